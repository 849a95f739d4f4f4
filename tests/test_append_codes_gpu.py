"""E4M3 codes of fp32 and bf16 rows under scales over the whole range of fp32: the code is that of the
fp32 quotient x / scale, also where x, or the rest of a division by it, is no normal number."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _rows(scale, dtype, seed):
    """Values beside the borders between two codes, times the scale; some of any size."""
    g = np.random.default_rng(seed)
    n = 256 * 64
    t = np.ldexp(1 + g.integers(0, 16, n) / 16.0, g.integers(-11, 9, n)) * g.choice([-1.0, 1.0], n)
    x = t * np.float64(np.float32(scale)) * (1 + g.integers(-2, 3, n) * 2.0 ** -24)
    x[::97] = 2.0 ** g.uniform(-149, 127, len(x[::97]))
    x = np.clip(x, -3.0e38, 3.0e38).astype(np.float32)
    return torch.from_numpy(x).view(256, 1, 64).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [3.8209197e-38, 4.3938958e-37, 7.5232194e-37, 3.082564e-33, 3.155444e-30, 2.0 ** -91, 1.3 * 2.0 ** -90,
                                   2.0 ** -89, 1.7e-20, 0.0093, 1.0, 3.3e5, 1.9e30, 1.7 * 2.0 ** 125, 1.5 * 2.0 ** 126, 3.0e38])
def test_codes_are_those_of_the_quotient(scale, dtype):
    import split_kv_decode_flashdecoding_b200 as fd
    k, v = _rows(scale, dtype, 1), _rows(scale, dtype, 2)
    pools = [torch.zeros((8, 1, 32, 64), dtype=torch.uint8, device="cuda") for _ in range(2)]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    fd.fd_pages_append_fp8(k.cuda(), v.cuda(), *pools, scale, scale, i32([list(range(8))]), i32([0]), i32([256]))
    assert fd.fd_poll_status() == 0
    for pool, x in zip(pools, (k, v)):
        q = (x.float() / torch.tensor(scale, dtype=torch.float32)).clamp(-448, 448)
        want = q.to(torch.float8_e4m3fn).view(torch.uint8)
        got = pool.cpu().view(256, 1, 64)
        wrong = (got != want).nonzero()
        assert len(wrong) == 0, f"{len(wrong)} codes, first {x[tuple(wrong[0])].item():g} / {scale:g}"
