"""Refusals of results and pools whose rows, heads or pages share memory."""

import ctypes

import split_kv_decode_flashdecoding_b200 as fd
from test_serving_cpu import _fake, _i, _prompt, _ref

UNS = fd.FD_ERR_UNSUPPORTED


def _message():
    return fd.lib.fd_last_error_message().decode()


def test_broadcast_results():
    for strides in ([0, 128, 1], [1024, 0, 1]):
        assert _prompt(out=_fake((9, 8, 128), strides=strides)) == UNS and "out's rows and heads" in _message()
    out, cache = _fake((9, 8, 128), strides=[1024, 0, 1]), _fake((3, 2, 50, 128))
    lse = ctypes.cast(ctypes.c_void_p(0x300000), ctypes.POINTER(ctypes.c_float))
    assert fd.lib.fd_tree_attention(_ref(_fake((9, 8, 128))), _ref(cache), _ref(cache), _i(), _i(), _i(), 1, _ref(out), lse, None) == UNS
    assert "out's rows and heads" in _message()


def test_broadcast_pools():
    new = _fake((9, 2, 128))
    for strides in ([0, 2048, 128, 1], [4096, 0, 128, 1]):
        pages = _fake((7, 2, 16, 128), strides=strides)
        for st in (fd.lib.fd_pages_append(_ref(new), _ref(new), _ref(pages), _ref(pages), _i(), 4, 3, _i(), _i(), None),
                   fd.lib.fd_pages_fork(_ref(pages), _ref(pages), _i(), _i(), 4, 3, _i(), _i(), _i(), 2, None),
                   fd.lib.fd_pages_compact(_ref(pages), _ref(pages), _i(), _i(), 4, 3, _i(), _i(), _i(), 5, _i(), None)):
            assert st == UNS and "must not share memory" in _message()
    one = _fake((1, 1, 16, 128), strides=[0, 0, 128, 1])  # one page of one head shares with none
    assert fd.lib.fd_pages_append(_ref(_fake((9, 1, 128))), _ref(_fake((9, 1, 128))), _ref(one), _ref(one), _i(), 4, 0, _i(), _i(), None) == fd.FD_OK
