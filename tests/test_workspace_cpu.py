"""Sizes of the workspace of the decode and chunk calls."""

import split_kv_decode_flashdecoding_b200 as fd

MB = 1 << 20


def test_header_and_sections():
    # the header (256 bytes), 1 item (32), no tile items, 1 row in three tables, one slot of 64 fp32 and
    # its log-sum-exp, each section in whole units of 256 bytes
    assert fd.fd_decode_workspace_bytes(1, 1, 1, 4096, 64, 1, 148) == 256 * (1 + 1 + 3 + 1 + 1)


def test_the_70b_shape():
    # 32 * 8 + max(8 * 148, 32 * 8 * 32768 / 1024) items and slots of 8 heads
    items = 32 * 8 + 8192
    assert fd.fd_decode_workspace_bytes(32, 64, 8, 32768, 128, 0, 148) == 256 + items * 32 + 2 * 256 + 1024 + items * 8 * 129 * 4


def test_a_shape_that_fits_the_static_scratch_by_a_little():
    assert fd.fd_decode_workspace_bytes(4, 1, 1, 4096, 64, 57455, 148) == 64 * MB - 256
