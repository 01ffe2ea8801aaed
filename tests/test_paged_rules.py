"""CPU checks of which of the two attention kernels a paged call takes, by the most rows that each has room for."""

import pytest

from test_paged_abi import UNSUPPORTED, args, attend, spec  # noqa: F401


@pytest.mark.parametrize("page,tensor_cores", [
    (8, True), (16, True), (32, True), (64, True), (128, True), (192, True), (320, True), (4160, True),
    (1, False), (4, False), (24, False), (48, False), (96, False), (160, False)])
def test_page_sizes_of_the_tensor_cores(spec, page, tensor_cores):  # noqa: F811
    """Whole pages in a block of 64 positions, or whole blocks in a page. 49,148 rows of 4 heads a KV head and two
    requests are 1,537 tiles of 128 rows and 12,289 of 16, one more than there may be."""
    c, _, d = args(spec)
    c.page_size, c.page_stride, c.layer_stride = page, page * 512, page * 5120
    got = attend(spec, c, d, rows=(12288 - 1) * 4, n=0)
    assert (got not in (0, UNSUPPORTED)) if tensor_cores else got == UNSUPPORTED
