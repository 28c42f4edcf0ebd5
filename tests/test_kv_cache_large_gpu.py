"""The paged cache's other calls at sizes that take their large forms: the rotation with
two rows per lane, page assignment for more requests than the default shared memory
holds.  Bounds as in test_kv_cache_gpu.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_kv_cache_gpu import check_pages, check_rope, pages_case  # noqa: E402


@pytest.mark.parametrize("T,H,Hkv,D,rot", [
    (2047, 12, 5, 128, 128),   # 8699 warps of rows, an odd number of heads per token
    (4099, 13, 4, 96, 64),     # eight lanes a row of which six hold data
    (1031, 10, 7, 256, 192),   # sixteen lanes a row, the second of them in another warp's part
    (601, 9, 6, 512, 512),     # a warp per row
    (5003, 31, 2, 64, 48),     # four lanes a row
])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("neighbours", [False, True])
def test_norm_rope_of_large_steps(T, H, Hkv, D, rot, norm, neighbours):
    lanes = 4 if D <= 64 else 8 if D <= 128 else 16 if D <= 256 else 32
    assert T * (H + Hkv) * lanes // 32 >= 8192  # two rows per lane from here on
    check_rope(T, H, Hkv, D, rot, norm, neighbours)
    check_rope(T, H, Hkv, D, rot, norm, neighbours, in_place=True, padded=False)


@pytest.mark.parametrize("n,page,max_len,max_new", [(16384, 16, 60, 5), (16384, 64, 500, 90), (6145, 32, 40, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_pages_of_as_many_requests_as_allowed(n, page, max_len, max_new, in_place):
    rng = np.random.default_rng(n + page)
    lens, new, free, table, tokens = pages_case(n, page, rng, max_len, max_new, spare=3, short=17)
    check_pages(lens, new, free, table, page, tokens, in_place=in_place)
