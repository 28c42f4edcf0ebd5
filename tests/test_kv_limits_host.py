"""Limits of the paged-cache entry points, on the host.  A call that has to pass the
checks of its sizes is given a misaligned pointer, which is refused after them, so that
nothing is launched wherever this runs."""
import pytest

import skinny_gemv_gb300 as sg
from test_kv_abi_host import A, ATTN, BAD, MIS, call, lib  # noqa: F401

TOP = 2 ** 31 - 1 - 1024  # largest batch, and query tokens of a request x heads


@pytest.mark.parametrize("sizes,code", [
    (dict(batch=1024, max_q=32768, tokens=33791, heads=64), MIS),     # a chunk beside 1023 decode requests
    (dict(batch=16384, max_q=131072, tokens=131072, heads=128), MIS),
    (dict(batch=TOP, max_q=1, tokens=1, heads=1), MIS), (dict(batch=TOP + 1, max_q=1, tokens=1, heads=1), BAD),
    (dict(batch=1, max_q=TOP // 64, tokens=2 ** 31 - 1, heads=64), MIS),
    (dict(batch=1, max_q=TOP // 64 + 1, tokens=2 ** 31 - 1, heads=64), BAD),
    (dict(batch=1, max_q=2 ** 40, tokens=TOP // 64, heads=64), MIS),  # the tokens bound max_q
    (dict(batch=2, max_q=4, tokens=4, heads=2 ** 31 // 128 - 1), MIS),
])
@pytest.mark.parametrize("name", ["attention_kv_nvfp4", "attention_kv_nvfp4_path"])
def test_attention_sizes(lib, name, sizes, code):  # noqa: F811
    heads = sizes["heads"]
    base = dict(ATTN, **sizes, kv_heads=1, ldq=heads * 128, ldo=heads * 128, pitch=16 * 144, Q=A + 2)
    if name == "attention_kv_nvfp4":
        assert call(lib, name, base) == code
    else:
        assert lib.attention_kv_nvfp4_path(*base.values(), sg.PATH_STREAM, None) == code
