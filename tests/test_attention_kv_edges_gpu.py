"""Attention over the paged NVFP4 cache at the edges of its inputs, on both kernels:
infinite queries, queries and scales far from 1, counts at the ends of their types,
weights whose larger partners meet zero values, the automatic choice of the kernel,
and a data error beside a timeout.

Tolerance as in test_attention_kv_gpu.py, with the weights' term by the kernel that
runs: fp16 weights on the streaming kernel (half a step is 2^-11), bf16 on the tcgen05
kernel (2^-8)."""
import numpy as np
import pytest

import oracle  # noqa: F401
import synthetic as syn

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import skinny_gemv_gb300 as sg  # noqa: E402
from test_attention_kv_gpu import D, PATHS, Case, clean, dev, f64, i32  # noqa: E402

ONES = 6 * 11 / 64  # what a block of ones reads back as: scale 11 / 64, code 6


def fill(c, k=None, v=None):
    """Writes K and V (float, [tokens, kv_heads, D], tokens of all requests one after
    another; None: ones) over the rows of a Case's cache."""
    rows = np.concatenate([np.arange(n) for n in c.lens]).astype(int)
    owner = np.repeat(np.arange(len(c.lens)), c.lens)
    slots = c.table[owner, rows // c.page] * c.page + rows % c.page
    one = np.ones((len(rows), c.kv_heads, D))
    k, v = (dev(syn.f64_to_bf16_bits(one if x is None else x)) for x in (k, v))
    sg.kv_append_nvfp4(k, v, c.view(), i32(slots), c.page, c.k_scale, c.v_scale)
    c.host = c.cache.cpu().numpy()


def check(c, path, causal=True, scale=None, auto=None):
    """Against the oracle, with the weights' bound of the kernel `path` (`auto`: run
    SG_PATH_AUTO, which takes that kernel)."""
    got = f64(c.run(causal, scale, path=sg.PATH_AUTO if auto else path))
    clean()
    ref, W = c.ref(causal, scale)
    weights = 2.0 ** (-11 if path == sg.PATH_STREAM else -8)
    assert np.isfinite(got).all()
    bound = 2.0 ** -8 * np.abs(ref) + weights * (W + np.abs(ref)) + 2.0 ** -12 * W
    d = np.abs(got - ref)
    assert (d <= bound).all(), (d - bound).max()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("value", [float("inf"), float("-inf")])
@pytest.mark.parametrize("scale", [None, -0.1, 0.0])
def test_infinite_queries_give_nan(path, value, scale):
    """Keys of one sign: every score of the row is an infinity of one sign, and a softmax
    of those is NaN, not a row that sees nothing.  Rows that see no key stay 0."""
    for q_lens, lens in (([1], [1]), ([1, 3], [200, 40]), ([50, 9], [600, 4]), ([200], [500])):
        c = Case(q_lens, lens, 8, 2, 16)
        fill(c, v=np.random.default_rng(1).standard_normal((sum(lens), 2, D)))
        ref = c.run(scale=scale, path=path).clone()
        q = dev(c.Q).clone()
        rows = [0, q_lens[0] - 1, int(c.cu[-1]) - 1]
        for t in rows:
            q[t, 6, 9] = value
        got = c.run(scale=scale, Q=q, path=path)
        clean()
        keep = torch.ones(got.shape[:2], dtype=torch.bool)
        keep[rows, 6] = False
        assert torch.equal(got[keep], ref[keep])
        for t in rows:
            assert torch.isnan(got[t, 6]).all(), t
        if lens[-1] < q_lens[-1]:  # the first of the last request's queries is blind
            t = int(c.cu[-2])
            q[t, 6, 9] = value
            assert (c.run(scale=scale, Q=q, path=path)[t] == 0).all()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("power", [115, 60, -100])
def test_powers_of_two_move_between_queries_and_scale(path, power):
    """Queries times 2^power with the scale times 2^-power: the same scores, the same bits."""
    for q_lens, lens in (([1, 3], [300, 70]), ([90], [200])):
        c = Case(q_lens, lens, 8, 2, 16)
        # magnitudes of at least 1, so that no element becomes subnormal
        c.Q = syn.f64_to_bf16_bits(np.sign(f64(dev(c.Q))) * np.maximum(np.abs(f64(dev(c.Q))), 1.0))
        want = c.run(scale=2.0 ** -4, path=path).clone()
        c.Q = syn.f64_to_bf16_bits(f64(dev(c.Q)) * 2.0 ** power)
        assert torch.equal(c.run(scale=2.0 ** (-4 - power), path=path), want)
        clean()


@pytest.mark.parametrize("path", PATHS)
def test_vanishing_scores_leave_masked_keys_masked(path):
    """Queries and scale so small that their product underflows: all visible keys weigh
    the same, and a masked one nothing (not 0 * infinity)."""
    for q_lens, lens in (([1], [37]), ([5], [5]), ([100], [150])):
        c = Case(q_lens, lens, 4, 2, 16)
        c.Q = syn.f64_to_bf16_bits(f64(dev(c.Q)) * 2.0 ** -115)
        check(c, path, scale=1e-30)


def test_the_longest_sequence_ends_where_it_says():
    """2^31 - 1 keys, the last page entry's last token past the end: its values are NaN
    and must stay unseen.  (One page serves as all the others: 19 MB of cache.)"""
    page = 65536
    cache = torch.empty(2, sg.kv_nvfp4_page_bytes(1, page), dtype=torch.uint8, device="cuda")
    ones = torch.ones(2 * page, 1, D, dtype=torch.bfloat16, device="cuda")
    v = ones.clone()
    v[-1] = float("nan")
    sg.kv_append_nvfp4(ones, v, cache, torch.arange(2 * page, dtype=torch.int32, device="cuda"), page)
    table = torch.zeros(1, 32768, dtype=torch.int32, device="cuda")
    table[0, -1] = 1
    for heads in (1, 16):  # 8 and 16 query rows per unit of the streaming kernel
        q = torch.zeros(1, heads, D, dtype=torch.bfloat16, device="cuda")
        out = sg.attention_kv_nvfp4(q, cache, table, i32([2 ** 31 - 1]), i32([0, 1]), 1, page, 1, path=sg.PATH_STREAM)
        clean()
        assert (out == ONES).all()


@pytest.mark.parametrize("path", PATHS)
def test_a_long_chunk_beside_thousands_of_decode_requests(path):
    """batch * max_q * heads past 2^31; sampled rows against the oracle, a row of the
    chunk as a single query over the keys it sees."""
    rng = np.random.default_rng(3)
    n, chunk, heads = 4097, 4097, 128
    at = 1000
    q_lens = [1] * n
    q_lens[at] = chunk
    lens = [int(x) for x in rng.integers(1, 30, n)]
    lens[at] = chunk
    assert n * chunk * heads >= 2 ** 31
    c = Case(q_lens, lens, heads, 8, 16)
    got = f64(c.run(path=path))
    clean()
    assert np.isfinite(got).all()
    reqs = np.concatenate([rng.choice(n, 40, replace=False), np.full(4, at)])
    tokens = np.where(reqs == at, rng.integers(0, chunk, len(reqs)), 0)
    rows = c.cu[reqs] + tokens
    sees = np.where(reqs == at, tokens + 1, np.array(lens)[reqs])
    ref, W = oracle.attention_kv(c.Q[rows], c.host, c.table[reqs], sees, np.arange(len(rows) + 1), 8, 16, True, None,
                                 c.k_scale, c.v_scale)
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** (-11 if path == sg.PATH_STREAM else -8) * (W + np.abs(ref)) + 2.0 ** -12 * W
    assert (np.abs(got[rows] - ref) <= bound).all()


@pytest.mark.parametrize("path", PATHS)
def test_a_timeout_is_reported_beside_a_data_error(path):
    """A bad page id (its keys masked, the output defined) and a copy that never arrives
    (the output undefined): the caller has to learn of the second, in either order."""
    lib = sg.load()
    c = Case([40, 1], [3000, 20], 8, 2, 16)
    whole = c.run(path=path).clone()
    clean()
    keep = int(c.table[1, 0])
    for first in ("data", "both"):
        try:
            c.table[1, 0] = -5
            if first == "data":  # an earlier launch leaves the data error, a later one times out
                c.run(path=path)
                torch.cuda.synchronize()
                c.table[1, 0] = keep
            sg.set_wait_timeout_ns(20_000_000)
            lib.sg_debug_inject_missing_tx(4096)
            c.run(path=path)
            st, detail = sg.check_device_errors()
            assert st == sg.SG_ERR_TIMEOUT and detail[0] in (1, 2, 3, 4), (st, detail)
        finally:
            lib.sg_debug_inject_missing_tx(0)
            sg.set_wait_timeout_ns(2_000_000_000)
            c.table[1, 0] = keep
        st, detail = sg.check_device_errors()  # the other record is still there, once
        assert st == sg.SG_ERR_BAD_INDEX and detail[0] == 17 and detail[3] == 1
        clean()
        assert torch.equal(c.run(path=path), whole)
        clean()
    c.table[1, 0] = -5  # alone it is still what it was
    c.run(path=path)
    st, detail = sg.check_device_errors()
    assert st == sg.SG_ERR_BAD_INDEX and detail[0] == 17 and detail[3] == 1
    clean()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("causal", [True, False])
def test_a_constant_value_comes_back(path, causal):
    """The sums are of the weights as they enter the product, so whatever their rounding
    the average of one value is that value: fp32 leaves 2^-20 of it, far inside half a
    step of bf16."""
    for q_lens, lens in (([1, 1], [700, 90]), ([5], [300]), ([60, 3], [900, 64]), ([200], [1500])):
        c = Case(q_lens, lens, 8, 2, 16, spread=1.5)
        k = np.random.default_rng(2).standard_normal((sum(lens), 2, D))
        fill(c, k=k, v=c.v_scale * np.ones_like(k))
        got = c.run(causal, path=path)
        clean()
        assert (got == ONES * c.v_scale).all(), (got.float() / (ONES * c.v_scale) - 1).abs().max()


@pytest.mark.parametrize("path", PATHS)
def test_a_constant_value_under_weights_that_round_alike(path):
    """256 keys of weight 1, which set the reference, then keys of a weight just past the
    middle of two bf16 numbers: rounded up, they are 2^-8 too heavy, which shows (half a
    step at 1.875 is 2^-9) unless the sum takes them the same way."""
    n = 152  # requests, each about one CTA's share
    c = Case([1] * n, [1500] * n, 1, 1, 16, v_scale=1.0)
    k = np.zeros((1500, 1, D))
    k[:, 0, 0], k[:, 0, 1] = np.where(np.arange(1500) < 256, 4.0, 6.0), 6.0  # held exactly: scale 1
    fill(c, k=np.tile(k, (n, 1, 1)), v=np.full((n * 1500, 1, D), 1.875))  # scale 5 / 16, code 6
    q = np.zeros((n, 1, D))
    q[:, 0, 0] = 16.0
    c.Q = syn.f64_to_bf16_bits(q)
    got = c.run(scale=np.log(1 + 2.0 ** -8 + 2.0 ** -11) / 32, path=path)
    clean()
    assert (got == 1.875).all(), got.float().unique()


@pytest.mark.parametrize("q_lens,lens,heads,kv_heads,page", [
    ([300], [1500], 8, 2, 16), ([150, 1, 40], [900, 2000, 41], 16, 2, 64), ([513, 0, 2], [513, 7, 1300], 12, 4, 128),
    ([33] * 20, [33 + 60 * i for i in range(20)], 4, 1, 32), ([1000], [3000], 2, 1, 48)])
def test_larger_prefill_calls_take_the_tensor_core_kernel(q_lens, lens, heads, kv_heads, page):
    c = Case(q_lens, lens, heads, kv_heads, page, seed=4)
    auto, forced = c.run().clone(), c.run(path=sg.PATH_TENSOR_CORE).clone()
    stream = c.run(path=sg.PATH_STREAM)
    clean()
    assert torch.equal(auto, forced) and not torch.equal(auto, stream)
    check(c, sg.PATH_TENSOR_CORE, auto=True)
    check(c, sg.PATH_STREAM)


@pytest.mark.parametrize("q_lens,lens,heads,kv_heads,page", [
    ([40], [700], 300, 1, 16),        # too many heads per kv head for the other kernel, 8250 steps
    ([8, 1], [5000, 3000], 16, 4, 64),   # 32 rows per kv head
    ([64], [64], 4, 1, 16), ([100, 7], [130, 500], 4, 2, 16)])  # little work
def test_other_calls_stream(q_lens, lens, heads, kv_heads, page):
    c = Case(q_lens, lens, heads, kv_heads, page, seed=4)
    auto, forced = c.run().clone(), c.run(path=sg.PATH_STREAM)
    clean()
    assert torch.equal(auto, forced)
    check(c, sg.PATH_STREAM, auto=True)


@pytest.mark.parametrize("q_lens,lens", [([1], [17]), ([2, 3], [700, 64]), ([4, 1, 4], [33, 2000, 129]), ([8], [300]),
                                         ([16, 5], [257, 1000]), ([70, 9], [400, 9])])
@pytest.mark.parametrize("heads,kv_heads,page", [(4, 4, 16), (8, 2, 32), (12, 1, 48), (32, 2, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_streaming_weights_keep_eleven_bits(q_lens, lens, heads, kv_heads, page, causal):
    """Both widths of the streaming kernel (8 and 16 query rows), within the bound of its
    fp16 weights."""
    check(Case(q_lens, lens, heads, kv_heads, page, seed=8), sg.PATH_STREAM, causal)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("below", [20, 30, 60, 90])
@pytest.mark.parametrize("order", ["heavy first", "light first", "mixed"])
def test_small_weights_count_where_the_larger_meet_zero(path, below, order):
    """Keys of two kinds, whose weights differ by 2^below; V is zero under the heavy ones,
    so the whole result comes from the light ones (and so does W, which the bound is
    relative to)."""
    rng = np.random.default_rng(below)
    for q_lens, lens in (([1], [50]), ([1, 2], [700, 90]), ([6], [400]), ([150], [1000])):
        c = Case(q_lens, lens, 8, 2, 16, v_scale=1.0)
        heavy = np.concatenate([np.arange(n) < (n + 1) // 2 if order == "heavy first" else
                                np.arange(n) >= n // 2 if order == "light first" else rng.random(n) < 0.5 for n in lens])
        k, v = np.zeros((2, sum(lens), 2, D))
        k[:, :, 0] = np.where(heavy, 6.0, -6.0)[:, None]  # held exactly: scale 1, code 6
        v[:] = np.where(heavy[:, None, None], 0.0, rng.standard_normal(v.shape))
        fill(c, k, v)
        q = np.zeros((int(c.cu[-1]), 8, D))
        q[:, :, 0] = 16.0
        c.Q = syn.f64_to_bf16_bits(q)
        check(c, path, scale=below * np.log(2.0) / (16 * 12))
        if order == "heavy first":
            ref, _ = c.ref(scale=below * np.log(2.0) / (16 * 12))
            assert 0 < np.abs(ref[-1]).max() < 2.0 ** (4 - below)
