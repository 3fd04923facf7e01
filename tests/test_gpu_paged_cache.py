"""The paged cache's write and read on the GPU against their definitions in 64 bits: exact codes, scale
bytes and rows; pages that end inside a call; rows that belong to no sequence; bad tables."""
import math

import pytest
import torch

from paged_common import D, HKV, Pool, prefix, quantise64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def raw(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.uint8)


def rows_of(n, seed, spread=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((n, HKV, D), generator=g, device="cuda")
    if spread:
        x = x * torch.exp2(20 * torch.rand((n, HKV, 1), generator=g, device="cuda") - 10)
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,lens_q,lens_k", [
    (16, [1], [1]), (1, [3], [5]), (12, [13, 0, 1, 25], [13, 7, 40, 31]), (64, [1] * 33, list(range(1, 34))),
    (5, [0, 0, 701, 0, 2], [0, 9, 701, 0, 1000]), (256, [4096], [5001])])
def test_write(qsa, fp8, page, lens_q, lens_k):
    pool = Pool(lens_k, page, fp8, seed=page)
    n, pad = sum(lens_q), 3
    k, v = rows_of(n + pad, 1), rows_of(n + pad, 2)
    want_k, want_v = pool.k.clone(), pool.v.clone()
    want_ks, want_vs = (pool.ks.clone(), pool.vs.clone()) if fp8 else (None, None)
    at = 0
    for s, (m, L) in enumerate(zip(lens_q, lens_k)):
        r = pool.rows(s, L - m, L)
        for x, w, ws in ((k, want_k, want_ks), (v, want_v, want_vs)):
            if fp8:
                code, e = quantise64(x[at:at + m])
                c8 = code.float().to(torch.float8_e4m3fn)
                assert torch.equal(c8.double(), code)                 # every code is a value of the type
                w.view(torch.uint8).view(-1, HKV, D)[r] = c8.view(torch.uint8)
                ws.view(-1, HKV)[r] = e
            else:
                w.view(-1, HKV, D)[r] = x[at:at + m]
        at += m
    qsa.cache_write_paged(k, v, pool.k, pool.v, pool.table, prefix(lens_q), prefix(lens_k), **pool.args())
    assert qsa.device_status(clear=True) == 0
    assert torch.equal(raw(pool.k), raw(want_k)) and torch.equal(raw(pool.v), raw(want_v))
    if fp8:
        assert torch.equal(pool.ks, want_ks) and torch.equal(pool.vs, want_vs)


def test_quantisation_at_its_edges(qsa):
    """Rows around the scale's steps, the smallest and the largest values, zeros and signed zeros."""
    tops = [448.0, 449.0, 450.0, 447.0, 224.0, 1.75, 1.7578125, 2.0, 3.3895313892515355e38, 1.1754943508222875e-38,
            9.183549615799121e-41, 2.0 ** -130, 2.0 ** -118, 2.0 ** -119, 1.75 * 2.0 ** -119, 0.0, -0.0, -448.0]
    x = rows_of(len(tops), 5, spread=False)
    for i, t in enumerate(tops):
        lead = torch.tensor(t, dtype=torch.float64).to(torch.bfloat16)
        x[i] = (torch.tanh(x[i].double()) * float(lead) * 0.99).to(torch.bfloat16)
        x[i, :, 17] = lead.cuda()
    pool = Pool([len(tops)], 8, True)
    cu = prefix([len(tops)])
    qsa.cache_write_paged(x, x, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    code, e = quantise64(x)
    r = pool.rows(0, 0, len(tops))
    assert torch.equal(pool.ks.view(-1, HKV)[r], e) and torch.equal(pool.vs.view(-1, HKV)[r], e)
    got = pool.k.view(torch.uint8).view(-1, HKV, D)[r].view(torch.float8_e4m3fn)
    assert torch.equal(got.double(), code)
    k, v = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, len(tops), **pool.args())
    # exact down to bf16's subnormals: code 2^e rounded once
    want = (code * torch.exp2(e.double() - 127)[..., None])
    assert torch.equal(k.double(), want.to(torch.bfloat16).double()) and torch.equal(raw(k), raw(v))


def test_rows_that_are_not_finite_read_back_as_nan(qsa):
    x = rows_of(4, 9, spread=False)
    x[0, 0, 3], x[1, 1, 255], x[2, 0, 0], x[2, 0, 9] = math.nan, math.inf, -math.inf, math.nan
    pool, cu = Pool([4], 3, True), prefix([4])
    qsa.cache_write_paged(x, x, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    r = pool.rows(0, 0, 4)
    bad = torch.tensor([[True, False], [False, True], [True, False], [False, False]], device="cuda")
    assert torch.equal(pool.ks.view(-1, HKV)[r] == 255, bad)
    assert (pool.k.view(torch.uint8).view(-1, HKV, D)[r][bad] == 0).all()
    k, _ = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, 4, **pool.args())
    assert torch.equal(torch.isnan(k).all(-1), bad) and not torch.isnan(k[~bad]).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,lens,begin", [
    (16, [1], None), (1, [5, 3], [0, 2]), (12, [13, 0, 40, 31], [13, 0, 7, 30]), (64, [701, 5000], None),
    (7, [100] * 20, list(range(0, 100, 5)))])
def test_read(qsa, fp8, page, lens, begin):
    pool = Pool(lens, page, fp8, seed=page).fill()
    b = begin or [0] * len(lens)
    count = [L - x for L, x in zip(lens, b)]
    n, pad = sum(count), 2
    out_k = torch.full((n + pad, HKV, D), -3.0, dtype=torch.bfloat16, device="cuda")
    out_v = out_k.clone()
    qsa.cache_read_paged(pool.k, pool.v, pool.table, prefix(lens), prefix(count), n + pad,
                         tok_begin=torch.tensor(b, dtype=torch.int32, device="cuda") if begin else None, k=out_k,
                         v=out_v, **pool.args())
    assert qsa.device_status(clear=True) == 0
    for x, got in (("k", out_k), ("v", out_v)):
        want = torch.cat([pool.values(x, s, b[s], L) for s, L in enumerate(lens) if L > b[s]])
        assert torch.equal(got[:n].double(), want)
        assert (got[n:] == -3.0).all()                                # rows behind the last sequence


@pytest.mark.parametrize("fp8", [False, True])
def test_write_read_write_gives_the_same_pool(qsa, fp8):
    lens = [37, 5, 128]
    pool, cu = Pool(lens, 12, fp8), prefix(lens)
    k, v = rows_of(170, 3), rows_of(170, 4)
    qsa.cache_write_paged(k, v, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    k2, v2 = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, 170, **pool.args())
    # within half a step of an e4m3 code, or of its subnormal step 2^(e - 9)
    for a, b in ((k, k2), (v, v2)):
        if fp8:
            _, e = quantise64(a)
            bound = torch.maximum(a.double().abs() * 2.0 ** -4, torch.exp2(e.double() - 127 - 10)[..., None])
            assert ((a.double() - b.double()).abs() <= bound).all()
        else:
            assert torch.equal(raw(a), raw(b))
    first = [raw(t).clone() for t in (pool.k, pool.v)]
    qsa.cache_write_paged(k2, v2, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    k3, v3 = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, 170, **pool.args())
    assert torch.equal(raw(k2), raw(k3)) and torch.equal(raw(v2), raw(v3))
    if not fp8:
        assert torch.equal(raw(pool.k), first[0]) and torch.equal(raw(pool.v), first[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_tokens_without_a_page(qsa, fp8):
    lens = [40, 20]
    pool, cu = Pool(lens, 8, fp8), prefix(lens)
    bad = pool.table.clone()
    bad[0, 1], bad[0, 2] = -1, pool.k.shape[0]                        # tokens 8 .. 23 of sequence 0
    short = bad[:, :4].contiguous()                                   # and 32 .. 39: past the table
    k, v = rows_of(60, 3, spread=False), rows_of(60, 4, spread=False)
    before = raw(pool.k).clone()
    qsa.cache_write_paged(k, v, pool.k, pool.v, short, cu, cu, **pool.args())
    assert qsa.device_status(clear=True) == qsa.QSA_ERR_DEVICE_CHECK
    gone = torch.cat([pool.rows(0, 8, 24), pool.rows(0, 32, 40)])
    assert torch.equal(raw(pool.k).view(-1, HKV, raw(pool.k).shape[-1])[gone],
                       before.view(-1, HKV, before.shape[-1])[gone])
    rk, rv = qsa.cache_read_paged(pool.k, pool.v, short, cu, cu, 60, **pool.args())
    assert qsa.device_status(clear=True) == qsa.QSA_ERR_DEVICE_CHECK
    zero = torch.zeros(60, dtype=torch.bool, device="cuda")
    zero[8:24] = zero[32:40] = True
    for x in (rk, rv):
        assert (x[zero] == 0).all() and (x[~zero] != 0).any(-1).all()
    # ranges outside the cached tokens
    qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, prefix([1, 1]), 2,
                         tok_begin=torch.tensor([-1, 20], dtype=torch.int32, device="cuda"), k=rk[:2], v=rv[:2],
                         **pool.args())
    assert qsa.device_status(clear=True) == qsa.QSA_ERR_DEVICE_CHECK
    assert (rk[:2] == 0).all() and (rv[:2] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(qsa, fp8):
    """The last rows of a pool of more than 2^32 bytes per array (a few written and read back)."""
    page = 1024
    pages = 2 ** 32 // (page * HKV * D * (1 if fp8 else 2)) + 2
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    kp, vp = (torch.empty((pages, page, HKV, D), dtype=dt, device="cuda") for _ in range(2))
    sc = [torch.empty((pages, page, HKV), dtype=torch.uint8, device="cuda") for _ in range(2)] if fp8 else [None] * 2
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    k, v = rows_of(1030, 1, spread=False), rows_of(1030, 2, spread=False)
    cu = prefix([1030])
    qsa.cache_write_paged(k, v, kp, vp, table, cu, cu, k_scales=sc[0], v_scales=sc[1])
    rk, rv = qsa.cache_read_paged(kp, vp, table, cu, cu, 1030, k_scales=sc[0], v_scales=sc[1])
    assert qsa.device_status(clear=True) == 0
    for a, b in ((k, rk), (v, rv)):
        if fp8:
            code, e = quantise64(a)
            assert torch.equal(b.double(), code * torch.exp2(e.double() - 127)[..., None])
        else:
            assert torch.equal(raw(a), raw(b))
    if not fp8:
        assert torch.equal(raw(kp[pages - 1]), raw(k[:1024])) and torch.equal(raw(kp[0, :6]), raw(k[1024:]))


def test_captured_write_and_read_replay_on_other_lengths(qsa):
    pool = Pool([50, 60], 16, True)
    k, v = rows_of(8, 1, spread=False), rows_of(8, 2, spread=False)
    cu_q, cu_k = prefix([4, 4]), prefix([4, 4])
    out_k, out_v = torch.zeros((8, HKV, D), dtype=torch.bfloat16, device="cuda"), torch.zeros(
        (8, HKV, D), dtype=torch.bfloat16, device="cuda")
    begin = torch.zeros(2, dtype=torch.int32, device="cuda")

    def step():
        qsa.cache_write_paged(k, v, pool.k, pool.v, pool.table, cu_q, cu_k, **pool.args())
        qsa.cache_read_paged(pool.k, pool.v, pool.table, cu_k, cu_q, 8, tok_begin=begin, k=out_k, v=out_v, **pool.args())

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for n, L in (([4, 4], [50, 60]), ([1, 5], [7, 33]), ([0, 3], [1, 3])):
        cu_q.copy_(prefix(n))
        cu_k.copy_(prefix(L))
        begin.copy_(torch.tensor([a - b for a, b in zip(L, n)], dtype=torch.int32))
        k.copy_(rows_of(8, sum(L), spread=False))
        out_k.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        code, e = quantise64(k)
        want = code * torch.exp2(e.double() - 127)[..., None]
        assert torch.equal(out_k[:sum(n)].double(), want[:sum(n)]) and (out_k[sum(n):] == 5.0).all()
    assert qsa.device_status(clear=True) == 0
