"""Attention of new tokens over a paged cache on the GPU against its definition in 64 bits, at the
lengths, pages, windows and stale memory where it can go wrong, and in the serving path it belongs to."""
import math

import pytest
import torch

from paged_common import D, HKV, HQ, Pool, U16, check_attend, prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def queries(n, seed=7, size=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((n, HQ, D), generator=g, device="cuda") * size).to(torch.bfloat16)


def attend(qsa, q, pool, lens_q, window=0, sinks=0, max_q=None, **kw):
    return qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(lens_q), prefix(pool.lens),
                                max(lens_q) if max_q is None else max_q, max(pool.lens), window=window, sinks=sinks,
                                want_lse=True, **pool.args(), **kw)


LENGTHS = [
    # page, new tokens, cached tokens
    (16, [1], [1]), (64, [1], [8191]), (1, [1, 1], [5, 130]), (12, [1] * 9, [1, 2, 63, 64, 65, 127, 128, 129, 700]),
    (64, [1] * 40, [100 + 37 * i for i in range(40)]),
    (16, [4, 3, 2, 1], [4, 300, 129, 1000]), (8, [0, 4, 0, 5, 0], [10, 300, 0, 5, 0]),
    (32, [21, 22, 43], [21, 150, 43]), (16, [10, 9, 1], [300, 9, 1000]), (48, [8] * 5, [8, 64, 65, 4000, 129]), (7, [10, 11, 64, 65], [300, 11, 64, 201]),
    (128, [701], [701]), (16, [128, 1, 300], [900, 2000, 300]), (64, [0, 0], [0, 5]), (5, [257], [2049]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page,lens_q,lens_k", LENGTHS)
def test_lengths(qsa, page, lens_q, lens_k, fp8):
    pool = Pool(lens_k, page, fp8, seed=page).fill(seed=sum(lens_k))
    q = queries(max(sum(lens_q), 1))
    o, lse = attend(qsa, q, pool, lens_q)
    assert qsa.device_status(clear=True) == 0
    check_attend(q, pool, lens_q, o, lse)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 3), (64, 0), (100, 4), (129, 200), (1000, 16), (5000, 7),
                                          (63, 64), (128, 65), (2 ** 31 - 1, 5), (3, 2 ** 31 - 1)])
@pytest.mark.parametrize("page,lens_q,lens_k", [(16, [1, 1, 1], [1, 500, 1300]), (12, [4, 3], [800, 130]),
                                                (64, [150, 1], [701, 90]), (32, [64, 33], [64, 901])])
def test_windows(qsa, page, lens_q, lens_k, window, sinks, fp8):
    pool = Pool(lens_k, page, fp8, seed=window).fill(seed=sinks)
    q = queries(sum(lens_q))
    o, lse = attend(qsa, q, pool, lens_q, window, sinks)
    assert qsa.device_status(clear=True) == 0
    check_attend(q, pool, lens_q, o, lse, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens_q", [[1, 1], [4, 2], [60, 70]])
def test_memory_that_no_row_sees_may_hold_anything(qsa, lens_q, fp8):
    """NaNs behind the sequences' ends and before the window, and a table without those pages."""
    lens_k, page, window, sinks = [1000, 333], 16, 100, 3
    pool = Pool(lens_k, page, fp8, seed=4).fill()      # the pool's other memory holds NaN already
    q = queries(sum(lens_q))
    for s, (n, L) in enumerate(zip(lens_q, lens_k)):
        a, b = sinks, max(L - n - window + 1, 0)       # tokens [a, b): no row sees them
        if b <= a:
            continue
        r = pool.rows(s, a, b)
        for x, sc in ((pool.k, pool.ks), (pool.v, pool.vs)):
            if fp8:
                x.view(torch.uint8).view(-1, HKV, D)[r] = 0x7F
                sc.view(-1, HKV)[r] = 255
            else:
                x.view(-1, HKV, D)[r] = math.nan
        pool.table[s, -(-a // page):b // page] = -1    # whole pages
    o, lse = attend(qsa, q, pool, lens_q, window, sinks)
    assert qsa.device_status(clear=True) == 0
    pool.table.clamp_(min=0)
    check_attend(q, pool, lens_q, o, lse, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens_q", [[1, 1, 1], [3, 4, 1], [70, 200, 5]])
def test_rows_without_keys_and_rows_of_no_sequence(qsa, lens_q, fp8):
    """More new tokens than cached ones: the first rows sit at negative positions.  Rows behind the last
    sequence stay as they were."""
    lens_k = [0, max(lens_q[1] - 2, 0), 5]
    pool = Pool(lens_k, 8, fp8).fill()
    n = sum(lens_q)
    q = queries(n + 5)
    o = torch.full_like(q, 3.0)
    lse = torch.full((n + 5, HQ), 4.0, device="cuda")
    attend(qsa, q, pool, lens_q, o=o, lse=lse)
    assert qsa.device_status(clear=True) == 0
    assert (o[n:] == 3.0).all() and (lse[n:] == 4.0).all()
    check_attend(q, pool, lens_q, o, lse)
    hidden = lens_q[0] + max(lens_q[1] - lens_k[1], 0)
    assert (o[:lens_q[0]] == 0).all() and torch.isneginf(lse[:lens_q[0]]).all()
    assert int(torch.isneginf(lse[:n]).all(1).sum()) == hidden + max(lens_q[2] - 5, 0)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 4, 64])
def test_large_scores(qsa, n, fp8):
    """Scores in the hundreds, one key far above the rest near the end: the running maximum moves late."""
    pool = Pool([1500], 16, fp8, seed=2).fill(spread=1.0)
    q = queries(n, size=12.0)
    o, lse = attend(qsa, q, pool, [n])
    check_attend(q, pool, [n], o, lse)
    r = pool.rows(0, 1499 - n, 1500 - n)
    if not fp8:
        pool.k.view(-1, HKV, D)[r] *= 8
    else:
        pool.ks.view(-1, HKV)[r] += 3
    o, lse = attend(qsa, q, pool, [n])
    check_attend(q, pool, [n], o, lse)


@pytest.mark.parametrize("n", [1, 64])
def test_scales_over_their_whole_range(qsa, n):
    """Scale bytes far from the usual ones: keys of 2^-100 beside values of 2^90."""
    pool = Pool([300], 16, True, seed=2).fill()
    r = pool.rows(0, 0, 300)
    pool.ks.view(-1, HKV)[r[::3]] = 27
    pool.vs.view(-1, HKV)[r] = 217 - 8
    q = queries(n)
    o, lse = attend(qsa, q, pool, [n])
    check_attend(q, pool, [n], o, lse)


def test_a_value_that_is_not_finite_reaches_the_rows_that_see_it(qsa):
    for fp8 in (False, True):
        for n in (1, 4, 64):
            pool = Pool([500], 16, fp8, seed=2).fill()
            r = pool.rows(0, 100, 101)
            if fp8:
                pool.ks.view(-1, HKV)[r, 0] = 255
            else:
                pool.k.view(-1, HKV, D)[r, 0, 5] = math.nan
            q = queries(n)
            o, lse = attend(qsa, q, pool, [n])
            assert torch.isnan(o[:, :12]).all() and torch.isnan(lse[:, :12]).all()
            assert not torch.isnan(o[:, 12:]).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens_q", [[1, 1], [40, 200]])
def test_visible_positions_without_a_page(qsa, lens_q, fp8):
    """They count as zero keys and values, and are flagged."""
    lens_k = [400, 300]
    pool = Pool(lens_k, 16, fp8, seed=3).fill()
    q = queries(sum(lens_q))
    gone = pool.rows(0, 32, 64)
    bad = pool.table.clone()
    bad[0, 2], bad[0, 3] = -7, pool.k.shape[0]
    for x, sc in ((pool.k, pool.ks), (pool.v, pool.vs)):
        x.view(torch.uint8).view(-1, HKV, D * x.element_size())[gone] = 0
        if fp8:
            sc.view(-1, HKV)[gone] = 120
    good, pool.table = pool.table, bad
    o, lse = attend(qsa, q, pool, lens_q)
    assert qsa.device_status(clear=True) == qsa.QSA_ERR_DEVICE_CHECK
    pool.table = good
    check_attend(q, pool, lens_q, o, lse)


def test_more_tokens_than_rows_are_flagged(qsa):
    pool = Pool([50], 16, False).fill()
    q = queries(8)
    o = torch.full_like(q, 3.0)
    qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix([9]), prefix([50]), 9, 50, o=o)
    assert qsa.device_status(clear=True) == qsa.QSA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("fp8", [False, True])
def test_the_bound_of_new_tokens_only_chooses_the_kernel(qsa, fp8):
    lens_q, lens_k = [30, 1, 7], [200, 300, 7]
    pool = Pool(lens_k, 16, fp8, seed=3).fill()
    q = queries(sum(lens_q))
    for max_q in (0, 1, 4, 30, 100000):
        o, lse = attend(qsa, q, pool, lens_q, max_q=max_q)
        check_attend(q, pool, lens_q, o, lse)
    assert qsa.device_status(clear=True) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 4, 90])
def test_two_runs_agree_to_the_bit(qsa, n, fp8):
    pool = Pool([3001, 17 + n, 900], 16, fp8, seed=3).fill()
    q = queries(3 * n)
    a = attend(qsa, q, pool, [n] * 3)
    b = attend(qsa, q, pool, [n] * 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 4, 50])
def test_captured_call_replays_on_other_lengths(qsa, n, fp8):
    """A graph captured for one batch holds for other lengths of the same total, and as caches grow."""
    lens = [900, 400, 1300]
    pool = Pool(lens, 16, fp8, seed=3).fill()
    q, cu_q, cu_k = queries(3 * n), prefix([n] * 3), prefix([n] * 3)
    o, lse = torch.empty_like(q), torch.empty((3 * n, HQ), device="cuda")
    ws = torch.empty(qsa.workspace_size(qsa.OP_CHUNK_PAGED, 3, 3 * n), dtype=torch.uint8, device="cuda")

    def step():
        qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, cu_q, cu_k, n, 1300, o=o, lse=lse, ws=ws, **pool.args())

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for lens_q, lens_k in (([n] * 3, lens), ([n] * 3, [n, 399, 1]), ([n, 0, n], [901 - n, 0, 1300])):
        cu_q.copy_(prefix(lens_q))
        cu_k.copy_(prefix(lens_k))
        o.fill_(9.0)
        ws.fill_(255)                                  # nothing may be left over from the last step
        graph.replay()
        torch.cuda.synchronize()
        pool.lens = lens_k
        check_attend(q, pool, lens_q, o, lse)
        assert (o[sum(lens_q):] == 9.0).all()
    assert qsa.device_status(clear=True) == 0


def test_two_streams_at_once(qsa):
    pools = [Pool([2000 + 100 * i, 600], 16, bool(i), seed=i).fill() for i in range(2)]
    q = [queries(41, seed=i) for i in range(2)]
    alone = [attend(qsa, q[i], pools[i], [40, 1]) for i in range(2)]
    torch.cuda.synchronize()
    streams, out = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(5):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                out[i] = attend(qsa, q[i], pools[i], [40, 1])
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(out[i][0], alone[i][0]) and torch.equal(out[i][1], alone[i][1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n", [1, 300])
def test_long_cache(qsa, n, fp8):
    """131072 cached tokens; rows checked against 64 bits."""
    pool = Pool([131072, 5], 64, fp8, seed=3).fill()
    q = queries(n + 5)
    o, lse = attend(qsa, q, pool, [n, 5])
    if n == 1:
        check_attend(q, pool, [n, 5], o, lse)
    else:  # the last rows alone: a call of fewer new tokens has the same result for them
        keep = torch.cat([q[n - 3:n], q[n:]])
        check_attend(keep, pool, [3, 5], torch.cat([o[n - 3:n], o[n:]]), torch.cat([lse[n - 3:n], lse[n:]]))


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(qsa, fp8):
    """A cache whose pages lie in the last rows of a pool of more than 2^32 bytes per array."""
    page = 1024
    pages = 2 ** 32 // (page * HKV * D * (1 if fp8 else 2)) + 4
    pool = Pool([2500, 700], page, fp8, seed=1).fill()
    used = pool.k.shape[0]
    big = [torch.empty((pages, page, HKV, D), dtype=pool.k.dtype, device="cuda") for _ in range(2)]
    sc = [torch.empty((pages, page, HKV), dtype=torch.uint8, device="cuda") if fp8 else None for _ in range(2)]
    for b, x in zip(big, (pool.k, pool.v)):
        b[pages - used:].view(torch.uint8).copy_(x.view(torch.uint8))
    for b, x in zip(sc, (pool.ks, pool.vs)):
        if fp8:
            b[pages - used:].copy_(x)
    table = torch.where(pool.table >= 0, pool.table + (pages - used), -1).to(torch.int32)
    for lens_q in ([1, 1], [30, 100]):
        q = queries(sum(lens_q))
        o, lse = qsa.chunk_attn_paged(q, big[0], big[1], table, prefix(lens_q), prefix(pool.lens), max(lens_q), 2500,
                                      k_scales=sc[0], v_scales=sc[1], want_lse=True)
        check_attend(q, pool, lens_q, o, lse)
    assert qsa.device_status(clear=True) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_calls_without_rows(qsa, fp8):
    """No new tokens, no rows to read, no tokens to rotate: nothing is touched, nothing raises."""
    pool = Pool([5, 9], 4, fp8).fill()
    before = pool.k.view(torch.uint8).clone()
    none = prefix([0, 0])
    kv = torch.empty((0, HKV, D), dtype=torch.bfloat16, device="cuda")
    qsa.cache_write_paged(kv, kv, pool.k, pool.v, pool.table, none, prefix(pool.lens), **pool.args())
    k, v = qsa.cache_read_paged(pool.k, pool.v, pool.table, prefix(pool.lens), none, 0, **pool.args())
    assert k.shape == v.shape == (0, HKV, D)
    o, lse = qsa.chunk_attn_paged(torch.empty((0, HQ, D), dtype=torch.bfloat16, device="cuda"), pool.k, pool.v,
                                  pool.table, none, prefix(pool.lens), 0, want_lse=True, **pool.args())
    assert o.shape == (0, HQ, D) and lse.shape == (0, HQ)
    qo, ko = qsa.rope_axes(o, k, torch.empty((3, 0), dtype=torch.int32, device="cuda"), (4, 2, 2))
    assert qo.shape == o.shape and ko.shape == k.shape
    assert torch.equal(pool.k.view(torch.uint8), before) and qsa.device_status(clear=True) == 0


def test_host_tensors_are_refused(qsa):
    pool = Pool([5], 4, False).fill()
    cu = prefix([1])
    q = queries(1)
    with pytest.raises(ValueError):
        qsa.chunk_attn_paged(q.cpu(), pool.k, pool.v, pool.table, cu, prefix([5]), 1)
    with pytest.raises(ValueError):
        qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table.cpu(), cu, prefix([5]), 1)
    with pytest.raises(qsa.QSAError):
        qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, cu, prefix([5]), 1, o=q)
    with pytest.raises(qsa.QSAError):
        qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, cu, prefix([5]), 1,
                             ws=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(qsa.QSAError):
        qsa.rope_axes(q, None, torch.zeros((3, 1), dtype=torch.int32, device="cuda"), (100, 20, 20))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("most", [1, 5, 30])
def test_large_batches(qsa, most, fp8):
    """More sequences than the kernels keep the lengths of at hand, some of them empty."""
    g = torch.Generator().manual_seed(most)
    lens_q = torch.randint(0, most + 1, (200,), generator=g).tolist()
    lens_q[7] = most
    lens_k = [n + int(x) for n, x in zip(lens_q, torch.randint(0, 400, (200,), generator=g))]
    pool = Pool(lens_k, 16, fp8, seed=most).fill()
    q = queries(sum(lens_q))
    for window, sinks in ((0, 0), (60, 4)):
        o, lse = attend(qsa, q, pool, lens_q, window, sinks)
        check_attend(q, pool, lens_q, o, lse, window, sinks)
    assert qsa.device_status(clear=True) == 0


def test_equals_the_packed_dense_attention(qsa):
    """A whole prompt at once: the packed dense kernel computes the same."""
    lens = [300, 129]
    pool = Pool(lens, 16, False, seed=5).fill()
    cu = prefix(lens)
    q = queries(429)
    k, v = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, 429)
    want, want_lse = qsa.dense_attn_prefill(q, k, v, cu, cu, 300, want_lse=True, max_len_k=300)
    o, lse = attend(qsa, q, pool, lens)
    check_attend(q, pool, lens, o, lse)
    # both within the bound of the definition: twice the probabilities' and the output's rounding
    assert (o.float() - want.float()).abs().max().item() <= 4 * U16 * float(v.float().abs().max())
    assert (lse - want_lse).abs().max().item() <= 1e-3


@pytest.mark.parametrize("fp8", [False, True])
def test_serving_path(qsa, fp8):
    """A layer's path as it is served: rotate by three axes, write, attend a prompt in chunks, then
    decode token by token (each step a captured one), then read the cache back for the sparse prefill
    with a full budget, which must agree with the dense result."""
    total, chunks, s = 140, [64, 50, 20, 1, 1, 4], (16, 8, 8)
    g = torch.Generator(device="cuda").manual_seed(11)
    q = torch.randn((total, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((total, HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    v = torch.randn((total, HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.arange(total, dtype=torch.int32, device="cuda").repeat(3, 1)
    pos[1, 20:60] = torch.arange(40, device="cuda", dtype=torch.int32) // 8 + 20  # an image's patches
    pos[2, 20:60] = torch.arange(40, device="cuda", dtype=torch.int32) % 8 + 20
    pool = Pool([total], 12, fp8)
    outs, lses, at = [], [], 0
    for n in chunks:
        sl = slice(at, at + n)
        at += n
        qr, kr = qsa.rope_axes(q[sl], k[sl], pos[:, sl].contiguous(), s, interleaved=True)
        cu_q, cu_k = prefix([n]), prefix([at])
        qsa.cache_write_paged(kr, v[sl], pool.k, pool.v, pool.table, cu_q, cu_k, **pool.args())
        o, lse = qsa.chunk_attn_paged(qr, pool.k, pool.v, pool.table, cu_q, cu_k, n, at, want_lse=True, **pool.args())
        outs.append(o)
        lses.append(lse)
    assert at == total
    qr, _ = qsa.rope_axes(q, None, pos, s, interleaved=True)
    o, lse = torch.cat(outs), torch.cat(lses)
    check_attend(qr, pool, [total], o, lse)
    cu = prefix([total])
    kk, vv = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, total, **pool.args())
    blocks = (total + 3) // 4
    sel = torch.full((total, 64), -1, dtype=torch.int32, device="cuda")
    for t in range(total):
        sel[t, :t // 4 + 1] = torch.arange(t // 4 + 1, dtype=torch.int32)
    assert blocks <= 64
    sparse = qsa.sparse_attn_prefill(qr, kk, vv, sel, cu, cu, cfg=qsa.default_config(budget_blocks=64))
    # the same attention of the same rows: twice the probabilities' and the output's rounding
    assert (o.float() - sparse.float()).abs().max().item() <= 4 * U16 * float(vv.float().abs().max())
    assert qsa.device_status(clear=True) == 0
