"""A pool that qsa_cache_write_paged fills, read by the sparse paged decode; and paged-cache calls whose first call
in a process is a captured one."""
import os
import subprocess
import sys
import textwrap

import numpy as np
import pytest
import torch

import oracle
from block_sparse_long_09_b200 import inputs
from paged_common import Pool, prefix
from parity_common import SCALE, check_attn

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


@pytest.mark.parametrize("page", [4, 64])
def test_sparse_decode_over_written_pages(qsa, page):
    """A prompt and then one decoded token per sequence written; every sequence attends 128 of its blocks."""
    batch, k = 6, 128
    d = inputs.make_decode(batch, 900, 5000, seed=92)
    lens = list(d.seqlens)
    pool, start = Pool(lens, page, False, seed=5), np.cumsum([0] + lens)
    kc, vc = d.k_cache.cuda(), d.v_cache.cuda()
    rows = torch.cat([torch.arange(a, b - 1) for a, b in zip(start[:-1], start[1:])]).cuda()
    last = torch.tensor([b - 1 for b in start[1:]]).cuda()
    short = [L - 1 for L in lens]
    qsa.cache_write_paged(kc[rows], vc[rows], pool.k, pool.v, pool.table, prefix(short), prefix(short))
    qsa.cache_write_paged(kc[last], vc[last], pool.k, pool.v, pool.table, prefix([1] * batch), prefix(lens))
    g = np.random.default_rng(6)
    sel = np.full((batch, k), -1, dtype=np.int32)
    for s, L in enumerate(lens):
        bt = (L - 1) // 4
        sel[s] = np.append(np.sort(g.choice(bt, size=k - 1, replace=False)), bt)
    o, lse = qsa.sparse_attn_decode_paged(d.q.cuda(), pool.k, pool.v, pool.table, prefix(lens),
                                          torch.from_numpy(sel).cuda(), want_lse=True,
                                          cfg=qsa.default_config(budget_blocks=k))
    assert qsa.device_status(clear=True) == 0
    for s, L in enumerate(lens):
        ref_o, ref_lse = oracle.attend(d.q[s:s + 1], d.k_cache[start[s]:start[s + 1]], d.v_cache[start[s]:start[s + 1]],
                                       sel[s:s + 1], 1, L, 4, SCALE)
        check_attn(o[s:s + 1].float().cpu().numpy(), ref_o)
        np.testing.assert_allclose(lse[s:s + 1].cpu().numpy(), ref_lse, rtol=0, atol=2e-3)


CHILD = textwrap.dedent("""
    import sys, torch
    sys.path[:0] = [{root!r}, {root!r} + "/tests"]
    from block_sparse_long_09_b200 import qsa
    from paged_common import HKV, HQ, D, Pool, check_attend, prefix
    fp8, n = {fp8}, {n}
    lens = [400, 900]
    pool = Pool(lens, 16, fp8, seed=3).fill()
    g = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn((2 * n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    k, v = (torch.randn((2 * n, HKV, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    pos = torch.arange(2 * n, dtype=torch.int32, device="cuda").repeat(3, 1)
    cu_q, cu_k, cu_n = prefix([n, n]), prefix(lens), prefix([n, n])
    begin = torch.tensor([L - n for L in lens], dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, kr = qsa.rope_axes(q, k, pos, (16, 8, 8))
        qsa.cache_write_paged(kr, v, pool.k, pool.v, pool.table, cu_q, cu_k, **pool.args())
        o, lse = qsa.chunk_attn_paged(qr, pool.k, pool.v, pool.table, cu_q, cu_k, n, 900, want_lse=True, **pool.args())
        rk, rv = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu_k, cu_n, 2 * n, tok_begin=begin, **pool.args())
    graph.replay()
    torch.cuda.synchronize()
    assert qsa.device_status(clear=True) == 0
    check_attend(qr, pool, [n, n], o, lse)
    want = torch.cat([pool.values("k", s, L - n, L) for s, L in enumerate(lens)])
    assert torch.equal(rk.double(), want)
    print("CHILD-OK")
""")


@pytest.mark.parametrize("fp8,n", [(False, 1), (False, 5), (False, 30), (True, 1), (True, 5), (True, 30)])
def test_first_call_of_a_process_is_captured(qsa, fp8, n):
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, fp8=fp8, n=n)], capture_output=True, text=True,
                       timeout=600)
    assert p.returncode == 0 and "CHILD-OK" in p.stdout, p.stdout[-2000:] + p.stderr[-4000:]
