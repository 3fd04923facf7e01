"""Argument checks of the paged-cache calls, the chunk attention and the axis rotation: they are
refused on the host, before any CUDA call."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    return q


def pool(pages=4, page=8, dtype=torch.bfloat16):
    return torch.zeros((pages, page, 2, 256), dtype=dtype), torch.zeros((pages, page, 2, 256), dtype=dtype)


def scales(pages=4, page=8):
    return torch.zeros((pages, page, 2), dtype=torch.uint8)


I32 = dict(dtype=torch.int32)
TABLE, CU = torch.zeros((1, 3), **I32), torch.zeros(2, **I32)
ROWS = torch.zeros((5, 2, 256), dtype=torch.bfloat16)
Q = torch.zeros((5, 24, 256), dtype=torch.bfloat16)


def bad_pools():
    k, v = pool()
    k8, v8 = pool(dtype=torch.float8_e4m3fn)
    yield k.half(), v.half(), {}                                            # another type
    yield k, v8, {}                                                         # K and V unlike
    yield k, v[:3], {}
    yield k[:, :, :, :128], v[:, :, :, :128], {}                            # another head size
    yield k[:, ::2], v[:, ::2], {}                                          # strided pages
    yield k, v, dict(k_scales=scales(), v_scales=scales())                  # scales of bf16 pages
    yield k8, v8, {}                                                        # no scales
    yield k8, v8, dict(k_scales=scales(), v_scales=scales(3))
    yield k8, v8, dict(k_scales=scales().float(), v_scales=scales())
    yield k8, v8, dict(k_scales=scales(4, 16)[:, ::2], v_scales=scales())   # strided scales


@pytest.mark.parametrize("n", range(10))
def test_pools_are_checked(qsa, n):
    k, v, sc = list(bad_pools())[n]
    with pytest.raises(ValueError):
        qsa.cache_write_paged(ROWS, ROWS, k, v, TABLE, CU, CU, **sc)
    with pytest.raises(ValueError):
        qsa.cache_read_paged(k, v, TABLE, CU, CU, 5, **sc)
    with pytest.raises(ValueError):
        qsa.chunk_attn_paged(Q, k, v, TABLE, CU, CU, 5, 5, **sc)


def test_rows_and_lengths_are_checked(qsa):
    k, v = pool()
    for rows in (ROWS.float(), ROWS[:, :1], torch.zeros((5, 4, 256), dtype=torch.bfloat16)[:, ::2], ROWS[0]):
        with pytest.raises(ValueError):
            qsa.cache_write_paged(rows, ROWS, k, v, TABLE, CU, CU)
    with pytest.raises(ValueError):
        qsa.cache_write_paged(ROWS, ROWS[:4], k, v, TABLE, CU, CU)
    for cu in (CU.long(), torch.zeros(3, **I32), torch.zeros((2, 1), **I32)):
        with pytest.raises(ValueError):
            qsa.cache_write_paged(ROWS, ROWS, k, v, TABLE, CU, cu)
        with pytest.raises(ValueError):
            qsa.cache_read_paged(k, v, TABLE, CU, cu, 5)
        with pytest.raises(ValueError):
            qsa.chunk_attn_paged(Q, k, v, TABLE, CU, cu, 5, 5)
    for table in (TABLE.long(), torch.zeros((2, 3), **I32), torch.zeros((1, 6), **I32)[:, ::2]):
        with pytest.raises(ValueError):
            qsa.chunk_attn_paged(Q, k, v, table, CU, CU, 5, 5)
    with pytest.raises(ValueError):
        qsa.cache_read_paged(k, v, TABLE, CU, CU, 5, tok_begin=torch.zeros(2, **I32))
    with pytest.raises(ValueError):
        qsa.cache_read_paged(k, v, TABLE, CU, CU, 4, k=ROWS)
    with pytest.raises(ValueError):
        qsa.chunk_attn_paged(Q, k, v, TABLE, CU, CU, 5, 5, o=Q[:4])
    with pytest.raises(ValueError):
        qsa.chunk_attn_paged(Q, k, v, TABLE, CU, CU, 5, 5, lse=torch.zeros((5, 2)))


def test_rope_axes_arguments(qsa):
    pos = torch.zeros((3, 5), **I32)
    for args in ((None, None, pos, (1, 1, 1)), (Q, ROWS[:4], pos, (1, 1, 1)), (Q, ROWS, pos[:2], (1, 1, 1)),
                 (Q, ROWS, pos.long(), (1, 1, 1)), (Q, ROWS, pos, (1, 1)), (Q.float(), ROWS, pos, (1, 1, 1)),
                 (Q[:, :, :128], ROWS, pos, (1, 1, 1))):
        with pytest.raises(ValueError):
            qsa.rope_axes(*args)
    with pytest.raises(ValueError):
        qsa.rope_axes(None, ROWS, pos, (1, 1, 1), q_out=Q)
    with pytest.raises(ValueError):
        qsa.rope_axes(Q, None, pos, (1, 1, 1), q_out=Q[:4])


FAKE = 1 << 20  # addresses that are never dereferenced: every call below returns before any device work


def p(i):
    return ctypes.c_void_p(FAKE + (i << 32)) if i else None


def test_write_and_read_statuses(qsa):
    lib, cfg = qsa.library(), qsa.default_config()
    C = ctypes.byref(cfg)

    def write(k=1, v=2, cu_q=3, cu_k=4, batch=1, total=5, fmt=0, kp=6, vp=7, ks=0, vs=0, pages=4, page=8, table=8,
              cols=2, shift=0):
        return lib.qsa_cache_write_paged(C, ctypes.c_void_p(FAKE + (k << 32) + shift) if k else None, p(v), p(cu_q),
                                         p(cu_k), batch, total, fmt, p(kp), p(vp), p(ks), p(vs), pages, page,
                                         p(table), cols, None)

    for bad in (dict(k=0), dict(v=0), dict(cu_q=0), dict(cu_k=0), dict(batch=0), dict(total=-1), dict(fmt=2),
                dict(kp=0), dict(vp=0), dict(pages=0), dict(page=0), dict(table=0), dict(cols=0), dict(fmt=1, ks=9),
                dict(fmt=1, vs=9), dict(shift=2), dict(k=6), dict(v=7)):
        assert write(**bad) == qsa.QSA_ERR_INVALID_ARG, bad
    assert write(pages=1 << 28, page=16) == qsa.QSA_ERR_UNSUPPORTED
    assert write(total=0, k=0, v=0) == qsa.QSA_OK

    def read(fmt=0, kp=1, vp=2, ks=0, vs=0, pages=4, page=8, table=3, cols=2, cu_k=4, begin=0, cu_o=5, batch=1,
             total=5, k=6, v=7):
        return lib.qsa_cache_read_paged(C, fmt, p(kp), p(vp), p(ks), p(vs), pages, page, p(table), cols, p(cu_k),
                                        p(begin), p(cu_o), batch, total, p(k), p(v), None)

    for bad in (dict(fmt=-1), dict(kp=0), dict(vp=0), dict(pages=0), dict(page=0), dict(table=0), dict(cols=0),
                dict(cu_k=0), dict(cu_o=0), dict(batch=0), dict(total=-1), dict(k=0), dict(v=0), dict(fmt=1),
                dict(k=1), dict(v=2), dict(k=7)):
        assert read(**bad) == qsa.QSA_ERR_INVALID_ARG, bad
    assert read(pages=1 << 28, page=16) == qsa.QSA_ERR_UNSUPPORTED
    assert read(total=0) == qsa.QSA_OK


def test_chunk_attention_statuses(qsa):
    lib, cfg = qsa.library(), qsa.default_config()
    need = qsa.workspace_size(qsa.OP_CHUNK_PAGED, 1, 5)
    assert need > 0

    def call(q=1, fmt=0, kp=2, vp=3, ks=0, vs=0, pages=4, page=8, table=4, cols=2, cu_q=5, cu_k=6, batch=1, total=5,
             max_q=5, window=0, sinks=0, o=7, lse=0, ws=8, size=need, c=cfg):
        return lib.qsa_chunk_attn_paged(ctypes.byref(c), p(q), fmt, p(kp), p(vp), p(ks), p(vs), pages, page, p(table),
                                        cols, p(cu_q), p(cu_k), batch, total, max_q, window, sinks, p(o), p(lse),
                                        p(ws), size, None)

    for bad in (dict(q=0), dict(fmt=3), dict(kp=0), dict(vp=0), dict(fmt=1, ks=9), dict(pages=0), dict(page=0),
                dict(table=0), dict(cols=0), dict(cu_q=0), dict(cu_k=0), dict(batch=0), dict(total=-1), dict(max_q=-1),
                dict(window=-1), dict(sinks=-1), dict(o=0), dict(o=1), dict(o=2), dict(lse=3)):
        assert call(**bad) == qsa.QSA_ERR_INVALID_ARG, bad
    assert call(ws=0) == qsa.QSA_ERR_WORKSPACE_TOO_SMALL
    assert call(size=need - 1) == qsa.QSA_ERR_WORKSPACE_TOO_SMALL
    assert call(pages=1 << 28, page=16) == qsa.QSA_ERR_UNSUPPORTED
    assert call(c=qsa.default_config(head_dim=128)) == qsa.QSA_ERR_UNSUPPORTED
    assert call(total=0, q=0, o=0, ws=0, size=0) == qsa.QSA_OK


def test_rope_axes_statuses(qsa):
    lib, cfg = qsa.library(), qsa.default_config()

    def call(q=1, k=2, pos=3, total=5, s=(4, 2, 2), flags=0, qo=4, ko=5, c=cfg):
        return lib.qsa_rope_axes(ctypes.byref(c), p(q), p(k), p(pos), total, s[0], s[1], s[2], flags, p(qo), p(ko),
                                 None)

    for bad in (dict(pos=0), dict(total=-1), dict(s=(-1, 2, 2)), dict(s=(0, 0, 0)), dict(s=(100, 20, 9)),
                dict(flags=4), dict(qo=0), dict(ko=0), dict(q=0), dict(k=0), dict(s=(1, 3, 1), flags=1),
                dict(s=(0, 0, 1), flags=1), dict(qo=2), dict(ko=1), dict(qo=5, ko=5),
                dict(c=qsa.default_config(rope_base=1.0)), dict(c=qsa.default_config(rope_base=float("inf"))),
                dict(c=qsa.default_config(rope_base=float("nan")))):
        assert call(**bad) == qsa.QSA_ERR_INVALID_ARG, bad
    assert call(total=0) == qsa.QSA_OK
    assert call(q=0, k=0, qo=0, ko=0) == qsa.QSA_OK


def test_constants_match_the_header(qsa):
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "qsa.h")).read()
    defs = {n: int(v, 0) for n, v in re.findall(r"#define\s+(QSA_[A-Z0-9_]+)\s+([0-9x]+)u?\b", text)}
    for name in ("QSA_CACHE_BF16", "QSA_CACHE_E4M3", "QSA_ROPE_INTERLEAVED", "QSA_ROPE_INVERSE"):
        assert getattr(qsa, name) == defs[name], name
    assert qsa.OP_CHUNK_PAGED == defs["QSA_OP_CHUNK_PAGED"]


def test_workspace_holds_every_kernel(qsa):
    """The workspace of any mix of lengths: pieces of two per worker, and two numbers per item of the
    smallest groups."""
    for batch, rows in ((1, 1), (64, 64), (3, 4096), (1000, 100000)):
        need = qsa.workspace_size(qsa.OP_CHUNK_PAGED, batch, rows)
        pairs = 2 * 80 * 252 * 257 * 4 + 2 * 8 * (rows // 10 + batch)
        single = 2 * 160 * 12 * 257 * 4 + 2 * 8 * (rows + batch)
        assert need >= max(pairs, single) and need % 4 == 0
