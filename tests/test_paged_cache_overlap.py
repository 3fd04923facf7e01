"""Memory that a paged-cache call writes and that overlaps what it reads or also writes: refused on the host, before
any CUDA call."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    return q


FAKE = 1 << 20  # addresses that are never dereferenced: every call below returns before any device work


def p(x):
    """A place: i, or (i, bytes behind it)."""
    i, off = x if isinstance(x, tuple) else (x, 0)
    return ctypes.c_void_p(FAKE + (i << 32) + off) if i else None


POOL = 4 * 8 * 2 * 256  # bytes of an e4m3 array of 4 pages of 8 tokens; bf16: twice as many


def test_write(qsa):
    lib, cfg = qsa.library(), qsa.default_config()

    def write(k=1, v=2, fmt=0, kp=3, vp=4, ks=0, vs=0):
        return lib.qsa_cache_write_paged(ctypes.byref(cfg), p(k), p(v), p(7), p(8), 1, 5, fmt, p(kp), p(vp), p(ks),
                                         p(vs), 4, 8, p(9), 2, None)

    f8 = dict(fmt=1, ks=5, vs=6)
    for bad in (dict(vp=3), dict(vp=(3, 16)), dict(vp=(3, 2 * POOL - 16)), dict(kp=(4, 2 * POOL - 16)),
                dict(f8, vp=3), dict(f8, vp=(3, POOL - 16)), dict(f8, vs=5), dict(f8, vs=(5, POOL // 256 - 1)),
                dict(f8, ks=(3, POOL - 1)), dict(f8, vs=(4, 0)), dict(f8, ks=(4, 100)), dict(k=(3, 64)),
                dict(f8, v=(6, 0))):
        assert write(**bad) == qsa.QSA_ERR_INVALID_ARG, bad


def test_attention(qsa):
    lib, cfg = qsa.library(), qsa.default_config()
    need = qsa.workspace_size(qsa.OP_CHUNK_PAGED, 1, 5)
    rows = 5 * 24 * 256 * 2  # bytes of q and o

    def call(q=1, o=2, lse=3, ws=4, fmt=0, ks=0, vs=0, size=need):
        return lib.qsa_chunk_attn_paged(ctypes.byref(cfg), p(q), fmt, p(5), p(6), p(ks), p(vs), 4, 8, p(9), 2, p(10),
                                        p(11), 1, 5, 5, 0, 0, p(o), p(lse), p(ws), size, None)

    f8 = dict(fmt=1, ks=7, vs=8)
    for bad in (dict(o=1), dict(o=(1, rows - 16)), dict(lse=(1, 4)), dict(lse=(1, rows - 4)), dict(lse=2),
                dict(lse=(2, rows - 4)), dict(ws=1), dict(ws=(2, 16)), dict(ws=(3, 0)), dict(o=(4, need // 16 * 16 - 16)),
                dict(lse=(4, need - 4)), dict(q=(4, 32)), dict(ws=5), dict(ws=(6, 64)), dict(f8, ws=(7, 0)),
                dict(f8, lse=(8, 0)), dict(o=(5, 16))):
        assert call(**bad) == qsa.QSA_ERR_INVALID_ARG, bad


def test_rotation(qsa):
    lib, cfg = qsa.library(), qsa.default_config()

    def call(q=1, k=2, pos=3, qo=4, ko=5):
        return lib.qsa_rope_axes(ctypes.byref(cfg), p(q), p(k), p(pos), 5, 4, 2, 2, 0, p(qo), p(ko), None)

    for bad in (dict(pos=4), dict(pos=(5, 16)), dict(pos=(1, 0), qo=1), dict(qo=(3, 48)), dict(qo=2), dict(ko=(1, 16)),
                dict(qo=(1, 16)), dict(ko=(4, 0))):
        assert call(**bad) == qsa.QSA_ERR_INVALID_ARG, bad
