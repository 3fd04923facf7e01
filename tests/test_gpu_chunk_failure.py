"""The chunk attention's bounded waits, single CTA and pair: the QSA_DEBUG_CHECKS library (20 ms waits)
withholds the arrival of one half tile when qsa_debug_inject(2) is set.  The kernel's roles give up: the
call ends, the status word reads QSA_ERR_TIMEOUT, and the next call
without the fault gives what the call before it gave.  In a child process, so that the release library
stays untouched."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent("""
    import sys, torch
    sys.path[:0] = [{root!r}, {root!r} + "/tests"]
    from block_sparse_long_09_b200 import qsa
    from paged_common import HQ, D, Pool, check_attend, prefix
    assert qsa.LIB_PATH.endswith("libqsa_debug.so"), qsa.LIB_PATH
    qsa.device_status(clear=True)
    for fp8 in (False, True):
        for lens_q, lens_k in (([4, 7], [300, 1500]), ([60, 90], [400, 2000])):  # one CTA per item, a pair
            pool = Pool(lens_k, 16, fp8, seed=3).fill()
            g = torch.Generator(device="cuda").manual_seed(1)
            q = torch.randn((sum(lens_q), HQ, D), generator=g, device="cuda").to(torch.bfloat16)

            def call():
                o, lse = qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(lens_q), prefix(lens_k),
                                              max(lens_q), max(lens_k), want_lse=True, **pool.args())
                torch.cuda.synchronize()
                return o, lse

            first = call()
            assert qsa.device_status(clear=True) == 0
            check_attend(q, pool, lens_q, *first)
            assert qsa.library().qsa_debug_inject(2) == qsa.QSA_OK
            call()
            st = qsa.device_status(clear=True)
            assert st == qsa.QSA_ERR_TIMEOUT, st
            assert qsa.library().qsa_debug_inject(0) == qsa.QSA_OK
            again = call()
            assert qsa.device_status(clear=True) == 0
            assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    assert qsa.library().qsa_debug_inject(3) == qsa.QSA_ERR_INVALID_ARG
    print("CHILD-OK")
""")


def test_wait_timeout_returns_status_and_leaves_the_kernel_usable():
    from block_sparse_long_09_b200 import build
    build.build_all()
    assert torch.cuda.is_available()
    env = dict(os.environ, QSA_DEBUG_BUILD="1")
    p = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert p.returncode == 0 and "CHILD-OK" in p.stdout, p.stdout[-2000:] + p.stderr[-4000:]
