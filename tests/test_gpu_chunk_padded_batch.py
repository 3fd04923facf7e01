"""A few new tokens in a batch that is mostly empty, as a captured step of the largest batch runs them: right, and
in a time that does not grow with the square of the batch."""
import pytest
import torch

from paged_common import D, HQ, Pool, check_attend, prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def queries(n):
    g = torch.Generator(device="cuda").manual_seed(n)
    return torch.randn((n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [14, 15, 30, 33, 130, 1500])
@pytest.mark.parametrize("most", [1, 4, 40])
def test_rows_among_empty_sequences(qsa, batch, most, fp8):
    """Tokens at the first, the last and a few sequences between; one of them sits before its cache."""
    lens_q, lens_k = [0] * batch, [0] * batch
    for i, s in enumerate((0, 3, batch // 2, batch - 1)):
        lens_q[s], lens_k[s] = max(1, most - i), 900 - 250 * i
    lens_k[3] = 0
    lens_k[5] = 77                                        # a cache without new tokens
    pool = Pool(lens_k, 16, fp8, seed=most).fill()
    q = queries(sum(lens_q) + 2)
    o = torch.full_like(q, 3.0)
    lse = torch.full((q.shape[0], HQ), 4.0, device="cuda")
    qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(lens_q), prefix(lens_k), max(lens_q), max(lens_k),
                         o=o, lse=lse, **pool.args())
    assert qsa.device_status(clear=True) == 0
    check_attend(q, pool, lens_q, o, lse)
    assert (o[-2:] == 3.0).all() and (lse[-2:] == 4.0).all()


def test_time_of_a_mostly_empty_batch(qsa):
    """Four tokens among 4096 sequences against four among 8: 7 times the small call's time (270 times it where
    the merge scanned every slot for every slot)."""
    def time(batch):
        lens_q, lens_k = [1] * 4 + [0] * (batch - 4), [1000] * 4 + [0] * (batch - 4)
        pool = Pool(lens_k, 64, True).fill()
        q, cu_q, cu_k = queries(4), prefix(lens_q), prefix(lens_k)
        best = float("inf")
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, cu_q, cu_k, 1, 1000, **pool.args())
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert time(4096) < 40 * time(8)
