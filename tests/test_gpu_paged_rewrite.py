"""What an e4m3 row is after it was written, read back and written again: the same values, in the same codes or
in codes of twice the size under a scale byte one less."""
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


def test_rewritten_rows(qsa):
    # maxima just above 448 2^e, from where rounding to the next byte's codes leads back down to it (the codes around
    # 224 lie 16 apart, so up to 464 for e = 0, 464 itself to the even code 224), and maxima that stay
    tops = [450.0, 456.0, 464.0, 900.0, 1.7578125, 466.0, 448.0, 470.0, 100.0, 1.0]
    falls = [True] * 5 + [False] * 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((len(tops), HKV, D), generator=g, device="cuda").clamp(-3, 3)
    for i, t in enumerate(tops):
        x[i] *= t / 4
        x[i, :, 17] = -t
    x = x.to(torch.bfloat16)
    assert torch.equal(x[:, 0, 17].float(), -torch.tensor(tops, device="cuda"))
    pool, cu = Pool([len(tops)], 4, True), prefix([len(tops)])
    r = pool.rows(0, 0, len(tops))
    qsa.cache_write_paged(x, x, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    byte = pool.ks.view(-1, HKV)[r].int()
    code = pool.k.view(torch.uint8).view(-1, HKV, D)[r].view(torch.float8_e4m3fn).double()
    k, v = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, len(tops), **pool.args())
    qsa.cache_write_paged(k, v, pool.k, pool.v, pool.table, cu, cu, **pool.args())
    byte2 = pool.ks.view(-1, HKV)[r].int()
    code2 = pool.k.view(torch.uint8).view(-1, HKV, D)[r].view(torch.float8_e4m3fn).double()
    k2, v2 = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, len(tops), **pool.args())
    assert torch.equal(k.view(torch.int16), k2.view(torch.int16)) and torch.equal(v.view(torch.int16), v2.view(torch.int16))
    down = torch.tensor(falls, device="cuda")[:, None].expand(len(tops), HKV)
    assert torch.equal(byte - byte2, down.int())
    assert torch.equal(code2, code * torch.where(down, 2.0, 1.0)[..., None])
    # both writes by the definition
    for rows, b, c in ((x, byte, code), (k, byte2, code2)):
        want_code, want_byte = quantise64(rows)
        assert torch.equal(b, want_byte.int()) and torch.equal(c, want_code)
