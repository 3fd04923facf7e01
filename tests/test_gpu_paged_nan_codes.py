"""e4m3 pools that hold the type's NaN codes (0x7F and 0xFF, which torch's own cast makes of whatever lies past
its range): every call that reads such a pool gives NaN where the definition does, and only there."""
import pytest
import torch

from paged_common import D, HKV, Pool, prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def test_read_gives_every_code_its_value(qsa):
    """All 256 codes in every place of a row, with scale bytes small, usual and large."""
    n = 256
    pool, cu = Pool([n], 16, True), prefix([n])
    codes = (torch.arange(n)[:, None, None] + torch.arange(D)[None, None, :] + torch.zeros((n, HKV, 1))).to(torch.int64)
    codes = (codes % 256).to(torch.uint8).cuda()
    r = pool.rows(0, 0, n)
    sc = torch.tensor([1, 40, 120, 127, 200, 246], dtype=torch.uint8, device="cuda")[torch.arange(n, device="cuda") % 6]
    for x, s in ((pool.k, pool.ks), (pool.v, pool.vs)):
        x.view(torch.uint8).view(-1, HKV, D)[r] = codes
        s.view(-1, HKV)[r] = sc[:, None].expand(n, HKV)
    k, v = qsa.cache_read_paged(pool.k, pool.v, pool.table, cu, cu, n, **pool.args())
    want = (codes.view(torch.float8_e4m3fn).double() * torch.exp2(sc.double() - 127)[:, None, None]).to(torch.bfloat16)
    bad = (codes & 0x7F) == 0x7F
    for got in (k, v):
        assert torch.equal(torch.isnan(got), bad)
        assert torch.equal(got[~bad].view(torch.int16), want[~bad].view(torch.int16))
