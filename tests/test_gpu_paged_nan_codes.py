"""e4m3 pools that hold the type's NaN codes (0x7F and 0xFF, which torch's own cast makes of whatever lies past
its range): every call that reads such a pool gives NaN where the definition does, and only there."""
import pytest
import torch

from paged_common import D, HKV, HQ, Pool, attend64, prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def queries(n, seed=7):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((n, HQ, D), generator=g, device="cuda").to(torch.bfloat16)


def attend(qsa, q, pool, lens_q):
    return qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(lens_q), prefix(pool.lens), max(lens_q),
                                max(pool.lens), want_lse=True, **pool.args())


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


@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("lens_q,lens_k", [([1], [500]), ([1] * 9, [200 + 31 * i for i in range(9)]), ([4], [500]),
                                           ([4, 7], [300, 1000]), ([64], [500]), ([130, 30], [700, 90])])
def test_value_codes(qsa, lens_q, lens_k, code):
    """NaN codes of V at keys that every new token sees: NaN in those dims of that KV head's rows alone."""
    pool = Pool(lens_k, 16, True, seed=2).fill()
    g = torch.Generator().manual_seed(code + len(lens_q))
    for s, (n, L) in enumerate(zip(lens_q, lens_k)):
        for dim in torch.randint(0, D, (12,), generator=g).tolist():
            key = int(torch.randint(0, L - n, (1,), generator=g))
            pool.v.view(torch.uint8).view(-1, HKV, D)[pool.rows(s, key, key + 1), s % 2, dim] = code
    q = queries(sum(lens_q))
    o, lse = attend(qsa, q, pool, lens_q)
    ro, rl, bo, bl = attend64(q, pool, lens_q)
    assert torch.isnan(ro).any() and not torch.isnan(rl).any()
    assert torch.equal(torch.isnan(o), torch.isnan(ro))
    good = ~torch.isnan(ro)
    assert ((o.double() - ro).abs()[good] <= bo[good]).all() and ((lse.double() - rl).abs() <= bl).all()


@pytest.mark.parametrize("code", [0x7F, 0xFF])
@pytest.mark.parametrize("n", [1, 4, 64])
def test_key_codes(qsa, n, code):
    """A NaN code of K: NaN rows and log-sum-exps of that KV head."""
    for dim in (0, 5, 127, 128, 250, 255):
        pool = Pool([500], 16, True, seed=2).fill()
        pool.k.view(torch.uint8).view(-1, HKV, D)[pool.rows(0, 100, 101), 1, dim] = code
        o, lse = attend(qsa, queries(n), pool, [n])
        assert torch.isnan(o[:, 12:]).all() and torch.isnan(lse[:, 12:]).all()
        assert not torch.isnan(o[:, :12]).any() and not torch.isnan(lse[:, :12]).any()


@pytest.mark.parametrize("what", ["byte", "code"])
@pytest.mark.parametrize("n", [1, 4, 64])
def test_values_of_keys_whose_probability_underflows(qsa, n, what):
    """A key 200 powers of two below the rest is seen all the same: its NaN reaches the row."""
    pool = Pool([500], 16, True, seed=2).fill()
    g = torch.Generator(device="cuda").manual_seed(1)
    u = torch.sign(torch.randn((HKV, D), generator=g, device="cuda"))
    q = u.repeat_interleave(HQ // HKV, 0).expand(n, HQ, D).to(torch.bfloat16).contiguous()
    r = pool.rows(0, 100, 101)
    pool.k.view(torch.uint8).view(-1, HKV, D)[r] = (u * -9).to(torch.float8_e4m3fn).view(torch.uint8)
    pool.ks.view(-1, HKV)[r] = 127
    if what == "byte":
        pool.vs.view(-1, HKV)[r, 0] = 255
    else:
        pool.v.view(torch.uint8).view(-1, HKV, D)[r, 0, :] = 0x7F
    o, lse = attend(qsa, q, pool, [n])
    assert torch.isnan(o[:, :12]).all() and not torch.isnan(o[:, 12:]).any() and not torch.isnan(lse).any()
