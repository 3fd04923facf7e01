"""Single new tokens over e4m3 caches whose values' scales differ by many powers of two between early and late
keys, with a late key far above the rest: what counts then is the late row, though an early one was the
largest that the kernel had seen.  Against the definition in 64 bits."""
import pytest
import torch

from paged_common import D, HKV, HQ, Pool, SCALE, attend64, prefix

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def fp16_bound(q, pool):
    """What the kernel's probabilities as fp16 add: below 2^-18 of the row's largest p 2^e an absolute
    2^-29 of it, for every key, times the key's code."""
    out = torch.zeros((len(pool.lens), HQ, D), dtype=torch.float64, device=q.device)
    for s, L in enumerate(pool.lens):
        r = pool.rows(s, 0, L)
        k = pool.values("k", s, 0, L)
        codes = pool.v.view(torch.uint8).view(-1, HKV, D)[r].view(torch.float8_e4m3fn).double().abs().sum(0)
        size = torch.exp2(pool.vs.view(-1, HKV)[r].double() - 127)
        for h in range(HQ):
            g = h // 12
            z = (k[:, g] @ q[s, h].double()) * SCALE
            p = torch.exp(z - torch.logsumexp(z, 0))
            out[s, h] = codes[g] * 2.0 ** -29 * (p * size[:, g]).max()
    return out


@pytest.mark.parametrize("lens", [[3000] * 64, [40000, 35001], [300, 129]])
@pytest.mark.parametrize("spread,top", [(20, 1.75), (30, 2.5), (40, 2.5), (40, 1.25), (24, 9.0), (60, 9.0)])
def test_late_key_with_small_values(qsa, lens, spread, top):
    """The last key scores 23 * top powers of two above the rest and its V scale is 2^-spread of theirs."""
    pool = Pool(lens, 64, True, seed=spread).fill(seed=len(lens))
    g = torch.Generator(device="cuda").manual_seed(3)
    u = torch.sign(torch.randn((HKV, D), generator=g, device="cuda"))
    q = u.repeat_interleave(HQ // HKV, 0).expand(len(lens), HQ, D).to(torch.bfloat16).contiguous()
    for s, L in enumerate(lens):
        r = pool.rows(s, L - 1, L)
        pool.k.view(torch.uint8).view(-1, HKV, D)[r] = (u * top).to(torch.float8_e4m3fn).view(torch.uint8)
        pool.ks.view(-1, HKV)[r] = 127
        pool.vs.view(-1, HKV)[r] -= spread
    ones = [1] * len(lens)
    o, lse = qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(ones), prefix(lens), 1, max(lens),
                                  want_lse=True, **pool.args())
    assert qsa.device_status(clear=True) == 0
    ro, rl, bo, bl = attend64(q, pool, ones)
    err = (o.double() - ro).abs() - (bo + fp16_bound(q, pool))
    assert not torch.isnan(err).any() and err.max().item() <= 0, (err.max().item(), ro.abs().max().item())
    assert ((lse.double() - rl).abs() <= bl).all()


@pytest.mark.parametrize("lens", [[3000] * 64, [40000, 35001]])
def test_maximum_that_moves_with_every_tile(qsa, lens):
    """Scores that climb by about 12 powers of two per 128 keys while the values' scales fall by as much, so
    that all tiles stay of one size in the sum."""
    pool = Pool(lens, 64, True, seed=5).fill(seed=6)
    g = torch.Generator(device="cuda").manual_seed(4)
    u = torch.sign(torch.randn((HKV, D), generator=g, device="cuda"))
    q = u.repeat_interleave(HQ // HKV, 0).expand(len(lens), HQ, D).to(torch.bfloat16).contiguous()
    for s, L in enumerate(lens):
        last = L // 128
        for i in range(max(0, last - 7), last + 1):  # the last eight tiles, one key of each
            r = pool.rows(s, min(128 * i + 5, L - 1), min(128 * i + 5, L - 1) + 1)
            step = i - last + 8                      # 1 .. 8: scores of 23 * 0.5 * step powers of two
            pool.k.view(torch.uint8).view(-1, HKV, D)[r] = (u * 0.5 * step).to(torch.float8_e4m3fn).view(torch.uint8)
            pool.ks.view(-1, HKV)[r] = 127
            pool.vs.view(-1, HKV)[r] = 120 - 11 * step
    ones = [1] * len(lens)
    o, lse = qsa.chunk_attn_paged(q, pool.k, pool.v, pool.table, prefix(ones), prefix(lens), 1, max(lens),
                                  want_lse=True, **pool.args())
    ro, rl, bo, bl = attend64(q, pool, ones)
    err = (o.double() - ro).abs() - (bo + fp16_bound(q, pool))
    assert not torch.isnan(err).any() and err.max().item() <= 0, (err.max().item(), ro.abs().max().item())
    assert ((lse.double() - rl).abs() <= bl).all()
