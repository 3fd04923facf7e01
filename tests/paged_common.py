"""Pools, 64-bit definitions and derived error bounds for the tests of the paged-cache calls."""
import math

import torch

HQ, HKV, D, GROUP = 24, 2, 256, 12
SCALE = 1.0 / 16.0
U16 = 2.0 ** -8      # bf16: half a step relative to the value
U8 = 2.0 ** -4       # e4m3, normal codes
U32 = 2.0 ** -24


def prefix(lens, device="cuda"):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


class Pool:
    """A paged K/V pool whose pages are dealt to the sequences at random; memory that no token
    owns holds `fill` (default: NaN, or the NaN row byte)."""

    def __init__(self, lens, page, fp8, seed=0, spare=2, device="cuda", extra_cols=1, fill=float("nan")):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.lens, self.page, self.fp8 = list(lens), page, fp8
        per = [-(-L // page) for L in lens]
        pages = max(1, sum(per) + spare)
        order = torch.randperm(pages, generator=g).tolist()
        self.table = torch.full((len(lens), max(max(per), 1) + extra_cols), -1, dtype=torch.int32)  # never a page
        at = 0
        for s, m in enumerate(per):
            self.table[s, :m] = torch.tensor(order[at:at + m], dtype=torch.int32)
            at += m
        self.table = self.table.to(device)
        if fp8:
            self.k = torch.full((pages, page, HKV, D), 0x7F, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            self.v = self.k.clone()
            self.ks = torch.full((pages, page, HKV), 255, dtype=torch.uint8, device=device)
            self.vs = self.ks.clone()
        else:
            self.k = torch.full((pages, page, HKV, D), fill, dtype=torch.bfloat16, device=device)
            self.v, self.ks, self.vs = self.k.clone(), None, None

    def rows(self, s, a, b):
        t = torch.arange(a, b, device=self.table.device)
        return self.table[s].long()[t // self.page] * self.page + t % self.page

    def fill(self, seed=1, spread=1.0):
        """Every token of every sequence: normal rows, or codes with scales around 2^-7."""
        g = torch.Generator(device=self.table.device).manual_seed(seed)
        for s, L in enumerate(self.lens):
            if L == 0:
                continue
            r = self.rows(s, 0, L)
            for x, sc in ((self.k, self.ks), (self.v, self.vs)):
                y = torch.randn((L, HKV, D), generator=g, device=self.table.device) * spread
                if self.fp8:
                    c = (y * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
                    x.view(torch.uint8).view(-1, HKV, D)[r] = c.view(torch.uint8)
                    sc.view(-1, HKV)[r] = torch.randint(117, 123, (L, HKV), generator=g, device=self.table.device,
                                                        dtype=torch.uint8)
                else:
                    x.view(-1, HKV, D)[r] = y.to(torch.bfloat16)
        return self

    def values(self, which, s, a, b):
        """fp64 rows [b - a, 2, 256] of sequence s."""
        x, sc = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        r = self.rows(s, a, b)
        if not self.fp8:
            return x.view(-1, HKV, D)[r].double()
        codes = x.view(torch.uint8).view(-1, HKV, D)[r].view(torch.float8_e4m3fn).double()
        e = sc.view(-1, HKV)[r].double() - 127
        return torch.where((e == 128)[..., None], math.nan, codes * torch.exp2(e)[..., None])

    def args(self):
        return dict(k_scales=self.ks, v_scales=self.vs)


def attend64(q, pool, lens_q, window=0, sinks=0):
    """(o, lse, bound of |o| errors, bound of |lse| errors) in fp64 for packed q."""
    o = torch.zeros((q.shape[0], HQ, D), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0], HQ), -math.inf, dtype=torch.float64, device=q.device)
    bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
    at = 0
    for s, (n, L) in enumerate(zip(lens_q, pool.lens)):
        if n == 0 or L == 0:
            at += n
            continue
        t = torch.arange(L - n, L, device=q.device)[:, None]
        j = torch.arange(L, device=q.device)
        seen = j <= t
        if window > 0:
            seen &= (t - j < window) | (j < sinks)
        k, v = pool.values("k", s, 0, L), pool.values("v", s, 0, L)
        anyone = seen.any(0)
        k, v = torch.where(anyone[:, None, None], k, 0.0), torch.where(anyone[:, None, None], v, 0.0)
        for h in range(HQ):
            x = q[at:at + n, h].double()
            z = (x @ k[:, h // GROUP].t()) * SCALE
            mag = ((x.abs() @ k[:, h // GROUP].abs().t()) * SCALE).masked_fill(~seen, 0).amax(1, keepdim=True)
            z = z.masked_fill(~seen, -math.inf)
            w = torch.logsumexp(z, 1, keepdim=True)
            p = torch.where(w > -math.inf, torch.exp(z - w), 0.0)
            r = p @ v[:, h // GROUP]
            o[at:at + n, h], lse[at:at + n, h] = r, w[:, 0]
            # A score is a sum of 256 products in fp32 (each of the sums within U32 of its partial
            # sum, at most `mag`), scaled twice; the exponent's argument rounds against |score| too.
            # dz bounds a score's error, and so the relative error of its probability beyond
            # the exponential's own 2^-22.  Probabilities round to bf16 before P V (U16), whose
            # fp32 sums over L terms and the merge of up to 2 * 512 pieces add L + 1024 roundings.
            dz = (256 + 8) * U32 * mag + 2.0 ** -22
            a = p @ v[:, h // GROUP].abs()
            bo[at:at + n, h] = a * (U16 + 2 * dz + (L + 1024) * U32) * 1.01 + r.abs() * U16
            bl[at:at + n, h] = (dz + (L + 1024) * U32 + 2.0 ** -22 + 2 * U32 * w.abs())[:, 0]
        at += n
    return o, lse, bo, bl


def check_attend(q, pool, lens_q, o, lse, window=0, sinks=0):
    ro, rl, bo, bl = attend64(q, pool, lens_q, window, sinks)
    n = sum(lens_q)
    err = (o[:n].double() - ro[:n]).abs() - bo[:n]
    assert n == 0 or (not torch.isnan(err).any() and err.max().item() <= 0), err.max().item()
    empty = rl == -math.inf
    assert torch.equal(lse[:n] == -math.inf, empty[:n])
    assert (o[:n][empty[:n]] == 0).all()
    dl = torch.where(empty, 0.0, (lse.double() - rl).abs() - bl)[:n]
    assert not torch.isnan(dl).any() and (n == 0 or dl.max().item() <= 0), dl.max().item()


def quantise64(x):
    """e4m3 codes (as fp64 values) and biased exponents of rows [..., 256] bf16, from the definition."""
    y = x.double()
    top = y.abs().amax(-1)
    e = torch.full(top.shape, -127, dtype=torch.int64, device=x.device)
    for cand in range(120, -128, -1):  # the smallest e with top <= 448 2^e
        e = torch.where(top <= 448 * 2.0 ** cand, cand, e)
    z = y * torch.exp2(-e.double())[..., None]
    m, ex = torch.frexp(z.abs())
    step = torch.exp2((ex - 1).clamp(min=-6).double() - 3)       # 3 mantissa bits, subnormals below 2^-6
    code = torch.round(z / step) * step                          # ties to even
    return code, (e + 127).to(torch.uint8)
