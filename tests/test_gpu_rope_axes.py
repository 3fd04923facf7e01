"""Rotary positions with three axes on the GPU against the rotation in 64 bits, its gradient against the
formula's and against differences."""
import math

import pytest
import torch

from paged_common import D, HKV, HQ, U16, U32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def qsa():
    from block_sparse_long_09_b200 import build
    build.build()
    from block_sparse_long_09_b200 import qsa as q
    q.device_status(clear=True)
    return q


def axis_of(i, s, mixed):
    if mixed:
        if i % 3 == 1 and i // 3 < s[1]:
            return 1
        return 2 if i % 3 == 2 and i // 3 < s[2] else 0
    return 0 if i < s[0] else (1 if i < s[0] + s[1] else 2)


def rotate64(x, pos, s, mixed, base, inverse=False):
    """(rotated rows, bound of the error): x fp64 [T, heads, 256]."""
    h = sum(s)
    y, b = x.clone(), torch.zeros_like(x)
    for i in range(h):
        a = pos[axis_of(i, s, mixed)].double() * float(base) ** (-i / h) * (-1.0 if inverse else 1.0)
        c, n = a.cos()[:, None], a.sin()[:, None]
        y[..., i], y[..., i + h] = x[..., i] * c - x[..., i + h] * n, x[..., i] * n + x[..., i + h] * c
        # sine and cosine rounded to fp32 (U32 each), two products and a sum (U32 each): 4 U32 of
        # both magnitudes covers them.  The angle in fp64, in units of 2^-53 of itself: the exponent
        # x <= log2(base) rounds three times here and once in the formula above (x ln 2 each), the
        # power, 1 / pi, and the products to the angle are 8 at most.  Then one rounding to bf16
        mag = x[..., i].abs() + x[..., i + h].abs()
        e = mag * (4 * U32 + a.abs()[:, None] * (4 * math.log2(base) * math.log(2) + 8) * 2.0 ** -53)
        b[..., i], b[..., i + h] = y[..., i].abs() * U16 + e, y[..., i + h].abs() * U16 + e
    return y, b


def case(T, far, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = torch.randn((T, HQ, D), generator=g, device="cuda").to(torch.bfloat16)
    k = torch.randn((T, HKV, D), generator=g, device="cuda").to(torch.bfloat16)
    return q, k, torch.randint(-far // 8, far, (3, T), generator=g, device="cuda", dtype=torch.int32)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("T,s,mixed,far", [
    (1, (16, 8, 8), False, 64), (9, (1, 0, 0), False, 1000), (7, (0, 0, 3), False, 1 << 20),
    (701, (12, 10, 10), True, 16384), (33, (5, 2, 1), True, 4096), (16, (64, 32, 32), False, 1 << 20),
    (5, (43, 43, 42), True, 2000000000), (8, (128, 0, 0), True, 1 << 24), (300, (3, 5, 7), False, 262144),
    (1500, (24, 20, 20), True, 262144)])
def test_rotation(qsa, T, s, mixed, far, inverse):
    q, k, pos = case(T, far, seed=T)
    qo, ko = qsa.rope_axes(q, k, pos, s, interleaved=mixed, inverse=inverse)
    h = sum(s)
    for x, got in ((q, qo), (k, ko)):
        want, bound = rotate64(x.double(), pos, s, mixed, 10000.0, inverse)
        assert ((got.double() - want).abs() <= bound).all()
        assert torch.equal(got[..., 2 * h:].view(torch.int16), x[..., 2 * h:].view(torch.int16))


def test_another_base(qsa):
    q, k, pos = case(40, 100000)
    cfg = qsa.default_config(rope_base=5000000.0)
    qo, _ = qsa.rope_axes(q, k, pos, (24, 20, 20), cfg=cfg)
    want, bound = rotate64(q.double(), pos, (24, 20, 20), False, 5000000.0)
    assert ((qo.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("s", [(16, 8, 8), (5, 2, 1), (3, 5, 7)])
def test_in_place_and_alone(qsa, s):
    q, k, pos = case(65, 4096)
    qo, ko = qsa.rope_axes(q, k, pos, s)
    only_q, none = qsa.rope_axes(q, None, pos, s)
    _, only_k = qsa.rope_axes(None, k, pos, s)
    assert none is None and torch.equal(only_q, qo) and torch.equal(only_k, ko)
    q2, k2 = q.clone(), k.clone()
    qsa.rope_axes(q2, k2, pos, s, q_out=q2, k_out=k2)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_values_that_are_not_finite_stay_in_their_pair(qsa):
    for s in ((16, 8, 8), (3, 5, 7)):
        h = sum(s)
        q, k, pos = case(4, 4096)
        clean, _ = qsa.rope_axes(q, k, pos, s)
        q[1, 3, 2] = float("nan")
        q[2, 5, h + 1] = float("inf")
        q[3, 7, 2 * h] = float("nan")
        out, _ = qsa.rope_axes(q, k, pos, s)
        touched = torch.zeros_like(q, dtype=torch.bool)
        touched[1, 3, 2] = touched[1, 3, h + 2] = touched[2, 5, 1] = touched[2, 5, h + 1] = touched[3, 7, 2 * h] = True
        assert torch.equal(out[~touched], clean[~touched]) and torch.isnan(out[1, 3, 2])


def test_gradient(qsa):
    """The gradient of <g, rope(x)> is the inverse rotation of g: against the formula, and against
    differences of the rotation in 64 bits along random directions."""
    s, mixed = (12, 10, 10), True
    x, _, pos = case(20, 16384, seed=3)
    gr, _, _ = case(20, 16384, seed=4)
    got, _ = qsa.rope_axes(gr, None, pos, s, interleaved=mixed, inverse=True)
    xr = x.double().requires_grad_()
    y, _ = rotate64(xr.clone(), pos, s, mixed, 10000.0)
    # rotate64 clones and writes in place: autograd differentiates the formula itself
    (y * gr.double()).sum().backward()
    _, bound = rotate64(gr.double(), pos, s, mixed, 10000.0, True)
    assert ((got.double() - xr.grad).abs() <= bound).all()
    for seed in range(3):
        d, _, _ = case(20, 16384, seed=10 + seed)
        d = d.double()
        # the rotation is linear: a difference quotient of any step is exact beyond 64-bit rounding
        up, _ = rotate64(x.double() + d, pos, s, mixed, 10000.0)
        dn, _ = rotate64(x.double() - d, pos, s, mixed, 10000.0)
        quotient = ((up - dn) / 2 * gr.double()).sum().item()
        slack = (bound * d.abs()).sum().item() + 1e-9
        assert abs((got.double() * d).sum().item() - quotient) <= slack


def test_there_and_back(qsa):
    q, k, pos = case(100, 1 << 20)
    qo, ko = qsa.rope_axes(q, k, pos, (16, 8, 8))
    qb, _ = qsa.rope_axes(qo, ko, pos, (16, 8, 8), inverse=True)
    _, b0 = rotate64(q.double(), pos, (16, 8, 8), False, 10000.0)
    _, b1 = rotate64(qo.double(), pos, (16, 8, 8), False, 10000.0, True)
    # the first rounding's error is rotated: both of its pair's errors may reach a value
    h = 32
    spread = b0.clone()
    spread[..., :h] += b0[..., h:2 * h]
    spread[..., h:2 * h] += b0[..., :h]
    assert ((qb.double() - q.double()).abs() <= b1 + spread).all()


def test_another_stream_and_a_graph(qsa):
    q, k, pos = case(50, 4096)
    want, _ = qsa.rope_axes(q, k, pos, (16, 8, 8))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        qsa.rope_axes(q, k, pos, (16, 8, 8), q_out=qo, k_out=ko)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want)
    pos.add_(17)
    want, _ = qsa.rope_axes(q, k, pos, (16, 8, 8))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(qo, want)
