"""The group norm with its activation, and its backward, against their formulas in 64 bits.

Tolerances are relative to 2-norms.  A bf16 result is rounded once, each value by 2^-8 of it at
most; an fp32 one, and a bf16 one before its rounding, is off by a few fp32 roundings and the error
of the exponential, 2^-20 of the values it is made of.  dx is a difference of terms of the size of
rstd dn, and each of its errors is relative to that; n is rstd times a difference of values of
the size of x, so that its own error is 2^-23 rstd |x|, which enters dx as a factor of rstd dn
three times (n, the mean of dn n, and the values dn of an activation of n).  dweight and dbias are
sums over the tokens of terms t, each off by 2^-20 |t| at most, so that a sum is off by 2^-20 of the
sum of |t|.  The sum itself may be any part of that, since the terms' signs differ: sqrt(M) |dbias|
is of the size of sum |t| only on the average over many channels.  With a single channel a sum of
0.033 of 300 terms of size one was off by 1.2e-6: 4e-5 of the sum, 2^-28 of the terms.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
ROUNDED = {BF: 2.0 ** -8, F32: 2.0 ** -24}
COMPUTED = 2.0 ** -20


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_85_amd as gdr
    return gdr


def inputs(M, G, D, x=BF, gate=None, bias=True, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    C = G * D
    return dict(x=(normal(M, C) * (0.2 + torch.rand(M, 1, device="cuda", generator=gen)) + 0.5 * normal(1, C)).to(x),
                weight=1 + 0.2 * normal(C), bias=0.3 * normal(C) if bias else None,
                gate=None if gate is None else normal(M, C).to(gate))


def exact(a, G, act, center, dout=None, eps=1e-5):
    """out, and with dout (dx, dweight, dbias, dgate) and the norm of what dx is a difference of."""
    C = a["x"].shape[-1]
    x = a["x"].double().reshape(-1, G, C // G)
    M = x.shape[0]
    size = x.abs().amax(-1, keepdim=True)
    x = x - x.mean(-1, keepdim=True) if center else x
    rstd = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    n = (x * rstd).reshape(M, C)
    w = torch.ones(C, dtype=torch.float64, device="cuda") if a["weight"] is None else a["weight"].double()
    y = n * w + (0 if a["bias"] is None else a["bias"].double())
    gated = a["gate"] is not None
    z = a["gate"].double().reshape(M, C) if gated else y
    s = 1 / (1 + torch.exp(-z))
    f, slope = {"silu": (z * s, s + z * s * (1 - s)), "sigmoid": (s, s * (1 - s)), None: (z, torch.ones_like(z))}[act]
    out = y * f if gated else f
    if dout is None:
        return out
    dout = dout.double().reshape(M, C)
    dy = dout * (f if gated else slope)
    dn = (dy * w).reshape(M, G, -1)
    nn = n.reshape(M, G, -1)
    dx = rstd * (dn - nn * (dn * nn).mean(-1, keepdim=True) - (dn.mean(-1, keepdim=True) if center else 0))
    return out, dx.reshape(M, C), Sum(dy * n), Sum(dy), dout * y * slope if gated else None, \
        (rstd * dn.abs().amax(-1, keepdim=True).expand(dn.shape) * (1 + size * rstd)).norm().item()


class Sum:
    """A sum over the tokens, and the norm of the sums of its terms' sizes."""

    def __init__(self, terms):
        self.value, self.scale = terms.sum(0), terms.abs().sum(0).norm().item()


def check(got, want, dtype, what, scale=0.0):
    if isinstance(want, Sum):
        want, scale = want.value, want.scale
    assert got.dtype == dtype, what
    d, n = (got.double().reshape(want.shape) - want).norm().item(), want.norm().item()
    tol = ROUNDED[dtype] * n + COMPUTED * max(n, scale)
    assert math.isfinite(d) and d <= tol, "%s: %.3g of %.3g, norm %.3g" % (what, d, tol, n)


WIDTHS = [1, 2, 7, 8, 16, 24, 65, 96, 128, 325, 512, 513, 520, 1024, 2048, 2056, 2600, 4096, 5000, 8191, 8192]


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("act", ["silu", "sigmoid", None])
@pytest.mark.parametrize("D", WIDTHS)
def test_forward_and_backward(gdr, D, act, center):
    for G, M in ((1, 1), (3, 67)) if D > 512 else ((1, 300), (18, 7), (5, 1), (32, 67)):
        for x, gate, out in ((BF, BF, BF), (F32, None, F32)) if act else ((F32, BF, BF), (BF, None, F32)):
            a = inputs(M, G, D, x, gate, bias=D % 3 != 0, seed=D)
            dout = torch.randn(M, G * D, device="cuda").to(out)
            y, dx, dw, db, dz, scale = exact(a, G, act, center, dout)
            got = gdr.group_norm(a["x"], G, a["weight"], a["bias"], a["gate"], activation=act, center=center,
                                 output_dtype=out)
            check(got, y, out, "out")
            g = gdr.group_norm_bwd(a["x"], G, dout, a["weight"], a["bias"], a["gate"], activation=act, center=center)
            check(g[0], dx, x, "dx", scale)
            check(g[1], dw, F32, "dweight")
            if a["bias"] is not None:
                check(g[2], db, F32, "dbias")
            if gate is not None:
                check(g[3], dz, gate, "dgate")


@pytest.mark.parametrize("x,gate,out", [(x, z, y) for x in (BF, F32) for z in (BF, F32) for y in (BF, F32)])
@pytest.mark.parametrize("D", [48, 65, 600, 3000, 8000])
def test_types(gdr, D, x, gate, out):
    a = inputs(9, 2, D, x, gate)
    dout = torch.randn(9, 2 * D, device="cuda").to(out)
    y, dx, dw, db, dz, scale = exact(a, 2, "silu", True, dout)
    check(gdr.group_norm(a["x"], 2, a["weight"], a["bias"], a["gate"], output_dtype=out), y, out, "out")
    g = gdr.group_norm_bwd(a["x"], 2, dout, a["weight"], a["bias"], a["gate"])
    check(g[0], dx, x, "dx", scale)
    check(g[3], dz, gate, "dgate")


def test_many_tokens_and_default_types(gdr):
    a = inputs(20011, 4, 64, F32, BF)
    y = gdr.group_norm(a["x"], 4, a["weight"], a["bias"], a["gate"])
    check(y, exact(a, 4, "silu", True), BF, "out")  # the gate's type
    y = gdr.group_norm(a["x"], 4, a["weight"], a["bias"])
    check(y, exact(dict(a, gate=None), 4, "silu", True), F32, "out")
    # no weight, no bias
    y = gdr.group_norm(a["x"], 4, activation=None)
    check(y, exact(dict(x=a["x"], weight=None, bias=None, gate=None), 4, None, True), F32, "out")
    assert gdr.group_norm(a["x"][:0], 4).shape == (0, 256)
    g = gdr.group_norm_bwd(a["x"][:0], 4, a["x"][:0], a["weight"], a["bias"])
    assert g[0].shape == (0, 256) and not g[1].any() and not g[2].any()


@pytest.mark.parametrize("D", [64, 65])
def test_rows_of_wider_tensors(gdr, D):
    """Slices of a projection, transposed and expanded rows, and rows off 16 bytes."""
    C, G = 2 * D, 2
    wide = torch.randn(3, 11, 3 * C + 8, device="cuda").to(BF)
    w = torch.randn(C, device="cuda")
    for x in (wide[..., :C], wide[..., 8:C + 8], wide[..., 1:C + 1], wide[:, ::2, :C], wide.transpose(0, 1)[..., :C],
              wide[:1, :1, :C].expand(3, 11, C), wide[0, :, :C], wide[0, 0, :C], wide[:, :1, :C].expand(3, 11, C)):
        gate = wide[..., C:2 * C].expand(x.shape) if x.shape == wide[..., :C].shape else None
        a = dict(x=x, weight=w, bias=None, gate=gate)
        want = exact(a, G, "silu", True)
        got = gdr.group_norm(x, G, w, gate=gate)
        assert got.shape == x.shape and got.is_contiguous()
        check(got, want, BF, "out")
        dout = torch.randn(x.shape, device="cuda")
        g = gdr.group_norm_bwd(x, G, dout, w, gate=gate)
        _, dx, dw, _, dz, scale = exact(a, G, "silu", True, dout)
        check(g[0], dx, BF, "dx", scale)
        check(g[1], dw, F32, "dweight")


def test_autograd_and_differences(gdr):
    gen = torch.Generator(device="cuda").manual_seed(3)
    for gated in (True, False):
        a = inputs(5, 3, 40, F32, F32 if gated else None, seed=4)
        leaves = {n: t.requires_grad_() for n, t in a.items() if t is not None}
        out = gdr.group_norm(a["x"], 3, a["weight"], a["bias"], a["gate"])
        dout = torch.randn(out.shape, device="cuda", generator=gen)
        grads = dict(zip(leaves, torch.autograd.grad(out, list(leaves.values()), dout)))
        for name, t in leaves.items():
            step = torch.randn(t.shape, device="cuda", generator=gen, dtype=torch.float64)
            at = lambda e: {n: None if u is None else u.detach().double() + (e * step if n == name else 0)  # noqa: E731
                            for n, u in a.items()}
            # central difference in 64 bits: its own error is about 1e-6 of the third derivative
            d = ((exact(at(1e-3), 3, "silu", True) - exact(at(-1e-3), 3, "silu", True)) / 2e-3 * dout.double()).sum()
            assert abs((grads[name].double() * step).sum() - d) <= 1e-4 * (grads[name].norm() * step.norm()), name
        # weights without gradients, and in bfloat16
        x = a["x"].detach().requires_grad_()
        w = a["weight"].detach().to(BF)
        gdr.group_norm(x, 3, w, activation=None).sum().backward()  # (an expanded gradient)
        want = exact(dict(x=x.detach(), weight=w, bias=None, gate=None), 3, None, True, torch.ones(x.shape, device="cuda"))
        check(x.grad, want[1], F32, "dx", want[5])


def test_values_that_are_not_finite_stay_in_their_group(gdr):
    a = inputs(8, 4, 64, BF, BF)
    clean = gdr.group_norm(a["x"], 4, a["weight"], a["bias"], a["gate"])
    for bad in (math.inf, -math.inf, math.nan):
        x = a["x"].clone()
        x[3, 70] = bad
        got = gdr.group_norm(x, 4, a["weight"], a["bias"], a["gate"])
        assert got[3, 64:128].isnan().all()
        got[3, 64:128] = clean[3, 64:128]
        assert torch.equal(got, clean)
    # constant groups, and values whose squares overflow bf16 sums
    x = torch.full((2, 128), 7.0, device="cuda")
    assert not gdr.group_norm(x, 2, activation=None).any()
    x = 1e15 * torch.randn(4, 128, device="cuda")
    check(gdr.group_norm(x, 2, activation=None), exact(dict(x=x, weight=None, bias=None, gate=None), 2, None, True), F32, "out")


def test_streams_graphs_and_repeats(gdr):
    a = inputs(500, 8, 128, F32, BF)
    dout = torch.randn(500, 1024, device="cuda").to(BF)

    def both():
        y = gdr.group_norm(a["x"], 8, a["weight"], a["bias"], a["gate"])
        return (y, *gdr.group_norm_bwd(a["x"], 8, dout, a["weight"], a["bias"], a["gate"]))

    want = both()
    assert all(torch.equal(p, q) for p, q in zip(want, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
        graph = torch.cuda.CUDAGraph()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = both()
    for seed in range(3):
        a["x"].copy_(inputs(500, 8, 128, F32, BF, seed=seed)["x"])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(both(), kept))


def test_offsets_past_32_bits(gdr):
    """2.5e9 values: the last tokens' results are bit for bit those of the tokens alone."""
    M, C, last = 300000, 8192, 100
    x = torch.zeros(M, C, dtype=BF, device="cuda")
    dout = torch.zeros(M, C, dtype=BF, device="cuda")
    x[-last:] = torch.randn(last, C, device="cuda").to(BF)
    dout[-last:] = torch.randn(last, C, device="cuda").to(BF)
    weight, bias = torch.rand(C, device="cuda"), torch.rand(C, device="cuda")
    args = 64, dout, weight, bias
    y = gdr.group_norm(x, 64, weight, bias)
    assert torch.equal(y[-last:], gdr.group_norm(x[-last:], 64, weight, bias))
    got = gdr.group_norm_bwd(x, *args)
    want = gdr.group_norm_bwd(x[-last:], 64, dout[-last:], weight, bias)
    assert torch.equal(got[0][-last:], want[0]) and not got[0][:-last].any()
    for a, b, name in zip(got[1:3], want[1:3], ("dweight", "dbias")):
        # (the other tokens add zeros; 100 terms in another order)
        assert (a - b).norm() <= 2 ** -24 * last * b.norm(), name


@pytest.mark.parametrize("D", [517, 1030, 2050, 4100, 8185, 8187, 8189, 8190, 8191])
def test_wide_groups_off_a_multiple_of_eight(gdr, D):
    """Aligned rows whose groups begin anywhere: the widest have more pieces than a workgroup has places.
    Memory that the allocator hands out next holds NaN, so that a channel that is not written shows."""
    for G in (8, 4) if D % 2 == 0 else (8,):
        for center, x, gate, out in ((True, BF, BF, BF), (False, F32, None, F32)):
            a = inputs(5, G, D, x, gate, seed=D)
            dout = torch.randn(5, G * D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(G)).to(out)
            y, dx, dw, db, dz, scale = exact(a, G, "silu", center, dout)
            junk = [torch.full((5 * G * D,), math.nan, device="cuda") for _ in range(4)]
            torch.cuda.synchronize()
            del junk
            got = gdr.group_norm(a["x"], G, a["weight"], a["bias"], a["gate"], center=center, output_dtype=out)
            check(got, y, out, "out")
            g = gdr.group_norm_bwd(a["x"], G, dout, a["weight"], a["bias"], a["gate"], center=center)
            check(g[0], dx, x, "dx", scale)
            check(g[1], dw, F32, "dweight")
            check(g[2], db, F32, "dbias")
            if gate is not None:
                check(g[3], dz, gate, "dgate")


@pytest.mark.parametrize("gated", [True, False])
def test_slope_of_a_sigmoid_near_one(gdr, gated):
    """Where the sigmoid is near 1 its slope is small, and every value of it is as precise as elsewhere: the
    exponential's argument is rounded, 2^-24 |z|, and fewer than sixteen roundings follow."""
    z = torch.linspace(-30, 30, 4096, device="cuda").view(4, 1024)
    ones = torch.ones_like(z)
    if gated:  # y = 1: dgate is the slope
        weight, bias = torch.zeros(1024, device="cuda"), torch.ones(1024, device="cuda")
        got = gdr.group_norm_bwd(torch.randn(4, 1024, device="cuda"), 8, ones, weight, bias, z, activation="sigmoid")[3]
        at = z.double()
    else:  # y = bias: dbias is the slope
        got = torch.stack([gdr.group_norm_bwd(ones[:1], 8, ones[:1], ones[0], row, activation="sigmoid")[2] for row in z])
        at = z.double()
    e = torch.exp(-at.abs())
    want = e / (1 + e) ** 2
    off = (got.double() - want).abs() / (want * 2.0 ** -24 * (16 + 2 * at.abs()))
    assert off.max() <= 1, "%.3g times the tolerance at %.3g" % (off.max(), at.flatten()[off.argmax()])
