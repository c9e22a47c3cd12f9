"""Linear attention with a decay for each head against its definition, token by token in 64 bits:
the chunked form and its backward.

Tolerances are relative to the 2-norm of the exact result.  A bf16 result is rounded once, each
value by 2^-8 of it at most; what is computed before that is off by less than 2^-15 (two bf16 pieces
of an fp32 operand, 2^-17 a term, and fp32 sums).  An fp32 result is a sum of up to 64 + K terms per
chunk of products of fp32 rounding, and a state goes through one rounding per chunk: 2^-24 times
the root of the number of roundings, under 64 for every case here, 2^-18.  Gate gradients are
sums over up to 1024 tokens of differences q . dq - v . dv, whose terms' errors are 2^-24 times
the root of 128 of their size, 2^-15 in all: relative to the result or, where strong gates leave
little of it, to those terms (a fixed gate's is their sum over the tokens).
"""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8 + 2.0 ** -15, F32: 2.0 ** -18}
TOL_GATES = 2.0 ** -15


@pytest.fixture(scope="module")
def gdr():
    import gated_delta_rule_85_amd as gdr
    return gdr


def inputs(B, T, Hq, Hv, K, V, dtype, gates="token", h0=False, lens=None, seed=0, g_scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *s: torch.randn(s, device="cuda", generator=gen)  # noqa: E731
    N = B if lens is None else len(lens)
    x = dict(q=normal(B, T, Hq, K).to(dtype), k=normal(B, T, Hq, K).to(dtype), v=normal(B, T, Hv, V).to(dtype))
    x["g"] = g_scale * torch.nn.functional.logsigmoid(2 * normal(B, T, Hv) + 3) if gates == "token" else \
        -g_scale * torch.rand(Hv, device="cuda", generator=gen)
    x["initial_state"] = normal(N, Hv, K, V) if h0 else None
    x["cu_seqlens"] = None
    if lens is not None:
        x["cu_seqlens"] = torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32, device="cuda")
    return x


def bounds(x):
    B, T = x["q"].shape[:2]
    return [T * i for i in range(B + 1)] if x["cu_seqlens"] is None else x["cu_seqlens"].tolist()


def exact(x, do=None, dht=None, scale=None):
    """o, final states and, with do or dht, the gradients, from the recurrence in 64 bits."""
    q, k, v = x["q"].double(), x["k"].double(), x["v"].double()
    B, T, Hq, K = q.shape
    Hv, V = v.shape[2:]
    G = Hv // Hq
    scale = K ** -0.5 if scale is None else scale
    g = x["g"].double().expand(B, T, Hv).reshape(B * T, Hv)
    q, k = (y.repeat_interleave(G, dim=2).reshape(B * T, Hv, K) for y in (q, k))
    v = v.reshape(B * T, Hv, V)
    b = bounds(x)
    o = torch.zeros_like(v)
    hT = torch.zeros(len(b) - 1, Hv, K, V, dtype=torch.float64, device="cuda")
    backward = do is not None or dht is not None
    dq, dk, dv, dg, dh0 = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(g), torch.zeros_like(hT)
    do = torch.zeros_like(v) if do is None else do.double().reshape(B * T, Hv, V)
    for j in range(len(b) - 1):
        h = hT[j].clone() if x["initial_state"] is None else x["initial_state"][j].double()
        before = []
        for t in range(b[j], b[j + 1]):
            before.append(h)
            h = h * g[t].exp()[:, None, None] + k[t][:, :, None] * v[t][:, None]
            o[t] = scale * (q[t][:, :, None] * h).sum(1)
            dq[t] = scale * (h * do[t][:, None]).sum(2)
        hT[j] = h
        if not backward:
            continue
        dh = torch.zeros_like(h) if dht is None else dht[j].double()
        for t in reversed(range(b[j], b[j + 1])):
            dh = dh + scale * q[t][:, :, None] * do[t][:, None]
            dk[t] = (dh * v[t][:, None]).sum(2)
            dv[t] = (dh * k[t][:, :, None]).sum(1)
            dh = dh * g[t].exp()[:, None, None]
            dg[t] = (dh * before.pop()).sum((1, 2))
        dh0[j] = dh
    out = (o.view(B, T, Hv, V), hT)
    if not backward:
        return out
    heads = lambda y: y.view(B, T, Hq, G, K).sum(3)  # noqa: E731
    dg = dg.sum(0) if x["g"].dim() == 1 else dg.view(B, T, Hv)
    terms = max((q * dq).sum(-1).norm().item(), (k * dk).sum(-1).norm().item()) * (math.sqrt(B * T) if x["g"].dim() == 1 else 1)
    return out + (heads(dq), heads(dk), dv.view(B, T, Hv, V), dg, None if x["initial_state"] is None else dh0, terms)


def check(got, want, tol, what, terms=0.0):
    assert got.shape == want.shape, what
    d, n = (got.double() - want).norm().item(), max(want.norm().item(), terms)
    assert math.isfinite(d) and d <= tol * n + 1e-30, "%s: %.3g of %.3g" % (what, d / max(n, 1e-300), tol)


LENGTHS = [1, 2, 63, 64, 65, 127, 200, 1100]


@pytest.mark.parametrize("K,V", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", LENGTHS)
def test_forward(gdr, T, dtype, K, V):
    x = inputs(2, T, 2, 4, K, V, dtype, gates="token" if T % 2 else "head", h0=T != 64, seed=T)
    o, hT = exact(x)
    for out in (BF, F32):
        got, last = gdr.chunk_linear_attention_fwd(**x, output_dtype=out)
        check(got, o, TOL[out], "o")
        check(last, hT, TOL[F32], "final_state")


@pytest.mark.parametrize("K,V", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", LENGTHS)
def test_backward(gdr, T, dtype, K, V):
    group = 1 if T in (2, 65) else 2
    x = inputs(2, T, 2, 2 * group, K, V, dtype, gates="token" if T % 2 else "head", h0=T != 64, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(T)
    do = torch.randn(x["v"].shape, device="cuda", generator=gen).to(dtype)
    dht = None if T == 65 else torch.randn((2, 2 * group, K, V), device="cuda", generator=gen)
    want = exact(x, do, dht)[2:]
    for grad in {dtype, F32}:
        got = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"],
                                             grad_dtype=grad)
        for name, a, b in zip(("dq", "dk", "dv"), got, want):
            check(a, b, TOL[grad], name)
        check(got[3], want[3], TOL_GATES, "dg", want[5])
        if want[4] is not None:
            check(got[4], want[4], TOL[F32], "dh0")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("lens", [[5, 0, 700, 64, 1, 0], [1], [0, 0], [0, 3000], [64] * 40])
def test_packed(gdr, lens, K, V, dtype):
    x = inputs(1, sum(lens), 2, 4, K, V, dtype, h0=True, lens=lens, seed=len(lens))
    do = torch.randn(x["v"].shape, device="cuda").to(dtype)
    dht = torch.randn(x["initial_state"].shape, device="cuda")
    o, hT, *want = exact(x, do, dht)
    got, last = gdr.chunk_linear_attention_fwd(**x, output_dtype=dtype)
    check(got, o, TOL[dtype], "o")
    check(last, hT, TOL[F32], "final_state")
    grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"], x["cu_seqlens"])
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dh0"), grads, want, [TOL[dtype]] * 3 + [TOL_GATES, TOL[F32]]):
        check(a, b, tol, name, want[5] if name == "dg" else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("segment", [1, 2, 5, 16, 1000])
def test_segments(gdr, segment, dtype):
    """Any split gives the same results."""
    lens = [700, 64, 1300, 3]
    x = inputs(1, sum(lens), 1, 2, 64, 128, dtype, h0=True, lens=lens)
    do = torch.randn(x["v"].shape, device="cuda").to(dtype)
    dht = torch.randn(x["initial_state"].shape, device="cuda")
    o, hT, *want = exact(x, do, dht)
    got, last = gdr.chunk_linear_attention_fwd(**x, segment_chunks=segment)
    check(got, o, TOL[F32], "o")
    check(last, hT, TOL[F32], "final_state")
    grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"],
                                           x["cu_seqlens"], segment_chunks=segment)
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dh0"), grads, want, [TOL[dtype]] * 3 + [TOL_GATES, TOL[F32]]):
        check(a, b, tol, name, want[5] if name == "dg" else 0.0)


@pytest.mark.parametrize("N", [1, 3, 40])
@pytest.mark.parametrize("group", [1, 3])
def test_heads(gdr, N, group):
    for Hq in (1, 5):
        x = inputs(N, 130, Hq, group * Hq, 64, 64, BF)
        do = torch.randn(x["v"].shape, device="cuda").to(BF)
        o, hT, *want = exact(x, do)
        got, _ = gdr.chunk_linear_attention_fwd(**x, output_dtype=BF)
        check(got, o, TOL[BF], "o")
        for a, b, tol, terms in zip(gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do), want,
                                    [TOL[BF]] * 3 + [TOL_GATES], [0, 0, 0, want[5]]):
            check(a, b, tol, "gradient", terms)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gates(gdr, dtype):
    """No decay, growth, decays that leave nothing of the last chunk, gates that empty the state."""
    for kind in ("none", "grow", "strong", "resets", "all"):
        x = inputs(1, 300, 1, 2, 64, 64, dtype, h0=True)
        g = x["g"]
        if kind == "none":
            g.zero_()
        elif kind == "grow":
            g.copy_(0.02 * torch.rand(g.shape, device="cuda"))
        elif kind == "strong":
            g.copy_(-5 * torch.rand(g.shape, device="cuda"))
        elif kind == "resets":
            g[0, torch.tensor([0, 17, 64, 65, 200]).cuda()] = torch.tensor([-math.inf, -1e38, -104, -200, -math.inf],
                                                                          device="cuda")[:, None]
        else:
            g.fill_(-math.inf)
        do = torch.randn(x["v"].shape, device="cuda").to(dtype)
        dht = torch.randn(x["initial_state"].shape, device="cuda")
        y = dict(x, g=g.clamp(min=-1000))  # (e^-1000 is 0 in 64 bits; 0 times infinity is not met)
        o, hT, *want = exact(y, do, dht)
        got, last = gdr.chunk_linear_attention_fwd(**x)
        # sums of gates to 104 within 16 tokens are rounded by 2^-18
        worse = 8 if kind in ("resets", "strong") else 1
        check(got, o, worse * TOL[F32], "o")
        check(last, hT, worse * TOL[F32], "final_state")
        grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"])
        for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dh0"), grads, want,
                                   [TOL[dtype] + worse * 2.0 ** -18] * 3 + [TOL_GATES, worse * TOL[F32]]):
            check(a, b, tol, name, want[5] if name == "dg" else 0.0)


def test_rows_read_in_place(gdr):
    """Slices of one projection, transposed batches, rows that have to be copied."""
    Hq, Hv, K, V = 2, 4, 64, 128
    wide = torch.randn(3, 150, 2 * Hq * K + Hv * V + 8, device="cuda").to(BF)
    cut = lambda w, at, H, D: w[..., at:at + H * D].unflatten(-1, (H, D))  # noqa: E731
    for w, off in ((wide, 0), (wide, 8), (wide, 1), (wide.transpose(0, 1).contiguous().transpose(0, 1), 0)):
        x = inputs(3, 150, Hq, Hv, K, V, BF)
        x.update(q=cut(w, off, Hq, K), k=cut(w, off + Hq * K, Hq, K), v=cut(w, off + 2 * Hq * K, Hv, V) if off < 8 else
                 cut(w, 8 + 2 * Hq * K, Hv, V))
        do = torch.randn(3, 150, Hv, V, device="cuda").to(BF)
        o, hT, *want = exact(x, do)
        got, last = gdr.chunk_linear_attention_fwd(**x, output_dtype=BF)
        check(got, o, TOL[BF], "o")
        for a, b in zip(gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do)[:3], want):
            check(a, b, TOL[BF], "gradient")
    # one head's rows for all heads, one row for all tokens
    x = inputs(2, 70, 2, 2, 64, 64, BF)
    x["k"], x["v"] = x["k"][:, :, :1].expand(-1, -1, 2, -1), x["v"][:, :1].expand(-1, 70, -1, -1)
    check(gdr.chunk_linear_attention_fwd(**x)[0], exact(x)[0], TOL[F32], "o")


def test_autograd(gdr):
    for out, dtype, per_head in ((BF, BF, True), (F32, BF, False), (F32, F32, True)):
        x = inputs(2, 100, 2, 4, 64, 64, dtype, gates="head" if per_head else "token", h0=True)
        leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "g", "initial_state")]
        o, hT = gdr.chunk_linear_attention(**x, output_final_state=True, output_dtype=out)
        do, dht = torch.randn(o.shape, device="cuda").to(out), torch.randn(hT.shape, device="cuda")
        detached = {n: t if t is None or n == "cu_seqlens" else t.detach() for n, t in x.items()}
        want = exact(detached, do, dht)
        check(o.detach(), want[0], TOL[out], "o")
        tols, terms = [TOL[dtype]] * 3 + [TOL_GATES, TOL[F32]], lambda w: [0, 0, 0, w[-1], 0]  # noqa: E731
        for a, b, leaf, tol, t in zip(torch.autograd.grad([o, hT], leaves, [do, dht]), want[2:], leaves, tols, terms(want)):
            assert a.dtype == leaf.dtype
            check(a, b, tol, "gradient", t)
        # of the final state alone, and an expanded gradient of o
        o, hT = gdr.chunk_linear_attention(**x, output_final_state=True, output_dtype=out)
        want = exact(detached, None, dht)[2:]
        grads = torch.autograd.grad(hT, leaves, dht, allow_unused=True)
        for a, b, tol, t in zip(grads[1:], want[1:], tols[1:], terms(want)[1:]):
            check(a, b, tol, "gradient", t)
        assert not grads[0].any()
        o, none = gdr.chunk_linear_attention(**x, output_dtype=out)
        assert none is None
        want = exact(detached, torch.ones(o.shape, device="cuda"))[2:]
        for a, b, tol, t in zip(torch.autograd.grad(o.sum(), leaves), want, tols, terms(want)):
            check(a, b, tol, "gradient", t)


def test_gradients_are_differences(gdr):
    x = inputs(1, 90, 1, 2, 64, 64, F32, h0=True)
    do, dht = torch.randn(1, 90, 2, 64, device="cuda"), torch.randn(1, 2, 64, 64, device="cuda")
    grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"])
    for name, grad in zip(("q", "k", "v", "g", "initial_state"), grads):
        step = torch.randn(x[name].shape, device="cuda", dtype=torch.float64)
        value = []
        for e in (1e-4, -1e-4):  # central differences in 64 bits, off by about 1e-8 of the third derivative
            o, hT = exact(dict(x, **{name: x[name].double() + e * step}))
            value.append((o * do.double()).sum() + (hT * dht.double()).sum())
        d = (value[0] - value[1]) / 2e-4
        assert abs((grad.double() * step).sum() - d) <= 1e-4 * grad.double().norm() * step.norm(), name


def test_values_that_are_not_finite_stay_in_their_sequence_and_head(gdr):
    lens = [100, 30, 200]
    x = inputs(1, sum(lens), 2, 4, 64, 64, BF, lens=lens)
    clean, last = gdr.chunk_linear_attention_fwd(**x)
    for name in ("q", "k", "v"):
        y = dict(x, **{name: x[name].clone()})
        y[name][0, 105, 1] = math.nan
        got, hT = gdr.chunk_linear_attention_fwd(**y)
        heads = slice(2, 4) if name != "v" else slice(1, 2)
        for t in (got, clean):
            t.view(-1, 4, 64)[100:130, heads] = 0
        assert torch.equal(got, clean)
        keep = torch.ones(3, 4, dtype=torch.bool)
        keep[1, heads] = False
        assert torch.equal(hT[keep.cuda()], last[keep.cuda()])
        clean, last = gdr.chunk_linear_attention_fwd(**x)


def test_bad_offsets_stay_in_bounds(gdr):
    """Offsets on the device are not read on the host: out-of-range ones are clamped."""
    x = inputs(1, 200, 1, 2, 64, 64, BF, lens=[100, 100], h0=True)
    for offsets, good in (([0, 100, 10 ** 6], [0, 100, 200]), ([-5, 100, 200], [0, 100, 200]), ([0, 300, 200], [0, 200, 200]),
                          ([50, 20, 200], [50, 50, 200])):
        bad = dict(x, cu_seqlens=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        o, hT = gdr.chunk_linear_attention_fwd(**bad)
        if offsets[1] == 100:
            want, last = gdr.chunk_linear_attention_fwd(**x)
            assert torch.equal(o, want) and torch.equal(hT, last)
        gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], torch.zeros_like(x["v"]), None, None,
                                       x["initial_state"], bad["cu_seqlens"])
    torch.cuda.synchronize()


def test_rows_behind_the_last_sequence_are_left(gdr):
    """With the C interface's own buffers: rows of no sequence keep what they held."""
    from gated_delta_rule_85_amd import _lib
    T, H, K, V = 200, 2, 64, 64
    x = inputs(1, T, H, H, K, V, BF)
    cu = torch.tensor([10, 60, 130], dtype=torch.int32, device="cuda")
    o = torch.full((1, T, H, V), 7.0, device="cuda")
    a = _lib.LaFwdArgs()
    a.B, a.T, a.H_q, a.H_v, a.K, a.V, a.n_seq = 1, T, H, H, K, V, 2
    a.q_row = a.k_row = H * K
    a.v_row, a.dtype, a.out_dtype, a.scale, a.segment_chunks = H * V, _lib.BF16, _lib.F32, 1.0, 1000
    a.q, a.k, a.v, a.g, a.cu_seqlens, a.o = (t.data_ptr() for t in (x["q"], x["k"], x["v"], x["g"], cu, o))
    _lib.la_fwd(a, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert (o[:, :10] == 7).all() and (o[:, 130:] == 7).all()
    y = {n: t[:, 10:130] for n, t in x.items() if n in ("q", "k", "v", "g")}
    y.update(initial_state=None, cu_seqlens=torch.tensor([0, 50, 120], dtype=torch.int32, device="cuda"))
    check(o[:, 10:130], exact(y, scale=1.0)[0], TOL[F32], "o")


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype,Hq,Hv", [(BF, 2, 4), (BF, 2, 2), (F32, 1, 3)])
@pytest.mark.parametrize("cu", [[0, 100, 130], [7, 90, 90, 200], [40, 40], [200], [0, 256], [255, 256]])
def test_padded_rows_are_zero(gdr, cu, dtype, Hq, Hv, per_head):
    """Rows of no sequence: whatever they hold, o and the gradients are zero there, and the others' are
    those of the sequences alone."""
    T, K, V = 256, 64, 128
    x = inputs(1, T, Hq, Hv, K, V, dtype, gates="head" if per_head else "token")
    first, end = (cu[0], cu[-1]) if len(cu) > 1 else (0, 0)
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[first:end] = False
    leaves = {n: x[n].clone() for n in ("q", "k", "v", "g")}
    for n in ("q", "k", "v") if per_head else ("q", "k", "v", "g"):
        leaves[n][:, rest] = math.nan
    do = torch.randn(1, T, Hv, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5)).to(dtype)
    pads = do.clone()
    pads[:, rest] = math.nan
    for t in leaves.values():
        t.requires_grad_()
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    junk = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(4)]  # what the allocator hands out next
    torch.cuda.synchronize()
    del junk
    o, _ = gdr.chunk_linear_attention(**leaves, cu_seqlens=offsets, output_dtype=dtype)
    assert (o[:, rest] == 0).all()
    o.backward(pads)
    assert all((leaves[n].grad[:, rest] == 0).all() for n in ("q", "k", "v"))
    assert per_head or (leaves["g"].grad[:, rest] == 0).all()
    if end == first:
        assert all((t.grad == 0).all() for t in leaves.values())
        return
    alone = {n: (t if n == "g" and per_head else t[:, first:end]).clone().requires_grad_() for n, t in x.items()
             if n in ("q", "k", "v", "g")}
    want, _ = gdr.chunk_linear_attention(**alone, cu_seqlens=offsets - first, output_dtype=dtype)
    want.backward(do[:, first:end])
    # both are off by the tolerances of the exact result (segments may start elsewhere)
    check(o[:, first:end], want.double(), 2 * TOL[dtype], "o")
    along = (alone["q"] * alone["q"].grad).double().sum(-1)
    terms = along.abs().sum(1).norm().item() if per_head else along.norm().item()
    for n, t in alone.items():
        got = leaves[n].grad if n == "g" and per_head else leaves[n].grad[:, first:end]
        check(got, t.grad.double(), 2 * (TOL_GATES if n == "g" else TOL[dtype]), n, terms if n == "g" else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K,V", [(128, 128), (128, 64), (64, 128), (64, 64)])
@pytest.mark.parametrize("N,T", [(1, 1), (5, 1), (33, 3), (2, 9)])
def test_step(gdr, N, T, K, V, dtype):
    for gates in ("token", "head"):
        x = inputs(N, T, 2, 4, K, V, dtype, gates=gates, h0=True)
        pool = torch.randn(N + 3, 4, K, V, device="cuda")
        slots = torch.randperm(N + 3)[:N].int().cuda()
        pool[slots.long()] = x["initial_state"]
        o, hT = exact(x)
        want = pool.double()
        want[slots.long()] = hT
        for out in (BF, F32):
            states = pool.clone()
            got = gdr.recurrent_linear_attention(x["q"], x["k"], x["v"], x["g"], states, slots=slots, output_dtype=out)
            check(got, o, TOL[out], "o")
            check(states, want, TOL[F32], "states")


def test_step_of_packed_padded_and_repeated_sequences(gdr):
    lens = [1, 4, 0, 2, 3]
    x = inputs(1, sum(lens), 2, 2, 64, 128, BF, lens=lens, h0=True)
    pool = torch.randn(6, 2, 64, 128, device="cuda")
    slots = torch.tensor([3, -1, 0, 5, 3], dtype=torch.int32, device="cuda")  # the second pads, the last repeats
    x["initial_state"] = pool[slots.clamp(min=0).long()]
    o, hT = exact(x)
    states, out = pool.clone(), torch.full((1, 10, 2, 128), 9.0, device="cuda")
    got = gdr.recurrent_linear_attention(x["q"], x["k"], x["v"], x["g"], states, cu_seqlens=x["cu_seqlens"], slots=slots, out=out)
    assert got is out or got.data_ptr() == out.data_ptr()
    check(got[:, :1], o[:, :1], TOL[F32], "o")
    check(got[:, 5:7], o[:, 5:7], TOL[F32], "o")
    assert not got[:, 1:5].any() and not got[:, 7:].any()
    want = pool.double()
    want[3], want[5] = hT[0], hT[3]
    check(states, want, TOL[F32], "states")
    keep = [0, 1, 2, 4]
    assert torch.equal(states[keep], pool[keep])


def test_a_layer_trained_and_served(gdr):
    """Prompts through the chunked form and the norm, their states into a pool, tokens from there on
    through the recurrent form: the same rows as one pass over the whole sequences."""
    Hq, Hv, K, V, lens, more = 2, 4, 128, 64, [70, 1, 130], 5
    whole = [n + more for n in lens]
    x = inputs(1, sum(whole), Hq, Hv, K, V, BF, gates="head", lens=whole)
    w = 1 + 0.1 * torch.randn(Hv * V, device="cuda")
    gate = torch.randn(1, sum(whole), Hv * V, device="cuda").to(BF)
    o, hT = gdr.chunk_linear_attention_fwd(**x)
    y = gdr.group_norm(o.flatten(2), Hv, w, gate=gate)
    at = bounds(x)
    pick = lambda t, n0, n1: torch.cat([t[:, a + n0(i):a + n1(i)] for i, a in enumerate(at[:-1])], 1)  # noqa: E731
    first = lambda t: pick(t, lambda i: 0, lambda i: lens[i])  # noqa: E731
    cu = torch.tensor([0] + list(itertools.accumulate(lens)), dtype=torch.int32, device="cuda")
    po, states = gdr.chunk_linear_attention(first(x["q"]), first(x["k"]), first(x["v"]), x["g"], cu_seqlens=cu,
                                            output_final_state=True)
    pool = torch.zeros(7, Hv, K, V, device="cuda")
    slots = torch.tensor([4, 0, 6], dtype=torch.int32, device="cuda")
    gdr.copy_states(pool, slots, torch.arange(3, dtype=torch.int32, device="cuda"), states)
    got = gdr.group_norm(po.flatten(2), Hv, w, gate=first(gate))
    check(got, first(y).double(), 2 * TOL[BF], "prompt")
    for i in range(more):
        token = lambda t: torch.stack([t[0, a + n + i] for a, n in zip(at, lens)])[:, None]  # noqa: E731
        so = gdr.recurrent_linear_attention(token(x["q"]), token(x["k"]), token(x["v"]), x["g"], pool, slots=slots)
        check(gdr.group_norm(so.flatten(2), Hv, w, gate=token(gate)), token(y).double(), 2 * TOL[BF], "token")
    check(pool[slots.long()], hT.double(), TOL[F32], "states")
    # trained: gradients through both operators
    leaves = [x[n].requires_grad_() for n in ("q", "k", "v", "g")] + [gate.requires_grad_(), w.requires_grad_()]
    o, _ = gdr.chunk_linear_attention(**x, output_dtype=BF)
    z = gdr.group_norm(o.flatten(2), Hv, w, gate=gate)
    dz = torch.randn(z.shape, device="cuda").to(BF)
    grads = torch.autograd.grad(z, leaves, dz)
    ref = [t.detach().double().requires_grad_() for t in leaves]
    ox = torch.cat([_plain(ref[0][:, a:b], ref[1][:, a:b], ref[2][:, a:b], ref[3]) for a, b in zip(at, at[1:])], 1)
    n = torch.nn.functional.layer_norm(ox, (V,)).flatten(2) * ref[5]
    want = torch.autograd.grad(n * torch.nn.functional.silu(ref[4]), ref, dz.double())
    for a, b in zip(grads, want):  # o, its gradient and the result are rounded to bf16
        check(a, b, 4 * TOL[BF], "gradient")


def _plain(q, k, v, g):
    """One sequence with a fixed decay per head, as a masked product (64 bits, differentiable)."""
    T, G = q.shape[1], v.shape[2] // q.shape[2]
    q, k = (y.repeat_interleave(G, 2).transpose(1, 2) for y in (q, k))
    d = torch.arange(T, device="cuda")[:, None] - torch.arange(T, device="cuda")
    p = (q @ k.transpose(-1, -2)) * torch.where(d >= 0, torch.exp(g[:, None, None] * d.clamp(min=0)), 0.0) / q.shape[-1] ** 0.5
    return (p @ v.transpose(1, 2)).transpose(1, 2)


def test_streams_graphs_and_repeats(gdr):
    """Captured with other calls' workspaces alive, replayed with eager work between."""
    x = inputs(1, 5000, 1, 2, 64, 64, BF, h0=True)  # long enough to be split
    do = torch.randn(x["v"].shape, device="cuda").to(BF)

    def both():
        o, hT = gdr.chunk_linear_attention_fwd(**x)
        return (o, hT, *gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, hT, None, x["initial_state"]))

    want = both()
    assert all(torch.equal(a, b) for a, b in zip(want, both()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    kept = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            kept.append(both())
    for seed in range(3):
        x["v"].copy_(inputs(1, 5000, 1, 2, 64, 64, BF, seed=seed)["v"])
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        fresh = both()
        for k in kept:
            assert all(torch.equal(a, b) for a, b in zip(fresh, k))


@pytest.mark.parametrize("N", [65, 300, 5000])
def test_many_packed_sequences_split(gdr, N):
    """The segments of more sequences than a wave has lanes, empty and long ones among them: split and
    unsplit scans are both off by the tolerances of the exact result."""
    gen = torch.Generator().manual_seed(N)
    lens = torch.randint(0, 4, (N,), generator=gen)
    for i in (0, 1, N // 2, N // 2 + 3, N - 1):
        lens[i] = 130 + 65 * (i % 3)
    T, H, K, V = int(lens.sum()) + 9, 2, 64, 64  # (and rows behind the last one)
    x = inputs(1, T, 1, H, K, V, BF, lens=lens.tolist(), h0=True)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(device="cuda", dtype=torch.int32)
    do = torch.randn(1, T, H, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(BF)
    dht = torch.randn(N, H, K, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(2))
    runs = []
    for segment in (1, 2, 1 << 20):
        o, hT = gdr.chunk_linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], None, x["initial_state"], cu,
                                               segment_chunks=segment)
        grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"], cu,
                                               segment_chunks=segment)
        runs.append((o, hT) + grads)
    terms = (x["q"].double() * runs[-1][2].double()).sum(-1).norm().item()
    for run in runs[:-1]:
        for name, got, want in zip(("o", "hT", "dq", "dk", "dv", "dg", "dh0"), run, runs[-1]):
            tol = TOL_GATES if name == "dg" else TOL[BF] if got.dtype == BF else TOL[F32]
            check(got, want.double(), 2 * tol, name, terms if name == "dg" else 0.0)


def test_offsets_past_32_bits(gdr):
    """v, o and do of 2.5e9 elements: a sequence at the end is as it is alone."""
    T, first, H, K, V = 300000, 299000, 64, 64, 128
    x = inputs(1, T, 32, H, K, V, BF)
    do = torch.randn(T - first, H * V, device="cuda").to(BF).view(1, -1, H, V)
    whole = torch.zeros(1, T, H, V, dtype=BF, device="cuda")
    whole[:, first:] = do
    cu = torch.tensor([0, first, T], dtype=torch.int32, device="cuda")
    leaves = [x[n] for n in ("q", "k", "v", "g")]
    alone = [t[:, first:].contiguous() for t in leaves]
    want, _ = gdr.chunk_linear_attention_fwd(*alone, output_dtype=BF)
    got, _ = gdr.chunk_linear_attention_fwd(*leaves, cu_seqlens=cu, output_dtype=BF)
    check(got[:, first:], want.double(), 2 * TOL[BF], "o")
    del got
    want = gdr.chunk_linear_attention_bwd(*alone, do)
    got = gdr.chunk_linear_attention_bwd(*leaves, whole, cu_seqlens=cu)
    for name, a, b in zip(("dq", "dk", "dv"), got, want):
        check(a[:, first:], b.double(), 2 * TOL[BF], name)
        assert (a[:, :first] == 0).all(), name  # (nothing reaches another sequence)
    terms = (alone[0].double() * want[0].double()).sum(-1).norm().item()
    check(got[3][:, first:], want[3].double(), 2 * TOL_GATES, "dg", terms)


def _resets(T, n, closed, seed):
    """Gates of T tokens of which n close at the start of every 16 and two more anywhere."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.nn.functional.logsigmoid(2 * torch.randn(1, T, 2, device="cuda", generator=gen) + 3)
    g[:, torch.arange(T, device="cuda") % 16 < n] = closed
    g[:, torch.randint(T, (2,), device="cuda", generator=gen)] = closed
    return g


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("closed", [-math.inf, -104.0, -60.0, -5.0])
@pytest.mark.parametrize("n", [0, 1, 4, 8])
def test_decays_between_tokens(gdr, n, closed, dtype):
    """Keys and values of a single one read the decay from every token to every later one out of o, and
    to the end out of the state.  Its error is relative to the gates between the two, whatever came
    before them: their sum S is made of at most twelve roundings, each 2^-24 of S at most, and what is
    made of it goes through fewer than sixteen more."""
    T = 128
    one = torch.eye(T, device="cuda").to(dtype).view(1, T, 1, T)
    g = _resets(T, n, closed, seed=n)
    total = g[0].double().clamp(min=-1000).cumsum(0)
    o, hT = gdr.chunk_linear_attention_fwd(torch.ones_like(one), one, one.expand(1, T, 2, T), g, 1.0)
    between = total[:, None] - total[None]  # [t, i, head]
    got = o[0].transpose(1, 2).double()
    past = torch.ones(T, T, dtype=torch.bool, device="cuda").tril()[:, :, None]
    for got, between in ((got.where(past, 0), between.where(past, -math.inf)),
                         (hT[0].diagonal(dim1=1, dim2=2).T.double(), between[-1])):
        off = (got - between.exp()).abs()
        tol = 2.0 ** -24 * (16 + 16 * between.abs().nan_to_num(posinf=0)) * between.exp() + 2.0 ** -120
        assert (off <= tol).all(), "%.3g times the tolerance" % (off / tol).max()
    assert not o[0].transpose(1, 2).where(past, 0).isnan().any() and not (o[0].transpose(1, 2) * ~past).any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [1, 4, 8])
def test_gradients_behind_resets(gdr, n, dtype):
    """Gates that empty the state do not make what follows them less precise."""
    x = inputs(1, 300, 1, 2, 64, 128, dtype, h0=True)
    x["g"] = _resets(300, n, -math.inf, seed=n)
    do = torch.randn(x["v"].shape, device="cuda").to(dtype)
    dht = torch.randn(x["initial_state"].shape, device="cuda")
    o, hT, *want = exact(dict(x, g=x["g"].clamp(min=-1000)), do, dht)
    got, last = gdr.chunk_linear_attention_fwd(**x)
    check(got, o, TOL[F32], "o")
    check(last, hT, TOL[F32], "final_state")
    grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"], grad_dtype=F32)
    for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dh0"), grads, want, [TOL[F32]] * 3 + [TOL_GATES, TOL[F32]]):
        check(a, b, tol, name, want[5] if name == "dg" else 0.0)


@pytest.mark.parametrize("kind", ["past the end", "before the start", "falls", "falls within", "long", "64", "80", "1500"])
def test_offsets_on_the_device_are_made_to_rise(gdr, kind):
    """Offsets outside [0, T], or smaller than one before them, give what the offsets give that they are
    taken as: no sequence shares a row with another, and rows of none are zero."""
    T, K, V = 200, 64, 128
    if kind in ("64", "80", "1500"):
        T = 3000
        offsets = torch.randint(-50, T + 50, (int(kind) + 1,), generator=torch.Generator().manual_seed(int(kind)))
        rising = (torch.arange(len(offsets)) * T / len(offsets)).long()
        mixed = torch.rand(len(offsets), generator=torch.Generator().manual_seed(1)) < 0.1
        offsets = torch.where(mixed, offsets.clamp(max=T // 2), rising).tolist()
    else:
        offsets = {"past the end": [0, 300, 200], "before the start": [-5, 100, 10 ** 6], "falls": [50, 20, 200],
                   "falls within": [0, 100, 50, 180, 150], "long": [7, 1500, 700, 2900, 100, 2901]}[kind]
        T = 3000 if kind == "long" else T
    good = list(itertools.accumulate((min(max(i, 0), T) for i in offsets), max))
    N = len(good) - 1
    x = inputs(1, T, 1, 2, K, V, BF)
    gen = torch.Generator(device="cuda").manual_seed(3)
    h0, dht = (torch.randn(N, 2, K, V, device="cuda", generator=gen) for _ in range(2))
    do = torch.randn(1, T, 2, V, device="cuda", generator=gen).to(BF)
    runs = []
    for cu in (good, offsets):
        cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        run = []
        for segment in (0, 1, 2, 1 << 20):
            run += gdr.chunk_linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], None, h0, cu, segment_chunks=segment)
            run += gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, h0, cu, segment_chunks=segment)
        torch.cuda.synchronize()
        runs.append(run)
    assert all(torch.equal(a, b) for a, b in zip(*runs))
    names = ["o", "hT", "dq", "dk", "dv", "dg", "dh0"]
    for name, t in zip(itertools.cycle(names), runs[1]):
        assert t.isfinite().all(), name
        if name not in ("hT", "dh0"):
            assert not t[:, :good[0]].any() and not t[:, good[-1]:].any(), name
    # what they are taken as is right
    want = exact(dict(x, initial_state=h0, cu_seqlens=torch.tensor(good)), do, dht)
    for name, got, b in zip(names, runs[1], want):
        check(got, b, TOL_GATES if name == "dg" else TOL[got.dtype], name, want[7] if name == "dg" else 0.0)


def test_many_sequences_and_heads(gdr):
    """640000 (sequence, head) pairs, most of them of one token: long sequences among them are bit for bit
    what they are alone, and single tokens what their products are."""
    N, long, H, K = 40000, 700, 16, 64
    lens = torch.ones(N, dtype=torch.int64)
    lens[[5, N - 2]] = long
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
    T = int(cu[-1])
    x = inputs(1, T, H, H, K, K, BF)
    do = torch.randn(1, T, H, K, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)).to(BF)
    leaves = [x[n] for n in ("q", "k", "v", "g")]
    offsets = cu.to(device="cuda", dtype=torch.int32)
    for segment in (2, 1 << 20):
        o, _ = gdr.chunk_linear_attention_fwd(*leaves, None, None, offsets, False, segment_chunks=segment)
        grads = gdr.chunk_linear_attention_bwd(*leaves, do, None, None, None, offsets, segment_chunks=segment)
        for j in (5, N - 2):
            at = slice(int(cu[j]), int(cu[j + 1]))
            alone = [t[:, at].contiguous() for t in leaves]
            want = gdr.chunk_linear_attention_fwd(*alone, None, None, None, False, segment_chunks=segment)[:1]
            want += gdr.chunk_linear_attention_bwd(*alone, do[:, at].contiguous(), segment_chunks=segment)
            assert all(torch.equal(a[:, at], b) for a, b in zip((o,) + grads[:4], want[:5]))
        single = torch.ones(T, dtype=torch.bool)
        single[cu[5]:cu[6]] = single[cu[N - 2]:cu[N - 1]] = False
        q, k, v, d = (t[0, single.cuda()].double() for t in (x["q"], x["k"], x["v"], do))
        qk, vd = K ** -0.5 * (q * k).sum(-1, keepdim=True), K ** -0.5 * (v * d).sum(-1, keepdim=True)
        for got, want, tol in zip((o,) + grads, (qk * v, vd * k, vd * q, qk * d), (TOL[F32], TOL[BF], TOL[BF], TOL[BF])):
            check(got[0, single.cuda()], want, tol, "single tokens")
        # (no state before them: nothing depends on their gates)
        assert grads[3][0, single.cuda()].abs().max() <= TOL_GATES * (q * k).sum(-1).abs().max() * (v * d).sum(-1).abs().max()


@pytest.mark.parametrize("K,V", [(128, 128), (64, 128), (128, 64)])
@pytest.mark.parametrize("N,T,Hq,Hv,segment", [(16, 131, 16, 16, 0), (32, 70, 4, 8, 0), (1, 4100, 2, 4, 1), (3, 700, 8, 8, 1)])
def test_full_device(gdr, N, T, Hq, Hv, segment, K, V):
    """256 and more (sequence or segment, head) pairs: a workgroup takes 128 columns."""
    x = inputs(N, T, Hq, Hv, K, V, BF, h0=True, seed=T)
    gen = torch.Generator(device="cuda").manual_seed(T)
    do = torch.randn(x["v"].shape, device="cuda", generator=gen).to(BF)
    dht = torch.randn(x["initial_state"].shape, device="cuda", generator=gen)
    o, hT, *want = exact(x, do, dht)
    for out in (BF, F32):
        got, last = gdr.chunk_linear_attention_fwd(**x, output_dtype=out, segment_chunks=segment)
        check(got, o, TOL[out], "o")
        check(last, hT, TOL[F32], "final_state")
    for grad in (BF, F32):
        grads = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, x["initial_state"],
                                               grad_dtype=grad, segment_chunks=segment)
        for name, a, b, tol in zip(("dq", "dk", "dv", "dg", "dh0"), grads, want, [TOL[grad]] * 3 + [TOL_GATES, TOL[F32]]):
            check(a, b, tol, name, want[5] if name == "dg" else 0.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_gate_gradients_over_long_segments(gdr, dtype):
    """Between two borders 1024 tokens apart a gate's gradient is a sum of differences a - b of two dots, tied at
    both ends.  A dot goes through about twelve roundings, each 2^-24 / sqrt(3) of it in the mean square, 2^-23 in
    all; a sum of n such differences that ends where it should is off by sqrt(2) sqrt(n / 6) of that in the mean.
    With fp32 operands the matrix instruction adds one product after the other, so that a sum of 128 goes through
    128 roundings of its parts so far, whose mean squares are i / 128 of one of the whole: 64 of those for the
    scores and 64 for what is made with the state, 140 in place of 12."""
    x = inputs(2, 4096, 2, 4, 128, 128, dtype, seed=11)
    do = torch.randn(x["v"].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(12)).to(dtype)
    want = exact(x, do)[2:]
    got = gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, segment_chunks=16)
    d = (got[3].double() - want[3]).norm().item()
    tol = 2.0 ** -24 * math.sqrt((12 if dtype == BF else 140) / 3) * math.sqrt(2 * 1024 / 6) * want[5]
    assert d <= tol, "%.3g of %.3g" % (d, tol)


@pytest.mark.parametrize("N", [5, 80])
def test_replays_read_the_offsets_again(gdr, N):
    """Captured with one batch's offsets, replayed with others' in the same tensor, some of them falling."""
    T, K, V = 2000, 64, 128
    x = inputs(1, T, 1, 2, K, V, BF)
    gen = torch.Generator(device="cuda").manual_seed(4)
    do = torch.randn(1, T, 2, V, device="cuda", generator=gen).to(BF)
    h0, dht = (torch.randn(N, 2, K, V, device="cuda", generator=gen) for _ in range(2))
    cu = torch.linspace(0, T, N + 1).int().cuda()

    def both():
        o, hT = gdr.chunk_linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], None, h0, cu, segment_chunks=3)
        return (o, hT, *gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], do, dht, None, h0, cu, segment_chunks=3))

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = both()
    for seed in range(4):
        new = torch.randint(-10, T + 10, (N + 1,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
        cu.copy_(new if seed == 3 else new.sort()[0])
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(both(), kept))
