"""Linear attention with a decay for each head against its definition, token by token in 64 bits:
the chunked form and its backward.

Tolerances are relative to the 2-norm of the exact result.  A bf16 result is rounded once: at
most 2^-9 relative to a value near the top of its binade and 2^-8 near the bottom, 2^-8 / sqrt(3)
at most in the 2-norm; what is computed before that is off by less than 2^-15 (two bf16 pieces of
an fp32 operand, 2^-17 a term, and fp32 sums).  An fp32 result is a sum of up to 64 + K terms per
chunk of products of fp32 rounding, and a state goes through one rounding per chunk: 2^-24 times
the root of the number of roundings, under 64 for every case here, 2^-18.  Gate gradients are
sums of differences of such values over up to 1024 tokens, each of the size of the result: 2^-24
times the root of 1024 x 128, 2^-15.
"""
import itertools
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TOL = {BF: 2.0 ** -8 / math.sqrt(3) + 2.0 ** -15, F32: 2.0 ** -18}
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
    return out + (heads(dq), heads(dk), dv.view(B, T, Hv, V), dg, None if x["initial_state"] is None else dh0)


def check(got, want, tol, what):
    assert got.shape == want.shape, what
    d, n = (got.double() - want).norm().item(), want.norm().item()
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
        check(got[3], want[3], TOL_GATES, "dg")
        if want[4] is not None:
            check(got[4], want[4], TOL[F32], "dh0")
