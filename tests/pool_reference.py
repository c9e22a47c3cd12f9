"""The operators on a pool of states in 64 bits, token by token on the host, the
inputs of their tests, and the tolerances.

Tolerances.  With unit k and q, 0 <= beta <= 1 and g <= 0 a token's update does not
enlarge an error of the state.  A product of a row with a state column is a sum
of K terms, whose fp32 error is at most K 2^-24 |k| |h column|; the few other
roundings of a token are counted as 16 more.  So n tokens leave at most
n (K + 16) 2^-24 X in any value, X being the largest norm of a state column or |v| on
the way (one more token's worth for the output's own product), and in the 2-norm
over all values (K + n + 16) 2^-24 of the values' own norm, the errors of different
tokens being as independent as the values.  An output in fewer bits adds its half
step, eps / 2 of the value."""
import torch


def unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def make(N, T, Hq, Hv, K, V, dtype=torch.bfloat16, lens=None, seed=0, extra_slots=2):
    """Inputs on the host: a dict of q, k, v, g, beta, states, slots (a shuffled part of
    the pool) and cu (None without lens)."""
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    cu = None
    B = N
    if lens is not None:
        cu = torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
        N, B, T = len(lens), 1, int(cu[-1])
    return dict(q=unit(r(B, T, Hq, K)).to(dtype), k=unit(r(B, T, Hq, K)).to(dtype), v=r(B, T, Hv, V).to(dtype),
                g=-0.5 * torch.nn.functional.softplus(r(B, T, Hv)), beta=torch.sigmoid(r(B, T, Hv)),
                states=0.1 * r(N + extra_slots, Hv, K, V),
                slots=torch.randperm(N + extra_slots, generator=gen)[:N].to(torch.int32), cu=cu)


def cuda(x):
    return {n: t.cuda() if isinstance(t, torch.Tensor) else t for n, t in x.items()}


def bounds(x):
    B, T = x["k"].shape[:2]
    cu = [T * i for i in range(B + 1)] if x["cu"] is None else x["cu"].tolist()
    return list(zip(cu[:-1], cu[1:]))


class Ref:
    """64-bit token steps over flattened tokens; `X` tracks the largest column norm or |v|."""

    def __init__(self, x, scale=None):
        B, T, Hq, K = x["k"].shape
        self.Hv, self.V = x["v"].shape[2:]
        head = torch.arange(self.Hv) // (self.Hv // Hq)
        flat = lambda t: t.double().reshape((B * T,) + t.shape[2:])  # noqa: E731
        self.q, self.k = flat(x.get("q", x["k"]))[:, head], flat(x["k"])[:, head]
        self.v, self.g, self.beta = flat(x["v"]), flat(x["g"]), flat(x["beta"])
        self.scale = K ** -0.5 if scale is None else scale
        self.o = torch.zeros(B * T, self.Hv, self.V, dtype=torch.float64)
        self.shape = (B, T, self.Hv, self.V)
        self.X = float(self.v.abs().nan_to_num(0, 0, 0).max()) if self.v.numel() else 0.0

    def seen(self, h):
        self.X = max(self.X, float(h.nan_to_num(0, 0, 0).norm(dim=1).max()))
        return h

    def step(self, h, i):
        """Token i from the state h [Hv, K, V]."""
        h = self.seen(h) * self.g[i].exp()[:, None, None]
        u = self.beta[i][:, None] * (self.v[i] - (self.k[i][:, :, None] * h).sum(1))
        h = self.seen(h + self.k[i][:, :, None] * u[:, None, :])
        self.o[i] = self.scale * (self.q[i][:, :, None] * h).sum(1)
        return h


def recurrent(x, scale=None):
    """(o, states, X)"""
    r, states = Ref(x, scale), x["states"].double().clone()
    for j, (b, e) in enumerate(bounds(x)):
        s = int(x["slots"][j])
        for i in range(b, e):
            states[s] = r.step(states[s], i)
    return r.o.view(r.shape), states, r.X


def tree(x, parents, scale=None):
    """(o, X); parents as [B, T]"""
    r, par = Ref(x, scale), parents.reshape(-1).tolist()
    for j, (b, e) in enumerate(bounds(x)):
        after = []
        for i in range(b, e):
            after.append(r.step(after[par[i]] if par[i] >= 0 else x["states"][int(x["slots"][j])].double(), i))
    return r.o.view(r.shape), r.X


def path_of(parents, node):
    p = []
    while node >= 0:
        p.append(node)
        node = parents[node]
    return p[::-1]


def accept(x, parents, accepted):
    """(states, X)"""
    r, par, states = Ref(x), parents.reshape(-1).tolist(), x["states"].double().clone()
    for j, (b, e) in enumerate(bounds(x)):
        s = int(x["slots"][j])
        for i in path_of(par[b:e], int(accepted[j])):
            states[s] = r.step(states[s], b + i)
    return states, r.X


def near(got, want, n, K, X, what=""):
    """got (a device tensor) is as near to want (64 bits) as n tokens of fp32 and got's type allow."""
    half = torch.finfo(got.dtype).eps / 2 if got.dtype != torch.float32 else 0.0
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert bool(torch.isfinite(got).all()), what
    d = (got - want).abs()
    most = (n + 1) * (K + 16) * 2.0 ** -24 * X
    assert bool((d <= half * want.abs() + most).all()), (what, float((d - half * want.abs()).max()), most)
    norm = float(want.norm())
    assert float(d.norm()) <= ((K + n + 16) * 2.0 ** -24 + half) * norm + 1e-30, (what, float(d.norm()) / norm)
