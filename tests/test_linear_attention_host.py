"""Refusals of linear attention and the group norm, and their C interface's checks, without a GPU:
everything here ends before anything is launched."""
import ctypes

import pytest
import torch

import gated_delta_rule_85_amd as gdr
from gated_delta_rule_85_amd import _lib
from test_abi import _struct_offsets_from_c

BF = torch.bfloat16


def inputs():
    return dict(q=torch.randn(2, 3, 2, 64).to(BF), k=torch.randn(2, 3, 2, 64).to(BF), v=torch.randn(2, 3, 4, 128).to(BF),
                g=-torch.rand(2, 3, 4), initial_state=None, cu_seqlens=None)


CHANGES = [
    ("v tokens", lambda x: x.update(v=x["v"][:, :2])),
    ("k shape", lambda x: x.update(k=x["k"][:, :, :1])),
    ("dimensions", lambda x: x.update(q=x["q"][0], k=x["k"][0])),
    ("v dtype", lambda x: x.update(v=x["v"].float())),
    ("fp16", lambda x: x.update(q=x["q"].half(), k=x["k"].half(), v=x["v"].half())),
    ("g shape", lambda x: x.update(g=x["g"][:, :, :2])),
    ("g tokens", lambda x: x.update(g=x["g"][0, :, 0])),
    ("g whole", lambda x: x.update(g=torch.zeros(4, dtype=torch.int64))),
    ("cu with a batch", lambda x: x.update(cu_seqlens=torch.tensor([0, 3], dtype=torch.int32))),
    ("host tensors", lambda x: None),
]


@pytest.mark.parametrize("name,change", CHANGES + [
    ("state shape", lambda x: x.update(initial_state=torch.zeros(1, 4, 64, 128))),
    ("offsets dtype", lambda x: x.update({n: x[n][:1] for n in "qkvg"}, cu_seqlens=torch.tensor([0, 3]))),
    ("offsets' end", lambda x: x.update({n: x[n][:1] for n in "qkvg"}, cu_seqlens=torch.tensor([0, 2], dtype=torch.int32))),
    ("offsets fall", lambda x: x.update({n: x[n][:1] for n in "qkvg"},
                                        cu_seqlens=torch.tensor([0, 2, 1, 3], dtype=torch.int32))),
    ("no offsets", lambda x: x.update({n: x[n][:1] for n in "qkvg"}, cu_seqlens=torch.tensor([], dtype=torch.int32))),
])
def test_chunked_arguments_are_refused(name, change):
    x = inputs()
    change(x)
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention(**x)
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention_fwd(**x)
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["v"], None, None, x["initial_state"], x["cu_seqlens"])
    leaf = dict(x, q=x["q"].requires_grad_())
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention(**leaf)


def test_chunked_types_of_results_are_refused():
    x = inputs()
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention_fwd(x["q"], x["k"], x["v"], x["g"], output_dtype=torch.float16)
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["v"][:, :1])
    with pytest.raises(ValueError):
        gdr.chunk_linear_attention_bwd(x["q"], x["k"], x["v"], x["g"], x["v"], grad_dtype=torch.float16)


@pytest.mark.parametrize("name,change", CHANGES + [
    ("states dtype", lambda x: x.update(states=x["states"].bfloat16())),
    ("states heads", lambda x: x.update(states=x["states"][:, :2])),
    ("too few slots", lambda x: x.update(states=x["states"][:1])),
    ("slots past the pool", lambda x: x.update(slots=torch.tensor([0, 9], dtype=torch.int32))),
    ("a slot twice", lambda x: x.update(slots=torch.tensor([1, 1], dtype=torch.int32))),
    ("out shape", lambda x: x.update(out=torch.zeros(2, 3, 4, 64))),
])
def test_recurrent_arguments_are_refused(name, change):
    x = inputs()
    x.update(states=torch.zeros(5, 4, 64, 128), slots=None, out=None)
    change(x)
    with pytest.raises(ValueError):
        gdr.recurrent_linear_attention(x["q"], x["k"], x["v"], x["g"], x["states"], cu_seqlens=x["cu_seqlens"],
                                       slots=x["slots"], out=x["out"])


def test_recurrent_form_has_no_gradient():
    x = inputs()
    with pytest.raises(ValueError, match="no gradient"):
        gdr.recurrent_linear_attention(x["q"].requires_grad_(), x["k"], x["v"], x["g"], torch.zeros(5, 4, 64, 128))
    with pytest.raises(TypeError):
        gdr.recurrent_linear_attention(x["q"], x["k"], x["v"], None, torch.zeros(5, 4, 64, 128))


@pytest.mark.parametrize("name,change", [
    ("x dtype", lambda a: a.update(x=a["x"].half())),
    ("groups", lambda a: a.update(num_groups=5)),
    ("no groups", lambda a: a.update(num_groups=0)),
    ("negative groups", lambda a: a.update(num_groups=-3)),
    ("weight", lambda a: a.update(weight=torch.ones(11))),
    ("weight whole", lambda a: a.update(weight=torch.ones(12, dtype=torch.int32))),
    ("bias", lambda a: a.update(bias=torch.ones(1, 12))),
    ("gate shape", lambda a: a.update(gate=torch.ones(12))),
    ("gate dtype", lambda a: a.update(gate=torch.ones(4, 12, dtype=torch.float16))),
    ("activation", lambda a: a.update(activation="relu")),
    ("scalar", lambda a: a.update(x=torch.tensor(1.0))),
    ("no channels", lambda a: a.update(x=torch.zeros(4, 0))),
    ("host tensors", lambda a: None),
])
def test_norm_arguments_are_refused(name, change):
    a = dict(x=torch.randn(4, 12), num_groups=3, weight=torch.ones(12), bias=torch.zeros(12), gate=torch.ones(4, 12),
             activation="silu")
    change(a)
    with pytest.raises(ValueError):
        gdr.group_norm(**a)
    if name != "scalar":
        with pytest.raises(ValueError):
            gdr.group_norm_bwd(a["x"], a["num_groups"], a["x"], a["weight"], a["bias"], a["gate"],
                               activation=a["activation"])
    with pytest.raises(ValueError):
        gdr.group_norm(**dict(a, x=a["x"].requires_grad_()))


def test_norm_types_are_refused():
    with pytest.raises(ValueError):
        gdr.group_norm(torch.ones(4, 12), 3, output_dtype=torch.float16)
    with pytest.raises(ValueError):
        gdr.group_norm(torch.ones(4, 12), 3, output_dtype="bf16")
    with pytest.raises(ValueError):
        gdr.group_norm_bwd(torch.ones(4, 12), 3, torch.ones(4, 12).half())
    with pytest.raises(TypeError):
        gdr.group_norm(None, 3)


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as fw
    x = inputs()
    with fw.dual_level():
        x["q"] = fw.make_dual(x["q"], torch.ones_like(x["q"]))
        with pytest.raises((NotImplementedError, RuntimeError, ValueError)):
            gdr.chunk_linear_attention(**x)
        with pytest.raises((NotImplementedError, RuntimeError, ValueError)):
            gdr.group_norm(fw.make_dual(torch.ones(4, 12), torch.ones(4, 12)), 3)


# ---------------------------------------------------------------- the C interface
@pytest.mark.parametrize("st,name", [(_lib.LaFwdArgs, "gdr_la_fwd_args"), (_lib.LaBwdArgs, "gdr_la_bwd_args"),
                                     (_lib.NormFwdArgs, "gdr_norm_fwd_args"), (_lib.NormBwdArgs, "gdr_norm_bwd_args")])
def test_struct_layouts_match_the_header(tmp_path, st, name):
    names = [f[0] for f in st._fields_]
    c = _struct_offsets_from_c(tmp_path, name, names)
    assert c["size"] == ctypes.sizeof(st)
    for n in names:
        assert c[n] == getattr(st, n).offset, n


def la_args(st, **kw):
    a = st()
    a.B, a.T, a.H_q, a.H_v, a.K, a.V, a.dtype, a.scale = 2, 300, 2, 4, 128, 64, _lib.BF16, 1.0
    a.q_row = a.k_row = 256
    a.v_row = 256
    a.q_batch = a.k_batch = a.v_batch = 300 * 256
    for n in (f for f in ("q", "k", "v", "g", "o", "dout", "dq", "dk", "dv", "dg") if hasattr(a, f)):
        setattr(a, n, 64)  # (never read here)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


BAD = [(dict(H_v=3), _lib.EINVAL), (dict(K=96), _lib.ENOTSUP), (dict(V=32), _lib.ENOTSUP), (dict(dtype=7), _lib.ENOTSUP),
       (dict(B=-1), _lib.EINVAL), (dict(T=-1), _lib.EINVAL), (dict(H_q=0), _lib.EINVAL), (dict(H_v=1 << 16), _lib.EINVAL),
       (dict(cu_seqlens=64, n_seq=2), _lib.EINVAL), (dict(cu_seqlens=64, B=1, n_seq=-1), _lib.EINVAL),
       (dict(segment_chunks=-1), _lib.EINVAL), (dict(q_row=4), _lib.EINVAL), (dict(k_row=-8), _lib.EINVAL),
       (dict(v_row=1 << 23), _lib.EINVAL), (dict(q_batch=-8), _lib.EINVAL), (dict(v_batch=4), _lib.EINVAL),
       (dict(q=8), _lib.EINVAL), (dict(initial_state=8), _lib.EINVAL), (dict(T=1 << 31), _lib.EINVAL),
       (dict(T=1 << 30), _lib.EINVAL), (dict(B=1 << 20, H_q=1 << 3, H_v=1 << 6), _lib.EINVAL)]


@pytest.mark.parametrize("kw,code", BAD)
@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_chunked_validation(which, kw, code):
    st = _lib.LaFwdArgs if which == "fwd" else _lib.LaBwdArgs
    n = ctypes.c_size_t(0)
    a = la_args(st, **kw)
    assert getattr(_lib.lib, "gdr_la_%s_workspace" % which)(ctypes.byref(a), ctypes.byref(n)) == code
    assert getattr(_lib.lib, "gdr_la_" + which)(ctypes.byref(a), None) == code


@pytest.mark.parametrize("T", [0, 1, 63, 64, 65, 128, 129, 1000, 70000])
@pytest.mark.parametrize("n_seq", [None, 0, 1, 2, 37, 5000])
@pytest.mark.parametrize("dtype", [_lib.BF16, _lib.F32])
def test_chunked_split_of_any_length(T, n_seq, dtype):
    """The split into segments, of sequences without tokens too."""
    n = ctypes.c_size_t(0)
    packed = {} if n_seq is None else dict(B=1, cu_seqlens=64, n_seq=n_seq)
    for st, which in ((_lib.LaFwdArgs, "fwd"), (_lib.LaBwdArgs, "bwd")):
        for segment in (0, 1, 7):
            a = la_args(st, T=T, dtype=dtype, segment_chunks=segment, q_batch=0, k_batch=0, v_batch=0, **packed)
            assert getattr(_lib.lib, "gdr_la_%s_workspace" % which)(ctypes.byref(a), ctypes.byref(n)) == 0


def test_chunked_pointers_and_workspace():
    n = ctypes.c_size_t(0)
    call = lambda f, a: getattr(_lib.lib, f)(ctypes.byref(a), None)  # noqa: E731
    for name in ("q", "k", "v", "g", "o"):
        assert call("gdr_la_fwd", la_args(_lib.LaFwdArgs, **{name: None})) == _lib.EINVAL
    assert call("gdr_la_fwd", la_args(_lib.LaFwdArgs, o=8)) == _lib.EINVAL
    for name in ("q", "k", "v", "g", "dout", "dq", "dk", "dv", "dg"):
        assert call("gdr_la_bwd", la_args(_lib.LaBwdArgs, **{name: None})) == _lib.EINVAL
    for name in ("dout", "dht", "dq", "dh0"):
        assert call("gdr_la_bwd", la_args(_lib.LaBwdArgs, **{name: 8})) == _lib.EINVAL
    assert call("gdr_la_bwd", la_args(_lib.LaBwdArgs)) == _lib.EWORKSPACE
    long = la_args(_lib.LaFwdArgs, B=1, T=65536)
    assert _lib.lib.gdr_la_fwd_workspace(ctypes.byref(long), ctypes.byref(n)) == 0 and n.value > 0
    assert call("gdr_la_fwd", long) == _lib.EWORKSPACE
    long.segment_chunks = 1 << 20
    assert _lib.lib.gdr_la_fwd_workspace(ctypes.byref(long), ctypes.byref(n)) == 0 and n.value == 0
    # rows to clear, and nowhere to
    none = dict(B=1, n_seq=0, cu_seqlens=64, zero_rest=1)
    assert call("gdr_la_fwd", la_args(_lib.LaFwdArgs, o=None, **none)) == _lib.EINVAL
    for name in ("dq", "dk", "dv", "dg"):
        assert call("gdr_la_bwd", la_args(_lib.LaBwdArgs, **{name: None}, **none)) == _lib.EINVAL
    # nothing to do
    for kw in (dict(B=0), dict(T=0), dict(cu_seqlens=64, B=1, n_seq=0)):
        assert call("gdr_la_fwd", la_args(_lib.LaFwdArgs, **kw)) == 0
    assert call("gdr_la_bwd", la_args(_lib.LaBwdArgs, B=0)) == 0
    # a gate per token and one per head are told apart, and beta is not asked for
    a = _lib.PoolArgs()
    a.B, a.T, a.H_q, a.H_v, a.K, a.V, a.n_slots, a.dtype, a.out_dtype = 1, 1, 1, 1, 64, 64, 1, 0, 0
    a.q = a.k = a.v = a.g = a.states = 64
    assert call("gdr_la_step", a) == _lib.EINVAL  # no o
    a.o, a.T = 64, 0
    assert call("gdr_la_step", a) == 0


def test_norm_validation():
    def args(st, **kw):
        a = st()
        a.M, a.C, a.groups, a.x_row, a.gate_row, a.activation, a.eps = 4, 96, 3, 96, 96, _lib.ACT_SILU, 1e-5
        for n in ("x", "out", "dout", "dx", "dweight", "dbias"):
            if hasattr(a, n):
                setattr(a, n, 64)
        for n, v in kw.items():
            setattr(a, n, v)
        return a

    n = ctypes.c_size_t(0)
    for kw, code in ((dict(groups=5), _lib.EINVAL), (dict(groups=0), _lib.EINVAL), (dict(M=-1), _lib.EINVAL),
                     (dict(C=0), _lib.EINVAL), (dict(x_dtype=3), _lib.ENOTSUP), (dict(gate_dtype=3), _lib.ENOTSUP),
                     (dict(out_dtype=-1), _lib.ENOTSUP), (dict(activation=3), _lib.ENOTSUP), (dict(x_row=-1), _lib.EINVAL),
                     (dict(C=8193, groups=1), _lib.ENOTSUP), (dict(M=1 << 31), _lib.EINVAL)):
        assert _lib.lib.gdr_group_norm(ctypes.byref(args(_lib.NormFwdArgs, **kw)), None) == code, kw
        assert _lib.lib.gdr_group_norm_bwd(ctypes.byref(args(_lib.NormBwdArgs, **kw)), None) == code, kw
        assert _lib.lib.gdr_group_norm_bwd_workspace(ctypes.byref(args(_lib.NormBwdArgs, **kw)), ctypes.byref(n)) == code
    for kw in (dict(x=None), dict(out=None), dict(x=65), dict(out=65), dict(weight=66), dict(gate=65)):
        assert _lib.lib.gdr_group_norm(ctypes.byref(args(_lib.NormFwdArgs, **kw)), None) == _lib.EINVAL, kw
    for kw in (dict(x=None), dict(dout=None), dict(dx=None), dict(gate=64), dict(dweight=66)):
        assert _lib.lib.gdr_group_norm_bwd(ctypes.byref(args(_lib.NormBwdArgs, **kw)), None) == _lib.EINVAL, kw
    assert _lib.lib.gdr_group_norm_bwd(ctypes.byref(args(_lib.NormBwdArgs)), None) == _lib.EWORKSPACE
    assert _lib.lib.gdr_group_norm(ctypes.byref(args(_lib.NormFwdArgs, M=0)), None) == 0
    assert _lib.lib.gdr_group_norm_bwd(ctypes.byref(args(_lib.NormBwdArgs, M=0, dweight=None, dbias=None)), None) == 0


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("N,length", [(4096, 64), (512, 1024), (100, 1100), (1, 70000), (3, 1)])
def test_workspace_holds_the_borders_alone(N, length, packed):
    """No state is kept of a sequence that has no border: the backward's borders are 1024 tokens apart at most,
    those of packed sequences as many as 1024 fits into all tokens."""
    H, K, V = 64, 128, 128
    sizes = dict(T=N * length, B=1, cu_seqlens=64, n_seq=N) if packed else dict(T=length, B=N)
    kw = dict(sizes, H_q=H, H_v=H, K=K, V=V, q_row=H * K, k_row=H * K, v_row=H * V, segment_chunks=16, q_batch=0, k_batch=0, v_batch=0)
    borders = N * length // 1024 if packed else N * (-(-length // 1024) - 1)
    places = N + N * length // 1024 if packed else N * -(-length // 1024)
    # two states a border, and per token, place and sequence no more than a few numbers a head
    few = 4 * H * (4 * N * length + 40 * places + 32 * N) + 16 * 256
    n = ctypes.c_size_t(0)
    assert _lib.lib.gdr_la_bwd_workspace(ctypes.byref(la_args(_lib.LaBwdArgs, **kw)), ctypes.byref(n)) == 0
    assert n.value <= 2 * borders * 4 * H * K * V + few
    assert _lib.lib.gdr_la_fwd_workspace(ctypes.byref(la_args(_lib.LaFwdArgs, **kw)), ctypes.byref(n)) == 0
    assert n.value <= borders * 4 * H * K * V + few


@pytest.mark.parametrize("which", ["fwd", "bwd"])
def test_chunked_sequences_times_heads(which):
    """Up to 2^22 (sequence, v head) pairs, and (segment, v head) pairs."""
    st = _lib.LaFwdArgs if which == "fwd" else _lib.LaBwdArgs
    n = ctypes.c_size_t(0)
    for N, H, T, segment, packed, ok in ((1 << 13, 64, 1, 0, False, True), ((1 << 22) - 1, 1, 1, 0, False, True),
                                         (1 << 22, 1, 1, 0, False, False), ((1 << 16) - 1, 64, 1 << 16, 0, True, True),
                                         (1 << 16, 64, 1 << 16, 0, True, False), (1, 63, 1 << 22, 1, False, True),
                                         (1, 64, 1 << 22, 1, False, False)):
        a = la_args(st, B=1 if packed else N, T=T, H_q=H, H_v=H, K=64, V=64, q_row=H * 64, k_row=H * 64, v_row=H * 64, q_batch=0,
                    k_batch=0, v_batch=0, segment_chunks=segment, **(dict(cu_seqlens=64, n_seq=N) if packed else {}))
        rc = getattr(_lib.lib, "gdr_la_%s_workspace" % which)(ctypes.byref(a), ctypes.byref(n))
        assert rc == (_lib.OK if ok else _lib.EINVAL), (N, H, T)


def test_too_many_sequences_are_refused_by_name():
    q = torch.zeros(1 << 16, 1, 64, 64, dtype=BF)[:, :0]
    with pytest.raises(ValueError, match="sequences"):
        gdr.chunk_linear_attention_fwd(q, q, q, torch.zeros(1 << 16, 0, 64))
