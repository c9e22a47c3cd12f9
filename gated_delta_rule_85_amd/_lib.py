"""ctypes binding of libgdr.so (the C ABI declared in include/gdr.h).

Argument marshalling only: every step of the operator runs in the library's
HIP kernels.  Importing this module fails loudly when the library has not
been built; there is no fallback.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

ABI_VERSION = 9
CHUNK = 64
FWD_STAGES = 3
BWD_STAGES = 4
TREE_MAX = 64    # GDR_TREE_MAX: nodes of a tree
COPY_MAX = 4096  # GDR_COPY_MAX: entries of one gdr_copy_states

OK, EINVAL, ENOTSUP, EWORKSPACE, ELAUNCH, ESCRATCH = 0, -1, -2, -3, -4, -5
SCRATCH_BYTES = 256 << 20  # GDR_SCRATCH_BYTES: gdr_fwd_noalloc's per-device scratch
BF16, F32 = 0, 1
ACT_NONE, ACT_SILU, ACT_SIGMOID = 0, 1, 2
CP_AUTO, CP_OFF, CP_WARMUP, CP_EXACT, CP_AUTO_EXACT, CP_AUTO_PAGES = 0, 1, 2, 3, 4, 5

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32


class FwdArgs(ctypes.Structure):
    """Mirror of gdr_fwd_args."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H_q", _i64), ("H_v", _i64), ("K", _i64), ("V", _i64),
        ("n_seq", _i64),
        ("dtype", _i32), ("out_dtype", _i32), ("scale", ctypes.c_float),
        ("cp_mode", _i32), ("cp_segment_chunks", _i32), ("cp_warmup_chunks", _i32),
        ("q", _p), ("k", _p), ("v", _p), ("g", _p), ("beta", _p), ("initial_state", _p),
        ("cu_seqlens", _p),
        ("o", _p), ("final_state", _p), ("g_cum", _p), ("A", _p), ("h", _p), ("h_bwd", _p), ("tblk_bwd", _p),
        ("w_out", _p), ("u_out", _p), ("events", _p),
        ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
    ]


class BwdArgs(ctypes.Structure):
    """Mirror of gdr_bwd_args."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H_q", _i64), ("H_v", _i64), ("K", _i64), ("V", _i64),
        ("n_seq", _i64),
        ("dtype", _i32), ("grad_dtype", _i32), ("cp_mode", _i32), ("cp_segment_chunks", _i32),
        ("scale", ctypes.c_float),
        ("q", _p), ("k", _p), ("v", _p), ("g_cum", _p), ("beta", _p), ("A", _p),
        ("dout", _p), ("dht", _p), ("initial_state", _p), ("cu_seqlens", _p), ("h_bwd", _p), ("tblk_bwd", _p),
        ("dq", _p), ("dk", _p), ("dv", _p), ("dbeta", _p), ("dg", _p), ("dh0", _p),
        ("events", _p), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
    ]


class PoolArgs(ctypes.Structure):
    """Mirror of gdr_pool_args."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H_q", _i64), ("H_v", _i64), ("K", _i64), ("V", _i64),
        ("n_seq", _i64), ("n_slots", _i64), ("slot_stride", _i64),
        ("q_row", _i64), ("k_row", _i64), ("v_row", _i64),
        ("q_batch", _i64), ("k_batch", _i64), ("v_batch", _i64),
        ("dtype", _i32), ("out_dtype", _i32), ("scale", ctypes.c_float),
        ("q", _p), ("k", _p), ("v", _p), ("g", _p), ("beta", _p), ("cu_seqlens", _p), ("slots", _p),
        ("parents", _p), ("accepted", _p), ("states", _p), ("o", _p), ("g_per_head", _i32),
    ]


class CopyArgs(ctypes.Structure):
    """Mirror of gdr_copy_args."""
    _fields_ = [
        ("n", _i64), ("n_dst", _i64), ("n_src", _i64), ("slot_bytes", _i64),
        ("dst_stride", _i64), ("src_stride", _i64), ("layers", _i64),
        ("dst_layer_stride", _i64), ("src_layer_stride", _i64),
        ("dst", _p), ("src", _p), ("states", _p), ("source", _p),
    ]


class LaFwdArgs(ctypes.Structure):
    """Mirror of gdr_la_fwd_args."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H_q", _i64), ("H_v", _i64), ("K", _i64), ("V", _i64), ("n_seq", _i64),
        ("q_row", _i64), ("k_row", _i64), ("v_row", _i64),
        ("q_batch", _i64), ("k_batch", _i64), ("v_batch", _i64),
        ("dtype", _i32), ("out_dtype", _i32), ("g_per_head", _i32), ("segment_chunks", _i32),
        ("scale", ctypes.c_float),
        ("q", _p), ("k", _p), ("v", _p), ("g", _p), ("initial_state", _p), ("cu_seqlens", _p),
        ("o", _p), ("final_state", _p), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
        ("zero_rest", _i32),
    ]


class LaBwdArgs(ctypes.Structure):
    """Mirror of gdr_la_bwd_args."""
    _fields_ = [
        ("B", _i64), ("T", _i64), ("H_q", _i64), ("H_v", _i64), ("K", _i64), ("V", _i64), ("n_seq", _i64),
        ("q_row", _i64), ("k_row", _i64), ("v_row", _i64),
        ("q_batch", _i64), ("k_batch", _i64), ("v_batch", _i64),
        ("dtype", _i32), ("grad_dtype", _i32), ("g_per_head", _i32), ("segment_chunks", _i32),
        ("scale", ctypes.c_float),
        ("q", _p), ("k", _p), ("v", _p), ("g", _p), ("initial_state", _p), ("cu_seqlens", _p),
        ("dout", _p), ("dht", _p),
        ("dq", _p), ("dk", _p), ("dv", _p), ("dg", _p), ("dh0", _p),
        ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
        ("zero_rest", _i32),
    ]


class NormFwdArgs(ctypes.Structure):
    """Mirror of gdr_norm_fwd_args."""
    _fields_ = [
        ("M", _i64), ("C", _i64), ("groups", _i64), ("x_row", _i64), ("gate_row", _i64),
        ("x_dtype", _i32), ("gate_dtype", _i32), ("out_dtype", _i32), ("activation", _i32), ("center", _i32),
        ("eps", ctypes.c_float),
        ("x", _p), ("weight", _p), ("bias", _p), ("gate", _p), ("out", _p),
    ]


class NormBwdArgs(ctypes.Structure):
    """Mirror of gdr_norm_bwd_args."""
    _fields_ = [
        ("M", _i64), ("C", _i64), ("groups", _i64), ("x_row", _i64), ("gate_row", _i64),
        ("x_dtype", _i32), ("gate_dtype", _i32), ("out_dtype", _i32), ("activation", _i32), ("center", _i32),
        ("eps", ctypes.c_float),
        ("x", _p), ("weight", _p), ("bias", _p), ("gate", _p), ("dout", _p),
        ("dx", _p), ("dgate", _p), ("dweight", _p), ("dbias", _p), ("workspace", _p), ("workspace_bytes", ctypes.c_size_t),
    ]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libgdr.so is not built (%s); run `python gated_delta_rule_85_amd/build.py` or "
            "__graft_entry__.build() first" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    lib.gdr_abi_version.restype = ctypes.c_int
    lib.gdr_abi_version.argtypes = []
    lib.gdr_strerror.restype = ctypes.c_char_p
    lib.gdr_strerror.argtypes = [ctypes.c_int]
    for name, st in (("gdr_fwd", FwdArgs), ("gdr_bwd", BwdArgs), ("gdr_la_fwd", LaFwdArgs), ("gdr_la_bwd", LaBwdArgs)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.POINTER(st), _p]
        fw = getattr(lib, name + "_workspace")
        fw.restype = ctypes.c_int
        fw.argtypes = [ctypes.POINTER(st), ctypes.POINTER(ctypes.c_size_t)]
    lib.gdr_fwd_noalloc.restype = ctypes.c_int
    lib.gdr_fwd_noalloc.argtypes = [ctypes.POINTER(FwdArgs), _p]
    lib.gdr_tblocks_bytes.restype = ctypes.c_int
    lib.gdr_tblocks_bytes.argtypes = [ctypes.POINTER(FwdArgs), ctypes.POINTER(ctypes.c_size_t)]
    for name, st in (("gdr_step", PoolArgs), ("gdr_la_step", PoolArgs), ("gdr_tree", PoolArgs), ("gdr_tree_accept", PoolArgs),
                     ("gdr_copy_states", CopyArgs), ("gdr_group_norm", NormFwdArgs),
                     ("gdr_group_norm_bwd", NormBwdArgs)):
        f = getattr(lib, name)
        f.restype = ctypes.c_int
        f.argtypes = [ctypes.POINTER(st), _p]
    lib.gdr_group_norm_bwd_workspace.restype = ctypes.c_int
    lib.gdr_group_norm_bwd_workspace.argtypes = [ctypes.POINTER(NormBwdArgs), ctypes.POINTER(ctypes.c_size_t)]
    if lib.gdr_abi_version() != ABI_VERSION:
        raise ImportError("libgdr ABI version %d, binding expects %d"
                          % (lib.gdr_abi_version(), ABI_VERSION))
    return lib


lib = _load()


class GdrError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__("%s failed: %s (%d)" % (fn, strerror(code), code))
        self.code = code


def strerror(code):
    return lib.gdr_strerror(int(code)).decode()


def abi_version():
    return lib.gdr_abi_version()


def fwd_workspace(args):
    n = ctypes.c_size_t(0)
    rc = lib.gdr_fwd_workspace(ctypes.byref(args), ctypes.byref(n))
    if rc:
        raise GdrError("gdr_fwd_workspace", rc)
    return n.value


def tblocks_bytes(args):
    n = ctypes.c_size_t(0)
    rc = lib.gdr_tblocks_bytes(ctypes.byref(args), ctypes.byref(n))
    if rc:
        raise GdrError("gdr_tblocks_bytes", rc)
    return n.value


def fwd(args, stream):
    rc = lib.gdr_fwd(ctypes.byref(args), _p(stream))
    if rc:
        raise GdrError("gdr_fwd", rc)


def fwd_noalloc(args, stream):
    """gdr_fwd on the library's static per-device scratch (args.workspace ignored)."""
    rc = lib.gdr_fwd_noalloc(ctypes.byref(args), _p(stream))
    if rc:
        raise GdrError("gdr_fwd_noalloc", rc)


def bwd_workspace(args):
    n = ctypes.c_size_t(0)
    rc = lib.gdr_bwd_workspace(ctypes.byref(args), ctypes.byref(n))
    if rc:
        raise GdrError("gdr_bwd_workspace", rc)
    return n.value


def bwd(args, stream):
    rc = lib.gdr_bwd(ctypes.byref(args), _p(stream))
    if rc:
        raise GdrError("gdr_bwd", rc)


def la_fwd(args, stream):
    rc = lib.gdr_la_fwd(ctypes.byref(args), _p(stream))
    if rc:
        raise GdrError("gdr_la_fwd", rc)
