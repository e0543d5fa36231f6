"""ctypes binding of ``liba2av.so`` (the C ABI in ``include/a2av.h``).

Argument marshalling only: every function takes torch tensors that already
live on the GPU, passes their device pointers and the stream to the C entry
point of the same name, and raises :class:`A2avError` for a nonzero host
return code. All computation runs in the library's HIP kernels; if the library
is missing the first call raises, there is no fallback.

torch is used for device memory and streams only. The stream defaults to
torch's current stream on the tensors' device.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "A2avError", "lib", "LIB_PATH",
    "OK", "EARG", "EHIP", "MAX_W", "MAX_SPLIT", "MAX_EXPERTS",
    "ST_BAD_SPLIT", "ST_SEND_OVERRUN", "ST_RECV_OVERFLOW", "ST_BAD_EXPERT", "ST_BAD_OFFSETS",
    "ST_BAD_PERM",
    "a2av_abi_version", "a2av_strerror", "a2av_exchange_splits", "a2av_offsets", "a2av_copy",
    "a2av_all_to_all_vdev",
    "moe_pack_workspace_bytes", "moe_pack", "moe_unpack", "moe_combine",
    "moe_regroup_workspace_bytes", "moe_regroup", "moe_dispatch_grouped_workspace_bytes",
    "moe_dispatch_grouped", "moe_combine_grouped_workspace_bytes", "moe_combine_grouped",
    "moe_pack_dispatch_workspace_bytes", "moe_pack_dispatch", "moe_unpack_return_workspace_bytes",
    "moe_unpack_return", "moe_combine_return_workspace_bytes", "moe_combine_return",
    "moe_route", "moe_route_backward", "moe_combine_backward_workspace_bytes",
    "moe_combine_backward", "moe_combine_return_backward_workspace_bytes",
    "moe_combine_return_backward", "moe_expert_linear_workspace_bytes", "moe_expert_linear",
    "moe_expert_linear_backward_workspace_bytes", "moe_expert_linear_backward",
    "moe_mx_row_bytes", "moe_mx_quantize", "moe_mx_dequantize", "moe_rms_norm",
    "moe_rms_norm_backward_workspace_bytes", "moe_rms_norm_backward",
    "moe_expert_linear_mx_workspace_bytes", "moe_expert_linear_mx", "MX_FP8", "MX_FP4",
    "SCORE_SOFTMAX", "SCORE_SIGMOID", "ACT_NONE", "ACT_RELU", "ACT_GELU", "ACT_SILU",
    "ACT_SWIGLU", "MAX_WIDTH",
    "keys_bucketize_workspace_bytes",
    "keys_bucketize", "keys_exchange_workspace_bytes", "keys_exchange",
    "keys_exchange_noalloc", "NOALLOC_SCRATCH_BYTES", "a2av_device_copy",
    "a2av_device_read", "a2av_device_fill", "SINK_WORDS",
    "MAX_TABLES",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liba2av.so")

OK, EARG, EHIP = 0, -1, -2
MAX_W = 64
MAX_SPLIT = 1 << 40
MAX_EXPERTS = 4096
MAX_TABLES = 4096
NOALLOC_SCRATCH_BYTES = 1 << 20
SINK_WORDS = 4096
ST_BAD_SPLIT = 1
ST_SEND_OVERRUN = 2
ST_RECV_OVERFLOW = 4
ST_BAD_EXPERT = 8
ST_BAD_OFFSETS = 16
ST_BAD_PERM = 32
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
ACT_NONE, ACT_RELU, ACT_GELU, ACT_SILU, ACT_SWIGLU = range(5)
MAX_WIDTH = 1 << 20
MX_FP8, MX_FP4 = 3, 4
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_lib = None


class A2avError(RuntimeError):
    def __init__(self, fn, code):
        super().__init__(f"{fn} returned {code}: {a2av_strerror(code)}")
        self.code = code


def lib():
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m embeddings_a2av_virtual_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
        vpp = ctypes.POINTER(ctypes.c_void_p)
        i64p = ctypes.POINTER(ctypes.c_int64)
        L.a2av_abi_version.argtypes = []
        L.a2av_abi_version.restype = i32
        L.a2av_strerror.argtypes = [i32]
        L.a2av_strerror.restype = ctypes.c_char_p
        L.a2av_exchange_splits.argtypes = [i32, vp, vp, vp, vp]
        L.a2av_offsets.argtypes = [i32, vp, vp, vp, vp, vp, vp]
        L.a2av_copy.argtypes = [i32, sz, vpp, i64p, vpp, i64p, vp, vp, vp, vp, vp]
        L.a2av_all_to_all_vdev.argtypes = [i32, sz, vpp, i64p, vpp, i64p, vp, vp, vp, vp, vp, vp]
        L.moe_pack_workspace_bytes.argtypes = [i32, i64, i32, i32]
        L.moe_pack_workspace_bytes.restype = sz
        L.moe_pack.argtypes = [i32, i64, i32, i32, sz, vpp, vpp, vpp, vpp, vp, vp, vp, sz, vp, vp]
        L.moe_unpack.argtypes = [i32, i64, i32, sz, vpp, vpp, vpp, vp, vp]
        L.moe_combine.argtypes = [i32, i64, i32, i64, vpp, vpp, vpp, vpp, vp, vp]
        L.moe_regroup_workspace_bytes.argtypes = [i32, i32]
        L.moe_regroup_workspace_bytes.restype = sz
        L.moe_regroup.argtypes = [i32, i32, sz, vp, vpp, i64p, vpp, i64p, vp, i32, vp, sz, vp, vp]
        L.moe_dispatch_grouped_workspace_bytes.argtypes = [i32, i32]
        L.moe_dispatch_grouped_workspace_bytes.restype = sz
        L.moe_dispatch_grouped.argtypes = [i32, i32, sz, vp, vpp, i64p, vpp, i64p, vp, i32, vp, sz,
                                           vp, vp]
        L.moe_combine_grouped_workspace_bytes.argtypes = [i32, i64, i32, i32]
        L.moe_combine_grouped_workspace_bytes.restype = sz
        L.moe_combine_grouped.argtypes = [i32, i64, i32, i32, i64, vp, vpp, vpp, vpp, i64p, vpp,
                                          vpp, vp, sz, vp, vp]
        L.moe_pack_dispatch_workspace_bytes.argtypes = [i32, i64, i32, i32]
        L.moe_pack_dispatch_workspace_bytes.restype = sz
        L.moe_pack_dispatch.argtypes = [i32, i64, i32, i32, sz, vpp, vpp, vpp, i64p, vpp, vp, vp,
                                        vp, i32, vp, sz, vp, vp]
        L.moe_unpack_return_workspace_bytes.argtypes = [i32, i32]
        L.moe_unpack_return_workspace_bytes.restype = sz
        L.moe_unpack_return.argtypes = [i32, i64, i32, i32, sz, vp, vpp, vpp, vpp, i64p, vpp, i32,
                                        vp, sz, vp, vp]
        L.moe_combine_return_workspace_bytes.argtypes = [i32, i64, i32, i32]
        L.moe_combine_return_workspace_bytes.restype = sz
        L.moe_combine_return.argtypes = [i32, i64, i32, i32, i64, vp, vpp, vpp, vpp, i64p, vpp, vpp,
                                         i32, vp, sz, vp, vp]
        L.moe_route.argtypes = [i32, i64, i32, i32, i32, i32, vpp, vp, i32, i32, i32, i32,
                                ctypes.c_float, vpp, vpp, vp, vp]
        L.moe_route_backward.argtypes = [i32, i64, i32, i32, i32, i32, vpp, vpp, vpp, i32,
                                         ctypes.c_float, vpp, vpp, vp, vp]
        L.moe_combine_backward_workspace_bytes.argtypes = [i32, i64, i32]
        L.moe_combine_backward_workspace_bytes.restype = sz
        L.moe_combine_backward.argtypes = [i32, i64, i32, i64, vpp, vpp, vpp, vpp, vpp, vpp, vp, sz,
                                           vp, vp]
        L.moe_combine_return_backward_workspace_bytes.argtypes = [i32, i64, i32, i32]
        L.moe_combine_return_backward_workspace_bytes.restype = sz
        L.moe_combine_return_backward.argtypes = [i32, i64, i32, i32, i64, vp, vpp, vpp, vpp, i64p,
                                                  vpp, vpp, vpp, vpp, i32, vp, sz, vp, vp]
        L.moe_expert_linear_workspace_bytes.argtypes = [i32, i32, i64, i64, i32, i64p]
        L.moe_expert_linear_workspace_bytes.restype = sz
        L.moe_expert_linear.argtypes = [i32, i32, i64, i64, i32, i32, vpp, i64p, vp, vpp, vpp, vpp,
                                        vpp, vpp, vp, sz, vp, vp]
        L.moe_expert_linear_backward_workspace_bytes.argtypes = [i32, i32, i64, i64, i32, i64p]
        L.moe_expert_linear_backward_workspace_bytes.restype = sz
        L.moe_expert_linear_backward.argtypes = [i32, i32, i64, i64, i32, i32, vpp, i64p, vp, vpp,
                                                 vpp, vpp, vpp, vpp, vpp, vpp, vp, sz, vp, vp]
        L.moe_mx_row_bytes.argtypes = [i32, i64]
        L.moe_mx_row_bytes.restype = sz
        L.moe_mx_quantize.argtypes = [i32, i64, i32, i32, vpp, i64p, vpp, vp, vp]
        L.moe_mx_dequantize.argtypes = [i32, i64, i32, i32, vpp, i64p, vpp, vp, vp]
        L.moe_rms_norm.argtypes = [i32, i64, i64, i32, ctypes.c_double, vpp, vpp, vp, vpp, vpp, vpp,
                                   i32, vp, vp]
        L.moe_rms_norm_backward_workspace_bytes.argtypes = [i32, i64, i64]
        L.moe_rms_norm_backward_workspace_bytes.restype = sz
        L.moe_rms_norm_backward.argtypes = [i32, i64, i64, i32, ctypes.c_double, vpp, vp, vpp, vpp,
                                            vpp, vp, vp, sz, vp, vp]
        L.moe_expert_linear_mx_workspace_bytes.argtypes = [i32, i32, i64, i64, i32, i64p]
        L.moe_expert_linear_mx_workspace_bytes.restype = sz
        L.moe_expert_linear_mx.argtypes = [i32, i32, i64, i64, i32, i32, vpp, i64p, vp, vpp, vpp,
                                           vpp, i32, vp, sz, vp, vp]
        L.keys_bucketize_workspace_bytes.argtypes = [i32, i32]
        L.keys_bucketize_workspace_bytes.restype = sz
        L.keys_bucketize.argtypes = [i32, i32, i64, vpp, vpp, i64p, vpp, vpp, vp, vp, vp, sz, vp,
                                     vp]
        L.keys_exchange_workspace_bytes.argtypes = [i32, i32]
        L.keys_exchange_workspace_bytes.restype = sz
        L.keys_exchange.argtypes = [i32, i32, i64, vpp, vpp, i64p, vpp, i64p, vpp, i64p, vp, vp, vp,
                                    vp, sz, vp, vp]
        L.keys_exchange_noalloc.argtypes = [i32, i32, i64, vpp, vpp, i64p, vpp, i64p, vpp, i64p,
                                            vp, vp, vp, vp, vp]
        L.a2av_device_copy.argtypes = [vp, vp, sz, vp]
        L.a2av_device_read.argtypes = [vp, sz, vp, vp]
        L.a2av_device_fill.argtypes = [vp, sz, ctypes.c_uint32, i32, vp]
        for f in ("a2av_exchange_splits", "a2av_offsets", "a2av_copy", "a2av_all_to_all_vdev",
                  "moe_pack", "moe_unpack", "moe_combine", "moe_regroup", "moe_dispatch_grouped",
                  "moe_combine_grouped", "moe_pack_dispatch", "moe_unpack_return",
                  "moe_combine_return", "moe_route", "moe_route_backward",
                  "moe_combine_backward", "moe_combine_return_backward", "moe_expert_linear",
                  "moe_expert_linear_backward", "moe_mx_quantize", "moe_mx_dequantize",
                  "moe_rms_norm", "moe_rms_norm_backward", "moe_expert_linear_mx",
                  "keys_bucketize", "keys_exchange", "keys_exchange_noalloc",
                  "a2av_device_copy", "a2av_device_read", "a2av_device_fill"):
            getattr(L, f).restype = i32
        _lib = L
    return _lib


# ------------------------------------------------------------------ marshalling helpers
def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _stream(stream, like: torch.Tensor) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(like.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr_array(tensors, name):
    arr = (ctypes.c_void_p * len(tensors))()
    for i, t in enumerate(tensors):
        arr[i] = None if t is None else _dev(t, f"{name}[{i}]")
    return arr


def _i64_array(vals):
    arr = (ctypes.c_int64 * len(vals))()
    for i, v in enumerate(vals):
        arr[i] = int(v)
    return arr


_PTRS = [ctypes.c_void_p * n for n in range(MAX_W + 1)]
_Tensor = torch.Tensor
# the current stream's handle without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _typed(tensors, name, dtype, sizes):
    """Pointers of one array per rank (None: no arrays), each on the GPU,
    contiguous, of this type and with at least this many elements."""
    if tensors is None:
        return None
    if len(tensors) != len(sizes):
        raise ValueError(f"{name} needs {len(sizes)} entries")
    ptrs = []
    add = ptrs.append
    for t, n in zip(tensors, sizes):
        # the usual case in one expression; anything else is looked into
        if (type(t) is _Tensor and t.dtype is dtype and t.is_cuda and t.is_contiguous()
                and t.numel() >= n):
            add(t.data_ptr())
        elif t is None:
            if n > 0:
                raise ValueError(f"{name}[{len(ptrs)}] needs {n} elements")
            add(None)
        else:
            add(_one(t, f"{name}[{len(ptrs)}]", dtype, n))
    return _PTRS[len(ptrs)](*ptrs) if len(ptrs) <= MAX_W else (ctypes.c_void_p * len(ptrs))(*ptrs)


def _one(t, name, dtype, n):
    p = _dev(t, name)
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    if t.numel() < n:
        raise ValueError(f"{name} needs {n} elements, has {t.numel()}")
    return p


def _check(fn, rc):
    if rc != OK:
        raise A2avError(fn, rc)


def _call(fn, like, stream, *args):
    """The C entry point on `stream` (or the current one of `like`'s GPU), with
    that GPU current: the kernels of a stream are launched on the GPU that is
    current."""
    f = getattr(_lib or lib(), fn)
    device = like.device.index
    s = _raw_stream(device) if stream is None and _raw_stream else _stream(stream, like)
    if device == torch.cuda.current_device():
        rc = f(*args, s)
    else:
        with torch.cuda.device(device):
            rc = f(*args, s)
    if rc != OK:
        raise A2avError(fn, rc)


# ------------------------------------------------------------------ entry points
def a2av_abi_version() -> int:
    return lib().a2av_abi_version()


def a2av_strerror(code: int) -> str:
    return lib().a2av_strerror(int(code)).decode()


def a2av_exchange_splits(S, O, status, stream=None):
    """O[d][s] = S[s][d]; S, O: int64 [W, W] on the GPU; status: int32 [1]."""
    W = S.shape[0]
    _check("a2av_exchange_splits",
           lib().a2av_exchange_splits(W, _dev(S, "S"), _dev(O, "O"), _dev(status, "status"),
                                      _stream(stream, S)))


def a2av_offsets(S, O, send_off, recv_off, status, stream=None):
    """Exclusive scans of the rows of S and O into [W, W+1] int64 offsets."""
    W = S.shape[0]
    _check("a2av_offsets",
           lib().a2av_offsets(W, _dev(S, "S"), _dev(O, "O"), _dev(send_off, "send_off"),
                              _dev(recv_off, "recv_off"), _dev(status, "status"),
                              _stream(stream, S)))


def a2av_copy(row_bytes, ins, in_rows, outs, out_cap_rows, S, send_off, recv_off, status,
              stream=None):
    """Payload step. ``ins``/``outs``: W GPU tensors (any dtype, contiguous);
    ``in_rows``/``out_cap_rows``: W host integers (rows each buffer holds)."""
    W = len(ins)
    if len(outs) != W or len(in_rows) != W or len(out_cap_rows) != W:
        raise ValueError("ins, outs, in_rows and out_cap_rows need W entries each")
    _check("a2av_copy",
           lib().a2av_copy(W, int(row_bytes), _ptr_array(ins, "ins"), _i64_array(in_rows),
                           _ptr_array(outs, "outs"), _i64_array(out_cap_rows), _dev(S, "S"),
                           _dev(send_off, "send_off"), _dev(recv_off, "recv_off"),
                           _dev(status, "status"), _stream(stream, S)))


def a2av_all_to_all_vdev(row_bytes, ins, in_rows, outs, out_cap_rows, S, O, send_off, recv_off,
                         status, stream=None):
    """Exchange, offsets and payload in one call (one launch for W <= 16)."""
    W = len(ins)
    if len(outs) != W or len(in_rows) != W or len(out_cap_rows) != W:
        raise ValueError("ins, outs, in_rows and out_cap_rows need W entries each")
    _check("a2av_all_to_all_vdev",
           lib().a2av_all_to_all_vdev(W, int(row_bytes), _ptr_array(ins, "ins"),
                                      _i64_array(in_rows), _ptr_array(outs, "outs"),
                                      _i64_array(out_cap_rows), _dev(S, "S"), _dev(O, "O"),
                                      _dev(send_off, "send_off"), _dev(recv_off, "recv_off"),
                                      _dev(status, "status"), _stream(stream, S)))


def moe_pack_workspace_bytes(W, T, k, E) -> int:
    return int(lib().moe_pack_workspace_bytes(int(W), int(T), int(k), int(E)))


def moe_pack(W, T, k, E, row_bytes, tokens, ids, send, perm, S, expert_counts, workspace,
             status, stream=None):
    """Stable pack of every rank's routing slots by expert id (see a2av.h)."""
    _check("moe_pack",
           lib().moe_pack(int(W), int(T), int(k), int(E), int(row_bytes),
                          _ptr_array(tokens, "tokens"), _ptr_array(ids, "ids"),
                          _ptr_array(send, "send"), _ptr_array(perm, "perm"), _dev(S, "S"),
                          _dev(expert_counts, "expert_counts"), _dev(workspace, "workspace"),
                          workspace.numel() * workspace.element_size(), _dev(status, "status"),
                          _stream(stream, S)))


def moe_unpack(W, T, k, row_bytes, back, perm, out, status, stream=None):
    """out[r][q] = back[r][perm[r][q]] for every rank r."""
    _check("moe_unpack",
           lib().moe_unpack(int(W), int(T), int(k), int(row_bytes), _ptr_array(back, "back"),
                            _ptr_array(perm, "perm"), _ptr_array(out, "out"),
                            _dev(status, "status"), _stream(stream, status)))


def moe_combine(W, T, k, H, back, perm, weights, out, status, stream=None):
    """Gate-weighted combine: out[r][t] = bf16(fma chain over j of
    weights[r][t][j] * back[r][perm[r][t*k+j]]), in slot order."""
    _check("moe_combine",
           lib().moe_combine(int(W), int(T), int(k), int(H), _ptr_array(back, "back"),
                             _ptr_array(perm, "perm"), _ptr_array(weights, "weights"),
                             _ptr_array(out, "out"), _dev(status, "status"),
                             _stream(stream, status)))


def moe_regroup_workspace_bytes(W, E) -> int:
    return int(lib().moe_regroup_workspace_bytes(int(W), int(E)))


def moe_regroup(W, E, row_bytes, counts, ins, in_rows, outs, out_cap_rows, expert_offsets,
                direction, workspace, status, stream=None):
    """Per-rank regroup between (source, expert) and (expert, source) row order."""
    if len(ins) != W or len(outs) != W or len(in_rows) != W or len(out_cap_rows) != W:
        raise ValueError("ins, outs, in_rows and out_cap_rows need W entries each")
    _check("moe_regroup",
           lib().moe_regroup(int(W), int(E), int(row_bytes), _dev(counts, "counts"),
                             _ptr_array(ins, "ins"), _i64_array(in_rows), _ptr_array(outs, "outs"),
                             _i64_array(out_cap_rows), _dev(expert_offsets, "expert_offsets"),
                             int(direction), _dev(workspace, "workspace"),
                             workspace.numel() * workspace.element_size(),
                             _dev(status, "status"), _stream(stream, status)))


def moe_dispatch_grouped_workspace_bytes(W, E) -> int:
    return int(lib().moe_dispatch_grouped_workspace_bytes(int(W), int(E)))


def moe_dispatch_grouped(W, E, row_bytes, counts, ins, in_rows, outs, out_cap_rows,
                         expert_offsets, direction, workspace, status, stream=None):
    """Dispatch a2av + expert regroup in one copy (direction 0), or its inverse (1)."""
    if len(ins) != W or len(outs) != W or len(in_rows) != W or len(out_cap_rows) != W:
        raise ValueError("ins, outs, in_rows and out_cap_rows need W entries each")
    _check("moe_dispatch_grouped",
           lib().moe_dispatch_grouped(int(W), int(E), int(row_bytes), _dev(counts, "counts"),
                                      _ptr_array(ins, "ins"), _i64_array(in_rows),
                                      _ptr_array(outs, "outs"), _i64_array(out_cap_rows),
                                      _dev(expert_offsets, "expert_offsets"), int(direction),
                                      _dev(workspace, "workspace"),
                                      workspace.numel() * workspace.element_size(),
                                      _dev(status, "status"), _stream(stream, status)))


def moe_combine_grouped_workspace_bytes(W, T, k, E) -> int:
    return int(lib().moe_combine_grouped_workspace_bytes(int(W), int(T), int(k), int(E)))


def moe_combine_grouped(W, T, k, E, H, counts, ids, perm, expert_side, exp_rows, weights, out,
                        workspace, status, stream=None):
    """The return trip and the weighted combine in one pass, reading every
    slot's row on its owner's expert side."""
    _check("moe_combine_grouped",
           lib().moe_combine_grouped(int(W), int(T), int(k), int(E), int(H),
                                     _dev(counts, "counts"), _ptr_array(ids, "ids"),
                                     _ptr_array(perm, "perm"),
                                     _ptr_array(expert_side, "expert_side"),
                                     _i64_array(exp_rows), _ptr_array(weights, "weights"),
                                     _ptr_array(out, "out"), _dev(workspace, "workspace"),
                                     workspace.numel() * workspace.element_size(),
                                     _dev(status, "status"), _stream(stream, status)))


def moe_pack_dispatch_workspace_bytes(W, T, k, E) -> int:
    return int(lib().moe_pack_dispatch_workspace_bytes(int(W), int(T), int(k), int(E)))


def moe_pack_dispatch(W, T, k, E, row_bytes, tokens, ids, recv, recv_cap_rows, perm, S,
                      expert_counts, block_offsets, layout, workspace, status, stream=None):
    """moe_pack and the dispatch in one step: every slot's token row written
    straight into its owner's receive buffer (layout 0: source-major, as the
    a2av delivers; 1: expert-major, as the grouped dispatch delivers)."""
    if (len(tokens) != W or len(ids) != W or len(recv) != W or len(recv_cap_rows) != W
            or len(perm) != W):
        raise ValueError("tokens, ids, recv, recv_cap_rows and perm need W entries each")
    _check("moe_pack_dispatch",
           lib().moe_pack_dispatch(int(W), int(T), int(k), int(E), int(row_bytes),
                                   _ptr_array(tokens, "tokens"), _ptr_array(ids, "ids"),
                                   _ptr_array(recv, "recv"), _i64_array(recv_cap_rows),
                                   _ptr_array(perm, "perm"), _dev(S, "S"),
                                   _dev(expert_counts, "expert_counts"),
                                   _dev(block_offsets, "block_offsets"), int(layout),
                                   _dev(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(),
                                   _dev(status, "status"), _stream(stream, status)))


def moe_unpack_return_workspace_bytes(W, E) -> int:
    return int(lib().moe_unpack_return_workspace_bytes(int(W), int(E)))


def moe_unpack_return(W, T, k, E, row_bytes, expert_counts, ids, perm, recv, recv_rows, out,
                      layout, workspace, status, stream=None):
    """The inverse of moe_pack_dispatch: every slot's row read back from its
    owner's receive buffer."""
    if len(ids) != W or len(perm) != W or len(recv) != W or len(recv_rows) != W or len(out) != W:
        raise ValueError("ids, perm, recv, recv_rows and out need W entries each")
    _check("moe_unpack_return",
           lib().moe_unpack_return(int(W), int(T), int(k), int(E), int(row_bytes),
                                   _dev(expert_counts, "expert_counts"), _ptr_array(ids, "ids"),
                                   _ptr_array(perm, "perm"), _ptr_array(recv, "recv"),
                                   _i64_array(recv_rows), _ptr_array(out, "out"), int(layout),
                                   _dev(workspace, "workspace"),
                                   workspace.numel() * workspace.element_size(),
                                   _dev(status, "status"), _stream(stream, status)))


def moe_combine_return_workspace_bytes(W, T, k, E) -> int:
    return int(lib().moe_combine_return_workspace_bytes(int(W), int(T), int(k), int(E)))


def moe_combine_return(W, T, k, E, H, expert_counts, ids, perm, recv, recv_rows, weights, out,
                       layout, workspace, status, stream=None):
    """The return trip and the gate-weighted combine in one pass, reading
    every slot's row where moe_pack_dispatch left it."""
    if (len(ids) != W or len(perm) != W or len(recv) != W or len(recv_rows) != W
            or len(weights) != W or len(out) != W):
        raise ValueError("ids, perm, recv, recv_rows, weights and out need W entries each")
    _check("moe_combine_return",
           lib().moe_combine_return(int(W), int(T), int(k), int(E), int(H),
                                    _dev(expert_counts, "expert_counts"), _ptr_array(ids, "ids"),
                                    _ptr_array(perm, "perm"), _ptr_array(recv, "recv"),
                                    _i64_array(recv_rows), _ptr_array(weights, "weights"),
                                    _ptr_array(out, "out"), int(layout),
                                    _dev(workspace, "workspace"),
                                    workspace.numel() * workspace.element_size(),
                                    _dev(status, "status"), _stream(stream, status)))


def moe_route(W, T, k, E, score, logits, bias, groups, topk_groups, group_top, renorm, scale, ids,
              weights, status, stream=None):
    """Expert ids (int32 [T, k] per rank) and gate weights (fp32) from router
    logits [T, E] (fp32, bf16 or fp16): softmax or sigmoid scores, a selection
    bias (fp32 [E] or None), the best topk_groups of groups, the k best
    experts, renormalised and scaled."""
    dtype = _logits_type(logits)
    _call("moe_route", status, stream, int(W), int(T), int(k), int(E), _TYPES[dtype], int(score),
          _typed(logits, "logits", dtype, [T * E] * W),
          None if bias is None else _one(bias, "bias", torch.float32, E), int(groups),
          int(topk_groups), int(group_top), int(bool(renorm)), float(scale),
          _typed(ids, "ids", torch.int32, [T * k] * W),
          _typed(weights, "weights", torch.float32, [T * k] * W), _dev(status, "status"))


def moe_route_backward(W, T, k, E, score, logits, ids, weights, renorm, scale, d_weights, d_logits,
                       status, stream=None):
    """The gradient of moe_route's weights in its logits, the ids held fixed."""
    dtype = _logits_type(logits)
    _call("moe_route_backward", status, stream, int(W), int(T), int(k), int(E), _TYPES[dtype],
          int(score), _typed(logits, "logits", dtype, [T * E] * W),
          _typed(ids, "ids", torch.int32, [T * k] * W),
          _typed(weights, "weights", torch.float32, [T * k] * W), int(bool(renorm)), float(scale),
          _typed(d_weights, "d_weights", torch.float32, [T * k] * W),
          _typed(d_logits, "d_logits", dtype, [T * E] * W), _dev(status, "status"))


def _logits_type(logits):
    if not logits or not isinstance(logits[0], torch.Tensor) or logits[0].dtype not in _TYPES:
        raise ValueError("logits must be a list of fp32, bf16 or fp16 tensors, one per rank")
    return logits[0].dtype


def moe_combine_backward_workspace_bytes(W, T, k) -> int:
    return int(lib().moe_combine_backward_workspace_bytes(int(W), int(T), int(k)))


def moe_combine_backward(W, T, k, H, back, perm, weights, d_out, d_back, d_weights, workspace,
                         status, stream=None):
    """The gradient of moe_combine in its rows (d_back, bf16) and its weights
    (d_weights, fp32), from d_out (bf16 [T, H] per rank)."""
    bf16, rows, toks = torch.bfloat16, [T * k * H] * W, [T * H] * W
    _call("moe_combine_backward", status, stream, int(W), int(T), int(k), int(H),
          _typed(back, "back", bf16, rows), _typed(perm, "perm", torch.int64, [T * k] * W),
          _typed(weights, "weights", torch.float32, [T * k] * W),
          _typed(d_out, "d_out", bf16, toks), _typed(d_back, "d_back", bf16, rows),
          _typed(d_weights, "d_weights", torch.float32, [T * k] * W),
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def moe_combine_return_backward_workspace_bytes(W, T, k, E) -> int:
    return int(lib().moe_combine_return_backward_workspace_bytes(int(W), int(T), int(k), int(E)))


def moe_combine_return_backward(W, T, k, E, H, expert_counts, ids, perm, recv, recv_rows, weights,
                                d_out, d_recv, d_weights, layout, workspace, status, stream=None):
    """The gradient of moe_combine_return: every slot's row read, and its
    gradient written, at the owner of its expert."""
    bf16, rows = torch.bfloat16, [int(n) * H for n in recv_rows]
    if len(rows) != W:
        raise ValueError("recv_rows needs W entries")
    _call("moe_combine_return_backward", status, stream, int(W), int(T), int(k), int(E), int(H),
          _one(expert_counts, "expert_counts", torch.int64, W * E),
          _typed(ids, "ids", torch.int32, [T * k] * W),
          _typed(perm, "perm", torch.int64, [T * k] * W), _typed(recv, "recv", bf16, rows),
          _i64_array(recv_rows), _typed(weights, "weights", torch.float32, [T * k] * W),
          _typed(d_out, "d_out", bf16, [T * H] * W), _typed(d_recv, "d_recv", bf16, rows),
          _typed(d_weights, "d_weights", torch.float32, [T * k] * W), int(layout),
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def _expert_type(x):
    for t in x:
        if isinstance(t, torch.Tensor):
            if t.dtype not in (torch.bfloat16, torch.float16):
                raise ValueError(f"expert rows must be bf16 or fp16, not {t.dtype}")
            return t.dtype
    raise ValueError("x must be a list of tensors, one per rank")


def moe_expert_linear_workspace_bytes(W, P, K, N, act, x_rows) -> int:
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    return int(lib().moe_expert_linear_workspace_bytes(int(W), int(P), int(K), int(N), int(act),
                                                       _i64_array(x_rows)))


def moe_expert_linear(W, P, K, N, act, x, x_rows, expert_offsets, weight, bias, residual, out, pre,
                      workspace, status, stream=None):
    """out = act(x . weight^T + bias) + residual for the rows of every expert
    (bf16 or fp16); bias, residual and pre may be None."""
    dtype, NW = _expert_type(weight), 2 * N if act == ACT_SWIGLU else N
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    narrow, wide = [int(n) * N for n in x_rows], [int(n) * NW for n in x_rows]
    _call("moe_expert_linear", status, stream, int(W), int(P), int(K), int(N), _TYPES[dtype],
          int(act), _typed(x, "x", dtype, [int(n) * K for n in x_rows]), _i64_array(x_rows),
          _one(expert_offsets, "expert_offsets", torch.int64, W * (P + 1)),
          _typed(weight, "weight", dtype, [P * NW * K] * W),
          _typed(bias, "bias", dtype, [P * NW] * W), _typed(residual, "residual", dtype, narrow),
          _typed(out, "out", dtype, narrow), _typed(pre, "pre", dtype, wide),
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def moe_expert_linear_backward_workspace_bytes(W, P, K, N, act, x_rows) -> int:
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    return int(lib().moe_expert_linear_backward_workspace_bytes(int(W), int(P), int(K), int(N),
                                                                int(act), _i64_array(x_rows)))


def moe_expert_linear_backward(W, P, K, N, act, x, x_rows, expert_offsets, weight, pre, d_out,
                               d_pre, d_x, d_weight, d_bias, workspace, status, stream=None):
    """The gradients of moe_expert_linear; d_x, d_weight and d_bias may be None
    (not wanted), pre and d_pre are None with ACT_NONE."""
    dtype, NW = _expert_type(weight), 2 * N if act == ACT_SWIGLU else N
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    wide, xs, ws = [int(n) * NW for n in x_rows], [int(n) * K for n in x_rows], [P * NW * K] * W
    _call("moe_expert_linear_backward", status, stream, int(W), int(P), int(K), int(N),
          _TYPES[dtype], int(act), _typed(x, "x", dtype, xs), _i64_array(x_rows),
          _one(expert_offsets, "expert_offsets", torch.int64, W * (P + 1)),
          _typed(weight, "weight", dtype, ws), _typed(pre, "pre", dtype, wide),
          _typed(d_out, "d_out", dtype, [int(n) * N for n in x_rows]),
          _typed(d_pre, "d_pre", dtype, wide), _typed(d_x, "d_x", dtype, xs),
          _typed(d_weight, "d_weight", dtype, ws), _typed(d_bias, "d_bias", dtype, [P * NW] * W),
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def moe_mx_row_bytes(format, H) -> int:
    return int(lib().moe_mx_row_bytes(int(format), int(H)))


def _value_type(lists, name):
    """The type of the first tensor in lists of fp32, bf16 or fp16 arrays."""
    for t in lists:
        if isinstance(t, torch.Tensor):
            if t.dtype not in _TYPES:
                raise ValueError(f"{name} must be fp32, bf16 or fp16, not {t.dtype}")
            return t.dtype
    raise ValueError(f"{name} must be a list of tensors, one per rank")


def moe_mx_quantize(W, H, format, x, n_rows, rows, status, stream=None):
    """Values [n_rows[r], H] (fp32, bf16 or fp16) to microscaled rows (uint8
    [n_rows[r], moe_mx_row_bytes(format, H)]) of MX_FP8 or MX_FP4 elements."""
    dtype, wide = _value_type(x, "x"), moe_mx_row_bytes(format, H)
    if len(n_rows) != W:
        raise ValueError("n_rows needs W entries")
    _call("moe_mx_quantize", status, stream, int(W), int(H), _TYPES[dtype], int(format),
          _typed(x, "x", dtype, [int(n) * H for n in n_rows]), _i64_array(n_rows),
          _typed(rows, "rows", torch.uint8, [int(n) * wide for n in n_rows]),
          _dev(status, "status"))


def moe_mx_dequantize(W, H, format, rows, n_rows, out, status, stream=None):
    """Microscaled rows back to values of out's type (fp32, bf16 or fp16)."""
    dtype, wide = _value_type(out, "out"), moe_mx_row_bytes(format, H)
    if len(n_rows) != W:
        raise ValueError("n_rows needs W entries")
    _call("moe_mx_dequantize", status, stream, int(W), int(H), _TYPES[dtype], int(format),
          _typed(rows, "rows", torch.uint8, [int(n) * wide for n in n_rows]), _i64_array(n_rows),
          _typed(out, "out", dtype, [int(n) * H for n in n_rows]), _dev(status, "status"))


def moe_rms_norm(W, T, H, eps, x, residual, weight, sum, out, rows, format, status, stream=None):
    """h = x + residual and y = h / sqrt(mean(h^2) + eps) * weight for rows
    [T, H] per rank (fp32, bf16 or fp16): h into sum, y into out and, as
    microscaled rows of the format, into rows. residual, sum, out and rows may
    be None (out and rows not both)."""
    dtype, n = _value_type([weight], "weight"), [T * H] * W
    _call("moe_rms_norm", status, stream, int(W), int(T), int(H), _TYPES[dtype], float(eps),
          _typed(x, "x", dtype, n), _typed(residual, "residual", dtype, n),
          _one(weight, "weight", dtype, H), _typed(sum, "sum", dtype, n),
          _typed(out, "out", dtype, n),
          _typed(rows, "rows", torch.uint8, [T * moe_mx_row_bytes(format, H)] * W), int(format),
          _dev(status, "status"))


def moe_rms_norm_backward_workspace_bytes(W, T, H) -> int:
    return int(lib().moe_rms_norm_backward_workspace_bytes(int(W), int(T), int(H)))


def moe_rms_norm_backward(W, T, H, eps, x, weight, d_out, d_sum, d_x, d_weight, workspace, status,
                          stream=None):
    """The gradients of moe_rms_norm in its rows (d_x, of x and of the residual
    alike) and its weight (d_weight, fp32 [H] over all ranks, or None); x is
    the sum that it wrote, d_sum that sum's gradient by other ways or None."""
    dtype, n = _value_type([weight], "weight"), [T * H] * W
    _call("moe_rms_norm_backward", status, stream, int(W), int(T), int(H), _TYPES[dtype],
          float(eps), _typed(x, "x", dtype, n), _one(weight, "weight", dtype, H),
          _typed(d_out, "d_out", dtype, n), _typed(d_sum, "d_sum", dtype, n),
          _typed(d_x, "d_x", dtype, n),
          None if d_weight is None else _one(d_weight, "d_weight", torch.float32, H),
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def moe_expert_linear_mx_workspace_bytes(W, P, K, N, act, x_rows) -> int:
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    return int(lib().moe_expert_linear_mx_workspace_bytes(int(W), int(P), int(K), int(N), int(act),
                                                          _i64_array(x_rows)))


def moe_expert_linear_mx(W, P, K, N, x_format, act, x, x_rows, expert_offsets, weight, bias, out,
                         workspace, status, stream=None):
    """out = act(x . weight^T + bias) for the rows of every expert: x in
    microscaled rows of x_format, the weight in MX_FP4 rows (uint8), bias fp32
    or None, out bf16, fp16 or (uint8) rows of MX_FP8."""
    NW = 2 * N if act == ACT_SWIGLU else N
    if len(x_rows) != W:
        raise ValueError("x_rows needs W entries")
    first = next((t for t in out if isinstance(t, torch.Tensor)), None)
    dtype = torch.bfloat16 if first is None else first.dtype
    if dtype not in (torch.bfloat16, torch.float16, torch.uint8):
        raise ValueError(f"out must be bf16, fp16 or uint8 (microscaled rows), not {dtype}")
    wide = moe_mx_row_bytes(MX_FP8, N) if dtype == torch.uint8 else N
    _call("moe_expert_linear_mx", status, stream, int(W), int(P), int(K), int(N), int(x_format),
          int(act),
          _typed(x, "x", torch.uint8, [int(n) * moe_mx_row_bytes(x_format, K) for n in x_rows]),
          _i64_array(x_rows), _one(expert_offsets, "expert_offsets", torch.int64, W * (P + 1)),
          _typed(weight, "weight", torch.uint8, [P * NW * moe_mx_row_bytes(MX_FP4, K)] * W),
          _typed(bias, "bias", torch.float32, [P * NW] * W),
          _typed(out, "out", dtype, [int(n) * wide for n in x_rows]),
          MX_FP8 if dtype == torch.uint8 else _TYPES[dtype],
          _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(),
          _dev(status, "status"))


def keys_bucketize_workspace_bytes(W, n_tables) -> int:
    return int(lib().keys_bucketize_workspace_bytes(int(W), int(n_tables)))


def keys_bucketize(W, n_tables, batch, lengths, keys, n_keys, lengths_out, keys_out, split_keys,
                   split_lengths, workspace, status, stream=None):
    """Owner-order bucketing of every rank's jagged keys (table t -> rank t mod W)."""
    if len(lengths) != W or len(keys) != W or len(n_keys) != W:
        raise ValueError("lengths, keys and n_keys need W entries each")
    _check("keys_bucketize",
           lib().keys_bucketize(int(W), int(n_tables), int(batch), _ptr_array(lengths, "lengths"),
                                _ptr_array(keys, "keys"), _i64_array(n_keys),
                                _ptr_array(lengths_out, "lengths_out"),
                                _ptr_array(keys_out, "keys_out"), _dev(split_keys, "split_keys"),
                                _dev(split_lengths, "split_lengths"), _dev(workspace, "workspace"),
                                workspace.numel() * workspace.element_size(),
                                _dev(status, "status"), _stream(stream, status)))


def keys_exchange_workspace_bytes(W, n_tables) -> int:
    return int(lib().keys_exchange_workspace_bytes(int(W), int(n_tables)))


def keys_exchange(W, n_tables, batch, lengths, keys, n_keys, lengths_out, lengths_cap, keys_out,
                  keys_cap, split_keys, split_lengths, recv_off_keys, workspace, status,
                  stream=None):
    """Bucketing and both exchanges of one batch's keys in one call."""
    if any(len(x) != W for x in (lengths, keys, n_keys, lengths_out, lengths_cap, keys_out,
                                 keys_cap)):
        raise ValueError("every per-rank list needs W entries")
    _check("keys_exchange",
           lib().keys_exchange(int(W), int(n_tables), int(batch), _ptr_array(lengths, "lengths"),
                               _ptr_array(keys, "keys"), _i64_array(n_keys),
                               _ptr_array(lengths_out, "lengths_out"), _i64_array(lengths_cap),
                               _ptr_array(keys_out, "keys_out"), _i64_array(keys_cap),
                               _dev(split_keys, "split_keys"), _dev(split_lengths, "split_lengths"),
                               _dev(recv_off_keys, "recv_off_keys"), _dev(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(),
                               _dev(status, "status"), _stream(stream, status)))


def keys_exchange_noalloc(W, n_tables, batch, lengths, keys, n_keys, lengths_out, lengths_cap,
                          keys_out, keys_cap, split_keys, split_lengths, recv_off_keys, status,
                          stream=None):
    """keys_exchange with the library's fixed per-GPU scratch instead of a
    workspace (allocates nothing)."""
    if any(len(x) != W for x in (lengths, keys, n_keys, lengths_out, lengths_cap, keys_out,
                                 keys_cap)):
        raise ValueError("every per-rank list needs W entries")
    _check("keys_exchange_noalloc",
           lib().keys_exchange_noalloc(int(W), int(n_tables), int(batch),
                                       _ptr_array(lengths, "lengths"), _ptr_array(keys, "keys"),
                                       _i64_array(n_keys), _ptr_array(lengths_out, "lengths_out"),
                                       _i64_array(lengths_cap), _ptr_array(keys_out, "keys_out"),
                                       _i64_array(keys_cap), _dev(split_keys, "split_keys"),
                                       _dev(split_lengths, "split_lengths"),
                                       _dev(recv_off_keys, "recv_off_keys"),
                                       _dev(status, "status"), _stream(stream, status)))


def a2av_device_copy(dst, src, nbytes, stream=None):
    """Plain contiguous copy of nbytes from src to dst (bandwidth ceiling)."""
    _check("a2av_device_copy",
           lib().a2av_device_copy(_dev(dst, "dst"), _dev(src, "src"), int(nbytes),
                                  _stream(stream, dst)))


def a2av_device_read(src, nbytes, sink, stream=None):
    """Read nbytes of src once (read-only bandwidth ceiling); each wave XORs
    the fold of what it read into one word of sink (SINK_WORDS int64)."""
    if sink.numel() * sink.element_size() < SINK_WORDS * 8:
        raise ValueError("sink needs SINK_WORDS int64 words")
    _check("a2av_device_read",
           lib().a2av_device_read(_dev(src, "src"), int(nbytes), _dev(sink, "sink"),
                                  _stream(stream, src)))


def a2av_device_fill(dst, nbytes, pattern, nontemporal=True, stream=None):
    """Write the 32-bit pattern over nbytes of dst (write-only bandwidth ceiling)."""
    _check("a2av_device_fill",
           lib().a2av_device_fill(_dev(dst, "dst"), int(nbytes), int(pattern) & 0xFFFFFFFF,
                                  1 if nontemporal else 0, _stream(stream, dst)))
