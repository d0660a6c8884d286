"""Thin ctypes binding over libgdn.so (the C ABI in include/gdn.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of libgdn.so. Tensors must already live on the GPU; the current torch
stream is passed to the library. If the library has not been built, the first
call raises -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
# GDN_LIB_PATH selects another build of the same library (e.g. a tuning variant).
LIB_PATH = os.environ.get("GDN_LIB_PATH") or os.path.join(HERE, "libgdn.so")

GDN_OK = 0
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_NULL", 2: "GDN_ERR_SHAPE", 3: "GDN_ERR_UNSUPPORTED",
                4: "GDN_ERR_OVERFLOW", 5: "GDN_ERR_ALIGN", 6: "GDN_ERR_WORKSPACE",
                7: "GDN_ERR_LAUNCH", 8: "GDN_ERR_SCRATCH"}
NOALLOC_SCRATCH_BYTES = 64 << 20
F32, F16, BF16 = 0, 1, 2
MAP_GROUPED, MAP_TILED = 0, 1
DECAY_LOG_RATE, DECAY_NEGATIVE_RATE = 0, 1
L2NORM_QK, RAW_GATES, GATED_NORM, STREAM_STATE, HEAD_DECAY = 1, 2, 4, 8, 16
CHUNK = 64
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
ROPE_PLAIN, ROPE_LINEAR, ROPE_BASE, ROPE_BANDS = 0, 1, 2, 3

EXPORTED = ["gdn_conv_update", "gdn_decode_step", "gdn_prefill_workspace_bytes",
            "gdn_prefill_chunked", "gdn_status_string", "gdn_version", "gdn_decode_layer",
            "gdn_decode_launch_info", "gdn_prefill_launch_info", "gdn_prefill_chunked_noalloc",
            "gdn_linattn_decode_step", "gdn_linattn_prefill_workspace_bytes",
            "gdn_linattn_prefill_chunked", "gdn_add_rms_norm", "gdn_quant_matmul",
            "gdn_quant_matmul_launch_info", "gdn_rope", "gdn_rope_frequencies",
            "gdn_attention_prefill_workspace_bytes", "gdn_attention_prefill",
            "gdn_attention_decode_workspace_bytes", "gdn_attention_decode", "gdn_pages_free",
            "gdn_pages_reserve", "gdn_pages_workspace_bytes", "gdn_pages_fork", "gdn_pages_compact"]

_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_VP = ctypes.c_void_p


class Dims(ctypes.Structure):
    _fields_ = [("num_k_heads", ctypes.c_int32), ("num_v_heads", ctypes.c_int32),
                ("head_dim_k", ctypes.c_int32), ("head_dim_v", ctypes.c_int32),
                ("head_map", ctypes.c_int32), ("decay", ctypes.c_int32),
                ("flags", ctypes.c_uint32), ("scale", ctypes.c_float),
                ("l2_eps", ctypes.c_float), ("norm_eps", ctypes.c_float)]


class Inputs(ctypes.Structure):
    _fields_ = [("q", _VP), ("k", _VP), ("v", _VP),
                ("q_stride", ctypes.c_int64), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("qkv_dtype", ctypes.c_int32),
                ("a", _VP), ("b", _VP), ("ab_dtype", ctypes.c_int32),
                ("decay_param", _VP), ("dt_bias", _VP),
                ("g", _VP), ("beta", _VP),
                ("z", _VP), ("z_dtype", ctypes.c_int32), ("norm_weight", _VP)]


class ConvArgs(ctypes.Structure):
    _fields_ = [("kernel_size", ctypes.c_int32), ("weight", _VP), ("state_in", _VP),
                ("state_out", _VP)]


class LaunchInfo(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("waves", "lanes_per_row", "token_mode", "nontemporal", "carry_kind",
                 "slices_per_workgroup", "workgroups", "threads", "prep_workgroups")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class NormArgs(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("x", _VP), ("x_stride", ctypes.c_int64),
                ("residual", _VP), ("residual_stride", ctypes.c_int64),
                ("residual_out", _VP), ("residual_out_stride", ctypes.c_int64),
                ("weight", _VP), ("eps", ctypes.c_float), ("out_dtype", ctypes.c_int32),
                ("out", _VP), ("out_stride", ctypes.c_int64),
                ("out_q", _VP), ("out_q_stride", ctypes.c_int64), ("out_scale", _VP)]


class RopeArgs(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("tokens", "q_heads", "kv_heads", "head_dim", "rotary_dim",
                                              "layout", "dtype")] + \
        [("magnitude", ctypes.c_float), ("positions", _VP), ("inv_freq", _VP),
         ("q", _VP), ("q_stride", ctypes.c_int64), ("q_out", _VP), ("q_out_stride", ctypes.c_int64),
         ("k", _VP), ("k_stride", ctypes.c_int64), ("k_out", _VP), ("k_out_stride", ctypes.c_int64),
         ("v", _VP), ("v_stride", ctypes.c_int64), ("k_pages", _VP), ("v_pages", _VP),
         ("page_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
         ("page_size", ctypes.c_int32), ("slots", _VP)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("q_heads", ctypes.c_int32), ("kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("scale", ctypes.c_float),
                ("q", _VP), ("q_stride", ctypes.c_int64), ("out", _VP), ("out_stride", ctypes.c_int64),
                ("lse", _VP), ("k", _VP), ("v", _VP), ("k_stride", ctypes.c_int64),
                ("v_stride", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("table", _VP), ("table_stride", ctypes.c_int64)]


class PageArgs(ctypes.Structure):
    _fields_ = [("table", _VP), ("table_stride", ctypes.c_int64), ("rows", ctypes.c_int32),
                ("width", ctypes.c_int32), ("refs", _VP), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("data", _VP), ("num_planes", ctypes.c_int32),
                ("plane_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64),
                ("page_bytes", ctypes.c_int64)]


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


_LIB = None


def load() -> ctypes.CDLL:
    """Load libgdn.so from the package directory (raises if it is not built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -c 'import __graft_entry__ as g; g.build()'` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    lib.gdn_status_string.restype = ctypes.c_char_p
    lib.gdn_status_string.argtypes = [ctypes.c_int]
    lib.gdn_version.restype = ctypes.c_int32
    lib.gdn_conv_update.restype = ctypes.c_int
    lib.gdn_conv_update.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _VP,
                                    ctypes.c_int32, ctypes.c_int32, _VP, ctypes.c_int64, _VP, _VP,
                                    ctypes.c_int32, _VP, ctypes.c_int64, _VP]
    lib.gdn_decode_step.restype = ctypes.c_int
    lib.gdn_decode_step.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int32,
                                    ctypes.POINTER(Inputs), _VP, _VP, ctypes.c_int32,
                                    ctypes.c_int32, _VP, _VP]
    lib.gdn_decode_layer.restype = ctypes.c_int
    lib.gdn_decode_layer.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int32,
                                     ctypes.POINTER(ConvArgs), ctypes.POINTER(Inputs), _VP, _VP,
                                     ctypes.c_int32, ctypes.c_int32, _VP, _VP]
    lib.gdn_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_prefill_workspace_bytes.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32,
                                                ctypes.c_int32]
    lib.gdn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_prefill_chunked.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, _VP, _VP,
                                        ctypes.c_int32, ctypes.POINTER(Inputs), _VP,
                                        ctypes.c_int32, _VP, _VP, ctypes.c_size_t, _VP]
    lib.gdn_prefill_chunked_noalloc.restype = ctypes.c_int
    lib.gdn_prefill_chunked_noalloc.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, _VP, _VP,
                                                ctypes.c_int32, ctypes.POINTER(Inputs), _VP,
                                                ctypes.c_int32, _VP, _VP]
    lib.gdn_decode_launch_info.restype = ctypes.c_int
    lib.gdn_decode_launch_info.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, ctypes.c_int32,
                                           ctypes.c_int32, ctypes.POINTER(LaunchInfo)]
    lib.gdn_prefill_launch_info.restype = ctypes.c_int
    lib.gdn_prefill_launch_info.argtypes = [ctypes.POINTER(Dims), ctypes.c_int32, _VP,
                                            ctypes.c_int32, ctypes.c_int32,
                                            ctypes.POINTER(LaunchInfo)]
    lib.gdn_linattn_decode_step.restype = ctypes.c_int
    lib.gdn_linattn_decode_step.argtypes = lib.gdn_decode_step.argtypes
    lib.gdn_linattn_prefill_workspace_bytes.restype = ctypes.c_size_t
    lib.gdn_linattn_prefill_workspace_bytes.argtypes = lib.gdn_prefill_workspace_bytes.argtypes
    lib.gdn_linattn_prefill_chunked.restype = ctypes.c_int
    lib.gdn_linattn_prefill_chunked.argtypes = lib.gdn_prefill_chunked.argtypes
    lib.gdn_add_rms_norm.restype = ctypes.c_int
    lib.gdn_add_rms_norm.argtypes = [ctypes.POINTER(NormArgs), _VP]
    lib.gdn_quant_matmul.restype = ctypes.c_int
    lib.gdn_quant_matmul.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, _VP,
                                     ctypes.c_int64, _VP, _VP, ctypes.c_int64, _VP,
                                     ctypes.c_int32, _VP, ctypes.c_int64, _VP]
    lib.gdn_quant_matmul_launch_info.restype = ctypes.c_int
    lib.gdn_quant_matmul_launch_info.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                                 ctypes.POINTER(LaunchInfo)]
    i32, ptr = ctypes.c_int32, ctypes.POINTER
    for name, restype, argtypes in (
            ("gdn_rope", ctypes.c_int, [ptr(RopeArgs), _VP]),
            ("gdn_rope_frequencies", ctypes.c_int,
             [i32, ctypes.c_double, i32] + [ctypes.c_double] * 4 + [_VP, _VP]),
            ("gdn_attention_prefill_workspace_bytes", ctypes.c_size_t, [i32] * 5),
            ("gdn_attention_prefill", ctypes.c_int,
             [ptr(AttentionArgs), i32, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            ("gdn_attention_decode_workspace_bytes", ctypes.c_size_t, [i32] * 7),
            ("gdn_attention_decode", ctypes.c_int,
             [ptr(AttentionArgs), i32, i32, _VP, i32, _VP, i32, _VP, ctypes.c_size_t, _VP]),
            ("gdn_pages_free", ctypes.c_int, [ptr(PageArgs), i32, _VP, _VP, _VP]),
            ("gdn_pages_reserve", ctypes.c_int, [ptr(PageArgs), i32, _VP, _VP, _VP, _VP]),
            ("gdn_pages_workspace_bytes", ctypes.c_size_t, [i32]),
            ("gdn_pages_fork", ctypes.c_int,
             [ptr(PageArgs), i32, _VP, _VP, _VP, _VP, _VP, ctypes.c_size_t, _VP]),
            ("gdn_pages_compact", ctypes.c_int, [ptr(PageArgs), _VP, _VP, _VP, ctypes.c_size_t, _VP])):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = restype, argtypes
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    return load().gdn_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != GDN_OK:
        raise GdnError(status, what)


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensor must be on the GPU")
    return ctypes.c_void_p(t.data_ptr())


def _dt(t) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _stream(stream=None) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _row_view(t, width: int, name: str):
    """(tensor, row stride in elements) for a [rows, ..., width-elements] activation."""
    if t.dim() < 2:
        raise ValueError(f"{name}: need at least 2 dims")
    flat_inner = 1
    for s in t.shape[1:]:
        flat_inner *= s
    if flat_inner != width:
        raise ValueError(f"{name}: inner size {flat_inner} != {width}")
    # inner dims must be contiguous; the row stride may be larger (views into a mixed row)
    exp = 1
    for d in range(t.dim() - 1, 0, -1):
        if t.shape[d] != 1 and t.stride(d) != exp:
            raise ValueError(f"{name}: inner dims must be contiguous")
        exp *= t.shape[d]
    return t, t.stride(0)


def _cu_device(cu, device):
    """cu_seqlens as the device int32 [N+1] tensor the kernels read (a copy when the
    caller's tensor has another dtype or lives elsewhere)."""
    if cu is None:
        return None
    if cu.dtype.is_floating_point or cu.dim() != 1:
        raise TypeError("cu_seqlens must be a 1-d integer tensor")
    return cu.to(device=device, dtype=torch.int32).contiguous()


def _cu_host(cu):
    """cu_seqlens as a host int32 [N+1] tensor (the prefill validates it there)."""
    if cu.dtype.is_floating_point or cu.dim() != 1:
        raise TypeError("cu_seqlens must be a 1-d integer tensor")
    return cu.to(device="cpu", dtype=torch.int32).contiguous()


def _check_state(state, Hv, dv, dk):
    if state.dtype != torch.float32 or not state.is_contiguous():
        raise ValueError("state must be contiguous float32")
    if state.dim() != 4 or tuple(state.shape[1:]) != (Hv, dv, dk):
        raise ValueError(f"state must be [slots][{Hv}][{dv}][{dk}], got {tuple(state.shape)}")


def _check_out(out, rows, Hv, dv):
    if out.dtype not in _DT or not out.is_contiguous():
        raise ValueError("out must be contiguous f32, f16 or bf16")
    if out.numel() != rows * Hv * dv or out.shape[0] != rows:
        raise ValueError(f"out must be [{rows}][{Hv}][{dv}], got {tuple(out.shape)}")


def _check_conv(conv_weight, conv_state_in, conv_state_out, qdtype, slots, channels):
    K = conv_weight.shape[1] if conv_weight.dim() == 2 else -1
    if tuple(conv_weight.shape) != (channels, K):
        raise ValueError(f"conv_weight must be [{channels}][K]")
    for name, t in (("conv_weight", conv_weight), ("conv_state_in", conv_state_in),
                    ("conv_state_out", conv_state_out)):
        if t.dtype != qdtype or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous in q's dtype")
    for name, t in (("conv_state_in", conv_state_in), ("conv_state_out", conv_state_out)):
        if tuple(t.shape) != (slots, channels, K - 1):
            raise ValueError(f"{name} must be [{slots}][{channels}][{K - 1}]")


def _check_slots(state_slots, batch):
    if state_slots is None:
        return
    if state_slots.dtype != torch.int32 or not state_slots.is_contiguous() or \
            state_slots.numel() != batch:
        raise ValueError(f"state_slots must be a contiguous int32 [{batch}] tensor")


def make_dims(Hk, Hv, dk, dv, head_map, flags, decay=DECAY_LOG_RATE, scale=0.0, l2_eps=0.0,
              norm_eps=0.0) -> Dims:
    return Dims(Hk, Hv, dk, dv, head_map, decay, flags, scale, l2_eps, norm_eps)


def make_inputs(q, k, v, *, Hk, Hv, dk, dv, a=None, b=None, decay_param=None, dt_bias=None,
                g=None, beta=None, z=None, norm_weight=None):
    q, qs = _row_view(q, Hk * dk, "q")
    k, ks = _row_view(k, Hk * dk, "k")
    v, vs = _row_view(v, Hv * dv, "v")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share a dtype")
    keep = [q, k, v]
    inp = Inputs(q=_ptr(q), k=_ptr(k), v=_ptr(v), q_stride=qs, k_stride=ks, v_stride=vs,
                 qkv_dtype=_dt(q))
    if a is not None:
        for t in (a, b):
            if not t.is_contiguous():
                raise ValueError("a, b must be contiguous [tokens][Hv]")
        if decay_param.dtype != torch.float32 or dt_bias.dtype != torch.float32:
            raise TypeError("decay_param and dt_bias must be float32")
        inp.a, inp.b, inp.ab_dtype = _ptr(a), _ptr(b), _dt(a)
        inp.decay_param, inp.dt_bias = _ptr(decay_param), _ptr(dt_bias)
        keep += [a, b, decay_param, dt_bias]
    if g is not None:
        if g.dtype != torch.float32 or beta.dtype != torch.float32:
            raise TypeError("g and beta must be float32")
        if not (g.is_contiguous() and beta.is_contiguous()):
            raise ValueError("g, beta must be contiguous [tokens][Hv]")
        inp.g, inp.beta = _ptr(g), _ptr(beta)
        keep += [g, beta]
    if z is not None:
        if not z.is_contiguous():
            raise ValueError("z must be contiguous [tokens][Hv][dv]")
        if norm_weight.dtype != torch.float32:
            raise TypeError("norm_weight must be float32")
        inp.z, inp.z_dtype, inp.norm_weight = _ptr(z), _dt(z), _ptr(norm_weight)
        keep += [z, norm_weight]
    return inp, keep


def decode_launch_info(*, Hk, Hv, dk, dv, batch, tokens_per_seq=1, fused_conv=True,
                       head_map=MAP_TILED, flags=L2NORM_QK | RAW_GATES | GATED_NORM) -> dict:
    """The decode kernel gdn_decode_layer (fused_conv) or gdn_decode_step would run."""
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags)
    info = LaunchInfo()
    _check(load().gdn_decode_launch_info(ctypes.byref(dims), batch, tokens_per_seq,
                                         int(fused_conv), ctypes.byref(info)),
           "gdn_decode_launch_info")
    return info.as_dict()


def prefill_launch_info(lengths, *, Hk, Hv, dk, dv, compute_units, head_map=MAP_GROUPED,
                        flags=L2NORM_QK | RAW_GATES) -> dict:
    """The prefill kernels gdn_prefill_chunked would run for these sequence lengths
    on a device with `compute_units` CUs."""
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + int(n))
    arr = (ctypes.c_int32 * len(cu))(*cu)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags)
    info = LaunchInfo()
    _check(load().gdn_prefill_launch_info(ctypes.byref(dims), len(lengths), arr, cu[-1],
                                          compute_units, ctypes.byref(info)),
           "gdn_prefill_launch_info")
    return info.as_dict()


def quant_matmul_launch_info(M, N, K) -> dict:
    """The kernel gdn_quant_matmul would run: its workgroups and threads per workgroup."""
    info = LaunchInfo()
    _check(load().gdn_quant_matmul_launch_info(M, N, K, ctypes.byref(info)),
           "gdn_quant_matmul_launch_info")
    return info.as_dict()


def conv_update(x, weight, conv_state, *, cu_seqlens=None, num_seqs=None, y=None,
                y_dtype=torch.float32, stream=None):
    """Causal depthwise conv + SiLU over x [tokens][C] (rows may be strided),
    weight [C][K], conv_state [N][C][K-1] (updated in place). Returns y."""
    total, C = x.shape
    if x.stride(1) != 1:
        raise ValueError("x channels must be contiguous")
    K = weight.shape[1]
    N = conv_state.shape[0] if num_seqs is None else num_seqs
    if weight.dtype != x.dtype or conv_state.dtype != x.dtype:
        raise TypeError("weight and conv_state must have x's dtype")
    if not (weight.is_contiguous() and conv_state.is_contiguous()):
        raise ValueError("weight and conv_state must be contiguous")
    if tuple(weight.shape) != (C, K) or tuple(conv_state.shape[1:]) != (C, K - 1) or \
            conv_state.shape[0] < N:
        raise ValueError("weight must be [C][K] and conv_state [N][C][K-1]")
    cu_seqlens = _cu_device(cu_seqlens, x.device)
    if cu_seqlens is not None and cu_seqlens.numel() != N + 1:
        raise ValueError("cu_seqlens must hold N + 1 offsets")
    if y is None:
        y = torch.empty((total, C), dtype=y_dtype, device=x.device)
    if y.dim() != 2 or y.shape[0] != total or y.shape[1] < C or y.stride(1) != 1:
        raise ValueError("y must be [tokens][>= C] with contiguous channels")
    st = load().gdn_conv_update(C, K, N, _ptr(cu_seqlens), total, _dt(x), _ptr(x), x.stride(0),
                                _ptr(weight), _ptr(conv_state), _dt(y), _ptr(y), y.stride(0),
                                _stream(stream))
    _check(st, "gdn_conv_update")
    return y


def decode_step(q, k, v, state, *, Hk, Hv, dk, dv, head_map, batch, tokens_per_seq=1,
                a=None, b=None, decay_param=None, dt_bias=None, g=None, beta=None, z=None,
                norm_weight=None, l2norm_qk=True, decay=DECAY_LOG_RATE, scale=0.0,
                state_slots=None, out=None, out_dtype=torch.float32, stream_state=False,
                stream=None):
    """One call of gdn_decode_step. q, k [B*T][Hk*dk] (views allowed), v [B*T][Hv*dv],
    state [slots][Hv][dv][dk] f32 updated in place. Returns out [B*T][Hv][dv].
    stream_state sets GDN_STREAM_STATE (non-temporal state loads and stores)."""
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0) | (STREAM_STATE if stream_state else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    _check_state(state, Hv, dv, dk)
    rows = batch * tokens_per_seq
    if out is None:
        out = torch.empty((rows, Hv, dv), dtype=out_dtype, device=state.device)
    _check_out(out, rows, Hv, dv)
    _check_slots(state_slots, batch)
    num_slots = state.shape[0]
    st = load().gdn_decode_step(ctypes.byref(dims), batch, tokens_per_seq, ctypes.byref(inp),
                                _ptr(state), _ptr(state_slots), num_slots, _dt(out), _ptr(out),
                                _stream(stream))
    _check(st, "gdn_decode_step")
    del keep
    return out


def decode_layer(q, k, v, state, conv_weight, conv_state_in, conv_state_out, *, Hk, Hv, dk, dv,
                 head_map, batch, tokens_per_seq=1, a=None, b=None, decay_param=None,
                 dt_bias=None, g=None, beta=None, z=None, norm_weight=None, l2norm_qk=True,
                 decay=DECAY_LOG_RATE, scale=0.0, state_slots=None, out=None,
                 out_dtype=torch.float32, stream_state=False, stream=None):
    """One call of gdn_decode_layer: q, k, v are the pre-conv projections (views of
    the mixed row allowed); conv_weight [channels][4], conv states [slots][channels][3]
    in q's dtype (read from conv_state_in, the new window written to conv_state_out);
    state [slots][Hv][dv][dk] f32 updated in place. Returns out [B*T][Hv][dv].
    stream_state sets GDN_STREAM_STATE (non-temporal state loads and stores)."""
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0) | (STREAM_STATE if stream_state else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    _check_state(state, Hv, dv, dk)
    _check_conv(conv_weight, conv_state_in, conv_state_out, q.dtype, state.shape[0],
                2 * Hk * dk + Hv * dv)
    conv = ConvArgs(conv_weight.shape[1], _ptr(conv_weight), _ptr(conv_state_in),
                    _ptr(conv_state_out))
    rows = batch * tokens_per_seq
    if out is None:
        out = torch.empty((rows, Hv, dv), dtype=out_dtype, device=state.device)
    _check_out(out, rows, Hv, dv)
    _check_slots(state_slots, batch)
    st = load().gdn_decode_layer(ctypes.byref(dims), batch, tokens_per_seq, ctypes.byref(conv),
                                 ctypes.byref(inp), _ptr(state), _ptr(state_slots), state.shape[0],
                                 _dt(out), _ptr(out), _stream(stream))
    _check(st, "gdn_decode_layer")
    del keep
    return out


def prefill_workspace_bytes(*, Hk, Hv, dk, dv, head_map=MAP_GROUPED, num_seqs, total_tokens,
                            gated_norm=False, flags=None):
    """Workspace gdn_prefill_chunked needs; the gated norm needs more, so pass
    gated_norm=True (or the call's flags) for calls that apply it."""
    if flags is None:
        flags = GATED_NORM if gated_norm else 0
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags)
    return int(load().gdn_prefill_workspace_bytes(ctypes.byref(dims), num_seqs, total_tokens))


def prefill_chunked(q, k, v, state, cu_seqlens, *, Hk, Hv, dk, dv, head_map, a=None, b=None,
                    decay_param=None, dt_bias=None, g=None, beta=None, z=None, norm_weight=None,
                    l2norm_qk=True, decay=DECAY_LOG_RATE, scale=0.0, out=None,
                    out_dtype=torch.float32, workspace=None, cu_seqlens_host=None, stream=None):
    """One call of gdn_prefill_chunked over packed sequences (cu_seqlens int32 [N+1]).
    state [N][Hv][dv][dk] f32: initial in, final out. Returns out [tokens][Hv][dv]."""
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    cu_seqlens_host = _cu_host(cu_seqlens if cu_seqlens_host is None else cu_seqlens_host)
    cu_dev = _cu_device(cu_seqlens, state.device)
    if cu_dev.numel() != cu_seqlens_host.numel():
        raise ValueError("cu_seqlens and cu_seqlens_host differ in length")
    N = cu_seqlens_host.numel() - 1
    total = int(cu_seqlens_host[-1])
    _check_state(state, Hv, dv, dk)
    if state.shape[0] != N:
        raise ValueError(f"state must hold one slot per sequence ({N})")
    if out is None:
        out = torch.empty((total, Hv, dv), dtype=out_dtype, device=state.device)
    _check_out(out, total, Hv, dv)
    need = load().gdn_prefill_workspace_bytes(ctypes.byref(dims), N, total)
    if workspace is None:
        workspace = torch.empty(max(int(need), 256), dtype=torch.uint8, device=state.device)
    host_ptr = ctypes.c_void_p(cu_seqlens_host.data_ptr())
    st = load().gdn_prefill_chunked(ctypes.byref(dims), N, host_ptr, _ptr(cu_dev), total,
                                    ctypes.byref(inp), _ptr(state), _dt(out), _ptr(out),
                                    _ptr(workspace), workspace.numel() * workspace.element_size(),
                                    _stream(stream))
    _check(st, "gdn_prefill_chunked")
    del keep
    return out


def prefill_chunked_noalloc(q, k, v, state, cu_seqlens, out, *, cu_seqlens_host, Hk, Hv, dk, dv,
                            head_map, a=None, b=None, decay_param=None, dt_bias=None, g=None,
                            beta=None, z=None, norm_weight=None, l2norm_qk=True,
                            decay=DECAY_LOG_RATE, scale=0.0, stream=None):
    """One call of gdn_prefill_chunked_noalloc: the prefill with the library's static
    scratch as its workspace. The caller passes every buffer, out included, and the
    offsets on both sides (int32 [N+1] on the GPU and on the host), so the binding
    itself allocates nothing. Returns out."""
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    for name, t, dev in (("cu_seqlens", cu_seqlens, True), ("cu_seqlens_host", cu_seqlens_host, False)):
        if t.dtype != torch.int32 or not t.is_contiguous() or t.is_cuda != dev:
            raise ValueError(f"{name} must be a contiguous int32 tensor on the "
                             f"{'GPU' if dev else 'host'}")
    N = cu_seqlens_host.numel() - 1
    total = int(cu_seqlens_host[-1])
    _check_state(state, Hv, dv, dk)
    _check_out(out, total, Hv, dv)
    st = load().gdn_prefill_chunked_noalloc(ctypes.byref(dims), N,
                                            ctypes.c_void_p(cu_seqlens_host.data_ptr()),
                                            _ptr(cu_seqlens), total, ctypes.byref(inp),
                                            _ptr(state), _dt(out), _ptr(out), _stream(stream))
    _check(st, "gdn_prefill_chunked_noalloc")
    del keep
    return out


class PreparedCall:
    """A library call with its ctypes arguments built once; ``launch()`` re-issues
    it on the stream captured at preparation time (for tight timing loops and
    graph capture, where per-call Python marshalling would dominate)."""

    def __init__(self, fn, args, what, keep):
        self._fn, self._args, self._what, self._keep = fn, args, what, keep

    def launch(self):
        st = self._fn(*self._args)
        if st != GDN_OK:
            raise GdnError(st, self._what)


def prepare_conv_update(x, weight, conv_state, y, *, cu_seqlens=None, num_seqs=None,
                        stream=None) -> PreparedCall:
    total, C = x.shape
    N = conv_state.shape[0] if num_seqs is None else num_seqs
    cu_seqlens = _cu_device(cu_seqlens, x.device)
    args = (C, weight.shape[1], N, _ptr(cu_seqlens), total, _dt(x), _ptr(x), x.stride(0),
            _ptr(weight), _ptr(conv_state), _dt(y), _ptr(y), y.stride(0), _stream(stream))
    return PreparedCall(load().gdn_conv_update, args, "gdn_conv_update",
                        [x, weight, conv_state, y, cu_seqlens])


def prepare_decode_step(q, k, v, state, out, *, Hk, Hv, dk, dv, head_map, batch,
                        tokens_per_seq=1, a=None, b=None, decay_param=None, dt_bias=None,
                        g=None, beta=None, z=None, norm_weight=None, l2norm_qk=True,
                        decay=DECAY_LOG_RATE, scale=0.0, state_slots=None,
                        stream_state=False, stream=None) -> PreparedCall:
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0) | (STREAM_STATE if stream_state else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    _check_state(state, Hv, dv, dk)
    _check_out(out, batch * tokens_per_seq, Hv, dv)
    _check_slots(state_slots, batch)
    args = (ctypes.byref(dims), batch, tokens_per_seq, ctypes.byref(inp), _ptr(state),
            _ptr(state_slots), state.shape[0], _dt(out), _ptr(out), _stream(stream))
    return PreparedCall(load().gdn_decode_step, args, "gdn_decode_step",
                        keep + [dims, inp, state, out, state_slots])


def prepare_decode_layer(q, k, v, state, conv_weight, conv_state_in, conv_state_out, out, *, Hk,
                         Hv, dk, dv, head_map, batch, tokens_per_seq=1, a=None, b=None,
                         decay_param=None, dt_bias=None, g=None, beta=None, z=None,
                         norm_weight=None, l2norm_qk=True, decay=DECAY_LOG_RATE, scale=0.0,
                         state_slots=None, stream_state=False, stream=None) -> PreparedCall:
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0) | (STREAM_STATE if stream_state else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    _check_state(state, Hv, dv, dk)
    _check_conv(conv_weight, conv_state_in, conv_state_out, q.dtype, state.shape[0],
                2 * Hk * dk + Hv * dv)
    _check_out(out, batch * tokens_per_seq, Hv, dv)
    _check_slots(state_slots, batch)
    conv = ConvArgs(conv_weight.shape[1], _ptr(conv_weight), _ptr(conv_state_in),
                    _ptr(conv_state_out))
    args = (ctypes.byref(dims), batch, tokens_per_seq, ctypes.byref(conv), ctypes.byref(inp),
            _ptr(state), _ptr(state_slots), state.shape[0], _dt(out), _ptr(out), _stream(stream))
    return PreparedCall(load().gdn_decode_layer, args, "gdn_decode_layer",
                        keep + [dims, inp, conv, state, out, state_slots, conv_weight,
                                conv_state_in, conv_state_out])


def prepare_prefill_chunked(q, k, v, state, cu_seqlens_dev, cu_seqlens_host, out, workspace, *,
                            Hk, Hv, dk, dv, head_map, a=None, b=None, decay_param=None,
                            dt_bias=None, g=None, beta=None, z=None, norm_weight=None,
                            l2norm_qk=True, decay=DECAY_LOG_RATE, scale=0.0,
                            stream=None) -> PreparedCall:
    flags = (L2NORM_QK if l2norm_qk else 0) | (RAW_GATES if a is not None else 0) | \
        (GATED_NORM if z is not None else 0)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv, a=a, b=b,
                            decay_param=decay_param, dt_bias=dt_bias, g=g, beta=beta, z=z,
                            norm_weight=norm_weight)
    if cu_seqlens_host.device.type != "cpu" or cu_seqlens_host.dtype != torch.int32:
        raise ValueError("cu_seqlens_host must be a CPU int32 tensor")
    cu_seqlens_dev = _cu_device(cu_seqlens_dev, state.device)
    N = cu_seqlens_host.numel() - 1
    total = int(cu_seqlens_host[-1])
    _check_state(state, Hv, dv, dk)
    _check_out(out, total, Hv, dv)
    args = (ctypes.byref(dims), N, ctypes.c_void_p(cu_seqlens_host.data_ptr()),
            _ptr(cu_seqlens_dev), total, ctypes.byref(inp), _ptr(state), _dt(out), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream))
    return PreparedCall(load().gdn_prefill_chunked, args, "gdn_prefill_chunked",
                        keep + [dims, inp, state, out, workspace, cu_seqlens_dev,
                                cu_seqlens_host])


# ---- decayed linear attention, residual RMS norm with 8-bit output, int8 product ----
# These calls run on the tensors' own device, whatever the current one is. What they
# allocate (outputs, workspaces, offset copies) is allocated on the stream they run on,
# so its memory is not handed out again before the kernels have read it. As for torch's own
# operators, tensors of another stream are ready, and kept until the call has run, by the caller.

def _device_of(**tensors):
    """The one GPU that every given tensor is on."""
    device = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be on the GPU")
        if device is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, other tensors are on {device}")
        device = t.device
    return device


class _RunOn:
    """The device and stream a call runs on, made current while it is prepared and
    issued. stream: the caller's, or the current stream of the tensors' device."""

    def __init__(self, device, stream):
        if stream is None:
            stream = torch.cuda.current_stream(device)
        elif stream.device != device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
        self.handle = ctypes.c_void_p(stream.cuda_stream)
        self._context = torch.cuda.stream(stream)

    def __enter__(self):
        self._context.__enter__()
        return self.handle

    def __exit__(self, *exc):
        return self._context.__exit__(*exc)


class DeviceCall(PreparedCall):
    """A prepared call that is issued on its tensors' device, whatever the current
    device is. ``out`` is what the call returns."""

    def __init__(self, fn, args, what, keep, device, out):
        super().__init__(fn, args, what, keep)
        self._device, self.out = device, out

    def launch(self):
        if torch.cuda.current_device() == self._device.index:
            st = self._fn(*self._args)
        else:
            with torch.cuda.device(self._device):
                st = self._fn(*self._args)
        if st != GDN_OK:
            raise GdnError(st, self._what)


def _linattn_args(q, k, v, state, out, tokens, *, Hk, Hv, dk, dv, head_map, g, decay_param, decay,
                  scale, stream_state=False):
    """(dims, inputs, tensors to keep) of a gdn_linattn_* call over `tokens` rows."""
    if (g is None) == (decay_param is None):
        raise ValueError("give g [tokens][Hv] or decay_param [Hv], one of the two")
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t.dim() < 2 or t.shape[0] != tokens:
            raise ValueError(f"{name} must have {tokens} token rows, got {tuple(t.shape)}")
    inp, keep = make_inputs(q, k, v, Hk=Hk, Hv=Hv, dk=dk, dv=dv)
    flags = STREAM_STATE if stream_state else 0
    name, t, shape = ("g", g, (tokens, Hv)) if decay_param is None else ("decay_param", decay_param, (Hv,))
    if t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape:
        raise ValueError(f"{name} must be contiguous float32 {list(shape)}")
    if decay_param is None:
        inp.g = _ptr(t)
    else:
        inp.decay_param = _ptr(t)
        flags |= HEAD_DECAY
    _check_state(state, Hv, dv, dk)
    _check_out(out, tokens, Hv, dv)
    dims = make_dims(Hk, Hv, dk, dv, head_map, flags, decay, scale)
    return dims, inp, keep + [t, state, out]


def prepare_linattn_decode_step(q, k, v, state, out, *, Hk, Hv, dk, dv, head_map, batch,
                                tokens_per_seq=1, g=None, decay_param=None,
                                decay=DECAY_LOG_RATE, scale=0.0, state_slots=None,
                                stream_state=False, stream=None) -> DeviceCall:
    """linattn_decode_step with its arguments checked and marshalled once."""
    device = _device_of(state=state, q=q, k=k, v=v, out=out, g=g, decay_param=decay_param,
                        state_slots=state_slots)
    dims, inp, keep = _linattn_args(q, k, v, state, out, batch * tokens_per_seq, Hk=Hk, Hv=Hv,
                                    dk=dk, dv=dv, head_map=head_map, g=g, decay_param=decay_param,
                                    decay=decay, scale=scale, stream_state=stream_state)
    _check_slots(state_slots, batch)
    args = (ctypes.byref(dims), batch, tokens_per_seq, ctypes.byref(inp), _ptr(state),
            _ptr(state_slots), state.shape[0], _dt(out), _ptr(out), _RunOn(device, stream).handle)
    return DeviceCall(load().gdn_linattn_decode_step, args, "gdn_linattn_decode_step",
                      keep + [dims, inp, state_slots], device, out)


def linattn_decode_step(q, k, v, state, *, Hk, Hv, dk, dv, head_map, batch, tokens_per_seq=1,
                        g=None, decay_param=None, decay=DECAY_LOG_RATE, scale=0.0,
                        state_slots=None, out=None, out_dtype=torch.float32, stream_state=False,
                        stream=None):
    """One call of gdn_linattn_decode_step: S <- exp(g) S + v k^T, o = scale (S q) for each
    token. q, k [B*T][Hk*dk], v [B*T][Hv*dv] (views of a mixed row allowed); the log decay is
    g [B*T][Hv] f32, or one rate per head from decay_param [Hv] f32; state [slots][Hv][dv][dk]
    f32 updated in place, the slots of one call distinct. Returns out [B*T][Hv][dv]."""
    with _RunOn(_device_of(state=state), stream):
        if out is None:
            out = torch.empty((batch * tokens_per_seq, Hv, dv), dtype=out_dtype, device=state.device)
        prepare_linattn_decode_step(q, k, v, state, out, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                                    head_map=head_map, batch=batch, tokens_per_seq=tokens_per_seq,
                                    g=g, decay_param=decay_param, decay=decay, scale=scale,
                                    state_slots=state_slots, stream_state=stream_state).launch()
    return out


def linattn_prefill_workspace_bytes(*, Hk, Hv, dk, dv, num_seqs, total_tokens,
                                    head_map=MAP_GROUPED):
    """Workspace gdn_linattn_prefill_chunked needs."""
    dims = make_dims(Hk, Hv, dk, dv, head_map, 0)
    return int(load().gdn_linattn_prefill_workspace_bytes(ctypes.byref(dims), num_seqs, total_tokens))


def prepare_linattn_prefill_chunked(q, k, v, state, cu_seqlens_dev, cu_seqlens_host, out, workspace,
                                    *, Hk, Hv, dk, dv, head_map, g=None, decay_param=None,
                                    decay=DECAY_LOG_RATE, scale=0.0, stream=None) -> DeviceCall:
    """linattn_prefill_chunked with its arguments checked and marshalled once: the offsets as
    int32 [N+1] tensors on the GPU and on the host, the workspace a contiguous uint8 tensor."""
    device = _device_of(state=state, q=q, k=k, v=v, out=out, g=g, decay_param=decay_param,
                        cu_seqlens_dev=cu_seqlens_dev, workspace=workspace)
    for name, t in (("cu_seqlens_dev", cu_seqlens_dev), ("cu_seqlens_host", cu_seqlens_host)):
        if t.dtype != torch.int32 or t.dim() != 1 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous 1-d int32 tensor")
    if cu_seqlens_host.device.type != "cpu" or cu_seqlens_host.numel() != cu_seqlens_dev.numel() or \
            cu_seqlens_host.numel() < 1:
        raise ValueError("cu_seqlens_host must hold cu_seqlens_dev's offsets on the host")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    N, total = cu_seqlens_host.numel() - 1, int(cu_seqlens_host[-1])
    if state.shape[0] != N:
        raise ValueError(f"state must hold one slot per sequence ({N})")
    dims, inp, keep = _linattn_args(q, k, v, state, out, total, Hk=Hk, Hv=Hv, dk=dk, dv=dv,
                                    head_map=head_map, g=g, decay_param=decay_param, decay=decay,
                                    scale=scale)
    args = (ctypes.byref(dims), N, ctypes.c_void_p(cu_seqlens_host.data_ptr()),
            _ptr(cu_seqlens_dev), total, ctypes.byref(inp), _ptr(state), _dt(out), _ptr(out),
            _ptr(workspace), workspace.numel() * workspace.element_size(),
            _RunOn(device, stream).handle)
    return DeviceCall(load().gdn_linattn_prefill_chunked, args, "gdn_linattn_prefill_chunked",
                      keep + [dims, inp, workspace, cu_seqlens_dev, cu_seqlens_host], device, out)


def linattn_prefill_chunked(q, k, v, state, cu_seqlens, *, Hk, Hv, dk, dv, head_map, g=None,
                            decay_param=None, decay=DECAY_LOG_RATE, scale=0.0, out=None,
                            out_dtype=torch.float32, workspace=None, cu_seqlens_host=None,
                            stream=None):
    """One call of gdn_linattn_prefill_chunked over packed sequences (cu_seqlens integer [N+1],
    on either side; cu_seqlens_host saves the copy to the host). The log decay is
    g [tokens][Hv] f32 or one rate per head from decay_param [Hv] f32. state [N][Hv][dv][dk] f32:
    initial in, final out. Returns out [tokens][Hv][dv]."""
    with _RunOn(_device_of(state=state), stream):
        cu_host = _cu_host(cu_seqlens if cu_seqlens_host is None else cu_seqlens_host)
        cu_dev = _cu_device(cu_seqlens, state.device)
        N, total = cu_host.numel() - 1, int(cu_host[-1]) if cu_host.numel() else 0
        if out is None:
            out = torch.empty((total, Hv, dv), dtype=out_dtype, device=state.device)
        if workspace is None:
            need = linattn_prefill_workspace_bytes(Hk=Hk, Hv=Hv, dk=dk, dv=dv, num_seqs=N,
                                                   total_tokens=total)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=state.device)
        prepare_linattn_prefill_chunked(q, k, v, state, cu_dev, cu_host, out, workspace, Hk=Hk,
                                        Hv=Hv, dk=dk, dv=dv, head_map=head_map, g=g,
                                        decay_param=decay_param, decay=decay, scale=scale).launch()
    return out


def _rows(name, t, rows, hidden, dtypes):
    if max(rows, hidden) > 2 ** 31 - 1:
        raise ValueError(f"{name}: counts must fit 32 bits")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.dim() != 2 or tuple(t.shape) != (rows, hidden) or (hidden > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be [{rows}][{hidden}] with contiguous rows, "
                         f"got {tuple(t.shape)}")
    return t.stride(0) if rows > 1 else hidden


def prepare_add_rms_norm(x, weight, *, residual=None, residual_out=None, out=None, out_q=None,
                         out_scale=None, eps=0.0, stream=None) -> DeviceCall:
    """add_rms_norm into the caller's buffers, checked and marshalled once: residual_out
    [rows][hidden] (x's or residual's own buffer allowed), out [rows][hidden], out_q int8
    [rows][hidden] with out_scale [rows] f32; each may be None, out and out_q not both."""
    device = _device_of(x=x, weight=weight, residual=residual, residual_out=residual_out, out=out,
                        out_q=out_q, out_scale=out_scale)
    if x.dim() != 2:
        raise ValueError("x must be [rows][hidden]")
    rows, hidden = x.shape
    args = NormArgs(rows=rows, hidden=hidden, dtype=_dt(x), x=_ptr(x),
                    x_stride=_rows("x", x, rows, hidden, _DT), weight=_ptr(weight), eps=eps)
    if weight.dtype != torch.float32 or not weight.is_contiguous() or tuple(weight.shape) != (hidden,):
        raise ValueError(f"weight must be contiguous float32 [{hidden}]")
    if residual is not None:
        args.residual, args.residual_stride = _ptr(residual), _rows("residual", residual, rows, hidden, (x.dtype,))
    if residual_out is not None:
        args.residual_out = _ptr(residual_out)
        args.residual_out_stride = _rows("residual_out", residual_out, rows, hidden, (x.dtype,))
    if out is not None:
        args.out, args.out_dtype, args.out_stride = _ptr(out), _dt(out), _rows("out", out, rows, hidden, _DT)
    if out_q is not None:
        args.out_q, args.out_q_stride = _ptr(out_q), _rows("out_q", out_q, rows, hidden, (torch.int8,))
    if out_scale is not None:
        if out_scale.dtype != torch.float32 or not out_scale.is_contiguous() or tuple(out_scale.shape) != (rows,):
            raise ValueError(f"out_scale must be contiguous float32 [{rows}]")
        args.out_scale = _ptr(out_scale)
    return DeviceCall(load().gdn_add_rms_norm, (ctypes.byref(args), _RunOn(device, stream).handle),
                      "gdn_add_rms_norm",
                      [args, x, weight, residual, residual_out, out, out_q, out_scale], device,
                      (out, residual_out, out_q, out_scale))


def add_rms_norm(x, weight, *, residual=None, residual_out=None, out=None, out_dtype=None,
                 quantize=False, eps=0.0, stream=None):
    """One call of gdn_add_rms_norm: h = x + residual; y = h rsqrt(mean h^2 + eps) weight.
    x, residual [rows][hidden] (rows may be strided), weight [hidden] f32. Returns a dict of
    new tensors: `out` y in out_dtype (default x's; with quantize only if out_dtype is given),
    `residual` h (with a residual; in residual_out if given, which may be x or residual
    itself), and with quantize `out_q` int8 and `out_scale` [rows] f32, ready for quant_matmul."""
    with _RunOn(_device_of(x=x), stream):
        if x.dim() != 2:
            raise ValueError("x must be [rows][hidden]")
        rows, hidden = x.shape
        new = lambda dtype, *shape: torch.empty(shape, dtype=dtype, device=x.device)  # noqa: E731
        if out is None and (out_dtype is not None or not quantize):
            out = new(out_dtype or x.dtype, rows, hidden)
        if residual is not None and residual_out is None:
            residual_out = new(x.dtype, rows, hidden)
        out_q, out_scale = (new(torch.int8, rows, hidden), new(torch.float32, rows)) if quantize else (None, None)
        prepare_add_rms_norm(x, weight, residual=residual, residual_out=residual_out, out=out,
                             out_q=out_q, out_scale=out_scale, eps=eps).launch()
    got = dict(out=out, residual=residual_out, out_q=out_q, out_scale=out_scale)
    return {name: t for name, t in got.items() if t is not None}


def prepare_quant_matmul(a, a_scale, w, w_scale, out, *, stream=None) -> DeviceCall:
    """quant_matmul into the caller's out [M][N], checked and marshalled once."""
    device = _device_of(a=a, a_scale=a_scale, w=w, w_scale=w_scale, out=out)
    if a.dim() != 2 or w.dim() != 2 or a.shape[1] != w.shape[1]:
        raise ValueError("a must be [M][K] and w [N][K]")
    (M, K), N = a.shape, w.shape[0]
    strides = [_rows("a", a, M, K, (torch.int8,)), _rows("w", w, N, K, (torch.int8,)),
               _rows("out", out, M, N, _DT)]
    for name, t, n in (("a_scale", a_scale, M), ("w_scale", w_scale, N)):
        if t.dtype != torch.float32 or not t.is_contiguous() or t.numel() != n:
            raise ValueError(f"{name} must be contiguous float32 [{n}]")
    args = (M, N, K, _ptr(a), strides[0], _ptr(a_scale), _ptr(w), strides[1], _ptr(w_scale), _dt(out),
            _ptr(out), strides[2], _RunOn(device, stream).handle)
    return DeviceCall(load().gdn_quant_matmul, args, "gdn_quant_matmul",
                      [a, a_scale, w, w_scale, out], device, out)


def quant_matmul(a, a_scale, w, w_scale, *, out=None, out_dtype=torch.bfloat16, stream=None):
    """One call of gdn_quant_matmul: out[m][n] = (sum_k a[m][k] w[n][k]) a_scale[m] w_scale[n].
    a [M][K] and w [N][K] int8 (rows may be strided by multiples of 16 bytes), a_scale [M] and
    w_scale [N] f32. Returns out [M][N]."""
    with _RunOn(_device_of(a=a), stream):
        if out is None:
            out = torch.empty((a.shape[0], w.shape[0]), dtype=out_dtype, device=a.device)
        prepare_quant_matmul(a, a_scale, w, w_scale, out).launch()
    return out


# ---- softmax attention layers: rotary positions, attention, the pages of the cache ----

def rope_frequencies(rotary_dim, theta=10000.0, *, scaling=ROPE_PLAIN, factor=1.0, original_length=0.0,
                     beta_fast=32.0, beta_slow=1.0):
    """The frequencies of gdn_rope_frequencies: (inv_freq [rotary_dim / 2] f64 on the host, magnitude)."""
    inv_freq = torch.empty(max(int(rotary_dim) // 2, 1), dtype=torch.float64)
    magnitude = ctypes.c_float()
    st = load().gdn_rope_frequencies(rotary_dim, theta, scaling, factor, original_length, beta_fast,
                                     beta_slow, ctypes.c_void_p(inv_freq.data_ptr()), ctypes.byref(magnitude))
    _check(st, "gdn_rope_frequencies")
    return inv_freq, magnitude.value


def _i32(name, t, *shape):
    """A contiguous int32 tensor of the shape; None in it is any size."""
    if t.dtype != torch.int32 or t.dim() != len(shape) or not t.is_contiguous() or \
            any(want is not None and n != want for n, want in zip(t.shape, shape)):
        raise ValueError(f"{name} must be contiguous int32 {['any' if n is None else n for n in shape]}, "
                         f"got {t.dtype} {list(t.shape)}")
    return t


def _head_rows(name, t, rows, heads, dim, dtype):
    """Row stride of t [rows][heads][dim], whose rows may be strided."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 3 or tuple(t.shape) != (rows, heads, dim):
        raise ValueError(f"{name} must be [{rows}][{heads}][{dim}], got {list(t.shape)}")
    if t.numel() > 0 and ((dim > 1 and t.stride(2) != 1) or (heads > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name}: the heads of a row must be contiguous")
    return t.stride(0) if rows > 1 else heads * dim


def _page_pool(name, t, heads, dim, dtype):
    """Page stride of the pool t [pages][heads][page_size][dim], whose pages may be strided."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 4 or t.shape[1] != heads or t.shape[3] != dim:
        raise ValueError(f"{name} must be [pages][{heads}][page_size][{dim}], got {list(t.shape)}")
    page = heads * t.shape[2] * dim
    if t.numel() > 0 and not t[0].is_contiguous():
        raise ValueError(f"{name}: a page must be contiguous")
    return t.stride(0) if t.shape[0] > 1 else page


def prepare_rope(positions, inv_freq, *, q=None, q_out=None, k=None, k_out=None, v=None, k_pages=None,
                 v_pages=None, slots=None, layout=ROPE_HALF, magnitude=1.0, stream=None) -> DeviceCall:
    """rope into the caller's buffers, checked and marshalled once: q_out and k_out like q and k (their
    own buffers allowed), or for k and v page pools [pages][kv_heads][page_size][head_dim] with
    slots [tokens] int32."""
    device = _device_of(positions=positions, inv_freq=inv_freq, q=q, q_out=q_out, k=k, k_out=k_out, v=v,
                        k_pages=k_pages, v_pages=v_pages, slots=slots)
    given = q if q is not None else k
    if given is None:
        raise ValueError("give q, k or both")
    if given.dim() != 3:
        raise ValueError("q and k must be [tokens][heads][head_dim]")
    tokens, _, dim = given.shape
    _i32("positions", positions, tokens)
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be contiguous float64 [rotary_dim / 2]")
    if magnitude == 0:
        raise ValueError("magnitude must not be 0")
    args = RopeArgs(tokens=tokens, head_dim=dim, rotary_dim=2 * inv_freq.numel(), layout=layout, dtype=_dt(given),
                    magnitude=magnitude, positions=_ptr(positions), inv_freq=_ptr(inv_freq))
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    if q is not None:
        args.q_heads = q.shape[1]
        args.q, args.q_stride = _ptr(q), _head_rows("q", q, tokens, args.q_heads, dim, given.dtype)
        args.q_out, args.q_out_stride = _ptr(q_out), _head_rows("q_out", q_out, tokens, args.q_heads, dim, given.dtype)
    paged = [t is not None for t in (k_pages, v_pages, slots, v)]
    if any(paged) and (not all(paged) or k is None or k_out is not None):
        raise ValueError("k_pages, v_pages, slots, k and v go together, without k_out")
    if not any(paged) and (k is None) != (k_out is None):
        raise ValueError("k goes to k_out or to pages")
    if k is not None:
        args.kv_heads = k.shape[1] if k.dim() == 3 else 0
        args.k, args.k_stride = _ptr(k), _head_rows("k", k, tokens, args.kv_heads, dim, given.dtype)
    if k_out is not None:
        args.k_out, args.k_out_stride = _ptr(k_out), _head_rows("k_out", k_out, tokens, args.kv_heads, dim, given.dtype)
    if k_pages is not None:
        args.v, args.v_stride = _ptr(v), _head_rows("v", v, tokens, args.kv_heads, dim, given.dtype)
        args.k_pages, args.v_pages = _ptr(k_pages), _ptr(v_pages)
        args.page_stride = _page_pool("k_pages", k_pages, args.kv_heads, dim, given.dtype)
        if _page_pool("v_pages", v_pages, args.kv_heads, dim, given.dtype) != args.page_stride or \
                k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must have one shape and stride")
        args.num_pages, args.page_size = k_pages.shape[0], k_pages.shape[2]
        args.slots = _ptr(_i32("slots", slots, tokens))
    return DeviceCall(load().gdn_rope, (ctypes.byref(args), _RunOn(device, stream).handle), "gdn_rope",
                      [args, positions, inv_freq, q, q_out, k, k_out, v, k_pages, v_pages, slots], device,
                      (q_out, k_out))


def rope(positions, inv_freq, *, q=None, k=None, v=None, k_pages=None, v_pages=None, slots=None,
         layout=ROPE_HALF, magnitude=1.0, stream=None):
    """One call of gdn_rope: turns the first 2 * len(inv_freq) elements of each head of q and k
    [tokens][heads][head_dim] (views of a mixed row allowed) by their positions [tokens] int32. With
    pages, k and v are stored in the slots and only q is returned; else new (q, k), None for one
    not given."""
    with _RunOn(_device_of(positions=positions), stream):
        q_out = None if q is None else torch.empty(q.shape, dtype=q.dtype, device=q.device)
        k_out = None if k is None or k_pages is not None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        prepare_rope(positions, inv_freq, q=q, q_out=q_out, k=k, k_out=k_out, v=v, k_pages=k_pages,
                     v_pages=v_pages, slots=slots, layout=layout, magnitude=magnitude).launch()
    return q_out if k_pages is not None else (q_out, k_out)


def _attention_args(q, k, v, out, lse, table, scale):
    """AttentionArgs of queries q [rows][q_heads][head_dim] and packed rows or, with a table, page pools."""
    if q.dim() != 3 or k.dim() != (3 if table is None else 4) or k.shape[-1] != q.shape[2]:
        raise ValueError("q must be [rows][q_heads][head_dim], k and v [keys][kv_heads][head_dim] or "
                         "[pages][kv_heads][page_size][head_dim] with a table")
    rows, Hq, dim = q.shape
    Hkv = k.shape[1]
    args = AttentionArgs(q_heads=Hq, kv_heads=Hkv, head_dim=dim, dtype=_dt(q), scale=scale, q=_ptr(q),
                         q_stride=_head_rows("q", q, rows, Hq, dim, q.dtype), out=_ptr(out),
                         out_stride=_head_rows("out", out, rows, Hq, dim, q.dtype), k=_ptr(k), v=_ptr(v))
    if lse is not None:
        if lse.dtype != torch.float32 or not lse.is_contiguous() or tuple(lse.shape) != (rows, Hq):
            raise ValueError(f"lse must be contiguous float32 [{rows}][{Hq}]")
        args.lse = _ptr(lse)
    if k.shape != v.shape:
        raise ValueError("k and v must have one shape")
    if table is None:
        args.k_stride = _head_rows("k", k, k.shape[0], Hkv, dim, q.dtype)
        args.v_stride = _head_rows("v", v, k.shape[0], Hkv, dim, q.dtype)
    else:
        args.k_stride = _page_pool("k", k, Hkv, dim, q.dtype)
        args.v_stride = _page_pool("v", v, Hkv, dim, q.dtype)
        args.num_pages, args.page_size = k.shape[0], k.shape[2]
        if table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table must be int32 [sequences][entries] with contiguous rows")
        args.table = _ptr(table)
        args.table_stride = table.stride(0) if table.shape[0] > 1 else table.shape[1]
        if args.table_stride < table.shape[1]:
            raise ValueError("table: rows overlap")
    return args


def _workspace(workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def attention_prefill_workspace_bytes(*, Hq, Hkv, head_dim, num_seqs, total_tokens):
    """Workspace gdn_attention_prefill needs for total_tokens queries."""
    return int(load().gdn_attention_prefill_workspace_bytes(Hq, Hkv, head_dim, num_seqs, total_tokens))


def prepare_attention_prefill(q, k, v, cu_q, cu_q_host, out, workspace, *, cu_k=None, cu_k_host=None,
                              table=None, lse=None, scale=0.0, stream=None) -> DeviceCall:
    """attention_prefill with its arguments checked and marshalled once: the offsets as int32 [N+1]
    tensors on the GPU and on the host, the workspace a contiguous uint8 tensor (None where none is needed)."""
    device = _device_of(q=q, k=k, v=v, cu_q=cu_q, out=out, workspace=workspace, cu_k=cu_k, table=table, lse=lse)
    if (cu_k is None) != (cu_k_host is None):
        raise ValueError("cu_k and cu_k_host go together")
    for name, t, host in (("cu_q", cu_q, cu_q_host), ("cu_k", cu_k, cu_k_host)):
        if t is None:
            continue
        _i32(name, t, None)
        _i32(name + "_host", host, t.numel())
        if host.device.type != "cpu" or t.numel() != cu_q.numel() or t.numel() < 1:
            raise ValueError(f"{name}_host must hold {name}'s offsets on the host, one more than sequences")
    args = _attention_args(q, k, v, out, lse, table, scale)
    N = cu_q.numel() - 1
    cu_keys = cu_q_host if cu_k_host is None else cu_k_host
    if q.shape[0] < int(cu_q_host[-1]):
        raise ValueError(f"q must hold {int(cu_q_host[-1])} rows")
    if table is None and k.shape[0] < int(cu_keys[-1]):
        raise ValueError(f"k and v must hold {int(cu_keys[-1])} rows")
    if table is not None:
        longest = int(cu_keys.diff().max()) if N > 0 else 0
        if table.shape[0] != N or table.shape[1] * k.shape[2] < longest:
            raise ValueError(f"table must hold {N} rows of pages for {longest} tokens")
    ws, ws_bytes = _workspace(workspace)
    call = (ctypes.byref(args), N, ctypes.c_void_p(cu_q_host.data_ptr()), _ptr(cu_q),
            None if cu_k is None else ctypes.c_void_p(cu_k_host.data_ptr()), _ptr(cu_k), ws, ws_bytes,
            _RunOn(device, stream).handle)
    return DeviceCall(load().gdn_attention_prefill, call, "gdn_attention_prefill",
                      [args, q, k, v, cu_q, cu_q_host, out, workspace, cu_k, cu_k_host, table, lse], device, out)


def attention_prefill(q, k, v, cu_seqlens, *, cu_k=None, table=None, out=None, lse=None, scale=0.0,
                      workspace=None, cu_seqlens_host=None, cu_k_host=None, stream=None):
    """One call of gdn_attention_prefill: causal attention of packed prompts, q [tokens][q_heads][head_dim]
    (f16 or bf16, views of a mixed row allowed), cu_seqlens integer [N+1] on either side. k and v are packed
    rows [keys][kv_heads][head_dim], or page pools [pages][kv_heads][page_size][head_dim] with a table
    [N][entries] int32; cu_k are the offsets of the keys where they are not those of the queries (the
    queries are then the last ones of the keys). lse [tokens][q_heads] f32 receives the log-sums. Returns
    out [tokens][q_heads][head_dim]."""
    with _RunOn(_device_of(q=q), stream):
        host = _cu_host(cu_seqlens if cu_seqlens_host is None else cu_seqlens_host)
        dev = _cu_device(cu_seqlens, q.device)
        k_host = k_dev = None
        if cu_k is not None:
            k_host = _cu_host(cu_k if cu_k_host is None else cu_k_host)
            k_dev = _cu_device(cu_k, q.device)
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if workspace is None and q.dim() == 3 and k.dim() > 2:
            need = attention_prefill_workspace_bytes(Hq=q.shape[1], Hkv=k.shape[1], head_dim=q.shape[2],
                                                     num_seqs=host.numel() - 1, total_tokens=int(host[-1]))
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        prepare_attention_prefill(q, k, v, dev, host, out, workspace, cu_k=k_dev, cu_k_host=k_host, table=table,
                                  lse=lse, scale=scale).launch()
    return out


def attention_decode_workspace_bytes(*, Hq, Hkv, head_dim, batch, tokens_per_seq=1, max_len, prefix_len=0):
    """Workspace gdn_attention_decode needs."""
    return int(load().gdn_attention_decode_workspace_bytes(Hq, Hkv, head_dim, batch, tokens_per_seq, max_len,
                                                           prefix_len))


def prepare_attention_decode(q, k_pages, v_pages, table, lens, out, workspace, *, batch, max_len,
                             tokens_per_seq=1, prefix_table=None, prefix_len=0, lse=None, scale=0.0,
                             stream=None) -> DeviceCall:
    """attention_decode with its arguments checked and marshalled once; the workspace a contiguous uint8
    tensor (None where none is needed). lens and the tables are read when the call runs."""
    device = _device_of(q=q, k_pages=k_pages, v_pages=v_pages, table=table, lens=lens, out=out,
                        workspace=workspace, prefix_table=prefix_table, lse=lse)
    if table is None:
        raise ValueError("the keys of a decode step are on pages: give a table")
    args = _attention_args(q, k_pages, v_pages, out, lse, table, scale)
    if q.shape[0] != batch * tokens_per_seq:
        raise ValueError(f"q must hold {batch * tokens_per_seq} rows")
    _i32("lens", lens, batch)
    if table.shape[0] < batch or table.shape[1] * k_pages.shape[2] < max_len:
        raise ValueError(f"table must hold {batch} rows of pages for {max_len} tokens")
    if (prefix_table is None) != (prefix_len == 0):
        raise ValueError("prefix_table and prefix_len go together")
    if prefix_table is not None:
        _i32("prefix_table", prefix_table, None)
        if prefix_table.numel() * k_pages.shape[2] < prefix_len:
            raise ValueError(f"prefix_table must hold pages for {prefix_len} tokens")
    ws, ws_bytes = _workspace(workspace)
    call = (ctypes.byref(args), batch, tokens_per_seq, _ptr(lens), max_len, _ptr(prefix_table), prefix_len, ws,
            ws_bytes, _RunOn(device, stream).handle)
    return DeviceCall(load().gdn_attention_decode, call, "gdn_attention_decode",
                      [args, q, k_pages, v_pages, table, lens, out, workspace, prefix_table, lse], device, out)


def attention_decode(q, k_pages, v_pages, table, lens, *, batch, max_len, tokens_per_seq=1, prefix_table=None,
                     prefix_len=0, out=None, lse=None, scale=0.0, workspace=None, stream=None):
    """One call of gdn_attention_decode: tokens_per_seq new queries of each sequence, q [B*T][q_heads]
    [head_dim], against a prefix that the batch shares (prefix_len tokens on the pages prefix_table) and each
    sequence's own lens[b] tokens (int32, on the GPU, the new ones among them, at most max_len) on the pages
    table[b]. Returns out [B*T][q_heads][head_dim]."""
    with _RunOn(_device_of(q=q), stream):
        if out is None:
            out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        if workspace is None and q.dim() == 3 and k_pages.dim() == 4:
            need = attention_decode_workspace_bytes(Hq=q.shape[1], Hkv=k_pages.shape[1], head_dim=q.shape[2],
                                                    batch=batch, tokens_per_seq=tokens_per_seq, max_len=max_len,
                                                    prefix_len=prefix_len)
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q.device)
        prepare_attention_decode(q, k_pages, v_pages, table, lens, out, workspace, batch=batch, max_len=max_len,
                                 tokens_per_seq=tokens_per_seq, prefix_table=prefix_table, prefix_len=prefix_len,
                                 lse=lse, scale=scale).launch()
    return out


def _page_args(table, refs, page_size=1, pool=None):
    if table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1) or \
            (table.shape[0] > 1 and table.stride(0) < table.shape[1]):
        raise ValueError("table must be int32 [rows][entries] with contiguous rows")
    _i32("refs", refs, None)
    args = PageArgs(table=_ptr(table), table_stride=table.stride(0) if table.shape[0] > 1 else table.shape[1],
                    rows=table.shape[0], width=table.shape[1], refs=_ptr(refs), num_pages=refs.numel(),
                    page_size=page_size)
    if pool is not None:
        if pool.dim() < 2 or pool.shape[1] != refs.numel():
            raise ValueError(f"pool must be [planes][{refs.numel()}][...]")
        size = pool.element_size()
        args.data, args.num_planes = _ptr(pool), pool.shape[0]
        page = 1
        for n in pool.shape[2:]:
            page *= n
        args.page_bytes = page * size
        args.page_stride = pool.stride(1) * size if pool.shape[1] > 1 else args.page_bytes
        args.plane_stride = pool.stride(0) * size if pool.shape[0] > 1 else pool.shape[1] * args.page_stride
        if pool.numel() > 0 and not pool[0, 0].is_contiguous():
            raise ValueError("pool: a page must be contiguous")
    return args


def prepare_pages_free(table, refs, rows, *, keep=None, stream=None) -> DeviceCall:
    """pages_free with its arguments checked and marshalled once."""
    device = _device_of(table=table, refs=refs, rows=rows, keep=keep)
    args = _page_args(table, refs)
    n = _i32("rows", rows, None).numel()
    if keep is not None:
        _i32("keep", keep, n)
    return DeviceCall(load().gdn_pages_free, (ctypes.byref(args), n, _ptr(rows), _ptr(keep),
                                              _RunOn(device, stream).handle), "gdn_pages_free",
                      [args, table, refs, rows, keep], device, None)


def pages_free(table, refs, rows, *, keep=None, stream=None):
    """One call of gdn_pages_free: the rows rows [n] int32 of table [rows][entries] int32 give their pages back,
    all or those from entry keep[i] on; refs [pages] int32."""
    with _RunOn(_device_of(table=table), stream):
        prepare_pages_free(table, refs, rows, keep=keep).launch()


def prepare_pages_reserve(table, refs, rows, lens, status, *, page_size, stream=None) -> DeviceCall:
    """pages_reserve into the caller's status [n] int32, checked and marshalled once."""
    device = _device_of(table=table, refs=refs, rows=rows, lens=lens, status=status)
    args = _page_args(table, refs, page_size)
    n = _i32("rows", rows, None).numel()
    _i32("lens", lens, n)
    _i32("status", status, n)
    return DeviceCall(load().gdn_pages_reserve, (ctypes.byref(args), n, _ptr(rows), _ptr(lens), _ptr(status),
                                                 _RunOn(device, stream).handle), "gdn_pages_reserve",
                      [args, table, refs, rows, lens, status], device, status)


def pages_reserve(table, refs, rows, lens, *, page_size, stream=None):
    """One call of gdn_pages_reserve: row rows[i] gets pages for its first lens[i] tokens where it has none.
    Returns status [n] int32: 0 done, 1 too few pages, 2 refused."""
    with _RunOn(_device_of(table=table), stream):
        status = torch.empty(rows.shape, dtype=torch.int32, device=table.device)
        prepare_pages_reserve(table, refs, rows, lens, status, page_size=page_size).launch()
    return status


def pages_workspace_bytes(num_pages):
    """Workspace gdn_pages_fork and gdn_pages_compact need."""
    return int(load().gdn_pages_workspace_bytes(num_pages))


def prepare_pages_fork(pool, table, refs, src, dst, lens, status, workspace, *, page_size,
                       stream=None) -> DeviceCall:
    """pages_fork into the caller's status [n] int32, checked and marshalled once."""
    device = _device_of(pool=pool, table=table, refs=refs, src=src, dst=dst, lens=lens, status=status,
                        workspace=workspace)
    args = _page_args(table, refs, page_size, pool)
    n = _i32("src", src, None).numel()
    for name, t in (("dst", dst), ("lens", lens), ("status", status)):
        _i32(name, t, n)
    ws, ws_bytes = _workspace(workspace)
    return DeviceCall(load().gdn_pages_fork, (ctypes.byref(args), n, _ptr(src), _ptr(dst), _ptr(lens), _ptr(status),
                                              ws, ws_bytes, _RunOn(device, stream).handle), "gdn_pages_fork",
                      [args, pool, table, refs, src, dst, lens, status, workspace], device, status)


def pages_fork(pool, table, refs, src, dst, lens, *, page_size, workspace=None, stream=None):
    """One call of gdn_pages_fork: the empty row dst[i] becomes the first lens[i] tokens of row src[i], full pages
    shared, a last one copied on every plane of pool [planes][pages][...]. Returns status [n] int32."""
    with _RunOn(_device_of(table=table), stream):
        status = torch.empty(src.shape, dtype=torch.int32, device=table.device)
        if workspace is None:
            workspace = torch.empty(pages_workspace_bytes(refs.numel()), dtype=torch.uint8, device=table.device)
        prepare_pages_fork(pool, table, refs, src, dst, lens, status, workspace, page_size=page_size).launch()
    return status


def prepare_pages_compact(pool, table, refs, page_map, used, workspace, *, stream=None) -> DeviceCall:
    """pages_compact into the caller's page_map [pages] and used [1] int32, checked and marshalled once."""
    device = _device_of(pool=pool, table=table, refs=refs, page_map=page_map, used=used, workspace=workspace)
    args = _page_args(table, refs, 1, pool)
    _i32("page_map", page_map, refs.numel())
    _i32("used", used, 1)
    ws, ws_bytes = _workspace(workspace)
    return DeviceCall(load().gdn_pages_compact, (ctypes.byref(args), _ptr(page_map), _ptr(used), ws, ws_bytes,
                                                 _RunOn(device, stream).handle), "gdn_pages_compact",
                      [args, pool, table, refs, page_map, used, workspace], device, (page_map, used))


def pages_compact(pool, table, refs, *, workspace=None, stream=None):
    """One call of gdn_pages_compact: the pages in use move to the front of pool [planes][pages][...], table and
    refs follow. Returns (page_map [pages] int32: where each page went, used [1] int32: how many are in use)."""
    with _RunOn(_device_of(table=table), stream):
        page_map = torch.empty(refs.shape, dtype=torch.int32, device=table.device)
        used = torch.empty(1, dtype=torch.int32, device=table.device)
        if workspace is None:
            workspace = torch.empty(pages_workspace_bytes(refs.numel()), dtype=torch.uint8, device=table.device)
        prepare_pages_compact(pool, table, refs, page_map, used, workspace).launch()
    return page_map, used
