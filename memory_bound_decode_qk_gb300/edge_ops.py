"""Thin ctypes binding over the C ABI of libedge_ops.so (include/edge_ops.h).

Argument marshalling only.  Every step of every op runs in the library's
CUDA kernels, and there is no CPU or eager fallback: if the library is
missing, the first call raises.  Torch is used for device memory, dtypes and
the current stream.  The binding allocates outputs through torch only when
the caller passes none.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

from . import _build

F32, F16, BF16, FP8_E4M3, INT8 = 0, 1, 2, 3, 4
ROTATE_HALF, INTERLEAVED = 0, 1
SILU, GELU_TANH = 0, 1
AXES_BLOCKS, AXES_CYCLED = 0, 1

STATUS = {
    0: "EDGE_OK", 1: "EDGE_ERR_NULL", 2: "EDGE_ERR_DTYPE", 3: "EDGE_ERR_SHAPE",
    4: "EDGE_ERR_ALIGN", 5: "EDGE_ERR_ALIAS", 6: "EDGE_ERR_UNSUPPORTED", 7: "EDGE_ERR_CUDA",
    8: "EDGE_ERR_VALUE",
}
EXPORTS = ("edge_rmsnorm", "edge_add_rmsnorm", "edge_glu_act", "edge_qk_norm_rope",
           "edge_qk_norm_rope_ex", "edge_rope", "edge_layernorm", "edge_quantize_fp8",
           "edge_qkv_rope_cache", "edge_copy",
           "edge_qk_norm_rope_axes", "edge_rope_axes", "edge_qkv_rope_cache_axes",
           "edge_paged_attention", "edge_paged_attention_workspace",
           "edge_pages_copy", "edge_pages_free", "edge_pages_fork", "edge_pages_compact",
           "edge_pages_compact_workspace",
           "edge_rmsnorm_q8", "edge_add_rmsnorm_q8", "edge_glu_act_q8", "edge_quantize_q8",
           "edge_matmul_q8",
           "edge_status_str", "edge_last_cuda_error", "edge_version")
QK_ROTATE_UNROUNDED = 1

_ACTS = {"silu": SILU, "gelu_tanh": GELU_TANH}
_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_LIB = None


class EdgeError(RuntimeError):
    def __init__(self, status: int, op: str):
        self.status = status
        msg = lib().edge_status_str(status).decode()
        extra = ""
        if status == 7:
            extra = f" (cudaError {lib().edge_last_cuda_error()})"
        super().__init__(f"{op}: {STATUS.get(status, status)}: {msg}{extra}")


def library_path() -> str:
    return _build.LIB


def lib(build_if_missing: bool = False) -> ctypes.CDLL:
    """The loaded C ABI.  Raises if libedge_ops.so is absent (no fallback)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB
    if not os.path.exists(path):
        if not build_if_missing:
            raise RuntimeError(
                f"libedge_ops.so is not built ({path}); run __graft_entry__.build() or "
                "python -m memory_bound_decode_qk_gb300._build")
        _build.build()
    L = ctypes.CDLL(path)
    P, I64, I32, I, F = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_int,
                         ctypes.c_float)
    L.edge_rmsnorm.argtypes = [P, I, P, P, I, I64, I64, F, I, F, P]
    L.edge_add_rmsnorm.argtypes = [P, I, P, P, P, I, I64, I64, F, I, F, P]
    L.edge_glu_act.argtypes = [P, I, P, I, I64, I64, I, F, P]
    L.edge_qk_norm_rope.argtypes = [P, P, I, P, P, P, P, I, I64, I32, I32, I32, I32, I, P, P, P,
                                    I64, F, I, F, P]
    L.edge_qk_norm_rope_ex.argtypes = [P, P, I, P, P, P, P, I, I64, I32, I32, I32, I32, I, P, P,
                                       P, I64, F, I, F, ctypes.c_uint32, P]
    L.edge_rope.argtypes = [P, P, I, P, P, I, I64, I32, I32, I32, I32, I, P, P, P, I64, F, P]
    L.edge_layernorm.argtypes = [P, I, P, P, P, I, I64, I64, F, F, P]
    L.edge_quantize_fp8.argtypes = [P, P, I, I64, F, P]
    L.edge_qkv_rope_cache.argtypes = [P, P, P, P, P, P, I, I64, I32, I32, I32, I32, I, P, P, P,
                                      I64, P, I64, F, I, I, P]
    L.edge_copy.argtypes = [P, P, I64, P]
    for name in ("edge_rmsnorm", "edge_add_rmsnorm", "edge_glu_act", "edge_qk_norm_rope",
                 "edge_qk_norm_rope_ex", "edge_rope", "edge_layernorm", "edge_quantize_fp8",
                 "edge_qkv_rope_cache", "edge_copy"):
        getattr(L, name).restype = I
    L.edge_qk_norm_rope_axes.argtypes = [P, P, I, P, P, P, P, I, I64, I32, I32, I32, I32, I, P,
                                         I32, P, I, P, P, I64, F, I, F, ctypes.c_uint32, P]
    L.edge_rope_axes.argtypes = [P, P, I, P, P, I, I64, I32, I32, I32, I32, I, P, I32, P, I, P, P,
                                 I64, F, P]
    L.edge_qkv_rope_cache_axes.argtypes = [P, P, P, P, P, P, I, I64, I32, I32, I32, I32, I, P, I32,
                                           P, I, P, P, I64, P, I64, F, I, I, P]
    for name in ("edge_qk_norm_rope_axes", "edge_rope_axes", "edge_qkv_rope_cache_axes"):
        getattr(L, name).restype = I
    L.edge_paged_attention.argtypes = [P, I, P, P, P, P, I, I64, I32, I32, I32, I64, I32, P, I32,
                                       I32, P, P, F, I, I32, F, P, I64, P]
    L.edge_paged_attention.restype = I
    L.edge_paged_attention_workspace.argtypes = [I, I32, I32, I32]
    L.edge_paged_attention_workspace.restype = I64
    L.edge_pages_copy.argtypes = [P, I32, I64, I32, P, P, I32, P]
    L.edge_pages_free.argtypes = [P, I32, I32, P, P, I32, P, I32, P]
    L.edge_pages_fork.argtypes = [P, I32, I64, I32, I32, P, I32, I32, P, P, P, P, I32, P, P, P]
    L.edge_pages_compact.argtypes = [P, I32, I64, I32, P, P, I32, I32, P, P, P, I64, P]
    for name in ("edge_pages_copy", "edge_pages_free", "edge_pages_fork", "edge_pages_compact"):
        getattr(L, name).restype = I
    L.edge_pages_compact_workspace.argtypes = [I32]
    L.edge_pages_compact_workspace.restype = I64
    L.edge_rmsnorm_q8.argtypes = [P, I, P, P, P, I, I64, I64, F, I, P]
    L.edge_add_rmsnorm_q8.argtypes = [P, I, P, P, P, P, I, I64, I64, F, I, P]
    L.edge_glu_act_q8.argtypes = [P, I, P, P, I, I64, I64, I, P]
    L.edge_quantize_q8.argtypes = [P, I, P, P, I, I64, I64, P]
    L.edge_matmul_q8.argtypes = [P, I, P, P, I, P, P, P, I64, I64, I64, P]
    for name in ("edge_rmsnorm_q8", "edge_add_rmsnorm_q8", "edge_glu_act_q8", "edge_quantize_q8",
                 "edge_matmul_q8"):
        getattr(L, name).restype = I
    L.edge_status_str.argtypes = [I]
    L.edge_status_str.restype = ctypes.c_char_p
    L.edge_last_cuda_error.restype = I
    L.edge_version.restype = I
    _LIB = L
    return L


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream's raw handle without building a Stream object (about 2
# us cheaper per call); the public route where torch lacks it.
_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _RAW_STREAM is not None:
            return _RAW_STREAM(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _dt(t: torch.Tensor) -> int:
    try:
        return _DT[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _out_dt(fp8: bool, dt: int) -> int:
    return FP8_E4M3 if fp8 else dt


def _check(st: int, op: str):
    if st != 0:
        raise EdgeError(st, op)


def _need_contig(*ts):
    for t in ts:
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous (row-major)")


def _alloc(like: torch.Tensor, shape, fp8: bool):
    return torch.empty(shape, dtype=torch.uint8 if fp8 else like.dtype, device=like.device)


def rmsnorm(x, w=None, *, eps=1e-6, weight_offset=0, out=None, fp8=False, inv_scale=1.0,
            stream=None):
    """RMSNorm over the last dim of x ([rows, hidden])."""
    _need_contig(x, w, out)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if out is None:
        out = _alloc(x, x.shape, fp8)
    dt = _dt(x)
    _check(lib().edge_rmsnorm(_ptr(out), _out_dt(fp8, dt), _ptr(x), _ptr(w), dt, rows, hidden,
                              eps, weight_offset, inv_scale, _stream(stream)), "edge_rmsnorm")
    return out


def add_rmsnorm(x, residual, w=None, *, eps=1e-6, weight_offset=0, out=None, fp8=False,
                inv_scale=1.0, stream=None):
    """residual <- x + residual (rounded to the dtype); returns RMSNorm(residual)."""
    _need_contig(x, residual, w, out)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if out is None:
        out = _alloc(x, x.shape, fp8)
    dt = _dt(x)
    _check(lib().edge_add_rmsnorm(_ptr(out), _out_dt(fp8, dt), _ptr(x), _ptr(residual), _ptr(w),
                                  dt, rows, hidden, eps, weight_offset, inv_scale,
                                  _stream(stream)), "edge_add_rmsnorm")
    return out


def layernorm(x, gamma=None, beta=None, *, eps=1e-6, out=None, fp8=False, inv_scale=1.0,
              stream=None):
    """One-read LayerNorm over the last dim of x ([rows, hidden])."""
    _need_contig(x, gamma, beta, out)
    hidden = x.shape[-1]
    rows = x.numel() // hidden if hidden else 0
    if out is None:
        out = _alloc(x, x.shape, fp8)
    dt = _dt(x)
    _check(lib().edge_layernorm(_ptr(out), _out_dt(fp8, dt), _ptr(x), _ptr(gamma), _ptr(beta), dt,
                                rows, hidden, eps, inv_scale, _stream(stream)), "edge_layernorm")
    return out


def copy(src, *, out=None, stream=None):
    """The yardstick copy: src's bytes into out (a new tensor like src when
    None), in the operators' launch form.  Returns out."""
    _need_contig(src, out)
    if out is None:
        out = torch.empty_like(src)
    nbytes = src.numel() * src.element_size()
    if out.numel() * out.element_size() != nbytes:
        raise ValueError("copy: out must hold as many bytes as src")
    _check(lib().edge_copy(_ptr(out), _ptr(src), nbytes, _stream(stream)), "edge_copy")
    return out


def quantize_fp8(x, inv_scale, *, out=None, stream=None):
    """Static-scale E4M3 codes of x (any shape, contiguous); uint8 output."""
    _need_contig(x, out)
    if out is None:
        out = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    _check(lib().edge_quantize_fp8(_ptr(out), _ptr(x), _dt(x), x.numel(), inv_scale,
                                   _stream(stream)), "edge_quantize_fp8")
    return out


_AXIS_ORDER = {"blocks": AXES_BLOCKS, "cycled": AXES_CYCLED}


@functools.lru_cache(maxsize=256)
def _section_array(sections):
    if any(not -2 ** 31 <= n < 2 ** 31 for n in sections):
        raise ValueError(f"sections must be 32-bit numbers, not {sections}")
    return (ctypes.c_int32 * max(1, len(sections)))(*sections)


def _axis_args(sections, axis_order, positions, tokens):
    """(axes, sections array, order) of a rotary embedding with several axes."""
    sections = tuple(sections)
    n = len(sections)
    if positions is not None and not (positions.dtype is torch.int64 and
                                      positions.shape == (n, tokens)):
        raise ValueError(f"positions must be int64 [{n}, {tokens}] for {n} sections")
    return n, _section_array(sections), _AXIS_ORDER.get(axis_order, axis_order)


def qkv_rope_cache(qkv, q_heads, kv_heads, wq, wk, positions, cos, sin, slots, k_cache, v_cache,
                   *, rotary_dim=None, layout=ROTATE_HALF, eps=1e-6, weight_offset=0,
                   normalize=True, q_out=None, cache_len=None, stream=None, sections=None,
                   axis_order="blocks"):
    """Fused QKV split + prologue + KV-cache write.  qkv: [T, (Hq + 2 Hk) D];
    k_cache, v_cache: [S, Hk, D] (written at rows slots[t]).  sections, axis_order:
    as in qk_norm_rope.  Returns q_out."""
    _need_contig(qkv, wq, wk, positions, cos, sin, slots, k_cache, v_cache, q_out)
    T = qkv.shape[0]
    D = qkv.shape[-1] // (q_heads + 2 * kv_heads)
    if rotary_dim is None:
        rotary_dim = D if cos is None else 2 * cos.shape[-1]
    if cache_len is None:
        cache_len = 0 if cos is None else cos.shape[0]
    if isinstance(layout, str):
        layout = {"rotate_half": ROTATE_HALF, "interleaved": INTERLEAVED}[layout]
    if q_out is None:
        q_out = torch.empty((T, q_heads, D), dtype=qkv.dtype, device=qkv.device)
    S = k_cache.shape[0] if k_cache is not None else 0
    if sections is not None:
        axes, counts, order = _axis_args(sections, axis_order, positions, T)
        _check(lib().edge_qkv_rope_cache_axes(
            _ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(qkv), _ptr(wq), _ptr(wk), _dt(qkv), T,
            q_heads, kv_heads, D, rotary_dim, layout, _ptr(positions), axes, counts, order,
            _ptr(cos), _ptr(sin), cache_len, _ptr(slots), S, eps, weight_offset,
            1 if normalize else 0, _stream(stream)), "edge_qkv_rope_cache_axes")
        return q_out
    _check(lib().edge_qkv_rope_cache(_ptr(q_out), _ptr(k_cache), _ptr(v_cache), _ptr(qkv),
                                     _ptr(wq), _ptr(wk), _dt(qkv), T, q_heads, kv_heads, D,
                                     rotary_dim, layout, _ptr(positions), _ptr(cos), _ptr(sin),
                                     cache_len, _ptr(slots), S, eps, weight_offset,
                                     1 if normalize else 0, _stream(stream)), "edge_qkv_rope_cache")
    return q_out


def glu_act(gate_up, act=SILU, *, out=None, fp8=False, inv_scale=1.0, stream=None):
    """act(gate) * up for gate_up = [rows, 2d] (gate first); returns [rows, d]."""
    _need_contig(gate_up, out)
    two_d = gate_up.shape[-1]
    d = two_d // 2
    rows = gate_up.numel() // two_d if two_d else 0
    if isinstance(act, str):
        act = _ACTS[act]
    if out is None:
        out = _alloc(gate_up, tuple(gate_up.shape[:-1]) + (d,), fp8)
    dt = _dt(gate_up)
    _check(lib().edge_glu_act(_ptr(out), _out_dt(fp8, dt), _ptr(gate_up), dt, rows, d, act,
                              inv_scale, _stream(stream)), "edge_glu_act")
    return out


def _qk_shapes(q, k, cos, rotary_dim, cache_len, layout, fp8, q_out, k_out):
    T, Hq, D = q.shape
    Hk = k.shape[1] if k is not None else 0
    if rotary_dim is None:
        rotary_dim = D if cos is None else 2 * cos.shape[-1]
    if cache_len is None:
        cache_len = 0 if cos is None else cos.shape[0]
    if isinstance(layout, str):
        layout = {"rotate_half": ROTATE_HALF, "interleaved": INTERLEAVED}[layout]
    if q_out is None:
        q_out = _alloc(q, q.shape, fp8)
    if k_out is None and k is not None:
        k_out = _alloc(k, k.shape, fp8)
    return T, Hq, Hk, D, rotary_dim, cache_len, layout, q_out, k_out


def qk_norm_rope(q, k, wq, wk, positions, cos, sin, *, rotary_dim=None, layout=ROTATE_HALF,
                 eps=1e-6, weight_offset=0, q_out=None, k_out=None, fp8=False, inv_scale=1.0,
                 cache_len=None, unrounded=False, stream=None, sections=None,
                 axis_order="blocks"):
    """Per-head QK-RMSNorm + RoPE.  q: [T, Hq, D], k: [T, Hk, D];
    cos/sin: [P, rotary_dim/2] fp32; positions: [T] int64.  Pass q_out=q and
    k_out=k for the in-place form.  unrounded=True rotates the fp32 normalized
    value (edge_qk_norm_rope_ex with EDGE_QK_ROTATE_UNROUNDED).  sections: the
    pairs of each of A axes, for positions [A, T] (rotary positions with several
    axes); axis_order "blocks" (one axis after the other) or "cycled" (dealt in
    turn).  Returns (q_out, k_out)."""
    _need_contig(q, k, wq, wk, positions, cos, sin, q_out, k_out)
    T, Hq, Hk, D, rotary_dim, cache_len, layout, q_out, k_out = _qk_shapes(
        q, k, cos, rotary_dim, cache_len, layout, fp8, q_out, k_out)
    dt = _dt(q)
    args = (_ptr(q_out), _ptr(k_out), _out_dt(fp8, dt), _ptr(q), _ptr(k), _ptr(wq), _ptr(wk), dt,
            T, Hq, Hk, D, rotary_dim, layout, _ptr(positions), _ptr(cos), _ptr(sin), cache_len,
            eps, weight_offset, inv_scale)
    if sections is not None:
        axes, counts, order = _axis_args(sections, axis_order, positions, T)
        _check(lib().edge_qk_norm_rope_axes(
            *args[:15], axes, counts, order, *args[15:], QK_ROTATE_UNROUNDED if unrounded else 0,
            _stream(stream)), "edge_qk_norm_rope_axes")
    elif unrounded:
        _check(lib().edge_qk_norm_rope_ex(*args, QK_ROTATE_UNROUNDED, _stream(stream)),
               "edge_qk_norm_rope_ex")
    else:
        _check(lib().edge_qk_norm_rope(*args, _stream(stream)), "edge_qk_norm_rope")
    return q_out, k_out


def rope(q, k, positions, cos, sin, *, rotary_dim=None, layout=ROTATE_HALF, q_out=None,
         k_out=None, fp8=False, inv_scale=1.0, cache_len=None, stream=None, sections=None,
         axis_order="blocks"):
    """Standalone rotary embedding of q: [T, Hq, D] and k: [T, Hk, D] (k may
    be None).  Pass q_out=q (k_out=k) for the in-place form.  sections,
    axis_order: as in qk_norm_rope.  Returns (q_out, k_out)."""
    _need_contig(q, k, positions, cos, sin, q_out, k_out)
    T, Hq, Hk, D, rotary_dim, cache_len, layout, q_out, k_out = _qk_shapes(
        q, k, cos, rotary_dim, cache_len, layout, fp8, q_out, k_out)
    dt = _dt(q)
    if sections is not None:
        axes, counts, order = _axis_args(sections, axis_order, positions, T)
        _check(lib().edge_rope_axes(
            _ptr(q_out), _ptr(k_out), _out_dt(fp8, dt), _ptr(q), _ptr(k), dt, T, Hq, Hk, D,
            rotary_dim, layout, _ptr(positions), axes, counts, order, _ptr(cos), _ptr(sin),
            cache_len, inv_scale, _stream(stream)), "edge_rope_axes")
        return q_out, k_out
    _check(lib().edge_rope(_ptr(q_out), _ptr(k_out), _out_dt(fp8, dt), _ptr(q), _ptr(k), dt, T, Hq,
                           Hk, D, rotary_dim, layout, _ptr(positions), _ptr(cos), _ptr(sin),
                           cache_len, inv_scale, _stream(stream)), "edge_rope")
    return q_out, k_out


# ---------------------------------------------------------------- paged cache

def _on(device, stream):
    """The context in which a call allocates and launches: the tensors' device,
    and `stream` as torch's current stream, so that memory taken for the call
    belongs to the stream that uses it.  A stream of another device is refused."""
    if stream is None:
        return torch.cuda.device(device)
    if getattr(stream, "device", device) != device:
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return torch.cuda.stream(stream)


# The current device without torch's lazy-initialization check (a CUDA tensor
# exists wherever it is asked for); the public route where torch lacks it.
_CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _here(index, stream):
    """Whether a call with tensors on device `index` can launch as it stands."""
    return stream is None and index == _CURRENT_DEVICE()


def _fits(index, dtype, *tensors):
    """Whether every tensor given has this dtype, is on device `index` and is
    contiguous: the quick form of _want, which names what is wrong."""
    for t in tensors:
        if t is not None and not (t.dtype is dtype and t.get_device() == index and
                                  t.is_contiguous()):
            return False
    return True


def _want(t, name, dtype, shape, device):
    """t is a contiguous tensor of this dtype, shape (None: any extent) and device."""
    if t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not {device}")
    if len(t.shape) != len(shape) or any(b is not None and a != b for a, b in zip(t.shape, shape)):
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")


def paged_attention_workspace(q, k_cache):
    """A workspace for paged_attention calls with heads like q's ([T, Hq, D]) over
    k_cache ([S, Hk, D]), of any batch and length.  Calls that may run at the
    same time need one each."""
    with torch.cuda.device(q.device):
        n = lib().edge_paged_attention_workspace(_dt(q), q.shape[-2], k_cache.shape[-2],
                                                 q.shape[-1])
        if n < 0:
            raise ValueError("paged_attention does not serve these heads")
        return torch.empty(n, dtype=torch.uint8, device=q.device)


def paged_attention(q, k_cache, v_cache, block_table, lens, *, page_size, q_starts=None,
                    scale=None, causal=True, window=0, out=None, lse=None, fp8=False,
                    inv_scale=1.0, workspace=None, stream=None):
    """Attention of new tokens over a paged KV cache.  q: [T, Hq, D]; k_cache,
    v_cache: [S, Hk, D] (slot = page * page_size + offset, as qkv_rope_cache
    writes them); block_table: [B, P] int32; lens: [B] int32, the keys of each
    sequence with its new tokens.  q_starts: [B + 1] int32, the rows of each
    sequence in q; None for one token per sequence (T == B).  scale: 1 /
    sqrt(D) when None.  lse: [T, Hq] fp32 to be filled with the log-sum-exp of
    each row.  workspace: from paged_attention_workspace; one is taken from
    torch for the call when None.  Returns out ([T, Hq, D])."""
    T, Hq, D = q.shape
    S, Hk, Dk = k_cache.shape
    B, pages = block_table.shape
    at = q.get_device()
    dt = _dt(q)
    if not (at >= 0 and Dk == D and v_cache.shape == k_cache.shape and lens.shape == (B,) and
            _fits(at, q.dtype, q, k_cache, v_cache) and
            _fits(at, torch.int32, block_table, lens, q_starts) and
            (q_starts is None or q_starts.shape == (B + 1,)) and
            (out is None or (out.shape == q.shape and
                             _fits(at, torch.uint8 if fp8 else q.dtype, out))) and
            (lse is None or (lse.shape == (T, Hq) and _fits(at, torch.float32, lse))) and
            (workspace is None or _fits(at, torch.uint8, workspace))):
        _explain_attention(q, k_cache, v_cache, block_table, lens, q_starts, out, lse, fp8,
                           workspace)
    if not _here(at, stream):
        with _on(q.device, stream):
            return paged_attention(q, k_cache, v_cache, block_table, lens, page_size=page_size,
                                   q_starts=q_starts, scale=scale, causal=causal, window=window,
                                   out=out, lse=lse, fp8=fp8, inv_scale=inv_scale,
                                   workspace=workspace)
    if out is None:
        out = _alloc(q, q.shape, fp8)
    if T == 0:
        return out  # no rows (an empty tensor has no address to pass on)
    if workspace is None:
        workspace = paged_attention_workspace(q, k_cache)
    if scale is None:
        scale = D ** -0.5
    st = lib().edge_paged_attention(
        out.data_ptr(), FP8_E4M3 if fp8 else dt, _ptr(lse), q.data_ptr(), k_cache.data_ptr(),
        v_cache.data_ptr(), dt, T, Hq, Hk, D, S, page_size, block_table.data_ptr(), B, pages,
        lens.data_ptr(), _ptr(q_starts), scale, 1 if causal else 0, window, inv_scale,
        workspace.data_ptr(), workspace.numel(), _stream(None))
    if st:
        raise EdgeError(st, "edge_paged_attention")
    return out


def _explain_attention(q, k_cache, v_cache, block_table, lens, q_starts, out, lse, fp8, workspace):
    """Raises for the first tensor of a paged_attention call that does not fit."""
    T, Hq, D = q.shape
    S, Hk, _ = k_cache.shape
    B, pages = block_table.shape
    dev = q.device
    if dev.type != "cuda":
        raise ValueError(f"q must be a CUDA tensor, not on {dev}")
    _want(q, "q", q.dtype, (T, Hq, D), dev)
    _want(k_cache, "k_cache", q.dtype, (S, Hk, D), dev)
    _want(v_cache, "v_cache", q.dtype, (S, Hk, D), dev)
    _want(block_table, "block_table", torch.int32, (B, pages), dev)
    _want(lens, "lens", torch.int32, (B,), dev)
    if q_starts is not None:
        _want(q_starts, "q_starts", torch.int32, (B + 1,), dev)
    if out is not None:
        _want(out, "out", torch.uint8 if fp8 else q.dtype, (T, Hq, D), dev)
    if lse is not None:
        _want(lse, "lse", torch.float32, (T, Hq), dev)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (None,), dev)


class PageCaches:
    """The caches of one page pool: tensors of one dtype and shape [S, ...] (S =
    pages * page_size slots, as qkv_rope_cache and paged_attention take them) on
    one device.  Holds the tensors and their addresses for the page calls."""

    def __init__(self, caches, page_size):
        caches = list(caches)
        if not caches:
            raise ValueError("PageCaches needs at least one cache")
        first = caches[0]
        if page_size < 1 or first.shape[0] % page_size:
            raise ValueError(f"{first.shape[0]} slots are not whole pages of {page_size}")
        if first.device.type != "cuda":
            raise ValueError(f"caches must be CUDA tensors, not on {first.device}")
        for t in caches:
            _want(t, "cache", first.dtype, first.shape, first.device)
        self.tensors = caches
        self.device = first.device
        self.page_size = page_size
        self.num_pages = first.shape[0] // page_size
        slot = first.numel() // first.shape[0] if first.shape[0] else 1
        self.page_bytes = max(1, slot * first.element_size()) * page_size
        self.pointers = (ctypes.c_void_p * len(caches))(*[t.data_ptr() for t in caches])
        self.index = first.get_device()
        self.count = len(caches)

    def __len__(self):
        return len(self.tensors)


def pages_copy(caches, src, dst, *, stream=None):
    """Copies page src[i] to page dst[i] in every cache of `caches` (PageCaches).
    src, dst: [n] int32.  See edge_pages_copy for pairs that meet."""
    n = src.shape[0]
    if not (src.dim() == 1 and dst.shape == src.shape and
            _fits(caches.index, torch.int32, src, dst)):
        _want(src, "src", torch.int32, (None,), caches.device)
        _want(dst, "dst", torch.int32, (n,), caches.device)
    if not _here(caches.index, stream):
        with _on(caches.device, stream):
            return pages_copy(caches, src, dst)
    st = lib().edge_pages_copy(caches.pointers, caches.count, caches.page_bytes, caches.num_pages,
                               src.data_ptr(), dst.data_ptr(), n, _stream(None))
    if st:
        raise EdgeError(st, "edge_pages_copy")


def _want_rows(block_table, lens, refs, pages, dev):
    _want(block_table, "block_table", torch.int32, (None, None), dev)
    if lens is not None:
        _want(lens, "lens", torch.int32, (block_table.shape[0],), dev)
    _want(refs, "refs", torch.int32, (pages,), dev)


def pages_free(block_table, lens, refs, seqs, *, stream=None):
    """Gives back the pages of sequences `seqs` ([n] int32): their entries of
    block_table ([B, P] int32) become -1, their lens ([B] int32) 0, and the
    counts refs ([pages] int32) of their pages go down."""
    at = refs.get_device()
    B, width = block_table.shape
    if not (at >= 0 and refs.dim() == 1 and seqs.dim() == 1 and lens.shape == (B,) and
            _fits(at, torch.int32, block_table, lens, refs, seqs)):
        _want_rows(block_table, lens, refs, None, refs.device)
        _want(seqs, "seqs", torch.int32, (None,), refs.device)
        raise ValueError(f"refs must be a CUDA tensor, not on {refs.device}")
    if not _here(at, stream):
        with _on(refs.device, stream):
            return pages_free(block_table, lens, refs, seqs)
    st = lib().edge_pages_free(block_table.data_ptr(), B, width, lens.data_ptr(), refs.data_ptr(),
                               refs.shape[0], seqs.data_ptr(), seqs.shape[0], _stream(None))
    if st:
        raise EdgeError(st, "edge_pages_free")


def pages_fork(caches, block_table, lens, refs, parents, children, *, status=None, pairs=None,
               stream=None):
    """Makes sequence children[i] a copy of parents[i] ([n] int32 each): full
    pages are shared, a partly filled last page is copied into the lowest free
    page of `caches` (PageCaches).  Returns status ([n] int32: 0 forked, 1 no
    free page, 2 refused); pairs ([n, 2] int32), where given, receives the pages
    copied."""
    n = parents.shape[0]
    B, width = block_table.shape
    if not (parents.dim() == 1 and children.shape == parents.shape and lens.shape == (B,) and
            refs.shape == (caches.num_pages,) and
            (status is None or status.shape == (n,)) and (pairs is None or pairs.shape == (n, 2)) and
            _fits(caches.index, torch.int32, block_table, lens, refs, parents, children, status,
                  pairs)):
        dev = caches.device
        _want_rows(block_table, lens, refs, caches.num_pages, dev)
        _want(parents, "parents", torch.int32, (None,), dev)
        _want(children, "children", torch.int32, (n,), dev)
        if status is not None:
            _want(status, "status", torch.int32, (n,), dev)
        if pairs is not None:
            _want(pairs, "pairs", torch.int32, (n, 2), dev)
    if not _here(caches.index, stream):
        with _on(caches.device, stream):
            return pages_fork(caches, block_table, lens, refs, parents, children, status=status,
                              pairs=pairs)
    if status is None:
        status = torch.empty_like(parents)
    if pairs is None:
        pairs = torch.empty((n, 2), dtype=torch.int32, device=caches.device)
    st = lib().edge_pages_fork(caches.pointers, caches.count, caches.page_bytes, caches.num_pages,
                               caches.page_size, block_table.data_ptr(), B, width, lens.data_ptr(),
                               refs.data_ptr(), parents.data_ptr(), children.data_ptr(), n,
                               status.data_ptr(), pairs.data_ptr(), _stream(None))
    if st:
        raise EdgeError(st, "edge_pages_fork")
    return status


def pages_compact_workspace(refs):
    """A workspace for pages_compact of a pool with counts refs ([pages] int32)."""
    n = lib().edge_pages_compact_workspace(refs.shape[0])
    return torch.empty(n, dtype=torch.uint8, device=refs.device)


def pages_compact(caches, block_table, refs, *, table_out=None, refs_out=None, workspace=None,
                  stream=None):
    """Moves the pages in use to the lowest numbers in every cache of `caches`
    (PageCaches), and renumbers block_table ([B, P] int32) and refs ([pages]
    int32), in place or into table_out and refs_out.  Returns the new number of
    each page ([pages] int32, -1 for free pages), a view of the workspace."""
    dev = caches.device
    table_out = block_table if table_out is None else table_out
    refs_out = refs if refs_out is None else refs_out
    _want_rows(block_table, None, refs, caches.num_pages, dev)
    _want(table_out, "table_out", torch.int32, tuple(block_table.shape), dev)
    _want(refs_out, "refs_out", torch.int32, tuple(refs.shape), dev)
    if workspace is not None:
        _want(workspace, "workspace", torch.uint8, (None,), dev)
    if not _here(caches.index, stream):
        with _on(dev, stream):
            return pages_compact(caches, block_table, refs, table_out=table_out, refs_out=refs_out,
                                 workspace=workspace)
    if workspace is None:
        workspace = pages_compact_workspace(refs)
    _check(lib().edge_pages_compact(caches.pointers, len(caches), caches.page_bytes,
                                    caches.num_pages, table_out.data_ptr(), block_table.data_ptr(),
                                    *block_table.shape, refs_out.data_ptr(), refs.data_ptr(),
                                    workspace.data_ptr(), workspace.numel(), _stream(None)),
           "edge_pages_compact")
    return workspace[:4 * caches.num_pages].view(torch.int32)


# ---------------------------------------------------------------- 8 bits, a scale per token

# dtypes of a tensor of codes, by fp8; the first is the one that the binding allocates
_CODES = {False: (torch.int8,), True: (torch.uint8, torch.float8_e4m3fn)}
_CODE_KIND = {torch.int8: INT8, torch.uint8: FP8_E4M3, torch.float8_e4m3fn: FP8_E4M3}


def _stream_of(index):
    """The current stream's raw handle on device `index`, the current one."""
    return _RAW_STREAM(index) if _RAW_STREAM is not None else torch.cuda.current_stream().cuda_stream


def _q8_fits(at, x, n, shape, fp8, out, scales):
    """Whether x, and out and scales where given, suit a call that turns the rows of x
    into n codes each, of shape `shape` in all."""
    return (at >= 0 and n > 0 and x.is_contiguous() and
            (out is None or (out.shape == shape and out.dtype in _CODES[fp8] and
                             out.get_device() == at and out.is_contiguous())) and
            (scales is None or (scales.shape == shape[:-1] and
                                _fits(at, torch.float32, scales))))


def _explain_q8(x, name, shape, fp8, out, scales):
    """Raises for the first tensor of a row call in 8 bits that does not fit."""
    dev = x.device
    if dev.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor, not on {dev}")
    if not shape or shape[-1] < 1:
        raise ValueError(f"{name} must have rows of at least one code, not shape {tuple(x.shape)}")
    _want(x, name, x.dtype, tuple(x.shape), dev)
    if out is not None:
        kind = out.dtype if out.dtype in _CODES[fp8] else _CODES[fp8][0]
        _want(out, "out", kind, tuple(shape), dev)
    if scales is not None:
        _want(scales, "scales", torch.float32, tuple(shape[:-1]), dev)


def _q8_results(x, shape, fp8, out, scales):
    if out is None:
        out = torch.empty(shape, dtype=_CODES[fp8][0], device=x.device)
    if scales is None:
        scales = torch.empty(shape[:-1], dtype=torch.float32, device=x.device)
    return out, scales


def rmsnorm_q8(x, w=None, *, eps=1e-6, weight_offset=0, fp8=False, out=None, scales=None,
               stream=None):
    """RMSNorm over the last dim of x ([..., n]) in 8 bits: int8 codes, or E4M3
    codes (uint8) with fp8=True, and an fp32 scale for each row.  w: [n].
    Returns (out, scales), out * scales[..., None] being the norm."""
    at, shape = x.get_device(), x.shape
    n = shape[-1] if shape else 0
    if not (_q8_fits(at, x, n, shape, fp8, out, scales) and
            (w is None or (w.shape == (n,) and _fits(at, x.dtype, w)))):
        _explain_q8(x, "x", shape, fp8, out, scales)
        if w is not None:
            _want(w, "w", x.dtype, (n,), x.device)
    if not _here(at, stream):
        with _on(x.device, stream):
            return rmsnorm_q8(x, w, eps=eps, weight_offset=weight_offset, fp8=fp8, out=out,
                              scales=scales)
    dt = _dt(x)
    out, scales = _q8_results(x, shape, fp8, out, scales)
    rows = scales.numel()
    if rows == 0:
        return out, scales  # (an empty tensor has no address to pass on)
    st = (_LIB or lib()).edge_rmsnorm_q8(out.data_ptr(), FP8_E4M3 if fp8 else INT8, scales.data_ptr(),
                               x.data_ptr(), _ptr(w), dt, rows, n, eps, weight_offset,
                               _stream_of(at))
    if st:
        raise EdgeError(st, "edge_rmsnorm_q8")
    return out, scales


def add_rmsnorm_q8(x, residual, w=None, *, eps=1e-6, weight_offset=0, fp8=False, out=None,
                   scales=None, stream=None):
    """residual <- x + residual (rounded to the dtype); returns rmsnorm_q8 of it."""
    at, shape = x.get_device(), x.shape
    n = shape[-1] if shape else 0
    if not (_q8_fits(at, x, n, shape, fp8, out, scales) and residual.shape == shape and
            _fits(at, x.dtype, residual) and
            (w is None or (w.shape == (n,) and _fits(at, x.dtype, w)))):
        _explain_q8(x, "x", shape, fp8, out, scales)
        _want(residual, "residual", x.dtype, tuple(shape), x.device)
        if w is not None:
            _want(w, "w", x.dtype, (n,), x.device)
    if not _here(at, stream):
        with _on(x.device, stream):
            return add_rmsnorm_q8(x, residual, w, eps=eps, weight_offset=weight_offset, fp8=fp8,
                                  out=out, scales=scales)
    dt = _dt(x)
    out, scales = _q8_results(x, shape, fp8, out, scales)
    rows = scales.numel()
    if rows == 0:
        return out, scales
    st = (_LIB or lib()).edge_add_rmsnorm_q8(out.data_ptr(), FP8_E4M3 if fp8 else INT8, scales.data_ptr(),
                                   x.data_ptr(), residual.data_ptr(), _ptr(w), dt, rows, n, eps,
                                   weight_offset, _stream_of(at))
    if st:
        raise EdgeError(st, "edge_add_rmsnorm_q8")
    return out, scales


def glu_act_q8(gate_up, act=SILU, *, fp8=False, out=None, scales=None, stream=None):
    """act(gate) * up for gate_up = [..., 2d] (gate first) in 8 bits, as rmsnorm_q8
    returns them: ([..., d], [...])."""
    if isinstance(act, str):
        act = _ACTS[act]
    at, two_d = gate_up.get_device(), gate_up.shape[-1] if gate_up.shape else 0
    shape = gate_up.shape[:-1] + (two_d // 2,)
    if not (_q8_fits(at, gate_up, two_d // 2, shape, fp8, out, scales) and two_d % 2 == 0):
        _explain_q8(gate_up, "gate_up", shape, fp8, out, scales)
        raise ValueError(f"gate_up must have rows of an even length, not {two_d}")
    if not _here(at, stream):
        with _on(gate_up.device, stream):
            return glu_act_q8(gate_up, act, fp8=fp8, out=out, scales=scales)
    dt = _dt(gate_up)
    out, scales = _q8_results(gate_up, shape, fp8, out, scales)
    rows = scales.numel()
    if rows == 0:
        return out, scales
    st = (_LIB or lib()).edge_glu_act_q8(out.data_ptr(), FP8_E4M3 if fp8 else INT8, scales.data_ptr(),
                               gate_up.data_ptr(), dt, rows, two_d // 2, act, _stream_of(at))
    if st:
        raise EdgeError(st, "edge_glu_act_q8")
    return out, scales


def quantize_q8(x, *, fp8=False, out=None, scales=None, stream=None):
    """The rows of x ([..., n]) in 8 bits, as rmsnorm_q8 returns them."""
    at, shape = x.get_device(), x.shape
    n = shape[-1] if shape else 0
    if not _q8_fits(at, x, n, shape, fp8, out, scales):
        _explain_q8(x, "x", shape, fp8, out, scales)
    if not _here(at, stream):
        with _on(x.device, stream):
            return quantize_q8(x, fp8=fp8, out=out, scales=scales)
    dt = _dt(x)
    out, scales = _q8_results(x, shape, fp8, out, scales)
    rows = scales.numel()
    if rows == 0:
        return out, scales
    st = (_LIB or lib()).edge_quantize_q8(out.data_ptr(), FP8_E4M3 if fp8 else INT8, scales.data_ptr(),
                                x.data_ptr(), dt, rows, n, _stream_of(at))
    if st:
        raise EdgeError(st, "edge_quantize_q8")
    return out, scales


def matmul_q8(a, w, a_scales, w_scales, *, bias=None, dtype=None, out=None, stream=None):
    """a w^T of 8-bit operands with a scale for each token and output channel.
    a: [..., k] and w: [n, k], both int8 or both E4M3 codes (uint8 or
    float8_e4m3fn); a_scales: [...], w_scales: [n] fp32; bias: [n].  The result
    ([..., n]) and bias have dtype `dtype` (out's, or bf16)."""
    at, k, n = a.get_device(), a.shape[-1] if a.shape else 0, w.shape[0] if w.shape else 0
    kind = _CODE_KIND.get(a.dtype)
    if dtype is None:
        dtype = torch.bfloat16 if out is None else out.dtype
    shape = a.shape[:-1] + (n,)
    if not (at >= 0 and kind is not None and k > 0 and n > 0 and w.shape == (n, k) and a.is_contiguous() and
            _CODE_KIND.get(w.dtype) == kind and w.get_device() == at and w.is_contiguous() and
            a_scales.shape == shape[:-1] and w_scales.shape == (n,) and
            _fits(at, torch.float32, a_scales, w_scales) and
            (bias is None or (bias.shape == (n,) and _fits(at, dtype, bias))) and
            (out is None or (out.shape == shape and _fits(at, dtype, out)))):
        _explain_matmul(a, w, a_scales, w_scales, bias, dtype, out)
    if not _here(at, stream):
        with _on(a.device, stream):
            return matmul_q8(a, w, a_scales, w_scales, bias=bias, dtype=dtype, out=out)
    try:
        dt = _DT[dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {dtype}") from None
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=a.device)
    tokens = a_scales.numel()
    if tokens == 0:
        return out
    st = (_LIB or lib()).edge_matmul_q8(out.data_ptr(), dt, a.data_ptr(), w.data_ptr(), kind,
                              a_scales.data_ptr(), w_scales.data_ptr(), _ptr(bias), tokens, n, k,
                              _stream_of(at))
    if st:
        raise EdgeError(st, "edge_matmul_q8")
    return out


def _explain_matmul(a, w, a_scales, w_scales, bias, dtype, out):
    """Raises for the first tensor of a matmul_q8 call that does not fit."""
    dev = a.device
    if dev.type != "cuda":
        raise ValueError(f"a must be a CUDA tensor, not on {dev}")
    if a.dtype not in _CODE_KIND:
        raise TypeError(f"a must hold int8 or E4M3 codes, not {a.dtype}")
    if w.dim() != 2 or a.dim() < 1 or a.shape[-1] < 1 or w.shape[0] < 1:
        raise ValueError(f"a and w must be [..., k] and [n, k] with n and k at least 1, not "
                         f"{tuple(a.shape)} and {tuple(w.shape)}")
    n, k = w.shape[0], a.shape[-1]
    same = w.dtype if _CODE_KIND.get(w.dtype) == _CODE_KIND[a.dtype] else a.dtype
    _want(a, "a", a.dtype, tuple(a.shape), dev)
    _want(w, "w", same, (n, k), dev)
    _want(a_scales, "a_scales", torch.float32, tuple(a.shape[:-1]), dev)
    _want(w_scales, "w_scales", torch.float32, (n,), dev)
    if bias is not None:
        _want(bias, "bias", dtype, (n,), dev)
    if out is not None:
        _want(out, "out", dtype, tuple(a.shape[:-1]) + (n,), dev)
