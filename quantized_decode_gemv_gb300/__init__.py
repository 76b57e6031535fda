"""Python binding of libqdecode (argument marshalling only).

Every function here forwards to the C entry point of the same name in ``include/qdecode.h``
(without the ``qd_`` prefix): device tensors are passed as ``data_ptr()`` and the stream as
``torch.cuda.current_stream().cuda_stream`` unless given.  All arithmetic runs in the CUDA
library.  There is no fallback: if ``libqdecode.so`` is missing or does not load, every call
raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqdecode.so")
_lib = None

FMT = {"q4_0": 0, "q8_0": 1, "q4_k": 2, "i8": 3, "q4_1": 4, "q5_0": 5, "q5_k": 6, "q6_k": 7, "f16": 8, "i4": 9}
PAIRING = {"adjacent": 0, "half": 1}
MAX_BATCH = 16
STATUS = {0: "QD_OK", 1: "QD_ERR_INVALID_ARG", 2: "QD_ERR_SHAPE", 3: "QD_ERR_ALIGN", 4: "QD_ERR_UNSUPPORTED",
          5: "QD_ERR_CUDA", 6: "QD_ERR_NOMEM", 7: "QD_ERR_DEVICE_FLAG"}

# Every symbol include/qdecode.h declares (checked by the CPU test suite).
EXPORTS = ["qd_status_str", "qd_abi_version", "qd_f16_to_f32", "qd_bf16_to_f32", "qd_src_bytes", "qd_packed_bytes",
           "qd_repack", "qd_unpack", "qd_dequant", "qd_quantize_i8_rows", "qd_quantize_i4_rows",
           "qd_q_gemv_workspace", "qd_q_gemv",
           "qd_q_gemv_ex", "qd_read_ceiling", "qd_q_gemm_workspace", "qd_q_gemm", "qd_q8_bytes",
           "qd_quantize_q8", "qd_q_gemv_q8", "qd_rmsnorm",
           "qd_rope_table", "qd_rope", "qd_kv_append", "qd_gqa_decode_attn_workspace", "qd_gqa_decode_attn",
           "qd_gqa_decode_attn_noalloc",
           "qd_swiglu", "qd_argmax", "qd_embed", "qd_tree_plan", "qd_tree_append", "qd_tree_attn_workspace",
           "qd_tree_attn", "qd_token_logprobs", "qd_tree_commit", "qd_rope_plan", "qd_rope_tokens", "qd_paged_append",
           "qd_paged_attn_workspace", "qd_paged_attn", "qd_paged_read", "qd_model_weight_bytes", "qd_model_state_bytes",
           "qd_model_create", "qd_model_destroy", "qd_decode_step", "qd_prefill_workspace", "qd_prefill",
           "qd_model_reset", "qd_model_set_pos",
           "qd_model_pos", "qd_model_kv_cache", "qd_model_act_q8_buffer", "qd_model_check",
           "qd_model_launches_per_step", "qd_model_set_step_path", "qd_model_step_path",
           "qd_model_cluster_available"]
STEP_AUTO, STEP_KERNEL_CHAIN, STEP_CLUSTER = 0, 1, 2
PREFILL_EXACT = 1
MAX_TREE = 64
MAX_TOP = 32
KV_BLOCK = 16
MAX_SEQS = 256
KV_FMT = {"i8": 0, "e4m3": 1}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "turns": 3, "pairs": 4}


class QDError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} returned {STATUS.get(status, status)}")


class Config(ctypes.Structure):
    _fields_ = [("layers", ctypes.c_int), ("dim", ctypes.c_int), ("ffn", ctypes.c_int),
                ("n_heads", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("vocab", ctypes.c_int), ("max_ctx", ctypes.c_int), ("max_batch", ctypes.c_int),
                ("rope_theta", ctypes.c_float), ("eps", ctypes.c_float), ("pairing", ctypes.c_int),
                ("w_fmt", ctypes.c_int), ("emb_fmt", ctypes.c_int), ("tied", ctypes.c_int),
                ("kv_f16", ctypes.c_int), ("act_q8", ctypes.c_int), ("mixed_fmt", ctypes.c_int),
                ("qkv_fmt", ctypes.c_int), ("wo_fmt", ctypes.c_int), ("gate_up_fmt", ctypes.c_int),
                ("down_fmt", ctypes.c_int)]


class PagedKVStruct(ctypes.Structure):
    _fields_ = [("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_table", ctypes.c_void_p), ("n_pages", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("n_kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("max_seqs", ctypes.c_int), ("max_pages", ctypes.c_int), ("fmt", ctypes.c_int)]


def build(force: bool = False) -> str:
    from . import builder as _b

    return _b.build(force=force)


def load():
    """Load libqdecode.so (built in-tree by ``build()``); raises if it is absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libqdecode.so not built ({LIB_PATH}); run __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    p, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
    f64 = ctypes.c_double
    sig = {
        "qd_status_str": ([i32], ctypes.c_char_p),
        "qd_abi_version": ([], i32),
        "qd_f16_to_f32": ([p, p, i64, p], i32),
        "qd_bf16_to_f32": ([p, p, i64, p], i32),
        "qd_src_bytes": ([i32, i64, i64], sz),
        "qd_packed_bytes": ([i32, i64, i64], sz),
        "qd_repack": ([i32, p, i64, i64, p, sz, p], i32),
        "qd_unpack": ([i32, p, i64, i64, p, sz, p], i32),
        "qd_dequant": ([i32, p, i64, i64, p, p], i32),
        "qd_quantize_i8_rows": ([p, i64, i64, p, sz, p], i32),
        "qd_quantize_i4_rows": ([p, i64, i64, p, sz, p], i32),
        "qd_q_gemv_workspace": ([i32, i64, i64, i32], sz),
        "qd_q_gemv": ([i32, p, i64, i64, p, p, i32, p, sz, p], i32),
        "qd_q_gemv_ex": ([i32, p, i64, i64, p, p, i32, ctypes.c_uint, p], i32),
        "qd_read_ceiling": ([p, sz, i32, i32, ctypes.c_uint, p, p], i32),
        "qd_q_gemm_workspace": ([i32, i64, i64, i32], sz),
        "qd_q_gemm": ([i32, p, i64, i64, p, p, i32, p, sz, p], i32),
        "qd_q8_bytes": ([i32, i64, i32], sz),
        "qd_quantize_q8": ([p, i32, i64, i32, p, sz, p], i32),
        "qd_q_gemv_q8": ([i32, p, i64, i64, p, sz, p, i32, p], i32),
        "qd_rmsnorm": ([p, p, p, i32, i32, f32, p], i32),
        "qd_rope_table": ([f32, i32, i32, p], i32),
        "qd_rope": ([p, i32, i32, i64, p, i32, p, i32, i32, p], i32),
        "qd_kv_append": ([p, p, i64, p, p, i32, i32, p, i32, i32, p], i32),
        "qd_gqa_decode_attn_workspace": ([i32, i32, i32, i32], sz),
        "qd_gqa_decode_attn": ([p, i64, p, p, p, i32, i32, i32, p, i32, i32, p, sz, p], i32),
        "qd_gqa_decode_attn_noalloc": ([p, i64, p, p, p, i32, i32, i32, p, i32, i32, p], i32),
        "qd_swiglu": ([p, p, p, i64, i32, p], i32),
        "qd_argmax": ([p, i64, i32, p, p], i32),
        "qd_embed": ([i32, p, i64, i64, p, i32, p, p], i32),
        "qd_tree_plan": ([p, i32, p, p], i32),
        "qd_tree_append": ([p, p, p, i64, i64, p, p, p, i32, i32, i32, i32, p, p, p, i32, i32, p, i32, i32, p], i32),
        "qd_tree_attn_workspace": ([i32] * 6, sz),
        "qd_tree_attn": ([p, i64, p, p, p, p, i32, p, i32, i32, i32, p, p, p, i32, i32, i32, p, sz, p], i32),
        "qd_token_logprobs": ([p, i64, i64, i32, p, i32, p, p, i32, p, p, p], i32),
        "qd_tree_commit": ([p, p, p, i64, p, i32, p, p, p, p, i32, i32, i64, i32, i32, p, i32, i32, p, p, p, p, p],
                           i32),
        "qd_rope_plan": ([f64, i32, i32, f64, i32, f64, f64, p, p], i32),
        "qd_rope_tokens": ([p, i64, p, i64, i32, i32, i32, i32, p, i32, p, f64, p], i32),
        "qd_paged_append": ([p, p, p, p, i64, p, i32, i32, p, p, i32, i32, i32, p, f64, p], i32),
        "qd_paged_attn_workspace": ([p, i32, i32, i32], sz),
        "qd_paged_attn": ([p, p, i64, p, i32, i32, p, p, i32, f32, i32, p, sz, p], i32),
        "qd_paged_read": ([p, p, i32, i32, p, p, i32, p], i32),
        "qd_model_weight_bytes": ([ctypes.POINTER(Config)], sz),
        "qd_model_state_bytes": ([ctypes.POINTER(Config)], sz),
        "qd_model_create": ([ctypes.POINTER(Config), p, p, sz, p, sz, p, ctypes.POINTER(p)], i32),
        "qd_model_destroy": ([p], None),
        "qd_decode_step": ([p, p, i32, p, p, p], i32),
        "qd_prefill_workspace": ([ctypes.POINTER(Config), i32], sz),
        "qd_prefill": ([p, i32, p, i32, ctypes.c_uint, p, sz, p, p, p], i32),
        "qd_model_reset": ([p, p], i32),
        "qd_model_set_pos": ([p, p, i32, p], i32),
        "qd_model_pos": ([p, p, i32, p], i32),
        "qd_model_kv_cache": ([p, ctypes.POINTER(p), ctypes.POINTER(p)], i32),
        "qd_model_act_q8_buffer": ([p, ctypes.POINTER(p), ctypes.POINTER(sz), ctypes.POINTER(i32)], i32),
        "qd_model_check": ([p, p], i32),
        "qd_model_launches_per_step": ([p], i32),
        "qd_model_set_step_path": ([p, i32], i32),
        "qd_model_step_path": ([p], i32),
        "qd_model_cluster_available": ([p], i32),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


# ------------------------------------------------------------------------------ marshalling

def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, st: int):
    if st != 0:
        raise QDError(fn, st)


def status_str(s: int) -> str:
    return load().qd_status_str(s).decode()


def src_bytes(fmt: str, rows: int, cols: int) -> int:
    return int(load().qd_src_bytes(FMT[fmt], rows, cols))


def packed_bytes(fmt: str, rows: int, cols: int) -> int:
    return int(load().qd_packed_bytes(FMT[fmt], rows, cols))


def f16_to_f32(inp, out, n=None, stream=None):
    n = inp.numel() if n is None else n
    _check("qd_f16_to_f32", load().qd_f16_to_f32(_ptr(inp), _ptr(out), n, _stream(stream)))


def bf16_to_f32(inp, out, n=None, stream=None):
    n = inp.numel() if n is None else n
    _check("qd_bf16_to_f32", load().qd_bf16_to_f32(_ptr(inp), _ptr(out), n, _stream(stream)))


def repack(fmt, src, rows, cols, dst, dst_bytes=None, stream=None):
    nbytes = dst.numel() * dst.element_size() if dst_bytes is None else dst_bytes
    _check("qd_repack", load().qd_repack(FMT[fmt], _ptr(src), rows, cols, _ptr(dst), nbytes, _stream(stream)))


def unpack(fmt, packed, rows, cols, dst, dst_bytes=None, stream=None):
    nbytes = dst.numel() * dst.element_size() if dst_bytes is None else dst_bytes
    _check("qd_unpack", load().qd_unpack(FMT[fmt], _ptr(packed), rows, cols, _ptr(dst), nbytes, _stream(stream)))


def dequant(fmt, packed, rows, cols, out, stream=None):
    _check("qd_dequant", load().qd_dequant(FMT[fmt], _ptr(packed), rows, cols, _ptr(out), _stream(stream)))


def quantize_i4_rows(w_bf16, rows, cols, out, out_bytes=None, stream=None):
    nbytes = out.numel() * out.element_size() if out_bytes is None else out_bytes
    _check("qd_quantize_i4_rows", load().qd_quantize_i4_rows(_ptr(w_bf16), rows, cols, _ptr(out), nbytes,
                                                             _stream(stream)))


def quantize_i8_rows(w_bf16, rows, cols, out, out_bytes=None, stream=None):
    """BF16 weights (uint16/int16/bfloat16 tensor [rows][cols]) -> per-row INT8 source layout."""
    nbytes = out.numel() * out.element_size() if out_bytes is None else out_bytes
    _check("qd_quantize_i8_rows",
           load().qd_quantize_i8_rows(_ptr(w_bf16), rows, cols, _ptr(out), nbytes, _stream(stream)))


def q_gemv_workspace(fmt, rows, cols, batch) -> int:
    return int(load().qd_q_gemv_workspace(FMT[fmt], rows, cols, batch))


def q_gemm_workspace(fmt, rows, cols, t) -> int:
    return int(load().qd_q_gemm_workspace(FMT[fmt], rows, cols, t))


def q_gemm(fmt, W, rows, cols, x, y, t, workspace, workspace_bytes=None, stream=None):
    """y[n][r] = sum_c deq(W)[r][c] x[n][c] for n < t on the tensor cores (see qdecode.h)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check("qd_q_gemm", load().qd_q_gemm(FMT[fmt], _ptr(W), rows, cols, _ptr(x), _ptr(y), t, _ptr(workspace),
                                         workspace_bytes, _stream(stream)))


def q8_bytes(batch, cols, with_sum=False) -> int:
    return int(load().qd_q8_bytes(batch, cols, 1 if with_sum else 0))


def quantize_q8(x, batch, cols, out, with_sum=False, out_bytes=None, stream=None):
    """ggml-exact Q8_0 (Q8_1 with with_sum) activations of x [batch][cols] into out."""
    nbytes = out.numel() * out.element_size() if out_bytes is None else out_bytes
    _check("qd_quantize_q8", load().qd_quantize_q8(_ptr(x), batch, cols, 1 if with_sum else 0, _ptr(out), nbytes,
                                                   _stream(stream)))


def q_gemv_q8(fmt, W, rows, cols, xq, y, batch, xq_bytes=None, stream=None):
    """y = W x over quantised activations xq (quantize_q8 output) in integers."""
    nbytes = xq.numel() * xq.element_size() if xq_bytes is None else xq_bytes
    _check("qd_q_gemv_q8", load().qd_q_gemv_q8(FMT[fmt], _ptr(W), rows, cols, _ptr(xq), nbytes, _ptr(y), batch,
                                               _stream(stream)))


def q_gemv(fmt, W, rows, cols, x, y, batch, workspace=None, workspace_bytes=0, stream=None):
    _check("qd_q_gemv", load().qd_q_gemv(FMT[fmt], _ptr(W), rows, cols, _ptr(x), _ptr(y), batch, _ptr(workspace),
                                         workspace_bytes, _stream(stream)))


GEMV_OVERLAP = 1


def q_gemv_ex(fmt, W, rows, cols, x, y, batch, flags=0, stream=None):
    _check("qd_q_gemv_ex", load().qd_q_gemv_ex(FMT[fmt], _ptr(W), rows, cols, _ptr(x), _ptr(y), batch, flags,
                                               _stream(stream)))


def read_ceiling(buf, nbytes, ctas_per_sm, threads, flags=0, sink=None, stream=None):
    """Roofline calibration: one plain read of nbytes of buf (see qd_read_ceiling)."""
    _check("qd_read_ceiling", load().qd_read_ceiling(_ptr(buf), nbytes, ctas_per_sm, threads, flags, _ptr(sink),
                                                     _stream(stream)))


def rmsnorm(x, g, out, n, batch, eps, stream=None):
    _check("qd_rmsnorm", load().qd_rmsnorm(_ptr(x), _ptr(g), _ptr(out), n, batch, eps, _stream(stream)))


def rope_table(theta, head_dim, ctx, dst_host_ptr):
    _check("qd_rope_table", load().qd_rope_table(theta, head_dim, ctx, dst_host_ptr))


def rope(v, n_heads, head_dim, batch_stride, pos, pairing, cos_sin, max_ctx, batch, stream=None):
    _check("qd_rope", load().qd_rope(_ptr(v), n_heads, head_dim, batch_stride, _ptr(pos), PAIRING[pairing],
                                     _ptr(cos_sin), max_ctx, batch, _stream(stream)))


def kv_append(k, v, src_batch_stride, k_cache, v_cache, n_kv_heads, head_dim, pos, max_ctx, batch, stream=None):
    _check("qd_kv_append", load().qd_kv_append(_ptr(k), _ptr(v), src_batch_stride, _ptr(k_cache), _ptr(v_cache),
                                               n_kv_heads, head_dim, _ptr(pos), max_ctx, batch, _stream(stream)))


def gqa_decode_attn_workspace(n_heads, head_dim, max_ctx, batch) -> int:
    return int(load().qd_gqa_decode_attn_workspace(n_heads, head_dim, max_ctx, batch))


def gqa_decode_attn(q, q_batch_stride, k_cache, v_cache, out, n_heads, n_kv_heads, head_dim, pos, max_ctx, batch,
                    workspace, workspace_bytes, stream=None):
    _check("qd_gqa_decode_attn",
           load().qd_gqa_decode_attn(_ptr(q), q_batch_stride, _ptr(k_cache), _ptr(v_cache), _ptr(out), n_heads,
                                     n_kv_heads, head_dim, _ptr(pos), max_ctx, batch, _ptr(workspace),
                                     workspace_bytes, _stream(stream)))


def gqa_decode_attn_noalloc(q, q_batch_stride, k_cache, v_cache, out, n_heads, n_kv_heads, head_dim, pos, max_ctx,
                            batch, stream=None):
    """Attention without a caller workspace (the library's fixed device scratch)."""
    _check("qd_gqa_decode_attn_noalloc",
           load().qd_gqa_decode_attn_noalloc(_ptr(q), q_batch_stride, _ptr(k_cache), _ptr(v_cache), _ptr(out),
                                             n_heads, n_kv_heads, head_dim, _ptr(pos), max_ctx, batch,
                                             _stream(stream)))


def swiglu(gate, up, out, n, batch, stream=None):
    _check("qd_swiglu", load().qd_swiglu(_ptr(gate), _ptr(up), _ptr(out), n, batch, _stream(stream)))


def argmax(logits, n, batch, out_idx, stream=None):
    _check("qd_argmax", load().qd_argmax(_ptr(logits), n, batch, _ptr(out_idx), _stream(stream)))


def embed(fmt, E, vocab, dim, tokens, batch, x, stream=None):
    _check("qd_embed", load().qd_embed(FMT[fmt], _ptr(E), vocab, dim, _ptr(tokens), batch, _ptr(x),
                                       _stream(stream)))


def _here(stream):
    """(raw stream, index of the current device); `stream` as in _stream."""
    import torch

    dev = torch.cuda.current_device()
    if stream is None:  # what torch.cuda.current_stream() wraps, without the wrapper's 3 us
        return torch._C._cuda_getCurrentRawStream(dev), dev
    return _stream(stream), dev


@functools.lru_cache(maxsize=1024)  # 0.4 us instead of 1.2 for a view of four dimensions
def _extent(shape, strides, steps):
    """Elements from a view's first one to its last; None where a dimension leaves a gap that is
    not one of `steps` (if there are any)."""
    n = dense = 1
    for size, stride in zip(reversed(shape), reversed(strides)):
        if size != 1:
            if stride != dense and steps and stride not in steps:
                return None
            n += (size - 1) * stride
            dense = size * stride
    return n


def _room(fn, name, t, dtype, dev, n, stepped=False, steps=()):
    """Pointer of t after a look at what only the tensor tells: its type, its device, that n
    elements lie behind its pointer, so that a tensor too small is an error here and not a read
    out of bounds on the device, and that they lie there in the order of its dimensions.  Only a
    `stepped` argument may be a view with gaps, and those have to be the `steps`, the strides that
    the call is given (none: any).  Raw pointers and None pass as they are."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is not dtype:
        raise ValueError(f"{fn}: {name} has type {t.dtype}, not {dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{fn}: {name} is on {t.device}, not on the current device")
    if t.is_contiguous():
        have = t.numel()
    elif not stepped:
        raise ValueError(f"{fn}: {name} is not contiguous")
    else:
        have = _extent(t.shape, t.stride(), steps)
        if have is None:
            raise ValueError(f"{fn}: {name} has strides {t.stride()}, the call takes {steps} and no other gaps")
    if have < n:
        if stepped:
            have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
        if have < n:
            raise ValueError(f"{fn}: {name} holds {have} elements, the call takes {n}")
    return t.data_ptr()


def tree_plan(parent):
    """Ancestor masks (int64 bit patterns) and depths (int32) of one tree, parent[i] that of node i, as
    CPU tensors; a batch stacks those of its trees."""
    import torch

    given = torch.as_tensor(parent, device="cpu")
    if given.dim() != 1:
        raise ValueError(f"qd_tree_plan: parent has {given.dim()} dimensions, one tree has one")
    par = given.to(torch.int32).contiguous()
    if not torch.equal(par.to(given.dtype), given):
        raise ValueError("qd_tree_plan: the parents are not whole numbers of 32 bits")
    mask, depth = torch.empty(par.numel(), dtype=torch.int64), torch.empty(par.numel(), dtype=torch.int32)
    _check("qd_tree_plan", load().qd_tree_plan(par.data_ptr(), par.numel(), mask.data_ptr(), depth.data_ptr()))
    return mask, depth


def tree_append(q, k, v, batch_stride, node_stride, q_out, k_draft, v_draft, n_heads, n_kv_heads, head_dim, pos, depth,
                n_valid, n_nodes, pairing, cos_sin, max_ctx, batch, kv_f16=False, stream=None):
    """Rotated queries into q_out, rotated keys and values into the draft buffers (see qdecode.h)."""
    import torch

    fn, f32, i32, (st, dev) = "qd_tree_append", torch.float32, torch.int32, _here(stream)
    kv = torch.float16 if kv_f16 else f32
    last = (batch - 1) * batch_stride + (n_nodes - 1) * node_stride
    qn, kn, steps = n_heads * head_dim, n_kv_heads * head_dim, (batch_stride, node_stride)
    _check(fn, load().qd_tree_append(
        _room(fn, "q", q, f32, dev, last + qn, True, steps),
        _room(fn, "k", k, f32, dev, last + kn, True, steps),
        _room(fn, "v", v, f32, dev, last + kn, True, steps), batch_stride, node_stride,
        _room(fn, "q_out", q_out, f32, dev, batch * n_nodes * qn),
        _room(fn, "k_draft", k_draft, kv, dev, batch * n_nodes * kn),
        _room(fn, "v_draft", v_draft, kv, dev, batch * n_nodes * kn), 1 if kv_f16 else 0, n_heads, n_kv_heads,
        head_dim, _room(fn, "pos", pos, i32, dev, batch), _room(fn, "depth", depth, i32, dev, batch * n_nodes),
        _room(fn, "n_valid", n_valid, i32, dev, batch), n_nodes, PAIRING[pairing],
        _room(fn, "cos_sin", cos_sin, f32, dev, max_ctx * head_dim), max_ctx, batch, st))


def tree_attn_workspace(n_heads, n_kv_heads, head_dim, n_nodes, max_ctx, batch) -> int:
    return int(load().qd_tree_attn_workspace(n_heads, n_kv_heads, head_dim, n_nodes, max_ctx, batch))


def tree_attn(q, q_batch_stride, k_cache, v_cache, k_draft, v_draft, out, n_heads, n_kv_heads, head_dim, pos, mask,
              n_valid, n_nodes, max_ctx, batch, workspace, workspace_bytes=None, kv_f16=False, stream=None):
    """Attention of the tree over the cache and its own drafts (see qdecode.h)."""
    import torch

    fn, f32, i32, (st, dev) = "qd_tree_attn", torch.float32, torch.int32, _here(stream)
    kv = torch.float16 if kv_f16 else f32
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    qn, kn = n_nodes * n_heads * head_dim, batch * n_nodes * n_kv_heads * head_dim
    cn = batch * n_kv_heads * max_ctx * head_dim
    _check(fn, load().qd_tree_attn(
        _room(fn, "q", q, f32, dev, (batch - 1) * q_batch_stride + qn, True, (q_batch_stride,)), q_batch_stride,
        _room(fn, "k_cache", k_cache, kv, dev, cn), _room(fn, "v_cache", v_cache, kv, dev, cn),
        _room(fn, "k_draft", k_draft, kv, dev, kn), _room(fn, "v_draft", v_draft, kv, dev, kn), 1 if kv_f16 else 0,
        _room(fn, "out", out, f32, dev, batch * qn), n_heads, n_kv_heads, head_dim,
        _room(fn, "pos", pos, i32, dev, batch), _room(fn, "mask", mask, torch.int64, dev, batch * n_nodes),
        _room(fn, "n_valid", n_valid, i32, dev, batch), n_nodes, max_ctx, batch,
        _room(fn, "workspace", workspace, torch.uint8, dev, workspace_bytes), workspace_bytes, st))


def token_logprobs(logits, row_stride, vocab, rows, tokens, n_tokens, logprob, entropy, top_k, top_idx, top_logprob,
                   stream=None):
    """Log probabilities of tokens, entropy and the top alternatives of each row of logits (see qdecode.h)."""
    import torch

    fn, f32, i32, (st, dev) = "qd_token_logprobs", torch.float32, torch.int32, _here(stream)
    _check(fn, load().qd_token_logprobs(
        _room(fn, "logits", logits, f32, dev, (rows - 1) * row_stride + vocab, True, (row_stride,)), row_stride, vocab,
        rows, _room(fn, "tokens", tokens, i32, dev, rows * n_tokens), n_tokens,
        _room(fn, "logprob", logprob, f32, dev, rows * n_tokens), _room(fn, "entropy", entropy, f32, dev, rows), top_k,
        _room(fn, "top_idx", top_idx, i32, dev, rows * top_k),
        _room(fn, "top_logprob", top_logprob, f32, dev, rows * top_k), st))


def tree_commit(tokens, parent, chosen, chosen_stride, n_valid, n_nodes, k_draft, v_draft, k_cache, v_cache, layers,
                cache_layer_stride, n_kv_heads, head_dim, pos, max_ctx, batch, path, n_accept, next_token, pos_out,
                kv_f16=False, stream=None):
    """Accept a path of each tree and copy its rows of every layer into the caches (see qdecode.h)."""
    import torch

    fn, i32, (st, dev) = "qd_tree_commit", torch.int32, _here(stream)
    kv = torch.float16 if kv_f16 else torch.float32
    nodes, dn = batch * n_nodes, layers * batch * n_nodes * n_kv_heads * head_dim
    cn = (layers - 1) * cache_layer_stride + batch * n_kv_heads * max_ctx * head_dim
    _check(fn, load().qd_tree_commit(
        _room(fn, "tokens", tokens, i32, dev, nodes), _room(fn, "parent", parent, i32, dev, nodes),
        _room(fn, "chosen", chosen, i32, dev, (nodes - 1) * chosen_stride + 1, True, (chosen_stride,)), chosen_stride,
        _room(fn, "n_valid", n_valid, i32, dev, batch), n_nodes, _room(fn, "k_draft", k_draft, kv, dev, dn),
        _room(fn, "v_draft", v_draft, kv, dev, dn),
        _room(fn, "k_cache", k_cache, kv, dev, cn, True, (cache_layer_stride,)),
        _room(fn, "v_cache", v_cache, kv, dev, cn, True, (cache_layer_stride,)), 1 if kv_f16 else 0, layers,
        cache_layer_stride, n_kv_heads, head_dim, _room(fn, "pos", pos, i32, dev, batch), max_ctx, batch,
        _room(fn, "path", path, i32, dev, nodes),
        _room(fn, "n_accept", n_accept, i32, dev, batch), _room(fn, "next_token", next_token, i32, dev, batch),
        _room(fn, "pos_out", pos_out, i32, dev, batch), st))


def rope_plan(theta, rot_dim, scaling="none", factor=1.0, trained_ctx=0, low=1.0, high=32.0):
    """(turns, magnitude) of qd_rope_plan: int64 bit patterns [rot_dim / 2] as a CPU tensor, and a float."""
    import torch

    turns = torch.empty(max(int(rot_dim) // 2, 1), dtype=torch.int64)
    magnitude = ctypes.c_double()
    _check("qd_rope_plan", load().qd_rope_plan(theta, rot_dim, ROPE_SCALING[scaling], factor, trained_ctx, low, high,
                                               turns.data_ptr(), ctypes.byref(magnitude)))
    return turns, magnitude.value


def rope_tokens(x, x_stride, out, out_stride, n_tokens, n_heads, head_dim, rot_dim, pos, pairing, turns, magnitude=1.0,
                stream=None):
    """RoPE of packed rows at positions pos, the first rot_dim dimensions of each head (see qdecode.h)."""
    import torch

    fn, f32, (st, dev) = "qd_rope_tokens", torch.float32, _here(stream)
    row = n_heads * head_dim
    _check(fn, load().qd_rope_tokens(
        _room(fn, "x", x, f32, dev, (n_tokens - 1) * x_stride + row, True, (x_stride,)), x_stride,
        _room(fn, "out", out, f32, dev, (n_tokens - 1) * out_stride + row, True, (out_stride,)), out_stride, n_tokens,
        n_heads, head_dim, rot_dim, _room(fn, "pos", pos, torch.int32, dev, n_tokens), PAIRING[pairing],
        _room(fn, "turns", turns, torch.int64, dev, rot_dim // 2), magnitude, st))


class PagedKV:
    """One layer's paged cache (qd_paged_kv) over the caller's tensors, which it keeps alive: codes
    [n_pages][n_kv_heads][page_tokens][head_dim] (int8 or uint8, float8_e4m3fn too for "e4m3"), scales f32
    [n_pages][n_kv_heads][page_tokens / 16], page_table int32 [max_seqs][max_pages]."""

    def __init__(self, k_pages, v_pages, k_scale, v_scale, page_table, fmt="i8"):
        import torch

        kinds = (torch.int8, torch.uint8) + ((torch.float8_e4m3fn,) if fmt == "e4m3" else ())
        if k_pages.dim() != 4 or k_scale.dim() != 3 or page_table.dim() != 2:
            raise ValueError("PagedKV: pages have 4 dimensions, scales 3, the page table 2")
        n, hk, tokens, hd = k_pages.shape
        dev = k_pages.get_device()
        for name, t, kind, shape in (("k_pages", k_pages, kinds, (n, hk, tokens, hd)),
                                     ("v_pages", v_pages, kinds, (n, hk, tokens, hd)),
                                     ("k_scale", k_scale, (torch.float32,), (n, hk, tokens // KV_BLOCK)),
                                     ("v_scale", v_scale, (torch.float32,), (n, hk, tokens // KV_BLOCK)),
                                     ("page_table", page_table, (torch.int32,), tuple(page_table.shape))):
            if t.dtype not in kind:
                raise ValueError(f"PagedKV: {name} has type {t.dtype}, not {' or '.join(map(str, kind))}")
            if tuple(t.shape) != shape:
                raise ValueError(f"PagedKV: {name} has shape {tuple(t.shape)}, not {shape}")
            if not t.is_contiguous():
                raise ValueError(f"PagedKV: {name} is not contiguous")
            if t.get_device() != dev:
                raise ValueError(f"PagedKV: {name} is on {t.device}, k_pages on {k_pages.device}")
        self.tensors = (k_pages, v_pages, k_scale, v_scale, page_table)
        self.device, self.n_kv_heads, self.head_dim = dev, hk, hd
        self.max_seqs, self.max_pages = page_table.shape
        self.struct = PagedKVStruct(*(t.data_ptr() for t in self.tensors), n, tokens, hk, hd, self.max_seqs,
                                    self.max_pages, KV_FMT[fmt])
        self.ptr = ctypes.addressof(self.struct)


def _paged(fn, kv, dev):
    if kv.device != dev:
        raise ValueError(f"{fn}: the cache is on device {kv.device}, not on the current device")
    return kv.ptr


def paged_append(kv, q, k, v, token_stride, q_out, n_heads, n_tokens, row_start, pos, n_seqs, rot_dim, pairing, turns,
                 magnitude=1.0, stream=None):
    """Rotated queries into q_out, rotated keys and values into the pages of kv (see qdecode.h)."""
    import torch

    fn, f32, i32, (st, dev) = "qd_paged_append", torch.float32, torch.int32, _here(stream)
    hd = kv.head_dim
    last, qn, kn, steps = (n_tokens - 1) * token_stride, n_heads * hd, kv.n_kv_heads * hd, (token_stride,)
    _check(fn, load().qd_paged_append(
        _paged(fn, kv, dev), _room(fn, "q", q, f32, dev, last + qn, True, steps),
        _room(fn, "k", k, f32, dev, last + kn, True, steps), _room(fn, "v", v, f32, dev, last + kn, True, steps),
        token_stride, _room(fn, "q_out", q_out, f32, dev, n_tokens * qn), n_heads, n_tokens,
        _room(fn, "row_start", row_start, i32, dev, n_seqs + 1), _room(fn, "pos", pos, i32, dev, n_seqs), n_seqs, rot_dim,
        PAIRING[pairing], _room(fn, "turns", turns, torch.int64, dev, rot_dim // 2), magnitude, st))


def paged_attn_workspace(kv, n_heads, n_tokens, n_seqs) -> int:
    return int(load().qd_paged_attn_workspace(kv.ptr, n_heads, n_tokens, n_seqs))


def paged_attn(kv, q, q_stride, out, n_heads, n_tokens, row_start, pos, n_seqs, scale, window, workspace,
               workspace_bytes=None, stream=None):
    """Causal attention of packed rows over the pages of kv (see qdecode.h)."""
    import torch

    fn, f32, i32, (st, dev) = "qd_paged_attn", torch.float32, torch.int32, _here(stream)
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    qn = n_heads * kv.head_dim
    _check(fn, load().qd_paged_attn(
        _paged(fn, kv, dev), _room(fn, "q", q, f32, dev, (n_tokens - 1) * q_stride + qn, True, (q_stride,)), q_stride,
        _room(fn, "out", out, f32, dev, n_tokens * qn), n_heads, n_tokens,
        _room(fn, "row_start", row_start, i32, dev, n_seqs + 1), _room(fn, "pos", pos, i32, dev, n_seqs), n_seqs, scale,
        window, _room(fn, "workspace", workspace, torch.uint8, dev, workspace_bytes), workspace_bytes, st))


def paged_read(kv, length, n_seqs, max_ctx, k_out, v_out, out_f16=False, stream=None):
    """Sequences of kv as contiguous f32 (binary16 with out_f16) caches (see qdecode.h)."""
    import torch

    fn, (st, dev) = "qd_paged_read", _here(stream)
    kind = torch.float16 if out_f16 else torch.float32
    n = n_seqs * kv.n_kv_heads * max_ctx * kv.head_dim
    _check(fn, load().qd_paged_read(
        _paged(fn, kv, dev), _room(fn, "len", length, torch.int32, dev, n_seqs), n_seqs, max_ctx,
        _room(fn, "k_out", k_out, kind, dev, n), _room(fn, "v_out", v_out, kind, dev, n), 1 if out_f16 else 0, st))


def make_config(cfg: dict, max_ctx: int, max_batch: int, tied: bool = True, kv_f16: bool | None = None,
                act_q8: bool | None = None) -> Config:
    """kv_f16: binary16 KV cache (default: cfg.get("kv_f16", False)); act_q8: products over
    Q8_0 activations (default: cfg.get("act_q8", False)).  A config naming any of qkv_fmt,
    wo_fmt, gate_up_fmt or down_fmt is a mixed-format model (the classes it does not name
    take w_fmt)."""
    f16 = cfg.get("kv_f16", False) if kv_f16 is None else kv_f16
    q8 = cfg.get("act_q8", False) if act_q8 is None else act_q8
    classes = ("qkv_fmt", "wo_fmt", "gate_up_fmt", "down_fmt")
    mixed = any(k in cfg for k in classes)
    per = [FMT[cfg.get(k, cfg["w_fmt"])] for k in classes]
    return Config(cfg["layers"], cfg["dim"], cfg["ffn"], cfg["n_heads"], cfg["n_kv_heads"], cfg["head_dim"],
                  cfg["vocab"], max_ctx, max_batch, cfg["rope_theta"], cfg["eps"], PAIRING[cfg["pairing"]],
                  FMT[cfg["w_fmt"]], FMT[cfg["emb_fmt"]], 1 if tied else 0, 1 if f16 else 0, 1 if q8 else 0,
                  1 if mixed else 0, *per)


class Model:
    """A decode model over caller-owned device memory (torch uint8 tensors)."""

    def __init__(self, cfg: Config, src_tensors: list, stream=None):
        import torch

        lib = load()
        self.cfg = cfg
        wb = lib.qd_model_weight_bytes(ctypes.byref(cfg))
        sb = lib.qd_model_state_bytes(ctypes.byref(cfg))
        if not wb or not sb:
            raise QDError("qd_model_weight_bytes", 4)
        self.weights = torch.empty(wb, dtype=torch.uint8, device="cuda")
        self.state = torch.empty(sb, dtype=torch.uint8, device="cuda")
        ptrs = (ctypes.c_void_p * len(src_tensors))(*[_ptr(t) for t in src_tensors])
        h = ctypes.c_void_p()
        _check("qd_model_create", lib.qd_model_create(ctypes.byref(cfg), ptrs, self.weights.data_ptr(), wb,
                                                      self.state.data_ptr(), sb, _stream(stream), ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            load().qd_model_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def decode_step(self, tokens, batch, out_tokens, logits_out=None, stream=None):
        """tokens / out_tokens / logits_out: torch tensors (host or device) or raw pointers."""
        _check("qd_decode_step", load().qd_decode_step(self.handle, _ptr(tokens), batch, _ptr(out_tokens),
                                                       _ptr(logits_out), _stream(stream)))

    def prefill_workspace(self, t):
        """Bytes of the workspace qd_prefill needs for t tokens (0: not available)."""
        return load().qd_prefill_workspace(ctypes.byref(self.cfg), t)

    def prefill(self, seq, tokens, t, out_token, logits_out=None, flags=0, workspace=None, stream=None):
        """Run t prompt tokens of sequence seq in one call (qd_prefill).  tokens, out_token,
        logits_out: torch tensors (host or device) or raw pointers; workspace: a device
        tensor of at least prefill_workspace(t) bytes (allocated here when None)."""
        import torch

        need = self.prefill_workspace(t)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
        nbytes = workspace.numel() * workspace.element_size() if hasattr(workspace, "numel") else need
        _check("qd_prefill", load().qd_prefill(self.handle, seq, _ptr(tokens), t, flags, _ptr(workspace), nbytes,
                                               _ptr(out_token), _ptr(logits_out), _stream(stream)))

    def reset(self, stream=None):
        _check("qd_model_reset", load().qd_model_reset(self.handle, _stream(stream)))

    def set_pos(self, pos_list, stream=None):
        arr = (ctypes.c_int32 * len(pos_list))(*pos_list)
        _check("qd_model_set_pos", load().qd_model_set_pos(self.handle, arr, len(pos_list), _stream(stream)))

    def pos(self, batch, stream=None):
        arr = (ctypes.c_int32 * batch)()
        _check("qd_model_pos", load().qd_model_pos(self.handle, arr, batch, _stream(stream)))
        return list(arr)

    def kv_cache_ptrs(self):
        k, v = ctypes.c_void_p(), ctypes.c_void_p()
        _check("qd_model_kv_cache", load().qd_model_kv_cache(self.handle, ctypes.byref(k), ctypes.byref(v)))
        return k.value, v.value

    def act_q8_buffer(self):
        """(device pointer, bytes per slot, slots) of the act_q8 quantised inputs of the last
        step ((None, 0, 0) without act_q8)."""
        b, n, k = ctypes.c_void_p(), ctypes.c_size_t(), ctypes.c_int()
        _check("qd_model_act_q8_buffer", load().qd_model_act_q8_buffer(self.handle, ctypes.byref(b), ctypes.byref(n),
                                                                       ctypes.byref(k)))
        return b.value, n.value, k.value

    def check(self, stream=None) -> int:
        return int(load().qd_model_check(self.handle, _stream(stream)))

    def set_step_path(self, path: int):
        """STEP_AUTO, STEP_KERNEL_CHAIN or STEP_CLUSTER (see qd_model_set_step_path)."""
        _check("qd_model_set_step_path", load().qd_model_set_step_path(self.handle, int(path)))

    def step_path(self) -> int:
        return int(load().qd_model_step_path(self.handle))

    def cluster_available(self) -> bool:
        return bool(load().qd_model_cluster_available(self.handle))

    def launches_per_step(self) -> int:
        return int(load().qd_model_launches_per_step(self.handle))
