"""Python binding of the paged quantized KV-cache library (libkvq.so, sm_103a).

Thin argument marshalling over the C ABI declared in ``include/kvq.h``: every
function below has the C function's name, checks dtypes/devices of the torch
tensors it is given, and passes raw device pointers, sizes and the current
CUDA stream.  All computation happens in the CUDA kernels of libkvq.so; there
is no CPU fallback, and importing a function whose library is missing raises.

Method: decode-step attention over a block-paged KV cache stored as INT8/FP8
codes with per-token, per-channel or per-group fp32 scales, or FP16
("KV Cache优化实战：大模型推理显存占用与加速方案详解", 0539edu.com/news/5800990,
§1.1, §2.1-§2.3, §3.3, §4.3).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "kvq.h")

# kvq_dtype
KVQ_FP16 = 0
KVQ_INT8_PER_TOKEN = 1
KVQ_INT8_PER_CHANNEL = 2
KVQ_INT8_PER_GROUP = 3
KVQ_FP8_E4M3_PER_TOKEN = 4
KVQ_INT4_PER_GROUP = 5
KVQ_FP8_E5M2 = 6
KVQ_INT8_PER_BLOCK = 7
KVQ_FP8_E4M3_PER_BLOCK = 8
GROUP_FORMATS = (KVQ_INT8_PER_GROUP, KVQ_INT4_PER_GROUP)
BLOCK_FORMATS = (KVQ_INT8_PER_BLOCK, KVQ_FP8_E4M3_PER_BLOCK)

# kvq_rope_layout, kvq_rope_scaling, kvq_x_type
KVQ_ROPE_HALF = 0
KVQ_ROPE_INTERLEAVED = 1
KVQ_ROPE_NONE = 0
KVQ_ROPE_LINEAR = 1
KVQ_ROPE_BASE = 2
KVQ_ROPE_PARTS = 3
KVQ_ROPE_BANDS = 4
KVQ_ROPE_MAX_PAIRS = 64
KVQ_X_FP16 = 0
KVQ_X_BF16 = 1

# kvq_status
KVQ_OK = 0
KVQ_ERR_INVALID_ARG = 1
KVQ_ERR_UNSUPPORTED = 2
KVQ_ERR_CUDA = 3
KVQ_ERR_OUT_OF_RANGE = 4
KVQ_ERR_WORKSPACE = 5
KVQ_ERR_TIMEOUT = 6

_lock = threading.Lock()
_lib = None


class KVQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (where, kvq_status_string(status), status))


class _Layout(ctypes.Structure):
    _fields_ = [("total_bytes", ctypes.c_size_t), ("code_bytes", ctypes.c_size_t),
                ("scale_bytes", ctypes.c_size_t), ("header_bytes", ctypes.c_size_t),
                ("page_bytes", ctypes.c_size_t)]


class _RopeConfig(ctypes.Structure):
    _fields_ = [("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int), ("scaling", ctypes.c_int),
                ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("orig_len", ctypes.c_double), ("low", ctypes.c_double), ("high", ctypes.c_double),
                ("magnitude", ctypes.c_double)]


class RopePlan(ctypes.Structure):
    """kvq_rope_plan: a rotation made by kvq_rope_init (plain host data)."""

    _fields_ = [("rotary_dim", ctypes.c_int), ("layout", ctypes.c_int),
                ("magnitude", ctypes.c_float), ("reserved", ctypes.c_int),
                ("turns", ctypes.c_uint64 * KVQ_ROPE_MAX_PAIRS)]


class PoolHandle(ctypes.c_void_p):
    """A kvq_pool* with the shape it was allocated with: (block_size, kv_heads,
    head_dim).  The library sees addresses only; tensors are held against this."""

    _shape = None
    rows = None  # (kv_heads, head_dim) of a token, as a tensor's shape would have them

    @property
    def shape(self):
        return self._shape

    @shape.setter
    def shape(self, shape):
        self._shape, self.rows = shape, tuple(shape[1:])


def header_functions() -> list[str]:
    """Names of the functions include/kvq.h declares."""
    text = open(HEADER_PATH).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvq_[a-z0-9_]+)\s*\(", text)))


def lib() -> ctypes.CDLL:
    """The loaded libkvq.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libkvq.so is not built (run __graft_entry__.build() or "
                                   "python -m paged_quantized_kv_kvq_gb300.build)")
            L = ctypes.CDLL(LIB_PATH)
            _declare(L)
            _lib = L
        return _lib


def _declare(L):
    P, i32, i64, sz, f32 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t,
                            ctypes.c_float)
    sigs = {
        "kvq_pool_layout_query": (i32, [i64, i32, i32, i32, i32, i32, ctypes.POINTER(_Layout)]),
        "kvq_pool_bytes": (sz, [i64, i32, i32, i32, i32, i32]),
        "kvq_alloc_pool": (i32, [i64, i32, i32, i32, i32, i32, P, sz, ctypes.POINTER(P)]),
        "kvq_free_pool": (i32, [P]),
        "kvq_set_channel_scales": (i32, [P, P, P, P]),
        "kvq_calibrate_channel_scales": (i32, [P, P, P, i64, P]),
        "kvq_append": (i32, [P, P, P, P, i64, P]),
        "kvq_copy_blocks": (i32, [P, P, P, i32, P]),
        "kvq_append_strided": (i32, [P, P, P, i64, P, i64, P]),
        "kvq_paged_decode_strided": (i32, [P, P, i64, i32, i32, P, i32, P, i32, f32, P, i64, P, sz,
                                           P]),
        "kvq_decode_workspace_bytes": (sz, [P, i32, i32, i32]),
        "kvq_decode_workspace_bytes_ex": (sz, [P, i32, i32, i32, i32]),
        "kvq_paged_decode": (i32, [P, P, i32, i32, P, i32, P, i32, f32, P, P, sz, P]),
        "kvq_paged_decode_ex": (i32, [P, P, i32, i32, P, i32, P, i32, f32, P, P, sz, i32, P]),
        "kvq_paged_decode_noalloc": (i32, [P, P, i32, i32, P, i32, P, i32, f32, P, i32, P]),
        "kvq_decode_step": (i32, [P, P, P, P, i32, i32, P, i32, P, i32, f32, P, P, sz, P]),
        "kvq_cascade_workspace_bytes": (sz, [P, i32, i32, i32]),
        "kvq_prefill": (i32, [P, P, i32, i32, P, i32, P, i32, P, i32, f32, P, P]),
        "kvq_prefill_workspace_bytes": (sz, [P, i32, i32]),
        "kvq_prefill_ex": (i32, [P, P, i32, i32, P, i32, P, i32, P, i32, f32, P, P, sz, P]),
        "kvq_selftest_decode_timeout": (i32, [P, P, i32, i32, P, i32, P, i32, P, P, sz, i32, P]),
        "kvq_cascade_decode": (i32, [P, P, i32, i32, P, i32, P, i32, i32, f32, P, P, sz, P]),
        "kvq_cascade_decode_step": (i32, [P, P, P, P, i32, i32, P, i32, P, i32, i32, f32, P, P, sz,
                                          P]),
        "kvq_rope_init": (i32, [ctypes.POINTER(_RopeConfig), ctypes.POINTER(RopePlan)]),
        "kvq_rope": (i32, [ctypes.POINTER(RopePlan), i32, P, i64, i32, P, i64, i32, i32, P, i64, P, P,
                           f32, P, i64, P, i64, P]),
        "kvq_rope_append": (i32, [P, ctypes.POINTER(RopePlan), i32, P, i64, i32, P, i64, P, i64, P,
                                  P, i64, P, P, f32, P, i64, P]),
        "kvq_paged_decode_lse": (i32, [P, P, i32, i32, P, i32, P, i32, f32, P, P, P, sz, i32, P]),
        "kvq_attention_weights": (i32, [P, P, i32, i32, P, i32, P, i32, f32, P, f32, P, P, i64, P]),
        "kvq_evict_blocks": (i32, [P, P, i64, i32, P, i32, P, i32, i32, i32, i32, P, P, P, P, i64, P]),
        "kvq_read_values": (i32, [P, P, i64, P, P, P]),
        "kvq_read_slots": (i32, [P, P, i64, P, P, P]),
        "kvq_get_error": (i32, [P, P]),
        "kvq_status_string": (ctypes.c_char_p, [i32]),
        "kvq_set_phase_events": (i32, [P, i32]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args


def _check(st: int, where: str) -> None:
    if st != KVQ_OK:
        raise KVQError(st, where)


_torch = None


def _th():
    """torch, imported at the first call that has tensors (the library itself does
    without it)."""
    global _torch
    if _torch is None:
        import torch

        _torch = torch
    return _torch


def _stream(stream):
    if stream is None:
        torch = _th()
        try:  # the handle itself: building a Stream object costs more than a launch
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        except AttributeError:
            stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _on(stream):
    """Context in which tensors are allocated for `stream`, the one that will use them:
    filled in its order, and given to no other stream's work when they are freed while
    it still runs.  (The current stream's needs none.)"""
    if stream is None:
        return contextlib.nullcontext()
    torch = _th()
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def _ptr(t, dtype=None, name="tensor"):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


# ------------------------------------------------------------------ C ABI
def kvq_status_string(status: int) -> str:
    return lib().kvq_status_string(int(status)).decode()


def kvq_pool_layout_query(num_blocks, block_size, kv_heads, head_dim, dtype, group=0) -> dict:
    lay = _Layout()
    _check(lib().kvq_pool_layout_query(num_blocks, block_size, kv_heads, head_dim, dtype, group,
                                       ctypes.byref(lay)), "kvq_pool_layout_query")
    return {f: int(getattr(lay, f)) for f, _ in _Layout._fields_}


def kvq_pool_bytes(num_blocks, block_size, kv_heads, head_dim, dtype, group=0) -> int:
    return int(lib().kvq_pool_bytes(num_blocks, block_size, kv_heads, head_dim, dtype, group))


def kvq_alloc_pool(num_blocks, block_size, kv_heads, head_dim, dtype, group=0, device_buf=None):
    """Returns an opaque handle (a ctypes.c_void_p).  device_buf: optional torch
    uint8 CUDA tensor of at least kvq_pool_bytes(..) bytes, owned by the caller."""
    h = PoolHandle()
    ptr = _ptr(device_buf, name="device_buf") if device_buf is not None else None
    nbytes = device_buf.numel() * device_buf.element_size() if device_buf is not None else 0
    _check(lib().kvq_alloc_pool(num_blocks, block_size, kv_heads, head_dim, dtype, group, ptr,
                                nbytes, ctypes.byref(h)), "kvq_alloc_pool")
    h.shape = (block_size, kv_heads, head_dim)
    return h


def kvq_free_pool(pool) -> None:
    _check(lib().kvq_free_pool(pool), "kvq_free_pool")


def kvq_set_channel_scales(pool, k_scale, v_scale, stream=None) -> None:
    torch = _th()
    _check(lib().kvq_set_channel_scales(pool, _ptr(k_scale, torch.float32, "k_scale"),
                                        _ptr(v_scale, torch.float32, "v_scale"), _stream(stream)),
           "kvq_set_channel_scales")


def kvq_calibrate_channel_scales(pool, k, v, stream=None) -> None:
    torch = _th()
    _check(lib().kvq_calibrate_channel_scales(pool, _ptr(k, torch.float16, "k"),
                                              _ptr(v, torch.float16, "v"), k.shape[0],
                                              _stream(stream)), "kvq_calibrate_channel_scales")


def kvq_append(pool, k, v, slot_mapping, stream=None) -> None:
    torch = _th()
    if k.shape != v.shape or k.shape[0] != slot_mapping.numel():
        raise ValueError("k, v must be [T, kv_heads, head_dim] and slot_mapping [T]")
    _check(lib().kvq_append(pool, _ptr(k, torch.float16, "k"), _ptr(v, torch.float16, "v"),
                            _ptr(slot_mapping, torch.int64, "slot_mapping"), k.shape[0],
                            _stream(stream)), "kvq_append")


def _device():
    """The current GPU, on whose stream the kernels are launched: the one that every
    tensor of a call must be on.  -2, no tensor's device, without a GPU."""
    try:
        return _th()._C._cuda_getDevice()
    except (AttributeError, AssertionError, RuntimeError):
        return -2


def _at(t, dtype, name, dev):
    """_ptr of a tensor on GPU dev."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _rows_view(t, dtype, name):
    """Pointer and row stride (elements) of a [rows, heads, head_dim] view whose
    heads and channels are contiguous (a head slice of wider rows)."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    stride = t.stride()
    if len(stride) != 3 or stride[2] != 1 or stride[1] != t.shape[2]:
        raise ValueError("%s must be [rows, heads, head_dim] with contiguous heads" % name)
    return t.data_ptr(), stride[0]


def kvq_append_strided(pool, k, v, slot_mapping, stream=None) -> None:
    """kvq_append for head slices of wider token rows (per-head mixed precision)."""
    torch = _th()
    kp, ks = _rows_view(k, torch.float16, "k")
    vp, vs = _rows_view(v, torch.float16, "v")
    if ks != vs or k.shape != v.shape or k.shape[0] != slot_mapping.numel():
        raise ValueError("k and v must be equal-shaped views with the same row stride")
    _check(lib().kvq_append_strided(pool, kp, vp, ks, _ptr(slot_mapping, torch.int64, "slot_mapping"),
                                    k.shape[0], _stream(stream)), "kvq_append_strided")


def kvq_rope_init(rotary_dim, interleaved=False, scaling=KVQ_ROPE_NONE, base=10000.0, factor=1.0,
                  orig_len=0.0, low=0.0, high=0.0, magnitude=0.0) -> RopePlan:
    """A rotation for kvq_rope and kvq_rope_append (kvq_rope_init in include/kvq.h)."""
    cfg = _RopeConfig(rotary_dim, KVQ_ROPE_INTERLEAVED if interleaved else KVQ_ROPE_HALF, scaling,
                      base, factor, orig_len, low, high, magnitude)
    plan = RopePlan()
    _check(lib().kvq_rope_init(ctypes.byref(cfg), ctypes.byref(plan)), "kvq_rope_init")
    return plan


def _x_rows(t, dtype, T, D, name, dev):
    """_rows_view of rows that agree with the others in type, tokens and head_dim, and
    their heads."""
    shape, stride = t.shape, t.stride()
    if t.dtype != dtype or len(shape) != 3 or shape[0] != T or shape[2] != D:
        raise ValueError("%s must be [%d, heads, %d] of %s like the other rows" % (name, T, D, dtype))
    H = shape[1]
    if stride[2] != 1 or (stride[1] != D and H != 1):
        raise ValueError("%s must be [rows, heads, head_dim] with contiguous heads" % name)
    if t.get_device() != dev:
        raise ValueError("%s must be on the current CUDA device" % name)
    # (the stride along a dimension of one says nothing)
    return t.data_ptr(), stride[0] if T > 1 else H * D, H


def _pool_rows(pool):
    """(kv_heads, head_dim) of a handle made by kvq_alloc_pool; None for any other,
    which has to be the caller's care."""
    return getattr(pool, "rows", None)


def _seqs(pool, q, block_table, context_lens):
    """S, Hq of q [S, Hq, head_dim] and max_blocks_per_seq, held against each other and
    the pool."""
    shape, table = q.shape, block_table.shape
    if len(shape) != 3:
        raise ValueError("q must be [num_seqs, num_q_heads, head_dim]")
    S, Hq, D = shape
    rows = _pool_rows(pool)
    if rows is not None and (D != rows[1] or Hq % rows[0] != 0):
        raise ValueError("q must have the pool's head_dim of %d and a multiple of its %d kv heads"
                         % (rows[1], rows[0]))
    if len(table) != 2 or table[0] != S:
        raise ValueError("block_table must be [num_seqs, max_blocks_per_seq]")
    if context_lens.numel() != S:
        raise ValueError("context_lens must be [num_seqs]")
    return S, Hq, table[1]


def _scores_width(pool, scores, S):
    """Tokens of scores [S, kv_heads, tokens], held against the pool."""
    shape = scores.shape
    if len(shape) != 3 or shape[0] != S:
        raise ValueError("scores must be [num_seqs, kv_heads, tokens]")
    rows = _pool_rows(pool)
    if rows is not None and shape[1] != rows[0]:
        raise ValueError("scores must have the pool's %d kv heads" % rows[0])
    return shape[2]


def _x_type(dtype, name):
    torch = _th()
    if dtype is torch.float16:
        return KVQ_X_FP16
    if dtype is torch.bfloat16:
        return KVQ_X_BF16
    raise ValueError("%s must be float16 or bfloat16, got %s" % (name, dtype))


def _weight(w, head_dim, name, dev):
    if w is None:
        return None
    if w.numel() != head_dim:
        raise ValueError("%s must be [head_dim]" % name)
    return _at(w, _th().float32, name, dev)


def _positions(plan, positions, T, dev):
    if plan is None:
        return None, None
    if positions is None or positions.numel() != T:
        raise ValueError("positions must be [T]")
    return ctypes.byref(plan), _at(positions, _th().int64, "positions", dev)


def kvq_rope(plan, q, k, positions, q_out=None, k_out=None, q_weight=None, k_weight=None, eps=1e-6,
             stream=None) -> None:
    """Per-head norm (where a weight is given) and rotation (where a plan is
    given) of query rows q [T, Hq, D] and key rows k [T, Hk, D], fp16 or bf16,
    into fp16 rows q_out and k_out (kvq_rope in include/kvq.h).  q or k may be
    None; fp16 rows without an out are turned in place."""
    half = _th().float16
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    dtype = ref.dtype
    x_type = _x_type(dtype, "q" if q is not None else "k")
    dev = _device()
    T, _, D = ref.shape

    def side(x, out, name):
        if x is None:
            return None, 0, 0, None, 0
        ptr, stride, heads = _x_rows(x, dtype, T, D, name, dev)
        if out is None:
            out = x
        optr, ostride, oheads = _x_rows(out, half, T, D, name + "_out", dev)
        if oheads != heads:
            raise ValueError("%s_out must have the shape of %s" % (name, name))
        return ptr, stride, heads, optr, ostride

    qp, qs, hq, qo, qos = side(q, q_out, "q")
    kp, ks, hk, ko, kos = side(k, k_out, "k")
    pl, pos = _positions(plan, positions, T, dev)
    _check(lib().kvq_rope(pl, x_type, qp, qs, hq, kp, ks, hk, D, pos, T,
                          _weight(q_weight, D, "q_weight", dev), _weight(k_weight, D, "k_weight", dev),
                          float(eps), qo, qos, ko, kos, _stream(stream)), "kvq_rope")


def kvq_rope_append(pool, plan, q, k, v, positions, slot_mapping, q_out=None, q_weight=None,
                    k_weight=None, eps=1e-6, stream=None) -> None:
    """kvq_rope of q (into fp16 q_out; in place if None) and k, and the append of
    the rotated k and of v to the pool, in one kernel (kvq_rope_append in
    include/kvq.h).  q may be None."""
    torch = _th()
    dtype = k.dtype
    x_type = _x_type(dtype, "k")
    dev = _device()
    shape, rows = k.shape, _pool_rows(pool)
    if v.shape != shape or len(shape) != 3 or slot_mapping.numel() != shape[0]:
        raise ValueError("k, v must be [T, kv_heads, head_dim] and slot_mapping [T]")
    T, H, D = shape
    if rows is not None and rows != (H, D):
        raise ValueError("k, v must have the pool's %d kv heads of %d channels" % rows)
    kp, ks, _ = _x_rows(k, dtype, T, D, "k", dev)
    vp, vs, _ = _x_rows(v, dtype, T, D, "v", dev)
    qp, qs, hq, qo, qos = None, 0, 0, None, 0
    if q is not None:
        qp, qs, hq = _x_rows(q, dtype, T, D, "q", dev)
        qo, qos, oheads = _x_rows(q if q_out is None else q_out, torch.float16, T, D, "q_out", dev)
        if oheads != hq:
            raise ValueError("q_out must have the shape of q")
    pl, pos = _positions(plan, positions, T, dev)
    _check(lib().kvq_rope_append(pool, pl, x_type, qp, qs, hq, kp, ks, vp, vs, pos,
                                 _at(slot_mapping, torch.int64, "slot_mapping", dev), T,
                                 _weight(q_weight, D, "q_weight", dev), _weight(k_weight, D, "k_weight", dev),
                                 float(eps), qo, qos, _stream(stream)), "kvq_rope_append")


def kvq_paged_decode_strided(pool, q, block_table, context_lens, max_context_len, sm_scale, out,
                             workspace=None, stream=None) -> None:
    """kvq_paged_decode for head slices of wider q / out rows (per-head mixed precision)."""
    torch = _th()
    qp, qs = _rows_view(q, torch.float16, "q")
    op, os_ = _rows_view(out, torch.float32, "out")
    S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_paged_decode_strided(
        pool, qp, qs, S, Hq, _ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len), float(sm_scale),
        op, os_, _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        _stream(stream)), "kvq_paged_decode_strided")


def kvq_copy_blocks(pool, src_blocks, dst_blocks, stream=None) -> None:
    """Block dst_blocks[i] becomes a copy of block src_blocks[i] (copy-on-write)."""
    torch = _th()
    if src_blocks.numel() != dst_blocks.numel():
        raise ValueError("src_blocks and dst_blocks must have the same length")
    _check(lib().kvq_copy_blocks(pool, _ptr(src_blocks, torch.int32, "src_blocks"),
                                 _ptr(dst_blocks, torch.int32, "dst_blocks"), src_blocks.numel(),
                                 _stream(stream)), "kvq_copy_blocks")


def kvq_decode_workspace_bytes(pool, num_seqs, num_q_heads, max_context_len, split_blocks=0) -> int:
    return int(lib().kvq_decode_workspace_bytes_ex(pool, num_seqs, num_q_heads, max_context_len,
                                                   split_blocks))


def kvq_paged_decode(pool, q, block_table, context_lens, max_context_len, sm_scale, out,
                     workspace=None, split_blocks=0, stream=None) -> None:
    torch = _th()
    S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_paged_decode_ex(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        float(sm_scale), _ptr(out, torch.float32, "out"),
        _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        int(split_blocks), _stream(stream)), "kvq_paged_decode")


def kvq_paged_decode_lse(pool, q, block_table, context_lens, max_context_len, sm_scale, out, lse,
                         workspace=None, split_blocks=0, stream=None) -> None:
    """kvq_paged_decode that also writes each row's log-sum-exp, lse [S, Hq] fp32
    (kvq_paged_decode_lse in include/kvq.h)."""
    torch = _th()
    S, Hq, max_blocks = _seqs(pool, q, block_table, context_lens)
    if lse.shape != (S, Hq):
        raise ValueError("lse must be [num_seqs, num_q_heads]")
    if out.numel() != q.numel():
        raise ValueError("out must have the size of q")
    dev = _device()
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_paged_decode_lse(
        pool, _at(q, torch.float16, "q", dev), S, Hq, _at(block_table, torch.int32, "block_table", dev),
        max_blocks, _at(context_lens, torch.int32, "context_lens", dev), int(max_context_len),
        float(sm_scale), _at(out, torch.float32, "out", dev), _at(lse, torch.float32, "lse", dev),
        None if workspace is None else _at(workspace, workspace.dtype, "workspace", dev), ws_bytes,
        int(split_blocks), _stream(stream)), "kvq_paged_decode_lse")


def kvq_attention_weights(pool, q, block_table, context_lens, max_context_len, sm_scale, lse, scores,
                          prev=None, decay=1.0, stream=None) -> None:
    """Attention weights of the cached tokens, summed over each kv head's Q heads and
    added to decay * prev: scores [S, Hkv, >= max_context_len] fp32
    (kvq_attention_weights in include/kvq.h).  prev may be scores itself."""
    torch = _th()
    S, Hq, max_blocks = _seqs(pool, q, block_table, context_lens)
    width = _scores_width(pool, scores, S)
    if lse.shape != (S, Hq):
        raise ValueError("lse must be [num_seqs, num_q_heads]")
    if prev is not None and prev is not scores and prev.shape != scores.shape:
        raise ValueError("prev must have the shape of scores")
    dev = _device()
    _check(lib().kvq_attention_weights(
        pool, _at(q, torch.float16, "q", dev), S, Hq, _at(block_table, torch.int32, "block_table", dev),
        max_blocks, _at(context_lens, torch.int32, "context_lens", dev), int(max_context_len),
        float(sm_scale), _at(lse, torch.float32, "lse", dev), float(decay),
        _at(prev, torch.float32, "prev", dev), _at(scores, torch.float32, "scores", dev), width,
        _stream(stream)), "kvq_attention_weights")


def kvq_evict_blocks(pool, scores, block_table, context_lens, max_context_len, budget_blocks,
                     sink_blocks, recent_blocks, table_out, lens_out, kept=None, scores_out=None,
                     stream=None) -> None:
    """Keep each sequence's heaviest budget_blocks blocks and permute its table row
    (kvq_evict_blocks in include/kvq.h): scores [S, Hkv, >= max_context_len], kept
    int32 [S, budget_blocks], scores_out [S, Hkv, >= budget_blocks * block_size].
    table_out and lens_out may be block_table and context_lens themselves."""
    torch = _th()
    S = context_lens.numel()
    width, table = _scores_width(pool, scores, S), block_table.shape
    if len(table) != 2 or table[0] != S:
        raise ValueError("block_table must be [num_seqs, blocks]")
    if (table_out is not block_table and table_out.shape != table) or lens_out.numel() != S:
        raise ValueError("table_out and lens_out must be shaped like block_table and context_lens")
    if kept is not None and kept.shape != (S, budget_blocks):
        raise ValueError("kept must be [num_seqs, budget_blocks]")
    if scores_out is not None and (scores_out.dim() != 3 or scores_out.shape[:2] != scores.shape[:2]):
        raise ValueError("scores_out must be [num_seqs, kv_heads, tokens]")
    dev = _device()
    _check(lib().kvq_evict_blocks(
        pool, _at(scores, torch.float32, "scores", dev), width, S,
        _at(block_table, torch.int32, "block_table", dev), table[1],
        _at(context_lens, torch.int32, "context_lens", dev), int(max_context_len), int(budget_blocks),
        int(sink_blocks), int(recent_blocks), _at(table_out, torch.int32, "table_out", dev),
        _at(lens_out, torch.int32, "lens_out", dev), _at(kept, torch.int32, "kept", dev),
        _at(scores_out, torch.float32, "scores_out", dev),
        0 if scores_out is None else scores_out.shape[2], _stream(stream)), "kvq_evict_blocks")


def kvq_decode_step(pool, k_new, v_new, q, block_table, context_lens, max_context_len, sm_scale,
                    out, workspace=None, stream=None) -> None:
    """Append each sequence's new token at position context_lens[s]-1, then
    decode (kvq_decode_step in include/kvq.h)."""
    torch = _th()
    S, Hq, _ = q.shape
    if k_new.shape != v_new.shape or k_new.shape[0] != S:
        raise ValueError("k_new, v_new must be [num_seqs, kv_heads, head_dim]")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_decode_step(
        pool, _ptr(k_new, torch.float16, "k_new"), _ptr(v_new, torch.float16, "v_new"),
        _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        float(sm_scale), _ptr(out, torch.float32, "out"),
        _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        _stream(stream)), "kvq_decode_step")


def kvq_cascade_workspace_bytes(pool, num_seqs, num_q_heads, max_context_len) -> int:
    return int(lib().kvq_cascade_workspace_bytes(pool, num_seqs, num_q_heads, max_context_len))


def kvq_cascade_decode(pool, q, block_table, context_lens, max_context_len, prefix_blocks,
                       sm_scale, out, workspace, stream=None) -> None:
    """Decode whose first prefix_blocks blocks (shared by every sequence) are
    attended once for all sequences (kvq_cascade_decode in include/kvq.h)."""
    torch = _th()
    S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_cascade_decode(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        int(prefix_blocks), float(sm_scale), _ptr(out, torch.float32, "out"),
        _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        _stream(stream)), "kvq_cascade_decode")


def kvq_cascade_decode_step(pool, k_new, v_new, q, block_table, context_lens, max_context_len,
                            prefix_blocks, sm_scale, out, workspace, stream=None) -> None:
    """kvq_decode_step with the shared-prefix cascade decode."""
    torch = _th()
    S, Hq, _ = q.shape
    if k_new.shape != v_new.shape or k_new.shape[0] != S:
        raise ValueError("k_new, v_new must be [num_seqs, kv_heads, head_dim]")
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_cascade_decode_step(
        pool, _ptr(k_new, torch.float16, "k_new"), _ptr(v_new, torch.float16, "v_new"),
        _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        int(prefix_blocks), float(sm_scale), _ptr(out, torch.float32, "out"),
        _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        _stream(stream)), "kvq_cascade_decode_step")


def kvq_prefill(pool, q, q_start, max_q_len, block_table, context_lens, max_context_len, sm_scale,
                out, stream=None) -> None:
    """Causal attention of each sequence's new query tokens over its cache
    (kvq_prefill in include/kvq.h).  q: [Tq, Hq, D] fp16, q_start: [S+1] int32."""
    torch = _th()
    Tq, Hq, _ = q.shape
    S = q_start.numel() - 1
    _check(lib().kvq_prefill(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(q_start, torch.int32, "q_start"),
        int(max_q_len), _ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len), float(sm_scale),
        _ptr(out, torch.float32, "out"), _stream(stream)), "kvq_prefill")


def kvq_prefill_workspace_bytes(pool, num_seqs, max_context_len) -> int:
    return int(lib().kvq_prefill_workspace_bytes(pool, int(num_seqs), int(max_context_len)))


def kvq_prefill_ex(pool, q, q_start, max_q_len, block_table, context_lens, max_context_len,
                   sm_scale, out, workspace, stream=None) -> None:
    """kvq_prefill in two passes through a caller workspace (kvq_prefill_ex in
    include/kvq.h); workspace: uint8 device tensor of at least
    kvq_prefill_workspace_bytes(...) bytes, or None when that is 0."""
    torch = _th()
    Tq, Hq, _ = q.shape
    S = q_start.numel() - 1
    ws = None if workspace is None else _ptr(workspace, torch.uint8, "workspace")
    nbytes = 0 if workspace is None else workspace.numel()
    _check(lib().kvq_prefill_ex(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(q_start, torch.int32, "q_start"),
        int(max_q_len), _ptr(block_table, torch.int32, "block_table"), block_table.shape[1],
        _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len), float(sm_scale),
        _ptr(out, torch.float32, "out"), ws, nbytes, _stream(stream)), "kvq_prefill_ex")


def kvq_selftest_decode_timeout(pool, q, block_table, context_lens, max_context_len, out,
                                workspace, wait_tries=20, stream=None) -> None:
    """Decode with one page copy withheld so that a bounded wait runs out
    (kvq_selftest_decode_timeout in include/kvq.h)."""
    torch = _th()
    S, Hq, _ = q.shape
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().kvq_selftest_decode_timeout(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        _ptr(out, torch.float32, "out"),
        _ptr(workspace, None, "workspace") if workspace is not None else None, ws_bytes,
        int(wait_tries), _stream(stream)), "kvq_selftest_decode_timeout")


KVQ_NOALLOC_SCRATCH_BYTES = 16 << 20


def kvq_paged_decode_noalloc(pool, q, block_table, context_lens, max_context_len, sm_scale, out,
                             split_blocks=0, stream=None) -> None:
    """kvq_paged_decode without a workspace argument, for callers that cannot
    allocate device memory: the split scratch is a fixed 16 MiB array inside
    the library (see kvq_paged_decode_noalloc in include/kvq.h)."""
    torch = _th()
    S, Hq, _ = q.shape
    _check(lib().kvq_paged_decode_noalloc(
        pool, _ptr(q, torch.float16, "q"), S, Hq, _ptr(block_table, torch.int32, "block_table"),
        block_table.shape[1], _ptr(context_lens, torch.int32, "context_lens"), int(max_context_len),
        float(sm_scale), _ptr(out, torch.float32, "out"), int(split_blocks), _stream(stream)),
        "kvq_paged_decode_noalloc")


def kvq_read_slots(pool, slots, codes_out, scales_out=None, stream=None) -> None:
    torch = _th()
    _check(lib().kvq_read_slots(pool, _ptr(slots, torch.int64, "slots"), slots.numel(),
                                _ptr(codes_out, None, "codes_out"),
                                _ptr(scales_out, torch.float32, "scales_out")
                                if scales_out is not None else None, _stream(stream)),
           "kvq_read_slots")


def kvq_read_values(pool, slots, k_out, v_out, stream=None) -> None:
    """Cached K and V of the slots as fp16 values, [n, kv_heads, head_dim] each
    (kvq_read_values in include/kvq.h)."""
    torch = _th()
    shape, rows, n = k_out.shape, _pool_rows(pool), slots.numel()
    if v_out.shape != shape or shape[0] != n or (rows is not None and k_out.numel() != n * rows[0] * rows[1]):
        raise ValueError("k_out, v_out must be [n, kv_heads, head_dim]")
    dev = _device()
    _check(lib().kvq_read_values(pool, _at(slots, torch.int64, "slots", dev), n,
                                 _at(k_out, torch.float16, "k_out", dev),
                                 _at(v_out, torch.float16, "v_out", dev), _stream(stream)),
           "kvq_read_values")


def kvq_get_error(pool, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the pool's device error status."""
    return int(lib().kvq_get_error(pool, _stream(stream)))


def kvq_set_phase_events(events) -> None:
    """Measurement aid: the calling thread's next len(events) kernel launches
    by the library each record one of these torch.cuda.Event objects on their
    stream right after the launch (an empty list clears them; see kvq.h)."""
    handles = []
    for ev in events:
        if not ev.cuda_event:  # torch creates the CUDA event at its first record
            ev.record()
        handles.append(ev.cuda_event)
    arr = (ctypes.c_void_p * len(handles))(*handles) if handles else None
    _check(lib().kvq_set_phase_events(arr, len(handles)), "kvq_set_phase_events")


# ------------------------------------------------------------------ convenience
class KVPool:
    """One layer's pool in caller-owned (torch) device memory.  Calls with a `stream`
    allocate what they return, and their workspaces, on that stream."""

    def __init__(self, num_blocks, block_size, kv_heads, head_dim, dtype, group=0, device="cuda",
                 fill_byte: int | None = None):
        torch = _th()
        self.num_blocks, self.block_size, self.kv_heads, self.head_dim = (
            num_blocks, block_size, kv_heads, head_dim)
        self.dtype, self.group = dtype, (group if dtype in GROUP_FORMATS else 0)
        nbytes = kvq_pool_bytes(num_blocks, block_size, kv_heads, head_dim, dtype, self.group)
        if nbytes == 0:
            kvq_pool_layout_query(num_blocks, block_size, kv_heads, head_dim, dtype, self.group)
            raise KVQError(KVQ_ERR_INVALID_ARG, "KVPool")
        self.buffer = torch.empty(nbytes, dtype=torch.uint8, device=device)
        if fill_byte is not None:
            self.buffer.fill_(fill_byte)
        self.handle = kvq_alloc_pool(num_blocks, block_size, kv_heads, head_dim, dtype, self.group,
                                     self.buffer)

    def close(self):
        if getattr(self, "handle", None) is not None:
            kvq_free_pool(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def append(self, k, v, slot_mapping, stream=None):
        kvq_append(self.handle, k, v, slot_mapping, stream)

    def rope_append(self, plan, q, k, v, positions, slot_mapping, q_out=None, q_weight=None,
                    k_weight=None, eps=1e-6, stream=None):
        """Rotated (and normed) fp16 queries; keys and values go to the pool."""
        torch = _th()
        if q is not None and q_out is None:
            with _on(stream):
                q_out = torch.empty(q.shape, dtype=torch.float16, device=q.device)
        kvq_rope_append(self.handle, plan, q, k, v, positions, slot_mapping, q_out, q_weight,
                        k_weight, eps, stream)
        return q_out

    def decode(self, q, block_table, context_lens, max_context_len, sm_scale=None, out=None,
               split_blocks=0, stream=None):
        torch = _th()
        S, Hq, D = q.shape
        if sm_scale is None:
            sm_scale = D ** -0.5
        nws = kvq_decode_workspace_bytes(self.handle, S, Hq, max_context_len, split_blocks)
        with _on(stream):
            if out is None:
                out = torch.empty((S, Hq, D), dtype=torch.float32, device=q.device)
            ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=q.device) if nws else None
        kvq_paged_decode(self.handle, q, block_table, context_lens, max_context_len, sm_scale, out,
                         ws, split_blocks, stream)
        return out

    def decode_step(self, k_new, v_new, q, block_table, context_lens, max_context_len,
                    sm_scale=None, out=None, stream=None):
        torch = _th()
        S, Hq, D = q.shape
        if sm_scale is None:
            sm_scale = D ** -0.5
        nws = kvq_decode_workspace_bytes(self.handle, S, Hq, max_context_len)
        with _on(stream):
            if out is None:
                out = torch.empty((S, Hq, D), dtype=torch.float32, device=q.device)
            ws = torch.empty(max(nws, 1), dtype=torch.uint8, device=q.device) if nws else None
        kvq_decode_step(self.handle, k_new, v_new, q, block_table, context_lens, max_context_len,
                        sm_scale, out, ws, stream)
        return out

    def decode_lse(self, q, block_table, context_lens, max_context_len, sm_scale=None, stream=None):
        """decode's output and each row's log-sum-exp [S, Hq]."""
        torch = _th()
        S, Hq, D = q.shape
        nws = kvq_decode_workspace_bytes(self.handle, S, Hq, max_context_len)
        with _on(stream):
            out = torch.empty((S, Hq, D), dtype=torch.float32, device=q.device)
            lse = torch.empty((S, Hq), dtype=torch.float32, device=q.device)
            ws = torch.empty(nws, dtype=torch.uint8, device=q.device) if nws else None
        kvq_paged_decode_lse(self.handle, q, block_table, context_lens, max_context_len,
                             D ** -0.5 if sm_scale is None else sm_scale, out, lse, ws, 0, stream)
        return out, lse

    def accumulate_weights(self, q, block_table, context_lens, max_context_len, lse, scores,
                           decay=1.0, sm_scale=None, stream=None):
        """scores = decay * scores + this step's attention weights, in place."""
        kvq_attention_weights(self.handle, q, block_table, context_lens, max_context_len,
                              q.shape[2] ** -0.5 if sm_scale is None else sm_scale, lse, scores,
                              scores, decay, stream)
        return scores

    def evict_blocks(self, scores, block_table, context_lens, max_context_len, budget_blocks,
                     sink_blocks=0, recent_blocks=1, stream=None):
        """(table, lens, kept, scores) after the eviction, in new tensors."""
        torch = _th()
        S = context_lens.numel()
        with _on(stream):
            table, lens = torch.empty_like(block_table), torch.empty_like(context_lens)
            kept = torch.empty((S, budget_blocks), dtype=torch.int32, device=scores.device)
            out = torch.zeros((S, self.kv_heads, max(budget_blocks * self.block_size, scores.shape[2])),
                              dtype=torch.float32, device=scores.device)
        kvq_evict_blocks(self.handle, scores, block_table, context_lens, max_context_len,
                         budget_blocks, sink_blocks, recent_blocks, table, lens, kept, out, stream)
        return table, lens, kept, out

    def cascade_decode(self, q, block_table, context_lens, max_context_len, prefix_blocks,
                       sm_scale=None, out=None, stream=None):
        torch = _th()
        S, Hq, D = q.shape
        if sm_scale is None:
            sm_scale = D ** -0.5
        nws = kvq_cascade_workspace_bytes(self.handle, S, Hq, max_context_len)
        with _on(stream):
            if out is None:
                out = torch.empty((S, Hq, D), dtype=torch.float32, device=q.device)
            ws = torch.empty(max(nws, 256), dtype=torch.uint8, device=q.device)
        kvq_cascade_decode(self.handle, q, block_table, context_lens, max_context_len,
                           prefix_blocks, sm_scale, out, ws, stream)
        return out

    def read_slots(self, slots, stream=None):
        torch = _th()
        n = slots.numel()
        cdt = torch.float16 if self.dtype == KVQ_FP16 else (
            torch.uint8 if self.dtype in (KVQ_FP8_E4M3_PER_TOKEN, KVQ_FP8_E5M2,
                                          KVQ_FP8_E4M3_PER_BLOCK) else torch.int8)
        with _on(stream):
            codes = torch.empty((n, 2, self.kv_heads, self.head_dim), dtype=cdt, device=slots.device)
            scales = None
            if self.dtype in GROUP_FORMATS:
                scales = torch.empty((n, 2, self.kv_heads, self.head_dim // self.group),
                                     dtype=torch.float32, device=slots.device)
            elif self.dtype in (KVQ_INT8_PER_TOKEN, KVQ_FP8_E4M3_PER_TOKEN):
                scales = torch.empty((n, 2), dtype=torch.float32, device=slots.device)
            elif self.dtype in BLOCK_FORMATS:
                scales = torch.empty((n, 2, self.kv_heads), dtype=torch.float32, device=slots.device)
        kvq_read_slots(self.handle, slots, codes, scales, stream)
        return codes, scales

    def read_values(self, slots, stream=None):
        """fp16 K and V [n, kv_heads, head_dim] of the slots; zeros for negative ones and
        for slots outside the pool."""
        torch = _th()
        with _on(stream):
            k = torch.zeros((slots.numel(), self.kv_heads, self.head_dim), dtype=torch.float16,
                            device=slots.device)
            v = torch.zeros_like(k)
        kvq_read_values(self.handle, slots, k, v, stream)
        return k, v

    def error(self, stream=None) -> int:
        return kvq_get_error(self.handle, stream)
