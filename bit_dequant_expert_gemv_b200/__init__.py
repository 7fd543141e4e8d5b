"""B200 (sm_100a) batch-1 MoE layer with 4-bit / 2-bit group-affine dequantising expert GEMVs,
and the token mixers before it: the gated delta rule, a paged 4-bit cache, attention over it.

Thin binding over the C ABI of ``libfmoe.so`` (``include/fmoe.h``): argument marshalling
only. Every step of the computation runs in the library's CUDA kernels; PyTorch only supplies
device memory and streams. There is no CPU fallback: importing the package fails loudly when
the compiled library is missing.
"""
from __future__ import annotations

import ctypes as C
import os

from ._build import LIB, build, stale  # noqa: F401

FMOE_OK, FMOE_ERR_INVALID, FMOE_ERR_ALIGN, FMOE_ERR_CUDA, FMOE_ERR_NOMEM, FMOE_ERR_TIMEOUT, \
    FMOE_ERR_UNSUPPORTED, FMOE_ERR_INDEX = 0, -1, -2, -3, -4, -5, -6, -7
FMOE_F32, FMOE_BF16, FMOE_F16 = 0, 1, 2


class FmoeError(RuntimeError):
    def __init__(self, fn: str, code: int, msg: str):
        super().__init__(f"{fn} failed with status {code}: {msg}")
        self.code = code


class View(C.Structure):
    """Mirror of fmoe_view and fmoe_out_view."""
    _fields_ = [("ptr", C.c_void_p), ("token_stride", C.c_int64), ("head_stride", C.c_int64)]


# The descriptors below hold their views field by field: the memory is that of a nested structure,
# and one call fills it.
def _view(name):
    return [(name, C.c_void_p), (name + "_token_stride", C.c_int64), (name + "_head_stride", C.c_int64)]


class DeltaDesc(C.Structure):
    """Mirror of fmoe_delta_desc."""
    _fields_ = [("heads_k", C.c_int), ("heads_v", C.c_int), ("dim_k", C.c_int), ("dim_v", C.c_int),
                ("dtype", C.c_int), ("l2norm", C.c_int), ("eps", C.c_float), ("scale", C.c_float),
                *_view("q"), *_view("k"), *_view("v"), ("g", C.c_void_p), ("beta", C.c_void_p),
                ("gate_stride", C.c_int64), ("state", C.c_void_p), ("state_stride", C.c_int64),
                ("n_slots", C.c_int), ("slots", C.c_void_p), *_view("out")]


class KvCacheDesc(C.Structure):
    """Mirror of fmoe_kv_cache."""
    _fields_ = [("pages", C.c_void_p), ("n_pages", C.c_int), ("heads", C.c_int), ("dim", C.c_int),
                ("page_size", C.c_int), ("page_table", C.c_void_p), ("table_stride", C.c_int64),
                ("n_seqs", C.c_int), ("max_pages", C.c_int)]


class KvTokens(C.Structure):
    """Mirror of fmoe_kv_tokens."""
    _fields_ = [("dtype", C.c_int), ("n_tokens", C.c_int), *_view("k"), *_view("v"),
                ("positions", C.c_void_p), ("seq", C.c_void_p), ("inv_freq", C.c_void_p),
                ("n_freq", C.c_int), ("interleaved", C.c_int), ("heads_q", C.c_int), *_view("q"),
                *_view("q_out")]


class AttnDesc(C.Structure):
    """Mirror of fmoe_attn_desc."""
    _fields_ = [("heads_q", C.c_int), ("dtype", C.c_int), ("n_tokens", C.c_int), ("max_q", C.c_int),
                ("max_len", C.c_int), ("scale", C.c_float), *_view("q"), ("cu_q", C.c_void_p),
                ("lens", C.c_void_p), *_view("out")]


_SIGS = {
    "fmoe_last_error": (C.c_char_p, []),
    "fmoe_version": (C.c_int, []),
    "fmoe_sync_status": (C.c_int, [C.c_void_p]),
    "fmoe_set_wait_budget_ns": (None, [C.c_uint64]),
    "fmoe_set_fault_injection": (None, [C.c_int]),
    "fmoe_qmat_bytes": (C.c_size_t, [C.c_int] * 3),
    "fmoe_expert_bytes": (C.c_size_t, [C.c_int] * 3),
    "fmoe_pack": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "fmoe_pack_q4": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "fmoe_pack_q2": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_void_p, C.c_void_p]),
    "fmoe_route": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int, C.c_int, C.c_int,
                             C.c_void_p, C.c_void_p, C.c_void_p]),
    "fmoe_expert_gemv": (C.c_int, [C.c_void_p, C.c_int, C.c_int, C.c_int, C.c_void_p,
                                   C.c_void_p, C.c_void_p]),
    "fmoe_moe_layer": (C.c_int, [C.c_void_p] * 8),
    "fmoe_moe_layer_noalloc": (C.c_int, [C.c_void_p] * 8),
    "fmoe_moe_layer_seq": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_int,
                                     C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "fmoe_moe_layer_seq_host": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_void_p, C.c_int,
                                          C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p,
                                          C.c_void_p]),
    "fmoe_moe_stack": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p, C.c_float,
                                 C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "fmoe_stack_graph_create": (C.c_int, [C.c_void_p, C.c_int, C.c_void_p, C.c_int, C.c_void_p,
                                          C.c_float, C.c_void_p, C.c_void_p, C.c_void_p, C.c_int,
                                          C.c_void_p]),
    "fmoe_stack_graph_launch": (C.c_int, [C.c_void_p, C.c_void_p]),
    "fmoe_stack_graph_destroy": (C.c_int, [C.c_void_p]),
    "fmoe_describe_geometry": (C.c_int, [C.c_int] * 8 + [C.c_void_p, C.c_int]),
    "fmoe_set_dot_form": (C.c_int, [C.c_int]),
    "fmoe_launch_count": (C.c_uint64, []),
    "fmoe_delta_step": (C.c_int, [C.POINTER(DeltaDesc), C.c_int, C.c_void_p]),
    "fmoe_delta_chunk": (C.c_int, [C.POINTER(DeltaDesc), C.c_void_p, C.c_int, C.c_int, C.c_int,
                                   C.c_void_p, C.c_void_p]),
    "fmoe_kv_block_bytes": (C.c_size_t, [C.c_int, C.c_int]),
    "fmoe_kv_append": (C.c_int, [C.POINTER(KvCacheDesc), C.POINTER(KvTokens), C.c_void_p]),
    "fmoe_kv_read": (C.c_int, [C.POINTER(KvCacheDesc), C.c_void_p, C.c_void_p, C.c_int, C.c_int,
                               View, View, C.c_void_p]),
    "fmoe_attn_q4": (C.c_int, [C.POINTER(KvCacheDesc), C.POINTER(AttnDesc), C.c_void_p]),
}
_lib = None


def lib():
    """The loaded libfmoe.so; raises ImportError when it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise ImportError(f"libfmoe.so is not built ({LIB}); run __graft_entry__.build() "
                              "or python -m bit_dequant_expert_gemv_b200._build")
        L = C.CDLL(LIB)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def last_error() -> str:
    return lib().fmoe_last_error().decode()


def _ck(name: str, rc: int):
    if rc != FMOE_OK:
        raise FmoeError(name, rc, last_error())


def _ptr(t):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    if stream is None:
        return C.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return C.c_void_p(stream)
    return C.c_void_p(stream.cuda_stream)


class LayerDesc(C.Structure):
    """Mirror of fmoe_layer_desc; keeps the tensors it points to alive."""
    _fields_ = [("hidden", C.c_int), ("inter", C.c_int), ("n_experts", C.c_int),
                ("top_k", C.c_int), ("bits", C.c_int), ("experts", C.c_void_p),
                ("expert_stride", C.c_size_t), ("shared_expert", C.c_void_p),
                ("router", C.c_void_p), ("shared_gate", C.c_void_p)]

    def __init__(self, hidden, inter, n_experts, top_k, bits, experts, expert_stride, shared,
                 router, shared_gate):
        super().__init__(hidden, inter, n_experts, top_k, bits, experts.data_ptr(), expert_stride,
                         None if shared is None else shared.data_ptr(), router.data_ptr(),
                         None if shared_gate is None else shared_gate.data_ptr())
        self._keep = (experts, shared, router, shared_gate)


def _descs(layers):
    if isinstance(layers, LayerDesc):
        layers = [layers]
    arr = (LayerDesc * len(layers))()
    for i, d in enumerate(layers):
        C.memmove(C.addressof(arr[i]), C.addressof(d), C.sizeof(LayerDesc))
    return arr, len(layers)


# --------------------------------------------------------------------------------- sizes
def qmat_bytes(rows: int, cols: int, bits: int) -> int:
    return int(lib().fmoe_qmat_bytes(rows, cols, bits))


def expert_bytes(hidden: int, inter: int, bits: int) -> int:
    return int(lib().fmoe_expert_bytes(hidden, inter, bits))


GEOMETRY_FIELDS = ("H I E K bits route_on shared_on routed_on gate_on rc_h rs_h rc_i rs_i q_gu nr "
                   "rseg rcols rrows au hr ad dr nseg sh wh gh si wi pi ji stage_bytes nA nB "
                   "o_ringA o_ringB o_x o_h o_red o_oacc o_misc o_bar oacc_n smem_bytes "
                   "consumer_warps max_rows_thread max_rows_warp red_slot gpass").split()


def describe_geometry(H, I, E, K, bits, flags=15, max_smem=232448, sms=148) -> dict:
    buf = (C.c_int64 * len(GEOMETRY_FIELDS))()
    n = lib().fmoe_describe_geometry(H, I, E, K, bits, flags, max_smem, sms, buf,
                                     len(GEOMETRY_FIELDS))
    if n < 0:
        raise FmoeError("fmoe_describe_geometry", n, last_error())
    return {k: int(buf[i]) for i, k in enumerate(GEOMETRY_FIELDS[:n])}


def set_dot_form(form: int):
    """0: digit planes + dp4a (default), 1: literal fma(q, s*x, z*x), 2: naive (q*s + z)*x."""
    _ck("fmoe_set_dot_form", lib().fmoe_set_dot_form(int(form)))


def launch_count() -> int:
    return int(lib().fmoe_launch_count())


def set_wait_budget_ns(ns: int):
    lib().fmoe_set_wait_budget_ns(int(ns))


def set_fault_injection(flags: int):
    lib().fmoe_set_fault_injection(int(flags))


def sync_status(stream=None) -> int:
    """Synchronise `stream`, return (and clear) the sticky device status (0 = OK)."""
    return int(lib().fmoe_sync_status(_stream(stream)))


# --------------------------------------------------------------------------------- entry points
def pack(w, bits: int, out=None, stream=None):
    import torch
    assert w.is_cuda and w.dtype == torch.float32 and w.is_contiguous() and w.dim() == 2
    rows, cols = w.shape
    if out is None:
        out = torch.empty(qmat_bytes(rows, cols, bits), dtype=torch.uint8, device=w.device)
    _ck("fmoe_pack", lib().fmoe_pack(_ptr(w), rows, cols, bits, _ptr(out), _stream(stream)))
    return out


def route(x, router, bias, top_k: int, idx=None, weight=None, stream=None):
    import torch
    E, H = router.shape
    idx = torch.empty(top_k, dtype=torch.int32, device=x.device) if idx is None else idx
    weight = torch.empty(top_k, dtype=torch.float32, device=x.device) if weight is None else weight
    _ck("fmoe_route", lib().fmoe_route(_ptr(x), _ptr(router), _ptr(bias), H, E, top_k, _ptr(idx),
                                      _ptr(weight), _stream(stream)))
    return idx, weight


def expert_gemv(blob, hidden: int, inter: int, bits: int, x, y=None, stream=None):
    import torch
    y = torch.empty(hidden, dtype=torch.float32, device=x.device) if y is None else y
    _ck("fmoe_expert_gemv", lib().fmoe_expert_gemv(_ptr(blob), hidden, inter, bits, _ptr(x), _ptr(y),
                                                  _stream(stream)))
    return y


def moe_layer(desc: LayerDesc, x, residual=None, bias=None, out=None, idx=None, weight=None,
              stream=None):
    import torch
    out = torch.empty_like(x) if out is None else out
    arr, _ = _descs(desc)
    _ck("fmoe_moe_layer", lib().fmoe_moe_layer(arr, _ptr(x), _ptr(residual), _ptr(bias), _ptr(out),
                                              _ptr(idx), _ptr(weight), _stream(stream)))
    return out


def moe_layer_noalloc(desc: LayerDesc, x, residual=None, bias=None, out=None, idx=None,
                      weight=None, stream=None):
    """fmoe_moe_layer_noalloc: one token with the library's fixed scratch array (no device
    allocation inside the call; `out` must be given by callers that allocate nothing)."""
    import torch
    out = torch.empty_like(x) if out is None else out
    arr, _ = _descs(desc)
    _ck("fmoe_moe_layer_noalloc",
        lib().fmoe_moe_layer_noalloc(arr, _ptr(x), _ptr(residual), _ptr(bias), _ptr(out),
                                     _ptr(idx), _ptr(weight), _stream(stream)))
    return out


NOALLOC_SCRATCH_BYTES = 128 * 1024


def moe_layer_seq(descs, x, residual=None, bias=None, out=None, idx=None, weight=None,
                  stream=None):
    import torch
    T = x.shape[0]
    out = torch.empty_like(x) if out is None else out
    arr, n = _descs(descs)
    _ck("fmoe_moe_layer_seq", lib().fmoe_moe_layer_seq(arr, n, _ptr(x), _ptr(residual), T,
                                                      _ptr(bias), _ptr(out), _ptr(idx),
                                                      _ptr(weight), _stream(stream)))
    return out


def moe_layer_seq_host(descs, x, residual, bias, out, idx=None, weight=None, stream=None):
    """Host-buffer variant (pinned torch CPU tensors): copies in, runs, copies out on `stream`."""
    arr, n = _descs(descs)
    _ck("fmoe_moe_layer_seq_host", lib().fmoe_moe_layer_seq_host(
        arr, n, _ptr(x), _ptr(residual), x.shape[0], _ptr(bias), _ptr(out), _ptr(idx), _ptr(weight),
        _stream(stream)))
    return out


def moe_stack(descs, h_in, bias=None, eps: float = 1e-6, h_out=None, idx_trace=None,
              h_trace=None, stream=None):
    import torch
    T = h_in.shape[0]
    h_out = torch.empty_like(h_in) if h_out is None else h_out
    arr, n = _descs(descs)
    _ck("fmoe_moe_stack", lib().fmoe_moe_stack(arr, n, _ptr(h_in), T, _ptr(bias), eps, _ptr(h_out),
                                              _ptr(idx_trace), _ptr(h_trace), _stream(stream)))
    return h_out


class StackGraph:
    """fmoe_moe_stack captured once into a CUDA graph (fixed buffers), replayed by launch()."""

    def __init__(self, descs, h_in, h_out, bias=None, eps: float = 1e-6, idx_trace=None,
                 h_trace=None, tokens_per_launch: int = 0):
        arr, n = _descs(descs)
        self._keep = (descs, h_in, h_out, bias, idx_trace, h_trace)
        self._g = C.c_void_p()
        _ck("fmoe_stack_graph_create", lib().fmoe_stack_graph_create(
            arr, n, _ptr(h_in), h_in.shape[0], _ptr(bias), eps, _ptr(h_out), _ptr(idx_trace),
            _ptr(h_trace), tokens_per_launch, C.byref(self._g)))

    def launch(self, stream=None):
        _ck("fmoe_stack_graph_launch", lib().fmoe_stack_graph_launch(self._g, _stream(stream)))

    def close(self):
        if self._g:
            lib().fmoe_stack_graph_destroy(self._g)
            self._g = C.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------------------------- token mixers
# These calls are short next to what they launch; their checks are written to cost little.
_DTYPES = {}


def _dtype(t):
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.float32: FMOE_F32, torch.bfloat16: FMOE_BF16, torch.float16: FMOE_F16})
    code = _DTYPES.get(t)
    if code is None:
        raise TypeError(f"element type {t} is not float32, bfloat16 or float16")
    return code


def _rows(t, dtype, dev, name, shape=None):
    """A [tokens, heads, dim] tensor as (pointer, token stride, head stride): contiguous columns, any strides."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 3:
        raise TypeError(f"{name} must be a [tokens, heads, dim] tensor of {dtype} on CUDA device {dev}")
    n, h, _ = got = t.shape
    if shape is not None and got != shape:
        raise ValueError(f"{name} has shape {tuple(got)}, expected {tuple(shape)}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise ValueError(f"the columns of {name} must be contiguous")
    return t.data_ptr(), st if n > 1 else 0, sh if h > 1 else 0


def _array(t, dtype, dev, name, n):
    """The pointer of a contiguous array of n elements (None stays None)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on CUDA device {dev}")
    return t.data_ptr()


def _device(t):
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on a CUDA device")
    return dev


def _empty(like, shape, dtype, stream):
    """Memory for a result that `stream` writes, on the device of `like`. Free memory of the current stream may still be
    written by what that stream has yet to run: another stream's result is allocated on that one, and outlives the
    current one's use of it."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=like.device)
    with torch.cuda.stream(stream):
        out = torch.empty(shape, dtype=dtype, device=like.device)
    out.record_stream(torch.cuda.current_stream(like.device))
    return out


def _call(fn, dev, stream, *args):
    """fn(*args, stream) with the tensors' device current; the stream is that device's current one by default."""
    import torch
    code = getattr(lib(), fn)
    if torch._C._cuda_getDevice() != dev:
        with torch.cuda.device(dev):
            return _call(fn, dev, stream, *args)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    rc = code(*args, stream)
    if rc:
        _ck(fn, rc)


def _delta(dev, q, k, v, g, beta, state, n, slots, scale, l2norm, eps, out, stream):
    import torch
    dt = v.dtype
    code = _dtype(dt)
    vv = _rows(v, dt, dev, "v")
    tokens, heads_v, dim_v = shape = v.shape
    kv = _rows(k, dt, dev, "k")
    tk, heads_k, dim_k = k.shape
    if tk != tokens:
        raise ValueError("k and v have different numbers of tokens")
    qv = _rows(q, dt, dev, "q", k.shape)
    f32 = torch.float32
    gs, bs = g.stride(), beta.stride()
    if g.dtype is not f32 or beta.dtype is not f32 or g.get_device() != dev or beta.get_device() != dev \
            or g.shape != (tokens, heads_v) or beta.shape != g.shape \
            or (heads_v > 1 and (gs[1] != 1 or bs[1] != 1)) or (tokens > 1 and gs[0] != bs[0]):
        raise ValueError("g and beta must be float32 [tokens, heads] tensors with the same strides")
    n_slots, *rest = state.shape
    ss = state.stride()
    if state.dtype is not f32 or state.get_device() != dev or rest != [heads_v, dim_k, dim_v] \
            or ss[2:] != (dim_v, 1) or (heads_v > 1 and ss[1] != dim_k * dim_v):
        raise ValueError("state must be float32 [slots, heads, dim_k, dim_v], contiguous within a slot")
    sp = _array(slots, torch.int32, dev, "slots", n)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=v.device) if stream is None else _empty(v, shape, dt, stream)
    ov = _rows(out, dt, dev, "out", shape)
    return out, DeltaDesc(heads_k, heads_v, dim_k, dim_v, code, l2norm, eps,
                          dim_k ** -0.5 if scale is None else scale, *qv, *kv, *vv, g.data_ptr(),
                          beta.data_ptr(), gs[0], state.data_ptr(),
                          ss[0] if n_slots > 1 else heads_v * dim_k * dim_v, n_slots, sp, *ov)


def delta_step(q, k, v, g, beta, state, slots=None, scale=None, l2norm: bool = True,
               eps: float = 1e-6, out=None, stream=None):
    """One token of every sequence through the gated delta rule; `state` is updated in place."""
    dev, n = _device(v), v.shape[0]
    out, d = _delta(dev, q, k, v, g, beta, state, n, slots, scale, l2norm, eps, out, stream)
    _call("fmoe_delta_step", dev, stream, d, n)
    return out


def delta_chunk(q, k, v, g, beta, state, cu_seqlens, max_len: int, slots=None, fresh=None,
                scale=None, l2norm: bool = True, eps: float = 1e-6, out=None, stream=None):
    """Packed sequences (prompts) through the gated delta rule; `state` is updated in place."""
    import torch
    dev, n = _device(v), cu_seqlens.numel() - 1
    out, d = _delta(dev, q, k, v, g, beta, state, n, slots, scale, l2norm, eps, out, stream)
    cu = _array(cu_seqlens, torch.int32, dev, "cu_seqlens", n + 1)
    if fresh is not None and fresh.dtype is torch.bool:
        fresh = fresh.view(torch.uint8)
    fr = _array(fresh, torch.uint8, dev, "fresh", n)
    _call("fmoe_delta_chunk", dev, stream, d, cu, n, v.shape[0], max_len, fr)
    return out


def kv_block_bytes(page_size: int, dim: int) -> int:
    return int(lib().fmoe_kv_block_bytes(page_size, dim))


def kv_pages(n_pages: int, heads: int, dim: int, page_size: int, device="cuda"):
    """Zeroed pages of a 4-bit cache: [n_pages, heads, block bytes]."""
    import torch
    block = kv_block_bytes(page_size, dim)
    if block == 0:
        raise ValueError(f"no 4-bit cache of page size {page_size} and dim {dim}")
    return torch.zeros(n_pages, heads, block, dtype=torch.uint8, device=device)


def _cache(dev, pages, table, dim):
    import torch
    if pages.dtype is not torch.uint8 or pages.get_device() != dev or pages.dim() != 3 or not pages.is_contiguous():
        raise ValueError(f"pages must be a contiguous uint8 [pages, heads, block bytes] tensor on CUDA device {dev}")
    if table.dtype is not torch.int32 or table.get_device() != dev or table.dim() != 2 \
            or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError(f"the page table must be an int32 [sequences, pages] tensor on CUDA device {dev}")
    n_pages, heads, block = pages.shape
    ps, rest = divmod(block, dim + dim // 8)
    if rest:
        raise ValueError(f"blocks of {block} bytes hold no whole rows of dim {dim}")
    n, most = table.shape
    return KvCacheDesc(pages.data_ptr(), n_pages, heads, dim, ps, table.data_ptr(), table.stride(0), n, most)


def kv_append(k, v, positions, pages, page_table, inv_freq, seq=None, q=None, q_out=None,
              interleaved: bool = False, stream=None):
    """Rotates and quantises k, quantises v, writes both into the pages; returns the rotated q
    (None without q)."""
    import torch
    dev, dt = _device(k), k.dtype
    code = _dtype(dt)
    kv = _rows(k, dt, dev, "k")
    tokens, heads, dim = shape = k.shape
    c = _cache(dev, pages, page_table, dim)
    if heads != c.heads:
        raise ValueError(f"k has {heads} heads, the pages {c.heads}")
    vv = _rows(v, dt, dev, "v", shape)
    n_freq = inv_freq.numel()
    pp = _array(positions, torch.int32, dev, "positions", tokens)
    sp = _array(seq, torch.int32, dev, "seq", tokens)
    if seq is None and tokens > c.n_seqs:
        raise ValueError(f"{tokens} tokens for {c.n_seqs} sequences without seq")
    fp = _array(inv_freq, torch.float32, dev, "inv_freq", n_freq)
    heads_q, qv, ov = 0, (None, 0, 0), (None, 0, 0)
    if q is not None:
        qv = _rows(q, dt, dev, "q")
        heads_q, q_shape = q.shape[1], q.shape
        if q_shape != (tokens, heads_q, dim):
            raise ValueError(f"q has shape {tuple(q_shape)}, expected ({tokens}, heads, {dim})")
        if q_out is None:
            q_out = torch.empty(q_shape, dtype=dt, device=k.device) if stream is None else _empty(k, q_shape, dt, stream)
        ov = _rows(q_out, dt, dev, "q_out", q_shape)
    a = KvTokens(code, tokens, *kv, *vv, pp, sp, fp, n_freq, interleaved, heads_q, *qv, *ov)
    _call("fmoe_kv_append", dev, stream, c, a)
    return q_out


def kv_read(pages, page_table, positions, dim: int, seq=None, dtype=None, k=None, v=None, stream=None):
    """The keys and values held at positions[t] of sequence seq[t] (default t): two [tokens, heads,
    dim] tensors of `dtype` (default bfloat16)."""
    import torch
    dev = _device(pages)
    c = _cache(dev, pages, page_table, dim)
    tokens = positions.numel()
    shape = (tokens, c.heads, dim)
    dt = dtype if dtype is not None else torch.bfloat16 if k is None else k.dtype
    if k is None:
        k = torch.empty(shape, dtype=dt, device=pages.device) if stream is None else _empty(pages, shape, dt, stream)
    if v is None:
        v = torch.empty(shape, dtype=dt, device=pages.device) if stream is None else _empty(pages, shape, dt, stream)
    pp = _array(positions, torch.int32, dev, "positions", tokens)
    sp = _array(seq, torch.int32, dev, "seq", tokens)
    _call("fmoe_kv_read", dev, stream, c, pp, sp, tokens, _dtype(dt), View(*_rows(k, dt, dev, "k", shape)),
          View(*_rows(v, dt, dev, "v", shape)))
    return k, v


def attn_q4(q, pages, page_table, lens, max_len: int, cu_q=None, max_q: int = 1, scale=None, out=None,
            stream=None):
    """Attention of the last positions of every sequence (one query each, or cu_q's) over the 4-bit
    cache; q and the result are [tokens, heads, dim]."""
    import torch
    dev, dt = _device(q), q.dtype
    code = _dtype(dt)
    qv = _rows(q, dt, dev, "q")
    tokens, heads, dim = shape = q.shape
    c = _cache(dev, pages, page_table, dim)
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device) if stream is None else _empty(q, shape, dt, stream)
    ov = _rows(out, dt, dev, "out", shape)
    lp = _array(lens, torch.int32, dev, "lens", c.n_seqs)
    cp = _array(cu_q, torch.int32, dev, "cu_q", c.n_seqs + 1)
    a = AttnDesc(heads, code, tokens, max_q, max_len, dim ** -0.5 if scale is None else scale, *qv, cp, lp, *ov)
    _call("fmoe_attn_q4", dev, stream, c, a)
    return out
