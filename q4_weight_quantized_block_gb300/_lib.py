"""ctypes binding over libfak.so: argument marshalling only (see include/fak.h)."""
import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfak.so")

if not os.path.exists(LIB_PATH):
    raise ImportError("libfak.so not built: run q4_weight_quantized_block_gb300.build.build() "
                      "(nvcc, sm_103a); there is no fallback implementation")

lib = ctypes.CDLL(LIB_PATH)

STATUS = {0: "FAK_OK", 1: "FAK_ERR_INVALID_ARG", 2: "FAK_ERR_SHAPE", 3: "FAK_ERR_ALIGN", 4: "FAK_ERR_CUDA",
          5: "FAK_ERR_TIMEOUT", 6: "FAK_ERR_NOMEM", 7: "FAK_ERR_DEVICE", 8: "FAK_ERR_UNSUPPORTED"}
FAK_ENGINE_MAX_K = 18432
FAK_MLP_NOALLOC_MAX_FF = 18432
FAK_LAYER_GDN, FAK_LAYER_FA = 0, 1
FAK_DECODE_ONE_LAUNCH, FAK_DECODE_PER_MATMUL, FAK_DECODE_ONE_LAUNCH_I8X, FAK_DECODE_PER_MATMUL_I8X = 0, 1, 2, 3
FAK_DECODE_PER_MATMUL_HOST_WAIT = 4
FAK_KV_BF16, FAK_KV_E4M3, FAK_KV_I8 = 0, 1, 2
FAK_ROWS_F32, FAK_ROWS_BF16 = 0, 1

P, I64, I32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t


class FakError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__("%s: %s (%s)" % (where, STATUS.get(status, status), fak_strerror(status)))


class LayerDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("w_in", P), ("w_k", P), ("w_v", P), ("w_out", P), ("w_gate", P),
                ("w_up", P), ("w_down", P)]


class MixerLayer(ctypes.Structure):
    _fields_ = [("conv_w", P), ("a_log", P), ("dt_bias", P), ("norm_w", P), ("q_norm_w", P), ("k_norm_w", P)]


class MixerDesc(ctypes.Structure):
    _fields_ = [("gdn_nk", ctypes.c_int32), ("gdn_nv", ctypes.c_int32), ("gdn_dk", ctypes.c_int32),
                ("gdn_dv", ctypes.c_int32), ("fa_nq", ctypes.c_int32), ("fa_nkv", ctypes.c_int32),
                ("fa_dh", ctypes.c_int32), ("fa_rot", ctypes.c_int32), ("rope_theta", ctypes.c_float),
                ("eps", ctypes.c_float), ("max_ctx", ctypes.c_int32), ("layers", ctypes.POINTER(MixerLayer))]


class DecodeDesc(ctypes.Structure):
    _fields_ = [("n_layers", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("vocab", ctypes.c_int32), ("gdn_in", ctypes.c_int32), ("fa_qg", ctypes.c_int32),
                ("fa_kv", ctypes.c_int32), ("n_mix", ctypes.c_int32), ("eps", ctypes.c_float),
                ("mode", ctypes.c_int32), ("layers", ctypes.POINTER(LayerDesc)), ("lm_head", P),
                ("embedding", P), ("mixer", ctypes.POINTER(MixerDesc))]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_kv", ctypes.c_int32), ("dh", ctypes.c_int32), ("page", ctypes.c_int32),
                ("n_pages", I64), ("k", P), ("v", P), ("k_scale", P), ("v_scale", P)]


class KvBatchDesc(ctypes.Structure):
    _fields_ = [("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("page_table", P), ("row_start", P),
                ("kv_len", P)]


class KvRows(ctypes.Structure):
    _fields_ = [("type", ctypes.c_int32), ("nq", ctypes.c_int32), ("rot", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rows", I64), ("q", P), ("k", P), ("v", P), ("q_row", I64), ("q_head", I64), ("k_row", I64),
                ("k_head", I64), ("v_row", I64), ("v_head", I64), ("q_norm_w", P), ("k_norm_w", P), ("rope", P),
                ("q_out", P)]


class AttnArgs(ctypes.Structure):
    _fields_ = [("nq", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("max_q", ctypes.c_int32), ("max_kv", ctypes.c_int32), ("scale", ctypes.c_float), ("rows", I64),
                ("q", P), ("q_row", I64), ("q_head", I64), ("gate", P), ("gate_row", I64), ("gate_head", I64),
                ("out", P), ("out_row", I64), ("out_head", I64), ("workspace", P), ("workspace_bytes", SZ)]


_SIGS = {
    "fak_strerror": ([I32], ctypes.c_char_p),
    "fak_version": ([], ctypes.c_char_p),
    "fak_q4k_pack": ([P, I64, I64, P, SZ], I32),
    "fak_q8_0_pack": ([P, I64, I64, P, SZ], I32),
    "fak_q4k_pack_device": ([P, I64, I64, P, SZ, P], I32),
    "fak_q8_0_pack_device": ([P, I64, I64, P, SZ, P], I32),
    "fak_q4k_gemv": ([P, I64, I64, P, P, P], I32),
    "fak_q4k_gemv_i8x": ([P, I64, I64, P, P, P], I32),
    "fak_q8_0_gemv": ([P, I64, I64, P, P, P], I32),
    "fak_q4k_gemv_batch": ([P, I64, I64, P, I32, P, P], I32),
    "fak_mlp_workspace_bytes": ([I64], SZ),
    "fak_mlp_decode": ([P, P, P, I64, I64, P, ctypes.c_float, P, P, SZ, P], I32),
    "fak_mlp_decode_noalloc": ([P, P, P, I64, I64, P, ctypes.c_float, P, P], I32),
    "fak_q4k_gemm": ([P, I64, I64, P, I64, P, P], I32),
    "fak_swiglu_bf16": ([P, I64, I64, P, P], I32),
    "fak_q4k_gemm_swiglu": ([P, I64, I64, P, I64, P, P], I32),
    "fak_q4k_interleave_gate_up": ([P, P, I64, I64, P, P], I32),
    "fak_decode_create": ([ctypes.POINTER(DecodeDesc), ctypes.POINTER(P)], I32),
    "fak_decode_step": ([P, P, P, P, P], I32),
    "fak_decode_status": ([P, P], I32),
    "fak_decode_read_state": ([P, I32, P, SZ, P], I32),
    "fak_decode_reset": ([P, P], I32),
    "fak_decode_launches_per_step": ([P], I32),
    "fak_decode_set_timeout_ns": ([P, I64], I32),
    "fak_decode_debug_unreachable_wait": ([P, I32], I32),
    "fak_decode_destroy": ([P], None),
    "fak_device_status": ([P], I32),
    "fak_rope_table": ([I32, ctypes.c_double, P], I32),
    "fak_kv_append": ([P, P, P, P], I32),
    "fak_kv_read": ([P, P, I64, I32, P, P, P], I32),
    "fak_paged_attn_workspace_bytes": ([P, P, P], SZ),
    "fak_paged_attn": ([P, P, P, P], I32),
    "fak_paged_attn_debug_wait": ([I64, I32], I32),
    "fak_prefill_create": ([ctypes.POINTER(DecodeDesc), I64, ctypes.POINTER(P)], I32),
    "fak_prefill_run": ([P, P, P, P, P], I32),
    "fak_prefill_read_hidden": ([P, P, SZ, P], I32),
    "fak_prefill_kernels": ([P], I32),
    "fak_prefill_status": ([P, P], I32),
    "fak_prefill_destroy": ([P], None),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def fak_strerror(status):
    return lib.fak_strerror(int(status)).decode()


def fak_version():
    return lib.fak_version().decode()


def _check(status, where):
    if status != 0:
        raise FakError(status, where)


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if isinstance(t, np.ndarray):
        return t.ctypes.data
    return t.data_ptr()


def _current_stream():
    """torch's current stream; through its raw form, which costs a tenth, where torch has one."""
    global _current_stream
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    device = getattr(torch._C, "_cuda_getDevice", None)
    torch.cuda.current_stream()  # initialises CUDA
    if raw is None or device is None:
        _current_stream = lambda: torch.cuda.current_stream().cuda_stream
    else:
        _current_stream = lambda: raw(device())
    return _current_stream()


def _stream(stream):
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


# ------------------------------------------------------------------ host packers
def fak_q4k_pack(w):
    """Host f32 [N, K] -> uint8 [N, K/256*144] Q4_K bytes."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    N, K = w.shape
    out = np.empty((N, K // 256 * 144), dtype=np.uint8)
    _check(lib.fak_q4k_pack(w.ctypes.data, N, K, out.ctypes.data, out.nbytes), "fak_q4k_pack")
    return out


def fak_q8_0_pack(w):
    """Host f32 [N, K] -> uint8 [N, K/32*34] Q8_0 bytes."""
    w = np.ascontiguousarray(w, dtype=np.float32)
    N, K = w.shape
    out = np.empty((N, K // 32 * 34), dtype=np.uint8)
    _check(lib.fak_q8_0_pack(w.ctypes.data, N, K, out.ctypes.data, out.nbytes), "fak_q8_0_pack")
    return out


def fak_q4k_pack_device(w, N, K, out, stream=None):
    """Device f32 [N, K] (tensor or pointer) -> device Q4_K bytes `out` (N*(K/256)*144 bytes)."""
    nbytes = N * (K // 256) * 144
    _check(lib.fak_q4k_pack_device(_ptr(w), N, K, _ptr(out), nbytes, _stream(stream)), "fak_q4k_pack_device")


def fak_q8_0_pack_device(w, N, K, out, stream=None):
    """Device f32 [N, K] -> device Q8_0 bytes `out` (N*(K/32)*34 bytes)."""
    nbytes = N * (K // 32) * 34
    _check(lib.fak_q8_0_pack_device(_ptr(w), N, K, _ptr(out), nbytes, _stream(stream)), "fak_q8_0_pack_device")


# ------------------------------------------------------------------ device calls
def fak_q4k_gemv(Wq, N, K, x, y, stream=None):
    _check(lib.fak_q4k_gemv(_ptr(Wq), N, K, _ptr(x), _ptr(y), _stream(stream)), "fak_q4k_gemv")


def fak_q4k_gemv_i8x(Wq, N, K, x, y, stream=None):
    """fak_q4k_gemv on int8 activations (one scale per 32-element sub-block of x)."""
    _check(lib.fak_q4k_gemv_i8x(_ptr(Wq), N, K, _ptr(x), _ptr(y), _stream(stream)), "fak_q4k_gemv_i8x")


def fak_q8_0_gemv(Wq, N, K, x, y, stream=None):
    _check(lib.fak_q8_0_gemv(_ptr(Wq), N, K, _ptr(x), _ptr(y), _stream(stream)), "fak_q8_0_gemv")


def fak_q4k_gemv_batch(Wq, N, K, X, M, Y, stream=None):
    _check(lib.fak_q4k_gemv_batch(_ptr(Wq), N, K, _ptr(X), M, _ptr(Y), _stream(stream)), "fak_q4k_gemv_batch")


def fak_mlp_workspace_bytes(d_ff):
    return int(lib.fak_mlp_workspace_bytes(d_ff))


def fak_mlp_decode(Wgate, Wup, Wdown, d_model, d_ff, x, eps, y, workspace, workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _check(lib.fak_mlp_decode(_ptr(Wgate), _ptr(Wup), _ptr(Wdown), d_model, d_ff, _ptr(x), float(eps), _ptr(y),
                              _ptr(workspace), workspace_bytes, _stream(stream)), "fak_mlp_decode")


def fak_mlp_decode_noalloc(Wgate, Wup, Wdown, d_model, d_ff, x, eps, y, stream=None):
    """fak_mlp_decode with the library's own static scratch (no allocation; calls must not overlap)."""
    _check(lib.fak_mlp_decode_noalloc(_ptr(Wgate), _ptr(Wup), _ptr(Wdown), d_model, d_ff, _ptr(x), float(eps),
                                      _ptr(y), _stream(stream)), "fak_mlp_decode_noalloc")


def fak_q4k_gemm(Wq, N, K, X, P_, Y, stream=None):
    _check(lib.fak_q4k_gemm(_ptr(Wq), N, K, _ptr(X), P_, _ptr(Y), _stream(stream)), "fak_q4k_gemm")


def fak_swiglu_bf16(Y1, P_, half, X2, stream=None):
    _check(lib.fak_swiglu_bf16(_ptr(Y1), P_, half, _ptr(X2), _stream(stream)), "fak_swiglu_bf16")


def fak_q4k_gemm_swiglu(W13, F, K, X, P_, X2, stream=None):
    _check(lib.fak_q4k_gemm_swiglu(_ptr(W13), F, K, _ptr(X), P_, _ptr(X2), _stream(stream)), "fak_q4k_gemm_swiglu")


def fak_q4k_interleave_gate_up(Wg, Wu, F, K, W13, stream=None):
    _check(lib.fak_q4k_interleave_gate_up(_ptr(Wg), _ptr(Wu), F, K, _ptr(W13), _stream(stream)),
           "fak_q4k_interleave_gate_up")


def fak_device_status(stream=None):
    return int(lib.fak_device_status(_stream(stream)))


# ------------------------------------------------------------------ paged KV cache and attention
# The kernels run on the current device and read what they are given there: every call looks whether all of it is on that
# device, and nothing on the host (whose tensors' device is -1).
def _current_device():
    """torch's current CUDA device; as _current_stream."""
    global _current_device
    import torch
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    return torch.cuda.current_device()


def _one_device(where, tensors):
    """The CUDA device of all the tensors that are given (-1: the host's)."""
    tensors = [t for t in tensors if t is not None]
    if any(t.device != tensors[0].device for t in tensors):
        raise FakError(8, where)
    return tensors[0].get_device()


class KVCache:
    """A paged cache's description: codes k, v [n_pages, n_kv, page, dh] (contiguous; bfloat16, or for e4m3 uint8 or
    float8_e4m3fn, for int8 int8 or uint8) and in the 8-bit kinds scales [n_pages, n_kv, page] f32.  Keeps the tensors
    alive.  Calls on tensors of the host or of another device than the current one are refused (FAK_ERR_UNSUPPORTED)."""

    def __init__(self, kind, k, v, k_scale=None, v_scale=None):
        import torch
        types = {FAK_KV_BF16: (torch.bfloat16,), FAK_KV_E4M3: (torch.uint8, torch.float8_e4m3fn),
                 FAK_KV_I8: (torch.int8, torch.uint8)}.get(kind, ())
        scales = [t for t in (k_scale, v_scale) if t is not None]
        if k.shape != v.shape or k.dim() != 4 or any(t.shape != k.shape[:3] for t in scales):
            raise FakError(2, "KVCache")
        if any(t.dtype not in types or not t.is_contiguous() for t in (k, v)) or any(
                t.dtype != torch.float32 or not t.is_contiguous() for t in scales):
            raise FakError(1, "KVCache")
        self.device = _one_device("KVCache", (k, v, k_scale, v_scale))
        self._keep = (k, v, k_scale, v_scale)
        n_pages, n_kv, page, dh = k.shape
        self.kind, self.n_kv, self.dh = kind, n_kv, dh
        self.desc = KvCacheDesc(kind, n_kv, dh, page, n_pages, _ptr(k), _ptr(v), _ptr(k_scale), _ptr(v_scale))
        self.ref = ctypes.addressof(self.desc)


class KVBatch:
    """A ragged batch's description: int32 device tensors page_table [n_seqs, max_pages], row_start [n_seqs + 1]
    and kv_len [n_seqs], read when the kernels run.  Keeps the tensors alive."""

    def __init__(self, page_table, row_start, kv_len):
        import torch
        n = page_table.shape[0]
        if page_table.dim() != 2 or row_start.shape != (n + 1,) or kv_len.shape != (n,):
            raise FakError(2, "KVBatch")
        if any(t.dtype != torch.int32 or not t.is_contiguous() for t in (page_table, row_start, kv_len)):
            raise FakError(1, "KVBatch")
        self.device = _one_device("KVBatch", (page_table, row_start, kv_len))
        self._keep = (page_table, row_start, kv_len)
        self.desc = KvBatchDesc(n, page_table.shape[1], _ptr(page_table), _ptr(row_start), _ptr(kv_len))
        self.ref = ctypes.addressof(self.desc)


def _float_types():
    """torch's float32 and bfloat16 (this module does without torch until a call brings tensors)."""
    global _float_types
    import torch
    types = torch.float32, torch.bfloat16
    _float_types = lambda: types
    return types


def _index_types():
    """torch's 64-bit integers."""
    global _index_types
    import torch
    types = torch.int64, torch.uint64
    _index_types = lambda: types
    return types


def _heads(t, heads, dh, dtype, where):
    """Pointer, row stride and head stride of rows [rows, heads, dh] with neighbouring values in a head."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dh:
        raise FakError(2, where)
    if t.dtype != dtype or stride[2] != 1:
        raise FakError(1, where)
    return t.data_ptr(), stride[0], stride[1]


def _gain(w, dh, f32, where):
    """Pointer of a norm's gain: f32, dh values next to each other; None: no norm."""
    if w is None:
        return None
    if w.dtype != f32 or not w.is_contiguous():
        raise FakError(1, where)
    if w.numel() != dh:
        raise FakError(2, where)
    return w.data_ptr()


def _rope(table, rot, where):
    """Pointer of a rotary table: 64-bit integers, rot / 2 or more of them."""
    if table is None:
        return None
    if table.dtype not in _index_types() or not table.is_contiguous():
        raise FakError(1, where)
    if 2 * table.numel() < rot:
        raise FakError(2, where)
    return table.data_ptr()


def fak_rope_table(rot, theta):
    """Host int64 [rot / 2]: the rotary frequencies as 64-bit fractions of a turn (copy it to the device)."""
    out = np.empty(max(0, rot // 2), dtype=np.int64)
    _check(lib.fak_rope_table(int(rot), float(theta), out.ctypes.data), "fak_rope_table")
    return out


def fak_kv_append(cache, batch, k, v, q=None, q_out=None, q_norm_w=None, k_norm_w=None, eps=1e-6, rope=None, rot=0,
                  stream=None):
    """k, v [rows, n_kv, dh] and q [rows, nq, dh], f32 or bf16 (views with strides are fine); q_out bf16; gains f32 [dh];
    rope int64, fak_rope_table's values on the device."""
    dtype, (f32, bf16) = k.dtype, _float_types()
    if (dtype != f32 and dtype != bf16) or (q is not None and (
            q_out is None or q_out.dtype != bf16 or not q_out.is_contiguous())):
        raise FakError(1, "fak_kv_append")
    if v.shape[0] != k.shape[0] or (q is not None and (q.shape[0] != k.shape[0] or q_out.shape != q.shape)):
        raise FakError(2, "fak_kv_append")
    kp, kr, kh = _heads(k, cache.n_kv, cache.dh, dtype, "fak_kv_append")
    vp, vr, vh = _heads(v, cache.n_kv, cache.dh, dtype, "fak_kv_append")
    nq = 0 if q is None else q.shape[1]
    qp, qr, qh = (None, 0, 0) if q is None else _heads(q, nq, cache.dh, dtype, "fak_kv_append")
    r = KvRows(FAK_ROWS_F32 if dtype == f32 else FAK_ROWS_BF16, nq, rot, eps, k.shape[0], qp, kp, vp, qr, qh, kr, kh, vr,
               vh, _gain(q_norm_w, cache.dh, f32, "fak_kv_append"), _gain(k_norm_w, cache.dh, f32, "fak_kv_append"),
               _rope(rope, rot, "fak_kv_append"), _ptr(q_out))
    # (written out: these calls are bound by the host where rows are few)
    d = cache.device
    if (d < 0 or batch.device != d or k.get_device() != d or v.get_device() != d
            or (q is not None and (q.get_device() != d or q_out.get_device() != d))
            or (q_norm_w is not None and q_norm_w.get_device() != d)
            or (k_norm_w is not None and k_norm_w.get_device() != d)
            or (rope is not None and rope.get_device() != d) or _current_device() != d):
        raise FakError(8, "fak_kv_append")
    _check(lib.fak_kv_append(cache.ref, batch.ref, ctypes.addressof(r), _stream(stream)), "fak_kv_append")


def fak_kv_read(cache, batch, k_out, v_out, stream=None):
    """k_out, v_out [rows, n_kv, dh] contiguous, both f32 or both bf16; either may be None."""
    outs = [t for t in (k_out, v_out) if t is not None]
    if not outs or any(not t.is_contiguous() or t.dtype not in _float_types() for t in outs) or (
            outs[0].dtype != outs[-1].dtype):
        raise FakError(1, "fak_kv_read")
    if any(t.dim() != 3 or t.shape[1:] != (cache.n_kv, cache.dh) or t.shape[0] != outs[0].shape[0] for t in outs):
        raise FakError(2, "fak_kv_read")
    kind = FAK_ROWS_F32 if outs[0].element_size() == 4 else FAK_ROWS_BF16
    d = cache.device
    if d < 0 or batch.device != d or any(t.get_device() != d for t in outs) or _current_device() != d:
        raise FakError(8, "fak_kv_read")
    _check(lib.fak_kv_read(cache.ref, batch.ref, outs[0].shape[0], kind, _ptr(k_out), _ptr(v_out), _stream(stream)),
           "fak_kv_read")


def fak_paged_attn_workspace_bytes(cache, batch, nq, rows, max_q, max_kv, window=0, sinks=0):
    a = AttnArgs(nq, window, sinks, max_q, max_kv, 1.0, rows)
    return int(lib.fak_paged_attn_workspace_bytes(cache.ref, batch.ref, ctypes.addressof(a)))


def fak_paged_attn(cache, batch, q, out, max_q, max_kv, scale=None, window=0, sinks=0, gate=None, workspace=None,
                   stream=None):
    """q, out [rows, nq, dh] bf16 and gate f32 (views with strides are fine); scale defaults to dh^-1/2."""
    nq, (f32, bf16) = q.shape[1], _float_types()
    if out.shape != q.shape or (gate is not None and gate.shape != q.shape):
        raise FakError(2, "fak_paged_attn")
    if workspace is not None and not workspace.is_contiguous():
        raise FakError(1, "fak_paged_attn")
    qp, qr, qh = _heads(q, nq, cache.dh, bf16, "fak_paged_attn")
    op, orow, oh = _heads(out, nq, cache.dh, bf16, "fak_paged_attn")
    gp, gr, gh = (None, 0, 0) if gate is None else _heads(gate, nq, cache.dh, f32, "fak_paged_attn")
    a = AttnArgs(nq, window, sinks, max_q, max_kv, cache.dh ** -0.5 if scale is None else scale, q.shape[0], qp, qr, qh,
                 gp, gr, gh, op, orow, oh, _ptr(workspace),
                 0 if workspace is None else workspace.numel() * workspace.element_size())
    d = cache.device
    if (d < 0 or batch.device != d or q.get_device() != d or out.get_device() != d
            or (gate is not None and gate.get_device() != d)
            or (workspace is not None and workspace.get_device() != d) or _current_device() != d):
        raise FakError(8, "fak_paged_attn")
    _check(lib.fak_paged_attn(cache.ref, batch.ref, ctypes.addressof(a), _stream(stream)), "fak_paged_attn")


def fak_paged_attn_debug_wait(timeout_ns=0, unreachable=0):
    """Test hooks: the limit of the attention's waits (0: the default), and a wait that can never complete."""
    _check(lib.fak_paged_attn_debug_wait(int(timeout_ns), int(unreachable)), "fak_paged_attn_debug_wait")


# ------------------------------------------------------------------ decode context
class DecodeContext:
    """Owns a fak_decode context.  `layers` is a list of dicts with keys kind, w_in,
    w_k, w_v, w_out, w_gate, w_up, w_down (device tensors or pointers)."""

    def __init__(self, d_model, d_ff, vocab, gdn_in, fa_qg, fa_kv, n_mix, layers, lm_head, embedding,
                 eps=1e-6, mode=FAK_DECODE_ONE_LAUNCH, mixer=None):
        """mixer: None (projections only), or a dict with the head counts gdn_nk, gdn_nv, fa_nq, fa_nkv,
        fa_rot, rope_theta, eps, max_ctx and `layers`: one dict per layer with the device tensors
        conv_w, a_log, dt_bias, norm_w (GDN layers) or q_norm_w, k_norm_w (FA layers)."""
        self._keep = (layers, lm_head, embedding, mixer)
        arr = (LayerDesc * max(1, len(layers)))()
        for i, L in enumerate(layers):
            arr[i].kind = L["kind"]
            for key in ("w_in", "w_k", "w_v", "w_out", "w_gate", "w_up", "w_down"):
                setattr(arr[i], key, _ptr(L.get(key)))
        self._arr = arr
        mptr = None
        if mixer is not None:
            ml = (MixerLayer * max(1, len(layers)))()
            for i, M in enumerate(mixer["layers"]):
                for key in ("conv_w", "a_log", "dt_bias", "norm_w", "q_norm_w", "k_norm_w"):
                    setattr(ml[i], key, _ptr(M.get(key)))
            self._ml = ml
            self._md = MixerDesc(mixer["gdn_nk"], mixer["gdn_nv"], 128, 128, mixer["fa_nq"], mixer["fa_nkv"], 256,
                                 mixer["fa_rot"], float(mixer["rope_theta"]), float(mixer["eps"]), mixer["max_ctx"],
                                 ctypes.cast(ml, ctypes.POINTER(MixerLayer)))
            mptr = ctypes.pointer(self._md)
        desc = DecodeDesc(len(layers), d_model, d_ff, vocab, gdn_in, fa_qg, fa_kv, n_mix, float(eps), mode,
                          ctypes.cast(arr, ctypes.POINTER(LayerDesc)), _ptr(lm_head), _ptr(embedding), mptr)
        h = P()
        _check(lib.fak_decode_create(ctypes.byref(desc), ctypes.byref(h)), "fak_decode_create")
        self.handle = h
        self.d_model, self.vocab, self.fa_kv = d_model, vocab, fa_kv
        self.n_fa = sum(1 for L in layers if L["kind"] == FAK_LAYER_FA)

    def step(self, tok_in, tok_out, logits=None, stream=None):
        _check(lib.fak_decode_step(self.handle, _ptr(tok_in), _ptr(tok_out), _ptr(logits), _stream(stream)),
               "fak_decode_step")

    def status(self, stream=None):
        return int(lib.fak_decode_status(self.handle, _stream(stream)))

    def reset(self, stream=None):
        """Start a new sequence: clear the mixer state (conv states, S, KV cache, position)."""
        _check(lib.fak_decode_reset(self.handle, _stream(stream)), "fak_decode_reset")

    def read_state(self, which, dst, stream=None):
        """which 0: hidden state [d_model]; 1: FA k/v projections [n_fa][2][fa_kv]; 2: the last
        layer's mixer output [n_mix]."""
        count = dst.numel() if hasattr(dst, "numel") else dst.size
        _check(lib.fak_decode_read_state(self.handle, int(which), _ptr(dst), count, _stream(stream)),
               "fak_decode_read_state")

    def launches_per_step(self):
        return int(lib.fak_decode_launches_per_step(self.handle))

    def set_timeout_ns(self, ns):
        _check(lib.fak_decode_set_timeout_ns(self.handle, int(ns)), "fak_decode_set_timeout_ns")

    def debug_unreachable_wait(self, op_index):
        _check(lib.fak_decode_debug_unreachable_wait(self.handle, int(op_index)), "fak_decode_debug_unreachable_wait")

    def close(self):
        if self.handle:
            lib.fak_decode_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def fak_decode_create(*args, **kw):
    return DecodeContext(*args, **kw)


# ------------------------------------------------------------------ prefill forward
class PrefillContext:
    """Owns a fak_prefill context: the projections-only prefill forward of P tokens as one CUDA graph.
    Same model arguments as DecodeContext (no mixer)."""

    def __init__(self, d_model, d_ff, vocab, gdn_in, fa_qg, fa_kv, n_mix, layers, lm_head, embedding, n_tokens,
                 eps=1e-6):
        self._keep = (layers, lm_head, embedding)
        arr = (LayerDesc * max(1, len(layers)))()
        for i, L in enumerate(layers):
            arr[i].kind = L["kind"]
            for key in ("w_in", "w_k", "w_v", "w_out", "w_gate", "w_up", "w_down"):
                setattr(arr[i], key, _ptr(L.get(key)))
        self._arr = arr
        desc = DecodeDesc(len(layers), d_model, d_ff, vocab, gdn_in, fa_qg, fa_kv, n_mix, float(eps), 0,
                          ctypes.cast(arr, ctypes.POINTER(LayerDesc)), _ptr(lm_head), _ptr(embedding), None)
        h = P()
        _check(lib.fak_prefill_create(ctypes.byref(desc), int(n_tokens), ctypes.byref(h)), "fak_prefill_create")
        self.handle = h
        self.P, self.d_model, self.vocab = int(n_tokens), d_model, vocab

    def run(self, tokens, tok_out, logits=None, stream=None):
        _check(lib.fak_prefill_run(self.handle, _ptr(tokens), _ptr(tok_out), _ptr(logits), _stream(stream)),
               "fak_prefill_run")

    def read_hidden(self, dst, stream=None):
        count = dst.numel() if hasattr(dst, "numel") else dst.size
        _check(lib.fak_prefill_read_hidden(self.handle, _ptr(dst), count, _stream(stream)), "fak_prefill_read_hidden")

    def kernels(self):
        return int(lib.fak_prefill_kernels(self.handle))

    def status(self, stream=None):
        return int(lib.fak_prefill_status(self.handle, _stream(stream)))

    def close(self):
        if self.handle:
            lib.fak_prefill_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
