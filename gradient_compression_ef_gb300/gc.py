"""ctypes binding of ``libgc.so`` (the C ABI declared in include/gc.h).

Argument marshalling only: every step of the compressor runs in the CUDA
kernels of the library.  Functions take torch CUDA tensors (or raw device
addresses as ints) and pass ``data_ptr()`` values through unchanged.  There
is no fallback: importing this module raises if the library is missing.

    from gradient_compression_ef_gb300 import gc
    ctx = gc.Context(max_n)                  # bound to the current stream
    gc.ef_topk(ctx, grad, err, k, idx, val)  # asynchronous on ctx's stream
    ctx.check()                              # sync + device status
"""
import ctypes
import os

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libgc.so")

MINMAX, QSGD, TERN, LOG = 0, 1, 2, 3
NEAREST_EVEN, STOCHASTIC = 0, 1
MODES = {"minmax": MINMAX, "qsgd": QSGD, "tern": TERN, "log": LOG}
ROUNDINGS = {"nearest_even": NEAREST_EVEN, "stochastic": STOCHASTIC}

F32, BF16, F16 = 0, 1, 2
DTYPES = {"f32": F32, "bf16": BF16, "f16": F16}
GELU, SILU = 0, 1
ACTS = {"gelu": GELU, "silu": SILU}

PHASE_COUNT = 35

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_WORKSPACE = -1, -2, -3, -4
ERR_CUDA, ERR_DEVICE_CHECK, ERR_NO_MEMORY = -5, -6, -7

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_u64 = ctypes.c_uint64
_int = ctypes.c_int

# (name, restype, argtypes) of every function declared in include/gc.h
SIGNATURES = [
    ("gc_version", _int, []),
    ("gc_status_string", ctypes.c_char_p, [_int]),
    ("gc_ctx_create", _int, [ctypes.POINTER(_vp), _vp, _i64]),
    ("gc_ctx_destroy", _int, [_vp]),
    ("gc_ctx_set_stream", _int, [_vp, _vp]),
    ("gc_ctx_reserve_powersgd", _int, [_vp, _i64, _i64, _int]),
    ("gc_ctx_check", _int, [_vp]),
    ("gc_phase_name", ctypes.c_char_p, [_int]),
    ("gc_ctx_enable_timing", _int, [_vp, _int]),
    ("gc_ctx_read_timing", _int, [_vp, ctypes.POINTER(ctypes.c_double),
                                  ctypes.POINTER(ctypes.c_int64)]),
    ("gc_ctx_launch_count", _i64, [_vp]),
    ("gc_codes_bytes", _i64, [_i64, _int, _int]),
    ("gc_scales_floats", _i64, [_i64, _i64, _int]),
    ("gc_ef_topk", _int, [_vp, _vp, _vp, _i64, _i64, _vp, _vp]),
    ("gc_quant", _int, [_vp, _vp, _i64, _int, _i64, _int, _int, _u64, _u64, _vp, _vp]),
    ("gc_dequant", _int, [_vp, _vp, _vp, _i64, _int, _i64, _int, _vp]),
    ("gc_ef_quant", _int, [_vp, _vp, _vp, _i64, _int, _i64, _int, _int, _u64, _u64, _vp, _vp]),
    ("gc_ef_topk_quant", _int, [_vp, _vp, _vp, _i64, _i64, _int, _i64, _int, _u64, _u64,
                                _vp, _vp, _vp]),
    ("gc_ef_diff_quant", _int, [_vp, _vp, _vp, _vp, _i64, _int, _i64, _int, _int, _u64, _u64,
                                _int, _vp, _vp]),
    ("gc_diff_dequant", _int, [_vp, _vp, _vp, _i64, _int, _i64, _int, _int, _vp]),
    ("gc_powersgd_step", _int, [_vp, _vp, _vp, _i64, _i64, _int, _vp, _vp]),
    ("gc_ef_topk_noalloc", _int, [_vp, _vp, _i64, _i64, _vp, _vp, _vp]),
    ("gc_bucket_seed", _u64, [_u64, _int]),
    ("gc_ctx_set_buckets", _int, [_vp, _int, ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    ("gc_ctx_set_deferred_residual", _int, [_vp, _int]),
    ("gc_bucket_flush", _int, [_vp]),
    ("gc_bucket_offsets", _int, [_int, ctypes.POINTER(_i64), _int, _i64, ctypes.POINTER(_i64),
                                 ctypes.POINTER(_i64), ctypes.POINTER(_i64)]),
    ("gc_ef_topk_buckets", _int, [_vp, _vp, _vp, _vp, _vp, _vp]),
    ("gc_ef_topk_quant_buckets", _int, [_vp, _vp, _vp, _int, _i64, _int, _u64, _u64, _vp, _vp,
                                        _vp, _vp]),
    ("gc_ef_randk", _int, [_vp, _vp, _vp, _i64, ctypes.c_float, _u64, _u64, _vp, _vp, _i64,
                           _vp]),
    ("gc_topk_aggregate", _int, [_vp, _int, _i64, _vp, _vp, _i64, _vp]),
    ("gc_topk_quant_aggregate", _int, [_vp, _int, _i64, _vp, _vp, _vp, _int, _i64, _i64, _vp]),
    ("gc_ckpt_codes_bytes", _i64, [_i64, _i64]),
    ("gc_ckpt_scales_bytes", _i64, [_i64, _i64]),
    ("gc_ctx_reserve_scratch", _int, [_vp, _i64]),
    ("gc_ckpt_save", _int, [_vp, _vp, _int, _i64, _i64, _i64, _vp, _vp]),
    ("gc_ckpt_restore", _int, [_vp, _vp, _vp, _int, _i64, _i64, _vp, _i64]),
    ("gc_act_forward", _int, [_vp, _int, _vp, _i64, _vp, _i64, _int, _i64, _i64, _vp, _i64,
                              _vp, _vp, _vp, _vp]),
    ("gc_act_backward", _int, [_vp, _int, _vp, _i64, _vp, _vp, _vp, _vp, _int, _i64, _i64, _vp,
                               _i64, _vp, _i64]),
    ("gc_layernorm_forward", _int, [_vp, _vp, _i64, _int, _i64, _i64, _vp, _vp, _int,
                                    ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _vp]),
    ("gc_layernorm_scratch_bytes", _i64, [_i64, _i64]),
    ("gc_layernorm_backward", _int, [_vp, _vp, _i64, _vp, _i64, _vp, _vp, _int, _i64, _i64, _vp,
                                     _int, _vp, _vp, _vp, _i64, _vp, _vp, _int]),
    ("gc_linear_wgrad_scratch_bytes", _i64, [_i64, _i64, _i64, _int]),
    ("gc_linear_wgrad", _int, [_vp, _vp, _int, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _vp,
                               _int]),
]

# largest n of gc_ef_topk_noalloc (GC_NOALLOC_MAX_N in include/gc.h)
NOALLOC_MAX_N = 1048576


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libgc.so is not built (%s); run `python -c \"import __graft_entry__ as g; "
            "g.build()\"` first -- there is no non-CUDA fallback" % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, res, args in SIGNATURES:
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class GCError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s (%d)" % (what, status_string(status), status))


def phase_name(phase):
    return lib.gc_phase_name(phase).decode()


def status_string(status):
    return lib.gc_status_string(status).decode()


def _check(status, what):
    if status != OK:
        raise GCError(status, what)


def _ptr(t):
    """Device address of a tensor (or an int address / None)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _mode(m):
    return MODES[m] if isinstance(m, str) else int(m)


def _rounding(r):
    return ROUNDINGS[r] if isinstance(r, str) else int(r)


def codes_bytes(n, bits, mode):
    return int(lib.gc_codes_bytes(n, bits, _mode(mode)))


def scales_floats(n, group, mode):
    return int(lib.gc_scales_floats(n, group, _mode(mode)))


class Context:
    """A gc_ctx: scratch for calls of up to ``max_n`` elements, bound to a
    CUDA stream (default: torch's current stream at creation)."""

    def __init__(self, max_n, stream=None):
        if stream is None:
            import torch
            stream = torch.cuda.current_stream()
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        self._stream_ref = stream
        h = _vp()
        _check(lib.gc_ctx_create(ctypes.byref(h), handle, max_n), "gc_ctx_create")
        self.handle = h
        self.max_n = max_n

    def set_stream(self, stream):
        handle = stream if isinstance(stream, int) else stream.cuda_stream
        _check(lib.gc_ctx_set_stream(self.handle, handle), "gc_ctx_set_stream")
        self._stream_ref = stream

    def reserve_powersgd(self, max_m, max_n, max_r):
        _check(lib.gc_ctx_reserve_powersgd(self.handle, max_m, max_n, max_r),
               "gc_ctx_reserve_powersgd")

    def reserve_scratch(self, nbytes):
        """At least nbytes of scratch for layernorm_backward and linear_wgrad
        (their *_scratch_bytes).  What it grows out of stays allocated (captured
        graphs may use it): reserve the largest size first."""
        _check(lib.gc_ctx_reserve_scratch(self.handle, nbytes), "gc_ctx_reserve_scratch")

    def check(self):
        _check(lib.gc_ctx_check(self.handle), "gc_ctx_check")

    def enable_timing(self, max_launches):
        """Brackets each later kernel launch with CUDA events on the stream."""
        _check(lib.gc_ctx_enable_timing(self.handle, max_launches), "gc_ctx_enable_timing")

    def read_timing(self):
        """{phase name: (total ms, launches)} of the timed launches since the
        last read (synchronises the stream)."""
        ms = (ctypes.c_double * PHASE_COUNT)()
        cnt = (ctypes.c_int64 * PHASE_COUNT)()
        _check(lib.gc_ctx_read_timing(self.handle, ms, cnt), "gc_ctx_read_timing")
        return {phase_name(p): (ms[p], cnt[p]) for p in range(PHASE_COUNT) if cnt[p]}

    def launch_count(self):
        return int(lib.gc_ctx_launch_count(self.handle))

    def set_buckets(self, bucket_n, bucket_k):
        """Bucket plan: consecutive slices of bucket_n[b] elements keeping
        bucket_k[b] entries each (synchronous)."""
        nb = len(bucket_n)
        if len(bucket_k) != nb:
            raise ValueError("bucket_n and bucket_k differ in length")
        an = (_i64 * max(nb, 1))(*[int(v) for v in bucket_n])
        ak = (_i64 * max(nb, 1))(*[int(v) for v in bucket_k])
        _check(lib.gc_ctx_set_buckets(self.handle, nb, an, ak), "gc_ctx_set_buckets")
        self.bucket_n = [int(v) for v in bucket_n]
        self.bucket_k = [int(v) for v in bucket_k]

    def set_deferred_residual(self, on):
        """on: the bucketed calls with error feedback keep the kept entries'
        residuals aside and the next bucketed call on the same err applies
        them as it reads e; err is exact only after bucket_flush().  off:
        flushes, then writes e' in full again."""
        _check(lib.gc_ctx_set_deferred_residual(self.handle, 1 if on else 0),
               "gc_ctx_set_deferred_residual")

    def bucket_flush(self):
        """Writes the pending residuals of the last deferred bucketed call into
        its err (asynchronous on the context's stream)."""
        _check(lib.gc_bucket_flush(self.handle), "gc_bucket_flush")

    def close(self):
        if getattr(self, "handle", None) is not None and self.handle.value:
            st = lib.gc_ctx_destroy(self.handle)
            self.handle = None
            _check(st, "gc_ctx_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            if getattr(self, "handle", None) is not None and self.handle.value:
                lib.gc_ctx_destroy(self.handle)
        except Exception:
            pass


def ef_topk(ctx, grad, err, k, idx_out, val_out, n=None):
    n = grad.numel() if n is None else n
    _check(lib.gc_ef_topk(ctx.handle, _ptr(grad), _ptr(err), n, k, _ptr(idx_out),
                          _ptr(val_out)), "gc_ef_topk")


def quant(ctx, x, bits, group, mode, rounding, seed, step, codes_out, scales_out, n=None):
    n = x.numel() if n is None else n
    _check(lib.gc_quant(ctx.handle, _ptr(x), n, bits, group, _mode(mode), _rounding(rounding),
                        seed, step, _ptr(codes_out), _ptr(scales_out)), "gc_quant")


def dequant(ctx, codes, scales, n, bits, group, mode, x_out):
    _check(lib.gc_dequant(ctx.handle, _ptr(codes), _ptr(scales), n, bits, group, _mode(mode),
                          _ptr(x_out)), "gc_dequant")


def ef_quant(ctx, grad, err, bits, group, mode, rounding, seed, step, codes_out, scales_out,
             n=None):
    n = grad.numel() if n is None else n
    _check(lib.gc_ef_quant(ctx.handle, _ptr(grad), _ptr(err), n, bits, group, _mode(mode),
                           _rounding(rounding), seed, step, _ptr(codes_out),
                           _ptr(scales_out)), "gc_ef_quant")


def ef_diff_quant(ctx, grad, err, ref, bits, group, mode, rounding, seed, step, refresh,
                  codes_out, scales_out, n=None):
    """Differential quantisation against the history ref (updated in place);
    err may be None."""
    n = grad.numel() if n is None else n
    _check(lib.gc_ef_diff_quant(ctx.handle, _ptr(grad), _ptr(err), _ptr(ref), n, bits, group,
                                _mode(mode), _rounding(rounding), seed, step,
                                1 if refresh else 0, _ptr(codes_out), _ptr(scales_out)),
           "gc_ef_diff_quant")


def diff_dequant(ctx, codes, scales, n, bits, group, mode, refresh, ref):
    _check(lib.gc_diff_dequant(ctx.handle, _ptr(codes), _ptr(scales), n, bits, group,
                               _mode(mode), 1 if refresh else 0, _ptr(ref)), "gc_diff_dequant")


def ef_topk_quant(ctx, grad, err, k, bits, group, rounding, seed, step, idx_out, codes_out,
                  scales_out, n=None):
    n = grad.numel() if n is None else n
    _check(lib.gc_ef_topk_quant(ctx.handle, _ptr(grad), _ptr(err), n, k, bits, group,
                                _rounding(rounding), seed, step, _ptr(idx_out),
                                _ptr(codes_out), _ptr(scales_out)), "gc_ef_topk_quant")


def powersgd_step(ctx, grad, err, m, n, r, P_out, Q_inout):
    _check(lib.gc_powersgd_step(ctx.handle, _ptr(grad), _ptr(err), m, n, r, _ptr(P_out),
                                _ptr(Q_inout)), "gc_powersgd_step")


def ef_topk_noalloc(grad, err, k, idx_out, val_out, stream=None, n=None):
    """gc_ef_topk_noalloc: EF + Top-K with no context and no allocation, on
    ``stream`` (default: torch's current stream); n <= NOALLOC_MAX_N."""
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    n = grad.numel() if n is None else n
    _check(lib.gc_ef_topk_noalloc(_ptr(grad), _ptr(err), n, k, _ptr(idx_out), _ptr(val_out),
                                  handle), "gc_ef_topk_noalloc")


def bucket_seed(seed, b):
    """The Philox key the bucketed calls give bucket b for ``seed``."""
    return int(lib.gc_bucket_seed(seed, b))


def bucket_offsets(bucket_k, bits=None, group=None):
    """gc_bucket_offsets: (idx_off, codes_off, scales_off), each a list of
    nb + 1 starts (the last is the total); codes_off / scales_off are None
    when bits / group are not given."""
    nb = len(bucket_k)
    ak = (_i64 * max(nb, 1))(*[int(v) for v in bucket_k])
    oi = (_i64 * (nb + 1))()
    oc = (_i64 * (nb + 1))() if bits is not None else None
    os_ = (_i64 * (nb + 1))() if group is not None else None
    _check(lib.gc_bucket_offsets(nb, ak, 0 if bits is None else bits,
                                 0 if group is None else group, oi, oc, os_),
           "gc_bucket_offsets")
    return (list(oi), list(oc) if oc is not None else None,
            list(os_) if os_ is not None else None)


def ef_topk_buckets(ctx, grad, err, idx_out, val_out, diag=None):
    """diag: None, or a device float64 tensor of 3 * nb values receiving per
    bucket (sum c^2, sum g_hat^2, sum e'^2)."""
    _check(lib.gc_ef_topk_buckets(ctx.handle, _ptr(grad), _ptr(err), _ptr(idx_out),
                                  _ptr(val_out), _ptr(diag)), "gc_ef_topk_buckets")


def ef_topk_quant_buckets(ctx, grad, err, bits, group, rounding, seed, step, idx_out,
                          codes_out, scales_out, diag=None):
    _check(lib.gc_ef_topk_quant_buckets(ctx.handle, _ptr(grad), _ptr(err), bits, group,
                                        _rounding(rounding), seed, step, _ptr(idx_out),
                                        _ptr(codes_out), _ptr(scales_out), _ptr(diag)),
           "gc_ef_topk_quant_buckets")



def topk_aggregate(ctx, W, k, idx, val, n, out):
    """gc_topk_aggregate: out[n] = rank-ordered sum of W ranks' (idx, val)."""
    _check(lib.gc_topk_aggregate(ctx.handle, W, k, _ptr(idx), _ptr(val), n, _ptr(out)),
           "gc_topk_aggregate")


def topk_quant_aggregate(ctx, W, k, idx, codes, scales, bits, group, n, out):
    """gc_topk_quant_aggregate: the same with QSGD-coded values per rank."""
    _check(lib.gc_topk_quant_aggregate(ctx.handle, W, k, _ptr(idx), _ptr(codes), _ptr(scales),
                                       bits, group, n, _ptr(out)), "gc_topk_quant_aggregate")


def ef_randk(ctx, grad, err, p, seed, step, idx_out, val_out, count_out, n=None, capacity=None):
    """gc_ef_randk: EF + random sparsification; count_out is a device int64
    tensor receiving the kept count."""
    n = grad.numel() if n is None else n
    capacity = idx_out.numel() if capacity is None else capacity
    _check(lib.gc_ef_randk(ctx.handle, _ptr(grad), _ptr(err), n, float(p), seed, step,
                           _ptr(idx_out), _ptr(val_out), capacity, _ptr(count_out)),
           "gc_ef_randk")


# --- the backward pass that fills the flat gradient: 8-bit activation
# checkpoints, activation functions, layer norm, linear weight gradients ----

_TORCH = {}  # torch dtype -> GC_* type, filled when the first tensor comes
_U8 = _F32 = None


def _types():
    global _U8, _F32
    import torch
    _U8, _F32 = torch.uint8, torch.float32
    _TORCH.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})


def _dtype(t):
    """GC_* type of a torch tensor, a torch dtype or a name."""
    if isinstance(t, str):
        return DTYPES[t]
    dt = getattr(t, "dtype", t)
    if not _TORCH:
        _types()
    try:
        return _TORCH[dt]
    except KeyError:
        raise TypeError("unsupported element type %s (float32, bfloat16 or float16)" % dt) from None


def _matrix(t, what, like=None):
    """(rows, cols, row stride) of a 2-D tensor with contiguous columns,
    which must have the shape and type of `like` if given."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got %d-D" % (what, len(shape)))
    rows, cols = shape
    sr, sc = t.stride()
    if sc != 1 and cols > 1:
        raise ValueError("%s: columns must be contiguous (stride %d)" % (what, sc))
    if rows <= 1:
        sr = cols
    elif sr < cols:
        raise ValueError("%s: overlapping rows (stride %d, %d columns)" % (what, sr, cols))
    if like is not None and (shape != like.shape or t.dtype != like.dtype):
        raise ValueError("%s: %s %s, expected %s %s" % (
            what, tuple(shape), t.dtype, tuple(like.shape), like.dtype))
    return rows, cols, sr


def _floats(t, n, what):
    """Address of a contiguous fp32 tensor (or None) of at least n elements."""
    if t is None:
        return None
    if not _TORCH:
        _types()
    if t.dtype != _F32 or t.numel() < n or not t.is_contiguous():
        raise ValueError("%s: needs %d contiguous float32" % (what, n))
    return t.data_ptr()


def _ckpt(codes, scales, rows, cols):
    """Addresses of a checkpoint's buffers (either may be None)."""
    if codes is None and scales is None:
        return None, None
    if not _TORCH:
        _types()
    groups = (cols + 31) >> 5
    if codes is not None and (codes.dtype != _U8 or codes.numel() < rows * groups * 32
                              or not codes.is_contiguous()):
        raise ValueError("codes: needs %d contiguous uint8" % (rows * groups * 32))
    if scales is not None and (scales.dtype != _U8
                               or scales.numel() < rows * (((groups + 15) >> 4) << 4)
                               or not scales.is_contiguous()):
        raise ValueError("scales: needs %d contiguous uint8" % (rows * (((groups + 15) >> 4) << 4)))
    return (None if codes is None else codes.data_ptr(),
            None if scales is None else scales.data_ptr())


def _param(t, cols, what):
    if t is None:
        return None
    if t.numel() != cols or not t.is_contiguous():
        raise ValueError("%s: needs %d contiguous values" % (what, cols))
    return t.data_ptr()


def _act(act):
    return ACTS[act] if isinstance(act, str) else int(act)


def ckpt_codes_bytes(rows, cols):
    return int(lib.gc_ckpt_codes_bytes(rows, cols))


def ckpt_scales_bytes(rows, cols):
    return int(lib.gc_ckpt_scales_bytes(rows, cols))


def ckpt_save(ctx, x, codes, scales):
    """Saves x [rows, cols] as an 8-bit checkpoint."""
    rows, cols, ldx = _matrix(x, "x")
    c, s = _ckpt(codes, scales, rows, cols)
    _check(lib.gc_ckpt_save(ctx.handle, x.data_ptr(), _dtype(x), rows, cols, ldx, c, s),
           "gc_ckpt_save")


def ckpt_restore(ctx, codes, scales, x_out):
    """Writes the values a checkpoint stands for into x_out [rows, cols]."""
    rows, cols, ldx = _matrix(x_out, "x_out")
    c, s = _ckpt(codes, scales, rows, cols)
    _check(lib.gc_ckpt_restore(ctx.handle, c, s, _dtype(x_out), rows, cols, x_out.data_ptr(),
                               ldx), "gc_ckpt_restore")


def act_forward(ctx, act, x, y, codes=None, scales=None, gate=None, gate_codes=None,
                gate_scales=None):
    """y = act(x) [* gate]; codes / scales receive the checkpoint of x (and
    gate_codes / gate_scales that of gate)."""
    rows, cols, ldx = _matrix(x, "x")
    _, _, ldy = _matrix(y, "y", x)
    ldg = _matrix(gate, "gate", x)[2] if gate is not None else 0
    c, s = _ckpt(codes, scales, rows, cols)
    gc_, gs = _ckpt(gate_codes, gate_scales, rows, cols)
    _check(lib.gc_act_forward(ctx.handle, _act(act), x.data_ptr(), ldx, None if gate is None else gate.data_ptr(), ldg,
                              _dtype(x), rows, cols, y.data_ptr(), ldy, c, s, gc_, gs),
           "gc_act_forward")


def act_backward(ctx, act, dy, dx, codes, scales, dgate=None, gate_codes=None, gate_scales=None):
    """dx (and dgate) of act_forward from its checkpoints."""
    rows, cols, lddy = _matrix(dy, "dy")
    _, _, lddx = _matrix(dx, "dx", dy)
    ldg = _matrix(dgate, "dgate", dy)[2] if dgate is not None else 0
    c, s = _ckpt(codes, scales, rows, cols)
    gc_, gs = _ckpt(gate_codes, gate_scales, rows, cols)
    _check(lib.gc_act_backward(ctx.handle, _act(act), dy.data_ptr(), lddy, c, s, gc_, gs, _dtype(dy), rows, cols,
                               dx.data_ptr(), lddx, None if dgate is None else dgate.data_ptr(),
                               ldg), "gc_act_backward")


def layernorm_scratch_bytes(rows, cols):
    return int(lib.gc_layernorm_scratch_bytes(rows, cols))


def layernorm_forward(ctx, x, gamma, beta, eps, y, mean, rstd, codes=None, scales=None):
    """Layer norm over the columns; gamma / beta may be None; codes / scales
    receive the checkpoint of x."""
    rows, cols, ldx = _matrix(x, "x")
    _, _, ldy = _matrix(y, "y", x)
    if gamma is not None and beta is not None and gamma.dtype != beta.dtype:
        raise ValueError("gamma and beta differ in type")
    p = gamma if gamma is not None else beta
    c, s = _ckpt(codes, scales, rows, cols)
    _check(lib.gc_layernorm_forward(
        ctx.handle, x.data_ptr(), ldx, _dtype(x), rows, cols, _param(gamma, cols, "gamma"),
        _param(beta, cols, "beta"), F32 if p is None else _dtype(p), eps, y.data_ptr(), ldy,
        _floats(mean, rows, "mean"), _floats(rstd, rows, "rstd"),
        c, s), "gc_layernorm_forward")


def layernorm_backward(ctx, dy, x, gamma, mean, rstd, dx, dgamma=None, dbeta=None, codes=None,
                       scales=None, accumulate=False):
    """Layer norm backward from x, or (x None) from its checkpoint; dgamma /
    dbeta: fp32 tensors of cols elements (slices of the flat gradient), or
    None."""
    rows, cols, lddy = _matrix(dy, "dy")
    _, _, lddx = _matrix(dx, "dx", dy)
    ldx = _matrix(x, "x", dy)[2] if x is not None else 0
    c, s = _ckpt(codes, scales, rows, cols)
    _check(lib.gc_layernorm_backward(
        ctx.handle, dy.data_ptr(), lddy, None if x is None else x.data_ptr(), ldx, c, s,
        _dtype(dy), rows, cols, _param(gamma, cols, "gamma"),
        F32 if gamma is None else _dtype(gamma), _floats(mean, rows, "mean"),
        _floats(rstd, rows, "rstd"), dx.data_ptr(), lddx,
        _floats(dgamma, cols, "dgamma"),
        _floats(dbeta, cols, "dbeta"), 1 if accumulate else 0),
        "gc_layernorm_backward")


def linear_wgrad_scratch_bytes(rows, out_features, in_features, dtype):
    return int(lib.gc_linear_wgrad_scratch_bytes(rows, out_features, in_features, _dtype(dtype)))


def linear_wgrad(ctx, dy, codes, scales, dw, db=None, accumulate=False):
    """dw [out, in] (and db [out]) of a linear layer, fp32, from dy
    [rows, out] and the checkpoint of its input [rows, in]."""
    rows, out, lddy = _matrix(dy, "dy")
    wo, in_features, lddw = _matrix(dw, "dw")
    if wo != out or _dtype(dw) != F32:
        raise ValueError("dw: %s %s, expected fp32 with %d rows" % (tuple(dw.shape), dw.dtype,
                                                                   out))
    c, s = _ckpt(codes, scales, rows, in_features)
    _check(lib.gc_linear_wgrad(ctx.handle, dy.data_ptr(), _dtype(dy), lddy, c, s, rows, out,
                               in_features, dw.data_ptr(), lddw,
                               _floats(db, out, "db"), 1 if accumulate else 0),
           "gc_linear_wgrad")
