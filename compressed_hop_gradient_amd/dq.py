"""Python binding of the C ABI in ``include/dq.h``.

Argument marshalling only: every stage runs in the HIP kernels of
``libdq.so``.  PyTorch supplies device memory (tensors) and the stream
(``torch.cuda.current_stream()``).  If the shared library is missing the
import of this module's functions raises; there is no CPU fallback.
"""
import ctypes as C
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdq.so")

DQ_OK, DQ_EINVAL, DQ_EBUDGET, DQ_ESTATE, DQ_EWORKSPACE, DQ_ENULL, DQ_EHIP, DQ_ENONFINITE = \
    0, -1, -2, -3, -4, -5, -6, -7
RING, BUTTERFLY = 0, 1
BF16, F32, PACKED, F32_PARTIAL = 0, 1, 2, 3
OWN_PACKED, OWN_F32 = 0, 1
CORRELATED, INDEPENDENT, STRATIFIED = 0, 1, 2
OPT_SEED, OPT_ROUND, OPT_ROUNDING, OPT_TIMING, OPT_ALLOC, OPT_TIMING_KINDS, OPT_OWN = 0, 1, 2, 3, 4, 5, 6
OPT_STREAMS = 7
OPT_MAX_WIDTH = 8
ALLOC_THRESHOLD, ALLOC_MEAN_CORRECTED, ALLOC_UNIFORM = 0, 1, 2
MX_FP8_E4M3, MX_FP6_E3M2, MX_FP6_E2M3, MX_FP4_E2M1 = 0, 1, 2, 3
OPT_EPS = 0   # dq_option_f64
ROUTE_RENORM = 1   # dq_route_flags
ROUTE_MAX_PARTS = 16
EXPERT_GATHER, EXPERT_TURNED = 1, 2   # dq_expert_flags
GATHER_NONE, GATHER_X, GATHER_DOUT = 0, 1, 2
KEEP_DITHER = 1
ACT_SWIGLU, ACT_RELU = 0, 1
KERNEL_KINDS = ("stats", "allocate", "reorder", "compress", "hop_grad", "hop_packed",
                "finalize", "mxfp8", "hop_final")


class dq_info(C.Structure):
    _fields_ = [("rho_bits", C.c_uint32), ("rho", C.c_float), ("t12", C.c_float),
                ("t24", C.c_float), ("t48", C.c_float), ("class_counts", C.c_int64 * 3),
                ("budget_bits", C.c_int64), ("used_bits", C.c_int64),
                ("achieved_bits", C.c_double), ("nonfinite", C.c_int32), ("t816", C.c_float),
                ("class_count16", C.c_int64)]


class dq_layout(C.Structure):
    _fields_ = [(n, C.c_size_t) for n in ("sum", "sumsq", "widths", "perm", "inv", "mu_stream",
                                          "tables", "ctrl", "total", "tables16")]


class dq_timing(C.Structure):
    _fields_ = [("ms", C.c_double * len(KERNEL_KINDS)), ("launches", C.c_int64 * len(KERNEL_KINDS)),
                ("coords", C.c_int64 * len(KERNEL_KINDS))]


class dq_route_worker(C.Structure):
    _fields_ = [("d_logits", C.c_void_p), ("tokens", C.c_int64), ("stride", C.c_int64), ("d_mask", C.c_void_p),
                ("d_ids", C.c_void_p), ("d_gates", C.c_void_p), ("d_part", C.c_void_p), ("part_bytes", C.c_size_t)]


class dq_route_grad(C.Structure):
    _fields_ = [("d_logits", C.c_void_p), ("tokens", C.c_int64), ("stride", C.c_int64), ("d_mask", C.c_void_p),
                ("d_ids", C.c_void_p), ("d_dgates", C.c_void_p), ("d_dlogits", C.c_void_p), ("dstride", C.c_int64)]


class dq_route_part(C.Structure):
    _fields_ = [("d_part", C.c_void_p), ("tokens", C.c_int64)]


class dq_expert_lists(C.Structure):
    _fields_ = [("d_offsets", C.c_void_p), ("d_source", C.c_void_p), ("d_row", C.c_void_p), ("tokens", C.c_int64),
                ("top_k", C.c_int32), ("n_experts", C.c_int32)]


class dq_keep_key(C.Structure):
    _fields_ = [("seed", C.c_uint64), ("d_round", C.c_void_p), ("round", C.c_uint32), ("worker", C.c_int32),
                ("site", C.c_uint32), ("flags", C.c_int32)]


class DQError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


_lib = None

# exported symbols and their signatures (every declaration of include/dq.h)
_SIGS = {
    "dq_plan_create": (C.c_int, [C.c_int64, C.c_int32, C.c_int32, C.c_float, C.POINTER(C.c_void_p)]),
    "dq_plan_destroy": (None, [C.c_void_p]),
    "dq_plan_set_u64": (C.c_int, [C.c_void_p, C.c_int32, C.c_uint64]),
    "dq_workspace_bytes": (C.c_size_t, [C.c_void_p]),
    "dq_plan_bind": (C.c_int, [C.c_void_p, C.c_void_p, C.c_size_t]),
    "dq_workspace_layout": (C.c_int, [C.c_void_p, C.POINTER(dq_layout)]),
    "dq_region_bytes_max": (C.c_size_t, [C.c_void_p, C.c_int64]),
    "dq_stats": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p]),
    "dq_allocate": (C.c_int, [C.c_void_p, C.c_void_p]),
    "dq_reorder": (C.c_int, [C.c_void_p, C.c_void_p]),
    "dq_compress": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p,
                              C.c_void_p]),
    "dq_hop": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_int32,
                         C.c_void_p, C.c_void_p, C.c_void_p]),
    "dq_finalize": (C.c_int, [C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p]),
    "dq_final_part": (C.c_int64, [C.c_void_p, C.c_int32]),
    "dq_arena_bytes": (C.c_size_t, [C.c_void_p]),
    "dq_allreduce": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_size_t,
                               C.c_void_p, C.c_void_p]),
    "dq_noalloc_max_bytes": (C.c_size_t, []),
    "dq_allreduce_noalloc": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_void_p]),
    "dq_mxfp8_arena_bytes": (C.c_size_t, [C.c_void_p]),
    "dq_mxfp8_allreduce": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_void_p, C.c_size_t,
                                     C.c_void_p, C.c_void_p]),
    "dq_mx_arena_bytes": (C.c_size_t, [C.c_void_p]),
    "dq_hop_finalize": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_int32,
                                  C.c_void_p, C.c_void_p, C.c_void_p]),
    "dq_partial_bytes_max": (C.c_size_t, [C.c_void_p, C.c_int64]),
    "dq_plan_set_f64": (C.c_int, [C.c_void_p, C.c_int32, C.c_double]),
    "dq_mx_allreduce": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_void_p, C.c_size_t,
                                  C.c_void_p, C.c_void_p]),
    "dq_check_reciprocal": (C.c_int, [C.c_uint32, C.c_uint32, C.c_void_p, C.c_void_p]),
    "dq_check_round_half_up": (C.c_int, [C.c_uint32, C.c_uint32, C.c_void_p, C.c_void_p]),
    "dq_probe_stream": (C.c_int, [C.c_void_p, C.c_size_t, C.c_void_p, C.c_size_t, C.c_int32,
                                  C.c_void_p]),
    "dq_dropout": (C.c_int, [C.c_void_p, C.c_void_p, C.c_void_p, C.c_int32, C.c_int64, C.c_int64, C.c_int64,
                             C.c_int64, C.c_int64, C.c_double, C.c_uint64, C.c_uint32, C.c_void_p,
                             C.c_int32, C.c_uint32, C.c_void_p]),
    "dq_route_part_bytes": (C.c_size_t, [C.c_int64, C.c_int32]),
    "dq_route": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_void_p]),
    "dq_balance": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p,
                             C.c_void_p, C.c_void_p, C.c_void_p]),
    "dq_route_backward": (C.c_int, [C.c_void_p, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_void_p,
                                    C.c_void_p, C.c_void_p]),
    "dq_expert_rows_bytes": (C.c_size_t, [C.c_int64, C.c_int32, C.c_int32]),
    "dq_expert_rows": (C.c_int, [C.c_void_p, C.c_int64, C.c_int32, C.c_int32, C.c_void_p, C.c_void_p, C.c_void_p,
                                 C.c_void_p, C.c_size_t, C.c_void_p]),
    "dq_expert_matmul": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_int32, C.c_void_p, C.c_int64, C.c_int64,
                                   C.c_void_p, C.c_int64, C.c_int32, C.c_int64, C.c_int64, C.c_void_p]),
    "dq_expert_matmul_grad_bytes": (C.c_size_t, [C.c_int64, C.c_int32, C.c_int32, C.c_int32, C.c_int32, C.c_int64,
                                                 C.c_int64, C.c_int32]),
    "dq_expert_matmul_grad": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p,
                                        C.c_int64, C.c_int32, C.c_void_p, C.c_int32, C.c_int32, C.c_int64,
                                        C.c_int64, C.c_void_p, C.c_size_t, C.c_void_p]),
    "dq_expert_sum": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64, C.c_void_p, C.c_int64,
                                C.c_int32, C.c_int64, C.c_void_p]),
    "dq_keep8": (C.c_int, [C.c_void_p, C.c_int32, C.c_int64, C.c_int64, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p,
                           C.c_void_p]),
    "dq_restore8": (C.c_int, [C.c_void_p, C.c_void_p, C.c_int32, C.c_int64, C.c_int64, C.c_void_p, C.c_int64,
                              C.c_void_p]),
    "dq_expert_act": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64,
                                C.c_int32, C.c_int64, C.c_void_p, C.c_void_p, C.c_void_p, C.c_void_p]),
    "dq_expert_act_backward": (C.c_int, [C.c_void_p, C.c_int32, C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p,
                                         C.c_void_p, C.c_int64, C.c_void_p, C.c_void_p, C.c_int64, C.c_void_p,
                                         C.c_int64, C.c_void_p, C.c_int32, C.c_int64, C.c_void_p]),
    "dq_get_info": (C.c_int, [C.c_void_p, C.POINTER(dq_info), C.c_void_p]),
    "dq_timing_read": (C.c_int, [C.c_void_p, C.POINTER(dq_timing)]),
    "dq_status_string": (C.c_char_p, [C.c_int32]),
    "dq_version": (C.c_int32, []),
}


def lib():
    """Load ``libdq.so`` (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} is missing "
                               "(run __graft_entry__.build())")
        L = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(s):
    return lib().dq_status_string(int(s)).decode()


def _check(rc, what):
    if rc != DQ_OK:
        raise DQError(rc, what)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return C.c_void_p(stream.cuda_stream)


def _ptr(t):
    return C.c_void_p(t.data_ptr())


def _kind(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    if t.dtype == torch.uint8:
        return PACKED
    raise TypeError(f"unsupported tensor dtype {t.dtype}")


def _tensor(t, what, device, numel=None, min_bytes=None, dtype=None):
    """Reject what the kernels cannot address safely: tensors on the host or on
    another device, non-contiguous views and buffers shorter than the call
    writes or reads (the C ABI takes bare pointers and cannot check sizes)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device != device:
        raise ValueError(f"{what}: tensor on {t.device}, the plan works on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what}: dtype {t.dtype}, expected {dtype}")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{what}: {t.numel()} elements, expected {numel}")
    if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
        raise ValueError(f"{what}: {t.numel() * t.element_size()} bytes, the call needs {min_bytes}")
    return t


def check_reciprocal(lo_bits, count, device=None, stream=None):
    """Mismatches between the codec's reciprocal and the IEEE quotient 1/x over
    the fp32 bit patterns [lo_bits, lo_bits + count) (runs on the GPU)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    cnt = torch.zeros(1, dtype=torch.int64, device=dev)
    _check(lib().dq_check_reciprocal(int(lo_bits), int(count), _ptr(cnt), _stream(stream)),
           "dq_check_reciprocal")
    return int(cnt.item())


def check_round_half_up(lo_bits, count, device=None, stream=None):
    """Mismatches between the codec's round-half-up conversion and the exact
    floor(x + 0.5) (NaN saturated by its sign) over the fp32 bit patterns
    [lo_bits, lo_bits + count)
    (runs on the GPU)."""
    dev = torch.device("cuda") if device is None else torch.device(device)
    cnt = torch.zeros(1, dtype=torch.int64, device=dev)
    _check(lib().dq_check_round_half_up(int(lo_bits), int(count), _ptr(cnt), _stream(stream)),
           "dq_check_round_half_up")
    return int(cnt.item())


def probe_stream(src, dst, reads_per_write, stream=None):
    """Run the streaming probe over the bytes of ``src`` (device tensor) with
    the given read:write mix, writing into ``dst``."""
    dev = src.device
    _tensor(src, "src", dev)
    _tensor(dst, "dst", dev)
    _check(lib().dq_probe_stream(_ptr(src), src.numel() * src.element_size(), _ptr(dst),
                                 dst.numel() * dst.element_size(), int(reads_per_write),
                                 _stream(stream)), "dq_probe_stream")


# ---- training step (every call takes stream=, as under torch.cuda.stream) --------

def _rows(t, what):
    """(rows, cols, row stride) of a tensor as a matrix of its last dimension:
    one row when contiguous; any views whose rows lie at one stride."""
    if t.is_contiguous():
        return 1, t.numel(), t.numel()
    if t.dim() == 0 or t.stride(-1) != 1 and t.size(-1) != 1:
        raise ValueError(f"{what}: the last dimension must be contiguous")
    rows, stride = 1, None
    for size, step in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if stride is None:
            stride = step
        elif step != rows * stride:
            raise ValueError(f"{what}: shape {tuple(t.shape)} with strides {t.stride()} has no common row stride")
        rows *= size
    return rows, t.size(-1), t.size(-1) if stride is None else stride


def _gpu(t, what):
    """A float tensor the kernels read: bf16 or fp32, on a GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.dtype != torch.bfloat16 and t.dtype != torch.float32:
        raise TypeError(f"{what}: dtype {t.dtype} (bf16 or fp32 only)")
    if t.device.type != "cuda":
        raise ValueError(f"{what}: tensor on {t.device}, the kernels run on a GPU")
    return t


def _raw_stream(dev):
    """The current stream's handle (torch.cuda.current_stream builds an object:
    2.9 us where a whole call takes about 10, against 0.1)."""
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _call(dev, name, *args):
    """Call a stateless entry point on ``dev``'s current stream."""
    stream = _raw_stream(dev)
    if dev.index == torch.cuda.current_device():
        rc = getattr(lib(), name)(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = getattr(lib(), name)(*args, stream)
    if rc != DQ_OK:
        raise DQError(rc, name)


def _on_stream(fn):
    """``stream=s`` means: as under ``torch.cuda.stream(s)``, so that results and
    scratch are allocated for the stream that uses them."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _like(t, x, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a torch.Tensor, got {type(t).__name__}")
    if t.shape != x.shape or t.dtype != x.dtype or t.device != x.device:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on {t.device}, "
                         f"x is {tuple(x.shape)} {x.dtype} on {x.device}")
    return t


def _opt(t):
    return None if t is None else t.data_ptr()


@_on_stream
def dropout(x, p, residual=None, seed=1, rnd=0, worker=0, site=0, out=None):
    """``residual + dropout(x)``, or ``dropout(x)`` (``dq_dropout``).

    The mask is a function of (seed, rnd, worker, site, element) and is never
    stored.  ``x``, ``residual`` and ``out`` are bf16 or fp32, of one dtype and
    shape, contiguous or with rows at one stride; ``out`` may be ``x`` or
    ``residual``.  ``rnd`` is the step: an int, or a one-element int32 GPU tensor that
    the kernel reads (for captured graphs: a replay takes the tensor's new value)."""
    dev = _gpu(x, "x").device
    rows, cols, xs = _rows(x, "x")
    flat, rs, ys = rows == 1, cols, cols
    if residual is not None:
        n, _, rs = _rows(_like(residual, x, "residual"), "residual")
        flat = flat and n == 1
    if out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
    else:
        n, _, ys = _rows(_like(out, x, "out"), "out")
        flat = flat and n == 1
    if not flat:                # rows at their strides; contiguous operands among them
        cols = x.size(-1)
        rows = x.numel() // cols
        xs, rs, ys = (cols if t is None or t.is_contiguous() else stride
                      for t, stride in ((x, xs), (residual, rs), (out, ys)))
    d_round = None
    if isinstance(rnd, torch.Tensor):
        d_round = _tensor(rnd, "rnd", dev, numel=1, dtype=torch.int32).data_ptr()
        rnd = 0
    # beyond these, marshalling would wrap them into other numbers
    if not (0 <= rnd < 1 << 32 and 0 <= worker < 1 << 16 and 0 <= site < 1 << 31 and 0 <= seed < 1 << 64):
        raise ValueError(f"seed {seed}, rnd {rnd}, worker {worker}, site {site}: expected 64, 32, 16 and 31 bits")
    _call(dev, "dq_dropout", x.data_ptr(), _opt(residual), out.data_ptr(),
          F32 if x.dtype == torch.float32 else BF16, rows, cols, xs, rs, ys, p,
          seed, rnd, d_round, worker, site)
    return out


def dropout_backward(dout, p, seed=1, rnd=0, worker=0, site=0, out=None, stream=None):
    """Gradient of :func:`dropout` by ``x``, from the same numbers as the
    forward call (the gradient by ``residual`` is ``dout`` itself)."""
    return dropout(dout, p, None, seed, rnd, worker, site, out, stream=stream)


def _logits(t, what="logits"):
    _gpu(t, what)
    if t.dim() != 2 or t.size(1) > 1 and t.stride(1) != 1 and t.numel():
        raise ValueError(f"{what}: {tuple(t.shape)} with strides {t.stride()}, expected [tokens, experts] "
                         "with contiguous rows")
    return t


def _token_mask(mask, tokens, dev):
    if mask is None:
        return None
    _tensor(mask, "mask", dev, numel=tokens)
    if mask.dtype != torch.bool and mask.dtype != torch.uint8:
        raise TypeError(f"mask: dtype {mask.dtype}, expected bool or uint8")
    return mask.data_ptr()


def _result(t, shape, what, dtype, dev):
    """A buffer of the caller's for a result, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if isinstance(t, torch.Tensor) and t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _tensor(t, what, dev, dtype=dtype)


class RouteStats:
    """Balance statistics of the workers routed so far: the parts that
    :func:`route` wrote, folded on demand.  The first part holds the scratch of a
    fold, so calls on one object must not run side by side on several streams (let
    the later stream wait for the earlier, as for any tensor)."""

    def __init__(self, experts, device):
        self.experts, self.device = experts, device
        self.parts = []        # (buffer of dq_route, the part in it, its tokens, the stream it was made on)
        self.sums = None       # what was folded before them, fp64 [2 experts + 1]
        self._sums_on = None   # the stream that was made on, if it was made here

    def _add(self, part, at, tokens):
        if len(self.parts) == ROUTE_MAX_PARTS:
            self.fold()
        self.parts.append((part, at, tokens, _raw_stream(self.device)))

    def _balance(self, top_k, stats, loss, coef, counts):
        n = len(self.parts)
        array = (dq_route_part * n)(*[p[1:3] for p in self.parts])
        now = _raw_stream(self.device)
        for part, _, _, made in self.parts:
            if made != now:       # its memory is not to be reused there before this call has read it
                part.record_stream(torch.cuda.current_stream(self.device))
        if self.sums is not None and self._sums_on != now:
            self.sums.record_stream(torch.cuda.current_stream(self.device))
        _call(self.device, "dq_balance", array, n, _opt(self.sums), self.experts, top_k, _opt(stats), _opt(loss),
              _opt(coef), _opt(counts))

    def fold(self):
        """The statistics as one tensor: choices per expert, summed
        probabilities per expert, routed tokens (fp64 [2 experts + 1]).  Those
        of several processes add up; a change to the latest such tensor is one to
        these statistics.  A fold that has new parts makes a new one and leaves
        earlier ones as they are."""
        if self.parts:
            stats = torch.empty(2 * self.experts + 1, dtype=torch.float64, device=self.device)
            self._balance(1, stats, None, None, None)
            self.sums, self._sums_on, self.parts = stats, _raw_stream(self.device), []
        return self.sums


@functools.lru_cache(maxsize=256)
def _part_bytes(tokens, experts):
    return lib().dq_route_part_bytes(tokens, experts)


def _workers(logits, masks):
    """The workers' logits and masks as lists, of one dtype, width and device."""
    masks = [None] * len(logits) if masks is None else masks
    if not logits or len(masks) != len(logits):
        raise ValueError(f"{len(logits)} logits with {len(masks)} masks")
    first = _logits(logits[0])
    for l in logits[1:]:
        if _logits(l).size(1) != first.size(1) or l.dtype != first.dtype or l.device != first.device:
            raise ValueError(f"the workers' logits differ: {tuple(l.shape)} {l.dtype} on {l.device}, "
                             f"{tuple(first.shape)} {first.dtype} on {first.device}")
    return masks


def _results(given, tokens, width, what, dtype, dev):
    """The caller's buffers for a [tokens, width] result of each worker, or new
    ones."""
    given = [None] * len(tokens) if given is None else given
    if len(given) != len(tokens):
        raise ValueError(f"{len(given)} {what} for {len(tokens)} workers")
    return [_result(t, (n, width), what, dtype, dev) for t, n in zip(given, tokens)]


def _route_stats(stats, logits, top_k):
    if top_k < 1:
        raise ValueError(f"top_k {top_k}")
    if stats is None:
        return RouteStats(logits.size(1), logits.device)
    if not isinstance(stats, RouteStats):
        raise TypeError(f"stats: expected a RouteStats, got {type(stats).__name__}")
    if stats.experts != logits.size(1) or stats.device != logits.device:
        raise ValueError(f"stats of {stats.experts} experts on {stats.device}, "
                         f"logits of {logits.size(1)} on {logits.device}")
    return stats


def _route(io, n, logits, top_k, renorm, stats):
    _call(stats.device, "dq_route", io, n, _kind(logits), stats.experts, top_k, ROUTE_RENORM if renorm else 0)


@_on_stream
def route(logits, top_k, renorm=True, mask=None, stats=None, ids=None, gates=None):
    """Expert choice of every token (``dq_route``): returns (ids, gates, stats).

    ``logits`` is [tokens, experts], bf16 or fp32, rows at any stride; ``mask``
    (bool or uint8, [tokens]) is false for tokens left out.  ``ids`` is int32 and
    ``gates`` fp32, both [tokens, top_k], best choice first; -1 and 0 where a
    token has fewer open experts (logits above -inf).  ``stats`` is a
    :class:`RouteStats` for :func:`balance`: one that is passed in takes these tokens
    in addition (the workers in rank order).

    With lists of the workers' ``logits`` (and ``mask``) one call takes them all, and
    ``ids`` and ``gates`` are lists."""
    if isinstance(logits, (list, tuple)):
        masks = _workers(logits, mask)
        stats = _route_stats(stats, logits[0], top_k)
        tokens = [l.size(0) for l in logits]
        ids = _results(ids, tokens, top_k, "ids", torch.int32, stats.device)
        gates = _results(gates, tokens, top_k, "gates", torch.float32, stats.device)
        nbytes = [_part_bytes(t, stats.experts) for t in tokens]
        part = torch.empty(sum(nbytes), dtype=torch.uint8, device=stats.device)
        at, io = part.data_ptr(), []
        for l, t, m, i, g, n in zip(logits, tokens, masks, ids, gates, nbytes):
            io.append((l.data_ptr(), t, l.stride(0), _token_mask(m, t, stats.device), i.data_ptr(), g.data_ptr(), at, n))
            at += n
        _route((dq_route_worker * len(io))(*io), len(io), logits[0], top_k, renorm, stats)
        for w in io:
            stats._add(part, w[6], w[1])
        return ids, gates, stats
    tokens, experts = _logits(logits).shape
    dev = logits.device
    stats = _route_stats(stats, logits, top_k)
    ids = _result(ids, (tokens, top_k), "ids", torch.int32, dev)
    gates = _result(gates, (tokens, top_k), "gates", torch.float32, dev)
    nbytes = _part_bytes(tokens, experts)
    part = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    at = part.data_ptr()
    io = dq_route_worker(logits.data_ptr(), tokens, logits.stride(0), _token_mask(mask, tokens, dev), ids.data_ptr(),
                         gates.data_ptr(), at, nbytes)
    _route(C.byref(io), 1, logits, top_k, renorm, stats)
    stats._add(part, at, tokens)
    return ids, gates, stats


@_on_stream
def balance(stats, top_k):
    """Balance loss of the tokens in ``stats`` (``dq_balance``), a
    :class:`RouteStats` or the tensor that its ``fold`` gives: returns (loss [1] fp32,
    coef [experts] fp32, counts [experts] int64).  ``top_k`` is that of the route
    calls.  ``coef`` is the loss's derivative by any token's probabilities, which
    :func:`route_backward` takes."""
    if isinstance(stats, torch.Tensor):
        if stats.dim() != 1 or stats.numel() < 3 or stats.numel() % 2 == 0:
            raise ValueError(f"stats: shape {tuple(stats.shape)}, expected [2 experts + 1]")
        if stats.device.type != "cuda":
            raise ValueError(f"stats: tensor on {stats.device}, the kernels run on a GPU")
        sums = _tensor(stats, "stats", stats.device, dtype=torch.float64)
        stats = RouteStats(sums.numel() // 2, sums.device)
        stats.sums = sums
    elif not isinstance(stats, RouteStats):
        raise TypeError(f"stats: expected a RouteStats or its tensor, got {type(stats).__name__}")
    dev = stats.device
    loss = torch.empty(1, dtype=torch.float32, device=dev)
    coef = torch.empty(stats.experts, dtype=torch.float32, device=dev)
    counts = torch.empty(stats.experts, dtype=torch.int64, device=dev)
    stats._balance(top_k, None, loss, coef, counts)
    return loss, coef, counts


def _grad_fields(logits, ids, dgates, mask, out):
    tokens, dev = logits.size(0), logits.device
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.size(0) != tokens:
        raise ValueError(f"ids: expected [{tokens}, top_k] of route()")
    _tensor(ids, "ids", dev, dtype=torch.int32)
    if dgates is not None:
        _result(dgates, ids.shape, "dgates", torch.float32, dev)
    if _logits(out, "out").shape != logits.shape or out.dtype != logits.dtype or out.device != dev:
        raise ValueError(f"out: {tuple(out.shape)} {out.dtype} on {out.device}, "
                         f"logits are {tuple(logits.shape)} {logits.dtype} on {dev}")
    return (logits.data_ptr(), tokens, logits.stride(0), _token_mask(mask, tokens, dev), ids.data_ptr(), _opt(dgates),
            out.data_ptr(), out.stride(0))


def _route_grad(io, n, logits, ids, coef, dloss, renorm):
    dev, experts = logits.device, logits.size(1)
    if coef is not None:
        _tensor(coef, "coef", dev, numel=experts, dtype=torch.float32)
    if dloss is not None:
        _tensor(dloss, "dloss", dev, numel=1, dtype=torch.float32)
    _call(dev, "dq_route_backward", io, n, _kind(logits), experts, ids.size(1), ROUTE_RENORM if renorm else 0,
          _opt(coef), _opt(dloss))


@_on_stream
def route_backward(logits, ids, dgates=None, coef=None, dloss=None, renorm=True, mask=None, out=None):
    """Gradient by the logits (``dq_route_backward``) from the gates' gradient
    ``dgates`` and the balance loss's, ``dloss`` (one fp32 element; None: 1) times
    ``coef`` of :func:`balance`; either part may be None.  ``ids``, ``renorm`` and ``mask``
    as in the forward call; ``out`` may be ``logits``.  Lists as in :func:`route`, with
    None in ``dgates`` for a worker without."""
    if isinstance(logits, (list, tuple)):
        masks = _workers(logits, mask)
        n = len(logits)
        dgates = [None] * n if dgates is None else dgates
        if len(ids) != n or len(dgates) != n or out is not None and len(out) != n:
            raise ValueError(f"{len(ids)} ids, {len(dgates)} dgates and {0 if out is None else len(out)} out "
                             f"for {n} workers")
        tops = {i.size(-1) for i in ids if isinstance(i, torch.Tensor) and i.dim() == 2}
        if len(tops) != 1:
            raise ValueError(f"ids: expected [tokens, top_k] of route() for every worker, got top_k of {sorted(tops)}")
        outs = out
        if out is None:
            outs = [torch.empty_like(l, memory_format=torch.contiguous_format) for l in logits]
        io = [_grad_fields(*w) for w in zip(logits, ids, dgates, masks, outs)]
        _route_grad((dq_route_grad * n)(*io), n, logits[0], ids[0], coef, dloss, renorm)
        return outs
    _logits(logits)
    if out is None:
        out = torch.empty_like(logits, memory_format=torch.contiguous_format)
    io = dq_route_grad(*_grad_fields(logits, ids, dgates, mask, out))
    _route_grad(C.byref(io), 1, logits, ids, coef, dloss, renorm)
    return out


# ---- experts (every call takes stream=, as above) ---------------------------------

_ACTS = {"swiglu": ACT_SWIGLU, "relu": ACT_RELU}


def _round_of(rnd, dev):
    """(number, device pointer) of a round index: an int, or one int32 element
    that the kernel reads."""
    if isinstance(rnd, torch.Tensor):
        return 0, _tensor(rnd, "rnd", dev, numel=1, dtype=torch.int32).data_ptr()
    return rnd, None


def _keep_key(dither, seed, rnd, worker, site, dev):
    rnd, d_round = _round_of(rnd, dev)
    # beyond these, marshalling would wrap them into other numbers
    if not (0 <= rnd < 1 << 32 and 0 <= worker < 1 << 16 and 0 <= site < 1 << 31 and 0 <= seed < 1 << 64):
        raise ValueError(f"seed {seed}, rnd {rnd}, worker {worker}, site {site}: expected 64, 32, 16 and 31 bits")
    return C.byref(dq_keep_key(seed, d_round, rnd, worker, site, KEEP_DITHER if dither else 0))


class Kept8:
    """A tensor kept in 8 bits by :func:`keep8`: int8 ``codes`` of its shape, uint8
    ``exponents`` (one for every 32 elements of its last dimension, which it
    replaces), and the ``dtype`` it had."""

    @classmethod
    def _made(cls, shape, x):
        """Buffers for what is to be kept of ``x``."""
        kept = cls.__new__(cls)
        kept.codes = x.new_empty(shape, dtype=torch.int8)
        kept.exponents = x.new_empty((*shape[:-1], (shape[-1] + 31) // 32), dtype=torch.uint8)
        kept.dtype = x.dtype
        return kept

    def __init__(self, codes, exponents, dtype):
        if not isinstance(codes, torch.Tensor) or codes.dim() == 0 or codes.device.type != "cuda":
            raise ValueError("codes: expected a tensor of at least one dimension on a GPU")
        _tensor(codes, "codes", codes.device, dtype=torch.int8)
        _tensor(exponents, "exponents", codes.device, dtype=torch.uint8)
        if exponents.shape != codes.shape[:-1] + ((codes.size(-1) + 31) // 32,):
            raise ValueError(f"exponents: shape {tuple(exponents.shape)} for codes of {tuple(codes.shape)}")
        if dtype != torch.bfloat16 and dtype != torch.float32:
            raise TypeError(f"dtype {dtype} (bf16 or fp32 only)")
        self.codes, self.exponents, self.dtype = codes, exponents, dtype

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def _matrix_rows(t, what):
    """(rows, cols, row stride) of a tensor as a matrix of its last dimension, the
    row kept whole."""
    if t.dim() == 0:
        raise ValueError(f"{what}: expected at least one dimension")
    cols = t.size(-1)
    if t.is_contiguous():
        return (t.numel() // cols if cols else 0), cols, cols
    _, _, stride = _rows(t, what)
    return t.numel() // cols, cols, stride


@_on_stream
def keep8(x, dither=True, seed=1, rnd=0, worker=0, site=0):
    """``x`` in 8 bits, for the backward pass (``dq_keep8``): a :class:`Kept8` of 33
    bytes for 32 elements of the last dimension, which share a power of two.

    With ``dither`` the rounding is random, by numbers of (seed, rnd, worker, site,
    element), and the kept value's mean is ``x``; without, it is the nearest.  ``x`` is
    bf16 or fp32, contiguous or with rows at one stride; ``rnd`` as in
    :func:`dropout`."""
    dev = _gpu(x, "x").device
    rows, cols, stride = _matrix_rows(x, "x")
    key = _keep_key(dither, seed, rnd, worker, site, dev)
    kept = Kept8._made(x.shape, x)
    _call(dev, "dq_keep8", x.data_ptr(), _kind(x), rows, cols, stride, kept.codes.data_ptr(),
          kept.exponents.data_ptr(), key)
    return kept


@_on_stream
def restore8(kept, out=None):
    """The values that ``kept`` stands for (``dq_restore8``), exactly, in the dtype of
    what was kept; NaN for a block that was not finite (or beyond 127 2^121)."""
    if not isinstance(kept, Kept8):
        raise TypeError(f"kept: expected a Kept8, got {type(kept).__name__}")
    if out is None:
        out = kept.codes.new_empty(kept.shape, dtype=kept.dtype)
    elif _gpu(out, "out").shape != kept.shape or out.dtype != kept.dtype or out.device != kept.device:
        raise ValueError(f"out: {tuple(out.shape)} {out.dtype} on {out.device}, "
                         f"kept is {tuple(kept.shape)} {kept.dtype} on {kept.device}")
    rows, cols, stride = _matrix_rows(out, "out")
    _call(kept.device, "dq_restore8", kept.codes.data_ptr(), kept.exponents.data_ptr(), _kind(out), rows, cols,
          out.data_ptr(), stride)
    return out


class ExpertRows:
    """Rows of every expert, as :func:`expert_rows` lists them: ``offsets`` int32
    [experts + 1], the experts' first rows; ``source`` int32 [tokens * top_k], the slot
    (token * top_k + choice) of every row, those without an expert last; ``row`` int32
    [tokens, top_k], the row of every slot, -1 without an expert."""

    def __init__(self, offsets, source, row):
        if not isinstance(row, torch.Tensor) or row.dim() != 2 or row.device.type != "cuda":
            raise ValueError("row: expected a tensor [tokens, top_k] on a GPU")
        dev = row.device
        _tensor(row, "row", dev, dtype=torch.int32)
        _tensor(source, "source", dev, numel=row.numel(), dtype=torch.int32)
        _tensor(offsets, "offsets", dev, dtype=torch.int32)
        if offsets.dim() != 1 or offsets.numel() < 2:
            raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected [experts + 1]")
        self._set(offsets, source, row, dev, *row.shape, offsets.numel() - 1)

    def _set(self, offsets, source, row, dev, tokens, top_k, experts):
        self.offsets, self.source, self.row, self.device = offsets, source, row, dev
        self.tokens, self.top_k, self.slots, self.experts = tokens, top_k, tokens * top_k, experts
        self._io = C.byref(dq_expert_lists(offsets.data_ptr(), source.data_ptr(), row.data_ptr(), tokens, top_k,
                                           experts))
        return self


@functools.lru_cache(maxsize=256)
def _rows_bytes(tokens, top_k, experts):
    return lib().dq_expert_rows_bytes(tokens, top_k, experts)


@_on_stream
def expert_rows(ids, experts):
    """:class:`ExpertRows` of the choices ``ids`` [tokens, top_k] int32 of
    :func:`route` (``dq_expert_rows``): every expert's slots in the order of the tokens.
    Ids outside 0 .. experts - 1 are no choice.  Nothing waits for the GPU: how many
    rows an expert has stays on the device."""
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2 or ids.device.type != "cuda":
        raise ValueError("ids: expected [tokens, top_k] of route() on a GPU")
    dev = ids.device
    _tensor(ids, "ids", dev, dtype=torch.int32)
    tokens, top_k = ids.shape
    need = _rows_bytes(tokens, top_k, experts)
    if not need:
        raise ValueError(f"{tokens} tokens of {top_k} choices among {experts} experts")
    offsets, source, row = ids.new_empty(experts + 1), ids.new_empty(tokens * top_k), ids.new_empty((tokens, top_k))
    work = None if need <= 256 else ids.new_empty(need // 4)
    _call(dev, "dq_expert_rows", ids.data_ptr(), tokens, top_k, experts, offsets.data_ptr(), source.data_ptr(),
          row.data_ptr(), _opt(work), need)
    return ExpertRows.__new__(ExpertRows)._set(offsets, source, row, dev, tokens, top_k, experts)


def _expert_rows(rows):
    if not isinstance(rows, ExpertRows):
        raise TypeError(f"rows: expected an ExpertRows, got {type(rows).__name__}")
    return rows


def _row_matrix(t, what, n, dev, cols=None, dtype=None):
    """An operand [n, cols] whose rows are contiguous; its row stride."""
    if isinstance(t, torch.Tensor) and t.dim() == 2 and t.size(0) == n and t.device == dev and t.is_contiguous() and \
            (cols is None or t.size(1) == cols) and (dtype is None or t.dtype == dtype) and \
            (t.dtype == torch.bfloat16 or t.dtype == torch.float32):
        return t.size(1)                        # what almost all are
    _gpu(t, what)
    if t.dim() != 2 or t.size(0) != n or cols is not None and t.size(1) != cols or t.device != dev or \
            dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what}: {tuple(t.shape)} {t.dtype} on {t.device}, expected [{n}, "
                         f"{'width' if cols is None else cols}] {dtype or 'bf16 or fp32'} on {dev}")
    if t.size(1) > 1 and t.stride(1) != 1 and t.numel():
        raise ValueError(f"{what}: strides {t.stride()}, the last dimension must be contiguous")
    return t.stride(0)


def _row_result(t, what, n, cols, x):
    """A caller's buffer [n, cols] for a result like ``x``, or a new one."""
    if t is None:
        return x.new_empty((n, cols)), cols
    return t, _row_matrix(t, what, n, x.device, cols, x.dtype)


@_on_stream
def expert_matmul(x, w, rows, gather=False, out=None):
    """``x[r] @ w[e(r)]`` for every expert's rows (``dq_expert_matmul``): [tokens *
    top_k, outer] of the dtype of ``x``.

    ``x`` is [tokens * top_k, inner] in the order of ``rows``, or with ``gather`` the tokens
    themselves, [tokens, inner], read where they lie.  ``w`` is [experts, inner, outer],
    contiguous along one of the last two: the gradient by ``x`` is
    ``expert_matmul(dout, w.transpose(1, 2), rows)``.  Rows of ``x`` and ``out`` may lie at any
    stride.  Rows without an expert are left as they were (uninitialised in a new
    ``out``)."""
    dev = _expert_rows(rows).device
    xs = _row_matrix(x, "x", rows.tokens if gather else rows.slots, dev)
    if not isinstance(w, torch.Tensor) or w.dim() != 3 or w.size(0) != rows.experts or w.size(1) != x.size(1) or \
            w.dtype != x.dtype or w.device != dev:
        raise ValueError(f"w: {tuple(w.shape)} {w.dtype} on {w.device}, expected [{rows.experts}, {x.size(1)}, outer] "
                         f"{x.dtype} on {dev}" if isinstance(w, torch.Tensor) else "w: expected a torch.Tensor")
    _, inner, outer = w.shape
    we, w1, w2 = w.stride()
    flags = EXPERT_GATHER if gather else 0
    if w2 == 1 or outer == 1:
        ws = w1
    elif w1 == 1 or inner == 1:
        ws, flags = w2, flags | EXPERT_TURNED
    else:
        raise ValueError(f"w: strides {w.stride()}, one of the last two dimensions must be contiguous")
    out, ys = _row_result(out, "out", rows.slots, outer, x)
    _call(dev, "dq_expert_matmul", rows._io, x.data_ptr(), xs, flags, w.data_ptr(), we, ws, out.data_ptr(), ys,
          _kind(x), inner, outer)
    return out


@functools.lru_cache(maxsize=256)
def _grad_bytes(tokens, top_k, experts, kind, gather, inner, outer, kept):
    return lib().dq_expert_matmul_grad_bytes(tokens, top_k, experts, kind, gather, inner, outer, kept)


@_on_stream
def expert_matmul_grad(x, dout, rows, gather=None, dtype=None, out=None):
    """The gradient of :func:`expert_matmul` by ``w``: the sum of ``x[r]^T dout[r]`` over
    every expert's rows (``dq_expert_matmul_grad``), [experts, inner, outer] of ``dtype``
    (that of ``dout``, or fp32); zeros for an expert without rows.

    ``gather`` names which of ``"x"`` and ``"dout"`` holds tokens instead of rows, if one
    does.  ``x`` may be a :class:`Kept8`: it is decoded as it is read, or for long products
    once into scratch memory."""
    dev = _expert_rows(rows).device
    if gather not in (None, "x", "dout"):
        raise ValueError(f"gather {gather!r}: expected None, 'x' or 'dout'")
    n = rows.tokens if gather == "x" else rows.slots
    ds = _row_matrix(dout, "dout", rows.tokens if gather == "dout" else rows.slots, dev)
    if isinstance(x, Kept8):
        if x.codes.dim() != 2 or x.shape[0] != n or x.dtype != dout.dtype or x.device != dev:
            raise ValueError(f"x: kept {tuple(x.shape)} {x.dtype} on {x.device}, expected [{n}, inner] {dout.dtype} "
                             f"on {dev}")
        at, xs, codes, exponents, inner = None, 0, x.codes.data_ptr(), x.exponents.data_ptr(), x.shape[1]
    else:
        xs = _row_matrix(x, "x", n, dev, dtype=dout.dtype)
        at, codes, exponents, inner = x.data_ptr(), None, None, x.size(1)
    outer = dout.size(1)
    dtype = dout.dtype if dtype is None else dtype
    if dtype != dout.dtype and dtype != torch.float32:
        raise TypeError(f"dtype {dtype}: expected {dout.dtype} or fp32")
    out = _result(out, (rows.experts, inner, outer), "out", dtype, dev)
    kind = _kind(dout)
    side = GATHER_X if gather == "x" else GATHER_DOUT if gather else GATHER_NONE
    need = _grad_bytes(rows.tokens, rows.top_k, rows.experts, kind, side, inner, outer, codes is not None)
    work = dout.new_empty(need, dtype=torch.uint8)
    _call(dev, "dq_expert_matmul_grad", rows._io, at, xs, codes, exponents, dout.data_ptr(), ds, side,
          out.data_ptr(), kind, _kind(out), inner, outer, work.data_ptr(), need)
    return out


@_on_stream
def expert_sum(y, rows, residual=None, out=None):
    """Every token's rows added up, and its ``residual``: ``residual[t] + sum_j y[row[t,
    j]]`` (``dq_expert_sum``), [tokens, width].  Choices without an expert add nothing.
    It is the way back of the experts' outputs and the gradient of gathering.
    ``out`` may be ``residual``."""
    dev = _expert_rows(rows).device
    ys = _row_matrix(y, "y", rows.slots, dev)
    width, rs = y.size(1), 0
    if residual is not None:
        rs = _row_matrix(residual, "residual", rows.tokens, dev, width, y.dtype)
    out, os_ = _row_result(out, "out", rows.tokens, width, y)
    _call(dev, "dq_expert_sum", rows._io, y.data_ptr(), ys, _opt(residual), rs, out.data_ptr(), os_, _kind(y), width)
    return out


def _act(act, columns):
    """(number, width) of an activation over so many columns of u."""
    if act not in _ACTS:
        raise ValueError(f"act {act!r}: expected one of {sorted(_ACTS)}")
    if act == "swiglu" and columns % 2:
        raise ValueError(f"u: {columns} columns, expected gate and value halves")
    return _ACTS[act], columns // 2 if act == "swiglu" else columns


def _gates(gates, rows):
    if not isinstance(gates, torch.Tensor) or gates.shape != rows.row.shape:
        raise ValueError(f"gates: expected [{rows.tokens}, {rows.top_k}] of route()")
    return _tensor(gates, "gates", rows.device, dtype=torch.float32).data_ptr()


@_on_stream
def expert_act(u, gates, rows, act="swiglu", keep=False, dither=True, seed=1, rnd=0, worker=0, site=0, out=None):
    """The activation between the experts' products, weighted by the router's
    ``gates`` (``dq_expert_act``): with ``act="swiglu"``, ``u`` = (g, v) in two halves and
    ``gate * silu(g) * v``; with ``"relu"``, ``gate * max(u, 0)``.

    ``u`` is [tokens * top_k, columns].  With ``keep`` returns (a, kept): the rows of
    ``u`` are also kept in 8 bits, as :func:`keep8` would keep them with the same
    numbers, in the same pass where the width is a multiple of 32."""
    dev = _expert_rows(rows).device
    us = _row_matrix(u, "u", rows.slots, dev)
    columns = u.size(1)
    number, width = _act(act, columns)
    at = _gates(gates, rows)
    a, as_ = _row_result(out, "out", rows.slots, width, u)
    kept = codes = exponents = key = None
    if keep:
        key = _keep_key(dither, seed, rnd, worker, site, dev)
        kept = Kept8._made((rows.slots, columns), u)
        codes, exponents = kept.codes.data_ptr(), kept.exponents.data_ptr()
    _call(dev, "dq_expert_act", rows._io, number, u.data_ptr(), us, at, a.data_ptr(), as_, _kind(u), width, codes,
          exponents, key)
    return (a, kept) if keep else a


@_on_stream
def expert_act_backward(u, da, gates, rows, act="swiglu", du=None, dgates=None, a=None, again=True):
    """Gradient of :func:`expert_act`, from ``u`` or the :class:`Kept8` of it: returns
    (du, dgates, a).  ``a`` is the activation once more, from the same ``u``, for
    :func:`expert_matmul_grad` of the next product (None without ``again``).  ``du``,
    ``dgates`` and ``a`` may be given as buffers; the gates of slots without an expert
    get 0."""
    dev = _expert_rows(rows).device
    das = _row_matrix(da, "da", rows.slots, dev)
    if isinstance(u, Kept8):
        if u.codes.dim() != 2 or u.shape[0] != rows.slots or u.dtype != da.dtype or u.device != dev:
            raise ValueError(f"u: kept {tuple(u.shape)} {u.dtype} on {u.device}, expected [{rows.slots}, columns] "
                             f"{da.dtype} on {dev}")
        columns, at, us, codes, exponents = u.shape[1], None, 0, u.codes.data_ptr(), u.exponents.data_ptr()
    else:
        us = _row_matrix(u, "u", rows.slots, dev, dtype=da.dtype)
        columns, at, codes, exponents = u.size(1), u.data_ptr(), None, None
    number, width = _act(act, columns)
    if da.size(1) != width:
        raise ValueError(f"da: {da.size(1)} columns, expected {width}")
    g = _gates(gates, rows)
    du, dus = _row_result(du, "du", rows.slots, columns, da)
    dgates = gates.new_empty(gates.shape) if dgates is None else _result(dgates, gates.shape, "dgates", torch.float32, dev)
    as_ = 0
    if again or a is not None:
        a, as_ = _row_result(a, "a", rows.slots, width, da)
    _call(dev, "dq_expert_act_backward", rows._io, number, at, us, codes, exponents, da.data_ptr(), das, g,
          du.data_ptr(), dus, _opt(a), as_, dgates.data_ptr(), _kind(da), width)
    return du, dgates, a


class Plan:
    """One gradient-synchronisation round over ``n_workers`` virtual workers.

    Mirrors ``include/dq.h``: create -> options -> bind workspace -> stats (rank
    order) -> allocate -> reorder -> compress / hop -> finalize.
    """

    def __init__(self, n_coords, n_workers, topology=RING, avg_bits=5.0, seed=1, rnd=0,
                 rounding=STRATIFIED, device="cuda", timing=False, alloc=ALLOC_THRESHOLD, eps=None,
                 own=OWN_PACKED, streams=1, max_width=8):
        self.d = int(n_coords)
        self.n = int(n_workers)
        self.J = self.d // 256
        self.topology = int(topology)
        self.log2n = max(0, (self.n - 1).bit_length())
        self.own = int(own)
        if torch.device(device).type != "cuda":
            raise ValueError(f"the plan's workspace must be GPU memory, not {device}")
        h = C.c_void_p()
        _check(lib().dq_plan_create(self.d, self.n, self.topology, float(avg_bits), C.byref(h)),
               "dq_plan_create")
        self.h = h
        self.set(OPT_SEED, seed)
        self.set(OPT_ROUND, rnd)
        self.set(OPT_ROUNDING, rounding)
        self.set(OPT_TIMING, 1 if timing else 0)
        self.set(OPT_ALLOC, alloc)
        self.set(OPT_OWN, own)
        self.max_width = int(max_width)
        if self.max_width != 8:
            self.set(OPT_MAX_WIDTH, self.max_width)
        if eps is not None:
            _check(lib().dq_plan_set_f64(self.h, OPT_EPS, float(eps)), "dq_plan_set_f64")
        if streams != 1:
            with torch.cuda.device(torch.device(device)):   # the second stream lives on this device
                self.set(OPT_STREAMS, streams)
        nbytes = lib().dq_workspace_bytes(self.h)
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.device = self.workspace.device
        _check(lib().dq_plan_bind(self.h, _ptr(self.workspace), nbytes), "dq_plan_bind")
        lay = dq_layout()
        _check(lib().dq_workspace_layout(self.h, C.byref(lay)), "dq_workspace_layout")
        self.layout = {n: getattr(lay, n) for n, _ in dq_layout._fields_}

    def __del__(self):
        h = getattr(self, "h", None)
        if h is not None and h.value and _lib is not None:
            _lib.dq_plan_destroy(h)
            self.h = None

    def set(self, option, value):
        _check(lib().dq_plan_set_u64(self.h, int(option), int(value)), "dq_plan_set_u64")

    # ---- buffer sizes the schedule implies (for the argument checks) ---------
    def _m_compress(self):
        """m of the part a compress writes: the whole vector for one worker,
        a ring part (m = n), or a butterfly level-1 half (m = 2)."""
        return 1 if self.n == 1 else (self.n if self.topology == RING else 2)

    def _m_hop(self, step):
        """(m of the part a hop reads, m of each region it writes), or None
        for a step outside the schedule (the library rejects those)."""
        if self.n == 1:
            return None
        if self.topology == RING:
            return (self.n, self.n) if 1 <= step < self.n else None
        if not 1 <= step <= self.log2n:
            return None
        m = 1 << step
        return (m, 2 * m if step < self.log2n else m)

    def _check_hop(self, worker, step, region_in, local, kind, outs):
        ms = self._m_hop(int(step))
        dev = self.device
        _tensor(region_in, "region_in", dev)
        _tensor(local, "local", dev)
        for i, o in enumerate(outs):
            if o is not None:
                _tensor(o, f"out{i}", dev)
        if ms is None:
            return
        m_in, m_out = ms
        _tensor(region_in, "region_in", dev, min_bytes=self.region_bytes_max(m_in))
        if kind in (BF16, F32):
            _tensor(local, "local", dev, numel=self.d)
        elif kind == PACKED:
            _tensor(local, "local", dev, min_bytes=self.region_bytes_max(m_in))
        elif kind == F32_PARTIAL:
            _tensor(local, "local", dev, min_bytes=self.partial_bytes_max(m_in))
        two = self.topology == BUTTERFLY and step < self.log2n
        # own-fp32: the child this worker keeps is written as fp32 partial sums
        keep = (int(worker) >> (self.log2n - int(step) - 1)) & 1 if two and self.own == OWN_F32 else -1
        for h, o in enumerate(outs):
            if o is not None:
                need = self.partial_bytes_max(m_out) if h == keep else self.region_bytes_max(m_out)
                _tensor(o, f"out{h}", dev, min_bytes=need)

    def _check_grads(self, grads):
        if len(grads) != self.n:
            raise ValueError(f"{len(grads)} gradients for {self.n} workers")
        kind = _kind(grads[0])
        for w, g in enumerate(grads):
            _tensor(g, f"grads[{w}]", self.device, numel=self.d, dtype=grads[0].dtype)
        return kind

    # ---- stages --------------------------------------------------------
    def stats(self, worker, grad, stream=None):
        _tensor(grad, "grad", self.device, numel=self.d)
        _check(lib().dq_stats(self.h, int(worker), _ptr(grad), _kind(grad), _stream(stream)),
               "dq_stats")

    def allocate(self, stream=None):
        _check(lib().dq_allocate(self.h, _stream(stream)), "dq_allocate")

    def reorder(self, stream=None):
        _check(lib().dq_reorder(self.h, _stream(stream)), "dq_reorder")

    def compress(self, worker, step, grad, region_out, stream=None):
        _tensor(grad, "grad", self.device, numel=self.d)
        _tensor(region_out, "region_out", self.device, min_bytes=self.region_bytes_max(self._m_compress()))
        _check(lib().dq_compress(self.h, int(worker), int(step), _ptr(grad), _kind(grad),
                                 _ptr(region_out), _stream(stream)), "dq_compress")

    def hop(self, worker, step, region_in, local, out0, out1=None, stream=None, local_kind=None):
        """local_kind: F32_PARTIAL for the own fp32 partial sums (OWN_F32);
        otherwise taken from the tensor's dtype."""
        kind = _kind(local) if local_kind is None else int(local_kind)
        self._check_hop(worker, step, region_in, local, kind, (out0, out1))
        _check(lib().dq_hop(self.h, int(worker), int(step), _ptr(region_in), _ptr(local),
                            kind, _ptr(out0), None if out1 is None else _ptr(out1),
                            _stream(stream)), "dq_hop")

    def hop_finalize(self, worker, step, region_in, local, region_out, out, stream=None, local_kind=None):
        kind = _kind(local) if local_kind is None else int(local_kind)
        self._check_hop(worker, step, region_in, local, kind, (region_out,))
        _tensor(out, "out", self.device, min_bytes=4 * self.d, dtype=torch.float32)
        _check(lib().dq_hop_finalize(self.h, int(worker), int(step), _ptr(region_in), _ptr(local), kind,
                                     _ptr(region_out), _ptr(out), _stream(stream)), "dq_hop_finalize")

    def finalize(self, part, region, out, stream=None):
        _tensor(region, "region", self.device, min_bytes=self.region_bytes_max(self.n))
        _tensor(out, "out", self.device, min_bytes=4 * self.d, dtype=torch.float32)
        _check(lib().dq_finalize(self.h, int(part), _ptr(region), _ptr(out), _stream(stream)),
               "dq_finalize")

    def final_part(self, worker):
        return int(lib().dq_final_part(self.h, int(worker)))

    # ---- whole round -----------------------------------------------------
    def region_bytes_max(self, m):
        return int(lib().dq_region_bytes_max(self.h, int(m)))

    def partial_bytes_max(self, m):
        return int(lib().dq_partial_bytes_max(self.h, int(m)))

    def new_region(self, m, device="cuda"):
        return torch.zeros(self.region_bytes_max(m), dtype=torch.uint8, device=device)

    def arena_bytes(self):
        return int(lib().dq_arena_bytes(self.h))

    def _round_buffers(self, grads, out, arena, arena_bytes):
        kind = self._check_grads(grads)
        if arena is None:
            arena = torch.empty(max(1, arena_bytes), dtype=torch.uint8, device=self.device)
        if out is None:
            out = torch.empty(self.d, dtype=torch.float32, device=self.device)
        _tensor(arena, "arena", self.device)
        _tensor(out, "out", self.device, min_bytes=4 * self.d, dtype=torch.float32)
        ptrs = (C.c_void_p * self.n)(*[g.data_ptr() for g in grads])
        return kind, out, arena, arena.numel() * arena.element_size(), ptrs

    def allreduce(self, grads, out=None, arena=None, stream=None):
        kind, out, arena, nbytes, ptrs = self._round_buffers(grads, out, arena, self.arena_bytes())
        _check(lib().dq_allreduce(self.h, ptrs, kind, _ptr(arena), nbytes, _ptr(out),
                                  _stream(stream)), "dq_allreduce")
        return out

    def allreduce_noalloc(self, grads, out, stream=None):
        """dq_allreduce_noalloc: the round in the library's static scratch
        (binds the plan there)."""
        kind = self._check_grads(grads)
        _tensor(out, "out", self.device, min_bytes=4 * self.d, dtype=torch.float32)
        ptrs = (C.c_void_p * self.n)(*[g.data_ptr() for g in grads])
        _check(lib().dq_allreduce_noalloc(self.h, ptrs, kind, _ptr(out), _stream(stream)),
               "dq_allreduce_noalloc")
        return out

    def mxfp8_allreduce(self, grads, out=None, arena=None, stream=None):
        kind, out, arena, nbytes, ptrs = self._round_buffers(
            grads, out, arena, int(lib().dq_mxfp8_arena_bytes(self.h)))
        _check(lib().dq_mxfp8_allreduce(self.h, ptrs, kind, _ptr(arena), nbytes, _ptr(out),
                                        _stream(stream)), "dq_mxfp8_allreduce")
        return out

    def mx_allreduce(self, fmt, grads, out=None, arena=None, stream=None):
        kind, out, arena, nbytes, ptrs = self._round_buffers(
            grads, out, arena, int(lib().dq_mx_arena_bytes(self.h)))
        _check(lib().dq_mx_allreduce(self.h, int(fmt), ptrs, kind, _ptr(arena), nbytes, _ptr(out),
                                     _stream(stream)), "dq_mx_allreduce")
        return out

    # ---- inspection ------------------------------------------------------
    def info(self, stream=None):
        i = dq_info()
        rc = lib().dq_get_info(self.h, C.byref(i), _stream(stream))
        if rc not in (DQ_OK, DQ_ENONFINITE):
            _check(rc, "dq_get_info")
        counts = list(i.class_counts) + ([i.class_count16] if self.max_width == 16 else [])
        return {"rho_bits": i.rho_bits, "rho": i.rho, "t12": i.t12, "t24": i.t24, "t48": i.t48,
                "t816": i.t816, "class_counts": counts, "budget_bits": i.budget_bits,
                "used_bits": i.used_bits, "achieved_bits": i.achieved_bits,
                "nonfinite": bool(i.nonfinite), "status": rc}

    def timing(self):
        t = dq_timing()
        _check(lib().dq_timing_read(self.h, C.byref(t)), "dq_timing_read")
        return {k: {"ms": t.ms[i], "launches": t.launches[i], "coords": t.coords[i]}
                for i, k in enumerate(KERNEL_KINDS)}

    def _view(self, name, dtype, count):
        off = self.layout[name]
        nbytes = count * torch.empty(0, dtype=dtype).element_size()
        return self.workspace[off:off + nbytes].view(dtype)

    def stats_arrays(self):
        return self._view("sum", torch.float32, self.J), self._view("sumsq", torch.float32, self.J)

    def widths(self):
        return self._view("widths", torch.uint8, self.J)

    def perm(self):
        return self._view("perm", torch.int32, self.J), self._view("inv", torch.int32, self.J)

    def mu_stream(self):
        return self._view("mu_stream", torch.float32, self.J)
