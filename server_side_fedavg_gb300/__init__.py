"""Server-side FedAvg aggregation on one GB300: Python binding of libfedavg.so.

Thin ctypes marshalling over the C ABI in include/fedavg.h; every function
has the C name and raises FedAvgError on a negative status.  All device work
happens in the library's CUDA kernels: there is no Python or CPU compute path,
and importing the binding without the built library fails loudly.

Pointers may be given as ints, as objects with .data_ptr() (torch tensors) or
as numpy arrays (host memory); streams as ints or objects with .cuda_stream.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libfedavg.so")

FA_OK = 0
FA_ERR_ARG = -1
FA_ERR_RANGE = -2
FA_ERR_DTYPE = -3
FA_ERR_WEIGHT = -4
FA_ERR_INCOMPLETE = -5
FA_ERR_STATE = -6
FA_ERR_NOMEM = -7
FA_ERR_CUDA = -8
FA_ERR_TIMEOUT = -9
FA_ERR_INTERNAL = -10

FA_F32 = 0
FA_BF16 = 1
FA_KEY_FLAT = -1
FA_FLAT_OUT = 1
FA_STAGE_HOST = 2
FA_COMPENSATED = 4
FA_TEST_WAIT_EXPIRES = 0x80000000
FA_NOALLOC_MAX_ELEMS = 1 << 22

FA_ACT_NONE = 0
FA_ACT_RELU = 1
FA_ACT_GELU = 2
FA_ACT_SILU = 3
FA_TRANS_A = 1
FA_TRANS_B = 2
FA_DISTILL_MAX_CLIENTS = 16
FA_DISTILL_MAX_TOPK = 2048
FA_ROTARY_INTERLEAVED = 1
FA_ROTARY_INVERSE = 2
FA_ROTARY_MAX_DIM = 512
FA_ROTARY_PLAIN = 0
FA_ROTARY_LINEAR = 1
FA_ROTARY_BASE = 2
FA_ROTARY_BANDED = 3
FA_NORM_MAX_CHANNELS = 8192
FA_ORTHO_NESTEROV = 1
FA_ORTHO_MAX_STEPS = 32

ACTS = {"none": FA_ACT_NONE, "relu": FA_ACT_RELU, "gelu": FA_ACT_GELU, "silu": FA_ACT_SILU,
        FA_ACT_NONE: FA_ACT_NONE, FA_ACT_RELU: FA_ACT_RELU, FA_ACT_GELU: FA_ACT_GELU,
        FA_ACT_SILU: FA_ACT_SILU}

SCALINGS = {"none": FA_ROTARY_PLAIN, "linear": FA_ROTARY_LINEAR, "base": FA_ROTARY_BASE, "banded": FA_ROTARY_BANDED,
            FA_ROTARY_PLAIN: FA_ROTARY_PLAIN, FA_ROTARY_LINEAR: FA_ROTARY_LINEAR, FA_ROTARY_BASE: FA_ROTARY_BASE,
            FA_ROTARY_BANDED: FA_ROTARY_BANDED}

DTYPES = {"f32": FA_F32, "bf16": FA_BF16, FA_F32: FA_F32, FA_BF16: FA_BF16}


class fa_key(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("numel", ctypes.c_uint64)]


class fa_opts(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("ring_slots", ctypes.c_uint32),
                ("slot_bytes", ctypes.c_uint64), ("timeout_ms", ctypes.c_uint32),
                ("flags", ctypes.c_uint32)]


class fa_stats(ctypes.Structure):
    _fields_ = [("kernel_launches", ctypes.c_uint64), ("client_bytes", ctypes.c_uint64),
                ("h2d_bytes", ctypes.c_uint64), ("d2h_bytes", ctypes.c_uint64),
                ("chunks", ctypes.c_uint64)]


class fa_partition_opts(ctypes.Structure):
    _fields_ = [("w_time", ctypes.c_double), ("w_energy", ctypes.c_double),
                ("ema_alpha", ctypes.c_double), ("deadband", ctypes.c_double)]


class fa_work_opts(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("timeout_ms", ctypes.c_uint32),
                ("workspace_bytes", ctypes.c_uint64), ("flags", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class fa_work_stats(ctypes.Structure):
    _fields_ = [("kernel_launches", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64)]


class fa_product_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype_in", ctypes.c_int32),
                ("dtype_out", ctypes.c_int32), ("act", ctypes.c_int32), ("reserved", ctypes.c_uint32),
                ("m", ctypes.c_uint64), ("n", ctypes.c_uint64), ("k", ctypes.c_uint64),
                ("a", ctypes.c_void_p), ("lda", ctypes.c_uint64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_uint64), ("bias", ctypes.c_void_p),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_uint64),
                ("out", ctypes.c_void_p), ("ldo", ctypes.c_uint64), ("pre", ctypes.c_void_p),
                ("alpha", ctypes.c_double), ("beta", ctypes.c_double)]


class fa_product_backward_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype_in", ctypes.c_int32),
                ("dtype_dout", ctypes.c_int32), ("dtype_grad", ctypes.c_int32), ("act", ctypes.c_int32),
                ("m", ctypes.c_uint64), ("n", ctypes.c_uint64), ("k", ctypes.c_uint64),
                ("a", ctypes.c_void_p), ("lda", ctypes.c_uint64),
                ("b", ctypes.c_void_p), ("ldb", ctypes.c_uint64),
                ("dout", ctypes.c_void_p), ("ldd", ctypes.c_uint64),
                ("pre", ctypes.c_void_p), ("ldp", ctypes.c_uint64),
                ("d_a", ctypes.c_void_p), ("ldda", ctypes.c_uint64),
                ("d_b", ctypes.c_void_p), ("lddb", ctypes.c_uint64),
                ("d_bias", ctypes.c_void_p), ("alpha", ctypes.c_double)]


class fa_distill_client(ctypes.Structure):
    _fields_ = [("index", ctypes.c_void_p), ("value", ctypes.c_void_p), ("topk", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("weight", ctypes.c_double)]


class fa_distill_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("n_clients", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("dtype_value", ctypes.c_int32), ("rows", ctypes.c_uint64), ("vocab", ctypes.c_uint64),
                ("logits", ctypes.c_void_p), ("ld", ctypes.c_uint64), ("clients", ctypes.c_void_p),
                ("temperature", ctypes.c_double), ("row_weight", ctypes.c_void_p),
                ("loss", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("ldg", ctypes.c_uint64)]


class fa_rotary_part(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32), ("batch_stride", ctypes.c_uint64),
                ("token_stride", ctypes.c_uint64), ("head_stride", ctypes.c_uint64),
                ("out_batch_stride", ctypes.c_uint64), ("out_token_stride", ctypes.c_uint64),
                ("out_head_stride", ctypes.c_uint64)]


class fa_rotary_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("head_dim", ctypes.c_uint32), ("rotary_dim", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("batch", ctypes.c_uint64), ("seq", ctypes.c_uint64), ("turns", ctypes.c_void_p),
                ("position", ctypes.c_void_p), ("first", ctypes.c_int64), ("scale", ctypes.c_double),
                ("q", fa_rotary_part), ("k", fa_rotary_part)]


class fa_group_norm_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("dtype_param", ctypes.c_int32), ("act", ctypes.c_int32), ("reserved", ctypes.c_uint32),
                ("n", ctypes.c_uint64), ("positions", ctypes.c_uint64), ("channels", ctypes.c_uint64),
                ("groups", ctypes.c_uint64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_uint64),
                ("step_x", ctypes.c_uint64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_uint64),
                ("step_y", ctypes.c_uint64), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("eps", ctypes.c_double), ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p)]


class fa_group_norm_backward_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype", ctypes.c_int32),
                ("dtype_param", ctypes.c_int32), ("act", ctypes.c_int32), ("reserved", ctypes.c_uint32),
                ("n", ctypes.c_uint64), ("positions", ctypes.c_uint64), ("channels", ctypes.c_uint64),
                ("groups", ctypes.c_uint64), ("x", ctypes.c_void_p), ("ldx", ctypes.c_uint64),
                ("step_x", ctypes.c_uint64), ("dout", ctypes.c_void_p), ("ldd", ctypes.c_uint64),
                ("step_d", ctypes.c_uint64), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("rstd", ctypes.c_void_p), ("dx", ctypes.c_void_p),
                ("lddx", ctypes.c_uint64), ("step_dx", ctypes.c_uint64), ("d_gamma", ctypes.c_void_p),
                ("d_beta", ctypes.c_void_p)]


class fa_orthogonalise_args(ctypes.Structure):
    _fields_ = [("size", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("dtype_in", ctypes.c_int32),
                ("dtype_out", ctypes.c_int32), ("steps", ctypes.c_uint32), ("reserved", ctypes.c_uint32),
                ("count", ctypes.c_uint64), ("rows", ctypes.c_uint64), ("cols", ctypes.c_uint64),
                ("update", ctypes.c_void_p), ("ldu", ctypes.c_uint64), ("step_u", ctypes.c_uint64),
                ("momentum", ctypes.c_void_p), ("ldm", ctypes.c_uint64), ("step_m", ctypes.c_uint64),
                ("momentum_out", ctypes.c_void_p), ("ldmo", ctypes.c_uint64), ("step_mo", ctypes.c_uint64),
                ("residual", ctypes.c_void_p), ("ldr", ctypes.c_uint64), ("step_r", ctypes.c_uint64),
                ("out", ctypes.c_void_p), ("ldo", ctypes.c_uint64), ("step_o", ctypes.c_uint64),
                ("mu", ctypes.c_double), ("eps", ctypes.c_double), ("alpha", ctypes.c_double), ("beta", ctypes.c_double),
                ("a", ctypes.c_double), ("b", ctypes.c_double), ("c", ctypes.c_double)]


class FedAvgError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.detail = detail
        super().__init__(f"{status} ({fa_strerror(status)}): {detail}")


_lib = None


def lib():
    """The loaded libfedavg.so; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(LIB_PATH)
        i32, u32, u64, i64, f64, vp = (ctypes.c_int32, ctypes.c_uint32, ctypes.c_uint64,
                                       ctypes.c_int64, ctypes.c_double, ctypes.c_void_p)
        L.fa_open.argtypes = [ctypes.POINTER(fa_key), u32, i32, i32, u32, ctypes.POINTER(fa_opts),
                              ctypes.POINTER(vp)]
        L.fa_accumulate.argtypes = [vp, u32, f64, i64, u64, vp, u64, vp]
        L.fa_accumulate_batch.argtypes = [vp, u32, ctypes.POINTER(u32), ctypes.POINTER(f64), i64,
                                          u64, ctypes.POINTER(vp), u64, vp]
        L.fa_accumulate_keys.argtypes = [vp, u32, f64, u32, ctypes.POINTER(i64), ctypes.POINTER(u64),
                                         ctypes.POINTER(vp), ctypes.POINTER(u64), vp]
        L.fa_accumulate_final.argtypes = [vp, u32, f64, i64, u64, vp, u64, ctypes.POINTER(vp), vp]
        L.fa_finalize.argtypes = [vp, ctypes.POINTER(vp), vp]
        L.fa_reduce_resident.argtypes = [vp, u32, ctypes.POINTER(u32), ctypes.POINTER(f64),
                                         ctypes.POINTER(vp), ctypes.POINTER(vp), vp]
        L.fa_finalize_apply.argtypes = [vp, ctypes.POINTER(vp), ctypes.POINTER(vp), f64, vp]
        L.fa_reduce_subsets.argtypes = [vp, u32, ctypes.POINTER(u32), ctypes.POINTER(f64),
                                        ctypes.POINTER(vp), ctypes.POINTER(u32), ctypes.POINTER(i64),
                                        ctypes.POINTER(vp), vp]
        L.fa_reset.argtypes = [vp]
        L.fa_close.argtypes = [vp]
        L.fa_key_total.argtypes = [vp, u32, ctypes.POINTER(f64), ctypes.POINTER(u32)]
        L.fa_sync.argtypes = [vp]
        L.fa_get_stats.argtypes = [vp, ctypes.POINTER(fa_stats)]
        L.fa_aggregate_noalloc.argtypes = [u32, ctypes.POINTER(f64), ctypes.POINTER(vp), u64, i32, i32,
                                           vp, vp]
        L.fa_aggregate_noalloc.restype = i32
        L.fa_aggregate_noalloc_status.argtypes = [vp, u32]
        L.fa_aggregate_noalloc_status.restype = i32
        L.fa_partition_plan.argtypes = [u32, vp, vp, vp, vp, vp, ctypes.POINTER(fa_partition_opts), vp]
        L.fa_partition_plan.restype = i32
        L.fa_work_open.argtypes = [ctypes.POINTER(fa_work_opts), ctypes.POINTER(vp)]
        L.fa_work_close.argtypes = [vp]
        L.fa_work_sync.argtypes = [vp]
        L.fa_work_get_stats.argtypes = [vp, ctypes.POINTER(fa_work_stats)]
        L.fa_work_last_error.argtypes = [vp]
        L.fa_work_last_error.restype = ctypes.c_char_p
        L.fa_product.argtypes = [vp, ctypes.POINTER(fa_product_args), vp]
        L.fa_product_backward.argtypes = [vp, ctypes.POINTER(fa_product_backward_args), vp]
        L.fa_rotary_turns.argtypes = [ctypes.c_uint32, ctypes.c_double, ctypes.c_int32, ctypes.c_double, ctypes.c_double,
                                      ctypes.c_double, ctypes.c_double, ctypes.POINTER(ctypes.c_uint64)]
        L.fa_orthogonalise.argtypes = [vp, ctypes.POINTER(fa_orthogonalise_args), vp]
        L.fa_rotary.argtypes = [vp, ctypes.POINTER(fa_rotary_args), vp]
        L.fa_group_norm.argtypes = [vp, ctypes.POINTER(fa_group_norm_args), vp]
        L.fa_group_norm_backward.argtypes = [vp, ctypes.POINTER(fa_group_norm_backward_args), vp]
        L.fa_distill_loss.argtypes = [vp, ctypes.POINTER(fa_distill_args), vp]
        L.fa_distill_grad.argtypes = [vp, ctypes.POINTER(fa_distill_args), vp]
        L.fa_strerror.argtypes = [i32]
        L.fa_strerror.restype = ctypes.c_char_p
        L.fa_last_error.argtypes = [vp]
        L.fa_last_error.restype = ctypes.c_char_p
        for name in ("fa_open", "fa_accumulate", "fa_accumulate_batch", "fa_accumulate_keys",
                     "fa_accumulate_final", "fa_finalize",
                     "fa_finalize_apply", "fa_reduce_resident", "fa_reduce_subsets", "fa_reset",
                     "fa_close", "fa_key_total", "fa_sync", "fa_get_stats", "fa_work_open", "fa_work_close",
                     "fa_work_sync", "fa_work_get_stats", "fa_product", "fa_product_backward",
                     "fa_distill_loss", "fa_distill_grad", "fa_rotary_turns", "fa_rotary", "fa_group_norm",
                     "fa_group_norm_backward", "fa_orthogonalise"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def _ptr(x) -> int:
    if x is None:
        return 0
    of = getattr(x, "data_ptr", None)      # a tensor, most often
    if of is not None:
        return of()
    if isinstance(x, int):
        return x
    if hasattr(x, "ctypes"):
        return int(x.ctypes.data)
    raise TypeError(f"cannot take a pointer of {type(x)!r}")


def _stream(s) -> int:
    if s is None:
        return 0
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(status: int, ctx=None):
    if status != FA_OK:
        detail = fa_last_error(ctx) if ctx is not None else ""
        raise FedAvgError(status, detail)


def fa_strerror(status: int) -> str:
    return lib().fa_strerror(status).decode()


def fa_last_error(ctx) -> str:
    r = lib().fa_last_error(ctx)
    return r.decode() if r else ""


def fa_open(layout, dtype_in, dtype_out, max_clients, ring_slots=0, slot_bytes=0,
            timeout_ms=0, flags=0):
    """layout: list of (name, numel).  Returns an opaque context handle."""
    n = len(layout)
    keys = (fa_key * max(n, 1))()
    names = []
    for i, (name, numel) in enumerate(layout):
        b = name.encode() if isinstance(name, str) else name
        names.append(b)
        keys[i].name = b
        keys[i].numel = int(numel)
    opts = fa_opts(ctypes.sizeof(fa_opts), ring_slots, slot_bytes, timeout_ms, flags)
    ctx = ctypes.c_void_p()
    _check(lib().fa_open(keys, n, DTYPES[dtype_in], DTYPES[dtype_out], max_clients,
                         ctypes.byref(opts), ctypes.byref(ctx)))
    return ctx


def fa_accumulate(ctx, client_id, weight_nk, key, offset_elems, chunk, len_elems, stream=None):
    _check(lib().fa_accumulate(ctx, client_id, float(weight_nk), key, offset_elems, _ptr(chunk),
                               len_elems, _stream(stream)), ctx)


def out_array(outs):
    """A C array of output pointers (per-key outputs, None allowed, or one flat output)."""
    return (ctypes.c_void_p * max(len(outs), 1))(*[_ptr(o) for o in outs])


def fa_accumulate_final(ctx, client_id, weight_nk, key, offset_elems, chunk, len_elems, outs,
                        stream=None):
    """outs: as for fa_finalize, or an array made by out_array (reused across calls)."""
    ps = outs if isinstance(outs, ctypes.Array) else out_array(outs)
    _check(lib().fa_accumulate_final(ctx, client_id, float(weight_nk), key, offset_elems, _ptr(chunk),
                                     len_elems, ps, _stream(stream)), ctx)


def _same_length(**seqs):
    n = {k: len(v) for k, v in seqs.items()}
    if len(set(n.values())) > 1:
        raise ValueError("lengths differ: " + ", ".join(f"{k}={v}" for k, v in n.items()))


def fa_accumulate_batch(ctx, client_ids, weights, key, offset_elems, chunks, len_elems,
                        stream=None):
    _same_length(client_ids=client_ids, weights=weights, chunks=chunks)
    J = len(client_ids)
    ids = (ctypes.c_uint32 * J)(*client_ids)
    ws = (ctypes.c_double * J)(*[float(w) for w in weights])
    ps = (ctypes.c_void_p * J)(*[_ptr(c) for c in chunks])
    _check(lib().fa_accumulate_batch(ctx, J, ids, ws, key, offset_elems, ps, len_elems,
                                     _stream(stream)), ctx)


def fa_accumulate_keys(ctx, client_id, weight_nk, keys, offsets, chunks, lens, stream=None):
    """One client's chunks in one call: chunk i is `lens[i]` elements at `offsets[i]` of
    key `keys[i]` (FA_KEY_FLAT: of the flat layout), read from `chunks[i]` (pointers as
    ints or a uint64 array, or tensors / arrays).  Sequences or NumPy arrays."""
    import numpy as np
    ks = np.ascontiguousarray(keys, dtype=np.int64)
    os_ = np.ascontiguousarray(offsets, dtype=np.uint64)
    ls = np.ascontiguousarray(lens, dtype=np.uint64)
    if isinstance(chunks, np.ndarray):
        ps = np.ascontiguousarray(chunks, dtype=np.uint64)
    else:
        ps = np.fromiter((_ptr(c) for c in chunks), dtype=np.uint64, count=len(chunks))
    n = ks.size
    if not (os_.size == ps.size == ls.size == n):
        raise ValueError("keys, offsets, chunks and lens must have the same length")
    _check(lib().fa_accumulate_keys(
        ctx, client_id, float(weight_nk), n, ks.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
        os_.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
        ps.ctypes.data_as(ctypes.POINTER(ctypes.c_void_p)),
        ls.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)), _stream(stream)), ctx)


def fa_finalize(ctx, outs, stream=None):
    """outs: list of per-key outputs (None allowed for keys that will not be written),
    or a one-element list with the flat output when opened with FA_FLAT_OUT."""
    ps = (ctypes.c_void_p * max(len(outs), 1))(*[_ptr(o) for o in outs])
    _check(lib().fa_finalize(ctx, ps, _stream(stream)), ctx)


def fa_finalize_apply(ctx, bases, outs, server_lr=1.0, stream=None):
    """Delta rounds: outs = round(bases + server_lr * weighted mean); outs may be bases."""
    bs = (ctypes.c_void_p * max(len(bases), 1))(*[_ptr(b) for b in bases])
    ps = (ctypes.c_void_p * max(len(outs), 1))(*[_ptr(o) for o in outs])
    _check(lib().fa_finalize_apply(ctx, bs, ps, float(server_lr), _stream(stream)), ctx)


def fa_reduce_resident(ctx, client_ids, weights, flat_updates, outs, stream=None):
    """Whole round from resident full updates (one flat buffer per client) straight to outs."""
    _same_length(client_ids=client_ids, weights=weights, flat_updates=flat_updates)
    J = len(client_ids)
    ids = (ctypes.c_uint32 * J)(*client_ids)
    ws = (ctypes.c_double * J)(*[float(w) for w in weights])
    ps = (ctypes.c_void_p * J)(*[_ptr(x) for x in flat_updates])
    os_ = (ctypes.c_void_p * max(len(outs), 1))(*[_ptr(o) for o in outs])
    _check(lib().fa_reduce_resident(ctx, J, ids, ws, ps, os_, _stream(stream)), ctx)


def subset_table(client_keys):
    """Marshal per-client key lists once: (n_keys uint32 array, concatenated int64 keys)."""
    import numpy as np
    nk = np.ascontiguousarray([len(k) for k in client_keys], dtype=np.uint32)
    ks = np.ascontiguousarray(np.concatenate([np.asarray(k, np.int64) for k in client_keys])
                              if len(client_keys) else np.zeros(0, np.int64), dtype=np.int64)
    return nk, ks


def fa_reduce_subsets(ctx, client_ids, weights, client_bufs, client_keys, outs, stream=None):
    """A round of key subsets resident in device memory, straight to outs: client j's
    buffer client_bufs[j] holds its keys client_keys[j] (a list of key ids) packed back to
    back in that order.  client_keys may also be a subset_table(...) result."""
    import numpy as np
    if isinstance(client_keys, tuple) and len(client_keys) == 2 and isinstance(client_keys[0], np.ndarray):
        nk, ks = client_keys
        _same_length(client_ids=client_ids, weights=weights, client_bufs=client_bufs, n_keys=nk)
    else:
        _same_length(client_ids=client_ids, weights=weights, client_bufs=client_bufs,
                     client_keys=client_keys)
        nk, ks = subset_table(client_keys)
    J = len(client_ids)
    ids = (ctypes.c_uint32 * J)(*client_ids)
    ws = (ctypes.c_double * J)(*[float(w) for w in weights])
    ps = (ctypes.c_void_p * J)(*[_ptr(b) for b in client_bufs])
    os_ = (ctypes.c_void_p * max(len(outs), 1))(*[_ptr(o) for o in outs])
    _check(lib().fa_reduce_subsets(ctx, J, ids, ws, ps, nk.ctypes.data_as(ctypes.POINTER(ctypes.c_uint32)),
                                   ks.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)), os_,
                                   _stream(stream)), ctx)


def fa_reset(ctx):
    _check(lib().fa_reset(ctx), ctx)


def fa_close(ctx):
    _check(lib().fa_close(ctx))


def fa_key_total(ctx, key):
    s = ctypes.c_double()
    n = ctypes.c_uint32()
    _check(lib().fa_key_total(ctx, key, ctypes.byref(s), ctypes.byref(n)), ctx)
    return s.value, n.value


def fa_sync(ctx):
    _check(lib().fa_sync(ctx), ctx)


def fa_get_stats(ctx) -> dict:
    st = fa_stats()
    _check(lib().fa_get_stats(ctx, ctypes.byref(st)), ctx)
    return {f: getattr(st, f) for f, _ in fa_stats._fields_}


def fa_aggregate_noalloc(weights, chunks, numel, dtype_in, dtype_out, out, stream=None):
    """One tensor, all clients resident, no allocation: the running sum lives in a
    fixed 16 MiB array of the library (see include/fedavg.h).  For callers that must
    not have a library allocate device memory."""
    _same_length(weights=weights, chunks=chunks)
    J = len(chunks)
    ws = (ctypes.c_double * max(J, 1))(*[float(w) for w in weights])
    ps = (ctypes.c_void_p * max(J, 1))(*[_ptr(c) for c in chunks])
    _check(lib().fa_aggregate_noalloc(J, ws, ps, numel, DTYPES[dtype_in], DTYPES[dtype_out],
                                      _ptr(out), _stream(stream)))


def fa_aggregate_noalloc_status(stream=None, timeout_ms=0):
    """Raises FedAvgError (FA_ERR_INTERNAL) if a device-side wait gave up in an
    fa_aggregate_noalloc call on the current device since the last check."""
    _check(lib().fa_aggregate_noalloc_status(_stream(stream), timeout_ms))


def fa_partition_plan(time_s, energy_j, samples, ema_tau=None, ema_eps=None, w_time=1.0,
                      w_energy=0.0, ema_alpha=0.5, deadband=0.05):
    """Next round's sample counts; returns (new_samples, ema_tau, ema_eps) as lists."""
    import numpy as np
    m = len(samples)
    t = np.ascontiguousarray(time_s, dtype=np.float64)
    e = np.ascontiguousarray(energy_j, dtype=np.float64)
    n = np.ascontiguousarray(samples, dtype=np.uint64)
    tau = np.full(m, np.nan) if ema_tau is None else np.array(ema_tau, dtype=np.float64)
    eps = np.full(m, np.nan) if ema_eps is None else np.array(ema_eps, dtype=np.float64)
    out = np.zeros(m, dtype=np.uint64)
    o = fa_partition_opts(w_time, w_energy, ema_alpha, deadband)
    _check(lib().fa_partition_plan(m, t.ctypes.data, e.ctypes.data, n.ctypes.data, tau.ctypes.data,
                                   eps.ctypes.data, ctypes.byref(o), out.ctypes.data))
    return [int(v) for v in out], tau.tolist(), eps.tolist()


# ---------------------------------------------------------------- training operators
def _check_work(status: int, work):
    if status != FA_OK:
        raise FedAvgError(status, fa_work_last_error(work))


def fa_work_last_error(work) -> str:
    r = lib().fa_work_last_error(work)
    return r.decode() if r else ""


def fa_work_open(timeout_ms=0, workspace_bytes=0, flags=0):
    """A work handle on the current device: what fa_product, fa_product_backward,
    fa_distill_loss and fa_distill_grad share (workspace, error word, order of calls)."""
    opts = fa_work_opts(ctypes.sizeof(fa_work_opts), timeout_ms, workspace_bytes, flags, 0)
    work = ctypes.c_void_p()
    _check(lib().fa_work_open(ctypes.byref(opts), ctypes.byref(work)))
    return work


def fa_work_close(work):
    _check_work(lib().fa_work_close(work), work)


def fa_work_sync(work):
    """Wait (bounded) for the handle's work; raises what its kernels reported."""
    _check_work(lib().fa_work_sync(work), work)


def fa_work_get_stats(work) -> dict:
    st = fa_work_stats()
    _check_work(lib().fa_work_get_stats(work, ctypes.byref(st)), work)
    return {f: getattr(st, f) for f, _ in fa_work_stats._fields_}


def fa_product(work, m, n, k, a, lda, b, ldb, out, ldo, dtype_in, dtype_out, trans_a=False,
               trans_b=False, alpha=1.0, bias=None, act="none", residual=None, ldr=0, beta=1.0,
               pre=None, stream=None):
    """out[m,n] = act(alpha * op(a) . op(b) + bias) + beta * residual.  a is [m,k] (trans_a:
    stored [k,m]), b is [k,n] (trans_b: stored [n,k], a linear layer's weight); `pre`, if
    given, receives the value before the activation (stride ldo)."""
    args = fa_product_args(ctypes.sizeof(fa_product_args), bool(trans_a) | bool(trans_b) << 1,
                           DTYPES[dtype_in], DTYPES[dtype_out], ACTS[act], 0, m, n, k, _ptr(a), lda,
                           _ptr(b), ldb, _ptr(bias), _ptr(residual), ldr, _ptr(out), ldo, _ptr(pre),
                           alpha, beta)
    _check_work(lib().fa_product(work, args, _stream(stream)), work)


def fa_product_backward(work, m, n, k, a, lda, b, ldb, dout, ldd, d_a, ldda, d_b, lddb, dtype_in,
                        dtype_dout, dtype_grad, trans_a=False, trans_b=False, alpha=1.0, act="none",
                        pre=None, ldp=0, d_bias=None, stream=None):
    """Gradients of fa_product with respect to a, b and the bias (None: not wanted), from
    dout and -- unless act is "none" -- the kept `pre`; each stored like its operand."""
    args = fa_product_backward_args(
        ctypes.sizeof(fa_product_backward_args), bool(trans_a) | bool(trans_b) << 1, DTYPES[dtype_in],
        DTYPES[dtype_dout], DTYPES[dtype_grad], ACTS[act], m, n, k, _ptr(a), lda, _ptr(b), ldb,
        _ptr(dout), ldd, _ptr(pre), ldp, _ptr(d_a), ldda, _ptr(d_b), lddb, _ptr(d_bias), alpha)
    _check_work(lib().fa_product_backward(work, args, _stream(stream)), work)


# the element types of lists, by name: what is read as int32, as fp32 and as bf16 bits; the types
# seen to be right are kept (None: a plain address)
_INDEX_TYPES, _VALUE_TYPES = ("int32", "uint32"), {FA_F32: ("float32",), FA_BF16: ("bfloat16", "uint16", "int16")}
_index_seen, _value_seen = {None}, {FA_F32: {None}, FA_BF16: {None}}


def _check_types(arrays, names, seen, what):
    for x in arrays:
        dt = getattr(x, "dtype", None)
        if dt not in seen:
            if str(dt).rsplit(".", 1)[-1] not in names:
                raise TypeError(f"{what}, not {dt}")
            seen.add(dt)


def distill_lists(index, value, topk, weights, dtype_value="f32"):
    """The clients' top-logit lists for fa_distill_loss and fa_distill_grad, marshalled once:
    per client its index array [rows, topk] (int32, negative: unused; torch.topk gives int64:
    TypeError), its value array, its topk and its weight (sample count).  The arrays are kept
    alive by the result."""
    n = len(index)
    if not n == len(value) == len(topk) == len(weights):
        _same_length(index=index, value=value, topk=topk, weights=weights)
    kind = DTYPES[dtype_value]
    _check_types(index, _INDEX_TYPES, _index_seen, "an index array is int32")
    _check_types(value, _VALUE_TYPES[kind], _value_seen[kind], f"a value array is of dtype_value, {dtype_value}")
    arr = (fa_distill_client * max(n, 1))(*[(_ptr(i), _ptr(v), t, 0, w)
                                            for i, v, t, w in zip(index, value, topk, weights)])
    return arr, n, kind, (list(index), list(value))


def _distill_args(rows, vocab, logits, ld, dtype, lists, temperature, row_weight, loss, lse, grad, ldg):
    return fa_distill_args(ctypes.sizeof(fa_distill_args), lists[1], DTYPES[dtype], lists[2], rows, vocab,
                           _ptr(logits), ld, ctypes.addressof(lists[0]), temperature, _ptr(row_weight),
                           _ptr(loss), _ptr(lse), _ptr(grad), ldg)


def fa_distill_loss(work, rows, vocab, logits, ld, dtype, lists, temperature, row_weight, loss,
                    lse=None, stream=None):
    """Per-row distillation loss of the student's logits from the clients' lists (a
    distill_lists result), and optionally the rows' log sum exp(z / T) for the gradient."""
    args = _distill_args(rows, vocab, logits, ld, dtype, lists, temperature, row_weight, loss, lse, None, 0)
    _check_work(lib().fa_distill_loss(work, args, _stream(stream)), work)


def fa_distill_grad(work, rows, vocab, logits, ld, dtype, lists, temperature, row_weight, lse, loss, grad,
                    ldg, stream=None):
    """Gradient of the rows' losses with respect to the logits (grad may be logits itself).
    lse: kept by fa_distill_loss, or None to compute it here; loss: written unless None."""
    args = _distill_args(rows, vocab, logits, ld, dtype, lists, temperature, row_weight, loss, lse, grad, ldg)
    _check_work(lib().fa_distill_grad(work, args, _stream(stream)), work)


# ---------------------------------------------------------------- layers of the student
def rotary_turns(rotary_dim, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=32.0):
    """A model's rotary frequencies for fa_rotary, made once (fa_rotary_turns): base^(-2 i /
    rotary_dim) per pair, for long contexts divided by `factor` ("linear"), taken from a larger
    base ("base"), or divided where a pair turns fewer than low..high times over the first
    `context` positions ("banded")."""
    turns = (ctypes.c_uint64 * max(1, rotary_dim // 2))()
    _check(lib().fa_rotary_turns(rotary_dim, base, SCALINGS[scaling], factor, context, low, high, turns))
    return turns


def fa_rotary(work, batch, seq, head_dim, turns, dtype, q, q_heads, q_out, k=None, k_heads=0, k_out=None,
              position=None, first=0, layout="half", inverse=False, scale=1.0, q_strides=None,
              q_out_strides=None, k_strides=None, k_out_strides=None, stream=None):
    """Rotary positions of q and k, [batch, seq, heads, head_dim] unless strides = (batch, token,
    head) in elements are given.  turns: a rotary_turns result; its length sets rotary_dim.
    position: int32 [batch, seq], negative in padding (left as it is), or None for first + s.
    layout "half" pairs (i, i + rotary_dim / 2), "interleaved" (2 i, 2 i + 1).  inverse: the
    gradient's direction.  An output may be its input itself."""
    dt = getattr(position, "dtype", None)
    if dt not in _position_seen:
        _check_types((position,), ("int32",), _position_seen, "position is int32")
    flags = _LAYOUTS.get(layout)
    if flags is None:
        raise ValueError(f"layout is 'half' or 'interleaved', not {layout!r}")
    if q_strides is None or (q_out_strides is None and q_out is not q):
        row = q_heads * head_dim
        q_own = (seq * row, row, head_dim)
    if k_strides is None or (k_out_strides is None and k_out is not k):
        row = k_heads * head_dim
        k_own = (seq * row, row, head_dim)
    if q_strides is None:
        q_strides = q_own
    if q_out_strides is None:
        q_out_strides = q_strides if q_out is q else q_own
    if k_strides is None:
        k_strides = k_own
    if k_out_strides is None:
        k_out_strides = k_strides if k_out is k else k_own
    args = fa_rotary_args(
        _ROTARY_SIZE, flags | FA_ROTARY_INVERSE if inverse else flags, DTYPES[dtype], head_dim, 2 * len(turns), 0, batch, seq,
        ctypes.addressof(turns), _ptr(position), first, scale,
        (_ptr(q), _ptr(q_out), q_heads, 0, *q_strides, *q_out_strides),
        (_ptr(k), _ptr(k_out), k_heads, 0, *k_strides, *k_out_strides))
    _check_work(lib().fa_rotary(work, args, _stream(stream)), work)


_LAYOUTS = {"half": 0, "interleaved": FA_ROTARY_INTERLEAVED}
_ROTARY_SIZE = ctypes.sizeof(fa_rotary_args)
_position_seen = {None}


def fa_group_norm(work, n, positions, channels, groups, x, y, dtype, gamma=None, beta=None, dtype_param="f32",
                  act="none", eps=1e-5, mean=None, rstd=None, ldx=None, step_x=0, ldy=None, step_y=0, stream=None):
    """Group norm with an activation of x [n, positions, channels] (channels last), to y, which may
    be x.  mean and rstd [n, groups] fp32 receive the statistics for the backward call."""
    args = fa_group_norm_args(
        ctypes.sizeof(fa_group_norm_args), 0, DTYPES[dtype], DTYPES[dtype_param], ACTS[act], 0, n, positions, channels,
        groups, _ptr(x), channels if ldx is None else ldx, step_x, _ptr(y), channels if ldy is None else ldy, step_y,
        _ptr(gamma), _ptr(beta), eps, _ptr(mean), _ptr(rstd))
    _check_work(lib().fa_group_norm(work, args, _stream(stream)), work)


def fa_group_norm_backward(work, n, positions, channels, groups, x, dout, dx, dtype, gamma, beta, dtype_param, mean, rstd,
                           act="none", d_gamma=None, d_beta=None, ldx=None, step_x=0, ldd=None, step_d=0, lddx=None,
                           step_dx=0, stream=None):
    """Gradients of fa_group_norm from dout, x and the kept mean and rstd: dx (which may be x or
    dout), and d_gamma and d_beta [channels] unless None."""
    args = fa_group_norm_backward_args(
        ctypes.sizeof(fa_group_norm_backward_args), 0, DTYPES[dtype], DTYPES[dtype_param], ACTS[act], 0, n, positions,
        channels, groups, _ptr(x), channels if ldx is None else ldx, step_x, _ptr(dout), channels if ldd is None else ldd,
        step_d, _ptr(gamma), _ptr(beta), _ptr(mean), _ptr(rstd), _ptr(dx), channels if lddx is None else lddx, step_dx,
        _ptr(d_gamma), _ptr(d_beta))
    _check_work(lib().fa_group_norm_backward(work, args, _stream(stream)), work)


# ---------------------------------------------------------------- the weight step
def fa_orthogonalise(work, count, rows, cols, update, out, dtype_in, dtype_out, steps=5,
                     coefficients=(3.4445, -4.7750, 2.0315), eps=1e-7, momentum=None, momentum_out=None, mu=0.0,
                     nesterov=False, residual=None, alpha=1.0, beta=1.0, ldu=None, step_u=0, ldm=None, step_m=0, ldmo=None,
                     step_mo=0, ldr=None, step_r=0, ldo=None, step_o=0, stream=None):
    """out = alpha * orthogonalised(update with momentum) + beta * residual, for `count` matrices
    [rows, cols] that lie ld... and step_... elements apart (a row, a matrix; by default one after
    the other).  momentum and momentum_out are fp32, and may be one buffer."""
    args = fa_orthogonalise_args(
        ctypes.sizeof(fa_orthogonalise_args), bool(nesterov), DTYPES[dtype_in], DTYPES[dtype_out], steps, 0, count, rows, cols,
        _ptr(update), cols if ldu is None else ldu, step_u, _ptr(momentum), cols if ldm is None else ldm, step_m,
        _ptr(momentum_out), cols if ldmo is None else ldmo, step_mo, _ptr(residual), cols if ldr is None else ldr, step_r,
        _ptr(out), cols if ldo is None else ldo, step_o, mu, eps, alpha, beta, *coefficients)
    _check_work(lib().fa_orthogonalise(work, args, _stream(stream)), work)
