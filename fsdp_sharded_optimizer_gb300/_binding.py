"""Thin ctypes binding of ``libzero.so`` (the C ABI declared in include/zero.h).

Argument marshalling only: torch tensors become device pointers and host
pointer tables, the caller's current torch stream becomes the ``cudaStream_t``,
and a negative return code becomes an exception.  Every step of the path runs
in the library's CUDA kernels; there is no CPU or PyTorch fallback, and
importing this module fails loudly if the library is missing.

Per-rank buffers may be given as a list of tensors (one per rank) or as the
rows of one 2-D tensor (row k = rank k).  Buffers may be CUDA memory or pinned
host memory, which the kernels read and write in place (no staging copy).  bf16 buffers may be ``torch.bfloat16``
or ``torch.int16``/``torch.uint16`` bit patterns.
"""
import ctypes as C
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libzero.so")

ZERO_OK, ZERO_EINVAL, ZERO_EALIGN, ZERO_ECUDA, ZERO_ETIMEOUT = 0, -1, -2, -3, -4
ZERO_MAX_RANKS = 64
ZERO_DEFAULT_ALIGN = 64
ZERO_CHUNK_ELEMS = 13107200  # fused-step launch granularity (include/zero.h)


class ZeroError(RuntimeError):
    """A negative return code of the C ABI."""

    def __init__(self, fn, code):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (fn, strerror(code), code))


class zero_hparams_t(C.Structure):
    _fields_ = [("lr", C.c_double), ("beta1", C.c_double), ("beta2", C.c_double),
                ("eps", C.c_double), ("weight_decay", C.c_double), ("step", C.c_int64)]


class zero_unit_t(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("n_params", "n_padded", "shard_len", "offset",
                                         "shard_offset", "param_offset", "pad")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}

    def __repr__(self):
        return "zero_unit_t(%s)" % ", ".join("%s=%d" % kv for kv in self.as_dict().items())


class zero_bytes_t(C.Structure):
    _fields_ = [(n, C.c_double) for n in ("weight_bytes", "grad_bytes", "optim_bytes",
                                          "state_bytes", "comm_volume", "comm_sent_elems",
                                          "comm_sent_bytes", "hbm_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class zero_op_t(C.Structure):
    _fields_ = [("kind", C.c_int32), ("stream", C.c_int32), ("unit", C.c_int32), ("arg", C.c_int32)]


class zero_regen_t(C.Structure):
    _fields_ = [("seed", C.c_uint64), ("sigma", C.c_double), ("outliers", C.c_int32)]


ZERO_OP_RECORD, ZERO_OP_WAIT, ZERO_OP_GATHER = 1, 2, 3
ZERO_OP_REDUCE_SCATTER, ZERO_OP_REGEN, ZERO_OP_USE = 4, 5, 6
OP_NAMES = {1: "record", 2: "wait", 3: "gather", 4: "reduce_scatter", 5: "regen", 6: "use",
            7: "norm", 8: "clip_coef", 9: "accumulate"}


class zero_clip_t(C.Structure):
    _fields_ = [("max_norm", C.c_double), ("scratch", C.c_void_p), ("scratch_bytes", C.c_int64),
                ("norm_coef", C.c_void_p), ("grad_shard", C.c_void_p)]


ZERO_TYPE_BF16, ZERO_TYPE_F32, ZERO_TYPE_I32, ZERO_TYPE_I64 = 1, 2, 3, 4
ZERO_NORM_RMS, ZERO_NORM_LAYER = 0, 1


class zero_block_norm_t(C.Structure):
    _fields_ = [("n_rows", C.c_int64), ("dim", C.c_int64), ("rows_per_gate", C.c_int64),
                ("kind", C.c_int32), ("post_norm", C.c_int32), ("pre_norm", C.c_int32),
                ("act_type", C.c_int32), ("res_type", C.c_int32), ("param_type", C.c_int32),
                ("gate_type", C.c_int32), ("eps", C.c_double), ("residual_scale", C.c_double),
                ("branch_scale", C.c_double)]


class zero_block_norm_grads_t(C.Structure):
    _fields_ = [("dgate", C.c_void_p), ("dpost_weight", C.c_void_p), ("dpost_bias", C.c_void_p),
                ("dpre_weight", C.c_void_p), ("dpre_bias", C.c_void_p),
                ("dgate_type", C.c_int32), ("grad_type", C.c_int32)]


class zero_distill_t(C.Structure):
    _fields_ = [("n_rows", C.c_int64), ("vocab", C.c_int64), ("logits_stride", C.c_int64),
                ("top", C.c_int32), ("logits_type", C.c_int32), ("teacher_type", C.c_int32),
                ("id_type", C.c_int32), ("label_type", C.c_int32), ("temperature", C.c_double),
                ("ce_weight", C.c_double), ("kl_weight", C.c_double)]


def clip_args(max_norm, scratch, norm_coef, grad_shard=None):
    """A zero_clip_t for zero3_step from device tensors (scratch of
    zero_clip_scratch_bytes(), norm_coef of 2 floats, and optionally the fp32
    gradient shard storage, N x S_total, that the norm pass fills and the
    updates read)."""
    table = _rows(grad_shard, 4, "grad_shard")[0] if grad_shard is not None else None
    c = zero_clip_t(float(max_norm), scratch.data_ptr(), scratch.numel() * scratch.element_size(),
                    norm_coef.data_ptr(),
                    C.cast(table, C.c_void_p).value if table is not None else None)
    # kept alive with the struct (a graph holds these addresses)
    c.tensors = (scratch, norm_coef, grad_shard, table)
    return c

# name -> (restype, argtypes); the same names as include/zero.h
_P, _I32, _I64, _U64, _F64 = C.c_void_p, C.c_int32, C.c_int64, C.c_uint64, C.c_double
SIGNATURES = {
    "zero_layout": (C.c_int, [_P, _I32, _I32, _I32, _P, _P]),
    "zero_step_stage12": (C.c_int, [_I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P]),
    "zero3_gather_unit": (C.c_int, [_P, _I32, _P, _P, _P]),
    "zero3_reduce_scatter_unit": (C.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "zero_state_bytes": (C.c_int, [_I64, _I32, _I32, _I32, _P]),
    "zero_clip_scratch_bytes": (C.c_int64, []),
    "zero_grad_sqnorm": (C.c_int, [_I32, _I64, _P, _I32, _P, _I64, _P]),
    "zero_clip_coef": (C.c_int, [_P, _I64, _F64, _P, _P]),
    "zero_step_stage12_clip": (C.c_int, [_I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P,
                                         _P]),
    "zero3_reduce_scatter_unit_clip": (C.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
    "zero_grad_reduce_sqnorm": (C.c_int, [_I32, _I64, _P, _P, _I32, _P, _I64, _P]),
    "zero3_update_unit_reduced": (C.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
    "zero_step_stage12_reduced": (C.c_int, [_I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P,
                                            _P]),
    "zero_clip_coef_units_noalloc": (C.c_int, [_P, _I32, _I32, _P, _F64, _P, _P, _P]),
    "zero_grad_nonfinite": (C.c_int, [_I32, _I64, _P, _P, _I32, _P]),
    "zero_step_stage12_checked": (C.c_int, [_I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64, _P,
                                            _P]),
    "zero3_reduce_scatter_unit_checked": (C.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P, _P]),
    "zero3_step_checked": (C.c_int, [_P, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                     _I32, _P, _P, _P]),
    "zero_step_stage12_f32grads": (C.c_int, [_I32, _I32, _I64, _P, _P, _P, _P, _P, _P, _I64,
                                             _P]),
    "zero3_reduce_scatter_unit_f32grads": (C.c_int, [_P, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "zero_gen_grads_unit_f32": (C.c_int, [_U64, _I64, _F64, _I32, _P, _I32, _P, _P]),
    "zero2_accumulate": (C.c_int, [_I32, _I64, _P, _P, _I32, _P]),
    "zero2_step_accumulated": (C.c_int, [_I32, _I64, _P, _P, _I32, _P, _P, _P, _P, _P, _P]),
    # from unit, n_from, src table, to unit, n_to, dst table, stream
    "zero_reshard_f32": (C.c_int, [_P, _I32, _P, _P, _I32, _P, _P]),
    # unit, n_ranks, unit grads, grad_acc storage, first, stream
    "zero3_accumulate_unit": (C.c_int, [_P, _I32, _P, _P, _I32, _P]),
    # unit, n_ranks, unit grads, grad_acc storage, micro_batches, master, m, v, shards, hp, stream
    "zero3_reduce_scatter_unit_accumulated": (C.c_int, [_P, _I32, _P, _P, _I32, _P, _P, _P, _P,
                                                        _P, _P]),
    "zero3_plan": (C.c_int, [_I32, _I32, _I32, _I32, _P, _I32, _P]),
    "zero3_plan_microbatch": (C.c_int, [_I32, _I32, _I32, _I32, _P, _I32, _P]),
    # units, n_units, n_ranks, grads, grad_acc, micro_batch, micro_batches, master, m, v,
    # shards, full_a, full_b, hp, reshard_after_forward, main stream, side stream
    "zero3_step_microbatch": (C.c_int, [_P, _I32, _I32, _P, _P, _I32, _I32, _P, _P, _P, _P, _P,
                                        _P, _P, _I32, _P, _P]),
    # units, n_units, n_ranks, grads, resident, master, m, v, shards, full_a, full_b, hp,
    # regen, clip, reshard_after_forward, main stream, side stream
    "zero3_step": (C.c_int, [_P, _I32, _I32, _P, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32,
                             _P, _P]),
    # units, n_units, n_ranks, grads, master, m, v, shards, full_a, full_b, hp,
    # reshard_after_forward, main stream, side stream
    "zero3_step_f32grads": (C.c_int, [_P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P,
                                      _P]),
    # units, n_units, n_ranks, grads, master, m, v, shards, full_a, full_b, hp, clip,
    # reshard_after_forward, capture stream, side stream, out handle
    "zero3_graph_create": (C.c_int, [_P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32,
                                     _P, _P, _P]),
    # units, n_units, n_ranks, grads (fp32), master, m, v, shards, full_a, full_b, hp,
    # reshard_after_forward, capture stream, side stream, out handle
    "zero3_graph_create_f32grads": (C.c_int, [_P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P,
                                              _I32, _P, _P, _P]),
    "zero3_graph_launch": (C.c_int, [_P, _P, _P]),
    "zero3_graph_destroy": (C.c_int, [_P]),
    "zero_gen_grads_unit": (C.c_int, [_U64, _I64, _F64, _I32, _P, _I32, _P, _P]),
    "zero_gen_master": (C.c_int, [_U64, _F64, _P, _I32, _I32, _P, _P]),
    "zero_cast_bf16": (C.c_int, [_P, _P, _I64, _P]),
    # table, type, vocab, dim, ids, type, n_tokens, scale, out, type, stream
    "zero_embed_forward": (C.c_int, [_P, _I32, _I64, _I64, _P, _I32, _I64, _F64, _P, _I32, _P]),
    "zero_embed_scratch_bytes": (_I64, [_I64, _I64, _I64]),
    # dout, type, ids, type, n_tokens, scale, dtable, type, vocab, dim, accumulate, scratch,
    # scratch bytes, stream
    "zero_embed_backward": (C.c_int, [_P, _I32, _P, _I32, _I64, _F64, _P, _I32, _I64, _I64, _I32,
                                      _P, _I64, _P]),
    # norm, x, branch, gate, post weight and bias, pre weight and bias, y, u, stream
    "zero_block_norm_forward": (C.c_int, [_P] * 11),
    "zero_block_norm_scratch_bytes": (_I64, [_I64, _I64, _I64]),
    # norm, dy, du, y, branch, gate, post weight and bias, pre weight, dx, dbranch, grads,
    # scratch, scratch bytes, stream
    "zero_block_norm_backward": (C.c_int, [_P] * 13 + [_I64, _P]),
    # distill, logits, teacher logits, teacher ids, labels, row weight, ce, kl, stream
    "zero_distill_forward": (C.c_int, [_P] * 9),
    # ..., ce, kl, dlogits, dlogits stride, stream
    "zero_distill_forward_backward": (C.c_int, [_P] * 9 + [_I64, _P]),
    "zero_stream_wait": (C.c_int, [_P, _I64]),
    "zero_strerror": (C.c_char_p, [C.c_int]),
}


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libzero.so is not built (%s). Run __graft_entry__.build() or "
            "python -m fsdp_sharded_optimizer_gb300.build; there is no fallback path." % LIB_PATH)
    lib = C.CDLL(LIB_PATH)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def strerror(code):
    return lib.zero_strerror(code).decode()


def _check(fn, rc):
    if rc != ZERO_OK:
        raise ZeroError(fn, rc)


def _addressable(t):
    """CUDA memory, or pinned host memory: the GPU reads and writes pinned host
    memory directly (unified addressing; over NVLink-C2C on Grace-Blackwell)."""
    return t.is_cuda or (t.device.type == "cpu" and t.is_pinned())


def _rows(x, dtype_bytes, what):
    """A host table of device-addressable pointers from a list of tensors or a 2-D tensor."""
    rows = list(x) if isinstance(x, (list, tuple)) else [x[i] for i in range(x.shape[0])]
    for t in rows:
        if not _addressable(t):
            raise ValueError("%s must be CUDA memory or pinned host memory" % what)
        if t.element_size() != dtype_bytes:
            raise ValueError("%s: expected %d-byte elements, got %s" % (what, dtype_bytes, t.dtype))
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % what)
    return (C.c_void_p * len(rows))(*[t.data_ptr() for t in rows]), rows


def _dev(t, dtype_bytes, what):
    if not _addressable(t) or t.element_size() != dtype_bytes or not t.is_contiguous():
        raise ValueError("%s must be a contiguous CUDA or pinned host tensor of %d-byte elements"
                         % (what, dtype_bytes))
    return C.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return C.c_void_p(s.cuda_stream)


def hparams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, step=1):
    return zero_hparams_t(lr, beta1, beta2, eps, weight_decay, step)


# ------------------------------------------------------------------ host calls
def zero_layout(unit_sizes, n_ranks, align_elems=ZERO_DEFAULT_ALIGN):
    """Layout of each unit and the total padded length (host only)."""
    sizes = (C.c_int64 * len(unit_sizes))(*[int(s) for s in unit_sizes])
    units = (zero_unit_t * len(unit_sizes))()
    total = C.c_int64()
    _check("zero_layout", lib.zero_layout(sizes, len(unit_sizes), n_ranks, align_elems, units,
                                          C.byref(total)))
    return list(units), total.value


def zero_state_bytes(n_params, n_ranks, stage, K=12):
    out = zero_bytes_t()
    _check("zero_state_bytes", lib.zero_state_bytes(int(n_params), n_ranks, stage, K, C.byref(out)))
    return out.as_dict()


def zero_stream_wait(stream=None, timeout_ms=10_000):
    """Wait for the stream with a wall-clock limit; raises ZeroError(ZERO_ETIMEOUT)."""
    _check("zero_stream_wait", lib.zero_stream_wait(_stream(stream), int(timeout_ms)))


# ------------------------------------------------------------------ device calls
def zero_step_stage12(stage, grads, master, m, v, params_bf16, hp, bucket_elems=0, stream=None):
    """The fused ZeRO-1/2 step: grads (N x P' bf16), master/m/v (N x S fp32),
    params_bf16 (P' bf16), all on the device."""
    g, grows = _rows(grads, 2, "grads")
    w, wrows = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    n_padded = grows[0].numel()
    _check("zero_step_stage12", lib.zero_step_stage12(
        stage, len(grows), n_padded, g, w, mm, vv, _dev(params_bf16, 2, "params_bf16"),
        C.byref(hp), int(bucket_elems), _stream(stream)))


def zero3_gather_unit(unit, shard_bf16, full_unit, stream=None):
    s, rows = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_gather_unit", lib.zero3_gather_unit(
        C.byref(unit), len(rows), s, _dev(full_unit, 2, "full_unit"), _stream(stream)))


def zero3_reduce_scatter_unit(unit, unit_grads, master, m, v, shard_bf16, hp, stream=None):
    g, grows = _rows(unit_grads, 2, "unit_grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_reduce_scatter_unit", lib.zero3_reduce_scatter_unit(
        C.byref(unit), len(grows), g, w, mm, vv, s, C.byref(hp), _stream(stream)))


def zero_clip_scratch_bytes():
    return lib.zero_clip_scratch_bytes()


def zero_grad_sqnorm(grads, scratch, accumulate=False, stream=None):
    """Add the squared norm of the averaged gradient of one buffer into the
    per-block partials in `scratch` (a device tensor of zero_clip_scratch_bytes())."""
    g, rows = _rows(grads, 2, "grads")
    _check("zero_grad_sqnorm", lib.zero_grad_sqnorm(
        len(rows), rows[0].numel(), g, 1 if accumulate else 0, C.c_void_p(scratch.data_ptr()),
        scratch.numel() * scratch.element_size(), _stream(stream)))


def zero_clip_coef(scratch, max_norm, norm_coef, stream=None):
    """norm_coef (device float[2]) <- (global norm, clip coefficient)."""
    _check("zero_clip_coef", lib.zero_clip_coef(
        C.c_void_p(scratch.data_ptr()), scratch.numel() * scratch.element_size(), float(max_norm),
        _dev(norm_coef, 4, "norm_coef"), _stream(stream)))


def zero_step_stage12_clip(stage, grads, master, m, v, params_bf16, hp, norm_coef, bucket_elems=0,
                           stream=None):
    g, grows = _rows(grads, 2, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    _check("zero_step_stage12_clip", lib.zero_step_stage12_clip(
        stage, len(grows), grows[0].numel(), g, w, mm, vv, _dev(params_bf16, 2, "params_bf16"),
        C.byref(hp), int(bucket_elems), _dev(norm_coef, 4, "norm_coef"), _stream(stream)))


def zero_grad_reduce_sqnorm(grads, grad_shard, scratch, accumulate=False, stream=None):
    """zero_grad_sqnorm that also stores the mean gradient to the owners' fp32
    shards: grads (N x P' bf16), grad_shard (N x S fp32)."""
    g, rows = _rows(grads, 2, "grads")
    gs, srows = _rows(grad_shard, 4, "grad_shard")
    if len(srows) != len(rows):
        raise ValueError("grad_shard needs one row per rank")
    _check("zero_grad_reduce_sqnorm", lib.zero_grad_reduce_sqnorm(
        len(rows), rows[0].numel(), g, gs, 1 if accumulate else 0, C.c_void_p(scratch.data_ptr()),
        scratch.numel() * scratch.element_size(), _stream(stream)))


def zero_step_stage12_reduced(stage, grad_shard, master, m, v, params_bf16, hp, norm_coef=None,
                              bucket_elems=0, stream=None):
    """The ZeRO-1/2 step from the reduced fp32 gradient shards (N x S), clipped
    by norm_coef (device float[2]) when given."""
    gs, rows = _rows(grad_shard, 4, "grad_shard")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    _check("zero_step_stage12_reduced", lib.zero_step_stage12_reduced(
        stage, len(rows), params_bf16.numel(), gs, w, mm, vv, _dev(params_bf16, 2, "params_bf16"),
        C.byref(hp), int(bucket_elems),
        _dev(norm_coef, 4, "norm_coef") if norm_coef is not None else None, _stream(stream)))


def zero3_update_unit_reduced(unit, grad_shard, master, m, v, shard_bf16, hp, norm_coef=None,
                              stream=None):
    """One unit's ZeRO-3 update from the fp32 gradient shard storage (N x S_total),
    clipped by norm_coef when given."""
    gs, rows = _rows(grad_shard, 4, "grad_shard")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    sh, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_update_unit_reduced", lib.zero3_update_unit_reduced(
        C.byref(unit), len(rows), gs, w, mm, vv, sh, C.byref(hp),
        _dev(norm_coef, 4, "norm_coef") if norm_coef is not None else None, _stream(stream)))


def zero3_reduce_scatter_unit_clip(unit, unit_grads, master, m, v, shard_bf16, hp, norm_coef,
                                   stream=None):
    g, grows = _rows(unit_grads, 2, "unit_grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_reduce_scatter_unit_clip", lib.zero3_reduce_scatter_unit_clip(
        C.byref(unit), len(grows), g, w, mm, vv, s, C.byref(hp), _dev(norm_coef, 4, "norm_coef"),
        _stream(stream)))


def zero_step_stage12_f32grads(stage, grads, master, m, v, params_bf16, hp, bucket_elems=0,
                               stream=None):
    """The fused ZeRO-1/2 step with fp32 rank gradients (N x P' fp32)."""
    g, grows = _rows(grads, 4, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    _check("zero_step_stage12_f32grads", lib.zero_step_stage12_f32grads(
        stage, len(grows), grows[0].numel(), g, w, mm, vv, _dev(params_bf16, 2, "params_bf16"),
        C.byref(hp), int(bucket_elems), _stream(stream)))


def zero3_reduce_scatter_unit_f32grads(unit, unit_grads, master, m, v, shard_bf16, hp,
                                       stream=None):
    g, grows = _rows(unit_grads, 4, "unit_grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_reduce_scatter_unit_f32grads", lib.zero3_reduce_scatter_unit_f32grads(
        C.byref(unit), len(grows), g, w, mm, vv, s, C.byref(hp), _stream(stream)))


def zero_gen_grads_unit_f32(seed, step, sigma, outliers, unit, unit_grads, stream=None):
    g, rows = _rows(unit_grads, 4, "unit_grads")
    _check("zero_gen_grads_unit_f32", lib.zero_gen_grads_unit_f32(
        int(seed), int(step), float(sigma), int(outliers), C.byref(unit), len(rows), g,
        _stream(stream)))


def zero2_accumulate(grads, grad_acc, first, stream=None):
    """One earlier micro-batch of ZeRO-2 gradient accumulation: grad_acc
    (N x S fp32, per owner) = (first ? 0 : grad_acc) + the micro-batch mean."""
    g, grows = _rows(grads, 2, "grads")
    a, _ = _rows(grad_acc, 4, "grad_acc")
    _check("zero2_accumulate", lib.zero2_accumulate(len(grows), grows[0].numel(), g, a,
                                                    1 if first else 0, _stream(stream)))


def zero2_step_accumulated(grads, grad_acc, micro_batches, master, m, v, params_bf16, hp,
                           stream=None):
    """The last micro-batch fused with the ZeRO-2 step: g = (grad_acc + mean) / m."""
    g, grows = _rows(grads, 2, "grads")
    a, _ = _rows(grad_acc, 4, "grad_acc")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    _check("zero2_step_accumulated", lib.zero2_step_accumulated(
        len(grows), grows[0].numel(), g, a, int(micro_batches), w, mm, vv,
        _dev(params_bf16, 2, "params_bf16"), C.byref(hp), _stream(stream)))


def zero_reshard_f32(from_unit, src, to_unit, dst, stream=None):
    """One unit's fp32 state (rows: ranks, laid out like master) re-laid from
    len(src) to len(dst) ranks."""
    a, _ = _rows(src, 4, "src")
    b, _ = _rows(dst, 4, "dst")
    n_from = len(src) if isinstance(src, (list, tuple)) else src.shape[0]
    n_to = len(dst) if isinstance(dst, (list, tuple)) else dst.shape[0]
    _check("zero_reshard_f32", lib.zero_reshard_f32(C.byref(from_unit), n_from, a,
                                                    C.byref(to_unit), n_to, b, _stream(stream)))


def zero3_accumulate_unit(unit, unit_grads, grad_acc, first, stream=None):
    """One earlier micro-batch of a ZeRO-3 unit: grad_acc (N x S_total fp32,
    laid out like master) at the unit's offset = (first ? 0 : it) + the mean."""
    g, grows = _rows(unit_grads, 2, "unit_grads")
    a, _ = _rows(grad_acc, 4, "grad_acc")
    _check("zero3_accumulate_unit", lib.zero3_accumulate_unit(
        C.byref(unit), len(grows), g, a, 1 if first else 0, _stream(stream)))


def zero3_reduce_scatter_unit_accumulated(unit, unit_grads, grad_acc, micro_batches, master, m, v,
                                          shard_bf16, hp, stream=None):
    """The unit's last micro-batch fused with its update: g = (grad_acc + mean) / m."""
    g, grows = _rows(unit_grads, 2, "unit_grads")
    a, _ = _rows(grad_acc, 4, "grad_acc")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_reduce_scatter_unit_accumulated", lib.zero3_reduce_scatter_unit_accumulated(
        C.byref(unit), len(grows), g, a, int(micro_batches), w, mm, vv, s, C.byref(hp),
        _stream(stream)))


def zero_grad_nonfinite(grads, counts, reset=True, stream=None):
    """counts (device int32/uint32[N]) (+)= per-rank number of non-finite bf16 gradients."""
    g, rows = _rows(grads, 2, "grads")
    _check("zero_grad_nonfinite", lib.zero_grad_nonfinite(
        len(rows), rows[0].numel(), g, _dev(counts, 4, "counts"), 1 if reset else 0,
        _stream(stream)))


def _flags(nonfinite_ranks):
    """The finite check's output: a device tensor of two 32-bit words (or more)."""
    if nonfinite_ranks.numel() * nonfinite_ranks.element_size() < 8:
        raise ValueError("nonfinite_ranks needs two 32-bit words")
    return _dev(nonfinite_ranks, 4, "nonfinite_ranks")


def zero_step_stage12_checked(stage, grads, master, m, v, params_bf16, hp, nonfinite_ranks,
                              bucket_elems=0, stream=None):
    """zero_step_stage12 with the pre-reduction finite check fused in: bit r of
    nonfinite_ranks (device int32/uint32[2]; word r // 32) is OR-ed in when rank
    r's gradient holds an infinity or a NaN.  Same results, no extra traffic."""
    g, grows = _rows(grads, 2, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    _check("zero_step_stage12_checked", lib.zero_step_stage12_checked(
        stage, len(grows), grows[0].numel(), g, w, mm, vv, _dev(params_bf16, 2, "params_bf16"),
        C.byref(hp), int(bucket_elems), _flags(nonfinite_ranks), _stream(stream)))


def zero3_reduce_scatter_unit_checked(unit, unit_grads, master, m, v, shard_bf16, hp,
                                      nonfinite_ranks, stream=None):
    """zero3_reduce_scatter_unit with the fused finite check (as
    zero_step_stage12_checked)."""
    g, grows = _rows(unit_grads, 2, "unit_grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    _check("zero3_reduce_scatter_unit_checked", lib.zero3_reduce_scatter_unit_checked(
        C.byref(unit), len(grows), g, w, mm, vv, s, C.byref(hp), _flags(nonfinite_ranks),
        _stream(stream)))


ZERO_NOALLOC_MAX_UNITS = 1024


def zero_clip_coef_units_noalloc(units, grads, max_norm, norm_coef, unit_norms=None, stream=None):
    """Global-norm clip coefficient over `units` (rank r's gradients of every
    unit concatenated in grads[r]) using the library's fixed internal scratch
    instead of caller memory: for callers that cannot allocate device memory.
    norm_coef (device float[2]) <- (norm, coef); unit_norms (optional device
    float[len(units)]) <- each unit's norm.  At most ZERO_NOALLOC_MAX_UNITS units.
    The C entry point has no lengths to check, so the sizes are checked here,
    before anything is launched: every gradient row must cover every unit."""
    n_rows = len(grads) if isinstance(grads, (list, tuple)) else grads.shape[0]
    need = max((int(u.offset) + int(u.n_padded) for u in units), default=0)
    for r in range(n_rows):
        if grads[r].numel() < need:
            raise ValueError("zero_clip_coef_units_noalloc: grads[%d] holds %d elements, the "
                             "units need %d" % (r, grads[r].numel(), need))
    if norm_coef.numel() < 2:
        raise ValueError("zero_clip_coef_units_noalloc: norm_coef needs 2 floats")
    if unit_norms is not None and unit_norms.numel() < len(units):
        raise ValueError("zero_clip_coef_units_noalloc: unit_norms needs %d floats, has %d"
                         % (len(units), unit_norms.numel()))
    g, rows = _rows(grads, 2, "grads")
    arr = (zero_unit_t * len(units))(*units)
    un = _dev(unit_norms, 4, "unit_norms") if unit_norms is not None else None
    _check("zero_clip_coef_units_noalloc", lib.zero_clip_coef_units_noalloc(
        arr, len(units), len(rows), g, float(max_norm), _dev(norm_coef, 4, "norm_coef"), un,
        _stream(stream)))


def zero3_plan(n_units, regen=False, clip=False, reshard_after_forward=True):
    """The operations of one ZeRO-3 step (host only): a list of
    (kind name, stream 0=main/1=side, unit, arg)."""
    cap = 18 * n_units + 8  # the header's bound (16 n + 7 with regeneration and clipping) and more
    ops = (zero_op_t * cap)()
    n = C.c_int32()
    _check("zero3_plan", lib.zero3_plan(n_units, 1 if regen else 0, 1 if clip else 0,
                                        1 if reshard_after_forward else 0, ops, cap, C.byref(n)))
    return [(OP_NAMES[o.kind], o.stream, o.unit, o.arg) for o in ops[:n.value]]


def zero3_plan_microbatch(n_units, micro_batch, micro_batches, reshard_after_forward=True):
    """The operations of one micro-batch of a ZeRO-3 step with gradient
    accumulation (host only), as zero3_plan's list."""
    cap = 18 * n_units + 8  # the header's bound (16 n + 7 with regeneration and clipping) and more
    ops = (zero_op_t * cap)()
    n = C.c_int32()
    _check("zero3_plan_microbatch", lib.zero3_plan_microbatch(
        n_units, 1 if reshard_after_forward else 0, int(micro_batch), int(micro_batches), ops, cap,
        C.byref(n)))
    return [(OP_NAMES[o.kind], o.stream, o.unit, o.arg) for o in ops[:n.value]]


def zero3_step_microbatch(units, grads, grad_acc, micro_batch, micro_batches, master, m, v,
                          shard_bf16, full_a, full_b, hp, reshard_after_forward=True,
                          main_stream=None, side_stream=None):
    """One micro-batch of a ZeRO-3 step with gradient accumulation (every
    unit's gradients resident); the update happens in the last micro-batch."""
    g, rows = _rows(grads, 2, "grads")
    a = _rows(grad_acc, 4, "grad_acc")[0] if grad_acc is not None else None
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    _check("zero3_step_microbatch", lib.zero3_step_microbatch(
        arr, len(units), len(rows), g, a, int(micro_batch), int(micro_batches), w, mm, vv, s,
        _dev(full_a, 2, "full_a"), _dev(full_b, 2, "full_b") if full_b is not None else None,
        C.byref(hp), 1 if reshard_after_forward else 0, _stream(main_stream),
        _stream(side_stream)))


def zero3_step(units, grads, master, m, v, shard_bf16, full_a, full_b, hp, grads_resident=True,
               regen=None, clip=None, reshard_after_forward=True, main_stream=None,
               side_stream=None):
    """One whole ZeRO-3 step issued by the native scheduler.  grads: per-rank
    gradients (all units concatenated when grads_resident, else one unit-sized
    buffer per rank refilled by `regen`, a zero_regen_t)."""
    g, rows = _rows(grads, 2, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    _check("zero3_step", lib.zero3_step(
        arr, len(units), len(rows), g, 1 if grads_resident else 0, w, mm, vv, s,
        _dev(full_a, 2, "full_a"), _dev(full_b, 2, "full_b") if full_b is not None else None,
        C.byref(hp),
        C.byref(regen) if regen is not None else None, C.byref(clip) if clip is not None else None,
        1 if reshard_after_forward else 0, _stream(main_stream), _stream(side_stream)))


def zero3_step_checked(units, grads, master, m, v, shard_bf16, full_a, full_b, hp,
                       nonfinite_ranks, grads_resident=True, regen=None,
                       reshard_after_forward=True, main_stream=None, side_stream=None):
    """zero3_step (no clipping) with the fused pre-reduction finite check:
    bit r of nonfinite_ranks (device int32/uint32[2], word r // 32) is OR-ed in
    when rank r's gradient of any unit holds an infinity or a NaN."""
    g, rows = _rows(grads, 2, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    _check("zero3_step_checked", lib.zero3_step_checked(
        arr, len(units), len(rows), g, 1 if grads_resident else 0, w, mm, vv, s,
        _dev(full_a, 2, "full_a"), _dev(full_b, 2, "full_b") if full_b is not None else None,
        C.byref(hp), C.byref(regen) if regen is not None else None,
        1 if reshard_after_forward else 0, _flags(nonfinite_ranks), _stream(main_stream),
        _stream(side_stream)))


def zero3_step_f32grads(units, grads, master, m, v, shard_bf16, full_a, full_b, hp,
                        reshard_after_forward=True, main_stream=None, side_stream=None):
    """zero3_step with fp32 rank gradients (every unit's, concatenated per rank)."""
    g, rows = _rows(grads, 4, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    _check("zero3_step_f32grads", lib.zero3_step_f32grads(
        arr, len(units), len(rows), g, w, mm, vv, s, _dev(full_a, 2, "full_a"),
        _dev(full_b, 2, "full_b") if full_b is not None else None, C.byref(hp),
        1 if reshard_after_forward else 0, _stream(main_stream), _stream(side_stream)))


class Zero3Graph:
    """A handle from zero3_graph_create(_f32grads).  It keeps the captured tensors alive
    (the graph holds their addresses) until zero3_graph_destroy."""

    def __init__(self, handle, keep):
        self.handle, self._keep = handle, keep

    def launch(self, hp, stream=None):
        zero3_graph_launch(self, hp, stream)

    def close(self):
        zero3_graph_destroy(self)


def zero3_graph_create(units, grads, master, m, v, shard_bf16, full_a, full_b, hp, capture_stream,
                       side_stream, clip=None, reshard_after_forward=True):
    """Capture one ZeRO-3 step (zero3_step's, gradients resident) as a CUDA
    graph; capture_stream and side_stream are two distinct torch.cuda.Streams."""
    if capture_stream is None or side_stream is None:
        raise ValueError("zero3_graph_create needs two explicit streams (the default stream "
                         "cannot be captured)")
    g, rows = _rows(grads, 2, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    h = C.c_void_p()
    _check("zero3_graph_create", lib.zero3_graph_create(
        arr, len(units), len(rows), g, w, mm, vv, s, _dev(full_a, 2, "full_a"),
        _dev(full_b, 2, "full_b") if full_b is not None else None, C.byref(hp),
        C.byref(clip) if clip is not None else None, 1 if reshard_after_forward else 0,
        _stream(capture_stream), _stream(side_stream), C.byref(h)))
    return Zero3Graph(h, (grads, master, m, v, shard_bf16, full_a, full_b, clip))


def zero3_graph_create_f32grads(units, grads, master, m, v, shard_bf16, full_a, full_b, hp,
                                capture_stream, side_stream, reshard_after_forward=True):
    """zero3_graph_create for fp32 rank gradients (zero3_step_f32grads's step,
    gradients resident, no clipping)."""
    if capture_stream is None or side_stream is None:
        raise ValueError("zero3_graph_create_f32grads needs two explicit streams (the default "
                         "stream cannot be captured)")
    g, rows = _rows(grads, 4, "grads")
    w, _ = _rows(master, 4, "master")
    mm, _ = _rows(m, 4, "m")
    vv, _ = _rows(v, 4, "v")
    s, _ = _rows(shard_bf16, 2, "shard_bf16")
    arr = (zero_unit_t * len(units))(*units)
    h = C.c_void_p()
    _check("zero3_graph_create_f32grads", lib.zero3_graph_create_f32grads(
        arr, len(units), len(rows), g, w, mm, vv, s, _dev(full_a, 2, "full_a"),
        _dev(full_b, 2, "full_b") if full_b is not None else None, C.byref(hp),
        1 if reshard_after_forward else 0, _stream(capture_stream), _stream(side_stream),
        C.byref(h)))
    return Zero3Graph(h, (grads, master, m, v, shard_bf16, full_a, full_b))


def zero3_graph_launch(graph, hp, stream=None):
    if graph.handle is None:
        raise ValueError("zero3_graph_launch: the graph was destroyed")
    _check("zero3_graph_launch", lib.zero3_graph_launch(graph.handle, C.byref(hp), _stream(stream)))


def zero3_graph_destroy(graph):
    if graph.handle is not None:
        h, graph.handle = graph.handle, None
        _check("zero3_graph_destroy", lib.zero3_graph_destroy(h))
        graph._keep = None


# ------------------------------------------------------------------ harness calls
def zero_gen_grads_unit(seed, step, sigma, outliers, unit, unit_grads, stream=None):
    g, rows = _rows(unit_grads, 2, "unit_grads")
    _check("zero_gen_grads_unit", lib.zero_gen_grads_unit(
        int(seed), int(step), float(sigma), int(outliers), C.byref(unit), len(rows), g,
        _stream(stream)))


def zero_gen_master(seed, sigma, units, master, stream=None):
    w, rows = _rows(master, 4, "master")
    arr = (zero_unit_t * len(units))(*units)
    _check("zero_gen_master", lib.zero_gen_master(
        int(seed), float(sigma), arr, len(units), len(rows), w, _stream(stream)))


def zero_cast_bf16(src, dst, stream=None):
    _check("zero_cast_bf16", lib.zero_cast_bf16(
        _dev(src, 4, "src"), _dev(dst, 2, "dst"), src.numel(), _stream(stream)))


# ------------------------------------------------- operators of the model
# These calls are short (a few microseconds on the GPU for a few tokens), so
# each tensor is looked at once and attributes are not read twice.
_FLOATS = {torch.bfloat16: ZERO_TYPE_BF16, torch.int16: ZERO_TYPE_BF16,
           torch.uint16: ZERO_TYPE_BF16, torch.float32: ZERO_TYPE_F32}
_INDEXES = {torch.int32: ZERO_TYPE_I32, torch.int64: ZERO_TYPE_I64}
_KINDS = {"rms": ZERO_NORM_RMS, "layer": ZERO_NORM_LAYER}


def _type(t, what, types=_FLOATS):
    """ZERO_TYPE_* of a tensor (bf16 may be given as its bits, int16 or uint16)."""
    try:
        return types[t.dtype]
    except KeyError:
        raise ValueError("%s must be %s, got %s" % (
            what, "bf16 or fp32" if types is _FLOATS else "int32 or int64", t.dtype)) from None


def _at(t, what, shape=None):
    """The address of a contiguous device-addressable tensor of a shape."""
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if not t.is_contiguous() or not _addressable(t):
        raise ValueError("%s must be a contiguous CUDA or pinned host tensor" % what)
    return t.data_ptr()


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def zero_embed_forward(table, ids, out, scale=1.0, stream=None):
    """out[t, :] = scale * table[ids[t], :]; a row of +0 where the id lies outside the
    table.  table (V x D) and out (tokens x D): bf16 or fp32; ids: int32 or int64."""
    if table.dim() != 2:
        raise ValueError("table must have two dimensions")
    V, D = table.shape
    _check("zero_embed_forward", lib.zero_embed_forward(
        _at(table, "table"), _type(table, "table"), V, D, _at(ids, "ids"),
        _type(ids, "ids", _INDEXES), ids.numel(), scale, _at(out, "out", (*ids.shape, D)),
        _type(out, "out"), _raw_stream(stream)))


def _bytes(fn, n):
    if n < 0:
        raise ZeroError(fn, int(n))
    return n


def zero_embed_scratch_bytes(n_tokens, vocab, dim):
    return _bytes("zero_embed_scratch_bytes",
                  lib.zero_embed_scratch_bytes(int(n_tokens), int(vocab), int(dim)))


def zero_embed_backward(dout, ids, dtable, scratch, scale=1.0, accumulate=False, stream=None):
    """dtable[v, :] = (dtable[v, :] if accumulate else 0) + scale * the sum of dout's
    rows whose id is v, by sorted tokens.  scratch: a device tensor of
    zero_embed_scratch_bytes(tokens, V, D) bytes."""
    if dtable.dim() != 2:
        raise ValueError("dtable must have two dimensions")
    V, D = dtable.shape
    _check("zero_embed_backward", lib.zero_embed_backward(
        _at(dout, "dout", (*ids.shape, D)), _type(dout, "dout"), _at(ids, "ids"),
        _type(ids, "ids", _INDEXES), ids.numel(), scale, _at(dtable, "dtable"),
        _type(dtable, "dtable"), V, D, 1 if accumulate else 0, _at(scratch, "scratch"),
        scratch.nbytes, _raw_stream(stream)))


class _Alike:
    """Addresses of tensors that share a shape and one of the float types; None
    for None."""

    def __init__(self, shape, what, type=None):
        self.shape, self.what, self.type = shape, what, type

    def __call__(self, t, name):
        if t is None:
            return None
        at, type = _at(t, name, self.shape), _type(t, name)
        if self.type is None:
            self.type = type
        elif self.type != type:
            raise ValueError("%s must have one type: %s" % (self.what, name))
        return at


def _norm_call(rows, kind, rows_per_gate):
    """Shape, gate span and kind of a call on the residual stream `rows`."""
    if rows.dim() != 2:
        raise ValueError("the residual stream must have two dimensions")
    if kind not in _KINDS:
        raise ValueError("kind must be 'rms' or 'layer'")
    return rows.shape, int(rows_per_gate) if rows_per_gate else max(1, rows.shape[0]), _KINDS[kind]


def zero_block_norm_forward(x, branch=None, gate=None, post_weight=None, post_bias=None,
                            pre_weight=None, pre_bias=None, y=None, u=None, kind="rms",
                            rows_per_gate=None, post_norm=True, pre_norm=True, eps=1e-6,
                            residual_scale=1.0, branch_scale=1.0, stream=None):
    """y = residual_scale * x + branch_scale * gate * norm(branch), u = norm(y).

    x, y (rows x D) of the residual type, branch, u (rows x D) of the activations'
    type, gate (gate rows x D; row i uses gate row i // rows_per_gate, all rows the
    one gate row by default), weights and biases (D).  post_norm / pre_norm False
    leaves out the branch's norm / the norm of y (u is then None).  Without a
    branch (before the first block) u = norm(x), and y is None."""
    shape, span, kind = _norm_call(x, kind, rows_per_gate)
    R, D = shape
    res, act = _Alike(shape, "x and y"), _Alike(shape, "branch and u")
    par = _Alike((D,), "weights and biases")
    gates = _Alike((max(1, -(-R // span)), D), "gate")
    args = (res(x, "x"), act(branch, "branch"), gates(gate, "gate"),
            par(post_weight, "post_weight"), par(post_bias, "post_bias"),
            par(pre_weight, "pre_weight"), par(pre_bias, "pre_bias"), res(y, "y"), act(u, "u"))
    spec = zero_block_norm_t(R, D, span, kind, 1 if post_norm and branch is not None else 0,
                             1 if pre_norm else 0, act.type or res.type, res.type,
                             par.type or ZERO_TYPE_BF16, gates.type or ZERO_TYPE_BF16, eps,
                             residual_scale, branch_scale)
    _check("zero_block_norm_forward", lib.zero_block_norm_forward(C.byref(spec), *args,
                                                                  _raw_stream(stream)))


def zero_block_norm_scratch_bytes(n_rows, dim, rows_per_gate=None):
    span = int(rows_per_gate) if rows_per_gate else max(1, int(n_rows))
    return _bytes("zero_block_norm_scratch_bytes",
                  lib.zero_block_norm_scratch_bytes(int(n_rows), int(dim), span))


def zero_block_norm_backward(y, scratch, dy=None, du=None, branch=None, gate=None,
                             post_weight=None, post_bias=None, pre_weight=None, dx=None,
                             dbranch=None, dgate=None, dpost_weight=None, dpost_bias=None,
                             dpre_weight=None, dpre_bias=None, kind="rms", rows_per_gate=None,
                             post_norm=True, pre_norm=True, eps=1e-6, residual_scale=1.0,
                             branch_scale=1.0, stream=None):
    """The gradient of zero_block_norm_forward, given dy and du (either may be None: 0;
    du exactly when pre_norm is False).  y: the stream the forward call wrote (x
    where it had no branch).  Writes the gradients that are given: dx, dbranch
    (with a branch), dgate, and the weights' and biases' sums over the rows, which
    may lie in a rank's gradient buffer.  scratch: a device tensor of
    zero_block_norm_scratch_bytes(rows, D, rows_per_gate) bytes."""
    shape, span, kind = _norm_call(y, kind, rows_per_gate)
    R, D = shape
    gate_shape = (max(1, -(-R // span)), D)
    res, act = _Alike(shape, "y, dy and dx"), _Alike(shape, "du, branch and dbranch")
    par, gates = _Alike((D,), "weights and biases"), _Alike(gate_shape, "gate")
    sums = _Alike((D,), "the gradients of weights and biases")
    gate_sums = _Alike(gate_shape, "dgate")
    y = res(y, "y")
    args = (res(dy, "dy"), act(du, "du"), y, act(branch, "branch"), gates(gate, "gate"),
            par(post_weight, "post_weight"), par(post_bias, "post_bias"),
            par(pre_weight, "pre_weight"), res(dx, "dx"), act(dbranch, "dbranch"))
    spec = zero_block_norm_t(R, D, span, kind, 1 if post_norm and branch is not None else 0,
                             1 if pre_norm else 0, act.type or res.type, res.type,
                             par.type or ZERO_TYPE_BF16, gates.type or ZERO_TYPE_BF16, eps,
                             residual_scale, branch_scale)
    grads = zero_block_norm_grads_t(
        gate_sums(dgate, "dgate"), sums(dpost_weight, "dpost_weight"),
        sums(dpost_bias, "dpost_bias"), sums(dpre_weight, "dpre_weight"),
        sums(dpre_bias, "dpre_bias"), gate_sums.type or ZERO_TYPE_BF16,
        sums.type or ZERO_TYPE_BF16)
    _check("zero_block_norm_backward", lib.zero_block_norm_backward(
        C.byref(spec), *args, C.byref(grads), _at(scratch, "scratch"), scratch.nbytes,
        _raw_stream(stream)))


def _matrix(t, what, shape=None):
    """Address and row stride of a matrix whose rows are contiguous."""
    if t.dim() != 2:
        raise ValueError("%s must have two dimensions" % what)
    if shape is not None and t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    rows, cols = t.shape
    if not _addressable(t) or (cols > 1 and t.stride(1) != 1):
        raise ValueError("%s must be CUDA or pinned host memory with contiguous rows" % what)
    return t.data_ptr(), t.stride(0) if rows > 1 else max(cols, t.stride(0))


def _distill_call(logits, teacher_logits, teacher_ids, ce, kl, labels, row_weight, temperature,
                  ce_weight, kl_weight):
    ptr, stride = _matrix(logits, "logits")
    R, V = logits.shape
    if teacher_ids.dim() != 2:
        raise ValueError("teacher_ids must have two dimensions")
    entries = (R, teacher_ids.shape[1])
    rows = _Alike((R,), "ce, kl and row_weight (fp32)", ZERO_TYPE_F32)
    spec = zero_distill_t(R, V, stride, entries[1], _type(logits, "logits"),
                          _type(teacher_logits, "teacher_logits"),
                          _type(teacher_ids, "teacher_ids", _INDEXES),
                          _type(labels, "labels", _INDEXES) if labels is not None
                          else ZERO_TYPE_I64, temperature, ce_weight, kl_weight)
    return spec, (C.byref(spec), ptr, _at(teacher_logits, "teacher_logits", entries),
                  _at(teacher_ids, "teacher_ids", entries),
                  _at(labels, "labels", (R,)) if labels is not None else None,
                  rows(row_weight, "row_weight"), rows(ce, "ce"), rows(kl, "kl"))


def zero_distill_forward(logits, teacher_logits, teacher_ids, ce, kl, labels=None,
                         row_weight=None, temperature=1.0, stream=None):
    """Each row's distillation loss kl (temperature^2 * KL(teacher || student), the
    teacher given by its top logits and their ids, -1 for no entry) and cross
    entropy ce (0 without a label in [0, V)).  logits (rows x V): bf16 or fp32,
    rows contiguous, any row stride; teacher_logits, teacher_ids (rows x K); ce,
    kl, row_weight (rows): fp32; rows of weight 0 are not read."""
    _, args = _distill_call(logits, teacher_logits, teacher_ids, ce, kl, labels, row_weight,
                            temperature, 0.0, 1.0)
    _check("zero_distill_forward", lib.zero_distill_forward(*args, _raw_stream(stream)))


def zero_distill_forward_backward(logits, teacher_logits, teacher_ids, ce, kl, dlogits,
                                  labels=None, row_weight=None, temperature=1.0, ce_weight=0.0,
                                  kl_weight=1.0, stream=None):
    """zero_distill_forward, and dlogits = the gradient of the sum over the rows of
    row_weight * (ce_weight * ce + kl_weight * kl).  dlogits may be logits."""
    spec, args = _distill_call(logits, teacher_logits, teacher_ids, ce, kl, labels, row_weight,
                               temperature, ce_weight, kl_weight)
    ptr, stride = _matrix(dlogits, "dlogits", logits.shape)
    if _type(dlogits, "dlogits") != spec.logits_type:
        raise ValueError("logits and dlogits must have one type")
    _check("zero_distill_forward_backward", lib.zero_distill_forward_backward(
        *args, ptr, stride, _raw_stream(stream)))
