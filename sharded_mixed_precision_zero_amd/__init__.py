"""Python binding of the MI355X ZeRO-1/2 shard optimizer step.

Argument marshalling only: every step of the path runs in the HIP kernels of
``libzeroshard.so`` behind the C ABI of ``include/zero_shard.h``.  The
functions below carry the C names; ``ZeroShard`` is a small owner object
over one handle.  PyTorch is used for device memory and streams only.

There is no fallback: importing this package without the built library
raises, and every call that returns a negative status raises ``ZeroShardError``.
"""

from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzeroshard.so")

ZS_OK, ZS_EINVAL, ZS_EALIGN, ZS_ENOMEM, ZS_EHIP, ZS_EDEVICE, ZS_ESTATE, ZS_ETOOBIG = (
    0, -1, -2, -3, -4, -5, -6, -7)
ZS_MAX_ND = 64
ZS_F32, ZS_BF16, ZS_F16 = 0, 1, 2
ZS_ORTHO_MAX_STEPS = 32
ZS_NORM_LAYER, ZS_NORM_RMS = 0, 1
ZS_GATE_NONE, ZS_GATE_COLUMN, ZS_GATE_SIGMOID = 0, 1, 2
ZS_BLOCKNORM_MAX_COLS = 16384
ZS_ADAMW_BLOCK, ZS_ADAMW_MAX_TENSORS, ZS_ADAMW_MAX_ELEMENTS = 256, 1 << 20, 1 << 33
ZS_STATE_32, ZS_STATE_8 = 0, 1
ZS_EMBEDDING_MAX_TOKENS, ZS_EMBEDDING_MAX_VOCAB = 1 << 27, 1 << 30
# how a call's work is split into kernel launches (zero_shard.h)
ZS_NORM_LAUNCH_LEN = 1 << 26
ZS_WIDE_LAUNCH_LEN = 1 << 25
ZS_WIDE_MIN_ROWS = 18
ZS_WIDE_MIN_ROWS_QUANT = 32
ZS_WIDE_MIN_ROWS_Q8 = 16
QUANT_BLOCKS = (32, 64, 128, 256, 512)

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() (hipcc, gfx950)")

# The library must run on the same HIP runtime as the PyTorch that owns the
# device memory and streams.  Loading torch first makes the library's
# libamdhip64.so.7 dependency resolve to torch's already-loaded runtime;
# the other order would map a second runtime into the process.
import torch  # noqa: E402,F401

_lib = ctypes.CDLL(LIB_PATH)


class zs_desc(ctypes.Structure):  # noqa: N801  (the C name)
    _fields_ = [
        ("phi", ctypes.c_int64),
        ("n_d", ctypes.c_int32),
        ("r", ctypes.c_int32),
        ("shard_len", ctypes.c_int64),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("bias_correction", ctypes.c_int32),
        ("max_norm", ctypes.c_float),
        ("quant_block", ctypes.c_int32),
        ("master", ctypes.c_void_p),
        ("m", ctypes.c_void_p),
        ("v", ctypes.c_void_p),
        ("param_out", ctypes.c_void_p),
        ("q_codes", ctypes.c_void_p),
        ("q_scales", ctypes.c_void_p),
        ("gbar_ws", ctypes.c_void_p),
        ("stream", ctypes.c_void_p),
    ]


class zs_layernorm_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("ld_x", ctypes.c_int64),
        ("ld_residual", ctypes.c_int64),
        ("ld_sum", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_dsum", ctypes.c_int64),
        ("ld_dx", ctypes.c_int64),
        ("stream", ctypes.c_void_p),
    ]


class zs_muon_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("n", ctypes.c_int64),
        ("n_d", ctypes.c_int32),
        ("nesterov", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("mu", ctypes.c_float),
        ("weight_decay", ctypes.c_float),
        ("stream", ctypes.c_void_p),
    ]


class zs_ortho_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("batch", ctypes.c_int64),
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("ld_in", ctypes.c_int64),
        ("ld_out", ctypes.c_int64),
        ("stride_in", ctypes.c_int64),
        ("stride_out", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("steps", ctypes.c_int32),
        ("coeffs", ctypes.POINTER(ctypes.c_float)),
        ("eps", ctypes.c_float),
        ("stream", ctypes.c_void_p),
    ]


class zs_blocknorm_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("rows", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32),
        ("kind", ctypes.c_int32),
        ("post", ctypes.c_int32),
        ("gate", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("residual_scale", ctypes.c_float),
        ("ld_x", ctypes.c_int64),
        ("ld_block", ctypes.c_int64),
        ("ld_gate", ctypes.c_int64),
        ("ld_sum", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_dsum", ctypes.c_int64),
        ("ld_dx", ctypes.c_int64),
        ("ld_dblock", ctypes.c_int64),
        ("ld_dgate", ctypes.c_int64),
        ("stream", ctypes.c_void_p),
    ]


class zs_embedding_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("tokens", ctypes.c_int64),
        ("vocab", ctypes.c_int64),
        ("cols", ctypes.c_int64),
        ("first", ctypes.c_int64),
        ("padding", ctypes.c_int64),
        ("pad_set", ctypes.c_int32),
        ("id_bytes", ctypes.c_int32),
        ("dtype", ctypes.c_int32),
        ("table_dtype", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("accumulate", ctypes.c_int32),
        ("scale", ctypes.c_float),
        ("ld_table", ctypes.c_int64),
        ("ld_y", ctypes.c_int64),
        ("ld_dy", ctypes.c_int64),
        ("ld_dtable", ctypes.c_int64),
        ("stream", ctypes.c_void_p),
    ]


class zs_adamw_tensor(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("n", ctypes.c_int64),
        ("master_in", ctypes.c_void_p),
        ("master_out", ctypes.c_void_p),
        ("m_in", ctypes.c_void_p),
        ("v_in", ctypes.c_void_p),
        ("m_out", ctypes.c_void_p),
        ("v_out", ctypes.c_void_p),
        ("m_scale_in", ctypes.c_void_p),
        ("v_scale_in", ctypes.c_void_p),
        ("m_scale_out", ctypes.c_void_p),
        ("v_scale_out", ctypes.c_void_p),
        ("param_out", ctypes.c_void_p),
        ("weight_decay", ctypes.c_float),
        ("lr_scale", ctypes.c_float),
        ("state", ctypes.c_int32),
        ("grad_dtype", ctypes.c_int32),
        ("param_dtype", ctypes.c_int32),
    ]


class zs_adamw_desc(ctypes.Structure):  # noqa: N801
    _fields_ = [
        ("count", ctypes.c_int64),
        ("beta1", ctypes.c_float),
        ("beta2", ctypes.c_float),
        ("eps", ctypes.c_float),
        ("bias_correction", ctypes.c_int32),
        ("max_norm", ctypes.c_float),
        ("stream", ctypes.c_void_p),
    ]


_handle_p = ctypes.c_void_p
_lib.zero_shard_init.restype = ctypes.c_int
_lib.zero_shard_init.argtypes = [ctypes.POINTER(zs_desc), ctypes.POINTER(_handle_p)]
_lib.zero_shard_gnorm.restype = ctypes.c_int
_lib.zero_shard_gnorm.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_step_consts.restype = ctypes.c_int
_lib.zero_shard_step_consts.argtypes = [ctypes.POINTER(zs_desc), ctypes.c_float, ctypes.c_int64,
                                        ctypes.c_void_p]
_lib.zero_shard_step_dev.restype = ctypes.c_int
_lib.zero_shard_step_dev.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_gnorm_noalloc.restype = ctypes.c_int
_lib.zero_shard_gnorm_noalloc.argtypes = [ctypes.POINTER(zs_desc), ctypes.c_void_p,
                                          ctypes.c_void_p]
_lib.zero_shard_step.restype = ctypes.c_int
_lib.zero_shard_step.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_float, ctypes.c_int64,
                                 ctypes.c_void_p]
_lib.zero_shard_gnorm_q8.restype = ctypes.c_int
_lib.zero_shard_gnorm_q8.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                     ctypes.c_void_p]
_lib.zero_shard_step_q8.restype = ctypes.c_int
_lib.zero_shard_step_q8.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                    ctypes.c_float, ctypes.c_int64, ctypes.c_void_p]
_lib.zero_shard_gnorm_bucketed.restype = ctypes.c_int
_lib.zero_shard_gnorm_bucketed.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_int64,
                                           ctypes.c_int32, ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_step_bucketed.restype = ctypes.c_int
_lib.zero_shard_step_bucketed.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_int32, ctypes.c_void_p, ctypes.c_float,
                                          ctypes.c_int64, ctypes.c_void_p]
_lib.zero_shard_gnorm_bucketed_q8.restype = ctypes.c_int
_lib.zero_shard_gnorm_bucketed_q8.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p,
                                              ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                              ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_step_bucketed_q8.restype = ctypes.c_int
_lib.zero_shard_step_bucketed_q8.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int32, ctypes.c_int64, ctypes.c_int32,
                                             ctypes.c_void_p, ctypes.c_float, ctypes.c_int64,
                                             ctypes.c_void_p]
_lib.zero_shard_dequant.restype = ctypes.c_int
_lib.zero_shard_dequant.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                    ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p,
                                    ctypes.c_void_p]
_lib.zero_shard_host_step.restype = ctypes.c_int
_lib.zero_shard_host_step.argtypes = [ctypes.POINTER(zs_desc), ctypes.c_void_p, ctypes.c_float,
                                      ctypes.c_int64, ctypes.c_double, ctypes.c_int32]
_lib.zero_shard_offload_init.restype = ctypes.c_int
_lib.zero_shard_offload_init.argtypes = [ctypes.POINTER(zs_desc), ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int32,
                                         ctypes.POINTER(_handle_p)]
_lib.zero_shard_offload_step.restype = ctypes.c_int
_lib.zero_shard_offload_step.argtypes = [_handle_p, ctypes.c_void_p, ctypes.c_float,
                                         ctypes.c_int64, ctypes.c_double]
_lib.zero_shard_offload_params.restype = ctypes.c_void_p
_lib.zero_shard_offload_params.argtypes = [_handle_p]
_lib.zero_shard_offload_wait.restype = ctypes.c_int
_lib.zero_shard_offload_wait.argtypes = [_handle_p]
_lib.zero_shard_offload_free.restype = ctypes.c_int
_lib.zero_shard_offload_free.argtypes = [_handle_p]
_lib.zero_shard_quant.restype = ctypes.c_int
_lib.zero_shard_quant.argtypes = [_handle_p, ctypes.c_int32]
_lib.zero_shard_layernorm.restype = ctypes.c_int
_lib.zero_shard_layernorm.argtypes = [ctypes.POINTER(zs_layernorm_desc)] + [ctypes.c_void_p] * 8
_lib.zero_shard_layernorm_workspace.restype = ctypes.c_int64
_lib.zero_shard_layernorm_workspace.argtypes = [ctypes.POINTER(zs_layernorm_desc)]
_lib.zero_shard_layernorm_bwd.restype = ctypes.c_int
_lib.zero_shard_layernorm_bwd.argtypes = ([ctypes.POINTER(zs_layernorm_desc)]
                                          + [ctypes.c_void_p] * 10 + [ctypes.c_int64])
_lib.zero_shard_muon_momentum.restype = ctypes.c_int
_lib.zero_shard_muon_momentum.argtypes = [ctypes.POINTER(zs_muon_desc)] + [ctypes.c_void_p] * 4
_lib.zero_shard_muon_apply.restype = ctypes.c_int
_lib.zero_shard_muon_apply.argtypes = [ctypes.POINTER(zs_muon_desc), ctypes.c_void_p,
                                       ctypes.c_float, ctypes.c_float, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_ortho_workspace.restype = ctypes.c_int64
_lib.zero_shard_ortho_workspace.argtypes = [ctypes.POINTER(zs_ortho_desc)]
_lib.zero_shard_ortho.restype = ctypes.c_int
_lib.zero_shard_ortho.argtypes = [ctypes.POINTER(zs_ortho_desc), ctypes.c_void_p, ctypes.c_void_p,
                                  ctypes.c_void_p, ctypes.c_int64]
_lib.zero_shard_blocknorm.restype = ctypes.c_int
_lib.zero_shard_blocknorm.argtypes = [ctypes.POINTER(zs_blocknorm_desc)] + [ctypes.c_void_p] * 10
_lib.zero_shard_blocknorm_workspace.restype = ctypes.c_int64
_lib.zero_shard_blocknorm_workspace.argtypes = [ctypes.POINTER(zs_blocknorm_desc)]
_lib.zero_shard_blocknorm_bwd.restype = ctypes.c_int
_lib.zero_shard_blocknorm_bwd.argtypes = ([ctypes.POINTER(zs_blocknorm_desc)]
                                          + [ctypes.c_void_p] * 17 + [ctypes.c_int64])
_lib.zero_shard_embedding.restype = ctypes.c_int
_lib.zero_shard_embedding.argtypes = [ctypes.POINTER(zs_embedding_desc)] + [ctypes.c_void_p] * 3
_lib.zero_shard_embedding_workspace.restype = ctypes.c_int64
_lib.zero_shard_embedding_workspace.argtypes = [ctypes.POINTER(zs_embedding_desc)]
_lib.zero_shard_embedding_bwd.restype = ctypes.c_int
_lib.zero_shard_embedding_bwd.argtypes = ([ctypes.POINTER(zs_embedding_desc)]
                                          + [ctypes.c_void_p] * 4 + [ctypes.c_int64])
_adamw_call = [ctypes.POINTER(zs_adamw_desc), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_adamw_plan_bytes.restype = ctypes.c_int64
_lib.zero_shard_adamw_plan_bytes.argtypes = [ctypes.POINTER(zs_adamw_desc), ctypes.c_void_p]
_lib.zero_shard_adamw_plan.restype = ctypes.c_int
_lib.zero_shard_adamw_plan.argtypes = [ctypes.POINTER(zs_adamw_desc), ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int64]
_lib.zero_shard_adamw_gnorm.restype = ctypes.c_int
_lib.zero_shard_adamw_gnorm.argtypes = _adamw_call + [ctypes.c_void_p]
_lib.zero_shard_adamw.restype = ctypes.c_int
_lib.zero_shard_adamw.argtypes = _adamw_call + [ctypes.c_float, ctypes.c_int64, ctypes.c_uint32,
                                                ctypes.c_void_p]
_lib.zero_shard_adamw_consts.restype = ctypes.c_int
_lib.zero_shard_adamw_consts.argtypes = [ctypes.POINTER(zs_adamw_desc), ctypes.c_float,
                                         ctypes.c_int64, ctypes.c_uint32, ctypes.c_void_p]
_lib.zero_shard_adamw_dev.restype = ctypes.c_int
_lib.zero_shard_adamw_dev.argtypes = _adamw_call + [ctypes.c_void_p, ctypes.c_void_p]
_lib.zero_shard_free.restype = ctypes.c_int
_lib.zero_shard_free.argtypes = [_handle_p]
_lib.zero_shard_strerror.restype = ctypes.c_char_p
_lib.zero_shard_strerror.argtypes = [ctypes.c_int]
_lib.zero_shard_len.restype = ctypes.c_int64
_lib.zero_shard_len.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32]

EXPORTS = ("zero_shard_init", "zero_shard_gnorm", "zero_shard_gnorm_noalloc", "zero_shard_step",
           "zero_shard_step_consts", "zero_shard_step_dev",
           "zero_shard_gnorm_q8",
           "zero_shard_step_q8", "zero_shard_gnorm_bucketed", "zero_shard_step_bucketed",
           "zero_shard_gnorm_bucketed_q8", "zero_shard_step_bucketed_q8",
           "zero_shard_quant", "zero_shard_dequant",
           "zero_shard_host_step", "zero_shard_offload_init", "zero_shard_offload_step",
           "zero_shard_offload_params", "zero_shard_offload_wait", "zero_shard_offload_free",
           "zero_shard_layernorm", "zero_shard_layernorm_workspace", "zero_shard_layernorm_bwd",
           "zero_shard_muon_momentum", "zero_shard_muon_apply", "zero_shard_ortho_workspace",
           "zero_shard_ortho", "zero_shard_blocknorm", "zero_shard_blocknorm_workspace",
           "zero_shard_blocknorm_bwd", "zero_shard_embedding", "zero_shard_embedding_workspace",
           "zero_shard_embedding_bwd", "zero_shard_adamw_plan_bytes", "zero_shard_adamw_plan",
           "zero_shard_adamw_gnorm", "zero_shard_adamw", "zero_shard_adamw_consts",
           "zero_shard_adamw_dev", "zero_shard_free", "zero_shard_strerror", "zero_shard_len")


class ZeroShardError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {zero_shard_strerror(code)} ({code})")


def _check(rc: int, what: str) -> None:
    if rc != ZS_OK:
        raise ZeroShardError(rc, what)


def check(rc: int) -> None:
    """Raise ZeroShardError if a C-named call returned a negative status."""
    _check(rc, "zero_shard call")


def _ptr(t) -> int | None:
    if t is None:
        return None
    return int(t.data_ptr())


def _ptrs(*tensors) -> list:
    return [None if t is None else t.data_ptr() for t in tensors]


def contrib_table(contrib) -> ctypes.Array | None:
    """Host array of device pointers: a list of 1-D tensors (or None), or the
    rows of a 2-D tensor (row k = rank k's contribution, codes or scales)."""
    if contrib is None:
        return None
    if isinstance(contrib, ctypes.Array):  # already a table (kept by the caller)
        return contrib
    if hasattr(contrib, "dim") and contrib.dim() == 2:
        rows = [contrib[k] for k in range(contrib.shape[0])]
    else:
        rows = list(contrib)
    tab = (ctypes.c_void_p * max(1, len(rows)))(*[_ptr(r) for r in rows])
    tab._keep = rows
    return tab


def _kept_table(table, owner, check):
    """A table that the caller keeps.  check(its tensors) runs when ``owner`` first sees
    it, and again if its entries have changed since; they have to be the tensors'."""
    entries, seen = bytes(table), getattr(table, "_seen", None)
    if seen is None or seen[0] is not owner or seen[1] != entries:
        check(table._keep)
        _require(entries == bytes(contrib_table(table._keep)), "a table's entries")
        table._seen = owner, entries
    return table


# ------------------------------------------------------------ C-named calls

def zero_shard_strerror(code: int) -> str:
    return _lib.zero_shard_strerror(int(code)).decode()


def zero_shard_len(phi: int, n_d: int, r: int) -> int:
    return int(_lib.zero_shard_len(int(phi), int(n_d), int(r)))


def zero_shard_init(desc: zs_desc) -> tuple[int, ctypes.c_void_p]:
    h = _handle_p()
    rc = _lib.zero_shard_init(ctypes.byref(desc), ctypes.byref(h))
    return rc, h


def zero_shard_gnorm(h, contrib, sumsq_dev) -> int:
    return _lib.zero_shard_gnorm(h, contrib_table(contrib), _ptr(sumsq_dev))


def zero_shard_gnorm_noalloc(desc: zs_desc, contrib, sumsq_dev) -> int:
    """zero_shard_gnorm without a handle and without allocating (desc: a
    zs_desc; its n_d, shard_len, gbar_ws and stream are used)."""
    return _lib.zero_shard_gnorm_noalloc(ctypes.byref(desc), contrib_table(contrib),
                                         _ptr(sumsq_dev))


def zero_shard_step(h, contrib, lr: float, t: int, global_sumsq_dev=None) -> int:
    return _lib.zero_shard_step(h, contrib_table(contrib), float(lr), int(t),
                                _ptr(global_sumsq_dev))


def zero_shard_step_consts(desc: zs_desc, lr: float, t: int):
    """-> (status, [lr, lr*wd, bc1, bc2]) as the library computes them."""
    out = (ctypes.c_double * 4)()
    rc = _lib.zero_shard_step_consts(ctypes.byref(desc), float(lr), int(t), out)
    return rc, list(out)


def zero_shard_step_dev(h, contrib, consts_dev, global_sumsq_dev=None) -> int:
    """consts_dev: a float64 device tensor of 4 (see zero_shard_step_consts)."""
    return _lib.zero_shard_step_dev(h, contrib_table(contrib), _ptr(consts_dev),
                                    _ptr(global_sumsq_dev))


def zero_shard_gnorm_q8(h, codes, scales, block: int, sumsq_dev) -> int:
    return _lib.zero_shard_gnorm_q8(h, contrib_table(codes), contrib_table(scales), int(block),
                                    _ptr(sumsq_dev))


def zero_shard_step_q8(h, codes, scales, block: int, lr: float, t: int,
                       global_sumsq_dev=None) -> int:
    return _lib.zero_shard_step_q8(h, contrib_table(codes), contrib_table(scales), int(block),
                                   float(lr), int(t), _ptr(global_sumsq_dev))


def event_table(ready) -> ctypes.Array | None:
    """Host array of hipEvent_t from a list of torch.cuda.Event (or None
    entries); None stays None.  Each event must have been recorded."""
    if ready is None:
        return None
    tab = (ctypes.c_void_p * max(1, len(ready)))(
        *[None if e is None else int(e.cuda_event) for e in ready])
    tab._keep = list(ready)
    return tab


def zero_shard_gnorm_bucketed(h, contrib, bucket_len: int, streams: int, ready,
                              sumsq_dev) -> int:
    return _lib.zero_shard_gnorm_bucketed(h, contrib_table(contrib), int(bucket_len),
                                          int(streams), event_table(ready), _ptr(sumsq_dev))


def zero_shard_step_bucketed(h, contrib, bucket_len: int, streams: int, ready, lr: float,
                             t: int, global_sumsq_dev=None) -> int:
    return _lib.zero_shard_step_bucketed(h, contrib_table(contrib), int(bucket_len),
                                         int(streams), event_table(ready), float(lr), int(t),
                                         _ptr(global_sumsq_dev))


def zero_shard_gnorm_bucketed_q8(h, codes, scales, block: int, bucket_len: int, streams: int,
                                 ready, sumsq_dev) -> int:
    return _lib.zero_shard_gnorm_bucketed_q8(h, contrib_table(codes), contrib_table(scales),
                                             int(block), int(bucket_len), int(streams),
                                             event_table(ready), _ptr(sumsq_dev))


def zero_shard_step_bucketed_q8(h, codes, scales, block: int, bucket_len: int, streams: int,
                                ready, lr: float, t: int, global_sumsq_dev=None) -> int:
    return _lib.zero_shard_step_bucketed_q8(h, contrib_table(codes), contrib_table(scales),
                                            int(block), int(bucket_len), int(streams),
                                            event_table(ready), float(lr), int(t),
                                            _ptr(global_sumsq_dev))


def zero_shard_quant(h, block: int) -> int:
    return _lib.zero_shard_quant(h, int(block))


def zero_shard_dequant(codes, scales, n_d: int, phi: int, block: int, param_out,
                       stream=None) -> int:
    """param_out: 16-bit tensor of phi elements; stream: a torch stream
    (default: the current one)."""
    if stream is None:
        import torch

        stream = torch.cuda.current_stream()
    return _lib.zero_shard_dequant(contrib_table(codes), contrib_table(scales), int(n_d), int(phi),
                                   int(block), _ptr(param_out), int(stream.cuda_stream))


def zero_shard_host_step(desc: zs_desc, gbar_host_ptr: int, lr: float, t: int,
                         global_sumsq: float = 0.0, threads: int = 1) -> int:
    """desc carries HOST pointers; gbar_host_ptr: address of fp32[shard_len]
    in host memory."""
    return _lib.zero_shard_host_step(ctypes.byref(desc), gbar_host_ptr, float(lr), int(t),
                                     float(global_sumsq), int(threads))


def host_desc(*, phi: int, n_d: int, r: int, shard_len: int, master, m, v, param_out,
              beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
              weight_decay: float = 0.0, bias_correction: bool = True, max_norm: float = 0.0,
              quant_block: int = 0, q_codes=None, q_scales=None) -> zs_desc:
    """A descriptor over host arrays (numpy arrays or CPU tensors) for
    zero_shard_host_step; keep the arrays alive while it is used."""
    def addr(a):
        if a is None:
            return None
        return int(a.ctypes.data) if hasattr(a, "ctypes") else int(a.data_ptr())

    return zs_desc(phi=int(phi), n_d=int(n_d), r=int(r), shard_len=int(shard_len),
                   beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
                   bias_correction=int(bool(bias_correction)), max_norm=max_norm,
                   quant_block=int(quant_block), master=addr(master), m=addr(m), v=addr(v),
                   param_out=addr(param_out), q_codes=addr(q_codes), q_scales=addr(q_scales),
                   gbar_ws=None, stream=None)


def zero_shard_offload_init(host: zs_desc, param_dev0, param_dev1, stream=None,
                            threads: int = 16):
    """-> (status, handle).  host: a host_desc(...); param_dev0/1: 16-bit
    device tensors of shard_len elements; stream: a torch stream (default:
    the current one)."""
    if stream is None:
        import torch

        stream = torch.cuda.current_stream()
    o = _handle_p()
    rc = _lib.zero_shard_offload_init(ctypes.byref(host), _ptr(param_dev0), _ptr(param_dev1),
                                      int(stream.cuda_stream), int(threads), ctypes.byref(o))
    return rc, o


def zero_shard_offload_step(o, contrib, lr: float, t: int, s_other: float = 0.0) -> int:
    return _lib.zero_shard_offload_step(o, contrib_table(contrib), float(lr), int(t),
                                        float(s_other))


def zero_shard_offload_params(o) -> int | None:
    return _lib.zero_shard_offload_params(o)


def zero_shard_offload_wait(o) -> int:
    return _lib.zero_shard_offload_wait(o)


def zero_shard_offload_free(o) -> int:
    return _lib.zero_shard_offload_free(o)


def zero_shard_free(h) -> int:
    return _lib.zero_shard_free(h)


def dtype_code(dtype) -> int:
    """zs_dtype of a torch dtype (float32, bfloat16, float16)."""
    try:
        return _DTYPES[dtype]
    except KeyError:
        raise ZeroShardError(ZS_EINVAL, f"dtype {dtype}") from None


_DTYPES = {torch.float32: ZS_F32, torch.bfloat16: ZS_BF16, torch.float16: ZS_F16}


def _stream(stream) -> int:
    """hipStream_t of a torch stream (default: the current one)."""
    return int((torch.cuda.current_stream() if stream is None else stream).cuda_stream)


def layernorm_desc(*, rows: int, cols: int, dtype=torch.bfloat16, param_dtype=None,
                   eps: float = 1e-5, stream=None, **ld: int) -> zs_layernorm_desc:
    """dtype, param_dtype: torch dtypes (param_dtype defaults to dtype); ld:
    the row strides ld_x, ld_residual, ... that are not cols; stream: a torch
    stream (default: the current one)."""
    return zs_layernorm_desc(
        rows=int(rows), cols=int(cols), dtype=dtype_code(dtype),
        param_dtype=dtype_code(dtype if param_dtype is None else param_dtype), eps=eps,
        stream=_stream(stream), **ld)


def zero_shard_layernorm(desc: zs_layernorm_desc, x, residual, gamma, beta, sum_out, y, mean,
                         rstd) -> int:
    return _lib.zero_shard_layernorm(ctypes.byref(desc),
                                     *_ptrs(x, residual, gamma, beta, sum_out, y, mean, rstd))


def zero_shard_layernorm_workspace(desc: zs_layernorm_desc) -> int:
    return int(_lib.zero_shard_layernorm_workspace(ctypes.byref(desc)))


def zero_shard_layernorm_bwd(desc: zs_layernorm_desc, dy, x, gamma, mean, rstd, dsum, dx, dgamma,
                             dbeta, workspace) -> int:
    """workspace: a contiguous device tensor (its size in bytes is passed on)
    or None."""
    return _lib.zero_shard_layernorm_bwd(
        ctypes.byref(desc), *_ptrs(dy, x, gamma, mean, rstd, dsum, dx, dgamma, dbeta, workspace),
        _nbytes(workspace))


def _nbytes(t) -> int:
    return 0 if t is None else int(t.numel() * t.element_size())


def muon_desc(*, n: int, n_d: int = 1, mu: float = 0.95, nesterov: bool = True,
              dtype=torch.bfloat16, weight_decay: float = 0.0, stream=None) -> zs_muon_desc:
    return zs_muon_desc(n=int(n), n_d=int(n_d), nesterov=int(bool(nesterov)),
                        dtype=dtype_code(dtype), mu=mu, weight_decay=weight_decay,
                        stream=_stream(stream))


def zero_shard_muon_momentum(desc: zs_muon_desc, contrib, m_in, m_out, update) -> int:
    table = contrib_table(contrib)
    if table is not None and len(table) < desc.n_d and desc.n > 0:
        return ZS_EINVAL
    return _lib.zero_shard_muon_momentum(ctypes.byref(desc), table, _ptr(m_in), _ptr(m_out),
                                         _ptr(update))


def zero_shard_muon_apply(desc: zs_muon_desc, o, lr: float, scale: float, master_in, master_out,
                          param_out) -> int:
    return _lib.zero_shard_muon_apply(ctypes.byref(desc), _ptr(o), float(lr), float(scale),
                                      _ptr(master_in), _ptr(master_out), _ptr(param_out))


def ortho_desc(*, batch: int = 1, rows: int, cols: int, dtype=torch.bfloat16, steps: int = 5,
               coeffs=None, eps: float = 1e-7, ld_in: int = 0, ld_out: int = 0,
               stride_in: int = 0, stride_out: int = 0, stream=None) -> zs_ortho_desc:
    """coeffs: (a, b, c) of every step, or one (a, b, c) per step, or None."""
    d = zs_ortho_desc(batch=int(batch), rows=int(rows), cols=int(cols), ld_in=int(ld_in),
                      ld_out=int(ld_out), stride_in=int(stride_in), stride_out=int(stride_out),
                      dtype=dtype_code(dtype), steps=int(steps), eps=eps, stream=_stream(stream))
    if coeffs is not None:
        each = list(coeffs) if hasattr(coeffs[0], "__len__") else [coeffs] * int(steps)
        if len(each) != int(steps) or any(len(k) != 3 for k in each):
            raise ZeroShardError(ZS_EINVAL, "coeffs")
        d._keep = (ctypes.c_float * (3 * len(each)))(*[float(v) for k in each for v in k])
        d.coeffs = ctypes.cast(d._keep, ctypes.POINTER(ctypes.c_float))
    return d


def zero_shard_ortho_workspace(desc: zs_ortho_desc) -> int:
    return int(_lib.zero_shard_ortho_workspace(ctypes.byref(desc)))


def zero_shard_ortho(desc: zs_ortho_desc, g, o, workspace) -> int:
    """workspace: a contiguous device tensor (its size in bytes is passed on)."""
    return _lib.zero_shard_ortho(ctypes.byref(desc), _ptr(g), _ptr(o), _ptr(workspace),
                                 _nbytes(workspace))


_KINDS = {"layer": ZS_NORM_LAYER, "rms": ZS_NORM_RMS}
_GATES = {"none": ZS_GATE_NONE, "column": ZS_GATE_COLUMN, "sigmoid": ZS_GATE_SIGMOID}


def blocknorm_desc(*, rows: int, cols: int, dtype=torch.bfloat16, param_dtype=None,
                   kind: str = "rms", post: bool = True, gate: str = "none", eps: float = 1e-5,
                   residual_scale: float = 1.0, stream=None, **ld: int) -> zs_blocknorm_desc:
    """kind: "layer" or "rms"; gate: "none", "column" or "sigmoid"; the rest as
    for layernorm_desc."""
    if kind not in _KINDS or gate not in _GATES:
        raise ZeroShardError(ZS_EINVAL, f"kind {kind!r}, gate {gate!r}")
    return zs_blocknorm_desc(
        rows=int(rows), cols=int(cols), dtype=dtype_code(dtype),
        param_dtype=dtype_code(dtype if param_dtype is None else param_dtype),
        kind=_KINDS[kind], post=int(bool(post)), gate=_GATES[gate], eps=eps,
        residual_scale=residual_scale, stream=_stream(stream), **ld)


def zero_shard_blocknorm(desc: zs_blocknorm_desc, x, block, gate, gamma_post, beta_post, gamma,
                         beta, sum_out, y, stats) -> int:
    return _lib.zero_shard_blocknorm(ctypes.byref(desc),
                                     *_ptrs(x, block, gate, gamma_post, beta_post, gamma, beta,
                                            sum_out, y, stats))


def zero_shard_blocknorm_workspace(desc: zs_blocknorm_desc) -> int:
    return int(_lib.zero_shard_blocknorm_workspace(ctypes.byref(desc)))


def zero_shard_blocknorm_bwd(desc: zs_blocknorm_desc, dy, dsum, total, block, gate, gamma_post,
                             beta_post, gamma, stats, dx, dblock, dgate, dgamma_post, dbeta_post,
                             dgamma, dbeta, workspace) -> int:
    """workspace: a contiguous device tensor (its size in bytes is passed on)
    or None."""
    return _lib.zero_shard_blocknorm_bwd(
        ctypes.byref(desc),
        *_ptrs(dy, dsum, total, block, gate, gamma_post, beta_post, gamma, stats, dx, dblock,
               dgate, dgamma_post, dbeta_post, dgamma, dbeta, workspace), _nbytes(workspace))


def embedding_desc(*, tokens: int, vocab: int, cols: int, dtype=torch.bfloat16, table_dtype=None,
                   grad_dtype=None, scale: float = 1.0, first: int = 0, padding: int | None = None,
                   id_dtype=torch.int64, accumulate: bool = False, stream=None,
                   **ld: int) -> zs_embedding_desc:
    """table_dtype, grad_dtype: of the table and its gradient (default: dtype);
    padding: the id that gives no gradient; id_dtype: torch.int64 or torch.int32;
    ld: the row strides ld_table, ... that are not cols."""
    if id_dtype not in _ID_BYTES:
        raise ZeroShardError(ZS_EINVAL, f"id_dtype {id_dtype}")
    return zs_embedding_desc(
        tokens=int(tokens), vocab=int(vocab), cols=int(cols), first=int(first),
        padding=0 if padding is None else int(padding), pad_set=int(padding is not None),
        id_bytes=_ID_BYTES[id_dtype], dtype=dtype_code(dtype),
        table_dtype=dtype_code(dtype if table_dtype is None else table_dtype),
        grad_dtype=dtype_code(dtype if grad_dtype is None else grad_dtype),
        accumulate=int(bool(accumulate)), scale=scale, stream=_stream(stream), **ld)


_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def zero_shard_embedding(desc: zs_embedding_desc, ids, table, y) -> int:
    return _lib.zero_shard_embedding(ctypes.byref(desc), *_ptrs(ids, table, y))


def zero_shard_embedding_workspace(desc: zs_embedding_desc) -> int:
    return int(_lib.zero_shard_embedding_workspace(ctypes.byref(desc)))


def zero_shard_embedding_bwd(desc: zs_embedding_desc, ids, dy, dtable, workspace) -> int:
    """workspace: a contiguous device tensor (its size in bytes is passed on)."""
    return _lib.zero_shard_embedding_bwd(ctypes.byref(desc), *_ptrs(ids, dy, dtable, workspace),
                                         _nbytes(workspace))


def adamw_tensor(master, m, v, *, param_out=None, m_scale=None, v_scale=None, master_out=None,
                 m_out=None, v_out=None, m_scale_out=None, v_scale_out=None,
                 grad_dtype=torch.bfloat16, weight_decay: float = 0.0,
                 lr_scale: float = 1.0) -> zs_adamw_tensor:
    """A tensor of an AdamW plan, from contiguous device tensors of any shape.
    master: float32; m, v: float32, or, for a state in 8 bits, float8_e4m3fn (or uint8
    patterns) of m and sqrt(v) with their scales, float32[ceil(n / 256)];
    param_out: bfloat16 or float16, or None; *_out: where the results go (default: in
    place).  The struct keeps the tensors alive."""
    n = master.numel()
    eight = m.dtype in _E4M3_LIKE
    scales = (n + ZS_ADAMW_BLOCK - 1) // ZS_ADAMW_BLOCK
    state = _E4M3_LIKE if eight else (torch.float32,)
    ins = {"master": master, "m": m, "v": v, "m_scale": m_scale, "v_scale": v_scale}
    outs = {"master": master_out, "m": m_out, "v": v_out, "m_scale": m_scale_out,
            "v_scale": v_scale_out}
    outs = {k: ins[k] if t is None else t for k, t in outs.items()}
    for what, types, size in (("master", (torch.float32,), n), ("m", state, n), ("v", state, n),
                              ("m_scale", (torch.float32,), scales),
                              ("v_scale", (torch.float32,), scales)):
        for t in (ins[what], outs[what]):
            if what.endswith("scale") and not eight:
                _require(t is None, what)
            else:
                _require(t is not None and t.dtype in types and t.numel() == size and t.is_cuda
                         and t.is_contiguous(), what)
    if param_out is not None:
        _require(param_out.dtype in (torch.bfloat16, torch.float16) and param_out.numel() == n
                 and param_out.is_cuda and param_out.is_contiguous(), "param_out")
    t = zs_adamw_tensor(
        n=n, weight_decay=weight_decay, lr_scale=lr_scale,
        state=ZS_STATE_8 if eight else ZS_STATE_32, grad_dtype=dtype_code(grad_dtype),
        param_dtype=ZS_BF16 if param_out is None else dtype_code(param_out.dtype),
        param_out=_ptr(param_out), **{k + "_in": _ptr(x) for k, x in ins.items()},
        **{k + "_out": _ptr(x) for k, x in outs.items()})
    t._keep = (ins, outs, param_out)
    return t


_E4M3_LIKE = (torch.float8_e4m3fn, torch.uint8)  # e4m3 numbers or their patterns


def adamw_state(n: int, bits: int = 32, device="cuda") -> dict:
    """The state that a tensor of n elements starts with, as arguments of
    adamw_tensor: m and v, and with 8 bits m_scale and v_scale."""
    _require(bits in (8, 32), f"bits {bits}")
    if bits == 32:
        return {k: torch.zeros(n, device=device) for k in ("m", "v")}
    blocks = (n + ZS_ADAMW_BLOCK - 1) // ZS_ADAMW_BLOCK
    state = {k: torch.zeros(n, device=device, dtype=torch.uint8).view(torch.float8_e4m3fn)
             for k in ("m", "v")}
    state.update({k: torch.zeros(blocks, device=device) for k in ("m_scale", "v_scale")})
    return state


def adamw_desc(*, count: int, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               bias_correction: bool = True, max_norm: float = 0.0, stream=None) -> zs_adamw_desc:
    return zs_adamw_desc(count=int(count), beta1=beta1, beta2=beta2, eps=eps,
                         bias_correction=int(bool(bias_correction)), max_norm=max_norm,
                         stream=_stream(stream))


def zero_shard_adamw_plan_bytes(desc: zs_adamw_desc, tensors) -> int:
    """tensors: an array of zs_adamw_tensor ((zs_adamw_tensor * n)(...))."""
    if tensors is not None and len(tensors) < desc.count:
        return -1
    return int(_lib.zero_shard_adamw_plan_bytes(ctypes.byref(desc), tensors))


def zero_shard_adamw_plan(desc: zs_adamw_desc, tensors, plan) -> int:
    """plan: a contiguous CPU tensor (its size in bytes is passed on)."""
    if tensors is not None and len(tensors) < desc.count or plan is not None and plan.is_cuda:
        return ZS_EINVAL
    return _lib.zero_shard_adamw_plan(ctypes.byref(desc), tensors, _ptr(plan), _nbytes(plan))


def _adamw_fits(desc: zs_adamw_desc, plan, table) -> bool:
    """What the call reads on the host is there: a gradient's address for each tensor, and a
    plan that is not the device's copy."""
    return ((table is None or len(table) >= desc.count)
            and (plan is None or not plan.is_cuda))


def zero_shard_adamw_gnorm(desc: zs_adamw_desc, plan, plan_dev, grads, sumsq_dev) -> int:
    """plan, plan_dev: the plan on the CPU and its copy on the device."""
    table = contrib_table(grads)
    if not _adamw_fits(desc, plan, table):
        return ZS_EINVAL
    return _lib.zero_shard_adamw_gnorm(ctypes.byref(desc), _ptr(plan), _ptr(plan_dev), table,
                                       _ptr(sumsq_dev))


def zero_shard_adamw(desc: zs_adamw_desc, plan, plan_dev, grads, lr: float, t: int, key: int,
                     global_sumsq_dev=None) -> int:
    table = contrib_table(grads)
    if not _adamw_fits(desc, plan, table):
        return ZS_EINVAL
    return _lib.zero_shard_adamw(ctypes.byref(desc), _ptr(plan), _ptr(plan_dev), table, float(lr),
                                 int(t), int(key) & 0xFFFFFFFF, _ptr(global_sumsq_dev))


def zero_shard_adamw_consts(desc: zs_adamw_desc, lr: float, t: int, key: int):
    """-> (status, [lr, bc1, bc2, key])."""
    out = (ctypes.c_double * 4)()
    rc = _lib.zero_shard_adamw_consts(ctypes.byref(desc), float(lr), int(t),
                                      int(key) & 0xFFFFFFFF, out)
    return rc, list(out)


def zero_shard_adamw_dev(desc: zs_adamw_desc, plan, plan_dev, grads, consts_dev,
                         global_sumsq_dev=None) -> int:
    table = contrib_table(grads)
    if not _adamw_fits(desc, plan, table):
        return ZS_EINVAL
    return _lib.zero_shard_adamw_dev(ctypes.byref(desc), _ptr(plan), _ptr(plan_dev), table,
                                     _ptr(consts_dev), _ptr(global_sumsq_dev))


# ------------------------------------------------------------ owner objects

class ZeroShard:
    """One rank's shard step over caller-owned torch tensors.

    master, m, v: float32[shard_len]; param_out: 16-bit [shard_len] (bf16
    patterns); q_codes int8[shard_len] and q_scales float32[ceil(n/block)]
    when quantizing; gbar_ws float32[shard_len] optional (clipping spill).
    All on the current device.  ``stream`` is a torch stream (default: the
    current stream at construction)."""

    def __init__(self, *, phi: int, n_d: int, r: int, shard_len: int, master, m, v, param_out,
                 beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 weight_decay: float = 0.0, bias_correction: bool = True,
                 max_norm: float = 0.0, quant_block: int = 0, q_codes=None, q_scales=None,
                 gbar_ws=None, stream=None):
        if stream is None:
            import torch

            stream = torch.cuda.current_stream()
        self._keep = (master, m, v, param_out, q_codes, q_scales, gbar_ws, stream)
        self.desc = zs_desc(
            phi=int(phi), n_d=int(n_d), r=int(r), shard_len=int(shard_len),
            beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay,
            bias_correction=int(bool(bias_correction)), max_norm=max_norm,
            quant_block=int(quant_block), master=_ptr(master), m=_ptr(m), v=_ptr(v),
            param_out=_ptr(param_out), q_codes=_ptr(q_codes), q_scales=_ptr(q_scales),
            gbar_ws=_ptr(gbar_ws), stream=int(stream.cuda_stream))
        rc, self.h = zero_shard_init(self.desc)
        _check(rc, "zero_shard_init")

    def gnorm(self, contrib, sumsq_dev) -> None:
        _check(zero_shard_gnorm(self.h, contrib, sumsq_dev), "zero_shard_gnorm")

    def step(self, contrib, lr: float, t: int, global_sumsq_dev=None) -> None:
        _check(zero_shard_step(self.h, contrib, lr, t, global_sumsq_dev), "zero_shard_step")

    def step_dev(self, contrib, consts_dev, global_sumsq_dev=None) -> None:
        _check(zero_shard_step_dev(self.h, contrib, consts_dev, global_sumsq_dev),
               "zero_shard_step_dev")

    def consts(self, lr: float, t: int) -> list[float]:
        rc, out = zero_shard_step_consts(self.desc, lr, t)
        _check(rc, "zero_shard_step_consts")
        return out

    def gnorm_q8(self, codes, scales, block: int, sumsq_dev) -> None:
        _check(zero_shard_gnorm_q8(self.h, codes, scales, block, sumsq_dev), "zero_shard_gnorm_q8")

    def step_q8(self, codes, scales, block: int, lr: float, t: int, global_sumsq_dev=None) -> None:
        _check(zero_shard_step_q8(self.h, codes, scales, block, lr, t, global_sumsq_dev),
               "zero_shard_step_q8")

    def gnorm_bucketed(self, contrib, bucket_len: int, sumsq_dev, streams: int = 2,
                       ready=None) -> None:
        _check(zero_shard_gnorm_bucketed(self.h, contrib, bucket_len, streams, ready, sumsq_dev),
               "zero_shard_gnorm_bucketed")

    def step_bucketed(self, contrib, bucket_len: int, lr: float, t: int, global_sumsq_dev=None,
                      streams: int = 2, ready=None) -> None:
        _check(zero_shard_step_bucketed(self.h, contrib, bucket_len, streams, ready, lr, t,
                                        global_sumsq_dev), "zero_shard_step_bucketed")

    def gnorm_bucketed_q8(self, codes, scales, block: int, bucket_len: int, sumsq_dev,
                          streams: int = 2, ready=None) -> None:
        _check(zero_shard_gnorm_bucketed_q8(self.h, codes, scales, block, bucket_len, streams,
                                            ready, sumsq_dev), "zero_shard_gnorm_bucketed_q8")

    def step_bucketed_q8(self, codes, scales, block: int, bucket_len: int, lr: float, t: int,
                         global_sumsq_dev=None, streams: int = 2, ready=None) -> None:
        _check(zero_shard_step_bucketed_q8(self.h, codes, scales, block, bucket_len, streams,
                                           ready, lr, t, global_sumsq_dev),
               "zero_shard_step_bucketed_q8")

    def quant(self, block: int) -> None:
        _check(zero_shard_quant(self.h, block), "zero_shard_quant")

    def free(self) -> None:
        if self.h is not None and self.h.value:
            _check(zero_shard_free(self.h), "zero_shard_free")
        self.h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.free()

    def __del__(self):
        try:
            if getattr(self, "h", None) is not None and self.h.value:
                zero_shard_free(self.h)
        except Exception:
            pass


def _require(ok: bool, what: str) -> None:
    if not ok:
        raise ZeroShardError(ZS_EINVAL, what)


class ZeroLayerNorm:
    """Layer norm of (rows, cols) tensors, forward and backward, with the
    saved statistics and the workspace of the gradient reduction.

    All tensors are on the current device; x, residual, sum_out, y, dy, dsum
    and dx are (rows, cols) of ``dtype`` with column stride 1 and rows that do
    not overlap (an expanded tensor, such as autograd's gradient of ``y.sum(0)``,
    needs ``.contiguous()`` first), the parameters and their gradients contiguous
    (cols,) of ``param_dtype`` (default: dtype).  ``stream`` is a torch stream
    (default: the current one at construction)."""

    def __init__(self, *, rows: int, cols: int, dtype=torch.bfloat16, param_dtype=None,
                 eps: float = 1e-5, stream=None):
        self.dtype, self.param_dtype = dtype, dtype if param_dtype is None else param_dtype
        self.shape = (int(rows), int(cols))
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.desc = layernorm_desc(rows=rows, cols=cols, dtype=dtype, param_dtype=param_dtype,
                                   eps=eps, stream=self._stream)
        self._ref = ctypes.byref(self.desc)
        self._workspace_bytes = size = zero_shard_layernorm_workspace(self.desc)
        _require(size >= 0, "layer norm's sizes")
        with torch.cuda.stream(self._stream):
            self.mean = torch.empty(rows, device="cuda", dtype=torch.float32)
            self.rstd = torch.empty(rows, device="cuda", dtype=torch.float32)
            self.workspace = torch.empty(size, device="cuda", dtype=torch.uint8)

    def _row(self, t, what: str) -> int:
        """Row stride of a (rows, cols) tensor; 0 for None and a single row.
        Rows that share memory (expanded tensors have row stride 0, which the
        descriptor takes for cols) are refused."""
        if t is None:
            return 0
        rows, cols = self.shape
        if t.shape != self.shape or t.dtype is not self.dtype or not t.is_cuda:
            raise ZeroShardError(ZS_EINVAL, what)
        ld, unit = t.stride()
        if (unit != 1 and cols != 1) or (rows > 1 and ld < cols):
            raise ZeroShardError(ZS_EINVAL, what)
        return ld if rows > 1 else 0

    def _param(self, t, what: str) -> None:
        if (t.shape != self.shape[1:] or t.dtype is not self.param_dtype or not t.is_cuda
                or not t.is_contiguous()):
            raise ZeroShardError(ZS_EINVAL, what)

    def forward(self, x, y, *, gamma=None, beta=None, residual=None, sum_out=None) -> None:
        """y = LN(x), or LN(sum_out) with sum_out = x + residual; keeps the
        rows' mean and rstd for backward."""
        d = self.desc
        d.ld_x, d.ld_y = self._row(x, "x"), self._row(y, "y")
        d.ld_residual, d.ld_sum = self._row(residual, "residual"), self._row(sum_out, "sum_out")
        if gamma is not None:
            self._param(gamma, "gamma")
        if beta is not None:
            self._param(beta, "beta")
        rc = _lib.zero_shard_layernorm(self._ref, *_ptrs(x, residual, gamma, beta, sum_out, y,
                                                         self.mean, self.rstd))
        if rc:
            _check(rc, "zero_shard_layernorm")

    def backward(self, dy, x, dx, *, gamma=None, dgamma=None, dbeta=None, dsum=None, mean=None,
                 rstd=None) -> None:
        """x: what was normalised (sum_out with a residual); mean, rstd: the
        saved statistics (default: those of the last forward)."""
        d = self.desc
        d.ld_dy, d.ld_x = self._row(dy, "dy"), self._row(x, "x")
        d.ld_dx, d.ld_dsum = self._row(dx, "dx"), self._row(dsum, "dsum")
        for t, what in ((gamma, "gamma"), (dgamma, "dgamma"), (dbeta, "dbeta")):
            if t is not None:
                self._param(t, what)
        for t in (mean, rstd):
            _require(t is None or (t.shape == self.shape[:1] and t.dtype is torch.float32
                                   and t.is_cuda and t.is_contiguous()), "mean, rstd")
        rc = _lib.zero_shard_layernorm_bwd(
            self._ref, *_ptrs(dy, x, gamma, self.mean if mean is None else mean,
                              self.rstd if rstd is None else rstd, dsum, dx, dgamma, dbeta,
                              self.workspace), self._workspace_bytes)
        if rc:
            _check(rc, "zero_shard_layernorm_bwd")


class ZeroBlockNorm:
    """The seam between two blocks: the norm of a block's output (``post``), its
    gate, the scaled residual sum and the norm before the next block, forward
    and backward, with the saved statistics and the workspace of the gradients'
    reduction.

    ``kind``: "rms" or "layer", of both norms; ``gate``: "none", "column" (a
    (cols,) parameter) or "sigmoid" (a (rows, cols) tensor z, of which the
    sigmoid is taken).  Tensors, parameters and ``stream`` as for ZeroLayerNorm."""

    def __init__(self, *, rows: int, cols: int, dtype=torch.bfloat16, param_dtype=None,
                 kind: str = "rms", post: bool = True, gate: str = "none", eps: float = 1e-5,
                 residual_scale: float = 1.0, stream=None):
        self.dtype, self.param_dtype = dtype, dtype if param_dtype is None else param_dtype
        self.shape, self.gate = (int(rows), int(cols)), gate
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.desc = blocknorm_desc(rows=rows, cols=cols, dtype=dtype, param_dtype=param_dtype,
                                   kind=kind, post=post, gate=gate, eps=eps,
                                   residual_scale=residual_scale, stream=self._stream)
        self._ref = ctypes.byref(self.desc)
        self._workspace_bytes = size = zero_shard_blocknorm_workspace(self.desc)
        _require(size >= 0, "block norm's sizes")
        with torch.cuda.stream(self._stream):
            # rstd of the first norm and the second, then (layer) their means
            self.stats = torch.zeros(4 if kind == "layer" else 2, rows, device="cuda")
            self.workspace = torch.empty(size, device="cuda", dtype=torch.uint8)

    _row = ZeroLayerNorm._row
    _param = ZeroLayerNorm._param

    def _gate(self, t, what: str) -> int:
        """Row stride of an element gate or its gradient; 0 for other gates."""
        if t is None or self.gate == "sigmoid":
            return self._row(t, what)
        self._param(t, what)
        return 0

    def forward(self, x, block, sum_out, y, *, gate=None, gamma_post=None, beta_post=None,
                gamma=None, beta=None) -> None:
        """sum_out = residual_scale x + gate N(block), y = N(sum_out); keeps the
        rows' statistics for backward.  block and sum_out None: y = N(x)."""
        d = self.desc
        d.ld_x, d.ld_block = self._row(x, "x"), self._row(block, "block")
        d.ld_sum, d.ld_y = self._row(sum_out, "sum_out"), self._row(y, "y")
        d.ld_gate = self._gate(gate, "gate")
        for t, what in ((gamma_post, "gamma_post"), (beta_post, "beta_post"), (gamma, "gamma"),
                        (beta, "beta")):
            if t is not None:
                self._param(t, what)
        rc = _lib.zero_shard_blocknorm(self._ref, *_ptrs(x, block, gate, gamma_post, beta_post,
                                                         gamma, beta, sum_out, y, self.stats))
        if rc:
            _check(rc, "zero_shard_blocknorm")

    def backward(self, dy, total, block, dx, dblock, *, dsum=None, gate=None, gamma_post=None,
                 beta_post=None, gamma=None, dgate=None, dgamma_post=None, dbeta_post=None,
                 dgamma=None, dbeta=None, stats=None) -> None:
        """total: the forward pass's sum_out (x without a block); dsum: the
        gradient that reaches it from elsewhere; stats: the saved statistics
        (default: those of the last forward)."""
        d = self.desc
        d.ld_dy, d.ld_sum = self._row(dy, "dy"), self._row(total, "total")
        d.ld_block, d.ld_dsum = self._row(block, "block"), self._row(dsum, "dsum")
        d.ld_dx, d.ld_dblock = self._row(dx, "dx"), self._row(dblock, "dblock")
        d.ld_gate, d.ld_dgate = self._gate(gate, "gate"), self._gate(dgate, "dgate")
        for t, what in ((gamma_post, "gamma_post"), (beta_post, "beta_post"), (gamma, "gamma"),
                        (dgamma_post, "dgamma_post"), (dbeta_post, "dbeta_post"),
                        (dgamma, "dgamma"), (dbeta, "dbeta")):
            if t is not None:
                self._param(t, what)
        if stats is None:
            stats = self.stats
        else:
            _require(stats.shape == self.stats.shape and stats.dtype is torch.float32
                     and stats.is_cuda and stats.is_contiguous(), "stats")
        rc = _lib.zero_shard_blocknorm_bwd(
            self._ref, *_ptrs(dy, dsum, total, block, gate, gamma_post, beta_post, gamma, stats,
                              dx, dblock, dgate, dgamma_post, dbeta_post, dgamma, dbeta,
                              self.workspace), self._workspace_bytes)
        if rc:
            _check(rc, "zero_shard_blocknorm_bwd")


class ZeroEmbedding:
    """The embedding of tokens out of a (vocab, cols) table, scaled, and the
    gradient of the table, with its workspace.

    The table's rows stand for the ids ``first``, ``first`` + 1, ...; other ids
    give rows of zeros and no gradient (a table split over ranks); tokens of the id
    ``padding`` give no gradient.  ids: contiguous, ``tokens`` of them in any shape;
    y and dy: (tokens, cols) of ``dtype``; the table and its gradient of
    ``table_dtype`` and ``grad_dtype`` (default: dtype).  Column stride 1, no
    rows that overlap; ``stream`` as for ZeroLayerNorm."""

    def __init__(self, *, tokens: int, vocab: int, cols: int, dtype=torch.bfloat16,
                 table_dtype=None, grad_dtype=None, scale: float = 1.0, first: int = 0,
                 padding: int | None = None, id_dtype=torch.int64, stream=None):
        self.dtype, self.id_dtype = dtype, id_dtype
        self.table_dtype = dtype if table_dtype is None else table_dtype
        self.grad_dtype = dtype if grad_dtype is None else grad_dtype
        self.rows, self.shape = (int(vocab), int(cols)), (int(tokens), int(cols))
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.desc = embedding_desc(tokens=tokens, vocab=vocab, cols=cols, dtype=dtype,
                                   table_dtype=table_dtype, grad_dtype=grad_dtype, scale=scale,
                                   first=first, padding=padding, id_dtype=id_dtype,
                                   stream=self._stream)
        self._ref = ctypes.byref(self.desc)
        self._workspace_bytes = size = zero_shard_embedding_workspace(self.desc)
        _require(size >= 0, "embedding's sizes")
        self._workspace = None

    @property
    def workspace(self):
        """Of the backward pass, from its first call on (or this property's first use,
        which a program that captures its first backward pass makes before)."""
        if self._workspace is None:
            with torch.cuda.stream(self._stream):
                self._workspace = torch.empty(self._workspace_bytes, device="cuda",
                                              dtype=torch.uint8)
        return self._workspace

    def _ids(self, ids) -> None:
        if (ids.numel() != self.shape[0] or ids.dtype is not self.id_dtype or not ids.is_cuda
                or not ids.is_contiguous()):
            raise ZeroShardError(ZS_EINVAL, "ids")

    @staticmethod
    def _matrix(t, shape, dtype, what: str) -> int:
        """Row stride of a matrix; 0 for a single row."""
        if t.shape != shape or t.dtype is not dtype or not t.is_cuda:
            raise ZeroShardError(ZS_EINVAL, what)
        (rows, cols), (ld, unit) = shape, t.stride()
        if (unit != 1 and cols != 1) or (rows > 1 and ld < cols):
            raise ZeroShardError(ZS_EINVAL, what)
        return ld if rows > 1 else 0

    def forward(self, ids, table, y) -> None:
        """y = scale table[ids - first]."""
        d = self.desc
        self._ids(ids)
        d.ld_table = self._matrix(table, self.rows, self.table_dtype, "table")
        d.ld_y = self._matrix(y, self.shape, self.dtype, "y")
        rc = _lib.zero_shard_embedding(self._ref, *_ptrs(ids, table, y))
        if rc:
            _check(rc, "zero_shard_embedding")

    def backward(self, ids, dy, dtable, accumulate: bool = False) -> None:
        """dtable = the table's gradient (all of its rows), or, with
        ``accumulate``, dtable + that."""
        d = self.desc
        self._ids(ids)
        d.ld_dy = self._matrix(dy, self.shape, self.dtype, "dy")
        d.ld_dtable = self._matrix(dtable, self.rows, self.grad_dtype, "dtable")
        d.accumulate = 1 if accumulate else 0
        rc = _lib.zero_shard_embedding_bwd(self._ref, *_ptrs(ids, dy, dtable, self.workspace),
                                           self._workspace_bytes)
        if rc:
            _check(rc, "zero_shard_embedding_bwd")


class ZeroAdamW:
    """The AdamW step of a list of tensors (adamw_tensor), with the plan of them.

    The gradients of a call are a list of contiguous device tensors, one a tensor of its
    ``grad_dtype`` and length (None for an empty one), or a table of theirs that the
    caller keeps (contrib_table), which is checked as a list is when it is first given.
    ``max_norm`` > 0: gnorm, the all-reduce of its sum across ranks, then step with it.
    ``stream`` as for ZeroLayerNorm."""

    def __init__(self, tensors, *, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                 bias_correction: bool = True, max_norm: float = 0.0, stream=None):
        self.tensors = list(tensors)
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.desc = adamw_desc(count=len(self.tensors), beta1=beta1, beta2=beta2, eps=eps,
                               bias_correction=bias_correction, max_norm=max_norm,
                               stream=self._stream)
        self._ref = ctypes.byref(self.desc)
        array = (zs_adamw_tensor * max(1, len(self.tensors)))(*self.tensors)
        size = zero_shard_adamw_plan_bytes(self.desc, array)
        _require(size >= 0, "adamw's sizes")
        self.plan = torch.empty(size, dtype=torch.uint8)
        _check(zero_shard_adamw_plan(self.desc, array, self.plan), "zero_shard_adamw_plan")
        with torch.cuda.stream(self._stream):
            self.plan_dev = self.plan.to("cuda")
        self._args = (self._ref, self.plan.data_ptr(), self.plan_dev.data_ptr())

    def _grads(self, grads):
        if isinstance(grads, ctypes.Array):  # kept by the caller
            _require(hasattr(grads, "_keep"), "grads: not a table of contrib_table's")
            return _kept_table(grads, self, self._check_grads)
        grads = list(grads)
        self._check_grads(grads)
        return contrib_table(grads)

    def _check_grads(self, grads) -> None:
        _require(len(grads) == len(self.tensors), "grads")
        for g, t in zip(grads, self.tensors):
            if t.n or g is not None:
                _require(g is not None and g.numel() == t.n and g.is_cuda and g.is_contiguous()
                         and _DTYPES.get(g.dtype) == t.grad_dtype, "grads")

    @staticmethod
    def _double(t, n: int, what: str):
        if t is not None:
            _require(t.dtype is torch.float64 and t.numel() >= n and t.is_cuda
                     and t.is_contiguous(), what)
        return _ptr(t)

    def gnorm(self, grads, sumsq_dev) -> None:
        """The sum of squares of all gradients, to sumsq_dev (float64)."""
        _check(_lib.zero_shard_adamw_gnorm(*self._args, self._grads(grads),
                                           self._double(sumsq_dev, 1, "sumsq_dev")),
               "zero_shard_adamw_gnorm")

    def step(self, grads, lr: float, t: int, global_sumsq_dev=None, key: int | None = None) -> None:
        """Step t.  key: of the rounding of 8-bit states, another one each step
        (default: t)."""
        _check(_lib.zero_shard_adamw(*self._args, self._grads(grads), float(lr), int(t),
                                     (int(t) if key is None else int(key)) & 0xFFFFFFFF,
                                     self._double(global_sumsq_dev, 1, "global_sumsq_dev")),
               "zero_shard_adamw")

    def consts(self, lr: float, t: int, key: int | None = None) -> list[float]:
        rc, out = zero_shard_adamw_consts(self.desc, lr, t, t if key is None else key)
        _check(rc, "zero_shard_adamw_consts")
        return out

    def step_dev(self, grads, consts_dev, global_sumsq_dev=None) -> None:
        """The step of the constants that consts_dev (float64[4], see consts) holds
        when the kernel runs."""
        _check(_lib.zero_shard_adamw_dev(*self._args, self._grads(grads),
                                         self._double(consts_dev, 4, "consts_dev"),
                                         self._double(global_sumsq_dev, 1, "global_sumsq_dev")),
               "zero_shard_adamw_dev")


class ZeroOrtho:
    """Newton-Schulz orthogonalisation of (batch, rows, cols) tensors of
    ``dtype`` into bf16 ones, with its workspace; a 2-D tensor is a batch of
    one.  Column stride 1, no expanded rows or matrices; ``stream`` as for
    ZeroLayerNorm."""

    def __init__(self, *, batch: int = 1, rows: int, cols: int, dtype=torch.bfloat16,
                 steps: int = 5, coeffs=None, eps: float = 1e-7, stream=None):
        self.shape, self.dtype = (int(batch), int(rows), int(cols)), dtype
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.desc = ortho_desc(batch=batch, rows=rows, cols=cols, dtype=dtype, steps=steps,
                               coeffs=coeffs, eps=eps, stream=self._stream)
        size = zero_shard_ortho_workspace(self.desc)
        _require(size >= 0, "ortho's sizes")
        with torch.cuda.stream(self._stream):
            self.workspace = torch.empty(size, device="cuda", dtype=torch.uint8)

    def _strides(self, t, dtype, what: str) -> tuple[int, int]:
        """Row and matrix strides.  Expanded tensors are refused: their strides of
        0 are the dense ones to the descriptor."""
        b, r, c = self.shape
        _require((t.shape == self.shape or (b == 1 and t.shape == self.shape[1:]))
                 and t.dtype == dtype and t.is_cuda and (t.stride(-1) == 1 or c == 1), what)
        ld = t.stride(-2) if r > 1 else c
        each = t.stride(0) if b > 1 else r * ld
        _require(t.numel() == 0 or (ld > 0 and each > 0), what)
        return ld, each

    def __call__(self, g, o) -> None:
        """o = the orthogonalised g."""
        d = self.desc
        d.ld_in, d.stride_in = self._strides(g, self.dtype, "g")
        d.ld_out, d.stride_out = self._strides(o, torch.bfloat16, "o")
        _check(zero_shard_ortho(d, g, o, self.workspace), "zero_shard_ortho")


_BF16_LIKE = (torch.bfloat16, torch.int16, torch.uint16)  # bf16 or its patterns


class ZeroMuon:
    """One rank's Muon step over ``batch`` matrices of rows x cols that lie one
    after another in caller-owned torch tensors.

    master, momentum: float32[n]; param_out: bf16[n] (or its patterns as int16
    or uint16), n = batch * rows * cols, 16-byte aligned.  ``update_dtype``: of the
    momentum's update matrix (bf16 or float32).  ``scale``: the update's scale
    (default 0.2 sqrt(max(rows, cols)), which matches an Adam update's size)."""

    def __init__(self, *, n_d: int, rows: int, cols: int, master, momentum, param_out,
                 batch: int = 1, mu: float = 0.95, nesterov: bool = True,
                 weight_decay: float = 0.0, steps: int = 5, coeffs=None, eps: float = 1e-7,
                 scale: float | None = None, update_dtype=torch.bfloat16, stream=None):
        n = int(batch) * int(rows) * int(cols)
        for t, types, what in ((master, (torch.float32,), "master"),
                               (momentum, (torch.float32,), "momentum"),
                               (param_out, _BF16_LIKE, "param_out")):
            _require(t.numel() == n and t.dtype in types and t.is_contiguous() and t.is_cuda, what)
            if t.data_ptr() % 16:
                raise ZeroShardError(ZS_EALIGN, what)
        self._stream = torch.cuda.current_stream() if stream is None else stream
        self.master, self.momentum, self.param_out = master, momentum, param_out
        self.scale = 0.2 * max(rows, cols) ** 0.5 if scale is None else float(scale)
        self.desc = muon_desc(n=n, n_d=n_d, mu=mu, nesterov=nesterov, dtype=update_dtype,
                              weight_decay=weight_decay, stream=self._stream)
        self._no_elements = muon_desc(n=0, weight_decay=weight_decay, stream=self._stream)
        self.ortho = ZeroOrtho(batch=batch, rows=rows, cols=cols, dtype=update_dtype, steps=steps,
                               coeffs=coeffs, eps=eps, stream=self._stream)
        with torch.cuda.stream(self._stream):
            self.update = torch.empty(batch, rows, cols, device="cuda", dtype=update_dtype)
            self.o = torch.empty(batch, rows, cols, device="cuda", dtype=torch.bfloat16)

    def _table(self, contrib):
        """The table of n_d contributions, each n contiguous bf16 elements or more
        (a row may be padded at its end)."""
        if isinstance(contrib, ctypes.Array):  # kept by the caller
            _require(len(contrib) == self.desc.n_d, "contrib")
            # one that contrib_table did not make is addresses, which nothing is known of
            return (_kept_table(contrib, self, self._check_rows) if hasattr(contrib, "_keep")
                    else contrib)
        rows = list(contrib)  # also of a 2-D tensor
        self._check_rows(rows)
        return contrib_table(rows)

    def _check_rows(self, rows) -> None:
        n, n_d = self.desc.n, self.desc.n_d
        _require(len(rows) == n_d, "contrib")
        for r in rows:
            _require(r is not None and r.numel() >= n and r.dtype in _BF16_LIKE
                     and r.is_contiguous() and r.is_cuda, "contrib")

    def step(self, contrib, lr: float) -> None:
        """Momentum over the mean of the contributions, its orthogonalisation,
        and the weight update; param_out holds the bf16 weights.  contrib: n_d
        bf16[n] tensors (or their patterns; longer ones are read up to n), the rows
        of an (n_d, n) one, or a table of theirs (contrib_table)."""
        table = self._table(contrib)
        # the rate is refused before the momentum moves on: the weight update of
        # no elements checks it and does nothing else
        _check(zero_shard_muon_apply(self._no_elements, None, lr, self.scale, None, None, None),
               "lr, scale")
        _check(zero_shard_muon_momentum(self.desc, table, self.momentum, self.momentum,
                                        self.update), "zero_shard_muon_momentum")
        self.ortho(self.update, self.o)
        _check(zero_shard_muon_apply(self.desc, self.o, lr, self.scale, self.master, self.master,
                                     self.param_out), "zero_shard_muon_apply")
