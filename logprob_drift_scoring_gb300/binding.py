"""Thin Python binding of liblpd (include/lpd.h): same names, marshalling only.

Every function here converts torch tensors to the C structs and pointers of
the C ABI and calls the library; all arithmetic runs in the CUDA kernels.
There is no CPU or library fallback: if liblpd.so cannot be loaded (or
built), importing the binding fails.
"""
from __future__ import annotations

import ctypes
import functools
import inspect
from dataclasses import dataclass

from . import _build

# ---- constants (mirror include/lpd.h) --------------------------------------
LPD_BF16, LPD_F32 = 0, 1
LPD_E4M3, LPD_E5M2 = 2, 3  # block-scaled operands only
LPD_OK = 0
LPD_ERR_NULL_POINTER = -1
LPD_ERR_BAD_SIZE = -2
LPD_ERR_BAD_DTYPE = -3
LPD_ERR_BAD_STRIDE = -4
LPD_ERR_BAD_CLIP = -5
LPD_ERR_BAD_SHARDS = -6
LPD_ERR_WORKSPACE = -7
LPD_ERR_CUDA = -8
LPD_ERR_ALIGNMENT = -9
LPD_ERR_UNSUPPORTED = -10
LPD_ERR_BAD_TRANSFORM = -11
LPD_ERR_BAD_MEMORY = -12
LPD_OP_SCALE, LPD_OP_SOFTCAP = 1, 2
LPD_STATUS_TOKEN_OOB = 1
LPD_STATUS_NONFINITE = 2
LPD_STATUS_TIMEOUT = 4
LPD_FLAG_NO_ACTIVE = 1
LPD_FLAG_NO_PERCENTILES = 2
LPD_KIND_SCORE, LPD_KIND_SHARDED, LPD_KIND_CONTROLLED = 0, 1, 2
LPD_TOPO_ALLGATHER_PARTIALS_FIXED_MERGE, LPD_TOPO_ALLREDUCE_PARTIALS, LPD_TOPO_ALLGATHER_LOGITS = 0, 1, 2
TOPOLOGIES = {"allgather_partials_fixed_merge": 0, "allreduce_partials": 1, "allgather_logits": 2}


class LpdLogits(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_stride", ctypes.c_int64)]


class LpdShard(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("v_start", ctypes.c_int64), ("v_end", ctypes.c_int64)]


class LpdTransform(ctypes.Structure):
    _fields_ = [("n_ops", ctypes.c_int32), ("kind", ctypes.c_int32 * 4), ("param", ctypes.c_float * 4)]


def transform_struct(ops):
    """lpd_transform from [(kind, param), ...] applied in order; None for the identity."""
    if ops is None:
        return None
    t = LpdTransform()
    t.n_ops = len(ops)
    for i, (k, p) in enumerate(ops):
        t.kind[i] = k
        t.param[i] = p
    return t


class LpdControls(ctypes.Structure):
    _fields_ = [("history", ctypes.c_void_p), ("n_history", ctypes.c_int64), ("hist_begin", ctypes.c_void_p),
                ("hist_split", ctypes.c_void_p), ("hist_end", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("frequency", ctypes.c_void_p), ("presence", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("bias_ids", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("n_bias", ctypes.c_int64),
                ("mask", ctypes.c_void_p), ("n_masks", ctypes.c_int64), ("mask_stride", ctypes.c_int64),
                ("mask_row", ctypes.c_void_p)]


class LpdFilter(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_void_p), ("min_p", ctypes.c_void_p), ("top_k", ctypes.c_void_p),
                ("top_p", ctypes.c_void_p)]


class LpdBlockScaled(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("block", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("scales", ctypes.c_void_p), ("scale_stride", ctypes.c_int64)]


class LpdMicroScaled(ctypes.Structure):
    _fields_ = [("ptr", ctypes.c_void_p), ("block", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("row_stride", ctypes.c_int64), ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p)]


class LpdMetrics(ctypes.Structure):
    _fields_ = [("n_active", ctypes.c_int64), ("argmax_row", ctypes.c_int64), ("flags", ctypes.c_uint32),
                ("status", ctypes.c_uint32), ("ratio0_mean", ctypes.c_double), ("clipfrac0", ctypes.c_double),
                ("approx_kl0", ctypes.c_double), ("mean_abs_dlogp", ctypes.c_double),
                ("p95_abs_dlogp", ctypes.c_double), ("p99_abs_dlogp", ctypes.c_double),
                ("max_abs_dlogp", ctypes.c_double)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_}


class LpdBackendInfo(ctypes.Structure):
    _fields_ = [("backend_id", ctypes.c_char * 32), ("op_name", ctypes.c_char * 48), ("arch", ctypes.c_char * 16),
                ("dtypes", ctypes.c_char * 32), ("deterministic", ctypes.c_int32),
                ("batch_invariant", ctypes.c_int32), ("fast_math", ctypes.c_int32),
                ("has_fallback", ctypes.c_int32), ("fingerprint", ctypes.c_char * 96)]


METRICS_BYTES = ctypes.sizeof(LpdMetrics)


class LpdMergeDrift(ctypes.Structure):
    _fields_ = [("max_abs_dout", ctypes.c_double), ("max_abs_dlse", ctypes.c_double),
                ("row_dout", ctypes.c_int64), ("row_dlse", ctypes.c_int64), ("scratch", ctypes.c_uint64 * 2)]

    def as_dict(self) -> dict:
        return {"max_abs_dout": self.max_abs_dout, "max_abs_dlse": self.max_abs_dlse,
                "row_dout": self.row_dout, "row_dlse": self.row_dlse}


MERGE_DRIFT_BYTES = ctypes.sizeof(LpdMergeDrift)


class LpdLogpDrift(ctypes.Structure):
    _fields_ = [("max_abs_dlogp_train", ctypes.c_double), ("max_abs_dlogp_rollout", ctypes.c_double),
                ("row_train", ctypes.c_int64), ("row_rollout", ctypes.c_int64), ("n_active", ctypes.c_int64),
                ("n_differ", ctypes.c_int64), ("frac_differ", ctypes.c_double), ("scratch", ctypes.c_uint64 * 4)]

    def as_dict(self) -> dict:
        return {name: getattr(self, name) for name, _ in self._fields_ if name != "scratch"}


LOGP_DRIFT_BYTES = ctypes.sizeof(LpdLogpDrift)

# every symbol include/lpd.h declares
EXPORTED = ("lpd_workspace_size", "lpd_backend_info", "lpd_strerror", "lpd_score", "lpd_score_host",
            "lpd_select_active",
            "lpd_token_logp", "lpd_drift_metrics", "lpd_score_sharded", "lpd_score_noalloc",
            "lpd_fused_workspace_size", "lpd_score_fused", "lpd_score_fused_transformed", "lpd_score_transformed",
            "lpd_score_entropy", "lpd_logprob_backward", "lpd_attn_merge", "lpd_attn_merge_order_drift",
            "lpd_topology_workspace_size", "lpd_score_sharded_topology", "lpd_drift_metrics_from_dlogp",
            "lpd_logp_drift_summary", "lpd_merge_rank_metrics", "lpd_controls_apply", "lpd_score_controlled",
            "lpd_logprob_backward_controlled", "lpd_sample", "lpd_filter_mask", "lpd_block_quantize",
            "lpd_block_workspace_size", "lpd_block_matmul", "lpd_micro_scale_bytes", "lpd_micro_quantize",
            "lpd_micro_workspace_size", "lpd_micro_matmul")
LPD_MAX_BIAS = 1024
LPD_SAMPLE_MAX_VOCAB = 393216
LPD_NOALLOC_MAX_ROWS = 32768
LPD_ATTN_MAX_PARTS = 64


class LpdError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {lib().lpd_strerror(code).decode()} (code {code})")


_LIB: ctypes.CDLL | None = None


def lib() -> ctypes.CDLL:
    """The loaded liblpd.so (built in-tree on first use if nvcc is present)."""
    global _LIB
    if _LIB is None:
        path = _build.build()
        L = ctypes.CDLL(str(path))
        P, I32, I64, SZ, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_double
        L.lpd_workspace_size.restype = SZ
        L.lpd_workspace_size.argtypes = [I32, I64, I64, I32]
        L.lpd_backend_info.restype = ctypes.c_int
        L.lpd_backend_info.argtypes = [P]
        L.lpd_strerror.restype = ctypes.c_char_p
        L.lpd_strerror.argtypes = [ctypes.c_int]
        L.lpd_score.restype = ctypes.c_int
        L.lpd_score.argtypes = [P, P, I64, I64, P, P, D, D, P, P, P, P, P, SZ, P]
        L.lpd_select_active.restype = ctypes.c_int
        L.lpd_select_active.argtypes = [I64, P, P, P, P, P, P, P, SZ, P]
        L.lpd_token_logp.restype = ctypes.c_int
        L.lpd_token_logp.argtypes = [P, P, I64, I64, P, P, P, P, P, SZ, P]
        L.lpd_drift_metrics.restype = ctypes.c_int
        L.lpd_drift_metrics.argtypes = [I64, D, D, P, P, SZ, P]
        L.lpd_score_sharded.restype = ctypes.c_int
        L.lpd_score_sharded.argtypes = [P, P, I32, I64, I64, P, P, D, D, P, P, P, P, P, P, P, P, SZ, P]
        L.lpd_fused_workspace_size.restype = SZ
        L.lpd_fused_workspace_size.argtypes = [I64, I64, I64]
        L.lpd_score_fused.restype = ctypes.c_int
        L.lpd_score_fused.argtypes = [P, P, P, I64, I64, I64, P, P, D, D, P, P, P, P, P, SZ, P]
        L.lpd_score_fused_transformed.restype = ctypes.c_int
        L.lpd_score_fused_transformed.argtypes = [P, P, P, P, P, I64, I64, I64, P, P, D, D, P, P, P, P, P, SZ, P]
        L.lpd_score_host.restype = ctypes.c_int
        L.lpd_score_host.argtypes = [P, P, P, P, I64, I64, P, P, P, P, D, D, P, P, P, P, P, SZ, P, P]
        L.lpd_score_transformed.restype = ctypes.c_int
        L.lpd_score_transformed.argtypes = [P, P, P, P, I64, I64, P, P, D, D, P, P, P, P, P, SZ, P]
        L.lpd_score_entropy.restype = ctypes.c_int
        L.lpd_score_entropy.argtypes = [P, P, I64, I64, P, P, D, D, P, P, P, P, P, P, P, SZ, P]
        L.lpd_logprob_backward.restype = ctypes.c_int
        L.lpd_logprob_backward.argtypes = [P, I64, I64, P, P, P, P, P, I32, I64, P]
        L.lpd_score_noalloc.restype = ctypes.c_int
        L.lpd_score_noalloc.argtypes = [P, P, I64, I64, P, P, D, D, P, P, P, P, P]
        L.lpd_drift_metrics_from_dlogp.restype = ctypes.c_int
        L.lpd_drift_metrics_from_dlogp.argtypes = [I64, P, P, D, D, P, P, SZ, P]
        L.lpd_topology_workspace_size.restype = SZ
        L.lpd_topology_workspace_size.argtypes = [I32, I64, I64, I32, I32, I32]
        L.lpd_score_sharded_topology.restype = ctypes.c_int
        L.lpd_score_sharded_topology.argtypes = [P, P, I32, I64, I64, P, P, D, D, I32, P, P, P, P, P, P, SZ, P]
        L.lpd_attn_merge.restype = ctypes.c_int
        L.lpd_attn_merge.argtypes = [P, I32, P, I32, I64, I32, I32, P, P, P, P]
        L.lpd_attn_merge_order_drift.restype = ctypes.c_int
        L.lpd_attn_merge_order_drift.argtypes = [P, I32, P, I32, I64, I32, I32, P, P, P, P, P, P, P, P]
        L.lpd_logp_drift_summary.restype = ctypes.c_int
        L.lpd_merge_rank_metrics.restype = ctypes.c_int
        L.lpd_merge_rank_metrics.argtypes = [P, P, I32, P]
        L.lpd_logp_drift_summary.argtypes = [I64, P, P, P, P, P, P, P]
        L.lpd_block_quantize.restype = ctypes.c_int
        L.lpd_block_quantize.argtypes = [P, I32, I64, I64, I64, I32, I32, P, P]
        L.lpd_block_workspace_size.restype = SZ
        L.lpd_block_workspace_size.argtypes = [I64, I64, I64]
        L.lpd_block_matmul.restype = ctypes.c_int
        L.lpd_block_matmul.argtypes = [P, P, I64, I64, I64, P, I32, I64, P, SZ, P]
        L.lpd_micro_scale_bytes.restype = SZ
        L.lpd_micro_scale_bytes.argtypes = [I32, I64, I64]
        L.lpd_micro_quantize.restype = ctypes.c_int
        L.lpd_micro_quantize.argtypes = [P, I32, I64, I64, I64, I32, P, P, I32, I64, P]
        L.lpd_micro_workspace_size.restype = SZ
        L.lpd_micro_workspace_size.argtypes = [I64, I64, I64]
        L.lpd_micro_matmul.restype = ctypes.c_int
        L.lpd_micro_matmul.argtypes = [P, P, I64, I64, I64, P, I32, I64, P, SZ, P]
        L.lpd_sample.restype = ctypes.c_int
        L.lpd_sample.argtypes = [P, P, I64, I64, P, P, P, P, P]
        L.lpd_filter_mask.restype = ctypes.c_int
        L.lpd_filter_mask.argtypes = [P, P, I64, I64, P, P, P, I64, P, P, P]
        L.lpd_controls_apply.restype = ctypes.c_int
        L.lpd_controls_apply.argtypes = [P, P, I64, I64, P, I32, I64, P]
        L.lpd_score_controlled.restype = ctypes.c_int
        L.lpd_score_controlled.argtypes = [P, P, P, P, I64, I64, P, P, D, D, P, P, P, P, P, SZ, P]
        L.lpd_logprob_backward_controlled.restype = ctypes.c_int
        L.lpd_logprob_backward_controlled.argtypes = [P, P, I64, I64, P, P, P, P, P, I32, I64, P]
        _LIB = L
    return _LIB


# ---- marshalling helpers ----------------------------------------------------

def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return LPD_BF16
    if t.dtype == torch.float32:
        return LPD_F32
    return 99  # rejected by the library with LPD_ERR_BAD_DTYPE


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        # (The handle alone, where this torch gives it: making a Stream object of it takes 3 us, a
        # fifth of a small call.  The name is not a public one.)
        handle = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        return handle(torch.cuda.current_device()) if handle else torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


def _with_its_stream(form):
    """A form that allocates: on a stream of the caller's, what it allocates belongs to that
    stream, and what it reads back is read there.  (Memory of torch's current stream may still be
    in use there, and is given out again there as soon as the form lets go of it.)"""
    at = list(inspect.signature(form).parameters).index("stream")

    @functools.wraps(form)
    def call(*args, **kwargs):
        stream = args[at] if len(args) > at else kwargs.get("stream")
        if stream is None:
            return form(*args, **kwargs)
        import torch

        if not isinstance(stream, torch.cuda.Stream):  # a handle, of the device of the call's tensors
            given = [*args, *kwargs.values()]
            given = sum(([*v] if isinstance(v, (list, tuple)) else [v] for v in given), [])
            given = [getattr(v, name, None) for v in given for name in ("codes", "values")] + given
            device = next(t.device for t in given if isinstance(t, torch.Tensor))
            stream = torch.cuda.ExternalStream(getattr(stream, "cuda_stream", stream), device=device)
        with torch.cuda.stream(stream):
            return form(*args, **kwargs)

    return call


def _row_stride(t) -> int:
    """Elements between the rows of a 2-D tensor.  A single row's stride has no
    meaning in torch, so where it is too small its width serves; rows that overlap
    or repeat keep theirs, which the library refuses (LPD_ERR_BAD_STRIDE)."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def logits_struct(t) -> LpdLogits:
    """lpd_logits for a 2-D tensor with unit column stride (rows may be padded)."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("logits must be 2-D with contiguous columns")
    return LpdLogits(t.data_ptr(), _dtype_code(t), 0, t.stride(0))


def shard_array(shards, v_ranges):
    arr = (LpdShard * len(shards))()
    for i, (t, (v0, v1)) in enumerate(zip(shards, v_ranges)):
        if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
            raise ValueError("shard logits must be 2-D with contiguous columns")
        arr[i] = LpdShard(t.data_ptr(), _dtype_code(t), 0, t.stride(0), int(v0), int(v1))
    return arr


def _check(rc: int, where: str) -> None:
    if rc != LPD_OK:
        raise LpdError(rc, where)


# ---- the C ABI, one Python function per entry point ---------------------------

def lpd_workspace_size(kind: int, n_rows: int, vocab: int = 0, n_shards: int = 0) -> int:
    return int(lib().lpd_workspace_size(kind, n_rows, vocab, n_shards))


def lpd_backend_info() -> dict:
    info = LpdBackendInfo()
    _check(lib().lpd_backend_info(ctypes.byref(info)), "lpd_backend_info")
    out = {}
    for name, _ in info._fields_:
        v = getattr(info, name)
        out[name] = v.decode() if isinstance(v, bytes) else v
    return out


def lpd_strerror(code: int) -> str:
    return lib().lpd_strerror(code).decode()


def lpd_score(train, rollout, token_ids, action_mask, clip_lo, clip_hi, out_logp_train, out_logp_rollout,
              out_dlogp, out_metrics, workspace, stream=None) -> None:
    t, r = logits_struct(train), logits_struct(rollout)
    rc = lib().lpd_score(ctypes.byref(t), ctypes.byref(r), train.shape[0], train.shape[1], _ptr(token_ids),
                         _ptr(action_mask), float(clip_lo), float(clip_hi), _ptr(out_logp_train),
                         _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics), _ptr(workspace),
                         workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(rc, "lpd_score")


def lpd_score_host(train_host, rollout_host, token_ids_host, action_mask_host, clip_lo, clip_hi, train_dev,
                   rollout_dev, token_ids_dev, action_mask_dev, out_logp_train, out_logp_rollout, out_dlogp,
                   out_metrics, workspace, stream=None) -> int:
    """lpd_score_host: host tensors in, device staging and outputs; returns
    the bytes copied to the device."""
    th, rh = logits_struct(train_host), logits_struct(rollout_host)
    td, rd = logits_struct(train_dev), logits_struct(rollout_dev)
    copied = ctypes.c_int64(0)
    rc = lib().lpd_score_host(ctypes.byref(th), ctypes.byref(rh), ctypes.byref(td), ctypes.byref(rd),
                              train_host.shape[0], train_host.shape[1], _ptr(token_ids_host), _ptr(action_mask_host),
                              _ptr(token_ids_dev), _ptr(action_mask_dev), float(clip_lo), float(clip_hi),
                              _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics),
                              _ptr(workspace), workspace.numel() if workspace is not None else 0,
                              ctypes.byref(copied), _stream(stream))
    _check(rc, "lpd_score_host")
    return int(copied.value)


def lpd_score_transformed(train, rollout, train_ops, rollout_ops, token_ids, action_mask, clip_lo, clip_hi,
                          out_logp_train, out_logp_rollout, out_dlogp, out_metrics, workspace, stream=None) -> None:
    t, r = logits_struct(train), logits_struct(rollout)
    ct, cr = transform_struct(train_ops), transform_struct(rollout_ops)
    rc = lib().lpd_score_transformed(ctypes.byref(t), ctypes.byref(r), ctypes.byref(ct) if ct else None,
                                     ctypes.byref(cr) if cr else None, train.shape[0], train.shape[1],
                                     _ptr(token_ids), _ptr(action_mask), float(clip_lo), float(clip_hi),
                                     _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "lpd_score_transformed")


def lpd_score_entropy(train, rollout, token_ids, action_mask, clip_lo, clip_hi, out_logp_train, out_logp_rollout,
                      out_dlogp, out_entropy_train, out_entropy_rollout, out_metrics, workspace, stream=None) -> None:
    t, r = logits_struct(train), logits_struct(rollout)
    rc = lib().lpd_score_entropy(ctypes.byref(t), ctypes.byref(r), train.shape[0], train.shape[1], _ptr(token_ids),
                                 _ptr(action_mask), float(clip_lo), float(clip_hi), _ptr(out_logp_train),
                                 _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_entropy_train),
                                 _ptr(out_entropy_rollout), _ptr(out_metrics), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(rc, "lpd_score_entropy")


def lpd_logprob_backward(logits, token_ids, action_mask, logp, grad_logp, out_dlogits, stream=None) -> None:
    x = logits_struct(logits)
    if out_dlogits.dim() != 2 or (out_dlogits.shape[1] > 1 and out_dlogits.stride(1) != 1):
        raise ValueError("out_dlogits must be 2-D with contiguous columns")
    rc = lib().lpd_logprob_backward(ctypes.byref(x), logits.shape[0], logits.shape[1], _ptr(token_ids),
                                    _ptr(action_mask), _ptr(logp), _ptr(grad_logp), _ptr(out_dlogits),
                                    _dtype_code(out_dlogits), out_dlogits.stride(0), _stream(stream))
    _check(rc, "lpd_logprob_backward")


def lpd_select_active(token_ids, action_mask, out_logp_train, out_logp_rollout, out_dlogp, out_metrics, workspace,
                      stream=None) -> None:
    n = action_mask.shape[0]
    rc = lib().lpd_select_active(n, _ptr(token_ids), _ptr(action_mask), _ptr(out_logp_train), _ptr(out_logp_rollout),
                                 _ptr(out_dlogp), _ptr(out_metrics), _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    _check(rc, "lpd_select_active")


def lpd_token_logp(train, rollout, out_logp_train, out_logp_rollout, out_dlogp, out_metrics, workspace,
                   stream=None) -> None:
    t, r = logits_struct(train), logits_struct(rollout)
    rc = lib().lpd_token_logp(ctypes.byref(t), ctypes.byref(r), train.shape[0], train.shape[1],
                              _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics),
                              _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "lpd_token_logp")


def lpd_drift_metrics(n_rows, clip_lo, clip_hi, out_metrics, workspace, stream=None) -> None:
    rc = lib().lpd_drift_metrics(n_rows, float(clip_lo), float(clip_hi), _ptr(out_metrics), _ptr(workspace),
                                 workspace.numel(), _stream(stream))
    _check(rc, "lpd_drift_metrics")


def lpd_score_sharded(train_shards, rollout_shards, v_ranges, token_ids, action_mask, clip_lo, clip_hi,
                      merge_perm, out_logp_train, out_logp_rollout, out_dlogp, out_perm_logp_train,
                      out_perm_logp_rollout, out_metrics, workspace, stream=None) -> None:
    ts, rs = shard_array(train_shards, v_ranges), shard_array(rollout_shards, v_ranges)
    n_rows = train_shards[0].shape[0]
    vocab = max(v1 for _, v1 in v_ranges)
    perm = None
    if merge_perm is not None:
        perm = (ctypes.c_int32 * len(merge_perm))(*[int(k) for k in merge_perm])
    rc = lib().lpd_score_sharded(ts, rs, len(train_shards), n_rows, vocab, _ptr(token_ids), _ptr(action_mask),
                                 float(clip_lo), float(clip_hi), perm, _ptr(out_logp_train), _ptr(out_logp_rollout),
                                 _ptr(out_dlogp), _ptr(out_perm_logp_train), _ptr(out_perm_logp_rollout),
                                 _ptr(out_metrics), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "lpd_score_sharded")


def lpd_drift_metrics_from_dlogp(dlogp, action_mask, clip_lo, clip_hi, out_metrics, workspace, stream=None) -> None:
    rc = lib().lpd_drift_metrics_from_dlogp(dlogp.shape[0], _ptr(dlogp), _ptr(action_mask), float(clip_lo),
                                            float(clip_hi), _ptr(out_metrics), _ptr(workspace), workspace.numel(),
                                            _stream(stream))
    _check(rc, "lpd_drift_metrics_from_dlogp")


@_with_its_stream
def drift_metrics_from_dlogp(dlogp, action_mask, clip=(0.8, 1.2), stream=None) -> dict:
    """The metrics record of given per-token dlogp (float32, device) over the active rows."""
    import torch

    dev = dlogp.device
    met = torch.empty(METRICS_BYTES, dtype=torch.uint8, device=dev)
    ws = torch.empty(lpd_workspace_size(LPD_KIND_SCORE, dlogp.shape[0]), dtype=torch.uint8, device=dev)
    lpd_drift_metrics_from_dlogp(dlogp, action_mask, clip[0], clip[1], met, ws, stream)
    return read_metrics(met)


def lpd_topology_workspace_size(topology: int, n_rows: int, vocab: int, n_shards: int, dtype_train: int,
                                dtype_rollout: int) -> int:
    return int(lib().lpd_topology_workspace_size(topology, n_rows, vocab, n_shards, dtype_train, dtype_rollout))


def lpd_score_sharded_topology(train_shards, rollout_shards, v_ranges, token_ids, action_mask, clip_lo, clip_hi,
                               topology, reduce_order, out_logp_train, out_logp_rollout, out_dlogp, out_metrics,
                               workspace, stream=None) -> None:
    ts, rs = shard_array(train_shards, v_ranges), shard_array(rollout_shards, v_ranges)
    n_rows = train_shards[0].shape[0]
    vocab = max(v1 for _, v1 in v_ranges)
    order = None
    if reduce_order is not None:
        order = (ctypes.c_int32 * len(reduce_order))(*[int(k) for k in reduce_order])
    rc = lib().lpd_score_sharded_topology(ts, rs, len(train_shards), n_rows, vocab, _ptr(token_ids),
                                          _ptr(action_mask), float(clip_lo), float(clip_hi), int(topology), order,
                                          _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp),
                                          _ptr(out_metrics), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(rc, "lpd_score_sharded_topology")


def lpd_fused_workspace_size(n_rows: int, hidden: int, vocab: int) -> int:
    return int(lib().lpd_fused_workspace_size(n_rows, hidden, vocab))


def lpd_score_fused(hidden_train, hidden_rollout, W, token_ids, action_mask, clip_lo, clip_hi, out_logp_train,
                    out_logp_rollout, out_dlogp, out_metrics, workspace, stream=None) -> None:
    n_rows, hidden = hidden_train.shape
    rc = lib().lpd_score_fused(_ptr(hidden_train), _ptr(hidden_rollout), _ptr(W), n_rows, hidden, W.shape[0],
                               _ptr(token_ids), _ptr(action_mask), float(clip_lo), float(clip_hi),
                               _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics),
                               _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(rc, "lpd_score_fused")


def lpd_score_fused_transformed(hidden_train, hidden_rollout, W, train_ops, rollout_ops, token_ids, action_mask,
                                clip_lo, clip_hi, out_logp_train, out_logp_rollout, out_dlogp, out_metrics, workspace,
                                stream=None) -> None:
    n_rows, hidden = hidden_train.shape
    ct, cr = transform_struct(train_ops), transform_struct(rollout_ops)
    rc = lib().lpd_score_fused_transformed(
        _ptr(hidden_train), _ptr(hidden_rollout), _ptr(W), ctypes.byref(ct) if ct else None,
        ctypes.byref(cr) if cr else None, n_rows, hidden, W.shape[0], _ptr(token_ids), _ptr(action_mask),
        float(clip_lo), float(clip_hi), _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp),
        _ptr(out_metrics), _ptr(workspace), workspace.numel() if workspace is not None else 0, _stream(stream))
    _check(rc, "lpd_score_fused_transformed")


def lpd_score_noalloc(train, rollout, token_ids, action_mask, clip_lo, clip_hi, out_logp_train, out_logp_rollout,
                      out_dlogp, out_metrics, stream=None) -> None:
    """lpd_score with the library's built-in scratch instead of a workspace
    (for callers that cannot allocate device memory; n_rows <= 32768)."""
    t, r = logits_struct(train), logits_struct(rollout)
    rc = lib().lpd_score_noalloc(ctypes.byref(t), ctypes.byref(r), train.shape[0], train.shape[1], _ptr(token_ids),
                                 _ptr(action_mask), float(clip_lo), float(clip_hi), _ptr(out_logp_train),
                                 _ptr(out_logp_rollout), _ptr(out_dlogp), _ptr(out_metrics), _stream(stream))
    _check(rc, "lpd_score_noalloc")


def _order(order, n_parts):
    if order is None:
        return None
    order = [int(k) for k in order]
    if len(order) != n_parts:
        raise ValueError(f"order has {len(order)} entries for {n_parts} parts")
    return (ctypes.c_int32 * n_parts)(*order)


def _parts_shape(out_parts, lse_parts):
    if out_parts.dim() != 3 or not out_parts.is_contiguous() or not lse_parts.is_contiguous():
        raise ValueError("out_parts must be a dense [K, n_rows, head_dim] tensor and lse_parts dense [K, n_rows]")
    K, n, d = out_parts.shape
    if tuple(lse_parts.shape) != (K, n):
        raise ValueError("lse_parts must be [K, n_rows]")
    return K, n, d


def lpd_attn_merge(out_parts, lse_parts, order, out, out_lse, lse_base2=False, stream=None) -> None:
    K, n, d = _parts_shape(out_parts, lse_parts)
    rc = lib().lpd_attn_merge(_ptr(out_parts), _dtype_code(out_parts), _ptr(lse_parts), K, n, d, int(bool(lse_base2)),
                              _order(order, K), _ptr(out), _ptr(out_lse), _stream(stream))
    _check(rc, "lpd_attn_merge")


def lpd_attn_merge_order_drift(out_parts, lse_parts, order_a, order_b, out, out_lse, row_dout, row_dlse, drift,
                               lse_base2=False, stream=None) -> None:
    K, n, d = _parts_shape(out_parts, lse_parts)
    rc = lib().lpd_attn_merge_order_drift(_ptr(out_parts), _dtype_code(out_parts), _ptr(lse_parts), K, n, d,
                                          int(bool(lse_base2)), _order(order_a, K), _order(order_b, K), _ptr(out),
                                          _ptr(out_lse), _ptr(row_dout), _ptr(row_dlse), _ptr(drift), _stream(stream))
    _check(rc, "lpd_attn_merge_order_drift")


def lpd_logp_drift_summary(logp_train_a, logp_rollout_a, logp_train_b, logp_rollout_b, action_mask, out,
                           stream=None) -> None:
    """Merge-order drift summary of per-token result b against result a over
    the active rows (device float32 [n] each, uint8 mask, out: a device buffer
    of LOGP_DRIFT_BYTES)."""
    n = action_mask.shape[0]
    for x in (logp_train_a, logp_rollout_a, logp_train_b, logp_rollout_b):
        if x.shape[0] != n:
            raise ValueError("per-token results and mask must have the same length")
    rc = lib().lpd_logp_drift_summary(n, _ptr(logp_train_a), _ptr(logp_rollout_a), _ptr(logp_train_b),
                                      _ptr(logp_rollout_b), _ptr(action_mask), _ptr(out), _stream(stream))
    _check(rc, "lpd_logp_drift_summary")


@dataclass(frozen=True)
class Controls:
    """One side's sampling controls as device tensors (lpd_controls; None leaves
    a step out).  Row arrays have one entry a logits row: hist_begin, hist_split
    and hist_end int64 into history int32; repetition, frequency, presence and
    scale float32; bias_ids int32 and bias float32 [rows, n_bias]; mask int32
    [n_masks, words] with bit j % 32 of word j / 32 set where token j is
    allowed; mask_row int32.  The tensors must live as long as this object."""
    history: object = None
    hist_begin: object = None
    hist_split: object = None
    hist_end: object = None
    repetition: object = None
    frequency: object = None
    presence: object = None
    scale: object = None
    bias_ids: object = None
    bias: object = None
    mask: object = None
    mask_row: object = None

    def __post_init__(self):
        import torch

        kinds = {"history": torch.int32, "hist_begin": torch.int64, "hist_split": torch.int64,
                 "hist_end": torch.int64, "repetition": torch.float32, "frequency": torch.float32,
                 "presence": torch.float32, "scale": torch.float32, "bias_ids": torch.int32, "bias": torch.float32,
                 "mask": torch.int32, "mask_row": torch.int32}
        rows, device = None, None
        for name, kind in kinds.items():
            t = getattr(self, name)
            if t is None:
                continue
            if t.dtype != kind:
                raise ValueError(f"{name} must be {kind}, got {t.dtype}")
            if device is not None and t.device != device:
                raise ValueError(f"{name} is on {t.device}, the other controls on {device}")
            device = t.device
            if t.dim() != (2 if name in ("bias_ids", "bias", "mask") else 1):
                raise ValueError(f"{name} has {t.dim()} dimensions")
            if name == "mask":
                if t.numel() and t.shape[1] > 1 and t.stride(1) != 1:
                    raise ValueError("mask must have contiguous words")
            elif not t.is_contiguous():
                raise ValueError(f"{name} must be dense")
            if name not in ("history", "mask"):
                if rows is not None and t.shape[0] != rows:
                    raise ValueError(f"{name} has {t.shape[0]} rows, the other controls {rows}")
                rows = t.shape[0]
        if self.history is not None and None in (self.hist_begin, self.hist_split, self.hist_end):
            raise ValueError("history needs hist_begin, hist_split and hist_end")
        if (self.bias_ids is None) != (self.bias is None):
            raise ValueError("bias_ids and bias go together")
        if self.bias is not None and self.bias.shape != self.bias_ids.shape:
            raise ValueError("bias and bias_ids must have one shape")
        m = self.mask
        n = lambda t: t.shape[0] if t is not None else 0  # noqa: E731
        # A table of no rows has no memory in torch, and NULL would mean "no
        # mask": it gets an address, through which nothing is read.
        mask_ptr = (m.data_ptr() or 256) if m is not None else None
        struct = LpdControls(_ptr(self.history), n(self.history), _ptr(self.hist_begin), _ptr(self.hist_split),
                             _ptr(self.hist_end), _ptr(self.repetition), _ptr(self.frequency), _ptr(self.presence),
                             _ptr(self.scale), _ptr(self.bias_ids), _ptr(self.bias),
                             self.bias.shape[1] if self.bias is not None else 0, mask_ptr, n(m),
                             (m.stride(0) if m.shape[0] > 1 else m.shape[1]) if m is not None else 0,
                             _ptr(self.mask_row))
        object.__setattr__(self, "_struct", struct)
        object.__setattr__(self, "_rows", rows)
        object.__setattr__(self, "_device", device)


def _controls(c, logits):
    """Pointer to the side's lpd_controls (None: no controls) after the checks
    that only the tensors allow."""
    if c is None:
        return None
    if c._rows is not None and c._rows != logits.shape[0]:
        raise ValueError(f"controls of {c._rows} rows for {logits.shape[0]} logits rows")
    if c._device is not None and c._device != logits.device:
        raise ValueError(f"controls on {c._device}, logits on {logits.device}")
    words = -(-logits.shape[1] // 32)
    if c.mask is not None and c.mask.shape[1] < words:
        # (the library sees the stride between rows only, which a slice keeps)
        raise ValueError(f"mask has {c.mask.shape[1]} words a row, {logits.shape[1]} columns need {words}")
    return ctypes.byref(c._struct)


def _same_rows(n, device, **tensors):
    for name, (t, kind) in tensors.items():
        if t is None:
            continue
        if t.dtype != kind or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous() or t.device != device:
            raise ValueError(f"{name} must be a dense {kind} tensor of {n} values on {device}")


def _bytes(t) -> int:
    return t.numel() * t.element_size() if t is not None else 0


def _buffer(name, t, device, size=0):
    """A dense tensor's storage that the library writes as bytes (None: its own check)."""
    if t is not None and (not t.is_contiguous() or t.device != device or _bytes(t) < size):
        raise ValueError(f"{name} must be a dense tensor on {device}, of {size} bytes at least")


class _on:
    """The device of the call's tensors made current, where it is not."""

    def __init__(self, t):
        import torch

        if not t.is_cuda:
            raise ValueError("the tensors must be in device memory")
        self._guard = None if t.device.index == torch.cuda.current_device() else torch.cuda.device(t.device)

    def __enter__(self):
        if self._guard is not None:
            self._guard.__enter__()

    def __exit__(self, *exc):
        if self._guard is not None:
            self._guard.__exit__(*exc)


def lpd_controls_apply(logits, controls, out, stream=None) -> None:
    """The controlled logits of every row into `out` (bf16 or f32; may be `logits`)."""
    x, o = logits_struct(logits), logits_struct(out)
    if out.shape != logits.shape or out.device != logits.device:
        raise ValueError("out must have the logits' shape and device")
    c = _controls(controls, logits)
    with _on(logits):
        rc = lib().lpd_controls_apply(ctypes.byref(x), c, logits.shape[0], logits.shape[1], o.ptr, o.dtype,
                                      o.row_stride, _stream(stream))
    _check(rc, "lpd_controls_apply")


def lpd_score_controlled(train, rollout, train_controls, rollout_controls, token_ids, action_mask, clip_lo, clip_hi,
                         out_logp_train, out_logp_rollout, out_dlogp, out_metrics, workspace, stream=None) -> None:
    import torch

    t, r = logits_struct(train), logits_struct(rollout)
    if train.shape != rollout.shape or train.device != rollout.device:
        raise ValueError("train and rollout must have one shape and device")
    _same_rows(train.shape[0], train.device, token_ids=(token_ids, torch.int32), action_mask=(action_mask, torch.uint8),
               out_logp_train=(out_logp_train, torch.float32), out_logp_rollout=(out_logp_rollout, torch.float32),
               out_dlogp=(out_dlogp, torch.float32))
    _buffer("out_metrics", out_metrics, train.device, METRICS_BYTES)
    _buffer("workspace", workspace, train.device)
    ct, cr = _controls(train_controls, train), _controls(rollout_controls, rollout)
    with _on(train):
        rc = lib().lpd_score_controlled(ctypes.byref(t), ctypes.byref(r), ct, cr, train.shape[0], train.shape[1],
                                        _ptr(token_ids), _ptr(action_mask), float(clip_lo), float(clip_hi),
                                        _ptr(out_logp_train), _ptr(out_logp_rollout), _ptr(out_dlogp),
                                        _ptr(out_metrics), _ptr(workspace), _bytes(workspace), _stream(stream))
    _check(rc, "lpd_score_controlled")


def lpd_logprob_backward_controlled(logits, controls, token_ids, action_mask, logp, grad_logp, out_dlogits,
                                    stream=None) -> None:
    import torch

    x, o = logits_struct(logits), logits_struct(out_dlogits)
    if out_dlogits.shape != logits.shape or out_dlogits.device != logits.device:
        raise ValueError("out_dlogits must have the logits' shape and device")
    _same_rows(logits.shape[0], logits.device, token_ids=(token_ids, torch.int32),
               action_mask=(action_mask, torch.uint8), logp=(logp, torch.float32), grad_logp=(grad_logp, torch.float32))
    c = _controls(controls, logits)
    with _on(logits):
        rc = lib().lpd_logprob_backward_controlled(ctypes.byref(x), c, logits.shape[0], logits.shape[1],
                                                   _ptr(token_ids), _ptr(action_mask), _ptr(logp), _ptr(grad_logp),
                                                   o.ptr, o.dtype, o.row_stride, _stream(stream))
    _check(rc, "lpd_logprob_backward_controlled")


@dataclass(frozen=True)
class Filter:
    """A sampler's filters as device tensors of one entry a row (lpd_filter; None
    leaves a step out): scale (1 / temperature), min_p and top_p float32, top_k
    int32.  The tensors must live as long as this object."""
    scale: object = None
    min_p: object = None
    top_k: object = None
    top_p: object = None

    def __post_init__(self):
        import torch

        rows, device = None, None
        for name in ("scale", "min_p", "top_k", "top_p"):
            t = getattr(self, name)
            if t is None:
                continue
            kind = torch.int32 if name == "top_k" else torch.float32
            if t.dtype != kind or t.dim() != 1 or not t.is_contiguous():
                raise ValueError(f"{name} must be a dense {kind} vector, got {t.dtype} {list(t.shape)}")
            if rows is not None and t.shape[0] != rows:
                raise ValueError(f"{name} has {t.shape[0]} rows, the other filters {rows}")
            if device is not None and t.device != device:
                raise ValueError(f"{name} is on {t.device}, the other filters on {device}")
            rows, device = t.shape[0], t.device
        object.__setattr__(self, "_struct", LpdFilter(_ptr(self.scale), _ptr(self.min_p), _ptr(self.top_k),
                                                      _ptr(self.top_p)))
        object.__setattr__(self, "_rows", rows)
        object.__setattr__(self, "_device", device)


def _filter(f, logits):
    """Pointer to the lpd_filter (None: no filter) after the checks that only the tensors allow."""
    if f is None:
        return None
    if f._rows is not None and f._rows != logits.shape[0]:
        raise ValueError(f"filters of {f._rows} rows for {logits.shape[0]} logits rows")
    if f._device is not None and f._device != logits.device:
        raise ValueError(f"filters on {f._device}, logits on {logits.device}")
    return ctypes.byref(f._struct)


def lpd_sample(logits, filter, uniform, out_ids, out_logp=None, out_kept=None, stream=None) -> None:
    """A token of each row's kept set, drawn with uniform [rows] float32, into out_ids
    (int32), its logprob into out_logp (float32) and the sets' sizes into out_kept (int32)."""
    import torch

    x = logits_struct(logits)
    x.row_stride = _row_stride(logits)
    _same_rows(logits.shape[0], logits.device, uniform=(uniform, torch.float32), out_ids=(out_ids, torch.int32),
               out_logp=(out_logp, torch.float32), out_kept=(out_kept, torch.int32))
    f = _filter(filter, logits)
    with _on(logits):
        rc = lib().lpd_sample(ctypes.byref(x), f, logits.shape[0], logits.shape[1], _ptr(uniform), _ptr(out_ids),
                              _ptr(out_logp), _ptr(out_kept), _stream(stream))
    _check(rc, "lpd_sample")


def lpd_filter_mask(logits, filter, token_ids, action_mask, out_mask, out_lse=None, out_kept=None,
                    stream=None) -> None:
    """The rows' kept sets as bits, into out_mask int32 [rows, words] (Controls.mask's form)."""
    import torch

    x = logits_struct(logits)
    x.row_stride = _row_stride(logits)
    words = -(-logits.shape[1] // 32)
    if out_mask.dtype != torch.int32 or out_mask.dim() != 2 or out_mask.shape[0] != logits.shape[0] \
            or out_mask.shape[1] < words or (out_mask.shape[1] > 1 and out_mask.stride(1) != 1):
        raise ValueError(f"out_mask must be int32 [{logits.shape[0]}, {words} or more] with contiguous words")
    if out_mask.device != logits.device:
        raise ValueError(f"out_mask on {out_mask.device}, logits on {logits.device}")
    _same_rows(logits.shape[0], logits.device, token_ids=(token_ids, torch.int32),
               action_mask=(action_mask, torch.uint8), out_lse=(out_lse, torch.float32),
               out_kept=(out_kept, torch.int32))
    f = _filter(filter, logits)
    with _on(logits):
        rc = lib().lpd_filter_mask(ctypes.byref(x), f, logits.shape[0], logits.shape[1], _ptr(token_ids),
                                   _ptr(action_mask), _ptr(out_mask), _row_stride(out_mask), _ptr(out_lse),
                                   _ptr(out_kept), _stream(stream))
    _check(rc, "lpd_filter_mask")


@dataclass(frozen=True)
class BlockScaled:
    """An 8-bit operand (lpd_block_scaled): values float8_e4m3fn or float8_e5m2
    [rows, k] with contiguous rows, scales float32 [rows, ceil(k / 128)], or
    [ceil(rows / 128), ceil(k / 128)] where `block` is true.  The tensors must
    live as long as this object."""
    values: object
    scales: object
    block: bool = False

    def __post_init__(self):
        import torch

        v, s = self.values, self.scales
        codes = {torch.float8_e4m3fn: LPD_E4M3, torch.float8_e5m2: LPD_E5M2}
        if v.dtype not in codes:
            raise ValueError(f"values must be float8_e4m3fn or float8_e5m2, got {v.dtype}")
        if v.dim() != 2 or (v.numel() and v.shape[1] > 1 and v.stride(1) != 1):
            raise ValueError("values must be 2-D with contiguous columns")
        want = (-(-v.shape[0] // 128) if self.block else v.shape[0], -(-v.shape[1] // 128))
        if s.dtype != torch.float32 or tuple(s.shape) != want or (s.numel() and s.shape[1] > 1 and s.stride(1) != 1):
            raise ValueError(f"scales must be float32 {list(want)} with contiguous columns, got {s.dtype} {list(s.shape)}")
        if s.device != v.device:
            raise ValueError(f"values on {v.device}, scales on {s.device}")
        # the stride of a single row has no meaning in torch: any legal one serves
        stride = v.stride(0) if v.shape[0] > 1 else -(-v.shape[1] // 16) * 16
        object.__setattr__(self, "_struct", LpdBlockScaled(
            v.data_ptr(), codes[v.dtype], int(bool(self.block)), stride, s.data_ptr(),
            s.stride(0) if s.shape[0] > 1 else want[1]))


def block_empty(rows: int, k: int, dtype, block: bool = False, device="cuda") -> BlockScaled:
    """An operand of these sizes to quantise into, its rows on 16-byte boundaries
    as the product needs them."""
    import torch

    room = torch.empty((rows, -(-k // 16) * 16), dtype=torch.uint8, device=device)
    scales = torch.empty((-(-rows // 128) if block else rows, -(-k // 128)), dtype=torch.float32, device=device)
    return BlockScaled(room.view(dtype)[:, :k], scales, block)


def lpd_block_quantize(x, out, transpose=False, pow2=False, stream=None) -> None:
    """x (bf16 or f32, 2-D) into the operand `out`, or its transpose."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with contiguous columns")
    if tuple(out.values.shape) != (tuple(x.shape)[::-1] if transpose else tuple(x.shape)):
        raise ValueError("out has another shape")
    if out.values.device != x.device:
        raise ValueError(f"x on {x.device}, out on {out.values.device}")
    with _on(x):
        rc = lib().lpd_block_quantize(_ptr(x), _dtype_code(x), _row_stride(x), x.shape[0], x.shape[1],
                                      int(bool(transpose)), int(bool(pow2)), ctypes.byref(out._struct),
                                      _stream(stream))
    _check(rc, "lpd_block_quantize")


def lpd_block_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().lpd_block_workspace_size(m, n, k))


def lpd_block_matmul(a, b, out, workspace, stream=None) -> None:
    """out [m, n] (bf16 or f32) = A [m, k] times B [n, k] transposed."""
    (m, k), n = a.values.shape, b.values.shape[0]
    if b.values.shape[1] != k or tuple(out.shape) != (m, n):
        raise ValueError(f"A {[m, k]}, B {list(b.values.shape)} and out {list(out.shape)} do not fit")
    if out.dim() != 2 or (n > 1 and out.stride(1) != 1):
        raise ValueError("out must have contiguous columns")
    if not a.values.device == b.values.device == out.device:
        raise ValueError("the operands and out must be on one device")
    _buffer("workspace", workspace, out.device)
    with _on(out):
        rc = lib().lpd_block_matmul(ctypes.byref(a._struct), ctypes.byref(b._struct), m, n, k, _ptr(out),
                                    _dtype_code(out), _row_stride(out), _ptr(workspace),
                                    _bytes(workspace), _stream(stream))
    _check(rc, "lpd_block_matmul")


def lpd_micro_scale_bytes(block: int, rows: int, k: int) -> int:
    return int(lib().lpd_micro_scale_bytes(block, rows, k))


@dataclass(frozen=True)
class MicroScaled:
    """A 4-bit operand (lpd_micro_scaled) of k columns: codes uint8 [rows, ceil(k / 2)
    or more] with contiguous rows, scales uint8, dense, in the tiled order of the
    header, block 16 or 32, tensor_scale a float32 tensor of one value or None (1).
    The tensors must live as long as this object."""
    codes: object
    scales: object
    k: int
    block: int = 16
    tensor_scale: object = None

    def __post_init__(self):
        import torch

        c, s, t = self.codes, self.scales, self.tensor_scale
        if self.block not in (16, 32):
            raise ValueError(f"block must be 16 or 32, got {self.block}")
        if self.k < 0 or c.dtype != torch.uint8 or c.dim() != 2 or c.shape[1] < -(-self.k // 2) \
                or (c.numel() and c.shape[1] > 1 and c.stride(1) != 1):
            raise ValueError(f"codes must be uint8 [rows, {-(-self.k // 2)} or more] with contiguous columns")
        want = -(-c.shape[0] // 128) * -(-self.k // (4 * self.block)) * 512
        if s.dtype != torch.uint8 or not s.is_contiguous() or s.numel() != want:
            raise ValueError(f"scales must be {want} dense uint8 values, got {s.dtype} {list(s.shape)}")
        if t is not None and (t.dtype != torch.float32 or t.numel() != 1):
            raise ValueError("tensor_scale must be one float32 value")
        for name, o in (("scales", s), ("tensor_scale", t)):
            if o is not None and o.device != c.device:
                raise ValueError(f"codes on {c.device}, {name} on {o.device}")
        # the stride of a single row has no meaning in torch: any legal one serves
        stride = c.stride(0) if c.shape[0] > 1 else -(-c.shape[1] // 16) * 16
        struct = LpdMicroScaled(c.data_ptr(), self.block, 0, stride, s.data_ptr(), _ptr(t))
        for name, value in (("_struct", struct), ("_ref", ctypes.byref(struct)), ("_rows", c.shape[0]), ("_device", c.device)):
            object.__setattr__(self, name, value)


def micro_empty(rows: int, k: int, block: int = 16, tensor_scale=None, device="cuda") -> MicroScaled:
    """An operand of these sizes to quantise into, its rows on 16-byte boundaries
    as the product needs them."""
    import torch

    room = torch.empty((rows, -(-k // 32) * 16), dtype=torch.uint8, device=device)
    scales = torch.empty(lpd_micro_scale_bytes(block, rows, k), dtype=torch.uint8, device=device)
    return MicroScaled(room[:, :-(-k // 2)], scales, k, block, tensor_scale)


def lpd_micro_quantize(x, out, transpose=False, out_values=None, stream=None) -> None:
    """x (bf16 or f32, 2-D) into the operand `out`, or its transpose; the values that
    it stands for into out_values (bf16 or f32), if given."""
    if x.dim() != 2 or (x.shape[1] > 1 and x.stride(1) != 1):
        raise ValueError("x must be 2-D with contiguous columns")
    rows, cols = x.shape
    shape = (cols, rows) if transpose else (rows, cols)
    device = x.device
    if (out._rows, out.k) != shape:
        raise ValueError("out has another shape")
    if out._device != device:
        raise ValueError(f"x on {device}, out on {out._device}")
    v, v_dtype, v_stride = out_values, 0, 0
    if v is not None:
        if v.shape != shape or v.device != device or (shape[1] > 1 and v.stride(1) != 1):
            raise ValueError("out_values must have out's shape and device and contiguous columns")
        v_dtype, v_stride = _dtype_code(v), _row_stride(v)
    with _on(x):
        rc = lib().lpd_micro_quantize(_ptr(x), _dtype_code(x), _row_stride(x), rows, cols, int(bool(transpose)),
                                      out._ref, _ptr(v), v_dtype, v_stride, _stream(stream))
    _check(rc, "lpd_micro_quantize")


def lpd_micro_workspace_size(m: int, n: int, k: int) -> int:
    return int(lib().lpd_micro_workspace_size(m, n, k))


def lpd_micro_matmul(a, b, out, workspace, stream=None) -> None:
    """out [m, n] (bf16 or f32) = A [m, k] times B [n, k] transposed."""
    m, n = a.codes.shape[0], b.codes.shape[0]
    if b.k != a.k or tuple(out.shape) != (m, n):
        raise ValueError(f"A {[m, a.k]}, B {[n, b.k]} and out {list(out.shape)} do not fit")
    if out.dim() != 2 or (n > 1 and out.stride(1) != 1):
        raise ValueError("out must have contiguous columns")
    if not a.codes.device == b.codes.device == out.device:
        raise ValueError("the operands and out must be on one device")
    _buffer("workspace", workspace, out.device)
    with _on(out):
        rc = lib().lpd_micro_matmul(a._ref, b._ref, m, n, a.k, _ptr(out),
                                    _dtype_code(out), _row_stride(out), _ptr(workspace), _bytes(workspace),
                                    _stream(stream))
    _check(rc, "lpd_micro_matmul")


# ---- convenience: allocate with torch, call, read back ------------------------

def read_merge_drift(buf) -> dict:
    """Copy a device lpd_merge_drift record (uint8 tensor) to the host as a dict."""
    host = buf.detach().to("cpu", copy=True).numpy().tobytes()
    return LpdMergeDrift.from_buffer_copy(host).as_dict()


@_with_its_stream
def attn_merge(out_parts, lse_parts, order=None, lse_base2=False, stream=None):
    """Merged (out [n, d] f32, lse [n] f32) of K partials, allocated with torch."""
    import torch

    K, n, d = _parts_shape(out_parts, lse_parts)
    out = torch.empty((n, d), dtype=torch.float32, device=out_parts.device)
    lse = torch.empty((n,), dtype=torch.float32, device=out_parts.device)
    lpd_attn_merge(out_parts, lse_parts, order, out, lse, lse_base2, stream)
    return out, lse


@_with_its_stream
def attn_merge_order_drift(out_parts, lse_parts, order_a=None, order_b=None, lse_base2=False, stream=None):
    """(out, lse, row_dout, row_dlse, summary dict) of the order_a vs order_b merge."""
    import torch

    K, n, d = _parts_shape(out_parts, lse_parts)
    dev = out_parts.device
    out = torch.empty((n, d), dtype=torch.float32, device=dev)
    lse = torch.empty((n,), dtype=torch.float32, device=dev)
    rdo = torch.empty((n,), dtype=torch.float32, device=dev)
    rdl = torch.empty((n,), dtype=torch.float32, device=dev)
    drift = torch.empty(MERGE_DRIFT_BYTES, dtype=torch.uint8, device=dev)
    lpd_attn_merge_order_drift(out_parts, lse_parts, order_a, order_b, out, lse, rdo, rdl, drift, lse_base2, stream)
    return out, lse, rdo, rdl, read_merge_drift(drift)


def read_logp_drift(buf) -> dict:
    """Copy a device lpd_logp_drift record (uint8 tensor) to the host as a dict."""
    host = buf.detach().to("cpu", copy=True).numpy().tobytes()
    return LpdLogpDrift.from_buffer_copy(host).as_dict()


@_with_its_stream
def logp_drift_summary(logp_train_a, logp_rollout_a, logp_train_b, logp_rollout_b, action_mask, stream=None) -> dict:
    """lpd_logp_drift_summary with a torch-allocated record, read back as a dict."""
    import torch

    out = torch.empty(LOGP_DRIFT_BYTES, dtype=torch.uint8, device=action_mask.device)
    lpd_logp_drift_summary(logp_train_a, logp_rollout_a, logp_train_b, logp_rollout_b, action_mask, out, stream)
    return read_logp_drift(out)


def merge_rank_metrics(per_rank: list[dict], row_offsets: list[int] | None = None) -> dict:
    """lpd_merge_rank_metrics (a host call) on metrics records given as dicts
    in rank order; returns the merged record as a dict."""
    n = len(per_rank)
    arr = (LpdMetrics * max(n, 1))()
    for k, rec in enumerate(per_rank):
        for name, _ in LpdMetrics._fields_:
            setattr(arr[k], name, rec.get(name, 0))
    offs = None if row_offsets is None else (ctypes.c_int64 * max(n, 1))(*[int(o) for o in row_offsets])
    out = LpdMetrics()
    rc = lib().lpd_merge_rank_metrics(ctypes.addressof(arr), None if offs is None else ctypes.addressof(offs), n,
                                      ctypes.addressof(out))
    _check(rc, "lpd_merge_rank_metrics")
    return out.as_dict()


def read_metrics(buf) -> dict:
    """Copy a device lpd_metrics record (uint8 tensor) to the host as a dict."""
    host = buf.detach().to("cpu", copy=True).numpy().tobytes()
    return LpdMetrics.from_buffer_copy(host).as_dict()


@_with_its_stream
def score_fused(hidden_train, hidden_rollout, W, token_ids, action_mask, clip=(0.8, 1.2), stream=None,
                train_ops=None, rollout_ops=None):
    """Allocate outputs and workspace with torch, run lpd_score_fused (or
    lpd_score_fused_transformed when a chain is given)."""
    import torch

    dev = hidden_train.device
    n = hidden_train.shape[0]
    outs = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3)]
    met = torch.empty(METRICS_BYTES, dtype=torch.uint8, device=dev)
    ws = torch.empty(lpd_fused_workspace_size(n, hidden_train.shape[1], W.shape[0]), dtype=torch.uint8, device=dev)
    if train_ops is None and rollout_ops is None:
        lpd_score_fused(hidden_train, hidden_rollout, W, token_ids, action_mask, clip[0], clip[1], *outs, met, ws,
                        stream=stream)
    else:
        lpd_score_fused_transformed(hidden_train, hidden_rollout, W, train_ops, rollout_ops, token_ids, action_mask,
                                    clip[0], clip[1], *outs, met, ws, stream=stream)
    return ScoreResult(outs[0], outs[1], outs[2], read_metrics(met))


@dataclass
class ScoreResult:
    logp_train: object
    logp_rollout: object
    dlogp: object
    metrics: dict


@_with_its_stream
def score(train, rollout, token_ids, action_mask, clip=(0.8, 1.2), stream=None, train_ops=None,
          rollout_ops=None) -> ScoreResult:
    """Allocate outputs and workspace with torch on the logits' device, run
    lpd_score (or lpd_score_transformed when a chain is given), and return
    per-token tensors plus the metrics as a dict."""
    import torch

    dev = train.device
    n = train.shape[0]
    outs = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3)]
    met = torch.empty(METRICS_BYTES, dtype=torch.uint8, device=dev)
    ws = torch.empty(lpd_workspace_size(LPD_KIND_SCORE, n), dtype=torch.uint8, device=dev)
    if train_ops is None and rollout_ops is None:
        lpd_score(train, rollout, token_ids, action_mask, clip[0], clip[1], *outs, met, ws, stream=stream)
    else:
        lpd_score_transformed(train, rollout, train_ops, rollout_ops, token_ids, action_mask, clip[0], clip[1],
                              *outs, met, ws, stream=stream)
    return ScoreResult(outs[0], outs[1], outs[2], read_metrics(met))


@_with_its_stream
def score_sharded_topology(train_shards, rollout_shards, v_ranges, token_ids, action_mask, topology,
                           reduce_order=None, clip=(0.8, 1.2), stream=None) -> ScoreResult:
    """lpd_score_sharded_topology with torch-allocated outputs and workspace."""
    import torch

    dev = token_ids.device
    n = token_ids.shape[0]
    vocab = max(v1 for _, v1 in v_ranges)
    outs = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3)]
    met = torch.empty(METRICS_BYTES, dtype=torch.uint8, device=dev)
    nbytes = lpd_topology_workspace_size(topology, n, vocab, len(train_shards), _dtype_code(train_shards[0]),
                                         _dtype_code(rollout_shards[0]))
    ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    lpd_score_sharded_topology(train_shards, rollout_shards, v_ranges, token_ids, action_mask, clip[0], clip[1],
                               topology, reduce_order, *outs, met, ws, stream)
    return ScoreResult(*outs, read_metrics(met))


@_with_its_stream
def controls_apply(logits, controls, out_dtype=None, stream=None):
    """The controlled logits in a new tensor (the logits' type unless given)."""
    import torch

    out = torch.empty(logits.shape, dtype=out_dtype or logits.dtype, device=logits.device)
    lpd_controls_apply(logits, controls, out, stream)
    return out


@_with_its_stream
def score_controlled(train, rollout, token_ids, action_mask, train_controls=None, rollout_controls=None,
                     clip=(0.8, 1.2), stream=None) -> ScoreResult:
    """lpd_score_controlled with torch-allocated outputs and workspace."""
    import torch

    dev = train.device
    n = train.shape[0]
    outs = [torch.empty(n, dtype=torch.float32, device=dev) for _ in range(3)]
    met = torch.empty(METRICS_BYTES, dtype=torch.uint8, device=dev)
    ws = torch.empty(lpd_workspace_size(LPD_KIND_CONTROLLED, n, train.shape[1]), dtype=torch.uint8, device=dev)
    lpd_score_controlled(train, rollout, train_controls, rollout_controls, token_ids, action_mask, clip[0], clip[1],
                         *outs, met, ws, stream)
    return ScoreResult(*outs, read_metrics(met))


@_with_its_stream
def sample(logits, uniform, filter=None, stream=None):
    """(ids int32, logprobs float32, kept int32) of a draw from each row, in new tensors."""
    import torch

    n, dev = logits.shape[0], logits.device
    ids, kept = (torch.empty(n, dtype=torch.int32, device=dev) for _ in range(2))
    logp = torch.empty(n, dtype=torch.float32, device=dev)
    lpd_sample(logits, filter, uniform, ids, logp, kept, stream)
    return ids, logp, kept


@_with_its_stream
def filter_mask(logits, filter, token_ids=None, action_mask=None, stream=None):
    """(mask int32 [rows, words], lse float32, kept int32) of the rows' kept sets, in new tensors."""
    import torch

    n, dev = logits.shape[0], logits.device
    mask = torch.empty((n, -(-logits.shape[1] // 32)), dtype=torch.int32, device=dev)
    lse = torch.empty(n, dtype=torch.float32, device=dev)
    kept = torch.empty(n, dtype=torch.int32, device=dev)
    lpd_filter_mask(logits, filter, token_ids, action_mask, mask, lse, kept, stream)
    return mask, lse, kept


@_with_its_stream
def block_quantize(x, dtype=None, block=False, transpose=False, pow2=False, stream=None) -> BlockScaled:
    """x as a new 8-bit operand (e4m3 unless given)."""
    import torch

    rows, k = tuple(x.shape)[::-1] if transpose else tuple(x.shape)
    out = block_empty(rows, k, dtype or torch.float8_e4m3fn, block, x.device)
    lpd_block_quantize(x, out, transpose, pow2, stream)
    return out


@_with_its_stream
def block_matmul(a, b, out_dtype=None, stream=None):
    """The product of two operands in a new tensor (bf16 unless given)."""
    import torch

    m, n = a.values.shape[0], b.values.shape[0]
    dev = a.values.device
    out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    ws = torch.empty(lpd_block_workspace_size(m, n, a.values.shape[1]), dtype=torch.uint8, device=dev)
    lpd_block_matmul(a, b, out, ws, stream)
    return out


@_with_its_stream
def micro_quantize(x, block=16, tensor_scale=None, transpose=False, stream=None) -> MicroScaled:
    """x as a new 4-bit operand."""
    rows, k = tuple(x.shape)[::-1] if transpose else tuple(x.shape)
    out = micro_empty(rows, k, block, tensor_scale, x.device)
    lpd_micro_quantize(x, out, transpose, None, stream)
    return out


@_with_its_stream
def micro_matmul(a, b, out_dtype=None, stream=None):
    """The product of two 4-bit operands in a new tensor (bf16 unless given)."""
    import torch

    m, n = a.codes.shape[0], b.codes.shape[0]
    dev = a.codes.device
    out = torch.empty((m, n), dtype=out_dtype or torch.bfloat16, device=dev)
    ws = torch.empty(lpd_micro_workspace_size(m, n, a.k), dtype=torch.uint8, device=dev)
    lpd_micro_matmul(a, b, out, ws, stream)
    return out
