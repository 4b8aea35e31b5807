"""Thin Python binding of libkda.so (argument marshalling only).

Every step of the forward pass runs in the library's CUDA kernels; torch only
provides device memory and the current CUDA stream.  There is no fallback: if
the library is missing or the tensors are not on a CUDA device the calls
raise.
"""
import ctypes
import os

import torch

from . import build as _build

KDA_OK = 0
KDA_BF16, KDA_F32 = 0, 1
STATUS_NAMES = {0: "KDA_OK", 1: "KDA_ERR_INVALID_ARG", 2: "KDA_ERR_UNSUPPORTED",
                3: "KDA_ERR_MISALIGNED", 4: "KDA_ERR_CUDA", 5: "KDA_ERR_TIMEOUT",
                6: "KDA_ERR_RANGE"}

# Entry points declared in include/kda.h and include/kda_layer.h (kept in sync
# by tests).
EXPORTS = ("kda_chunk_fwd", "kda_chunk_fwd_staged", "kda_recurrent_step",
           "kda_chunk_fwd_plan", "kda_selftest_umma", "kda_device_status",
           "kda_status_string", "kda_last_cuda_error", "kda_version",
           "kda_chunk_fwd_staged_noalloc", "kda_chunk_fwd_gated",
           "kda_recurrent_step_gated", "kda_chunk_fwd_ex",
           "kda_recurrent_step_ex", "kda_selftest_timeout", "kda_chunk_bwd",
           "kda_chunk_bwd_plan", "kda_chunk_fwd_split", "kda_workspace_pool",
           "kda_chunk_fwd_twopass", "kda_chunk_fwd_paired",
           "kda_chunk_fwd_split_plan", "kda_profile_pass_event",
           "kda_chunk_bwd_layout", "kda_short_conv_fwd", "kda_short_conv_bwd",
           "kda_short_conv_step", "kda_ssm_scan_fwd", "kda_ssm_scan_bwd",
           "kda_ssm_scan_bwd_plan", "kda_ssm_step", "kda_block_norm_fwd",
           "kda_block_norm_bwd")
GATES = {"channel": 0, "head": 1, "none": 2}
ACTS = {"none": 0, "silu": 1, "sigmoid": 2}


class KdaShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("H", ctypes.c_int),
                ("dk", ctypes.c_int), ("dv", ctypes.c_int),
                ("chunk", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("io_dtype", ctypes.c_int)]


class KdaPrologue(ctypes.Structure):
    _fields_ = [("normalize_qk", ctypes.c_int), ("q_scale", ctypes.c_float),
                ("gate_logits", ctypes.c_int), ("gate_scale", ctypes.c_float)]


class KdaConvShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("W", ctypes.c_int), ("n_seqs", ctypes.c_int),
                ("io_dtype", ctypes.c_int), ("activation", ctypes.c_int),
                ("x_stride", ctypes.c_int64)]


class KdaSsmShape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("D", ctypes.c_int),
                ("S", ctypes.c_int), ("G", ctypes.c_int),
                ("n_seqs", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("softplus", ctypes.c_int), ("u_stride", ctypes.c_int64),
                ("delta_stride", ctypes.c_int64), ("z_stride", ctypes.c_int64),
                ("b_stride", ctypes.c_int64),
                ("b_group_stride", ctypes.c_int64),
                ("c_stride", ctypes.c_int64),
                ("c_group_stride", ctypes.c_int64)]


class KdaNormShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("heads", ctypes.c_int),
                ("width", ctypes.c_int), ("io_dtype", ctypes.c_int),
                ("residual_dtype", ctypes.c_int), ("gate_act", ctypes.c_int),
                ("gate_first", ctypes.c_int), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("gate_stride", ctypes.c_int64)]


def _prologue(pro):
    """dict(normalize_qk=bool, q_scale=float, gate_logits=bool,
    gate_scale=float) -> KdaPrologue (missing keys: no-op defaults)."""
    pro = dict(pro or {})
    return KdaPrologue(int(bool(pro.get("normalize_qk", False))),
                       float(pro.get("q_scale", 1.0)),
                       int(bool(pro.get("gate_logits", False))),
                       float(pro.get("gate_scale", 1.0)))


class KdaError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)} "
                         f"({library().kda_status_string(status).decode()})"
                         + (f" cuda error {library().kda_last_cuda_error()}"
                            if status == 4 else ""))


_lib = None


def library_path():
    return _build.LIB


def library():
    """The loaded libkda.so.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"libkda.so not found at {path}; build it with "
                "`python -m gated_delta_rule_156_b200.build`")
        lib = ctypes.CDLL(path)
        vp, fp = ctypes.c_void_p, ctypes.c_void_p
        chunk_args = [ctypes.POINTER(KdaShape), vp, vp, vp, fp, fp, fp, vp, vp,
                      fp, vp]
        for name in ("kda_chunk_fwd", "kda_chunk_fwd_staged",
                     "kda_chunk_fwd_staged_noalloc"):
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            fn.argtypes = chunk_args
        lib.kda_chunk_fwd_gated.restype = ctypes.c_int
        lib.kda_chunk_fwd_gated.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, vp, vp, vp, fp, fp, fp, vp,
            vp, fp, ctypes.c_int, vp]
        lib.kda_recurrent_step_gated.restype = ctypes.c_int
        lib.kda_recurrent_step_gated.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, vp, vp, vp, fp, fp, fp, vp,
            vp]
        lib.kda_chunk_fwd_ex.restype = ctypes.c_int
        lib.kda_chunk_fwd_ex.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.POINTER(KdaPrologue),
            vp, vp, vp, fp, fp, fp, vp, vp, fp, ctypes.c_int, vp]
        for name in ("kda_chunk_fwd_twopass", "kda_chunk_fwd_paired"):
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            fn.argtypes = [
                ctypes.POINTER(KdaShape), ctypes.c_int,
                ctypes.POINTER(KdaPrologue), vp, vp, vp, fp, fp, fp, vp, vp,
                fp, vp]
        lib.kda_recurrent_step_ex.restype = ctypes.c_int
        lib.kda_recurrent_step_ex.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.POINTER(KdaPrologue),
            vp, vp, vp, fp, fp, fp, vp, vp]
        lib.kda_recurrent_step.restype = ctypes.c_int
        lib.kda_recurrent_step.argtypes = [ctypes.POINTER(KdaShape), vp, vp, vp,
                                           fp, fp, fp, vp, vp]
        lib.kda_chunk_fwd_plan.restype = ctypes.c_int
        lib.kda_chunk_fwd_plan.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.c_int,
            ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
            ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_chunk_fwd_split.restype = ctypes.c_int
        lib.kda_chunk_fwd_split.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, vp, vp, vp, fp, fp, fp, vp,
            fp, ctypes.c_int, vp]
        lib.kda_chunk_fwd_split_plan.restype = ctypes.c_int
        lib.kda_chunk_fwd_split_plan.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.c_int, ctypes.c_int,
            ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
            ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_chunk_bwd.restype = ctypes.c_int
        lib.kda_chunk_bwd.argtypes = [ctypes.POINTER(KdaShape)] + [vp] * 16
        lib.kda_chunk_bwd_plan.restype = ctypes.c_int
        lib.kda_chunk_bwd_plan.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.POINTER(ctypes.c_int),
            ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_chunk_bwd_layout.restype = ctypes.c_int
        lib.kda_chunk_bwd_layout.argtypes = [
            ctypes.POINTER(KdaShape), ctypes.c_int, ctypes.c_int,
            ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t),
            ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
            ctypes.POINTER(ctypes.c_int)]
        lib.kda_selftest_umma.restype = ctypes.c_int
        lib.kda_selftest_umma.argtypes = [ctypes.c_int] * 5 + [vp, vp, vp, vp]
        lib.kda_selftest_timeout.restype = ctypes.c_int
        lib.kda_selftest_timeout.argtypes = [ctypes.c_int, vp]
        lib.kda_device_status.restype = ctypes.c_int
        lib.kda_device_status.argtypes = [vp]
        lib.kda_status_string.restype = ctypes.c_char_p
        lib.kda_status_string.argtypes = [ctypes.c_int]
        for name, struct, n in (("kda_short_conv_fwd", KdaConvShape, 7),
                                ("kda_short_conv_bwd", KdaConvShape, 11),
                                ("kda_short_conv_step", KdaConvShape, 5),
                                ("kda_ssm_scan_fwd", KdaSsmShape, 12),
                                ("kda_ssm_scan_bwd", KdaSsmShape, 21),
                                ("kda_ssm_step", KdaSsmShape, 10),
                                ("kda_block_norm_fwd", KdaNormShape, 8),
                                ("kda_block_norm_bwd", KdaNormShape, 14)):
            fn = getattr(lib, name)
            fn.restype = ctypes.c_int
            # the shape, n tensors, the stream
            fn.argtypes = [ctypes.POINTER(struct)] + [vp] * (n + 1)
        lib.kda_ssm_scan_bwd_plan.restype = ctypes.c_int
        lib.kda_ssm_scan_bwd_plan.argtypes = [
            ctypes.POINTER(KdaSsmShape), ctypes.c_int,
            ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_workspace_pool.restype = ctypes.c_int
        lib.kda_workspace_pool.argtypes = [ctypes.POINTER(ctypes.c_size_t),
                                           ctypes.POINTER(ctypes.c_size_t)]
        lib.kda_profile_pass_event.restype = ctypes.c_int
        lib.kda_profile_pass_event.argtypes = [ctypes.c_void_p]
        lib.kda_last_cuda_error.restype = ctypes.c_int
        lib.kda_last_cuda_error.argtypes = []
        lib.kda_version.restype = ctypes.c_int
        lib.kda_version.argtypes = []
        _lib = lib
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check_dev(name, t, dtype=None):
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")


def _io(q):
    if q.dtype == torch.bfloat16:
        return KDA_BF16
    if q.dtype == torch.float32:
        return KDA_F32
    raise ValueError(f"unsupported io dtype {q.dtype}")


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def chunk_fwd(q, k, v, log_alpha, beta, initial_state=None, cu_seqlens=None,
              chunk=64, out=None, final_state=None, staged=False, stream=None,
              gate="channel", prologue=None, twopass=False, paired=False):
    """Chunkwise KDA forward (kda_chunk_fwd / kda_chunk_fwd_staged, or
    kda_chunk_fwd_gated when ``gate`` is not "channel").

    q, k [B, T, H, d_k]; v [B, T, H, d_v] (bf16 or fp32, same dtype);
    log_alpha fp32 [B, T, H, d_k] (gate="channel"), [B, T, H] (gate="head")
    or None (gate="none"); beta [B, T, H] fp32; initial_state
    [N, H, d_k, d_v] fp32 or None; cu_seqlens int32 [N + 1] or None (then
    B == 1 and T is the packed total).  ``prologue`` (dict, see
    kda_prologue) normalises q and k and/or maps gate logits in-kernel
    (kda_chunk_fwd_ex).  ``twopass`` forces the factorisation pass + chain
    kernel (kda_chunk_fwd_twopass, the default for bf16 d in {64, 128},
    chunk 64); ``paired`` the one-kernel cluster-pair path
    (kda_chunk_fwd_paired).  Returns (out, final_state).
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32,
                                  device=q.device)
    for name, t, dt in (("q", q, None), ("k", k, q.dtype), ("v", v, q.dtype),
                        ("log_alpha", log_alpha, torch.float32),
                        ("beta", beta, torch.float32),
                        ("initial_state", initial_state, torch.float32),
                        ("cu_seqlens", cu_seqlens, torch.int32),
                        ("out", out, q.dtype),
                        ("final_state", final_state, torch.float32)):
        _check_dev(name, t, dt)
    shape = KdaShape(B, T, H, dk, dv, chunk, n if cu_seqlens is not None else 0,
                     _io(q))
    if twopass or paired:  # an explicit tensor-core evaluation
        name = "kda_chunk_fwd_twopass" if twopass else "kda_chunk_fwd_paired"
        pro = None if prologue is None else _prologue(prologue)
        st = getattr(library(), name)(
            ctypes.byref(shape), GATES[gate],
            None if pro is None else ctypes.byref(pro), _ptr(q), _ptr(k),
            _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state),
            _ptr(cu_seqlens), _ptr(out), _ptr(final_state), _stream(stream))
        if st != KDA_OK:
            raise KdaError(st, name)
        return out, final_state
    if prologue is not None:
        pro = _prologue(prologue)
        st = library().kda_chunk_fwd_ex(
            ctypes.byref(shape), GATES[gate], ctypes.byref(pro), _ptr(q),
            _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(initial_state),
            _ptr(cu_seqlens), _ptr(out), _ptr(final_state), int(staged),
            _stream(stream))
        if st != KDA_OK:
            raise KdaError(st, "kda_chunk_fwd_ex")
        return out, final_state
    if gate != "channel":
        st = library().kda_chunk_fwd_gated(
            ctypes.byref(shape), GATES[gate], _ptr(q), _ptr(k), _ptr(v),
            _ptr(log_alpha), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
            _ptr(out), _ptr(final_state), int(staged), _stream(stream))
        if st != KDA_OK:
            raise KdaError(st, "kda_chunk_fwd_gated")
        return out, final_state
    fn = library().kda_chunk_fwd_staged if staged else library().kda_chunk_fwd
    st = fn(ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
            _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out),
            _ptr(final_state), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_staged" if staged else "kda_chunk_fwd")
    return out, final_state


def chunk_fwd_split(q, k, v, log_alpha, beta, initial_state=None,
                    n_segments=2, chunk=64, out=None, final_state=None,
                    gate="channel", stream=None):
    """Prefill of one long sequence as ``n_segments`` segments evaluated side
    by side and joined by a scan of their state transitions
    (kda_chunk_fwd_split; ``n_segments=0`` lets the library pick the count
    from the SM count).  Shapes as chunk_fwd with B == 1 and no cu_seqlens.
    Returns (out, final_state)."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((B, H, dk, dv), dtype=torch.float32,
                                  device=q.device)
    for name, t, dt in (("q", q, None), ("k", k, q.dtype), ("v", v, q.dtype),
                        ("log_alpha", log_alpha, torch.float32),
                        ("beta", beta, torch.float32),
                        ("initial_state", initial_state, torch.float32),
                        ("out", out, q.dtype),
                        ("final_state", final_state, torch.float32)):
        _check_dev(name, t, dt)
    shape = KdaShape(B, T, H, dk, dv, chunk, 0, _io(q))
    st = library().kda_chunk_fwd_split(
        ctypes.byref(shape), GATES[gate], _ptr(q), _ptr(k), _ptr(v),
        _ptr(log_alpha), _ptr(beta), _ptr(initial_state), _ptr(out),
        _ptr(final_state), int(n_segments), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_split")
    return out, final_state


def chunk_fwd_split_plan(T, H, dk, dv, chunk, dtype, n_segments,
                         gate="channel", num_sms=148):
    """(segments, kernels, workspace_bytes) of a chunk_fwd_split call
    (``num_sms`` matters only for ``n_segments=0``)."""
    io = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    shape = KdaShape(1, T, H, dk, dv, chunk, 0, io)
    seg, kern, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    st = library().kda_chunk_fwd_split_plan(
        ctypes.byref(shape), GATES[gate], int(n_segments), int(num_sms),
        ctypes.byref(seg), ctypes.byref(kern), ctypes.byref(ws))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_split_plan")
    return seg.value, kern.value, ws.value


def chunk_bwd(q, k, v, log_alpha, beta, initial_state, cu_seqlens, d_out,
              d_final_state=None, chunk=64, want_initial_state=True,
              stream=None):
    """Backward pass of chunk_fwd (kda_chunk_bwd; per-channel gate, no input
    prologue): the gradients of sum(d_out * out) + sum(d_final_state *
    final_state).  Shapes as chunk_fwd; d_out like out; d_final_state fp32
    [N, H, d_k, d_v] or None.  Returns (dq, dk, dv, dlog_alpha, dbeta,
    d_initial_state) with d_initial_state None unless want_initial_state.
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    for name, t, dt in (("q", q, None), ("k", k, q.dtype), ("v", v, q.dtype),
                        ("log_alpha", log_alpha, torch.float32),
                        ("beta", beta, torch.float32),
                        ("initial_state", initial_state, torch.float32),
                        ("cu_seqlens", cu_seqlens, torch.int32),
                        ("d_out", d_out, q.dtype),
                        ("d_final_state", d_final_state, torch.float32)):
        _check_dev(name, t, dt)
    dq = torch.empty_like(q)
    dkk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    dla = torch.empty((B, T, H, dk), dtype=torch.float32, device=q.device)
    dbeta = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    ds0 = (torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
           if want_initial_state else None)
    shape = KdaShape(B, T, H, dk, dv, chunk, n if cu_seqlens is not None else 0,
                     _io(q))
    st = library().kda_chunk_bwd(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
        _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), _ptr(d_out),
        _ptr(d_final_state), _ptr(dq), _ptr(dkk), _ptr(dvv), _ptr(dla),
        _ptr(dbeta), _ptr(ds0), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd")
    return dq, dkk, dvv, dla, dbeta, ds0


def chunk_bwd_plan(B, T, H, dk, dv, chunk, dtype, packed=False, n_seqs=0):
    """(kernels, workspace_bytes) of a chunk_bwd call of this shape."""
    io = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    shape = KdaShape(B, T, H, dk, dv, chunk, n_seqs if packed else 0, io)
    kern, ws = ctypes.c_int(), ctypes.c_size_t()
    st = library().kda_chunk_bwd_plan(ctypes.byref(shape), int(packed),
                                      ctypes.byref(kern), ctypes.byref(ws))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd_plan")
    return kern.value, ws.value


def chunk_bwd_layout(B, T, H, dk, dv, chunk, dtype, packed=False, n_seqs=0):
    """The workspace arrays of a chunk_bwd call of this shape, as (offset,
    bytes, first launch, last launch) tuples (kda_chunk_bwd_layout); empty on
    the fp32 path, whose arrays are all apart."""
    io = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    shape = KdaShape(B, T, H, dk, dv, chunk, n_seqs if packed else 0, io)
    cap = 64
    offs, sizes = (ctypes.c_size_t * cap)(), (ctypes.c_size_t * cap)()
    first, last, count = (ctypes.c_int * cap)(), (ctypes.c_int * cap)(), \
        ctypes.c_int()
    st = library().kda_chunk_bwd_layout(ctypes.byref(shape), int(packed), cap,
                                        offs, sizes, first, last,
                                        ctypes.byref(count))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_bwd_layout")
    return [(offs[i], sizes[i], first[i], last[i])
            for i in range(min(count.value, cap))]


def recurrent_step(q, k, v, log_alpha, beta, state, out=None, stream=None,
                   gate="channel", prologue=None):
    """Token-by-token KDA (kda_recurrent_step, or kda_recurrent_step_gated
    when ``gate`` is "head" or "none"); ``state`` [B, H, d_k, d_v] fp32 is
    updated in place.  q, k [B, T, H, d_k] (T >= 1 tokens per sequence).
    Returns out [B, T, H, d_v]."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    for name, t, dt in (("q", q, None), ("k", k, q.dtype), ("v", v, q.dtype),
                        ("log_alpha", log_alpha, torch.float32),
                        ("beta", beta, torch.float32),
                        ("state", state, torch.float32), ("out", out, q.dtype)):
        _check_dev(name, t, dt)
    shape = KdaShape(B, T, H, dk, dv, 0, 0, _io(q))
    if prologue is not None:
        pro = _prologue(prologue)
        st = library().kda_recurrent_step_ex(
            ctypes.byref(shape), GATES[gate], ctypes.byref(pro), _ptr(q),
            _ptr(k), _ptr(v), _ptr(log_alpha), _ptr(beta), _ptr(state),
            _ptr(out), _stream(stream))
        if st != KDA_OK:
            raise KdaError(st, "kda_recurrent_step_ex")
        return out
    st = library().kda_recurrent_step_gated(
        ctypes.byref(shape), GATES[gate], _ptr(q), _ptr(k), _ptr(v),
        _ptr(log_alpha), _ptr(beta), _ptr(state), _ptr(out), _stream(stream)) \
        if gate != "channel" else library().kda_recurrent_step(
            ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
            _ptr(beta), _ptr(state), _ptr(out), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_recurrent_step")
    return out


def chunk_fwd_plan(B, T, H, dk, dv, chunk, dtype, packed=False, n_seqs=0,
                   staged=False):
    """(path, kernels, workspace_bytes) of a chunk_fwd call of this shape:
    path is "twopass" or "staged"; no device work is done."""
    io = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    shape = KdaShape(B, T, H, dk, dv, chunk, n_seqs if packed else 0, io)
    path, kern, ws = ctypes.c_int(), ctypes.c_int(), ctypes.c_size_t()
    st = library().kda_chunk_fwd_plan(ctypes.byref(shape), int(packed),
                                      int(staged), ctypes.byref(path),
                                      ctypes.byref(kern), ctypes.byref(ws))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_plan")
    return ({2: "twopass", 1: "fused"}.get(path.value, "staged"), kern.value,
            ws.value)


def chunk_fwd_kernel_count(B, T, H, dk, dv, chunk, dtype, packed=False):
    return chunk_fwd_plan(B, T, H, dk, dv, chunk, dtype, packed, 1)[1]


def chunk_fwd_path(B, T, H, dk, dv, chunk, dtype, packed=False):
    return chunk_fwd_plan(B, T, H, dk, dv, chunk, dtype, packed, 1)[0]


def selftest_umma(A, B, a_mn, b_mn, panel_rows=None, stream=None):
    """Diagnostic tensor-core product through the fused kernel's operand
    layouts (kda_selftest_umma).  A is [128, K] (a_mn=False) or [K, 128]
    (a_mn=True); B is [N, K] (b_mn=False) or [K, N] (b_mn=True); bf16.
    Returns D = A_logical @ B_logical as [128, N] fp32."""
    K = A.shape[1] if not a_mn else A.shape[0]
    N = B.shape[0] if not b_mn else B.shape[1]
    D = torch.empty((128, N), dtype=torch.float32, device=A.device)
    for name, t in (("A", A), ("B", B)):
        _check_dev(name, t, torch.bfloat16)
    st = library().kda_selftest_umma(int(a_mn), int(b_mn), N, K,
                                     panel_rows or K, _ptr(A), _ptr(B),
                                     _ptr(D), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_umma")
    return D


def profile_pass_event(event):
    """Set (a torch.cuda.Event, already recorded once so that it exists) or
    clear (None) the event that two-pass calls on this thread record between
    their factorisation pass and their chain kernel
    (kda_profile_pass_event)."""
    h = None if event is None else ctypes.c_void_p(event.cuda_event)
    if event is not None and not event.cuda_event:
        raise ValueError("record the event once before passing it")
    st = library().kda_profile_pass_event(h)
    if st != 0:
        raise KdaError(st, "kda_profile_pass_event")


def workspace_pool():
    """(reserved, used) bytes of the device memory pool the library's
    stream-ordered workspace comes from (kda_workspace_pool)."""
    r, u = ctypes.c_size_t(), ctypes.c_size_t()
    st = library().kda_workspace_pool(ctypes.byref(r), ctypes.byref(u))
    if st != KDA_OK:
        raise KdaError(st, "kda_workspace_pool")
    return r.value, u.value


def device_status(stream=None):
    """Synchronise the stream and return the library's device-side status
    code (0 = no bounded wait ran out since the last call)."""
    return library().kda_device_status(_stream(stream))


NOALLOC_SCRATCH_BYTES = 16 << 20  # KDA_NOALLOC_SCRATCH_BYTES in include/kda.h


def chunk_fwd_noalloc(q, k, v, log_alpha, beta, initial_state=None,
                      cu_seqlens=None, chunk=64, out=None, final_state=None,
                      stream=None):
    """kda_chunk_fwd_staged_noalloc: the four-stage fp32 pipeline with its
    workspace in the library's fixed device array, for callers that must not
    allocate device memory during the call.  ``out`` and ``final_state``
    should be passed in by such callers (they are allocated here only when
    omitted).  Calls that overlap on the GPU race on the shared array."""
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    n = B if cu_seqlens is None else cu_seqlens.numel() - 1
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    if final_state is None:
        final_state = torch.empty((n, H, dk, dv), dtype=torch.float32,
                                  device=q.device)
    for name, t, dt in (("q", q, None), ("k", k, q.dtype), ("v", v, q.dtype),
                        ("log_alpha", log_alpha, torch.float32),
                        ("beta", beta, torch.float32),
                        ("initial_state", initial_state, torch.float32),
                        ("cu_seqlens", cu_seqlens, torch.int32),
                        ("out", out, q.dtype),
                        ("final_state", final_state, torch.float32)):
        _check_dev(name, t, dt)
    shape = KdaShape(B, T, H, dk, dv, chunk, n if cu_seqlens is not None else 0,
                     _io(q))
    st = library().kda_chunk_fwd_staged_noalloc(
        ctypes.byref(shape), _ptr(q), _ptr(k), _ptr(v), _ptr(log_alpha),
        _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens), _ptr(out),
        _ptr(final_state), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_chunk_fwd_staged_noalloc")
    return out, final_state


def selftest_timeout(limit_us=1000, stream=None):
    """Diagnostic (kda_selftest_timeout): a kernel whose bounded wait runs out
    after limit_us; the next device_status() then reports KDA_ERR_TIMEOUT."""
    st = library().kda_selftest_timeout(int(limit_us), _stream(stream))
    if st != KDA_OK:
        raise KdaError(st, "kda_selftest_timeout")


# ---- the operators around a recurrent layer (include/kda_layer.h) ----------

class _On:
    """The device of a call's tensors and the stream it is queued on.  The
    call runs with that device current, and what it allocates belongs to that
    stream, so it may be made from any device or stream; the caller orders
    the stream behind whatever wrote the inputs."""
    __slots__ = ("dev", "stream", "old_dev", "old_stream")

    def __init__(self, dev, stream):
        self.dev, self.stream = dev, stream

    def __enter__(self):
        dev, stream = self.dev, self.stream
        self.old_dev = self.old_stream = None
        if dev != torch.cuda.current_device():
            self.old_dev = torch.cuda.current_device()
            torch.cuda.set_device(dev)
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(dev)
        cur = torch.cuda.current_stream(dev)
        if stream != cur:
            if stream.device_index != dev:
                self.__exit__()
                raise ValueError("the stream must be on the tensors' device")
            self.old_stream = cur
            torch.cuda.set_stream(stream)
        return stream.cuda_stream

    def __exit__(self, *exc):
        if self.old_stream is not None:
            torch.cuda.set_stream(self.old_stream)
        if self.old_dev is not None:
            torch.cuda.set_device(self.old_dev)


def _device(name, t, dims=0):
    """The device index of a call's first tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dims and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got "
                         f"{tuple(t.shape)}")
    return t.get_device()


def _is(name, t, dev, dtype, shape):
    """Checks a tensor's device, dtype and shape."""
    if isinstance(t, torch.Tensor) and t.get_device() == dev and \
            t.dtype is dtype and t.shape == shape:
        return
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise ValueError(f"{name} must be a CUDA tensor on one device with "
                         "the others")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must have shape {tuple(shape)}, got "
                     f"{tuple(t.shape)}")


def _need(name, t, dev, dtype, shape, optional=False):
    """Checks a dense tensor of this dtype and shape (None where optional)."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    _is(name, t, dev, dtype, shape)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _tokens(name, t, dev, dtype, shape, inner=1):
    """Checks a tensor of this shape whose leading dims are tokens and whose
    last `inner` dims are one token's elements: dense within a token, tokens
    at one stride (a slice of a wider tensor will do).  Returns the stride."""
    _is(name, t, dev, dtype, shape)
    if t.is_contiguous() or t.numel() == 0:
        return 0
    stride = _token_stride(t, inner)
    if stride is None:
        raise ValueError(f"{name}: a token's elements must be dense and "
                         "consecutive tokens one stride apart")
    return stride


def _token_stride(t, inner):
    """The stride between the tokens of t (0: there is one token at most),
    None where its elements do not lie that way."""
    shape, st, lead = t.shape, t.stride(), t.dim() - inner
    width = 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if shape[i] != 1 and st[i] != width:
            return None
        width *= shape[i]
    stride = None  # dims of size 1 have no stride
    for i in range(lead - 1, -1, -1):
        if shape[i] == 1:
            continue
        if stride is None:
            stride = st[i]
            if stride < width:
                return None
            span = stride * shape[i]
        elif st[i] == span:
            span *= shape[i]
        else:
            return None
    return stride or 0


def _groups(name, t, dev, dtype, shape):
    """(token stride, group stride) of B or C [B, T, G, S]."""
    _is(name, t, dev, dtype, shape)
    if t.is_contiguous() or t.numel() == 0:
        return 0, 0
    b, n, g, s = shape
    st = t.stride()
    if s > 1 and st[3] != 1:
        raise ValueError(f"{name}: a group's states must be dense")
    group = st[2] if g > 1 else s
    if b > 1 and n > 1 and st[0] != n * st[1]:
        raise ValueError(f"{name}: consecutive tokens must be one stride "
                         "apart")
    token = st[1] if n > 1 else st[0] if b > 1 else g * group
    if group < s or token < (g - 1) * group + s:
        raise ValueError(f"{name}: tokens and groups must not overlap")
    return token, group


def _sequences(x, dev, cu_seqlens):
    """Sequences of a [B, T, ...] tensor, dense or packed, and the n_seqs that
    its shape struct takes."""
    if cu_seqlens is None:
        return x.shape[0], 0
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or \
            cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must hold n_seqs + 1 offsets")
    if x.shape[0] != 1:
        raise ValueError("a packed batch has B == 1")
    n = cu_seqlens.numel() - 1
    _need("cu_seqlens", cu_seqlens, dev, torch.int32, (n + 1,))
    return n, n


def _dims(*sizes):
    """The sizes of a call, refused where one does not fit the C ABI's 32-bit
    fields (ctypes would cut it)."""
    if max(sizes) > 0x7fffffff:
        raise ValueError(f"every size must be below 2^31, got {sizes}")
    return sizes


def _empty(t):
    """An uninitialised dense tensor of t's shape and dtype."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _run(name, shape, tensors, stream):
    st = getattr(library(), name)(
        ctypes.byref(shape),
        *[None if t is None else t.data_ptr() for t in tensors], stream)
    if st != KDA_OK:
        raise KdaError(st, name)


def _conv_shape(x, weight, bias, cu_seqlens, activation):
    """(shape struct, device, dims of x, dims of the states)"""
    dev, f32 = _device("x", x, 3), torch.float32
    full = x.shape
    n, packed = _sequences(x, dev, cu_seqlens)
    B, T, D = full
    if not isinstance(weight, torch.Tensor) or weight.dim() != 2:
        raise ValueError("weight must be [D, W]")
    W = weight.shape[1]
    _need("weight", weight, dev, f32, (D, W))
    _need("bias", bias, dev, f32, (D,), optional=True)
    shape = KdaConvShape(*_dims(B, T, D, W, packed), _io(x), ACTS[activation],
                         _tokens("x", x, dev, x.dtype, full))
    return shape, dev, full, (n, W - 1, D)


def short_conv_fwd(x, weight, bias=None, initial_state=None, cu_seqlens=None,
                   activation="silu", want_final_state=True, out=None,
                   stream=None):
    """Depthwise causal convolution over each sequence (kda_short_conv_fwd).

    x [B, T, D] (bf16 or fp32; may be a slice of a projection's output),
    weight [D, W] fp32 with W in {2, 3, 4}, bias [D] fp32 or None,
    initial_state [N, W-1, D] like x or None (zeros), activation "silu" or
    "none".  Returns (out [B, T, D], final_state [N, W-1, D] or None).
    """
    shape, dev, full, state = _conv_shape(x, weight, bias, cu_seqlens,
                                          activation)
    dt = x.dtype
    _need("initial_state", initial_state, dev, dt, state, optional=True)
    _need("out", out, dev, dt, full, optional=True)
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(x)
        final = x.new_empty(state) if want_final_state else None
        _run("kda_short_conv_fwd", shape,
             (x, weight, bias, initial_state, cu_seqlens, out, final), s)
    return out, final


def short_conv_bwd(x, weight, bias, initial_state, cu_seqlens, d_out,
                   d_final_state=None, activation="silu",
                   want_initial_state=True, stream=None):
    """Gradients of short_conv_fwd (kda_short_conv_bwd): (dx, d_weight,
    d_bias or None, d_initial_state or None)."""
    shape, dev, full, state = _conv_shape(x, weight, bias, cu_seqlens,
                                          activation)
    dt = x.dtype
    _need("initial_state", initial_state, dev, dt, state, optional=True)
    _need("d_out", d_out, dev, dt, full)
    _need("d_final_state", d_final_state, dev, dt, state, optional=True)
    with _On(dev, stream) as s:
        dx = _empty(x)
        dw = torch.empty_like(weight)
        db = None if bias is None else torch.empty_like(bias)
        d0 = x.new_empty(state) if want_initial_state else None
        _run("kda_short_conv_bwd", shape,
             (x, weight, bias, initial_state, cu_seqlens, d_out,
              d_final_state, dx, dw, db, d0), s)
    return dx, dw, db, d0


def short_conv_step(x, weight, bias, state, activation="silu", out=None,
                    stream=None):
    """The convolution of T >= 1 new tokens (kda_short_conv_step): x
    [N, T, D]; ``state`` [N, W-1, D] is updated in place.  Returns out."""
    shape, dev, full, st = _conv_shape(x, weight, bias, None, activation)
    dt = x.dtype
    _need("state", state, dev, dt, st)
    _need("out", out, dev, dt, full, optional=True)
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(x)
        _run("kda_short_conv_step", shape, (x, weight, bias, state, out), s)
    return out


def _ssm_shape(u, delta, A, Bm, Cm, D, z, delta_bias, cu_seqlens, softplus):
    """(shape struct, device, dims of u, dims of the states)"""
    dev, dt, f32 = _device("u", u, 3), u.dtype, torch.float32
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or \
            not isinstance(Bm, torch.Tensor) or Bm.dim() != 4:
        raise ValueError("A must be [D, S], Bm [B, T, G, S]")
    full = u.shape
    n, packed = _sequences(u, dev, cu_seqlens)
    B, T, C = full
    S, G = A.shape[1], Bm.shape[2]
    _need("A", A, dev, f32, (C, S))
    _need("D", D, dev, f32, (C,), optional=True)
    _need("delta_bias", delta_bias, dev, f32, (C,), optional=True)
    us = _tokens("u", u, dev, dt, full)
    ds = _tokens("delta", delta, dev, dt, full)
    zs = 0 if z is None else _tokens("z", z, dev, dt, full)
    bs, bg = _groups("Bm", Bm, dev, dt, (B, T, G, S))
    cs, cg = _groups("Cm", Cm, dev, dt, (B, T, G, S))
    shape = KdaSsmShape(*_dims(B, T, C, S, G, packed), _io(u),
                        1 if softplus else 0, us, ds, zs, bs, bg, cs, cg)
    return shape, dev, full, (n, C, S)


def ssm_scan_fwd(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None,
                 initial_state=None, cu_seqlens=None, softplus=True, out=None,
                 final_state=None, stream=None):
    """Selective state space scan (kda_ssm_scan_fwd).

    u, delta, z [B, T, D] and Bm, Cm [B, T, G, S] (bf16 or fp32, one dtype;
    slices of a projection's output will do; z may be None), A [D, S], D and
    delta_bias [D] fp32 (may be None), initial_state [N, D, S] fp32 or None.
    Returns (out [B, T, D], final_state [N, D, S] fp32); ``final_state`` may
    be the initial state itself.
    """
    shape, dev, full, state = _ssm_shape(u, delta, A, Bm, Cm, D, z,
                                         delta_bias, cu_seqlens, softplus)
    dt, f32 = u.dtype, torch.float32
    _need("initial_state", initial_state, dev, f32, state, optional=True)
    _need("out", out, dev, dt, full, optional=True)
    _need("final_state", final_state, dev, f32, state, optional=True)
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(u)
        if final_state is None:
            final_state = A.new_empty(state)
        _run("kda_ssm_scan_fwd", shape,
             (u, delta, A, Bm, Cm, D, z, delta_bias, initial_state,
              cu_seqlens, out, final_state), s)
    return out, final_state


def ssm_scan_bwd(u, delta, A, Bm, Cm, D=None, z=None, delta_bias=None,
                 initial_state=None, cu_seqlens=None, d_out=None,
                 d_final_state=None, softplus=True, want_initial_state=True,
                 stream=None):
    """Gradients of ssm_scan_fwd (kda_ssm_scan_bwd): (du, d_delta, dA, dBm,
    dCm, dD, dz, d_delta_bias, d_initial_state), None where the input is
    None (d_initial_state: unless want_initial_state)."""
    shape, dev, full, state = _ssm_shape(u, delta, A, Bm, Cm, D, z,
                                         delta_bias, cu_seqlens, softplus)
    dt, f32 = u.dtype, torch.float32
    _need("initial_state", initial_state, dev, f32, state, optional=True)
    _need("d_out", d_out, dev, dt, full)
    _need("d_final_state", d_final_state, dev, f32, state, optional=True)
    with _On(dev, stream) as s:
        du, dd = _empty(u), _empty(u)
        dA = torch.empty_like(A)
        dB, dC = _empty(Bm), _empty(Bm)
        dD = None if D is None else torch.empty_like(D)
        dz = None if z is None else _empty(u)
        db = None if delta_bias is None else torch.empty_like(delta_bias)
        d0 = A.new_empty(state) if want_initial_state else None
        _run("kda_ssm_scan_bwd", shape,
             (u, delta, A, Bm, Cm, D, z, delta_bias, initial_state,
              cu_seqlens, d_out, d_final_state, du, dd, dA, dB, dC, dD, dz,
              db, d0), s)
    return du, dd, dA, dB, dC, dD, dz, db, d0


def ssm_scan_bwd_plan(B, T, D, S, G, dtype, packed=False, n_seqs=0):
    """(kernels, workspace_bytes) of an ssm_scan_bwd call of this shape."""
    io = KDA_BF16 if dtype == torch.bfloat16 else KDA_F32
    shape = KdaSsmShape(*_dims(B, T, D, S, G, n_seqs if packed else 0), io, 1)
    kern, ws = ctypes.c_int(), ctypes.c_size_t()
    st = library().kda_ssm_scan_bwd_plan(ctypes.byref(shape), int(packed),
                                         ctypes.byref(kern), ctypes.byref(ws))
    if st != KDA_OK:
        raise KdaError(st, "kda_ssm_scan_bwd_plan")
    return kern.value, ws.value


def ssm_step(u, delta, A, Bm, Cm, state, D=None, z=None, delta_bias=None,
             softplus=True, out=None, stream=None):
    """The scan over T >= 1 new tokens (kda_ssm_step): u, delta, z [N, T, D],
    Bm, Cm [N, T, G, S]; ``state`` [N, D, S] fp32 is updated in place.
    Returns out [N, T, D]."""
    shape, dev, full, st = _ssm_shape(u, delta, A, Bm, Cm, D, z, delta_bias,
                                      None, softplus)
    dt = u.dtype
    _need("state", state, dev, torch.float32, st)
    _need("out", out, dev, dt, full, optional=True)
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(u)
        _run("kda_ssm_step", shape,
             (u, delta, A, Bm, Cm, D, z, delta_bias, state, out), s)
    return out


def _norm_shape(x, post_weight, gate, residual, scale, pre_weight, rt,
                gate_act, gate_first, eps):
    """(shape struct, device)"""
    dev, dt, f32 = _device("x", x), x.dtype, torch.float32
    if x.dim() < 2 or x.shape[-1] == 0:
        raise ValueError("x must be [..., width]")
    width = x.shape[-1]
    # rows at one stride, else tokens of `heads` dense rows at one stride
    inner = 1
    for t in (x, gate):
        if isinstance(t, torch.Tensor) and not t.is_contiguous() and \
                t.dim() > 2 and _token_stride(t, 1) is None:
            inner = 2
    heads = x.shape[-2] if inner == 2 else 1
    tokens = x.numel() // (heads * width) if x.numel() else 0
    _need("post_weight", post_weight, dev, f32, (width,), optional=True)
    _need("scale", scale, dev, f32, (width,), optional=True)
    _need("pre_weight", pre_weight, dev, f32, (width,), optional=True)
    _need("residual", residual, dev, rt, x.shape, optional=True)
    xs = _tokens("x", x, dev, dt, x.shape, inner)
    gs = 0 if gate is None else _tokens("gate", gate, dev, dt, x.shape, inner)
    if rt not in (dt, f32):
        raise ValueError(f"the residual must be {dt} or float32, got {rt}")
    return KdaNormShape(tokens, *_dims(max(heads, 1), width), _io(x),
                        KDA_BF16 if rt == torch.bfloat16 else KDA_F32,
                        ACTS[gate_act], 1 if gate_first else 0, eps, xs,
                        gs), dev


def block_norm_fwd(x, post_weight=None, gate=None, residual=None, scale=None,
                   pre_weight=None, gate_act="sigmoid", gate_first=False,
                   eps=1e-6, out=None, normed=None, stream=None):
    """The norm after a block with its gate, the residual scale and sum, and
    the next block's norm (kda_block_norm_fwd), each part optional:

        h = x [act(gate) with gate_first]
        p = rms(h) post_weight [act(gate) otherwise]
        out = residual + scale p;  normed = rms(out) pre_weight

    x, gate [..., width] (bf16 or fp32; the norms are over the last dim;
    slices of a projection's output will do: rows at one stride, or tokens
    [..., heads, width] at one stride with dense heads, and x and gate in the
    same of these two forms unless one of them is contiguous), residual the
    same shape in x's dtype or fp32, weights and scale [width] fp32,
    ``gate_act`` "sigmoid", "silu" or "none".  ``out`` may be the residual
    itself.  Returns (out in the residual's dtype, normed in x's or None).
    """
    rt = residual.dtype if isinstance(residual, torch.Tensor) else \
        out.dtype if isinstance(out, torch.Tensor) else x.dtype
    shape, dev = _norm_shape(x, post_weight, gate, residual, scale,
                             pre_weight, rt, gate_act, gate_first, eps)
    dt = x.dtype
    _need("out", out, dev, rt, x.shape, optional=True)
    _need("normed", normed, dev, dt, x.shape, optional=True)
    with _On(dev, stream) as s:
        if out is None:
            out = _empty(x if residual is None else residual)
        if normed is None and pre_weight is not None:
            normed = _empty(x)
        _run("kda_block_norm_fwd", shape,
             (x, post_weight, gate, residual, scale, pre_weight, out, normed),
             s)
    return out, normed


def block_norm_bwd(x, post_weight=None, gate=None, residual=None, scale=None,
                   pre_weight=None, d_out=None, d_normed=None,
                   gate_act="sigmoid", gate_first=False, eps=1e-6,
                   stream=None):
    """Gradients of block_norm_fwd (kda_block_norm_bwd): (dx, dgate,
    d_residual, d_post_weight, d_scale, d_pre_weight), None where the input
    is None.  d_out has the dtype of out, d_normed of x; either may be None
    (zero)."""
    rt = residual.dtype if isinstance(residual, torch.Tensor) else \
        d_out.dtype if isinstance(d_out, torch.Tensor) else x.dtype
    shape, dev = _norm_shape(x, post_weight, gate, residual, scale,
                             pre_weight, rt, gate_act, gate_first, eps)
    dt = x.dtype
    _need("d_out", d_out, dev, rt, x.shape, optional=True)
    _need("d_normed", d_normed, dev, dt, x.shape, optional=True)

    def like(t):
        return None if t is None else _empty(t)
    with _On(dev, stream) as s:
        dx, dg, dr = like(x), like(gate), like(residual)
        dpost, dscale, dpre = like(post_weight), like(scale), like(pre_weight)
        _run("kda_block_norm_bwd", shape,
             (x, post_weight, gate, residual, scale, pre_weight, d_out,
              d_normed, dx, dg, dr, dpost, dscale, dpre), s)
    return dx, dg, dr, dpost, dscale, dpre
