"""DeepSeek sparse attention (DSA) hot path on GB300: lightning indexer ->
top-k -> absorbed sparse latent attention, in hand-written sm_103a CUDA
behind the C ABI of ``libdsa.so`` (include/dsa.h).

This module is the thin Python binding: it marshals torch tensors (device
memory, the current stream) into the C calls of the same names.  Every
arithmetic step runs in the CUDA kernels; there is no CPU fallback, and a
missing ``libdsa.so`` raises.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import functools

import torch

from . import _abi
from ._abi import DSA_BF16, DSA_E4M3, DSA_F32, KERNEL_BITS

__all__ = [
    "Seqs", "DSAError", "dsa_quant_e4m3_ue8m0", "dsa_indexer_scores", "dsa_topk_select",
    "dsa_sparse_mla_workspace_size", "dsa_sparse_mla_fwd", "dsa_forward_workspace_size", "dsa_forward",
    "dsa_check_device_error", "dsa_selftest_bounded_wait", "dsa_set_wait_limit", "dsa_set_fused_topk", "dsa_kv_prologue",
    "dsa_output_proj", "dsa_sparse_mla_fwd_fp8kv", "dsa_forward_host", "last_kernels", "last_launch_count", "build",
    "Pages", "LatentCache", "Heads", "dsa_latent_cache_write", "dsa_latent_cache_read", "dsa_tree_mla_workspace_size",
    "dsa_tree_mla_fwd", "dsa_head_norm_rope",
]


class DSAError(RuntimeError):
    def __init__(self, fn: str, status: int):
        lib = _abi.load()
        msg = lib.dsa_status_string(status).decode()
        if status == _abi.DSA_ERR_CUDA:
            msg += f" (cudaError {lib.dsa_last_cuda_error()})"
        super().__init__(f"{fn}: {msg}")
        self.status = status


def build(force: bool = False) -> str:
    from .build import build as _b
    return _b(force=force)


def _check(fn: str, status: int):
    if status != _abi.DSA_OK:
        raise DSAError(fn, status)


def _int32s(values):
    """A C array of the values (through ``array``, which takes a list ten times as fast as ctypes does)."""
    values = values if isinstance(values, list) else list(values)  # (array would take the bytes of a bytes object as memory)
    try:
        a = array.array("i", values)
    except TypeError:  # tensors of one value and other things that only int() takes
        a = array.array("i", [int(x) for x in values])
    return (ctypes.c_int32 * len(a)).from_buffer(a) if a else (ctypes.c_int32 * 1)()


class Seqs:
    """A batch description (host arrays): cu_q [B+1], cu_k [B+1], start_pos [B]."""

    def __init__(self, cu_q, cu_k, start_pos):
        B = len(start_pos)
        assert len(cu_q) == B + 1 and len(cu_k) == B + 1
        self._q, self._k, self._p = _int32s(cu_q), _int32s(cu_k), _int32s(start_pos)
        self.struct = _abi.dsa_seqs(B, self._q, self._k, self._p)
        self.B = B
        self.total_q = self._q[B]
        self.total_k = self._k[B]

    @functools.cached_property
    def max_S(self) -> int:
        k = self._k[:]
        return max((b - a for a, b in zip(k, k[1:])), default=0)

    @classmethod
    def from_lengths(cls, T, S, start_pos):
        cu_q, cu_k = [0], [0]
        for t, s in zip(T, S):
            cu_q.append(cu_q[-1] + int(t))
            cu_k.append(cu_k[-1] + int(s))
        return cls(cu_q, cu_k, start_pos)

    def ref(self):
        return ctypes.byref(self.struct)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DSA_F32
    if t.dtype == torch.bfloat16:
        return DSA_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return DSA_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _row_stride(t: torch.Tensor) -> int:
    assert t.dim() == 2 and t.stride(1) == 1, "rows must be contiguous"
    return t.stride(0)


def last_kernels() -> set:
    bits = _abi.load().dsa_last_kernels()
    return {k for k, v in KERNEL_BITS.items() if bits & v}


def last_launch_count() -> int:
    return _abi.load().dsa_last_launch_count()


def dsa_check_device_error(stream=None):
    site = ctypes.c_int(0)
    st = _abi.load().dsa_check_device_error(_stream(stream), ctypes.byref(site))
    return st, site.value


def dsa_selftest_bounded_wait(limit_cycles: int, completed_ok=None, stream=None):
    """Launch the bounded-wait self-test (a wait that runs out after limit_cycles);
    read its outcome with dsa_check_device_error."""
    _check("dsa_selftest_bounded_wait",
           _abi.load().dsa_selftest_bounded_wait(int(limit_cycles), _ptr(completed_ok) if completed_ok is not None else None,
                                                 _stream(stream)))


def dsa_set_wait_limit(cycles: int):
    """Wait limit (SM cycles) of the tensor-core kernels' bounded waits; 0 restores the default."""
    _check("dsa_set_wait_limit", _abi.load().dsa_set_wait_limit(int(cycles)))


def dsa_set_fused_topk(mode):
    """Fused indexer + top-k for the dsa_forward calls that follow on large batches:
    True/1 wherever it applies, False/0 never, -1 the library's choice (default)."""
    m = -1 if mode == -1 else (1 if mode else 0)
    _check("dsa_set_fused_topk", _abi.load().dsa_set_fused_topk(m))


def dsa_quant_e4m3_ue8m0(x: torch.Tensor, codes=None, scales=None, stream=None):
    """x: [..., 128k] f32/bf16 -> (codes uint8 same shape, scales f32 [numel/128])."""
    x = x.contiguous()
    nb = x.numel() // 128
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device) if codes is None else codes
    scales = torch.empty(nb, dtype=torch.float32, device=x.device) if scales is None else scales
    _check("dsa_quant_e4m3_ue8m0", _abi.load().dsa_quant_e4m3_ue8m0(_ptr(x), _dt(x), nb, _ptr(codes), _ptr(scales),
                                                                    _stream(stream)))
    return codes, scales


def dsa_indexer_scores(q_idx, k_idx, w, seqs: Seqs, q_scale=None, k_scale=None, scores=None, ld=None, stream=None):
    H_I, D_I = q_idx.shape[-2], q_idx.shape[-1]
    if ld is None:
        ld = (max(seqs.max_S, 1) + 3) // 4 * 4
    if scores is None:
        scores = torch.empty((seqs.total_q, ld), dtype=torch.float32, device=q_idx.device)
    st = _abi.load().dsa_indexer_scores(_ptr(q_idx), _ptr(q_scale), _ptr(k_idx), _ptr(k_scale), _dt(q_idx), _ptr(w),
                                        H_I, D_I, seqs.ref(), _ptr(scores), scores.stride(0), _stream(stream))
    _check("dsa_indexer_scores", st)
    return scores


def dsa_topk_select(scores, seqs: Seqs, k: int, idx=None, stream=None):
    if idx is None:
        idx = torch.empty((seqs.total_q, k), dtype=torch.int32, device=scores.device)
    st = _abi.load().dsa_topk_select(_ptr(scores), scores.stride(0), seqs.ref(), k, _ptr(idx), _stream(stream))
    _check("dsa_topk_select", st)
    return idx


def dsa_sparse_mla_workspace_size(dtype: int, H: int, d_n: int, d_r: int, d_c: int, d_v: int, k: int,
                                  seqs: Seqs) -> int:
    return _abi.load().dsa_sparse_mla_workspace_size(dtype, H, d_n, d_r, d_c, d_v, k, seqs.ref())


def dsa_sparse_mla_fwd(q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, idx, seqs: Seqs, softmax_scale: float, out=None,
                       lse=None, workspace=None, want_lse=True, stream=None, k=None):
    """kv_cache and k_pe are 2-D views [sum S, d_c] / [sum S, d_r] with contiguous rows
    (k_pe may be a column slice of a packed cache).  idx=None selects the dense causal
    pattern (entry e of a row is key e) for k entries per row."""
    M, H, d_n = q_nope.shape
    d_r = q_pe.shape[2]
    d_c = W_UK.shape[2]
    d_v = W_UV.shape[2]
    if idx is not None:
        k = idx.shape[1]
    elif k is None:
        raise ValueError("dsa_sparse_mla_fwd: idx=None needs k")
    dt = _dt(q_nope)
    dev = q_nope.device
    if out is None:
        out = torch.empty((M, H, d_v), dtype=q_nope.dtype, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((M, H), dtype=torch.float32, device=dev)
    need = dsa_sparse_mla_workspace_size(dt, H, d_n, d_r, d_c, d_v, k, seqs)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = _abi.load().dsa_sparse_mla_fwd(_ptr(q_nope), _ptr(q_pe), dt, _ptr(kv_cache), _row_stride(kv_cache), _ptr(k_pe),
                                        _row_stride(k_pe), _ptr(W_UK), _ptr(W_UV), H, d_n, d_r, d_c, d_v, _ptr(idx), k,
                                        seqs.ref(), float(softmax_scale), _ptr(out), _ptr(lse), _ptr(workspace),
                                        workspace.numel(), _stream(stream))
    _check("dsa_sparse_mla_fwd", st)
    return out, lse


def dsa_kv_prologue(x, W_proj, kv_gain, k_gain, k_bias, rope_cos, rope_sin, seqs: Seqs, kv_cache, k_cache, w=None,
                    k_scale=None, d_c=512, d_r=64, D_I=128, H_I=64, workspace=None, stream=None):
    """The step before the path for the new tokens x [sum T, dim]: writes their
    rows of kv_cache ([sum S, >= d_c + d_r] bf16) and k_cache ([sum S, D_I] bf16,
    or uint8 e4m3 codes with k_scale [sum S]) and returns w [sum T, H_I]."""
    dim = x.shape[1]
    dev = x.device
    if w is None:
        w = torch.empty((seqs.total_q, H_I), dtype=torch.float32, device=dev)
    k_dtype = DSA_E4M3 if k_cache.dtype in (torch.uint8, torch.float8_e4m3fn) else DSA_BF16
    lib = _abi.load()
    need = lib.dsa_kv_prologue_workspace_size(dim, d_c, d_r, D_I, H_I, seqs.ref())
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = lib.dsa_kv_prologue(_ptr(x), dim, _ptr(W_proj), _ptr(kv_gain), _ptr(k_gain), _ptr(k_bias), _ptr(rope_cos),
                             _ptr(rope_sin), rope_cos.shape[0], d_c, d_r, D_I, H_I, seqs.ref(), _ptr(kv_cache),
                             _row_stride(kv_cache), _ptr(k_cache), k_dtype, _ptr(k_scale), _ptr(w), _ptr(workspace),
                             workspace.numel(), _stream(stream))
    _check("dsa_kv_prologue", st)
    return w


def dsa_output_proj(out, wo, y=None, stream=None):
    """y = out wo^T with out [M, H, d_v] (or [M, H * d_v]) and wo [d_model, H * d_v], bf16."""
    M = out.shape[0]
    K = out[0].numel() if M else wo.shape[1]
    d_model = wo.shape[0]
    if y is None:
        y = torch.empty((M, d_model), dtype=out.dtype, device=out.device)
    _check("dsa_output_proj", _abi.load().dsa_output_proj(_ptr(out), _ptr(wo), M, K, d_model, _ptr(y), _stream(stream)))
    return y


def dsa_sparse_mla_fwd_fp8kv(q_nope, q_pe, kv_codes, kv_scale, k_pe, W_UK, W_UV, idx, seqs: Seqs,
                             softmax_scale: float, out=None, lse=None, workspace=None, stream=None):
    """The sparse attention over an FP8 latent cache: kv_codes [sum S, >= d_c] uint8
    e4m3 codes with kv_scale [sum S, d_c / 128] fp32 block scales; k_pe bf16."""
    M, H, d_n = q_nope.shape
    d_r, d_c, d_v = q_pe.shape[2], W_UK.shape[2], W_UV.shape[2]
    k = idx.shape[1]
    dev = q_nope.device
    if out is None:
        out = torch.empty((M, H, d_v), dtype=q_nope.dtype, device=dev)
    if lse is None:
        lse = torch.empty((M, H), dtype=torch.float32, device=dev)
    need = dsa_sparse_mla_workspace_size(DSA_BF16, H, d_n, d_r, d_c, d_v, k, seqs)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
    st = _abi.load().dsa_sparse_mla_fwd_fp8kv(_ptr(q_nope), _ptr(q_pe), _ptr(kv_codes), _row_stride(kv_codes),
                                              _ptr(kv_scale), _ptr(k_pe), _row_stride(k_pe), _ptr(W_UK), _ptr(W_UV), H,
                                              d_n, d_r, d_c, d_v, _ptr(idx), k, seqs.ref(), float(softmax_scale),
                                              _ptr(out), _ptr(lse), _ptr(workspace), workspace.numel(),
                                              _stream(stream))
    _check("dsa_sparse_mla_fwd_fp8kv", st)
    return out, lse


def _problem(q_idx, k_idx, w, q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, top_k, softmax_scale, idx_fp8, out, lse,
             idx_out, wo=None, y=None, kv_scale=None):
    p = _abi.dsa_problem()
    p.H_I, p.D_I = q_idx.shape[-2], q_idx.shape[-1]
    p.top_k = top_k
    p.H, p.d_n = q_nope.shape[1], q_nope.shape[2]
    p.d_r = q_pe.shape[2]
    p.d_c = W_UK.shape[2]
    p.d_v = W_UV.shape[2]
    p.dtype = _dt(q_nope)
    p.idx_fp8 = 1 if idx_fp8 else 0
    p.softmax_scale = float(softmax_scale)
    p.q_idx, p.k_idx, p.w = q_idx.data_ptr(), k_idx.data_ptr(), w.data_ptr()
    p.q_nope, p.q_pe = q_nope.data_ptr(), q_pe.data_ptr()
    p.kv_cache, p.ld_kv = kv_cache.data_ptr(), _row_stride(kv_cache)
    p.k_pe, p.ld_pe = k_pe.data_ptr(), _row_stride(k_pe)
    p.W_UK, p.W_UV = W_UK.data_ptr(), W_UV.data_ptr()
    p.out = out.data_ptr() if out is not None else None
    p.lse = lse.data_ptr() if lse is not None else None
    p.idx_out = idx_out.data_ptr() if idx_out is not None else None
    if wo is not None:
        p.wo, p.d_model, p.y = wo.data_ptr(), wo.shape[0], y.data_ptr()
    if kv_scale is not None:
        p.kv_fp8, p.kv_scale = 1, kv_scale.data_ptr()
    return p


def dsa_forward_workspace_size(problem, seqs: Seqs) -> int:
    return _abi.load().dsa_forward_workspace_size(ctypes.byref(problem), seqs.ref())


def dsa_forward(q_idx, k_idx, w, q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, seqs: Seqs, top_k: int,
                softmax_scale: float, idx_fp8: bool = False, out=None, lse=None, idx_out=None, workspace=None,
                want_lse=True, want_idx=True, stream=None, wo=None, y=None, want_out=True, kv_scale=None):
    """The whole path.  Returns (out [sum T, H, d_v] or None, lse [sum T, H] or None,
    idx [sum T, top_k] or None), plus y [sum T, d_model] = out wo^T when wo is given
    (the step after the path; with want_out=False the attention output stays in
    the workspace).  With kv_scale, kv_cache holds the latent rows as e4m3 codes
    (uint8) with kv_scale [sum S, d_c / 128] block scales."""
    dev = q_nope.device
    M, H = q_nope.shape[0], q_nope.shape[1]
    if out is None and (want_out or wo is None):
        out = torch.empty((M, H, W_UV.shape[2]), dtype=q_nope.dtype, device=dev)
    if lse is None and want_lse:
        lse = torch.empty((M, H), dtype=torch.float32, device=dev)
    if idx_out is None and want_idx:
        idx_out = torch.empty((M, top_k), dtype=torch.int32, device=dev)
    if wo is not None and y is None:
        y = torch.empty((M, wo.shape[0]), dtype=q_nope.dtype, device=dev)
    p = _problem(q_idx, k_idx, w, q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, top_k, softmax_scale, idx_fp8, out, lse,
                 idx_out, wo, y, kv_scale)
    need = dsa_forward_workspace_size(p, seqs)
    if need == 0 and M > 0:
        raise DSAError("dsa_forward_workspace_size", _abi.DSA_ERR_INVALID_ARG)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=dev)
        if stream is not None:  # freed on return while the call's kernels may still run on `stream`
            workspace.record_stream(stream)
    st = _abi.load().dsa_forward(ctypes.byref(p), seqs.ref(), _ptr(workspace), workspace.numel(), _stream(stream))
    _check("dsa_forward", st)
    if wo is not None:
        return out, lse, idx_out, y
    return out, lse, idx_out


def dsa_forward_host(host: dict, q_idx, k_idx, w, q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, seqs: Seqs, top_k: int,
                     softmax_scale: float, idx_fp8: bool = False, out=None, lse=None, idx_out=None, workspace=None,
                     stream=None, wo=None, y=None, kv_scale=None, compute_after=None, compute_done=None,
                     copy_after=None, copy_done=None):
    """One step from HOST tensors (the end-to-end call).  ``host`` maps names to CPU
    tensors (pinned for asynchronous copies): inputs ``q_idx``, ``w``, ``q_nope``,
    ``q_pe`` (the step's queries) and ``kv_new``, ``k_pe_new``, ``k_idx_new``,
    ``kv_scale_new`` (the cache rows the step appends: rows start_pos[b] .. S_b - 1
    of every sequence, concatenated), outputs ``out`` (y with wo), ``lse``, ``idx``;
    a missing name is not copied.  The device tensors are the buffers the copies fill
    and the forward reads and writes.  Everything is enqueued on ``stream``, except the
    copies of q_nope and q_pe, which run on the library's side stream while the indexer
    runs (the attention waits for them on ``stream``); returns without synchronising.  ``compute_after`` / ``compute_done`` (torch.cuda.Event):
    the forward waits for the first after the input copies and records the second
    before the output copies, to chain the forwards of calls on two streams;
    ``copy_after`` / ``copy_done``: the input copies wait for the first and the
    second is recorded once they (and the append kernel) are enqueued, to chain
    the input copies of calls on two streams."""
    lib = _abi.load()
    p = _problem(q_idx, k_idx, w, q_nope, q_pe, kv_cache, k_pe, W_UK, W_UV, top_k, softmax_scale, idx_fp8, out, lse,
                 idx_out, wo, y, kv_scale)
    io = _abi.dsa_host_io()
    for name in ("q_idx", "w", "q_nope", "q_pe", "kv_new", "k_pe_new", "k_idx_new", "kv_scale_new", "out", "lse",
                 "idx"):
        ten = host.get(name)
        if ten is not None:
            if ten.device.type != "cpu" or not ten.is_contiguous():
                raise ValueError(f"host tensor {name} must be a contiguous CPU tensor")
            setattr(io, name, ten.data_ptr())
    for name, ev in (("compute_after", compute_after), ("compute_done", compute_done), ("copy_after", copy_after),
                     ("copy_done", copy_done)):
        if ev is not None:
            if not ev.cuda_event:  # torch creates the CUDA event on its first record
                ev.record()
            setattr(io, name, ev.cuda_event)
    need = dsa_forward_workspace_size(p, seqs)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=q_nope.device)
        if stream is not None:  # freed on return while the call's kernels may still run on `stream`
            workspace.record_stream(stream)
    st = lib.dsa_forward_host(ctypes.byref(p), seqs.ref(), ctypes.byref(io), _ptr(workspace), workspace.numel(),
                              _stream(stream))
    _check("dsa_forward_host", st)


def set_stage_events(events):
    """Record ``events`` (DSA_STAGE_EVENTS torch.cuda.Event objects, or None to
    switch off) at the stage boundaries of the next dsa_forward calls."""
    lib = _abi.load()
    if events is None:
        _check("dsa_set_stage_events", lib.dsa_set_stage_events(None, 0))
        return
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check("dsa_set_stage_events", lib.dsa_set_stage_events(arr, len(events)))


# ---------------------------------------------------------------------------------------------------------------
# Speculative decoding over a served latent cache
# ---------------------------------------------------------------------------------------------------------------
def _on_one_device(fn: str, tensors) -> int:
    """The index of the CUDA device that every tensor (of pairs of a name and a tensor or None) is on."""
    dev = -1
    for name, t in tensors:
        if t is None:
            continue
        d = t.get_device()
        if d < 0:
            raise ValueError(f"{fn}: {name} must be a CUDA tensor, is on {t.device}")
        if dev >= 0 and d != dev:
            raise ValueError(f"{fn}: {name} is on {t.device}, other arguments on cuda:{dev}")
        dev = d
    return dev


_NOTHING = contextlib.nullcontext()


def _launching(dev: int, stream):
    """The context of a call on device ``dev``: launches go to ``stream`` (default: the current one) with ``dev``
    current, and what is allocated meanwhile belongs to that stream."""
    if stream is None:
        return _NOTHING if torch._C._cuda_getDevice() == dev else torch.cuda.device(dev)
    if stream.device.index != dev:
        raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{dev}")
    return torch.cuda.stream(stream)


def _int32(fn: str, name: str, t, n: int):
    if t is not None and (t.dtype != torch.int32 or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{fn}: {name} must be a contiguous int32 tensor [{n}]")


class Pages:
    """Where the sequences' tokens sit in a paged cache: token s of sequence b is row
    ``block_table[b, s // page_size] * page_size + s % page_size``.  ``block_table``: int32
    [B, pages per sequence] on the device, -1 (or any page that is none) for no page."""

    def __init__(self, block_table: torch.Tensor, page_size: int, n_pages: int):
        if block_table.dim() != 2 or block_table.dtype != torch.int32 or \
                (block_table.shape[1] > 1 and block_table.stride(1) != 1):
            raise ValueError("Pages: block_table must be a 2-D int32 tensor with contiguous rows")
        rows, width = block_table.shape
        ld = block_table.stride(0) if rows > 1 else width
        if ld < width:
            raise ValueError("Pages: the rows of block_table overlap")
        self.block_table, self.rows = block_table, rows
        self.struct = _abi.dsa_pages(block_table.data_ptr(), ld, width, page_size, n_pages)

    def ref(self, fn: str, seqs: Seqs):
        if self.rows < seqs.B:
            raise ValueError(f"{fn}: block_table has {self.rows} rows for {seqs.B} sequences")
        return ctypes.byref(self.struct)


class LatentCache:
    """A latent cache: ``kv`` [rows, d_c] values (fp32 or bf16) or e4m3 codes (uint8 or float8_e4m3fn) with
    ``kv_scale`` [rows, d_c / 128] fp32, and the rotary keys ``k_pe`` [rows, d_r] (bf16 with codes, else kv's
    type).  Both may be column slices of a packed buffer.  A cache cut into pages is given flat."""

    def __init__(self, kv: torch.Tensor, k_pe: torch.Tensor, kv_scale: torch.Tensor | None = None):
        dt = _dt(kv)
        rows, d_c = _rows_2d("LatentCache", "kv", kv)
        _, d_r = _rows_2d("LatentCache", "k_pe", k_pe, None, rows)
        if k_pe.dtype != (torch.bfloat16 if dt == DSA_E4M3 else kv.dtype):
            raise ValueError(f"LatentCache: k_pe is {k_pe.dtype} beside {kv.dtype} latents")
        if (kv_scale is not None) != (dt == DSA_E4M3):
            raise ValueError("LatentCache: kv_scale goes with e4m3 codes, and only with them")
        if kv_scale is not None and (kv_scale.dtype != torch.float32 or not kv_scale.is_contiguous() or
                                     kv_scale.shape != (rows, d_c // 128)):
            raise ValueError("LatentCache: kv_scale must be contiguous fp32 [rows, d_c / 128]")
        self.kv, self.k_pe, self.kv_scale = kv, k_pe, kv_scale
        self.d_c, self.d_r, self.rows = d_c, d_r, rows
        self.struct = _abi.dsa_latent_cache(
            kv.data_ptr(), _ld(kv), None if kv_scale is None else kv_scale.data_ptr(),
            k_pe.data_ptr() if d_r else None, _ld(k_pe), dt, rows)

    def ref(self):
        return ctypes.byref(self.struct)

    def tensors(self):
        return ("cache.kv", self.kv), ("cache.k_pe", self.k_pe), ("cache.kv_scale", self.kv_scale)


def _rows_2d(fn: str, name: str, t: torch.Tensor, width=None, rows=None):
    shape = t.shape
    if len(shape) != 2 or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{fn}: {name} must be 2-D with contiguous rows")
    if (width is not None and shape[1] != width) or (rows is not None and shape[0] != rows):
        raise ValueError(f"{fn}: {name} has shape {tuple(shape)}, expected ({rows}, {width})")
    return shape


def _ld(t: torch.Tensor) -> int:
    """Row stride; a single row's is its width rounded up to 16 bytes (torch gives such a stride any value)."""
    if t.shape[0] > 1:
        return t.stride(0)
    per = 16 // t.element_size()
    return (t.shape[1] + per - 1) // per * per


def _table(pages):
    return "block_table", None if pages is None else pages.block_table


def _ref_pages(fn, pages, seqs):
    return None if pages is None else pages.ref(fn, seqs)


def _addr(t):
    return None if t is None else t.data_ptr()


def dsa_latent_cache_write(c_kv, k_pe, cache: LatentCache, seqs: Seqs, pages: Pages | None = None, stream=None):
    """Write the new tokens' latent rows c_kv [sum T, d_c] and rotary keys k_pe [sum T, d_r] (fp32 or bf16) into the
    cache as tokens start_pos[b] + t of their sequences, quantising them when the cache holds e4m3 codes."""
    fn = "dsa_latent_cache_write"
    dev = _on_one_device(fn, (("c_kv", c_kv), ("k_pe", k_pe), _table(pages)) + cache.tensors())
    _rows_2d(fn, "c_kv", c_kv, cache.d_c, seqs.total_q)
    _rows_2d(fn, "k_pe", k_pe, cache.d_r, seqs.total_q)
    if k_pe.dtype != c_kv.dtype:
        raise ValueError(f"{fn}: k_pe is {k_pe.dtype}, c_kv {c_kv.dtype}")
    with _launching(dev, stream):
        _check(fn, _abi.load().dsa_latent_cache_write(
            c_kv.data_ptr(), _ld(c_kv), k_pe.data_ptr() if cache.d_r else None, _ld(k_pe), _dt(c_kv), cache.d_c,
            cache.d_r, cache.ref(), seqs.ref(), _ref_pages(fn, pages, seqs), torch._C._cuda_getCurrentRawStream(dev)))


def dsa_latent_cache_read(cache: LatentCache, seqs: Seqs, pages: Pages | None = None, pos=None, dtype=torch.bfloat16,
                          c_kv=None, k_pe=None, stream=None):
    """Read tokens back, dequantised: row cu_q[b] + t is token pos[row] (int32 [sum T]) of sequence b, or
    start_pos[b] + t without pos; zeros where there is no such token.  Returns (c_kv [sum T, d_c],
    k_pe [sum T, d_r]) of ``dtype``."""
    fn = "dsa_latent_cache_read"
    dev = _on_one_device(fn, (("pos", pos), ("c_kv", c_kv), ("k_pe", k_pe), _table(pages)) + cache.tensors())
    _int32(fn, "pos", pos, seqs.total_q)
    with _launching(dev, stream):
        if c_kv is None:
            c_kv = torch.empty((seqs.total_q, cache.d_c), dtype=dtype, device=cache.kv.device)
        else:
            _rows_2d(fn, "c_kv", c_kv, cache.d_c, seqs.total_q)
        if k_pe is None:
            k_pe = torch.empty((seqs.total_q, cache.d_r), dtype=c_kv.dtype, device=c_kv.device)
        else:
            _rows_2d(fn, "k_pe", k_pe, cache.d_r, seqs.total_q)
            if k_pe.dtype != c_kv.dtype:
                raise ValueError(f"{fn}: k_pe is {k_pe.dtype}, c_kv {c_kv.dtype}")
        _check(fn, _abi.load().dsa_latent_cache_read(
            cache.ref(), cache.d_c, cache.d_r, seqs.ref(), _ref_pages(fn, pages, seqs), _addr(pos), c_kv.data_ptr(),
            _ld(c_kv), k_pe.data_ptr() if cache.d_r else None, _ld(k_pe), _dt(c_kv),
            torch._C._cuda_getCurrentRawStream(dev)))
    return c_kv, k_pe


def dsa_tree_mla_workspace_size(dtype: int, H: int, d_n: int, d_r: int, d_c: int, d_v: int, seqs: Seqs) -> int:
    return _abi.load().dsa_tree_mla_workspace_size(dtype, H, d_n, d_r, d_c, d_v, seqs.ref())


def dsa_tree_mla_fwd(q_nope, q_pe, cache: LatentCache, W_UK, W_UV, seqs: Seqs, softmax_scale: float, tree_mask=None,
                     pages: Pages | None = None, out=None, lse=None, workspace=None, want_lse=True, stream=None):
    """Attention of drafted tokens over the cache: the query rows of sequence b are the nodes of a tree on top of
    tokens 0 .. start_pos[b] - 1, their own keys are tokens start_pos[b] + j (write them first).  ``tree_mask``
    [sum T, words] int64 (or uint64): bit j of a row lets it see node j of its sequence (its ancestors and itself);
    None: a chain, node t sees nodes 0 .. t.  Returns (out [sum T, H, d_v], lse [sum T, H] or None)."""
    fn = "dsa_tree_mla_fwd"
    dev = _on_one_device(fn, (("q_nope", q_nope), ("q_pe", q_pe), ("W_UK", W_UK), ("W_UV", W_UV),
                              ("tree_mask", tree_mask), ("out", out), ("lse", lse), ("workspace", workspace),
                              _table(pages)) + cache.tensors())
    N, H, d_n = q_nope.shape
    d_r, d_c, d_v = q_pe.shape[2], W_UK.shape[2], W_UV.shape[2]
    dtype = q_nope.dtype
    for name, t, shape in (("q_nope", q_nope, (seqs.total_q, H, d_n)), ("q_pe", q_pe, (N, H, d_r)),
                           ("W_UK", W_UK, (H, d_n, d_c)), ("W_UV", W_UV, (H, d_c, d_v)), ("out", out, (N, H, d_v))):
        if t is not None and (t.shape != shape or t.dtype != dtype or not t.is_contiguous()):
            raise ValueError(f"{fn}: {name} must be contiguous {shape} of {dtype}")
    if (cache.d_c, cache.d_r) != (d_c, d_r):
        raise ValueError(f"{fn}: the cache holds {cache.d_c} + {cache.d_r} values a row, expected {d_c} + {d_r}")
    words = 0
    if tree_mask is not None:
        if tree_mask.dtype not in (torch.int64, torch.uint64) or tree_mask.dim() != 2 or tree_mask.shape[0] != N or \
                not tree_mask.is_contiguous():
            raise ValueError(f"{fn}: tree_mask must be contiguous int64 or uint64 [{N}, words]")
        words = tree_mask.shape[1]
        if words == 0 and N > 0:  # its address would be NULL, which means a chain
            raise ValueError(f"{fn}: tree_mask has no words for {N} rows")
    if lse is not None and (lse.shape != (N, H) or lse.dtype != torch.float32 or not lse.is_contiguous()):
        raise ValueError(f"{fn}: lse must be contiguous fp32 [{N}, {H}]")
    if workspace is not None and (workspace.dtype != torch.uint8 or not workspace.is_contiguous()):
        raise ValueError(f"{fn}: workspace must be a contiguous uint8 tensor")
    dt = _dt(q_nope)
    lib = _abi.load()
    with _launching(dev, stream):
        on = q_nope.device
        if out is None:
            out = torch.empty((N, H, d_v), dtype=dtype, device=on)
        if lse is None and want_lse:
            lse = torch.empty((N, H), dtype=torch.float32, device=on)
        if workspace is None:
            need = lib.dsa_tree_mla_workspace_size(dt, H, d_n, d_r, d_c, d_v, seqs.ref())
            workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=on)
        _check(fn, lib.dsa_tree_mla_fwd(
            q_nope.data_ptr(), q_pe.data_ptr() if d_r else None, dt, cache.ref(), W_UK.data_ptr(), W_UV.data_ptr(), H,
            d_n, d_r, d_c, d_v, _addr(tree_mask), words, seqs.ref(), _ref_pages(fn, pages, seqs), softmax_scale,
            out.data_ptr(), _addr(lse), workspace.data_ptr(), workspace.numel(),
            torch._C._cuda_getCurrentRawStream(dev)))
    return out, lse


_NORMS = {None: _abi.DSA_NORM_NONE, "none": _abi.DSA_NORM_NONE, "rms": _abi.DSA_NORM_RMS,
          "layer": _abi.DSA_NORM_LAYER}
_ROPES = {"pairs": _abi.DSA_ROPE_PAIRS, "halves": _abi.DSA_ROPE_HALVES}


class Heads:
    """The heads of one tensor for dsa_head_norm_rope: x [sum T, n_heads, D] (fp32 or bf16, any strides but a
    contiguous last dimension), their norm ("rms", "layer", "none") with gain and bias [D] fp32 (None: 1 and 0).
    Outputs that are given: ``y`` ([sum T, n_heads, D], or the D - d_r unrotated dims beside ``y_pe``
    [sum T, n_heads, d_r]); y may be x."""

    def __init__(self, x, norm="rms", gain=None, bias=None, y=None, y_pe=None):
        if norm not in _NORMS:
            raise ValueError(f"Heads: norm must be 'rms', 'layer' or 'none', not {norm!r}")
        self.x, self.norm, self.gain, self.bias, self.y, self.y_pe = x, norm, gain, bias, y, y_pe

    def tensors(self, which):
        return ((which + ".x", self.x), (which + ".gain", self.gain), (which + ".bias", self.bias),
                (which + ".y", self.y), (which + ".y_pe", self.y_pe))


def _head_strides(fn, name, t, N, n, w, dtype):
    """Row and head stride of a tensor [N, n, w] with contiguous heads (0 where there is one row, or one head)."""
    if t.shape != (N, n, w) or t.dtype != dtype:
        raise ValueError(f"{fn}: {name} must be [{N}, {n}, {w}] of {dtype}")
    a, b, c = t.stride()
    if w > 1 and c != 1:
        raise ValueError(f"{fn}: {name} must have contiguous heads")
    return a if N > 1 else 0, b if n > 1 else 0


def dsa_head_norm_rope(q: Heads | None, k: Heads | None, rope_cos, rope_sin, seqs: Seqs, pos=None, rope="pairs",
                       rope_first=False, eps=1e-6, split=False, dtype=None, stream=None):
    """Norm every head of q and k and rotate its rotary dims (the last 2 * rope_cos.shape[1] of the D, or the first)
    to position pos[row] (int32 [sum T]; None: start_pos[b] + t) in one pass.  ``rope``: "pairs" turns (2i, 2i+1) into
    dims i and d_r/2 + i, "halves" turns (i, d_r/2 + i) in place.  Returns the pair of q's and k's results (None for a
    tensor that is None): y [sum T, heads, D], or with ``split`` (y without the rotary dims, y_pe) as the attention
    takes them."""
    fn = "dsa_head_norm_rope"
    if q is None and k is None:
        raise ValueError(f"{fn}: neither q nor k")
    if rope not in _ROPES:
        raise ValueError(f"{fn}: rope must be 'pairs' or 'halves', not {rope!r}")
    both = ([] if q is None else [q]) + ([] if k is None else [k])
    named = (("rope_cos", rope_cos), ("rope_sin", rope_sin), ("pos", pos))
    for name, h in (("q", q), ("k", k)):
        if h is not None:
            named += h.tensors(name)
    dev = _on_one_device(fn, named)
    x0 = both[0].x
    N, D, d_r = seqs.total_q, x0.shape[-1], 2 * rope_cos.shape[-1]
    for name, t in (("rope_cos", rope_cos), ("rope_sin", rope_sin)):
        if t.dtype != torch.float32 or t.dim() != 2 or t.shape != rope_cos.shape or not t.is_contiguous():
            raise ValueError(f"{fn}: {name} must be contiguous fp32 [positions, d_r / 2]")
    _int32(fn, "pos", pos, N)
    if d_r > D:
        raise ValueError(f"{fn}: {d_r} rotary dims in heads of {D}")
    split = split or any(h.y_pe is not None for h in both)
    if split and d_r == 0:
        raise ValueError(f"{fn}: no rotary dims to split off")
    y_dtype = next((h.y.dtype for h in both if h.y is not None), dtype or x0.dtype)
    width = D - d_r if split else D
    with _launching(dev, stream):
        structs, results = [], []
        for h in (q, k):
            if h is None:
                structs.append(None)
                results.append(None)
                continue
            x, y, pe = h.x, h.y, h.y_pe
            n = x.shape[1]
            for t in (h.gain, h.bias):
                if t is not None and (t.dtype != torch.float32 or t.shape != (D,) or not t.is_contiguous()):
                    raise ValueError(f"{fn}: gain and bias must be contiguous fp32 [{D}]")
            strides = _head_strides(fn, "x", x, N, n, D, x0.dtype)
            if y is None:
                y = torch.empty((N, n, width), dtype=y_dtype, device=x0.device)
                strides_y = n * width, width
            else:
                strides_y = _head_strides(fn, "y", y, N, n, width, y_dtype)
            strides_pe = 0, 0
            if split and pe is None:
                pe = torch.empty((N, n, d_r), dtype=y_dtype, device=x0.device)
                strides_pe = n * d_r, d_r
            elif split:
                strides_pe = _head_strides(fn, "y_pe", pe, N, n, d_r, y_dtype)
            st = _abi.dsa_heads(x.data_ptr(), *strides, n, _NORMS[h.norm], _addr(h.gain), _addr(h.bias), y.data_ptr(),
                                *strides_y, _addr(pe), *strides_pe)
            structs.append(ctypes.byref(st))
            results.append((y, pe) if split else y)
        _check(fn, _abi.load().dsa_head_norm_rope(
            structs[0], structs[1], _dt_of(x0.dtype), _dt_of(y_dtype), D, d_r, 1 if rope_first else 0, _ROPES[rope],
            eps, rope_cos.data_ptr(), rope_sin.data_ptr(), rope_cos.shape[0], _addr(pos), seqs.ref(),
            torch._C._cuda_getCurrentRawStream(dev)))
    return tuple(results)


def _dt_of(dtype: torch.dtype) -> int:
    if dtype == torch.float32:
        return DSA_F32
    if dtype == torch.bfloat16:
        return DSA_BF16
    raise TypeError(f"unsupported dtype {dtype}")
