"""Python binding of libentmaxkv (ctypes). Argument marshalling only.

Every step of the decode runs in the library's CUDA kernels; this module
allocates caller-owned buffers with torch, passes their device pointers and
the current CUDA stream, and turns non-zero return codes into exceptions.
There is no fallback: if the library is missing or fails to load, calls
raise.
"""

from __future__ import annotations

import contextlib
import copy
import ctypes
import os
from dataclasses import dataclass

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libentmaxkv.so")

F32, BF16, I8, E4M3 = 0, 1, 2, 3
POLICY_FULL, POLICY_TOPK, POLICY_GAUSSIAN, POLICY_SOFTMAX, POLICY_SOFTMAX_TOPK = 0, 1, 2, 3, 4
POLICIES = {"full": POLICY_FULL, "topk": POLICY_TOPK, "gaussian": POLICY_GAUSSIAN,
            "softmax": POLICY_SOFTMAX, "softmax_topk": POLICY_SOFTMAX_TOPK}
FLAG_DENSE_V, FLAG_EXACT_DELTA, FLAG_EXPIRE_WAITS = 0x1, 0x2, 0x100
DELTA_ZERO, DELTA_CERTIFIED, DELTA_MODEL, DELTA_EXACT = 0, 1, 2, 3
DEV_BAD_PAGE_TABLE, DEV_CAPACITY, DEV_TAUHAT_NOCONV = 0x1, 0x2, 0x4
DEV_CAND_OVERFLOW, DEV_TAU_NOCONV, DEV_BAD_SEQ_ID, DEV_TIMEOUT = 0x8, 0x10, 0x20, 0x40
DEV_BAD_BATCH, DEV_NONFINITE = 0x80, 0x100

# Symbols the header declares (kept in step with include/entmaxkv.h by a test).
EXPORTS = ("entmaxkv_version", "entmaxkv_status_string", "entmaxkv_append",
           "entmaxkv_workspace_bytes", "entmaxkv_decode", "entmaxkv_decode_profiled",
           "entmaxkv_workspace_layout", "entmaxkv_noalloc_scratch_bytes",
           "entmaxkv_decode_softmax_noalloc", "entmaxkv_workspace_bytes_flags",
           "entmaxkv_delta_kind", "entmaxkv_read_status", "entmaxkv_gaussian_alpha_supported",
           "entmaxkv_moment_fit_eval", "entmaxkv_plan_pages", "entmaxkv_plan_pages_bounded",
           "entmaxkv_release_pages",
           "entmaxkv_append_q8", "entmaxkv_read_q8", "entmaxkv_attend_q8_workspace",
           "entmaxkv_attend_q8")
STAGE_EVENTS = 6
STAGES = ("clear", "score", "select", "pass_a", "pass_b")


class Config(ctypes.Structure):
    _fields_ = [("num_kv_heads", ctypes.c_int32), ("group", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_seqs", ctypes.c_int32), ("max_pages_per_seq", ctypes.c_int32),
                ("num_phys_pages", ctypes.c_int32), ("kv_dtype", ctypes.c_int32)]


class CacheView(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("kmin", ctypes.c_void_p), ("kmax", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("m2", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("status", ctypes.c_void_p), ("mean_bf16", ctypes.c_void_p),
                ("m2_bf16", ctypes.c_void_p)]


class WorkspaceView(ctypes.Structure):
    _fields_ = [("bbox_u", ctypes.c_size_t), ("bbox_uhat", ctypes.c_size_t),
                ("gauss_ms", ctypes.c_size_t), ("tauhat", ctypes.c_size_t),
                ("sel_bitmap", ctypes.c_size_t), ("tauhat_iters", ctypes.c_size_t),
                ("page_zmax", ctypes.c_size_t),
                ("cap_pages", ctypes.c_int32), ("splits", ctypes.c_int32),
                ("total", ctypes.c_size_t), ("z_scores", ctypes.c_size_t)]


class Q8CacheView(ctypes.Structure):
    _fields_ = [("k_pool", ctypes.c_void_p), ("v_pool", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("status", ctypes.c_void_p)]


class RowsView(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("token_stride", ctypes.c_int64),
                ("head_stride", ctypes.c_int64)]


class BatchView(ctypes.Structure):
    _fields_ = [("seq_ids", ctypes.c_void_p), ("start", ctypes.c_void_p), ("count", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("total", ctypes.c_int32), ("max_count", ctypes.c_int32)]


class ScoreView(ctypes.Structure):
    _fields_ = [("scale", ctypes.c_float), ("softcap", ctypes.c_float), ("window", ctypes.c_int32),
                ("slopes", ctypes.c_void_p), ("prefix", ctypes.c_void_p), ("first_key", ctypes.c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libentmaxkv.so (build it with ``python -m sparse_entmax_attention_gb300.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libentmaxkv.so not built ({LIB_PATH}); run "
                          "`python -m sparse_entmax_attention_gb300.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, u32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float, ctypes.c_size_t
    L.entmaxkv_version.restype = i32
    L.entmaxkv_status_string.restype = ctypes.c_char_p
    L.entmaxkv_status_string.argtypes = [i32]
    L.entmaxkv_append.restype = i32
    L.entmaxkv_append.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(CacheView), vp, vp, vp, i32, i32, vp]
    L.entmaxkv_workspace_bytes.restype = sz
    L.entmaxkv_workspace_bytes.argtypes = [ctypes.POINTER(Config), i32, i32, i32]
    L.entmaxkv_workspace_bytes_flags.restype = sz
    L.entmaxkv_workspace_bytes_flags.argtypes = [ctypes.POINTER(Config), i32, i32, i32, ctypes.c_uint32]
    L.entmaxkv_delta_kind.restype = i32
    L.entmaxkv_delta_kind.argtypes = [i32, ctypes.c_uint32]
    L.entmaxkv_read_status.restype = i32
    L.entmaxkv_read_status.argtypes = [ctypes.POINTER(CacheView), ctypes.POINTER(ctypes.c_uint32), i32, vp]
    L.entmaxkv_gaussian_alpha_supported.restype = i32
    L.entmaxkv_gaussian_alpha_supported.argtypes = [ctypes.c_float]
    L.entmaxkv_moment_fit_eval.restype = i32
    L.entmaxkv_moment_fit_eval.argtypes = [ctypes.c_float, i32, vp, i32, vp]
    L.entmaxkv_decode.restype = i32
    L.entmaxkv_decode.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(CacheView), vp, vp, i32,
                                  f32, i32, i32, f32, u32, vp, sz, vp, vp, i32, vp, vp, vp, vp]
    L.entmaxkv_decode_profiled.restype = i32
    L.entmaxkv_decode_profiled.argtypes = L.entmaxkv_decode.argtypes + [ctypes.POINTER(ctypes.c_void_p)]
    L.entmaxkv_noalloc_scratch_bytes.restype = sz
    L.entmaxkv_noalloc_scratch_bytes.argtypes = []
    L.entmaxkv_decode_softmax_noalloc.restype = i32
    L.entmaxkv_decode_softmax_noalloc.argtypes = [ctypes.POINTER(Config), ctypes.POINTER(CacheView),
                                                  vp, vp, i32, vp, vp, vp]
    L.entmaxkv_workspace_layout.restype = i32
    L.entmaxkv_workspace_layout.argtypes = [ctypes.POINTER(Config), i32, i32, i32,
                                            ctypes.POINTER(WorkspaceView)]
    cfg_p, q8_p = ctypes.POINTER(Config), ctypes.POINTER(Q8CacheView)
    bat_p, row_p = ctypes.POINTER(BatchView), ctypes.POINTER(RowsView)
    L.entmaxkv_plan_pages.restype = i32
    L.entmaxkv_plan_pages.argtypes = [cfg_p, vp, vp, vp, vp, vp, i32, i32] + [vp] * 9
    L.entmaxkv_plan_pages_bounded.restype = i32
    L.entmaxkv_plan_pages_bounded.argtypes = [cfg_p, vp, vp, vp, vp, vp, i32, i32, i32] + [vp] * 9
    L.entmaxkv_release_pages.restype = i32
    L.entmaxkv_release_pages.argtypes = [cfg_p, vp, vp, vp, vp, i32, vp, vp, vp]
    L.entmaxkv_append_q8.restype = i32
    L.entmaxkv_append_q8.argtypes = [cfg_p, q8_p, bat_p, row_p, row_p, vp]
    L.entmaxkv_read_q8.restype = i32
    L.entmaxkv_read_q8.argtypes = [cfg_p, q8_p, bat_p, vp, row_p, row_p, vp]
    L.entmaxkv_attend_q8_workspace.restype = sz
    L.entmaxkv_attend_q8_workspace.argtypes = [cfg_p, i32, i32, i32, f32]
    L.entmaxkv_attend_q8.restype = i32
    L.entmaxkv_attend_q8.argtypes = [cfg_p, q8_p, bat_p, row_p, ctypes.POINTER(ScoreView), f32, vp, sz,
                                     row_p, vp, vp]
    _lib = L
    return L


class EntmaxKVError(RuntimeError):
    pass


def _check(code: int):
    if code != 0:
        raise EntmaxKVError(f"entmaxkv: {lib().entmaxkv_status_string(code).decode()} (code {code})")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _allocating(stream):
    """Where a call given `stream` makes its tensors: on that stream, so that their first fill, the
    call's launches and the reuse of what the call drops come one behind the other."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _for_caller(stream, *tensors):
    """Tensors made on `stream` and returned are kept until the caller's current stream is done with
    them too (it waits for `stream` before it reads them)."""
    if stream is not None:
        for t in tensors:
            t.record_stream(torch.cuda.current_stream(t.device))


_DT = {torch.float32: F32, torch.bfloat16: BF16}


class PagedCache:
    """Caller-owned paged KV cache plus per-page key metadata (torch memory).

    meta_bf16: also keep bf16 copies of the page means and m2, which the
    Gaussian scorer then streams instead of the fp32 arrays.
    """

    def __init__(self, num_kv_heads, group, head_dim, page_size, max_seqs, max_pages_per_seq,
                 num_phys_pages, kv_dtype=torch.bfloat16, device="cuda", meta_bf16=False):
        self.cfg = Config(num_kv_heads, group, head_dim, page_size, max_seqs,
                          max_pages_per_seq, num_phys_pages, _DT[kv_dtype])
        self.dtype, self.device = kv_dtype, torch.device(device)
        Hkv, d, P = num_kv_heads, head_dim, page_size
        self.k_pool = torch.zeros(num_phys_pages, Hkv, P, d, dtype=kv_dtype, device=device)
        self.v_pool = torch.zeros_like(self.k_pool)
        self.kmin = torch.zeros(num_phys_pages, Hkv, d, dtype=kv_dtype, device=device)
        self.kmax = torch.zeros_like(self.kmin)
        self.mean = torch.zeros(num_phys_pages, Hkv, d, dtype=torch.float32, device=device)
        self.m2 = torch.zeros_like(self.mean)
        self.block_table = torch.zeros(max_seqs, max_pages_per_seq, dtype=torch.int32, device=device)
        self.seq_lens = torch.zeros(max_seqs, dtype=torch.int32, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)
        self.mean_bf16 = self.m2_bf16 = None
        if meta_bf16:
            self.mean_bf16 = torch.zeros(num_phys_pages, Hkv, d, dtype=torch.bfloat16, device=device)
            self.m2_bf16 = torch.zeros_like(self.mean_bf16)
        self.view = CacheView(self.k_pool.data_ptr(), self.v_pool.data_ptr(), self.kmin.data_ptr(),
                              self.kmax.data_ptr(), self.mean.data_ptr(), self.m2.data_ptr(),
                              self.block_table.data_ptr(), self.seq_lens.data_ptr(),
                              self.status.data_ptr(),
                              self.mean_bf16.data_ptr() if meta_bf16 else None,
                              self.m2_bf16.data_ptr() if meta_bf16 else None)

    def fp32_metadata(self) -> "PagedCache":
        """The same cache seen without its bf16 metadata copies (the Gaussian
        scorer then streams the fp32 mean and m2); tensors are shared."""
        other = copy.copy(self)
        other.view = CacheView(*[getattr(self.view, f) for f, _ in CacheView._fields_])
        other.view.mean_bf16 = None
        other.view.m2_bf16 = None
        other.mean_bf16 = None  # (this view streams none; self keeps the tensors alive)
        other.m2_bf16 = None
        return other

    @property
    def num_q_heads(self):
        return self.cfg.num_kv_heads * self.cfg.group

    def device_status(self) -> int:
        return int(self.status.item()) & 0xffffffff

    def read_status(self, clear=False, stream=None) -> int:
        """entmaxkv_read_status: the ENTMAXKV_DEV_* bits after the stream's work."""
        out = ctypes.c_uint32(0)
        _check(lib().entmaxkv_read_status(ctypes.byref(self.view), ctypes.byref(out), int(bool(clear)),
                                          _stream(stream)))
        return int(out.value)


def append(cache: PagedCache, k, v, seq_ids=None, stream=None):
    """entmaxkv_append: k, v [n_seqs, Hkv, n_tokens, d] in the cache dtype."""
    assert k.is_contiguous() and v.is_contiguous() and k.dtype == cache.dtype
    n_seqs, _, n_tok, _ = k.shape
    _check(lib().entmaxkv_append(ctypes.byref(cache.cfg), ctypes.byref(cache.view), _ptr(k),
                                 _ptr(v), _ptr(seq_ids), n_seqs, n_tok, _stream(stream)))


def workspace_bytes(cache: PagedCache, n_seqs, policy, budget_tokens=0, flags=0) -> int:
    return int(lib().entmaxkv_workspace_bytes_flags(ctypes.byref(cache.cfg), n_seqs,
                                                    POLICIES.get(policy, policy), budget_tokens,
                                                    int(flags)))


def delta_kind(policy, flags=0) -> int:
    return int(lib().entmaxkv_delta_kind(POLICIES.get(policy, policy), int(flags)))


def workspace_layout(cache: PagedCache, n_seqs, policy, budget_tokens=0) -> WorkspaceView:
    v = WorkspaceView()
    _check(lib().entmaxkv_workspace_layout(ctypes.byref(cache.cfg), n_seqs,
                                           POLICIES.get(policy, policy), budget_tokens,
                                           ctypes.byref(v)))
    return v


def alloc_workspace(cache: PagedCache, n_seqs, policy, budget_tokens=0, flags=0):
    n = workspace_bytes(cache, n_seqs, policy, budget_tokens, flags)
    if n == 0:
        raise EntmaxKVError("invalid decode arguments for workspace sizing")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)  # caching allocator: 256-B aligned


@dataclass
class DecodeOutputs:
    out: torch.Tensor
    page_ids: torch.Tensor
    n_sel: torch.Tensor
    tau: torch.Tensor
    delta: torch.Tensor


def page_capacity(cache: PagedCache, policy, budget_tokens) -> int:
    p = POLICIES.get(policy, policy)
    maxp, P = cache.cfg.max_pages_per_seq, cache.cfg.page_size
    if p in (POLICY_TOPK, POLICY_SOFTMAX_TOPK):
        return min(budget_tokens // P, maxp)
    if p == POLICY_GAUSSIAN and budget_tokens > 0:
        return min(budget_tokens // P, maxp)
    return maxp


def alloc_outputs(cache: PagedCache, n_seqs, policy, budget_tokens=0) -> DecodeOutputs:
    dev, Hq, Hkv = cache.device, cache.num_q_heads, cache.cfg.num_kv_heads
    cap = page_capacity(cache, policy, budget_tokens)
    return DecodeOutputs(
        out=torch.empty(n_seqs, Hq, cache.cfg.head_dim, dtype=torch.float32, device=dev),
        page_ids=torch.full((n_seqs, Hkv, cap), -1, dtype=torch.int32, device=dev),
        n_sel=torch.empty(n_seqs, Hkv, dtype=torch.int32, device=dev),
        tau=torch.empty(n_seqs, Hq, dtype=torch.float32, device=dev),
        delta=torch.empty(n_seqs, Hq, dtype=torch.float32, device=dev))


def decode(cache: PagedCache, q, alpha=1.5, policy="gaussian", budget_tokens=0, margin=0.0,
           flags=0, seq_ids=None, workspace=None, outputs: DecodeOutputs | None = None,
           stream=None, events=None) -> DecodeOutputs:
    """entmaxkv_decode: q [n_seqs, Hq, d] in the cache dtype.

    With ``events`` (STAGE_EVENTS torch.cuda.Event objects) this calls
    entmaxkv_decode_profiled, which records them between the stages. A workspace and
    outputs that are not given are allocated on ``stream``.
    """
    assert q.is_contiguous() and q.dtype == cache.dtype
    n_seqs = q.shape[0]
    pol = POLICIES.get(policy, policy)
    made = outputs is None
    if made or workspace is None:
        with _allocating(stream):
            if workspace is None:
                workspace = alloc_workspace(cache, n_seqs, pol, budget_tokens, flags)
            if made:
                outputs = alloc_outputs(cache, n_seqs, pol, budget_tokens)
    o = outputs
    if made:
        _for_caller(stream, o.out, o.page_ids, o.n_sel, o.tau, o.delta)
    args = [ctypes.byref(cache.cfg), ctypes.byref(cache.view), _ptr(q), _ptr(seq_ids), n_seqs,
            float(alpha), pol, int(budget_tokens), float(margin), int(flags), _ptr(workspace),
            workspace.numel(), _ptr(o.out), _ptr(o.page_ids), o.page_ids.shape[-1], _ptr(o.n_sel),
            _ptr(o.tau), _ptr(o.delta), _stream(stream)]
    if events is None:
        _check(lib().entmaxkv_decode(*args))
    else:
        assert len(events) == STAGE_EVENTS
        arr = (ctypes.c_void_p * STAGE_EVENTS)(*[ctypes.c_void_p(e.cuda_event) for e in events])
        _check(lib().entmaxkv_decode_profiled(*args, arr))
    return o


class DecodeStep:
    """One serving step, append one token per sequence and decode, captured
    once as CUDA graphs of the library's launches over fixed buffers.

    `run(k, v, q)` takes device tensors: it copies them into the step's
    buffers and replays the launches. `run_host(k, v, q)` takes host tensors:
    they are copied into one pinned staging buffer, and a second graph moves
    them to the device in one copy, runs the launches and returns out, τ, δ
    and n_sel to pinned host memory in one copy; it returns those host views
    once the step is done. Capturing launches nothing: the cache changes only
    on replay. Arguments as for `append` and `decode`; k and v are
    [n_seqs, Hkv, 1, d], q is [n_seqs, Hq, d]."""

    def __init__(self, cache: PagedCache, n_seqs, alpha=1.5, policy="gaussian", budget_tokens=0,
                 margin=0.0, flags=0, seq_ids=None):
        dev, d = cache.device, cache.cfg.head_dim
        self.cache = cache
        Hkv, Hq = cache.cfg.num_kv_heads, cache.num_q_heads
        el = torch.tensor([], dtype=cache.dtype).element_size()
        shapes_in = [(n_seqs, Hkv, 1, d), (n_seqs, Hkv, 1, d), (n_seqs, Hq, d)]
        n_in = [int(torch.Size(sh).numel()) * el for sh in shapes_in]
        self.dev_in = torch.zeros(sum(n_in), dtype=torch.uint8, device=dev)
        self.host_in = torch.zeros(sum(n_in), dtype=torch.uint8).pin_memory()

        def views(buf):
            out, off = [], 0
            for sh, n in zip(shapes_in, n_in):
                out.append(buf[off:off + n].view(cache.dtype).view(sh))
                off += n
            return out

        self.k, self.v, self.q = views(self.dev_in)
        self._hk, self._hv, self._hq = views(self.host_in)
        # outputs: out, τ, δ, n_sel packed in one buffer (one copy back); page ids apart
        cap = page_capacity(cache, policy, budget_tokens)
        shapes_out = [((n_seqs, Hq, d), torch.float32), ((n_seqs, Hq), torch.float32),
                      ((n_seqs, Hq), torch.float32), ((n_seqs, Hkv), torch.int32)]
        n_out = [int(torch.Size(sh).numel()) * 4 for sh, _ in shapes_out]
        self.dev_out = torch.zeros(sum(n_out), dtype=torch.uint8, device=dev)
        self.host_out = torch.zeros(sum(n_out), dtype=torch.uint8).pin_memory()

        def out_views(buf):
            res, off = [], 0
            for (sh, dt), n in zip(shapes_out, n_out):
                res.append(buf[off:off + n].view(dt).view(sh))
                off += n
            return res

        out, tau, delta, n_sel = out_views(self.dev_out)
        self.outputs = DecodeOutputs(out=out, tau=tau, delta=delta, n_sel=n_sel,
                                     page_ids=torch.full((n_seqs, Hkv, cap), -1, dtype=torch.int32, device=dev))
        self.host_outputs = out_views(self.host_out)
        self.workspace = alloc_workspace(cache, n_seqs, policy, budget_tokens, flags)
        args = (alpha, policy, budget_tokens, margin, flags)

        def launches():
            append(cache, self.k, self.v, seq_ids=seq_ids)
            decode(cache, self.q, *args, seq_ids=seq_ids, workspace=self.workspace, outputs=self.outputs)

        # one decode outside the captures: first-launch set-up (shared-memory
        # attributes, moment fits) happens here, and no token is appended
        decode(cache, self.q, *args, seq_ids=seq_ids, workspace=self.workspace, outputs=self.outputs)
        torch.cuda.synchronize(dev)
        self.graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph):
            launches()
        self.graph_io = torch.cuda.CUDAGraph()
        with torch.cuda.graph(self.graph_io):
            self.dev_in.copy_(self.host_in, non_blocking=True)
            launches()
            self.host_out.copy_(self.dev_out, non_blocking=True)

    def run(self, k, v, q) -> DecodeOutputs:
        """Device tensors in; the outputs stay on the device."""
        self.k.copy_(k, non_blocking=True)
        self.v.copy_(v, non_blocking=True)
        self.q.copy_(q, non_blocking=True)
        self.graph.replay()
        return self.outputs

    def run_host(self, k, v, q, wait=True):
        """Host tensors in; returns (out, τ, δ, n_sel) as pinned host tensors.
        With wait=True the call returns once the step has finished; with
        wait=False the caller synchronises the current stream before reading
        them (and before the next call reuses the staging buffer)."""
        self._hk.copy_(k)
        self._hv.copy_(v)
        self._hq.copy_(q)
        self.graph_io.replay()
        if wait:
            torch.cuda.current_stream(self.cache.device).synchronize()
        return self.host_outputs


def stage_events():
    """STAGE_EVENTS timing events with their CUDA handles already created."""
    evs = [torch.cuda.Event(enable_timing=True) for _ in range(STAGE_EVENTS)]
    for e in evs:
        e.record()
    torch.cuda.synchronize()
    return evs


def gaussian_alpha_supported(alpha: float) -> bool:
    """entmaxkv_gaussian_alpha_supported (host only)."""
    return bool(lib().entmaxkv_gaussian_alpha_supported(float(alpha)))


def moment_fit_eval(alpha: float, order: int, t):
    """entmaxkv_moment_fit_eval: the fitted J_ν(t), ν = β − order, on the host
    in the kernels' float arithmetic. t: 1-d float32 array-like."""
    import numpy as np
    ta = np.ascontiguousarray(np.asarray(t, dtype=np.float32))
    out = np.empty_like(ta)
    _check(lib().entmaxkv_moment_fit_eval(float(alpha), int(order), ta.ctypes.data_as(ctypes.c_void_p),
                                          int(ta.size), out.ctypes.data_as(ctypes.c_void_p)))
    return out


# ---------------------------------------------------------------------------
# The 8-bit paged cache: plan, append, attend.

_CODES = {torch.int8: I8, torch.float8_e4m3fn: E4M3}
_I32, _F32, _BF16 = torch.int32, torch.float32, torch.bfloat16


def _need(ok, what):
    if not ok:
        raise EntmaxKVError(what)


def _i32(t, shape, dev, name):
    """The pointer of a contiguous int32 tensor of this shape on device number `dev`."""
    if t.dtype is not _I32 or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise EntmaxKVError(f"{name}: a contiguous int32 tensor of shape {tuple(shape)} on device {dev} is wanted")
    return t.data_ptr()


def _q8_call(dev, stream, fn, *args):
    """fn(*args, stream) on the tensors' device, whichever device is current."""
    if stream is not None and stream.device_index != dev:
        raise EntmaxKVError("stream: on another device than the tensors")
    if torch._C._cuda_getDevice() == dev:
        code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(dev):
            code = fn(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    if code:
        _check(code)


def _rows(t, shape, dev, name):
    """entmaxkv_rows of a [tokens, heads, d] bf16 tensor (its first two strides are free)."""
    if t.dtype is not _BF16 or t.shape != shape or t.get_device() != dev:
        raise EntmaxKVError(f"{name}: a bfloat16 tensor of shape {shape} on device {dev} is wanted")
    ts, hs, es = t.stride()
    if es != 1:
        raise EntmaxKVError(f"{name}: the head dimension must be contiguous")
    if shape[0] == 1:
        ts = max(8, shape[1] * shape[2])
    if shape[1] == 1:
        hs = max(8, shape[2])
    return RowsView(t.data_ptr(), ts, hs)


class PageTable:
    """A block table and lengths alone, for planning pages of caches kept elsewhere."""

    def __init__(self, block_table, seq_lens, page_size, num_phys_pages, status=None):
        self.device, self._dev = block_table.device, block_table.get_device()
        max_seqs, max_pages = block_table.shape
        _i32(block_table, (max_seqs, max_pages), self._dev, "block_table")
        _i32(seq_lens, (max_seqs,), self._dev, "seq_lens")
        self.cfg = Config(1, 1, 64, page_size, max_seqs, max_pages, num_phys_pages, I8)
        self.block_table, self.seq_lens = block_table, seq_lens
        self.status = status if status is not None else torch.zeros(1, dtype=torch.int32, device=self.device)

    def device_status(self) -> int:
        return int(self.status.item()) & 0xffffffff


class PagePool:
    """A stack of free physical pages on the device: free_pages[0 .. free_count - 1].
    PagePool.full(n, device) starts with all n pages, page 0 handed out first."""

    def __init__(self, free_pages, free_count):
        self.free_pages, self.free_count = free_pages, free_count
        self._dev, self._n = free_pages.get_device(), free_pages.numel()
        self._pages = _i32(free_pages, (self._n,), self._dev, "free_pages")
        self._count = _i32(free_count, (1,), self._dev, "free_count")

    @classmethod
    def full(cls, num_phys_pages, device="cuda"):
        return cls(torch.arange(num_phys_pages - 1, -1, -1, dtype=torch.int32, device=device),
                   torch.full((1,), num_phys_pages, dtype=torch.int32, device=device))


class Batch:
    """Rows of a ragged batch (entmaxkv_batch): slot b owns rows start[b] .. start[b] + count[b] - 1
    of `total`, the last count[b] tokens of sequence seq_ids[b] (b without seq_ids)."""

    def __init__(self, start, count, total, max_count, seq_ids=None):
        self._n, self._dev = start.shape[0], start.get_device()
        shape = (self._n,)
        self.start, self.count, self.seq_ids = start, count, seq_ids
        self.total, self.max_count, self.device = int(total), int(max_count), start.device
        self.view = BatchView(None if seq_ids is None else _i32(seq_ids, shape, self._dev, "seq_ids"),
                              _i32(start, shape, self._dev, "start"), _i32(count, shape, self._dev, "count"),
                              self._n, self.total, self.max_count)

    @classmethod
    def uniform(cls, n_seqs, count=1, seq_ids=None, device="cuda"):
        """count rows of every sequence, one sequence behind the other."""
        start = torch.arange(n_seqs, dtype=torch.int32, device=device) * count
        return cls(start, torch.full_like(start, count), n_seqs * count, count, seq_ids)


class PagePlan:
    """What plan_pages writes: the batch's rows (start, count [n_seqs]), positions and slots [total]
    of its tokens (int32, int64)."""

    def __init__(self, start, count, positions, slots):
        self.start, self.count, self.positions, self.slots = start, count, positions, slots
        self._n, self._total, self._dev = start.shape[0], positions.shape[0], start.get_device()
        _need(slots.dtype == torch.int64 and slots.shape == positions.shape and slots.is_contiguous()
              and slots.get_device() == self._dev, "slots: a contiguous int64 tensor beside positions is wanted")
        self._ptrs = (_i32(start, (self._n,), self._dev, "start"), _i32(count, (self._n,), self._dev, "count"),
                      _i32(positions, (self._total,), self._dev, "positions"), slots.data_ptr())

    def batch(self, max_count, seq_ids=None) -> Batch:
        return Batch(self.start, self.count, self._total, max_count, seq_ids)


def alloc_plan(n_seqs, total, device="cuda") -> PagePlan:
    i32 = dict(dtype=torch.int32, device=device)
    return PagePlan(torch.zeros(n_seqs, **i32), torch.zeros(n_seqs, **i32), torch.full((total,), -1, **i32),
                    torch.full((total,), -1, dtype=torch.int64, device=device))


def plan_pages(cache, pool: PagePool, n_new, plan: PagePlan, seq_ids=None, advance=True, lens_out=None,
               count_out=None, stream=None, max_count=0) -> PagePlan:
    """entmaxkv_plan_pages_bounded: pages, positions and slots for n_new[b] more tokens of each sequence.

    max_count: the bound of the batch that comes next (append_q8, attend_q8); a slot with more new
    tokens is refused here, as it would be there. 0: none.
    cache: a QuantCache, a PagedCache or a PageTable. With advance the lengths count the new
    tokens in (into lens_out when given, else in place); a PagedCache, whose append counts them
    itself, is planned with advance=False. The free list's new height goes to count_out, or in place.
    """
    n, dev, cfg = plan._n, plan._dev, cache.cfg
    table, lens = cache.block_table, cache.seq_lens
    if table.get_device() != dev or pool._dev != dev:
        raise EntmaxKVError("cache, pool and plan: on one device are wanted")
    if pool._n < cfg.num_phys_pages:
        raise EntmaxKVError("pool: a free list of num_phys_pages entries is wanted")
    start, count, positions, slots = plan._ptrs
    lens_p = lens.data_ptr()
    if not advance:
        to = None
    elif lens_out is None:
        to = lens_p
    else:
        to = _i32(lens_out, lens.shape, dev, "lens_out")
    _q8_call(dev, stream, lib().entmaxkv_plan_pages_bounded, cfg, table.data_ptr(), lens_p, cache.status.data_ptr(),
             None if seq_ids is None else _i32(seq_ids, (n,), dev, "seq_ids"), _i32(n_new, (n,), dev, "n_new"), n,
             plan._total, int(max_count), pool._pages, pool._count,
             pool._count if count_out is None else _i32(count_out, (1,), dev, "count_out"), to, start, count,
             positions, slots)
    return plan


def release_pages(cache, pool: PagePool, seq_ids, stream=None):
    """entmaxkv_release_pages: the sequences' pages go back to the pool, their lengths become 0."""
    dev, n = pool._dev, seq_ids.shape[0]
    _need(cache.block_table.get_device() == dev, "cache and pool: on one device are wanted")
    _need(pool._n >= cache.cfg.num_phys_pages, "pool: a free list of num_phys_pages entries is wanted")
    _q8_call(dev, stream, lib().entmaxkv_release_pages, cache.cfg, cache.block_table.data_ptr(),
             cache.seq_lens.data_ptr(), cache.status.data_ptr(), _i32(seq_ids, (n,), dev, "seq_ids"), n,
             pool._pages, pool._count)


class QuantCache:
    """Caller-owned paged KV cache in 8 bits (torch memory): codes in int8 or float8_e4m3fn and a
    float32 scale for the K and one for the V rows of each (physical page, KV head). seq_lens
    counts the tokens of the step under way (plan_pages advances it)."""

    def __init__(self, num_kv_heads, group, head_dim, page_size, max_seqs, max_pages_per_seq, num_phys_pages,
                 code_dtype=torch.int8, device="cuda"):
        shape = (num_phys_pages, num_kv_heads, page_size, head_dim)
        pools = [torch.zeros(shape, dtype=torch.int8, device=device).view(code_dtype) for _ in range(2)]
        scales = [torch.zeros(shape[:2], dtype=torch.float32, device=device) for _ in range(2)]
        self._init(*pools, *scales, torch.zeros(max_seqs, max_pages_per_seq, dtype=torch.int32, device=device),
                   torch.zeros(max_seqs, dtype=torch.int32, device=device), group, None)

    @classmethod
    def of(cls, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, group, status=None):
        """The cache over tensors the caller already has (scales of pages in use are positive)."""
        c = cls.__new__(cls)
        c._init(k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, group, status)
        return c

    def _init(self, k_pool, v_pool, k_scale, v_scale, block_table, seq_lens, group, status):
        dev, shape = k_pool.get_device(), k_pool.shape
        _need(k_pool.dtype in _CODES, "k_pool: int8 or float8_e4m3fn codes are wanted")
        _need(v_pool.dtype == k_pool.dtype and v_pool.shape == shape and len(shape) == 4
              and v_pool.get_device() == dev and k_pool.is_contiguous() and v_pool.is_contiguous(),
              "k_pool, v_pool: contiguous [pages, KV heads, page size, head dim] of one type are wanted")
        for t in (k_scale, v_scale):
            _need(t.dtype is _F32 and t.shape == shape[:2] and t.is_contiguous() and t.get_device() == dev,
                  "k_scale, v_scale: contiguous float32 [pages, KV heads] are wanted")
        max_seqs, max_pages = block_table.shape
        _i32(block_table, (max_seqs, max_pages), dev, "block_table")
        _i32(seq_lens, (max_seqs,), dev, "seq_lens")
        self.device, self._dev, self.code_dtype = k_pool.device, dev, k_pool.dtype
        self.k_pool, self.v_pool, self.k_scale, self.v_scale = k_pool, v_pool, k_scale, v_scale
        self.block_table, self.seq_lens = block_table, seq_lens
        self.status = status if status is not None else torch.zeros(1, dtype=torch.int32, device=self.device)
        self.cfg = Config(shape[1], group, shape[3], shape[2], max_seqs, max_pages, shape[0], _CODES[k_pool.dtype])
        self.num_q_heads = shape[1] * group
        self.view = Q8CacheView(k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                block_table.data_ptr(), seq_lens.data_ptr(), self.status.data_ptr())

    def device_status(self) -> int:
        return int(self.status.item()) & 0xffffffff


def _on_cache(cache, batch):
    if batch._dev != cache._dev:
        raise EntmaxKVError("batch: on another device than the cache")
    return cache._dev


def append_q8(cache: QuantCache, k, v, batch: Batch, stream=None):
    """entmaxkv_append_q8: k, v [total, Hkv, d] bf16 (any token and head strides that are multiples
    of 8): the last count[b] tokens of each sequence become codes."""
    dev, shape = _on_cache(cache, batch), (batch.total, cache.cfg.num_kv_heads, cache.cfg.head_dim)
    _q8_call(dev, stream, lib().entmaxkv_append_q8, cache.cfg, cache.view, batch.view, _rows(k, shape, dev, "k"),
             _rows(v, shape, dev, "v"))


def read_q8(cache: QuantCache, first, batch: Batch, k=None, v=None, stream=None):
    """entmaxkv_read_q8: tokens first[b] .. first[b] + count[b] - 1 of each sequence as bf16 rows
    [total, Hkv, d] in k and v (allocated on the call's stream when not given). Returns (k, v)."""
    dev, shape = _on_cache(cache, batch), (batch.total, cache.cfg.num_kv_heads, cache.cfg.head_dim)
    if k is None or v is None:
        with _allocating(stream):
            made = [torch.empty(shape, dtype=torch.bfloat16, device=cache.device) for t in (k, v) if t is None]
        _for_caller(stream, *made)
        v = made.pop() if v is None else v
        k = made.pop() if k is None else k
    _q8_call(dev, stream, lib().entmaxkv_read_q8, cache.cfg, cache.view, batch.view,
             _i32(first, (batch._n,), dev, "first"), _rows(k, shape, dev, "k"), _rows(v, shape, dev, "v"))
    return k, v


class AttendOutputs:
    """out [total, Hq, d] bf16 and tau [total, Hq] float32 (log-sum-exp of a softmax, the entmax
    threshold), or tau None."""

    def __init__(self, out, tau):
        self.out, self.tau = out, tau


def alloc_attend_outputs(cache: QuantCache, batch: Batch) -> AttendOutputs:
    Hq = cache.num_q_heads
    return AttendOutputs(torch.zeros(batch.total, Hq, cache.cfg.head_dim, dtype=torch.bfloat16, device=cache.device),
                         torch.zeros(batch.total, Hq, dtype=torch.float32, device=cache.device))


def attend_workspace_bytes(cache: QuantCache, batch: Batch, alpha=1.0) -> int:
    b = batch.view
    return int(lib().entmaxkv_attend_q8_workspace(cache.cfg, b.n_seqs, b.total, b.max_count, float(alpha)))


def alloc_attend_workspace(cache: QuantCache, batch: Batch, alpha=1.0):
    n = attend_workspace_bytes(cache, batch, alpha)
    if n == 0:
        raise EntmaxKVError("invalid attention arguments for workspace sizing")
    return torch.empty(n, dtype=torch.uint8, device=cache.device)  # caching allocator: 256-B aligned


def attend_q8(cache: QuantCache, q, batch: Batch, alpha=1.0, scale=0.0, softcap=0.0, slopes=None, window=0,
              prefix=None, first_key=None, workspace=None, outputs: AttendOutputs | None = None,
              stream=None) -> AttendOutputs:
    """entmaxkv_attend_q8: q [total, Hq, d] bf16 against each row's sequence. alpha = 1 is softmax;
    alpha > 1 is alpha-entmax, for one new token a sequence.

    softcap: s becomes softcap * tanh(s / softcap). slopes: float32 [Hq], slopes[h] * distance is
    taken off. window: keys seen back from the row's own. prefix: int32 [n_seqs], keys in front
    that every row sees. first_key: int32 [total], where each row's document begins.
    A workspace and outputs that are not given are allocated on the call's stream.
    """
    dev, Hq = _on_cache(cache, batch), cache.num_q_heads
    shape = (batch.total, Hq, cache.cfg.head_dim)
    if workspace is not None and workspace.get_device() != dev:
        raise EntmaxKVError("workspace: on another device than the cache")
    made = outputs is None
    if made or workspace is None:
        with _allocating(stream):
            if made:
                outputs = alloc_attend_outputs(cache, batch)
            if workspace is None:
                workspace = alloc_attend_workspace(cache, batch, alpha)
        if made:
            _for_caller(stream, outputs.out, outputs.tau)
    score = ScoreView(scale, softcap, window, None, None, None)
    if slopes is not None:
        if slopes.dtype is not _F32 or slopes.shape != (Hq,) or not slopes.is_contiguous() or slopes.get_device() != dev:
            raise EntmaxKVError("slopes: contiguous float32 [Hq] is wanted")
        score.slopes = slopes.data_ptr()
    if prefix is not None:
        score.prefix = _i32(prefix, (batch._n,), dev, "prefix")
    if first_key is not None:
        score.first_key = _i32(first_key, (batch.total,), dev, "first_key")
    t = outputs.tau
    if t is not None and (t.dtype is not _F32 or t.shape != shape[:2] or not t.is_contiguous() or t.get_device() != dev):
        raise EntmaxKVError("tau: contiguous float32 [total, Hq] is wanted")
    _q8_call(dev, stream, lib().entmaxkv_attend_q8, cache.cfg, cache.view, batch.view, _rows(q, shape, dev, "q"),
             score, alpha, workspace.data_ptr(), workspace.nbytes, _rows(outputs.out, shape, dev, "out"),
             None if t is None else t.data_ptr())
    return outputs


class QuantStep:
    """One serving step over an 8-bit cache for n_seqs slots of up to max_count new tokens each:
    plan pages, append, attend, captured once as a CUDA graph of the library's launches over fixed
    buffers. Arguments as for attend_q8; prefix and first_key are fixed buffers too.

    run(n_new, seq_ids, q, k, v): n_new and seq_ids int32 [n_seqs] (a slot with n_new 0 is idle),
    q, k, v the new tokens' rows one slot behind the other, in the first sum(n_new) rows of at most
    n_seqs * max_count. Rows past the last token, and those of refused slots, are left as they were.
    A slot with more than max_count tokens is refused (DEV_BAD_BATCH): its sequence, pages and the pool
    stay as they were.
    Capturing launches nothing: the cache changes only on replay."""

    def __init__(self, cache: QuantCache, pool: PagePool, n_seqs, max_count=1, alpha=1.0, **score):
        dev, c = cache.device, cache.cfg
        total, Hq = n_seqs * max_count, cache.num_q_heads
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.cache, self.pool = cache, pool
        self.n_new = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.seq_ids = torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.q = torch.zeros(total, Hq, c.head_dim, **bf)
        self.k = torch.zeros(total, c.num_kv_heads, c.head_dim, **bf)
        self.v = torch.zeros_like(self.k)
        self.plan = alloc_plan(n_seqs, total, dev)
        self.batch = self.plan.batch(max_count, self.seq_ids)
        self.outputs = alloc_attend_outputs(cache, self.batch)
        self.workspace = alloc_attend_workspace(cache, self.batch, alpha)
        self._score = dict(score, alpha=alpha)

        def launches():
            plan_pages(cache, pool, self.n_new, self.plan, seq_ids=self.seq_ids, max_count=max_count)
            append_q8(cache, self.k, self.v, self.batch)
            attend_q8(cache, self.q, self.batch, workspace=self.workspace, outputs=self.outputs, **self._score)

        with torch.cuda.device(dev):
            launches()  # every slot idle: first-launch set-up outside the capture
            torch.cuda.synchronize(dev)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                launches()

    def run(self, n_new, seq_ids, q, k, v) -> AttendOutputs:
        """Device tensors in; the outputs (and plan) stay on the device."""
        rows = q.shape[0]
        _need(rows <= self.q.shape[0], "more rows than the step was made for")
        for t, own, name in ((q, self.q, "q"), (k, self.k, "k"), (v, self.v, "v")):
            _need(t.shape == (rows, *own.shape[1:]), f"{name}: rows of shape {(rows, *own.shape[1:])} are wanted")
        for t, name in ((n_new, "n_new"), (seq_ids, "seq_ids")):
            _need(t.shape == self.n_new.shape, f"{name}: a tensor of shape {tuple(self.n_new.shape)} is wanted")
        self.n_new.copy_(n_new, non_blocking=True)
        self.seq_ids.copy_(seq_ids, non_blocking=True)
        self.q[:rows].copy_(q, non_blocking=True)
        self.k[:rows].copy_(k, non_blocking=True)
        self.v[:rows].copy_(v, non_blocking=True)
        self.graph.replay()
        return self.outputs
