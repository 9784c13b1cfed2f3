"""prefix_tree_block_gb300 -- prefix-tree attention (forward and backward) for
one NVIDIA GB300, as a C-ABI library (libpt.so, declared in include/pt.h)
with this thin Python binding.

The binding only marshals arguments: it passes raw device pointers and the
current CUDA stream to the library and allocates outputs with PyTorch.  Every
step of the computation runs in the library's CUDA kernels; if libpt.so is
missing the calls raise, there is no other implementation behind them.
Build the library with ``prefix_tree_block_gb300.build.build()``.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional, Tuple

__all__ = [
    "PTError", "BlockMap", "HostStep", "load_library", "build_blockmap_tree", "build_blockmap_seg",
    "build_blockmap_draft",
    "attn_fwd", "attn_bwd", "bwd_workspace_bytes", "sync_status", "launch_count", "LIB_PATH",
    "profile_enable", "profile_read", "profile_reset", "attn_bwd_noalloc", "FoldPlan", "fold_plan",
    "cache_tables", "cache_write", "DecodePlan", "decode_plan", "attn_decode", "draft_tree", "cache_keep", "rotary",
    "token_logprobs", "token_logprobs_bwd",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpt.so")

PT_OK, PT_ERR_INVALID_ARG, PT_ERR_UNSUPPORTED, PT_ERR_CUDA, PT_ERR_TIMEOUT, PT_ERR_NOMEM = range(6)
PT_BF16, PT_F32 = 0, 1
_STATUS_NAMES = {0: "PT_OK", 1: "PT_ERR_INVALID_ARG", 2: "PT_ERR_UNSUPPORTED", 3: "PT_ERR_CUDA",
                 4: "PT_ERR_TIMEOUT", 5: "PT_ERR_NOMEM"}

_lib = None
_lock = threading.Lock()
_alloc_hook = None


def set_output_allocator(fn=None):
    """Route the binding's device output allocations (O, LSE, gradients,
    workspaces, fold outputs) through fn(shape, dtype, device) -> tensor, or
    back to torch.empty with None.  Tests use it to surround every output
    with guard bands."""
    global _alloc_hook
    _alloc_hook = fn


def _empty(shape, dtype, device):
    import torch

    if _alloc_hook is not None:
        return _alloc_hook(tuple(shape), dtype, device)
    return torch.empty(tuple(shape), dtype=dtype, device=device)


class PTError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


def load_library(path: Optional[str] = None):
    """Load libpt.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with prefix_tree_block_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, i32, i64, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        pp = ctypes.POINTER(ctypes.c_void_p)
        i32p, i64p = ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int64)
        sig = {
            "pt_build_blockmap_tree": [vp, i32, vp, vp, i32, i32, i32, vp, pp],
            "pt_build_blockmap_seg": [vp, vp, i32, i32, i32, vp, pp],
            "pt_blockmap_dense": [vp, vp, pp],
            "pt_build_blockmap_draft": [i32, i32, i32, vp, vp, i32, i32, vp, vp, i32, i32, vp, pp],
            "pt_blockmap_info": [vp, i32p, i32p, i32p, i32p, i32p, i64p, i64p],
            "pt_blockmap_export": [vp, vp, vp, vp, vp, vp, vp],
            "pt_blockmap_export_masks": [vp, vp, vp, vp, vp],
            "pt_attn_fwd": [vp, vp, vp, ctypes.c_int, i32, i32, i32, i32, f32, vp, vp, vp, vp],
            "pt_attn_bwd": [vp, vp, vp, vp, vp, vp, ctypes.c_int, i32, i32, i32, i32, f32, vp, vp, vp, vp, vp, sz, vp],
            "pt_sync_status": [vp],
            "pt_debug_wait_timeout": [vp],
            "pt_debug_status": [vp, i32],
            "pt_debug_exp2": [vp, vp, i64, i32, vp],
            "pt_debug_pack_dkdv": [vp, i32, i32, i32, i32, i32, i32, vp, i64, vp, i32p, i32p, i32p],
            "pt_debug_pack_dq": [vp, i32, i32, i32, vp, i64, vp, i32p, i32p, i32p],
            "pt_debug_tree_lists": [vp, i32, vp, vp, i32, i32, i32, vp, i64, vp, i64, i64p],
            "pt_debug_draft_lists": [i32, i32, i32, vp, vp, i32, i32, vp, vp, vp, i64, vp, i64, i64p, i64p],
            "pt_blockmap_prepare_bwd": [vp, i32, i32, i32, vp],
            "pt_attn_bwd_noalloc": [vp, vp, vp, vp, vp, vp, ctypes.c_int, i32, i32, i32, i32, f32, vp, vp, vp, vp,
                                    vp],
            "pt_hoststep_create": [ctypes.c_int, i32, i32, i32, i32, pp],
            "pt_hoststep_run": [vp, vp, vp, vp, vp, f32, vp, vp, vp, vp, vp],
            "pt_hoststep_sync": [vp, vp],
            "pt_hoststep_last_forward": [vp, vp, vp],
            "pt_fold_plan": [vp, i32, vp, vp, i32, i32, vp, pp],
            "pt_foldplan_info": [vp, i32p, i32p, i32p],
            "pt_fold": [vp, vp, i64, vp, vp],
            "pt_unfold": [vp, vp, i64, vp, vp],
            "pt_unfold_grad": [vp, vp, ctypes.c_int, i64, vp, vp],
            "pt_fold_positions": [vp, vp, vp],
            "pt_fold_successors": [vp, vp, vp, vp],
            "pt_fold_mismatches": [vp, vp, i64, vp, vp],
            "pt_debug_pool_usage": [i32, ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_uint64)],
            "pt_cache_tables": [vp, vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, vp, vp, i32, vp, vp],
            "pt_cache_write": [vp, vp, i64, i64, ctypes.c_int, i32, i32, i32, vp, vp, vp, i32, i32, vp],
            "pt_decode_plan": [i32, vp, vp, i32, i32, i32, i32, vp, pp],
            "pt_attn_decode": [vp, i64, vp, vp, ctypes.c_int, i32, i32, i32, vp, i32, vp, vp, f32, vp, vp, vp, vp, sz,
                               vp],
            "pt_attn_decode_drafts": [vp, i64, vp, vp, ctypes.c_int, i32, i32, i32, vp, i32, vp, vp, vp, f32, vp, vp, vp,
                                      vp, sz, vp],
            "pt_draft_tree": [vp, vp, vp, vp, vp, vp, vp, vp],
            "pt_cache_keep": [vp, vp, vp, vp, i32, ctypes.c_int, i32, vp, vp, i32, i32, vp, vp],
            "pt_rotary": [vp, i64, ctypes.c_int, i32, i32, i32, vp, vp, i32, vp, i32, i32, i32, vp, i64, vp],
            "pt_token_logprobs": [vp, i64, ctypes.c_int, i32, i32, vp, vp, vp, i32, f32, i32, vp, vp, vp, vp, vp, vp],
            "pt_token_logprobs_bwd": [vp, vp, vp, i64, ctypes.c_int, i32, i32, vp, vp, vp, i32, f32, vp, vp, vp, i64, vp],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.pt_blockmap_free.argtypes = [vp]
        lib.pt_blockmap_free.restype = None
        lib.pt_foldplan_free.argtypes = [vp]
        lib.pt_foldplan_free.restype = None
        lib.pt_decodeplan_free.argtypes = [vp]
        lib.pt_decodeplan_free.restype = None
        lib.pt_decode_workspace_bytes.argtypes = [vp, i32]
        lib.pt_decode_workspace_bytes.restype = sz
        lib.pt_hoststep_free.argtypes = [vp]
        lib.pt_hoststep_free.restype = None
        lib.pt_bwd_workspace_bytes.argtypes = [i32, i32, i32]
        lib.pt_bwd_workspace_bytes.restype = sz
        lib.pt_last_error.argtypes = []
        lib.pt_last_error.restype = ctypes.c_char_p
        lib.pt_launch_count.argtypes = []
        lib.pt_launch_count.restype = ctypes.c_uint64
        lib.pt_bwd_noalloc_max_scratch_bytes.argtypes = []
        lib.pt_bwd_noalloc_max_scratch_bytes.restype = sz
        lib.pt_debug_drop_listed_tile.argtypes = [i32]
        lib.pt_debug_drop_listed_tile.restype = None
        lib.pt_profile_enable.argtypes = [ctypes.c_int]
        lib.pt_profile_enable.restype = None
        lib.pt_profile_read.argtypes = [ctypes.c_char_p, i64p, ctypes.POINTER(ctypes.c_double)]
        lib.pt_profile_read.restype = ctypes.c_int
        lib.pt_profile_reset.argtypes = []
        lib.pt_profile_reset.restype = None
        _lib = lib
        return lib


def _check(rc: int):
    if rc != PT_OK:
        msg = load_library().pt_last_error()
        raise PTError(rc, msg.decode() if msg else "")


def _stream(stream=None) -> int:
    import torch

    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _ptr(t) -> int:
    return int(t.data_ptr())


class BlockMap:
    """Owner of a device-resident block map built by the library."""

    def __init__(self, handle: int):
        self._h = ctypes.c_void_p(handle)
        self._lib = load_library()
        T, bm_, bn_, nq, nk = (ctypes.c_int32() for _ in range(5))
        _check(self._lib.pt_blockmap_info(self._h, ctypes.byref(T), ctypes.byref(bm_), ctypes.byref(bn_),
                                          ctypes.byref(nq), ctypes.byref(nk), None, None))
        self.T, self.block_m, self.block_n = T.value, bm_.value, bn_.value
        self.nq, self.nk = nq.value, nk.value
        self._counts = None

    def _list_sizes(self):
        # the list sizes reach the host after the build's device work: asked for lazily
        if self._counts is None:
            nnz, nfull = ctypes.c_int64(), ctypes.c_int64()
            _check(self._lib.pt_blockmap_info(self._h, None, None, None, None, None, ctypes.byref(nnz),
                                              ctypes.byref(nfull)))
            self._counts = (nnz.value, nfull.value)
        return self._counts

    @property
    def nnz(self) -> int:
        """Non-empty tiles (waits for the build on the device the first time)."""
        return self._list_sizes()[0]

    @property
    def n_full(self) -> int:
        """Fully kept tiles (waits for the build on the device the first time)."""
        return self._list_sizes()[1]

    @property
    def handle(self):
        return self._h

    def prepare_bwd(self, Hq: int, Hkv: int, D: int, stream=None):
        """Build the work lists attn_bwd_noalloc needs for this head layout."""
        _check(load_library().pt_blockmap_prepare_bwd(self._h, Hq, Hkv, D, ctypes.c_void_p(_stream(stream))))

    def dense(self, stream=None) -> "BlockMap":
        """The same tree with every tile marked partial (no skipping)."""
        out = ctypes.c_void_p()
        _check(self._lib.pt_blockmap_dense(self._h, ctypes.c_void_p(_stream(stream)), ctypes.byref(out)))
        return BlockMap(out.value)

    def export(self) -> dict:
        """Host copies (numpy) of the q-major list and its kv-major transpose."""
        import numpy as np

        n = max(self.nnz, 1)
        q_ptr = np.zeros(self.nq + 1, np.int32)
        k_ptr = np.zeros(self.nk + 1, np.int32)
        kv_idx = np.zeros(n, np.int32)
        q_idx = np.zeros(n, np.int32)
        kind = np.zeros(n, np.uint8)
        kindT = np.zeros(n, np.uint8)
        _check(self._lib.pt_blockmap_export(self._h, q_ptr.ctypes.data, kv_idx.ctypes.data, kind.ctypes.data,
                                            k_ptr.ctypes.data, q_idx.ctypes.data, kindT.ctypes.data))
        e = self.nnz
        return dict(q_ptr=q_ptr, kv_idx=kv_idx[:e], kind=kind[:e], k_ptr=k_ptr, q_idx=q_idx[:e], kindT=kindT[:e],
                    nnz=e, nq=self.nq, nk=self.nk)

    def export_masks(self) -> dict:
        """Host copies (numpy) of the partial tiles' keep bitmasks."""
        import numpy as np

        npart = self.nnz - self.n_full
        pidx = np.zeros(max(self.nnz, 1), np.int32)
        pidxT = np.zeros(max(self.nnz, 1), np.int32)
        rows = np.zeros((max(npart, 1), 128, 4), np.uint32)
        cols = np.zeros((max(npart, 1), 128, 4), np.uint32)
        _check(self._lib.pt_blockmap_export_masks(self._h, pidx.ctypes.data, pidxT.ctypes.data, rows.ctypes.data,
                                                  cols.ctypes.data))
        return dict(pidx=pidx[: self.nnz], pidxT=pidxT[: self.nnz], mask_rows=rows[:npart], mask_cols=cols[:npart])

    def free(self):
        if self._h is not None and self._h.value:
            self._lib.pt_blockmap_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def build_blockmap_tree(node_lengths, path_ptr, path_nodes, block_m: int = 128, block_n: int = 128,
                        stream=None) -> BlockMap:
    """Block map from (node_lengths, CSR sample paths), all host int32 arrays."""
    import numpy as np

    lib = load_library()
    nl = np.ascontiguousarray(np.asarray(node_lengths, dtype=np.int32))
    pp = np.ascontiguousarray(np.asarray(path_ptr, dtype=np.int32))
    pn = np.ascontiguousarray(np.asarray(path_nodes, dtype=np.int32))
    out = ctypes.c_void_p()
    _check(lib.pt_build_blockmap_tree(nl.ctypes.data if nl.size else None, int(nl.size), pp.ctypes.data,
                                      pn.ctypes.data if pn.size else None, int(pp.size - 1), int(block_m),
                                      int(block_n), ctypes.c_void_p(_stream(stream)), ctypes.byref(out)))
    return BlockMap(out.value)


def build_blockmap_draft(ctx_len: int, anchors, block_size: int, block_keep=None, causal: bool = False,
                         window: int = 0, ctx_doc=None, anchor_doc=None, block_m: int = 128, block_n: int = 128,
                         stream=None) -> BlockMap:
    """Block map of the draft-block (DFlash) mask (pt_build_blockmap_draft):
    context [ctx_len] then len(anchors) blocks of block_size tokens; host arrays."""
    import numpy as np

    lib = load_library()
    an = np.ascontiguousarray(np.asarray(anchors, dtype=np.int32))
    keep = None if block_keep is None else np.ascontiguousarray(np.asarray(block_keep, dtype=np.uint8))
    cd = None if ctx_doc is None else np.ascontiguousarray(np.asarray(ctx_doc, dtype=np.int32))
    ad = None if anchor_doc is None else np.ascontiguousarray(np.asarray(anchor_doc, dtype=np.int32))
    ptr = lambda a: (a.ctypes.data if a.size else None) if a is not None else None
    out = ctypes.c_void_p()
    _check(lib.pt_build_blockmap_draft(int(ctx_len), int(an.size), int(block_size), ptr(an), ptr(keep), int(bool(causal)),
                                       int(window), ptr(cd), ptr(ad), int(block_m), int(block_n),
                                       ctypes.c_void_p(_stream(stream)), ctypes.byref(out)))
    return BlockMap(out.value)


def build_blockmap_seg(group_id, suffix_id, block_m: int = 128, block_n: int = 128, stream=None) -> BlockMap:
    """Block map from per-token segment labels (CUDA int32 tensors [T])."""
    import torch

    lib = load_library()
    for t in (group_id, suffix_id):
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == torch.int32 and t.is_contiguous()):
            raise TypeError("group_id and suffix_id must be contiguous CUDA int32 tensors")
    if group_id.numel() != suffix_id.numel():
        raise ValueError("group_id and suffix_id differ in length")
    out = ctypes.c_void_p()
    T = int(group_id.numel())
    _check(lib.pt_build_blockmap_seg(_ptr(group_id) if T else None, _ptr(suffix_id) if T else None, T,
                                     int(block_m), int(block_n), ctypes.c_void_p(_stream(stream)),
                                     ctypes.byref(out)))
    return BlockMap(out.value)


def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return PT_BF16
    if t.dtype == torch.float32:
        return PT_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _check_tensors(*ts):
    import torch

    dt = ts[0].dtype
    for t in ts:
        if not (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous()):
            raise TypeError("tensors must be contiguous CUDA tensors")
        if t.dtype != dt:
            raise TypeError("all tensors must share one dtype")


def attn_fwd(Q, K, V, bm: BlockMap, scale: float = 0.0, O=None, LSE=None, stream=None) -> Tuple:
    """O [T,Hq,D] and LSE [Hq,T] (fp32).  Q [T,Hq,D], K/V [T,Hkv,D]."""
    import torch

    _check_tensors(Q, K, V)
    T, Hq, D = Q.shape
    Hkv = K.shape[1]
    if O is None:
        O = _empty(Q.shape, Q.dtype, Q.device)
    if LSE is None:
        LSE = _empty((Hq, T), torch.float32, Q.device)
    lib = load_library()
    _check(lib.pt_attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _dtype_code(Q), T, Hq, Hkv, D, float(scale), bm.handle,
                           _ptr(O), _ptr(LSE), ctypes.c_void_p(_stream(stream))))
    return O, LSE


def bwd_workspace_bytes(T: int, Hq: int, D: int) -> int:
    return int(load_library().pt_bwd_workspace_bytes(int(T), int(Hq), int(D)))


def attn_bwd(dO, Q, K, V, O, LSE, bm: BlockMap, scale: float = 0.0, dQ=None, dK=None, dV=None, workspace=None,
             stream=None) -> Tuple:
    """dQ [T,Hq,D], dK/dV [T,Hkv,D] from the upstream gradient dO."""
    import torch

    _check_tensors(dO, Q, K, V, O)
    T, Hq, D = Q.shape
    Hkv = K.shape[1]
    dQ = _empty(Q.shape, Q.dtype, Q.device) if dQ is None else dQ
    dK = _empty(K.shape, K.dtype, K.device) if dK is None else dK
    dV = _empty(V.shape, V.dtype, V.device) if dV is None else dV
    need = bwd_workspace_bytes(T, Hq, D)
    if workspace is None:
        workspace = _empty((need,), torch.uint8, Q.device)
    lib = load_library()
    _check(lib.pt_attn_bwd(_ptr(dO), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _dtype_code(Q), T, Hq, Hkv, D,
                           float(scale), bm.handle, _ptr(dQ), _ptr(dK), _ptr(dV), _ptr(workspace),
                           workspace.numel() * workspace.element_size(), ctypes.c_void_p(_stream(stream))))
    return dQ, dK, dV


def attn_bwd_noalloc(dO, Q, K, V, O, LSE, bm: BlockMap, scale: float = 0.0, dQ=None, dK=None, dV=None,
                     stream=None) -> Tuple:
    """attn_bwd without a workspace: the library's built-in scratch array is
    used instead (for callers that cannot allocate device memory; calls that
    overlap on the GPU race on that array)."""
    import torch

    _check_tensors(dO, Q, K, V, O)
    T, Hq, D = Q.shape
    Hkv = K.shape[1]
    dQ = _empty(Q.shape, Q.dtype, Q.device) if dQ is None else dQ
    dK = _empty(K.shape, K.dtype, K.device) if dK is None else dK
    dV = _empty(V.shape, V.dtype, V.device) if dV is None else dV
    lib = load_library()
    _check(lib.pt_attn_bwd_noalloc(_ptr(dO), _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), _dtype_code(Q), T, Hq,
                                   Hkv, D, float(scale), bm.handle, _ptr(dQ), _ptr(dK), _ptr(dV),
                                   ctypes.c_void_p(_stream(stream))))
    return dQ, dK, dV


def sync_status(stream=None):
    """Synchronise and raise PTError if an in-kernel wait timed out, a
    device-side check failed or a cache ran out of pages since the last call."""
    _check(load_library().pt_sync_status(ctypes.c_void_p(_stream(stream))))


def debug_exp2(x, method: int):
    """2^x on the device with the MUFU instruction (method 0) or the kernels'
    FMA-pipe polynomial (method 1); x is a contiguous float32 CUDA tensor."""
    import torch

    if x.dtype != torch.float32 or not x.is_cuda or not x.is_contiguous():
        raise ValueError("x must be a contiguous float32 CUDA tensor")
    y = _empty(x.shape, x.dtype, x.device)
    _check(load_library().pt_debug_exp2(ctypes.c_void_p(x.data_ptr()), ctypes.c_void_p(y.data_ptr()), x.numel(),
                                        method, ctypes.c_void_p(_stream(None))))
    return y


def launch_count() -> int:
    return int(load_library().pt_launch_count())


def profile_enable(on: bool = True):
    """Start (or stop) per-kernel CUDA-event timing inside the library."""
    load_library().pt_profile_enable(1 if on else 0)


def profile_read(kernel: str):
    """(launches, total milliseconds) recorded for one kernel name."""
    n, ms = ctypes.c_int64(), ctypes.c_double()
    _check(load_library().pt_profile_read(kernel.encode(), ctypes.byref(n), ctypes.byref(ms)))
    return int(n.value), float(ms.value)


def profile_reset():
    load_library().pt_profile_reset()


class HostStep:
    """Forward and backward from pinned host tensors, double-buffered on the
    device so that consecutive run() calls overlap their copies with the
    kernels (pt_hoststep_*).  Host tensors: Q, dO, dQ [T, Hq, D]; K, V, dK,
    dV [T, Hkv, D], contiguous, of the dtype given at creation."""

    def __init__(self, dtype, T: int, Hq: int, Hkv: int, D: int):
        import torch

        self._lib = load_library()
        self._dt = dtype
        self._code = PT_BF16 if dtype == torch.bfloat16 else PT_F32 if dtype == torch.float32 else None
        if self._code is None:
            raise TypeError("HostStep: dtype must be torch.bfloat16 or torch.float32")
        self.shape = (T, Hq, Hkv, D)
        out = ctypes.c_void_p()
        _check(self._lib.pt_hoststep_create(self._code, T, Hq, Hkv, D, ctypes.byref(out)))
        self._h = out

    def run(self, Q, K, V, dO, bm: BlockMap, dQ, dK, dV, scale: float = 0.0, stream=None):
        """Queue one step; the host outputs are valid after sync() and a
        synchronisation of the stream."""
        T, Hq, Hkv, D = self.shape
        for t, h in ((Q, Hq), (dO, Hq), (dQ, Hq), (K, Hkv), (V, Hkv), (dK, Hkv), (dV, Hkv)):
            if t.is_cuda or t.dtype != self._dt or tuple(t.shape) != (T, h, D) or not t.is_contiguous():
                raise ValueError("HostStep.run: host tensors of the creation dtype and shape expected")
        _check(self._lib.pt_hoststep_run(self._h, _ptr(Q), _ptr(K), _ptr(V), _ptr(dO), float(scale), bm.handle,
                                         _ptr(dQ), _ptr(dK), _ptr(dV), ctypes.c_void_p(_stream(stream))))

    def sync(self, stream=None):
        """Make the stream wait for every download queued so far."""
        _check(self._lib.pt_hoststep_sync(self._h, ctypes.c_void_p(_stream(stream))))

    def last_forward(self):
        """O [T, Hq, D] and LSE [Hq, T] of the most recent run(), as new host
        tensors (waits for that step's kernels)."""
        import torch

        T, Hq, Hkv, D = self.shape
        O = torch.empty((T, Hq, D), dtype=self._dt)
        L = torch.empty((Hq, T), dtype=torch.float32)
        _check(self._lib.pt_hoststep_last_forward(self._h, _ptr(O), _ptr(L)))
        return O, L

    def free(self):
        if self._h is not None and self._h.value:
            self._lib.pt_hoststep_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


class FoldPlan:
    """Shared-prefix fold of rollouts and its inverse (pt_fold_plan and the
    calls after it): the flat layout of the tree (node_lengths, CSR sample
    paths) against n_samples rollout rows of row_len tokens.  Tensors carry
    one row of data per token: flat [T, ...], rollouts [n_samples, row_len, ...]."""

    def __init__(self, node_lengths, path_ptr, path_nodes, row_len: int, stream=None):
        import numpy as np

        self._lib = load_library()
        nl = np.ascontiguousarray(np.asarray(node_lengths, dtype=np.int32))
        pp = np.ascontiguousarray(np.asarray(path_ptr, dtype=np.int32))
        pn = np.ascontiguousarray(np.asarray(path_nodes, dtype=np.int32))
        out = ctypes.c_void_p()
        _check(self._lib.pt_fold_plan(nl.ctypes.data if nl.size else None, int(nl.size), pp.ctypes.data,
                                      pn.ctypes.data if pn.size else None, int(pp.size - 1), int(row_len),
                                      ctypes.c_void_p(_stream(stream)), ctypes.byref(out)))
        self._h = out
        T, S, L = (ctypes.c_int32() for _ in range(3))
        _check(self._lib.pt_foldplan_info(self._h, ctypes.byref(T), ctypes.byref(S), ctypes.byref(L)))
        self.T, self.n_samples, self.row_len = T.value, S.value, L.value

    @staticmethod
    def _row_bytes(t, lead: int) -> int:
        """Bytes of one token's row: the trailing dimensions (valid for empty leading ones)."""
        n = t.element_size()
        for d in t.shape[lead:]:
            n *= d
        return n

    def _need(self, t, shape, name):
        if not t.is_cuda or not t.is_contiguous() or tuple(t.shape[:len(shape)]) != shape:
            raise ValueError(f"{name} must be a contiguous CUDA tensor of leading shape {shape}")

    def fold(self, roll, out=None, stream=None):
        """flat[t] = roll[first sample holding t][its position]."""
        import torch

        self._need(roll, (self.n_samples, self.row_len), "roll")
        rb = self._row_bytes(roll, 2)
        out = _empty((self.T,) + tuple(roll.shape[2:]), roll.dtype, roll.device) if out is None else out
        _check(self._lib.pt_fold(self._h, _ptr(roll), rb, _ptr(out), ctypes.c_void_p(_stream(stream))))
        return out

    def unfold(self, flat, out=None, stream=None):
        """roll[s][j] = flat[token at position j of sample s]; padding zero."""
        import torch

        self._need(flat, (self.T,), "flat")
        rb = self._row_bytes(flat, 1)
        out = _empty((self.n_samples, self.row_len) + tuple(flat.shape[1:]), flat.dtype, flat.device) \
            if out is None else out
        _check(self._lib.pt_unfold(self._h, _ptr(flat), rb, _ptr(out), ctypes.c_void_p(_stream(stream))))
        return out

    def unfold_grad(self, droll, out=None, stream=None):
        """dflat[t] = sum of droll over every copy of t (fp32 sums, rounded once)."""
        import torch

        self._need(droll, (self.n_samples, self.row_len), "droll")
        width = 1
        for d in droll.shape[2:]:
            width *= d
        out = _empty((self.T,) + tuple(droll.shape[2:]), droll.dtype, droll.device) if out is None else out
        _check(self._lib.pt_unfold_grad(self._h, _ptr(droll), _dtype_code(droll), width, _ptr(out),
                                        ctypes.c_void_p(_stream(stream))))
        return out

    def positions(self, device=None, stream=None):
        """Position ids of the flat tokens (int64 [T])."""
        import torch

        out = _empty((self.T,), torch.int64, device or torch.device("cuda"))
        _check(self._lib.pt_fold_positions(self._h, _ptr(out), ctypes.c_void_p(_stream(stream))))
        return out

    def successors(self, device=None, stream=None) -> Tuple:
        """Which flat tokens follow which: succ_ptr [T + 1] and succ [T] (int32),
        the row_ptr and index of token_logprobs for the flat layout."""
        import torch

        device = device or torch.device("cuda")
        ptr, succ = _empty((self.T + 1,), torch.int32, device), _empty((self.T,), torch.int32, device)
        if isinstance(stream, torch.cuda.Stream):
            ptr.record_stream(stream)
            succ.record_stream(stream)
        _check(self._lib.pt_fold_successors(self._h, _ptr(ptr), _ptr(succ), ctypes.c_void_p(_stream(stream))))
        return ptr, succ

    def mismatches(self, roll, stream=None) -> int:
        """Rollout entries whose bytes differ from the entry the fold keeps (synchronises)."""
        import torch

        self._need(roll, (self.n_samples, self.row_len), "roll")
        cnt = _empty((1,), torch.int64, roll.device)
        _check(self._lib.pt_fold_mismatches(self._h, _ptr(roll), self._row_bytes(roll, 2), _ptr(cnt),
                                            ctypes.c_void_p(_stream(stream))))
        return int(cnt.item())

    def free(self):
        if getattr(self, "_h", None) is not None and self._h.value:
            self._lib.pt_foldplan_free(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def fold_plan(node_lengths, path_ptr, path_nodes, row_len: int, stream=None) -> FoldPlan:
    """Plan of the shared-prefix fold for a tree and a rollout row length."""
    return FoldPlan(node_lengths, path_ptr, path_nodes, row_len, stream)


# The calls below run once per layer and step, next to kernels of a few
# microseconds, so their Python side is kept short: one attribute or method of
# a tensor costs about 0.1 us here, an allocation 1.5 us.
_T = None  # torch, its int32, int64, float32 and bfloat16, a device's current stream, and the current device


def _torch():
    global _T
    if _T is None:
        import torch

        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is None:
            raw = lambda dev: torch.cuda.current_stream(dev).cuda_stream  # noqa: E731
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _T = torch, torch.int32, torch.int64, torch.float32, torch.bfloat16, raw, device
    return _T


def _bad(t, name: str, dtype, dev):
    """Raise for a tensor of the cache calls that is not dense, of this dtype
    and on the current device."""
    if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or dev < 0:
        raise TypeError(f"{name} must be a contiguous CUDA tensor of {dtype}")
    raise ValueError(f"{name} is on device {t.get_device()}, the current device is {dev}")


def _need(t, name: str, dtype, shape, dev):
    """dev: the current device, or -1 when the call's first tensor is not on one."""
    if t.dtype != dtype or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _bad(t, name, dtype, dev)
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} expected")


def _out(shape, dtype, like):
    return _T[0].empty(shape, dtype=dtype, device=like.device) if _alloc_hook is None else \
        _alloc_hook(tuple(shape), dtype, like.device)


def _launch_stream(stream, dev, *held):
    """The raw stream of a call.  On a stream of the caller's choice, the
    tensors allocated here (`held`) are marked as used on it.  They are allocated
    on the current stream: what the caller's stream does behind that stream's
    work (stream.wait_stream(torch.cuda.current_stream())) finds their memory
    free."""
    if stream is None:
        return _T[5](dev)
    if isinstance(stream, _T[0].cuda.Stream):
        for t in held:
            t.record_stream(stream)
    return int(stream.cuda_stream)


def cache_tables(held, added, tables, ring, counters, page_size: int, max_new: int, start=None, stream=None) -> Tuple:
    """One step of a paged cache's rows (pt_cache_tables): row i goes from
    held[i] to held[i] + added[i] tokens, taking pages from the ring of free
    ids or giving them back.  CUDA int32 tensors held, added, start [n], tables
    [n, max_pages] and ring [cap]; counters int64 [2].  tables and ring change
    in place; returns new lens [n], counters [2], row_ptr [n + 1], and the
    added tokens' slots and position ids (int64 [max_new])."""
    _, i32, i64, _, _, _, device = _torch()
    n, cap = held.numel(), ring.numel()
    if cap > 1 << 30:
        raise ValueError(f"a ring of {cap} ids is out of range")
    row = (n,)
    dev = device() if held.is_cuda else -1
    _need(held, "held", i32, row, dev)
    _need(added, "added", i32, row, dev)
    _need(ring, "ring", i32, (cap,), dev)
    _need(counters, "counters", i64, (2,), dev)
    width = tables.shape[1] if tables.dim() == 2 else 0
    _need(tables, "tables", i32, (n, width), dev)
    if start is not None:
        _need(start, "start", i32, row, dev)
    if not 0 <= max_new <= 1 << 30:
        raise ValueError(f"max_new = {max_new} is out of range")
    lens, row_ptr = _out(row, i32, held), _out((n + 1,), i32, held)
    slots, positions, out = _out((max_new,), i64, held), _out((max_new,), i64, held), _out((2,), i64, held)
    rc = load_library().pt_cache_tables(
        held.data_ptr(), added.data_ptr(), None if start is None else start.data_ptr(), n, page_size,
        tables.data_ptr(), width, ring.data_ptr(), cap, counters.data_ptr(), lens.data_ptr(), row_ptr.data_ptr(),
        slots.data_ptr(), positions.data_ptr(), max_new, out.data_ptr(),
        _launch_stream(stream, dev, lens, row_ptr, slots, positions, out))
    if rc:
        _check(rc)
    return lens, out, row_ptr, slots, positions


def _cache_shape(Kc, Vc, dtype, dev):
    """(code of the dtype, cache shape)."""
    code = PT_BF16 if dtype == _T[4] else PT_F32 if dtype == _T[3] else None
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    shape = Kc.shape
    if len(shape) != 4:
        raise ValueError("Kc and Vc are [n_pages, Hkv, page_size, D]")
    if Kc.dtype != dtype or Kc.get_device() != dev or dev < 0 or not Kc.is_contiguous():
        _bad(Kc, "Kc", dtype, dev)
    _need(Vc, "Vc", dtype, shape, dev)
    return code, shape


def _token_rows(t, name, dtype, T, heads, D, dev):
    """[T, heads, D] tokens whose heads are dense (a slice of a fused
    projection will do); returns the elements between tokens."""
    if t.dtype != dtype or t.get_device() != dev or dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor [T, heads, head_dim] of {dtype} on the current device")
    if t.shape != (T, heads, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, ({T}, {heads}, {D}) expected")
    s, h, d = t.stride()
    if (d != 1 and D > 1) or (h != D and heads > 1) or (s < heads * D and T > 1):
        if T and heads and D:
            raise ValueError(f"{name}: the heads of a token must be dense and tokens must not overlap")
    return s if T > 1 else heads * D


def cache_write(K, V, slots, Kc, Vc, stream=None) -> None:
    """Put tokens' K and V [T, Hkv, D] into their slots (int64 [T], negative:
    passed over) of the cache Kc, Vc [n_pages, Hkv, page_size, D], in place."""
    i64, device = _torch()[2], _T[6]
    dev = device() if K.is_cuda else -1
    dtype = K.dtype
    code, (n_pages, Hkv, ps, D) = _cache_shape(Kc, Vc, dtype, dev)
    T = K.shape[0]
    ks, vs = _token_rows(K, "K", dtype, T, Hkv, D, dev), _token_rows(V, "V", dtype, T, Hkv, D, dev)
    _need(slots, "slots", i64, (T,), dev)
    rc = load_library().pt_cache_write(K.data_ptr(), V.data_ptr(), ks, vs, code, T, Hkv, D, slots.data_ptr(),
                                       Kc.data_ptr(), Vc.data_ptr(), n_pages, ps, _launch_stream(stream, dev))
    if rc:
        _check(rc)


class DecodePlan:
    """Plan of the decoding attention for a tree's paths and a head layout
    (pt_decode_plan).  It holds no lengths: one plan serves every layer and
    step until a path changes."""

    def __init__(self, n_nodes: int, path_ptr, path_nodes, Hq: int, Hkv: int, q_len: int = 1, stream=None):
        import numpy as np

        self._h = None
        self._lib = load_library()
        pp = np.ascontiguousarray(np.asarray(path_ptr, dtype=np.int32))
        pn = np.ascontiguousarray(np.asarray(path_nodes, dtype=np.int32))
        if pp.size < 1 or (pp.size > 1 and int(pp[-1]) > pn.size):
            raise ValueError("path_ptr runs past path_nodes")
        out = ctypes.c_void_p()
        _check(self._lib.pt_decode_plan(int(n_nodes), pp.ctypes.data, pn.ctypes.data if pn.size else None,
                                        int(pp.size - 1), int(Hq), int(Hkv), int(q_len),
                                        ctypes.c_void_p(_stream(stream)), ctypes.byref(out)))
        self._h = out
        self.n_nodes, self.n_samples, self.Hq, self.Hkv, self.q_len = n_nodes, int(pp.size - 1), Hq, Hkv, q_len
        self.n_rows = self.n_samples * q_len  # query tokens of a call

    @property
    def handle(self):
        return self._h

    def workspace_bytes(self, D: int) -> int:
        """Bytes of scratch attn_decode needs at this head_dim."""
        return int(self._lib.pt_decode_workspace_bytes(self._h, int(D)))

    def free(self):
        if self._h is not None and self._h.value:
            self._lib.pt_decodeplan_free(self._h)
        self._h = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def decode_plan(n_nodes: int, path_ptr, path_nodes, Hq: int, Hkv: int, q_len: int = 1, stream=None) -> DecodePlan:
    """Plan of the decoding attention: host int32 CSR paths over cache rows."""
    return DecodePlan(n_nodes, path_ptr, path_nodes, Hq, Hkv, q_len, stream)


def attn_decode(Q, Kc, Vc, tables, lens, plan: DecodePlan, q_count=None, scale: float = 0.0, O=None, LSE=None,
                workspace=None, stream=None, draft_mask=None) -> Tuple:
    """O [n_samples * q_len, Hq, D] and LSE [Hq, n_samples * q_len] (fp32) of
    the samples' newest tokens Q over the cache Kc, Vc [n_pages, Hkv,
    page_size, D], tables [n_nodes, max_pages], lens [n_nodes] (pt_attn_decode).
    With q_count, rows behind a sample's queries keep what O and LSE held.
    draft_mask [n_samples * q_len, ceil(q_len / 32)] (int32, as draft_tree gives
    it): the queries are a tree of drafts (pt_attn_decode_drafts)."""
    torch, i32, _, f32, _, _, device = _torch()
    dev = device() if Q.is_cuda else -1
    dtype = Q.dtype
    code, (n_pages, Hkv, ps, D) = _cache_shape(Kc, Vc, dtype, dev)
    T, Hq, N = plan.n_rows, plan.Hq, plan.n_nodes
    if Hkv != plan.Hkv:
        raise ValueError(f"the cache has {Hkv} kv heads, the plan {plan.Hkv}")
    qs = _token_rows(Q, "Q", dtype, T, Hq, D, dev)
    width = tables.shape[1] if tables.dim() == 2 else 0
    _need(tables, "tables", i32, (N, width), dev)
    _need(lens, "lens", i32, (N,), dev)
    if q_count is not None:
        _need(q_count, "q_count", i32, (plan.n_samples,), dev)
    held = []
    if O is None:
        O = _out((T, Hq, D), dtype, Q)
        held.append(O)
    else:
        _need(O, "O", dtype, (T, Hq, D), dev)
    if LSE is None:
        LSE = _out((Hq, T), f32, Q)
        held.append(LSE)
    else:
        _need(LSE, "LSE", f32, (Hq, T), dev)
    if workspace is None:
        workspace = _out((plan.workspace_bytes(D),), torch.uint8, Q)
        held.append(workspace)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous CUDA tensor on the current device")
    call, masked = load_library().pt_attn_decode, ()
    if draft_mask is not None:
        _need(draft_mask, "draft_mask", i32, (T, (plan.q_len + 31) // 32), dev)
        call, masked = _lib.pt_attn_decode_drafts, (draft_mask.data_ptr(),)
    rc = call(
        Q.data_ptr(), qs, Kc.data_ptr(), Vc.data_ptr(), code, D, n_pages, ps, tables.data_ptr(), width,
        lens.data_ptr(), None if q_count is None else q_count.data_ptr(), *masked, scale, plan.handle, O.data_ptr(),
        LSE.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
        _launch_stream(stream, dev, *held))
    if rc:
        _check(rc)
    return O, LSE


def draft_tree(parents, lens, plan: DecodePlan, q_count=None, start=None, stream=None) -> Tuple:
    """Trees of drafts (pt_draft_tree): parents [n_samples * q_len] (CUDA int32,
    the draft above each, or -1) become draft_mask [n_samples * q_len, ceil(q_len
    / 32)] (int32) for attn_decode, and the drafts' position ids (int64
    [n_samples * q_len]) from lens and start (int32 [n_nodes])."""
    _, i32, i64, _, _, _, device = _torch()
    dev = device() if parents.is_cuda else -1
    n, N = plan.n_rows, plan.n_nodes
    _need(parents, "parents", i32, (n,), dev)
    _need(lens, "lens", i32, (N,), dev)
    if q_count is not None:
        _need(q_count, "q_count", i32, (plan.n_samples,), dev)
    if start is not None:
        _need(start, "start", i32, (N,), dev)
    mask, positions = _out((n, (plan.q_len + 31) // 32), i32, parents), _out((n,), i64, parents)
    rc = load_library().pt_draft_tree(
        parents.data_ptr(), lens.data_ptr(), None if q_count is None else q_count.data_ptr(),
        None if start is None else start.data_ptr(), plan.handle, mask.data_ptr(), positions.data_ptr(),
        _T[5](dev) if stream is None else _launch_stream(stream, dev, mask, positions))
    if rc:
        _check(rc)
    return mask, positions


def cache_keep(kept, Kc, Vc, tables, lens, plan: DecodePlan, q_count=None, stream=None) -> None:
    """Move the accepted drafts' keys and values together (pt_cache_keep): of
    each sample, draft kept[s, i] (CUDA int32 [n_samples, q_len], ascending, ended
    by a negative one) becomes draft i of its own node, in place in Kc and Vc."""
    _, i32, _, _, _, _, device = _torch()
    dev = device() if kept.is_cuda else -1
    code, (n_pages, Hkv, ps, D) = _cache_shape(Kc, Vc, Kc.dtype, dev)
    if Hkv != plan.Hkv:
        raise ValueError(f"the cache has {Hkv} kv heads, the plan {plan.Hkv}")
    _need(kept, "kept", i32, (plan.n_samples, plan.q_len), dev)
    width = tables.shape[1] if tables.dim() == 2 else 0
    _need(tables, "tables", i32, (plan.n_nodes, width), dev)
    _need(lens, "lens", i32, (plan.n_nodes,), dev)
    if q_count is not None:
        _need(q_count, "q_count", i32, (plan.n_samples,), dev)
    rc = load_library().pt_cache_keep(
        kept.data_ptr(), None if q_count is None else q_count.data_ptr(), lens.data_ptr(), tables.data_ptr(), width,
        code, D, Kc.data_ptr(), Vc.data_ptr(), n_pages, ps, plan.handle, _launch_stream(stream, dev))
    if rc:
        _check(rc)


def _code(dtype) -> int:
    code = PT_BF16 if dtype == _T[4] else PT_F32 if dtype == _T[3] else None
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def rotary(X, positions, inv_freq, sections=None, interleaved: bool = False, inverse: bool = False, out=None,
           stream=None):
    """X [T, H, D] with its pairs of columns turned by position (pt_rotary).
    positions: CUDA int64 [T], or [axes, T] with sections, the pairs of each axis;
    inv_freq: fp32 [rot_dim / 2].  inverse gives the inverse, which is also the
    gradient.  X and out may be slices of a fused projection; out may be X."""
    _, _, i64, f32, _, _, device = _torch()
    dev = device() if X.is_cuda else -1
    shape = X.shape
    if len(shape) != 3:
        raise ValueError("X is [T, H, head_dim]")
    T, H, D = shape
    dtype = X.dtype
    code = _code(dtype)
    xs = _token_rows(X, "X", dtype, T, H, D, dev)
    axes = 1 if sections is None else len(sections)
    _need(positions, "positions", i64, (T,) if axes == 1 and positions.dim() == 1 else (axes, T), dev)
    half = inv_freq.numel()
    _need(inv_freq, "inv_freq", f32, (half,), dev)
    given = out is not None
    if given:
        ys = _token_rows(out, "out", dtype, T, H, D, dev)
    else:
        out, ys = _out(shape, dtype, X), H * D
    if T == 1:  # (a token has no neighbour: one stride for both, whatever the slices')
        xs = ys = H * D
    pairs = None if sections is None else (ctypes.c_int32 * max(axes, 1))(*sections)
    rc = load_library().pt_rotary(
        X.data_ptr(), xs, code, T, H, D, positions.data_ptr(), inv_freq.data_ptr(), 2 * half, pairs, axes, interleaved,
        inverse, out.data_ptr(), ys,
        _T[5](dev) if stream is None else _launch_stream(stream, dev, *(() if given else (out,))))
    if rc:
        _check(rc)
    return out


def _logit_rows(t, name, dtype, shape, dev) -> int:
    """[R, V] rows of dense elements; returns the elements between rows."""
    if t.dtype != dtype or t.get_device() != dev or dev < 0:
        raise TypeError(f"{name} must be a CUDA tensor [rows, vocabulary] of {dtype} on the current device")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, {tuple(shape)} expected")
    R, V = shape
    s, d = t.stride()
    if R and V and ((d != 1 and V > 1) or (s < V and R > 1)):
        raise ValueError(f"{name}: the logits of a row must be dense and rows must not overlap")
    return s if R > 1 else V


def _entries(targets, row_ptr, index, R, dev):
    """The checked tokens of the rows: (N, pointers of targets, row_ptr and index)."""
    i32, i64 = _T[1], _T[2]
    N = targets.numel()
    _need(targets, "targets", i64, (N,), dev)
    if row_ptr is not None:
        _need(row_ptr, "row_ptr", i32, (R + 1,), dev)
    elif N != R:
        raise ValueError(f"{N} targets for {R} rows need a row_ptr")
    if index is not None:
        _need(index, "index", i32, (N,), dev)
    return N, targets.data_ptr(), None if row_ptr is None else row_ptr.data_ptr(), None if index is None else index.data_ptr()


def token_logprobs(logits, targets, row_ptr=None, index=None, top_k: int = 0, entropy: bool = False,
                   scale: float = 1.0, stream=None) -> Tuple:
    """Log probabilities of given tokens (pt_token_logprobs): logits [R, V],
    targets int64 [N] (negative: not scored).  Row r scores token r, or tokens
    index[row_ptr[r]:row_ptr[r + 1]] (int32, every token once; FoldPlan.successors
    gives both for a tree).  Returns logp [N], LSE [R], entropy [R] or None, and the top_k most
    likely tokens' log probabilities and ids [R, top_k] or None."""
    _, _, i64, f32, _, _, device = _torch()
    dev = device() if logits.is_cuda else -1
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits is [rows, vocabulary]")
    R, V = shape
    dtype = logits.dtype
    code = _code(dtype)
    rs = _logit_rows(logits, "logits", dtype, shape, dev)
    N, targets_p, ptr_p, index_p = _entries(targets, row_ptr, index, R, dev)
    logp, lse = _out((N,), f32, logits), _out((R,), f32, logits)
    H = top = ids = None
    H_p = top_p = ids_p = None
    if entropy:
        H = _out((R,), f32, logits)
        H_p = H.data_ptr()
    if top_k > 0:
        top, ids = _out((R, top_k), f32, logits), _out((R, top_k), i64, logits)
        top_p, ids_p = top.data_ptr(), ids.data_ptr()
    rc = load_library().pt_token_logprobs(
        logits.data_ptr(), rs, code, R, V, targets_p, ptr_p, index_p, N, scale, top_k, logp.data_ptr(), lse.data_ptr(),
        H_p, top_p, ids_p, _T[5](dev) if stream is None else
        _launch_stream(stream, dev, *[t for t in (logp, lse, H, top, ids) if t is not None]))
    if rc:
        _check(rc)
    return logp, lse, H, top, ids


def token_logprobs_bwd(dlogp, logits, targets, lse, row_ptr=None, index=None, dentropy=None, entropy=None,
                       scale: float = 1.0, dlogits=None, stream=None):
    """dlogits [R, V] from dlogp [N] and, with the forward's entropy, dentropy
    [R] (pt_token_logprobs_bwd); lse and entropy as token_logprobs returned them.
    dlogits may be logits.  Beside logits that are columns of a wider buffer give
    one with their row stride (without, it is dense and stored by elements)."""
    _, _, _, f32, _, _, device = _torch()
    dev = device() if logits.is_cuda else -1
    if logits.dim() != 2:
        raise ValueError("logits is [rows, vocabulary]")
    R, V = logits.shape
    code = _code(logits.dtype)
    rs = _logit_rows(logits, "logits", logits.dtype, (R, V), dev)
    N, *entries = _entries(targets, row_ptr, index, R, dev)
    _need(dlogp, "dlogp", f32, (N,), dev)
    _need(lse, "lse", f32, (R,), dev)
    if dentropy is not None:
        if entropy is None:
            raise ValueError("dentropy needs the forward's entropy")
        _need(dentropy, "dentropy", f32, (R,), dev)
        _need(entropy, "entropy", f32, (R,), dev)
    held = ()
    if dlogits is None:
        dlogits = _out((R, V), logits.dtype, logits)
        held, ds = (dlogits,), V
    else:
        ds = _logit_rows(dlogits, "dlogits", logits.dtype, (R, V), dev)
    rc = load_library().pt_token_logprobs_bwd(
        dlogp.data_ptr(), None if dentropy is None else dentropy.data_ptr(), logits.data_ptr(), rs, code, R, V, *entries,
        N, scale, lse.data_ptr(), None if entropy is None else entropy.data_ptr(), dlogits.data_ptr(), ds,
        _launch_stream(stream, dev, *held))
    if rc:
        _check(rc)
    return dlogits
