"""ctypes binding over libmla_prefill.so (argument marshalling only).

Every function mirrors one C entry point of ``include/mla_prefill.h`` under
the same name.  Tensors are torch tensors: device memory and the current
CUDA stream come from torch, all arithmetic happens in the library's
kernels.  There is no fallback: if the shared library cannot be built or
loaded, the first call raises.
"""
from __future__ import annotations

import ctypes
import threading

import numpy as np

from . import _build

_lib = None
_lock = threading.Lock()

MLA_OK = 0
_c_int, _c_i64, _c_f, _c_vp = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p
_i32p = ctypes.POINTER(ctypes.c_int32)
_i64p = ctypes.POINTER(ctypes.c_int64)

_SIGNATURES = {
    "mla_error_string": (ctypes.c_char_p, [_c_int]),
    "mla_abi_version": (_c_int, []),
    "mla_prefill_plan": (_c_int, [ctypes.POINTER(_c_vp), _i32p, _i32p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                  _c_f, _c_int, _c_f, _c_vp]),
    "mla_prefill_run": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_prefill_run_merge": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_prefill_run_shared_rope": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp, _c_vp, _c_int,
                                             _c_vp]),
    "mla_prefill_status": (_c_int, [_c_vp]),
    "mla_plan_destroy": (_c_int, [_c_vp]),
    "mla_plan_query": (_c_int, [_c_vp, _c_int, _i64p]),
    "mla_plan_units_host": (_c_int, [_i32p, _i32p, _c_int, _c_int, _c_int, _c_int, _c_int, _i32p, _c_i64, _i32p,
                                     _i64p]),
    "mla_gather_latent": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64,
                                   _c_vp, _c_vp, _c_vp]),
    "mla_gather_latent_fp8": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64,
                                       _c_vp, _c_vp, _c_vp]),
    "mla_cache_write": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "mla_up_proj": (_c_int, [_c_vp, _c_vp, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_up_proj_paged": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64,
                                   _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_up_proj_paged_split": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int,
                                         _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_merge_state": (_c_int, [_c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_i64, _c_int, _c_int, _c_vp]),
    "mla_prefill_run_noalloc": (_c_int, [_i32p, _i32p, _c_int, _c_int, _c_int, _c_int, _c_int, _c_f, _c_int, _c_f,
                                         _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_absorbed_plan": (_c_int, [ctypes.POINTER(_c_vp), _i32p, _i32p, _c_int, _c_int, _c_int, _c_int, _c_f, _c_f,
                                   _c_vp]),
    "mla_absorbed_run": (_c_int, [_c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_int, _c_vp, _c_vp, _c_vp]),
    "mla_block_table_update": (_c_int, [_c_vp, _c_vp, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_vp,
                                        _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "mla_tree_mask": (_c_int, [_c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_int, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_tree_workspace": (_c_int, [_c_i64, _c_int, _i64p]),
    "mla_tree_workspace_fp4": (_c_int, [_c_i64, _c_int, _c_int, _c_i64, _c_int, _i64p]),
    "mla_tree_attention": (_c_int, [_c_vp, _c_vp, _c_i64, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_int,
                                    _c_i64, _c_int, _c_f, _c_f, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "mla_tree_attention_fp4": (_c_int, [_c_vp, _c_vp, _c_i64, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_vp, _c_int, _c_int,
                                        _c_i64, _c_int, _c_f, _c_f, _c_vp, _c_vp, _c_vp, _c_i64, _c_vp, _c_vp]),
    "mla_tree_verify": (_c_int, [_c_vp, _c_vp, _c_int, _c_i64, _c_vp, _c_vp, _c_vp, _c_int, _c_i64, _c_vp, _c_vp, _c_vp,
                                 _c_int, _c_vp, _c_vp, _c_vp, _c_vp]),
    "mla_cache_append": (_c_int, [_c_vp, _c_int, _c_i64, _c_int, _c_vp, _c_i64, _c_vp, _c_f, _c_vp, _c_vp, _c_i64, _c_int,
                                  _c_vp, _c_i64, _c_vp, _c_i64, _c_i64, _c_int, _c_vp, _c_i64, _c_i64, _c_vp, _c_vp]),
    "mla_gather_latent_fp4": (_c_int, [_c_vp, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_int, _c_i64,
                                       _c_vp, _c_vp, _c_vp]),
    "mla_tree_commit": (_c_int, [_c_vp, _c_int, _c_i64, _c_i64, _c_int, _c_int, _c_vp, _c_int, _c_vp, _c_vp, _c_vp,
                                 _c_int, _c_int, _c_vp, _c_vp]),
}
EXPORTED = tuple(_SIGNATURES)


class MlaError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {error_string(code)} ({code})")


def library(build_if_stale: bool = True) -> ctypes.CDLL:
    """Load (building first if needed) the shared library."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build_if_stale else _build.LIB_PATH
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _lib = lib
    return _lib


def library_path() -> str:
    return _build.LIB_PATH


def error_string(code: int) -> str:
    return library().mla_error_string(code).decode()


def _check(code: int, what: str):
    if code != MLA_OK:
        raise MlaError(code, what)


def _host_i32(x) -> np.ndarray:
    if hasattr(x, "detach"):
        x = x.detach().cpu().numpy()
    return np.ascontiguousarray(np.asarray(x, dtype=np.int32))


def _ptr(a: np.ndarray):
    return a.ctypes.data_as(_i32p)


def _stream(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev(t, dtype, name):
    import torch
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


# ---------------------------------------------------------------------------- plan
class PrefillPlan:
    """Owns an ``mla_plan_t``; created by :func:`mla_prefill_plan`."""

    def __init__(self, handle: ctypes.c_void_p, num_heads: int, total_q: int, total_kv: int):
        self._h = handle
        self.num_heads = num_heads
        self.total_q = total_q
        self.total_kv = total_kv

    @property
    def handle(self):
        return self._h

    def query(self, which: int) -> int:
        v = ctypes.c_int64(0)
        _check(library().mla_plan_query(self._h, which, ctypes.byref(v)), "mla_plan_query")
        return int(v.value)

    num_units = property(lambda self: self.query(0))
    num_ctas = property(lambda self: self.query(1))
    allowed_pairs = property(lambda self: self.query(4))
    kv_tiles = property(lambda self: self.query(5))
    cta_pairs = property(lambda self: bool(self.query(6)))

    def run(self, q, k, v, o=None, lse=None, return_lse=True, stream=None):
        return mla_prefill_run(self, q, k, v, o, lse, return_lse, stream)

    def run_merge(self, q, k, v, o, lse, stream=None):
        return mla_prefill_run_merge(self, q, k, v, o, lse, stream)

    def status(self) -> int:
        return mla_prefill_status(self)

    def destroy(self):
        if self._h:
            h, self._h = self._h, None
            _check(library().mla_plan_destroy(h), "mla_plan_destroy")

    def __del__(self):
        try:
            if self._h and _lib is not None:
                _lib.mla_plan_destroy(self._h)
                self._h = None
        except Exception:
            pass


def mla_prefill_plan(qo_indptr, kv_indptr, num_heads: int, head_dim_qk: int = 192, head_dim_vo: int = 128,
                     causal: bool = True, sm_scale: float | None = None, window_left: int = -1,
                     logits_soft_cap: float = 0.0, stream=None) -> PrefillPlan:
    """Plan a ragged prefill (host indptrs).  ``sm_scale`` is required, as on the pages."""
    if sm_scale is None:
        raise ValueError("sm_scale must be given explicitly")
    qo, kv = _host_i32(qo_indptr), _host_i32(kv_indptr)
    if qo.ndim != 1 or kv.shape != qo.shape or qo.size < 1:
        raise ValueError("qo_indptr and kv_indptr must be 1-D of equal length batch+1")
    h = ctypes.c_void_p()
    _check(library().mla_prefill_plan(ctypes.byref(h), _ptr(qo), _ptr(kv), qo.size - 1, num_heads, head_dim_qk,
                                      head_dim_vo, int(bool(causal)), float(sm_scale), int(window_left),
                                      float(logits_soft_cap), _stream(stream)), "mla_prefill_plan")
    return PrefillPlan(h, num_heads, int(qo[-1]), int(kv[-1]))


class AbsorbedPlan(PrefillPlan):
    """An ``mla_plan_t`` made by :func:`mla_absorbed_plan` (absorbed-weight MQA prefill over
    the paged latent cache); status, query and destroy as for :class:`PrefillPlan`."""

    def __init__(self, handle, num_heads: int, total_q: int, batch: int, block_size: int, max_kv_blocks: int):
        super().__init__(handle, num_heads, total_q, 0)
        self.batch = batch
        self.block_size = block_size
        self.max_kv_blocks = max_kv_blocks

    def run(self, q_abs, cache, block_table, o=None, lse=None, return_lse=True, stream=None):
        return mla_absorbed_run(self, q_abs, cache, block_table, o, lse, return_lse, stream)

    def run_merge(self, *args, **kwargs):
        raise TypeError("an absorbed plan runs with mla_absorbed_run")


def mla_absorbed_plan(qo_indptr, kv_lens, num_heads: int, block_size: int, causal: bool = True,
                      sm_scale: float | None = None, logits_soft_cap: float = 0.0, stream=None) -> AbsorbedPlan:
    """Plan an absorbed-weight prefill: request r has qo_indptr[r+1]-qo_indptr[r] new query
    rows, the last ones of its kv_lens[r] cache positions.  ``sm_scale`` is required."""
    if sm_scale is None:
        raise ValueError("sm_scale must be given explicitly")
    qo, kl = _host_i32(qo_indptr), _host_i32(kv_lens)
    if qo.ndim != 1 or qo.size < 1 or kl.shape != (qo.size - 1,):
        raise ValueError("qo_indptr must be 1-D [batch+1] and kv_lens [batch]")
    h = ctypes.c_void_p()
    _check(library().mla_absorbed_plan(ctypes.byref(h), _ptr(qo), _ptr(kl), qo.size - 1, num_heads, int(block_size),
                                       int(bool(causal)), float(sm_scale), float(logits_soft_cap), _stream(stream)),
           "mla_absorbed_plan")
    max_blocks = int(max(((int(x) + block_size - 1) // block_size for x in kl), default=0))
    return AbsorbedPlan(h, num_heads, int(qo[-1]), qo.size - 1, int(block_size), max_blocks)


def mla_absorbed_run(plan: AbsorbedPlan, q_abs, cache, block_table, o=None, lse=None, return_lse=True, stream=None):
    """Run an absorbed plan: q_abs [T, H, 576], cache [NB, BS, 576], block_table [B, M] int32
    (device) -> (o_lat [T, H, 512], lse [T, H] or None)."""
    import torch
    H, T = plan.num_heads, plan.total_q
    if tuple(q_abs.shape) != (T, H, 576):
        raise ValueError(f"q_abs must be [{T}, {H}, 576], got {tuple(q_abs.shape)}")
    if cache.dim() != 3 or cache.shape[1] != plan.block_size or cache.shape[2] != 576:
        raise ValueError(f"cache must be [num_blocks, {plan.block_size}, 576], got {tuple(cache.shape)}")
    if block_table.dim() != 2 or block_table.shape[0] != plan.batch or block_table.shape[1] < plan.max_kv_blocks:
        raise ValueError(f"block_table must be [{plan.batch}, >= {plan.max_kv_blocks}], got {tuple(block_table.shape)}")
    if o is None:
        o = torch.empty((T, H, 512), dtype=torch.bfloat16, device=q_abs.device)
    if return_lse and lse is None:
        lse = torch.empty((T, H), dtype=torch.float32, device=q_abs.device)
    if tuple(o.shape) != (T, H, 512) or (lse is not None and tuple(lse.shape) != (T, H)):
        raise ValueError("o/lse shapes do not match the plan")
    bf = torch.bfloat16
    _check(library().mla_absorbed_run(plan.handle, _dev(q_abs, bf, "q_abs"), _dev(cache, bf, "cache"),
                                      int(cache.shape[0]), _dev(block_table, torch.int32, "block_table"),
                                      int(block_table.shape[1]), _dev(o, bf, "o"),
                                      _dev(lse, torch.float32, "lse"), _stream(stream)),
           "mla_absorbed_run")
    return o, lse


def mla_prefill_run(plan: PrefillPlan, q, k, v, o=None, lse=None, return_lse=True, stream=None):
    """Run a plan; returns (o, lse) (lse None when not requested)."""
    import torch
    H = plan.num_heads
    if tuple(q.shape) != (plan.total_q, H, 192):
        raise ValueError(f"q must be [{plan.total_q}, {H}, 192], got {tuple(q.shape)}")
    if tuple(k.shape) != (plan.total_kv, H, 192) or tuple(v.shape) != (plan.total_kv, H, 128):
        raise ValueError("k/v shapes do not match the plan")
    if o is None:
        o = torch.empty((plan.total_q, H, 128), dtype=torch.bfloat16, device=q.device)
    if return_lse and lse is None:
        lse = torch.empty((plan.total_q, H), dtype=torch.float32, device=q.device)
    if tuple(o.shape) != (plan.total_q, H, 128) or (lse is not None and tuple(lse.shape) != (plan.total_q, H)):
        raise ValueError("o/lse shapes do not match the plan")
    bf = torch.bfloat16
    _check(library().mla_prefill_run(plan.handle, _dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"),
                                     _dev(o, bf, "o"), _dev(lse, torch.float32, "lse"), _stream(stream)),
           "mla_prefill_run")
    return o, lse


def mla_prefill_run_merge(plan: PrefillPlan, q, k, v, o, lse, stream=None):
    """Run a plan and merge the result into the partial state (o, lse) in place; returns (o, lse)."""
    import torch
    H = plan.num_heads
    if tuple(q.shape) != (plan.total_q, H, 192):
        raise ValueError(f"q must be [{plan.total_q}, {H}, 192], got {tuple(q.shape)}")
    if tuple(k.shape) != (plan.total_kv, H, 192) or tuple(v.shape) != (plan.total_kv, H, 128):
        raise ValueError("k/v shapes do not match the plan")
    if o is None or lse is None:
        raise ValueError("mla_prefill_run_merge needs the partial state o and lse")
    if tuple(o.shape) != (plan.total_q, H, 128) or tuple(lse.shape) != (plan.total_q, H):
        raise ValueError("o/lse shapes do not match the plan")
    bf = torch.bfloat16
    _check(library().mla_prefill_run_merge(plan.handle, _dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"),
                                           _dev(o, bf, "o"), _dev(lse, torch.float32, "lse"), _stream(stream)),
           "mla_prefill_run_merge")
    return o, lse


def mla_prefill_run_shared_rope(plan: PrefillPlan, q, k_nope, k_rope, v, o=None, lse=None, merge: bool = False,
                                stream=None):
    """Run a plan with K = [k_nope (per head) || k_rope (one row per key, shared by all heads)].

    k_nope [T_kv, H, 128]; k_rope: a 2-D [T_kv, 64] view whose rows may be strided (e.g.
    latent[:, 512:] of a gathered [T_kv, 576] latent).  merge=True merges into (o, lse)."""
    import torch
    H = plan.num_heads
    if tuple(q.shape) != (plan.total_q, H, 192):
        raise ValueError(f"q must be [{plan.total_q}, {H}, 192], got {tuple(q.shape)}")
    if tuple(k_nope.shape) != (plan.total_kv, H, 128) or tuple(v.shape) != (plan.total_kv, H, 128):
        raise ValueError("k_nope/v shapes do not match the plan")
    if k_rope.dim() != 2 or tuple(k_rope.shape) != (plan.total_kv, 64) or k_rope.stride(1) != 1:
        raise ValueError("k_rope must be a [T_kv, 64] view with unit column stride")
    if merge and (o is None or lse is None):
        raise ValueError("merge needs the partial state o and lse")
    if k_rope.dtype != torch.bfloat16 or not k_rope.is_cuda:
        raise TypeError("k_rope must be a bf16 CUDA tensor")
    if o is None:
        o = torch.empty((plan.total_q, H, 128), dtype=torch.bfloat16, device=q.device)
    if lse is None:
        lse = torch.empty((plan.total_q, H), dtype=torch.float32, device=q.device)
    if tuple(o.shape) != (plan.total_q, H, 128) or tuple(lse.shape) != (plan.total_q, H):
        raise ValueError("o/lse shapes do not match the plan")
    bf = torch.bfloat16
    _check(library().mla_prefill_run_shared_rope(plan.handle, _dev(q, bf, "q"), _dev(k_nope, bf, "k_nope"),
                                                 ctypes.c_void_p(k_rope.data_ptr()), int(k_rope.stride(0)),
                                                 _dev(v, bf, "v"), _dev(o, bf, "o"), _dev(lse, torch.float32, "lse"),
                                                 int(bool(merge)), _stream(stream)), "mla_prefill_run_shared_rope")
    return o, lse


def mla_prefill_status(plan: PrefillPlan) -> int:
    """Read-and-clear the plan's device status word; raises on a device-side error."""
    code = library().mla_prefill_status(plan.handle)
    _check(code, "mla_prefill_status")
    return code


def mla_plan_destroy(plan: PrefillPlan):
    plan.destroy()


def mla_plan_units_host(qo_indptr, kv_indptr, num_heads: int, causal: bool, window_left: int, num_ctas: int):
    """Host planner only: returns (units [n, 8] int32, cta_offsets [num_ctas+1] int32)."""
    qo, kv = _host_i32(qo_indptr), _host_i32(kv_indptr)
    n = ctypes.c_int64(0)
    offs = np.zeros(num_ctas + 1, dtype=np.int32)
    lib = library()
    args = (_ptr(qo), _ptr(kv), qo.size - 1, num_heads, int(bool(causal)), int(window_left), num_ctas)
    code = lib.mla_plan_units_host(*args, None, 0, _ptr(offs), ctypes.byref(n))
    if code not in (MLA_OK, -2):
        _check(code, "mla_plan_units_host")
    units = np.zeros((max(1, n.value), 8), dtype=np.int32)
    _check(lib.mla_plan_units_host(*args, _ptr(units), n.value, _ptr(offs), ctypes.byref(n)),
           "mla_plan_units_host")
    return units[:n.value], offs


# ---------------------------------------------------------------------------- gather / up-proj / merge
def mla_gather_latent(cache, block_table, cu_seq_lens, chunk_starts, total_tokens: int, out=None, status=None,
                      stream=None):
    """Copy one prefix chunk out of the paged latent cache (device tensors)."""
    import torch
    nb, bs, e = cache.shape
    if out is None:
        out = torch.empty((total_tokens, e), dtype=cache.dtype, device=cache.device)
    batch = block_table.shape[0]
    i32 = torch.int32
    _check(library().mla_gather_latent(_dev(cache, torch.bfloat16, "cache"), nb, bs, e,
                                       _dev(block_table, i32, "block_table"), block_table.shape[1],
                                       _dev(cu_seq_lens, i32, "cu_seq_lens"), _dev(chunk_starts, i32, "chunk_starts"),
                                       batch, int(total_tokens), _dev(out, torch.bfloat16, "out"),
                                       _dev(status, i32, "status"), _stream(stream)), "mla_gather_latent")
    return out


def mla_gather_latent_fp8(cache, block_table, cu_seq_lens, chunk_starts, total_tokens: int, out=None, status=None,
                          stream=None):
    """One prefix chunk out of an fp8 paged cache (uint8 [NB, BS, 648]), dequantized to
    bf16 [total_tokens, 576]."""
    import torch
    nb, bs, e = cache.shape
    t = int(total_tokens)
    if out is None:
        out = torch.empty((t, 576), dtype=torch.bfloat16, device=cache.device)
    if tuple(out.shape) != (t, 576):
        raise ValueError(f"out must be [{t}, 576]")
    batch = block_table.shape[0]
    if tuple(cu_seq_lens.shape) != (batch + 1,) or tuple(chunk_starts.shape) != (batch,):
        raise ValueError("cu_seq_lens must be [B+1] and chunk_starts [B] for a block table of B rows")
    i32 = torch.int32
    _check(library().mla_gather_latent_fp8(_dev(cache, torch.uint8, "cache"), nb, bs, e,
                                           _dev(block_table, i32, "block_table"), block_table.shape[1],
                                           _dev(cu_seq_lens, i32, "cu_seq_lens"),
                                           _dev(chunk_starts, i32, "chunk_starts"), batch, t,
                                           _dev(out, torch.bfloat16, "out"), _dev(status, i32, "status"),
                                           _stream(stream)), "mla_gather_latent_fp8")
    return out


def mla_cache_write(cache, latent, slot_mapping, status=None, stream=None):
    """Store latent [T, E] rows into the paged cache [NB, BS, E] at slot_mapping [T] (int64,
    device; negative = padding token).  Returns the cache (written in place)."""
    import torch
    nb, bs, e = cache.shape
    t = latent.shape[0]
    if latent.shape[1] != e or slot_mapping.shape[0] != t:
        raise ValueError("latent must be [T, entry_dim] and slot_mapping [T]")
    _check(library().mla_cache_write(_dev(cache, torch.bfloat16, "cache"), nb, bs, e,
                                     _dev(latent, torch.bfloat16, "latent"),
                                     _dev(slot_mapping, torch.int64, "slot_mapping"), int(t),
                                     _dev(status, torch.int32, "status"), _stream(stream)), "mla_cache_write")
    return cache


def mla_up_proj(latent, w_kvb, num_heads: int, k_out=None, v_out=None, status=None, stream=None):
    """latent [T, 576] x w_kvb [512, H*256] -> K [T, H, 192], V [T, H, 128]."""
    import torch
    t = latent.shape[0]
    if tuple(latent.shape[1:]) != (576,) or tuple(w_kvb.shape) != (512, num_heads * 256):
        raise ValueError("latent must be [T, 576] and w_kvb [512, H*256]")
    if k_out is None:
        k_out = torch.empty((t, num_heads, 192), dtype=torch.bfloat16, device=latent.device)
    if v_out is None:
        v_out = torch.empty((t, num_heads, 128), dtype=torch.bfloat16, device=latent.device)
    bf = torch.bfloat16
    _check(library().mla_up_proj(_dev(latent, bf, "latent"), _dev(w_kvb, bf, "w_kvb"), t, num_heads,
                                 _dev(k_out, bf, "k_out"), _dev(v_out, bf, "v_out"),
                                 _dev(status, torch.int32, "status"), _stream(stream)), "mla_up_proj")
    return k_out, v_out


def mla_up_proj_paged(cache, block_table, cu_seq_lens, chunk_starts, total_tokens: int, w_kvb, num_heads: int,
                      k_out=None, v_out=None, status=None, stream=None):
    """One prefix chunk decompressed straight from the paged cache [NB, BS, 576]:
    K [T, H, 192], V [T, H, 128] (T = total_tokens), as gather + up-projection would give."""
    import torch
    nb, bs, e = cache.shape
    t = int(total_tokens)
    if e != 576 or tuple(w_kvb.shape) != (512, num_heads * 256):
        raise ValueError("cache must be [NB, BS, 576] and w_kvb [512, H*256]")
    batch = block_table.shape[0]
    if tuple(cu_seq_lens.shape) != (batch + 1,) or tuple(chunk_starts.shape) != (batch,):
        raise ValueError("cu_seq_lens must be [B+1] and chunk_starts [B] for a block table of B rows")
    if k_out is None:
        k_out = torch.empty((t, num_heads, 192), dtype=torch.bfloat16, device=cache.device)
    if v_out is None:
        v_out = torch.empty((t, num_heads, 128), dtype=torch.bfloat16, device=cache.device)
    if tuple(k_out.shape) != (t, num_heads, 192) or tuple(v_out.shape) != (t, num_heads, 128):
        raise ValueError("k_out/v_out shapes do not match total_tokens and num_heads")
    bf, i32 = torch.bfloat16, torch.int32
    _check(library().mla_up_proj_paged(_dev(cache, bf, "cache"), nb, bs, e, _dev(block_table, i32, "block_table"),
                                       block_table.shape[1], _dev(cu_seq_lens, i32, "cu_seq_lens"),
                                       _dev(chunk_starts, i32, "chunk_starts"), batch, t, _dev(w_kvb, bf, "w_kvb"),
                                       num_heads, _dev(k_out, bf, "k_out"), _dev(v_out, bf, "v_out"),
                                       _dev(status, i32, "status"), _stream(stream)), "mla_up_proj_paged")
    return k_out, v_out


def mla_up_proj_paged_split(cache, block_table, cu_seq_lens, chunk_starts, total_tokens: int, w_kvb, num_heads: int,
                            k_nope_out=None, v_out=None, rope_out=None, status=None, stream=None):
    """mla_up_proj_paged with K split into K_nope [T, H, 128] and one rope row per token [T, 64]."""
    import torch
    nb, bs, e = cache.shape
    t = int(total_tokens)
    if e != 576 or tuple(w_kvb.shape) != (512, num_heads * 256):
        raise ValueError("cache must be [NB, BS, 576] and w_kvb [512, H*256]")
    batch = block_table.shape[0]
    if tuple(cu_seq_lens.shape) != (batch + 1,) or tuple(chunk_starts.shape) != (batch,):
        raise ValueError("cu_seq_lens must be [B+1] and chunk_starts [B] for a block table of B rows")
    bf, i32 = torch.bfloat16, torch.int32
    if k_nope_out is None:
        k_nope_out = torch.empty((t, num_heads, 128), dtype=bf, device=cache.device)
    if v_out is None:
        v_out = torch.empty((t, num_heads, 128), dtype=bf, device=cache.device)
    if rope_out is None:
        rope_out = torch.empty((t, 64), dtype=bf, device=cache.device)
    if (tuple(k_nope_out.shape) != (t, num_heads, 128) or tuple(v_out.shape) != (t, num_heads, 128)
            or tuple(rope_out.shape) != (t, 64)):
        raise ValueError("k_nope_out/v_out/rope_out shapes do not match total_tokens and num_heads")
    _check(library().mla_up_proj_paged_split(_dev(cache, bf, "cache"), nb, bs, e, _dev(block_table, i32, "block_table"),
                                             block_table.shape[1], _dev(cu_seq_lens, i32, "cu_seq_lens"),
                                             _dev(chunk_starts, i32, "chunk_starts"), batch, t,
                                             _dev(w_kvb, bf, "w_kvb"), num_heads, _dev(k_nope_out, bf, "k_nope_out"),
                                             _dev(v_out, bf, "v_out"), _dev(rope_out, bf, "rope_out"),
                                             _dev(status, i32, "status"), _stream(stream)), "mla_up_proj_paged_split")
    return k_nope_out, v_out, rope_out


def mla_merge_state(o_a, lse_a, o_b, lse_b, o_out=None, lse_out=None, stream=None):
    """Merge two partial states by LSE; o_out/lse_out may be o_a/lse_a (in place)."""
    import torch
    rows, h, d = o_a.shape
    if tuple(o_b.shape) != (rows, h, d):
        raise ValueError(f"o_b must be {(rows, h, d)} like o_a, got {tuple(o_b.shape)}")
    if tuple(lse_a.shape) != (rows, h) or tuple(lse_b.shape) != (rows, h):
        raise ValueError(f"lse_a and lse_b must be {(rows, h)}")
    if o_out is not None and tuple(o_out.shape) != (rows, h, d):
        raise ValueError(f"o_out must be {(rows, h, d)}")
    if lse_out is not None and tuple(lse_out.shape) != (rows, h):
        raise ValueError(f"lse_out must be {(rows, h)}")
    if o_out is None:
        o_out = torch.empty_like(o_a)
    if lse_out is None:
        lse_out = torch.empty_like(lse_a)
    bf, f32 = torch.bfloat16, torch.float32
    _check(library().mla_merge_state(_dev(o_a, bf, "o_a"), _dev(lse_a, f32, "lse_a"), _dev(o_b, bf, "o_b"),
                                     _dev(lse_b, f32, "lse_b"), _dev(o_out, bf, "o_out"),
                                     _dev(lse_out, f32, "lse_out"), rows, h, d, _stream(stream)),
           "mla_merge_state")
    return o_out, lse_out


def mla_prefill_run_noalloc(qo_indptr, kv_indptr, num_heads: int, q, k, v, o, lse=None, *, causal: bool = True,
                            sm_scale: float, window_left: int = -1, logits_soft_cap: float = 0.0, status=None,
                            stream=None):
    """Plan + run without any device allocation by the library (outputs are caller-provided).

    For callers that cannot allocate device memory; the work list goes into a fixed
    array inside the library, so overlapping calls must be serialised by the caller."""
    import torch
    qo, kv = _host_i32(qo_indptr), _host_i32(kv_indptr)
    if qo.ndim != 1 or kv.shape != qo.shape or qo.size < 1:
        raise ValueError("qo_indptr and kv_indptr must be 1-D of equal length batch+1")
    total_q, total_kv = int(qo[-1]), int(kv[-1])
    H = int(num_heads)
    for t, shape, name in ((q, (total_q, H, 192), "q"), (k, (total_kv, H, 192), "k"), (v, (total_kv, H, 128), "v"),
                           (o, (total_q, H, 128), "o")):
        if t is None or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be {list(shape)}, got {None if t is None else tuple(t.shape)}")
    if lse is not None and tuple(lse.shape) != (total_q, H):
        raise ValueError(f"lse must be [{total_q}, {H}], got {tuple(lse.shape)}")
    if status is not None and status.numel() < 1:
        raise ValueError("status must hold at least one int32 word")
    bf = torch.bfloat16
    _check(library().mla_prefill_run_noalloc(
        _ptr(qo), _ptr(kv), qo.size - 1, num_heads, 192, 128, int(bool(causal)), float(sm_scale), int(window_left),
        float(logits_soft_cap), _dev(q, bf, "q"), _dev(k, bf, "k"), _dev(v, bf, "v"), _dev(o, bf, "o"),
        _dev(lse, torch.float32, "lse"), _dev(status, torch.int32, "status"), _stream(stream)),
        "mla_prefill_run_noalloc")
    return o, lse


# ---------------------------------------------------------------------------- speculative decoding
# These calls are made once per step or layer on a few rows, so the time to make them counts
# (about 2 us of launch each): one look per tensor, the raw current stream, no context manager
# unless a stream is given.
def _bad_tensor(t, dtype, dev, name):
    import torch
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, the current device is cuda:{dev}")
    raise ValueError(f"{name} must be contiguous")


def _arg(t, dtype, dev, name, shape=None):
    """Address of a contiguous tensor of this type (and shape) on the current device; None for None."""
    if t is None:
        return None
    try:
        ok = t.dtype is dtype and t.get_device() == dev and dev >= 0 and t.is_contiguous()
    except AttributeError:
        ok = False
    if not ok:
        _bad_tensor(t, dtype, dev, name)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _status_arg(t, dtype, dev):
    """Address of a status word; one without an element would pass for none."""
    if t is None:
        return None
    at = _arg(t, dtype, dev, "status")
    if t.numel() == 0:
        raise ValueError("status must have an element")
    return at


class _Torch:
    """What these calls use of torch, looked up once (the module is imported by the first call)."""

    def __init__(self):
        import torch
        self.int32, self.int64, self.uint8 = torch.int32, torch.int64, torch.uint8
        self.bf16, self.f32 = torch.bfloat16, torch.float32
        self.empty, self.out_of_memory = torch.empty, torch.OutOfMemoryError
        self.device, self.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


_torch_parts = None


def _here(stream, t, name):
    """(torch parts, current device, stream object or None, its handle); t: a tensor without
    which the call means nothing."""
    global _torch_parts
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    T = _torch_parts
    if T is None:
        T = _torch_parts = _Torch()
    dev = T.device()
    if stream is None:
        return T, dev, None, T.raw_stream(dev)
    if not hasattr(stream, "cuda_stream"):
        import torch
        stream = torch.cuda.ExternalStream(int(stream))
    elif stream.device.index != dev:
        raise ValueError(f"stream is on cuda:{stream.device.index}, the current device is cuda:{dev}")
    return T, dev, stream, stream.cuda_stream


def _new(T, shape, dtype, device, stream):
    """Memory in the order of the stream that the kernels are launched on."""
    if stream is None:
        return T.empty(shape, dtype=dtype, device=device)
    import torch
    with torch.cuda.stream(stream):
        return T.empty(shape, dtype=dtype, device=device)


def mla_block_table_update(seq_lens, new_lens, block_table, num_held, free_blocks, free_count, block_size: int,
                           num_tokens: int = 0, qo_indptr=None, kv_lens=None, slot_mapping=None, status=None,
                           stream=None):
    """Fit block_table [B, M] to seq_lens + new_lens [B] (device int32), taking blocks from and
    giving them back to the stack free_blocks / free_count; block_table, num_held, free_blocks
    and free_count are updated in place.  Returns (qo_indptr [B+1], kv_lens [B], slot_mapping
    [num_tokens] int64), the new tokens' prefix sums, the lengths with them, and their slots."""
    T, dev, st, handle = _here(stream, block_table, "block_table")
    int32, int64 = T.int32, T.int64
    if seq_lens.dim() != 1 or block_table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("seq_lens must be [B], block_table [B, M] and free_blocks [N]")
    b, n, m = seq_lens.shape[0], int(num_tokens), block_table.shape[1]
    device = block_table.device
    if qo_indptr is None:
        qo_indptr = _new(T, (b + 1,), int32, device, st)
    if kv_lens is None:
        kv_lens = _new(T, (b,), int32, device, st)
    if slot_mapping is None:
        slot_mapping = _new(T, (n,), int64, device, st)
    _check((_lib or library()).mla_block_table_update(
        _arg(seq_lens, int32, dev, "seq_lens"), _arg(new_lens, int32, dev, "new_lens", (b,)), b, int(block_size),
        _arg(block_table, int32, dev, "block_table", (b, m)), m, _arg(num_held, int32, dev, "num_held", (b,)),
        _arg(free_blocks, int32, dev, "free_blocks"), free_blocks.shape[0],
        _arg(free_count, int32, dev, "free_count", (1,)), _arg(qo_indptr, int32, dev, "qo_indptr", (b + 1,)),
        _arg(kv_lens, int32, dev, "kv_lens", (b,)), _arg(slot_mapping, int64, dev, "slot_mapping", (n,)), n,
        _status_arg(status, int32, dev), handle), "mla_block_table_update")
    return qo_indptr, kv_lens, slot_mapping


def mla_tree_mask(parents, qo_indptr, mask_words: int, kv_lens=None, mask=None, positions=None, status=None,
                  stream=None):
    """Trees given by parents [T] (node indices inside the request, -1: child of the context)
    -> (mask [T, mask_words] int64 of visibility bits, positions [T] int32: depth, plus the
    context length when kv_lens is given)."""
    T, dev, st, handle = _here(stream, parents, "parents")
    int32, int64 = T.int32, T.int64
    w = int(mask_words)
    if parents.dim() != 1 or qo_indptr.dim() != 1 or qo_indptr.shape[0] < 1 or w < 1:
        raise ValueError("parents must be [T], qo_indptr [B+1] and mask_words at least 1")
    t, b = parents.shape[0], qo_indptr.shape[0] - 1
    if mask is None:
        mask = _new(T, (t, w), int64, parents.device, st)
    if positions is None:
        positions = _new(T, (t,), int32, parents.device, st)
    _check((_lib or library()).mla_tree_mask(
        _arg(parents, int32, dev, "parents"), _arg(qo_indptr, int32, dev, "qo_indptr"),
        _arg(kv_lens, int32, dev, "kv_lens", (b,)), b, t, w, _arg(mask, int64, dev, "mask", (t, w)),
        _arg(positions, int32, dev, "positions", (t,)), _status_arg(status, int32, dev), handle), "mla_tree_mask")
    return mask, positions


_workspace_bytes: dict = {}   # device index -> bytes (a fact of the device)


def mla_tree_workspace(total_rows: int, num_heads: int) -> int:
    """Bytes of workspace that mla_tree_attention needs on the current device."""
    n = ctypes.c_int64(0)
    _check(library().mla_tree_workspace(int(total_rows), int(num_heads), ctypes.byref(n)), "mla_tree_workspace")
    return int(n.value)


def mla_tree_workspace_fp4(total_rows: int, num_heads: int, batch: int, num_blocks: int, block_size: int) -> int:
    """Bytes of workspace with which mla_tree_attention_fp4 is fastest on the current device (it does
    with those of mla_tree_workspace): with many pairs a request, room for the cache's rows in bf16."""
    n = ctypes.c_int64()
    _check((_lib or library()).mla_tree_workspace_fp4(int(total_rows), int(num_heads), int(batch), int(num_blocks),
                                                      int(block_size), ctypes.byref(n)), "mla_tree_workspace_fp4")
    return n.value


def _tree_attention(name, kind, width, q_abs, cache, block_table, qo_indptr, kv_lens, tree_mask, sm_scale,
                    logits_soft_cap, o, lse, return_lse, workspace, status, stream):
    T, dev, st, handle = _here(stream, q_abs, "q_abs")
    int32, bfloat16, float32, uint8 = T.int32, T.bf16, T.f32, T.uint8
    if q_abs.dim() != 3 or q_abs.shape[2] != 576 or cache.dim() != 3 or cache.shape[2] != width:
        raise ValueError(f"q_abs must be [T, H, 576] and cache [NB, BS, {width}]")
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, M]")
    t, h, _ = q_abs.shape
    b, m = block_table.shape
    words = 0
    if tree_mask is not None:
        if tree_mask.dim() != 2 or tree_mask.shape[0] != t or tree_mask.shape[1] < 1:
            raise ValueError(f"tree_mask must be [{t}, words], got {list(tree_mask.shape)}")
        words = tree_mask.shape[1]
    device = q_abs.device
    if o is None:
        o = _new(T, (t, h, 512), bfloat16, device, st)
    if return_lse and lse is None:
        lse = _new(T, (t, h), float32, device, st)
    if workspace is None:
        n = _workspace_bytes.get(dev)
        if n is None:
            n = _workspace_bytes[dev] = mla_tree_workspace(t, h)
        if kind == "uint8" and t * h > 128 * b:   # (for fewer it is the same)
            try:
                workspace = _new(T, (mla_tree_workspace_fp4(t, h, b, cache.shape[0], cache.shape[1]),), uint8, device, st)
            except T.out_of_memory:   # the rows in bf16 are 2.9 times the cache: without room for them the call is slower
                pass
        if workspace is None:
            workspace = _new(T, (n,), uint8, device, st)
    _check(getattr(_lib or library(), name)(
        _arg(q_abs, bfloat16, dev, "q_abs"), _arg(cache, getattr(T, kind), dev, "cache"), cache.shape[0], cache.shape[1],
        _arg(block_table, int32, dev, "block_table"), m, _arg(qo_indptr, int32, dev, "qo_indptr", (b + 1,)),
        _arg(kv_lens, int32, dev, "kv_lens", (b,)), _arg(tree_mask, T.int64, dev, "tree_mask"), words, b, t, h,
        float(sm_scale), float(logits_soft_cap), _arg(o, bfloat16, dev, "o", (t, h, 512)),
        _arg(lse, float32, dev, "lse", (t, h)), _arg(workspace, uint8, dev, "workspace"), workspace.numel(),
        _status_arg(status, int32, dev), handle), name)
    return o, lse


def mla_tree_attention(q_abs, cache, block_table, qo_indptr, kv_lens, tree_mask=None, *, sm_scale: float,
                       logits_soft_cap: float = 0.0, o=None, lse=None, return_lse: bool = True, workspace=None,
                       status=None, stream=None):
    """Drafted nodes (or single new tokens) over the paged latent cache: q_abs [T, H, 576],
    cache [NB, BS, 576] bf16, block_table [B, M], qo_indptr [B+1], kv_lens [B] int32 (all on the
    device), tree_mask [T, W] int64 from mla_tree_mask (None: each node sees those before it)
    -> (o_lat [T, H, 512] bf16, lse [T, H] fp32 or None).  The workspace (uint8) is allocated
    for the call when not given; one that is given must not serve two calls at a time."""
    return _tree_attention("mla_tree_attention", "bf16", 576, q_abs, cache, block_table, qo_indptr, kv_lens, tree_mask,
                           sm_scale, logits_soft_cap, o, lse, return_lse, workspace, status, stream)


def mla_tree_attention_fp4(q_abs, cache, block_table, qo_indptr, kv_lens, tree_mask=None, *, sm_scale: float,
                           logits_soft_cap: float = 0.0, o=None, lse=None, return_lse: bool = True, workspace=None,
                           status=None, stream=None):
    """mla_tree_attention over a cache of 4-bit entries, uint8 [NB, BS, 400]; the rest as there.  With many
    pairs a request the workspace that is allocated has room for the cache's rows in bf16 (see
    mla_tree_workspace_fp4) unless memory is short; one of mla_tree_workspace bytes may be given instead."""
    return _tree_attention("mla_tree_attention_fp4", "uint8", 400, q_abs, cache, block_table, qo_indptr, kv_lens,
                           tree_mask, sm_scale, logits_soft_cap, o, lse, return_lse, workspace, status, stream)


def mla_tree_verify(target_probs, tokens, qo_indptr, uniforms, final_uniforms, max_accepted: int, parents=None,
                    draft_probs=None, accepted=None, accepted_counts=None, next_tokens=None, status=None, stream=None):
    """Which drafted nodes are kept: target_probs [T, V] (fp32 or bf16) after each node, tokens [T],
    parents [T] (None: chains), qo_indptr [B+1] int32, uniforms [T] and final_uniforms [B] fp32 in
    [0, 1), draft_probs [T, V] like target_probs if the nodes were drawn from them (None: given)
    -> (accepted [B, max_accepted] int32, -1 behind each path, accepted_counts [B], next_tokens [B])."""
    T, dev, st, handle = _here(stream, target_probs, "target_probs")
    int32, f32 = T.int32, T.f32
    if target_probs.dim() != 2 or tokens.dim() != 1 or final_uniforms.dim() != 1:
        raise ValueError("target_probs must be [T, V], tokens [T] and final_uniforms [B]")
    t, vocab = target_probs.shape
    b, n, device, kind = final_uniforms.shape[0], int(max_accepted), target_probs.device, target_probs.dtype
    if kind is not f32 and kind is not T.bf16:
        raise TypeError(f"target_probs must be torch.float32 or torch.bfloat16, got {kind}")
    if n < 1:
        raise ValueError("max_accepted must be at least 1")
    if accepted is None:
        accepted = _new(T, (b, n), int32, device, st)
    if accepted_counts is None:
        accepted_counts = _new(T, (b,), int32, device, st)
    if next_tokens is None:
        next_tokens = _new(T, (b,), int32, device, st)
    _check((_lib or library()).mla_tree_verify(
        _arg(target_probs, kind, dev, "target_probs"), _arg(draft_probs, kind, dev, "draft_probs", (t, vocab)),
        0 if kind is f32 else 1, vocab, _arg(tokens, int32, dev, "tokens", (t,)), _arg(parents, int32, dev, "parents", (t,)),
        _arg(qo_indptr, int32, dev, "qo_indptr", (b + 1,)), b, t, _arg(uniforms, f32, dev, "uniforms", (t,)),
        _arg(final_uniforms, f32, dev, "final_uniforms"), _arg(accepted, int32, dev, "accepted", (b, n)), n,
        _arg(accepted_counts, int32, dev, "accepted_counts", (b,)), _arg(next_tokens, int32, dev, "next_tokens", (b,)),
        _status_arg(status, int32, dev), handle), "mla_tree_verify")
    return accepted, accepted_counts, next_tokens


def mla_tree_commit(cache, block_table, seq_lens, accepted, accepted_counts, status=None, stream=None):
    """Move the rows of accepted nodes (accepted [B, A] int32, the first accepted_counts[r] of a
    row, strictly increasing) from position seq_lens[r] + node to seq_lens[r] + i, in cache
    [NB, BS, E] or, all layers at once, [L, NB, BS, E].  Returns the cache (written in place)."""
    T, dev, _, handle = _here(stream, cache, "cache")
    int32, bfloat16 = T.int32, T.bf16
    if cache.dim() not in (3, 4) or block_table.dim() != 2 or accepted.dim() != 2:
        raise ValueError("cache must be [NB, BS, E] or [L, NB, BS, E], block_table [B, M], accepted [B, A]")
    layers = cache.shape[0] if cache.dim() == 4 else 1
    nb, bs, e = cache.shape[-3:]
    b, m = block_table.shape
    a = accepted.shape[1]
    _check((_lib or library()).mla_tree_commit(
        _arg(cache, bfloat16, dev, "cache"), layers, nb * bs * e, nb, bs, e,
        _arg(block_table, int32, dev, "block_table"), m, _arg(seq_lens, int32, dev, "seq_lens", (b,)),
        _arg(accepted, int32, dev, "accepted", (b, a)), _arg(accepted_counts, int32, dev, "accepted_counts", (b,)),
        b, a, _status_arg(status, int32, dev), handle), "mla_tree_commit")
    return cache


# ---------------------------------------------------------------------------- entries of several formats
def _view(t, dtype, dev, name):
    """Address of a tensor whose last dimension is contiguous, on the current device."""
    try:
        ok = t.dtype is dtype and t.get_device() == dev and dev >= 0
    except AttributeError:
        ok = False
    if not ok:
        _bad_tensor(t, dtype, dev, name)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    return t.data_ptr()


def mla_cache_append(cache, latent, slot_mapping, positions, cos_sin, norm_weight=None, norm_eps: float = 1e-6,
                     interleaved: bool = True, q_rope=None, q_out=None, status=None, stream=None):
    """New tokens into the paged cache, [NB, BS, 576] bf16, [NB, BS, 648] uint8 (fp8) or [NB, BS, 400]
    uint8 (fp4): latent [T, 576] bf16 (rows may be strided, its rope not rotated), slot_mapping [T]
    int64 (negative: padding), positions [T] int32, cos_sin [P, 64] fp32 (32 cosines, 32 sines),
    norm_weight [512] bf16 or None.  q_rope [T, H, 64] bf16 (a strided view, e.g. q[..., 128:]) is
    rotated into q_out (another view, e.g. q_abs[..., 512:]; None: in place).  Returns the cache."""
    T, dev, _, handle = _here(stream, cache, "cache")
    bf16 = T.bf16
    if cache.dim() != 3 or latent.dim() != 2 or latent.shape[1] != 576 or cos_sin.dim() != 2:
        raise ValueError("cache must be [NB, BS, E], latent [T, 576] and cos_sin [P, 64]")
    nb, bs, e = cache.shape
    if cache.dtype is bf16:
        entry = 0 if e == 576 else None
    else:
        entry = {648: 1, 400: 2}.get(e)
    if entry is None:
        raise ValueError("cache must be [NB, BS, 576] bf16 or [NB, BS, 648 or 400] uint8")
    t = latent.shape[0]
    h, q = 0, (None, 0, 0, 0, None, 0, 0)
    if q_rope is not None:
        if q_out is None:
            q_out = q_rope
        if q_rope.dim() != 3 or q_rope.shape[0] != t or q_rope.shape[2] != 64 or q_out.shape != q_rope.shape:
            raise ValueError(f"q_rope and q_out must be [{t}, H, 64]")
        h = q_rope.shape[1]
        if h and t:
            # (torch gives a dimension of one element any stride)
            at = lambda x: (x.stride(0) if t > 1 else 64 * h, x.stride(1) if h > 1 else 64)  # noqa: E731
            q = (_view(q_rope, bf16, dev, "q_rope"), *at(q_rope), h, _view(q_out, bf16, dev, "q_out"), *at(q_out))
    elif q_out is not None:
        raise ValueError("q_out without q_rope")
    _check((_lib or library()).mla_cache_append(
        _arg(cache, bf16 if entry == 0 else T.uint8, dev, "cache"), entry, nb, bs, _view(latent, bf16, dev, "latent"),
        latent.stride(0) if t > 1 else 576, _arg(norm_weight, bf16, dev, "norm_weight", (512,)), float(norm_eps),
        _arg(positions, T.int32, dev, "positions", (t,)), _arg(cos_sin, T.f32, dev, "cos_sin", (cos_sin.shape[0], 64)),
        cos_sin.shape[0], int(bool(interleaved)), _arg(slot_mapping, T.int64, dev, "slot_mapping", (t,)), t, *q,
        _status_arg(status, T.int32, dev), handle), "mla_cache_append")
    return cache


def mla_gather_latent_fp4(cache, block_table, cu_seq_lens, chunk_starts, total_tokens: int, out=None, status=None,
                          stream=None):
    """One prefix chunk out of a 4-bit paged cache (uint8 [NB, BS, 400]), dequantized to
    bf16 [total_tokens, 576]."""
    T, dev, st, handle = _here(stream, cache, "cache")
    if cache.dim() != 3 or cache.shape[2] != 400 or block_table.dim() != 2:
        raise ValueError("cache must be [NB, BS, 400] and block_table [B, M]")
    nb, bs, e = cache.shape
    t, (batch, width) = int(total_tokens), block_table.shape
    if out is None:
        out = _new(T, (t, 576), T.bf16, cache.device, st)
    i32 = T.int32
    _check((_lib or library()).mla_gather_latent_fp4(
        _arg(cache, T.uint8, dev, "cache"), nb, bs, e, _arg(block_table, i32, dev, "block_table"), width,
        _arg(cu_seq_lens, i32, dev, "cu_seq_lens", (batch + 1,)), _arg(chunk_starts, i32, dev, "chunk_starts", (batch,)),
        batch, t, _arg(out, T.bf16, dev, "out", (t, 576)), _status_arg(status, i32, dev), handle),
        "mla_gather_latent_fp4")
    return out
