"""ctypes binding of libkvsel (include/kvsel.h): same entry-point names, argument
marshalling only.  Device buffers are torch CUDA tensors (torch is the allocator and
the stream provider); every step of the computation runs in libkvsel's kernels.

There is no fallback: if the shared library is missing or fails to load, every call
raises ``KvselUnavailable``.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libkvsel.so")

KVSEL_OK = 0
KVSEL_EINVAL = -1
KVSEL_EBUDGET = -2
KVSEL_EUNSUPPORTED = -3
KVSEL_EWORKSPACE = -4
KVSEL_ECUDA = -5
KVSEL_ETIMEOUT = -6
KVSEL_EDEVICE = -7

REDUCE = {"sum": 0, "mean": 1, "max": 2, "max_logit": 3}
POOL = {"none": 0, "max": 1, "avg": 2}
BUDGET = {"head": 0, "layer": 1, "anchor": 2}
WO_MODE = {"group_sum": 0, "per_head": 1}
VALUE_NORM = {"l1": 0, "l2": 1}
VERIFY = {"sampled": 0, "point": 1, "greedy": 2}
DTYPE = {"fp32": 0, "bf16": 1}
ROPE_LAYOUT = {"half": 0, "interleaved": 1}
ROPE_DIRECTION = {"forward": 0, "transpose": 1, "inverse": 2}
ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}
LAYOUT_CONTIGUOUS, LAYOUT_PAGED, LAYOUT_PACKED = 0, 1, 2
MAX_BATCH = 128

EXPORTS = ("kvsel_workspace_size", "kvsel_output_size", "kvsel_workspace_init", "kvsel_score",
           "kvsel_select", "kvsel_compact", "kvsel_partition", "kvsel_run_layer", "kvsel_get_device_status",
           "kvsel_set_stage_events", "kvsel_strerror", "kvsel_version",
           "kvsel_score_noalloc", "kvsel_launch_count", "kvsel_head_scores", "kvsel_anchor_project",
           "kvsel_run_anchors", "kvsel_perturbation_workspace_size", "kvsel_perturbation",
           "kvsel_query_agnostic_split", "kvsel_prepared_w_o_size", "kvsel_prepare_w_o",
           "kvsel_attend_workspace_size", "kvsel_attend", "kvsel_evict_append_workspace_size",
           "kvsel_evict_append", "kvsel_compact_in_place", "kvsel_tree_masks", "kvsel_attend_tree_workspace_size",
           "kvsel_attend_tree", "kvsel_verify_workspace_size", "kvsel_verify", "kvsel_pages_workspace_size",
           "kvsel_pages_fork", "kvsel_pages_reserve", "kvsel_pages_trim", "kvsel_pages_accept", "kvsel_rope_table",
           "kvsel_rope", "kvsel_rope_cache")
NOALLOC_SCRATCH_BYTES = 16 << 20
STAGES = ("rowstats", "keysum", "wbar", "vnorm", "finalize", "select", "compact", "project", "perturb")


class KvselUnavailable(RuntimeError):
    pass


class KvselError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {strerror(code)} ({code})")


class kvsel_params(ctypes.Structure):
    _fields_ = [
        ("h_kv", ctypes.c_int32), ("group", ctypes.c_int32), ("head_dim", ctypes.c_int32),
        ("d_model", ctypes.c_int32), ("n_ctx", ctypes.c_int32), ("window", ctypes.c_int32),
        ("q_chunk", ctypes.c_int32), ("causal", ctypes.c_int32), ("scale", ctypes.c_float),
        ("reduce", ctypes.c_int32), ("pool", ctypes.c_int32), ("pool_kernel", ctypes.c_int32),
        ("value_aware", ctypes.c_int32), ("wo_mode", ctypes.c_int32), ("eps", ctypes.c_float),
        ("alpha", ctypes.c_float), ("n_sink", ctypes.c_int32), ("n_recent", ctypes.c_int32),
        ("budget_mode", ctypes.c_int32), ("budget_ratio", ctypes.c_double),
        ("floor_ratio", ctypes.c_double), ("batch", ctypes.c_int32),
        ("n_ctx_per_req", ctypes.POINTER(ctypes.c_int32)), ("value_norm", ctypes.c_int32),
        ("w_o_prepared", ctypes.c_int32), ("wait_cycles", ctypes.c_uint64), ("sm_budget", ctypes.c_int32),
        ("concurrent", ctypes.c_int32),
    ]


class kvsel_kv(ctypes.Structure):
    _fields_ = [
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("layout", ctypes.c_int32),
        ("stride_req", ctypes.c_int64), ("stride_head", ctypes.c_int64), ("stride_tok", ctypes.c_int64),
        ("block_table", ctypes.c_void_p), ("block_size", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32), ("num_blocks", ctypes.c_int32),
    ]


class _RowParams(ctypes.Structure):
    """Parameters that describe tensors of bf16 rows.  rows: what those tensors have to be (_rows), worked out
    by the first call with the present values."""
    rows = None

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name != "rows":
            self.rows = None


class kvsel_attn_params(_RowParams):
    _fields_ = [
        ("h_kv", ctypes.c_int32), ("group", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("batch", ctypes.c_int32),
        ("n_new", ctypes.c_int32), ("max_len", ctypes.c_int32), ("causal", ctypes.c_int32), ("window", ctypes.c_int32),
        ("n_sink", ctypes.c_int32), ("scale", ctypes.c_float), ("lens_per_head", ctypes.c_int32),
        ("q_stride_req", ctypes.c_int64), ("q_stride_head", ctypes.c_int64), ("q_stride_tok", ctypes.c_int64),
        ("o_stride_req", ctypes.c_int64), ("o_stride_head", ctypes.c_int64), ("o_stride_tok", ctypes.c_int64),
        ("n_rows", ctypes.c_int64), ("acc_stride", ctypes.c_int64), ("wait_cycles", ctypes.c_uint64),
        ("tree_window", ctypes.c_int32),
    ]


class kvsel_evict_params(_RowParams):
    _fields_ = [
        ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("batch", ctypes.c_int32), ("n_new", ctypes.c_int32),
        ("capacity", ctypes.c_int32), ("budget", ctypes.c_int32), ("n_sink", ctypes.c_int32),
        ("n_recent", ctypes.c_int32),
        ("new_stride_req", ctypes.c_int64), ("new_stride_head", ctypes.c_int64), ("new_stride_tok", ctypes.c_int64),
    ]


class kvsel_verify_params(_RowParams):
    _fields_ = [
        ("batch", ctypes.c_int32), ("n_new", ctypes.c_int32), ("vocab", ctypes.c_int32), ("mode", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("stride_req", ctypes.c_int64), ("stride_node", ctypes.c_int64),
        ("wait_cycles", ctypes.c_uint64),
    ]


class kvsel_pages_params(_RowParams):
    _fields_ = [
        ("h_kv", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("batch", ctypes.c_int32), ("block_size", ctypes.c_int32),
        ("max_blocks", ctypes.c_int32), ("num_blocks", ctypes.c_int32), ("layers", ctypes.c_int32),
        ("n_new", ctypes.c_int32), ("lens_per_head", ctypes.c_int32), ("stride_layer", ctypes.c_int64),
    ]


class kvsel_rope_params(ctypes.Structure):
    _fields_ = [
        ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("direction", ctypes.c_int32), ("scaling", ctypes.c_int32),
        ("orig_len", ctypes.c_int32), ("theta", ctypes.c_double), ("factor", ctypes.c_double),
        ("beta_fast", ctypes.c_double), ("beta_slow", ctypes.c_double), ("low_freq", ctypes.c_double),
        ("high_freq", ctypes.c_double), ("value_scale", ctypes.c_double),
    ]


class kvsel_rope_angles(ctypes.Structure):
    _fields_ = [
        ("turns", ctypes.c_uint64 * 64), ("rot_dim", ctypes.c_int32), ("layout", ctypes.c_int32), ("scale", ctypes.c_float),
        ("back", ctypes.c_int32),
    ]


class kvsel_rope_rows(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("n_tok", ctypes.c_int32), ("heads", ctypes.c_int32), ("k_heads", ctypes.c_int32)] + [
        (f"{t}_{s}", ctypes.c_int64) for t in ("q", "qo", "k", "ko") for s in ("req", "head", "tok")] + [
        ("pos_req", ctypes.c_int64)]


class kvsel_rope_cache_params(ctypes.Structure):
    _fields_ = [
        ("h_kv", ctypes.c_int32), ("batch", ctypes.c_int32), ("max_len", ctypes.c_int32), ("lens_per_head", ctypes.c_int32),
        ("pos_stride", ctypes.c_int64), ("o_req", ctypes.c_int64), ("o_head", ctypes.c_int64), ("o_tok", ctypes.c_int64),
    ]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libkvsel.so (built by __graft_entry__.build()); raise if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise KvselUnavailable(f"libkvsel.so not built ({p}); run __graft_entry__.build()")
    try:
        lib = ctypes.CDLL(p)
    except OSError as e:  # pragma: no cover - depends on the machine
        raise KvselUnavailable(f"cannot load {p}: {e}") from e
    P, K = ctypes.POINTER(kvsel_params), ctypes.POINTER(kvsel_kv)
    PA, PE = ctypes.POINTER(kvsel_attn_params), ctypes.POINTER(kvsel_evict_params)
    PV, PP = ctypes.POINTER(kvsel_verify_params), ctypes.POINTER(kvsel_pages_params)
    PR, RA, i32 = ctypes.POINTER(kvsel_rope_params), ctypes.POINTER(kvsel_rope_angles), ctypes.c_int32
    vp, sz, i64p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_int64)
    sig = {
        "kvsel_workspace_size": ([P, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_output_size": ([P, i64p, i64p, i64p], ctypes.c_int),
        "kvsel_workspace_init": ([vp, sz, vp], ctypes.c_int),
        "kvsel_score": ([P, vp, K, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvsel_select": ([P, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvsel_compact": ([P, K, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvsel_partition": ([P, K] + [vp] * 11 + [sz, vp], ctypes.c_int),
        "kvsel_run_layer": ([P, vp, K, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
        "kvsel_get_device_status": ([vp, vp, ctypes.POINTER(ctypes.c_int)], ctypes.c_int),
        "kvsel_set_stage_events": ([ctypes.c_void_p], None),
        "kvsel_score_noalloc": ([P, vp, K, vp, vp, vp, vp], ctypes.c_int),
        "kvsel_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "kvsel_version": ([], ctypes.c_char_p),
        "kvsel_launch_count": ([], ctypes.c_uint64),
        "kvsel_head_scores": ([P, vp, vp, vp], ctypes.c_int),
        "kvsel_prepared_w_o_size": ([P, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_prepare_w_o": ([P, vp, vp, sz, vp, sz, vp], ctypes.c_int),
        "kvsel_query_agnostic_split": ([P, ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)],
                                       ctypes.c_int),
        "kvsel_anchor_project": ([P, K] + [vp] * 10 + [sz, vp], ctypes.c_int),
        "kvsel_run_anchors": ([P, vp, K] + [vp] * 12 + [sz, vp], ctypes.c_int),
        "kvsel_attend_workspace_size": ([PA, ctypes.c_int, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_attend": ([PA, vp, K] + [vp] * 7 + [sz, vp], ctypes.c_int),
        "kvsel_evict_append_workspace_size": ([PE, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_evict_append": ([PE, K] + [vp] * 8 + [sz, vp], ctypes.c_int),
        "kvsel_compact_in_place": ([P, K] + [vp] * 8 + [ctypes.c_int64, vp, sz, vp], ctypes.c_int),
        "kvsel_tree_masks": ([vp, vp, vp, i32, i32, vp, vp, vp], ctypes.c_int),
        "kvsel_attend_tree_workspace_size": ([PA, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_attend_tree": ([PA, vp, K] + [vp] * 7 + [sz, vp], ctypes.c_int),
        "kvsel_verify_workspace_size": ([PV, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_verify": ([PV] + [vp] * 10 + [sz, vp], ctypes.c_int),
        "kvsel_pages_workspace_size": ([PP, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_pages_fork": ([PP] + [vp] * 7 + [sz, vp], ctypes.c_int),
        "kvsel_pages_reserve": ([PP] + [vp] * 8 + [sz, vp], ctypes.c_int),
        "kvsel_pages_trim": ([PP] + [vp] * 4 + [sz, vp], ctypes.c_int),
        "kvsel_pages_accept": ([PP] + [vp] * 9 + [sz, vp], ctypes.c_int),
        "kvsel_rope_table": ([PR, RA], ctypes.c_int),
        "kvsel_rope": ([RA, ctypes.POINTER(kvsel_rope_rows)] + [vp] * 7, ctypes.c_int),
        "kvsel_rope_cache": ([RA, ctypes.POINTER(kvsel_rope_cache_params), K] + [vp] * 4 + [sz, vp], ctypes.c_int),
        "kvsel_perturbation_workspace_size": ([P, ctypes.POINTER(sz)], ctypes.c_int),
        "kvsel_perturbation": ([P, vp, K, vp, vp, vp, vp, vp, vp, sz, vp], ctypes.c_int),
    }
    for name, (args, res) in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    if path is None:
        _lib = lib
    return lib


# ------------------------------------------------------------------------------ helpers
def make_params(*, h_kv: int, group: int, n_ctx: int, window: int, head_dim: int = 128,
                d_model: int = 0, q_chunk: int = 0, causal: bool = True, scale: float = 0.0,
                reduce: str = "mean", pool: str = "max", pool_kernel: int = 7,
                value_aware: bool = False, wo_mode: str = "group_sum", eps: float = 1e-4,
                alpha: float = 0.5, n_sink: int = 4, n_recent: int = 32,
                budget_mode: str = "head", budget_ratio: float = 0.2, floor_ratio: float = 0.0,
                n_ctx_per_req: Optional[Sequence[int]] = None, value_norm: str = "l1",
                wait_cycles: int = 0, w_o_prepared: bool = False, sm_budget: int = 0,
                concurrent: bool = False) -> kvsel_params:
    p = kvsel_params()
    p.h_kv, p.group, p.head_dim, p.d_model = h_kv, group, head_dim, d_model
    p.n_ctx, p.window, p.q_chunk, p.causal = n_ctx, window, q_chunk, int(bool(causal))
    p.scale = scale
    p.reduce, p.pool, p.pool_kernel = REDUCE[reduce], POOL[pool], pool_kernel
    p.value_aware, p.wo_mode, p.eps, p.alpha = int(bool(value_aware)), WO_MODE[wo_mode], eps, alpha
    p.n_sink, p.n_recent = n_sink, n_recent
    p.budget_mode, p.budget_ratio, p.floor_ratio = BUDGET[budget_mode], budget_ratio, floor_ratio
    p.value_norm = VALUE_NORM[value_norm]
    p.wait_cycles = int(wait_cycles)
    p.sm_budget = int(sm_budget)
    p.concurrent = int(bool(concurrent))
    p.w_o_prepared = int(bool(w_o_prepared))
    if n_ctx_per_req is not None:
        arr = (ctypes.c_int32 * len(n_ctx_per_req))(*[int(x) for x in n_ctx_per_req])
        p._n_arr = arr  # keep alive
        p.n_ctx_per_req = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int32))
        p.batch = len(n_ctx_per_req)
    else:
        p.batch = 1
    return p


def params_from_workload(wl, n_ctx_per_req: Optional[Sequence[int]] = None, **override) -> kvsel_params:
    kw = dict(h_kv=wl.h_kv, group=wl.group, n_ctx=wl.n_ctx, window=wl.window, head_dim=wl.head_dim,
              d_model=wl.d_model if wl.value_aware else 0, q_chunk=wl.q_chunk, causal=wl.causal,
              reduce=wl.reduce, pool=wl.pool, pool_kernel=wl.pool_kernel, value_aware=wl.value_aware,
              eps=wl.eps, alpha=wl.alpha, n_sink=wl.n_sink, n_recent=wl.n_recent,
              budget_mode=wl.budget_mode, budget_ratio=wl.budget_ratio, floor_ratio=wl.floor_ratio,
              n_ctx_per_req=n_ctx_per_req, value_norm=wl.value_norm)
    kw.update(override)
    return make_params(**kw)


def make_attn_params(*, h_kv: int, group: int, batch: int, max_len: int, n_new: int = 1, head_dim: int = 128,
                     causal: bool = True, window: int = 0, n_sink: int = 0, scale: float = 0.0,
                     lens_per_head: bool = False, q_strides: Sequence[int] = (0, 0, 0),
                     o_strides: Sequence[int] = (0, 0, 0), n_rows: int = 0, acc_stride: int = 0,
                     wait_cycles: int = 0, tree_window: bool = False) -> kvsel_attn_params:
    """q_strides / o_strides: (request, query head, token) in elements; zeros = dense
    [batch][h_kv*group][n_new][head_dim].  tree_window: the window counts a tree's own rows too."""
    return kvsel_attn_params(h_kv, group, head_dim, batch, n_new, max_len, int(bool(causal)), window, n_sink, scale,
                             int(bool(lens_per_head)), *[int(x) for x in q_strides], *[int(x) for x in o_strides],
                             n_rows, acc_stride, int(wait_cycles), int(bool(tree_window)))


def make_evict_params(*, h_kv: int, batch: int, capacity: int, budget: int, n_new: int = 1, head_dim: int = 128,
                      n_sink: int = 4, n_recent: int = 32,
                      new_strides: Sequence[int] = (0, 0, 0)) -> kvsel_evict_params:
    """new_strides: (request, KV head, token) of k_new and v_new in elements; zeros = dense
    [batch][h_kv][n_new][head_dim]."""
    return kvsel_evict_params(h_kv, head_dim, batch, n_new, capacity, budget, n_sink, n_recent,
                              *[int(x) for x in new_strides])


def make_verify_params(*, batch: int, n_new: int, vocab: int, mode: str = "sampled", dtype: str = "fp32",
                       stride_req: int = 0, stride_node: int = 0, wait_cycles: int = 0) -> kvsel_verify_params:
    """Strides of target and draft in elements; zeros = dense [batch][n_new][vocab]."""
    return kvsel_verify_params(batch, n_new, vocab, VERIFY[mode], DTYPE[dtype], stride_req, stride_node, int(wait_cycles))


def make_pages_params(*, batch: int, max_blocks: int, num_blocks: int, block_size: int, h_kv: int, layers: int = 1,
                      n_new: int = 1, head_dim: int = 128, lens_per_head: bool = False,
                      stride_layer: int = 0) -> kvsel_pages_params:
    """Pools [layers][num_blocks][block_size][h_kv][head_dim] under a table [batch][max_blocks]; stride_layer: elements
    between layers (0: dense)."""
    return kvsel_pages_params(h_kv, head_dim, batch, block_size, max_blocks, num_blocks, layers, n_new,
                              int(bool(lens_per_head)), stride_layer)


def _refuse(where: str, why: str) -> None:
    raise KvselError(KVSEL_EINVAL, f"{where}: {why}")


_BF16 = None   # torch's type, once it is loaded


def _is_bf16(t) -> bool:
    """bf16, or its bit patterns in 16-bit integers."""
    global _BF16
    if t.dtype is _BF16:
        return True
    import torch

    _BF16 = torch.bfloat16
    return t.dtype is _BF16 or (t.element_size() == 2 and not t.is_floating_point())


def _same_rows(where: str, k, v) -> None:
    """A view has one set of strides and sizes, taken from k: refuse a v that they do not describe (a v that is
    absent or a bare address is the caller's own matter)."""
    if v is None or isinstance(v, int):
        v = k
    for t in (k, v):
        if not _is_bf16(t):
            _refuse(where, f"rows of {t.dtype}, not bf16")
        if t.shape[-1] > 1 and t.stride(-1) != 1:
            _refuse(where, f"columns {t.stride(-1)} elements apart")
    if v.device != k.device or v.shape[-1] != k.shape[-1]:
        _refuse(where, f"k {tuple(k.shape)} on {k.device}, v {tuple(v.shape)} on {v.device}")
    for i in range(1, max(k.dim(), v.dim()) + 1):
        nk, nv = (t.shape[-i] if i <= t.dim() else 1 for t in (k, v))
        if nv < nk or (nk > 1 and v.stride(-i) != k.stride(-i)):
            _refuse(where, f"k {tuple(k.shape)} with strides {k.stride()}, v {tuple(v.shape)} with strides {v.stride()}")


def make_kv_contiguous(k, v, *, stride_req: int = 0) -> kvsel_kv:
    """K/V tensors [H][n][d] (one request) or [B][H][n][d] (bf16, CUDA), of the same strides."""
    if k.dim() < 3:
        _refuse("make_kv_contiguous", f"k {tuple(k.shape)}")
    _same_rows("make_kv_contiguous", k, v)
    kv = kvsel_kv()
    kv.k, kv.v = _ptr(k), _ptr(v)
    kv.layout = LAYOUT_CONTIGUOUS
    kv.stride_tok = k.stride(-2)
    kv.stride_head = k.stride(-3)
    kv.stride_req = k.stride(-4) if k.dim() == 4 else stride_req
    return kv


def make_kv_paged(k_pool, v_pool, block_table) -> kvsel_kv:
    """Pools [num_blocks][block][H][d] bf16 and block_table [B][max_blocks] int32 (CUDA), all dense."""
    _same_rows("make_kv_paged", k_pool, v_pool)
    if not k_pool.is_contiguous():   # (v_pool has its strides)
        _refuse("make_kv_paged", f"a pool with strides {k_pool.stride()}")
    t = block_table
    if t.dim() != 2 or t.element_size() != 4 or t.is_floating_point() or not t.is_contiguous():
        _refuse("make_kv_paged", f"block table {tuple(t.shape)} of {t.dtype} with strides {t.stride()}")
    kv = kvsel_kv()
    kv.k, kv.v = _ptr(k_pool), _ptr(v_pool)
    kv.layout = LAYOUT_PAGED
    kv.block_table = _ptr(block_table)
    kv.block_size = k_pool.shape[1]
    kv.max_blocks = block_table.shape[1]
    kv.num_blocks = k_pool.shape[0]
    return kv


def make_kv_packed(k, v) -> kvsel_kv:
    """Rows [n_rows][d] bf16 (CUDA) of segments placed by an offsets array, as kvsel_compact
    writes them (kvsel_attend only), of the same stride."""
    if k.dim() != 2:
        _refuse("make_kv_packed", f"k {tuple(k.shape)}")
    _same_rows("make_kv_packed", k, v)
    kv = kvsel_kv()
    kv.k, kv.v = _ptr(k), _ptr(v)
    kv.layout = LAYOUT_PACKED
    kv.stride_tok = k.stride(0)
    return kv


def _ptr(t) -> Optional[int]:
    return t if t is None or isinstance(t, int) else t.data_ptr()


def _rows(batch: int, heads: int, toks: int, req: int, head: int, tok: int):
    """Of bf16 rows [batch][heads][toks][128] with these strides (all zero: dense): their type, whether they
    are dense, and the bytes from the first element to the end of the last."""
    import torch

    if req or head or tok:
        return torch.bfloat16, False, 2 * ((batch - 1) * req + (heads - 1) * head + (toks - 1) * tok + 128)
    return torch.bfloat16, True, 256 * batch * heads * toks


def _row_ptr(t, rows, where: str) -> Optional[int]:
    """Address of a tensor that has to be as `rows` says, else refused (an address is the caller's own matter)."""
    if t is None or isinstance(t, int):
        return t
    dtype, dense, need = rows
    holds = t.is_contiguous() and t.nbytes >= need
    if not holds and not dense:
        holds = t.untyped_storage().nbytes() - 2 * t.storage_offset() >= need and t.stride()[-1] == 1
    if not holds or (t.dtype is not dtype and not _is_bf16(t)):
        _refuse(where, f"{tuple(t.shape)} of {t.dtype} with strides {t.stride()} for {need} bytes of {'dense ' * dense}rows")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _current_stream() -> int:
    """Handle of torch's current stream (the raw getter: a Stream object costs more than a launch)."""
    import torch

    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return torch.cuda.current_stream().cuda_stream
    return raw(torch.cuda.current_device())


@functools.lru_cache(maxsize=None)
def _cuda():
    """torch's getters of the current device and of a device's current stream (a handle); the raw ones cost a
    third of torch.cuda's."""
    import torch

    torch.cuda.init()
    return (getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device),
            getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream))


def _place(ws, stream, where: str) -> int:
    """Handle of the stream of a call with workspace ws.  The call runs on the current device; a workspace
    elsewhere (and what belongs to it) is refused."""
    device, current = _cuda()
    dev = device()
    if ws.get_device() != dev:
        raise KvselError(KVSEL_EINVAL, f"{where}: workspace on {ws.device}, current device cuda:{dev}")
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    return current(dev)


def _check(rc: int, where: str) -> None:
    if rc != KVSEL_OK:
        raise KvselError(rc, where)


# ------------------------------------------------------------------------------ the ABI
def strerror(code: int) -> str:
    try:
        return load().kvsel_strerror(code).decode()
    except KvselUnavailable:
        return f"error {code}"


def kvsel_version() -> str:
    return load().kvsel_version().decode()


def kvsel_strerror(code: int) -> str:
    return load().kvsel_strerror(code).decode()


def kvsel_launch_count() -> int:
    return int(load().kvsel_launch_count())


def kvsel_prepared_w_o_size(params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_prepared_w_o_size(ctypes.byref(params), ctypes.byref(out)), "kvsel_prepared_w_o_size")
    return out.value


def kvsel_prepare_w_o(params, w_o, w_prep, ws=None, stream=None) -> None:
    """The value-norm weights of W_O (W_h, or its Gram matrix for the L2 norm) into w_prep,
    once per model; scoring calls with w_o_prepared=True then take w_prep as their w_o."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().kvsel_prepare_w_o(ctypes.byref(params), _ptr(w_o), _ptr(w_prep),
                                    w_prep.numel() * w_prep.element_size(), _ptr(ws), nbytes, _stream(stream)),
           "kvsel_prepare_w_o")


def kvsel_query_agnostic_split(params) -> tuple:
    """(key blocks per head, query-row slices per key block) of query-agnostic scoring."""
    kb, rs = ctypes.c_int32(), ctypes.c_int32()
    _check(load().kvsel_query_agnostic_split(ctypes.byref(params), ctypes.byref(kb), ctypes.byref(rs)),
           "kvsel_query_agnostic_split")
    return kb.value, rs.value


def kvsel_head_scores(params, scores, head_out, stream=None) -> None:
    """head_out[b*h_kv + h] = max over the sequence of request b, head h of `scores`."""
    _check(load().kvsel_head_scores(ctypes.byref(params), _ptr(scores), _ptr(head_out), _stream(stream)),
           "kvsel_head_scores")


def kvsel_set_stage_events(events) -> None:
    """events: None, or a ctypes array of 2*len(STAGES) cudaEvent_t handles (kept alive
    by the caller while set)."""
    load().kvsel_set_stage_events(None if events is None else ctypes.cast(events, ctypes.c_void_p))


def kvsel_workspace_size(params: kvsel_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_workspace_size(ctypes.byref(params), ctypes.byref(out)), "kvsel_workspace_size")
    return out.value


def kvsel_output_size(params: kvsel_params):
    a, b, c = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int64()
    _check(load().kvsel_output_size(ctypes.byref(params), ctypes.byref(a), ctypes.byref(b), ctypes.byref(c)),
           "kvsel_output_size")
    return a.value, b.value, c.value


def kvsel_workspace_init(ws, stream=None) -> None:
    _check(load().kvsel_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "kvsel_workspace_init")


def kvsel_score(params, q, kv: kvsel_kv, w_o, s_attn, s_val, ws, stream=None) -> None:
    _check(load().kvsel_score(ctypes.byref(params), _ptr(q), ctypes.byref(kv), _ptr(w_o), _ptr(s_attn),
                              _ptr(s_val), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "kvsel_score")


def kvsel_score_noalloc(params, q, kv: kvsel_kv, w_o, s_attn, s_val, stream=None) -> None:
    """kvsel_score with the library's built-in scratch buffer instead of a workspace, for
    callers that cannot allocate device memory (see include/kvsel.h)."""
    _check(load().kvsel_score_noalloc(ctypes.byref(params), _ptr(q), ctypes.byref(kv), _ptr(w_o), _ptr(s_attn),
                                      _ptr(s_val), _stream(stream)), "kvsel_score_noalloc")


def kvsel_select(params, s_attn, s_val, idx, counts, offsets, ws=None, stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().kvsel_select(ctypes.byref(params), _ptr(s_attn), _ptr(s_val), _ptr(idx), _ptr(counts),
                               _ptr(offsets), _ptr(ws), nbytes, _stream(stream)), "kvsel_select")


def kvsel_compact(params, kv: kvsel_kv, idx, counts, offsets, k_out, v_out, ws=None, stream=None) -> None:
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().kvsel_compact(ctypes.byref(params), ctypes.byref(kv), _ptr(idx), _ptr(counts), _ptr(offsets),
                                _ptr(k_out), _ptr(v_out), _ptr(ws), nbytes, _stream(stream)), "kvsel_compact")


def kvsel_partition(params, kv: kvsel_kv, idx, counts, offsets, ev_idx, ev_counts, ev_offsets, k_ev, v_ev,
                    k_kept=None, v_kept=None, ws=None, stream=None) -> None:
    """Kept set and its complement: evicted positions and the evicted (and optionally the
    kept) K/V rows, bit-exact."""
    nbytes = 0 if ws is None else ws.numel() * ws.element_size()
    _check(load().kvsel_partition(ctypes.byref(params), ctypes.byref(kv), _ptr(idx), _ptr(counts), _ptr(offsets),
                                  _ptr(ev_idx), _ptr(ev_counts), _ptr(ev_offsets), _ptr(k_ev), _ptr(v_ev),
                                  _ptr(k_kept), _ptr(v_kept), _ptr(ws), nbytes, _stream(stream)), "kvsel_partition")


def kvsel_run_layer(params, q, kv: kvsel_kv, w_o, s_attn, s_val, idx, counts, offsets, k_out, v_out, ws,
                    stream=None) -> None:
    _check(load().kvsel_run_layer(ctypes.byref(params), _ptr(q), ctypes.byref(kv), _ptr(w_o), _ptr(s_attn),
                                  _ptr(s_val), _ptr(idx), _ptr(counts), _ptr(offsets), _ptr(k_out),
                                  _ptr(v_out), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "kvsel_run_layer")


def kvsel_anchor_project(params, kv: kvsel_kv, anchor_k, anchor_v, idx, counts, offsets, slot_k, gamma_k,
                         slot_v, gamma_v, ws, stream=None) -> None:
    _check(load().kvsel_anchor_project(ctypes.byref(params), ctypes.byref(kv), _ptr(anchor_k), _ptr(anchor_v),
                                       _ptr(idx), _ptr(counts), _ptr(offsets), _ptr(slot_k), _ptr(gamma_k),
                                       _ptr(slot_v), _ptr(gamma_v), _ptr(ws), ws.numel() * ws.element_size(),
                                       _stream(stream)), "kvsel_anchor_project")


def kvsel_run_anchors(params, q, kv: kvsel_kv, rand_keys, s_attn, idx, counts, offsets, anchor_k, anchor_v,
                      slot_k, gamma_k, slot_v, gamma_v, ws, stream=None) -> None:
    _check(load().kvsel_run_anchors(ctypes.byref(params), _ptr(q), ctypes.byref(kv), _ptr(rand_keys),
                                    _ptr(s_attn), _ptr(idx), _ptr(counts), _ptr(offsets), _ptr(anchor_k),
                                    _ptr(anchor_v), _ptr(slot_k), _ptr(gamma_k), _ptr(slot_v), _ptr(gamma_v),
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "kvsel_run_anchors")


def kvsel_perturbation_workspace_size(params: kvsel_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_perturbation_workspace_size(ctypes.byref(params), ctypes.byref(out)),
           "kvsel_perturbation_workspace_size")
    return out.value


def kvsel_perturbation(params, q, kv: kvsel_kv, w_o, idx, counts, offsets, out, ws, stream=None) -> None:
    _check(load().kvsel_perturbation(ctypes.byref(params), _ptr(q), ctypes.byref(kv), _ptr(w_o), _ptr(idx),
                                     _ptr(counts), _ptr(offsets), _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(stream)), "kvsel_perturbation")


def kvsel_attend_workspace_size(params: kvsel_attn_params, acc: bool = False) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_attend_workspace_size(ctypes.byref(params), int(bool(acc)), ctypes.byref(out)),
           "kvsel_attend_workspace_size")
    return out.value


def kvsel_attend(params: kvsel_attn_params, q, kv: kvsel_kv, lens, out, ws, new_lens=None, offsets=None, lse=None,
                 acc=None, stream=None) -> None:
    """Attention of new tokens over the cache; with acc every cached row's weight is added."""
    if params.rows is None:
        p, B, H = params, params.batch, params.h_kv * params.group
        p.rows = (_rows(B, H, p.n_new, p.q_stride_req, p.q_stride_head, p.q_stride_tok),
                  _rows(B, H, p.n_new, p.o_stride_req, p.o_stride_head, p.o_stride_tok))
    q_rows, o_rows = params.rows
    q, out = _row_ptr(q, q_rows, "kvsel_attend: q"), _row_ptr(out, o_rows, "kvsel_attend: out")
    st = _place(ws, stream, "kvsel_attend")
    rc = (_lib or load()).kvsel_attend(params, q, kv, _ptr(lens), _ptr(new_lens), _ptr(offsets), out, _ptr(lse),
                                       _ptr(acc), ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, "kvsel_attend")


def kvsel_evict_append_workspace_size(params: kvsel_evict_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_evict_append_workspace_size(ctypes.byref(params), ctypes.byref(out)),
           "kvsel_evict_append_workspace_size")
    return out.value


def kvsel_evict_append(params: kvsel_evict_params, kv: kvsel_kv, lens, seen, pos, acc, k_new, v_new, ws,
                       new_lens=None, stream=None) -> None:
    """Evict by accumulated weight until the new rows fit the budget, then append them."""
    if params.rows is None:
        p = params
        p.rows = _rows(p.batch, p.h_kv, p.n_new, p.new_stride_req, p.new_stride_head, p.new_stride_tok)
    k_new = _row_ptr(k_new, params.rows, "kvsel_evict_append: k_new")
    v_new = _row_ptr(v_new, params.rows, "kvsel_evict_append: v_new")
    st = _place(ws, stream, "kvsel_evict_append")
    rc = (_lib or load()).kvsel_evict_append(params, kv, _ptr(lens), _ptr(seen), _ptr(pos), _ptr(acc), k_new, v_new,
                                             _ptr(new_lens), ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, "kvsel_evict_append")


_INT32 = _FP32 = None   # torch's types, once it is loaded


def _int32(t, count: int, where: str) -> Optional[int]:
    """Address of a dense tensor of at least `count` 32-bit integers, else refused (an address is the caller's own
    matter)."""
    if t is None or t.__class__ is int:
        return t
    if t.dtype is _INT32 and t.numel() >= count and t.is_contiguous():
        return t.data_ptr()
    return _other_words(t, count, where, False)


def _fp32(t, count: int, where: str) -> Optional[int]:
    if t is None or t.__class__ is int:
        return t
    if t.dtype is _FP32 and t.numel() >= count and t.is_contiguous():
        return t.data_ptr()
    return _other_words(t, count, where, True)


def _other_words(t, count: int, where: str, real: bool) -> int:
    """The first tensor of its type, one of unsigned integers, or one that is refused."""
    global _INT32, _FP32
    import torch

    _INT32, _FP32 = torch.int32, torch.float32
    if t.dtype not in ((_FP32,) if real else (_INT32, torch.uint32)) or t.numel() < count or not t.is_contiguous():
        _refuse(where, f"{tuple(t.shape)} of {t.dtype} with strides {t.stride()} for {count} dense {'fp32 numbers' if real else '32-bit integers'}")
    return t.data_ptr()


def kvsel_compact_in_place(params, kv: kvsel_kv, idx, counts, offsets, lens, seen, pos, ws=None, scores=None, acc=None,
                           stream=None) -> None:
    """The kept rows of every segment become its first ones, in the cache itself; lens, seen, pos and acc as
    kvsel_evict_append goes on with them.  pos (and acc): [batch][h_kv][capacity]."""
    where, segs = "kvsel_compact_in_place", params.batch * params.h_kv
    capacity = pos.shape[-1]
    if acc is not None and acc.shape[-1] != capacity:
        _refuse(where, f"pos {tuple(pos.shape)}, acc {tuple(acc.shape)}")
    n_scores, n_kept, _ = kvsel_output_size(params)
    if offsets.element_size() != 8 or not offsets.is_contiguous() or offsets.numel() < segs:
        _refuse(where, f"offsets {tuple(offsets.shape)} of {offsets.dtype}")
    st = _place(pos, stream, where)
    _check(load().kvsel_compact_in_place(
        params, kv, _int32(idx, n_kept, where), _int32(counts, segs, where), _ptr(offsets), _fp32(scores, n_scores, where),
        _int32(lens, segs, where), _int32(seen, segs, where), _int32(pos, segs * capacity, where),
        _fp32(acc, segs * capacity, where), capacity, _ptr(ws), 0 if ws is None else ws.nbytes, st), where)


def kvsel_tree_masks(parents, tree, pos=None, first=None, new_lens=None, stream=None) -> None:
    """Masks (and positions first + depth) of trees: parents [batch][n_new] -> tree [batch][n_new][words]."""
    where = "kvsel_tree_masks"
    B, m = parents.shape
    st = _place(parents, stream, where)
    _check((_lib or load()).kvsel_tree_masks(
        _int32(parents, B * m, where), _int32(new_lens, B, where), _int32(first, B, where), B, m,
        _int32(tree, B * m * ((m + 31) // 32), where), _int32(pos, B * m, where), st), where)


def kvsel_attend_tree_workspace_size(params: kvsel_attn_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_attend_tree_workspace_size(ctypes.byref(params), ctypes.byref(out)),
           "kvsel_attend_tree_workspace_size")
    return out.value


def kvsel_attend_tree(params: kvsel_attn_params, q, kv: kvsel_kv, lens, tree, out, ws, new_lens=None, offsets=None,
                      lse=None, stream=None) -> None:
    """Attention of the nodes of a tree over the cache; tree: the masks [batch][n_new][words]."""
    if params.rows is None:
        p, B, H = params, params.batch, params.h_kv * params.group
        p.rows = (_rows(B, H, p.n_new, p.q_stride_req, p.q_stride_head, p.q_stride_tok),
                  _rows(B, H, p.n_new, p.o_stride_req, p.o_stride_head, p.o_stride_tok))
    q_rows, o_rows = params.rows
    q, out = _row_ptr(q, q_rows, "kvsel_attend_tree: q"), _row_ptr(out, o_rows, "kvsel_attend_tree: out")
    m = params.n_new
    tree = _int32(tree, params.batch * m * ((m + 31) // 32), "kvsel_attend_tree: tree")
    st = _place(ws, stream, "kvsel_attend_tree")
    rc = (_lib or load()).kvsel_attend_tree(params, q, kv, _ptr(lens), _ptr(new_lens), _ptr(offsets), tree, out, _ptr(lse),
                                            ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, "kvsel_attend_tree")


def kvsel_verify_workspace_size(params: kvsel_verify_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_verify_workspace_size(ctypes.byref(params), ctypes.byref(out)), "kvsel_verify_workspace_size")
    return out.value


def _values_of(p: kvsel_verify_params):
    """What target and draft have to be: types, elements between requests and nodes, and bytes (dense: of all)."""
    import torch

    dense = not (p.stride_req or p.stride_node)
    req, node = (p.n_new * p.vocab, p.vocab) if dense else (p.stride_req, p.stride_node)
    size = 2 if p.dtype else 4
    types = (torch.bfloat16, torch.int16, torch.uint16) if p.dtype else (torch.float32,)
    return types, dense, req, node, size * ((p.batch - 1) * req + (p.n_new - 1) * node + p.vocab), (p.batch, p.n_new, p.vocab)


def _values(t, params: kvsel_verify_params, where: str) -> Optional[int]:
    """Address of target or draft, whose type and strides have to be as the parameters say."""
    if t is None or isinstance(t, int):
        return t
    if params.rows is None:
        params.rows = _values_of(params)
    types, dense, req, node, need, shape = params.rows
    holds = t.dtype in types
    if holds and not (t.shape == shape and dense and t.is_contiguous()):
        holds = t.stride()[-1] == 1 and t.untyped_storage().nbytes() - t.element_size() * t.storage_offset() >= need
        if holds and t.dim() == 3:
            holds = all(a >= b for a, b in zip(t.shape, shape)) and (shape[0] == 1 or t.stride(0) == req) and (
                shape[1] == 1 or t.stride(1) == node)
        elif holds:                                  # rows one after another
            holds = t.is_contiguous() and t.nbytes >= need and (t.dim() == 1 or t.shape[-1] % node == 0)
    if not holds:
        _refuse(where, f"{tuple(t.shape)} of {t.dtype} with strides {t.stride()}")
    return t.data_ptr()


def kvsel_verify(params: kvsel_verify_params, tokens, parents, target, path, counts, next, ws, draft=None, u=None,
                 new_lens=None, stream=None) -> None:
    """Which drafted tokens stay (path, counts) and the token after them (next)."""
    where, B, n = "kvsel_verify", params.batch, params.batch * params.n_new
    st = _place(ws, stream, where)
    rc = (_lib or load()).kvsel_verify(
        params, _int32(tokens, n, where), _int32(parents, n, where), _values(target, params, where), _values(draft, params, where),
        _fp32(u, n, where), _int32(new_lens, B, where), _int32(path, n, where), _int32(counts, B, where), _int32(next, B, where),
        ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_pages_workspace_size(params: kvsel_pages_params) -> int:
    out = ctypes.c_size_t()
    _check(load().kvsel_pages_workspace_size(ctypes.byref(params), ctypes.byref(out)), "kvsel_pages_workspace_size")
    return out.value


def _pool(t, params: kvsel_pages_params, where: str) -> Optional[int]:
    if t.__class__ is int:
        return t
    if params.rows is None:
        p = params
        layer = p.num_blocks * p.block_size * p.h_kv * p.head_dim
        stride = p.stride_layer or layer
        params.rows = 2 * ((p.layers - 1) * stride + layer), layer, stride if p.layers > 1 and stride != layer else 0
    need, layer, stride = params.rows
    holds = t.is_contiguous() and t.nbytes >= need
    if stride and t.dim() > 1:                       # (else flat)
        holds = t.shape[0] >= params.layers and t.stride(0) == stride and t[0].is_contiguous() and t[0].numel() >= layer and (
            t.untyped_storage().nbytes() - 2 * t.storage_offset() >= need)
    if not holds or not _is_bf16(t):
        _refuse(where, f"{tuple(t.shape)} of {t.dtype} with strides {t.stride()} for pools of {need} bytes" + f", {stride} elements apart" * bool(stride))
    return t.data_ptr()


def _segments(params: kvsel_pages_params) -> int:
    return params.batch * params.h_kv if params.lens_per_head else params.batch


def kvsel_pages_fork(params: kvsel_pages_params, table_in, lens_in, src, table_out, lens_out, ref, ws, stream=None) -> None:
    """Row b of table_out is row src[b] of table_in (-1: none); the uses of the pages follow."""
    where, n, segs = "kvsel_pages_fork", params.batch * params.max_blocks, _segments(params)
    st = _place(ws, stream, where)
    rc = (_lib or load()).kvsel_pages_fork(
        params, _int32(table_in, n, where), _int32(lens_in, segs, where), _int32(src, params.batch, where),
        _int32(table_out, n, where), _int32(lens_out, segs, where), _int32(ref, params.num_blocks, where), ws.data_ptr(),
        ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_pages_reserve(params: kvsel_pages_params, k, v, table, ref, lens, granted, ws, new_lens=None, stream=None) -> None:
    """Pages for the new rows of every request; a shared page that they go to is copied, in every layer."""
    where, B = "kvsel_pages_reserve", params.batch
    st = _place(ws, stream, where)
    rc = (_lib or load()).kvsel_pages_reserve(
        params, _pool(k, params, where), _pool(v, params, where), _int32(table, B * params.max_blocks, where),
        _int32(ref, params.num_blocks, where), _int32(lens, _segments(params), where), _int32(new_lens, B, where),
        _int32(granted, B, where), ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_pages_trim(params: kvsel_pages_params, table, ref, lens, ws, stream=None) -> None:
    """Pages behind a request's rows are given back."""
    where = "kvsel_pages_trim"
    st = _place(ws, stream, where)
    rc = (_lib or load()).kvsel_pages_trim(
        params, _int32(table, params.batch * params.max_blocks, where), _int32(ref, params.num_blocks, where),
        _int32(lens, _segments(params), where), ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_pages_accept(params: kvsel_pages_params, k, v, table, lens, path, counts, lens_out, ws, new_lens=None,
                       stream=None) -> None:
    """The rows of the accepted nodes move to the front of the tree's, in every layer."""
    where, B, segs = "kvsel_pages_accept", params.batch, _segments(params)
    st = _place(ws, stream, where)
    rc = (_lib or load()).kvsel_pages_accept(
        params, _pool(k, params, where), _pool(v, params, where), _int32(table, B * params.max_blocks, where),
        _int32(lens, segs, where), _int32(new_lens, B, where), _int32(path, B * params.n_new, where), _int32(counts, B, where),
        _int32(lens_out, segs, where), ws.data_ptr(), ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_rope_table(*, rot_dim: int = 128, layout: str = "half", theta: float = 10000.0, scaling: str = "none",
                     factor: float = 1.0, orig_len: int = 0, direction: str = "forward", beta_fast: float = 32.0,
                     beta_slow: float = 1.0, low_freq: float = 1.0, high_freq: float = 4.0,
                     value_scale: float = 0.0) -> kvsel_rope_angles:
    """The angles that kvsel_rope and kvsel_rope_cache take, made once per model and direction."""
    p = kvsel_rope_params(rot_dim, ROPE_LAYOUT[layout], ROPE_DIRECTION[direction], ROPE_SCALING[scaling], orig_len, theta,
                          factor, beta_fast, beta_slow, low_freq, high_freq, value_scale)
    t = kvsel_rope_angles()
    _check(load().kvsel_rope_table(p, t), "kvsel_rope_table")
    return t


@functools.lru_cache(maxsize=256)
def _rope_rows(q_shape, q, qo_shape, qo, k_shape, k, ko_shape, ko, pos_shape, pos) -> kvsel_rope_rows:
    """What kvsel_rope is told of tensors with these shapes and strides."""
    where = "kvsel_rope"
    if len(q_shape) != 4 or qo_shape != q_shape or (k_shape and (len(k_shape) != 4 or ko_shape != k_shape)):
        _refuse(where, f"q {q_shape} to {qo_shape}, k {k_shape} to {ko_shape}")
    B, h, n, d = q_shape
    hk = k_shape[1] if k_shape else 0
    if d != 128 or (k_shape and (k_shape[0], *k_shape[2:]) != (B, n, d)) or any(s[3] != 1 for s in (q, qo, k, ko) if s):
        _refuse(where, f"q {q_shape} with strides {q} and {qo}, k {k_shape} with strides {k} and {ko}")
    if tuple(pos_shape) not in ((B, n), (n,)) or (n > 1 and pos[-1] != 1):
        _refuse(where, f"pos {pos_shape} with strides {pos}")
    zero = (0, 0, 0, 0)
    return kvsel_rope_rows(B, n, h, hk, *q[:3], *qo[:3], *(k or zero)[:3], *(ko or zero)[:3], pos[0] if len(pos_shape) == 2 else 0)


def kvsel_rope(table: kvsel_rope_angles, q, pos, q_out=None, k=None, k_out=None, new_lens=None, stream=None) -> None:
    """Rows q [batch][heads][tokens][128] (and k, with other heads) turned by pos [batch][tokens] or [tokens];
    without an output in place."""
    where = "kvsel_rope"
    q_out = q if q_out is None else q_out
    if k is None:
        if k_out is not None:
            _refuse(where, "k_out without k")
        keys, k_ptr, ko_ptr = (None,) * 4, None, None
    else:
        k_out = k if k_out is None else k_out
        keys, k_ptr, ko_ptr = (k.shape, k.stride(), k_out.shape, k_out.stride()), k.data_ptr(), k_out.data_ptr()
    for t in (q, q_out) if k is None else (q, q_out, k, k_out):
        if not _is_bf16(t):
            _refuse(where, f"{tuple(t.shape)} of {t.dtype}")
    if pos.dtype is not _INT32 and (pos.element_size() != 4 or pos.is_floating_point()):
        _refuse(where, f"pos of {pos.dtype}")
    p = _rope_rows(q.shape, q.stride(), q_out.shape, q_out.stride(), *keys, pos.shape, pos.stride())
    st = _place(q, stream, where)
    rc = (_lib or load()).kvsel_rope(table, p, q.data_ptr(), q_out.data_ptr(), k_ptr, ko_ptr, pos.data_ptr(),
                                     new_lens if new_lens is None else _int32(new_lens, p.batch, where), st)
    if rc:
        _check(rc, where)


def kvsel_rope_cache(table: kvsel_rope_angles, kv: kvsel_kv, lens, pos=None, ws=None, out=None, batch: int = 0,
                     h_kv: int = 0, max_len: int = 0, stream=None) -> None:
    """Cached keys turned by pos [batch][h_kv][rows] (None: row j's position is j, with batch, h_kv and max_len
    given), in place or into out [batch][h_kv][rows][128].  lens: [batch] or [batch][h_kv]."""
    where = "kvsel_rope_cache"
    if pos is not None:
        B, H, n = pos.shape
    else:
        B, H, n = batch, h_kv, max_len
    per_head = lens.numel() != B
    o = (0, 0, 0)
    if out is not None:
        o = out.stride()[:3]
        if not _is_bf16(out) or out.dim() != 4 or out.stride()[3] != 1 or out.shape[3] != 128 or out.shape[0] < B or (
                out.shape[1] < H or out.shape[2] < n):
            _refuse(where, f"out {tuple(out.shape)} of {out.dtype} with strides {out.stride()}")
    p = kvsel_rope_cache_params(H, B, n, int(per_head), n if pos is not None else 0, *o)
    st = _place(lens, stream, where)
    rc = (_lib or load()).kvsel_rope_cache(table, p, kv, _int32(lens, B * H if per_head else B, where), _int32(pos, B * H * n, where),
                                           _ptr(out), _ptr(ws), 0 if ws is None else ws.nbytes, st)
    if rc:
        _check(rc, where)


def kvsel_get_device_status(ws, stream=None) -> int:
    """Read and clear the status word of workspace `ws`, or with ws=None the one of the
    built-in buffer that kvsel_score_noalloc uses on the current device."""
    st = ctypes.c_int()
    _check(load().kvsel_get_device_status(_ptr(ws), _stream(stream), ctypes.byref(st)), "kvsel_get_device_status")
    return st.value


# ------------------------------------------------------------------------------ buffers
class LayerBuffers:
    """Device outputs and workspace for one layer call (torch allocations)."""

    def __init__(self, params: kvsel_params, device="cuda"):
        import torch

        n_scores, n_kept, n_seg = kvsel_output_size(params)
        ws_bytes = kvsel_workspace_size(params)
        self.s_attn = torch.empty(max(n_scores, 1), dtype=torch.float32, device=device)
        self.s_val = torch.empty(max(n_scores, 1), dtype=torch.float32, device=device) if params.value_aware else None
        self.idx = torch.empty(max(n_kept, 1), dtype=torch.int32, device=device)
        self.counts = torch.empty(max(n_seg, 1), dtype=torch.int32, device=device)
        self.offsets = torch.empty(max(n_seg, 1), dtype=torch.int64, device=device)
        self.k_out = torch.empty((max(n_kept, 1), params.head_dim), dtype=torch.bfloat16, device=device)
        self.v_out = torch.empty((max(n_kept, 1), params.head_dim), dtype=torch.bfloat16, device=device)
        self.ws = torch.empty(max(ws_bytes, 256) // 4 + 64, dtype=torch.int32, device=device)
        if params.budget_mode == BUDGET["anchor"]:
            # anchors: per-position slot and gamma for K and V (k_out / v_out hold the anchors)
            self.slot_k = torch.empty(max(n_scores, 1), dtype=torch.int32, device=device)
            self.slot_v = torch.empty(max(n_scores, 1), dtype=torch.int32, device=device)
            self.gamma_k = torch.empty(max(n_scores, 1), dtype=torch.float32, device=device)
            self.gamma_v = torch.empty(max(n_scores, 1), dtype=torch.float32, device=device)
        kvsel_workspace_init(self.ws)
        self.n_scores, self.n_kept, self.n_seg = n_scores, n_kept, n_seg
