"""Python binding of libpw.so (include/pw.h): argument marshalling only.

Every function keeps its C name and signature; device buffers are passed as torch
tensors (or raw integer addresses), host buffers as numpy arrays.  A call that returns
a status other than PW_OK raises ``PwError`` with ``pw_last_error``'s message.  There is
no fallback: if libpw.so has not been built, importing works but the first call raises.
"""
from __future__ import annotations

import ctypes as C
import os

import numpy as np

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpw.so")

PW_OK, PW_ERR_INVALID, PW_ERR_CUDA, PW_ERR_OOM, PW_ERR_STATE, PW_ERR_TIMEOUT, PW_ERR_BUSY, PW_ERR_RANGE = range(8)
PW_FLAG_POISON = 1
PW_ACCUMULATE = 1
PW_PRENORM = 2
PW_PAGE_GPU, PW_PAGE_CPU, PW_PAGE_TO_CPU, PW_PAGE_TO_GPU = range(4)
PW_BF16, PW_FP16 = range(2)
PW_TREE_NODES = 256
STATUS_NAMES = {0: "PW_OK", 1: "PW_ERR_INVALID", 2: "PW_ERR_CUDA", 3: "PW_ERR_OOM",
                4: "PW_ERR_STATE", 5: "PW_ERR_TIMEOUT", 6: "PW_ERR_BUSY",
                7: "PW_ERR_RANGE"}


class PwError(RuntimeError):
    def __init__(self, status, msg):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


class pw_desc(C.Structure):
    _fields_ = [("L", C.c_int), ("E", C.c_int), ("H", C.c_int), ("I", C.c_int), ("K", C.c_int),
                ("Is", C.c_int), ("bmax", C.c_int), ("bits_mask", C.c_uint32), ("renorm", C.c_int),
                ("device", C.c_int), ("max_tokens", C.c_int), ("flags", C.c_int)]


class pw_block_info(C.Structure):
    _fields_ = [("layer", C.c_int), ("expert", C.c_int), ("u", C.c_int), ("N", C.c_int), ("K", C.c_int),
                ("q", C.c_int), ("d", C.c_int), ("pending_q", C.c_int), ("state", C.c_int * 8),
                ("M", C.c_int64 * 9)]


class pw_mem_info(C.Structure):
    _fields_ = [("resident_bytes", C.c_int64), ("device_pool_bytes", C.c_int64),
                ("device_pool_free", C.c_int64), ("pinned_bytes", C.c_int64), ("scratch_bytes", C.c_int64),
                ("held_bytes", C.c_int64)]


class pw_kv_stats(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("budget_bytes", "block_bytes", "weight_bytes", "capacity_blocks",
                                         "used_blocks", "pending_blocks", "free_blocks", "headroom_bytes")]


class pw_obs(C.Structure):
    _fields_ = [("T_blk", C.c_int), ("F_blk", C.c_int), ("B_KV", C.c_double), ("R", C.c_int),
                ("mass", C.c_void_p), ("phi", C.c_void_p), ("rho_hat", C.c_void_p)]


class pw_request_signals(C.Structure):
    _fields_ = [("mass", C.c_void_p), ("rho_hat", C.c_void_p), ("conf", C.c_void_p), ("rho_min", C.c_double),
                ("rho_max", C.c_double), ("kv_blocks", C.c_double)]


class pw_offline(C.Structure):
    _fields_ = [("n_bits", C.c_int), ("s", C.c_void_p), ("head_w", C.c_void_p), ("head_a", C.c_void_p),
                ("head_c", C.c_void_p), ("alpha", C.c_double), ("rho_min", C.c_double),
                ("rho_max", C.c_double), ("eps", C.c_double), ("n_buckets", C.c_int), ("mu", C.c_void_p),
                ("floors", C.c_void_p), ("n_stages", C.c_int)]


class pw_plan_entry(C.Structure):
    _fields_ = [("block", C.c_int), ("from_bits", C.c_int), ("to_bits", C.c_int), ("delta", C.c_double)]


class pw_plan(C.Structure):
    _fields_ = [("entries", C.POINTER(pw_plan_entry)), ("capacity", C.c_int), ("n", C.c_int),
                ("kind", C.c_int), ("stage", C.c_int), ("D", C.c_double), ("total", C.c_double)]


class pw_plan_problem(C.Structure):
    _fields_ = [("n_blocks", C.c_int), ("n_bits", C.c_int), ("L", C.c_int), ("E", C.c_int),
                ("bits", C.c_void_p), ("q", C.c_void_p), ("q_init", C.c_void_p), ("utype", C.c_void_p),
                ("layer", C.c_void_p), ("expert", C.c_void_p), ("M", C.c_void_p)]


class pw_attn_desc(C.Structure):
    _fields_ = [(n, C.c_int) for n in ("L", "n_heads", "n_kv_heads", "head_dim", "dtype", "n_blocks", "block_tokens",
                                       "max_requests", "max_tokens", "max_shared_tokens", "n_plans", "device", "max_tree_tokens")]


class pw_kv_step(C.Structure):
    _fields_ = [("R", C.c_int), ("n_tokens", C.c_int), ("max_new", C.c_int), ("table_rows", C.c_int),
                ("table_stride", C.c_int), ("ctx_len", C.c_void_p), ("new_len", C.c_void_p), ("rows", C.c_void_p),
                ("table", C.c_void_p), ("q_start", C.c_void_p), ("kv_len", C.c_void_p), ("slot", C.c_void_p),
                ("pos", C.c_void_p), ("n_groups", C.c_int), ("group_start", C.c_void_p), ("shared_len", C.c_void_p)]


class pw_rope_desc(C.Structure):
    _fields_ = [("rot_dim", C.c_int), ("interleaved", C.c_int), ("n_axes", C.c_int), ("inv_freq", C.c_void_p),
                ("axis", C.c_void_p), ("scale", C.c_float), ("q_gain", C.c_void_p), ("k_gain", C.c_void_p), ("eps", C.c_float)]


class pw_tree(C.Structure):
    _fields_ = [("tree_len", C.c_void_p), ("parent", C.c_void_p), ("parent_stride", C.c_int), ("pos", C.c_void_p)]


_P = C.c_void_p
_I = C.c_int
_L = C.c_int64
_F = C.c_float
_SIGS = {
    "pw_create": [C.POINTER(pw_desc), C.POINTER(_P)],
    "pw_destroy": [_P],
    "pw_last_error": [_P],
    "pw_version": [],
    "pw_set_stream": [_P, _P],
    "pw_get_stream": [_P, C.POINTER(_P)],
    "pw_pack": [_P, _I, _I, _I, _P, _P, _I],
    "pw_set_router": [_P, _I, _P, _P],
    "pw_set_shared": [_P, _I, _P, _P],
    "pw_set_shared_gate": [_P, _I, _P],
    "pw_routing_features": [_P, _I, _P, _I],
    "pw_moe_forward": [_P, _I, _P, _I, _P, _P, _P, _I, _P],
    "pw_check": [_P],
    "pw_stack_forward": [_P, _P, _I, _P],
    "pw_stack_forward_host": [_P, _P, _I, _P],
    "pw_routing_stats": [_P, _I, _P, _P, _I],
    "pw_set_bits": [_P, _I, _I],
    "pw_offload": [_P, _I, _I],
    "pw_reload": [_P, _I, _I],
    "pw_commit": [_P, C.POINTER(_I)],
    "pw_sync_io": [_P],
    "pw_query": [_P, _I, C.POINTER(pw_block_info)],
    "pw_memory": [_P, C.POINTER(pw_mem_info)],
    "pw_set_fault": [_P, _I, _I],
    "pw_plan_host": [C.POINTER(pw_plan_problem), C.POINTER(pw_obs), C.POINTER(pw_offline), C.POINTER(pw_plan)],
    "pw_plan_step": [_P, C.POINTER(pw_obs), C.POINTER(pw_offline), C.POINTER(pw_plan)],
    "pw_merge_requests": [C.POINTER(pw_request_signals), _I, _I, _I, _I, _I, _P, _P, _P, C.POINTER(C.c_double),
                          C.POINTER(C.c_double)],
    "pw_route_noalloc": [_P, _I, _P, _I, _P, _P, _I, _P],
    "pw_kv_create": [C.c_int64, C.c_int64, C.POINTER(C.c_void_p)],
    "pw_kv_destroy": [_P],
    "pw_kv_set_weight_bytes": [_P, C.c_int64],
    "pw_kv_attach": [_P, _P],
    "pw_kv_announce": [_P, C.c_int64, C.c_int64],
    "pw_kv_grow": [_P, C.c_int64, C.c_int64, _P],
    "pw_kv_release": [_P, C.c_int64, C.POINTER(C.c_int64)],
    "pw_kv_request": [_P, C.c_int64, C.POINTER(C.c_int64), C.POINTER(C.c_int64)],
    "pw_kv_blocks": [_P, C.c_int64, _P, C.c_int64, C.POINTER(C.c_int64)],
    "pw_kv_get_stats": [_P, C.POINTER(pw_kv_stats)],
    "pw_kv_fork": [_P, C.c_int64, C.c_int64, C.c_int64],
    "pw_kv_unshare": [_P, C.c_int64, C.c_int64, C.POINTER(C.c_int32), C.POINTER(C.c_int32)],
    "pw_kv_trim": [_P, C.c_int64, C.c_int64, C.POINTER(C.c_int64)],
    "pw_kv_compact": [_P, C.c_int64, _P, _P, C.c_int64, C.POINTER(C.c_int64)],
    "pw_attn_create": [C.POINTER(pw_attn_desc), C.POINTER(C.c_void_p)],
    "pw_attn_destroy": [_P],
    "pw_attn_bind": [_P, _I, _P, _P, _L, _L, _L],
    "pw_kv_map": [_P, _P, _P, _I, _P],
    "pw_attn_plan": [_P, _I, _P, _I, _P, _P, _P],
    "pw_attn_append": [_P, _I, _P, _P, _L, _L, _P, _L, _L, _P],
    "pw_attn_forward": [_P, _I, _I, _P, _L, _L, _P, _L, _L, _P, _F, _F, _P, _P],
    "pw_attn_set_rope": [_P, _I, C.POINTER(pw_rope_desc)],
    "pw_attn_rope_append": [_P, _I, _P, _P, _L, _L, _P, _L, _L, _P, _L, _L, _P, _L, _L, _P, _P],
    "pw_attn_plan_tree": [_P, _I, _P, _I, C.POINTER(pw_tree), _P],
    "pw_kv_keep": [_P, _P, _P, _P, _I, _P, _P, _P],
    "pw_kv_copy": [_P, _P, _P, _I, _P, _I, _I, _P],
    "pw_attn_check": [_P, _P],
    "pw_attn_set_fault": [_P, _I, _I],
    "pw_set_profiling": [_P, _I],
    "pw_set_gemv_tokens": [_P, _I],
    "pw_profile_read": [_P, _I, _P],
    "pw_tc_selftest": [_P, _P, _I, _I, _I, _P, _P, _P],
    "pw_unpack_indices": [_P, _I, _I, _P],
    "pw_dequant": [_P, _I, _I, _P],
    "pw_pack_planes_host": [_P, _I, _I, _I, _P],
    "pw_tile_planes_host": [_P, _I, _I, _I, _I, _P],
    "pw_untile_planes_host": [_P, _I, _I, _I, _I, _P],
}

_lib = None


def lib():
    """The loaded libpw.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libpw.so is not built; run any_precision_bit_gb300._build.build()")
        L = C.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            f = getattr(L, name)
            f.argtypes = args
            f.restype = None if name in ("pw_destroy", "pw_kv_destroy", "pw_attn_destroy") else (C.c_char_p if name in ("pw_last_error", "pw_version") else C.c_int)
        _lib = L
    return _lib


def _ptr(obj):
    """Address of a torch tensor, numpy array, integer address or None."""
    if obj is None:
        return None
    if isinstance(obj, int):
        return obj
    if isinstance(obj, np.ndarray):
        if not obj.flags["C_CONTIGUOUS"]:
            raise ValueError("numpy arrays must be C-contiguous")
        return obj.ctypes.data
    if hasattr(obj, "data_ptr"):
        if hasattr(obj, "is_contiguous") and not obj.is_contiguous():
            raise ValueError("tensors must be contiguous")
        return obj.data_ptr()
    if hasattr(obj, "cuda_stream"):
        return obj.cuda_stream
    raise TypeError(f"cannot take the address of {type(obj)}")


def _check(st, ctx=None):
    if st != PW_OK:
        msg = lib().pw_last_error(ctx)
        raise PwError(st, msg.decode() if msg else "")
    return st


def _stream(s):
    if s is None:
        return None
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


# ------------------------------------------------------------------ the ABI, one to one
def pw_version():
    return lib().pw_version().decode()


def pw_create(desc: pw_desc):
    h = C.c_void_p()
    _check(lib().pw_create(C.byref(desc), C.byref(h)))
    return h.value


def pw_destroy(ctx):
    lib().pw_destroy(ctx)


def pw_last_error(ctx=None):
    return lib().pw_last_error(ctx).decode()


def pw_set_stream(ctx, stream):
    _check(lib().pw_set_stream(ctx, _stream(stream)), ctx)


def pw_get_stream(ctx):
    s = C.c_void_p()
    _check(lib().pw_get_stream(ctx, C.byref(s)), ctx)
    return s.value or 0


def pw_pack(ctx, layer, expert, u, idx, lut, q_init):
    _check(lib().pw_pack(ctx, layer, expert, u, _ptr(idx), _ptr(lut), q_init), ctx)


def pw_set_router(ctx, layer, Wr, bias=None):
    _check(lib().pw_set_router(ctx, layer, _ptr(Wr), _ptr(bias)), ctx)


def pw_set_shared(ctx, layer, wgu, wd):
    _check(lib().pw_set_shared(ctx, layer, _ptr(wgu), _ptr(wd)), ctx)


def pw_set_shared_gate(ctx, layer, wsg=None):
    if wsg is not None and not hasattr(wsg, "data_ptr"):
        wsg = np.ascontiguousarray(wsg, dtype=np.float32)
    _check(lib().pw_set_shared_gate(ctx, layer, _ptr(wsg)), ctx)


def pw_moe_forward(ctx, layer, x, T, y, ids=None, w=None, flags=0, stream=None):
    _check(lib().pw_moe_forward(ctx, layer, _ptr(x), T, _ptr(y), _ptr(ids), _ptr(w), flags, _stream(stream)), ctx)


def pw_check(ctx):
    _check(lib().pw_check(ctx), ctx)


def pw_stack_forward(ctx, x, T, stream=None):
    _check(lib().pw_stack_forward(ctx, _ptr(x), T, _stream(stream)), ctx)


def pw_stack_forward_host(ctx, x_host, T, y_host):
    _check(lib().pw_stack_forward_host(ctx, _ptr(x_host), T, _ptr(y_host)), ctx)


def pw_routing_stats(ctx, layer, E, reset=False):
    cnt = np.zeros(E, dtype=np.float64)
    ws = np.zeros(E, dtype=np.float64)
    _check(lib().pw_routing_stats(ctx, layer, _ptr(cnt), _ptr(ws), int(reset)), ctx)
    return cnt, ws


def pw_routing_features(ctx, layer, E, reset=False):
    phi = np.zeros((E, 3), dtype=np.float64)
    _check(lib().pw_routing_features(ctx, layer, _ptr(phi), int(reset)), ctx)
    return phi


def pw_set_bits(ctx, block, q):
    _check(lib().pw_set_bits(ctx, block, q), ctx)


def pw_offload(ctx, block, q_new):
    _check(lib().pw_offload(ctx, block, q_new), ctx)


def pw_reload(ctx, block, q_new):
    _check(lib().pw_reload(ctx, block, q_new), ctx)


def pw_commit(ctx):
    n = C.c_int(0)
    _check(lib().pw_commit(ctx, C.byref(n)), ctx)
    return n.value


def pw_sync_io(ctx):
    _check(lib().pw_sync_io(ctx), ctx)


def pw_query(ctx, block) -> pw_block_info:
    info = pw_block_info()
    _check(lib().pw_query(ctx, block, C.byref(info)), ctx)
    return info


def pw_memory(ctx) -> pw_mem_info:
    info = pw_mem_info()
    _check(lib().pw_memory(ctx, C.byref(info)), ctx)
    return info


def pw_set_fault(ctx, kind, n):
    _check(lib().pw_set_fault(ctx, kind, n), ctx)


def pw_route_noalloc(ctx, layer, x, T, ids, w, flags=0, stream=None):
    _check(lib().pw_route_noalloc(ctx, layer, _ptr(x), T, _ptr(ids), _ptr(w), flags, _stream(stream)), ctx)


def pw_set_gemv_tokens(ctx, max_tokens):
    _check(lib().pw_set_gemv_tokens(ctx, int(max_tokens)), ctx)


def pw_set_profiling(ctx, on):
    _check(lib().pw_set_profiling(ctx, int(on)), ctx)


def pw_profile_read(ctx, layer):
    ms = np.zeros(4, dtype=np.float32)
    _check(lib().pw_profile_read(ctx, layer, _ptr(ms)), ctx)
    return ms


def pw_tc_selftest(A, B, N, K, D, err, stream=None, a_in_tmem=False):
    _check(lib().pw_tc_selftest(_ptr(A), _ptr(B), N, K, 1 if a_in_tmem else 0, _ptr(D), _ptr(err), _stream(stream)))


def pw_unpack_indices(ctx, block, b, N, K):
    out = np.zeros((N, K), dtype=np.uint8)
    _check(lib().pw_unpack_indices(ctx, block, b, _ptr(out)), ctx)
    return out


def pw_dequant(ctx, block, b, N, K):
    out = np.zeros((N, K), dtype=np.uint16)
    _check(lib().pw_dequant(ctx, block, b, _ptr(out)), ctx)
    return out


def pw_pack_planes_host(idx: np.ndarray, bmax: int) -> np.ndarray:
    idx = np.ascontiguousarray(idx, dtype=np.uint8)
    N, K = idx.shape
    W = (K + 127) // 128 * 4
    out = np.zeros((bmax, N, W), dtype=np.uint32)
    _check(lib().pw_pack_planes_host(_ptr(idx), N, K, bmax, _ptr(out)))
    return out


def pw_tile_planes_host(planes: np.ndarray, K: int, u: int) -> np.ndarray:
    planes = np.ascontiguousarray(planes, dtype=np.uint32)
    nplanes, N, W = planes.shape
    out = np.zeros_like(planes)
    _check(lib().pw_tile_planes_host(_ptr(planes), N, K, nplanes, u, _ptr(out)))
    return out


def pw_untile_planes_host(tiled: np.ndarray, K: int, u: int) -> np.ndarray:
    tiled = np.ascontiguousarray(tiled, dtype=np.uint32)
    nplanes, N, W = tiled.shape
    out = np.zeros_like(tiled)
    _check(lib().pw_untile_planes_host(_ptr(tiled), N, K, nplanes, u, _ptr(out)))
    return out


def _plan_result(plan, entries):
    return dict(kind=plan.kind, stage=plan.stage, D=plan.D, total=plan.total,
                entries=[(entries[i].block, entries[i].from_bits, entries[i].to_bits, entries[i].delta)
                         for i in range(plan.n)])


def _offline_struct(off, keep):
    def arr(v, dt):
        a = np.ascontiguousarray(v, dtype=dt)
        keep.append(a)
        return a.ctypes.data
    return pw_offline(n_bits=int(np.asarray(off["s"]).shape[1]), s=arr(off["s"], np.float64),
                      head_w=arr(off["head_w"], np.float64), head_a=arr(off["head_a"], np.float64),
                      head_c=arr(off["head_c"], np.float64), alpha=float(off["alpha"]),
                      rho_min=float(off["rho_min"]), rho_max=float(off["rho_max"]), eps=float(off["eps"]),
                      n_buckets=len(off["mu"]), mu=arr(off["mu"], np.float64),
                      floors=arr(off["floors"], np.int32), n_stages=int(off["n_stages"]))


def pw_plan_host(bits, q, q_init, utype, layer, expert, M, L, E, obs: dict, off: dict, capacity=None):
    keep = []

    def arr(v, dt):
        a = np.ascontiguousarray(v, dtype=dt)
        keep.append(a)
        return a.ctypes.data
    n = len(q)
    prob = pw_plan_problem(n_blocks=n, n_bits=len(bits), L=L, E=E, bits=arr(bits, np.int32), q=arr(q, np.int32),
                           q_init=arr(q_init, np.int32), utype=arr(utype, np.int32), layer=arr(layer, np.int32),
                           expert=arr(expert, np.int32), M=arr(M, np.float64))
    o = pw_obs(T_blk=int(obs["T_blk"]), F_blk=int(obs["F_blk"]), B_KV=float(obs["B_KV"]), R=int(obs.get("R", 0)),
               mass=arr(obs["mass"], np.float64),
               phi=arr(obs["phi"], np.float64) if obs.get("phi") is not None else None,
               rho_hat=arr(obs["rho_hat"], np.float64) if obs.get("rho_hat") is not None else None)
    f = _offline_struct(off, keep)
    cap = capacity if capacity is not None else max(n, 1)
    entries = (pw_plan_entry * cap)()
    plan = pw_plan(entries=C.cast(entries, C.POINTER(pw_plan_entry)), capacity=cap)
    _check(lib().pw_plan_host(C.byref(prob), C.byref(o), C.byref(f), C.byref(plan)))
    return _plan_result(plan, entries)


def pw_plan_step(ctx, n_blocks, obs: dict, off: dict):
    keep = []

    def arr(v, dt):
        a = np.ascontiguousarray(v, dtype=dt)
        keep.append(a)
        return a.ctypes.data
    o = pw_obs(T_blk=int(obs["T_blk"]), F_blk=int(obs["F_blk"]), B_KV=float(obs["B_KV"]), R=int(obs.get("R", 0)),
               mass=arr(obs["mass"], np.float64) if obs.get("mass") is not None else None,
               phi=arr(obs["phi"], np.float64) if obs.get("phi") is not None else None,
               rho_hat=arr(obs["rho_hat"], np.float64) if obs.get("rho_hat") is not None else None)
    f = _offline_struct(off, keep)
    entries = (pw_plan_entry * n_blocks)()
    plan = pw_plan(entries=C.cast(entries, C.POINTER(pw_plan_entry)), capacity=n_blocks)
    _check(lib().pw_plan_step(ctx, C.byref(o), C.byref(f), C.byref(plan)), ctx)
    return _plan_result(plan, entries)


def pw_merge_requests(requests, kv_blocks, L, E, n_blocks, n_bits):
    """requests: dicts with mass [L][E], rho_hat [n_blocks][n_bits-1], conf [2][n_bits-1],
    rho_min, rho_max; kv_blocks: one weight per request.  Returns the merged table as a dict."""
    keep = []

    def arr(v):
        a = np.ascontiguousarray(v, dtype=np.float64)
        keep.append(a)
        return a.ctypes.data
    reqs = (pw_request_signals * len(requests))()
    for r, (q, kv) in enumerate(zip(requests, kv_blocks)):
        reqs[r] = pw_request_signals(mass=arr(q["mass"]), rho_hat=arr(q["rho_hat"]), conf=arr(q["conf"]),
                                     rho_min=float(q["rho_min"]), rho_max=float(q["rho_max"]), kv_blocks=float(kv))
    mass = np.zeros((L, E))
    rho = np.zeros((n_blocks, n_bits - 1))
    conf = np.zeros((2, n_bits - 1))
    lo, hi = C.c_double(), C.c_double()
    _check(lib().pw_merge_requests(reqs, len(requests), L, E, n_blocks, n_bits, _ptr(mass), _ptr(rho), _ptr(conf),
                                   C.byref(lo), C.byref(hi)))
    return dict(mass=mass, rho_hat=rho, conf=conf, rho_min=lo.value, rho_max=hi.value)


# ---------------------------------------------------------------- KV-block allocator
def pw_kv_create(budget_bytes, block_bytes):
    """A KV-block allocator over `budget_bytes` shared with the weight pages (handle)."""
    kv = C.c_void_p()
    _check(lib().pw_kv_create(int(budget_bytes), int(block_bytes), C.byref(kv)))
    return kv


def pw_kv_destroy(kv):
    lib().pw_kv_destroy(kv)


def pw_kv_set_weight_bytes(kv, weight_bytes):
    _check(lib().pw_kv_set_weight_bytes(kv, int(weight_bytes)))


def pw_kv_attach(kv, ctx):
    _check(lib().pw_kv_attach(kv, ctx))


def pw_kv_announce(kv, request, n_blocks):
    _check(lib().pw_kv_announce(kv, int(request), int(n_blocks)))


def pw_kv_grow(kv, request, n_blocks) -> np.ndarray:
    """Grow a request; returns the granted block ids (int32).  PwError(PW_ERR_OOM) when the
    free blocks do not suffice."""
    ids = np.zeros(max(int(n_blocks), 1), dtype=np.int32)
    _check(lib().pw_kv_grow(kv, int(request), int(n_blocks), ids.ctypes.data))
    return ids[:int(n_blocks)]


def pw_kv_release(kv, request) -> int:
    n = C.c_int64()
    _check(lib().pw_kv_release(kv, int(request), C.byref(n)))
    return n.value


def pw_kv_fork(kv, parent, child, n_blocks):
    """`child` shares the first n_blocks blocks of `parent`."""
    _check(lib().pw_kv_fork(kv, int(parent), int(child), int(n_blocks)))


def pw_kv_unshare(kv, request, index):
    """(source, destination) of the copy to make before the request writes to its block number `index`; the same where
    the block is the request's alone."""
    src, dst = C.c_int32(), C.c_int32()
    _check(lib().pw_kv_unshare(kv, int(request), int(index), C.byref(src), C.byref(dst)))
    return src.value, dst.value


def pw_kv_trim(kv, request, n_keep) -> int:
    n = C.c_int64()
    _check(lib().pw_kv_trim(kv, int(request), int(n_keep), C.byref(n)))
    return n.value


def pw_kv_compact(kv, limit):
    """Blocks that move below `limit`, as int32 arrays (sources, destinations)."""
    cap = pw_kv_get_stats(kv)["used_blocks"]
    src, dst, n = np.zeros(max(cap, 1), dtype=np.int32), np.zeros(max(cap, 1), dtype=np.int32), C.c_int64()
    _check(lib().pw_kv_compact(kv, int(limit), src.ctypes.data, dst.ctypes.data, cap, C.byref(n)))
    return src[:n.value], dst[:n.value]


def pw_kv_request(kv, request):
    """(blocks held, blocks announced) of a request."""
    held, ann = C.c_int64(), C.c_int64()
    _check(lib().pw_kv_request(kv, int(request), C.byref(held), C.byref(ann)))
    return held.value, ann.value


def pw_kv_blocks(kv, request) -> np.ndarray:
    n = C.c_int64()
    _check(lib().pw_kv_blocks(kv, int(request), None, 0, C.byref(n)))
    ids = np.zeros(max(n.value, 1), dtype=np.int32)
    _check(lib().pw_kv_blocks(kv, int(request), ids.ctypes.data, n.value, C.byref(n)))
    return ids[:n.value]


def pw_kv_get_stats(kv) -> dict:
    st = pw_kv_stats()
    _check(lib().pw_kv_get_stats(kv, C.byref(st)))
    return {name: getattr(st, name) for name, _ in pw_kv_stats._fields_}


# ---------------------------------------------------------------- paged attention
# (Called once or several times a layer, so argument marshalling is kept short here.)
# handle: (n_heads, n_kv_heads, head_dim, the caches' and rows' type, device, desc, plans, caches), with
# {plan: (its step's n_tokens, the step's tensors)} and {layer: its caches}: the library keeps their addresses
# Every call works on `stream` (None: the device's default stream) and returns before it has run.  Its tensors are lent to that
# stream where it is not torch's current one, so that a tensor made for the call alone is not given out again too early; other
# tensors of a foreign stream are the caller's to keep or to record, as with torch's own operators.
_attn_shapes = {}
_rope_axes = {}  # axes of a (handle, layer)'s rotation
_types = {}  # torch's, by name
_raw_stream = None  # torch's current stream of a device, as a number


def _load_types():
    global _raw_stream
    if not _types:
        import torch
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda d: torch.cuda.current_stream(d).cuda_stream)
        _types.update((n, getattr(torch, n)) for n in ("int32", "int64", "float32", "bfloat16", "float16"))


def _addr(t, device, n=0, kind="int32"):
    """Address of a contiguous tensor of at least n elements of a type on a CUDA device, or None."""
    if t is None:
        return None
    if t.dtype is not _types[kind] or not t.is_contiguous() or t.numel() < n or t.get_device() != device:
        raise ValueError(f"needs a contiguous {kind} tensor of {n} or more elements on device {device}, not {_what(t)}")
    return t.data_ptr()


def _nodes(t, device, R):
    """Address of a contiguous int32 tensor of at least R rows, and the length of a row."""
    if t.dim() != 2:
        raise ValueError(f"needs a tensor [{R}][nodes], not {_what(t)}")
    n = t.shape[1]
    return _addr(t, device, R * n), n


def _rows(t, n, heads, dim, dtype, device):
    """Address and the strides of [n or more rows][heads][dim] (unit last stride)."""
    rows, h, d = t.shape
    a, b, c = t.stride()
    if rows < n or h != heads or d != dim or c != 1 or t.dtype is not dtype or t.get_device() != device:
        raise ValueError(f"needs a tensor [{n}][{heads}][{dim}] of {dtype} on device {device}, the last dimension "
                         f"contiguous, not {_what(t)}")
    return t.data_ptr(), a, b


def _what(t):
    return f"{list(t.shape)} of {t.dtype} on {t.device}, strides {t.stride()}"


def _step_on(step, device):
    if step.device != device:
        raise ValueError(f"the step's tensors are on device {step.device}, the handle is for {device}")
    return step.address


def _cuda_stream(s):
    return 0 if s is None else getattr(s, "cuda_stream", s)


def _lend(stream, device, *tensors):
    """Tensors that a call uses on a stream that is not torch's current one (whose freed tensors are given out again at once):
    their memory stays theirs until the stream has come past the call."""
    if not hasattr(stream, "cuda_stream"):
        import torch
        raw = getattr(stream, "value", stream) or 0
        if raw == _raw_stream(device):
            return
        stream = torch.cuda.ExternalStream(raw, device=device) if raw else torch.cuda.default_stream(device)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def pw_attn_create(desc: pw_attn_desc):
    """An attention handle (pass it to the pw_attn_* calls and pw_kv_map)."""
    _load_types()
    h = C.c_void_p()
    _check(lib().pw_attn_create(C.byref(desc), C.byref(h)))
    kept = pw_attn_desc.from_buffer_copy(desc)
    dtype = _types["bfloat16" if kept.dtype == PW_BF16 else "float16"]
    _attn_shapes[h.value] = kept.n_heads, kept.n_kv_heads, kept.head_dim, dtype, kept.device, kept, {}, {}
    return h.value


def pw_attn_destroy(attn):
    kept = _attn_shapes.pop(attn, None)  # noqa: F841 (until the device's work is done)
    for key in [k for k in _rope_axes if k[0] == attn]:
        del _rope_axes[key]
    lib().pw_attn_destroy(attn)


def pw_attn_bind(attn, layer, k_cache, v_cache):
    """Caches as tensors [n_blocks][block_tokens][n_kv_heads][head_dim], views included, of the
    same strides and a unit last one.  The handle keeps them until others are bound to the layer (which does not wait for
    work on them)."""
    _, _, _, dtype, device, d, _, caches = _attn_shapes[attn]
    for c in (k_cache, v_cache):
        if (tuple(c.shape) != (d.n_blocks, d.block_tokens, d.n_kv_heads, d.head_dim) or c.dtype is not dtype
                or c.get_device() != device):
            raise ValueError(f"the caches must be tensors of the handle's shape, {dtype} and on device {device}, not {_what(c)}")
    if k_cache.stride() != v_cache.stride() or k_cache.stride(3) != 1:
        raise ValueError("the caches must have the same strides and a contiguous last dimension")
    _check(lib().pw_attn_bind(attn, layer, k_cache.data_ptr(), v_cache.data_ptr(), *k_cache.stride()[:3]))
    caches[layer] = k_cache, v_cache


def pw_make_step(ctx_len, new_len, table, q_start, kv_len, slot, pos, max_new, rows=None, groups=None, shared_len=None):
    """A pw_kv_step over device tensors, which it keeps alive: lengths int32 [R], table int32
    [rows][blocks], q_start int32 [R + 1], kv_len int32 [R], slot int64 and pos int32 [n_tokens];
    groups int32 [n_groups + 1] and shared_len int32 [n_groups] for shared prefixes.  All on one device."""
    _load_types()
    dev = ctx_len.get_device()
    if dev < 0:
        raise ValueError("a step's tensors are on a CUDA device")
    R, n, n_groups = ctx_len.numel(), pos.numel(), 0 if groups is None else groups.numel() - 1
    s = pw_kv_step(R=R, n_tokens=n, max_new=int(max_new), table_rows=table.shape[0], table_stride=table.shape[1],
                   ctx_len=_addr(ctx_len, dev), new_len=_addr(new_len, dev, R), rows=_addr(rows, dev, R),
                   table=_addr(table, dev), q_start=_addr(q_start, dev, R + 1), kv_len=_addr(kv_len, dev, R),
                   slot=_addr(slot, dev, n, "int64"), pos=_addr(pos, dev), n_groups=n_groups,
                   group_start=_addr(groups, dev), shared_len=_addr(shared_len, dev, n_groups))
    s.device = dev
    s.refs = (ctx_len, new_len, table, q_start, kv_len, slot, pos, rows, groups, shared_len)
    s.address = C.addressof(s)
    return s


def pw_kv_map(attn, step, new_ids, stream=None):
    dev = _attn_shapes[attn][4]
    raw = _cuda_stream(stream)
    st = lib().pw_kv_map(attn, _step_on(step, dev), _addr(new_ids, dev), 0 if new_ids is None else new_ids.numel(), raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, new_ids, *step.refs)


def pw_attn_plan(attn, plan, step, window=0, doc_start=None, bidir_len=None, stream=None):
    """The handle keeps the step's tensors until the plan is laid out again."""
    _, _, _, _, dev, _, plans, _ = _attn_shapes[attn]
    raw = _cuda_stream(stream)
    st = lib().pw_attn_plan(attn, plan, _step_on(step, dev), window, _addr(doc_start, dev, step.n_tokens),
                            _addr(bidir_len, dev, step.R), raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, doc_start, bidir_len, *step.refs)
    plans[plan] = step.n_tokens, step.refs


def pw_attn_append(attn, layer, step, k, v, stream=None):
    """k and v: [n_tokens][n_kv_heads][head_dim], any strides with a unit last one."""
    _, h, d, dtype, dev, _, _, _ = _attn_shapes[attn]
    n = step.n_tokens
    raw = _cuda_stream(stream)
    st = lib().pw_attn_append(attn, layer, _step_on(step, dev), *_rows(k, n, h, d, dtype, dev), *_rows(v, n, h, d, dtype, dev),
                              raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, k, v, *step.refs)


def pw_attn_forward(attn, layer, plan, q, o, lse=None, scale=None, softcap=0.0, slopes=None, stream=None):
    """q and o: [n_tokens][n_heads][head_dim], any strides with a unit last one; scale defaults to
    1 / sqrt(head_dim)."""
    h, _, d, dtype, dev, _, plans, _ = _attn_shapes[attn]
    n = plans[plan][0] if plan in plans else 0
    raw = _cuda_stream(stream)
    st = lib().pw_attn_forward(attn, layer, plan, *_rows(q, n, h, d, dtype, dev), *_rows(o, n, h, d, dtype, dev),
                               _addr(lse, dev, n * h, "float32"), d ** -0.5 if scale is None else scale, softcap,
                               _addr(slopes, dev, h, "float32"), raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, q, o, lse, slopes, *plans[plan][1])


def pw_attn_set_rope(attn, layer, inv_freq, axis=None, n_axes=1, interleaved=False, scale=1.0, q_gain=None, k_gain=None,
                     eps=1e-6):
    """inv_freq: [rot_dim / 2] on the host (empty: no rotation); axis: as many ints; gains: fp32 [head_dim], host or device."""
    _, _, d, _, dev, _, _, _ = _attn_shapes[attn]
    freq = np.ascontiguousarray(inv_freq, dtype=np.float64)
    axes = None if axis is None else np.ascontiguousarray(axis, dtype=np.int32)
    if axes is not None and axes.size != freq.size:
        raise ValueError("inv_freq and axis have an element for each pair")

    def gain(g):
        if g is None or hasattr(g, "get_device") and g.get_device() >= 0:
            return _addr(g, dev, d, "float32")
        g = np.ascontiguousarray(g, dtype=np.float32)
        if g.size < d:
            raise ValueError("a gain has an element for each of the head's")
        keep.append(g)
        return g.ctypes.data
    keep = []
    desc = pw_rope_desc(rot_dim=2 * freq.size, interleaved=int(interleaved), n_axes=int(n_axes), inv_freq=freq.ctypes.data,
                        axis=None if axes is None else axes.ctypes.data, scale=float(scale), q_gain=gain(q_gain),
                        k_gain=gain(k_gain), eps=float(eps))
    _check(lib().pw_attn_set_rope(attn, layer, C.byref(desc)))
    _rope_axes[attn, layer] = desc.n_axes


def pw_attn_rope_append(attn, layer, step, q, q_out, k, v, pos=None, stream=None):
    """q and q_out: [n_tokens][n_heads][head_dim], k and v: [n_tokens][n_kv_heads][head_dim], any strides with a unit last
    one; pos: int32 [n_axes][n_tokens], or None for the step's."""
    hq, h, d, dtype, dev, _, _, _ = _attn_shapes[attn]
    n = step.n_tokens
    if pos is not None and pos.dim() > 1 and pos.shape[-1] != n:
        raise ValueError(f"needs positions [n_axes][{n}], not {_what(pos)}")
    raw = _cuda_stream(stream)
    st = lib().pw_attn_rope_append(attn, layer, _step_on(step, dev), *_rows(q, n, hq, d, dtype, dev),
                                   *_rows(q_out, n, hq, d, dtype, dev), *_rows(k, n, h, d, dtype, dev),
                                   *_rows(v, n, h, d, dtype, dev), _addr(pos, dev, n * _rope_axes.get((attn, layer), 1)),
                                   raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, q, q_out, k, v, pos, *step.refs)


def pw_attn_plan_tree(attn, plan, step, tree_len, parent, pos=None, window=0, stream=None):
    """tree_len: int32 [R]; parent: int32 [R][nodes]; pos: int32 [n_tokens], filled.  The handle keeps the step's tensors
    and these until the plan is laid out again."""
    _, _, _, _, dev, _, plans, _ = _attn_shapes[attn]
    nodes, stride = _nodes(parent, dev, step.R)
    tree = pw_tree(tree_len=_addr(tree_len, dev, step.R), parent=nodes, parent_stride=stride, pos=_addr(pos, dev, step.n_tokens))
    raw = _cuda_stream(stream)
    st = lib().pw_attn_plan_tree(attn, plan, _step_on(step, dev), window, C.byref(tree), raw)
    if st:
        _check(st)
    plans[plan] = step.n_tokens, (*step.refs, tree_len, parent, pos)
    if raw != _raw_stream(dev):
        _lend(stream, dev, *plans[plan][1])


def pw_kv_keep(attn, step, tree_len, keep, n_keep, ctx_out=None, stream=None):
    """tree_len and n_keep: int32 [R]; keep: int32 [R][nodes]; ctx_out: int32 [R], filled."""
    dev, R = _attn_shapes[attn][4], step.R
    raw = _cuda_stream(stream)
    st = lib().pw_kv_keep(attn, _step_on(step, dev), _addr(tree_len, dev, R), *_nodes(keep, dev, R), _addr(n_keep, dev, R),
                          _addr(ctx_out, dev, R), raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, tree_len, keep, n_keep, ctx_out, *step.refs)


def pw_kv_copy(attn, src, dst, table=None, stream=None):
    """src and dst: int32 [n]; table: int32 [rows][blocks] whose entries src become dst."""
    dev, n = _attn_shapes[attn][4], src.numel()
    rows, stride = (0, 0) if table is None else table.shape
    raw = _cuda_stream(stream)
    st = lib().pw_kv_copy(attn, _addr(src, dev), _addr(dst, dev, n), n, _addr(table, dev), rows, stride, raw)
    if st:
        _check(st)
    if raw != _raw_stream(dev):
        _lend(stream, dev, src, dst, table)


def pw_attn_check(attn, stream=None):
    _check(lib().pw_attn_check(attn, _cuda_stream(stream)))


def pw_attn_set_fault(attn, kind, n):
    _check(lib().pw_attn_set_fault(attn, kind, n))
