"""Thin ctypes binding of libtps.so (C ABI in include/tps.h).

Argument marshalling only: every step of the path runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (device memory and streams are
PyTorch's); calls are enqueued on the current torch stream unless ``stream``
is given. A missing or unloadable library raises immediately -- there is no
fallback.
"""
from __future__ import annotations

import ctypes as C
import os

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtps.so")
_lib = None

OK, INVALID_ARG, SHAPE, ALIGN, CUDA, TIMEOUT, BOUNDS, WORKSPACE = range(8)
SELECT_THRESHOLD, SELECT_TOPK = 0, 1
OP_SELECT, OP_GROUP, OP_SCHEDULE, OP_FRONT = 0, 1, 2, 3
FRONT_THRESHOLD, FRONT_TOPK, FRONT_GROUP = 0, 1, 2

_P = C.c_void_p
_I64 = C.c_int64
_INT = C.c_int

# name -> (restype, argtypes); mirrors include/tps.h
SIGNATURES = {
    "lipar_score": (_INT, [_P, _P, _P, _I64, _I64, _I64, _P, _P]),
    "lipar_select": (_INT, [_P, _I64, _INT, C.c_float, _I64, _P, _P, _P, C.c_size_t, _P]),
    "lipar_select_static": (_INT, [_P, _I64, _INT, C.c_float, _I64, _P, _P, _P]),
    "lipar_front": (_INT, [_P, _P, _P, _I64, _I64, _I64, _INT, C.c_float, _I64, _INT, _P, _P, _P, _P, _P,
                           C.c_size_t, _P]),
    "lipar_group": (_INT, [_P, _I64, _INT, _P, _P, C.c_size_t, _P]),
    "lipar_schedule": (_INT, [_P, _I64, _INT, _P, _INT, _INT, _INT, _P, _P, _P, C.c_size_t, _P]),
    "tps_gather_rows": (_INT, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "kv_sync": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P, _P]),
    "kv_rerotate": (_INT, [_P, _P, _P, _I64, _I64, _INT, _INT, _P, _P, _P]),
    "pruned_attn": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, C.c_float, _P, _INT, _P, _P, _P]),
    "pruned_attn_ws": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, C.c_float, _P, _INT, _P, _P, _P,
                              C.c_size_t, _P]),
    "tps_attn_workspace_size": (C.c_size_t, [_I64, _I64, _INT, _INT]),
    "tps_attn_split": (_INT, [_I64, _I64, _INT, _INT]),
    "tps_attn_plan": (_INT, [_I64, _I64, _INT, _INT, _P, _P, _P]),
    "tps_rope_table": (_INT, [_P, _P, _P, _P, C.c_float]),
    "rope_rows": (_INT, [_P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _INT, _P]),
    "kv_sync_q8": (_INT, [_P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, _P, _P]),
    "pruned_attn_q8": (_INT, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, C.c_float, _P, _INT, _P, _P, _P,
                              C.c_size_t, _P]),
    "tps_attn_q8_workspace_size": (C.c_size_t, [_I64, _I64, _INT, _INT]),
    "pruned_attn_pair": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, C.c_float, _P, _INT, _P, _P, _P]),
    "pruned_attn_mma": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _INT, _INT, C.c_float, _P, _INT, _P, _P, _P]),
    "scatter_out": (_INT, [_P, _P, _P, _P, _I64, _I64, _INT, _INT, _P]),
    "hsa_euler_update": (_INT, [_P, _P, _P, _P, _P, _I64, _I64, _I64, C.c_float, _P]),
    "lipar_score_motion": (_INT, [_P, _I64, _I64, _I64, _INT, _P, _P]),
    "attn_lse_merge": (_INT, [_P, _P, _P, _P, _P, _I64, _INT, _INT, _P, _P, _P]),
    "timeripple_score": (_INT, [_P, _I64, _I64, _I64, _INT, _INT, _P, _P, _P, _P, _P, _P]),
    "timeripple_theta": (C.c_float, [_INT, C.c_float, C.c_float, _INT, _INT]),
    "tps_workspace_size": (C.c_size_t, [_INT, _I64, _INT]),
    "tps_workspace_min_size": (C.c_size_t, [_INT, _I64, _INT]),
    "tps_last_error": (C.c_char_p, []),
    "tps_pointer_is_device_accessible": (_INT, [_P]),
    "tps_check": (_INT, [_P]),
    "tps_philox_fill": (_INT, [_P, C.c_uint64, _I64, C.c_uint64, C.c_uint32, C.c_uint32, _P]),
    "tps_wait_probe": (_INT, [_I64, _P]),
    "tps_debug_inject_launch_failures": (None, [_INT]),
    "tps_version": (C.c_char_p, []),
}


class TPSError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[tps status {code}] {msg}")
        self.code = code


class Renoise(C.Structure):
    """tps_renoise: eff = a * cache + b * eps for pruned rows."""
    _fields_ = [("a", C.c_float), ("b", C.c_float), ("seed", C.c_uint64),
                ("step", C.c_uint32), ("pad_", C.c_uint32)]


def lib() -> C.CDLL:
    """Loads libtps.so once; raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libtps.so is not built ({_LIB_PATH}); run "
                               "`python -m token_pruned_sparse_b200.build`")
        l = C.CDLL(_LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            if not hasattr(l, name):
                continue            # calling it raises AttributeError; the ABI test flags it
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _chk(code: int):
    if code != OK:
        raise TPSError(code, lib().tps_last_error().decode())


def _ptr(t):
    return None if t is None else _P(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return _P(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def workspace_size(op: int, N: int, K: int = 0) -> int:
    return int(lib().tps_workspace_size(op, N, K))


def workspace_min_size(op: int, N: int, K: int = 0) -> int:
    return int(lib().tps_workspace_min_size(op, N, K))


def workspace(op: int, N: int, K: int = 0, device=None, minimal: bool = False) -> torch.Tensor:
    n = workspace_min_size(op, N, K) if minimal else workspace_size(op, N, K)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda")


# ---- the path -----------------------------------------------------------------------
def lipar_score(x, x_ref=None, x_prev_frame=None, out=None, stream=None):
    """x [F, HW, C] bf16 -> float32 [F*HW] relative-L1 change."""
    F, HW, Cc = x.shape
    if out is None:
        out = torch.empty(F * HW, dtype=torch.float32, device=x.device)
    _chk(lib().lipar_score(_ptr(x), _ptr(x_ref), _ptr(x_prev_frame), F, HW, Cc, _ptr(out), _stream(stream)))
    return out


def lipar_select(score, mode, tau=0.0, k=0, idx=None, count=None, ws=None, stream=None):
    """Returns (idx int32, count int32[1]) on the device."""
    N = score.numel()
    if idx is None:
        idx = torch.empty(max(N if mode == SELECT_THRESHOLD else k, 1), dtype=torch.int32, device=score.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=score.device)
    if ws is None:
        ws = workspace(OP_SELECT, N, 0, score.device)
    _chk(lib().lipar_select(_ptr(score), N, mode, float(tau), int(k), _ptr(idx), _ptr(count),
                            _ptr(ws), ws.numel(), _stream(stream)))
    return idx, count


def lipar_select_static(score, mode, tau=0.0, k=0, idx=None, count=None, stream=None):
    """lipar_select without a workspace: the library's own static scratch
    (N <= 4,194,304; calls on one device must not overlap on the GPU)."""
    N = score.numel()
    if idx is None:
        idx = torch.empty(max(N if mode == SELECT_THRESHOLD else k, 1), dtype=torch.int32, device=score.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=score.device)
    _chk(lib().lipar_select_static(_ptr(score), N, mode, float(tau), int(k), _ptr(idx), _ptr(count),
                                   _stream(stream)))
    return idx, count


def lipar_front(x, mode, x_ref=None, x_prev_frame=None, tau=0.0, k=0, K=1, score=None, idx=None, count=None,
                group=None, ws=None, stream=None):
    """Score + selection (mode FRONT_THRESHOLD / FRONT_TOPK -> (idx, count)) or
    score + group split (FRONT_GROUP -> group), in one launch where it applies.
    x [F, HW, C] bf16. Pass a tensor as `score` to also receive the scores."""
    F, HW, Cc = x.shape
    N = F * HW
    dev = x.device
    if mode == FRONT_GROUP:
        if group is None:
            group = torch.empty(N, dtype=torch.int8, device=dev)
    else:
        if idx is None:
            idx = torch.empty(max(N if mode == FRONT_THRESHOLD else k, 1), dtype=torch.int32, device=dev)
        if count is None:
            count = torch.empty(1, dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(OP_FRONT, N, K, dev)
    _chk(lib().lipar_front(_ptr(x), _ptr(x_ref), _ptr(x_prev_frame), F, HW, Cc, int(mode), float(tau), int(k),
                           int(K), _ptr(score), _ptr(idx), _ptr(count), _ptr(group), _ptr(ws), ws.numel(),
                           _stream(stream)))
    return group if mode == FRONT_GROUP else (idx, count)


def lipar_group(score, K, group=None, ws=None, stream=None):
    N = score.numel()
    if group is None:
        group = torch.empty(N, dtype=torch.int8, device=score.device)
    if ws is None:
        ws = workspace(OP_GROUP, N, K, score.device)
    _chk(lib().lipar_group(_ptr(score), N, K, _ptr(group), _ptr(ws), ws.numel(), _stream(stream)))
    return group


def lipar_schedule(group, K, budgets, T, step, m=0, idx=None, count=None, ws=None, stream=None):
    N = group.numel()
    b = (C.c_int32 * K)(*budgets)
    if idx is None:
        idx = torch.empty(max(N, 1), dtype=torch.int32, device=group.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=group.device)
    if ws is None:
        ws = workspace(OP_SCHEDULE, N, K, group.device)
    _chk(lib().lipar_schedule(_ptr(group), N, K, C.cast(b, _P), T, step, m, _ptr(idx), _ptr(count),
                              _ptr(ws), ws.numel(), _stream(stream)))
    return idx, count


def tps_gather_rows(dst, src, idx, count, cap=None, stream=None):
    N = src.shape[0]
    row_bytes = src[0].numel() * src.element_size()
    cap = dst.shape[0] if cap is None else cap
    _chk(lib().tps_gather_rows(_ptr(dst), _ptr(src), _ptr(idx), _ptr(count), cap, N, row_bytes, _stream(stream)))
    return dst


def kv_sync(k_cache, v_cache, k_fresh, v_fresh, idx, count, cap=None, renoise=None, k_eff=None,
            v_eff=None, stream=None):
    """renoise = (a, b, seed, step) or None."""
    N, H, d = k_cache.shape
    cap = k_fresh.shape[0] if cap is None else cap
    rn = None
    if renoise is not None:
        a, b, seed, step = renoise
        rn = Renoise(float(a), float(b), int(seed), int(step), 0)
        if k_eff is None:
            k_eff = torch.empty_like(k_cache)
        if v_eff is None:
            v_eff = torch.empty_like(v_cache)
    _chk(lib().kv_sync(_ptr(k_cache), _ptr(v_cache), _ptr(k_fresh), _ptr(v_fresh), _ptr(idx), _ptr(count),
                       cap, N, H, d, None if rn is None else C.cast(C.byref(rn), _P), _ptr(k_eff), _ptr(v_eff),
                       _stream(stream)))
    return k_eff, v_eff


class Rope(C.Structure):
    """tps_rope: rotary groups (t, x, y), the offset given to pruned rows, base."""
    _fields_ = [("dims", C.c_int32 * 3), ("shift", C.c_int32 * 3), ("base", C.c_float), ("pad_", C.c_int32)]


def kv_rerotate(k_cache, idx, count, dims, shift, base=10000.0, k_eff=None, cap=None, stream=None):
    """k_eff [N, H, d]: active rows copied, pruned rows turned by `shift`."""
    N, H, d = k_cache.shape
    cap = idx.shape[0] if cap is None else cap
    if k_eff is None:
        k_eff = torch.empty_like(k_cache)
    r = Rope((C.c_int32 * 3)(*[int(v) for v in dims]), (C.c_int32 * 3)(*[int(v) for v in shift]), float(base), 0)
    _chk(lib().kv_rerotate(_ptr(k_cache), _ptr(idx), _ptr(count), cap, N, H, d, C.cast(C.byref(r), _P),
                           _ptr(k_eff), _stream(stream)))
    return k_eff


def _attn(fn, q_act, k, v, idx, count, scale, blockmask, block, o_act, lse, cap, stream):
    N, H, d = k.shape
    cap = q_act.shape[0] if cap is None else cap
    if o_act is None:
        o_act = torch.empty_like(q_act)
    _chk(fn(_ptr(q_act), _ptr(k), _ptr(v), _ptr(idx), _ptr(count), cap, N, H, d, float(scale),
            _ptr(blockmask), int(block), _ptr(o_act), _ptr(lse), _stream(stream)))
    return o_act


def pruned_attn(q_act, k, v, idx, count, scale, blockmask=None, block=128, o_act=None, lse=None,
                cap=None, stream=None):
    return _attn(lib().pruned_attn, q_act, k, v, idx, count, scale, blockmask, block, o_act, lse, cap, stream)


def attn_workspace(cap, N, H, d, device=None):
    n = int(lib().tps_attn_workspace_size(cap, N, H, d))
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device or "cuda"), n


def attn_split(cap, N, H, d) -> int:
    """Whole-grid key-range split a dense pruned_attn call of this shape uses (1 = none)."""
    return int(lib().tps_attn_split(int(cap), int(N), int(H), int(d)))


def attn_plan(cap, N, H, d):
    """(split, main_rows, tail_split) of a dense pruned_attn call of this shape."""
    split, tail = C.c_int(0), C.c_int(0)
    main = C.c_int64(0)
    _chk(lib().tps_attn_plan(int(cap), int(N), int(H), int(d), C.byref(split), C.byref(main), C.byref(tail)))
    return split.value, main.value, tail.value


def pruned_attn_ws(q_act, k, v, idx, count, scale, blockmask=None, block=128, o_act=None, lse=None, cap=None,
                   ws=None, stream=None):
    N, H, d = k.shape
    cap = q_act.shape[0] if cap is None else cap
    if o_act is None:
        o_act = torch.empty_like(q_act)
    if ws is None:
        ws, _ = attn_workspace(cap, N, H, d, q_act.device)
    _chk(lib().pruned_attn_ws(_ptr(q_act), _ptr(k), _ptr(v), _ptr(idx), _ptr(count), cap, N, H, d, float(scale),
                              _ptr(blockmask), int(block), _ptr(o_act), _ptr(lse), _ptr(ws), ws.numel(),
                              _stream(stream)))
    return o_act


def pruned_attn_pair(q_act, k, v, idx, count, scale, blockmask=None, block=128, o_act=None, lse=None,
                     cap=None, stream=None):
    return _attn(lib().pruned_attn_pair, q_act, k, v, idx, count, scale, blockmask, block, o_act, lse, cap,
                 stream)


def pruned_attn_mma(q_act, k, v, idx, count, scale, blockmask=None, block=128, o_act=None, lse=None,
                    cap=None, stream=None):
    return _attn(lib().pruned_attn_mma, q_act, k, v, idx, count, scale, blockmask, block, o_act, lse, cap,
                 stream)


# ---- rotary rows and the 8-bit cache --------------------------------------------------
# These check their tensors on the host (the library sees addresses only) and run on
# the tensors' device, on its current stream unless one is given. A call costs the host
# about 10 us, so a check that passes builds no message, and addresses go to ctypes as ints.
_T, _BF16, _F32, _I32 = torch.Tensor, torch.bfloat16, torch.float32, torch.int32
_CODES = (torch.uint8, torch.float8_e4m3fn)
_MASKS = (torch.uint8, torch.bool)
_I3 = C.c_int32 * 3


def _need(cond, msg, code=INVALID_ARG):
    if not cond:
        raise TPSError(code, msg)


def _refuse(who, name, t, dtypes, shape, index):
    """Raises what is wrong with a tensor that _check did not take."""
    _need(isinstance(t, _T), f"{who}: {name} must be a tensor")
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    _need(t.dtype in dtypes, f"{who}: {name} is {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    _need(tuple(t.shape) == tuple(shape), f"{who}: {name} has shape {tuple(t.shape)}, expected {tuple(shape)}", SHAPE)
    _need(index >= 0 and t.get_device() == index,
          f"{who}: {name} is on {t.device}, expected {'a CUDA device' if index < 0 else f'cuda:{index}'}")
    _need(t.is_contiguous(), f"{who}: {name} must be contiguous")


def _check(who, name, t, dtype, shape, index):
    """t: a contiguous tensor of that type (or of one of them) and shape on CUDA device `index`; returns its address."""
    if not (isinstance(t, _T) and (t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)) and t.shape == shape
            and t.get_device() == index >= 0 and t.is_contiguous()):
        _refuse(who, name, t, dtype, shape, index)
    return t.data_ptr()


def _rows_of(who, name, t, H, d):
    _need(isinstance(t, _T) and t.dim() == 3, f"{who}: {name} must be a [rows, H, d] tensor", SHAPE)
    return t.shape[0]


def _active(who, idx, count, cap, rows, index):
    """Checks the active list against the rows at hand; returns (cap, address of idx, address of count)."""
    cap = rows if cap is None else int(cap)
    if not 0 <= cap <= rows:
        raise TPSError(SHAPE, f"{who}: cap={cap} must be in [0, {rows}]")
    _need(isinstance(idx, _T) and idx.dim() == 1, f"{who}: idx must be a one-dimensional tensor")
    if idx.shape[0] < cap:
        raise TPSError(SHAPE, f"{who}: idx holds {idx.shape[0]} entries, cap={cap}")
    return (cap, _check(who, "idx", idx, _I32, idx.shape, index), _check(who, "count", count, _I32, (1,), index))


def _call(fn, index, stream, *args):
    """fn(*args, stream) with CUDA device `index` current; raises on an error status."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(index)
    else:
        raw = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    if torch.cuda.current_device() == index:
        code = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            code = fn(*args, raw)
    if code != OK:
        _chk(code)


def _made_for(stream, index, *made):
    """Tells torch's allocator that tensors made by this call are used on `stream`. It hands memory on in the
    order of the current stream, so the other stream also waits for that one first."""
    if stream is None:
        return
    on = stream if hasattr(stream, "cuda_stream") else torch.cuda.ExternalStream(int(stream), index)
    now = torch.cuda.current_stream(index)
    if on.cuda_stream == now.cuda_stream:
        return
    on.wait_stream(now)
    for t in made:
        t.record_stream(on)


class RopeGrid(C.Structure):
    """tps_rope_grid: channels and positions of the t, x, y axes, and the table."""
    _fields_ = [("dims", C.c_int32 * 3), ("size", C.c_int32 * 3), ("table", C.c_void_p)]


class _RopeGridFlat(C.Structure):
    """The same bytes, in fields that are cheaper to fill (0.4 us against 1.4)."""
    _fields_ = [(n, C.c_int32) for n in ("dt", "dx", "dy", "F", "Ws", "Hs")] + [("table", C.c_void_p)]


def rope_table(dims, grid, origin=(0, 0, 0), base=10000.0, device=None):
    """The (cos, sin) table of a latent grid (F, Hs, Ws) for rope_rows and kv_sync_q8:
    float32 [entries, 2] on `device`, computed on the host in double precision. dims:
    channels of the t, x, y groups; origin: position of the first token on t, x, y."""
    F, Hs, Ws = (int(v) for v in grid)
    size = (F, Ws, Hs)
    _need(all(s >= 1 for s in size), f"rope_table: grid {tuple(grid)} must be positive", SHAPE)
    _need(all(int(v) >= 0 and int(v) % 2 == 0 for v in dims), f"rope_table: dims {tuple(dims)} must be even and >= 0")
    t = torch.empty((sum(s * (int(v) // 2) for s, v in zip(size, dims)), 2), dtype=torch.float32)
    arr = [C.cast(_I3(*[int(v) for v in a]), _P) for a in (dims, size, origin)]
    _chk(lib().tps_rope_table(_P(t.data_ptr()), *arr, float(base)))
    return t.to(device or "cuda")


def _rope_grid(who, table, dims, grid, index):
    F, Hs, Ws = grid
    dt, dx, dy = dims
    if min(dt, dx, dy) < 0 or (dt | dx | dy) & 1 or min(F, Hs, Ws) < 1:
        raise TPSError(INVALID_ARG, f"{who}: dims {tuple(dims)} must be even and >= 0, grid {tuple(grid)} positive")
    at = _check(who, "table", table, _F32, (F * (dt // 2) + Ws * (dx // 2) + Hs * (dy // 2), 2), index)
    return _RopeGridFlat(dt, dx, dy, F, Ws, Hs, at)


def rope_rows(src, idx, count, table, dims, grid, dst=None, src2=None, dst2=None, inverse=False, cap=None,
              stream=None):
    """Rows of src (and src2) [cap, H, d] bf16 turned to the position of token idx[j]
    on the grid (F, Hs, Ws), or back with inverse=True (the gradient). table:
    rope_table(dims, grid). idx and count None: row j is token j. Returns dst, or
    (dst, dst2); dst may be src."""
    who = "rope_rows"
    _need(isinstance(src, _T) and src.dim() == 3, "rope_rows: src must be a [rows, H, d] tensor", SHAPE)
    shape = src.shape
    A, H, d = shape
    dev = src.get_device()
    a_src = _check(who, "src", src, _BF16, shape, dev)
    made = []
    if dst is None:
        dst = torch.empty_like(src)
        made.append(dst)
    a_dst = _check(who, "dst", dst, _BF16, shape, dev)
    a_src2 = a_dst2 = None
    if src2 is not None:
        a_src2 = _check(who, "src2", src2, _BF16, shape, dev)
        if dst2 is None:
            dst2 = torch.empty_like(src2)
            made.append(dst2)
        a_dst2 = _check(who, "dst2", dst2, _BF16, shape, dev)
    elif dst2 is not None:
        raise TPSError(INVALID_ARG, "rope_rows: dst2 without src2")
    if idx is None:
        cap, a_idx = A if cap is None else int(cap), None
        _need(0 <= cap <= A, "rope_rows: cap must be in [0, rows of src]", SHAPE)
        a_cnt = None if count is None else _check(who, "count", count, _I32, (1,), dev)
    else:
        cap, a_idx, a_cnt = _active(who, idx, count, cap, A, dev)
    if cap == 0:
        return dst if src2 is None else (dst, dst2)
    g = _rope_grid(who, table, dims, grid, dev)
    F, Hs, Ws = grid
    if made:
        _made_for(stream, dev, *made)
    _call(lib().rope_rows, dev, stream, a_dst, a_src, a_dst2, a_src2, a_idx, a_cnt, cap, F * Hs * Ws, H, d,
          C.addressof(g), 1 if inverse else 0)
    return dst if src2 is None else (dst, dst2)


def _cache_q8(who, k_cache, v_cache, k_scale, v_scale):
    """Checks a cache; returns its sizes, device index and addresses."""
    _need(isinstance(k_cache, _T) and k_cache.dim() == 3, "the 8-bit k_cache must be a [N, H, d] tensor", SHAPE)
    shape = k_cache.shape
    N, H, d = shape
    dev = k_cache.get_device()
    nb = (N + 127) // 128
    return (N, H, d, dev, _check(who, "k_cache", k_cache, _CODES, shape, dev),
            _check(who, "v_cache", v_cache, _CODES, shape, dev), _check(who, "k_scale", k_scale, _F32, (nb, H), dev),
            _check(who, "v_scale", v_scale, _F32, (nb, H), dev))


def cache_q8(N, H, d, device=None):
    """An empty 8-bit cache: (k_cache, v_cache, k_scale, v_scale), e4m3 codes [N, H, d] and
    float32 scales [ceil(N / 128), H], all zero."""
    dev = device or "cuda"
    codes = [torch.zeros((N, H, d), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn) for _ in range(2)]
    scales = [torch.zeros(((N + 127) // 128, H), dtype=torch.float32, device=dev) for _ in range(2)]
    return (*codes, *scales)


def kv_sync_q8(k_cache, v_cache, k_scale, v_scale, k_fresh, v_fresh, idx, count, rope=None, cap=None, stream=None):
    """Fresh K/V rows [cap, H, d] bf16 of the active tokens into the 8-bit cache, in
    place. rope = (table, dims, grid) turns the keys to their position on the way."""
    who = "kv_sync_q8"
    N, H, d, dev, a_kc, a_vc, a_ks, a_vs = _cache_q8(who, k_cache, v_cache, k_scale, v_scale)
    nk, nv = _rows_of(who, "k_fresh", k_fresh, H, d), _rows_of(who, "v_fresh", v_fresh, H, d)
    a_kf = _check(who, "k_fresh", k_fresh, _BF16, (nk, H, d), dev)
    a_vf = _check(who, "v_fresh", v_fresh, _BF16, (nv, H, d), dev)
    cap, a_idx, a_cnt = _active(who, idx, count, cap, min(nk, nv), dev)
    if cap == 0:
        return
    g = None if rope is None else _rope_grid(who, *rope, dev)
    _call(lib().kv_sync_q8, dev, stream, a_kc, a_vc, a_ks, a_vs, a_kf, a_vf, a_idx, a_cnt, cap, N, H, d,
          None if g is None else C.addressof(g))


def attn_q8_workspace(cap, N, H, d, device=None):
    """The workspace of a dense pruned_attn_q8 call of this shape (its size depends on the
    device's SM count, so ask on the device that runs it)."""
    dev = torch.device(device or "cuda")
    with torch.cuda.device(dev):
        n = int(lib().tps_attn_q8_workspace_size(int(cap), int(N), int(H), int(d)))
    return torch.empty(n, dtype=torch.uint8, device=dev)


def pruned_attn_q8(q_act, k_cache, v_cache, k_scale, v_scale, idx, count, scale, blockmask=None, block=128,
                   o_act=None, lse=None, cap=None, ws=None, stream=None):
    """pruned_attn over the 8-bit cache. ws None: a workspace from torch's allocator, where the
    call takes one."""
    who = "pruned_attn_q8"
    N, H, d, dev, a_kc, a_vc, a_ks, a_vs = _cache_q8(who, k_cache, v_cache, k_scale, v_scale)
    rows = _rows_of(who, "q_act", q_act, H, d)
    a_q = _check(who, "q_act", q_act, _BF16, (rows, H, d), dev)
    made = []
    if o_act is None:
        o_act = torch.empty_like(q_act)
        made.append(o_act)
    n = _rows_of(who, "o_act", o_act, H, d)
    a_o = _check(who, "o_act", o_act, _BF16, (n, H, d), dev)
    rows = min(rows, n)
    a_lse = a_mask = a_ws = None
    if lse is not None:
        _need(isinstance(lse, _T) and lse.dim() == 2, "pruned_attn_q8: lse must be a [rows, H] tensor", SHAPE)
        n = lse.shape[0]
        a_lse = _check(who, "lse", lse, _F32, (n, H), dev)
        rows = min(rows, n)
    if blockmask is not None:
        nb = (N + 127) // 128
        a_mask = _check(who, "blockmask", blockmask, _MASKS, (nb, nb), dev)
    cap, a_idx, a_cnt = _active(who, idx, count, cap, rows, dev)
    if cap == 0:
        return o_act
    n_ws = 0
    if ws is not None:
        n_ws = ws.numel() * ws.element_size()
        a_ws = _check(who, "ws", ws, ws.dtype, ws.shape, dev)
    elif blockmask is None:
        if torch.cuda.current_device() == dev:
            n_ws = lib().tps_attn_q8_workspace_size(cap, N, H, d)
        else:
            with torch.cuda.device(dev):
                n_ws = lib().tps_attn_q8_workspace_size(cap, N, H, d)
        if n_ws:
            ws = torch.empty(n_ws, dtype=torch.uint8, device=q_act.device)
            a_ws = ws.data_ptr()
            made.append(ws)
    if made:
        _made_for(stream, dev, *made)
    _call(lib().pruned_attn_q8, dev, stream, a_q, a_kc, a_vc, a_ks, a_vs, a_idx, a_cnt, cap, N, H, d, float(scale), a_mask,
          int(block), a_o, a_lse, a_ws, n_ws)
    return o_act


def scatter_out(o_full, o_act, idx, count, cap=None, stream=None):
    N, H, d = o_full.shape
    cap = o_act.shape[0] if cap is None else cap
    _chk(lib().scatter_out(_ptr(o_full), _ptr(o_act), _ptr(idx), _ptr(count), cap, N, H, d, _stream(stream)))
    return o_full


def hsa_euler_update(x, v_cache, v_fresh, idx, count, dsigma, cap=None, stream=None):
    """x [N, C] float32 and v_cache [N, C] bf16 updated in place."""
    N, Cc = x.shape
    cap = v_fresh.shape[0] if cap is None else cap
    _chk(lib().hsa_euler_update(_ptr(x), _ptr(v_cache), _ptr(v_fresh), _ptr(idx), _ptr(count), cap, N, Cc,
                                float(dsigma), _stream(stream)))
    return x


def lipar_score_motion(x, L, out=None, stream=None):
    F, HW, Cc = x.shape
    if out is None:
        out = torch.empty(F * HW, dtype=torch.float32, device=x.device)
    _chk(lib().lipar_score_motion(_ptr(x), F, HW, Cc, int(L), _ptr(out), _stream(stream)))
    return out


def attn_lse_merge(o1, lse1, o2, lse2, count, o=None, lse=None, cap=None, stream=None):
    A, H, d = o1.shape
    cap = A if cap is None else cap
    if o is None:
        o = torch.empty_like(o1)
    _chk(lib().attn_lse_merge(_ptr(o1), _ptr(lse1), _ptr(o2), _ptr(lse2), _ptr(count), cap, H, d, _ptr(o),
                              _ptr(lse), _stream(stream)))
    return o


def timeripple_score(x, F, Hs, Ws, windows, theta, reuse=None, delta=False, score=False, stream=None):
    """x [F*Hs*Ws, H, d] bf16. windows: ((start, len),) * 3 for t, x, y; theta:
    3 floats. Returns (reuse uint8 [N, H], delta float32 [3, N, H] or None,
    score float32 [N] or None); pass tensors as delta/score to reuse buffers."""
    N, H, d = x.shape
    if reuse is None:
        reuse = torch.empty((N, H), dtype=torch.uint8, device=x.device)
    if delta is True:
        delta = torch.empty((3, N, H), dtype=torch.float32, device=x.device)
    if score is True:
        score = torch.empty(N, dtype=torch.float32, device=x.device)
    delta = delta if isinstance(delta, torch.Tensor) else None
    score = score if isinstance(score, torch.Tensor) else None
    win = (C.c_int32 * 6)(*[int(v) for w in windows for v in w])
    th = (C.c_float * 3)(*[float(v) for v in theta])
    _chk(lib().timeripple_score(_ptr(x), F, Hs, Ws, H, d, C.cast(win, _P), C.cast(th, _P), _ptr(reuse),
                                _ptr(delta), _ptr(score), _stream(stream)))
    return reuse, delta, score


def timeripple_theta(step, theta_lo, theta_hi, i0=11, i1=21) -> float:
    return float(lib().timeripple_theta(int(step), float(theta_lo), float(theta_hi), int(i0), int(i1)))


def pointer_is_device_accessible(t) -> bool:
    """True if library kernels may read/write tensor t in place (device memory,
    or pinned host memory mapped into the device address space)."""
    return bool(lib().tps_pointer_is_device_accessible(_P(t.data_ptr())))


def tps_check(stream=None):
    _chk(lib().tps_check(_stream(stream)))


def tps_philox_fill(q0, nq, seed, step, tensor, out=None, stream=None):
    if out is None:
        out = torch.empty(nq * 4, dtype=torch.int32, device="cuda")
    _chk(lib().tps_philox_fill(_ptr(out), q0, nq, seed, step, tensor, _stream(stream)))
    return out


def tps_wait_probe(limit_cycles, stream=None):
    _chk(lib().tps_wait_probe(int(limit_cycles), _stream(stream)))


def debug_inject_launch_failures(n: int):
    lib().tps_debug_inject_launch_failures(int(n))


def version() -> str:
    return lib().tps_version().decode()
