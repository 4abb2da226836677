"""Rotary rows and the 8-bit cache without a GPU: the oracle's pins, the host-built rope table, and the
refusals of the C ABI and of the binding."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle as O
from oracle import q8_oracle as Q
from token_pruned_sparse_b200 import synth, tps

F = C.c_void_p(0x1000)        # fake, 16-byte aligned, never dereferenced
MIS = C.c_void_p(0x1001)
NULL = None


# ---- oracle pins ----------------------------------------------------------------------------------------
def test_e4m3_decode_matches_torch_for_every_code():
    codes = np.arange(256, dtype=np.uint8)
    ref = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(Q.e4m3_decode(codes), ref)
    assert Q.e4m3_decode([0x7E])[()] == 448.0 and Q.e4m3_decode([0x01])[()] == 2.0 ** -9


def test_e4m3_round_is_nearest_even_and_saturates():
    grid = np.unique(Q.e4m3_decode([c for c in range(256) if c & 0x7F != 0x7F]))
    np.testing.assert_array_equal(Q.e4m3_round(grid), grid)
    mid = (grid[1:] + grid[:-1]) / 2
    lower = {v: (int(c) & 1) for c in range(0x7F) for v in [float(Q.e4m3_decode([c])[0])]}
    for a, b, m in zip(grid[:-1], grid[1:], mid):
        got = float(Q.e4m3_round(m))
        assert got in (a, b) and lower[abs(got)] == 0, m            # ties go to the even mantissa
        assert Q.e4m3_round(m + 1e-9 * abs(b - a)) == b and Q.e4m3_round(m - 1e-9 * abs(b - a)) == a
    assert Q.e4m3_round(1e9) == 448.0 and Q.e4m3_round(-np.inf) == -448.0 and np.isnan(Q.e4m3_round(np.nan))


@pytest.mark.parametrize("amax,scale", [(0.0, 0.0), (448.0, 1.0), (448.0000001, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8),
                                        (1.7500001, 2.0 ** -7), (1e-40, 2.0 ** -100), (3e38, 2.0 ** 100)])
def test_q8_scale(amax, scale):
    assert Q.q8_scale(amax) == scale


def test_rope_rows_oracle_inverse_and_positions():
    rng = np.random.default_rng(5)
    grid, dims = (3, 5, 7), synth.rope_dims(64)
    idx = rng.choice(105, 40, replace=False)
    x = rng.standard_normal((40, 2, 64))
    y = O.rope_rows(x, idx, dims, grid, origin=(4, -1, 2))
    np.testing.assert_allclose(O.rope_rows(y, idx, dims, grid, origin=(4, -1, 2), inverse=True), x, rtol=0, atol=1e-12)
    n = int(idx[0])
    f, y0, x0 = n // 35, (n // 7) % 5, n % 7
    np.testing.assert_allclose(y[0], O.rope_rotate(x[0], dims, (f + 4, x0 - 1, y0 + 2)), rtol=0, atol=1e-15)


def test_rope_gradient_is_the_turn_back():
    """R^T g against central differences of <R x, g>."""
    rng = np.random.default_rng(6)
    grid, dims = (2, 3, 4), synth.rope_dims(64)
    idx = np.array([23, 0, 7])
    x, g = rng.standard_normal((2, 3, 1, 64))
    grad = O.rope_rows(g, idx, dims, grid, inverse=True)
    for at in [(0, 0, 0), (1, 0, 31), (2, 0, 63), (0, 0, 40)]:
        e = np.zeros_like(x)
        e[at] = 1e-4
        diff = np.sum((O.rope_rows(x + e, idx, dims, grid) - O.rope_rows(x - e, idx, dims, grid)) * g) / 2e-4
        assert abs(diff - grad[at]) < 1e-8


def test_kv_sync_q8_oracle_scales_grow_and_do_not_drift():
    rng = np.random.default_rng(7)
    N, H, d = 300, 2, 64
    vals, sc = np.zeros((N, H, d)), np.zeros((3, H))
    every = np.arange(N)
    vals, sc = Q.kv_sync_q8(vals, sc, rng.standard_normal((N, H, d)), every)
    held = vals * np.repeat(sc, 128, 0)[:N, :, None]
    loud = 100.0 * rng.standard_normal((1, H, d))
    v2, s2 = Q.kv_sync_q8(vals, sc, loud, [5])
    assert (s2[0] > sc[0]).all() and (s2[1:] == sc[1:]).all()
    kept = np.setdiff1d(every, [5])
    now = (v2 * np.repeat(s2, 128, 0)[:N, :, None])[kept]
    big = np.abs(held[kept]) >= 2.0 ** -6 * np.repeat(s2, 128, 0)[kept, :, None]
    np.testing.assert_array_equal(now[big], held[kept][big])         # normal codes keep their value
    v3, s3 = Q.kv_sync_q8(v2, s2, 0.01 * loud, [5])                  # the scale does not fall back ...
    np.testing.assert_array_equal(s3, s2)
    np.testing.assert_array_equal(v3[kept], v2[kept])
    _, s4 = Q.kv_sync_q8(v3, s3, 0.01 * rng.standard_normal((128, H, d)), np.arange(128))
    assert (s4[0] < s3[0]).all()                                     # ... until the whole block is fresh


def test_two_e4m3_parts_hold_a_bf16_row():
    """q = 2^e (hi + lo): exact down to 2^-9 of the row's largest channel, within 2^-17 of the largest below that; and
    not 2^-10 and 2^-18 (largest 225, channel 225 * 2^-10)."""
    mant = (128 + np.arange(128)) / 128.0
    values = np.concatenate([mant * 2.0 ** e for e in range(-30, 9)])
    values = values[values <= 448]
    hi = Q.e4m3_round(values)
    miss = np.abs(hi + Q.e4m3_round(values - hi) - values)
    least, most = 224.0 * (1 + 2.0 ** -7), 448.0                     # the scaled largest lies there
    assert not miss[values >= 2.0 ** -9 * least].any()
    assert miss.max() <= 2.0 ** -17 * least
    at = np.flatnonzero(values == 225 * 2.0 ** -10)[0]
    assert values[at] < 0.25 and miss[at] > 2.0 ** -18 * 225 and Q.q8_scale(225.0) == 1.0 and Q.q8_scale(most) == 1.0


# ---- the host-built table --------------------------------------------------------------------------------
@pytest.mark.parametrize("d,grid,origin,base", [(64, (4, 8, 8), (0, 0, 0), 10000.0), (128, (3, 5, 7), (9, -2, 1000), 500.0)])
def test_rope_table(d, grid, origin, base):
    dims = synth.rope_dims(d)
    t = tps.rope_table(dims, grid, origin, base, device="cpu").double().numpy()
    at = 0
    for da, size, o in zip(dims, (grid[0], grid[2], grid[1]), origin):
        for s in range(size):
            phi = (o + s) * base ** (-2.0 * np.arange(da // 2) / da)
            # cos and sin in double, rounded once to fp32 (half a step: 2^-24 of a value <= 1), plus the
            # angle's own rounding in double (2^-52 of it)
            tol = 2.0 ** -24 + 2.0 ** -51 * np.abs(phi).max()
            assert np.abs(t[at:at + da // 2, 0] - np.cos(phi)).max() <= tol
            assert np.abs(t[at:at + da // 2, 1] - np.sin(phi)).max() <= tol
            at += da // 2
    assert at == t.shape[0]


def test_rope_table_refusals():
    arr = lambda *v: C.cast((C.c_int32 * 3)(*v), C.c_void_p)        # noqa: E731
    l = tps.lib()
    buf = C.cast((C.c_float * 64)(), C.c_void_p)
    ok = (arr(2, 2, 4), arr(1, 1, 1), arr(0, 0, 0))
    assert l.tps_rope_table(buf, *ok, 10000.0) == tps.OK
    assert l.tps_rope_table(NULL, *ok, 10000.0) == tps.INVALID_ARG
    assert l.tps_rope_table(buf, arr(3, 1, 4), *ok[1:], 10000.0) == tps.INVALID_ARG
    assert l.tps_rope_table(buf, ok[0], arr(0, 1, 1), ok[2], 10000.0) == tps.SHAPE
    assert l.tps_rope_table(buf, *ok[:2], arr((1 << 24) + 1, 0, 0), 10000.0) == tps.SHAPE
    for base in (0.0, -1.0, float("inf"), float("nan")):
        assert l.tps_rope_table(buf, *ok, base) == tps.INVALID_ARG
    with pytest.raises(tps.TPSError):
        tps.rope_table((24, 20, 20), (0, 8, 8), device="cpu")


# ---- refusals of the C ABI ----------------------------------------------------------------------------------
def _grid(dims=(24, 20, 20), size=(4, 5, 5), table=0x1000):
    return tps.RopeGrid((C.c_int32 * 3)(*dims), (C.c_int32 * 3)(*size), table)


def _p(g):
    return C.cast(C.byref(g), C.c_void_p)


BAD_GRIDS = [(_grid(dims=(23, 21, 20)), tps.INVALID_ARG), (_grid(dims=(24, 20, 18)), tps.INVALID_ARG),
             (_grid(dims=(-2, 46, 20)), tps.INVALID_ARG), (_grid(size=(4, 5, 6)), tps.SHAPE),
             (_grid(size=(4, 5, 4)), tps.SHAPE), (_grid(size=(0, 5, 5)), tps.SHAPE), (_grid(table=None), tps.INVALID_ARG),
             (_grid(table=0x1008), tps.ALIGN), (_grid(size=(1 << 24, 1 << 24, 1 << 24)), tps.SHAPE)]


def test_rope_rows_refusals():
    l, g = tps.lib(), _grid()
    call = lambda dst=F, src=F, dst2=NULL, src2=NULL, idx=F, count=F, cap=10, N=100, H=2, d=64, rope=g, inv=0: \
        l.rope_rows(dst, src, dst2, src2, idx, count, cap, N, H, d, _p(rope) if rope else NULL, inv, NULL)   # noqa: E731
    assert call(dst=NULL) == tps.INVALID_ARG and call(src=NULL) == tps.INVALID_ARG and call(rope=None) == tps.INVALID_ARG
    assert call(src2=F) == tps.INVALID_ARG and call(dst2=F) == tps.INVALID_ARG and call(count=NULL) == tps.INVALID_ARG
    assert call(cap=-1) == tps.SHAPE and call(cap=1 << 31) == tps.SHAPE and call(N=0) == tps.SHAPE
    assert call(N=1 << 31) == tps.SHAPE
    assert call(d=96) == tps.INVALID_ARG and call(H=0) == tps.SHAPE and call(H=257) == tps.SHAPE
    assert call(dst=MIS) == tps.ALIGN and call(src=MIS) == tps.ALIGN and call(src2=MIS, dst2=F) == tps.ALIGN
    assert call(idx=NULL, count=NULL, cap=101) == tps.SHAPE
    for bad, code in BAD_GRIDS:
        assert call(rope=bad) == code
    assert call(cap=0) == tps.OK                                     # nothing to do: no launch


def test_kv_sync_q8_refusals():
    l, g = tps.lib(), _grid()
    base = dict(kc=F, vc=F, ks=F, vs=F, kf=F, vf=F, idx=F, count=F, cap=10, N=100, H=2, d=64, rope=g)

    def call(**kw):
        a = {**base, **kw}
        return l.kv_sync_q8(a["kc"], a["vc"], a["ks"], a["vs"], a["kf"], a["vf"], a["idx"], a["count"], a["cap"], a["N"],
                            a["H"], a["d"], _p(a["rope"]) if a["rope"] else NULL, NULL)
    for k in ("kc", "vc", "ks", "vs", "kf", "vf", "idx", "count"):
        assert call(**{k: NULL}) == tps.INVALID_ARG, k
    for k in ("kc", "vc", "kf", "vf", "ks", "vs"):
        assert call(**{k: MIS}) == tps.ALIGN, k
    assert call(cap=-1) == tps.SHAPE and call(N=0) == tps.SHAPE and call(N=1 << 31) == tps.SHAPE
    assert call(d=32) == tps.INVALID_ARG and call(H=0) == tps.SHAPE and call(H=300) == tps.SHAPE
    for bad, code in BAD_GRIDS:
        assert call(rope=bad) == code
    assert call(cap=0) == tps.OK and call(cap=0, rope=None) == tps.OK


def test_pruned_attn_q8_refusals():
    l = tps.lib()
    base = dict(q=F, k=F, v=F, ks=F, vs=F, idx=F, count=F, cap=10, N=100, H=2, d=64, scale=0.1, bm=NULL, block=128,
                o=F, lse=NULL)

    def call(**kw):
        a = {**base, **kw}
        return l.pruned_attn_q8(a["q"], a["k"], a["v"], a["ks"], a["vs"], a["idx"], a["count"], a["cap"], a["N"], a["H"],
                                a["d"], a["scale"], a["bm"], a["block"], a["o"], a["lse"], NULL, 0, NULL)
    for k in ("q", "k", "v", "ks", "vs", "idx", "count", "o"):
        assert call(**{k: NULL}) == tps.INVALID_ARG, k
    for k in ("q", "k", "v", "o", "ks", "vs", "lse"):
        assert call(**{k: MIS}) == tps.ALIGN, k
    assert call(d=80) == tps.INVALID_ARG and call(H=0) == tps.SHAPE and call(H=257) == tps.SHAPE
    assert call(N=0) == tps.SHAPE and call(cap=-1) == tps.SHAPE
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == tps.INVALID_ARG
    assert call(bm=F, block=64) == tps.INVALID_ARG and call(bm=F, N=4097 * 128) == tps.SHAPE
    assert call(cap=0) == tps.OK
    assert tps.lib().tps_attn_q8_workspace_size(10, 0, 2, 64) == 0
    assert tps.lib().tps_attn_q8_workspace_size(10, 100, 2, 96) == 0


# ---- refusals of the binding (CPU tensors: everything is decided before the library is called) ------------------
def _cpu_state(N=300, H=2, d=64, A=20):
    kc, vc, ks, vs = tps.cache_q8(N, H, d, device="cpu")
    q = torch.zeros((A, H, d), dtype=torch.bfloat16)
    return kc, vc, ks, vs, q, torch.zeros(A, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)


@pytest.mark.parametrize("change", ["dtype", "shape", "strides", "idx dtype", "idx short", "scale shape", "cap"])
def test_binding_refuses_what_the_library_cannot_see(change):
    kc, vc, ks, vs, q, idx, cnt = _cpu_state()
    kw = {}
    if change == "dtype":
        q = q.half()
    elif change == "shape":
        q = q[:, :1].contiguous()
    elif change == "strides":
        q = q.transpose(0, 1).contiguous().transpose(0, 1)
    elif change == "idx dtype":
        idx = idx.long()
    elif change == "idx short":
        idx = idx[:3]
    elif change == "scale shape":
        ks = ks[:-1].contiguous()
    elif change == "cap":
        kw["cap"] = 21
    with pytest.raises(tps.TPSError):
        tps.pruned_attn_q8(q, kc, vc, ks, vs, idx, cnt, 0.1, **kw)
    with pytest.raises(tps.TPSError):
        tps.kv_sync_q8(kc, vc, ks, vs, q, q, idx, cnt, **kw)
    if change not in ("scale shape", "shape"):
        table = tps.rope_table((24, 20, 20), (3, 10, 10), device="cpu")
        with pytest.raises(tps.TPSError):
            tps.rope_rows(q, idx, cnt, table, (24, 20, 20), (3, 10, 10), **kw)


def test_binding_refuses_a_table_of_another_grid():
    kc, vc, ks, vs, q, idx, cnt = _cpu_state()
    table = tps.rope_table((24, 20, 20), (3, 10, 10), device="cpu")
    with pytest.raises(tps.TPSError):
        tps.rope_rows(q, idx, cnt, table, (24, 20, 20), (3, 10, 11))
    with pytest.raises(tps.TPSError):
        tps.kv_sync_q8(kc, vc, ks, vs, q, q, idx, cnt, rope=(table, (20, 24, 20), (3, 11, 10)))
