"""GPU parity of the rotary rows and of the 8-bit key/value cache (update and attention) with the fp64
oracle, through the binding; their edge cases; and a run of them together."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from oracle import q8_oracle as Q
from token_pruned_sparse_b200 import synth, tps

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _idx(N, A, seed):
    return np.sort(np.random.default_rng(seed).choice(N, A, replace=False)).astype(np.int32)


def _dev(idx, count=None, room=0):
    full = np.concatenate([np.asarray(idx, np.int32), np.zeros(room + (len(idx) + room == 0), np.int32)])
    n = len(idx) if count is None else count
    return torch.from_numpy(full).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)


# ---- rope_rows ---------------------------------------------------------------------------------------------
def _rope_bound(ref, x):
    """bf16 rounding (2^-8 |y|) + the fp32 turn: table entries within 2^-24, two products and a sum, so
    within 2^-22 (|a| + |b|) of the pair's exact turn."""
    a = np.abs(O.f64(x))
    pair = np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)
    return 2.0 ** -8 * np.abs(ref) + 2.0 ** -22 * pair * (1 + 2.0 ** -8) + 2.0 ** -134


@pytest.mark.parametrize("grid,H,d,A,room", [((4, 8, 8), 2, 64, 100, 28), ((1, 1, 1), 1, 64, 1, 0), ((3, 5, 7), 3, 128, 104, 1),
                                             ((2, 31, 53), 5, 64, 777, 0), ((7, 6, 5), 24, 128, 210, 3),
                                             ((2, 3, 4), 128, 128, 11, 0), ((33, 2, 3), 17, 64, 0, 5)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_rows_parity(grid, H, d, A, room, inverse):
    N = grid[0] * grid[1] * grid[2]
    dims, origin = synth.rope_dims(d), (3, -2, 500)
    idx = _idx(N, A, N + A)
    x, x2 = (synth.gaussian_bf16((A + room, H, d), 11 + i) for i in range(2))
    di, dc = _dev(idx, room=room)
    table = tps.rope_table(dims, grid, origin)
    dst = torch.full((A + room, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    dst2 = dst.clone()
    tps.rope_rows(x.to(DEV), di, dc, table, dims, grid, dst=dst, src2=x2.to(DEV), dst2=dst2, inverse=inverse)
    tps.tps_check()
    for got, src in ((dst, x), (dst2, x2)):
        ref = O.rope_rows(src[:A], idx, dims, grid, origin, inverse=inverse)
        assert np.all(np.abs(O.f64(got[:A].cpu()) - ref) <= _rope_bound(ref, src[:A]))
        assert bool((got[A:] == 7.0).all())                          # rows behind the count
    # one tensor, in place: the same bits
    y = x.to(DEV)
    tps.rope_rows(y, di, dc, table, dims, grid, dst=y, inverse=inverse)
    assert torch.equal(y[:A], dst[:A]) and torch.equal(y[A:].cpu(), x[A:])


def test_rope_rows_any_order_repeats_bounds_and_all_rows():
    grid, H, d = (3, 4, 5), 2, 64
    dims = synth.rope_dims(d)
    table = tps.rope_table(dims, grid)
    x = synth.gaussian_bf16((60, H, d), 3)
    xd = x.to(DEV)
    every = tps.rope_rows(xd, None, None, table, dims, grid)
    ref = O.rope_rows(x, np.arange(60), dims, grid)
    assert np.all(np.abs(O.f64(every.cpu()) - ref) <= _rope_bound(ref, x))
    some = tps.rope_rows(xd, None, torch.tensor([17], dtype=torch.int32, device=DEV), table, dims, grid, dst=xd.clone())
    assert torch.equal(some[:17], every[:17]) and torch.equal(some[17:], xd[17:])
    idx = np.array([9, 9, 59, 0, 33], np.int32)                       # unsorted, repeated
    di, dc = _dev(idx)
    got = tps.rope_rows(xd[:5].contiguous(), di, dc, table, dims, grid)
    ref = O.rope_rows(x[:5], idx, dims, grid)
    assert np.all(np.abs(O.f64(got.cpu()) - ref) <= _rope_bound(ref, x[:5]))
    tps.tps_check()
    di, dc = _dev(np.array([1, 60, -1, 2], np.int32))
    dst = torch.full((4, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    tps.rope_rows(xd[:4].contiguous(), di, dc, table, dims, grid, dst=dst)
    with pytest.raises(tps.TPSError) as e:
        tps.tps_check()
    assert e.value.code == tps.BOUNDS
    assert bool((dst[1:3] == 7.0).all()) and not bool((dst[[0, 3]] == 7.0).any())


def test_rope_rows_gradient_through_the_turn_back():
    """The turn back of the turned rows is the input again, within two roundings; <R x, g> = <x, R^T g>."""
    grid, H, d, A = (5, 6, 7), 3, 128, 123
    dims, idx = synth.rope_dims(d), _idx(210, 123, 4)
    table = tps.rope_table(dims, grid)
    di, dc = _dev(idx)
    x, g = (synth.gaussian_bf16((A, H, d), 20 + i) for i in range(2))
    fwd = tps.rope_rows(x.to(DEV), di, dc, table, dims, grid)
    bwd = tps.rope_rows(g.to(DEV), di, dc, table, dims, grid, inverse=True)
    lhs, rhs = (O.f64(fwd.cpu()) * O.f64(g)).sum(-1), (O.f64(x) * O.f64(bwd.cpu())).sum(-1)
    # each side is off by at most 2^-8 of the sum of its products' magnitudes, and 2^-22 for the turn
    tol = (2.0 ** -8 + 2.0 ** -20) * ((np.abs(O.f64(fwd.cpu()) * O.f64(g))).sum(-1) + (np.abs(O.f64(x) * O.f64(bwd.cpu()))).sum(-1))
    assert np.all(np.abs(lhs - rhs) <= tol * (1 + 2.0 ** -7))


# ---- kv_sync_q8 ------------------------------------------------------------------------------------------------
def _cache(N, H, d, seed, spread=True):
    """A cache of unequal blocks and heads: (values of the codes, scales) in float64."""
    rng = np.random.default_rng(seed)
    nb = (N + 127) // 128
    out = []
    for _ in range(2):
        x = rng.standard_normal((N, H, d))
        if spread:
            x = x * np.repeat(np.exp(0.7 * rng.standard_normal((nb, H))), 128, 0)[:N, :, None]
        out.append(Q.kv_sync_q8(np.zeros((N, H, d)), np.zeros((nb, H)), x, np.arange(N)))
    return out


def _to_dev(cache):
    (kv, ks), (vv, vs) = cache
    return (Q.codes_of(kv).to(DEV), Q.codes_of(vv).to(DEV), torch.from_numpy(ks).float().to(DEV),
            torch.from_numpy(vs).float().to(DEV))


def _check_codes(got, got_scale, ref, ref_scale, x=None, idx=None, slack=None):
    """Codes and scales of one tensor. slack [A, H, d]: how far the fp32 fresh value may be from the exact x (the
    turned keys; None: the values are exact, and so must the codes be)."""
    np.testing.assert_array_equal(got_scale.cpu().double().numpy(), ref_scale)
    val = Q.e4m3_decode(got.cpu().view(torch.uint8).numpy())
    if slack is None:
        np.testing.assert_array_equal(val, ref)
        return
    stale = np.setdiff1d(np.arange(ref.shape[0]), idx)
    np.testing.assert_array_equal(val[stale], ref[stale])
    per = np.repeat(ref_scale, 128, 0)[idx][:, :, None]
    per = np.where(per > 0, per, 1.0)
    v, s = np.abs(x / per), slack / per
    half = np.exp2(np.maximum(np.floor(np.log2(np.maximum(v + s, 2.0 ** -30))), -6.0) - 4.0)
    assert np.all(np.abs(val[idx] - x / per) <= half + s)


@pytest.mark.parametrize("grid,H,d,A,room", [((4, 8, 8), 2, 64, 100, 28), ((1, 1, 1), 1, 64, 1, 0), ((3, 5, 7), 3, 128, 104, 1),
                                             ((2, 31, 53), 5, 64, 777, 0), ((3, 9, 19), 24, 128, 513, 3),
                                             ((2, 8, 16), 128, 128, 200, 0), ((5, 13, 10), 7, 128, 3, 0),
                                             ((5, 13, 10), 1, 64, 0, 4)])
@pytest.mark.parametrize("turn", [False, True])
@pytest.mark.parametrize("loud", [0.2, 1.0, 6.0])
def test_kv_sync_q8_parity(grid, H, d, A, room, turn, loud):
    N = grid[0] * grid[1] * grid[2]
    dims, origin = synth.rope_dims(d), (0, 0, 7)
    idx = _idx(N, A, 3 * N + A)
    cache = _cache(N, H, d, N)
    kf, vf = ((loud * synth.gaussian_bf16((A + room, H, d), 31 + i).float()).bfloat16() for i in range(2))
    dev = _to_dev(cache)
    di, dc = _dev(idx, room=room)
    rope = (tps.rope_table(dims, grid, origin), dims, grid) if turn else None
    tps.kv_sync_q8(*dev, kf.to(DEV), vf.to(DEV), di, dc, rope=rope)
    tps.tps_check()
    x = O.rope_rows(kf[:A], idx, dims, grid, origin) if turn else O.f64(kf[:A])
    ref_k = Q.kv_sync_q8(*cache[0], x, idx)
    ref_v = Q.kv_sync_q8(*cache[1], O.f64(vf[:A]), idx)
    a = np.abs(O.f64(kf[:A]))
    slack = 2.0 ** -22 * np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1) if turn else None
    _check_codes(dev[0], dev[2], *ref_k, x, idx, slack)
    _check_codes(dev[1], dev[3], *ref_v)
    # the same update again changes nothing
    before = [t.clone() for t in dev]
    tps.kv_sync_q8(*dev, kf.to(DEV), vf.to(DEV), di, dc, rope=rope)
    assert all(torch.equal(a, b) for a, b in zip(before, dev))


def test_kv_sync_q8_whole_blocks_lower_the_scale_and_partial_last_block():
    N, H, d = 300, 2, 64                                            # blocks of 128, 128, 44
    cache = _cache(N, H, d, 8)
    idx = np.concatenate([np.arange(128), np.arange(256, 300)]).astype(np.int32)
    kf, vf = ((2.0 ** -6 * synth.gaussian_bf16((len(idx), H, d), 41 + i).float()).bfloat16() for i in range(2))
    dev = _to_dev(cache)
    tps.kv_sync_q8(*dev, kf.to(DEV), vf.to(DEV), *_dev(idx))
    for c, (f, i) in zip(cache, ((kf, 0), (vf, 1))):
        ref = Q.kv_sync_q8(*c, O.f64(f), idx)
        _check_codes(dev[i], dev[2 + i], *ref)
        assert (ref[1][0] < c[1][0]).all() and (ref[1][2] < c[1][2]).all() and (ref[1][1] == c[1][1]).all()


def test_kv_sync_q8_empty_cache_zero_rows_and_odd_old_scales():
    N, H, d = 256, 2, 128
    kc, vc, ks, vs = tps.cache_q8(N, H, d, DEV)
    idx = _idx(128, 50, 1)
    kf, vf = synth.gaussian_bf16((50, H, d), 51), torch.zeros((50, H, d), dtype=torch.bfloat16)
    tps.kv_sync_q8(kc, vc, ks, vs, kf.to(DEV), vf.to(DEV), *_dev(idx))
    zero = (np.zeros((N, H, d)), np.zeros((2, H)))
    _check_codes(kc, ks, *Q.kv_sync_q8(*zero, O.f64(kf), idx))
    assert bool((vs == 0).all()) and bool((vc.view(torch.uint8) & 0x7F == 0).all())
    # a NaN or negative old scale is no scale; one that is no power of two is kept while it is the larger
    cache = _cache(N, H, d, 9)
    dev = _to_dev(cache)
    dev[2][0, 0], dev[2][0, 1], dev[3][0, 0] = float("nan"), -1.0, 3.0
    tps.kv_sync_q8(*dev, kf.to(DEV), kf.to(DEV), *_dev(idx))
    tps.tps_check()
    (kv, ksc), (vv, vsc) = cache
    ksc, vsc = ksc.copy(), vsc.copy()
    ksc[0], vsc[0, 0] = 0.0, 3.0
    _check_codes(dev[0], dev[2], *Q.kv_sync_q8(kv, ksc, O.f64(kf), idx))
    ref = Q.kv_sync_q8(vv, vsc, O.f64(kf), idx)
    np.testing.assert_array_equal(dev[3].cpu().double().numpy(), ref[1])
    got = Q.e4m3_decode(dev[1].cpu().numpy())
    # x * (1 / 3): two roundings of 2^-24 before the code's half step
    v = np.abs(O.f64(kf)[:, 0] / 3.0)
    half = np.exp2(np.maximum(np.floor(np.log2(np.maximum(v * (1 + 2.0 ** -22), 2.0 ** -30))), -6.0) - 4.0)
    assert np.all(np.abs(got[idx, 0] - O.f64(kf)[:, 0] / 3.0) <= half + 2.0 ** -22 * v)


def test_kv_sync_q8_infinities_and_nan():
    N, H, d = 128, 1, 64
    cache = _cache(N, H, d, 10)
    idx = _idx(N, 40, 2)
    vf = synth.gaussian_bf16((40, H, d), 61)
    vf[0, 0, 0], vf[1, 0, 1], vf[2, 0, 2] = float("inf"), float("-inf"), float("nan")
    dev = _to_dev(cache)
    tps.kv_sync_q8(*dev, vf.to(DEV), vf.to(DEV), *_dev(idx))
    for i in range(2):
        _check_codes(dev[i], dev[2 + i], *Q.kv_sync_q8(*cache[i], O.f64(vf), idx))
    tps.tps_check()


def test_kv_sync_q8_flags_bad_lists_and_keeps_other_rows():
    N, H, d = 300, 2, 64
    cache = _cache(N, H, d, 11)
    kf, vf = (synth.gaussian_bf16((6, H, d), 71 + i) for i in range(2))
    for idx, good in ((np.array([3, 3, 9, 140, 141, 299], np.int32), [0, 2, 3, 4, 5]),      # repeated: the first counts
                      (np.array([3, 5, 9, 140, 141, 300], np.int32), [0, 1, 2, 3, 4]),      # behind the last token
                      (np.array([-4, 5, 9, 140, 141, 299], np.int32), [1, 2, 3, 4, 5])):
        dev = _to_dev(cache)
        tps.kv_sync_q8(*dev, kf.to(DEV), vf.to(DEV), *_dev(idx))
        with pytest.raises(tps.TPSError) as e:
            tps.tps_check()
        assert e.value.code == tps.BOUNDS
        _check_codes(dev[1], dev[3], *Q.kv_sync_q8(*cache[1], O.f64(vf)[good], idx[good]))


# ---- pruned_attn_q8 ----------------------------------------------------------------------------------------------
def _attn_case(N, A, H, d, seed, spread=True, q_amp=1.0):
    cache = _cache(N, H, d, seed, spread)
    q = (q_amp * synth.gaussian_bf16((A, H, d), seed + 1).float()).bfloat16()
    return cache, q, _idx(N, A, seed + 2)


def _values(cache):
    return [v * np.repeat(s, 128, 0)[: v.shape[0], :, None] for v, s in cache]


def _run_attn(cache, q, idx, scale, bm=None, room=0, ws=None, lse=True, dev=None):
    A, H, d = q.shape
    dev = _to_dev(cache) if dev is None else dev
    qd = torch.cat([q, torch.full((room, H, d), float("nan"), dtype=torch.bfloat16)]).to(DEV)
    o = torch.full((A + room, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    l = torch.full((A + room, H), 7.0, device=DEV) if lse else None
    di, dc = _dev(idx, room=room)
    tps.pruned_attn_q8(qd, *dev, di, dc, scale, blockmask=None if bm is None else torch.from_numpy(bm).to(DEV),
                       o_act=o, lse=l, ws=ws)
    tps.tps_check()
    assert bool((o[A:] == 7.0).all()) and (l is None or bool((l[A:] == 7.0).all()))   # rows behind the count
    return O.f64(o[:A].cpu()), None if l is None else l[:A].cpu().double().numpy()


def _check_attn(o, lse, cache, q, idx, scale, bm=None):
    k, v = _values(cache)
    ref, rlse = O.pruned_attn(q, k, v, idx, scale, blockmask=bm)
    ot, lt = Q.q8_attn_bound(q, k, v, cache[1][1], idx, scale, bm)
    err = np.abs(o - ref)
    assert np.all(err <= ot), (float(err.max()), float((err / ot).max()))
    if lse is not None:
        fin = np.isfinite(rlse)
        assert np.array_equal(np.isneginf(lse), ~fin)
        miss = np.abs(lse[fin] - rlse[fin])
        assert np.all(miss <= lt[fin]), float((miss / lt[fin]).max())


ATTN = [(1, 1, 1, 64), (1, 1, 1, 128), (127, 5, 2, 64), (128, 128, 1, 128), (129, 129, 4, 128), (256, 256, 2, 64),
        (300, 113, 2, 64), (517, 131, 3, 128), (1000, 1, 1, 128), (1000, 257, 2, 128), (2000, 1999, 1, 128),
        (4099, 700, 2, 64), (6000, 33, 5, 128), (9001, 17, 3, 64)]


@pytest.mark.parametrize("N,A,H,d", ATTN)
@pytest.mark.parametrize("sharp", [False, True])
def test_attn_q8_dense(N, A, H, d, sharp):
    cache, q, idx = _attn_case(N, A, H, d, N + A)
    scale = 0.35 if sharp else 1.0 / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale, room=3)
    _check_attn(o, lse, cache, q, idx, scale)


@pytest.mark.parametrize("N,A,H,d", [(1, 1, 3, 64), (15, 8, 2, 128), (129, 9, 2, 64), (300, 16, 2, 128), (1000, 2, 24, 128),
                                     (5003, 16, 3, 64), (9001, 9, 2, 128), (20280, 1, 12, 128), (2049, 3, 128, 64)])
@pytest.mark.parametrize("sharp", [False, True])
def test_attn_q8_few_rows(N, A, H, d, sharp):
    cache, q, idx = _attn_case(N, A, H, d, N + A)
    scale = 0.35 if sharp else 1.0 / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale, room=3)
    _check_attn(o, lse, cache, q, idx, scale)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    o1, _ = _run_attn(cache, q, idx, scale, ws=none, lse=False)       # one key range per head
    _check_attn(o1, None, cache, q, idx, scale)


def test_attn_q8_full_waves_then_a_split_tail():
    """More row tiles than one wave of this GPU holds: the last ones go in a second, split launch."""
    N, A, H, d = 2100, 2000, 24, 64
    cache, q, idx = _attn_case(N, A, H, d, 3)
    scale = 1.0 / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale, room=5)
    _check_attn(o, lse, cache, q, idx, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [3, 16, 60, 128, 300])
@pytest.mark.parametrize("where", [[0], [1], [17], list(range(0, 20, 2)), list(range(1, 20, 2)), list(range(20))])
def test_attn_q8_nan_keys_reach_every_row(d, A, where):
    """A key block whose codes are all NaN makes every attending row NaN, whichever key range, stream or warp sees
    it and even where that part sees nothing else."""
    N, H = 20 * 128 - 5, 1
    cache, q, idx = _attn_case(N, A, H, d, 41)
    dev = list(_to_dev(cache))
    for b in where:
        dev[0][b * 128:(b + 1) * 128] = 0x7F
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        o, lse = _run_attn(cache, q, idx, 1.0 / math.sqrt(d), dev=dev, ws=ws)
        assert np.isnan(o).all() and np.isnan(lse).all()


@pytest.mark.parametrize("N,A,H,d", [(6000, 33, 5, 128), (4099, 700, 2, 64)])
def test_attn_q8_without_workspace_and_without_lse(N, A, H, d):
    cache, q, idx = _attn_case(N, A, H, d, 5)
    scale = 1.0 / math.sqrt(d)
    none = torch.empty(0, dtype=torch.uint8, device=DEV)
    o, lse = _run_attn(cache, q, idx, scale, ws=none)
    _check_attn(o, lse, cache, q, idx, scale)
    o2, _ = _run_attn(cache, q, idx, scale, ws=none, lse=False)
    assert np.array_equal(o, o2)


@pytest.mark.parametrize("N,A,H,d,keep", [(300, 113, 2, 64, 2), (1000, 600, 2, 128, 3), (2000, 1999, 1, 128, 7),
                                          (1290, 40, 3, 64, 1), (4099, 700, 2, 128, 20)])
def test_attn_q8_blocks(N, A, H, d, keep):
    cache, q, idx = _attn_case(N, A, H, d, N + A)
    nb = (N + 127) // 128
    rng = np.random.default_rng(keep)
    bm = (rng.random((nb, nb)).argsort(1) < keep).astype(np.uint8)
    bm[idx[0] // 128] = 0                                            # a query block that keeps nothing
    scale = 1.0 / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale, bm=bm, room=2)
    _check_attn(o, lse, cache, q, idx, scale, bm)
    gone = idx // 128 == idx[0] // 128
    assert not o[gone].any() and np.isneginf(lse[gone]).all()


@pytest.mark.parametrize("d", [64, 128])
def test_attn_q8_nan_only_where_it_is_attended(d):
    """NaN codes and NaN scales in key blocks that no query keeps leave every result alone; one in a kept block
    reaches the rows that keep it, and no other."""
    N, H = 900, 2
    cache, q, idx = _attn_case(N, 500, H, d, 77)
    nb = 8
    bm = np.ones((nb, nb), np.uint8)
    bm[:, 3] = 0
    bm[2, 3] = 1                                                     # only query block 2 keeps key block 3
    scale = 1.0 / math.sqrt(d)
    clean, clean_l = _run_attn(cache, q, idx, scale, bm=bm)
    dev = list(_to_dev(cache))
    dev[0][3 * 128 + 5, 0, 1] = 0x7F
    dev[1][3 * 128 + 9] = 0xFF
    o, lse = _run_attn(cache, q, idx, scale, bm=bm, dev=dev)
    hit = idx // 128 == 2
    assert np.array_equal(o[~hit], clean[~hit]) and np.array_equal(lse[~hit], clean_l[~hit])
    assert np.isnan(o[hit]).all() and np.isnan(lse[hit][:, 0]).all()
    np.testing.assert_array_equal(lse[hit][:, 1], clean_l[hit][:, 1])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [200, 100, 11])
def test_attn_q8_rising_maxima_force_rescales(d, A):
    """Keys that grow along the cache: the running maximum moves again and again, far beyond what f16 holds."""
    N, H = 1500, 1
    rng = np.random.default_rng(3)
    u = rng.standard_normal(d)
    grow = np.linspace(0.1, 12.0, N)[:, None, None]
    k = u[None, None] * grow + 0.1 * rng.standard_normal((N, H, d))
    v = rng.standard_normal((N, H, d)) * np.repeat(2.0 ** rng.integers(-6, 7, 12), 128)[:N, None, None]
    zero = (np.zeros((N, H, d)), np.zeros((12, H)))
    cache = [Q.kv_sync_q8(*zero, x, np.arange(N)) for x in (k, v)]
    q = torch.from_numpy(u[None, None] * rng.choice([-1.0, 1.0], (A, 1, 1)) + 0.1 * rng.standard_normal((A, H, d))).bfloat16()
    idx = _idx(N, A, 4)
    for scale in (1.0 / math.sqrt(d), 1.0):
        o, lse = _run_attn(cache, q, idx, scale)
        _check_attn(o, lse, cache, q, idx, scale)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [150, 40, 5])
def test_attn_q8_scales_zero_far_apart_and_any_number(d, A):
    N, H = 700, 2
    cache, q, idx = _attn_case(N, A, H, d, 31)
    (kv, ks), (vv, vs) = cache
    ks, vs = ks.copy(), vs.copy()
    ks[1], vs[2] = 0.0, 0.0                                          # values of 0 under those blocks
    vs[4] *= 2.0 ** 30
    ks[3] = np.float32(0.0123)
    vs[3] = np.float32(0.0077)
    cache = [(kv, ks), (vv, vs)]
    o, lse = _run_attn(cache, q, idx, 1.0 / math.sqrt(d))
    _check_attn(o, lse, cache, q, idx, 1.0 / math.sqrt(d))


def test_attn_q8_queries_of_every_magnitude():
    """Rows from 2^-90 to 2^60 in size, a zero row, rows with one outlying channel, and an infinite entry."""
    N, H, d = 400, 1, 128
    cache, q, _ = _attn_case(N, 8, H, d, 91, spread=False)
    q = q.float()
    q[0] *= 2.0 ** -90
    q[1] = 0
    q[2, 0, 5] = 4000.0
    q[3, 0, ::2] *= 2.0 ** -12
    q[4] *= 2.0 ** 10
    q = q.bfloat16()
    idx = _idx(N, 8, 1)
    o, lse = _run_attn(cache, q, idx, 2.0 ** -10)
    _check_attn(o, lse, cache, q, idx, 2.0 ** -10)
    q[7, 0, 3] = float("inf")
    bad, bl = _run_attn(cache, q, idx, 2.0 ** -10)
    assert np.isnan(bad[7]).all() and np.isnan(bl[7]).all()
    # a NaN row makes its warp look for new maxima: its neighbours' probabilities are then rounded against
    # another reference, each again within 2^-11, so the same bound holds (not the same bits)
    _check_attn(bad[:7], bl[:7], cache, q[:7], idx[:7], 2.0 ** -10)


def test_attn_q8_active_count_below_cap_and_zero():
    N, A, H, d = 3000, 700, 2, 128
    cache, q, idx = _attn_case(N, A, H, d, 13)
    scale = 1.0 / math.sqrt(d)
    dev = _to_dev(cache)
    full, _ = _run_attn(cache, q, idx, scale, dev=dev)
    for n in (0, 1, 129, 300):
        o = torch.full((A, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
        tps.pruned_attn_q8(q.to(DEV), *dev, *_dev(idx, count=n), scale, o_act=o)
        tps.tps_check()
        assert bool((o[n:] == 7.0).all())
        ot, _ = Q.q8_attn_bound(q[:n], *_values(cache), cache[1][1], idx[:n], scale) if n else (0, 0)
        assert np.all(np.abs(O.f64(o[:n].cpu()) - full[:n]) <= 2 * ot)


def test_attn_q8_bounds_flag_with_mask():
    N, H, d = 300, 1, 64
    cache, q, _ = _attn_case(N, 4, H, d, 17)
    bm = np.ones((3, 3), np.uint8)
    good = np.array([5, 140, 299], np.int32)
    ref, _ = _run_attn(cache, q[:3], good, 0.125, bm=bm)
    o = torch.full((4, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    tps.pruned_attn_q8(q.to(DEV), *_to_dev(cache), *_dev(np.array([5, 140, 299, 300], np.int32)), 0.125,
                       blockmask=torch.from_numpy(bm).to(DEV), o_act=o)
    with pytest.raises(tps.TPSError) as e:
        tps.tps_check()
    assert e.value.code == tps.BOUNDS
    assert np.array_equal(O.f64(o[:3].cpu()), ref) and bool((o[3] == 7.0).all())


# ---- together, and how they are called -----------------------------------------------------------------------------
def _step(grid, H, d, A, seed):
    N = grid[0] * grid[1] * grid[2]
    dims = synth.rope_dims(d)
    return dict(N=N, dims=dims, grid=grid, idx=_idx(N, A, seed), scale=1.0 / math.sqrt(d),
                full=[synth.gaussian_bf16((N, H, d), seed + i) for i in range(2)],
                act=[synth.gaussian_bf16((A, H, d), seed + 5 + i) for i in range(3)])


@pytest.mark.parametrize("grid,H,d,A", [((4, 8, 8), 2, 64, 100), ((5, 13, 21), 3, 128, 400)])
def test_a_step_over_the_8_bit_cache(grid, H, d, A):
    """Fill the cache, then one pruned step: turn Q, update the cache with turned K, attend, restore."""
    s = _step(grid, H, d, A, 7)
    N, idx, dims = s["N"], s["idx"], s["dims"]
    table = tps.rope_table(dims, grid)
    kc, vc, ks, vs = tps.cache_q8(N, H, d)
    every = torch.arange(N, dtype=torch.int32, device=DEV)
    tps.kv_sync_q8(kc, vc, ks, vs, *(t.to(DEV) for t in s["full"]), every,
                   torch.tensor([N], dtype=torch.int32, device=DEV), rope=(table, dims, grid))
    q, k, v = (t.to(DEV) for t in s["act"])
    di, dc = _dev(idx)
    qr = tps.rope_rows(q, di, dc, table, dims, grid)
    tps.kv_sync_q8(kc, vc, ks, vs, k, v, di, dc, rope=(table, dims, grid))
    o = tps.pruned_attn_q8(qr, kc, vc, ks, vs, di, dc, s["scale"])
    out = torch.full((N, H, d), 3.0, dtype=torch.bfloat16, device=DEV)
    tps.scatter_out(out, o, di, dc)
    tps.tps_check()
    cache = [(Q.e4m3_decode(c.cpu().view(torch.uint8).numpy()), sc.cpu().double().numpy()) for c, sc in ((kc, ks), (vc, vs))]
    _check_attn(O.f64(o.cpu()), None, cache, qr.cpu(), idx, s["scale"])
    assert torch.equal(out[di.long()], o) and bool((out[np.setdiff1d(np.arange(N), idx)] == 3.0).all())
    # against the step in 64 bits from the bf16 inputs, nothing rounded in between: the cache's values are within
    # 2^-4 (half a step of e4m3) of the exact ones (or 2^-10 of the scale), and so is a mean of them
    kx = O.rope_rows(s["full"][0], np.arange(N), dims, grid)
    kx[idx] = O.rope_rows(s["act"][1], idx, dims, grid)
    vx = O.f64(s["full"][1]).copy()
    vx[idx] = O.f64(s["act"][2])
    for (c, sc), x in zip(cache, (kx, vx)):
        per = np.repeat(sc, 128, 0)[:N, :, None]
        assert np.all(np.abs(c * per - x) <= 2.0 ** -4 * np.abs(x) * (1 + 2.0 ** -16) + 2.0 ** -10 * per + 2.0 ** -20)


def test_another_stream_a_captured_step_and_repeats_agree():
    grid, H, d, A = (5, 13, 21), 3, 128, 400
    s = _step(grid, H, d, A, 9)
    N, dims = s["N"], s["dims"]
    table = tps.rope_table(dims, grid)
    di, dc = _dev(s["idx"])
    q, k, v = (t.to(DEV) for t in s["act"])
    start = _to_dev(_cache(N, H, d, 3))
    ws = tps.attn_q8_workspace(A, N, H, d)

    def step(cache, qr, o, lse, w):
        tps.rope_rows(q, di, dc, table, dims, grid, dst=qr)
        tps.kv_sync_q8(*cache, k, v, di, dc, rope=(table, dims, grid))
        tps.pruned_attn_q8(qr, *cache, di, dc, s["scale"], o_act=o, lse=lse, ws=w)

    def buffers():
        return [t.clone() for t in start], torch.empty_like(q), torch.empty_like(q), torch.empty((A, H), device=DEV)

    ref = buffers()
    step(*ref, ws)
    tps.tps_check()
    other = torch.cuda.Stream()
    two = buffers()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        step(*two, None)
    torch.cuda.current_stream().wait_stream(other)
    tps.tps_check()
    three = buffers()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(*three, ws)
    for t, f in zip(three[0], start):
        t.copy_(f)
    g.replay()
    torch.cuda.synchronize()
    tps.tps_check()
    for got in (two, three):
        for a, b in zip(ref[0] + list(ref[1:]), got[0] + list(got[1:])):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    """Calls in flight on two streams share nothing: each gives what it gives alone."""
    jobs = []
    for N, A, H, d, seed in ((3000, 700, 3, 128, 1), (6000, 9, 5, 64, 2)):
        cache, q, idx = _attn_case(N, A, H, d, seed)
        jobs.append((q.to(DEV), _to_dev(cache), _dev(idx), 1.0 / math.sqrt(d), torch.cuda.Stream()))
    alone = [tps.pruned_attn_q8(q, *c, *i, s) for q, c, i, s, _ in jobs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for k, (q, c, i, s, st) in enumerate(jobs):
            with torch.cuda.stream(st):
                got[k].append(tps.pruned_attn_q8(q, *c, *i, s))
    torch.cuda.synchronize()
    tps.tps_check()
    for a, outs in zip(alone, got):
        assert all(torch.equal(a, o) for o in outs)
    # the same with the stream given by argument, and as a raw handle
    q, c, i, s, st = jobs[0]
    for handle in (st, st.cuda_stream):
        o = torch.empty_like(q)
        st.wait_stream(torch.cuda.current_stream())
        tps.pruned_attn_q8(q, *c, *i, s, o_act=o, stream=handle)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(o, alone[0])


@pytest.mark.parametrize("raw", [False, True])
def test_outputs_made_for_another_stream_wait_for_the_memory(raw):
    """With stream= given, an output may get memory that the current stream still reads: the call waits for it."""
    grid, H, d = (5, 20, 20), 4, 128
    N, dims = 2000, synth.rope_dims(128)
    table = tps.rope_table(dims, grid)
    cache, q, idx = _attn_case(N, N, H, d, 11)
    q, cache, idx = q.to(DEV), _to_dev(cache), _dev(idx)
    other = torch.cuda.Stream()
    want = tps.rope_rows(q, None, None, table, dims, grid)
    want_o = tps.pruned_attn_q8(q, *cache, *idx, 0.1)
    torch.cuda.synchronize()
    for call, ref in ((lambda st: tps.rope_rows(q, None, None, table, dims, grid, stream=st), want),
                      (lambda st: tps.pruned_attn_q8(q, *cache, *idx, 0.1, stream=st), want_o)):
        victim = torch.full_like(q, 3.0)
        torch.cuda.synchronize()
        torch.cuda._sleep(20_000_000)            # about 10 ms ahead of the read of victim
        read = victim + 1.0
        del victim
        out = call(other.cuda_stream if raw else other)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
        assert bool((read == 4.0).all())
    tps.tps_check()


def test_two_captured_graphs_share_a_workspace_and_one_makes_its_own():
    N, A, H, d = 4000, 100, 3, 128               # few rows of work: the keys are split
    ws = tps.attn_q8_workspace(A, N, H, d)
    assert ws.numel() > 0
    jobs = []
    for seed in (1, 2, 3):
        cache, q, idx = _attn_case(N, A, H, d, seed)
        q, cache, idx = q.to(DEV), _to_dev(cache), _dev(idx)
        want = tps.pruned_attn_q8(q, *cache, *idx, 0.1)
        o, g = torch.empty_like(q), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            tps.pruned_attn_q8(q, *cache, *idx, 0.1, o_act=o, ws=None if seed == 3 else ws)
        jobs.append((g, o, want, (q, cache, idx)))
    for _ in range(3):
        for g, o, *_ in jobs:
            o.fill_(float("nan"))
        for g, *_ in jobs:                       # one after the other on one stream
            g.replay()
        torch.cuda.synchronize()
        for _, o, want, _ in jobs:
            assert torch.equal(o, want)
    tps.tps_check()


def test_empty_lists_and_zero_capacity():
    H, d, N = 2, 64, 200
    cache, q, _ = _attn_case(N, 5, H, d, 4)
    cache, q = _to_dev(cache), q.to(DEV)
    before = [t.view(torch.uint8).clone() for t in cache]
    none = (torch.empty(0, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV))
    empty = q[:0]
    assert tps.pruned_attn_q8(empty, *cache, *none, 0.1).shape == (0, H, d)
    tps.kv_sync_q8(*cache, empty, empty, *none)
    dims, grid = synth.rope_dims(64), (1, 10, 20)
    assert tps.rope_rows(empty, *none, tps.rope_table(dims, grid), dims, grid).shape == (0, H, d)
    o = torch.full_like(q, 7.0)
    tps.pruned_attn_q8(q, *cache, *_dev(np.arange(5), 0), 0.1, o_act=o)      # capacity 5, none active
    tps.kv_sync_q8(*cache, q, q, *_dev(np.arange(5), 0))
    assert bool((o == 7.0).all())
    assert all(torch.equal(a, b.view(torch.uint8)) for a, b in zip(before, cache))
    tps.tps_check()


def test_a_chunk_of_frames_with_an_origin():
    """Streaming: a window of the video, its first frame at position 7, gives the keys of the whole video's table."""
    H, d, grid = 2, 128, (3, 4, 5)
    N, dims = 60, synth.rope_dims(128)
    k = synth.gaussian_bf16((N, H, d), 5)
    every = torch.arange(N, dtype=torch.int32, device=DEV)
    count = torch.tensor([N], dtype=torch.int32, device=DEV)
    got = []
    long_grid = (10, 4, 5)
    for table, g, shift in ((tps.rope_table(dims, grid, origin=(7, 0, 0)), grid, 0),
                            (tps.rope_table(dims, long_grid), long_grid, 7 * 20)):
        n = g[0] * g[1] * g[2]
        cache = tps.cache_q8(n, H, d)
        tps.kv_sync_q8(*cache, k.to(DEV), k.to(DEV), every + shift, count, rope=(table, dims, g))
        got.append((tps.rope_rows(k.to(DEV), every + shift, count, table, dims, g), cache))
    tps.tps_check()
    assert torch.equal(got[0][0], got[1][0])
    a = Q.q8_values(got[0][1][0].cpu().view(torch.uint8).numpy(), got[0][1][2].cpu().numpy())
    b = Q.q8_values(got[1][1][0].cpu().view(torch.uint8).numpy(), got[1][1][2].cpu().numpy())[140:200]
    # the same values on grids whose scales may differ by a power of two: equal where both are normal
    big = np.abs(a) >= 2.0 ** -6 * np.maximum(got[0][1][2].cpu().numpy().max(), got[1][1][2].cpu().numpy().max())
    np.testing.assert_array_equal(a[big], b[big])


def test_offsets_beyond_32_bits():
    """A cache of more than 2^32 code bytes: the last blocks are written and attended at their own place."""
    H, d = 128, 128
    N = (1 << 18) + 200                                              # N * H * d = 4.3e9 bytes a tensor
    kc, vc, ks, vs = tps.cache_q8(N, H, d)
    idx = np.concatenate([np.arange(64), np.arange(N - 200, N)]).astype(np.int32)
    k, v, q = (synth.gaussian_bf16((len(idx), H, d), 80 + i) for i in range(3))
    grid, dims = (1, 8, N // 8), synth.rope_dims(d)
    table = tps.rope_table(dims, grid)
    di, dc = _dev(idx)
    tps.kv_sync_q8(kc, vc, ks, vs, k.to(DEV), v.to(DEV), di, dc, rope=(table, dims, grid))
    tps.tps_check()
    rows = torch.from_numpy(idx).long().to(DEV)
    for h in (0, 127):
        for codes, sc, x in ((kc, ks, O.rope_rows(k[:, h:h + 1], idx, dims, grid)), (vc, vs, O.f64(v[:, h:h + 1]))):
            per = sc[rows // 128, h].cpu().double().numpy()[:, None]
            got = Q.e4m3_decode(codes.view(torch.uint8)[rows, h].cpu().numpy()) * per
            assert np.all(np.abs(got - x[:, 0]) <= 2.0 ** -4 * np.abs(x[:, 0]) * (1 + 2.0 ** -12) + 2.0 ** -10 * per + 2.0 ** -12)
    # a mask that keeps only the last key blocks for the last query block
    assert int((kc.view(torch.uint8)[64:N - 200] != 0).sum()) == 0
    scale = 0.5
    few = slice(len(idx) - 3, len(idx))
    o = tps.pruned_attn_q8(q[few].contiguous().to(DEV), kc, vc, ks, vs, *_dev(idx[few]), scale)
    tps.tps_check()
    h = 127
    kd = torch.zeros((N, d), dtype=torch.float64)
    vd = torch.zeros((N, d), dtype=torch.float64)
    for codes, sc, to in ((kc, ks, kd), (vc, vs, vd)):
        per = sc[rows // 128, h].cpu().double().numpy()[:, None]
        to[torch.from_numpy(idx).long()] = torch.from_numpy(Q.e4m3_decode(codes.view(torch.uint8)[rows, h].cpu().numpy()) * per)
    qh = q[few][:, h:h + 1]
    ref, _ = O.pruned_attn(qh, kd[:, None].numpy(), vd[:, None].numpy(), idx[few], scale)
    ot, _ = Q.q8_attn_bound(qh, kd[:, None].numpy(), vd[:, None].numpy(), vs[:, h:h + 1].cpu().double().numpy(), idx[few], scale)
    assert np.all(np.abs(O.f64(o[:, h:h + 1].cpu()) - ref) <= ot)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A,keep", [(900, 11), (900, 3), (100, 0), (17, 0)])
def test_attn_q8_one_set_calls_repeat_bit_for_bit_beside_a_copy(A, keep, d):
    """Calls whose two issuers share the key ring, over a cache that a copy on another stream drives out of L2: a load
    may land late, and every call still gives the same bits, within the bound."""
    N, H = 6000, 4
    cache, q, idx = _attn_case(N, A, H, d, 29)
    nb = (N + 127) // 128
    bm = (np.random.default_rng(keep).random((nb, nb)).argsort(1) < keep).astype(np.uint8) if keep else None
    scale = 1.0 / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale, bm=bm)
    _check_attn(o, lse, cache, q, idx, scale, bm)
    qd, dev, act = q.to(DEV), _to_dev(cache), _dev(idx)
    mask = None if bm is None else torch.from_numpy(bm).to(DEV)
    ws = None if keep else tps.attn_q8_workspace(A, N, H, d)
    big, other = torch.zeros(1 << 28, dtype=torch.uint8, device=DEV), torch.cuda.Stream()
    to = torch.empty_like(big)
    want, bad = torch.from_numpy(o).bfloat16().to(DEV), torch.zeros((), dtype=torch.int64, device=DEV)
    got = torch.empty_like(qd)
    torch.cuda.synchronize()
    for i in range(1500):
        if i % 3 == 0:
            with torch.cuda.stream(other):
                to.copy_(big)
        tps.pruned_attn_q8(qd, *dev, *act, scale, blockmask=mask, o_act=got, ws=ws)
        bad += (got != want).sum()
    torch.cuda.synchronize()
    tps.tps_check()
    assert int(bad) == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [3, 16, 60, 300])
@pytest.mark.parametrize("split", [False, True])
def test_attn_q8_nan_values_reach_every_row_however_small_their_weight(d, A, split):
    """A NaN code of V makes its channel NaN in every row that attends it, also where its key range, stream or warp has
    a weight that is zero in fp32 (256 nats and more below the others)."""
    N, H = 20 * 128 - 5, 1
    rng = np.random.default_rng(5)
    u = rng.choice([-1.0, 1.0], d)
    low = (np.arange(N) // 128 % 2 == 1) | (np.arange(N) < 512)       # odd blocks, and the first four
    k = np.where(low, -16.0, 16.0)[:, None, None] * u
    v = rng.standard_normal((N, H, d))
    zero = (np.zeros((N, H, d)), np.zeros((20, H)))
    cache = [Q.kv_sync_q8(*zero, x, np.arange(N)) for x in (k, v)]
    q = torch.from_numpy(np.broadcast_to(u, (A, H, d)).copy()).bfloat16()
    idx = _idx(N, A, 3)
    ws = None if split else torch.empty(0, dtype=torch.uint8, device=DEV)
    scale = 0.125
    o, lse = _run_attn(cache, q, idx, scale, ws=ws)
    _check_attn(o, lse, cache, q, idx, scale)
    for b in (0, 1, 5, 19):                                           # all of them low
        dev = list(_to_dev(cache))
        dev[1][b * 128 + 7, 0, 9] = 0x7F
        got, glse = _run_attn(cache, q, idx, scale, dev=dev, ws=ws)
        assert np.isnan(got[:, 0, 9]).all(), b
        rest = np.delete(np.arange(d), 9)
        assert np.array_equal(got[..., rest], o[..., rest]) and np.array_equal(glse, lse)


# per block of 128 keys: (log2 of V's scale or None for 0, the keys' logit in log2 units)
SPREADS = {
    "two empty blocks": [(0, 0)] * 2 + [(None, 0)] * 2 + [(0, 0)] * 8,
    "empty beside 2^30": [(30, 0), (None, 0)] * 6,
    "empty beside 2^30, reversed": [(None, 0), (30, 0)] * 6,
    "one block 2^200 above the rest": [(-100, 0)] * 5 + [(100, 0)] + [(-100, 0)] * 6,
    "the weight on small values, large ones first": [(100, -250)] + [(-100, 0)] * 11,
    "the weight on small values, large ones last": [(-100, 0)] * 11 + [(100, -250)],
    "large and small values that count alike": [(-100, 0), (100, -198)] * 6,
    "the same, other way round": [(100, -198), (-100, 0)] * 6,
    "the weight on empty blocks": [(None, 40)] * 6 + [(0, 0)] * 6,
    "the weight on empty blocks behind": [(0, 0)] * 6 + [(None, 40)] * 6,
    "a little weight on empty blocks": [(0, 0)] * 3 + [(None, -12)] * 9,
    "half of the weight on a block 2^70 below": [(-40, 0), (30, 0)] * 6,
    "steps of 2^50": [(-100 + 50 * (i % 5), -10 * (i % 3)) for i in range(12)],
    "weights of 2^-150 on values that are 2^167 larger": [(-72, 150)] * 6 + [(95, 0)] * 6,
    "the same, larger values first": [(95, 0)] * 6 + [(-72, 150)] * 6,
    "all empty": [(None, 3 * (i % 2)) for i in range(12)],
    "all small": [(-100, i) for i in range(12)],
    "all large": [(100, -i) for i in range(12)],
}


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A,masked", [(5, False), (16, False), (60, False), (128, False), (300, False), (300, True)])
@pytest.mark.parametrize("name", list(SPREADS))
def test_attn_q8_sums_hold_over_the_whole_range_of_value_scales(name, A, masked, d):
    """Scales of V from 0 over 2^-100 to 2^100 in one head: a key counts in the sum whatever its V's scale is."""
    H, N = 2, 12 * 128 - 5
    rng = np.random.default_rng(7)
    u, scale = rng.choice([-1.0, 1.0], d), 0.25
    blocks = SPREADS[name]
    at = np.array([x for _, x in blocks], float) * math.log(2) / (scale * d)
    k = at[np.arange(N) // 128][:, None, None] * u + 0.02 * rng.standard_normal((N, H, d))
    cache = [Q.kv_sync_q8(np.zeros((N, H, d)), np.zeros((12, H)), x, np.arange(N)) for x in (k, rng.standard_normal((N, H, d)))]
    vs = np.array([0.0 if e is None else 2.0 ** e for e, _ in blocks])[:, None].repeat(H, 1)
    cache[1] = (cache[1][0], vs)
    q = torch.from_numpy(u + 0.02 * rng.standard_normal((A, H, d))).bfloat16()
    idx = _idx(N, A, 3)
    bm = np.ones((12, 12), np.uint8) if masked else None
    kk, vv = _values(cache)
    ref, rlse = O.pruned_attn(q, kk, vv, idx, scale, blockmask=bm)
    ot, lt = Q.q8_attn_bound(q, kk, vv, vs, idx, scale, bm, floor=2.0 ** -25)
    for ws in (None, torch.empty(0, dtype=torch.uint8, device=DEV)):
        o, lse = _run_attn(cache, q, idx, scale, bm=bm, ws=None if masked else ws)
        assert np.all(np.abs(lse - rlse) <= lt), float((np.abs(lse - rlse) / lt).max())
        # bf16 and fp32 hold normal numbers down to 2^-126; what is smaller may become 0
        assert np.all(np.abs(o - ref) <= ot + 2.0 ** -126), float((np.abs(o - ref) / ot).max())


def _one_loud_key(A, d, loud, ws):
    """A million keys at 2^-26 of the weight of key `loud` hold 1.5% of the sum. Their values are 1, its values 0.
    Returns (o, lse), the exact ones, and q8_attn_bound's bound e of a logit."""
    N, H, scale = 1 << 20, 1, 0.25
    codes = [torch.zeros((N, H, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    sc = [torch.full((N // 128, H), 2.0 ** -8, device=DEV) for _ in range(2)]
    codes[1][:] = 0x78                                               # 256: values of 1
    codes[1][loud] = 0                                               # and 0 under the large weight
    u = np.random.default_rng(1).choice([-1.0, 1.0], d)
    codes[0][loud, 0] = Q.codes_of(256.0 * u)
    assert Q.e4m3_decode([0x78])[0] == 256.0
    at = 26.0 * math.log(2) / (scale * d)                            # the logit in log2 units is 26
    q = torch.from_numpy(np.broadcast_to(at * u, (A, H, d)).copy()).bfloat16()
    x = float((O.f64(q[0, 0]) * u).sum() * scale)
    total = math.exp(x) + (N - 1)
    e = scale * (2.0 ** -17 * at * d + 2 * d * 2.0 ** -23 * at * d) + 2.0 ** -22 * (x * math.log2(math.e) + 4)
    ws = None if ws else torch.empty(0, dtype=torch.uint8, device=DEV)
    return _run_attn(None, q, np.arange(A, dtype=np.int32), scale, ws=ws, dev=(*codes, *sc)), ((N - 1) / total, math.log(total)), e


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [5, 16, 60, 300])
@pytest.mark.parametrize("loud", [3, (1 << 20) - 9])
@pytest.mark.parametrize("split", [False, True])
def test_attn_q8_a_long_sum_loses_no_small_terms(A, d, loud, split):
    """16,384 additions of 2^-24 to a sum of 1: rounded one by one, fp32 would drop them all (lse off by 2^-10)."""
    (_, lse), (_, rlse), e = _one_loud_key(A, d, loud, split)
    assert np.abs(lse - rlse).max() <= e + 2.0 ** -22 * (rlse + 1)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [5, 16, 60, 300])
@pytest.mark.parametrize("loud", [3, (1 << 20) - 9])
@pytest.mark.parametrize("split", [False, True])
def test_attn_q8_many_small_weights_count_beside_a_large_one(A, d, loud, split):
    """As above: the values under the small weights must not get lost in f16."""
    (o, _), (ref, _), e = _one_loud_key(A, d, loud, split)
    # as q8_attn_bound: f16's normal rounding, e twice, bf16, and N 2^-33 of the largest p vs by 448
    tol = (2.0 ** -11 + 2 * e + 2.0 ** -8) * ref + 2.0 ** 20 * 2.0 ** -33 * 448 * 2.0 ** -8
    assert np.abs(o - ref).max() <= tol, (float(np.abs(o - ref).max()), tol, ref)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("A", [5, 60, 300])
@pytest.mark.parametrize("power", [-115, -104, 104, 112, 125])
def test_attn_q8_queries_at_the_ends_of_bf16(A, d, power):
    """Rows of Q of 2^power, with a softmax scale that makes their logits ordinary ones."""
    N, H = 700, 2
    cache, q, idx = _attn_case(N, A, H, d, 37)
    q = (q.double().clamp(-3.5, 3.5) * 2.0 ** power).bfloat16()
    assert bool(q.isfinite().all())
    scale = 2.0 ** -power / math.sqrt(d)
    o, lse = _run_attn(cache, q, idx, scale)
    _check_attn(o, lse, cache, q, idx, scale)


def test_attn_q8_takes_its_scale_as_pruned_attn_does():
    """Whatever converts to a float, a zero-dimensional tensor among it."""
    cache, q, idx = _attn_case(300, 20, 2, 64, 3)
    q, cache, idx = q.to(DEV), _to_dev(cache), _dev(idx)
    want = tps.pruned_attn_q8(q, *cache, *idx, 0.125)
    kv = torch.zeros((300, 2, 64), dtype=torch.bfloat16, device=DEV)
    for scale in (torch.tensor(0.125), np.float32(0.125), torch.tensor(0.125, device=DEV)):
        tps.pruned_attn(q, kv, kv, *idx, scale)
        assert torch.equal(tps.pruned_attn_q8(q, *cache, *idx, scale), want)
    tps.tps_check()


def test_attn_q8_the_tail_plan_is_the_one_that_is_tested():
    """The shape of test_attn_q8_full_waves_then_a_split_tail splits its last row tiles alone: a plan that split all
    rows would need room for two parts of each."""
    N, A, H, d = 2100, 2005, 24, 64
    need = tps.attn_q8_workspace(A, N, H, d).numel()
    assert 0 < need < 2 * A * H * (d + 1) * 4


@pytest.mark.parametrize("d", [64, 128])
def test_attn_q8_nan_scales_of_blocks_that_no_query_keeps(d):
    N, H, nb = 900, 2, 8
    cache, q, idx = _attn_case(N, 500, H, d, 77)
    bm = np.ones((nb, nb), np.uint8)
    bm[:, [0, 3, 7]] = 0                                             # the first, one between, the last (part of a tile)
    clean = _run_attn(cache, q, idx, 0.125, bm=bm)
    _check_attn(*clean, cache, q, idx, 0.125, bm)
    dev = list(_to_dev(cache))
    for b in (0, 3, 7):
        for codes, sc in ((dev[0], dev[2]), (dev[1], dev[3])):
            codes[b * 128:(b + 1) * 128] = 0x7F
            sc[b] = float("nan")
    for got, want in zip(_run_attn(cache, q, idx, 0.125, bm=bm, dev=dev), clean):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("A,masked", [(40, False), (130, False), (130, True)])
def test_attn_q8_offsets_beyond_32_bits_on_the_tensor_cores(A, masked):
    """A cache of more than 2^32 code bytes through the tensor maps and the converters, dense (one set, two sets) and
    with a mask that keeps the first and the last key blocks."""
    H, d, scale = 128, 128, 0.5
    N = (1 << 18) + 200
    nb = (N + 127) // 128
    kc, vc, ks, vs = tps.cache_q8(N, H, d)
    idx = np.concatenate([np.arange(64), np.arange(N - 200, N)]).astype(np.int32)
    k, v, q = (synth.gaussian_bf16((len(idx), H, d), 90 + i) for i in range(3))
    tps.kv_sync_q8(kc, vc, ks, vs, k.to(DEV), v.to(DEV), *_dev(idx))
    last = slice(len(idx) - A, len(idx))
    bm = None
    if masked:
        bm = np.zeros((nb, nb), np.uint8)
        bm[:, [0, nb - 2, nb - 1]] = 1
    o, lse = _run_attn(None, q[last], idx[last], scale, bm=bm, dev=(kc, vc, ks, vs))
    rows = torch.from_numpy(idx).long().to(DEV)
    for h in (0, 127):
        full = []
        for codes, sc, x in ((kc, ks, k), (vc, vs, v)):
            per = sc[rows // 128, h].cpu().double().numpy()[:, None]
            got = Q.e4m3_decode(codes.view(torch.uint8)[rows, h].cpu().numpy()) * per
            x = O.f64(x[:, h])
            assert np.all(np.abs(got - x) <= 2.0 ** -4 * np.abs(x) + 2.0 ** -10 * per)
            at = np.zeros((N, 1, d))
            at[idx, 0] = got
            full.append(at)
        qh, v_scale = q[last][:, h:h + 1], vs[:, h:h + 1].cpu().double().numpy()
        ref, rlse = O.pruned_attn(qh, *full, idx[last], scale, blockmask=bm)
        ot, lt = Q.q8_attn_bound(qh, *full, v_scale, idx[last], scale, bm, floor=2.0 ** -25)
        assert np.all(np.abs(o[:, h:h + 1] - ref) <= ot)
        assert np.all(np.abs(lse[:, h:h + 1] - rlse) <= lt)


@pytest.mark.parametrize("old", [1e-40, 2.0 ** -127, 2.0 ** -126, 3e38])
def test_kv_sync_q8_zero_rows_under_an_old_scale_at_the_ends_of_fp32(old):
    """Zero values are codes of zero whatever positive scale the block has (its reciprocal may be beyond fp32)."""
    N, H, d = 200, 2, 64
    cache = _cache(N, H, d, 12)
    dev = _to_dev(cache)
    dev[2][0], dev[3][0] = old, old
    idx = _idx(128, 30, 4)
    zero = torch.zeros((30, H, d), dtype=torch.bfloat16)
    tps.kv_sync_q8(*dev, zero.to(DEV), zero.to(DEV), *_dev(idx))
    tps.tps_check()
    for i in range(2):
        vals, sc = cache[i][0], cache[i][1].copy()
        sc[0] = float(np.float32(old))
        _check_codes(dev[i], dev[2 + i], *Q.kv_sync_q8(vals, sc, O.f64(zero), idx))


@pytest.mark.parametrize("N,A,H,d,masked", [(700, 5, 2, 64, False), (700, 60, 2, 128, False), (700, 300, 2, 64, False),
                                            (2100, 2000, 24, 64, False), (700, 300, 2, 128, True), (300, 40, 256, 128, False),
                                            (300, 140, 256, 128, True)])
def test_attn_q8_in_place_a_smaller_capacity_and_a_mask_of_bools(N, A, H, d, masked):
    """o_act may be q_act; with cap given, rows behind it stay whatever the count says; a mask may be bool."""
    cache, q, idx = _attn_case(N, A, H, d, 19)
    nb = (N + 127) // 128
    bm = (np.random.default_rng(2).random((nb, nb)) < 0.6) if masked else None
    scale = 1.0 / math.sqrt(d)
    dev = _to_dev(cache)
    want, lse = _run_attn(cache, q, idx, scale, bm=None if bm is None else bm.astype(np.uint8), dev=dev)
    if H < 100:
        _check_attn(want, lse, cache, q, idx, scale, bm)
    else:                                                            # a few of many heads
        some = [0, 100, H - 1]
        part = [(v[:, some], s[:, some]) for v, s in cache]
        _check_attn(want[:, some], lse[:, some], part, q[:, some], idx, scale, bm)
    mask = None if bm is None else torch.from_numpy(bm).to(DEV)
    di, dc = _dev(idx)
    o = q.to(DEV)
    tps.pruned_attn_q8(o, *dev, di, dc, scale, blockmask=mask, o_act=o)
    assert np.array_equal(O.f64(o.cpu()), want)
    cap = A - A // 3
    o = torch.full((A, H, d), 7.0, dtype=torch.bfloat16, device=DEV)
    tps.pruned_attn_q8(q.to(DEV), *dev, di, dc, scale, blockmask=mask, o_act=o, cap=cap)
    tps.tps_check()
    assert bool((o[cap:] == 7.0).all())
    tol, _ = Q.q8_attn_bound(q[:cap, :1], *(v[:, :1] for v in _values(cache)), cache[1][1][:, :1], idx[:cap], scale, bm)
    assert np.all(np.abs(O.f64(o[:cap, :1].cpu()) - want[:cap, :1]) <= 2 * tol)      # (another plan, other roundings)


def test_attn_q8_a_mask_of_the_largest_size():
    """4,096 key blocks: a query block that keeps all of them, and one that keeps the last alone."""
    N, H, d, A = 4096 * 128, 1, 64, 40
    kc, vc, ks, vs = tps.cache_q8(N, H, d)
    rows = np.unique(np.concatenate([np.random.default_rng(0).integers(0, N, 400), [0, N - 1]])).astype(np.int32)
    k, v = (synth.gaussian_bf16((len(rows), H, d), 95 + i) for i in range(2))
    tps.kv_sync_q8(kc, vc, ks, vs, k.to(DEV), v.to(DEV), *_dev(rows))
    idx = np.concatenate([np.arange(5, 25), np.arange(N - 60, N - 40)]).astype(np.int32)
    bm = np.zeros((4096, 4096), np.uint8)
    bm[0], bm[4095, 4095] = 1, 1
    q = synth.gaussian_bf16((A, H, d), 99)
    o, lse = _run_attn(None, q, idx, 1.0, bm=bm, dev=(kc, vc, ks, vs))
    cache = [(Q.e4m3_decode(c.cpu().view(torch.uint8).numpy()), s.cpu().double().numpy()) for c, s in ((kc, ks), (vc, vs))]
    _check_attn(o, lse, cache, q, idx, 1.0, bm)


def test_kv_sync_q8_all_heads_of_a_large_cache_in_one_block():
    """256 heads and enough blocks that a thread block takes all heads of its tokens."""
    N, H, d = 60000, 256, 64
    kc, vc, ks, vs = tps.cache_q8(N, H, d)
    idx = np.concatenate([np.arange(256, 384), [5, 1000, 1001, 59999]]).astype(np.int32)
    idx.sort()
    k, v = (synth.gaussian_bf16((len(idx), H, d), 85 + i) for i in range(2))
    for scale in (1.0, 4.0):                                         # the second time every scale grows
        tps.kv_sync_q8(kc, vc, ks, vs, (scale * k.float()).bfloat16().to(DEV), (scale * v.float()).bfloat16().to(DEV), *_dev(idx))
    tps.tps_check()
    for codes, sc, x in ((kc, ks, k), (vc, vs, v)):
        touched = np.unique(idx // 128)
        assert int((sc != 0).any(1).sum()) == len(touched)
        for b in touched:
            mine = idx // 128 == b
            n = min(128, N - b * 128)
            ref = Q.kv_sync_q8(np.zeros((n, H, d)), np.zeros((1, H)), O.f64(x)[mine] * 4.0, idx[mine] - b * 128)
            _check_codes(codes[b * 128:b * 128 + n], sc[b:b + 1], *ref)


@pytest.mark.parametrize("dims", [(64, 0, 0), (0, 64, 0), (0, 0, 64), (0, 30, 34), (2, 60, 2)])
def test_rope_groups_of_any_width(dims):
    grid, H, d = (3, 5, 7), 2, 64
    table = tps.rope_table(dims, grid)
    x = synth.gaussian_bf16((40, H, d), 3)
    idx = _idx(105, 40, 6)
    got = tps.rope_rows(x.to(DEV), *_dev(idx), table, dims, grid)
    ref = O.rope_rows(x, idx, dims, grid)
    assert np.all(np.abs(O.f64(got.cpu()) - ref) <= _rope_bound(ref, x))
    cache = tps.cache_q8(105, H, d)
    tps.kv_sync_q8(*cache, x.to(DEV), x.to(DEV), *_dev(idx), rope=(table, dims, grid))
    tps.tps_check()
    zero = (np.zeros((105, H, d)), np.zeros((1, H)))
    a = np.abs(O.f64(x))
    slack = 2.0 ** -22 * np.repeat(a[..., 0::2] + a[..., 1::2], 2, axis=-1)
    _check_codes(cache[0], cache[2], *Q.kv_sync_q8(*zero, ref, idx), ref, idx, slack)
