// kv_sync_q8: the fresh K and V rows of the active tokens go into a cache held in
// 8 bits, the keys turned to their rotary position on the way.
//
// [HSA] 2.2 (2): fresh K/V of the active tokens overwrite their cache rows, the
// others stay stale but valid; [TR] Metodologia 1: rotary groups t, x, y. The
// cache is e4m3 with one scale for each block of 128 tokens, head and tensor.
//
// Scale of a block: need = the smallest 2^e with amax <= 448 * 2^e over its fresh
// values (fp32, after the turn, |.| finite). Every token of the block fresh:
// scale = need. Otherwise scale = max(old scale, need): it only grows, so the
// stale rows need not be read for a maximum, and are re-encoded only when the scale
// does grow. Powers of two make that exact: e4m3 is a floating-point format, so a
// code keeps its value at another power of two unless it leaves the normal
// range below (steps of 2^-9 of the scale); repeated updates do not drift.
//
// HBM-bound: 2 bytes read and 1 written per fresh element. A CTA takes one block of 128
// tokens of one tensor (and of a run of heads, where blocks alone would not fill the GPU):
// it finds the block's part of the ascending idx with two warp searches, lists its tokens
// and, for keys, gathers their (cos, sin) entries into shared memory. Then it streams the
// rows once: a warp takes 512 contiguous bytes of each of a part of the rows, 8 loads in
// flight, turns them, keeps the maximum, and writes the codes against the OLD scale, which
// is the new one as long as the block got no louder. Heads whose scale does change are
// read again (from L2) and encoded again. Measured at the HSA size (39,600 rows, 0.73 GB, floor 111
// us) with scales that stay: CTA-wide passes of 128 (row, head) slots with the block's values held in
// registers 466 us, a warp holding its head's rows 210-220 us, this 151-155 us (3 CTAs per SM of 80
// registers instead of 2 of 116: 173), 183 as a single call after a flush of L2.
// The price: where scales change the second pass has one load in flight per warp and stale rows go 8
// bytes a lane. Single calls after a flush: the same update four times as loud, so that every scale
// grows (1.70 GB with the stale rows, floor 260 us), 900 us; the first fill of all 118,800 rows (2.19
// GB, 334 us) 1,190 us; five new frames of 1,560 tokens, 12 heads (72 MB, 11 us) 27 us where no scale
// changes, 45 us where 7% of the keys' do.
#include <climits>

#include "q8.cuh"
#include "rope_grid.cuh"
#include "trace.cuh"
#include "warp_search.cuh"

namespace tps {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 8;       // rows of a warp in flight
constexpr int kPart = 16;        // rows of one task: a block's tasks spread evenly over the warps
constexpr int kMaxHeads = 256;
constexpr int kCtasWanted = 6;   // CTAs of a launch per SM (2 run at a time)

struct SyncQ8 {
  uint8_t* cache[2];
  float* scale[2];
  const uint16_t* fresh[2];
  const int32_t* idx;
  const int32_t* count;
  int64_t cap;
  int64_t N;
  int H;
  int vpr;         // 16-byte vectors of a fresh row
  int groups;      // 32-vector groups per CTA
  RopeGrid grid;
  unsigned int* status;
};

// The 8 channels of one vector in fp32, turned by the entries cs of their 4 pairs.
template <bool kTurn>
__device__ __forceinline__ void values_of(uint4 x, const float4* cs, float (&v)[8]) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if constexpr (kTurn) {
    const float4 a = cs[0], b = cs[1];
    const float2 e[4] = {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float2 r = rope_turn(w[q], e[q]);
      v[2 * q] = r.x;
      v[2 * q + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = bf16lo(w[q]);
      v[2 * q + 1] = bf16hi(w[q]);
    }
  }
}
__device__ __forceinline__ uint2 codes_of(const float (&v)[8], float inv) {
  return make_uint2(pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                    pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
}
// (finite: below 2^-128 the reciprocal is not, and 0 times it would be NaN)
__device__ __forceinline__ float factor_of(float scale) { return scale > 0.f ? fminf(1.f / scale, 3e38f) : 1.f; }

template <int D, bool kTurn>
__device__ __forceinline__ void sync_block(const SyncQ8& p, int tensor) {
  constexpr int kLanes = D / 8;              // lanes of a head's row, 8 channels each
  constexpr int kHeads = 32 / kLanes;        // heads of a 32-vector group
  __shared__ int64_t s_run[2];
  __shared__ int s_src[kScaleBlock];     // fresh row of each token of the block, or INT_MAX
  __shared__ int2 s_list[kScaleBlock];   // (token of the block, fresh row), ascending
  __shared__ int s_cnt[kScaleBlock / 32];
  __shared__ int s_top[kMaxHeads];       // bits of each head's maximum (non-negative floats order as ints)
  __shared__ float s_was[kMaxHeads], s_inv[kMaxHeads];
  extern __shared__ float4 s_cs[];       // kTurn: (cos, sin) of two pairs per entry, D / 4 entries per listed token

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const int64_t n0 = b * kScaleBlock;
  const int64_t cnt = active_count(p.count, p.cap);
  if (warp < 2) {
    const int64_t at = warp_lower_bound(p.idx, cnt, n0 + warp * kScaleBlock, lane);
    if (lane == 0) s_run[warp] = at;
  }
  if (tid < kScaleBlock) s_src[tid] = INT_MAX;
  __syncthreads();
  const int64_t lo = s_run[0], hi = s_run[1];
  if (blockIdx.y == 0 && tensor == 0 && tid == 0 && cnt > 0 &&
      ((b == 0 && p.idx[0] < 0) || (b == gridDim.x - 1 && p.idx[cnt - 1] >= p.N)))
    raise_status(p.status, STATUS_BOUNDS);
  if (hi <= lo) return;

  const int size = static_cast<int>(p.N - n0 < kScaleBlock ? p.N - n0 : kScaleBlock);
  const int g0 = blockIdx.y * p.groups;                          // this CTA's groups and heads
  const int ng = min(p.groups, (p.vpr + 31) / 32 - g0);
  const int h0 = g0 * kHeads, nh = min(ng * kHeads, p.H - h0);
  float* scale = p.scale[tensor] + b * p.H + h0;
  for (int64_t j = lo + tid; j < hi; j += kThreads) {
    const int64_t n = static_cast<int64_t>(p.idx[j]) - n0;
    const bool in = n >= 0 && n < size;
    if (in) atomicMin(&s_src[n], static_cast<int>(j));   // of equal entries the first counts
    // out of order, outside [0, N) or a repeated token
    if (!in || (j > lo && p.idx[j - 1] >= p.idx[j])) raise_status(p.status, STATUS_BOUNDS);
  }
  if (tid < nh) {
    s_top[tid] = 0;
    s_was[tid] = scale[tid];
    s_inv[tid] = factor_of(s_was[tid]);
  }
  __syncthreads();
  unsigned int mine = 0;
  if (tid < kScaleBlock) {
    mine = __ballot_sync(0xffffffffu, s_src[tid] != INT_MAX);
    if (lane == 0) s_cnt[warp] = __popc(mine);
  }
  __syncthreads();
  int nact = 0;
#pragma unroll
  for (int w = 0; w < kScaleBlock / 32; ++w) {
    if (w == warp && ((mine >> lane) & 1u))
      s_list[nact + __popc(mine & ((1u << lane) - 1u))] = make_int2(tid, s_src[tid]);
    nact += s_cnt[w];
  }
  __syncthreads();
  if (nact == 0) return;
  const bool whole = nact == size;
  if constexpr (kTurn) {
    for (int i = tid; i < nact * kLanes; i += kThreads) {
      const int c = i / kLanes, l = i % kLanes;
      float2 e[4];
      rope_lookup(p.grid, static_cast<uint32_t>(n0) + s_list[c].x, l * 4, e);
      s_cs[i * 2] = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
      s_cs[i * 2 + 1] = make_float4(e[2].x, e[2].y, e[3].x, e[3].y);
    }
    __syncthreads();
  }

  const uint4* fresh = reinterpret_cast<const uint4*>(p.fresh[tensor]);
  uint2* cache = reinterpret_cast<uint2*>(p.cache[tensor]);
  const int lane8 = lane % kLanes;
  const int ntasks = ng * ((nact + kPart - 1) / kPart);
  // A task is one group of one part of the rows; f(v, head, first row, end) with this lane's vector v.
  auto tasks = [&](auto&& f) {
    for (int k = warp; k < ntasks; k += kWarps) {
      const int g = k % ng, c0 = k / ng * kPart;
      const int v = (g0 + g) * 32 + lane;
      f(v, g * kHeads + lane / kLanes, c0, min(c0 + kPart, nact));
    }
  };
  auto load = [&](int v, int c) { return fresh[static_cast<int64_t>(s_list[c].y) * p.vpr + v]; };
  auto entries = [&](int c) { return s_cs + (c * kLanes + lane8) * 2; };
  auto store = [&](int v, int c, uint2 o) { cache[(n0 + s_list[c].x) * p.vpr + v] = o; };
  auto largest = [](const float(&x)[8]) {
    float a = fmaxf(fabsf(x[0]), fabsf(x[1]));           // (NaN is passed over)
#pragma unroll
    for (int q = 2; q < 8; ++q) a = fmaxf(a, fabsf(x[q]));
    return a;
  };
  auto keep_top = [&](float top, int head, bool on) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (on && lane8 == 0) atomicMax(&s_top[head], __float_as_int(top));
  };

  // ---- one pass: codes against the old scale, and the maxima -----------------------------------
  tasks([&](int v, int head, int c0, int c1) {
    const bool on = v < p.vpr;
    const float inv = on ? s_inv[head] : 1.f;
    float top = 0.f;
    for (int c = c0; c < c1; c += kUnroll) {
      uint4 x[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)     // rows behind the last repeat it: the same codes to the same place
        if (on) x[u] = load(v, min(c + u, c1 - 1));
      if (on) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
          float f[8];
          values_of<kTurn>(x[u], entries(min(c + u, c1 - 1)), f);
          top = fmaxf(top, largest(f));
          store(v, min(c + u, c1 - 1), codes_of(f, inv));
        }
      }
    }
    keep_top(top, head, on);
  });
  __syncthreads();

  // ---- the new scales -------------------------------------------------------------------------------
  bool infinite = tid < nh && s_top[tid] == 0x7F800000;
  if (__syncthreads_or(infinite)) {         // infinities set no scale: look again without them
    if (infinite) s_top[tid] = 0;
    __syncthreads();
    tasks([&](int v, int head, int c0, int c1) {
      const bool on = v < p.vpr;
      float top = 0.f;
      for (int c = c0; on && c < c1; ++c) {
        float f[8];
        values_of<kTurn>(load(v, c), entries(c), f);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (fabsf(f[q]) < INFINITY) top = fmaxf(top, fabsf(f[q]));
      }
      keep_top(top, head, on);
    });
    __syncthreads();
  }
  bool changed = false;
  float ratio = 0.f;
  if (tid < nh) {
    const float was = s_was[tid], need = scale_of_amax(__int_as_float(s_top[tid]));
    const float sc = whole ? need : fmaxf(need, was);     // a NaN old scale counts as none
    changed = !(sc == was);
    if (changed) {
      scale[tid] = sc;
      ratio = !(was > 0.f) ? 0.f : was / sc;
      s_inv[tid] = factor_of(sc);
    }
    s_top[tid] = changed;
    s_was[tid] = ratio;
  }
  if (!__syncthreads_or(changed)) return;

  // ---- the heads whose scale changed: fresh rows again, and the stale ones --------------------------
  tasks([&](int v, int head, int c0, int c1) {
    if (v >= p.vpr || !s_top[head]) return;
    const float inv = s_inv[head];
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
      float f[8];
      values_of<kTurn>(load(v, c), entries(c), f);
      store(v, c, codes_of(f, inv));
    }
  });
  if (whole) return;
  for (int k = warp; k < ng * (kScaleBlock / kPart); k += kWarps) {
    const int g = k % ng, r0 = k / ng * kPart;
    const int v = (g0 + g) * 32 + lane, head = g * kHeads + lane / kLanes;
    if (v >= p.vpr || !s_top[head]) continue;
    const float r = s_was[head];
#pragma unroll 4
    for (int n = r0; n < min(r0 + kPart, size); ++n) {
      if (s_src[n] != INT_MAX) continue;
      uint2* at = cache + (n0 + n) * p.vpr + v;
      const uint2 w = *at;
      uint32_t o[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t u = q ? w.y : w.x;
        const float2 e = f16x2_to_f2(e4m3x2_to_f16x2(u)), f = f16x2_to_f2(e4m3x2_to_f16x2(u >> 16));
        o[q] = pack_e4m3x4(e.x * r, e.y * r, f.x * r, f.y * r);
      }
      *at = make_uint2(o[0], o[1]);
    }
  }
}

// blockIdx.z: 0 = K, 1 = V
template <int D, bool kTurnK>
__global__ void __launch_bounds__(kThreads, 2) sync_q8_kernel(const __grid_constant__ SyncQ8 p) {
  if (kTurnK && blockIdx.z == 0) sync_block<D, true>(p, 0);
  else sync_block<D, false>(p, blockIdx.z);
}

}  // namespace
}  // namespace tps

using namespace tps;

extern "C" int kv_sync_q8(uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale, const tps_bf16* k_fresh,
                          const tps_bf16* v_fresh, const int32_t* idx, const int32_t* count, int64_t cap, int64_t N,
                          int H, int d, const tps_rope_grid* rope, tps_stream stream) {
  TPS_TRACE("kv_sync_q8");
  if (!k_cache || !v_cache || !k_scale || !v_scale || !k_fresh || !v_fresh || !idx || !count)
    return fail(TPS_ERR_INVALID_ARG, "kv_sync_q8: null pointer");
  if (cap < 0 || cap >= (INT64_C(1) << 31) || N < 1 || N >= (INT64_C(1) << 31))
    return fail(TPS_ERR_SHAPE, "kv_sync_q8: need 0 <= cap < 2^31 and 1 <= N < 2^31");
  if (d != 64 && d != 128) return fail(TPS_ERR_INVALID_ARG, "kv_sync_q8: d=%d must be 64 or 128", d);
  if (H < 1 || static_cast<int64_t>(H) * d > 16384)
    return fail(TPS_ERR_SHAPE, "kv_sync_q8: H=%d must satisfy 1 <= H*d <= 16384", H);
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_fresh) || !aligned16(v_fresh))
    return fail(TPS_ERR_ALIGN, "kv_sync_q8: rows must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale)) & 3u)
    return fail(TPS_ERR_ALIGN, "kv_sync_q8: scales must be 4-byte aligned");
  SyncQ8 p{};
  if (rope)
    if (int e = rope_grid_check("kv_sync_q8", rope, N, d, &p.grid)) return e;
  if (cap == 0) return ok();
  int err;
  p.status = device_status(&err);
  if (!p.status) return err;
  p.cache[0] = k_cache;
  p.cache[1] = v_cache;
  p.scale[0] = k_scale;
  p.scale[1] = v_scale;
  p.fresh[0] = k_fresh;
  p.fresh[1] = v_fresh;
  p.idx = idx;
  p.count = count;
  p.cap = cap;
  p.N = N;
  p.H = H;
  const int64_t nb = (N + kScaleBlock - 1) / kScaleBlock;
  // Every CTA pays the search of its run and the gathering of its entries, so it takes all heads where the
  // blocks alone fill the GPU; small caches spread over the heads instead.
  p.vpr = H * (d / 8);
  const int64_t all = (p.vpr + 31) / 32;
  int64_t chunks = (static_cast<int64_t>(sm_count()) * kCtasWanted + 2 * nb - 1) / (2 * nb);
  chunks = chunks < 1 ? 1 : (chunks > all ? all : chunks);
  p.groups = static_cast<int>((all + chunks - 1) / chunks);
  const dim3 grid(static_cast<unsigned>(nb), static_cast<unsigned>((all + p.groups - 1) / p.groups), 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t smem = rope ? static_cast<size_t>(kScaleBlock) * (d / 2) * sizeof(float2) : 0;
  if (d == 128 && rope) {
    const cudaError_t e = cudaFuncSetAttribute(sync_q8_kernel<128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(smem));   // per device; a host-side call
    if (e != cudaSuccess) return cuda_status(e, "kv_sync_q8: smem attribute");
    sync_q8_kernel<128, true><<<grid, kThreads, smem, st>>>(p);
  } else if (d == 128) {
    sync_q8_kernel<128, false><<<grid, kThreads, 0, st>>>(p);
  } else if (rope) {
    sync_q8_kernel<64, true><<<grid, kThreads, smem, st>>>(p);
  } else {
    sync_q8_kernel<64, false><<<grid, kThreads, 0, st>>>(p);
  }
  if (int e = launch_status("kv_sync_q8")) return e;
  return ok();
}
