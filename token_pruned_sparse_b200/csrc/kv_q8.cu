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
// tokens of one tensor, for a run of heads: it finds the block's part of the ascending
// idx with two warp searches, lists its tokens and, for keys, gathers their (cos, sin)
// entries into shared memory. Then each warp takes a head: it loads all of the head's
// fresh rows of the block into registers at once (16 bytes per lane, up to 32 loads in
// flight, 64 rows of 128 or 128 rows of 64 channels) and goes over them once: turn,
// maximum, and codes against the OLD scale, which is the new one as long as the block
// got no louder. Only where the scale changes are the rows loaded again (from L2)
// and encoded again. No warp waits for another, except with more than 64 rows of 128
// channels: then two warps share a head and exchange their maxima. What it measured at
// the HSA size: CTA-wide passes of 128 (row, head) slots with three barriers each 466
// us; this layout with two turns from the table in global memory 375 us.
#include <climits>

#include "q8.cuh"
#include "rope_grid.cuh"
#include "trace.cuh"
#include "warp_search.cuh"

namespace tps {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kVecs = 32;        // 16-byte vectors per lane in registers
constexpr int kCtasWanted = 24;  // CTAs of a launch per SM (3 run at a time)

struct SyncQ8 {
  uint8_t* cache[2];
  float* scale[2];
  const uint16_t* fresh[2];
  const int32_t* idx;
  const int32_t* count;
  int64_t cap;
  int64_t N;
  int H;
  int heads;       // heads per CTA
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
__device__ __forceinline__ float factor_of(float scale) { return scale > 0.f ? 1.f / scale : 1.f; }
// Largest of the non-negative floats of a warp.
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x)));
}

template <int D, bool kTurn>
__device__ __forceinline__ void sync_block(const SyncQ8& p, int tensor) {
  constexpr int kLanes = D / 8;              // lanes of a row, 8 channels each
  constexpr int kRows = 32 / kLanes;         // rows of one warp-wide vector
  constexpr int kHeld = kVecs * kRows;       // rows a warp holds
  __shared__ int64_t s_run[2];
  __shared__ int s_src[kScaleBlock];     // fresh row of each token of the block, or INT_MAX
  __shared__ int2 s_list[kScaleBlock];   // (token of the block, fresh row), ascending
  __shared__ int s_cnt[kWarps];
  __shared__ float s_top[kWarps];
  extern __shared__ float4 s_cs[];       // kTurn: (cos, sin) of two pairs per entry, D / 4 entries per listed token

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const int64_t n0 = b * kScaleBlock;
  const int64_t cnt = active_count(p.count, p.cap);
  if (warp < 2) {
    const int64_t at = warp_lower_bound(p.idx, cnt, n0 + warp * kScaleBlock, lane);
    if (lane == 0) s_run[warp] = at;
  }
  s_src[tid] = INT_MAX;
  __syncthreads();
  const int64_t lo = s_run[0], hi = s_run[1];
  if (blockIdx.y == 0 && tensor == 0 && tid == 0 && cnt > 0 &&
      ((b == 0 && p.idx[0] < 0) || (b == gridDim.x - 1 && p.idx[cnt - 1] >= p.N)))
    raise_status(p.status, STATUS_BOUNDS);
  if (hi <= lo) return;

  const int size = static_cast<int>(p.N - n0 < kScaleBlock ? p.N - n0 : kScaleBlock);
  for (int64_t j = lo + tid; j < hi; j += kThreads) {
    const int64_t n = static_cast<int64_t>(p.idx[j]) - n0;
    const bool in = n >= 0 && n < size;
    if (in) atomicMin(&s_src[n], static_cast<int>(j));   // of equal entries the first counts
    // out of order, outside [0, N) or a repeated token
    if (!in || (j > lo && p.idx[j - 1] >= p.idx[j])) raise_status(p.status, STATUS_BOUNDS);
  }
  __syncthreads();
  static_assert(kThreads == kScaleBlock, "one thread per token of the block");
  const unsigned int mine = __ballot_sync(0xffffffffu, s_src[tid] != INT_MAX);
  if (lane == 0) s_cnt[warp] = __popc(mine);
  __syncthreads();
  int nact = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? s_cnt[w] : 0;
    nact += s_cnt[w];
  }
  if ((mine >> lane) & 1u) s_list[before + __popc(mine & ((1u << lane) - 1u))] = make_int2(tid, s_src[tid]);
  __syncthreads();
  if (nact == 0) return;
  const bool whole = nact == size;
  if constexpr (kTurn) {
    // a quarter-warp's worth of threads per token: 4 pairs each
    for (int i = tid; i < nact * kLanes; i += kThreads) {
      const int c = i / kLanes, l = i % kLanes;
      float2 e[4];
      rope_lookup(p.grid, static_cast<uint32_t>(n0) + s_list[c].x, l * 4, e);
      s_cs[(c * kLanes + l) * 2] = make_float4(e[0].x, e[0].y, e[1].x, e[1].y);
      s_cs[(c * kLanes + l) * 2 + 1] = make_float4(e[2].x, e[2].y, e[3].x, e[3].y);
    }
    __syncthreads();
  }

  const int lane8 = lane % kLanes, sub = lane / kLanes;
  const uint4* fresh = reinterpret_cast<const uint4*>(p.fresh[tensor]);
  uint2* cache = reinterpret_cast<uint2*>(p.cache[tensor]);
  float* scale = p.scale[tensor] + b * p.H;
  const int hend = min(p.H, (static_cast<int>(blockIdx.y) + 1) * p.heads);
  const int share = nact > kHeld ? 2 : 1;              // warps per head
  const int c0 = share == 2 ? (warp & 1) * kHeld : 0;  // this warp's first row in the list
  const int mylen = min(nact - c0, kHeld);

  for (int h0 = blockIdx.y * p.heads; h0 < hend; h0 += kWarps / share) {
    const int h = h0 + warp / share;
    const bool on = h < hend;
    auto row_of = [&](int c) { return fresh + (static_cast<int64_t>(s_list[c0 + c].y) * p.H + h) * kLanes + lane8; };
    auto entries = [&](int c) { return s_cs + ((c0 + c) * kLanes + lane8) * 2; };
    auto place = [&](int c) { return cache + ((n0 + s_list[c0 + c].x) * p.H + h) * kLanes + lane8; };
    uint4 x[kVecs];
    if (on) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (i * kRows + sub < mylen) x[i] = *row_of(i * kRows + sub);
    }
    const float was = on ? scale[h] : 0.f;
    const float inv_was = factor_of(was);
    float top = 0.f;
    if (on) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) {
        const int c = i * kRows + sub;
        if (c < mylen) {
          float v[8];
          values_of<kTurn>(x[i], entries(c), v);
#pragma unroll
          for (int q = 0; q < 8; ++q) top = fmaxf(top, fabsf(v[q]));   // (NaN is passed over)
          const uint2 o = codes_of(v, inv_was);
          x[i].x = o.x;
          x[i].y = o.y;
        }
      }
      top = warp_max(top);
      if (top == INFINITY) {                           // infinities set no scale: look again without them
        top = 0.f;
#pragma unroll 1
        for (int c = sub; c < mylen; c += kRows) {
          float v[8];
          values_of<kTurn>(*row_of(c), entries(c), v);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (fabsf(v[q]) < INFINITY) top = fmaxf(top, fabsf(v[q]));
        }
        top = warp_max(top);
      }
    }
    if (share == 2) {                                  // uniform over the CTA
      __syncthreads();
      if (lane == 0) s_top[warp] = top;
      __syncthreads();
      top = fmaxf(s_top[warp], s_top[warp ^ 1]);
    }
    if (!on) continue;                                 // no barrier from here to the next head's
    const float need = scale_of_amax(top);
    const float sc = whole ? need : fmaxf(need, was);  // a NaN old scale counts as none
    if (sc == was) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i)
        if (i * kRows + sub < mylen) *place(i * kRows + sub) = make_uint2(x[i].x, x[i].y);
    } else {
      const float inv = factor_of(sc);
#pragma unroll 4
      for (int c = sub; c < mylen; c += kRows) {
        float v[8];
        values_of<kTurn>(*row_of(c), entries(c), v);
        *place(c) = codes_of(v, inv);
      }
    }
    if (share == 1 || (warp & 1) == 0) {
      if (!whole && (sc > was || was != was)) {        // the scale grew: the stale rows move to it
        const float ratio = was > 0.f ? was / sc : 0.f;
#pragma unroll 4
        for (int r = sub; r < size; r += kRows) {
          if (s_src[r] != INT_MAX) continue;
          uint2* at = cache + ((n0 + r) * p.H + h) * kLanes + lane8;
          const uint2 w = *at;
          uint32_t o[2];
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t u = q ? w.y : w.x;
            const float2 e = f16x2_to_f2(e4m3x2_to_f16x2(u)), f = f16x2_to_f2(e4m3x2_to_f16x2(u >> 16));
            o[q] = pack_e4m3x4(e.x * ratio, e.y * ratio, f.x * ratio, f.y * ratio);
          }
          *at = make_uint2(o[0], o[1]);
        }
      }
      __syncwarp();
      if (lane == 0) scale[h] = sc;                    // (a second warp of the head read the old one before its barrier)
    }
  }
}

// blockIdx.z: 0 = K, 1 = V
template <int D, bool kTurnK>
__global__ void __launch_bounds__(kThreads, 3) sync_q8_kernel(const __grid_constant__ SyncQ8 p) {
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
  // Heads per CTA: every CTA pays the search of its run, so it takes several heads per warp where the
  // blocks fill the GPU; small caches spread over the heads instead.
  int64_t chunks = (static_cast<int64_t>(sm_count()) * kCtasWanted + 2 * nb - 1) / (2 * nb);
  const int64_t most = (H + kWarps - 1) / kWarps;
  chunks = chunks < 1 ? 1 : (chunks > most ? most : chunks);
  p.heads = static_cast<int>((H + chunks - 1) / chunks);
  p.heads = (p.heads + kWarps - 1) / kWarps * kWarps;
  const dim3 grid(static_cast<unsigned>(nb), static_cast<unsigned>((H + p.heads - 1) / p.heads), 2);
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
