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
// One CTA owns a block of 128 tokens of one tensor, for a run of heads. It finds
// the block's part of the ascending idx with two warp searches, then takes as
// many heads at a time as fill its 128 (row, head) slots: all values are
// loaded once into registers (16 bytes per lane and slot), reduced to each
// head's maximum through shared memory, and encoded from the registers.
// HBM-bound: 2 bytes read and 1 written per fresh element.
#include "q8.cuh"
#include "rope_grid.cuh"
#include "trace.cuh"
#include "warp_search.cuh"

namespace tps {
namespace {

constexpr int kThreads = 256;
constexpr int kSlots = 128;      // (row, head) pairs in registers at a time

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
  bool turn;       // keys are turned by `grid`
  RopeGrid grid;
  unsigned int* status;
};

template <int D>
__global__ void __launch_bounds__(kThreads) sync_q8_kernel(const __grid_constant__ SyncQ8 p) {
  constexpr int kLanes = D / 8;                     // lanes of a slot, 8 channels each
  constexpr int kPer = kSlots * kLanes / kThreads;  // slots per thread
  constexpr int kStep = kThreads / kLanes;          // slots of one pass
  __shared__ int64_t s_run[2];
  __shared__ int s_src[kScaleBlock];     // fresh row of each token of the block, or INT_MAX
  __shared__ int s_list[kScaleBlock];    // the block's active tokens, ascending
  __shared__ int s_cnt[kScaleBlock / 32];
  __shared__ int s_amax[kSlots];         // bits of each head's maximum (non-negative floats order as ints)
  __shared__ float s_old[kSlots];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t b = blockIdx.x;
  const int64_t n0 = b * kScaleBlock;
  const int tensor = blockIdx.z;
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
  for (int64_t j = lo + tid; j < hi; j += kThreads) {
    const int64_t n = static_cast<int64_t>(p.idx[j]) - n0;
    const bool in = n >= 0 && n < size;
    if (in) atomicMin(&s_src[n], static_cast<int>(j));   // of equal entries the first counts
    // out of order, outside [0, N) or a repeated token
    if (!in || (j > lo && p.idx[j - 1] >= p.idx[j])) raise_status(p.status, STATUS_BOUNDS);
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
    if (tid < kScaleBlock && w == warp && ((mine >> lane) & 1u))
      s_list[nact + __popc(mine & ((1u << lane) - 1u))] = tid;
    nact += s_cnt[w];
  }
  __syncthreads();
  if (nact == 0) return;
  const bool whole = nact == size;

  // heads at a time: the power of two that still fits nact rows of each into the slots
  int lg = 0;
  while ((nact << (lg + 1)) <= kSlots) ++lg;
  const int group = 1 << lg;
  const int lane8 = tid % kLanes, slot0 = tid / kLanes;
  const uint4* fresh = reinterpret_cast<const uint4*>(p.fresh[tensor]);
  uint2* cache = reinterpret_cast<uint2*>(p.cache[tensor]);
  float* scale = p.scale[tensor] + b * p.H;
  const bool turn = p.turn && tensor == 0;
  const int hend = min(p.H, (static_cast<int>(blockIdx.y) + 1) * p.heads);

  for (int h0 = blockIdx.y * p.heads; h0 < hend; h0 += group) {
    const int nh = min(group, hend - h0);
    uint4 x[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kStep + slot0, hh = s & (group - 1), c = s >> lg;
      if (c < nact && hh < nh)
        x[i] = fresh[(static_cast<int64_t>(s_src[s_list[c]]) * p.H + h0 + hh) * kLanes + lane8];
    }
    if (tid < nh) {
      s_amax[tid] = 0;
      s_old[tid] = scale[h0 + tid];
    }
    __syncthreads();
    // the values of slot i: fp32, turned
    auto values = [&](int i, int c, float (&v)[8]) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
      if (turn) {
        float2 cs[4];
        rope_lookup(p.grid, static_cast<uint32_t>(n0) + s_list[c], lane8 * 4, cs);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 r = rope_turn(w[q], cs[q]);
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
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kStep + slot0, hh = s & (group - 1), c = s >> lg;
      float top = 0.f;
      if (c < nact && hh < nh) {
        float v[8];
        values(i, c, v);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float a = fabsf(v[q]);
          if (a < INFINITY) top = fmaxf(top, a);     // infinities and NaN set no scale
        }
      }
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (lane8 == 0 && c < nact && hh < nh) atomicMax(&s_amax[hh], __float_as_int(top));
    }
    __syncthreads();
    auto new_scale = [&](int hh) {
      const float need = scale_of_amax(__int_as_float(s_amax[hh]));
      return whole ? need : fmaxf(need, s_old[hh]);   // a NaN old scale counts as none
    };
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int s = i * kStep + slot0, hh = s & (group - 1), c = s >> lg;
      if (c >= nact || hh >= nh) continue;
      float v[8];
      values(i, c, v);
      const float sc = new_scale(hh);
      const float inv = sc > 0.f ? 1.f / sc : 1.f;
      cache[((n0 + s_list[c]) * p.H + h0 + hh) * kLanes + lane8] =
          make_uint2(pack_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                     pack_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    }
    for (int hh = 0; hh < nh; ++hh) {
      const float sc = new_scale(hh), was = s_old[hh];
      if (tid == 0) scale[h0 + hh] = sc;
      if (whole || !(sc > was || was != was)) continue;   // stale rows keep their codes
      const float ratio = was > 0.f ? was / sc : 0.f;
      for (int r = slot0; r < size; r += kStep) {
        if (s_src[r] != INT_MAX) continue;
        uint2* at = cache + ((n0 + r) * p.H + h0 + hh) * kLanes + lane8;
        const uint2 w = *at;
        uint32_t o[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t u = q ? w.y : w.x;
          const float2 a = f16x2_to_f2(e4m3x2_to_f16x2(u)), c = f16x2_to_f2(e4m3x2_to_f16x2(u >> 16));
          o[q] = pack_e4m3x4(a.x * ratio, a.y * ratio, c.x * ratio, c.y * ratio);
        }
        *at = make_uint2(o[0], o[1]);
      }
    }
    __syncthreads();   // s_amax and s_old are rewritten for the next heads
  }
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
  p.turn = rope != nullptr;
  const int64_t nb = (N + kScaleBlock - 1) / kScaleBlock;
  // Heads per CTA: as many as leave about 8 CTAs per SM, since each one pays the search
  // of its run; small caches spread over the heads instead.
  int64_t chunks = (static_cast<int64_t>(sm_count()) * 8 + 2 * nb - 1) / (2 * nb);
  chunks = chunks < 1 ? 1 : (chunks > H ? H : chunks);
  p.heads = static_cast<int>((H + chunks - 1) / chunks);
  const dim3 grid(static_cast<unsigned>(nb), static_cast<unsigned>((H + p.heads - 1) / p.heads), 2);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d == 128) sync_q8_kernel<128><<<grid, kThreads, 0, st>>>(p);
  else sync_q8_kernel<64><<<grid, kThreads, 0, st>>>(p);
  if (int e = launch_status("kv_sync_q8")) return e;
  return ok();
}
