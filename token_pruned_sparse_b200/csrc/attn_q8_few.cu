// pruned_attn_q8 for at most 16 active rows: a few changed tokens (down to one) over a long
// 8-bit cache.
//
// The mathematics is that of attn_q8.cu: x = scale log2(e) ks_b (q . k8), P' =
// 2^(x + log2 vs_b - m) times V's codes, the sums of P' / vs_b. What bounds it is HBM:
// 2 H d bytes per key and 4 rows d FLOP, 111 us for one token over the HSA cache (0.73
// GB) at the measured copy rate. The tcgen05 kernel pays a 128-row product for it: 156 us
// in a single call, 180 us back to back, where its MMAs draw the clock down. This
// one takes 126 us with the merge in a graph (5.8 TB/s) and 133-138 us as a call; loads of the same
// addresses without any arithmetic take 120 us. The 12 warps per SM wait for memory half of the time. Slower (than
// an earlier 141 us a call, which spilled 12 bytes at D = 128): a ring of 4 steps through shared memory instead of
// the registers (156-165 us), adjacent heads side by side in a CTA (152-160), a prefetch of lines into L2 (145-177),
// e4m3 products for S (162, more registers), two chains of products for S instead of four (146). A warp works on its own, without shared memory, barriers or TMEM:
// - It owns whole blocks of 128 keys (one scale each) and goes over them 16 keys at
//   a time, the next 16 keys' codes (4 KB a warp) in flight meanwhile.
// - S = Q K^T and O^T = V^T P'^T are warp-level f16 products of 16 x 8 x 16; the codes
//   become f16 in registers (exact). The order of the channels inside the sum of S
//   is free, so a thread takes 16 consecutive codes of its key, and Q's fragments
//   are permuted to match once. The order of the output channels is free too, so a
//   thread takes D / 8 consecutive channels of V for its 4 keys; pairs of keys are
//   interleaved with byte permutes. S's result has just the layout in which P' enters the
//   second product.
// - A running reference maximum as in attn_q8.cu; rows that outgrow it are rescaled.
// The warps of a CTA merge through shared memory, the CTAs of a head (key ranges) through
// the caller's workspace and a second launch.
#include "attn_common.cuh"
#include "attn_q8.cuh"
#include "q8.cuh"

namespace tps {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 16;             // keys of a step
constexpr float kSumLimit = 16384.f;  // P' stays finite in f16 (a thread's four P' of a row sum to at most this)

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8-row sets of a call, and the CTAs that an SM holds (by registers)
constexpr int few_sets(int64_t cap) { return cap <= 8 ? 1 : 2; }
constexpr int few_ctas(int sets) { return sets == 1 ? 3 : 2; }

// kSets: 8-row sets (1 or 2).
template <int D, int kSets>
__global__ void __launch_bounds__(kThreads, few_ctas(kSets)) attn_q8_few_kernel(const __grid_constant__ Q8Args prm) {
  constexpr int kSteps = D / 16;        // 16-channel steps of S
  constexpr int kTilesM = D / 16;       // 16-channel tiles of O^T
  constexpr int kKV = D / 64;           // 16-byte vectors of a thread's key (4 threads hold D channels)
  constexpr int kVW = D / 32;           // words of a thread's V channels (D / 8 of them) of one key
  __shared__ __align__(16) float s_o[kWarps][8 * kSets][D + 4];   // written 8 bytes, read 16 bytes at a time
  static_assert((D + 4) * sizeof(float) % 16 == 0, "rows of s_o keep its alignment");
  __shared__ float4 s_msl[kWarps][8 * kSets];

  const AttnArgs& p = prm.a;
  const int rows = static_cast<int>(active_count(p.count, p.cap));
  if (rows == 0) return;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int h = blockIdx.x;
  const int nb = static_cast<int>((p.N + kScaleBlock - 1) / kScaleBlock);
  // this CTA's blocks, and this warp's among them
  const int b0 = static_cast<int>(static_cast<int64_t>(nb) * blockIdx.y / gridDim.y);
  const int b1 = static_cast<int>(static_cast<int64_t>(nb) * (blockIdx.y + 1) / gridDim.y);

  // ---- Q: rows g and g + 8 as f16 fragments, one power of two per row ------------------------------
  // k index 2t, 2t + 1, 2t + 8, 2t + 9 of step s stand for the channels 64 v + 16 t + 4 w + 0..3, s = 4 v + w
  uint32_t qf[kSteps][4];
  float rowc[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = g + 8 * r;
    const bool on = r < kSets && row < rows;
    uint4 x[2 * kKV];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 2 * kKV; ++i) {
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (on)
        x[i] = *(reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(row) * p.H + h) * D + 64 * (i >> 1) + 16 * t) +
                 (i & 1));
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float a = fabsf(bf16lo(w[k])), b = fabsf(bf16hi(w[k]));
        if (a < INFINITY) top = fmaxf(top, a);
        if (b < INFINITY) top = fmaxf(top, b);
      }
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const float sc = scale_of_row(top);
    rowc[r] = prm.scale_log2 * sc;
    const float inv = 1.f / sc;
#pragma unroll
    for (int i = 0; i < 2 * kKV; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 2; ++k) {            // channels 8 i' + 4 k .. + 3 of this thread
        float f[4] = {bf16lo(w[2 * k]) * inv, bf16hi(w[2 * k]) * inv, bf16lo(w[2 * k + 1]) * inv,
                      bf16hi(w[2 * k + 1]) * inv};
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!(fabsf(f[c]) < INFINITY)) f[c] = NAN;     // an infinite logit makes the row NaN
        const int s = (i >> 1) * 4 + (i & 1) * 2 + k;
        qf[s][r] = pack_f16x2(f[0], f[1]);
        qf[s][2 + r] = pack_f16x2(f[2], f[3]);
      }
    }
  }

  float o[kSets][kTilesM][4];
#pragma unroll
  for (int e = 0; e < kSets; ++e)
#pragma unroll
    for (int i = 0; i < kTilesM; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) o[e][i][k] = 0.f;
  float m_run[2] = {-INFINITY, -INFINITY}, s_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
  float l_low[2] = {0.f, 0.f};           // what l_run's additions rounded off

  // codes of 16 keys: K of keys g and g + 8 (channels 64 v + 16 t ..), V of keys 2t, 2t + 1, 2t + 8, 2t + 9
  // (channels g D / 8 ..)
  struct Codes {
    uint4 k[2][kKV];
    uint32_t v[4][kVW];
  };
  const int64_t row_bytes = static_cast<int64_t>(p.H) * D;
  const uint8_t* kbase = reinterpret_cast<const uint8_t*>(p.k) + static_cast<int64_t>(h) * D + 16 * t;
  const uint8_t* vbase = prm.v8 + static_cast<int64_t>(h) * D + g * (D / 8);
  auto load = [&](Codes& c, int64_t key0) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t key = key0 + g + 8 * r;
#pragma unroll
      for (int i = 0; i < kKV; ++i)
        c.k[r][i] = key < p.N ? __ldg(reinterpret_cast<const uint4*>(kbase + key * row_bytes + 64 * i))
                              : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t key = key0 + 2 * t + (r & 1) + 8 * (r >> 1);
      const uint8_t* at = vbase + key * row_bytes;
      if constexpr (D == 128) {
        const uint4 x = key < p.N ? __ldg(reinterpret_cast<const uint4*>(at)) : make_uint4(0u, 0u, 0u, 0u);
        c.v[r][0] = x.x;
        c.v[r][1] = x.y;
        c.v[r][2] = x.z;
        c.v[r][3] = x.w;
      } else {
        const uint2 x = key < p.N ? __ldg(reinterpret_cast<const uint2*>(at)) : make_uint2(0u, 0u);
        c.v[r][0] = x.x;
        c.v[r][1] = x.y;
      }
    }
  };

  auto step = [&](const Codes& c, int64_t key0, const float (&cc)[2], float lv, float (&share)[kSets]) {
    // ---- S = Q K^T: sf[n] = rows g, g + 8 x keys 8 n + 2t, 8 n + 2t + 1 -----------------------------
    // (even and odd steps apart: the four chains of products are half as long)
    float sf[2][4], sg[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) sf[n][k] = sg[n][k] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint4 x = c.k[n][s >> 2];
        const uint32_t w = (s & 3) == 0 ? x.x : ((s & 3) == 1 ? x.y : ((s & 3) == 2 ? x.z : x.w));
        mma_f16((s & 1) ? sg[n] : sf[n], qf[s], e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
      }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) sf[n][k] += sg[n][k];
    const bool whole = key0 + kKeys <= p.N;
    if (!whole) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (key0 + 8 * n + 2 * t + (k & 1) >= p.N) sf[n][k] = -INFINITY;
    }
    // ---- P' against the running reference, which moves when a sum outgrows f16 -------------------------
    float pf[kSets][4];                // set e: keys 2t, 2t + 1, 2t + 8, 2t + 9 of row g + 8 e
    float lt[kSets];
    auto probabilities = [&]() {
#pragma unroll
      for (int e = 0; e < kSets; ++e) {
        const float add = lv - m_run[e];
        lt[e] = 0.f;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            pf[e][2 * n + k] = fast_exp2(fmaf(sf[n][2 * e + k], cc[e], add));
            lt[e] += pf[e][2 * n + k];
          }
      }
    };
    probabilities();                   // (no reference yet: sums are +inf)
    bool outgrown = !whole;
#pragma unroll
    for (int e = 0; e < kSets; ++e) outgrown = outgrown || !(lt[e] <= kSumLimit && share[e] <= kShareMax);
    if (__any_sync(0xffffffffu, outgrown)) {
#pragma unroll
      for (int e = 0; e < kSets; ++e) {
        float mx = fmaxf(fmaxf(sf[0][2 * e], sf[0][2 * e + 1]), fmaxf(sf[1][2 * e], sf[1][2 * e + 1]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // a step has a key below N, so the maximum is finite (or S is NaN, and so is the row); m stays -inf
        // until a key has a value
        mx *= cc[e];
        const float m_new = fmaxf(m_run[e], mx + (lv - kRaise)), s_new = fmaxf(s_run[e], mx);
        const float alpha = m_run[e] == -INFINITY ? 0.f : fast_exp2(m_run[e] - m_new);
        m_run[e] = m_new;
        const float beta = fast_exp2(s_run[e] - s_new);
        l_run[e] *= beta;
        l_low[e] *= beta;
        s_run[e] = s_new;
        share[e] = share_of(m_new, lv, s_new);
        const float a0 = __shfl_sync(0xffffffffu, alpha, 8 * t), a1 = __shfl_sync(0xffffffffu, alpha, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < kTilesM; ++i) {    // O^T holds rows 2t and 2t + 1
          o[e][i][0] *= a0;
          o[e][i][1] *= a1;
          o[e][i][2] *= a0;
          o[e][i][3] *= a1;
        }
      }
      probabilities();
      bool alone = false;
#pragma unroll
      for (int e = 0; e < kSets; ++e) alone = alone || !(share[e] <= kShareMax);
      if (__any_sync(0xffffffffu, alone)) {
#pragma unroll
        for (int e = 0; e < kSets; ++e) {
          float sum = 0.f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              sum += fast_exp2(fmaf(sf[n][2 * e + k], cc[e], -s_run[e]));
              if (lv == -INFINITY) pf[e][2 * n + k] = 0.f;
            }
          add_low(l_low[e] + sum, l_run[e], l_low[e]);
          lt[e] = 0.f;
        }
      }
    }
    // ---- O^T += V^T P'^T ---------------------------------------------------------------------------------
    uint32_t pb[kSets][2];
#pragma unroll
    for (int e = 0; e < kSets; ++e) {
      add_low(fmaf(lt[e], share[e], l_low[e]), l_run[e], l_low[e]);
      pb[e][0] = pack_f16x2(pf[e][0], pf[e][1]);
      pb[e][1] = pack_f16x2(pf[e][2], pf[e][3]);
    }
#pragma unroll
    for (int w = 0; w < kVW; ++w) {
      // channels 4 w .. 4 w + 3 of the key pairs (2t, 2t + 1) and (2t + 8, 2t + 9), interleaved
      uint32_t z[2][2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        z[r][0] = __byte_perm(c.v[2 * r][w], c.v[2 * r + 1][w], 0x5140);
        z[r][1] = __byte_perm(c.v[2 * r][w], c.v[2 * r + 1][w], 0x7362);
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t a[4] = {e4m3x2_to_f16x2(z[0][k]), e4m3x2_to_f16x2(z[0][k] >> 16), e4m3x2_to_f16x2(z[1][k]),
                               e4m3x2_to_f16x2(z[1][k] >> 16)};
#pragma unroll
        for (int e = 0; e < kSets; ++e) mma_f16(o[e][2 * w + k], a, pb[e][0], pb[e][1]);
      }
    }
  };

  // ---- the keys -------------------------------------------------------------------------------------------
  const int first = b0 + warp;
  Codes buf[2];
  if (first < b1) load(buf[0], static_cast<int64_t>(first) * kScaleBlock);
  for (int b = first; b < b1; b += kWarps) {
    const int64_t at = static_cast<int64_t>(b) * p.H + h;
    const float ks = __ldg(prm.ks + at);
    const float lv = log2_scale(__ldg(prm.vs + at));
    float share[kSets];
#pragma unroll
    for (int e = 0; e < kSets; ++e) share[e] = share_of(m_run[e], lv, s_run[e]);
    const float cc[2] = {fmaxf(rowc[0] * ks, kFactorMin), fmaxf(rowc[1] * ks, kFactorMin)};
    const int64_t key0 = static_cast<int64_t>(b) * kScaleBlock;
    const int nstep = static_cast<int>(((p.N - key0 < kScaleBlock ? p.N - key0 : kScaleBlock) + kKeys - 1) / kKeys);
    const int64_t next_block = b + kWarps < b1 ? key0 + static_cast<int64_t>(kWarps) * kScaleBlock : p.N;
#pragma unroll 1
    for (int i = 0; i < nstep; i += 2) {       // two steps, so that the two buffers keep their registers
      const int64_t k0 = key0 + i * kKeys;
      load(buf[1], i + 1 < nstep ? k0 + kKeys : p.N);
      step(buf[0], k0, cc, lv, share);
      load(buf[0], i + 2 < nstep ? k0 + 2 * kKeys : next_block);
      if (i + 1 < nstep) step(buf[1], k0 + kKeys, cc, lv, share);
    }
  }

  // ---- merge: the warps of the CTA -----------------------------------------------------------------------
#pragma unroll
  for (int e = 0; e < kSets; ++e) {
    float l = l_run[e];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (t == 0) s_msl[warp][8 * e + g] = make_float4(m_run[e], s_run[e], l, 0.f);
#pragma unroll
    for (int i = 0; i < kTilesM; ++i) {
      const int ch = g * (D / 8) + 2 * i;
      *reinterpret_cast<float2*>(&s_o[warp][8 * e + 2 * t][ch]) = make_float2(o[e][i][0], o[e][i][2]);
      *reinterpret_cast<float2*>(&s_o[warp][8 * e + 2 * t + 1][ch]) = make_float2(o[e][i][1], o[e][i][3]);
    }
  }
  __syncthreads();
  for (int i = tid; i < rows * (D / 4); i += kThreads) {
    const int r = i / (D / 4), c4 = i % (D / 4);
    float ref = -INFINITY, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ref = fmaxf(ref, s_msl[w][r].y);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) l = fmaf(part_weight(s_msl[w][r].y, s_msl[w][r].z, ref), s_msl[w][r].z, l);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = value_weight(s_msl[w][r].x, ref) * inv;   // (a weight of 0 keeps a NaN of V)
      const float4 x = *reinterpret_cast<const float4*>(&s_o[w][r][4 * c4]);
      a.x = fmaf(f, x.x, a.x);
      a.y = fmaf(f, x.y, a.y);
      a.z = fmaf(f, x.z, a.z);
      a.w = fmaf(f, x.w, a.w);
    }
    const float lse = l == 0.f ? -INFINITY : (ref + log2f(l)) * kLn2;
    const int64_t orow = static_cast<int64_t>(r) * p.H + h;
    if (gridDim.y > 1) {
      const int64_t prow = static_cast<int64_t>(blockIdx.y) * prm.part_rows * p.H + orow;
      reinterpret_cast<float4*>(prm.o_part + prow * D)[c4] = a;
      if (c4 == 0) prm.lse_part[prow] = lse;
    } else {
      reinterpret_cast<uint2*>(p.o + orow * D)[c4] =
          make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
      if (c4 == 0 && p.lse) p.lse[orow] = lse;
    }
  }
}

}  // namespace

int launch_attn_q8_few(const Q8Args& prm, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(prm.a.H), static_cast<unsigned>(prm.nsplit));
  const bool one = few_sets(prm.a.cap) == 1;
  if (prm.a.d == 128 && one) attn_q8_few_kernel<128, 1><<<grid, kThreads, 0, st>>>(prm);
  else if (prm.a.d == 128) attn_q8_few_kernel<128, 2><<<grid, kThreads, 0, st>>>(prm);
  else if (one) attn_q8_few_kernel<64, 1><<<grid, kThreads, 0, st>>>(prm);
  else attn_q8_few_kernel<64, 2><<<grid, kThreads, 0, st>>>(prm);
  return launch_status("pruned_attn_q8");
}

// Key ranges of a head, from the time in units of a warp's block (2.6 us while latency counts): waves of CTAs times
// the most blocks of a warp and kEnds for the rest of a CTA, and the merge. One block a warp is enough: 8 rows x 64
// over 11,501 keys, 5 heads, took 12.7 us in 11 ranges (3 blocks) and take 8.7 us in 23 (one). A wave that is
// not full costs more than longer ranges: 16 rows (2 CTAs per SM) over 118,800 keys, 24 heads: 157 us in 12 ranges,
// 187 us in 18.
int few_split(int64_t cap, int64_t N, int H) {
  constexpr double kEnds = 2.0, kMerge = 0.6, kPart = 0.03;
  const int64_t nb = (N + kScaleBlock - 1) / kScaleBlock;
  const int64_t resident = static_cast<int64_t>(sm_count()) * few_ctas(few_sets(cap));
  int best = 1;
  double cost = 1e300;
  for (int s = 1; s <= kFewMaxSplit && (s == 1 || s * kWarps < nb + kWarps); ++s) {
    const int64_t waves = (static_cast<int64_t>(H) * s + resident - 1) / resident;
    const int64_t blocks = ((nb + s - 1) / s + kWarps - 1) / kWarps;
    const double c = static_cast<double>(waves) * (blocks + kEnds) + (s > 1 ? kMerge + kPart * s : 0.0);
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

}  // namespace tps
