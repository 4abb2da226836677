// Rotary positions on the latent grid: the host-side check of a tps_rope_grid
// and the device-side lookup of a token's (cos, sin) entries, shared by
// rope_rows and kv_sync_q8.
//
// A head's d channels are the groups [t | x | y] of dims[0..2] channels; the
// adjacent channels (o_a + 2j, o_a + 2j + 1) of group a are pair j. Token
// n = (f * Hs + y) * Ws + x has the positions (f, x, y). The table holds the
// axes one after the other, entry (position, pair) of axis a at
// off_a + position * dims[a] / 2 + pair.
#pragma once

#include "tps_internal.cuh"

namespace tps {

struct RopeGrid {
  const float2* tab;
  uint32_t Ws, HW;       // grid width, tokens of a frame
  uint32_t Hs;
  int end0, end1;        // pairs [0, end0) turn with t, [end0, end1) with x, the rest with y
  int half[3];           // dims[a] / 2
  uint32_t off[3];       // first entry of axis a
};

// Checks a rope grid against the call's N and d and fills `r`.
inline int rope_grid_check(const char* who, const tps_rope_grid* g, int64_t N, int d, RopeGrid* r) {
  if (!g || !g->table) return fail(TPS_ERR_INVALID_ARG, "%s: rope grid and its table must be non-null", who);
  int64_t cells = 1, off = 0;
  int sum = 0;
  for (int a = 0; a < 3; ++a) {
    if (g->dims[a] < 0 || g->dims[a] > d || g->dims[a] % 2)
      return fail(TPS_ERR_INVALID_ARG, "%s: rope group %d has %d channels (must be even and in [0, d])", who, a,
                  g->dims[a]);
    if (g->size[a] < 1 || g->size[a] > (1 << 24))
      return fail(TPS_ERR_SHAPE, "%s: rope axis %d has %d positions (must be in [1, 2^24])", who, a, g->size[a]);
    sum += g->dims[a];
    cells *= g->size[a];
    if (cells > N) return fail(TPS_ERR_SHAPE, "%s: the rope grid has more than N=%lld tokens", who, static_cast<long long>(N));
    r->half[a] = g->dims[a] / 2;
    r->off[a] = static_cast<uint32_t>(off);
    off += static_cast<int64_t>(g->size[a]) * (g->dims[a] / 2);
  }
  if (sum != d) return fail(TPS_ERR_INVALID_ARG, "%s: rope groups sum to %d channels, d=%d", who, sum, d);
  if (cells != N)
    return fail(TPS_ERR_SHAPE, "%s: the rope grid has %lld tokens, N=%lld", who, static_cast<long long>(cells),
                static_cast<long long>(N));
  if (!aligned16(g->table)) return fail(TPS_ERR_ALIGN, "%s: the rope table must be 16-byte aligned", who);
  r->tab = reinterpret_cast<const float2*>(g->table);
  r->Ws = static_cast<uint32_t>(g->size[1]);
  r->Hs = static_cast<uint32_t>(g->size[2]);
  r->HW = r->Ws * r->Hs;
  r->end0 = r->half[0];
  r->end1 = r->half[0] + r->half[1];
  return TPS_OK;
}

// The (cos, sin) entries of pairs p0 .. p0+3 for token n.
__device__ __forceinline__ void rope_lookup(const RopeGrid& g, uint32_t n, int p0, float2 (&cs)[4]) {
  const uint32_t f = n / g.HW, in = n - f * g.HW;
  const uint32_t y = in / g.Ws, x = in - y * g.Ws;
  const uint32_t b0 = g.off[0] + f * g.half[0];
  const uint32_t b1 = g.off[1] + x * g.half[1] - g.end0;
  const uint32_t b2 = g.off[2] + y * g.half[2] - g.end1;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int p = p0 + i;
    cs[i] = __ldg(g.tab + ((p < g.end0 ? b0 : (p < g.end1 ? b1 : b2)) + p));
  }
}

// (x, y) -> (x cos - y sin, x sin + y cos) on one word of two bf16
__device__ __forceinline__ float2 rope_turn(uint32_t w, float2 cs) {
  const float x = bf16lo(w), y = bf16hi(w);
  return make_float2(fmaf(x, cs.x, -y * cs.y), fmaf(x, cs.y, y * cs.x));
}

}  // namespace tps
