// rope_rows: rows of Q (and K) turned to the rotary position of their token on
// the latent grid, or turned back (the gradient of the turn).
//
// [TR] "Timeripple", Metodologia 1: a head's rotary channels form temporal, x
// and y groups. [LIPAR] Dutch summary 2.C takes the RoPE rotations into account
// when keys are reused. Pair j of group a of token n turns by
// position_a(n) * base^(-2j / dims[a]):
//   (x, y) -> (x cos - y sin, x sin + y cos);
// the turn back negates the sine (R is orthogonal, so R^T = R^-1 is the gradient).
//
// HBM-bound: 4 bytes per element (2 read, 2 written). A warp owns 4 vectors of
// 16 bytes per lane of one row (blockIdx.y picks the tensor and the part of the row); a
// lane's vectors all hold the same channels of different heads, so its four
// (cos, sin) entries are looked up once, from a table that stays in L1, while
// the row's loads are in flight. Q and K of the HSA step (39,600 rows of 24 x 128
// channels each, 0.97 GB): 163 us, 5.97 TB/s, 91% of the measured copy rate.
#include <cmath>

#include "rope_grid.cuh"
#include "trace.cuh"

namespace tps {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;   // 16-byte vectors per lane and row part

struct RopeRows {
  const uint4* src[2];
  uint4* dst[2];
  const int32_t* idx;
  const int32_t* count;
  int64_t cap;
  int64_t N;
  int vpr;      // 16-byte vectors per row
  int vph;      // ... per head (8 or 16)
  int parts;    // row parts of 32 * kUnroll vectors
  float sign;   // +1, or -1 for the turn back
  RopeGrid grid;
  unsigned int* status;
};

__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const __grid_constant__ RopeRows p) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = p.count ? active_count(p.count, p.cap) : p.cap;
  const int tensor = blockIdx.y / p.parts;
  const int v0 = (blockIdx.y - tensor * p.parts) * (32 * kUnroll) + lane;
  const uint4* src = p.src[tensor];
  uint4* dst = p.dst[tensor];
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t j = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); j < rows; j += nwarps) {
    uint4 x[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (v0 + 32 * u < p.vpr) x[u] = src[j * p.vpr + v0 + 32 * u];
    const int64_t n = p.idx ? p.idx[j] : j;
    if (n < 0 || n >= p.N) {
      if (lane == 0 && blockIdx.y == 0) raise_status(p.status, STATUS_BOUNDS);
      continue;
    }
    float2 cs[4];
    rope_lookup(p.grid, static_cast<uint32_t>(n), (lane % p.vph) * 4, cs);   // 32 % vph == 0
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i].y *= p.sign;
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (v0 + 32 * u >= p.vpr) continue;
      const float2 a = rope_turn(x[u].x, cs[0]), b = rope_turn(x[u].y, cs[1]);
      const float2 c = rope_turn(x[u].z, cs[2]), d = rope_turn(x[u].w, cs[3]);
      dst[j * p.vpr + v0 + 32 * u] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(b.x, b.y), pack_bf16x2(c.x, c.y),
                                                pack_bf16x2(d.x, d.y));
    }
  }
}

}  // namespace
}  // namespace tps

using namespace tps;

extern "C" int tps_rope_table(float* table, const int32_t* dims, const int32_t* size, const int32_t* origin,
                              float base) {
  if (!table || !dims || !size || !origin) return fail(TPS_ERR_INVALID_ARG, "tps_rope_table: null pointer");
  if (!(base > 0.f) || !std::isfinite(base))
    return fail(TPS_ERR_INVALID_ARG, "tps_rope_table: base must be finite and > 0");
  for (int a = 0; a < 3; ++a) {
    if (dims[a] < 0 || dims[a] % 2)
      return fail(TPS_ERR_INVALID_ARG, "tps_rope_table: group %d has %d channels (must be even and >= 0)", a, dims[a]);
    if (size[a] < 1 || size[a] > (1 << 24) || origin[a] < -(1 << 24) || origin[a] > (1 << 24))
      return fail(TPS_ERR_SHAPE, "tps_rope_table: axis %d needs 1 <= size <= 2^24 and |origin| <= 2^24", a);
  }
  for (int a = 0; a < 3; ++a) {
    const int half = dims[a] / 2;
    for (int64_t s = 0; s < size[a]; ++s)
      for (int j = 0; j < half; ++j) {
        const double phi = static_cast<double>(origin[a] + s) *
                           std::pow(static_cast<double>(base), -2.0 * j / static_cast<double>(dims[a]));
        *table++ = static_cast<float>(std::cos(phi));
        *table++ = static_cast<float>(std::sin(phi));
      }
  }
  return ok();
}

extern "C" int rope_rows(tps_bf16* dst, const tps_bf16* src, tps_bf16* dst2, const tps_bf16* src2, const int32_t* idx,
                         const int32_t* count, int64_t cap, int64_t N, int H, int d, const tps_rope_grid* rope,
                         int inverse, tps_stream stream) {
  TPS_TRACE("rope_rows");
  if (!dst || !src || !rope) return fail(TPS_ERR_INVALID_ARG, "rope_rows: null pointer");
  if (!dst2 != !src2) return fail(TPS_ERR_INVALID_ARG, "rope_rows: dst2 and src2 go together");
  if (idx && !count) return fail(TPS_ERR_INVALID_ARG, "rope_rows: idx needs count");
  if (cap < 0 || cap >= (INT64_C(1) << 31) || N < 1 || N >= (INT64_C(1) << 31))
    return fail(TPS_ERR_SHAPE, "rope_rows: need 0 <= cap < 2^31 and 1 <= N < 2^31");
  if (!idx && cap > N) return fail(TPS_ERR_SHAPE, "rope_rows: without idx, cap must be <= N");
  if (d != 64 && d != 128) return fail(TPS_ERR_INVALID_ARG, "rope_rows: d=%d must be 64 or 128", d);
  if (H < 1 || static_cast<int64_t>(H) * d > 16384)
    return fail(TPS_ERR_SHAPE, "rope_rows: H=%d must satisfy 1 <= H*d <= 16384", H);
  if (!aligned16(dst) || !aligned16(src) || !aligned16(dst2) || !aligned16(src2))
    return fail(TPS_ERR_ALIGN, "rope_rows: rows must be 16-byte aligned");
  RopeRows p{};
  if (int e = rope_grid_check("rope_rows", rope, N, d, &p.grid)) return e;
  if (cap == 0) return ok();
  int err;
  p.status = device_status(&err);
  if (!p.status) return err;
  p.src[0] = reinterpret_cast<const uint4*>(src);
  p.dst[0] = reinterpret_cast<uint4*>(dst);
  p.src[1] = reinterpret_cast<const uint4*>(src2);
  p.dst[1] = reinterpret_cast<uint4*>(dst2);
  p.idx = idx;
  p.count = count;
  p.cap = cap;
  p.N = N;
  p.vpr = H * d / 8;
  p.vph = d / 8;
  p.parts = (p.vpr + 32 * kUnroll - 1) / (32 * kUnroll);
  p.sign = inverse ? -1.f : 1.f;
  const int ny = p.parts * (src2 ? 2 : 1);
  int64_t g = (cap + kWarps - 1) / kWarps;
  const int64_t gmax = (static_cast<int64_t>(sm_count()) * 16 + ny - 1) / ny;
  g = g > gmax ? gmax : g;
  rope_rows_kernel<<<dim3(static_cast<unsigned>(g), static_cast<unsigned>(ny)), kThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(p);
  if (int e = launch_status("rope_rows")) return e;
  return ok();
}
