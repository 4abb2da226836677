// pruned_attn_q8: active queries attend all N keys of a cache held in 8 bits
// (e4m3 codes, one scale for each block of 128 tokens, head and tensor), on the
// Blackwell tensor cores (tcgen05 + TMEM + TMA).
//
// [HSA] 2.2 (3)-(4): the active tokens' queries attend the full cached K/V.
// [SVOO] part 2: with a mask, a query attends only the 128-key blocks that its
// ORIGINAL 128-token block keeps.
//
// The mathematics, for query row i, key n of block b (a key tile is one scale block):
//   x = scale log2(e) ks_b (q_i . k8_n),  o_i = sum_n 2^(x - m) vs_b v8_n / sum_n 2^(x - m).
// Nothing of the cache is dequantised to the scaled value:
// - Q K^T runs as e4m3 MMAs on the codes. A bf16 value has 8 significant bits and an
//   e4m3 value 4, so q = 2^e (hi + lo) with hi = e4m3(q / 2^e), lo = e4m3(rest) and one
//   power of two per row with amax(q) <= 448 * 2^e: exact for channels down to 2^-9 of
//   the row's largest, and within 2^-17 of the largest below that. Two e4m3 MMAs cost what
//   one bf16 MMA costs, K stays 8 bits wide in shared memory, and no key is converted.
// - ks_b enters as the factor of the exponent's FMA. vs_b enters as log2(vs_b) in its
//   addend, so that P' = 2^(x + log2 vs_b - m) multiplies the codes of V directly; the row
//   sum takes P' / vs_b, with a reference of its own (attn_q8.cuh). Neither costs an
//   instruction per element, but in blocks whose vs_b is 0 or 2^60 below others'.
// - P' V needs V as wide as P: four converter warps turn the codes into f16 (exact, e4m3 is
//   a subset of f16) on the way from global to the swizzled shared tile. P' is f16: 11
//   bits against bf16's 8 make its rounding (2^-11 per probability) vanish beside the
//   output's. The reference m is up to 2^8 below the running maximum of x + log2 vs_b, the more the
//   longer the range (attn_q8.cuh), so that what underflows is below 2^-13 of the row; P' <= 2^15 always (kSumLimit).
//
// Two layouts of a CTA's two 128-row MMA tiles t = 0, 1 (template kOneSet):
// - false: 256 compacted rows of one head; both tiles consume every K/V tile.
// - true: one set of at most 128 rows (few active tokens, or the rows of one
//   query block when a mask is given); tile t takes every second key tile, and the
//   two partial results are merged through shared memory at the end. A masked row set
//   streams only the key tiles its query block keeps, so a block that is not kept is
//   never read, whatever it holds.
// Warps: 0-3 / 4-7 softmax of tile 0 / 1 (one TMEM lane = one row per thread), 8-11 converters of V, 12 TMA
// producer, 13 MMA issuer and TMEM owner, 14 MMA issuer of tile 1 (one set), 15 idle. Every wait is bounded: on
// expiry the CTA sets the device status word (TPS_ERR_TIMEOUT), drains what it issued, frees TMEM and returns.
//
// What bounds it, and what the steps towards it measured (middle video, 6,084 rows x 20,280 keys, 12 heads, d =
// 128, 0.758 TFLOP; single calls; clocks of an SM per step of 256 rows x 128 keys):
//   MMAs alone: 2,484 clocks (S in halves of N = 64: 50.7 clocks each, bound by the shared-memory reads of Q;
//   P' V 65.6 each); exp2 on 16 lanes a clock: 2,048.
//   - first form, descriptors built before each MMA by "lane 0": 897 us (a step 4,900 clocks, the issuer 100
//     clocks per MMA);
//   - one elected thread and precomputed descriptors (22 clocks per MMA): 760 us;
//   - S through the registers 32 columns at a time instead of 128 (no spills): 680 us;
//   - S in two halves per tile, so that MMAs run under the exponentials: 620 us;
//   - registers moved to the roles that spilled, Q's parts made by rows: 616 us;
//   - the sum against a reference of its own, with a factor per tile instead of a division: 608 us = 1,250 TFLOP/s.
// Back to back the GPU's power limit holds it to 690-715 us (1.70 GHz), and the bf16 kernel, which reads twice the
// cache, to 675-715. With d = 64 the exponentials bound it: 552 us for the same rows and keys, of which exp2 alone
// takes 318 at 1.965 GHz (unit 66% active, tensor pipe 32%); the bf16 kernel takes 543-553.
#include "attn_q8.cuh"
#include "q8.cuh"
#include "tc_ptx.cuh"
#include "tma_host.cuh"
#include "trace.cuh"
#include "warp_search.cuh"

namespace tps {
namespace {

using namespace tc;

constexpr int kBM = 128;        // rows of an MMA tile
constexpr int kBN = 128;        // keys of a tile = scale block = mask block
constexpr int kTiles = 2;
constexpr int kSoftmaxThreads = kTiles * kBM;
constexpr int kConvThreads = 128;
constexpr int kThreads = kSoftmaxThreads + kConvThreads + 128;
constexpr int kConvWarp = kSoftmaxThreads / 32;
constexpr int kTmaWarp = kConvWarp + kConvThreads / 32;
constexpr int kMmaWarp = kTmaWarp + 1;
// 16 warps launch with 128 registers per thread; the warpgroups re-divide them
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 144, kConvRegs = 104, kProducerRegs = 120;
static_assert(8 * kSoftmaxRegs + 4 * kConvRegs + 4 * kProducerRegs <= 16 * kLaunchRegs, "register split");
constexpr int kTmemCols = 512;
constexpr int kListMax = 4096;
constexpr float kSumLimit = 32768.f;   // largest sum of a row's half tile kept without a new reference: P' stays finite in f16
static_assert(64.f * (1 << kRaise) <= kSumLimit, "a half tile against its own reference: 64 P' of 2^kRaise");
static_assert(kBN == kScaleBlock, "a key tile has one scale");

template <int D, bool kOneSet>
struct Layout {
  // A wait on a barrier's parity tells a phase from its neighbours only: a role must have seen phase n of a
  // stage before it waits for phase n + 1. With one set the two issuers take alternate tiles and each waits
  // for its own alone, so their rings (K, V) have an even number of stages: a stage then belongs to one issuer.
  // (With three K stages issuer 1 could take tile 0's stage for tile 3's before tile 0 had landed.)
  static constexpr int kKStages = D == 64 || kOneSet ? 4 : 3;
  static constexpr int kVStages = D == 64 ? 4 : (kOneSet ? 2 : 3);
  static_assert(!kOneSet || (kKStages % kTiles == 0 && kVStages % kTiles == 0), "a stage belongs to one issuer");
  // kOneSet: V's codes come through a ring of their own, so that enough bytes are in flight to stream a
  // long cache for few rows (one tile ahead in the converters' registers reached 2.2 TB/s)
  static constexpr int kCStages = kOneSet ? (D == 64 ? 6 : 3) : 0;
  static constexpr int kQPart = kBM * D;                 // one e4m3 tile
  static constexpr int kKTile = kBN * D;
  static constexpr int kSub = kBN * 128;                 // [128 keys x 64 f16], 128-byte swizzle
  static constexpr int kVTile = (D / 64) * kSub;
  static constexpr int kV = 0;
  static constexpr int kK = kV + kVStages * kVTile;
  static constexpr int kC = kK + kKStages * kKTile;      // V's codes
  static constexpr int kQ = kC + kCStages * kKTile;      // [tile][hi, lo]; not first: see the lane shift
  static constexpr int kList = kQ + (kOneSet ? 1 : kTiles) * 2 * kQPart;   // uint16 kept key blocks (kOneSet)
  static constexpr int kBar = kList + (kOneSet ? 2 * kListMax : 0);
  static constexpr int kBytes = kBar + 512;
  static constexpr int kAlloc = kBytes + 1024;           // slack for 1024-byte alignment
  // mbarrier indices
  static constexpr int q_full = 0;
  // + 2 * tile + half: each has one phase per key tile. (One barrier for both halves would let a warp that
  // is through with its second half arrive in the place of one that is still at its first.)
  static constexpr int s_full = q_full + 1;
  static constexpr int p_full = s_full + 2 * kTiles;
  static constexpr int o_part = p_full + 2 * kTiles;     // + tile: the last step's first half is in O_t
  static constexpr int o_full = o_part + kTiles;         // + tile: all of O_t
  static constexpr int k_full = o_full + kTiles;         // + stage
  static constexpr int k_empty = k_full + kKStages;
  static constexpr int v_full = k_empty + kKStages;
  static constexpr int v_empty = v_full + kVStages;
  static constexpr int c_full = v_empty + kVStages;
  static constexpr int c_empty = c_full + kCStages;
  static constexpr int drain = c_empty + kCStages;
  static_assert((drain + 1) * 8 <= 512, "barrier block");
  static_assert(kAlloc + 1536 <= 232448, "shared memory, with the static part");
  // the merge of the two tiles stages half of 2 x 128 fp32 rows over the V and K rings
  static_assert(!kOneSet || kVStages * kVTile + kKStages * kKTile >= kBM * D * 4, "merge staging");
};

__device__ __forceinline__ void barrier_all() { asm volatile("barrier.sync 0;" ::: "memory"); }
__device__ __forceinline__ void barrier_softmax() {
  asm volatile("barrier.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory");
}

// P' = 2^(S * c - base) of 32 columns as f16 pairs; the unrounded P' are added to acc.
__device__ __forceinline__ void exp_cols_f16(const uint32_t (&sr)[32], uint64_t c2, uint64_t nb2, uint32_t* pk,
                                             uint64_t (&acc)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 4) {
    const uint64_t a01 = ffma2(f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1])), c2, nb2);
    const uint64_t a23 = ffma2(f2_pack(__uint_as_float(sr[i + 2]), __uint_as_float(sr[i + 3])), c2, nb2);
    float a0, a1, a2, a3;
    f2_unpack(a01, a0, a1);
    f2_unpack(a23, a2, a3);
    const float p0 = fast_exp2(a0), p1 = fast_exp2(a1), p2 = fast_exp2(a2), p3 = fast_exp2(a3);
    acc[0] = fadd2(acc[0], f2_pack(p0, p1));
    acc[1] = fadd2(acc[1], f2_pack(p2, p3));
    pk[i >> 1] = pack_f16x2(p0, p1);
    pk[(i >> 1) + 1] = pack_f16x2(p2, p3);
  }
}

template <int D, bool kOneSet>
__global__ void __launch_bounds__(kThreads, 1)
attn_q8_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
               const __grid_constant__ Q8Args prm) {
  using L = Layout<D, kOneSet>;
  constexpr int kIssuers = kOneSet ? kTiles : 1;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ int s_run[2];
  __shared__ float s_rowc[(kOneSet ? 1 : kTiles) * kBM];   // scale * log2(e) * 2^e of each row of Q
  __shared__ volatile int s_abort;
  __shared__ unsigned int s_wcnt[kThreads / 32];
  constexpr int kChunks = D / 8;                    // 16-byte chunks of half a row of O

  const AttnArgs& p = prm.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.y;
  const int64_t rows = active_count(p.count, p.cap);
  const bool masked = kOneSet && p.bm != nullptr;

  // ---- this CTA's rows: [row0, row0 + nrows) of the compacted queries -----------------------
  int64_t row0 = (static_cast<int64_t>(blockIdx.x) + prm.tile0) * (kOneSet ? kBM : kTiles * kBM);
  int nrows = static_cast<int>(rows - row0 < kTiles * kBM ? rows - row0 : kTiles * kBM);
  if constexpr (kOneSet) {
    if (masked) {
      // lower bounds in idx of this query block and of the next (or of N)
      if (warp < 2) {
        const int64_t key = (static_cast<int64_t>(blockIdx.x) + warp) * kBN;
        const int64_t at = warp_lower_bound(p.idx, rows, key < p.N ? key : p.N, lane);
        if (lane == 0) s_run[warp] = static_cast<int>(at);
      } else if (warp == 2 && h == 0 && blockIdx.x == 0 && rows > 0 && lane == 0 &&
                 (p.idx[0] < 0 || p.idx[rows - 1] >= p.N)) {
        raise_status(prm.status, STATUS_BOUNDS);   // entries outside [0, N): those rows are skipped
      }
      __syncthreads();
      row0 = s_run[0];
      nrows = s_run[1] - s_run[0];
      if (nrows > kBM) {                           // more rows than tokens: an index repeated
        if (tid == 0 && h == 0) raise_status(prm.status, STATUS_BOUNDS);
        nrows = kBM;
      }
    } else if (nrows > kBM) {
      nrows = kBM;
    }
  }
  if (nrows <= 0) return;   // uniform: before TMEM or barriers

  const uint32_t sbase = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (sbase - smem_u32(smem_raw));
  const uint32_t bar0 = sbase + L::kBar;
  auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
  uint16_t* sList = reinterpret_cast<uint16_t*>(gbase + L::kList);

  // ---- setup: barriers, TMEM, key tiles ---------------------------------------------------------
  const int rows_t0 = nrows < kBM ? nrows : kBM;
  const int rows_t1 = kOneSet ? rows_t0 : (nrows > kBM ? nrows - kBM : 0);
  // Warp w of tile t (lanes 32 w .. 32 w + 31) works if it has a row; warp 0's row 0 always counts as one.
  // One set of at most 64 rows: tile 1 holds them in lanes 64-127 (its A operand starts 64 rows before Q's;
  // what lanes 0-63 then compute is not used), so that the two tiles' warps sit on different schedulers.
  const int shift = kOneSet && nrows <= kBM / 2 ? kBM / 2 : 0;
  auto first_row = [&](int t, int w) { return (w * 32 - (t == 1 ? shift : 0)) & (kBM - 1); };
  auto has_rows = [&](int t, int w) { return first_row(t, w) < (t ? rows_t1 : rows_t0) || first_row(t, w) == 0; };
  if (tid == 0) {
    s_abort = 0;
    mbar_init(bar(L::q_full), kSoftmaxThreads);
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(bar(L::o_part + t), 1);
      mbar_init(bar(L::o_full + t), 1);
      int warps = 0;                // that store P'_t
      for (int w = 0; w < 4; ++w) warps += has_rows(t, w) ? 1 : 0;
      for (int u = 0; u < 2; ++u) {
        mbar_init(bar(L::s_full + 2 * t + u), 1);
        mbar_init(bar(L::p_full + 2 * t + u), 32 * warps);
      }
    }
    for (int s = 0; s < L::kKStages; ++s) {
      mbar_init(bar(L::k_full + s), 1);
      mbar_init(bar(L::k_empty + s), 1);
    }
    for (int s = 0; s < L::kVStages; ++s) {
      mbar_init(bar(L::v_full + s), kConvThreads);
      mbar_init(bar(L::v_empty + s), 1);
    }
    for (int s = 0; s < L::kCStages; ++s) {
      mbar_init(bar(L::c_full + s), 1);
      mbar_init(bar(L::c_empty + s), kConvThreads);
    }
    mbar_init(bar(L::drain), kIssuers);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) tmem_alloc<kTmemCols>(smem_u32(&s_tmem));
  if (warp == kTmaWarp && lane == 0) {
    tma_prefetch_desc(&tmK);
    if (kOneSet) tma_prefetch_desc(&tmV);
  }
  const int nkt = static_cast<int>((p.N + kBN - 1) / kBN);
  // split z covers the key tiles [kt0, kt0 + ntiles)
  const int kt0 = static_cast<int>((static_cast<int64_t>(nkt) * blockIdx.z) / prm.nsplit);
  int ntiles = static_cast<int>((static_cast<int64_t>(nkt) * (blockIdx.z + 1)) / prm.nsplit) - kt0;
  if (masked) {
    // the key blocks this query block keeps, ascending
    const uint8_t* mrow = p.bm + static_cast<int64_t>(blockIdx.x) * p.nb;
    int base = 0;
    for (int kb0 = 0; kb0 < p.nb; kb0 += kThreads) {
      const int kb = kb0 + tid;
      const unsigned int m = __ballot_sync(0xffffffffu, kb < p.nb && mrow[kb] != 0);
      if (lane == 0) s_wcnt[warp] = __popc(m);
      __syncthreads();
      int off = base;
      for (int i = 0; i < kThreads / 32; ++i) {
        off += i < warp ? s_wcnt[i] : 0;
        base += s_wcnt[i];
      }
      if ((m >> lane) & 1u) sList[off + __popc(m & ((1u << lane) - 1u))] = static_cast<uint16_t>(kb);
      __syncthreads();
    }
    ntiles = base;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // S_t of half u of a key tile (64 keys); P'_t (f16 pairs) later takes its first 32 columns
  auto tS = [&](int t, int u) { return tmem + 256u * t + 64u * u; };
  auto tO = [&](int t) { return tmem + 256u * t + 128u; };
  // the loaded key tiles are numbered q = 0 .. ntiles - 1; step j of tile t reads tile seq(t, j)
  auto seq = [&](int t, int j) { return kOneSet ? 2 * j + t : j; };
  auto steps = [&](int t) { return kOneSet ? (ntiles - t + 1) / 2 : ntiles; };
  auto key_tile = [&](int q) -> int { return masked ? sList[q] : kt0 + q; };

  auto tma_role = [&]() {
    // ================================ TMA producer =====================================
    if (elect_one()) {
      int issued_k = 0, issued_c = 0;
      for (int q = 0; q < ntiles; ++q) {
        const int st = q % L::kKStages, key0 = key_tile(q) * kBN;
        if (q >= L::kKStages &&
            !mbar_wait(bar(L::k_empty + st), ((q / L::kKStages) - 1) & 1, &s_abort, prm.status))
          break;
        mbar_expect_tx(bar(L::k_full + st), L::kKTile);
        tma_load_3d(sbase + L::kK + st * L::kKTile, &tmK, 0, h, key0, bar(L::k_full + st));
        issued_k = q + 1;
        if constexpr (kOneSet) {
          const int sc = q % L::kCStages;
          if (q >= L::kCStages &&
              !mbar_wait(bar(L::c_empty + sc), ((q / L::kCStages) - 1) & 1, &s_abort, prm.status))
            break;
          mbar_expect_tx(bar(L::c_full + sc), L::kKTile);
          tma_load_3d(sbase + L::kC + sc * L::kKTile, &tmV, 0, h, key0, bar(L::c_full + sc));
          issued_c = q + 1;
        }
      }
      // every load issued above must land before the CTA may exit
      for (int q = issued_k > L::kKStages ? issued_k - L::kKStages : 0; q < issued_k; ++q)
        drain_wait(bar(L::k_full + q % L::kKStages), (q / L::kKStages) & 1);
      if constexpr (kOneSet)
        for (int q = issued_c > L::kCStages ? issued_c - L::kCStages : 0; q < issued_c; ++q)
          drain_wait(bar(L::c_full + q % L::kCStages), (q / L::kCStages) & 1);
    }
    __syncwarp();
  };

  auto conv_role = [&]() {
    // ================================ V converters ======================================
    // kLanes threads hold a key's D codes (16 each), kRows keys at a time. The swizzle of a thread's chunks
    // is the same in every pass (kRows is a multiple of 8): channels 16 l .. 16 l + 15 are the 16-byte chunks
    // 2 l and 2 l + 1 of the f16 row; with D = 128 lanes 4-7 (second 64-channel sub-tile) store theirs in the
    // other order, so 8 lanes cover all banks.
    constexpr int kLanes = D / 16;
    constexpr int kRows = kConvThreads / kLanes;   // keys of one pass
    constexpr int kPass = kBN / kRows;
    static_assert(kRows % 8 == 0, "swizzle");
    const int ct = tid - kConvWarp * 32;
    const int l = ct % kLanes, r0 = ct / kLanes;
    const int odd = l >> 2, c0 = (2 * l) & 7;
    const uint32_t row = (l / 4) * L::kSub + r0 * 128;
    const uint32_t to_a = row + (((c0 + odd) ^ (r0 & 7)) << 4), to_b = row + (((c0 + 1 - odd) ^ (r0 & 7)) << 4);
    auto convert = [&](uint8_t* tile, int i, uint4 w) {
      const uint4 a = make_uint4(e4m3x2_to_f16x2(w.x), e4m3x2_to_f16x2(w.x >> 16), e4m3x2_to_f16x2(w.y),
                                 e4m3x2_to_f16x2(w.y >> 16));
      const uint4 b = make_uint4(e4m3x2_to_f16x2(w.z), e4m3x2_to_f16x2(w.z >> 16), e4m3x2_to_f16x2(w.w),
                                 e4m3x2_to_f16x2(w.w >> 16));
      *reinterpret_cast<uint4*>(tile + to_a + i * kRows * 128) = odd ? b : a;
      *reinterpret_cast<uint4*>(tile + to_b + i * kRows * 128) = odd ? a : b;
    };
    auto wait_slot = [&](int q) -> bool {
      return q < L::kVStages ||
             mbar_wait(bar(L::v_empty + q % L::kVStages), ((q / L::kVStages) - 1) & 1, &s_abort, prm.status);
    };
    uint4 buf[kPass];
    if constexpr (kOneSet) {
      for (int q = 0; q < ntiles; ++q) {
        const int st = q % L::kVStages, sc = q % L::kCStages;
        if (!mbar_wait(bar(L::c_full + sc), (q / L::kCStages) & 1, &s_abort, prm.status)) break;
        const uint4* codes = reinterpret_cast<const uint4*>(gbase + L::kC + sc * L::kKTile) + ct;
#pragma unroll
        for (int i = 0; i < kPass; ++i) buf[i] = codes[i * kConvThreads];
        mbar_arrive(bar(L::c_empty + sc));
        if (!wait_slot(q)) break;
#pragma unroll
        for (int i = 0; i < kPass; ++i) convert(gbase + L::kV + st * L::kVTile, i, buf[i]);
        fence_proxy_async_smem();
        mbar_arrive(bar(L::v_full + st));
      }
    } else {
      // the codes of the next tile are loaded as those of this one leave the registers
      const int64_t step = static_cast<int64_t>(kRows) * p.H * D;
      const uint8_t* mine = prm.v8 + (static_cast<int64_t>(r0) * p.H + h) * D + l * 16;
      auto load = [&](const uint8_t* at, int q, int i) {
        // keys past N become zeros (their P' is 0)
        const bool in = static_cast<int64_t>(key_tile(q)) * kBN + i * kRows + r0 < p.N;
        buf[i] = in ? __ldg(reinterpret_cast<const uint4*>(at + i * step)) : make_uint4(0u, 0u, 0u, 0u);
      };
      const int64_t tile_bytes = static_cast<int64_t>(kBN) * p.H * D;
      if (ntiles > 0)
#pragma unroll
        for (int i = 0; i < kPass; ++i) load(mine + key_tile(0) * tile_bytes, 0, i);
      for (int q = 0; q < ntiles; ++q) {
        const int st = q % L::kVStages;
        if (!wait_slot(q)) break;
        const int qn = q + 1 < ntiles ? q + 1 : q;
        const uint8_t* next = mine + key_tile(qn) * tile_bytes;
#pragma unroll
        for (int i = 0; i < kPass; ++i) {
          const uint4 w = buf[i];
          load(next, qn, i);
          convert(gbase + L::kV + st * L::kVTile, i, w);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(L::v_full + st));
      }
    }
  };

  auto mma_role = [&](int me) {
    // ================================ MMA issuer =======================================
    // One thread issues the MMAs of both tiles, in turns, or (one set) each tile has its own. The tensor
    // pipe queues 8 MMAs, about 400 clocks of work, and a commit, a wait that finds its barrier ready and a
    // tcgen05 fence cost the issuer 50-200 clocks each, so a single one leaves the pipe waiting: two took 154 us
    // instead of 179 for one set of rows (a single one) over 118,800 keys, 24 heads, before such calls got a kernel
    // of their own. With shared key tiles two issuers lose: the
    // tiles fall into step and both softmaxes wait for MMAs at once (middle video 656 us instead of 622).
    // Descriptors are a base plus a constant in the 14-bit address field (shared memory ends
    // below 2^18 bytes: no carry).
    const int t_lo = kOneSet ? me : 0, t_hi = kOneSet ? me + 1 : kTiles;
    if (elect_one()) {
      constexpr uint32_t kIdescS = idesc_fmt0(kBM, kBN / 2, false, false);  // e4m3: Q (hi, lo) K^T, both K-major
      constexpr uint32_t kIdescO = idesc_fmt0(kBM, D, false, true);         // f16: P' V, V is MN-major
      auto base = [&](uint32_t a) { return D == 128 ? sdesc_sw128(a, 16, 1024) : sdesc_sw64(a, 16, 512); };
      const uint64_t dq = base(sbase + L::kQ), dk = base(sbase + L::kK);
      const uint64_t dv = sdesc_sw128(sbase + L::kV, L::kSub, 1024);
      auto issue_s = [&](int t, int u, int st) {
        const uint64_t da = kOneSet ? dq - (t == 1 ? shift * D >> 4 : 0) : dq + (t * 2 * L::kQPart >> 4);
        const uint64_t db = dk + ((st * L::kKTile + u * (L::kKTile / 2)) >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {     // hi parts, then lo parts, 32 channels each
          const int part = i / (D / 32), kk = i % (D / 32);
          mma_f8_ss(tS(t, u), da + ((part * L::kQPart + kk * 32) >> 4), db + (kk * 32 >> 4), kIdescS, i > 0 ? 1u : 0u);
        }
        mma_commit(bar(L::s_full + 2 * t + u));
        if (u == 1 && (kOneSet || t == kTiles - 1)) mma_commit(bar(L::k_empty + st));   // last reader
      };
      auto issue_o = [&](int t, int u, int st, bool first) {
        const uint64_t db = dv + ((st * L::kVTile + u * 64 * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < kBN / 32; ++kk)
          mma_f16_ts(tO(t), tS(t, u) + 8 * kk, db + (kk * 16 * 128 >> 4), kIdescO, (u > 0 || kk > 0 || !first) ? 1u : 0u);
        if (u == 1 && (kOneSet || t == kTiles - 1)) mma_commit(bar(L::v_empty + st));
      };
      auto wait_k = [&](int q) -> bool {
        return mbar_wait(bar(L::k_full + q % L::kKStages), (q / L::kKStages) & 1, &s_abort, prm.status);
      };
      auto wait_v = [&](int q) -> bool {
        return mbar_wait(bar(L::v_full + q % L::kVStages), (q / L::kVStages) & 1, &s_abort, prm.status);
      };
      bool ok = true;
      for (int t = t_lo; t < t_hi; ++t) {
        if (!ok || steps(t) == 0) continue;
        ok = mbar_wait(bar(L::q_full), 0, &s_abort, prm.status) && wait_k(seq(t, 0));
        tc_fence_after();
        if (!ok) continue;
        issue_s(t, 0, seq(t, 0) % L::kKStages);
        issue_s(t, 1, seq(t, 0) % L::kKStages);
      }
      // Step j: for each half O_t += P'_t V, and S_t of that half of the next key tile in its place (it overwrites
      // the columns P'_t was read from: MMAs of one thread run in issue order). While a softmax warp is at one
      // half, the MMAs of its other half run.
      const int n = steps(t_lo);
      for (int j = 0; ok && j < n; ++j) {
        const int q = seq(t_lo, j), qn = seq(t_lo, j + 1);
        const bool more = j + 1 < n;
        ok = wait_v(q) && (!more || wait_k(qn));
        const int sv = q % L::kVStages, sk = qn % L::kKStages;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          for (int t = t_lo; t < t_hi; ++t) {
            ok = ok && mbar_wait(bar(L::p_full + 2 * t + u), j & 1, &s_abort, prm.status);
            if (!ok) break;
            tc_fence_after();
            issue_o(t, u, sv, j == 0);
            if (more) issue_s(t, u, sk);
            else mma_commit(bar((u == 0 ? L::o_part : L::o_full) + t));
          }
        }
      }
      mma_commit(bar(L::drain));   // fires once every MMA issued above has completed
    }
    __syncwarp();
  };

  auto softmax_role = [&]() {
    // ================================ softmax warps ====================================
    const int t = warp >> 2;
    const int off_lane = t == 1 ? shift : 0;
    const int r = ((warp & 3) * 32 + lane - off_lane) & (kBM - 1);   // row of the tile, in TMEM lane r + off_lane
    const int lrow = (kOneSet ? 0 : t * kBM) + r;
    const bool valid = lrow < nrows;
    const int64_t row = row0 + lrow;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const bool works = has_rows(t, warp & 3);

    // ---- Q as hi + lo e4m3 codes: kLanesQ lanes per row, all softmax warps over all rows -------------------
    {
      constexpr int kLanesQ = D / 8;                            // 8 channels each
      constexpr int kRowsP = kSoftmaxThreads / kLanesQ;         // rows of a pass
      constexpr int kAhead = 4;                                 // passes whose loads are in flight
      const int lq = tid % kLanesQ;
      // the working warps' other lanes get zeros (warp 0 of a tile without rows included)
      const int need = kOneSet || nrows > kBM ? (nrows + 31) & ~31 : kBM + 32;
      for (int r0 = tid / kLanesQ; r0 < need; r0 += kAhead * kRowsP) {
        uint4 x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int r = r0 + i * kRowsP;
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (r < nrows) x[i] = *(reinterpret_cast<const uint4*>(p.q + ((row0 + r) * p.H + h) * D) + lq);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int r = r0 + i * kRowsP;
          float f[8] = {bf16lo(x[i].x), bf16hi(x[i].x), bf16lo(x[i].y), bf16hi(x[i].y),
                        bf16lo(x[i].z), bf16hi(x[i].z), bf16lo(x[i].w), bf16hi(x[i].w)};
          float top = 0.f;
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (fabsf(f[c]) < INFINITY) top = fmaxf(top, fabsf(f[c]));
#pragma unroll
          for (int o = kLanesQ / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float sc = scale_of_row(top);
          const float inv = 1.f / sc;
          uint32_t hi[2], lo[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float* g = f + 4 * k;
#pragma unroll
            for (int c = 0; c < 4; ++c) g[c] = fabsf(g[c]) < INFINITY ? g[c] * inv : NAN;   // an infinite logit: NaN
            hi[k] = pack_e4m3x4(g[0], g[1], g[2], g[3]);
            const float2 a = f16x2_to_f2(e4m3x2_to_f16x2(hi[k])), b = f16x2_to_f2(e4m3x2_to_f16x2(hi[k] >> 16));
            lo[k] = pack_e4m3x4(g[0] - a.x, g[1] - a.y, g[2] - b.x, g[3] - b.y);
          }
          if (r < need) {
            const int rt = r & (kBM - 1), c = lq >> 1;          // row of its tile, 16-byte chunk
            uint8_t* to = gbase + L::kQ + (r / kBM) * 2 * L::kQPart + 8 * (lq & 1) +
                          (D == 128 ? rt * 128 + ((c ^ (rt & 7)) << 4) : rt * 64 + ((c ^ ((rt >> 1) & 3)) << 4));
            *reinterpret_cast<uint2*>(to) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2*>(to + L::kQPart) = make_uint2(lo[0], lo[1]);
            if (lq == 0) s_rowc[r] = prm.scale_log2 * sc;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(L::q_full));
      barrier_softmax();                                        // s_rowc
    }
    const float rowc = works ? s_rowc[lrow] : 1.f;
    float m_run = -INFINITY, s_run = -INFINITY, l_run = 0.f;   // references of P' and O, and of the sum
    float l_low = 0.f;                            // what l_run's additions rounded off
    bool ok = true;
    const int nsteps = steps(t);
    auto scales = [&](int j, float& ks, float& vs) {
      const int64_t at = static_cast<int64_t>(key_tile(seq(t, j))) * p.H + h;
      ks = __ldg(prm.ks + at);
      vs = __ldg(prm.vs + at);
    };
    float ks_next = 0.f, vs_next = 0.f;
    if (works && nsteps > 0) scales(0, ks_next, vs_next);
    for (int j = 0; works && j < nsteps; ++j) {
      const float c = fmaxf(rowc * ks_next, kFactorMin);
      const float lv = log2_scale(vs_next);
      float share = share_of(m_run, lv, s_run);
      if (j + 1 < nsteps) scales(j + 1, ks_next, vs_next);
      const int64_t key0 = static_cast<int64_t>(key_tile(seq(t, j))) * kBN;
      const int nvalid = static_cast<int>(p.N - key0 < kBN ? p.N - key0 : kBN);
      // The tile goes in two halves of 64 keys, each with its own S: the MMAs of one half run while the
      // exponentials of the other are taken.
      const uint64_t c2 = f2_pack(c, c);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        // every wait result is made warp-uniform: tcgen05.ld/st are .sync.aligned
        if (!__all_sync(0xffffffffu, mbar_wait(bar(L::s_full + 2 * t + u), j & 1, &s_abort, prm.status))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t at = tS(t, u) + lane_off;
        uint32_t pk[32];
        uint64_t acc[2] = {f2_pack(0.f, 0.f), f2_pack(0.f, 0.f)};
        auto sum = [&]() -> float {
          float x0, x1, x2, x3;
          f2_unpack(acc[0], x0, x1);
          f2_unpack(acc[1], x2, x3);
          return (x0 + x1) + (x2 + x3);
        };
        // Fast path: keep the running reference. Softmax is exact for any reference; the half's sum bounds
        // every P', so P' stays finite in f16 while the sum is at most kSumLimit. S passes through the
        // registers 32 columns at a time, the next 32 on their way meanwhile: no branch may come between the
        // two ends of such a load, since the compiler may move registers there that are still to be written.
        float lt = 0.f;
        bool slow = (j == 0 && u == 0) || nvalid < kBN;
        if (!slow) {
          const uint64_t nb2 = f2_pack(lv - m_run, lv - m_run);
          uint32_t s0[32], s1[32];
          tmem_ld32_begin(at, s0);
          tmem_ld32_end(s0);
          tmem_ld32_begin(at + 32, s1);
          exp_cols_f16(s0, c2, nb2, pk, acc);
          tmem_ld32_end(s1);
          exp_cols_f16(s1, c2, nb2, pk + 16, acc);
          lt = sum();
          slow = __any_sync(0xffffffffu, !(lt <= kSumLimit && share <= kShareMax));
        }
        if (slow) {                                 // S is intact: P' of this half has not been stored yet
          uint32_t sr[64];
          tmem_ld64(at, sr);
          if (nvalid < kBN) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (64 * u + i >= nvalid) sr[i] = __float_as_uint(-INFINITY);
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int i = 0; i < 64; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(sr[i]));
          // a tile's first half has a key below N, so the first maximum is finite (or S is NaN, and so is
          // the row); m stays -inf until a key has a value
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
          const float m_new = fmaxf(m_run, top + (lv - raise_of(ntiles)));
          const float s_new = fmaxf(s_run, top);
          const float beta = fast_exp2(s_run - s_new);
          l_run *= beta;
          l_low *= beta;
          s_run = s_new;
          if (j == 0 && u == 0) {
            m_run = m_new;
          } else if (__any_sync(0xffffffffu, m_new > m_run)) {
            // O, complete up to the half before, is rescaled. The MMAs of that half are followed by those of the
            // next S in its columns (or, in the last step, by a commit of their own).
            const float alpha = fast_exp2(m_run - m_new);
            const bool last = u == 1 && j + 1 == nsteps;
            const uint32_t before = last ? bar(L::o_part + t) : bar(L::s_full + 2 * t + 1 - u);
            if (!__all_sync(0xffffffffu, mbar_wait(before, last ? 0 : (j + u) & 1, &s_abort, prm.status))) ok = false;
            tc_fence_after();
#pragma unroll
            for (int i0 = 0; i0 < D; i0 += 16) {    // few registers: sr is held meanwhile
              float o[16];
              tmem_ld16(tO(t) + lane_off + i0, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= alpha;
              tmem_st16(tO(t) + lane_off + i0, o);
            }
            m_run = m_new;
          }
          uint32_t(&lo)[32] = *reinterpret_cast<uint32_t(*)[32]>(sr);
          uint32_t(&hi)[32] = *reinterpret_cast<uint32_t(*)[32]>(sr + 32);
          auto exponentials = [&](float base) {
            const uint64_t nb2 = f2_pack(base, base);
            acc[0] = acc[1] = f2_pack(0.f, 0.f);
            exp_cols_f16(lo, c2, nb2, pk, acc);
            exp_cols_f16(hi, c2, nb2, pk + 16, acc);
            lt = sum();
          };
          share = share_of(m_run, lv, s_run);
          const bool alone = __any_sync(0xffffffffu, !(share <= kShareMax));
          if (alone) {
            exponentials(-s_run);
            add_low(l_low + lt, l_run, l_low);
          }
          if (lv == -INFINITY) {
#pragma unroll
            for (int i = 0; i < 32; ++i) pk[i] = 0u;
          } else {
            exponentials(lv - m_run);
          }
          if (!alone) add_low(fmaf(lt, share, l_low), l_run, l_low);
        } else {
          add_low(fmaf(lt, share, l_low), l_run, l_low);
        }
        tmem_st32_words(at, pk);                    // P' over S columns that have been read
        tc_fence_before();
        mbar_arrive(bar(L::p_full + 2 * t + u));
      }
      if (!ok) break;
    }
    // ---- epilogue ------------------------------------------------------------------------
    if (ok && nsteps > 0) ok = mbar_wait(bar(L::o_full + t), 0, &s_abort, prm.status);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    float w1 = 0.f;
    constexpr int kMine = kOneSet ? D / 2 : D;    // columns of the output that this thread writes, from c0
    const int c0 = kOneSet ? t * kMine : 0;
    const float* other = nullptr;
    if constexpr (kOneSet) {
      // Each tile stages the half of its row that the other will write over the rings (free once both tiles' last
      // products are complete), chunks rotated by row so the 16-byte accesses of a warp hit distinct banks.
      // With shifted lanes the two threads of a row sit in different warps: both have r.
      float4* stage = reinterpret_cast<float4*>(gbase + L::kV);
      float4* s_msl = reinterpret_cast<float4*>(gbase + L::kList);   // [tile][row]; the list is done with
      barrier_softmax();
      s_msl[t * kBM + r] = make_float4(m_run, s_run, l_run, 0.f);
      if (ok && works && nsteps > 0) {
#pragma unroll
        for (int i0 = 0; i0 < kMine; i0 += 32) {
          float o[32];
          tmem_ld32(tO(t) + lane_off + (1 - t) * kMine + i0, o);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            stage[(t * kBM + r) * kChunks + (i0 / 4 + q + r) % kChunks] =
                make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
        }
      }
      barrier_softmax();
      ok = __all_sync(0xffffffffu, ok && !s_abort);
      const float4 msl = s_msl[(1 - t) * kBM + r];
      const float s = fmaxf(s_run, msl.y);
      l_run = part_weight(s_run, l_run, s) * l_run + part_weight(msl.y, msl.z, s) * msl.z;
      s_run = s;
      w1 = value_weight(msl.x, s);
      other = reinterpret_cast<const float*>(stage + (1 - t) * kBM * kChunks);
    }
    if (!ok || !works) return;
    // a row with no key has l = 0: o = 0, lse = -inf; a NaN sum stays NaN
    const float inv = l_run == 0.f ? 0.f : 1.f / l_run;
    const float w0 = value_weight(m_run, s_run) * inv;   // weights of this tile's and the other tile's O
    w1 *= inv;
    const float lse = l_run == 0.f ? -INFINITY : (s_run + log2f(l_run)) * kLn2;
    const int64_t orow = row * p.H + h;
    const int64_t prow = prm.nsplit > 1 ? static_cast<int64_t>(blockIdx.z) * prm.part_rows * p.H + orow - prm.part_row0 * p.H : 0;
#pragma unroll
    for (int i0 = 0; i0 < kMine; i0 += 32) {
      float o[32];
      __syncwarp();
      if (nsteps > 0) tmem_ld32(tO(t) + lane_off + c0 + i0, o);
#pragma unroll
      for (int i = 0; i < 32; ++i) o[i] = nsteps > 0 ? o[i] * w0 : 0.f;   // (a weight of 0 keeps a NaN of V)
      if constexpr (kOneSet) {
        if (ntiles > 1 - t) {                     // the other tile has steps
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            const float4 x = reinterpret_cast<const float4*>(other)[r * kChunks + (i0 / 4 + q + r) % kChunks];
            o[4 * q] = fmaf(w1, x.x, o[4 * q]);
            o[4 * q + 1] = fmaf(w1, x.y, o[4 * q + 1]);
            o[4 * q + 2] = fmaf(w1, x.z, o[4 * q + 2]);
            o[4 * q + 3] = fmaf(w1, x.w, o[4 * q + 3]);
          }
        }
      }
      if (valid && prm.nsplit > 1) {
        float4* dst = reinterpret_cast<float4*>(prm.o_part + prow * D + c0 + i0);
#pragma unroll
        for (int q = 0; q < 8; ++q) dst[q] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      } else if (valid) {
        uint4* dst = reinterpret_cast<uint4*>(p.o + orow * D + c0 + i0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
          dst[q] = make_uint4(pack_bf16x2(o[8 * q], o[8 * q + 1]), pack_bf16x2(o[8 * q + 2], o[8 * q + 3]),
                              pack_bf16x2(o[8 * q + 4], o[8 * q + 5]), pack_bf16x2(o[8 * q + 6], o[8 * q + 7]));
      }
    }
    if (valid && (!kOneSet || t == 0)) {
      if (prm.nsplit > 1) prm.lse_part[prow] = lse;
      else if (p.lse) p.lse[orow] = lse;
    }
  };

  // teardown; each role runs its own copy (ptxas allots a region the registers of its setmaxnreg only
  // if the region does not rejoin the other warps' code)
  auto tail = [&]() {
    if (warp == kMmaWarp) drain_wait(bar(L::drain), 0);   // no MMA may still write TMEM
    tc_fence_before();
    barrier_all();
    tc_fence_after();
    if (warp == kMmaWarp) {
      __syncwarp();
      tmem_dealloc<kTmemCols>(tmem);
    }
  };
  if (warp >= kTmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    if (warp == kTmaWarp) tma_role();
    else if (warp >= kMmaWarp && warp < kMmaWarp + kIssuers) mma_role(warp - kMmaWarp);
    tail();
  } else if (warp >= kConvWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kConvRegs));
    conv_role();
    tail();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    softmax_role();
    tail();
  }
}

// ---- host ------------------------------------------------------------------------------------
// [N, H, d] e4m3 codes -> 3-D map (d, H, N), box (d, 1, 128): one row per key (K: one swizzle row).
int make_map(EncodeTiledFn enc, CUtensorMap* m, const void* base, int64_t N, int H, int d, CUtensorMapSwizzle swizzle) {
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(N)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(H) * d};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(d), 1, kBN};
  cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(TPS_ERR_CUDA, "pruned_attn_q8: cuTensorMapEncodeTiled failed (%d)", static_cast<int>(r));
  return TPS_OK;
}

// How a call runs. A unit of work is one row tile (256 rows, or one set of 128) of one head; U units on P SMs
// take ceil(U / P) unit times. Two ways out of a mostly empty last wave: all units split S ways along the
// keys, or the units of the full waves whole and the remaining tiles split S_t ways in a second launch.
// Costs in steps of key tiles (of a pair of them in the one-set layout; 1.7 us each): a CTA of n steps takes
// n + kEnds (prologue and epilogue), a split adds the merge. A plan must gain 2% on the one before it. Ranges of
// down to two key tiles pay: 64 rows x 4,096 keys, 12 heads, took 16.3 us in 4 ranges of 8 tiles and take 13.5 in 8 of 4;
// 67 x 11,501, 5 heads x 64: 18.1 us in 11, 13.9 in 23 (steps counted whole: 15.2 in 22). A second wave does not:
// 128 x 32,760, 5 heads: 20.6 us in 29 ranges, 32.3 in 32.
// Masked calls are one CTA per query block and head.
struct Plan {
  bool few;             // the kernel of attn_q8_few.cu
  bool one_set;
  int split;            // of the launch that has all tiles (main_tiles = 0), or of the tail
  int64_t main_tiles;   // tiles of an unsplit first launch; 0: none
};
constexpr double kEnds = 6.0, kMerge = 1.5, kPart = 0.06;
constexpr int kMaxSplit = 64;

Plan make_plan(int64_t cap, int64_t N, int H, bool masked) {
  Plan best{!masked && cap <= kFewRows, masked || cap <= kBM, 1, 0};
  if (masked || cap < 1) return best;
  if (best.few) {
    best.split = few_split(cap, N, H);
    return best;
  }
  const int64_t tiles = best.one_set ? 1 : (cap + kTiles * kBM - 1) / (kTiles * kBM);
  const int64_t units = tiles * H;
  const int64_t nkt = (N + kBN - 1) / kBN;
  const int64_t P = sm_count();
  auto cost_of = [&](int64_t u, int s) {
    const int64_t own = (nkt + s - 1) / s, steps = best.one_set ? (own + 1) / 2 : own;
    return static_cast<double>((u * s + P - 1) / P) * (steps + kEnds) + (s > 1 ? kMerge + kPart * s : 0.0);
  };
  double cost = 1e300;
  for (int s = 1; s <= kMaxSplit && (s == 1 || nkt >= 2 * s); ++s)
    if (const double c = cost_of(units, s); c < 0.98 * cost) {
      cost = c;
      best.split = s;
    }
  const int64_t whole = units / P * P / H;          // tiles that fit the full waves
  if (whole >= 1 && whole < tiles)
    for (int s = 2; s <= kMaxSplit && nkt >= 2 * s; ++s)
      if (const double c = cost_of(whole * H, 1) + cost_of((tiles - whole) * H, s); c < 0.98 * cost) {
        cost = c;
        best.split = s;
        best.main_tiles = whole;
      }
  return best;
}

int64_t part_rows_of(const Plan& plan, int64_t cap) { return cap - plan.main_tiles * (kTiles * kBM); }

size_t ws_bytes_of(const Plan& plan, int64_t cap, int H, int d) {
  if (plan.split <= 1) return 0;
  const size_t rows = static_cast<size_t>(plan.split) * part_rows_of(plan, cap) * H;
  return (rows * d * sizeof(float) + 255) / 256 * 256 + rows * sizeof(float);
}

// The S-way merge of the partials: o = sum_s w_s o_s / sum_s w_s with w_s = exp(lse_s - max). Latency is all it
// costs, so a thread (4 channels of a row) loads values and statistics of 8 parts at a time, guarded rather than
// in a remainder loop, against a running maximum. A weight enters as its root, twice: below 2^-126 it can still count,
// where the part's values are as much larger than the others'.
template <int D>
__global__ void __launch_bounds__(128) merge_kernel(const __grid_constant__ Q8Args prm) {
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched ahead of the partials' end
  const AttnArgs& p = prm.a;
  const int64_t rows = active_count(p.count, p.cap) - prm.part_row0;
  const int64_t plane = prm.part_rows * p.H;
  const int64_t total = rows * p.H * (D / 4);
  constexpr int kParts = 8;                            // loads in flight
  const float4* op = reinterpret_cast<const float4*>(prm.o_part);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t rh = i / (D / 4);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, ref = 0.f, sum = 0.f;
    for (int s0 = 0; s0 < prm.nsplit; s0 += kParts) {
      float4 x[kParts];
      float l[kParts];
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const bool in = s0 + u < prm.nsplit;
        x[u] = in ? op[(s0 + u) * plane * (D / 4) + i] : make_float4(0.f, 0.f, 0.f, 0.f);
        l[u] = in ? prm.lse_part[(s0 + u) * plane + rh] : -INFINITY;   // (a part without a key: zeros and -inf)
      }
      const float was = m;
#pragma unroll
      for (int u = 0; u < kParts; ++u) m = fmaxf(m, l[u]);              // NaN is passed over here, not by w
      ref = m == -INFINITY ? 0.f : m;
      const float f = expf(0.5f * (was - ref));
      a = make_float4(a.x * f * f, a.y * f * f, a.z * f * f, a.w * f * f);
      sum *= f * f;
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const float w = expf(0.5f * (l[u] - ref));
        a.x = fmaf(w, w * x[u].x, a.x);
        a.y = fmaf(w, w * x[u].y, a.y);
        a.z = fmaf(w, w * x[u].z, a.z);
        a.w = fmaf(w, w * x[u].w, a.w);
        sum = fmaf(w, w, sum);
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int64_t orow = prm.part_row0 * p.H + rh;
    reinterpret_cast<uint2*>(p.o + orow * D)[i % (D / 4)] =
        make_uint2(pack_bf16x2(a.x * inv, a.y * inv), pack_bf16x2(a.z * inv, a.w * inv));
    if (p.lse && i % (D / 4) == 0) p.lse[orow] = sum == 0.f ? -INFINITY : ref + logf(sum);
  }
}

int launch_merge(const Q8Args& prm, cudaStream_t st) {
  const int64_t threads = prm.part_rows * prm.a.H * (prm.a.d / 4);
  int64_t grid = (threads + 127) / 128;
  const int64_t most = static_cast<int64_t>(sm_count()) * 16;
  grid = grid < most ? grid : most;
  // the launch itself overlaps the kernels of the partials; the merge kernel waits for their end
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(128);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = prm.a.d == 128 ? cudaLaunchKernelEx(&cfg, merge_kernel<128>, prm)
                                       : cudaLaunchKernelEx(&cfg, merge_kernel<64>, prm);
  if (e != cudaSuccess) return cuda_status(e, "pruned_attn_q8: merge launch");
  return launch_status("pruned_attn_q8: merge");
}

template <int D, bool kOneSet>
int launch(const CUtensorMap& mk, const CUtensorMap& mv, const Q8Args& prm, int64_t tiles, cudaStream_t st) {
  constexpr int kSmem = Layout<D, kOneSet>::kAlloc;
  if (int e = smem_attribute<attn_q8_kernel<D, kOneSet>>(kSmem, "pruned_attn_q8")) return e;
  const dim3 grid(static_cast<unsigned>(tiles), static_cast<unsigned>(prm.a.H), static_cast<unsigned>(prm.nsplit));
  attn_q8_kernel<D, kOneSet><<<grid, kThreads, kSmem, st>>>(mk, mv, prm);
  return launch_status("pruned_attn_q8");
}

}  // namespace

}  // namespace tps

extern "C" size_t tps_attn_q8_workspace_size(int64_t cap, int64_t N, int H, int d) {
  using namespace tps;
  if (cap <= 0 || cap >= (INT64_C(1) << 31) || N <= 0 || N >= (INT64_C(1) << 31) || H <= 0 || H > 256 ||
      (d != 64 && d != 128))
    return 0;
  return ws_bytes_of(make_plan(cap, N, H, false), cap, H, d);
}

extern "C" int pruned_attn_q8(const tps_bf16* q_act, const uint8_t* k_cache, const uint8_t* v_cache,
                              const float* k_scale, const float* v_scale, const int32_t* idx, const int32_t* count,
                              int64_t cap, int64_t N, int H, int d, float scale, const uint8_t* blockmask, int block,
                              tps_bf16* o_act, float* lse, void* ws, size_t ws_bytes, tps_stream stream) {
  TPS_TRACE("pruned_attn_q8");
  using namespace tps;
  Q8Args prm{};
  if (int e = attn_validate("pruned_attn_q8", q_act, reinterpret_cast<const tps_bf16*>(k_cache),
                            reinterpret_cast<const tps_bf16*>(v_cache), idx, count, cap, N, H, d, scale, blockmask,
                            block, o_act, lse, &prm.a))
    return e;
  if (!k_scale || !v_scale) return fail(TPS_ERR_INVALID_ARG, "pruned_attn_q8: null scales");
  if ((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) | reinterpret_cast<uintptr_t>(lse)) & 3u)
    return fail(TPS_ERR_ALIGN, "pruned_attn_q8: scales and lse must be 4-byte aligned");
  if (cap == 0) return ok();
  Plan plan = make_plan(cap, N, H, blockmask != nullptr);
  if (!ws || !aligned16(ws) || ws_bytes < ws_bytes_of(plan, cap, H, d)) {
    plan.split = 1;
    plan.main_tiles = 0;
  }
  int err;
  prm.status = device_status(&err);
  if (!prm.status) return err;
  prm.v8 = v_cache;
  prm.ks = k_scale;
  prm.vs = v_scale;
  prm.scale_log2 = scale * kLog2e;
  prm.nsplit = plan.split;
  if (plan.split > 1) {
    prm.part_row0 = plan.main_tiles * (kTiles * kBM);
    prm.part_rows = part_rows_of(plan, cap);
    prm.o_part = static_cast<float*>(ws);
    prm.lse_part = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                            (static_cast<size_t>(plan.split) * prm.part_rows * H * d * sizeof(float) + 255) / 256 * 256);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int e;
  if (plan.few) {
    e = launch_attn_q8_few(prm, st);
  } else {
    EncodeTiledFn enc;
    if (int r = tensor_map_encoder(&enc, "pruned_attn_q8")) return r;
    CUtensorMap mk, mv;
    if (int r = make_map(enc, &mk, k_cache, N, H, d, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return r;
    if (int r = make_map(enc, &mv, v_cache, N, H, d, CU_TENSOR_MAP_SWIZZLE_NONE)) return r;
    if (plan.one_set) {
      const int64_t tiles = blockmask ? prm.a.nb : 1;
      e = d == 64 ? launch<64, true>(mk, mv, prm, tiles, st) : launch<128, true>(mk, mv, prm, tiles, st);
    } else {
      const int64_t tiles = (cap + kTiles * kBM - 1) / (kTiles * kBM);
      auto run = [&](const Q8Args& a, int64_t n) {
        return d == 64 ? launch<64, false>(mk, mv, a, n, st) : launch<128, false>(mk, mv, a, n, st);
      };
      e = TPS_OK;
      if (plan.main_tiles) {
        Q8Args whole = prm;
        whole.nsplit = 1;
        e = run(whole, plan.main_tiles);
        prm.tile0 = static_cast<int>(plan.main_tiles);
      }
      if (!e) e = run(prm, tiles - plan.main_tiles);
    }
  }
  if (!e && plan.split > 1) e = launch_merge(prm, st);
  return e ? e : ok();
}
