// Attention over an 8-bit cache for many query rows: the tensor-core kernel.
//
// One CTA = (KV split, head, group of query rows): up to two 128-row main tiles and, on the last
// group, a tail of at most 8 rows, as in the bf16 kernel (spk_attn_tc.cu).  Keys are processed in
// units of 64 (the planner's chunks).
//
// Operands.  The codes are widened to fp16 in shared memory once per CTA and unit, with their
// scales: K' = c 2^(b - RK), V' = c 2^(b - RV), RK and RV the largest scale bytes of the split, so
// that |K'|, |V'| <= 448 (exact down to 2^-15 of the largest scale, below that rounded by up to 2^-25;
// fp16 because 8-bit weights would cost the output four bits and bf16 three).  Q' = q 2^(127 - e) with
// the row's largest value in [1, 2).  Scores are x = rf (Q' K') in log2 units, rf = log2(e) / sqrt(D)
// 2^(e - 127) 2^(RK - 127) one factor per row; P' = 2^(x - m + 8) in fp16 with m a running maximum that
// moves only when 32 P' sum to 2^14 (a score 6 above m at the latest).  The row's largest P' is thus at
// least 2^7; a P' is rounded by 2^-11 of itself down to 2^-14, below that by up to 2^-25: 2^-32 of the
// row's largest weight.  Row sums are taken from the fp32 weights.
//
// Warps:
//   0-3    widen the units;
//   4-7    the tail;
//   8-     softmax of the main tiles, one thread per row (= TMEM lane). head_dim 64: 16 warps, four
//          each for the even and the odd units of tile 0 and of tile 1.  The two warps of a tile and
//          SM sub-partition take turns, so one loads scores, stores P and waits while the other
//          exponentiates.  They share m through shared memory: before a unit's warps publish their P they
//          wait until the unit before has published its own (the barrier that tells the issuer so) and
//          correct what they hold if it moved m; a unit that moves m rescales O after every earlier
//          product has completed.  So P, O and the sums always refer to one m.  head_dim 128 (twice the
//          products per score): 8 warps, four per tile.
//   then   a TMA producer (codes of a unit by the cache's tensor map, its 2 x 64 scale bytes by bulk
//          copies, into a ring of raw units) and an MMA issuer per main tile.
//
// Score buffers of 64 columns, three per tile (head_dim 128: two), P over the scores: the product of unit
// g + 3 (g + 2) goes into the buffer that P V of unit g has just read, so a warpgroup finds its next scores
// nearly done when it has published a P.
// TMEM, D = 64: S 2 x 3 x 64 | O 2 x 64; D = 128: S 2 x 2 x 64 | O 2 x 128: all 512 columns.
//
// The tail (at most 8 rows) needs no TMEM: four warps, two for the even and two for the odd units, 32 keys
// each, as fp16 warp products with the widened tiles (ldmatrix; keys and dims in the products' M, the rows
// in N), each a running softmax of its own; they are joined at the end.
//
// A unit's slot is free once every consumer's P V of it has completed (slot_free, which the rare
// path that moves m waits on too).  Every wait is bounded, as in the bf16 kernel.
//
// Measured with the merge: 78,432 keys of 16 heads of 64 dims, 262 rows 113 to 118 us (747 to 715
// TFLOP/s; 107 where scores spread so little that m hardly moves); 51,960 keys, 1005 rows 271 to 278 us
// (790 to 770; 261); 4 x 63,792 keys of 8 heads of 128 dims, 262 rows 272 to 276 us (1,005 to 990; 270).
// DRAM is at 6 to 27 %, the tensor pipe at 38 to 53 %.  A unit of 64 dims takes some 1,350 cycles:
// 520 of products, 720 of exponentials and packing at the rate of four warps by themselves, 66 % of the
// issue slots; the softmax warps and the widening warps are both busy all the time, a third of it with
// the latency of waits, TMEM loads and hand-overs.  Four softmax warps a sub-partition hide that better
// than two with twice the registers (1005 rows 291 and 331 us).
#include "ptx_sm100.cuh"
#include "spk_e4m3.cuh"
#include "spk_internal.h"

#include <cuda_bf16.h>

#include <atomic>

namespace spk {
namespace {

constexpr int kUnit = kUnitTokens;         // keys of a unit
constexpr int kWarpTail = 4;
constexpr int kWarpMain = 8;
constexpr int kBias = 8;                   // P' = 2^(x - m + kBias)
// Tail: a score may pass m by this much before m moves.
constexpr float kHeadroom = 6.f;
// Main tiles: m moves when the sum of 32 P' reaches this, so no P' does.  With every score at most m the
// sum is at most 2^13.  The sum is taken anyway; a maximum took a twelfth of the instructions.
constexpr float kSumLimit = 16384.f;

template <int D>
struct Cfg {
  // Score buffers per tile, P over the scores, each with its p_ready: P of unit g + kBuffers needs P V of
  // unit g, so a barrier is never two phases ahead of who waits for it (a wait only tells a phase
  // from the one before it).
  static constexpr int kBuffers = D == 64 ? 3 : 2;
  static constexpr int kPar = D == 64 ? 2 : 1;        // softmax warpgroups per main tile
  static constexpr int kWarpTma = kWarpMain + 8 * kPar;
  static constexpr int kWarpMma = kWarpTma + 1;
  static constexpr int kThreads = 32 * (kWarpMma + 2);
  // registers a thread (7 or 5 warps on an SM sub-partition; D = 64 spills 4 bytes)
  static constexpr int kRegs = D == 64 ? 72 : 96;
  static constexpr int kTile = kUnit * D * 2;         // one widened K' or V' unit
  static constexpr int kBlock = kUnit * 128;          // its 64-column block (128-byte rows)
  static constexpr int kRawTile = kUnit * D;
  static constexpr int kSlots = 2 * kBuffers;         // widened units (twice: see the widening warps)
  static constexpr int kRaw = D == 64 ? 6 : 2;        // raw units
  // shared memory
  static constexpr int kQ = 0;                                      // two Q' tiles
  static constexpr int kK = 2 * 128 * D * 2;
  static constexpr int kV = kK + kSlots * kTile;
  static constexpr int kRawOff = kV + kSlots * kTile;               // K codes, V codes of each raw unit
  static constexpr int kScales = kRawOff + kRaw * 2 * kRawTile;     // [kRaw][K, V][64]
  // what a tile's two warpgroups share: running max [2][128], rf [2][128], row sums [2][2][128]
  static constexpr int kRowM = kScales + kRaw * 2 * kUnit;
  static constexpr int kRowF = kRowM + 1024;
  static constexpr int kRowL = kRowF + 1024;
  static constexpr int kBars = kPar == 2 ? kRowL + 2048 : kRowM;
  // raw_full, raw_empty [kRaw]; kv_full, slot_free [kSlots]; q_full, s_full [2][3], p_ready [2][3],
  // o_done [2]
  static constexpr int kNumBars = 2 * kRaw + 2 * kSlots + 15;
  static constexpr int kMisc = kBars + 8 * kNumBars;                // TMEM address, abort flag, RK, RV
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kLaunch = kBytes + 1024;
  // TMEM columns
  static constexpr uint32_t kO0 = 2 * kBuffers * kUnit;
  static_assert(kO0 + 2 * D <= 512, "TMEM budget");
  // the tail's join: fp32 O [4][8][D], m and l [4][8] over the raw ring
  static_assert(4 * 8 * (D + 2) * 4 <= kRaw * 2 * kRawTile, "join fits");
  static_assert(kK % 1024 == 0 && kV % 1024 == 0 && kRawOff % 1024 == 0, "swizzled tiles");
  static_assert(kLaunch <= 227 * 1024, "shared memory per CTA");
  // scores and P of unit g of tile t
  __device__ static uint32_t s_col(int t, int g) { return uint32_t(kUnit * (kBuffers * t + g % kBuffers)); }
};

__device__ __forceinline__ void signal_abort(int32_t* status, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicExch(status, kStatusWaitTimeout);
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ int lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return int(v);
}

// 2^d as a pair of fp16 values, d <= 0 (0 below fp16's least value)
__device__ __forceinline__ uint32_t pow2_f16x2(int d) {
  const float f = __uint_as_float(uint32_t(127 + max(d, -126)) << 23);
  return e4m3::pack_f16(f, f);
}

// Widen a raw unit (K and V, 64 rows of D codes, swizzled over D bytes) into fp16 rows (64-column
// blocks of 128-byte rows, 128-byte swizzle) with 128 threads.  A thread takes 16 codes of a row at
// a time, four loads ahead of their use; the pieces are dealt so that neither the reads nor the
// writes of eight threads meet in a bank.  Rows of V at or past `keys` become zero (whatever their
// slots hold).
template <int D>
__device__ __forceinline__ void widen_unit(uint32_t raw, uint32_t scales, uint32_t dst_k, uint32_t dst_v, int ref_k,
                                           int ref_v, int keys, int tid) {
  constexpr int kPasses = kUnit * (D / 16) / 128;     // pieces of a thread and tile: 2 or 4
  constexpr int kGroup = 2 * kPasses < 4 ? 2 * kPasses : 4;
#pragma unroll 1
  for (int i0 = 0; i0 < 2 * kPasses; i0 += kGroup) {
    uint4 v[kGroup];
    int b[kGroup];
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const int i = i0 + k, kv = i / kPasses, j = i % kPasses;
      const int r = (D == 64 ? j : j >> 1) * 32 + (tid >> 2);
      const int c = D == 64 ? tid & 3 : (tid & 3) + 4 * ((r ^ j) & 1);
      v[k] = lds128(raw + uint32_t(kv * Cfg<D>::kRawTile) +
                    uint32_t(D == 64 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4)));
      b[k] = lds_u8(scales + uint32_t(kv * kUnit + r));
    }
#pragma unroll
    for (int k = 0; k < kGroup; ++k) {
      const int i = i0 + k, kv = i / kPasses, j = i % kPasses;
      const int r = (D == 64 ? j : j >> 1) * 32 + (tid >> 2);
      const int c = D == 64 ? tid & 3 : (tid & 3) + 4 * ((r ^ j) & 1);
      const uint32_t f = pow2_f16x2(b[k] - (kv ? ref_v : ref_k));
      const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
      uint32_t h[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        h[2 * q] = ptx::mul_f16x2(e4m3::widen_lo(w[q]), f);
        h[2 * q + 1] = ptx::mul_f16x2(e4m3::widen_hi(w[q]), f);
      }
      if (kv && r >= keys) {
#pragma unroll
        for (int q = 0; q < 8; ++q) h[q] = 0;
      }
      const uint32_t row = (kv ? dst_v : dst_k) + uint32_t((c >> 2) * Cfg<D>::kBlock + r * 128);
      const int p = 2 * (c & 3);
      sts128(row + uint32_t((p ^ (r & 7)) << 4), h[0], h[1], h[2], h[3]);
      sts128(row + uint32_t(((p + 1) ^ (r & 7)) << 4), h[4], h[5], h[6], h[7]);
    }
  }
}

// A query row as fp16, scaled by 2^(127 - e) with e the exponent of its largest value; returns
// log2(e)/sqrt(D) 2^(e - 127).
template <int D>
__device__ __forceinline__ float row_exponent(const uint4* src, bool valid, float sl2, float* scale) {
  uint32_t amax = 0;
  if (valid) {
#pragma unroll 4
    for (int c = 0; c < D / 8; ++c) {
      const uint4 v = __ldg(src + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) amax = max(amax, max((w[j] << 16) & 0x7FFFFFFFu, w[j] & 0x7FFF0000u));
    }
  }
  const uint32_t e = min(max(amax >> 23, 1u), 253u);
  *scale = __uint_as_float((254u - e) << 23);
  return sl2 * __uint_as_float(e << 23);
}
__device__ __forceinline__ uint32_t to_f16x2(uint32_t bf16x2, float scale) {
  return e4m3::pack_f16(__uint_as_float(bf16x2 << 16) * scale, __uint_as_float(bf16x2 & 0xFFFF0000u) * scale);
}

// The scores of the keys past a ragged unit's last one become -inf where they lie: the code that
// every unit passes through then needs no mask (nor the moves that a conditional one leaves).
__device__ __noinline__ void mask_scores(uint32_t tS, int keys) {
#pragma unroll 1
  for (int c = keys; c < kUnit; ++c)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(tS + uint32_t(c)), "r"(0xFF800000u) : "memory");
  ptx::tmem_wait_st();
}

__device__ __forceinline__ float max32(const uint32_t (&s)[32], float mx) {
  float a = mx, b = -INFINITY;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    a = ptx::max3(a, __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
    b = ptx::max3(b, __uint_as_float(s[e + 2]), __uint_as_float(s[e + 3]));
  }
  return fmaxf(a, b);
}

// Scores to words of two P' = 2^(rf s + c); sums in (h0, h1)
template <int kScores>
__device__ __forceinline__ void exps(const uint32_t (&s)[kScores], float rf, float c, uint32_t* pk, float& h0, float& h1) {
#pragma unroll
  for (int e = 0; e < kScores / 2; ++e) {
    float x0, x1;
    ptx::fma2(x0, x1, __uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1]), rf, c);
    x0 = ptx::ex2(x0);
    x1 = ptx::ex2(x1);
    ptx::add2(h0, h1, x0, x1);
    pk[e] = e4m3::pack_f16(x0, x1);
  }
}

__device__ __forceinline__ void rescale_o(uint32_t tO, int cols, float corr) {
#pragma unroll 1
  for (int j = 0; j < cols; j += 32) {
    uint32_t o[32];
    ptx::tmem_ld32(tO + j, o);
    ptx::tmem_wait_ld();
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
    ptx::tmem_st32(tO + j, o);
    ptx::tmem_wait_st();
  }
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void tail_bar_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }
// every warp but the producer
template <int kThreads>
__device__ __forceinline__ void workers_sync() {
  asm volatile("bar.sync 2, %0;" ::"n"(kThreads - 32) : "memory");
}
// the 256 softmax threads of a tile (head_dim 64)
__device__ __forceinline__ void tile_sync(int t) {
  if (t == 0) asm volatile("bar.sync 3, 256;" ::: "memory");
  else asm volatile("bar.sync 4, 256;" ::: "memory");
}

__device__ __forceinline__ uint32_t byte_max(uint32_t v) {
  v = __vmaxu4(v, v >> 16);
  return max(v & 255u, (v >> 8) & 255u);
}

template <int D, bool kPlanRegs>
__global__ void __launch_bounds__(Cfg<D>::kThreads, 1)
    attention_e4m3_tc_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kv_map) {
  using C = Cfg<D>;
  constexpr int S = C::kSlots, SR = C::kRaw;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  auto sK = [&](int s) { return sbase + uint32_t(C::kK + s * C::kTile); };
  auto sV = [&](int s) { return sbase + uint32_t(C::kV + s * C::kTile); };
  auto sRaw = [&](int s) { return sbase + uint32_t(C::kRawOff + s * 2 * C::kRawTile); };
  auto sScale = [&](int s) { return sbase + uint32_t(C::kScales + s * 2 * kUnit); };
  const uint32_t bars = sbase + C::kBars;
  auto raw_full = [&](int s) { return bars + 8 * s; };
  auto raw_empty = [&](int s) { return bars + 8 * (SR + s); };
  auto kv_full = [&](int s) { return bars + 8 * (2 * SR + s); };
  auto slot_free = [&](int s) { return bars + 8 * (2 * SR + S + s); };
  const uint32_t q_full = bars + 8 * (2 * SR + 2 * S);
  auto s_full = [&](int t, int b) { return q_full + 8 * (1 + 3 * t + b); };
  auto p_ready = [&](int t, int g) { return q_full + 8 * (7 + 3 * t + g % C::kBuffers); };  // of unit g, with its phase
  auto p_phase = [&](int g) { return uint32_t(g / C::kBuffers) & 1u; };
  auto o_done = [&](int t) { return q_full + 8 * (13 + t); };
  float* row_m = reinterpret_cast<float*>(smem + C::kRowM);
  float* row_f = reinterpret_cast<float*>(smem + C::kRowF);
  float* row_l = reinterpret_cast<float*>(smem + C::kRowL);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  int* refs = reinterpret_cast<int*>(smem + C::kMisc + 8);  // RK, RV

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  int x = blockIdx.x;
  const int group = x % p.ngroups;
  x /= p.ngroups;
  const int head = x % p.H;
  const int split = x / p.H;
  const WorkDesc work = p.works[split];
  const ChunkDesc* chunks = p.chunks + work.chunk_begin;
  const int n = work.chunk_end - work.chunk_begin;  // units
  auto unit_keys = [&](int g) { return __ldg(&chunks[g].start_len) >> 16; };
  const int row0 = group * 2 * kTileRows;
  const int n_main = min(2, p.main_tiles - 2 * group);
  const bool has_tail = group == p.ngroups - 1 && p.tail_rows > 0;
  const int tail_row0 = p.main_tiles * kTileRows;
  const long long limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < SR; ++i) {
      ptx::mbar_init(raw_full(i), 1);
      ptx::mbar_init(raw_empty(i), 4);
    }
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(kv_full(i), 4);
      ptx::mbar_init(slot_free(i), max(1, n_main + (has_tail ? 2 : 0)));
    }
    ptx::mbar_init(q_full, 8);
    for (int t = 0; t < 2; ++t) {
      for (int b = 0; b < C::kBuffers; ++b) ptx::mbar_init(s_full(t, b), 1);
      // the four softmax warps (P of unit g) and the four widening warps (unit g + kBuffers): all that
      // the issuer's next step needs in one wait
      for (int b = 0; b < C::kBuffers; ++b) ptx::mbar_init(p_ready(t, b), 8);
    }
    for (int t = 0; t < 2; ++t) ptx::mbar_init(o_done(t), 1);
    *abort_flag = 0;
    refs[0] = refs[1] = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // launched as a programmatic dependent (see attention_tc_kernel)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == C::kWarpTma) {
    // ------------------------------------------------------------ producer
    if (lane == 0) ptx::prefetch_tmap(&kv_map);
    e4m3::ChunkReader reader(chunks, n, lane);
    int issued = 0;
    for (; issued < n; ++issued) {
      const int st = issued % SR;
      const ChunkDesc cd = reader.get(issued);
      if (!e4m3::wait_warp(raw_empty(st), ((issued / SR) & 1) ^ 1, limit, abort_flag)) {
        if (lane == 0) signal_abort(p.status, abort_flag);
        break;
      }
      if (lane == 0) {
        const int start = cd.start_len & 0xFFFF;
        const uint8_t* scales = p.scales + (int64_t(cd.page) * 2 * p.H + head) * p.scale_row + start;
        ptx::mbar_arrive_expect_tx(raw_full(st), 2 * C::kRawTile + 2 * kUnit);
        ptx::tma_load_4d(sRaw(st), &kv_map, 0, head, start, 2 * cd.page, raw_full(st));
        ptx::tma_load_4d(sRaw(st) + C::kRawTile, &kv_map, 0, head, start, 2 * cd.page + 1, raw_full(st));
        ptx::bulk_load(sScale(st), scales, kUnit, raw_full(st));
        ptx::bulk_load(sScale(st) + kUnit, scales + int64_t(p.H) * p.scale_row, kUnit, raw_full(st));
      }
    }
    if (lane == 0) {
      // copies must land before exit
      for (int i = issued > SR ? issued - SR : 0; i < issued; ++i)
        ptx::mbar_wait_bounded(raw_full(i % SR), (i / SR) & 1, limit, nullptr);
    }
    __syncwarp();
  } else {
    // RK and RV: the largest scale bytes of the split's keys, 16 at a time
    {
      const int worker = threadIdx.x < C::kWarpTma * 32 ? threadIdx.x : threadIdx.x - 32;
      uint32_t mk = 0, mv = 0;
      for (int i = worker; i < 8 * n; i += C::kThreads - 32) {
        const ChunkDesc cd = chunks[i >> 3];
        const int is_v = (i >> 2) & 1, off = (i & 3) * 16, left = (cd.start_len >> 16) - off;
        if (left <= 0) continue;
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(
            p.scales + (int64_t(2 * cd.page + is_v) * p.H + head) * p.scale_row + (cd.start_len & 0xFFFF) + off));
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // bytes past the last key do not count
          const int b = left - 4 * j;
          if (b < 4) w[j] = b <= 0 ? 0u : w[j] & (0xFFFFFFFFu >> (8 * (4 - b)));
        }
        const uint32_t m = __vmaxu4(__vmaxu4(w[0], w[1]), __vmaxu4(w[2], w[3]));
        if (is_v) mv = __vmaxu4(mv, m);
        else mk = __vmaxu4(mk, m);
      }
      const uint32_t k = __reduce_max_sync(0xffffffffu, byte_max(mk)), v = __reduce_max_sync(0xffffffffu, byte_max(mv));
      if (lane == 0) {
        atomicMax(refs, int(k));
        atomicMax(refs + 1, int(v));
      }
    }
    workers_sync<C::kThreads>();
    const int RK = refs[0], RV = refs[1];
    if (warp >= C::kWarpMma) {
      // ---------------------------------------------------------- MMA issuers
      // The whole warp runs the loop and an elected lane issues.  elect.sync tells the compiler that one
      // lane is left; behind `lane == 0` it guards the uniform operands of each tcgen05 instruction
      // against lanes that differ, and issuing, which every unit waits for, took 1,000 cycles a unit
      // and tile instead of 400.
      const int t = __shfl_sync(0xffffffffu, warp - C::kWarpMma, 0);
      if (t < n_main) {
        const uint32_t hi = uint32_t(ptx::smem_desc_sw128(sbase, 16, 1024) >> 32);
        auto lo_of = [&](uint32_t addr) { return uint32_t(ptx::smem_desc_sw128(addr, 16, 1024)); };
        constexpr uint32_t idesc_qk = ptx::idesc_f16_f32(128, kUnit, 0, 0);
        constexpr uint32_t idesc_pv = ptx::idesc_f16_f32(128, D, 0, 1);
        const uint32_t q_lo = lo_of(sbase + C::kQ + t * 128 * D * 2);
        const uint32_t tO = tmem + C::kO0 + uint32_t(t * D);
        const uint32_t tS0 = tmem + C::s_col(t, 0);
        // V' as an MN-major operand: the leading offset is the distance between 64-column blocks
        const uint32_t k_lo0 = lo_of(sK(0)), v_lo0 = uint32_t(ptx::smem_desc_sw128(sV(0), C::kBlock, 1024));
        constexpr uint32_t kStep = C::kTile >> 4;
        // Q K^T of the unit in slot `slot` into score buffer `buf`
        auto issue_qk = [&](int slot, int buf) {
          const uint32_t k_lo = k_lo0 + uint32_t(slot) * kStep, tS = tS0 + uint32_t(kUnit * buf);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = uint32_t((k >> 2) * (C::kBlock >> 4) + (k & 3) * 2);
            const uint32_t qoff = uint32_t((k >> 2) * (128 * 128 >> 4) + (k & 3) * 2);
            if (k == 0) ptx::mma_ss_lh<0>(tS, q_lo + qoff, k_lo + off, hi, idesc_qk);
            else ptx::mma_ss_lh<1>(tS, q_lo + qoff, k_lo + off, hi, idesc_qk);
          }
          ptx::mma_commit(s_full(t, 0) + 8 * buf);
        };
        // P V of unit g in slot `slot`, P in buffer `buf`
        auto issue_pv = [&](int g, int slot, int buf) {
          const uint32_t v_lo = v_lo0 + uint32_t(slot) * kStep;
          const uint32_t tP = tS0 + uint32_t(kUnit * buf);
#pragma unroll
          for (int k = 0; k < kUnit / 16; ++k)
            ptx::mma_ts_lh(tO, tP + 8 * k, v_lo + uint32_t(128 * k), hi, idesc_pv, (g > 0 || k > 0) ? 1u : 0u);
          ptx::mma_commit(slot_free(0) + 8 * slot);
        };
        bool ok = e4m3::wait_warp(q_full, 0, limit, abort_flag);
        // Positions in the rings are kept by counting.  i: slot of unit g; a: slot of the unit whose
        // scores are requested next; b: the buffer of unit g.
        int i = 0, a = 0, b = 0;
        uint32_t a_phase = 0, b_phase = 0;
        auto next_ahead = [&]() {
          if (++a == S) a = 0, a_phase ^= 1;
        };
        for (int g = 0; ok && g < C::kBuffers && g < n; ++g) {
          if (!(ok = e4m3::wait_warp(kv_full(a), a_phase, limit, abort_flag))) break;
          if (ptx::elect_one()) {
            ptx::tc_fence_after();
            issue_qk(a, g);
          }
          next_ahead();
        }
        for (int g = 0; ok && g < n; ++g) {
          const bool more = g + C::kBuffers < n;
          // P of unit g, and unit g + kBuffers widened
          if (!(ok = e4m3::wait_warp(p_ready(t, 0) + 8 * b, b_phase, limit, abort_flag))) break;
          if (ptx::elect_one()) {
            ptx::tc_fence_after();
            issue_pv(g, i, b);
            if (more) issue_qk(a, b);  // into the buffer that P V of unit g reads (in order)
          }
          __syncwarp();
          next_ahead();
          if (++i == S) i = 0;
          if (++b == C::kBuffers) b = 0, b_phase ^= 1;
        }
        if (ptx::elect_one()) {  // (the same lane every time)
          if (!ok) signal_abort(p.status, abort_flag);
          ptx::mma_commit(o_done(t));  // arrives once every MMA this thread issued has completed
          ptx::mbar_wait_bounded(o_done(t), 0, limit, nullptr);
        }
      }
      __syncwarp();
    } else if (warp >= kWarpMain) {
      // ---------------------------------------------------------- main-tile softmax
      if constexpr (kPlanRegs) ptx::regs_keep<C::kRegs>();
      const int t = (warp - kWarpMain) / (4 * C::kPar), par = C::kPar == 2 ? (warp >> 2) & 1 : 0, q4 = warp & 3;
      const int r = q4 * 32 + lane;
      const int row = row0 + t * kTileRows + r;
      const bool tile_on = t < n_main;
      const bool row_ok = tile_on && row < p.T;
      const uint32_t lane_off = uint32_t(q4 * 32) << 16;
      const uint32_t tO = tmem + C::kO0 + uint32_t(t * D) + lane_off;
      float rf = 0.f;
      if (par == 0) {
        if (tile_on) {
          const int64_t qrow = int64_t(work.stream) * p.T + row;
          const uint4* src =
              reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.q) + (qrow * p.H + head) * D);
          float scale;
          const float f = row_exponent<D>(src, row_ok, p.scale_log2, &scale);
          // (not 0: it multiplies the -inf of masked keys)
          rf = fmaxf(f * e4m3::scale_of(RK), 1.17549435e-38f);
          if constexpr (C::kPar == 2) {
            row_f[t * 128 + r] = rf;
            row_m[t * 128 + r] = -INFINITY;
          }
          {
            const uint32_t dst = sbase + uint32_t(C::kQ + t * 128 * D * 2 + r * 128);
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
              const uint4 v = row_ok ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
              sts128(dst + uint32_t((c >> 3) * 128 * 128 + (((c & 7) ^ (r & 7)) << 4)), to_f16x2(v.x, scale),
                     to_f16x2(v.y, scale), to_f16x2(v.z, scale), to_f16x2(v.w, scale));
            }
          }
        }
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_before();
        e4m3::arrive_warp(q_full);
      }
      if (tile_on) {
        bool ok = e4m3::wait_warp(q_full, 0, limit, abort_flag);
        if constexpr (C::kPar == 2) rf = row_f[t * 128 + r];
        float m = -INFINITY, l = 0.f;  // running max in log2 units; sum of this thread's P'
        // buffer of unit g and its phase, kept by counting
        const uint32_t tS0 = tmem + C::s_col(t, 0) + lane_off;
        int buf = par, phase = 0;
        for (int g = par; ok && g < n; g += C::kPar) {
          const int keys = unit_keys(g);
          if (!(ok = e4m3::wait_warp(s_full(t, 0) + 8 * buf, phase, limit, abort_flag))) break;
          ptx::tc_fence_after();
          const uint32_t tS = tS0 + uint32_t(kUnit * buf);
          if (keys < kUnit) mask_scores(tS, keys);
          float h0 = 0.f, h1 = 0.f;
          // What refers to m when it becomes m_new: this thread's sums, and the P' of this unit's
          // first `words` 16-column words that are already stored (m only takes whole numbers, so
          // the corrections are exact).
          auto adopt = [&](float m_new, int words) {
            const float corr = m_new == m ? 1.f : ptx::ex2(m - m_new);  // 0 while m is -inf
            if (words > 0) {
              // (as two factors: corr alone may lie below fp16's least value)
              const float e0 = truncf((m - m_new) * 0.5f), f0 = ptx::ex2(e0), f1 = ptx::ex2(m - m_new - e0);
              const uint32_t c0 = e4m3::pack_f16(f0, f0), c1 = e4m3::pack_f16(f1, f1);
              ptx::tmem_wait_st();
#pragma unroll 1
              for (int w = 0; w < words; ++w) {
                uint32_t pk[16];
                ptx::tmem_ld16(tS + 16 * w, pk);
                ptx::tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 16; ++e) pk[e] = ptx::mul_f16x2(ptx::mul_f16x2(pk[e], c0), c1);
                ptx::tmem_st16(tS + 16 * w, pk);
              }
            }
            if (m_new != m) {
              l *= corr;
              h0 *= corr;
              h1 *= corr;
              m = m_new;
            }
            return corr;
          };
          // head_dim 64: the unit before has published its P, and with it m.  Waited for once per
          // unit, as late as can be, so that the exponentials of two units overlap.
          bool token = C::kPar == 1 || g == 0;
          auto take_token = [&](int words) -> bool {
            token = true;
            const bool wrapped = buf == 0;  // unit g - 1 is in the buffer before this one
            if (!e4m3::wait_warp(p_ready(t, 0) + 8 * (wrapped ? C::kBuffers - 1 : buf - 1), phase ^ (wrapped ? 1 : 0), limit,
                                 abort_flag))
              return false;
            const float ms = row_m[t * 128 + r];
            if (__any_sync(0xffffffffu, ms != m)) adopt(ms, words);
            return true;
          };
          // Move m up to the next whole number above a score and rescale O, once every earlier
          // product has completed.
          auto move_max = [&](bool need, float mx, int words) -> bool {
            if (!token && !take_token(words)) return false;
            const float m_new = need ? fmaxf(m, ceilf(mx * rf)) : m;
            bool good = true;
            const float corr = adopt(m_new, words);
            if (g > 0) {
              good = e4m3::wait_warp(slot_free((g - 1) % S), ((g - 1) / S) & 1, limit, abort_flag);
              ptx::tc_fence_after();
              rescale_o(tO, D, corr);
            }
            if constexpr (C::kPar == 2) row_m[t * 128 + r] = m;
            return good;
          };
          // 32 keys at a time, P over the scores they came from: the first half's P' takes the
          // columns of scores already read
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[16];
            float u0, u1;
            bool moved = false;
            for (;;) {
              uint32_t sv[32];
              u0 = u1 = 0.f;
              ptx::tmem_ld32(tS + 32 * half, sv);
              ptx::tmem_wait_ld();
              exps(sv, rf, float(kBias) - m, pk, u0, u1);
              const bool need = !(u0 + u1 < kSumLimit);
              if (moved || !__any_sync(0xffffffffu, need)) break;
              // rare: the first unit, and jumps of the maximum
              moved = true;
              ptx::tmem_ld32(tS + 32 * half, sv);
              ptx::tmem_wait_ld();
              if (!(ok = move_max(need, max32(sv, -INFINITY), half))) break;
            }
            if (!ok) break;
            h0 += u0;
            h1 += u1;
            ptx::tmem_st16(tS + 16 * half, pk);
          }
          if (!ok || !(ok = token || take_token(2))) break;
          l += h0 + h1;
          ptx::tmem_wait_st();
          ptx::tc_fence_before();
          e4m3::arrive_warp(p_ready(t, 0) + 8 * buf);
          buf += C::kPar;
          if (buf >= C::kBuffers) {
            buf -= C::kBuffers;
            phase ^= 1;
          }
        }
        if (!ok) signal_abort(p.status, abort_flag);
        ok = e4m3::wait_warp(o_done(t), 0, limit, abort_flag) && ok;
        if constexpr (C::kPar == 2) {
          // the two parts of the row sum, both against the final m
          if (ok) {
            const float ms = row_m[t * 128 + r];
            if (ms != m) l *= ptx::ex2(m - ms);
            m = ms;
            row_l[(t * 2 + par) * 128 + r] = l;
          }
          tile_sync(t);
          l = row_l[t * 256 + r] + row_l[t * 256 + 128 + r];
        }
        if (ok && *abort_flag == 0) {
          ptx::tc_fence_after();
          const float inv = e4m3::scale_of(RV) / l;
          const bool direct = work.nsplit == 1 && !p.force_part;
#pragma unroll 1
          for (int j = 0; j < D / 32 / C::kPar; ++j) {  // this warpgroup's columns
            const int col = par * (D / 2) + 32 * j;
            uint32_t v[32];
            ptx::tmem_ld32(tO + col, v);
            ptx::tmem_wait_ld();
            if (!row_ok) continue;
            if (direct) {
              const int64_t qrow = int64_t(work.stream) * p.T + row;
              uint4* dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + (qrow * p.H + head) * D + col);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(v[8 * k + 2 * i]) * inv,
                                                                 __uint_as_float(v[8 * k + 2 * i + 1]) * inv);
                  w[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
                dst[k] = make_uint4(w[0], w[1], w[2], w[3]);
              }
            } else {
#pragma unroll
              for (int k = 0; k < 8; ++k)
                *reinterpret_cast<float4*>(p.part_o + part_o_offset<D>(split, head, row, col + 4 * k, p.H, p.T)) =
                    make_float4(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv,
                                __uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv);
            }
          }
          if (row_ok && par == 0) {
            const float lse = m - float(kBias) + log2f(l);
            if (!direct) p.part_lse[(int64_t(split) * p.H + head) * p.T + row] = lse;
            else if (p.lse != nullptr) p.lse[(int64_t(work.stream) * p.T + row) * p.H + head] = e4m3::kLn2 * lse;
          }
        }
      }
    } else if (warp < kWarpTail) {
      // ---------------------------------------------------------- widening
      if constexpr (kPlanRegs) ptx::regs_keep<C::kRegs>();
      bool ok = true;
      int s = 0, raw = 0;
      uint32_t phase = 0, raw_phase = 0;
      for (int i = 0; i < n; ++i) {
        const int keys = unit_keys(i);
        ok = e4m3::wait_warp(raw_full(raw), raw_phase, limit, abort_flag) &&
             (i < S || e4m3::wait_warp(slot_free(s), phase ^ 1, limit, abort_flag));
        if (!ok) break;
        widen_unit<D>(sRaw(raw), sScale(raw), sK(s), sV(s), RK, RV, keys, threadIdx.x);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(kv_full(s));
          ptx::mbar_arrive(raw_empty(raw));
          // (unit i - kBuffers has the same buffer, and its phase is open: the slot that this unit took
          // was freed by P V of unit i - S, S = 2 kBuffers)
          if (i >= C::kBuffers)
            for (int t = 0; t < n_main; ++t) ptx::mbar_arrive(p_ready(t, i));
        }
        if (++s == S) s = 0, phase ^= 1;
        if (++raw == SR) raw = 0, raw_phase ^= 1;
      }
      // the last units have none behind them: their P alone is waited for
      for (int i = max(n, C::kBuffers); ok && i < n + C::kBuffers; ++i)
        for (int t = 0; ok && t < n_main; ++t) {
          ok = i < 2 * C::kBuffers || e4m3::wait_warp(p_ready(t, i), p_phase(i - 2 * C::kBuffers), limit, abort_flag);
          if (ok && lane == 0) ptx::mbar_arrive(p_ready(t, i));
        }
      if (!ok) signal_abort(p.status, abort_flag);
    } else {
      // ---------------------------------------------------------- tail
      if constexpr (kPlanRegs) ptx::regs_keep<C::kRegs>();
      if (has_tail) {
        const int q = warp & 3, gr = lane >> 2, tq = lane & 3;
        const int par = q >> 1, k0 = 32 * (q & 1);  // this warp's units and its keys of them
        const bool have = gr < p.tail_rows;
        // Q' fragments of row gr
        uint32_t qa[D / 16][2];
        float rf[2];  // of rows 2 tq and 2 tq + 1
        {
          const uint32_t* src = reinterpret_cast<const uint32_t*>(
              static_cast<const __nv_bfloat16*>(p.q) +
              ((int64_t(work.stream) * p.T + tail_row0 + (have ? gr : 0)) * p.H + head) * D);
          uint32_t amax = 0;
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t v = have ? __ldg(src + 8 * k + 4 * h + tq) : 0u;
              qa[k][h] = v;
              amax = max(amax, max((v << 16) & 0x7FFFFFFFu, v & 0x7FFF0000u));
            }
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
          amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
          const uint32_t e = min(max(amax >> 23, 1u), 253u);
          const float scale = __uint_as_float((254u - e) << 23);
          const float f = p.scale_log2 * __uint_as_float(e << 23) * e4m3::scale_of(RK);
          rf[0] = __shfl_sync(0xffffffffu, f, 8 * tq);
          rf[1] = __shfl_sync(0xffffffffu, f, 8 * tq + 4);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            qa[k][0] = to_f16x2(qa[k][0], scale);
            qa[k][1] = to_f16x2(qa[k][1], scale);
          }
        }
        // O^T = V'^T P^T (16 dims x 8 rows a product): dims gr and gr + 8 of 16, rows 2 tq + {0, 1}
        float o[D / 16][4];
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        bool ok = true;
        // ldmatrix rows and pieces of this lane, four 8 x 8 blocks: K' keys and dims, V' dims and keys
        const int k_row = k0 + (lane & 15), k_piece = lane >> 4;
        const int v_row = k0 + (lane & 7) + 8 * (lane >> 4), v_piece = (lane >> 3) & 1;
        auto at = [&](uint32_t tile, int row, int pc) {
          return tile + uint32_t((pc >> 3) * C::kBlock + row * 128 + (((pc & 7) ^ (row & 7)) << 4));
        };
        int s = par;
        uint32_t phase = 0;
        for (int j = par; j < n; j += 2) {
          const int keys = unit_keys(j);
          if (!(ok = e4m3::wait_warp(kv_full(s), phase, limit, abort_flag))) break;
          if (k0 < keys) {
            // x[kk][2 h + i]: key k0 + 16 kk + 8 h + gr, row 2 tq + i.  The sums over even and odd k-steps
            // apart: one warp a sub-partition has only its own instructions to hide latencies with.
            float x[2][4], mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              uint32_t a[D / 16][4];
#pragma unroll
              for (int k = 0; k < D / 16; ++k) ldmatrix4(a[k], at(sK(s), k_row + 16 * kk, 2 * k + k_piece));
              float odd[4] = {0.f, 0.f, 0.f, 0.f};
              x[kk][0] = x[kk][1] = x[kk][2] = x[kk][3] = 0.f;
#pragma unroll
              for (int k = 0; k < D / 16; k += 2) {
                e4m3::mma_16816(x[kk], a[k], qa[k][0], qa[k][1]);
                e4m3::mma_16816(odd, a[k + 1], qa[k + 1][0], qa[k + 1][1]);
              }
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const bool in = k0 + 16 * kk + 8 * (e >> 1) + gr < keys;
                x[kk][e] = in ? (x[kk][e] + odd[e]) * rf[e & 1] : -INFINITY;
                mx[e & 1] = fmaxf(mx[e & 1], x[kk][e]);
              }
            }
            if (__any_sync(0xffffffffu, mx[0] > m[0] + kHeadroom || mx[1] > m[1] + kHeadroom)) {
              float corr[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int d = 4; d < 32; d *= 2) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
                const float m_new = fmaxf(m[i], mx[i]);
                corr[i] = m_new == m[i] ? 1.f : ptx::ex2(m[i] - m_new);  // 0 while m is -inf
                m[i] = m_new;
                l[i] *= corr[i];
              }
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                o[i][0] *= corr[0];
                o[i][1] *= corr[1];
                o[i][2] *= corr[0];
                o[i][3] *= corr[1];
              }
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                x[kk][e] = ptx::ex2(x[kk][e] + (float(kBias) - m[e & 1]));
                l[e & 1] += x[kk][e];
              }
              const uint32_t p0 = e4m3::transpose_8x8(e4m3::pack_f16(x[kk][0], x[kk][1]));
              const uint32_t p1 = e4m3::transpose_8x8(e4m3::pack_f16(x[kk][2], x[kk][3]));
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                uint32_t a[4];
                ldmatrix4_trans(a, at(sV(s), v_row + 16 * kk, 2 * i + v_piece));
                e4m3::mma_16816(o[i], a, p0, p1);
              }
            }
          }
          e4m3::arrive_warp(slot_free(s));
          s += 2;
          if (s >= S) s -= S, phase ^= 1;
        }
        if (!ok) signal_abort(p.status, abort_flag);
        // Join of the four warps over the raw ring, which nothing uses once the warps of the last unit have
        // found it widened
        tail_bar_sync();
        float* jo = reinterpret_cast<float*>(smem + C::kRawOff);
        float* jm = jo + 4 * 8 * D;
        float* jl = jm + 32;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int d = 4; d < 32; d *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
        if (ok) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              jo[(q * 8 + 2 * tq + (k & 1)) * D + 16 * i + gr + 8 * (k >> 1)] = o[i][k];
          if (gr == 0) {
            jm[q * 8 + 2 * tq] = m[0];
            jm[q * 8 + 2 * tq + 1] = m[1];
            jl[q * 8 + 2 * tq] = l[0];
            jl[q * 8 + 2 * tq + 1] = l[1];
          }
        }
        tail_bar_sync();
        if (ok && *abort_flag == 0) {
          for (int u = threadIdx.x - 32 * kWarpTail; u < p.tail_rows * (D / 4); u += 128) {
            const int r = u / (D / 4), c4 = u % (D / 4), row = tail_row0 + r;
            float M = -INFINITY, L = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int w = 0; w < 4; ++w) M = fmaxf(M, jm[w * 8 + r]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float mw = jm[w * 8 + r], f = mw == M ? 1.f : ptx::ex2(mw - M);
              const float4 v = *reinterpret_cast<const float4*>(jo + (w * 8 + r) * D + 4 * c4);
              L = fmaf(f, jl[w * 8 + r], L);
              acc.x = fmaf(f, v.x, acc.x);
              acc.y = fmaf(f, v.y, acc.y);
              acc.z = fmaf(f, v.z, acc.z);
              acc.w = fmaf(f, v.w, acc.w);
            }
            const float inv = e4m3::scale_of(RV) / L;
            if (work.nsplit == 1 && !p.force_part) {
              const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                   b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
              uint2 pk;
              pk.x = *reinterpret_cast<const uint32_t*>(&a);
              pk.y = *reinterpret_cast<const uint32_t*>(&b);
              *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                        ((int64_t(work.stream) * p.T + row) * p.H + head) * D + 4 * c4) = pk;
              if (p.lse != nullptr && c4 == 0)
                p.lse[(int64_t(work.stream) * p.T + row) * p.H + head] = e4m3::kLn2 * (M - float(kBias) + log2f(L));
            } else {
              *reinterpret_cast<float4*>(p.part_o + part_o_offset<D>(split, head, row, 4 * c4, p.H, p.T)) =
                  make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
              if (c4 == 0) p.part_lse[(int64_t(split) * p.H + head) * p.T + row] = M - float(kBias) + log2f(L);
            }
          }
        }
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// regs_keep may only name the count that a launch gives, which is the build's: ptxas takes the most that
// the launch bounds leave, 72 and 96, with every flag tried.  A build that comes to another count runs
// the kernel without it (2 to 7 % slower; asking in the kernel costs the same, the roles' registers are
// then planned together).
template <int D>
std::atomic<bool> g_plan_regs{false};

template <int D>
cudaError_t configure_tc() {
  cudaFuncAttributes a;
  cudaError_t e = cudaFuncGetAttributes(&a, attention_e4m3_tc_kernel<D, true>);
  if (e != cudaSuccess) return e;
  const bool plan = a.numRegs == Cfg<D>::kRegs;
  g_plan_regs<D> = plan;
  return cudaFuncSetAttribute(plan ? attention_e4m3_tc_kernel<D, true> : attention_e4m3_tc_kernel<D, false>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kLaunch);
}

template <int D>
cudaError_t launch_tc(const AttnParams& p, const CUtensorMap* map, cudaStream_t s) {
  const int64_t grid = int64_t(p.num_splits) * p.H * p.ngroups;
  if (grid <= 0 || grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent(g_plan_regs<D> ? attention_e4m3_tc_kernel<D, true> : attention_e4m3_tc_kernel<D, false>,
                          dim3(unsigned(grid)), dim3(Cfg<D>::kThreads), Cfg<D>::kLaunch, s, p, *map);
}

}  // namespace

cudaError_t configure_attention_e4m3_tc() {
  const cudaError_t e = configure_tc<64>();
  return e != cudaSuccess ? e : configure_tc<128>();
}

cudaError_t launch_attention_e4m3_tc(const AttnParams& p, const CUtensorMap* unit_map, cudaStream_t s) {
  return p.D == 64 ? launch_tc<64>(p, unit_map, s) : launch_tc<128>(p, unit_map, s);
}

}  // namespace spk
