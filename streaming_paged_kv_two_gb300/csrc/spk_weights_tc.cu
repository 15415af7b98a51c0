// Accumulated attention weights of the special keys on the tensor cores (SPK_BF16, SPK_E4M3):
//   part[s][h][j] = sum over the call's query rows i of 2^(a_j (q_i k_j) - lse_i log2(e)),
// a second pass over K alone, the rows' log-sum-exps being known.
//
// The scores are taken transposed, S^T = K Q^T (M = 128 keys, N = query rows), so a thread owns a
// key (= TMEM lane): its scale is one register, and its sum needs no exchange.  One CTA = (split of
// the stream's special keys, head, stream).  Q stays in shared memory for the whole CTA, K streams
// through a ring, and nothing is written but one fp32 per key and head.  What bounds it is the
// exponentials, n H T of them at 4 cycles per warp and SM sub-partition, so four warpgroups share
// them: warpgroup w takes the tiles w, w + 4, ... and has a 128-column score buffer of its own; while
// it waits for its next scores the other three keep the exponential unit busy.  Products are few and
// wide: a thread issues one in some tens of cycles whatever its width.
//
// SPK_E4M3: the codes are the operand as they lie in the pool, and q, scaled by one power of two per
// head so that its largest value is in (224, 448], is the sum of two e4m3 values (q's 8 significant
// bits are 4 + 4): exact but for values below 2^-9 of the largest, which lose at most 2^-17 of it (half
// of e4m3's least step, 2^-9, of 224).  Where a row needs a power of two more than 2^kApart above that,
// so that it would lose more than 2^-13 of its own largest value, each row has its own, undone in its
// scores (exactly; that multiplies every score: 67 us become 76, so rows near one another share one).
// Both products go into the same accumulator; nothing is widened.  SPK_BF16: both as they are.
//
// Measured: 60,000 keys of 16 heads of 64 dims, 262 rows, e4m3: 61 us with the heads' sum over one set of
// inputs, 68 over inputs that change, where the exponentials alone would take 31 (16 scores a load: 4 us
// more; 16 scores loaded ahead of their use: 6; more score buffers or more issuers, measured with slower
// issuers: 15 to 18); bf16 60; 1,200 keys, bf16: 9 us.
#include "ptx_sm100.cuh"
#include "spk_e4m3.cuh"
#include "spk_internal.h"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace spk {
namespace {

constexpr int kGroups = 4;                          // exponential warpgroups
constexpr int kIssuers = 2;                         // each serves every other warpgroup
constexpr int kWarpExp = 4;                         // warp 0: producer, 1 and 2: issuers; 3 only loads Q
constexpr int kThreads = 32 * (kWarpExp + 4 * kGroups);
constexpr int kTileKeys = 128;
constexpr int kBufCols = 128;                       // TMEM columns of a warpgroup's score buffer
constexpr int kCols = 32;                           // scores a thread loads at a time
constexpr int kApart = 4;                           // e4m3: see above
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool kE4m3>
struct WCfg {
  static constexpr int kElem = kE4m3 ? 1 : 2;
  static constexpr int kRowBytes = kE4m3 ? D : 128;  // a swizzled row: all of D (e4m3) or 64 dims
  static constexpr int kBlocks = kE4m3 ? 1 : D / 64; // column blocks of K (and Q)
  static constexpr int kTile = kTileKeys * D * kElem;
  static constexpr int kKBlock = kTileKeys * kRowBytes;
  // query rows of one pass: Q takes 2 D bytes a row (two e4m3 terms, or bf16)
  static constexpr int kRows = D == 64 ? 768 : 384;
  // an even number, so that a slot's tiles always belong to one issuer (a wait only tells a phase
  // from the one before it, so nobody may skip one)
  static constexpr int kStages = D == 64 ? (kE4m3 ? 8 : 6) : kE4m3 ? 6 : 4;
  static constexpr int kQBytes = kRows * 2 * D;
  static constexpr int kK = kQBytes;
  static constexpr int kLse = kK + kStages * kTile;
  static constexpr int kRowF = kLse + kRows * 4;     // e4m3: the rows' own factors, where they are apart
  static constexpr int kBars = kRowF + (kE4m3 ? kRows * 4 : 0);
  // k_full, k_empty [kStages], s_full, s_free [kGroups], done [kIssuers]
  static constexpr int kMisc = kBars + 8 * (2 * kStages + 2 * kGroups + kIssuers);
  static constexpr int kBytes = kMisc + 16;
  static constexpr int kLaunch = kBytes + 1024;
  static_assert(kStages >= kGroups && kStages % kIssuers == 0, "four tiles are held at a time");
  static_assert(kLaunch <= 227 * 1024 && kK % 1024 == 0, "shared memory");
};

struct WeightTcParams {
  WeightParams w;
  int32_t row0, rows;         // query rows of this pass
  int32_t groups, group_rows; // its row groups (<= kBufCols rows, a multiple of kCols, each)
  int32_t splits;             // CTAs per (stream, head)
  int32_t unit_tokens;        // tokens of a planner chunk
  int32_t add;                // add to `part` (passes after the first)
};

// 128-byte or 64-byte swizzled K-major operand
template <int kRowBytes>
__device__ __forceinline__ uint64_t desc(uint32_t addr) {
  return uint64_t((addr >> 4) & 0x3FFFu) | (uint64_t(1) << 16) | (uint64_t((8 * kRowBytes) >> 4) << 32) |
         (uint64_t(1) << 46) | (uint64_t(kRowBytes == 128 ? 2 : 4) << 61);
}

// 16-byte piece c of row r in a tile of kRowBytes-byte swizzled rows
template <int kRowBytes>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return kRowBytes == 128 ? uint32_t(r * 128 + ((c ^ (r & 7)) << 4)) : uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ float4 lds_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

// Four values x[0..3] scaled by s as e4m3 codes hi and the codes lo of what they leave.
__device__ __forceinline__ void split4(const uint32_t (&bf16x2)[2], float s, uint32_t& hi, uint32_t& lo) {
  float x[4] = {__uint_as_float(bf16x2[0] << 16) * s, __uint_as_float(bf16x2[0] & 0xFFFF0000u) * s,
                __uint_as_float(bf16x2[1] << 16) * s, __uint_as_float(bf16x2[1] & 0xFFFF0000u) * s};
  hi = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3)) |
       uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3)) << 16;
  const uint32_t a = e4m3::widen_lo(hi), b = e4m3::widen_hi(hi);
  const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
  lo = uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[0] - fa.x, x[1] - fa.y), __NV_SATFINITE, __NV_E4M3)) |
       uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(x[2] - fb.x, x[3] - fb.y), __NV_SATFINITE, __NV_E4M3)) << 16;
}

// Largest finite magnitude of a row, whose D / 8 consecutive lanes hold 8 values each (fp32 bits).
template <int D>
__device__ __forceinline__ uint32_t row_amax(uint4 v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = (x[j] << 16) & 0x7FFFFFFFu, b = x[j] & 0x7FFF0000u;
    amax = max(amax, max(a < 0x7F800000u ? a : 0u, b < 0x7F800000u ? b : 0u));
  }
#pragma unroll
  for (int o = 1; o < D / 8; o *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  return amax;
}

// k with 2^k |q| in (224, 448]: with |q| = 1.m 2^(E - 127), k = 8 - (E - 127) - (1.m > 1.75)
__device__ __forceinline__ int scale_exponent(uint32_t amax) {
  return amax == 0 ? 0 : min(max(135 - int(amax >> 23) - ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0), -120), 120);
}

// Sum over `cols` score columns of 2^(a s f + m): m and f one value a column at shared addresses m_at and
// f_at (f = 1 without kOwnFactors).  Arrives at `free_bar` once the scores are in registers.
template <bool kOwnFactors>
__device__ __forceinline__ float add_terms(uint32_t tS, uint32_t m_at, uint32_t f_at, float a, int cols, uint32_t free_bar) {
  float h0 = 0.f, h1 = 0.f;
#pragma unroll 1
  for (int j = 0; j < cols; j += kCols) {
    uint32_t s[kCols];
    ptx::tmem_ld32(tS + uint32_t(j), s);
    ptx::tmem_wait_ld();
    if (j + kCols >= cols) {
      ptx::tc_fence_before();
      e4m3::arrive_warp(free_bar);
    }
#pragma unroll
    for (int e = 0; e < kCols; e += 4) {
      float x0 = __uint_as_float(s[e]), x1 = __uint_as_float(s[e + 1]), x2 = __uint_as_float(s[e + 2]),
            x3 = __uint_as_float(s[e + 3]);
      const float4 m = lds_f4(m_at + uint32_t(4 * (j + e)));
      if constexpr (kOwnFactors) {
        const float4 f = lds_f4(f_at + uint32_t(4 * (j + e)));
        x0 *= f.x, x1 *= f.y, x2 *= f.z, x3 *= f.w;
      }
      ptx::fma2(x0, x1, x0, x1, a, m.x, m.y);
      ptx::fma2(x2, x3, x2, x3, a, m.z, m.w);
      ptx::add2(h0, h1, ptx::ex2(x0), ptx::ex2(x1));
      ptx::add2(h0, h1, ptx::ex2(x2), ptx::ex2(x3));
    }
  }
  return h0 + h1;
}
// (out of line: inlined beside the common path it costs that 3 of 67 us, so 1)
__device__ __noinline__ float add_terms_apart(uint32_t tS, uint32_t m_at, uint32_t f_at, float a, int cols, uint32_t free_bar) {
  return add_terms<true>(tS, m_at, f_at, a, cols, free_bar);
}

template <int D, bool kE4m3>
__global__ void __launch_bounds__(kThreads, 1)
    weight_tc_kernel(const WeightTcParams p, const __grid_constant__ CUtensorMap kv_map) {
  using C = WCfg<D, kE4m3>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  auto k_full = [&](int s) { return sbase + uint32_t(C::kBars + 8 * s); };
  auto k_empty = [&](int s) { return sbase + uint32_t(C::kBars + 8 * (S + s)); };
  auto s_full = [&](int i) { return sbase + uint32_t(C::kBars + 8 * (2 * S + i)); };
  auto s_free = [&](int i) { return sbase + uint32_t(C::kBars + 8 * (2 * S + kGroups + i)); };
  auto done = [&](int i) { return sbase + uint32_t(C::kBars + 8 * (2 * S + 2 * kGroups + i)); };
  float* neg_lse = reinterpret_cast<float*>(smem + C::kLse);
  float* row_f = reinterpret_cast<float*>(smem + C::kRowF);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kMisc);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kMisc + 4);
  uint32_t* q_amax = reinterpret_cast<uint32_t*>(smem + C::kMisc + 8);   // of all rows
  uint32_t* q_least = reinterpret_cast<uint32_t*>(smem + C::kMisc + 12);  // of the row with the smallest but 0

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WeightParams& w = p.w;
  const int head = blockIdx.y, stream = blockIdx.z;
  const long long limit = w.wait_limit_ns;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(k_full(i), 1);
      ptx::mbar_init(k_empty(i), 1);
    }
    for (int i = 0; i < kGroups; ++i) {
      ptx::mbar_init(s_full(i), 1);
      ptx::mbar_init(s_free(i), 4);
    }
    for (int i = 0; i < kIssuers; ++i) ptx::mbar_init(done(i), 1);
    *abort_flag = 0;
    *q_amax = 0;
    *q_least = 0xFFFFFFFFu;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  if (warp == 0) {
    ptx::tmem_alloc(ptx::smem_u32(tmem_slot), 512);
    ptx::tmem_relinquish();
  }
  // launched as a programmatic dependent (see attention_tc_kernel)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const StreamDesc sd = w.streams[stream];
  const ChunkDesc* chunks = w.chunks + sd.special_chunk;
  // units (planner chunks) of the stream's special tokens, and the tiles of 128 keys made of them
  const int full_pages = sd.specials / w.ps, rest = sd.specials - full_pages * w.ps;
  const int units = full_pages * w.chunks_per_page + (rest + p.unit_tokens - 1) / p.unit_tokens;
  constexpr int kPerTile = kE4m3 ? 2 : 1;
  const int tiles = (units + kPerTile - 1) / kPerTile;
  const int t0 = int(int64_t(tiles) * blockIdx.x / p.splits), t1 = int(int64_t(tiles) * (blockIdx.x + 1) / p.splits);
  const int n = t1 - t0;
  const int64_t q_stride = int64_t(w.H) * D;
  const __nv_bfloat16* q0 =
      static_cast<const __nv_bfloat16*>(w.q) + (int64_t(stream) * w.T + p.row0) * q_stride + int64_t(head) * D;
  __syncthreads();
  const uint32_t tmem = *tmem_slot;
  constexpr int kPieces = D / 8;  // 16-byte pieces of a bf16 row
  const int padded = p.groups * p.group_rows;
  if (n > 0) {
    // (past the last row: that row again, at weight 0 below.  Zeros would turn an infinite key's score
    // into a NaN that no row has.)
    auto piece_of = [&](int i) {
      return __ldg(reinterpret_cast<const uint4*>(q0 + min(i / kPieces, p.rows - 1) * q_stride) + i % kPieces);
    };
    // (padded rows are whole warps of pieces, which take each step together)
    if constexpr (kE4m3) {
      uint32_t amax = 0, least = 0xFFFFFFFFu;
      for (int i = threadIdx.x; i < padded * kPieces; i += kThreads) {
        const uint32_t a = row_amax<D>(piece_of(i));
        amax = max(amax, a);
        if (a) least = min(least, a);
      }
      amax = __reduce_max_sync(0xffffffffu, amax);
      least = __reduce_min_sync(0xffffffffu, least);
      if (lane == 0) {
        atomicMax(q_amax, amax);
        atomicMin(q_least, least);
      }
    }
    __syncthreads();
    float factor = w.scale_log2;  // score of a key: factor (its scale) (product)
    int k_head = 0;
    bool apart = false;
    if constexpr (kE4m3) {
      k_head = scale_exponent(*q_amax);
      factor *= __uint_as_float(uint32_t(127 - k_head) << 23);
      apart = *q_amax > 0 && scale_exponent(*q_least) - k_head > kApart;
    }
    for (int i = threadIdx.x; i < padded * kPieces; i += kThreads) {
      const int r = i / kPieces, c = i % kPieces;
      const uint4 v = piece_of(i);
      if constexpr (kE4m3) {
        int k = k_head;
        if (apart) {
          k = min(max(scale_exponent(row_amax<D>(v)), k_head), k_head + 126);
          if (c == 0) row_f[r] = __uint_as_float(uint32_t(127 + k_head - k) << 23);
        }
        const float scale = __uint_as_float(uint32_t(127 + k) << 23);
        const uint32_t x0[2] = {v.x, v.y}, x1[2] = {v.z, v.w};
        uint32_t hi[2], lo[2];
        split4(x0, scale, hi[0], lo[0]);
        split4(x1, scale, hi[1], lo[1]);
        const uint32_t at = sbase + piece<C::kRowBytes>(r, c >> 1) + uint32_t((c & 1) * 8);
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(hi[0]), "r"(hi[1]) : "memory");
        asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at + uint32_t(padded * C::kRowBytes)), "r"(lo[0]), "r"(lo[1])
                     : "memory");
      } else {
        sts128(sbase + uint32_t((c >> 3) * padded * 128) + piece<128>(r, c & 7), v);
      }
    }
    for (int r = threadIdx.x; r < padded; r += kThreads)  // rows past the last weigh nothing
      neg_lse[r] = r < p.rows ? -kLog2e * w.lse[(int64_t(stream) * w.T + p.row0 + r) * w.H + head] : -INFINITY;
    ptx::fence_proxy_async_smem();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();

    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) ptx::prefetch_tmap(&kv_map);
      const int u1 = min(t1 * kPerTile, units);
      e4m3::ChunkReader reader(chunks + t0 * kPerTile, u1 - t0 * kPerTile, lane);
      int issued = 0;
      for (; issued < n; ++issued) {
        const int st = issued % S;
        const uint32_t dst = sbase + uint32_t(C::kK + st * C::kTile);
        const int count = min(kPerTile, units - (t0 + issued) * kPerTile);
        if (!e4m3::wait_warp(k_empty(st), ((issued / S) & 1) ^ 1, limit, abort_flag)) {
          *abort_flag = 1;
          if (lane == 0) atomicExch(w.status, kStatusWaitTimeout);
          break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(k_full(st), uint32_t(count * C::kTile / kPerTile));
        for (int u = 0; u < count; ++u) {
          const ChunkDesc cd = reader.get(issued * kPerTile + u);
          if (lane == 0) {
#pragma unroll
            for (int b = 0; b < C::kBlocks; ++b)
              ptx::tma_load_4d(dst + uint32_t(u * (C::kTile / kPerTile) + b * C::kKBlock), &kv_map, b * 64, head,
                               cd.start_len & 0xFFFF, 2 * cd.page, k_full(st));
          }
        }
      }
      if (lane == 0) {
        for (int i = issued > S ? issued - S : 0; i < issued; ++i)
          ptx::mbar_wait_bounded(k_full(i % S), (i / S) & 1, limit, nullptr);
      }
      __syncwarp();
    } else if (warp <= kIssuers) {
      // ---------------------------------------------------------- issuers
      // In order: for each four tiles (one per warpgroup), for each row group, this thread's tiles.
      // The whole warp runs the loops and an elected lane issues (see attention_e4m3_tc_kernel).
      const int me = __shfl_sync(0xffffffffu, warp, 0) - 1;
      const uint32_t idesc = kE4m3 ? ptx::idesc_f16_f32(128, p.group_rows, 0, 0)  // (all formats 0: e4m3)
                                   : ptx::idesc_bf16_f32(128, p.group_rows, 0, 0);
      const uint64_t d0 = desc<C::kRowBytes>(sbase);
      const uint32_t hi = uint32_t(d0 >> 32), lo = uint32_t(d0);  // of the start of shared memory
      const uint32_t q_step = uint32_t(p.group_rows * C::kRowBytes) >> 4, q_block = uint32_t(padded * C::kRowBytes) >> 4;
      bool ok = true;
      for (int c0 = 0; ok && c0 < n; c0 += kGroups)
        for (int g = 0; ok && g < p.groups; ++g)
          for (int wg = me; wg < kGroups && c0 + wg < n; wg += kIssuers) {
            const int c = c0 + wg, st = c % S, use = (c0 / kGroups) * p.groups + g;
            ok = (g > 0 || e4m3::wait_warp(k_full(st), (c / S) & 1, limit, abort_flag)) &&
                 (use == 0 || e4m3::wait_warp(s_free(wg), (use - 1) & 1, limit, abort_flag));
            if (!ok) break;
            if (ptx::elect_one()) {
              ptx::tc_fence_after();
              const uint32_t k_lo = lo + uint32_t((C::kK + st * C::kTile) >> 4);
              const uint32_t q_lo = lo + uint32_t(g) * q_step;
              const uint32_t tS = tmem + uint32_t(wg * kBufCols);
              if constexpr (kE4m3) {
#pragma unroll
                for (int k = 0; k < 2 * (D / 32); ++k) {
                  const uint32_t step = uint32_t(2 * (k % (D / 32)));
                  ptx::mma_f8_lh(tS, k_lo + step, q_lo + (k >= D / 32 ? q_block : 0u) + step, hi, idesc, k > 0 ? 1u : 0u);
                }
              } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                  const uint32_t step = uint32_t(2 * (k & 3));
                  if (k == 0) ptx::mma_ss_lh<0>(tS, k_lo, q_lo, hi, idesc);
                  else ptx::mma_ss_lh<1>(tS, k_lo + uint32_t((k >> 2) * (C::kKBlock >> 4)) + step,
                                         q_lo + uint32_t(k >> 2) * q_block + step, hi, idesc);
                }
              }
              ptx::mma_commit(s_full(wg));
              if (g == p.groups - 1) ptx::mma_commit(k_empty(st));
            }
            __syncwarp();
          }
      if (!ok && lane == 0) {
        *abort_flag = 1;
        atomicExch(w.status, kStatusWaitTimeout);
      }
      if (ptx::elect_one()) {
        ptx::mma_commit(done(me));  // arrives once every product of this warp has completed
        ptx::mbar_wait_bounded(done(me), 0, limit, nullptr);
      }
      __syncwarp();
    } else if (warp >= kWarpExp) {
      // ---------------------------------------------------------- exponentials
      const int wg = (warp - kWarpExp) >> 2, q4 = warp & 3;
      const int r = q4 * 32 + lane;  // key of the tile
      const uint32_t nl = sbase + uint32_t(C::kLse);
      bool ok = true;
      int use = 0;
      for (int c = wg; ok && c < n; c += kGroups) {
        const int u = (t0 + c) * kPerTile + (kE4m3 ? r >> 6 : 0);
        const int key = kE4m3 ? r & 63 : r;
        bool valid = u < units;
        int pos = 0;
        float a = factor;
        if (valid) {
          const ChunkDesc cd = chunks[u];
          valid = key < (cd.start_len >> 16);
          pos = (u / w.chunks_per_page) * w.ps + (cd.start_len & 0xFFFF) + key;
          if (kE4m3 && valid)
            a *= e4m3::scale_of(__ldg(w.scales + (int64_t(cd.page) * 2 * w.H + head) * w.scale_row +
                                      (cd.start_len & 0xFFFF) + key));
        }
        float sum = 0.f;
        for (int g = 0; ok && g < p.groups; ++g, ++use) {
          if (!(ok = e4m3::wait_warp(s_full(wg), use & 1, limit, abort_flag))) break;
          ptx::tc_fence_after();
          const uint32_t tS = tmem + uint32_t(wg * kBufCols) + (uint32_t(q4 * 32) << 16);
          // (columns past the last row of the pass weigh nothing)
          const int cols = min(p.group_rows, p.rows - g * p.group_rows);
          const uint32_t m = nl + uint32_t(4 * g * p.group_rows);
          if (kE4m3 && apart) sum += add_terms_apart(tS, m, m + uint32_t(C::kRowF - C::kLse), a, cols, s_free(wg));
          else sum += add_terms<false>(tS, m, 0, a, cols, s_free(wg));
        }
        if (ok && valid) {
          float* dst = w.part + (int64_t(stream) * w.H + head) * w.cap + pos;
          *dst = p.add ? *dst + sum : sum;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicExch(w.status, kStatusWaitTimeout);
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

template <int D, bool kE4m3>
cudaError_t launch(const WeightParams& w, const CUtensorMap* map, int num_sms, cudaStream_t s) {
  using C = WCfg<D, kE4m3>;
  cudaError_t e = cudaSuccess;
  WeightTcParams p{};
  p.w = w;
  p.unit_tokens = kE4m3 ? kUnitTokens : kChunkTokens;
  const int passes = (w.T + C::kRows - 1) / C::kRows;
  // enough CTAs for the SMs, no more than there are tiles
  const int tiles = (w.max_specials + kTileKeys - 1) / kTileKeys;
  p.splits = num_sms / (w.B * w.H);
  p.splits = p.splits < 1 ? 1 : p.splits > tiles ? tiles : p.splits;
  for (int i = 0; i < passes && e == cudaSuccess; ++i) {
    p.row0 = int(int64_t(w.T) * i / passes);
    p.rows = int(int64_t(w.T) * (i + 1) / passes) - p.row0;
    p.groups = (p.rows + kBufCols - 1) / kBufCols;
    p.group_rows = ((p.rows + p.groups - 1) / p.groups + kCols - 1) / kCols * kCols;
    p.groups = (p.rows + p.group_rows - 1) / p.group_rows;
    p.add = i > 0;
    e = launch_dependent(weight_tc_kernel<D, kE4m3>, dim3(unsigned(p.splits), unsigned(w.H), unsigned(w.B)),
                         dim3(kThreads), C::kLaunch, s, p, *map);
  }
  return e;
}

template <int D, bool kE4m3>
cudaError_t configure() {
  return cudaFuncSetAttribute(weight_tc_kernel<D, kE4m3>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              WCfg<D, kE4m3>::kLaunch);
}

}  // namespace

cudaError_t configure_weights_tc() {
  cudaError_t e;
  if ((e = configure<64, false>()) != cudaSuccess) return e;
  if ((e = configure<64, true>()) != cudaSuccess) return e;
  if ((e = configure<128, false>()) != cudaSuccess) return e;
  return configure<128, true>();
}

cudaError_t launch_weights_tc(const WeightParams& w, const CUtensorMap* map, bool e4m3, int num_sms, cudaStream_t s) {
  if (e4m3) return w.D == 64 ? launch<64, true>(w, map, num_sms, s) : launch<128, true>(w, map, num_sms, s);
  return w.D == 64 ? launch<64, false>(w, map, num_sms, s) : launch<128, false>(w, map, num_sms, s);
}

}  // namespace spk
