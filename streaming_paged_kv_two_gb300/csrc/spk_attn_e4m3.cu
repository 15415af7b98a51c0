// Attention over an 8-bit cache: softmax(q k^T / sqrt(D)) v with k = 2^(b_k - 127) c_k and
// v = 2^(b_v - 127) c_v, c the stored e4m3 codes and b one scale byte per (token, head).
// Calls with more query rows than kRowsMost go to the tensor-core kernel (spk_attn_e4m3_tc.cu).
//
// Rows kernel (attention_e4m3_rows_kernel): 8 or 16 query rows per CTA.  With few rows the call is
// a stream through K and V, 2 (D + 1) bytes per key and head, so everything is arranged around
// keeping loads in flight: one producer warp fills a ring of 64-key stages (codes by tensor-map
// copies, the two 64-byte runs of scale bytes by plain bulk copies), two CTAs fit an SM, and
// pairs of consumer warps take the stages in turn, 32 keys a warp, with no barrier among them: every
// warp is a running softmax of its own (maximum, sum, output), joined once at the end.  A warp widens
// its codes to fp16 in registers (exact) and multiplies with fp16 warp products, fp32 sums:
//   S = Q K^T: Q is scaled by a power of two per row so that its largest value is in [1, 2)
//   (exact in fp16 but for values below 2^-24 of the row's largest); a key's scale multiplies
//   its scores in fp32.
//   O += P' V: P' = p 2^(b_v - R) 2^12 in fp16, p <= 1 the softmax weight against the running
//   maximum and R the running largest scale byte.  The scale of V thus enters once, exactly,
//   and 2^12 puts P' high in fp16's range: it is rounded by 2^-11 of itself down to 2^-14 (2^-26 of
//   the largest there can be), below that by up to 2^-25, which times a code of at most 448 is 2^-36
//   of the largest |v| a key.  Row sums are those of the fp32 p.
// The order of a warp product's contraction is free, so each thread takes 16 consecutive dims
// of a key (one 16-byte shared-memory load) for Q K^T, and 8 or 16 consecutive dims of its four
// keys for P V; the swizzle of the copies keeps both free of bank conflicts (D = 128's K: two-way).
// Measured: one row over 78,432 keys of 16 heads of 64 dims (163 MB) 30.5 us in the kernel, 5.3 TB/s
// (0.79 of a plain copy, start included), 34.5 us with the merge; more or larger CTAs an SM, or more
// consumer warps, change it by less than 2 %.  16 rows 42 us: twice the products and exponentials.
#include "ptx_sm100.cuh"
#include "spk_e4m3.cuh"
#include "spk_internal.h"

#include <cuda_bf16.h>

namespace spk {
namespace {

__device__ __forceinline__ void signal_abort(int32_t* status, volatile int* abort_flag) {
  *abort_flag = 1;
  atomicExch(status, kStatusWaitTimeout);
}

// ------------------------------------------------------------------ rows kernel

constexpr float kPBias = 4096.f;                     // 2^12 (see above)
constexpr int kPBiasLog2 = 12;

template <int D, int kRows>
struct RowsCfg {
  static constexpr int kTile = kUnitTokens * D;      // codes of one K or V stage
  static constexpr int kScales = 2 * kUnitTokens;    // K then V scale bytes
  // about 200 KB in flight per SM: two CTAs, but one for 16 rows of 128 dims (whose registers
  // would not fit twice; ptxas spills 12 to 20 bytes a thread, none for 8 rows of 64 dims)
  static constexpr int kCtas = D == 128 && kRows == 16 ? 1 : 2;
  static constexpr int kStages = D == 128 && kCtas == 2 ? 6 : 12;
  static constexpr int kPairs = kStages == 6 ? 3 : 4;  // of consumer warps, which take the stages in turn
  static constexpr int kConsumers = 2 * kPairs;
  static constexpr int kThreads = 32 * (kConsumers + 1);
  // a pair that came to a stage every second time around could not tell its barrier's phases apart
  static_assert(kStages % kPairs == 0, "every stage belongs to one pair");
  static constexpr int kScaleOff = kStages * 2 * kTile;
  static constexpr int kBars = kScaleOff + kStages * kScales;
  static constexpr int kBytes = kBars + 2 * kStages * 8 + 16;
  static constexpr int kLaunch = kBytes + 1024;      // slack for 1024-byte alignment
  // the join of the warps reuses the ring: fp32 O [consumers][rows][D], then m, l [consumers][rows]
  // and R [consumers]
  static_assert(kConsumers * kRows * (D + 2) * 4 + kConsumers * 4 <= kScaleOff, "join fits the ring");
  static_assert(kLaunch * kCtas <= 227 * 1024, "shared memory per SM");
};

// 16-byte piece c of row r in a swizzled tile of D-byte rows
template <int D>
__device__ __forceinline__ uint32_t piece(int r, int c) {
  return D == 64 ? uint32_t(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)) : uint32_t(r * 128 + ((c ^ (r & 7)) << 4));
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// A thread's part of a query row, dims 64 h + 16 t + [0, 16) as words w[4 h + s][2] of two fp16,
// scaled by 2^(127 - e), e the fp32 exponent of the row's largest value (over the four lanes that
// share it).  Returns what turns a product back into log2 units; rows past the last are zero.
template <int D>
__device__ __forceinline__ float load_row(const AttnParams& p, int stream, int row, int head, int t,
                                          uint32_t (&f)[D / 16][2]) {
  constexpr int kHalves = D / 64;
  uint32_t w[kHalves][8];
  uint32_t amax = 0;
#pragma unroll
  for (int h = 0; h < kHalves; ++h) {
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    if (row < p.T) {
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const __nv_bfloat16*>(p.q) + ((int64_t(stream) * p.T + row) * p.H + head) * D + 64 * h + 16 * t);
      a = __ldg(src);
      b = __ldg(src + 1);
    }
    w[h][0] = a.x, w[h][1] = a.y, w[h][2] = a.z, w[h][3] = a.w;
    w[h][4] = b.x, w[h][5] = b.y, w[h][6] = b.z, w[h][7] = b.w;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, max((w[h][j] << 16) & 0x7FFFFFFFu, w[h][j] & 0x7FFF0000u));
  }
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const uint32_t e = min(max(amax >> 23, 1u), 253u);
  const float scale = __uint_as_float((254u - e) << 23);
#pragma unroll
  for (int h = 0; h < kHalves; ++h)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      f[4 * h + j / 2][j % 2] =
          e4m3::pack_f16(__uint_as_float(w[h][j] << 16) * scale, __uint_as_float(w[h][j] & 0xFFFF0000u) * scale);
  return p.scale_log2 * __uint_as_float(e << 23);
}

// Codes of V's keys r0 + {0, 1, 8, 9}, dims (D / 8) g + [0, D / 8).  Keys from len on are zeroed
// where the unit is ragged: their slots may hold anything.
template <int D>
__device__ __forceinline__ void load_v(uint32_t sv, int r0, int g, int len, bool ragged, uint32_t (&w)[4][D / 32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int r = r0 + (q & 1) + 8 * (q >> 1);
    if constexpr (D == 64) {
      const uint2 v = lds64(sv + piece<D>(r, g >> 1) + 8 * (g & 1));
      w[q][0] = v.x, w[q][1] = v.y;
    } else {
      const uint4 v = lds128(sv + piece<D>(r, g));
      w[q][0] = v.x, w[q][1] = v.y, w[q][2] = v.z, w[q][3] = v.w;
    }
    if (ragged && r >= len) {
#pragma unroll
      for (int z = 0; z < D / 32; ++z) w[q][z] = 0;
    }
  }
}

// A warp's running softmax over 16 query rows, the rows in the products' M: rows g and g + 8 of
// the thread, keys and dims in N.
template <int D, int kRows>
struct RowsState {
  static constexpr int kHalves = D / 64;
  uint32_t qf[4 * kHalves][4];
  float rf[2], m[2], l[2], o[D / 8][4];
  int R;  // largest V scale byte met

  __device__ __forceinline__ void init() {
    R = 0;
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) m[hr] = -INFINITY, l[hr] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // Fragments of the thread's rows, dims 64 h + 16 t + [0, 16)
  __device__ __forceinline__ void load_q(const AttnParams& p, int stream, int row0, int head, int g, int t) {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      uint32_t w[4 * kHalves][2];
      rf[hr] = load_row<D>(p, stream, row0 + g + 8 * hr, head, t, w);
#pragma unroll
      for (int j = 0; j < 4 * kHalves; ++j) qf[j][hr] = w[j][0], qf[j][2 + hr] = w[j][1];
    }
  }

  __device__ __forceinline__ void step(uint32_t sk, uint32_t sv, uint32_t sc, int k0, int len, int g, int t) {
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
          const uint4 v = lds128(sk + piece<D>(k0 + 8 * nt + g, 4 * h + t));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            e4m3::mma_16816(s[nt], qf[4 * h + q], e4m3::widen_lo(w[q]), e4m3::widen_hi(w[q]));
        }
      }
      // scores in log2 units; keys k0 + 8 nt + 2 t + {0, 1}
      float mx[2] = {-INFINITY, -INFINITY};
      uint32_t vb[4];
      int r_new = R;
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        const int key = k0 + 8 * nt + 2 * t;
        const uint32_t kb = lds_u16(sc + key);
        vb[nt] = lds_u16(sc + kUnitTokens + key);
        const float ks[2] = {e4m3::scale_of(kb & 255), e4m3::scale_of(kb >> 8)};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool in = key + j < len;
#pragma unroll
          for (int hr = 0; hr < 2; ++hr) {
            const float v = in ? s[nt][2 * hr + j] * rf[hr] * ks[j] : -INFINITY;
            s[nt][2 * hr + j] = v;
            mx[hr] = fmaxf(mx[hr], v);
          }
          if (in) r_new = max(r_new, int((vb[nt] >> (8 * j)) & 255));
        }
      }
      r_new = __reduce_max_sync(0xffffffffu, r_new);
      float corr[2];
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 1));
        mx[hr] = fmaxf(mx[hr], __shfl_xor_sync(0xffffffffu, mx[hr], 2));
        const float m_new = fmaxf(m[hr], mx[hr]);
        corr[hr] = m_new == m[hr] ? 1.f : ptx::ex2(m[hr] - m_new);  // 0 while m is -inf
        m[hr] = m_new;
        l[hr] *= corr[hr];
      }
      const float rdown = r_new == R ? 1.f : e4m3::scale_of(max(127 + R - r_new, 0));
      if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f || r_new != R)) {
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= corr[0] * rdown;
          o[j][1] *= corr[0] * rdown;
          o[j][2] *= corr[1] * rdown;
          o[j][3] *= corr[1] * rdown;
        }
      }
      R = r_new;
      uint32_t pa[2][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float vs[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e = int((vb[nt] >> (8 * j)) & 255) - R + 127 + kPBiasLog2;
          vs[j] = e > 0 ? __uint_as_float(uint32_t(min(e, 254)) << 23) : 0.f;
        }
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const float p0 = ptx::ex2(s[nt][2 * hr] - m[hr]), p1 = ptx::ex2(s[nt][2 * hr + 1] - m[hr]);
          l[hr] += p0 + p1;
          pa[nt >> 1][2 * (nt & 1) + hr] = e4m3::pack_f16(p0 * vs[0], p1 * vs[1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        constexpr int kWords = D / 32;
        uint32_t w[4][kWords];
        load_v<D>(sv, k0 + 16 * j + 2 * t, g, len, len < k0 + 32, w);
#pragma unroll
        for (int z = 0; z < kWords; ++z) {
          const uint32_t b0a = __byte_perm(w[0][z], w[1][z], 0x5140), b0b = __byte_perm(w[0][z], w[1][z], 0x7362);
          const uint32_t b1a = __byte_perm(w[2][z], w[3][z], 0x5140), b1b = __byte_perm(w[2][z], w[3][z], 0x7362);
          e4m3::mma_16816(o[4 * z], pa[j], e4m3::widen_lo(b0a), e4m3::widen_lo(b1a));
          e4m3::mma_16816(o[4 * z + 1], pa[j], e4m3::widen_hi(b0a), e4m3::widen_hi(b1a));
          e4m3::mma_16816(o[4 * z + 2], pa[j], e4m3::widen_lo(b0b), e4m3::widen_lo(b1b));
          e4m3::mma_16816(o[4 * z + 3], pa[j], e4m3::widen_hi(b0b), e4m3::widen_hi(b1b));
        }
      }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
      l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
    }
  }

  // Tile i of o holds dims (D / 8) n + i, n the column of the product.
  __device__ __forceinline__ void put(float* jo, float* jm, float* jl, int g, int t) const {
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float* dst = jo + (g + 8 * hr) * D + (D / 8) * 2 * t;
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < D / 8; i += 4)
          *reinterpret_cast<float4*>(dst + j * (D / 8) + i) =
              make_float4(o[i][2 * hr + j], o[i + 1][2 * hr + j], o[i + 2][2 * hr + j], o[i + 3][2 * hr + j]);
      if (t == 0) {
        jm[g + 8 * hr] = m[hr];
        jl[g + 8 * hr] = l[hr];
      }
    }
  }
};

// Up to 8 query rows: keys and dims in the products' M, the rows in N (rows 2 t and 2 t + 1 of the
// thread).  Half the products and half the exponentials of the 16-row form; the weights reach
// the second product's layout through a transpose of 8 x 8 halves among the lanes.
template <int D>
struct RowsState<D, 8> {
  static constexpr int kHalves = D / 64;
  uint32_t qf[4 * kHalves][2];
  float rf[2], m[2], l[2], o[D / 16][4];
  int R;  // largest V scale byte met

  __device__ __forceinline__ void init() {
    R = 0;
#pragma unroll
    for (int r = 0; r < 2; ++r) m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  __device__ __forceinline__ void load_q(const AttnParams& p, int stream, int row0, int head, int g, int t) {
    const float f = load_row<D>(p, stream, row0 + g, head, t, qf);
    rf[0] = __shfl_sync(0xffffffffu, f, 8 * t);
    rf[1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);
  }

  __device__ __forceinline__ void step(uint32_t sk, uint32_t sv, uint32_t sc, int k0, int len, int g, int t) {
    float s[2][4];  // [16 keys][2 kk + r]: key k0 + 16 mt + 8 kk + g, row 2 t + r
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      s[mt][0] = s[mt][1] = s[mt][2] = s[mt][3] = 0.f;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint4 a = lds128(sk + piece<D>(k0 + 16 * mt + g, 4 * h + t));
        const uint4 b = lds128(sk + piece<D>(k0 + 16 * mt + 8 + g, 4 * h + t));
        const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t f[4] = {e4m3::widen_lo(wa[q]), e4m3::widen_lo(wb[q]), e4m3::widen_hi(wa[q]),
                                 e4m3::widen_hi(wb[q])};
          e4m3::mma_16816(s[mt], f, qf[4 * h + q][0], qf[4 * h + q][1]);
        }
      }
    }
    // scores in log2 units
    float mx[2] = {-INFINITY, -INFINITY};
    int vb[2][2];
    int r_new = R;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int key = k0 + 16 * mt + 8 * kk + g;
        const float ks = e4m3::scale_of(int(lds_u8(sc + key)));
        vb[mt][kk] = int(lds_u8(sc + kUnitTokens + key));
        const bool in = key < len;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float v = in ? s[mt][2 * kk + r] * rf[r] * ks : -INFINITY;
          s[mt][2 * kk + r] = v;
          mx[r] = fmaxf(mx[r], v);
        }
        if (in) r_new = max(r_new, vb[mt][kk]);
      }
    r_new = __reduce_max_sync(0xffffffffu, r_new);
    float corr[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], d));
      const float m_new = fmaxf(m[r], mx[r]);
      corr[r] = m_new == m[r] ? 1.f : ptx::ex2(m[r] - m_new);  // 0 while m is -inf
      m[r] = m_new;
      l[r] *= corr[r];
    }
    if (__any_sync(0xffffffffu, corr[0] != 1.f || corr[1] != 1.f || r_new != R)) {
      const float rdown = r_new == R ? 1.f : e4m3::scale_of(max(127 + R - r_new, 0));
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {
        o[j][0] *= corr[0] * rdown;
        o[j][1] *= corr[1] * rdown;
        o[j][2] *= corr[0] * rdown;
        o[j][3] *= corr[1] * rdown;
      }
    }
    R = r_new;
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      uint32_t pb[2];
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        const int e = vb[mt][kk] - R + 127 + kPBiasLog2;
        const float vs = e > 0 ? __uint_as_float(uint32_t(min(e, 254)) << 23) : 0.f;
        const float p0 = ptx::ex2(s[mt][2 * kk] - m[0]), p1 = ptx::ex2(s[mt][2 * kk + 1] - m[1]);
        l[0] += p0;
        l[1] += p1;
        pb[kk] = e4m3::transpose_8x8(e4m3::pack_f16(p0 * vs, p1 * vs));
      }
      uint32_t w[4][D / 32];
      load_v<D>(sv, k0 + 16 * mt + 2 * t, g, len, len < k0 + 32, w);
#pragma unroll
      for (int z = 0; z < D / 32; ++z) {
        const uint32_t b0a = __byte_perm(w[0][z], w[1][z], 0x5140), b0b = __byte_perm(w[0][z], w[1][z], 0x7362);
        const uint32_t b1a = __byte_perm(w[2][z], w[3][z], 0x5140), b1b = __byte_perm(w[2][z], w[3][z], 0x7362);
        const uint32_t fa[4] = {e4m3::widen_lo(b0a), e4m3::widen_hi(b0a), e4m3::widen_lo(b1a), e4m3::widen_hi(b1a)};
        const uint32_t fb[4] = {e4m3::widen_lo(b0b), e4m3::widen_hi(b0b), e4m3::widen_lo(b1b), e4m3::widen_hi(b1b)};
        e4m3::mma_16816(o[2 * z], fa, pb[0], pb[1]);
        e4m3::mma_16816(o[2 * z + 1], fb, pb[0], pb[1]);
      }
    }
  }

  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int d = 4; d < 32; d *= 2) l[r] += __shfl_xor_sync(0xffffffffu, l[r], d);
  }

  // o[2 z] and o[2 z + 1] hold dims (D / 8) g + 4 z + [0, 4), two each, of rows 2 t and 2 t + 1.
  __device__ __forceinline__ void put(float* jo, float* jm, float* jl, int g, int t) const {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int z = 0; z < D / 32; ++z)
        *reinterpret_cast<float4*>(jo + (2 * t + r) * D + (D / 8) * g + 4 * z) =
            make_float4(o[2 * z][r], o[2 * z][2 + r], o[2 * z + 1][r], o[2 * z + 1][2 + r]);
      if (g == 0) {
        jm[2 * t + r] = m[r];
        jl[2 * t + r] = l[r];
      }
    }
  }
};

template <int D, int kRows>
__global__ void __launch_bounds__((RowsCfg<D, kRows>::kThreads), (RowsCfg<D, kRows>::kCtas))
    attention_e4m3_rows_kernel(const AttnParams p, const __grid_constant__ CUtensorMap kv_map) {
  using C = RowsCfg<D, kRows>;
  constexpr int S = C::kStages;
  constexpr int kRowsConsumers = C::kConsumers;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = ptx::smem_u32(smem);
  auto full_bar = [&](int st) { return sbase + uint32_t(C::kBars + 8 * st); };
  auto empty_bar = [&](int st) { return sbase + uint32_t(C::kBars + 8 * (S + st)); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBars + 16 * S);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_tiles = (p.T + kRows - 1) / kRows;
  int x = blockIdx.x;
  const int tile = x % row_tiles;
  x /= row_tiles;
  const int head = x % p.H;
  const int split = x / p.H;
  const WorkDesc work = p.works[split];
  const int c0 = work.chunk_begin, n = work.chunk_end - work.chunk_begin;
  const long long limit = p.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full_bar(i), 1);
      ptx::mbar_init(empty_bar(i), 2);
    }
    *abort_flag = 0;
    ptx::fence_mbar_init();
    ptx::fence_proxy_async_smem();
  }
  __syncthreads();
  // launched as a programmatic dependent (see attention_tc_kernel)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int g = lane >> 2, t = lane & 3;
  RowsState<D, kRows> z;
  z.init();

  if (warp == kRowsConsumers) {
    // ---------------------------------------------------------------- producer
    if (lane == 0) ptx::prefetch_tmap(&kv_map);
    e4m3::ChunkReader reader(p.chunks + c0, n, lane);
    int issued = 0;
    for (; issued < n; ++issued) {
      const int st = issued % S;
      const ChunkDesc cd = reader.get(issued);
      if (!e4m3::wait_warp(empty_bar(st), ((issued / S) & 1) ^ 1, limit, abort_flag)) {
        if (lane == 0) signal_abort(p.status, abort_flag);
        break;
      }
      if (lane == 0) {
        const int start = cd.start_len & 0xFFFF;
        const uint32_t kv = sbase + uint32_t(st * 2 * C::kTile), sc = sbase + uint32_t(C::kScaleOff + st * C::kScales);
        const uint8_t* scales = p.scales + (int64_t(cd.page) * 2 * p.H + head) * p.scale_row + start;
        ptx::mbar_arrive_expect_tx(full_bar(st), 2 * C::kTile + C::kScales);
        ptx::tma_load_4d(kv, &kv_map, 0, head, start, 2 * cd.page, full_bar(st));
        ptx::tma_load_4d(kv + C::kTile, &kv_map, 0, head, start, 2 * cd.page + 1, full_bar(st));
        ptx::bulk_load(sc, scales, kUnitTokens, full_bar(st));
        ptx::bulk_load(sc + kUnitTokens, scales + int64_t(p.H) * p.scale_row, kUnitTokens, full_bar(st));
      }
    }
    if (lane == 0) {
      // copies must land before the ring is reused or the CTA exits
      for (int i = issued > S ? issued - S : 0; i < issued; ++i)
        ptx::mbar_wait_bounded(full_bar(i % S), (i / S) & 1, limit, nullptr);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- consumers
    z.load_q(p, work.stream, tile * kRows, head, g, t);
    const int k0 = 32 * (warp & 1);  // this warp's keys [k0, k0 + 32) of its stages
    bool ok = true;
    for (int i = warp >> 1; i < n; i += kRowsConsumers / 2) {
      const int st = i % S;
      const int len = __ldg(&p.chunks[c0 + i].start_len) >> 16;
      if (!(ok = e4m3::wait_warp(full_bar(st), (i / S) & 1, limit, abort_flag))) break;
      if (k0 < len) {
        const uint32_t sk = sbase + uint32_t(st * 2 * C::kTile), sv = sk + C::kTile;
        const uint32_t sc = sbase + uint32_t(C::kScaleOff + st * C::kScales);
        z.step(sk, sv, sc, k0, len, g, t);
      }
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(empty_bar(st));
    }
    if (!ok) signal_abort(p.status, abort_flag);
    z.finish();
  }

  // ---------------------------------------------------------------- join of the warps
  __syncthreads();  // every stage has been consumed (or the wait gave up: no output then)
  if (*abort_flag) return;
  float* jo = reinterpret_cast<float*>(smem);
  float* jm = jo + kRowsConsumers * kRows * D;
  float* jl = jm + kRowsConsumers * kRows;
  int* jr = reinterpret_cast<int*>(jl + kRowsConsumers * kRows);
  if (warp < kRowsConsumers) {
    z.put(jo + warp * kRows * D, jm + warp * kRows, jl + warp * kRows, g, t);
    if (lane == 0) jr[warp] = z.R;
  }
  __syncthreads();
  for (int u = threadIdx.x; u < kRows * (D / 4); u += C::kThreads) {
    // rows fastest: a warp's partial stores are runs of consecutive rows
    const int r = u % kRows, c4 = u / kRows;
    const int row = tile * kRows + r;
    if (row >= p.T) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kRowsConsumers; ++w) M = fmaxf(M, jm[w * kRows + r]);
    float L = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kRowsConsumers; ++w) {
      const float mw = jm[w * kRows + r];
      const float f = mw == M ? 1.f : ptx::ex2(mw - M);
      L = fmaf(f, jl[w * kRows + r], L);
      const float fo = f * (e4m3::scale_of(jr[w]) * (1.f / kPBias));
      const float4 v = *reinterpret_cast<const float4*>(jo + (w * kRows + r) * D + 4 * c4);
      acc.x = fmaf(fo, v.x, acc.x);
      acc.y = fmaf(fo, v.y, acc.y);
      acc.z = fmaf(fo, v.z, acc.z);
      acc.w = fmaf(fo, v.w, acc.w);
    }
    const float inv = 1.f / L;
    acc.x *= inv;
    acc.y *= inv;
    acc.z *= inv;
    acc.w *= inv;
    if (work.nsplit == 1 && !p.force_part) {
      const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x, acc.y), b = __floats2bfloat162_rn(acc.z, acc.w);
      uint2 pk;
      pk.x = *reinterpret_cast<const uint32_t*>(&a);
      pk.y = *reinterpret_cast<const uint32_t*>(&b);
      *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) +
                                ((int64_t(work.stream) * p.T + row) * p.H + head) * D + 4 * c4) = pk;
      if (p.lse != nullptr && c4 == 0)
        p.lse[(int64_t(work.stream) * p.T + row) * p.H + head] = e4m3::kLn2 * (M + log2f(L));
    } else {
      *reinterpret_cast<float4*>(p.part_o + part_o_offset<D>(split, head, row, 4 * c4, p.H, p.T)) = acc;
      if (c4 == 0) p.part_lse[(int64_t(split) * p.H + head) * p.T + row] = M + log2f(L);
    }
  }
}

template <int D, int kRows>
cudaError_t launch_rows(const AttnParams& p, const CUtensorMap* map, cudaStream_t s) {
  const int64_t grid = int64_t(p.num_splits) * p.H * ((p.T + kRows - 1) / kRows);
  if (grid <= 0 || grid > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_dependent(attention_e4m3_rows_kernel<D, kRows>, dim3(unsigned(grid)),
                          dim3(RowsCfg<D, kRows>::kThreads),
                          RowsCfg<D, kRows>::kLaunch, s, p, *map);
}

template <int D, int kRows>
cudaError_t configure_rows() {
  return cudaFuncSetAttribute(attention_e4m3_rows_kernel<D, kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              RowsCfg<D, kRows>::kLaunch);
}

}  // namespace

// Query rows up to which the 8-row tile and the rows kernel at all serve a call.  A tile of 16 rows is a
// pass of its own over K and V (by way of L2 for the second), the many-row kernel pays for 128 rows
// whatever their number.  Measured with a cold L2, us, rows kernel / many-row kernel, over 78,432 keys
// of 16 heads of 64 dims: 1 row 47 / 78, 16 rows 53 / 90, 32 rows 84 / 92, 48 rows 119 / 92; over 4 x
// 63,792 keys of 8 heads of 128 dims: 16 rows 121 / 205, 32 rows 202 / 207, 48 rows 287 / 209.  Up to 8
// rows the tile of 8 takes 47 where that of 16 takes 53 (D = 128: 107 and 119).
constexpr int kRowsOne = 8, kRowsMost = kE4m3RowsMost;

cudaError_t configure_attention_e4m3() {
  for (const cudaError_t e : {configure_rows<64, 8>(), configure_rows<64, 16>(), configure_rows<128, 8>(),
                              configure_rows<128, 16>()})
    if (e != cudaSuccess) return e;
  return configure_attention_e4m3_tc();
}

cudaError_t launch_attention_e4m3(const AttnParams& p, const CUtensorMap* kv_map, cudaStream_t s) {
  if (p.T > kRowsMost) return launch_attention_e4m3_tc(p, kv_map, s);
  if (p.T > kRowsOne) return p.D == 64 ? launch_rows<64, 16>(p, kv_map, s) : launch_rows<128, 16>(p, kv_map, s);
  return p.D == 64 ? launch_rows<64, 8>(p, kv_map, s) : launch_rows<128, 8>(p, kv_map, s);
}

int e4m3_row_tiles(int T, int head_dim) {
  if (T > kRowsMost) return attention_bf16_tiles(T, head_dim).ngroups;
  return T > kRowsOne ? (T + 15) / 16 : 1;
}

// The merge kernel, 3.6 us, in units of 64 keys.  Measured, us, without / with: 18 rows over 96 keys in
// pages of 16 8.1 / 7.1, one row over 268 keys 5.8 / 4.1, over 536 6.3 / 5.5; for the many-row kernel
// 8 instead of 4 takes 262 rows over 524 keys from 14.4 to 16.9.
double e4m3_merge_charge(int T) { return T > kRowsMost ? 4.0 : 8.0; }

int e4m3_ctas_per_sm(int T, int head_dim) {
  if (T > kRowsMost) return 1;
  if (T > kRowsOne) return head_dim == 64 ? RowsCfg<64, 16>::kCtas : RowsCfg<128, 16>::kCtas;
  return head_dim == 64 ? RowsCfg<64, 8>::kCtas : RowsCfg<128, 8>::kCtas;
}

}  // namespace spk
