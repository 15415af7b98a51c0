// Append to an 8-bit cache: a frame's K/V rows quantised on their way into the pool,
// optionally with the 3-D rotary embedding of q and k in the same pass.
//
// For each (token, head) row x of D values: s = 2^(b - 127) the smallest power of two with
// max|x| <= 448 s, code = x / s rounded once to e4m3.  With max|x| = 1.m * 2^(E - 127) that is
// b = E - 8 + (1.m > 1.75): 448 = 1.75 * 2^8.
//
// What bounds it: the frame's rows are a megabyte or two, so the launch is a chain of latencies
// (one load, one reduction, one store per thread).  One CTA per token row, one 8-value piece
// per thread and 8 (D = 64) or 16 threads per (token, head) row: the row's maximum is three or
// four shuffles, every load and store of a row is contiguous.  Measured: 2.1 us a launch of 262
// tokens of 16 heads of 64 dims (1.6 MB), 3.9 us of 1005 (6.2 MB, 1.6 TB/s); a host call takes 3 us, the
// caller's indexing of the rows twice that (24 blocks 75 us with the rows at hand, 226 to 325 without).
#include "spk_rope.cuh"

#include <cuda_bf16.h>
#include <cuda_fp8.h>

namespace spk {
namespace {

constexpr int kThreads = 256;

// scale byte of a row whose largest finite magnitude has these fp32 bits
__device__ __forceinline__ int scale_byte(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int b = int(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(b, 0), 254);
}

// 2^(127 - b): the reciprocal of the scale (a subnormal for b = 254)
__device__ __forceinline__ float inverse_scale(int b) {
  return __uint_as_float(b < 254 ? uint32_t(254 - b) << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ const AppendParams& rows_of(const AppendParams& r) { return r; }
__device__ __forceinline__ const AppendParams& rows_of(const AppendRopeParams& r) { return r.a; }

// Unit u of a token row is 8 consecutive values: units [0, upr) are K, [upr, 2 upr) V,
// [2 upr, 3 upr) Q.
template <int D, typename Rows>
__global__ void __launch_bounds__(kThreads) append_e4m3_kernel(const __grid_constant__ AppendE4m3Params<Rows> p) {
  constexpr bool kRope = sizeof(Rows) == sizeof(AppendRopeParams);
  constexpr int kGroup = D / 8;  // threads of a (token, head) row
  __shared__ float2 cs[kRope ? kMaxRopePairs : 1];
  // launched as a programmatic dependent (see append_kernel)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const AppendParams& a = rows_of(p.r);
  const int32_t r = blockIdx.x;
  int32_t page, slot;
  if (r < a.P) {
    page = a.patch_page;
    slot = r;
  } else {
    page = a.special_page[r - a.P];
    slot = a.special_slot[r - a.P];
  }
  const int32_t upr = p.H * kGroup;
  int32_t units = 2 * upr;
  if constexpr (kRope) {
    if (p.r.q) units += upr;
  }
  const int64_t in_off = int64_t(r) * p.in_row_bytes;
  if constexpr (kRope) {
    for (int i = threadIdx.x; i < p.r.rot_pairs; i += kThreads) cs[i] = pair_cos_sin(p.r, r, i);
    __syncthreads();
  }
  // whole groups take each step together (units is a multiple of the group), so a group's
  // shuffles always find all of its lanes
  for (int32_t u = threadIdx.x; u < units; u += kThreads) {
    const int32_t t = u / upr;
    const int32_t c = u - t * upr;
    const char* src = t == 0 ? a.k : a.v;
    if constexpr (kRope) {
      if (t == 2) src = p.r.q;
    }
    src += in_off + int64_t(c) * 16;
    const uint4 raw = *reinterpret_cast<const uint4*>(src);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(w[j] << 16);
      x[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
    if constexpr (kRope) {
      const int32_t pair0 = (c % kGroup) * 4;
      if (t != 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (pair0 + j < p.r.rot_pairs) {
            const float2 v = cs[pair0 + j];
            const float x0 = x[2 * j], x1 = x[2 * j + 1];
            x[2 * j] = fmaf(x0, v.x, -x1 * v.y);
            x[2 * j + 1] = fmaf(x0, v.y, x1 * v.x);
          }
        }
      }
      if (t == 2) {
        *reinterpret_cast<uint4*>(p.r.q_out + in_off + int64_t(c) * 16) = make_uint4(
            pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
        continue;
      }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t m = __float_as_uint(x[j]) & 0x7FFFFFFFu;
      amax = max(amax, m < 0x7F800000u ? m : 0u);  // finite values only
    }
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t mask = (kGroup == 16 ? 0xFFFFu : 0xFFu) << (lane & ~uint32_t(kGroup - 1));
#pragma unroll
    for (int o = kGroup / 2; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(mask, amax, o));
    const int b = scale_byte(amax);
    const float inv = inverse_scale(b);
    uint32_t code[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t lo =
          __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j] * inv, x[4 * j + 1] * inv), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi =
          __nv_cvt_float2_to_fp8x2(make_float2(x[4 * j + 2] * inv, x[4 * j + 3] * inv), __NV_SATFINITE, __NV_E4M3);
      code[j] = lo | (hi << 16);
    }
    char* dst = a.pool + int64_t(page) * a.page_bytes + t * a.half_bytes + int64_t(slot) * a.row_bytes + int64_t(c) * 8;
    *reinterpret_cast<uint2*>(dst) = make_uint2(code[0], code[1]);
    if ((lane & (kGroup - 1)) == 0)
      p.scales[((int64_t(page) * 2 + t) * p.H + c / kGroup) * p.scale_row + slot] = uint8_t(b);
  }
}

template <typename Rows>
cudaError_t launch(const AppendE4m3Params<Rows>& p, int tokens, int head_dim, cudaStream_t s) {
  const dim3 grid{unsigned(tokens)}, block(kThreads);
  return head_dim == 64 ? launch_dependent(append_e4m3_kernel<64, Rows>, grid, block, 0, s, p)
                        : launch_dependent(append_e4m3_kernel<128, Rows>, grid, block, 0, s, p);
}

}  // namespace

cudaError_t launch_append_e4m3(const AppendE4m3Params<AppendParams>& p, int head_dim, cudaStream_t s) {
  return launch(p, p.r.T, head_dim, s);
}

cudaError_t launch_append_e4m3(const AppendE4m3Params<AppendRopeParams>& p, int head_dim, cudaStream_t s) {
  return launch(p, p.r.a.T, head_dim, s);
}

}  // namespace spk
