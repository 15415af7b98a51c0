// The special stream held at a budget: records of its tokens, the attention weight each one
// receives, and the eviction of the tokens of least weight.
#include <cooperative_groups.h>

#include "spk_internal.h"

namespace spk {
namespace {

// ------------------------------------------------------------------ records
__global__ void track_kernel(const TrackParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < p.count) {
    p.weights[i] = 0.f;
    p.ids[i] = p.first_id + i;
  }
}

// ------------------------------------------------------------------ accumulated weights
// w_j += sum over heads and query rows of exp(q k_j / sqrt(D) - lse): a second pass over K
// alone, with the rows' log-sum-exps known.  The heads' sums go to `part` (spk_weights_tc.cu, or
// the fp32 kernel here) and are added, in head order, by weight_sum_kernel, so no result depends
// on the order of execution.
// fp32 caches: CUDA-core arithmetic as in attention_f32_kernel.  One CTA takes 64 special keys of
// one head and walks the query rows in tiles of 64; a key's terms are added in registers and, over
// the 16 threads of a row group, in a fixed order.
constexpr int kWKeys = 64;
constexpr int kWRows = 64;
constexpr int kWThreads = 256;

template <int D>
struct WeightCfg {
  static constexpr int kLd = D + 4;  // floats per shared-memory row
  static constexpr int kBytes = ((kWKeys + kWRows) * kLd + kWRows + 16 * kWKeys) * 4;
};

// Page and slot of the special token at position pos.
__device__ __forceinline__ void special_slot(const WeightParams& p, const StreamDesc& sd, int pos, int& page, int& slot) {
  const int ord = pos / p.ps;
  slot = pos - ord * p.ps;
  page = p.chunks[sd.special_chunk + ord * p.chunks_per_page].page;
}

template <int D>
__global__ void __launch_bounds__(kWThreads) weight_f32_kernel(const WeightParams p) {
  using C = WeightCfg<D>;
  extern __shared__ float4 w_smem4[];
  float* Ks = reinterpret_cast<float*>(w_smem4);
  float* Qs = Ks + kWKeys * C::kLd;
  float* Ls = Qs + kWRows * C::kLd;
  float* Xs = Ls + kWRows;  // [16][64] partial sums
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int head = blockIdx.y, stream = blockIdx.z;
  const StreamDesc sd = p.streams[stream];
  const int key0 = blockIdx.x * kWKeys;
  if (key0 >= sd.specials) return;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  for (int i = tid; i < kWKeys * (D / 4); i += kWThreads) {
    const int key = i / (D / 4), d = 4 * (i % (D / 4));
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (key0 + key < sd.specials) {
      int page, slot;
      special_slot(p, sd, key0 + key, page, slot);
      v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.pool) +
                                                ((int64_t(page) * 2 * p.ps + slot) * p.H + head) * D + d));
    }
    *reinterpret_cast<float4*>(Ks + key * C::kLd + d) = v;
  }
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r0 = 0; r0 < p.T; r0 += kWRows) {
    __syncthreads();
    for (int i = tid; i < kWRows * (D / 4); i += kWThreads) {
      const int r = i / (D / 4), d = 4 * (i % (D / 4));
      // (past the last row: that row again, with an lse of +inf.  Zeros would turn an infinite key's
      // score into a NaN that no row has.)
      const int64_t at = ((int64_t(stream) * p.T + min(r0 + r, p.T - 1)) * p.H + head) * D + d;
      const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p.q) + at));
      *reinterpret_cast<float4*>(Qs + r * C::kLd + d) = v;
    }
    if (tid < kWRows)  // rows past the last get +inf: weight 0
      Ls[tid] = r0 + tid < p.T ? p.lse[(int64_t(stream) * p.T + r0 + tid) * p.H + head] * 1.4426950408889634f : INFINITY;
    __syncthreads();
    float s[4][4];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[r][j] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 q4[4], k4[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) q4[r] = *reinterpret_cast<const float4*>(Qs + (4 * ty + r) * C::kLd + d);
#pragma unroll
      for (int j = 0; j < 4; ++j) k4[j] = *reinterpret_cast<const float4*>(Ks + (tx + 16 * j) * C::kLd + d);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[r][j] = fmaf(q4[r].x, k4[j].x, s[r][j]);
          s[r][j] = fmaf(q4[r].y, k4[j].y, s[r][j]);
          s[r][j] = fmaf(q4[r].z, k4[j].z, s[r][j]);
          s[r][j] = fmaf(q4[r].w, k4[j].w, s[r][j]);
        }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float lse = Ls[4 * ty + r];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] += exp2f(fmaf(s[r][j], p.scale_log2, -lse));
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) Xs[ty * kWKeys + tx + 16 * j] = w[j];
  __syncthreads();
  if (tid < kWKeys && key0 + tid < sd.specials) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += Xs[i * kWKeys + tid];
    p.part[(int64_t(stream) * p.H + head) * p.cap + key0 + tid] = sum;
  }
}

// weights[s][j] += sum over heads, in head order.  Nothing is added where a wait of this call (or of
// an earlier one whose report has not been read) gave up: `part` is then incomplete, and the weights
// are a running total that could not be put right again.
__global__ void __launch_bounds__(256) weight_sum_kernel(const WeightParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int stream = blockIdx.y;
  const int j = blockIdx.x * 256 + threadIdx.x;
  if (j >= p.streams[stream].specials || *p.status == kStatusWaitTimeout) return;
  const float* src = p.part + int64_t(stream) * p.H * p.cap + j;
  float sum = 0.f;
  for (int h = 0; h < p.H; ++h) sum += src[int64_t(h) * p.cap];
  p.weights[int64_t(stream) * p.cap + j] += sum;
}

// ------------------------------------------------------------------ eviction: the choice
// The r = n - keep tokens of least (weight, position) among the tokens that are not recent: a
// radix select of the r-th smallest 32-bit key (digits of 11, 11 and 10 bits of the weights), then
// ordered counts that give the vacated positions below `keep` and the survivors at or past it,
// both ascending.  What bounds it are the steps themselves (three digits, two ordered counts, each
// with its barriers), so they are few, the digits are found by a prefix sum over the bins, and a
// long record is split over a cluster whose CTAs read one another's counts.
// Measured, us, one CTA / a cluster of 8: 1,264 tokens 9.9 / 15.3, 4,864 14.1 / 16.8, 9,664 20.1 /
// 17.2, 30,064 113 / 19.1, 96,064 429 / 29.6; hence kSelOneCta.
constexpr int kSelThreads = 1024;
constexpr int kSelBins = 2048;
constexpr int kSelOneCta = 8192;
constexpr uint32_t kProtected = 0xFFFFFFFFu;

// Order-preserving key of a weight; a NaN sorts after every number, recent tokens last of all.
__device__ __forceinline__ uint32_t weight_key(float w, int id, int first_recent) {
  if (int(uint32_t(id) - uint32_t(first_recent)) >= 0) return kProtected;  // (arrival numbers wrap)
  if (w != w) return kProtected - 1;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);  // -0 and 0 are equal
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive prefix of v over the block and its total, through shared memory xs[32] and a
// following barrier pair.
__device__ __forceinline__ int block_exclusive(int v, int* xs, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) xs[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    int s = xs[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    xs[lane] = s;
  }
  __syncthreads();
  total = xs[31];
  const int base = warp ? xs[warp - 1] : 0;
  __syncthreads();
  return base + inc - v;
}

// What a CTA shows the others of its cluster.
struct SelectShared {
  int hist[3][kSelBins];  // one per digit: a digit's reads need no barrier before the next one's counts
  int equals, holes, sources;
};

template <int kCtas>
__global__ void __cluster_dims__(kCtas) __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ SelectShared sh;
  __shared__ int xs[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_rank;
  const cooperative_groups::cluster_group cluster = cooperative_groups::this_cluster();
  const int tid = threadIdx.x, cta = int(cluster.block_rank());
  for (int i = tid; i < 3 * kSelBins; i += kSelThreads) (&sh.hist[0][0])[i] = 0;
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int n = int(p.n), keep = int(p.keep);
  // each thread's tokens: a run, so that ranks within the block are the records' order
  const int per = (n + kCtas * kSelThreads - 1) / (kCtas * kSelThreads);
  const int lo = int(min(int64_t(cta * kSelThreads + tid) * per, int64_t(n)));
  const int hi = min(lo + per, n);
  auto each = [&](auto&& f) {  // f(i, key), four loads at a time
    for (int i0 = lo; i0 < hi; i0 += 4) {
      uint32_t k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        k[j] = i0 + j < hi ? weight_key(p.weights[i0 + j], p.ids[i0 + j], p.first_recent_id) : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i0 + j < hi) f(i0 + j, k[j]);
    }
  };
  uint32_t prefix = 0;
  int rank = n - keep - 1;  // rank (from 0) of the last token that leaves
#pragma unroll
  for (int d = 0; d < 3; ++d) {
    constexpr int kShift[3] = {21, 10, 0};
    const int shift = kShift[d], bits = d < 2 ? 11 : 10;
    each([&](int, uint32_t k) {
      if (d == 0 || (k >> (d == 1 ? 21 : 10)) == prefix) atomicAdd(&sh.hist[d][(k >> shift) & ((1 << bits) - 1)], 1);
    });
    cluster.sync();
    int x = 0, y = 0;  // bins 2 tid and 2 tid + 1 over the whole cluster
#pragma unroll
    for (int c = 0; c < kCtas; ++c) {
      const int2 v = reinterpret_cast<const int2*>(cluster.map_shared_rank(sh.hist[d], c))[tid];
      x += v.x;
      y += v.y;
    }
    int total;
    const int before = block_exclusive(x + y, xs, total);
    if (rank >= before && rank < before + x + y) {
      const int up = rank >= before + x;
      s_prefix = (prefix << bits) | uint32_t(2 * tid + up);
      s_rank = rank - before - (up ? x : 0);
    }
    __syncthreads();
    prefix = s_prefix;
    rank = s_rank;
  }
  // tokens below the key `prefix` leave, and the first rank + 1 of those at it
  const uint32_t pivot = prefix;
  const int take = rank + 1;
  int mine = 0, total;
  each([&](int, uint32_t k) { mine += k == pivot; });
  int equals = block_exclusive(mine, xs, total);
  if (tid == 0) sh.equals = total;
  cluster.sync();
  for (int c = 0; c < cta; ++c) equals += *cluster.map_shared_rank(&sh.equals, c);
  auto split = [&](auto&& hole, auto&& source) {
    int e = equals;
    each([&](int i, uint32_t k) {
      const bool leaves = k < pivot || (k == pivot && e < take);
      e += k == pivot;
      if (leaves && i < keep) hole(i);
      if (!leaves && i >= keep) source(i);
    });
  };
  int nh = 0, ns = 0, all_h, all_s;
  split([&](int) { ++nh; }, [&](int) { ++ns; });
  int h = block_exclusive(nh, xs, all_h), s = block_exclusive(ns, xs, all_s);
  if (tid == 0) {
    sh.holes = all_h;
    sh.sources = all_s;
  }
  cluster.sync();
  int holes = 0;
  for (int c = 0; c < cta; ++c) {
    holes += *cluster.map_shared_rank(&sh.holes, c);
    s += *cluster.map_shared_rank(&sh.sources, c);
  }
  h += holes;
  split([&](int i) { p.holes[h++] = i; }, [&](int i) { p.sources[s++] = i; });
  if (cta == kCtas - 1 && tid == 0) *p.count = holes + all_h;  // = sources: keep tokens stay
  cluster.sync();  // no CTA leaves while another reads its memory
}

// ------------------------------------------------------------------ eviction: the page list
// The stream's special pages in order, by way of the launch's parameters: a copy from pinned memory
// would make a host that evicts several streams a frame wait for a staging buffer until the frame's
// GPU work is done.
__global__ void __launch_bounds__(256) page_list_kernel(const __grid_constant__ PageListParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (int i = threadIdx.x; i < p.count; i += blockDim.x) p.dst[i] = p.pages[i];
}

// ------------------------------------------------------------------ eviction: the moves
// Survivor sources[i] into holes[i], K and V (and scale bytes) of every pool of the launch.
// Sources lie at or past `keep`, holes below it: no move reads what another writes.  As many CTAs as
// there can be moves and pools: the count is only known on the device.  6 moves in 24 pools: 3 us.
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ MoveParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int count = *p.count;
  char* pool = p.pools[blockIdx.y];
  const int units = int(p.row_bytes >> 4);  // 16-byte pieces of a token's K or V
  for (int i = blockIdx.x; i < count; i += gridDim.x) {
    const int a = p.sources[i], b = p.holes[i];
    const int64_t page_a = p.pages[a / p.ps], page_b = p.pages[b / p.ps];
    const int slot_a = a % p.ps, slot_b = b % p.ps;
    const char* src = pool + page_a * p.page_bytes + slot_a * p.row_bytes;
    char* dst = pool + page_b * p.page_bytes + slot_b * p.row_bytes;
    for (int u = threadIdx.x; u < 2 * units; u += blockDim.x) {
      const int64_t off = u < units ? int64_t(u) * 16 : p.half_bytes + int64_t(u - units) * 16;
      *reinterpret_cast<uint4*>(dst + off) = *reinterpret_cast<const uint4*>(src + off);
    }
    if (p.scales_off) {
      char* scales = pool + p.scales_off;
      for (int u = threadIdx.x; u < 2 * p.H; u += blockDim.x)
        scales[(page_b * 2 * p.H + u) * p.scale_row + slot_b] = scales[(page_a * 2 * p.H + u) * p.scale_row + slot_a];
    }
    if (p.weights != nullptr && blockIdx.y == 0 && threadIdx.x == 0) {
      p.weights[b] = p.weights[a];
      p.ids[b] = p.ids[a];
    }
  }
}

template <int D>
cudaError_t launch_weight_f32(const WeightParams& p, cudaStream_t s) {
  const dim3 grid(unsigned((p.max_specials + kWKeys - 1) / kWKeys), unsigned(p.H), unsigned(p.B));
  return launch_dependent(weight_f32_kernel<D>, grid, dim3(kWThreads), WeightCfg<D>::kBytes, s, p);
}

}  // namespace

cudaError_t launch_track(const TrackParams& p, cudaStream_t s) {
  const int threads = p.count < 256 ? 64 : 256;
  return launch_dependent(track_kernel, dim3(unsigned((p.count + threads - 1) / threads)), dim3(unsigned(threads)), 0, s,
                          p);
}

cudaError_t configure_weights_f32() {
  cudaError_t e = cudaFuncSetAttribute(weight_f32_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       WeightCfg<64>::kBytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(weight_f32_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, WeightCfg<128>::kBytes);
}

cudaError_t launch_weights(const WeightParams& p, int dtype, const CUtensorMap* map, int num_sms, cudaStream_t s) {
  const cudaError_t e = dtype != 1   ? launch_weights_tc(p, map, dtype == 2, num_sms, s)
                        : p.D == 64 ? launch_weight_f32<64>(p, s)
                                    : launch_weight_f32<128>(p, s);
  if (e != cudaSuccess) return e;
  return launch_dependent(weight_sum_kernel, dim3(unsigned((p.max_specials + 255) / 256), unsigned(p.B)), dim3(256), 0,
                          s, p);
}

cudaError_t launch_page_list(const PageListParams& p, cudaStream_t s) {
  return launch_dependent(page_list_kernel, dim3(1), dim3(256), 0, s, p);
}

cudaError_t launch_evict_select(const EvictParams& p, cudaStream_t s) {
  if (p.n <= kSelOneCta) return launch_dependent(evict_select_kernel<1>, dim3(1), dim3(kSelThreads), 0, s, p);
  return launch_dependent(evict_select_kernel<8>, dim3(8), dim3(kSelThreads), 0, s, p);
}

cudaError_t launch_evict_move(const MoveParams& p, cudaStream_t s) {
  const int moves = p.max_moves < 2048 ? p.max_moves : 2048;
  return launch_dependent(evict_move_kernel, dim3(unsigned(moves), unsigned(p.num_pools)), dim3(256), 0, s, p);
}

}  // namespace spk
