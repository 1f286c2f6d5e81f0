// expert.cu -- token slots sorted by expert, rows copied to that order and added back.
//
// The sort is a stable counting sort in one launch: every warp counts the experts of its
// own run of slots, the counts become first rows by prefix sums over warps, CTAs (a
// cluster reads each other's counts through distributed shared memory) and experts, and
// every warp walks its run again to hand out rows. Row order is slot order within an
// expert, so the result does not depend on timing. The copies and sums are bound by the
// bytes of the rows; one CTA a token, 16-byte accesses where the rows allow them.
#include <cooperative_groups.h>

#include "lbq_common.cuh"
#include "sm100_async.cuh"

namespace {

using namespace lbq;
namespace cg = cooperative_groups;

constexpr int kSortThreads = 512, kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8, kSortMost = 16;  // CTAs of a cluster
// Slots of a warp's run that stay in registers, 32 at a time (a run of more is read twice).
constexpr int kSortKeep = 8;

template <typename Id>
__device__ __forceinline__ int expert_of(const Id* ids, int64_t i, int64_t end, int E) {
  if (i >= end) return E;
  const Id v = ids[i];
  return v >= 0 && v < static_cast<Id>(E) ? static_cast<int>(v) : E;
}

// The lanes with this lane's value (bits 0 .. bits-1): one ballot a bit. (A match
// instruction costs more.)
__device__ __forceinline__ unsigned peers_of(int v, int bits) {
  unsigned peers = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const bool set = (v >> b) & 1;
    const unsigned m = __ballot_sync(0xffffffffu, set);
    peers &= set ? m : ~m;
  }
  return peers;
}

// Shared memory: hist [warps][E], tot [E], base [E].
template <typename Id>
__global__ void __launch_bounds__(kSortThreads, 1)
    expert_sort_kernel(const Id* ids, int64_t R, int E, int64_t per_warp,
                       int32_t* __restrict__ offsets, int32_t* __restrict__ rows,
                       int32_t* __restrict__ slots) {
  pdl_launch_dependents();
  pdl_wait();
  extern __shared__ int32_t sm[];
  __shared__ int32_t wsum[kSortWarps];
  int32_t* hist = sm;
  int32_t* tot = hist + kSortWarps * E;
  int32_t* base = tot + E;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = tid; i < kSortWarps * E; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  const int64_t w0 = (static_cast<int64_t>(rank) * kSortWarps + warp) * per_warp;
  const int64_t w1 = w0 + per_warp < R ? w0 + per_warp : R;
  int32_t* mine = hist + warp * E;
  const int bits = 32 - __clz(E);  // of the values 0 .. E
  // a batch of the warp's ids, all loads at once (one at a time, 262144 slots took 70 us);
  // the first one stays
  auto fetch = [&](int64_t i, int (&v)[kSortKeep]) {
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k) v[k] = i + 32 * k < w1 ? expert_of(ids, i + 32 * k + lane, w1, E) : E;
  };
  int kept[kSortKeep], more[kSortKeep];
  fetch(w0, kept);
  auto count = [&](int e) {
    const unsigned peers = peers_of(e, bits);
    if (e < E && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
  };
#pragma unroll
  for (int k = 0; k < kSortKeep; ++k)
    if (w0 + 32 * k < w1) count(kept[k]);
  for (int64_t i = w0 + 32 * kSortKeep; i < w1; i += 32 * kSortKeep) {
    fetch(i, more);
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k)
      if (i + 32 * k < w1) count(more[k]);
  }
  __syncthreads();
  // each expert's counts of the warps before, and the CTA's total
  for (int e = tid; e < E; e += kSortThreads) {
    int32_t c[kSortWarps], run = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) c[w] = hist[w * E + e];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      hist[w * E + e] = run;
      run += c[w];
    }
    tot[e] = run;
  }
  cluster.sync();
  // thread e: totals of all CTAs and of those before this one, and their running sum over
  // the experts (kSortThreads at a time)
  int32_t total = 0;
  for (int e0 = 0; e0 < E; e0 += kSortThreads) {
    const int e = e0 + tid;
    int32_t all = 0, before = 0;
    if (e < E) {
      int32_t v[kSortMost];
#pragma unroll
      for (int c = 0; c < kSortMost; ++c) v[c] = c < C ? *cluster.map_shared_rank(tot + e, c) : 0;
#pragma unroll
      for (int c = 0; c < kSortMost; ++c) {
        all += v[c];
        if (c < rank) before += v[c];
      }
    }
    int32_t scan = all;  // inclusive over the warp, then over the CTA
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t v = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += v;
    }
    if (lane == 31) wsum[warp] = scan;
    __syncthreads();
    int32_t ahead = total;
    for (int w = 0; w < kSortWarps; ++w) {
      if (w < warp) ahead += wsum[w];
      total += wsum[w];
    }
    if (e < E) {
      const int32_t first = ahead + scan - all;
      base[e] = first + before;
      if (rank == 0) offsets[e] = first;
    }
    __syncthreads();
  }
  if (rank == 0 && tid == 0) offsets[E] = total;
  cluster.sync();  // no CTA leaves while another still reads its totals
  const unsigned below = (1u << lane) - 1u;
  auto place = [&](int e, int64_t i) {
    const unsigned peers = peers_of(e, bits);
    int32_t row = -1;
    if (e < E) row = base[e] + mine[e] + __popc(peers & below);
    __syncwarp();
    if (e < E && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
    __syncwarp();
    if (i + lane < w1) {
      rows[i + lane] = row;
      if (row >= 0) slots[row] = static_cast<int32_t>(i + lane);
    }
  };
#pragma unroll
  for (int k = 0; k < kSortKeep; ++k)
    if (w0 + 32 * k < w1) place(kept[k], w0 + 32 * k);
  for (int64_t i = w0 + 32 * kSortKeep; i < w1; i += 32 * kSortKeep) {
    fetch(i, more);
#pragma unroll
    for (int k = 0; k < kSortKeep; ++k)
      if (i + 32 * k < w1) place(more[k], i + 32 * k);
  }
  for (int64_t r = total + static_cast<int64_t>(rank) * kSortThreads + tid; r < R; r += static_cast<int64_t>(C) * kSortThreads)
    slots[r] = -1;
}

// kVec bf16 values as one access, widened to fp32.
template <int kVec>
struct Vec;
template <>
struct Vec<8> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32_to_bf16_bits(f[2 * i]) | (static_cast<uint32_t>(f32_to_bf16_bits(f[2 * i + 1])) << 16);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<1> {
  uint16_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *p = v; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = bf16_bits_to_f32(v); }
  __device__ __forceinline__ void set(const float (&f)[1]) { v = f32_to_bf16_bits(f[0]); }
};

constexpr int kRowThreads = 256;

struct RouteArgs {
  const int32_t* rows;
  const float* weights;  // null: all 1
  int64_t R, N;
  int32_t topk;
};

// The row of slot i, or -1 when it names none.
__device__ __forceinline__ int64_t row_of(const RouteArgs& a, int64_t i) {
  const int32_t r = a.rows[i];
  return r >= 0 && r < a.R ? r : -1;
}

template <int kVec, bool kWeighted>
__global__ void __launch_bounds__(kRowThreads)
    dispatch_kernel(const uint16_t* X, const RouteArgs a, uint16_t* out) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t t = blockIdx.x;
  for (int64_t n = static_cast<int64_t>(threadIdx.x) * kVec; n < a.N; n += static_cast<int64_t>(blockDim.x) * kVec) {
    Vec<kVec> v;
    v.load(X + t * a.N + n);
    float f[kVec];
    if (kWeighted) v.get(f);
    for (int j = 0; j < a.topk; ++j) {
      const int64_t r = row_of(a, t * a.topk + j);
      if (r < 0) continue;
      if (kWeighted) {
        const float w = a.weights[t * a.topk + j];
        float p[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) p[i] = w * f[i];
        Vec<kVec> o;
        o.set(p);
        o.store(out + r * a.N + n);
      } else {
        v.store(out + r * a.N + n);
      }
    }
  }
}

// Slots of a token taken together: their rows' loads are all in flight at once.
constexpr int kSlotsAtOnce = 8;

// The rows (and weights) of up to eight slots of a token, lane j's of slot j0 + j. CTAs
// walk over the tokens and read the next token's ahead: looked up when they were needed,
// they put a second memory latency before every token's rows (32768 rows of 2048: 27 us to
// add up); in every lane's registers all eight, they spilled.
template <bool kWeighted>
struct Slots {
  int32_t r;
  float w;
  __device__ __forceinline__ void load(const RouteArgs& a, int64_t t, int64_t T, int j0) {
    const int j = j0 + (threadIdx.x & 31);
    const bool in = t < T && j < j0 + kSlotsAtOnce && j < a.topk;
    r = in ? a.rows[t * a.topk + j] : -1;
    w = kWeighted && in ? a.weights[t * a.topk + j] : 0.0f;
    if (r >= a.R) r = -1;
    if (r < 0) w = 0.0f;  // whatever it is: the slot adds nothing
  }
  __device__ __forceinline__ void spread(int32_t (&rows)[kSlotsAtOnce], float (&weights)[kSlotsAtOnce]) const {
#pragma unroll
    for (int j = 0; j < kSlotsAtOnce; ++j) {
      rows[j] = __shfl_sync(0xffffffffu, r, j);
      if (kWeighted) weights[j] = __shfl_sync(0xffffffffu, w, j);
    }
  }
};

template <int kVec, bool kWeighted>
__global__ void __launch_bounds__(kRowThreads, 4)
    combine_kernel(const uint16_t* Y, const RouteArgs a, int64_t T, uint16_t* out) {
  pdl_launch_dependents();
  pdl_wait();
  const int N = static_cast<int>(a.N), threads = static_cast<int>(blockDim.x);
  const int cols = (N + kVec - 1) / kVec, rounds = (cols + threads - 1) / threads;
  Slots<kWeighted> next;
  next.load(a, blockIdx.x, T, 0);
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    const Slots<kWeighted> first = next;
    next.load(a, t + gridDim.x, T, 0);
    for (int k = 0; k < rounds; ++k) {  // (whole warps, for the shuffles)
      const int c = k * threads + static_cast<int>(threadIdx.x);
      const uint16_t* const y = Y + kVec * c;
      float acc[kVec] = {};
      for (int j0 = 0; j0 < a.topk; j0 += kSlotsAtOnce) {
        Slots<kWeighted> s = first;
        if (j0) s.load(a, t, T, j0);
        int32_t r[kSlotsAtOnce];
        float w[kSlotsAtOnce];
        s.spread(r, w);
        Vec<kVec> v[kSlotsAtOnce];
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
          v[j] = {};
          if (r[j] >= 0 && c < cols) v[j].load(y + static_cast<int64_t>(r[j]) * N);
        }
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {  // (a slot left out adds 0 times zeros)
          float f[kVec];
          v[j].get(f);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[i] += kWeighted ? w[j] * f[i] : f[i];
        }
      }
      Vec<kVec> o;
      o.set(acc);
      if (c < cols) o.store(out + t * N + kVec * c);
    }
  }
}

// (The form for single columns, odd widths and addresses, spills 68 bytes a thread.)
template <int kVec>
__global__ void __launch_bounds__(kRowThreads, 3)
    combine_grad_kernel(const uint16_t* dout, const uint16_t* Y, const RouteArgs a, int64_t T, uint16_t* dY,
                        float* dweights) {
  pdl_launch_dependents();
  pdl_wait();
  __shared__ float red[2][kRowThreads / 32][kSlotsAtOnce];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = static_cast<int>(blockDim.x) >> 5;
  const int N = static_cast<int>(a.N);
  int buf = 0;
  Slots<true> next;
  next.load(a, blockIdx.x, T, 0);
  for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
    for (int j0 = 0; j0 < a.topk; j0 += kSlotsAtOnce, buf ^= 1) {
      int32_t r[kSlotsAtOnce];
      float w[kSlotsAtOnce];
      next.spread(r, w);
      const bool more = j0 + kSlotsAtOnce < a.topk;
      next.load(a, more ? t : t + gridDim.x, T, more ? j0 + kSlotsAtOnce : 0);
      float dot[kSlotsAtOnce] = {};
      for (int n = static_cast<int>(threadIdx.x) * kVec; n < N; n += static_cast<int>(blockDim.x) * kVec) {
        Vec<kVec> v, y[kSlotsAtOnce];
        v.load(dout + t * N + n);
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
          y[j] = {};
          if (r[j] >= 0) y[j].load(Y + n + static_cast<int64_t>(r[j]) * N);
        }
        float g[kVec];
        v.get(g);
#pragma unroll
        for (int j = 0; j < kSlotsAtOnce; ++j) {
          if (r[j] < 0) continue;  // (its gradient is 0, whatever dout holds)
          float f[kVec], p[kVec];
          y[j].get(f);
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            dot[j] += g[i] * f[i];
            p[i] = w[j] * g[i];
          }
          Vec<kVec> d;
          d.set(p);
          d.store(dY + n + static_cast<int64_t>(r[j]) * N);
        }
      }
      // lanes by a fixed tree, then warps in order (two buffers: one barrier a round)
#pragma unroll
      for (int j = 0; j < kSlotsAtOnce; ++j) {
        const float v = warp_sum(dot[j]);
        if (lane == 0) red[buf][warp][j] = v;
      }
      __syncthreads();
      if (threadIdx.x < kSlotsAtOnce && j0 + static_cast<int>(threadIdx.x) < a.topk) {
        float v = 0.0f;
        for (int q = 0; q < warps; ++q) v += red[buf][q][threadIdx.x];
        dweights[t * a.topk + j0 + threadIdx.x] = v;
      }
    }
  }
}

// Threads a token: one 16-byte (or single) column each, whole warps.
int threads_for(int64_t N, int vec) {
  const int64_t n = ((N + vec - 1) / vec + 31) / 32 * 32;
  return n < kRowThreads ? static_cast<int>(n) : kRowThreads;
}

// Launches early beside the previous kernel of the stream; the kernels wait for it themselves.
template <typename... P, typename... A>
cudaError_t launch_rows(void (*k)(P...), unsigned grid, int threads, cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, P(args)...);
}

// CTAs that walk over T tokens: as many as are resident, at `full` CTAs of kRowThreads an SM.
unsigned walkers(int64_t T, int threads, int full) {
  const int64_t most = static_cast<int64_t>(sm_count()) * (full * kRowThreads / threads < 16 ? full * kRowThreads / threads : 16);
  return static_cast<unsigned>(T < most ? T : most);
}

bool vec8(int64_t N, const void* a, const void* b, const void* c = nullptr, const void* d = nullptr) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) |
                      reinterpret_cast<uintptr_t>(c) | reinterpret_cast<uintptr_t>(d);
  return N % 8 == 0 && (u & 15) == 0;
}

template <typename Id>
cudaError_t launch_sort(const Id* ids, int64_t R, int32_t E, int32_t* offsets, int32_t* rows,
                        int32_t* slots, cudaStream_t s) {
  static PerDevice<int> configured;  // CTAs of the largest cluster this device takes
  int largest = 0;
  const cudaError_t e = configured.get(
      [](int, int* v) {
        constexpr int smem = (kSortWarps + 2) * LBQ_MAX_EXPERTS * 4;
        cudaError_t r = cudaFuncSetAttribute(expert_sort_kernel<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (r == cudaSuccess)
          r = cudaFuncSetAttribute(expert_sort_kernel<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r != cudaSuccess) return r;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(kSortMost);
        cfg.blockDim = dim3(kSortThreads);
        cfg.dynamicSmemBytes = smem;
        return cudaOccupancyMaxPotentialClusterSize(v, expert_sort_kernel<Id>, &cfg);
      },
      &largest);
  if (e != cudaSuccess) return e;
  // one CTA for few slots, a cluster for more (128 experts, one / eight CTAs: 64 slots 3.3 /
  // 3.7 us, 512 3.9 / 4.3, 1024 4.8 / 4.4, 4096 9.4 / 4.3; eight / sixteen: 16384 slots 6.6 /
  // 5.4, 32768 9.6 / 6.9, 262144 56 / 30)
  const int C = R <= kSortThreads ? 1 : (R <= 8192 || largest < kSortMost ? kSortCluster : kSortMost);
  const int64_t warps = static_cast<int64_t>(C) * kSortWarps;
  const int64_t per_warp = ((R + warps - 1) / warps + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(C));
  cfg.blockDim = dim3(kSortThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(kSortWarps + 2) * E * 4;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(C);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, expert_sort_kernel<Id>, ids, R, static_cast<int>(E), per_warp, offsets, rows, slots);
}

}  // namespace

cudaError_t lbq_launch_expert_sort(const void* ids, int id_bytes, int64_t R, int32_t E,
                                   int32_t* offsets, int32_t* rows, int32_t* slots, cudaStream_t s) {
  return id_bytes == 8 ? launch_sort(static_cast<const long long*>(ids), R, E, offsets, rows, slots, s)
                       : launch_sort(static_cast<const int*>(ids), R, E, offsets, rows, slots, s);
}

cudaError_t lbq_launch_expert_dispatch(const uint16_t* X, const int32_t* rows, const float* weights,
                                       int64_t T, int32_t topk, int64_t K, int64_t R, uint16_t* out,
                                       cudaStream_t s) {
  const RouteArgs a = {rows, weights, R, K, topk};
  const unsigned grid = static_cast<unsigned>(T);
  const bool v8 = vec8(K, X, out);
  return launch_rows(v8 ? (weights ? dispatch_kernel<8, true> : dispatch_kernel<8, false>)
                        : (weights ? dispatch_kernel<1, true> : dispatch_kernel<1, false>),
                     grid, threads_for(K, v8 ? 8 : 1), s, X, a, out);
}

cudaError_t lbq_launch_expert_combine(const uint16_t* Y, const int32_t* rows, const float* weights,
                                      int64_t T, int32_t topk, int64_t N, int64_t R, uint16_t* out,
                                      cudaStream_t s) {
  const RouteArgs a = {rows, weights, R, N, topk};
  const bool v8 = vec8(N, Y, out);
  const int threads = threads_for(N, v8 ? 8 : 1);
  return launch_rows(v8 ? (weights ? combine_kernel<8, true> : combine_kernel<8, false>)
                        : (weights ? combine_kernel<1, true> : combine_kernel<1, false>),
                     walkers(T, threads, 4), threads, s, Y, a, T, out);
}

cudaError_t lbq_launch_expert_combine_grad(const uint16_t* dout, const uint16_t* Y,
                                           const int32_t* rows, const float* weights, int64_t T,
                                           int32_t topk, int64_t N, int64_t R, uint16_t* dY,
                                           float* dweights, cudaStream_t s) {
  const RouteArgs a = {rows, weights, R, N, topk};
  const bool v8 = vec8(N, dout, Y, dY);
  const int threads = threads_for(N, v8 ? 8 : 1);
  return launch_rows(v8 ? combine_grad_kernel<8> : combine_grad_kernel<1>, walkers(T, threads, 3), threads, s, dout,
                     Y, a, T, dY, dweights);
}
