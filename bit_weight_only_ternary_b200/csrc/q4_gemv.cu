// q4_gemv.cu -- 4-bit products for few tokens: y[m][n] = sum_k s[n][k/g] (q[n][k] - 8) x[m][k].
//
// One CTA computes 32 weight rows (eight groups of four) over all of K for up to eight
// tokens; its eight warps take the 128-weight chunks of K in turn and their fp32 sums are
// added in warp order, so the result does not depend on timing. Bound: the bytes of the
// packed weights.
//
// A 16-byte load brings one 32-bit word (eight neighbouring weights) of four rows. Lane
// (g, t) = (lane / 4, lane % 4) reads word 4 s + t of row group g, which is, up to the
// order of rows and of K, the weight operand of m16n8k16 matrix instructions: rows 4g and
// 4g+1 are rows g and g+8 of a first tile, 4g+2 and 4g+3 of a second, and a word's eight
// weights are the lane's K values of two instructions. The activations need only the same
// order of K: lane (g, t) reads the eight activations of its word for token g with one
// 16-byte load. A code becomes a bf16 integer without a conversion: 0x4300 | q is 128 + q,
// minus 136 is q - 8, both exact. Products of these integers with bf16 activations are
// exact in fp32, sums are fp32, and the group's scale multiplies the group's sum in fp32:
// nothing is rounded to fewer bits before the final bf16 (or fp32) store.
#include <algorithm>

#include "lbq_common.cuh"
#include "sm100_async.cuh"

namespace {

using namespace lbq;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowTile = 32;
constexpr int kMaxTokens = 8;  // columns of one matrix instruction

struct Q4Prod {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* x;   // [M][K]
  void* y;             // bf16 (or fp32) [M][N]
  int64_t gcode;       // code bytes per group of four rows
  int32_t gscale;      // scales per group of four rows
  int32_t N, nc;       // rows; 128-weight chunks of K
  int32_t tile0;       // first CTA of this product
};

template <int kCap>
struct Q4List {
  int32_t n, M;
  Q4Prod p[kCap];
};

// 16 bytes of packed weights: streamed, not kept in L1.
__device__ __forceinline__ uint4 ldg_w(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
// Activations: plain loads (they may have been written just before this kernel).
__device__ __forceinline__ uint4 ldg_x(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Pair j of a word's codes (weights 2j, 2j+1) as two bf16 integers q - 8.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, int j) {
  const uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | 0x43004300u;  // 128 + q
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));  // - 136
  return r;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// One chunk of K in flight: 4 x 16 bytes of codes, the scales and the activations.
template <int kG>
struct Chunk {
  uint4 w[4];
  uint2 s[kG == 32 ? 4 : 1];  // fp16 of rows 4g .. 4g+3 per group of K
  uint4 x[4];
};

// acc[tile][..] += this warp's chunks of the 32-row tile; xrow: this lane's token's
// activations (null: zeros).
template <int kG>
__device__ __forceinline__ void warp_sum_tile(const uint8_t* codes, const uint16_t* scales, int nc,
                                              const uint16_t* xrow, int warp, int lane,
                                              float (&acc)[2][4]) {
  const int t = lane & 3;
  const uint8_t* wp = codes + 16 * t;
  Chunk<kG> buf[2];
  auto load = [&](Chunk<kG>& b, int c) {
    if (c >= nc) return;
#pragma unroll
    for (int s = 0; s < 4; ++s) b.w[s] = ldg_w(wp + static_cast<int64_t>(c) * 256 + 64 * s);
    constexpr int kS = kG == 32 ? 4 : 1;
#pragma unroll
    for (int s = 0; s < kS; ++s)
      b.s[s] = __ldg(reinterpret_cast<const uint2*>(scales + 4 * (static_cast<int64_t>(c) * kS + s)));
#pragma unroll
    for (int s = 0; s < 4; ++s)
      b.x[s] = xrow ? ldg_x(xrow + static_cast<int64_t>(c) * kQ4Chunk + 32 * s + 8 * t) : make_uint4(0, 0, 0, 0);
  };
  auto use = [&](const Chunk<kG>& b) {
    float part[2][4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      if (kG == 32 || s == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) part[i >> 2][i & 3] = 0.0f;
      }
      const uint4 w = b.w[s], x = b.x[s];
      mma_bf16(part[0], q4_pair(w.x, 0), q4_pair(w.y, 0), q4_pair(w.x, 1), q4_pair(w.y, 1), x.x, x.y);
      mma_bf16(part[1], q4_pair(w.z, 0), q4_pair(w.w, 0), q4_pair(w.z, 1), q4_pair(w.w, 1), x.x, x.y);
      mma_bf16(part[0], q4_pair(w.x, 2), q4_pair(w.y, 2), q4_pair(w.x, 3), q4_pair(w.y, 3), x.z, x.w);
      mma_bf16(part[1], q4_pair(w.z, 2), q4_pair(w.w, 2), q4_pair(w.z, 3), q4_pair(w.w, 3), x.z, x.w);
      if (kG == 32 || s == 3) {
        const uint2 sc = b.s[kG == 32 ? s : 0];
        const float2 s01 = __half22float2(*reinterpret_cast<const __half2*>(&sc.x));
        const float2 s23 = __half22float2(*reinterpret_cast<const __half2*>(&sc.y));
        acc[0][0] += s01.x * part[0][0];
        acc[0][1] += s01.x * part[0][1];
        acc[0][2] += s01.y * part[0][2];
        acc[0][3] += s01.y * part[0][3];
        acc[1][0] += s23.x * part[1][0];
        acc[1][1] += s23.x * part[1][1];
        acc[1][2] += s23.y * part[1][2];
        acc[1][3] += s23.y * part[1][3];
      }
    }
  };
  load(buf[0], warp);
  load(buf[1], warp + kWarps);
  for (int c = warp; c < nc; c += 2 * kWarps) {
    use(buf[0]);
    load(buf[0], c + 2 * kWarps);
    if (c + kWarps >= nc) break;
    use(buf[1]);
    load(buf[1], c + 3 * kWarps);
  }
}

// The warps' sums added in warp order; put(token, row in tile, value).
template <typename Put>
__device__ __forceinline__ void join_warps(float (*red)[kRowTile * kMaxTokens], const float (&acc)[2][4],
                                           int warp, int lane, Put put) {
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int c = 0; c < 2; ++c)  // token 2t + c, row 4g + 2i + h
        red[warp][(2 * t + c) * kRowTile + 4 * g + 2 * i + h] = acc[i][2 * h + c];
  __syncthreads();
  const int o = threadIdx.x;
  float v = red[0][o];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += red[w][o];
  put(o / kRowTile, o % kRowTile, v);
}

template <int kG, int kCap, bool kF32>
__global__ void __launch_bounds__(kThreads, 2)
    q4_list_kernel(const __grid_constant__ Q4List<kCap> a) {
  __shared__ float red[kWarps][kRowTile * kMaxTokens];
  const int tile = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  int lo = 0;
  if (kCap > 1) {  // the last product whose first tile is at most this one
    int hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.p[mid].tile0 <= tile) lo = mid; else hi = mid;
    }
  }
  const Q4Prod& P = a.p[lo];
  pdl_launch_dependents();
  const int row0 = (tile - P.tile0) * kRowTile;
  const int ng = (P.N + 3) >> 2;
  int64_t grp = (row0 >> 2) + g;
  if (grp >= ng) grp = ng - 1;  // rows behind the last: read it again, store nothing
  const int m0 = blockIdx.y * kMaxTokens, K = P.nc * kQ4Chunk;
  pdl_wait();
  float acc[2][4] = {};
  const uint16_t* xrow = m0 + g < a.M ? P.x + static_cast<int64_t>(m0 + g) * K : nullptr;
  warp_sum_tile<kG>(P.codes + grp * P.gcode, P.scales + grp * P.gscale, P.nc, xrow, warp, lane, acc);
  join_warps(red, acc, warp, lane, [&](int m, int r, float v) {
    if (m0 + m >= a.M || row0 + r >= P.N) return;
    const int64_t o = static_cast<int64_t>(m0 + m) * P.N + row0 + r;
    if (kF32) static_cast<float*>(P.y)[o] = v;
    else static_cast<uint16_t*>(P.y)[o] = f32_to_bf16_bits(v);
  });
}

struct Q4ExpertArgs {
  const uint8_t* codes;
  const uint16_t* scales;
  int64_t gcode, ecode, escale;  // code bytes per group, per expert; scales per expert
  int32_t gscale, N, nc;
  lbq_expert_rows r;
};

template <int kG>
__global__ void __launch_bounds__(kThreads, 2) q4_expert_kernel(const __grid_constant__ Q4ExpertArgs a) {
  __shared__ float red[kWarps][kRowTile * kMaxTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2;
  const int e = blockIdx.y, row0 = blockIdx.x * kRowTile;
  pdl_launch_dependents();
  pdl_wait();
  const int R = static_cast<int>(a.r.R);
  int lo = __ldcg(a.r.offsets + e), hi = __ldcg(a.r.offsets + e + 1);
  lo = lo < 0 ? 0 : lo;
  hi = hi > R ? R : hi;
  if (lo >= hi) return;
  const int ng = (a.N + 3) >> 2, K = a.nc * kQ4Chunk;
  int64_t grp = (row0 >> 2) + g;
  if (grp >= ng) grp = ng - 1;
  const uint8_t* codes = a.codes + e * a.ecode + grp * a.gcode;
  const uint16_t* scales = a.scales + e * a.escale + grp * a.gscale;
  for (int m0 = lo; m0 < hi; m0 += kMaxTokens) {
    const uint16_t* xrow = nullptr;
    if (m0 + g < hi) {
      int64_t src = m0 + g;
      if (a.r.slots) {
        const int slot = __ldcg(a.r.slots + src);
        src = slot < 0 ? -1 : slot / a.r.topk;
      }
      if (src >= 0 && src < a.r.T) xrow = a.r.X + src * K;
    }
    float acc[2][4] = {};
    warp_sum_tile<kG>(codes, scales, a.nc, xrow, warp, lane, acc);
    join_warps(red, acc, warp, lane, [&](int m, int r, float v) {
      if (m0 + m < hi && row0 + r < a.N)
        a.r.Y[static_cast<int64_t>(m0 + m) * a.N + row0 + r] = f32_to_bf16_bits(v);
    });
    __syncthreads();  // red is read before the next tokens' sums
  }
}

// Programmatic dependent launch on stream s: the kernel starts early and waits itself.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*k)(KArgs...), dim3 grid, dim3 block, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args...);
}

Q4Prod make_prod(const lbq_weights& w, const uint16_t* x, void* y) {
  Q4Prod p;
  p.codes = static_cast<const uint8_t*>(w.codes);
  p.scales = static_cast<const uint16_t*>(w.scales);
  p.x = x;
  p.y = y;
  p.gcode = 4 * w.code_stride;
  p.gscale = static_cast<int32_t>(4 * w.scale_stride);
  p.N = static_cast<int32_t>(w.N);
  p.nc = static_cast<int32_t>(w.K / kQ4Chunk);
  p.tile0 = 0;
  return p;
}

unsigned tiles_of(int64_t N) { return static_cast<unsigned>((N + kRowTile - 1) / kRowTile); }

}  // namespace

cudaError_t lbq_launch_q4_list(const lbq_product* ps, int32_t n, float* y32, cudaStream_t s) {
  const bool g32 = ps[0].w.fmt == LBQ_Q4G32;
  if (n == 1) {
    Q4List<1> a;
    a.n = 1;
    a.M = 1;
    a.p[0] = make_prod(ps[0].w, ps[0].x, y32 ? static_cast<void*>(y32) : ps[0].y);
    const dim3 grid(tiles_of(ps[0].w.N));
    if (y32) return launch_pdl(g32 ? q4_list_kernel<32, 1, true> : q4_list_kernel<128, 1, true>, grid, kThreads, s, a);
    return launch_pdl(g32 ? q4_list_kernel<32, 1, false> : q4_list_kernel<128, 1, false>, grid, kThreads, s, a);
  }
  static thread_local Q4List<LBQ_BATCH_MAX> a;  // 18 KB: off the stack
  a.n = n;
  a.M = 1;
  // longest K first: its CTAs take longest, so they should not be the last to start
  int32_t order[LBQ_BATCH_MAX];
  for (int32_t i = 0; i < n; ++i) order[i] = i;
  std::stable_sort(order, order + n, [&](int32_t i, int32_t k) { return ps[i].w.K > ps[k].w.K; });
  int64_t tiles = 0;
  for (int32_t i = 0; i < n; ++i) {
    const lbq_product& q = ps[order[i]];
    a.p[i] = make_prod(q.w, q.x, q.y);
    a.p[i].tile0 = static_cast<int32_t>(tiles);
    tiles += tiles_of(q.w.N);
  }
  if (tiles > INT32_MAX) return cudaErrorInvalidValue;
  return launch_pdl(g32 ? q4_list_kernel<32, LBQ_BATCH_MAX, false> : q4_list_kernel<128, LBQ_BATCH_MAX, false>,
                    dim3(static_cast<unsigned>(tiles)), kThreads, s, a);
}

cudaError_t lbq_launch_q4_few(const lbq_weights* w, const uint16_t* X, int64_t M, uint16_t* Y,
                              cudaStream_t s) {
  if (M > static_cast<int64_t>(65535) * kMaxTokens) return cudaErrorInvalidValue;
  Q4List<1> a;
  a.n = 1;
  a.M = static_cast<int32_t>(M);
  a.p[0] = make_prod(*w, X, Y);
  const dim3 grid(tiles_of(w->N), static_cast<unsigned>((M + kMaxTokens - 1) / kMaxTokens));
  return launch_pdl(w->fmt == LBQ_Q4G32 ? q4_list_kernel<32, 1, false> : q4_list_kernel<128, 1, false>, grid,
                    kThreads, s, a);
}

cudaError_t lbq_launch_q4_expert_few(const lbq_weights* w, const lbq_expert_rows& r, cudaStream_t s) {
  Q4ExpertArgs a;
  a.codes = static_cast<const uint8_t*>(w->codes);
  a.scales = static_cast<const uint16_t*>(w->scales);
  a.gcode = 4 * w->code_stride;
  a.gscale = static_cast<int32_t>(4 * w->scale_stride);
  const int64_t ng = (w->N + 3) / 4;
  a.ecode = ng * a.gcode;
  a.escale = ng * a.gscale;
  a.N = static_cast<int32_t>(w->N);
  a.nc = static_cast<int32_t>(w->K / kQ4Chunk);
  a.r = r;
  const dim3 grid(tiles_of(w->N), static_cast<unsigned>(r.E));
  return launch_pdl(w->fmt == LBQ_Q4G32 ? q4_expert_kernel<32> : q4_expert_kernel<128>, grid, kThreads, s, a);
}
