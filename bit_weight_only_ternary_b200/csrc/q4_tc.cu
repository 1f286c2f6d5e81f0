// q4_tc.cu -- 4-bit products of many tokens on the 5th-generation tensor cores: one
// matrix for all rows (lbq_gemm) or a matrix per expert (lbq_expert_gemm).
//
// Y[m][n] = sum_k s[n][k/g] (q[n][k] - 8) x[m][k]. The kernel decodes tiles of 128 weight
// rows x 128 K into tensor memory as fp16 and multiplies them with fp16 activations
// (tcgen05.mma kind::f16, fp32 accumulators in tensor memory).
//
// Roundings. Activations: each row is scaled by a power of two into fp16, exactly; a row
// that spans more than fp16 holds is flagged and recomputed in fp32 (as in the ternary
// product). Weights: s (q - 8) has up to 15 significant bits and is rounded to fp16's 11,
// at most 2^-11 of each term (bf16 would be 2^-8, as much as the final rounding of y
// itself; keeping q - 8 exact and scaling the accumulators would cost one tensor-memory
// read and one multiply per accumulator and group of K: for groups of 32 as many fp32
// operations as the SM has in that time). Every weight row's scales are first multiplied
// by a power of two that brings the row's largest scale to [2^11, 2^12), so that neither
// large nor tiny scales leave fp16's normal range; the epilogue undoes both powers.
//
// Persistent: each pair of CTAs (a cluster of two, cta_group::2) walks over output tiles of
// 256 weight rows, 128 a CTA, x up to 256 tokens (balanced: a batch or an expert's rows are
// cut into equal tiles, the matrix instruction takes the tile's own token count rounded up
// to 16). Each CTA fetches half of the tile's activations, and the tensor cores read both
// halves: with a CTA on its own every SM fetched all 256 tokens, 64 KB per 128 K and so 17
// TB/s from L2 at the MMA's own rate, and that bound it (1.42 ms for 4096 x 5120 x 34816).
// Warp roles:
//   warp 0   one lane copies activations (128 K x tokens), one 3D TMA a block: issuing four
//            or eight boxes of 32 rows a block took longer than the matrix instructions
//   warp 1   allocates tensor memory; in the pair's first CTA one lane issues the MMAs
//   warp 2   one lane copies packed weights and scales, 256 K x 128 rows a copy
//   warp 3   finds the tiles ahead of the others and leaves their exponents and flags
//   warps 4-19 decode, four warps a weight stage; then, one block later (the stages are
//            refilled for the next tile first, so the tensor cores go on as soon as the
//            accumulators have been read), the tile's epilogue
// Every wait is bounded (sm100_async.cuh). Measured: 4096 tokens x 5120 x 34816 in 0.92 ms
// by a cool chip, 1.07 to 1.11 in a row of passes (1.59 to 1.31 PFLOP/s, by the power that
// is left), 333 x 5120 x 7001 in 30 us, 4096 tokens x 8 of 128 experts of 2048 x 1536 in 250
// to 260 us with other inputs each pass (820 to 790 TFLOP/s) and 215 to 226 in a graph of
// the same one again and again, which finds its weights in L2 (the times beside the choices
// below are of such graphs); 45 us are the preparation. A row that is recomputed in fp32
// costs 5 to 8 ns a weight in every weight tile: 1024 rows of 17408 x 5120 take 0.14 to 0.16
// ms, with one in 16 so 3.1, behind a squared relu (two rows in five) 21. A block of 128 K
// cannot take less than 0.27 us: the tensor cores read its weights, 128 x 128 a CTA, from
// tensor memory in 8 x 64 cycles.
#include <cudaTypedefs.h>

#include <algorithm>

#include "sm100_async.cuh"

namespace {

using namespace lbq;

constexpr int kTileN = 128, kTileK = 128, kMaxTileM = 256;
constexpr int kStages = 4;             // stages of one 128 x 128 weight block and its activations
constexpr int kDec = 4 * kTileN;       // decoder threads
constexpr int kThreads = 128 + kDec;
constexpr uint32_t kSlabBytes = kMaxTileM / 2 * 128;  // activations: 64 K of half the tile's tokens
// An activation copy brings 128 K (two 128-byte swizzled halves) of a CTA's tokens at once:
// a tensor map for every multiple of kBoxStep tokens up to 128.
constexpr int kBoxStep = 16, kBoxes = kMaxTileM / 2 / kBoxStep;
struct XMaps {
  CUtensorMap m[kBoxes];
};
// A weight copy: 32 row groups x (2 blocks = 32 words of four rows, plus one word of
// four rows so that a group's row is 33 16-byte units, an odd number: the eight groups a
// warp decodes then read from different banks).
constexpr int kChunkBlocks = 2;
constexpr uint32_t kGroupWords = 4 * 32 + 4;
constexpr uint32_t kRawBytes = kGroupWords * 4 * (kTileN / 4);
constexpr int kRawStages = 4;
constexpr uint32_t kScaleStage = 2048;  // bytes reserved for a chunk's scales
// Tensor memory: accumulators in columns [0, 256), weight stage s at 256 + 64 s.
constexpr uint32_t kTmemCols = 512, kTmemA = 256;
// Shared memory, from a 1 KB boundary.
constexpr uint32_t kOffSlab = 0;
constexpr uint32_t kOffRaw = kOffSlab + kStages * 2 * kSlabBytes;
constexpr uint32_t kOffScale = kOffRaw + kRawStages * kRawBytes;
// Tiles that are known in shared memory, found by a warp that walks ahead: (found by every
// decoder warp itself, a tile of experts cost some 1500 of 23000 cycles twice). Of each, in
// words: 2^exponent of its tokens; exponent * 2 + flag of its tokens; its weight rows'
// exponents; then the fields of Info.
constexpr int kInfos = 4;
constexpr int kInfoExp = kMaxTileM, kInfoRow = 2 * kMaxTileM, kInfoFields = 2 * kMaxTileM + kTileN;
struct Info {
  int m0, cnt, n0;  // as in Tile
  int row0;         // the CTA's first weight row among all matrices'
  int nkb, kb0, split;
  int special;      // some token is flagged, or two powers of two cannot be multiplied into one normal float
};
constexpr uint32_t kInfoBytes = kInfoFields * 4 + sizeof(Info);
constexpr uint32_t kOffInfo = kOffScale + kRawStages * kScaleStage;
constexpr uint32_t kOffRed = kOffInfo + kInfos * kInfoBytes;  // [512] floats
constexpr uint32_t kOffPre = kOffRed + kDec * 4;                     // [E + 1] tiles before the i-th expert
constexpr uint32_t kOffFirst = kOffPre + (LBQ_MAX_EXPERTS + 2) * 4;  // [E + 1] offsets, clamped
constexpr uint32_t kOffOrder = kOffFirst + (LBQ_MAX_EXPERTS + 2) * 4;  // [E] the i-th expert (16 bits)
constexpr uint32_t kOffBar = kOffOrder + LBQ_MAX_EXPERTS * 2;
constexpr uint32_t kBarBytes = 8 * (2 * kStages + 2 * kRawStages + 2 * kInfos + 5) + 8;  // and the TMEM slot
constexpr uint32_t kSmem = kOffBar + kBarBytes + 1024;
static_assert(kSmem <= 232448, "over the shared-memory limit");
constexpr unsigned kFaultX = 14, kFaultMma = 15, kFaultW = 16, kFaultDecode = 17, kFaultEpilogue = 18;

struct Args {
  int64_t K;
  int32_t N, M;              // rows of one matrix; token rows (sorted rows for experts)
  int32_t E, groups;         // matrices; row groups of one matrix
  int32_t tile_m, ntm, splits, kb_split;  // dense: tokens a tile, token tiles, K splits, blocks a split
  const int32_t* offsets;    // experts: rows of each (null: dense)
  const int32_t* slots;
  int32_t topk;
  int64_t T;
  const int* xexp;           // token row m was scaled by 2^-xexp[m]
  const int* xflag;          // 1: row m is recomputed in fp32
  const int* plan;           // experts: [E + 1] tiles before the i-th expert, [E] the i-th expert
  const int* wexp;           // weight row was scaled by 2^-wexp (rows padded to groups)
  const uint16_t* X;
  const uint8_t* codes;
  const uint16_t* scales;
  int64_t code_stride, scale_stride;
  uint16_t* Y;
  float* part;               // [splits][M][N] partial sums, or null
  unsigned* fault;
};

// What an earlier kernel of the stream may still be writing when this one starts (early) is
// read after the wait, from L2 or by plain loads: not through the read-only path, which
// __ldg takes for weights.
// Source row of sorted row r: its slot's token, or -1.
__device__ __forceinline__ int64_t source_row(const int32_t* slots, int topk, int64_t T, int64_t r) {
  if (slots) {
    const int32_t s = __ldcg(slots + r);
    r = s < 0 ? -1 : s / topk;
  }
  return r < T ? r : -1;
}

__device__ __forceinline__ int clamp_row(int v, int R) { return v < 0 ? 0 : (v > R ? R : v); }

// Token tiles of `cnt` rows: as few as fit, all alike up to 16 rows (none is empty: all
// but the last hold at most 256 rows each, and cnt is more than they can hold).
__device__ __forceinline__ int tiles_for(int cnt) { return (cnt + kMaxTileM - 1) / kMaxTileM; }
__device__ __forceinline__ int tile_rows(int cnt, int nt) { return ((cnt + nt - 1) / nt + 15) / 16 * 16; }

// ------------------------------------------------------------------- preparation
// The order of the experts' tiles, by one block: experts whose tiles have the most tokens
// come first, so that the tiles of a round, one a pair of CTAs, take about the same time
// and the last round's are the shortest. (2048 tokens x 8
// of 128 experts 149 us in the experts' order, 140 in this one; 4096 226 and 222. Equal
// shares of the time, each of tiles in a row, took 257: all activations are then in use at
// once, more than L2 holds.) A counting sort by sixteenths of a tile, stable.
__device__ __forceinline__ void plan_tiles(const Args& a, int ntn, int* __restrict__ plan) {
  constexpr int kClasses = kMaxTileM / 16 + 1, kChunks = LBQ_MAX_EXPERTS / 32;
  __shared__ int off[LBQ_MAX_EXPERTS + 1], hist[kChunks][kClasses], sum[kClasses];
  __shared__ short order[LBQ_MAX_EXPERTS];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, E = a.E;
  for (int e = tid; e <= E; e += 256) off[e] = clamp_row(__ldcg(a.offsets + e), a.M);
  for (int i = tid; i < kChunks * kClasses; i += 256) (&hist[0][0])[i] = 0;
  __syncthreads();
  // Offsets that descend somewhere would name rows twice, and more tiles than are counted
  // in 32 bits: no row then.
  bool down = false;
  for (int e = tid; e < E; e += 256) down = down || off[e + 1] < off[e];
  down = __syncthreads_or(down);
  auto class_of = [&](int e) {  // 0: the largest tiles; kClasses - 1: none; kClasses: no expert
    if (e >= E) return kClasses;
    const int rows = off[e + 1] - off[e];
    return kClasses - 1 - (rows > 0 ? tile_rows(rows, tiles_for(rows)) / 16 : 0);
  };
  auto peers_of = [](int k) {
    unsigned p = 0xffffffffu;
#pragma unroll
    for (int b = 0; b < 5; ++b) {
      const unsigned m = __ballot_sync(0xffffffffu, (k >> b) & 1);
      p &= (k >> b) & 1 ? m : ~m;
    }
    return p;
  };
  static_assert(kClasses < 32, "five bits");
  if (!down) {
    for (int e0 = 32 * warp; e0 < E; e0 += 256) {
      const int k = class_of(e0 + lane);
      const unsigned p = peers_of(k);
      if (k < kClasses && lane == __ffs(p) - 1) hist[e0 / 32][k] = __popc(p);
    }
    __syncthreads();
    if (tid < kClasses) {
      int run = 0;
      for (int c = 0; c < kChunks; ++c) {
        const int n = hist[c][tid];
        hist[c][tid] = run;
        run += n;
      }
      sum[tid] = run;
    }
    __syncthreads();
    for (int e0 = 32 * warp; e0 < E; e0 += 256) {
      const int k = class_of(e0 + lane);
      const unsigned p = peers_of(k);
      if (k < kClasses) {
        int at = hist[e0 / 32][k] + __popc(p & ((1u << lane) - 1u));
        for (int j = 0; j < k; ++j) at += sum[j];
        order[at] = static_cast<short>(e0 + lane);
      }
    }
  }
  __syncthreads();
  if (warp != 0) return;
  int run = 0;  // a running sum, 32 experts at a time
  for (int i0 = 0; i0 < E; i0 += 32) {
    const int i = i0 + lane, e = i < E && !down ? order[i] : 0;
    const int rows = i < E && !down ? off[e + 1] - off[e] : 0;
    const int c = rows > 0 ? tiles_for(rows) * ntn : 0;
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (i < E) {
      plan[i] = run + inc - c;
      plan[E + 1 + i] = e;
    }
    run += __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) plan[E] = run;
}

// Lanes that share a weight row group's scales: experts have many groups of few scales (128
// experts of 2048 x 1536, 512 tokens: 95.5 us with a warp a group, 89.8 with eight lanes).
__host__ __device__ inline int scale_lanes(int ns) { return ns <= 64 ? 8 : 32; }

// Rows are converted by a block each, or by a warp each where they are many and short (a
// block's launch, some 3 ns, is then more than a row's share of the time). Measured, whole
// products, a warp / a block: 512 x 2048, 600 rows 14.6 / 16.5 us, 2000 rows 16.5 / 26.8; 2048 x
// 1536, 1000 rows 19.9 / 18.5, 2500 rows 27.8 / 28.0; 5120 x 5120, 333 rows 34.9 / 26.8, 8192
// rows 337 / 333; 17408 x 2048, 2000 rows 146 / 116; the conversion of 32768 rows of 2048 45 /
// 107.
inline bool warp_a_row(int64_t K, int64_t rows) { return K <= 4096 && rows >= K; }

// The first blocks convert activation rows to fp16, kRow threads a row (exact power-of-two
// scaling, flag if not exact). An expert's rows are written once each, in their order, so that one
// copy brings a block of a tile: with the tokens converted once and the rows gathered by
// the product, 4096 tokens x 8 took 334 us by asynchronous copies of 16 bytes and 535 by
// four-row tensor copies, where this takes 222. The blocks behind take groups of four
// weight rows: the exponent that brings a row's largest scale to [2^11, 2^12).
template <int kRow>
__global__ void __launch_bounds__(256, 8)
    q4_prepare_kernel(const Args a, uint16_t* __restrict__ Xh, int* __restrict__ xexp,
                      int* __restrict__ xflag, int* __restrict__ wexp, int* __restrict__ plan, int ngroups,
                      int group) {
  pdl_launch_dependents();
  pdl_wait();
  if (a.offsets && blockIdx.x == gridDim.x - 1) {
    plan_tiles(a, (a.N + 2 * kTileN - 1) / (2 * kTileN), plan);
    return;
  }
  constexpr int kRows = 256 / kRow;  // rows a block
  __shared__ uint2 red[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t xblocks = (static_cast<int64_t>(a.M) + kRows - 1) / kRows;
  if (static_cast<int64_t>(blockIdx.x) >= xblocks) {
    const int ns = static_cast<int>(a.K / group), width = scale_lanes(ns), l = lane & (width - 1);
    const int64_t grp = (static_cast<int64_t>(blockIdx.x) - xblocks) * (256 / width) + threadIdx.x / width;
    bool used = grp < ngroups;
    if (used && a.offsets) {  // experts without rows need none
      const int e = static_cast<int>(grp) / a.groups;
      used = a.offsets[e] < a.offsets[e + 1];  // (cached: many blocks read the same)
    }
    uint32_t m01 = 0, m23 = 0;
    if (used) {
      const uint2* s = reinterpret_cast<const uint2*>(a.scales + grp * 4 * a.scale_stride);
#pragma unroll 4
      for (int e = l; e < ns; e += width) {
        const uint2 v = __ldg(s + e);
        m01 = __vmaxu2(m01, v.x & 0x7fff7fffu);
        m23 = __vmaxu2(m23, v.y & 0x7fff7fffu);
      }
    }
    for (int o = width / 2; o > 0; o >>= 1) {
      m01 = __vmaxu2(m01, __shfl_xor_sync(0xffffffffu, m01, o));
      m23 = __vmaxu2(m23, __shfl_xor_sync(0xffffffffu, m23, o));
    }
    if (used && l < 4) {
      const uint32_t h = (l & 2 ? m23 : m01) >> (16 * (l & 1)) & 0xffffu;
      // an infinite or NaN scale makes its row's outputs so whatever the exponent
      wexp[grp * 4 + l] = h == 0 ? 0 : (h >= 0x7c00u ? 4 : max(-30, ilogbf(f16_bits_to_f32(static_cast<uint16_t>(h))) - 11));
    }
    return;
  }
  // this thread's row and its place among the row's threads (kRow = 256: all on one row)
  const int64_t m = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kRow;
  const int u = threadIdx.x % kRow;
  if (m >= a.M) return;
  int64_t src = m;
  if (a.offsets) {
    if (m >= clamp_row(__ldcg(a.offsets + a.E), a.M)) return;
    src = source_row(a.slots, a.topk, a.T, m);
  }
  uint4* hr = reinterpret_cast<uint4*>(Xh + m * a.K);
  const int K8 = static_cast<int>(a.K / 8);
  if (src < 0) {  // a slot of no token: zeros
    for (int k = u; k < K8; k += kRow) hr[k] = make_uint4(0, 0, 0, 0);
    if (u == 0) xexp[m] = xflag[m] = 0;
    return;
  }
  const uint4* xr = reinterpret_cast<const uint4*>(a.X + src * a.K);
  auto lo = [](uint32_t w) { return __uint_as_float(w << 16); };
  auto hi = [](uint32_t w) { return __uint_as_float(w & 0xffff0000u); };
  // the row's first kKeep x kRow vectors stay in registers, what is behind is read twice
  constexpr int kKeep = 2;
  uint4 kept[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) kept[i] = u + i * kRow < K8 ? xr[u + i * kRow] : make_uint4(0, 0, 0, 0);
  // largest and smallest non-zero magnitude, as bf16 bits in both halves (the smallest less
  // one, so that zeros, 0xffff, come last; a magnitude's top bit is zero and is set while
  // the one is taken off, so that no half borrows from the other: borrowed bits hid a 2^-133
  // above a zero and flagged every row of zeros)
  uint32_t mb = 0, sb = 0xffffffffu;
  auto largest = [&](const uint4& v) {
    const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      mb = __vmaxu2(mb, w[i]);
      sb = __vminu2(sb, ((w[i] | 0x80008000u) - 0x00010001u) ^ 0x80008000u);
    }
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i) largest(kept[i]);
#pragma unroll 4
  for (int k = u + kKeep * kRow; k < K8; k += kRow) largest(xr[k]);
  uint32_t mag = max(mb & 0xffffu, mb >> 16), small = min(sb & 0xffffu, sb >> 16);
  mag = __reduce_max_sync(0xffffffffu, mag);
  small = __reduce_min_sync(0xffffffffu, small);
  if (kRow == 256) {
    if (lane == 0) red[warp] = make_uint2(mag, small);
    __syncthreads();
    for (int i = 0; i < 8; ++i) {
      mag = max(mag, red[i].x);
      small = min(small, red[i].y);
    }
  }
  const float mx = __uint_as_float(mag << 16);
  // max |x| 2^-e in [2^14, 2^15); a row of zeros, or with NaN or Inf (flagged below), as it is
  const int e = mag == 0 || mag >= 0x7f80u ? 0 : ilogbf(mx) - 14;
  // fp16 holds a bf16 value of 2^-17 or more exactly (its last bit is then at least fp16's
  // smallest step, 2^-24): a row is flagged when its smallest value, 31 powers of two below
  // the largest, may not be (or when it has NaN or Inf)
  const bool inexact = mag >= 0x7f80u || (small != 0xffffu && ilogbf(__uint_as_float((small + 1u) << 16)) - e < -17);
  auto pack = [](float a0, float a1) {
    const __half2 h = __floats2half2_rn(a0, a1);
    return *reinterpret_cast<const uint32_t*>(&h);
  };
  auto convert = [&](auto scale) {
    auto put = [&](int k, const uint4& v) {
      hr[k] = make_uint4(pack(scale(lo(v.x)), scale(hi(v.x))), pack(scale(lo(v.y)), scale(hi(v.y))),
                         pack(scale(lo(v.z)), scale(hi(v.z))), pack(scale(lo(v.w)), scale(hi(v.w))));
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (u + i * kRow < K8) put(u + i * kRow, kept[i]);
#pragma unroll 2
    for (int k = u + kKeep * kRow; k < K8; k += kRow) put(k, xr[k]);
  };
  if (-e >= -126 && -e <= 127) {
    const float f = __int_as_float((127 - e) << 23);
    convert([f](float x) { return x * f; });
  } else {
    convert([e](float x) { return ldexpf(x, -e); });
  }
  if (u == 0) {
    xexp[m] = e;
    xflag[m] = inexact ? 1 : 0;
  }
}

// ----------------------------------------------------------------------- the tiles
struct Tile {
  int e, n0;     // matrix, this CTA's first weight row (may lie behind the last)
  int m0, cnt;   // first token row, token rows
  int split, kb0, nkb;
};

// Tile `i` of the walk. Token tiles run fastest: the CTAs at work share weight tiles
// (read from HBM once), and all activations stay in L2.
__device__ __forceinline__ Tile tile_at(const Args& a, const int* pre, const int* off, const uint16_t* order,
                                        int ntn, int rank, int i) {
  Tile t;
  const int nkb = static_cast<int>(a.K / kTileK);
  if (!a.offsets) {
    const int tm = i % a.ntm, r = i / a.ntm;
    t.e = 0;
    t.n0 = (2 * (r % ntn) + rank) * kTileN;
    t.split = r / ntn;
    t.m0 = tm * a.tile_m;
    t.cnt = a.M - t.m0 < a.tile_m ? a.M - t.m0 : a.tile_m;
    t.kb0 = t.split * a.kb_split;
    t.nkb = nkb - t.kb0 < a.kb_split ? nkb - t.kb0 : a.kb_split;
    return t;
  }
  int lo = 0, hi = a.E;  // the expert's place: the last with pre[] <= i
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid; else hi = mid;
  }
  const int e = order[lo], r0 = off[e], r1 = off[e + 1];
  const int nt = tiles_for(r1 - r0), rows = tile_rows(r1 - r0, nt), l = i - pre[lo];
  t.e = e;
  t.n0 = (2 * (l / nt) + rank) * kTileN;
  t.m0 = r0 + (l % nt) * rows;
  t.cnt = r1 - t.m0 < rows ? r1 - t.m0 : rows;
  t.split = 0;
  t.kb0 = 0;
  t.nkb = nkb;
  return t;
}

// Tokens of the matrix instruction, and how many accumulators take its K steps in turn
// (an instruction on the previous one's accumulator waits for it; small ones are shorter
// than that wait).
__device__ __forceinline__ int mma_n(int cnt) { return cnt <= 16 ? 16 : (cnt + 15) / 16 * 16; }
__device__ __forceinline__ int accs_for(int n) { return n > 64 ? 1 : (n > 32 ? 2 : 4); }
// Where they lie: a tile of up to 128 tokens takes the half of the accumulators' columns
// that the tile before it does not, if that is as small, and starts while its sums are read.
__device__ __forceinline__ uint32_t acc_column(int n, uint32_t tile) { return n <= kMaxTileM / 2 ? (tile & 1) * (kMaxTileM / 2) : 0u; }

__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
  uint64_t d = static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
__device__ __forceinline__ uint32_t idesc_f16_m256(int n) {
  return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(256 >> 4) << 24);
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(d) : "r"(a), "r"(b), "r"(c));  // (a & b) | c
  return d;
}

// The eight codes of a word as fp16 pairs s (q - 8), in K order. 0x6400 | q is 1024 + q
// and 0x6400 | 16 q is 1024 + 16 q: q - 8 exactly after one subtraction or one fused
// multiply-add; the product with s is rounded to fp16.
__device__ __forceinline__ void decode_word(uint32_t w, __half2 s, uint32_t* out) {
  const __half2 c1032 = __half2half2(__ushort_as_half(0x6408));   // 1032
  const __half2 c16th = __half2half2(__ushort_as_half(0x2c00));   // 1/16
  const __half2 cm72 = __half2half2(__ushort_as_half(0xd480));    // -72
  const uint32_t w8 = w >> 8;
  const uint32_t v[4] = {and_or(w, 0x000f000fu, 0x64006400u), and_or(w, 0x00f000f0u, 0x64006400u),
                         and_or(w8, 0x000f000fu, 0x64006400u), and_or(w8, 0x00f000f0u, 0x64006400u)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __half2 h = *reinterpret_cast<const __half2*>(&v[j]);
    const __half2 q = (j & 1) ? __hfma2(h, c16th, cm72) : __hsub2(h, c1032);
    const __half2 p = __hmul2(q, s);
    out[j] = *reinterpret_cast<const uint32_t*>(&p);
  }
}

// fp32 recomputation of a tile's flagged tokens by all decoder threads d (four a weight
// row, each every fourth block of K); put(token, row, value) on threads d < kTileN. The
// flags are shared, so every warp comes to every meeting (a bounded wait, like all).
// All other warps of both CTAs may wait for its end, which takes 5 to 8 ns a token and
// weight of a row (256 tokens of K = 17408: 24 ms; of K = 2^21: 4.2 s): it beats in both,
// once a token.
template <int kG, typename Meet, typename Put>
__device__ __forceinline__ void fixup_flagged(const Args& a, const Info& t, const int* xe, float* red,
                                              int d, uint32_t beat, Meet meet, Put put) {
  const int row = d & (kTileN - 1), qtr = d / kTileN, n = t.n0 + row;
  const int64_t grow = t.row0 + row;
  for (int i = 0; i < t.cnt; ++i) {
    if (!(xe[i] & 1)) continue;
    if (d < 2)
      asm volatile("st.volatile.shared::cluster.b32 [%0], %1;" ::"r"(map_to_rank(beat, d)), "r"(beat_now()) : "memory");
    const int64_t src = a.offsets ? source_row(a.slots, a.topk, a.T, t.m0 + i) : t.m0 + i;
    float acc = 0.0f;
    if (n < a.N && src >= 0) {
      const uint16_t* x = a.X + src * a.K;
      for (int kb = t.kb0 + qtr; kb < t.kb0 + t.nkb; kb += 4) {
        for (int g = 0; g < kTileK / kG; ++g) {
          const float s = f16_bits_to_f32(__ldg(a.scales + g4_scale_elem(grow, kb * (kTileK / kG) + g, a.scale_stride)));
          float p = 0.0f;
          for (int w = 0; w < kG / 8; ++w) {
            const int64_t wi = static_cast<int64_t>(kb) * (kTileK / 8) + g * (kG / 8) + w;
            const uint32_t c = __ldg(reinterpret_cast<const uint32_t*>(a.codes + g4_word_byte(grow, wi, a.code_stride)));
#pragma unroll
            for (int q = 0; q < 8; ++q) {
              const int v = static_cast<int>((c >> (4 * ((q >> 1) + 4 * (q & 1)))) & 15u) - 8;
              p += static_cast<float>(v) * bf16_bits_to_f32(__ldcg(x + 8 * wi + q));
            }
          }
          acc += s * p;
        }
      }
    }
    red[qtr * kTileN + row] = acc;
    meet();
    if (d < kTileN && n < a.N)
      put(i, row, ((red[row] + red[kTileN + row]) + red[2 * kTileN + row]) + red[3 * kTileN + row]);
    meet();
  }
}

// v * 2^e with one rounding.
__device__ __forceinline__ float scale_pow2(float v, int e) {
  return (e >= -126 && e <= 127) ? v * __int_as_float((e + 127) << 23) : ldexpf(v, e);
}

template <int kG>
__global__ void __launch_bounds__(kThreads, 1)
    q4_tc_kernel(const __grid_constant__ XMaps tm_x, const __grid_constant__ CUtensorMap tm_w,
                 const __grid_constant__ CUtensorMap tm_s, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  unsigned char* sp = smem_raw + (base - smem_u32(smem_raw));
  int* pre = reinterpret_cast<int*>(sp + kOffPre);
  int* off = reinterpret_cast<int*>(sp + kOffFirst);
  uint16_t* order = reinterpret_cast<uint16_t*>(sp + kOffOrder);
  const uint32_t bars = base + kOffBar;
  const uint32_t full = bars, empty = full + 8 * kStages, fullR = empty + 8 * kStages,
                 emptyR = fullR + 8 * kRawStages, accum = emptyR + 8 * kRawStages, dfree = accum + 16,
                 meet = dfree + 16, fullI = meet + 8, emptyI = fullI + 8 * kInfos, tslot = emptyI + 8 * kInfos,
                 beat = tslot + 4;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto wait = [&](uint32_t bar, uint32_t parity, unsigned code, bool give_up = true) {
    // (a token of the largest K, 2^28, is recomputed in some 2 s)
    return mbar_wait(bar, parity, a.fault, code, give_up, 2 * kWaitLimitNs, beat);
  };
  if (tid == 0) {
    asm volatile("st.shared.b32 [%0], %1;" ::"r"(beat), "r"(0u) : "memory");
    for (int s = 0; s < kStages; ++s) {
      // the stage's four decoder warps of both CTAs, and the first CTA's activation lane
      mbar_init(full + 8 * s, 2 * kDec / 32 / kStages + 1);
      mbar_init(empty + 8 * s, 1);
    }
    for (int s = 0; s < kRawStages; ++s) {
      mbar_init(fullR + 8 * s, 1);
      mbar_init(emptyR + 8 * s, kChunkBlocks * kDec / 32 / kStages);
    }
    for (int s = 0; s < kInfos; ++s) {
      mbar_init(fullI + 8 * s, 1);
      mbar_init(emptyI + 8 * s, kDec / 32);
    }
    for (int s = 0; s < 2; ++s) {  // of even and odd tiles
      mbar_init(accum + 8 * s, 1);
      mbar_init(dfree + 8 * s, 2 * kDec / 32);
    }
    mbar_init(meet, kDec / 32);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc_pair(tslot, kTmemCols);
  pdl_wait();
  const int rank = static_cast<int>(cluster_rank());
  const int ntn = (a.N + 2 * kTileN - 1) / (2 * kTileN);
  if (a.offsets)
    for (int e = tid; e <= a.E; e += kThreads) {
      off[e] = clamp_row(__ldcg(a.offsets + e), a.M);
      pre[e] = __ldcg(a.plan + e);
      if (e < a.E) order[e] = static_cast<uint16_t>(__ldcg(a.plan + a.E + 1 + e));
    }
  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // the other CTA's barriers and tensor memory are ready too
  tc_fence_after_sync();
  const int total = a.offsets ? pre[a.E] : a.ntm * ntn * a.splits;
  // All 512 columns are allocated, so the allocation starts at column 0; a constant keeps
  // the MMA loop's addresses in uniform registers.
  constexpr uint32_t tmem = 0;
  const int first = static_cast<int>(blockIdx.x >> 1), step = static_cast<int>(gridDim.x >> 1);
  // the barriers the first CTA waits on for both
  const uint32_t full0 = map_to_rank(full, 0), dfree0 = map_to_rank(dfree, 0);

  if (warp == 0) {
    // ---------------- activations
    if (lane == 0) {
      uint32_t blk = 0;  // stages filled
      bool ok = true;
      for (int i = first; i < total && ok; i += step) {
        const Tile t = tile_at(a, pre, off, order, ntn, rank, i);
        const int half = mma_n(t.cnt) / 2, box = (half + kBoxStep - 1) / kBoxStep;
        const CUtensorMap* map = &tm_x.m[box - 1];
        for (int kb = 0; kb < (t.nkb + 1) / 2 * 2; ++kb, ++blk) {
          const uint32_t s = blk % kStages;
          if (!wait(empty + 8 * s, ((blk / kStages) & 1) ^ 1, kFaultX)) {
            ok = false;
            break;
          }
          if (kb == t.nkb) {  // an odd number of blocks: the last chunk's second stage stays unused
            if (rank == 0) mbar_arrive(full + 8 * s);
            continue;
          }
          if (rank == 0) mbar_arrive_expect_tx(full + 8 * s, static_cast<uint32_t>(box) * (2 * 2 * kBoxStep * 128));
          tma_load_3d_pair(base + kOffSlab + 2 * s * kSlabBytes, map, 0, t.m0 + rank * half, t.kb0 * 2 + 2 * kb, full0 + 8 * s);
        }
      }
      // every issued copy lands before the CTAs end (both halves complete on the first's barriers)
      if (rank == 0)
        for (uint32_t q = blk > kStages ? blk - kStages : 0; q < blk; ++q)
          wait(full + 8 * (q % kStages), (q / kStages) & 1, kFaultX, false);
    }
  } else if (warp == 1) {
    // ---------------- MMA issue: eight K = 16 steps a stage, one wait and one commit. The
    // whole warp walks the loop and one elected lane issues, so that the loop's values
    // stay in uniform registers (issued from a branch on lane 0, and with separate
    // barriers for weights and two activation slabs, a block took 0.74 us at any size).
    if (rank == 0) {
      uint32_t blk = 0, nt = 0;
      int before = 0;  // tokens of the tile before
      bool ok = true;
      for (int i = first; i < total && ok; i += step) {
        // (the tile's info stays until its epilogues, which come after its last instruction)
        ok = wait(fullI + 8 * (nt % kInfos), (nt / kInfos) & 1, kFaultMma);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const Info& t = *reinterpret_cast<const Info*>(sp + kOffInfo + (nt % kInfos) * kInfoBytes + kInfoFields * 4);
        const int n = mma_n(t.cnt), nacc = accs_for(n), nkb = t.nkb;
        const uint32_t acc = tmem + acc_column(n, nt);
        const uint32_t idesc = idesc_f16_m256(n);
        const uint32_t half_k = static_cast<uint32_t>((n / 2 + kBoxStep - 1) / kBoxStep) * (kBoxStep * 128 >> 4);
        // the accumulators are free once the tile before the last has been read, and the last
        // if one of the two is larger than half of them
        ok = wait(dfree + 8 * (nt & 1), ((nt >> 1) & 1) ^ 1, kFaultMma);
        if (ok && nt > 0 && (n > kMaxTileM / 2 || before > kMaxTileM / 2))
          ok = wait(dfree + 8 * ((nt & 1) ^ 1), ((nt - 1) >> 1) & 1, kFaultMma);
        before = n;
        for (int kb = 0; kb < (nkb + 1) / 2 * 2; ++kb, ++blk) {
          const uint32_t s = blk % kStages;
          if (ok) ok = wait(full + 8 * s, (blk / kStages) & 1, kFaultMma);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_fence_after_sync();
          if (elect_one()) {
            if (kb < nkb) {
              const uint32_t ta = tmem + kTmemA + 64u * s;
              const uint64_t bdesc = sw128_desc(base + kOffSlab + 2 * s * kSlabBytes);
#pragma unroll
              for (int ks = 0; ks < 8; ++ks)
                mma_f16_ts_pair(acc + static_cast<uint32_t>((ks & (nacc - 1)) * n), ta + 8u * ks,
                                bdesc + (ks >> 2) * half_k + 2u * (ks & 3), idesc,
                                (kb > 0 || ks >= nacc) ? 1u : 0u);
            }
            mma_commit_pair(empty + 8 * s);
          }
          __syncwarp();
        }
        if (elect_one()) mma_commit_pair(accum + 8 * (nt & 1));
        __syncwarp();
        ++nt;
      }
    }
  } else if (warp == 2) {
    // ---------------- packed weights and scales
    if (lane == 0) {
      prefetch_tmap(&tm_w);
      prefetch_tmap(&tm_s);
      constexpr uint32_t kScaleBytes = (kChunkBlocks * kTileK / kG) * 8 * (kTileN / 4);
      uint32_t c = 0;
      bool ok = true;
      for (int i = first; i < total && ok; i += step) {
        const Tile t = tile_at(a, pre, off, order, ntn, rank, i);
        const int g0 = t.e * a.groups + t.n0 / 4;
        for (int kb = t.kb0; kb < t.kb0 + t.nkb; kb += kChunkBlocks) {
          const uint32_t r = c % kRawStages;
          if (!wait(emptyR + 8 * r, ((c / kRawStages) & 1) ^ 1, kFaultW)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(fullR + 8 * r, kRawBytes + kScaleBytes);
          tma_load_2d(base + kOffRaw + r * kRawBytes, &tm_w, kb * (kTileK / 8) * 4, g0, fullR + 8 * r);
          tma_load_2d(base + kOffScale + r * kScaleStage, &tm_s, kb * (kTileK / kG) * 4, g0, fullR + 8 * r);
          ++c;
        }
      }
      for (uint32_t q = c > kRawStages ? c - kRawStages : 0; q < c; ++q)
        wait(fullR + 8 * (q % kRawStages), (q / kRawStages) & 1, kFaultW, false);
    }
  } else if (warp == 3) {
    // ---------------- what the decoders have to know of the tiles
    uint32_t k = 0;
    for (int i = first; i < total; i += step, ++k) {
      const Tile t = tile_at(a, pre, off, order, ntn, rank, i);
      const int row0 = t.e * a.groups * 4 + t.n0;
      const uint32_t s = k % kInfos;
      int* info = reinterpret_cast<int*>(sp + kOffInfo + s * kInfoBytes);
      int e[kMaxTileM / 32], f[kMaxTileM / 32], we[kTileN / 32];
#pragma unroll
      for (int x = 0; x < kMaxTileM / 32; ++x) {
        const int m = 32 * x + lane;
        e[x] = m < t.cnt ? __ldcg(a.xexp + t.m0 + m) : 0;
        f[x] = m < t.cnt ? __ldcg(a.xflag + t.m0 + m) : 0;
      }
#pragma unroll
      for (int x = 0; x < kTileN / 32; ++x)
        we[x] = t.n0 + 32 * x + lane < a.N ? __ldcg(a.wexp + row0 + 32 * x + lane) : 0;
      bool ok = wait(emptyI + 8 * s, ((k / kInfos) & 1) ^ 1, kFaultEpilogue);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      bool special = false;
#pragma unroll
      for (int x = 0; x < kMaxTileM / 32; ++x) {
        const int m = 32 * x + lane;
        info[m] = (e[x] + 127) << 23;
        info[kInfoExp + m] = 2 * e[x] + f[x];
        special = special || f[x] != 0 || e[x] < -85 || e[x] > 115;
      }
#pragma unroll
      for (int x = 0; x < kTileN / 32; ++x) info[kInfoRow + 32 * x + lane] = we[x];
      special = __any_sync(0xffffffffu, special);
      if (lane == 0)
        *reinterpret_cast<Info*>(info + kInfoFields) = {t.m0, t.cnt, t.n0, row0, t.nkb, t.kb0, t.split, special};
      __syncwarp();
      if (lane == 0) mbar_arrive(fullI + 8 * s);
    }
  } else if (warp >= 4) {
    // ---------------- decode: weight stage g belongs to warp group g (four warps, one
    // thread a weight row), which decodes every fourth block into it. The groups' chains
    // (wait for the codes, decode, wait for the stage, store) overlap; with all sixteen
    // warps on every block the chain's latency bounded the rate (0.88 us a block, 128 x 64)
    const int d = tid - 128, row = d & (kTileN - 1), grp = d >> 7;
    const int q = warp & 3;  // row = 32 q + lane
    float* red = reinterpret_cast<float*>(sp + kOffRed);
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    const uint32_t tA = lane_base + kTmemA + 64u * grp;
    constexpr uint32_t kScales = kTileK / kG;  // scales a block
    const uint32_t myword = base + kOffRaw + 4u * (static_cast<uint32_t>(row >> 2) * kGroupWords + (row & 3)) + 256u * (grp & 1);
    const uint32_t myscale = base + kOffScale + static_cast<uint32_t>(row >> 2) * (kChunkBlocks * kScales * 8) +
                             2u * (row & 3) + 8u * kScales * (grp & 1);
    bool ok = true;
    uint32_t tiles = 0, done_tiles = 0;  // begun, and epilogues finished
    uint32_t meetings = 0;    // of the decoder warps
    auto meeting = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(meet);
      if (ok) ok = wait(meet, meetings & 1, kFaultEpilogue);
      __syncwarp();
      ++meetings;
    };

    auto info_of = [&](uint32_t k) { return reinterpret_cast<const int*>(sp + kOffInfo + (k % kInfos) * kInfoBytes); };
    // of the oldest tile without one (its info is there: the warp has decoded for it)
    auto epilogue = [&]() {
      const int* const info = info_of(done_tiles);
      const Info& t = *reinterpret_cast<const Info*>(info + kInfoFields);
      const float* xs = reinterpret_cast<const float*>(info);
      const int* xe = info + kInfoExp;
      const int n = mma_n(t.cnt), nacc = accs_for(n);
      const int nr = t.n0 + 32 * q + lane;
      const int we = info[kInfoRow + 32 * q + lane];
      const float ws = __int_as_float((127 + we) << 23);  // 2^we (we is in -30 .. 4)
      const bool special = ok && t.special;
      if (ok) ok = wait(accum + 8 * (done_tiles & 1), (done_tiles >> 1) & 1, kFaultEpilogue);
      __syncwarp();
      tc_fence_after_sync();
      // this warp's columns 16 grp + 64 c + (0..15), the accumulators summed in order
      const uint32_t acc = lane_base + acc_column(n, done_tiles);
      auto read16 = [&](int c0, uint32_t (&v)[16]) {
        tmem_ld16(acc + static_cast<uint32_t>(c0), v);
        tmem_ld_wait();
        for (int j = 1; j < nacc; ++j) {
          uint32_t u[16];
          tmem_ld16(acc + static_cast<uint32_t>(j * n + c0), u);
          tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 16; ++x) v[x] = __float_as_uint(__uint_as_float(v[x]) + __uint_as_float(u[x]));
        }
      };
      auto release = [&]() {  // the accumulators may be overwritten
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(dfree0 + 8 * (done_tiles & 1));
      };
      if (!special && !a.part) {
        // all columns are read, scaled and rounded first, so that the tensor cores wait for
        // the reads only; the stores run beside the next tile's instructions
        uint32_t y[4][8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int c0 = 16 * grp + 64 * c;
          if (c0 >= n) break;
          uint32_t v[16];
          read16(c0, v);
#pragma unroll
          for (int x = 0; x < 16; x += 2) {
            const float2 f = *reinterpret_cast<const float2*>(xs + c0 + x);
            y[c][x / 2] = f32_to_bf16_bits(__uint_as_float(v[x]) * (f.x * ws)) |
                          static_cast<uint32_t>(f32_to_bf16_bits(__uint_as_float(v[x + 1]) * (f.y * ws))) << 16;
          }
        }
        release();
        if (ok && nr < a.N) {
          uint16_t* yp = a.Y + static_cast<int64_t>(t.m0) * a.N + nr;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int c0 = 16 * grp + 64 * c;
            if (c0 >= t.cnt) break;
            uint16_t* yc = yp + static_cast<int64_t>(c0) * a.N;
#pragma unroll
            for (int x = 0; x < 16; ++x)
              if (c0 + x < t.cnt) yc[static_cast<int64_t>(x) * a.N] = static_cast<uint16_t>(y[c][x / 2] >> (16 * (x & 1)));
          }
        }
      } else {
        float* const part = a.part ? a.part + static_cast<int64_t>(t.split) * a.M * a.N : nullptr;
        for (int c0 = 16 * grp; c0 < n; c0 += 64) {
          uint32_t v[16];
          read16(c0, v);
          if (!ok || nr >= a.N) continue;
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int m = c0 + x;
            if (m < t.cnt && !(xe[m] & 1)) {
              const float y = special ? scale_pow2(__uint_as_float(v[x]), (xe[m] >> 1) + we) : __uint_as_float(v[x]) * (xs[m] * ws);
              const int64_t o = static_cast<int64_t>(t.m0 + m) * a.N + nr;
              if (part) part[o] = y;
              else a.Y[o] = f32_to_bf16_bits(y);
            }
          }
        }
        release();
        if (special)
          fixup_flagged<kG>(a, t, xe, red, d, beat, meeting, [&](int m, int r, float y) {
            if (!ok) return;
            const int64_t o = static_cast<int64_t>(t.m0 + m) * a.N + t.n0 + r;
            if (part) part[o] = y;
            else a.Y[o] = f32_to_bf16_bits(y);
          });
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(emptyI + 8 * (done_tiles % kInfos));
      ++done_tiles;
    };
    uint32_t chunk0 = 0;  // chunks of the tiles before
    for (int i = first; i < total; i += step, ++tiles) {
      if (ok) ok = wait(fullI + 8 * (tiles % kInfos), (tiles / kInfos) & 1, kFaultEpilogue);
      __syncwarp();
      const int* const info = info_of(tiles);
      const int we = ok ? info[kInfoRow + row] : 0;
      const int nkb = ok ? reinterpret_cast<const Info*>(info + kInfoFields)->nkb : 0;
      // 2^-we as two fp16 factors (we is in -30 .. 4)
      const int we1 = we < -15 ? -15 : we;
      const __half2 f1 = __half2half2(__ushort_as_half(static_cast<uint16_t>((15 - we1) << 10)));
      const __half2 f2 = __half2half2(__ushort_as_half(static_cast<uint16_t>((15 - (we - we1)) << 10)));
      // the tile's blocks are dealt to the groups two by two: chunk c (two blocks) to the
      // groups 0 and 1 or 2 and 3
      const uint32_t nch = static_cast<uint32_t>(nkb + kChunkBlocks - 1) / kChunkBlocks;
      for (uint32_t c = ((chunk0 & 1) ^ static_cast<uint32_t>(grp >> 1)); c < nch; c += 2) {
        const uint32_t r = (chunk0 + c) % kRawStages;
        if (ok) ok = wait(fullR + 8 * r, ((chunk0 + c) / kRawStages) & 1, kFaultDecode);
        __syncwarp();
        uint32_t w[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) w[x] = lds32(myword + r * kRawBytes + 16u * x);
        uint32_t sc[kScales];
#pragma unroll
        for (int x = 0; x < static_cast<int>(kScales); ++x) sc[x] = lds16(myscale + r * kScaleStage + 8u * x);
        __syncwarp();
        if (lane == 0) mbar_arrive(emptyR + 8 * r);
        // (an odd number of blocks: the last chunk's second one is zeros to its group)
        const uint32_t use = (chunk0 + c) / 2;  // the stage's uses before this one
        if (ok) ok = wait(empty + 8 * grp, (use & 1) ^ 1, kFaultDecode);
        __syncwarp();
        tc_fence_after_sync();
#pragma unroll
        for (int x = 0; x < 4; ++x) {  // 32 weights at a time
          const __half2 sx = __half2half2(__ushort_as_half(static_cast<uint16_t>(sc[kG == 32 ? x : 0])));
          const __half2 s2 = __hmul2(__hmul2(sx, f1), f2);
          uint32_t hv[16];
#pragma unroll
          for (int y = 0; y < 4; ++y) decode_word(w[4 * x + y], s2, hv + 4 * y);
          tmem_st16(tA + 16u * x, hv);
        }
        tmem_st_wait();
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(full0 + 8 * grp);
        // Tiles that ended before this block: their epilogues. The stages then hold later
        // blocks, so the tensor cores go on as soon as the accumulators are read. (Each
        // group comes here after its first block behind the tile, which waits only for
        // blocks of that tile or earlier ones: no circle of waits.)
        while (done_tiles < tiles) epilogue();
      }
      chunk0 += nch;
    }
    while (done_tiles < tiles) epilogue();
  }

  tc_fence_before_sync();
  __syncthreads();
  cluster_sync_all();  // neither CTA leaves while the other's MMAs or arrivals reach into it
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// Y = bf16(sum over splits of the fp32 partial products), splits in order; four outputs a
// thread (kVec: their number is a multiple of four and Y is aligned to them).
template <bool kVec>
__global__ void __launch_bounds__(256) q4_split_sum_kernel(const float* __restrict__ part, int splits,
                                                           int64_t MN, uint16_t* __restrict__ Y) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t i = 4 * (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x);
  if (i >= MN) return;
  if (kVec) {
    float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
    for (int z = 0; z < splits; ++z) {
      const float4 v = __ldcg(reinterpret_cast<const float4*>(part + z * MN + i));
      sum.x += v.x;
      sum.y += v.y;
      sum.z += v.z;
      sum.w += v.w;
    }
    const uint32_t lo = f32_to_bf16_bits(sum.x) | (static_cast<uint32_t>(f32_to_bf16_bits(sum.y)) << 16);
    const uint32_t hi = f32_to_bf16_bits(sum.z) | (static_cast<uint32_t>(f32_to_bf16_bits(sum.w)) << 16);
    *reinterpret_cast<uint2*>(Y + i) = make_uint2(lo, hi);
  } else {
    for (int64_t j = i; j < i + 4 && j < MN; ++j) {
      float sum = 0.0f;
      for (int z = 0; z < splits; ++z) sum += __ldcg(part + z * MN + j);
      Y[j] = f32_to_bf16_bits(sum);
    }
  }
}

struct Plan {
  int tile_m, ntm, splits, kb_split;
};

// Dense: how many token tiles, and whether K is split where the tiles leave half of the
// pairs of SMs idle or more. Modelled time in us: rounds of tiles over the pairs, each 1.5
// and its blocks; a block of 128 K takes 0.36 up to some 120 tokens, where the decoding and
// the reading of the weight operand bound it, and 0.085 + 0.0023 a token beyond (measured:
// 0.42 at 144, 0.57 at 208, 0.68 at 256); a split 3 and 3.3 a million partial sums, for their
// way to memory and back. Over 84 sizes (40 to 1500 tokens, 512 x 8192 to 5120 x 34816) the
// plan is within a few percent of the best of all; 256 tokens of 5120 x 7168: one tile of
// tokens 39.1 us, one with K in two 37.9, two tiles 27.8.
Plan plan_for(const lbq_weights* w, int64_t M) {
  Plan p = {};
  const int64_t ntn = (w->N + 2 * kTileN - 1) / (2 * kTileN), pairs = sm_count() / 2;
  const int nkb = static_cast<int>(w->K / kTileK), most = (nkb + 3) / 4;  // splits: at least four blocks each
  const int64_t least = (M + kMaxTileM - 1) / kMaxTileM;
  double best = 0.0;
  for (int64_t nt = least; nt <= 4 * least && nt <= (M + 15) / 16; ++nt) {
    const int64_t rows = ((M + nt - 1) / nt + 15) / 16 * 16, ntm = (M + rows - 1) / rows, tiles = ntm * ntn;
    int splits = tiles < pairs ? static_cast<int>(pairs / tiles) : 1;
    if (splits > most) splits = most;
    const int kb_split = ((nkb + splits - 1) / splits + kChunkBlocks - 1) / kChunkBlocks * kChunkBlocks;
    splits = (nkb + kb_split - 1) / kb_split;
    const double r = static_cast<double>(rows), block = 0.35 + 0.0002 * r, large = 0.085 + 0.0023 * r;
    const double cost = static_cast<double>((tiles * splits + pairs - 1) / pairs) *
                            (1.5 + kb_split * (block > large ? block : large)) +
                        (splits > 1 ? 3.0 + 3.3e-6 * splits * static_cast<double>(M) * static_cast<double>(w->N) : 0.0);
    if (nt == least || cost < best) {
      best = cost;
      p = {static_cast<int>(rows), static_cast<int>(ntm), splits, kb_split};
    }
  }
  return p;
}

inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

struct Scratch {
  size_t xh, xexp, xflag, wexp, plan, part, total;
};
Scratch scratch_for(const lbq_weights* w, int64_t rows, int E, size_t part_floats) {
  Scratch s;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes, 1024);
    return at;
  };
  s.xh = take(static_cast<size_t>(rows) * w->K * 2);
  s.xexp = take(static_cast<size_t>(rows) * 4);
  s.xflag = take(static_cast<size_t>(rows) * 4);
  s.wexp = take(static_cast<size_t>(E) * g4_rows(w->N) * 4);
  s.plan = take((2 * static_cast<size_t>(E) + 1) * 4);
  s.part = take(part_floats * 4);
  s.total = o;
  return s;
}

template <int kG>
cudaError_t configure() {
  static PerDevice<bool> configured;
  bool done = false;
  return configured.get(
      [](int, bool* v) {
        *v = true;
        return cudaFuncSetAttribute(q4_tc_kernel<kG>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(kSmem));
      },
      &done);
}

template <int kG>
cudaError_t launch(const lbq_weights* w, const Plan& plan, const lbq_expert_rows* er, const uint16_t* X,
                   int64_t rows, uint16_t* Y, char* ws, cudaStream_t s) {
  cudaError_t e = configure<kG>();
  if (e != cudaSuccess) return e;
  auto encode = tensor_map_encoder();
  if (!encode) return cudaErrorInvalidValue;
  const int E = er ? er->E : 1;
  const int64_t ng = (w->N + 3) / 4;
  const size_t part_floats = plan.splits > 1 ? static_cast<size_t>(plan.splits) * rows * w->N : 0;
  const Scratch sc = scratch_for(w, rows, E, part_floats);
  Args a = {};
  a.K = w->K;
  a.N = static_cast<int32_t>(w->N);
  a.M = static_cast<int32_t>(rows);
  a.E = E;
  a.groups = static_cast<int32_t>(ng);
  a.tile_m = plan.tile_m;
  a.ntm = plan.ntm;
  a.splits = plan.splits;
  if (er) {
    a.offsets = er->offsets;
    a.slots = er->slots;
    a.topk = er->topk;
    a.T = er->T;
  }
  uint16_t* Xh = reinterpret_cast<uint16_t*>(ws + sc.xh);
  int* xexp = reinterpret_cast<int*>(ws + sc.xexp);
  int* xflag = reinterpret_cast<int*>(ws + sc.xflag);
  int* wexp = reinterpret_cast<int*>(ws + sc.wexp);
  a.xexp = xexp;
  a.xflag = xflag;
  a.wexp = wexp;
  int* tiles = reinterpret_cast<int*>(ws + sc.plan);
  a.plan = tiles;
  a.X = X;
  a.codes = static_cast<const uint8_t*>(w->codes);
  a.scales = static_cast<const uint16_t*>(w->scales);
  a.code_stride = w->code_stride;
  a.scale_stride = w->scale_stride;
  a.Y = Y;
  a.part = part_floats ? reinterpret_cast<float*>(ws + sc.part) : nullptr;
  a.fault = lbq_fault_word();
  if (!a.fault) return cudaErrorInvalidDevicePointer;

  XMaps tx;
  CUtensorMap tw, ts;
  const cuuint32_t estr[2] = {1, 1};
  auto map = [&](CUtensorMap* m, CUtensorMapDataType dt, void* p, cuuint64_t cols, cuuint64_t n, cuuint64_t pitch,
                 cuuint32_t bx, cuuint32_t by, CUtensorMapSwizzle sw) {
    const cuuint64_t dims[2] = {cols, n};
    const cuuint64_t strides[1] = {pitch};
    const cuuint32_t box[2] = {bx, by};
    return encode(m, dt, 2, p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  // (rows of weights end with K: what a chunk holds behind it arrives as zeros, not from the
  // padding or from behind the last group)
  const cuuint64_t G = static_cast<cuuint64_t>(E) * ng, cw = static_cast<cuuint64_t>(w->K / 2),
                   se = static_cast<cuuint64_t>(w->K / kG) * 4;
  // (dense: only the boxes of the full and the last token tile are used)
  const int64_t last = rows - static_cast<int64_t>(plan.ntm - 1) * plan.tile_m;
  auto box_of = [](int64_t cnt) { return static_cast<int>((((cnt + 15) / 16 * 16) / 2 + kBoxStep - 1) / kBoxStep) - 1; };
  for (int i = 0; i < kBoxes; ++i) {
    if (!er && i != box_of(plan.tile_m) && i != box_of(last)) continue;
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(w->K / 64)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(w->K) * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>((i + 1) * kBoxStep), 2};
    const cuuint32_t estr3[3] = {1, 1, 1};
    if (encode(&tx.m[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, Xh, dims, strides, box, estr3,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (!map(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT32, const_cast<void*>(w->codes), cw, G,
           static_cast<cuuint64_t>(w->code_stride) * 4, kGroupWords, kTileN / 4,
           CU_TENSOR_MAP_SWIZZLE_NONE) ||
      !map(&ts, CU_TENSOR_MAP_DATA_TYPE_UINT16, const_cast<void*>(w->scales), se, G,
           static_cast<cuuint64_t>(w->scale_stride) * 8,
           (kChunkBlocks * kTileK / kG) * 4, kTileN / 4, CU_TENSOR_MAP_SWIZZLE_NONE))
    return cudaErrorInvalidValue;

  a.kb_split = plan.kb_split;
  const int per_block = 256 / scale_lanes(static_cast<int>(w->K / kG));
  const unsigned wblocks = static_cast<unsigned>((static_cast<int64_t>(E) * ng + per_block - 1) / per_block);
  const int ngroups = static_cast<int>(E * ng);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  const bool many = warp_a_row(w->K, rows);
  cfg.gridDim = dim3(static_cast<unsigned>(many ? (rows + 7) / 8 : rows) + wblocks + (er ? 1 : 0));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, many ? q4_prepare_kernel<32> : q4_prepare_kernel<256>, a, Xh, xexp, xflag, wexp, tiles, ngroups, kG);
  if (e != cudaSuccess) return e;
  const int64_t ntn = (w->N + 2 * kTileN - 1) / (2 * kTileN), pairs = sm_count() / 2;
  // experts: at most rows / 256 + E token tiles
  const int64_t most = er ? (rows / kMaxTileM + E) * ntn : static_cast<int64_t>(plan.ntm) * ntn * plan.splits;
  cfg.gridDim = dim3(2 * static_cast<unsigned>(most < pairs ? most : pairs));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, q4_tc_kernel<kG>, tx, tw, ts, a);
  if (e != cudaSuccess || plan.splits == 1) return e;
  const int64_t MN = rows * w->N;
  cfg.gridDim = dim3(static_cast<unsigned>((MN + 1023) / 1024));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  const bool vec = MN % 4 == 0 && (reinterpret_cast<uintptr_t>(Y) & 7) == 0;
  return cudaLaunchKernelEx(&cfg, vec ? q4_split_sum_kernel<true> : q4_split_sum_kernel<false>,
                            static_cast<const float*>(a.part), plan.splits, MN, Y);
}

}  // namespace

// Partial sums of the batches of up to M tokens that plan_for may split: at most pairs /
// tiles splits, with at least a token tile for every kMaxTileM tokens. (A plan of few tokens
// may need more of them than one of many: a workspace for M tokens serves all batches up to
// M.)
static size_t most_part_floats(const lbq_weights* w, int64_t M) {
  const int64_t ntn = (w->N + 2 * kTileN - 1) / (2 * kTileN), pairs = sm_count() / 2;
  const int64_t most = (w->K / kTileK + 3) / 4;
  int64_t floats = 0;
  for (int64_t c = 1; c <= (M + kMaxTileM - 1) / kMaxTileM && 2 * c * ntn <= pairs; ++c) {
    const int64_t splits = std::min(pairs / (c * ntn), most), rows = std::min<int64_t>(M, c * kMaxTileM);
    if (splits > 1) floats = std::max(floats, splits * rows * w->N);
  }
  return static_cast<size_t>(floats);
}

// [64 KB left alone: the counter rule][fp16 X][exponents, flags][weight exponents][tile order][partials]
size_t lbq_q4_tc_workspace(const lbq_weights* w, int64_t M) {
  return std::max(lbq_q4_few_workspace(8), kWsCounterBytes + scratch_for(w, M, 1, most_part_floats(w, M)).total);
}

cudaError_t lbq_launch_q4_tc(const lbq_weights* w, const uint16_t* X, int64_t M, uint16_t* Y, void* ws,
                             cudaStream_t s) {
  const Plan p = plan_for(w, M);
  char* base = static_cast<char*>(ws) + kWsCounterBytes;
  return w->fmt == LBQ_Q4G32 ? launch<32>(w, p, nullptr, X, M, Y, base, s)
                             : launch<128>(w, p, nullptr, X, M, Y, base, s);
}

size_t lbq_q4_expert_tc_workspace(const lbq_weights* w, int32_t E, int64_t R) {
  return std::max(lbq_q4_few_workspace(8), kWsCounterBytes + scratch_for(w, R, E, 0).total);
}

cudaError_t lbq_launch_q4_expert_tc(const lbq_weights* w, const lbq_expert_rows& r, void* ws, cudaStream_t s) {
  const Plan p = {kMaxTileM, 1, 1, static_cast<int>(w->K / kTileK)};
  char* base = static_cast<char*>(ws) + kWsCounterBytes;
  return w->fmt == LBQ_Q4G32 ? launch<32>(w, p, &r, r.X, r.R, r.Y, base, s)
                             : launch<128>(w, p, &r, r.X, r.R, r.Y, base, s);
}
