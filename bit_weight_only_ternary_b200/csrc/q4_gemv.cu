// q4_gemv.cu -- 4-bit products of few tokens: y[m][n] = sum_k s[n][k/g] (q[n][k] - 8) x[m][k],
// for a list of products (one token), one matrix and a few tokens, or a matrix per expert.
// Bound: the bytes of the packed weights, with the decoding close behind.
//
// Work. A tile is 32 weight rows (eight groups of four) x up to 8 tokens over all of K;
// its chunks are 128 of K (2 KB of codes). All tiles' chunks lie in one line, cut into
// equal runs, one a warp: however many rows a product has, every SM streams until the end,
// and a warp adds up its stretch of K alone. It streams through slots of shared memory
// of its own that asynchronous copies fill ahead, across tiles. A tile that lies in one
// warp's run is stored by the warp; the parts of a tile that several warps share are
// joined in K order, once, when the CTA's runs are done; where the CTA's runs end inside a
// tile, its part goes to the workspace and the last of the tile's CTAs to get there adds
// the parts in K order. Every order of sums is fixed, so results do not depend on timing.
// (A CTA a tile, its warps taking chunks in turn and two chunks ahead in registers, took
// 50 us for a 27B layer; the warps of a persistent CTA joined at every tile 47 us.)
//
// Arithmetic. A 16-byte load brings one 32-bit word (eight neighbouring weights) of four
// rows. Lane (g, t) = (lane / 4, lane % 4) reads word 4 s + t of row group g, which is, up
// to the order of rows and of K, the weight operand of m16n8k16 matrix instructions: rows
// 4g and 4g+1 are rows g and g+8 of a first tile, 4g+2 and 4g+3 of a second, and a word's
// eight weights are the lane's K values of two instructions. The activations need only
// the same order of K: lane (g, t) reads the eight activations of its word for token g. A
// code becomes a bf16 integer without a conversion: 0x4300 | q is 128 + q, minus 136 is
// q - 8, both exact. Products of these integers with bf16 activations are exact in fp32,
// sums are fp32, and the group's scale multiplies the group's sum in fp32: nothing is
// rounded to fewer bits before the final bf16 (or fp32) store. (Summing 128 + q and
// taking 136 sum x off at the end would save the subtractions, but an activation on a
// zero weight would then leave its rounding error behind.)
#include <algorithm>

#include "lbq_common.cuh"
#include "sm100_async.cuh"

namespace {

using namespace lbq;

// One CTA an SM. Twenty-four warps in three CTAs took 43 us for a 27B layer (the CTAs of an
// SM advanced unevenly, 24 to 37 us), 24 in one CTA 41, 12 in one 40.5, 16 in one 39: more
// bytes in flight fill longer at the start and drain longer at the end.
constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kRowTile = 32;
// Asynchronous copies global -> shared of this thread's own bytes (L1 is bypassed for 16).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kLeft>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}

// Pair j of a word's codes (weights 2j, 2j+1) as two bf16 integers q - 8.
__device__ __forceinline__ uint32_t q4_pair(uint32_t w, int j) {
  uint32_t v, r;
  // ((w >> 4 j) & 0x000f000f) | 0x43004300, 128 + q twice, as one three-input operation
  // (left to the compiler it became two, with an immediate each)
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(v) : "r"(w >> (4 * j)), "r"(0x000f000fu), "r"(0x43004300u));
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(0x43084308u));  // - 136
  return r;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b: the first instruction of a group's sum.
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Division by a number the host knows: a product with ceil(2^(31 + l) / d), l = ceil(log2 d),
// and a shift, exact for 0 <= n < 2^31 (the product's error is below n d / 2^(31 + l) / d <
// 1 / d). A run's start has half a dozen divisions one after another, and a division by a
// variable takes some hundred cycles.
struct Div {
  uint32_t d, mul;
  int shift;
  Div() = default;
  explicit Div(int64_t v) : d(static_cast<uint32_t>(v)) {
    int l = 0;
    while ((int64_t{1} << l) < v) ++l;
    shift = 31 + l;
    mul = static_cast<uint32_t>(((uint64_t{1} << shift) + v - 1) / v);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * mul) >> shift);
  }
  __device__ __forceinline__ int64_t wide(int64_t n) const {  // any n >= 0
    return (n >> 31) == 0 ? (*this)(static_cast<int>(n)) : n / d;
  }
};

// a / b for a >= 0, b > 0 of any size: in 32 bits where they fit.
__device__ __forceinline__ int64_t quot(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// ---------------------------------------------------------------- where the tiles are
// A source gives the tiles of its products (or experts): tiles and chunks of product p,
// the lane's pointers into tile i, and where its outputs go.
struct LanePtr {
  const uint8_t* w;        // the tile's first row group's codes
  const uint16_t* s;       // and scales
  int64_t gcode;           // from one row group to the next
  int32_t gscale;
  int groups;              // row groups of the tile that exist (of 8)
  const uint16_t* x;       // its token's activations + 8 t; null: no token, or (zero) zeros
  const uint16_t* x0;      // where x stood at chunk 0 of the tile
  bool zero;
};

struct Q4Prod {
  const uint8_t* codes;
  const uint16_t* scales;
  const uint16_t* x;   // [M][K]
  void* y;             // bf16 (or fp32) [M][N]
  int64_t q0;          // chunks of the products before
  int64_t gcode;       // code bytes per group of four rows
  int32_t gscale;      // scales per group of four rows
  int32_t N;           // rows
  Div nc;              // chunks of a tile
};

template <int kCap>
struct Q4List {
  int64_t chunks;
  int64_t share;       // chunks a CTA; the first `extra` CTAs take one more
  int32_t extra;
  Div ntok;            // token tiles
  float* part;         // workspace: parts of tiles cut by a run's end
  unsigned* count;     // arrivals on such a tile (zero before and after)
  int32_t n, M;
  Q4Prod p[kCap];
};

template <int kCap, int kTok, bool kF32>
struct ListSource {
  static constexpr bool kZeros = false;
  static constexpr bool kWarpFind = false;  // (see ExpertSource)
  static constexpr bool kEarly = true;  // the list and the weights are known before the previous kernel ends
  const Q4List<kCap>& a;
  __device__ __forceinline__ int64_t chunks() const { return a.chunks; }
  __device__ __forceinline__ int64_t start(int p) const { return a.p[p].q0; }
  __device__ __forceinline__ const Div& nc(int p) const { return a.p[p].nc; }
  __device__ __forceinline__ int64_t share(int) const { return a.share; }
  __device__ __forceinline__ int extra(int) const { return a.extra; }
  __device__ __forceinline__ int ntok() const { return kTok == 1 ? 1 : static_cast<int>(a.ntok.d); }
  __device__ __forceinline__ int tiles(int p) const { return (a.p[p].N + kRowTile - 1) / kRowTile * ntok(); }
  __device__ __forceinline__ int next(int p) const { return p + 1; }
  __device__ __forceinline__ int find(int64_t q) const {
    int lo = 0;
    if (kCap > 1) {
      int hi = a.n;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.p[mid].q0 <= q) lo = mid; else hi = mid;
      }
    }
    return lo;
  }
  __device__ __forceinline__ void point(int p, int i, int lane, bool, LanePtr& l) const {
    const Q4Prod& P = a.p[p];
    const int g = lane >> 2, t = lane & 3, ng = (P.N + 3) >> 2;
    const int rt = kTok == 1 ? i : a.ntok(i), m = (i - rt * ntok()) * kTok + g;  // token tiles run fastest
    const int64_t grp = rt * (kRowTile / 4);
    l.w = P.codes + grp * P.gcode;
    l.s = P.scales + grp * P.gscale;
    l.gcode = P.gcode;
    l.gscale = P.gscale;
    l.groups = ng - static_cast<int>(grp);
    const int64_t K = static_cast<int64_t>(P.nc.d) * kQ4Chunk;
    l.x0 = kTok == 1 ? P.x + 8 * lane : (g < kTok && m < a.M ? P.x + m * K + 8 * t : nullptr);
    l.zero = false;
  }
  __device__ __forceinline__ void store(int p, int i, int m, int r, float v) const {
    const Q4Prod& P = a.p[p];
    const int rt = kTok == 1 ? i : a.ntok(i), row = rt * kRowTile + r;
    m += (i - rt * ntok()) * kTok;
    if (m >= a.M || row >= P.N) return;
    const int64_t o = static_cast<int64_t>(m) * P.N + row;
    if (kF32) static_cast<float*>(P.y)[o] = v;
    else static_cast<uint16_t*>(P.y)[o] = f32_to_bf16_bits(v);
  }
};

struct Q4Experts {
  const uint8_t* codes;
  const uint16_t* scales;
  int64_t gcode, ecode, escale;  // code bytes per group, per expert; scales per expert
  int32_t gscale, N;
  Div nc, ntn, topk;             // chunks of a tile, row tiles
  lbq_expert_rows r;
  float* part;
  unsigned* count;
};

// Tiles of expert e: its token tiles, each with all row tiles behind one another (so the
// lanes' token rows, found through the slots, change rarely).
template <int kTok>
struct ExpertSource {
  static constexpr bool kZeros = true;  // slots may name no token
  static constexpr bool kWarpFind = true;  // find() is the whole warp's, for one q
  static constexpr bool kEarly = false;
  const Q4Experts& a;
  const int* off;  // [E + 1] first rows, clamped (shared memory)
  const int* pre;  // [E + 1] tiles of the experts before
  __device__ __forceinline__ int ntn() const { return static_cast<int>(a.ntn.d); }
  __device__ __forceinline__ int64_t chunks() const { return static_cast<int64_t>(pre[a.r.E]) * a.nc.d; }
  __device__ __forceinline__ int64_t share(int grid) const { return quot(chunks(), grid); }
  __device__ __forceinline__ int extra(int grid) const { return static_cast<int>(chunks() - share(grid) * grid); }
  __device__ __forceinline__ int64_t start(int e) const { return static_cast<int64_t>(pre[e]) * a.nc.d; }
  __device__ __forceinline__ const Div& nc(int) const { return a.nc; }
  __device__ __forceinline__ int tiles(int e) const { return pre[e + 1] - pre[e]; }
  __device__ __forceinline__ int next(int e) const {
    do ++e; while (e < a.r.E && pre[e + 1] == pre[e]);
    return e;
  }
  __device__ __forceinline__ int find(int64_t q) const {
    // the last expert with pre[e] <= tile (the ones before it may be empty): one count, 32
    // experts at a time (a search by halves takes a dependent load a step)
    const int tile = static_cast<int>(a.nc.wide(q)), lane = threadIdx.x & 31;
    int n = 0;
#pragma unroll 4
    for (int e0 = 0; e0 < a.r.E; e0 += 32)
      n += __popc(__ballot_sync(0xffffffffu, e0 + lane < a.r.E && pre[e0 + lane] <= tile));
    return n - 1;
  }
  // (next: the lane stood in the tile before this one, which mostly has the same tokens)
  __device__ __forceinline__ void point(int e, int i, int lane, bool next, LanePtr& l) const {
    const int g = lane >> 2, t = lane & 3, ng = (a.N + 3) >> 2, nt = a.ntn(i), rt = i - nt * ntn();
    const int64_t grp = rt * (kRowTile / 4);
    l.w = a.codes + e * a.ecode + grp * a.gcode;
    l.s = a.scales + e * a.escale + grp * a.gscale;
    l.gcode = a.gcode;
    l.gscale = a.gscale;
    l.groups = ng - static_cast<int>(grp);
    if (next && rt > 0) return;
    const int row = off[e] + nt * kTok + g;
    l.x0 = nullptr;
    l.zero = false;
    if (g < kTok && row < off[e + 1]) {
      int64_t src = row;
      if (a.r.slots) {
        const int slot = __ldcg(a.r.slots + row);
        src = slot < 0 ? -1 : a.topk(slot);
      }
      l.zero = src < 0 || src >= a.r.T;  // a slot of no token: a row of zeros
      if (!l.zero) l.x0 = a.r.X + src * (static_cast<int64_t>(a.nc.d) * kQ4Chunk) + 8 * t;
    }
  }
  __device__ __forceinline__ void store(int e, int i, int m, int r, float v) const {
    const int nt = a.ntn(i), row = (i - nt * ntn()) * kRowTile + r, y = off[e] + nt * kTok + m;
    if (y < off[e + 1] && row < a.N) a.r.Y[static_cast<int64_t>(y) * a.N + row] = f32_to_bf16_bits(v);
  }
};

// -------------------------------------------------------------------- the stream
// A slot: 4 x 512 bytes of codes, 8 bytes of scales a row group and group of K, 256 bytes
// of activations a token. Every lane copies the codes it will read itself; the scales of a
// row group serve four lanes, and lanes of columns behind the last token read any bytes:
// a column of the product depends on its own token only, and theirs are not stored.
template <int kG, int kTok>
struct Slot {  // (kDepth a warp)
  static constexpr uint32_t kScale = 2048;
  static constexpr uint32_t kX = kScale + (kG == 32 ? 256 : 64);
  static constexpr uint32_t kXStep = 64 * kTok;  // a lane's next 16 bytes
  static constexpr uint32_t kBytes = kX + kTok * 256;
  static constexpr int kDepth = 2;
};

// A place in the line of chunks: chunk c of tile i of product p.
struct Place {
  int p, i, c;
};
template <typename Src>
__device__ __forceinline__ Place place_of(const Src& src, int64_t q) {
  Place a;
  a.p = src.find(q);
  const int64_t r = q - src.start(a.p);
  a.i = static_cast<int>(src.nc(a.p).wide(r));
  a.c = static_cast<int>(r - static_cast<int64_t>(a.i) * src.nc(a.p).d);
  return a;
}

template <int kG, int kTok, typename Src>
__device__ __forceinline__ void stream_tiles(const Src& src, float* part, unsigned* count, int grid) {
  using S = Slot<kG, kTok>;
  constexpr int kOut = kRowTile * kTok;  // outputs of a tile
  extern __shared__ __align__(128) unsigned char slots[];
  // Of every warp's run: the end of a tile that began in an earlier run (0), the start of
  // one that goes on in the next (1). Kept in registers while the runs last, then in the
  // slots' place.
  float (*ends)[2][kOut] = reinterpret_cast<float (*)[2][kOut]>(slots);
  static_assert(2 * kOut * sizeof(float) <= S::kDepth * S::kBytes, "ends do not fit");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int b = static_cast<int>(blockIdx.x);
  if (b >= grid) return;
  // The CTA's chunks: an equal share, its ends moved to the nearest start of a tile where
  // tiles are short (then no tile is joined across CTAs, some 2 us at the end: experts with
  // K = 2048, three tokens 20.1 us to 18.6, 64 tokens 54 us to 51; but shares that differ by
  // half a tile of K = 5120 cost as much as they saved).
  const int64_t share = src.share(grid);
  const int extra = src.extra(grid);
  auto bound = [&](int i) {
    const int64_t q = i * share + (i < extra ? i : extra);
    if (i == 0 || i == grid) return q;
    const Place a = place_of(src, q);
    const int nc = static_cast<int>(src.nc(a.p).d);
    if (nc > 24 || 6 * static_cast<int64_t>(nc) > share) return q;
    return 2 * a.c < nc ? q - a.c : q + (nc - a.c);
  };
  int64_t c0, c1;
  if (Src::kWarpFind) {
    c0 = bound(b);
    c1 = bound(b + 1);
  } else {  // two lanes' work, side by side
    const int64_t bounds = bound(b + (lane & 1));
    c0 = __shfl_sync(0xffffffffu, bounds, 0);
    c1 = __shfl_sync(0xffffffffu, bounds, 1);
  }
  auto run_start = [&](int w) { return c0 + (c1 - c0) * w / kWarps; };

  // --- fetching: chunks 0 .. n - 1 of this warp's run
  const int64_t q0 = run_start(warp);
  const int n = static_cast<int>(run_start(warp + 1) - q0);
  const uint32_t slot0 = smem_u32(slots) + warp * (S::kDepth * S::kBytes);
  Place u = {0, 0, 0};
  if (n > 0) u = place_of(src, q0);
  Place f = u;
  LanePtr l = {};
  int left = 0, qf = 0;  // chunks left of the tile being fetched; of the run, those fetched
  // A copy instruction brings 256 bytes of two row groups (lanes 0-15 and 16-31); row groups
  // behind the last are left out, and the rows computed from what is there are not stored.
  const int hi = lane >> 4, lo = lane & 15;
  const uint32_t wdst = 512u * (lo >> 2) + 16u * (lo & 3) + 64u * hi;
  auto point = [&](bool next) {   // the pointers to chunk f.c
    src.point(f.p, f.i, lane, next, l);
    l.x = l.x0;
    l.w += static_cast<int64_t>(f.c) * 256 + hi * l.gcode + 16 * lo;
    if (kG == 32) l.s += static_cast<int64_t>(f.c) * 16 + (lo >> 1) * static_cast<int64_t>(l.gscale) + 8 * (lo & 1);
    else l.s += static_cast<int64_t>(f.c) * 4 + (lane & 7) * static_cast<int64_t>(l.gscale);
    if (l.x) l.x += static_cast<int64_t>(f.c) * kQ4Chunk;
    left = static_cast<int>(src.nc(f.p).d) - f.c;
  };
  if (n > 0) point(false);
  auto fetch_w = [&](uint32_t d) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (2 * i + hi < l.groups) cp16(d + wdst + 128u * i, l.w + 2 * i * l.gcode);
    if (kG == 32) {
      if (lane < 16 && (lane >> 1) < l.groups) cp16(d + S::kScale + 16u * lane, l.s);
    } else if (lane < 8 && lane < l.groups) {
      cp8(d + S::kScale + 8u * lane, l.s);
    }
  };
  auto fetch_x = [&](uint32_t d, const uint16_t* x, bool zero) {
    d += S::kX + 16u * lane;
    if (kTok == 1) {  // 128 activations: 16 lanes
      if (lane < 16) cp16(d, x);
    } else if (x) {
#pragma unroll
      for (int s = 0; s < 4; ++s) cp16(d + S::kXStep * s, x + 32 * s);
    } else if (Src::kZeros && zero) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(d + S::kXStep * s), "r"(0u) : "memory");
    }
  };
  auto advance = [&]() {  // to the next chunk of the run
    l.w += 256;
    l.s += kG == 32 ? 16 : 4;
    if (kTok == 1 || l.x) l.x += kQ4Chunk;
    if (++qf < n && --left == 0) {
      f.c = 0;
      if (++f.i == src.tiles(f.p)) {
        f.i = 0;
        f.p = src.next(f.p);
      }
      point(true);
    }
  };
  // The first chunks: their codes and scales before the previous kernel has finished
  // (where that kernel decides nothing about them), the activations after it.
  const uint16_t* x0[S::kDepth] = {};
  bool z0[S::kDepth] = {};
#pragma unroll
  for (int i = 0; i < S::kDepth; ++i)
    if (i < n) {
      fetch_w(slot0 + i * S::kBytes);
      x0[i] = l.x;
      z0[i] = l.zero;
      advance();
    }
  if (Src::kEarly) pdl_wait();
#pragma unroll
  for (int i = 0; i < S::kDepth; ++i) {
    if (i < n) fetch_x(slot0 + i * S::kBytes, x0[i], z0[i]);
    cp_commit();
  }
  uint32_t cslot = slot0;
  auto fetch = [&]() {  // the next chunk into the slot just read
    if (qf < n) {
      fetch_w(cslot);
      fetch_x(cslot, l.x, l.zero);
      advance();
    }
    cp_commit();
  };

  // --- the run's tiles, whole or in part
  const uint32_t xoff = S::kX + 16u * (lane & (4 * kTok - 1));
  Place head = {-1, 0, 0}, tail = {-1, 0, 0};  // the tiles of this run's ends
  int64_t tail_q = 0;                          // where the second begins
  const int head_c = u.c;
  float acc[2][4], first[2][4];  // first: the sums of place 0
  for (int q = 0; q < n;) {
    const int nc = static_cast<int>(src.nc(u.p).d);
    const int qe = nc - u.c < n - q ? q + (nc - u.c) : n;
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i >> 2][i & 3] = 0.0f;
    const int part_c = u.c, part_q = q;
    for (; q < qe; ++q) {
      cp_wait<S::kDepth - 1>();
      __syncwarp();  // (the other lanes' scales)
      float sum[2][4];
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        const uint4 w = lds128(cslot + 512u * s + 16u * lane);
        const uint4 x = lds128(cslot + xoff + S::kXStep * s);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a0[4] = {q4_pair(w.x, 2 * j), q4_pair(w.y, 2 * j), q4_pair(w.x, 2 * j + 1), q4_pair(w.y, 2 * j + 1)};
          const uint32_t a1[4] = {q4_pair(w.z, 2 * j), q4_pair(w.w, 2 * j), q4_pair(w.z, 2 * j + 1), q4_pair(w.w, 2 * j + 1)};
          const uint32_t b0 = j ? x.z : x.x, b1 = j ? x.w : x.y;
          if (j == 0 && (kG == 32 || s == 0)) {
            mma_bf16_first(sum[0], a0, b0, b1);
            mma_bf16_first(sum[1], a1, b0, b1);
          } else {
            mma_bf16(sum[0], a0, b0, b1);
            mma_bf16(sum[1], a1, b0, b1);
          }
        }
        if (kG == 32 || s == 3) {
          const uint2 sc = lds64(cslot + S::kScale + (kG == 32 ? 32u * g + 8u * s : 8u * g));
          const float2 s01 = __half22float2(*reinterpret_cast<const __half2*>(&sc.x));
          const float2 s23 = __half22float2(*reinterpret_cast<const __half2*>(&sc.y));
#pragma unroll
          for (int c = 0; c < (kTok == 1 ? 1 : 2); ++c) {  // tokens 2t, 2t + 1
            acc[0][c] += s01.x * sum[0][c];
            acc[0][2 + c] += s01.y * sum[0][2 + c];
            acc[1][c] += s23.x * sum[1][c];
            acc[1][2 + c] += s23.y * sum[1][2 + c];
          }
        }
      }
      __syncwarp();  // every lane has read the slot
      fetch();
      cslot = cslot == slot0 + (S::kDepth - 1) * S::kBytes ? slot0 : cslot + S::kBytes;
    }
    const bool whole = part_c == 0 && qe - part_q == nc;
    if (part_c > 0) {
      head = u;
#pragma unroll
      for (int i = 0; i < 8; ++i) first[i >> 2][i & 3] = acc[i >> 2][i & 3];
    } else if (!whole) {
      tail = u;
      tail_q = q0 + part_q;
    }
    if (whole) {
#pragma unroll
      for (int c = 0; c < (kTok == 1 ? 1 : 2); ++c)
        if (2 * t + c < kTok)
#pragma unroll
          for (int r = 0; r < 4; ++r)  // row 4g + r of token 2t + c
            src.store(u.p, u.i, 2 * t + c, 4 * g + r, acc[r >> 1][2 * (r & 1) + c]);
    }
    u.c = 0;
    if (q < n && ++u.i == src.tiles(u.p)) {
      u.i = 0;
      u.p = src.next(u.p);
    }
  }
  cp_wait<0>();
  __shared__ int64_t starts[kWarps + 1];  // of the runs
  if (lane == 0) starts[warp] = q0;
  if (threadIdx.x == 0) starts[kWarps] = c1;
  __syncthreads();  // every warp has left its slots
#pragma unroll
  for (int c = 0; c < (kTok == 1 ? 1 : 2); ++c)
    if (2 * t + c < kTok)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int o = (2 * t + c) * kRowTile + 4 * g + r;
        if (head.p >= 0) ends[warp][0][o] = first[r >> 1][2 * (r & 1) + c];
        if (tail.p >= 0) ends[warp][1][o] = acc[r >> 1][2 * (r & 1) + c];
      }
  __syncthreads();

  // --- tiles that several warps share: joined by the warp in whose run the tile (or the
  // CTA's part of it) begins
  auto join = [&](const Place& at, int64_t qt, int which) {
    const int64_t qn = qt + src.nc(at.p).d;
    float v[kTok], next[kTok];  // row `lane` of every token
#pragma unroll
    for (int m = 0; m < kTok; ++m) v[m] = ends[warp][which][m * kRowTile + lane];
    // the later warps whose runs, if not empty, begin inside the tile; a part's loads are
    // in flight while the one before is added
    const int64_t s0 = starts[lane < kWarps ? lane : kWarps], s1 = starts[lane < kWarps ? lane + 1 : kWarps];
    unsigned more = __ballot_sync(0xffffffffu, lane > warp && s0 < qn && s0 < s1);
    auto fetch_part = [&]() {
#pragma unroll
      for (int m = 0; m < kTok; ++m) next[m] = ends[__ffs(more) - 1][0][m * kRowTile + lane];
    };
    if (more) fetch_part();
    while (more) {
      float part[kTok];
#pragma unroll
      for (int m = 0; m < kTok; ++m) part[m] = next[m];
      more &= more - 1;
      if (more) fetch_part();
#pragma unroll
      for (int m = 0; m < kTok; ++m) v[m] += part[m];
    }
    if (which == 1 && qn <= c1) {
#pragma unroll
      for (int m = 0; m < kTok; ++m) src.store(at.p, at.i, m, lane, v[m]);
      return;
    }
    // shared with other CTAs
#pragma unroll
    for (int m = 0; m < kTok; ++m) __stcg(part + static_cast<int64_t>(2 * b + which) * kOut + m * kRowTile + lane, v[m]);
    __syncwarp();
    auto cta_of = [&](int64_t q) {
      const int64_t r = q - extra * (share + 1);
      return static_cast<int>(r < 0 ? quot(q, share + 1) : extra + quot(r, share));
    };
    const int first = which == 1 ? b : cta_of(qt), parts = cta_of(qn - 1) - first + 1;
    unsigned before = 0;
    // (one atomic that releases this warp's stores and acquires the others')
    if (lane == 0)
      asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(count + first) : "memory");
    before = __shfl_sync(0xffffffffu, before, 0);
    if (before != static_cast<unsigned>(parts - 1)) return;
    __syncwarp();  // lane 0's acquire comes before every lane's reads (a shuffle orders no memory)
#pragma unroll
    for (int m = 0; m < kTok; ++m) {
      float y = __ldcg(part + static_cast<int64_t>(2 * first + 1) * kOut + m * kRowTile + lane);
      for (int k = 1; k < parts; ++k) y += __ldcg(part + static_cast<int64_t>(2 * (first + k)) * kOut + m * kRowTile + lane);
      src.store(at.p, at.i, m, lane, y);
    }
    if (lane == 0) count[first] = 0;  // as it was found
  };
  if (head.p >= 0 && q0 == starts[0]) join(head, q0 - head_c, 0);
  if (tail.p >= 0) join(tail, tail_q, 1);
}

// Enough CTAs to fill the GPU, but at least a chunk for every warp of each.
__device__ __forceinline__ int runs_for(int64_t chunks, int most) {
  const int64_t n = (chunks + kWarps - 1) / kWarps;
  return static_cast<int>(n < most ? n : most);
}

template <int kG, int kTok, int kCap, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    q4_list_kernel(const __grid_constant__ Q4List<kCap> a) {
  pdl_launch_dependents();
  const ListSource<kCap, kTok, kF32> src = {a};
  stream_tiles<kG, kTok>(src, a.part, a.count, static_cast<int>(gridDim.x));
}

template <int kG, int kTok>
__global__ void __launch_bounds__(kThreads, 1)
    q4_expert_kernel(const __grid_constant__ Q4Experts a) {
  extern __shared__ __align__(128) unsigned char slots[];
  int* const off = reinterpret_cast<int*>(slots + kWarps * Slot<kG, kTok>::kDepth * Slot<kG, kTok>::kBytes);  // [E + 1]
  int* const pre = off + a.r.E + 1;                                                                           // [E + 1]
  pdl_launch_dependents();
  pdl_wait();
  // Tiles before each expert: a running sum over the warp, then over the warps. Offsets that
  // descend somewhere would name rows twice, and more tiles than are counted in 32 bits: no
  // row then.
  __shared__ int wsum[kWarps];
  const int R = static_cast<int>(a.r.R), E = a.r.E, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto clamped = [&](int e) {
    const int v = __ldcg(a.r.offsets + e);
    return v < 0 ? 0 : (v > R ? R : v);
  };
  int run = 0;
  bool down = false;
  for (int e0 = 0; e0 < E; e0 += kThreads) {
    const int e = e0 + threadIdx.x;
    int c = 0;
    if (e < E) {
      const int r0 = clamped(e), r1 = clamped(e + 1);
      off[e] = r0;
      if (e == E - 1) off[E] = r1;
      down = down || r1 < r0;
      c = r1 > r0 ? (r1 - r0 + kTok - 1) / kTok * static_cast<int>(a.ntn.d) : 0;
    }
    int inc = c;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) wsum[warp] = inc;
    down = __syncthreads_or(down);
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += wsum[w];
      all += wsum[w];
    }
    if (e < E) pre[e] = run + before + inc - c;
    run += all;
    if (e0 + kThreads < E) __syncthreads();  // (wsum is written again)
  }
  if (threadIdx.x == 0) pre[E] = down ? 0 : run;
  __syncthreads();
  if (pre[E] == 0) return;
  const ExpertSource<kTok> src = {a, off, pre};
  stream_tiles<kG, kTok>(src, a.part, a.count, runs_for(src.chunks(), static_cast<int>(gridDim.x)));
}

// Programmatic dependent launch on stream s: the kernel starts early and waits itself.
template <typename A>
cudaError_t launch_pdl(void (*k)(A), size_t smem, unsigned grid, cudaStream_t s, const A& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, args);
}

// The kernel's shared-memory limit, set once per device.
template <auto kKernel>
cudaError_t allow_smem(size_t bytes) {
  static PerDevice<bool> configured;
  bool done = false;
  return configured.get(
      [&](int, bool* v) {
        *v = true;
        return cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
      },
      &done);
}

int most_runs() { return sm_count(); }

// Tokens a tile of the experts' products, by the average rows of an expert. Four move fewer
// activations, eight decode an expert's weights once for more rows. Measured, four / eight:
// 16 experts of 5120 x 5120, 4 rows in all 22.7 / 25.0 us, 16 rows 39.0 / 41.5, 32 rows 48.7 /
// 47.8; 128 of 2048 x 1536, 8 rows 15.2 / 16.8, 64 rows 24.1 / 24.2, 128 rows 31.8 / 31.0, 256
// rows 43.8 / 38.5.
int few_tok(int32_t E, int64_t R) { return R <= E ? 4 : 8; }

// Workspace: the counters' 64 KB (one for every run), then two parts of a tile a run.
float* part_of(void* ws) { return reinterpret_cast<float*>(static_cast<char*>(ws) + kWsCounterBytes); }

template <int kG, int kTok, int kCap, bool kF32>
cudaError_t launch_list(Q4List<kCap>& a, void* ws, cudaStream_t s) {
  constexpr size_t smem = kWarps * Slot<kG, kTok>::kDepth * Slot<kG, kTok>::kBytes;
  a.part = part_of(ws);
  a.count = static_cast<unsigned*>(ws);
  const int64_t runs = (a.chunks + kWarps - 1) / kWarps;
  const unsigned grid = static_cast<unsigned>(runs < most_runs() ? runs : most_runs());
  a.share = a.chunks / grid;
  a.extra = static_cast<int32_t>(a.chunks % grid);
  a.ntok = Div((a.M + kTok - 1) / kTok);
  const cudaError_t e = allow_smem<q4_list_kernel<kG, kTok, kCap, kF32>>(smem);
  return e != cudaSuccess ? e : launch_pdl(q4_list_kernel<kG, kTok, kCap, kF32>, smem, grid, s, a);
}

template <int kG, int kTok>
cudaError_t launch_experts(const Q4Experts& a, cudaStream_t s) {
  constexpr size_t slots = kWarps * Slot<kG, kTok>::kDepth * Slot<kG, kTok>::kBytes;
  const cudaError_t e = allow_smem<q4_expert_kernel<kG, kTok>>(slots + 8 * (LBQ_MAX_EXPERTS + 1));
  return e != cudaSuccess ? e : launch_pdl(q4_expert_kernel<kG, kTok>, slots + 8 * static_cast<size_t>(a.r.E + 1),
                                           static_cast<unsigned>(most_runs()), s, a);
}

// Product p of a list, each row tile with `ntok` token tiles: q0 chunks lie before it.
Q4Prod make_prod(const lbq_weights& w, const uint16_t* x, void* y, int64_t* q0, int64_t ntok = 1) {
  Q4Prod p;
  p.codes = static_cast<const uint8_t*>(w.codes);
  p.scales = static_cast<const uint16_t*>(w.scales);
  p.x = x;
  p.y = y;
  p.q0 = *q0;
  p.gcode = 4 * w.code_stride;
  p.gscale = static_cast<int32_t>(4 * w.scale_stride);
  p.N = static_cast<int32_t>(w.N);
  p.nc = Div(w.K / kQ4Chunk);
  *q0 += (w.N + kRowTile - 1) / kRowTile * ntok * p.nc.d;
  return p;
}

}  // namespace

size_t lbq_q4_few_workspace(int64_t M) {
  const int tok = M == 1 ? 1 : (M <= 4 ? 4 : 8);
  return kWsCounterBytes + static_cast<size_t>(most_runs()) * 2 * kRowTile * tok * sizeof(float);
}

cudaError_t lbq_launch_q4_list(const lbq_product* ps, int32_t n, float* y32, void* ws, cudaStream_t s) {
  const bool g32 = ps[0].w.fmt == LBQ_Q4G32;
  if (n == 1) {
    Q4List<1> a;
    a.n = 1;
    a.M = 1;
    a.chunks = 0;
    a.p[0] = make_prod(ps[0].w, ps[0].x, y32 ? static_cast<void*>(y32) : ps[0].y, &a.chunks);
    if (y32) return g32 ? launch_list<32, 1, 1, true>(a, ws, s) : launch_list<128, 1, 1, true>(a, ws, s);
    return g32 ? launch_list<32, 1, 1, false>(a, ws, s) : launch_list<128, 1, 1, false>(a, ws, s);
  }
  static thread_local Q4List<LBQ_BATCH_MAX> a;  // 18 KB: off the stack
  a.n = n;
  a.M = 1;
  a.chunks = 0;
  for (int32_t i = 0; i < n; ++i) a.p[i] = make_prod(ps[i].w, ps[i].x, ps[i].y, &a.chunks);
  return g32 ? launch_list<32, 1, LBQ_BATCH_MAX, false>(a, ws, s) : launch_list<128, 1, LBQ_BATCH_MAX, false>(a, ws, s);
}

cudaError_t lbq_launch_q4_few(const lbq_weights* w, const uint16_t* X, int64_t M, uint16_t* Y, void* ws,
                              cudaStream_t s) {
  const bool g32 = w->fmt == LBQ_Q4G32;
  const int tok = M <= 4 ? 4 : 8;
  Q4List<1> a;
  a.n = 1;
  a.M = static_cast<int32_t>(M);
  a.chunks = 0;
  a.p[0] = make_prod(*w, X, Y, &a.chunks, (M + tok - 1) / tok);
  if (tok == 4) return g32 ? launch_list<32, 4, 1, false>(a, ws, s) : launch_list<128, 4, 1, false>(a, ws, s);
  return g32 ? launch_list<32, 8, 1, false>(a, ws, s) : launch_list<128, 8, 1, false>(a, ws, s);
}

cudaError_t lbq_launch_q4_expert_few(const lbq_weights* w, const lbq_expert_rows& r, void* ws, cudaStream_t s) {
  Q4Experts a;
  a.codes = static_cast<const uint8_t*>(w->codes);
  a.scales = static_cast<const uint16_t*>(w->scales);
  a.gcode = 4 * w->code_stride;
  a.gscale = static_cast<int32_t>(4 * w->scale_stride);
  const int64_t ng = (w->N + 3) / 4;
  a.ecode = ng * a.gcode;
  a.escale = ng * a.gscale;
  a.N = static_cast<int32_t>(w->N);
  a.nc = Div(w->K / kQ4Chunk);
  a.ntn = Div((w->N + kRowTile - 1) / kRowTile);
  a.topk = Div(r.topk);
  a.r = r;
  a.part = part_of(ws);
  a.count = static_cast<unsigned*>(ws);
  const bool g32 = w->fmt == LBQ_Q4G32;
  if (few_tok(r.E, r.R) == 4) return g32 ? launch_experts<32, 4>(a, s) : launch_experts<128, 4>(a, s);
  return g32 ? launch_experts<32, 8>(a, s) : launch_experts<128, 8>(a, s);
}
