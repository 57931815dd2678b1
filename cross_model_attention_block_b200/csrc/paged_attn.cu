// Attention of one new token per sequence over a paged key-value cache.
//
// MapFlow article (163.com, "让复用真正省时，还需要解决存储和执行问题"): the
// receiver works with PagedAttention; after a mapped prefill its own tokens
// attend to the keys and values it keeps in pages.
//
//   x_j = scale q.k_j + band_bias [L-1-j < band_width]   (j < L, inside the window)
//   O = sum_j 2^(x_j log2e - m) v_j / l,  m = max, l = sum of the same powers,
//   lse = (m + log2 l) ln 2.
//
// Bound by memory: each key and value is read once for the G = Hq / Hkv query
// heads that share it, 4 G operations per element, G / 2 to 2 G a byte.  What
// counts is that every SM keeps enough bytes in flight and that all SMs stop
// at the same time, whatever the lengths:
//
//  * A unit is 16 keys and values of one KV head (16 tokens never straddle a
//    page).  The units of all rows (sequence, KV head, group of query heads),
//    laid end to end, are cut into runs, one per block and in equal parts one
//    per warp; every block finds the cuts itself from `lens`, so the host needs
//    no lengths and a captured call follows them.
//  * A warp runs alone: it copies its units by TMA into its own ring of
//    shared memory (one box of 16 tokens x 1 head for K, one for V, 128-byte
//    swizzled) and waits on its own barriers; no block-wide step in the loop.
//  * A row inside one run is finished there.  Rows that a block's warps share
//    are joined in shared memory when all are through; the pieces (maximum,
//    sum, unnormalised O) of those that blocks share, two a block at most, go
//    to the workspace, and a second, dependent launch joins them.
//
// The cuts and the order of the sums follow from the lengths of all sequences,
// the sizes of the pool and the table, and the heads, never from timing: a call
// repeats its bits.  A sequence's differ (within the rounding of float32 sums)
// beside other sequences or behind a table of another width.
//
// Measured (bf16, d 128, 32 heads over 8, pages of 16): 64 sequences of 1 K to
// 16 K tokens, 1.39 GB, 217 us (6.4 TB/s).  32 K tokens 31.2 us: 1.8 to find the
// cuts, 2.9 more until the first keys are there, 21 until the last are read (6.4
// TB/s), 1.3 to join in the blocks, 2.3 for the second launch, 2 around them.  1 K
// tokens 9.4 us, all latency: 1.4, 1.8, 1.3, 0.9, 1.5 and 2.4 of the same.
#include <algorithm>
#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdio>

#include "mf_sm100.cuh"

namespace mf {
using namespace sm100;
namespace {

constexpr int kUnit = 16;      // keys of one unit
// What a row costs a warp besides its units, in units (a batch of many rows of a
// unit or two: 22.5 us with 2 to 5, 26.3 with 0).
constexpr int kRowCost = 2;
constexpr int kCtas = 148;     // one block per SM of a B200
constexpr int kWarps = 8;      // of the main kernel's blocks
// A line of kLarge places a block leaves 1 / kRest of itself to kExtra more
// blocks.  Measured, 64 sequences of 1 K to 16 K tokens: 215 us with 8, 219 with
// 6 or with half as many blocks, 224 without; batches of 540 and 600 places a
// block lose (97 -> 103 us) and break even (111 -> 112), of 1000 and 1280 gain
// (172 -> 167, 211 -> 205).  A table with room for such a line brings the blocks
// whatever the lengths: where these are short they leave at once, for 1 us (64
// sequences of 200 tokens 16.8 -> 17.7).
constexpr int kExtra = 2 * kCtas;
constexpr int kRest = 8;
constexpr int kLarge = 800;
constexpr int kThreads = kWarps * 32;
// A row's reference m is not its running maximum: it moves when a logit lies
// more than 2^kSlack above it, about once a row, and only then are the sums
// rescaled.  Weights stay below 2^kSlack.
constexpr float kSlack = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Shared {  // a row that blocks v0 .. v1 share (v1 < v0: none)
  int s, r;      // its sequence, and which of the sequence's rows (marked)
  int v0, v1;
};

struct Params {
  const void* Q;
  void* O;
  float* lse;
  const int32_t* page_table;
  const int32_t* lens;
  int64_t q_stride, o_stride, npages;
  int nseq, Hq, page_size, max_pages, len_add, band, window;
  int Hkv, G, groups, gh;  // as in Rows
  bool pair;
  bool by_rows;    // blocks take whole rows
  int extra;       // blocks past the first kCtas
  float scale2, bias2;  // times log2 e
  float bias;           // as it is: of rows that lie inside the band
  // workspace: pieces of the rows that blocks share (two per block: of the row
  // its run begins in and of the row it ends in); entry b of `shared`: the row
  // whose first block boundary is the one before block b
  float* part_o;   // [2 blocks][gh][D]
  float2* part_ml; // [2 blocks][gh]
  Shared* shared;  // [blocks]
  unsigned* status;
};

// ------------------------------------------------------------------ the plan

// In Span's band_lo (keys lie below 2^31 - 16): no key is in the band; every key
// is, and its bias, which moves no weight, is left to the log-sum-exp.  A bias of
// any size takes no digits from the logits of such rows.
constexpr int kNoBand = INT32_MAX - 1;
constexpr int kAllBand = INT32_MAX;

struct Span {  // the keys [lo, len) of a sequence, and its units
  int lo, len, band_lo;  // keys from band_lo on get the bias
  int first, n;          // first unit, units
};

__device__ __forceinline__ int clamp_int(int64_t x) {
  return int(max(int64_t(0), min(x, int64_t(INT32_MAX))));
}

__device__ __forceinline__ Span span_of(const Params& p, int s) {
  const int64_t L = int64_t(p.lens[s]) + p.len_add;
  Span k;
  k.len = int(max(int64_t(0), min(L, int64_t(p.max_pages) * p.page_size)));
  k.lo = p.window > 0 ? min(clamp_int(L - p.window), k.len) : 0;
  k.band_lo = p.band > 0 ? min(clamp_int(L - p.band), kNoBand) : kNoBand;
  if (k.band_lo <= k.lo) k.band_lo = kAllBand;
  k.first = k.lo / kUnit;
  k.n = k.len > k.lo ? (k.len + kUnit - 1) / kUnit - k.first : 0;
  return k;
}

// The line is made of the rows' units, each row's behind kRowCost places that
// stand for what a row costs besides its units (queries, sums, output).  It is
// cut into a run for every block, and that into equal runs for its warps.  The
// first kCtas blocks, which fill the GPU, share `head` places evenly, and
// `extra` blocks what is left.
//
// SMs do not read at one speed: those that share their path to L2 with more
// others are slower (with equal runs the first is done after 170 us, most after
// 190, the last after 215).  So a large line leaves a part to short runs, of
// blocks that the hardware starts where others have ended.
struct Cuts {
  int64_t total, head;
  int extra;
  __device__ __forceinline__ static int64_t part(int64_t n, int i, uint32_t of) {
    const uint64_t x = uint64_t(n) * uint32_t(i);
    return int64_t(x >> 32 ? x / of : uint32_t(x) / of);
  }
  __device__ __forceinline__ static int which(int64_t n, int64_t u, uint32_t of) {
    const uint64_t x = uint64_t(u + 1) * of - 1;
    return x >> 32 ? int(x / uint64_t(n)) : int(uint32_t(x) / uint32_t(n));
  }
  // first place of block b
  __device__ __forceinline__ int64_t at(int b) const {
    return b <= kCtas ? part(head, b, kCtas) : head + part(total - head, b - kCtas, extra);
  }
  // the block that holds place u
  __device__ __forceinline__ int holder(int64_t u) const {
    return u < head ? which(head, u, kCtas) : kCtas + which(total - head, u - head, extra);
  }
};

__device__ __forceinline__ Cuts cuts_of(const Params& p, int64_t total) {
  const bool large = p.extra > 0 && total >= int64_t(kCtas) * kLarge;
  return Cuts{total, large ? total - total / kRest : total, p.extra};
}

// Which of a sequence's rows, below 2^16, with a mark where it lies inside the
// band: whoever ends a shared row need not look up its span.
__device__ __forceinline__ int marked(int r, const Span& k) {
  return k.band_lo == kAllBand ? r | 1 << 16 : r;
}
__device__ __forceinline__ int row_of(int mark) { return mark & 0xffff; }
__device__ __forceinline__ float bias_of(const Params& p, int mark) {
  return mark >> 16 ? p.bias : 0.f;
}

// A place in the line: a unit, and how much of the run is left from there.
struct Walk {
  int s, r, g;  // sequence, its row, unit of the row
  int left;     // <= 0: the run is over
  Span k;
  // the next unit; rows of a sequence have equally many
  __device__ __forceinline__ void step(const Params& p) {
    --left;
    if (++g < k.n) return;
    g = 0;
    left -= kRowCost;
    if (left <= 0 || ++r < p.Hkv * p.groups) return;
    r = 0;
    do {
      if (++s >= p.nseq) return;
      k = span_of(p, s);
    } while (k.n == 0);
  }
};

struct PlanSmem {
  int64_t before[kThreads + 1];  // places of the sequences before thread t's
  int64_t warp_sum[kThreads / 32];
};

// Places of every thread's share of the sequences, added up over the block.
__device__ __forceinline__ void plan_places(const Params& p, PlanSmem& sm, bool report) {
  const int per = (p.nseq + kThreads - 1) / kThreads;
  const int s0 = min(int(threadIdx.x) * per, p.nseq), s1 = min(s0 + per, p.nseq);
  int64_t mine = 0;
  for (int s = s0; s < s1; ++s) {
    const int n = span_of(p, s).n;
    mine += n > 0 ? n + kRowCost : 0;
    if (report && int64_t(p.lens[s]) + p.len_add > int64_t(p.max_pages) * p.page_size)
      atomicOr(p.status, kStatusBadPage);
  }
  mine *= p.Hkv * p.groups;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int64_t sum = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  if (lane == 31) sm.warp_sum[warp] = sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t x = sm.warp_sum[w];
    if (w < warp) sum += x;
  }
  sm.before[threadIdx.x] = sum - mine;
  if (threadIdx.x == kThreads - 1) sm.before[kThreads] = sum;
  __syncthreads();
}

// The place where the row before which `row` others come begins; rows of
// sequences without keys count, but have no places.
__device__ __forceinline__ int64_t place_of_row(const Params& p, const PlanSmem& sm, int row) {
  const int rows = p.Hkv * p.groups, s = row / rows;
  if (s >= p.nseq) return sm.before[kThreads];
  const int per = (p.nseq + kThreads - 1) / kThreads, t = s / per;
  int64_t at = sm.before[t];
  for (int i = t * per; i < s; ++i) {
    const int n = span_of(p, i).n;
    at += n > 0 ? (n + kRowCost) * rows : 0;
  }
  const int n = span_of(p, s).n;
  return at + (n > 0 ? (row - s * rows) * (n + kRowCost) : 0);
}

// The first unit of the run of `n` places from place u on (the same in the
// whole warp).
__device__ __forceinline__ Walk find_place(const Params& p, const PlanSmem& sm, int64_t u,
                                           int n) {
  constexpr int kSub = kThreads / 32;
  const int lane = threadIdx.x % 32;
  const int t0 = (__popc(__ballot_sync(0xffffffffu, sm.before[lane * kSub] <= u)) - 1) * kSub;
  const bool below = lane < kSub && sm.before[t0 + lane % kSub] <= u;
  const int t = t0 - 1 + __popc(__ballot_sync(0xffffffffu, below));
  int64_t at = u - sm.before[t];
  Walk w;
  w.s = t * ((p.nseq + kThreads - 1) / kThreads);
  const int rows = p.Hkv * p.groups;
  while (true) {
    w.k = span_of(p, w.s);
    const int64_t places = w.k.n > 0 ? int64_t(w.k.n + kRowCost) * rows : 0;
    if (at < places || w.s + 1 >= p.nseq) break;
    at -= places;
    ++w.s;
  }
  const uint32_t row = w.k.n + kRowCost;
  w.r = at >> 32 ? int(at / row) : int(uint32_t(at) / row);
  const int into = int(at - int64_t(w.r) * row);  // below kRowCost: before the row's units
  w.g = max(0, into - kRowCost);
  w.left = n - max(0, kRowCost - into);
  return w;
}

// ------------------------------------------------------- joining two pieces

// In place of a piece's sum of weights: its unnormalised O was never written.  A
// sum of zero is not that: keys whose logits are all -inf weigh nothing, but zero
// times a NaN or an infinity among their values is a NaN, wherever a row is cut.
constexpr float kNoSums = -1.f;

// The factors of two pieces with maxima a and b, relative to their maximum m.
struct Join {
  float m, ca, cb;
  __device__ __forceinline__ Join(float a, float b) {
    m = fmaxf(a, b);
    const float ref = m == -INFINITY ? 0.f : m;  // nothing seen: keep 2^(-inf)
    ca = ex2(a - ref);
    cb = ex2(b - ref);
  }
};

// ------------------------------------------------------------ bf16: mma.sync
//
// The query heads of a group are the rows of a 16-row matrix product: S = Q K^T
// per unit, then O += P V.  The weights are kept to 2^-17 as two bf16 terms
// (the first rounded, the second its remainder), so that they lose no more
// than the float32 arithmetic around them.  Up to 8 heads leave half the rows
// of a product free: rows 8..15 then take the remainders and the two terms
// cost one product.
//
// A remainder is zero or negative as often as not, and must not meet an infinity
// among the values, which the first terms' products already carry: sums of packed
// remainders are dropped where those of the first terms are infinite, and the
// unpacked remainders' products are taken with the values held to the largest
// finite bf16 (one instruction a register, 32 a unit at 128 dims).
//
// Why warp-level products: a unit's 32 take 256 cycles of an SM quarter's tensor
// pipe, and HBM brings its two warps a unit each in 1.48 us, 2720 cycles at the
// 1837 MHz of such a call, so a fifth of that pipe is enough (up to 48 products
// and three tenths with 16 heads); operands and sums stay in one warp's registers
// and no warp waits for another.  The same work as
// tcgen05 products of 128 keys x heads, with P through shared memory and sums
// in TMEM, took 237 us where this took 226 then, and 48 where 17 (short
// rows): each tile is a chain of five hand-offs, and a row's end another two.
//
// A unit takes a warp 2420 cycles of the 64 sequences' call (clock64, 1837 MHz), 4
// heads a group: 350 S, 320 weights, 250 O, 640 to issue the next copies, 110
// between these, and 760 waiting; with keys in L2 1610, 90 of them waiting.
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Infinities to the largest finite bf16, with their sign.  Their products with
// remainders stay finite unless three keys of a unit have infinities in a dim and
// weights above 2^7 (a remainder is at most 2^-8 of its weight's power of two).
__device__ __forceinline__ uint32_t finite_bf16(uint32_t v) {
  asm("min.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(v) : "r"(0x7f7f7f7fu));
  return v;
}

// HEADS: 4 (at 128 dims), 8 or 16 query heads of a row at most.  PAIR: a row has two KV heads,
// whose 64 dims lie side by side, and the query heads of both; the products are
// taken with both, and a query head keeps the one that is its own.
template <int D_, int HEADS, bool PAIR = false>
struct Bf16Body {
  using T = __nv_bfloat16;
  static constexpr int D = D_, kHeads = HEADS;
  static constexpr int KD = PAIR ? 2 * D : D;  // dims of a key as it is copied
  static constexpr int kTile = kUnit * KD * 2;
  // what the pieces of shared rows leave of 227 KB
  static constexpr int kStages = KD == 64 ? (HEADS == 16 ? 5 : 6) : HEADS * D <= 512 ? 3 : 2;
  static constexpr int kScratch = 0;  // bytes of shared memory per warp besides the ring
  static constexpr bool kPacked = HEADS <= 8;
  static constexpr int NR = kPacked ? 1 : 2;  // rows of the product a thread holds
  static constexpr int KS = D / 16;

  int lane;
  uint32_t q[KS][2 * NR];
  float o[KD / 8][4];
  float m[NR], l[NR];
  bool second[NR];  // PAIR: the row's KV head is the second

  __device__ __forceinline__ Bf16Body(int lane_, void*) : lane(lane_) {}

  __device__ __forceinline__ int row(int n) const { return n * 8 + lane / 4; }

  __device__ __forceinline__ void begin(const T* Q, int heads) {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      const bool live = row(n) < heads;
      second[n] = PAIR && row(n) >= heads / 2;
      const T* x = Q + (live ? row(n) : 0) * D + 2 * (lane % 4);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        q[k][n] = live ? *reinterpret_cast<const uint32_t*>(x + k * 16) : 0u;
        q[k][NR + n] = live ? *reinterpret_cast<const uint32_t*>(x + k * 16 + 8) : 0u;
      }
      m[n] = -INFINITY;
      l[n] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < KD / 8; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  }

  // One unit: keys j0 .. j0+15 at `K`, values at `V`; keys outside [lo, len)
  // take no part, those from band_lo on get the bias.
  __device__ __forceinline__ void step(const Params& p, char* K, char* V, int j0, const Span& k) {
    float s[2][4] = {}, s2[2][4] = {};
    {
      const int r = (lane / 16) * 8 + lane % 8;
      const uint32_t base = smem_u32(K) + r * 128;
#pragma unroll
      for (int i = 0; i < KD / 16; ++i) {
        const int c = 2 * i + (lane / 8) % 2;
        uint32_t b[4];
        ldsm4(b, base + (c / 8) * 2048 + (((c % 8) ^ (r % 8)) << 4));
        const uint32_t* a = q[i % KS];
        const uint32_t a1 = kPacked ? 0u : a[1], a3 = kPacked ? 0u : a[NR + 1];
        float(&to)[2][4] = i < KS ? s : s2;
        mma16816(to[0], a[0], a1, a[NR], a3, b[0], b[1]);
        mma16816(to[1], a[0], a1, a[NR], a3, b[2], b[3]);
      }
    }
    const bool inside = j0 >= k.lo && j0 + kUnit <= k.len;
    const bool band = j0 + kUnit > k.band_lo;
    if (!inside) {  // what lies outside may hold anything: zero times it is not zero
      constexpr int kRow = KD * 2 / 16;
      for (int i = lane; i < kUnit * kRow; i += 32) {
        const int r = i / kRow, c = i % kRow;
        if (j0 + r < k.lo || j0 + r >= k.len)
          *reinterpret_cast<uint4*>(V + (c / 8) * 2048 + r * 128 + (c % 8) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();  // the ring's next copy comes after these writes
      __syncwarp();
    }
    uint32_t hi[NR][2], lo[NR][2];
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      float x[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        x[c] = (PAIR && second[n] ? s2[c / 2][2 * n + c % 2] : s[c / 2][2 * n + c % 2]) * p.scale2;
      if (band || !inside) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + (c / 2) * 8 + 2 * (lane % 4) + c % 2;
          if (j >= k.band_lo) x[c] += p.bias2;
          if (j < k.lo || j >= k.len) x[c] = -INFINITY;
        }
      }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      if (__any_sync(0xffffffffu, mx > m[n] + kSlack)) {
        const Join f(m[n], mx);
        m[n] = f.m;
        l[n] *= f.ca;
#pragma unroll
        for (int i = 0; i < KD / 8; ++i) {
          o[i][2 * n] *= f.ca;
          o[i][2 * n + 1] *= f.ca;
          if (kPacked) {
            o[i][2] *= f.ca;
            o[i][3] *= f.ca;
          }
        }
      }
      const float ref = m[n] == -INFINITY ? 0.f : m[n];
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] = ex2(x[c] - ref);
      l[n] += (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * c], x[2 * c + 1]);
        hi[n][c] = *reinterpret_cast<const uint32_t*>(&h);
        lo[n][c] = pack_bf16(x[2 * c] - __low2float(h), x[2 * c + 1] - __high2float(h));
      }
    }
    {
      const int r = ((lane / 8) % 2) * 8 + lane % 8;
      const uint32_t base = smem_u32(V) + r * 128;
      constexpr int n = NR - 1;
#pragma unroll
      for (int i = 0; i < KD / 16; ++i) {
        const int c = 2 * i + lane / 16;
        uint32_t v[4];
        ldsm4_t(v, base + (c / 8) * 2048 + (((c % 8) ^ (r % 8)) << 4));
        if (kPacked) {
          mma16816(o[2 * i], hi[0][0], lo[0][0], hi[0][1], lo[0][1], v[0], v[1]);
          mma16816(o[2 * i + 1], hi[0][0], lo[0][0], hi[0][1], lo[0][1], v[2], v[3]);
        } else {
          mma16816(o[2 * i], hi[0][0], hi[n][0], hi[0][1], hi[n][1], v[0], v[1]);
          mma16816(o[2 * i + 1], hi[0][0], hi[n][0], hi[0][1], hi[n][1], v[2], v[3]);
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = finite_bf16(v[k]);
          mma16816(o[2 * i], lo[0][0], lo[n][0], lo[0][1], lo[n][1], v[0], v[1]);
          mma16816(o[2 * i + 1], lo[0][0], lo[n][0], lo[0][1], lo[n][1], v[2], v[3]);
        }
      }
    }
  }

  // Completes the sums over the warp's lanes.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 1);
      l[n] += __shfl_xor_sync(0xffffffffu, l[n], 2);
    }
    if (kPacked)
#pragma unroll
      for (int i = 0; i < KD / 8; ++i)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (fabsf(o[i][c]) != INFINITY) o[i][c] += o[i][2 + c];
  }
  // Hands every row to `sink`.
  template <class Sink>
  __device__ __forceinline__ void put(int heads, const Sink& sink) const {
#pragma unroll
    for (int n = 0; n < NR; ++n)
      if (row(n) < heads) {
        if (lane % 4 == 0) sink.stats(row(n), m[n], l[n]);
        const float f = sink.factor(l[n]);
        auto* to = sink.at(row(n)) + 2 * (lane % 4);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          constexpr int kNext = PAIR ? D / 8 : 0;  // to the second KV head's sums
          sink.store(to + i * 8, f, second[n] ? o[i + kNext][2 * n] : o[i][2 * n],
                     second[n] ? o[i + kNext][2 * n + 1] : o[i][2 * n + 1]);
        }
      }
  }
};

// ------------------------------------------------------ float32: packed FMAs
//
// Logits: a lane sums a quarter of the dims for two keys (k and k + 8) and every
// head; the four lanes of a key trade partial sums so that each ends with a
// quarter of the heads.  Weights go through shared memory; then a lane owns
// D / 32 dims of every head.
//
// What bounds it: at few heads a group memory (30 sequences of 300 to 3000
// tokens, 8 heads over 8 of 128: 47 us, 78 % of the copy rate); from 4 on the
// reads of shared memory, 16 bytes a lane in 4 cycles however many lanes share
// an address.  Two keys a lane halve those of the queries (40 heads over 2 of
// 128: 41 us; 46 with a key and half of the dims a lane).  8 warps with a stage
// each hide more than 4 warps with 3.
template <int D_, int GT>  // GT: query heads of a group at most (4 or 8)
struct F32Body {
  using T = float;
  static constexpr int D = D_, kHeads = GT;
  static constexpr int kTile = kUnit * D * 4;
  static constexpr int kStages = D == 128 ? 1 : GT == 4 ? 3 : 2;
  static constexpr int kPieces = D / 16;     // 16-byte pieces of a quarter row
  static constexpr int kQuarter = D / 4 + 4; // floats of a query's quarter: the four lie in
                                             // different banks
  static constexpr int NH = GT / 4;          // heads a lane ends with
  // queries [GT][4][kQuarter], weights [16 keys][GT], factors [GT]
  static constexpr int kScratch = (GT * 4 * kQuarter + kUnit * GT + GT) * 4;
  static constexpr int NO = D / 32;          // dims a lane owns

  int lane, key, head;  // key: of the two, the first; head: the first it ends with
  float *qs, *ws, *cs;
  float2 o[GT][NO / 2];
  float m[NH], l[NH];

  __device__ __forceinline__ F32Body(int lane_, void* scratch)
      : lane(lane_),
        key(lane_ % 8),
        head((lane_ & 16 ? GT / 2 : 0) + (lane_ & 8 ? GT / 4 : 0)),
        qs(static_cast<float*>(scratch)),
        ws(qs + GT * 4 * kQuarter),
        cs(ws + kUnit * GT) {}

  __device__ __forceinline__ void begin(const T* Q, int heads) {
    __syncwarp();
    constexpr int kLoads = GT * D / 128;
    float4 x[kLoads];  // all on their way before the first is stored
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const int i = c * 128 + lane * 4;
      x[c] = i / D < heads ? *reinterpret_cast<const float4*>(Q + i) : make_float4(0, 0, 0, 0);
    }
#pragma unroll
    for (int c = 0; c < kLoads; ++c) {
      const int i = c * 128 + lane * 4;
      *reinterpret_cast<float4*>(qs + i / (D / 4) * kQuarter + i % (D / 4)) = x[c];
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < GT; ++g)
#pragma unroll
      for (int c = 0; c < NO / 2; ++c) o[g][c] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const Params& p, char* K, char* V, int j0, const Span& k) {
    const int quarter = lane / 8;
    float x[GT][2];
    {
      float2 acc[GT][2];
#pragma unroll
      for (int g = 0; g < GT; ++g) acc[g][0] = acc[g][1] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < kPieces; ++i) {
        const int piece = quarter * kPieces + i;
        const char* at = K + (piece / 8) * 2048 + key * 128 + (((piece % 8) ^ key) << 4);
        const float4 k0 = *reinterpret_cast<const float4*>(at);
        const float4 k1 = *reinterpret_cast<const float4*>(at + 8 * 128);
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          const float4 q = *reinterpret_cast<const float4*>(qs + (g * 4 + quarter) * kQuarter +
                                                            i * 4);
          const float2 qa = make_float2(q.x, q.y), qb = make_float2(q.z, q.w);
          acc[g][0] = ffma2(make_float2(k0.x, k0.y), qa, acc[g][0]);
          acc[g][0] = ffma2(make_float2(k0.z, k0.w), qb, acc[g][0]);
          acc[g][1] = ffma2(make_float2(k1.x, k1.y), qa, acc[g][1]);
          acc[g][1] = ffma2(make_float2(k1.z, k1.w), qb, acc[g][1]);
        }
      }
#pragma unroll
      for (int g = 0; g < GT; ++g)
#pragma unroll
        for (int n = 0; n < 2; ++n) x[g][n] = acc[g][n].x + acc[g][n].y;
    }
    // the quarters' sums: half of the heads to the lane 16 away, then a quarter
    // to the one 8 away
    const auto trade = [&](int half, int mask) {
      const bool up = lane & mask;
#pragma unroll
      for (int g = 0; g < GT / 2; ++g)
        if (g < half)
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            const float other =
                __shfl_xor_sync(0xffffffffu, up ? x[g][n] : x[g + half][n], mask);
            x[g][n] = (up ? x[g + half][n] : x[g][n]) + other;
          }
    };
    trade(GT / 2, 16);
    trade(GT / 4, 8);

    float mx[NH];
    bool up = false;
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const int j = j0 + key + 8 * n;
        x[i][n] = j >= k.lo && j < k.len
                      ? fmaf(x[i][n], p.scale2, j >= k.band_lo ? p.bias2 : 0.f)
                      : -INFINITY;
      }
      mx[i] = fmaxf(x[i][0], x[i][1]);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1)
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
      up |= mx[i] > m[i] + kSlack;
    }
    const bool any_up = __any_sync(0xffffffffu, up);
    if (any_up) {
#pragma unroll
      for (int i = 0; i < NH; ++i) {
        const Join f(m[i], mx[i]);
        m[i] = f.m;
        l[i] *= f.ca;
        if (key == 0) cs[head + i] = f.ca;
      }
    }
#pragma unroll
    for (int i = 0; i < NH; ++i) {
      const float ref = m[i] == -INFINITY ? 0.f : m[i];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const float w = ex2(x[i][n] - ref);
        l[i] += w;
        ws[(key + 8 * n) * GT + head + i] = w;
      }
    }
    __syncwarp();
    if (any_up) {
#pragma unroll
      for (int g = 0; g < GT; ++g) {
        const float c = cs[g];
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) {
          o[g][n].x *= c;
          o[g][n].y *= c;
        }
      }
    }
    // only the keys that are seen: what lies outside may hold anything
    const int r0 = max(k.lo - j0, 0), r1 = min(k.len - j0, kUnit);
#pragma unroll 4
    for (int r = r0; r < r1; ++r) {
      float2 v[NO / 2];
      const int dim = lane * NO, piece = dim / 4;
      const char* at =
          V + (piece / 8) * 2048 + r * 128 + (((piece % 8) ^ (r % 8)) << 4) + (dim % 4) * 4;
      if (NO == 4) {
        const float4 t = *reinterpret_cast<const float4*>(at);
        v[0] = make_float2(t.x, t.y);
        v[NO / 2 - 1] = make_float2(t.z, t.w);
      } else {
        v[0] = *reinterpret_cast<const float2*>(at);
      }
#pragma unroll
      for (int g = 0; g < GT; g += 4) {
        const float4 w = *reinterpret_cast<const float4*>(ws + r * GT + g);
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) {
          o[g][n] = ffma2(make_float2(w.x, w.x), v[n], o[g][n]);
          o[g + 1][n] = ffma2(make_float2(w.y, w.y), v[n], o[g + 1][n]);
          o[g + 2][n] = ffma2(make_float2(w.z, w.z), v[n], o[g + 2][n]);
          o[g + 3][n] = ffma2(make_float2(w.w, w.w), v[n], o[g + 3][n]);
        }
      }
    }
    __syncwarp();  // the weights are read before the next unit's are written
  }

  // Completes the sums over the warp's lanes; every lane gets all heads' m and l.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < NH; ++i) {
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (key == 0) {
        cs[head + i] = m[i];
        ws[head + i] = l[i];
      }
    }
    __syncwarp();
  }
  // The statistics a head a lane: their code, once a head in a row, would be
  // fetched for longer than it runs.
  template <class Sink>
  __device__ __forceinline__ void put(int heads, const Sink& sink) const {
    if (lane < heads) {
      sink.stats(lane, cs[lane], ws[lane]);
      qs[lane] = sink.factor(ws[lane]);
    }
    __syncwarp();
#pragma unroll
    for (int g = 0; g < GT; ++g)
      if (g < heads) {
        auto* to = sink.at(g) + lane * NO;
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) sink.store(to + 2 * n, qs[g], o[g][n].x, o[g][n].y);
      }
  }
};

// ------------------------------------------------------------------ outputs

__device__ __forceinline__ void store2(float* p, float a, float b) {
  *reinterpret_cast<float2*>(p) = make_float2(a, b);
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float a, float b) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(a, b);
}

// A finished row: O and lse of query heads h0 .. of sequence s.
template <typename T_, int D>
struct Finished {
  using T = T_;
  const Params& p;
  int s, h0;
  float bias;  // what its log-sum-exp lacks
  __device__ __forceinline__ void stats(int head, float m, float l) const {
    if (p.lse)
      p.lse[int64_t(h0 + head) * p.nseq + s] =
          l == 0.f ? -INFINITY : fmaf(m + log2f(l), kLn2, bias);
  }
  // of the sums; 0: no weight (the sums are zero, or NaN)
  __device__ __forceinline__ static float factor(float l) { return l == 0.f ? 0.f : 1.f / l; }
  __device__ __forceinline__ T* at(int head) const {
    return static_cast<T*>(p.O) + s * p.o_stride + int64_t(h0 + head) * D;
  }
  __device__ __forceinline__ static void store(T* o, float f, float a, float b) {
    store2(o, a * f, b * f);
  }
};

// A piece of a row: unnormalised sums [heads][D], maxima and sums of weights.
template <int D>
struct PieceAt {
  using T = float;
  float* o;
  float2* ml;
  __device__ __forceinline__ void stats(int head, float m, float l) const {
    ml[head] = make_float2(m, l);
  }
  __device__ __forceinline__ static float factor(float) { return 1.f; }
  __device__ __forceinline__ float* at(int head) const { return o + head * D; }
  __device__ __forceinline__ static void store(float* o, float, float a, float b) {
    store2(o, a, b);
  }
};

template <int D>
__device__ __forceinline__ PieceAt<D> piece_at(const Params& p, int64_t slot) {
  return PieceAt<D>{p.part_o + slot * p.gh * D, p.part_ml + slot * p.gh};
}

template <int D>
struct Piece {  // running joint result; a lane owns D / 32 dims
  float m = -INFINITY, l = 0.f, o[D / 32] = {};
  __device__ __forceinline__ void add(float m2, float l2, const float* o2) {
    const Join f(m, m2);
    m = f.m;
    l = fmaf(l, f.ca, l2 * f.cb);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) o[i] = fmaf(o[i], f.ca, o2[i] * f.cb);
  }
};

template <int D, class Sink>
__device__ __forceinline__ void put_row(const Sink& sink, int head, const Piece<D>& x) {
  const int lane = threadIdx.x % 32;
  if (lane == 0) sink.stats(head, x.m, x.l);
  const float f = sink.factor(x.l);
  auto* to = sink.at(head) + lane * (D / 32);
#pragma unroll
  for (int i = 0; i < D / 32; i += 2) sink.store(to + i, f, x.o[i], x.o[i + 1]);
}

// ------------------------------------------------------------ the main kernel

// What a warp tells its block of its run: the rows it shares with its
// neighbours (sequence, row of it; s < 0: none), and whether the first goes on
// past the run.
struct Cut {
  int s, r, through;  // the row the run begins in, if the run before has a part
  int s_end, r_end;   // the row it ends in, if only the runs after have another
  int any;            // the run is not empty
};

template <class Body>
struct Layout {
  static constexpr int kStageBytes = 2 * Body::kTile;
  static constexpr int kRing = kWarps * Body::kStages * kStageBytes;
  static constexpr int kPiece = Body::kHeads * Body::D * 4;  // a row's sums
  static constexpr int kOffPieces = kRing + kWarps * Body::kScratch;
  static constexpr int kBytes = kOffPieces + kWarps * kPiece + 1024;  // 1024: alignment
  static_assert(Body::kStages * kStageBytes >= kPiece);
};

template <class Body>
__global__ void __launch_bounds__(kThreads, 1)
    k_paged_attn(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const Params p) {
  using T = typename Body::T;
  using S = Layout<Body>;
  constexpr int D = Body::D, kStages = Body::kStages;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ PlanSmem plan;
  __shared__ uint64_t bars[kWarps][kStages];
  // the pieces of rows that the block's warps share: [0] of the row a warp's run
  // begins in, [1] of the row it ends in
  __shared__ float2 join_ml[2][kWarps][Body::kHeads];
  __shared__ Cut cuts_in[kWarps];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0 && p.npages > 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  // all before this ran beside the end of the launch before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan_places(p, plan, blockIdx.x == 0);
  // the joining kernel may take its place now; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const Cuts cuts = cuts_of(p, plan.before[kThreads]);
  if (blockIdx.x >= kCtas && cuts.head == cuts.total) {  // a wide table's short lengths
    if (threadIdx.x == 0) p.shared[blockIdx.x] = Shared{0, 0, 0, -1};
    return;
  }
  int64_t c0, c1;  // the block's run
  if (p.by_rows) {
    const int rows = p.nseq * p.Hkv * p.groups;  // few: 32 bits
    c0 = place_of_row(p, plan, rows * blockIdx.x / kCtas);
    c1 = place_of_row(p, plan, rows * (blockIdx.x + 1) / kCtas);
  } else {
    c0 = cuts.at(blockIdx.x);
    c1 = cuts.at(blockIdx.x + 1);
  }
  const int64_t u0 = c0 + (c1 - c0) * warp / kWarps, u1 = c0 + (c1 - c0) * (warp + 1) / kWarps;
  Walk at = {};
  bool begun = false;  // the row the run begins in is begun before it
  if (u1 > u0) {
    at = find_place(p, plan, u0, int(u1 - u0));
    begun = at.g > 0;
  }
  Cut cut{-1, 0, 0, -1, 0, at.left > 0};

  char* ring = smem + warp * kStages * S::kStageBytes;
  Body body(lane, smem + S::kRing + warp * Body::kScratch);
  bool ok = true;

  // ---- the copies: `ahead` runs up to kStages units before `at`
  Walk ahead = at;
  int issued = 0, batch = -1;      // batch: first unit of the row that `slots` covers
  int slots = -1, slots_next = -1; // lane i: pool slot of unit batch + i (+ 32), or -1
  uint32_t bad = 0;                // bit: that stage's page is outside the pool
  const int per_page = p.page_size / kUnit;
  auto load_slots = [&](int g) {
    if (g + lane >= ahead.k.n) return -1;
    const int unit = ahead.k.first + g + lane;
    const int page = p.page_table[int64_t(ahead.s) * p.max_pages + unit / per_page];
    if (page < 0 || page >= p.npages) {
      atomicOr(p.status, kStatusBadPage);
      return -1;
    }
    return page * p.page_size + (unit % per_page) * kUnit;
  };
  auto issue = [&](int stage) {
    if (batch < 0) {
      batch = ahead.g;
      slots = load_slots(batch);
      slots_next = load_slots(batch + 32);
    } else if (ahead.g >= batch + 32) {
      batch += 32;
      slots = slots_next;
      slots_next = load_slots(batch + 32);
    }
    const int slot = __shfl_sync(0xffffffffu, slots, ahead.g - batch);
    bad = (bad & ~(1u << stage)) | (uint32_t(slot < 0) << stage);
    if (lane == 0) {
      uint64_t* bar = &bars[warp][stage];
      if (slot < 0) {
        mbar_arrive(bar);
      } else {
        char* dst = ring + stage * S::kStageBytes;
        const int head = ahead.r / p.groups;
        mbar_expect_tx(bar, S::kStageBytes);
        tma_load_4d(dst, &tk, bar, 0, slot, 0, head);
        tma_load_4d(dst + Body::kTile, &tv, bar, 0, slot, 0, head);
      }
    }
    ++issued;
    if (ahead.left > 1) {
      const int s = ahead.s, r = ahead.r;
      ahead.step(p);
      // another row begins; its units have the same pages if they are still at hand
      if (ahead.s != s || (ahead.r != r && batch > 0)) batch = -1;
    } else {
      ahead.left = 0;
    }
  };
#pragma unroll 1  // `issue` is long, and this runs once
  for (int i = 0; i < kStages; ++i)
    if (ahead.left > 0) issue(i);

  // ---- while they are on their way: the row to join that the block begins in
  if (!p.by_rows && lane == 0) {
    if (u0 == c0 && u1 > u0) {
      const int64_t row = u0 - at.g;  // its first unit, if that is before the block
      const bool full = cuts.total >= kCtas;  // else blocks hold a place or none
      Shared x{at.s, marked(at.r, at.k), 0, -1};
      if (begun && row >= (full ? cuts.at(blockIdx.x - 1) : u0 - 1)) {
        x.v0 = full ? blockIdx.x - 1 : cuts.holder(row);
        x.v1 = cuts.holder(row + at.k.n - 1);
      }
      p.shared[blockIdx.x] = x;
    } else if (warp == 0 && c1 == c0) {  // an empty block
      p.shared[blockIdx.x] = Shared{0, 0, 0, -1};
      for (int i = 0; i < 2 * p.gh; ++i)
        p.part_ml[int64_t(2) * blockIdx.x * p.gh + i] = make_float2(-INFINITY, kNoSums);
    }
  }

  int done = 0, stage = 0;
  uint32_t phase = 0;
  while (at.left > 0 && ok) {
    const int group = at.r % p.groups, kvh = at.r / p.groups;
    const int h0 = kvh * p.G + group * p.gh, heads = min(p.gh, p.G - group * p.gh);
    const int n = min(at.left, at.k.n - at.g);
    const bool whole = at.g == 0 && n == at.k.n;
    body.begin(static_cast<const T*>(p.Q) + at.s * p.q_stride + int64_t(h0) * D, heads);
    for (int i = 0; i < n; ++i) {
      ok = mbar_wait(&bars[warp][stage], phase, p.status);
      if (__any_sync(0xffffffffu, !ok)) {
        ok = false;
        break;
      }
      char* src = ring + stage * S::kStageBytes;
      if (!((bad >> stage) & 1))
        body.step(p, src, src + Body::kTile, (at.k.first + at.g + i) * kUnit, at.k);
      __syncwarp();
      ++done;
      if (ahead.left > 0) issue(stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;
    body.finish();
    if (whole) {
      body.put(heads, Finished<T, D>{p, at.s, h0, at.k.band_lo == kAllBand ? p.bias : 0.f});
    } else {
      // the first row's piece keeps out of the ring, which may be in use; the
      // last's, when all is read, goes there
      const int end = begun ? 0 : 1;
      float* to = reinterpret_cast<float*>(begun ? smem + S::kOffPieces + warp * S::kPiece : ring);
      body.put(heads, PieceAt<D>{to, join_ml[end][warp]});
      if (begun)
        cut.s = at.s, cut.r = marked(at.r, at.k), cut.through = at.g + n < at.k.n;
      else
        cut.s_end = at.s, cut.r_end = marked(at.r, at.k);
    }
    begun = false;
    at.g += n - 1;
    at.left -= n - 1;
    at.step(p);
  }
  // a wait that gave up: the copies still in flight end before the block does
  if (!ok)
    for (int i = done; i < issued; ++i) {
      mbar_wait(&bars[warp][stage], phase, p.status);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }

  // ---- the rows that the block's warps share.  A chain of pieces begins with a
  // warp's last row, or with the row the block begins in, and goes on over the
  // next warps' first rows.
  if (lane == 0) cuts_in[warp] = cut;
  __syncthreads();
  {
    const Cut c = cuts_in[lane % kWarps];
    const bool one = lane < kWarps;
    const uint32_t any = __ballot_sync(0xffffffffu, one && c.any);
    const uint32_t first = __ballot_sync(0xffffffffu, one && c.s >= 0);
    const uint32_t through = __ballot_sync(0xffffffffu, one && c.s >= 0 && c.through);
    const uint32_t last = __ballot_sync(0xffffffffu, one && c.s_end >= 0);
    // chain 0: of the block's first row, chain v + 1: of warp v's last
    const uint32_t chains = (first & any & -any ? 1u : 0u) | last << 1;
    const int share = min(p.gh, kWarps);  // warps that take a chain's heads in turn
    for (int t = warp; t < __popc(chains) * share; t += kWarps) {
      uint32_t rest = chains;
      for (int i = t / share; i > 0; --i) rest &= rest - 1;
      const int v = __ffs(rest) - 2;
      const int lead = v < 0 ? __ffs(any) - 1 : v;  // the warp of its first piece
      const Cut& of = cuts_in[lead];
      const int s = v < 0 ? of.s : of.s_end, mark = v < 0 ? of.r : of.r_end, r = row_of(mark);
      const int group = r % p.groups, heads = min(p.gh, p.G - group * p.gh);
      bool open = v >= 0 || ((through >> lead) & 1);  // goes on after the pieces so far
      uint32_t more = 0;                              // warps with its further pieces
      for (uint32_t w = any >> 1 >> lead << 1 << lead; w && open; w &= w - 1) {
        more |= w & -w;
        open = through & w & -w;
      }
      for (int h = t % share; h < heads; h += share) {
        Piece<D> acc;
        auto add = [&](const char* from, float2 ml) {
          float o[D / 32];
          const float* x = reinterpret_cast<const float*>(from) + h * D + lane * (D / 32);
#pragma unroll
          for (int i = 0; i < D / 32; ++i) o[i] = x[i];
          acc.add(ml.x, ml.y, o);
        };
        add(v < 0 ? smem + S::kOffPieces + lead * S::kPiece
                  : smem + lead * kStages * S::kStageBytes,
            join_ml[v < 0 ? 0 : 1][lead][h]);
        for (uint32_t w = more; w; w &= w - 1) {
          const int k = __ffs(w) - 1;
          add(smem + S::kOffPieces + k * S::kPiece, join_ml[0][k][h]);
        }
        if (v >= 0 && !open)
          put_row(Finished<T, D>{p, s, r / p.groups * p.G + group * p.gh, bias_of(p, mark)}, h,
                  acc);
        else
          put_row(piece_at<D>(p, 2 * blockIdx.x + (v < 0 ? 0 : 1)), h, acc);
      }
    }
  }
  // sequences without keys
  for (int s = blockIdx.x; s < p.nseq && blockIdx.x < kCtas; s += kCtas) {
    if (span_of(p, s).n > 0) continue;
    for (int i = threadIdx.x; i < p.Hq * (D / 2); i += kThreads)
      store2(static_cast<T*>(p.O) + s * p.o_stride + 2 * i, 0.f, 0.f);
    for (int h = threadIdx.x; h < p.Hq && p.lse; h += kThreads)
      p.lse[int64_t(h) * p.nseq + s] = -INFINITY;
  }
}

// ---------------------------------------------------------- joining the rows

// One warp per block boundary that is the first inside its row, and a query
// head (blockIdx.y); a row that many blocks share takes the whole block.
constexpr int kJoinWarps = 8;
constexpr int kJoinAlone = 8;  // blocks of a row whose pieces one warp joins by itself

template <int D>
__device__ __forceinline__ void join_blocks(const Params& p, const Shared& row, int head, int warp,
                                            int warps, Piece<D>& acc) {
  const int lane = threadIdx.x % 32;
  for (int base = row.v0; base <= row.v1; base += 32 * warps) {
    const int v = base + lane * warps + warp;
    const int slot = v <= row.v1 ? 2 * v + (v == row.v0) : -1;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (slot >= 0) ml = __ldcg(&p.part_ml[int64_t(slot) * p.gh + head]);
    unsigned left = __ballot_sync(0xffffffffu, slot >= 0);
    while (left) {
      constexpr int kBatch = 3;
      float o[kBatch][D / 32];
      unsigned now = left;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int at = __shfl_sync(0xffffffffu, slot, now ? __ffs(now) - 1 : 0);
        const float* x = p.part_o + (int64_t(at) * p.gh + head) * D + lane * (D / 32);
        if (now) {
          if (D == 128) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(x));
            o[i][0] = t.x, o[i][1] = t.y, o[i][D / 32 - 2] = t.z, o[i][D / 32 - 1] = t.w;
          } else {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(x));
            o[i][0] = t.x, o[i][1] = t.y;
          }
        }
        now &= now - 1;
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int src = left ? __ffs(left) - 1 : 0;
        const float m = __shfl_sync(0xffffffffu, ml.x, src);
        const float l = __shfl_sync(0xffffffffu, ml.y, src);
        if (left && l != kNoSums) acc.add(m, l, o[i]);
        left &= left - 1;
      }
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kJoinWarps * 32, 4) k_paged_join(const Params p) {
  __shared__ float sm_o[kJoinWarps][D];
  __shared__ float2 sm_ml[kJoinWarps];
  const int head = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int w = blockIdx.x * kJoinWarps + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // lane i: the boundary before block blockIdx.x * 8 + i
  Shared row{0, 0, 0, -1};
  if (lane < kJoinWarps && w < kCtas + p.extra) row = p.shared[w];
  const bool split = row.v0 <= row.v1 && head < min(p.gh, p.G - row_of(row.r) % p.groups * p.gh);
  const unsigned mine = __ballot_sync(0xffffffffu, split && row.v1 - row.v0 < kJoinAlone);
  unsigned shared = __ballot_sync(0xffffffffu, split && row.v1 - row.v0 >= kJoinAlone);
  auto get_row = [&](int i) {
    return Shared{__shfl_sync(0xffffffffu, row.s, i), __shfl_sync(0xffffffffu, row.r, i),
                  __shfl_sync(0xffffffffu, row.v0, i), __shfl_sync(0xffffffffu, row.v1, i)};
  };
  auto finish = [&](const Shared& x, const Piece<D>& acc) {
    const int r = row_of(x.r);
    put_row(Finished<T, D>{p, x.s, r / p.groups * p.G + r % p.groups * p.gh, bias_of(p, x.r)},
            head, acc);
  };
  if ((mine >> warp) & 1) {
    const Shared x = get_row(warp);
    Piece<D> acc;
    join_blocks<D>(p, x, head, 0, 1, acc);
    finish(x, acc);
  }
  while (shared) {  // the same in every warp
    const Shared x = get_row(__ffs(shared) - 1);
    shared &= shared - 1;
    Piece<D> acc;
    join_blocks<D>(p, x, head, warp, kJoinWarps, acc);
    __syncthreads();
#pragma unroll
    for (int d = 0; d < D / 32; ++d) sm_o[warp][lane * (D / 32) + d] = acc.o[d];
    if (lane == 0) sm_ml[warp] = make_float2(acc.m, acc.l);
    __syncthreads();
    if (warp == 0) {
      Piece<D> all;
      for (int v = 0; v < kJoinWarps; ++v) {
        float o[D / 32];
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[d] = sm_o[v][lane * (D / 32) + d];
        all.add(sm_ml[v].x, sm_ml[v].y, o);
      }
      finish(x, all);
    }
  }
}

// ------------------------------------------------------------------ the host

mf_status fail(mf_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

mf_status check(const mf_kv_cache* cache, const mf_paged_attn_desc* a) {
  const mf_status st = check_kv_cache(cache);
  if (st != MF_OK) return st;
  if (!a) return fail(MF_ERR_INVALID_ARG, "attention descriptor is NULL");
  if (a->Hq < 1 || a->Hq % cache->Hkv != 0)
    return fail(MF_ERR_INVALID_ARG, "Hq must be a positive multiple of Hkv");
  if (a->Hq > 256) return fail(MF_ERR_UNSUPPORTED, "more than 256 query heads");
  if (!std::isfinite(a->scale) || !std::isfinite(a->band_bias))
    return fail(MF_ERR_INVALID_ARG, "scale or band_bias not finite");
  if (a->band_width < 0 || a->window < 0)
    return fail(MF_ERR_INVALID_ARG, "band_width or window < 0");
  if (!std::isfinite(a->scale * kLog2e) ||
      (a->band_width > 0 && a->band_bias * kLog2e == INFINITY))
    return fail(MF_ERR_INVALID_ARG, "scale or band_bias times log2 e not finite");
  return MF_OK;
}

// What a row is.  Query heads of one KV head are taken together, up to what a
// warp's registers hold (16 for bf16, 8 for float32); more are cut into even
// groups, each of which reads the keys again.
//
// Where a key is 128 bytes (bf16, d 64), two KV heads make a row if the query
// heads of both have room in it, for HBM is slow to bring pieces of 128 bytes:
// 64 sequences of 3 K to 8 K tokens, 32 heads over 8, 111 us, 141 with a head a
// row.  Tables with room for few units keep a head a row, which is more rows to
// share out (one sequence of 1000 tokens 9.0 us, 9.9 in pairs; 16 of up to 1000,
// with room for 54 a block, 12.1 and 12.2; 30 of them 18.4 and 17.4).
constexpr int kPairs = 40;  // units a block

struct Rows {
  bool pair;
  int Hkv, G;      // as if two KV heads were one
  int groups, gh;  // groups of query heads per KV head, heads of a group
};

Rows rows_of(const mf_kv_cache& c, int Hq) {
  const int G = Hq / c.Hkv, most = c.dt == MF_BF16 ? 16 : 8;
  const int64_t room = int64_t(c.max_pages_per_seq) * (c.page_size / kUnit) * c.nseq * c.Hkv;
  if (c.dt == MF_BF16 && c.d == 64 && c.Hkv % 2 == 0 && 2 * G <= most && room >= kCtas * kPairs)
    return Rows{true, c.Hkv / 2, 2 * G, 1, 2 * G};
  const int groups = (G + most - 1) / most;
  return Rows{false, c.Hkv, G, groups, (G + groups - 1) / groups};
}

// Where the table has room for few places a block, blocks take whole rows:
// nothing is left to join, and the second launch, 1 to 3 of the 7 to 10 us
// that short rows take, is not made.  Few: those that its warps are through
// with in that time (14 sequences of up to 215 tokens, 8 heads a KV head: 11.1
// us with the second launch, 9.0 without; float32, 19 of up to 491 tokens, 2
// heads a KV head: 10.2 with, 15.1 without).
bool whole_rows(const mf_kv_cache& c, const Rows& of) {
  const int64_t few = kWarps * (c.dt == MF_BF16 ? 4 : 2);  // so rows are few, too
  const int64_t places = int64_t(c.max_pages_per_seq) * (c.page_size / kUnit) + kRowCost;
  const int64_t rows = int64_t(c.nseq) * of.Hkv * of.groups;
  return places <= few && (rows + kCtas - 1) / kCtas * places <= few;
}

// Blocks past the first kCtas, where the table has room for a large line.
int extra_blocks(const mf_kv_cache& c, const Rows& of) {
  const int64_t units = int64_t(c.max_pages_per_seq) * (c.page_size / kUnit);
  return units * c.nseq * of.Hkv * of.groups >= int64_t(kCtas) * kLarge ? kExtra : 0;
}

size_t layout(const mf_kv_cache& c, int Hq, void* ws, Params* p) {
  const Rows of = rows_of(c, Hq);
  const int gh = of.gh, extra = extra_blocks(c, of), blocks = kCtas + extra;
  Carve k(ws);
  float* part_o = k.take<float>(size_t(2 * blocks) * gh * c.d);
  float2* part_ml = k.take<float2>(size_t(2 * blocks) * gh);
  Shared* shared = k.take<Shared>(blocks);
  if (p) {
    p->pair = of.pair;
    p->Hkv = of.Hkv;
    p->G = of.G;
    p->groups = of.groups;
    p->gh = gh;
    p->by_rows = whole_rows(c, of);
    p->extra = extra;
    p->part_o = part_o;
    p->part_ml = part_ml;
    p->shared = shared;
  }
  return (k.used + 255) & ~size_t(255);
}

template <class Body>
cudaError_t launch(const Params& p, const CUtensorMap& tk, const CUtensorMap& tv,
                   cudaStream_t st) {
  constexpr int kSmem = Layout<Body>::kBytes;
  // once per device: the call costs as much as a fifth of a launch
  static std::atomic<uint64_t> set{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);  // status_word() refuses devices past 63
  if (!(set.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(k_paged_attn<Body>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem);
    if (e != cudaSuccess) return e;
    set.fetch_or(bit, std::memory_order_relaxed);
  }
  // either launch may take its place before the one ahead of it has ended
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kCtas + p.extra);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_paged_attn<Body>, tk, tv, p);
  if (e != cudaSuccess || p.by_rows) return e;
  cfg.gridDim = dim3((kCtas + p.extra + kJoinWarps - 1) / kJoinWarps, p.gh);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_paged_join<typename Body::T, Body::D>, p);
}

// The kernel with room for the row's heads.  Measured on the batch of 64 sequences
// (1 K to 16 K tokens; float32: to 4 K), with the next larger one for comparison:
// 4 heads of bf16 217.9 us, 221.6; 8 of them 224.7, 230.7; 4 of float32 172.7,
// 189.5; 4 of bf16 with 64 dims (12 over 3) 59.9 with room for 8, 69.1 for 16.
template <int D>
cudaError_t launch_d(const Params& p, mf_dtype dt, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  if (dt == MF_BF16) {
    if constexpr (D == 64)
      if (p.pair)
        return p.gh <= 8 ? launch<Bf16Body<D, 8, true>>(p, tk, tv, st)
                         : launch<Bf16Body<D, 16, true>>(p, tk, tv, st);
    if constexpr (D == 128)  // at 64 dims the rings of 4 and 8 heads are of one depth
      if (p.gh <= 4) return launch<Bf16Body<D, 4>>(p, tk, tv, st);
    if (p.gh <= 8) return launch<Bf16Body<D, 8>>(p, tk, tv, st);
    return launch<Bf16Body<D, 16>>(p, tk, tv, st);
  }
  if (p.gh <= 4) return launch<F32Body<D, 4>>(p, tk, tv, st);
  return launch<F32Body<D, 8>>(p, tk, tv, st);
}

}  // namespace
}  // namespace mf

using namespace mf;

extern "C" {

size_t mf_paged_attn_workspace(const mf_kv_cache* cache, const mf_paged_attn_desc* attn) {
  if (check(cache, attn) != MF_OK) return 0;
  return layout(*cache, attn->Hq, nullptr, nullptr);
}

mf_status mf_paged_attn(const mf_kv_cache* cache, const mf_paged_attn_desc* attn,
                        const int32_t* lens, const void* Q, int64_t q_stride, void* O,
                        int64_t o_stride, float* lse, void* ws, size_t ws_bytes,
                        mf_stream_t stream) {
  const mf_status st = check(cache, attn);
  if (st != MF_OK) return st;
  const mf_kv_cache& c = *cache;
  const mf_paged_attn_desc& a = *attn;
  if (c.nseq > 0 && (!lens || !Q || !O)) return fail(MF_ERR_INVALID_ARG, "lens, Q or O is NULL");
  const size_t elem = c.dt == MF_BF16 ? 2 : 4;
  if (q_stride < int64_t(a.Hq) * c.d || o_stride < int64_t(a.Hq) * c.d)
    return fail(MF_ERR_INVALID_ARG, "a token stride is below heads * d");
  if (reinterpret_cast<uintptr_t>(Q) % 16 || reinterpret_cast<uintptr_t>(O) % 16 ||
      uint64_t(q_stride) * elem % 16 || uint64_t(o_stride) * elem % 16)
    return fail(MF_ERR_INVALID_ARG, "Q or O is not 16-byte aligned");
  Params p = {};
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < layout(c, a.Hq, ws, &p))
    return fail(MF_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or too small");
  if (c.nseq == 0) return MF_OK;
  p.Q = Q;
  p.O = O;
  p.lse = lse;
  p.page_table = c.page_table;
  p.lens = lens;
  p.q_stride = q_stride;
  p.o_stride = o_stride;
  p.npages = c.npages;
  p.nseq = c.nseq;
  p.Hq = a.Hq;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages_per_seq;
  p.len_add = a.len_add;
  p.band = a.band_width;
  p.window = a.window;
  p.scale2 = a.scale * kLog2e;
  p.bias = a.band_bias;
  p.bias2 = std::fmax(a.band_bias * kLog2e, -FLT_MAX);  // the type's lowest value stays finite
  p.status = status_word();
  if (!p.status) return fail(MF_ERR_CUDA, "no CUDA device");

  // The pools as [Hkv][128-byte chunks of a row][tokens][128 bytes], two bytes
  // an element whatever the type (the copies move bytes): a box is 16 tokens
  // of one head.  Without pages nothing is copied.
  CUtensorMap tk = {}, tv = {};
  if (c.npages > 0) {
    const uint64_t row = uint64_t(c.d) * elem * (p.pair ? 2 : 1);
    const uint64_t dims[4] = {64, uint64_t(c.npages) * c.page_size, row / 128, uint64_t(p.Hkv)};
    const uint64_t strides[3] = {p.Hkv * row, 128, row};
    const uint32_t box[4] = {64, kUnit, uint32_t(row / 128), 1};
    const int l2 = row < 256 ? 128 : 256;
    if (make_tmap_bf16(&tk, c.K, 4, dims, strides, box, 128, l2) != cudaSuccess ||
        make_tmap_bf16(&tv, c.V, 4, dims, strides, box, 128, l2) != cudaSuccess)
      return fail(MF_ERR_CUDA, "paged attention: no tensor map of the page pools");
  }
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = c.d == 128 ? launch_d<128>(p, c.dt, tk, tv, s)
                                   : launch_d<64>(p, c.dt, tk, tv, s);
  if (e == cudaSuccess) return MF_OK;
  char msg[160];
  std::snprintf(msg, sizeof msg, "paged attention: %s", cudaGetErrorString(e));
  return fail(MF_ERR_CUDA, msg);
}

}  // extern "C"
