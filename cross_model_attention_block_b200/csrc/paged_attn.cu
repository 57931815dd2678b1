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
//    laid end to end, are cut into equal runs, one per warp of a fixed grid;
//    every block finds the cuts itself from `lens`, so the host needs no
//    lengths and a captured call follows them.
//  * A warp runs alone: it copies its units by TMA into its own ring of
//    shared memory (one box of 16 tokens x 1 head for K, one for V, 128-byte
//    swizzled) and waits on its own barriers; no block-wide step in the loop.
//  * A row inside one warp's run is finished there.  The pieces of a cut row
//    (running maximum, sum, unnormalised O) go to the workspace, first joined
//    in shared memory when a whole block works on one row, and a second,
//    dependent launch joins them.  The cuts and the order of the sums depend
//    on the lengths alone.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdio>

#include "mf_sm100.cuh"

namespace mf {
using namespace sm100;
namespace {

constexpr int kUnit = 16;      // keys of one unit
constexpr int kRowCost = 2;    // of a row besides its units, in units
constexpr int kCtas = 148;     // one block per SM of a B200
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Start {  // where a warp's run begins
  int s, r;     // sequence and row of the sequence
  int g, n;     // units of that row before the run, and in all
};

struct Params {
  const void* Q;
  void* O;
  float* lse;
  const int32_t* page_table;
  const int32_t* lens;
  int64_t q_stride, o_stride, npages;
  int nseq, Hq, Hkv, G, page_size, max_pages, len_add, band, window;
  int groups, gh;  // groups of query heads per KV head, heads of a group
  int min_run;     // units of a run, if there are fewer than that for every warp
  float scale2, bias2;  // times log2 e
  // workspace: pieces of cut rows (two per warp: the row its run begins in,
  // the row it ends in), where the runs begin, the number of units
  float* part_o;   // [2 warps][gh][D]
  float2* part_ml; // [2 warps][gh]
  Start* starts;   // [warps]
  int64_t* total;
  unsigned* status;
};

// ------------------------------------------------------------------ the plan

struct Span {  // the keys [lo, len) of a sequence, and its units
  int lo, len, band_lo;  // the band covers keys from band_lo on
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
  k.band_lo = p.band > 0 ? clamp_int(L - p.band) : INT32_MAX;
  k.first = k.lo / kUnit;
  k.n = k.len > k.lo ? (k.len + kUnit - 1) / kUnit - k.first : 0;
  return k;
}

// The line is made of the rows' units, each row's behind kRowCost places that
// stand for what a row costs besides its units (queries, sums, output), and cut
// into kCtas << shift equal runs, 1 << shift per block.
struct Cuts {
  int64_t total;
  int shift;
  // first place of run w
  __device__ __forceinline__ int64_t at(int w) const {
    const uint64_t x = uint64_t(total) * uint32_t(w);
    return int64_t((x >> 32 ? x / kCtas : uint32_t(x) / uint32_t(kCtas)) >> shift);
  }
  // the run that holds place u
  __device__ __forceinline__ int holder(int64_t u) const {
    const uint64_t x = uint64_t(u + 1) * uint32_t(kCtas << shift) - 1;
    return x >> 32 ? int(x / uint64_t(total)) : int(uint32_t(x) / uint32_t(total));
  }
};

// Runs shorter than this cost more in pieces to join than they save: a piece
// (gh rows of float32, written and read once) is gh / 4 of a unit's bytes in
// bf16, half that in float32.
template <int WARPS>
__device__ __forceinline__ Cuts cuts_of(const Params& p, int64_t total) {
  int shift = WARPS == 8 ? 3 : 2;
  while (shift > 0 && total < (int64_t(kCtas) << shift) * p.min_run) --shift;
  return Cuts{total, shift};
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

template <int THREADS>
struct PlanSmem {
  int64_t before[THREADS + 1];  // places of the sequences before thread t's
  int64_t warp_sum[THREADS / 32];
};

// Places of every thread's share of the sequences, added up over the block.
template <int THREADS>
__device__ __forceinline__ void plan_units(const Params& p, PlanSmem<THREADS>& sm, bool report) {
  const int per = (p.nseq + THREADS - 1) / THREADS;
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
  for (int w = 0; w < warp; ++w) sum += sm.warp_sum[w];
  sm.before[threadIdx.x] = sum - mine;
  if (threadIdx.x == THREADS - 1) sm.before[THREADS] = sum;
  __syncthreads();
}

// Where a run of `n` places from place u on begins: `into` is u's place in its
// row, below kRowCost if it lies before the row's first unit.  The same u in
// the whole warp.
template <int THREADS>
__device__ __forceinline__ Walk find_place(const Params& p, const PlanSmem<THREADS>& sm, int64_t u,
                                           int n, int* into) {
  constexpr int kSub = THREADS / 32;
  const int lane = threadIdx.x % 32;
  const int t0 = (__popc(__ballot_sync(0xffffffffu, sm.before[lane * kSub] <= u)) - 1) * kSub;
  const int t = t0 - 1 + __popc(__ballot_sync(0xffffffffu, lane < kSub && sm.before[t0 + lane % kSub] <= u));
  int64_t at = u - sm.before[t];
  Walk w;
  w.s = t * ((p.nseq + THREADS - 1) / THREADS);
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
  *into = int(at - int64_t(w.r) * row);
  w.g = max(0, *into - kRowCost);
  w.left = n - max(0, kRowCost - *into);
  return w;
}

// ------------------------------------------------------- joining two pieces

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
// The query heads of a group are the rows of 16-row matrix products: S = Q K^T
// per unit, then O += P V.  The weights are kept to 2^-17 as two bf16 terms
// (the first rounded, the second its remainder), so that they lose no more
// than the float32 arithmetic around them.  Up to 8 heads leave half the rows
// of a product free: rows 8..15 then take the remainders and the two terms
// cost one product.  The tensor pipe is at most a fifth busy at G = 4, which
// is why the products are the warp-level ones: their operands and results
// stay in one warp's registers, and no warp waits for another.
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

template <int D_, int ROWS>  // ROWS: 8, 16 or 32 query heads of a group at most
struct Bf16Body {
  using T = __nv_bfloat16;
  static constexpr int D = D_, kWarps = 8;
  static constexpr int kTile = kUnit * D * 2;
  static constexpr int kStages = D == 128 ? 3 : 6;
  static constexpr int kScratch = 0;  // bytes of shared memory per warp besides the ring
  static constexpr bool kPacked = ROWS == 8;
  static constexpr int NB = ROWS == 32 ? 2 : 1;  // 16-row products
  static constexpr int NR = kPacked ? 1 : 2;     // rows of one product a thread holds
  static constexpr int KS = D / 16;

  int lane;
  uint32_t q[NB][KS][2 * NR];
  float o[NB][D / 8][4];
  float m[NB][NR], l[NB][NR];

  __device__ __forceinline__ Bf16Body(int lane_, void*) : lane(lane_) {}

  __device__ __forceinline__ int row(int b, int n) const { return b * 16 + n * 8 + lane / 4; }

  __device__ __forceinline__ void begin(const T* Q, int heads) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const bool live = row(b, n) < heads;
        const T* x = Q + (live ? row(b, n) : 0) * D + 2 * (lane % 4);
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          q[b][k][n] = live ? *reinterpret_cast<const uint32_t*>(x + k * 16) : 0u;
          q[b][k][NR + n] = live ? *reinterpret_cast<const uint32_t*>(x + k * 16 + 8) : 0u;
        }
        m[b][n] = -INFINITY;
        l[b][n] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < D / 8; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[b][i][c] = 0.f;
    }
  }

  // One unit: keys j0 .. j0+15 at `K`, values at `V`; keys outside [lo, len)
  // take no part, those from band_lo on get the bias.
  __device__ __forceinline__ void step(const Params& p, char* K, char* V, int j0, const Span& k) {
    float s[NB][2][4] = {};
    {
      const int r = (lane / 16) * 8 + lane % 8;
      const uint32_t base = smem_u32(K) + r * 128;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int c = 2 * i + (lane / 8) % 2;
        uint32_t b[4];
        ldsm4(b, base + (c / 8) * 2048 + (((c % 8) ^ (r % 8)) << 4));
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint32_t* a = q[n][i];
          mma16816(s[n][0], a[0], kPacked ? 0u : a[1], a[NR], kPacked ? 0u : a[NR + 1], b[0], b[1]);
          mma16816(s[n][1], a[0], kPacked ? 0u : a[1], a[NR], kPacked ? 0u : a[NR + 1], b[2], b[3]);
        }
      }
    }
    const bool inside = j0 >= k.lo && j0 + kUnit <= k.len;
    const bool band = j0 + kUnit > k.band_lo;
    if (!inside) {  // what lies outside may hold anything: zero times it is not zero
      constexpr int kRow = D * 2 / 16;
      for (int i = lane; i < kUnit * kRow; i += 32) {
        const int r = i / kRow, c = i % kRow;
        if (j0 + r < k.lo || j0 + r >= k.len)
          *reinterpret_cast<uint4*>(V + (c / 8) * 2048 + r * 128 + (c % 8) * 16) =
              make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();  // the ring's next copy comes after these writes
      __syncwarp();
    }
    uint32_t hi[NB][NR][2], lo[NB][NR][2];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        float x[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = s[b][c / 2][2 * n + c % 2] * p.scale2;
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
        if (__any_sync(0xffffffffu, mx > m[b][n])) {
          const Join f(m[b][n], mx);
          m[b][n] = f.m;
          l[b][n] *= f.ca;
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[b][i][2 * n] *= f.ca;
            o[b][i][2 * n + 1] *= f.ca;
            if (kPacked) {
              o[b][i][2] *= f.ca;
              o[b][i][3] *= f.ca;
            }
          }
        }
        const float ref = m[b][n] == -INFINITY ? 0.f : m[b][n];
#pragma unroll
        for (int c = 0; c < 4; ++c) x[c] = ex2(x[c] - ref);
        l[b][n] += (x[0] + x[1]) + (x[2] + x[3]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * c], x[2 * c + 1]);
          hi[b][n][c] = *reinterpret_cast<const uint32_t*>(&h);
          lo[b][n][c] = pack_bf16(x[2 * c] - __low2float(h), x[2 * c + 1] - __high2float(h));
        }
      }
    }
    {
      const int r = ((lane / 8) % 2) * 8 + lane % 8;
      const uint32_t base = smem_u32(V) + r * 128;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int c = 2 * i + lane / 16;
        uint32_t v[4];
        ldsm4_t(v, base + (c / 8) * 2048 + (((c % 8) ^ (r % 8)) << 4));
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          if (kPacked) {
            mma16816(o[b][2 * i], hi[b][0][0], lo[b][0][0], hi[b][0][1], lo[b][0][1], v[0], v[1]);
            mma16816(o[b][2 * i + 1], hi[b][0][0], lo[b][0][0], hi[b][0][1], lo[b][0][1], v[2],
                     v[3]);
          } else {
            constexpr int n = NR - 1;
            mma16816(o[b][2 * i], hi[b][0][0], hi[b][n][0], hi[b][0][1], hi[b][n][1], v[0], v[1]);
            mma16816(o[b][2 * i + 1], hi[b][0][0], hi[b][n][0], hi[b][0][1], hi[b][n][1], v[2],
                     v[3]);
            mma16816(o[b][2 * i], lo[b][0][0], lo[b][n][0], lo[b][0][1], lo[b][n][1], v[0], v[1]);
            mma16816(o[b][2 * i + 1], lo[b][0][0], lo[b][n][0], lo[b][0][1], lo[b][n][1], v[2],
                     v[3]);
          }
        }
      }
    }
  }

  // Completes the sums over the warp's lanes.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        l[b][n] += __shfl_xor_sync(0xffffffffu, l[b][n], 1);
        l[b][n] += __shfl_xor_sync(0xffffffffu, l[b][n], 2);
        if (kPacked)
#pragma unroll
          for (int i = 0; i < D / 8; ++i) {
            o[b][i][0] += o[b][i][2];
            o[b][i][1] += o[b][i][3];
          }
      }
  }
  // Hands every row to `sink`, pair of dims by pair of dims.
  template <class Sink>
  __device__ __forceinline__ void put(int heads, const Sink& sink) const {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int n = 0; n < NR; ++n)
        if (row(b, n) < heads) {
          const auto to = sink.row(row(b, n), m[b][n], l[b][n], lane % 4 == 0);
#pragma unroll
          for (int i = 0; i < D / 8; ++i)
            to.store(i * 8 + 2 * (lane % 4), o[b][i][2 * n], o[b][i][2 * n + 1]);
        }
  }
};

// ------------------------------------------------------ float32: packed FMAs
//
// Logits: lane (half, key) sums half of the dims for every head, the two
// halves trade partial sums so that each ends with half of the heads (head
// 2 i + half).  Weights go through shared memory, each twice in a row, the
// operand of a packed FMA; then a lane owns D / 32 dims of every head.
template <int D_, int GT>  // GT: query heads of a group at most (even)
struct F32Body {
  using T = float;
  static constexpr int D = D_, kWarps = D == 128 ? 4 : 8;
  static constexpr int kTile = kUnit * D * 4;
  static constexpr int kStages = GT == 16 ? 2 : 3;
  // queries [GT][D], weights [16 keys][GT][2], factors [GT]
  static constexpr int kScratch = GT * D * 4 + kUnit * GT * 8 + GT * 4 + 64;
  static constexpr int NO = D / 32;       // dims a lane owns

  int lane;
  float *qs, *ws, *cs;
  float2 o[GT][NO / 2];
  float m[GT / 2], l[GT / 2];

  __device__ __forceinline__ F32Body(int lane_, void* scratch)
      : lane(lane_), qs(static_cast<float*>(scratch)), ws(qs + GT * D), cs(ws + kUnit * GT * 2) {}

  __device__ __forceinline__ void begin(const T* Q, int heads) {
    __syncwarp();
    for (int i = lane * 4; i < GT * D; i += 128)
      *reinterpret_cast<float4*>(qs + i) =
          i / D < heads ? *reinterpret_cast<const float4*>(Q + i) : make_float4(0, 0, 0, 0);
    __syncwarp();
#pragma unroll
    for (int g = 0; g < GT; ++g)
#pragma unroll
      for (int c = 0; c < NO / 2; ++c) o[g][c] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < GT / 2; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }

  __device__ __forceinline__ void step(const Params& p, char* K, char* V, int j0, const Span& k) {
    const int key = lane % 16, half = lane / 16;
    float x[GT / 2];
    {
      float2 acc[GT];
#pragma unroll
      for (int g = 0; g < GT; ++g) acc[g] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {  // 16-byte pieces of this half's dims
        const int piece = half * (D / 8) + i;
        const float4 kv = *reinterpret_cast<const float4*>(
            K + (piece / 8) * 2048 + key * 128 + (((piece % 8) ^ (key % 8)) << 4));
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          const float4 qv = *reinterpret_cast<const float4*>(qs + g * D + piece * 4);
          acc[g] = ffma2(make_float2(kv.x, kv.y), make_float2(qv.x, qv.y), acc[g]);
          acc[g] = ffma2(make_float2(kv.z, kv.w), make_float2(qv.z, qv.w), acc[g]);
        }
      }
#pragma unroll
      for (int i = 0; i < GT / 2; ++i) {
        const float a = acc[2 * i].x + acc[2 * i].y, b = acc[2 * i + 1].x + acc[2 * i + 1].y;
        const float other = __shfl_xor_sync(0xffffffffu, half ? a : b, 16);
        x[i] = ((half ? b : a) + other) * p.scale2;
      }
    }
    const int j = j0 + key;
    const bool seen = j >= k.lo && j < k.len;
    const float bias = j >= k.band_lo ? p.bias2 : 0.f;
    bool up = false;
    float mx[GT / 2];
#pragma unroll
    for (int i = 0; i < GT / 2; ++i) {
      x[i] = seen ? x[i] + bias : -INFINITY;
      mx[i] = x[i];
#pragma unroll
      for (int d = 8; d > 0; d >>= 1)
        mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
      up |= mx[i] > m[i];
    }
    const bool any_up = __any_sync(0xffffffffu, up);
    if (any_up) {
#pragma unroll
      for (int i = 0; i < GT / 2; ++i) {
        const Join f(m[i], mx[i]);
        m[i] = f.m;
        l[i] *= f.ca;
        if (key == 0) cs[2 * i + half] = f.ca;
      }
    }
#pragma unroll
    for (int i = 0; i < GT / 2; ++i) {
      const float w = ex2(x[i] - (m[i] == -INFINITY ? 0.f : m[i]));
      l[i] += w;
      *reinterpret_cast<float2*>(ws + (key * GT + 2 * i + half) * 2) = make_float2(w, w);
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
      for (int g = 0; g < GT; g += 2) {
        const float4 w = *reinterpret_cast<const float4*>(ws + (r * GT + g) * 2);
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) {
          o[g][n] = ffma2(make_float2(w.x, w.y), v[n], o[g][n]);
          o[g + 1][n] = ffma2(make_float2(w.z, w.w), v[n], o[g + 1][n]);
        }
      }
    }
    __syncwarp();  // the weights are read before the next unit's are written
  }

  // Completes the sums over the warp's lanes; every lane gets all heads' m and l.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int i = 0; i < GT / 2; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      if (lane % 16 == 0) {
        cs[2 * i + lane / 16] = m[i];
        ws[2 * i + lane / 16] = l[i];
      }
    }
    __syncwarp();
  }
  template <class Sink>
  __device__ __forceinline__ void put(int heads, const Sink& sink) const {
#pragma unroll
    for (int g = 0; g < GT; ++g)
      if (g < heads) {
        const auto to = sink.row(g, cs[g], ws[g], lane == 0);
#pragma unroll
        for (int n = 0; n < NO / 2; ++n) to.store(lane * NO + 2 * n, o[g][n].x, o[g][n].y);
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
template <typename T, int D>
struct Finished {
  const Params& p;
  int s, h0;
  struct To {
    T* o;
    float inv;
    bool none;  // nothing seen: zero, whatever was summed
    __device__ __forceinline__ void store(int dim, float a, float b) const {
      store2(o + dim, none ? 0.f : a * inv, none ? 0.f : b * inv);
    }
  };
  __device__ __forceinline__ To row(int head, float m, float l, bool first) const {
    const bool none = l == 0.f;
    if (first && p.lse)
      p.lse[int64_t(h0 + head) * p.nseq + s] = none ? -INFINITY : (m + log2f(l)) * kLn2;
    return To{static_cast<T*>(p.O) + s * p.o_stride + int64_t(h0 + head) * D, 1.f / l, none};
  }
};

// A piece of a row: unnormalised sums [heads][D], maxima and sums of weights.
template <int D>
struct PieceAt {
  float* o;
  float2* ml;
  struct To {
    float* o;
    __device__ __forceinline__ void store(int dim, float a, float b) const {
      store2(o + dim, a, b);
    }
  };
  __device__ __forceinline__ To row(int head, float m, float l, bool first) const {
    if (first) ml[head] = make_float2(m, l);
    return To{o + head * D};
  }
};

template <int D>
__device__ __forceinline__ PieceAt<D> piece_at(const Params& p, int64_t slot) {
  return PieceAt<D>{p.part_o + slot * p.gh * D, p.part_ml + slot * p.gh};
}

// ------------------------------------------------------------ the main kernel

template <class Body>
struct Shared {
  static constexpr int kStageBytes = 2 * Body::kTile;
  static constexpr int kRing = Body::kWarps * Body::kStages * kStageBytes;
  static constexpr int kBytes = kRing + Body::kWarps * Body::kScratch + 1024;  // 1024: alignment
};

template <class Body>
__global__ void __launch_bounds__(Body::kWarps * 32, 1)
    k_paged_attn(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                 const Params p) {
  using T = typename Body::T;
  using S = Shared<Body>;
  constexpr int D = Body::D, kWarps = Body::kWarps, kStages = Body::kStages;
  constexpr int kThreads = kWarps * 32;
  extern __shared__ char smem_raw[];
  char* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ PlanSmem<kThreads> plan;
  __shared__ uint64_t bars[kWarps][kStages];
  __shared__ float2 join_ml[kWarps][32];

  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(&bars[warp][i], 1);
    fence_barrier_init();
    fence_proxy_async_smem();
  }
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  // all before this ran beside the end of the launch before
  asm volatile("griddepcontrol.wait;" ::: "memory");
  plan_units<kThreads>(p, plan, blockIdx.x == 0);
  // the joining kernel may take its place now; it waits for this one's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const Cuts cuts = cuts_of<kWarps>(p, plan.before[kThreads]);
  const int w0 = blockIdx.x << cuts.shift, w = w0 + warp;
  const int64_t c0 = cuts.at(w0), c1 = cuts.at(w0 + (1 << cuts.shift));
  int64_t u0 = c1, u1 = c1;
  if (warp >> cuts.shift == 0) {
    u0 = cuts.at(w);
    u1 = cuts.at(w + 1);
  }
  Walk at = {};
  bool mine = false;   // this block's whole run lies in one row
  bool begun = false;  // the row the run begins in, at a unit of it
  if (u1 > u0) {
    int into;
    at = find_place<kThreads>(p, plan, u0, int(u1 - u0), &into);
    const int64_t row = u0 - into + kRowCost;  // its first unit
    begun = u0 >= row;
    mine = row <= c0 && row + at.k.n >= c1;
  }
  if (lane == 0 && warp >> cuts.shift == 0) p.starts[w] = Start{at.s, at.r, at.g, at.k.n};
  if (w == 0 && lane == 0) *p.total = cuts.total;
  join_ml[warp][lane] = make_float2(-INFINITY, 0.f);

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
    if (whole && !mine) {
      body.put(heads, Finished<T, D>{p, at.s, h0});
    } else {
      PieceAt<D> to = piece_at<D>(p, begun ? 2 * w : 2 * w + 1);
      if (mine) to = PieceAt<D>{reinterpret_cast<float*>(ring), join_ml[warp]};
      body.put(heads, to);
    }
    begun = false;
    if (mine) break;
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

  if (__syncthreads_or(mine)) {
    // the warps' pieces of the row are in the (now idle) ring; the row is that
    // of the first warp whose run is not empty
    __shared__ int row_s, row_r;
    __shared__ bool row_whole;
    if (mine && u0 == c0 && lane == 0) {
      row_s = at.s;
      row_r = at.r;
      row_whole = at.g == 0 && c1 - c0 == at.k.n;
    }
    __syncthreads();
    const int g2 = row_r % p.groups, hh = row_r / p.groups * p.G + g2 * p.gh;
    const int nh = min(p.gh, p.G - g2 * p.gh);
    for (int i = threadIdx.x; i < nh * (D / 2); i += kThreads) {
      const int h = i / (D / 2), d = i % (D / 2) * 2;
      float2 ml[kWarps], t[kWarps];
      float m = -INFINITY, l = 0.f, a = 0.f, b = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        ml[v] = join_ml[v][h];
        t[v] = *reinterpret_cast<const float2*>(smem + v * kStages * S::kStageBytes +
                                                (h * D + d) * 4);
        m = fmaxf(m, ml[v].x);
      }
      const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const float c = ex2(ml[v].x - ref);
        const bool some = ml[v].y != 0.f;  // else its sums are not there
        l = fmaf(ml[v].y, c, l);
        a = fmaf(some ? t[v].x : 0.f, c, a);
        b = fmaf(some ? t[v].y : 0.f, c, b);
      }
      if (row_whole)
        Finished<T, D>{p, row_s, hh}.row(h, m, l, d == 0).store(d, a, b);
      else
        piece_at<D>(p, int64_t(2) * w0).row(h, m, l, d == 0).store(d, a, b);
    }
  }
  // sequences without keys
  for (int s = blockIdx.x; s < p.nseq; s += kCtas) {
    if (span_of(p, s).n > 0) continue;
    for (int i = threadIdx.x; i < p.Hq * (D / 2); i += kThreads)
      store2(static_cast<T*>(p.O) + s * p.o_stride + 2 * i, 0.f, 0.f);
    for (int h = threadIdx.x; h < p.Hq && p.lse; h += kThreads)
      p.lse[int64_t(h) * p.nseq + s] = -INFINITY;
  }
}

// ---------------------------------------------------------- joining the rows

// One warp per cut that is the first inside its row, and a query head
// (blockIdx.y); a row of many pieces takes the whole block.
constexpr int kJoinWarps = 8;
constexpr int kJoinAlone = 8;  // runs of a row that one warp joins by itself

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

struct Row {
  int64_t a, e;  // units
  int s, r;
  int v0, v1;    // first and last run that holds one of them
};

template <int D>
__device__ __forceinline__ void join_runs(const Params& p, const Row& row, const Cuts& cuts,
                                          int head, int warp, int warps, Piece<D>& acc) {
  const int lane = threadIdx.x % 32;
  // eights of runs go round the warps, so that the pieces of whole blocks do too
  for (int base = row.v0 & ~7; base <= row.v1; base += 32 * warps) {
    const int v = base + (lane / 8 * warps + warp) * 8 + lane % 8;
    int slot = -1;
    if (v >= row.v0 && v <= row.v1) {
      const int64_t u0 = cuts.at(v), u1 = cuts.at(v + 1);
      const int w0 = v >> cuts.shift << cuts.shift;
      const int64_t c0 = cuts.at(w0), c1 = cuts.at(w0 + (1 << cuts.shift));
      if (u0 < u1) {
        if (c0 >= row.a && c1 <= row.e)  // joined by its block
          slot = u0 == c0 ? 2 * w0 : -1;
        else
          slot = u0 >= row.a ? 2 * v : 2 * v + 1;
      }
    }
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
        if (left && l != 0.f) acc.add(m, l, o[i]);  // l = 0: an empty piece, its sums void
        left &= left - 1;
      }
    }
  }
}

template <typename T, int D>
__device__ __forceinline__ void put_row(const Params& p, const Row& row, int head,
                                        const Piece<D>& x) {
  const int group = row.r % p.groups;
  const int lane = threadIdx.x % 32;
  const Finished<T, D> sink{p, row.s, row.r / p.groups * p.G + group * p.gh};
  const auto to = sink.row(head, x.m, x.l, lane == 0);
#pragma unroll
  for (int i = 0; i < D / 32; i += 2) to.store(lane * (D / 32) + i, x.o[i], x.o[i + 1]);
}

template <typename T, int D, int WARPS>  // WARPS of the main kernel's blocks
__global__ void __launch_bounds__(kJoinWarps * 32, 4) k_paged_join(const Params p) {
  __shared__ float sm_o[kJoinWarps][D];
  __shared__ float2 sm_ml[kJoinWarps];
  const int head = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int w = blockIdx.x * kJoinWarps + lane;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Start st = lane < kJoinWarps ? p.starts[w] : Start{};
  const Cuts cuts = cuts_of<WARPS>(p, *p.total);
  if (blockIdx.x * kJoinWarps >= kCtas << cuts.shift) return;

  // lane i: the cut before run blockIdx.x * 8 + i
  Row row = {};
  bool split = false;
  if (lane < kJoinWarps && w > 0 && w < kCtas << cuts.shift) {
    const int64_t u = cuts.at(w);
    const int group = st.r % p.groups, heads = min(p.gh, p.G - group * p.gh);
    if (cuts.at(w + 1) > u && st.g > 0 && head < heads) {
      row = Row{u - st.g, u - st.g + st.n, st.s, st.r, 0, 0};
      // the first cut inside the row: the run before, the last that is not
      // empty, begins no later than the row
      const bool full = cuts.total >= kCtas << cuts.shift;
      split = row.a >= (full ? cuts.at(w - 1) : u - 1);
      if (split) {
        row.v0 = full ? w - 1 : cuts.holder(row.a);
        row.v1 = cuts.holder(row.e - 1);
        const int w0 = row.v0 >> cuts.shift << cuts.shift;
        // a block that held just this row is done with it
        if (row.a == cuts.at(w0) && row.e == cuts.at(w0 + (1 << cuts.shift))) split = false;
      }
    }
  }
  const unsigned mine = __ballot_sync(0xffffffffu, split && row.v1 - row.v0 < kJoinAlone);
  unsigned shared = __ballot_sync(0xffffffffu, split && row.v1 - row.v0 >= kJoinAlone);
  auto row_of = [&](int i) {
    Row x;
    x.a = __shfl_sync(0xffffffffu, row.a, i);
    x.e = __shfl_sync(0xffffffffu, row.e, i);
    x.s = __shfl_sync(0xffffffffu, row.s, i);
    x.r = __shfl_sync(0xffffffffu, row.r, i);
    x.v0 = __shfl_sync(0xffffffffu, row.v0, i);
    x.v1 = __shfl_sync(0xffffffffu, row.v1, i);
    return x;
  };
  if ((mine >> warp) & 1) {
    const Row x = row_of(warp);
    Piece<D> acc;
    join_runs<D>(p, x, cuts, head, 0, 1, acc);
    put_row<T, D>(p, x, head, acc);
  }
  while (shared) {  // the same in every warp
    const Row x = row_of(__ffs(shared) - 1);
    shared &= shared - 1;
    Piece<D> acc;
    join_runs<D>(p, x, cuts, head, warp, kJoinWarps, acc);
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
      put_row<T, D>(p, x, head, all);
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
  return MF_OK;
}

// Query heads of one KV head are taken together, up to what a warp's registers
// hold (32 for bf16, 16 for float32); more are cut into even groups, each of
// which reads the keys again.
int head_groups(const mf_kv_cache& c, int Hq) {
  const int G = Hq / c.Hkv, most = c.dt == MF_BF16 ? 32 : 16;
  return (G + most - 1) / most;
}

int warps_of(const mf_kv_cache& c) { return c.dt == MF_F32 && c.d == 128 ? 4 : 8; }

size_t layout(const mf_kv_cache& c, int Hq, void* ws, Params* p) {
  const int groups = head_groups(c, Hq), G = Hq / c.Hkv, gh = (G + groups - 1) / groups;
  const size_t runs = size_t(kCtas) * warps_of(c);
  Carve k(ws);
  float* part_o = k.take<float>(2 * runs * gh * c.d);
  float2* part_ml = k.take<float2>(2 * runs * gh);
  Start* starts = k.take<Start>(runs);
  int64_t* total = k.take<int64_t>(1);
  if (p) {
    p->groups = groups;
    p->gh = gh;
    p->min_run = std::max(1, gh / (c.dt == MF_BF16 ? 8 : 16));
    p->part_o = part_o;
    p->part_ml = part_ml;
    p->starts = starts;
    p->total = total;
  }
  return (k.used + 255) & ~size_t(255);
}

template <class Body>
cudaError_t launch(const Params& p, const CUtensorMap& tk, const CUtensorMap& tv,
                   cudaStream_t st) {
  constexpr int kSmem = Shared<Body>::kBytes;
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
  cfg.gridDim = dim3(kCtas);
  cfg.blockDim = dim3(Body::kWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_paged_attn<Body>, tk, tv, p);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((kCtas * Body::kWarps + kJoinWarps - 1) / kJoinWarps, p.gh);
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_paged_join<typename Body::T, Body::D, Body::kWarps>, p);
}

template <int D>
cudaError_t launch_d(const Params& p, mf_dtype dt, const CUtensorMap& tk, const CUtensorMap& tv,
                     cudaStream_t st) {
  if (dt == MF_BF16) {
    if (p.gh <= 8) return launch<Bf16Body<D, 8>>(p, tk, tv, st);
    if (p.gh <= 16) return launch<Bf16Body<D, 16>>(p, tk, tv, st);
    return launch<Bf16Body<D, 32>>(p, tk, tv, st);
  }
  if (p.gh <= 4) return launch<F32Body<D, 4>>(p, tk, tv, st);
  if (p.gh <= 8) return launch<F32Body<D, 8>>(p, tk, tv, st);
  return launch<F32Body<D, 16>>(p, tk, tv, st);
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
  p.Hkv = c.Hkv;
  p.G = a.Hq / c.Hkv;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages_per_seq;
  p.len_add = a.len_add;
  p.band = a.band_width;
  p.window = a.window;
  p.scale2 = a.scale * kLog2e;
  p.bias2 = a.band_bias * kLog2e;
  p.status = status_word();
  if (!p.status) return fail(MF_ERR_CUDA, "no CUDA device");

  // The pools as [Hkv][128-byte chunks of a row][tokens][128 bytes], two bytes
  // an element whatever the type (the copies move bytes): a box is 16 tokens
  // of one head.  Without pages nothing is copied.
  CUtensorMap tk = {}, tv = {};
  if (c.npages > 0) {
    const uint64_t row = uint64_t(c.d) * elem;
    const uint64_t dims[4] = {64, uint64_t(c.npages) * c.page_size, row / 128, uint64_t(c.Hkv)};
    const uint64_t strides[3] = {c.Hkv * row, 128, row};
    const uint32_t box[4] = {64, kUnit, uint32_t(row / 128), 1};
    if (make_tmap_bf16(&tk, c.K, 4, dims, strides, box, 128) != cudaSuccess ||
        make_tmap_bf16(&tv, c.V, 4, dims, strides, box, 128) != cudaSuccess)
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
