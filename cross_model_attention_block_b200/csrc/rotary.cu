// Rotary positions, and the append of new keys and values to a paged cache
// with the rotation on the way.
//
// MapFlow article (163.com, "让复用真正省时，还需要解决存储和执行问题"): the
// receiver keeps its own V and works with PagedAttention; the maps a sender
// hands over are those of its rotated queries and keys.
//
// A token's pair i turns by position * f_i.  The angle is held as 64-bit
// fixed-point turns: position * phase_i modulo 2^64 drops whole turns without
// rounding, at any 32-bit position (a float32 product is off by 0.004 rad at
// position 100,000).  The nearest quarter turn is taken off in the integer and
// turns cosine and sine afterwards; what is left, at most an eighth of a turn,
// goes to sincospif as float32 half turns, good to 2^-24 of itself.
//
// Bound by memory: every element is read and written once, a few FMAs each.
// A block first places its tokens (sequence, position, page) and computes
// their sines into shared memory, each once; then its warps walk the tokens'
// heads (Q, K and V alike), two 16-byte packs a lane and step, and read the
// sines where they are used.  Loads are hidden by the number of warps: six
// blocks on an SM at 39 registers.  Measured at 32,768 tokens of 40 + 40 heads
// of 128: sines kept in registers and four heads loaded ahead (115 registers,
// two blocks) 317 us; two steps loaded ahead 257; as here 205 (6.6 TB/s).
#include <algorithm>
#include <cmath>
#include <cstdio>

#include "mf_device.cuh"
#include "mf_internal.h"

namespace mf {
namespace {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryBlocks = 6;  // resident on an SM
constexpr int kSms = 148;

struct RotaryParams {
  // rotation (half = 0: none)
  const uint64_t* phases;
  float scale;
  int half;  // rot_dim / 2
  bool backward;
  // tokens
  int64_t ntok;
  int nseq;
  const int32_t* cu;
  const int32_t* start;
  // rows
  int Hq, Hk, Hv, d;
  const void *Q, *K, *V;
  int64_t q_stride, k_stride, v_stride;
  void *Qo, *Ko, *Vo;
  int64_t qo_stride, ko_stride;
  bool paged;  // Ko and Vo are page pools
  const int32_t* page_table;
  int page_size, max_pages;
  int64_t npages;
  unsigned* status;
  int tokens;  // of a block
};

constexpr int kMaxTokens = 4;  // of a block

// Rows of K's and V's outputs that do not exist.
constexpr int64_t kNoSlot = -1;   // the token's place is outside the table or the pool
constexpr int64_t kPadding = -2;  // no token: its query is left alone, too

template <typename T, int N>
struct alignas(sizeof(T) * N) Pack {
  T v[N];
};

// A unit: two packs of VEC elements of one head: the first and second halves
// of VEC pairs (half layout), 2 VEC neighbours (interleaved), or 2 VEC copied
// elements.
template <typename T, int VEC, bool INTERLEAVED>
__device__ __forceinline__ void turn_pair(Pack<T, VEC>& a, Pack<T, VEC>& b, int i, float co,
                                          float si) {
  constexpr bool I = INTERLEAVED;
  const bool first = 2 * i < VEC;
  const T ta = !I ? a.v[i] : first ? a.v[2 * i % VEC] : b.v[2 * i % VEC];
  const T tb = !I ? b.v[i] : 2 * i + 1 < VEC ? a.v[(2 * i + 1) % VEC] : b.v[(2 * i + 1) % VEC];
  const float x = to_f32(ta), y = to_f32(tb);
  const T ra = from_f32<T>(fmaf(x, co, -y * si)), rb = from_f32<T>(fmaf(x, si, y * co));
  if (!I) {
    a.v[i] = ra;
    b.v[i] = rb;
  } else {
    if (first)
      a.v[2 * i % VEC] = ra;
    else
      b.v[2 * i % VEC] = ra;
    if (2 * i + 1 < VEC)
      a.v[(2 * i + 1) % VEC] = rb;
    else
      b.v[(2 * i + 1) % VEC] = rb;
  }
}

template <typename T, int VEC, bool INTERLEAVED, int D>
__global__ void __launch_bounds__(kRotaryThreads, kRotaryBlocks) k_rotary(const RotaryParams p) {
  constexpr int kUnits = D / (2 * VEC);  // of a head
  constexpr int kPairs = D / 2;
  // cosines and sines, two pairs in a row: pairs 2 c and 2 c + 1 of unit u at
  // [token][c][u], so that neighbouring lanes read neighbouring 16 bytes
  constexpr int kC = VEC >= 2 ? VEC / 2 : 1, kIn = VEC >= 2 ? 2 : 1;
  __shared__ alignas(16) float2 turns[kMaxTokens][kPairs];
  __shared__ int64_t rows[kMaxTokens], positions[kMaxTokens];
  const int64_t t0 = int64_t(blockIdx.x) * p.tokens;
  const int live = int(min(int64_t(p.tokens), p.ntok - t0));
  asm volatile("griddepcontrol.wait;" ::: "memory");

  if (threadIdx.x < live) {
    const int64_t t = t0 + threadIdx.x;
    const int s = p.cu ? upper_index(p.cu, p.nseq + 1, t) : int(t);
    const bool padding = s == p.nseq;  // behind the last sequence
    const int32_t first = p.start && !padding ? p.start[s] : 0;
    const int64_t pos = int64_t(first) + (p.cu ? t - p.cu[s] : 0);
    int64_t row = t;  // of K's and V's outputs
    if (padding || p.paged) {
      row = kPadding;
      if (!padding && first >= 0) {  // else a padding sequence
        row = kNoSlot;
        int32_t at = -1;
        if (pos >= 0 && pos < int64_t(p.max_pages) * p.page_size)
          at = p.page_table[int64_t(s) * p.max_pages + int(pos) / p.page_size];
        if (at < 0 || at >= p.npages)
          atomicOr(p.status, kStatusBadPage);
        else
          row = int64_t(at) * p.page_size + int(pos) % p.page_size;
      }
    }
    rows[threadIdx.x] = row;
    positions[threadIdx.x] = pos;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < live * kPairs; i += kRotaryThreads) {
    const int token = i / kPairs, pair = i % kPairs;
    if (pair >= p.half) continue;
    const uint64_t angle = uint64_t(positions[token]) * p.phases[pair];
    float si, co;
    const int quarters = int((angle + (uint64_t(1) << 61)) >> 62);
    const int64_t rest = int64_t(angle - (uint64_t(quarters) << 62));
    sincospif(float(rest) * 0x1p-63f, &si, &co);
    if (quarters & 1) {
      const float x = co;
      co = -si;
      si = x;
    }
    if (quarters & 2) {
      co = -co;
      si = -si;
    }
    const int u = pair / VEC, c = pair % VEC / kIn;
    turns[token][(c * kUnits + u) * kIn + pair % kIn] =
        make_float2(co * p.scale, si * (p.backward ? -p.scale : p.scale));
  }
  __syncthreads();

  // 32 units a step; the warps take steps in turn
  const int H = p.Hq + p.Hk + p.Hv, per_token = (H * kUnits + 31) / 32;
  int token = 0;
  for (int step = threadIdx.x / 32;; step += kRotaryThreads / 32) {
    while (step >= per_token) {
      step -= per_token;
      ++token;
    }
    if (token >= live) break;
    const int item = step * 32 + threadIdx.x % 32, h = item / kUnits, u = item % kUnits;
    const int64_t t = t0 + token, row = rows[token];
    if (h >= H || row == kPadding || (row == kNoSlot && h >= p.Hq)) continue;
    const T* in;
    T* out;
    if (h < p.Hq) {
      in = static_cast<const T*>(p.Q) + t * p.q_stride + h * D;
      out = static_cast<T*>(p.Qo) + t * p.qo_stride + h * D;
    } else if (h < p.Hq + p.Hk) {
      in = static_cast<const T*>(p.K) + t * p.k_stride + (h - p.Hq) * D;
      out = static_cast<T*>(p.Ko) + row * p.ko_stride + (h - p.Hq) * D;
    } else {
      in = static_cast<const T*>(p.V) + t * p.v_stride + (h - p.Hq - p.Hk) * D;
      out = static_cast<T*>(p.Vo) + row * p.ko_stride + (h - p.Hq - p.Hk) * D;
    }
    // units 0 .. half/VEC-1 rotate, the rest copy the dims past rot_dim; V's
    // are copied at the same offsets
    const bool pairs = u * VEC < p.half;
    const int off_a = pairs && !INTERLEAVED ? u * VEC : 2 * u * VEC;
    const int off_b = off_a + (pairs && !INTERLEAVED ? p.half : VEC);
    Pack<T, VEC> a = *reinterpret_cast<const Pack<T, VEC>*>(in + off_a);
    Pack<T, VEC> b = *reinterpret_cast<const Pack<T, VEC>*>(in + off_b);
    if (pairs && h < p.Hq + p.Hk) {
      const float2* cs = &turns[token][u * kIn];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if constexpr (VEC >= 2) {
          const float4 w = *reinterpret_cast<const float4*>(cs + c * kUnits * 2);
          turn_pair<T, VEC, INTERLEAVED>(a, b, 2 * c, w.x, w.y);
          turn_pair<T, VEC, INTERLEAVED>(a, b, 2 * c + 1, w.z, w.w);
        } else {
          turn_pair<T, VEC, INTERLEAVED>(a, b, 0, cs->x, cs->y);
        }
      }
    }
    *reinterpret_cast<Pack<T, VEC>*>(out + off_a) = a;
    *reinterpret_cast<Pack<T, VEC>*>(out + off_b) = b;
  }
}

template <typename T, int VEC, int D>
cudaError_t launch_vec(RotaryParams& p, bool interleaved, cudaStream_t st) {
  // Tokens of a block: as many as leave every SM its blocks kTurns times
  // over, so that the last ones to end hold up little, but where the tokens go
  // round, enough of them for kSteps steps, against the block's fixed cost, and
  // never more than kMaxTokens (32K tokens of 80 heads: 205 us with at most 4,
  // 210 with 8, 217 without the limit; a packed float32 batch of 8 heads: 7.1
  // us with 4 tokens each, 8.1 with 2).
  constexpr int64_t kTurns = 4, kSteps = 20;
  const int64_t steps = (int64_t(p.Hq + p.Hk + p.Hv) * (D / (2 * VEC)) + 31) / 32;
  const int64_t many = p.ntok / (kSms * kRotaryBlocks * kTurns);
  const int64_t enough = std::min((kSteps + steps - 1) / steps, p.ntok / kSms);
  p.tokens = int(std::clamp<int64_t>(std::max(many, enough), 1, kMaxTokens));
  cudaLaunchAttribute attr;  // it may take its place before the launch ahead has ended
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned((p.ntok + p.tokens - 1) / p.tokens));
  cfg.blockDim = dim3(kRotaryThreads);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return interleaved ? cudaLaunchKernelEx(&cfg, k_rotary<T, VEC, true, D>, p)
                     : cudaLaunchKernelEx(&cfg, k_rotary<T, VEC, false, D>, p);
}

// 16-byte packs need every row and both halves of the rotation on 16-byte
// boundaries; anything else (an odd storage offset, rot_dim not a multiple of
// two packs) goes element by element.
template <typename T>
cudaError_t launch_rotary(RotaryParams& p, bool interleaved, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  uintptr_t bits = 0;
  const void* ptrs[] = {p.Q, p.Qo, p.K, p.Ko, p.V, p.Vo};
  for (const void* x : ptrs) bits |= reinterpret_cast<uintptr_t>(x);
  const int64_t strides[] = {p.q_stride, p.qo_stride, p.k_stride, p.v_stride, p.ko_stride};
  for (int64_t x : strides) bits |= uintptr_t(x) * sizeof(T);
  bits |= uintptr_t(p.half) * sizeof(T);
  if (p.d == 128)
    return bits % 16 == 0 ? launch_vec<T, kVec, 128>(p, interleaved, st)
                          : launch_vec<T, 1, 128>(p, interleaved, st);
  return bits % 16 == 0 ? launch_vec<T, kVec, 64>(p, interleaved, st)
                        : launch_vec<T, 1, 64>(p, interleaved, st);
}

mf_status fail(mf_status st, const char* msg) {
  set_last_error(msg);
  return st;
}

mf_status check_rope(const mf_rope_desc* r, int d) {
  if (r->rot_dim < 2 || r->rot_dim % 2 != 0 || r->rot_dim > d)
    return fail(MF_ERR_INVALID_ARG, "rot_dim must be even and in [2, d]");
  if (!r->phases) return fail(MF_ERR_INVALID_ARG, "rope phases are NULL");
  if (!std::isfinite(r->scale)) return fail(MF_ERR_INVALID_ARG, "rope scale not finite");
  return MF_OK;
}

mf_status check_batch(const mf_token_batch* b) {
  if (!b) return fail(MF_ERR_INVALID_ARG, "batch is NULL");
  if (b->ntok < 0 || b->nseq < 0 || (b->nseq == 0 && b->ntok > 0))
    return fail(MF_ERR_INVALID_ARG, "negative token or sequence count, or tokens without sequences");
  if (b->ntok > INT32_MAX) return fail(MF_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
  if (b->cu_seqlens && b->nseq == INT32_MAX)
    return fail(MF_ERR_UNSUPPORTED, "more than 2^31 - 2 sequences");
  if (!b->cu_seqlens && b->ntok != b->nseq)
    return fail(MF_ERR_INVALID_ARG, "without cu_seqlens every sequence has one token");
  return MF_OK;
}

// One set of rows [ntok][H][d] and its output.
mf_status check_rows(const void* in, int64_t stride, const void* out, int64_t out_stride, int H,
                     int d, size_t elem, bool empty) {
  if (H == 0) return MF_OK;
  if ((!in || !out) && !empty) return fail(MF_ERR_INVALID_ARG, "Q, K, V or an output is NULL");
  if (stride < int64_t(H) * d || out_stride < int64_t(H) * d)
    return fail(MF_ERR_INVALID_ARG, "a token stride is below heads * d");
  if (reinterpret_cast<uintptr_t>(in) % elem || reinterpret_cast<uintptr_t>(out) % elem)
    return fail(MF_ERR_INVALID_ARG, "a pointer is not aligned to its element");
  return MF_OK;
}

mf_status launch(RotaryParams& p, mf_dtype dt, bool interleaved, mf_stream_t stream) {
  if (p.ntok == 0) return MF_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dt == MF_BF16 ? launch_rotary<__nv_bfloat16>(p, interleaved, s)
                                      : launch_rotary<float>(p, interleaved, s);
  if (e == cudaSuccess) return MF_OK;
  char msg[160];
  std::snprintf(msg, sizeof msg, "rotary: %s", cudaGetErrorString(e));
  return fail(MF_ERR_CUDA, msg);
}

}  // namespace

mf_status check_kv_cache(const mf_kv_cache* c) {
  if (!c) return fail(MF_ERR_INVALID_ARG, "cache is NULL");
  if (c->dt != MF_BF16 && c->dt != MF_F32) return fail(MF_ERR_INVALID_ARG, "unknown dtype");
  if (c->d != 64 && c->d != 128) return fail(MF_ERR_UNSUPPORTED, "head dim d must be 64 or 128");
  if (c->nseq < 0 || c->Hkv < 1 || c->npages < 0 || c->max_pages_per_seq < 0)
    return fail(MF_ERR_INVALID_ARG, "cache sizes out of range");
  if (c->Hkv > 256) return fail(MF_ERR_UNSUPPORTED, "more than 256 KV heads");
  if (c->page_size < 16 || c->page_size % 16 != 0)
    return fail(MF_ERR_INVALID_ARG, "page_size must be a positive multiple of 16");
  if (c->npages > INT32_MAX / c->page_size || c->max_pages_per_seq > INT32_MAX / c->page_size)
    return fail(MF_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens in the pool or in a sequence");
  if ((c->npages > 0 && (!c->K || !c->V)) ||
      (!c->page_table && c->nseq > 0 && c->max_pages_per_seq > 0))
    return fail(MF_ERR_INVALID_ARG, "a page pool or the page table is NULL");
  if (reinterpret_cast<uintptr_t>(c->K) % 16 || reinterpret_cast<uintptr_t>(c->V) % 16)
    return fail(MF_ERR_INVALID_ARG, "a page pool is not 16-byte aligned");
  return MF_OK;
}

}  // namespace mf

using namespace mf;

extern "C" {

mf_status mf_rope_freqs(int32_t rot_dim, double base, mf_rope_scaling kind, double factor,
                        double original_length, double low, double high, double* inv_freq) {
  if (!inv_freq) return fail(MF_ERR_INVALID_ARG, "inv_freq is NULL");
  if (rot_dim < 2 || rot_dim % 2 != 0) return fail(MF_ERR_INVALID_ARG, "rot_dim must be even and >= 2");
  if (!(base > 0.0) || !std::isfinite(base)) return fail(MF_ERR_INVALID_ARG, "base must be > 0");
  if (kind != MF_ROPE_NONE && kind != MF_ROPE_LINEAR && kind != MF_ROPE_NTK &&
      kind != MF_ROPE_PARTS)
    return fail(MF_ERR_INVALID_ARG, "unknown scaling");
  if (kind != MF_ROPE_NONE && (!(factor > 0.0) || !std::isfinite(factor)))
    return fail(MF_ERR_INVALID_ARG, "factor must be > 0");
  if (kind == MF_ROPE_PARTS && (!(original_length > 0.0) || !std::isfinite(original_length) ||
                                !std::isfinite(low) || !std::isfinite(high) || !(high > low)))
    return fail(MF_ERR_INVALID_ARG, "parts need original_length > 0 and high > low");
  if (kind == MF_ROPE_NTK && rot_dim == 2)
    return fail(MF_ERR_INVALID_ARG, "ntk needs rot_dim > 2");
  const double b = kind == MF_ROPE_NTK ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (kind == MF_ROPE_LINEAR) f /= factor;
    if (kind == MF_ROPE_PARTS) {
      const double turns = original_length * f / (2.0 * M_PI);
      const double g = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f = (1.0 - g) * f / factor + g * f;
    }
    inv_freq[i] = f;
  }
  return MF_OK;
}

mf_status mf_rope_phases(const double* inv_freq, int32_t n, uint64_t* phases) {
  if (n < 0 || (n > 0 && (!inv_freq || !phases)))
    return fail(MF_ERR_INVALID_ARG, "n < 0 or a NULL array");
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(inv_freq[i])) return fail(MF_ERR_INVALID_ARG, "a frequency is not finite");
  for (int i = 0; i < n; ++i) {
    // turns per position modulo 1, to 64 bits (the quotient keeps the 64-bit
    // significand of long double: relative error 2^-64)
    const long double turns = static_cast<long double>(inv_freq[i]) /
                              6.283185307179586476925286766559005768L;
    const long double frac = turns - floorl(turns);
    const long double scaled = rintl(ldexpl(frac, 64));
    phases[i] = scaled >= 18446744073709551616.0L ? 0 : static_cast<uint64_t>(scaled);
  }
  return MF_OK;
}

mf_status mf_rope(const mf_rope_desc* rope, const mf_token_batch* batch, int32_t d, mf_dtype dt,
                  int32_t Hq, const void* Q, int64_t q_stride, void* Q_out, int64_t qo_stride,
                  int32_t Hk, const void* K, int64_t k_stride, void* K_out, int64_t ko_stride,
                  int32_t backward, mf_stream_t stream) {
  if (!rope) return fail(MF_ERR_INVALID_ARG, "rope is NULL");
  if (d != 64 && d != 128) return fail(MF_ERR_UNSUPPORTED, "head dim d must be 64 or 128");
  if (dt != MF_BF16 && dt != MF_F32) return fail(MF_ERR_INVALID_ARG, "unknown dtype");
  mf_status st = check_rope(rope, d);
  if (st != MF_OK) return st;
  st = check_batch(batch);
  if (st != MF_OK) return st;
  if (Hq < 1 || Hk < 0 || Hq > 65536 || Hk > 65536)
    return fail(MF_ERR_INVALID_ARG, "Hq must be positive, Hk not negative");
  const size_t elem = dt == MF_BF16 ? 2 : 4;
  st = check_rows(Q, q_stride, Q_out, qo_stride, Hq, d, elem, batch->ntok == 0);
  if (st != MF_OK) return st;
  st = check_rows(K, k_stride, K_out, ko_stride, Hk, d, elem, batch->ntok == 0);
  if (st != MF_OK) return st;
  RotaryParams p = {};
  p.phases = rope->phases;
  p.scale = rope->scale;
  p.half = rope->rot_dim / 2;
  p.backward = backward != 0;
  p.ntok = batch->ntok;
  p.nseq = batch->nseq;
  p.cu = batch->cu_seqlens;
  p.start = batch->start;
  p.Hq = Hq;
  p.d = d;
  p.Q = Q;
  p.q_stride = q_stride;
  p.Qo = Q_out;
  p.qo_stride = qo_stride;
  if (Hk > 0) {
    p.Hk = Hk;
    p.K = K;
    p.k_stride = k_stride;
    p.Ko = K_out;
    p.ko_stride = ko_stride;
  }
  return launch(p, dt, rope->interleaved != 0, stream);
}

mf_status mf_kv_append(const mf_kv_cache* cache, const mf_rope_desc* rope,
                       const mf_token_batch* batch, const void* K, int64_t k_stride,
                       const void* V, int64_t v_stride, int32_t Hq, const void* Q,
                       int64_t q_stride, void* Q_out, int64_t qo_stride, mf_stream_t stream) {
  mf_status st = check_kv_cache(cache);
  if (st != MF_OK) return st;
  const mf_kv_cache& c = *cache;
  if (rope && (st = check_rope(rope, c.d)) != MF_OK) return st;
  st = check_batch(batch);
  if (st != MF_OK) return st;
  if (batch->nseq != c.nseq)
    return fail(MF_ERR_INVALID_ARG, "the batch's sequences are not the cache's");
  if (Hq < 0 || Hq > 65536) return fail(MF_ERR_INVALID_ARG, "Hq must not be negative");
  const size_t elem = c.dt == MF_BF16 ? 2 : 4;
  const bool empty = batch->ntok == 0;
  const int64_t pool_row = int64_t(c.Hkv) * c.d;
  st = check_rows(K, k_stride, c.K, pool_row, c.Hkv, c.d, elem, empty || c.npages == 0);
  if (st != MF_OK) return st;
  st = check_rows(V, v_stride, c.V, pool_row, c.Hkv, c.d, elem, empty || c.npages == 0);
  if (st != MF_OK) return st;
  st = check_rows(Q, q_stride, Q_out, qo_stride, Hq, c.d, elem, empty);
  if (st != MF_OK) return st;
  if (empty) return MF_OK;
  RotaryParams p = {};
  if (rope) {
    p.phases = rope->phases;
    p.scale = rope->scale;
    p.half = rope->rot_dim / 2;
  }
  p.ntok = batch->ntok;
  p.nseq = batch->nseq;
  p.cu = batch->cu_seqlens;
  p.start = batch->start;
  p.Hk = p.Hv = c.Hkv;
  p.d = c.d;
  p.K = K;
  p.V = V;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.Ko = c.K;
  p.Vo = c.V;
  p.ko_stride = pool_row;
  if (Hq > 0) {
    p.Hq = Hq;
    p.Q = Q;
    p.q_stride = q_stride;
    p.Qo = Q_out;
    p.qo_stride = qo_stride;
  }
  p.paged = true;
  p.page_table = c.page_table;
  p.page_size = c.page_size;
  p.max_pages = c.max_pages_per_seq;
  p.npages = c.npages;
  p.status = status_word();
  if (!p.status) return fail(MF_ERR_CUDA, "no CUDA device");
  return launch(p, c.dt, rope && rope->interleaved != 0, stream);
}

}  // extern "C"
