// Attention of one new token per sequence over a paged key-value cache.
//
// MapFlow article (163.com, "让复用真正省时，还需要解决存储和执行问题"): the
// receiver works with PagedAttention; after a mapped prefill its own tokens
// attend to the keys and values it keeps in pages.
//
//   x_j = scale q.k_j + band_bias [L-1-j < band_width]   (j < L, inside the window)
//   O = sum_j 2^(x_j log2e - m) v_j / l,  m = max, l = sum of the same powers,
//   lse = (m + log2 l) ln 2.
#include <cmath>
#include <cstdio>

#include "mf_sm100.cuh"

namespace mf {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxG = 8;  // query heads of one KV head that one CTA takes
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const void *K, *V, *Q;
  void* O;
  float* lse;
  const int32_t* page_table;
  const int32_t* lens;
  int64_t q_stride, o_stride, npages;
  int nseq, Hq, Hkv, G, page_size, max_pages, len_add, band, window;
  float scale2, bias2;  // times log2 e
  unsigned* status;
};

// One CTA per (sequence, KV head, up to 8 of its query heads); the warps take
// every eighth key and keep their own running maximum and sum, joined at the
// end.
template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) k_paged_attn(const Params p) {
  constexpr int E = D / 32;
  const int s = blockIdx.x, kvh = blockIdx.y, g0 = blockIdx.z * kMaxG;
  const int ng = min(kMaxG, p.G - g0);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __shared__ float sm_m[kWarps][kMaxG], sm_l[kWarps][kMaxG];
  __shared__ float sm_o[kWarps][kMaxG][D];

  const int64_t L = int64_t(p.lens[s]) + p.len_add;
  const int len = int(max(int64_t(0), min(L, int64_t(p.max_pages) * p.page_size)));
  if (L > len && L > 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadPage);
  const int lo = p.window > 0 ? int(max(int64_t(0), L - p.window)) : 0;

  float q[kMaxG][E], o[kMaxG][E] = {}, m[kMaxG], l[kMaxG];
  const int h0 = kvh * p.G + g0;
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    m[g] = -INFINITY;
    l[g] = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e)
      q[g][e] = g < ng ? to_f32(static_cast<const T*>(p.Q)[s * p.q_stride +
                                                         int64_t(h0 + g) * D + e * 32 + lane])
                       : 0.f;
  }
  for (int j = lo + warp; j < len; j += kWarps) {
    const int32_t page = p.page_table[int64_t(s) * p.max_pages + j / p.page_size];
    if (page < 0 || page >= p.npages) {
      if (lane == 0) atomicOr(p.status, kStatusBadPage);
      continue;
    }
    const int64_t row = ((int64_t(page) * p.page_size + j % p.page_size) * p.Hkv + kvh) * D;
    float k[E], v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = to_f32(static_cast<const T*>(p.K)[row + e * 32 + lane]);
      v[e] = to_f32(static_cast<const T*>(p.V)[row + e * 32 + lane]);
    }
    const float bias = L - 1 - j < p.band ? p.bias2 : 0.f;
#pragma unroll
    for (int g = 0; g < kMaxG; ++g) {
      float x = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) x = fmaf(q[g][e], k[e], x);
      x = fmaf(warp_sum(x), p.scale2, bias);
      const float mn = fmaxf(m[g], x);
      // an infinite maximum stays out of the differences
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float c = exp2f(m[g] - ref), w = exp2f(x - ref);
      m[g] = mn;
      l[g] = fmaf(l[g], c, w);
#pragma unroll
      for (int e = 0; e < E; ++e) o[g][e] = fmaf(o[g][e], c, w * v[e]);
    }
  }
#pragma unroll
  for (int g = 0; g < kMaxG; ++g) {
    if (lane == 0) {
      sm_m[warp][g] = m[g];
      sm_l[warp][g] = l[g];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][g][e * 32 + lane] = o[g][e];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < ng * D; i += kWarps * 32) {
    const int g = i / D, dim = i % D;
    float mx = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm_m[w][g]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f, acc = 0.f;
    for (int w = 0; w < kWarps; ++w) {
      const float c = exp2f(sm_m[w][g] - ref);
      sum = fmaf(sm_l[w][g], c, sum);
      acc = fmaf(sm_o[w][g][dim], c, acc);
    }
    static_cast<T*>(p.O)[s * p.o_stride + int64_t(h0 + g) * D + dim] =
        from_f32<T>(sum == 0.f ? 0.f : acc / sum);
    if (dim == 0 && p.lse)
      p.lse[int64_t(h0 + g) * p.nseq + s] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * kLn2;
  }
}

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

}  // namespace
}  // namespace mf

using namespace mf;

extern "C" {

size_t mf_paged_attn_workspace(const mf_kv_cache* cache, const mf_paged_attn_desc* attn) {
  if (check(cache, attn) != MF_OK) return 0;
  return 256;
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
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255) || ws_bytes < mf_paged_attn_workspace(cache, attn))
    return fail(MF_ERR_WORKSPACE, "workspace missing, not 256-byte aligned or too small");
  if (c.nseq == 0) return MF_OK;
  Params p = {};
  p.K = c.K;
  p.V = c.V;
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
  const dim3 grid(c.nseq, c.Hkv, (p.G + kMaxG - 1) / kMaxG);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (c.dt == MF_BF16 && c.d == 128)
    k_paged_attn<__nv_bfloat16, 128><<<grid, kWarps * 32, 0, s>>>(p);
  else if (c.dt == MF_BF16)
    k_paged_attn<__nv_bfloat16, 64><<<grid, kWarps * 32, 0, s>>>(p);
  else if (c.d == 128)
    k_paged_attn<float, 128><<<grid, kWarps * 32, 0, s>>>(p);
  else
    k_paged_attn<float, 64><<<grid, kWarps * 32, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) return MF_OK;
  char msg[160];
  std::snprintf(msg, sizeof msg, "paged attention: %s", cudaGetErrorString(e));
  return fail(MF_ERR_CUDA, msg);
}

}  // extern "C"
