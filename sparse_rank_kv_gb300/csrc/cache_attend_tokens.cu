// Attention of several tokens per sequence over the 8-bit block cache
// (shadowkv_cache_attend_tokens): a piece of a prompt, drafted tokens, or queries
// over an encoder's states.
#include <cmath>
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

struct TokensArgs {
  CacheDev c;
  const void* q;
  void* out;
  float* lse;
  const int32_t* lens;
  long long qb, qh, qs, ob, oh, os;
  float scale_log2;   // scale log2(e)
  int s, h_q, G, causal;
};

__device__ __forceinline__ int tokens_len(const TokensArgs& a, int seq) {
  const int n = a.lens ? a.lens[seq] : a.s;
  if (a.lens && static_cast<unsigned>(n) > static_cast<unsigned>(a.s)) flag_error(a.c.status, DEV_BAD_COUNT);
  return min(max(n, 0), a.s);
}
// Tokens query j of `len` sees of the n held.
__device__ __forceinline__ int tokens_seen(const TokensArgs& a, int n, int len, int j) {
  return a.causal ? max(n - len + j + 1, 0) : n;
}

// CTA = (query, head).
template <typename T, int D>
__global__ void __launch_bounds__(128)
k_attend_tokens(const __grid_constant__ TokensArgs a) {
  __shared__ float sq[D], sp[128], red[8];
  const int tid = threadIdx.x, j = blockIdx.x, h = blockIdx.y, seq = blockIdx.z, pair = seq * a.c.h_kv + h / a.G;
  tc::grid_dep_wait();
  const int len = tokens_len(a, seq), n = cache_tokens(a.c, pair);
  if (j >= len) return;
  const int seen = tokens_seen(a, n, len, j), B = 1 << a.c.shift;
  const T* q = static_cast<const T*>(a.q) + seq * a.qb + h * a.qh + j * a.qs;
  if (tid < D) sq[tid] = Ty<T>::to_f(q[tid]);
  float m = -INFINITY, l = 0.f, acc = 0.f;
  for (int t0 = 0; t0 < seen; t0 += 128) {
    __syncthreads();
    const int t = t0 + tid;
    float x = -INFINITY, vs = 0.f;
    if (t < seen) {
      const int id = cache_block(a.c, pair, t >> a.c.shift), r = t & (B - 1);
      const uint8_t* k = a.c.kc + static_cast<size_t>(id) * B * D + (r / 8) * 8 * D + (r % 8) * 16;
      float z = 0.f;
      for (int e = 0; e < D; e += 2) {
        const float2 f = e4m3_unpack2(*reinterpret_cast<const uint16_t*>(k + (e / 16) * 128 + e % 16));
        z = fmaf(sq[e], f.x, fmaf(sq[e + 1], f.y, z));
      }
      x = z * a.c.ks[id] * a.scale_log2;
      vs = a.c.vs[id];
    }
    float w = warp_max(x);
    if ((tid & 31) == 0) red[tid >> 5] = w;
    __syncthreads();
    const float mn = fmaxf(m, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float ref = mn == -INFINITY ? 0.f : mn, p = exp2f(x - ref), scale = exp2f(m - ref);
    m = mn;
    sp[tid] = t < seen ? p * vs : 0.f;
    w = warp_sum(p);
    if ((tid & 31) == 0) red[4 + (tid >> 5)] = w;
    __syncthreads();
    l = l * scale + (red[4] + red[5] + red[6] + red[7]);
    acc *= scale;
    if (tid < D)
      for (int u = 0; u < min(128, seen - t0); ++u) {
        const int id = cache_block(a.c, pair, (t0 + u) >> a.c.shift), r = (t0 + u) & (B - 1);
        const uint8_t c = a.c.vc[static_cast<size_t>(id) * B * D + (r / 16) * 16 * D + tid * 16 + r % 16];
        acc = fmaf(sp[u], e4m3_unpack2(c).x, acc);
      }
  }
  T* out = static_cast<T*>(a.out) + seq * a.ob + h * a.oh + j * a.os;
  if (tid < D) out[tid] = Ty<T>::from_f(seen > 0 ? acc / l : 0.f);
  if (a.lse && tid == 0)
    a.lse[(static_cast<size_t>(seq) * a.h_q + h) * a.s + j] = seen > 0 ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int D>
static cudaError_t attend_tokens_t(const TokensArgs& a, const shadowkv_cache& c, cudaStream_t st) {
  return launch_pdl(k_attend_tokens<T, D>, dim3(a.s, a.h_q, c.b), dim3(128), 0, st, a);
}

static const char* tokens_fault(const shadowkv_cache& c, int h_q, int s, skv_status* st) {
  *st = SKV_ERR_INVALID_ARG;
  if (s < 0) return "s must be >= 0";
  *st = SKV_ERR_UNSUPPORTED;
  if (h_q < 1 || h_q % c.h_kv || h_q / c.h_kv > 128) return "h_q must be a multiple of h_kv, of at most 128";
  if (static_cast<long long>(s) * (h_q / c.h_kv) > 1 << 24) return "s h_q / h_kv must be at most 2^24";
  *st = SKV_OK;
  return nullptr;
}

static const char* tokens_rows_fault(const shadowkv_rows* r, int b, int h, int s, uintptr_t E, bool written) {
  if (!r || !r->ptr) return "q and out must be non-NULL";
  const long long sb = b > 1 ? r->sb : 1, sh = h > 1 ? r->sh : 1, ss = s > 1 ? r->ss : 1;
  if (sb < 0 || sh < 0 || ss < 0) return "row strides must not be negative";
  if (written && (!sb || !sh || !ss)) return "an output stride is 0";
  if (reinterpret_cast<uintptr_t>(r->ptr) % E) return "q and out must be aligned to their elements";
  return nullptr;
}

}  // namespace skv

extern "C" {

size_t shadowkv_cache_attend_tokens_workspace(const shadowkv_cache* c, int h_q, int s) try {
  if (skv::cache_checked(c) != SKV_OK) return 0;
  skv_status st;
  if (const char* f = skv::tokens_fault(*c, h_q, s, &st)) {
    skv::set_error(st, f);
    return 0;
  }
  return 256;
} catch (...) {   // host memory for an error text or a table ran out
  return 0;
}

skv_status shadowkv_cache_attend_tokens(const shadowkv_cache* c, int dtype, int h_q, int s, const shadowkv_rows* q,
                                        const int32_t* lens, int causal, float scale, const shadowkv_rows* out, float* lse,
                                        void* work, size_t work_bytes, void* stream) try {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (dtype != SKV_DTYPE_F32 && dtype != SKV_DTYPE_BF16) return set_error(SKV_ERR_INVALID_ARG, "bad dtype");
  if (const char* f = skv::tokens_fault(*c, h_q, s, &st)) return set_error(st, f);
  if (s == 0) return SKV_OK;
  const uintptr_t E = dtype == SKV_DTYPE_BF16 ? 2 : 4;
  const char* f = skv::tokens_rows_fault(q, c->b, h_q, s, E, false);
  if (!f) f = skv::tokens_rows_fault(out, c->b, h_q, s, E, true);
  if (!f && (reinterpret_cast<uintptr_t>(lens) % 4 || reinterpret_cast<uintptr_t>(lse) % 4))
    f = "lens and lse must be 4-byte aligned";
  if (!f && !std::isfinite(scale)) f = "scale must be finite";
  if (!f && causal != 0 && causal != 1) f = "causal must be 0 or 1";
  if (!f && (!work || reinterpret_cast<uintptr_t>(work) % 256)) f = "the workspace must be non-NULL and 256-byte aligned";
  if (!f && work_bytes < 256) f = "the workspace is smaller than shadowkv_cache_attend_tokens_workspace";
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  skv::TokensArgs a;
  a.c = skv::cache_dev(*c);
  a.q = q->ptr;
  a.out = out->ptr;
  a.lse = lse;
  a.lens = lens;
  // the stride of an extent of 1 is not used
  a.qb = c->b > 1 ? q->sb : 0; a.qh = h_q > 1 ? q->sh : 0; a.qs = s > 1 ? q->ss : 0;
  a.ob = c->b > 1 ? out->sb : 0; a.oh = h_q > 1 ? out->sh : 0; a.os = s > 1 ? out->ss : 0;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.s = s;
  a.h_q = h_q;
  a.G = h_q / c->h_kv;
  a.causal = causal;
  cudaStream_t p = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  cudaError_t e;
  if (dtype == SKV_DTYPE_BF16)
    e = c->d == 128 ? skv::attend_tokens_t<skv::bf16, 128>(a, *c, p) : skv::attend_tokens_t<skv::bf16, 64>(a, *c, p);
  else
    e = c->d == 128 ? skv::attend_tokens_t<float, 128>(a, *c, p) : skv::attend_tokens_t<float, 64>(a, *c, p);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
