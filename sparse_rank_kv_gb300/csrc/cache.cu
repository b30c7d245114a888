// The 8-bit block cache (include/shadowkv.h): its checks, the append that
// quantises new tokens into it, and the eviction of whole blocks by gathered
// attention weight.
#include <cfloat>
#include <cstdint>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

// ------------------------------------------------------------------ append
constexpr int kApThreads = 256;

struct AppendArgs {
  CacheDev c;
  const void *k, *v;
  long long kb, kh, ks, vb, vh, vs;   // strides of k and v: sequence, head, token
  const int32_t* lens;
  int s;
};

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= FLT_MAX ? a : 0.f;   // infinities and NaN do not count
}

// x / s: by the reciprocal where s is a power of two (then the exact
// quotient), else (a partly filled block the caller made with a scale of its
// own) by division.
__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0u; }
__device__ __forceinline__ float quotient(float x, float s, float inv, bool pow2) { return pow2 ? x * inv : x / s; }

// The tokens a pair's append covers: [n0, end) of the pair.
__device__ __forceinline__ void append_range(const AppendArgs& a, int pair, int* n0, int* end) {
  const int n = cache_tokens(a.c, pair);
  int cnt = a.s;
  if (a.lens) {
    cnt = a.lens[pair / a.c.h_kv];
    if (cnt < 0 || cnt > a.s) {
      flag_error(a.c.status, DEV_BAD_COUNT);
      cnt = cnt < 0 ? 0 : a.s;
    }
  }
  const int cap = a.c.max_blocks << a.c.shift;
  if (cnt > cap - n) {
    flag_error(a.c.status, DEV_BAD_COUNT);
    cnt = cap - n;
  }
  *n0 = n;
  *end = n + cnt;
}

// Quantises the new tokens [n0, end) that fall into the pair's block blk, for
// K (which = 0) or V (1).  Two passes over the tokens' rows: the largest
// magnitude, then the codes (the second pass hits L1).
template <typename T, int D>
__device__ __forceinline__ void append_block(const AppendArgs& a, int pair, int blk, int n0, int end, int which,
                                             float* red) {
  constexpr int VE = 16 / sizeof(T);        // elements per 16-byte load
  const CacheDev& c = a.c;
  const int B = 1 << c.shift, tid = threadIdx.x;
  const int b0 = blk << c.shift;
  const int e0 = max(n0 - b0, 0), e1 = min(end - b0, B);   // new rows of the block
  if (e0 >= e1) return;
  const int id = cache_block(c, pair, blk);
  const int seq = pair / c.h_kv, head = pair - seq * c.h_kv;
  const T* src = which ? static_cast<const T*>(a.v) + seq * a.vb + head * a.vh
                       : static_cast<const T*>(a.k) + seq * a.kb + head * a.kh;
  const long long ss = which ? a.vs : a.ks;
  src += (static_cast<long long>(b0) + e0 - n0) * ss;       // row e0 of the block
  uint8_t* dst = (which ? c.vc : c.kc) + static_cast<size_t>(id) * (D << c.shift);
  float* scale = (which ? c.vs : c.ks) + id;

  float m = 0.f;
  for (int u = tid; u < (e1 - e0) * (D / VE); u += kApThreads) {
    const int r = u / (D / VE), p = u % (D / VE);
    float x[VE];
    Ty<T>::load16(src + r * ss + p * VE, x);
#pragma unroll
    for (int e = 0; e < VE; ++e) m = fmaxf(m, finite_abs(x[e]));
  }
  m = warp_max(m);
  __syncthreads();
  if ((tid & 31) == 0) red[tid >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kApThreads / 32; ++w) m = fmaxf(m, red[w]);
  const float fresh = cache_scale_of(m);
  const float was = e0 > 0 ? *scale : 0.f;
  const float sc = fmaxf(fresh, was);
  const bool grow = e0 > 0 && sc > was;
  const float ratio = e0 > 0 ? was / sc : 1.f;
  const float inv = 1.f / sc;
  const bool pow2 = is_pow2(sc);
  auto dv = [&](float x) { return quotient(x, sc, inv, pow2); };
  auto rescale2 = [&](uint32_t c2) {
    const float2 f = e4m3_unpack2(c2);
    return e4m3_pack2(f.x * ratio, f.y * ratio);
  };

  if (which == 0) {
    // K: unit = 16 dimensions of a row (16 bytes); 8 consecutive threads take
    // 8 rows, whose units are adjacent in the block
    const int r0 = grow ? 0 : e0 & ~7;
    for (int u = tid; u < (((e1 + 7) & ~7) - r0) * (D / 16); u += kApThreads) {
      const int r = r0 + ((u / (8 * (D / 16))) << 3) + (u & 7), p = (u >> 3) % (D / 16);
      if (r >= e1 || (r < e0 && !grow)) continue;
      uint4* w = reinterpret_cast<uint4*>(dst + (r >> 3) * (8 * D) + p * 128 + (r & 7) * 16);
      uint32_t o[4];
      if (r < e0) {
        const uint4 old = *w;
        const uint32_t in[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = rescale2(in[e]) | (rescale2(in[e] >> 16) << 16);
      } else {
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; e += VE) Ty<T>::load16(src + (r - e0) * ss + p * 16 + e, x + e);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = e4m3_pack2(dv(x[4 * e]), dv(x[4 * e + 1])) | (e4m3_pack2(dv(x[4 * e + 2]), dv(x[4 * e + 3])) << 16);
      }
      *w = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
    // V: unit = 16 tokens of two dimensions (32 bytes); bytes of tokens
    // that are neither held nor new stay as they are
    const int g0 = grow ? 0 : e0 >> 4, g1 = (e1 + 15) >> 4;
    for (int u = tid; u < (g1 - g0) * (D / 2); u += kApThreads) {
      const int t0 = (g0 + u / (D / 2)) << 4, j = (u % (D / 2)) * 2;
      uint4* w = reinterpret_cast<uint4*>(dst + (t0 >> 4) * (16 * D) + j * 16);
      uint32_t o[2][4] = {};
      if (t0 < e0 || t0 + 16 > e1) {
        const uint4 a0 = w[0], a1 = w[1];
        o[0][0] = a0.x; o[0][1] = a0.y; o[0][2] = a0.z; o[0][3] = a0.w;
        o[1][0] = a1.x; o[1][1] = a1.y; o[1][2] = a1.z; o[1][3] = a1.w;
      }
#pragma unroll
      for (int t = 0; t < 16; ++t) {
        const int r = t0 + t, sh = (t & 3) * 8;
        uint32_t c2;
        if (r >= e0 && r < e1) {
          const T* p = src + (r - e0) * ss + j;
          c2 = e4m3_pack2(dv(Ty<T>::to_f(p[0])), dv(Ty<T>::to_f(p[1])));
        } else if (r < e0 && grow) {
          c2 = rescale2(((o[0][t >> 2] >> sh) & 0xffu) | (((o[1][t >> 2] >> sh) & 0xffu) << 8));
        } else {
          continue;
        }
        o[0][t >> 2] = (o[0][t >> 2] & ~(0xffu << sh)) | ((c2 & 0xffu) << sh);
        o[1][t >> 2] = (o[1][t >> 2] & ~(0xffu << sh)) | ((c2 >> 8) << sh);
      }
      w[0] = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
      w[1] = make_uint4(o[1][0], o[1][1], o[1][2], o[1][3]);
    }
  }
  __syncthreads();   // every thread has read the old scale
  if (tid == 0) {
    *scale = sc;
    if (which == 0 && e0 == 0 && c.weight) c.weight[static_cast<size_t>(pair) * c.max_blocks + blk] = 0.f;
  }
}

// Few new tokens (s <= block): one CTA per pair covers the at most two
// blocks they touch and moves the pair's count.
template <typename T, int D>
__global__ void __launch_bounds__(kApThreads) k_append_few(const __grid_constant__ AppendArgs a) {
  __shared__ float red[kApThreads / 32];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int pair = blockIdx.x;
  int n0, end;
  append_range(a, pair, &n0, &end);
  for (int blk = n0 >> a.c.shift; blk << a.c.shift < end; ++blk)
    for (int which = 0; which < 2; ++which) append_block<T, D>(a, pair, blk, n0, end, which, red);
  __syncthreads();
  if (threadIdx.x == 0) a.c.n_tok[pair] = end;
}

// Many: CTA (block, pair) for K and V; k_append_count moves the counts after.
template <typename T, int D>
__global__ void __launch_bounds__(kApThreads) k_append_many(const __grid_constant__ AppendArgs a, int nblk) {
  __shared__ float red[kApThreads / 32];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int pair = blockIdx.x / nblk, bi = blockIdx.x - pair * nblk;
  int n0, end;
  append_range(a, pair, &n0, &end);
  append_block<T, D>(a, pair, (n0 >> a.c.shift) + bi, n0, end, blockIdx.y, red);
}

__global__ void __launch_bounds__(kApThreads) k_append_count(const __grid_constant__ AppendArgs a) {
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int pair = blockIdx.x * kApThreads + threadIdx.x;
  if (pair >= a.c.pairs) return;
  int n0, end;
  append_range(a, pair, &n0, &end);
  a.c.n_tok[pair] = end;
}

template <typename T, int D>
static cudaError_t append_t(const AppendArgs& a, cudaStream_t st) {
  const int B = 1 << a.c.shift;
  if (a.s <= B)
    return launch_pdl(k_append_few<T, D>, dim3(a.c.pairs), dim3(kApThreads), 0, st, a);
  const long long touched = (static_cast<long long>(a.s) + B - 1) / B + 1;
  const int nblk = static_cast<int>(touched < a.c.max_blocks ? touched : a.c.max_blocks);
  cudaError_t e = launch_pdl(k_append_many<T, D>, dim3(static_cast<unsigned>(a.c.pairs) * nblk, 2), dim3(kApThreads), 0, st,
                             a, nblk);
  if (e == cudaSuccess)
    e = launch_pdl(k_append_count, dim3((a.c.pairs + kApThreads - 1) / kApThreads), dim3(kApThreads), 0, st, a);
  return e;
}

// ------------------------------------------------------------------ evict
constexpr int kEvThreads = 512;
constexpr int kEvMax = 16384;   // blocks per pair
constexpr int kEvRegs = kEvMax / kEvThreads;

static size_t evict_smem(int mb) {
  const size_t nw = (mb + 31) / 32;
  return 4 * (2 * static_cast<size_t>(mb) + 2 * nw + topk_scratch_ints(kEvThreads));
}

// CTA = pair.  The blocks' weights become order-preserving keys (protected
// blocks the largest), block_topk marks the `keep` largest, and a block's new
// place follows from the marked blocks before it.  Entries pass through
// registers, so that the tables may be rewritten in place.
__global__ void __launch_bounds__(kEvThreads)
k_evict(const __grid_constant__ CacheDev c, int32_t* table, int32_t* n_tok, float* weight, int32_t* kept, int keep,
        int sink, int recent) {
  extern __shared__ __align__(16) unsigned char smem[];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int mb = c.max_blocks, nw_max = (mb + 31) >> 5, tid = threadIdx.x;
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem);   // [mb]
  int* order = reinterpret_cast<int*>(keys + mb);       // [mb] old index of every new place
  uint32_t* bits = reinterpret_cast<uint32_t*>(order + mb);
  int* wpref = reinterpret_cast<int*>(bits + nw_max);
  int* scratch = wpref + nw_max;
  const int pair = blockIdx.x;
  const size_t row = static_cast<size_t>(pair) * mb;
  const int tok = cache_tokens(c, pair);
  const int B = 1 << c.shift, n = (tok + B - 1) >> c.shift;
  const bool over = n > keep;
  const int nk = over ? keep : n;
  if (over) {
    for (int i = tid; i < n; i += kEvThreads) {
      const float w = c.weight[row + i];
      keys[i] = i < sink || i >= n - recent ? 0xffffffffu : w == w ? order_key(w + 0.f) : 1u;   // -0 as 0, NaN last
    }
    __syncthreads();
    block_topk(keys, n, keep, order, scratch, bits, wpref);   // order[0, keep): the kept, ascending
    for (int i = tid; i < n; i += kEvThreads) {
      const uint32_t b = bits[i >> 5], bit = 1u << (i & 31);
      if (!(b & bit)) order[keep + i - wpref[i >> 5] - __popc(b & (bit - 1u))] = i;
    }
    for (int i = n + tid; i < mb; i += kEvThreads) order[i] = i;
    __syncthreads();
  } else {
    for (int i = tid; i < mb; i += kEvThreads) order[i] = i;
    __syncthreads();
  }
  int32_t id[kEvRegs];
  float wt[kEvRegs];
#pragma unroll
  for (int r = 0; r < kEvRegs; ++r) {
    const int i = tid + r * kEvThreads;
    if (i < mb) {
      id[r] = c.table[row + order[i]];
      wt[r] = i < nk ? c.weight[row + order[i]] : 0.f;
    }
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kEvRegs; ++r) {
    const int i = tid + r * kEvThreads;
    if (i < mb) {
      table[row + i] = id[r];
      weight[row + i] = wt[r];
    }
  }
  if (kept)
    for (int i = tid; i < keep; i += kEvThreads) kept[static_cast<size_t>(pair) * keep + i] = i < nk ? order[i] : -1;
  if (tid == 0) {
    const bool last = nk > 0 && order[nk - 1] == n - 1;   // the newest block is still held
    n_tok[pair] = last ? (nk - 1) * B + tok - (n - 1) * B : nk * B;
  }
}

}  // namespace skv

// ------------------------------------------------------------------ C ABI
namespace {

const char* cache_fault(const shadowkv_cache* c, skv_status* st) {
  *st = SKV_ERR_INVALID_ARG;
  if (!c) return "cache is NULL";
  if (c->b < 1 || c->h_kv < 1) return "cache: b and h_kv must be >= 1";
  if (c->max_blocks < 1 || c->n_pool < 1) return "cache: max_blocks and n_pool must be >= 1";
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->table || !c->n_tok || !c->status)
    return "cache: a required pointer is NULL";
  if (reinterpret_cast<uintptr_t>(c->k_codes) % 16 || reinterpret_cast<uintptr_t>(c->v_codes) % 16)
    return "cache: codes must be 16-byte aligned";
  const uintptr_t words = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale) |
                          reinterpret_cast<uintptr_t>(c->table) | reinterpret_cast<uintptr_t>(c->n_tok) |
                          reinterpret_cast<uintptr_t>(c->weight) | reinterpret_cast<uintptr_t>(c->status);
  if (words % 4) return "cache: scales, table, counts, weights and status must be 4-byte aligned";
  *st = SKV_ERR_UNSUPPORTED;
  if (c->d != 64 && c->d != 128) return "cache: d must be 64 or 128";
  if (c->block != 16 && c->block != 32 && c->block != 64 && c->block != 128)
    return "cache: block must be 16, 32, 64 or 128";
  if (c->max_blocks > skv::kEvMax) return "cache: max_blocks must be <= 16384";
  if (static_cast<long long>(c->b) * c->h_kv * c->max_blocks >= (1LL << 31))
    return "cache: b * h_kv * max_blocks must be < 2^31";
  *st = SKV_OK;
  return nullptr;
}

// Rows read 16 bytes at a time.
const char* rows16_fault(const shadowkv_rows* r, int E) {
  if (!r || !r->ptr) return "k and v must be non-NULL";
  if (r->sb < 0 || r->sh < 0 || r->ss < 0) return "row strides must not be negative";
  if (reinterpret_cast<uintptr_t>(r->ptr) % 16 || (r->sb * E) % 16 || (r->sh * E) % 16 || (r->ss * E) % 16)
    return "row pointers and strides must be multiples of 16 bytes";
  return nullptr;
}

}  // namespace

namespace skv {
skv_status cache_checked(const shadowkv_cache* c) {
  skv_status st;
  const char* f = cache_fault(c, &st);
  return f ? set_error(st, f) : SKV_OK;
}
}  // namespace skv

extern "C" {

skv_status shadowkv_cache_validate(const shadowkv_cache* c) { return skv::cache_checked(c); }

skv_status shadowkv_cache_append(const shadowkv_cache* c, int dtype, const shadowkv_rows* k, const shadowkv_rows* v,
                                 int s, const int32_t* lens, void* stream) {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (dtype != SKV_DTYPE_F32 && dtype != SKV_DTYPE_BF16) return set_error(SKV_ERR_INVALID_ARG, "bad dtype");
  if (s < 0) return set_error(SKV_ERR_INVALID_ARG, "s must be >= 0");
  const int E = dtype == SKV_DTYPE_BF16 ? 2 : 4;
  const char* f = rows16_fault(k, E);
  if (!f) f = rows16_fault(v, E);
  if (!f && reinterpret_cast<uintptr_t>(lens) % 4) f = "lens must be 4-byte aligned";
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  if (s == 0) return SKV_OK;
  skv::AppendArgs a;
  a.c = skv::cache_dev(*c);
  a.k = k->ptr; a.kb = k->sb; a.kh = k->sh; a.ks = k->ss;
  a.v = v->ptr; a.vb = v->sb; a.vh = v->sh; a.vs = v->ss;
  a.lens = lens;
  a.s = s;
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == SKV_DTYPE_BF16)
    e = c->d == 128 ? skv::append_t<skv::bf16, 128>(a, q) : skv::append_t<skv::bf16, 64>(a, q);
  else
    e = c->d == 128 ? skv::append_t<float, 128>(a, q) : skv::append_t<float, 64>(a, q);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
}

skv_status shadowkv_cache_evict(const shadowkv_cache* src, const shadowkv_cache* dst, int keep, int sink, int recent,
                                int32_t* kept, void* stream) {
  using skv::set_error;
  skv_status st = skv::cache_checked(src);
  if (st != SKV_OK) return st;
  if (!dst) dst = src;
  st = skv::cache_checked(dst);
  if (st != SKV_OK) return st;
  if (dst->b != src->b || dst->h_kv != src->h_kv || dst->max_blocks != src->max_blocks || dst->block != src->block)
    return set_error(SKV_ERR_INVALID_ARG, "dst and src differ in b, h_kv, max_blocks or block");
  if (!src->weight || !dst->weight) return set_error(SKV_ERR_INVALID_ARG, "the cache keeps no weights");
  if (keep < 1 || keep > src->max_blocks) return set_error(SKV_ERR_INVALID_ARG, "need 1 <= keep <= max_blocks");
  if (sink < 0 || recent < 0 || sink > keep || recent > keep - sink)
    return set_error(SKV_ERR_INVALID_ARG, "need sink, recent >= 0 and sink + recent <= keep");
  if (reinterpret_cast<uintptr_t>(kept) % 4) return set_error(SKV_ERR_INVALID_ARG, "kept must be 4-byte aligned");
  const size_t smem = skv::evict_smem(src->max_blocks);
  cudaError_t e = skv::set_smem_once(reinterpret_cast<const void*>(skv::k_evict), static_cast<int>(smem));
  if (e == cudaSuccess)
    e = skv::launch_pdl(skv::k_evict, dim3(src->b * src->h_kv), dim3(skv::kEvThreads), smem,
                        static_cast<cudaStream_t>(stream), skv::cache_dev(*src), dst->table, dst->n_tok, dst->weight,
                        kept, keep, sink, recent);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
}

skv_status shadowkv_cache_check(const shadowkv_cache* c) {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  int word = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&word, c->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  if (word == skv::DEV_TIMEOUT) return set_error(SKV_ERR_TIMEOUT, "a bounded device wait gave up");
  if (word) return set_error(SKV_ERR_DEVICE_CHECK, "a kernel met a block id, length or token count out of range");
  return SKV_OK;
}

}  // extern "C"
