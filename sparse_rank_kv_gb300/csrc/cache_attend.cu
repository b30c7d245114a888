// Attention of one token per sequence over the 8-bit block cache
// (shadowkv_cache_attend): out = softmax(scale q K^T) V per query head, the
// log of each head's sum, and the weight every block receives.
//
// Every pair's tokens are cut into 128-token tiles; the tiles of all pairs, in
// order, are dealt evenly to the CTAs (consecutive tiles to a CTA), so that
// ragged lengths and few long sequences both fill the GPU.  A CTA leaves one
// partial (max, sum, sum p v) per pair it meets, and k_attend_merge joins a
// pair's partials in order and turns the tiles' sums of p into block weights.
// Lengths are only known on the device: every CTA forms the prefix of the tile counts itself.
#include <cmath>
#include <cstdint>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

constexpr int kCaT = 128;         // tokens per tile

// Workspace, in order: per pair the index of its first tile, the total tile
// count, the CTAs' partials, and for the weights every tile's reference
// maximum and the sums of p over granules of min(block, 32) tokens.
struct AttendWork {
  int* first;      // [pairs] then the total
  float* part;     // [ctas + pairs][G][d + 2]
  float* tmax;     // [pairs][tiles][G]
  float* psum;     // [pairs][granules][G]
  int tiles, granules;   // per pair, at most
};

inline int attend_ctas(const shadowkv_cache& c, int nsm) {
  const long long tiles = (static_cast<long long>(c.max_blocks) * c.block + kCaT - 1) / kCaT * c.b * c.h_kv;
  return static_cast<int>(tiles < 2LL * nsm ? tiles : 2LL * nsm);
}

inline size_t attend_layout(const shadowkv_cache& c, int G, int nsm, void* base, AttendWork* w) {
  const size_t pairs = static_cast<size_t>(c.b) * c.h_kv;
  const long long tok = static_cast<long long>(c.max_blocks) * c.block;
  const int gran = c.block < 32 ? c.block : 32;
  AttendWork v;
  v.tiles = static_cast<int>((tok + kCaT - 1) / kCaT);
  v.granules = v.tiles * (kCaT / gran);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = static_cast<char*>(base) + off;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  v.first = reinterpret_cast<int*>(take((pairs + 1) * sizeof(int)));
  v.part = reinterpret_cast<float*>(take((attend_ctas(c, nsm) + pairs) * G * (c.d + 2) * sizeof(float)));
  v.tmax = reinterpret_cast<float*>(take(pairs * v.tiles * G * sizeof(float)));
  v.psum = reinterpret_cast<float*>(take(pairs * v.granules * G * sizeof(float)));
  if (w) *w = v;
  return off;
}

struct AttendArgs {
  CacheDev c;
  AttendWork w;
  const void* q;
  void* out;
  float* lse;
  long long qb, qh, ob, oh;
  float scale_log2;   // scale log2(e)
  float decay;
  int gather;
};

__device__ __forceinline__ int tiles_of(const CacheDev& c, int pair) {
  return (cache_tokens(c, pair) + kCaT - 1) / kCaT;
}

// A CTA's share [t0, t1) of the T tiles when n CTAs take part (n <= T).
__device__ __forceinline__ int share_begin(int cta, int n, int T) {
  return static_cast<int>(static_cast<long long>(cta) * T / n);
}
// The CTA whose share holds tile x.
__device__ __forceinline__ int share_owner(int x, int n, int T) {
  return static_cast<int>(((static_cast<long long>(x) + 1) * n - 1) / T);
}

// Total of the tile counts, and the pair and tile at which this CTA's share
// begins (s_where = {pair, tile in the pair, total}).  Every thread calls it.
// The CTA that holds a pair's first tile also writes the pair's first tile
// index for the merge (share_note).
template <int NT>
__device__ __forceinline__ void share_find(const AttendArgs& a, int cta, int ncta, int* s_where, int* s_scan) {
  const int tid = threadIdx.x, P = a.c.pairs;
  const int per = (P + NT - 1) / NT;
  const int p0 = min(P, tid * per), p1 = min(P, p0 + per);
  int sum = 0;
  for (int p = p0; p < p1; ++p) sum += tiles_of(a.c, p);
  int T;
  int before = block_exclusive_scan(sum, s_scan, &T);
  if (tid == 0) s_where[2] = T;
  if (cta == 0 && tid == 0) a.w.first[P] = T;
  const int n = min(ncta, T);
  if (cta < n && sum > 0) {
    const int t0 = share_begin(cta, n, T);
    if (before <= t0 && t0 < before + sum) {
      int p = p0, b = before;
      for (;; ++p) {
        const int k = tiles_of(a.c, p);
        if (t0 < b + k) break;
        b += k;
      }
      s_where[0] = p;
      s_where[1] = t0 - b;
    }
  }
  __syncthreads();
}

// ------------------------------------------------------------ CUDA cores
template <typename T, int D, int G>
__global__ void __launch_bounds__(kCaT) k_attend(const __grid_constant__ AttendArgs a) {
  __shared__ int s_where[3], s_scan[32];
  __shared__ float sq[G][D], sp[G][kCaT], red[4][G];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int cta = blockIdx.x;
  share_find<kCaT>(a, cta, gridDim.x, s_where, s_scan);
  const int total = s_where[2], n = min(static_cast<int>(gridDim.x), total);
  if (cta >= n) return;
  const int t0 = share_begin(cta, n, total), t1 = share_begin(cta + 1, n, total);
  const int gran = min(1 << a.c.shift, 32);
  int pair = s_where[0], tile = s_where[1], left = t1 - t0, at = t0;
  while (left > 0) {
    const int ntok = cache_tokens(a.c, pair), nt = (ntok + kCaT - 1) / kCaT;
    if (tile >= nt) {   // the next pair (one without tokens has no tile)
      if (pair + 1 >= a.c.pairs) break;
      ++pair;
      tile = 0;
      continue;
    }
    if (tile == 0 && tid == 0) a.w.first[pair] = at;
    const int seq = pair / a.c.h_kv, head = pair - seq * a.c.h_kv;
    __syncthreads();
    for (int i = tid; i < G * D; i += kCaT) {
      const int g = i / D, j = i - g * D;
      sq[g][j] = Ty<T>::to_f(static_cast<const T*>(a.q)[seq * a.qb + (static_cast<long long>(head) * G + g) * a.qh + j]);
    }
    __syncthreads();
    const int end = min(nt, tile + left);
    float m[G], l[G], acc[G];
#pragma unroll
    for (int g = 0; g < G; ++g) { m[g] = -INFINITY; l[g] = 0.f; acc[g] = 0.f; }
    for (int t = tile; t < end; ++t) {
      const int tok0 = t * kCaT, cnt = min(kCaT, ntok - tok0);
      float s[G];
      const int tok = tok0 + tid;
      if (tid < cnt) {
        const int id = cache_block(a.c, pair, tok >> a.c.shift), r = tok & ((1 << a.c.shift) - 1);
        const uint8_t* row = a.c.kc + static_cast<size_t>(id) * (D << a.c.shift) + (r >> 3) * (8 * D) + (r & 7) * 16;
#pragma unroll
        for (int g = 0; g < G; ++g) s[g] = 0.f;
        for (int p = 0; p < D / 16; ++p) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + p * 128);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 f = e4m3_unpack2(w[e >> 1] >> (16 * (e & 1)));
#pragma unroll
            for (int g = 0; g < G; ++g)
              s[g] = fmaf(f.x, sq[g][p * 16 + 2 * e], fmaf(f.y, sq[g][p * 16 + 2 * e + 1], s[g]));
          }
        }
        const float ks = a.c.ks[id] * a.scale_log2;
#pragma unroll
        for (int g = 0; g < G; ++g) s[g] *= ks;
      } else {
#pragma unroll
        for (int g = 0; g < G; ++g) s[g] = -INFINITY;
      }
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float x = warp_max(s[g]);
        if (lane == 0) red[warp][g] = x;
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float mn = fmaxf(fmaxf(fmaxf(red[0][g], red[1][g]), fmaxf(red[2][g], red[3][g])), m[g]);
        const float ref = mn == -INFINITY ? 0.f : mn;
        const float al = exp2f(m[g] - ref);
        m[g] = mn;
        const float p = exp2f(s[g] - ref);
        l[g] = l[g] * al + p;
        acc[g] *= al;
        sp[g][tid] = p;
        if (a.gather) {
          float z = p;
          for (int o = 1; o < gran; o <<= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
          if ((tid & (gran - 1)) == 0)
            a.w.psum[(static_cast<size_t>(pair) * a.w.granules + (tok0 + tid) / gran) * G + g] = z;
          if (tid == 0) a.w.tmax[(static_cast<size_t>(pair) * a.w.tiles + t) * G + g] = ref;
        }
      }
      __syncthreads();
      if (tid < D) {
        for (int u = 0; u < cnt; ++u) {
          const int tk = tok0 + u, id = cache_block(a.c, pair, tk >> a.c.shift), r = tk & ((1 << a.c.shift) - 1);
          const uint8_t c8 = a.c.vc[static_cast<size_t>(id) * (D << a.c.shift) + (r >> 4) * (16 * D) + tid * 16 + (r & 15)];
          const float v = e4m3_unpack2(c8).x * a.c.vs[id];
#pragma unroll
          for (int g = 0; g < G; ++g) acc[g] = fmaf(sp[g][u], v, acc[g]);
        }
      }
      __syncthreads();
    }
    // the partial of (this CTA, pair)
    float* part = a.w.part + static_cast<size_t>(cta + pair) * G * (D + 2);
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float z = warp_sum(l[g]);
      if (lane == 0) red[warp][g] = z;
      if (tid < D) part[g * (D + 2) + tid] = acc[g];
    }
    __syncthreads();
    if (tid == 0)
#pragma unroll
      for (int g = 0; g < G; ++g) {
        part[g * (D + 2) + D] = m[g];
        part[g * (D + 2) + D + 1] = red[0][g] + red[1][g] + red[2][g] + red[3][g];
      }
    at += end - tile;
    left -= end - tile;
    tile = end;
  }
}

// ------------------------------------------------------------ merge
constexpr int kCmThreads = 256;

// Blocks 0 .. pairs G - 1: the output of a query head.  The others, with
// weights: `chunk` cache blocks of a pair.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kCmThreads)
k_attend_merge(const __grid_constant__ AttendArgs a, int ncta, int chunk, int nchunk) {
  __shared__ float s_M[G], s_L[G], s_acc[kCmThreads / D][D];
  const int tid = threadIdx.x;
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int P = a.c.pairs, bx = blockIdx.x;
  const bool head_role = bx < P * G;
  const int pair = head_role ? bx / G : (bx - P * G) / nchunk;
  const int ntok = cache_tokens(a.c, pair), nt = (ntok + kCaT - 1) / kCaT;
  const int seq = pair / a.c.h_kv, kvh = pair - seq * a.c.h_kv;
  if (nt == 0) {
    if (head_role) {
      const int h = kvh * G + bx % G;
      if (tid < D) static_cast<T*>(a.out)[seq * a.ob + h * a.oh + tid] = Ty<T>::from_f(0.f);
      if (a.lse && tid == 0) a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h] = -INFINITY;
    }
    return;
  }
  const int T_all = a.w.first[P], n = min(ncta, T_all), f = a.w.first[pair];
  const int c0 = share_owner(f, n, T_all), c1 = share_owner(f + nt - 1, n, T_all);
  // the heads' largest maximum and total sum over the pair's partials
  if (tid < 32 * G && tid / 32 < G) {
    const int g = tid / 32, lane = tid & 31;
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
      M = fmaxf(M, a.w.part[(static_cast<size_t>(c + pair) * G + g) * (D + 2) + D]);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float* p = a.w.part + (static_cast<size_t>(c + pair) * G + g) * (D + 2) + D;
      L = fmaf(p[1], exp2f(p[0] - ref), L);
    }
    L = warp_sum(L);
    if (lane == 0) { s_M[g] = ref; s_L[g] = L; }
  }
  __syncthreads();
  if (head_role) {
    const int g = bx % G, j = tid % D, sl = tid / D;
    float acc = 0.f;
    for (int c = c0 + sl; c <= c1; c += kCmThreads / D) {
      const float* p = a.w.part + (static_cast<size_t>(c + pair) * G + g) * (D + 2);
      acc = fmaf(p[j], exp2f(p[D] - s_M[g]), acc);
    }
    s_acc[sl][j] = acc;
    __syncthreads();
    if (sl == 0) {
      for (int u = 1; u < kCmThreads / D; ++u) acc += s_acc[u][j];
      const int h = kvh * G + g;
      static_cast<T*>(a.out)[seq * a.ob + h * a.oh + j] = Ty<T>::from_f(acc / s_L[g]);
      if (a.lse && j == 0)
        a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h] = (s_M[g] + log2f(s_L[g])) * 0.6931471805599453f;
    }
    return;
  }
  const int B = 1 << a.c.shift, gran = min(B, 32), nb = (ntok + B - 1) >> a.c.shift;
  const int i0 = ((bx - P * G) % nchunk) * chunk;
  for (int i = i0 + tid; i < min(nb, i0 + chunk); i += kCmThreads) {
    float w = 0.f;
    const int tile = i * B / kCaT;
    for (int g = 0; g < G; ++g) {
      float z = 0.f;
      for (int u = 0; u < B / gran; ++u)
        z += a.w.psum[(static_cast<size_t>(pair) * a.w.granules + i * (B / gran) + u) * G + g];
      w += z * exp2f(a.w.tmax[(static_cast<size_t>(pair) * a.w.tiles + tile) * G + g] - s_M[g]) / s_L[g];
    }
    float* dst = a.c.weight + static_cast<size_t>(pair) * a.c.max_blocks + i;
    *dst = a.decay == 0.f ? w : fmaf(a.decay, *dst, w);
  }
}

template <typename T, int D, int G>
static cudaError_t attend_t(const AttendArgs& a, int ncta, cudaStream_t st) {
  cudaError_t e = launch_pdl(k_attend<T, D, G>, dim3(ncta), dim3(kCaT), 0, st, a);
  if (e != cudaSuccess) return e;
  const int chunk = 512;
  const int nchunk = a.gather ? (a.c.max_blocks + chunk - 1) / chunk : 0;
  return launch_pdl(k_attend_merge<T, D, G>, dim3(a.c.pairs * (G + nchunk)), dim3(kCmThreads), 0, st, a, ncta, chunk,
                    nchunk);
}

template <typename T, int D>
static cudaError_t attend_g(const AttendArgs& a, int G, int ncta, cudaStream_t st) {
  switch (G) {
    case 1: return attend_t<T, D, 1>(a, ncta, st);
    case 2: return attend_t<T, D, 2>(a, ncta, st);
    case 4: return attend_t<T, D, 4>(a, ncta, st);
    default: return attend_t<T, D, 8>(a, ncta, st);
  }
}

// SMs of the current device (asked once per device).
static cudaError_t device_sms(int* n) {
  static int have[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && have[dev]) { *n = have[dev]; return cudaSuccess; }
  e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
  if (e == cudaSuccess && dev >= 0 && dev < 64) have[dev] = *n;
  return e;
}

static bool attend_heads_ok(const shadowkv_cache& c, int h_q) {
  if (h_q < 1 || h_q % c.h_kv) return false;
  const int G = h_q / c.h_kv;
  return G == 1 || G == 2 || G == 4 || G == 8;
}

}  // namespace skv

extern "C" {

size_t shadowkv_cache_attend_workspace(const shadowkv_cache* c, int h_q) {
  if (skv::cache_checked(c) != SKV_OK) return 0;
  if (!skv::attend_heads_ok(*c, h_q)) {
    skv::set_error(SKV_ERR_UNSUPPORTED, "h_q / h_kv must be 1, 2, 4 or 8");
    return 0;
  }
  int nsm = 0;
  const cudaError_t e = skv::device_sms(&nsm);
  if (e != cudaSuccess) {
    skv::set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
    return 0;
  }
  return skv::attend_layout(*c, h_q / c->h_kv, nsm, nullptr, nullptr);
}

skv_status shadowkv_cache_attend(const shadowkv_cache* c, int dtype, int h_q, const shadowkv_rows* q, float scale,
                                 int gather, float decay, const shadowkv_rows* out, float* lse, void* work,
                                 size_t work_bytes, void* stream) {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (dtype != SKV_DTYPE_F32 && dtype != SKV_DTYPE_BF16) return set_error(SKV_ERR_INVALID_ARG, "bad dtype");
  if (!skv::attend_heads_ok(*c, h_q))
    return set_error(SKV_ERR_UNSUPPORTED, "h_q must be 1, 2, 4 or 8 times h_kv");
  if (!q || !q->ptr || !out || !out->ptr) return set_error(SKV_ERR_INVALID_ARG, "q and out must be non-NULL");
  if (q->sb < 0 || q->sh < 0 || out->sb < 0 || out->sh < 0)
    return set_error(SKV_ERR_INVALID_ARG, "row strides must not be negative");
  if ((c->b > 1 && !out->sb) || (h_q > 1 && !out->sh)) return set_error(SKV_ERR_INVALID_ARG, "an output stride is 0");
  const uintptr_t E = dtype == SKV_DTYPE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(q->ptr) % E || reinterpret_cast<uintptr_t>(out->ptr) % E ||
      reinterpret_cast<uintptr_t>(lse) % 4)
    return set_error(SKV_ERR_INVALID_ARG, "q, out and lse must be aligned to their elements");
  if (!std::isfinite(scale)) return set_error(SKV_ERR_INVALID_ARG, "scale must be finite");
  if (gather != 0 && gather != 1) return set_error(SKV_ERR_INVALID_ARG, "gather must be 0 or 1");
  if (gather && !c->weight) return set_error(SKV_ERR_INVALID_ARG, "the cache keeps no weights");
  if (gather && !std::isfinite(decay)) return set_error(SKV_ERR_INVALID_ARG, "decay must be finite");
  if (!work || reinterpret_cast<uintptr_t>(work) % 256)
    return set_error(SKV_ERR_INVALID_ARG, "the workspace must be non-NULL and 256-byte aligned");
  int nsm = 0;
  cudaError_t e = skv::device_sms(&nsm);
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  const int G = h_q / c->h_kv;
  skv::AttendArgs a;
  if (work_bytes < skv::attend_layout(*c, G, nsm, work, &a.w))
    return set_error(SKV_ERR_INVALID_ARG, "the workspace is smaller than shadowkv_cache_attend_workspace");
  a.c = skv::cache_dev(*c);
  a.q = q->ptr;
  a.out = out->ptr;
  a.lse = lse;
  a.qb = q->sb; a.qh = q->sh;
  a.ob = out->sb; a.oh = out->sh;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.gather = gather;
  a.decay = decay;
  const int ncta = skv::attend_ctas(*c, nsm);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == SKV_DTYPE_BF16)
    e = c->d == 128 ? skv::attend_g<skv::bf16, 128>(a, G, ncta, s) : skv::attend_g<skv::bf16, 64>(a, G, ncta, s);
  else
    e = c->d == 128 ? skv::attend_g<float, 128>(a, G, ncta, s) : skv::attend_g<float, 64>(a, G, ncta, s);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
}

}  // extern "C"
