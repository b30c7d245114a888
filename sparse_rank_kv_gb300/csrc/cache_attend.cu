// Attention of one token per sequence over the 8-bit block cache
// (shadowkv_cache_attend): out = softmax(scale q K^T) V per query head, the
// log of each head's sum, and the weight every block receives.
//
// Memory bounds it: 2 d bytes of codes per token and KV head are read once.
// Measured, 32 query and 8 KV heads of 128 in bf16, weights gathered: batch 8 at
// 128K (2.15 GB) 313 us, 6.9 TB/s; batch 1 at 128K 47 us (39 at that rate); 16
// ragged sequences of up to 9001 tokens (163 MB) 34.4 us (24 at that rate: a
// few CTAs' copies come at half the speed of the others', and the shares are
// fixed beforehand); 90 tokens 5.1 us, all latency.  16 sequences of 9001 tokens
// (295 MB, 43 us at that rate): 51 us, with 64 query heads 57, fp32 51, both 66; heads
// of 64 (22 at that rate) 37.7.  The softmax warps' latency bounds those above 51 and the last.  The CUDA-core form of the
// same split took 8.0 ms at batch 8, 128K.
//
// Every pair's tokens are cut into 128-token tiles; the tiles of all pairs, in
// order, are dealt evenly to the CTAs (consecutive tiles to a CTA), so that
// ragged lengths and few long sequences both fill the GPU.  A CTA leaves one
// partial (max, sum, sum p v) per pair it meets, and k_attend_merge joins a
// pair's partials in order and turns the tiles' sums of p into block weights.
// Lengths are only known on the device: every CTA forms the prefix of the tile counts itself.
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

constexpr int kCaT = 128;         // tokens per tile
constexpr int kCaMostPerSm = 3;   // CTAs per SM, at most

// Small caches: one CTA works a pair's tiles off and finishes it, without the
// prefix sums, the partials and the second launch.  Measured with weights,
// device time of the split form and of this one: 8 pairs of 2 tiles 8.3 and
// 6.6 us, of 4 tiles 8.4 and 9.4 (4 us of host time less), of 8 tiles 8.6 and
// 14.1; 152 pairs of 8 tiles 14.5 and 14.6; 256 pairs of 4 tiles 17.2 and 10.6,
// of 8 tiles 20.6 and 16.1; 16 tiles go either way with the number of waves
// (384 pairs 44 and 36, 512 pairs 56 and 63).
inline bool attend_solo(const shadowkv_cache& c, int nsm) {
  const long long tiles = (static_cast<long long>(c.max_blocks) * c.block + kCaT - 1) / kCaT;
  return tiles <= 4 || (tiles <= 8 && static_cast<long long>(c.b) * c.h_kv >= nsm);
}

// Workspace, in order: per pair the index of its first tile, the total tile
// count, the CTAs' partials, and for the weights every tile's reference
// maximum and the sums of p over granules of min(block, 32) tokens.  (The
// form without a second launch uses the last two alone.)
struct AttendWork {
  int* first;      // [pairs] then the total
  float* part;     // [ctas + pairs][G][d + 2]
  float* tmax;     // [pairs][tiles][G]
  float* psum;     // [pairs][granules][G]
  int tiles, granules;   // per pair, at most
};

// CTAs that share the tiles, at `per_sm` on every SM.
inline int attend_ctas(const shadowkv_cache& c, int nsm, int per_sm) {
  const long long tiles = (static_cast<long long>(c.max_blocks) * c.block + kCaT - 1) / kCaT * c.b * c.h_kv;
  const long long most = static_cast<long long>(per_sm) * nsm;
  return static_cast<int>(tiles < most ? tiles : most);
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
  v.part = reinterpret_cast<float*>(take((attend_ctas(c, nsm, kCaMostPerSm) + pairs) * G * (c.d + 2) * sizeof(float)));
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
  int solo;           // one CTA per pair, which finishes it: no second launch
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
template <int NT>
__device__ __forceinline__ void share_find(const AttendArgs& a, int cta, int ncta, int* s_where, int* s_scan) {
  const int tid = threadIdx.x, P = a.c.pairs;
  const int per = (P + NT - 1) / NT;
  const int p0 = min(P, tid * per), p1 = min(P, p0 + per);
  int sum = 0;
  for (int p = p0; p < p1; ++p) sum += tiles_of(a.c, p);
  if (tid < 2) s_where[tid] = 0;
  int T;
  int before = block_exclusive_scan(sum, s_scan, &T);
  if (tid == 0) s_where[2] = T;
  if (cta == 0 && tid == 0) a.w.first[P] = T;
  const int n = min(ncta, T);
  if (cta < n && sum > 0) {
    const int t0 = share_begin(cta, n, T);
    if (before <= t0 && t0 < before + sum) {
      int p = p0, b = before;
      for (; p < p1 - 1; ++p) {
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

// 2^x by the special function unit (2^-22 relative); results below 2^-126 are 0
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// G adjacent floats (16-byte aligned where G >= 4).
template <int G>
__device__ __forceinline__ void load_heads(const float* p, float* o) {
  if constexpr (G >= 4) {
#pragma unroll
    for (int e = 0; e < G; e += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + e);
      o[e] = v.x; o[e + 1] = v.y; o[e + 2] = v.z; o[e + 3] = v.w;
    }
  } else if constexpr (G == 2) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    o[0] = v.x; o[1] = v.y;
  } else {
    o[0] = *p;
  }
}

// Weight of a pair's block i from its granules' sums of p, its tile's
// references and the heads' maxima M and sums L; stored with the decayed old one.
template <int G>
__device__ __forceinline__ void store_weight(const AttendArgs& a, int pair, int i, const float* M, const float* L) {
  const int B = 1 << a.c.shift, gran = min(B, 32);
  const int tile = i * B / kCaT, ng = B / gran;   // one granule, or 2 or 4 of 32 tokens
  const float* ps = a.w.psum + (static_cast<size_t>(pair) * a.w.granules + static_cast<size_t>(i) * ng) * G;
  float z[4][G], t[G], w = 0.f;
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (u < ng) load_heads<G>(ps + u * G, z[u]);
  load_heads<G>(a.w.tmax + (static_cast<size_t>(pair) * a.w.tiles + tile) * G, t);
#pragma unroll
  for (int g = 0; g < G; ++g) {
    float sum = z[0][g];
#pragma unroll
    for (int u = 1; u < 4; ++u) sum += u < ng ? z[u][g] : 0.f;
    w += sum * ex2(t[g] - M[g]) / L[g];
  }
  float* dst = a.c.weight + static_cast<size_t>(pair) * a.c.max_blocks + i;
  *dst = a.decay == 0.f ? w : fmaf(a.decay, *dst, w);
}
__device__ __forceinline__ float natural_lse(float M, float L) { return (M + log2f(L)) * 0.6931471805599453f; }

// ------------------------------------------------------------ tensor cores
// The codes go to the tensor core as they are (tcgen05 kind::f8f6f4, one
// K-major tile per 128 tokens, straight from bulk copies of whole blocks):
//   S = K Q^T   (M = 128 tokens, K = d),        Q: QP rows per query head
//   O = V^T P^T (M = d, K = 128 tokens),        P: PP rows per query head
// q and p are not e4m3 numbers but sums of them: x = x0 + x1/16 + x2/256 + ...,
// each term the e4m3 rounding of what the ones before leave, 4 bits each.
// Beside a bf16 output four terms hold p to 2^-16 of itself; six hold an fp32 value.
// e4m3's range ends the terms at 2^-10 16^(1-terms) under a largest value of 256 (a
// tile's largest p and largest V scale, whichever tokens have them) or above 224 (a q row): 2^-30 and 2^-29 for bf16, 2^-38 and 2^-37
// for fp32.  Two terms would hold a bf16 query's 8 bits, but only down to 2^-13 of
// its row's largest; rows with an outlier have entries below that, and four hold them down to 2^-21.  Decoding has
// G <= 8 query rows for a tile of at least 16, so the terms fill rows that
// would be padding, and no code is ever converted.  Products of e4m3 numbers accumulate in fp32 (measured: within
// 2^-22 of the sum of magnitudes, as an fp32 matrix product).
constexpr int kCaSoft = 128;                  // softmax threads: warps 0..3, thread = token, then dimension
constexpr int kCaThreads = kCaSoft + 64;      // warp 4: copies, warp 5: tcgen05.mma

template <typename T, int D, int G>
struct Ca {
  static constexpr int QP = sizeof(T) == 2 ? 4 : 6, PP = sizeof(T) == 2 ? 4 : 6;
  static constexpr int N1 = (G * QP + 15) / 16 * 16, N2 = (G * PP + 15) / 16 * 16;
  static constexpr int KB = kCaT * D, Stage = 2 * KB;       // K tile, V tile
  static constexpr int QB = N1 * D, PB = N2 * kCaT;
  static constexpr int Misc = 2048;
  // CTAs per SM: while one waits for its barriers the others compute; three
  // where the registers allow it: 18 warps on four schedulers leave 96 each, which
  // bf16 with four heads and fp32 with two keep to (fp32 with four takes 111 to
  // 114, bf16 with eight 146).  Measured against two: 16 sequences of
  // 9001 tokens with heads of 64 42.2 -> 36.8 us, batch 8 at 128K with heads of 128
  // 320 -> 313 us; a fourth for one or two heads of 64 gave nothing.
  static constexpr int PerSm = G <= (sizeof(T) == 2 ? 4 : 2) ? 3 : 2;
  static constexpr int SmemMax = (228 / PerSm - 1) * 1024;
  static constexpr int NST = (SmemMax - 128 - QB - 2 * PB - Misc) / Stage;
  static constexpr int Smem = 128 + NST * Stage + QB + 2 * PB + Misc;
  static constexpr int Cols0 = 2 * N1 + 2 * N2;
  static constexpr int Cols = Cols0 <= 32 ? 32 : Cols0 <= 64 ? 64 : Cols0 <= 128 ? 128 : 256;
  static_assert(NST >= 2 && NST <= 7 && Cols0 <= 256, "attention tile");
};

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f8f6f4, e4m3 A and B (format 0), fp32 D, M = 128; A K-major, B
// K-major or (bn: bit 16) N-major
constexpr uint32_t idesc_e4m3(int N, bool bn = false) {
  return (1u << 4) | (bn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
// x[g] = the sum of a head's products over its terms, v[i G + g] 16^-i, on pairs
// of heads (fma.f32x2).
template <int G, int Terms>
__device__ __forceinline__ void join_terms(const float* v, float* x) {
  if constexpr (G == 1) {
    x[0] = v[Terms - 1];
#pragma unroll
    for (int i = Terms - 2; i >= 0; --i) x[0] = fmaf(x[0], 1.f / 16.f, v[i]);
  } else {
#pragma unroll
    for (int g = 0; g < G; g += 2) {
      const float* a = v + (Terms - 1) * G + g;
      float2 y = make_float2(a[0], a[1]);
#pragma unroll
      for (int i = Terms - 2; i >= 0; --i) y = __ffma2_rn(y, make_float2(1.f / 16.f, 1.f / 16.f), make_float2(v[i * G + g], v[i * G + g + 1]));
      x[g] = y.x;
      x[g + 1] = y.y;
    }
  }
}
// Sum of z[g] over groups of `gran` (16 or 32) lanes: lanes exchange half of
// their heads at each step until one is left (G = 4: 6 shuffles instead of 20).
// Lane l of a group holds the sum of head head_of_lane<G>(l) for l < G.
template <int G>
__device__ __forceinline__ float granule_sum(const float* z, int lane, int gran) {
  float v[G];
#pragma unroll
  for (int g = 0; g < G; ++g) v[g] = z[g];
  int o = 1;
#pragma unroll
  for (int h = G / 2; h > 0; h >>= 1, o <<= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int g = 0; g < h; ++g) {
      const float mine = up ? v[g + h] : v[g], other = up ? v[g] : v[g + h];
      v[g] = mine + __shfl_xor_sync(0xffffffffu, other, o);
    }
  }
#pragma unroll
  for (int w = G; w < 16; w <<= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], w);
  if (gran == 32) v[0] += __shfl_xor_sync(0xffffffffu, v[0], 16);
  return v[0];
}
template <int G>
__device__ __forceinline__ int head_of_lane(int l) {
  int h = 0;
#pragma unroll
  for (int b = G / 2, o = 1; b > 0; b >>= 1, o <<= 1) h += l & o ? b : 0;
  return h;
}
__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// of a tile in its stage, beside its tokens (at most kCaT)
enum : int { kFirst = 256, kLast = 512, kEnd = 1024 };

// A CTA's tiles in order: `left` tiles from tile `tile` of pair `pair`.
struct TileCursor {
  int pair, tile, left, ntok, nt;
  __device__ __forceinline__ void begin(const CacheDev& c, int p, int t, int n) {
    pair = p;
    tile = t;
    left = n;
    ntok = cache_tokens(c, p);
    nt = (ntok + kCaT - 1) / kCaT;
  }
  // to the next tile; true when it is another pair's
  __device__ __forceinline__ bool next(const CacheDev& c) {
    if (--left <= 0) return false;
    if (++tile < nt) return false;
    tile = 0;
    do {
      if (++pair >= c.pairs) { left = 0; return false; }
      ntok = cache_tokens(c, pair);
      nt = (ntok + kCaT - 1) / kCaT;
    } while (nt == 0);
    return true;
  }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kCaThreads, (Ca<T, D, G>::PerSm)) k_attend(const __grid_constant__ AttendArgs a) {
  using C = Ca<T, D, G>;
  constexpr int N1 = C::N1, N2 = C::N2, NST = C::NST;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  unsigned char* stages = smem;
  unsigned char* qbuf = stages + NST * C::Stage;        // the pair's q
  unsigned char* pbuf = qbuf + C::QB;                   // [2], by tile
  unsigned char* misc = pbuf + 2 * C::PB;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);   // [NST <= 7]
  uint64_t* empty = full + 8;                           // [NST]
  uint64_t* sfull = empty + 8;                          // [2]
  uint64_t* pfull = sfull + 2;
  uint64_t* ofull = pfull + 2;
  uint64_t* qfull = ofull + 2;                          // [2]
  float* sqs = reinterpret_cast<float*>(misc + 192);    // [8] q scales
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 640);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 644);
  int* s_where = reinterpret_cast<int*>(misc + 648);    // [3]
  float* red = reinterpret_cast<float*>(misc + 256);    // [2][4][G] maxima, [4][G] sums
  int* s_scan = reinterpret_cast<int*>(misc + 512);     // [32], before the sums are used
  float* ssc = reinterpret_cast<float*>(misc + 672);    // [NST][20]: K scales, V factors, V reference
  int* sinfo = reinterpret_cast<int*>(misc + 1248);     // [NST][4]: the stage's tile (below)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!a.solo) tc::grid_dep_launch();   // (a call's last kernel lets nothing start early)

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(&full[i], 2);   // the copies, and the scales
      tc::mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sfull[i], 1);
      tc::mbar_init(&pfull[i], kCaSoft / 32);
      tc::mbar_init(&ofull[i], 1);
      tc::mbar_init(&qfull[i], kCaSoft / 32);
    }
    tc::fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == 5) {
    tc::tmem_alloc(tmem_slot, C::Cols);
    tc::tmem_relinquish();
  }
  // q rows past the terms stay zero
  for (int i = tid; i < C::QB / 16; i += kCaThreads)
    reinterpret_cast<uint4*>(qbuf)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  tc::fence_before();
  tc::grid_dep_wait();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const int cta = blockIdx.x;
  int t0 = 0, ntile = 0;
  if (a.solo) {
    if (tid == 0) {
      s_where[0] = cta;
      s_where[1] = 0;
      s_where[2] = tiles_of(a.c, cta);
    }
    __syncthreads();
    ntile = s_where[2];
  } else {
    share_find<kCaThreads>(a, cta, gridDim.x, s_where, s_scan);
    const int total = s_where[2], n = min(static_cast<int>(gridDim.x), total);
    if (cta < n) {
      t0 = share_begin(cta, n, total);
      ntile = share_begin(cta + 1, n, total) - t0;
    }
  }
  const int shift = a.c.shift, B = 1 << shift;
  auto abort_now = [&]() {
    *s_abort = 1;
    flag_error(a.c.status, DEV_TIMEOUT);
  };

  if (ntile > 0 && warp == 4) {
    // ------------------------------------------------------------ copies
    // This warp alone walks the pairs; what the others need to know of a
    // tile lies in its stage: pair, tile, the tile's tokens and kFirst, kLast
    // (of the CTA's tiles of that pair), kEnd and, above them, the next tile's pair.
    // lane = block of the tile; block ids are loaded two tiles ahead, the
    // blocks' scales one ahead.  The codes are read once: evicted first from
    // L2 (338 us without and 322 with it, at batch 8, 128K and two CTAs per SM)
    TileCursor cur, nx1, nx2;
    cur.begin(a.c, s_where[0], s_where[1], ntile);
    auto tokens = [&](const TileCursor& c) { return c.left > 0 ? max(0, min(kCaT, c.ntok - c.tile * kCaT)) : 0; };
    auto blocks = [&](const TileCursor& c) { return (tokens(c) + B - 1) >> shift; };
    auto id_of = [&](const TileCursor& c) {
      return lane < blocks(c) ? cache_block(a.c, c.pair, ((c.tile * kCaT) >> shift) + lane) : 0;
    };
    const uint64_t once = tc::l2_evict_first_policy();
    int id = id_of(cur), id1 = 0;
    float ks = 0.f, vs = 0.f;
    int it = 0, before = -1;   // before: the previous tile's pair
    for (;; ++it) {
      const int st = it % NST, use = it / NST;
      bool ok = true;
      if (lane == 0) ok = !*s_abort && tc::mbar_wait(&empty[st], (use & 1) ^ 1, kWaitLimit);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) {
        if (lane == 0) abort_now();
        break;
      }
      const int nb = blocks(cur);
      if (lane == 0) tc::mbar_expect_tx(&full[st], static_cast<uint32_t>(nb) * 2u * (B * D));
      __syncwarp();
      if (lane < nb) {
        unsigned char* dst = stages + st * C::Stage + lane * (B * D);
        const size_t src = static_cast<size_t>(id) * (B * D);
        tc::bulk_load_hint(dst, a.c.kc + src, B * D, &full[st], once);
        tc::bulk_load_hint(dst + C::KB, a.c.vc + src, B * D, &full[st], once);
      }
      if (it == 0) {
        ks = a.c.ks[id];
        vs = a.c.vs[id];
        nx1 = cur;
        nx1.next(a.c);
        id1 = id_of(nx1);
      }
      nx2 = nx1;
      if (nx2.left > 0) nx2.next(a.c);
      const int id2 = id_of(nx2);
      const float ks1 = a.c.ks[id1], vs1 = a.c.vs[id1];
      float* sc = ssc + st * 20;
      // V's scales relative to the tile's largest, which O is multiplied by
      float vref = lane < nb ? fabsf(vs) : 0.f;
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) vref = fmaxf(vref, __shfl_xor_sync(0xffffffffu, vref, o));
      if (lane < nb) {
        sc[lane] = ks;
        sc[8 + lane] = vref > 0.f ? vs / vref * 256.f : vs == vs ? 0.f : vs;
      }
      if (lane == 0) {
        sc[16] = vref * (1.f / 256.f);
        const bool end = nx1.left <= 0;
        reinterpret_cast<int4*>(sinfo)[st] =
            make_int4(cur.pair, cur.tile, tokens(cur) | (cur.pair != before ? kFirst : 0) |
                                              (end || nx1.pair != cur.pair ? kLast : 0) | (end ? kEnd : 0),
                      nx1.pair);
        if (cur.tile == 0 && !a.solo) a.w.first[cur.pair] = t0 + it;
      }
      before = cur.pair;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&full[st]);
      if (nx1.left <= 0) { ++it; break; }
      cur = nx1;
      nx1 = nx2;
      id = id1;
      id1 = id2;
      ks = ks1;
      vs = vs1;
    }
    // after an abort, no copy may still be on its way when the CTA ends
    if (lane == 0 && *s_abort)
      for (int u = max(0, it - NST); u < it; ++u) tc::mbar_wait(&full[u % NST], (u / NST) & 1, kWaitLimit);
    __syncwarp();
  } else if (ntile > 0 && warp == 5) {
    // ------------------------------------------------------------ tensor core
    if (lane == 0) {
      const uint32_t tS = tmem, tO = tmem + 2 * N1;
      // S(i) needs its K, its pair's q, and the softmax to be done with S(i - 2)
      // (P(i - 2) is there); O(j) needs P(j).  Whichever is ready goes, O
      // first: it frees a stage for the next copy
      int i = 0, j = 0, runs = 0;      // next S, next O; runs: pair's turn of tile i
      bool more = true;
      uint64_t t_last = 0;
      int idle = 0;
      while (more || j < i) {
        bool did = false;
        if (j < i && tc::mbar_test(&pfull[j & 1], (j >> 1) & 1)) {
          tc::fence_after();
          const int st = j % NST;
          const uint32_t v0 = tc::smem_u32(stages + st * C::Stage + C::KB), p0 = tc::smem_u32(pbuf + (j & 1) * C::PB);
#pragma unroll
          for (int k = 0; k < kCaT / 32; ++k)
            mma_e4m3(tO + (j & 1) * N2, tc::desc_k_none(v0 + k * (2 * D * 16), D * 16, 128),
                     tc::desc_k_none(p0 + k * 512, 128, kCaT * 16), idesc_e4m3(N2, true), k > 0);
          tc::mma_commit(&ofull[j & 1]);
          tc::mma_commit(&empty[st]);
          ++j;
          did = true;
        }
        int flags = 0, turn = runs;
        bool go = more && j >= i - 1 && tc::mbar_test(&full[i % NST], (i / NST) & 1);
        if (go) {
          flags = sinfo[(i % NST) * 4 + 2];
          if (i > 0 && (flags & kFirst)) ++turn;
          go = tc::mbar_test(&qfull[turn & 1], (turn >> 1) & 1);
        }
        if (go) {
          runs = turn;
          tc::fence_after();
          const uint32_t k0 = tc::smem_u32(stages + (i % NST) * C::Stage), q0 = tc::smem_u32(qbuf);
#pragma unroll
          for (int k = 0; k < D / 32; ++k)
            mma_e4m3(tS + (i & 1) * N1, tc::desc_k_none(k0 + k * 256, 128, 8 * D),
                     tc::desc_k_none(q0 + k * (2 * N1 * 16), N1 * 16, 128), idesc_e4m3(N1), k > 0);
          tc::mma_commit(&sfull[i & 1]);
          ++i;
          more = !(flags & kEnd);
          did = true;
        }
        if (did) {
          idle = 0;
          continue;
        }
        // nothing ready: look at the clock now and then
        if (idle == 0) t_last = tc::globaltimer_ns();
        if ((++idle & 63) == 0 && (*s_abort || tc::globaltimer_ns() - t_last > kWaitLimit)) {
          abort_now();
          break;
        }
      }
    }
    __syncwarp();
  } else if (ntile > 0) {
    // ------------------------------------------------------------ softmax
    const uint32_t tS = tmem + (static_cast<uint32_t>(warp) << 21), tO = tS + 2 * N1;
    const int gran = min(B, 32);
    bool ok = true;
    // q's terms, each head scaled by a power of two so that the largest
    // entry is at most 448; an entry that is not finite makes the head NaN
    auto lay_q = [&](int pair, int turn) {
      const int seq = pair / a.c.h_kv, kvh = pair - seq * a.c.h_kv;
      for (int g = warp; g < G; g += 4) {
        const T* row = static_cast<const T*>(a.q) + seq * a.qb + (static_cast<long long>(kvh) * G + g) * a.qh;
        float x[D / 32], m = 0.f;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
          x[e] = Ty<T>::to_f(row[lane + 32 * e]);
          const float ax = fabsf(x[e]);
          m = fmaxf(m, ax < INFINITY ? ax : 0.f);
          if (!(ax < INFINITY)) x[e] = __int_as_float(0x7fffffff);
        }
        m = warp_max(m);
        const float s = cache_scale_of(m), inv = 1.f / s;
#pragma unroll
        for (int e = 0; e < D / 32; e += 2) {
          float u = x[e] * inv, v = x[e + 1] * inv;
          const int j = lane + 32 * e;
          unsigned char* dst = qbuf + (j >> 4) * (N1 * 16) + (j & 15);
#pragma unroll
          for (int i = 0; i < C::QP; ++i) {
            const uint32_t c2 = e4m3_pack2(u, v);
            dst[(i * G + g) * 16] = static_cast<unsigned char>(c2);
            dst[(i * G + g) * 16 + 2 * N1 * 16] = static_cast<unsigned char>(c2 >> 8);
            const float2 f = e4m3_unpack2(c2);
            u = (u - f.x) * 16.f;
            v = (v - f.y) * 16.f;
          }
        }
        if (lane == 0) sqs[g] = s * a.scale_log2;
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&qfull[turn & 1]);
      ok = tc::named_sync_and(1, kCaSoft, ok);
    };
    lay_q(s_where[0], 0);
    int turn = 0;
    // running maximum, sum and output of the pair's run; p is relative to its own
    // tile's maximum, whatever larger one came before (a token with most of
    // the weight and little value must not push other tiles' terms out)
    float m[G], l[G], acc[G], al[G], be[G];
    // adds tile j's O to the run's sums
    auto take_o = [&](int j) {
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&ofull[j & 1], (j >> 1) & 1, kWaitLimit));
      if (!ok) return;
      tc::fence_after();
      float o[N2], x[G];
#pragma unroll
      for (int c = 0; c < N2; c += 16) tc::tmem_ld16(tO + (j & 1) * N2 + c, o + c);
      join_terms<G, C::PP>(o, x);
#pragma unroll
      for (int g = 0; g < G; ++g) acc[g] = fmaf(acc[g], al[g], x[g] * be[g]);
    };
    // (a wait that gave up shows at the next barrier, so that all 128 threads
    // leave together)
    for (int it = 0;; ++it) {
      const int st = it % NST;
      ok = __all_sync(0xffffffffu, ok && tc::mbar_wait(&full[st], (it / NST) & 1, kWaitLimit) &&
                                       tc::mbar_wait(&sfull[it & 1], (it >> 1) & 1, kWaitLimit));
      const int4 info = reinterpret_cast<const int4*>(sinfo)[st];
      const int pair = info.x, t = info.y, cnt = info.z & 255, flags = info.z;
      if (flags & kFirst) {
#pragma unroll
        for (int g = 0; g < G; ++g) {
          m[g] = -INFINITY;
          l[g] = acc[g] = al[g] = be[g] = 0.f;
        }
      }
      float s[G];
      const float* sc = ssc + st * 20;
      const int blk = tid >> shift;
      if (ok) {
        tc::fence_after();
        float v[N1];
#pragma unroll
        for (int c = 0; c < N1; c += 16) tc::tmem_ld16(tS + (it & 1) * N1 + c, v + c);
        const float ks = sc[blk];
        float qs[G], x[G];
        load_heads<G>(sqs, qs);
        join_terms<G, C::QP>(v, x);
#pragma unroll
        for (int g = 0; g < G; ++g) s[g] = tid < cnt ? x[g] * (qs[g] * ks) : -INFINITY;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float x = redux_max(s[g]);
          if (lane == 0) red[(it & 1) * 32 + warp * G + g] = x;
        }
      }
      ok = tc::named_sync_and(1, kCaSoft, ok);
      if (!ok) break;
      float al_new[G], be_new[G];
      unsigned char* pb = pbuf + (it & 1) * C::PB + tid * 16;
      const float vf = tid < cnt ? sc[8 + blk] : 0.f, vref = sc[16];
      float p[G], rd[4][G];
#pragma unroll
      for (int w = 0; w < 4; ++w) load_heads<G>(red + (it & 1) * 32 + w * G, rd[w]);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float mt = fmaxf(fmaxf(rd[0][g], rd[1][g]), fmaxf(rd[2][g], rd[3][g]));
        const float tref = mt == -INFINITY ? 0.f : mt, mn = fmaxf(mt, m[g]), ref = mn == -INFINITY ? 0.f : mn;
        al_new[g] = ex2(m[g] - ref);
        be_new[g] = ex2(mt - ref);
        m[g] = mn;
        p[g] = ex2(s[g] - tref);
        l[g] = fmaf(l[g], al_new[g], p[g] * be_new[g]);
        be_new[g] *= vref;
        if (a.gather && tid == 0) a.w.tmax[(static_cast<size_t>(pair) * a.w.tiles + t) * G + g] = tref;
      }
      if (a.gather) {
        const float z = granule_sum<G>(p, lane, gran);
        const int l = lane & (gran - 1);
        if (l < G)
          a.w.psum[(static_cast<size_t>(pair) * a.w.granules + (t * kCaT + tid) / gran) * G + head_of_lane<G>(l)] = z;
      }
      // p's terms, times the token's V scale; row term G + head.  The operand is
      // N-major ([N2/16][token][16 rows]), so that a token's rows are 16-byte stores
      uint32_t pw[N2 / 4] = {};
#pragma unroll
      for (int g = 0; g < G; g += 2) {
        float u = p[g] * vf, v = G > 1 ? p[g + (G > 1)] * vf : 0.f;
        __half2 x;
#pragma unroll
        for (int i = 0; i < C::PP; ++i) {
          uint32_t c2;
          if (sizeof(T) == 4 || i == 0) {
            c2 = e4m3_pack2(u, v);
            const float2 f = e4m3_unpack2(c2);
            u = (u - f.x) * 16.f;
            v = (v - f.y) * 16.f;
            // What the first term leaves (exact, below 2^-4 of p) as an fp16, whose 11 bits
            // three terms hold exactly: 2^-16 of p, as four terms from fp32 in half the
            // operations.  (p as one fp16 in three terms, 2^-11: 1% faster, and it shows in the output where
            // values cancel)
            x = __floats2half2_rn(u, v);
          } else {
            c2 = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
            const __half2 f = __half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2), __NV_E4M3));
            x = __hmul2(__hsub2(x, f), __float2half2_rn(16.f));
          }
          const int n = i * G + g;
          pw[n >> 2] |= (G > 1 ? c2 : c2 & 0xffu) << (8 * (n & 3));
        }
      }
#pragma unroll
      for (int c = 0; c < N2 / 16; ++c)
        *reinterpret_cast<uint4*>(pb + c * (kCaT * 16)) = make_uint4(pw[4 * c], pw[4 * c + 1], pw[4 * c + 2], pw[4 * c + 3]);
      // V past the tokens may be any bytes, NaN too: zero under zero weights
      if (cnt < kCaT && tid < D) {
        unsigned char* vb = stages + st * C::Stage + C::KB + tid * 16;
        for (int u = cnt >> 4; u < kCaT / 16; ++u) {
          uint4* w = reinterpret_cast<uint4*>(vb + u * (D * 16));
          const int keep = cnt - u * 16;   // bytes kept, if any
          if (keep <= 0) {
            *w = make_uint4(0, 0, 0, 0);
          } else {
            uint4 x = *w;
            uint32_t* xw = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int kb = keep - 4 * e;
              xw[e] = kb >= 4 ? xw[e] : kb <= 0 ? 0u : xw[e] & ((1u << (8 * kb)) - 1u);
            }
            *w = x;
          }
        }
      }
      tc::fence_proxy_async_smem();
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&pfull[it & 1]);
      // the next pair's q, so that its S can start while this pair ends (this
      // tile's S, which is here, was the last reader of the pair's own)
      if ((flags & (kLast | kEnd)) == kLast) lay_q(info.w, turn + 1);
      if (!(flags & kFirst)) take_o(it - 1);
#pragma unroll
      for (int g = 0; g < G; ++g) {
        al[g] = al_new[g];
        be[g] = be_new[g];
      }
      if (!(flags & kLast)) continue;
      take_o(it);
      tc::fence_before();
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float z = warp_sum(l[g]);
        if (lane == 0) red[64 + warp * G + g] = z;
      }
      if (a.solo) {
        ok = tc::named_sync_and(1, kCaSoft, ok);
        if (!ok) break;
        const int seq = pair / a.c.h_kv, h0 = (pair - seq * a.c.h_kv) * G;
#pragma unroll
        for (int g = 0; g < G; ++g) {
          const float* rd = red + 64 + g;
          l[g] = rd[0] + rd[G] + rd[2 * G] + rd[3 * G];
          m[g] = m[g] == -INFINITY ? 0.f : m[g];
          if (tid < D) static_cast<T*>(a.out)[seq * a.ob + (h0 + g) * a.oh + tid] = Ty<T>::from_f(acc[g] / l[g]);
          if (a.lse && tid == g) a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h0 + g] = natural_lse(m[g], l[g]);
        }
        if (a.gather)   // (the barrier stands between the sums' stores and these loads)
          for (int i = tid; i < (t * kCaT + cnt + B - 1) >> shift; i += kCaSoft) store_weight<G>(a, pair, i, m, l);
        break;
      }
      // the partial of (this CTA, pair)
      float* part = a.w.part + static_cast<size_t>(cta + pair) * G * (D + 2);
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (tid < D) part[g * (D + 2) + tid] = acc[g];
      ok = tc::named_sync_and(1, kCaSoft, ok);
      if (tid < G) {
        const float* rd = red + 64 + tid;
        float mm = m[0];
#pragma unroll
        for (int g = 1; g < G; ++g) mm = tid == g ? m[g] : mm;
        part[tid * (D + 2) + D] = mm;
        part[tid * (D + 2) + D + 1] = rd[0] + rd[G] + rd[2 * G] + rd[3 * G];
      }
      ++turn;
      if (!ok || (flags & kEnd)) break;
    }
    if (!ok && tid == 0) abort_now();
  } else if (a.solo && ntile == 0) {
    // a pair without tokens
    const int seq = cta / a.c.h_kv, h0 = (cta - seq * a.c.h_kv) * G;
    for (int i = tid; i < G * D; i += kCaThreads)
      static_cast<T*>(a.out)[seq * a.ob + (h0 + i / D) * a.oh + i % D] = Ty<T>::from_f(0.f);
    if (a.lse && tid < G) a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h0 + tid] = -INFINITY;
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 5) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, C::Cols);
  }
}

// ------------------------------------------------------------ merge
constexpr int kCmThreads = 256;
constexpr int kCmChunk = 512;    // cache blocks whose weights a CTA forms

// Blocks 0 .. pairs G - 1: the output of a query head.  The others, with
// weights: kCmChunk cache blocks of a pair.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kCmThreads)
k_attend_merge(const __grid_constant__ AttendArgs a, int ncta, int nchunk) {
  constexpr int SL = kCmThreads / D, Pre = 8;   // partials per pass; rows held while the maxima are formed
  __shared__ float s_M[G], s_L[G], s_acc[SL][D];
  const int tid = threadIdx.x;
  tc::grid_dep_wait();
  const int P = a.c.pairs, bx = blockIdx.x;
  const bool head_role = bx < P * G;
  const int pair = head_role ? bx / G : (bx - P * G) / nchunk;
  const int total = a.w.first[P], f = a.w.first[pair];   // (f is not written for a pair without tokens)
  const int ntok = cache_tokens(a.c, pair), nt = (ntok + kCaT - 1) / kCaT;
  const int seq = pair / a.c.h_kv, kvh = pair - seq * a.c.h_kv;
  if (nt == 0 || total <= 0) {
    if (head_role) {
      const int h = kvh * G + bx % G;
      if (tid < D) static_cast<T*>(a.out)[seq * a.ob + h * a.oh + tid] = Ty<T>::from_f(0.f);
      if (a.lse && tid == 0) a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h] = -INFINITY;
    }
    return;
  }
  const int n = min(ncta, total);
  // (the bounds hold anyway unless the counts changed since the first launch)
  const int f0 = min(max(f, 0), total - 1);
  const int c0 = share_owner(f0, n, total), c1 = share_owner(min(f0 + nt, total) - 1, n, total);
  const int g_out = bx % G, j = tid % D, sl = tid / D;
  const float* rows = a.w.part + (static_cast<size_t>(c0 + pair) * G + g_out) * (D + 2);   // partial c0 + u: + u G (D + 2)
  float pre[Pre], pm[Pre];
  if (head_role) {
#pragma unroll
    for (int u = 0; u < Pre; ++u) {
      const bool on = c0 + sl + u * SL <= c1;
      const float* p = rows + static_cast<size_t>(sl + u * SL) * G * (D + 2);
      pre[u] = on ? p[j] : 0.f;
      pm[u] = on ? p[D] : -INFINITY;
    }
  }
  // the heads' largest maximum and total sum over the pair's partials
  if (tid < 32 * G) {
    const int g = tid / 32, lane = tid & 31;
    float M = -INFINITY;
    for (int c = c0 + lane; c <= c1; c += 32)
      M = fmaxf(M, a.w.part[(static_cast<size_t>(c + pair) * G + g) * (D + 2) + D]);
    M = warp_max(M);
    const float ref = M == -INFINITY ? 0.f : M;
    float L = 0.f;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float* p = a.w.part + (static_cast<size_t>(c + pair) * G + g) * (D + 2) + D;
      L = fmaf(p[1], ex2(p[0] - ref), L);
    }
    L = warp_sum(L);
    if (lane == 0) { s_M[g] = ref; s_L[g] = L; }
  }
  __syncthreads();
  if (head_role) {
    float acc = 0.f;
#pragma unroll
    for (int u = 0; u < Pre; ++u) acc = fmaf(pre[u], ex2(pm[u] - s_M[g_out]), acc);
#pragma unroll 4
    for (int c = c0 + sl + Pre * SL; c <= c1; c += SL) {
      const float* p = rows + static_cast<size_t>(c - c0) * G * (D + 2);
      acc = fmaf(p[j], ex2(p[D] - s_M[g_out]), acc);
    }
    s_acc[sl][j] = acc;
    __syncthreads();
    if (sl == 0) {
#pragma unroll
      for (int u = 1; u < SL; ++u) acc += s_acc[u][j];
      const int h = kvh * G + g_out;
      static_cast<T*>(a.out)[seq * a.ob + h * a.oh + j] = Ty<T>::from_f(acc / s_L[g_out]);
      if (a.lse && j == 0)
        a.lse[static_cast<size_t>(seq) * a.c.h_kv * G + h] = natural_lse(s_M[g_out], s_L[g_out]);
    }
    return;
  }
  const int nb = (ntok + (1 << a.c.shift) - 1) >> a.c.shift;
  const int i0 = ((bx - P * G) % nchunk) * kCmChunk;
  for (int i = i0 + tid; i < min(nb, i0 + kCmChunk); i += kCmThreads) {
    store_weight<G>(a, pair, i, s_M, s_L);
  }
}

template <typename T, int D, int G>
static cudaError_t attend_t(const AttendArgs& a, const shadowkv_cache& c, int nsm, cudaStream_t st) {
  const int ncta = attend_ctas(c, nsm, Ca<T, D, G>::PerSm);
  const auto kern = k_attend<T, D, G>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), Ca<T, D, G>::Smem);
  if (e == cudaSuccess)
    e = launch_pdl(kern, dim3(a.solo ? a.c.pairs : ncta), dim3(kCaThreads), Ca<T, D, G>::Smem, st, a);
  if (e != cudaSuccess || a.solo) return e;
  const int nchunk = a.gather ? (a.c.max_blocks + kCmChunk - 1) / kCmChunk : 0;
  return launch_pdl(k_attend_merge<T, D, G>, dim3(a.c.pairs * (G + nchunk)), dim3(kCmThreads), 0, st, a, ncta, nchunk);
}

template <typename T, int D>
static cudaError_t attend_g(const AttendArgs& a, int G, const shadowkv_cache& c, int nsm, cudaStream_t st) {
  switch (G) {
    case 1: return attend_t<T, D, 1>(a, c, nsm, st);
    case 2: return attend_t<T, D, 2>(a, c, nsm, st);
    case 4: return attend_t<T, D, 4>(a, c, nsm, st);
    default: return attend_t<T, D, 8>(a, c, nsm, st);
  }
}

// SMs of the current device (asked once per device).
cudaError_t device_sms(int* n) {
  static std::atomic<int> have[64] = {};   // (any thread may ask)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 0 && dev < 64 && (*n = have[dev])) return cudaSuccess;
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

size_t shadowkv_cache_attend_workspace(const shadowkv_cache* c, int h_q) try {
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
} catch (...) {   // host memory for an error text or a table ran out
  return 0;
}

skv_status shadowkv_cache_attend(const shadowkv_cache* c, int dtype, int h_q, const shadowkv_rows* q, float scale,
                                 int gather, float decay, const shadowkv_rows* out, float* lse, void* work,
                                 size_t work_bytes, void* stream) try {
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
  if (static_cast<long long>(c->b) * c->h_kv * (8 + (c->max_blocks + skv::kCmChunk - 1) / skv::kCmChunk) >= (1LL << 31))
    return set_error(SKV_ERR_UNSUPPORTED, "too many sequences and heads for one call");
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
  a.solo = skv::attend_solo(*c, nsm);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  if (dtype == SKV_DTYPE_BF16)
    e = c->d == 128 ? skv::attend_g<skv::bf16, 128>(a, G, *c, nsm, s) : skv::attend_g<skv::bf16, 64>(a, G, *c, nsm, s);
  else
    e = c->d == 128 ? skv::attend_g<float, 128>(a, G, *c, nsm, s) : skv::attend_g<float, 64>(a, G, *c, nsm, s);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
