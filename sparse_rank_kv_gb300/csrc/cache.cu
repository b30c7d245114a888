// The 8-bit block cache (include/shadowkv.h): its checks, the append that
// quantises new tokens into it, and the eviction of whole blocks by gathered
// attention weight.
//
// Every kernel waits for its stream's previous kernel before it touches
// memory.  Only a call's inner kernels let their dependents start early: a
// call's last kernel does not, since kernels of the library read some of
// their inputs before their own grid-dependency wait.
#include <cfloat>
#include <cstdint>
#include <mutex>

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

__device__ __forceinline__ bool is_pow2(float s) { return (__float_as_uint(s) & 0x7fffffu) == 0u; }

// Two held codes (low 16 bits) under a scale larger by 1 / ratio.
__device__ __forceinline__ uint32_t rescale2(uint32_t c2, float ratio) {
  const float2 f = e4m3_unpack2(c2);
  return e4m3_pack2(f.x * ratio, f.y * ratio);
}
__device__ __forceinline__ uint32_t rescale4(uint32_t c4, float ratio) {
  return rescale2(c4, ratio) | (rescale2(c4 >> 16, ratio) << 16);
}

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

// Bytes t of w0, w1 (t < 4) replaced by the low and the high code of c2.
__device__ __forceinline__ void put_codes(uint32_t* w0, uint32_t* w1, int t, uint32_t c2) {
  const int sh = t * 8;
  *w0 = (*w0 & ~(0xffu << sh)) | ((c2 & 0xffu) << sh);
  *w1 = (*w1 & ~(0xffu << sh)) | (((c2 >> 8) & 0xffu) << sh);
}

__device__ __forceinline__ void load32(uint32_t* w, const void* p) {
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void store32(void* p, const uint32_t* a, const uint32_t* b) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]),
               "r"(b[0]), "r"(b[1]), "r"(b[2]), "r"(b[3])
               : "memory");
}

// One block's K or V in the hands of TPJ threads: 16 code bytes of K per unit
// (16 dimensions of a row), 2 x 16 of V (16 tokens of two dimensions), so that
// every store is 16 bytes and the loads of a unit's elements are all in
// flight together.  Elements are loaded once and wait in registers while the
// block's largest magnitude is found.
template <typename T, int D, int B>
struct Ap {
  static constexpr int TPJ = B * D / 32;                     // 32 to 512
  static constexpr int NT = TPJ < kApThreads ? kApThreads : TPJ;   // threads per CTA
  static constexpr int UV = 1, UK = 2;                       // units per thread
  // CTAs per SM the registers are cut for.  Measured at 2, 3 and 4 (four ragged
  // prompts of up to 6000 tokens, d = 128): blocks of 16 27.3, 29.1 and 26.0 us,
  // of 32 27.4, 28.0 and 22.7, of 64 29.4, 24.4 and 23.6; d = 64, blocks of 16:
  // 13.1, 14.5 and 16.7
  static constexpr int MinCtas = sizeof(T) == 4 ? 1 : TPJ == 32 || TPJ == 512 ? 2 : 4;
  static constexpr int E = sizeof(T) / 2;                    // 32-bit words per two elements
  static constexpr int Words = 16 * UV * E;                  // raw words per thread
  // unit u of K: 8 consecutive threads take a group's 8 rows (128 adjacent code bytes)
  __device__ __forceinline__ static int k_row(int u) { return (u / (D / 2) << 3) + (u & 7); }
  __device__ __forceinline__ static int k_piece(int u) { return (u >> 3) % (D / 16); }
  __device__ __forceinline__ static int v_tok(int u) { return u / (D / 2) << 4; }
  __device__ __forceinline__ static int v_dim(int u) { return u % (D / 2) * 2; }
  // the two elements at pair index p of the raw words
  __device__ __forceinline__ static float2 pair(const uint32_t* w, int p) {
    if constexpr (E == 1) return make_float2(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u));
    else return make_float2(__uint_as_float(w[2 * p]), __uint_as_float(w[2 * p + 1]));
  }

  // rows [e0, e1) of the block from src (row 0's address; rows outside are
  // not read).  Full: all of them.
  template <bool Full>
  __device__ __forceinline__ static void load_rows(uint32_t* w, const T* src, long long ss, int which, int e0, int e1, int tid) {
    // 32-byte loads where the rows are 32-byte aligned
    const bool wide = ((reinterpret_cast<uintptr_t>(src) | static_cast<uintptr_t>(ss * static_cast<long long>(sizeof(T)))) & 31u) == 0;
    if (which == 0) {
#pragma unroll
      for (int i = 0; i < UK; ++i) {
        const int u = tid + i * TPJ, r = k_row(u);
        const bool on = Full || (r >= e0 && r < e1);
        const T* p = src + r * ss + k_piece(u) * 16;
        if (Full && wide) {
#pragma unroll
          for (int e = 0; e < E; ++e) load32(w + (i * E + e) * 8, p + e * (16 / E));
        } else {
#pragma unroll
          for (int e = 0; e < 2 * E; ++e) {
            const uint4 x = on ? reinterpret_cast<const uint4*>(p)[e] : make_uint4(0, 0, 0, 0);
            uint32_t* o = w + i * 8 * E + 4 * e;
            o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < UV; ++i) {
        const int u = tid + i * TPJ, t0 = v_tok(u);
        const T* p = src + t0 * ss + v_dim(u);
#pragma unroll
        for (int t = 0; t < 16; ++t, p += ss) {
          const bool on = Full || (t0 + t >= e0 && t0 + t < e1);
          uint32_t* o = w + (i * 16 + t) * E;
          if constexpr (E == 1) {
            o[0] = on ? *reinterpret_cast<const uint32_t*>(p) : 0u;
          } else {
            const uint2 x = on ? *reinterpret_cast<const uint2*>(p) : make_uint2(0, 0);
            o[0] = x.x; o[1] = x.y;
          }
        }
      }
    }
  }
  __device__ __forceinline__ static void load(uint32_t* w, const T* src, long long ss, int which, int e0, int e1, int tid) {
    if (e0 == 0 && e1 == B) load_rows<true>(w, src, ss, which, e0, e1, tid);
    else load_rows<false>(w, src, ss, which, e0, e1, tid);
  }

  // the largest magnitude, as fp32 bits (integer order is magnitude order);
  // 0x7f800000 and above: something is infinite or NaN
  __device__ __forceinline__ static uint32_t top(const uint32_t* w) {
    uint32_t m = 0;
    if constexpr (E == 1) {
#pragma unroll
      for (int i = 0; i < Words; ++i)
        asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %1;\n\tmax.NaN.bf16x2 %0, %0, t;\n\t}" : "+r"(m) : "r"(w[i]));
      return max(m & 0xffff0000u, m << 16);
    } else {
#pragma unroll
      for (int i = 0; i < Words; ++i) m = max(m, w[i] & 0x7fffffffu);
      return m;
    }
  }
  __device__ __forceinline__ static uint32_t top_finite(const uint32_t* w) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < Words / E; ++p) {
      const float2 f = pair(w, p);
      const uint32_t a = __float_as_uint(f.x) & 0x7fffffffu, b = __float_as_uint(f.y) & 0x7fffffffu;
      m = max(m, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
    }
    return m;
  }

  // four K codes, or two tokens' codes of V's two dimensions, of whole rows
  // under a power-of-two scale
  __device__ __forceinline__ static uint32_t code2(const uint32_t* w, int p, float inv) {
    const float2 f = __fmul2_rn(pair(w, p), make_float2(inv, inv));
    return e4m3_pack2(f.x, f.y);
  }
  // codes of a block that is all new
  __device__ __forceinline__ static void store_full(const uint32_t* w, uint8_t* dst, float sc, int which, int tid) {
    const float inv = 1.f / sc;   // exact for a power of two
    if (which == 0) {
#pragma unroll
      for (int i = 0; i < UK; ++i) {
        const int u = tid + i * TPJ;
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          o[e] = __byte_perm(code2(w + i * 8 * E, 2 * e, inv), code2(w + i * 8 * E, 2 * e + 1, inv), 0x5410);
        reinterpret_cast<uint4*>(dst)[u] = make_uint4(o[0], o[1], o[2], o[3]);   // units lie in the block's order
      }
    } else {
#pragma unroll
      for (int i = 0; i < UV; ++i) {
        const int u = tid + i * TPJ;
        uint32_t a[4], b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t* x = w + (i * 16 + 4 * t) * E;
          const uint32_t p = __byte_perm(code2(x, 0, inv), code2(x, 1, inv), 0x5140);   // t0 t1 of j, of j + 1
          const uint32_t q = __byte_perm(code2(x, 2, inv), code2(x, 3, inv), 0x5140);
          a[t] = __byte_perm(p, q, 0x5410);
          b[t] = __byte_perm(p, q, 0x7632);
        }
        store32(dst + 32 * static_cast<size_t>(u), a, b);
      }
    }
  }
  // codes of rows [e0, e1) read again from src, under any scale sc; with
  // grow, the rows [0, e0) held, too, whose scale was smaller by ratio.  At
  // most two blocks of an append go here: kept out of the other path's way.
  __device__ __noinline__ static void store_part(const T* src, long long ss, uint8_t* dst, float sc, bool grow, float ratio,
                                                 int which, int e0, int e1, int tid) {
    const float inv = 1.f / sc;
    const bool pow2 = is_pow2(sc);
    auto one = [&](const T* p) {
      const float x = Ty<T>::to_f(p[0]), y = Ty<T>::to_f(p[1]);
      // a partly filled block the caller made may have another scale: divide
      return pow2 ? e4m3_pack2(x * inv, y * inv) : e4m3_pack2(x / sc, y / sc);
    };
    if (which == 0) {
      for (int u = tid; u < B * D / 16; u += TPJ) {
        const int r = k_row(u);
        if (r >= e1 || (r < e0 && !grow)) continue;
        uint4* d = reinterpret_cast<uint4*>(dst) + u;
        if (r < e0) {
          const uint4 o = *d;
          *d = make_uint4(rescale4(o.x, ratio), rescale4(o.y, ratio), rescale4(o.z, ratio), rescale4(o.w, ratio));
        } else {
          const T* p = src + r * ss + k_piece(u) * 16;
          uint32_t o[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) o[e] = one(p + 4 * e) | (one(p + 4 * e + 2) << 16);
          *d = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    } else {
      // bytes of tokens that are neither held nor new stay as they are
      for (int u = tid; u < B * D / 32; u += TPJ) {
        const int t0 = v_tok(u), j = v_dim(u);
        if (t0 >= e1 || (t0 + 16 <= e0 && !grow)) continue;
        uint4* d = reinterpret_cast<uint4*>(dst) + 2 * u;
        uint4 oa = d[0], ob = d[1];
        uint32_t* a = reinterpret_cast<uint32_t*>(&oa);
        uint32_t* b = reinterpret_cast<uint32_t*>(&ob);
#pragma unroll
        for (int t = 0; t < 16; ++t) {
          const int r = t0 + t, sh = (t & 3) * 8;
          if (r >= e0 && r < e1) {
            put_codes(&a[t >> 2], &b[t >> 2], t & 3, one(src + r * ss + j));
          } else if (r < e0 && grow) {
            const uint32_t old = ((a[t >> 2] >> sh) & 0xffu) | (((b[t >> 2] >> sh) & 0xffu) << 8);
            put_codes(&a[t >> 2], &b[t >> 2], t & 3, rescale2(old, ratio));
          }
        }
        d[0] = oa;
        d[1] = ob;
      }
    }
  }
};

// Group of TPJ threads = a run of `per` blocks of a pair's K or V, the next
// block's rows loading while the current block is quantised (without that
// every block pays its loads' latency, which bounds a CTA per block).
// k_append_count moves the token counts after.  Measured, 8 heads of 128 in
// bf16, blocks of 64: four prompts of up to 16,000 tokens, 39,600 in all (243 MB read and written),
// 45 us, 5.4 TB/s; four full ones (393 MB) 65 us, 6.0 TB/s.  A CTA per block took 84 us,
// one load per element and the next block's loads in flight 66, a path of
// its own for whole new blocks 48.5, 32-byte accesses 45.
template <typename T, int D, int B>
__global__ void __launch_bounds__((Ap<T, D, B>::NT), (Ap<T, D, B>::MinCtas))
k_append_many(const __grid_constant__ AppendArgs a, int per, int nrun) {
  typedef Ap<T, D, B> A;
  constexpr int NW = (A::TPJ + 31) / 32;
  __shared__ uint32_t red[2][A::NT / 32];
  __shared__ int2 s_range[A::NT / A::TPJ];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int grp = threadIdx.x / A::TPJ, tid = threadIdx.x % A::TPJ, warp = threadIdx.x >> 5;
  const uint32_t job = blockIdx.x * (A::NT / A::TPJ) + grp;   // 2 pairs nrun < 2^32
  const uint32_t pw = job / static_cast<uint32_t>(nrun);
  const int run = static_cast<int>(job - pw * static_cast<uint32_t>(nrun));
  const int which = static_cast<int>(pw & 1u), pair = static_cast<int>(pw >> 1);
  if (pair >= a.c.pairs) return;
  const CacheDev& c = a.c;
  // one thread reads the counts, so that the group agrees on them whatever
  // else happens to the cache
  if (tid == 0) append_range(a, pair, &s_range[grp].x, &s_range[grp].y);
  if (NW > 1) tc::named_sync(1 + grp, A::TPJ);
  else __syncwarp();
  const int n0 = s_range[grp].x, end = s_range[grp].y;
  constexpr int S = B == 16 ? 4 : B == 32 ? 5 : B == 64 ? 6 : 7;
  int blk = (n0 >> S) + run * per;
  const int last = min(blk + per, (end + B - 1) >> S);   // blocks [blk, last)
  if (blk >= last) return;
  const int seq = pair / c.h_kv, head = pair - seq * c.h_kv;
  const T* src = which ? static_cast<const T*>(a.v) + seq * a.vb + head * a.vh
                       : static_cast<const T*>(a.k) + seq * a.kb + head * a.kh;
  const long long ss = which ? a.vs : a.ks;
  src -= static_cast<long long>(n0) * ss;               // the pair's token 0
  auto all_max = [&](uint32_t m, int turn) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (NW > 1) {
      if ((tid & 31) == 0) red[turn][warp] = m;
      tc::named_sync(1 + grp, A::TPJ);
      m = __reduce_max_sync(0xffffffffu, red[turn][grp * NW + (tid & (NW - 1))]);
    }
    return m;
  };
  uint32_t w[A::Words], nx[A::Words];
  int id = cache_block_or_none(c, pair, blk);
  A::load(nx, src + static_cast<long long>(blk) * B * ss, ss, which, max(n0 - blk * B, 0), min(end - blk * B, B), tid);
  for (int turn = 0; blk < last; ++blk, turn ^= 1) {
    const int e0 = max(n0 - blk * B, 0), e1 = min(end - blk * B, B);
#pragma unroll
    for (int i = 0; i < A::Words; ++i) w[i] = nx[i];
    int id_next = 0;
    if (blk + 1 < last) {
      id_next = cache_block_or_none(c, pair, blk + 1);
      A::load(nx, src + static_cast<long long>(blk + 1) * B * ss, ss, which, 0, min(end - (blk + 1) * B, B), tid);
    }
    // a block whose id is out of range is dropped: its loads and barriers are
    // everyone's, its stores nobody's
    float* scale = (which ? c.vs : c.ks) + id;
    const float was = e0 > 0 && id >= 0 ? *scale : 0.f;
    // two reductions of one block use both halves of red; the next block's
    // first one, `turn` later, is behind another barrier of the group
    uint32_t m = all_max(A::top(w), turn);
    if (m >= 0x7f800000u) {
      tc::named_sync(1 + grp, A::TPJ);
      m = all_max(A::top_finite(w), turn ^ 1);
      tc::named_sync(1 + grp, A::TPJ);
    }
    // (a caller's own scale may be negative: held codes then change sign)
    const float sc = fmaxf(cache_scale_of(__uint_as_float(m)), fabsf(was));
    const bool grow = e0 > 0 && sc != was;
    if (NW == 1) __syncwarp();   // every lane has read the old scale
    if (tid == 0) {
      if (id >= 0) *scale = sc;
      if (which == 0 && e0 == 0 && c.weight) c.weight[static_cast<size_t>(pair) * c.max_blocks + blk] = 0.f;
    }
    uint8_t* dst = (which ? c.vc : c.kc) + static_cast<size_t>(id) * (D * B);
    if (e0 == 0 && e1 == B && id >= 0) A::store_full(w, dst, sc, which, tid);
    else A::store_part(src + static_cast<long long>(blk) * B * ss, ss, dst, sc, grow, was / sc, which, e0, id < 0 ? 0 : e1, tid);
    id = id_next;
  }
}

__global__ void __launch_bounds__(kApThreads) k_append_count(const __grid_constant__ AppendArgs a) {
  tc::grid_dep_wait();
  const int pair = blockIdx.x * kApThreads + threadIdx.x;
  if (pair >= a.c.pairs) return;
  int n0, end;
  append_range(a, pair, &n0, &end);
  a.c.n_tok[pair] = end;
}

// One new token: a warp for a pair's K, one for its V, lane = D/32 adjacent
// dimensions.  Only where the token needs a larger scale does the warp pass over
// the block's codes.  Three dependent loads (count, table, scale) bound it: 384 pairs about 3 us.
template <typename T, int D>
__global__ void __launch_bounds__(kApThreads) k_append_one(const __grid_constant__ AppendArgs a) {
  constexpr int N = D / 32;
  tc::grid_dep_wait();
  const CacheDev& c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, which = warp & 1;
  const int pair = blockIdx.x * (kApThreads / 64) + (warp >> 1);
  int n0 = 0, end = 0;
  if (pair < c.pairs) {
    const int seq = pair / c.h_kv, head = pair - seq * c.h_kv;
    const T* src = which ? static_cast<const T*>(a.v) + seq * a.vb + head * a.vh
                         : static_cast<const T*>(a.k) + seq * a.kb + head * a.kh;
    // the row is there whatever the counts say, except where lens gives the
    // sequence no token
    float x[N] = {};
    const bool any = !a.lens || a.lens[seq] > 0;
    if (any) {
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = Ty<T>::to_f(src[lane * N + e]);
    }
    if (lane == 0) append_range(a, pair, &n0, &end);
    n0 = __shfl_sync(0xffffffffu, n0, 0);
    end = __shfl_sync(0xffffffffu, end, 0);
    const int blk = n0 >> c.shift, e0 = n0 - (blk << c.shift);
    const int id = end > n0 ? cache_block_or_none(c, pair, blk) : -1;
    if (id >= 0) {   // (a token for a block whose id is out of range is dropped)
      uint8_t* dst = (which ? c.vc : c.kc) + static_cast<size_t>(id) * (D << c.shift);
      float* scale = (which ? c.vs : c.ks) + id;
      const float was = e0 > 0 ? *scale : 0.f;
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < N; ++e) m = max(m, __float_as_uint(finite_abs(x[e])));
      m = __reduce_max_sync(0xffffffffu, m);
      const float sc = fmaxf(cache_scale_of(__uint_as_float(m)), fabsf(was));
      if (e0 > 0 && sc != was) {
        const float ratio = was / sc;
        for (int u = lane; u < (D << c.shift) / 16; u += 32) {
          // 16 bytes: one row of K, 16 tokens of V
          const int r = which ? (u / D) << 4 : (u / (D / 2) << 3) + (u & 7);
          if (r >= e0) continue;
          uint4* w = reinterpret_cast<uint4*>(dst) + u;
          const uint4 o = *w;
          const uint32_t in[4] = {o.x, o.y, o.z, o.w};
          uint32_t y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = rescale4(in[e], ratio);
            const int left = which ? e0 - r - 4 * e : 4;   // tokens of this word that are held
            if (left < 4) {
              const uint32_t keep = left <= 0 ? 0u : (1u << (8 * left)) - 1u;
              y[e] = (y[e] & keep) | (in[e] & ~keep);
            }
          }
          *w = make_uint4(y[0], y[1], y[2], y[3]);
        }
      }
      __syncwarp();
      const float inv = 1.f / sc;
      const bool pow2 = is_pow2(sc);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const uint32_t c2 = pow2 ? e4m3_pack2(x[e] * inv, x[e + 1] * inv) : e4m3_pack2(x[e] / sc, x[e + 1] / sc);
        const int j = lane * N + e;
        if (which == 0) {
          *reinterpret_cast<uint16_t*>(dst + (e0 >> 3) * (8 * D) + (j >> 4) * 128 + (e0 & 7) * 16 + (j & 15)) =
              static_cast<uint16_t>(c2);
        } else {
          uint8_t* w = dst + (e0 >> 4) * (16 * D) + j * 16 + (e0 & 15);
          w[0] = static_cast<uint8_t>(c2);
          w[16] = static_cast<uint8_t>(c2 >> 8);
        }
      }
      if (lane == 0) *scale = sc;
    }
    if (lane == 0 && which == 0 && end > n0 && e0 == 0 && c.weight)
      c.weight[static_cast<size_t>(pair) * c.max_blocks + blk] = 0.f;
  }
  __syncthreads();   // both warps of a pair have read its count
  if (pair < c.pairs && which == 0 && lane == 0) c.n_tok[pair] = end;
}

template <typename T, int D, int B>
static cudaError_t append_many(const AppendArgs& a, cudaStream_t st) {
  typedef Ap<T, D, B> A;
  const long long touched = (static_cast<long long>(a.s) + B - 1) / B + 1;
  const int nblk = static_cast<int>(touched < a.c.max_blocks ? touched : a.c.max_blocks);
  // runs of up to 8 blocks as long as about 1200 groups are left.  Measured,
  // four full prompts of 16,000 tokens: 67 us, one block per run 82 us; four
  // ragged ones of up to 4000: 14.7 us, with 4096 groups 19.0
  const long long jobs = 2LL * a.c.pairs * nblk;
  const int per = static_cast<int>(jobs / 1200 < 1 ? 1 : jobs / 1200 > 8 ? 8 : jobs / 1200);
  const int nrun = (nblk + per - 1) / per;
  const long long groups = 2LL * a.c.pairs * nrun, gpc = A::NT / A::TPJ;
  cudaError_t e = launch_pdl(k_append_many<T, D, B>, dim3(static_cast<unsigned>((groups + gpc - 1) / gpc)),
                             dim3(A::NT), 0, st, a, per, nrun);
  if (e == cudaSuccess)
    e = launch_pdl(k_append_count, dim3((a.c.pairs + kApThreads - 1) / kApThreads), dim3(kApThreads), 0, st, a);
  return e;
}

template <typename T, int D>
static cudaError_t append_t(const AppendArgs& a, cudaStream_t st) {
  // one token, 384 pairs: 4.1 us with the count's copy, 9.6 through the other path
  if (a.s == 1) {
    constexpr int ppc = kApThreads / 64;   // pairs per CTA
    return launch_pdl(k_append_one<T, D>, dim3((a.c.pairs + ppc - 1) / ppc), dim3(kApThreads), 0, st, a);
  }
  switch (a.c.shift) {
    case 4: return append_many<T, D, 16>(a, st);
    case 5: return append_many<T, D, 32>(a, st);
    case 6: return append_many<T, D, 64>(a, st);
    default: return append_many<T, D, 128>(a, st);
  }
}

// ------------------------------------------------------------------ evict
constexpr int kEvMax = 16384;   // blocks per pair

// CTA = pair; thread t holds the entries t, t + NT, ... in registers (so the
// tables may be rewritten in place).  Weights become
// order-preserving keys, protected blocks the largest; the `keep`-th largest
// key is found two bits at a time by counting over the block (one barrier a step, ending
// as soon as some prefix has exactly `keep` keys above it), and every block's
// new place from ballots.  A few microseconds of latency bound it, whatever the size:
// measured, 8 pairs of 63 blocks 2.5 us, 64 pairs of 2049 blocks 7.1 us (8.8 and
// 13.3 with a radix select in shared memory).
template <int NT, int R>
__global__ void __launch_bounds__(NT)
k_evict(const __grid_constant__ CacheDev c, int32_t* table, int32_t* n_tok, float* weight, int32_t* kept, int keep,
        int sink, int recent) {
  constexpr int NW = NT / 32;
  __shared__ uint2 s_cnt[2][NW];
  __shared__ int s_pre[R * NW];
  __shared__ int s_tok;
  tc::grid_dep_wait();
  const int mb = c.max_blocks, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x;
  const size_t row = static_cast<size_t>(pair) * mb;
  // the weights, as keys; what the tables hold is read once more below
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + r * NT;
    key[r] = i < mb ? __float_as_uint(c.weight[row + i]) : 0u;
  }
  if (tid == 0) s_tok = cache_tokens(c, pair);
  __syncthreads();
  const int tok = s_tok;
  const int B = 1 << c.shift, n = (tok + B - 1) >> c.shift;
  const int nk = min(n, keep);
  const int rows = (n + NT - 1) / NT;   // registers in use: the same for every thread
  // 0: no block (never chosen); 1: NaN, below every number; -0 as 0
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + r * NT;
    const float w = __uint_as_float(key[r]);
    key[r] = i >= n ? 0u : i < sink || i >= n - recent ? 0xffffffffu : w == w ? order_key(w + 0.f) : 1u;
  }
  // sums over the block of three counts of at most 16384 each
  int turn = 0;
  auto count3 = [&](uint32_t c1, uint32_t c2, uint32_t c3) {
    const uint32_t a = __reduce_add_sync(0xffffffffu, c1 | (c2 << 16)), b = __reduce_add_sync(0xffffffffu, c3);
    if (lane == 0) s_cnt[turn][warp] = make_uint2(a, b);
    __syncthreads();
    const uint2 v = lane < NW ? s_cnt[turn][lane] : make_uint2(0, 0);
    turn ^= 1;
    const uint32_t t = __reduce_add_sync(0xffffffffu, v.x);
    return make_int3(t & 0xffffu, t >> 16, __reduce_add_sync(0xffffffffu, v.y));
  };
  // exclusive prefix, in index order, of one flag per block
  auto prefix = [&](uint32_t flags, int* out) {
    uint32_t bal[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      bal[r] = __ballot_sync(0xffffffffu, (flags >> r) & 1u);
      if (lane == 0) s_pre[r * NW + warp] = __popc(bal[r]);
    }
    __syncthreads();
    if (warp == 0) {
      int run = 0;
      for (int e0 = 0; e0 < R * NW; e0 += 32) {
        const int v = e0 + lane < R * NW ? s_pre[e0 + lane] : 0;
        int x = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += y;
        }
        if (e0 + lane < R * NW) s_pre[e0 + lane] = run + x - v;
        run += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) out[r] = s_pre[r * NW + warp] + __popc(bal[r] & ((1u << lane) - 1u));
    __syncthreads();   // s_pre may be written again
  };

  uint32_t stay = 0;   // bit r: block tid + r NT is kept
  if (n > keep) {
    uint32_t T = 0;
    int ge = n;   // keys >= T
    for (int sh = 30; sh >= 0 && ge != keep; sh -= 2) {
      uint32_t c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r >= rows) break;
        const uint32_t k = key[r];
        c1 += k >= (T | (1u << sh));
        c2 += k >= (T | (2u << sh));
        c3 += k >= (T | (3u << sh));
      }
      const int3 s = count3(c1, c2, c3);
      if (s.z >= keep) { T |= 3u << sh; ge = s.z; }
      else if (s.y >= keep) { T |= 2u << sh; ge = s.y; }
      else if (s.x >= keep) { T |= 1u << sh; ge = s.x; }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) stay |= (key[r] >= T && key[r] != 0u ? 1u : 0u) << r;
    if (ge != keep) {
      // more keys equal T than fit: those of the lowest index
      uint32_t eq = 0, gt = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        eq |= (key[r] == T ? 1u : 0u) << r;
        gt += key[r] > T;
      }
      const int need = keep - count3(gt, 0, 0).x;
      int at[R];
      prefix(eq, at);
#pragma unroll
      for (int r = 0; r < R; ++r)
        if (((eq >> r) & 1u) && at[r] >= need) stay &= ~(1u << r);
    }
  } else {
#pragma unroll
    for (int r = 0; r < R; ++r) stay |= (tid + r * NT < n ? 1u : 0u) << r;
  }
  int32_t id[R];
  float w[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + r * NT;
    id[r] = i < mb ? c.table[row + i] : 0;
    w[r] = i < mb ? c.weight[row + i] : 0.f;
  }
  int at[R];
  prefix(stay, at);   // its barriers also stand between every read and write of the tables
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int i = tid + r * NT;
    if (i >= mb) continue;
    const bool s = (stay >> r) & 1u;
    const int to = i >= n ? i : s ? at[r] : nk + i - at[r];   // kept, then freed, then the rest
    table[row + to] = id[r];
    weight[row + to] = s ? w[r] : 0.f;
    if (s && kept) kept[static_cast<size_t>(pair) * keep + to] = i;
    if (i == n - 1) n_tok[pair] = s ? (nk - 1) * B + tok - (n - 1) * B : nk * B;
  }
  if (n == 0 && tid == 0) n_tok[pair] = 0;
  if (kept)
    for (int i = nk + tid; i < keep; i += NT) kept[static_cast<size_t>(pair) * keep + i] = -1;
}

static cudaError_t launch_evict(const shadowkv_cache& src, const shadowkv_cache& dst, int keep, int sink, int recent,
                                int32_t* kept, cudaStream_t st) {
  auto go = [&](auto kern, int nt) {
    return launch_pdl(kern, dim3(src.b * src.h_kv), dim3(nt), 0, st, cache_dev(src), dst.table, dst.n_tok, dst.weight, kept,
                      keep, sink, recent);
  };
  const int mb = src.max_blocks;
  if (mb <= 256) return go(k_evict<256, 1>, 256);
  if (mb <= 1024) return go(k_evict<1024, 1>, 1024);
  if (mb <= 4096) return go(k_evict<1024, 4>, 1024);
  return go(k_evict<1024, 16>, 1024);
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
  if (reinterpret_cast<uintptr_t>(c->k_codes) % 32 || reinterpret_cast<uintptr_t>(c->v_codes) % 32)
    return "cache: codes must be 32-byte aligned";
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

// Rows read 16 bytes at a time, of b sequences, h heads and s tokens (the stride
// of a single one is not looked at).
const char* rows16_fault(const shadowkv_rows* r, int b, int h, int s, int E) {
  if (!r || !r->ptr) return "k and v must be non-NULL";
  const long long sb = b > 1 ? r->sb : 0, sh = h > 1 ? r->sh : 0, ss = s > 1 ? r->ss : 0;
  if (sb < 0 || sh < 0 || ss < 0) return "row strides must not be negative";
  if (reinterpret_cast<uintptr_t>(r->ptr) % 16 || (sb * E) % 16 || (sh * E) % 16 || (ss * E) % 16)
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
std::mutex& cache_enqueue() {
  static std::mutex m;
  return m;
}
}  // namespace skv

extern "C" {

skv_status shadowkv_cache_validate(const shadowkv_cache* c) try {
  return skv::cache_checked(c);
} catch (...) {   // host memory for an error text ran out
  return SKV_ERR_OOM;
}

skv_status shadowkv_cache_append(const shadowkv_cache* c, int dtype, const shadowkv_rows* k, const shadowkv_rows* v,
                                 int s, const int32_t* lens, void* stream) try {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (dtype != SKV_DTYPE_F32 && dtype != SKV_DTYPE_BF16) return set_error(SKV_ERR_INVALID_ARG, "bad dtype");
  if (s < 0) return set_error(SKV_ERR_INVALID_ARG, "s must be >= 0");
  if (s == 0) return SKV_OK;
  const int E = dtype == SKV_DTYPE_BF16 ? 2 : 4;
  const char* f = rows16_fault(k, c->b, c->h_kv, s, E);
  if (!f) f = rows16_fault(v, c->b, c->h_kv, s, E);
  if (!f && reinterpret_cast<uintptr_t>(lens) % 4) f = "lens must be 4-byte aligned";
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  skv::AppendArgs a;
  a.c = skv::cache_dev(*c);
  a.k = k->ptr; a.kb = k->sb; a.kh = k->sh; a.ks = k->ss;
  a.v = v->ptr; a.vb = v->sb; a.vh = v->sh; a.vs = v->ss;
  a.lens = lens;
  a.s = s;
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  cudaError_t e;
  if (dtype == SKV_DTYPE_BF16)
    e = c->d == 128 ? skv::append_t<skv::bf16, 128>(a, q) : skv::append_t<skv::bf16, 64>(a, q);
  else
    e = c->d == 128 ? skv::append_t<float, 128>(a, q) : skv::append_t<float, 64>(a, q);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

skv_status shadowkv_cache_evict(const shadowkv_cache* src, const shadowkv_cache* dst, int keep, int sink, int recent,
                                int32_t* kept, void* stream) try {
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
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  const cudaError_t e = skv::launch_evict(*src, *dst, keep, sink, recent, kept, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

skv_status shadowkv_cache_check(const shadowkv_cache* c) try {
  using skv::set_error;
  skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  int word = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpy(&word, c->status, sizeof(int), cudaMemcpyDeviceToHost);
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  if (word == skv::DEV_TIMEOUT) return set_error(SKV_ERR_TIMEOUT, "a bounded device wait gave up");
  if (word == skv::DEV_BAD_SEQUENCE)
    return set_error(SKV_ERR_DEVICE_CHECK, "a call met a sequence number out of range or named twice");
  if (word == skv::DEV_POOL_FULL) return set_error(SKV_ERR_DEVICE_CHECK, "the pool has fewer blocks than are in use");
  if (word) return set_error(SKV_ERR_DEVICE_CHECK, "a kernel met a block id, length or token count out of range");
  return SKV_OK;
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
