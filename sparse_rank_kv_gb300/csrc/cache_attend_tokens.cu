// Attention of several tokens per sequence over the 8-bit block cache
// (shadowkv_cache_attend_tokens): a piece of a prompt, drafted tokens, or queries
// over an encoder's states.
//
// Rows: the queries of a sequence and the G query heads of a KV head together, row
// r = query r / G, head r % G; a tile of 128 rows is the M of the tensor core's
// products, 128 tokens are their N (S = Q K^T) and K (O += P V).  The codes become fp16 on
// their way (exact: e4m3 has 4 bits and fp16 more range), their scales go to the
// logits and to p in fp32.  A bf16 query row is exact in fp16 after division by the power
// of two of its largest entry (entries down to 2^-31 of it, the others to 2^-39 of it); an fp32
// row, and p times its V scale beside both, are sums of two fp16 terms (2^-22 of themselves).  p's are relative to
// the largest scale so far and good to 2^-36 of the largest: p is at most 2^4 (the running maximum is only raised where
// a tile passes it by more than 4 in base 2, so that O is rarely rescaled).  One term of p, 2^-11 of itself, would
// show in bf16 where values cancel, and took a prompt of 16,384 tokens 2.23 ms in place of 2.45.
//
// All row tiles and the tiles (of 128 tokens) that each sees are numbered through in units, five for a row tile's start
// and end and one for each of its tiles, and every CTA takes an equal run of units: one prompt, ragged batches and few rows over
// a long cache fill the GPU alike.  A row tile that several CTAs work on is joined by k_tokens_merge.
//
// Measured, 32 query and 8 KV heads of 128 in bf16: a prompt of 16,384 tokens 2.45 ms, 899 TFLOP/s (0.46 of a
// cuBLAS product's rate; the products with V run once for each term of p, and that is counted once); 6 tokens over
// 8 x 131,072 538 us, 4.0 TB/s of codes.  What bounds it: the chain S -> softmax -> P -> O of a stream (with one term of p 2300
// cycles of softmax and 500 of waits between warps beside 2200 of products for two streams); the shared memory, which
// the products' operands, the codes and their fp16 forms share; and at a row tile's start and end about 20,000 cycles.
#include <cuda_fp16.h>

#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

constexpr int kCtT = 128;       // tokens of a tile, rows of an MMA
constexpr int kCtThreads = 576; // warps 0-3 and 4-7: softmax of stream 0 and 1; 8-11 and 12-15: conversion of K and of V; 16: copies; 17: tcgen05.mma
constexpr int kCtInfo = 8;      // tiles described ahead
constexpr int kCtBatch = 8;     // pieces that a conversion thread has in flight (2 and 4: 1 to 3% slower)

struct TokensArgs {
  CacheDev c;
  const void* q;
  void* out;
  float* lse;
  const int32_t* lens;
  int4* rec;          // [ctas]: row tile in whose midst the CTA's run begins (pair, tile, its first unit, all units), pair -1: none
  float* part_o;      // [2 ctas][Rows][d]
  float2* part_ml;    // [2 ctas][Rows]
  uint32_t* nan;      // [ctas][3][128][4]
  long long qb, qh, qs, ob, oh, os;
  float scale_log2, scale_rest;   // scale log2(e), and what its rounding leaves over it
  int s, h_q, G, causal, wide_q, wide_o;   // wide: rows in 16-byte pieces
};

__device__ __forceinline__ int tokens_len(const TokensArgs& a, int seq) {
  const int n = a.lens ? a.lens[seq] : a.s;
  if (static_cast<unsigned>(n) <= static_cast<unsigned>(a.s)) return n;
  flag_error(a.c.status, DEV_BAD_COUNT);
  return n < 0 ? 0 : a.s;
}
// Tokens query j of `len` sees of the n held.
__device__ __forceinline__ int tokens_seen(const TokensArgs& a, int n, int len, int j) {
  return a.causal ? max(n - len + j + 1, 0) : n;
}

// One of bf16's or fp32's forms.  Two: a CTA works on two row tiles with the same tokens at a
// time (stream 0 and 1); else on one, whose tokens' tiles the streams take in turn.  Copies = 4: at most
// 32 rows, which stand in the MMA's rows four times, so that each of the softmax's warps takes 32 of a tile's 128 columns (its
// P is zero elsewhere) and has sums of its own.
template <typename T, int D, bool Two, int Copies>
struct Ct {
  static constexpr int NQ = sizeof(T) == 2 ? 1 : 2;        // fp16 terms of q
  static constexpr int NP = 2;                             // and of p
  static constexpr int Rows = (Two ? 256 : 128) / Copies;
  static constexpr int PartRows = Two ? 256 : 128;          // rows of a part, copies and all
  static constexpr int QT = kCtT * D * 2;                   // an operand tile in fp16
  static constexpr int QB = (Two ? 2 : NQ) * QT;
  static constexpr int KB = kCtT * D;                       // codes of K or of V: a stage
  static constexpr int Misc = 2928;
  static constexpr int Most = 227 * 1024 - 128 - Misc;
  static constexpr int NST0 = (Most - QB - 4 * QT) / KB, NST = NST0 > 8 ? 8 : NST0;
  static constexpr int Smem = 128 + QB + 4 * QT + NST * KB + Misc;
  static_assert(NST >= 2 && NST % 2 == 0 && !(Two && (NQ > 1 || Copies > 1)), "tile");
};

// ------------------------------------------------------------ tensor core
// D (+)= A B^T, fp16, A in TMEM (lane = row, two elements of K to a column)
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// kind::f16, fp16 A and B (format 0), fp32 D, both K-major, M = 128
constexpr uint32_t idesc_f16(int N) { return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24); }

// One lane of the warp (the compiler knows that one thread runs what depends on it, and keeps
// descriptors in uniform registers: the eight products of a tile are issued in half the time of `lane == 0`)
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {   // 2^-22 relative; results below 2^-126 are 0
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float lg2(float x) {   // of a normal number: within 2^-22
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Two numbers as a pair, each rounded as by itself
__device__ __forceinline__ unsigned long long pair_of(float2 a) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
  return r;
}
__device__ __forceinline__ float2 of_pair(unsigned long long a) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)), "l"(pair_of(c)));
  return of_pair(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pair_of(a)), "l"(pair_of(b)));
  return of_pair(r);
}
// The two fp16 terms of two numbers: each to the nearest, then what it leaves over (exact in fp32; -1 times the fp16
// number as it is, in place of two conversions back and two sums: a prompt of 16,384 2.63 -> 2.44 ms).
__device__ __forceinline__ void terms2(float2 p, uint32_t* first, uint32_t* rest) {
  const __half2 z = __floats2half2_rn(p.x, p.y);
  *first = *reinterpret_cast<const uint32_t*>(&z);
  float x, y;
  asm("{\n\t.reg .b16 l, h, m;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "mov.b16 m, 0xBC00;\n\t"
      "fma.rn.f32.f16 %0, l, m, %3;\n\t"
      "fma.rn.f32.f16 %1, h, m, %4;\n\t}"
      : "=f"(x), "=f"(y)
      : "r"(*first), "f"(p.x), "f"(p.y));
  const __half2 w = __floats2half2_rn(x, y);
  *rest = *reinterpret_cast<const uint32_t*>(&w);
}
// e >= -110 with x < 2^e, of a largest V scale
__device__ __forceinline__ int scale_exp(float x) { return max(static_cast<int>(__float_as_uint(x) >> 23) - 126, -110); }
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// ------------------------------------------------------------ the tiles in order
// A run of tiles: row tile q of a pair, its tiles from `tile` on.
struct Walk {
  int pair, q, tile, left;
  int n, len, nq, nt, seen0;   // of the pair: tokens, queries, row tiles; of the row tile: tiles, tokens its first row sees
  int lim;                     // tokens its last row sees
};
template <int Rows>
__device__ __forceinline__ int row_tiles(const TokensArgs& a, int len) { return (len * a.G + Rows - 1) / Rows; }
// Tokens that row tile q sees (its last row), and its tiles: one at least, so that rows that see nothing are written.
template <int Rows>
__device__ __forceinline__ int tile_lim(const TokensArgs& a, int n, int len, int q) {
  return tokens_seen(a, n, len, min(len - 1, (q * Rows + Rows - 1) / a.G));
}
__device__ __forceinline__ int lim_tiles(int lim) { return max(1, (lim + kCtT - 1) / kCtT); }

template <int Rows>
__device__ __forceinline__ void walk_item(const TokensArgs& a, Walk& w) {
  w.lim = tile_lim<Rows>(a, w.n, w.len, w.q);
  w.seen0 = tokens_seen(a, w.n, w.len, w.q * Rows / a.G);
  w.nt = lim_tiles(w.lim);
}
template <int Rows>
__device__ __forceinline__ void walk_pair(const TokensArgs& a, Walk& w) {
  w.n = cache_tokens(a.c, w.pair);
  w.len = tokens_len(a, w.pair / a.c.h_kv);
  w.nq = row_tiles<Rows>(a, w.len);
}
// To the next tile; true when it is another row tile's.
template <int Rows>
__device__ __forceinline__ bool walk_next(const TokensArgs& a, Walk& w) {
  if (--w.left <= 0) return false;
  if (++w.tile < w.nt) return false;
  w.tile = 0;
  if (++w.q >= w.nq) {
    w.q = 0;
    do {
      if (++w.pair >= a.c.pairs) { w.left = 0; return false; }
      walk_pair<Rows>(a, w);
    } while (w.nq == 0);
  }
  walk_item<Rows>(a, w);
  return true;
}

__device__ __forceinline__ int run_begin(int cta, int n, int total) {
  return static_cast<int>(static_cast<long long>(cta) * total / n);
}
__device__ __forceinline__ int run_owner(int x, int n, int total) {
  return static_cast<int>(((static_cast<long long>(x) + 1) * n - 1) / total);
}

// The runs are dealt in units: a row tile has kCtCost units for its start and end (queries laid, outputs stored:
// about as long as five tiles take), then one for each of its tiles.  Measured against tiles alone: a prompt of 2048
// 127.7 -> 88 us, of 8192 845 -> 629, of 16,384 2645 -> 2215; four pieces of up to 2048 over up to 20,001 1391 -> 1210.
//
// Where this CTA's run begins: s_where = {pair, row tile, its first tile here, all units}, s_run = {the row tile's
// first unit, tiles before the run, tiles before the next CTA's}.  Groups of 2^lg lanes take runs of pairs, a lane every
// 2^lg-th row tile.
constexpr int kCtCost = 5;
template <int Rows>
__device__ __forceinline__ void run_find(const TokensArgs& a, int cta, int ncta, int* s_where, int* s_run, int* s_scan) {
  const int tid = threadIdx.x, P = a.c.pairs, most = row_tiles<Rows>(a, a.s);
  const int lg = most <= 2 ? 0 : most <= 8 ? 2 : 5, gs = 1 << lg, sub = tid & (gs - 1);
  const int ng = kCtThreads >> lg, per = (P + ng - 1) / ng, p0 = min(P, (tid >> lg) * per), p1 = min(P, p0 + per);
  auto pair_sum = [&](int p, int* items) {   // this lane's part
    const int n = cache_tokens(a.c, p), len = tokens_len(a, p / a.c.h_kv), nq = row_tiles<Rows>(a, len);
    int x = 0;
    for (int q = sub; q < nq; q += gs) x += kCtCost + lim_tiles(tile_lim<Rows>(a, n, len, q));
    *items = sub == 0 ? nq : 0;
    return x;
  };
  auto group_sum = [&](int x) {
    for (int o = gs >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
  };
  int sum = 0, items = 0;
  for (int i = 0; i < per; ++i)
    if (p0 + i < p1) {
      int k;
      sum += pair_sum(p0 + i, &k);
      items += k;
    }
  sum = group_sum(sum);
  if (tid < 4) s_where[tid] = tid == 0 ? -1 : 0;
  if (tid < 3) s_run[tid] = 0;
  int total, all_items;
  const int scan = block_exclusive_scan(sub == 0 ? sum : 0, s_scan, &total);
  const int scan_items = block_exclusive_scan(items, s_scan, &all_items);
  const int lead = tid & 31 & ~(gs - 1);
  int before = __shfl_sync(0xffffffffu, scan, lead), items_before = __shfl_sync(0xffffffffu, scan_items, lead);
  const int n = min(ncta, total);
  const int t0 = cta < n ? run_begin(cta, n, total) : -1, t1 = cta < n ? run_begin(cta + 1, n, total) : -1;
  if (tid == 0) {
    s_where[3] = total;
    if (t1 == total) s_run[2] = total - kCtCost * all_items;
  }
  // the groups walk their pairs once more, in step within the warp
  for (int i = 0; i < per; ++i) {
    const int p = p0 + i;
    int nq = 0;
    const int mine = p < p1 ? pair_sum(p, &nq) : 0, all = group_sum(mine);
    nq = __shfl_sync(0xffffffffu, nq, lead);
    const bool here = (before <= t0 && t0 < before + all) || (before <= t1 && t1 < before + all);
    if (__any_sync(0xffffffffu, here)) {
      const int cn = p < p1 ? cache_tokens(a.c, p) : 0, len = p < p1 ? tokens_len(a, p / a.c.h_kv) : 0;
      int run = before;
      for (int q0 = 0; __any_sync(0xffffffffu, here && q0 < nq); q0 += gs) {
        const int q = q0 + sub, x = here && q < nq ? kCtCost + lim_tiles(tile_lim<Rows>(a, cn, len, q)) : 0;
        int inc = x;
        for (int o = 1; o < gs; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, inc, o);
          if (sub >= o) inc += y;
        }
        const int at = run + inc - x;   // the row tile's first unit
        const int tiles = at - kCtCost * (items_before + q);
        if (x > 0 && at <= t0 && t0 < at + x) {
          const int first = max(t0 - at - kCtCost, 0);
          s_where[0] = p;
          s_where[1] = q;
          s_where[2] = first;
          s_run[0] = at;
          s_run[1] = tiles + first;
        }
        if (x > 0 && at <= t1 && t1 < at + x) s_run[2] = tiles + max(t1 - at - kCtCost, 0);
        run += __shfl_sync(0xffffffffu, inc, tid & 31 | (gs - 1));
      }
    }
    before += all;
    items_before += nq;
  }
  __syncthreads();
}

// of a tile, beside its tokens (at most 128)
enum : int {
  kSFirst = 1024,   // first that its stream has of the row tile
  kSLast = 2048,
  kMixed = 4096,    // some rows do not see some of its tokens
  kOdd = 8192,      // a K scale that is negative, a V scale that is not positive, or one that is no number
  kWhole = 16384,   // this CTA has all of the row tile
  kKexp = 16        // (a shift) the exponent of its largest K scale, as a float holds it
};
// Logits up to this much (a row's factor times the largest K scale, by the sum of their exponents as floats hold them: with
// 2^15 448 128 of S, below 2^23) are sure to be resolved to a half: more than that is rounded before it is compared and
// subtracted, since what is left between a logit and its rounding could be any power of two.
constexpr int kLargeSum = 2 * 127 - 10;
struct TileInfo {
  int tile, flags, vexp, vlow;   // all V scales are below 2^vexp, and 2^vlow or more
  float ks[8], vs[8];            // of every 16 tokens
  int pair, q, n, len;
  int turn, end, pad[2];         // number of the row tile in this CTA; of its last tile here
};

// One row of a row tile from its parts (numbers u of n; a part's Copies sub-rows lie `step` apart): a warp's work.
template <typename T, int D, int Copies, typename At>
__device__ __forceinline__ void join_row(const TokensArgs& a, int seq, int h, int j, bool sees, int n, int step, At&& at) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31, parts = n * Copies;
  auto row_of = [&](int u) { return at(u / Copies) + u % Copies * step; };
  float M = -INFINITY;
  for (int u = lane; u < parts; u += 32) M = fmaxf(M, __ldcg(&a.part_ml[row_of(u)].x));
  M = warp_max(M);
  const float ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, o[E] = {};
  constexpr int B = Copies > 1 ? 8 : 2;   // (without copies a row has two or three parts as a rule)
  // 32 parts at a time: a lane forms one's weight, then the parts' values, B loads in flight
  for (int u0 = 0; u0 < parts; u0 += 32) {
    const float2 ml = u0 + lane < parts ? __ldcg(&a.part_ml[row_of(u0 + lane)]) : make_float2(-INFINITY, 0.f);
    const float mine = ex2(ml.x - ref);
    L = fmaf(ml.y, mine, L);
    const int k = min(32, parts - u0);
    for (int v = 0; v < k; v += B) {
      float x[B][E];
#pragma unroll
      for (int e = 0; e < B; ++e) {
        const float* src = a.part_o + row_of(u0 + min(v + e, k - 1)) * D + lane * E;
        if constexpr (E == 4) *reinterpret_cast<float4*>(x[e]) = __ldcg(reinterpret_cast<const float4*>(src));
        else *reinterpret_cast<float2*>(x[e]) = __ldcg(reinterpret_cast<const float2*>(src));
      }
#pragma unroll
      for (int e = 0; e < B; ++e) {
        const float w = __shfl_sync(0xffffffffu, mine, min(v + e, 31));
        if (v + e < k)
#pragma unroll
          for (int c = 0; c < E; ++c) o[c] = fmaf(x[e][c], w, o[c]);
      }
    }
  }
  L = warp_sum(L);
  T* dst = static_cast<T*>(a.out) + seq * a.ob + h * a.oh + j * a.os + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) dst[e] = Ty<T>::from_f(sees ? o[e] / L : 0.f);
  if (a.lse && lane == 0)
    a.lse[(static_cast<size_t>(seq) * a.h_q + h) * a.s + j] = sees ? (ref + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

template <typename T, int D, bool Two, int Copies>
__global__ void __launch_bounds__(kCtThreads, 1) k_attend_tokens(const __grid_constant__ TokensArgs a) {
  using C = Ct<T, D, Two, Copies>;
  constexpr int NST = C::NST, Rows = C::Rows;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  unsigned char* qbuf = smem;
  unsigned char* kbuf = qbuf + C::QB;                    // [2] K in fp16
  unsigned char* vbuf = kbuf + 2 * C::QT;                // [2] V
  unsigned char* stages = vbuf + 2 * C::QT;              // [NST] codes
  unsigned char* misc = stages + NST * C::KB;
  uint64_t* full = reinterpret_cast<uint64_t*>(misc);    // [8] codes are there: K and V of the tiles in turn
  uint64_t* sempty = full + 8;                           // [8] codes are converted
  uint64_t* kfull = full + 16;                           // [2]
  uint64_t* kempty = full + 18;
  uint64_t* vfull = full + 20;
  uint64_t* vempty = full + 22;
  uint64_t* sfull = full + 24;                           // [2], by stream
  uint64_t* pfull = full + 26;
  uint64_t* ofin = full + 28;                            // a row tile's last product is done
  uint64_t* qfull = full + 30;
  uint64_t* jfull = full + 32;                           // stream 1's sums are there
  uint64_t* jdone = full + 33;                           // stream 0 has joined the two
  uint64_t* ifull = full + 34;                           // [8]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(misc + 336);
  volatile int* s_abort = reinterpret_cast<volatile int*>(misc + 340);
  int* s_where = reinterpret_cast<int*>(misc + 344);     // [4]
  int* s_run = reinterpret_cast<int*>(misc + 400);       // [3]
  volatile int* s_nan = reinterpret_cast<volatile int*>(misc + 360);   // [2]: V's tile has NaN
  int* s_scan = reinterpret_cast<int*>(misc + 448);      // [32], before the tiles are described
  TileInfo* infos = reinterpret_cast<TileInfo*>(misc + 448);
  float* sqs = reinterpret_cast<float*>(misc + 1344);    // [128] rows' factors (one row tile), then stream 1's vexp
  float2* s_ml = reinterpret_cast<float2*>(misc + 1856); // [128] stream 1's maxima and sums
  int2* s_join = reinterpret_cast<int2*>(misc + 2880);   // [4 warps] whether it had tiles, and whether NaN is recorded
  // (the warps wait for one another at these, never at named barriers: a wait that gives up must not leave others behind)
  uint64_t* vote_bar = reinterpret_cast<uint64_t*>(misc + 2912);             // the conversion of V
  uint64_t* parts_bar = vote_bar + 1;                                        // stream 0, its copies' parts
  volatile int* s_vote = reinterpret_cast<volatile int*>(misc + 368);        // [2][4]
  static_assert(sizeof(TileInfo) == 112, "misc");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cta = blockIdx.x;
  if (gridDim.x > 1) tc::grid_dep_launch();   // (a call's last kernel lets nothing start early)

  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(&full[i], i & 1 ? 1 : 2);   // K's also waits for the tile's description
      tc::mbar_init(&sempty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&kfull[i], 4);
      tc::mbar_init(&kempty[i], 1);
      tc::mbar_init(&vfull[i], 4);
      tc::mbar_init(&vempty[i], 1);
      tc::mbar_init(&sfull[i], 1);
      tc::mbar_init(&pfull[i], 4);
      tc::mbar_init(&ofin[i], 1);
      tc::mbar_init(&qfull[i], 4);
    }
    tc::mbar_init(jfull, 4);
    tc::mbar_init(jdone, 4);
    for (int i = 0; i < kCtInfo; ++i) tc::mbar_init(&ifull[i], 1);
    tc::mbar_init(vote_bar, 4);
    tc::mbar_init(parts_bar, 4);
    tc::fence_mbar_init();
    *s_abort = 0;
  }
  if (warp == 17) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  tc::fence_before();
  tc::grid_dep_wait();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  run_find<Rows>(a, cta, gridDim.x, s_where, s_run, s_scan);
  const int ntile = s_where[0] >= 0 ? s_run[2] - s_run[1] : 0;
  if (tid == 0)
    a.rec[cta] = ntile > 0 && s_where[2] > 0 ? make_int4(s_where[0], s_where[1], s_run[0], s_where[3]) : make_int4(-1, 0, 0, s_where[3]);
  const int shift = a.c.shift, B = 1 << shift;
  uint32_t* nan_masks = a.nan + static_cast<size_t>(cta) * 3 * 128 * 4;
  auto abort_now = [&]() {
    *s_abort = 1;
    flag_error(a.c.status, DEV_TIMEOUT);
  };
  auto warp_wait = [&](uint64_t* bar, uint32_t phase) {
    if (__all_sync(0xffffffffu, tc::mbar_try_wait(bar, phase & 1))) return true;
    const bool ok = __all_sync(0xffffffffu, !*s_abort && tc::mbar_wait(bar, phase & 1, kWaitLimit));
    if (!ok && lane == 0) abort_now();
    return ok;
  };

  if (ntile > 0 && warp == 16) {
    // ------------------------------------------------------------ copies
    // Block ids are loaded two tiles ahead, scales one.
    Walk cur;
    cur.pair = s_where[0];
    cur.q = s_where[1];
    cur.tile = s_where[2];
    cur.left = ntile;
    walk_pair<Rows>(a, cur);
    walk_item<Rows>(a, cur);
    auto tokens = [&](const Walk& w) { return w.left > 0 ? max(0, min(kCtT, w.lim - w.tile * kCtT)) : 0; };
    auto blocks = [&](const Walk& w) { return (tokens(w) + B - 1) >> shift; };
    auto id_of = [&](const Walk& w) {
      return lane < blocks(w) ? cache_block(a.c, w.pair, ((w.tile * kCtT) >> shift) + lane) : 0;
    };
    Walk nx = cur;
    int id = id_of(cur);
    walk_next<Rows>(a, nx);
    int id1 = id_of(nx), turn = 0, seg0 = 0;   // seg0: number of the row tile's first tile here
    int whole = cur.tile == 0 && cur.left >= cur.nt ? kWhole : 0;
    int seg_end = min(ntile, cur.nt - cur.tile);
    float ks = a.c.ks[id], vs = a.c.vs[id];
    int it = 0, copied = 0;
    int st = 0;           // stage and its turn
    uint32_t ph = 1;
    auto next_stage = [&]() {
      if (++st == NST) {
        st = 0;
        ph ^= 1;
      }
    };
    // (one row tile per pair: the codes are read once and evicted first from L2)
    const bool once = row_tiles<Rows>(a, a.s) == 1;
    const uint64_t policy = tc::l2_evict_first_policy();
    auto load = [&](void* dst, const uint8_t* src) {
      if (once) tc::bulk_load_hint(dst, src, B * D, &full[st], policy);
      else tc::bulk_load(dst, src, B * D, &full[st]);
    };
    for (;; ++it) {
      const int nb = blocks(cur), cnt = tokens(cur);
      if (!warp_wait(&sempty[st], ph)) break;
      if (lane == 0) tc::mbar_expect_tx(&full[st], static_cast<uint32_t>(nb * B * D));
      __syncwarp();
      const size_t src = static_cast<size_t>(id) * (B * D);
      if (lane < nb) load(stages + st * C::KB + lane * (B * D), a.c.kc + src);
      ++copied;
      // (the stage is free: the tile kCtInfo before this one has been described to all and used)
      TileInfo* in = infos + it % kCtInfo;
      if (lane >= nb) ks = vs = 0.f;
      // largest finite V scale, as an exponent above it
      const bool odd = __any_sync(0xffffffffu, lane < nb && !(ks * a.scale_log2 >= 0.f && vs > 0.f && vs < INFINITY));
      const float least = -warp_max(lane < nb ? -fabsf(vs) : -INFINITY);
      const float top = warp_max(fabsf(vs) < INFINITY ? fabsf(vs) : 0.f);
      const uint32_t kexp = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(ks))) >> 23;   // (NaN above all)
      const int g16 = lane << 4 >> shift;   // block of 16-token group `lane`
      const float ksg = __shfl_sync(0xffffffffu, ks, g16 & 7), vsg = __shfl_sync(0xffffffffu, vs, g16 & 7);
      if (lane < 8) {
        in->ks[lane] = ksg;
        in->vs[lane] = vsg;
      }
      if (lane == 0) {
        const int k = it - seg0, stride = Two ? 1 : 2;
        in->pair = cur.pair;
        in->q = cur.q;
        in->tile = cur.tile;
        in->flags = cnt | (k < stride ? kSFirst : 0) |
                    (it >= seg_end - stride ? kSLast : 0) | (cur.tile * kCtT + cnt > cur.seen0 ? kMixed : 0) | (odd ? kOdd : 0) | whole |
                    static_cast<int>(kexp) << kKexp;
        in->n = cur.n;
        in->len = cur.len;
        in->turn = turn;
        in->end = seg_end - 1;
        in->vlow = static_cast<int>(__float_as_uint(least) >> 23) - 127;
        in->vexp = scale_exp(top);
      }
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&ifull[it % kCtInfo]);
        tc::mbar_arrive(&full[st]);
      }
      __syncwarp();
      next_stage();
      if (!warp_wait(&sempty[st], ph)) break;
      if (lane == 0) tc::mbar_expect_tx(&full[st], static_cast<uint32_t>(nb * B * D));
      __syncwarp();
      if (lane < nb) load(stages + st * C::KB + lane * (B * D), a.c.vc + src);
      ++copied;
      next_stage();
      Walk nx2 = nx;
      if (nx2.left > 0) walk_next<Rows>(a, nx2);
      const int id2 = id_of(nx2);
      const float ks1 = a.c.ks[id1], vs1 = a.c.vs[id1];
      if (nx.left <= 0) break;
      if (it + 1 == seg_end) {   // another row tile
        ++turn;
        seg0 = seg_end;
        whole = nx.left >= nx.nt ? kWhole : 0;
        seg_end = min(ntile, seg0 + nx.nt);
      }
      cur = nx;
      nx = nx2;
      id = id1;
      id1 = id2;
      ks = ks1;
      vs = vs1;
    }
    // after an abort, no copy may still be on its way when the CTA ends
    if (lane == 0 && *s_abort)
      for (int u = max(0, copied - NST); u < copied; ++u) tc::mbar_wait(&full[u % NST], (u / NST) & 1, kWaitLimit);
    __syncwarp();
  } else if (ntile > 0 && warp == 17) {
    // ------------------------------------------------------------ tensor core
    if (elect_one()) {
      // Steps v in a fixed order: tile and stream in turn.  S two steps ahead of O += P V, so that one stream's
      // softmax runs while the other's products do; not past the end of a row tile, though, whose last O has to come
      // before the next one's queries can (the thread waits for what it needs next, and for nothing else).
      const int steps = Two ? 2 * ntile : ntile;
      // (a descriptor's low bits are its address / 16)
      const uint64_t dq = tc::desc_k_none(tc::smem_u32(qbuf), 2048, 128), dk = tc::desc_k_none(tc::smem_u32(kbuf), 2048, 128),
                     dv = tc::desc_k_none(tc::smem_u32(vbuf), D * 16, 128);
      // (what a wait has shown is not asked for again: a wait costs its 100 to 300 cycles also when it need not wait)
      int next = 0, turn_p = 0, turn_s = 0;   // next S; row tiles of the next product with V and of the next S
      int flags_s = 0, flags_p[2] = {0, 0};   // of the next S's tile, of the streams' next products with V
      int asked = -1, laid[2] = {-1, -1};     // last tile whose K is known to be there; row tiles whose queries are
      bool ok = true;
      for (int v = 0; ok && v < steps; ++v) {
        while (next < steps && next < v + 2) {
          const int i = Two ? next >> 1 : next, x = next & 1;
          if (asked != i) {
            ok = tc::mbar_wait(&kfull[i & 1], (i >> 1) & 1, kWaitLimit);
            if (!ok) break;
            asked = i;
            flags_s = infos[i % kCtInfo].flags;
            turn_s = infos[i % kCtInfo].turn;
          }
          if (next == v) turn_p = turn_s;
          if (turn_s != turn_p) break;
          if (laid[Two ? x : 0] != turn_s) {
            ok = tc::mbar_wait(&qfull[Two ? x : 0], turn_s & 1, kWaitLimit);
            if (!ok) break;
            laid[Two ? x : 0] = turn_s;
          }
          tc::fence_after();
          const uint64_t d0 = dk + (i & 1) * (C::QT / 16), q0 = dq + (Two ? x : 0) * (C::QT / 16);
          const uint32_t tS = tmem + x * kCtT;
#pragma unroll
          for (int t = C::NQ - 1; t >= 0; --t)   // (the small terms first)
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc::mma_bf16(tS, q0 + t * (C::QT / 16) + k * 256, d0 + k * 256, idesc_f16(kCtT), t < C::NQ - 1 || k > 0);
          tc::mma_commit(&sfull[x]);
          if (!Two || x == 1) tc::mma_commit(&kempty[i & 1]);
          flags_p[x] = flags_s;
          ++next;
        }
        if (!ok) break;
        const int i = Two ? v >> 1 : v, x = v & 1, flags = flags_p[x];
        if (!Two || x == 0) ok = tc::mbar_wait(&vfull[i & 1], (i >> 1) & 1, kWaitLimit);
        ok = ok && tc::mbar_wait(&pfull[x], (Two ? i : i >> 1) & 1, kWaitLimit);
        if (!ok) break;
        tc::fence_after();
        const uint64_t d0 = dv + (i & 1) * (C::QT / 16);
        const uint32_t tS = tmem + x * kCtT, tO = tmem + 2 * kCtT + x * D;
#pragma unroll
        for (int t = 0; t < C::NP; ++t)
#pragma unroll
          for (int k = 0; k < kCtT / 16; ++k)
            mma_f16_ts(tO, tS + k / 2 * 32 + k % 2 * 8 + t * 16, d0 + k * (2 * D), idesc_f16(D), !(flags & kSFirst) || t + k > 0);
        if (!Two || x == 1) tc::mma_commit(&vempty[i & 1]);
        if (flags & kSLast) tc::mma_commit(&ofin[x]);
      }
      if (!ok) abort_now();
    }
    __syncwarp();
  } else if (ntile > 0 && warp >= 8 && warp < 16) {
    // ------------------------------------------------------------ conversion
    const int t = tid & 127;
    const bool v = warp >= 12;
    auto to_half = [](const uint4& w, uint4* lo, uint4* hi) {
      auto four = [](uint32_t c, uint32_t* a, uint32_t* b) {
        asm("{\n\t.reg .b16 x, y;\n\t"
            "mov.b32 {x, y}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, x;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
            : "=r"(*a), "=r"(*b)
            : "r"(c));
      };
      four(w.x, &lo->x, &lo->y);
      four(w.y, &lo->z, &lo->w);
      four(w.z, &hi->x, &hi->y);
      four(w.w, &hi->z, &hi->w);
    };
    constexpr int U = D / 16;   // 16-byte pieces of a thread
    // (one code for K and V: the kernel's instructions should stay in the instruction cache)
    const int sstep = v ? 2048 : 128, dhalf = v ? D * 16 : 2048;
    const int src = v ? t * 16 : (t >> 3) * (8 * D) + (t & 7) * 16;
    unsigned char* dst0 = v ? vbuf + t / D * (2 * D * 16) + t % D * 16 : kbuf + t * 16;
    uint64_t* done = v ? vfull : kfull;
    uint64_t* room = v ? vempty : kempty;
    uint32_t votes = 0;
    constexpr int Batch = kCtBatch < U ? kCtBatch : U;
    for (int i = 0; i < ntile; ++i) {
      const int b = i & 1, n = 2 * i + v, st = n % NST;
      if (!warp_wait(&full[st], n / NST)) break;
      unsigned char* codes = stages + st * C::KB + src;
      const int flags = infos[i % kCtInfo].flags, cnt = flags & 255;
      if (!warp_wait(&room[b], (i >> 1) ^ 1)) break;
      // (keys past the tokens are whatever was there: their logits are not used)
      if (v && (flags & kMixed || cnt < kCtT)) {
        // V past the tokens counts as zero.  NaN that not all rows see is taken out and noted.  (In the codes,
        // of which each thread changes those that it converts)
        uint32_t nan = 0;
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const int keep = cnt - (u * 128 + t) / D * 16;   // of the piece's 16 tokens
          uint32_t* ww = reinterpret_cast<uint32_t*>(codes + u * sstep);
#pragma unroll 1
          for (int e = 0; e < 4; ++e) {
            const int k = keep - 4 * e;
            uint32_t w = ww[e];
            if (k < 4) ww[e] = w = k <= 0 ? 0u : w & ((1u << (8 * k)) - 1u);
            nan |= (w & 0x7f7f7f7fu) + 0x01010101u;        // a NaN's byte carries into its sign
          }
        }
        if (flags & kMixed) {
          const int mine = __any_sync(0xffffffffu, nan & 0x80808080u);
          if (lane == 0) {
            s_vote[(votes & 1) * 4 + (warp & 3)] = mine;
            tc::mbar_arrive(vote_bar);
          }
          if (!warp_wait(vote_bar, votes)) break;
          const volatile int* all = s_vote + (votes & 1) * 4;
          const bool any = all[0] | all[1] | all[2] | all[3];
          ++votes;
          if (t == 0) s_nan[b] = any;
          if (any)
#pragma unroll 1
            for (int u = 0; u < U; ++u) {
              uint32_t bits = 0;   // bit e: token e of the piece
#pragma unroll 1
              for (int e = 0; e < 16; ++e)
                if ((codes[u * sstep + e] & 0x7f) == 0x7f) {
                  codes[u * sstep + e] = 0;
                  bits |= 1u << e;
                }
              const int x = u * 128 + t;
              reinterpret_cast<uint16_t*>(nan_masks)[(b * 128 + x % D) * 8 + x / D] = static_cast<uint16_t>(bits);
            }
        }
      }
      unsigned char* dst = dst0 + b * C::QT;
#pragma unroll 1
      for (int h = 0; h < U; h += Batch) {
        uint4 w[Batch], lo, hi;
#pragma unroll
        for (int u = 0; u < Batch; ++u) w[u] = *reinterpret_cast<const uint4*>(codes + (h + u) * sstep);
#pragma unroll
        for (int u = 0; u < Batch; ++u) {
          to_half(w[u], &lo, &hi);
          *reinterpret_cast<uint4*>(dst + (h + u) * 4096) = lo;
          *reinterpret_cast<uint4*>(dst + (h + u) * 4096 + dhalf) = hi;
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(&done[b]);
        tc::mbar_arrive(&sempty[st]);
      }
    }
  } else if (ntile > 0 && warp < 8) {
    // ------------------------------------------------------------ softmax
    const int x = warp >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>(wq) << 21;
    const uint32_t tS = tmem + x * kCtT + lanes, tO0 = tmem + 2 * kCtT + lanes, tO = tO0 + x * D;
    float m = -INFINITY, l = 0.f, rowf = 0.f;
    int lim = 0, vexp = 0, seq = 0, j = 0, h = 0;
    bool valid = false, active = false, used = false;
    uint32_t nanrow[D / 32];
    uint32_t use = 0, fin0 = 0, fin1 = 0;
    [[maybe_unused]] uint32_t whole_parts = 0;
    int joined = 0;   // stream 1: row tiles that stream 0 is known to have joined
    auto wait_joined = [&](int turn) {
      if (joined >= turn) return true;
      joined = turn;
      return warp_wait(jdone, turn - 1);
    };

    // The warp's 32 queries, in fp16 terms, and the factors of their logits.  A lane loads 16-byte pieces
    // of rows lane % 8 + 8 g: four lanes take 64 adjacent bytes, and eight rows' pieces are 128 adjacent bytes of
    // the operand.
    constexpr int V = Ty<T>::kVec, N = D / V;   // elements of a piece, pieces of a row
    auto row_of = [&](int g) { return g * 8 + (lane & 7); };   // of the warp's
    auto lay_q = [&]() {
      const long long mine = valid ? seq * a.qb + h * a.qh + j * a.qs : -1;
      auto load = [&](int g, uint4* r) {
        const long long off = __shfl_sync(0xffffffffu, mine, row_of(g & 3));
        const T* src = static_cast<const T*>(a.q) + off + (lane >> 3) * V;
#pragma unroll
        for (int u = 0; u < N / 4; ++u) {
          r[u] = make_uint4(0, 0, 0, 0);
          if (off < 0 || g > 3) continue;
          if (a.wide_q) {
            r[u] = *reinterpret_cast<const uint4*>(src + u * 4 * V);
          } else {
#pragma unroll
            for (int e = 0; e < V; ++e) reinterpret_cast<T*>(&r[u])[e] = src[u * 4 * V + e];
          }
        }
      };
      // (rolled, the next group's pieces on their way: unrolled, the code of a row tile's start and end was fetched
      // anew each time, and a prompt of 2048 took 128 us)
      uint4 raw[N / 4], ahead[N / 4];
      load(0, ahead);
#pragma unroll 1
      for (int g = 0; g < 4; ++g) {
#pragma unroll
        for (int u = 0; u < N / 4; ++u) raw[u] = ahead[u];
        load(g + 1, ahead);
        float top = 0.f;
#pragma unroll
        for (int u = 0; u < N / 4; ++u)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float z = fabsf(Ty<T>::to_f(reinterpret_cast<const T*>(&raw[u])[e]));
            top = fmaxf(top, z < INFINITY ? z : INFINITY);   // (NaN, too)
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        const bool bad = !(top < INFINITY);   // an entry that is not finite: the row is NaN
        const int ex = bad ? 0 : max(static_cast<int>(__float_as_uint(top) >> 23) - 127, -100);
        const float down = exp2i(14 - ex);    // the largest to [2^14, 2^15)
        const float f = __shfl_sync(0xffffffffu, exp2i(ex - 14) * a.scale_log2, lane & 7);
        if (lane >> 3 == g) rowf = f;
        unsigned char* dst = qbuf + (Two ? x : 0) * C::QT + (wq * 32 + row_of(g)) * 16;
#pragma unroll
        for (int u = 0; u < N / 4; ++u) {
          // a piece of fp32 is half a piece of the operand
          const int at = (u * 4 + (lane >> 3)) * V;   // its first element
          uint32_t w[C::NQ][V / 2];
#pragma unroll
          for (int e = 0; e < V; e += 2) {
            float y0 = Ty<T>::to_f(reinterpret_cast<const T*>(&raw[u])[e]) * down;
            float y1 = Ty<T>::to_f(reinterpret_cast<const T*>(&raw[u])[e + 1]) * down;
            if (bad) y0 = y1 = __int_as_float(0x7fffffff);
#pragma unroll
            for (int n = 0; n < C::NQ; ++n) {
              const __half2 z = __floats2half2_rn(y0, y1);
              w[n][e / 2] = *reinterpret_cast<const uint32_t*>(&z);
              y0 -= __low2float(z);
              y1 -= __high2float(z);
            }
          }
#pragma unroll
          for (int n = 0; n < C::NQ; ++n) {
            unsigned char* d = dst + n * C::QT + (at >> 3) * 2048 + (at & 7) * 2;
            if constexpr (V == 8) *reinterpret_cast<uint4*>(d) = make_uint4(w[n][0], w[n][1], w[n][2], w[n][3]);
            else *reinterpret_cast<uint2*>(d) = make_uint2(w[n][0], w[n][1]);
          }
        }
      }
      if (!Two) sqs[row] = rowf;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&qfull[Two ? x : 0]);
    };

    // S of one tile to P over its columns, 32 columns at a time (the loops are short on purpose: unrolled over
    // the tile, instruction fetch bound them).  General: tokens the row does not see, scales of any kind.
    constexpr int W = kCtT / Copies;            // columns of this warp
    const int col0 = Copies > 1 ? wq * W : 0;
    // The references m and 2^vexp of a tile whose largest logit is mt and whose V scales that the row sees are below 2^vt; O and
    // l follow.  m is a whole number, so that what was formed by one reference is brought to another's exactly, here
    // and where parts are joined.  (Rows that do not see all of a tile have vt's of their own: by a hidden token's scale
    // theirs would lose bits.  Such tiles are a row tile's last ones.)
    auto raise = [&](int vt, bool first, float mt) {
      const int v2 = first ? vt : max(vexp, vt);
      if (first) {
        m = floorf(mt);
      } else if (__any_sync(0xffffffffu, mt > m + 4.f || v2 > vexp)) {
        const float m2 = fmaxf(m, floorf(mt)), al = m2 == -INFINITY ? 1.f : exp2i(static_cast<int>(fmaxf(m - m2, -126.f)));
        m = m2;
        l *= al;
        const float r = al * exp2i(max(vexp - v2, -126));
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tc::tmem_ld16(tO + c, o);
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[e] * r);
          tmem_st16(tO + c, w);
        }
      }
      vexp = v2;
    };
    auto zero_others = [&]() {   // P in the other warps' columns
      const uint32_t zero[16] = {};
#pragma unroll
      for (int c = 0; c < kCtT; c += W)
#pragma unroll
        for (int n = 0; n < C::NP; ++n)
          if (c != col0) tmem_st16(tS + c + 16 * n, zero);
    };
    // x f + off; beside fp32 with what f's rounding leaves (one relative error of all logits otherwise, 3e-7 of p)
    auto exponent = [&](float x, float f, float off, float rest) {
      const float y = fmaf(x, f, off);
      return C::NQ > 1 ? fmaf(x * f, rest, y) : y;
    };
    // All tokens seen, scales positive and not too far apart: bf16's V scale v goes into the exponent, w = 2^(x - m + log2 v), and
    // comes out of the sum of 16 tokens' w again; four and a half instructions an element, two of them w's second term.
    auto softmax_plain = [&](const TileInfo& in, bool first) {
      float mt = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < W; c += 32) {
        float s[32];
        tc::tmem_ld32(tS + col0 + c, s);
        const float2 k2 = *reinterpret_cast<const float2*>(in.ks + (col0 + c) / 16);
        float t0 = s[0], t1 = s[16];
#pragma unroll
        for (int e = 1; e < 15; e += 2) {
          t0 = max3(t0, s[e], s[e + 1]);
          t1 = max3(t1, s[16 + e], s[17 + e]);
        }
        mt = max3(mt, fmaxf(t0, s[15]) * (rowf * k2.x), fmaxf(t1, s[31]) * (rowf * k2.y));
      }
      raise(in.vexp, first, mt);
      const float ref = m == -INFINITY ? 0.f : m, up = exp2i(11 - vexp);
#pragma unroll 1
      for (int c = 0; c < W; c += 32) {
        const float2 k2 = *reinterpret_cast<const float2*>(in.ks + (col0 + c) / 16);
        const float2 v2 = *reinterpret_cast<const float2*>(in.vs + (col0 + c) / 16);
        float s[32];
        tc::tmem_ld32(tS + col0 + c, s);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          // (not beside fp32: with the scale's 11 binades the exponent's own rounding would show)
          constexpr bool Fold = C::NQ == 1;
          const float fg = rowf * (g ? k2.y : k2.x), fv = (g ? v2.y : v2.x) * up, off = Fold ? lg2(fv) - ref : -ref;
          float2 sum = make_float2(0.f, 0.f);
          uint32_t w[C::NP][8];
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            const float s0 = s[16 * g + e], s1 = s[16 * g + e + 1];
            const float2 x = Fold ? fma2(make_float2(s0, s1), make_float2(fg, fg), make_float2(off, off))
                                  : make_float2(exponent(s0, fg, off, a.scale_rest), exponent(s1, fg, off, a.scale_rest));
            float2 p = make_float2(ex2(x.x), ex2(x.y));
            sum = add2(sum, p);
            if (!Fold) p = make_float2(p.x * fv, p.y * fv);
            terms2(p, &w[0][e / 2], &w[1][e / 2]);
          }
          l = Fold ? fmaf(sum.x + sum.y, __fdividef(1.f, fv), l) : l + (sum.x + sum.y);
          // P of 32 tokens over their own columns of S: 16 columns a term
#pragma unroll
          for (int n = 0; n < C::NP; ++n) tmem_st8(tS + col0 + c + 16 * n + 8 * g, w[n]);
        }
      }
      if constexpr (Copies > 1) zero_others();
      tmem_wait_st();
    };
    // Any tokens, any scales; large: logits of any size, S is replaced by them, rounded.
    auto softmax_any = [&](const TileInfo& in, bool first, bool large) {
      const int rem = lim - in.tile * kCtT - col0;
      const float rest = large ? 0.f : a.scale_rest;
      if (large) {
#pragma unroll 1
        for (int c = 0; c < W; c += 16) {
          float s[16];
          tc::tmem_ld16(tS + col0 + c, s);
          const float fg = rowf * in.ks[(col0 + c) / 16];
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(s[e] * fg);
          tmem_st16(tS + col0 + c, w);
        }
        tmem_wait_st();
      }
      float mt = -INFINITY;
#pragma unroll 1
      for (int c = 0; c < W; c += 16) {
        float s[16];
        tc::tmem_ld16(tS + col0 + c, s);
        const float fg = large ? 1.f : rowf * in.ks[(col0 + c) / 16];
#pragma unroll
        for (int e = 0; e < 16; ++e) mt = fmaxf(mt, c + e < rem ? s[e] * fg : -INFINITY);
      }
      int vt = in.vexp;
      if (in.flags & kMixed) {   // of the scales that the row sees
        float top = 0.f;
#pragma unroll
        for (int g = 0; g < 8; ++g) {
          const float v = fabsf(in.vs[g]);
          if (16 * g < rem + col0 && v < INFINITY) top = fmaxf(top, v);
        }
        vt = scale_exp(top);
      }
      raise(vt, first, mt);
      const float ref = m == -INFINITY ? 0.f : m, up = exp2i(11 - vexp);
      float sum = 0.f;
#pragma unroll 1
      for (int c = 0; c < W; c += 32) {
        uint32_t w[C::NP][16];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          float s[16];
          tc::tmem_ld16(tS + col0 + c + 16 * g, s);
          const float fg = large ? 1.f : rowf * in.ks[(col0 + c) / 16 + g], fv = in.vs[(col0 + c) / 16 + g] * up;
#pragma unroll
          for (int e = 0; e < 16; e += 2) {
            float p[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const bool seen = c + 16 * g + e + u < rem;
              p[u] = seen ? ex2(exponent(s[e + u], fg, -ref, rest)) : 0.f;
              sum += p[u];
              p[u] = seen ? p[u] * fv : 0.f;   // (a scale that is no number under a hidden token)
            }
            terms2(make_float2(p[0], p[1]), &w[0][8 * g + e / 2], &w[1][8 * g + e / 2]);
          }
          if (!(fabsf(fv) < INFINITY))   // an infinite scale's p is its first term
#pragma unroll
            for (int e = 0; e < 8; ++e) w[1][8 * g + e] = 0;
        }
#pragma unroll
        for (int n = 0; n < C::NP; ++n) tmem_st16(tS + col0 + c + 16 * n, w[n]);
      }
      if constexpr (Copies > 1) zero_others();
      l += sum;
      tmem_wait_st();
    };

    // The warp's finished rows (fin), or this CTA's part of them, 16 columns at a time from o(c, v): 64 bytes of eight
    // rows to a store, by way of the warp's own queries' place, which is free by now (no other warp's next
    // queries go there).
    auto store_rows = [&](bool fin, size_t part, auto&& o) {
      unsigned char* buf = qbuf + (Two ? x : 0) * C::QT + wq * 512;   // pieces of 32 rows, 2048 bytes apart
      const long long mine = !valid ? -1 : fin ? seq * a.ob + h * a.oh + j * a.os : static_cast<long long>(part * D);
      const int E = fin ? static_cast<int>(sizeof(T)) : 4;
      unsigned char* base = fin ? static_cast<unsigned char*>(a.out) : reinterpret_cast<unsigned char*>(a.part_o);
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        float v[16];
        o(c, v);
        __syncwarp();
        if (fin && sizeof(T) == 2) {
          T y[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = Ty<T>::from_f(v[e]);
#pragma unroll
          for (int e = 0; e < 2; ++e) *reinterpret_cast<uint4*>(buf + e * 2048 + lane * 16) = reinterpret_cast<const uint4*>(y)[e];
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) *reinterpret_cast<float4*>(buf + e * 2048 + lane * 16) = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
        __syncwarp();
        // 16 columns are 32 or 64 bytes: two or four lanes to a row
        const int per = E, rows = 32 / per;   // lanes to a row (E == 2: 2, 4: 4), rows at a time
#pragma unroll 1
        for (int g = 0; g < 32; g += rows) {
          const int r = g + lane % rows, piece = lane / rows;
          const long long off = __shfl_sync(0xffffffffu, mine, r);
          const uint4 z = *reinterpret_cast<const uint4*>(buf + piece * 2048 + r * 16);
          if (off < 0) continue;
          unsigned char* dst = base + (off + c) * E + piece * 16;
          if (!fin || a.wide_o) {
            *reinterpret_cast<uint4*>(dst) = z;
          } else {
#pragma unroll
            for (int e = 0; e < static_cast<int>(16 / sizeof(T)); ++e) reinterpret_cast<T*>(dst)[e] = reinterpret_cast<const T*>(&z)[e];
          }
        }
      }
    };

    for (int i = 0, end; i < ntile; i = end + 1) {
      if (!warp_wait(&ifull[i % kCtInfo], i / kCtInfo)) break;
      const TileInfo& head = infos[i % kCtInfo];
      const int flags = head.flags, turn = head.turn, head_n = head.n, head_len = head.len, head_q = head.q;
      const int kvh = head.pair % a.c.h_kv;
      end = head.end;
      {
        const int r = head_q * Rows + (Two ? x * kCtT : 0) + row % (kCtT / Copies);
        seq = head.pair / a.c.h_kv;
        valid = r < head_len * a.G;
        j = valid ? r / a.G : 0;
        h = kvh * a.G + (valid ? r - j * a.G : 0);
        lim = valid ? tokens_seen(a, head_n, head_len, j) : 0;
        active = __any_sync(0xffffffffu, valid);
        m = -INFINITY;
        l = 0.f;
        used = false;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) nanrow[e] = 0;
      }
      if (Two || x == 0) {
        lay_q();
      } else {
        if (!warp_wait(&qfull[0], turn)) break;
        rowf = sqs[row];
      }
      const int rexp = static_cast<int>(__float_as_uint(warp_max(fabsf(rowf))) >> 23);   // of the warp's largest factor
      // this stream's tiles
      int t = Two ? i : i + ((i ^ x) & 1);
      bool ok = true;
      for (; t <= end; t += Two ? 1 : 2) {
        ok = warp_wait(&ifull[t % kCtInfo], t / kCtInfo) && warp_wait(&sfull[x], use);
        if (!ok) break;
        const TileInfo& in = infos[t % kCtInfo];
        ++use;
        tc::fence_after();
        if (!Two && x == 1 && !(ok = wait_joined(turn))) break;   // O is free
        if (active) {
          const int4 what = *reinterpret_cast<const int4*>(&in);   // tile, flags, vexp, vlow
          const int rem = lim - what.x * kCtT, tf = what.y;
          const bool large = (tf >> kKexp) + rexp > kLargeSum;
          if (large || (tf & (kMixed | kOdd)) || (tf & 255) < kCtT ||
              what.w + 71 < (used ? max(vexp, what.z) : what.z))   // (below 2^-60 of the largest, w could vanish before p does)
            softmax_any(in, !used, large);
          else
            softmax_plain(in, !used);
          if (tf & kMixed) {
            if (!(ok = warp_wait(&vfull[t & 1], t >> 1))) break;
            if (s_nan[t & 1])
#pragma unroll 1
              for (int d = 0; d < D; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int k = rem - 32 * e;   // tokens of this word that the row sees
                  const uint32_t see = k >= 32 ? 0xffffffffu : k <= 0 ? 0u : (1u << k) - 1u;
                  const uint32_t hit = nan_masks[((t & 1) * 128 + d) * 4 + e] & see ? 1u << (d & 31) : 0u;
#pragma unroll
                  for (int u = 0; u < D / 32; ++u) nanrow[u] |= d / 32 == u ? hit : 0u;
                }
          }
        }
        used = true;
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&pfull[x]);
      }
      if (!ok) break;
      // ---- the row tile's end
      bool nan_any = false;
#pragma unroll
      for (int e = 0; e < D / 32; ++e) nan_any |= nanrow[e] != 0;
      nan_any = __any_sync(0xffffffffu, nan_any);
      if (!Two && x == 1) {
        if (!wait_joined(turn)) break;
        s_ml[row] = make_float2(m, l);
        if (nan_any)
#pragma unroll
          for (int e = 0; e < D / 32; ++e) nan_masks[(2 * 128 + row) * 4 + e] = nanrow[e];
        sqs[row] = __int_as_float(vexp);   // (this row's factor has been read, and is written anew after jfull)
        if (lane == 0) s_join[wq] = make_int2(used, nan_any);
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(jfull);
        continue;
      }
      float m1 = -INFINITY, l1 = 0.f;
      int vexp1 = 0;
      bool had1 = false;   // stream 1 had tiles of it
      if (!Two) {
        if (!warp_wait(jfull, turn)) break;
        const float2 ml = s_ml[row];
        const int2 sj = s_join[wq];
        had1 = sj.x;
        if (had1) {
          vexp1 = __float_as_int(sqs[row]);
          m1 = ml.x;
          l1 = ml.y;
          if (!warp_wait(&ofin[1], fin1++)) break;
        }
        if (sj.y) {
#pragma unroll
          for (int e = 0; e < D / 32; ++e) nanrow[e] |= nan_masks[(2 * 128 + row) * 4 + e];
          nan_any = true;
        }
      }
      if (used && !warp_wait(&ofin[Two ? x : 0], fin0++)) break;
      tc::fence_after();
      if (active) {
        const float mm = fmaxf(m, m1), ref = mm == -INFINITY ? 0.f : mm;
        float r0 = used ? ex2(m - ref) : 0.f, r1 = had1 ? ex2(m1 - ref) : 0.f;
        const float sum = (used ? l * r0 : 0.f) + (had1 ? l1 * r1 : 0.f);
        r0 *= exp2i(used ? vexp - 11 : 0);
        r1 *= exp2i(had1 ? vexp1 - 11 : 0);
        const bool whole = Copies == 1 && (flags & kWhole);   // (copies are joined below)
        const float inv = whole ? 1.f / sum : 1.f;
        const size_t part = static_cast<size_t>(2 * cta + (turn > 0)) * C::PartRows + (Two ? x * kCtT : 0) + row;
        store_rows(whole, part, [&](int c, float* o) {
          if (used) {
            tc::tmem_ld16(tO + c, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] *= r0;
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = 0.f;
          }
          if (!Two && had1) {
            float z[16];
            tc::tmem_ld16(tO0 + D + c, z);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = fmaf(z[e], r1, o[e]);
          }
          if (nan_any) {
            uint32_t bits = 0;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) bits = c / 32 == u ? nanrow[u] : bits;
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (bits >> ((c & 31) + e) & 1) o[e] = __int_as_float(0x7fffffff);
          }
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = lim > 0 ? o[e] * inv : 0.f;
          }
        });
        if (valid && !whole) a.part_ml[part] = make_float2(mm, sum);
        if (valid && whole && a.lse)
          a.lse[(static_cast<size_t>(seq) * a.h_q + h) * a.s + j] = lim > 0 ? (ref + log2f(sum)) * 0.6931471805599453f : -INFINITY;
      }
      if (Copies > 1 && (flags & kWhole)) {
        // (the next parts are written after jdone)
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(parts_bar);
        if (!warp_wait(parts_bar, whole_parts++)) break;
        const size_t part = static_cast<size_t>(2 * cta + (turn > 0)) * C::PartRows;
        for (int u = wq; u < Rows && head_q * Rows + u < head_len * a.G; u += 4) {
          const int r = head_q * Rows + u, jr = r / a.G;
          join_row<T, D, Copies>(a, seq, kvh * a.G + r - jr * a.G, jr, tokens_seen(a, head_n, head_len, jr) > 0, 1, Rows,
                                 [&](int) { return part + u; });
        }
      }
      tc::fence_before();
      if (!Two) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(jdone);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 17) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------ merge
constexpr int kCgThreads = 256, kCgRows = 8;

// Row (x) = boundary between two CTAs' runs: the first one inside a row tile joins its
// parts, in order; kCgRows rows to a CTA, a warp to a row.
template <typename T, int D, bool Two, int Copies>
__global__ void __launch_bounds__(kCgThreads) k_tokens_merge(const __grid_constant__ TokensArgs a, int ncta) {
  using C = Ct<T, D, Two, Copies>;
  constexpr int Rows = C::Rows;
  tc::grid_dep_wait();
  const int c = blockIdx.x + 1;
  const int4 rec = a.rec[c];
  if (rec.x < 0) return;
  const int total = rec.w, n = min(ncta, total), first = rec.z;
  if (run_begin(c - 1, n, total) > first + kCtCost) return;
  const int seq = rec.x / a.c.h_kv, kvh = rec.x - seq * a.c.h_kv, len = tokens_len(a, seq), tok = cache_tokens(a.c, rec.x);
  const int nt = lim_tiles(tile_lim<Rows>(a, tok, len, rec.y));
  const int c1 = run_owner(min(first + kCtCost + nt, total) - 1, n, total);
  const int slot0 = 2 * (c - 1) + (run_begin(c - 1, n, total) < first);   // CTA c - 1's last part; the others' first
  for (int u = threadIdx.x >> 5; u < kCgRows; u += kCgThreads / 32) {
    const int row = blockIdx.y * kCgRows + u, r = rec.y * Rows + row;
    if (row >= Rows || r >= len * a.G) return;
    const int j = r / a.G;
    join_row<T, D, Copies>(a, seq, kvh * a.G + r - j * a.G, j, tokens_seen(a, tok, len, j) > 0, c1 - c + 2, Rows, [&](int v) {
      return static_cast<size_t>(v == 0 ? slot0 : 2 * (c - 1 + v)) * C::PartRows + row;
    });
  }
}

static int tokens_ctas(const shadowkv_cache& c, int rows, int per, int nsm) {
  const long long tiles = (static_cast<long long>(c.max_blocks) * c.block + kCtT - 1) / kCtT;
  const long long all = (tiles + kCtCost) * ((rows + per - 1) / per) * c.b * c.h_kv;
  return static_cast<int>(all < nsm ? all : nsm);
}

static size_t tokens_layout(const shadowkv_cache& c, int nsm, char* base, TokensArgs* a) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base + off;
    off += (bytes + 255) / 256 * 256;
    return p;
  };
  char* rec = take(nsm * sizeof(int4));
  char* ml = take(static_cast<size_t>(2 * nsm) * 256 * sizeof(float2));
  char* nan = take(static_cast<size_t>(nsm) * 3 * 128 * 4 * sizeof(uint32_t));
  char* o = take(static_cast<size_t>(2 * nsm) * 256 * c.d * sizeof(float));
  if (a) {
    a->rec = reinterpret_cast<int4*>(rec);
    a->part_ml = reinterpret_cast<float2*>(ml);
    a->nan = reinterpret_cast<uint32_t*>(nan);
    a->part_o = reinterpret_cast<float*>(o);
  }
  return off;
}

template <typename T, int D, bool Two, int Copies>
static cudaError_t attend_tokens_t(const TokensArgs& a, const shadowkv_cache& c, int nsm, cudaStream_t st) {
  using C = Ct<T, D, Two, Copies>;
  const int ncta = tokens_ctas(c, a.s * a.G, C::Rows, nsm);
  const auto kern = k_attend_tokens<T, D, Two, Copies>;
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(kern), C::Smem);
  if (e == cudaSuccess) e = launch_pdl(kern, dim3(ncta), dim3(kCtThreads), C::Smem, st, a);
  if (e != cudaSuccess || ncta == 1) return e;
  const int rows = a.s * a.G < C::Rows ? a.s * a.G : C::Rows;
  return launch_pdl(k_tokens_merge<T, D, Two, Copies>, dim3(ncta - 1, (rows + kCgRows - 1) / kCgRows), dim3(kCgThreads), 0, st, a, ncta);
}

// Rows of a sequence and KV head: up to 32 stand four times in one tile; bf16's take two tiles at a time from
// 129 on (an fp32 row's terms take the room of the second).
template <int D>
static cudaError_t attend_tokens_d(const TokensArgs& a, const shadowkv_cache& c, int dtype, int nsm, cudaStream_t st) {
  const int rows = a.s * a.G;
  if (dtype != SKV_DTYPE_BF16)
    return rows <= 32 ? attend_tokens_t<float, D, false, 4>(a, c, nsm, st) : attend_tokens_t<float, D, false, 1>(a, c, nsm, st);
  return rows <= 32    ? attend_tokens_t<bf16, D, false, 4>(a, c, nsm, st)
         : rows <= kCtT ? attend_tokens_t<bf16, D, false, 1>(a, c, nsm, st)
                        : attend_tokens_t<bf16, D, true, 1>(a, c, nsm, st);
}

static const char* tokens_fault(const shadowkv_cache& c, int h_q, int s, skv_status* st) {
  *st = SKV_ERR_INVALID_ARG;
  if (s < 0) return "s must be >= 0";
  *st = SKV_ERR_UNSUPPORTED;
  if (h_q < 1 || h_q % c.h_kv || h_q / c.h_kv > 128) return "h_q must be a multiple of h_kv, of at most 128";
  const long long rows = static_cast<long long>(s) * (h_q / c.h_kv);
  if (rows > 1 << 24) return "s h_q / h_kv must be at most 2^24";
  if (((rows + 127) / 128) * ((static_cast<long long>(c.max_blocks) * c.block + 127) / 128 + kCtCost) >= (1LL << 31) / (static_cast<long long>(c.b) * c.h_kv))
    return "too many queries and tokens for one call";
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
  int nsm = 0;
  const cudaError_t e = skv::device_sms(&nsm);
  if (e != cudaSuccess) {
    skv::set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
    return 0;
  }
  return skv::tokens_layout(*c, nsm, nullptr, nullptr);
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
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  int nsm = 0;
  cudaError_t e = skv::device_sms(&nsm);
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  skv::TokensArgs a;
  if (work_bytes < skv::tokens_layout(*c, nsm, static_cast<char*>(work), &a))
    return set_error(SKV_ERR_INVALID_ARG, "the workspace is smaller than shadowkv_cache_attend_tokens_workspace");
  a.c = skv::cache_dev(*c);
  a.q = q->ptr;
  a.out = out->ptr;
  a.lse = lse;
  a.lens = lens;
  // the stride of an extent of 1 is not used
  a.qb = c->b > 1 ? q->sb : 0; a.qh = h_q > 1 ? q->sh : 0; a.qs = s > 1 ? q->ss : 0;
  a.ob = c->b > 1 ? out->sb : 0; a.oh = h_q > 1 ? out->sh : 0; a.os = s > 1 ? out->ss : 0;
  const double scale_log2 = static_cast<double>(scale) * 1.4426950408889634;
  a.scale_log2 = static_cast<float>(scale_log2);
  a.scale_rest = a.scale_log2 != 0.f ? static_cast<float>((scale_log2 - a.scale_log2) / a.scale_log2) : 0.f;
  a.s = s;
  a.h_q = h_q;
  a.G = h_q / c->h_kv;
  a.causal = causal;
  auto wide = [&](const void* ptr, long long sb, long long sh, long long ss) {
    return reinterpret_cast<uintptr_t>(ptr) % 16 == 0 && (sb * E) % 16 == 0 && (sh * E) % 16 == 0 && (ss * E) % 16 == 0;
  };
  a.wide_q = wide(q->ptr, a.qb, a.qh, a.qs);
  a.wide_o = wide(out->ptr, a.ob, a.oh, a.os);
  cudaStream_t p = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  e = c->d == 128 ? skv::attend_tokens_d<128>(a, *c, dtype, nsm, p) : skv::attend_tokens_d<64>(a, *c, dtype, nsm, p);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
