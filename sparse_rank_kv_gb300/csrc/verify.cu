// Verification of drafted tokens against the target's logits
// (shadowkv_verify_drafts): how many of a sequence's drafts stand, and the token
// that follows them, from given random numbers.
//
// Which token a number falls on is decided next to borders (a vocabulary of 2^17 has as
// many), so the weights w_v = exp((l_v - max) / T) of the row that is sampled from are
// whole numbers: 2^43 w_v, each within 2^-37 of itself and half a unit, by a table of 2^(j/64) and a
// short polynomial (Tang, "Table-driven implementation of the exponential function",
// 1989) on pairs of floats.  Their sums are exact and do not depend on the order; the half units of a long flat tail add
// up to vocab 2^-44 of a total at most (2^-27 of 131,072 tokens).  The rows'
// sums for the acceptance tests are fp32 and good to 2^-13; a test that close to its
// border (one in 5,000) is decided again with the row's whole-number sum.
//
// The logits are read once by k_verify_rows; one row per sequence is read again by
// k_verify_pick (from L2), with the draft's distribution.  Measured in a graph: 64 sequences of up to
// 7 drafts over 128,256 tokens in bf16 99 us (the 107 MB it cannot do without: 16 us); one
// sequence of 4 over 32,000 16.5 us.  Profiled at the first, k_verify_rows is 0.3 of it
// (DRAM at 30%, issue slots at 47%: it waits for loads) and k_verify_pick 0.7: 39 million warp
// instructions, 60% of the issue slots of SMs that have work, but 36 clusters fit at a time
// and 64 take two rounds, so over its duration it issues at 37%.
#include <cooperative_groups.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {
namespace cg = cooperative_groups;

struct VerifyArgs {
  const void* logits;
  const int32_t* drafts;
  const float* probs;
  const float *accept, *sample;
  const int32_t* lens;
  const float* temperatures;
  int32_t *tokens, *accepted;
  float4* part;        // [b (s + 1)][splits]: maximum, its index, sum
  long long lb, ls, pb, ps;
  float ch, cl;        // log2(e) / T as two floats, where no temperatures are given; 0: greedy
  int b, s, vocab, splits;
  int held;            // elements of a CTA of k_verify_pick whose weights it keeps, or 0
};

// Logits are taken as finite: NaN counts as -inf (the maximum's other operand), +inf as the largest float.
__device__ __forceinline__ float logit(float x) { return fminf(fmaxf(x, -INFINITY), 3.402823466e38f); }

// Eight logits from element v on (those past the vocabulary: -inf), in 16-byte pieces where
// the row's address allows and the piece ends within the row.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int v, int vocab, bool wide, float* x) {
  constexpr int V = Ty<T>::kVec;
#pragma unroll
  for (int e = 0; e < 8; e += V) {
    if (wide && v + e + V <= vocab) {
      Ty<T>::load16(row + v + e, x + e);
#pragma unroll
      for (int u = 0; u < V; ++u) x[e + u] = logit(x[e + u]);
    } else {
#pragma unroll
      for (int u = 0; u < V; ++u) x[e + u] = v + e + u < vocab ? logit(Ty<T>::to_f(row[v + e + u])) : -INFINITY;
    }
  }
}
__device__ __forceinline__ bool wide_row(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
__device__ __forceinline__ float ex2(float x) {   // 2^-22 relative
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The temperature's factor of the logits, log2(e) / T, as two floats; 0: greedy.  (64-bit arithmetic runs at a hundredth of
// the fp32 rate: one thread, or the host, does what there is of it.)
__host__ __device__ inline void log2_factor(double t, float* ch, float* cl) {
  const double f = t >= 1e-30 ? 1.4426950408889634 / (t < 1e30 ? t : 1e30) : 0.0;
  *ch = static_cast<float>(f);
  *cl = static_cast<float>(f - *ch);
}
__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int seq) {
  return a.lens ? min(max(a.lens[seq], 0), a.s) : a.s;
}

// ------------------------------------------------------------------ rows
constexpr int kVrThreads = 256;

struct Best {
  float m;
  int at;
};
__device__ __forceinline__ Best better(Best x, Best y) {
  return y.m > x.m || (y.m == x.m && y.at < x.at) ? y : x;
}
__device__ __forceinline__ Best warp_best(Best x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Best y;
    y.m = __shfl_xor_sync(0xffffffffu, x.m, o);
    y.at = __shfl_xor_sync(0xffffffffu, x.at, o);
    x = better(x, y);
  }
  return x;
}

// CTA = (split of the vocabulary: 2048 N logits, row): its largest logit, the first index of it (greedy
// sequences), and the sum of 2^(c (l - max)).  The logits stay in registers between the two.
template <typename T, int N>
__global__ void __launch_bounds__(kVrThreads)
k_verify_rows(const __grid_constant__ VerifyArgs a) {
  __shared__ Best s_best[kVrThreads / 32];
  __shared__ float s_sum[kVrThreads / 32];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int row = blockIdx.y, seq = row / (a.s + 1), j = row - seq * (a.s + 1), tid = threadIdx.x;
  if (j > drafts_of(a, seq)) return;
  const T* l = static_cast<const T*>(a.logits) + seq * a.lb + j * a.ls;
  const bool wide = wide_row(l);
  float x[N][8], top = -INFINITY;
  const int v0 = blockIdx.x * (kVrThreads * 8 * N) + tid * 8;
#pragma unroll
  for (int n = 0; n < N; ++n) load8(l, v0 + n * (kVrThreads * 8), a.vocab, wide, x[n]);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e) top = fmaxf(top, x[n][e]);
  const float t = a.temperatures ? a.temperatures[seq] : 1.f;
  const float c = !a.temperatures ? a.ch : t >= 1e-30f ? __fdividef(1.44269504f, fminf(t, 1e30f)) : 0.f;
  Best best{top, a.vocab};
  if (c == 0.f)
#pragma unroll
    for (int n = N - 1; n >= 0; --n)
#pragma unroll
      for (int e = 7; e >= 0; --e)
        if (x[n][e] == top) best.at = v0 + n * (kVrThreads * 8) + e;
  best = warp_best(best);
  if ((tid & 31) == 0) s_best[tid >> 5] = best;
  __syncthreads();
  best = s_best[0];
#pragma unroll
  for (int w = 1; w < kVrThreads / 32; ++w) best = better(best, s_best[w]);
  float z = 0.f;
  if (best.m > -INFINITY)
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int e = 0; e < 8; ++e) z += ex2((x[n][e] - best.m) * c);
  z = warp_sum(z);
  if ((tid & 31) == 0) s_sum[tid >> 5] = z;
  __syncthreads();
  if (tid == 0) {
    z = 0.f;
#pragma unroll
    for (int w = 0; w < kVrThreads / 32; ++w) z += s_sum[w];
    a.part[static_cast<size_t>(row) * a.splits + blockIdx.x] = make_float4(best.m, __int_as_float(best.at), z, 0.f);
  }
}

// ------------------------------------------------------------------ whole-number weights
struct Exp {
  float m;          // the row's largest logit
  float ch, cl;     // log2(e) / T
  const ulonglong2* table;   // 2^(43 + j/64), rounded; its leading 24 bits and the rest as floats
};

// round(2^43 2^((l - m) log2(e) / T))
__device__ __forceinline__ unsigned long long weight_of(const Exp& e, float l) {
  // l - m and its error, times the factor, as a sum of two floats
  const float s = l - e.m, bb = s - l, err = (l - (s - bb)) + (-e.m - bb);
  const float th = s * e.ch;
  if (!(th >= -50.f)) return 0;   // below half a unit (-inf, too)
  const float tl = fmaf(s, e.ch, -th) + fmaf(s, e.cl, err * e.ch);
  const float kf = rintf(th * 64.f);
  const int k = static_cast<int>(kf);
  const float g = fmaf(kf, -1.f / 64.f, th);   // exact; |g| <= 1/128
  // 2^(g + tl) - 1 = yh + e2, y = (g + tl) ln 2
  const float yh = g * 0.693147182f;
  const float yl = fmaf(g, 0.693147182f, -yh) + fmaf(g, -1.90465421e-9f, tl * 0.693147182f);
  const float e2 = yl + yh * yh * fmaf(yh, fmaf(yh, 1.f / 24.f, 1.f / 6.f), 0.5f);
  const ulonglong2 t = e.table[k & 63];
  const float tf = __uint_as_float(static_cast<uint32_t>(t.y)), tr = __uint_as_float(static_cast<uint32_t>(t.y >> 32));
  const float ph = tf * yh, pl = fmaf(tf, yh, -ph) + fmaf(tr, yh, tf * e2);
  // the table's value is in [1, 2): ph below 2^-6, pl below 2^-14
  const float a0 = rintf(ph * 0x1p36f);
  const float b0 = rintf((pl + fmaf(a0, -0x1p-36f, ph)) * 0x1p43f);
  const unsigned long long w = t.x + (static_cast<long long>(static_cast<int>(a0)) << 7) + static_cast<long long>(static_cast<int>(b0));
  const int sh = -(k >> 6);   // 0 .. 50
  return sh ? ((w >> (sh - 1)) + 1) >> 1 : w;
}

// floor(f x) of a float f >= 0 (infinite or above: the largest) and a whole number.
__device__ __forceinline__ unsigned long long times(float f, unsigned long long x) {
  const uint32_t u = __float_as_uint(f);
  const int e = static_cast<int>(u >> 23) - 127 - 23;       // f = m 2^e, m < 2^24
  if (!(f > 0.f)) return 0;
  const unsigned long long m = u >> 23 ? (u & 0x7fffffu) | 0x800000u : (u & 0x7fffffu) << 1;
  const unsigned long long lo = m * x, hi = __umul64hi(m, x);   // below 2^88
  if (e >= 0) return hi || e > 40 || (lo >> (63 - e)) ? 0x7fffffffffffffffull : lo << e;
  const int r = -e;
  if (r >= 128) return 0;
  if (r >= 64) return hi >> (r - 64);
  return hi >> r ? 0x7fffffffffffffffull : (hi << (64 - r)) | (lo >> r);
}

// ------------------------------------------------------------------ pick
constexpr int kVpCtas = 8, kVpThreads = 512, kVpWarps = kVpThreads / 32;
constexpr int kVpChunk = 256;   // elements whose sum is kept, one warp's work: eight adjacent ones a lane

// 2^(43 + j/64), rounded; its leading 24 bits and the rest as floats.  (Made on the host once: 64-bit exponentials
// took the kernel 1.4 us.)
struct VerifyTable {
  ulonglong2 e[64];
};
static const VerifyTable& verify_table() {
  static const VerifyTable t = [] {
    VerifyTable v;
    for (int j = 0; j < 64; ++j) {
      const double x = std::exp2(j / 64.0);
      const float lead = static_cast<float>(x), rest = static_cast<float>(x - lead);
      uint32_t a, b;
      std::memcpy(&a, &lead, 4);
      std::memcpy(&b, &rest, 4);
      v.e[j].x = static_cast<unsigned long long>(std::llrint(x * 0x1p43));
      v.e[j].y = a | static_cast<unsigned long long>(b) << 32;
    }
    return v;
  }();
  return t;
}

struct PickShared {
  ulonglong2 table[64];
  unsigned long long cta[2][kVpCtas];   // the CTAs' sums
  unsigned long long warp[kVpWarps];
};

__device__ __forceinline__ unsigned long long warp_add(unsigned long long x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// Sum over the cluster; ahead: of the CTAs before this one.  `turn` alternates between calls.
__device__ __forceinline__ unsigned long long cluster_add(cg::cluster_group& cl, PickShared* sh, unsigned long long warp_sum,
                                                          int turn, unsigned long long* ahead) {
  const int tid = threadIdx.x;
  if ((tid & 31) == 0) sh->warp[tid >> 5] = warp_sum;
  __syncthreads();
  if (tid < kVpCtas) {
    unsigned long long x = 0;
    for (int w = 0; w < kVpWarps; ++w) x += sh->warp[w];
    *cl.map_shared_rank(&sh->cta[turn][cl.block_rank()], tid) = x;
  }
  cl.sync();
  unsigned long long all = 0, before = 0;
#pragma unroll
  for (unsigned u = 0; u < kVpCtas; ++u) {
    if (u < cl.block_rank()) before += sh->cta[turn][u];
    all += sh->cta[turn][u];
  }
  if (ahead) *ahead = before;
  return all;
}

// Cluster = sequence.  Every CTA decides the acceptance tests by itself (on the same
// numbers), a warp to a draft; the sampled row is dealt in chunks, a run of them to each CTA.
template <typename T>
__global__ void __cluster_dims__(kVpCtas, 1, 1) __launch_bounds__(kVpThreads, 2)
k_verify_pick(const __grid_constant__ VerifyArgs a, const __grid_constant__ VerifyTable table) {
  extern __shared__ unsigned long long s_chunk[];   // sums of this CTA's chunks, then (held) its weights
  __shared__ PickShared sh;
  __shared__ float s_top[kVpWarps], s_ch, s_cl;   // largest logits of the rows looked at, the factor
  __shared__ int s_at[kVpWarps], s_state[kVpWarps], s_yes;
  cg::cluster_group cl = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 64) sh.table[tid] = table.e[tid];
  tc::grid_dep_wait();
  const int seq = blockIdx.x / kVpCtas, n = drafts_of(a, seq), rank = cl.block_rank();
  if (tid == 0) {
    s_ch = a.ch;
    s_cl = a.cl;
    if (a.temperatures) log2_factor(a.temperatures[seq], &s_ch, &s_cl);
  }
  cl.sync();   // every CTA's shared memory is there
  const float ch = s_ch, cl_ = s_cl;
  const int chunks = (a.vocab + kVpChunk - 1) / kVpChunk, c0 = static_cast<int>(static_cast<long long>(chunks) * rank / kVpCtas),
            c1 = static_cast<int>(static_cast<long long>(chunks) * (rank + 1) / kVpCtas);
  const T* rows = static_cast<const T*>(a.logits) + seq * a.lb;
  unsigned long long* weights = s_chunk + c1 - c0;   // element 8 lane + e of a chunk at 32 e + lane
  const bool held = a.held > 0;
  int turn = 0;

  // The row's maximum, its index and its fp32 sum, from its splits (by one warp).
  auto row_stats = [&](int j, float* z_out) {
    const float4* p = a.part + (static_cast<size_t>(seq) * (a.s + 1) + j) * a.splits;
    Best best{-INFINITY, a.vocab};
    for (int u = lane; u < a.splits; u += 32) best = better(best, Best{p[u].x, __float_as_int(p[u].y)});
    best = warp_best(best);
    float z = 0.f;
    for (int u = lane; u < a.splits; u += 32)
      if (p[u].x > -INFINITY) z = fmaf(p[u].z, ex2((p[u].x - best.m) * ch), z);
    *z_out = warp_sum(z);
    return best;
  };
  // Whole-number sum of row j's weights, and of each of this CTA's chunks.
  auto row_sum = [&](int j, float top, unsigned long long* ahead) {
    const Exp e{top, ch, cl_, sh.table};
    const T* l = rows + j * a.ls;
    const bool wide = wide_row(l);
    unsigned long long sum = 0;
    for (int c = c0 + warp; c < c1; c += kVpWarps) {
      unsigned long long x = 0;
      float y[8];
      load8(l, c * kVpChunk + lane * 8, a.vocab, wide, y);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const unsigned long long w = weight_of(e, y[u]);
        if (held) weights[(c - c0) * kVpChunk + u * 32 + lane] = w;
        x += w;
      }
      x = warp_add(x);
      if (lane == 0) s_chunk[c - c0] = x;
      sum += x;
    }
    const unsigned long long all = cluster_add(cl, &sh, sum, turn, ahead);
    turn ^= 1;
    return all;
  };

  int j = 0;
  int j0 = 0;
  for (bool all = true; all;) {
    j0 = j;
    const int k = j0 + warp;
    if (k <= n) {
      float z;
      const Best best = row_stats(k, &z);
      if (lane == 0) {
        s_top[warp] = best.m;
        s_at[warp] = best.at;
      }
      if (lane == 0 && k < n) {
        const size_t at = static_cast<size_t>(seq) * a.s + k;
        const int y = a.drafts[at];
        int state = 0;   // 1: it stands; 2: too near to say
        if (static_cast<unsigned>(y) < static_cast<unsigned>(a.vocab) && best.m > -INFINITY) {
          const float q = a.probs ? a.probs[seq * a.pb + k * a.ps + y] : 1.f, u = a.accept[at];
          if (ch == 0.f) {
            state = y == best.at && static_cast<double>(u) * q < 1.0;
          } else {
            const float w = ex2((logit(Ty<T>::to_f(rows[k * a.ls + y])) - best.m) * ch), uz = u * q * z;
            // (below 2^-100 the products' roundings are not relative any more)
            state = !(fabsf(uz - w) > 0x1p-13f * w && (uz > 0x1p-100f || w > 0x1p-100f)) ? 2 : uz < w;
          }
        }
        s_state[warp] = state;
      }
    }
    __syncthreads();
    for (; j < min(n, j0 + kVpWarps); ++j) {
      int state = s_state[j - j0];
      if (state == 2) {
        const float top = s_top[j - j0];
        const unsigned long long z = row_sum(j, top, nullptr);
        if (tid == 0) {
          const size_t at = static_cast<size_t>(seq) * a.s + j;
          const int y = a.drafts[at];
          const double u = static_cast<double>(a.accept[at]) * (a.probs ? a.probs[seq * a.pb + j * a.ps + y] : 1.f);   // exact
          const double d = static_cast<double>(logit(Ty<T>::to_f(rows[j * a.ls + y]))) - top;
          s_yes = u * (static_cast<double>(z) * 0x1p-43) < exp2(d * (static_cast<double>(ch) + cl_));
        }
        __syncthreads();
        state = s_yes;
      }
      if (state != 1) {
        all = false;
        break;
      }
    }
    if (j == n && n < j0 + kVpWarps) all = false;
    if (all) __syncthreads();   // the states are written again
  }
  // the drafts that stand, and what follows them
  if (rank == 0) {
    for (int i = tid; i <= a.s; i += kVpThreads)
      if (i != j) a.tokens[static_cast<size_t>(seq) * (a.s + 1) + i] = i < j ? a.drafts[static_cast<size_t>(seq) * a.s + i] : -1;
    if (tid == 0) a.accepted[seq] = j;
  }
  int32_t* next = a.tokens + static_cast<size_t>(seq) * (a.s + 1) + j;
  const float top = s_top[j - j0];
  if (ch == 0.f || top == -INFINITY) {
    if (rank == 0 && tid == 0) *next = top == -INFINITY ? -1 : s_at[j - j0];
    return;
  }
  unsigned long long ahead, total = row_sum(j, top, &ahead);
  const Exp e{top, ch, cl_, sh.table};
  const T* l = rows + j * a.ls;
  const float* q = j < n && a.probs ? a.probs + seq * a.pb + j * a.ps : nullptr;
  const int out = j < n && !a.probs ? a.drafts[static_cast<size_t>(seq) * a.s + j] : -1;   // the token left out
  const unsigned long long z = total;
  // what is left of a lane's eight weights of chunk c
  bool plain = j == n;
  const bool wide_l = wide_row(l), wide_q = q && wide_row(q);
  auto left = [&](int c, unsigned long long* w) {
    const int v = c * kVpChunk + lane * 8;
    if (held) {
#pragma unroll
      for (int u = 0; u < 8; ++u) w[u] = weights[(c - c0) * kVpChunk + u * 32 + lane];
    } else {
      float y[8];
      load8(l, v, a.vocab, wide_l, y);
#pragma unroll
      for (int u = 0; u < 8; ++u) w[u] = weight_of(e, y[u]);
    }
    if (plain) return;
    if (!q) {
#pragma unroll
      for (int u = 0; u < 8; ++u) w[u] = v + u == out ? 0ull : w[u];
      return;
    }
    float y[8];
    load8(q, v, a.vocab, wide_q, y);   // (what is past the vocabulary has no weight)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const unsigned long long t = times(y[u], z);
      w[u] = w[u] > t ? w[u] - t : 0ull;
    }
  };
  auto left_sum = [&](unsigned long long* before) {
    unsigned long long sum = 0;
    for (int c = c0 + warp; c < c1; c += kVpWarps) {
      unsigned long long w[8], x = 0;
      left(c, w);
#pragma unroll
      for (int u = 0; u < 8; ++u) x += w[u];
      x = warp_add(x);
      if (lane == 0) s_chunk[c - c0] = x;
      sum += x;
    }
    const unsigned long long all = cluster_add(cl, &sh, sum, turn, before);
    turn ^= 1;
    return all;
  };
  if (!plain) {
    total = left_sum(&ahead);
    if (total == 0) {   // nothing left: from the row itself
      plain = true;
      total = left_sum(&ahead);
    }
  }
  // the first token whose running sum passes sample times the total
  const float r = a.sample[seq];
  const unsigned long long at = times(r >= 1.f ? 0x1.fffffep-1f : r, total);   // below the total
  __syncthreads();
  // the chunk (warp 0 of the CTA that has it), then the token in it
  if (warp == 0) {
    unsigned long long run = ahead;
    int found = -1;
    for (int c = c0; c < c1 && found < 0; c += 32) {
      const unsigned long long mine = c + lane < c1 ? s_chunk[c + lane - c0] : 0;
      unsigned long long x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, c + lane < c1 && run + x > at);
      if (past) {
        found = __ffs(past) - 1;
        run += __shfl_sync(0xffffffffu, x - mine, found);
        found += c;
      } else {
        run += __shfl_sync(0xffffffffu, x, 31);
      }
    }
    if (found >= 0 && ahead <= at) {
      unsigned long long w[8], mine = 0;
      left(found, w);
#pragma unroll
      for (int u = 0; u < 8; ++u) mine += w[u];
      unsigned long long x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, run + x > at);
      if (past && lane == __ffs(past) - 1) {
        run += x - mine;
        int u = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (run + w[k] <= at && u == k) {
            run += w[k];
            ++u;
          }
        *next = found * kVpChunk + lane * 8 + u;
      }
    }
  }
}

// Logits per CTA of k_verify_rows / 2048: four, where that still gives every SM of a GB300 two CTAs.  (Not asked of the device: the
// workspace's size goes by it, which is known without one.)
constexpr int kGbSms = 152;
static int verify_vectors(const shadowkv_verify_params& p) {
  const long long rows = static_cast<long long>(p.b) * (p.s + 1);
  for (int n = 4; n > 1; n /= 2)
    if (rows * ((p.vocab + 2048 * n - 1) / (2048 * n)) >= 2 * kGbSms) return n;
  return 1;
}
static int verify_splits(const shadowkv_verify_params& p) {
  const int per = 2048 * verify_vectors(p);
  return (p.vocab + per - 1) / per;
}

template <typename T>
static cudaError_t verify_t(VerifyArgs a, int n, cudaStream_t st) {
  const dim3 grid(a.splits, a.b * (a.s + 1)), block(kVrThreads);
  cudaError_t e = n == 4   ? launch_pdl(k_verify_rows<T, 4>, grid, block, 0, st, a)
                  : n == 2 ? launch_pdl(k_verify_rows<T, 2>, grid, block, 0, st, a)
                           : launch_pdl(k_verify_rows<T, 1>, grid, block, 0, st, a);
  if (e != cudaSuccess) return e;
  // a CTA keeps the weights of its share of the row in shared memory where two CTAs still fit on an SM (104,000
  // tokens); else it forms them twice
  const int chunks = (a.vocab + kVpChunk - 1) / kVpChunk, mine = (chunks + kVpCtas - 1) / kVpCtas;
  constexpr int kMost = 104 * 1024;
  size_t smem = mine * sizeof(unsigned long long);
  a.held = smem + static_cast<size_t>(mine) * kVpChunk * 8 <= kMost ? mine * kVpChunk : 0;
  smem += static_cast<size_t>(a.held) * 8;
  e = set_smem_once(reinterpret_cast<const void*>(k_verify_pick<T>), kMost);
  return e == cudaSuccess ? launch_pdl(k_verify_pick<T>, dim3(a.b * kVpCtas), dim3(kVpThreads), smem, st, a, verify_table()) : e;
}

static const char* verify_fault(const shadowkv_verify_params* p, skv_status* st) {
  *st = SKV_ERR_INVALID_ARG;
  if (!p) return "params is NULL";
  if (p->b < 0 || p->s < 0) return "b and s must be >= 0";
  if (p->vocab < 1) return "vocab must be >= 1";
  if (p->dtype != SKV_DTYPE_F32 && p->dtype != SKV_DTYPE_BF16) return "bad dtype";
  if (!(p->temperature >= 0.0) || !std::isfinite(p->temperature)) return "temperature must be finite and >= 0";
  if (p->logits_sb < 0 || p->logits_ss < 0 || p->probs_sb < 0 || p->probs_ss < 0) return "strides must not be negative";
  *st = SKV_ERR_UNSUPPORTED;
  if (p->vocab > 1 << 19) return "vocab must be at most 2^19";
  if (p->s > 65534 || static_cast<long long>(p->b) * (p->s + 1) > 65535) return "b * (s + 1) must be at most 65535";
  *st = SKV_OK;
  return nullptr;
}

}  // namespace skv

extern "C" {

size_t shadowkv_verify_workspace(const shadowkv_verify_params* p) try {
  skv_status st;
  if (const char* f = skv::verify_fault(p, &st)) {
    skv::set_error(st, f);
    return 0;
  }
  if (p->b == 0) return 256;
  return static_cast<size_t>(p->b) * (p->s + 1) * skv::verify_splits(*p) * sizeof(float4);
} catch (...) {   // host memory for an error text ran out
  return 0;
}

skv_status shadowkv_verify_drafts(const shadowkv_verify_params* p, const void* logits, const int32_t* drafts,
                                  const float* probs, const float* accept, const float* sample, const int32_t* lens,
                                  const float* temperatures, int32_t* tokens, int32_t* accepted, void* work,
                                  size_t work_bytes, void* stream) try {
  using skv::set_error;
  skv_status st;
  if (const char* f = skv::verify_fault(p, &st)) return set_error(st, f);
  if (p->b == 0) return SKV_OK;
  if (!logits || !sample || !tokens || !accepted || (p->s > 0 && (!drafts || !accept)))
    return set_error(SKV_ERR_INVALID_ARG, "a required pointer is NULL");
  const uintptr_t words = reinterpret_cast<uintptr_t>(drafts) | reinterpret_cast<uintptr_t>(probs) |
                          reinterpret_cast<uintptr_t>(accept) | reinterpret_cast<uintptr_t>(sample) |
                          reinterpret_cast<uintptr_t>(lens) | reinterpret_cast<uintptr_t>(temperatures) |
                          reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(accepted);
  if (words % 4 || reinterpret_cast<uintptr_t>(logits) % (p->dtype == SKV_DTYPE_BF16 ? 2 : 4))
    return set_error(SKV_ERR_INVALID_ARG, "pointers must be aligned to their elements");
  if (!work || reinterpret_cast<uintptr_t>(work) % 256)
    return set_error(SKV_ERR_INVALID_ARG, "the workspace must be non-NULL and 256-byte aligned");
  skv::VerifyArgs a;
  a.splits = skv::verify_splits(*p);
  if (work_bytes < static_cast<size_t>(p->b) * (p->s + 1) * a.splits * sizeof(float4))
    return set_error(SKV_ERR_INVALID_ARG, "the workspace is smaller than shadowkv_verify_workspace");
  a.logits = logits;
  a.drafts = drafts;
  a.probs = probs;
  a.accept = accept;
  a.sample = sample;
  a.lens = lens;
  a.temperatures = temperatures;
  a.tokens = tokens;
  a.accepted = accepted;
  a.part = static_cast<float4*>(work);
  a.lb = p->logits_sb; a.ls = p->logits_ss;
  a.pb = p->probs_sb; a.ps = p->probs_ss;
  skv::log2_factor(p->temperature, &a.ch, &a.cl);
  a.b = p->b; a.s = p->s; a.vocab = p->vocab;
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  const int n = skv::verify_vectors(*p);
  const cudaError_t e = p->dtype == SKV_DTYPE_BF16 ? skv::verify_t<skv::bf16>(a, n, q) : skv::verify_t<float>(a, n, q);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
