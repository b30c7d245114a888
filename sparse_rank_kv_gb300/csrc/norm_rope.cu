// Norm of query and key heads with the rotation to the token's position
// (shadowkv_qk_norm_rope): y = x / sqrt(mean x^2 + eps) w, then rotate-half
// over the first `rot` dimensions by pos theta^(-2i/rot).
//
// D/8 lanes hold a row, each with two 4-element pieces: a rotated lane the
// pieces at 4l and 4l + rot/2, so that a pair's two elements are in one
// thread; the other lanes two adjacent pieces.
#include <cmath>
#include <cstdint>

#include "common.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {

struct RopeFreq {
  unsigned long long f[64];   // theta^(-2i/rot) / (2 pi), in units of 2^-64 turns
};

struct NormRopeArgs {
  const void *x[2], *w[2];                 // q, k
  void* y[2];
  long long xb[2], xh[2], xs[2], yb[2], yh[2], ys[2];
  const int32_t* pos;
  uint32_t tokens;                         // b s
  int s, h_q, heads, chunk, rot, norm, per_token;
  float eps;
};

// Sine and cosine of pos f turns (f in units of 2^-64).  The product's low 64
// bits are the fraction of a turn, exact up to f's own rounding at any
// position; its top 32 bits are split into the nearest quarter and a rest
// within an eighth of a turn, which fp32 holds to 2^-28.
template <bool kFast>
__device__ __forceinline__ void rope_turn(long long pos, unsigned long long f, float* sn, float* cs) {
  const uint32_t u = static_cast<uint32_t>((static_cast<unsigned long long>(pos) * f + 0x80000000ull) >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float r = static_cast<float>(static_cast<int32_t>(u - (quarter << 30)));
  float s, c;
  // the hardware sine and cosine: within an eighth of a turn their errors are
  // absolute, near 2^-22, far below a bf16 result's rounding; fp32 keeps small sines, too
  if (kFast) __sincosf(r * (6.283185307179586f / 4294967296.f), &s, &c);
  else sincospif(r * (2.f / 4294967296.f), &s, &c);
  const float a = quarter & 1 ? c : s, b = quarter & 1 ? s : c;
  *sn = quarter & 2 ? -a : a;
  *cs = (quarter + 1) & 2 ? -b : b;
}

// 4 elements of a row, as loaded and as two float pairs.
template <typename T> struct Quad;
template <> struct Quad<float> {
  typedef float4 Raw;
  __device__ __forceinline__ static void get(Raw v, float2* o) {
    o[0] = make_float2(v.x, v.y);
    o[1] = make_float2(v.z, v.w);
  }
  __device__ __forceinline__ static Raw put(const float2* o) { return make_float4(o[0].x, o[0].y, o[1].x, o[1].y); }
};
template <> struct Quad<bf16> {
  typedef uint2 Raw;
  __device__ __forceinline__ static void get(Raw v, float2* o) {
    o[0] = make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u));
    o[1] = make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u));
  }
  __device__ __forceinline__ static Raw put(const float2* o) {
    __nv_bfloat162 a = __float22bfloat162_rn(o[0]), b = __float22bfloat162_rn(o[1]);
    return make_uint2(*reinterpret_cast<uint32_t*>(&a), *reinterpret_cast<uint32_t*>(&b));
  }
};

constexpr int kNrThreads = 256;
constexpr int kNrTokens = 4;    // tokens per CTA
constexpr int kNrCtas = 5;      // per SM (48 registers)

// CTA = 4 tokens x `chunk` heads.  The tokens' sines and cosines are formed
// once, a pair per thread, and every D/8-lane group keeps its token's in
// registers over its heads, which it loads two (fp32: one) at a time; the other
// CTAs of the SM cover its loads.  The arithmetic is on pairs (fma.f32x2).
// Measured at 32768 tokens of 32 + 8 heads of 128 in bf16 (671 MB): 101 us, 6.6
// TB/s, bound by DRAM; without the L2 prefetch 116 us, then with scalar
// arithmetic 141 us (bound by its instructions), with four CTAs per SM 122 us, with four rows at
// a time 147 us, with the next rows prefetched into registers 144 us.
template <typename T, int D>
__global__ void __launch_bounds__(kNrThreads, kNrCtas)
k_norm_rope(const __grid_constant__ NormRopeArgs a, const __grid_constant__ RopeFreq freq) {
  constexpr int LPR = D / 8, Sub = kNrThreads / LPR / kNrTokens;   // row groups per token
  constexpr int Rows = 4 / sizeof(T);                              // rows in flight per group
  typedef typename Quad<T>::Raw Raw;
  __shared__ float2 s_cs[kNrTokens][D / 2];
  // no early launch of dependents: the decode step's selection reads the new
  // token's key, this kernel's output, before its own grid-dependency wait
  const int half = a.rot >> 1;
  const uint32_t tok0 = blockIdx.x * kNrTokens;
  tc::grid_dep_wait();
  auto place = [&](uint32_t token, int* i, int* t) {
    *i = static_cast<int>(token / static_cast<uint32_t>(a.s));
    *t = static_cast<int>(token - static_cast<uint32_t>(*i) * static_cast<uint32_t>(a.s));
  };
  const int l = threadIdx.x % LPR, grp = threadIdx.x / LPR, u = grp / Sub, sub = grp % Sub;
  const uint32_t token = tok0 + u;
  const bool live = token < a.tokens;
  int i = 0, t = 0;
  if (live) place(token, &i, &t);
  const int c0 = blockIdx.y * a.chunk, c1 = min(a.heads, c0 + a.chunk);
  // with several rounds of rows ahead, all of them go to L2 while the angles are formed
  for (int h = c0 + sub + l * Sub; live && a.chunk > Sub * Rows && h < c1; h += Sub * LPR) {
    const int w = h < a.h_q ? 0 : 1;
    const char* p = reinterpret_cast<const char*>(static_cast<const T*>(a.x[w]) + i * a.xb[w] + t * a.xs[w] +
                                                  (w ? h - a.h_q : h) * a.xh[w]);
#pragma unroll
    for (int e = 0; e < D * static_cast<int>(sizeof(T)); e += 128)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p + e));
  }
  for (int e = threadIdx.x; e < kNrTokens * half; e += kNrThreads) {
    const int u = e / half, p = e - u * half;
    if (tok0 + u >= a.tokens) break;
    int i, t;
    place(tok0 + u, &i, &t);
    const long long pos = !a.pos ? t : a.per_token ? a.pos[tok0 + u] : static_cast<long long>(a.pos[i]) + t;
    float sn, cs;
    rope_turn<sizeof(T) == 2>(pos, freq.f[p], &sn, &cs);
    s_cs[u][p] = make_float2(cs, sn);
  }
  __syncthreads();
  const int nrot = a.rot >> 3;
  const bool turned = l < nrot;
  const int o0 = turned ? 4 * l : a.rot + 8 * (l - nrot);
  const int o1 = turned ? 4 * l + half : o0 + 4;
  float2 cs[2], sn[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float2 x = turned ? s_cs[u][4 * l + 2 * e] : make_float2(1.f, 0.f);
    const float2 y = turned ? s_cs[u][4 * l + 2 * e + 1] : make_float2(1.f, 0.f);
    cs[e] = make_float2(x.x, y.x);
    sn[e] = make_float2(x.y, y.y);
  }
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    // this part's heads of the chunk, as indexes into q or k
    const int base = which ? a.h_q : 0;
    const int h0 = max(c0, base) - base, h1 = min(c1, which ? a.heads : a.h_q) - base;
    if (h0 >= h1) continue;
    const long long xh = a.xh[which], yh = a.yh[which];
    const int first = h0 + sub;
    const int mine = live && first < h1 ? (h1 - first + Sub - 1) / Sub : 0;   // rows of this group
    const T* src = static_cast<const T*>(a.x[which]) + i * a.xb[which] + t * a.xs[which] + first * xh;
    T* dst = static_cast<T*>(a.y[which]) + i * a.yb[which] + t * a.ys[which] + first * yh;
    float2 w[4] = {{1.f, 1.f}, {1.f, 1.f}, {1.f, 1.f}, {1.f, 1.f}};
    if (a.norm && a.w[which]) {
      Quad<T>::get(*reinterpret_cast<const Raw*>(static_cast<const T*>(a.w[which]) + o0), w);
      Quad<T>::get(*reinterpret_cast<const Raw*>(static_cast<const T*>(a.w[which]) + o1), w + 2);
    }
    const int most = (h1 - h0 + Sub - 1) / Sub;   // the same count for every lane of the warp
    for (int n = 0; n < most; n += Rows) {
      Raw r0[Rows], r1[Rows];
#pragma unroll
      for (int v = 0; v < Rows; ++v) {
        r0[v] = Raw{};
        r1[v] = Raw{};
        if (n + v < mine) {
          const T* p = src + v * Sub * xh;
          r0[v] = *reinterpret_cast<const Raw*>(p + o0);
          r1[v] = *reinterpret_cast<const Raw*>(p + o1);
        }
      }
      src += Rows * Sub * xh;
#pragma unroll
      for (int v = 0; v < Rows; ++v) {
        float2 x[4];
        Quad<T>::get(r0[v], x);
        Quad<T>::get(r1[v], x + 2);
        if (a.norm) {
          float2 s2 = __fmul2_rn(x[0], x[0]);
#pragma unroll
          for (int e = 1; e < 4; ++e) s2 = __ffma2_rn(x[e], x[e], s2);
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(fmaf(ss, 1.f / D, a.eps));
          const float2 rr = make_float2(r, r);
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = __fmul2_rn(__fmul2_rn(x[e], rr), w[e]);
        }
        if (turned) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float2 x1 = x[e], x2 = x[2 + e], m = __fmul2_rn(x2, sn[e]);
            x[e] = __ffma2_rn(x1, cs[e], make_float2(-m.x, -m.y));
            x[2 + e] = __ffma2_rn(x2, cs[e], __fmul2_rn(x1, sn[e]));
          }
        }
        if (n + v < mine) {
          T* p = dst + v * Sub * yh;
          *reinterpret_cast<Raw*>(p + o0) = Quad<T>::put(x);
          *reinterpret_cast<Raw*>(p + o1) = Quad<T>::put(x + 2);
        }
      }
      dst += Rows * Sub * yh;
    }
  }
}

static cudaError_t launch_norm_rope(const shadowkv_norm_rope_params& p, NormRopeArgs& a, const RopeFreq& f,
                                    cudaStream_t st) {
  const long long groups = (static_cast<long long>(a.tokens) + kNrTokens - 1) / kNrTokens;
  // all heads in one CTA, which then forms its angles once, or with few
  // tokens the heads split over up to 400 CTAs.  Measured at 32 + 8 heads of 128
  // in bf16, all in one against one head per row group: 8 tokens 5.3 and 2.7 us,
  // 512 tokens 5.5 and 7.7 (as split here 5.3), 2048 tokens 9.4 and 23.7
  const int sub = kNrThreads / (p.d / 8) / kNrTokens;
  const int most = (a.heads + sub - 1) / sub;
  const int parts = static_cast<int>(groups >= 400 ? 1 : 400 / groups < most ? 400 / groups : most);
  a.chunk = ((a.heads + parts - 1) / parts + sub - 1) / sub * sub;
  const dim3 grid(static_cast<unsigned>(groups), (a.heads + a.chunk - 1) / a.chunk);
  const bool bf = p.dtype == SKV_DTYPE_BF16;
  auto k = bf ? (p.d == 128 ? k_norm_rope<bf16, 128> : k_norm_rope<bf16, 64>)
              : (p.d == 128 ? k_norm_rope<float, 128> : k_norm_rope<float, 64>);
  return launch_pdl(k, grid, dim3(kNrThreads), 0, st, a, f);
}

// The frequencies of one (theta, rot), kept for the thread's next call with the
// same ones (64 extended-precision powers take longer than the kernel).
static const RopeFreq& rope_freq(float theta, int rot) {
  thread_local RopeFreq f;
  thread_local float have_theta = -1.f;
  thread_local int have_rot = -1;
  if (have_theta != theta || have_rot != rot) {
    const long double two_pi = 6.283185307179586476925286766559005768L;
    for (int i = 0; i < rot / 2; ++i) {
      const long double turns = powl(static_cast<long double>(theta), -2.0L * i / rot) / two_pi;
      const long double frac = turns - floorl(turns);
      f.f[i] = static_cast<unsigned long long>(ldexpl(frac, 63)) << 1;
    }
    have_theta = theta;
    have_rot = rot;
  }
  return f;
}

// b x heads x s x d rows of E-byte elements: pointer and strides in whole
// 4-element pieces (a stride nothing is reached by, of one sequence, head or
// token, is not looked at); an output's tokens must not share rows.
static const char* rows_fault(const shadowkv_rows& r, int b, int h, int s, int E, bool out) {
  if (!r.ptr) return "a row pointer is NULL";
  if (reinterpret_cast<uintptr_t>(r.ptr) % (4 * E)) return "row pointers must be aligned to 4 elements";
  const long long sb = b > 1 ? r.sb : 4, sh = h > 1 ? r.sh : 4, ss = s > 1 ? r.ss : 4;
  if (sb < 0 || sh < 0 || ss < 0) return "row strides must not be negative";
  if (sb % 4 || sh % 4 || ss % 4) return "row strides must be multiples of 4 elements";
  if (out && (!sb || !sh || !ss)) return "an output stride is 0";
  return nullptr;
}

}  // namespace skv

extern "C" skv_status shadowkv_qk_norm_rope(const shadowkv_norm_rope_params* p, const shadowkv_rows* q,
                                            const shadowkv_rows* k, const void* q_weight, const void* k_weight,
                                            const int32_t* pos, const shadowkv_rows* q_out,
                                            const shadowkv_rows* k_out, void* stream) try {
  using skv::set_error;
  if (!p) return set_error(SKV_ERR_INVALID_ARG, "params is NULL");
  if (!q && !k) return set_error(SKV_ERR_INVALID_ARG, "q and k are both NULL");
  if ((q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return set_error(SKV_ERR_INVALID_ARG, "q and q_out, k and k_out must be given together");
  if ((!q && q_weight) || (!k && k_weight)) return set_error(SKV_ERR_INVALID_ARG, "a weight without its rows");
  const int hq = q ? p->h_q : 0, hk = k ? p->h_kv : 0;
  if (p->b < 0 || p->s < 0 || (q && hq < 1) || (k && hk < 1))
    return set_error(SKV_ERR_INVALID_ARG, "need b, s >= 0 and h_q, h_kv >= 1");
  if (hq > 65536 || hk > 65536) return set_error(SKV_ERR_UNSUPPORTED, "more than 65536 heads");
  if (static_cast<long long>(p->b) * p->s >= (1LL << 31))
    return set_error(SKV_ERR_UNSUPPORTED, "b * s must be < 2^31");
  if (p->d != 64 && p->d != 128) return set_error(SKV_ERR_UNSUPPORTED, "d must be 64 or 128");
  if (p->rot < 0 || p->rot > p->d || p->rot % 8)
    return set_error(SKV_ERR_INVALID_ARG, "rot must be a multiple of 8 in 0..d");
  if (p->dtype != SKV_DTYPE_F32 && p->dtype != SKV_DTYPE_BF16) return set_error(SKV_ERR_INVALID_ARG, "bad dtype");
  if (p->norm != 0 && p->norm != 1) return set_error(SKV_ERR_INVALID_ARG, "norm must be 0 or 1");
  if (p->pos_per_token != 0 && p->pos_per_token != 1)
    return set_error(SKV_ERR_INVALID_ARG, "pos_per_token must be 0 or 1");
  if (p->norm && (!(p->eps > 0.f) || !std::isfinite(p->eps)))
    return set_error(SKV_ERR_INVALID_ARG, "eps must be > 0 and finite");
  if (p->rot && (!(p->theta > 0.f) || !std::isfinite(p->theta)))
    return set_error(SKV_ERR_INVALID_ARG, "theta must be > 0 and finite");
  if (p->b == 0 || p->s == 0) return SKV_OK;
  const int E = p->dtype == SKV_DTYPE_BF16 ? 2 : 4;
  const shadowkv_rows* in[2] = {q, k};
  const shadowkv_rows* out[2] = {q_out, k_out};
  const void* w[2] = {q_weight, k_weight};
  skv::NormRopeArgs a{};
  for (int i = 0; i < 2; ++i) {
    if (!in[i]) continue;
    const char* f = skv::rows_fault(*in[i], p->b, i ? hk : hq, p->s, E, false);
    if (!f) f = skv::rows_fault(*out[i], p->b, i ? hk : hq, p->s, E, true);
    if (!f && reinterpret_cast<uintptr_t>(w[i]) % (4 * E)) f = "weights must be aligned to 4 elements";
    if (f) return set_error(SKV_ERR_INVALID_ARG, f);
    a.x[i] = in[i]->ptr;
    a.xb[i] = in[i]->sb; a.xh[i] = in[i]->sh; a.xs[i] = in[i]->ss;
    a.y[i] = out[i]->ptr;
    a.yb[i] = out[i]->sb; a.yh[i] = out[i]->sh; a.ys[i] = out[i]->ss;
    a.w[i] = w[i];
  }
  if (reinterpret_cast<uintptr_t>(pos) % 4) return set_error(SKV_ERR_INVALID_ARG, "pos must be 4-byte aligned");
  a.pos = pos;
  a.s = p->s;
  a.tokens = static_cast<uint32_t>(p->b) * static_cast<uint32_t>(p->s);
  a.h_q = hq;
  a.heads = hq + hk;
  a.rot = p->rot;
  a.norm = p->norm;
  a.per_token = p->pos_per_token;
  a.eps = p->eps;
  const cudaError_t e = skv::launch_norm_rope(*p, a, skv::rope_freq(p->theta, p->rot), static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  return SKV_OK;
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}
