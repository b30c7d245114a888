// Device view of the 8-bit block cache (include/shadowkv.h) and the helpers
// its kernels share.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/shadowkv.h"
#include "common.cuh"

namespace skv {

struct CacheDev {
  uint8_t *kc, *vc;
  float *ks, *vs;
  int32_t *table, *n_tok;
  float* weight;
  int* status;
  int pairs, h_kv, max_blocks, n_pool;
  int shift;   // block = 1 << shift
};

inline CacheDev cache_dev(const shadowkv_cache& c) {
  CacheDev d;
  d.kc = static_cast<uint8_t*>(c.k_codes);
  d.vc = static_cast<uint8_t*>(c.v_codes);
  d.ks = c.k_scale;
  d.vs = c.v_scale;
  d.table = c.table;
  d.n_tok = c.n_tok;
  d.weight = c.weight;
  d.status = c.status;
  d.pairs = c.b * c.h_kv;
  d.h_kv = c.h_kv;
  d.max_blocks = c.max_blocks;
  d.n_pool = c.n_pool;
  d.shift = c.block == 16 ? 4 : c.block == 32 ? 5 : c.block == 64 ? 6 : 7;
  return d;
}

// Tokens a pair holds; a count out of range is recorded and clamped.
__device__ __forceinline__ int cache_tokens(const CacheDev& c, int pair) {
  const int n = c.n_tok[pair], cap = c.max_blocks << c.shift;
  if (n >= 0 && n <= cap) return n;
  flag_error(c.status, DEV_BAD_COUNT);
  return n < 0 ? 0 : cap;
}

// Pool block of a pair's block i, or -1; an id out of range is recorded.
__device__ __forceinline__ int cache_block_or_none(const CacheDev& c, int pair, int i) {
  const int id = c.table[static_cast<size_t>(pair) * c.max_blocks + i];
  if (static_cast<unsigned>(id) < static_cast<unsigned>(c.n_pool)) return id;
  flag_error(c.status, DEV_BAD_SLOT);
  return -1;
}

// The same for kernels that only read: block 0 for an id out of range.
__device__ __forceinline__ int cache_block(const CacheDev& c, int pair, int i) {
  return max(cache_block_or_none(c, pair, i), 0);
}

// The smallest power of two 2^e, e >= -100, with amax <= 448 2^e
// (448 = 1.75 2^8, the largest e4m3 value); amax finite and not negative.
__device__ __forceinline__ float cache_scale_of(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, -100);
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Two floats to two e4m3 codes (the first in the low byte), rounded to
// nearest even, saturated to +-448; NaN stays NaN.
__device__ __forceinline__ uint32_t e4m3_pack2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3_unpack2(uint32_t c2) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c2 & 0xffffu), __NV_E4M3);
  return __half22float2(__half2(h));
}

}  // namespace skv
