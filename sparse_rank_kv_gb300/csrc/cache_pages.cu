// The 8-bit block cache's pool as one that sequences share: every pool block has
// a count of the table entries that name it, and a block with the count 0 is free.
//   shadowkv_cache_share     forks: tables copied, counts raised, no codes moved
//   shadowkv_cache_reserve   room for an append: free blocks handed out, and a
//                            partly filled block that others name too copied first
//   shadowkv_cache_truncate  tokens taken off the end, their blocks given back
//   shadowkv_cache_compact   the blocks in use moved to the start of another pool
//
// The counts are the only state: who gets which block follows from them alone (the
// lowest free ids, in order of sequence, head and entry), so a call's result does not
// depend on timing, and a cache's copy of tables and counts is a whole one.
#include <cooperative_groups.h>

#include <cstdint>
#include <mutex>

#include "cache.cuh"
#include "internal.h"
#include "tc.cuh"

namespace skv {
namespace cg = cooperative_groups;

__device__ __forceinline__ bool in_pool(const CacheDev& c, int id) {
  return static_cast<unsigned>(id) < static_cast<unsigned>(c.n_pool);
}

// One table entry less names block `id`.
__device__ __forceinline__ void give_back(const CacheDev& c, int32_t* refs, int id) {
  if (in_pool(c, id)) {
    if (atomicSub(&refs[id], 1) <= 0) flag_error(c.status, DEV_BAD_COUNT);
  } else if (id != -1) {
    flag_error(c.status, DEV_BAD_SLOT);
  }
}

// ------------------------------------------------------------------ share
constexpr int kPgThreads = 256;

// CTA = (fork, KV head, kPgThreads table entries).  A few dependent loads and one
// write per entry: latency bounds it.
__global__ void __launch_bounds__(kPgThreads)
k_share(const __grid_constant__ CacheDev c, int32_t* refs, int b, int n, const int32_t* src, const int32_t* dst) {
  tc::grid_dep_wait();
  const int k = blockIdx.x / c.h_kv, g = blockIdx.x - k * c.h_kv, tid = threadIdx.x;
  const int s = src[k], d = dst[k];
  bool bad = static_cast<unsigned>(s) >= static_cast<unsigned>(b) || static_cast<unsigned>(d) >= static_cast<unsigned>(b);
  // a sequence that another fork reads, or that an earlier one writes, is not written
  for (int u = tid; u < n; u += kPgThreads) bad |= src[u] == d || (u < k && dst[u] == d);
  if (__syncthreads_or(bad)) {
    if (tid == 0) flag_error(c.status, DEV_BAD_SEQUENCE);
    return;
  }
  const int from = s * c.h_kv + g, to = d * c.h_kv + g, tok = cache_tokens(c, from);
  const int nb = (tok + (1 << c.shift) - 1) >> c.shift, i = blockIdx.y * kPgThreads + tid;
  if (i >= c.max_blocks) return;
  const size_t rf = static_cast<size_t>(from) * c.max_blocks + i, rt = static_cast<size_t>(to) * c.max_blocks + i;
  int id = i < nb ? c.table[rf] : -1;
  if (i < nb && !in_pool(c, id)) {
    flag_error(c.status, DEV_BAD_SLOT);
    id = -1;
  }
  give_back(c, refs, c.table[rt]);
  if (id >= 0) atomicAdd(&refs[id], 1);
  c.table[rt] = id;
  if (c.weight) c.weight[rt] = c.weight[rf];
  if (i == 0) c.n_tok[to] = tok;
}

// --------------------------------------------------------------- truncate
// CTA = pair.
__global__ void __launch_bounds__(kPgThreads)
k_truncate(const __grid_constant__ CacheDev c, int32_t* refs, const int32_t* drop) {
  tc::grid_dep_wait();
  const int pair = blockIdx.x, tid = threadIdx.x;
  int off = drop ? drop[pair / c.h_kv] : 0;
  if (off < 0) {
    if (tid == 0) flag_error(c.status, DEV_BAD_COUNT);
    off = 0;
  }
  const int was = cache_tokens(c, pair), tok = max(was - off, 0);
  __syncthreads();   // every thread has the old count
  if (tid == 0) c.n_tok[pair] = tok;
  const size_t row = static_cast<size_t>(pair) * c.max_blocks;
  for (int i = ((tok + (1 << c.shift) - 1) >> c.shift) + tid; i < c.max_blocks; i += kPgThreads) {
    if (refs) {
      give_back(c, refs, c.table[row + i]);
      c.table[row + i] = -1;
    }
    if (c.weight) c.weight[row + i] = 0.f;
  }
}

// ------------------------------------------------- numbering a list's members
// A cluster of kClCtas CTAs walks a list once to count its members and once more to
// number them in order: every warp takes a run of the list, and the counts of the
// warps before it come from its CTA's and the other CTAs' shared memory.
constexpr int kClCtas = 8, kClThreads = 1024, kClWarps = kClCtas * kClThreads / 32;

struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run warp_run(int n, unsigned rank) {
  const int per = (static_cast<int>((static_cast<long long>(n) + kClWarps - 1) / kClWarps) + 31) / 32 * 32;
  const long long lo = static_cast<long long>(per) * (rank * (kClThreads / 32) + threadIdx.x / 32);
  return {static_cast<int>(min(lo, static_cast<long long>(n))), static_cast<int>(min(lo + per, static_cast<long long>(n)))};
}
template <typename F>
__device__ __forceinline__ int count_run(Run r, F&& member) {
  const int lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll 4
  for (int i = r.lo; i < r.hi; i += 32) n += __popc(__ballot_sync(0xffffffffu, i + lane < r.hi && member(i + lane)));
  return n;
}
// visit(i, number of members before i, is one) for every i of the run
template <typename F, typename V>
__device__ __forceinline__ void number_run(Run r, int before, F&& member, V&& visit) {
  const int lane = threadIdx.x & 31;
#pragma unroll 4
  for (int i = r.lo; i < r.hi; i += 32) {
    const bool on = i + lane < r.hi && member(i + lane);
    const uint32_t bal = __ballot_sync(0xffffffffu, on);
    if (i + lane < r.hi) visit(i + lane, before + __popc(bal & ((1u << lane) - 1u)), on);
    before += __popc(bal);
  }
}
// Members before this warp's run (one count per warp given by every lane) and in all.
__device__ __forceinline__ int before_run(cg::cluster_group& cl, int mine, int* s_scan, int* s_tot, int* total) {
  const int lane = threadIdx.x & 31;
  int cta;
  const int before = block_exclusive_scan(lane == 0 ? mine : 0, s_scan, &cta);
  if (threadIdx.x < kClCtas) *cl.map_shared_rank(&s_tot[cl.block_rank()], threadIdx.x) = cta;
  cl.sync();
  int ahead = 0, all = 0;
#pragma unroll
  for (unsigned u = 0; u < kClCtas; ++u) {
    if (u < cl.block_rank()) ahead += s_tot[u];
    all += s_tot[u];
  }
  *total = all;
  return ahead + __shfl_sync(0xffffffffu, before, 0);
}

// ---------------------------------------------------------------- reserve
struct ReserveArgs {
  CacheDev c;
  int32_t* refs;
  const int32_t* lens;
  int32_t* granted;
  int32_t* rank;     // [pairs][slots]: a needed block's number, or -1
  int32_t* start;    // [b + 1]: blocks needed by the sequences before
  int32_t* list;     // free ids, ascending
  int2* copy;        // [pairs]: block copied, and where to (or -1)
  int b, s, slots;   // slots: table entries an append of s tokens can touch
};

__device__ __forceinline__ int reserve_len(const ReserveArgs& a, int seq) {
  const int n = a.lens ? a.lens[seq] : a.s;
  return min(max(n, 0), a.s);
}

// One cluster: which entries need a block (slot k of a pair: its k-th entry from the
// one the next token goes to), the needs and the free blocks numbered, then handed
// out.  Latency of the walks and of the cluster's barriers
// bounds it (profiled: 16 us for 48 sequences over 55,000 blocks).
__global__ void __cluster_dims__(kClCtas, 1, 1) __launch_bounds__(kClThreads)
k_reserve(const __grid_constant__ ReserveArgs a) {
  __shared__ int s_scan[32], s_tot[2][kClCtas];
  cg::cluster_group cl = cg::this_cluster();
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const CacheDev& c = a.c;
  const int B = 1 << c.shift, E = a.slots, items = c.pairs * E;
  const int me = static_cast<int>(cl.block_rank()) * kClThreads + threadIdx.x, all = kClCtas * kClThreads;
  for (int i = me; i < a.b; i += all) {
    if (a.lens && static_cast<unsigned>(a.lens[i]) > static_cast<unsigned>(a.s)) flag_error(c.status, DEV_BAD_COUNT);
    a.granted[i] = reserve_len(a, i);
  }
  cl.sync();
  for (int x = me; x < items; x += all) {
    const int pair = x / E, k = x - pair * E, seq = pair / c.h_kv, len = reserve_len(a, seq);
    const int tok = cache_tokens(c, pair), e = (tok >> c.shift) + k;
    bool need = false;
    if (tok + static_cast<long long>(len) > static_cast<long long>(c.max_blocks) * B) {
      a.granted[seq] = -1;   // more than the table holds
    } else if (static_cast<long long>(e) * B < tok + static_cast<long long>(len)) {
      const int id = c.table[static_cast<size_t>(pair) * c.max_blocks + e];
      const bool have = in_pool(c, id), partial = k == 0 && (tok & (B - 1));
      if (!have && (id != -1 || partial)) flag_error(c.status, DEV_BAD_SLOT);
      if (!have && partial) a.granted[seq] = -1;   // tokens without a block
      const int r = have ? a.refs[id] : 0;
      if (have && r < 1) flag_error(c.status, DEV_BAD_COUNT);
      need = r != 1;
    }
    a.rank[x] = need;
  }
  cl.sync();
  const Run pool = warp_run(c.n_pool, cl.block_rank()), mine = warp_run(items, cl.block_rank());
  const auto is_free = [&](int i) { return a.refs[i] == 0; };
  const auto needs = [&](int x) { return a.rank[x] && a.granted[x / E / c.h_kv] >= 0; };
  int nfree, total;
  const int f0 = before_run(cl, count_run(pool, is_free), s_scan, s_tot[0], &nfree);
  const int n0 = before_run(cl, count_run(mine, needs), s_scan, s_tot[1], &total);
  if (f0 < total) number_run(pool, f0, is_free, [&](int i, int r, bool on) { if (on && r < total) a.list[r] = i; });
  number_run(mine, n0, needs, [&](int x, int r, bool on) {
    a.rank[x] = on ? r : -1;
    if (x % (E * c.h_kv) == 0) a.start[x / (E * c.h_kv)] = r;
  });
  if (me == 0) a.start[a.b] = total;
  cl.sync();
  for (int x = me; x < items; x += all) {
    const int pair = x / E, k = x - pair * E, seq = pair / c.h_kv, r = a.rank[x];
    // a sequence gets all its blocks or none
    const bool ok = a.start[seq + 1] <= nfree || a.start[seq + 1] == a.start[seq];
    int2 cp = make_int2(-1, -1);
    if (r >= 0 && ok) {
      const int tok = cache_tokens(c, pair);
      int32_t* entry = c.table + static_cast<size_t>(pair) * c.max_blocks + (tok >> c.shift) + k;
      const int old = *entry, id = a.list[r];
      if (in_pool(c, old)) {
        atomicSub(&a.refs[old], 1);
        if (k == 0 && (tok & (B - 1))) cp = make_int2(old, id);
      }
      a.refs[id] = 1;
      *entry = id;
    }
    if (k == 0) a.copy[pair] = cp;
    if (x % (E * c.h_kv) == 0 && (!ok || a.granted[seq] < 0)) a.granted[seq] = 0;
  }
}

// Codes and scales of one block to another.  Memory bounds it: a compaction that moves 1.18 GB (read and
// written) takes 223 us with its numbering, 5.3 TB/s.
__device__ __forceinline__ void copy_codes(const CacheDev& from, int id, const CacheDev& to, int id2, int d, int tid, int nt) {
  const int n16 = d << from.shift >> 4;
  const uint4* k0 = reinterpret_cast<const uint4*>(from.kc) + static_cast<size_t>(id) * n16;
  const uint4* v0 = reinterpret_cast<const uint4*>(from.vc) + static_cast<size_t>(id) * n16;
  uint4* k1 = reinterpret_cast<uint4*>(to.kc) + static_cast<size_t>(id2) * n16;
  uint4* v1 = reinterpret_cast<uint4*>(to.vc) + static_cast<size_t>(id2) * n16;
  // four pieces of each in flight, read once and not kept
  for (int i = tid; i < n16; i += 4 * nt) {
    uint4 k[4], v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * nt < n16) {
        k[u] = __ldcs(k0 + i + u * nt);
        v[u] = __ldcs(v0 + i + u * nt);
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i + u * nt < n16) {
        __stcs(k1 + i + u * nt, k[u]);
        __stcs(v1 + i + u * nt, v[u]);
      }
  }
  if (tid == 0) {
    to.ks[id2] = from.ks[id];
    to.vs[id2] = from.vs[id];
  }
}

// CTA = pair: its partly filled block, where it was shared.
__global__ void __launch_bounds__(kPgThreads)
k_reserve_copy(const __grid_constant__ CacheDev c, int d, const int2* copy) {
  tc::grid_dep_wait();
  const int2 cp = copy[blockIdx.x];
  if (cp.x >= 0) copy_codes(c, cp.x, c, cp.y, d, threadIdx.x, kPgThreads);
}

// ---------------------------------------------------------------- compact
struct CompactArgs {
  CacheDev c, to;
  const int32_t* refs;
  int32_t* to_refs;
  int32_t* number;   // [n_pool]: a block's place in the new pool, or -1
  int32_t* list;     // [n_pool]: the blocks in use, ascending
  int32_t* count;    // blocks in use, or -1 where the new pool has too few
  int d;
};

__global__ void __cluster_dims__(kClCtas, 1, 1) __launch_bounds__(kClThreads)
k_compact_number(const __grid_constant__ CompactArgs a) {
  __shared__ int s_scan[32], s_tot[kClCtas];
  cg::cluster_group cl = cg::this_cluster();
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  cl.sync();   // every CTA's shared memory is there
  const Run pool = warp_run(a.c.n_pool, cl.block_rank());
  const auto live = [&](int i) { return a.refs[i] > 0; };
  int total;
  const int n0 = before_run(cl, count_run(pool, live), s_scan, s_tot, &total);
  const bool fits = total <= a.to.n_pool;
  number_run(pool, n0, live, [&](int i, int r, bool on) {
    a.number[i] = on && fits ? r : -1;
    if (on && fits) {
      a.list[r] = i;
      a.to_refs[r] = a.refs[i];
    }
  });
  const int me = static_cast<int>(cl.block_rank()) * kClThreads + threadIdx.x;
  for (int i = (fits ? total : 0) + me; i < a.to.n_pool; i += kClCtas * kClThreads) a.to_refs[i] = 0;
  if (me == 0) {
    *a.count = fits ? total : -1;
    if (!fits) flag_error(a.to.status, DEV_POOL_FULL);
  }
}

__global__ void __launch_bounds__(kPgThreads)
k_compact_move(const __grid_constant__ CompactArgs a) {
  tc::grid_dep_wait();
  // (n = -1 where the new pool has too few blocks: all of these are compared as signed numbers)
  const int n = *a.count, first = blockIdx.x, ctas = gridDim.x;
  // (the next block's id is on its way while one is copied)
  int id = first < n ? a.list[first] : 0;
  for (int i = first; i < n; i += ctas) {
    const int next = i + ctas < n ? a.list[i + ctas] : 0;
    copy_codes(a.c, id, a.to, i, a.d, threadIdx.x, kPgThreads);
    id = next;
  }
  const size_t entries = static_cast<size_t>(a.c.pairs) * a.c.max_blocks, step = static_cast<size_t>(gridDim.x) * kPgThreads;
  for (size_t e = static_cast<size_t>(blockIdx.x) * kPgThreads + threadIdx.x; e < entries; e += step) {
    const int id = a.c.table[e];
    const int to = in_pool(a.c, id) ? a.number[id] : -1;
    if (n >= 0 && to < 0 && id != -1) flag_error(a.to.status, DEV_BAD_SLOT);
    a.to.table[e] = to;
    if (a.to.weight) a.to.weight[e] = n >= 0 && a.c.weight ? a.c.weight[e] : 0.f;
    if (e < static_cast<size_t>(a.c.pairs)) a.to.n_tok[e] = n >= 0 ? a.c.n_tok[e] : 0;
  }
}

static int reserve_slots(const shadowkv_cache& c, int s) {
  const long long n = (static_cast<long long>(s) + c.block - 2) / c.block + 1;   // s >= 1
  return static_cast<int>(n < c.max_blocks ? n : c.max_blocks);
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

static size_t reserve_layout(const shadowkv_cache& c, int s, char* base, ReserveArgs* a) {
  const size_t pairs = static_cast<size_t>(c.b) * c.h_kv, items = pairs * reserve_slots(c, s);
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base + off;
    off += up256(bytes);
    return p;
  };
  char* rank = take(items * 4);
  char* start = take((static_cast<size_t>(c.b) + 1) * 4);
  char* list = take((items < static_cast<size_t>(c.n_pool) ? items : c.n_pool) * 4);
  char* copy = take(pairs * 8);
  if (a) {
    a->rank = reinterpret_cast<int32_t*>(rank);
    a->start = reinterpret_cast<int32_t*>(start);
    a->list = reinterpret_cast<int32_t*>(list);
    a->copy = reinterpret_cast<int2*>(copy);
  }
  return off;
}

static size_t compact_bytes(const shadowkv_cache& c) { return 256 + 2 * up256(static_cast<size_t>(c.n_pool) * 4); }

}  // namespace skv

// ------------------------------------------------------------------ C ABI
namespace {
// What the walks count in 32 bits.
const char* large_fault(const shadowkv_cache* c, int s) {
  if (c->n_pool > 1 << 30) return "the pool must have at most 2^30 blocks";
  if (static_cast<long long>(c->b) * c->h_kv * skv::reserve_slots(*c, s > 0 ? s : 1) > 1 << 30)
    return "too many blocks for one call";
  return nullptr;
}
bool odd4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 != 0; }
const char* work_fault(const void* work, size_t have, size_t need) {
  if (!work || reinterpret_cast<uintptr_t>(work) % 256) return "the workspace must be non-NULL and 256-byte aligned";
  return have < need ? "the workspace is too small" : nullptr;
}
}  // namespace

extern "C" {

skv_status shadowkv_cache_share(const shadowkv_cache* c, int32_t* refs, int n, const int32_t* src, const int32_t* dst,
                                void* stream) try {
  using skv::set_error;
  const skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (n < 0 || n > c->b) return set_error(SKV_ERR_INVALID_ARG, "need 0 <= n <= b");
  if (n == 0) return SKV_OK;
  if (!refs || !src || !dst || odd4(refs) || odd4(src) || odd4(dst))
    return set_error(SKV_ERR_INVALID_ARG, "refs, src and dst must be non-NULL and 4-byte aligned");
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  const cudaError_t e = skv::launch_pdl(
      skv::k_share, dim3(n * c->h_kv, (c->max_blocks + skv::kPgThreads - 1) / skv::kPgThreads), dim3(skv::kPgThreads), 0,
      static_cast<cudaStream_t>(stream), skv::cache_dev(*c), refs, c->b, n, src, dst);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

skv_status shadowkv_cache_truncate(const shadowkv_cache* c, int32_t* refs, const int32_t* drop, void* stream) try {
  using skv::set_error;
  const skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (odd4(refs) || odd4(drop)) return set_error(SKV_ERR_INVALID_ARG, "refs and drop must be 4-byte aligned");
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  const cudaError_t e = skv::launch_pdl(skv::k_truncate, dim3(c->b * c->h_kv), dim3(skv::kPgThreads), 0,
                                        static_cast<cudaStream_t>(stream), skv::cache_dev(*c), refs, drop);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

size_t shadowkv_cache_reserve_workspace(const shadowkv_cache* c, int s) try {
  if (skv::cache_checked(c) != SKV_OK) return 0;
  if (s < 0) {
    skv::set_error(SKV_ERR_INVALID_ARG, "s must be >= 0");
    return 0;
  }
  return skv::reserve_layout(*c, s > 0 ? s : 1, nullptr, nullptr);
} catch (...) {   // host memory for an error text or a table ran out
  return 0;
}

skv_status shadowkv_cache_reserve(const shadowkv_cache* c, int32_t* refs, int s, const int32_t* lens, int32_t* granted,
                                  void* work, size_t work_bytes, void* stream) try {
  using skv::set_error;
  const skv_status st = skv::cache_checked(c);
  if (st != SKV_OK) return st;
  if (s < 0) return set_error(SKV_ERR_INVALID_ARG, "s must be >= 0");
  if (const char* f = large_fault(c, s)) return set_error(SKV_ERR_UNSUPPORTED, f);
  if (!refs || !granted || odd4(refs) || odd4(granted) || odd4(lens))
    return set_error(SKV_ERR_INVALID_ARG, "refs and granted must be non-NULL, and 4-byte aligned as lens");
  skv::ReserveArgs a;
  const char* f = work_fault(work, work_bytes, skv::reserve_layout(*c, s > 0 ? s : 1, static_cast<char*>(work), &a));
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  a.c = skv::cache_dev(*c);
  a.refs = refs;
  a.lens = lens;
  a.granted = granted;
  a.b = c->b;
  a.s = s;
  a.slots = skv::reserve_slots(*c, s > 0 ? s : 1);
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  cudaError_t e = skv::launch_pdl(skv::k_reserve, dim3(skv::kClCtas), dim3(skv::kClThreads), 0, q, a);
  if (e == cudaSuccess)
    e = skv::launch_pdl(skv::k_reserve_copy, dim3(c->b * c->h_kv), dim3(skv::kPgThreads), 0, q, a.c, c->d,
                        static_cast<const int2*>(a.copy));
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

size_t shadowkv_cache_compact_workspace(const shadowkv_cache* src) try {
  return skv::cache_checked(src) == SKV_OK ? skv::compact_bytes(*src) : 0;
} catch (...) {   // host memory for an error text or a table ran out
  return 0;
}

skv_status shadowkv_cache_compact(const shadowkv_cache* src, const int32_t* refs, const shadowkv_cache* dst,
                                  int32_t* dst_refs, void* work, size_t work_bytes, void* stream) try {
  using skv::set_error;
  skv_status st = skv::cache_checked(src);
  if (st != SKV_OK) return st;
  st = skv::cache_checked(dst);
  if (st != SKV_OK) return st;
  if (src->n_pool > 1 << 30 || dst->n_pool > 1 << 30)
    return set_error(SKV_ERR_UNSUPPORTED, "the pool must have at most 2^30 blocks");
  if (dst->b != src->b || dst->h_kv != src->h_kv || dst->d != src->d || dst->max_blocks != src->max_blocks ||
      dst->block != src->block)
    return set_error(SKV_ERR_INVALID_ARG, "dst and src differ in b, h_kv, d, max_blocks or block");
  if (dst->k_codes == src->k_codes || dst->v_codes == src->v_codes || dst->k_scale == src->k_scale ||
      dst->v_scale == src->v_scale || dst->table == src->table || dst->n_tok == src->n_tok || dst_refs == refs ||
      (dst->weight && dst->weight == src->weight))
    return set_error(SKV_ERR_INVALID_ARG, "dst shares memory with src");
  if (!refs || !dst_refs || odd4(refs) || odd4(dst_refs))
    return set_error(SKV_ERR_INVALID_ARG, "refs must be non-NULL and 4-byte aligned");
  const char* f = work_fault(work, work_bytes, skv::compact_bytes(*src));
  if (f) return set_error(SKV_ERR_INVALID_ARG, f);
  skv::CompactArgs a;
  a.c = skv::cache_dev(*src);
  a.to = skv::cache_dev(*dst);
  a.refs = refs;
  a.to_refs = dst_refs;
  a.count = static_cast<int32_t*>(work);
  a.number = a.count + 64;
  a.list = a.number + skv::up256(static_cast<size_t>(src->n_pool) * 4) / 4;
  a.d = src->d;
  int nsm = 0;
  cudaError_t e = skv::device_sms(&nsm);
  if (e != cudaSuccess) return set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
  cudaStream_t q = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> together(skv::cache_enqueue());
  e = skv::launch_pdl(skv::k_compact_number, dim3(skv::kClCtas), dim3(skv::kClThreads), 0, q, a);
  if (e == cudaSuccess) e = skv::launch_pdl(skv::k_compact_move, dim3(8 * nsm), dim3(skv::kPgThreads), 0, q, a);
  return e == cudaSuccess ? SKV_OK : set_error(SKV_ERR_CUDA, cudaGetErrorString(e));
} catch (...) {   // host memory for an error text or a table ran out
  return SKV_ERR_OOM;
}

}  // extern "C"
