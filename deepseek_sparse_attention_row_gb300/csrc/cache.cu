// cache.cu -- forking, freeing and compacting the pages of a cache: the C ABI
// of include/dsa_cache.h.
//
// A fork and a compaction are two launches: one CTA plans (which page goes
// where: ranks by block-wide prefix sums over the pairs and over refs), then
// many CTAs copy the page contents and write the tables. All decisions are
// ranks in index order, and refs change by integer atomics only, so results
// do not depend on the order of the work. The copies are bound by HBM: a
// thread has four 16-byte loads under way before it stores (128 pages of 128
// KiB in 16 planes move in 75.6 us, 1.04 of a plain copy's rate; with one load
// under way 100 us).
#include "../../include/dsa_cache.h"

#include <cuda_runtime.h>

#include <cstdint>

#include "follow.cuh"

namespace dsa {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr unsigned kMoveCtas = 152 * 8;  // a full SM's worth each
constexpr int64_t kMaxPairs = 65535;

// The plan of one pair of a fork: tokens of the parent (-1: nothing to do),
// and the copy of its partial page (from, to; -1 without one).
struct ForkPair {
  int32_t tokens, from, to;
};

struct CacheArgs {
  char* cache;
  int64_t planes, plane_stride, num_pages, page_stride;
  int32_t page_size;
  int64_t token_bytes;
  int32_t* refs;
  int32_t* tables;
  int64_t seqs, max_pages, ld_tables;
  int32_t* lens;
  // scales that go with the pages, whole pages of words; 0 words for none
  char* scales;
  int64_t scale_plane, scale_page;  // strides in bytes
  int32_t scale_words;
};

constexpr int kPlanPages = 4;  // pages of a thread in one round

// Sum of x over the lanes up to this one.
__device__ __forceinline__ uint32_t warp_sum_upto(uint32_t x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}

// Exclusive prefix sum of x over the CTA in thread order; `total` is the sum.
// `part` holds one word per warp; begins with a barrier behind its last use.
__device__ __forceinline__ uint32_t cta_scan(uint32_t x, uint32_t* part, uint32_t& total) {
  static_assert(kPlanThreads == 32 * 32, "one lane per warp below");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t upto = warp_sum_upto(x);
  __syncthreads();
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  const uint32_t sums = warp_sum_upto(part[lane]);
  total = __shfl_sync(~0u, sums, 31);
  const uint32_t before = __shfl_sync(~0u, sums, (warp - 1) & 31);
  return (warp > 0 ? before : 0) + upto - x;
}

// Bit i: whether page n0 + i is in use; the pages past the last one count as
// used too if `past`.
__device__ __forceinline__ uint32_t used_pages(const CacheArgs& a, int64_t n0, bool past) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < kPlanPages; ++i) {
    const int64_t n = n0 + i;
    if (n < a.num_pages ? a.refs[n] > 0 : past) bits |= 1u << i;
  }
  return bits;
}

// Which pairs are forked, and onto which pages: the r-th pair that needs a
// page gets the r-th free page.
__global__ void __launch_bounds__(kPlanThreads)
    fork_plan_kernel(const CacheArgs a, const int32_t* parents, const int32_t* children,
                     int32_t pairs, int32_t* status, ForkPair* plan, int32_t* want) {
  __shared__ uint32_t part[kPlanThreads / 32];
  __shared__ uint32_t again[(kMaxPairs + 31) / 32];  // children that were named before
  // Pass 0: a warp per pair looks through the pairs before it.
  for (int32_t w = threadIdx.x; w < (pairs + 31) / 32; w += kPlanThreads) again[w] = 0;
  __syncthreads();
  for (int32_t i = threadIdx.x >> 5; i < pairs; i += kPlanThreads / 32) {
    const int32_t c = children[i];
    bool named = false;
#pragma unroll 4
    for (int32_t k = threadIdx.x & 31; k < i; k += 32) named |= children[k] == c;
    if (__any_sync(~0u, named) && (threadIdx.x & 31) == 0) atomicOr(&again[i >> 5], 1u << (i & 31));
  }
  __syncthreads();
  // Pass 1: what each pair needs; want[r] = the pair of rank r.
  uint32_t needed = 0;
  for (int32_t i0 = 0; i0 < pairs; i0 += kPlanThreads) {
    const int32_t i = i0 + threadIdx.x;
    int32_t need = 0;
    if (i < pairs) {
      const int32_t p = parents[i], c = children[i];
      bool ok = p >= 0 && p < a.seqs && c >= 0 && c < a.seqs;
      int32_t tokens = 0, from = -1;
      if (ok) {
        const int32_t* crow = a.tables + c * a.ld_tables;
        ok = a.lens[c] == 0 && crow[0] < 0 && !((again[i >> 5] >> (i & 31)) & 1);
      }
      if (ok) {
        const int64_t most = a.max_pages * a.page_size;
        const int32_t len = a.lens[p];
        tokens = len < 0 ? 0 : (len > most ? static_cast<int32_t>(most) : len);
        if (tokens % a.page_size != 0) {
          from = a.tables[p * a.ld_tables + tokens / a.page_size];
          ok = from >= 0 && from < a.num_pages;
          need = ok;
        }
      }
      status[i] = ok ? DSA_FORK_OK : DSA_FORK_REFUSED;
      plan[i] = ForkPair{ok ? tokens : -1, from, -1};
    }
    uint32_t total;
    const uint32_t rank = needed + cta_scan(need, part, total);
    if (need) want[rank] = i;
    needed += total;
  }
  __syncthreads();  // want is read by other threads below
  // Pass 2: the free pages in order, until every need is met.
  uint32_t found = 0;
  for (int64_t n0 = 0; n0 < a.num_pages && found < needed; n0 += kPlanThreads * kPlanPages) {
    const int64_t n = n0 + threadIdx.x * kPlanPages;
    const uint32_t used = used_pages(a, n, true);
    uint32_t total;
    uint32_t rank = found + cta_scan(kPlanPages - __popc(used), part, total);
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) {
      if ((used >> i) & 1) continue;
      if (rank < needed) plan[want[rank]].to = static_cast<int32_t>(n + i);
      ++rank;
    }
    found += total;
  }
  for (uint32_t r = found + threadIdx.x; r < needed; r += kPlanThreads) {
    const int32_t i = want[r];
    status[i] = DSA_FORK_NO_PAGE;
    plan[i].tokens = -1;
  }
}

constexpr int kInFlight = 4;  // 16-byte loads of a thread
constexpr int64_t kPiece = 16ll * kInFlight * kCopyThreads;

// Bytes [at, at + kPiece) of a copy of `bytes`, by the whole CTA.
__device__ __forceinline__ void copy_piece(char* to, const char* from, int64_t bytes, int64_t at) {
  uint4 x[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int64_t o = at + 16ll * (i * kCopyThreads + threadIdx.x);
    if (o < bytes) x[i] = __ldcs(reinterpret_cast<const uint4*>(from + o));
  }
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    const int64_t o = at + 16ll * (i * kCopyThreads + threadIdx.x);
    if (o < bytes) __stcs(reinterpret_cast<uint4*>(to + o), x[i]);
  }
}

// The scales of a page in one plane, by the whole CTA.
__device__ __forceinline__ void copy_scales(const CacheArgs& a, int64_t plane, int32_t to,
                                            int32_t from) {
  char* base = a.scales + plane * a.scale_plane;
  uint32_t* x = reinterpret_cast<uint32_t*>(base + to * a.scale_page);
  const uint32_t* y = reinterpret_cast<const uint32_t*>(base + from * a.scale_page);
  for (int32_t i = threadIdx.x; i < a.scale_words; i += kCopyThreads) x[i] = y[i];
}

// CTA (x, y): pair x, planes y, y + gridDim.y, ...; the CTAs of y = 0 also
// write the child's row.
__global__ void __launch_bounds__(kCopyThreads)
    fork_copy_kernel(const CacheArgs a, const int32_t* parents, const int32_t* children,
                     const ForkPair* plan) {
  follow();
  const ForkPair f = plan[blockIdx.x];
  if (f.tokens < 0) return;
  const int32_t whole = f.tokens / a.page_size;
  if (blockIdx.y == 0) {
    const int32_t p = parents[blockIdx.x], c = children[blockIdx.x];
    const int32_t* prow = a.tables + p * a.ld_tables;
    int32_t* crow = a.tables + c * a.ld_tables;
    for (int64_t j = threadIdx.x; j < a.max_pages; j += kCopyThreads) {
      // an empty parent may be another pair's child: its row is not read
      const int32_t id = j < whole ? prow[j] : (j == whole ? f.to : -1);
      crow[j] = id;
      if (id >= 0 && id < a.num_pages) atomicAdd(a.refs + id, 1);
    }
    if (threadIdx.x == 0) a.lens[c] = f.tokens;
  }
  if (f.to < 0) return;
  const int64_t bytes = (f.tokens % a.page_size) * a.token_bytes;
  for (int64_t pl = blockIdx.y; pl < a.planes; pl += gridDim.y) {
    char* plane = a.cache + pl * a.plane_stride;
    for (int64_t at = 0; at < bytes; at += kPiece)
      copy_piece(plane + f.to * a.page_stride, plane + f.from * a.page_stride, bytes, at);
    if (a.scale_words > 0) copy_scales(a, pl, f.to, f.from);
  }
}

__global__ void __launch_bounds__(kCopyThreads)
    free_kernel(const CacheArgs a, const int32_t* list) {
  const int32_t s = list[blockIdx.x];
  if (s < 0 || s >= a.seqs) return;
  int32_t* row = a.tables + s * a.ld_tables;
  for (int64_t j = threadIdx.x; j < a.max_pages; j += kCopyThreads) {
    // exchanged, so that a slot named twice gives each page back once
    const int32_t id = atomicExch(row + j, -1);
    if (id >= 0 && id < a.num_pages) {
      // what goes below 0 is given back: whatever the order, refs end at
      // max(0, refs - frees)
      if (atomicSub(a.refs + id, 1) <= 0) atomicAdd(a.refs + id, 1);
    }
  }
  if (threadIdx.x == 0) a.lens[s] = 0;
}

// moves: [0] how many, then from[k], to[k] pairs.
__global__ void __launch_bounds__(kPlanThreads)
    compact_plan_kernel(const CacheArgs a, int32_t* remap, int32_t* live, int32_t* count,
                        int2* moves) {
  __shared__ uint32_t part[kPlanThreads / 32];
  constexpr int kRound = kPlanThreads * kPlanPages;
  uint32_t mine = 0, used;
#pragma unroll 4
  for (int64_t n = threadIdx.x; n < a.num_pages; n += kPlanThreads) mine += a.refs[n] > 0;
  cta_scan(mine, part, used);
  uint32_t holes = 0, movers = 0;
  for (int64_t n0 = 0; n0 < a.num_pages; n0 += kRound) {
    const int64_t n = n0 + threadIdx.x * kPlanPages;
    const uint32_t bits = used_pages(a, n, false);
    // bits of the pages below the number of used ones, and of real pages
    const uint32_t low = n >= used ? 0 : used - n >= kPlanPages ? ~0u : (1u << (used - n)) - 1;
    const uint32_t real =
        n >= a.num_pages ? 0
                         : (1u << min(a.num_pages - n, static_cast<int64_t>(kPlanPages))) - 1;
    const uint32_t hole = ~bits & low & real, mover = bits & ~low;
    // both counts in one sum: a round has fewer than 2^16 pages
    static_assert(kRound < 65536, "counts of 16 bits");
    uint32_t total;
    const uint32_t rank = cta_scan(__popc(hole) | (__popc(mover) << 16), part, total);
    uint32_t h = holes + (rank & 0xffff), m = movers + (rank >> 16);
#pragma unroll
    for (int i = 0; i < kPlanPages; ++i) {
      const int32_t page = static_cast<int32_t>(n + i);
      if ((hole >> i) & 1) moves[h++].y = page;
      if ((mover >> i) & 1) moves[m++].x = page;
      if ((real >> i) & 1) remap[page] = (bits >> i) & 1 ? page : -1;
    }
    holes += total & 0xffff;
    movers += total >> 16;
  }
  __syncthreads();  // moves and remap are read and rewritten by other threads
  for (uint32_t k = threadIdx.x; k < movers; k += kPlanThreads) {
    const int2 m = moves[k];
    remap[m.x] = m.y;
    a.refs[m.y] = a.refs[m.x];
    a.refs[m.x] = 0;
  }
  if (threadIdx.x == 0) {
    *live = used;
    *count = movers;
  }
}

// The moves of all planes, dealt to the CTAs in turn, then the tables.
__global__ void __launch_bounds__(kCopyThreads)
    compact_move_kernel(const CacheArgs a, const int32_t* remap, const int32_t* count,
                        const int2* moves) {
  follow();
  const int64_t bytes = a.page_size * a.token_bytes;
  const int64_t pieces = (bytes + kPiece - 1) / kPiece, units = *count * a.planes * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t page = u / pieces;
    const int2 m = moves[page / a.planes];
    char* plane = a.cache + (page % a.planes) * a.plane_stride;
    copy_piece(plane + m.y * a.page_stride, plane + m.x * a.page_stride, bytes,
               (u - page * pieces) * kPiece);
  }
  if (a.scale_words > 0)
    for (int64_t u = blockIdx.x; u < *count * a.planes; u += gridDim.x) {
      const int2 m = moves[u / a.planes];
      copy_scales(a, u % a.planes, m.y, m.x);
    }
  const int64_t entries = a.seqs * a.max_pages;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kCopyThreads + threadIdx.x; e < entries;
       e += static_cast<int64_t>(gridDim.x) * kCopyThreads) {
    int32_t* at = a.tables + (e / a.max_pages) * a.ld_tables + e % a.max_pages;
    const int32_t id = *at;
    if (id >= 0 && id < a.num_pages) {
      const int32_t to = remap[id];
      if (to != id) *at = to;
    }
  }
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dsa_status check_tables(int64_t num_pages, const int32_t* refs, const int32_t* tables,
                        int64_t seqs, int64_t max_pages, int64_t ld_tables) {
  if (num_pages < 0 || seqs < 0 || max_pages < 0 || ld_tables < max_pages) return DSA_EINVAL;
  if (num_pages > INT32_MAX || seqs > INT32_MAX || max_pages > INT32_MAX) return DSA_EUNSUPPORTED;
  if ((num_pages > 0 && !refs) || (seqs > 0 && max_pages > 0 && !tables)) return DSA_EINVAL;
  return DSA_OK;
}

dsa_status check_cache(const CacheArgs& a) {
  if (a.planes < 0 || a.page_size < 1 || a.token_bytes < 0) return DSA_EINVAL;
  if (a.max_pages * a.page_size > INT32_MAX || a.token_bytes > INT32_MAX || a.planes > INT32_MAX)
    return DSA_EUNSUPPORTED;
  if (a.planes > 0 && a.num_pages > 0 && a.token_bytes > 0 && !a.cache) return DSA_EINVAL;
  if (!aligned16(a.cache) || a.plane_stride % 16 != 0 || a.page_stride % 16 != 0 ||
      a.token_bytes % 16 != 0)
    return DSA_EUNSUPPORTED;
  return DSA_OK;
}

// Scales of `bytes` a page beside the pages of `a`; none for 0.
dsa_status add_scales(CacheArgs& a, void* scales, int64_t plane_stride, int64_t page_stride,
                      int64_t bytes) {
  if (bytes < 0 || plane_stride < 0 || page_stride < 0) return DSA_EINVAL;
  if (bytes > INT32_MAX) return DSA_EUNSUPPORTED;
  if (bytes == 0) return DSA_OK;
  if (!scales && a.planes > 0 && a.num_pages > 0) return DSA_EINVAL;
  if ((reinterpret_cast<uintptr_t>(scales) & 3u) != 0 ||
      (plane_stride | page_stride | bytes) % 4 != 0)
    return DSA_EUNSUPPORTED;
  a.scales = static_cast<char*>(scales);
  a.scale_plane = plane_stride;
  a.scale_page = page_stride;
  a.scale_words = static_cast<int32_t>(bytes / 4);
  return DSA_OK;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Fork: want [pairs], plan [pairs]. Compaction: count (256 bytes), moves.
size_t fork_bytes(int64_t pairs) { return up256(pairs * 4) + up256(pairs * sizeof(ForkPair)); }
size_t compact_bytes(int64_t pages) { return 256 + up256(pages * sizeof(int2)); }

}  // namespace
}  // namespace dsa

extern "C" size_t dsa_cache_workspace_bytes(int64_t pairs, int64_t num_pages) {
  if (pairs < 0 || num_pages < 0) return 0;
  const size_t f = dsa::fork_bytes(pairs), c = pairs ? 0 : dsa::compact_bytes(num_pages);
  return f > c ? f : c;
}

namespace {

dsa_status fork(const dsa::CacheArgs& a, const int32_t* parents, const int32_t* children,
                int64_t pairs, int32_t* status, void* workspace, size_t workspace_bytes,
                void* stream) {
  dsa_status st = dsa::check_tables(a.num_pages, a.refs, a.tables, a.seqs, a.max_pages,
                                    a.ld_tables);
  if (st != DSA_OK) return st;
  st = dsa::check_cache(a);
  if (st != DSA_OK) return st;
  if (pairs < 0) return DSA_EINVAL;
  if (pairs > dsa::kMaxPairs) return DSA_EUNSUPPORTED;
  if (pairs == 0) return DSA_OK;
  if (a.max_pages < 1 || !parents || !children || !status || (a.seqs > 0 && !a.lens))
    return DSA_EINVAL;
  if (!workspace || workspace_bytes < dsa::fork_bytes(pairs) || !dsa::aligned16(workspace))
    return DSA_EINVAL;
  int32_t* want = static_cast<int32_t*>(workspace);
  auto* plan = reinterpret_cast<dsa::ForkPair*>(static_cast<char*>(workspace) +
                                                dsa::up256(pairs * 4));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int32_t n = static_cast<int32_t>(pairs);
  dsa::fork_plan_kernel<<<1, dsa::kPlanThreads, 0, s>>>(a, parents, children, n, status, plan,
                                                        want);
  if (cudaGetLastError() != cudaSuccess) return DSA_ECUDA;
  const unsigned ys =
      static_cast<unsigned>(a.planes < 1 ? 1 : (a.planes < 65535 ? a.planes : 65535));
  return dsa::launch_after(dsa::fork_copy_kernel, dim3(n, ys), dsa::kCopyThreads, s, a, parents,
                           children, static_cast<const dsa::ForkPair*>(plan))
             ? DSA_OK
             : DSA_ECUDA;
}

}  // namespace

extern "C" dsa_status dsa_cache_fork(void* cache, int64_t planes, int64_t plane_stride,
                                     int64_t num_pages, int64_t page_stride, int32_t page_size,
                                     int64_t token_bytes, int32_t* refs, int32_t* tables,
                                     int64_t seqs, int64_t max_pages, int64_t ld_tables,
                                     int32_t* lens, const int32_t* parents,
                                     const int32_t* children, int64_t pairs, int32_t* status,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  const dsa::CacheArgs a{static_cast<char*>(cache), planes, plane_stride, num_pages, page_stride,
                         page_size, token_bytes, refs, tables, seqs, max_pages, ld_tables, lens,
                         nullptr, 0, 0, 0};
  return fork(a, parents, children, pairs, status, workspace, workspace_bytes, stream);
}

extern "C" dsa_status dsa_cache_fork_scaled(
    void* cache, int64_t planes, int64_t plane_stride, int64_t num_pages, int64_t page_stride,
    int32_t page_size, int64_t token_bytes, void* scales, int64_t scale_plane_stride,
    int64_t scale_page_stride, int64_t scale_bytes, int32_t* refs, int32_t* tables, int64_t seqs,
    int64_t max_pages, int64_t ld_tables, int32_t* lens, const int32_t* parents,
    const int32_t* children, int64_t pairs, int32_t* status, void* workspace,
    size_t workspace_bytes, void* stream) {
  dsa::CacheArgs a{static_cast<char*>(cache), planes, plane_stride, num_pages, page_stride,
                   page_size, token_bytes, refs, tables, seqs, max_pages, ld_tables, lens,
                   nullptr, 0, 0, 0};
  const dsa_status st =
      dsa::add_scales(a, scales, scale_plane_stride, scale_page_stride, scale_bytes);
  if (st != DSA_OK) return st;
  return fork(a, parents, children, pairs, status, workspace, workspace_bytes, stream);
}

extern "C" dsa_status dsa_cache_free(int32_t* refs, int64_t num_pages, int32_t* tables,
                                     int64_t seqs, int64_t max_pages, int64_t ld_tables,
                                     int32_t* lens, const int32_t* seqs_list, int64_t count,
                                     void* stream) {
  const dsa_status st = dsa::check_tables(num_pages, refs, tables, seqs, max_pages, ld_tables);
  if (st != DSA_OK) return st;
  if (count < 0) return DSA_EINVAL;
  if (count > INT32_MAX) return DSA_EUNSUPPORTED;
  if (count == 0) return DSA_OK;
  if (!seqs_list || (seqs > 0 && !lens)) return DSA_EINVAL;
  dsa::CacheArgs a{};
  a.num_pages = num_pages;
  a.refs = refs;
  a.tables = tables;
  a.seqs = seqs;
  a.max_pages = max_pages;
  a.ld_tables = ld_tables;
  a.lens = lens;
  dsa::free_kernel<<<static_cast<unsigned>(count), dsa::kCopyThreads, 0,
                     static_cast<cudaStream_t>(stream)>>>(a, seqs_list);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

namespace {

dsa_status compact(const dsa::CacheArgs& a, int32_t* remap, int32_t* live, void* workspace,
                   size_t workspace_bytes, void* stream) {
  dsa_status st = dsa::check_tables(a.num_pages, a.refs, a.tables, a.seqs, a.max_pages,
                                    a.ld_tables);
  if (st != DSA_OK) return st;
  st = dsa::check_cache(a);
  if (st != DSA_OK) return st;
  if (!live || (a.num_pages > 0 && !remap)) return DSA_EINVAL;
  if (!workspace || workspace_bytes < dsa::compact_bytes(a.num_pages) ||
      !dsa::aligned16(workspace))
    return DSA_EINVAL;
  int32_t* count = static_cast<int32_t*>(workspace);
  int2* moves = reinterpret_cast<int2*>(static_cast<char*>(workspace) + 256);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  dsa::compact_plan_kernel<<<1, dsa::kPlanThreads, 0, s>>>(a, remap, live, count, moves);
  if (cudaGetLastError() != cudaSuccess) return DSA_ECUDA;
  return dsa::launch_after(dsa::compact_move_kernel, dim3(dsa::kMoveCtas), dsa::kCopyThreads, s, a,
                           static_cast<const int32_t*>(remap), static_cast<const int32_t*>(count),
                           static_cast<const int2*>(moves))
             ? DSA_OK
             : DSA_ECUDA;
}

}  // namespace

extern "C" dsa_status dsa_cache_compact(void* cache, int64_t planes, int64_t plane_stride,
                                        int64_t num_pages, int64_t page_stride, int32_t page_size,
                                        int64_t token_bytes, int32_t* refs, int32_t* tables,
                                        int64_t seqs, int64_t max_pages, int64_t ld_tables,
                                        int32_t* remap, int32_t* live, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  const dsa::CacheArgs a{static_cast<char*>(cache), planes, plane_stride, num_pages, page_stride,
                         page_size, token_bytes, refs, tables, seqs, max_pages, ld_tables,
                         nullptr, nullptr, 0, 0, 0};
  return compact(a, remap, live, workspace, workspace_bytes, stream);
}

extern "C" dsa_status dsa_cache_compact_scaled(
    void* cache, int64_t planes, int64_t plane_stride, int64_t num_pages, int64_t page_stride,
    int32_t page_size, int64_t token_bytes, void* scales, int64_t scale_plane_stride,
    int64_t scale_page_stride, int64_t scale_bytes, int32_t* refs, int32_t* tables, int64_t seqs,
    int64_t max_pages, int64_t ld_tables, int32_t* remap, int32_t* live, void* workspace,
    size_t workspace_bytes, void* stream) {
  dsa::CacheArgs a{static_cast<char*>(cache), planes, plane_stride, num_pages, page_stride,
                   page_size, token_bytes, refs, tables, seqs, max_pages, ld_tables, nullptr,
                   nullptr, 0, 0, 0};
  const dsa_status st =
      dsa::add_scales(a, scales, scale_plane_stride, scale_page_stride, scale_bytes);
  if (st != DSA_OK) return st;
  return compact(a, remap, live, workspace, workspace_bytes, stream);
}
