// attend.cuh -- the attention kernel on the tensor cores, shared by prompt
// attention and by decode attention on pages.
//
// Mathematics. For a row q over the keys that it sees (c = scale * log2 e):
// x_j = c <q, k_j>, m = max x_j, l = sum 2^(x_j - m), O = sum 2^(x_j - m) v_j.
// Keys go by in tiles of 128. The row keeps a base b, m - 8 / c <= b <= m (in
// units of <q, k>), and adds 2^(c (s_j - b)) to l and to O; only when a new
// maximum passes the base by more than 2^8 in weight are l and O multiplied
// down and the base moved. Weights then stay below 2^8, and the largest is at
// least 1, so that neither fp32 sums nor 16-bit weights lose anything by it.
// Weights are rounded to the operands' type for the product with V: the tensor
// cores take one type for both operands. l sums them unrounded.
//
// Rows. The G query heads of one key/value head share every key, so a matrix
// tile of 128 rows holds 128 / G tokens of G heads each.
//
// One CTA per SM with 12 warps: four warps for each of two streams (one row
// per thread: maxima, exponentials, sums, and at the end the output), one
// warp that issues matrix products, one that loads, one that schedules. A
// stream has its own 128 columns of tensor memory for the scores S = Q K^T
// (the weights P overwrite them, as 16-bit pairs) and up to 128 for O += P V.
// While one stream's warps are busy with exponentials, the tensor cores run
// the other's products. The streams either take two row tiles over the same
// keys (shared: each K and V tile is loaded once for 256 rows) or one row
// tile over alternate key tiles (split: few rows, both streams busy; the
// results are two partial outputs).
//
// A persistent CTA walks a list of segments (row tiles x a range of key
// tiles) that the scheduling warp writes to a ring of eight, so that loads and
// products of the next segment run under the current one's end.
//
// What bounds it. Prompts: the tensor cores, active in 78% of the cycles (one
// full attention of 8192 tokens, 16 heads of 128: 316 us, 1740 TFLOP/s, 0.91
// of a plain product's burst rate; 16389 causal tokens: 645 us, 1705); the rest
// is the chain scores - softmax - weights of a stream, about 1100 cycles of
// softmax a tile, and the ends of segments. Decode on pages: HBM (64 sequences
// of up to 4096 tokens: 95 us for 527 MB with the join; the loads alone 93).
//
// Every wait is bounded (kWaitTurns); one that gives up records its site in
// g_pipe_error, and all roles leave.
//
// Values that a row does not see have weight 0, which an infinite or NaN value
// turns into NaN. What lies behind a sequence's end in its last tile (often
// memory never written) is cleared by a warp of its own before the products;
// what a row does not see of its own sequence (causal rows) or of the prefix
// (lengths that end in it) is finite in any sane call. Where an output is not
// finite and its row does not see all of its tiles, the CTA goes through its
// list again: the clearing warp makes the tiles finite that some row does not
// see whole, and at the end each row gets what it sees of the values that were
// not (add_seen). Such a CTA takes about twice as long (262144 tokens, one
// hidden infinity: 20 ms, 10 without; rows computed again one by one took 6.8
// s). A prefix that rows end in, with a NaN behind them, is read by four warps
// of each CTA: 128 sequences on 32768 tokens 4.8 ms, 0.15 without. In the
// softmax warps this costs one store: with more code there, 128 sequences
// behind a shared document took 122 us instead of 105.
//
// Code size matters: the roles of an SM run different code at the same time,
// and a call with short segments runs each piece only a few times. Loops that
// need no registers as arrays are therefore not unrolled, and each wait and
// product sequence stands in as few places as possible.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "follow.cuh"
#include "umma.cuh"

namespace dsa {
namespace {

constexpr int kTile = 128;           // rows of a row tile, keys of a key tile
constexpr int kAttendThreads = 384;  // no calls in the kernel: ptxas could not split registers
constexpr int kParts = 2;            // parts of a weight tile handed to the products one by one
constexpr float kGrow = 8.0f;        // log2 of the growth that moves a row's base
constexpr int kSegs = 8;             // segments that the scheduling warp may be ahead
// A wait gives up when its CTA has got on with nothing between the second and
// third turn of the global timer's high word, for 8.6 to 12.9 seconds. What
// counts are the loads (every 64 steps): a wait may be as long as the call, like
// that for the next value behind a sequence's end, of which a call may have
// none.
constexpr int32_t kWaitTurns = 3;

__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_f(float x) { return __float2half_rn(x); }
// {lo, hi} rounded to nearest even, lo in the low half
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __int_as_float(0x7f800000); }

// What a stream of segments is made of. Sizes are below 2^31.
struct Seg {
  int32_t n[2];     // key tiles of each stream; n[0] < 0: the list's end
  int32_t split;    // streams: 0 two row tiles, 1 alternate key tiles
  int32_t first;    // split: the stream of the first key tile
  int32_t t0;       // first key tile
  int32_t kh;       // key/value head
  int32_t tok[2];   // first token of each row tile
  int32_t ntok[2];  // its tokens
  // prompt: keys [k0, k0 + kv_len); the token before q_end sees all of them
  int32_t k0, kv_len, q_end;
  // pages: the sequence whose own tokens these are (kv_len of them), or ~r for
  // the prefix (kv_len 0), whose pages stand r rows of tables behind
  // prefix_pages; whether a page of the segment is missing
  int32_t seq, gaps;
  int32_t slot;     // of the partial outputs (-1: written out at once)
  // Pass 1: the key tile from which on some row does not see all, whose values
  // are made finite. kNone in pass 0.
  int32_t sane;
  // The key tile from which on values go through the clearing warp: sane, or
  // where values lie behind the sequence's last key (the next sequence's, or
  // what a page holds that is not full).
  int32_t tail;
};
constexpr int32_t kNone = 0x7fffffff;
// A V tile for the clearing warp.
struct Tail {
  int32_t stage, parity;
  int32_t sane;      // whether the rows below `from` are made finite
  int32_t from, to;  // the rows to clear
};

struct AttendArgs {
  const void *q, *k, *v;
  int64_t q_st, q_sh;
  int32_t heads, kv_heads, group, dim, tile_tokens;
  float c;  // scale * log2 e
  int64_t tokens;
  // prompt
  int64_t total_k, k_st, k_sh, v_st, v_sh;
  const int32_t *cu_q, *cu_k;
  int32_t seqs, causal;
  void* out;
  int64_t o_st, o_sh;
  float* lse;
  int64_t l_st, l_sh;
  int32_t cut;                     // whether blocks may be cut, with room for it:
  struct CutBlock* cuts;           // [CTAs], and the parts in prefix_o, prefix_lse
  // pages
  int64_t k_sn, v_sn;
  int64_t num_pages, max_pages, ld_tables;
  int32_t page_size, page_log2;
  const int32_t *prefix_pages, *tables, *lens;
  int64_t prefix_len;
  int32_t prefix_tiles, prefix_blocks, prefix_split;
  int32_t* starts;                 // [tokens + 1]: own units before each sequence
  // [slot][2][DP / 4][128][4] (neighbouring rows write neighbouring 16 bytes),
  // [slot][256]
  float *prefix_o, *prefix_lse;
  float *own_o, *own_lse;          // [slot][2 G][DP], [slot][2 G]
};

template <int DP>
struct Layout {
  static constexpr int kHalves = DP / 64;
  static constexpr uint32_t kHalf = kTile * 128;  // [128 rows][64 elements], swizzled
  static constexpr uint32_t kBytes = kHalf * kHalves;
  static constexpr int kStages = DP == 128 ? 5 : 10;
  static constexpr uint32_t kRing = 2 * kBytes;
  static constexpr uint32_t kCtrl = kRing + kStages * kBytes;
};

constexpr int kMaxStages = 10;
constexpr int kTails = 16;  // more than V tiles in the ring
struct Ctrl {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2][kParts], o_done[2], o_free[2];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t tail_full[kTails], tail_done[kTails];
  Seg seg[kSegs];
  Tail tail[kTails];
  uint32_t tmem;
  uint32_t beat;  // global_turns() when the CTA last got on
  int dead;
  int doubt;  // an output may hold what its row does not see
  int pass;   // 0; 1: once more, with finite values
};
constexpr size_t attend_smem(uint32_t ctrl) { return 1024 + ctrl + sizeof(Ctrl); }

__device__ __forceinline__ uint32_t global_turns() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_hi;" : "=r"(t));
  return t;
}
__device__ __forceinline__ void get_on(Ctrl* c) {
  *reinterpret_cast<volatile uint32_t*>(&c->beat) = global_turns();
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, Ctrl* c, unsigned site) {
  if (mbar_try_wait(bar, parity)) return true;
#pragma unroll 1
  for (;;) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&c->dead)) return false;
    const uint32_t beat = *reinterpret_cast<volatile uint32_t*>(&c->beat);
    if (static_cast<int32_t>(global_turns() - beat) >= kWaitTurns) {
      atomicCAS(&g_pipe_error, 0u, site);
      *reinterpret_cast<volatile int*>(&c->dead) = 1;
      return false;
    }
  }
}

// The same for a whole warp: all lanes go on, or none.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, Ctrl* c,
                                          unsigned site) {
  return __all_sync(~0u, wait(bar, parity, c, site));
}

__device__ __forceinline__ int32_t clamp_to(int32_t x, int64_t top) {
  return x < 0 ? 0 : (x > top ? static_cast<int32_t>(top) : x);
}
// Sum of x over the lanes up to this one.
__device__ __forceinline__ uint32_t warp_sum_upto(uint32_t x) {
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(~0u, x, o);
    if ((threadIdx.x & 31) >= o) x += y;
  }
  return x;
}
// Key tiles of n keys (in 32 bits without a sign: n may be 2^31 - 1).
__host__ __device__ inline int32_t tiles_of(int32_t n) {
  return n <= 0 ? 0 : static_cast<int32_t>((static_cast<uint32_t>(n) + kTile - 1) / kTile);
}

// ---- keys on pages ----------------------------------------------------------

// The page of the segment's token t (counted from the prefix's start, or from
// the sequence's first own token), or num_pages when there is none.
__device__ __forceinline__ int32_t page_of(const AttendArgs& a, int32_t seq, int64_t t) {
  int64_t p = t >> a.page_log2;
  const int32_t none = static_cast<int32_t>(a.num_pages);
  const int64_t pre = a.prefix_len >> a.page_log2;
  int32_t id;
  if (seq < 0) {
    if (p >= pre) return none;
    id = __ldg(a.prefix_pages + ~seq * a.ld_tables + p);
  } else {
    p += pre;
    if (p >= a.max_pages) return none;
    id = __ldg(a.tables + seq * a.ld_tables + p);
  }
  return id < 0 || id > none ? none : id;
}

// ---- schedules ------------------------------------------------------------

// Prompts: the work is a line of units, cut into equal shares, one per CTA:
// (sequence, key/value head, block of 2 * tile_tokens tokens). A block is as
// long as the keys that its last token sees, and kBlockCost for itself; a key
// tile falls to the share that holds its first unit, so that CTAs finish
// together whatever the lengths are. A share is a list of segments, a block's
// tiles each. Blocks that lie in one share are written out at once; of a block
// that is cut, each share holds a partial output, in slot 2 x of CTA x where
// the block begins in an earlier share, 2 x + 1 where it goes on in the next,
// and join_blocks_kernel joins them.
// Without cuts (a.cut = 0: few keys, where the join would cost more than it
// evens out) every block is one unit. kBlockCost = 2, 4, 6, 8 tiles: packed
// prefill chunk 351, 339, 349, 350 us, one long prompt 665, 645, 662, 664.
constexpr int32_t kBlockCost = 4 * kTile;
constexpr int32_t kMinShare = 4 * kTile;

// A cut block: what the joining kernel needs of it, with the CTA that begins it.
struct CutBlock {
  int32_t tok, ntok[2], kh;
  int32_t more;  // CTAs behind this one that hold parts; 0: no block is cut here
};
// Whether CTA x of `ctas` left a block to join, with all of its parts in the
// workspace and its rows in the output. Every share keeps to that while the
// offsets stay as they are; a caller who changes them under the call gets
// wrong rows, but no access out of range.
__host__ __device__ inline bool joinable(const CutBlock& b, const AttendArgs& a, int64_t x,
                                         int64_t ctas) {
  return b.more > 0 && b.more < ctas - x && b.tok >= 0 && b.ntok[0] >= 0 &&
         b.ntok[0] <= a.tile_tokens && b.ntok[1] >= 0 && b.ntok[1] <= a.tile_tokens &&
         static_cast<int64_t>(b.tok) + b.ntok[0] + b.ntok[1] <= a.tokens && b.kh >= 0 &&
         b.kh < a.kv_heads;
}

struct PromptSchedule {
  int64_t pos, end, share;
  int64_t start;         // unit at which the current block begins
  int32_t chunk = 0;     // first of the 32 sequences that the lanes hold
  int32_t l_q0, l_q1, l_k0, l_k1;
  int32_t lane_of = -1;  // lane of the current sequence
  int32_t q0, q1, k0, kv, blocks, kh, b;

  __device__ void hold(const AttendArgs& a) {
    const int32_t i = chunk + (threadIdx.x & 31);
    l_q0 = l_q1 = l_k0 = l_k1 = 0;
    if (i < a.seqs) {
      l_q0 = clamp_to(a.cu_q[i], a.tokens);
      l_q1 = max(l_q0, clamp_to(a.cu_q[i + 1], a.tokens));
      l_k0 = clamp_to(a.cu_k[i], a.total_k);
      l_k1 = max(l_k0, clamp_to(a.cu_k[i + 1], a.total_k));
    }
  }
  __device__ static int32_t blocks_of(const AttendArgs& a, int32_t tokens) {
    const uint32_t block = 2 * a.tile_tokens;
    return static_cast<int32_t>((static_cast<uint32_t>(tokens) + block - 1) / block);
  }
  // Keys that token e - 1 of n sees of kv, and units of the block that ends there.
  __device__ static int32_t keys_of(const AttendArgs& a, int32_t n, int32_t kv, int32_t e) {
    return a.causal ? max(kv - (n - e), 0) : kv;
  }
  __device__ static int32_t cost_of(const AttendArgs& a, int32_t keys) {
    return a.cut ? kBlockCost + keys : 1;
  }
  // Units of the first m blocks of n tokens on kv keys (m below the number of
  // blocks: all of them whole).
  __device__ static int64_t units_of(const AttendArgs& a, int32_t n, int32_t kv, int32_t m) {
    if (!a.cut) return m;
    const int64_t own = static_cast<int64_t>(m) * kBlockCost;
    if (!a.causal) return own + static_cast<int64_t>(m) * kv;
    // block i sees kv - n + (i + 1) * block keys, none below i = none
    const int32_t block = 2 * a.tile_tokens;
    const int32_t none = kv >= n ? 0 : min((n - kv) / block, m);
    const int64_t some = m - none;
    return own + some * (static_cast<int64_t>(kv) - n) + block * (some * (none + 1 + m) / 2);
  }
  __device__ static int64_t all_of(const AttendArgs& a, int32_t n, int32_t kv) {
    const int32_t m = blocks_of(a, n);
    return m == 0 ? 0 : units_of(a, n, kv, m - 1) + cost_of(a, kv);
  }
  // Makes lane `src`'s sequence the current one.
  __device__ void enter(const AttendArgs& a, int src) {
    lane_of = src;
    q0 = __shfl_sync(~0u, l_q0, src);
    q1 = __shfl_sync(~0u, l_q1, src);
    k0 = __shfl_sync(~0u, l_k0, src);
    kv = __shfl_sync(~0u, l_k1, src) - k0;
    blocks = blocks_of(a, q1 - q0);
    kh = b = 0;
  }

  __device__ explicit PromptSchedule(const AttendArgs& a) {
    // No block is cut here until next() says so: before any wait, so that the
    // join finds no stale entry where a wait gives up.
    if (a.cut && (threadIdx.x & 31) == 0) a.cuts[blockIdx.x].more = 0;
    int64_t all = 0;
#pragma unroll 1
    for (chunk = 0; chunk < a.seqs; chunk += 32) {
      hold(a);
      int64_t n = all_of(a, l_q1 - l_q0, l_k1 - l_k0);
#pragma unroll 1
      for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(~0u, n, o);
      all += n * a.kv_heads;
    }
    share = (all + gridDim.x - 1) / gridDim.x;
    if (a.cut) share = max(share, static_cast<int64_t>(kMinShare));
    pos = min(share * blockIdx.x, all);
    end = min(pos + share, all);
    start = 0;
    if (pos >= end) return;
    // the sequence, the head and the block that hold unit pos
#pragma unroll 1
    for (chunk = 0;; chunk += 32) {
      if (a.seqs > 32) hold(a);
      const int64_t n = all_of(a, l_q1 - l_q0, l_k1 - l_k0) * a.kv_heads;
      int64_t upto = n;
#pragma unroll 1
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(~0u, upto, o);
        if ((threadIdx.x & 31) >= o) upto += y;
      }
      const uint32_t found = __ballot_sync(~0u, upto > pos - start);
      if (found != 0) {
        const int src = __ffs(found) - 1;
        start += __shfl_sync(~0u, upto - n, src);
        enter(a, src);
        break;
      }
      start += __shfl_sync(~0u, upto, 31);
    }
    const int64_t per = all_of(a, q1 - q0, kv);
    kh = static_cast<int32_t>((pos - start) / per);
    start += kh * per;
    int32_t lo = 0, hi = blocks;  // units_of(lo) <= pos - start < those of hi blocks
#pragma unroll 1
    while (hi - lo > 1) {
      const int32_t mid = (lo + hi) >> 1;
      if (units_of(a, q1 - q0, kv, mid) <= pos - start) lo = mid; else hi = mid;
    }
    b = lo;
    start += units_of(a, q1 - q0, kv, b);
  }

  // The key tile from which on some row of the segment does not see all keys.
  __device__ static int32_t first_masked(const AttendArgs& a, const Seg& g) {
    return a.causal ? max(g.kv_len - (g.q_end - 1 - g.tok[0]), 0) / kTile : kNone;
  }

  __device__ bool next(const AttendArgs& a, Seg& g) {
    const int32_t block = 2 * a.tile_tokens;
#pragma unroll 1
    for (;;) {
      if (pos >= end) return false;
      const int32_t e = min((b + 1) * static_cast<int64_t>(block), static_cast<int64_t>(q1 - q0));
      const int32_t keys = keys_of(a, q1 - q0, kv, e), cost = cost_of(a, keys);
      const int32_t from = static_cast<int32_t>(pos - start);
      const int32_t to = static_cast<int32_t>(min(static_cast<int64_t>(cost), end - start));
      const int64_t at = start;
      const int32_t tiles = tiles_of(keys), my_kh = kh, my_k0 = k0, my_kv = kv, my_q1 = q1;
      const int32_t tok = q0 + b * block;
      const int32_t t0 = a.cut ? tiles_of(from - kBlockCost) : 0;
      const int32_t t1 = a.cut ? tiles_of(to - kBlockCost) : tiles;
      pos = start + to;
      if (to == cost) {
        start = pos;
        if (++b == blocks) {
          b = 0;
          if (++kh == a.kv_heads && pos < end) {
            // the next sequence that has any tokens
            uint32_t found =
                __ballot_sync(~0u, l_q1 > l_q0) & (lane_of == 31 ? 0u : ~0u << (lane_of + 1));
#pragma unroll 1
            while (found == 0 && chunk < a.seqs) {
              chunk += 32;
              hold(a);
              found = __ballot_sync(~0u, l_q1 > l_q0);
            }
            if (found == 0) end = pos;  // the offsets changed under the call
            else enter(a, __ffs(found) - 1);
          }
        }
      }
      // a block without keys goes to the share where it begins
      if (t1 <= t0 && !(tiles == 0 && from == 0)) continue;
      g.kh = my_kh;
      g.k0 = my_k0;
      g.kv_len = my_kv;
      g.q_end = my_q1;
      g.tok[0] = tok;
      g.ntok[0] = min(a.tile_tokens, my_q1 - tok);
      g.tok[1] = tok + g.ntok[0];
      g.ntok[1] = min(a.tile_tokens, my_q1 - g.tok[1]);
      g.split = g.first = g.seq = g.gaps = 0;
      g.t0 = t0;
      for (int s = 0; s < 2; ++s) {
        // tiles up to the last key that the row tile's last token sees
        const int32_t lim = a.causal ? my_kv - (my_q1 - g.tok[s] - g.ntok[s]) : my_kv;
        g.n[s] = g.ntok[s] > 0 ? max(min(tiles_of(lim), t1) - t0, 0) : 0;
      }
      g.slot = -1;
      if (t1 - t0 < tiles) {
        g.slot = 2 * static_cast<int32_t>(blockIdx.x) + (t0 == 0);
        if (t0 == 0 && (threadIdx.x & 31) == 0) {
          const int64_t last = (at + kBlockCost + static_cast<int64_t>(tiles - 1) * kTile) / share;
          a.cuts[blockIdx.x] = CutBlock{tok, {g.ntok[0], g.ntok[1]}, my_kh,
                                        static_cast<int32_t>(last - blockIdx.x)};
        }
      }
      return true;
    }
  }
};

// Keys of sequence b, and those of them that lie behind the prefix.
__device__ __forceinline__ int32_t seen_tokens(const AttendArgs& a, int64_t b) {
  return clamp_to(a.lens[b], a.max_pages << a.page_log2);
}
__device__ __forceinline__ int32_t own_of(const AttendArgs& a, int32_t len) {
  return max(clamp_to(len, a.max_pages << a.page_log2) - static_cast<int32_t>(a.prefix_len), 0);
}
__device__ __forceinline__ int32_t own_tokens(const AttendArgs& a, int64_t b) {
  return own_of(a, a.lens[b]);
}

// Pages: the work is a line of units (fewer than 2^31), cut into equal shares,
// one per CTA: first the prefix (key/value head, block of the batch), then
// every sequence's own tokens (sequence, key/value head). Each such group is
// as long as it is dear: kSegCost for itself and a cost for each of its key
// tiles, which falls to the share that holds the tile's first unit. A share is
// a list of segments, a group's tiles each; segment (group g, CTA x) has slot
// g + x, which grows along the line: no two segments share one. The costs are
// fitted to two batches, and where the cuts fall moves the best point with any
// change of the kernel: (group, one row tile, two) = (12, 4, 6) takes 53.8 us
// for 64 chat sequences behind 8192 shared tokens and 105 for 128 behind 32768;
// (8, 4, 5) 53.0 and 104, (12, 4, 7) 56.0 and 117, (20, 4, 7) 51.1 and 108.
constexpr int32_t kSegCost = 12;
constexpr int32_t kTileCost = 4;        // one row tile
constexpr int32_t kTwoTileCost = 6;     // two row tiles, bound by products

struct PagedSchedule {
  int32_t pos, end, prefix_units;
  int32_t prefix_row = 0;
  int32_t turn = 0;     // tiles of split segments so far: the streams take turns
  int32_t chunk = 0;
  int32_t before = 0;   // own units before the chunk
  bool loaded = false;
  int32_t mine;         // own tokens of the lane's sequence
  int32_t upto;

  // Units of a group with n key tiles.
  __device__ static int32_t group_units(int32_t n, int32_t cost) {
    return n > 0 ? n * cost + kSegCost : 0;
  }
  __device__ static int32_t prefix_cost(const AttendArgs& a) {
    return a.prefix_split || a.prefix_tiles == 0 ? kTileCost : kTwoTileCost;
  }
  // Never less than a tile: between a group's first and last segment each
  // share then begins some tile, so that no slot between theirs is empty.
  __device__ static int32_t share_of(const AttendArgs& a, int32_t all, int32_t grid) {
    return max(static_cast<int32_t>((static_cast<uint32_t>(all) + grid - 1) / grid),
               prefix_cost(a));
  }
  __device__ static int32_t prefix_group(const AttendArgs& a) {
    return group_units(a.prefix_tiles, prefix_cost(a));
  }
  __device__ static int32_t own_group(int32_t tokens) {
    return group_units(tiles_of(tokens), kTileCost);
  }
  __device__ static int32_t units(const AttendArgs& a) {
    return a.kv_heads * a.prefix_blocks * prefix_group(a);
  }
  __device__ explicit PagedSchedule(const AttendArgs& a) {
    const int lane = threadIdx.x & 31;
    prefix_units = units(a);
    // By default the prefix is the first row's that holds pages: empty slots
    // of a cache (length 0, first entry negative) may stand before it.
    bool look = a.prefix_pages == a.tables && a.prefix_tiles > 0;
    // CTA 0 also writes down where each sequence's units start.
    const bool first = blockIdx.x == 0;
    int32_t own_units = 0, next_len = lane < a.tokens ? a.lens[lane] : 0;
#pragma unroll 1
    for (int64_t b0 = 0; b0 < a.tokens; b0 += 32) {
      const int64_t b = b0 + lane;
      const int32_t len = next_len, n = own_group(own_of(a, len)) * a.kv_heads;
      next_len = b + 32 < a.tokens ? a.lens[b + 32] : 0;
      if (look) {
        const uint32_t found = __ballot_sync(
            ~0u, len > 0 || (b < a.tokens && a.tables[b * a.ld_tables] >= 0));
        if (found != 0) {
          prefix_row = static_cast<int32_t>(b0) + __ffs(found) - 1;
          look = false;
        }
      }
      if (first) {
        const int32_t inc = static_cast<int32_t>(warp_sum_upto(n));
        if (b < a.tokens) a.starts[b] = own_units + inc - n;
        own_units += __shfl_sync(~0u, inc, 31);
      } else {
        own_units += n;  // the lane's share of the sum
      }
    }
    if (!first) own_units = __shfl_sync(~0u, warp_sum_upto(own_units), 31);
    if (first && lane == 0) a.starts[a.tokens] = own_units;
    const int32_t all = prefix_units + own_units, share = share_of(a, all, gridDim.x);
    const int64_t from = static_cast<int64_t>(share) * blockIdx.x;
    pos = static_cast<int32_t>(min(from, static_cast<int64_t>(all)));
    end = static_cast<int32_t>(min(from + share, static_cast<int64_t>(all)));
  }

  // The tiles of a group of `units` whose units at, at + 1, ... are next in
  // this CTA's share: from t0, n of them (0: only a part of a cost).
  __device__ int32_t take(int32_t at, int32_t units, int32_t cost, int32_t& t0) {
    const int32_t m = min(units - at, end - pos);
    pos += m;
    t0 = max(at - kSegCost + cost - 1, 0) / cost;
    return max(at + m - kSegCost + cost - 1, 0) / cost - t0;
  }
  __device__ void split(Seg& g, int32_t n) {
    g.first = turn & 1;
    turn += n;
    g.n[g.first] = (n + 1) / 2;
    g.n[1 - g.first] = n / 2;
  }

  // As above, of the prefix; rows that see nothing of it do not count.
  __device__ static int32_t first_masked(const AttendArgs& a, const Seg& g) {
    if (g.seq >= 0) return kNone;
    int32_t least = kNone;
#pragma unroll 1
    for (int32_t b = g.tok[0] + (threadIdx.x & 31); b < g.tok[1] + g.ntok[1]; b += 32) {
      const int32_t n = seen_tokens(a, b);
      if (n > 0 && n < a.prefix_len) least = min(least, n);
    }
    least = __reduce_min_sync(~0u, least);
    return least == kNone ? kNone : least / kTile;
  }

  // Whether a page of the segment's tiles is missing: looked up here, ahead
  // of the streams, which then need no table.
  __device__ static void find_gaps(const AttendArgs& a, Seg& g, int32_t n) {
    const int32_t end = g.seq < 0 ? static_cast<int32_t>(a.prefix_len) : g.kv_len;
    const int32_t k1 = end - g.t0 * kTile > n * kTile ? (g.t0 + n) * kTile : end;
    const int32_t p1 = (k1 + a.page_size - 1) >> a.page_log2;
    bool none = false;
#pragma unroll 1
    for (int32_t p = ((g.t0 * kTile) >> a.page_log2) + (threadIdx.x & 31); p < p1; p += 32)
      none |= page_of(a, g.seq, static_cast<int64_t>(p) << a.page_log2) >= a.num_pages;
    g.gaps = __any_sync(~0u, none);
  }

  __device__ bool next(const AttendArgs& a, Seg& g) {
    const int lane = threadIdx.x & 31;
    int32_t n = 0;
#pragma unroll 1
    while (n == 0) {
      if (pos >= end) return false;
      if (pos < prefix_units) {
        const int32_t per = prefix_group(a), pg = pos / per;
        n = take(pos - pg * per, per, prefix_cost(a), g.t0);
        g.kh = pg / a.prefix_blocks;
        g.seq = ~prefix_row;
        g.kv_len = 0;
        g.slot = pg + static_cast<int32_t>(blockIdx.x);
        g.split = a.prefix_split;
        g.tok[0] = (pg - g.kh * a.prefix_blocks) * (g.split ? 1 : 2) * a.tile_tokens;
      } else {
        const int32_t at = pos - prefix_units;
#pragma unroll 1
        for (;; chunk += 32, loaded = false) {
          if (chunk >= a.tokens) return false;  // the lengths changed under the call
          if (!loaded) {
            const int64_t b = static_cast<int64_t>(chunk) + lane;
            mine = b < a.tokens ? own_tokens(a, b) : 0;
            upto = static_cast<int32_t>(
                warp_sum_upto(own_group(mine) * a.kv_heads));
            loaded = true;
          }
          const int32_t all = __shfl_sync(~0u, upto, 31);
          if (at - before < all) break;
          before += all;
        }
        const int src = __ffs(__ballot_sync(~0u, upto > at - before)) - 1;
        g.kv_len = __shfl_sync(~0u, mine, src);
        const int32_t per = own_group(g.kv_len);
        const int32_t rel = at - before - (__shfl_sync(~0u, upto, src) - per * a.kv_heads);
        g.kh = rel / per;
        n = take(rel - g.kh * per, per, kTileCost, g.t0);
        g.seq = chunk + src;
        g.slot = g.seq * a.kv_heads + g.kh + static_cast<int32_t>(blockIdx.x);
        g.split = 1;
        g.tok[0] = g.seq;
      }
    }
    const int32_t rows = static_cast<int32_t>(a.tokens);
    g.k0 = g.q_end = 0;
    g.ntok[0] = g.seq < 0 ? min(a.tile_tokens, rows - g.tok[0]) : 1;
    g.tok[1] = g.tok[0] + g.ntok[0];
    g.ntok[1] = g.split ? 0 : min(a.tile_tokens, rows - g.tok[1]);
    if (g.split) {
      split(g, n);
    } else {
      g.first = 0;
      g.n[0] = n;
      g.n[1] = g.ntok[1] > 0 ? n : 0;
    }
    find_gaps(a, g, n);
    return true;
  }
};

template <bool PAGED>
struct ScheduleOf { using type = PromptSchedule; };
template <>
struct ScheduleOf<true> { using type = PagedSchedule; };

// Address of key (or value) j of a segment; nullptr where none is.
template <typename T, bool PAGED>
__device__ __forceinline__ const T* row_at(const AttendArgs& a, const Seg& g, const void* base,
                                           int64_t sn, int64_t st, int64_t sh, int64_t j) {
  if constexpr (PAGED) {
    const int32_t id = page_of(a, g.seq, j);
    if (id >= a.num_pages) return nullptr;
    return static_cast<const T*>(base) + id * sn + (j & (a.page_size - 1)) * st + g.kh * sh;
  } else {
    if (g.k0 + j >= a.total_k) return nullptr;
    return static_cast<const T*>(base) + (g.k0 + j) * st + g.kh * sh;
  }
}

// ---- rows with infinities or NaN in places that they do not see ------------

// A masked weight is 0, but 0 times an infinite or NaN value is NaN.

// To 32 rows of a segment (rows 32 w ... of stream s) the values that were made
// finite in the products and that the row sees. Rows are taken in the order of
// their ends, so that each key is read once. Weights are over 0, so that the
// sum of such values is what they make of an output, infinite or NaN.
template <typename T, int DP, bool PAGED>
__device__ __forceinline__ void add_seen(const AttendArgs& a, const Seg& g, int s, int w) {
  const int lane = threadIdx.x & 31, row = 32 * w + lane, rt = row / a.group;
  const int qs = g.split ? 0 : s;
  const bool valid = rt < g.ntok[qs];
  const int32_t tok = g.tok[qs] + rt, head = g.kh * a.group + row % a.group;
  int32_t lim = 0;
  T* out = nullptr;
  float* part = nullptr;
  if (valid) {
    if constexpr (PAGED) lim = min(seen_tokens(a, tok), static_cast<int32_t>(a.prefix_len));
    else lim = g.kv_len - (g.q_end - 1 - tok);
    if (PAGED || g.slot >= 0)
      part = a.prefix_o + (g.slot * 256ll + (s ^ g.first) * kTile) * DP + row * 4;
    else
      out = static_cast<T*>(a.out) + tok * a.o_st + head * a.o_sh;
  }
  const int32_t step = g.split ? 2 : 1, first = g.t0 + (g.split ? s ^ g.first : 0);
  float sum[4] = {0.f, 0.f, 0.f, 0.f};  // of dimension lane + 32 e
  uint32_t rows = __ballot_sync(~0u, lim > 0);
  int32_t i = max(g.sane - first + step - 1, 0) / step, at = 0;  // tile, key of it
#pragma unroll 1
  while (rows != 0) {
    const int32_t mine = (rows >> lane) & 1 ? lim : kNone;
    const int32_t least = __reduce_min_sync(~0u, mine);
    const int src = __ffs(__ballot_sync(~0u, mine == least) & rows) - 1;
    rows &= ~(1u << src);
#pragma unroll 1
    while (i < g.n[s]) {
      const int64_t j = static_cast<int64_t>(first + i * step) * kTile + at;
      if (j >= least) break;
      const T* v = row_at<T, PAGED>(a, g, a.v, a.v_sn, a.v_st, a.v_sh, j);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = v && lane + 32 * e < a.dim ? to_f(v[lane + 32 * e]) : 0.f;
        if (!finite(x)) sum[e] += x;
      }
      if (++at == kTile) {
        at = 0;
        ++i;
      }
    }
    T* o = reinterpret_cast<T*>(
        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(out), src));
    float* p = reinterpret_cast<float*>(
        __shfl_sync(~0u, reinterpret_cast<unsigned long long>(part), src));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = lane + 32 * e;
      if (d >= a.dim || sum[e] == 0.f) continue;
      if (PAGED || p) p[d / 4 * (4 * kTile) + d % 4] += sum[e];
      else o[d] = from_f<T>(to_f(o[d]) + sum[e]);
    }
  }
}

// Behind pass 1: that for all segments of the CTA, by four warps (number w).
template <typename T, int DP, bool PAGED>
__device__ __forceinline__ void add_all_seen(const AttendArgs& a, int w) {
  typename ScheduleOf<PAGED>::type list(a);
  Seg g;
#pragma unroll 1
  while (list.next(a, g)) {
    g.sane = list.first_masked(a, g);
#pragma unroll 1
    for (int i = w; i < 8 && g.sane != kNone; i += 4) add_seen<T, DP, PAGED>(a, g, i >> 2, i & 3);
  }
}

// ---- roles ------------------------------------------------------------------

template <int DP>
struct Cta {
  unsigned char* base;
  __device__ unsigned char* q(int s) const { return base + s * Layout<DP>::kBytes; }
  __device__ unsigned char* stage(int i) const {
    return base + Layout<DP>::kRing + i * Layout<DP>::kBytes;
  }
  __device__ Ctrl* ctrl() const { return reinterpret_cast<Ctrl*>(base + Layout<DP>::kCtrl); }
};

// Where a role stands in the ring of K and V stages.
template <int DP>
struct Ring {
  int stage = 0;
  uint32_t round = 0;
  __device__ void next() {
    if (++stage == Layout<DP>::kStages) stage = 0, ++round;
  }
};

// Segment `k` of the list, for one warp (or for one thread alone); `last` lets
// go of its entry.
template <bool WARP>
__device__ __forceinline__ bool take_seg(Ctrl* c, uint32_t k, Seg& g, bool last, unsigned site) {
  const int i = k % kSegs;
  const uint32_t parity = (k / kSegs) & 1;
  if (!(WARP ? wait_warp(&c->seg_full[i], parity, c, site)
             : wait(&c->seg_full[i], parity, c, site)))
    return false;
  g = c->seg[i];
  if (last) {
    if (WARP) __syncwarp();
    if (!WARP || (threadIdx.x & 31) == 0) mbar_arrive(&c->seg_empty[i]);
  }
  return true;
}

// A place in the list of key tiles of all segments; n = 0 in a segment without
// any.
template <bool WARP>
struct Place {
  Seg g;
  uint32_t k = 0;         // segments taken
  int32_t j = -1, n = 0;  // tile of n in the segment
  bool more = true;       // false behind the last segment

  __device__ __forceinline__ bool next(Ctrl* c, bool last, unsigned site) {
    if (++j < n) return true;
    if (!take_seg<WARP>(c, k, g, last, site)) return false;
    ++k;
    j = 0;
    more = g.n[0] >= 0;
    n = g.split ? g.n[0] + g.n[1] : max(g.n[0], g.n[1]);
    return true;
  }
};

// The order of the products, and of the loads for them. A tile's scores
// (Q K^T, which need K) lead its values (P V, which need V) by one tile where
// both streams take each tile (shared), by two where they take turns (split),
// across segments of one kind. `ahead`: tiles that have scores but no values.
// One step is the values of place p, or the scores of place q, or both;
// neither where both stand at a segment without tiles. (q never looks past
// such a segment: it would wait for entries that p has yet to let go of.)
template <bool WARP>
__device__ __forceinline__ void order(const Place<WARP>& p, const Place<WARP>& q, int ahead,
                                      bool& values, bool& scores) {
  const int lead = (ahead > 0 ? p.g.split : q.g.split) ? 2 : 1;
  scores = q.more && q.n > 0 && (ahead == 0 || p.g.split == q.g.split);
  values = ahead > 0 && (ahead >= lead || !scores);
}

template <int DP, bool PAGED>
__device__ void schedule(const AttendArgs& a, Cta<DP> cta) {
  Ctrl* c = cta.ctrl();
  typename ScheduleOf<PAGED>::type list(a);
  const bool again = c->pass > 0;
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    Seg g;
    const int i = k % kSegs;
    const bool more = list.next(a, g);
    if (!more) g.n[0] = -1;
    g.sane = again && more ? list.first_masked(a, g) : kNone;
    g.tail = min(g.sane, g.kv_len > 0 ? g.kv_len / kTile : kNone);
    if (k >= kSegs && !wait_warp(&c->seg_empty[i], (k / kSegs - 1) & 1, c, 16)) return;
    if ((threadIdx.x & 31) == 0) {
      c->seg[i] = g;
      mbar_arrive(&c->seg_full[i]);
    }
    __syncwarp();
    if (!more) return;
  }
}

// The loading warp: row tiles, K and V, in the order in which the products
// take them. Lane i looks up the tile's i-th page, a step ahead and compared
// only when the load is due, so that nothing waits for the table. One elected
// lane issues every copy: copies that several lanes issue at once are taken
// one by one, at about 150 cycles each (16 per tile of 16-token pages).
template <int DP, bool PAGED>
__device__ void load(const AttendArgs& a, const CUtensorMap* qm, const CUtensorMap* qm1,
                     const CUtensorMap* km, const CUtensorMap* vm, Cta<DP> cta) {
  using L = Layout<DP>;
  Ctrl* c = cta.ctrl();
  const int lane = threadIdx.x & 31;
  Ring<DP> ring;
  uint32_t used = 0, phase = 0;  // row-tile buffers: in use before, parity of the next wait
  uint32_t turn = 0;
  const int pages = PAGED && a.page_size < kTile ? kTile >> a.page_log2 : 1;
  const uint32_t page_bytes = kTile * 128 / pages;
  const uint32_t none = static_cast<uint32_t>(a.num_pages);
  const auto look_up = [&](const Place<true>& p) -> uint32_t {
    if (!PAGED || !p.more) return none;
    // the list's table, from its first page on, and how many pages are seen
    const int32_t pre = static_cast<int32_t>(a.prefix_len >> a.page_log2);
    const bool own = p.g.seq >= 0;
    const int32_t* table = (own ? a.tables + pre : a.prefix_pages) +
                           (own ? p.g.seq : ~p.g.seq) * a.ld_tables;
    const int32_t count = own ? (p.g.kv_len + a.page_size - 1) >> a.page_log2 : pre;
    const int32_t at = (((p.g.t0 + p.j) * kTile) >> a.page_log2) + lane;
    return lane < pages && at < count ? static_cast<uint32_t>(__ldg(table + at)) : none;
  };
  // A K or V tile into the ring's next stage.
  const auto put = [&](const CUtensorMap* map, const Place<true>& p, uint32_t ids) -> bool {
    uint64_t* bar = &c->kv_full[ring.stage];
    if (ring.round > 0 && !wait_warp(&c->kv_empty[ring.stage], (ring.round - 1) & 1, c, 19))
      return false;
    unsigned char* dst = cta.stage(ring.stage);
    ring.next();
    if (elect_one()) mbar_arrive_expect_tx(bar, L::kBytes);
    const int32_t t = (p.g.t0 + p.j) * kTile;
    if constexpr (PAGED) {
#pragma unroll 1
      for (int i = 0; i < pages; ++i) {
        // a page that is not there: behind the last one, where zeros are read
        const uint32_t id = min(__shfl_sync(~0u, ids, i), none);
        if (elect_one()) {
#pragma unroll
          for (int h = 0; h < L::kHalves; ++h)
            tma_load4(dst + h * L::kHalf + i * page_bytes, map, h * 64, p.g.kh,
                      t & (a.page_size - 1), static_cast<int>(id), bar);
        }
      }
    } else if (elect_one()) {
#pragma unroll
      for (int h = 0; h < L::kHalves; ++h)
        tma_load3(dst + h * L::kHalf, map, h * 64, p.g.kh, p.g.k0 + t, bar);
    }
    __syncwarp();
    return true;
  };
  Place<true> p, q;  // of the values and of the scores
  if (!q.next(c, false, 17) || !p.next(c, true, 17)) return;
  int ahead = 0;
  uint32_t tails = 0;
  uint32_t p_ids = look_up(p), q_ids = p_ids, steps = 0;
#pragma unroll 1
  while (p.more) {
    if (++steps % 64 == 0) get_on(c);
    bool values, scores;
    order(p, q, ahead, values, scores);
    if (values) {
      const Ring<DP> at = ring;
      if (!put(vm, p, p_ids)) return;
      if (p.g.t0 + p.j >= p.g.tail) {
        const uint32_t i = tails++ % kTails;
        if (lane == 0) {
          // whole pages behind the end are not loaded (zeros are)
          const int32_t t = p.g.t0 + p.j;
          const int32_t from = p.g.kv_len > 0 ? min(p.g.kv_len - t * kTile, kTile) : kTile;
          const int32_t to = PAGED ? min((from + a.page_size - 1) & -a.page_size, kTile) : kTile;
          c->tail[i] = Tail{at.stage, static_cast<int32_t>(at.round & 1), t >= p.g.sane, from, to};
          mbar_arrive(&c->tail_full[i]);
        }
        __syncwarp();
      }
    }
    if (scores) {
      if (q.j == 0) {
        // Split segments take the two row-tile buffers in turn, so that the
        // next segment's rows load while this one's are in use; shared ones
        // take both. A segment of one sequence needs that token's rows alone.
        const int first = q.g.split ? turn++ & 1 : 0;
        const int count = !q.g.split && q.g.ntok[1] > 0 ? 2 : 1;
        const bool one = PAGED && q.g.seq >= 0;
#pragma unroll 1
        for (int r = first; r < first + count; ++r) {
          if ((used >> r) & 1) {
            if (!wait_warp(&c->q_empty[r], (phase >> r) & 1, c, 18)) return;
            phase ^= 1u << r;
          }
          used |= 1u << r;
          if (elect_one()) {
            mbar_arrive_expect_tx(&c->q_full[r],
                                  L::kHalves * (one ? 1 : a.tile_tokens) * a.group * 128);
#pragma unroll
            for (int h = 0; h < L::kHalves; ++h)
              tma_load3(cta.q(r) + h * L::kHalf, one ? qm1 : qm, h * 64, q.g.kh * a.group,
                        q.g.tok[q.g.split ? 0 : r], &c->q_full[r]);
          }
          __syncwarp();
        }
      }
      if (!put(km, q, q_ids)) return;
    }
    if (scores || !values) {  // q first: p lets go of the entries it takes
      if (!q.next(c, false, 17)) return;
      q_ids = look_up(q);
      ahead += scores;
    }
    if (values || !scores) {
      if (!p.next(c, true, 17)) return;
      p_ids = look_up(p);
      ahead -= values;
    }
  }
  if (lane == 0) {
    c->tail[tails % kTails].stage = -1;  // no more
    mbar_arrive(&c->tail_full[tails % kTails]);
  }
  __syncwarp();
  // The last arrivals of the products on these barriers come before the
  // shared memory is given back.
#pragma unroll 1
  for (int i = 0; i < L::kStages; ++i) {
    const uint32_t uses = ring.round + (i < ring.stage ? 1 : 0);
    if (uses > 0 && !wait_warp(&c->kv_empty[i], (uses - 1) & 1, c, 19)) return;
  }
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    if (((used >> i) & 1) && !wait_warp(&c->q_empty[i], (phase >> i) & 1, c, 18)) return;
}

// Two values, 0 in place of those that are not finite (exponents of ones).
template <typename T>
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  constexpr uint32_t kOnes = std::is_same<T, __nv_bfloat16>::value ? 0x7f807f80u : 0x7c007c00u;
  return x & ~__vcmpeq2(x & kOnes, kOnes);
}

// The warp that clears V tiles behind their sequences' ends and, in pass 1,
// makes the rows before that finite where some row does not see them.
template <typename T, int DP>
__device__ void clear_tails(Cta<DP> cta) {
  using L = Layout<DP>;
  Ctrl* c = cta.ctrl();
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    const int i = k % kTails;
    if (!wait_warp(&c->tail_full[i], (k / kTails) & 1, c, 29)) return;
    const Tail t = c->tail[i];
    if (t.stage < 0) return;
    if (!wait_warp(&c->kv_full[t.stage], t.parity, c, 30)) return;
    if (t.sane) {
#pragma unroll 1
      for (int j = lane; j < t.from * 8 * L::kHalves; j += 32) {
        uint4* at = reinterpret_cast<uint4*>(cta.stage(t.stage) +
                                             (j >= t.from * 8 ? L::kHalf - t.from * 128 : 0)) + j;
        const uint4 x = *at;
        *at = make_uint4(finite2<T>(x.x), finite2<T>(x.y), finite2<T>(x.z), finite2<T>(x.w));
      }
    }
    // 16-byte pieces of the rows behind the end; swizzling keeps a row's
    // pieces within the row
#pragma unroll 2
    for (int j = t.from * 8 + lane; j < t.to * 8; j += 32) {
#pragma unroll
      for (int h = 0; h < L::kHalves; ++h)
        *reinterpret_cast<uint4*>(cta.stage(t.stage) + h * L::kHalf + j * 16) =
            make_uint4(0, 0, 0, 0);
    }
    async_proxy_fence();
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->tail_done[i]);
  }
}

// The thread that issues the products. In program order: the values of a
// stream's tile, then the scores of its next one into the same columns. It is
// on the way of every product, so that its loops are kept short: one for
// segments of two row tiles, with both streams written out (one copy for both,
// or the steps of order() here, cost prompts 8 to 13%), one for runs of split
// segments.
template <typename T, int DP, bool PAGED>
__device__ void multiply(const AttendArgs& a, Cta<DP> cta, uint32_t tmem) {
  using L = Layout<DP>;
  Ctrl* c = cta.ctrl();
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr uint32_t kShapeS = mma_shape(kBf16, kTile, false);
  // The products stop at the head dimension, in steps of 16.
  const int steps = (a.dim + 15) / 16;
  const uint32_t shape_o = mma_shape(kBf16, 16 * steps, true);
  const uint32_t q0 = operand(smem_addr(cta.q(0)), 16);
  const uint32_t k0 = operand(smem_addr(cta.stage(0)), 16);
  const uint32_t v0 = operand(smem_addr(cta.stage(0)), L::kHalf);
  Ring<DP> ring;
  // Bit s (or i): parities of the next waits, and whether O_s was used before.
  uint32_t q_phase = 0, p_phase = 0, o_phase = 0, o_used = 0;

  const auto full = [&]() { return wait(&c->kv_full[ring.stage], ring.round & 1, c, 20); };
  // Q K^T of stream s
  const auto scores = [&](int s, int q, int stage) {
    tc_fence_after();
    const uint32_t qa = q0 + q * (L::kBytes >> 4), kb = k0 + stage * (L::kBytes >> 4);
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) {
      const uint32_t off = ((i / 4) * L::kHalf + (i % 4) * 32) >> 4;
      if (i < (DP == 128 ? 5 : 1) || i < steps)
        mma_ss(tmem + s * kTile, qa + off, kb + off, kShapeS, i > 0);
    }
    mma_commit(&c->s_full[s]);
  };
  uint32_t tails = 0;
  const auto clean = [&]() {
    const uint32_t k = tails++;
    return wait(&c->tail_done[k % kTails], (k / kTails) & 1, c, 31);
  };
  // P V of stream s
  const auto values = [&](int s, bool first, int stage) -> bool {
    if (first) {
      if ((o_used >> s) & 1) {
        if (!wait(&c->o_free[s], (o_phase >> s) & 1, c, 22)) return false;
        o_phase ^= 1u << s;
      }
      o_used |= 1u << s;
    }
    const uint32_t vb = v0 + stage * (L::kBytes >> 4);
    const uint32_t o = tmem + 2 * kTile + s * kTile, w = tmem + s * kTile;
#pragma unroll
    for (int p = 0; p < kParts; ++p) {
      if (!wait(&c->p_full[s][p], (p_phase >> s) & 1, c, 21)) return false;
      tc_fence_after();
      constexpr int kSteps = kTile / 16 / kParts;
#pragma unroll
      for (int e = 0; e < kSteps; ++e)
        mma_ts(o, w + (p * kSteps + e) * 8, vb + (((p * kSteps + e) * 2048) >> 4), shape_o,
               !first || p > 0 || e > 0);
    }
    p_phase ^= 1u << s;
    mma_commit(&c->o_done[s]);
    return true;
  };

  Place<false> p;
  if (!p.next(c, true, 23)) return;
  uint32_t turn = 0;
#pragma unroll 1
  while (p.more) {
    if (!PAGED || !p.g.split) {
      const Seg& g = p.g;
      const int32_t n = p.n;
      const int tiles = g.ntok[1] > 0 ? 2 : 1;
      const int32_t tail = g.tail - g.t0;
      if (n > 0) {
#pragma unroll 1
        for (int i = 0; i < tiles; ++i) {
          if (!wait(&c->q_full[i], (q_phase >> i) & 1, c, 24)) return;
          q_phase ^= 1u << i;
        }
        if (!full()) return;
#pragma unroll
        for (int s = 0; s < 2; ++s)
          if (g.n[s] > 0) scores(s, s, ring.stage);
        mma_commit(&c->kv_empty[ring.stage]);
        ring.next();
      }
#pragma unroll 1
      for (int32_t j = 0; j < n; ++j) {
        // V_j in the current stage, K_{j+1} in the next one
        if (j + 1 == n) {
#pragma unroll 1
          for (int i = 0; i < tiles; ++i) mma_commit(&c->q_empty[i]);
        }
        if (!full()) return;
        if (j >= tail && !clean()) return;
        const int v = ring.stage;
        ring.next();
        bool have = false;
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          if (j < g.n[s]) {
            if (!values(s, j == 0, v)) return;
          }
          if (s == 1) mma_commit(&c->kv_empty[v]);
          if (j + 1 < g.n[s]) {
            if (!have && !full()) return;
            have = true;
            scores(s, s, ring.stage);
          }
        }
        if (j + 1 < n) {
          mma_commit(&c->kv_empty[ring.stage]);
          ring.next();
        }
      }
      p.j = n;
      if (!p.next(c, true, 23)) return;
      continue;
    }
    // A run of split segments: scores at place q, two tiles before the values
    // at p, the streams taking turns.
    Place<false> q = p;
    int ahead = 0, rows = 0;
#pragma unroll 1
    for (;;) {
      const bool more = q.more && q.g.split, late = ahead == 2 || !more;
      if (late) {
        if (ahead == 0) break;
        if (!full()) return;
        if (p.g.t0 + p.j >= p.g.tail && !clean()) return;
        const int v = ring.stage;
        ring.next();
        if (!values((p.j & 1) ^ p.g.first, p.j < 2, v)) return;
        mma_commit(&c->kv_empty[v]);
      }
      if (more) {
        if (q.j == 0) {
          rows = turn++ & 1;
          if (!wait(&c->q_full[rows], (q_phase >> rows) & 1, c, 24)) return;
          q_phase ^= 1u << rows;
        }
        if (!full()) return;
        scores((q.j & 1) ^ q.g.first, rows, ring.stage);
        mma_commit(&c->kv_empty[ring.stage]);
        ring.next();
        if (q.j + 1 == q.n) mma_commit(&c->q_empty[rows]);
        if (!q.next(c, false, 23)) return;
        ++ahead;
      }
      if (late) {
        if (!p.next(c, true, 23)) return;
        --ahead;
      }
    }
  }
}

// Four warps of stream s, one row per thread. What the output needs of the
// segment is read again behind the tiles: between them 128 scores fill the
// registers.
template <typename T, int DP, bool PAGED>
__device__ void soften(const AttendArgs& a, Cta<DP> cta, uint32_t tmem, int s) {
  Ctrl* c = cta.ctrl();
  const int lane = threadIdx.x & 31;
  const int32_t row = threadIdx.x & 127;
  const int32_t rt = row / a.group, head0 = row % a.group;  // token of the tile, head of the group
  const uint32_t lanes = static_cast<uint32_t>(row & ~31) << 16;
  const uint32_t ts = tmem + lanes + s * kTile, to = tmem + lanes + 2 * kTile + s * kTile;
  const float grow = fminf(kGrow / a.c, 3e38f);  // finite, so that -inf + grow stays -inf
  uint32_t done = 0;
#pragma unroll 1
  for (uint32_t k = 0;; ++k) {
    if (!wait_warp(&c->seg_full[k % kSegs], (k / kSegs) & 1, c, 25)) return;
    const Seg& g = c->seg[k % kSegs];
    if (g.n[0] < 0) return;
    const int qs = g.split ? 0 : s;
    const int32_t n = g.n[s];
    const bool valid = rt < g.ntok[qs];  // ntok <= tile_tokens
    const int32_t tile0 = g.split ? g.t0 + (s ^ g.first) : g.t0, tile_step = g.split ? 2 : 1;
    const bool gaps = PAGED && g.gaps;
    // keys that the row sees, of the segment's list; rows of no token are
    // not masked at all (nothing is written for them)
    int32_t lim = 0x7fffffff;
    if (valid) {
      const int32_t tok = g.tok[qs] + rt;
      if constexpr (PAGED) {
        lim = g.seq < 0 ? min(seen_tokens(a, tok), static_cast<int32_t>(a.prefix_len))
                        : g.kv_len;
      } else {
        lim = a.causal ? g.kv_len - (g.q_end - 1 - tok) : g.kv_len;
      }
    }
    const bool busy = __any_sync(~0u, valid);  // else the warp only keeps step
    float base = neg_inf(), l = 0.f;  // the row's base, in units of <q, k>
#pragma unroll 1
    for (int32_t i = 0; i < n; ++i) {
      const int32_t t = tile0 + i * tile_step;
      uint32_t bad = 0;  // groups of 16 keys whose page is not there
      if (gaps) {
        bool none = false;
        if (lane < kTile / 16)
          none = page_of(a, g.seq, static_cast<int64_t>(t) * kTile + lane * 16) >= a.num_pages;
        bad = __ballot_sync(~0u, none);
      }
      if (!wait_warp(&c->s_full[s], done & 1, c, 26)) return;
      ++done;
      tc_fence_after();
      if (!busy) {
        for (int p = 0; p < kParts; ++p) mbar_arrive(&c->p_full[s][p]);
        continue;
      }
      float x[kTile];
#pragma unroll
      for (int b = 0; b < kTile / 16; ++b)
        tmem_load16(ts + 16 * b, *reinterpret_cast<uint32_t(*)[16]>(x + 16 * b));
      tmem_wait_load();
      const int32_t rel = lim - t * kTile;
      if (rel < kTile || bad != 0) {
        // bit j of word b: key 32 b + j of the tile is seen
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int r = rel - 32 * b;
          uint32_t see = r >= 32 ? ~0u : r <= 0 ? 0u : (1u << r) - 1;
          if (PAGED) {
            if ((bad >> (2 * b)) & 1) see &= 0xffff0000u;
            if ((bad >> (2 * b + 1)) & 1) see &= 0x0000ffffu;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) x[32 * b + j] = (see >> j) & 1 ? x[32 * b + j] : neg_inf();
        }
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int j = 4; j < kTile - 4; j += 8) {
#pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], x[j + e], x[j + 4 + e]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], x[kTile - 4 + e]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      if (__any_sync(~0u, valid && top > base + grow)) {
        const float was = base;
        base = fmaxf(base, top);
        if (i > 0) {
          const float f = was == base ? 1.f : ex2((was - base) * a.c);
          l *= f;
          if (!wait_warp(&c->o_done[s], (done - 2) & 1, c, 27)) return;
          tc_fence_after();
#pragma unroll 1
          for (int b = 0; b < DP; b += 32) {
            uint32_t o[32];
            tmem_load32(to + b, o);
            tmem_wait_load();
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_store32(to + b, o);
          }
        }
      }
      // base is -inf while the row has seen no key: every x is -inf then
      const float shift = base == neg_inf() ? 0.f : -base * a.c;
      const float2 cc = make_float2(a.c, a.c), sh = make_float2(shift, shift);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        uint32_t p[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int e = b * 32 + 2 * j;
          float2 y = fma2(make_float2(x[e], x[e + 1]), cc, sh);
          y.x = ex2(y.x);
          y.y = ex2(y.y);
          sum[j & 1] = add2(sum[j & 1], y);
          p[j] = pack2(y.x, y.y, T());
        }
        tmem_store16(ts + 16 * b, p);
        if ((b + 1) % (4 / kParts) == 0) {
          tmem_wait_store();
          tc_fence_before();
          mbar_arrive(&c->p_full[s][b / (4 / kParts)]);
        }
      }
      sum[0] = add2(sum[0], sum[1]);
      l += sum[0].x + sum[0].y;
    }

    // The output. l is 0 only where no key was seen.
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float lse = l == 0.f ? neg_inf() : base * a.c + log2f(l);
    const int32_t head = g.kh * a.group + head0, tok = g.tok[qs] + rt;
    T* out = nullptr;
    float *part = nullptr, *lse_at = nullptr;
    // from four values of a partial output to the next
    const int step = !PAGED || g.seq < 0 ? 4 * kTile : 4;
    if (valid) {
      if (PAGED && g.seq >= 0) {
        const int64_t r = (g.slot * 2ll + (s ^ g.first)) * a.group + row;
        part = a.own_o + r * DP;
        lse_at = a.own_lse + r;
      } else if (PAGED || g.slot >= 0) {
        const int64_t r = g.slot * 256ll + (s ^ g.first) * kTile;
        part = a.prefix_o + r * DP + row * 4;
        lse_at = a.prefix_lse + r + row;
      } else {
        out = static_cast<T*>(a.out) + tok * a.o_st + head * a.o_sh;
        if (a.lse) lse_at = a.lse + tok * a.l_st + head * a.l_sh;
      }
    }
    T* quad[4];  // the rows of this thread and its three neighbours
#pragma unroll
    for (int j = 0; j < 4; ++j)
      quad[j] = PAGED ? nullptr
                      : reinterpret_cast<T*>(__shfl_sync(
                            ~0u, reinterpret_cast<unsigned long long>(out), (lane & ~3) + j));
    // NaN once a value is not finite: 0 times each, summed in pairs (a test of
    // each took 10 us of 115 for 128 sequences behind a shared document)
    float2 odd = make_float2(0.f, 0.f);
    if (n > 0) {
      if (!wait_warp(&c->o_done[s], (done - 1) & 1, c, 28)) return;
      tc_fence_after();
    }
#pragma unroll 1
    for (int b = 0; b < DP; b += 32) {
      float o[32];
      if (n > 0 && busy) {
        tmem_load32(to + b, *reinterpret_cast<uint32_t(*)[32]>(o));
        tmem_wait_load();
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = l == 0.f ? 0.f : o[j] * inv;
      // columns behind the last step of 16 of the products hold anything
#pragma unroll
      for (int h = 0; h < 32; h += 16) {
        float2 z = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = h; j < h + 16; j += 2)
          z = fma2(make_float2(o[j], o[j + 1]), make_float2(0.f, 0.f), z);
        if (b + h < a.dim) odd = add2(odd, z);
      }
      if (part) {
#pragma unroll
        for (int j = 0; j < 32; j += 4)
          *reinterpret_cast<float4*>(part + (b + j) / 4 * step) =
              make_float4(o[j], o[j + 1], o[j + 2], o[j + 3]);
      } else if (!PAGED && g.slot < 0) {
        // Rows lie apart: four neighbouring threads change their 16-byte
        // pieces about, so that each row gets 64 bytes at a time (a quarter
        // of the lines per store).
        uint32_t u[4][4];
#pragma unroll
        for (int j = 0; j < 32; j += 2) u[j / 8][j % 8 / 2] = pack2(o[j], o[j + 1], T());
#pragma unroll
        for (int m = 1; m <= 2; m *= 2) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (j & m) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t mine = lane & m ? u[j][e] : u[j | m][e];
              const uint32_t other = __shfl_xor_sync(~0u, mine, m);
              if (lane & m) u[j][e] = other;
              else u[j | m][e] = other;
            }
          }
        }
        const int32_t d = b + 8 * (lane & 3);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (quad[j] && d < a.dim)
            *reinterpret_cast<uint4*>(quad[j] + d) = make_uint4(u[j][0], u[j][1], u[j][2], u[j][3]);
      }
    }
    if (n > 0) {
      tc_fence_before();
      mbar_arrive(&c->o_free[s]);
    }
    if (lse_at) *lse_at = lse;

    // whether the tiles hold keys that the row does not see (what lies behind
    // the sequence's end was cleared)
    const int32_t tiles = n > 0 ? tile0 + (n - 1) * tile_step + 1 : 0;
    if (valid && !finite(odd.x + odd.y) && lim < static_cast<int64_t>(tiles) * kTile &&
        lim < (PAGED && g.seq < 0 ? a.prefix_len : g.kv_len))
      c->doubt = 1;
    __syncwarp();
    if (lane == 0) mbar_arrive(&c->seg_empty[k % kSegs]);
  }
}

// By one warp, each lane the barriers of its number; with `old` ones to give up.
template <int DP>
__device__ __forceinline__ void init_barriers(Ctrl* c, bool old = false) {
  const int i = threadIdx.x & 31;
  const auto init = [&](uint64_t* bar, uint32_t count) {
    if (old) mbar_inval(bar);
    mbar_init(bar, count);
  };
  if (i < Layout<DP>::kStages) {
    init(&c->kv_full[i], 1);
    init(&c->kv_empty[i], 1);
  }
  if (i < 2) {
    init(&c->q_full[i], 1);
    init(&c->q_empty[i], 1);
    init(&c->s_full[i], 1);
    for (int p = 0; p < kParts; ++p) init(&c->p_full[i][p], kTile);
    init(&c->o_done[i], 1);
    init(&c->o_free[i], kTile);
  }
  if (i < kSegs) {
    init(&c->seg_full[i], 1);
    init(&c->seg_empty[i], 10);  // the loading and multiplying roles, eight warps
  }
  if (i < kTails) {
    init(&c->tail_full[i], 1);
    init(&c->tail_done[i], 1);
  }
}

// The end of every role in a pass: whether there is another one. All copies and
// products have landed by then (load() and soften() waited for them), so that
// the barriers can start anew.
template <int DP>
__device__ __forceinline__ bool again(Ctrl* c) {
  const auto together = [] {
    asm volatile("bar.sync 1, %0;" ::"n"(kAttendThreads) : "memory");
  };
  __syncwarp();
  tc_fence_before();
  together();
  if (c->doubt == 0 || c->pass > 0 || c->dead) return false;
  together();
  if (threadIdx.x >= kAttendThreads - 32) {
    init_barriers<DP>(c, true);
    c->pass = 1;
    get_on(c);
    mbar_init_fence();
  }
  together();
  tc_fence_after();
  return true;
}

template <typename T, int DP, bool PAGED>
__global__ void __launch_bounds__(kAttendThreads, 1)
    attend_kernel(const __grid_constant__ CUtensorMap qm, const __grid_constant__ CUtensorMap q1,
                  const __grid_constant__ CUtensorMap km, const __grid_constant__ CUtensorMap vm,
                  const __grid_constant__ AttendArgs a) {
  using L = Layout<DP>;
  extern __shared__ unsigned char raw[];
  Cta<DP> cta;
  cta.base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);  // swizzle atoms are 1 KiB
  Ctrl* c = cta.ctrl();
  const int warp = threadIdx.x >> 5;
  if (warp == 0) {
    init_barriers<DP>(c);
    if (threadIdx.x == 0) c->dead = c->doubt = c->pass = 0;
    mbar_init_fence();
  }
  if (warp == 8) {
    tmem_alloc(&c->tmem);
  } else if (warp == 10) {
    get_on(c);
  } else if (warp == 9 && (threadIdx.x & 31) == 0) {
    tma_prefetch(PAGED ? &q1 : &qm);
    tma_prefetch(&km);
    tma_prefetch(&vm);
  }
  // Rows that no token of a tile fills are products of zeros.
  const int used = a.tile_tokens * a.group;
  for (int i = threadIdx.x; i < 2 * L::kHalves * (kTile - used) * 8; i += kAttendThreads) {
    const int tile = i / ((kTile - used) * 8), rest = i % ((kTile - used) * 8);
    *reinterpret_cast<uint4*>(cta.base + tile * L::kHalf + used * 128 + rest * 16) =
        make_uint4(0, 0, 0, 0);
  }
  async_proxy_fence();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  // 168 registers a thread at the launch: 256 x 216 + 128 x 72 = 384 x 168.
  if (warp < 8) {
    reg_grow<216>();
#pragma unroll 1
    do soften<T, DP, PAGED>(a, cta, tmem, warp >> 2);
    while (again<DP>(c));
  } else {
    reg_shrink<72>();
#pragma unroll 1
    do {
      if (warp == 8) {
        if (elect_one()) multiply<T, DP, PAGED>(a, cta, tmem);
      } else if (warp == 9) {
        load<DP, PAGED>(a, &qm, &q1, &km, &vm, cta);
      } else if (warp == 10) {
        schedule<DP, PAGED>(a, cta);
      } else {
        clear_tails<T, DP>(cta);
      }
    } while (again<DP>(c));
    if (c->pass > 0 && !c->dead) add_all_seen<T, DP, PAGED>(a, warp - 8);
  }
  if (c->dead) {
    // A wait gave up: loads and products may still be under way. Give them
    // time to land before the memory is handed on.
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 10000000ull) __nanosleep(100000);
    __syncthreads();
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_free(tmem);
  }
}

// ---- partial outputs of the paged form joined -------------------------------

// One warp per (sequence, head): the partial outputs of its prefix segments
// and of its own ones, weighted by 2^(lse_i - F) with F the log-sum-exp of
// their log-sum-exps. Bound by its chain of loads (starts, log-sum-exps,
// outputs): 9 us for 2048 rows, launched under the kernel before it.
struct JoinArgs {
  void* out;
  int64_t o_sb, o_sh;
  float* lse;
  int64_t l_sb, l_sh;
  int32_t grid;  // CTAs that shared the work
};
constexpr int kJoinWarps = 4;

template <typename T, int DP>
__global__ void __launch_bounds__(kJoinWarps * 32)
    join_kernel(const __grid_constant__ AttendArgs a, const JoinArgs j) {
  follow();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * kJoinWarps + (threadIdx.x >> 5);
  if (r >= a.tokens * a.heads) return;
  const int64_t b = r / a.heads;
  const int32_t h = static_cast<int32_t>(r - b * a.heads), kh = h / a.group, e = h - kh * a.group;
  const int32_t pre = PagedSchedule::units(a), from = a.starts[b], upto = a.starts[b + 1];
  const int32_t share = PagedSchedule::share_of(a, pre + a.starts[a.tokens], j.grid);
  // Partial i < np: prefix; np <= i < np + no: own. In both the segments of
  // one group have consecutive slots, each with one or two partials.
  int64_t p0 = 0, o0 = 0;
  int32_t np = 0, no = 0, prow = 0;
  if (a.prefix_tiles > 0) {
    const int32_t block = (a.prefix_split ? 1 : 2) * a.tile_tokens, bi = static_cast<int32_t>(b);
    const int32_t rb = bi / block, in = bi - rb * block, pg = kh * a.prefix_blocks + rb;
    const int32_t u = pg * PagedSchedule::prefix_group(a) + kSegCost;
    const int32_t c0 = u / share,
                  c1 = (u + (a.prefix_tiles - 1) * PagedSchedule::prefix_cost(a)) / share;
    const int32_t s = in >= a.tile_tokens;
    np = (c1 - c0 + 1) << a.prefix_split;
    p0 = static_cast<int64_t>(pg + c0) * 256 + s * kTile;
    prow = (in - s * a.tile_tokens) * a.group + e;
  }
  if (upto > from) {
    const int32_t per = (upto - from) / a.kv_heads, u = pre + from + kh * per + kSegCost;
    const int32_t c0 = u / share, c1 = (u + per - kSegCost - kTileCost) / share;
    no = (c1 - c0 + 1) * 2;
    o0 = (b * a.kv_heads + kh + c0) * 2 * a.group + e;
  }
  // Prefix partials: tiles of 128 rows, [DP / 4][128][4] each; own ones: rows.
  // Partial i's row is a step behind partial i - 1's.
  constexpr int kPer = DP / 32;  // values of a lane
  const int32_t all = np + no, d = lane * kPer;
  const int64_t p_step = a.prefix_split ? kTile : 2 * kTile;
  const float* p_lse = a.prefix_lse + p0 + prow;
  const float* o_lse = a.own_lse + o0;
  const float* p_out = a.prefix_o + p0 * DP + (d / 4 * kTile + prow) * 4 + d % 4;
  const float* o_out = a.own_o + o0 * DP + d;
  const auto lse_of = [&](int32_t i) {
    return i >= all ? neg_inf() : i < np ? p_lse[i * p_step] : o_lse[(i - np) * a.group];
  };
  // Lane i keeps the log-sum-exp of partial i; more than 32 are read again.
  const float held = lse_of(lane);
  float m = held;
#pragma unroll 1
  for (int32_t i = lane + 32; i < all; i += 32) m = fmaxf(m, lse_of(i));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  const float base = m == neg_inf() ? 0.f : m;
  float sum = ex2(held - base);
#pragma unroll 1
  for (int32_t i = lane + 32; i < all; i += 32) sum += ex2(lse_of(i) - base);
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const bool any = sum != 0.f;  // NaN counts
  const float lse = any ? base + log2f(sum) : neg_inf();
  using Vec = typename std::conditional<kPer == 4, float4, float2>::type;
  float acc[kPer];
  for (int d = 0; d < kPer; ++d) acc[d] = 0.f;
  // Every partial holds an output (zeros where it saw nothing), so that the
  // loads wait for no log-sum-exp.
#pragma unroll 1
  for (int32_t i0 = 0; i0 < all; i0 += 32) {
    const float w = any ? ex2((i0 == 0 ? held : lse_of(i0 + lane)) - lse) : 0.f;
    const int32_t n = min(all - i0, 32);
#pragma unroll 4
    for (int32_t i = 0; i < n; ++i) {
      const float wi = __shfl_sync(~0u, w, i);
      const int32_t k = i0 + i;
      const float* o = k < np ? p_out + k * p_step * DP
                              : o_out + static_cast<int64_t>(k - np) * a.group * DP;
      const Vec v = *reinterpret_cast<const Vec*>(o);
      acc[0] = fmaf(wi, v.x, acc[0]);
      acc[1] = fmaf(wi, v.y, acc[1]);
      if constexpr (kPer == 4) {
        acc[2] = fmaf(wi, v.z, acc[2]);
        acc[3] = fmaf(wi, v.w, acc[3]);
      }
    }
  }
  if (lane * kPer < a.dim) {
    T* out = static_cast<T*>(j.out) + b * j.o_sb + h * j.o_sh + lane * kPer;
    for (int d = 0; d < kPer; ++d) out[d] = from_f<T>(acc[d]);
  }
  if (j.lse && lane == 0) j.lse[b * j.l_sb + h * j.l_sh] = lse;
}

// The partial outputs of the blocks that are cut: CTAs (x, y) join the block
// that begins in share x and goes on, one row per thread, 32 columns each
// (14 us for 152 cut blocks of 256 rows, two parts each: 40 MB of fp32 parts;
// 15.5 us with all 128 columns in one thread).
constexpr int kJoinRows = 2 * kTile;
constexpr int kJoinCols = 32;

template <typename T, int DP>
__global__ void __launch_bounds__(kJoinRows)
    join_blocks_kernel(const __grid_constant__ AttendArgs a) {
  follow();
  const CutBlock cut = a.cuts[blockIdx.x];
  if (!joinable(cut, a, blockIdx.x, gridDim.x)) return;
  const int s = threadIdx.x >> 7, row = threadIdx.x & 127, rt = row / a.group;
  if (rt >= cut.ntok[s]) return;
  const int64_t x = blockIdx.x;
  // part i's row tile
  const auto tile_at = [&](int32_t i) -> int64_t {
    return (2 * (x + i) + (i == 0)) * 256 + s * kTile;
  };
  float m = neg_inf();
#pragma unroll 4
  for (int32_t i = 0; i <= cut.more; ++i) m = fmaxf(m, a.prefix_lse[tile_at(i) + row]);
  const float base = m == neg_inf() ? 0.f : m;
  float sum = 0.f;
  float acc[kJoinCols];
#pragma unroll
  for (int d = 0; d < kJoinCols; ++d) acc[d] = 0.f;
  const int d0 = blockIdx.y * kJoinCols;
#pragma unroll 2
  for (int32_t i = 0; i <= cut.more; ++i) {
    const int64_t r = tile_at(i);
    const float w = ex2(a.prefix_lse[r + row] - base);
    sum += w;
    const float4* o =
        reinterpret_cast<const float4*>(a.prefix_o + r * DP) + d0 / 4 * kTile + row;
#pragma unroll
    for (int d = 0; d < kJoinCols; d += 4) {
      const float4 v = o[d / 4 * kTile];
      acc[d] = fmaf(w, v.x, acc[d]);
      acc[d + 1] = fmaf(w, v.y, acc[d + 1]);
      acc[d + 2] = fmaf(w, v.z, acc[d + 2]);
      acc[d + 3] = fmaf(w, v.w, acc[d + 3]);
    }
  }
  const bool any = sum != 0.f;  // NaN counts
  const float inv = any ? 1.f / sum : 0.f;
  const int64_t tok = cut.tok + s * cut.ntok[0] + rt, head = cut.kh * a.group + row % a.group;
  T* out = static_cast<T*>(a.out) + tok * a.o_st + head * a.o_sh + d0;
#pragma unroll
  for (int d = 0; d < kJoinCols; d += 8)
    if (d0 + d < a.dim)
      *reinterpret_cast<uint4*>(out + d) =
          make_uint4(pack2(acc[d] * inv, acc[d + 1] * inv, T()),
                     pack2(acc[d + 2] * inv, acc[d + 3] * inv, T()),
                     pack2(acc[d + 4] * inv, acc[d + 5] * inv, T()),
                     pack2(acc[d + 6] * inv, acc[d + 7] * inv, T()));
  if (a.lse && d0 == 0)
    a.lse[tok * a.l_st + head * a.l_sh] = any ? base + log2f(sum) : neg_inf();
}

}  // namespace
}  // namespace dsa
