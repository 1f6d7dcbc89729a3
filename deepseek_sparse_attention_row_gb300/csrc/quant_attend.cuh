// quant_attend.cuh -- the kernels of dsa_quant_attention (include/dsa_quant.h):
// single tokens over pages of e4m3 codes.
//
// The heads that share a key/value head are the columns (8 or 16) of both
// products, and keys and dimensions their rows, so that no row of a tensor
// instruction is padding:
//   S^T [keys x heads] = K [keys x dim] Q^T,   O^T [dim x heads] += V^T P^T.
// A warp works alone: it goes through a line of 4 KiB tiles of keys (32 of up to
// 128 dimensions, 64 of up to 64), and as many of values, that cp.async brings
// into a ring of three of its own in shared memory, whole rows at a time; no
// barrier stands between a load and its use. Codes become fp16 in registers,
// which is exact; so are queries after a power of two that brings the largest of
// a row to 2^14. Weights are two fp16 numbers each, so that V^T P^T is two products.
//
// The tiles of all sequences lie on one line, in front of each sequence's a unit for
// its start. It is cut into equal shares, one for each team of as many warps as there
// are key/value heads; the warps of a team go through its share side by side, each
// with a head of its own, so that what the heads of a token have in common of a line
// of memory is there once for all (with heads of 80 bytes, a warp after the other,
// 264 MB were read where 174 would do). Sequences that lie within a share are
// finished by its warps; of the others each leaves a piece, and a second launch joins
// those by their log-sum-exps.
//
// Bound by HBM where contexts are long: 302,000 tokens of 8 heads of 128, 619 MB,
// take 100 us (6.2 TB/s, 7.3 TB/s in the loop alone), 459,000 tokens of 4 heads 80
// us (5.9 TB/s). About 8 us pass before the first tiles are done (lengths, page,
// codes: a chain of loads, then all SMs' first ones at once) and 5 at the end (the
// join). With heads of 80, 174 MB in 49.5 us, these are a quarter of the time; in the
// loop, at 5.2 TB/s, a scheduler has three warps, each of which issues every sixth
// cycle.
// What was tried while weights were one fp16 number (100.0 us for the first case, 47.9
// for heads of 80): codes through registers instead of the ring 161 us (too few bytes
// under way); 14 or 16 warps of 128 registers 110 and 117 us (heads of 80, 16 warps:
// 47.4); 8 warps with tiles of 8 KiB 102 us; pieces joined in the CTA and rows in turn
// instead of side by side 122 us; rings of four slots, with loads a whole tile further
// ahead, 108 us; heads of 80 in rows of 80 bytes, tiles of 64 keys, 54 us.
#pragma once

#include <cuda_runtime.h>

#include <cfloat>

#include "follow.cuh"
#include "quant.cuh"
#include "umma.cuh"

namespace dsa {

constexpr int kQuantTileBytes = 4096;
// What the start of a sequence takes of a share, in tiles. 128 sequences of up to 300
// tokens, 8 heads of 128: 18.7 us with 0, 17.4 with 1, 18.3 with 2; 300 of up to 700, 4
// heads of 64: 21.7, 20.9, 22.1; 33 of up to 8000, 8 heads of 80: 50.2, 49.6, 49.9; 64
// of up to 9216, 8 heads of 128: 101.0, 100.6, 101.0.
constexpr int32_t kQuantStart = 1;

struct QuantAttnArgs {
  QuantPool pool;
  const void* q;
  int64_t q_sb, q_sh;
  int64_t batch;
  int32_t group, splits, split_heads;  // a group's heads, its parts, and heads of a part
  int32_t rows;                        // kv_heads * splits
  const int32_t* lens;
  float c;  // scale * log2 e
  void* out;
  int64_t o_sb, o_sh;
  float* lse;
  int64_t l_sb, l_sh;
  int32_t bf16;
  int32_t warps;    // of the first launch
  int2* spans;      // [batch] the first and the last share of each sequence
  float* part_o;    // [2 warps][columns][DP]
  float* part_lse;  // [2 warps][columns]
};

template <int DP, int NT>
struct QuantLayout {
  static constexpr int kTile = kQuantTileBytes / DP;  // keys
  static constexpr int kHeads = 8 * NT;
  // As many as the registers let be: 16 columns take 235 to 255 of a thread (12 warps
  // of them, spilled, took 79 us where 8 took 62: groups of 16, 64 sequences, weights
  // of one fp16 number).
  static constexpr int kWarps = NT == 1 ? 12 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kRing = 3 * kQuantTileBytes;
  static constexpr int kPiece = kHeads * DP;  // floats
  static constexpr int kSmem = kWarps * kRing;
  static_assert(kPiece * 4 <= kRing, "a piece lies over its warp's ring");
};

// ---- instructions ----------------------------------------------------------

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The same, but zeros where `yes` is false (nothing is read then).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool yes) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %2, 0;\n\t"
      "cp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst),
      "l"(src), "r"(static_cast<uint32_t>(yes))
      : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void shared_words(uint32_t (&x)[4], uint32_t at) {
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void shared_words(uint32_t (&x)[2], uint32_t at) {
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(x[0]), "=r"(x[1]) : "r"(at) : "memory");
}
__device__ __forceinline__ void shared_words(uint32_t (&x)[1], uint32_t at) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(x[0]) : "r"(at) : "memory");
}
__device__ __forceinline__ uint32_t shared_half_word(uint32_t at) {
  uint32_t x;
  asm volatile("{\n\t.reg .b16 h;\n\tld.shared.u16 h, [%1];\n\tcvt.u32.u16 %0, h;\n\t}"
               : "=r"(x)
               : "r"(at)
               : "memory");
  return x;
}
// Four codes as two pairs of fp16.
__device__ __forceinline__ void decode4(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, y;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}
// [16 x 16] by [16 x 8] of fp16, added in fp32.
__device__ __forceinline__ void product(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of 16-bit elements, two of a row in each lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  return fma2(a, b, make_float2(-0.f, -0.f));
}

// ---- the line of tiles -----------------------------------------------------

// A line of `total` units cut into n shares, in 32 bits (n up to 65535): share i
// begins at floor(total * i / n). None is empty if n is not above the total.
struct Shares {
  uint32_t n, whole, rest;
  __device__ __forceinline__ Shares(int32_t total, uint32_t parts)
      : n(parts), whole(total / parts), rest(total - whole * parts) {}
  __device__ __forceinline__ int32_t begin(uint32_t i) const {
    return static_cast<int32_t>(whole * i + rest * i / n);
  }
  // The last one that begins at or before `unit` of the line.
  __device__ __forceinline__ int32_t of(int32_t total, int32_t unit) const {
    const float guess = static_cast<float>(unit) * static_cast<float>(n) / static_cast<float>(total);
    uint32_t i = min(static_cast<uint32_t>(guess), n - 1);
    while (i > 0 && begin(i) > unit) --i;
    while (i + 1 < n && begin(i + 1) <= unit) ++i;
    return static_cast<int32_t>(i);
  }
};

// Teams among which a line is cut: of as many warps as there are rows, and none
// without a unit.
__device__ __forceinline__ uint32_t quant_teams(const QuantAttnArgs& a, int32_t total) {
  return static_cast<uint32_t>(min(max(a.warps / a.rows, 1), max(total, 1)));
}

__device__ __forceinline__ int32_t quant_length(const QuantAttnArgs& a, int64_t b) {
  const int64_t most = a.pool.max_pages << a.pool.page_log2, n = a.lens[b];
  return static_cast<int32_t>(n < 0 ? 0 : (n < most ? n : most));
}

// A place on the line.
struct Spot {
  int64_t b;
  int32_t tile, tiles, tokens;
};

// (Lengths go up to 2^31 - 16: tokens behind a tile's start do not fit then.)
template <int TILE>
__device__ __forceinline__ int32_t tiles_of(int32_t tokens) {
  return static_cast<int32_t>((static_cast<uint32_t>(tokens) + TILE - 1) / TILE);
}
template <int TILE>
__device__ __forceinline__ void enter(const QuantAttnArgs& a, Spot& s) {
  s.tokens = quant_length(a, s.b);
  s.tiles = tiles_of<TILE>(s.tokens);
}
// Units of a sequence on the line: its start and its tiles.
__device__ __forceinline__ int32_t units_of(int32_t tiles) {
  return tiles > 0 ? tiles + kQuantStart : 0;
}
// To the next tile; never called behind the last one of the line.
template <int TILE>
__device__ __forceinline__ void advance(const QuantAttnArgs& a, Spot& s) {
  if (++s.tile < s.tiles) return;
  s.tile = 0;
  do {
    ++s.b;
    enter<TILE>(a, s);
  } while (s.tiles == 0 && s.b + 1 < a.batch);
}

// ---- output ----------------------------------------------------------------

__device__ __forceinline__ uint32_t pack_pair(const QuantAttnArgs& a, float lo, float hi) {
  if (a.bf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  return half_pair(lo, hi);
}

// The first query head of a row, and how many it has.
__device__ __forceinline__ int32_t row_heads(const QuantAttnArgs& a, int32_t row, int32_t& first) {
  const int32_t kv = row / a.splits, part = row - kv * a.splits;
  first = kv * a.group + part * a.split_heads;
  return min(a.split_heads, a.group - part * a.split_heads);
}

__device__ __forceinline__ uint16_t* out_row(const QuantAttnArgs& a, int64_t b, int32_t head) {
  return static_cast<uint16_t*>(a.out) + b * a.o_sb + head * a.o_sh;
}

// A warp's joined output of a head, kDims elements in each lane, `sum` times too
// large, and its log-sum-exp relative to `top`.
template <int kDims>
__device__ __forceinline__ void write_joined(const QuantAttnArgs& a, int64_t b, int32_t head,
                                             const float (&x)[kDims], float sum, float top) {
  const int lane = threadIdx.x & 31;
  const float f = sum == 0.f ? 0.f : 1.f / sum;
  if (lane * kDims < a.pool.dim) {
    uint32_t* to = reinterpret_cast<uint32_t*>(out_row(a, b, head) + lane * kDims);
#pragma unroll
    for (int j = 0; j < kDims; j += 2)
      to[j / 2] = sum == 0.f ? 0u : pack_pair(a, x[j] * f, x[j + 1] * f);
  }
  if (lane == 0 && a.lse)
    a.lse[b * a.l_sb + head * a.l_sh] = (top == -INFINITY ? 0.f : top) + log2f(sum);
}

// ---- the kernels -----------------------------------------------------------

// KD: the dimensions that are multiplied. The first MD of them, 64 or 128, are dealt
// to the lanes in whole chunks; 80 and 96 have a tail of one or two steps of 16.
template <int DP, int NT, int KD>
struct QuantWarp {
  using L = QuantLayout<DP, NT>;
  static constexpr int kTail = KD == 80 ? 1 : KD == 96 ? 2 : 0, MD = KD - 16 * kTail;
  static_assert(MD == 64 || MD == 128, "whole chunks");
  static constexpr int kTile = L::kTile;
  static constexpr int kGroups = kTile / 16;  // of 16 keys
  static constexpr int kChunks = MD / 64;     // 16-byte chunks of a key in a lane
  static constexpr int kWords = MD / 32;      // 4-byte words of a value in a lane
  static constexpr int kSteps = KD / 16;      // of 16 dimensions
  static constexpr int kMasks = kTile / 32;
  static constexpr int kRowLanes = DP / 16;          // lanes that load a row
  static constexpr int kRows = 32 / kRowLanes;       // rows of one copy
  static constexpr int kCopies = 16 / kRows;         // of 16 keys

  // A tile whose loads are under way or its turn.
  struct Tile {
    bool some;            // there is one
    bool full;            // all keys are seen
    int32_t page[kGroups];  // of 16 keys; -1: none
    int32_t inside;       // its first token's place on its page
    uint32_t seen[kMasks];
    float sk[kMasks], sv[kMasks];  // scales, of key 32 x + lane
  };

  const QuantAttnArgs& a;
  const int lane, g, t;
  const uint32_t ring;     // this warp's shared memory
  uint32_t fill, read;     // slots of the next tile to load and to use
  // This lane copies 16 bytes of every kRows-th row; what is its place where it
  // does not (behind the head dimension) is 0 from the start.
  const bool copies;
  uint32_t copy_to[2];     // where to, in even and odd steps of kRows
  uint32_t key_from[2];    // where this lane's chunks of keys are, on even and odd rows
  uint32_t value_from[2];  // its parts of values
  uint32_t key_tail, value_tail[2];  // the same of the tail

  Spot due;       // the tile whose keys are loaded next
  int32_t left;   // tiles from it to the share's end
  int32_t page[kGroups];
  int32_t row;    // this warp's
  const uint8_t *keys, *values;  // what this lane copies of it, on page 0
  const float *k_scales, *v_scales;
  Tile now, next;

  uint32_t qf[NT][kSteps][2];
  float2 q_power[NT];  // of the columns' heads
  float o[NT][KD / 16][4];
  float2 l[NT], m[NT], big[NT];  // sums; bases of the sums and of the weights

  // Rows of 128 bytes, or pairs of rows of 64, are swizzled by 16-byte chunks: the
  // eight lanes that read together (two keys of four chunks, or two chunks of
  // values that lie two rows apart) find theirs on different banks.
  static __device__ __forceinline__ uint32_t place(int row, int chunk) {
    if constexpr (DP == 128)
      return row * 128 + ((chunk ^ (row & 6) ^ ((row & 1) << 2)) << 4);
    return (row >> 1) * 128 + (((((row & 1) << 2) | chunk) ^ (row & 6)) << 4);
  }

  __device__ __forceinline__ QuantWarp(const QuantAttnArgs& args, uint32_t smem)
      : a(args),
        lane(threadIdx.x & 31),
        g(lane >> 2),
        t(lane & 3),
        ring(smem),
        fill(smem),
        read(smem),
        copies(lane % kRowLanes * 16 < args.pool.dim) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      copy_to[i] = place(lane / kRowLanes + i * kRows, lane % kRowLanes) - i * kRows * DP;
      key_from[i] = place(g, MD == 128 ? 4 * i + t : t);
      value_from[i] = place(2 * t + i, MD == 128 ? g : g >> 1) + (MD == 128 ? 0 : (g & 1) * 8);
      if constexpr (kTail > 0)
        value_tail[i] = place(2 * t + i, 4 + 2 * kTail * g / 16) + 2 * kTail * g % 16;
    }
    if constexpr (kTail > 0) key_tail = place(g, 4 + 4 * kTail * t / 16) + 4 * kTail * t % 16;
    if (!copies)
#pragma unroll 1
      for (uint32_t i = 0; i < 3 * kTile / kRows; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                         ring + (i & 1 ? copy_to[1] : copy_to[0]) + i * kRows * DP),
                     "r"(0)
                     : "memory");
  }

  __device__ __forceinline__ void step(uint32_t& slot) {
    slot += kQuantTileBytes;
    if (slot == ring + 3 * kQuantTileBytes) slot = ring;
  }

  __device__ __forceinline__ void take_row(int32_t r) {
    row = r;
    const int32_t head = r / a.splits;
    const int from = lane / kRowLanes, byte = lane % kRowLanes * 16;
    keys = a.pool.codes[0] + head * a.pool.sh[0] + from * a.pool.st[0] + byte;
    values = a.pool.codes[1] + head * a.pool.sh[1] + from * a.pool.st[1] + byte;
    k_scales = a.pool.scales[0] + head;
    v_scales = a.pool.scales[1] + head;
  }
  __device__ __forceinline__ bool one_page() const { return (1 << a.pool.page_log2) >= kTile; }
  __device__ __forceinline__ void look_up() {
    if (left <= 0) return;
    const int32_t t0 = due.tile * kTile, rest = due.tokens - t0;
    page[0] = quant_page(a.pool, due.b, t0);
#pragma unroll
    for (int i = 1; i < kGroups; ++i)
      page[i] = one_page() ? page[0]
                           : 16 * i < rest ? quant_page(a.pool, due.b, t0 + 16 * i) : -1;
  }

  // The rows of a tile into the next slot; `from`: what this lane copies, on page 0.
  __device__ __forceinline__ void copy_rows(const Tile& x, const uint8_t* from, int kv) {
    const int64_t sn = a.pool.sn[kv], st = a.pool.st[kv];
    const int32_t mask = (1 << a.pool.page_log2) - 1;
    const uint32_t to[2] = {fill + copy_to[0], fill + copy_to[1]};
    if (copies) {
      const uint8_t* p = from + x.page[0] * sn + x.inside * st;
      if (x.full) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          if (i > 0 && !one_page())
            p = from + x.page[i] * sn + ((x.inside + 16 * i) & mask) * st;
#pragma unroll
          for (int j = 0; j < kCopies; ++j) {
            copy16(to[j & 1] + (16 * i + j * kRows) * DP, p);
            p += kRows * st;
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
          p = from + x.page[i] * sn + ((x.inside + 16 * i) & mask) * st;
#pragma unroll
          for (int j = 0; j < kCopies; ++j) {
            const int at = 16 * i + j * kRows + lane / kRowLanes;
            const bool yes = x.seen[i / 2] >> (at & 31) & 1;
            copy16(to[j & 1] + (16 * i + j * kRows) * DP, yes ? p : a.pool.codes[kv], yes);
            p += kRows * st;
          }
        }
      }
    }
    step(fill);
  }

  // Keys and scales of the due tile, which becomes `next`; the one behind it is
  // due then.
  __device__ __forceinline__ void load_keys() {
    next.some = left > 0;
    if (next.some) {
      const int32_t t0 = due.tile * kTile, mask = (1 << a.pool.page_log2) - 1;
      next.inside = t0 & mask;
      const int32_t rest = due.tokens - t0;
      bool full = rest >= kTile;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        next.page[i] = page[i];
        full &= page[i] >= 0;
      }
      next.full = full;
#pragma unroll
      for (int x = 0; x < kMasks; ++x) {
        const int32_t mine = lane < 16 ? page[2 * x] : page[2 * x + 1];
        const bool ok = mine >= 0 && 32 * x + lane < rest;
        next.seen[x] = full ? ~0u : __ballot_sync(~0u, ok);
        const int64_t in =
            static_cast<int64_t>(((next.inside + 32 * x + lane) & mask) >> a.pool.block_log2) *
            a.pool.kv_heads;
        next.sk[x] = next.sv[x] = 0.f;
        if (ok) {
          next.sk[x] = k_scales[mine * a.pool.ssn[0] + in];
          next.sv[x] = v_scales[mine * a.pool.ssn[1] + in];
        }
      }
      copy_rows(next, keys, 0);
      if (--left > 0) {
        advance<kTile>(a, due);
        if (due.tile == 0) {
          fetch_queries();
          left -= kQuantStart;
        }
      }
      look_up();
    }
    copies_commit();
  }
  __device__ __forceinline__ void load_values() {
    if (next.some) copy_rows(next, values, 1);
    copies_commit();
  }

  // Brings the queries of the due sequence nearer, which begins in two tiles.
  __device__ __forceinline__ void fetch_queries() {
    int32_t first;
    const int32_t heads = row_heads(a, row, first);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + g;
      if (h < heads && 32 * t < a.pool.dim)
        asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const uint16_t*>(a.q) +
                                                      due.b * a.q_sb + (first + h) * a.q_sh +
                                                      32 * t));
    }
  }

  // The queries of a sequence as the products' right-hand side: column g is a head,
  // and this lane has the dimensions that it has of a key. Each head is
  // multiplied by a power of two that brings its largest element to 2^14, which
  // fp16 then holds exactly to 2^-38 of it.
  __device__ __forceinline__ float2 unpack_pair(uint32_t w) const {
    if (a.bf16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  __device__ __forceinline__ void begin(int64_t b) {
    int32_t first;
    const int32_t heads = row_heads(a, row, first);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int h = 8 * n + g;
      const uint16_t* from =
          static_cast<const uint16_t*>(a.q) + b * a.q_sb + (first + h) * a.q_sh;
      float2 x[2 * kSteps];
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int d = 64 * j + 16 * t;
        uint4 u[2] = {};
        if (h < heads && d < a.pool.dim) {
          u[0] = reinterpret_cast<const uint4*>(from + d)[0];
          u[1] = reinterpret_cast<const uint4*>(from + d)[1];
        }
        const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[8 * j + i] = unpack_pair(w[i]);
      }
      if constexpr (kTail > 0) {
        uint2 u[kTail] = {};
#pragma unroll
        for (int i = 0; i < kTail; ++i) {
          if (h < heads)
            u[i] = *reinterpret_cast<const uint2*>(from + MD + 4 * (kTail * t + i));
          x[8 * kChunks + 2 * i] = unpack_pair(u[i].x);
          x[8 * kChunks + 2 * i + 1] = unpack_pair(u[i].y);
        }
      }
#pragma unroll
      for (int i = 0; i < 2 * kSteps; ++i)
        top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
      top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
      // the power's exponent: what brings `top` to [2^14, 2^15), from 2^-126 on
      // (bf16's smallest number is 2^-133: 2^-7 then)
      int e = static_cast<int>(__float_as_uint(top) >> 23) - 127 - 14;
      e = max(e, -126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int r = 0; r < kSteps; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          qf[n][r][i] = half_pair(x[2 * r + i].x * down, x[2 * r + i].y * down);
      q_power[n].x = __shfl_sync(~0u, up, 8 * t);
      q_power[n].y = __shfl_sync(~0u, up, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < KD / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[n][i][j] = 0.f;
      l[n] = make_float2(0.f, 0.f);
      m[n] = big[n] = make_float2(-FLT_MAX, -FLT_MAX);
    }
  }

  // One tile. Weights with their values' scales, 2^(x + log2 sv), are kept
  // relative to a base of their own, as 2^7 at most 2^8 times over: the largest
  // is then from 2^7 to 2^15 of fp16's range, and what is lost lies 2^-32 below
  // it. The sums of 2^x have another base. Both move rarely.
  // Products take a weight as two fp16 numbers, the nearest one and what is left,
  // so that it is held to 2^-22 of itself. With the nearest one alone (2^-11) fp16
  // outputs were 13 % further from exact ones than rounding makes them (33 sequences,
  // 8 heads of 80: 2.37e-4 instead of 2.09e-4 of their norm), and those of values
  // that cancel lost all they had. The second product costs 0.4 us of 100 (302,000
  // tokens of 8 heads of 128), 1.5 of 48 (136,000 of 80) and, with 16 columns, 6 of
  // 62 (64 sequences of up to 4000 tokens, 128 heads on 8 of 128).
  __device__ __forceinline__ void tile(bool work) {
    float s[kGroups][NT][4];
    if (work) scores(s);
    load_values();
    if (work) outputs(s);
    now = next;
    load_keys();
  }

  // The products of queries and keys.
  __device__ __forceinline__ void scores(float (&s)[kGroups][NT][4]) {
    copies_wait<2>();
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kGroups; ++x)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[x][n][j] = 0.f;
#pragma unroll
    for (int j = 0; j < kChunks; ++j) score_steps<4>(s, key_from[j], 4 * j);
    if constexpr (kTail > 0) score_steps<kTail>(s, key_tail, 4 * kChunks);
    step(read);
    __syncwarp();  // the slot has been read
  }

  // STEPS of them, from step `r0` on, whose codes are at `from` of a tile.
  template <int STEPS>
  __device__ __forceinline__ void score_steps(float (&s)[kGroups][NT][4], uint32_t from, int r0) {
    uint32_t k[kGroups][2][STEPS];
#pragma unroll
    for (int x = 0; x < kGroups; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) shared_words(k[x][y], read + from + (16 * x + 8 * y) * DP);
#pragma unroll
    for (int r = 0; r < STEPS; ++r)
#pragma unroll
      for (int x = 0; x < kGroups; ++x) {
        uint32_t a0, a1, a2, a3;
        decode4(k[x][0][r], a0, a2);
        decode4(k[x][1][r], a1, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          product(s[x][n], a0, a1, a2, a3, qf[n][r0 + r][0], qf[n][r0 + r][1]);
      }
  }

  // Weights, sums and the products with values.
  __device__ __forceinline__ void outputs(float (&s)[kGroups][NT][4]) {
    float ck[kMasks], lv[kMasks];
#pragma unroll
    for (int x = 0; x < kMasks; ++x) {
      ck[x] = a.c * now.sk[x];
      lv[x] = __log2f(now.sv[x]);
    }
    // scores, and with the values' scales
    float2 w[kGroups][2][NT];
    float2 top[NT], wide[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) top[n] = wide[n] = make_float2(-INFINITY, -INFINITY);
#pragma unroll
    for (int x = 0; x < kGroups; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int from = (16 * x + 8 * y + g) & 31;
        const float fk = __shfl_sync(~0u, ck[x / 2], from);
        const float fv = __shfl_sync(~0u, lv[x / 2], from);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float2 z = mul2(make_float2(s[x][n][2 * y], s[x][n][2 * y + 1]),
                          mul2(q_power[n], make_float2(fk, fk)));
          if (!now.full && !(now.seen[x / 2] >> from & 1)) z = make_float2(-INFINITY, -INFINITY);
          s[x][n][2 * y] = z.x;
          s[x][n][2 * y + 1] = z.y;
          const float2 v = add2(z, make_float2(fv, fv));
          w[x][y][n] = v;
          top[n] = make_float2(fmaxf(top[n].x, z.x), fmaxf(top[n].y, z.y));
          wide[n] = make_float2(fmaxf(wide[n].x, v.x), fmaxf(wide[n].y, v.y));
        }
      }
    bool move = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
      move |= top[n].x > m[n].x + 64.f || top[n].y > m[n].y + 64.f ||
              wide[n].x > big[n].x + 8.f || wide[n].y > big[n].y + 8.f;
    if (__any_sync(~0u, move)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float2 m0 = m[n], big0 = big[n];
        m[n] = make_float2(column_max(top[n].x, m0.x), column_max(top[n].y, m0.y));
        big[n] = make_float2(column_max(wide[n].x, big0.x), column_max(wide[n].y, big0.y));
        l[n].x *= ex2(m0.x - m[n].x);
        l[n].y *= ex2(m0.y - m[n].y);
        const float fx = ex2(big0.x - big[n].x), fy = ex2(big0.y - big[n].y);
#pragma unroll
        for (int i = 0; i < KD / 16; ++i) {
          o[n][i][0] *= fx;
          o[n][i][1] *= fy;
          o[n][i][2] *= fx;
          o[n][i][3] *= fy;
        }
      }
    }
    uint32_t p[kGroups][NT][2], rest[kGroups][NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float2 m0 = make_float2(-m[n].x, -m[n].y);
      const float2 b0 = make_float2(7.f - big[n].x, 7.f - big[n].y);
#pragma unroll
      for (int x = 0; x < kGroups; ++x)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float2 z = add2(make_float2(s[x][n][2 * y], s[x][n][2 * y + 1]), m0);
          const float2 v = add2(w[x][y][n], b0);
          l[n] = add2(l[n], make_float2(ex2(z.x), ex2(z.y)));
          const float2 e = make_float2(ex2(v.x), ex2(v.y));
          const uint32_t near = half_pair(e.x, e.y);
          const float2 have = __half22float2(*reinterpret_cast<const __half2*>(&near));
          p[x][n][y] = transposed(near);
          rest[x][n][y] = transposed(half_pair(e.x - have.x, e.y - have.y));
        }
    }
    copies_wait<2>();
    __syncwarp();
#pragma unroll
    for (int x = 0; x < kGroups; ++x) {
      uint32_t v[4][kWords];
#pragma unroll
      for (int y = 0; y < 4; ++y)
        shared_words(v[y], read + value_from[y & 1] + (16 * x + 8 * (y >> 1)) * DP);
      const auto steps = [&](uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, int i, int to) {
        // codes of neighbouring keys side by side, of two dimensions
        uint32_t a0, a1, a2, a3;
        decode4(__byte_perm(v0, v1, i ? 0x7362 : 0x5140), a0, a1);
        decode4(__byte_perm(v2, v3, i ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          product(o[n][to], a0, a1, a2, a3, p[x][n][0], p[x][n][1]);
          product(o[n][to], a0, a1, a2, a3, rest[x][n][0], rest[x][n][1]);
        }
      };
#pragma unroll
      for (int r = 0; r < kWords; ++r)
#pragma unroll
        for (int i = 0; i < 2; ++i) steps(v[0][r], v[1][r], v[2][r], v[3][r], i, 2 * r + i);
      if constexpr (kTail > 0) {
        uint32_t z[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint32_t at = read + value_tail[y & 1] + (16 * x + 8 * (y >> 1)) * DP;
          if constexpr (kTail == 1) {
            z[y] = shared_half_word(at);
          } else {
            uint32_t word[1];
            shared_words(word, at);
            z[y] = word[0];
          }
        }
#pragma unroll
        for (int i = 0; i < kTail; ++i) steps(z[0], z[1], z[2], z[3], i, 2 * kWords + i);
      }
    }
    step(read);
    __syncwarp();
  }

  // The largest of a column, and of `x`.
  __device__ __forceinline__ float column_max(float v, float x) {
#pragma unroll
    for (int i = 4; i < 32; i <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, i));
    return fmaxf(v, x);
  }

  // The outputs of what this warp has of a sequence, and its log-sum-exps, in
  // place: o and m.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float sum = h ? l[n].y : l[n].x;
        float& base = h ? m[n].y : m[n].x;
        const float weights = h ? big[n].y : big[n].x;
#pragma unroll
        for (int i = 4; i < 32; i <<= 1) sum += __shfl_xor_sync(~0u, sum, i);
        const bool none = sum == 0.f;
        // 2^(weights - base) is near the values' scales, and subnormal with a sum of
        // many tokens below it where these are near 2^-126: half of it at a time
        const float half = exp2f(0.5f * (weights - 7.f - base)), f = half / sum;
#pragma unroll
        for (int i = 0; i < KD / 16; ++i) {
          o[n][i][h] = none ? 0.f : o[n][i][h] * f * half;
          o[n][i][2 + h] = none ? 0.f : o[n][i][2 + h] * f * half;
        }
        base = none ? -INFINITY : base + log2f(sum);
      }
  }

  __device__ __forceinline__ void store(int64_t b) {
    constexpr int kDims = MD / 8;  // of a lane
    int32_t first;
    const int32_t heads = row_heads(a, row, first);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t at = 8 * n + 2 * t + h;
        if (at >= heads) continue;
        if (g * kDims < a.pool.dim) {
          uint4* to = reinterpret_cast<uint4*>(out_row(a, b, first + at) + g * kDims);
#pragma unroll
          for (int i = 0; i < MD / 64; ++i) {
            uint32_t u[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              u[j] = pack_pair(a, o[n][4 * i + j][h], o[n][4 * i + j][2 + h]);
            to[i] = make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
        if constexpr (kTail > 0) {
          uint32_t* to =
              reinterpret_cast<uint32_t*>(out_row(a, b, first + at) + MD + 2 * kTail * g);
#pragma unroll
          for (int i = 0; i < kTail; ++i)
            to[i] = pack_pair(a, o[n][MD / 16 + i][h], o[n][MD / 16 + i][2 + h]);
        }
        if (g == 0 && a.lse) a.lse[b * a.l_sb + (first + at) * a.l_sh] = h ? m[n].y : m[n].x;
      }
  }

  // To a piece [columns][DP], the first KD of each, and its log-sum-exps.
  __device__ __forceinline__ void keep(float* piece, float* lse) {
    int32_t first;
    const int32_t heads = row_heads(a, row, first);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int32_t at = 8 * n + 2 * t + h;
        if (at >= heads) continue;
        float4* to = reinterpret_cast<float4*>(piece + at * DP + g * (MD / 8));
#pragma unroll
        for (int i = 0; i < MD / 32; ++i)
          to[i] = make_float4(o[n][2 * i][h], o[n][2 * i][2 + h], o[n][2 * i + 1][h],
                              o[n][2 * i + 1][2 + h]);
        if constexpr (kTail > 0) {
          float2* tail = reinterpret_cast<float2*>(piece + at * DP + MD + 2 * kTail * g);
#pragma unroll
          for (int i = 0; i < kTail; ++i)
            tail[i] = make_float2(o[n][MD / 16 + i][h], o[n][MD / 16 + i][2 + h]);
        }
        if (g == 0) lse[at] = h ? m[n].y : m[n].x;
      }
  }

  // `units` of the line, from the tile of `spot` on. What it has of a sequence in part
  // goes to `piece(b, whether the sequence begins here)` instead of the output.
  template <typename F>
  __device__ __forceinline__ void run(Spot spot, int32_t units, F piece) {
    due = spot;
    left = units;
    look_up();
    next.some = false;
    bool began = spot.tile == 0, fresh = true;
    // two rounds ahead of the first tile only load
    for (int32_t i = -2; units > 0; ++i) {
      if (i >= 0 && fresh) begin(spot.b);
      tile(i >= 0);
      if (i < 0) continue;
      fresh = false;
      --units;
      const bool ends = spot.tile + 1 == spot.tiles;
      if (!ends && units > 0) {
        ++spot.tile;
        continue;
      }
      if (ends) units -= kQuantStart;
      finish();
      if (began && ends)
        store(spot.b);
      else
        piece(began);
      if (units > 0) {
        advance<kTile>(a, spot);
        began = fresh = true;
      }
    }
  }
};

// Where `unit` of the line lies (in a sequence's start: a tile below 0); all lanes of
// a warp together. sums[i]: units in front of chunk i (of `chunk` sequences each).
template <int TILE, int THREADS>
__device__ __forceinline__ Spot find_spot(const QuantAttnArgs& a, int32_t unit,
                                          const int32_t* sums, int64_t chunk) {
  const int lane = threadIdx.x & 31;
  int below = 0;
#pragma unroll
  for (int i = 0; i < THREADS; i += 32) below += sums[i + lane] <= unit;
  below = __reduce_add_sync(~0u, below) - 1;  // the last chunk that begins at or before it
  int32_t before = sums[below];
  for (int64_t b0 = below * chunk;; b0 += 32) {
    Spot s;
    s.b = b0 + lane;
    s.tiles = s.tokens = 0;
    if (s.b < a.batch) enter<TILE>(a, s);
    const int32_t units = units_of(s.tiles);
    int32_t upto = units;
#pragma unroll
    for (int i = 1; i < 32; i <<= 1) {
      const int32_t y = __shfl_up_sync(~0u, upto, i);
      if (lane >= i) upto += y;
    }
    const uint32_t past = __ballot_sync(~0u, before + upto > unit);
    if (past) {
      const int who = __ffs(past) - 1;
      s.tile = __shfl_sync(~0u, unit - (before + upto - units), who) - kQuantStart;
      s.b = b0 + who;
      s.tiles = __shfl_sync(~0u, s.tiles, who);
      s.tokens = __shfl_sync(~0u, s.tokens, who);
      return s;
    }
    before += __shfl_sync(~0u, upto, 31);
  }
}

template <int DP, int NT, int KD>
__global__ void __launch_bounds__(QuantLayout<DP, NT>::kThreads, 1)
    quant_attend_kernel(const QuantAttnArgs a) {
  using L = QuantLayout<DP, NT>;
  constexpr int W = L::kWarps;
  // A ring for each warp. Rows of 128 bytes have to begin at multiples of 128 (with
  // others, copies took twice the sectors).
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int32_t sums[L::kThreads];
  __shared__ int32_t part[W];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  launch_followers();
  const int64_t chunk = (a.batch + L::kThreads - 1) / L::kThreads;
  const int64_t b0 = threadIdx.x * chunk, b1 = min(b0 + chunk, a.batch);
  int32_t mine = 0;
  for (int64_t b = b0; b < b1; ++b) mine += units_of(tiles_of<L::kTile>(quant_length(a, b)));
  int32_t upto = mine;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int32_t y = __shfl_up_sync(~0u, upto, i);
    if (lane >= i) upto += y;
  }
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  int32_t before = upto - mine, total = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < warp) before += part[i];
    total += part[i];
  }
  sums[threadIdx.x] = before;
  __syncthreads();
  // Neighbouring warps of a team are on different SMs, so that short lines use
  // many. With more rows than warps each goes through several.
  const int32_t self = warp * gridDim.x + blockIdx.x;
  const Shares shares(total, quant_teams(a, total));
  if (threadIdx.x % gridDim.x == blockIdx.x) {  // this CTA's part of the spans
    int32_t at = before;
    for (int64_t b = b0; b < b1; ++b) {
      const int32_t tiles = tiles_of<L::kTile>(quant_length(a, b));
      const int32_t from = at + kQuantStart;
      a.spans[b] = tiles > 0 ? make_int2(shares.of(total, from), shares.of(total, from + tiles - 1))
                             : make_int2(0, -1);
      at += units_of(tiles);
    }
  }
  const uint32_t team = self / a.rows;
  if (total == 0 || team >= shares.n) return;
  const int32_t first = shares.begin(team);
  int32_t units = shares.begin(team + 1) - first;
  Spot spot = find_spot<L::kTile, L::kThreads>(a, first, sums, chunk);
  if (spot.tile < 0) {  // it begins with a start
    units += spot.tile;
    spot.tile = 0;
  }
  if (units <= 0) return;
  QuantWarp<DP, NT, KD> w(a, smem_addr(smem) + warp * L::kRing);
  for (int32_t row = self - team * a.rows; row < a.rows; row += a.warps) {
    w.take_row(row);
    w.run(spot, units, [&](bool began) {
      const int64_t slot = 2ll * self + began;
      w.keep(a.part_o + slot * L::kPiece, a.part_lse + slot * L::kHeads);
    });
  }
}

// A CTA for each row of few tiles, whose warps share them: nothing is left to be
// joined by a second launch.
template <int DP, int NT, int KD>
__global__ void __launch_bounds__(QuantLayout<DP, NT>::kThreads, 1)
    quant_attend_row_kernel(const QuantAttnArgs a) {
  using L = QuantLayout<DP, NT>;
  constexpr int W = L::kWarps, kDims = DP / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float piece_lse[W][L::kHeads];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Spot spot{};
  spot.b = blockIdx.x / a.rows;
  const int32_t row = static_cast<int32_t>(blockIdx.x - spot.b * a.rows);
  enter<L::kTile>(a, spot);
  int32_t first;
  const int32_t heads = row_heads(a, row, first);
  const uint32_t used = min(spot.tiles, W);
  if (warp < used) {
    const Shares shares(spot.tiles, used);
    spot.tile = shares.begin(warp);
    QuantWarp<DP, NT, KD> w(a, smem_addr(smem) + warp * L::kRing);
    w.take_row(row);
    w.run(spot, shares.begin(warp + 1) - spot.tile, [&](bool) {
      __syncwarp();  // the ring has been read
      w.keep(reinterpret_cast<float*>(smem + warp * L::kRing), piece_lse[warp]);
    });
    if (used == 1) return;  // has stored them
  }
  if (used == 1) return;
  __syncthreads();
  for (int h = warp; h < heads; h += W) {
    float top = -INFINITY, sum = 0.f, x[kDims] = {};
    for (int i = 0; i < used; ++i) top = fmaxf(top, piece_lse[i][h]);
    const float base = top == -INFINITY ? 0.f : top;
    for (int i = 0; i < used; ++i) {
      const float f = ex2(piece_lse[i][h] - base);
      const float* y = reinterpret_cast<const float*>(smem + i * L::kRing) + h * DP + lane * kDims;
      sum += f;
#pragma unroll
      for (int j = 0; j < kDims; ++j) x[j] += f * y[j];
    }
    write_joined<kDims>(a, spot.b, first + h, x, sum, top);
  }
}

// Joins what the first launch left of sequences that lie in several shares, and
// writes those without tiles: TEAM warps for each query head. Loads of pieces do
// not wait for one another.
template <int TEAM>
struct JoinShape {
  static constexpr int kWarps = TEAM < 8 ? 8 : TEAM, kThreads = 32 * kWarps;
};
template <int DP, int NT, int TEAM>
__global__ void __launch_bounds__(JoinShape<TEAM>::kThreads) quant_join_kernel(const QuantAttnArgs a) {
  constexpr int kHeads = 8 * NT, kDims = DP / 32, kAtOnce = 8, kWarps = JoinShape<TEAM>::kWarps;
  __shared__ float shared_o[TEAM][DP];
  __shared__ float shared_top[TEAM], shared_sum[TEAM];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mate = warp % TEAM;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (kWarps / TEAM) + warp / TEAM;
  const int32_t all = a.pool.kv_heads * a.group;
  const int64_t b = item / all;
  const int32_t head = static_cast<int32_t>(item - b * all);
  const int32_t kv = head / a.group, in = head - kv * a.group;
  const int32_t row = kv * a.splits + in / a.split_heads, h = in % a.split_heads;
  follow();
  if (b >= a.batch) return;  // (only where a team is a warp)
  const int2 span = a.spans[b];
  const int32_t s0 = span.x, s1 = span.y;
  if (s0 == s1) return;
  float top = -INFINITY, sum = 0.f, x[kDims] = {};
  for (int32_t s = s0 + mate; s <= s1; s += TEAM * kAtOnce) {
    float lse[kAtOnce], y[kAtOnce][kDims];
    float most = top;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      lse[i] = -INFINITY;
#pragma unroll
      for (int j = 0; j < kDims; ++j) y[i][j] = 0.f;
      const int32_t at = s + i * TEAM;
      if (at <= s1) {
        // the first one's piece is where the sequence begins
        const int64_t slot = (2ll * (at * a.rows + row) + (at == s0)) * kHeads + h;
        lse[i] = a.part_lse[slot];
        const float* from = a.part_o + slot * DP + lane * kDims;
#pragma unroll
        for (int j = 0; j < kDims; ++j) y[i][j] = from[j];
      }
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) most = fmaxf(most, lse[i]);
    const float base = most == -INFINITY ? 0.f : most, keep = ex2(top - base);
    sum *= keep;
#pragma unroll
    for (int j = 0; j < kDims; ++j) x[j] *= keep;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float f = ex2(lse[i] - base);
      sum += f;
#pragma unroll
      for (int j = 0; j < kDims; ++j) x[j] += f * y[i][j];
    }
    top = most;
  }
  if constexpr (TEAM > 1) {
#pragma unroll
    for (int j = 0; j < kDims; ++j) shared_o[mate][lane * kDims + j] = x[j];
    if (lane == 0) {
      shared_top[mate] = top;
      shared_sum[mate] = sum;
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) top = fmaxf(top, shared_top[i]);
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < kDims; ++j) x[j] = 0.f;
#pragma unroll
    for (int i = 0; i < TEAM; ++i) {
      const float f = ex2(shared_top[i] - (top == -INFINITY ? 0.f : top));
      sum += f * shared_sum[i];
#pragma unroll
      for (int j = 0; j < kDims; ++j) x[j] += f * shared_o[i][lane * kDims + j];
    }
  }
  write_joined<kDims>(a, b, head, x, sum, top);
}

}  // namespace dsa
