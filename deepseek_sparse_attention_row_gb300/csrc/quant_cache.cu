// quant_cache.cu -- writing keys and values into pages of e4m3 codes and
// reading them back: dsa_quant_cache_write and dsa_quant_cache_read of
// include/dsa_quant.h.
//
// Scales are powers of two: x / scale then is exact in fp32, so that a code is the
// one next to x and does not depend on how it is computed, and a scale that grows
// changes the held codes only where they fall below the smallest normal one.
//
// Reading is bound by HBM: 20541 tokens of 8 heads of 128, 126 MB, take 22.8 us (5.5
// TB/s; 25 us with eight rows to a warp). Writing is bound by how many loads are under
// way: it reads a block's tokens once, into the registers of a team of warps that agree
// on their largest size, and a CTA has none under way while it agrees and stores. 16389
// tokens of 8 heads of 128, 101 MB, take 22.2 us (4.5 TB/s); 72 us when a warp went
// through the block twice, 30 with sizes taken as floats, 27 with registers for two
// CTAs of an SM instead of four. Small blocks have a CTA each: 16000 tokens take 21.7 us
// in blocks of 128, 21.2 of 16, 46 of 4 and 161 of 1.
#include <cuda_runtime.h>

#include <cmath>

#include "quant.cuh"

namespace dsa {
namespace {

struct WriteArgs {
  QuantPool pool;
  const void* x[2];
  int64_t xt[2], xh[2];  // elements
  int64_t total;
  const int32_t* cu;
  int32_t seqs;
  const int32_t* lens;
};

__device__ __forceinline__ int64_t clamped(int32_t x, int64_t most) {
  return x < 0 ? 0 : (x < most ? x : most);
}

// The last of the first n of nondecreasing marks that is not above `x` (0 if all
// are), by a warp: each step reads 32 of them at once.
template <typename F>
__device__ __forceinline__ int32_t last_upto(int32_t n, int64_t x, F mark) {
  const int lane = threadIdx.x & 31;
  int32_t lo = 0;  // what is sought is in [lo, lo + n)
  while (n > 1) {
    const int32_t step = (n + 31) / 32, at = lane * step;
    const uint32_t upto = __ballot_sync(~0u, at < n && mark(lo + at) <= x);
    // marks may decrease against the rules: the first ones that hold count
    const int32_t held = max(__ffs(~upto) - 2, upto == ~0u ? 31 : 0);
    lo += held * step;
    n = min(step, n - held * step);
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ float2 pair(uint32_t two);
template <>
__device__ __forceinline__ float2 pair<__nv_bfloat16>(uint32_t two) {
  return make_float2(__uint_as_float(two << 16), __uint_as_float(two & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 pair<__half>(uint32_t two) {
  return __half22float2(*reinterpret_cast<const __half2*>(&two));
}

// Sizes of 16-bit numbers are ordered as integers; from this one on they are not
// finite. (Both halves alike.)
template <typename T>
constexpr uint32_t kInfinite = 0x7f80u;
template <>
constexpr uint32_t kInfinite<__half> = 0x7c00u;

__device__ __forceinline__ float nan_for_infinite(float x) {
  return fabsf(x) < INFINITY ? x : NAN;
}
// The larger of the two halves of each word.
__device__ __forceinline__ uint32_t largest2(uint32_t x, uint32_t sizes) {
  return __vmaxu2(x, sizes & 0x7fff7fffu);
}
// The same, of finite numbers.
template <typename T>
__device__ __forceinline__ uint32_t largest_finite2(uint32_t x, uint32_t sizes) {
  sizes &= 0x7fff7fffu;
  if ((sizes & 0xffffu) >= kInfinite<T>) sizes &= 0xffff0000u;
  if ((sizes >> 16) >= kInfinite<T>) sizes &= 0xffffu;
  return __vmaxu2(x, sizes);
}

// A block of a sequence that gets new tokens. Sequence s of n tokens touches at
// most n / block + 2 blocks, and floor(cu[s] / block) + 2 s counts that many
// between one sequence and the next: item numbers are found from cu alone.
struct Block {
  int32_t seq;       // -1: nothing to do
  int32_t start;     // its first token
  int32_t from, to;  // the new ones
  int64_t row;       // of the token `from`
};

__device__ __forceinline__ Block find_block(const WriteArgs& a, int64_t item) {
  const int lg = a.pool.block_log2;
  Block b{};
  b.seq = -1;
  const int32_t s = last_upto(a.seqs, item, [&](int32_t i) {
    return (clamped(a.cu[i], a.total) >> lg) + 2ll * i;
  });
  const int64_t r0 = clamped(a.cu[s], a.total), r1 = clamped(a.cu[s + 1], a.total);
  const int64_t held = a.lens[s] > 0 ? a.lens[s] : 0, end = held + (r1 - r0);
  const int64_t most = a.pool.max_pages << a.pool.page_log2;
  const int64_t at = item - (r0 >> lg) - 2ll * s;  // below 0: rows in front of the first sequence
  const int64_t start = ((held >> lg) + at) << lg;
  if (at < 0 || r1 <= r0 || start >= end || start >= most) return b;
  b.seq = s;
  b.start = static_cast<int32_t>(start);
  b.from = static_cast<int32_t>(held > start ? held : start);
  b.to = static_cast<int32_t>(end < start + (1ll << lg) ? end : start + (1ll << lg));
  b.row = r0 + b.from - held;
  return b;
}

constexpr int kWriteWarps = 8;
constexpr int kAtOnce = 8;  // 16-byte loads of a lane

// A team of `team` warps (a power of two, up to 16) for each block, head and one of
// keys and values; the teams of a CTA share the block. Where a block's new tokens
// are no more than a team has registers for, they are read once. The team is laid out
// for the mean of the sequences: a prompt of 2048 tokens, alone 4.6 us, takes 24.4 among
// 255 single tokens (alone 7.5), as its blocks' warps go through them twice.
// (64 registers, none spilled, for twice the warps.)
template <typename T>
__global__ void __launch_bounds__(512, 2) write_kernel(const WriteArgs a, int team) {
  __shared__ uint32_t tops[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const Block b = find_block(a, blockIdx.x);
  if (b.seq < 0) return;
  const int32_t page = quant_page(a.pool, b.seq, b.start);  // not waited for yet
  const int parts = a.pool.dim / 8, rows = 32 / parts;      // 8 elements of a lane
  const int row = lane / parts, part = lane - row * parts;
  const int mate = warp & (team - 1), each = warps / team;  // teams of a CTA
  const int step = team * rows;                             // rows of a team at a time
  const int from = row < rows ? mate * rows + row : 1 << 20;  // idle lanes: behind every row
  const int count = b.to - b.from;
  // This team's work number w: keys or values of a head.
  const auto source = [&](int w) {
    const int kv = w & 1;
    return static_cast<const char*>(a.x[kv]) +
           (b.row * a.xt[kv] + (w >> 1) * a.xh[kv]) * static_cast<int64_t>(sizeof(T)) + part * 16;
  };
  const auto load = [&](uint4 (&u)[kAtOnce], int w, int i0) {
    const char* x = source(w);
    const int64_t x_step = a.xt[w & 1] * static_cast<int64_t>(sizeof(T));
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int at = i0 + from + i * step;
      u[i] = make_uint4(0, 0, 0, 0);
      if (at < count) u[i] = *reinterpret_cast<const uint4*>(x + at * x_step);
    }
  };
  // The largest finite size of them and of `x` (two halves); `special`: this warp
  // has some that are not finite.
  const auto largest = [&](const uint4 (&u)[kAtOnce], uint32_t x, bool& special) {
    uint32_t y = x;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      for (uint32_t two : {u[i].x, u[i].y, u[i].z, u[i].w}) y = largest2(y, two);
    if (!__any_sync(~0u, max(y & 0xffffu, y >> 16) >= kInfinite<T>)) return y;
    special = true;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      for (uint32_t two : {u[i].x, u[i].y, u[i].z, u[i].w}) x = largest_finite2<T>(x, two);
    return x;
  };
  const int works = 2 * a.pool.kv_heads;
  const bool once = count <= kAtOnce * step;
  for (int w0 = blockIdx.y * each; w0 < works; w0 += gridDim.y * each) {
    const int w = w0 + warp / team;
    const bool mine = w < works;
    const int kv = w & 1, head = mine ? w >> 1 : 0;
    uint4 u[kAtOnce];
    uint32_t sizes = 0;
    bool special = false;
    if (mine)
      for (int i0 = 0; i0 < count; i0 += kAtOnce * step) {
        load(u, w, i0);
        sizes = largest(u, sizes, special);
      }
    uint32_t most = __reduce_max_sync(~0u, max(sizes & 0xffffu, sizes >> 16));
    float* scale = quant_scale(a.pool, kv, page, b.start, head);
    const float was = mine && page >= 0 && b.from > b.start ? *scale : 0.f;
    if (team > 1) {
      if (lane == 0) tops[warp] = most;
      __syncthreads();  // and the scale has been read
      for (int i = 0; i < team; ++i) most = max(most, tops[(warp & ~(team - 1)) + i]);
      __syncthreads();
    } else {
      __syncwarp();
    }
    if (!mine || page < 0) continue;
    uint32_t e = need_exponent(pair<T>(most).x);
    if (b.from > b.start) e = max(e, held_exponent(was));
    if (mate == 0 && lane == 0) *scale = power(e);
    const float i1 = inverse_power(e);
    uint8_t* codes = quant_code(a.pool, kv, page, b.start, head) + part * 8;
    const int64_t c_step = a.pool.st[kv];
    if (b.from > b.start && power(e) != was) {
      for (int at = from; at < b.from - b.start; at += step) {
        uint2* to = reinterpret_cast<uint2*>(codes + at * c_step);
        const uint2 v = *to;
        const auto again = [&](uint32_t four) {
          const float2 lo = decode2f(four & 0xffffu), hi = decode2f(four >> 16);
          return encode2(lo.x * was * i1, lo.y * was * i1) |
                 (encode2(hi.x * was * i1, hi.y * was * i1) << 16);
        };
        *to = make_uint2(again(v.x), again(v.y));
      }
    }
    codes += (b.from - b.start) * c_step;
    for (int i0 = 0; i0 < count; i0 += kAtOnce * step) {
      if (!once) load(u, w, i0);
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) {
        const int at = i0 + from + i * step;
        const auto code = [&](uint32_t two) {
          float2 f = pair<T>(two);
          if (special) f = make_float2(nan_for_infinite(f.x), nan_for_infinite(f.y));
          return encode2(f.x * i1, f.y * i1);
        };
        if (at < count)
          *reinterpret_cast<uint2*>(codes + at * c_step) =
              make_uint2(code(u[i].x) | (code(u[i].y) << 16),
                         code(u[i].z) | (code(u[i].w) << 16));
      }
    }
  }
}

struct ReadArgs {
  QuantPool pool;
  void* x[2];
  int64_t xt[2], xh[2];
  int64_t total;
  const int32_t* cu;
  int32_t seqs;
};

template <typename T>
__device__ __forceinline__ uint32_t pack(float2 f);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 h = __float22bfloat162_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float2 f) {
  const __half2 h = __float22half2_rn(f);
  return *reinterpret_cast<const uint32_t*>(&h);
}

constexpr int kReadWarps = 4;
constexpr int kReadRows = 2;  // of a warp

// A warp for two rows: lane i finds row i's page, and then 16 codes at a time are
// dealt to the lanes over all of them. WIDE: 32 bytes of an output at once.
template <typename T, bool WIDE>
__global__ void __launch_bounds__(kReadWarps * 32) read_kernel(const ReadArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t r0 =
      (static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5)) * kReadRows;
  if (r0 >= a.total) return;
  int32_t s = last_upto(a.seqs, r0, [&](int32_t i) { return clamped(a.cu[i], a.total); });
  // -2: a row of no sequence, -1: no page
  int32_t page = -2, tok = 0;
  const int64_t r = r0 + lane;
  if (lane < kReadRows && r < a.total) {
    while (s + 1 < a.seqs && r >= clamped(a.cu[s + 1], a.total)) ++s;
    const int64_t c0 = clamped(a.cu[s], a.total), c1 = clamped(a.cu[s + 1], a.total);
    if (r >= c0 && r < c1) {
      tok = static_cast<int32_t>(r - c0);
      page = tok < (a.pool.max_pages << a.pool.page_log2) ? quant_page(a.pool, s, tok) : -1;
    }
  }
  const uint32_t parts = a.pool.dim / 16, half = a.pool.kv_heads * parts, units = 2 * half;
  const uint32_t all = units * kReadRows;
  constexpr int kUnroll = 4;
  for (uint32_t e0 = 0; e0 < all; e0 += 32 * kUnroll) {
    uint4 c[kUnroll];
    float scale[kUnroll];
    T* to[kUnroll];
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      const uint32_t e = e0 + 32 * i + lane, row = min(e / units, kReadRows - 1u);
      const int32_t p = __shfl_sync(~0u, page, row), t = __shfl_sync(~0u, tok, row);
      const uint32_t u = e - row * units, kv = u >= half, rest = u - (kv ? half : 0);
      const int32_t head = rest / parts, part = rest - head * parts;
      c[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 0.f;
      to[i] = nullptr;
      if (e < all && p >= -1)
        to[i] = static_cast<T*>(a.x[kv]) + (r0 + row) * a.xt[kv] + head * a.xh[kv] + part * 16;
      if (e < all && p >= 0) {
        c[i] = *reinterpret_cast<const uint4*>(quant_code(a.pool, kv, p, t, head) + part * 16);
        scale[i] = *quant_scale(a.pool, kv, p, t, head);
      }
    }
#pragma unroll
    for (int i = 0; i < kUnroll; ++i) {
      if (!to[i]) continue;
      const auto two = [&](uint32_t codes) {
        const float2 f = decode2f(codes);
        return pack<T>(make_float2(f.x * scale[i], f.y * scale[i]));
      };
      const uint32_t x[8] = {two(c[i].x & 0xffff), two(c[i].x >> 16), two(c[i].y & 0xffff),
                             two(c[i].y >> 16),    two(c[i].z & 0xffff), two(c[i].z >> 16),
                             two(c[i].w & 0xffff), two(c[i].w >> 16)};
      if constexpr (WIDE) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(to[i]), "r"(x[0]),
                     "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                     : "memory");
      } else {
        reinterpret_cast<uint4*>(to[i])[0] = make_uint4(x[0], x[1], x[2], x[3]);
        reinterpret_cast<uint4*>(to[i])[1] = make_uint4(x[4], x[5], x[6], x[7]);
      }
    }
  }
}

// What writing and reading check alike: rows of 16-bit elements.
dsa_status check_rows(const void* k, const void* v, int32_t dtype, int64_t total, int64_t k_st,
                      int64_t k_sh, int64_t v_st, int64_t v_sh, const int32_t* cu, int32_t seqs,
                      int32_t kv_heads) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (total < 0 || seqs < 0) return DSA_EINVAL;
  if (dtype == DSA_DTYPE_F32 || total > INT32_MAX || seqs >= (1 << 28)) return DSA_EUNSUPPORTED;
  if (total == 0 || seqs == 0 || kv_heads == 0) return DSA_OK;
  if (!k || !v || !cu) return DSA_EINVAL;
  if (!quant_aligned16(k) || !quant_aligned16(v)) return DSA_EUNSUPPORTED;
  for (int64_t s : {k_st, k_sh, v_st, v_sh})
    if (s < 0 || s % 8 != 0) return DSA_EUNSUPPORTED;
  return DSA_OK;
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_quant_cache_write(const dsa_quant_pages* pages, const void* k,
                                            const void* v, int32_t dtype, int64_t total,
                                            int64_t k_st, int64_t k_sh, int64_t v_st,
                                            int64_t v_sh, const int32_t* cu, int32_t seqs,
                                            const int32_t* lens, void* stream) {
  dsa::WriteArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, pages, seqs);
  if (st != DSA_OK) return st;
  st = dsa::check_rows(k, v, dtype, total, k_st, k_sh, v_st, v_sh, cu, seqs, a.pool.kv_heads);
  if (st != DSA_OK) return st;
  const int32_t kv_heads = a.pool.kv_heads, block = 1 << a.pool.block_log2;
  if (block > 256) return DSA_EUNSUPPORTED;
  if (total == 0 || seqs == 0 || kv_heads == 0) return DSA_OK;
  if (!lens) return DSA_EINVAL;
  if (a.pool.max_pages == 0 || a.pool.num_pages == 0) return DSA_OK;
  a.x[0] = k;
  a.x[1] = v;
  a.xt[0] = k_st;
  a.xt[1] = v_st;
  a.xh[0] = k_sh;
  a.xh[1] = v_sh;
  a.total = total;
  a.cu = cu;
  a.seqs = seqs;
  a.lens = lens;
  const int64_t items = total / block + 2ll * seqs;
  if (items > INT32_MAX) return DSA_EUNSUPPORTED;
  // A team's registers hold the new tokens that a block gets on average: one warp
  // for single tokens, the whole block where more come to a sequence.
  const int64_t rows = 32 / (a.pool.dim / 8) * dsa::kAtOnce, mean = (total + seqs - 1) / seqs;
  int team = 1;
  while (team < 16 && team * rows < (mean < block ? mean : block)) team *= 2;
  const int warps = team > dsa::kWriteWarps ? team : dsa::kWriteWarps;
  const int64_t ys = (2ll * kv_heads + warps / team - 1) / (warps / team);
  const dim3 grid(static_cast<unsigned>(items), static_cast<unsigned>(ys < 65535 ? ys : 65535));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == DSA_DTYPE_BF16)
    dsa::write_kernel<__nv_bfloat16><<<grid, warps * 32, 0, s>>>(a, team);
  else
    dsa::write_kernel<__half><<<grid, warps * 32, 0, s>>>(a, team);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

extern "C" dsa_status dsa_quant_cache_read(const dsa_quant_pages* pages, const int32_t* cu,
                                           int32_t seqs, int64_t total, int32_t dtype, void* k,
                                           int64_t k_st, int64_t k_sh, void* v, int64_t v_st,
                                           int64_t v_sh, void* stream) {
  dsa::ReadArgs a{};
  dsa_status st = dsa::quant_pool(a.pool, pages, seqs);
  if (st != DSA_OK) return st;
  st = dsa::check_rows(k, v, dtype, total, k_st, k_sh, v_st, v_sh, cu, seqs, a.pool.kv_heads);
  if (st != DSA_OK) return st;
  if (total == 0 || seqs == 0 || a.pool.kv_heads == 0) return DSA_OK;
  a.x[0] = k;
  a.x[1] = v;
  a.xt[0] = k_st;
  a.xt[1] = v_st;
  a.xh[0] = k_sh;
  a.xh[1] = v_sh;
  a.total = total;
  a.cu = cu;
  a.seqs = seqs;
  constexpr int64_t kRows = dsa::kReadWarps * dsa::kReadRows;
  const unsigned grid = static_cast<unsigned>((total + kRows - 1) / kRows);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool wide = (k_st | k_sh | v_st | v_sh) % 16 == 0 &&
                    ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0;
  auto* kernel =
      dtype == DSA_DTYPE_BF16
          ? (wide ? dsa::read_kernel<__nv_bfloat16, true> : dsa::read_kernel<__nv_bfloat16, false>)
          : (wide ? dsa::read_kernel<__half, true> : dsa::read_kernel<__half, false>);
  kernel<<<grid, dsa::kReadWarps * 32, 0, s>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}
