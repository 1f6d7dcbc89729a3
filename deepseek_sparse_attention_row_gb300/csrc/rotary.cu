// rotary.cu -- rotary positions of queries and keys: the C ABI of
// include/dsa_rotary.h.
//
// A CTA takes a few tokens: it computes the cosines and sines of their positions
// once, into shared memory. Each thread owns a chunk of pairs of one head and goes
// through the tokens with it, so that its addresses only step. Chunks are as wide
// as alignment lets them be, up to 16 bytes; neighbouring threads take neighbouring
// chunks. The first loads are on their way while the angles are computed.
//
// Bound by HBM: 8192 tokens of 40 heads of 128, bf16, take 31.3 us (5.4 TB/s read
// and written; 48 us with the angles in registers, computed by every thread, 35 us
// with chunks dealt to the threads by division); 4099 tokens of 16 heads of 96,
// fp32, neighbours, 9.0 us (5.6 TB/s). Four tokens to a CTA and two under way in a
// thread were the best of 2, 4, 8 and 16, and of 2 and 4 (or 4 and 8).
#include "../../include/dsa_rotary.h"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

namespace dsa {
namespace {

struct RotaryArgs {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh;
  int32_t heads, all_heads;  // all_heads counts those of k too
  int64_t tokens;
  const int32_t* positions;
  const int64_t* turns;
  int32_t pairs;
  int32_t turned, chunks;  // chunks of a head: those of the pairs, and all
  int32_t step, other;     // from chunk to chunk, and to its second half (SPLIT)
  int32_t each;            // tokens of a CTA
  int32_t part, width;     // heads of a CTA, and chunks of each
  float factor;
  int32_t transpose;
};

// cos and sin of the angle of position p. The fraction of a turn is exact; what is
// left after the nearest quarter turn, at most an eighth, is rounded once, to fp32
// relative to itself, so that both are good to two ulps of their own at any p, however
// small they are. (Cut to 32 bits first, 2^-34 of a turn at the most, the sine of an
// angle of 3e-8 was off by 1 %.)
__device__ __forceinline__ float2 cos_sin(int32_t p, int64_t turn, bool transpose) {
  const uint64_t t = static_cast<uint64_t>(static_cast<int64_t>(p)) * static_cast<uint64_t>(turn);
  const uint64_t v = t + (1ull << 61);
  const uint32_t quarter = static_cast<uint32_t>(v >> 62);
  const int64_t rest = static_cast<int64_t>((v << 2) ^ (1ull << 63));  // 2^-66 of a turn
  float s, c;
  sincospif(static_cast<float>(rest) * 0x1p-65f, &s, &c);  // half turns
  float2 r = quarter & 1 ? make_float2(-s, c) : make_float2(c, s);
  if (quarter & 2) r = make_float2(-r.x, -r.y);
  if (transpose) r.y = -r.y;
  return r;
}

// Two neighbouring elements of T, and as floats.
template <typename T>
struct Two;
template <>
struct Two<float> {
  using Raw = float2;
  static __device__ __forceinline__ float2 widen(Raw x) { return x; }
  static __device__ __forceinline__ Raw narrow(float2 x) { return x; }
};
template <>
struct Two<__nv_bfloat16> {
  using Raw = __nv_bfloat162;
  static __device__ __forceinline__ float2 widen(Raw x) { return __bfloat1622float2(x); }
  static __device__ __forceinline__ Raw narrow(float2 x) { return __float22bfloat162_rn(x); }
};
template <>
struct Two<__half> {
  using Raw = __half2;
  static __device__ __forceinline__ float2 widen(Raw x) { return __half22float2(x); }
  static __device__ __forceinline__ Raw narrow(float2 x) { return __float22half2_rn(x); }
};

// V elements of T, in memory as one load or store.
template <typename T, int V>
struct alignas(V * sizeof(T)) Chunk {
  typename Two<T>::Raw x[V / 2];
};
template <typename T>
struct Chunk<T, 1> {
  T x;
};

// (a, b) turned by (cos, sin).
__device__ __forceinline__ float2 turned(float xa, float xb, float2 cs) {
  return make_float2(fmaf(xa, cs.x, -(xb * cs.y)), fmaf(xb, cs.x, xa * cs.y));
}

constexpr int kMaxThreads = 512;

// V elements of T at a time. SPLIT: a chunk is V pairs, whose first and second
// elements lie apart; otherwise it is V / 2 pairs of neighbours.
template <typename T, int V, bool SPLIT>
__global__ void __launch_bounds__(kMaxThreads) rotary_kernel(const RotaryArgs a) {
  constexpr int P = SPLIT ? V : V / 2;  // pairs of a chunk
  constexpr int kAtOnce = 2;  // tokens
  using C = Chunk<T, V>;
  // [token][two pairs of a chunk][chunk]: neighbouring threads read neighbours
  extern __shared__ __align__(16) float2 angles[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.each;
  const int tokens = static_cast<int>(min(static_cast<int64_t>(a.each), a.tokens - t0));
  const int in = threadIdx.x / a.width, head = blockIdx.y * a.part + in;
  const int c = blockIdx.z * a.width + threadIdx.x - in * a.width;
  const bool mine = in < a.part && head < a.all_heads && c < a.chunks, turn = c < a.turned;
  const int at = turn ? c * a.step : 2 * a.pairs + (c - a.turned) * V;
  const bool q = head < a.heads;
  const int64_t st = q ? a.q_st : a.k_st, ot = q ? a.qo_st : a.ko_st;
  const T* from = q ? static_cast<const T*>(a.q) + head * a.q_sh
                    : static_cast<const T*>(a.k) + (head - a.heads) * a.k_sh;
  T* to = q ? static_cast<T*>(a.q_out) + head * a.qo_sh
            : static_cast<T*>(a.k_out) + (head - a.heads) * a.ko_sh;
  from += t0 * st + at;
  to += t0 * ot + at;
  C u[kAtOnce], w[SPLIT ? kAtOnce : 1];
  const auto load = [&](int t) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (!mine || t + i >= tokens) continue;
      const T* x = from + (t + i) * st;
      u[i] = *reinterpret_cast<const C*>(x);
      if constexpr (SPLIT)
        if (turn) w[i] = *reinterpret_cast<const C*>(x + a.other);
    }
  };
  load(0);
  for (int i = threadIdx.x; i < tokens * a.pairs; i += blockDim.x) {
    const int token = i / a.pairs, pair = i - token * a.pairs, chunk = pair / P, n = pair % P;
    float2 cs = cos_sin(a.positions[t0 + token], a.turns[pair], a.transpose);
    cs.x *= a.factor;
    cs.y *= a.factor;
    angles[token * a.pairs + (P > 1 ? ((n >> 1) * a.turned + chunk) * 2 + (n & 1) : chunk)] = cs;
  }
  __syncthreads();
  if (!mine) return;
  for (int t = 0;;) {
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (t + i >= tokens) continue;
      T* y = to + (t + i) * ot;
      if (turn) {
        const float2* cs = angles + (t + i) * a.pairs + (P > 1 ? c * 2 : c);
        if constexpr (V == 1) {
          const float2 z = turned(static_cast<float>(u[i].x), static_cast<float>(w[i].x), *cs);
          u[i].x = static_cast<T>(z.x);
          w[i].x = static_cast<T>(z.y);
        } else if constexpr (SPLIT) {
#pragma unroll
          for (int n = 0; n < V / 2; ++n) {
            const float4 f = *reinterpret_cast<const float4*>(cs + n * a.turned * 2);
            const float2 xa = Two<T>::widen(u[i].x[n]), xb = Two<T>::widen(w[i].x[n]);
            const float2 y0 = turned(xa.x, xb.x, make_float2(f.x, f.y));
            const float2 y1 = turned(xa.y, xb.y, make_float2(f.z, f.w));
            u[i].x[n] = Two<T>::narrow(make_float2(y0.x, y1.x));
            w[i].x[n] = Two<T>::narrow(make_float2(y0.y, y1.y));
          }
        } else {
#pragma unroll
          for (int n = 0; n < P; ++n) {
            const float2 f = cs[P > 1 ? (n >> 1) * a.turned * 2 + (n & 1) : 0];
            const float2 x = Two<T>::widen(u[i].x[n]);
            u[i].x[n] = Two<T>::narrow(turned(x.x, x.y, f));
          }
        }
        if constexpr (SPLIT) *reinterpret_cast<C*>(y + a.other) = w[i];
      }
      *reinterpret_cast<C*>(y) = u[i];
    }
    t += kAtOnce;
    if (t >= tokens) return;
    load(t);
  }
}

// Tokens of a CTA, and angles; CTAs that are wanted before a CTA gets several
// tokens.
constexpr int64_t kTokens = 4, kAngles = 2048, kCtas = 152 * 4;

template <typename T, int V>
dsa_status launch(RotaryArgs a, int32_t head_dim, bool halves, cudaStream_t stream) {
  // neighbours at addresses that hold no pair whole are taken one by one
  const bool split = halves || V == 1;
  a.turned = split ? a.pairs / V : 2 * a.pairs / V;
  a.chunks = a.turned + (head_dim - 2 * a.pairs) / V;
  a.step = halves ? V : V == 1 ? 2 : V;
  a.other = halves ? a.pairs : 1;
  a.width = a.chunks < kMaxThreads ? a.chunks : kMaxThreads;
  const int64_t most = kMaxThreads / a.width;
  a.part = static_cast<int32_t>(a.all_heads < most ? a.all_heads : most);
  const unsigned parts = (a.all_heads + a.part - 1) / a.part;
  int64_t each = a.tokens * parts / kCtas;
  if (each > kTokens) each = kTokens;
  if (a.pairs > 0 && each > kAngles / a.pairs) each = kAngles / a.pairs;
  if (each < 1) each = 1;
  a.each = static_cast<int32_t>(each);
  const dim3 grid(static_cast<unsigned>((a.tokens + each - 1) / each), parts,
                  (a.chunks + a.width - 1) / a.width);
  const unsigned threads = (a.part * a.width + 31) / 32 * 32;
  const size_t smem = static_cast<size_t>(each) * a.pairs * sizeof(float2);
  if (split)
    rotary_kernel<T, V, true><<<grid, threads, smem, stream>>>(a);
  else if constexpr (V > 1)
    rotary_kernel<T, V, false><<<grid, threads, smem, stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ECUDA;
}

// The widest chunk of which `bits` (addresses and steps in bytes, or'ed) and
// the pairs and what is behind them are whole numbers.
template <typename T>
dsa_status launch(const RotaryArgs& a, int32_t head_dim, bool halves, uint64_t bits,
                  cudaStream_t stream) {
  constexpr int e = sizeof(T);
  bits |= static_cast<uint64_t>(halves ? a.pairs : 2 * a.pairs) * e;
  bits |= static_cast<uint64_t>(head_dim - 2 * a.pairs) * e;
  if (bits % 16 == 0) return launch<T, 16 / e>(a, head_dim, halves, stream);
  if (bits % 8 == 0) return launch<T, 8 / e>(a, head_dim, halves, stream);
  if constexpr (e == 2)
    if (bits % 4 == 0) return launch<T, 2>(a, head_dim, halves, stream);
  return launch<T, 1>(a, head_dim, halves, stream);
}

}  // namespace
}  // namespace dsa

extern "C" dsa_status dsa_rotary(const void* q, void* q_out, int32_t heads, int64_t q_st,
                                 int64_t q_sh, int64_t qo_st, int64_t qo_sh, const void* k,
                                 void* k_out, int32_t kv_heads, int64_t k_st, int64_t k_sh,
                                 int64_t ko_st, int64_t ko_sh, int32_t dtype, int64_t tokens,
                                 int32_t head_dim, const int32_t* positions, const int64_t* turns,
                                 int32_t pairs, int32_t interleaved, float factor,
                                 int32_t transpose, void* stream) {
  if (dtype != DSA_DTYPE_F32 && dtype != DSA_DTYPE_BF16 && dtype != DSA_DTYPE_F16)
    return DSA_EINVAL;
  if (heads < 0 || kv_heads < 0 || tokens < 0 || head_dim < 0 || pairs < 0 ||
      pairs > head_dim / 2 || !std::isfinite(factor))
    return DSA_EINVAL;
  const int64_t all = static_cast<int64_t>(heads) + kv_heads;
  const int64_t strides[] = {q_st, q_sh, qo_st, qo_sh, k_st, k_sh, ko_st, ko_sh};
  for (int i = heads > 0 ? 0 : 4; i < (kv_heads > 0 ? 8 : 4); ++i)
    if (strides[i] < 0) return DSA_EINVAL;
  if (tokens > INT32_MAX || head_dim > 4096 || all > 65535)
    return DSA_EUNSUPPORTED;
  if (tokens == 0 || head_dim == 0 || all == 0) return DSA_OK;
  if ((heads > 0 && (!q || !q_out)) || (kv_heads > 0 && (!k || !k_out)) ||
      (pairs > 0 && (!positions || !turns)))
    return DSA_EINVAL;
  const uint64_t e = dtype == DSA_DTYPE_F32 ? 4 : 2;
  uint64_t bits = 0;
  if (heads > 0)
    bits |= reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(q_out) |
            static_cast<uint64_t>(q_st | q_sh | qo_st | qo_sh) * e;
  if (kv_heads > 0)
    bits |= reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(k_out) |
            static_cast<uint64_t>(k_st | k_sh | ko_st | ko_sh) * e;
  if (bits % e != 0) return DSA_EINVAL;
  dsa::RotaryArgs a{};
  a.q = q;
  a.k = k;
  a.q_out = q_out;
  a.k_out = k_out;
  a.q_st = q_st;
  a.q_sh = q_sh;
  a.qo_st = qo_st;
  a.qo_sh = qo_sh;
  a.k_st = k_st;
  a.k_sh = k_sh;
  a.ko_st = ko_st;
  a.ko_sh = ko_sh;
  a.heads = heads;
  a.all_heads = static_cast<int32_t>(all);
  a.tokens = tokens;
  a.positions = positions;
  a.turns = turns;
  a.pairs = pairs;
  a.factor = factor;
  a.transpose = transpose != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool halves = interleaved == 0;
  if (dtype == DSA_DTYPE_F32) return dsa::launch<float>(a, head_dim, halves, bits, s);
  if (dtype == DSA_DTYPE_BF16) return dsa::launch<__nv_bfloat16>(a, head_dim, halves, bits, s);
  return dsa::launch<__half>(a, head_dim, halves, bits, s);
}
