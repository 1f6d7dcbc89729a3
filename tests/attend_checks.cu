// attend_checks.cu -- host-side checks of the attention kernel's bookkeeping
// (csrc/attend.cuh), run without a GPU by test_attend_checks.py.
#include <cstdint>
#include <cstdio>
#include <random>

#include "attend.cuh"

using namespace dsa;

// Whatever an entry of the cut blocks holds (a workspace is not initialised),
// the join reads parts inside the workspace and writes rows inside the output.
static int joins_stay_in_range() {
  std::mt19937_64 rng(7);
  const int32_t edges[] = {0, 1, -1, 2, 17, 127, 128, 129, 255, 256, INT32_MAX, INT32_MIN,
                           INT32_MAX - 1, 0x7f7f7f7f, static_cast<int32_t>(0xffc00000u)};
  const auto any = [&](int32_t near) -> int32_t {
    switch (rng() % 4) {
      case 0: return edges[rng() % (sizeof(edges) / sizeof(edges[0]))];
      case 1: return static_cast<int32_t>(rng());
      default: return static_cast<int32_t>(rng() % (2 * static_cast<uint64_t>(near) + 2)) - 1;
    }
  };
  int64_t taken = 0;
  for (int i = 0; i < 2000000; ++i) {
    AttendArgs a{};
    a.group = 1 + static_cast<int32_t>(rng() % 128);
    a.tile_tokens = kTile / a.group;
    a.kv_heads = 1 + static_cast<int32_t>(rng() % 8);
    a.heads = a.kv_heads * a.group;
    a.tokens = 1 + static_cast<int64_t>(rng() % (rng() % 2 ? 300 : INT32_MAX));
    const int64_t ctas = 1 + static_cast<int64_t>(rng() % 152), x = rng() % ctas;
    CutBlock b{any(static_cast<int32_t>(a.tokens)), {any(a.tile_tokens), any(a.tile_tokens)},
               any(a.kv_heads), any(152)};
    if (!joinable(b, a, x, ctas)) continue;
    ++taken;
    for (int s = 0; s < 2; ++s) {
      if (b.ntok[s] == 0) continue;
      // the join's rows (rt < ntok) and parts (slot 2 (x + i), one of 2 ctas)
      const int64_t row = static_cast<int64_t>(b.ntok[s]) * a.group - 1;
      const int64_t tok = b.tok + static_cast<int64_t>(s) * b.ntok[0] + b.ntok[s] - 1;
      const int64_t head = static_cast<int64_t>(b.kh) * a.group + a.group - 1;
      const int64_t slot = 2 * (x + b.more) + 1;
      if (row >= kTile || b.tok < 0 || tok >= a.tokens || b.kh < 0 || head >= a.heads ||
          b.more < 1 || slot >= 2 * ctas) {
        std::printf("tok %d ntok %d %d kh %d more %d x %lld\n", b.tok, b.ntok[0], b.ntok[1], b.kh,
                    b.more, static_cast<long long>(x));
        return 1;
      }
    }
  }
  const CutBlock none{5, {3, 2}, 0, 0}, good{5, {3, 2}, 0, 4};
  AttendArgs a{};
  a.tile_tokens = 3;
  a.tokens = 10;
  a.kv_heads = 1;
  return taken < 1000 || joinable(none, a, 0, 8) || !joinable(good, a, 3, 8) ||
         joinable(good, a, 4, 8);
}

// Up to the longest table of pages of 16 tokens and the longest sequence.
static int tiles_hold_the_longest_lengths() {
  const int64_t most = INT32_MAX;
  for (const int64_t n : {int64_t{-5}, int64_t{0}, int64_t{1}, int64_t{128}, int64_t{129},
                          most - 4096, most - 127, most - 63, most - 15, most - 1, most}) {
    const int64_t want = n <= 0 ? 0 : (n + kTile - 1) / kTile;
    if (tiles_of(static_cast<int32_t>(n)) != want) {
      std::printf("%lld keys: %d tiles\n", static_cast<long long>(n),
                  tiles_of(static_cast<int32_t>(n)));
      return 1;
    }
  }
  return 0;
}

int main() {
  if (joins_stay_in_range() || tiles_hold_the_longest_lengths()) return 1;
  std::puts("ok");
  return 0;
}
