// CPU proof that the library's per-element division (fp8q_math.h) is a binary32 division for every
// binary32 dividend, not only bf16 ones: the norm and the gate quantize binary32 rows.
//
// Let x = X 2^a and s = S 2^b with X, S in [2^23, 2^24), all steps normal (then they scale exactly), and
// count in steps of the quotient's last place: t = x / s = X 2^j / S in [2^23, 2^24), j = 23 or 24.
//   y = RN(1 / s) = (1 + e) / s, |e| <= 2^-24: x y is off t by at most 1, q = RN(x y) by at most 2 (half a
//   step, or a whole one where q reaches the next binade).  r = RN(q s - x) and r y are off by a factor of
//   at most (1 + 2^-24)^2, so that the last step rounds t + d with |d| <= 2 (2^-23 + 2^-48) < 2^-22 + 2^-46.
// That is RN(t) unless a border between two numbers, M / 2 with M odd, lies within |d| of t; t itself is no
// border (M S = 2^(j+1) X would make M > 2^24 divide X).  Such pairs have |2^(j+1) X - M S| <= 2 S |d|, which is
// below 8 + 2^-21: a whole number D of 1 to 8 either way.  For every S, j and D the equation M S = -D modulo
// 2^(j+1) leaves few M: all of them are tried.  A randomized pass backs the argument up.
#include <cstdint>
#include <cstdio>
#include <random>

#include "fp8q_math.h"

using fp8q::bits_to_f32;
using fp8q::f32_to_bits;

static uint64_t inverse(uint64_t odd) {  // modulo 2^64
  uint64_t v = odd;
  for (int i = 0; i < 6; ++i) v *= 2 - odd * v;
  return v;
}

// X, S in [2^23, 2^24) as numbers of [1, 2), times 2^ex and 2^es
static bool differs(uint32_t X, uint32_t S, int ex, int es) {
  const float x = bits_to_f32(uint32_t(127 + ex) << 23 | (X & 0x7FFFFF));
  const float s = bits_to_f32(uint32_t(127 + es) << 23 | (S & 0x7FFFFF));
  const float y = 1.0f / s, want = x / s;
  return f32_to_bits(fp8q::div_by_scale(x, s, y)) != f32_to_bits(want) ||
         f32_to_bits(fp8q::div_by_scale(-x, s, y)) != f32_to_bits(-want);
}

int main() {
  long long bad = 0, tried = 0, caught = 0;
#pragma omp parallel for reduction(+ : bad, tried, caught) schedule(static)
  for (int64_t S = 1 << 23; S < 1 << 24; ++S) {
    const int v = __builtin_ctzll(uint64_t(S));
    if (v > 3) continue;  // M is odd: D has as many factors of 2 as S
    const uint64_t inv = inverse(uint64_t(S) >> v);
    for (int j = 23; j <= 24; ++j) {
      const uint64_t modulus = uint64_t(1) << (j + 1 - v);
      for (int D = -8; D <= 8; ++D) {
        if (D == 0 || __builtin_ctz(unsigned(D)) != v) continue;
        const uint64_t M0 = uint64_t(-(int64_t(D) >> v)) * inv & (modulus - 1);
        for (uint64_t M = M0; M < uint64_t(1) << 25; M += modulus) {
          if (M < uint64_t(1) << 24) continue;
          const uint64_t at = M * uint64_t(S) + uint64_t(int64_t(D));
          const uint64_t X = at >> (j + 1);
          if (X << (j + 1) != at || X < 1 << 23 || X >= 1 << 24 || (j == 23) != (X >= uint64_t(S))) continue;
          ++tried;
          const float x = bits_to_f32(127u << 23 | (uint32_t(X) & 0x7FFFFF));
          const float s = bits_to_f32(127u << 23 | (uint32_t(S) & 0x7FFFFF));
          caught += x * (1.0f / s) != x / s;  // what the correction is for
          bad += differs(uint32_t(X), uint32_t(S), 0, 0);
          bad += differs(uint32_t(X), uint32_t(S), 0, -42);   // the smallest scales of groups
          bad += differs(uint32_t(X), uint32_t(S), 126, 119); // the largest
        }
      }
    }
  }
  fprintf(stderr, "pairs next to a border: %lld, uncorrected products off: %lld\n", tried, caught);
  printf("border_mismatches %lld\n", bad);
  printf("products_without_a_correction_all_right %d\n", caught > 0 ? 0 : 1);
  long long bad2 = 0;
#pragma omp parallel for reduction(+ : bad2)
  for (int chunk = 0; chunk < 64; ++chunk) {
    std::mt19937_64 rng(chunk + 1);
    for (int i = 0; i < 1000000; ++i) {
      const uint64_t z = rng();
      // quotients of 2^-11 to 2^9 by scales of 2^-43 to 2^118
      const int es = int(z >> 46 & 0x7F) - 43 + int(z >> 53 & 31), eq = int(z >> 58) % 20 - 10;
      if (es > 118 || es + eq > 127 || es + eq < -126) continue;
      bad2 += differs(uint32_t(z) | 1u << 23, uint32_t(z >> 23) | 1u << 23, es + eq, es);
    }
  }
  printf("random_mismatches %lld\n", bad2);
  return bad || bad2 || !caught;
}
