// Score rules: what the attention calls ending in _rules do to a score before
// the softmax, and which keys a query sees.
//
// For a query at position i of a sequence of L tokens, and key j:
//   s = scale q.k_j;  with a cap c: s = c tanh(s / c);  with a slope m of the
//   query's head: s = s - m |i - j|;
//   seen: max(0, i - W + 1 (with a window W), begin) <= j < min(L, end), end
//   being i + 1 where the call gives none.
// Scores are held in the exp2 domain (times log2 e), as everywhere here.
#pragma once

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace pagedkv {

constexpr float kLog2e = 1.4426950408889634f;

// The cap for packed pairs, as a polynomial in the dot product: tanh(z) = z
// P(z^2) for |z| <= 1, P of degree 5, within 6e-7 of it (the fit of soft_cap's,
// two terms shorter: rounding the weights to 16 bits leaves 5e-4 and more).
// With z = a dot the coefficients take the powers of a^2 and scale_log2; the
// squares of dots it holds for end at 1 / a^2.  They are made on the host.
struct CapPoly {
  float2 c[6];  // each coefficient twice
  float limit;
  // base + the capped scores of two dots; `big` collects the largest square,
  // which the caller compares with limit.
  __device__ __forceinline__ uint64_t run(uint64_t dots, uint64_t base, float& big) const {
    const uint64_t u = tc::fmul2(dots, dots);
    const float2 u2 = tc::f2_split(u);
    big = max3(big, u2.x, u2.y);
    uint64_t y = tc::ffma2(tc::f2(c[5].x, c[5].y), u, tc::f2(c[4].x, c[4].y));
#pragma unroll
    for (int j = 3; j >= 0; --j) y = tc::ffma2(y, u, tc::f2(c[j].x, c[j].y));
    return tc::ffma2(dots, y, base);
  }
};

struct ScoreRules {
  float cap_log2;            // cap * log2(e); 0: no cap
  float cap_arg;             // scale / cap: dot * cap_arg is tanh's argument
  const float* slopes;       // [num_heads], or null
  const int32_t* key_begin;  // [query rows] first key seen, or null
  const int32_t* key_end;    // [query rows] one past the last key seen, or null (prefill only)
  int32_t window;            // keys seen up to and with the query's own; 0: all
  CapPoly poly;              // the cap's polynomial
};

// The rules of a call, checked.
inline int make_rules(float scale, float softcap, const float* slopes, int32_t window, const int32_t* key_begin,
                      const int32_t* key_end, ScoreRules* out) {
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < 0) return KV_ERR_INVALID_ARG;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(slopes) | reinterpret_cast<uintptr_t>(key_begin) |
                         reinterpret_cast<uintptr_t>(key_end);
  if (bits % 4 != 0) return KV_ERR_INVALID_ARG;
  ScoreRules r{0.f, 0.f, slopes, key_begin, key_end, window, {}};
  if (softcap > 0.f) {
    r.cap_log2 = softcap * kLog2e;
    r.cap_arg = scale / softcap;
    // a cap so large or small that these, or the former's reciprocal, leave float32
    if (!std::isfinite(r.cap_log2) || !(r.cap_log2 >= FLT_MIN) || !std::isfinite(r.cap_arg)) return KV_ERR_INVALID_ARG;
    constexpr float k[6] = {0.9999994039535522f,    -0.3332904279232025f,  0.13281433284282684f,
                            -0.051605675369501114f, 0.016743117943406105f, -0.0030670613050460815f};
    // Where a^2 is so small that a^10 would leave float32 (a cap over 3162 times
    // the scale: 50 with a scale of 1/128, say) nothing is in range and every score
    // takes the exact form, at a cost in time.
    const double a2 = static_cast<double>(r.cap_arg) * r.cap_arg;
    const bool fits = a2 >= 1e-7 && a2 <= 1e7;
    double power = static_cast<double>(scale) * kLog2e;
    for (int i = 0; i < 6; ++i) {
      r.poly.c[i].x = r.poly.c[i].y = fits ? static_cast<float>(k[i] * power) : 0.f;
      power *= a2;
    }
    r.poly.limit = fits ? static_cast<float>(1.0 / a2) : -1.f;
  }
  *out = r;
  return KV_OK;
}

// The keys lo .. hi - 1 that query row `row`, at position i of L tokens, sees
// (none: hi <= lo).  Both are 0 or more whatever the arrays hold, so that taking
// a position of the sequence from them stays in 32 bits.
struct KeySpan {
  int lo, hi;
};
__device__ __forceinline__ KeySpan keys_seen(const ScoreRules& r, int64_t row, int i, int L) {
  KeySpan s{0, i + 1};
  if (r.window > 0) s.lo = max(0, i - r.window + 1);
  if (r.key_begin) s.lo = max(s.lo, __ldg(r.key_begin + row));
  if (r.key_end) s.hi = __ldg(r.key_end + row);
  s.hi = max(0, min(s.hi, L));
  return s;
}

// Bits lo .. hi - 1 of a word, as far as it has them.
__device__ __forceinline__ uint32_t bits_between(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 32);
  return lo < hi ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
}

// c tanh(s / c) log2(e) of a score s = dot * scale: tanh(z) = z P(z^2) for
// |z| <= 1, P the polynomial of least relative error (4e-9, so float32's
// rounding is what is left: below 1.1e-7 over the interval), fitted by exchange
// against 40 digits; beyond, 1 - 2 / (1 + e^2|z|), whose two approximations are
// off by less than 4e-7 of it there.  z P(z^2) keeps small scores' relative
// precision, which the second form would lose under a large cap.
__device__ __forceinline__ float soft_cap(float dot, float scale_log2, float cap_log2, float cap_arg) {
  const float z = dot * cap_arg, u = z * z;
  if (u <= 1.f) {
    float p = -3.533457638695836e-4f;
    p = fmaf(p, u, 2.2822304163128138e-3f);
    p = fmaf(p, u, -7.917446084320545e-3f);
    p = fmaf(p, u, 2.1464820951223373e-2f);
    p = fmaf(p, u, -5.387091264128685e-2f);
    p = fmaf(p, u, 1.333215981721878e-1f);
    p = fmaf(p, u, -3.3333277702331543e-1f);
    p = fmaf(p, u, 1.f);
    return dot * scale_log2 * p;
  }
  const float e = fast_exp2(fabsf(z) * (2.f * kLog2e));
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(1.f + e));
  return copysignf(fmaf(-2.f * cap_log2, inv, cap_log2), z);  // NaN: copysign keeps it
}

// soft_cap out of line, for the rare scores beyond the cap.
static __device__ __noinline__ float soft_cap_far(float dot, float scale_log2, float cap_log2, float cap_arg) {
  return soft_cap(dot, scale_log2, cap_log2, cap_arg);
}

// The rules of one decode tile for one lane of its warp (heads ng * 8 +
// (lane % 4) * 2 + c), and their absence.
struct NoRules {
  static constexpr bool kOn = false;
};
template <int NG, bool CAP>
struct TileRules {
  static constexpr bool kOn = true, kCap = CAP;
  float cap_log2, cap_arg;
  CapPoly poly;
  uint64_t fall[NG];  // -slope * log2(e) of the lane's two heads
  int lo;             // first key seen
  int pos;            // the query's position
};

template <typename R>
__device__ __forceinline__ bool rule_sees(const R& r, int t, int L) {
  if constexpr (R::kOn) return t >= r.lo && t < L;
  else return t < L;
}

// The dots of NS 16-token sub-tiles (tokens t0 + 16 u and + 8 further, two
// heads each) into scores under the rules, in the exp2 domain.
template <int NS, int NG, bool CAP>
__device__ __forceinline__ void rule_scores(const TileRules<NG, CAP>& r, float (&sc)[NS][NG][4], float scale_log2,
                                            int t0) {
  const CapPoly& cap = r.poly;
  const float from = static_cast<float>(r.pos - t0);  // distance of the first token
  const uint64_t sl2 = tc::f2(scale_log2, scale_log2);
  if constexpr (CAP) {
    // Scores beyond the cap (or in slots that are not seen, at a cost in time
    // only): the exact form, out of line.
    float far = 0.f;
#pragma unroll
    for (int u = 0; u < NS; ++u)
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int e = 0; e < 4; e += 2) far = max3(far, fabsf(sc[u][ng][e]), fabsf(sc[u][ng][e + 1]));
    if (__any_sync(0xffffffffu, far * far > cap.limit)) {
#pragma unroll
      for (int u = 0; u < NS; ++u)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float away = from - (u * 16 + (e >> 1) * 8);
            const float2 fall = tc::f2_split(r.fall[ng]);
            sc[u][ng][e] = fmaf(e & 1 ? fall.y : fall.x, away,
                                soft_cap_far(sc[u][ng][e], scale_log2, r.cap_log2, r.cap_arg));
          }
      return;
    }
  }
#pragma unroll
  for (int u = 0; u < NS; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float away = from - (u * 16 + h * 8);
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) {
        float* d = &sc[u][ng][2 * h];
        const uint64_t bias = tc::fmul2(r.fall[ng], tc::f2(away, away)), x = tc::f2(d[0], d[1]);
        float unused = 0.f;
        const float2 y = tc::f2_split(CAP ? cap.run(x, bias, unused) : tc::ffma2(x, sl2, bias));
        d[0] = y.x;
        d[1] = y.y;
      }
    }
}

}  // namespace pagedkv
