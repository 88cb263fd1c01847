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

#include <cmath>

#include "common.cuh"

namespace pagedkv {

constexpr float kLog2e = 1.4426950408889634f;

struct ScoreRules {
  float cap_log2;            // cap * log2(e); 0: no cap
  float cap_arg;             // scale / cap: dot * cap_arg is tanh's argument
  const float* slopes;       // [num_heads], or null
  const int32_t* key_begin;  // [query rows] first key seen, or null
  const int32_t* key_end;    // [query rows] one past the last key seen, or null (prefill only)
  int32_t window;            // keys seen up to and with the query's own; 0: all
};

// The rules of a call, checked.
inline int make_rules(float scale, float softcap, const float* slopes, int32_t window, const int32_t* key_begin,
                      const int32_t* key_end, ScoreRules* out) {
  if (!(softcap >= 0.f) || !std::isfinite(softcap) || window < 0) return KV_ERR_INVALID_ARG;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(slopes) | reinterpret_cast<uintptr_t>(key_begin) |
                         reinterpret_cast<uintptr_t>(key_end);
  if (bits % 4 != 0) return KV_ERR_INVALID_ARG;
  ScoreRules r{0.f, 0.f, slopes, key_begin, key_end, window};
  if (softcap > 0.f) {
    r.cap_log2 = softcap * kLog2e;
    r.cap_arg = scale / softcap;
    // a cap so large or small that these leave float32
    if (!std::isfinite(r.cap_log2) || !(r.cap_log2 > 0.f) || !std::isfinite(r.cap_arg)) return KV_ERR_INVALID_ARG;
  }
  *out = r;
  return KV_OK;
}

// The keys lo .. hi - 1 that query row `row`, at position i of L tokens, sees
// (none: hi <= lo).
struct KeySpan {
  int lo, hi;
};
__device__ __forceinline__ KeySpan keys_seen(const ScoreRules& r, int64_t row, int i, int L) {
  KeySpan s{0, i + 1};
  if (r.window > 0) s.lo = max(0, i - r.window + 1);
  if (r.key_begin) s.lo = max(s.lo, __ldg(r.key_begin + row));
  if (r.key_end) s.hi = __ldg(r.key_end + row);
  s.hi = min(s.hi, L);
  return s;
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

// The rules of one decode tile for one lane of its warp (heads ng * 8 +
// (lane % 4) * 2 + c), and their absence.
struct NoRules {
  static constexpr bool kOn = false;
};
template <int NG>
struct TileRules {
  static constexpr bool kOn = true;
  float cap_log2, cap_arg;
  float slope[NG][2];  // slope * log2(e)
  int lo;              // first key seen
  int pos;             // the query's position
};

// A key's score in the exp2 domain from its dot product.
template <typename R>
__device__ __forceinline__ float rule_score(const R& r, float dot, float scale_log2, int t, int ng, int c) {
  if constexpr (!R::kOn) {
    return dot * scale_log2;
  } else {
    const float x = r.cap_log2 > 0.f ? soft_cap(dot, scale_log2, r.cap_log2, r.cap_arg) : dot * scale_log2;
    return fmaf(-r.slope[ng][c], static_cast<float>(r.pos - t), x);
  }
}
template <typename R>
__device__ __forceinline__ bool rule_sees(const R& r, int t, int L) {
  if constexpr (R::kOn) return t >= r.lo && t < L;
  else return t < L;
}

}  // namespace pagedkv
