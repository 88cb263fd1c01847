// Position rotation on the way into the cache: the rotary embedding of a
// step's queries and keys, the queries to their own buffer, the keys and the
// values to the paged pool at their slots.
//
// Per token at position p, per head, the first R = rot_dim of its D values
// form R / 2 pairs; pair i is (x_i, x_{i + R/2}), or (x_{2i}, x_{2i+1}) in the
// interleaved form, and is turned by the angle whose cosine c and sine s the
// table's row p holds (c_0 .. c_{R/2-1}, s_0 .. s_{R/2-1}, float32):
//   y_a = x_a c - x_b s,   y_b = x_b c + x_a s.
// The other D - R values pass through.  Each product and each sum is rounded
// to float32 by itself (no fused multiply-add), so the result is defined to
// the bit; it is rounded once more to the output type, or, for an fp8 cache,
// quantised from float32 with no 16-bit rounding between ("paged-attention-
// impl-detail", 实践建议 4: the row steps of the fp8 cache write).
// With several axes (time, height, width of an image's or a film's tokens) a
// token has one position per axis, and pair i is turned by the angle i of its
// axis' position: row positions[axis(i)][t] of the table.
// A slot of -1 marks a padded token: nothing is written for it
// ("MiniPaged-Qwen" §11-§12, the cache write's rules).
//
// What bounds it: memory.  A token's q, k and v are read once, its q and its
// two cache rows written once; the table row (4 R bytes, shared by all its
// heads) is the only other traffic.
//
// Kernel shape: a lane owns 16 values of a head as two 8-value runs chosen so
// that both members of every pair lie in the lane (the halves at c and
// c + R/2, or 16 consecutive values when interleaved).  D / 16 lanes make a
// head and a CTA's thread count is a multiple of D / 16, so a thread keeps
// one column, and one set of 8 cosines and sines in registers, over all the
// heads it walks.  Heads come in rounds of kUnits whose loads all go out
// before any is used, the first round's beside the position and the slot.
// Few tokens: one CTA per token and round of heads, so that a decode step's
// latency is one chain of loads (position, table row, then the stores); many
// tokens: one CTA per token walks all its heads.
//
// Measured on the device: 32768 tokens of 28 + 2 x 4 heads of 128, bf16: 96.7
// us, 621 MB, 0.95 of the copy rate; 4581 of 32 + 2 x 8: 19.8 us (0.82: 152
// SMs of 12 CTAs hold 1824 tokens, so its 2.5 rounds take three), in float32
// 34.2 us, 216 MB (0.94), into fp8 caches 23.4 us (0.64: a token's second round
// of heads, where all its K and V rows lie, is loaded after the first is
// stored and is half empty; 20.8 with a product in the place of the correctly
// rounded divisions that the codes' definition asks for); 8 tokens: 2.0 us.

#include <type_traits>

#include "common.cuh"
#include "token_rows.h"

namespace pagedkv {
namespace {

constexpr int kRopeThreads = 128;
// Heads a thread has in flight, and CTAs that must fit an SM (a bound on the
// registers): warps in flight pay more than loads per thread.  32768 tokens of
// 28 + 2 x 4 heads of 128, bf16: 122.7 us with four heads and no bound, 96.6
// with one and twelve CTAs; 4581 tokens of 32 + 2 x 8 into fp8: 31.0 us, and
// 23.2 with two and eight (whose rows need more registers).
template <typename T, bool F8> struct RopeShape {
  static constexpr int kUnits = F8 ? 2 : 1;
  static constexpr int kCtas = F8 || sizeof(T) == 4 ? 8 : 12;
};

constexpr int kRopeAxes = 4, kRopeAxisPairs = 256;

// One position a token; several, with the pairs in runs of eight (a lane's
// share) of one axis; several in any order.
enum RopeAxes { kOneAxis = 0, kAxisRuns = 1, kAnyAxis = 2 };

struct RopeParams {
  void* q_out;
  const void* q;
  const void* k;
  const void* v;
  const int32_t* positions;
  const float* cos_sin;
  void* k_cache;
  void* v_cache;
  float* k_scales;  // fp8 caches: [num_blocks][num_kv_heads][block_size]
  float* v_scales;
  const int32_t* slot_mapping;
  int32_t num_heads, num_kv_heads, head_dim, rot_dim, block_size;
  int64_t max_positions, num_slots;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // elements between tokens
  // several axes (num_axes > 1): positions [num_axes][num_tokens], and the axis
  // of each pair, two bits each from the lowest on
  int64_t num_tokens;
  int32_t num_axes, axis_runs;  // axis_runs: pairs 8 i .. 8 i + 7 are of one axis
  uint64_t axis_of_pair[kRopeAxisPairs / 32];
};

// The position that pair `pair` of a token turns by.
__device__ __forceinline__ int32_t rope_position(const RopeParams& p, const int32_t (&pos)[kRopeAxes], int pair) {
  const int axis = static_cast<int>(p.axis_of_pair[pair >> 5] >> (2 * (pair & 31))) & 3;
  int32_t at = pos[0];
#pragma unroll
  for (int a = 1; a < kRopeAxes; ++a) at = axis == a ? pos[a] : at;
  return at;
}

// Position and slot of token t; false when the token is padded or out of
// range (recorded by one thread of the CTA).
__device__ __forceinline__ bool rope_token(const RopeParams& p, int32_t pos, int32_t slot, bool reporter) {
  if (slot == -1) return false;
  if (slot < 0 || slot >= p.num_slots || pos < 0 || pos >= p.max_positions) {
    if (reporter) record_error(KV_ERR_DEVICE_BOUNDS);
    return false;
  }
  return true;
}

// The same for a token with several positions; pos[a] of axis a.
__device__ __forceinline__ bool rope_token_axes(const RopeParams& p, const int32_t (&pos)[kRopeAxes], int32_t slot,
                                                bool reporter) {
  bool in = true;
#pragma unroll
  for (int a = 0; a < kRopeAxes; ++a) in = in && (a >= p.num_axes || (pos[a] >= 0 && pos[a] < p.max_positions));
  return rope_token(p, in ? 0 : -1, slot, reporter);
}

__device__ __forceinline__ void rotate_pair(float& a, float& b, float c, float s) {
  const float ya = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = ya;
}

// Eight values of type T as one or two 16-byte vectors, held as they came.
template <typename T>
struct Run8 {
  static constexpr int kVecs = 8 * static_cast<int>(sizeof(T)) / 16;
  uint4 v[kVecs];
  // plain loads: q_out may be q, so no read-only path
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < kVecs; ++i) reinterpret_cast<uint4*>(p)[i] = v[i];
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const T* e = reinterpret_cast<const T*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = DType<T>::to_float(e[i]);
  }
  __device__ __forceinline__ void put(const float (&x)[8]) {
    T* e = reinterpret_cast<T*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = DType<T>::from_float(x[i]);
  }
};

template <bool INTER>
__device__ __forceinline__ void rotate16(float (&x0)[8], float (&x1)[8], const float (&c)[8], const float (&s)[8]) {
  if constexpr (INTER) {  // pairs 0..3 in the first run, 4..7 in the second
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rotate_pair(x0[2 * i], x0[2 * i + 1], c[i], s[i]);
      rotate_pair(x1[2 * i], x1[2 * i + 1], c[i + 4], s[i + 4]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) rotate_pair(x0[i], x1[i], c[i], s[i]);
  }
}

// One CTA per (token, part): the part's rounds of heads.  F8: K and V are
// quantised, a head's D / 16 lanes (4, 8 or 16, so within one warp) taking
// the row's largest magnitude by shuffles.
template <typename T, bool INTER, bool F8, RopeAxes AXES>
__global__ void __launch_bounds__(kRopeThreads, (RopeShape<T, F8>::kCtas))
rope_cache_kernel(const RopeParams p, int threads) {
  constexpr int kUnits = RopeShape<T, F8>::kUnits;
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int lph = p.head_dim >> 4;                     // lanes per head
  const int heads = p.num_heads + 2 * p.num_kv_heads;  // q, k, v heads of a token
  const int per = threads / lph;                       // heads the CTA touches at once
  const int col = tid % lph;
  const int half = p.rot_dim >> 1;
  const bool turn = col * 16 < p.rot_dim;
  // element offsets of the lane's two runs
  const int e0 = INTER || !turn ? col * 16 : col * 8;
  const int e1 = INTER || !turn ? e0 + 8 : e0 + half;
  const int first = blockIdx.y * (per * kUnits) + tid / lph, step = gridDim.y * (per * kUnits);

  const int32_t slot = __ldg(p.slot_mapping + t);
  int32_t pos[kRopeAxes];
#pragma unroll
  for (int a = 0; a < (AXES != kOneAxis ? kRopeAxes : 1); ++a)
    if (a == 0 || a < p.num_axes) pos[a] = __ldg(p.positions + (AXES != kOneAxis ? a * p.num_tokens : 0) + t);
  Run8<T> r[kUnits][2];
  auto load = [&](int h0) {
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int h = h0 + u * per;
      if (h >= heads) break;
      const T* src;
      if (h < p.num_heads) src = static_cast<const T*>(p.q) + t * p.q_stride + h * p.head_dim;
      else if (h < p.num_heads + p.num_kv_heads)
        src = static_cast<const T*>(p.k) + t * p.k_stride + (h - p.num_heads) * p.head_dim;
      else src = static_cast<const T*>(p.v) + t * p.v_stride + (h - p.num_heads - p.num_kv_heads) * p.head_dim;
      r[u][0].load(src + e0);
      r[u][1].load(src + e1);
    }
  };
  // the first heads' rows depend on neither position nor slot: their loads go
  // out beside those (a padded token's rows are read and dropped)
  load(first);
  const bool reporter = tid == 0 && blockIdx.y == 0;
  if (AXES != kOneAxis ? !rope_token_axes(p, pos, slot, reporter) : !rope_token(p, pos[0], slot, reporter)) return;
  // With axes in any order the CTA first gathers the token's own row of angles,
  // a thread per pair from its axis' row of the table (each lane picking its
  // pairs from up to four rows took 40 registers into spills: 43.0 us instead of
  // 33.1 for 8192 tokens of 28 + 2 x 4 heads of 128).  Where a lane's eight pairs
  // are of one axis it reads them from that axis' row (31.1 us; with one position
  // a token 29.4).
  const float* row;
  __shared__ __align__(16) float own_row[AXES == kAnyAxis ? 2 * kRopeAxisPairs : 4];
  if constexpr (AXES == kAnyAxis) {
    for (int i = tid; i < half; i += threads) {
      const float* from = p.cos_sin + rope_position(p, pos, i) * static_cast<int64_t>(p.rot_dim) + i;
      own_row[i] = __ldg(from);
      own_row[half + i] = __ldg(from + half);
    }
    __syncthreads();
    row = own_row + col * 8;
  } else {
    const int32_t at = AXES == kOneAxis || !turn ? pos[0] : rope_position(p, pos, col * 8);
    row = p.cos_sin + static_cast<int64_t>(at) * p.rot_dim + col * 8;
  }
  float c[8], s[8];
  if (turn) {
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      float4 cv, sv;
      if constexpr (AXES == kAnyAxis) {
        cv = *reinterpret_cast<const float4*>(row + i);
        sv = *reinterpret_cast<const float4*>(row + half + i);
      } else {
        cv = __ldg(reinterpret_cast<const float4*>(row + i));
        sv = __ldg(reinterpret_cast<const float4*>(row + half + i));
      }
      c[i] = cv.x, c[i + 1] = cv.y, c[i + 2] = cv.z, c[i + 3] = cv.w;
      s[i] = sv.x, s[i + 1] = sv.y, s[i + 2] = sv.z, s[i + 3] = sv.w;
    }
  }
  const int64_t blk = slot / p.block_size, off = slot % p.block_size;
  // every thread of a warp runs the same rounds: the bound goes by the round's first head
  for (int h0 = first; h0 - tid / lph < heads; h0 += step) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int h = h0 + u * per;
      const bool in = h < heads;
      const bool is_v = h >= p.num_heads + p.num_kv_heads;
      const int hk = h - p.num_heads - (is_v ? p.num_kv_heads : 0);  // kv head (h >= num_heads)
      if (!F8) {
        if (!in) break;
        if (turn && !is_v) {
          float x0[8], x1[8];
          r[u][0].get(x0);
          r[u][1].get(x1);
          rotate16<INTER>(x0, x1, c, s);
          r[u][0].put(x0);
          r[u][1].put(x1);
        }
        T* dst = h < p.num_heads
                     ? static_cast<T*>(p.q_out) + t * p.q_out_stride + h * p.head_dim
                     : static_cast<T*>(is_v ? p.v_cache : p.k_cache) +
                           (static_cast<int64_t>(slot) * p.num_kv_heads + hk) * p.head_dim;
        r[u][0].store(dst + e0);
        r[u][1].store(dst + e1);
      } else {
        float x0[8], x1[8], amax = 0.f;
        if (in) {
          r[u][0].get(x0);
          r[u][1].get(x1);
          if (turn && !is_v) rotate16<INTER>(x0, x1, c, s);
        }
        if (__any_sync(0xffffffffu, in && h >= p.num_heads)) {  // the warp holds K or V heads
          if (in) {
#pragma unroll
            for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fmaxf(fabsf(x0[i]), fabsf(x1[i])));
          }
          for (int o = lph >> 1; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        }
        if (!in) continue;
        if (h < p.num_heads) {
          T* dst = static_cast<T*>(p.q_out) + t * p.q_out_stride + h * p.head_dim;
          r[u][0].put(x0);
          r[u][1].put(x1);
          r[u][0].store(dst + e0);
          r[u][1].store(dst + e1);
        } else {
          const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
          uint16_t w0[4], w1[4];
#pragma unroll
          for (int i = 0; i < 8; i += 2) {
            w0[i / 2] = e4m3x2_from(__fdiv_rn(x0[i], scale), __fdiv_rn(x0[i + 1], scale));
            w1[i / 2] = e4m3x2_from(__fdiv_rn(x1[i], scale), __fdiv_rn(x1[i + 1], scale));
          }
          uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) +
                         (static_cast<int64_t>(slot) * p.num_kv_heads + hk) * p.head_dim;
          *reinterpret_cast<uint2*>(dst + e0) = make_uint2(w0[0] | static_cast<uint32_t>(w0[1]) << 16,
                                                           w0[2] | static_cast<uint32_t>(w0[3]) << 16);
          *reinterpret_cast<uint2*>(dst + e1) = make_uint2(w1[0] | static_cast<uint32_t>(w1[1]) << 16,
                                                           w1[2] | static_cast<uint32_t>(w1[3]) << 16);
          if (col == 0) (is_v ? p.v_scales : p.k_scales)[(blk * p.num_kv_heads + hk) * p.block_size + off] = scale;
        }
      }
    }
  }
}

// Any head_dim, any even rot_dim, any alignment of the elements: one warp
// per (token, head), lanes over the pairs and then over the values that pass
// through.  F8 walks a K or V row twice (its largest magnitude, its codes).
template <typename T, bool INTER, bool F8, RopeAxes AXES>
__global__ void __launch_bounds__(kRopeThreads) rope_cache_any_kernel(const RopeParams p, int64_t num_tokens) {
  const int lane = threadIdx.x & 31;
  const int heads = p.num_heads + 2 * p.num_kv_heads, D = p.head_dim, half = p.rot_dim >> 1;
  const int64_t total = num_tokens * heads, nwarps = static_cast<int64_t>(gridDim.x) * (kRopeThreads / 32);
  for (int64_t w = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5); w < total; w += nwarps) {
    const int64_t t = w / heads;
    const int h = static_cast<int>(w % heads);
    const int32_t slot = __ldg(p.slot_mapping + t);
    int32_t pos[kRopeAxes];
#pragma unroll
    for (int a = 0; a < (AXES != kOneAxis ? kRopeAxes : 1); ++a)
      if (a == 0 || a < p.num_axes) pos[a] = __ldg(p.positions + (AXES != kOneAxis ? a * p.num_tokens : 0) + t);
    const bool reporter = lane == 0 && h == 0;
    if (AXES != kOneAxis ? !rope_token_axes(p, pos, slot, reporter) : !rope_token(p, pos[0], slot, reporter)) continue;
    const bool is_q = h < p.num_heads, is_v = h >= p.num_heads + p.num_kv_heads;
    const int hk = h - p.num_heads - (is_v ? p.num_kv_heads : 0);
    const T* src = is_q ? static_cast<const T*>(p.q) + t * p.q_stride + static_cast<int64_t>(h) * D
                        : static_cast<const T*>(is_v ? p.v : p.k) + t * (is_v ? p.v_stride : p.k_stride) +
                              static_cast<int64_t>(hk) * D;
    auto row_of = [&](int i) {  // the table row of pair i
      return p.cos_sin + static_cast<int64_t>(AXES != kOneAxis ? rope_position(p, pos, i) : pos[0]) * p.rot_dim;
    };
    const int turned = is_v ? 0 : p.rot_dim;
    // visit(e, y): every output value of the row once, pairs first
    auto walk = [&](auto visit) {
      for (int i = lane; i < turned / 2; i += 32) {
        const int ea = INTER ? 2 * i : i, eb = INTER ? 2 * i + 1 : i + half;
        float a = DType<T>::to_float(src[ea]), b = DType<T>::to_float(src[eb]);
        const float* row = row_of(i);
        rotate_pair(a, b, __ldg(row + i), __ldg(row + half + i));
        visit(ea, a);
        visit(eb, b);
      }
      for (int e = turned + lane; e < D; e += 32) visit(e, DType<T>::to_float(src[e]));
    };
    const int64_t at = (static_cast<int64_t>(slot) * p.num_kv_heads + hk) * D;
    if (is_q || !F8) {
      T* dst = is_q ? static_cast<T*>(p.q_out) + t * p.q_out_stride + static_cast<int64_t>(h) * D
                    : static_cast<T*>(is_v ? p.v_cache : p.k_cache) + at;
      walk([&](int e, float y) { dst[e] = DType<T>::from_float(y); });
    } else {
      float amax = 0.f;
      walk([&](int, float y) { amax = fmaxf(amax, fabsf(y)); });
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float scale = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
      uint8_t* dst = static_cast<uint8_t*>(is_v ? p.v_cache : p.k_cache) + at;
      walk([&](int e, float y) { dst[e] = static_cast<uint8_t>(e4m3x2_from(__fdiv_rn(y, scale), 0.f) & 0xff); });
      if (lane == 0)
        (is_v ? p.v_scales : p.k_scales)[(slot / p.block_size * static_cast<int64_t>(p.num_kv_heads) + hk) *
                                             p.block_size + slot % p.block_size] = scale;
    }
  }
}

bool rope_aligned(const void* x, int64_t a) { return reinterpret_cast<uintptr_t>(x) % a == 0; }

int rope_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

template <typename T, bool INTER, bool F8, RopeAxes AXES>
cudaError_t launch_rope(const RopeParams& p, int64_t n, bool vec, cudaStream_t st) {
  const int heads = p.num_heads + 2 * p.num_kv_heads;
  const int64_t sms = rope_sms();
  if (!vec) {
    const int64_t need = (n * heads + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
    rope_cache_any_kernel<T, INTER, F8, AXES == kAxisRuns ? kAnyAxis : AXES>
        <<<static_cast<unsigned>(need < sms * 64 ? need : sms * 64), kRopeThreads, 0, st>>>(p, n);
    return cudaGetLastError();
  }
  const int lph = p.head_dim / 16;
  const int threads = kRopeThreads / lph * lph;  // <= kRopeThreads: head_dim is at most 16 kRopeThreads
  constexpr int kUnits = RopeShape<T, F8>::kUnits;
  const int rounds = (heads + threads / lph * kUnits - 1) / (threads / lph * kUnits);
  // all rounds side by side while the tokens alone leave SMs short of CTAs
  const int parts = n < sms * 8 ? (rounds < 65535 ? rounds : 65535) : 1;
  rope_cache_kernel<T, INTER, F8, AXES><<<dim3(static_cast<unsigned>(n), parts), threads, 0, st>>>(p, threads);
  return cudaGetLastError();
}

template <typename T, bool F8>
cudaError_t launch_rope_form(const RopeParams& p, int64_t n, bool vec, bool inter, cudaStream_t st) {
  // one axis: the single-position kernels, its row of positions being the only one
  if (p.num_axes <= 1)
    return inter ? launch_rope<T, true, F8, kOneAxis>(p, n, vec, st)
                 : launch_rope<T, false, F8, kOneAxis>(p, n, vec, st);
  if (p.axis_runs)
    return inter ? launch_rope<T, true, F8, kAxisRuns>(p, n, vec, st)
                 : launch_rope<T, false, F8, kAxisRuns>(p, n, vec, st);
  return inter ? launch_rope<T, true, F8, kAnyAxis>(p, n, vec, st)
               : launch_rope<T, false, F8, kAnyAxis>(p, n, vec, st);
}

// Checks shared by the entry points, then the launch.
int rope_impl(const RopeParams& in, int64_t num_tokens, int32_t interleaved, int64_t num_blocks, int dtype, bool f8,
              cudaStream_t st) {
  RopeParams p = in;
  if (num_tokens < 0 || num_tokens > INT32_MAX || p.num_heads < 0 || p.num_kv_heads <= 0 || p.head_dim <= 0 ||
      p.block_size <= 0 || num_blocks <= 0 || p.max_positions <= 0)
    return KV_ERR_INVALID_ARG;
  if (p.rot_dim <= 0 || p.rot_dim % 2 != 0 || p.rot_dim > p.head_dim) return KV_ERR_INVALID_ARG;
  if (p.num_heads > 65535 || p.num_kv_heads > 65535 || p.head_dim > 65535) return KV_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(p.num_heads) * p.head_dim;
  const int64_t kv_row = static_cast<int64_t>(p.num_kv_heads) * p.head_dim;
  if (q_row > INT32_MAX || kv_row > INT32_MAX) return KV_ERR_INVALID_ARG;
  if (p.k_stride < kv_row || p.v_stride < kv_row) return KV_ERR_INVALID_ARG;
  if (p.num_heads > 0 && (p.q_stride < q_row || p.q_out_stride < q_row)) return KV_ERR_INVALID_ARG;
  if (num_blocks > INT32_MAX / p.block_size) return KV_ERR_INVALID_ARG;
  p.num_slots = num_blocks * p.block_size;
  if (num_tokens == 0) return KV_OK;
  if (!p.k || !p.v || !p.positions || !p.cos_sin || !p.k_cache || !p.v_cache || !p.slot_mapping)
    return KV_ERR_INVALID_ARG;
  if (p.num_heads > 0 && (!p.q || !p.q_out)) return KV_ERR_INVALID_ARG;
  if (f8 && (!p.k_scales || !p.v_scales)) return KV_ERR_INVALID_ARG;
  const int64_t es = static_cast<int64_t>(dtype_bytes(dtype));
  if (p.num_heads > 0) {
    // rotating in place is token by token: the same rows, or none in common;
    // k and v are read while q_out is written
    if (p.q_out == p.q && p.q_out_stride != p.q_stride) return KV_ERR_INVALID_ARG;
    auto rows = [&](const void* x, int64_t row, int64_t stride) {
      return TokenRows{reinterpret_cast<uintptr_t>(x), row * es, stride * es};
    };
    const TokenRows qo = rows(p.q_out, q_row, p.q_out_stride);
    if ((p.q_out != p.q && rows_overlap(qo, rows(p.q, q_row, p.q_stride), num_tokens)) ||
        rows_overlap(qo, rows(p.k, kv_row, p.k_stride), num_tokens) ||
        rows_overlap(qo, rows(p.v, kv_row, p.v_stride), num_tokens))
      return KV_ERR_INVALID_ARG;
  }
  const void* elems[] = {p.num_heads ? p.q : p.k, p.num_heads ? p.q_out : p.k, p.k, p.v};
  for (const void* x : elems)
    if (!rope_aligned(x, es)) return KV_ERR_INVALID_ARG;
  if (!rope_aligned(p.k_cache, f8 ? 1 : es) || !rope_aligned(p.v_cache, f8 ? 1 : es) ||
      !rope_aligned(p.cos_sin, 4) || (f8 && (!rope_aligned(p.k_scales, 4) || !rope_aligned(p.v_scales, 4))))
    return KV_ERR_INVALID_ARG;
  // the vector kernel: whole 16-byte runs, and columns of 16 values
  bool vec = p.head_dim % 16 == 0 && p.rot_dim % 16 == 0 && p.head_dim <= 16 * kRopeThreads;
  for (const void* x : elems) vec = vec && rope_aligned(x, 16);
  vec = vec && rope_aligned(p.cos_sin, 16) && rope_aligned(p.k_cache, f8 ? 8 : 16) &&
        rope_aligned(p.v_cache, f8 ? 8 : 16);
  vec = vec && p.k_stride * es % 16 == 0 && p.v_stride * es % 16 == 0 &&
        (p.num_heads == 0 || (p.q_stride * es % 16 == 0 && p.q_out_stride * es % 16 == 0));
  const bool inter = interleaved != 0;
  cudaError_t e;
  if (f8) {
    e = dtype == KV_DTYPE_F16 ? launch_rope_form<__half, true>(p, num_tokens, vec, inter, st)
                              : launch_rope_form<__nv_bfloat16, true>(p, num_tokens, vec, inter, st);
  } else if (dtype == KV_DTYPE_F32) {
    e = launch_rope_form<float, false>(p, num_tokens, vec, inter, st);
  } else {
    e = dtype == KV_DTYPE_F16 ? launch_rope_form<__half, false>(p, num_tokens, vec, inter, st)
                              : launch_rope_form<__nv_bfloat16, false>(p, num_tokens, vec, inter, st);
  }
  return cuda_status(e);
}

// The axes of a call with several positions per token, checked, into `p`.
int rope_axes(RopeParams& p, int64_t num_tokens, int32_t num_axes, const uint8_t* pair_axes) {
  if (num_axes < 1 || num_axes > kRopeAxes) return KV_ERR_INVALID_ARG;
  if (p.rot_dim <= 0 || p.rot_dim % 2 != 0 || p.rot_dim / 2 > kRopeAxisPairs || !pair_axes) return KV_ERR_INVALID_ARG;
  p.num_tokens = num_tokens;
  p.num_axes = num_axes;
  p.axis_runs = 1;
  for (int i = 0; i < p.rot_dim / 2; ++i) {
    if (pair_axes[i] >= num_axes) return KV_ERR_INVALID_ARG;
    if (pair_axes[i] != pair_axes[i & ~7]) p.axis_runs = 0;
    p.axis_of_pair[i >> 5] |= static_cast<uint64_t>(pair_axes[i]) << (2 * (i & 31));
  }
  return KV_OK;
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_rope_and_cache(void* q_out, const void* q, const void* k, const void* v, const int32_t* positions,
                                    const float* cos_sin, void* k_cache, void* v_cache, const int32_t* slot_mapping,
                                    int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                    int32_t rot_dim, int64_t max_positions, int32_t interleaved, int32_t block_size,
                                    int64_t num_blocks, int64_t q_out_token_stride, int64_t q_token_stride,
                                    int64_t k_token_stride, int64_t v_token_stride, int dtype, void* stream) {
  if (dtype != KV_DTYPE_F32 && dtype != KV_DTYPE_F16 && dtype != KV_DTYPE_BF16) return KV_ERR_INVALID_ARG;
  const RopeParams p{q_out, q, k, v, positions, cos_sin, k_cache, v_cache, nullptr, nullptr, slot_mapping, num_heads,
                     num_kv_heads, head_dim, rot_dim, block_size, max_positions, 0, q_out_token_stride,
                     q_token_stride, k_token_stride, v_token_stride};
  return rope_impl(p, num_tokens, interleaved, num_blocks, dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" int paged_rope_and_cache_fp8(void* q_out, const void* q, const void* k, const void* v,
                                        const int32_t* positions, const float* cos_sin, void* k_cache, void* v_cache,
                                        float* k_scales, float* v_scales, const int32_t* slot_mapping,
                                        int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
                                        int32_t rot_dim, int64_t max_positions, int32_t interleaved,
                                        int32_t block_size, int64_t num_blocks, int64_t q_out_token_stride,
                                        int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                                        int dtype, void* stream) {
  if (dtype != KV_DTYPE_F16 && dtype != KV_DTYPE_BF16) return KV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KV_ERR_INVALID_ARG;
  const RopeParams p{q_out, q, k, v, positions, cos_sin, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_heads,
                     num_kv_heads, head_dim, rot_dim, block_size, max_positions, 0, q_out_token_stride,
                     q_token_stride, k_token_stride, v_token_stride};
  return rope_impl(p, num_tokens, interleaved, num_blocks, dtype, true, static_cast<cudaStream_t>(stream));
}

extern "C" int paged_rope_and_cache_axes(void* q_out, const void* q, const void* k, const void* v,
                                         const int32_t* positions, int32_t num_axes, const uint8_t* pair_axes,
                                         const float* cos_sin, void* k_cache, void* v_cache,
                                         const int32_t* slot_mapping, int64_t num_tokens, int32_t num_heads,
                                         int32_t num_kv_heads, int32_t head_dim, int32_t rot_dim,
                                         int64_t max_positions, int32_t interleaved, int32_t block_size,
                                         int64_t num_blocks, int64_t q_out_token_stride, int64_t q_token_stride,
                                         int64_t k_token_stride, int64_t v_token_stride, int dtype, void* stream) {
  if (dtype != KV_DTYPE_F32 && dtype != KV_DTYPE_F16 && dtype != KV_DTYPE_BF16) return KV_ERR_INVALID_ARG;
  RopeParams p{q_out, q, k, v, positions, cos_sin, k_cache, v_cache, nullptr, nullptr, slot_mapping, num_heads,
               num_kv_heads, head_dim, rot_dim, block_size, max_positions, 0, q_out_token_stride, q_token_stride,
               k_token_stride, v_token_stride};
  const int st = rope_axes(p, num_tokens, num_axes, pair_axes);
  if (st != KV_OK) return st;
  return rope_impl(p, num_tokens, interleaved, num_blocks, dtype, false, static_cast<cudaStream_t>(stream));
}

extern "C" int paged_rope_and_cache_axes_fp8(
    void* q_out, const void* q, const void* k, const void* v, const int32_t* positions, int32_t num_axes,
    const uint8_t* pair_axes, const float* cos_sin, void* k_cache, void* v_cache, float* k_scales, float* v_scales,
    const int32_t* slot_mapping, int64_t num_tokens, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t rot_dim, int64_t max_positions, int32_t interleaved, int32_t block_size, int64_t num_blocks,
    int64_t q_out_token_stride, int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int dtype,
    void* stream) {
  if (dtype != KV_DTYPE_F16 && dtype != KV_DTYPE_BF16) return KV_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return KV_ERR_INVALID_ARG;
  RopeParams p{q_out, q, k, v, positions, cos_sin, k_cache, v_cache, k_scales, v_scales, slot_mapping, num_heads,
               num_kv_heads, head_dim, rot_dim, block_size, max_positions, 0, q_out_token_stride, q_token_stride,
               k_token_stride, v_token_stride};
  const int st = rope_axes(p, num_tokens, num_axes, pair_axes);
  if (st != KV_OK) return st;
  return rope_impl(p, num_tokens, interleaved, num_blocks, dtype, true, static_cast<cudaStream_t>(stream));
}

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_rope_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
