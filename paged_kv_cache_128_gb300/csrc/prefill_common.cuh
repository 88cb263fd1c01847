// What the chunked-prefill kernels share: their arguments, the mma.sync kernel
// (any block size), and the tensor maps of the tcgen05 kernels.
#pragma once

#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "score_rules.cuh"
#include "tcgen05.cuh"

namespace pagedkv {
namespace {

constexpr int kPfWarps = 4;
constexpr int kPfRows = 16 * kPfWarps;  // query tokens (of one head) per CTA
constexpr int kPfKeys = 32;             // keys per shared-memory tile

struct PrefillParams {
  static constexpr bool kRules = false;
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* query_start;  // [B + 1]: sequence b's chunk tokens are rows query_start[b] ..
  int32_t num_seqs, num_heads, num_kv_heads, group, block_size;
  int64_t num_blocks;
  int32_t max_blocks_per_seq;
  float scale_log2;  // scale * log2(e)
  int64_t num_tokens;  // rows of q and out
  int32_t hg_log2;     // tensor-core kernel: log2 of the query heads per row tile
  int32_t row_tiles;   // tensor-core kernel: row tiles per (sequence, head group) in the grid
  int32_t test_skip;   // tensor-core kernel, test control (-1: off): CTA 0 never loads this K tile
};

// The same with score rules (score_rules.cuh).
struct RulesPrefillParams : PrefillParams {
  static constexpr bool kRules = true;
  ScoreRules rules;
  // tensor-core kernel: pieces that an item's keys may be cut into, how many
  // they are cut into, each piece's unnormalised outputs [splits][num_tokens
  // num_heads][D] and (reference, sum) of the weights (unused where one is most)
  int32_t splits;
  int32_t* ws_pieces;
  float* ws_o;
  float* ws_ml;
};

// Byte offset of (key, dim) in a [kPfKeys][D] 16-bit tile: 128-byte slabs of
// 64 dims, 16-byte chunks XOR-swizzled by key % 8 (conflict-free ldmatrix).
__device__ __forceinline__ uint32_t pf_off(int key, int d) {
  return static_cast<uint32_t>((d >> 6) * (kPfKeys * 128) + key * 128 + ((((d & 63) >> 3) ^ (key & 7)) << 4) +
                               (d & 7) * 2);
}

template <typename T, int D, typename Params>
__global__ void __launch_bounds__(kPfWarps * 32) prefill_kernel(const Params p) {
  using M = Mma<T>;
  constexpr int KS = D / 16;                 // k-steps of Q K^T over head_dim
  constexpr int kTile = kPfKeys * D * 2;     // bytes of one K or V tile
  constexpr int kChunks = kPfKeys * (D / 8);  // 16-byte chunks of one tile
  __shared__ __align__(1024) uint8_t sm[2][2][kTile];  // [stage][K, V]

  const int qt = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qs = __ldg(p.query_start + b), n = __ldg(p.query_start + b + 1) - qs;
  // rows past the grid's reach (a chunk longer than max_query_len) would be
  // left uncomputed: the last row tile of the sequence reports it
  if (qt == gridDim.x - 1 && h == 0 && tid == 0 && n > static_cast<int64_t>(gridDim.x) * kPfRows)
    record_error(KV_ERR_DEVICE_BOUNDS);
  if (n <= 0 || qt * kPfRows >= n) return;
  if (qs < 0 || qs + n > p.num_tokens) {  // the chunk's rows must lie inside q
    if (tid == 0) record_error(KV_ERR_DEVICE_BOUNDS);
    return;
  }
  int L = __ldg(p.seq_lens + b);
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  if (L < n || L > cap) {  // the chunk must lie inside the sequence and its table
    if (tid == 0) record_error(KV_ERR_DEVICE_BOUNDS);
    if (L > cap) L = static_cast<int>(cap);
    if (L < n) return;
  }
  const int ctx = L - n, kvh = h / p.group;
  const int g = lane >> 2, t2 = (lane & 3) * 2;
  const int row0 = qt * kPfRows + warp * 16;  // this warp's first chunk token
  const int64_t stride = static_cast<int64_t>(p.num_heads) * D;

  // Q as the A operand: rows row0 + g and row0 + g + 8, dims kk*16 + t2 (+1), + 8
  uint32_t qa[KS][4];
  {
    const T* qb = static_cast<const T*>(p.q) + static_cast<int64_t>(qs) * stride + static_cast<int64_t>(h) * D;
    const bool vlo = row0 + g < n, vhi = row0 + g + 8 < n;
    const T* qlo = qb + static_cast<int64_t>(row0 + g) * stride;
    const T* qhi = qlo + 8 * stride;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk) {
      const int d = kk * 16 + t2;
      qa[kk][0] = vlo ? __ldg(reinterpret_cast<const uint32_t*>(qlo + d)) : 0u;
      qa[kk][1] = vhi ? __ldg(reinterpret_cast<const uint32_t*>(qhi + d)) : 0u;
      qa[kk][2] = vlo ? __ldg(reinterpret_cast<const uint32_t*>(qlo + d + 8)) : 0u;
      qa[kk][3] = vhi ? __ldg(reinterpret_cast<const uint32_t*>(qhi + d + 8)) : 0u;
    }
  }
  const int pos_lo = ctx + row0 + g, pos_hi = pos_lo + 8;
  // keys the CTA needs: 0 .. position of its last row, or, with rules, what
  // its rows see; span_lo, span_hi: of this lane's two rows
  const int last_row = min(n, (qt + 1) * kPfRows) - 1;
  int first_key = 0, nkeys = ctx + last_row + 1;
  KeySpan span_lo{0, pos_lo + 1}, span_hi{0, pos_hi + 1};
  float slope = 0.f;  // times log2(e)
  // rules: the keys of tile kt that some row of warp w sees, [kt % 2][w] (a key
  // between the rows' intervals is not loaded, whatever its value holds)
  __shared__ uint32_t seen[2][kPfWarps];
  auto note_seen = [&](int kt) {
    const int k0 = kt * kPfKeys;
    static_assert(kPfKeys == 32, "a bit per key of a tile");
    const uint32_t mine = bits_between(span_lo.lo - k0, span_lo.hi - k0) | bits_between(span_hi.lo - k0, span_hi.hi - k0);
    const uint32_t all = __reduce_or_sync(0xffffffffu, mine);
    if (lane == 0) seen[kt & 1][warp] = all;
  };
  if constexpr (Params::kRules) {
    __shared__ int first, end;
    if (tid == 0) first = INT32_MAX, end = 0;
    __syncthreads();
    auto span_of = [&](int row) {
      const KeySpan s = row < n ? keys_seen(p.rules, static_cast<int64_t>(qs) + row, ctx + row, L) : KeySpan{0, 0};
      if (s.lo < s.hi) {
        atomicMin(&first, s.lo);
        atomicMax(&end, s.hi);
      }
      return s;
    };
    span_lo = span_of(row0 + g);
    span_hi = span_of(row0 + g + 8);
    __syncthreads();
    first_key = first;  // no row sees a key: no tile, rows of zeros
    nkeys = end;
    if (p.rules.slopes) slope = __ldg(p.rules.slopes + h) * kLog2e;
  }
  const int tile0 = first_key / kPfKeys;
  const int ntiles = (nkeys + kPfKeys - 1) / kPfKeys;
  if constexpr (Params::kRules) {
    if (tile0 < ntiles) {
      note_seen(tile0);
      note_seen(tile0 + 1);
    }
    __syncthreads();
  }

  auto load_tile = [&](int kt, int stage) {
    uint32_t keys = 0xffffffffu;
    if constexpr (Params::kRules) keys = seen[kt & 1][0] | seen[kt & 1][1] | seen[kt & 1][2] | seen[kt & 1][3];
    static_assert(kPfWarps == 4, "the words of every warp");
    for (int c = tid; c < 2 * kChunks; c += kPfWarps * 32) {
      const int which = c / kChunks, cc = c - which * kChunks;
      const int key = cc / (D / 8), d = (cc % (D / 8)) * 8;
      const int j = kt * kPfKeys + key;
      const bool valid = j < nkeys && (keys >> key & 1u);
      const T* src = static_cast<const T*>(which ? p.v_cache : p.k_cache);
      if (valid) {
        int pb = __ldg(p.block_tables + static_cast<int64_t>(b) * p.max_blocks_per_seq + j / p.block_size);
        if (pb < 0 || pb >= p.num_blocks) {
          record_error(KV_ERR_DEVICE_BOUNDS);
          pb = 0;
        }
        const int64_t row = static_cast<int64_t>(pb) * p.block_size + j % p.block_size;
        src += (row * p.num_kv_heads + kvh) * D + d;
      }
      cp_async16(smem_u32(&sm[stage][which][0]) + pf_off(key, d), src, valid);
    }
    cp_async_commit();
  };

  float o[D / 8][4];
#pragma unroll
  for (int i = 0; i < D / 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m_lo = -INFINITY, m_hi = -INFINITY, l_lo = 0.f, l_hi = 0.f;  // l: this lane's partial row sums
  // ldmatrix x4 lane -> matrix m = lane / 8, row lane % 8
  const int lm = lane >> 3, lr = lane & 7;

  if (tile0 < ntiles) load_tile(tile0, tile0 & 1);
  for (int kt = tile0; kt < ntiles; ++kt) {
    if (kt + 1 < ntiles) {
      load_tile(kt + 1, (kt + 1) & 1);
      cp_async_wait<1>();
    } else {
      cp_async_wait<0>();
    }
    __syncthreads();
    if constexpr (Params::kRules) note_seen(kt + 2);  // every warp has read this tile's words
    const uint32_t kb = smem_u32(&sm[kt & 1][0][0]), vb = smem_u32(&sm[kt & 1][1][0]);
    // S[16 rows x 32 keys] = Q K^T, four n8 blocks of keys
    float s[4][4];
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) s[nb][0] = s[nb][1] = s[nb][2] = s[nb][3] = 0.f;
#pragma unroll
    for (int kk = 0; kk < KS; ++kk)
#pragma unroll
      for (int nb = 0; nb < 4; nb += 2) {
        uint32_t r0, r1, r2, r3;  // (keys nb*8.., dims kk*16 + 0/8), (keys (nb+1)*8.., dims + 0/8)
        ldmatrix_x4(kb + pf_off((nb + (lm >> 1)) * 8 + lr, kk * 16 + (lm & 1) * 8), r0, r1, r2, r3);
        M::run(s[nb], qa[kk], r0, r1);
        M::run(s[nb + 1], qa[kk], r2, r3);
      }
    // mask keys past each row's position; online softmax in the exp2 domain
    float x[4][4];
    float mx_lo = -INFINITY, mx_hi = -INFINITY;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const int j = kt * kPfKeys + nb * 8 + t2;
      auto score = [&](float dot, const KeySpan& span, int pos, int key) {
        if constexpr (Params::kRules) {
          if (key < span.lo || key >= span.hi) return -INFINITY;
          const float v = p.rules.cap_log2 > 0.f ? soft_cap(dot, p.scale_log2, p.rules.cap_log2, p.rules.cap_arg)
                                                 : dot * p.scale_log2;
          return fmaf(-slope, fabsf(static_cast<float>(pos - key)), v);
        } else {
          return key <= pos ? dot * p.scale_log2 : -INFINITY;
        }
      };
      x[nb][0] = score(s[nb][0], span_lo, pos_lo, j);
      x[nb][1] = score(s[nb][1], span_lo, pos_lo, j + 1);
      x[nb][2] = score(s[nb][2], span_hi, pos_hi, j);
      x[nb][3] = score(s[nb][3], span_hi, pos_hi, j + 1);
      mx_lo = fmaxf(mx_lo, fmaxf(x[nb][0], x[nb][1]));
      mx_hi = fmaxf(mx_hi, fmaxf(x[nb][2], x[nb][3]));
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      mx_lo = fmaxf(mx_lo, __shfl_xor_sync(0xffffffffu, mx_lo, off));
      mx_hi = fmaxf(mx_hi, __shfl_xor_sync(0xffffffffu, mx_hi, off));
    }
    const float mn_lo = fmaxf(m_lo, mx_lo), mn_hi = fmaxf(m_hi, mx_hi);
    const float mu_lo = mn_lo == -INFINITY ? 0.f : mn_lo, mu_hi = mn_hi == -INFINITY ? 0.f : mn_hi;
    const float al_lo = fast_exp2(m_lo - mu_lo), al_hi = fast_exp2(m_hi - mu_hi);
    m_lo = mn_lo;
    m_hi = mn_hi;
    uint32_t pa[2][4];  // P as the A operand of two k16 steps over the 32 keys
    float sum_lo = 0.f, sum_hi = 0.f;
#pragma unroll
    for (int nb = 0; nb < 4; ++nb) {
      const float p0 = fast_exp2(x[nb][0] - mu_lo), p1 = fast_exp2(x[nb][1] - mu_lo);
      const float p2 = fast_exp2(x[nb][2] - mu_hi), p3 = fast_exp2(x[nb][3] - mu_hi);
      const uint32_t lo2 = M::pack(p0, p1), hi2 = M::pack(p2, p3);
      pa[nb >> 1][(nb & 1) * 2 + 0] = lo2;  // row g: a0 (keys 0-7 of the step) or a2 (keys 8-15)
      pa[nb >> 1][(nb & 1) * 2 + 1] = hi2;  // row g + 8: a1 or a3
      if constexpr (Params::kRules) {
        // the weights as rounded for the product: what the output is divided
        // by is then what it was built from, and their rounding cancels in part
        const float2 flo = M::unpack(lo2), fhi = M::unpack(hi2);
        sum_lo += flo.x + flo.y;
        sum_hi += fhi.x + fhi.y;
      } else {
        sum_lo += p0 + p1;
        sum_hi += p2 + p3;
      }
    }
    l_lo = l_lo * al_lo + sum_lo;
    l_hi = l_hi * al_hi + sum_hi;
#pragma unroll
    for (int i = 0; i < D / 8; ++i) {
      o[i][0] *= al_lo;
      o[i][1] *= al_lo;
      o[i][2] *= al_hi;
      o[i][3] *= al_hi;
    }
    // O[16 x D] += P V: V fragments by ldmatrix.trans, two n8 blocks of dims per x4
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
      for (int db = 0; db < D / 8; db += 2) {
        uint32_t r0, r1, r2, r3;  // (keys ks*16 + 0/8, dims db*8..), (same keys, dims (db+1)*8..)
        ldmatrix_x4_trans(vb + pf_off(ks * 16 + (lm & 1) * 8 + lr, (db + (lm >> 1)) * 8), r0, r1, r2, r3);
        M::run(o[db], pa[ks], r0, r1);
        M::run(o[db + 1], pa[ks], r2, r3);
      }
    __syncthreads();  // every warp is done with this stage before it is loaded again
  }
  // row sums over the quad, normalise, one rounding to the output type
#pragma unroll
  for (int off = 1; off < 4; off <<= 1) {
    l_lo += __shfl_xor_sync(0xffffffffu, l_lo, off);
    l_hi += __shfl_xor_sync(0xffffffffu, l_hi, off);
  }
  const float inv_lo = l_lo > 0.f ? 1.f / l_lo : 0.f, inv_hi = l_hi > 0.f ? 1.f / l_hi : 0.f;
  T* ob = static_cast<T*>(p.out) + static_cast<int64_t>(qs) * stride + static_cast<int64_t>(h) * D;
  const bool vlo = row0 + g < n, vhi = row0 + g + 8 < n;
#pragma unroll
  for (int db = 0; db < D / 8; ++db) {
    const int d = db * 8 + t2;
    if (vlo)
      *reinterpret_cast<uint32_t*>(ob + static_cast<int64_t>(row0 + g) * stride + d) =
          M::pack(o[db][0] * inv_lo, o[db][1] * inv_lo);
    if (vhi)
      *reinterpret_cast<uint32_t*>(ob + static_cast<int64_t>(row0 + g + 8) * stride + d) =
          M::pack(o[db][2] * inv_hi, o[db][3] * inv_hi);
  }
}

template <typename T, typename P>
cudaError_t launch_prefill(const P& p, int head_dim, int max_query_len, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(max_query_len) + kPfRows - 1) / kPfRows), p.num_heads,
                  p.num_seqs);
  if (head_dim == 64) prefill_kernel<T, 64, P><<<grid, kPfWarps * 32, 0, st>>>(p);
  else prefill_kernel<T, 128, P><<<grid, kPfWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

// tcgen05 kernels
constexpr int kTcRows = 128;                      // MMA M: rows of a query tile
constexpr int kTcKeys = 128;                      // keys per tile: N of S, K of P V

PFN_cuTensorMapEncodeTiled_v12000 tc_encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  });
  return fn;
}

// A 3-D tensor {n0, n1, n2} of 16-bit elements (dim 0 contiguous, dim 1
// `n0` apart, dim 2 `n0 * n1` apart) with 128-byte-swizzled boxes
// {64, box1, box2}.  Encoded maps are kept in a small table keyed by all the
// arguments, so a caller that reuses its buffers pays the encoding once.
bool tc_map(const void* base, int64_t n0, int64_t n1, int64_t n2, int box1, int box2, CUtensorMap* out) {
  struct Key {
    const void* base;
    int64_t n0, n1, n2;
    int box1, box2;
    bool operator==(const Key& o) const {
      return base == o.base && n0 == o.n0 && n1 == o.n1 && n2 == o.n2 && box1 == o.box1 && box2 == o.box2;
    }
  };
  constexpr int kSlots = 32;
  static std::mutex mu;
  static Key keys[kSlots];
  static CUtensorMap maps[kSlots];
  static int used = 0, next = 0;
  const Key key{base, n0, n1, n2, box1, box2};
  std::lock_guard<std::mutex> lock(mu);
  for (int i = 0; i < used; ++i)
    if (keys[i] == key) {
      *out = maps[i];
      return true;
    }
  auto fn = tc_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(n0) * 2, static_cast<cuuint64_t>(n0 * n1) * 2};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)};
  cuuint32_t estr[3] = {1, 1, 1};
  CUtensorMap m;
  if (fn(&m, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(base), dims, strides, box, estr,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return false;
  const int slot = used < kSlots ? used++ : (next++ % kSlots);
  keys[slot] = key;
  maps[slot] = m;
  *out = m;
  return true;
}

bool tc_supported(int block_size) { return block_size >= 16 && block_size % 16 == 0 && kTcKeys % block_size == 0; }

bool aligned16(const void* x) { return (reinterpret_cast<uintptr_t>(x) & 15u) == 0; }

// Rows of the longest chunk: what the caller allows for, and no more than q
// has (the largest int32 says "no limit"; grids and reaches go by this).
int32_t longest_chunk(int32_t max_query_len, int64_t num_query_tokens) {
  return static_cast<int32_t>(std::min<int64_t>(max_query_len, num_query_tokens));
}

// A call's arguments, checked, as kernel parameters (num_seqs 0: nothing to do).
int prefill_params(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* seq_lens, const int32_t* query_start_loc, int64_t num_query_tokens, int32_t num_seqs,
                   int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
                   int32_t max_blocks_per_seq, int32_t max_query_len, float scale, int dtype, PrefillParams* params) {
  if (dtype != KV_DTYPE_F16 && dtype != KV_DTYPE_BF16) return KV_ERR_INVALID_ARG;
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 || block_size <= 0 ||
      num_blocks <= 0 || max_blocks_per_seq <= 0 || max_query_len < 0 || (head_dim != 64 && head_dim != 128))
    return KV_ERR_INVALID_ARG;
  if (num_blocks > INT32_MAX / block_size || num_heads > 65535 || num_seqs > 65535) return KV_ERR_INVALID_ARG;
  if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return KV_ERR_INVALID_ARG;
  if (num_query_tokens < 0 || num_query_tokens > INT32_MAX) return KV_ERR_INVALID_ARG;
  if (num_seqs == 0 || max_query_len == 0 || num_query_tokens == 0) return KV_OK;  // nothing to do: params->num_seqs stays 0
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens || !query_start_loc) return KV_ERR_INVALID_ARG;
  if (!aligned16(out) || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache)) return KV_ERR_INVALID_ARG;
  PrefillParams& p = *params;
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_start = query_start_loc;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.block_size = block_size;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.num_tokens = num_query_tokens;
  return KV_OK;
}

}  // namespace
}  // namespace pagedkv
