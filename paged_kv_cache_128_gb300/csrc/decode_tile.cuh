// Decode attention over one tile of a sequence's tokens by one warp, on
// mma.sync: the tile layout that TMA writes, the warp's online-softmax state,
// and the step that takes a tile into it.
#pragma once

#include "common.cuh"

namespace pagedkv {

// =========================================================================
// Tensor-core path: shared consumer math.
//
// Each consumer warp owns whole tiles (one physical block of one kv head,
// BS tokens) and keeps its own online-softmax state for the current unit
// (sequence, kv head).  Per 16-token sub-tile:
//   S^T[16 tok x 8*NG heads] = K[16 x D] Q^T          (mma m16n8k16, fp32 acc)
//   softmax update in the exp2 domain, P^T packed to the MMA type,
//   movmatrix turns the P^T accumulator fragment into a B operand,
//   O^T[D x 8*NG] += V^T[D x 16] P^T                   (V^T via ldmatrix.trans)
// =========================================================================

template <int D, int BS>
struct Tile {
  static constexpr int kSub = D / 64;              // 128-byte column slabs per row
  static constexpr int kSlabBytes = BS * 128;      // one slab of one tile
  static constexpr int kTileBytes = BS * D * 2;    // K or V of one block, one kv head
  static constexpr int kStageBytes = 2 * kTileBytes;
  static_assert(D % 64 == 0, "head_dim must be a multiple of 64");
  static_assert(BS % 16 == 0, "block_size must be a multiple of 16");
  static_assert(kSlabBytes % 1024 == 0, "slabs must keep 1024-byte swizzle alignment");
};

// Byte offset of element (row t, column d) inside a tile written by TMA with
// 128-byte swizzle.  The tile holds whole physical blocks of PB rows, block
// by block; inside a block, 64-column slab by slab (PB rows of 128 bytes
// each); inside a row, 16-byte chunk (d%64)/8 XOR (t%8) (PB is a multiple of
// 8, so a row's swizzle phase is t % 8 wherever its block sits).
template <int D, int PB>
__device__ __forceinline__ uint32_t swz(int t, int d) {
  return static_cast<uint32_t>(((t / PB) * (D / 64) + (d >> 6)) * (PB * 128) + (t % PB) * 128 +
                               ((((d & 63) >> 3) ^ (t & 7)) << 4));
}

template <int D, int NG>
struct WarpState {
  static constexpr int KS = D / 16;  // k-steps of S^T = K Q^T, and m-tiles of O^T
  uint32_t qf[KS][NG][2];            // Q^T as B operand
  float acc[KS][NG][4];              // O^T accumulator fragments
  float m[NG][2], l[NG][2];          // running max (exp2 domain) and sum, 2 heads per lane
};

// B operand of S^T = K Q^T: b0 = Q[g][kk*16 + 2*(lane%4) + {0,1}], b1 at d + 8,
// g = ng*8 + lane/4; heads past G are zero.
template <typename T, int D, int NG>
__device__ __forceinline__ void load_q_frags(uint32_t (&qf)[D / 16][NG][2], const T* qb, int G, int lane) {
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    const int g = ng * 8 + (lane >> 2);
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
      const int d = kk * 16 + (lane & 3) * 2;
      if (g < G) {
        qf[kk][ng][0] = __ldg(reinterpret_cast<const uint32_t*>(qb + g * D + d));
        qf[kk][ng][1] = __ldg(reinterpret_cast<const uint32_t*>(qb + g * D + d + 8));
      } else {
        qf[kk][ng][0] = 0u;
        qf[kk][ng][1] = 0u;
      }
    }
  }
}

template <typename T, int D, int NG>
__device__ __forceinline__ void load_q(WarpState<D, NG>& st, const T* qb, int G, int lane) {
  load_q_frags<T, D, NG>(st.qf, qb, G, lane);
}

template <int D, int NG>
__device__ __forceinline__ void reset_state(WarpState<D, NG>& st) {
#pragma unroll
  for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
      for (int e = 0; e < 4; ++e) st.acc[mt][ng][e] = 0.f;
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    st.m[ng][0] = st.m[ng][1] = -INFINITY;
    st.l[ng][0] = st.l[ng][1] = 0.f;
  }
}

// Accumulate NS 16-token sub-tiles (tokens tok0 .. tok0 + 16 * NS - 1) of
// one tile held in shared memory at kt_a (K) and vt_a (V) as one step of the
// online softmax: the score chains of the sub-tiles are interleaved, and
// the running max, the rescale of the accumulator and l are updated once.
template <typename T, int D, int PB, int NG, int NS>
__device__ __forceinline__ void consume_subtiles(WarpState<D, NG>& st, uint32_t kt_a, uint32_t vt_a, int tok0, int L,
                                                 float sl2, int lane) {
  using M = Mma<T>;
  constexpr int KS = D / 16;
  // ldmatrix lane -> (row, column) of the 8x8 matrix it addresses
  const int k_row = (lane & 7) + ((lane >> 3) & 1) * 8, k_col = (lane >> 4) * 8;  // A = K (non-trans)
  const int v_row = (lane & 7) + (lane >> 4) * 8, v_col = ((lane >> 3) & 1) * 8;  // A = V^T (trans)
  float sc[NS][NG][4];
#pragma unroll
  for (int u = 0; u < NS; ++u)
#pragma unroll
    for (int ng = 0; ng < NG; ++ng) sc[u][ng][0] = sc[u][ng][1] = sc[u][ng][2] = sc[u][ng][3] = 0.f;
#pragma unroll
  for (int kk = 0; kk < KS; ++kk) {
    uint32_t a[NS][4];
#pragma unroll
    for (int u = 0; u < NS; ++u)
      ldmatrix_x4(kt_a + swz<D, PB>(u * 16 + k_row, kk * 16 + k_col), a[u][0], a[u][1], a[u][2], a[u][3]);
#pragma unroll
    for (int u = 0; u < NS; ++u)
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) M::run(sc[u][ng], a[u], st.qf[kk][ng][0], st.qf[kk][ng][1]);
  }
  uint32_t pb[NS][NG][2];
#pragma unroll
  for (int ng = 0; ng < NG; ++ng) {
    // scores in the exp2 domain; rows past the sequence end are -inf
    float x[NS][4];
    float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      const int t_lo = tok0 + u * 16 + (lane >> 2);
      const bool in_lo = t_lo < L, in_hi = t_lo + 8 < L;
      x[u][0] = in_lo ? sc[u][ng][0] * sl2 : -INFINITY;
      x[u][1] = in_lo ? sc[u][ng][1] * sl2 : -INFINITY;
      x[u][2] = in_hi ? sc[u][ng][2] * sl2 : -INFINITY;
      x[u][3] = in_hi ? sc[u][ng][3] * sl2 : -INFINITY;
      mx0 = fmaxf(mx0, fmaxf(x[u][0], x[u][2]));
      mx1 = fmaxf(mx1, fmaxf(x[u][1], x[u][3]));
    }
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, off));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, off));
    }
    const float mn0 = fmaxf(st.m[ng][0], mx0), mn1 = fmaxf(st.m[ng][1], mx1);
    const float mu0 = (mn0 == -INFINITY) ? 0.f : mn0, mu1 = (mn1 == -INFINITY) ? 0.f : mn1;
    const float al0 = fast_exp2(st.m[ng][0] - mu0), al1 = fast_exp2(st.m[ng][1] - mu1);
    float s0 = 0.f, s1 = 0.f;
#pragma unroll
    for (int u = 0; u < NS; ++u) {
      // l sums the probabilities as rounded for the PV product
      const uint32_t lo = M::pack(fast_exp2(x[u][0] - mu0), fast_exp2(x[u][1] - mu1));
      const uint32_t hi = M::pack(fast_exp2(x[u][2] - mu0), fast_exp2(x[u][3] - mu1));
      const float2 flo = M::unpack(lo), fhi = M::unpack(hi);
      s0 += flo.x + fhi.x;
      s1 += flo.y + fhi.y;
      pb[u][ng][0] = movmatrix_trans(lo);
      pb[u][ng][1] = movmatrix_trans(hi);
    }
    st.l[ng][0] = st.l[ng][0] * al0 + s0;
    st.l[ng][1] = st.l[ng][1] * al1 + s1;
    st.m[ng][0] = mn0;
    st.m[ng][1] = mn1;
#pragma unroll
    for (int mt = 0; mt < KS; ++mt) {
      st.acc[mt][ng][0] *= al0;
      st.acc[mt][ng][1] *= al1;
      st.acc[mt][ng][2] *= al0;
      st.acc[mt][ng][3] *= al1;
    }
  }
#pragma unroll
  for (int mt = 0; mt < KS; ++mt) {
    uint32_t a[NS][4];
#pragma unroll
    for (int u = 0; u < NS; ++u)
      ldmatrix_x4_trans(vt_a + swz<D, PB>(u * 16 + v_row, mt * 16 + v_col), a[u][0], a[u][1], a[u][2], a[u][3]);
#pragma unroll
    for (int u = 0; u < NS; ++u)
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) M::run(st.acc[mt][ng], a[u], pb[u][ng][0], pb[u][ng][1]);
  }
}

// Accumulate one tile (tokens tok0 .. tok0 + BS - 1 of a sequence of length
// L) held in shared memory at kt (K) and vt (V).  Sub-tiles wholly past the
// sequence end are skipped.
// BS: tokens of the tile; PB: rows of each physical block in it (the tile's
// layout, see swz).
template <typename T, int D, int BS, int NG, int PB = BS>
__device__ __forceinline__ void consume_tile(WarpState<D, NG>& st, uint8_t* kt, uint8_t* vt, int tok0, int L,
                                             float sl2, int lane) {
  const int valid = min(BS, L - tok0);
  if (valid < BS) {
    // zero the V rows past the sequence end: P is 0 there, but 0 * NaN is not
    const int chunks = (BS - valid) * (D / 8);
    for (int c = lane; c < chunks; c += 32) {
      const int t = valid + c / (D / 8), d = (c % (D / 8)) * 8;
      *reinterpret_cast<uint4*>(vt + swz<D, PB>(t, d)) = make_uint4(0u, 0u, 0u, 0u);
    }
    fence_proxy_async_smem();  // these bytes are TMA-written again later
    __syncwarp();
  }
  const uint32_t kt_a = smem_u32(kt), vt_a = smem_u32(vt);
  if constexpr (BS == 32) {
    if (valid > 16) consume_subtiles<T, D, PB, NG, 2>(st, kt_a, vt_a, tok0, L, sl2, lane);
    else consume_subtiles<T, D, PB, NG, 1>(st, kt_a, vt_a, tok0, L, sl2, lane);
  } else {
    static_assert(BS == 16, "tiles are 16 or 32 tokens");
    consume_subtiles<T, D, PB, NG, 1>(st, kt_a, vt_a, tok0, L, sl2, lane);
  }
}

}  // namespace pagedkv
