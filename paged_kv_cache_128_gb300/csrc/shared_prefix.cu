// Decode attention for groups of sequences that share a prefix.
//
// Sequence b of group g (consecutive sequences of the batch) has its first
// P_g tokens in the blocks that the group's first sequence has them in
// ("paged-attention-impl-detail", section Copy-on-Write共享).  Its output is
// plain decode attention ("MiniPaged-Qwen" §13, §14),
//   out[b, qh] = sum_{j < L_b} softmax_j(scale * q[b, qh] . K_j) V_j,
// and the softmax splits over keys (§17.3): with m, l, o the running max, sum
// and unnormalised output of a range of keys,
//   out = (e^{m1 - m} o1 + e^{m2 - m} o2) / (e^{m1 - m} l1 + e^{m2 - m} l2).
// So the work falls into units of two kinds, each a set of query rows against
// a range of keys of one kv head:
//   prefix unit (group, row tile, kv head): the G query heads of up to
//     128 / G sequences of the group against keys 0 .. P_g - 1, which are
//     read once for all of them: matrix products with 128 rows;
//   rest unit (sequence, kv head): G rows against keys P_g .. L_b - 1: the
//     few rows of ordinary decode attention.
//
// What bounds it: every group's prefix and every sequence's rest are read
// once (a second row tile of a group finds the prefix in L2), 4 D flops per
// query row and key; memory until about 280 query rows share each key, then
// the tensor cores.
//
// Partition.  The prefix units in order (group; kv head; row tile) lie on one
// line, each a fixed charge followed by its 64-key tiles, the rest units
// (sequence; kv head) on another, each a charge and its 16-token tiles.  The
// first CTAs of one wave (two per SM) share the first line, the warps of the
// others the second one, in equal lengths, and the number of CTAs on each
// side follows the lines' weights; so a unit is cut only where a share ends.
// A rest unit of a sequence without prefix that falls whole into one warp's
// share is written to `out`; every other piece writes (o, m, l) in float32 to
// the workspace, and shared_merge_kernel joins a row's pieces in their order
// along the lines, so results do not depend on timing.  Every CTA rebuilds
// the lines from group_start, prefix_lens and seq_lens in shared memory;
// nothing in the workspace outlives the call.
//
// A prefix CTA is the tcgen05 pipeline of the chunked prefill, at 64 keys a
// tile and with two score buffers:
//   warp 5: TMA: K and V tiles through the block table into one ring of
//     stages, K_0 K_1 V_0 K_2 V_1 ..., across unit boundaries;
//   warp 4: one lane issues the MMAs, M 128: S = Q K^T (N 64) into one of two
//     buffers, so that the next tile's scores are made while the softmax is at
//     the last one's, and O += P V (N D) with P from tensor memory;
//   warps 0-3: softmax, one query row per thread, as in the prefill: P, the
//     sum and O are relative to a reference that moves only when a tile's
//     maximum passes it by far; warps without a row of the unit skip the
//     arithmetic.  They also lay a unit's Q into shared memory (any G: the
//     rows are gathered) and write its results.
// P is rounded to the cache's 16-bit type, on both lines and as in the other
// attention kernels: the tensor cores take both operands of P V in one type.
// The sum is taken over the rounded P, so a rounding moves a result by at most
// u sum_j p_j |V_j - out| (u 2^-8 in bf16, 2^-11 in fp16).  Scores, sums, O and
// the pieces are float32.
// In a rest CTA each of warps 0-3 works by itself: its own ring of 16-token
// tiles, its own copies, the decode kernels' mma.sync step (tokens in M, heads
// in N) and its unit's whole softmax state in registers, so that a unit of a
// few tokens costs no exchange between warps.  (Rest units through the
// tcgen05 pipeline cost 3.3 us each at one 64-key tile, with 5 of 128 rows
// in use.)
//
// Measured on the device (bf16, 32 query heads on 8 kv heads of 128; beside
// it paged_decode_attention, which reads the prefix for every sequence):
//   64 sequences, prefix 4096, rests up to 1024: 29 us, 75 MB (125 us);
//   7 sequences, prefix 32768, rests up to 300: 34 us, 135 MB (128 us);
//   256 sequences, prefix 8192, rests up to 512: 70 us, 131 MB, 35 GFLOP (740 us).
// Time stamps in a copy of the kernel: the lines are built after 2.0 us (4
// sequences) to 3.0 (256); the first scores are there after 3.9 to 7.4; the
// last CTA's end is followed by 4 to 7 us of launch and merge.  So 8 of the
// smallest call's 9.6 us (4 sequences of 512) and 12.5 to 13.5 us of the others
// lie before the first tile and after the last.  A prefix CTA, two to an SM,
// takes a tile in 1.16 us (256 sequences) to 1.4 (7, whose 16-token blocks take
// four copies a tile).
// Of the 70 us of 256 sequences, 6.6 go by before the first scores, 46 on 38 to
// 42 tiles a CTA (0.8 PFLOP/s on the 113 SMs of the prefix line), 9 between the
// median CTA's end (55 us, on both lines) and the last one's, and the rest after
// it.  In those tiles an SM's tensor pipe is busy for 0.33 of 0.58 us (N 64: 48
// clocks for 16 dims where N 128 takes 64); neither L2 (22 %) nor memory (27 %)
// is near its limit.
// Slower than paged_decode_attention where the rests are most of what is read:
// 64 sequences, prefix 128, rests 1024 to 2048, 79 against 70 us; prefix 2048,
// rests 2048 to 4096, 165 against 160; nothing shared, 512 tokens each, 28
// against 27.
// Slower in part of the cases, so not taken: one CTA per SM whose K and V
// stages serve two row tiles (31 / 41 / 74 us: its one issuing lane sets the
// pace); a fifth stage (30 / 37 / 71 us).

#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "decode_tile.cuh"
#include "tcgen05.cuh"

namespace pagedkv {
namespace {

constexpr int kSpRows = 128;   // MMA M: query rows of a prefix unit
constexpr int kSpKeys = 64;    // keys per prefix tile: N of S, K of P V
constexpr int kSpSoftWarps = 4;
constexpr int kSpMmaWarp = kSpSoftWarps, kSpTmaWarp = kSpSoftWarps + 1;
constexpr int kSpThreads = 32 * (kSpSoftWarps + 2);
constexpr uint32_t kSpCols = 256;  // S buffers at columns 0 and 64 (P over the first half of each), O at 128
// At least three stages: a thread that waits for a tile's V then knows that
// what the stage held before has landed (with two, and units of one tile, it
// would be the V of the tile before, whose P V may not have run), so its
// parity wait is one phase behind at most.
constexpr int kSpMinStages = 3, kSpMaxStages = 8;
constexpr int kSpMaxSeqs = 4096;
constexpr int kSpMaxGroup = 16;  // query heads per kv head: rows of a rest unit (two n8 blocks)
constexpr int kSpTok = 16;       // tokens per rest tile
constexpr int kSpMaxRest = 6;    // stages of a warp's ring of rest tiles
// Charges, in tiles of the unit's line, for what a unit costs beyond its
// tiles, and the weight of a prefix tile against a rest tile.
constexpr int kSpPrefixCost = 3, kSpRestCost = 2;
constexpr int kSpPrefixWeight = 4, kSpRestWeight = 1;

struct SpParams {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* seq_lens;
  const int32_t* group_start;
  const int32_t* prefix_lens;
  int32_t num_seqs, num_groups, num_heads, num_kv_heads, group, block_size, tile_seqs;
  int64_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t stages, rest_stages;
  float scale_log2;  // scale * log2(e)
  int32_t num_sms, num_ctas;
  int32_t test_skip;  // test control (-1: off): the prefix line's first share never loads this copy
  // workspace
  float* unit_o;   // [2][B][Hq][D] whole units: prefix, rest
  float* unit_ml;  // [2][B][Hq][2] (reference, sum)
  float* pre_o;    // [CTA][2][kSpRows][D] pieces of prefix units cut by a CTA's share: its first, its last
  float* pre_ml;   // [CTA][2][kSpRows][2]
  float* rest_o;   // [warp][2][G][D] the same of rest units and a warp's share
  float* rest_ml;  // [warp][2][G][2]
  int4* pre_span;   // [B][Hkv] first and last share of the sequence's prefix unit, its first row there
  int4* rest_span;  // [B][Hkv] first and last share of its rest unit
  int2* seq;        // [B] (tokens taken from the prefix unit, length)
};

template <int D>
struct SpLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr int kQSlab = kSpRows * 128;  // 64 dims of the 128 rows
  static constexpr int kQ = kSlabs * kQSlab;
  static constexpr int kAtom = 8 * 128;           // 64 dims of 8 keys
  static constexpr int kEight = kSlabs * kAtom;   // 8 keys of a K or V tile, slab by slab
  static constexpr int kTile = kSpKeys / 8 * kEight;
  static constexpr int kRestTile = kSpTok * D * 2;  // K or V of a rest tile
  static constexpr int kBars = 8 * (2 * kSpMaxStages + 9 + kSpSoftWarps * kSpMaxRest) + 56;
  // a rest CTA uses the bytes of Q and the stages for its warps' rings
  static int rest_stages(int stages) {
    return std::min(kSpMaxRest, (kQ + stages * kTile) / (kSpSoftWarps * 2 * kRestTile));
  }
  static int bytes(int stages, int num_seqs, int num_groups) {
    return 1024 + kQ + stages * kTile + kBars + 4 * (3 * num_seqs + 3 * num_groups + 3);
  }
};

// The lines of units, in shared memory.
struct SpLine {
  int* pre;     // [groups + 1] prefix line: cost per kv head before each group
  int* rest;    // [seqs + 1] rest line: cost per kv head before each sequence
  int* start;   // [groups + 1] group_start
  int* prefix;  // [groups] tokens of the group's prefix that are shared (whole blocks)
  int* first;   // [seqs] tokens the sequence takes from its group's prefix unit
  int* len;     // [seqs]
};

// The last entity of a line (cost prefix sums cum[0..n]) that begins at or
// before place x < hkv cum[n]; it is not empty.
__device__ __forceinline__ int sp_entity(const int* cum, int n, int hkv, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (hkv * cum[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// A line of length W cut into `shares` parts of W / shares places, the first
// W mod shares of them one longer (the host has checked that places fit an
// int).
struct SpCut {
  int shares, q, r;
  __device__ __forceinline__ SpCut(int W, int most) : shares(min(W, most)), q(W / shares), r(W - q * shares) {}
  __device__ __forceinline__ int begin(int s) const { return s * q + min(s, r); }
  __device__ __forceinline__ int of(int place) const {  // the share that holds a place
    const int longer = r * (q + 1);
    return place < longer ? place / (q + 1) : r + (place - longer) / q;
  }
};

// Prefix units of a share of the prefix line, in order.
struct SpPrefixWalk {
  const SpParams& p;
  const SpLine& ln;
  int x, x1, base;  // place reached, the share's end, the unit's place
  int e, u, cs, row_tiles, n;  // group, unit in it, a unit's cost, row tiles, sequences
  // the unit; lead: the group's first sequence, whose table row holds the prefix (b0, the row tile's first, may
  // be shorter than the prefix, or empty, and its row another)
  int b0, lead, rows, kvh, keys, t0, t1, T;
  int at;

  __device__ __forceinline__ SpPrefixWalk(const SpParams& p_, const SpLine& ln_, int x0, int x1_)
      : p(p_), ln(ln_), x(x0), x1(x1_) {
    enter(sp_entity(ln.pre, p.num_groups, p.num_kv_heads, x));
    u = (x - base) / cs;
    base += u * cs;
  }
  __device__ __forceinline__ void enter(int g) {
    e = g;
    u = 0;
    n = ln.start[g + 1] - ln.start[g];
    row_tiles = (n + p.tile_seqs - 1) / p.tile_seqs;
    cs = (ln.pre[g + 1] - ln.pre[g]) / row_tiles;
    base = p.num_kv_heads * ln.pre[g];
  }
  // To the next unit with a tile in the share; false when there is none.
  __device__ __forceinline__ bool next() {
    while (x < x1) {
      T = cs - kSpPrefixCost;
      t0 = max(0, x - base - kSpPrefixCost);
      t1 = min(T, x1 - base - kSpPrefixCost);
      at = base;
      kvh = u / row_tiles;
      const int rt = u - kvh * row_tiles;
      lead = ln.start[e];
      b0 = lead + rt * p.tile_seqs;
      rows = min(p.tile_seqs, n - rt * p.tile_seqs) * p.group;
      keys = ln.prefix[e];
      base += cs;
      x = base;
      if (++u == p.num_kv_heads * row_tiles && x < x1) {
        int g = e + 1;
        while (ln.pre[g + 1] == ln.pre[g]) ++g;  // x < x1: a group with units follows
        enter(g);
      }
      if (t1 > t0) return true;
    }
    return false;
  }
};

// Tiles of a share of the rest line, in order: tile t of unit (b, kvh).
struct SpRestWalk {
  int b, kvh, t, t0, t1, T, first, len;
  int base, x1;

  __device__ __forceinline__ void enter(const SpLine& ln, int b_) {
    b = b_;
    T = ln.rest[b + 1] - ln.rest[b] - kSpRestCost;
    first = ln.first[b];
    len = ln.len[b];
  }
  __device__ __forceinline__ bool span(int x) {  // tiles of the unit from place x on
    t0 = max(0, x - base - kSpRestCost);
    t1 = min(T, x1 - base - kSpRestCost);
    t = t0;
    return t0 < t1;
  }
  __device__ __forceinline__ bool begin(const SpParams& p, const SpLine& ln, int x0, int x1_) {
    x1 = x1_;
    if (x0 >= x1) return false;
    enter(ln, sp_entity(ln.rest, p.num_seqs, p.num_kv_heads, x0));
    base = p.num_kv_heads * ln.rest[b];
    kvh = (x0 - base) / (T + kSpRestCost);
    base += kvh * (T + kSpRestCost);
    return span(x0) || next_unit(p, ln);
  }
  __device__ __forceinline__ bool next_unit(const SpParams& p, const SpLine& ln) {
    base += T + kSpRestCost;
    if (base + kSpRestCost >= x1) return false;  // its first tile is another share's
    if (++kvh == p.num_kv_heads) {
      kvh = 0;
      int n = b + 1;
      while (ln.rest[n + 1] == ln.rest[n]) ++n;  // base < x1: a sequence with a rest follows
      enter(ln, n);
    }
    return span(base);
  }
  __device__ __forceinline__ bool next(const SpParams& p, const SpLine& ln) {
    return ++t < t1 || next_unit(p, ln);
  }
};

// Where 16-byte chunk c of row r of a prefix unit lies within the row in the
// workspace: moved so that eight rows' chunks fall into different banks when
// the rows are laid into shared memory for a bulk store.
__device__ __forceinline__ int sp_chunk(int c, int r) { return c ^ (r & 7); }

// Bulk store of contiguous shared memory, both ends 16-byte aligned.
__device__ __forceinline__ void bulk_store(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_store_wait() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group 0;" ::: "memory");
}

// One warp's share of the rest line.
template <typename T, int D, int NG>
__device__ __forceinline__ void rest_warp(const SpParams& p, const SpLine& ln, const CUtensorMap& tmK,
                                          const CUtensorMap& tmV, uint8_t* ring, uint64_t* full, const SpCut& cut,
                                          int share, int lane) {
  constexpr int kRestTile = SpLayout<D>::kRestTile;
  const int G = p.group, bs = p.block_size, nst = p.rest_stages;
  const int x0 = cut.begin(share), x1 = cut.begin(share + 1);
  SpRestWalk iw, cw;  // where the copies are, where the arithmetic is
  bool imore = iw.begin(p, ln, x0, x1);
  bool more = cw.begin(p, ln, x0, x1);
  // Table entries are fetched 32 at a time, one per lane, and the chunk the
  // walk is likely to need next is fetched along.
  auto fetch = [&](int b, int chunk) -> int {
    const int e = (chunk << 5) + lane;
    return e < p.max_blocks_per_seq ? p.block_tables[static_cast<int64_t>(b) * p.max_blocks_per_seq + e] : 0;
  };
  int have_b = -1, have_c = -1, mine = 0, next_b = -1, next_c = -1, nxt = 0;
  int issued = 0, ist = 0;
  auto issue = [&]() {  // the copies of the issue walk's tile into stage ist
    const int tok = iw.first + iw.t * kSpTok, blk = tok / bs, off = tok - blk * bs;
    const int c = blk >> 5;
    if (iw.b != have_b || c != have_c) {
      mine = iw.b == next_b && c == next_c ? nxt : fetch(iw.b, c);
      have_b = iw.b;
      have_c = c;
      next_b = iw.b;
      next_c = c + 1;
      if ((next_c << 5) * bs >= iw.len) {  // the sequence's last chunk
        next_b = iw.b + 1;
        next_c = next_b < p.num_seqs ? ln.first[next_b] / bs >> 5 : 0;
      }
      if (next_b < p.num_seqs) nxt = fetch(next_b, next_c);
    }
    int pb = __shfl_sync(0xffffffffu, mine, blk & 31);
    if (lane == 0) {
      if (pb < 0 || pb >= p.num_blocks) {
        record_error(KV_ERR_DEVICE_BOUNDS);
        pb = 0;
      }
      uint8_t* dst = ring + ist * 2 * kRestTile;
      mbar_arrive_expect_tx(full + ist, 2 * kRestTile);
      const int at = (pb * bs + off) / kSpTok;
      tma_load_5d(dst, &tmK, full + ist, 0, 0, 0, at, iw.kvh);
      tma_load_5d(dst + kRestTile, &tmV, full + ist, 0, 0, 0, at, iw.kvh);
    }
    ++issued;
    if (++ist == nst) ist = 0;
    imore = iw.next(p, ln);
  };
  auto q_of = [&](const SpRestWalk& w) {
    return static_cast<const T*>(p.q) + (static_cast<int64_t>(w.b) * p.num_heads + w.kvh * G) * D;
  };
  WarpState<D, NG> st;
  // the next unit's Q is fetched one unit ahead where the registers allow
  constexpr bool kAheadQ = (D / 16) * NG * 2 <= 16;
  uint32_t qn[D / 16][NG][2];
  auto fetch_next_q = [&]() {
    if constexpr (kAheadQ) {
      SpRestWalk w = cw;
      if (w.next_unit(p, ln)) load_q_frags<T, D, NG>(qn, q_of(w), G, lane);
    }
  };
  for (int i = 0; i < nst && imore; ++i) issue();
  if (more) {
    load_q<T, D, NG>(st, q_of(cw), G, lane);
    fetch_next_q();
  }
  reset_state(st);
  int cst = 0, phase = 0, ok = 1;
  while (more && ok) {
    if (lane == 0) ok = mbar_wait_bounded(full + cst, phase);
    ok = __shfl_sync(0xffffffffu, ok, 0);
    if (!ok) break;
    __syncwarp();
    uint8_t* kt = ring + cst * 2 * kRestTile;
    consume_tile<T, D, kSpTok, NG>(st, kt, kt + kRestTile, cw.first + cw.t * kSpTok, cw.len, p.scale_log2, lane);
    __syncwarp();
    if (imore) issue();  // into the stage just read
    if (++cst == nst) {
      cst = 0;
      phase ^= 1;
    }
    if (cw.t + 1 < cw.t1) {
      ++cw.t;
      continue;
    }
    // ---- the share's piece of the unit is complete
    const bool whole = cw.t0 == 0 && cw.t1 == cw.T, direct = whole && cw.first == 0;
    const int64_t orow = static_cast<int64_t>(cw.b) * p.num_heads + cw.kvh * G;
    const int64_t urow = orow + static_cast<int64_t>(p.num_seqs) * p.num_heads;
    const int64_t crow = (static_cast<int64_t>(share) * 2 + (cw.t0 == 0 ? 1 : 0)) * G;
#pragma unroll
    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) st.l[ng][c] += __shfl_xor_sync(0xffffffffu, st.l[ng][c], o);
    float* po = whole ? p.unit_o + urow * D : p.rest_o + crow * D;
    float* pml = whole ? p.unit_ml + urow * 2 : p.rest_ml + crow * 2;
#pragma unroll
    for (int ng = 0; ng < NG; ++ng)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int g = ng * 8 + (lane & 3) * 2 + c;
        if (g >= G) continue;
        if (direct) {
          const float inv = st.l[ng][c] > 0.f ? __fdiv_rn(1.f, st.l[ng][c]) : 0.f;
          T* o = static_cast<T*>(p.out) + (orow + g) * D + (lane >> 2);
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[mt * 16] = DType<T>::from_float(st.acc[mt][ng][c] * inv);
            o[mt * 16 + 8] = DType<T>::from_float(st.acc[mt][ng][c + 2] * inv);
          }
        } else {
          float* o = po + static_cast<int64_t>(g) * D + (lane >> 2);
#pragma unroll
          for (int mt = 0; mt < D / 16; ++mt) {
            o[mt * 16] = st.acc[mt][ng][c];
            o[mt * 16 + 8] = st.acc[mt][ng][c + 2];
          }
          if (lane < 4) *reinterpret_cast<float2*>(pml + g * 2) = make_float2(st.m[ng][c], st.l[ng][c]);
        }
      }
    if (cw.t0 == 0 && lane == 0) {  // the unit's first share says where its pieces lie
      const int last = whole ? share : cut.of(cw.base + kSpRestCost + cw.T - 1);
      p.rest_span[static_cast<int64_t>(cw.b) * p.num_kv_heads + cw.kvh] = make_int4(share, last, 0, 0);
    }
    more = cw.next_unit(p, ln);
    if (more) {
      if constexpr (kAheadQ) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int ng = 0; ng < NG; ++ng) {
            st.qf[kk][ng][0] = qn[kk][ng][0];
            st.qf[kk][ng][1] = qn[kk][ng][1];
          }
        fetch_next_q();
      } else {
        load_q<T, D, NG>(st, q_of(cw), G, lane);
      }
      reset_state(st);
    }
  }
  if (!ok && lane == 0) drain_fills(full, issued, nst, true);  // a wait ran out: no copy in flight as the CTA ends
}

// A CTA's share [x0, x1) of the prefix line.
template <typename T, int D>
__device__ __forceinline__ void prefix_cta(const SpParams& p, const SpLine& ln, const CUtensorMap& tmK,
                                           const CUtensorMap& tmV, uint8_t* sm, uint64_t* bars, uint32_t tmem,
                                           const SpCut& cut, int share) {
  using Lay = SpLayout<D>;
  constexpr int kSlabs = Lay::kSlabs;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nst = p.stages, bs = p.block_size;
  uint8_t* ring = sm + Lay::kQ;
  uint64_t* bar_full = bars;                      // [stage] tile landed
  uint64_t* bar_empty = bar_full + kSpMaxStages;  // [stage] its MMAs done
  uint64_t* bar_q = bar_empty + kSpMaxStages;     // a unit's Q laid down (every softmax thread)
  uint64_t* bar_o = bar_q + 1;                    // a unit's O read (every softmax thread)
  uint64_t* bar_s = bar_o + 1;                    // [2] S written
  uint64_t* bar_p = bar_s + 2;                    // [2] P written (every softmax thread)
  uint64_t* bar_pv = bar_p + 2;                   // [2] P V done
  uint64_t* bar_end = bar_pv + 2;                 // after a wait ran out: all MMAs done
  SpPrefixWalk w(p, ln, cut.begin(share), cut.begin(share + 1));
  if (warp == kSpTmaWarp) {
    // ---- K and V tiles, one box per block (up to 64 of its tokens by all
    // dims).  A copy costs the warp some 58 clocks to issue, one after another
    // whichever lanes issue them; boxes of 64 dims took twice as many.
    const int rows = min(bs, kSpKeys), at = lane * rows;
    const uint32_t box_bytes = static_cast<uint32_t>(rows / 8 * Lay::kEight);
    // Table entries are fetched 32 at a time, one per lane, and the row's next
    // 32 along with them: a load per tile held the tile's copies up by its
    // latency.  All of a group's units read its first sequence's row.
    auto fetch = [&](int seq, int chunk) -> int {
      const int e = (chunk << 5) + lane;
      return e < p.max_blocks_per_seq ? __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + e)
                                      : 0;
    };
    int have_b = -1, have_c = -1, mine = 0, next_c = -1, nxt = 0;
    const int skip = share == 0 ? p.test_skip : -1;
    int ok = 1, st = 0, phase = 0, armed = 0;
    const int shift = __ffs(bs) - 1;  // (a power of two)
    // Copies go out in the order in which the MMA lane takes the tiles: K of
    // the next tile before V of this one.  (In the order K V K V a K copy
    // waited, behind the V copy before it, for a P V that its own stage did
    // not need.)
    auto copy = [&](const CUtensorMap& map, bool box, int eight, uint32_t bytes) {
      if (lane == 0) {
        if (armed >= nst) ok = mbar_wait_bounded(bar_empty + st, phase ^ 1);
        if (ok && armed != skip) mbar_arrive_expect_tx(bar_full + st, bytes);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) return;
      if (box && armed != skip)
        tma_load_5d(ring + st * Lay::kTile + (at >> 3) * Lay::kEight, &map, bar_full + st, 0, 0, 0, eight, w.kvh);
      ++armed;
      if (++st == nst) {
        st = 0;
        phase ^= 1;
      }
    };
    while (ok && w.next()) {
      bool v_box = false;  // the V copy that is due
      int v_eight = 0;
      uint32_t v_bytes = 0;
      for (int t = w.t0; t < w.t1 && ok; ++t) {
        const int tok = t * kSpKeys, c = tok >> shift >> 5;  // a tile's blocks lie in one chunk
        if (w.lead != have_b || c != have_c) {
          mine = w.lead == have_b && c == next_c ? nxt : fetch(w.lead, c);
          have_b = w.lead;
          have_c = c;
          // the row's next chunk; after its last, the first again (the next unit's)
          next_c = (c + 1) * 32 < (w.keys + bs - 1) >> shift ? c + 1 : 0;
          if (next_c != have_c) nxt = fetch(have_b, next_c);
        }
        const int here = tok + at;
        const bool box = at < kSpKeys && here < w.keys;
        int pb = __shfl_sync(0xffffffffu, mine, here >> shift & 31);
        const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, box)) * box_bytes;
        if (box && (pb < 0 || pb >= p.num_blocks)) {
          record_error(KV_ERR_DEVICE_BOUNDS);
          pb = 0;
        }
        const int eight = ((pb << shift) + (here & (bs - 1))) >> 3;
        copy(tmK, box, eight, bytes);
        if (ok && t > w.t0) copy(tmV, v_box, v_eight, v_bytes);
        v_box = box;
        v_eight = eight;
        v_bytes = bytes;
      }
      if (ok) copy(tmV, v_box, v_eight, v_bytes);
    }
    // At exit no copy or commit is in flight: every stage's last MMAs have
    // completed, or, where a wait ran out (the MMA lane may be gone), at least
    // the copies have landed.
    if (lane == 0) {
      if (!ok || !drain_fills(bar_empty, armed, nst, false)) drain_fills(bar_full, armed, nst, true);
    }
  } else if (warp == kSpMmaWarp) {
    if (lane == 0) {
      // ---- MMA issue
      constexpr uint32_t idS = tc::idesc_f16(kBf16, kSpRows, kSpKeys, false);
      constexpr uint32_t idPV = tc::idesc_f16(kBf16, kSpRows, D, true);
      constexpr uint32_t kQHi = tc::sdesc_hi(1024), kKvHi = tc::sdesc_hi(Lay::kEight);
      const uint32_t q_lo = tc::sdesc_lo(smem_u32(sm), 16), k_lo = tc::sdesc_lo(smem_u32(ring), 16);
      const uint32_t v_lo = tc::sdesc_lo(smem_u32(ring), Lay::kAtom);
      int st = 0, phase = 0;  // the ring's stage that is taken next
      auto taken = [&]() {
        tc::commit(bar_empty + st);
        if (++st == nst) {
          st = 0;
          phase ^= 1;
        }
      };
      // S of tile j (first: of unit number un) once its K, the unit's Q
      // and its buffer (P V of tile j - 2 done) are ready
      auto issue_s = [&](int j, bool first, int un) -> bool {
        if (first && !mbar_wait_bounded(bar_q, un & 1)) return false;
        if (!mbar_wait_bounded(bar_full + st, phase)) return false;
        if (j >= 2 && !mbar_wait_bounded(bar_pv + (j & 1), ((j >> 1) - 1) & 1)) return false;
        tc::fence_after();
        const uint32_t d = tmem + (j & 1) * 64, kb = k_lo + st * (Lay::kTile / 16);
        tc::mma_f16_words<false>(d, q_lo, kQHi, kb, kKvHi, idS);
#pragma unroll
        for (int kk = 1; kk < D / 16; ++kk)
          tc::mma_f16_words<true>(d, q_lo + ((kk >> 2) * Lay::kQSlab + (kk & 3) * 32) / 16, kQHi,
                                  kb + ((kk >> 2) * Lay::kAtom + (kk & 3) * 32) / 16, kKvHi, idS);
        tc::commit(bar_s + (j & 1));
        taken();
        return true;
      };
      auto issue_pv = [&](int j, bool first, int un) -> bool {
        if (!mbar_wait_bounded(bar_full + st, phase)) return false;
        // P lands after the softmax warps have zeroed a last tile's V tail
        if (!mbar_wait_bounded(bar_p + (j & 1), (j >> 1) & 1)) return false;
        if (first && un > 0 && !mbar_wait_bounded(bar_o, (un - 1) & 1)) return false;
        tc::fence_after();
        const uint32_t a = tmem + (j & 1) * 64, vb = v_lo + st * (Lay::kTile / 16);
#pragma unroll
        for (int kk = 0; kk < kSpKeys / 16; ++kk)
          tc::mma_f16_ts_words(tmem + 128, a + kk * 8, vb + kk * (2 * Lay::kEight / 16), kKvHi, idPV,
                               (!first || kk > 0) ? 1u : 0u);
        tc::commit(bar_pv + (j & 1));
        taken();
        return true;
      };
      const bool any = w.next();
      int t = w.t0, j = 0, un = 0;
      bool ok = any && issue_s(0, true, 0);
      while (ok) {
        const bool last = t + 1 == w.t1;
        if (!last) ok = issue_s(j + 1, false, un);
        ok = ok && issue_pv(j, t == w.t0, un);
        ++j;
        ++t;
        if (last) {
          if (!w.next()) break;
          t = w.t0;
          ++un;
          ok = ok && issue_s(j, true, un);
        }
      }
      if (any && !ok) {  // a wait ran out: what was issued ends before the tensor memory goes
        tc::commit(bar_end);
        mbar_wait_bounded(bar_end, 0);
      }
    }
  } else {
    // ---- softmax: thread r owns query row r
    const int r = tid;
    const uint32_t tS = tmem + (static_cast<uint32_t>(warp * 32) << 16), tO = tS + 128;
    const float c2 = p.scale_log2;
    const uint64_t c2x2 = tc::f2(c2, c2);
    // A row's reference moves when a score passes it by more than kSlack (in
    // powers of two), or when its first tile lies more than kLow below it.
    // bf16 P has float32's exponents, so 2^30 costs no precision and the sums
    // stay far from overflow (|V| < 2^90).  fp16 P stays below 2^14, and its
    // largest is 1 or more, so that weights down to 2^-25 of the largest count
    // (rounded to P's step of 2^-24), as in the decode kernels; with the
    // largest at 2^-8 those below 2^-17 of it were lost.  A move costs the
    // warp a second pass and, past the unit's first tile, a wait for the last
    // P V and a read and write of O (about 2 us): with 2^8 for both types, a
    // warp of 32 rows of ordinary scores (standard deviation 1.5) moved in one
    // tile of four.
    constexpr float kSlack = kBf16 ? 30.f : 14.f, kLow = kBf16 ? 30.f : 0.f;
    bool ok = true;
    // A unit's Q into shared memory in the MMA's swizzled layout, 16-byte
    // chunks copied asynchronously, all of a thread's in flight at once
    auto load_q = [&]() {
      constexpr int kCh = D / 8;
      const uint32_t dst = smem_u32(sm);
      const int sq0 = w.b0, h0 = w.kvh * p.group;
      for (int i = tid; i < w.rows * kCh; i += kSpSoftWarps * 32) {
        const int row = i / kCh, ch = i % kCh, sq = row / p.group;
        cp_async16(dst + (ch >> 3) * Lay::kQSlab + row * 128 + (((ch & 7) ^ (row & 7)) << 4),
                   static_cast<const T*>(p.q) +
                       (static_cast<int64_t>(sq0 + sq) * p.num_heads + h0 + row - sq * p.group) * D + ch * 8,
                   true);
      }
      cp_async_commit();
      cp_async_wait<0>();
      fence_proxy_async_smem();  // read by the tensor cores
      mbar_arrive(bar_q);
    };
    bool more = w.next();
    if (more) load_q();
    int j = 0;
    while (more) {
      const bool mine = warp * 32 < w.rows, valid = r < w.rows;
      float m_ref = 0.f, l = 0.f;
      for (int t = w.t0; t < w.t1; ++t, ++j) {
        const int buf = (j & 1) * 64;
        // after a timeout (recorded) the remaining waits are skipped
        if (ok && !mbar_wait_bounded(bar_s + (j & 1), (j >> 1) & 1)) ok = false;
        tc::fence_after();
        const int keys = min(kSpKeys, w.keys - t * kSpKeys);
        if (mine) {
          uint32_t x[64];
          uint64_t ls[2];
          float me;
          bool rescale = false;
          float alpha = 1.f;
          // one pass: e = S c2 - m_ref (no key: -inf), P = exp2(e) rounded
          // to T, its sum, the row's max of e; repeated against a new
          // reference only where that max calls for one
#pragma unroll 1
          for (int attempt = 0; attempt < 2; ++attempt) {
            const uint64_t negm = tc::f2(-m_ref, -m_ref);
            ls[0] = ls[1] = tc::f2(0.f, 0.f);
            tc::ld_32x32b_x32(tS + buf, x);
            tc::ld_32x32b_x32(tS + buf + 32, x + 32);
            tc::wait_ld();
            float ma = -INFINITY, mb = -INFINITY;
            if (keys < kSpKeys) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                float2 ev = tc::f2_split(
                    tc::ffma2(tc::f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2x2, negm));
                ev.x = 2 * i < keys ? ev.x : -INFINITY;
                ev.y = 2 * i + 1 < keys ? ev.y : -INFINITY;
                softmax_pair<T>(ev, i, ma, mb, ls, x);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                softmax_pair<T>(tc::f2_split(tc::ffma2(tc::f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])),
                                                       c2x2, negm)),
                                i, ma, mb, ls, x);
            }
            me = fmaxf(ma, mb);
            if (attempt == 1) break;
            const bool need = valid && (me > kSlack || (l == 0.f && me != -INFINITY && me < -kLow));
            rescale = __any_sync(0xffffffffu, need);
            if (!rescale) break;
            const float m_new = need ? m_ref + me : m_ref;
            // before the row's first key of weight l and O are 0: nothing to
            // rescale, and a move down by 2^128 or more would make it 0 inf
            alpha = l == 0.f ? 1.f : fast_exp2(m_ref - m_new);
            l *= alpha;
            m_ref = m_new;
          }
          tc::st_32x32b_x32(tS + buf, x);
          const float2 a = tc::f2_split(ls[0]), b2 = tc::f2_split(ls[1]);
          l += (a.x + a.y) + (b2.x + b2.y);
          if (rescale && t > w.t0) {
            // O holds the unit's tiles up to the last one: its P V is done
            if (ok && !mbar_wait_bounded(bar_pv + ((j - 1) & 1), ((j - 1) >> 1) & 1)) ok = false;
            tc::fence_after();
            const uint64_t a2 = tc::f2(alpha, alpha);
#pragma unroll
            for (int oc = 0; oc < D; oc += 32) {
              uint32_t v[32];
              tc::ld_32x32b_x32(tO + oc, v);
              tc::wait_ld();
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 y = tc::f2_split(tc::fmul2(tc::f2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), a2));
                v[k] = __float_as_uint(y.x);
                v[k + 1] = __float_as_uint(y.y);
              }
              tc::st_32x32b_x32(tO + oc, v);
            }
          }
          tc::wait_st();
        }
        if (keys < kSpKeys) {
          // V rows past the last key (blocks not loaded) are zeroed: their P
          // is 0, and 0 times what lies there must be 0
          const int i = 2 * j + 1, st = i % nst;  // (the unit's last tile: no K lies before its V)
          if (ok && !mbar_wait_bounded(bar_full + st, (i / nst) & 1)) ok = false;
          uint8_t* vt = ring + st * Lay::kTile;
#pragma unroll 1
          for (int k = keys * 8 * kSlabs + tid; k < kSpKeys * 8 * kSlabs; k += kSpSoftWarps * 32) {
            const int row = k / (8 * kSlabs), rest = k % (8 * kSlabs);
            *reinterpret_cast<uint4*>(vt + (row >> 3) * Lay::kEight + (rest >> 3) * Lay::kAtom + (row & 7) * 128 +
                                      (rest & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tc::fence_before();
        mbar_arrive(bar_p + (j & 1));
      }
      // all scores of the unit are read: the next unit's Q goes down while
      // the last P V runs
      const bool whole = w.t0 == 0 && w.t1 == w.T, begins = w.t0 == 0;
      const int b0 = w.b0, kvh = w.kvh;
      const int end = w.at + kSpPrefixCost + w.T - 1, rows = w.rows;
      more = w.next();
      if (more) load_q();
      if (ok && !mbar_wait_bounded(bar_pv + ((j - 1) & 1), ((j - 1) >> 1) & 1)) ok = false;
      tc::fence_after();
      // The results: after the CTA's last unit Q and the stages are free, and
      // the rows go out through them in bulk stores (0.6 us for 128 rows of
      // 128 floats; from the registers, 16 bytes of 32 rows at a time, 2.9 us);
      // other units' rows are stored from the registers.
      const int sq = r / p.group, b = b0 + sq, g = r - sq * p.group;
      const int64_t orow = static_cast<int64_t>(b) * p.num_heads + kvh * p.group + g;
      const int64_t crow = (static_cast<int64_t>(share) * 2 + (begins ? 1 : 0)) * kSpRows + r;
      float* po = (whole ? p.unit_o + orow * D : p.pre_o + crow * D);
      if (mine) {
        uint4* dst = more ? reinterpret_cast<uint4*>(po) : reinterpret_cast<uint4*>(sm) + r * (D / 4);
#pragma unroll 1
        for (int oc = 0; oc < D; oc += 32) {
          uint32_t v[32];
          tc::ld_32x32b_x32(tO + oc, v);
          tc::wait_ld();
          if (valid) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[sp_chunk(oc / 4 + k, r)] = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
          }
        }
        if (valid) {
          *reinterpret_cast<float2*>(whole ? p.unit_ml + orow * 2 : p.pre_ml + crow * 2) = make_float2(m_ref, l);
          // the unit's first CTA says where its pieces lie, once per sequence
          if (g == 0 && begins)
            p.pre_span[static_cast<int64_t>(b) * p.num_kv_heads + kvh] =
                make_int4(share, whole ? share : cut.of(end), r, 0);
        }
      }
      if (!more) {
        fence_proxy_async_smem();
        named_barrier_sync(1, kSpSoftWarps * 32);
        // a cut unit's rows lie together; a whole one's sequence by sequence
        if (!whole && r == 0) bulk_store(po, sm, static_cast<uint32_t>(rows * D * 4));
        if (whole && valid && g == 0) bulk_store(po, sm + r * D * 4, static_cast<uint32_t>(p.group * D * 4));
        bulk_store_wait();
      }
      tc::fence_before();
      mbar_arrive(bar_o);
    }
  }
}

// Registers: two CTAs of six warps, at most 168 a thread (as the prefill).
// NG: n8 blocks of a rest unit's query rows.
template <typename T, int D, int NG>
__global__ void __launch_bounds__(kSpThreads, 2)
    shared_prefix_kernel(const SpParams p, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmRK,
                         const __grid_constant__ CUtensorMap tmRV) {
  using Lay = SpLayout<D>;
  extern __shared__ uint8_t sp_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sp_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Lay::kQ + p.stages * Lay::kTile);
  uint64_t* rest_full = bars + 2 * kSpMaxStages + 9;  // [warp][rest stage] tile landed
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(rest_full + kSpSoftWarps * kSpMaxRest);
  const int B = p.num_seqs, NGR = p.num_groups;
  SpLine ln;
  ln.pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bars) + Lay::kBars);
  ln.rest = ln.pre + NGR + 1;
  ln.start = ln.rest + B + 1;
  ln.prefix = ln.start + NGR + 1;
  ln.first = ln.prefix + NGR;
  ln.len = ln.first + B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = p.block_size;

  // ---- barriers, tensor memory, the maps
  if (warp == kSpMmaWarp) tc::alloc(tmem_slot, kSpCols);
  if (warp == kSpTmaWarp) {
    if (lane < 4) prefetch_tensormap(lane == 0 ? &tmK : lane == 1 ? &tmV : lane == 2 ? &tmRK : &tmRV);
    for (int s = lane; s < 2 * kSpMaxStages; s += 32) mbar_init(bars + s, 1);
    // Q and O: every softmax thread; S, P (every softmax thread) and P V of two buffers; the end
    if (lane < 9) mbar_init(bars + 2 * kSpMaxStages + lane, lane < 2 || (lane >= 4 && lane < 6) ? kSpSoftWarps * 32 : 1);
    for (int s = lane; s < kSpSoftWarps * kSpMaxRest; s += 32) mbar_init(rest_full + s, 1);
    fence_mbar_init();
  }

  // ---- the lines: lengths, groups, costs, their prefix sums
  int bad = 0;
  const int64_t columns = static_cast<int64_t>(p.max_blocks_per_seq) * bs;
  const int cap = columns < INT32_MAX ? static_cast<int>(columns) : INT32_MAX;
  bool out = false;
#pragma unroll 4
  for (int b = tid; b < B; b += kSpThreads) {
    const int L = p.seq_lens[b], in = max(0, min(L, cap));
    out |= in != L;
    ln.len[b] = in;
  }
  if (out) record_error(KV_ERR_DEVICE_BOUNDS);
  for (int g = tid; NGR > 0 && g <= NGR; g += kSpThreads) {
    const int s = p.group_start[g], nx = g < NGR ? p.group_start[g + 1] : B;
    if (g < NGR) ln.prefix[g] = p.prefix_lens[g];
    ln.start[g] = s;
    if (s < 0 || s > nx || nx > B || (g == 0 && s != 0) || (g == NGR && s != B)) bad = 1;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) record_error(KV_ERR_DEVICE_BOUNDS);  // no group: every sequence reads its whole table
  auto shared_of = [&](int g) -> int {  // tokens that group g shares
    if (bad || ln.start[g + 1] - ln.start[g] < 2) return 0;  // a group of one shares with nobody
    return max(0, min(ln.prefix[g], ln.len[ln.start[g]])) & -bs;  // (a power of two)
  };
  // each thread takes neighbours of either kind, so that their sums are its own
  const int pg = (NGR + kSpThreads - 1) / kSpThreads, pb = (B + kSpThreads - 1) / kSpThreads;
  const int g0 = min(NGR, tid * pg), g1 = min(NGR, g0 + pg), b0 = min(B, tid * pb), b1 = min(B, b0 + pb);
  int lg = 0, lb = 0;
  for (int g = g0; g < g1; ++g) {
    if (!bad && ln.prefix[g] < 0) record_error(KV_ERR_DEVICE_BOUNDS);
    const int P = shared_of(g);
    if (P > 0)
      lg += (ln.start[g + 1] - ln.start[g] + p.tile_seqs - 1) / p.tile_seqs * ((P + kSpKeys - 1) / kSpKeys + kSpPrefixCost);
    ln.pre[g + 1] = lg;
  }
  for (int b = b0; b < b1; ++b) {
    int first = 0;
    const int L = ln.len[b];
    if (!bad && NGR > 0) {
      int lo = 0, hi = NGR - 1;  // the last group that begins at or before b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ln.start[mid] <= b) lo = mid; else hi = mid - 1;
      }
      // a sequence shorter than its group's prefix (an empty slot of the
      // batch) reads its own table
      const int P = shared_of(lo);
      if (L >= P) first = P;
    }
    ln.first[b] = first;
    if (L > first) lb += (L - first + kSpTok - 1) / kSpTok + kSpRestCost;
    ln.rest[b + 1] = lb;
  }
  int ig = lg, ib = lb;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int yg = __shfl_up_sync(0xffffffffu, ig, off), yb = __shfl_up_sync(0xffffffffu, ib, off);
    if (lane >= off) {
      ig += yg;
      ib += yb;
    }
  }
  __shared__ int2 warp_tot[kSpThreads / 32];
  if (lane == 31) warp_tot[warp] = make_int2(ig, ib);
  __syncthreads();  // nobody looks at the prefixes as given any more
  ig -= lg;
  ib -= lb;
  for (int i = 0; i < warp; ++i) {
    ig += warp_tot[i].x;
    ib += warp_tot[i].y;
  }
  if (tid == 0) ln.pre[0] = ln.rest[0] = 0;
  for (int g = g0; g < g1; ++g) {
    ln.pre[g + 1] += ig;
    ln.prefix[g] = shared_of(g);
  }
  for (int b = b0; b < b1; ++b) ln.rest[b + 1] += ib;
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  for (int b = blockIdx.x + tid * gridDim.x; b < B; b += kSpThreads * gridDim.x)
    p.seq[b] = make_int2(ln.first[b], ln.len[b]);

  // ---- SMs on each line, by weight: both CTAs of an SM take the same one
  // (blocks i and i + SMs share an SM where the device places blocks in turn;
  // nothing but speed rests on that)
  const int Wp = p.num_kv_heads * ln.pre[NGR], Wr = p.num_kv_heads * ln.rest[B];
  const int pid = blockIdx.x, sms = p.num_sms, sm_of = pid % sms, layer = pid / sms, layers = gridDim.x / sms;
  int Sp = 0;  // SMs on the prefix line
  if (Wp > 0) {
    const float tp = static_cast<float>(Wp) * kSpPrefixWeight, tr = static_cast<float>(Wr) * kSpRestWeight;
    Sp = Wr == 0 ? sms : max(1, min(sms - 1, static_cast<int>(sms * (tp / (tp + tr)) + 0.5f)));
  }
  if (sm_of < Sp) {
    const SpCut cut(Wp, Sp * layers);
    const int share = layer * Sp + sm_of;
    if (share < cut.shares) prefix_cta<T, D>(p, ln, tmK, tmV, sm, bars, *tmem_slot, cut, share);
  } else if (warp < kSpSoftWarps && Wr > 0) {
    // the first shares go to warp 0 of every CTA, and so on
    const int ctas = (sms - Sp) * layers;
    const SpCut cut(Wr, ctas * kSpSoftWarps);
    const int share = warp * ctas + layer * (sms - Sp) + sm_of - Sp;
    if (share < cut.shares)
      rest_warp<T, D, NG>(p, ln, tmRK, tmRV, sm + warp * p.rest_stages * 2 * Lay::kRestTile,
                          rest_full + warp * kSpMaxRest, cut, share, lane);
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kSpMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::dealloc(*tmem_slot, kSpCols);
  }
}

// Joins a row's pieces.  WPR warps per (sequence, query head): warp w of them
// takes pieces w, w + WPR, ..., a lane D / 32 outputs, and the first one adds
// up the others' in order.  A piece's statistics and its values are loaded
// together, so a row costs two round trips (where its pieces lie, what they
// hold).  Rows that the first kernel wrote whole are left alone; a sequence
// of no tokens gets zeros.  (Programmatic dependent launches of the two kernels
// saved nothing: 9.5 against 9.7 us for the smallest batches, and up to 2 us
// more for large ones.)
constexpr int kSpMergeWarps = 8;

template <typename T, int D, int WPR>
__global__ void __launch_bounds__(kSpMergeWarps * 32) shared_merge_kernel(const SpParams p) {
  constexpr int kV = D / 32, kAhead = 4, kRows = kSpMergeWarps / WPR;
  __shared__ float part[WPR > 1 ? kRows : 1][WPR][D + 2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rw = warp / WPR, w = warp % WPR;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + rw;
  const bool real = row < static_cast<int64_t>(p.num_seqs) * p.num_heads;
  const int b = real ? static_cast<int>(row / p.num_heads) : 0;
  const int h = real ? static_cast<int>(row - static_cast<int64_t>(b) * p.num_heads) : 0;
  const int kvh = h / p.group, g = h - kvh * p.group;
  const int64_t at = static_cast<int64_t>(b) * p.num_kv_heads + kvh;
  const int2 sq = p.seq[b];  // tokens from the prefix unit, length
  int4 ps = p.pre_span[at], rs = p.rest_span[at];
  auto clamped = [&](int4 v, int shares) {  // in range whatever a call that timed out left there
    v.x = max(0, min(v.x, shares - 1));
    v.y = max(v.x, min(v.y, shares - 1));
    v.z = max(0, min(v.z, kSpRows - p.group));
    return v;
  };
  ps = sq.x > 0 ? clamped(ps, p.num_ctas) : make_int4(0, -1, 0, 0);
  rs = sq.y > sq.x ? clamped(rs, p.num_ctas * kSpSoftWarps) : make_int4(0, -1, 0, 0);
  const int np = ps.y - ps.x + 1, nr = rs.y - rs.x + 1;
  const bool skip = !real || (sq.x == 0 && nr == 1);  // written by the first kernel
  const int n = skip ? 0 : np + nr;
  float m = -INFINITY, den = 0.f, acc[kV];
#pragma unroll
  for (int v = 0; v < kV; ++v) acc[v] = 0.f;
  for (int i0 = w; i0 < n; i0 += WPR * kAhead) {
    float2 ml[kAhead];
    float y[kAhead][kV];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * WPR;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (i < n) {
        // piece i: a row of the whole units' array, or of a share's cut pieces
        // (the first share's is its last piece, the others' their first)
        const bool pre = i < np;
        const int4 s = pre ? ps : rs;
        const int c = pre ? i : i - np;
        const bool cut = s.x != s.y;
        const int64_t slot = static_cast<int64_t>(s.x + c) * 2 + (c == 0 ? 1 : 0);
        const int64_t pr = !cut  ? row + (pre ? 0 : static_cast<int64_t>(p.num_seqs) * p.num_heads)
                           : pre ? slot * kSpRows + s.z + g
                                 : slot * p.group + g;
        ml[k] = *reinterpret_cast<const float2*>((!cut ? p.unit_ml : pre ? p.pre_ml : p.rest_ml) + pr * 2);
        // a prefix row's 16-byte chunks are moved (sp_chunk)
        const int at = pre ? sp_chunk(lane * kV / 4, s.z + g) * 4 + lane * kV % 4 : lane * kV;
        const float* src = (!cut ? p.unit_o : pre ? p.pre_o : p.rest_o) + pr * D + at;
        if constexpr (kV == 4) *reinterpret_cast<float4*>(y[k]) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(y[k]) = *reinterpret_cast<const float2*>(src);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      // no such piece, or one without weight; a piece whose sum is NaN (a score
      // that is NaN or +inf) makes the row NaN
      if (ml[k].y == 0.f) continue;
      const float mx = fmaxf(m, ml[k].x);
      const float old = fast_exp2(m - mx), wt = fast_exp2(ml[k].x - mx);
      m = mx;
      den = den * old + wt * ml[k].y;
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[v] = acc[v] * old + wt * y[k][v];
    }
  }
  if constexpr (WPR > 1) {
    if (w > 0) {
#pragma unroll
      for (int v = 0; v < kV; ++v) part[rw][w][lane * kV + v] = acc[v];
      if (lane == 0) {
        part[rw][w][D] = m;
        part[rw][w][D + 1] = den;
      }
    }
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 1; k < WPR; ++k) {
      const float mk = part[rw][k][D], dk = part[rw][k][D + 1];
      if (dk == 0.f) continue;
      const float mx = fmaxf(m, mk), old = fast_exp2(m - mx), wt = fast_exp2(mk - mx);
      m = mx;
      den = den * old + wt * dk;
#pragma unroll
      for (int v = 0; v < kV; ++v) acc[v] = acc[v] * old + wt * part[rw][k][lane * kV + v];
    }
  }
  if (skip) return;
  T* o = static_cast<T*>(p.out) + row * D + lane * kV;
  const float inv = den > 0.f ? __fdiv_rn(1.f, den) : 0.f;
  if constexpr (kV == 4)
    *reinterpret_cast<uint2*>(o) =
        make_uint2(Mma<T>::pack(acc[0] * inv, acc[1] * inv), Mma<T>::pack(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(o) = Mma<T>::pack(acc[0] * inv, acc[1] * inv);
}

// ------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 sp_encode_fn() {
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

// A layer's cache as a tensor {64 dims, `rows` slots, D / 64 slabs, slots /
// rows, Hkv}, boxes of all D dims of one head in `groups` times `rows`
// consecutive slots (a block's slots are a multiple of `rows`): shared memory
// holds `rows` slots slab by slab, then the next ones.  128-byte swizzle.
bool sp_map(const void* cache, int64_t slots, int hkv, int d, int rows, int groups, CUtensorMap* out) {
  auto fn = sp_encode_fn();
  if (!fn) return false;
  const cuuint64_t slot = static_cast<cuuint64_t>(hkv) * d * 2;
  cuuint64_t dims[5] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(d / 64),
                        static_cast<cuuint64_t>(slots / rows), static_cast<cuuint64_t>(hkv)};
  cuuint64_t strides[4] = {slot, 128, slot * rows, static_cast<cuuint64_t>(d) * 2};
  cuuint32_t box[5] = {64, static_cast<cuuint32_t>(rows), static_cast<cuuint32_t>(d / 64),
                       static_cast<cuuint32_t>(groups), 1};
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 5, const_cast<void*>(cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int sp_sm_count() {
  int dev = 0, n = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  return n > 0 ? n : 1;
}

// Whether the shapes take the tensor-core kernels; the rest is
// paged_decode_attention.
bool sp_shapes(int B, int G, int D, int bs, int dtype) {
  return dtype != KV_DTYPE_F32 && (D == 64 || D == 128) && (bs == 16 || bs == 32 || bs == 64 || bs == 128) &&
         G <= kSpMaxGroup && B <= kSpMaxSeqs;
}
// Places on the lines fit an int (with room for the units' places to be
// stepped past the end): at most B units per kv head of the tiles of a whole
// table row and the charge.
bool sp_line_fits(int B, int Hkv, int64_t row_tokens) {
  const int64_t unit = row_tokens / kSpTok + 1 + std::max(kSpPrefixCost, kSpRestCost);
  return unit < (1 << 24) && unit * B < INT32_MAX / 2 / Hkv;
}

size_t sp_align(size_t x) { return (x + 255) & ~size_t(255); }

struct SpWorkspace {
  size_t unit_o, unit_ml, pre_o, pre_ml, rest_o, rest_ml, pre_span, rest_span, seq, bytes;
};

SpWorkspace sp_workspace(int B, int Hq, int Hkv, int D, int ctas) {
  SpWorkspace w{};
  size_t at = 0;
  auto take = [&](size_t n) {
    const size_t here = at;
    at += sp_align(n);
    return here;
  };
  const size_t rows = static_cast<size_t>(B) * Hq, spans = static_cast<size_t>(B) * Hkv;
  const size_t pre = static_cast<size_t>(ctas) * 2 * kSpRows;
  const size_t rest = static_cast<size_t>(ctas) * kSpSoftWarps * 2 * (Hq / Hkv);
  w.unit_o = take(2 * rows * D * 4);
  w.unit_ml = take(2 * rows * 2 * 4);
  w.pre_o = take(pre * D * 4);
  w.pre_ml = take(pre * 2 * 4);
  w.rest_o = take(rest * D * 4);
  w.rest_ml = take(rest * 2 * 4);
  w.pre_span = take(spans * sizeof(int4));
  w.rest_span = take(spans * sizeof(int4));
  w.seq = take(static_cast<size_t>(B) * sizeof(int2));
  w.bytes = at;
  return w;
}

// Shared memory per CTA with two CTAs on an SM, and with one.
constexpr int kSpSmemTwo = 112 * 1024, kSpSmemOne = 226 * 1024;

template <typename T, int D, int WPR>
cudaError_t launch_merge(const SpParams& p, int64_t rows, cudaStream_t st) {
  constexpr int kRows = kSpMergeWarps / WPR;
  shared_merge_kernel<T, D, WPR>
      <<<static_cast<unsigned>((rows + kRows - 1) / kRows), kSpMergeWarps * 32, 0, st>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, int NG>
cudaError_t launch_shared(SpParams& p, const CUtensorMap (&maps)[4], int sms, cudaStream_t st) {
  using Lay = SpLayout<D>;
  // as many stages as fit beside the batch's lines (4 at head_dim 128, 8 at
  // 64, for small batches); a batch whose lines leave no three gets an SM per CTA
  p.stages = D == 128 ? 4 : kSpMaxStages;
  while (p.stages > kSpMinStages && Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemTwo) --p.stages;
  int per_sm = 2;
  if (Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemTwo) {
    per_sm = 1;
    p.stages = D == 128 ? 4 : kSpMaxStages;
    while (p.stages > kSpMinStages && Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemOne) --p.stages;
  }
  p.rest_stages = Lay::rest_stages(p.stages);
  const int smem = Lay::bytes(p.stages, p.num_seqs, p.num_groups);
  p.num_sms = sms;
  p.num_ctas = sms * per_sm;
  auto kern = shared_prefix_kernel<T, D, NG>;
  static std::atomic<uint64_t> configured{0};  // devices (of the first 64) whose limits are set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !(configured.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpSmemOne);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured.fetch_or(uint64_t{1} << dev);
  }
  kern<<<p.num_ctas, kSpThreads, smem, st>>>(p, maps[0], maps[1], maps[2], maps[3]);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // few rows: up to eight warps join one
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_heads;
  if (rows * 8 <= static_cast<int64_t>(sms) * 64) return launch_merge<T, D, 8>(p, rows, st);
  if (rows * 2 <= static_cast<int64_t>(sms) * 64) return launch_merge<T, D, 2>(p, rows, st);
  return launch_merge<T, D, 1>(p, rows, st);
}

template <typename T>
cudaError_t launch_shared_shape(SpParams& p, int head_dim, const CUtensorMap (&maps)[4], int sms, cudaStream_t st) {
  if (head_dim == 64)
    return p.group <= 8 ? launch_shared<T, 64, 1>(p, maps, sms, st) : launch_shared<T, 64, 2>(p, maps, sms, st);
  return p.group <= 8 ? launch_shared<T, 128, 1>(p, maps, sms, st) : launch_shared<T, 128, 2>(p, maps, sms, st);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_shared_prefix_workspace_size(int32_t num_seqs, int32_t num_heads, int32_t num_kv_heads,
                                                  int32_t head_dim, int32_t block_size, int64_t max_seq_len,
                                                  int dtype, size_t* bytes_out) {
  // the shapes' own checks, and the size where the call is plain decode
  const int st = paged_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size, max_seq_len, 0,
                                             dtype, bytes_out);
  if (st != KV_OK) return st;
  if (sp_shapes(num_seqs, num_heads / num_kv_heads, head_dim, block_size, dtype))
    *bytes_out = std::max(*bytes_out,
                          sp_workspace(num_seqs, num_heads, num_kv_heads, head_dim, 2 * sp_sm_count()).bytes);
  return KV_OK;
}

extern "C" int paged_decode_attention_shared_prefix(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* group_start, const int32_t* prefix_lens, int32_t num_seqs,
    int32_t num_groups, int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
    int64_t num_blocks, int32_t max_blocks_per_seq, int64_t max_seq_len, float scale, int dtype, void* workspace,
    size_t workspace_bytes, void* stream) {
  size_t need = 0;
  const int chk = paged_shared_prefix_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim, block_size,
                                                     max_seq_len, dtype, &need);
  if (chk != KV_OK) return chk;
  if (max_blocks_per_seq <= 0 || num_blocks <= 0 || num_blocks > INT32_MAX / block_size || num_groups < 0 || num_groups > num_seqs ||
      !std::isfinite(scale))
    return KV_ERR_INVALID_ARG;
  if (num_seqs == 0) return KV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !seq_lens) return KV_ERR_INVALID_ARG;
  if (num_groups > 0 && (!group_start || !prefix_lens)) return KV_ERR_INVALID_ARG;
  const uintptr_t bits = reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(q) |
                         reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
  if (bits % 16 != 0) return KV_ERR_INVALID_ARG;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return KV_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) % 256 != 0) return KV_ERR_INVALID_ARG;
  }
  const int G = num_heads / num_kv_heads;
  if (!sp_shapes(num_seqs, G, head_dim, block_size, dtype) ||
      !sp_line_fits(num_seqs, num_kv_heads, static_cast<int64_t>(max_blocks_per_seq) * block_size))
    return paged_decode_attention(out, q, k_cache, v_cache, block_tables, seq_lens, num_seqs, num_heads, num_kv_heads,
                                  head_dim, block_size, num_blocks, max_blocks_per_seq, max_seq_len, scale, 0, dtype,
                                  workspace, workspace_bytes, stream);
  SpParams p{};
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.group_start = group_start;
  p.prefix_lens = prefix_lens;
  p.num_seqs = num_seqs;
  p.num_groups = num_groups;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = G;
  p.block_size = block_size;
  p.tile_seqs = kSpRows / G;
  p.num_blocks = num_blocks;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.test_skip = debug_skip_tile();
  const int sms = sp_sm_count();
  const SpWorkspace w = sp_workspace(num_seqs, num_heads, num_kv_heads, head_dim, 2 * sms);
  char* ws = static_cast<char*>(workspace);
  p.unit_o = reinterpret_cast<float*>(ws + w.unit_o);
  p.unit_ml = reinterpret_cast<float*>(ws + w.unit_ml);
  p.pre_o = reinterpret_cast<float*>(ws + w.pre_o);
  p.pre_ml = reinterpret_cast<float*>(ws + w.pre_ml);
  p.rest_o = reinterpret_cast<float*>(ws + w.rest_o);
  p.rest_ml = reinterpret_cast<float*>(ws + w.rest_ml);
  p.pre_span = reinterpret_cast<int4*>(ws + w.pre_span);
  p.rest_span = reinterpret_cast<int4*>(ws + w.rest_span);
  p.seq = reinterpret_cast<int2*>(ws + w.seq);
  CUtensorMap maps[4];  // prefix K, V; rest K, V
  const int64_t slots = num_blocks * block_size;
  const int rows = std::min(block_size, kSpKeys);
  if (!sp_map(k_cache, slots, num_kv_heads, head_dim, 8, rows / 8, &maps[0]) ||
      !sp_map(v_cache, slots, num_kv_heads, head_dim, 8, rows / 8, &maps[1]) ||
      !sp_map(k_cache, slots, num_kv_heads, head_dim, kSpTok, 1, &maps[2]) ||
      !sp_map(v_cache, slots, num_kv_heads, head_dim, kSpTok, 1, &maps[3]))
    return cuda_status(cudaErrorInvalidValue, "cuTensorMapEncodeTiled failed");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return cuda_status(dtype == KV_DTYPE_F16 ? launch_shared_shape<__half>(p, head_dim, maps, sms, st)
                                           : launch_shared_shape<__nv_bfloat16>(p, head_dim, maps, sms, st));
}

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_shared_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
