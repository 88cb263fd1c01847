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
//     read once for all of them;
//   rest unit (sequence, kv head): G rows against keys P_g .. L_b - 1.
//
// What bounds it: every group's prefix and every sequence's rest are read
// once (a second row tile of a group finds the prefix in L2), 4 D flops per
// query row and key; memory until about 280 query rows share each key, then
// the tensor cores.
//
// Partition.  The units in order (groups, then sequences; kv head; row tile)
// lie on a line, each a fixed charge followed by its 64-key tiles.  The line
// is cut into equal lengths, one per CTA (two persistent CTAs per SM), so the
// load is even whatever the mix of group sizes and lengths, and a unit is cut
// only where a CTA's share ends.  A rest unit of a sequence without prefix
// that falls whole into one CTA is written to `out`; every other piece writes
// (o, m, l) in float32 to the workspace, and shared_merge_kernel joins a
// row's pieces, in their order along the line, so results do not depend on
// timing.  Every CTA rebuilds the line from group_start, prefix_lens and
// seq_lens in shared memory; nothing in the workspace outlives the call.
//
// Warps of a CTA (the tcgen05 pipeline of the chunked prefill, at 64 keys a
// tile and with two score buffers):
//   warp 5: TMA: K and V tiles through the block table into one ring of
//     stages, K_0 V_0 K_1 V_1 ..., across unit boundaries;
//   warp 4: one lane issues the MMAs, M 128: S = Q K^T (N 64) into one of two
//     buffers, so that the next tile's scores are made while the softmax is at
//     the last one's, and O += P V (N D) with P from tensor memory;
//   warps 0-3: softmax, one query row per thread, as in the prefill: P, the
//     sum and O are relative to a reference that moves only when a tile's
//     maximum passes it by 2^8; warps without a row of the unit skip the
//     arithmetic.  They also lay a unit's Q into shared memory (any G: the
//     rows are gathered) and write its results.
// Rest units fill only G of the 128 rows; a 64-key tile's MMAs then take about
// 0.27 us of an SM's tensor pipe against 0.73 us of its share of the memory
// rate (D 128), so the idle rows cost no time.

#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "tcgen05.cuh"

namespace pagedkv {
namespace {

constexpr int kSpRows = 128;   // MMA M: query rows of a unit
constexpr int kSpKeys = 64;    // keys per tile: N of S, K of P V
constexpr int kSpSoftWarps = 4;
constexpr int kSpMmaWarp = kSpSoftWarps, kSpTmaWarp = kSpSoftWarps + 1;
constexpr int kSpThreads = 32 * (kSpSoftWarps + 2);
constexpr uint32_t kSpCols = 256;  // S buffers at columns 0 and 64 (P over the first half of each), O at 128
// At least three stages: a thread that waits for a tile's V then knows that
// what the stage held before has landed (with two it would be the V of the
// tile before, whose P V may not have run), so its parity wait is one phase
// behind at most.
constexpr int kSpMinStages = 3, kSpMaxStages = 8;
constexpr int kSpMaxSeqs = 4096;
// Tiles' worth of time that a unit costs beyond its tiles (its Q, the
// pipeline's turn-round, its partial result).
constexpr int kSpUnitCost = 3;

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
  int32_t stages;
  float scale_log2;  // scale * log2(e)
  int32_t num_ctas;
  // workspace
  float* unit_o;    // [2][B][Hq][D] whole units: prefix, rest
  float* unit_ml;   // [2][B][Hq][2] (reference, sum)
  float* cut_o;     // [CTA][2][kSpRows][D] pieces of units cut by a CTA's share: its first, its last
  float* cut_ml;    // [CTA][2][kSpRows][2]
  int4* pre_span;   // [B][Hkv] first and last CTA of the sequence's prefix unit, its first row there
  int4* rest_span;  // [B][Hkv] the same of its rest unit
  int2* seq;        // [B] (tokens taken from the prefix unit, length)
};

template <int D>
struct SpLayout {
  static constexpr int kSlabs = D / 64;
  static constexpr int kQSlab = kSpRows * 128;  // 64 dims of the 128 rows
  static constexpr int kQ = kSlabs * kQSlab;
  static constexpr int kSlab = kSpKeys * 128;   // 64 dims of a tile's 64 keys
  static constexpr int kTile = kSlabs * kSlab;
  static constexpr int kBars = 256;
  static int bytes(int stages, int num_seqs, int num_groups) {
    return 1024 + kQ + stages * kTile + kBars + 4 * (3 * num_seqs + 3 * num_groups + 2);
  }
};

// The line of units, in shared memory.
struct SpLine {
  int* cum;    // [groups + seqs + 1] cost per kv head before each entity (a group's prefix units, a sequence's rest)
  int* start;  // [groups + 1] group_start
  int* prefix;  // [groups] tokens of the group's prefix that are shared (whole blocks)
  int* first;  // [seqs] tokens the sequence takes from its group's prefix unit
  int* len;    // [seqs]
};

struct SpUnit {
  int b0, rows;    // first sequence, query rows
  int kvh;
  int key0, key1;  // keys
  int t0, t1, T;   // tiles of it in this CTA, its tiles in all
  int64_t base;    // its place on the line
  bool prefix;
};

// Walks the units of CTA pid's share in order.  Every role of the CTA walks
// for itself.
struct SpWalk {
  const SpParams& p;
  const SpLine& ln;
  int64_t x, x1, base;
  int e, u, units, cs, rt_n, n;

  __device__ __forceinline__ SpWalk(const SpParams& p_, const SpLine& ln_, int64_t x0_, int64_t x1_)
      : p(p_), ln(ln_), x(x0_), x1(x1_), base(0), e(0), u(0), units(0), cs(1), rt_n(1), n(1) {
    int lo = 0, hi = p.num_groups + p.num_seqs - 1;  // the last entity that begins at or before x: it is not empty
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (static_cast<int64_t>(p.num_kv_heads) * ln.cum[mid] <= x) lo = mid; else hi = mid - 1;
    }
    enter(lo);
    u = static_cast<int>((x - base) / cs);
    base += static_cast<int64_t>(u) * cs;
  }
  __device__ __forceinline__ void enter(int e_) {
    e = e_;
    u = 0;
    const int per_head = ln.cum[e + 1] - ln.cum[e];
    rt_n = 1;
    n = 1;
    if (e < p.num_groups) {
      n = ln.start[e + 1] - ln.start[e];
      rt_n = (n + p.tile_seqs - 1) / p.tile_seqs;
    }
    cs = per_head / rt_n;
    units = p.num_kv_heads * rt_n;
    base = static_cast<int64_t>(p.num_kv_heads) * ln.cum[e];
  }
  // The next unit with a tile in the share, or false.
  __device__ __forceinline__ bool next(SpUnit& s) {
    while (x < x1) {
      s.T = cs - kSpUnitCost;
      s.t0 = static_cast<int>(max(static_cast<int64_t>(0), x - base - kSpUnitCost));
      s.t1 = static_cast<int>(min(static_cast<int64_t>(s.T), x1 - base - kSpUnitCost));
      s.base = base;
      s.kvh = u / rt_n;
      if (e < p.num_groups) {
        const int rt = u - s.kvh * rt_n;
        s.prefix = true;
        s.b0 = ln.start[e] + rt * p.tile_seqs;
        s.rows = min(p.tile_seqs, n - rt * p.tile_seqs) * p.group;
        s.key0 = 0;
        s.key1 = ln.prefix[e];
      } else {
        s.prefix = false;
        s.b0 = e - p.num_groups;
        s.rows = p.group;
        s.key0 = ln.first[s.b0];
        s.key1 = ln.len[s.b0];
      }
      base += cs;
      x = base;
      if (++u == units && x < x1) {
        int en = e + 1;
        const int E = p.num_groups + p.num_seqs;
        while (en < E && ln.cum[en + 1] == ln.cum[en]) ++en;
        if (en < E) enter(en);
        else x1 = x;
      }
      if (s.t1 > s.t0) return true;
    }
    return false;
  }
};

// The CTA whose share [c W / P, (c + 1) W / P) holds place t.
__device__ __forceinline__ int sp_cta_of(int64_t t, int64_t W, int P) {
  return static_cast<int>(((t + 1) * P + W - 1) / W - 1);
}

// 32-byte store: a thread's piece of its row is a whole sector.
__device__ __forceinline__ void st_global_32b(float* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

__device__ __forceinline__ int sp_len(const SpParams& p, int b) {
  int L = __ldg(p.seq_lens + b);
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  if (L < 0 || L > cap) {
    record_error(KV_ERR_DEVICE_BOUNDS);
    L = L < 0 ? 0 : static_cast<int>(cap);
  }
  return L;
}

// Registers: two CTAs of six warps, at most 168 a thread (as the prefill).
template <typename T, int D>
__global__ void __launch_bounds__(kSpThreads, 2)
    shared_prefix_kernel(const SpParams p, const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV) {
  using Lay = SpLayout<D>;
  constexpr int kSlabs = Lay::kSlabs;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t sp_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(sp_smem_raw) + 1023) & ~uintptr_t(1023));
  const int nst = p.stages;
  uint8_t* ring = sm + Lay::kQ;
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(ring + nst * Lay::kTile);  // [stage] tile landed
  uint64_t* bar_empty = bar_full + kSpMaxStages;  // [stage] its MMAs done
  uint64_t* bar_q = bar_empty + kSpMaxStages;     // a unit's Q laid down (every softmax thread)
  uint64_t* bar_o = bar_q + 1;                    // a unit's O read (every softmax thread)
  uint64_t* bar_s = bar_o + 1;                    // [2] S written
  uint64_t* bar_p = bar_s + 2;                    // [2] P written (every softmax thread)
  uint64_t* bar_pv = bar_p + 2;                   // [2] P V done
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bar_pv + 2);
  const int B = p.num_seqs, NG = p.num_groups, E = NG + B;
  SpLine ln;
  ln.cum = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(bar_full) + Lay::kBars);
  ln.start = ln.cum + E + 1;
  ln.prefix = ln.start + NG + 1;
  ln.first = ln.prefix + NG;
  ln.len = ln.first + B;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int bs = p.block_size;

  if (tid == 0) {
    for (int s = 0; s < nst; ++s) {
      mbar_init(bar_full + s, 1);
      mbar_init(bar_empty + s, 1);
    }
    mbar_init(bar_q, kSpSoftWarps * 32);
    mbar_init(bar_o, kSpSoftWarps * 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, kSpSoftWarps * 32);
      mbar_init(bar_pv + i, 1);
    }
    fence_mbar_init();
  }
  if (warp == kSpTmaWarp && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kSpMmaWarp) tc::alloc(tmem_slot, kSpCols);

  // ---- the line: lengths, groups, costs, their prefix sums (all global
  // loads before the first barrier)
  int bad = 0;
  for (int g = tid; NG > 0 && g <= NG; g += kSpThreads) {
    const int s = __ldg(p.group_start + g), nx = g < NG ? __ldg(p.group_start + g + 1) : B;
    if (g < NG) ln.prefix[g] = __ldg(p.prefix_lens + g);
    ln.start[g] = s;
    if (s < 0 || s > nx || nx > B || (g == 0 && s != 0) || (g == NG && s != B)) bad = 1;
  }
  for (int b = tid; b < B; b += kSpThreads) ln.len[b] = sp_len(p, b);
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) record_error(KV_ERR_DEVICE_BOUNDS);  // no group: every sequence reads its whole table
  for (int g = tid; g < NG; g += kSpThreads) {
    int P = 0, cost = 0;
    if (!bad) {
      const int n = ln.start[g + 1] - ln.start[g];
      if (ln.prefix[g] < 0) record_error(KV_ERR_DEVICE_BOUNDS);
      if (n > 1) {  // a group of one shares with nobody
        P = max(0, min(ln.prefix[g], ln.len[ln.start[g]])) / bs * bs;
        if (P > 0)
          cost = (n + p.tile_seqs - 1) / p.tile_seqs * ((P + kSpKeys - 1) / kSpKeys + kSpUnitCost);
      }
    }
    ln.prefix[g] = P;
    ln.cum[g + 1] = cost;
  }
  __syncthreads();
  for (int b = tid; b < B; b += kSpThreads) {
    int first = 0;
    const int L = ln.len[b];
    if (!bad && NG > 0) {
      int lo = 0, hi = NG - 1;  // the last group that begins at or before b
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (ln.start[mid] <= b) lo = mid; else hi = mid - 1;
      }
      // a sequence shorter than its group's prefix (an empty slot of the
      // batch) reads its own table
      if (L >= ln.prefix[lo]) first = ln.prefix[lo];
    }
    ln.first[b] = first;
    ln.cum[NG + b + 1] = L > first ? (L - first + kSpKeys - 1) / kSpKeys + kSpUnitCost : 0;
    if (b % gridDim.x == blockIdx.x) p.seq[b] = make_int2(first, L);
  }
  __syncthreads();
  {
    const int per = (E + kSpThreads - 1) / kSpThreads;
    const int beg = min(E, tid * per), end = min(E, beg + per);
    int local = 0;
    for (int i = beg; i < end; ++i) local += ln.cum[i + 1];
    int incl = local;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += y;
    }
    __shared__ int warp_tot[kSpThreads / 32];
    if (lane == 31) warp_tot[warp] = incl;
    if (tid == 0) ln.cum[0] = 0;
    __syncthreads();
    int run = incl - local;
    for (int w = 0; w < warp; ++w) run += warp_tot[w];
    for (int i = beg; i < end; ++i) {
      run += ln.cum[i + 1];
      ln.cum[i + 1] = run;
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  const int64_t W = static_cast<int64_t>(p.num_kv_heads) * ln.cum[E];
  const int P = static_cast<int>(min(static_cast<int64_t>(gridDim.x), W)), pid = blockIdx.x;
  const int64_t x0 = pid < P ? pid * W / P : 0, x1 = pid < P ? (pid + 1) * W / P : 0;

  // the merge kernel may be launched into what this one leaves free; it waits
  // for this grid's end itself
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (x0 < x1) {
    SpWalk walk(p, ln, x0, x1);
    SpUnit s;
    if (warp == kSpTmaWarp) {
      // ---- K and V tiles, one box of up to 64 rows per (block, 64-dim slab)
      const int rpc = min(bs, kSpKeys);  // rows of a box
      const int ci = lane / kSlabs, slab = lane % kSlabs;
      // table entry of this lane's box of tile t and the box's offset in the
      // block (-1: no box); the entry is looked at only when the box is copied
      auto entry = [&](const SpUnit& un, int t, int& off) -> int {
        const int tok = un.key0 + t * kSpKeys + ci * rpc;
        off = -1;
        if (ci * rpc >= kSpKeys || tok >= un.key1) return 0;
        const int blk = tok / bs;
        off = tok - blk * bs;
        return __ldg(p.block_tables + static_cast<int64_t>(un.b0) * p.max_blocks_per_seq + blk);
      };
      // advances (unit, tile); false past the share's end
      auto step = [&](SpUnit& un, int& t) -> bool {
        if (++t < un.t1) return true;
        if (!walk.next(un)) return false;
        t = un.t0;
        return true;
      };
      // the table entries of two tiles are in flight ahead of their copies
      bool more = walk.next(s);
      int t = s.t0, ok = 1, i = 0;
      int off = -1, off1 = -1, off2 = -1;
      int pb = more ? entry(s, t, off) : 0, kvh = s.kvh;
      bool more1 = more && step(s, t);
      int pb1 = more1 ? entry(s, t, off1) : 0, kvh1 = s.kvh;
      while (more && ok) {
        const bool more2 = more1 && step(s, t);
        off2 = -1;
        const int pb2 = more2 ? entry(s, t, off2) : 0, kvh2 = s.kvh;
        const int boxes = __popc(__ballot_sync(0xffffffffu, off >= 0));
        if (off >= 0 && (pb < 0 || pb >= p.num_blocks)) {
          record_error(KV_ERR_DEVICE_BOUNDS);
          pb = 0;
        }
        const int row = pb * bs + off;
        for (int v = 0; v < 2 && ok; ++v, ++i) {
          const int st = i % nst;
          if (lane == 0) {
            if (i >= nst) ok = mbar_wait_bounded(bar_empty + st, (i / nst - 1) & 1);
            if (ok) mbar_arrive_expect_tx(bar_full + st, static_cast<uint32_t>(boxes * rpc * 128));
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (ok && off >= 0)
            tma_load_3d(ring + st * Lay::kTile + slab * Lay::kSlab + ci * rpc * 128, v ? &tmV : &tmK, bar_full + st,
                        slab * 64, kvh, row);
        }
        pb = pb1, off = off1, kvh = kvh1, more = more1;
        pb1 = pb2, off1 = off2, kvh1 = kvh2, more1 = more2;
      }
      // every stage's last MMAs have completed: no copy or commit in flight at exit
      if (lane == 0 && ok)
        for (int k = max(0, i - nst); k < i; ++k) mbar_wait_bounded(bar_empty + k % nst, (k / nst) & 1);
    } else if (warp == kSpMmaWarp) {
      if (lane == 0) {
        // ---- MMA issue
        constexpr uint32_t idS = tc::idesc_f16(kBf16, kSpRows, kSpKeys, false);
        constexpr uint32_t idPV = tc::idesc_f16(kBf16, kSpRows, D, true);
        const uint32_t aQ = smem_u32(sm), ring_a = smem_u32(ring);
        // S of tile j (first: of unit number un) once its K, the unit's Q
        // and its buffer (P V of tile j - 2 done) are ready
        auto issue_s = [&](int j, bool first, int un) -> bool {
          const int i = 2 * j, st = i % nst;
          if (first && !mbar_wait_bounded(bar_q, un & 1)) return false;
          if (!mbar_wait_bounded(bar_full + st, (i / nst) & 1)) return false;
          if (j >= 2 && !mbar_wait_bounded(bar_pv + (j & 1), ((j >> 1) - 1) & 1)) return false;
          tc::fence_after();
          const uint32_t kb = ring_a + st * Lay::kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            tc::mma_f16(tmem + (j & 1) * 64,
                        tc::sdesc_sw128(aQ + (kk >> 2) * Lay::kQSlab + (kk & 3) * 32, 16, 1024),
                        tc::sdesc_sw128(kb + (kk >> 2) * Lay::kSlab + (kk & 3) * 32, 16, 1024), idS, kk > 0);
          tc::commit(bar_s + (j & 1));
          tc::commit(bar_empty + st);
          return true;
        };
        auto issue_pv = [&](int j, bool first, int un) -> bool {
          const int i = 2 * j + 1, st = i % nst;
          if (!mbar_wait_bounded(bar_full + st, (i / nst) & 1)) return false;
          // P lands after the softmax warps have zeroed a last tile's V tail
          if (!mbar_wait_bounded(bar_p + (j & 1), (j >> 1) & 1)) return false;
          if (first && un > 0 && !mbar_wait_bounded(bar_o, (un - 1) & 1)) return false;
          tc::fence_after();
          const uint32_t vb = ring_a + st * Lay::kTile;
#pragma unroll
          for (int kk = 0; kk < kSpKeys / 16; ++kk)
            tc::mma_f16_ts(tmem + 128, tmem + (j & 1) * 64 + kk * 8,
                           tc::sdesc_sw128(vb + kk * 16 * 128, Lay::kSlab, 1024), idPV, (!first || kk > 0) ? 1u : 0u);
          tc::commit(bar_pv + (j & 1));
          tc::commit(bar_empty + st);
          return true;
        };
        bool more = walk.next(s);
        int t = s.t0, j = 0, un = 0;
        bool ok = more && issue_s(0, true, 0);
        while (ok) {
          const bool last = t + 1 == s.t1;
          if (!last) ok = issue_s(j + 1, false, un);
          ok = ok && issue_pv(j, t == s.t0, un);
          ++j;
          ++t;
          if (last) {
            if (!walk.next(s)) break;
            t = s.t0;
            ++un;
            ok = ok && issue_s(j, true, un);
          }
        }
      }
    } else {
      // ---- softmax: thread r owns query row r
      const int r = tid;
      const uint32_t tS = tmem + (static_cast<uint32_t>(warp * 32) << 16), tO = tS + 128;
      const float c2 = p.scale_log2;
      const uint64_t c2x2 = tc::f2(c2, c2);
      constexpr float kSlack = 8.f, kLow = 8.f;  // as the prefill: P stays <= 2^8, and not all tiny
      bool ok = true;
      // A unit's Q goes to shared memory in the MMA's swizzled layout, 16-byte
      // chunk i of the rows by thread i mod 128, loads in batches of kQBatch.
      // The first batch (all of a rest unit's Q when G D <= 2048) is fetched
      // while the unit before is still at work.
      constexpr int kCh = D / 8, kQBatch = 2;
      uint4 qv[kQBatch];
      auto fetch_q = [&](const SpUnit& un, int i0) {
#pragma unroll
        for (int k = 0; k < kQBatch; ++k) {
          const int i = i0 + k * kSpSoftWarps * 32;
          if (i < un.rows * kCh) {
            const int row = i / kCh, sq = row / p.group;
            qv[k] = __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(p.q) +
                                                         (static_cast<int64_t>(un.b0 + sq) * p.num_heads +
                                                          un.kvh * p.group + row - sq * p.group) * D) +
                          i % kCh);
          }
        }
      };
      auto store_q = [&](const SpUnit& un) {
        for (int i0 = tid;; ) {
#pragma unroll
          for (int k = 0; k < kQBatch; ++k) {
            const int i = i0 + k * kSpSoftWarps * 32;
            if (i < un.rows * kCh) {
              const int row = i / kCh, ch = i % kCh;
              *reinterpret_cast<uint4*>(sm + (ch >> 3) * Lay::kQSlab + row * 128 + (((ch & 7) ^ (row & 7)) << 4)) =
                  qv[k];
            }
          }
          i0 += kQBatch * kSpSoftWarps * 32;
          if (i0 >= un.rows * kCh) break;
          fetch_q(un, i0);
        }
        fence_proxy_async_smem();  // read by the tensor cores
        mbar_arrive(bar_q);
      };
      bool more = walk.next(s);
      if (more) {
        fetch_q(s, tid);
        store_q(s);
      }
      int j = 0;
      while (more) {
        const bool mine = warp * 32 < s.rows, valid = r < s.rows;
        SpUnit nx;
        bool nmore = false;
        float m_ref = 0.f, l = 0.f;
        for (int t = s.t0; t < s.t1; ++t, ++j) {
          const int buf = (j & 1) * 64;
          if (t + 1 == s.t1) {
            nmore = walk.next(nx);
            if (nmore) fetch_q(nx, tid);
          }
          // after a timeout (recorded) the remaining waits are skipped
          if (ok && !mbar_wait_bounded(bar_s + (j & 1), (j >> 1) & 1)) ok = false;
          tc::fence_after();
          const int keys = min(kSpKeys, s.key1 - s.key0 - t * kSpKeys);
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
                  softmax_pair<T>(tc::f2_split(tc::ffma2(
                                      tc::f2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), c2x2, negm)),
                                  i, ma, mb, ls, x);
              }
              me = fmaxf(ma, mb);
              if (attempt == 1) break;
              const bool need = valid && (me > kSlack || (l == 0.f && me != -INFINITY && me < -kLow));
              rescale = __any_sync(0xffffffffu, need);
              if (!rescale) break;
              const float m_new = need ? m_ref + me : m_ref;
              alpha = fast_exp2(m_ref - m_new);
              l *= alpha;
              m_ref = m_new;
            }
            tc::st_32x32b_x32(tS + buf, x);
            const float2 a = tc::f2_split(ls[0]), b2 = tc::f2_split(ls[1]);
            l += (a.x + a.y) + (b2.x + b2.y);
            if (rescale && t > s.t0) {
              // O holds the unit's tiles up to the last one: its P V is done
              if (ok && !mbar_wait_bounded(bar_pv + ((j - 1) & 1), ((j - 1) >> 1) & 1)) ok = false;
              tc::fence_after();
              const uint64_t a2 = tc::f2(alpha, alpha);
#pragma unroll
              for (int oc = 0; oc < D; oc += 32) {
                uint32_t w[32];
                tc::ld_32x32b_x32(tO + oc, w);
                tc::wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k += 2) {
                  const float2 y =
                      tc::f2_split(tc::fmul2(tc::f2(__uint_as_float(w[k]), __uint_as_float(w[k + 1])), a2));
                  w[k] = __float_as_uint(y.x);
                  w[k + 1] = __float_as_uint(y.y);
                }
                tc::st_32x32b_x32(tO + oc, w);
              }
            }
            tc::wait_st();
          }
          if (keys < kSpKeys) {
            // V rows past the last key (a block's tail, blocks not loaded) are
            // zeroed: their P is 0, and 0 times what lies there must be 0
            const int i = 2 * j + 1, st = i % nst;
            if (ok && !mbar_wait_bounded(bar_full + st, (i / nst) & 1)) ok = false;
            uint8_t* vt = ring + st * Lay::kTile;
#pragma unroll 1
            for (int k = keys * 8 * kSlabs + tid; k < kSpKeys * 8 * kSlabs; k += kSpSoftWarps * 32) {
              const int row = k / (8 * kSlabs), rest = k % (8 * kSlabs);
              *reinterpret_cast<uint4*>(vt + (rest >> 3) * Lay::kSlab + row * 128 + (rest & 7) * 16) =
                  make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
          }
          tc::fence_before();
          mbar_arrive(bar_p + (j & 1));
        }
        // all scores of the unit are read: the next unit's Q goes down while
        // the last P V runs
        const SpUnit d = s;
        const float m_out = m_ref, l_out = l;
        more = nmore;
        if (more) {
          s = nx;
          store_q(s);
        }
        if (ok && !mbar_wait_bounded(bar_pv + ((j - 1) & 1), ((j - 1) >> 1) & 1)) ok = false;
        tc::fence_after();
        const bool whole = d.t0 == 0 && d.t1 == d.T;
        const bool direct = whole && !d.prefix && d.key0 == 0;
        if (mine) {
          const int b = d.b0 + r / p.group, g = r % p.group, h = d.kvh * p.group + g;
          const int64_t orow = static_cast<int64_t>(b) * p.num_heads + h;
          const int64_t prow = (static_cast<int64_t>(pid) * 2 + (d.t0 == 0 ? 1 : 0)) * kSpRows + r;
          const int64_t urow = orow + (d.prefix ? 0 : static_cast<int64_t>(p.num_seqs) * p.num_heads);
          float* po = whole ? p.unit_o + urow * D : p.cut_o + prow * D;
          float* pml = whole ? p.unit_ml + urow * 2 : p.cut_ml + prow * 2;
          const float inv = l_out > 0.f ? __fdiv_rn(1.f, l_out) : 0.f;
#pragma unroll 1
          for (int oc = 0; oc < D; oc += 32) {
            uint32_t w[32];
            tc::ld_32x32b_x32(tO + oc, w);
            tc::wait_ld();
            if (valid && direct) {
              uint4* o4 = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + orow * D + oc);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                uint32_t y[4];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  y[c] = Mma<T>::pack(__uint_as_float(w[8 * k + 2 * c]) * inv,
                                      __uint_as_float(w[8 * k + 2 * c + 1]) * inv);
                o4[k] = make_uint4(y[0], y[1], y[2], y[3]);
              }
            } else if (valid) {
#pragma unroll
              for (int k = 0; k < 32; k += 8) st_global_32b(po + oc + k, w + k);
            }
          }
          if (valid && !direct) *reinterpret_cast<float2*>(pml) = make_float2(m_out, l_out);
          // the unit's first CTA says where its pieces lie, once per sequence
          if (valid && g == 0 && d.t0 == 0) {
            const int a1 = whole ? pid : sp_cta_of(d.base + kSpUnitCost + d.T - 1, W, P);
            (d.prefix ? p.pre_span : p.rest_span)[static_cast<int64_t>(b) * p.num_kv_heads + d.kvh] =
                make_int4(pid, a1, r, 0);
          }
        }
        tc::fence_before();
        mbar_arrive(bar_o);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kSpMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::dealloc(tmem, kSpCols);
  }
}

// Joins a row's pieces.  WPR warps per (sequence, query head): warp w of them
// takes pieces w, w + WPR, ..., a lane D / 32 outputs, and the first one adds
// up the others' in order.  A piece's statistics and its values are loaded
// together, so a row costs two round trips (where its pieces lie, what they
// hold).  Rows that the first kernel wrote whole are left alone; a sequence
// of no tokens gets zeros.  Launched early (programmatic dependent launch): it
// waits for the first kernel's end before it reads anything.
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int64_t at = static_cast<int64_t>(b) * p.num_kv_heads + kvh;
  const int2 sq = p.seq[b];  // tokens from the prefix unit, length
  int4 ps = p.pre_span[at], rs = p.rest_span[at];
  auto clamped = [&](int4 v) {  // CTAs in range whatever a call that timed out left there
    v.x = max(0, min(v.x, p.num_ctas - 1));
    v.y = max(v.x, min(v.y, p.num_ctas - 1));
    v.z = max(0, min(v.z, kSpRows - p.group));
    return v;
  };
  ps = sq.x > 0 ? clamped(ps) : make_int4(0, -1, 0, 0);
  rs = sq.y > sq.x ? clamped(rs) : make_int4(0, -1, 0, 0);
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
        // piece i: row of the whole units' array, or of a CTA's cut pieces
        // (the first CTA's is its last piece, the others' their first)
        const bool pre = i < np;
        const int4 s = pre ? ps : rs;
        const int c = pre ? i : i - np;
        const bool cut = s.x != s.y;
        const int64_t pr = cut ? (static_cast<int64_t>(s.x + c) * 2 + (c == 0 ? 1 : 0)) * kSpRows + s.z + g
                               : row + (pre ? 0 : static_cast<int64_t>(p.num_seqs) * p.num_heads);
        ml[k] = *reinterpret_cast<const float2*>((cut ? p.cut_ml : p.unit_ml) + pr * 2);
        const float* src = (cut ? p.cut_o : p.unit_o) + pr * D + lane * kV;
        if constexpr (kV == 4) *reinterpret_cast<float4*>(y[k]) = *reinterpret_cast<const float4*>(src);
        else *reinterpret_cast<float2*>(y[k]) = *reinterpret_cast<const float2*>(src);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      if (!(ml[k].y > 0.f)) continue;  // no such piece, or one without weight
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
      if (!(dk > 0.f)) continue;
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

// A layer's cache as a tensor {D, Hkv, slots}, boxes of 64 dims of one head
// in `box_rows` consecutive slots, 128-byte swizzle.
bool sp_map(const void* cache, int64_t slots, int hkv, int d, int box_rows, CUtensorMap* out) {
  auto fn = sp_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(hkv), static_cast<cuuint64_t>(slots)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(hkv) * d * 2};
  cuuint32_t box[3] = {64, 1, static_cast<cuuint32_t>(box_rows)};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT16, 3, const_cast<void*>(cache), dims, strides, box, estr,
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
         G <= kSpRows && B <= kSpMaxSeqs;
}
// The line's cost per kv head fits an int: at most 2 B units of the tiles of
// a whole table row and the charge.
bool sp_line_fits(int B, int64_t row_tokens) {
  return 2 * static_cast<int64_t>(B) * (row_tokens / kSpKeys + 1 + kSpUnitCost) < INT32_MAX;
}

size_t sp_align(size_t x) { return (x + 255) & ~size_t(255); }

struct SpWorkspace {
  size_t unit_o, unit_ml, cut_o, cut_ml, pre_span, rest_span, seq, bytes;
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
  const size_t cuts = static_cast<size_t>(ctas) * 2 * kSpRows;
  w.unit_o = take(2 * rows * D * 4);
  w.unit_ml = take(2 * rows * 2 * 4);
  w.cut_o = take(cuts * D * 4);
  w.cut_ml = take(cuts * 2 * 4);
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
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((rows + kRows - 1) / kRows));
  cfg.blockDim = dim3(kSpMergeWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, shared_merge_kernel<T, D, WPR>, p);
}

template <typename T, int D>
cudaError_t launch_shared(SpParams& p, const CUtensorMap& mk, const CUtensorMap& mv, int sms, cudaStream_t st) {
  using Lay = SpLayout<D>;
  // as many stages as fit beside the batch's line (4 at head_dim 128, 8 at 64,
  // for small batches); a batch whose line leaves no three gets an SM per CTA
  p.stages = D == 128 ? 4 : kSpMaxStages;
  while (p.stages > kSpMinStages && Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemTwo) --p.stages;
  int per_sm = 2;
  if (Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemTwo) {
    per_sm = 1;
    p.stages = D == 128 ? 4 : kSpMaxStages;
    while (p.stages > kSpMinStages && Lay::bytes(p.stages, p.num_seqs, p.num_groups) > kSpSmemOne) --p.stages;
  }
  const int smem = Lay::bytes(p.stages, p.num_seqs, p.num_groups);
  p.num_ctas = sms * per_sm;
  auto kern = shared_prefix_kernel<T, D>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpSmemOne);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, 100);
  if (e != cudaSuccess) return e;
  kern<<<p.num_ctas, kSpThreads, smem, st>>>(p, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // few rows: up to eight warps join one
  const int64_t rows = static_cast<int64_t>(p.num_seqs) * p.num_heads;
  if (rows * 8 <= static_cast<int64_t>(sms) * 64) return launch_merge<T, D, 8>(p, rows, st);
  if (rows * 2 <= static_cast<int64_t>(sms) * 64) return launch_merge<T, D, 2>(p, rows, st);
  return launch_merge<T, D, 1>(p, rows, st);
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
      !sp_line_fits(num_seqs, static_cast<int64_t>(max_blocks_per_seq) * block_size))
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
  const int sms = sp_sm_count();
  const SpWorkspace w = sp_workspace(num_seqs, num_heads, num_kv_heads, head_dim, 2 * sms);
  char* ws = static_cast<char*>(workspace);
  p.unit_o = reinterpret_cast<float*>(ws + w.unit_o);
  p.unit_ml = reinterpret_cast<float*>(ws + w.unit_ml);
  p.cut_o = reinterpret_cast<float*>(ws + w.cut_o);
  p.cut_ml = reinterpret_cast<float*>(ws + w.cut_ml);
  p.pre_span = reinterpret_cast<int4*>(ws + w.pre_span);
  p.rest_span = reinterpret_cast<int4*>(ws + w.rest_span);
  p.seq = reinterpret_cast<int2*>(ws + w.seq);
  CUtensorMap mk, mv;
  const int64_t slots = num_blocks * block_size;
  const int box = std::min(block_size, kSpKeys);
  if (!sp_map(k_cache, slots, num_kv_heads, head_dim, box, &mk) ||
      !sp_map(v_cache, slots, num_kv_heads, head_dim, box, &mv))
    return cuda_status(cudaErrorInvalidValue, "cuTensorMapEncodeTiled failed");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dtype == KV_DTYPE_F16)
    e = head_dim == 64 ? launch_shared<__half, 64>(p, mk, mv, sms, st) : launch_shared<__half, 128>(p, mk, mv, sms, st);
  else
    e = head_dim == 64 ? launch_shared<__nv_bfloat16, 64>(p, mk, mv, sms, st)
                       : launch_shared<__nv_bfloat16, 128>(p, mk, mv, sms, st);
  return cuda_status(e);
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
