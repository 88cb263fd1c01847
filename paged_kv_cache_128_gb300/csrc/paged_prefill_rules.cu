// Chunked-prefill attention under score rules (score_rules.cuh): capped
// scores, a bias that falls with the distance, windows, documents and spans
// seen both ways, each query row over its own interval of keys.

#include <algorithm>
#include <cfloat>
#include <type_traits>

#include "prefill_common.cuh"

namespace pagedkv {
namespace {

// ---------------------------------------------------------------------------
// Tensor-core (tcgen05) kernel under rules, for block sizes that divide 128
// and are multiples of 16.
//
// Persistent CTAs, one per SM, walk items (head group, sequence, pair of row
// tiles).  An item is two 128-row query tiles over one stream of 128-key tiles:
// each K and V tile is loaded once for both, and one tile's softmax runs while
// the tensor cores work for the other.  Rows are packed as in the plain
// kernel: HG query heads of one kv head (the largest power of two dividing the
// group, at most 8) times 128 / HG tokens.
//
// Each row sees an interval of keys, so a query tile needs the key tiles from
// the smallest first key of its rows to their largest end; what neither tile
// of the pair needs is not loaded.  The key tiles are walked from the last to
// the first: under a falling bias, and in causal attention, a row's largest
// scores then tend to come first, and the softmax reference, which moves only
// when a tile's weights have outgrown it, stays where it is.
//
// Tensor memory (512 columns): S of the two tiles at 0 and 128 (P, two keys to
// a column, over the upper half of its S), O at 256 and 256 + D.
//   warp 17, scheduler and TMA producer: works out an item's ranges, hands them
//     to the others through a two-deep ring in shared memory, and loads Q and
//     the K tiles (one box per block and 64-dim slab, a lane each) into a ring of
//     slots, running ahead into the next item; warp 18 does so for the V tiles;
//   warp 16 issues, for each key tile and for the two query tiles in turn, O +=
//     P V of the previous key tile and S = Q K^T of this one (a warp for each
//     query tile was slower, 558 us for 500: their MMAs interleave, both softmaxes
//     run at once and the tensor cores wait for both);
//   warps 0-7 and 8-15: the softmax of the first and second query tile, half a
//     row's keys per thread.
// V rows that lie in no row's interval are cleared before P V reads them: the
// warp that loads a V tile notes which of its keys some row of the pair sees.
// Where few rows see many keys an item's key tiles are cut into pieces, whose
// parts join_pieces_kernel joins.
//
// What bounds it: no pipe alone.  A key tile costs a pair some 3300 cycles, of
// which the tensor cores work 2050; the chain of one query tile, S (500), softmax
// (1100; with a cap 2200) and P V (650), is 2250 long and the two run side by side,
// so that a thousand cycles are accounted for by neither.  Measured: 8192 causal
// tokens of 32/8 heads of 128, bf16: 428 us, 1.28 PFLOP/s of the keys seen (0.68 of
// the measured peak), with a cap 517, with a bias 460, with both 628; a chunk of
// 8192 under a window of 4096, 28/4 heads: 388 us, 1.24 PFLOP/s.
// ---------------------------------------------------------------------------
constexpr int kRlSoftWarps = 8;  // per query tile: a row's keys are halved between two warps
constexpr int kRlMmaWarp = 2 * kRlSoftWarps, kRlTmaWarp = kRlMmaWarp + 1, kRlValueWarp = kRlTmaWarp + 1;
constexpr int kRlThreads = 32 * (kRlValueWarp + 1);
constexpr uint32_t kRlCols = 512;

// mbar_wait_bounded with the wait itself out of line: the many waits of this
// kernel's roles are short in its code then, and their instructions stay cached.
__device__ __noinline__ bool rl_wait_on(uint64_t* bar, uint32_t parity) { return mbar_wait_bounded(bar, parity); }
__device__ __forceinline__ bool rl_wait(uint64_t* bar, uint32_t parity) {
  return mbar_try_wait(bar, parity) || rl_wait_on(bar, parity);
}

template <int D>
struct RlLayout {
  static constexpr int kDeep = D == 64 ? 4 : 2;      // slots for K tiles, and for V tiles
  static constexpr int kRing = 2 * kDeep;            // tile n: K in slot n % kDeep, V kDeep further on
  static constexpr int kSlab = kTcRows * 128;        // one 64-column slab of 128 rows
  static constexpr int kTile = (D / 64) * kSlab;     // a Q, K or V tile
  static constexpr int kOffRing = 2 * kTile;         // after the two Q tiles
  static constexpr int kOffBar = kOffRing + kRing * kTile;
  static constexpr int kOffRow = kOffBar + 512;       // [query tile][half][row] floats: a half's maxima and sums
  static constexpr int kBytes = kOffRow + 2 * 2 * kTcRows * 4;
  static constexpr int kSmem = kBytes + 1024;        // slack for 1024-byte alignment
};

// An item as the scheduler hands it on.
struct RlItem {
  int seq;          // -1: no more items
  int q_row, n;     // first row of the sequence's chunk in q, its tokens
  int ctx, len;     // positions before the chunk, and in all
  int tok0, head0;  // first chunk token of the pair, first head of the group
  int key_lo, key_hi;          // from the first key that some row of the pair sees to the last
  int gaps;                    // there may be keys between that none sees
  int whole_lo, whole_hi;      // tiles all of whose keys some row sees (with gaps: none are said to be)
  int pieces, piece;           // what they are cut into, and which of it this is
  int first, end;              // its tiles, first down to end (none: first < end)
  int tile_lo[2], tile_hi[2];  // key tiles of each query tile in the piece (none: equal)
  int tile0;                   // tiles before the item's first
};

// What a launch costs, in key tiles' time, when items that need `work` tiles
// together and `longest` at most are cut into n pieces each: the longest piece or
// the mean of the CTAs, six tiles for a piece's start, end and parts, three for
// the join.
__host__ __device__ inline float rl_cost(float items, float work, float longest, int n, float ctas) {
  const float piece = longest / n + 6.f, mean = (work + 6.f * items * n) / ctas;
  return (piece > mean ? piece : mean) + (n > 1 ? 3.f : 0.f);
}

// The key tiles of an item as they are walked: first down to end, of which
// own() says whether query tile q needs one, other() whether the other one does.
struct RlSpan {
  int first, end, own_lo, own_hi, other_lo, other_hi, tile0;
  __device__ __forceinline__ RlSpan(const RlItem& it, int q)
      : first(it.first), end(it.end), own_lo(it.tile_lo[q]), own_hi(it.tile_hi[q]), other_lo(it.tile_lo[q ^ 1]),
        other_hi(it.tile_hi[q ^ 1]), tile0(it.tile0) {}
  __device__ __forceinline__ bool own(int kt) const { return kt >= own_lo && kt < own_hi; }
  __device__ __forceinline__ bool other(int kt) const { return kt >= other_lo && kt < other_hi; }
  __device__ __forceinline__ bool any(int kt) const { return own(kt) || other(kt); }
  __device__ __forceinline__ int below(int kt) const {  // the next tile down that either query tile needs
    do --kt;
    while (kt >= end && !any(kt));
    return kt;
  }
};

// sum += both halves of a packed pair, in float32.
template <typename T>
__device__ __forceinline__ void add_pair(float& sum, uint32_t w) {
  if constexpr (std::is_same<T, __nv_bfloat16>::value)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, l, %0;\n\tadd.rn.f32.bf16 %0, h, %0;\n\t}"
        : "+f"(sum)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.f16 %0, l, %0;\n\tadd.rn.f32.f16 %0, h, %0;\n\t}"
        : "+f"(sum)
        : "r"(w));
}

// One lane of the warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}

// Barrier `id` over `threads` threads, with the OR of their predicates.
__device__ __forceinline__ bool barrier_or(int id, int threads, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(id), "r"(threads)
      : "memory");
  return r != 0;
}

// The rows of a V tile whose bit in `keys` is not set, cleared by 256 threads;
// out of line, as tiles that need it are few.
template <int D>
__device__ __noinline__ void clear_unseen(uint8_t* tile, const uint4* keys, int thread) {
  constexpr int kChunks = D / 8;  // 16-byte chunks of a row
  const uint4 m = *keys;
  const uint32_t words[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (words[w] == 0xffffffffu) continue;
#pragma unroll
    for (int i = 0; i < 32 * kChunks; i += 2 * kTcRows) {
      const int key = (i + thread) / kChunks, rest = thread % kChunks;
      if (!(words[w] >> key & 1u))
        *reinterpret_cast<uint4*>(tile + (rest >> 3) * RlLayout<D>::kSlab + (w * 32 + key) * 128 + (rest & 7) * 16) =
            make_uint4(0, 0, 0, 0);
    }
  }
}

template <typename T, int D, bool CAP, bool BIAS>
__global__ void __launch_bounds__(kRlThreads, 1)
    prefill_rules_kernel(const RulesPrefillParams p, const __grid_constant__ CUtensorMap tmQ,
                         const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV) {
  using Lay = RlLayout<D>;
  constexpr int kSlabs = D / 64, kRing = Lay::kRing, kDeep = Lay::kDeep;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ uint8_t rl_smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(rl_smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bar_full = reinterpret_cast<uint64_t*>(sm + Lay::kOffBar);  // [kRing] tile landed
  uint64_t* bar_empty = bar_full + kRing;       // [kRing] tile read
  uint64_t* bar_qfull = bar_empty + kRing;      // Q landed
  uint64_t* bar_qempty = bar_qfull + 1;         // the item's last S done
  uint64_t* bar_s = bar_qempty + 1;             // [2] S written
  uint64_t* bar_p = bar_s + 2;                  // [2] P written (one arrival per softmax warp)
  uint64_t* bar_pv = bar_p + 2;                 // [2] P V done
  uint64_t* bar_o = bar_pv + 2;                 // [2] O read (one arrival per softmax warp)
  uint64_t* bar_item = bar_o + 2;               // [2] item slot filled
  uint64_t* bar_free = bar_item + 2;            // [2] item slot read (MMA, V and softmax warps)
  uint64_t* bar_end = bar_free + 2;             // after a wait ran out: all MMAs done
  RlItem* items = reinterpret_cast<RlItem*>(bar_end + 1);  // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(items + 2);
  uint4* seen = reinterpret_cast<uint4*>(sm + Lay::kOffBar + 512) - kDeep;  // [kDeep] keys of a V tile that are seen
  static_assert((2 * kRing + 15) * 8 + 2 * sizeof(RlItem) + 4 <= 512 - kDeep * 16, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hg = 1 << p.hg_log2, tpt = kTcRows >> p.hg_log2;  // heads and tokens of a row tile
  const int bs = p.block_size;

  if (warp == kRlTmaWarp && lane == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(bar_full + i, 1);
      mbar_init(bar_empty + i, 1);
    }
    mbar_init(bar_qfull, 1);
    mbar_init(bar_qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar_s + i, 1);
      mbar_init(bar_p + i, kRlSoftWarps);
      mbar_init(bar_pv + i, 1);
      mbar_init(bar_o + i, kRlSoftWarps);
      mbar_init(bar_item + i, 1);
      mbar_init(bar_free + i, 2 + 2 * kRlSoftWarps);
    }
    mbar_init(bar_end, 1);
    fence_mbar_init();
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == kRlMmaWarp) tc::alloc(tmem_slot, kRlCols);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp >= kRlTmaWarp) {
    // ---- TMA producers: one warp schedules and loads Q and K, the other V (a
    // copy per block and slab is issued at a time, so that one warp took longer
    // over the 32 copies of a K and a V tile of 16-token blocks than the tensor
    // cores over their products: 481 us, and 436 with two)
    const bool values = warp == kRlValueWarp;
    int loaded = 0;  // tiles
    bool ok = true;
    // a wait by lane 0 for the whole warp
    auto wait = [&](uint64_t* bar, int parity) {
      int w = 1;
      if (lane == 0) w = rl_wait(bar, parity);
      ok = __shfl_sync(0xffffffffu, w, 0) != 0;
      return ok;
    };
    // This lane's copy of a tile: slab lane % kSlabs of its block lane / kSlabs;
    // a tile has the blocks that hold keys key_lo .. key_hi - 1.
    const int my_blk = lane / kSlabs, my_slab = lane % kSlabs;
    // table entry of this lane's block in tile kt (-1: none)
    auto entry = [&](int seq, int key_lo, int key_hi, int kt) {
      const int blk = kt * (kTcKeys / bs) + my_blk;
      const bool in = my_blk < kTcKeys / bs && (blk + 1) * static_cast<int64_t>(bs) > key_lo &&
                      static_cast<int64_t>(blk) * bs < key_hi;
      int e = -1;
      if (in) {
        e = __ldg(p.block_tables + static_cast<int64_t>(seq) * p.max_blocks_per_seq + blk);
        if (e < 0 || e >= p.num_blocks) {
          record_error(KV_ERR_DEVICE_BOUNDS);
          e = 0;
        }
      }
      return e;
    };
    auto load = [&](const CUtensorMap* map, int kvh, int e, const uint4& keys) {
      const int slot = (values ? kDeep : 0) + loaded % kDeep;
      if (loaded >= kDeep && !wait(bar_empty + slot, ((loaded / kDeep) - 1) & 1)) return;
      if (!values && p.test_skip >= 0 && blockIdx.x == 0 && loaded == p.test_skip) {
        ok = false;  // test control: this tile never lands, and none after it
        return;
      }
      const int copies = __popc(__ballot_sync(0xffffffffu, e >= 0));
      if (lane == 0) {
        if (values) seen[slot - kDeep] = keys;
        mbar_arrive_expect_tx(bar_full + slot, static_cast<uint32_t>(copies * bs * 128));
      }
      __syncwarp();
      if (e >= 0)
        tma_load_3d(sm + Lay::kOffRing + slot * Lay::kTile + my_slab * Lay::kSlab + my_blk * bs * 128, map,
                    bar_full + slot, my_slab * 64, kvh, e * bs);
      ++loaded;
    };
    int q_loads = 0;
    if (values) {
      for (int k = 0;; ++k) {
        const int slot = k & 1;
        if (!wait(bar_item + slot, (k >> 1) & 1)) break;
        const RlSpan walk(items[slot], 0);
        const int seq = items[slot].seq, key_lo = items[slot].key_lo, key_hi = items[slot].key_hi;
        const int kvh = items[slot].head0 / p.group;
        const bool gaps = items[slot].gaps;
        const int tok0 = items[slot].tok0, rows = min(2 * tpt, items[slot].n - tok0), pos0 = items[slot].ctx + tok0,
                  len = items[slot].len;
        const int64_t row0 = static_cast<int64_t>(items[slot].q_row) + tok0;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free + slot);
        if (seq < 0) break;
        // a bit for each key of tile kt that some row of the pair sees
        auto seen_in = [&](int kt) {
          uint4 m = make_uint4(0, 0, 0, 0);
          auto add = [&](int lo, int hi) {
            lo -= kt * kTcKeys;
            hi -= kt * kTcKeys;
            m.x |= bits_between(lo, hi);
            m.y |= bits_between(lo - 32, hi - 32);
            m.z |= bits_between(lo - 64, hi - 64);
            m.w |= bits_between(lo - 96, hi - 96);
          };
          if (!gaps) {
            add(key_lo, key_hi);
          } else {
            for (int t = lane; t < rows; t += 32) {
              const KeySpan s = keys_seen(p.rules, row0 + t, pos0 + t, len);
              add(s.lo, s.hi);
            }
            m.x = __reduce_or_sync(0xffffffffu, m.x);
            m.y = __reduce_or_sync(0xffffffffu, m.y);
            m.z = __reduce_or_sync(0xffffffffu, m.z);
            m.w = __reduce_or_sync(0xffffffffu, m.w);
          }
          return m;
        };
        int kt = walk.below(walk.first + 1);
        int e = kt >= walk.end ? entry(seq, key_lo, key_hi, kt) : -1;
        while (kt >= walk.end && ok) {
          const int next = walk.below(kt);
          const int e_next = next >= walk.end ? entry(seq, key_lo, key_hi, next) : -1;
          load(&tmV, kvh, e, seen_in(kt));
          kt = next;
          e = e_next;
        }
        if (!ok) break;
      }
    } else {
      const int ngroups = p.num_heads >> p.hg_log2;
      int handed = 0;
      auto hand_on = [&](const RlItem& it) {
        const int slot = handed & 1;
        if (handed >= 2 && !wait(bar_free + slot, ((handed >> 1) - 1) & 1)) return;
        if (lane == 0) {
          items[slot] = it;
          mbar_arrive(bar_item + slot);
        }
        ++handed;
      };
      // Items in order: sequence by sequence, a sequence's pairs counted down
      // (the longest first), head groups innermost.  CTA c takes items c, c +
      // grid, ..., every other round in reverse, so that the sums even out.
      // Sequences are looked at 32 at a time, a lane each, and once: what has
      // no rows has no items, whatever max_query_len allows for.
      const int64_t reach = static_cast<int64_t>(p.row_tiles) * 2 * tpt;
      // lane's sequence: first row, rows, length, pairs of row tiles (0 of a bad one)
      int my_row = 0, my_n = 0, my_len = 0, my_pairs = 0;
      auto look = [&](int seq, bool report) {
        my_row = my_n = my_len = my_pairs = 0;
        if (seq >= p.num_seqs) return;
        my_row = __ldg(p.query_start + seq);
        my_n = __ldg(p.query_start + seq + 1) - my_row;
        my_len = __ldg(p.seq_lens + seq);
        const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) * bs;
        // rows past the reach of max_query_len are left uncomputed; the chunk must
        // lie inside its sequence and in q, the sequence in its table row
        const bool bad =
            my_n > 0 && (my_len < my_n || my_row < 0 || my_row + static_cast<int64_t>(my_n) > p.num_tokens);
        if (report && (bad || (my_n > 0 && (my_n > reach || my_len > cap)))) record_error(KV_ERR_DEVICE_BOUNDS);
        if (my_len > cap) my_len = static_cast<int>(cap);
        if (bad || my_n < 0 || my_len < my_n) my_n = 0;
        my_pairs = min(my_n / (2 * tpt) + (my_n % (2 * tpt) != 0), p.row_tiles);
      };
      // The pieces of each item's keys: up to those that the workspace has room
      // for, by the rule of rl_plan on the rows and lengths there are (the host
      // knows only the width of the table).
      int splits = 1;
      if (p.splits > 1) {
        float items = 0.f, work = 0.f, longest = 0.f;
        for (int b0 = 0; b0 < p.num_seqs; b0 += 32) {
          look(b0 + lane, false);
          // keys of the sequence's last pair of row tiles and of its first
          int64_t most = my_len, least = my_len - my_n + 2 * tpt;
          if (p.rules.window > 0) most = min(most, p.rules.window + 2 * static_cast<int64_t>(tpt));
          least = min(least, most);
          const float last = static_cast<float>((most + kTcKeys - 1) / kTcKeys);
          items += my_pairs;
          work += my_pairs * 0.5f * (last + static_cast<float>((least + kTcKeys - 1) / kTcKeys));
          if (my_pairs > 0) longest = fmaxf(longest, last);
        }
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          items += __shfl_xor_sync(0xffffffffu, items, off);
          work += __shfl_xor_sync(0xffffffffu, work, off);
          longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, off));
        }
        const int n = lane + 1;
        uint32_t key = 0xffffffffu;  // the least cost (positive: in the order of its bits), then the fewest pieces
        if (n <= p.splits && (n == 1 || 2 * n <= longest))
          key = (__float_as_uint(rl_cost(items * ngroups, work * ngroups, longest, n, gridDim.x)) & ~31u) | lane;
        splits = static_cast<int>(__reduce_min_sync(0xffffffffu, key) & 31) + 1;
        if (blockIdx.x == 0 && lane == 0) *p.ws_pieces = splits;
      }
      const int64_t per_pair = static_cast<int64_t>(ngroups) * splits;
      int64_t round = 0, before = 0;  // items of the sequences before this chunk of 32
      auto item_of = [&](int64_t r) {
        return r * gridDim.x + ((r & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
      };
      for (int b0 = 0; b0 < p.num_seqs && ok; b0 += 32) {
        look(b0 + lane, blockIdx.x == 0);
        int64_t upto = static_cast<int64_t>(my_pairs) * per_pair;  // items up to and with this lane's sequence
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
          const int64_t y = __shfl_up_sync(0xffffffffu, upto, off);
          if (lane >= off) upto += y;
        }
        upto += before;
        const int64_t end = __shfl_sync(0xffffffffu, upto, 31);
        for (; item_of(round) < end && ok; ++round) {
          const int64_t x = item_of(round);
          const int src = __ffs(__ballot_sync(0xffffffffu, x < upto)) - 1;  // the lane whose sequence x lies in
          const int pairs = __shfl_sync(0xffffffffu, my_pairs, src);
          const int64_t rel = x - (__shfl_sync(0xffffffffu, upto, src) - static_cast<int64_t>(pairs) * per_pair);
          const int b = b0 + src, gi = static_cast<int>(rel % per_pair / splits);
          const int pair = pairs - 1 - static_cast<int>(rel / per_pair);
          RlItem it;
          it.seq = b;
          it.pieces = splits;
          it.piece = static_cast<int>(rel % splits);
          it.q_row = __shfl_sync(0xffffffffu, my_row, src);
          it.n = __shfl_sync(0xffffffffu, my_n, src);
          it.len = __shfl_sync(0xffffffffu, my_len, src);
          it.tok0 = pair * 2 * tpt;
          it.head0 = gi * hg;
          it.ctx = it.len - it.n;
          it.key_lo = INT32_MAX;
          it.key_hi = 0;
          it.gaps = 0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const int t0 = it.tok0 + q * tpt, t1 = min(t0 + tpt, it.n);
            int lo = INT32_MAX, hi = 0;
            if (p.rules.key_begin || p.rules.key_end) {
              for (int t = t0 + lane; t < t1; t += 32) {
                const KeySpan s = keys_seen(p.rules, static_cast<int64_t>(it.q_row) + t, it.ctx + t, it.len);
                if (s.lo < s.hi) {
                  lo = min(lo, s.lo);
                  hi = max(hi, s.hi);
                }
                // where every row's interval meets the next one's, all keys between
                // the pair's first and last are seen
                if (t + 1 < min(it.tok0 + 2 * tpt, it.n)) {
                  const KeySpan u =
                      keys_seen(p.rules, static_cast<int64_t>(it.q_row) + t + 1, it.ctx + t + 1, it.len);
                  if (s.lo >= s.hi || u.lo >= u.hi || s.lo > u.hi || u.lo > s.hi) it.gaps = 1;
                }
              }
              it.gaps = __any_sync(0xffffffffu, it.gaps);
              lo = __reduce_min_sync(0xffffffffu, lo);
              hi = __reduce_max_sync(0xffffffffu, hi);
            } else if (t0 < t1) {  // a window's ends move with the row
              lo = keys_seen(p.rules, 0, it.ctx + t0, it.len).lo;
              hi = keys_seen(p.rules, 0, it.ctx + t1 - 1, it.len).hi;
            }
            it.tile_lo[q] = lo < hi ? lo / kTcKeys : 0;
            it.tile_hi[q] = lo < hi ? (hi + kTcKeys - 1) / kTcKeys : 0;
            if (lo < hi) {
              it.key_lo = min(it.key_lo, lo);
              it.key_hi = max(it.key_hi, hi);
            }
          }
          // The piece: an equal share of the tiles, of which each query tile has
          // what it needs; first and end are tiles that one of them needs.  An item
          // of fewer tiles has fewer pieces, the rest are empty.
          it.first = -1;
          it.end = 0;
          it.whole_lo = it.gaps ? INT32_MAX : it.key_lo / kTcKeys + (it.key_lo % kTcKeys != 0);
          it.whole_hi = it.key_hi / kTcKeys;
          if (it.key_lo < it.key_hi) {
            const int lowest = it.key_lo / kTcKeys, tiles = (it.key_hi + kTcKeys - 1) / kTcKeys - lowest;
            const int pieces = min(splits, max(1, tiles / 2)), at = min(it.piece, pieces);
            const int from = lowest + static_cast<int>(static_cast<int64_t>(tiles) * at / pieces);
            const int to = lowest + static_cast<int>(static_cast<int64_t>(tiles) * min(at + 1, pieces) / pieces);
            int end = INT32_MAX;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              it.tile_lo[q] = max(it.tile_lo[q], from);
              it.tile_hi[q] = min(it.tile_hi[q], to);
              if (it.tile_lo[q] < it.tile_hi[q]) {
                end = min(end, it.tile_lo[q]);
                it.first = max(it.first, it.tile_hi[q] - 1);
              } else {
                it.tile_lo[q] = it.tile_hi[q] = 0;
              }
            }
            if (it.first >= 0) it.end = end;
          }
          it.tile0 = loaded;
          hand_on(it);
          if (!ok || it.first < it.end) continue;
          const int kvh = it.head0 / p.group;
          const RlSpan walk(it, 0);
          int kt = walk.below(walk.first + 1);
          int e = entry(b, it.key_lo, it.key_hi, kt);
          bool first = true;
          while (kt >= walk.end && ok) {
            const int next = walk.below(kt);
            const int e_next = next >= walk.end ? entry(b, it.key_lo, it.key_hi, next) : -1;
            load(&tmK, kvh, e, make_uint4(0, 0, 0, 0));
            if (first && ok) {  // Q after the first K tile, which waits for less
              first = false;
              if (q_loads > 0 && !wait(bar_qempty, (q_loads - 1) & 1)) break;
              if (lane == 0) {
                mbar_arrive_expect_tx(bar_qfull, 2 * Lay::kTile);
                for (int q = 0; q < 2; ++q)
                  for (int s = 0; s < kSlabs; ++s)
                    tma_load_3d(sm + q * Lay::kTile + s * Lay::kSlab, &tmQ, bar_qfull, s * 64, it.head0,
                                it.q_row + it.tok0 + q * tpt);
              }
              ++q_loads;
            }
            kt = next;
            e = e_next;
          }
        }
        before = end;
      }
      if (ok) {
        RlItem stop;
        stop.seq = -1;
        hand_on(stop);
      }
    }
    // At exit no copy or commit is in flight: the warp's last tiles have been
    // read, or, where a wait ran out, their copies have at least landed.
    __syncwarp();
    if (lane == 0) {
      uint64_t* const full = bar_full + (values ? kDeep : 0);
      uint64_t* const empty = bar_empty + (values ? kDeep : 0);
      bool drained = ok;
      if (drained) drained = drain_fills(empty, loaded, kDeep, false);
      if (drained && q_loads > 0) drained = rl_wait(bar_qempty, (q_loads - 1) & 1);
      if (!drained) {
        if (q_loads > 0) rl_wait(bar_qfull, (q_loads - 1) & 1);
        drain_fills(full, loaded, kDeep, true);
      }
    }
  } else if (warp == kRlMmaWarp) {
    // ---- MMA issue.  The warp runs as one, on values that are the same in all
    // lanes by construction (broadcasts and votes), so that the descriptors stay
    // in uniform registers, which the MMA instructions take; one elected lane
    // issues.  With all of it in a single lane's branch the issue of a step's
    // products took as long as the products.
    constexpr uint32_t idS = tc::idesc_f16(kBf16, kTcRows, kTcKeys, false);
    constexpr uint32_t idPV = tc::idesc_f16(kBf16, kTcRows, D, true);
    constexpr uint32_t kHi = tc::sdesc_hi(1024);
    const bool leader = elect_one();
    auto all = [](uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); };
    const uint32_t tm = all(tmem);
    const uint32_t q_lo = all(tc::sdesc_lo(smem_u32(sm), 16));
    const uint32_t k_lo = all(tc::sdesc_lo(smem_u32(sm + Lay::kOffRing), 16));
    const uint32_t v_lo = all(tc::sdesc_lo(smem_u32(sm + Lay::kOffRing), Lay::kSlab));
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = __all_sync(0xffffffffu, rl_wait(bar, parity));
      return ok;
    };
    int q_loads = 0, pvs0 = 0, pvs1 = 0;  // Q loads, P V products
    int outs0 = 0, outs1 = 0;             // items with an output
    int n = 0;                            // tiles before this step's
    for (int k = 0; ok; ++k) {
      const int slot = k & 1;
      if (!wait(bar_item + slot, (k >> 1) & 1)) break;
      const RlSpan mine(items[slot], 0);
      const int last = all(items[slot].seq < 0);
      const int first = all(mine.first), end = all(mine.end), lo0 = all(mine.own_lo), hi0 = all(mine.own_hi),
                lo1 = all(mine.other_lo), hi1 = all(mine.other_hi);
      __syncwarp();
      if (leader) mbar_arrive(bar_free + slot);
      if (last) break;
      if (first < end) continue;
      if (!wait(bar_qfull, q_loads & 1)) break;
      ++q_loads;
      bool had0 = false, had1 = false, begun0 = false, begun1 = false;
      for (int kt = first; ok && kt >= end - 1; --kt) {
        const bool need0 = kt >= end && kt >= lo0 && kt < hi0, need1 = kt >= end && kt >= lo1 && kt < hi1;
        if (!(need0 || need1) && !(had0 || had1)) continue;  // a gap between the two tiles' intervals
        const int vslot = kDeep + (n + kDeep - 1) % kDeep, kslot = n % kDeep;  // V of the tile before, K of this one
        // one query tile's turn: P V of the key tile before, then S of this one
        auto turn = [&](int q, bool had, bool need, bool& begun, int& pvs, int outs, bool frees_v, bool frees_k) {
          const uint32_t tS = tm + q * 128, tO = tm + 256 + q * D;
          if (had) {
            if (!wait(bar_full + vslot, ((n - 1) / kDeep) & 1)) return;
            // a new item's O overwrites the previous one's, which has to be read
            if (!begun && outs > 0 && !wait(bar_o + q, (outs - 1) & 1)) return;
            if (!wait(bar_p + q, pvs & 1)) return;
            tc::fence_after();
            const uint32_t b_lo = v_lo + vslot * (Lay::kTile >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kTcKeys / 16; ++kk)
                tc::mma_f16_ts_words(tO, tS + 64 + kk * 8, b_lo + kk * 128, kHi, idPV, (begun || kk > 0) ? 1u : 0u);
              tc::commit(bar_pv + q);
              if (frees_v) tc::commit(bar_empty + vslot);
            }
            begun = true;
            ++pvs;
          }
          if (need) {
            if (!wait(bar_full + kslot, (n / kDeep) & 1)) return;
            // S overwrites the tile's last P, whose product must be done
            if (pvs > 0 && !wait(bar_pv + q, (pvs - 1) & 1)) return;
            tc::fence_after();
            const uint32_t a_lo = q_lo + q * (Lay::kTile >> 4), b_lo = k_lo + kslot * (Lay::kTile >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * Lay::kSlab + (kk & 3) * 32) >> 4;  // 64-dim slab, 16-dim step
                if (kk == 0) tc::mma_f16_words<false>(tS, a_lo + off, kHi, b_lo + off, kHi, idS);
                else tc::mma_f16_words<true>(tS, a_lo + off, kHi, b_lo + off, kHi, idS);
              }
              tc::commit(bar_s + q);
              if (frees_k) {
                tc::commit(bar_empty + kslot);
                if (kt == end) tc::commit(bar_qempty);  // the item's last S
              }
            }
          }
        };
        turn(0, had0, need0, begun0, pvs0, outs0, !had1, !need1);
        if (ok) turn(1, had1, need1, begun1, pvs1, outs1, true, true);
        had0 = need0;
        had1 = need1;
        if (need0 || need1) ++n;
      }
      outs0 += lo0 < hi0;
      outs1 += lo1 < hi1;
    }
    if (!ok && leader) {  // a wait ran out: what was issued ends before the tensor memory goes
      tc::commit(bar_end);
      rl_wait(bar_end, 0);
    }
    __syncwarp();
  } else {
    // ---- softmax of query tile q: thread t of the tile's warps w and w + 4 has
    // row 32 w + t, the first its keys 0-63 and the second its keys 64-127
    const int q = warp / kRlSoftWarps, wq = warp & 3, half = (warp >> 2) & 1, r = wq * 32 + lane;
    const uint32_t tS = tmem + q * 128 + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tO = tmem + 256 + q * D + half * (D / 2) + (static_cast<uint32_t>(wq * 32) << 16);
    const int hh = r & (hg - 1), tok = q * tpt + (r >> p.hg_log2);
    const int pair = 1 + q * 4 + wq;  // named barrier of the two warps of a row
    float* const row_own = reinterpret_cast<float*>(sm + Lay::kOffRow) + (q * 2 + half) * kTcRows + r;
    const float* const row_other = row_own + (half ? -kTcRows : kTcRows);
    const float c2 = p.scale_log2;
    const uint64_t c2x2 = tc::f2(c2, c2);
    const CapPoly cap = p.rules.poly;
    // a tile whose weights sum to more than this has moved too far above its row's reference
    constexpr float kGrown = kBf16 ? 4294967296.f : 16384.f;  // 2^32: P V stays in float32; 2^14: P in fp16
    bool ok = true;
    int scores = 0;  // S tiles so far
    for (int k = 0;; ++k) {
      const int slot = k & 1;
      // a row's two warps go on together: a wait that ran out for a lane of either ends both
      if (barrier_or(pair, 64, !(ok && rl_wait(bar_item + slot, (k >> 1) & 1)))) break;
      const RlSpan walk(items[slot], q);
      const bool last = items[slot].seq < 0;
      const int t = items[slot].tok0 + tok;
      const bool real = t < items[slot].n;
      const int pos = items[slot].ctx + t, head = items[slot].head0 + hh, len = items[slot].len;
      // tiles whole_lo .. whole_hi - 1 hold no key that no row of the pair sees
      const int whole_lo = items[slot].whole_lo, whole_hi = items[slot].whole_hi;
      const int64_t row = static_cast<int64_t>(items[slot].q_row) + t;
      const int piece = items[slot].piece;
      const bool whole = items[slot].pieces == 1;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_free + slot);
      if (last) break;
      KeySpan span{0, 0};
      if (real) span = keys_seen(p.rules, row, pos, len);
      float slope = 0.f;
      if constexpr (BIAS) slope = __ldg(p.rules.slopes + head) * kLog2e;
      // Weights and sums are relative to m_ref, the largest score of the first
      // tile in which the row sees a key (set: there was one).  It moves again
      // only when a tile's weights sum to more than kGrown.
      float m_ref = 0.f, l = 0.f;
      bool set = false, begun = false;
      int n = walk.tile0;  // tiles up to and with this one
      for (int kt = walk.first; kt >= walk.end; --kt) {
        if (!walk.any(kt)) continue;
        ++n;
        if (!walk.own(kt)) continue;
        // after a timeout (recorded) the remaining waits are skipped
        if (ok && !rl_wait(bar_s + q, scores & 1)) ok = false;
        ++scores;
        tc::fence_after();
        const int k0 = kt * kTcKeys + 64 * half;  // this half's first key
        // columns lo .. hi - 1 are keys of this row
        const int lo = span.lo - k0, hi = span.hi - k0;
        // some row of the warp does not see all of the half, or (with a bias) sees ahead
        const bool part = __any_sync(0xffffffffu, lo > 0 || hi < 64 || (BIAS && pos - k0 < 63));
        const float ahead = static_cast<float>(pos - k0);  // distance of column 0
        const uint32_t tSh = tS + 64 * half;
        uint32_t pk[32];  // P, two keys to a column
        float sum;
        // The row's largest score, over both halves (-inf: none has a weight).
        // The cap grows with the score, so that without a bias it is taken of the
        // largest alone (the lowest number stands for a seen -inf until then, which
        // the cap gives a weight); with one, every score is capped, by the polynomial
        // unless one lies beyond it.
        auto row_max = [&]() {
          float m = -INFINITY;
          auto scan = [&](auto in_full) -> bool {
            [[maybe_unused]] constexpr bool kExact = decltype(in_full)::value;
            float big = 0.f;
            m = -INFINITY;
#pragma unroll 1
            for (int c0 = 0; c0 < 64; c0 += 32) {
              uint32_t s[32];
              tc::ld_32x32b_x32(tSh + c0, s);
              tc::wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const int c = c0 + i;
                const float d = c >= lo && c < hi ? __uint_as_float(s[i]) : NAN;  // fmaxf passes a NaN over
                float x = d * c2;
                if constexpr (CAP && BIAS) {
                  if constexpr (kExact) {
                    x = soft_cap(d, c2, p.rules.cap_log2, p.rules.cap_arg);
                  } else {
                    const float u = d * d;
                    big = fmaxf(big, u);
                    float y = fmaf(cap.c[5].x, u, cap.c[4].x);
#pragma unroll
                    for (int j = 3; j >= 0; --j) y = fmaf(y, u, cap.c[j].x);
                    x = d * y;
                  }
                }
                if (BIAS) x = fmaf(-slope, fabsf(ahead - c), x);
                m = fmaxf(m, x);
              }
            }
            return __any_sync(0xffffffffu, big > cap.limit);
          };
          if (scan(std::false_type())) {
            if constexpr (CAP && BIAS) scan(std::true_type());
          }
          if (CAP && !BIAS && lo < min(hi, 64) && hi > 0) m = fmaxf(m, -FLT_MAX);  // a key of this half is seen
          *row_own = m;
          named_barrier_sync(pair, 64);
          m = fmaxf(m, *row_other);
          named_barrier_sync(pair, 64);  // read before it is written again
          if (CAP && !BIAS && m != -INFINITY)
            m = soft_cap(m == -FLT_MAX ? -INFINITY : m, 1.f, p.rules.cap_log2, __fdiv_rn(1.f, p.rules.cap_log2));
          return m;
        };
        // P = exp2(score - m_ref) rounded to T (keys the row does not see: 0), and
        // the sum of the rounded P.  `masked`: some key is not seen.  `in_full`: the
        // cap in its exact form, for scores beyond it, where the polynomial does
        // not hold (true returned: it was needed and not used).
        auto pass = [&](auto masked, auto in_full) -> bool {
          constexpr bool kPart = decltype(masked)::value, kExact = decltype(in_full)::value;
          float s0 = 0.f, s1 = 0.f, big = 0.f;
          const uint64_t negm = tc::f2(-m_ref, -m_ref);
          const uint64_t sl2 = tc::f2(slope, slope);
#pragma unroll
          for (int c0 = 0; c0 < 64; c0 += 32) {
            uint32_t s[32];
            tc::ld_32x32b_x32(tSh + c0, s);
            tc::wait_ld();
            const float b0 = BIAS ? fmaf(-slope, ahead - c0, -m_ref) : 0.f;
            const uint64_t b0x2 = tc::f2(b0, b0);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = c0 + 2 * i;
              float2 x = make_float2(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), e;
              const bool in0 = !kPart || (c >= lo && c < hi), in1 = !kPart || (c + 1 >= lo && c + 1 < hi);
              uint64_t base = negm;
              if constexpr (BIAS) {
                if (kPart)
                  base = tc::f2(fmaf(-slope, fabsf(ahead - c), -m_ref), fmaf(-slope, fabsf(ahead - (c + 1)), -m_ref));
                else
                  base = tc::ffma2(sl2, tc::f2(2.f * i, 2.f * i + 1.f), b0x2);
              }
              if constexpr (CAP && kExact) {
                const float2 b = tc::f2_split(base);
                e.x = soft_cap(x.x, c2, p.rules.cap_log2, p.rules.cap_arg) + b.x;
                e.y = soft_cap(x.y, c2, p.rules.cap_log2, p.rules.cap_arg) + b.y;
              } else if constexpr (CAP) {
                if (kPart) {  // what lies in a slot that is not seen must not call for the exact form
                  x.x = in0 ? x.x : 0.f;
                  x.y = in1 ? x.y : 0.f;
                }
                e = tc::f2_split(cap.run(tc::f2(x.x, x.y), base, big));
              } else {
                e = tc::f2_split(tc::ffma2(tc::f2(x.x, x.y), c2x2, base));
              }
              if (kPart) {
                e.x = in0 ? e.x : -INFINITY;
                e.y = in1 ? e.y : -INFINITY;
              }
              const uint32_t w = Mma<T>::pack(fast_exp2(e.x), fast_exp2(e.y));
              pk[c / 2] = w;
              // the sum is taken over the rounded P that P V multiplies, so that the
              // weights the output is normalised by are the ones it was built from
              if (i & 1) add_pair<T>(s1, w);
              else add_pair<T>(s0, w);
            }
          }
          sum = s0 + s1;
          return CAP && !kExact && __any_sync(0xffffffffu, big > cap.limit);
        };
        auto weigh = [&]() {
          using std::false_type;
          using std::true_type;
          const bool beyond = part ? pass(true_type(), false_type()) : pass(false_type(), false_type());
          if constexpr (CAP) {
            if (beyond) pass(true_type(), true_type());
          }
        };
        // (both warps of a row know the same `set`, so they agree on what follows)
        if (!__all_sync(0xffffffffu, set)) {
          const float m = row_max();
          if (!set && m != -INFINITY) {
            m_ref = m;
            set = true;
          }
        }
        weigh();
        // Do the row's two warps agree that the reference holds?  The barrier
        // also says that both have read S, which P goes over.
        tc::fence_before();
        const bool grown = barrier_or(pair, 64, sum > kGrown);
        tc::fence_after();
        if (grown) {
          const float m = row_max();
          const float m_new = fmaxf(m_ref, m), alpha = fast_exp2(m_ref - m_new);
          l *= alpha;
          m_ref = m_new;
          if (begun) {
            // O holds the tiles before this one: their P V were done before this S was written
            const uint64_t a2 = tc::f2(alpha, alpha);
#pragma unroll 1
            for (int oc = 0; oc < D / 2; oc += 32) {
              uint32_t w[32];
              tc::ld_32x32b_x32(tO + oc, w);
              tc::wait_ld();
#pragma unroll
              for (int j = 0; j < 32; j += 2) {
                const float2 y = tc::f2_split(tc::fmul2(tc::f2(__uint_as_float(w[j]), __uint_as_float(w[j + 1])), a2));
                w[j] = __float_as_uint(y.x);
                w[j + 1] = __float_as_uint(y.y);
              }
              tc::st_32x32b_x32(tO + oc, w);
            }
          }
          weigh();
          tc::fence_before();
          named_barrier_sync(pair, 64);
          tc::fence_after();
        }
        tc::st_32x32b_x32(tS + 64 + 32 * half, pk);
        l += sum;
        if (kt < whole_lo || kt >= whole_hi) {  // clear the V rows that no row of the pair sees
          // (both tiles' warps clear the same rows, each before its own P V)
          const int at = (n - 1) % kDeep;
          if (ok && !rl_wait(bar_full + kDeep + at, ((n - 1) / kDeep) & 1)) ok = false;
          clear_unseen<D>(sm + Lay::kOffRing + (kDeep + at) * Lay::kTile, seen + at, half * kTcRows + r);
          fence_proxy_async_smem();  // the zeros are read by the tensor cores
        }
        begun = true;
        tc::wait_st();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + q);
      }
      T* orow = static_cast<T*>(p.out) + (row * p.num_heads + head) * D + half * (D / 2);
      const int64_t part = static_cast<int64_t>(piece) * p.num_tokens * p.num_heads + row * p.num_heads + head;
      if (!begun) {  // the tile sees no key
        if (real && !whole) {
          if (half == 0) *reinterpret_cast<float2*>(p.ws_ml + part * 2) = make_float2(-INFINITY, 0.f);
        } else if (real)
          for (int oc = 0; oc < D / 2; oc += 8) *reinterpret_cast<uint4*>(orow + oc) = make_uint4(0, 0, 0, 0);
        continue;
      }
      *row_own = l;
      named_barrier_sync(pair, 64);
      l += *row_other;
      named_barrier_sync(pair, 64);
      if (ok && !rl_wait(bar_pv + q, (scores - 1) & 1)) ok = false;
      tc::fence_after();
      const float inv = l > 0.f ? __fdiv_rn(1.f, l) : 0.f;
      const bool store = ok && real;
      if (!whole && store && half == 0)
        *reinterpret_cast<float2*>(p.ws_ml + part * 2) = make_float2(l == 0.f ? -INFINITY : m_ref, l);
#pragma unroll 1
      for (int oc = 0; oc < D / 2; oc += 32) {
        uint32_t w[32];
        tc::ld_32x32b_x32(tO + oc, w);
        tc::wait_ld();
        if (!whole) {  // joined by join_pieces_kernel
          if (store) {
            float4* to = reinterpret_cast<float4*>(p.ws_o + part * D + half * (D / 2) + oc);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              to[j] = make_float4(__uint_as_float(w[4 * j]), __uint_as_float(w[4 * j + 1]),
                                  __uint_as_float(w[4 * j + 2]), __uint_as_float(w[4 * j + 3]));
          }
          continue;
        }
        uint32_t o[16];
#pragma unroll
        for (int j = 0; j < 16; ++j)
          o[j] = Mma<T>::pack(__uint_as_float(w[2 * j]) * inv, __uint_as_float(w[2 * j + 1]) * inv);
        if (store) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            reinterpret_cast<uint4*>(orow + oc)[j] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_o + q);
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == kRlMmaWarp) {
    __syncwarp();
    tc::fence_after();
    tc::dealloc(tmem, kRlCols);
  }
}

// Joins the pieces of a row, a warp per (row, head): M = max_s m_s, out =
// sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s, in the order of the pieces.
// Rows that no sequence's chunk has, or past what was computed, are left.
template <typename T, int D>
__global__ void __launch_bounds__(128) join_pieces_kernel(const RulesPrefillParams p) {
  const int lane = threadIdx.x & 31;
  const int splits = *p.ws_pieces;
  if (splits == 1) return;  // written by the attention kernel
  const int64_t rows = p.num_tokens * p.num_heads;
  const int64_t idx = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (idx >= rows) return;
  const int64_t row = idx / p.num_heads;
  // the last sequence that starts at or before the row, among those with rows
  int lo = 0, hi = p.num_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(p.query_start + mid) <= row) lo = mid; else hi = mid - 1;
  }
  const int q_row = __ldg(p.query_start + lo), n = __ldg(p.query_start + lo + 1) - q_row;
  int len = __ldg(p.seq_lens + lo);
  const int64_t cap = static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size;
  if (len >= n && len > cap) len = static_cast<int>(cap);
  const int64_t reach = static_cast<int64_t>(p.row_tiles) * 2 * (kTcRows >> p.hg_log2);
  if (q_row < 0 || row < q_row || row - q_row >= n || row - q_row >= reach || len < n ||
      q_row + static_cast<int64_t>(n) > p.num_tokens)
    return;
  constexpr int kPer = D / 32;
  float m = -INFINITY;
  for (int s = 0; s < splits; ++s) m = fmaxf(m, __ldg(p.ws_ml + (s * rows + idx) * 2));
  float num[kPer] = {}, den = 0.f;
  for (int s = 0; s < splits; ++s) {
    const float2 ml = __ldg(reinterpret_cast<const float2*>(p.ws_ml + (s * rows + idx) * 2));
    if (ml.y == 0.f) continue;  // no key of weight; its O was not written, perhaps (a sum of NaN goes on)
    const float f = fast_exp2(ml.x - m);
    den += f * ml.y;
    const float* o = p.ws_o + (s * rows + idx) * D + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) num[i] += f * __ldg(o + i);
  }
  T* out = static_cast<T*>(p.out) + idx * D + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; ++i) out[i] = DType<T>::from_float(den == 0.f ? 0.f : num[i] / den);  // NaN stays
}

int device_sms() {
  static int cached[64] = {0};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) dev = 0;
  if (!cached[dev]) {
    int n = 0;
    cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    cached[dev] = n > 0 ? n : 1;
  }
  return cached[dev];
}

// Pieces that each item's keys may be cut into: the number of least cost for
// the most items and tiles that the arguments allow for (the lengths are on the
// device, where the scheduler decides by them, up to this number).  Measured,
// 32/8 heads of 128, whole and in pieces: 40 rows after 20000 tokens 449 and 50
// us (19 pieces), 64 after 2000 41 and 27 (8), 300 after 4000 107 and 60 (4), 1000
// after 8000 210 and 156 (2); 2600 causal rows of 16/2 heads 60, and 79 in 3
// pieces, which this cost does not call for.  It counts on the mean of the CTAs and
// not on whole rounds of them: 8 chunks to 128 rows after to 1000 tokens take 37 us
// whole, and 50 in the two pieces that it asks for behind a wide table.  Calls that give key_begin are not
// cut: what their rows see has little to do with the lengths.
struct RlPlan {
  int hg_log2, splits;
};
RlPlan rl_plan(int64_t num_tokens, int num_seqs, int group, int num_heads, int block_size, int max_blocks,
               int max_query_len, int window, bool begins) {
  RlPlan pl{0, 1};
  while (pl.hg_log2 < 3 && group % (2 << pl.hg_log2) == 0) ++pl.hg_log2;
  if (begins) return pl;
  const int64_t tokens = 2 * (kTcRows >> pl.hg_log2);  // chunk tokens of an item
  const int64_t longest = std::min<int64_t>(max_query_len, num_tokens);
  const int64_t pairs = std::min((longest + tokens - 1) / tokens * num_seqs, num_tokens / tokens + num_seqs);
  const int64_t items = pairs * (num_heads >> pl.hg_log2);
  int64_t keys = static_cast<int64_t>(max_blocks) * block_size;
  if (window > 0) keys = std::min<int64_t>(keys, window + tokens);
  const int64_t tiles = (keys + kTcKeys - 1) / kTcKeys;
  float best = 0.f;
  for (int n = 1; n <= 32 && (n == 1 || 2 * n <= tiles); ++n) {
    const float cost = rl_cost(items, static_cast<float>(items) * tiles, tiles, n, device_sms());
    if (n == 1 || cost < best) {
      best = cost;
      pl.splits = n;
    }
  }
  return pl;
}

int64_t rl_workspace(const RlPlan& pl, int64_t num_tokens, int num_heads, int head_dim) {
  return pl.splits > 1 ? 16 + pl.splits * num_tokens * num_heads * (head_dim + 2) * 4 : 0;
}

template <typename T, int D, bool CAP, bool BIAS>
cudaError_t launch_rules(const RulesPrefillParams& p, int max_query_len, const CUtensorMap& mq, const CUtensorMap& mk,
                         const CUtensorMap& mv, cudaStream_t st) {
  constexpr int kSmem = RlLayout<D>::kSmem;
  auto kern = prefill_rules_kernel<T, D, CAP, BIAS>;
  static bool ready[64] = {false};  // per device: the kernel may use its shared memory
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int tokens = 2 * (kTcRows >> p.hg_log2);  // chunk tokens of an item
  const int64_t pairs = (static_cast<int64_t>(max_query_len) + tokens - 1) / tokens;
  const int64_t items = pairs * (p.num_heads >> p.hg_log2) * p.num_seqs * p.splits;
  if (pairs > INT32_MAX) return cudaErrorInvalidConfiguration;
  RulesPrefillParams a = p;
  a.row_tiles = static_cast<int32_t>(pairs);
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(items, device_sms()));
  kern<<<grid, kRlThreads, kSmem, st>>>(a, mq, mk, mv);
  e = cudaGetLastError();
  if (e != cudaSuccess || p.splits <= 1) return e;
  const int64_t rows = p.num_tokens * p.num_heads;
  if (rows > static_cast<int64_t>(INT32_MAX) * 4) return cudaErrorInvalidConfiguration;
  join_pieces_kernel<T, D><<<static_cast<unsigned>((rows + 3) / 4), 128, 0, st>>>(a);
  return cudaGetLastError();
}

template <typename T, int D>
cudaError_t launch_rules_form(const RulesPrefillParams& p, int max_query_len, const CUtensorMap& mq,
                              const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t st) {
  const bool cap = p.rules.cap_log2 > 0.f, bias = p.rules.slopes != nullptr;
  if (cap) return bias ? launch_rules<T, D, true, true>(p, max_query_len, mq, mk, mv, st)
                       : launch_rules<T, D, true, false>(p, max_query_len, mq, mk, mv, st);
  return bias ? launch_rules<T, D, false, true>(p, max_query_len, mq, mk, mv, st)
              : launch_rules<T, D, false, false>(p, max_query_len, mq, mk, mv, st);
}

}  // namespace
}  // namespace pagedkv

using namespace pagedkv;

extern "C" int paged_prefill_rules_workspace_size(int64_t num_query_tokens, int32_t num_seqs, int32_t num_heads,
                                                  int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                                  int32_t max_blocks_per_seq, int32_t max_query_len, int32_t window,
                                                  int32_t begins, size_t* bytes_out) {
  if (!bytes_out || num_query_tokens < 0 || num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 ||
      num_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128) || block_size <= 0 ||
      max_blocks_per_seq <= 0 || max_query_len < 0 || window < 0)
    return KV_ERR_INVALID_ARG;
  *bytes_out = 0;
  if (num_query_tokens == 0 || num_seqs == 0 || max_query_len == 0 || !tc_supported(block_size)) return KV_OK;
  const RlPlan pl = rl_plan(num_query_tokens, num_seqs, num_heads / num_kv_heads, num_heads, block_size,
                            max_blocks_per_seq, max_query_len, window, begins != 0);
  *bytes_out = static_cast<size_t>(rl_workspace(pl, num_query_tokens, num_heads, head_dim));
  return KV_OK;
}

extern "C" int paged_prefill_attention_rules(
    void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
    const int32_t* seq_lens, const int32_t* query_start_loc, int64_t num_query_tokens, int32_t num_seqs,
    int32_t num_heads, int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks,
    int32_t max_blocks_per_seq, int32_t max_query_len, float scale, float softcap, const float* slopes, int32_t window,
    const int32_t* key_begin, const int32_t* key_end, int dtype, void* workspace, size_t workspace_bytes,
    void* stream) {
  RulesPrefillParams p{};
  int s = make_rules(scale, softcap, slopes, window, key_begin, key_end, &p.rules);
  if (s != KV_OK) return s;
  s = prefill_params(out, q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, num_query_tokens, num_seqs,
                     num_heads, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq, max_query_len,
                     scale, dtype, &p);
  if (s != KV_OK || p.num_seqs == 0) return s;
  max_query_len = longest_chunk(max_query_len, num_query_tokens);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!tc_supported(block_size)) {
    const cudaError_t e = dtype == KV_DTYPE_F16 ? launch_prefill<__half>(p, head_dim, max_query_len, st)
                                                : launch_prefill<__nv_bfloat16>(p, head_dim, max_query_len, st);
    return cuda_status(e);
  }
  p.test_skip = debug_skip_tile();
  const RlPlan pl = rl_plan(num_query_tokens, num_seqs, p.group, num_heads, block_size, max_blocks_per_seq,
                            max_query_len, window, key_begin != nullptr);
  p.hg_log2 = pl.hg_log2;
  p.splits = 1;
  const size_t need = static_cast<size_t>(rl_workspace(pl, num_query_tokens, num_heads, head_dim));
  if (workspace && need > 0) {
    if (workspace_bytes < need) return KV_ERR_WORKSPACE;
    if (!aligned16(workspace)) return KV_ERR_INVALID_ARG;
    p.splits = pl.splits;
    p.ws_pieces = static_cast<int32_t*>(workspace);
    p.ws_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + 16);
    p.ws_ml = p.ws_o + pl.splits * num_query_tokens * num_heads * head_dim;
  }
  CUtensorMap mq, mk, mv;
  const int64_t rows = num_blocks * block_size;
  if (!tc_map(q, head_dim, num_heads, num_query_tokens, 1 << p.hg_log2, kTcRows >> p.hg_log2, &mq) ||
      !tc_map(k_cache, head_dim, num_kv_heads, rows, 1, block_size, &mk) ||
      !tc_map(v_cache, head_dim, num_kv_heads, rows, 1, block_size, &mv))
    return cuda_status(cudaErrorInvalidValue, "cuTensorMapEncodeTiled failed");
  cudaError_t e;
  if (dtype == KV_DTYPE_F16)
    e = head_dim == 64 ? launch_rules_form<__half, 64>(p, max_query_len, mq, mk, mv, st)
                       : launch_rules_form<__half, 128>(p, max_query_len, mq, mk, mv, st);
  else
    e = head_dim == 64 ? launch_rules_form<__nv_bfloat16, 64>(p, max_query_len, mq, mk, mv, st)
                       : launch_rules_form<__nv_bfloat16, 128>(p, max_query_len, mq, mk, mv, st);
  return cuda_status(e);
}

// Read (and optionally clear) this translation unit's device error word.
extern "C" int pagedkv_internal_prefill_rules_error(int reset, int* code) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_error, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  if (reset) {
    int zero = 0;
    if (cudaMemcpyToSymbol(g_device_error, &zero, sizeof(int)) != cudaSuccess) return KV_ERR_CUDA;
  }
  *code = v;
  return KV_OK;
}
