// Attention of drafted tokens over the paged cache: every sequence's last n
// tokens form a tree (or a chain), and each attends the tokens before the step,
// itself and its ancestors. bf16, head_dim 64 or 128, on the 5th-generation
// tensor cores. ("Paged Attention", klaylearn.com glossary, definition: the
// kernel reads K and V through the block table; the attention arithmetic is
// unchanged.)
//
// What bounds it: n rows x G query heads of a KV head share each K/V row, 4 d n G
// flops per 4 d bytes, so up to about 240 rows a KV head it is the cache's
// bytes. The rows are the M side of the MMA (a tile of 128, row = token * G +
// head of the group), the keys of a 64-key tile the N side.
//
// Work is counted in units: one 64-key tile for one KV head and one item of
// query rows (QT tiles of 128), and a few for each item itself; ordered by
// sequence, KV head, item, key. A fixed number of pipelines take equal,
// contiguous stretches of units (each finds its own from the context lengths, so
// that a captured call follows them), whatever the lengths are: a stretch may end
// inside one (sequence, head, item) and start inside another. A run that holds
// all key tiles of its item writes the output; otherwise (m, l, O) go to the
// workspace (two slots a pipeline: the item it starts inside, and the item it
// ends inside) with a header, and the merge kernel combines the parts of an item
// in key order. So the result depends on the lengths of the batch (which set the
// cuts), not on placement or block size.
//
// One CTA per SM, of one pipeline (QT = 2: each K/V tile is read once for 256
// rows) or of two (QT = 1: two streams of loads and two softmaxes hide each
// other's latency). A pipeline:
//  * warp 0 / warp 1 (producers): K (and Q) / V tiles by TMA, boxes of {64
//    columns, min(block_size, 64) tokens} with the 128-byte swizzle, into a
//    ring of 64-key tiles each, running ahead across items.
//  * warps 2, 3: S_x = Q_x K^T (M 128, N 64), two tiles ahead, and O_x += P_x V: one each, or
//    (QT = 2) a query tile each.
//  * 4 QT softmax warps, thread = row: as in the prefill kernel (base-2
//    exponentials against a reference that moves when exceeded by 2^8, P in
//    tensor memory over its S). P is rounded to bf16 (the type of V), and the row
//    sum adds the rounded weights, so that they sum to 1 exactly.
//
// Measured (32 query and 8 KV heads, head_dim 128, with the merge): 256 sequences of
// lognormal lengths (621 MB of K and V) with 1 to 16 rows each 117 us, 5.3 TB/s; 4
// sequences of 32,768 tokens with 64 rows each 144 us, 950 TFLOP/s: there a tile takes a
// pipeline 2,000 clocks, its exponentials 1,024 and its MMAs 1,244 of them. That is a
// dozen launches at 1,965 MHz; launched without a pause the SM clock falls to about 1,480
// MHz under the power limit, and the same launches take 126 and 172 us (4.9 TB/s, 800 TFLOP/s).
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_launch.cuh"
#include "pa_prefill_order.h"
#include "pa_tc.cuh"

namespace pa {

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();

namespace {

constexpr int kTreeKeys = 64;    // keys per tile
constexpr int kTreeRows = 128;   // rows per query tile
// Starting and ending an item (Q, the first tile's latency, the output) costs about
// as much as this many tiles: each item counts that many units more, so that a
// pipeline with several short items takes fewer tiles.
constexpr int kTreeItemCost = 2;
constexpr int kTreeMinUnits = 3;  // least units a pipeline takes
// An item of at most so many units is not cut: the merge would cost more than the
// uneven stretches (1,024 sequences of 166 tokens: 239 us cut, 224 whole).
constexpr int kTreeWhole = 8;

// What one partial result belongs to: rows [0, rows) of an item, whose first
// output row is out_row, split over pipelines first .. last; first < 0: none.
struct TreeHeader {
  int64_t out_row;
  int rows, first, last, pad[3];
};

struct TreeParams {
  __nv_bfloat16* out;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  const int32_t* parents;
  unsigned* err;
  TreeHeader* hdr;  // [pipelines][2]
  float2* ws_ml;    // [pipelines][2][slot_rows]: reference maximum, sum
  float* ws_acc;    // [pipelines][2][D / 4][slot_rows][4]
  int num_heads, num_kv_heads, lg_group, block_size, log2_block_size, num_blocks;
  int max_blocks_per_seq, num_seqs, total_q, max_query_len, slot_rows;
  int q_box_tokens;  // tokens of a query tile that are loaded
  float q_scale;     // scale * log2(e)
};

template <int D, int QT>
struct TreeConfig {
  static constexpr int kQBytes = kTreeRows * D * 2;
  static constexpr int kQHalf = kTreeRows * 128;       // a 64-column half of a Q tile
  static constexpr int kGran = kTreeKeys * D * 2;      // one K or V tile
  static constexpr int kGranHalf = kTreeKeys * 128;
  static constexpr int kHalves = D / 64;
  static constexpr int kPipes = QT == 1 ? 2 : 1;       // pipelines of a CTA
  // K and V tiles in flight. Two rings, each with one producer: its wait for a tile
  // to be free can then never be a whole phase ahead of its barrier (in one ring
  // that both producers filled in turns it could, when a commit came late).
  static constexpr int kNK = QT == 1 ? (D == 128 ? 2 : 5) : (D == 128 ? 5 : 6);
  static constexpr int kNV = QT == 1 ? (D == 128 ? 3 : 6) : (D == 128 ? 5 : 6);
  static constexpr int kNG = kNK + kNV;
  static constexpr int kRing = QT * kQBytes;           // a pipeline's Q, then its K and V rings
  static constexpr int kPipeBytes = kRing + kNG * kGran;
  static constexpr int kBars = kPipes * kPipeBytes;
  static constexpr int kNumBars = 2 * kNG + 2 + 6 * QT;  // of a pipeline
  static constexpr int kScratch = kBars + kPipes * kNumBars * 8;  // tensor-memory address, work search
  static constexpr int kSmemBytes = kScratch + 256;
  static constexpr int kPipeThreads = 128 + 128 * QT;
  static constexpr int kThreads = kPipes * kPipeThreads;
  static constexpr uint32_t kTmemCols = 512, kPipeCols = 512 / kPipes;
  static_assert(2 * 64 * QT + D * QT <= static_cast<int>(kPipeCols), "S and O fit");
  static_assert(kScratch % 8 == 0 && kSmemBytes <= 232448, "one CTA per SM");
};

__device__ __forceinline__ void tree_tma_3d(uint32_t dst, const CUtensorMap* map, int c0, int c1,
                                            int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// A sequence's rows and key tiles; nt = 0: no work (or bad arguments).
struct TreeSeq {
  int q0, n, L, nt, items;
  bool bad;
};

__device__ __forceinline__ TreeSeq tree_seq(const TreeParams& p, int s, int item_tokens) {
  TreeSeq t{};
  t.q0 = __ldg(p.query_start + s);
  const int q1 = __ldg(p.query_start + s + 1);
  t.L = __ldg(p.context_lens + s);
  if (!prefill_order::chunk_ok(t.q0, q1, t.L, p.total_q, p.max_query_len,
                               static_cast<int64_t>(p.max_blocks_per_seq) * p.block_size)) {
    t.bad = true;
    return t;
  }
  t.n = q1 - t.q0;
  if (t.n == 0) return t;
  t.nt = (t.L + kTreeKeys - 1) / kTreeKeys;
  t.items = (t.n + item_tokens - 1) / item_tokens;
  return t;
}

// (all sequences' together fit 31 bits: checked on the host for the longest)
__device__ __forceinline__ int tree_units(const TreeParams& p, const TreeSeq& t) {
  return (t.nt + (t.nt > 0 ? kTreeItemCost : 0)) * t.items * p.num_kv_heads;
}

// One run of key tiles of one item. Units count from the pipeline's first.
struct TreeRun {
  int s, q0, n, L, nt, h, row_item, t0, t1;
  int tile_unit;  // the unit of the item's first tile
};

// Calls f(run) for each run of the units [0, units), from sequence s on, whose
// first unit is `base` (<= 0); stops when f returns false.
template <typename F>
__device__ __forceinline__ void tree_runs(const TreeParams& p, int units, int s, int base,
                                          int item_tokens, F&& f) {
  int u = 0;
  while (u < units && s < p.num_seqs) {
    const TreeSeq t = tree_seq(p, s, item_tokens);
    const int own = tree_units(p, t);
    const int w = t.nt + kTreeItemCost;  // units of an item: its cost, then its tiles
    while (u < units && u - base < own) {
      const unsigned item = static_cast<unsigned>(u - base) / static_cast<unsigned>(w);
      TreeRun r;
      r.s = s;
      r.q0 = t.q0;
      r.n = t.n;
      r.L = t.L;
      r.nt = t.nt;
      r.h = t.items == 1 ? item : item / static_cast<unsigned>(t.items);
      r.row_item = static_cast<int>(item) - r.h * t.items;
      r.tile_unit = base + static_cast<int>(item) * w + kTreeItemCost;
      const int from = u - (r.tile_unit - kTreeItemCost), to = units - (r.tile_unit - kTreeItemCost);
      r.t0 = max(0, u - r.tile_unit);
      r.t1 = min(t.nt, units - r.tile_unit);
      if (w <= kTreeWhole) {
        // a short item goes whole to the stretch that holds its middle
        r.t0 = 0;
        r.t1 = 2 * from < w && 2 * to >= w ? t.nt : 0;
      }
      if (r.t1 > r.t0 && !f(r)) return;
      u = r.tile_unit + t.nt;
    }
    base += own;
    ++s;
  }
}

// A place in a ring of N tiles from `first` on, and the parity of its use.
template <int N>
struct RingPos {
  int st;
  uint32_t ph;
  int first;
  __device__ __forceinline__ explicit RingPos(int first_) : st(first_), ph(0), first(first_) {}
  __device__ __forceinline__ void step() {
    if (++st == first + N) {
      st = first;
      ph ^= 1;
    }
  }
};

template <int D, int QT>
__global__ void __launch_bounds__(TreeConfig<D, QT>::kThreads, 1)
    pa_tree_kernel(const __grid_constant__ CUtensorMap q_map,
                   const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const TreeParams p) {
  using Cfg = TreeConfig<D, QT>;
  constexpr int NK = Cfg::kNK, NV = Cfg::kNV, NG = Cfg::kNG, KEYN = kTreeKeys, HALVES = Cfg::kHalves;
  extern __shared__ __align__(1024) uint8_t sm[];
  // (the warp by a shuffle, so that the compiler knows it, and what the issuing warps derive
  // from it, to be uniform: an MMA's operands then stay in uniform registers. Moved there
  // for each, an MMA of 64 keys took 80 to 110 clocks to issue that runs in 48.)
  const int cta_warp = __shfl_sync(kFullMask, static_cast<int>(threadIdx.x) >> 5, 0);
  const int pipe = Cfg::kPipes == 1 ? 0 : cta_warp / (Cfg::kPipeThreads / 32);
  const int tid = static_cast<int>(threadIdx.x) - pipe * Cfg::kPipeThreads;  // of the pipeline
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + Cfg::kBars) + pipe * Cfg::kNumBars;
  auto bar = [&](int i) { return smem_u32(bars + i); };
  // barriers: a tile (K's, then V's) full, empty; Q full, empty; per query tile and parity of
  // the tile count: S full, P full, P V done
  constexpr int kFull = 0, kEmpty = NG, kQFull = 2 * NG, kQEmpty = 2 * NG + 1, kS = 2 * NG + 2;
  constexpr int kP = kS + 2 * QT, kO = kP + 2 * QT;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + Cfg::kScratch);
  int* s_sum = reinterpret_cast<int*>(sm + Cfg::kScratch + 16);  // [16]: one a warp
  int* s_base = s_sum + 16;                                      // [2], then [2]
  int* s_seq = s_base + 2;
  const uint32_t pipe_s = smem_u32(sm) + pipe * Cfg::kPipeBytes;
  auto q_s = [&](int x) { return pipe_s + x * Cfg::kQBytes; };
  auto gran = [&](int st) { return pipe_s + Cfg::kRing + st * Cfg::kGran; };

  const int warp = cta_warp - pipe * (Cfg::kPipeThreads / 32), lane = threadIdx.x & 31;  // (warp of the pipeline)
  const int G = 1 << p.lg_group, TOK = kTreeRows >> p.lg_group;
  const int item_tokens = QT * TOK;
  const int bs = p.block_size, lg = p.log2_block_size;
  auto wait_all = [&](uint32_t b, uint32_t parity) {
    return __all_sync(kFullMask, mbar_wait(b, parity, p.err));
  };

  if (smem_u32(sm) & 1023) {  // the swizzled operand layout needs this
    if (threadIdx.x == 0) atomicOr(p.err, PA_DEVERR_CONTEXT);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < NG; ++i) {
      mbar_init(bar(kFull + i), 1);
      mbar_init(bar(kEmpty + i), QT);  // (two query tiles have an issuer each)
    }
    mbar_init(bar(kQFull), 1);
    mbar_init(bar(kQEmpty), QT);
    for (int i = 0; i < 2 * QT; ++i) {
      mbar_init(bar(kS + i), 1);
      mbar_init(bar(kP + i), 128);
      mbar_init(bar(kO + i), 1);
    }
    fence_barrier_init();
    if (pipe == 0) {  // descriptors are kernel parameters: fetch them early
      prefetch_tensormap(&q_map);
      prefetch_tensormap(&k_map);
      prefetch_tensormap(&v_map);
    }
  }
  if (cta_warp == 2) tc::tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
  pdl_wait();  // inputs may come from the previous kernel in the stream
  pdl_launch_dependents();

  // The units of the batch, then each pipeline's stretch and the sequence it starts in:
  // each thread sums its own consecutive sequences, one scan joins the threads,
  // and the thread whose sequences hold the first unit finds the one.
  constexpr int NT = Cfg::kThreads, NW = NT / 32;
  const int per = (p.num_seqs + NT - 1) / NT;
  const int sa = threadIdx.x * per, sb = min(sa + per, p.num_seqs);
  int own = 0;
#pragma unroll 4
  for (int s = sa; s < sb; ++s) {
    const TreeSeq t = tree_seq(p, s, item_tokens);
    if (t.bad && blockIdx.x == 0) atomicOr(p.err, PA_DEVERR_CONTEXT);
    own += tree_units(p, t);
  }
  int incl = own;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(kFullMask, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) s_sum[cta_warp] = incl;
  if (tid == 0) s_seq[pipe] = p.num_seqs;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const int v = s_sum[w];
    if (w < cta_warp) incl += v;
    total += v;
  }
  const unsigned pipes = gridDim.x * Cfg::kPipes;
  const int share = max(static_cast<int>((static_cast<unsigned>(total) + pipes - 1) / pipes), kTreeMinUnits);
  const int me = static_cast<int>(blockIdx.x) * Cfg::kPipes + pipe;  // this pipeline among all
  const int64_t u0 = static_cast<int64_t>(me) * share;
  const int units = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(share), total - u0)));
#pragma unroll
  for (int q = 0; q < Cfg::kPipes; ++q) {
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * Cfg::kPipes + q) * share;
    if (incl - own <= first && first < incl) {
      int at = incl - own;
      for (int s = sa; s < sb; ++s) {
        const int n = tree_units(p, tree_seq(p, s, item_tokens));
        if (first < at + n) {
          s_seq[q] = s;
          s_base[q] = at - static_cast<int>(first);
          break;
        }
        at += n;
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = *tmem_slot + pipe * Cfg::kPipeCols;
  const int seq0 = s_seq[pipe];
  const int base0 = s_base[pipe];
  auto t_s = [&](int x, int b) { return tmem + (2 * x + b) * KEYN; };
  auto t_o = [&](int x) { return tmem + 2 * QT * KEYN + x * D; };
  auto runs = [&](auto&& f) {
    if (units > 0) tree_runs(p, units, seq0, base0, item_tokens, f);
  };

  // Two pipelines: 512 threads launched with 128 registers each; the producers and
  // issuers hand 56 of theirs to the softmax warpgroups (72 + 184 = 2 * 128).
  auto fewer = [] {
    if constexpr (QT == 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
  };
  if (warp < 2) {
    fewer();
    // ------------------------------------------------- producers: K and Q, V
    const CUtensorMap* map = warp == 0 ? &k_map : &v_map;
    const int rows = bs < KEYN ? bs : KEYN, lgr = bs < KEYN ? lg : 6;  // tokens per box
    int st = warp == 0 ? 0 : NK;  // the place in this producer's ring
    const int first = st, last = warp == 0 ? NK - 1 : NG - 1;
    uint32_t ph = 0, qph = 0;
    runs([&](const TreeRun& r) {
      const int32_t* trow = p.block_tables + static_cast<int64_t>(r.s) * p.max_blocks_per_seq;
      auto boxes = [&](int t) { return (min(KEYN, r.L - t * KEYN) + rows - 1) >> lgr; };  // <= 8
      // the block of this lane's box of tile t (lanes past the boxes: of the second
      // half of the columns), read one tile ahead
      auto entry = [&](int t, int nbox) {
        const int b = lane < nbox ? lane : lane - nbox;
        return lane < nbox * HALVES ? __ldg(trow + ((t * KEYN + b * rows) >> lg)) : 0;
      };
      int next = entry(r.t0, boxes(r.t0));
      if (warp == 0) {
        bool ok = true;
        if (lane == 0) {
          ok = mbar_wait(bar(kQEmpty), qph ^ 1, p.err);
          if (ok) {
            const int box = p.q_box_tokens * G * 128;
            mbar_arrive_expect_tx(bar(kQFull), QT * HALVES * box);
            for (int x = 0; x < QT; ++x)
              for (int c = 0; c < HALVES; ++c)
                tree_tma_3d(q_s(x) + c * Cfg::kQHalf, &q_map, c * 64, r.h * G,
                            r.q0 + r.row_item * item_tokens + x * TOK, bar(kQFull));
          }
        }
        if (!__shfl_sync(kFullMask, ok, 0)) return false;
        qph ^= 1;
      }
      for (int t = r.t0; t < r.t1; ++t) {
        const int nbox = boxes(t), blk = next;
        if (t + 1 < r.t1) next = entry(t + 1, boxes(t + 1));
        bool ok = true;
        if (lane == 0) {
          ok = mbar_wait(bar(kEmpty + st), ph ^ 1, p.err);
          if (ok) mbar_arrive_expect_tx(bar(kFull + st), static_cast<uint32_t>(nbox * rows * 128 * HALVES));
        }
        if (!__shfl_sync(kFullMask, ok, 0)) return false;
        if (lane < nbox * HALVES) {
          // an id outside the pool is flagged; TMA reads an out-of-range box as zeros
          if (static_cast<unsigned>(blk) >= static_cast<unsigned>(p.num_blocks))
            atomicOr(p.err, PA_DEVERR_BLOCK_ID);
          const int half = lane >= nbox, b = half ? lane - nbox : lane;
          tma_load_4d(gran(st) + half * Cfg::kGranHalf + b * rows * 128, map, half * 64,
                      (t * KEYN + b * rows) & (bs - 1), r.h, blk, bar(kFull + st));
        }
        if (++st > last) {
          st = first;
          ph ^= 1;
        }
      }
      return true;
    });
  } else if (warp < 4) {
    // ------------------------------------------------------------------- MMAs
    fewer();
    constexpr uint32_t kIdS = tc::idesc_bf16_f32(kTreeRows, KEYN, 0);
    constexpr uint32_t kIdPV = tc::idesc_bf16_f32(kTreeRows, D, 1);
    const bool one = tc::elect_one();
    RingPos<NK> kpos(0);
    RingPos<NV> vpos(NK);
    // S of tile it (over all runs), of query tile x; false: a wait gave up
    auto scores = [&](int x, int it) {
      // this buffer of S held P of tile it - 2 until its P V was done
      if (it >= 2 && !wait_all(bar(kO + 2 * x + (it & 1)), ((it - 2) >> 1) & 1)) return false;
      if (!wait_all(bar(kFull + kpos.st), kpos.ph)) return false;
      tc::fence_after_sync();
      if (one) {
        // (a k-step's operands lie a constant on: added to the descriptor, in 16 bytes)
        const uint64_t kd = tc::smem_desc_sw128(gran(kpos.st), 16, 1024);
        const uint64_t qd = tc::smem_desc_sw128(q_s(x), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc::mma_bf16(t_s(x, it & 1), qd + (((ks >> 2) * Cfg::kQHalf + (ks & 3) * 32) >> 4),
                       kd + (((ks >> 2) * Cfg::kGranHalf + (ks & 3) * 32) >> 4), kIdS, ks > 0);
        tc::commit(bar(kS + 2 * x + (it & 1)));
        tc::commit(bar(kEmpty + kpos.st));
      }
      __syncwarp();
      kpos.step();
      return true;
    };
    // O += P V of tile it, the run's first or not
    auto outputs = [&](int x, int it, bool first) {
      if (!wait_all(bar(kFull + vpos.st), vpos.ph)) return false;
      if (!wait_all(bar(kP + 2 * x + (it & 1)), (it >> 1) & 1)) return false;
      tc::fence_after_sync();
      if (one) {
        const uint64_t vd = tc::smem_desc_sw128(gran(vpos.st), Cfg::kGranHalf, 1024);
#pragma unroll
        for (int ks = 0; ks < KEYN / 16; ++ks)
          tc::mma_bf16_tmem_a(t_o(x), t_s(x, it & 1) + ks * 8, vd + ((ks * 2048) >> 4), kIdPV, !first || ks > 0);
        tc::commit(bar(kO + 2 * x + (it & 1)));
        tc::commit(bar(kEmpty + vpos.st));
      }
      __syncwarp();
      vpos.step();
      return true;
    };
    uint32_t qph = 0;
    int it = 0;  // tiles so far, over all runs
    bool ended = false;
    if (QT == 2) {
      // warp 2 + x: all of query tile x, S two tiles ahead of P V, so that neither query tile
      // waits for the other's barriers (one warp for S and one for P V of both: four
      // sequences of 32,768 tokens with 64 rows of 4 heads 151 us, this 147).
      const int x = warp - 2;
      runs([&](const TreeRun& r) {
        ended = false;
        if (!wait_all(bar(kQFull), qph)) return false;
        qph ^= 1;
        const int tiles = r.t1 - r.t0;
        for (int t = 0; t < tiles + 2; ++t) {
          if (t >= 2 && !outputs(x, it + t - 2, t == 2)) return false;
          if (t < tiles) {
            if (!scores(x, it + t)) return false;
            if (t == tiles - 1 && one) tc::commit(bar(kQEmpty));
          }
        }
        it += tiles;
        ended = true;
        return true;
      });
    } else if (warp == 2) {
      runs([&](const TreeRun& r) {
        ended = false;
        if (!wait_all(bar(kQFull), qph)) return false;
        qph ^= 1;
        for (int t = r.t0; t < r.t1; ++t, ++it)
          if (!scores(0, it)) return false;
        if (one) tc::commit(bar(kQEmpty));
        ended = true;
        return true;
      });
    } else {
      runs([&](const TreeRun& r) {
        ended = false;
        for (int t = r.t0; t < r.t1; ++t, ++it)
          if (!outputs(0, it, t == r.t0)) return false;
        ended = true;
        return true;
      });
    }
    // The CTA must not leave while a commit is still to arrive on its barriers.
    // The last phases of "S full" and "P V done" are waited for by their readers;
    // the last of each K and V place's and of Q's "empty" have no reader left, so
    // they are waited for here, by a warp that has taken the place's last tile: the
    // tile was loaded after the phase before. (A warp that has not could find that
    // phase still open, and the one before it, of the same parity, passed: two
    // commits of a thread arrive in no order that is promised.)
    if (ended) {
      const bool mine = QT == 2 ? warp == 2 : (lane < NK) == (warp == 2);
      if (lane < NG && mine) {
        const int n = lane < NK ? NK : NV, at = lane < NK ? lane : lane - NK;
        const int uses = (it - at + n - 1) / n;  // of this lane's place
        if (it > at) mbar_wait(bar(kEmpty + lane), (uses - 1) & 1, p.err);
      }
      if (warp == 2) mbar_wait(bar(kQEmpty), qph ^ 1, p.err);
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------------- softmax
    if constexpr (QT == 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    const int x = (warp - 4) >> 2;  // query tile of this warpgroup
    const int wq = warp & 3;        // tensor-memory lanes 32 wq .. 32 wq + 31
    const int r_ = wq * 32 + lane;  // row
    const int tok = r_ >> p.lg_group, g = r_ & (G - 1);
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const float qs = p.q_scale;
    RingPos<NV> vpos(NK);
    int it = 0;
    TreeHeader none{};
    none.first = -1;
    const bool teller = warp == 4 && lane == 0;
    TreeHeader* hdr = p.hdr + 2 * me;
    if (teller) hdr[0] = hdr[1] = none;
    // Up to 64 rows an item, warps wq = 2, 3 have no rows: they store the outputs
    // that warps 0, 1 leave in shared memory (barriers "there" and "taken", 64
    // threads), while those go on with the next run.
    const bool relay = QT == 1 && p.slot_rows <= 64;
    const int there = 1 + pipe * 4 + (wq & 1) * 2, taken = there + 1;
    bool left_some = false, failed = false;
    auto fail = [&] {  // a wait gave up
      failed = true;
      return false;
    };
    runs([&](const TreeRun& r) {
      const int my_tok = r.row_item * item_tokens + x * TOK + tok;  // token of this sequence's n
      const bool real = my_tok < r.n;
      // (warps without a row compute nothing, but take part in every barrier)
      const bool warp_real = (r.row_item * item_tokens + x * TOK + ((wq * 32) >> p.lg_group)) < r.n;
      const int before = r.L - r.n;  // tokens every row sees
      // the row's parent, read here so that it (and its line) is there for the
      // tiles of the step's own rows
      int parent = -1;
      if (p.parents != nullptr && real) parent = __ldg(p.parents + r.q0 + my_tok);
      float m_use = -INFINITY, l_run = 0.0f;
      for (int t = r.t0; t < r.t1; ++t, ++it) {
        if (!wait_all(bar(kS + 2 * x + (it & 1)), (it >> 1) & 1)) return fail();
        tc::fence_after_sync();
        const int key0 = t * KEYN;
        float alpha = 1.0f;
        uint32_t pw[KEYN / 2];
        if (warp_real) {
          uint32_t sv[KEYN];
          tc::ld64_wait(t_s(x, it & 1) + lane_off, sv);
          if (key0 + KEYN > before) {
            // bit i: key key0 + i is seen. Keys before the step, then the row's
            // own and its ancestors' (a parent comes before its child).
            const int rel = key0 - before;  // row of the step that key 0 of the tile is
            uint64_t seen = rel >= 0 ? 0ull : rel <= -64 ? ~0ull : (1ull << -rel) - 1;
            if (real) {
              if (p.parents == nullptr) {
                const int top = my_tok - rel;  // a chain: every earlier row
                if (top >= 63) seen = ~0ull;
                else if (top >= 0) seen |= (2ull << top) - 1;
              } else {
                // (a load for each ancestor, one after the other, in each of the row's own
                // tiles: 4 sequences of 8,192 tokens and a chain of 64 rows 52.6 us, of 512
                // 538, of 2,048 14,150; without parents 51.0, 298 and 1,270)
                int a = my_tok, up = parent;
                while (a >= rel) {
                  if (a - rel < 64) seen |= 1ull << (a - rel);
                  if (up >= a || up < -1) {
                    atomicOr(p.err, PA_DEVERR_DRAFT);
                    break;
                  }
                  a = up;
                  if (a < 0) break;
                  up = __ldg(p.parents + r.q0 + a);
                }
              }
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const uint32_t bits = static_cast<uint32_t>(seen >> (32 * c));
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (!((bits >> i) & 1)) sv[32 * c + i] = 0xff800000u;  // -inf
            }
          }
          float mx4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(__uint_as_float(sv[i]), __uint_as_float(sv[i + 4]));
#pragma unroll
          for (int i = 8; i < KEYN; i += 2)
            mx4[(i >> 1) & 3] = max3(mx4[(i >> 1) & 3], __uint_as_float(sv[i]), __uint_as_float(sv[i + 1]));
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * qs;
          const bool move = mx > m_use + 8.0f;
          const float m_new = move ? mx : m_use;
          alpha = move ? exp2_fast(m_use - m_new) : 1.0f;
          // a row that has seen no key yet keeps m = -inf and weights of 0
          const float m_sub = m_new == -INFINITY ? 0.0f : -m_new;
          const uint64_t q2 = pair_of(qs, qs), m2 = pair_of(m_sub, m_sub);
          uint64_t rs = 0;
#pragma unroll
          for (int e = 0; e < KEYN / 2; ++e) {
            float a, b;
            floats_of(fma2(pair_of(__uint_as_float(sv[2 * e]), __uint_as_float(sv[2 * e + 1])), q2, m2), a, b);
            pw[e] = pack_bf16x2(exp2_fast(a), exp2_fast(b));
            rs = add2(rs, pair_of(__uint_as_float(pw[e] << 16), __uint_as_float(pw[e] & 0xffff0000u)));
          }
          float rs0, rs1;
          floats_of(rs, rs0, rs1);
          l_run = l_run * alpha + (rs0 + rs1);
          m_use = m_new;
        }
        const bool rescale = t > r.t0 && __any_sync(kFullMask, alpha != 1.0f);
        if (rescale) {
          if (!wait_all(bar(kO + 2 * x + ((it - 1) & 1)), ((it - 1) >> 1) & 1)) return fail();
          tc::fence_after_sync();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tc::ld32_wait(t_o(x) + lane_off + c * 32, ov);
#pragma unroll
            for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
            tc::st32(t_o(x) + lane_off + c * 32, ov);
          }
        }
        __syncwarp();  // (lanes parted over their ancestors; the store is the warp's)
        if (warp_real) {
          tc::st32(t_s(x, it & 1) + lane_off, pw);
          tc::wait_st();
        }
        if (key0 + KEYN > r.L) {
          // keys past the context: stale or unwritten V rows become zeros (their
          // P is 0, but 0 * NaN would not be), by each query tile for its own P V
          if (!wait_all(bar(kFull + vpos.st), vpos.ph)) return fail();
          const int nkeys = r.L - key0;
          const uint32_t vb = gran(vpos.st);
          constexpr int kVecs = 8 * HALVES;
          for (int i = r_; i < (KEYN - nkeys) * kVecs; i += 128) {
            const int row = nkeys + i / kVecs, c = i % kVecs;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                             vb + (c >> 3) * Cfg::kGranHalf + row * 128 + ((c & 7) << 4)),
                         "r"(0u)
                         : "memory");
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        vpos.step();
        tc::fence_before_sync();
        mbar_arrive(bar(kP + 2 * x + (it & 1)));
      }
      // the run's end: O of all its tiles. (A phase of "P V done" that is waited for is the
      // next one of its barrier: S of tile i is issued after P V of tile i - 2.)
      if (r.t1 - r.t0 > 1 && !wait_all(bar(kO + 2 * x + (it & 1)), ((it - 2) >> 1) & 1)) return fail();
      if (!wait_all(bar(kO + 2 * x + ((it - 1) & 1)), ((it - 1) >> 1) & 1)) return fail();
      tc::fence_after_sync();
      const bool whole = r.t0 == 0 && r.t1 == r.nt;
      // row r_ of the item is output row base + (r_ >> lg_group) * num_heads + its head
      const int64_t base = (static_cast<int64_t>(r.q0) + r.row_item * item_tokens + x * TOK) * p.num_heads +
                           (r.h << p.lg_group);
      // the relay's place: Q's rows 64 .. 127 hold nothing; 32 rows a warp (8 KB, 16-byte
      // pieces swizzled by row), so that the stores are whole rows
      const uint32_t place = q_s(0) + 64 * 128 + (D == 128 ? (wq & 1) * Cfg::kQHalf : (wq & 1) * 4096);
      if (relay && wq >= 2) {
        const int left = ((r.n - r.row_item * item_tokens) << p.lg_group) - (wq - 2) * 32;  // rows from the warp's on
        if (!whole || left <= 0) return true;
        // a store takes kPer rows: row i kPer + (lane / kPieces), piece lane % kPieces
        constexpr int kPieces = D / 8, kPer = 32 / kPieces, kN = 32 / kPer;
        const int sub = lane / kPieces, c = lane % kPieces;
        const uint32_t from = place + sub * D * 2;
        __nv_bfloat16* dst = p.out + base * D + c * 8;
        const int skip = (p.num_heads - G) * D;  // elements between the rows of two tokens, beyond a row
        asm volatile("bar.sync %0, 64;" ::"r"(there) : "memory");
        uint4 w[kN];
#pragma unroll
        for (int i = 0; i < kN; ++i)
          w[i] = lds128(from + i * kPer * D * 2 + ((c ^ ((i * kPer + sub) & 7)) << 4));
        asm volatile("bar.arrive %0, 64;" ::"r"(taken) : "memory");
#pragma unroll
        for (int i = 0; i < kN; ++i) {
          const int row = i * kPer + sub, rr = (wq - 2) * 32 + row;
          if (row < left)
            *reinterpret_cast<uint4*>(dst + rr * D + static_cast<int64_t>(rr >> p.lg_group) * skip) = w[i];
        }
        return true;
      }
      if (!warp_real) return true;
      if (whole) {
        const float inv = 1.0f / l_run;
        if (relay) {
          if (left_some) asm volatile("bar.sync %0, 64;" ::"r"(taken) : "memory");
          left_some = true;
          const uint32_t row_at = place + lane * D * 2;
          const int sw = (lane & 7) << 4;
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t ov[64];
            tc::ld64_wait(t_o(x) + lane_off + c * 64, ov);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                w[i] = pack_bf16x2(__uint_as_float(ov[8 * v + 2 * i]) * inv, __uint_as_float(ov[8 * v + 2 * i + 1]) * inv);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(row_at + (((c * 8 + v) << 4) ^ sw)),
                           "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                           : "memory");
            }
          }
          asm volatile("bar.arrive %0, 64;" ::"r"(there) : "memory");
        } else {
          __nv_bfloat16* dst = p.out + (base + static_cast<int64_t>(tok) * p.num_heads + g) * D;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t ov[32];
            tc::ld32_wait(t_o(x) + lane_off + c * 32, ov);
            if (real) {
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                uint4 w;
                w.x = pack_bf16x2(__uint_as_float(ov[8 * v]) * inv, __uint_as_float(ov[8 * v + 1]) * inv);
                w.y = pack_bf16x2(__uint_as_float(ov[8 * v + 2]) * inv, __uint_as_float(ov[8 * v + 3]) * inv);
                w.z = pack_bf16x2(__uint_as_float(ov[8 * v + 4]) * inv, __uint_as_float(ov[8 * v + 5]) * inv);
                w.w = pack_bf16x2(__uint_as_float(ov[8 * v + 6]) * inv, __uint_as_float(ov[8 * v + 7]) * inv);
                *reinterpret_cast<uint4*>(dst + c * 32 + v * 8) = w;
              }
            }
          }
        }
      } else {
        // a part of an item: [D / 4][rows][4] so that a warp's stores are whole lines
        const int side = r.t0 > 0 ? 0 : 1;
        const int64_t slot = 2 * static_cast<int64_t>(me) + side;
        const int row = x * kTreeRows + r_;
        if (real) {
          p.ws_ml[slot * p.slot_rows + row] = make_float2(m_use, l_run);
        }
        float* dst = p.ws_acc + (slot * D * p.slot_rows) + row * 4;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t ov[32];
          tc::ld32_wait(t_o(x) + lane_off + c * 32, ov);
          if (real) {
#pragma unroll
            for (int v = 0; v < 8; ++v)
              *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(c * 8 + v) * p.slot_rows * 4) =
                  make_uint4(ov[4 * v], ov[4 * v + 1], ov[4 * v + 2], ov[4 * v + 3]);
          }
        }
        if (teller) {
          TreeHeader hd{};
          const int tok0 = r.row_item * item_tokens;
          hd.out_row = (static_cast<int64_t>(r.q0) + tok0) * p.num_heads + (r.h << p.lg_group);
          hd.rows = min(item_tokens, r.n - tok0) << p.lg_group;
          hd.first = static_cast<int>((u0 + r.tile_unit) / share);
          hd.last = static_cast<int>((u0 + r.tile_unit + r.nt - 1) / share);
          hdr[side] = hd;
        }
      }
      // (the next run's first P V overwrites O once P of its first tile is
      // published, which these threads do after the loads above)
      return true;
    });
    if (relay && failed) {  // let the other warp go
      asm volatile("bar.arrive %0, 64;" ::"r"(wq >= 2 ? taken : there) : "memory");
    } else if (left_some) {
      asm volatile("bar.sync %0, 64;" ::"r"(taken) : "memory");
    }
  }

  tc::fence_before_sync();
  __syncthreads();
  if (cta_warp == 2) tc::tmem_dealloc(*tmem_slot, Cfg::kTmemCols);
}

// Merge of the items that were split:
//   M = max m_j,  out = sum 2^(m_j - M) O_j / sum 2^(m_j - M) l_j
// over all parts j in which the row saw a key: those whose sum l_j is not 0. (Not by m_j:
// it is -inf as well where all that the row saw are NaN, whose sum is NaN, and so is the
// row then.) An item's pieces (32 rows x 4 kMergeCols columns, a lane one row)
// are dealt to as many CTAs as it has parts, times one per 128 rows. With fewer pieces
// than warps, W warps share a piece, taking the parts in turn and joining in shared
// memory in their order; so the sums' order goes by the item's rows and parts alone.
// Bound by the round trips of a warp, kMergeParts W parts each: with 16 columns a lane
// (eight loads in flight; of 7 parts and 4 columns two were, most items having two parts)
// the merge adds 4.4 us to 8 requests (7.3 before) and 5 to 256 (9).
constexpr int kMergeParts = 2, kMergeCols = 4, kMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(kMergeWarps * 32, 2) tree_merge_kernel(const TreeParams p) {
  __shared__ float s_m[kMergeWarps][32], s_l[kMergeWarps][32];
  __shared__ float4 s_acc[kMergeWarps][kMergeCols][32];
  pdl_wait();
  pdl_launch_dependents();
  const int slot = blockIdx.x, cta = slot >> 1;
  const TreeHeader hd = p.hdr[slot];
  if (hd.first < 0) return;
  const int parts = hd.last - hd.first + 1;
  const int rank = (cta - hd.first) * gridDim.y + blockIdx.y, ctas = parts * gridDim.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int groups = (hd.rows + 31) >> 5, pieces = groups * (D / 4 / kMergeCols);
  const int mine = (pieces - rank + ctas - 1) / ctas;  // pieces rank, rank + ctas, ...
  if (mine <= 0) return;
  const int W = mine >= 5 ? 1 : mine >= 3 ? 2 : mine == 2 ? 4 : 8;
  const int sub = warp & (W - 1);
  for (int k0 = 0; k0 < mine; k0 += kMergeWarps / W) {
    const int k = k0 + warp / W;
    const int w = rank + k * ctas;
    const int row = (w % groups) * 32 + lane, col = w / groups * kMergeCols;  // (columns in fours)
    const bool on = k < mine && row < hd.rows;
    float M = -INFINITY, l = 0.0f;
    float4 acc[kMergeCols];
#pragma unroll
    for (int c = 0; c < kMergeCols; ++c) acc[c] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    auto scale = [&](float f) {
      l *= f;
#pragma unroll
      for (int c = 0; c < kMergeCols; ++c) {
        acc[c].x *= f;
        acc[c].y *= f;
        acc[c].z *= f;
        acc[c].w *= f;
      }
    };
    auto add = [&](float f, float l2, const float4 (&v)[kMergeCols]) {
      l = fmaf(f, l2, l);
#pragma unroll
      for (int c = 0; c < kMergeCols; ++c) {
        acc[c].x = fmaf(f, v[c].x, acc[c].x);
        acc[c].y = fmaf(f, v[c].y, acc[c].y);
        acc[c].z = fmaf(f, v[c].z, acc[c].z);
        acc[c].w = fmaf(f, v[c].w, acc[c].w);
      }
    };
    if (on) {
      const float* ml = reinterpret_cast<const float*>(p.ws_ml + row);
      const float* av = p.ws_acc + (static_cast<int64_t>(col) * p.slot_rows + row) * 4;
      for (int j0 = sub; j0 < parts; j0 += kMergeParts * W) {
        float2 mq[kMergeParts];
        float4 v[kMergeParts][kMergeCols];
#pragma unroll
        for (int j = 0; j < kMergeParts; ++j) {
          const int jj = j0 + j * W;
          mq[j] = make_float2(-INFINITY, 0.0f);
          if (jj < parts) {
            // the first part lies in its pipeline's second slot, the others in the first
            const int64_t sl = 2 * static_cast<int64_t>(hd.first + jj) + (jj == 0 ? 1 : 0);
            mq[j] = ld_cg_f32x2(ml + sl * p.slot_rows * 2);
#pragma unroll
            for (int c = 0; c < kMergeCols; ++c) v[j][c] = ld_cg_f32x4(av + (sl * D + c * 4) * p.slot_rows);
          }
        }
        float bm = M;
        bool any = false;
#pragma unroll
        for (int j = 0; j < kMergeParts; ++j) {
          bm = fmaxf(bm, mq[j].x);
          any |= mq[j].y != 0.0f;
        }
        if (!any) continue;  // this row saw no key in these parts
        scale(exp2f(M - bm));
#pragma unroll
        for (int j = 0; j < kMergeParts; ++j)
          if (mq[j].y != 0.0f) add(exp2f(mq[j].x - bm), mq[j].y, v[j]);  // (else no part, or none of its keys seen)
        M = bm;
      }
    }
    if (W > 1) {  // (the same for the whole CTA)
      __syncthreads();
      s_m[warp][lane] = M;
      s_l[warp][lane] = l;
#pragma unroll
      for (int c = 0; c < kMergeCols; ++c) s_acc[warp][c][lane] = acc[c];
      __syncthreads();
      if (sub != 0) continue;
      for (int i = 1; i < W; ++i) {
        const float m2 = s_m[warp + i][lane], l2 = s_l[warp + i][lane];
        if (l2 == 0.0f) continue;
        const float bm = fmaxf(M, m2);
        float4 v[kMergeCols];
#pragma unroll
        for (int c = 0; c < kMergeCols; ++c) v[c] = s_acc[warp + i][c][lane];
        scale(exp2f(M - bm));
        add(exp2f(m2 - bm), l2, v);
        M = bm;
      }
    }
    if (!on) continue;
    const float inv = 1.0f / l;
    const int64_t out = hd.out_row + static_cast<int64_t>(row >> p.lg_group) * p.num_heads +
                        (row & ((1 << p.lg_group) - 1));
    __nv_bfloat16* dst = p.out + out * D + col * 4;
#pragma unroll
    for (int c = 0; c < kMergeCols; ++c)
      *reinterpret_cast<uint2*>(dst + 4 * c) =
          make_uint2(pack_bf16x2(acc[c].x * inv, acc[c].y * inv), pack_bf16x2(acc[c].z * inv, acc[c].w * inv));
  }
}

cudaError_t encode_tree_q(CUtensorMap* map, const void* q, int total_q, int num_heads, int head_dim,
                          int group, int box_tokens) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t row = static_cast<cuuint64_t>(head_dim) * 2;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(head_dim), static_cast<cuuint64_t>(num_heads),
                              static_cast<cuuint64_t>(total_q)};
  const cuuint64_t strides[2] = {row, static_cast<cuuint64_t>(num_heads) * row};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(box_tokens)};
  const cuuint32_t es[3] = {1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(q), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Cache [num_blocks][block_size][Hkv][D] viewed (column, token, head, block).
cudaError_t encode_tree_kv(CUtensorMap* map, const void* base, const TreeShape& sh, int rows) {
  auto enc = tensor_map_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t row = static_cast<cuuint64_t>(sh.head_dim) * 2;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(sh.head_dim), static_cast<cuuint64_t>(sh.block_size),
                              static_cast<cuuint64_t>(sh.num_kv_heads),
                              static_cast<cuuint64_t>(sh.num_blocks)};
  const cuuint64_t strides[3] = {row * sh.num_kv_heads, row,
                                 row * sh.num_kv_heads * static_cast<cuuint64_t>(sh.block_size)};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                   box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, int QT>
cudaError_t launch_tree_t(const TreeShape& sh, const TreeParams& p, const void* q, const void* k_cache,
                          const void* v_cache, cudaStream_t stream) {
  using Cfg = TreeConfig<D, QT>;
  static std::atomic<unsigned long long> configured{0};
  cudaError_t e = ensure_smem(pa_tree_kernel<D, QT>, Cfg::kSmemBytes, configured);
  if (e != cudaSuccess) return e;
  CUtensorMap qmap, kmap, vmap;
  const int rows = sh.block_size < kTreeKeys ? sh.block_size : kTreeKeys;
  if ((e = encode_tree_q(&qmap, q, sh.total_q, sh.num_heads, D, 1 << p.lg_group, p.q_box_tokens)) != cudaSuccess) return e;
  if ((e = encode_tree_kv(&kmap, k_cache, sh, rows)) != cudaSuccess) return e;
  if ((e = encode_tree_kv(&vmap, v_cache, sh, rows)) != cudaSuccess) return e;
  const unsigned parts = static_cast<unsigned>(tree_pipelines(QT));
  e = launch_pdl(pa_tree_kernel<D, QT>, dim3(parts / Cfg::kPipes), dim3(Cfg::kThreads), Cfg::kSmemBytes, stream,
                 qmap, kmap, vmap, p);
  // Where no table holds an item long enough to be cut there is nothing to merge. The host
  // knows the tables' width, not the lengths: one request of 300 tokens takes 10.0 us with a
  // table of its length, and 11.7, with the empty launch, with one for 32,768 tokens.
  const int64_t tiles = (static_cast<int64_t>(sh.max_blocks_per_seq) * sh.block_size + kTreeKeys - 1) / kTreeKeys;
  if (e != cudaSuccess || tiles + kTreeItemCost <= kTreeWhole) return e;
  // (two CTAs for each part of an item of 256 rows; more only add CTAs, which cost more than
  // they save: of smaller items 592 are launched, eight times as many took 7 us longer)
  return launch_pdl(tree_merge_kernel<D>, dim3(2 * parts, std::max(1, p.slot_rows / 128)), dim3(kMergeWarps * 32), 0,
                    stream, p);
}

}  // namespace

int tree_query_tiles(int num_heads, int num_kv_heads, int max_query_len) {
  const int64_t rows = static_cast<int64_t>(max_query_len) * (num_heads / num_kv_heads);
  return rows > kTreeRows ? 2 : 1;
}

int tree_pipelines(int query_tiles) { return query_tiles == 1 ? 2 * 148 : 148; }

TreeWorkspace tree_workspace(int num_heads, int num_kv_heads, int head_dim, int max_query_len) {
  TreeWorkspace w{};
  const int qt = tree_query_tiles(num_heads, num_kv_heads, max_query_len);
  const int64_t rows = static_cast<int64_t>(max_query_len) * (num_heads / num_kv_heads);
  w.slots = 2 * tree_pipelines(qt);
  // (grows with max_query_len: a workspace for more rows serves fewer)
  w.slot_rows = qt == 2 ? 2 * kTreeRows : static_cast<int>((rows + 31) / 32 * 32);
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const size_t each = static_cast<size_t>(w.slots) * w.slot_rows;
  w.ml_off = up(static_cast<size_t>(2 * tree_pipelines(1)) * sizeof(TreeHeader));
  w.acc_off = w.ml_off + up(each * sizeof(float2));
  w.total = w.acc_off + each * head_dim * sizeof(float);
  return w;
}

cudaError_t launch_decode_tree(const TreeShape& sh, void* out, const void* q, const void* k_cache,
                               const void* v_cache, const int32_t* block_tables,
                               const int32_t* context_lens, const int32_t* query_start,
                               const int32_t* parents, void* workspace, cudaStream_t stream) {
  const TreeWorkspace w =
      tree_workspace(sh.num_heads, sh.num_kv_heads, sh.head_dim, sh.max_query_len);
  TreeParams p{};
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.out = static_cast<__nv_bfloat16*>(out);
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.parents = parents;
  cudaError_t e = device_error_word(&p.err);
  if (e != cudaSuccess) return e;
  p.hdr = reinterpret_cast<TreeHeader*>(ws);
  p.ws_ml = reinterpret_cast<float2*>(ws + w.ml_off);
  p.ws_acc = reinterpret_cast<float*>(ws + w.acc_off);
  p.num_heads = sh.num_heads;
  p.num_kv_heads = sh.num_kv_heads;
  const int group = sh.num_heads / sh.num_kv_heads;
  p.lg_group = group == 1 ? 0 : group == 2 ? 1 : group == 4 ? 2 : 3;
  p.block_size = sh.block_size;
  int lg = 0;
  while ((1 << lg) < sh.block_size) ++lg;
  p.log2_block_size = lg;
  p.num_blocks = sh.num_blocks;
  p.max_blocks_per_seq = sh.max_blocks_per_seq;
  p.num_seqs = sh.num_seqs;
  p.total_q = sh.total_q;
  p.max_query_len = sh.max_query_len;
  p.slot_rows = w.slot_rows;
  p.q_box_tokens = sh.max_query_len < kTreeRows / group ? sh.max_query_len : kTreeRows / group;
  p.q_scale = sh.scale * 1.4426950408889634f;  // log2(e)
  const int qt = tree_query_tiles(sh.num_heads, sh.num_kv_heads, sh.max_query_len);
  if (sh.head_dim == 64)
    return qt == 1 ? launch_tree_t<64, 1>(sh, p, q, k_cache, v_cache, stream)
                   : launch_tree_t<64, 2>(sh, p, q, k_cache, v_cache, stream);
  return qt == 1 ? launch_tree_t<128, 1>(sh, p, q, k_cache, v_cache, stream)
                 : launch_tree_t<128, 2>(sh, p, q, k_cache, v_cache, stream);
}

}  // namespace pa
