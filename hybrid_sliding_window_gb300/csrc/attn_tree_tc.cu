// Draft-tree attention on the 5th-generation tensor cores (tcgen05 + TMEM + TMA):
// bf16 KV with D = 64 or 128, or E4M3 KV with D = 128; any GQA group and page
// size.
//
// Method: node i of a request reads the cached columns of its window and its
// ancestors' columns behind the prefix (include/swa.h, swa_attn_tree).  With T
// nodes and G query heads per KV head, T x G query rows share every K and V
// row, 4 D T G flops on 4 D bytes (bf16): up to about 256 rows the kernel is
// bound by reading the cache once, beyond that by the tensor cores and the
// softmax between them.
//
// Work: an item is a block of up to 2 * floor(128 / G) nodes of one request for
// one KV head; its keys are cut into tiles of 128 columns.  The tiles of all
// items of one head form one line, and the CTAs of that head - groups =
// #SMs / Hkv of them - take equal stretches of it, whatever the requests'
// lengths are, so one long request fills the GPU and a ragged batch has no
// tail.  CTAs of the same stretch and different heads are neighbours: a token's
// head rows lie next to each other and are read at about the same time.  A
// CTA's piece of an item is a segment.  Segments that hold an item's whole key
// range write its output; the others write (max, sum, unnormalised output)
// partials - at most two per CTA - which a second, dependent launch merges in
// group order, so results do not depend on timing and the workspace needs no
// initial contents.  Layers whose items have few keys (short windows) are dealt
// out in whole items and need no second launch.
//
// A CTA (one per SM) has warp-specialised roles that meet on mbarriers, with
// phases following running counts so that nothing drains between segments:
//   * warp 9, the producer, finds the CTA's segments (warp-wide prefix sums over
//     the requests), hands them to the other roles through a two-slot ring,
//     looks page rows up 32 page slots at a time and loads K tiles by TMA; warp
//     11 does the same for V.  K and V tiles share one ring, in the order in
//     which the products use them.  (One warp for both: a TMA box costs its
//     issuing thread 75 to 100 cycles, sixteen of them per tile pair on pages
//     of 16 rows, which was the pace of such layers.)
//     Pages that are no TMA box (fewer than 16 rows, more than 64, no power of
//     two) are gathered instead: the same two warps look up a row per key and copy
//     it with 16-byte cp.async into the same layout, 64 copies a lane and tile
//     (16 requests of 4K to 32K tokens, full layer, floor 95 us: 174 us on pages of
//     1 or 8, 116 on pages of 16 or 64, 24.7 ms on the generic kernel; the two
//     warps' copy instructions are the pace).
//   * warp 10 loads each segment's Q tiles once the previous segment's last
//     QK^T has read them;
//   * warp 8 issues S = Q K^T and O += P V with P in TMEM over S;
//   * warps 0-3 and 4-7 are two softmax groups.  Rows of an item that fill two
//     Q tiles: one tile each, both read the same key tiles.  Rows that fit one
//     Q tile: the groups take alternate key tiles with an accumulator each, so
//     that one group's softmax overlaps the other's products, and the two
//     accumulators are joined in TMEM's own lanes at the segment's end (warps i
//     and i + 4 can read the same lanes).
// E4M3 KV: K and V tiles arrive as bytes in a ring of their own; four more warps
// turn them into f16 tiles (exact: E4M3 is a subset of f16) and each Q tile from
// bf16 to f16 in place, the products run on f16 operands, P is packed as f16, the
// K scale joins the softmax scale and the V scale the output.  (With 16 warps the
// launch has 128 registers a thread; the other roles give the softmax groups 24
// each, setmaxnreg.)
// Key columns that some row may not read (window edge, non-ancestors) get -inf
// scores from a 64-bit mask per row and 64-column chunk; chunks that no row of
// a warp reads are skipped.
// Roundings: scores, maxima, sums, accumulators and partials are float32; weights
// are rounded to the products' type (half a step: bf16 2^-8, f16 2^-11 of each)
// and their sum is of the unrounded ones.  Against 64 bits the error of bf16
// outputs is 2.3e-3 of their size, 1.7e-3 with float32 weights (the rounding of the
// output); E4M3 KV 1.7e-3 both ways.  Float32 weights would need TF32 products,
// twice the time of PV.  A weight that is rescaled in place (when its row's
// reference rises in the tile's second chunk) is rounded again.
// Every mbarrier wait has a poll limit; on expiry the kernel sets
// SWA_DEVERR_TIMEOUT, every role leaves its loop, loads and products in flight
// are waited for, and the TMEM is released.
//
// Measured (device time with the plan; floors at 6788 GB/s and 1946 TFLOP/s):
// MiMo full layer, 64 requests of 4K to 32K tokens, 8 nodes: 409-420 us (6.6-6.75
// TB/s, floor 407); D = 64, 128 ragged trees of up to 13 nodes: 268 us (5.9 TB/s,
// floor 231); one request of 131072 tokens, 64 nodes: 200 us (1375 TFLOP/s, floor
// 141); E4M3, 4 x 131072 tokens, 16 nodes: 241 us (4.5 TB/s, floor 158); sliding
// layer, 64 requests, 8 nodes: 22 us (floor 7.7).  Past the cache's bytes the bound
// is a softmax group's loop - softmax of a tile (about 1600 cycles), its PV and its
// next S, which overwrites P - of which two run in turn.  At D = 128 TMEM holds no
// third S; at D = 64 columns 384 to 511 are free and would.  The loop is not at its
// limit: swa_attn_extend takes chains of 64 nodes at 1542 TFLOP/s, this kernel at
// 1422.  E4M3 tiles also pass shared memory twice (conversions left out: 210 us).
// Sliding layers are latency: 8 us for one request, 7.4 us for each further pair
// of items of a CTA, which has room for no second CTA beside it.
#include <algorithm>

#include <math.h>

#include "spec_internal.h"
#include "tc_ptx.cuh"

namespace swa {
namespace {

using namespace tc;

constexpr int kTileRows = 128;               // rows of a Q tile (M)
constexpr int kKeys = 128;                   // keys of a K/V tile
constexpr int kBlock = kTileRows * 64 * 2;   // one 64-column block of a tile
constexpr int kTreeThreads = 384;            // 8 softmax warps, MMA, and three that load
constexpr int kConvThreads = 128;            // E4M3 KV: warps 12-15 convert
constexpr float kRescaleGap = 8.f;           // log2 units: rescale O when the max grows more
constexpr float kSumCap = 32768.f;           // a chunk's weight sum that forces a maximum pass
constexpr int kMergeThreads = 256;
constexpr int kMergeRows = 32;               // rows of one merge CTA: one per lane

template <int D, bool F8>
struct TreeGeo {
  static constexpr int kTileBytes = kKeys * D * 2;
  static constexpr int kStages = F8 ? 3 : D == 128 ? 5 : 8;   // operand tiles
  static constexpr int kRawBytes = kKeys * D;                 // E4M3 tiles as loaded
  static constexpr int kRawStages = F8 ? 4 : 0;
  static constexpr int kOffRing = 2 * kTileBytes;             // after the Q tiles
  static constexpr int kOffRaw = kOffRing + kStages * kTileBytes;
  static constexpr int kOffStat = kOffRaw + kRawStages * kRawBytes;
  static constexpr int kOffBars = kOffStat + 2 * kTileRows * 8;
  static constexpr int kOffCtl = kOffBars + 40 * 8;           // Control
  static constexpr int kThreads = kTreeThreads + (F8 ? kConvThreads : 0);
};

struct TreeParams {
  int kind, window, hkv, G, T, ps, ps_shift;   // T: nodes of a Q tile
  int64_t page_stride, pool_rows;
  KvAddr addr;               // gathered pages: where rows live
  const int32_t *rt;
  int64_t rt_stride;
  const int64_t *req_idx, *pre, *qo_indptr;
  int bs, groups, max_new;
  int blocks;                // most blocks of 2 T nodes of a request
  int whole;                 // 1: CTAs take whole items, nothing is merged
  int wide_out;              // out is 32-byte aligned
  int64_t n_tokens;
  int lookback;              // the plan's
  PlanView plan;
  TreeView tree;
  const float *sinks;
  float scale_log2;          // E4M3 KV: with the K scale
  float v_scale;             // 1 unless E4M3 KV
  __nv_bfloat16 *out;
  float *partials;           // [CTA][2][D / 4][rows][4], then [rows][2] (max, sum)
  int rows_max;              // rows of an item
  int64_t part_stride;       // floats of one partial
  struct MergeDesc *desc;    // [CTA]
  int32_t *err;
};

// A CTA's last segment when it starts an item that goes on in the next groups.
struct MergeDesc {
  int32_t parts;     // contributing CTAs (0: nothing to merge)
  int32_t n_tok;     // nodes of the item
  int32_t q0;        // first query row
};

// A piece of the CTA's work.
//   alternate  one Q tile; step u takes key tile u, the groups' accumulators are
//              joined at the end
//   shared     two Q tiles of one item, a key tile serves both groups
//   pair       two whole items of one Q tile each, one per group, each with its
//              own key tiles (the shorter one's are padded: masked, so 0)
enum { kAlternate = 0, kShared = 1, kPair = 2 };
struct Piece {                 // what a group works on
  int b, n0, n_tok;            // request, first node, nodes
  int q0, col0, prefix;        // first query row, first key column, cached columns
};
struct Segment {
  int mode, n_tiles;           // mode -1: end; key tiles (of each piece)
  int part;                    // -1: whole item; else the partial's slot
  Piece piece[2];              // [1]: pairs only
};
// Key tiles that pass through the ring, in steps' order.
__device__ __forceinline__ int ring_tiles(int mode, int n) { return mode == kPair ? 2 * n : n; }

// Shared words of the roles.  (Everything lives in the dynamic array, whose
// start is 1024-byte aligned: the tiles leave no room for an alignment gap.)
struct Control {
  Segment seg[2];
  int fills[8];              // fills of each slot of the loads' ring
  uint32_t tmem;
  int abort;
};

enum { B_IFULL = 0, B_IEMPTY = 2, B_FULLQ = 4, B_QFREE = 5, B_SDONE = 6, B_PREADY = 8,
       B_ODONE = 10, B_STAT = 12, B_EPI = 13, B_DRAIN = 14, B_FULL = 15, B_EMPTY = 23,
       B_RAWFULL = 31, B_RAWEMPTY = 35, B_QCONV = 39, B_COUNT = 40 };

// Position in the ring of key tile i's K or V, of the n tiles of a segment: K0
// K1 V0 K2 V1 ... - the order in which the products release them.
__device__ __forceinline__ int seq_k(int i) { return i == 0 ? 0 : 2 * i - 1; }
__device__ __forceinline__ int seq_v(int i, int n) { return min(2 * i + 2, 2 * n - 1); }

// One request's nodes and keys as the schedule sees them.
struct Request {
  int q0, prefix, col0, n;
};
constexpr int kMaxCol = 0x7fffffff - 2 * SWA_TREE_MAX_NODES;
__device__ __forceinline__ int n_blocks(const TreeParams &P, const Request &r) {
  return (r.n + 2 * P.T - 1) / (2 * P.T);
}
// Key tiles of one of its blocks of nodes.
__device__ __forceinline__ int block_tiles(const TreeParams &P, const Request &r, int blk) {
  const int last = min((blk + 1) * 2 * P.T, r.n);   // nodes up to the block's end
  return ((r.prefix + last - 1 - r.col0) >> 7) + 1;
}
__device__ __forceinline__ Request request(const TreeParams &P, int b) {
  Request r{0, 0, 0, 0};
  if (b >= P.bs) return r;
  const int64_t q0 = P.qo_indptr[b], end = P.qo_indptr[b + 1], prefix = P.pre[b];
  int64_t n = end - q0;
  if (n <= 0) return r;
  const int64_t room =
      (P.kind == SWA_LAYER_FULL && P.rt_stride < kMaxCol ? P.rt_stride : kMaxCol) - prefix;
  if (q0 < 0 || end > P.n_tokens || n > P.max_new || prefix < 0 || n > room) {
    set_error(P.err, SWA_DEVERR_RANGE);
    if (q0 < 0 || q0 >= P.n_tokens || prefix < 0 || room <= 0) return r;
    n = min(min(n, P.n_tokens - q0), min((int64_t)P.max_new, room));
  }
  r.q0 = (int)q0;
  r.prefix = (int)prefix;
  r.n = (int)n;
  r.col0 = (int)first_position(P.kind, P.window, prefix) >> P.ps_shift << P.ps_shift;
  return r;
}

// First row (in the layer's K/V view) of the page holding column `col`; rec is
// its req_to_token entry (full layers) or its page in the request's plan, -1
// when the plan has none.  An offending page reads as page 0.
__device__ __forceinline__ int32_t page_rec(bool full, int ps_shift, const int32_t *rt_row,
                                            const int32_t *hdr, const int32_t *pages, int first,
                                            int max_pages, int col) {
  if (full) return rt_row[col];
  // The plan's first page is known (`first`), so the entry's load does not wait
  // for the header's, which is checked afterwards.
  const int4 h = *reinterpret_cast<const int4 *>(hdr);   // lo, hi, first page, pages
  const int k = (col >> ps_shift) - first;
  const int32_t page = k >= 0 && k < max_pages ? pages[k] : -1;
  return (col >= h.x && h.z == first && k < h.w) ? page : -1;
}
__device__ __forceinline__ int32_t page_row(const TreeParams &P, bool full, int32_t rec) {
  int64_t page = full ? (rec >= 0 ? rec >> P.ps_shift : -1) : rec;
  if (!full && page == 0) set_error(P.err, SWA_DEVERR_WINDOW_EVICTED);
  if (page < 0 || page >= P.pool_rows >> P.ps_shift) {
    set_error(P.err, SWA_DEVERR_RANGE);
    page = 0;
  }
  return (int32_t)(page * P.page_stride);
}

// Bits [x, y) of a 64-bit mask, clipped to it.
__device__ __forceinline__ uint64_t bit_range(int x, int y) {
  x = max(x, 0);
  y = min(y, 64);
  return x < y ? (~0ull >> (64 - (y - x))) << x : 0ull;
}
// Bits o .. o + 63 of an ancestor row of more than 64 bits (o may be negative;
// zeros outside).
__device__ __forceinline__ uint64_t row_bits(const uint32_t *row, int words, int o) {
  const int w = o >> 5, s = o & 31;
  uint32_t x[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) x[i] = (w + i >= 0 && w + i < words) ? row[w + i] : 0u;
  return (uint64_t)__funnelshift_r(x[0], x[1], s) | (uint64_t)__funnelshift_r(x[1], x[2], s) << 32;
}
// The same of a row of at most 64 bits.
__device__ __forceinline__ uint64_t shift_bits(uint64_t row, int o) {
  return o >= 64 || o <= -64 ? 0ull : o >= 0 ? row >> o : row << -o;
}

// (row r, 16-byte chunk c) of an operand tile: blocks of [128 rows][128 B] with the
// 128-byte swizzle.
__device__ __forceinline__ int tile_off(int r, int c) {
  return (c >> 3) * kBlock + r * 128 + (((c & 7) ^ (r & 7)) << 4);
}

template <int kD, bool kF8, bool kGather>
__global__ void __launch_bounds__(TreeGeo<kD, kF8>::kThreads, 1)
    k_tree_tc(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ TreeParams P) {
  using Gm = TreeGeo<kD, kF8>;
  static_assert(!kF8 || kD == 128, "E4M3 KV: D = 128");
  constexpr int kTileBytes = Gm::kTileBytes, kStages = Gm::kStages;
  static_assert(kStages <= 8, "barrier slots");
  // The ring that TMA fills: the operand tiles, or the E4M3 bytes.
  constexpr int kLoads = kF8 ? Gm::kRawStages : kStages;
  constexpr int kLoadBytes = kF8 ? Gm::kRawBytes : kTileBytes;
  constexpr int kOffLoad = kF8 ? Gm::kOffRaw : Gm::kOffRing;
  constexpr int bLoadFull = kF8 ? B_RAWFULL : B_FULL, bLoadEmpty = kF8 ? B_RAWEMPTY : B_EMPTY;
  extern __shared__ __align__(1024) char smem[];
  const uint32_t sb = smem_u32(smem);
  float2 *s_stat = reinterpret_cast<float2 *>(smem + Gm::kOffStat);   // [group][row] max, sum
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Gm::kOffBars);
  Control *ctl = reinterpret_cast<Control *>(smem + Gm::kOffCtl);
  volatile int &s_abort = ctl->abort;
  Segment *s_seg = ctl->seg;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int kvh = blockIdx.x % P.hkv, group_id = blockIdx.x / P.hkv;
  const int G = P.G, T = P.T, TG = T * G;
  auto bar = [&](int i) { return smem_u32(&bars[i]); };
  auto wait_all = [&](uint32_t b, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(b, parity, &s_abort));
  };

  if (sb & 1023) {   // the operand layouts need it
    if (tid == 0) set_error(P.err, SWA_DEVERR_RANGE);
    return;
  }
  if (tid == 0) s_abort = 0;
  if (tid == 32) {
    for (const CUtensorMap *m : {&tmK, &tmV, &tmQ})
      asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
  }
  if (tid < 8) ctl->fills[tid] = 0;
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     smem_u32(&ctl->tmem)),
                 "r"(512u));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::);
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_IFULL + i), 1);
      // 8 softmax warps, the MMA warp, the Q and V loaders (and four converters)
      mbar_init(bar(B_IEMPTY + i), kF8 ? 15 : 11);
      mbar_init(bar(B_SDONE + i), 1);
      mbar_init(bar(B_PREADY + i), kTileRows);
      mbar_init(bar(B_ODONE + i), 1);
    }
    mbar_init(bar(B_FULLQ), 1);
    mbar_init(bar(B_QFREE), 1);
    mbar_init(bar(B_STAT), 2 * kTileRows);
    mbar_init(bar(B_EPI), 2 * kTileRows);
    mbar_init(bar(B_DRAIN), 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(B_FULL + i), kF8 ? kConvThreads : kGather ? 32 : 1);
      mbar_init(bar(B_EMPTY + i), 1);
    }
    for (int i = 0; i < Gm::kRawStages; ++i) {
      mbar_init(bar(B_RAWFULL + i), kGather ? 32 : 1);
      mbar_init(bar(B_RAWEMPTY + i), kConvThreads / 32);
    }
    mbar_init(bar(B_QCONV), kConvThreads);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  __syncthreads();
  tc_fence_after();
  // All 512 columns: the allocation starts at address 0, which the addresses
  // below then hold as constants.
  constexpr uint32_t tmem = 0;
  constexpr uint32_t kIdS = idesc_f16(128, 128, false, kF8);
  constexpr uint32_t kIdO = idesc_f16(128, kD, true, kF8);

  int q_issued = 0;                          // Q fills, for the abort path

  // Launched as a programmatic dependent: what comes before each role's call
  // overlaps the kernel before this one on the stream, everything that reads or
  // writes global memory comes after that kernel's completion.
  auto after_previous = [] {
    asm volatile("griddepcontrol.wait;\n" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  };

  // Warp-collective, warp 10: the Q tiles of the CTA's segment nd, once the last
  // QK^T of the one before has read the buffers.
  auto load_q = [&](const Segment &sg, int nd) {
    if (nd >= 1 && !wait_all(bar(B_QFREE), (nd - 1) & 1)) return false;
    if (lane == 0) {
      const int tiles = sg.mode == kAlternate ? 1 : 2;
      mbar_expect_tx(bar(B_FULLQ), (uint32_t)(tiles * TG * 128 * (kD / 64)));
#pragma unroll
      for (int i = 0; i < 2; ++i)
        for (int h = 0; i < tiles && h < kD / 64; ++h)
          tma_load_3d(sb + i * kTileBytes + h * kBlock, &tmQ, h * 64, kvh * G,
                      (int)(sg.mode == kPair && i ? sg.piece[1].q0 : sg.piece[0].q0 + i * T),
                      bar(B_FULLQ));
      ++q_issued;
    }
    __syncwarp();
    return true;
  };

  // Warp-collective: the K tiles (warp 9) or the V tiles (warp 11) of a segment
  // whose first tile has position `base` in the ring of the loads.
  const bool full_layer = P.kind == SWA_LAYER_FULL;
  const int ppt = kGather ? 1 : kKeys >> P.ps_shift;   // pages per key tile
  auto stream = [&](const Segment &sg, int base) {
    const bool pair = sg.mode == kPair;
    // Page records and rows of piece w: 32 page slots at a time, lane i slot i.
    auto rec_of = [&](int w, int k) {
      const Piece &pc = sg.piece[w];
      const int pg0 = pc.col0 >> P.ps_shift;
      const int hi = pc.prefix + pc.n0 + pc.n_tok - 1;       // the item's last column
      // A windowed request's first page may start before its first planned
      // column: look it up by a column that is in the plan.  Page slots behind
      // the last column load its page again: finite values, zero weight.
      const int lo = (int)first_position(P.kind, P.window, pc.prefix);
      const int i = min(32 * k + lane, (hi >> P.ps_shift) - pg0);
      const int col = max((pg0 + i) << P.ps_shift, lo);
      return page_rec(full_layer, P.ps_shift,
                      full_layer ? P.rt + P.req_idx[pc.b] * P.rt_stride : nullptr,
                      full_layer ? nullptr : P.plan.hdr + pc.b * 4,
                      full_layer ? nullptr : P.plan.pages + (int64_t)pc.b * P.plan.max_pages,
                      max(pc.prefix - P.lookback, 0) >> P.ps_shift, P.plan.max_pages, col);
    };
    const int n = ring_tiles(sg.mode, sg.n_tiles), n_slots = sg.n_tiles * ppt;
    const int32_t rec0 = rec_of(0, 0), rec1 = pair ? rec_of(1, 0) : 0;
    int32_t rows = page_row(P, full_layer, rec0);           // of batch `cur`
    const int32_t rows_two = pair ? page_row(P, full_layer, rec1) : 0;   // a pair's second piece
    int32_t rec_next = !pair && n_slots > 32 ? rec_of(0, 1) : 0;
    int cur = 0;
    auto load_tile = [&](int x, int pos, const CUtensorMap *map) {
      const int i0 = (pair ? x >> 1 : x) * ppt;
      if (!pair && (i0 >> 5) > cur) {
        ++cur;
        rows = page_row(P, full_layer, rec_next);
        rec_next = 32 * (cur + 1) < n_slots ? rec_of(0, cur + 1) : 0;
      }
      const int32_t held = !pair || (x & 1) == 0 ? rows : rows_two;
      int32_t row[8];                        // first rows of the tile's pages
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < ppt) row[i] = __shfl_sync(0xffffffffu, held, (i0 + i) & 31);
      // The slot's fill before this one may be the other warp's.  Its phase is
      // told by parity alone, which is enough: this warp's previous tile lies at
      // most three places back and its wait saw a place released that only the
      // next place's release can precede, so the fill before that one is gone.
      const int s = pos % kLoads, f = pos / kLoads;
      if (f >= 1 && !wait_all(bar(bLoadEmpty + s), (f - 1) & 1)) return false;
      const uint32_t dst = sb + kOffLoad + s * kLoadBytes, full = bar(bLoadFull + s);
      if (elect_one()) {
        mbar_expect_tx(full, (uint32_t)kLoadBytes);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i < ppt)
#pragma unroll
            for (int h = 0; h < (kF8 ? 1 : kD / 64); ++h)
              tma_load_3d(dst + h * kBlock + (i << P.ps_shift) * 128, map, h * 64, kvh, row[i],
                          full);
        ctl->fills[s] = f + 1;
      }
      __syncwarp();
      return true;
    };
    for (int t = 0; t < n; ++t)
      if (!load_tile(t, base + (warp == 9 ? seq_k(t) : seq_v(t, n)), warp == 9 ? &tmK : &tmV))
        return false;
    return true;
  };

  // The same by 16-byte copies of every key's row.
  auto gather = [&](const Segment &sg, int base) {
    constexpr int kChunks = (kF8 ? kD : 2 * kD) / 16;      // of a head's row
    const bool pair = sg.mode == kPair, is_v = warp == 11;
    const int n = ring_tiles(sg.mode, sg.n_tiles);
    // Rows of the ring's tile x: lane i those of columns i, 32 + i, ...  Columns
    // behind the last one read it again (finite values, zero weight).
    auto slots_of = [&](int x, int64_t (&slot)[4]) {
      const Piece pc = pair && (x & 1) ? sg.piece[1] : sg.piece[0];
      const int hi = pc.prefix + pc.n0 + pc.n_tok - 1;
      const int first = max(pc.prefix - P.lookback, 0) / P.ps;   // the plan's first page
      const int32_t *rt_row = full_layer ? P.rt + P.req_idx[pc.b] * P.rt_stride : nullptr;
      const int4 h = full_layer ? make_int4(0, 0, 0, 0)
                                : *reinterpret_cast<const int4 *>(P.plan.hdr + pc.b * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = min(pc.col0 + (pair ? x >> 1 : x) * kKeys + 32 * i + lane, hi);
        if (full_layer) {
          slot[i] = rt_row[col];
        } else {
          const int pg = col / P.ps, k = pg - first;
          const bool in = k >= 0 && k < P.plan.max_pages && k < h.w && col >= h.x && h.z == first;
          const int32_t page = in ? P.plan.pages[(int64_t)pc.b * P.plan.max_pages + k] : -1;
          if (page == 0) set_error(P.err, SWA_DEVERR_WINDOW_EVICTED);
          slot[i] = page < 0 ? -1 : (int64_t)page * P.ps + (col - pg * P.ps);
        }
      }
    };
    const char *pool = (is_v ? P.addr.v : P.addr.k) + kvh * (kChunks * 16);
    int64_t next[4];
    slots_of(0, next);
    for (int t = 0; t < n; ++t) {
      int64_t from[4];                       // byte offsets of this lane's rows
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int64_t slot = next[i];
        if (slot < 0 || slot >= P.pool_rows) {
          set_error(P.err, SWA_DEVERR_RANGE);
          slot = 0;
        }
        from[i] = kv_row(P.addr, slot) * P.addr.row_bytes;
      }
      __syncwarp();
      if (t + 1 < n) slots_of(t + 1, next);  // in flight while this tile is copied
      const int pos = base + (is_v ? seq_v(t, n) : seq_k(t)), s = pos % kLoads, f = pos / kLoads;
      if (f >= 1 && !wait_all(bar(bLoadEmpty + s), (f - 1) & 1)) return false;
      const uint32_t dst = sb + kOffLoad + s * kLoadBytes;
      const int c = lane % kChunks;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll 4
        for (int q = 0; q < kChunks; ++q) {
          const int e = q * (32 / kChunks) + lane / kChunks;   // row of the 32
          const char *src = pool + __shfl_sync(0xffffffffu, from[i], e) + c * 16;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(
                           dst + tile_off(32 * i + e, c)),
                       "l"(src)
                       : "memory");
        }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(
                       bar(bLoadFull + s))
                   : "memory");
    }
    return true;
  };
  auto load_tiles = [&](const Segment &sg, int base) {
    if constexpr (kGather) return gather(sg, base);
    else return stream(sg, base);
  };

  if (warp >= 8) {
  // E4M3 KV: 512 threads x 128 registers = 256 x 152 (softmax) + 256 x 104; whole
  // warpgroups on each side.
  if constexpr (kF8) asm volatile("setmaxnreg.dec.sync.aligned.u32 104;\n");
  after_previous();
  if (warp == 9) {
    // ===================== producer: segments, K tiles =====================
    int n_pub = 0, base = 0;                 // segments published; ring position

    bool ok = true;
    MergeDesc mine{0, 0, 0};
    auto publish = [&](const Segment &sg) {
      const int slot = n_pub & 1;
      if (n_pub >= 2 && !wait_all(bar(B_IEMPTY + slot), ((n_pub >> 1) - 1) & 1)) return false;
      if (lane == 0) {
        s_seg[slot] = sg;
        mbar_arrive(bar(B_IFULL + slot));
      }
      __syncwarp();
      ++n_pub;
      return true;
    };
    Piece held{};                            // the first item of a pair, and its tiles
    int held_n = 0;
    auto emit = [&](int mode, int n, int part, const Piece &p0, const Piece &p1) {
      Segment sg;
      sg.mode = mode;
      sg.n_tiles = n;
      sg.part = part;
      sg.piece[0] = p0;
      sg.piece[1] = p1;
      const bool good = publish(sg) && load_tiles(sg, base);
      base += 2 * ring_tiles(mode, n);
      return good;
    };

    auto bcast = [&](int x, int l) { return __shfl_sync(0xffffffffu, x, l); };
    if (P.whole) {
      // The head's blocks, every request's the same number of them (some empty),
      // so nothing is summed up: neighbours to a CTA where a request has one, in
      // turn where it may have more (a large tree among small ones is spread).
      // This CTA's, 32 at a time.
      const unsigned per = P.blocks, total = P.bs * per, share = (total + P.groups - 1) / P.groups;
      const unsigned step = per == 1 ? 1 : P.groups, x_lo = per == 1 ? group_id * share : group_id;
      const unsigned x_hi = per == 1 ? min(total, x_lo + share) : total;
      for (unsigned x0 = x_lo; ok && x0 < x_hi; x0 += 32 * step) {
        const unsigned x = x0 + lane * step;
        const int b = per == 1 ? x : x / per, blk = x - b * per;
        const Request r = request(P, x < x_hi ? b : P.bs);
        Piece mp{b, blk * 2 * T, min(2 * T, r.n - blk * 2 * T), r.q0 + blk * 2 * T, r.col0, r.prefix};
        const int tiles = mp.n_tok > 0 ? block_tiles(P, r, blk) : 0;
        unsigned hit = __ballot_sync(0xffffffffu, mp.n_tok > 0);
        while (ok && hit) {
          const int l = __ffs(hit) - 1;
          hit &= hit - 1;
          const Piece pc{bcast(mp.b, l),  bcast(mp.n0, l),   bcast(mp.n_tok, l),
                         bcast(mp.q0, l), bcast(mp.col0, l), bcast(mp.prefix, l)};
          const int n = bcast(tiles, l);
          // Items of one Q tile and few pages go in pairs.
          if (pc.n_tok <= T && n * ppt <= 32) {
            if (held_n) {
              ok = emit(kPair, max(held_n, n), -1, held, pc);
              held_n = 0;
            } else {
              held = pc;
              held_n = n;
            }
          } else {
            ok = emit(pc.n_tok <= T ? kAlternate : kShared, n, -1, pc, pc);
          }
        }
      }
    } else {
      // The head's line of tiles, and this CTA's stretch of it.
      auto tiles_of = [&](const Request &r) {
        int64_t n = 0;
        for (int i = 0; i < n_blocks(P, r); ++i) n += block_tiles(P, r, i);
        return n;
      };
      int64_t total = 0;
      for (int b0 = 0; b0 < P.bs; b0 += 64) {
        const Request a = request(P, b0 + lane), b = request(P, b0 + 32 + lane);
        total += tiles_of(a) + tiles_of(b);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      const int64_t share = (total + P.groups - 1) / P.groups;
      const int64_t w0 = group_id * share, w1 = min(total, w0 + share);
      int64_t at = 0;                        // line position of the batch's first request
      for (int b0 = 0; ok && b0 < P.bs && at < w1; b0 += 32) {
        const Request r = request(P, b0 + lane);
        const int64_t mine_tiles = tiles_of(r);
        int64_t incl = mine_tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const int64_t s0 = at + incl - mine_tiles;
        unsigned hit = __ballot_sync(0xffffffffu, mine_tiles > 0 && s0 < w1 && s0 + mine_tiles > w0);
        while (ok && hit) {
          const int l = __ffs(hit) - 1;
          hit &= hit - 1;
          const Request q{bcast(r.q0, l), bcast(r.prefix, l), bcast(r.col0, l), bcast(r.n, l)};
          int64_t s = __shfl_sync(0xffffffffu, s0, l);
          for (int blk = 0; ok && blk < n_blocks(P, q) && s < w1; ++blk) {
            const int64_t e = s + block_tiles(P, q, blk);
            if (e > w0) {
              const int64_t from = max(s, w0), to = min(e, w1);
              const int n0 = blk * 2 * T;
              const Piece pc{b0 + l,     n0, min(2 * T, q.n - n0), q.q0 + n0,
                             q.col0 + (int)(from - s) * kKeys, q.prefix};
              int part = -1;
              if (from == s && to < e) {
                part = 1;
                mine.parts = (int)((e - 1) / share) - group_id + 1;
                mine.n_tok = pc.n_tok;
                mine.q0 = pc.q0;
              } else if (from > s) {
                part = 0;
              }
              ok = emit(pc.n_tok <= T ? kAlternate : kShared, (int)(to - from), part, pc, pc);
            }
            s = e;
          }
        }
        at += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    if (ok && held_n) ok = emit(kAlternate, held_n, -1, held, held);
    if (!P.whole && lane == 0) P.desc[blockIdx.x] = mine;
    if (ok) {
      Segment end{};
      end.mode = -1;
      publish(end);
    }
  } else if (warp == 10 || warp == 11) {
    // ===================== Q tiles (warp 10), V tiles (warp 11) =====================
    int base = 0;
    for (int nd = 0;; ++nd) {
      const int slot = nd & 1;
      if (!wait_all(bar(B_IFULL + slot), (nd >> 1) & 1)) break;
      const Segment sg = s_seg[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + slot));
      if (sg.mode < 0 || !(warp == 10 ? load_q(sg, nd) : load_tiles(sg, base))) break;
      base += 2 * ring_tiles(sg.mode, sg.n_tiles);
    }
  } else if (warp >= 12) {
    if constexpr (kF8) {
      // ============ converters (E4M3 KV): Q, K and V to f16 ============
      const int ct = tid - kTreeThreads;     // 0 .. 127
      int pos = 0;                           // ring position, both rings
      bool ok = true;
      for (int nd = 0; ok; ++nd) {
        const int slot = nd & 1;
        if (!wait_all(bar(B_IFULL + slot), (nd >> 1) & 1)) break;
        const Segment sg = s_seg[slot];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_IEMPTY + slot));
        if (sg.mode < 0) break;
        if (!wait_all(bar(B_FULLQ), nd & 1)) break;
        const int q_chunks = (sg.mode == kAlternate ? 1 : 2) * kTileBytes / 16;
#pragma unroll 4
        for (int i = ct; i < q_chunks; i += kConvThreads) {
          uint4 *q16 = reinterpret_cast<uint4 *>(smem + i * 16);
          uint4 v = *q16;
          v.x = bf16x2_to_f16x2(v.x);
          v.y = bf16x2_to_f16x2(v.y);
          v.z = bf16x2_to_f16x2(v.z);
          v.w = bf16x2_to_f16x2(v.w);
          *q16 = v;
        }
        fence_async_smem();                  // read by the tensor core (the async proxy)
        mbar_arrive(bar(B_QCONV));
        for (int j = 0; j < 2 * ring_tiles(sg.mode, sg.n_tiles); ++j, ++pos) {
          const int rs = pos % kLoads, s = pos % kStages;
          if (!(ok = wait_all(bar(B_RAWFULL + rs), (pos / kLoads) & 1))) break;
          if (pos >= kStages && !(ok = wait_all(bar(B_EMPTY + s), (pos / kStages - 1) & 1))) break;
          const char *src = smem + Gm::kOffRaw + rs * Gm::kRawBytes;
          char *dst = smem + Gm::kOffRing + s * kTileBytes;
          // Eight lanes take chunks 0-3 of an even row and 4-7 of the next (then
          // the other halves): neither the reads of 16 E4M3 values nor the two
          // 16-byte writes that they become meet in a bank.
          const int odd = (ct >> 2) & 1;
          uint4 w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = (((i & 1) ^ odd) << 2) + (ct & 3);
            const int r = 2 * ((i >> 1) * 16 + (ct >> 3)) + odd;
            w[i] = *reinterpret_cast<const uint4 *>(src + r * 128 + ((c ^ (r & 7)) << 4));
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int c = (((i & 1) ^ odd) << 2) + (ct & 3);
            const int r = 2 * ((i >> 1) * 16 + (ct >> 3)) + odd;
            uint4 a, b;
            e4m3x4_to_f16x4(w[i].x, a.x, a.y);
            e4m3x4_to_f16x4(w[i].y, a.z, a.w);
            e4m3x4_to_f16x4(w[i].z, b.x, b.y);
            e4m3x4_to_f16x4(w[i].w, b.z, b.w);
            *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * c)) = a;
            *reinterpret_cast<uint4 *>(dst + tile_off(r, 2 * c + 1)) = b;
          }
          fence_async_smem();
          mbar_arrive(bar(B_FULL + s));
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(B_RAWEMPTY + rs));
        }
      }
    }
  } else if (warp == 8) {
    // ===================== MMA issue =====================
    // Step u of a segment belongs to softmax group u & 1 and the ring's tile u / 2
    // (shared) or u; the order is S(0), S(1), then per step O(u), S(u + 2).  An
    // elected lane runs a segment's steps: with the segment's numbers made
    // uniform by a warp reduction, descriptors are computed in uniform registers
    // (in a branch on the lane number a product cost 67 cycles to issue, whatever
    // its size).
    auto uni = [](int x) { return (int)__reduce_max_sync(0xffffffffu, x); };
    const uint64_t dq = smem_desc(sb, 16, 1024);
    const uint64_t dk = smem_desc(sb + Gm::kOffRing, 16, 1024);
    const uint64_t dv = smem_desc(sb + Gm::kOffRing, kBlock, 1024);
    int steps0 = 1, steps1 = 1;              // PREADY phases of each group so far (the first: warm-up)
    int base = 0;                            // ring position of the segment's first tile
    for (int nd = 0;; ++nd) {
      const int slot = nd & 1;
      if (!wait_all(bar(B_IFULL + slot), (nd >> 1) & 1)) break;
      const int mode = uni(s_seg[slot].mode), tiles = uni(s_seg[slot].n_tiles);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + slot));
      if (mode < 0) break;
      const int U = mode == kAlternate ? tiles : 2 * tiles, n = ring_tiles(mode, tiles);
      const bool shared = mode == kShared;   // a K/V tile serves two steps
      if (!wait_all(bar(kF8 ? B_QCONV : B_FULLQ), nd & 1)) break;
      if (nd == 0 && !(wait_all(bar(B_PREADY), 0) && wait_all(bar(B_PREADY + 1), 0))) break;
      int ok = 1;
      if (elect_one()) {
        // Ring slots (and phases) of the next K and V tile.
        auto advance = [](int &slot, uint32_t &phase, int by) {
          slot += by;
          if (slot >= kStages) {
            slot -= kStages;
            phase ^= 1u;
          }
        };
        int ks = base % kStages, vs = ks, kt = 0, vt = 0;   // slots; tiles of the segment
        uint32_t kp = (base / kStages) & 1, vp = kp;
        advance(vs, vp, min(2, 2 * n - 1));
        for (int u = -2; u < U; ++u) {       // u = -2, -1: S(0) and S(1) only
          const int g = u & 1;
          const bool fresh = !shared || !g, last = !shared || g;   // first, last use of a tile
          if (u >= 0) {
            if (fresh && !(ok = mbar_wait_ready(bar(B_FULL + vs), vp, &s_abort))) break;
            if (kGather && !kF8) fence_async_smem();   // copied through the generic proxy
            if (!(ok = mbar_wait(bar(B_PREADY + g), ((g ? steps1 : steps0) + (u >> 1)) & 1, &s_abort)))
              break;
            tc_fence_after();
            const uint64_t vd = dv + (uint64_t)(vs * kTileBytes >> 4);
#pragma unroll
            for (int e = 0; e < kKeys / 16; ++e)
              mma_ts(tmem + 256 + g * kD, tmem + g * 128 + e * 8,
                     vd + (uint64_t)(e * 16 * 128 >> 4), kIdO, (u >= 2 || e > 0) ? 1u : 0u);
            if (last) {
              tc_commit(bar(B_EMPTY + vs));
              advance(vs, vp, ++vt == n - 1 ? 1 : 2);
            }
            if (u + 2 >= U) tc_commit(bar(B_ODONE + g));
          }
          if (u + 2 < U) {                   // S(u + 2), of the same group
            if (fresh && !(ok = mbar_wait_ready(bar(B_FULL + ks), kp, &s_abort))) break;
            if (kGather && !kF8) fence_async_smem();
            tc_fence_after();
            const uint64_t kd = dk + (uint64_t)(ks * kTileBytes >> 4);
            const uint64_t qd = dq + (uint64_t)((mode != kAlternate && g ? kTileBytes : 0) >> 4);
#pragma unroll
            for (int e = 0; e < kD / 16; ++e) {
              const uint64_t off = ((e >> 2) * kBlock + (e & 3) * 32) >> 4;
              mma_ss(tmem + g * 128, qd + off, kd + off, kIdS, e > 0);
            }
            tc_commit(bar(B_SDONE + g));
            if (last) {
              tc_commit(bar(B_EMPTY + ks));
              advance(ks, kp, kt++ == 0 ? 1 : 2);
            }
            if (u + 3 == U) tc_commit(bar(B_QFREE));
          }
        }
      }
      if (!__all_sync(0xffffffffu, ok)) break;
      steps0 += (U + 1) >> 1;
      steps1 += U >> 1;
      base += 2 * n;
    }
  }
  } else {
    if constexpr (kF8) asm volatile("setmaxnreg.inc.sync.aligned.u32 152;\n");
    // ===================== softmax group =====================
    const int grp = warp >> 2;
    const int r = tid & 127;                 // row of the Q tile = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + grp * 128 + lane_off;
    const uint32_t tO = tmem + 256 + grp * kD + lane_off;
    const int head = kvh * G + r % G;
    const float sc = P.scale_log2;
    const uint64_t sc2 = f2pack(sc, sc);
    int steps = 0, joins = 0;
    int both = 0;                            // segments in which both groups have a step
    // A segment as this row sees it, with what it loads of its node: taken from
    // the ring before the previous segment's epilogue, which covers the loads.
    struct Mine {
      int mode, n_tiles, part, tr, depth;
      Piece pc;
      bool valid;
      uint64_t above;          // ancestors, in trees of at most 64 nodes
    };
    const bool few = P.tree.words <= 2;
    auto take = [&](int nd, Mine &m) {
      const int slot = nd & 1;
      if (!wait_all(bar(B_IFULL + slot), (nd >> 1) & 1)) return false;
      m.mode = s_seg[slot].mode;
      m.n_tiles = s_seg[slot].n_tiles;
      m.part = s_seg[slot].part;
      m.pc = s_seg[slot].piece[m.mode == kPair ? grp : 0];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(B_IEMPTY + slot));
      m.tr = (m.mode == kShared ? grp * T : 0) + r / G;       // node of the item
      m.valid = m.mode >= 0 && r < TG && m.tr < m.pc.n_tok;
      m.depth = 0;
      m.above = 0ull;
      if (m.valid) {
        const uint32_t *row = P.tree.mask + (int64_t)(m.pc.q0 + m.tr) * P.tree.words;
        m.depth = P.tree.depth[m.pc.q0 + m.tr];
        if (few) m.above = row[0] | (P.tree.words == 2 ? (uint64_t)row[1] << 32 : 0ull);
      }
      __syncwarp();
      return true;
    };
    // Turn -1 runs the tile loop on whatever the tensor memory holds, for the
    // instruction cache: cold, a CTA's first tile took 6400 cycles instead of
    // 2700, and these warps have nothing to do until the first S is there.  Its
    // PREADY lets the first S in.
    Mine next{kShared, 1, -1, 0, 0, Piece{0, 0, 0, 0, 0, 32}, false, 0ull};
    float sg2 = -INFINITY;
    for (int nd = -1;; ++nd) {
      const bool warming = nd < 0;
      const Mine cur = next;
      if (cur.mode < 0) break;
      const int mode = cur.mode, n_tiles = cur.n_tiles, tr = cur.tr, part_slot = cur.part;
      const Piece pc = cur.pc;
      const bool alone = mode != kAlternate;           // this group's rows are its own
      const bool row_valid = cur.valid;
      const uint64_t above = cur.above;
      const bool any_row = warming || __any_sync(0xffffffffu, row_valid);
      const uint32_t *row = P.tree.mask + (int64_t)(pc.q0 + (row_valid ? tr : 0)) * P.tree.words;
      // Relative to the piece's first column: the row's first column, and the
      // first behind the cached ones.
      int lo_row = 0;
      const int behind = pc.prefix - pc.col0;
      if (row_valid)
        lo_row = (int)tree_first_col(first_position(P.kind, P.window, pc.prefix + cur.depth),
                                     pc.prefix, pc.n0 + tr, cur.depth, row) -
                 pc.col0;
      float m_run = row_valid || warming ? -INFINITY : 0.f, l_run = 0.f;
      bool alive = true, first = true;
      // Uniform over the warp: no row's columns begin after `lo_most`, and every
      // row has a reference maximum (`settled`); interior chunks then need no vote
      // before their exponentials.
      const int lo_most = __reduce_max_sync(0xffffffffu, row_valid ? lo_row : -0x7fffffff);
      bool settled = false;
      for (int t = alone ? 0 : grp; t < n_tiles; t += alone ? 1 : 2) {
        if (!warming) {
          if (!wait_all(bar(B_SDONE + grp), steps & 1)) {
            alive = false;
            break;
          }
          ++steps;
        }
        tc_fence_after();
        uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll 1
        for (int cb = 0; any_row && cb < 2; ++cb) {
          const int c0 = t * kKeys + cb * 64;        // the chunk's first column
          // Columns of the chunk this row reads.
          uint64_t allow = row_valid ? ~0ull : 0ull;
          const bool any_edge = warming || c0 < lo_most || c0 + 64 > behind;
          if (any_edge) {
            if (row_valid || warming) {
              allow = bit_range(lo_row - c0, behind - c0);
              // (The warm-up must not read the tree: it may still be written.)
              if (c0 + 64 > behind)
                allow |= (few || warming ? shift_bits(above, c0 - behind)
                                         : row_bits(row, P.tree.words, c0 - behind)) &
                         bit_range(max(lo_row, behind) - c0, 64);
            }
            if (!__any_sync(0xffffffffu, allow != 0ull)) {
              uint32_t zero[32];
#pragma unroll
              for (int e = 0; e < 32; ++e) zero[e] = 0u;
              TC_ST32(tS + cb * 32, zero);
              continue;
            }
          }
          uint32_t rr[64];
          TC_LD32(tS + cb * 64, rr);
          TC_LD32(tS + cb * 64 + 32, (rr + 32));
          tc_wait_ld();
          if (any_edge) {
            const uint32_t a0 = (uint32_t)allow, a1 = (uint32_t)(allow >> 32);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(a0 >> e & 1u)) rr[e] = 0xff800000u;
              if (!(a1 >> e & 1u)) rr[32 + e] = 0xff800000u;
            }
          }
          // The exponentials are taken against the row's reference maximum; the
          // chunk's own maximum is computed only for a row's first chunk and
          // when the weights' sum shows that a score outgrew the reference.
          // Raising the reference rescales what was summed against the old one.
          bool redo = false;
          if (!settled) {
            redo = __any_sync(0xffffffffu, m_run == -INFINITY);
            settled = !redo;
          }
          uint32_t pk[32];
          uint64_t c2[2];
#pragma unroll 1
          for (int pass = 0;; ++pass) {
            if (redo) {
              float m2[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int e = 0; e < 64; e += 2)
                m2[(e >> 1) & 3] =
                    max3(m2[(e >> 1) & 3], __uint_as_float(rr[e]), __uint_as_float(rr[e + 1]));
              float cm = max3(m2[0], m2[1], fmaxf(m2[2], m2[3]));
              cm = cm == -INFINITY ? -INFINITY : cm * sc;
              float corr = 1.f;
              if (row_valid &&
                  (cm > m_run + kRescaleGap || (m_run == -INFINITY && cm != -INFINITY))) {
                corr = m_run == -INFINITY ? 1.f : exp2f(m_run - cm);
                m_run = cm;
              }
              if (__any_sync(0xffffffffu, corr != 1.f)) {
                if (!first) {
#pragma unroll 1
                  for (int ob = 0; ob < kD / 32; ++ob) {
                    uint32_t ro[32];
                    TC_LD32(tO + ob * 32, ro);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                      ro[e] = __float_as_uint(__uint_as_float(ro[e]) * corr);
                    TC_ST32(tO + ob * 32, ro);
                  }
                }
                if (cb == 1) {
                  uint32_t pp[32];
                  tc_wait_st();
                  TC_LD32(tS, pp);
                  tc_wait_ld();
#pragma unroll
                  for (int e = 0; e < 32; ++e) {
                    const float2 f = unpack_p<kF8>(pp[e]);
                    pp[e] = pack_p<kF8>(f.x * corr, f.y * corr);
                  }
                  TC_ST32(tS, pp);
                }
                float a0, a1, b0, b1;
                f2unpack(acc2[0], a0, a1);
                f2unpack(acc2[1], b0, b1);
                acc2[0] = f2pack(a0 * corr, a1 * corr);
                acc2[1] = f2pack(b0 * corr, b1 * corr);
                l_run *= corr;
              }
            }
            const float mu = m_run == -INFINITY ? 0.f : m_run;
            const uint64_t nmu2 = f2pack(-mu, -mu);
            c2[0] = c2[1] = 0ull;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              float t0, t1;
              f2unpack(fma2(f2pack(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1])), sc2,
                            nmu2),
                       t0, t1);
              const float a0 = ex2(t0), a1 = ex2(t1);
              c2[e & 1] = add2(c2[e & 1], f2pack(a0, a1));
              pk[e] = pack_p<kF8>(a0, a1);
            }
            if (pass == 1) break;
            float s0, s1, s2, s3;
            f2unpack(c2[0], s0, s1);
            f2unpack(c2[1], s2, s3);
            redo = __any_sync(0xffffffffu, row_valid && (s0 + s1) + (s2 + s3) > kSumCap);
            if (!redo) break;
          }
          acc2[0] = add2(acc2[0], c2[0]);
          acc2[1] = add2(acc2[1], c2[1]);
          TC_ST32(tS + cb * 32, pk);
        }
        {
          float s0, s1, s2, s3;
          f2unpack(acc2[0], s0, s1);
          f2unpack(acc2[1], s2, s3);
          l_run += (s0 + s1) + (s2 + s3);
        }
        first = false;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_PREADY + grp));
      }
      if (warming) {
        after_previous();
        if (P.sinks && r < TG) sg2 = P.sinks[head] * 1.4426950408889634f;
      }
      if (!alive || !take(nd + 1, next)) break;
      if (warming) continue;
      // ---- epilogue ----
      // A segment of one step is group 0's: group 1's O is not written, and its
      // barrier has no phase (one that completed without a step of group 1 could
      // complete before group 1 has seen the phase before it, whose parity would
      // then be gone).
      const bool one_step = !alone && n_tiles == 1;
      const uint32_t done0 = nd & 1, done1 = both & 1;   // phases of the two O
      if (!(grp && one_step) && !wait_all(bar(B_ODONE + grp), grp ? done1 : done0)) break;
      float w0 = 1.f, w1 = 0.f;              // weights of this group's and the other's O
      if (!alone) {
        // Join the groups' halves of the keys: row statistics through shared
        // memory, accumulators read from TMEM; group i writes half i of D.
        s_stat[grp * kTileRows + r] = make_float2(m_run, l_run);
        mbar_arrive(bar(B_STAT));
        if (!wait_all(bar(B_STAT), joins & 1)) break;
        if ((grp || !one_step) && !wait_all(bar(B_ODONE + (grp ^ 1)), grp ? done0 : done1)) break;
        const float2 o = s_stat[(grp ^ 1) * kTileRows + r];
        const float m = fmaxf(m_run, o.x);
        w0 = m_run == -INFINITY ? 0.f : exp2f(m_run - m);
        w1 = o.x == -INFINITY ? 0.f : exp2f(o.x - m);
        m_run = m;
        l_run = l_run * w0 + o.y * w1;
      }
      tc_fence_after();
      float f = 1.f;
      if (part_slot < 0) {
        const float mr = m_run == -INFINITY ? 0.f : m_run;
        const float mfin = fmaxf(mr, sg2);
        const float rsc = exp2f(mr - mfin);
        const float denom = l_run * rsc + (P.sinks ? exp2f(sg2 - mfin) : 0.f);
        f = rsc / denom * P.v_scale;         // (no row is without a key: it attends itself)
      }
      w0 *= f;
      w1 *= f;
      const int row_i = (mode == kShared ? grp * TG : 0) + r;      // row of the item
      float *part = part_slot < 0 ? nullptr
                                : P.partials + ((int64_t)blockIdx.x * 2 + part_slot) * P.part_stride;
      if (part && row_valid && (alone || grp == 0))
        reinterpret_cast<float2 *>(part + P.rows_max * kD)[row_i] = make_float2(m_run, l_run);
      __nv_bfloat16 *orow = P.out + ((int64_t)(pc.q0 + tr) * (P.hkv * G) + head) * kD;
      const int d_lo = alone ? 0 : grp * (kD / 2), d_hi = alone ? kD : d_lo + kD / 2;
      const uint32_t tO2 = tmem + 256 + (grp ^ 1) * kD + lane_off;
      __syncwarp();
#pragma unroll 1
      for (int d = d_lo; any_row && d < d_hi; d += 32) {
        uint32_t a[32];
        TC_LD32(tO + d, a);
        if (alone) {
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * w0);
        } else {
          uint32_t b[32];
          TC_LD32(tO2 + d, b);
          tc_wait_ld();
          // An accumulator without weight may hold anything.
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float x = w0 != 0.f ? __uint_as_float(a[e]) * w0 : 0.f;
            a[e] = __float_as_uint(w1 != 0.f ? fmaf(__uint_as_float(b[e]), w1, x) : x);
          }
        }
        if (part && row_valid) {
          // Four dims of all rows together: a warp's rows are neighbours.
          float4 *dst = reinterpret_cast<float4 *>(part) + (d / 4) * P.rows_max + row_i;
#pragma unroll
          for (int e = 0; e < 8; ++e)
            dst[e * P.rows_max] = make_float4(__uint_as_float(a[4 * e]), __uint_as_float(a[4 * e + 1]),
                                 __uint_as_float(a[4 * e + 2]), __uint_as_float(a[4 * e + 3]));
        } else if (row_valid) {
          // Every lane has a row of its own, so a store costs the load-store unit
          // a cycle per lane: 32 bytes at a time where the output allows it.
          uint32_t w[16];
#pragma unroll
          for (int k = 0; k < 16; ++k)
            w[k] = pack_p<false>(__uint_as_float(a[2 * k]), __uint_as_float(a[2 * k + 1]));
          if (P.wide_out) {
#pragma unroll
            for (int k = 0; k < 16; k += 8)
              asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(
                               orow + d + 2 * k),
                           "r"(w[k]), "r"(w[k + 1]), "r"(w[k + 2]), "r"(w[k + 3]), "r"(w[k + 4]),
                           "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7])
                           : "memory");
          } else {
#pragma unroll
            for (int k = 0; k < 16; k += 4)
              *reinterpret_cast<uint4 *>(orow + d + 2 * k) =
                  make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
          }
        }
        __syncwarp();   // the TMEM loads are warp-collective
      }
      __syncwarp();
      if (!alone) {
        // Both groups have read both accumulators (and the statistics) before
        // the next segment's products overwrite them.
        tc_fence_before();
        mbar_arrive(bar(B_EPI));
        if (!wait_all(bar(B_EPI), joins & 1)) break;
        tc_fence_after();
        ++joins;
      }
      both += !one_step;
    }
  }
  if (kGather) asm volatile("cp.async.wait_all;\n" ::: "memory");
  // Every role has left its loop: s_abort is final.
  __syncthreads();
  if (s_abort) {
    // Loads and products already issued complete on their own; wait for them
    // before the shared memory and TMEM they write are released.
    if (tid == 0) set_error(P.err, SWA_DEVERR_TIMEOUT);
    if (warp == 9 && lane == 0)
      for (int s = 0; s < kLoads; ++s)
        if (ctl->fills[s]) mbar_drain(bar(bLoadFull + s), (ctl->fills[s] - 1) & 1);
    if (warp == 10 && lane == 0 && q_issued) mbar_drain(bar(B_FULLQ), (q_issued - 1) & 1);
    if (warp == 8 && elect_one()) {
      tc_commit(bar(B_DRAIN));
      mbar_drain(bar(B_DRAIN), 0);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
}

// Merges the partials of the items that cross CTAs: CTA (chunk, c) the rows
// [32 chunk, 32 chunk + 32) of the item that CTA c of the main launch began and
// left, in group order.  A lane has a row and a warp D / 8 of its dims, so that
// partials are read as they were written, whole lines at a time.
template <int kD>
__global__ void __launch_bounds__(kMergeThreads) k_tree_merge(const __grid_constant__ TreeParams P) {
  constexpr int kQuads = kD / 4 / (kMergeThreads / 32);   // float4s of a lane
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const MergeDesc d = P.desc[blockIdx.y];
  const int q0 = (threadIdx.x >> 5) * kQuads, r = blockIdx.x * kMergeRows + (threadIdx.x & 31);
  const int kvh = blockIdx.y % P.hkv, G = P.G;
  if (d.parts < 2 || r >= d.n_tok * G) return;
  const int head = kvh * G + r % G;
  auto part = [&](int i) {
    return P.partials +
           (((int64_t)blockIdx.y + (int64_t)i * P.hkv) * 2 + (i == 0 ? 1 : 0)) * P.part_stride;
  };
  auto stat = [&](int i) {
    return reinterpret_cast<const float2 *>(part(i) + P.rows_max * kD)[r];
  };
  const float sg2 = P.sinks ? P.sinks[head] * 1.4426950408889634f : -INFINITY;
  float M = sg2;
#pragma unroll 4
  for (int i = 0; i < d.parts; ++i) M = fmaxf(M, stat(i).x);
  float L = P.sinks ? exp2f(sg2 - M) : 0.f;
  float4 acc[kQuads];
#pragma unroll
  for (int e = 0; e < kQuads; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < d.parts; ++i) {
    const float2 s = stat(i);
    const float w = s.x == -INFINITY ? 0.f : exp2f(s.x - M);
    L += w * s.y;
    const float4 *src = reinterpret_cast<const float4 *>(part(i)) + q0 * P.rows_max + r;
#pragma unroll
    for (int e = 0; e < kQuads; ++e) {
      const float4 v = src[e * P.rows_max];
      acc[e].x = fmaf(v.x, w, acc[e].x);
      acc[e].y = fmaf(v.y, w, acc[e].y);
      acc[e].z = fmaf(v.z, w, acc[e].z);
      acc[e].w = fmaf(v.w, w, acc[e].w);
    }
  }
  const float f = P.v_scale / L;
  __nv_bfloat16 *dst = P.out + ((int64_t)(d.q0 + r / G) * (P.hkv * G) + head) * kD + q0 * 4;
#pragma unroll
  for (int e = 0; e < kQuads; e += 2)
    *reinterpret_cast<uint4 *>(dst + 4 * e) =
        make_uint4(pack_p<false>(acc[e].x * f, acc[e].y * f), pack_p<false>(acc[e].z * f, acc[e].w * f),
                   pack_p<false>(acc[e + 1].x * f, acc[e + 1].y * f),
                   pack_p<false>(acc[e + 1].z * f, acc[e + 1].w * f));
}

int tile_nodes(const Ctx &c, int layer, int max_new) {
  return std::min(kTileRows / (c.cfg.num_q_heads / c.layers[layer].hkv), max_new);
}

struct TreeWs {
  int groups, rows;          // CTAs per KV head; rows of an item
  bool whole;                // items are not split
  int64_t part_stride;       // floats
  size_t desc_off, part_off, total;
};

// [reserved][tickets] as in the other attention families, which this one leaves
// untouched (so calls of either may share a workspace), then the descriptors and
// partials.
TreeWs tree_ws(const Ctx &c, int layer, int bs, int64_t nq, int max_new, int max_seq_len) {
  const LayerInfo &L = c.layers[layer];
  TreeWs w;
  const int G = c.cfg.num_q_heads / L.hkv, T = tile_nodes(c, layer, max_new);
  w.groups = std::max(1, (c.num_sms > 0 ? c.num_sms : 148) / L.hkv);
  w.rows = std::min(2 * T, max_new) * G;
  // Whole items or equal stretches of the keys?  Whole items save the batch scan,
  // the partials and the merge; stretches keep every CTA busy.  Device time of
  // plan and attention, 8 nodes, whole against stretches: 2 requests of 500 / 1000
  // / 2000 / 4000 tokens 13.2 / 16.3 / 22.5 / 34.8 against 18.4 / 21.7 / 27.7 / 28.2
  // us (MiMo full layer); 64 requests of up to 1000 / 2000 / 4000 / 8000 tokens 25.4
  // / 43.8 / 75.5 / 129.5 against 39.6 / 54.9 / 77.5 / 120.0 us.  Where the items of
  // a group come out uneven (40 requests on 19 groups: three for some, two for
  // most) whole items lose from 2000 tokens on: 40.7 against 38.5 us (D = 64), 61.2
  // against 54.3 us (E4M3).
  const int64_t keys = tree_max_keys(c, layer, max_new, max_seq_len);
  const int64_t items = (int64_t)bs * ((max_new + 2 * T - 1) / (2 * T));
  const int64_t most = (items + w.groups - 1) / w.groups;
  w.whole = keys <= 1024 || (keys <= 2048 && (most <= 1 || 4 * most * w.groups <= 5 * items));
  // whole 128-byte lines of four dims x 32 rows
  w.rows = (w.rows + 31) / 32 * 32;
  w.part_stride = (int64_t)w.rows * (c.cfg.head_dim + 2);
  w.desc_off = ws_partials_off(c, nq);
  const size_t ctas = (size_t)w.groups * L.hkv;
  w.part_off = w.desc_off + (ctas * sizeof(MergeDesc) + 255) / 256 * 256;
  w.total = w.whole ? w.desc_off : w.part_off + ctas * 2 * w.part_stride * sizeof(float);
  return w;
}

template <int D, bool F8, bool G>
cudaError_t launch_tree(const LayerInfo &L, const CUtensorMap &tmq, const TreeParams &P, int rows,
                        int device, cudaStream_t s) {
  using Gm = TreeGeo<D, F8>;
  const size_t smem = Gm::kOffCtl + sizeof(Control);
  static_assert(B_COUNT == 40 && Gm::kOffCtl + sizeof(Control) <= 227 * 1024,
                "shared memory of a CTA");
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(k_tree_tc<D, F8, G>, smem, device, done);
  if (e != cudaSuccess) return e;
  const int ctas = P.groups * P.hkv;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(Gm::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, k_tree_tc<D, F8, G>, L.tmk, L.tmv, tmq, P);
  if (e != cudaSuccess || P.whole) return e;
  cfg.gridDim = dim3((rows + kMergeRows - 1) / kMergeRows, ctas);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  return cudaLaunchKernelEx(&cfg, k_tree_merge<D>, P);
}

}  // namespace

// Pages that are TMA boxes of the layer's tensor maps.
static bool boxed_pages(const Ctx &c, int layer) {
  return c.layers[layer].tma && c.cfg.page_size <= 64;
}

bool tc_tree_supported(const Ctx &c, int layer) {
  const KvAddr &a = c.layers[layer].addr;
  const int d = c.cfg.head_dim;
  return ((reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v)) & 15) == 0 &&
         ((c.cfg.kv_dtype == SWA_DTYPE_BF16 && (d == 64 || d == 128)) ||
          (c.cfg.kv_dtype == SWA_DTYPE_E4M3 && d == 128));
}

size_t tc_tree_ws_bytes(const Ctx &c, int layer, int bs, int64_t nq, int max_new,
                        int max_seq_len) {
  return (tree_ws(c, layer, bs, nq, max_new, max_seq_len).total + 255) / 256 * 256;
}

cudaError_t launch_attn_tree_tc(Ctx &c, const AttnArgs &a, const TreeView &tree, cudaStream_t s) {
  if (a.nq == 0) return cudaSuccess;
  const LayerInfo &L = c.layers[a.layer];
  const TreeWs w = tree_ws(c, a.layer, a.bs, a.nq, a.max_new, a.max_seq_len);
  TreeParams P{};
  P.kind = L.kind;
  P.window = L.window;
  P.hkv = L.hkv;
  P.G = c.cfg.num_q_heads / L.hkv;
  P.T = tile_nodes(c, a.layer, a.max_new);
  P.ps = c.cfg.page_size;
  const bool boxed = boxed_pages(c, a.layer);
  P.ps_shift = boxed ? __builtin_ctz((unsigned)P.ps) : 0;
  P.addr = L.addr;
  P.page_stride = (int64_t)P.ps * (L.addr.blocks ? L.addr.blocks : 1);
  P.pool_rows = (L.in_full ? c.cfg.size_full : c.cfg.size_swa) + c.cfg.page_size;
  P.rt = a.rt;
  P.rt_stride = a.rt_stride;
  P.req_idx = a.req_idx;
  P.pre = a.pre;
  P.qo_indptr = a.qo_indptr;
  P.bs = a.bs;
  P.groups = w.groups;
  P.blocks = (a.max_new + 2 * P.T - 1) / (2 * P.T);
  P.max_new = a.max_new;
  P.whole = w.whole ? 1 : 0;
  P.n_tokens = a.nq;
  P.lookback = c.lookback;
  P.plan = a.plan;
  P.tree = tree;
  P.sinks = a.sinks;
  const bool f8 = c.cfg.kv_dtype == SWA_DTYPE_E4M3;
  P.scale_log2 = a.scale * 1.4426950408889634f * (f8 ? a.k_scale : 1.f);
  P.v_scale = f8 ? a.v_scale : 1.f;
  P.out = static_cast<__nv_bfloat16 *>(a.out);
  P.wide_out = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 ? 1 : 0;
  char *ws = static_cast<char *>(a.ws);
  P.desc = reinterpret_cast<MergeDesc *>(ws + w.desc_off);
  P.partials = reinterpret_cast<float *>(ws + w.part_off);
  P.part_stride = w.part_stride;
  P.rows_max = w.rows;
  P.err = c.err_word;
  CUtensorMap tmq;
  if (!make_q_tile_map(&tmq, a.q, a.nq, c.cfg.num_q_heads, c.cfg.head_dim, P.G, P.T))
    return cudaErrorInvalidValue;
  auto go = [&](auto gather) {
    constexpr bool g = decltype(gather)::value;
    if (f8) return launch_tree<128, true, g>(L, tmq, P, w.rows, c.device, s);
    return c.cfg.head_dim == 64 ? launch_tree<64, false, g>(L, tmq, P, w.rows, c.device, s)
                                : launch_tree<128, false, g>(L, tmq, P, w.rows, c.device, s);
  };
  return boxed ? go(std::false_type{}) : go(std::true_type{});
}

}  // namespace swa
