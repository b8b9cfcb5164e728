// Moves of K/V rows between slots of all layers: copies between given slots (a
// fork's open page), and the commit of a verified draft tree, whose accepted
// nodes' rows move to the columns that follow the prefix.
//
// A token's row is Hkv x D elements at its full slot on full layers and at
// full_to_swa[slot] on the others ("SWA in SGLang" design note, "two pools and
// the mapping"), K and V of every layer.  The moves are pure copies, bound by
// HBM: bytes read + bytes written.  A warp moves 512 bytes at a time (32 lanes x
// 16 bytes, coalesced both ways), looks the slots of its moves up with its lanes
// in one go, and keeps kAhead loads in flight before it stores any.  A copy gives
// a warp one 512-byte column of one layer's K or V rows for kAhead moves (48
// layers: 100 rows 5.8 us, 1504 rows, 536 MB, 80.8 us, 6.6 TB/s; with 32 moves a
// warp 7.4 and 82.6 us).  A commit has few rows per request, so there a warp takes
// whole rows of one layer's K or V, and the chain of lookups (length, row, two
// slots, two mappings) is paid once for all their columns (48 layers: 64 requests,
// 65 MB, 10.0 us, with a warp per column 15.1 us; 16 requests of 12 nodes, 7.4 us,
// with K and V both on one warp 11.6 us).
#include <cuda_runtime.h>

#include "spec_internal.h"

namespace swa {
namespace {

constexpr int kMoveLayers = 64;    // layers per launch (the table is a kernel parameter)
constexpr int kMoveWarps = 4;
constexpr int64_t kCopyMoves = 1 << 24;   // moves per launch
constexpr int kAhead = 8;          // loads in flight per warp; moves of a copying warp

struct MoveLayer {
  char *k, *v;
  int32_t row_bytes;
  int32_t blocks;      // envelope: row blocks of a page; per-layer: 0
  int32_t in_full;
};
struct MoveParams {
  MoveLayer layer[kMoveLayers];
  int32_t ps;
  int64_t rows_full, rows_swa;   // slots of each pool, padding page included
  const int64_t *mapping;        // longer than rows_full
  int32_t *err;
  // copy
  const int64_t *src, *dst;
  int64_t n;
  // commit
  const int32_t *rt;
  int64_t rt_stride;
  const int64_t *req_idx, *prefix;
  const int32_t *accepted, *n_accepted;
  int32_t max_accept;
};

// Rows of the move (full slots a -> b) in the layer's pool; false: nothing to
// move there.  A copy's source may have left the window (kNode false); a node of
// this step has its SWA slot, or the tables are broken.
template <bool kNode>
__device__ __forceinline__ bool move_rows(const MoveParams &P, const MoveLayer &L, int64_t a,
                                          int64_t b, int64_t &ra, int64_t &rb) {
  if (a < 0 || b < 0 || a >= P.rows_full || b >= P.rows_full) {
    set_error(P.err, SWA_DEVERR_RANGE);
    return false;
  }
  if (!L.in_full) {
    a = P.mapping[a];
    b = P.mapping[b];
    if (!kNode && a <= 0) return false;   // full layers only
    if (a <= 0 || b <= 0) {
      set_error(P.err, SWA_DEVERR_WINDOW_EVICTED);
      return false;
    }
    if (a >= P.rows_swa || b >= P.rows_swa) {
      set_error(P.err, SWA_DEVERR_RANGE);
      return false;
    }
  }
  if (a == b) return false;
  const KvAddr addr{nullptr, nullptr, 0, P.ps, L.blocks};
  ra = kv_row(addr, a) * L.row_bytes;
  rb = kv_row(addr, b) * L.row_bytes;
  return true;
}

// The moves held by the warp's lanes (lane i: rows ra -> rb when live), in
// lane order, for one 16-byte column of the row per lane.  Rows are loaded
// kAhead at a time before any of them is stored.
__device__ __forceinline__ void run_moves(char *base, int64_t col, bool in_row, bool live,
                                          int64_t ra, int64_t rb) {
  unsigned todo = __ballot_sync(0xffffffffu, live);
  while (todo) {
    uint4 x[kAhead];
    int64_t to[kAhead];
    int m = 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (todo) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1;
        const int64_t from = __shfl_sync(0xffffffffu, ra, l);
        to[u] = __shfl_sync(0xffffffffu, rb, l);
        if (in_row) x[u] = *reinterpret_cast<const uint4 *>(base + from + col);
        m = u + 1;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (u < m && in_row) *reinterpret_cast<uint4 *>(base + to[u] + col) = x[u];
  }
}

// grid: x = batches of kAhead moves x 512-byte columns, y = 2 x layer + (K or V)
__global__ void __launch_bounds__(kMoveWarps * 32)
    k_copy_kv(const __grid_constant__ MoveParams P, int cols) {
  const int lane = threadIdx.x & 31;
  const int64_t w = blockIdx.x * (int64_t)kMoveWarps + (threadIdx.x >> 5);
  const MoveLayer &L = P.layer[blockIdx.y >> 1];
  const int64_t i = (w / cols) * kAhead + lane;
  const int64_t col = (w % cols) * 512 + lane * 16;
  if ((w / cols) * kAhead >= P.n || (w % cols) * 512 >= L.row_bytes) return;
  int64_t ra = 0, rb = 0;
  bool live = false;
  if (lane < kAhead && i < P.n) {
    const int64_t a = P.src[i], b = P.dst[i];
    live = a != -1 && b != -1 && move_rows<false>(P, L, a, b, ra, rb);
  }
  run_moves((blockIdx.y & 1) ? L.v : L.k, col, col < L.row_bytes, live, ra, rb);
}

// The same for whole rows: their columns, in move order, so that every column
// sees its moves in lane order.
__device__ __forceinline__ void run_row_moves(char *rows, int row_bytes, int lane, bool live,
                                              int64_t ra, int64_t rb) {
  const int end = (row_bytes + 511) / 512 * 512;
  unsigned todo = __ballot_sync(0xffffffffu, live);
  int l = todo ? __ffs(todo) - 1 : 0, col = 0;   // move, column of it
  while (todo) {
    uint4 x[kAhead];
    char *to[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      to[u] = nullptr;
      if (todo) {
        char *base = rows + col + lane * 16;
        const int64_t from = __shfl_sync(0xffffffffu, ra, l), dst = __shfl_sync(0xffffffffu, rb, l);
        if (col + lane * 16 < row_bytes) {
          x[u] = *reinterpret_cast<const uint4 *>(base + from);
          to[u] = base + dst;
        }
        if ((col += 512) == end) {
          col = 0;
          todo &= todo - 1;
          l = todo ? __ffs(todo) - 1 : 0;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (to[u]) *reinterpret_cast<uint4 *>(to[u]) = x[u];
  }
}

// grid: x = requests, y = 2 x layer + (K or V).  Node accepted[j] >= j moves to
// column prefix + j.  Ascending order makes the moves safe in place: a move writes
// a column below every later source, and its own source is only overwritten by a
// later move - whose stores follow this warp's loads of the earlier moves (batches
// go in order; within a batch loads precede stores), and no other warp touches
// these bytes.
__global__ void __launch_bounds__(kMoveWarps * 32)
    k_commit_tree(const __grid_constant__ MoveParams P, int bs) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.x * kMoveWarps + (threadIdx.x >> 5);
  const MoveLayer &L = P.layer[blockIdx.y >> 1];
  if (b >= bs) return;
  const int64_t pre = P.prefix[b];
  const int32_t *row = P.rt + P.req_idx[b] * P.rt_stride;
  int a = lane < P.max_accept ? P.accepted[(int64_t)b * P.max_accept + lane] : 0;
  const int n = P.n_accepted[b];
  if (n < 0 || n > P.max_accept || pre < 0) {
    set_error(P.err, SWA_DEVERR_RANGE);
    return;
  }
  int prev = -1;
  for (int j0 = 0; j0 < n; j0 += 32) {
    const int j = j0 + lane;
    if (j0 > 0) a = j < n ? P.accepted[(int64_t)b * P.max_accept + j] : 0;
    int before = __shfl_up_sync(0xffffffffu, a, 1);
    if (lane == 0) before = prev;
    prev = __shfl_sync(0xffffffffu, a, 31);
    // Strictly ascending node indices inside the row; nothing moves from the
    // first offending entry on.
    const bool bad = j < n && (a <= before || a >= SWA_TREE_MAX_NODES || pre + a >= P.rt_stride);
    const unsigned wrong = __ballot_sync(0xffffffffu, bad);
    int64_t ra = 0, rb = 0;
    bool live = j < n && (!wrong || lane < __ffs(wrong) - 1) && a != j;
    if (live) live = move_rows<true>(P, L, row[pre + a], row[pre + j], ra, rb);
    run_row_moves((blockIdx.y & 1) ? L.v : L.k, L.row_bytes, lane, live, ra, rb);
    if (wrong) {
      set_error(P.err, SWA_DEVERR_RANGE);
      return;
    }
  }
}

// Launches `fn(params, layers of this launch, most 512-byte columns of a row)`
// over all layers.
template <typename F>
cudaError_t for_layers(const Ctx &c, MoveParams &P, F fn) {
  P.ps = c.cfg.page_size;
  P.rows_full = c.cfg.size_full + c.cfg.page_size;
  P.rows_swa = c.cfg.size_swa + c.cfg.page_size;
  P.mapping = c.mapping;
  P.err = c.err_word;
  const int total = (int)c.layers.size();
  for (int l0 = 0; l0 < total; l0 += kMoveLayers) {
    const int nl = total - l0 < kMoveLayers ? total - l0 : kMoveLayers;
    int64_t most = 0;
    for (int i = 0; i < nl; ++i) {
      const LayerInfo &L = c.layers[l0 + i];
      P.layer[i] = MoveLayer{L.addr.k, L.addr.v, (int32_t)L.addr.row_bytes, L.addr.blocks,
                             L.in_full ? 1 : 0};
      if (L.addr.row_bytes > most) most = L.addr.row_bytes;
    }
    fn(P, nl, (int)((most + 511) / 512));
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_copy_kv(Ctx &c, const int64_t *src, const int64_t *dst, int64_t n,
                           cudaStream_t s) {
  MoveParams P{};
  // A launch's moves keep its grid within 2^31 - 1 blocks whatever the row size.
  for (int64_t i = 0; i < n; i += kCopyMoves) {
    P.src = src + i;
    P.dst = dst + i;
    P.n = n - i < kCopyMoves ? n - i : kCopyMoves;
    const cudaError_t e = for_layers(c, P, [&](const MoveParams &p, int nl, int cols) {
      const int64_t warps = (p.n + kAhead - 1) / kAhead * cols;
      dim3 grid((unsigned)((warps + kMoveWarps - 1) / kMoveWarps), 2 * nl);
      k_copy_kv<<<grid, kMoveWarps * 32, 0, s>>>(p, cols);
    });
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_commit_tree(Ctx &c, int bs, const int32_t *rt, int64_t rt_stride,
                               const int64_t *req_idx, const int64_t *prefix,
                               const int32_t *accepted, int max_accept, const int32_t *n_accepted,
                               cudaStream_t s) {
  if (bs == 0) return cudaSuccess;
  MoveParams P{};
  P.rt = rt;
  P.rt_stride = rt_stride;
  P.req_idx = req_idx;
  P.prefix = prefix;
  P.accepted = accepted;
  P.n_accepted = n_accepted;
  P.max_accept = max_accept;
  return for_layers(c, P, [&](const MoveParams &p, int nl, int) {
    dim3 grid((bs + kMoveWarps - 1) / kMoveWarps, 2 * nl);
    k_commit_tree<<<grid, kMoveWarps * 32, 0, s>>>(p, bs);
  });
}

}  // namespace swa
