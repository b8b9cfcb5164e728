// Internal declarations of the speculative-step operators: the draft-tree plan
// and tree attention, the q/k norm + rotation + store, and the row moves.
#pragma once

#include <atomic>

#include "swa_internal.h"

namespace swa {

// Draft-tree plan in the caller's `tree` buffer, shared by every layer of a
// step: depth int32 [n_tokens], then one ancestor bit row per node, uint32
// [n_tokens][words] (bit j of node i's row: node j of the same request is i
// itself or an ancestor of i), words = ceil(max_new / 32).
struct TreeView {
  int32_t *depth;
  uint32_t *mask;
  int32_t words;
};
inline size_t tree_depth_bytes(int64_t n_tokens) {
  return ((size_t)n_tokens * sizeof(int32_t) + 255) / 256 * 256;
}
inline TreeView tree_view(const void *tree, int64_t n_tokens, int max_new) {
  TreeView t;
  char *p = const_cast<char *>(static_cast<const char *>(tree));
  t.depth = reinterpret_cast<int32_t *>(p);
  t.mask = p ? reinterpret_cast<uint32_t *>(p + tree_depth_bytes(n_tokens)) : nullptr;
  t.words = (max_new + 31) / 32;
  return t;
}

// First column of req_to_token that node `node` (of depth `depth`, ancestor
// row `mask`) may read on a layer whose first attended position is lo, given
// the request's prefix length.  Cached columns are positions; a node's
// ancestors have one position each, d levels up being position p - d, and
// ascend in node index, so when lo falls behind the prefix (a window shorter
// than the node's depth) the columns allowed are those from the
// (p - lo + 1)-th set bit counted from the top on.
__device__ inline int64_t tree_first_col(int64_t lo, int64_t prefix, int node, int depth,
                                         const uint32_t *mask) {
  if (lo <= prefix) return lo;
  int keep = (int)(prefix + depth - lo + 1);   // nodes allowed, the query's own included
  for (int w = node >> 5; w >= 0; --w) {
    uint32_t m = mask[w];
    const int c = __popc(m);
    if (c < keep) {
      keep -= c;
      continue;
    }
    while (--keep) m &= ~(0x80000000u >> __clz(m));
    return prefix + 32 * w + 31 - __clz(m);
  }
  return prefix;   // unreachable for a valid row: it has depth + 1 > keep bits
}

__host__ __device__ inline int64_t first_position(int kind, int window, int64_t p) {
  if (kind == SWA_LAYER_FULL) return 0;
  if (kind == SWA_LAYER_SLIDING) return p - window > 0 ? p - window : 0;
  return (p / window) * window;
}

// Raises a kernel's dynamic shared memory limit, once per device and kernel
// (`done`: one bit per device; a repeated call is harmless).
template <typename K>
cudaError_t allow_smem(K *kernel, size_t bytes, int device, std::atomic<uint64_t> &done) {
  const uint64_t bit = 1ull << (device & 63);
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && device < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// ---- tree_plan.cu -----------------------------------------------------------
cudaError_t launch_tree_plan(Ctx &c, int bs, const int32_t *parents, const int64_t *prefix,
                             const int64_t *qo_indptr, int64_t n_tokens, int max_new,
                             int64_t *positions, const TreeView &tree, cudaStream_t s);

// ---- attn_simt.cu: generic tree attention ------------------------------------
// The most keys a node may have: its window before it, and the nodes.
int64_t tree_max_keys(const Ctx &c, int layer, int max_new, int max_seq_len);
size_t simt_tree_ws_bytes(const Ctx &c, int layer, int64_t nq, int max_new, int max_seq_len);
cudaError_t launch_attn_tree_simt(Ctx &c, const AttnArgs &a, const TreeView &tree, cudaStream_t s);

// ---- tma.cu -------------------------------------------------------------------
// TMA tensor map over queries x [nq][hq][d] (bf16) whose box is one tile of t
// tokens x g heads, 64 dims wide.  False as for make_qo_tensor_map.
bool make_q_tile_map(CUtensorMap *m, const void *x, int64_t nq, int hq, int d, int g, int t);

// ---- attn_tree_tc.cu ------------------------------------------------------------
bool tc_tree_supported(const Ctx &c, int layer);
size_t tc_tree_ws_bytes(const Ctx &c, int layer, int bs, int64_t nq, int max_new,
                        int max_seq_len);
cudaError_t launch_attn_tree_tc(Ctx &c, const AttnArgs &a, const TreeView &tree, cudaStream_t s);

// ---- qk_norm_rope.cu ----------------------------------------------------------
struct QkNormArgs {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  int64_t n;
  const int64_t *positions;
  const float *q_weight, *k_weight;
  float eps;
  const float *cos_sin;
  int64_t max_pos;
  int rot_dim;
  bool interleaved;
  const int64_t *full_loc, *swa_loc;
  float k_scale, v_scale;
  void *q_out;
};
cudaError_t launch_qk_norm_rope_store(Ctx &c, int layer, const QkNormArgs &a, cudaStream_t s);

// ---- kv_move.cu ---------------------------------------------------------------
cudaError_t launch_copy_kv(Ctx &c, const int64_t *src, const int64_t *dst, int64_t n,
                           cudaStream_t s);
cudaError_t launch_commit_tree(Ctx &c, int bs, const int32_t *rt, int64_t rt_stride,
                               const int64_t *req_idx, const int64_t *prefix,
                               const int32_t *accepted, int max_accept, const int32_t *n_accepted,
                               cudaStream_t s);

}  // namespace swa
