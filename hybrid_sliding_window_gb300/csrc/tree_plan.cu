// Draft-tree plan: each node's depth, position and ancestor bit row, built once
// per step and read by every layer's tree attention.
//
// A drafted tree comes as parent indices (node j of a request is a child of
// node parents[j] < j, or of the request's last cached token when -1).  A
// node's depth is the number of its proper ancestors among the nodes, its
// position prefix + depth, and its bit row the set of nodes it may attend:
// itself and its ancestors.
//
// One CTA per request: the parents go to shared memory and each thread walks
// one node's path to the root.  Parents have smaller indices, so the path
// visits the words of the bit row from high to low and every word is written
// once, from a register.  The walk costs one shared-memory load per level
// (about 30 cycles); the launch is latency: 2.3 us for 64 trees of 8 nodes, 3.7
// for one of 64.
#include <cuda_runtime.h>

#include "spec_internal.h"

namespace swa {
namespace {

constexpr int kPlanThreads = 128;

__global__ void __launch_bounds__(kPlanThreads)
    k_tree_plan(const int32_t *parents, const int64_t *prefix, const int64_t *qo_indptr,
                int64_t n_tokens, int max_new, int64_t *positions, TreeView tree, int32_t *err) {
  __shared__ int16_t s_parent[SWA_TREE_MAX_NODES];
  // The attention launched next may set itself up meanwhile (it waits for this
  // kernel's end before it reads anything).
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  const int b = blockIdx.x;
  const int64_t q0 = qo_indptr[b];
  int64_t n = qo_indptr[b + 1] - q0;
  const int64_t pre = prefix[b];
  if (n <= 0) return;
  // Rows outside the buffers, or more nodes than the bit rows hold.
  if (q0 < 0 || q0 + n > n_tokens || n > max_new || pre < 0) {
    if (threadIdx.x == 0) set_error(err, SWA_DEVERR_RANGE);
    if (q0 < 0 || q0 >= n_tokens || pre < 0) return;
    n = min(min(n, n_tokens - q0), (int64_t)max_new);
  }
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    int p = parents[q0 + i];
    if (p < -1 || p >= i) {
      set_error(err, SWA_DEVERR_RANGE);
      p = -1;
    }
    s_parent[i] = (int16_t)p;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kPlanThreads) {
    uint32_t *row = tree.mask + (q0 + i) * tree.words;
    for (int w = tree.words - 1; w > (i >> 5); --w) row[w] = 0u;
    int depth = -1, w = i >> 5;
    uint32_t bits = 0u;
    for (int j = i; j >= 0; j = s_parent[j]) {
      while (w > (j >> 5)) {
        row[w--] = bits;
        bits = 0u;
      }
      bits |= 1u << (j & 31);
      ++depth;
    }
    for (; w >= 0; --w) {
      row[w] = bits;
      bits = 0u;
    }
    tree.depth[q0 + i] = depth;
    if (positions) positions[q0 + i] = pre + depth;
  }
}

}  // namespace

cudaError_t launch_tree_plan(Ctx &c, int bs, const int32_t *parents, const int64_t *prefix,
                             const int64_t *qo_indptr, int64_t n_tokens, int max_new,
                             int64_t *positions, const TreeView &tree, cudaStream_t s) {
  if (bs == 0 || n_tokens == 0) return cudaSuccess;
  k_tree_plan<<<bs, kPlanThreads, 0, s>>>(parents, prefix, qo_indptr, n_tokens, max_new, positions,
                                          tree, c.err_word);
  return cudaGetLastError();
}

}  // namespace swa
