// tree_accept.cu -- the walk down a drafted tree along the tokens that were sampled
// behind its nodes (sm_103a).
//
// From node 0 on: of the current node's children the first one whose token is the
// node's sampled token is accepted and becomes the current node; where there is none
// the walk ends.  A CTA takes a request.  All children look at their parents at
// once: next[p] = min over children c of p with token(c) = sampled(p), an integer
// minimum in shared memory, whose order does not matter.  What is left of the walk is
// one shared-memory read a step.
//
// Bound by the chain of dependent steps: offsets, nodes, next, walk, results.  128 trees of 40 to
// 64 nodes take 3 us on the device, of which 2 are the launch; a call 4.4 on the host.
#include <limits.h>

#include "common.cuh"
#include "internal.h"

namespace dflash {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxNodes = DFLASH_TREE_MAX_NODES;

__global__ void __launch_bounds__(kThreads) accept_kernel(const __grid_constant__ AcceptArgs a) {
  __shared__ int32_t s_next[kMaxNodes], s_sampled[kMaxNodes];
  const int r = blockIdx.x, tid = threadIdx.x;
  const int t0 = a.offsets[r], t1 = a.offsets[r + 1], n = t1 - t0;
  int32_t* path = a.path + (long long)r * a.max_path;
  int32_t* out = a.out + (long long)r * a.max_path;
  // (t1 < t0 by itself: of offsets far apart the difference wraps)
  const bool bad = t0 < 0 || t1 < t0 || t1 > a.total || n > kMaxNodes;
  if (bad && tid == 0) record_error(a.err, DFLASH_ERR_INVALID);
  const int nodes = bad ? 0 : n;
  for (int j = tid; j < nodes; j += kThreads) {
    s_next[j] = INT_MAX;
    s_sampled[j] = a.sampled[t0 + j];
  }
  __syncthreads();
  for (int j = tid; j < nodes; j += kThreads) {
    const int p = a.parents[t0 + j];
    if (j > 0 && p >= 0 && p < j && a.tokens[t0 + j] == s_sampled[p]) atomicMin(&s_next[p], j);
  }
  __syncthreads();
  // every thread walks for itself and writes the steps that are its
  int count = 0;
  for (int at = 0; at < nodes && count < a.max_path; at = s_next[at], ++count)
    if (count % kThreads == tid) {
      path[count] = at;
      out[count] = s_sampled[at];
    }
  for (int j = count + tid; j < a.max_path; j += kThreads) path[j] = out[j] = -1;
  if (tid == 0) a.count[r] = count;
}

}  // namespace

cudaError_t launch_tree_accept(const AcceptArgs& a, cudaStream_t stream) {
  accept_kernel<<<a.R, kThreads, 0, stream>>>(a);
  count_launch();
  return cudaGetLastError();
}

}  // namespace dflash
