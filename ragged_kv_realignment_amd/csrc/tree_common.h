// Trees of drafted tokens: node 0 is the root, parent[i] < i, anything else
// marks a node that is not used.  Shared by the tree kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include "device_common.h"
#include "launch.h"
#include "specdec.h"

namespace sd {

// Node i's parent as the kernels use it: 0 for the root itself, -1 for a node
// that is not used.  `bad` is set where the value is no mark of that (a parent
// that does not come before its child, or below -1).
__device__ __forceinline__ int node_parent(int i, int raw, bool &bad) {
  if (i == 0) return 0;
  bad = bad || raw >= i || raw < -1;
  return raw >= 0 && raw < i ? raw : -1;
}

// Pointer doubling over the tree in LDS: after ceil(log2 N) rounds every node's
// pointer has reached the root (0) or an unused node (-1), in place of a walk
// of up to N - 1 dependent steps.  ptr[i] holds node_parent and steps[i] the
// number of edges ptr[i] spans (0 for the root); thread i owns node i
// (NT >= N).  On return steps[i] is the depth of node i where ptr[i] is 0.
template <int NT>
__device__ __forceinline__ void tree_depths(int N, int *ptr, int *steps) {
  static_assert(NT >= kMaxNodes, "one node per thread");
  const int i = threadIdx.x;
  for (int span = 1; span < N; span <<= 1) {
    __syncthreads();
    int q = -1, d = 0;
    if (i < N) {
      q = ptr[i];
      d = steps[i];
      if (q > 0) {
        d += steps[q];
        q = ptr[q];
      }
    }
    __syncthreads();
    if (i < N) {
      ptr[i] = q;
      steps[i] = d;
    }
  }
  __syncthreads();
}

}  // namespace sd
