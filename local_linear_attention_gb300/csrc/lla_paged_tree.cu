// Trees of drafted tokens: what the attention kernels of many rows and of fp32 need of a tree. For every
// node the nodes that it sees, as bits (itself and its ancestors, less those that fell out of the window),
// and its depth. The few-rows and the fp32 kernel do the same between a warp's lanes for up to 64 nodes.
//
// A thread per node goes up the tree by parents in shared memory. Indices fall on the way, so the words of a
// node's bits are met from the last to the first and each is written once, without atomics. What bounds
// it: the launch and the longest way up (6 us by itself with cold caches for 16 trees of 32 nodes; a call without it takes
// 1.8 us less); the attention is set up meanwhile and waits only where it meets the first masked keys.
#include "lla_paged.cuh"

namespace lla {
namespace paged {
namespace {

__global__ void __launch_bounds__(256) tree_kernel(Params p, uint32_t* bits, int* depth) {
  __shared__ int parent[kMaxNodes];
  let_next();  // which waits for this kernel's end itself
  const int b = blockIdx.x;
  const Seq sq = load_seq<true>(p, b);
  if (sq.n == 0) return;
  if (!mine(p, sq.n)) {
    if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(p.status, kStatusBadIndex);  // beyond max_new
    return;
  }
  const int upto = min(sq.n, (int)(blockIdx.y + 1) * 256);
  for (int i = threadIdx.x; i < upto; i += 256) {
    const int a = __ldg(p.parents + sq.t0 + i);
    const bool good = a >= -1 && a < i;
    if (!good) atomicOr(p.status, kStatusBadIndex);
    parent[i] = good ? a : -1;
  }
  __syncthreads();
  const int i = blockIdx.y * 256 + threadIdx.x;
  if (i >= sq.n) return;
  int d = 0;
  for (int a = parent[i]; a >= 0; a = parent[a]) ++d;
  depth[sq.t0 + i] = d;
  uint32_t* const out = bits + (long long)(sq.t0 + i) * p.words;
  int word = p.words - 1;
  uint32_t have = 0;
  int up = 0;
  for (int a = i; a >= 0; a = parent[a], ++up) {
    for (; word > a >> 5; --word) {
      out[word] = have;
      have = 0;
    }
    if (up < p.window || sq.first + d - up < p.sinks) have |= 1u << (a & 31);
  }
  for (; word >= 0; --word) {
    out[word] = have;
    have = 0;
  }
}

}  // namespace

cudaError_t launch_tree(const Params& p, uint32_t* bits, int* depth, int max_nodes, cudaStream_t s) {
  return launch(tree_kernel, dim3((unsigned)p.B, (unsigned)(max_nodes + 255) / 256), 256, 0, 1, false, s, p, bits, depth);
}

}  // namespace paged
}  // namespace lla
