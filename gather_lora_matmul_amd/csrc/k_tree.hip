// Trees of drafted tokens: which of their sequence's new tokens each token sees.
//
// A thread walks from its token up to the root through the parents in LDS, of whom
// every one has a lower number, so that the words of a row are finished one after
// another from the highest down.  Bound by the launch and by one LDS read a level.
#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

__global__ __launch_bounds__(256) void k_tree_build(TreeBuildArgs a) {
  __shared__ int16_t up[kTreeTokens];
  const int s = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
  int b = a.q_start[s], e = a.q_start[s + 1];
  b = b < 0 ? 0 : (b > a.n_tokens ? a.n_tokens : b);
  e = e < b ? b : (e > a.n_tokens ? a.n_tokens : e);
  const int n = e - b, in = min(n, 64 * a.words);   // tokens from 64 words on are in no tree
  for (int t = tid; t < in; t += threads) {
    const int p = a.parent[b + t];
    up[t] = (int16_t)(p >= 0 && p < t ? p : -1);
  }
  __syncthreads();
  for (int t = tid; t < n; t += threads) {
    uint64_t* row = a.seen + (int64_t)(b + t) * a.words;
    int word = a.words - 1, depth = 0;
    uint64_t bits = 0;
    for (int p = t < in ? t : -1; p >= 0; p = up[p], ++depth) {
      if (a.window > 0 && depth >= a.window) continue;
      for (; word > p >> 6; --word, bits = 0) row[word] = bits;
      bits |= (uint64_t)1 << (p & 63);
    }
    for (; word >= 0; --word, bits = 0) row[word] = bits;
    a.depth[b + t] = depth > 0 ? depth - 1 : 0;
  }
}

}  // namespace

hipError_t launch_tree_build(const TreeBuildArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_tree_build, dim3(a.n_seqs), dim3(64 * (a.words < 4 ? a.words : 4)), 0, s, a);
  return hipGetLastError();
}

}  // namespace lora
