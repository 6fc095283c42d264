// Trees of drafted tokens: which of their sequence's new tokens each token sees.
//
// A wave has 64 of a sequence's tokens, those of one word of the rows.  Within these a
// token's ancestors come by doubling: the path up to a link, and from there the link's own path,
// so that all are there after log2 of the longest path.  The lower words are the paths of the
// links that leave the 64, one hop a word.  Ancestors lie in the order of their numbers, so a
// window keeps a row's highest bits.  Bound by the launch: 128 trees of up to 250 tokens take
// 4.1 us, a chain of 1024 11 (each token's walk up its whole path: 4.1 and 273).
#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

__global__ __launch_bounds__(kTreeTokens) void k_tree_build(TreeBuildArgs a) {
  __shared__ uint64_t paths[kTreeTokens];
  __shared__ int16_t links[kTreeTokens];
  const int s = blockIdx.x, t = threadIdx.x, first = t & ~63;
  int b = a.q_start[s], e = a.q_start[s + 1];
  b = b < 0 ? 0 : (b > a.n_tokens ? a.n_tokens : b);
  e = e < b ? b : (e > a.n_tokens ? a.n_tokens : e);
  const int n = e - b, in = min(n, 64 * a.words);   // tokens from 64 words on are in no tree
  int link = t < in ? a.parent[b + t] : -1;   // the path from t ends below it
  link = link >= 0 && link < t ? link : -1;
  uint64_t path = (uint64_t)1 << (t & 63);
  while (__any(link >= first)) {
    const uint64_t path_on = __shfl(path, link & 63);
    const int link_on = __shfl(link, link & 63);
    const bool on = link >= first;
    path |= on ? path_on : 0;
    link = on ? link_on : link;
  }
  paths[t] = path;
  links[t] = (int16_t)link;
  __syncthreads();
  if (t < in) {
    int depth = -1, left = a.window > 0 ? a.window : kTreeTokens;   // bits that the row still may have
    uint64_t* row = a.seen + (int64_t)(b + t) * a.words;
    link = t;
    for (int i = a.words - 1; i >= 0; --i) {
      uint64_t bits = 0;
      if (link >> 6 == i) {
        bits = paths[link];
        link = links[link];
        depth += __popcll(bits);
      }
      for (int drop = __popcll(bits) - left; drop > 0; --drop) bits &= bits - 1;
      left -= __popcll(bits);
      row[i] = bits;
    }
    a.depth[b + t] = depth;
  }
  for (int i = in + t; i < n; i += blockDim.x) {
    for (int w = 0; w < a.words; ++w) a.seen[(int64_t)(b + i) * a.words + w] = 0;
    a.depth[b + i] = 0;
  }
}

}  // namespace

hipError_t launch_tree_build(const TreeBuildArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(k_tree_build, dim3(a.n_seqs), dim3(64 * a.words), 0, s, a);
  return hipGetLastError();
}

}  // namespace lora
