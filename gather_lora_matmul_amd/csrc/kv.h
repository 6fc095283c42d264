// KV cache in the unified page pool: geometry, device view and kernel
// launchers (internal).
//
// A sequence's cached tokens lie in blocks of T tokens.  Of every block each kv
// head has one K page and one V page.  With E elements in 16 bytes (8 of 16
// bits, 16 of FP8):
//   K page  [D / E][T][E]  element d of token slot t at ((d / E) * T + t) * E + d % E
//   V page  [T / E][D][E]  ... at ((t / E) * D + d) * E + t % E
// Both are the order in which the matrix instructions of the attention take
// their first operand (K rows: 16-byte pieces of the head dimension, one lane a
// token; V columns: 16-byte pieces of tokens, one lane an element of the head
// dimension), so a wave's 16-byte loads cover contiguous memory and no operand
// is transposed on the way.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lora_mi355x.h"

namespace lora {

constexpr int kKvMaxSeqs = 1024;   // sequences of one batch
constexpr int kKvMaxHeads = 256;   // kv heads

struct KvView {
  char* pages;             // pool base
  uint8_t* scales;         // FP8: exponent bytes [n_pages][T], else null
  int64_t page_bytes;
  int32_t n_pages;
  int32_t T;               // tokens of a page, a multiple of E
  uint32_t div_m;          // x / T = (x * div_m >> 32) >> div_s for 0 <= x < 2^31
  int32_t div_s;
  int32_t H;               // kv heads
  int32_t n_seqs;
  int32_t n_tokens;        // rows of the new tensors
  int32_t nb;              // blocks of a table row
  const int32_t* q_start;  // [n_seqs + 1]
  const int32_t* kv_len;   // [n_seqs]
  const int32_t* table;    // [n_seqs][2][H][nb]
};

__host__ __device__ inline uint32_t kv_div(const KvView& v, uint32_t x) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __umulhi(x, v.div_m) >> v.div_s;
#else
  return (uint32_t)(((uint64_t)x * v.div_m) >> 32) >> v.div_s;
#endif
}
// The multiplier of division by d >= 2: with 2^(k-1) < d <= 2^k,
// m = ceil(2^(31 + k) / d) < 2^32, and x * m >> (31 + k) is exact below 2^31.
inline void div_init(int32_t d, uint32_t& m, int32_t& s) {
  int k = 1;
  while ((1 << k) < d) ++k;
  m = (uint32_t)((((uint64_t)1 << (31 + k)) + (uint64_t)d - 1) / (uint64_t)d);
  s = k - 1;
}

// Rows of one sequence's new tokens, their positions, and its cached tokens, with
// everything that comes from device memory held inside the buffers: rows inside
// [0, n_tokens], cached tokens inside the table's row.  Positions follow the lengths
// as they are given (the first row's is kv_len - q_len, and what rows before row 0
// there are), so that cutting rows or tokens off moves none of the others.
struct KvSeq {
  int32_t q0, q_len;   // rows q0 .. q0 + q_len - 1
  int32_t base;        // position of row q0, held inside +-2^29 (no token is there)
  int32_t end;         // cached tokens that the table has place for
};
__host__ __device__ inline KvSeq kv_seq(const KvView& v, int s) {
  KvSeq r;
  const int cap = v.nb * v.T, far = 1 << 29;   // (cap <= 2^28, checked on the host)
  const int a = v.q_start[s], b = v.q_start[s + 1], n = v.kv_len[s] < 0 ? 0 : v.kv_len[s];
  r.q0 = a < 0 ? 0 : (a > v.n_tokens ? v.n_tokens : a);
  const int e = b < r.q0 ? r.q0 : (b > v.n_tokens ? v.n_tokens : b);
  r.q_len = e - r.q0;
  // n - (b - a) + (q0 - a); sums past 32 bits stay at their ends, beyond far
  const int base = __builtin_elementwise_add_sat(__builtin_elementwise_sub_sat(n, b), r.q0);
  r.base = base < -far ? -far : (base > far ? far : base);
  r.end = n > cap ? cap : n;
  return r;
}

// Element types: act of q/k/v/out rows (LORA_F16 or LORA_BF16), kv of the cache
// (the same, or LORA_FP8_E4M3).
struct KvTypes {
  int act, kv, D;
};

hipError_t launch_kv_write(const KvTypes& ty, const KvView& v, const void* k, const void* vv,
                           int64_t ld, hipStream_t s);
hipError_t launch_kv_read(const KvTypes& ty, const KvView& v, void* k, void* vv, int64_t ld,
                          hipStream_t s);

struct AttendArgs {
  KvView kv;
  const void* q;
  int64_t q_ld;            // elements between tokens
  void* out;
  int64_t out_ld;
  float* lse;              // [n_tokens][n_q_heads] or null
  int32_t n_q_heads;
  int32_t group;           // query heads of a kv head, and the multiplier of division
  uint32_t group_m;        // by it (if it is not 1)
  int32_t group_s;
  int32_t max_q_len;
  bool two_terms;          // of the weights, in long work too
  float scale_log2;        // scale * log2(e)
  int32_t window;          // 0: none
  char* ws;
  int32_t n_cu;
};
// Rows that are tokens of trees: which of their sequence's new tokens they see, and how
// deep they are.
struct TreeArgs : AttendArgs {
  const uint64_t* seen;    // [n_tokens][words]
  const int32_t* depth;    // [n_tokens], read if there is a window
  int32_t words;
};
size_t attend_workspace(const KvTypes& ty, int32_t n_cu, int32_t group, int32_t max_q_len, int32_t n_seqs,
                        int32_t H);
// A bound of the units of work of a call, to stay below 2^31.
int64_t attend_units(const KvView& v, int32_t group, int32_t max_q_len);
hipError_t launch_attend(const KvTypes& ty, const AttendArgs& a, hipStream_t s);
hipError_t launch_attend_tree(const KvTypes& ty, const TreeArgs& a, hipStream_t s);

struct VerifyArgs {
  int32_t n_seqs, n_tokens, n_drafts, vocab, dtype;
  int64_t target_ld, draft_ld;
  const int32_t* q_start;
  const int32_t* drafted;
  const void* target;
  const void* draft;       // null: the draft gave its token with certainty
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;
  int32_t* n_out;
  char* ws;
};
size_t verify_workspace(int32_t n_seqs, int32_t vocab);
hipError_t launch_verify(const VerifyArgs& a, hipStream_t s);


// Trees of drafted tokens.
struct TreeBuildArgs {
  int32_t n_seqs, n_tokens, words, window;
  const int32_t* q_start;
  const int32_t* parent;
  uint64_t* seen;          // [n_tokens][words]
  int32_t* depth;          // [n_tokens]
};
hipError_t launch_tree_build(const TreeBuildArgs& a, hipStream_t s);

constexpr int kTreeTokens = 1024;   // tokens of a tree (16 words)

struct TreeVerifyArgs {
  int32_t n_seqs, n_tokens, vocab, dtype, path_ld;
  int64_t target_ld;
  const int32_t* q_start;
  const int32_t* parent;
  const int32_t* drafted;
  const void* target;
  const float* u_accept;
  const float* u_sample;
  int32_t* tokens;         // [n_seqs][path_ld]
  int32_t* path;           // [n_seqs][path_ld]
  int32_t* n_out;
  char* ws;
};
size_t tree_verify_workspace(int32_t n_seqs, int32_t vocab);
hipError_t launch_tree_verify(const TreeVerifyArgs& a, hipStream_t s);

// The attention that cached tokens get.
struct WeighArgs {
  KvView kv;
  const void* q;
  int64_t q_ld;
  const float* lse;        // [n_tokens][n_q_heads]
  const float* before;     // [n_seqs][H][w_ld] or null
  float* weights;
  int64_t w_ld;
  int32_t n_q_heads;
  int32_t group;           // as in AttendArgs
  uint32_t group_m;
  int32_t group_s;
  int32_t max_q_len;
  float scale_log2;
  float decay;
  int32_t window;
  char* ws;
  int32_t n_cu;
};
size_t weigh_workspace(int32_t n_cu, int32_t group, int32_t max_q_len);
int64_t weigh_units(const KvView& v);
hipError_t launch_weigh(const KvTypes& ty, const WeighArgs& a, hipStream_t s);

// Eviction: the tokens that stay, and their way to the front.
struct SelectArgs {
  KvView kv;
  const float* weights;    // [n_seqs][H][w_ld]
  int64_t w_ld;
  int32_t budget, sinks, recent;
  int32_t* keep;           // [n_seqs][H][keep_ld]
  int64_t keep_ld;
  int32_t* n_keep;         // [n_seqs]
  char* ws;
};
size_t select_workspace(int32_t n_seqs, int32_t H, int64_t tokens);   // tokens: that a table's row has place for
hipError_t launch_select(const SelectArgs& a, hipStream_t s);

struct CompactArgs {
  KvView kv;
  const int32_t* keep;     // [n_seqs][keep_heads][keep_ld]
  int64_t keep_ld;
  int32_t keep_heads;      // 1 or H
  const int32_t* n_keep;
  bool from_new;           // numbers count from the first new token
  float* weights;          // [n_seqs][H][w_ld] or null
  int64_t w_ld;
};
hipError_t launch_compact(const KvTypes& ty, const CompactArgs& a, hipStream_t s);

}  // namespace lora
