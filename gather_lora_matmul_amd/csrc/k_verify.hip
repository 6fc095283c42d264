// Verification of drafted tokens.
//
// Row i of a sequence with k drafted tokens d_0 .. d_{k-1}: the target's
// probabilities p_i and the draft's q_i.  d_i is accepted while
//   u_i q_i(d_i) < p_i(d_i)
// and at the first refusal (or after the last acceptance, with q = 0) one more
// token is drawn with weights max(p_i - q_i, 0): the smallest v whose cumulative
// weight exceeds u times the total.  Weights are whole multiples of 2^-44, so
// that their sums, and with them the token, are the same for every split and
// order of the work.
//
// Bound by the reads of one p row and (after a refusal) one q row a sequence.
// Two launches: the sums of pieces of kPiece probabilities, all sequences' pieces
// at once; then one block a sequence finds the piece that holds the level, reads
// that piece again and finds the token.
#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

constexpr int kPiece = 2048;
constexpr int kThreads = 256;
constexpr int kPer = kPiece / kThreads;

struct VerifySums {
  uint64_t rest, all;   // of max(p - q, 0) and of p
};

// x clamped to [0, 1] (NaN: 0) in whole multiples of 2^-44, rounded down.
__device__ __forceinline__ uint64_t fixed44(float x) {
  if (!(x > 0.f)) return 0;
  if (x >= 1.f) return 1ull << 44;
  const uint32_t b = __float_as_uint(x);
  const int e = (int)(b >> 23);
  const uint32_t mant = (b & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = e - 106;   // mant * 2^(e - 150) * 2^44
  return sh >= 0 ? (uint64_t)mant << sh : (sh > -24 ? mant >> -sh : 0);
}

template <typename T>
__device__ __forceinline__ float prob(const void* base, int64_t i) {
  return load_y<T>(base, i);
}

struct VerifySeq {
  int q0, k;        // first row, drafted tokens (-1: no rows)
  int first;        // accepted tokens
  int64_t drow;     // draft row of the first drafted token
};

// Rows [b, e) of a sequence, held inside the target's.
__device__ __forceinline__ void rows_of(const VerifyArgs& a, int s, int& b, int& e) {
  b = a.q_start[s];
  e = a.q_start[s + 1];
  b = b < 0 ? 0 : (b > a.n_tokens ? a.n_tokens : b);
  e = e < b ? b : (e > a.n_tokens ? a.n_tokens : e);
}

// The drafted tokens of one sequence that are accepted; the same in every wave.
// Every thread of the block calls it.
template <typename T>
__device__ __forceinline__ VerifySeq accept(const VerifyArgs& a, int s) {
  VerifySeq r;
  int b, e;
  rows_of(a, s, b, e);
  r.q0 = b;
  r.k = e - b - 1;
  // each sequence with rows before this one has one row that is no draft's
  r.drow = (int64_t)b;
  for (int i0 = 0; i0 < s; i0 += kThreads) {
    const int i = i0 + (int)threadIdx.x;
    int ib = 0, ie = 0;
    if (i < s) rows_of(a, i, ib, ie);
    r.drow -= __syncthreads_count(ie > ib);
  }
  r.first = 0;
  if (r.k > 0 && (r.drow < 0 || r.drow + r.k > a.n_drafts)) r.k = 0;  // rows that are not there
  const int lane = threadIdx.x & 63;
  for (int t0 = 0; t0 < r.k; t0 += 64) {
    const int t = t0 + lane;
    bool ok = false;
    if (t < r.k) {
      const int tok = a.drafted[r.drow + t];
      if ((unsigned)tok < (unsigned)a.vocab) {
        const float p = prob<T>(a.target, (int64_t)(r.q0 + t) * a.target_ld + tok);
        const float q = a.draft ? prob<T>(a.draft, (r.drow + t) * a.draft_ld + tok) : 1.f;
        ok = a.u_accept[r.drow + t] * q < p;
      }
    }
    const unsigned long long no = __ballot(!ok);
    const int n = no ? __builtin_ctzll(no) : 64;
    r.first += n;
    if (n < 64) break;
  }
  return r;
}

// Weights of the thread's probabilities of a piece: element piece * kPiece +
// e(j) with e(j) = j * 256 + tid, or 4 (8) consecutive ones where rows are
// aligned for 16-byte loads.
template <typename T, bool VEC>
__device__ __forceinline__ int elem(int j) {
  constexpr int E = 16 / ET<T>::bytes;
  return VEC ? (j / E * kThreads + (int)threadIdx.x) * E + j % E : j * kThreads + (int)threadIdx.x;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_piece(const void* base, int64_t row0, int v0, int vocab, float* f) {
  constexpr int E = 16 / ET<T>::bytes;
  if constexpr (VEC) {
#pragma unroll
    for (int j = 0; j < kPer; j += E) {
      const int v = v0 + elem<T, true>(j);
      if (v + E <= vocab) {
        unpack16<T>(ld16(reinterpret_cast<const char*>(base) + (row0 + v) * ET<T>::bytes), f + j);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) f[j + i] = v + i < vocab ? prob<T>(base, row0 + v + i) : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int v = v0 + elem<T, false>(j);
      f[j] = v < vocab ? prob<T>(base, row0 + v) : 0.f;
    }
  }
}

// (p, max(p - q, 0)) of the thread's elements of a piece at the row of the new token.
template <typename T, bool VEC>
__device__ __forceinline__ void piece_weights(const VerifyArgs& a, const VerifySeq& r, int piece, float* p,
                                              float* rest) {
  const int v0 = piece * kPiece;
  load_piece<T, VEC>(a.target, (int64_t)(r.q0 + r.first) * a.target_ld, v0, a.vocab, p);
  if (r.first >= r.k) {
#pragma unroll
    for (int j = 0; j < kPer; ++j) rest[j] = p[j];
  } else if (a.draft) {
    load_piece<T, VEC>(a.draft, (r.drow + r.first) * a.draft_ld, v0, a.vocab, rest);
#pragma unroll
    for (int j = 0; j < kPer; ++j) rest[j] = p[j] - rest[j];
  } else {
    const int tok = a.drafted[r.drow + r.first] - v0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) rest[j] = elem<T, VEC>(j) == tok ? 0.f : p[j];
  }
}

__device__ __forceinline__ uint64_t wave_add(uint64_t x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void k_verify_sums(VerifyArgs a, VerifySums* __restrict__ sums) {
  __shared__ VerifySums sh[kThreads / 64];
  const int s = blockIdx.y, piece = blockIdx.x;
  const VerifySeq r = accept<T>(a, s);
  if (r.k < 0) return;
  float p[kPer], rest[kPer];
  piece_weights<T, VEC>(a, r, piece, p, rest);
  VerifySums w{0, 0};
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    w.rest += fixed44(rest[j]);
    w.all += fixed44(p[j]);
  }
  w.rest = wave_add(w.rest);
  w.all = wave_add(w.all);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = w;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int i = 1; i < kThreads / 64; ++i) {
      w.rest += sh[i].rest;
      w.all += sh[i].all;
    }
    sums[(int64_t)s * gridDim.x + piece] = w;
  }
}

// Inclusive prefix sums of x over the block; total returned.
__device__ __forceinline__ uint64_t block_scan(uint64_t x, uint64_t* sh, uint64_t& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  total = 0;
  for (int i = 0; i < kThreads / 64; ++i) {
    if (i < wave) x += sh[i];
    total += sh[i];
  }
  __syncthreads();
  return x;
}

template <typename T, bool VEC>
__global__ __launch_bounds__(kThreads) void k_verify_pick(VerifyArgs a, const VerifySums* __restrict__ sums,
                                                           int pieces) {
  __shared__ uint64_t sh[kThreads / 64];
  __shared__ uint64_t weight[kPiece];
  __shared__ uint64_t sh_before;
  __shared__ int sh_piece, sh_token;
  const int s = blockIdx.x, tid = threadIdx.x;
  const VerifySeq r = accept<T>(a, s);
  if (r.k < 0) {
    if (tid == 0) a.n_out[s] = 0;
    return;
  }
  // pieces <= 256: a thread each
  VerifySums mine{0, 0};
  if (tid < pieces) mine = sums[(int64_t)s * pieces + tid];
  uint64_t total, total_all;
  const uint64_t up = block_scan(mine.rest, sh, total);
  const uint64_t up_all = block_scan(mine.all, sh, total_all);
  const bool rest = total > 0;   // else the draft covers the target: its own probabilities
  const uint64_t T_ = rest ? total : total_all;
  float u = a.u_sample[s];
  u = u > 0.f ? (u < 0x1.fffffep-1f ? u : 0x1.fffffep-1f) : 0.f;
  const uint64_t part = (uint64_t)(uint32_t)(u * 0x1p31f);
  const uint64_t level = (T_ >> 31) * part + (((T_ & 0x7fffffffull) * part) >> 31);
  const uint64_t x = rest ? up : up_all, m = rest ? mine.rest : mine.all;
  if (tid == 0) sh_token = -1;
  if (x > level && x - m <= level) {
    sh_piece = tid;
    sh_before = x - m;
  }
  __syncthreads();
  if (T_ > 0) {
    float p[kPer], re[kPer];
    const int piece = sh_piece;
    piece_weights<T, VEC>(a, r, piece, p, re);
#pragma unroll
    for (int j = 0; j < kPer; ++j) weight[elem<T, VEC>(j)] = fixed44(rest ? re[j] : p[j]);
    __syncthreads();
    uint64_t own = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) own += weight[tid * kPer + j];
    uint64_t all;
    const uint64_t end = sh_before + block_scan(own, sh, all);
    if (end > level && end - own <= level) {
      uint64_t c = end - own;
      int j = 0;
      for (; j < kPer - 1; ++j) {
        c += weight[tid * kPer + j];
        if (c > level) break;
      }
      sh_token = piece * kPiece + tid * kPer + j;
    }
    __syncthreads();
  }
  for (int t = tid; t <= (r.k > 0 ? r.k : 0); t += kThreads)
    a.tokens[r.q0 + t] = t < r.first ? a.drafted[r.drow + t] : (t == r.first ? sh_token : -1);
  if (tid == 0) a.n_out[s] = r.first + 1;
}

template <typename T>
hipError_t launch(const VerifyArgs& a, hipStream_t s) {
  const int pieces = (a.vocab + kPiece - 1) / kPiece;
  VerifySums* sums = reinterpret_cast<VerifySums*>(a.ws);
  auto ok16 = [](const void* p, int64_t ld) {
    return ((uintptr_t)p & 15) == 0 && (ld * ET<T>::bytes & 15) == 0;
  };
  const dim3 grid((unsigned)pieces, (unsigned)a.n_seqs);
  if (ok16(a.target, a.target_ld) && (!a.draft || ok16(a.draft, a.draft_ld))) {
    hipLaunchKernelGGL((k_verify_sums<T, true>), grid, dim3(kThreads), 0, s, a, sums);
    hipLaunchKernelGGL((k_verify_pick<T, true>), dim3(a.n_seqs), dim3(kThreads), 0, s, a, sums, pieces);
  } else {
    hipLaunchKernelGGL((k_verify_sums<T, false>), grid, dim3(kThreads), 0, s, a, sums);
    hipLaunchKernelGGL((k_verify_pick<T, false>), dim3(a.n_seqs), dim3(kThreads), 0, s, a, sums, pieces);
  }
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace(int32_t n_seqs, int32_t vocab) {
  return (size_t)n_seqs * (size_t)((vocab + kPiece - 1) / kPiece) * sizeof(VerifySums);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  if (a.dtype == LORA_F32) return launch<float>(a, s);
  return a.dtype == LORA_F16 ? launch<f16_t>(a, s) : launch<bf16_t>(a, s);
}

}  // namespace lora
