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
// Bound by the reads of one p row and (after a refusal) one q row a sequence.  The
// rows are summed in regions of 512 probabilities (a wave each), a scan of the
// regions' sums finds the one that holds the level, and that one is read again for
// the token.  Enough sequences, or few probabilities, are one launch with a block
// of 16 waves a sequence; else the regions' sums are a launch over the whole chip
// and the scan is a second one.  Measured: one sequence of 4 drafted tokens, 32000
// probabilities, f32, 7.4 us (a launch and three dependent rounds of loads); 128 of
// none to 7, 131071 probabilities, 108 MB, 25.5 us, 4.2 TB/s.
#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

constexpr int kRegion = 512;             // probabilities of a region: 8 a lane
constexpr int kMaxRegions = (1 << 18) / kRegion;

// A weight in whole multiples of 2^-44 as hi * 2^22 + lo: two exact products and
// two conversions that round down.  Sums of 512 of them fit 32 bits.
struct Weight {
  uint32_t hi, lo;
};
__device__ __forceinline__ Weight fixed44(float x) {
  const float t = fminf(fmaxf(x, 0.f), 1.f) * 0x1p22f;   // NaN: 0
  Weight w;
  w.hi = (uint32_t)t;
  w.lo = (uint32_t)(__builtin_amdgcn_fractf(t) * 0x1p22f);
  return w;
}
__device__ __forceinline__ uint64_t whole(uint32_t hi, uint32_t lo) { return ((uint64_t)hi << 22) + lo; }

template <typename T>
__device__ __forceinline__ float prob(const void* base, int64_t i) {
  return load_y<T>(base, i);
}

struct VerifySeq {
  int q0, k;        // first row, drafted tokens (-1: no rows)
  int first;        // accepted tokens
  int rows;         // all of the sequence's, which are k + 1 unless its drafts are not there
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
// Every one of the block's THREADS threads calls it.
template <typename T, int THREADS>
__device__ __forceinline__ VerifySeq accept(const VerifyArgs& a, int s) {
  VerifySeq r;
  int b, e;
  rows_of(a, s, b, e);
  r.q0 = b;
  r.rows = e - b;
  r.k = r.rows - 1;
  // each sequence with rows before this one has one row that is no draft's
  r.drow = (int64_t)b;
  for (int i0 = 0; i0 < s; i0 += THREADS) {
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

// Rows of the token that follows the accepted ones: p, and q after a refusal.
struct VerifyRows {
  const char* p;
  const char* q;   // null: nothing to subtract
  int drop;        // token that the draft proposed with certainty, -1: none
};
template <typename T>
__device__ __forceinline__ VerifyRows rows_at(const VerifyArgs& a, const VerifySeq& r) {
  VerifyRows w;
  w.p = reinterpret_cast<const char*>(a.target) + (int64_t)(r.q0 + r.first) * a.target_ld * ET<T>::bytes;
  w.q = nullptr;
  w.drop = -1;
  if (r.first < r.k) {
    if (a.draft) w.q = reinterpret_cast<const char*>(a.draft) + (r.drow + r.first) * a.draft_ld * ET<T>::bytes;
    else w.drop = a.drafted[r.drow + r.first];
  }
  return w;
}

// Eight consecutive probabilities from v on, rows aligned to their elements only
// (16-byte loads need no more here); past the row's end 0.
template <typename T>
__device__ __forceinline__ void load8(const char* row, int v, int vocab, float* f) {
  constexpr int B = 8 * ET<T>::bytes;
  if (v + 8 <= vocab) {
    uint4 u[B / 16];
    __builtin_memcpy(u, row + (int64_t)v * ET<T>::bytes, B);
#pragma unroll
    for (int i = 0; i < B / 16; ++i) unpack16<T>(u[i], f + i * (16 / ET<T>::bytes));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = v + j < vocab ? prob<T>(row, v + j) : 0.f;
  }
}

// The lane's eight differences of a region (SELF: the target's own probabilities).
template <typename T, bool SELF>
__device__ __forceinline__ void region_rest(const VerifyRows& w, int region, int vocab, float* f) {
  const int v = region * kRegion + (threadIdx.x & 63) * 8;
  load8<T>(w.p, v, vocab, f);
  if (SELF) return;
  if (w.q) {
    float q[8];
    load8<T>(w.q, v, vocab, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] -= q[j];
  }
  const int d = w.drop - v;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = j == d ? 0.f : f[j];
}

__device__ __forceinline__ uint32_t wave_add(uint32_t x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ uint64_t region_sum(const float* f) {
  uint32_t hi = 0, lo = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const Weight w = fixed44(f[j]);
    hi += w.hi;
    lo += w.lo;
  }
  return whole(wave_add(hi), wave_add(lo));
}

__device__ __forceinline__ uint64_t wave_scan(uint64_t x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint64_t y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Sums of the regions first, first + step, .. of a sequence's rows, by one wave.
template <typename T, bool SELF>
__device__ __forceinline__ void sum_regions(const VerifyArgs& a, const VerifyRows& w, int first, int step,
                                            int regions, uint64_t* sums) {
  constexpr int U = 2;   // regions on their way at a time
  for (int g = first; g < regions; g += U * step) {
    float f[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g + u * step < regions) region_rest<T, SELF>(w, g + u * step, a.vocab, f[u]);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (g + u * step < regions) {
        const uint64_t x = region_sum(f[u]);
        if ((threadIdx.x & 63) == 0) sums[g + u * step] = x;
      }
  }
}

// From the regions' sums (LDS) to the token, by one wave: total, level, region,
// token.  -2: all weights are 0.
template <typename T, bool SELF>
__device__ __forceinline__ int pick(const VerifyArgs& a, int s, const VerifyRows& w, int regions,
                                    const uint64_t* sums) {
  const int lane = threadIdx.x & 63;
  constexpr int N = kMaxRegions / 64;
  uint64_t own = 0, x[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int g = lane * N + i;
    x[i] = g < regions ? sums[g] : 0;
    own += x[i];
  }
  const uint64_t end = wave_scan(own);
  const uint64_t total = __shfl(end, 63);
  if (total == 0) return -2;
  float u = a.u_sample[s];
  u = u > 0.f ? (u < 0x1.fffffep-1f ? u : 0x1.fffffep-1f) : 0.f;
  const uint64_t part = (uint64_t)(uint32_t)(u * 0x1p31f);
  const uint64_t level = (total >> 31) * part + (((total & 0x7fffffffull) * part) >> 31);
  // the lane, then its region, that pass the level (total > level, so there is one)
  const int src = __builtin_ctzll(__ballot(end > level));
  uint64_t before = end - own;
  int at = N - 1;
#pragma unroll
  for (int i = N - 2; i >= 0; --i) {
    uint64_t upto = end - own;
#pragma unroll
    for (int j = 0; j <= i; ++j) upto += x[j];
    if (upto > level) at = i;
  }
#pragma unroll
  for (int i = 0; i < N - 1; ++i)
    if (i < at) before += x[i];
  const int region = __shfl(lane * N + at, src);
  before = __shfl(before, src);
  float f[8];
  region_rest<T, SELF>(w, region, a.vocab, f);
  uint64_t y[8], sum = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const Weight e = fixed44(f[j]);
    y[j] = whole(e.hi, e.lo);
    sum += y[j];
  }
  const uint64_t up = before + wave_scan(sum);
  const int tl = __builtin_ctzll(__ballot(up > level));
  uint64_t c = up - sum;
  int tok = 7;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    c += y[j];
    if (c > level && tok == 7) tok = j;
  }
  return __shfl(region * kRegion + lane * 8 + tok, tl);
}

// The token and the outputs of one sequence, from the regions' sums in LDS.
template <typename T, int THREADS>
__device__ __forceinline__ void finish(const VerifyArgs& a, int s, const VerifySeq& r, const VerifyRows& w,
                                       int regions, uint64_t* sums, int* sh) {
  const int tid = threadIdx.x, wave = tid >> 6;
  if (wave == 0) {
    const int tok = pick<T, false>(a, s, w, regions, sums);
    if (tid == 0) *sh = tok;
  }
  __syncthreads();
  int tok = *sh;
  if (tok == -2) {   // the draft covers the target: the target's own probabilities
    sum_regions<T, true>(a, w, wave, THREADS / 64, regions, sums);
    __syncthreads();
    if (wave == 0) {
      tok = pick<T, true>(a, s, w, regions, sums);
      if (tid == 0) *sh = tok == -2 ? -1 : tok;
    }
    __syncthreads();
    tok = *sh;
  }
  for (int t = tid; t < r.rows; t += THREADS)
    a.tokens[r.q0 + t] = t < r.first ? a.drafted[r.drow + t] : (t == r.first ? tok : -1);
  if (tid == 0) a.n_out[s] = r.first + 1;
}

// What the first of two launches leaves for the second, ahead of a sequence's sums.
struct VerifyHead {
  VerifySeq r;
  int64_t pad;
};
static_assert(sizeof(VerifyHead) % 8 == 0, "sums follow");
__host__ __device__ inline size_t seq_words(int regions) { return sizeof(VerifyHead) / 8 + (size_t)regions; }

template <typename T>
__global__ __launch_bounds__(1024) void k_verify_one(VerifyArgs a, int regions) {
  __shared__ uint64_t sums[kMaxRegions];
  __shared__ int sh;
  const int s = blockIdx.x, tid = threadIdx.x;
  const VerifySeq r = accept<T, 1024>(a, s);
  if (r.k < 0) {
    if (tid == 0) a.n_out[s] = 0;
    return;
  }
  const VerifyRows w = rows_at<T>(a, r);
  sum_regions<T, false>(a, w, tid >> 6, 16, regions, sums);
  __syncthreads();
  finish<T, 1024>(a, s, r, w, regions, sums, &sh);
}

template <typename T>
__global__ __launch_bounds__(256) void k_verify_sums(VerifyArgs a, uint64_t* __restrict__ ws, int regions) {
  const int s = blockIdx.y, tid = threadIdx.x;
  uint64_t* head = ws + s * seq_words(regions);
  const VerifySeq r = accept<T, 256>(a, s);
  if (blockIdx.x == 0 && tid == 0) reinterpret_cast<VerifyHead*>(head)->r = r;
  if (r.k < 0) return;
  const VerifyRows w = rows_at<T>(a, r);
  sum_regions<T, false>(a, w, blockIdx.x * 4 + (tid >> 6), gridDim.x * 4, regions,
                        head + sizeof(VerifyHead) / 8);
}

template <typename T>
__global__ __launch_bounds__(512) void k_verify_pick(VerifyArgs a, const uint64_t* __restrict__ ws, int regions) {
  __shared__ uint64_t sums[kMaxRegions];
  __shared__ int sh;
  const int s = blockIdx.x, tid = threadIdx.x;
  const uint64_t* head = ws + s * seq_words(regions);
  const VerifySeq r = reinterpret_cast<const VerifyHead*>(head)->r;
  if (tid < regions) sums[tid] = head[sizeof(VerifyHead) / 8 + tid];
  if (r.k < 0) {
    if (tid == 0) a.n_out[s] = 0;
    return;
  }
  __syncthreads();
  finish<T, 512>(a, s, r, rows_at<T>(a, r), regions, sums, &sh);
}

// One launch where a block a sequence is enough to read the rows.  Measured on
// MI355X, us of a call by one launch / by two, by sequences of 4 drafted tokens, f32 with
// the draft's probabilities: 32000 probabilities 7.6 / 7.8 (1), 8.7 / 8.3 (16), 10.7 /
// 12.4 (128); 131071 16.3 / 7.5 (1), 21.8 / 16.6 (64), 28.9 / 26.9 (128), 46.6 / 49.6
// (256); 262144 30.8 / 7.4 (1), 56.2 / 46.1 (128), 83 / 86 (256).
bool one_launch(const VerifyArgs& a) { return a.vocab <= 32768 || a.n_seqs >= 192; }

template <typename T>
hipError_t launch(const VerifyArgs& a, hipStream_t s) {
  const int regions = (a.vocab + kRegion - 1) / kRegion;
  if (one_launch(a)) {
    hipLaunchKernelGGL((k_verify_one<T>), dim3(a.n_seqs), dim3(1024), 0, s, a, regions);
  } else {
    uint64_t* ws = reinterpret_cast<uint64_t*>(a.ws);
    hipLaunchKernelGGL((k_verify_sums<T>), dim3((regions + 7) / 8, a.n_seqs), dim3(256), 0, s, a, ws, regions);
    hipLaunchKernelGGL((k_verify_pick<T>), dim3(a.n_seqs), dim3(512), 0, s, a, ws, regions);
  }
  return hipGetLastError();
}

}  // namespace

size_t verify_workspace(int32_t n_seqs, int32_t vocab) {
  return (size_t)n_seqs * seq_words((vocab + kRegion - 1) / kRegion) * sizeof(uint64_t);
}

hipError_t launch_verify(const VerifyArgs& a, hipStream_t s) {
  if (a.dtype == LORA_F32) return launch<float>(a, s);
  return a.dtype == LORA_F16 ? launch<f16_t>(a, s) : launch<bf16_t>(a, s);
}

}  // namespace lora
