// Eviction from the cache: which tokens of a sequence and kv head stay, and their way to
// the front of the sequence's pages.
#include <algorithm>

#include "kvtiles.h"

namespace lora {

namespace {

// ---- select ------------------------------------------------------------------------
// The K tokens of largest rank: a weight's bits as a number that grows with it (NaN
// below all others), the first and the latest tokens above all, absent ones last.
__device__ __forceinline__ uint32_t rank_of(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);   // -0: 0
  const uint32_t x = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return w != w ? 1u : x;
}
__device__ __forceinline__ int select_tokens(const SelectArgs& a, int s) {
  return (int)min((int64_t)kv_seq(a.kv, s).end, a.w_ld);
}
// The tokens of one (sequence, head).
struct Ranks {
  const float* w;
  const int32_t *ktab, *vtab;
  int n, sinks, late;   // tokens; the first `sinks` and those from `late` on stay
  bool all;             // every token has pages
};
__device__ __forceinline__ Ranks ranks_of(const SelectArgs& a, int s, int h) {
  const KvView& kv = a.kv;
  Ranks r;
  r.w = a.weights + ((int64_t)s * kv.H + h) * a.w_ld;
  r.ktab = kv.table + ((int64_t)s * 2 * kv.H + h) * kv.nb;
  r.vtab = r.ktab + (int64_t)kv.H * kv.nb;
  r.n = select_tokens(a, s);
  r.sinks = a.sinks;
  r.late = kv_seq(a.kv, s).end - a.recent;
  r.all = true;
  return r;
}
__device__ __forceinline__ bool has_pages(const KvView& kv, const Ranks& r, int b) {
  return (unsigned)r.ktab[b] < (unsigned)kv.n_pages && (unsigned)r.vtab[b] < (unsigned)kv.n_pages;
}
// Ranks of a wave's per * 64 tokens from j0 on (per <= PER), 64 at a time; 0: there is none.
// (Values are selected, not written on a condition: the compiler keeps the array in registers
// and loses such a write.)
template <int PER>
__device__ __forceinline__ void load_weights(const Ranks& r, int j0, int per, float (&w)[PER]) {
  const int lane = threadIdx.x & 63, last = max(r.n - 1, 0);
  const float* at = r.w + j0 + lane;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    if (j0 + i * 64 + 63 < r.n) w[i] = at[i * 64];
    else if (i == 0 || i < per) w[i] = r.w[min(j0 + i * 64 + lane, last)];   // (w_ld is at least 1)
  }
}
template <int PER>
__device__ __forceinline__ void to_ranks(const KvView& kv, const Ranks& r, int j0, int per, const float (&w)[PER],
                                         uint32_t (&x)[PER]) {
  const int lane = threadIdx.x & 63, last = max(r.n - 1, 0);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int a = j0 + i * 64, j = a + lane;
    x[i] = 0u;
    if (i < per) {
      const uint32_t y = rank_of(w[i]);
      x[i] = y;
      // (the first and the latest tokens, and the last ones)
      if (a < r.sinks || a + 63 >= r.late || a + 63 >= r.n) x[i] = j >= r.n ? 0u : (j < r.sinks || j >= r.late ? 0xffffffffu : y);
    }
  }
  if (r.all) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = (int)kv_div(kv, (uint32_t)min(j0 + i * 64 + lane, last));
    const bool ok = (unsigned)r.ktab[b] < (unsigned)kv.n_pages & (unsigned)r.vtab[b] < (unsigned)kv.n_pages;
    x[i] = ok ? x[i] : 0u;
  }
}
template <int PER>
__device__ __forceinline__ void load_ranks(const KvView& kv, const Ranks& r, int j0, int per, uint32_t (&x)[PER]) {
  float w[PER];
  load_weights<PER>(r, j0, per, w);
  to_ranks<PER>(kv, r, j0, per, w, x);
}

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ int wave_min(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x = min(x, __shfl_xor(x, d));
  return x;
}
// Tokens of a head that have pages, by a wave.
__device__ __forceinline__ int count_present(const KvView& kv, const Ranks& r) {
  int c = 0;
  for (int b = threadIdx.x & 63; (int64_t)b * kv.T < r.n; b += 64)
    if (has_pages(kv, r, b)) c += min(kv.T, r.n - b * kv.T);
  return wave_sum(c);
}

__device__ __forceinline__ int lanes_below(unsigned long long m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Whether the thread, of a block's THREADS, finds a page of the sequence's n tokens missing, of
// any head.
template <int THREADS>
__device__ __forceinline__ bool some_absent(const KvView& kv, int s, int n) {
  constexpr int U = 8;   // ids on their way at a time
  const int used = (n + kv.T - 1) / kv.T, ids = 2 * kv.H * kv.nb, step = THREADS % kv.nb;
  const int32_t* tab = kv.table + (int64_t)s * ids;
  int column = (int)threadIdx.x % kv.nb;
  bool bad = false;
  for (int i0 = threadIdx.x; i0 < ids; i0 += U * THREADS) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = tab[min(i0 + u * THREADS, ids - 1)];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      bad |= i0 + u * THREADS < ids & column < used & (unsigned)id[u] >= (unsigned)kv.n_pages;
      column += step;
      column -= column >= kv.nb ? kv.nb : 0;
    }
  }
  return bad;
}

// What a block finds out in LDS.
template <int THREADS, int BINS>
struct SelectShared {
  uint32_t bins[BINS];
  alignas(16) uint32_t key[THREADS];   // ranks that begin alike, where they are few, and their tokens
  alignas(16) int index[THREADS];
  int part[THREADS / 64], part2[THREADS / 64];
  uint32_t found[3];
  int last;
  uint32_t fill;
};
// The last rank that stays: all larger ones do, of the equal ones those of tokens up to `last`.
struct Border {
  uint32_t rank;
  int last;
};
// The bin, from the top, in which the need-th of the ranks in sh.bins lies; need becomes what
// that bin has to give, `count` what it has.  No wave reads sh.bins after the last barrier here:
// another one may be clearing them by then.
template <int NB, int THREADS, int BINS>
__device__ __forceinline__ uint32_t find_bin(SelectShared<THREADS, BINS>& sh, uint32_t& need, uint32_t& count) {
  constexpr int W = THREADS / 64, EACH = NB > THREADS ? NB / THREADS : 1;
  static_assert(NB <= BINS && (NB % THREADS == 0 || THREADS % NB == 0), "bins divide over the threads");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int low = NB - (tid + 1) * EACH;   // the thread's bins: low .. low + EACH - 1, the top one first
  uint32_t bin[EACH], own = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) own += bin[i] = low >= 0 ? sh.bins[low + i] : 0u;
  uint32_t sum = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t z = __shfl_up(sum, d);
    if (lane >= d) sum += z;
  }
  if (lane == 63) sh.part[wave] = (int)sum;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) sum += w < wave ? (uint32_t)sh.part[w] : 0u;
  if (sum >= need && sum - own < need) {   // one thread
    uint32_t before = sum - own, at = low, left = need, has = own;
#pragma unroll
    for (int i = EACH - 1; i >= 0; --i) {
      const bool here = before < need && before + bin[i] >= need;
      at = here ? low + i : at;
      left = here ? need - before : left;
      has = here ? bin[i] : has;
      before += bin[i];
    }
    sh.found[0] = at;
    sh.found[1] = left;
    sh.found[2] = has;
  }
  __syncthreads();
  need = sh.found[1];
  count = sh.found[2];
  return sh.found[0];
}
// Of ranks that begin with `prefix` down to bit `shift` the border, `need` of them above or
// at it: the ranks that each(f) gives f(rank, token) for, in any order.  `count` of them.  What
// sh.bins had may be gone from the call on.
template <int THREADS, int BINS, typename Each>
__device__ __forceinline__ Border border_of(SelectShared<THREADS, BINS>& sh, uint32_t prefix, int shift, uint32_t need,
                                            uint32_t count, Each each) {
  const int tid = threadIdx.x;
  while (count > THREADS && shift > 0) {
    // 11 bits at a time, the last ones together with 0s
    const int next = max(shift - 11, 0), less = 11 - (shift - next);
    for (int i = tid; i < 2048; i += THREADS) sh.bins[i] = 0;
    __syncthreads();
    each([&](uint32_t x, int) {
      if (((uint64_t)x >> shift) == ((uint64_t)prefix >> shift)) atomicAdd(&sh.bins[(x >> next << less) & 2047u], 1u);
    });
    __syncthreads();
    prefix |= find_bin<2048>(sh, need, count) >> less << next;
    shift = next;
  }
  if (count > THREADS) {   // equal ranks: the need-th token of them, bit by bit
    int last = 0;
    for (int bit = 30; bit >= 0; --bit) {
      int c = 0;
      each([&](uint32_t x, int j) { c += x == prefix && j < (last | 1 << bit); });
      c = wave_sum(c);
      if ((tid & 63) == 0) sh.part[tid >> 6] = c;
      __syncthreads();
      c = 0;
#pragma unroll
      for (int w = 0; w < THREADS / 64; ++w) c += sh.part[w];
      __syncthreads();
      if ((uint32_t)c < need) last |= 1 << bit;
    }
    return Border{prefix, last};   // fewer than `need` lie before it
  }
  if (tid == 0) sh.fill = 0;
  if (tid >= (int)count && tid < (int)((count + 3) & ~3u)) sh.key[tid] = 0;
  __syncthreads();
  each([&](uint32_t x, int j) {
    if (((uint64_t)x >> shift) == ((uint64_t)prefix >> shift)) {
      const uint32_t at = atomicAdd(&sh.fill, 1u);
      sh.key[at] = x;
      sh.index[at] = j;
    }
  });
  __syncthreads();
  if (tid < (int)count) {
    const uint32_t x = sh.key[tid];
    const int j = sh.index[tid];
    uint32_t before = 0;
#pragma unroll 2
    for (uint32_t i = 0; i < count; i += 4) {
      const u32x4 y = *reinterpret_cast<const u32x4*>(sh.key + i), k = *reinterpret_cast<const u32x4*>(sh.index + i);
#pragma unroll
      for (int e = 0; e < 4; ++e) before += y[e] > x || (y[e] == x && (int)k[e] < j);
    }
    if (before == need - 1) {   // one thread
      sh.found[0] = x;
      sh.last = j;
    }
  }
  __syncthreads();
  return Border{sh.found[0], sh.last};
}
__device__ __forceinline__ bool stays(const Border& b, uint32_t x, int j) {
  return x > b.rank || (x == b.rank && j <= b.last);
}
// The tokens of a block's waves (per * 64 each, from j0 + wave * per * 64 on) that stay, to out,
// which has `room` for that many.
template <int THREADS, int PER, int BINS>
__device__ __forceinline__ void emit(SelectShared<THREADS, BINS>& sh, const Border& b, int j0, int per,
                                     const uint32_t (&x)[PER], int32_t* out, int room) {
  constexpr int W = THREADS / 64;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, first = j0 + wave * per * 64;
  unsigned long long stay[PER];
  int count = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    stay[i] = __ballot(x[i] && stays(b, x[i], first + i * 64 + lane));
    count += __popcll(stay[i]);
  }
  if (lane == 0) sh.part[wave] = count;
  __syncthreads();
  int at = 0;
#pragma unroll
  for (int w = 0; w < W; ++w) at += w < wave ? sh.part[w] : 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int place = at + lanes_below(stay[i]);
    if (((stay[i] >> lane) & 1) && place < room) out[place] = first + i * 64 + lane;
    at += __popcll(stay[i]);
  }
}

// ---- caches of up to 16384 tokens: a block for each ---------------------------------
// A block has a (sequence, head) with its ranks in registers: the 11 leading bits of all of
// them in bins, then the few that share the border's bin compared one with another.  Bound by
// its rounds through LDS (about a dozen barriers): the fewest waves that hold the ranks wait
// the least for one another.  2048 heads of up to 2048 tokens take 15.1 us with 256 threads
// (with 128 17.8, 512 20.3, 1024 26; a wave by itself for each head 17.6; ranks that wait for
// the page ids 15.7), half of it for the weights and the look for missing pages.
constexpr int kBlockTokens = 16384;

template <int THREADS, int PER>
__global__ __launch_bounds__(THREADS) void k_select(SelectArgs a, const int32_t* __restrict__ counts) {
  constexpr int W = THREADS / 64, BINS = 2048;
  __shared__ SelectShared<THREADS, BINS> sh;
  __shared__ int present[kKvMaxHeads];
  const KvView& kv = a.kv;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  Ranks r = ranks_of(a, s, h);
  const int n = uni(r.n), per = (n + THREADS - 1) / THREADS, first = wave * per * 64;
  r.n = n;
  r.late = uni(r.late);
  int least = n;   // tokens that the head with fewest has
  uint32_t x[PER];
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < per && x[i]) f(x[i], first + i * 64 + lane);
  };
  auto clear = [&] {
    for (int i = tid; i < BINS; i += THREADS) sh.bins[i] = 0;
    __syncthreads();
  };
  auto to_bins = [&] { each([&](uint32_t y, int) { atomicAdd(&sh.bins[y >> 21], 1u); }); };
  float w[PER];
  load_weights<PER>(r, first, per, w);
  if (!counts) {
    // the ranks go to their bins as if all pages were there, while the ids are on their way
    const bool bad = some_absent<THREADS>(kv, s, n);
    clear();
    to_ranks<PER>(kv, r, first, per, w, x);
    if (n > a.budget) to_bins();
    if (__syncthreads_or(bad)) {
      for (int o = wave; o < kv.H; o += W) {
        const int c = count_present(kv, ranks_of(a, s, o));
        if (lane == 0) present[o] = c;
      }
      __syncthreads();
      for (int o = lane; o < kv.H; o += 64) least = min(least, present[o]);
      least = wave_min(least);
      r.all = present[h] == n;
    }
  } else {
    for (int o = lane; o < kv.H; o += 64) least = min(least, counts[(int64_t)s * kv.H + o]);
    least = wave_min(least);
    r.all = counts[(int64_t)s * kv.H + h] == n;
    to_ranks<PER>(kv, r, first, per, w, x);
  }
  const int K = min(a.budget, uni(least));
  if (h == 0 && tid == 0) a.n_keep[s] = K;
  if (K == 0) return;
  int32_t* out = a.keep + ((int64_t)s * kv.H + h) * a.keep_ld;
  if (K == n) {   // all of them
    for (int j = tid; j < n; j += THREADS) out[j] = j;
    return;
  }
  if (counts || !r.all || n <= a.budget) {   // there are no bins yet, or not of these ranks
    if (!r.all) to_ranks<PER>(kv, r, first, per, w, x);
    __syncthreads();
    clear();
    to_bins();
    __syncthreads();
  }
  uint32_t need = (uint32_t)K, count;
  const uint32_t bin = find_bin<BINS>(sh, need, count);
  const Border b = border_of(sh, bin << 21, 21, need, count, each);
  emit(sh, b, 0, per, x, out, K);
}

// Tokens of every (sequence, head) that have pages.
__global__ __launch_bounds__(64) void k_select_count(SelectArgs a, int32_t* __restrict__ counts) {
  const int h = blockIdx.x, s = blockIdx.y, c = count_present(a.kv, ranks_of(a, s, h));
  if (threadIdx.x == 0) counts[(int64_t)s * a.kv.H + h] = c;
}

// ---- long caches: three launches over chunks of them -------------------------------
// 1: a chunk's ranks in bins (12 bits) and its present tokens; 2: every block adds up the
// chunks' bins, finds the border's bin and leaves its own ranks of that bin in one list; 3: every
// block finds the border among these and writes the tokens of its chunk that stay.  Two sequences
// of 100001 and 131071 tokens, 8 heads, to 16384 take 26 us (one block a head 161; chunks of
// 4096 30): 7, 9 and 10 of the launches, none of which moves more than 13 MB.
constexpr int kChunk = 8192, kLongThreads = 512, kLongPer = kChunk / kLongThreads, kLongBins = 4096;
// Ranks of the border's bin (an eighth of an octave) that have a place in the list.  With more,
// every block of the third launch reads its whole head again for each pass: a second one and a third
// for ranks that lie close, a pass for each bit of a token's number too where they are equal.  4096 holds
// the bins of 131071 log-normal weights with a sigma of 2 (1700 to 3100).  8 heads of them to 65536
// take 26 us with sigma 2, 193 with 1 or 0.5; to 16384 25 to 26 with each, but 2.04 ms if all
// weights are equal or most are 0.
constexpr int kListed = 4096;

struct ChunkInfo {
  int32_t present;   // tokens with pages
  int32_t above;     // ranks above the border's bin, and in it (from the second launch)
  int32_t in;
  int32_t pad;
};
// The workspace of a (sequence, head).
struct LongSpace {
  ChunkInfo* info;       // [chunks]
  uint2* list;           // [kListed] rank, token
  uint16_t* bins;        // [chunks][kLongBins]
  static __host__ __device__ size_t bytes(int chunks) {
    return (size_t)chunks * (sizeof(ChunkInfo) + kLongBins * sizeof(uint16_t)) + kListed * sizeof(uint2);
  }
  __device__ LongSpace(char* ws, int64_t i, int chunks) {
    ws += i * bytes(chunks);
    info = reinterpret_cast<ChunkInfo*>(ws);
    list = reinterpret_cast<uint2*>(ws + chunks * sizeof(ChunkInfo));
    bins = reinterpret_cast<uint16_t*>(list + kListed);
  }
};
using LongShared = SelectShared<kLongThreads, kLongBins>;

// Tokens that stay, from the chunks' counts of all heads, and whether the head's are all there.
__device__ __forceinline__ int long_budget(const SelectArgs& a, int s, int h, int chunks, Ranks& r, int* sh) {
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, used = (r.n + kChunk - 1) / kChunk;
  int least = r.n;
  for (int o = wave; o < kv.H; o += kLongThreads / 64) {
    const LongSpace sp(a.ws, (int64_t)s * kv.H + o, chunks);
    int c = 0;
    for (int i = lane; i < used; i += 64) c += sp.info[i].present;
    c = wave_sum(c);
    least = min(least, c);
    if (o == h && lane == 0) sh[kLongThreads / 64] = c;
  }
  if (lane == 0) sh[wave] = least;
  __syncthreads();
  for (int w = 0; w < kLongThreads / 64; ++w) least = min(least, sh[w]);
  r.all = sh[kLongThreads / 64] == r.n;
  return min(a.budget, least);
}

__global__ __launch_bounds__(kLongThreads) void k_select_bins(SelectArgs a, int chunks) {
  __shared__ uint32_t bins[kLongBins];
  __shared__ int part[kLongThreads / 64];
  const int h = blockIdx.x, ch = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, wave = tid >> 6;
  Ranks r = ranks_of(a, s, h);
  const int j0 = ch * kChunk;
  if (j0 >= r.n) return;
  uint32_t x[kLongPer];
  for (int i = tid; i < kLongBins; i += kLongThreads) bins[i] = 0;
  load_ranks<kLongPer>(a.kv, r, j0 + wave * kLongPer * 64, kLongPer, x);
  bool bad = false;
  for (int b = (int)kv_div(a.kv, (uint32_t)j0) + tid; b * a.kv.T < min(r.n, j0 + kChunk); b += kLongThreads) bad |= !has_pages(a.kv, r, b);
  if (__syncthreads_or(bad)) {
    r.all = false;
    load_ranks<kLongPer>(a.kv, r, j0 + wave * kLongPer * 64, kLongPer, x);
  }
  int c = 0;
#pragma unroll
  for (int i = 0; i < kLongPer; ++i)
    if (x[i]) {
      atomicAdd(&bins[x[i] >> 20], 1u);
      ++c;
    }
  c = wave_sum(c);
  if ((tid & 63) == 0) part[wave] = c;
  __syncthreads();
  const LongSpace sp(a.ws, (int64_t)s * a.kv.H + h, chunks);
  for (int i = tid; i < kLongBins / 2; i += kLongThreads)
    reinterpret_cast<uint32_t*>(sp.bins + (int64_t)ch * kLongBins)[i] = bins[2 * i] | bins[2 * i + 1] << 16;
  if (tid == 0) {
    c = 0;
    for (int w = 0; w < kLongThreads / 64; ++w) c += part[w];
    sp.info[ch].present = c;
  }
}

__global__ __launch_bounds__(kLongThreads) void k_select_list(SelectArgs a, int chunks) {
  __shared__ LongShared sh;
  __shared__ int counts[kLongThreads / 64 + 1];
  const int h = blockIdx.x, ch = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Ranks r = ranks_of(a, s, h);
  const int j0 = ch * kChunk;
  if (ch == 0 && h == 0 && r.n == 0 && tid == 0) a.n_keep[s] = 0;
  if (j0 >= r.n) return;
  float wt[kLongPer];
  load_weights<kLongPer>(r, j0 + wave * kLongPer * 64, kLongPer, wt);
  const LongSpace sp(a.ws, (int64_t)s * a.kv.H + h, chunks);
  const int used = (r.n + kChunk - 1) / kChunk;
  // thread t adds up the bins 8 t .. 8 t + 7
  constexpr int PER = kLongBins / kLongThreads;
  static_assert(PER == 8, "16 bytes a thread");
  constexpr int AHEAD = 8;
  uint4 v[AHEAD];
  auto bins_from = [&](int i0) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) v[i] = ld16(sp.bins + (int64_t)min(i0 + i, used - 1) * kLongBins + tid * PER);
  };
  bins_from(0);
  const int K = long_budget(a, s, h, chunks, r, counts);
  if (ch == 0 && h == 0 && tid == 0) a.n_keep[s] = K;
  if (K == 0 || K == r.n) return;
  uint32_t sum[PER] = {}, earlier[PER] = {};   // of all chunks, of those before this one
  for (int i0 = 0; i0 < used; i0 += AHEAD) {
    if (i0 > 0) bins_from(i0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      const uint32_t in = i0 + i < used ? 0xffffu : 0u, before = i0 + i < ch ? 0xffffu : 0u;
#pragma unroll
      for (int j = 0; j < PER; ++j) {
        const uint32_t c = w[j / 2] >> (16 * (j & 1));
        sum[j] += c & in;
        earlier[j] += c & before;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) sh.bins[tid * PER + j] = sum[j];
  __syncthreads();
  uint32_t x[kLongPer];
  to_ranks<kLongPer>(a.kv, r, j0 + wave * kLongPer * 64, kLongPer, wt, x);
  uint32_t need = (uint32_t)K, count;
  const uint32_t bin = find_bin<kLongBins>(sh, need, count);
  if (tid == (int)bin / PER) {   // the list's places before this chunk's
    uint32_t c = 0;
#pragma unroll
    for (int j = 0; j < PER; ++j) c = j == (int)bin % PER ? earlier[j] : c;
    sh.last = (int)c;
  }
  int above = 0, in = 0;
#pragma unroll
  for (int i = 0; i < kLongPer; ++i) {
    above += __popcll(__ballot(x[i] >> 20 > bin));
    in += __popcll(__ballot(x[i] >> 20 == bin && x[i]));
  }
  if (lane == 0) {
    sh.part[wave] = in;
    sh.part2[wave] = above;
  }
  __syncthreads();
  int at = sh.last;
  for (int w = 0; w < wave; ++w) at += sh.part[w];
#pragma unroll
  for (int i = 0; i < kLongPer; ++i) {
    const bool mine = x[i] >> 20 == bin && x[i];
    const unsigned long long m = __ballot(mine);
    const int place = at + __popcll(m & ((1ull << lane) - 1));
    if (mine && place < kListed) sp.list[place] = uint2{x[i], (uint32_t)(j0 + (wave * kLongPer + i) * 64 + lane)};
    at += __popcll(m);
  }
  if (tid == 0) {
    in = above = 0;
    for (int w = 0; w < kLongThreads / 64; ++w) {
      in += sh.part[w];
      above += sh.part2[w];
    }
    sp.info[ch].above = above;
    sp.info[ch].in = in;
  }
}

__global__ __launch_bounds__(kLongThreads) void k_select_long(SelectArgs a, int chunks) {
  __shared__ LongShared sh;
  __shared__ int counts[kLongThreads / 64 + 1];
  const int h = blockIdx.x, ch = blockIdx.y, s = blockIdx.z, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  Ranks r = ranks_of(a, s, h);
  const int j0 = ch * kChunk;
  if (j0 >= r.n) return;
  const LongSpace sp(a.ws, (int64_t)s * a.kv.H + h, chunks);
  const int used = (r.n + kChunk - 1) / kChunk;
  float wt[kLongPer];
  load_weights<kLongPer>(r, j0 + wave * kLongPer * 64, kLongPer, wt);
  constexpr int LISTED = kListed / kLongThreads;
  uint2 listed[LISTED];   // (asked for ahead of how many there are)
#pragma unroll
  for (int i = 0; i < LISTED; ++i) listed[i] = sp.list[i * kLongThreads + tid];
  int above = 0, in = 0, above_before = 0;
  for (int i = lane; i < used; i += 64) {
    const ChunkInfo c = sp.info[i];
    above += c.above;
    in += c.in;
    if (i < ch) above_before += c.above;
  }
  const int K = long_budget(a, s, h, chunks, r, counts);
  if (K == 0) return;
  int32_t* out = a.keep + ((int64_t)s * a.kv.H + h) * a.keep_ld;
  if (K == r.n) {
    for (int j = j0 + tid; j < min(r.n, j0 + kChunk); j += kLongThreads) out[j] = j;
    return;
  }
  uint32_t x[kLongPer];
  to_ranks<kLongPer>(a.kv, r, j0 + wave * kLongPer * 64, kLongPer, wt, x);
  above = wave_sum(above);
  in = wave_sum(in);
  above_before = wave_sum(above_before);
  const uint32_t need = (uint32_t)(K - above);
  Border b;
  int at = above_before;   // tokens of the chunks before that stay
  auto with = [&](auto each, uint32_t prefix) {
    b = border_of(sh, prefix, 20, need, (uint32_t)in, each);
    int c = 0;
    each([&](uint32_t y, int j) { c += y >> 20 == prefix >> 20 && j < j0 && stays(b, y, j); });
    c = wave_sum(c);
    if (lane == 0) sh.part2[wave] = c;
    __syncthreads();
    for (int w = 0; w < kLongThreads / 64; ++w) at += sh.part2[w];
  };
  const uint32_t prefix = sp.list[0].x >> 20 << 20;
  if (in <= kListed) {
    with([&](auto f) {
#pragma unroll
      for (int i = 0; i < LISTED; ++i)
        if (i * kLongThreads + tid < in) f(listed[i].x, (int)listed[i].y);
    }, prefix);
  } else {   // (ranks that are nearly all alike)
    with([&](auto f) {
      for (int j = tid; j < r.n; j += kLongThreads) {
        if (!r.all && !has_pages(a.kv, r, (int)kv_div(a.kv, (uint32_t)j))) continue;
        f(j < r.sinks || j >= r.late ? 0xffffffffu : rank_of(r.w[j]), j);
      }
    }, prefix);
  }
  emit(sh, b, j0, kLongPer, x, out + at, K - at);
}

// ---- compact -----------------------------------------------------------------------
// Place first + i of a (sequence, head) gets the token at first + keep[i] >= first + i, in
// place.  Both pages' layouts hold 16 bytes of one token (K) or of E tokens (V), so that a
// list that keeps every fifth token reads nearly every line of its pages: the bytes moved
// are fewer than those that memory has to give.
constexpr int64_t kNone = -1;

struct Places {
  int n, first, end;   // entries of the list; position of place 0; tokens with a place in the table
  const int32_t* keep;
  const int32_t* tab;  // K's page ids, then [H * nb] further V's
};
__device__ __forceinline__ Places places_of(const CompactArgs& a, int s, int h) {
  const KvView& kv = a.kv;
  const KvSeq q = kv_seq(kv, s);
  Places p;
  p.end = uni(q.end);
  p.first = a.from_new ? uni(q.base) : 0;
  p.n = (int)min((int64_t)max(uni(a.n_keep[s]), 0), a.keep_ld);
  p.n = min(p.n, p.end - p.first);
  p.keep = a.keep + ((int64_t)s * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_ld;
  p.tab = kv.table + ((int64_t)s * 2 * kv.H + h) * kv.nb;
  return p;
}
// Bytes of the K (which 0) or V of a token in page `page` of the pool: of K its 16 bytes of piece
// 0, of V its element 0.  kNone: it has no page.
template <int E, int D>
__device__ __forceinline__ int64_t token_at(const KvView& kv, int which, int slot, int page) {
  if ((unsigned)page >= (unsigned)kv.n_pages) return kNone;
  return (int64_t)page * kv.page_bytes + (which ? slot / E * (D * 16) + slot % E * (16 / E) : slot * 16);
}
// The scale byte of the token at `at` (K or V) in the pages.
template <int E, int D>
__device__ __forceinline__ int64_t scale_at(const KvView& kv, int which, int64_t at) {
  const int64_t page = at / kv.page_bytes;
  const int in = (int)(at - page * kv.page_bytes);
  return page * kv.T + (which ? in / (D * 16) * E + in % 16 : in / 16);
}

// The list's entries in steps of N positions, resolved once for all of a block's columns:
// slot x stands for position pos0 + x, pos0 a multiple of E.
template <int N>
struct Steps {
  int64_t from[2][N], to[2][N];   // of K and V; from kNone: the place keeps what it has
  int32_t w[N];                   // position that the weight comes from, -1: none
};
// One place of the list on its way: the token's number, then the page ids of both, then what
// the block's waves go by.
__device__ __forceinline__ int number_of(const Places& p, int pos) {
  const int i = pos - p.first, k = p.keep[max(min(i, p.n - 1), 0)];   // (p.n is at least 1)
  return i >= 0 && i < p.n ? k : -1;
}
struct Entry {
  int src, pos;   // from which position to which; src -1: none
  int from[2], to[2];   // page ids
};
__device__ __forceinline__ Entry entry_of(const KvView& kv, const Places& p, int pos, int k) {
  Entry e;
  e.src = k >= 0 && k < p.end - p.first ? p.first + k : -1;
  e.src = e.src >= 0 && pos >= 0 && pos < p.end ? e.src : -1;
  e.pos = pos;
  const int a = (int)kv_div(kv, (uint32_t)max(e.src, 0)), b = (int)kv_div(kv, (uint32_t)(e.src >= 0 ? pos : 0));
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int32_t* tab = p.tab + (which ? (int64_t)kv.H * kv.nb : 0);
    e.from[which] = tab[a];
    e.to[which] = tab[b];
  }
  return e;
}
// Returns whether something moves.
template <int E, int D, int N>
__device__ __forceinline__ bool put(const CompactArgs& a, const Entry& e, int x, Steps<N>& st) {
  const KvView& kv = a.kv;
  const bool move = e.src >= 0 && e.src != e.pos;
  st.w[x] = move && e.src < a.w_ld && e.pos < a.w_ld ? e.src : -1;   // (of lists that do not ascend src may be below)
  const int fs = e.src - (int)kv_div(kv, (uint32_t)max(e.src, 0)) * kv.T, ts = e.pos - (int)kv_div(kv, (uint32_t)max(e.pos, 0)) * kv.T;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const int64_t f = token_at<E, D>(kv, which, fs, e.from[which]), t = token_at<E, D>(kv, which, ts, e.to[which]);
    const bool ok = e.src >= 0 && t != kNone;
    st.from[which][x] = ok ? f : kNone;
    st.to[which][x] = ok ? t : kNone;
  }
  return move;
}

// E tokens' values of an element of V, gathered and in their places: what is in registers
// between the reads and the writes.
template <int E>
struct Gathered {
  using B = typename std::conditional<E == 16, uint8_t, uint16_t>::type;
  uint32_t w[4];
  uint32_t have;   // bits of the E tokens that have one
};
// Group x0 .. x0 + E - 1 of the step's positions, element d.
template <int E, int N>
__device__ __forceinline__ Gathered<E> gather_v(const char* pages, const Steps<N>& st, int x0, int d) {
  using B = typename Gathered<E>::B;
  B v[E];
  Gathered<E> g;
  g.have = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int64_t f = st.from[1][x0 + e];
    v[e] = *reinterpret_cast<const B*>(pages + (f == kNone ? 0 : f) + d * 16);   // (of page 0 where there is none)
    g.have |= (uint32_t)(f != kNone) << e;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) g.w[i] = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) g.w[e * (int)sizeof(B) / 4] |= (uint32_t)v[e] << (e * (int)sizeof(B) % 4 * 8);
  return g;
}
template <int E, int N>
__device__ __forceinline__ void place_v(char* pages, const Steps<N>& st, int x0, int d, const Gathered<E>& g) {
  using B = typename Gathered<E>::B;
  if (g.have == (1u << E) - 1u) {
    *reinterpret_cast<u32x4*>(pages + st.to[1][x0] + d * 16) = u32x4{g.w[0], g.w[1], g.w[2], g.w[3]};
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((g.have >> e) & 1u)
        *reinterpret_cast<B*>(pages + st.to[1][x0 + e] + d * 16) = (B)(g.w[e * (int)sizeof(B) / 4] >> (e * (int)sizeof(B) % 4 * 8));
  }
}

// Lists of up to 65 - E entries (the path of a tree): a block moves everything of a
// (sequence, head).  All is read before anything is written.  Bound by its four dependent
// reads (lengths, list, page ids, tokens): the paths of 64 trees of up to 25 tokens, 32 heads in
// FP8, take 11 us (a wave a column as below 22; reads of places that have nothing too 22).
template <int E, int D>
__global__ __launch_bounds__(256) void k_compact_few(CompactArgs a) {
  constexpr int N = 64, KU = N * (D / E) / 256, VU = N / E * D / 256;
  __shared__ Steps<N> st;
  const KvView& kv = a.kv;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const Places p = places_of(a, s, h);
  const int pos0 = max(p.first, 0) / E * E;
  if (p.n <= 0) return;
  bool moves = false;
  if (tid < N) moves = put<E, D>(a, entry_of(kv, p, pos0 + tid, number_of(p, pos0 + tid)), tid, st);
  if (!__syncthreads_or(moves)) return;
  const int x = tid & 63;
  u32x4 k[KU];
  Gathered<E> v[VU > 0 ? VU : 1];
  uint8_t sc = 0;
  float w = 0.f;
#pragma unroll
  for (int u = 0; u < KU; ++u)
    if (st.from[0][x] != kNone) k[u] = ldv(kv.pages + st.from[0][x] + (int64_t)(u * 4 + (tid >> 6)) * kv.T * 16);
#pragma unroll
  for (int u = 0; u < VU; ++u) {
    const int x0 = uni((u * 256 + tid) / D * E);   // the same for a wave
    v[u].have = 0;
    if (x0 < p.first + p.n - pos0) v[u] = gather_v<E>(kv.pages, st, x0, (u * 256 + tid) % D);
  }
  if (E == 16 && tid < 128 && st.from[tid >> 6][x] != kNone)
    sc = kv.scales[scale_at<E, D>(kv, tid >> 6, st.from[tid >> 6][x])];
  float* weights = a.weights ? a.weights + ((int64_t)s * kv.H + h) * a.w_ld : nullptr;
  if (weights && tid < N && st.w[tid] >= 0) w = weights[st.w[tid]];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < KU; ++u)
    if (st.from[0][x] != kNone) *reinterpret_cast<u32x4*>(kv.pages + st.to[0][x] + (int64_t)(u * 4 + (tid >> 6)) * kv.T * 16) = k[u];
#pragma unroll
  for (int u = 0; u < VU; ++u) place_v<E>(kv.pages, st, (u * 256 + tid) / D * E, (u * 256 + tid) % D, v[u]);
  if (E == 16 && tid < 128 && st.from[tid >> 6][x] != kNone)
    kv.scales[scale_at<E, D>(kv, tid >> 6, st.to[tid >> 6][x])] = sc;
  if (weights && tid < N && st.w[tid] >= 0) weights[pos0 + tid] = w;
}

// Lists of any length.  A wave owns a column (a 16-byte piece of K, 8 elements of V, the
// scale bytes or the weights) of one (sequence, head) and goes through the list in order: what
// it reads for a step lies at or behind what this step writes, and before that only earlier
// steps have written.  The block's waves share the look-up of 256 places, whose numbers and page
// ids are on their way one step ahead.  Bound by HBM's lines: 16 sequences of 4001 to 16000
// tokens, 8 heads in bf16, down to 2048 with their weights take 153 us (places looked up by
// each wave 675, by the block 327, 8 elements of V a wave instead of 64 222, reads that wait
// for no condition 153); where heads are few by the steps, 3 us each: 30000 tokens of 8 heads to
// 4096 63 us (looked up when their step comes, 512 at a time, 72), of one head to 15000 177 (203).
// Tokens read a step ahead of their writes too made these 67 and 199: one loop for all kinds of
// columns waits for all that is on its way.
template <int E, int D>
__global__ __launch_bounds__(256) void k_compact(CompactArgs a, int columns) {
  constexpr int N = 256, KC = D / E, VC = D / 8, U = 4, UV = 16 / E;
  __shared__ Steps<N> steps[2];
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 63, c = blockIdx.x * 4 + uni((int)threadIdx.x >> 6), h = blockIdx.y, s = blockIdx.z;
  const Places p = places_of(a, s, h);
  float* weights = a.weights ? a.weights + ((int64_t)s * kv.H + h) * a.w_ld : nullptr;
  if (p.n <= 0) return;
  const int end = p.first + p.n, tid = threadIdx.x;
  // while a step's tokens move, the next one's page ids and the numbers of the one behind are on their way
  int pos0 = max(p.first, 0) / E * E;
  Entry entry = entry_of(kv, p, pos0 + tid, number_of(p, pos0 + tid));
  int number = number_of(p, pos0 + N + tid);
  for (int i = 0; pos0 < end; pos0 += N, i ^= 1) {
    Steps<N>& st = steps[i];
    const bool moves = put<E, D>(a, entry, tid, st);
    entry = entry_of(kv, p, pos0 + N + tid, number);
    number = number_of(p, pos0 + 2 * N + tid);
    if (__syncthreads_or(moves)) {   // (the other half of `steps` has been read by all when a wave writes there)
      const int n = min(N, end - pos0);
      if (c < KC) {
        const int64_t column = (int64_t)c * kv.T * 16;
        for (int x0 = 0; x0 < n; x0 += 64 * U) {
          u32x4 v[U];
          int64_t f[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            f[u] = x0 + 64 * u < n ? st.from[0][x0 + 64 * u + lane] : kNone;
            v[u] = ldv(kv.pages + (f[u] == kNone ? 0 : f[u]) + column);   // (of page 0 where there is none)
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (f[u] != kNone) *reinterpret_cast<u32x4*>(kv.pages + st.to[0][x0 + 64 * u + lane] + column) = v[u];
        }
      } else if (c < KC + VC) {
        const int d = (c - KC) * 8 + (lane & 7);   // (8 elements are a line of 128 bytes)
        for (int x0 = 0; x0 < n; x0 += 8 * UV * E) {
          Gathered<E> v[UV];
#pragma unroll
          for (int u = 0; u < UV; ++u) v[u] = gather_v<E>(kv.pages, st, x0 + (u * 8 + (lane >> 3)) * E, d);
#pragma unroll
          for (int u = 0; u < UV; ++u) place_v<E>(kv.pages, st, x0 + (u * 8 + (lane >> 3)) * E, d, v[u]);
        }
      } else if (E == 16 && c < KC + VC + 2) {
        const int which = c - KC - VC;
        for (int x = lane; x < n; x += 64) {
          const int64_t f = st.from[which][x];
          uint8_t v = 0;
          if (f != kNone) v = kv.scales[scale_at<E, D>(kv, which, f)];
          if (f != kNone) kv.scales[scale_at<E, D>(kv, which, st.to[which][x])] = v;
        }
      } else if (c < columns) {
        for (int x = lane; x < n; x += 64) {
          const int f = st.w[x];
          float v = 0.f;
          if (f >= 0) v = weights[f];
          if (f >= 0) weights[pos0 + x] = v;
        }
      }
    }
  }
}

template <int E, int D>
hipError_t compact(const CompactArgs& a, hipStream_t s) {
  if (a.keep_ld <= 64 - E + 1) {
    hipLaunchKernelGGL((k_compact_few<E, D>), dim3(a.kv.H, a.kv.n_seqs), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  const int columns = D / E + D / 8 + (E == 16 ? 2 : 0) + (a.weights ? 1 : 0);
  hipLaunchKernelGGL((k_compact<E, D>), dim3((columns + 3) / 4, a.kv.H, a.kv.n_seqs), dim3(256), 0, s, a, columns);
  return hipGetLastError();
}

}  // namespace

// Caches of up to 16384 tokens, as far as the host can tell, are one launch, or two where
// one block would have to look at too many page ids of the other heads.  Many heads go to blocks
// of fewer threads, of which a CU has more at a time: us with 512 / 1024 threads, 2048 heads of 2000 to
// 4000 tokens 33 / 77, of 4100 to 8100 49 / 87, 512 heads of 8200 to 16000 36 / 44; 4 heads of 3000 6.3 /
// 7.3, of 8000 9.2 / 8.4, of 10845 13.7 / 12.0 (in chunks 21).
static int64_t select_most(const KvView& v, int64_t w_ld) { return std::min<int64_t>((int64_t)v.nb * v.T, w_ld); }
static bool counts_apart(const KvView& v) { return (int64_t)2 * v.H * v.nb > 8192; }

size_t select_workspace(int32_t n_seqs, int32_t H, int64_t tokens) {
  const size_t pairs = (size_t)n_seqs * H;
  return std::max(pairs * sizeof(int32_t), tokens > kBlockTokens ? pairs * LongSpace::bytes((int)((tokens + kChunk - 1) / kChunk)) : 0);
}

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  const int64_t most = select_most(a.kv, a.w_ld);
  if (most > kBlockTokens) {
    const int chunks = (int)((most + kChunk - 1) / kChunk);
    const dim3 grid(a.kv.H, chunks, a.kv.n_seqs);
    hipLaunchKernelGGL(k_select_bins, grid, dim3(kLongThreads), 0, s, a, chunks);
    hipLaunchKernelGGL(k_select_list, grid, dim3(kLongThreads), 0, s, a, chunks);
    hipLaunchKernelGGL(k_select_long, grid, dim3(kLongThreads), 0, s, a, chunks);
    return hipGetLastError();
  }
  const dim3 grid(a.kv.H, a.kv.n_seqs);
  int32_t* counts = nullptr;
  if (counts_apart(a.kv)) {
    counts = reinterpret_cast<int32_t*>(a.ws);
    hipLaunchKernelGGL(k_select_count, grid, dim3(64), 0, s, a, counts);
  }
  const bool few = (int64_t)a.kv.H * a.kv.n_seqs <= 256;   // a block a CU
  const auto run = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, a, counts); };
  if (most <= 2048) run(k_select<256, 8>, 256);
  else if (most <= 4096) run(k_select<512, 8>, 512);
  else if (most <= 8192) few ? run(k_select<1024, 8>, 1024) : run(k_select<512, 16>, 512);
  else few ? run(k_select<1024, 16>, 1024) : run(k_select<512, 32>, 512);
  return hipGetLastError();
}

hipError_t launch_compact(const KvTypes& ty, const CompactArgs& a, hipStream_t s) {
  if (ty.kv == LORA_FP8_E4M3) return ty.D == 128 ? compact<16, 128>(a, s) : compact<16, 64>(a, s);
  return ty.D == 128 ? compact<8, 128>(a, s) : compact<8, 64>(a, s);
}

}  // namespace lora
