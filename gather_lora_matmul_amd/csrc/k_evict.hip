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
  if ((b & 0x7fffffffu) > 0x7f800000u) return 1u;
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
struct Ranks {
  const float* w;
  const int32_t *ktab, *vtab;
  int n, sinks, late;   // tokens; the first `sinks` and those from `late` on stay
  bool all;             // every token has pages
  __device__ uint32_t of(const KvView& kv, int j, float x) const {
    if (!all) {
      const int b = (int)kv_div(kv, (uint32_t)j);
      if ((unsigned)ktab[b] >= (unsigned)kv.n_pages || (unsigned)vtab[b] >= (unsigned)kv.n_pages) return 0u;
    }
    return j < sinks || j >= late ? 0xffffffffu : rank_of(x);
  }
};
__device__ __forceinline__ int select_tokens(const SelectArgs& a, int s) {
  return (int)min((int64_t)kv_seq(a.kv, s).end, a.w_ld);
}

// Tokens of a (sequence, head) that have pages.
__global__ __launch_bounds__(256) void k_select_count(SelectArgs a, int32_t* __restrict__ counts) {
  const KvView& kv = a.kv;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const int n = select_tokens(a, s);
  const int32_t* ktab = kv.table + ((int64_t)s * 2 * kv.H + h) * kv.nb;
  const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
  int c = 0;
  for (int b = tid; (int64_t)b * kv.T < n; b += 256)
    if ((unsigned)ktab[b] < (unsigned)kv.n_pages && (unsigned)vtab[b] < (unsigned)kv.n_pages) c += min(kv.T, n - b * kv.T);
  __shared__ int part[4];
#pragma unroll
  for (int d = 32; d; d >>= 1) c += __shfl_xor(c, d);
  if ((tid & 63) == 0) part[tid >> 6] = c;
  __syncthreads();
  if (tid == 0) counts[(int64_t)s * kv.H + h] = part[0] + part[1] + part[2] + part[3];
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void k_select(SelectArgs a, const int32_t* __restrict__ counts) {
  constexpr int W = THREADS / 64, BINS = 2048;
  __shared__ uint32_t bins[BINS];
  __shared__ uint32_t part[W], part2[W];
  __shared__ uint32_t found[2];
  const KvView& kv = a.kv;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n = select_tokens(a, s);
  int least = n;   // present tokens of the head that has fewest
  for (int i = tid; i < kv.H; i += THREADS) least = min(least, counts[(int64_t)s * kv.H + i]);
#pragma unroll
  for (int d = 32; d; d >>= 1) least = min(least, __shfl_xor(least, d));
  if (lane == 0) part[wave] = (uint32_t)least;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < W; ++w) least = min(least, (int)part[w]);
  __syncthreads();
  const int K = min(a.budget, least);
  if (h == 0 && tid == 0) a.n_keep[s] = K;
  Ranks r;
  r.w = a.weights + ((int64_t)s * kv.H + h) * a.w_ld;
  r.ktab = kv.table + ((int64_t)s * 2 * kv.H + h) * kv.nb;
  r.vtab = r.ktab + (int64_t)kv.H * kv.nb;
  r.n = n;
  r.sinks = a.sinks;
  r.late = kv_seq(a.kv, s).end - a.recent;
  r.all = counts[(int64_t)s * kv.H + h] == n;
  // the rank of the last token that stays, 11, 11 and 10 bits at a time
  uint32_t prefix = 0, need = (uint32_t)K;   // of the ranks that begin like prefix, need stay
  if (K > 0)
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0), nb = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < nb; i += THREADS) bins[i] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += THREADS) {
        const uint32_t x = r.of(kv, j, r.w[j]);
        const bool in = pass == 0 || (pass == 1 ? x >> 21 == prefix >> 21 : x >> 10 == prefix >> 10);
        if (in) atomicAdd(&bins[(x >> shift) & (uint32_t)(nb - 1)], 1u);
      }
      __syncthreads();
      // bins from the top: thread t has `each` of them
      const int each = nb / THREADS > 0 ? nb / THREADS : 1;
      uint32_t own = 0;
      const int top = nb - 1 - tid * each;
      if (top >= 0)
        for (int i = 0; i < each; ++i) own += bins[top - i];
      uint32_t sum = own;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t z = __shfl_up(sum, d);
        if (lane >= d) sum += z;
      }
      if (lane == 63) part[wave] = sum;
      __syncthreads();
      for (int w = 0; w < wave; ++w) sum += part[w];
      if (sum >= need && sum - own < need) {   // one thread
        uint32_t before = sum - own;
        int i = 0;
        while (before + bins[top - i] < need) before += bins[top - i++];
        found[0] = (uint32_t)(top - i);
        found[1] = need - before;
      }
      __syncthreads();
      prefix |= found[0] << shift;
      need = found[1];
      __syncthreads();
    }
  // the list: every wave an equal run of tokens, those of larger rank and the first of the
  // equal ones
  const int each = (n + THREADS - 1) / THREADS * 64, j0 = min(wave * each, n), j1 = min(j0 + each, n);
  uint32_t more = 0, same = 0;
  if (K > 0)
    for (int j = j0; j < j1; j += 64) {
      const uint32_t x = j + lane < j1 ? r.of(kv, j + lane, r.w[j + lane]) : 0u;
      more += (uint32_t)__popcll(__ballot(j + lane < j1 && x > prefix));
      same += (uint32_t)__popcll(__ballot(j + lane < j1 && x == prefix));
    }
  if (lane == 0) {
    part[wave] = more;
    part2[wave] = same;
  }
  __syncthreads();
  uint32_t at = 0, equal = 0;
  for (int w = 0; w < wave; ++w) {
    at += part[w];
    equal += part2[w];
  }
  at += min(equal, need);
  int32_t* out = a.keep + ((int64_t)s * kv.H + h) * a.keep_ld;
  if (K > 0)
    for (int j = j0; j < j1; j += 64) {
      const bool in = j + lane < j1;
      const uint32_t x = in ? r.of(kv, j + lane, r.w[j + lane]) : 0u;
      const unsigned long long below = (1ull << lane) - 1, eq = __ballot(in && x == prefix);
      const bool stay = in && (x > prefix || (x == prefix && equal + (uint32_t)__popcll(eq & below) < need));
      const unsigned long long st = __ballot(stay);
      if (stay) out[at + (uint32_t)__popcll(st & below)] = j + lane;
      at += (uint32_t)__popcll(st);
      equal += (uint32_t)__popcll(eq);
    }
}

// ---- compact -----------------------------------------------------------------------
// Place i of a (sequence, head) gets token keep[i] >= i, in place.  A wave owns a column (a
// 16-byte piece of K, 16 elements of V, the scale bytes or the weights) of one (sequence,
// head) and goes through the list in order: what it reads for a step lies at or behind what
// this step writes, and before that only earlier steps have written.
struct Places {
  int n, first, end;   // entries of the list; position of place 0; tokens with a place in the table
  const int32_t* keep;
  const int32_t* tab;
};
// Page and slot of a position; false: none.
__device__ __forceinline__ bool page_of(const KvView& kv, const int32_t* tab, int pos, int end, int& page, int& slot) {
  if (pos < 0 || pos >= end) return false;
  const int b = (int)kv_div(kv, (uint32_t)pos);
  slot = pos - b * kv.T;
  page = tab[b];
  return (unsigned)page < (unsigned)kv.n_pages;
}
__device__ __forceinline__ Places places_of(const CompactArgs& a, int s, int h, int which) {
  const KvView& kv = a.kv;
  const KvSeq q = kv_seq(kv, s);
  Places p;
  p.end = uni(q.end);
  p.first = a.from_new ? uni(q.base) : 0;
  p.n = (int)min((int64_t)max(uni(a.n_keep[s]), 0), a.keep_ld);
  p.n = min(p.n, p.end - p.first);
  p.keep = a.keep + ((int64_t)s * a.keep_heads + (a.keep_heads > 1 ? h : 0)) * a.keep_ld;
  p.tab = kv.table + (((int64_t)s * 2 + which) * kv.H + h) * kv.nb;
  return p;
}
// The position that place i takes from; -1: none.
__device__ __forceinline__ int source_of(const Places& p, int i) {
  const int k = i < p.n ? p.keep[i] : -1;
  return k >= 0 && k < p.end - p.first ? p.first + k : -1;
}

template <typename V>
__device__ __forceinline__ void move_units(const KvView& kv, const Places& p, int lane, char* base, int64_t page_bytes,
                                           int64_t column) {   // one unit V a token, at page, column + slot sizeof(V)
  for (int i0 = 0; i0 < p.n; i0 += 64) {
    const int i = i0 + lane, src = source_of(p, i), dst = p.first + i;
    int sp = 0, ss = 0, dp = 0, ds = 0;
    const bool ok = i < p.n && src != dst && page_of(kv, p.tab, src, p.end, sp, ss) && page_of(kv, p.tab, dst, p.end, dp, ds);
    V v{};
    if (ok) v = *reinterpret_cast<const V*>(base + sp * page_bytes + column + (int64_t)ss * sizeof(V));
    if (ok) *reinterpret_cast<V*>(base + dp * page_bytes + column + (int64_t)ds * sizeof(V)) = v;
  }
}

template <int E, int D>
__device__ __forceinline__ void move_v(const KvView& kv, const Places& p, int lane, int column) {
  using B = typename std::conditional<E == 16, uint8_t, uint16_t>::type;
  const int d = column * 16 + (lane & 15);
  // four groups of E places at a time, aligned in the page
  for (int pos0 = p.first / E * E; pos0 < p.first + p.n; pos0 += 4 * E) {
    const int g0 = pos0 + (lane >> 4) * E;
    int dp = 0, ds = 0;
    const bool there = g0 < p.first + p.n && page_of(kv, p.tab, g0, p.end, dp, ds);
    B v[E];
    uint32_t have = 0, moved = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = g0 + e - p.first, src = there && i >= 0 ? source_of(p, i) : -1;
      int sp = 0, ss = 0;
      v[e] = 0;
      if (src >= 0 && page_of(kv, p.tab, src, p.end, sp, ss)) {
        v[e] = *reinterpret_cast<const B*>(kv.pages + (int64_t)sp * kv.page_bytes + ((int64_t)(ss / E) * D + d) * 16 +
                                           (ss % E) * sizeof(B));
        have |= 1u << e;
        moved |= (uint32_t)(src != g0 + e) << e;
      }
    }
    char* dst = kv.pages + (int64_t)dp * kv.page_bytes + ((int64_t)(ds / E) * D + d) * 16;
    if (have == (1u << E) - 1u && moved) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < E; ++e) w[e * (int)sizeof(B) / 4] |= (uint32_t)v[e] << (e * (int)sizeof(B) % 4 * 8);
      *reinterpret_cast<u32x4*>(dst) = u32x4{w[0], w[1], w[2], w[3]};
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if ((moved >> e) & 1u) reinterpret_cast<B*>(dst)[e] = v[e];
    }
  }
}

template <int E, int D>
__global__ __launch_bounds__(256) void k_compact(CompactArgs a, int columns) {
  constexpr int KC = D / E, VC = D / 16;
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 63, c = blockIdx.x * 4 + uni((int)threadIdx.x >> 6), h = blockIdx.y, s = blockIdx.z;
  if (c >= columns) return;
  if (c < KC) {
    const Places p = places_of(a, s, h, 0);
    move_units<u32x4>(kv, p, lane, kv.pages, kv.page_bytes, (int64_t)c * kv.T * 16);
  } else if (c < KC + VC) {
    const Places p = places_of(a, s, h, 1);
    move_v<E, D>(kv, p, lane, c - KC);
  } else if (E == 16 && c < KC + VC + 2) {
    const Places p = places_of(a, s, h, c - KC - VC);
    move_units<uint8_t>(kv, p, lane, reinterpret_cast<char*>(kv.scales), kv.T, 0);
  } else {
    const Places p = places_of(a, s, h, 0);
    float* w = a.weights + ((int64_t)s * kv.H + h) * a.w_ld;
    for (int i0 = 0; i0 < p.n; i0 += 64) {
      const int i = i0 + lane, src = source_of(p, i), dst = p.first + i;
      const bool ok = src >= 0 && src < a.w_ld && dst >= 0;
      const float x = ok ? w[src] : 0.f;
      if (ok && src != dst) w[dst] = x;
    }
  }
}

template <int E, int D>
hipError_t compact(const CompactArgs& a, hipStream_t s) {
  const int columns = D / E + D / 16 + (E == 16 ? 2 : 0) + (a.weights ? 1 : 0);
  hipLaunchKernelGGL((k_compact<E, D>), dim3((columns + 3) / 4, a.kv.H, a.kv.n_seqs), dim3(256), 0, s, a, columns);
  return hipGetLastError();
}

}  // namespace

size_t select_workspace(int32_t n_seqs, int32_t H) { return (size_t)n_seqs * H * sizeof(int32_t); }

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  int32_t* counts = reinterpret_cast<int32_t*>(a.ws);
  const dim3 grid(a.kv.H, a.kv.n_seqs);
  hipLaunchKernelGGL(k_select_count, grid, dim3(256), 0, s, a, counts);
  if ((int64_t)a.kv.nb * a.kv.T <= 8192) hipLaunchKernelGGL((k_select<256>), grid, dim3(256), 0, s, a, counts);
  else hipLaunchKernelGGL((k_select<1024>), grid, dim3(1024), 0, s, a, counts);
  return hipGetLastError();
}

hipError_t launch_compact(const KvTypes& ty, const CompactArgs& a, hipStream_t s) {
  if (ty.kv == LORA_FP8_E4M3) return ty.D == 128 ? compact<16, 128>(a, s) : compact<16, 64>(a, s);
  return ty.D == 128 ? compact<8, 128>(a, s) : compact<8, 64>(a, s);
}

}  // namespace lora
