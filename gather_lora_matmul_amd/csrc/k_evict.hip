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
// Bytes of a token's K (which 0) or V rows in the pool's pages: of K its 16 bytes of piece
// 0, of V its element 0.  kNone: it has no page.
template <int E, int D>
__device__ __forceinline__ int64_t token_at(const KvView& kv, const Places& p, int which, int pos) {
  if (pos < 0 || pos >= p.end) return kNone;
  const int b = (int)kv_div(kv, (uint32_t)pos), slot = pos - b * kv.T;
  const int page = p.tab[(which ? (int64_t)kv.H * kv.nb : 0) + b];
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
template <int E, int D, int N, int THREADS>
__device__ __forceinline__ bool resolve(const CompactArgs& a, const Places& p, int pos0, Steps<N>& st) {
  bool moves = false;
  for (int x = threadIdx.x; x < N; x += THREADS) {
    const int pos = pos0 + x, i = pos - p.first;
    const int k = i >= 0 && i < p.n ? p.keep[i] : -1;
    const int src = k >= 0 && k < p.end - p.first ? p.first + k : -1;
    const bool move = src >= 0 && src != pos && pos >= 0;
    moves |= move;
    st.w[x] = move && src < a.w_ld ? src : -1;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const int64_t f = src >= 0 ? token_at<E, D>(a.kv, p, which, src) : kNone;
      const int64_t t = src >= 0 ? token_at<E, D>(a.kv, p, which, pos) : kNone;
      st.from[which][x] = t == kNone ? kNone : f;
      st.to[which][x] = t;
    }
  }
  return __syncthreads_or(moves) != 0;
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
    v[e] = 0;
    if (f != kNone) {
      v[e] = *reinterpret_cast<const B*>(pages + f + d * 16);
      g.have |= 1u << e;
    }
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

// Lists of up to 64 - E entries (the path of a tree): a block moves everything of a
// (sequence, head).  All is read before anything is written.
template <int E, int D>
__global__ __launch_bounds__(256) void k_compact_few(CompactArgs a) {
  constexpr int N = 64, KU = N * (D / E) / 256, VU = N / E * D / 256;
  __shared__ Steps<N> st;
  const KvView& kv = a.kv;
  const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const Places p = places_of(a, s, h);
  const int pos0 = max(p.first, 0) / E * E;
  if (p.n <= 0 || !resolve<E, D, N, 256>(a, p, pos0, st)) return;
  const int x = tid & 63;
  u32x4 k[KU];
  Gathered<E> v[VU > 0 ? VU : 1];
  uint8_t sc[2] = {0, 0};
  float w = 0.f;
#pragma unroll
  for (int u = 0; u < KU; ++u)
    if (st.from[0][x] != kNone) k[u] = ldv(kv.pages + st.from[0][x] + (int64_t)(u * 4 + (tid >> 6)) * kv.T * 16);
#pragma unroll
  for (int u = 0; u < VU; ++u) v[u] = gather_v<E>(kv.pages, st, (u * 256 + tid) / D * E, (u * 256 + tid) % D);
  if (E == 16 && tid < 128 && st.from[tid >> 6][x] != kNone)
    sc[0] = kv.scales[scale_at<E, D>(kv, tid >> 6, st.from[tid >> 6][x])];
  float* weights = a.weights ? a.weights + ((int64_t)s * kv.H + h) * a.w_ld : nullptr;
  if (weights && tid < N && st.w[tid] >= 0) w = weights[st.w[tid]];
  __syncthreads();
#pragma unroll
  for (int u = 0; u < KU; ++u)
    if (st.from[0][x] != kNone) *reinterpret_cast<u32x4*>(kv.pages + st.to[0][x] + (int64_t)(u * 4 + (tid >> 6)) * kv.T * 16) = k[u];
#pragma unroll
  for (int u = 0; u < VU; ++u) place_v<E>(kv.pages, st, (u * 256 + tid) / D * E, (u * 256 + tid) % D, v[u]);
  if (E == 16 && tid < 128 && st.from[tid >> 6][x] != kNone)
    kv.scales[scale_at<E, D>(kv, tid >> 6, st.to[tid >> 6][x])] = sc[0];
  if (weights && tid < N && st.w[tid] >= 0) weights[pos0 + tid] = w;
}

// Lists of any length.  A wave owns a column (a 16-byte piece of K, 8 elements of V, the
// scale bytes or the weights) of one (sequence, head) and goes through the list in order: what
// it reads for a step lies at or behind what this step writes, and before that only earlier
// steps have written.
template <int E, int D>
__global__ __launch_bounds__(256) void k_compact(CompactArgs a, int columns) {
  constexpr int N = 512, KC = D / E, VC = D / 8, U = 4, UV = 16 / E;
  __shared__ Steps<N> st;
  const KvView& kv = a.kv;
  const int lane = threadIdx.x & 63, c = blockIdx.x * 4 + uni((int)threadIdx.x >> 6), h = blockIdx.y, s = blockIdx.z;
  const Places p = places_of(a, s, h);
  float* weights = a.weights ? a.weights + ((int64_t)s * kv.H + h) * a.w_ld : nullptr;
  const int end = p.first + p.n;
  for (int pos0 = max(p.first, 0) / E * E; pos0 < end; pos0 += N) {
    if (resolve<E, D, N, 256>(a, p, pos0, st)) {
      const int n = min(N, end - pos0);
      if (c < KC) {
        const int64_t column = (int64_t)c * kv.T * 16;
        for (int x0 = 0; x0 < n; x0 += 64 * U) {
          u32x4 v[U];
          int64_t f[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            f[u] = x0 + 64 * u < n ? st.from[0][x0 + 64 * u + lane] : kNone;
            if (f[u] != kNone) v[u] = ldv(kv.pages + f[u] + column);
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
    __syncthreads();   // the step's places have been read
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
