// The attention that cached tokens get from the new ones.
//
//   w_j = decay before_j + sum_i exp(scale q_i . k_j - lse_i)
//
// over the rows i of a kv head (its G query heads times the sequence's new tokens) that
// see token j, with the rows' log-sum-exps as the attention left them: one product, no
// running maximum.  S = Q K^T with the keys as columns: a lane holds scores of one key,
// adds their exponentials up in a register and needs other lanes only at a key's end.
// A key belongs to one wave, so that sums have one order and no atomics.
#include <algorithm>

#include "kvtiles.h"
#include "per_device.h"

namespace lora {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Tiles of KT cached tokens of a (sequence, head), in that order of sequences.
__device__ __forceinline__ int tokens_of(const WeighArgs& a, const KvSeq& q) {
  return (int)min((int64_t)q.end, a.w_ld);
}
// Prefix sums of the sequences' tiles in LDS (and, if wanted, the sequences); returns all.
template <int KT, int THREADS>
__device__ __forceinline__ int tile_sums(const WeighArgs& a, int* pre, KvSeq* seqs = nullptr) {
  const int n = a.kv.n_seqs, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __shared__ int wsum[THREADS / 64];
  int run = 0;
  for (int s0 = 0; s0 < n; s0 += THREADS) {
    const int s = s0 + tid;
    int sum = 0;
    if (s < n) {
      const KvSeq q = kv_seq(a.kv, s);
      if (seqs) seqs[s] = q;
      sum = (tokens_of(a, q) + KT - 1) / KT * a.kv.H;
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int z = __shfl_up(sum, d);
      if (lane >= d) sum += z;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < THREADS / 64; ++w) {
      if (w < wave) sum += wsum[w];
      all += wsum[w];
    }
    if (s < n) pre[s + 1] = run + sum;
    run += all;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  return run;
}
// The sequence of unit u, by every lane.
__device__ __forceinline__ int seq_of(const int* pre, int n, int u) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A (sequence, head) and a tile of it, the same in all lanes.
struct Unit {
  int seq, head, tile;
  int n;   // tokens of the sequence
  KvSeq q;
};
__device__ __forceinline__ void unit_seq(const WeighArgs& a, Unit& u, const KvSeq* seqs) {
  u.q = seqs ? seqs[u.seq] : kv_seq(a.kv, u.seq);
  u.q.q0 = uni(u.q.q0);
  u.q.q_len = uni(u.q.q_len);
  u.q.base = uni(u.q.base);
  u.q.end = uni(u.q.end);
  u.n = tokens_of(a, u.q);
}
template <int KT>
__device__ __forceinline__ Unit unit_of(const WeighArgs& a, const int* pre, int at, const KvSeq* seqs = nullptr) {
  Unit r;
  r.seq = uni(seq_of(pre, a.kv.n_seqs, at));
  unit_seq(a, r, seqs);
  const int tiles = (r.n + KT - 1) / KT, rem = at - pre[r.seq];
  r.head = uni(rem / tiles);
  r.tile = uni((rem - r.head * tiles) * KT);
  return r;
}

// What a token had before, faded; new tokens had nothing.
__device__ __forceinline__ float old_weight(const WeighArgs& a, const Unit& u, int64_t at, int j) {
  return a.before && a.decay > 0.f && j < u.q.base ? a.decay * a.before[at + j] : 0.f;
}

// ---- up to 32 rows a head and sequence ---------------------------------------------
// A wave for itself: KT keys straight to registers, the rows in tiles of 16.  A wave's units are
// neighbours; the next one's keys are asked for ahead of this one's products, the page ids of the
// one after behind them.  Bound by the reads of K, which do not overlap the products in full: what a token
// had before is faded, and in FP8 a scale byte widened, as soon as it is there, and these are the
// last of a unit's loads, so that a wave waits for all of them before it multiplies.  64 sequences
// of 20 to 2048 tokens, 32 heads on 32, in FP8 (268 MB of keys) take 74 us, 3.6 TB/s (with nothing
// from before 69; with 48 keys in three waves a SIMD 75, with 32 in four 74.5), in bf16 128, 4.2 TB/s (123).
// A key's exponentials are 16 a row tile whether its rows are there or not, and every tile
// of rows is read again for each unit: from about 32 rows on the tiles below are faster.  us of rows /
// tiles: bf16, 32 heads on 32, 17 rows over 500 tokens 5.0 / 7.8; 24 over 5000 15.9 / 17.0, 32 16.2 /
// 15.1; four sequences over 2500, 24 rows 25.5 / 23.9 (FP8 19.0 / 21.8), 32 27.1 / 21.4 (20.1 / 19.9),
// 48 34.4 / 26.4 (23.9 / 25.4), 64 41.5 / 23.5 (28.0 / 22.5); 64 heads on 8, 24 rows over 30000 20.0 /
// 19.3, 40 24.8 / 20.9, 64 30.9 / 19.7.
constexpr int kFewRows = 32, kRowsBlocks = 2;   // rows; blocks a CU
template <typename A, typename KV, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(kRowsBlocks, kRowsBlocks))) void k_weigh_rows(WeighArgs a) {
  constexpr bool Q8 = is_quant<KV>();
  constexpr int E = ET<KV>::E, NB = Q8 ? 4 : 2, KT = 16 * NB, NC = D / (4 * E), NQ = D / 32;
  __shared__ int pre[kKvMaxSeqs + 1];
  __shared__ KvSeq seqs[kKvMaxSeqs];
  const KvView& kv = a.kv;
  const int units = tile_sums<KT, 256>(a, pre, seqs);
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int workers = (int)gridDim.x * 4, worker = (int)blockIdx.x * 4 + uni(tid >> 6);
  const int from = (int)((int64_t)units * worker / workers), to = (int)((int64_t)units * (worker + 1) / workers);
  if (from >= to) return;
  const int win = a.window > 0 ? a.window : 0x40000000;
  struct Ids {
    int k[NB], v[NB];
  };
  struct Keys {
    u32x4 k[NB][NC];
    uint32_t scale[NB];
    uint32_t there;   // of block b: bit b
    float old;        // what the lane's token had before
  };
  auto find = [&](const Unit& u) {
    const int32_t* ktab = kv.table + ((int64_t)u.seq * 2 * kv.H + u.head) * kv.nb;
    Ids r;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int blk = (int)kv_div(kv, (uint32_t)(u.tile + 16 * b + col));
      r.k[b] = blk < kv.nb ? ktab[blk] : -1;
      r.v[b] = blk < kv.nb ? ktab[(int64_t)kv.H * kv.nb + blk] : -1;
    }
    return r;
  };
  auto load = [&](const Unit& u, const Ids& id) {
    Keys r;
    r.there = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int t = u.tile + 16 * b + col, slot = t - (int)kv_div(kv, (uint32_t)t) * kv.T;
      const bool ok = (unsigned)id.k[b] < (unsigned)kv.n_pages && (unsigned)id.v[b] < (unsigned)kv.n_pages;
      r.there |= (uint32_t)ok << b;
      const int pg = ok ? id.k[b] : 0, sl = ok ? slot : 0;
      const char* src = kv.pages + (int64_t)pg * kv.page_bytes + (g * kv.T + sl) * 16;
#pragma unroll
      for (int c = 0; c < NC; ++c) r.k[b][c] = ldv(src + c * 4 * kv.T * 16);
      r.scale[b] = Q8 ? kv.scales[(int64_t)pg * kv.T + sl] : 0u;
    }
    const int j = u.tile + 16 * g + col;
    const int64_t at = ((int64_t)u.seq * kv.H + u.head) * a.w_ld;
    r.old = g < NB && j < u.n ? old_weight(a, u, at, j) : 0.f;
    return r;
  };
  auto next = [&](Unit& u) {   // the unit behind u
    u.tile += KT;
    if (u.tile < u.n) return;
    u.tile = 0;
    if (++u.head < kv.H) return;
    u.head = 0;
    do ++u.seq;
    while (pre[u.seq + 1] == pre[u.seq]);
    unit_seq(a, u, seqs);
  };
  u32x4 qf[NQ];
  float ls[4];
  int pos[4];
  auto rows_at = [&](const Unit& u, int r0) {
    const KvSeq& q = u.q;
    const int rows = q.q_len * a.group;
    {
      const int row = min(r0 + col, rows - 1), t = token_of(a, row);
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(q.q0 + t) * a.q_ld +
                            (int64_t)(u.head * a.group + row - t * a.group) * D;
#pragma unroll
      for (int i = 0; i < NQ; ++i) qf[i] = ldv(src + (Q8 ? (4 * (i >> 1) + g) * 16 + (i & 1) * 8 : (4 * i + g) * 8));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = r0 + 4 * g + i, r = min(row, rows - 1), t = token_of(a, r);
      ls[i] = a.lse[(int64_t)(q.q0 + t) * a.n_q_heads + u.head * a.group + r - t * a.group] * kLog2e;
      pos[i] = row < rows ? q.base + t : -0x40000000;
    }
  };
  Unit u = unit_of<KT>(a, pre, from, seqs), un = u;
  Keys key = load(u, find(u));
  Ids idn{};
  bool fresh = true;   // the rows in registers are not u's
  if (from + 1 < to) {
    next(un);
    idn = find(un);
  }
  for (int i = from; i < to; ++i) {
    const bool more = i + 1 < to;
    const int rows = u.q.q_len * a.group;
    if (fresh && rows > 0) rows_at(u, 0);
    Keys kn;
    Unit u2 = un;
    if (more) {
      kn = load(un, idn);
      if (i + 2 < to) {
        next(u2);
        idn = find(u2);
      }
    }
    float sum[NB] = {};
    for (int r0 = 0; r0 < rows; r0 += 16) {
      if (r0 > 0) rows_at(u, r0);
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if constexpr (Q8) {
            s = mfma16<A>(qf[2 * c], fp8_to16<A>(key.k[b][c].x, key.k[b][c].y), s);
            s = mfma16<A>(qf[2 * c + 1], fp8_to16<A>(key.k[b][c].z, key.k[b][c].w), s);
          } else {
            s = mfma16<A>(qf[c], key.k[b][c], s);
          }
        }
        const int j = u.tile + 16 * b + col;
        const float f = Q8 ? a.scale_log2 * __uint_as_float(key.scale[b] << 23) : a.scale_log2;
        float part = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x], f, -ls[x]));
          part += j <= pos[x] && j > pos[x] - win ? p : 0.f;
        }
        sum[b] += part;
      }
    }
    // the lane groups' rows together; group g writes the 16 keys of block g
    float mine = 0.f;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x = sum[b];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      mine = g == b ? x : mine;
    }
    const int j = u.tile + 16 * g + col;
    if (g < NB && j < u.n)
      a.weights[((int64_t)u.seq * kv.H + u.head) * a.w_ld + j] = (key.there >> g) & 1u ? key.old + mine : 0.f;
    if (more) {
      fresh = un.head != u.head || un.seq != u.seq || rows > 16;
      key = kn;
      u = un;
      un = u2;
    }
  }
}

// ---- more rows -------------------------------------------------------------------
// A block's four waves have 64 keys each, in registers for all of the rows, which go
// through LDS in steps of 128 (two slots, one barrier a step).  32 products of 32x32x16 and 32
// exponentials of a wave cost about the same, so they are woven: the last 2048 of 16384
// tokens, 64 heads on 8 in bf16, take 600 to 620 us, 830 to 860 TFLOP/s, at 2.0 to 2.1 GHz
// (its cycles by its time).  (Products of one step, then its exponentials: 640.)
// Rows in LDS, 64 of them in B blocks of 1 KB, each what one load brings: row r is number r / B
// of block r % B, and a block begins 16 bytes further in the banks than the one before.  The
// loads cover whole rows, a product's lanes read all banks alike, and all operands of a lane
// are at constant distances from one address.
template <int D>
struct WeighShared {
  // (64 rows of P pieces in 1 KB blocks: B = P)
  static constexpr int P = D / 8, B = P, STEP = 1024 + 16, HALF = B * STEP;
  static constexpr int RT = 128, SLOT = RT / 64 * HALF;
  __align__(16) char q[2 * SLOT];
  float lse[4][RT];        // of the tile before, this one and the two after
  int pre[kKvMaxSeqs + 1];   // units of the sequences before
  int slot[kKvMaxSeqs];      // of the first sums of a sequence whose tiles are cut
  static __device__ __forceinline__ int row_at(int r) { return r % B * STEP + r / B * (16 * P); }
};

constexpr int kKeys = 256, kRows = 128;   // keys of a block's tile, rows of a step

// A unit is a tile, or where a call's tiles are few or differ a part of its rows; the parts'
// sums are joined by a second launch in their order.  Units are ordered by sequence, head, part
// and tile, so that neighbours read the same rows, and an eighth of the work (not of the
// units) goes to each XCD, whose blocks take its units in turn and find their rows in its
// L2.  us with whole tiles, in equal numbers / so: 4096 tokens over 4096, 8 heads on 1, 741 / 78;
// 1000 over 30000 216 / 105; 512 over 4096, 64 heads on 8, 162 / 68; 2048 over 2048 in FP8 401 /
// 101; 2 x 2048 over 5000 427 / 335; one of 2048 over 4096 among 63 of 1 over 2000 1187 / 348; 32
// sequences of 1 to 1024 over 1024 to 4096 1025 / 865; 64 of 1 to 512, 32 heads on 32, 472 / 394.
// (One more part for each block: 10 of 1 to 1672 over 1672 198 / 190, but 2 x 2048 over 5000
// 335 / 359.  Equal shares of all rows, cut wherever they end, were slower: the last 2048 of
// 16384 736 for 600, with rows from HBM instead of L2.)
struct WeighTile {
  int32_t seq, head, tile;
  int32_t parts;   // 0: not the first part of its tile
};
struct WeighCut {
  int32_t slots;   // sums that the second launch finds
  int32_t pad[63];
};
constexpr int kCuts = 2, kMaxParts = 32;
inline __host__ __device__ int most_slots(int G) { return 4 * kCuts * G; }
struct Plan {
  int x0, x1;    // units of the block's XCD
  int quantum;   // steps of a part
};
// Steps of rows that a tile of the sequence has at most.
__device__ __forceinline__ int steps_of(const WeighArgs& a, const KvSeq& q) {
  const int tokens = a.window > 0 ? min(q.q_len, a.window + kKeys) : q.q_len;
  return (tokens * a.group + kRows - 1) / kRows;
}
__device__ __forceinline__ int parts_of(int steps, int quantum) { return min((steps + quantum - 1) / quantum, kMaxParts); }

// Sums over a wave's lanes up to each.
template <typename T>
__device__ __forceinline__ T lanes_up_to(T x) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const T z = __shfl_up(x, d);
    x += lane >= d ? z : 0;
  }
  return x;
}
// The block's part of the call, by each of its waves.  A unit's work is its steps and two more
// for its keys.  A cut tile has more steps than the quantum, and all tiles' steps are twice the work
// at most, 2 kCuts G quanta: so cut tiles are 2 kCuts G and their parts 4 kCuts G at most.
template <class S>
__device__ __forceinline__ Plan plan_work(const WeighArgs& a, S& sh, WeighCut* cut) {
  using I64 = long long;
  const int n = a.kv.n_seqs, lane = threadIdx.x & 63, G = (int)gridDim.x, xcd = (int)blockIdx.x & 7;
  struct Work {
    int tiles, steps;
    I64 all;   // in half steps; a tile of new tokens has half of the steps, about
  };
  auto of = [&](int s) {
    if (s >= n) return Work{0, 0, 0};
    const KvSeq q = kv_seq(a.kv, s);
    const int tiles = (tokens_of(a, q) + kKeys - 1) / kKeys, steps = steps_of(a, q);
    return Work{tiles * a.kv.H, steps, a.kv.H * ((I64)(2 * tiles - min(q.q_len / kKeys, tiles)) * steps + 4 * tiles)};
  };
  const Work mine = of(lane);
  I64 total = mine.all;
  int whole = mine.tiles, longest = mine.tiles ? mine.steps + 2 : 0;
  for (int s = lane + 64; s < n; s += 64) {
    const Work w = of(s);
    total += w.all;
    whole += w.tiles;
    longest = max(longest, w.tiles ? w.steps + 2 : 0);
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) {
    total += __shfl_xor(total, d);
    whole += __shfl_xor(whole, d);
    longest = max(longest, __shfl_xor(longest, d));
  }
  Plan p;
  // (whole tiles where their rounds are within a tenth of the work)
  p.quantum = cut && (I64)((whole + G - 1) / G) * longest > total / 2 / G * 11 / 10
                  ? (int)min(max((total / 2 + kCuts * G) / (kCuts * G), (I64)4), (I64)1 << 30)
                  : 1 << 30;
  const I64 v[2] = {total * xcd / 8, total * (xcd + 1) / 8};
  int bound[2] = {0, 0}, units = 0, slots = 0;
  I64 before = 0;
  for (int s0 = 0; s0 < n; s0 += 64) {
    const int s = s0 + lane;
    const Work w = s0 ? of(s) : mine;
    const int parts = max(parts_of(w.steps, p.quantum), 1), own = w.tiles * parts, in_slots = parts > 1 ? own : 0;
    const int u = lanes_up_to(own), t = lanes_up_to(in_slots);
    const I64 c = lanes_up_to(w.all);
    if (s < n) {   // (every wave writes the same)
      sh.pre[s] = units + u - own;
      sh.slot[s] = slots + t - in_slots;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const I64 in = v[i] - (before + c - w.all);
      const unsigned long long hit = __ballot(in >= 0 && in < w.all);
      const int at = units + u - own + min((int)((double)in / (double)w.all * (double)own), own);
      if (hit) bound[i] = __builtin_amdgcn_readlane(at, __builtin_ctzll(hit));
    }
    units += __builtin_amdgcn_readlane(u, 63);
    slots += __builtin_amdgcn_readlane(t, 63);
    before += __shfl(c, 63);
  }
  if (threadIdx.x == 0) {
    sh.pre[n] = units;
    if (cut && blockIdx.x == 0) cut->slots = slots;
  }
  __syncthreads();
  p.quantum = uni(p.quantum);
  p.x0 = uni(bound[0]);
  p.x1 = uni(xcd == 7 ? units : bound[1]);
  return p;
}

template <typename A, typename KV, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_weigh_tiles(WeighArgs a, WeighCut* cut) {
  constexpr bool Q8 = is_quant<KV>();
  using S = WeighShared<D>;
  constexpr int KT = kKeys, NQ = D / 16, RT = S::RT, P = S::P, B = S::B;
  static_assert(RT == kRows, "steps");
  extern __shared__ __align__(16) char smem[];
  S& sh = *reinterpret_cast<S*>(smem);
  const KvView& kv = a.kv;
  const Plan plan = plan_work(a, sh, cut);
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), col = lane & 31, hi = lane >> 5;
  WeighTile* const tiles = reinterpret_cast<WeighTile*>(cut + 1);   // of each slot
  float* const sums = reinterpret_cast<float*>(tiles + most_slots((int)gridDim.x));
  for (int un = plan.x0 + ((int)blockIdx.x >> 3); un < plan.x1; un += (int)gridDim.x >> 3) {
    Unit u;
    u.seq = uni(seq_of(sh.pre, kv.n_seqs, un));
    unit_seq(a, u, nullptr);
    const int n_tiles = (u.n + KT - 1) / KT, parts = max(parts_of(steps_of(a, u.q), plan.quantum), 1);
    const int rem = un - uni(sh.pre[u.seq]);
    u.head = rem / (parts * n_tiles);
    const int part_no = (rem - u.head * parts * n_tiles) / n_tiles, tile_no = rem - (u.head * parts + part_no) * n_tiles;
    u.tile = tile_no * KT;
    const KvSeq& q = u.q;
    const int32_t* ktab = kv.table + ((int64_t)u.seq * 2 * kv.H + u.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    const int k0 = u.tile + wave * 64;
    const int win = a.window > 0 ? a.window : 0x40000000;
    u32x4 kf[2][NQ];
    float f[2], sum[2] = {0.f, 0.f};
    bool there[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int t = k0 + 32 * c + col;
      const int blk = (int)kv_div(kv, (uint32_t)t), slot = t - blk * kv.T;
      const int kp = blk < kv.nb ? ktab[blk] : -1, vp = blk < kv.nb ? vtab[blk] : -1;
      there[c] = (unsigned)kp < (unsigned)kv.n_pages && (unsigned)vp < (unsigned)kv.n_pages;
      const int pg = there[c] ? kp : 0, sl = there[c] ? slot : 0;
      const char* src = kv.pages + (int64_t)pg * kv.page_bytes + sl * 16;
#pragma unroll
      for (int k = 0; k < NQ; ++k) {
        if constexpr (Q8) {
          const uint2 w = *reinterpret_cast<const uint2*>(src + (int64_t)k * kv.T * 16 + hi * 8);
          kf[c][k] = fp8_to16<A>(w.x, w.y);
        } else {
          kf[c][k] = ldv(src + (int64_t)(2 * k + hi) * kv.T * 16);
        }
      }
      f[c] = a.scale_log2;
      if (Q8) f[c] *= __uint_as_float((uint32_t)kv.scales[(int64_t)pg * kv.T + sl] << 23);
    }
    // of the sequence's rows those of tokens [t0, t1) see something of the block's keys
    // (none of either where positions lie far from the keys: both stay within the sequence)
    const int t0 = min(max(u.tile - q.base, 0), q.q_len);
    const int t1 = a.window > 0 ? max(min(q.q_len, u.tile + KT - 1 + a.window - q.base), 0) : q.q_len;
    int r0 = t0 * a.group, r1 = t1 * a.group;
    if (parts > 1) {   // the part's steps of them
      const int steps = max(r1 - r0 + RT - 1, 0) / RT;
      r1 = min(r1, r0 + steps * (part_no + 1) / parts * RT);
      r0 += steps * part_no / parts * RT;
    }
    // rows rt .. rt + RT - 1 to a slot, their lse to LDS.  A lane finds the place of a row of
    // each 64, the loads take it from the lanes that have theirs
    auto issue = [&](int rt, int n) {
      float ls[RT / 64];
#pragma unroll
      for (int h = 0; h < RT / 64; ++h) {
        const int r = min(rt + 64 * h + lane, r1 - 1), t = token_of(a, r), in = u.head * a.group + r - t * a.group;
        const int64_t at = (int64_t)(q.q0 + t) * a.q_ld + (int64_t)in * D;
#pragma unroll
        for (int i = 0; i < B / 4; ++i) {
          const int b = wave + 4 * i, mine = b + B * (lane / P);   // the load's block, the lane's row
          const uint32_t lo = (uint32_t)__builtin_amdgcn_ds_bpermute(mine * 4, (int)(uint32_t)at);
          const int high = __builtin_amdgcn_ds_bpermute(mine * 4, (int)(at >> 32));
          const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + ((int64_t)high << 32 | lo) + lane % P * 8;
          load_lds16(src, sh.q + (n & 1) * S::SLOT + h * S::HALF + b * S::STEP);
        }
        if (wave == 0) ls[h] = a.lse[(int64_t)(q.q0 + t) * a.n_q_heads + in] * kLog2e;
      }
      if (wave == 0)
#pragma unroll
        for (int h = 0; h < RT / 64; ++h) sh.lse[n & 3][64 * h + lane] = ls[h];
    };
    // One step: the exponentials of 32 rows' scores s (rows ra on) and the products of the
    // 32 rows at `at`, woven, which keeps the matrix cores and the vector ALUs busy at the same
    // time.  Operands are read four products ahead, of the step after this one too if its
    // rows are there (then, at `after`), and that step's lse.
    constexpr int R = 4, M = 2 * NQ, EACH = 32 / M;   // operands read ahead, products, exponentials to each
    u32x4 fr[R];
    f32x4 ls[4];
    const char* const mine = sh.q + S::row_at(col) + hi * 16;
    auto operand = [&](int at, int k) { return *reinterpret_cast<const u32x4*>(mine + at + k * 32); };
    auto lse_of = [&](const float* lse, int b) { return *reinterpret_cast<const f32x4*>(lse + 8 * b + 4 * hi); };
    auto step = [&](auto then, f32x16(&s)[2], f32x16(&sn)[2], int at, int after, const float* next_ls, int ra)
        __attribute__((always_inline)) {
      float part[2] = {0.f, 0.f};   // of 32 rows: the long sum's terms are of one size
      const int rz = min(ra + 31, r1 - 1), pa = q.base + token_of(a, ra), pz = q.base + token_of(a, rz);
      const bool edge = k0 + 63 > pa || k0 <= pz - win || ra + 31 >= r1;
      auto product = [&](int m) __attribute__((always_inline)) {
        const int k = m >> 1, c = m & 1;
        sn[c] = mfma32<A>(fr[k % R], kf[c][k], k ? sn[c] : f32x16{});
        if (!c) return;
        if (k + R < NQ) fr[k % R] = operand(at, k + R);
        else if (decltype(then)::value) fr[k % R] = operand(after, k + R - NQ);
      };
      if (__builtin_expect(edge, 0)) {
#pragma unroll
        for (int m = 0; m < M; ++m) product(m);
        float fe[2] = {f[0], f[1]};   // (unknown to the compiler, which would take the exponentials of both ways ahead of them)
        asm volatile("" : "+v"(fe[0]), "+v"(fe[1]));
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int r = ra + 8 * (i >> 2) + 4 * hi + (i & 3), pos = q.base + token_of(a, r);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int j = k0 + 32 * c + col;
            const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][i], fe[c], -ls[i >> 2][i & 3]));
            part[c] += r < r1 && j <= pos && j > pos - win ? p : 0.f;
          }
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) ls[b] = lse_of(next_ls, b);
      } else {
        constexpr int L = 4;   // a sum follows its exponential by so many others
        float y[L] = {};
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          __builtin_amdgcn_sched_barrier(0);
          const int i = e >> 1, c = e & 1;
          const float x = __builtin_fmaf(s[c][i], f[c], -ls[i >> 2][i & 3]);
          if (e % EACH == 0) product(e / EACH);
          if (e >= L) {
            part[c] += y[e % L];
            asm volatile("" : "+v"(part[c]));   // (else the sums gather after the last product)
          }
          y[e % L] = __builtin_amdgcn_exp2f(x);
          if (e % 8 == 7) ls[e / 8] = lse_of(next_ls, e / 8);
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int e = 0; e < L; ++e) part[e & 1] += y[e];
      }
      sum[0] += part[0];
      sum[1] += part[1];
    };
    auto arrived = [&] {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
    };
    auto begin = [&](int at) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < R; ++k) fr[k] = operand(at, k);
    };
    if (r0 < r1) {
      issue(r0, 0);
      arrived();
      if (r0 + RT < r1) issue(r0 + RT, 1);
      f32x16 s0[2], s1[2];
#pragma unroll
      for (int k = 0; k < NQ; ++k)
#pragma unroll
        for (int c = 0; c < 2; ++c) s0[c] = mfma32<A>(operand(0, k), kf[c][k], k ? s0[c] : f32x16{});
      constexpr int HALF32 = 32 / B * 16 * P;   // distance of 32 rows
      begin(HALF32);
#pragma unroll
      for (int b = 0; b < 4; ++b) ls[b] = lse_of(&sh.lse[0][0], b);
      int n = 0;
      for (int rt = r0; rt < r1; rt += RT, ++n) {
        const int here = (n & 1) * S::SLOT, next = S::SLOT - here;
        const float* lse = &sh.lse[n & 3][0];
        step(std::true_type{}, s0, s1, here + HALF32, here + S::HALF, lse + 32, rt);
        if (rt + 32 >= r1) break;
        step(std::true_type{}, s1, s0, here + S::HALF, here + S::HALF + HALF32, lse + 64, rt + 32);
        if (rt + 64 >= r1) break;
        step(std::false_type{}, s0, s1, here + S::HALF + HALF32, 0, lse + 96, rt + 64);
        if (rt + 96 >= r1) break;
        arrived();   // the next tile; this one's slot has been read
        if (rt + 2 * RT < r1) issue(rt + 2 * RT, n + 2);
        begin(next);
        step(std::true_type{}, s1, s0, next, next + HALF32, &sh.lse[(n + 1) & 3][0], rt + 96);
      }
    }
    __syncthreads();   // the slots have been read
#pragma unroll
    for (int c = 0; c < 2; ++c) sum[c] += __shfl_xor(sum[c], 32);
    const int j = k0 + lane;
    const int64_t at = ((int64_t)u.seq * kv.H + u.head) * a.w_ld;
    const float got = hi ? sum[1] : sum[0];
    if (parts > 1) {
      const int slot = uni(sh.slot[u.seq]) + (u.head * n_tiles + tile_no) * parts + part_no;
      sums[(int64_t)slot * KT + wave * 64 + lane] = got;
      if (tid == 0) tiles[slot] = WeighTile{u.seq, u.head, u.tile, part_no ? 0 : parts};
    } else if (j < u.n) {
      a.weights[at + j] = (hi ? there[1] : there[0]) ? old_weight(a, u, at, j) + got : 0.f;
    }
  }
}

// The parts of a tile together, a thread a key.
__global__ __launch_bounds__(kKeys) void k_weigh_join(WeighArgs a, const WeighCut* __restrict__ cut, int G) {
  const KvView& kv = a.kv;
  const WeighTile* tiles = reinterpret_cast<const WeighTile*>(cut + 1);
  const float* sums = reinterpret_cast<const float*>(tiles + most_slots(G)) + threadIdx.x;
  const int slots = cut->slots;
  for (int i = blockIdx.x; i < slots; i += gridDim.x) {
    const WeighTile d = tiles[i];
    if (d.parts == 0) continue;
    float sum = 0.f;
    for (int p = 0; p < d.parts; ++p) sum += sums[(int64_t)(i + p) * kKeys];
    Unit u;
    u.seq = d.seq;
    unit_seq(a, u, nullptr);
    const int j = d.tile + (int)threadIdx.x;
    if (j >= u.n) continue;
    const int blk = (int)kv_div(kv, (uint32_t)j);
    const int32_t* ktab = kv.table + ((int64_t)d.seq * 2 * kv.H + d.head) * kv.nb;
    const bool there = (unsigned)ktab[blk] < (unsigned)kv.n_pages && (unsigned)ktab[(int64_t)kv.H * kv.nb + blk] < (unsigned)kv.n_pages;
    const int64_t at = ((int64_t)d.seq * kv.H + d.head) * a.w_ld;
    a.weights[at + j] = there ? old_weight(a, u, at, j) + sum : 0.f;
  }
}

// Tiles may be cut where a head has more rows than four steps take.
inline bool may_cut(int32_t group, int32_t max_q_len) { return (int64_t)max_q_len * group > 4 * kRows; }
inline int blocks_of(int n_cu) { return 2 * n_cu / 8 * 8; }

template <typename A, typename KV, int D>
hipError_t launch_tiles(const WeighArgs& a, hipStream_t s) {
  const size_t lds = sizeof(WeighShared<D>);
  static PerDevice limit;   // the kernel's LDS, more than a block gets unasked, is a setting of each device
  int device = -1;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess)
    e = limit.done(device, [&] {
      return hipFuncSetAttribute(reinterpret_cast<const void*>(&k_weigh_tiles<A, KV, D>),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
  if (e != hipSuccess) return e;
  const int G = blocks_of(a.n_cu);
  WeighCut* cut = may_cut(a.group, a.max_q_len) ? reinterpret_cast<WeighCut*>(a.ws) : nullptr;
  hipLaunchKernelGGL((k_weigh_tiles<A, KV, D>), dim3(G), dim3(256), lds, s, a, cut);
  if (cut) hipLaunchKernelGGL(k_weigh_join, dim3(2 * G), dim3(kKeys), 0, s, a, cut, G);
  return hipGetLastError();
}

template <typename A, typename KV, int D>
hipError_t launch(const WeighArgs& a, hipStream_t s) {
  if ((int64_t)a.max_q_len * a.group <= kFewRows)
    hipLaunchKernelGGL((k_weigh_rows<A, KV, D>), dim3(kRowsBlocks * a.n_cu), dim3(256), 0, s, a);
  else
    return launch_tiles<A, KV, D>(a, s);
  return hipGetLastError();
}
template <typename A, typename KV>
hipError_t launch_d(const KvTypes& ty, const WeighArgs& a, hipStream_t s) {
  return ty.D == 128 ? launch<A, KV, 128>(a, s) : launch<A, KV, 64>(a, s);
}

}  // namespace

size_t weigh_workspace(int32_t n_cu, int32_t group, int32_t max_q_len) {
  if (!may_cut(group, max_q_len)) return 0;
  return sizeof(WeighCut) + (size_t)most_slots(blocks_of(n_cu)) * (sizeof(WeighTile) + kKeys * sizeof(float));
}

int64_t weigh_units(const KvView& v) { return (int64_t)v.n_seqs * v.H * ((int64_t)v.nb * v.T / 32 + 1); }

hipError_t launch_weigh(const KvTypes& ty, const WeighArgs& a, hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  if (ty.act == LORA_F16) return q ? launch_d<f16_t, fp8_t>(ty, a, s) : launch_d<f16_t, f16_t>(ty, a, s);
  return q ? launch_d<bf16_t, fp8_t>(ty, a, s) : launch_d<bf16_t, bf16_t>(ty, a, s);
}

}  // namespace lora
