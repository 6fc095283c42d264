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

namespace lora {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// Tiles of KT cached tokens of a (sequence, head), in that order of sequences.
__device__ __forceinline__ int tokens_of(const WeighArgs& a, const KvSeq& q) {
  return (int)min((int64_t)q.end, a.w_ld);
}
// Prefix sums of the sequences' tiles in LDS (n_seqs + 1); returns all of them.
template <int KT, int THREADS>
__device__ __forceinline__ int tile_sums(const WeighArgs& a, int* pre) {
  const int n = a.kv.n_seqs, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  __shared__ int wsum[THREADS / 64];
  int run = 0;
  for (int s0 = 0; s0 < n; s0 += THREADS) {
    const int s = s0 + tid;
    int sum = 0;
    if (s < n) sum = (tokens_of(a, kv_seq(a.kv, s)) + KT - 1) / KT * a.kv.H;
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

struct Unit {
  int seq, head, tile;
  KvSeq q;
};
template <int KT>
__device__ __forceinline__ Unit unit_of(const WeighArgs& a, const int* pre, int u) {
  Unit r;
  r.seq = uni(seq_of(pre, a.kv.n_seqs, u));
  r.q = kv_seq(a.kv, r.seq);
  r.q.q0 = uni(r.q.q0);
  r.q.q_len = uni(r.q.q_len);
  r.q.base = uni(r.q.base);
  r.q.end = uni(r.q.end);
  const int tiles = (tokens_of(a, r.q) + KT - 1) / KT, rem = u - pre[r.seq];
  r.head = uni(rem / tiles);
  r.tile = uni((rem - r.head * tiles) * KT);
  return r;
}

// What a token had before, faded; new tokens had nothing.
__device__ __forceinline__ float old_weight(const WeighArgs& a, const Unit& u, int64_t at, int j) {
  return a.before && a.decay > 0.f && j < u.q.base ? a.decay * a.before[at + j] : 0.f;
}

// ---- up to 16 rows ---------------------------------------------------------------
// A wave for itself: KT keys straight to registers, the rows in tiles of 16.
template <typename A, typename KV, int D>
__global__ __launch_bounds__(256) void k_weigh_rows(WeighArgs a) {
  constexpr bool Q8 = is_quant<KV>();
  constexpr int E = ET<KV>::E, KT = 4 * E, NB = KT / 16, NC = D / (4 * E), NQ = D / 32;
  __shared__ int pre[kKvMaxSeqs + 1];
  const KvView& kv = a.kv;
  const int units = tile_sums<KT, 256>(a, pre);
  const int tid = threadIdx.x, lane = tid & 63, col = lane & 15, g = lane >> 4;
  const int workers = (int)gridDim.x * 4, worker = (int)blockIdx.x * 4 + uni(tid >> 6);
  const int from = (int)((int64_t)units * worker / workers), to = (int)((int64_t)units * (worker + 1) / workers);
  for (int un = from; un < to; ++un) {
    const Unit u = unit_of<KT>(a, pre, un);
    const KvSeq& q = u.q;
    const int32_t* ktab = kv.table + ((int64_t)u.seq * 2 * kv.H + u.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    const int rows = q.q_len * a.group, n = tokens_of(a, q);
    const int win = a.window > 0 ? a.window : 0x40000000;
    u32x4 kf[NB][NC];
    float f[NB], sum[NB];
    bool there[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int t = u.tile + 16 * b + col;
      const int blk = (int)kv_div(kv, (uint32_t)t), slot = t - blk * kv.T;
      const int kp = blk < kv.nb ? ktab[blk] : -1, vp = blk < kv.nb ? vtab[blk] : -1;
      there[b] = (unsigned)kp < (unsigned)kv.n_pages && (unsigned)vp < (unsigned)kv.n_pages;
      const int pg = there[b] ? kp : 0;
      const char* src = kv.pages + (int64_t)pg * kv.page_bytes + (g * kv.T + (there[b] ? slot : 0)) * 16;
#pragma unroll
      for (int c = 0; c < NC; ++c) kf[b][c] = ldv(src + c * 4 * kv.T * 16);
      f[b] = a.scale_log2;
      if (Q8) f[b] *= __uint_as_float((uint32_t)kv.scales[(int64_t)pg * kv.T + (there[b] ? slot : 0)] << 23);
      sum[b] = 0.f;
    }
    // of the sequence's rows those of tokens [t0, t1) see something of the tile
    const int t0 = max(u.tile - q.base, 0);
    const int t1 = a.window > 0 ? min(q.q_len, u.tile + KT - 1 + a.window - q.base) : q.q_len;
    for (int r0 = t0 * a.group; r0 < min(t1 * a.group, rows); r0 += 16) {
      u32x4 qf[NQ];
      {
        const int row = min(r0 + col, rows - 1), t = token_of(a, row);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(q.q0 + t) * a.q_ld +
                              (int64_t)(u.head * a.group + row - t * a.group) * D;
#pragma unroll
        for (int i = 0; i < NQ; ++i) qf[i] = ldv(src + (Q8 ? (4 * (i >> 1) + g) * 16 + (i & 1) * 8 : (4 * i + g) * 8));
      }
      float ls[4];
      int pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + 4 * g + i, r = min(row, rows - 1), t = token_of(a, r);
        ls[i] = a.lse[(int64_t)(q.q0 + t) * a.n_q_heads + u.head * a.group + r - t * a.group] * kLog2e;
        pos[i] = row < rows ? q.base + t : -0x40000000;
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x4 s = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          if constexpr (Q8) {
            s = mfma16<A>(qf[2 * c], fp8_to16<A>(kf[b][c].x, kf[b][c].y), s);
            s = mfma16<A>(qf[2 * c + 1], fp8_to16<A>(kf[b][c].z, kf[b][c].w), s);
          } else {
            s = mfma16<A>(qf[c], kf[b][c], s);
          }
        }
        const int j = u.tile + 16 * b + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i], f[b], -ls[i]));
          sum[b] += j <= pos[i] && j > pos[i] - win ? p : 0.f;
        }
      }
    }
    // the lane groups' rows together; group g writes the 16 keys of block g
    float mine = 0.f;
    bool ok = false;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x = sum[b];
      x += __shfl_xor(x, 16);
      x += __shfl_xor(x, 32);
      if (g == b) {
        mine = x;
        ok = there[b];
      }
    }
    const int j = u.tile + 16 * g + col;
    const int64_t at = ((int64_t)u.seq * kv.H + u.head) * a.w_ld;
    if (g < NB && j < n) a.weights[at + j] = ok ? old_weight(a, u, at, j) + mine : 0.f;
  }
}

// ---- more rows -------------------------------------------------------------------
// A block's four waves have 64 keys each, in registers for all of the rows, which go
// through LDS in tiles of 64 (two slots, one barrier a tile).
template <int D>
struct WeighShared {
  u32x4 q[2][D / 8][64];
  float lse[2][64];
};
template <typename A, typename KV, int D>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_weigh_tiles(WeighArgs a) {
  constexpr bool Q8 = is_quant<KV>();
  constexpr int KT = 256, NQ = D / 16, RT = 64;
  __shared__ int pre[kKvMaxSeqs + 1];
  __shared__ __align__(16) WeighShared<D> sh;
  const KvView& kv = a.kv;
  const int units = tile_sums<KT, 256>(a, pre);
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6), col = lane & 31, hi = lane >> 5;
  // an eighth of the units to each XCD: the tiles of one head, which read the same rows, share its L2
  const int per = (units + 7) / 8, x0 = min(((int)blockIdx.x & 7) * per, units), x1 = min(x0 + per, units);
  for (int un = x0 + ((int)blockIdx.x >> 3); un < x1; un += (int)gridDim.x >> 3) {
    const Unit u = unit_of<KT>(a, pre, un);
    const KvSeq& q = u.q;
    const int32_t* ktab = kv.table + ((int64_t)u.seq * 2 * kv.H + u.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    const int n = tokens_of(a, q), k0 = u.tile + wave * 64;
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
    const int t0 = max(u.tile - q.base, 0);
    const int t1 = a.window > 0 ? min(q.q_len, u.tile + KT - 1 + a.window - q.base) : q.q_len;
    const int r0 = t0 * a.group, r1 = t1 * a.group;
    auto row_of = [&](int r) { return min(r, r1 - 1); };
    float next_lse = 0.f;
    auto issue = [&](int rt, int slot) {   // rows rt .. rt + 63 to a slot; their lse to a register
#pragma unroll
      for (int i = 0; i < D / 8 / 4; ++i) {
        const int piece = wave + 4 * i, r = row_of(rt + lane), t = token_of(a, r);
        const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(q.q0 + t) * a.q_ld +
                              (int64_t)(u.head * a.group + r - t * a.group) * D + piece * 8;
        load_lds16(src, &sh.q[slot][piece][0]);
      }
      if (tid < RT) {
        const int r = row_of(rt + tid), t = token_of(a, r);
        next_lse = a.lse[(int64_t)(q.q0 + t) * a.n_q_heads + u.head * a.group + r - t * a.group] * kLog2e;
      }
    };
    int slot = 0;
    if (r0 < r1) {
      issue(r0, 0);
      if (tid < RT) sh.lse[0][tid] = next_lse;
    }
    for (int rt = r0; rt < r1; rt += RT, slot ^= 1) {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
      const bool more = rt + RT < r1;
      if (more) issue(rt + RT, slot ^ 1);
#pragma unroll 1
      for (int rb = 0; rb < 2; ++rb) {
        const int ra = rt + 32 * rb, rz = min(ra + 31, r1 - 1);
        if (ra >= r1) break;
        const int pa = q.base + token_of(a, ra), pz = q.base + token_of(a, rz);
        if (k0 > pz || k0 + 63 <= pa - win) continue;   // nothing of the wave's keys is seen
        f32x16 s[2] = {f32x16{}, f32x16{}};
#pragma unroll
        for (int k = 0; k < NQ; ++k) {
          const u32x4 qf = sh.q[slot][2 * k + hi][32 * rb + col];
          s[0] = mfma32<A>(qf, kf[0][k], s[0]);
          s[1] = mfma32<A>(qf, kf[1][k], s[1]);
        }
        const bool edge = k0 + 63 > pa || k0 <= pz - win || ra + 31 >= r1;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const f32x4 ls = *reinterpret_cast<const f32x4*>(&sh.lse[slot][32 * rb + 8 * b + 4 * hi]);
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float p = __builtin_amdgcn_exp2f(__builtin_fmaf(s[c][4 * b + i], f[c], -ls[i]));
              if (edge) {
                const int row = ra + 8 * b + 4 * hi + i, j = k0 + 32 * c + col;
                const int pos = q.base + token_of(a, row);
                p = row < r1 && j <= pos && j > pos - win ? p : 0.f;
              }
              sum[c] += p;
            }
        }
      }
      if (more && tid < RT) sh.lse[slot ^ 1][tid] = next_lse;
    }
    __syncthreads();   // the slots have been read
#pragma unroll
    for (int c = 0; c < 2; ++c) sum[c] += __shfl_xor(sum[c], 32);
    const int j = k0 + lane;
    const int64_t at = ((int64_t)u.seq * kv.H + u.head) * a.w_ld;
    if (j < n) a.weights[at + j] = (hi ? there[1] : there[0]) ? old_weight(a, u, at, j) + (hi ? sum[1] : sum[0]) : 0.f;
  }
}

template <typename A, typename KV, int D>
hipError_t launch(const WeighArgs& a, hipStream_t s) {
  if ((int64_t)a.max_q_len * a.group <= 16)
    hipLaunchKernelGGL((k_weigh_rows<A, KV, D>), dim3(4 * a.n_cu), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_weigh_tiles<A, KV, D>), dim3(2 * a.n_cu / 8 * 8), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename A, typename KV>
hipError_t launch_d(const KvTypes& ty, const WeighArgs& a, hipStream_t s) {
  return ty.D == 128 ? launch<A, KV, 128>(a, s) : launch<A, KV, 64>(a, s);
}

}  // namespace

size_t weigh_workspace(const KvTypes&, int32_t, int32_t, int32_t) { return 0; }

int64_t weigh_units(const KvView& v) { return (int64_t)v.n_seqs * v.H * ((int64_t)v.nb * v.T / 32 + 1); }

hipError_t launch_weigh(const KvTypes& ty, const WeighArgs& a, hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  if (ty.act == LORA_F16) return q ? launch_d<f16_t, fp8_t>(ty, a, s) : launch_d<f16_t, f16_t>(ty, a, s);
  return q ? launch_d<bf16_t, fp8_t>(ty, a, s) : launch_d<bf16_t, bf16_t>(ty, a, s);
}

}  // namespace lora
