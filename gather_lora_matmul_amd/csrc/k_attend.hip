// Attention of new tokens over the paged cache.
//
//   s_ij = scale q_i . k_j,  p_ij = exp(s_ij - m_i),  o_i = sum_j p_ij v_j / sum_j p_ij
//
// over the keys j that query i sees: pos_i - window < j <= pos_i whose pages are
// there.  One pass over the keys with a running maximum and sum.
//
// The rows of one kv head are its G query heads times the sequence's new tokens:
// row r is token r / G, head h G + r % G.  The longest sequence's row count chooses
// one of two kernels: up to 16 rows (FP8 caches: 32; single tokens and few drafted
// ones: bound by HBM) and more (chunks: bound by the matrix cores and the vector
// ALUs).  Both compute the transposed products
//   S^T = K Q^T      O^T = V^T P^T
// so that a query is a column: its scores lie in one lane group's registers, the
// row maximum and sum need one exchange between lanes, and P leaves the first
// product in the very registers in which the second one takes it.  For that the
// rows of the K operand are tokens in an order that makes a lane's scores E
// consecutive tokens (E elements in 16 bytes), which is how the V pages hold
// them: neither K, V nor P is moved between lanes.
//
// Work is cut as the adapter products' planned launches cut theirs: all (sequence,
// head, row tile, key unit) units form one sequence, of which every block takes an
// equal contiguous range, found from the lengths on the device (no plan, no host
// wait).  A tile that several blocks share leaves unnormalised partial results in
// the workspace, and a second launch joins them in block order (run to run the
// same bits; the cut, and with it the rounding, depends on the batch).
#include <algorithm>
#include <type_traits>

#include "kcommon.h"
#include "kv.h"
#include "per_device.h"

namespace lora {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ u32x4 ldv(const void* p) { return *reinterpret_cast<const u32x4*>(p); }

constexpr float kLn2 = 0.69314718055994530942f;

template <typename T>
__device__ __forceinline__ f32x4 mfma16(const u32x4& a, const u32x4& b, f32x4 c) {
  if constexpr (std::is_same<T, bf16_t>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ f32x16 mfma32(const u32x4& a, const u32x4& b, f32x16 c) {
  if constexpr (std::is_same<T, bf16_t>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Eight FP8 codes (two words) -> eight 16-bit values, exact.
template <typename T>
__device__ __forceinline__ u32x4 fp8_to16(uint32_t w0, uint32_t w1) {
  u32x4 r;
  if constexpr (std::is_same<T, bf16_t>::value) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, 1.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, 1.0f, true));
  }
  return r;
}

// 2^(byte - 127), less `down` (0 or 1) in the exponent.
__device__ __forceinline__ float scale_of(uint32_t byte, int down) {
  return __uint_as_float((byte > (uint32_t)down ? byte - (uint32_t)down : 0u) << 23);
}

// Element e of eight 16-bit values kept where bit e is set, else zero.
__device__ __forceinline__ u32x4 keep8(u32x4 u, uint32_t bits) {
  auto m = [](uint32_t b) { return ((b & 1) ? 0xffffu : 0u) | ((b & 2) ? 0xffff0000u : 0u); };
  u.x &= m(bits);
  u.y &= m(bits >> 2);
  u.z &= m(bits >> 4);
  u.w &= m(bits >> 6);
  return u;
}

// P in the 16 bits of the second product's operands: rounded, relative 2^-8 (bf16)
// or 2^-11 (f16) at most, and what the rounding left as a second operand (together
// 2^-16 of bf16, 2^-22 of f16): the results' error is that of fp32 weights.  Only the
// tiles of 256 rows, bound by the matrix cores, take the first term alone.  The sums
// take P unrounded: lse is an fp32 result.
//   f16 has no numbers between 0 and 2^-24, and many small weights may be what a row's
// result is made of.  There P is 2^7 exp(s - m): with a maximum that P passes by 2^8
// at most it stays below 2^15, and is off by 2^-32 of a weight 1 at most, whatever its
// size.  m - 7 takes the maximum's place in the exponent and in what is stored.
template <typename T>
__device__ __forceinline__ float origin(float m) {
  const float x = m == -INFINITY ? 0.f : m;
  return std::is_same<T, f16_t>::value ? x - 7.f : x;
}
template <typename T>
__device__ __forceinline__ void p_operand(const float* p, u32x4& hi, u32x4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack2<T>(p[2 * i], p[2 * i + 1]);
    if constexpr (std::is_same<T, f16_t>::value) {
      // p - h in one instruction a value, which takes h as it lies in its half (the compiler
      // left alone rounds each half once more by itself and converts it back)
      float less = -1.f;
      asm("" : "+v"(h[i]));
      asm("" : "+v"(less));
      const f16x2_t v = __builtin_bit_cast(f16x2_t, h[i]);
      l[i] = pack2<T>(__builtin_fmaf((float)v[0], less, p[2 * i]), __builtin_fmaf((float)v[1], less, p[2 * i + 1]));
    } else {
      l[i] = pack2<T>(p[2 * i] - bits_to_f<T>(h[i] & 0xffffu), p[2 * i + 1] - bits_to_f<T>(h[i] >> 16));
    }
  }
  hi = u32x4{h[0], h[1], h[2], h[3]};
  lo = u32x4{l[0], l[1], l[2], l[3]};
}

// Values without a finite number in V must reach the rows that see their token
// and no others (0 * inf is not 0 in a matrix product).  For tiles that some row
// does not see whole: v loses them, and for each class (+inf, -inf, NaN) an
// indicator takes their place in a product with the visibility of the tokens,
// whose result says which rows get that value.  (Tiles seen whole: settle.)
template <typename T>
__device__ __forceinline__ uint32_t class_bits(const u32x4& u, int cls) {
  constexpr uint32_t kInf = std::is_same<T, bf16_t>::value ? 0x7f80u : 0x7c00u;
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t bits = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t x = (w[e / 2] >> (16 * (e & 1))) & 0xffffu;
    const bool in = cls == 0   ? x == kInf
                    : cls == 1 ? x == (kInf | 0x8000u)
                    : cls == 2 ? (x & 0x7fffu) > kInf
                               : (x & kInf) == kInf;
    bits |= (uint32_t)in << e;
  }
  return bits;
}
// Byte e of sixteen kept where bit e is set, else zero.
__device__ __forceinline__ u32x4 keep16b(u32x4 u, uint32_t bits) {
  auto m = [](uint32_t b) {
    return ((b & 1) ? 0xffu : 0u) | ((b & 2) ? 0xff00u : 0u) | ((b & 4) ? 0xff0000u : 0u) | ((b & 8) ? 0xff000000u : 0u);
  };
  u.x &= m(bits);
  u.y &= m(bits >> 4);
  u.z &= m(bits >> 8);
  u.w &= m(bits >> 12);
  return u;
}
// Not zero if one of sixteen FP8 codes is NaN (all ones but for the sign).
__device__ __forceinline__ uint32_t nan_codes(const u32x4& u) {
  constexpr uint32_t kM = 0x7f7f7f7fu, kO = 0x01010101u;
  return (((u.x & kM) + kO) | ((u.y & kM) + kO) | ((u.z & kM) + kO) | ((u.w & kM) + kO)) & 0x80808080u;
}
// Bits of the N tokens from k0 on that lie in [lo, up].
template <int N>
__device__ __forceinline__ uint32_t run_bits(int k0, int lo, int up) {
  const int x = min(max(lo - k0, 0), N), y = min(max(up - k0 + 1, 0), N);
  return ((1u << y) - 1u) & ~((1u << x) - 1u);
}
// Not zero if one of eight values is not finite: adding one to an exponent of all
// ones carries into the sign's place.
template <typename T>
__device__ __forceinline__ uint32_t not_finite(const u32x4& u) {
  constexpr uint32_t kExp = std::is_same<T, bf16_t>::value ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = std::is_same<T, bf16_t>::value ? 0x00800080u : 0x04000400u;
  return (((u.x & kExp) + kOne) | ((u.y & kExp) + kOne) | ((u.z & kExp) + kOne) | ((u.w & kExp) + kOne)) &
         0x80008000u;
}
template <typename T>
__device__ __forceinline__ u32x4 ones8(uint32_t bits) {
  constexpr uint32_t kOne = std::is_same<T, bf16_t>::value ? 0x3f803f80u : 0x3c003c00u;
  return keep8(u32x4{kOne, kOne, kOne, kOne}, bits);
}
__device__ __forceinline__ float class_value(int cls) {
  return __uint_as_float(cls == 0 ? 0x7f800000u : (cls == 1 ? 0xff800000u : 0x7fc00000u));
}

// ---- the cut of the work -----------------------------------------------------------

// A part of one row tile: keys [unit0, unit0 + units) * KU of sequence s, head h,
// rows [row0, row0 + rows).
struct Piece {
  int seq, head, row0, rows;
  int key0, key1;        // keys to visit, key0 a multiple of KU
  int start;             // the tile's first unit in the whole sequence of units
  int first;             // block that has it (-1: a tile given out whole)
  bool begins, ends;     // the piece has the tile's first / last unit
  KvSeq q;
};
struct PartDesc {        // a tile whose last of several parts a block has
  int32_t last;          // that block, -1: none
  int32_t first;         // block of its first part
  int32_t first_slot;
  int32_t head, row0, rows, q0;
  int32_t share;         // groups of lanes of the joining launch that a row gets
};

__device__ __forceinline__ int token_of(const AttendArgs& a, int row) {  // row / group
  return a.group == 1 ? row : (int)(__umulhi((uint32_t)row, a.group_m) >> a.group_s);
}
// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ int uni(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Keys that the rows [row0, row0 + rows) of a sequence visit: from the first
// row's window, down to a multiple of KU, to the last row's own position or the
// table's end.
template <int KU>
__device__ __forceinline__ void tile_keys(const AttendArgs& a, const KvSeq& q, int row0, int rows,
                                          int& lo, int& hi) {
  const int t0 = token_of(a, row0), t1 = token_of(a, row0 + rows - 1);
  hi = min(q.base + t1 + 1, q.end);
  lo = 0;
  if (a.window > 0 && q.base + t0 + 1 - a.window > 0)
    lo = min(q.base + t0 + 1 - a.window, max(q.end - 1, 0)) / KU * KU;
  if (hi <= lo) hi = lo + 1;  // nothing is seen: one unit, all of it masked
}
template <int KU, int TR>
__device__ __forceinline__ int tile_units(const AttendArgs& a, const KvSeq& q, int tile) {
  const int row0 = tile * TR, rows = min(TR, q.q_len * a.group - row0);
  if (rows <= 0) return 0;
  int lo, hi;
  tile_keys<KU>(a, q, row0, rows, lo, hi);
  return (hi - lo + KU - 1) / KU;
}
// Units of the tiles before `tile`, by the whole wave (q and tile uniform).
__device__ __forceinline__ int wave_add(int x) {
#pragma unroll
  for (int d = 32; d; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

// All units of a call are fewer than 2^31 (attend_units, checked on the host), if its
// q_start ascend; a call whose units are more all the same does nothing.
struct Cut {               // ("block": the worker, which may be a wave)
  int pos, end;          // this block's range of units
  int each, over;        // block L's range begins at L each + min(L, over)
  int block, blocks;     // its number in the order of the ranges, and the blocks that have one
  int seq;
  int unit0;             // the first unit that is cut into ranges: the tiles before it are given
  int tile, tiles, step; // out whole, tile, tile + step, .. < tiles to this block
  __device__ int begin_of(int L) const { return unit0 + L * each + min(L, over); }
  __device__ int block_of(int x) const {
    const int big = (each + 1) * over;
    x -= unit0;
    return x < big ? (int)((uint32_t)x / (uint32_t)(each + 1)) : over + (int)((uint32_t)(x - big) / (uint32_t)each);
  }
};

// Prefix sums of the sequences' units in LDS, and this block's range.  Every
// block computes them itself: the lengths are a few KB that stay in L2.  A lane
// adds up the tiles of its sequence if they are few, all lanes together those of
// each other one.
// Of `workers` workers (blocks, or waves) this is number i of those on its XCD.
//
// With preT (prefix sums of the tiles) and tiles about equally long, as many whole
// rounds of tiles as the workers can take go out whole first, neighbouring tiles to
// the workers of one XCD: they walk the same keys at the same time, which ranges cut
// anywhere do not, and find them in their L2 (a chunk of 2048 tokens over 16384, 8
// heads: 54 % of the L2's reads missed without it).
template <int KU, int TR, int THREADS>
__device__ __forceinline__ void cut_work(const AttendArgs& a, int* pre, Cut& c, int workers, int i,
                                         int* preT = nullptr) {
  const int n = a.kv.n_seqs;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int W = THREADS / 64, FEW = 2;
  int* wsum = pre + kKvMaxSeqs + 1;
  uint32_t run = 0;
  bool past = false;            // too many units
  const bool small = n <= 64;   // every wave for itself
  int longest = 0;              // units of the longest tile, if no window is set
  for (int s0 = 0; s0 < n; s0 += small ? 64 : THREADS) {
    const int s = s0 + (small ? lane : tid);
    int units = 0;
    KvSeq q{0, 0, 0, 0};
    if (s < n) q = kv_seq(a.kv, s);
    const int tiles = (q.q_len * a.group + TR - 1) / TR;
#pragma unroll
    for (int t = 0; t < FEW; ++t)
      if (t < tiles) units += tile_units<KU, TR>(a, q, t);
    for (unsigned long long more = __ballot(tiles > FEW); more; more &= more - 1) {
      const int src = __builtin_ctzll(more);
      const KvSeq u{0, __shfl(q.q_len, src), __shfl(q.base, src), __shfl(q.end, src)};
      const int tu = __shfl(tiles, src);
      int part = 0;
      for (int t = FEW + lane; t < tu; t += 64) part += tile_units<KU, TR>(a, u, t);
      part = wave_add(part);
      if (lane == src) units += part;
    }
    uint32_t sum = (uint32_t)(units * a.kv.H);   // (of one sequence: below 2^31)
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t z = __shfl_up(sum, d);
      if (lane >= d) sum += z;
    }
    if (preT && small) {
      longest = tiles > 0 ? (q.end + KU - 1) / KU : 0;
      int st = tiles * a.kv.H;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(st, d);
        longest = max(longest, __shfl_xor(longest, d));
        if (lane >= d) st += z;
      }
      if (s < n) preT[s + 1] = st;
      if (lane == 0) preT[0] = 0;
    }
    if (!small) {
      if (lane == 63) wsum[wave] = (int)sum;
      __syncthreads();
      uint32_t before = run, all = 0;
      for (int w = 0; w < W; ++w) {
        if (w < wave) before += (uint32_t)wsum[w];
        all += (uint32_t)wsum[w];
      }
      sum += before;
      if (s < n) pre[s + 1] = (int)sum;
      run += all;
      __syncthreads();
    } else if (s < n) {
      pre[s + 1] = (int)sum;   // the same from every wave
    }
    // the first prefix sum past 2^31 is below 2^32: its bit 31 shows
    past |= s < n && (int)sum < 0;
  }
  if (small ? lane == 0 : tid == 0) pre[0] = 0;
  past = small ? __ballot(past) != 0 : __syncthreads_or(past) != 0;
  const int all_units = past ? 0 : uni(pre[n]);
  c.unit0 = c.tile = c.tiles = 0;
  c.step = workers;
  if (preT && small && all_units > 0) {
    const int T = uni(preT[n]), whole = T / workers * workers;
    // (8 T longest <= 9 units: the longest tile at most an eighth over the average)
    if (whole > 0 && (int64_t)T * uni(longest) * 8 <= (int64_t)all_units * 9) {
      c.tiles = whole;
      c.tile = ((int)blockIdx.x & 7) * (workers >> 3) + i;
      c.unit0 = all_units;
      if (whole < T) {   // the units before tile `whole`
        const int s = __popcll(__ballot(lane < n && preT[min(lane, n - 1) + 1] <= whole));
        const KvSeq q = kv_seq(a.kv, s);
        const uint32_t th = (uint32_t)(uni(preT[s + 1]) - uni(preT[s])) / (uint32_t)a.kv.H;
        const uint32_t hu = (uint32_t)(uni(pre[s + 1]) - uni(pre[s])) / (uint32_t)a.kv.H;
        const uint32_t rem = (uint32_t)(whole - uni(preT[s])), h = rem / th;
        int part = 0;
        for (int t = lane; t < (int)(rem - h * th); t += 64) part += tile_units<KU, TR>(a, q, t);
        c.unit0 = uni(pre[s]) + (int)(h * hu) + uni(wave_add(part));
      }
    }
  }
  const int total = all_units - c.unit0;
  // blocks b, b + 8, ... run on one XCD: give each XCD one contiguous eighth of
  // the ranges, so that the tiles that read the same keys share an L2
  c.blocks = min(total, workers);
  const int per = (c.blocks + 7) >> 3;
  const int L = ((int)blockIdx.x & 7) * per + i;
  c.block = L;
  c.pos = c.end = 0;
  if (i >= per || L >= c.blocks) return;
  c.each = (int)((uint32_t)total / (uint32_t)c.blocks);
  c.over = total - c.each * c.blocks;
  c.pos = c.begin_of(L);
  c.end = c.begin_of(L + 1);
  // the sequence of the first unit
  if (small) {
    c.seq = __popcll(__ballot(lane < n && pre[min(lane, n - 1) + 1] <= c.pos));
  } else {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= c.pos) lo = mid;
      else hi = mid;
    }
    c.seq = uni(lo);
  }
}

// The next piece of the range; advances c.  Sequences without units are passed.
// Every wave computes it for itself, with all its lanes.
template <int KU, int TR>
__device__ __forceinline__ bool next_piece(const AttendArgs& a, const int* pre, Cut& c, Piece& p,
                                           const int* preT = nullptr) {
  if (preT && c.tile < c.tiles) {
    const int n = a.kv.n_seqs, lane = threadIdx.x & 63;
    p.seq = __popcll(__ballot(lane < n && preT[min(lane, n - 1) + 1] <= c.tile));
    p.q = kv_seq(a.kv, p.seq);
    p.q.q0 = uni(p.q.q0);
    p.q.q_len = uni(p.q.q_len);
    p.q.base = uni(p.q.base);
    p.q.end = uni(p.q.end);
    const uint32_t th = (uint32_t)(p.q.q_len * a.group + TR - 1) / (uint32_t)TR;
    const uint32_t rem = (uint32_t)(c.tile - uni(preT[p.seq]));
    p.head = (int)(rem / th);
    p.row0 = (int)(rem - p.head * th) * TR;
    p.rows = min(TR, p.q.q_len * a.group - p.row0);
    tile_keys<KU>(a, p.q, p.row0, p.rows, p.key0, p.key1);
    p.begins = p.ends = true;
    p.start = 0;
    p.first = -1;   // no piece of the range
    c.tile += c.step;
    return true;
  }
  if (c.pos >= c.end) return false;
  while (uni(pre[c.seq + 1]) <= c.pos) ++c.seq;
  p.seq = c.seq;
  p.q = kv_seq(a.kv, c.seq);
  p.q.q0 = uni(p.q.q0);
  p.q.q_len = uni(p.q.q_len);
  p.q.base = uni(p.q.base);
  p.q.end = uni(p.q.end);
  const int before = uni(pre[c.seq]);
  const uint32_t hu = (uint32_t)(uni(pre[c.seq + 1]) - before) / (uint32_t)a.kv.H;
  p.head = (int)((uint32_t)(c.pos - before) / hu);
  int rem = c.pos - before - p.head * (int)hu;
  const int rows = p.q.q_len * a.group;
  int tile = 0;
  if (rows > TR) {
    const int lane = threadIdx.x & 63;
    for (;; tile += 64) {
      int sum = tile_units<KU, TR>(a, p.q, tile + lane);
      const int own = sum;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int z = __shfl_up(sum, d);
        if (lane >= d) sum += z;
      }
      const unsigned long long past = __ballot(sum > rem);
      if (past) {
        const int at = __builtin_ctzll(past);
        rem -= __shfl(sum - own, at);
        tile += at;
        break;
      }
      rem -= __shfl(sum, 63);
    }
    tile = uni(tile);
    rem = uni(rem);
  }
  p.row0 = tile * TR;
  p.rows = min(TR, rows - p.row0);
  int lo = 0, hi = 0;
  tile_keys<KU>(a, p.q, p.row0, p.rows, lo, hi);
  const int units = (hi - lo + KU - 1) / KU;
  const int take = min(c.end - c.pos, units - rem);
  p.begins = rem == 0;
  p.ends = rem + take == units;
  p.key0 = lo + rem * KU;
  p.key1 = p.ends ? hi : p.key0 + take * KU;
  p.start = c.pos - rem;
  p.first = p.begins ? c.block : c.block_of(p.start);
  c.pos += take;
  return true;
}

// Partial results of a block: slot 0 its first piece, slot 1 its last one if
// that is another.
template <int TR, int D>
struct Parts {
  static __host__ __device__ size_t desc_bytes(int G) { return (size_t)G * (sizeof(PartDesc) + sizeof(int)); }
  static __host__ __device__ size_t ml_bytes(int G) { return (size_t)G * 2 * TR * 2 * sizeof(float); }
  static __host__ __device__ size_t o_bytes(int G) { return (size_t)G * 2 * TR * D * sizeof(float); }
  PartDesc* desc;
  int* items;   // of each desc, for the list of the joining launch
  float2* ml;   // [slot][row]: maximum (log2 scale), sum
  float* o;     // [slot][row][D]
  __device__ Parts(char* ws, int G) {
    desc = reinterpret_cast<PartDesc*>(ws);
    items = reinterpret_cast<int*>(ws + G * sizeof(PartDesc));
    ml = reinterpret_cast<float2*>(ws + desc_bytes(G));
    o = reinterpret_cast<float*>(ws + desc_bytes(G) + ml_bytes(G));
  }
};

// Tell the joining launch about this block's first piece: a tile's parts are
// joined by the block whose first piece is the last of several.  One lane.
__device__ __forceinline__ void describe(PartDesc* at, const Cut& c, const Piece* p) {
  PartDesc d{};
  d.last = -1;
  if (p && p->ends && !p->begins) {
    d.last = c.block;
    d.first = p->first;
    // the first part is its block's first piece iff that block's range begins with the tile
    d.first_slot = c.begin_of(p->first) == p->start ? 0 : 1;
    d.head = p->head;
    d.row0 = p->row0;
    d.rows = p->rows;
    d.q0 = p->q.q0;
  }
  *at = d;
}

// Maximum of three in one instruction (fmaxf would quiet every operand first).  A
// NaN among them is the result: then the running maximum stays, and the row's sum
// becomes NaN by the exponential.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }

// What an infinity or NaN in V does to a row that sees its token: the result's element
// is that value, whatever its weight (NaN where they differ).  The products of tiles
// that all rows see whole, and factors that round to 0 later, make NaN of some (0 *
// inf: of a weight or a second term that has rounded to 0), but never hide one: an
// element is finite only if all that its row saw of V was.  So the elements of a
// piece that are not finite are settled at its end by a look at their column of V,
// and where all is finite nothing is looked at.  FP8 has NaN only, and needs none of this.
template <typename A>
__device__ __forceinline__ uint32_t classes_of(const u32x4& u, uint32_t see) {   // bits: +inf, -inf, NaN
  uint32_t found = 0;
#pragma unroll
  for (int cls = 0; cls < 3; ++cls) found |= (class_bits<A>(u, cls) & see) ? 1u << cls : 0u;
  return found;
}
// Eight tokens' values of the head's first element, from token t on (a multiple of 8), and
// which of them lie in [lo, hi] and have pages.
__device__ __forceinline__ const char* eight_values(const KvView& kv, const int32_t* ktab, const int32_t* vtab, int D,
                                                    int t, int lo, int hi, uint32_t& see) {
  const int b = (int)kv_div(kv, (uint32_t)t);
  const bool in = t <= hi && b < kv.nb;
  const int kp = in ? ktab[b] : -1, vp = in ? vtab[b] : -1;
  const bool ok = (unsigned)kp < (unsigned)kv.n_pages && (unsigned)vp < (unsigned)kv.n_pages;
  see = ok ? run_bits<8>(t, lo, hi) : 0u;
  return kv.pages + (int64_t)(ok ? vp : 0) * kv.page_bytes + (int64_t)(ok ? (t - b * kv.T) / 8 : 0) * D * 16;
}
// The wave's results o of rows that see the tokens lo .. hi of a piece's keys each and
// [all_lo, all_hi] in common (the same in all lanes): element i of o[n] is number
// dim(n E + i) of the head's.  Only lanes with `mine` are settled (a row whose scores are
// not finite is NaN).  The common tokens are walked once, all columns at a
// time; the few others of a row (as many as the wave's rows are apart) by its lanes.
template <typename A, int D, typename V, int N, typename Dim>
__device__ __forceinline__ void settle(const KvView& kv, const int32_t* ktab, const int32_t* vtab, int lo, int hi,
                                       int all_lo, int all_hi, bool mine, V (&o)[N], Dim dim) {
  constexpr int E = sizeof(V) / sizeof(float), C = D / 64, U = 4;
  const int lane = threadIdx.x & 63;
  uint32_t found[C] = {};
#pragma unroll 1
  for (int t0 = all_lo & ~7; t0 <= all_hi; t0 += 8 * U) {
    u32x4 u[U][C];
    uint32_t see[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const char* src = eight_values(kv, ktab, vtab, D, t0 + 8 * j, all_lo, all_hi, see[j]);
#pragma unroll
      for (int c = 0; c < C; ++c) u[j][c] = ldv(src + (c * 64 + lane) * 16);
    }
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int c = 0; c < C; ++c) found[c] |= classes_of<A>(u[j][c], see[j]);
  }
  unsigned long long column[3][C];   // of all columns, in every lane
#pragma unroll
  for (int cls = 0; cls < 3; ++cls)
#pragma unroll
    for (int c = 0; c < C; ++c) column[cls][c] = __ballot((found[c] >> cls) & 1u);
  const bool common = all_lo <= all_hi;
  uint64_t odd = 0, is[3] = {};
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < E; ++i) odd |= (uint64_t)(mine && !(fabsf(o[n][i]) < INFINITY)) << (n * E + i);
#pragma unroll 1
  for (uint64_t left = odd; left; left &= left - 1) {
    const int bit = __builtin_ctzll(left), d = dim(bit);
    uint32_t f = 0;
#pragma unroll
    for (int cls = 0; cls < 3; ++cls) {
      unsigned long long w = column[cls][0];
      if (C > 1 && d >= 64) w = column[cls][C - 1];
      f |= (uint32_t)((w >> (d & 63)) & 1u) << cls;
    }
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      const int from = side ? (common ? max(all_hi + 1, lo) : hi + 1) : lo;
      const int to = side ? hi : (common ? min(all_lo - 1, hi) : hi);
#pragma unroll 1
      for (int t = from & ~7; t <= to; t += 8) {
        uint32_t see;
        const char* src = eight_values(kv, ktab, vtab, D, t, from, to, see);
        f |= classes_of<A>(ldv(src + d * 16), see);
      }
    }
#pragma unroll
    for (int cls = 0; cls < 3; ++cls)
      is[cls] |= (uint64_t)(cls < 2 ? f == 1u << cls : f > 2) << bit;
  }
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < E; ++i)
#pragma unroll
      for (int cls = 0; cls < 3; ++cls)
        if ((is[cls] >> (n * E + i)) & 1u) o[n][i] = class_value(cls);
}
// NaN if one of the values is not finite, else 0.
template <typename V, int N, int E = sizeof(V) / sizeof(float)>
__device__ __forceinline__ float residue(const V (&o)[N]) {
  float z[4] = {0.f, 0.f, 0.f, 0.f};   // (in four chains, none of which waits for another)
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < E; ++i) z[i & 3] = __builtin_fmaf(o[n][i], 0.f, z[i & 3]);
  return (z[0] + z[1]) + (z[2] + z[3]);
}
// The weight of a part's sums, above 0 where it has rounded to 0, so that an infinity
// among them stays one: the least number instead, which makes less than 2^-20 of any
// finite sum.  (A branch for it in the joins costs 2 us of 5, a selection 0.3.)
__device__ __forceinline__ float weight(float w) { return fmaxf(w, 0x1p-149f); }

// ---- the joining launch ----------------------------------------------------------
// RB rows a block: weights of the parts by their maxima, then a
// weighted sum, D / 4 lanes a part and several parts at a time.  Bound by the reads
// of the parts; each is a contiguous D * 4 bytes.  Measured 3.1 us (one token of 517,
// 32 heads, 2.3 at the least) to 8 us (32 sequences of 40 rows, 8 heads).
template <typename A, int D, int TR, int RB>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a, int G) {
  constexpr int LR = D / 4, PG = 256 / RB / LR;            // lanes of a part, parts at a time
  constexpr int RW = 256 / RB < 64 ? 256 / RB : 64;        // lanes of a row in a wave
  __shared__ __align__(16) f32x4 sh_acc[4][LR];
  __shared__ float sh_sum[4];
  const Parts<TR, D> parts(a.ws, G);
  const PartDesc d = parts.desc[blockIdx.x];
  const int L = d.last;
  if (L < 0) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int li = tid % LR, pg = tid % (256 / RB) / LR;
  auto slot = [&](int j) { return (int64_t)(2 * j + (j == d.first ? d.first_slot : 0)) * TR; };
  for (int r0 = blockIdx.y * RB; r0 < d.rows; r0 += gridDim.y * RB) {
    const int r = r0 + tid / (256 / RB);
    const bool in = r < d.rows;
    float M = -INFINITY;
    if (in)
      for (int j = d.first + lane % RW; j <= L; j += RW) M = fmaxf(M, parts.ml[slot(j) + r].x);
#pragma unroll
    for (int x = RW / 2; x; x >>= 1) M = fmaxf(M, __shfl_xor(M, x));
    const float Mu = safe_max(M);
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
    if (in)
#pragma unroll 4
      for (int j = d.first + pg; j <= L; j += PG) {
        const int64_t at = slot(j) + r;
        const float2 ml = parts.ml[at];
        const float w = exp2f(ml.x - Mu);  // an empty part: exp2(-inf) = 0
        sum += w * ml.y;
        acc += weight(w) * *reinterpret_cast<const f32x4*>(parts.o + at * D + li * 4);
      }
#pragma unroll
    for (int x = LR; x < RW; x <<= 1) {
      sum += __shfl_xor(sum, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] += __shfl_xor(acc[i], x);
    }
    if constexpr (RB < 4) {   // the row's other waves
      if (lane < LR) sh_acc[wave][li] = acc;
      if (lane == 0) sh_sum[wave] = sum;
      __syncthreads();
      if (wave % (4 / RB) == 0) {
#pragma unroll
        for (int w = 1; w < 4 / RB; ++w) {
          acc += sh_acc[wave + w][li];
          sum += sh_sum[wave + w];
        }
      }
      __syncthreads();
    }
    if (!in || pg != 0) continue;
    const int row = d.row0 + r;
    const int t = token_of(a, row), head = d.head * a.group + row - t * a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (sum == 0.f) acc = f32x4{0.f, 0.f, 0.f, 0.f};
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(d.q0 + t) * a.out_ld + (int64_t)head * D + li * 4;
    *reinterpret_cast<uint2*>(out) = uint2{pack2<A>(acc[0] * inv, acc[1] * inv), pack2<A>(acc[2] * inv, acc[3] * inv)};
    if (a.lse && li == 0)
      a.lse[(int64_t)(d.q0 + t) * a.n_q_heads + head] = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
  }
}

// The same for few tiles of 128 rows with very many parts: the rows of all tiles that have parts are items of one list,
// which the blocks take in turn.  The NG groups of D / 4 lanes of a block take NG /
// P rows at a time, P groups the parts of each, where P leaves a group four parts
// or more (PartDesc::share).
template <typename A, int D, int TR>
__global__ __launch_bounds__(256) void k_attend_join_list(AttendArgs a, int G) {
  constexpr int LR = D / 4, NG = 256 / LR, W = 4, MAXG = 1024;
  __shared__ __align__(16) f32x4 sh_acc[NG][LR];
  __shared__ float sh_sum[NG];
  __shared__ int pre[MAXG + 1], wsum[W];
  const Parts<TR, D> parts(a.ws, G);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int li = tid % LR, gi = tid / LR;
  int run = 0;
  for (int g0 = 0; g0 < G; g0 += 256) {
    int sum = g0 + tid < G ? parts.items[g0 + tid] : 0;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int z = __shfl_up(sum, d);
      if (lane >= d) sum += z;
    }
    if (lane == 63) wsum[wave] = sum;
    __syncthreads();
    int all = 0;
    for (int w = 0; w < W; ++w) {
      if (w < wave) sum += wsum[w];
      all += wsum[w];
    }
    if (g0 + tid < G) pre[g0 + tid + 1] = run + sum;
    run += all;
    __syncthreads();
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  for (int it = blockIdx.x; it < run; it += gridDim.x) {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pre[mid] <= it) lo = mid;
      else hi = mid;
    }
    const PartDesc d = parts.desc[lo];
    const int L = d.last, P = d.share, R = NG / P;
    const int r = (it - pre[lo]) * R + gi / P, pg = gi % P;
    const bool in = r < d.rows;
    auto slot = [&](int j) { return (int64_t)(2 * j + (j == d.first ? d.first_slot : 0)) * TR; };
    float M = -INFINITY;
    if (in)
      for (int j = d.first + li; j <= L; j += LR) M = fmaxf(M, parts.ml[slot(j) + r].x);
#pragma unroll
    for (int x = LR / 2; x; x >>= 1) M = fmaxf(M, __shfl_xor(M, x));
    const float Mu = safe_max(M);
    f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
    float sum = 0.f;
    if (in)
#pragma unroll 4
      for (int j = d.first + pg; j <= L; j += P) {
        const int64_t at = slot(j) + r;
        const float2 ml = parts.ml[at];
        const float w = exp2f(ml.x - Mu);
        sum += w * ml.y;
        acc += weight(w) * *reinterpret_cast<const f32x4*>(parts.o + at * D + li * 4);
      }
    if (P > 1) {
      sh_acc[gi][li] = acc;
      if (li == 0) sh_sum[gi] = sum;
      __syncthreads();
      if (pg == 0)
        for (int k = 1; k < P; ++k) {
          acc += sh_acc[gi + k][li];
          sum += sh_sum[gi + k];
        }
      __syncthreads();
    }
    if (!in || pg != 0) continue;
    const int row = d.row0 + r;
    const int t = token_of(a, row), head = d.head * a.group + row - t * a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (sum == 0.f) acc = f32x4{0.f, 0.f, 0.f, 0.f};
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(d.q0 + t) * a.out_ld + (int64_t)head * D + li * 4;
    *reinterpret_cast<uint2*>(out) = uint2{pack2<A>(acc[0] * inv, acc[1] * inv), pack2<A>(acc[2] * inv, acc[3] * inv)};
    if (a.lse && li == 0)
      a.lse[(int64_t)(d.q0 + t) * a.n_q_heads + head] = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
  }
}

// ---- up to 16 rows ---------------------------------------------------------------
// K and V go from memory to registers (every byte is used once: LDS would only add
// a trip).  A wave's tile is 4 E keys: 16 KB at D = 128, its next pieces loaded
// as soon as the products have taken the last ones.  With few (sequence, head)
// pairs the four waves of a block take a tile of rows together, each every fourth
// tile of keys, and join their results in LDS; with many (SOLO) every wave works
// for itself, its range of the units cut as the blocks' ones are: no wave waits
// for another, and short sequences take their turns on 4 times as many workers.
// Measured: 64 sequences of 20 to 2048 tokens, 32 heads of 128, bf16, 1.15 GB of K and
// V, 213 us, 5.4 TB/s; 3 of 40001 to 131071 tokens, 8 heads for 64, FP8, 600 MB, 115 us,
// 5.2 TB/s (a device copy of 1 GiB moves 4.8 TB/s, a sum reads 4.0); one of 517 tokens,
// 32 heads, 9.7 us, of which two empty launches are 4.6.
template <typename A, typename KV, int D, bool SOLO>
struct Skinny {
  static constexpr bool Q8 = is_quant<KV>();
  static constexpr int E = ET<KV>::E;
  static constexpr int KT = 4 * E;       // keys of a wave's tile
  static constexpr int KU = SOLO ? KT : 4 * KT;   // keys of a unit
  static constexpr int TR = 16;
  static constexpr int NT = E / 4;       // K operands of 16 tokens
  static constexpr int NC = D / (4 * E); // 16-byte pieces of a K row a lane loads
  static constexpr int ND = D / 16;      // 16-element blocks of the head dimension
  static constexpr int NQ = D / 32;      // k steps of the first product
  using PT = typename std::conditional<Q8, bf16_t, A>::type;  // type of P and V in the second one
};

template <typename A, typename KV, int D, bool SOLO>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_attend_rows(AttendArgs a) {
  using S = Skinny<A, KV, D, SOLO>;
  using PT = typename S::PT;
  constexpr int E = S::E, KT = S::KT, KU = S::KU, TR = S::TR, NT = S::NT, NC = S::NC, ND = S::ND;
  constexpr bool Q8 = S::Q8;
  __shared__ int pre[kKvMaxSeqs + 1 + 4];
  __shared__ float sh_ml[SOLO ? 1 : 4][TR][2];
  __shared__ __align__(16) float sh_o[SOLO ? 1 : 4][TR][D + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int col = lane & 15, g = lane >> 4;   // query column, lane group
  const KvView& kv = a.kv;
  Cut c;
  const int workers = SOLO ? 4 * (int)gridDim.x : (int)gridDim.x;
  cut_work<KU, TR, 256>(a, pre, c, workers, SOLO ? ((int)blockIdx.x >> 3) * 4 + wave : (int)blockIdx.x >> 3);
  const Parts<TR, D> parts(a.ws, workers);
  PartDesc* desc = parts.desc + (SOLO ? (int)blockIdx.x * 4 + wave : (int)blockIdx.x);
  const bool speaker = SOLO ? lane == 0 : tid == 0;
  Piece p;
  int n_piece = 0;
  if (c.pos >= c.end && speaker) describe(desc, c, nullptr);
  while (next_piece<KU, TR>(a, pre, c, p)) {
    // ---- queries: operand B of the first product, column = row of the tile
    const int row = p.row0 + min(col, p.rows - 1);
    const int tq = token_of(a, row);
    const int pos = p.q.base + tq;
    const int posmin = p.q.base + token_of(a, p.row0);
    const int posmax = p.q.base + token_of(a, p.row0 + p.rows - 1);
    const int win = a.window > 0 ? a.window : 0x40000000;
    u32x4 qf[S::NQ];
    {
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(p.q.q0 + tq) * a.q_ld +
                           (int64_t)(p.head * a.group + row - tq * a.group) * D;
#pragma unroll
      for (int i = 0; i < S::NQ; ++i) {
        // 16 bits: piece c = 4 i + g of 8 elements; FP8: half i & 1 of piece 4 (i / 2) + g of 16
        const int d = Q8 ? (4 * (i >> 1) + g) * 16 + (i & 1) * 8 : (4 * i + g) * 8;
        qf[i] = ldv(qp + d);
      }
    }
    const int32_t* ktab = kv.table + ((int64_t)p.seq * 2 * kv.H + p.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    // the lane's tokens of a tile: K operand t's row col is token (col / 4) E + 4 t + col % 4,
    // so that the lane's scores are those of tokens g E .. g E + E - 1
    const int ktok = (col >> 2) * E + (col & 3);
    f32x4 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, l = 0.f;

    // page of the lane's K tokens (they lie in one aligned group of E) and of its V group
    struct Ids {
      int kp, vp, slot, vslot;
    };
    const int nblk = kv.nb;
    auto find = [&](int tile) {
      Ids r;
      const int kt = tile + (col >> 2) * E, vt = tile + g * E;
      const int kb = (int)kv_div(kv, (uint32_t)kt), vb = (int)kv_div(kv, (uint32_t)vt);
      r.slot = kt - kb * kv.T + (col & 3);
      r.vslot = vt - vb * kv.T;
      r.kp = kb < nblk ? ktab[kb] : -1;
      r.vp = vb < nblk ? vtab[vb] : -1;
      return r;
    };
    u32x4 kf[NT][NC], vf[ND];
    u32x4 kscale, vscale;
    auto load_k = [&](const Ids& id) {
      const bool ok = (unsigned)id.kp < (unsigned)kv.n_pages;
      const char* base = kv.pages + (int64_t)(ok ? id.kp : 0) * kv.page_bytes + (g * kv.T + id.slot) * 16;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int t = 0; t < NT; ++t) kf[t][n] = ldv(base + (n * 4 * kv.T + 4 * t) * 16);
    };
    auto load_v = [&](const Ids& id) {
      const bool ok = (unsigned)id.vp < (unsigned)kv.n_pages;
      const char* base = kv.pages + (int64_t)(ok ? id.vp : 0) * kv.page_bytes +
                         ((int64_t)(id.vslot / E) * D + col) * 16;
#pragma unroll
      for (int n = 0; n < ND; ++n) vf[n] = ldv(base + n * 256);
      if (Q8) vscale = ldv(kv.scales + (int64_t)(ok ? id.vp : 0) * kv.T + id.vslot);
    };
    // scale bytes of the lane's score tokens: group g, which is the V group's token range
    auto load_ks = [&](int tile) {
      if (!Q8) return;
      const int vt = tile + g * E;
      const int vb = (int)kv_div(kv, (uint32_t)vt);
      const int kp = vb < nblk ? ktab[vb] : -1;
      const bool ok = (unsigned)kp < (unsigned)kv.n_pages;
      kscale = ldv(kv.scales + (int64_t)(ok ? kp : 0) * kv.T + (vt - vb * kv.T));
    };

    int tile = p.key0 + (SOLO ? 0 : wave * KT);
    const bool any = tile < p.key1;
    Ids id, idn;
    if (any) {
      id = find(tile);
      load_k(id);
      load_ks(tile);
      load_v(id);
      idn = find(tile + KU);
    }
    for (; tile < p.key1; tile += KU) {
      const bool more = tile + KU < p.key1;
      const bool kbad = (unsigned)id.kp >= (unsigned)kv.n_pages, vbad = (unsigned)id.vp >= (unsigned)kv.n_pages;
      const bool edge = tile + KT - 1 > posmin || tile <= posmax - win || __ballot(kbad || vbad);
      uint32_t seen = 0xffffu;   // of the lane's tokens g E + e: seen by the lane's row
      if (edge) {
        // group g's K page is known to the lanes with col / 4 == g
        const unsigned long long kb = __ballot(kbad);
        const bool gone = vbad || ((kb >> (g * 4)) & 1);
        const int k0 = tile + g * E;
        seen = gone ? 0u : run_bits<E>(k0, pos - win + 1, pos);
        // what no row sees is taken out of V (0 times what lies there need not be 0);
        // values that are not finite go to the rows that see them, then they leave V
        const uint32_t live = gone ? 0u : run_bits<E>(k0, posmin - win + 1, min(posmax, p.key1 - 1));
        uint32_t odd = 0;
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          vf[n] = Q8 ? keep16b(vf[n], live) : keep8(vf[n], live);
          odd |= Q8 ? nan_codes(vf[n]) : not_finite<A>(vf[n]);
        }
        if (Q8) vscale = keep16b(vscale, live);
        if (__builtin_expect(__ballot(odd != 0) != 0, 0)) {
#pragma unroll
          for (int n = 0; n < ND; ++n)
#pragma unroll 1
            for (int q = 0; q < E / 8; ++q) {
              const u32x4 vis = ones8<PT>(seen >> (8 * q));
              const u32x4 v = Q8 ? (q ? fp8_to16<PT>(vf[n].z, vf[n].w) : fp8_to16<PT>(vf[n].x, vf[n].y)) : vf[n];
#pragma unroll 1
              for (int cls = 0; cls < 3; ++cls) {
                const f32x4 hit = mfma16<PT>(ones8<PT>(class_bits<PT>(v, cls)), vis, f32x4{0.f, 0.f, 0.f, 0.f});
                const float val = class_value(cls);
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] += hit[i] > 0.f ? val : 0.f;
              }
            }
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            if constexpr (Q8) {
              vf[n] = keep16b(vf[n], ~(class_bits<PT>(fp8_to16<PT>(vf[n].x, vf[n].y), 3) |
                                       class_bits<PT>(fp8_to16<PT>(vf[n].z, vf[n].w), 3) << 8));
            } else {
              vf[n] = keep8(vf[n], ~class_bits<A>(vf[n], 3));
            }
          }
        }
      }
      // ---- S^T = K Q^T
      f32x4 s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          if constexpr (Q8) {
            s[t] = mfma16<A>(fp8_to16<A>(kf[t][n].x, kf[t][n].y), qf[2 * n], s[t]);
            s[t] = mfma16<A>(fp8_to16<A>(kf[t][n].z, kf[t][n].w), qf[2 * n + 1], s[t]);
          } else {
            s[t] = mfma16<A>(kf[t][n], qf[n], s[t]);
          }
        }
      if constexpr (Q8) {
        const uint32_t w[4] = {kscale.x, kscale.y, kscale.z, kscale.w};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] *= __uint_as_float(((w[t] >> (8 * i)) & 0xffu) << 23);
      }
      // the ids after next are asked for ahead of the V loads: waiting for them
      // does not wait for those
      Ids idn2 = idn;
      if (more) {
        load_k(idn);
        load_ks(tile + KU);
        idn2 = find(tile + 2 * KU);
      }
      if (edge) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (4 * t + i)) & 1)) s[t][i] = -INFINITY;
      }
      // ---- running maximum and sum
      float top = s[0][0];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        top = max3(top, s[t][0], s[t][1]);
        top = max3(top, s[t][2], s[t][3]);
      }
      top = max3(top, __shfl_xor(top, 16), top);
      top = max3(top, __shfl_xor(top, 32), top);
      top *= a.scale_log2;
      // the maximum follows only when it would grow by more than 8 (a factor of
      // 256, which every type of P holds): else no rescaling
      if (__ballot(top > m + 8.f)) {
        const float mn = top > m ? top : m;
        const float f = m == -INFINITY ? 1.f : exp2f(m - mn);   // (nothing yet, or what is not finite)
        l *= f;
#pragma unroll
        for (int n = 0; n < ND; ++n) o[n] *= f;
        m = mn;
      }
      const float mu = origin<PT>(m);
      float pr[4 * NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          l += pr[4 * t + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], a.scale_log2, -mu));
      if constexpr (Q8) {
        const uint32_t w[4] = {vscale.x, vscale.y, vscale.z, vscale.w};
#pragma unroll
        for (int e = 0; e < 16; ++e) pr[e] *= __uint_as_float(((w[e / 4] >> (8 * (e & 3))) & 0xffu) << 23);
      }
      u32x4 pf[E / 8], pl[E / 8];
#pragma unroll
      for (int q = 0; q < E / 8; ++q) p_operand<PT>(pr + 8 * q, pf[q], pl[q]);
      // ---- O^T += V^T P^T
#pragma unroll
      for (int n = 0; n < ND; ++n) {
        if constexpr (Q8) {
          const u32x4 v0 = fp8_to16<PT>(vf[n].x, vf[n].y), v1 = fp8_to16<PT>(vf[n].z, vf[n].w);
          o[n] = mfma16<PT>(v0, pf[0], o[n]);
          o[n] = mfma16<PT>(v1, pf[E / 8 - 1], o[n]);
          o[n] = mfma16<PT>(v0, pl[0], o[n]);
          o[n] = mfma16<PT>(v1, pl[E / 8 - 1], o[n]);
        } else {
          o[n] = mfma16<PT>(vf[n], pf[0], o[n]);
          o[n] = mfma16<PT>(vf[n], pl[0], o[n]);
        }
      }
      if (more) {
        load_v(idn);
        id = idn;
        idn = idn2;
      }
    }
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (std::is_same<PT, f16_t>::value) m -= 7.f;   // the exponents' origin
    if constexpr (!Q8) {
      const bool mine = residue(o) != 0.f && l < INFINITY;
      if (__builtin_expect(__ballot(mine) != 0, 0))
        settle<A, D>(kv, ktab, vtab, max(pos - win + 1, p.key0), min(pos, p.key1 - 1), max(posmax - win + 1, p.key0),
                     min(posmin, p.key1 - 1), mine, o, [&](int bit) { return (bit >> 2) * 16 + 4 * g + (bit & 3); });
    }
    if constexpr (SOLO) {
      const int slot = n_piece == 0 ? 0 : 1;
      if (col < p.rows) {
        if (p.begins && p.ends) {
          const int head = p.head * a.group + row - tq * a.group;
          const float inv = l == 0.f ? 0.f : 1.f / l;
          uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(p.q.q0 + tq) * a.out_ld + (int64_t)head * D + 4 * g;
#pragma unroll
          for (int n = 0; n < ND; ++n) {
            const f32x4 x = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f} : o[n];
            *reinterpret_cast<uint2*>(out + 16 * n) = uint2{pack2<A>(x[0] * inv, x[1] * inv), pack2<A>(x[2] * inv, x[3] * inv)};
          }
          if (a.lse && g == 0)
            a.lse[(int64_t)(p.q.q0 + tq) * a.n_q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
        } else {
          const int64_t at = ((int64_t)c.block * 2 + slot) * TR + col;
#pragma unroll
          for (int n = 0; n < ND; ++n) *reinterpret_cast<f32x4*>(parts.o + at * D + 16 * n + 4 * g) = o[n];
          if (g == 0) parts.ml[at] = float2{m, l};
        }
      }
      if (n_piece == 0 && speaker) describe(desc, c, &p);
      ++n_piece;
      continue;
    }
    // ---- the waves' results
    if (lane < 16) {
      sh_ml[SOLO ? 0 : wave][col][0] = m;
      sh_ml[SOLO ? 0 : wave][col][1] = l;
    }
    if (col < p.rows)
#pragma unroll
      for (int n = 0; n < ND; ++n) *reinterpret_cast<f32x4*>(&sh_o[SOLO ? 0 : wave][col][16 * n + 4 * g]) = o[n];
    __syncthreads();
    const bool whole = p.begins && p.ends;
    const int slot = n_piece == 0 ? 0 : 1;
    for (int i = tid; i < p.rows * (D / 4); i += 256) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < (SOLO ? 1 : 4); ++w) M = fmaxf(M, sh_ml[w][r][0]);
      const float Mu = safe_max(M);
      float sum = 0.f;
      f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < (SOLO ? 1 : 4); ++w) {
        const float f = exp2f(sh_ml[w][r][0] - Mu);
        sum += f * sh_ml[w][r][1];
        acc += weight(f) * *reinterpret_cast<const f32x4*>(&sh_o[w][r][d]);
      }
      if (whole) {
        const int rr = p.row0 + r, t = token_of(a, rr), head = p.head * a.group + rr - t * a.group;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        if (sum == 0.f) acc = f32x4{0.f, 0.f, 0.f, 0.f};
        uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(p.q.q0 + t) * a.out_ld + (int64_t)head * D + d;
        *reinterpret_cast<uint2*>(out) = uint2{pack2<A>(acc[0] * inv, acc[1] * inv), pack2<A>(acc[2] * inv, acc[3] * inv)};
        if (a.lse && d == 0)
          a.lse[(int64_t)(p.q.q0 + t) * a.n_q_heads + head] = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
      } else {
        const int64_t at = ((int64_t)c.block * 2 + slot) * TR + r;
        *reinterpret_cast<f32x4*>(parts.o + at * D + d) = acc;
        if (d == 0) parts.ml[at] = float2{M, sum};
      }
    }
    if (n_piece == 0 && speaker) describe(desc, c, &p);
    ++n_piece;
    __syncthreads();
  }
}

// ---- more rows -------------------------------------------------------------------
// Tiles of 128 or 256 rows: four or eight waves of 32, which share tiles of 64 keys
// through LDS (two slots, one barrier a tile).  The LDS image is the 16-bit pages' own
// order, [piece][token] and [token group][element] of 16 bytes, so that operand reads
// are contiguous over lanes and free of bank conflicts; 16-bit pages are loaded there
// directly, FP8 ones through registers, where the codes get their scales (2 scales
// a pair of V codes, one a K row: the products and the softmax then know nothing
// of FP8).
//
// Of 64 keys of 128 elements a wave's 32 rows cost 1024 cycles of the matrix cores and
// about 1130 of the vector ALUs (32 exponentials of 16 cycles, about 150 other
// instructions a lane): only what overlaps is fast.  Two waves share a SIMD.
//   Four waves (short work): two blocks share a CU, drifting apart because no barrier
// ties them; a tile's products and its exponentials overlap within the second product
// only.  P goes in two 16-bit terms: the results are as near as fp32 weights make them,
// and the matrix cores wait for loads anyway (measured in turn, one term / two: 32 x 5 over
// 900 to 4100 tokens, 64 heads on 8, 86.3 / 88.4 us; 4 x 128 over 2000 70.2 / 82.0; 16 x 300
// over 300 of 32 heads on 32 68.2 / 72.3; 15 heads of 64 in a window of 1000, 1 to 255 new
// tokens each, 59.1 / 65.6).  2048 over 16384 tokens, 64 heads on 8, bf16, takes 1490 us.
//   Eight waves (long work): a step weaves the exponentials of one tile with its second
// product and the first product of the next tile, and spreads the loads among them (4390
// cycles a pair of wave tiles; that chunk 950 to 1000 us by the card's clock, 1030 to 1086
// TFLOP/s: a matrix product of 8192^3 runs at 1236).  The loads to LDS arrive at 53 bytes a
// cycle and CU, and issuing a tile's at once stops a wave for 600 to 1300 cycles; 256 rows
// halve them a row.  P goes in one term here, because the matrix cores bound the kernel:
// with two the chunk takes 1493 us against 1011 in turn, and what one costs is that an
// output's error grows from its own rounding's to 1.4 times that.  A caller who wants two
// gets four waves, which take as long.
__device__ __forceinline__ void load_lds16(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

// Eight FP8 codes times a power of two -> eight 16-bit values.
template <typename T>
__device__ __forceinline__ u32x4 fp8_to16s(uint32_t w0, uint32_t w1, float sc) {
  u32x4 r;
  if constexpr (std::is_same<T, bf16_t>::value) {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, sc, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, sc, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, sc, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, sc, true));
  } else {
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, sc, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w0, sc, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, sc, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w1, sc, true));
  }
  return r;
}
// Eight codes of eight tokens, each times its token's power of two (scale bytes
// s0, s1), less `down` (0 or 1) in the exponent.
template <typename T>
__device__ __forceinline__ u32x4 fp8_to16v(uint32_t w0, uint32_t w1, uint32_t s0, uint32_t s1, int down) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? w0 : w1, sb = i < 2 ? s0 : s1;
    const float fa = scale_of((sb >> (16 * (i & 1))) & 0xffu, down);
    const float fb = scale_of((sb >> (16 * (i & 1) + 8)) & 0xffu, down);
    uint32_t a, b;
    if constexpr (std::is_same<T, bf16_t>::value) {
      a = __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, fa, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, fa, false));
      b = __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, fb, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, fb, false));
    } else {
      a = __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, fa, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, fa, false));
      b = __builtin_bit_cast(uint32_t, (i & 1) ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, fb, true)
                                               : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, fb, false));
    }
    o[i] = __builtin_amdgcn_perm(b, a, 0x07060100u);  // token 2 i of a, token 2 i + 1 of b
  }
  return u32x4{o[0], o[1], o[2], o[3]};
}

// The order of the products of a step beside its 32 exponentials: op below 64 is
// product n = op / 2 of half op % 2 of the next scores, else 64 + q ND + n block n of
// the output with the 16 tokens of step q, whose P is complete after exponential
// 8 q + 7.  at: the exponential before which it goes.
template <int NQ, int ND>
struct Weave {
  static constexpr int n = 2 * NQ + 4 * ND, ring = 4;
  struct Table {
    int op[n], at[n];
  };
  static constexpr Table make() {
    Table t{};
    constexpr int share[4] = {3, 2, 2, 1};
    int j = 0, k = 0;
    for (int q = 0; q < 4; ++q) {
      const int ks = share[q] * NQ / 4, vs = q ? ND : 0, all = ks + vs;
      for (int i = 0, ki = 0, vi = 0; i < all; ++i, ++j) {
        const bool key = vi == vs || (ki < ks && ki * vs <= vi * ks);
        if (key) ++ki, t.op[j] = k++;
        else t.op[j] = 64 + (q - 1) * ND + vi++;
        t.at[j] = 8 * q + i * 8 / all;
      }
    }
    for (int i = 0; i < ND; ++i, ++j) t.op[j] = 64 + 3 * ND + i, t.at[j] = 32;
    return t;
  }
  static constexpr Table table = make();
  static constexpr const int (&op)[n] = table.op;
  static constexpr const int (&at)[n] = table.at;
};

template <typename A, typename KV, int D, int NW>
struct Tiles {
  static constexpr int TR = 32 * NW, KU = 64, NS = 2;
  static constexpr int NIDS = 512;   // blocks of the page-id window in LDS
  struct Shared {
    u32x4 k[NS][D / 8][KU];
    u32x4 v[NS][KU / 8][D];
    int pre[kKvMaxSeqs + 1 + NW];
    int preT[64 + 1];
    int ids[2][NIDS];
  };
};

template <typename A, typename KV, int D, int NW>
__global__ __launch_bounds__(NW * 64) __attribute__((amdgpu_waves_per_eu(2, 2))) void k_attend_tiles(AttendArgs a) {
  using TT = Tiles<A, KV, D, NW>;
  constexpr bool Q8 = is_quant<KV>();
  constexpr int TR = TT::TR, KU = TT::KU, NIDS = TT::NIDS;
  constexpr int E = ET<KV>::E;
  constexpr int ND = D / 32, NQ = D / 16;
  constexpr int KL = D / E;                 // wave loads of K (and of V) of a tile
  constexpr int LPW = KL / NW;              // ... of a wave
  static_assert(KL % NW == 0, "loads divide over the waves");
  // f16 over FP8: values at half their size, so that the 65536 = 256 * 2^8 that codes of f16
  // rows may stand for fits; made good in the score's scale and in the output.  Halves of
  // less than 2^-14 are f16's subnormals: codes of rows whose largest value is below
  // 2^-6 may lose their last bits, 2^-24 at most, which is f16's own step there.
  constexpr int DOWN = Q8 && std::is_same<A, f16_t>::value ? 1 : 0;
  extern __shared__ __align__(16) char smem[];
  typename TT::Shared& sh = *reinterpret_cast<typename TT::Shared*>(smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hi = lane >> 5;
  const KvView& kv = a.kv;
  Cut c;
  cut_work<KU, TR, NW * 64>(a, sh.pre, c, (int)gridDim.x, (int)blockIdx.x >> 3, sh.preT);
  const Parts<TR, D> parts(a.ws, (int)gridDim.x);
  Piece p;
  int n_piece = 0;
  auto tell = [&](const Piece* q) {
    PartDesc* d = parts.desc + blockIdx.x;
    describe(d, c, q);
    constexpr int NG = 1024 / D;
    int n = 0;
    if (d->last >= 0) {
      int P = 1;
      while (P < NG && 8 * P <= d->last - d->first + 1) P *= 2;
      d->share = P;
      n = (d->rows * P + NG - 1) / NG;
    }
    parts.items[blockIdx.x] = n;
  };
  if (c.pos >= c.end && tid == 0) tell(nullptr);
  // row col of a K operand is this token of a tile of 32: a lane's 16 scores are
  // those of tokens hi * 8 .. + 7 and 16 + hi * 8 .. + 7
  const int ktok = (col >> 4) * 16 + ((col >> 2) & 1) * 8 + ((col >> 3) & 1) * 4 + (col & 3);
  const float sl = DOWN ? a.scale_log2 * 2.f : a.scale_log2;
  while (next_piece<KU, TR>(a, sh.pre, c, p, sh.preT)) {
    const int wrow0 = p.row0 + wave * 32;
    const int wrows = min(32, p.rows - wave * 32);   // <= 0: no rows of its own
    const int base = p.q.base;
    const int row = min(wrow0 + col, p.row0 + p.rows - 1);
    const int tq = token_of(a, row);
    const int pos = base + tq;
    const int win = a.window > 0 ? a.window : 0x40000000;
    const int posmin = base + token_of(a, wrow0);
    const int posmax = base + token_of(a, wrow0 + max(wrows, 1) - 1);
    u32x4 qf[NQ];
    {
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(p.q.q0 + tq) * a.q_ld +
                           (int64_t)(p.head * a.group + row - tq * a.group) * D + hi * 8;
#pragma unroll
      for (int i = 0; i < NQ; ++i) qf[i] = ldv(qp + 16 * i);
    }
    const int32_t* ktab = kv.table + ((int64_t)p.seq * 2 * kv.H + p.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    const int bmin = base + token_of(a, p.row0), bmax = base + token_of(a, p.row0 + p.rows - 1);
    // ---- page ids of the blocks from b0 on, in LDS (absent ones as they are).  Blocks
    // before the first row's window may be given back without any care
    const int vis0 = a.window > 0 ? bmin - a.window + 1 : 0;
    const int b_last = min((int)kv_div(kv, (uint32_t)max(p.key1 - 1, 0)), kv.nb - 1);
    int b0 = 0;
    bool any_bad = false;
    auto load_ids = [&](int tile) {
      b0 = (int)kv_div(kv, (uint32_t)tile);
      bool bad = false;
      for (int i = tid; i < 2 * NIDS; i += NW * 64) {
        const int w = i / NIDS, b = b0 + i % NIDS;
        int id = -1;
        if (b <= b_last) {
          id = (w ? vtab : ktab)[b];
          bad |= (unsigned)id >= (unsigned)kv.n_pages && (b + 1) * kv.T > vis0;
        }
        sh.ids[w][i % NIDS] = id;
      }
      // (of rows past the table every tile is taken as one with absent pages)
      any_bad = __syncthreads_or(bad || bmax >= p.q.end);
    };
    // ---- loads of one tile; lane = token for the page lookups
    u32x4 stk[Q8 ? LPW : 1], stv[Q8 ? LPW : 1], vsc[Q8 ? LPW : 1];
    float ksc = 0.f;
    // where a lane's token of K and V lies: page and slot of it
    int kpg = 0, kst = 0, vpg = 0, vst = 0;
    auto find = [&](int which, int tile, int& page, int& slot_of) {
      const int t = tile + lane, b = (int)kv_div(kv, (uint32_t)t);
      slot_of = t - b * kv.T;
      const int id = sh.ids[which][min(b - b0, NIDS - 1)];
      page = (unsigned)id < (unsigned)kv.n_pages ? id : 0;
    };
    auto load_k = [&](int i, int slot) {
      const char* src = kv.pages + (int64_t)kpg * kv.page_bytes + ((wave + i * NW) * kv.T + kst) * 16;
      if constexpr (!Q8) load_lds16(src, &sh.k[slot][wave + NW * i][0]);
      else stk[i] = ldv(src);
      if constexpr (Q8)
        if (i == 0) ksc = scale_of(kv.scales[(int64_t)kpg * kv.T + kst], DOWN);
    };
    auto load_v = [&](int i, int slot) {
      const int j = wave * LPW + i, gr = j * 64 / D, d0 = j * 64 % D;
      const int pg = __builtin_amdgcn_readlane(vpg, gr * E), s0 = __builtin_amdgcn_readlane(vst, gr * E);
      const char* src = kv.pages + (int64_t)pg * kv.page_bytes + ((s0 / E) * D + d0 + lane) * 16;
      if constexpr (!Q8) {
        load_lds16(src, &sh.v[slot][gr][d0]);
      } else {
        stv[i] = ldv(src);
        vsc[i] = ldv(kv.scales + (int64_t)pg * kv.T + s0);
      }
    };
    auto issue_k = [&](int tile, int slot) {
      find(0, tile, kpg, kst);
#pragma unroll
      for (int i = 0; i < LPW; ++i) load_k(i, slot);
    };
    auto issue_v = [&](int tile, int slot) {
      find(1, tile, vpg, vst);
#pragma unroll
      for (int i = 0; i < LPW; ++i) load_v(i, slot);
    };
    auto commit_k = [&](int slot) {   // FP8: what was loaded goes to LDS
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
          const int ch = wave + NW * i;
          sh.k[slot][2 * ch][lane] = fp8_to16s<A>(stk[i].x, stk[i].y, ksc);
          sh.k[slot][2 * ch + 1][lane] = fp8_to16s<A>(stk[i].z, stk[i].w, ksc);
        }
      }
    };
    auto commit_v = [&](int slot) {
      if constexpr (Q8) {
#pragma unroll
        for (int i = 0; i < LPW; ++i) {
          const int j = wave * LPW + i, gr = j * 64 / D, d = j * 64 % D + lane;
          sh.v[slot][2 * gr][d] = fp8_to16v<A>(stv[i].x, stv[i].y, vsc[i].x, vsc[i].y, DOWN);
          sh.v[slot][2 * gr + 1][d] = fp8_to16v<A>(stv[i].z, stv[i].w, vsc[i].z, vsc[i].w, DOWN);
        }
      }
    };
    f32x16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) o[i] = f32x16{};
    float m = -INFINITY, l = 0.f;
    load_ids(p.key0);
    issue_k(p.key0, 0);
    issue_v(p.key0, 0);
    commit_k(0);
    commit_v(0);
    // tiles from clean0 to before clean1 are seen whole by all rows of the block, if their pages are there
    const int clean1 = bmin - KU + 2, clean0 = a.window > 0 ? bmax - a.window + 1 : 0;
    auto is_edge = [&](int tile) { return tile < clean0 || tile >= clean1 || any_bad; };
    auto sees = [&](int tile) {   // this wave's rows see something of it
      return wrows > 0 && tile <= posmax && tile + KU - 1 > posmin - win;
    };
    // An edge tile's V before the products: tokens that no row of the block sees are
    // taken out in LDS (0 times what lies there need not be 0), and what is not finite
    // goes to the rows that see it.  Returns the tokens without pages.
    auto clean = [&](int tile, int slot) {
      unsigned long long bad = 0;
      if (__builtin_expect(any_bad, 0)) {
        const int b = (int)kv_div(kv, (uint32_t)(tile + lane)) - b0;
        bad = __ballot((unsigned)sh.ids[0][b] >= (unsigned)kv.n_pages ||
                       (unsigned)sh.ids[1][b] >= (unsigned)kv.n_pages);
      }
      const int first = max(bmin - win + 1 - tile, 0), last = min(bmax - tile, KU - 1);   // seen tokens
      unsigned long long alive = last >= first ? (~0ull >> (63 - last + first)) << first : 0;
      alive &= ~bad;
      u32x4* vt = &sh.v[slot][0][0];
      uint32_t odd = 0;
#pragma unroll 1
      for (int i = tid; i < KU / 8 * D; i += NW * 64) {
        const uint32_t byte = (uint32_t)(alive >> (i / D * 8)) & 0xffu;
        u32x4 v = vt[i];
        if (byte != 0xffu) {
          v = keep8(v, byte);
          vt[i] = v;
        }
        odd |= not_finite<A>(v);
      }
      if (__builtin_expect(__syncthreads_or(odd != 0), 0)) {
        // their values go to the rows that see their tokens, then they leave V
        if (wrows > 0)
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            const int k0 = (q >> 1) * 32 + (q & 1) * 16 + hi * 8;
            const u32x4 vis = ones8<A>(run_bits<8>(k0, pos - win + 1 - tile, pos - tile) & ~(uint32_t)(bad >> k0));
#pragma unroll
            for (int n = 0; n < ND; ++n) {
              const u32x4 v = sh.v[slot][2 * q + hi][n * 32 + col];
#pragma unroll 1
              for (int cls = 0; cls < 3; ++cls) {
                const f32x16 hit = mfma32<A>(ones8<A>(class_bits<A>(v, cls)), vis, f32x16{});
                const float val = class_value(cls);
#pragma unroll
                for (int r = 0; r < 16; ++r) o[n][r] += hit[r] > 0.f ? val : 0.f;
              }
            }
          }
        __syncthreads();
#pragma unroll 1
        for (int i = tid; i < KU / 8 * D; i += NW * 64) vt[i] = keep8(vt[i], ~class_bits<A>(vt[i], 3));
        __syncthreads();
      }
      return bad;
    };
    auto mask = [&](f32x16(&s)[2], int tile, unsigned long long bad) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int k0 = (h >> 1) * 32 + (h & 1) * 16 + hi * 8;
        const uint32_t seen = run_bits<8>(k0, pos - win + 1 - tile, pos - tile) & ~(uint32_t)(bad >> k0);
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (!((seen >> r) & 1)) s[h >> 1][8 * (h & 1) + r] = -INFINITY;
      }
    };
    auto top_of = [](const f32x16(&x)[2]) {
      float t = x[0][0];
#pragma unroll
      for (int r = 0; r < 16; ++r) t = max3(t, x[0][r], x[1][r]);
      return t;
    };
    // The running maximum follows the lane's largest score (and its partner's, which
    // has the row's other keys); returns what the exponentials subtract.
    auto follow = [&](float top) {
      const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
      top = __builtin_elementwise_maximum(__uint_as_float(both[0]), __uint_as_float(both[1])) * sl;
      if (__ballot(top > m + 8.f)) {
        const float mn = top > m ? top : m;
        const float f = m == -INFINITY ? 1.f : exp2f(m - mn);   // (nothing yet, or what is not finite)
        l *= f;
#pragma unroll
        for (int n = 0; n < ND; ++n) o[n] *= f;
        m = mn;
      }
      return origin<A>(m);
    };
    // the loads have arrived, of every wave (a barrier alone does not wait for loads
    // that go to LDS), and what the next ones will overwrite is read
    auto arrived = [&] {
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
      __syncthreads();
    };
    if constexpr (NW == 4) {
      int slot = 0;
      for (int tile = p.key0; tile < p.key1; tile += KU, slot ^= 1) {
        const bool more = tile + KU < p.key1;
        arrived();
        if (more) {
          if ((int)kv_div(kv, (uint32_t)(tile + 2 * KU - 1)) - b0 >= NIDS) load_ids(tile);
          issue_k(tile + KU, slot ^ 1);
          issue_v(tile + KU, slot ^ 1);
        }
        const bool edge = is_edge(tile);
        unsigned long long bad = 0;
        if (edge) bad = clean(tile, slot);
        if (sees(tile)) {
          // ---- S^T = K Q^T
          // in groups of four products, whose operands were read a group ahead (the
          // scheduler, left alone, reads each just before its use)
          f32x16 s[2] = {f32x16{}, f32x16{}};
          const u32x4* kp = &sh.k[slot][hi][ktok];   // piece 2 n of half kt: kp[2 * n * KU + kt * 32]
          u32x4 kf[2][4];
#pragma unroll
          for (int i = 0; i < 4; ++i) kf[0][i] = kp[2 * (i >> 1) * KU + (i & 1) * 32];
#pragma unroll
          for (int g = 0; g < NQ / 2; ++g) {
            if (g + 1 < NQ / 2) {
#pragma unroll
              for (int i = 0; i < 4; ++i) kf[(g + 1) & 1][i] = kp[2 * (2 * g + 2 + (i >> 1)) * KU + (i & 1) * 32];
            }
            __builtin_amdgcn_sched_barrier(0x6);
#pragma unroll
            for (int i = 0; i < 4; ++i) s[i & 1] = mfma32<A>(kf[g & 1][i], qf[2 * g + (i >> 1)], s[i & 1]);
            __builtin_amdgcn_sched_barrier(0x6);
          }
          if (edge) mask(s, tile, bad);
          const float mu = follow(top_of(s));
          u32x4 pf[4], pl[4];
          auto take_exp = [&](int q) {   // P of the 16 tokens of step q
            float pr[8];
#pragma unroll
            for (int r = 0; r < 8; ++r)
              l += pr[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[q >> 1][8 * (q & 1) + r], sl, -mu));
            p_operand<A>(pr, pf[q], pl[q]);
          };
          // ---- O^T += V^T P^T
          // the exponentials of one step and the operands' reads beside the products of
          // the step before
          const u32x4* vp = &sh.v[slot][hi][col];    // step q, block n: vp[2 * q * D + n * 32]
          u32x4 vf[2][ND];
#pragma unroll
          for (int n = 0; n < ND; ++n) vf[0][n] = vp[n * 32];
          take_exp(0);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            __builtin_amdgcn_sched_barrier(0);
            if (q < 3) {
#pragma unroll
              for (int n = 0; n < ND; ++n) vf[(q + 1) & 1][n] = vp[2 * (q + 1) * D + n * 32];
            }
#pragma unroll
            for (int n = 0; n < ND; ++n) o[n] = mfma32<A>(vf[q & 1][n], pf[q], o[n]);
#pragma unroll
            for (int n = 0; n < ND; ++n) o[n] = mfma32<A>(vf[q & 1][n], pl[q], o[n]);
            if (q < 3) take_exp(q + 1);
          }
        }
        if (more) {
          commit_k(slot ^ 1);
          commit_v(slot ^ 1);
        }
      }
    } else {
      float next_top = 0.f;   // of the lane's scores of the next tile, before they are masked
      // One tile, whose scores s the step before has computed; sn becomes the next tile's.
      // K is loaded two tiles ahead, V one.  The step before the first tile only does the
      // latter.
      auto step = [&](auto parity, f32x16(&s)[2], f32x16(&sn)[2], const int tile, const bool before) {
        constexpr int par = decltype(parity)::value;
        const bool kmore = tile + 2 * KU < p.key1, vmore = !before && tile + KU < p.key1;
        arrived();
        if (kmore && (int)kv_div(kv, (uint32_t)(tile + 3 * KU - 1)) - b0 >= NIDS) load_ids(max(tile, p.key0));
        const bool edge = !before && is_edge(tile);
        unsigned long long bad = 0;
        if (edge) bad = clean(tile, par);
        const u32x4* kp = &sh.k[par ^ 1][hi][ktok];   // piece 2 n of half kt: kp[2 * n * KU + kt * 32]
        const u32x4* vp = &sh.v[par][hi][col];        // step q, block n: vp[2 * q * D + n * 32]
        if (!before && sees(tile)) {
          find(0, tile + 2 * KU, kpg, kst);
          find(1, tile + KU, vpg, vst);
          if (edge) mask(s, tile, bad);
          const float mu = follow(edge ? top_of(s) : next_top);
          // ---- P of this tile, the next tile's S^T = K Q^T and O^T += V^T P^T, woven: a
          // product and an exponential (32 cycles and about 26) at a time, in this order
          using Order = Weave<NQ, ND>;
          constexpr int R = Order::ring;
          u32x4 fr[R];
          auto read = [&](int j) {   // operand of product j
            const int w = Order::op[j];
            if (w < 64) fr[j % R] = kp[2 * (w >> 1) * KU + (w & 1) * 32];
            else fr[j % R] = vp[2 * ((w - 64) / ND) * D + (w - 64) % ND * 32];
          };
          u32x4 pf[4];
          auto product = [&](int j) {
            const int w = Order::op[j];
            if (w < 64) sn[w & 1] = mfma32<A>(fr[j % R], qf[w >> 1], w < 2 ? f32x16{} : sn[w & 1]);
            else o[(w - 64) % ND] = mfma32<A>(fr[j % R], pf[(w - 64) / ND], o[(w - 64) % ND]);
            if (j + R < Order::n) read(j + R);
          };
#pragma unroll
          for (int j = 0; j < R; ++j) read(j);
          float y[2] = {0.f, 0.f};   // the pair before
          int j = 0;
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            __builtin_amdgcn_sched_barrier(0);
            const float x = __builtin_fmaf(s[e >> 4][e & 15], sl, -mu);
            if (e && !(e & 1)) pf[(e - 1) >> 3][((e - 1) >> 1) & 3] = pack2<A>(y[0], y[1]);
            if (j < Order::n && Order::at[j] == e) product(j++);
            if (e % (16 / LPW) == 0) {   // the loads, one at a time
              const int i = e / (16 / LPW);
              if (i < LPW) load_k(i, par);
              else load_v(i - LPW, par ^ 1);
            }
            if (e) l += y[(e - 1) & 1];
            asm volatile("" : "+v"(l));   // (else the sums gather after the last product)
            y[e & 1] = __builtin_amdgcn_exp2f(x);
          }
          __builtin_amdgcn_sched_barrier(0);
          pf[3][3] = pack2<A>(y[0], y[1]);
          l += y[1];
          float t0 = sn[0][0], t1 = sn[1][0];
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            if (j < Order::n && (r & 1) == 0) product(j++);
            t0 = max3(t0, sn[0][2 * r], sn[0][2 * r + 1]);
            t1 = max3(t1, sn[1][2 * r], sn[1][2 * r + 1]);
            asm volatile("" : "+v"(t0), "+v"(t1));
            __builtin_amdgcn_sched_barrier(0);
          }
#pragma unroll
          for (; j < Order::n; ++j) product(j);
          next_top = max3(t0, t1, t1);
        } else {
          if (kmore) issue_k(tile + 2 * KU, par);
          if (vmore) issue_v(tile + KU, par ^ 1);
          if (tile + KU < p.key1 && sees(tile + KU)) {
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int h = 0; h < 2; ++h)
                sn[h] = mfma32<A>(kp[2 * n * KU + h * 32], qf[n], n ? sn[h] : f32x16{});
            next_top = top_of(sn);
          }
        }
        if (kmore) commit_k(par);
        if (vmore) commit_v(par ^ 1);
      };
      f32x16 s0[2], s1[2];
      int tile = p.key0 - KU;
      step(std::integral_constant<int, 1>{}, s1, s0, tile, true);
      for (tile += KU;; tile += KU) {
        step(std::integral_constant<int, 0>{}, s0, s1, tile, false);
        if ((tile += KU) >= p.key1) break;
        step(std::integral_constant<int, 1>{}, s1, s0, tile, false);
        if (tile + KU >= p.key1) break;
      }
      // the loads past the last tile, ahead of the next piece's into the same slots
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    // ---- results: a lane has four consecutive elements of its query at a time
    l += __shfl_xor(l, 32);
    if (std::is_same<A, f16_t>::value) m -= 7.f;   // the exponents' origin
    if constexpr (!Q8) {
      const bool mine = residue(o) != 0.f && l < INFINITY;
      if (__builtin_expect(__ballot(mine) != 0, 0))
        settle<A, D>(kv, ktab, vtab, max(pos - win + 1, p.key0), min(pos, p.key1 - 1), max(posmax - win + 1, p.key0),
                     min(posmin, p.key1 - 1), mine, o,
                     [&](int bit) { return (bit >> 4) * 32 + (bit >> 2 & 3) * 8 + hi * 4 + (bit & 3); });
    }
    const bool whole = p.begins && p.ends;
    if (col < wrows) {
      if (whole) {
        const int head = p.head * a.group + row - tq * a.group;
        const float inv = l == 0.f ? 0.f : (DOWN ? 2.f : 1.f) / l;
        uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(p.q.q0 + tq) * a.out_ld + (int64_t)head * D;
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const f32x4 x = l == 0.f ? f32x4{0.f, 0.f, 0.f, 0.f}
                                     : f32x4{o[n][4 * b], o[n][4 * b + 1], o[n][4 * b + 2], o[n][4 * b + 3]};
            *reinterpret_cast<uint2*>(out + n * 32 + b * 8 + hi * 4) =
                uint2{pack2<A>(x[0] * inv, x[1] * inv), pack2<A>(x[2] * inv, x[3] * inv)};
          }
        if (a.lse && hi == 0)
          a.lse[(int64_t)(p.q.q0 + tq) * a.n_q_heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      } else {
        const int64_t at = ((int64_t)c.block * 2 + (n_piece == 0 ? 0 : 1)) * TR + wave * 32 + col;
        const float up = DOWN ? 2.f : 1.f;
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *reinterpret_cast<f32x4*>(parts.o + at * D + n * 32 + b * 8 + hi * 4) =
                f32x4{o[n][4 * b] * up, o[n][4 * b + 1] * up, o[n][4 * b + 2] * up, o[n][4 * b + 3] * up};
        if (hi == 0) parts.ml[at] = float2{m, l};
      }
    }
    if (p.first >= 0) {
      if (n_piece == 0 && tid == 0) tell(&p);
      ++n_piece;
    }
    __syncthreads();  // the slots of this piece have been read
  }
}

// Rows of a head of the longest sequence choose the kernel for all of a batch.
// One tile of 16 of them, or of FP8 caches two (the tiles of 128 rows convert every code
// for whatever rows there are).  Measured, us by k_attend_rows / k_attend_tiles, new
// tokens of 64 query heads on 8 unless said: 16 rows, bf16, 2 over 500 11.3 / 15.5, 2
// over 30000 32.2 / 40.1, 32 x 2 over 2000 52.4 / 52.8; 32 rows, bf16, 4 over 500 11.7 /
// 15.6, 4 over 30000 47.1 / 41.6, 32 x 4 over 2000 47.3 / 54.0, 64 x 32 over 500 of 32
// heads on 32 207 / 121; 32 rows, FP8, 12.7 / 15.6, 32.2 / 40.2, 94.8 / 115 (the last as of
// bf16); 40 and 48 rows, FP8, 5 over 30000 40.1 / 44.5, 32 x 5 over 2000 84.3 / 61.6, 32 x 6
// 85.1 / 62.4.
inline bool few_rows(bool fp8, int32_t group, int32_t max_q_len) {
  return (int64_t)max_q_len * group <= (fp8 ? 32 : 16);
}
inline int blocks_of(int n_cu) { return std::min(2 * n_cu / 8 * 8, 1024); }

// Every wave for itself once there are two (sequence, head) pairs a block.  Measured, us
// by blocks / by waves: 64 sequences of 16 tokens, 32 heads, 19 / 12, of 20 to 2048 233 /
// 214; with fewer pairs a wave's range ends inside its tiles and the parts cost more.
inline bool solo_waves(int32_t n_seqs, int32_t H, int n_cu) { return (int64_t)n_seqs * H >= 2 * blocks_of(n_cu); }

// Tiles of 256 rows in eight waves, one block a CU, where sequences have 512 rows on
// average and a block gets 24 units or more, as far as the host can tell: if the caches
// are as long as their tables (or the window).  Measured, us of a call with four / eight
// waves, 64 query heads on 8 unless said, bf16 (FP8), by new tokens over keys: 2048 over
// 16384 1490 / 958 (1485 / 984), the same in a window of 1000 142 / 100 (145 / 100), 2 x 256
// over 4096 126 / 99 (128 / 106), 512 over 4096 123 / 98, 4000 over 4000 of 32 heads on 32
// 255 / 198, 1000 over 30000 of 8 on 1 205 / 151; and below the line 4 x 128 over 2000 81 /
// 72, 512 over 512 50 / 57, 1000 over 1000 of 32 on 32 54 / 55, 4096 over 4096 of 8 on 1 119 /
// 131, 32 x 5 over 4096 115 / 117 (112 / 130), 16 x 300 over 300 of 32 on 32 69 / 80.
inline bool wide_tiles(const AttendArgs& a, int blocks) {
  const int64_t rows = (int64_t)a.kv.n_tokens * a.group;
  if (a.two_terms || rows < 512 * (int64_t)a.kv.n_seqs) return false;
  int64_t keys = (int64_t)a.kv.nb * a.kv.T - a.max_q_len / 2;
  if (a.window > 0) keys = std::min<int64_t>(keys, a.window);
  return rows / 256 * a.kv.H * (keys / 64) >= 24 * (int64_t)blocks;
}

template <typename A, typename KV, int D, int NW>
hipError_t launch_tiles(const AttendArgs& a, int G, hipStream_t s) {
  using TT = Tiles<A, KV, D, NW>;
  const size_t lds = sizeof(typename TT::Shared);
  static PerDevice limit;   // the kernel's LDS, more than a block gets unasked, is a setting of each device
  int device = -1;
  hipError_t e = hipGetDevice(&device);
  if (e == hipSuccess)
    e = limit.done(device, [&] {
      return hipFuncSetAttribute(reinterpret_cast<const void*>(&k_attend_tiles<A, KV, D, NW>),
                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    });
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_attend_tiles<A, KV, D, NW>), dim3(G), dim3(NW * 64), lds, s, a);
  // tiles of which none has many parts: four blocks each; else the list.  Measured
  // (us of a call, list / this): 32 sequences of 5 x 8 rows over 2500 tokens 78.4 / 76.1,
  // 2 of 256 x 8 rows over 4096 130 / 126, 64 x 4 rows of 8 heads over 2000 33.6 / 83.6,
  // 100 x 8 rows of one head over 30000 49.5 / 123
  const int64_t tiles = a.kv.H * std::max<int64_t>(a.kv.n_seqs, (int64_t)a.kv.n_tokens * a.group / TT::TR);
  if (2 * tiles >= G) {
    constexpr int RB = 256 / (D / 4);
    const int rows = (int)std::min<int64_t>((int64_t)a.max_q_len * a.group, TT::TR);
    hipLaunchKernelGGL((k_attend_join<A, D, TT::TR, RB>), dim3(G, (unsigned)std::min((rows + RB - 1) / RB, 4)),
                       dim3(256), 0, s, a, G);
  } else {
    hipLaunchKernelGGL((k_attend_join_list<A, D, TT::TR>), dim3(2 * G), dim3(256), 0, s, a, G);
  }
  return hipGetLastError();
}

template <typename A, typename KV, int D>
hipError_t launch(const AttendArgs& a, hipStream_t s) {
  const int64_t most = std::min<int64_t>((int64_t)a.max_q_len * a.group, 16);   // rows of a tile
  const bool few = few_rows(is_quant<KV>(), a.group, a.max_q_len);
  const int G = blocks_of(a.n_cu);
  if (few && solo_waves(a.kv.n_seqs, a.kv.H, a.n_cu)) {
    hipLaunchKernelGGL((k_attend_rows<A, KV, D, true>), dim3(G), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_attend_join<A, D, 16, 1>), dim3(4 * G, (unsigned)most), dim3(256), 0, s, a, 4 * G);
  } else if (few) {
    hipLaunchKernelGGL((k_attend_rows<A, KV, D, false>), dim3(G), dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_attend_join<A, D, 16, 1>), dim3(G, (unsigned)most), dim3(256), 0, s, a, G);
  } else {
    // FP8 of 64 elements has too few loads in a tile for eight waves
    constexpr bool wide = D / ET<KV>::E % 8 == 0;
    if (wide && wide_tiles(a, G / 16 * 8)) return launch_tiles<A, KV, D, wide ? 8 : 4>(a, G / 16 * 8, s);
    return launch_tiles<A, KV, D, 4>(a, G, s);
  }
  return hipGetLastError();
}

template <typename A, typename KV>
hipError_t launch_d(const KvTypes& ty, const AttendArgs& a, hipStream_t s) {
  return ty.D == 128 ? launch<A, KV, 128>(a, s) : launch<A, KV, 64>(a, s);
}

}  // namespace

size_t attend_workspace(const KvTypes& ty, int32_t n_cu, int32_t group, int32_t max_q_len, int32_t n_seqs,
                        int32_t H) {
  const bool few = few_rows(ty.kv == LORA_FP8_E4M3, group, max_q_len);
  const size_t G = (size_t)blocks_of(n_cu) * (few && solo_waves(n_seqs, H, n_cu) ? 4 : 1);
  const size_t TR = few ? 16 : 128, D = (size_t)ty.D;
  return G * (sizeof(PartDesc) + sizeof(int) + 2 * TR * 2 * sizeof(float) + 2 * TR * D * sizeof(float));
}

int64_t attend_units(const KvView& v, int32_t group, int32_t max_q_len) {
  const bool few = few_rows(v.scales != nullptr, group, max_q_len);
  const int TR = few ? 16 : 128, KU = few ? 32 : 64;
  const int64_t tiles = ((int64_t)v.n_tokens * group + TR - 1) / TR + v.n_seqs;
  return tiles * v.H * ((int64_t)v.nb * v.T / KU + 2);
}

hipError_t launch_attend(const KvTypes& ty, const AttendArgs& a, hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  if (ty.act == LORA_F16) return q ? launch_d<f16_t, fp8_t>(ty, a, s) : launch_d<f16_t, f16_t>(ty, a, s);
  return q ? launch_d<bf16_t, fp8_t>(ty, a, s) : launch_d<bf16_t, bf16_t>(ty, a, s);
}

}  // namespace lora
