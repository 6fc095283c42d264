// Attention of new tokens over the paged cache.
//
//   s_ij = scale q_i . k_j,  p_ij = exp(s_ij - m_i),  o_i = sum_j p_ij v_j / sum_j p_ij
//
// over the keys j that query i sees: pos_i - window < j <= pos_i whose pages are
// there.  One pass over the keys with a running maximum and sum.
//
// The rows of one kv head are its G query heads times the sequence's new tokens:
// row r is token r / G, head h G + r % G.  Two kernels share the sequences by
// their row count: up to 16 rows (single tokens and few drafted ones: bound by
// HBM) and more (chunks: bound by the matrix cores).  Both compute the transposed
// products
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
#include <type_traits>

#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr float kLn2 = 0.69314718055994530942f;

template <typename T>
__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, f32x4 c) {
  if constexpr (std::is_same<T, bf16_t>::value)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}
template <typename T>
__device__ __forceinline__ f32x16 mfma32(const uint4& a, const uint4& b, f32x16 c) {
  if constexpr (std::is_same<T, bf16_t>::value)
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a),
                                                  __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Eight FP8 codes (two words) -> eight 16-bit values, exact.
template <typename T>
__device__ __forceinline__ uint4 fp8_to16(uint32_t w0, uint32_t w1) {
  uint4 r;
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

// Element e of eight 16-bit values kept where bit e is set, else zero.
__device__ __forceinline__ uint4 keep8(uint4 u, uint32_t bits) {
  auto m = [](uint32_t b) { return ((b & 1) ? 0xffffu : 0u) | ((b & 2) ? 0xffff0000u : 0u); };
  u.x &= m(bits);
  u.y &= m(bits >> 2);
  u.z &= m(bits >> 4);
  u.w &= m(bits >> 6);
  return u;
}

// P in the 16 bits of the second product's operand: rounded, relative 2^-8 (bf16)
// or 2^-11 (f16) a term at most, and where SPLIT what the rounding left as a
// second operand (together 2^-16 of bf16, 2^-22 of f16).  The sums take P
// unrounded: lse is an fp32 result.
template <typename T, bool SPLIT>
__device__ __forceinline__ void p_operand(const float* p, uint4& hi, uint4& lo) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = pack2<T>(p[2 * i], p[2 * i + 1]);
    if (SPLIT)
      l[i] = pack2<T>(p[2 * i] - bits_to_f<T>(h[i] & 0xffffu), p[2 * i + 1] - bits_to_f<T>(h[i] >> 16));
  }
  hi = uint4{h[0], h[1], h[2], h[3]};
  if (SPLIT) lo = uint4{l[0], l[1], l[2], l[3]};
}

// Values without a finite number in V must reach the rows that see their token
// and no others (0 * inf is not 0 in a matrix product).  For tiles that some row
// does not see whole: v loses them, and for each class (+inf, -inf, NaN) an
// indicator takes their place in a product with the visibility of the tokens,
// whose result says which rows get that value.
template <typename T>
__device__ __forceinline__ uint32_t class_bits(const uint4& u, int cls) {
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
template <typename T>
__device__ __forceinline__ uint4 ones8(uint32_t bits) {
  constexpr uint32_t kOne = std::is_same<T, bf16_t>::value ? 0x3f803f80u : 0x3c003c00u;
  return keep8(uint4{kOne, kOne, kOne, kOne}, bits);
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
  int64_t start;         // the tile's first unit in the whole sequence of units
  int first;             // block that has it
  bool begins, ends;     // the piece has the tile's first / last unit
  KvSeq q;
};
struct PartDesc {        // a tile whose last of several parts a block has
  int32_t last;          // that block, -1: none
  int32_t first;         // block of its first part
  int32_t first_slot;
  int32_t head, row0, rows, q0, pad;
};

// Keys that the rows [row0, row0 + rows) of a sequence visit: from the first
// row's window, down to a multiple of KU, to the last row's own position.
template <int KU>
__device__ __forceinline__ void tile_keys(const AttendArgs& a, const KvSeq& q, int row0, int rows,
                                          int& lo, int& hi) {
  const int t0 = row0 / a.group, t1 = (row0 + rows - 1) / a.group;
  const int base = q.kv_len - q.q_len;
  hi = base + t1 + 1;
  lo = 0;
  if (a.window > 0 && base + t0 + 1 - a.window > 0) lo = (base + t0 + 1 - a.window) / KU * KU;
  if (hi <= lo) hi = lo + 1;  // nothing is seen: one unit, all of it masked
}

// Units of one head of a sequence whose rows are cut into tiles of TR.
template <int KU, int TR>
__device__ __forceinline__ int head_units(const AttendArgs& a, const KvSeq& q, int row_lo, int row_hi) {
  const int64_t rows64 = (int64_t)q.q_len * a.group;
  if (rows64 < row_lo || rows64 > row_hi || rows64 == 0) return 0;
  const int rows = (int)rows64;
  int u = 0;
  for (int r = 0; r < rows; r += TR) {
    int lo, hi;
    tile_keys<KU>(a, q, r, min(TR, rows - r), lo, hi);
    u += (hi - lo + KU - 1) / KU;
  }
  return u;
}

struct Cut {
  int64_t pos, end, total;   // this block's range of units
  int block, blocks;         // its number in the order of the ranges, and the blocks that have one
  int seq;
};

// Prefix sums of the sequences' units in LDS, and this block's range.  Every
// block computes them itself: the lengths are a few KB that stay in L2.
template <int KU, int TR, int THREADS>
__device__ __forceinline__ void cut_work(const AttendArgs& a, int row_lo, int row_hi, int64_t* pre,
                                         Cut& c) {
  const int n = a.kv.n_seqs;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  constexpr int W = THREADS / 64;
  int64_t* wsum = pre + kKvMaxSeqs + 1;
  int64_t run = 0;
  for (int s0 = 0; s0 < n; s0 += THREADS) {
    const int s = s0 + tid;
    int64_t x = 0;
    if (s < n) x = (int64_t)head_units<KU, TR>(a, kv_seq(a.kv, s), row_lo, row_hi) * a.kv.H;
    int64_t sum = x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up(sum, d);
      if (lane >= d) sum += y;
    }
    if (n > 64) {
      if (lane == 63) wsum[wave] = sum;
      __syncthreads();
      int64_t before = run, all = 0;
      for (int w = 0; w < W; ++w) {
        if (w < wave) before += wsum[w];
        all += wsum[w];
      }
      if (s < n) pre[s + 1] = before + sum;
      run += all;
      __syncthreads();
    } else if (s < n) {
      pre[s + 1] = sum;
    }
  }
  if (tid == 0) pre[0] = 0;
  __syncthreads();
  c.total = pre[n];
  // blocks b, b + 8, ... run on one XCD: give each XCD one contiguous eighth of
  // the ranges, so that the tiles that read the same keys share an L2
  const int G = (int)gridDim.x;
  const int b = (int)blockIdx.x;
  c.blocks = c.total < G ? (int)c.total : G;
  const int each = (c.blocks + 7) >> 3;
  const int L = (b & 7) * each + (b >> 3);
  c.block = L;
  if ((b >> 3) >= each || L >= c.blocks) {
    c.pos = c.end = 0;
    return;
  }
  c.pos = c.total * L / c.blocks;
  c.end = c.total * (L + 1) / c.blocks;
  // the sequence of the first unit
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= c.pos) lo = mid;
    else hi = mid;
  }
  c.seq = lo;
}

// The next piece of the range; advances c.  Sequences without units are passed.
template <int KU, int TR>
__device__ __forceinline__ bool next_piece(const AttendArgs& a, int row_lo, int row_hi,
                                           const int64_t* pre, Cut& c, Piece& p) {
  if (c.pos >= c.end) return false;
  while (pre[c.seq + 1] <= c.pos) ++c.seq;
  p.seq = c.seq;
  p.q = kv_seq(a.kv, c.seq);
  const int64_t seq_units = pre[c.seq + 1] - pre[c.seq];
  const int64_t off = c.pos - pre[c.seq];
  const int hu = (int)(seq_units / a.kv.H);
  p.head = (int)(off / hu);
  int rem = (int)(off - (int64_t)p.head * hu);
  const int rows = p.q.q_len * a.group;
  int lo = 0, hi = 0, units = 0;
  for (p.row0 = 0;; p.row0 += TR) {
    p.rows = min(TR, rows - p.row0);
    tile_keys<KU>(a, p.q, p.row0, p.rows, lo, hi);
    units = (hi - lo + KU - 1) / KU;
    if (rem < units) break;
    rem -= units;
  }
  const int64_t left = c.end - c.pos;
  const int take = left < units - rem ? (int)left : units - rem;
  p.begins = rem == 0;
  p.ends = rem + take == units;
  p.key0 = lo + rem * KU;
  p.key1 = p.ends ? hi : p.key0 + take * KU;
  // the block of the tile's first unit: L with L total / B <= first < (L + 1) total / B
  p.start = c.pos - rem;
  p.first = (int)(((p.start + 1) * c.blocks - 1) / c.total);
  c.pos += take;
  return true;
}

// Partial results of a block: slot 0 its first piece, slot 1 its last one if
// that is another.
template <int TR, int D>
struct Parts {
  static __host__ __device__ size_t desc_bytes(int G) { return (size_t)G * sizeof(PartDesc); }
  static __host__ __device__ size_t ml_bytes(int G) { return (size_t)G * 2 * TR * 2 * sizeof(float); }
  static __host__ __device__ size_t o_bytes(int G) { return (size_t)G * 2 * TR * D * sizeof(float); }
  PartDesc* desc;
  float2* ml;   // [slot][row]: maximum (log2 scale), sum
  float* o;     // [slot][row][D]
  __device__ Parts(char* ws, int G) {
    desc = reinterpret_cast<PartDesc*>(ws);
    ml = reinterpret_cast<float2*>(ws + desc_bytes(G));
    o = reinterpret_cast<float*>(ws + desc_bytes(G) + ml_bytes(G));
  }
};

// Tell the joining launch about this block's first piece: a tile's parts are
// joined by the block whose first piece is the last of several.
template <int TR, int D>
__device__ __forceinline__ void describe(const Parts<TR, D>& parts, const Cut& c, const Piece* p) {
  if (threadIdx.x != 0) return;
  PartDesc d{};
  d.last = -1;
  if (p && p->ends && !p->begins) {
    d.last = c.block;
    d.first = p->first;
    // the first part is its block's first piece iff that block's range begins with the tile
    d.first_slot = c.total * p->first / c.blocks == p->start ? 0 : 1;
    d.head = p->head;
    d.row0 = p->row0;
    d.rows = p->rows;
    d.q0 = p->q.q0;
  }
  parts.desc[blockIdx.x] = d;
}

__device__ __forceinline__ float safe_max(float m) { return m == -INFINITY ? 0.f : m; }

// ---- the joining launch ----------------------------------------------------------
// One wave a row: weights of the parts by their maxima, then a weighted sum.
// Bound by the reads of the parts; each is a contiguous D * 4 bytes.
template <typename A, int D, int TR>
__global__ __launch_bounds__(256) void k_attend_join(AttendArgs a, int G) {
  const Parts<TR, D> parts(a.ws, G);
  const PartDesc d = parts.desc[blockIdx.x];
  const int L = d.last;
  if (L < 0) return;
  const int lane = threadIdx.x & 63;
  constexpr int V = D / 64;
  for (int r = blockIdx.y * 4 + (threadIdx.x >> 6); r < d.rows; r += gridDim.y * 4) {
    float M = -INFINITY;
    auto slot = [&](int j) { return 2 * j + (j == d.first ? d.first_slot : 0); };
    for (int j = d.first + lane; j <= L; j += 64)
      M = fmaxf(M, parts.ml[(int64_t)slot(j) * TR + r].x);
#pragma unroll
    for (int x = 32; x; x >>= 1) M = fmaxf(M, __shfl_xor(M, x));
    const float Mu = safe_max(M);
    float acc[V], sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
#pragma unroll 8
    for (int j = d.first; j <= L; ++j) {
      const int64_t at = (int64_t)slot(j) * TR + r;
      const float2 ml = parts.ml[at];
      const float w = exp2f(ml.x - Mu);  // an empty part: exp2(-inf) = 0
      sum += w * ml.y;
      const float* o = parts.o + at * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += w * o[i];
    }
    const int row = d.row0 + r;
    const int t = row / a.group, head = d.head * a.group + row % a.group;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* out = reinterpret_cast<uint16_t*>(a.out) + (int64_t)(d.q0 + t) * a.out_ld + (int64_t)head * D + lane * V;
#pragma unroll
    for (int i = 0; i < V; ++i) out[i] = (uint16_t)f_to_bits<A>(sum == 0.f ? 0.f : acc[i] * inv);
    if (a.lse && lane == 0)
      a.lse[(int64_t)(d.q0 + t) * a.n_q_heads + head] = sum == 0.f ? -INFINITY : (Mu + log2f(sum)) * kLn2;
  }
}

// ---- up to 16 rows ---------------------------------------------------------------
// Four waves a block, each with its own keys, all with all of the tile's rows; K
// and V go from memory to registers (every byte is used once: LDS would only add
// a trip).  A wave's tile is 4 E keys: 16 KB at D = 128, its next pieces loaded
// as soon as the products have taken the last ones.
template <typename A, typename KV, int D>
struct Skinny {
  static constexpr bool Q8 = is_quant<KV>();
  static constexpr int E = ET<KV>::E;
  static constexpr int KT = 4 * E;       // keys of a wave's tile
  static constexpr int KU = 4 * KT;      // keys of a unit (all waves)
  static constexpr int TR = 16;
  static constexpr int NT = E / 4;       // K operands of 16 tokens
  static constexpr int NC = D / (4 * E); // 16-byte pieces of a K row a lane loads
  static constexpr int ND = D / 16;      // 16-element blocks of the head dimension
  static constexpr int NQ = D / 32;      // k steps of the first product
  using PT = typename std::conditional<Q8, bf16_t, A>::type;  // type of P and V in the second one
};

template <typename A, typename KV, int D>
__global__ __launch_bounds__(256, 2) void k_attend_rows(AttendArgs a, int row_lo, int row_hi) {
  using S = Skinny<A, KV, D>;
  using PT = typename S::PT;
  constexpr int E = S::E, KT = S::KT, KU = S::KU, TR = S::TR, NT = S::NT, NC = S::NC, ND = S::ND;
  constexpr bool Q8 = S::Q8;
  __shared__ int64_t pre[kKvMaxSeqs + 1 + 4];
  __shared__ float sh_ml[4][TR][2];
  __shared__ __align__(16) float sh_o[4][TR][D + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int col = lane & 15, g = lane >> 4;   // query column, lane group
  const KvView& kv = a.kv;
  Cut c;
  cut_work<KU, TR, 256>(a, row_lo, row_hi, pre, c);
  const Parts<TR, D> parts(a.ws, (int)gridDim.x);
  Piece p;
  int n_piece = 0;
  if (c.pos >= c.end) describe<TR, D>(parts, c, nullptr);
  while (next_piece<KU, TR>(a, row_lo, row_hi, pre, c, p)) {
    // ---- queries: operand B of the first product, column = row of the tile
    const int row = p.row0 + min(col, p.rows - 1);
    const int tq = row / a.group;
    const int pos = p.q.kv_len - p.q.q_len + tq;
    const int posmin = p.q.kv_len - p.q.q_len + p.row0 / a.group;
    const int posmax = p.q.kv_len - p.q.q_len + (p.row0 + p.rows - 1) / a.group;
    const int vislo = a.window > 0 ? pos - a.window + 1 : 0;
    uint4 qf[S::NQ];
    {
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(p.q.q0 + tq) * a.q_ld +
                           (int64_t)(p.head * a.group + row % a.group) * D;
#pragma unroll
      for (int i = 0; i < S::NQ; ++i) {
        // 16 bits: piece c = 4 i + g of 8 elements; FP8: half i & 1 of piece 4 (i / 2) + g of 16
        const int d = Q8 ? (4 * (i >> 1) + g) * 16 + (i & 1) * 8 : (4 * i + g) * 8;
        qf[i] = ld16(qp + d);
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
    uint4 kf[NT][NC], vf[ND];
    uint4 kscale, vscale;
    auto load_k = [&](const Ids& id) {
      const bool ok = (unsigned)id.kp < (unsigned)kv.n_pages;
      const char* base = kv.pages + (int64_t)(ok ? id.kp : 0) * kv.page_bytes + (g * kv.T + id.slot) * 16;
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int t = 0; t < NT; ++t) kf[t][n] = ld16(base + (n * 4 * kv.T + 4 * t) * 16);
    };
    auto load_v = [&](const Ids& id) {
      const bool ok = (unsigned)id.vp < (unsigned)kv.n_pages;
      const char* base = kv.pages + (int64_t)(ok ? id.vp : 0) * kv.page_bytes +
                         ((int64_t)(id.vslot / E) * D + col) * 16;
#pragma unroll
      for (int n = 0; n < ND; ++n) vf[n] = ld16(base + n * 256);
      if (Q8) vscale = ld16(kv.scales + (int64_t)(ok ? id.vp : 0) * kv.T + id.vslot);
    };
    // scale bytes of the lane's score tokens: group g, which is the V group's token range
    auto load_ks = [&](int tile) {
      if (!Q8) return;
      const int vt = tile + g * E;
      const int vb = (int)kv_div(kv, (uint32_t)vt);
      const int kp = vb < nblk ? ktab[vb] : -1;
      const bool ok = (unsigned)kp < (unsigned)kv.n_pages;
      kscale = ld16(kv.scales + (int64_t)(ok ? kp : 0) * kv.T + (vt - vb * kv.T));
    };

    int tile = p.key0 + wave * KT;
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
      // ---- S^T = K Q^T
      f32x4 s[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          if constexpr (Q8) {
            s[t] = mfma16<A>(fp8_to16<A>(kf[t][n].x, kf[t][n].y), qf[2 * n], s[t]);
            s[t] = mfma16<A>(fp8_to16<A>(kf[t][n].z, kf[t][n].w), qf[2 * n + 1], s[t]);
          } else {
            s[t] = mfma16<A>(kf[t][n], qf[n], s[t]);
          }
        }
      }
      const Ids idc = id;
      if constexpr (Q8) {
        const uint32_t w[4] = {kscale.x, kscale.y, kscale.z, kscale.w};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[t][i] *= __uint_as_float(((w[t] >> (8 * i)) & 0xffu) << 23);
      }
      if (more) {
        load_k(idn);
        load_ks(tile + KU);
      }
      // ---- mask
      const bool kbad = (unsigned)idc.kp >= (unsigned)kv.n_pages, vbad = (unsigned)idc.vp >= (unsigned)kv.n_pages;
      const bool edge = tile + KT - 1 > posmin || (a.window > 0 && tile <= posmax - a.window) ||
                        __ballot(kbad || vbad);
      uint32_t live = 0xffffu;   // of the lane's tokens g E + e: seen by some row
      uint32_t seen = 0xffffu;   // ... by the lane's row
      if (edge) {
        // group g's K page is known to the lanes with col / 4 == g
        const unsigned long long kb = __ballot(kbad);
        const bool gone = vbad || ((kb >> (g * 4)) & 1);
        live = seen = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int key = tile + g * E + e;
          const bool lv = !gone && key <= posmax && key < p.key1 &&
                          (a.window <= 0 || key > posmin - a.window);
          const bool sv = lv && key <= pos && key >= vislo;
          live |= (uint32_t)lv << e;
          seen |= (uint32_t)sv << e;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((seen >> (4 * t + i)) & 1)) s[t][i] = -INFINITY;
      }
      // ---- running maximum and sum
      float top = s[0][0];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, s[t][i]);
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      top *= a.scale_log2;
      // the maximum follows only when it would grow by more than 8 (a factor of
      // 256, which every type of P holds): else no rescaling
      if (__ballot(top > m + 8.f)) {
        const float mn = fmaxf(m, top);
        const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
        l *= f;
#pragma unroll
        for (int n = 0; n < ND; ++n) o[n] *= f;
        m = mn;
      }
      const float mu = safe_max(m);
      float pr[4 * NT];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          l += pr[4 * t + i] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[t][i], a.scale_log2, -mu));
      if constexpr (Q8) {
        const uint32_t w[4] = {vscale.x, vscale.y, vscale.z, vscale.w};
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          pr[e] *= __uint_as_float(((w[e / 4] >> (8 * (e & 3))) & 0xffu) << 23);
          if (edge && !((seen >> e) & 1)) pr[e] = 0.f;
        }
      }
      uint4 pf[E / 8], pl[E / 8];
#pragma unroll
      for (int q = 0; q < E / 8; ++q) p_operand<PT, true>(pr + 8 * q, pf[q], pl[q]);
      // ---- O^T += V^T P^T
      if (!edge) {
#pragma unroll
        for (int n = 0; n < ND; ++n) {
          if constexpr (Q8) {
            const uint4 v0 = fp8_to16<PT>(vf[n].x, vf[n].y), v1 = fp8_to16<PT>(vf[n].z, vf[n].w);
            o[n] = mfma16<PT>(v0, pf[0], o[n]);
            o[n] = mfma16<PT>(v1, pf[E / 8 - 1], o[n]);
            o[n] = mfma16<PT>(v0, pl[0], o[n]);
            o[n] = mfma16<PT>(v1, pl[E / 8 - 1], o[n]);
          } else {
            o[n] = mfma16<PT>(vf[n], pf[0], o[n]);
            o[n] = mfma16<PT>(vf[n], pl[0], o[n]);
          }
        }
      } else {
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
          for (int q = 0; q < E / 8; ++q) {
            uint4 v = vf[n];
            if constexpr (Q8) v = q ? fp8_to16<PT>(vf[n].z, vf[n].w) : fp8_to16<PT>(vf[n].x, vf[n].y);
            v = keep8(v, live >> (8 * q));
            const uint32_t odd = class_bits<PT>(v, 3);
            if (__ballot(odd != 0)) {
              const uint4 vis = ones8<PT>(seen >> (8 * q));
              for (int cls = 0; cls < 3; ++cls) {
                const f32x4 hit = mfma16<PT>(ones8<PT>(class_bits<PT>(v, cls)), vis, f32x4{0.f, 0.f, 0.f, 0.f});
#pragma unroll
                for (int i = 0; i < 4; ++i) o[n][i] += hit[i] > 0.f ? class_value(cls) : 0.f;
              }
              v = keep8(v, ~odd);
            }
            o[n] = mfma16<PT>(v, pf[q], o[n]);
            o[n] = mfma16<PT>(v, pl[q], o[n]);
          }
      }
      if (more) {
        load_v(idn);
        id = idn;
        idn = find(tile + 2 * KU);
      }
    }
    // ---- the waves' results
    l += __shfl_xor(l, 16);
    l += __shfl_xor(l, 32);
    if (lane < 16) {
      sh_ml[wave][col][0] = m;
      sh_ml[wave][col][1] = l;
    }
    if (col < p.rows)
#pragma unroll
      for (int n = 0; n < ND; ++n) *reinterpret_cast<f32x4*>(&sh_o[wave][col][16 * n + 4 * g]) = o[n];
    __syncthreads();
    const bool whole = p.begins && p.ends;
    const int slot = n_piece == 0 ? 0 : 1;
    for (int i = tid; i < p.rows * (D / 4); i += 256) {
      const int r = i / (D / 4), d = (i % (D / 4)) * 4;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, sh_ml[w][r][0]);
      const float Mu = safe_max(M);
      float sum = 0.f;
      f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float f = exp2f(sh_ml[w][r][0] - Mu);
        sum += f * sh_ml[w][r][1];
        acc += f * *reinterpret_cast<const f32x4*>(&sh_o[w][r][d]);
      }
      if (whole) {
        const int rr = p.row0 + r, t = rr / a.group, head = p.head * a.group + rr % a.group;
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
    if (n_piece == 0) describe<TR, D>(parts, c, &p);
    ++n_piece;
    __syncthreads();
  }
}

// ---- more rows -------------------------------------------------------------------
// Tiles of 128 rows: four waves of 32, which share every tile of 64 keys through
// LDS (loaded there directly, two buffers, one barrier a tile).  The LDS image is
// the pages' own order, [piece][token] and [token group][element] of 16 bytes, so
// that all reads of operands are contiguous over lanes and free of bank conflicts.
template <typename KV>
__device__ __forceinline__ int key_of(int r, int hi) {  // token of score register r in a tile of 32
  return is_quant<KV>() ? hi * 16 + r : (r >> 3) * 16 + hi * 8 + (r & 7);
}

__device__ __forceinline__ void load_lds16(const void* src, void* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}

template <typename A, typename KV, int D>
__global__ __launch_bounds__(256, 2) void k_attend_tiles(AttendArgs a, int row_lo, int row_hi) {
  constexpr bool Q8 = is_quant<KV>();
  using PT = typename std::conditional<Q8, bf16_t, A>::type;
  // f16 rows over an FP8 cache: bf16 holds the scaled P's range, two terms of it f16's precision
  constexpr bool SPLIT = !std::is_same<A, PT>::value;
  constexpr int E = ET<KV>::E, KU = 64, TR = 128;
  constexpr int NCK = D / E;          // 16-byte pieces of a K row
  constexpr int NGV = KU / E;         // token groups of a tile
  constexpr int ND = D / 32;
  constexpr int NQ = D / 16;
  constexpr int KLOADS = NCK / 4, VLOADS = NGV * D / 256;  // 1 KB loads of a wave
  __shared__ __align__(16) uint4 sk[2][NCK][KU];
  __shared__ __align__(16) uint4 sv[2][NGV][D];
  __shared__ float ss[2][2][KU];      // FP8: scales of K and V
  __shared__ int64_t pre[kKvMaxSeqs + 1 + 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, hi = lane >> 5;
  const KvView& kv = a.kv;
  Cut c;
  cut_work<KU, TR, 256>(a, row_lo, row_hi, pre, c);
  const Parts<TR, D> parts(a.ws, (int)gridDim.x);
  Piece p;
  int n_piece = 0;
  if (c.pos >= c.end) describe<TR, D>(parts, c, nullptr);
  // row col of the K operand is this token of a tile of 32, so that a lane's
  // scores are runs of E tokens
  const int ktok = Q8 ? ((col >> 2) & 1) * 16 + (col >> 3) * 4 + (col & 3)
                      : (col >> 4) * 16 + ((col >> 2) & 1) * 8 + ((col >> 3) & 1) * 4 + (col & 3);
  while (next_piece<KU, TR>(a, row_lo, row_hi, pre, c, p)) {
    const int wrow0 = p.row0 + wave * 32;
    const int wrows = min(32, p.rows - wave * 32);   // <= 0: no rows of its own
    const int base = p.q.kv_len - p.q.q_len;
    const int row = min(wrow0 + col, p.row0 + p.rows - 1);
    const int tq = row / a.group;
    const int pos = base + tq;
    const int posmin = base + wrow0 / a.group;
    const int posmax = base + (wrow0 + max(wrows, 1) - 1) / a.group;
    const int vislo = a.window > 0 ? pos - a.window + 1 : 0;
    uint4 qf[NQ];
    {
      const uint16_t* qp = reinterpret_cast<const uint16_t*>(a.q) + (int64_t)(p.q.q0 + tq) * a.q_ld +
                           (int64_t)(p.head * a.group + row % a.group) * D;
#pragma unroll
      for (int i = 0; i < NQ; ++i) {
        const int d = Q8 ? (2 * (i >> 1) + hi) * 16 + (i & 1) * 8 : (2 * i + hi) * 8;
        qf[i] = ld16(qp + d);
      }
    }
    const int32_t* ktab = kv.table + ((int64_t)p.seq * 2 * kv.H + p.head) * kv.nb;
    const int32_t* vtab = ktab + (int64_t)kv.H * kv.nb;
    // pages of the tile's tokens, lane = token; every wave looks up all of them
    struct Ids {
      int kp, vp, slot;
    };
    auto find = [&](int tile) {
      Ids r;
      const int t = tile + lane;
      const int b = (int)kv_div(kv, (uint32_t)t);
      r.slot = t - b * kv.T;
      r.kp = r.vp = -1;
      if (b < kv.nb) {
        r.kp = ktab[b];
        r.vp = vtab[b];
      }
      return r;
    };
    float sc_next = 0.f;
    auto stage = [&](const Ids& id, int buf) {
      const int kp = (unsigned)id.kp < (unsigned)kv.n_pages ? id.kp : 0;
      const int vp = (unsigned)id.vp < (unsigned)kv.n_pages ? id.vp : 0;
      const char* kb = kv.pages + (int64_t)kp * kv.page_bytes + (int64_t)id.slot * 16;
#pragma unroll
      for (int i = 0; i < KLOADS; ++i) {
        const int ch = wave + 4 * i;
        load_lds16(kb + (int64_t)ch * kv.T * 16, &sk[buf][ch][0]);
      }
#pragma unroll
      for (int i = 0; i < VLOADS; ++i) {
        const int j = wave * VLOADS + i;
        const int gr = j * 64 / D, d0 = j * 64 % D;
        const int pg = __builtin_amdgcn_readlane(vp, gr * E), sl = __builtin_amdgcn_readlane(id.slot, gr * E);
        const char* vb = kv.pages + (int64_t)pg * kv.page_bytes + ((int64_t)(sl / E) * D + d0) * 16;
        load_lds16(vb + lane * 16, &sv[buf][gr][d0]);
      }
      if (Q8 && wave < 2)
        sc_next = __uint_as_float((uint32_t)kv.scales[(int64_t)(wave ? vp : kp) * kv.T + id.slot] << 23);
    };
    f32x16 o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] = 0.f;
    float m = -INFINITY, l = 0.f;
    auto bad_of = [&](const Ids& id) {
      return (unsigned long long)__ballot((unsigned)id.kp >= (unsigned)kv.n_pages ||
                                          (unsigned)id.vp >= (unsigned)kv.n_pages);
    };
    Ids idn = find(p.key0);
    unsigned long long bad = bad_of(idn), badn = 0;
    stage(idn, 0);
    idn = find(p.key0 + KU);
    int buf = 0;
    for (int tile = p.key0; tile < p.key1; tile += KU, buf ^= 1) {
      const bool more = tile + KU < p.key1;
      if (Q8 && wave < 2) ss[buf][wave][lane] = sc_next;
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      if (more) {
        badn = bad_of(idn);
        stage(idn, buf ^ 1);
        idn = find(tile + 2 * KU);
      }
      const bool mine = wrows > 0 && tile <= posmax && (a.window <= 0 || tile + KU - 1 > posmin - a.window);
      if (mine) {
        // ---- S^T = K Q^T
        f32x16 s[2];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
          for (int r = 0; r < 16; ++r) s[kt][r] = 0.f;
#pragma unroll
          for (int n = 0; n < NCK / 2; ++n) {
            const uint4 kf = sk[buf][2 * n + hi][kt * 32 + ktok];
            if constexpr (Q8) {
              s[kt] = mfma32<A>(fp8_to16<A>(kf.x, kf.y), qf[2 * n], s[kt]);
              s[kt] = mfma32<A>(fp8_to16<A>(kf.z, kf.w), qf[2 * n + 1], s[kt]);
            } else {
              s[kt] = mfma32<A>(kf, qf[n], s[kt]);
            }
          }
        }
        if constexpr (Q8) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int r = 0; r < 16; ++r) s[kt][r] *= ss[buf][0][kt * 32 + key_of<KV>(r, hi)];
        }
        // ---- mask
        const bool edge = tile + KU - 1 > posmin || (a.window > 0 && tile <= posmax - a.window) || bad;
        uint32_t live[2], seen[2];
        if (edge) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt) {
            live[kt] = seen[kt] = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              const int k = kt * 32 + key_of<KV>(r, hi), key = tile + k;
              const bool lv = !((bad >> k) & 1) && key <= posmax && (a.window <= 0 || key > posmin - a.window);
              const bool sv = lv && key <= pos && key >= vislo;
              live[kt] |= (uint32_t)lv << r;
              seen[kt] |= (uint32_t)sv << r;
              s[kt][r] = sv ? s[kt][r] : -INFINITY;
            }
          }
        }
        // ---- running maximum and sum
        float top = s[0][0];
#pragma unroll
        for (int r = 0; r < 16; ++r) top = fmaxf(top, fmaxf(s[0][r], s[1][r]));
        top = fmaxf(top, __shfl_xor(top, 32)) * a.scale_log2;
        if (__ballot(top > m + 8.f)) {
          const float mn = fmaxf(m, top);
          const float f = m == -INFINITY ? 0.f : exp2f(m - mn);
          l *= f;
#pragma unroll
          for (int n = 0; n < ND; ++n) o[n] *= f;
          m = mn;
        }
        const float mu = safe_max(m);
        uint4 pf[4], pl[4];
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          float pr[16];
#pragma unroll
          for (int r = 0; r < 16; ++r)
            l += pr[r] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[kt][r], a.scale_log2, -mu));
          if constexpr (Q8) {
#pragma unroll
            for (int r = 0; r < 16; ++r) {
              pr[r] *= ss[buf][1][kt * 32 + key_of<KV>(r, hi)];
              if (edge && !((seen[kt] >> r) & 1)) pr[r] = 0.f;
            }
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) p_operand<PT, SPLIT>(pr + 8 * q, pf[2 * kt + q], pl[2 * kt + q]);
        }
        // ---- O^T += V^T P^T
        auto v_of = [&](int kt, int q, int n) -> uint4 {
          if constexpr (Q8) {
            const uint4 u = sv[buf][kt * 2 + hi][n * 32 + col];
            return q ? fp8_to16<PT>(u.z, u.w) : fp8_to16<PT>(u.x, u.y);
          } else {
            return sv[buf][kt * 4 + q * 2 + hi][n * 32 + col];
          }
        };
        if (!edge) {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int n = 0; n < ND; ++n) {
                const uint4 v = v_of(kt, q, n);
                o[n] = mfma32<PT>(v, pf[2 * kt + q], o[n]);
                if (SPLIT) o[n] = mfma32<PT>(v, pl[2 * kt + q], o[n]);
              }
        } else {
#pragma unroll
          for (int kt = 0; kt < 2; ++kt)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
              for (int n = 0; n < ND; ++n) {
                uint4 v = keep8(v_of(kt, q, n), live[kt] >> (8 * q));
                const uint32_t odd = class_bits<PT>(v, 3);
                if (__ballot(odd != 0)) {
                  const uint4 vis = ones8<PT>(seen[kt] >> (8 * q));
                  for (int cls = 0; cls < 3; ++cls) {
                    f32x16 hit;
#pragma unroll
                    for (int r = 0; r < 16; ++r) hit[r] = 0.f;
                    hit = mfma32<PT>(ones8<PT>(class_bits<PT>(v, cls)), vis, hit);
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[n][r] += hit[r] > 0.f ? class_value(cls) : 0.f;
                  }
                  v = keep8(v, ~odd);
                }
                o[n] = mfma32<PT>(v, pf[2 * kt + q], o[n]);
                if (SPLIT) o[n] = mfma32<PT>(v, pl[2 * kt + q], o[n]);
              }
        }
      }
      bad = badn;
    }
    // ---- results: a lane has four consecutive elements of its query at a time
    l += __shfl_xor(l, 32);
    const bool whole = p.begins && p.ends;
    if (col < wrows) {
      if (whole) {
        const int head = p.head * a.group + row % a.group;
        const float inv = l == 0.f ? 0.f : 1.f / l;
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
#pragma unroll
        for (int n = 0; n < ND; ++n)
#pragma unroll
          for (int b = 0; b < 4; ++b)
            *reinterpret_cast<f32x4*>(parts.o + at * D + n * 32 + b * 8 + hi * 4) =
                f32x4{o[n][4 * b], o[n][4 * b + 1], o[n][4 * b + 2], o[n][4 * b + 3]};
        if (hi == 0) parts.ml[at] = float2{m, l};
      }
    }
    if (n_piece == 0) describe<TR, D>(parts, c, &p);
    ++n_piece;
    __syncthreads();  // the buffers of this piece have been read
  }
}

template <typename A, typename KV, int D>
hipError_t launch(const AttendArgs& a, hipStream_t s) {
  const int G = a.n_cu * 2 / 8 * 8;
  const int64_t most = (int64_t)a.max_q_len * a.group;  // rows of a head of the longest sequence
  const int split = 16;
  // up to `split` rows; alone if no sequence has more
  const bool wide = most > split;
  const int small = (int)(most < 16 ? most : 16);
  hipLaunchKernelGGL((k_attend_rows<A, KV, D>), dim3(G), dim3(256), 0, s, a, 1, wide ? split : INT32_MAX);
  hipLaunchKernelGGL((k_attend_join<A, D, 16>), dim3(G, (small + 3) / 4), dim3(256), 0, s, a, G);
  if (wide) {
    const int rows = (int)(most < 128 ? most : 128);
    hipLaunchKernelGGL((k_attend_tiles<A, KV, D>), dim3(G), dim3(256), 0, s, a, split + 1, INT32_MAX);
    hipLaunchKernelGGL((k_attend_join<A, D, 128>), dim3(G, (rows + 3) / 4), dim3(256), 0, s, a, G);
  }
  return hipGetLastError();
}

template <typename A, typename KV>
hipError_t launch_d(const KvTypes& ty, const AttendArgs& a, hipStream_t s) {
  return ty.D == 128 ? launch<A, KV, 128>(a, s) : launch<A, KV, 64>(a, s);
}

}  // namespace

size_t attend_workspace(const KvTypes& ty, int32_t n_cu, int32_t group, int32_t max_q_len) {
  const int G = n_cu * 2 / 8 * 8;
  const int TR = (int64_t)max_q_len * group > 16 ? 128 : 16;
  const size_t D = (size_t)ty.D;
  return (size_t)G * (sizeof(PartDesc) + 2 * TR * 2 * sizeof(float) + 2 * TR * D * sizeof(float));
}

hipError_t launch_attend(const KvTypes& ty, const AttendArgs& a, hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  if (ty.act == LORA_F16) return q ? launch_d<f16_t, fp8_t>(ty, a, s) : launch_d<f16_t, f16_t>(ty, a, s);
  return q ? launch_d<bf16_t, fp8_t>(ty, a, s) : launch_d<bf16_t, bf16_t>(ty, a, s);
}

}  // namespace lora
