// KV cache write and read: new rows to their places in the pool's pages and
// cached rows back to dense ones.
//
// Both are copies bounded by HBM (FP8: 3 bytes an element moved, 4 in 16 bits).
// One wave owns one group of E consecutive positions (E elements in 16 bytes: 8
// of 16 bits, 16 of FP8) of one head, because that is the smallest piece of a V
// page whose bytes are contiguous: E tokens x D elements.  Its rows are read and
// its pieces written 16 bytes (FP8: 8) a lane, and a wave's lanes cover whole
// 128-byte lines on both sides, save the tokens at a sequence's ends.  Measured (a
// device copy of 1 GiB moves 4.8 TB/s): write of 32 requests of 32 to 600 tokens, 40
// heads of 128, bf16 into FP8, 313 MB, 79 us, 4.0 TB/s, the same into bf16, 416 MB,
// 97 us, 4.3 TB/s; read of 16 requests of 200 to 3000 tokens, 32 heads, FP8 to f16, 565
// MB, 123 us, 4.6 TB/s; one token each of 64 requests written, 5.5 us, and 4001 tokens of
// 8 heads read, 33 MB, 8.1 us, are mostly the launch.
#include "kcommon.h"
#include "kv.h"

namespace lora {

namespace {

constexpr int kWaves = 4;  // waves of a block

// The groups of sequence s take the numbers from q0 / E + 2 s on: E + (E - 1)
// positions may touch 2 groups, so q_len tokens touch at most
// (q_len + 2 E - 2) / E <= q_len / E + 2 of them, which is less than the
// distance to the next sequence's first number.  A number therefore names its
// sequence without any prefix sums, and a wave finds it with two probes of 64.
// The lengths of the sequences probed last come with the probe: they are a load
// less on the way to the rows.
template <int E>
__device__ __forceinline__ int kv_find_seq(const KvView& v, int w, int lane, KvSeq& q) {
  int base = 0;
  for (int stride = v.n_seqs > 64 ? 64 : 1;; stride = 1) {
    const int s = base + lane * stride;
    KvSeq mine{0, 0, 0, 0};
    bool le = false;
    if (s < v.n_seqs) {
      mine = kv_seq(v, s);
      le = mine.q0 / E + 2 * s <= w;
    }
    const unsigned long long m = __ballot(le);
    const int at = m ? 63 - __builtin_clzll(m) : 0;
    base += at * stride;
    if (stride == 1) {
      q.q0 = __builtin_amdgcn_readlane(mine.q0, at);
      q.q_len = __builtin_amdgcn_readlane(mine.q_len, at);
      q.base = __builtin_amdgcn_readlane(mine.base, at);
      q.end = __builtin_amdgcn_readlane(mine.end, at);
      return base;
    }
  }
}

struct Group {
  int row;       // row of the first covered position in the new tensors
  int lo, hi;    // covered positions of the group: [lo, hi) of 0 .. E
  int64_t k, v;  // byte offsets of the group's K slot 0 and V piece (-1: no page)
  int64_t ks, vs;// FP8: offsets of its scale bytes
};

template <int E, int D>
__device__ __forceinline__ bool kv_group(const KvView& v, int w, int h, int lane, Group& g) {
  KvSeq q;
  const int s = kv_find_seq<E>(v, w, lane, q);
  // rows before position 0 and past the table have no place
  const int p0 = q.base > 0 ? q.base : 0;
  const int p1 = q.base + q.q_len < q.end ? q.base + q.q_len : q.end;
  const int first = p0 / E;
  const int pos = (first + (w - (q.q0 / E + 2 * s))) * E;
  if (w < q.q0 / E + 2 * s || pos >= p1 || p0 >= p1) return false;
  g.lo = p0 > pos ? p0 - pos : 0;
  g.hi = p1 - pos < E ? p1 - pos : E;
  g.row = q.q0 + (pos + g.lo - q.base);
  const int b = (int)kv_div(v, (uint32_t)pos);
  const int slot = pos - b * v.T;
  const int32_t* t = v.table + ((int64_t)s * 2 * v.H + h) * v.nb + b;
  const int kp = t[0], vp = t[(int64_t)v.H * v.nb];
  const bool kok = (unsigned)kp < (unsigned)v.n_pages, vok = (unsigned)vp < (unsigned)v.n_pages;
  g.k = kok ? (int64_t)kp * v.page_bytes + (int64_t)slot * 16 : -1;
  g.v = vok ? (int64_t)vp * v.page_bytes + (int64_t)(slot / E) * D * 16 : -1;
  g.ks = kok ? (int64_t)kp * v.T + slot : -1;
  g.vs = vok ? (int64_t)vp * v.T + slot : -1;
  return true;
}

// ---- 16-bit caches: bits are moved as they are ------------------------------
template <int D>
__global__ __launch_bounds__(kWaves * 64) void k_kv_write16(KvView v, const uint16_t* __restrict__ k,
                                                             const uint16_t* __restrict__ vv, int64_t ld,
                                                             int items) {
  const int lane = threadIdx.x & 63;
  const int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (item >= items) return;
  const int w = item / v.H, h = item - w * v.H;
  Group g;
  if (!kv_group<8, D>(v, w, h, lane, g)) return;
  constexpr int C = D / 8;  // 16-byte pieces of a row
  // rows by token slot; slots outside [lo, hi) are not touched
  const uint16_t* kr = k + ((int64_t)g.row - g.lo) * ld + h * D;
  const uint16_t* vr = vv + ((int64_t)g.row - g.lo) * ld + h * D;
  uint4 kb[C / 8];
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    const int p = i * 64 + lane, t = p / C, c = p % C;
    kb[i] = uint4{0, 0, 0, 0};
    if (t >= g.lo && t < g.hi) kb[i] = ld16(kr + t * ld + c * 8);
  }
  const int d = lane * 2;
  uint32_t vb[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    vb[t] = 0;
    if (d < D && t >= g.lo && t < g.hi) vb[t] = *reinterpret_cast<const uint32_t*>(vr + t * ld + d);
  }
  if (g.k >= 0) {
#pragma unroll
    for (int i = 0; i < C / 8; ++i) {
      const int p = i * 64 + lane, t = p / C, c = p % C;
      if (t >= g.lo && t < g.hi)
        *reinterpret_cast<uint4*>(v.pages + g.k + ((int64_t)c * v.T + t) * 16) = kb[i];
    }
  }
  if (g.v >= 0 && d < D) {
    uint16_t* dst = reinterpret_cast<uint16_t*>(v.pages + g.v) + d * 8;
    if (g.lo == 0 && g.hi == 8) {
      uint4 a, b;  // eight tokens of element d, then of d + 1
      a.x = __builtin_amdgcn_perm(vb[1], vb[0], 0x05040100u);
      a.y = __builtin_amdgcn_perm(vb[3], vb[2], 0x05040100u);
      a.z = __builtin_amdgcn_perm(vb[5], vb[4], 0x05040100u);
      a.w = __builtin_amdgcn_perm(vb[7], vb[6], 0x05040100u);
      b.x = __builtin_amdgcn_perm(vb[1], vb[0], 0x07060302u);
      b.y = __builtin_amdgcn_perm(vb[3], vb[2], 0x07060302u);
      b.z = __builtin_amdgcn_perm(vb[5], vb[4], 0x07060302u);
      b.w = __builtin_amdgcn_perm(vb[7], vb[6], 0x07060302u);
      reinterpret_cast<uint4*>(dst)[0] = a;
      reinterpret_cast<uint4*>(dst)[1] = b;
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t >= g.lo && t < g.hi) {
          dst[t] = (uint16_t)vb[t];
          dst[8 + t] = (uint16_t)(vb[t] >> 16);
        }
    }
  }
}

template <int D>
__global__ __launch_bounds__(kWaves * 64) void k_kv_read16(KvView v, uint16_t* __restrict__ k,
                                                            uint16_t* __restrict__ vv, int64_t ld,
                                                            int items) {
  const int lane = threadIdx.x & 63;
  const int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (item >= items) return;
  const int w = item / v.H, h = item - w * v.H;
  Group g;
  if (!kv_group<8, D>(v, w, h, lane, g)) return;
  constexpr int C = D / 8;
  uint16_t* kr = k + ((int64_t)g.row - g.lo) * ld + h * D;
  uint16_t* vr = vv + ((int64_t)g.row - g.lo) * ld + h * D;
  uint4 kb[C / 8];
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    const int p = i * 64 + lane, t = p / C, c = p % C;
    kb[i] = uint4{0, 0, 0, 0};
    if (g.k >= 0 && t < g.hi) kb[i] = ld16(v.pages + g.k + ((int64_t)c * v.T + t) * 16);
  }
  const int d = lane * 2;
  uint4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
  if (g.v >= 0 && d < D) {
    a = ld16(v.pages + g.v + (int64_t)d * 16);
    b = ld16(v.pages + g.v + (int64_t)d * 16 + 16);
  }
#pragma unroll
  for (int i = 0; i < C / 8; ++i) {
    const int p = i * 64 + lane, t = p / C, c = p % C;
    if (t >= g.lo && t < g.hi) *reinterpret_cast<uint4*>(kr + t * ld + c * 8) = kb[i];
  }
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int t = 0; t < 8; ++t)
    if (d < D && t >= g.lo && t < g.hi)
      *reinterpret_cast<uint32_t*>(vr + t * ld + d) =
          __builtin_amdgcn_perm(bw[t / 2], aw[t / 2], (t & 1) ? 0x07060302u : 0x05040100u);
}

// ---- FP8 caches ----------------------------------------------------------------
// A row x of one token and head is stored as codes c_d = e4m3(x_d 2^-e), nearest
// even, with the smallest e in [-126, 127] for which 448 2^e is at least the
// largest finite |x_d|, and the byte e + 127.  A power of two costs no precision
// next to max / 448 (codes are floating, 3 bits of fraction either way), makes
// the product with 2^-e exact, so that a code depends on nothing but its row,
// and lets the scale be one byte.
__device__ __forceinline__ int fp8_exponent(uint32_t top_bits) {
  // top = 1.f * 2^x; 448 = 1.75 * 2^8
  const int x = (int)(top_bits >> 23) - 127;
  const int e = x - 8 + ((top_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;  // (e <= 120 for any finite top)
}

// Largest over the lanes of aligned groups of W = 8 or 16.
template <int W>
__device__ __forceinline__ uint32_t group_max(uint32_t x) {
  auto mx = [](uint32_t a, uint32_t b) { return a > b ? a : b; };
  auto mov = [](uint32_t a, auto ctrl) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, decltype(ctrl)::value, 0xF, 0xF, false);
  };
  x = mx(x, mov(x, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
  x = mx(x, mov(x, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
  x = mx(x, mov(x, std::integral_constant<int, 0x141>{}));  // row_half_mirror: 8 lanes
  if (W == 16) x = mx(x, mov(x, std::integral_constant<int, 0x140>{}));  // row_mirror
  return x;
}

template <typename A, int D>
__global__ __launch_bounds__(kWaves * 64) void k_kv_write8(KvView v, const uint16_t* __restrict__ k,
                                                            const uint16_t* __restrict__ vv, int64_t ld,
                                                            int items) {
  __shared__ __align__(16) uint32_t sh[kWaves][16][D / 4];  // V codes [token][element]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int item = blockIdx.x * kWaves + wave;
  if (item >= items) return;
  const int w = item / v.H, h = item - w * v.H;
  Group g;
  if (!kv_group<16, D>(v, w, h, lane, g)) return;
  constexpr int C = D / 8;        // lanes of a row (8 elements each)
  constexpr int R = 64 / C;       // rows of one pass over the wave
  const int c = lane % C;
  auto quant = [&](const uint4 u, int& e) {
    float f[8];
    unpack16<A>(u, f);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = __float_as_uint(f[i]) & 0x7fffffffu;
      if (b >= 0x7f800000u) f[i] = __uint_as_float(0x7fc00000u);  // no infinities: NaN codes
      else top = b > top ? b : top;
    }
    e = fp8_exponent(group_max<C>(top));
    const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
    uint2 r;
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0] * inv, f[1] * inv, lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2] * inv, f[3] * inv, lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4] * inv, f[5] * inv, hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6] * inv, f[7] * inv, hi, true);
    r.x = (uint32_t)lo;
    r.y = (uint32_t)hi;
    return r;
  };
  const uint16_t* kr = k + ((int64_t)g.row - g.lo) * ld + h * D + c * 8;
  const uint16_t* vr = vv + ((int64_t)g.row - g.lo) * ld + h * D + c * 8;
  uint4 kb[16 / R], vb[16 / R];
#pragma unroll
  for (int i = 0; i < 16 / R; ++i) {
    const int t = i * R + lane / C;
    kb[i] = vb[i] = uint4{0, 0, 0, 0};
    if (t >= g.lo && t < g.hi) {
      kb[i] = ld16(kr + t * ld);
      vb[i] = ld16(vr + t * ld);
    }
  }
#pragma unroll
  for (int i = 0; i < 16 / R; ++i) {
    const int t = i * R + lane / C;
    const bool in = t >= g.lo && t < g.hi;
    int e;
    const uint2 kc = quant(kb[i], e);
    if (in && g.k >= 0) {
      *reinterpret_cast<uint2*>(v.pages + g.k + ((int64_t)(c / 2) * v.T + t) * 16 + (c & 1) * 8) = kc;
      if (c == 0) v.scales[g.ks + t] = (uint8_t)(e + 127);
    }
    const uint2 vc = quant(vb[i], e);
    *reinterpret_cast<uint2*>(&sh[wave][t][c * 2]) = vc;
    if (in && g.v >= 0 && c == 0) v.scales[g.vs + t] = (uint8_t)(e + 127);
  }
  if (g.v < 0) return;
  __builtin_amdgcn_wave_barrier();
  // four elements d of eight tokens a lane: 4 x 4 bytes transposed twice, and
  // eight tokens of one element are 8 contiguous bytes of the page
  constexpr int Q = D / 4;
#pragma unroll
  for (int u = lane; u < 2 * Q; u += 64) {
    const int dq = u % Q, th = u / Q;
    uint32_t in[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) in[t] = sh[wave][th * 8 + t][dq];
    char* dst = v.pages + g.v + (int64_t)dq * 64 + th * 8;
    if (g.lo == 0 && g.hi == 16) {
      uint32_t o[2][4];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const uint32_t p01l = __builtin_amdgcn_perm(in[4 * q + 1], in[4 * q], 0x05010400u);
        const uint32_t p23l = __builtin_amdgcn_perm(in[4 * q + 3], in[4 * q + 2], 0x05010400u);
        const uint32_t p01h = __builtin_amdgcn_perm(in[4 * q + 1], in[4 * q], 0x07030602u);
        const uint32_t p23h = __builtin_amdgcn_perm(in[4 * q + 3], in[4 * q + 2], 0x07030602u);
        o[q][0] = __builtin_amdgcn_perm(p23l, p01l, 0x05040100u);
        o[q][1] = __builtin_amdgcn_perm(p23l, p01l, 0x07060302u);
        o[q][2] = __builtin_amdgcn_perm(p23h, p01h, 0x05040100u);
        o[q][3] = __builtin_amdgcn_perm(p23h, p01h, 0x07060302u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2*>(dst + i * 16) = uint2{o[0][i], o[1][i]};
    } else {
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (th * 8 + t >= g.lo && th * 8 + t < g.hi)
#pragma unroll
          for (int i = 0; i < 4; ++i) dst[i * 16 + t] = (char)(in[t] >> (8 * i));
    }
  }
}

template <typename A, int D>
__global__ __launch_bounds__(kWaves * 64) void k_kv_read8(KvView v, uint16_t* __restrict__ k,
                                                           uint16_t* __restrict__ vv, int64_t ld,
                                                           int items) {
  const int lane = threadIdx.x & 63;
  const int item = blockIdx.x * kWaves + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (item >= items) return;
  const int w = item / v.H, h = item - w * v.H;
  Group g;
  if (!kv_group<16, D>(v, w, h, lane, g)) return;
  constexpr int C = D / 16;
  uint16_t* kr = k + ((int64_t)g.row - g.lo) * ld + h * D;
  uint16_t* vr = vv + ((int64_t)g.row - g.lo) * ld + h * D;
  uint4 kb[C / 4];
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    const int p = i * 64 + lane, t = p / C, c = p % C;
    kb[i] = uint4{0, 0, 0, 0};
    if (g.k >= 0 && t < g.hi) kb[i] = ld16(v.pages + g.k + ((int64_t)c * v.T + t) * 16);
  }
  const int d = lane * 2;
  uint4 a{0, 0, 0, 0}, b{0, 0, 0, 0};
  if (g.v >= 0 && d < D) {
    a = ld16(v.pages + g.v + (int64_t)d * 16);
    b = ld16(v.pages + g.v + (int64_t)d * 16 + 16);
  }
#pragma unroll
  for (int i = 0; i < C / 4; ++i) {
    const int p = i * 64 + lane, t = p / C, c = p % C;
    if (t < g.lo || t >= g.hi) continue;
    float f[16];
    unpack16<fp8_t>(kb[i], f);
    const float sc = g.k >= 0 ? __uint_as_float((uint32_t)v.scales[g.ks + t] << 23) : 0.f;
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = pack2<A>(f[2 * j] * sc, f[2 * j + 1] * sc);
    uint4* dst = reinterpret_cast<uint4*>(kr + t * ld + c * 16);
    dst[0] = uint4{o[0], o[1], o[2], o[3]};
    dst[1] = uint4{o[4], o[5], o[6], o[7]};
  }
  if (d >= D) return;
  float fa[16], fb[16];
  unpack16<fp8_t>(a, fa);
  unpack16<fp8_t>(b, fb);
#pragma unroll
  for (int t = 0; t < 16; ++t) {
    if (t < g.lo || t >= g.hi) continue;
    const float sc = g.v >= 0 ? __uint_as_float((uint32_t)v.scales[g.vs + t] << 23) : 0.f;
    *reinterpret_cast<uint32_t*>(vr + t * ld + d) = pack2<A>(fa[t] * sc, fb[t] * sc);
  }
}

int64_t group_items(const KvView& v, int E) {
  return ((int64_t)v.n_tokens / E + 2 * (int64_t)v.n_seqs) * v.H;
}

}  // namespace

#define KV_LAUNCH(kern, ...)                                                                      \
  hipLaunchKernelGGL(kern, dim3((unsigned)((items + kWaves - 1) / kWaves)), dim3(kWaves * 64), 0, \
                     s, __VA_ARGS__)

hipError_t launch_kv_write(const KvTypes& ty, const KvView& v, const void* k, const void* vv,
                           int64_t ld, hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  const int items = (int)group_items(v, q ? 16 : 8);
  const uint16_t* kp = reinterpret_cast<const uint16_t*>(k);
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(vv);
  if (!q) {
    if (ty.D == 128) KV_LAUNCH(k_kv_write16<128>, v, kp, vp, ld, items);
    else KV_LAUNCH(k_kv_write16<64>, v, kp, vp, ld, items);
  } else if (ty.act == LORA_F16) {
    if (ty.D == 128) KV_LAUNCH((k_kv_write8<f16_t, 128>), v, kp, vp, ld, items);
    else KV_LAUNCH((k_kv_write8<f16_t, 64>), v, kp, vp, ld, items);
  } else {
    if (ty.D == 128) KV_LAUNCH((k_kv_write8<bf16_t, 128>), v, kp, vp, ld, items);
    else KV_LAUNCH((k_kv_write8<bf16_t, 64>), v, kp, vp, ld, items);
  }
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvTypes& ty, const KvView& v, void* k, void* vv, int64_t ld,
                          hipStream_t s) {
  const bool q = ty.kv == LORA_FP8_E4M3;
  const int items = (int)group_items(v, q ? 16 : 8);
  uint16_t* kp = reinterpret_cast<uint16_t*>(k);
  uint16_t* vp = reinterpret_cast<uint16_t*>(vv);
  if (!q) {
    if (ty.D == 128) KV_LAUNCH(k_kv_read16<128>, v, kp, vp, ld, items);
    else KV_LAUNCH(k_kv_read16<64>, v, kp, vp, ld, items);
  } else if (ty.act == LORA_F16) {
    if (ty.D == 128) KV_LAUNCH((k_kv_read8<f16_t, 128>), v, kp, vp, ld, items);
    else KV_LAUNCH((k_kv_read8<f16_t, 64>), v, kp, vp, ld, items);
  } else {
    if (ty.D == 128) KV_LAUNCH((k_kv_read8<bf16_t, 128>), v, kp, vp, ld, items);
    else KV_LAUNCH((k_kv_read8<bf16_t, 64>), v, kp, vp, ld, items);
  }
  return hipGetLastError();
}

}  // namespace lora
