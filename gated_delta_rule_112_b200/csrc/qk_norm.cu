// Per-head norm and position rotation of queries and keys, their gradients,
// and the 8-bit checkpoint that stands for the raw rows between the forward
// and the backward pass (gdn_qk_norm_rope_*).
//
// For a row x of d elements (one token, one head), with n = 1 (L2) or d (RMS):
//   r = (sum x^2 / n + eps)^-1/2 (1 without a norm),  h = x r,  z = (w + w0) h
//   y = scale [ m R(theta) z_rot , z_rest ]
// R turns the pairs of the first `rot` elements -- (2j, 2j + 1), or
// (j, j + rot / 2) -- by theta_j = position * inv_freq_j. Gradients for dy:
//   dz = scale [ m R(-theta) dy_rot , dy_rest ],  dw = sum over rows of dz h
//   dh = (w + w0) dz,   dx = r (dh - h (dh . h) / n)
// A row is read once and written once: the kernels are bound by HBM.
//
// A group of G lanes holds a row, two chunks of E elements a lane (E = 8 in the
// forward kernels, 4 in the backward ones, which hold more a row), so the sums
// are log2 G shuffles. For pairs of halves the chunks lie rot / 2 apart (rot a
// multiple of 2 E), otherwise side by side: a pair's two elements are in one
// lane either way and nothing is exchanged. Only halves that do not fall into
// chunks (odd rot, rows off their alignment) meet in the warp's own shared
// memory. With y = r (x C + x' S), x' the partner's element, C and S hold
// cosine, sine, weight and scale, formed once for all heads of q and of k of a
// token, and a row's arithmetic is two or three paired instructions an element
// pair and part of the sum.
//
// A warp takes an item: rows of one token, q's heads and then k's. It forms the
// item's cosines and sines once: the angle in turns is position * inv_freq /
// 2 pi as a sum of two fp64 numbers, less its whole turns, so far positions lose
// nothing; fp32 sine and cosine of the remainder follow.
//
// Measured (B200, 16384 tokens, 16 + 16 heads of d = 128, bf16): forward 46.6 us
// = 88 % of the copy rate, gradients from fp32 ones 92 us = 89 %, forward with the
// checkpoint 68 us = 76 %, gradients with weights from the checkpoint 103 us = 70
// %. fp32 rows: forward 97 us = 85 %, gradients 131 us = 94 %, but 171 us forward
// with halves through shared memory, where a step's raw rows, 64 registers a lane,
// spill. The first two wait for HBM; the 8-bit ones issue two to three instructions
// an element pair and are bound by both. What brought them there from 83, 128,
// 117 and 140 us: a pair's elements in one lane (no exchange), factors formed
// once a token, paired multiply-adds, sixteen elements a lane, reads without
// conditions. Two CTAs of 128 registers a thread an SM, with four rows a lane in
// flight: three CTAs of 80 with two were slower (89 us with the checkpoint).
//
// Checkpoint: 32 consecutive elements of a row share a power of two 2^e, the
// smallest (e >= -127) with max|x| <= 448 * 2^e over the block's finite
// elements, and are stored as e4m3 of x 2^-e (to nearest even); an element that
// is not finite becomes NaN. One byte e + 127 a block: no code is rounded twice
// and 2^e times a code is exact in bf16 (for e >= -124, or rows that were bf16).
#include <cuda_fp8.h>

#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

// What bounds checks need beside the kernels' own arguments (GDN_CHECKS builds).
#if GDN_CHECKS
#define QK_CHECKED(...) __VA_ARGS__
#else
#define QK_CHECKED(...)
#endif

constexpr int kQkThreads = 256;
constexpr int kMaxD = 256;
constexpr int kBlocksPerSm = 2;
// Gradients without weights hold fewer values a row: five CTAs of four warps an
// SM (102 registers a thread) instead of two of eight, 91 us against 95 us for
// 16384 x 32 rows. The other kernels lose by it (forward 46 -> 52 us).
constexpr int kPlainBwdThreads = 128, kPlainBwdBlocksPerSm = 5;

// How the pairs lie. Split: halves that fall into chunks; shared: any halves.
enum { kPairNone, kPairInterleaved, kPairSplit, kPairShared };

struct Part {                     // q or k
  const void *x;                  // rows (dtype), or e4m3 codes
  const uint8_t *x_scales;        // set when x holds codes
  const void *dy;
  void *out;                      // y or dx; may be null when only codes are wanted
  uint8_t *codes, *scales;        // checkpoint to write, or null
  const void *w;
  int64_t x_ts, dy_ts, out_ts;    // bytes between tokens
  int x_hs, dy_hs, out_hs;        // bytes between heads
  int H;                          // heads
  float scale;
};

struct QkArgs {
  Part p[2];
  const int32_t *pos;
  const double *inv_freq;
  float *dw_part;                 // [2][gridDim.x][d] partial weight gradients
  int T, d, rot, norm;
  int lg;                         // log2 of the lanes of a row
  int rpi, splits;                // rows an item, items a token
  float eps, w0, rope_scale, inv_n;
  QK_CHECKED(uint32_t *err; int64_t dw_extent;)
};

// A lane's place in a row: chunks of E elements at a and b, of which na and nb
// exist.
struct Lane { int a, b, na, nb; };
template <int E, int PAIR>
__device__ __forceinline__ Lane lane_place(const QkArgs &A, int l) {
  Lane L;
  const bool split = PAIR == kPairSplit && 2 * E * l < A.rot;
  L.a = split ? E * l : 2 * E * l;
  L.b = split ? A.rot / 2 + E * l : 2 * E * l + E;
  L.na = max(0, min(E, A.d - L.a));
  L.nb = max(0, min(E, A.d - L.b));
  return L;
}

// Two chunks as they lie in memory.
template <typename T, int E>
struct Raw;
template <int E>
struct Raw<__nv_bfloat16, E> { uint32_t w[E]; };
template <int E>
struct Raw<float, E> { float w[2 * E]; };
template <int E>
struct Codes { uint32_t w[E / 2]; uint32_t ea, eb; };

// ACC: elements an access may take; all pointers and strides are multiples of
// it. Where a chunk is one access or several whole ones (ACC >= E) it exists or
// not as a whole: it is then read without a condition, what does not exist from
// the row's beginning, and left out of the sums. Otherwise n elements are read
// and the rest is zero.
template <int E, int ACC>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, int n, uint32_t *w) {
  if (ACC >= E && E == 8) {
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if (ACC >= E) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) w[i] = 0;
    if (ACC == 4) {
#pragma unroll
      for (int i = 0; i < E; i += 4)
        if (i < n) {
          const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p + i));
          w[i / 2] = v.x; w[i / 2 + 1] = v.y;
        }
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < n) w[i / 2] |= uint32_t(*reinterpret_cast<const uint16_t *>(p + i)) << (16 * (i & 1));
    }
  }
}
template <int E, int ACC>
__device__ __forceinline__ void load_chunk(const float *p, int n, float *w) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ACC >= E) {
      v = __ldcs(reinterpret_cast<const float4 *>(p + i));
    } else if (ACC == 4) {
      if (i < n) v = __ldcs(reinterpret_cast<const float4 *>(p + i));
    } else {
      if (i + 0 < n) v.x = p[i];
      if (i + 1 < n) v.y = p[i + 1];
      if (i + 2 < n) v.z = p[i + 2];
      if (i + 3 < n) v.w = p[i + 3];
    }
    w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
  }
}
template <int E, int ACC>
__device__ __forceinline__ void load_chunk(const uint8_t *p, int n, uint32_t *w) {
  if (ACC >= E && E == 8) {
    const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
    w[0] = v.x; w[1] = v.y;
  } else if (ACC >= E) {
    w[0] = __ldcs(reinterpret_cast<const uint32_t *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < E; i += 4) {
      w[i / 4] = 0;
      if (ACC == 4) {
        if (i < n) w[i / 4] = __ldcs(reinterpret_cast<const uint32_t *>(p + i));
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i + k < n) w[i / 4] |= uint32_t(p[i + k]) << (8 * k);
      }
    }
  }
}

// The lane's elements as E pairs: chunk a, then chunk b.
template <int E>
struct Row { Pair v[E]; };

template <int E>
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16, E> &r, Row<E> &x) {
#pragma unroll
  for (int i = 0; i < E; ++i) x.v[i] = pair(bf_lo(r.w[i]), bf_hi(r.w[i]));
}
template <int E>
__device__ __forceinline__ void unpack(const Raw<float, E> &r, Row<E> &x) {
#pragma unroll
  for (int i = 0; i < E; ++i) x.v[i] = pair(r.w[2 * i], r.w[2 * i + 1]);
}
// 2^(b - 127), b in [0, 254]: 2^-127 lies below the normal range.
__device__ __forceinline__ float pow2_biased(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}
// Codes without their scales, which go into the row's sums and factor.
template <int E>
__device__ __forceinline__ void unpack(const Codes<E> &r, Row<E> &x) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((r.w[i / 2] >> (16 * (i & 1))) & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x.v[i] = pair(f.x, f.y);
  }
}
// What the unpacked chunks are to be multiplied by.
struct Scales { float a, b; };
template <typename D>
__device__ __forceinline__ Scales scales_of(const D &) { return {1.f, 1.f}; }
template <int E>
__device__ __forceinline__ Scales scales_of(const Codes<E> &r) {
  return {pow2_biased(r.ea), pow2_biased(r.eb)};
}

template <int E, int ACC>
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, int n, const Pair *v) {
  uint32_t w[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const float2 f = unpair(v[i]);
    w[i] = bf_pack(f.x, f.y);
  }
  if (ACC >= E && E == 8) {
    if (n > 0) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (ACC >= 4) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      if (i < n) *reinterpret_cast<uint2 *>(p + i) = make_uint2(w[i / 2], w[i / 2 + 1]);
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) *reinterpret_cast<uint16_t *>(p + i) = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
}
template <int E, int ACC>
__device__ __forceinline__ void store_chunk(float *p, int n, const Pair *v) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float2 f = unpair(v[i / 2]), g = unpair(v[i / 2 + 1]);
    if (ACC >= 4) {
      if (i < n) *reinterpret_cast<float4 *>(p + i) = make_float4(f.x, f.y, g.x, g.y);
    } else {
      if (i + 0 < n) p[i] = f.x;
      if (i + 1 < n) p[i + 1] = f.y;
      if (i + 2 < n) p[i + 2] = g.x;
      if (i + 3 < n) p[i + 3] = g.y;
    }
  }
}
template <int E, int ACC>
__device__ __forceinline__ void store_codes(uint8_t *p, int n, const uint32_t *w) {
  if (ACC >= E && E == 8) {
    if (n > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else if (ACC >= 4) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      if (i < n) *reinterpret_cast<uint32_t *>(p + i) = w[i / 4];
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < n) p[i] = uint8_t(w[i / 4] >> (8 * (i & 3)));
  }
}

// Heads' rows of one token, at the lane's chunks: one multiply-add an address.
template <typename P>
struct Rows {
  P *a, *b;
  int hs;
  __device__ __forceinline__ Rows(P *p, int64_t offset, int head_stride, const Lane &L, bool reads) {
    char *q = const_cast<char *>(reinterpret_cast<const char *>(p)) + offset;
    // chunks that do not exist are read at the row's beginning
    a = reinterpret_cast<P *>(q) + (reads && L.na == 0 ? 0 : L.a);
    b = reinterpret_cast<P *>(q) + (reads && L.nb == 0 ? 0 : L.b);
    hs = head_stride;
  }
  static __device__ __forceinline__ P *at(P *p, int h, int hs) {
    return reinterpret_cast<P *>(const_cast<char *>(reinterpret_cast<const char *>(p)) + int64_t(h) * hs);
  }
  __device__ __forceinline__ P *first(int h) const { return at(a, h, hs); }
  __device__ __forceinline__ P *second(int h) const { return at(b, h, hs); }
  // Whether what a lane's access to row h touches lies in the buffer.
  QK_CHECKED(const P *base; int64_t extent; uint32_t *err;)
  template <int E, int ACC>
  __device__ __forceinline__ bool in_bounds(int h, const Lane &L, bool reads) const {
#if GDN_CHECKS
    const int na = reads && ACC >= E ? E : L.na, nb = reads && ACC >= E ? E : L.nb;
    return (na == 0 || GDN_IN_BOUNDS(err, first(h) - base, extent - na + 1)) &&
           (nb == 0 || GDN_IN_BOUNDS(err, second(h) - base, extent - nb + 1));
#else
    return true;
#endif
  }
};
#if GDN_CHECKS
template <typename P>
__device__ __forceinline__ void bound(Rows<P> &r, const QkArgs &A, const void *base, int64_t extent) {
  r.base = static_cast<const P *>(base);
  r.extent = extent;
  r.err = A.err;
}
// Elements from the first of a part's rows to the last; strides in bytes.
template <typename P>
__device__ __forceinline__ void bound(Rows<P> &r, const QkArgs &A, const void *base, int64_t ts, int64_t hs,
                                      int H) {
  bound(r, A, base, (int64_t(A.T - 1) * ts + int64_t(H - 1) * hs) / int64_t(sizeof(P)) + A.d);
}
#endif
template <int E, int ACC, typename T>
__device__ __forceinline__ void load_row(const Rows<const T> &P, int h, const Lane &L, Raw<T, E> &r) {
  constexpr int half = sizeof(r.w) / sizeof(r.w[0]) / 2;
  if (!P.template in_bounds<E, ACC>(h, L, true)) {
    r = Raw<T, E>{};
    return;
  }
  if (ACC == 8 && E == 4 && sizeof(T) == 2) {        // side by side (see with_variant)
    const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(P.first(h)));
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 2 * half; ++i) reinterpret_cast<uint32_t &>(r.w[i]) = w[i & 3];
  } else {
    load_chunk<E, ACC>(P.first(h), L.na, r.w);
    load_chunk<E, ACC>(P.second(h), L.nb, r.w + half);
  }
}

// Sum over the 2^lg lanes of a row; LG: lg where the compiler knows it, else 0.
template <int LG>
__device__ __forceinline__ float group_sum(float x, int lg) {
  if (LG) lg = LG;
  if (lg > 4) x += __shfl_xor_sync(0xffffffffu, x, 16);
  if (lg > 3) x += __shfl_xor_sync(0xffffffffu, x, 8);
  if (lg > 2) x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 2);
  x += __shfl_xor_sync(0xffffffffu, x, 1);
  return x;
}
// x . y over each of the lane's chunks; chunks that do not exist count for nothing.
template <int E, bool WHOLE>
__device__ __forceinline__ float2 dots(const Lane &L, const Row<E> &x, const Row<E> &y) {
  Pair s = mul2(x.v[0], y.v[0]), t = mul2(x.v[E / 2], y.v[E / 2]);
#pragma unroll
  for (int i = 1; i < E / 2; ++i) {
    s = fma2(x.v[i], y.v[i], s);
    t = fma2(x.v[E / 2 + i], y.v[E / 2 + i], t);
  }
  const float2 f = unpair(s), g = unpair(t);
  float2 d = make_float2(f.x + f.y, g.x + g.y);
  if (WHOLE) {
    if (L.na == 0) d.x = 0.f;
    if (L.nb == 0) d.y = 0.f;
  }
  return d;
}

// The lane's part of x C + x' S, x' the partner of every element. What does
// not turn takes no partner: it must not meet another element's infinity.
// row: this group's part of the warp's buffer.
template <int E, int PAIR>
__device__ __forceinline__ void turn(const QkArgs &A, const Lane &L, float *row, const Row<E> &C,
                                     const Row<E> &S, Row<E> &x) {
  Row<E> y;
#pragma unroll
  for (int i = 0; i < E; ++i) y.v[i] = mul2(x.v[i], C.v[i]);
  if (PAIR == kPairInterleaved) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float2 f = unpair(x.v[i]);
      if (L.a + 2 * i < A.rot) y.v[i] = fma2(pair(f.y, f.x), S.v[i], y.v[i]);
    }
  } else if (PAIR == kPairSplit) {
    if (L.a < A.rot) {
#pragma unroll
      for (int i = 0; i < E; ++i) y.v[i] = fma2(x.v[i ^ (E / 2)], S.v[i], y.v[i]);
    }
  } else if (PAIR == kPairShared) {
    const int half = A.rot / 2;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < E; ++i)
      *reinterpret_cast<float2 *>(row + L.a + 2 * i) = unpair(x.v[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < E; ++i) {
      float2 f;
      const int e = L.a + 2 * i, g = e + 1;
      f.x = e < A.rot ? row[e < half ? e + half : e - half] : 0.f;
      f.y = g < A.rot ? row[g < half ? g + half : g - half] : 0.f;
      y.v[i] = fma2(pair(f.x, f.y), S.v[i], y.v[i]);
    }
  }
  x = y;
}

// The item's cosines and sines, in the warp's buffer: cs[j], cs[kMaxD / 2 + j];
// 1 and 0 for the pairs that do not turn. inv_freq / 2 pi and its product with
// the position are each a rounded fp64 number and the remainder that a fused
// multiply-add gives exactly: rounded alone they are off by 4e-7 of a radian at
// 3e8 turns, seven times fp32's own rounding.
__device__ __forceinline__ void make_angles(const QkArgs &A, int t, int lane, int pairs, float *cs) {
  constexpr double kInv2Pi = 0.15915494309189535, kInv2PiRest = -9.839338337591243e-18;   // 1 / (2 pi)
  const double p = GDN_IN_BOUNDS(A.err, t, A.T) ? double(A.pos[t]) : 0.0;
  __syncwarp();
  for (int j = lane; j < pairs; j += 32) {
    float s = 0.f, c = 1.f;
    if (j < A.rot / 2) {
      const double f = A.inv_freq[j], h = __dmul_rn(f, kInv2Pi), n = __dmul_rn(p, h);
      const double h_rest = fma(f, kInv2PiRest, fma(f, kInv2Pi, -h));
      const double turns = __dadd_rn(n, -rint(n)) + fma(p, h_rest, fma(p, h, -n));
      sincospif(float(2.0 * turns), &s, &c);
      c *= A.rope_scale;
      s *= A.rope_scale;
    }
    cs[j] = c;
    cs[kMaxD / 2 + j] = s;
  }
  __syncwarp();
}

__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <int E>
__device__ __forceinline__ void lds(const float *p, float *x) {
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    const float4 v = lds4(p + i);
    x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
  }
}

// C and S for a turn by +angle (sign 1) or -angle, with the element's weight in
// C and its partner's in S. w: a weight for each element.
template <int E, int PAIR>
__device__ __forceinline__ void factors(const QkArgs &A, const Lane &L, int l, const float *cs, const float *w,
                                        float sign, Row<E> &C, Row<E> &S) {
  float wa[2 * E];
  lds<E>(w + L.a, wa);
  lds<E>(w + L.b, wa + E);
  float c[2 * E], s[2 * E];
  if (PAIR == kPairNone) {
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) c[i] = wa[i], s[i] = 0.f;
  } else if (PAIR == kPairShared) {
    const int half = A.rot / 2;
#pragma unroll
    for (int i = 0; i < 2 * E; ++i) {
      const int e = L.a + i, j = e < half ? e : e - half;
      const bool on = e < A.rot;
      c[i] = (on ? cs[j] : 1.f) * wa[i];
      s[i] = on ? sign * cs[kMaxD / 2 + j] * (e < half ? -w[e + half] : w[e - half]) : 0.f;
    }
  } else {
    float cj[E], sj[E];
    lds<E>(cs + E * l, cj);
    lds<E>(cs + kMaxD / 2 + E * l, sj);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      // the pair's elements: neighbours, or one of each chunk
      const int i = PAIR == kPairInterleaved ? 2 * j : j, k = PAIR == kPairInterleaved ? 2 * j + 1 : j + E;
      c[i] = cj[j] * wa[i];
      c[k] = cj[j] * wa[k];
      s[i] = -sign * sj[j] * wa[k];
      s[k] = sign * sj[j] * wa[i];
    }
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    C.v[i] = pair(c[2 * i], c[2 * i + 1]);
    S.v[i] = pair(s[2 * i], s[2 * i + 1]);
  }
}

__device__ __forceinline__ float rnorm(const QkArgs &A, float ss) {
  return A.norm == GDN_NORM_NONE ? 1.f : rsqrtf(ss * A.inv_n + A.eps);
}

// (w + w0) * scale of q's and of k's elements, 1 * scale without weights.
template <typename T, int THREADS>
__device__ __forceinline__ void stage_weights(const QkArgs &A, bool scaled, bool weighted, float (*w)[kMaxD]) {
  for (int i = threadIdx.x; i < 2 * kMaxD; i += THREADS) {
    const Part &P = A.p[i / kMaxD];
    const int e = i % kMaxD;
    float x = 1.f;
    if (weighted && P.w && e < A.d) x = to_f32(static_cast<const T *>(P.w)[e]) + A.w0;
    w[i / kMaxD][e] = scaled ? x * P.scale : x;
  }
  __syncthreads();
}

// Source of the rows: T in memory, or codes.
template <typename T, bool PACKED, int E, int PAIR, int ACC>
struct Source {
  using Data = Raw<T, E>;
  Rows<const T> rows;
  __device__ __forceinline__ Source(const QkArgs &A, const Part &P, int64_t t, const Lane &L)
      : rows(static_cast<const T *>(P.x), t * P.x_ts, P.x_hs, L, true) {
    QK_CHECKED(bound(rows, A, P.x, P.x_ts, P.x_hs, P.H);)
  }
  __device__ __forceinline__ void load(int h, const Lane &L, Data &r) const {
    load_row<E, ACC>(rows, h, L, r);
  }
};
template <typename T, int E, int PAIR, int ACC>
struct Source<T, true, E, PAIR, ACC> {
  using Data = Codes<E>;
  Rows<const uint8_t> rows;
  const uint8_t *e;
  int blocks, ea, eb;
  __device__ __forceinline__ Source(const QkArgs &A, const Part &P, int64_t t, const Lane &L)
      : rows(static_cast<const uint8_t *>(P.x), t * P.H * A.d, A.d, L, true) {
    blocks = (A.d + 31) / 32;
    e = P.x_scales + t * P.H * blocks;
    ea = L.na > 0 ? L.a / 32 : 0;
    eb = L.nb > 0 ? L.b / 32 : 0;
    QK_CHECKED(bound(rows, A, P.x, int64_t(A.T) * P.H * A.d); scales = P.x_scales;
               scales_extent = int64_t(A.T) * P.H * blocks;)
  }
  QK_CHECKED(const uint8_t *scales; int64_t scales_extent;)
  __device__ __forceinline__ void load(int h, const Lane &L, Data &r) const {
    const uint8_t *s = e + int64_t(h) * blocks;
    if (!rows.template in_bounds<E, ACC>(h, L, true) ||
        !GDN_IN_BOUNDS(rows.err, s + ea - scales, scales_extent) ||
        !GDN_IN_BOUNDS(rows.err, s + eb - scales, scales_extent)) {
      r = Codes<E>{};
      return;
    }
    load_chunk<E, ACC>(rows.first(h), L.na, r.w);
    load_chunk<E, ACC>(rows.second(h), L.nb, r.w + E / 4);
    r.ea = s[ea];
    r.eb = PAIR == kPairSplit ? s[eb] : r.ea;        // side by side, both are of one block
  }
};

// The biased exponent that a block's largest finite magnitude (its bits) asks
// for. 448 = 1.75 * 2^8: its exponent - 8, one more where the significand is
// above 1.75, and not below 2^-127.
__device__ __forceinline__ int block_exponent(uint32_t bits) {
  return max(int((bits + 0x1fffffu) >> 23) - 8, 0);
}
// Largest magnitude of each chunk, as bits of an fp32: of non-negative floats
// the bits compare alike, with infinities and NaN above the rest. bf16 is
// compared two at a time (a NaN wins).
struct Top { uint32_t a, b; };
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int E>
__device__ __forceinline__ Top chunk_tops(const Raw<__nv_bfloat16, E> &r) {
  const uint32_t m = 0x7fff7fffu;
  uint32_t a = r.w[0] & m, b = r.w[E / 2] & m;
#pragma unroll
  for (int i = 1; i < E / 2; ++i) {
    a = max2(a, r.w[i] & m);
    b = max2(b, r.w[E / 2 + i] & m);
  }
  const uint32_t t = max2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  return {t << 16, t & 0xffff0000u};
}
template <int E>
__device__ __forceinline__ Top chunk_tops(const Raw<float, E> &r) {
  Top t = {0, 0};
#pragma unroll
  for (int i = 0; i < E; ++i) {
    t.a = max(t.a, __float_as_uint(r.w[i]) & 0x7fffffffu);
    t.b = max(t.b, __float_as_uint(r.w[E + i]) & 0x7fffffffu);
  }
  return t;
}

// Writes the lane's elements in 8 bits. Side by side, 32 / 2E lanes hold a
// block; with halves in chunks 32 / E lanes' first chunks do, and their second
// chunks, where rot / 2 is a multiple of 32; for other rot the blocks' maxima
// meet in shared memory. The exponents go to scales, in shared memory too.
template <typename T, int E, int PAIR, int ACC>
__device__ __forceinline__ void write_codes(const QkArgs &A, const Rows<uint8_t> &codes, uint8_t *scales,
                                            int h, const Lane &L, bool on, uint32_t *tops,
                                            const Raw<T, E> &raw, const Row<E> &x) {
  constexpr uint32_t kInf = 0x7f800000u;
  Top t = chunk_tops<E>(raw);
  if (ACC >= E) {
    t.a = L.na > 0 ? t.a : 0;
    t.b = L.nb > 0 ? t.b : 0;
  }
  const bool odd = __any_sync(0xffffffffu, max(t.a, t.b) >= kInf);
  if (odd) {                           // what is not finite counts for nothing
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float2 f = unpair(x.v[i]);
      uint32_t &top = u[i / (E / 2)];
      const uint32_t fx = __float_as_uint(f.x) & 0x7fffffffu, fy = __float_as_uint(f.y) & 0x7fffffffu;
      if (fx < kInf) top = max(top, fx);
      if (fy < kInf) top = max(top, fy);
    }
    t.a = ACC < E || L.na > 0 ? u[0] : 0;
    t.b = ACC < E || L.nb > 0 ? u[1] : 0;
  }
  const bool split = PAIR == kPairSplit && L.a < A.rot;
  if (PAIR == kPairSplit && A.rot % 64) {
    __syncwarp();
    if ((L.a & 31) == 0) tops[L.a / 32] = 0;
    if ((L.b & 31) == 0) tops[L.b / 32] = 0;
    __syncwarp();
    atomicMax(&tops[L.a / 32], t.a);
    atomicMax(&tops[L.b / 32], t.b);
    __syncwarp();
    t = {tops[L.a / 32], tops[L.b / 32]};
  } else {
    if (!split) t.a = t.b = max(t.a, t.b);
    if (PAIR == kPairSplit && sizeof(T) == 2) {          // both chunks' 16 bits in one word
      uint32_t w = __byte_perm(t.a, t.b, 0x7632);
#pragma unroll
      for (int off = 1; off < 32 / E; off <<= 1) {
        const uint32_t o = __shfl_xor_sync(0xffffffffu, w, off);
        if (2 * off < 32 / E || split) w = max2(w, o);
      }
      t = {w << 16, w & 0xffff0000u};
    } else {
#pragma unroll
      for (int off = 1; off < 32 / E; off <<= 1) {
        const bool takes = 2 * off < 32 / E || split;
        if (PAIR != kPairSplit && 2 * off >= 32 / E) break;
        const uint32_t oa = __shfl_xor_sync(0xffffffffu, t.a, off);
        if (takes) t.a = max(t.a, oa);
        if (PAIR == kPairSplit) {
          const uint32_t ob = __shfl_xor_sync(0xffffffffu, t.b, off);
          if (takes) t.b = max(t.b, ob);
        }
      }
    }
  }
  const int ea = block_exponent(t.a), eb = PAIR == kPairSplit ? block_exponent(t.b) : ea;
  const float ia = __uint_as_float(uint32_t(254 - ea) << 23);     // 2^-(ea - 127)
  const float ib = __uint_as_float(uint32_t(254 - eb) << 23);
  uint32_t c[E / 2];
#pragma unroll
  for (int i = 0; i < E; i += 2) {
    const Pair inv = i < E / 2 ? pair(ia, ia) : pair(ib, ib);
    const float2 f = unpair(mul2(x.v[i], inv)), g = unpair(mul2(x.v[i + 1], inv));
    c[i / 2] = __nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) |
               uint32_t(__nv_cvt_float2_to_fp8x2(g, __NV_SATFINITE, __NV_E4M3)) << 16;
  }
  if (odd) {                           // infinities, 448 so far, become NaN as NaN does
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float2 f = unpair(x.v[i]);
      if (fabsf(f.x) > 3.402823466e38f) c[i / 2] |= 0x7fu << (16 * (i & 1));
      if (fabsf(f.y) > 3.402823466e38f) c[i / 2] |= 0x7f00u << (16 * (i & 1));
    }
  }
  if ((L.a & 31) == 0 && L.na > 0) scales[L.a / 32] = uint8_t(ea);
  if (PAIR == kPairSplit && (L.b & 31) == 0 && L.nb > 0) scales[L.b / 32] = uint8_t(eb);
  if (!on || !codes.template in_bounds<E, ACC>(h, L, false)) return;
  store_codes<E, ACC>(codes.first(h), L.na, c);
  store_codes<E, ACC>(codes.second(h), L.nb, c + E / 4);
}

// Where a warp's item lies.
struct Item { int t, r0, r1; };
__device__ __forceinline__ Item item_at(const QkArgs &A, int64_t item) {
  Item I;
  // tokens are shared out only where they are fewer than the warps
  I.t = A.splits == 1 ? int(item) : int(unsigned(item) / unsigned(A.splits));
  I.r0 = int(item - int64_t(I.t) * A.splits) * A.rpi;
  I.r1 = min(A.p[0].H + A.p[1].H, I.r0 + A.rpi);
  return I;
}

// PACK: also write codes.
constexpr int kFwdE = 8, kBwdE = 4;
template <typename T, bool PACKED, bool PACK, int PAIR, int ACC, int LG>
__global__ void __launch_bounds__(kQkThreads, kBlocksPerSm) gdn_qk_fwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int E = kFwdE, U = 4, kWarps = kQkThreads / 32;
  __shared__ __align__(16) float w_all[2][kMaxD];
  __shared__ __align__(16) float cs_all[PAIR == kPairNone ? 1 : kWarps][kMaxD];
  __shared__ __align__(16) float rows_all[PAIR == kPairShared ? kWarps : 1][2 * kMaxD];
  __shared__ uint32_t tops_all[PACK && PAIR == kPairSplit ? kWarps * 64 : 1];
  const int lg = LG ? LG : A.lg, G = 1 << lg, R = 32 >> lg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> lg, l = lane & (G - 1);
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[PAIR == kPairShared ? warp : 0] + (lane & -G) * 2 * E;
  uint32_t *tops = tops_all + (PACK && PAIR == kPairSplit ? warp * 64 + sub * 8 : 0);
  // a step's exponents: R U rows of up to 8 (R halves as a row's lanes double)
  __shared__ uint8_t scales_all[PACK ? kWarps : 1][64];
  uint8_t *exps = scales_all[PACK ? warp : 0];
  const int blocks = (A.d + 31) / 32;
  const Lane L = lane_place<E, PAIR>(A, l);
  stage_weights<T, kQkThreads>(A, true, true, w_all);
  const int64_t nwarps = int64_t(gridDim.x) * kWarps, items = int64_t(A.T) * A.splits;
  for (int64_t item = int64_t(blockIdx.x) * kWarps + warp; item < items; item += nwarps) {
    const Item I = item_at(A, item);
    if (PAIR != kPairNone) make_angles(A, I.t, lane, E << lg, cs);
    for (int part = 0; part < 2; ++part) {
      const Part &P = A.p[part];
      const int first = part ? A.p[0].H : 0;
      const int h0 = max(I.r0 - first, 0), h1 = min(I.r1 - first, P.H);
      if (h0 >= h1) continue;
      Row<E> C, S;
      factors<E, PAIR>(A, L, l, cs, w_all[part], 1.f, C, S);
      using Src = Source<T, PACKED, E, PAIR, ACC>;
      const Src src(A, P, I.t, L);
      Rows<T> out(static_cast<T *>(P.out), I.t * P.out_ts, P.out_hs, L, false);
      const int64_t row0 = int64_t(I.t) * P.H;
      Rows<uint8_t> codes(P.codes, row0 * A.d, A.d, L, false);
      QK_CHECKED(bound(out, A, P.out, P.out_ts, P.out_hs, P.H);
                 bound(codes, A, P.codes, int64_t(A.T) * P.H * A.d);)
      for (int h = h0 + sub; h - sub < h1; h += R * U) {
        typename Src::Data raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) src.load(min(h + u * R, h1 - 1), L, raw[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h - sub + u * R >= h1) break;
          const bool on = h + u * R < h1;
          Row<E> x;
          unpack(raw[u], x);
          Scales sc = scales_of(raw[u]);
          if constexpr (PACK)
            if (P.codes)
              write_codes<T, E, PAIR, ACC>(A, codes, exps + (u * R + sub) * blocks, h + u * R, L, on, tops,
                                           raw[u], x);
          if (A.norm != GDN_NORM_NONE) {
            const float2 d = dots<E, (ACC >= E)>(L, x, x);
            // (d s) s and not d s^2, which could leave the range where the sum does not
            const float ss = PACKED ? d.x * sc.a * sc.a + d.y * sc.b * sc.b : d.x + d.y;
            const float r = rnorm(A, group_sum<LG>(ss, A.lg));
            sc.a *= r;
            sc.b *= r;
          }
          if (PACKED || A.norm != GDN_NORM_NONE) {
#pragma unroll
            for (int i = 0; i < E; ++i)
              x.v[i] = mul2(x.v[i], i < E / 2 || !PACKED ? pair(sc.a, sc.a) : pair(sc.b, sc.b));
          }
          turn<E, PAIR>(A, L, row_buf, C, S, x);
          if (on && (!PACK || P.out) && out.template in_bounds<E, ACC>(h + u * R, L, false)) {
            store_chunk<E, ACC>(out.first(h + u * R), L.na, x.v);
            store_chunk<E, ACC>(out.second(h + u * R), L.nb, x.v + E / 2);
          }
        }
        // consecutive heads' exponents are consecutive bytes: written together
        // (71 -> 67 us for 16384 x 32 rows, against a byte a lane as they arise)
        if (PACK && P.codes) {
          const int h_first = h - sub, bytes = min(R * U, h1 - h_first) * blocks;
          __syncwarp();
          for (int i = lane; i < bytes; i += 32)
            if (GDN_IN_BOUNDS(A.err, (row0 + h_first) * blocks + i, int64_t(A.T) * P.H * blocks))
              P.scales[(row0 + h_first) * blocks + i] = exps[i];
          __syncwarp();
        }
      }
    }
  }
}

// WEIGHTS: weights and their gradients.
template <typename T, typename DT, bool PACKED, bool WEIGHTS, int PAIR, int ACC, int LG>
__global__ void __launch_bounds__(WEIGHTS ? kQkThreads : kPlainBwdThreads,
                                  WEIGHTS ? kBlocksPerSm : kPlainBwdBlocksPerSm)
    gdn_qk_bwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int E = kBwdE, U = 2, kThreads = WEIGHTS ? kQkThreads : kPlainBwdThreads, kWarps = kThreads / 32;
  constexpr bool kWhole = ACC >= E;
  __shared__ __align__(16) float w_all[2][kMaxD], one[2][kMaxD];
  __shared__ __align__(16) float cs_all[PAIR == kPairNone ? 1 : kWarps][kMaxD];
  __shared__ __align__(16) float rows_all[PAIR == kPairShared || WEIGHTS ? kWarps : 1][kMaxD];
  const int lg = LG ? LG : A.lg, G = 1 << lg, R = 32 >> lg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> lg, l = lane & (G - 1);
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[PAIR == kPairShared || WEIGHTS ? warp : 0] + (lane & -G) * 2 * E;
  const Lane L = lane_place<E, PAIR>(A, l);
  if (WEIGHTS) stage_weights<T, kThreads>(A, false, true, w_all);
  stage_weights<T, kThreads>(A, true, false, one);
  const int64_t nwarps = int64_t(gridDim.x) * kWarps, items = int64_t(A.T) * A.splits;
  Row<E> dw[2];
#pragma unroll
  for (int i = 0; i < 2 * E; ++i) dw[i / E].v[i % E] = pair(0.f, 0.f);
  for (int64_t item = int64_t(blockIdx.x) * kWarps + warp; item < items; item += nwarps) {
    const Item I = item_at(A, item);
    if (PAIR != kPairNone) make_angles(A, I.t, lane, E << lg, cs);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const Part &P = A.p[part];
      const int first = part ? A.p[0].H : 0;
      const int h0 = max(I.r0 - first, 0), h1 = min(I.r1 - first, P.H);
      if (h0 >= h1) continue;
      Row<E> C, S, W;
      factors<E, PAIR>(A, L, l, cs, one[part], -1.f, C, S);
      if (WEIGHTS) {
        float w[2 * E];
        lds<E>(w_all[part] + L.a, w);
        lds<E>(w_all[part] + L.b, w + E);
#pragma unroll
        for (int i = 0; i < E; ++i) W.v[i] = pair(w[2 * i], w[2 * i + 1]);
      }
      using Src = Source<T, PACKED, E, PAIR, ACC>;
      const Src src(A, P, I.t, L);
      Rows<const DT> dy(static_cast<const DT *>(P.dy), I.t * P.dy_ts, P.dy_hs, L, true);
      Rows<T> out(static_cast<T *>(P.out), I.t * P.out_ts, P.out_hs, L, false);
      QK_CHECKED(bound(dy, A, P.dy, P.dy_ts, P.dy_hs, P.H); bound(out, A, P.out, P.out_ts, P.out_hs, P.H);)
      for (int h = h0 + sub; h - sub < h1; h += R * U) {
        typename Src::Data raw[U];
        Raw<DT, E> grad[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int hu = min(h + u * R, h1 - 1);
          src.load(hu, L, raw[u]);
          load_row<E, ACC>(dy, hu, L, grad[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h - sub + u * R >= h1) break;
          const bool on = h + u * R < h1;
          Row<E> x, z;
          unpack(raw[u], x);
          unpack(grad[u], z);
          Scales sc = scales_of(raw[u]);
          turn<E, PAIR>(A, L, row_buf, C, S, z);
          float r = 1.f, m = 0.f;
          Row<E> dh = z;
          if (WEIGHTS) {
#pragma unroll
            for (int i = 0; i < E; ++i) dh.v[i] = mul2(z.v[i], W.v[i]);
          }
          if (A.norm != GDN_NORM_NONE) {
            const float2 d = dots<E, kWhole>(L, x, x), e = dots<E, kWhole>(L, x, dh);
            const float ss = PACKED ? d.x * sc.a * sc.a + d.y * sc.b * sc.b : d.x + d.y;
            const float xd = PACKED ? e.x * sc.a + e.y * sc.b : e.x + e.y;
            r = rnorm(A, group_sum<LG>(ss, A.lg));
            m = group_sum<LG>(xd, A.lg) * r * A.inv_n;
          }
          const Pair rr = pair(r, r), mm = pair(-m, -m);
          const Pair ra = pair(r * sc.a, r * sc.a), rb = PACKED ? pair(r * sc.b, r * sc.b) : ra;
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const Pair hx = mul2(x.v[i], i < E / 2 ? ra : rb);
            if (WEIGHTS && on) dw[part].v[i] = fma2(z.v[i], hx, dw[part].v[i]);
            x.v[i] = A.norm == GDN_NORM_NONE ? dh.v[i] : mul2(fma2(hx, mm, dh.v[i]), rr);
          }
          if (on && out.template in_bounds<E, ACC>(h + u * R, L, false)) {
            store_chunk<E, ACC>(out.first(h + u * R), L.na, x.v);
            store_chunk<E, ACC>(out.second(h + u * R), L.nb, x.v + E / 2);
          }
        }
      }
    }
  }
  if (WEIGHTS) {    // the block's rows in a fixed order: warps 0..7, and in each its groups
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2 * E; ++i) {
        const float2 f = unpair(dw[part].v[i / 2]);
        const int e = i < E ? L.a + i : L.b + i - E;
        if (e < A.d) row_buf[e] = i & 1 ? f.y : f.x;
      }
      __syncthreads();
      for (int e = threadIdx.x; e < A.d; e += kThreads) {
        float s = 0.f;
        for (int i = 0; i < kWarps * R; ++i) s += rows_all[i / R][(i % R) * G * 2 * E + e];
        if (GDN_IN_BOUNDS(A.err, (int64_t(part) * gridDim.x + blockIdx.x) * A.d + e, A.dw_extent))
          A.dw_part[(int64_t(part) * gridDim.x + blockIdx.x) * A.d + e] = s;
      }
    }
  }
}

// dw = the sum of the blocks' partial sums, in a fixed order.
__global__ void __launch_bounds__(1024) gdn_qk_dw_kernel(const float *part, int blocks, int d,
                                                         float *dw_q, float *dw_k) {
  __shared__ float sm[32][33];
  float *out = blockIdx.y ? dw_k : dw_q;
  if (!out) return;
  const int e = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float s = 0.f;
  if (e < d)
    for (int b = w; b < blocks; b += 32) s += part[(int64_t(blockIdx.y) * blocks + b) * d + e];
  sm[w][threadIdx.x & 31] = s;
  __syncthreads();
  s = warp_sum(sm[threadIdx.x & 31][w]);
  const int eo = blockIdx.x * 32 + w;
  if ((threadIdx.x & 31) == 0 && eo < d) out[eo] = s;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Elements per access: the most that every pointer and stride (in bytes) allows.
int access_width(const QkArgs &A, int xe, int dye, bool packed) {
  for (int acc = 8; acc > 1; acc -= 4) {
    if (A.d % acc) continue;
    bool ok = true;
    for (const Part &P : A.p) {
      if (!P.H) continue;
      const int xb = xe == 4 ? 16 : acc * xe, db = dye == 4 ? 16 : acc * dye;
      if (packed) ok &= aligned(P.x, acc);
      else ok &= aligned(P.x, xb) && P.x_ts % xb == 0 && P.x_hs % xb == 0;
      if (P.dy) ok &= aligned(P.dy, db) && P.dy_ts % db == 0 && P.dy_hs % db == 0;
      if (P.out) ok &= aligned(P.out, xb) && P.out_ts % xb == 0 && P.out_hs % xb == 0;
      if (P.codes) ok &= aligned(P.codes, acc);
    }
    if (ok) return acc;
  }
  return 1;
}

// The way the pairs are handled: halves go in chunks where they fall into them.
int pair_mode(const gdn_qk_params *p, int acc, int e) {
  if (!p->rot) return kPairNone;
  if (p->interleaved) return kPairInterleaved;
  return acc >= 4 && p->rot % (2 * e) == 0 ? kPairSplit : kPairShared;
}

// Rows an item and items a token: whole tokens, whose cosines then serve every
// head, where there are enough of them for all warps; else fewer rows, down to
// one step of a warp.
unsigned plan(QkArgs &A, int e, int threads, int per_sm) {
  for (A.lg = 2; (2 * e) << A.lg < A.d; ++A.lg) {}
  const int rows = A.p[0].H + A.p[1].H, step = 32 >> A.lg, sms = device_sms();
  const int64_t warps = int64_t(sms > 0 ? sms : 1) * per_sm * (threads / 32);
  int64_t want = (int64_t(A.T) * rows + warps - 1) / warps;          // rows a warp
  want = (want + step - 1) / step * step;
  A.rpi = int(want < 1 ? 1 : want < rows ? want : rows > 0 ? rows : 1);
  A.splits = (rows + A.rpi - 1) / A.rpi;
  const int64_t blocks = (int64_t(A.T) * A.splits + threads / 32 - 1) / (threads / 32);
  const int64_t most = int64_t(sms > 0 ? sms : 1) * per_sm;
  return unsigned(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

// Turns the run-time choices into template arguments. Accesses of eight
// elements: a chunk of eight (E = 8), or two chunks of four side by side.
//
// Measured for 16384 x 32 rows of 128, in us. The common width of a head, 65 to
// 128 elements, is known to the compiler where the accesses are wide. That pays
// in the backward kernels (92 against 97 without weights and 103 against 112 with
// them, 103 against 117 from codes, fp32 rows 117 against 126) and a little in
// the forward ones (46.5 against 47.4, with codes 68 against 70, fp32 rows 0 to 3
// %). Eight elements an access instead of four, width unknown: forward 47 against
// 50 (interleaved 50 against 56, with codes 70 against 77); in the backward
// kernels nothing (112.3 against 112.3, and within 0.5 % for rows of 64, 192 and
// 256) but for bf16 rows with halves through shared memory (111 against 113), so
// there it comes with the known width or with those.
template <int V> struct Const { static constexpr int value = V; };
template <int E, typename F>
void with_variant(int pair, int acc, int lg, F f) {
  constexpr int known = E == 8 ? 3 : 4;
  auto pick = [&](auto a, auto g) {
    constexpr int wide = decltype(a)::value, split = wide >= E ? E : 4;
    if (pair == kPairNone) f(Const<kPairNone>{}, a, g);
    else if (pair == kPairInterleaved) f(Const<kPairInterleaved>{}, a, g);
    else f(Const<kPairSplit>{}, Const<split>{}, g);
  };
  if (pair == kPairShared) {
    if (acc == 8) f(Const<kPairShared>{}, Const<8>{}, Const<0>{});
    else if (acc >= 4) f(Const<kPairShared>{}, Const<4>{}, Const<0>{});
    else f(Const<kPairShared>{}, Const<1>{}, Const<0>{});
  } else if (acc == 8 && lg == known) {
    pick(Const<8>{}, Const<known>{});
  } else if (acc >= 4) {
    if (E == 8 && acc == 8) pick(Const<E>{}, Const<0>{});
    else pick(Const<4>{}, Const<0>{});
  } else if (pair == kPairNone) {            // halves in chunks need accesses of four
    f(Const<kPairNone>{}, Const<1>{}, Const<0>{});
  } else {
    f(Const<kPairInterleaved>{}, Const<1>{}, Const<0>{});
  }
}

template <bool PACKED, bool PACK>
cudaError_t fwd_launch(const QkArgs &A, int dtype, int pair, int acc, unsigned grid, cudaStream_t s) {
  auto go = [&](auto type) {
    using T = decltype(type);
    with_variant<kFwdE>(pair, acc, A.lg, [&](auto p, auto a, auto g) {
      gdn_qk_fwd_kernel<T, PACKED, PACK, decltype(p)::value, decltype(a)::value, decltype(g)::value>
          <<<grid, kQkThreads, 0, s>>>(A);
    });
  };
  if (dtype == GDN_BF16) go(__nv_bfloat16{});
  else go(float{});
  return cudaGetLastError();
}
template <bool PACKED, bool WEIGHTS>
cudaError_t bwd_launch(const QkArgs &A, int dtype, int grad_dtype, int pair, int acc, unsigned grid,
                       cudaStream_t s) {
  auto go = [&](auto type, auto grad) {
    using T = decltype(type);
    using DT = decltype(grad);
    with_variant<kBwdE>(pair, acc, A.lg, [&](auto p, auto a, auto g) {
      gdn_qk_bwd_kernel<T, DT, PACKED, WEIGHTS, decltype(p)::value, decltype(a)::value, decltype(g)::value>
          <<<grid, WEIGHTS ? kQkThreads : kPlainBwdThreads, 0, s>>>(A);
    });
  };
  if (dtype == GDN_F32) go(float{}, float{});
  else if (grad_dtype == GDN_F32) go(__nv_bfloat16{}, float{});
  else go(__nv_bfloat16{}, __nv_bfloat16{});
  return cudaGetLastError();
}

int check_params(const gdn_qk_params *p) {
  if (!p || (p->dtype != GDN_BF16 && p->dtype != GDN_F32)) return GDN_ERR_INVALID_ARG;
  if (p->T < 0 || p->H_q < 0 || p->H_k < 0 || p->d < 1 || p->rot < 0 || p->rot % 2 ||
      p->rot > p->d || p->norm < GDN_NORM_NONE || p->norm > GDN_NORM_RMS)
    return GDN_ERR_INVALID_ARG;
  // a token's heads, and the step past the last of them, are counted in 32 bits
  if (p->d > kMaxD || int64_t(p->H_q) + p->H_k > 1 << 30) return GDN_ERR_UNSUPPORTED;
  if (p->rot && p->T && (!p->positions || !p->inv_freq)) return GDN_ERR_INVALID_ARG;
  const size_t e = p->dtype == GDN_BF16 ? 2 : 4;
  if (!aligned(p->positions, 4) || !aligned(p->inv_freq, 8) || !aligned(p->w_q, e) ||
      !aligned(p->w_k, e))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// Rows that do not overlap, token by token or head by head.
bool rows_ok(const gdn_rows *r, int T, int H, int d, size_t e) {
  if (!r || !r->data || !aligned(r->data, e)) return false;
  const int64_t ts = r->token_stride, hs = r->head_stride;
  if (ts < d || hs < d || hs >= (1 << 28)) return false;
  return ts >= int64_t(H - 1) * hs + d || hs >= int64_t(T - 1) * ts + d;
}

int fill(QkArgs &A, const gdn_qk_params *p, const gdn_rows *const x[2],
         const gdn_packed *const x8[2], const gdn_rows *const dy[2], size_t dye,
         const gdn_rows *const out[2], const gdn_packed *const out8[2]) {
  const size_t e = p->dtype == GDN_BF16 ? 2 : 4;
  QK_CHECKED(A.err = static_cast<uint32_t *>(qk_checked_block());)
  A.pos = p->positions;
  A.inv_freq = p->inv_freq;
  A.T = p->T; A.d = p->d; A.rot = p->rot; A.norm = p->norm;
  A.eps = p->eps; A.w0 = p->weight_offset; A.rope_scale = p->rope_scale;
  A.inv_n = p->norm == GDN_NORM_RMS ? 1.f / float(p->d) : 1.f;
  for (int i = 0; i < 2; ++i) {
    Part &P = A.p[i];
    P.H = i ? p->H_k : p->H_q;
    P.w = i ? p->w_k : p->w_q;
    P.scale = i ? 1.f : p->q_scale;
    if (!P.H || !p->T) { P.H = 0; continue; }
    if (x8) {
      if (!x8[i] || !x8[i]->codes || !x8[i]->scales) return GDN_ERR_INVALID_ARG;
      P.x = x8[i]->codes;
      P.x_scales = x8[i]->scales;
    } else {
      if (!rows_ok(x[i], p->T, P.H, p->d, e)) return GDN_ERR_INVALID_ARG;
      P.x = x[i]->data; P.x_ts = x[i]->token_stride * e; P.x_hs = int(x[i]->head_stride * e);
    }
    if (dy) {
      if (!rows_ok(dy[i], p->T, P.H, p->d, dye)) return GDN_ERR_INVALID_ARG;
      P.dy = dy[i]->data; P.dy_ts = dy[i]->token_stride * dye; P.dy_hs = int(dy[i]->head_stride * dye);
    }
    if (out8 && out8[i] && out8[i]->codes) {
      if (!out8[i]->scales) return GDN_ERR_INVALID_ARG;
      P.codes = out8[i]->codes;
      P.scales = out8[i]->scales;
    }
    if (out[i] && out[i]->data) {
      if (!rows_ok(out[i], p->T, P.H, p->d, e)) return GDN_ERR_INVALID_ARG;
      P.out = out[i]->data; P.out_ts = out[i]->token_stride * e; P.out_hs = int(out[i]->head_stride * e);
    } else if (!P.codes) {
      return GDN_ERR_INVALID_ARG;
    }
  }
  return GDN_OK;
}

template <bool PACKED>
int run_fwd(const gdn_qk_params *p, const gdn_rows *const x[2], const gdn_packed *const x8[2],
            const gdn_rows *const out[2], const gdn_packed *const out8[2], void *stream) {
  int rc = check_params(p);
  if (rc != GDN_OK) return rc;
  QkArgs A{};
  rc = fill(A, p, x, PACKED ? x8 : nullptr, nullptr, 0, out, out8);
  if (rc != GDN_OK) return rc;
  if (!A.p[0].H && !A.p[1].H) return GDN_OK;
  const bool pack = A.p[0].codes || A.p[1].codes;
  const unsigned grid = plan(A, kFwdE, kQkThreads, kBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, 2, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pair = pair_mode(p, acc, kFwdE);
  cudaError_t e;
  if constexpr (PACKED) e = fwd_launch<true, false>(A, p->dtype, pair, acc, grid, s);
  else if (pack) e = fwd_launch<false, true>(A, p->dtype, pair, acc, grid, s);
  else e = fwd_launch<false, false>(A, p->dtype, pair, acc, grid, s);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <bool PACKED>
int run_bwd(const gdn_qk_params *p, const gdn_rows *const dy[2], int grad_dtype,
            const gdn_rows *const x[2], const gdn_packed *const x8[2], const gdn_rows *const out[2],
            float *dw_q, float *dw_k, void *ws, size_t ws_bytes, void *stream) {
  int rc = check_params(p);
  if (rc != GDN_OK) return rc;
  if (grad_dtype != GDN_BF16 && grad_dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
  if (p->dtype == GDN_F32 && grad_dtype == GDN_BF16) return GDN_ERR_UNSUPPORTED;
  if (!p->w_q != !dw_q || !p->w_k != !dw_k) return GDN_ERR_INVALID_ARG;
  if (!aligned(dw_q, 4) || !aligned(dw_k, 4)) return GDN_ERR_INVALID_ARG;
  if (ws_bytes < gdn_qk_norm_rope_bwd_workspace_size(p)) return GDN_ERR_WORKSPACE;
  if ((dw_q || dw_k) && (!ws || !aligned(ws, 256))) return GDN_ERR_WORKSPACE;
  QkArgs A{};
  rc = fill(A, p, x, PACKED ? x8 : nullptr, dy, grad_dtype == GDN_BF16 ? 2 : 4, out, nullptr);
  if (rc != GDN_OK) return rc;
  A.dw_part = static_cast<float *>(ws);
  QK_CHECKED(A.dw_extent = ws_bytes / sizeof(float);)
  const unsigned grid = dw_q || dw_k ? plan(A, kBwdE, kQkThreads, kBlocksPerSm)
                                     : plan(A, kBwdE, kPlainBwdThreads, kPlainBwdBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, grad_dtype == GDN_BF16 ? 2 : 4, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!A.p[0].H && !A.p[1].H && !dw_q && !dw_k) return GDN_OK;
  const int pair = pair_mode(p, acc, kBwdE);
  const cudaError_t e =
      dw_q || dw_k ? bwd_launch<PACKED, true>(A, p->dtype, grad_dtype, pair, acc, grid, s)
                   : bwd_launch<PACKED, false>(A, p->dtype, grad_dtype, pair, acc, grid, s);
  if (e != cudaSuccess) return GDN_ERR_CUDA;
  if (dw_q || dw_k) {
    gdn_qk_dw_kernel<<<dim3((p->d + 31) / 32, 2), 1024, 0, s>>>(A.dw_part, int(grid), p->d, dw_q, dw_k);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

}  // namespace

#if GDN_CHECKS
namespace {
__device__ uint32_t g_checked[64];
}
void *qk_checked_block() {
  void *p = nullptr;
  return cudaGetSymbolAddress(&p, g_checked) == cudaSuccess ? p : nullptr;
}
#endif
}  // namespace gdn

using namespace gdn;

extern "C" {

int gdn_qk_norm_rope_fwd(const gdn_qk_params *p, const gdn_rows *q, const gdn_rows *k,
                         const gdn_rows *q_out, const gdn_rows *k_out, const gdn_packed *q_packed,
                         const gdn_packed *k_packed, void *stream) {
  const gdn_rows *x[2] = {q, k}, *out[2] = {q_out, k_out};
  const gdn_packed *out8[2] = {q_packed, k_packed};
  return run_fwd<false>(p, x, nullptr, out, out8, stream);
}

int gdn_qk_norm_rope_fwd_packed(const gdn_qk_params *p, const gdn_packed *q, const gdn_packed *k,
                                const gdn_rows *q_out, const gdn_rows *k_out, void *stream) {
  const gdn_packed *x8[2] = {q, k};
  const gdn_rows *out[2] = {q_out, k_out};
  return run_fwd<true>(p, nullptr, x8, out, nullptr, stream);
}

size_t gdn_qk_norm_rope_bwd_workspace_size(const gdn_qk_params *p) {
  if (check_params(p) != GDN_OK || (!p->w_q && !p->w_k)) return 0;
  return align_up(size_t(2) * device_sms() * kBlocksPerSm * p->d * sizeof(float), 256);
}

int gdn_qk_norm_rope_bwd(const gdn_qk_params *p, const gdn_rows *dq_out, const gdn_rows *dk_out,
                         int grad_dtype, const gdn_rows *q, const gdn_rows *k, const gdn_rows *dq,
                         const gdn_rows *dk, float *dw_q, float *dw_k, void *workspace,
                         size_t workspace_bytes, void *stream) {
  const gdn_rows *x[2] = {q, k}, *dy[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
  return run_bwd<false>(p, dy, grad_dtype, x, nullptr, out, dw_q, dw_k, workspace, workspace_bytes,
                        stream);
}

int gdn_qk_norm_rope_bwd_packed(const gdn_qk_params *p, const gdn_rows *dq_out,
                                const gdn_rows *dk_out, int grad_dtype, const gdn_packed *q,
                                const gdn_packed *k, const gdn_rows *dq, const gdn_rows *dk,
                                float *dw_q, float *dw_k, void *workspace, size_t workspace_bytes,
                                void *stream) {
  const gdn_packed *x8[2] = {q, k};
  const gdn_rows *dy[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
  return run_bwd<true>(p, dy, grad_dtype, nullptr, x8, out, dw_q, dw_k, workspace, workspace_bytes,
                       stream);
}

}  // extern "C"
