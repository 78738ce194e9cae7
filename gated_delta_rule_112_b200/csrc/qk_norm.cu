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
// A group of G lanes (the power of two from d / 8 up) holds a row, eight
// consecutive elements a lane, so the sums are log2 G shuffles and a pair's
// partner is in the same lane (interleaved), G' lanes away (halves, rot a
// multiple of 16), or fetched through a warp's own shared memory (other rot).
// A warp takes an item: up to RPI heads of q or of k of one token. It forms
// the item's cosines and sines once: the angle in turns is position *
// inv_freq / 2 pi in fp64, less its whole turns, so far positions lose
// nothing; fp32 sine and cosine of the remainder follow.
//
// Checkpoint: 32 consecutive elements of a row share a power of two 2^e, the
// smallest (e >= -127) with max|x| <= 448 * 2^e over the block's finite
// elements, and are stored as e4m3 of x 2^-e (to nearest even); an element that
// is not finite becomes NaN. One byte e + 127 a block: no code is rounded twice
// and 2^e times a code is exact in bf16.
#include <cuda_fp8.h>

#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kQkThreads = 256, kQkWarps = kQkThreads / 32;
constexpr int kMaxD = 256;

enum { kPairNone, kPairInterleaved, kPairHalfLanes, kPairHalfShared };

struct Part {                     // q or k
  const void *x;                  // rows (dtype), or e4m3 codes
  const uint8_t *x_scales;        // set when x holds codes
  const void *dy;
  void *out;                      // y or dx; may be null when only codes are wanted
  uint8_t *codes, *scales;        // checkpoint to write, or null
  const void *w;
  int64_t x_ts, x_hs, dy_ts, dy_hs, out_ts, out_hs;
  int H, splits;                  // heads, items per token
  float scale;
};

struct QkArgs {
  Part p[2];
  const int32_t *pos;
  const double *inv_freq;
  float *dw_part;                 // [2][gridDim.x][d] partial weight gradients
  int T, d, rot, rpi, norm, lg;     // lg: log2 of the lanes of a row
  float eps, w0, rope_scale, inv_n;
};

// Eight elements of a row as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> { uint32_t w[4]; };
template <>
struct Raw<float> { float w[8]; };
struct Codes { uint2 w; uint32_t e; };

// n: how many of the eight exist; ACC: elements per access (all pointers and
// strides are multiples of it).
template <int ACC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, int n, Raw<__nv_bfloat16> &r) {
  r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0;
  if (ACC == 8) {
    if (n > 0) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p));
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
  } else if (ACC == 4) {
    if (n > 0) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
      r.w[0] = v.x; r.w[1] = v.y;
    }
    if (n > 4) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p + 4));
      r.w[2] = v.x; r.w[3] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n)
        r.w[i / 2] |= uint32_t(*reinterpret_cast<const uint16_t *>(p + i)) << (16 * (i & 1));
  }
}
template <int ACC>
__device__ __forceinline__ void load8(const float *p, int n, Raw<float> &r) {
  if (ACC >= 4) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (n > 0) a = __ldcs(reinterpret_cast<const float4 *>(p));
    if (n > 4) b = __ldcs(reinterpret_cast<const float4 *>(p + 4));
    r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
    r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = i < n ? p[i] : 0.f;
  }
}
template <int ACC>
__device__ __forceinline__ void load_codes(const uint8_t *p, const uint8_t *e, int n, Codes &r) {
  r.w = make_uint2(0, 0);
  r.e = n > 0 ? *e : 127;
  if (ACC == 8) {
    if (n > 0) r.w = __ldcs(reinterpret_cast<const uint2 *>(p));
  } else if (ACC == 4) {
    if (n > 0) r.w.x = __ldcs(reinterpret_cast<const uint32_t *>(p));
    if (n > 4) r.w.y = __ldcs(reinterpret_cast<const uint32_t *>(p + 4));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) (i < 4 ? r.w.x : r.w.y) |= uint32_t(p[i]) << (8 * (i & 3));
  }
}

__device__ __forceinline__ void unpack8(const Raw<__nv_bfloat16> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) { x[2 * i] = bf_lo(r.w[i]); x[2 * i + 1] = bf_hi(r.w[i]); }
}
__device__ __forceinline__ void unpack8(const Raw<float> &r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = r.w[i];
}
// 2^(b - 127), b in [0, 254]: 2^-127 lies below the normal range.
__device__ __forceinline__ float pow2_biased(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ void unpack8(const Codes &r, float (&x)[8]) {
  const float s = pow2_biased(r.e);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? r.w.x : r.w.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((w >> (16 * (i & 1))) & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x[2 * i] = f.x * s;
    x[2 * i + 1] = f.y * s;
  }
}

template <int ACC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, int n, const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = bf_pack(x[2 * i], x[2 * i + 1]);
  if (ACC == 8) {
    if (n > 0) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else if (ACC == 4) {
    if (n > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    if (n > 4) *reinterpret_cast<uint2 *>(p + 4) = make_uint2(w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) *reinterpret_cast<uint16_t *>(p + i) = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
}
template <int ACC>
__device__ __forceinline__ void store8(float *p, int n, const float (&x)[8]) {
  if (ACC >= 4) {
    if (n > 0) *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
    if (n > 4) *reinterpret_cast<float4 *>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = x[i];
  }
}
template <int ACC>
__device__ __forceinline__ void store_codes(uint8_t *p, int n, uint2 w) {
  if (ACC == 8) {
    if (n > 0) *reinterpret_cast<uint2 *>(p) = w;
  } else if (ACC == 4) {
    if (n > 0) *reinterpret_cast<uint32_t *>(p) = w.x;
    if (n > 4) *reinterpret_cast<uint32_t *>(p + 4) = w.y;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = uint8_t((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

// Sum over the G = 2^lg lanes of a row (8, 16 or 32).
__device__ __forceinline__ float group_sum(float x, int lg) {
  if (lg > 4) x += __shfl_xor_sync(0xffffffffu, x, 16);
  if (lg > 3) x += __shfl_xor_sync(0xffffffffu, x, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// The lane's share of an item's cosines and sines: c[i], s[i] for element
// e0 + i (interleaved: for pair e0 / 2 + i), the sine signed for that element.
struct Turn { float c[8], s[8]; };

template <int PAIR>
__device__ __forceinline__ void make_turn(const QkArgs &A, int t, float sign, int e0, int lane,
                                          float *cs, Turn &R) {
  if (PAIR == kPairNone) return;
  const int half = A.rot / 2;
  const double p = double(A.pos[t]);
  __syncwarp();
  for (int j = lane; j < half; j += 32) {
    double turns = p * A.inv_freq[j] * 0.15915494309189533577;   // 1 / (2 pi)
    turns -= rint(turns);
    float s, c;
    sincospif(float(2.0 * turns), &s, &c);
    cs[j] = c * A.rope_scale;
    cs[kMaxD / 2 + j] = s * A.rope_scale * sign;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (PAIR == kPairInterleaved) {
      if (i < 4) {
        const int j = e0 / 2 + i;
        R.c[i] = j < half ? cs[j] : 1.f;
        R.s[i] = j < half ? cs[kMaxD / 2 + j] : 0.f;
      }
    } else {
      const int e = e0 + i, j = e < half ? e : e - half;
      const bool on = e < A.rot;
      R.c[i] = on ? cs[j] : 1.f;
      R.s[i] = on ? (e < half ? -cs[kMaxD / 2 + j] : cs[kMaxD / 2 + j]) : 0.f;
    }
  }
}

template <int PAIR>
__device__ __forceinline__ void turn8(const QkArgs &A, const Turn &R, int e0, int lane, float *row,
                                      float (&z)[8]) {
  if (PAIR == kPairInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = z[2 * i], b = z[2 * i + 1];
      if (e0 + 2 * i < A.rot) {
        z[2 * i] = a * R.c[i] - b * R.s[i];
        z[2 * i + 1] = b * R.c[i] + a * R.s[i];
      }
    }
  } else if (PAIR == kPairHalfLanes) {
    const int off = A.rot / 16;
    const int src = e0 < A.rot / 2 ? lane + off : e0 < A.rot ? lane - off : lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, z[i], src);
      if (e0 < A.rot) z[i] = z[i] * R.c[i] + o * R.s[i];
    }
  } else if (PAIR == kPairHalfShared) {   // row: this group's part of the warp's buffer
    const int half = A.rot / 2;
    __syncwarp();
    *reinterpret_cast<float4 *>(row + e0) = make_float4(z[0], z[1], z[2], z[3]);
    *reinterpret_cast<float4 *>(row + e0 + 4) = make_float4(z[4], z[5], z[6], z[7]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = e0 + i;
      if (e < A.rot) z[i] = z[i] * R.c[i] + row[e < half ? e + half : e - half] * R.s[i];
    }
  }
}

__device__ __forceinline__ float rnorm(const QkArgs &A, float ss) {
  return A.norm == GDN_NORM_NONE ? 1.f : rsqrtf(ss * A.inv_n + A.eps);
}

template <typename T, int ACC>
__device__ __forceinline__ void load_w(const QkArgs &A, const Part &P, int e0, int n, float (&w)[8]) {
  if (P.w) {
    const T *p = static_cast<const T *>(P.w) + e0;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = i < n ? to_f32(p[i]) + A.w0 : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
  }
}

// Where an item's rows are.
struct Item { int t, h0, h1; };
__device__ __forceinline__ Item item_at(const QkArgs &A, const Part &P, int64_t item) {
  Item I;
  I.t = int(item / P.splits);
  I.h0 = int(item % P.splits) * A.rpi;
  I.h1 = min(P.H, I.h0 + A.rpi);
  return I;
}

// Source of the rows: T in memory, or codes.
template <typename T, bool PACKED, int ACC>
struct Source {
  Raw<T> raw;
  __device__ __forceinline__ void load(const QkArgs &, const Part &P, int t, int h, int e0, int n) {
    load8<ACC>(static_cast<const T *>(P.x) + t * P.x_ts + h * P.x_hs + e0, n, raw);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack8(raw, x); }
};
template <typename T, int ACC>
struct Source<T, true, ACC> {
  Codes raw;
  __device__ __forceinline__ void load(const QkArgs &A, const Part &P, int t, int h, int e0, int n) {
    const int64_t row = int64_t(t) * P.H + h;
    load_codes<ACC>(static_cast<const uint8_t *>(P.x) + row * A.d + e0,
                    P.x_scales + row * ((A.d + 31) / 32) + e0 / 32, n, raw);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const { unpack8(raw, x); }
};

template <int ACC>
__device__ __forceinline__ void write_codes(const QkArgs &A, const Part &P, int64_t row, int e0, int n,
                                            bool on, const float (&x)[8]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    top = fmaxf(top, a <= 3.402823466e38f ? a : 0.f);     // false for infinities and NaN
  }
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
  // 448 = 1.75 * 2^8: e = exponent - 8, and one more where the significand is above 1.75
  const uint32_t bits = __float_as_uint(top);
  const int be = max(int(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), 0);
  const float inv = __uint_as_float(uint32_t(254 - be) << 23);     // 2^-(be - 127)
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 v = make_float2(x[2 * i] * inv, x[2 * i + 1] * inv);
    v.x = fabsf(x[2 * i]) <= 3.402823466e38f ? v.x : __int_as_float(0x7fffffff);
    v.y = fabsf(x[2 * i + 1]) <= 3.402823466e38f ? v.y : __int_as_float(0x7fffffff);
    c[i] = __nv_cvt_float2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
  }
  if (!on) return;
  store_codes<ACC>(P.codes + row * A.d + e0, n, make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16));
  if ((e0 & 31) == 0 && n > 0) P.scales[row * ((A.d + 31) / 32) + e0 / 32] = uint8_t(be);
}

template <typename T, bool PACKED, int PAIR, int ACC>
__global__ void __launch_bounds__(kQkThreads) gdn_qk_fwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int U = 4;
  const int G = 1 << A.lg, R = 32 >> A.lg;
  __shared__ float cs_all[PAIR == kPairNone ? 1 : kQkWarps][kMaxD];
  __shared__ __align__(16) float rows_all[PAIR == kPairHalfShared ? kQkWarps : 1][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> A.lg;
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[PAIR == kPairHalfShared ? warp : 0] + (lane & -G) * 8;
  const int e0 = (lane & (G - 1)) * 8, n = max(0, min(8, A.d - e0));
  const int64_t nwarps = int64_t(gridDim.x) * kQkWarps;
  for (int part = 0; part < 2; ++part) {
    const Part &P = A.p[part];
    const int64_t items = int64_t(A.T) * P.splits;
    float w[8];
    load_w<T, ACC>(A, P, e0, n, w);
    for (int64_t item = int64_t(blockIdx.x) * kQkWarps + warp; item < items; item += nwarps) {
      const Item I = item_at(A, P, item);
      Turn turn;
      make_turn<PAIR>(A, I.t, 1.f, e0, lane, cs, turn);
      for (int h0 = I.h0; h0 < I.h1; h0 += R * U) {
        Source<T, PACKED, ACC> src[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * R + sub;
          src[u].load(A, P, I.t, h < I.h1 ? h : I.h0, e0, h < I.h1 ? n : 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h0 + u * R >= I.h1) break;
          const int h = h0 + u * R + sub;
          const bool on = h < I.h1;
          float x[8];
          src[u].get(x);
          if (!PACKED && P.codes)
            write_codes<ACC>(A, P, int64_t(I.t) * P.H + h, e0, n, on, x);
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
          const float r = rnorm(A, group_sum(ss, A.lg));
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
          turn8<PAIR>(A, turn, e0, lane, row_buf, x);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] *= P.scale;
          if (on && P.out)
            store8<ACC>(static_cast<T *>(P.out) + I.t * P.out_ts + h * P.out_hs + e0, n, x);
        }
      }
    }
  }
}

template <typename T, typename DT, bool PACKED, int PAIR, int ACC>
__global__ void __launch_bounds__(kQkThreads) gdn_qk_bwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int U = 2;
  const int G = 1 << A.lg, R = 32 >> A.lg;
  __shared__ float cs_all[PAIR == kPairNone ? 1 : kQkWarps][kMaxD];
  __shared__ __align__(16) float rows_all[kQkWarps][kMaxD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> A.lg;
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[warp] + (lane & -G) * 8;
  const int e0 = (lane & (G - 1)) * 8, n = max(0, min(8, A.d - e0));
  const int64_t nwarps = int64_t(gridDim.x) * kQkWarps;
  for (int part = 0; part < 2; ++part) {
    const Part &P = A.p[part];
    const int64_t items = int64_t(A.T) * P.splits;
    float w[8], dw[8];
    load_w<T, ACC>(A, P, e0, n, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[i] = 0.f;
    for (int64_t item = int64_t(blockIdx.x) * kQkWarps + warp; item < items; item += nwarps) {
      const Item I = item_at(A, P, item);
      Turn turn;
      make_turn<PAIR>(A, I.t, -1.f, e0, lane, cs, turn);
      for (int h0 = I.h0; h0 < I.h1; h0 += R * U) {
        Source<T, PACKED, ACC> src[U];
        Raw<DT> grad[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int h = h0 + u * R + sub;
          const bool on = h < I.h1;
          src[u].load(A, P, I.t, on ? h : I.h0, e0, on ? n : 0);
          load8<ACC>(static_cast<const DT *>(P.dy) + I.t * P.dy_ts + (on ? h : I.h0) * P.dy_hs + e0,
                     on ? n : 0, grad[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h0 + u * R >= I.h1) break;
          const int h = h0 + u * R + sub;
          float x[8], z[8];
          src[u].get(x);
          unpack8(grad[u], z);
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] *= P.scale;
          turn8<PAIR>(A, turn, e0, lane, row_buf, z);
          float ss = 0.f, dot = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) { ss += x[i] * x[i]; dot += z[i] * w[i] * x[i]; }
          const float r = rnorm(A, group_sum(ss, A.lg));
          const float m = A.norm == GDN_NORM_NONE ? 0.f : group_sum(dot, A.lg) * r * A.inv_n;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float hx = x[i] * r;
            if (P.w) dw[i] += z[i] * hx;
            x[i] = A.norm == GDN_NORM_NONE ? z[i] * w[i] : r * (z[i] * w[i] - hx * m);
          }
          if (h < I.h1)
            store8<ACC>(static_cast<T *>(P.out) + I.t * P.out_ts + h * P.out_hs + e0, n, x);
        }
      }
    }
    if (P.w) {      // the block's rows in a fixed order: warps 0..7, and in each its groups
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) row_buf[e0 + i] = dw[i];
      __syncthreads();
      for (int e = threadIdx.x; e < A.d; e += kQkThreads) {
        float s = 0.f;
        for (int i = 0; i < kQkWarps * R; ++i) s += rows_all[i / R][(i % R) * G * 8 + e];
        A.dw_part[(int64_t(part) * gridDim.x + blockIdx.x) * A.d + e] = s;
      }
      __syncthreads();
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

// Elements per access: the most that every pointer and stride allows.
int access_width(const QkArgs &A, size_t xe, size_t dye, bool packed) {
  for (int acc = 8; acc > 1; acc -= 4) {
    if (A.d % acc) continue;
    bool ok = true;
    for (const Part &P : A.p) {
      if (!P.H) continue;
      const size_t xb = xe == 4 ? 16 : acc * xe, db = dye == 4 ? 16 : acc * dye;
      if (packed) ok &= aligned(P.x, acc);
      else ok &= aligned(P.x, xb) && P.x_ts % acc == 0 && P.x_hs % acc == 0;
      if (P.dy) ok &= aligned(P.dy, db) && P.dy_ts % acc == 0 && P.dy_hs % acc == 0;
      if (P.out) ok &= aligned(P.out, xb) && P.out_ts % acc == 0 && P.out_hs % acc == 0;
      if (P.codes) ok &= aligned(P.codes, acc);
    }
    if (ok) return acc;
  }
  return 1;
}

int pair_mode(const gdn_qk_params *p) {
  if (!p->rot) return kPairNone;
  if (p->interleaved) return kPairInterleaved;
  return p->rot % 16 == 0 ? kPairHalfLanes : kPairHalfShared;
}

// Blocks of a launch over `items` warps' worth of work.
unsigned grid_for(int64_t items, int sms, int per_sm) {
  const int64_t blocks = (items + kQkWarps - 1) / kQkWarps, most = int64_t(sms) * per_sm;
  return unsigned(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

constexpr int kFwdBlocksPerSm = 4, kBwdBlocksPerSm = 4;

// Turns the run-time choices into template arguments. A variant for each way
// the pairs lie, at the widest access (16 bytes of T); narrower accesses, which
// unaligned rows take, share partners through shared memory in every case of
// halves.
template <int V> struct Const { static constexpr int value = V; };
template <typename T, typename F>
void with_variant(int pair, int acc, F f) {
  constexpr int wide = sizeof(T) == 2 ? 8 : 4;
  auto pick = [&](auto a) {
    if (pair == kPairNone) f(Const<kPairNone>{}, a);
    else if (pair == kPairInterleaved) f(Const<kPairInterleaved>{}, a);
    else f(Const<kPairHalfShared>{}, a);
  };
  if (acc >= wide && pair == kPairHalfLanes) f(Const<kPairHalfLanes>{}, Const<wide>{});
  else if (acc >= wide) pick(Const<wide>{});
  else if (acc >= 4) pick(Const<4>{});
  else pick(Const<1>{});
}

template <bool PACKED>
cudaError_t fwd_launch(const QkArgs &A, int dtype, int pair, int acc, unsigned grid, cudaStream_t s) {
  auto go = [&](auto type) {
    using T = decltype(type);
    with_variant<T>(pair, acc, [&](auto p, auto a) {
      gdn_qk_fwd_kernel<T, PACKED, decltype(p)::value, decltype(a)::value>
          <<<grid, kQkThreads, 0, s>>>(A);
    });
  };
  if (dtype == GDN_BF16) go(__nv_bfloat16{});
  else go(float{});
  return cudaGetLastError();
}
template <bool PACKED>
cudaError_t bwd_launch(const QkArgs &A, int dtype, int grad_dtype, int pair, int acc, unsigned grid,
                       cudaStream_t s) {
  auto go = [&](auto type, auto grad) {
    using T = decltype(type);
    using DT = decltype(grad);
    with_variant<T>(pair, acc, [&](auto p, auto a) {
      gdn_qk_bwd_kernel<T, DT, PACKED, decltype(p)::value, decltype(a)::value>
          <<<grid, kQkThreads, 0, s>>>(A);
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
  if (p->d > kMaxD) return GDN_ERR_UNSUPPORTED;
  if (p->rot && p->T && (!p->positions || !p->inv_freq)) return GDN_ERR_INVALID_ARG;
  const size_t e = p->dtype == GDN_BF16 ? 2 : 4;
  if (!aligned(p->positions, 4) || !aligned(p->inv_freq, 8) || !aligned(p->w_q, e) ||
      !aligned(p->w_k, e))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

bool rows_ok(const gdn_rows *r, int H, int d, size_t e) {
  return r && r->data && aligned(r->data, e) && r->head_stride >= d &&
         r->token_stride >= (H > 0 ? int64_t(H - 1) * r->head_stride + d : 0);
}

int fill(QkArgs &A, const gdn_qk_params *p, const gdn_rows *const x[2],
         const gdn_packed *const x8[2], const gdn_rows *const dy[2], size_t dye,
         const gdn_rows *const out[2], const gdn_packed *const out8[2]) {
  const size_t e = p->dtype == GDN_BF16 ? 2 : 4;
  A.pos = p->positions;
  A.inv_freq = p->inv_freq;
  A.T = p->T; A.d = p->d; A.rot = p->rot; A.norm = p->norm;
  A.eps = p->eps; A.w0 = p->weight_offset; A.rope_scale = p->rope_scale;
  A.lg = p->d <= 64 ? 3 : p->d <= 128 ? 4 : 5;
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
      if (!rows_ok(x[i], P.H, p->d, e)) return GDN_ERR_INVALID_ARG;
      P.x = x[i]->data; P.x_ts = x[i]->token_stride; P.x_hs = x[i]->head_stride;
    }
    if (dy) {
      if (!rows_ok(dy[i], P.H, p->d, dye)) return GDN_ERR_INVALID_ARG;
      P.dy = dy[i]->data; P.dy_ts = dy[i]->token_stride; P.dy_hs = dy[i]->head_stride;
    }
    if (out8 && out8[i] && out8[i]->codes) {
      if (!out8[i]->scales) return GDN_ERR_INVALID_ARG;
      P.codes = out8[i]->codes;
      P.scales = out8[i]->scales;
    }
    if (out[i] && out[i]->data) {
      if (!rows_ok(out[i], P.H, p->d, e)) return GDN_ERR_INVALID_ARG;
      P.out = out[i]->data; P.out_ts = out[i]->token_stride; P.out_hs = out[i]->head_stride;
    } else if (!P.codes) {
      return GDN_ERR_INVALID_ARG;
    }
  }
  // Heads per item: enough items for every warp of the device where there are
  // tokens enough, else one step of a warp.
  A.rpi = 16;
  for (Part &P : A.p) P.splits = (P.H + A.rpi - 1) / A.rpi;
  return GDN_OK;
}

int64_t total_items(const QkArgs &A) {
  int64_t most = 0;
  for (const Part &P : A.p) most = most < int64_t(A.T) * P.splits ? int64_t(A.T) * P.splits : most;
  return most;
}

template <bool PACKED>
int run_fwd(const gdn_qk_params *p, const gdn_rows *const x[2], const gdn_packed *const x8[2],
            const gdn_rows *const out[2], const gdn_packed *const out8[2], void *stream) {
  int rc = check_params(p);
  if (rc != GDN_OK) return rc;
  QkArgs A{};
  rc = fill(A, p, x, PACKED ? x8 : nullptr, nullptr, 0, out, out8);
  if (rc != GDN_OK) return rc;
  if (total_items(A) == 0) return GDN_OK;
  const unsigned grid = grid_for(total_items(A), device_sms(), kFwdBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, 2, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = fwd_launch<PACKED>(A, p->dtype, pair_mode(p), acc, grid, s);
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
  const unsigned grid = grid_for(total_items(A), device_sms(), kBwdBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, grad_dtype == GDN_BF16 ? 2 : 4, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (total_items(A) > 0 || dw_q || dw_k) {
    const cudaError_t e = bwd_launch<PACKED>(A, p->dtype, grad_dtype, pair_mode(p), acc, grid, s);
    if (e != cudaSuccess) return GDN_ERR_CUDA;
  }
  if (dw_q || dw_k) {
    gdn_qk_dw_kernel<<<dim3((p->d + 31) / 32, 2), 1024, 0, s>>>(A.dw_part, int(grid), p->d, dw_q, dw_k);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  return GDN_OK;
}

}  // namespace
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
  return align_up(size_t(2) * device_sms() * kBwdBlocksPerSm * p->d * sizeof(float), 256);
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
