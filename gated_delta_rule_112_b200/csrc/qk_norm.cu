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
// A group of G lanes (8, 16 or 32: from d / 8 up) holds a row, eight elements
// a lane in two chunks of four, so the sums are log2 G shuffles. For pairs of
// halves the chunks lie rot / 2 apart (rot a multiple of 8), otherwise side by
// side: a pair's two elements are in one lane either way and nothing is
// exchanged. Only halves that do not fall into chunks of four (odd rot, rows
// off their alignment) meet in the warp's own shared memory. With
// y = r (x C + x' S), x' the partner's element, C and S hold cosine, sine,
// weight and scale, formed once for all heads of q and of k of a token, and the
// row's arithmetic is 12 paired instructions for 8 elements.
//
// A warp takes an item: rows of one token, q's heads and then k's. It forms the
// item's cosines and sines once: the angle in turns is position * inv_freq /
// 2 pi in fp64, less its whole turns, so far positions lose nothing; fp32 sine
// and cosine of the remainder follow.
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

// How the pairs lie. Split: halves in chunks of four; shared: any halves.
enum { kPairNone, kPairInterleaved, kPairSplit, kPairShared };

struct Part {                     // q or k
  const void *x;                  // rows (dtype), or e4m3 codes
  const uint8_t *x_scales;        // set when x holds codes
  const void *dy;
  void *out;                      // y or dx; may be null when only codes are wanted
  uint8_t *codes, *scales;        // checkpoint to write, or null
  const void *w;
  int64_t x_ts, x_hs, dy_ts, dy_hs, out_ts, out_hs;
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
};

// A lane's place in a row: chunks of four elements at a and b, of which na and
// nb exist.
struct Lane { int a, b, na, nb; };
template <int PAIR>
__device__ __forceinline__ Lane lane_place(const QkArgs &A, int l) {
  Lane L;
  const bool split = PAIR == kPairSplit && 8 * l < A.rot;
  L.a = split ? 4 * l : 8 * l;
  L.b = split ? A.rot / 2 + 4 * l : 8 * l + 4;
  L.na = max(0, min(4, A.d - L.a));
  L.nb = max(0, min(4, A.d - L.b));
  return L;
}

// Eight elements as they lie in memory.
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> { uint32_t w[4]; };
template <>
struct Raw<float> { float w[8]; };
struct Codes { uint32_t w[2]; uint32_t ea, eb; };

// ACC: elements an access may take; all pointers and strides are multiples of it.
template <int ACC>
__device__ __forceinline__ void load_chunk(const __nv_bfloat16 *p, int n, uint32_t *w) {
  w[0] = w[1] = 0;
  if (ACC >= 4) {
    if (n > 0) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p));
      w[0] = v.x; w[1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) w[i / 2] |= uint32_t(*reinterpret_cast<const uint16_t *>(p + i)) << (16 * (i & 1));
  }
}
template <int ACC>
__device__ __forceinline__ void load_chunk(const float *p, int n, float *w) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (ACC >= 4) {
    if (n > 0) v = __ldcs(reinterpret_cast<const float4 *>(p));
  } else {
    if (n > 0) v.x = p[0];
    if (n > 1) v.y = p[1];
    if (n > 2) v.z = p[2];
    if (n > 3) v.w = p[3];
  }
  w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
}
template <int PAIR, int ACC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *p, const Lane &L, bool on, Raw<__nv_bfloat16> &r) {
  if (ACC == 8 && PAIR != kPairSplit) {
    r.w[0] = r.w[1] = r.w[2] = r.w[3] = 0;
    if (on && L.na > 0) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p + L.a));
      r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
  } else {
    load_chunk<ACC>(p + L.a, on ? L.na : 0, r.w);
    load_chunk<ACC>(p + L.b, on ? L.nb : 0, r.w + 2);
  }
}
template <int PAIR, int ACC>
__device__ __forceinline__ void load8(const float *p, const Lane &L, bool on, Raw<float> &r) {
  load_chunk<ACC>(p + L.a, on ? L.na : 0, r.w);
  load_chunk<ACC>(p + L.b, on ? L.nb : 0, r.w + 4);
}
template <int ACC>
__device__ __forceinline__ uint32_t load_codes(const uint8_t *p, int n) {
  uint32_t w = 0;
  if (ACC >= 4) {
    if (n > 0) w = __ldcs(reinterpret_cast<const uint32_t *>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) w |= uint32_t(p[i]) << (8 * i);
  }
  return w;
}

// The lane's elements as four pairs: chunk a, then chunk b.
struct Row { Pair v[4]; };

__device__ __forceinline__ void unpack8(const Raw<__nv_bfloat16> &r, Row &x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = pair(bf_lo(r.w[i]), bf_hi(r.w[i]));
}
__device__ __forceinline__ void unpack8(const Raw<float> &r, Row &x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x.v[i] = pair(r.w[2 * i], r.w[2 * i + 1]);
}
// 2^(b - 127), b in [0, 254]: 2^-127 lies below the normal range.
__device__ __forceinline__ float pow2_biased(uint32_t b) {
  return __uint_as_float(b ? b << 23 : 0x00400000u);
}
__device__ __forceinline__ void unpack8(const Codes &r, Row &x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float s = pow2_biased(i < 2 ? r.ea : r.eb);
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(
        static_cast<__nv_fp8x2_storage_t>((r.w[i / 2] >> (16 * (i & 1))) & 0xffff), __NV_E4M3);
    const float2 f = __half22float2(__half2(h));
    x.v[i] = mul2(pair(f.x, f.y), pair(s, s));
  }
}

template <int ACC>
__device__ __forceinline__ void store_chunk(__nv_bfloat16 *p, int n, Pair lo, Pair hi) {
  const float2 f = unpair(lo), g = unpair(hi);
  const uint32_t w[2] = {bf_pack(f.x, f.y), bf_pack(g.x, g.y)};
  if (ACC >= 4) {
    if (n > 0) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) *reinterpret_cast<uint16_t *>(p + i) = uint16_t(w[i / 2] >> (16 * (i & 1)));
  }
}
template <int ACC>
__device__ __forceinline__ void store_chunk(float *p, int n, Pair lo, Pair hi) {
  const float2 f = unpair(lo), g = unpair(hi);
  if (ACC >= 4) {
    if (n > 0) *reinterpret_cast<float4 *>(p) = make_float4(f.x, f.y, g.x, g.y);
  } else {
    if (n > 0) p[0] = f.x;
    if (n > 1) p[1] = f.y;
    if (n > 2) p[2] = g.x;
    if (n > 3) p[3] = g.y;
  }
}
template <int PAIR, int ACC>
__device__ __forceinline__ void store8(__nv_bfloat16 *p, const Lane &L, const Row &y) {
  if (ACC == 8 && PAIR != kPairSplit) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(y.v[i]);
      w[i] = bf_pack(f.x, f.y);
    }
    if (L.na > 0) *reinterpret_cast<uint4 *>(p + L.a) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    store_chunk<ACC>(p + L.a, L.na, y.v[0], y.v[1]);
    store_chunk<ACC>(p + L.b, L.nb, y.v[2], y.v[3]);
  }
}
template <int PAIR, int ACC>
__device__ __forceinline__ void store8(float *p, const Lane &L, const Row &y) {
  store_chunk<ACC>(p + L.a, L.na, y.v[0], y.v[1]);
  store_chunk<ACC>(p + L.b, L.nb, y.v[2], y.v[3]);
}
template <int ACC>
__device__ __forceinline__ void store_codes(uint8_t *p, int n, uint32_t w) {
  if (ACC >= 4) {
    if (n > 0) *reinterpret_cast<uint32_t *>(p) = w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = uint8_t(w >> (8 * i));
  }
}

// Sum over the 2^lg lanes of a row.
__device__ __forceinline__ float group_sum(float x, int lg) {
  if (lg > 4) x += __shfl_xor_sync(0xffffffffu, x, 16);
  if (lg > 3) x += __shfl_xor_sync(0xffffffffu, x, 8);
#pragma unroll
  for (int off = 4; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}
__device__ __forceinline__ float dot8(const Row &x, const Row &y) {
  Pair s = mul2(x.v[0], y.v[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) s = fma2(x.v[i], y.v[i], s);
  const float2 f = unpair(s);
  return f.x + f.y;
}

// The lane's part of y = x C + x' S, x' the partner of every element. What does
// not turn takes no partner: it must not meet another element's infinity.
// row: this group's part of the warp's buffer.
template <int PAIR>
__device__ __forceinline__ void turn(const QkArgs &A, const Lane &L, float *row, const Row &C, const Row &S,
                                     Row &x) {
  Row y;
#pragma unroll
  for (int i = 0; i < 4; ++i) y.v[i] = mul2(x.v[i], C.v[i]);
  if (PAIR == kPairInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(x.v[i]);
      if (L.a + 2 * i < A.rot) y.v[i] = fma2(pair(f.y, f.x), S.v[i], y.v[i]);
    }
  } else if (PAIR == kPairSplit) {
    if (L.a < A.rot) {
#pragma unroll
      for (int i = 0; i < 4; ++i) y.v[i] = fma2(x.v[i ^ 2], S.v[i], y.v[i]);
    }
  } else if (PAIR == kPairShared) {
    const int half = A.rot / 2;
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<float2 *>(row + L.a + 2 * i) = unpair(x.v[i]);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
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
// 1 and 0 for the pairs that do not turn.
__device__ __forceinline__ void make_angles(const QkArgs &A, int t, int lane, float *cs) {
  const double p = double(A.pos[t]);
  __syncwarp();
  for (int j = lane; j < 4 << A.lg; j += 32) {
    float s = 0.f, c = 1.f;
    if (j < A.rot / 2) {
      double turns = p * A.inv_freq[j] * 0.15915494309189533577;   // 1 / (2 pi)
      turns -= rint(turns);
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
// Element i (0..7) of the lane: its place in the row.
__device__ __forceinline__ int element(const Lane &L, int i) { return i < 4 ? L.a + i : L.b + i - 4; }

// C and S for a turn by +angle (sign 1) or -angle, with the element's weight in
// C and its partner's in S. w: a weight for each element.
template <int PAIR>
__device__ __forceinline__ void factors(const QkArgs &A, const Lane &L, int l, const float *cs, const float *w,
                                        float sign, Row &C, Row &S) {
  const float4 wa = lds4(w + L.a), wb = lds4(w + L.b);
  if (PAIR == kPairNone) {
    C.v[0] = pair(wa.x, wa.y); C.v[1] = pair(wa.z, wa.w);
    C.v[2] = pair(wb.x, wb.y); C.v[3] = pair(wb.z, wb.w);
    return;
  }
  if (PAIR == kPairShared) {
    float c[8], s[8];
    const int half = A.rot / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = L.a + i, j = e < half ? e : e - half;
      const bool on = e < A.rot;
      c[i] = (on ? cs[j] : 1.f) * w[e];
      s[i] = on ? sign * cs[kMaxD / 2 + j] * (e < half ? -w[e + half] : w[e - half]) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      C.v[i] = pair(c[2 * i], c[2 * i + 1]);
      S.v[i] = pair(s[2 * i], s[2 * i + 1]);
    }
    return;
  }
  const float4 c = lds4(cs + 4 * l);
  float4 s = lds4(cs + kMaxD / 2 + 4 * l);
  s = make_float4(s.x * sign, s.y * sign, s.z * sign, s.w * sign);
  if (PAIR == kPairInterleaved) {
    C.v[0] = pair(c.x * wa.x, c.x * wa.y); S.v[0] = pair(-s.x * wa.y, s.x * wa.x);
    C.v[1] = pair(c.y * wa.z, c.y * wa.w); S.v[1] = pair(-s.y * wa.w, s.y * wa.z);
    C.v[2] = pair(c.z * wb.x, c.z * wb.y); S.v[2] = pair(-s.z * wb.y, s.z * wb.x);
    C.v[3] = pair(c.w * wb.z, c.w * wb.w); S.v[3] = pair(-s.w * wb.w, s.w * wb.z);
  } else {
    C.v[0] = pair(c.x * wa.x, c.y * wa.y); S.v[0] = pair(-s.x * wb.x, -s.y * wb.y);
    C.v[1] = pair(c.z * wa.z, c.w * wa.w); S.v[1] = pair(-s.z * wb.z, -s.w * wb.w);
    C.v[2] = pair(c.x * wb.x, c.y * wb.y); S.v[2] = pair(s.x * wa.x, s.y * wa.y);
    C.v[3] = pair(c.z * wb.z, c.w * wb.w); S.v[3] = pair(s.z * wa.z, s.w * wa.w);
  }
}

__device__ __forceinline__ float rnorm(const QkArgs &A, float ss) {
  return A.norm == GDN_NORM_NONE ? 1.f : rsqrtf(ss * A.inv_n + A.eps);
}

// (w + w0) * scale of q's and of k's elements, 1 * scale without weights.
template <typename T>
__device__ __forceinline__ void stage_weights(const QkArgs &A, bool scaled, bool weighted, float (*w)[kMaxD]) {
  for (int i = threadIdx.x; i < 2 * kMaxD; i += kQkThreads) {
    const Part &P = A.p[i / kMaxD];
    const int e = i % kMaxD;
    float x = 1.f;
    if (weighted && P.w && e < A.d) x = to_f32(static_cast<const T *>(P.w)[e]) + A.w0;
    w[i / kMaxD][e] = scaled ? x * P.scale : x;
  }
  __syncthreads();
}

// Source of the rows: T in memory, or codes. The pointers are those of the
// lane's first row and step from row to row.
template <typename T, bool PACKED, int PAIR, int ACC>
struct Source {
  using Data = Raw<T>;
  const T *p;
  int64_t step;
  __device__ __forceinline__ Source(const QkArgs &, const Part &P, int64_t t, int h, int rows) {
    p = static_cast<const T *>(P.x) + t * P.x_ts + h * P.x_hs;
    step = rows * P.x_hs;
  }
  __device__ __forceinline__ void load(const Lane &L, bool on, Data &r) {
    load8<PAIR, ACC>(p, L, on, r);
    p += step;
  }
};
template <typename T, int PAIR, int ACC>
struct Source<T, true, PAIR, ACC> {
  using Data = Codes;
  const uint8_t *p, *e;
  int step, estep;
  __device__ __forceinline__ Source(const QkArgs &A, const Part &P, int64_t t, int h, int rows) {
    const int64_t row = t * P.H + h;
    const int blocks = (A.d + 31) / 32;
    p = static_cast<const uint8_t *>(P.x) + row * A.d;
    e = P.x_scales + row * blocks;
    step = rows * A.d;
    estep = rows * blocks;
  }
  __device__ __forceinline__ void load(const Lane &L, bool on, Data &r) {
    if (ACC == 8 && PAIR != kPairSplit) {
      r.w[0] = r.w[1] = 0;
      r.ea = 127;
      if (on && L.na > 0) {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(p + L.a));
        r.w[0] = v.x; r.w[1] = v.y;
        r.ea = e[L.a / 32];
      }
      r.eb = r.ea;
    } else {
      r.w[0] = load_codes<ACC>(p + L.a, on ? L.na : 0);
      r.w[1] = load_codes<ACC>(p + L.b, on ? L.nb : 0);
      r.ea = on && L.na > 0 ? e[L.a / 32] : 127;
      r.eb = on && L.nb > 0 ? e[L.b / 32] : 127;
    }
    p += step;
    e += estep;
  }
};

// The biased exponent that a block's largest finite magnitude (its bits) asks
// for. 448 = 1.75 * 2^8: its exponent - 8, one more where the significand is
// above 1.75, and not below 2^-127.
__device__ __forceinline__ int block_exponent(uint32_t bits) {
  return max(int((bits + 0x1fffffu) >> 23) - 8, 0);
}
__device__ __forceinline__ uint32_t encode4(Pair lo, Pair hi, int be) {
  const float inv = __uint_as_float(uint32_t(254 - be) << 23);     // 2^-(be - 127)
  const float2 a = unpair(mul2(lo, pair(inv, inv))), b = unpair(mul2(hi, pair(inv, inv)));
  return __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3) |
         uint32_t(__nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3)) << 16;
}

// Largest magnitude of each chunk, as the upper 16 (bf16) or all (fp32) bits of
// an fp32: of non-negative floats the bits compare alike, with infinities and
// NaN above the rest. Two chunks' 16 bits share a word.
struct Top { uint32_t a, b; };
__device__ __forceinline__ Top chunk_tops(const Raw<__nv_bfloat16> &r) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(r.w[0] & m, r.w[1] & m), b = __vmaxu2(r.w[2] & m, r.w[3] & m);
  const uint32_t t = __vmaxu2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
  return {t << 16, t & 0xffff0000u};
}
__device__ __forceinline__ Top chunk_tops(const Raw<float> &r) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(r.w[i]) & 0x7fffffffu;
  return {max(max(u[0], u[1]), max(u[2], u[3])), max(max(u[4], u[5]), max(u[6], u[7]))};
}

// Writes the lane's eight elements in 8 bits. Side by side, four lanes hold a
// block; with halves in chunks eight lanes' first chunks do, and their second
// chunks, where rot / 2 is a multiple of 32; for other rot the blocks' maxima
// meet in shared memory.
template <typename T, int PAIR, int ACC>
__device__ __forceinline__ void write_codes(const QkArgs &A, const Part &P, int64_t row, const Lane &L,
                                            bool on, uint32_t *tops, const Raw<T> &raw, const Row &x) {
  constexpr uint32_t kInf = 0x7f800000u;
  Top t = chunk_tops(raw);
  Row z = x;
  if (__any_sync(0xffffffffu, max(t.a, t.b) >= kInf)) {
    // what is not finite counts for nothing, and becomes NaN
    uint32_t u[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 f = unpair(x.v[i]);
      const uint32_t fx = __float_as_uint(f.x) & 0x7fffffffu, fy = __float_as_uint(f.y) & 0x7fffffffu;
      if (fx < kInf) u[i / 2] = max(u[i / 2], fx);
      else f.x = __int_as_float(0x7fffffff);
      if (fy < kInf) u[i / 2] = max(u[i / 2], fy);
      else f.y = __int_as_float(0x7fffffff);
      z.v[i] = pair(f.x, f.y);
    }
    t = {u[0], u[1]};
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
      w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, 1));
      w = __vmaxu2(w, __shfl_xor_sync(0xffffffffu, w, 2));
      const uint32_t o = __shfl_xor_sync(0xffffffffu, w, 4);
      if (split) w = __vmaxu2(w, o);
      t = {w << 16, w & 0xffff0000u};
    } else {
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) {
        const uint32_t oa = __shfl_xor_sync(0xffffffffu, t.a, off);
        if (off < 4 || split) t.a = max(t.a, oa);
        if (PAIR == kPairSplit) {
          const uint32_t ob = __shfl_xor_sync(0xffffffffu, t.b, off);
          if (off < 4 || split) t.b = max(t.b, ob);
        }
      }
    }
  }
  const int ea = block_exponent(t.a), eb = PAIR == kPairSplit ? block_exponent(t.b) : ea;
  const uint32_t ca = encode4(z.v[0], z.v[1], ea), cb = encode4(z.v[2], z.v[3], eb);
  if (!on) return;
  uint8_t *p = P.codes + row * A.d, *e = P.scales + row * ((A.d + 31) / 32);
  if (ACC == 8 && PAIR != kPairSplit) {
    if (L.na > 0) *reinterpret_cast<uint2 *>(p + L.a) = make_uint2(ca, cb);
  } else {
    store_codes<ACC>(p + L.a, L.na, ca);
    store_codes<ACC>(p + L.b, L.nb, cb);
  }
  if ((L.a & 31) == 0 && L.na > 0) e[L.a / 32] = uint8_t(ea);
  if (PAIR == kPairSplit && (L.b & 31) == 0 && L.nb > 0) e[L.b / 32] = uint8_t(eb);
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
template <typename T, bool PACKED, bool PACK, int PAIR, int ACC>
__global__ void __launch_bounds__(kQkThreads, 3) gdn_qk_fwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int U = 4;
  __shared__ __align__(16) float w_all[2][kMaxD];
  __shared__ __align__(16) float cs_all[PAIR == kPairNone ? 1 : kQkWarps][kMaxD];
  __shared__ __align__(16) float rows_all[PAIR == kPairShared ? kQkWarps : 1][kMaxD];
  __shared__ uint32_t tops_all[PACK && PAIR == kPairSplit ? kQkWarps * 32 : 1];
  const int G = 1 << A.lg, R = 32 >> A.lg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> A.lg, l = lane & (G - 1);
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[PAIR == kPairShared ? warp : 0] + (lane & -G) * 8;
  uint32_t *tops = tops_all + (PACK && PAIR == kPairSplit ? warp * 32 + sub * 8 : 0);
  const Lane L = lane_place<PAIR>(A, l);
  stage_weights<T>(A, true, true, w_all);
  const int64_t nwarps = int64_t(gridDim.x) * kQkWarps, items = int64_t(A.T) * A.splits;
  for (int64_t item = int64_t(blockIdx.x) * kQkWarps + warp; item < items; item += nwarps) {
    const Item I = item_at(A, item);
    if (PAIR != kPairNone) make_angles(A, I.t, lane, cs);
    for (int part = 0; part < 2; ++part) {
      const Part &P = A.p[part];
      const int first = part ? A.p[0].H : 0;
      const int h0 = max(I.r0 - first, 0), h1 = min(I.r1 - first, P.H);
      if (h0 >= h1) continue;
      Row C, S;
      factors<PAIR>(A, L, l, cs, w_all[part], 1.f, C, S);
      using Src = Source<T, PACKED, PAIR, ACC>;
      Src src(A, P, I.t, h0 + sub, R);
      T *out = static_cast<T *>(P.out) + I.t * P.out_ts + (h0 + sub) * P.out_hs;
      const int64_t out_step = R * P.out_hs;
      for (int h = h0 + sub; h - sub < h1; h += R * U) {
        typename Src::Data raw[U];
#pragma unroll
        for (int u = 0; u < U; ++u) src.load(L, h + u * R < h1, raw[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h - sub + u * R >= h1) break;
          const bool on = h + u * R < h1;
          Row x;
          unpack8(raw[u], x);
          if constexpr (PACK)
            if (P.codes)
              write_codes<T, PAIR, ACC>(A, P, int64_t(I.t) * P.H + h + u * R, L, on, tops, raw[u], x);
          if (A.norm != GDN_NORM_NONE) {
            const float r = rnorm(A, group_sum(dot8(x, x), A.lg));
#pragma unroll
            for (int i = 0; i < 4; ++i) x.v[i] = mul2(x.v[i], pair(r, r));
          }
          turn<PAIR>(A, L, row_buf, C, S, x);
          if (on && (!PACK || P.out)) store8<PAIR, ACC>(out, L, x);
          out += out_step;
        }
      }
    }
  }
}

// WEIGHTS: weights and their gradients.
template <typename T, typename DT, bool PACKED, bool WEIGHTS, int PAIR, int ACC>
__global__ void __launch_bounds__(kQkThreads, 2) gdn_qk_bwd_kernel(const __grid_constant__ QkArgs A) {
  constexpr int U = 2;
  __shared__ __align__(16) float w_all[2][kMaxD], one[2][kMaxD];
  __shared__ __align__(16) float cs_all[PAIR == kPairNone ? 1 : kQkWarps][kMaxD];
  __shared__ __align__(16) float rows_all[PAIR == kPairShared || WEIGHTS ? kQkWarps : 1][kMaxD];
  const int G = 1 << A.lg, R = 32 >> A.lg;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane >> A.lg, l = lane & (G - 1);
  float *cs = cs_all[PAIR == kPairNone ? 0 : warp];
  float *row_buf = rows_all[PAIR == kPairShared || WEIGHTS ? warp : 0] + (lane & -G) * 8;
  const Lane L = lane_place<PAIR>(A, l);
  if (WEIGHTS) stage_weights<T>(A, false, true, w_all);
  stage_weights<T>(A, true, false, one);
  const int64_t nwarps = int64_t(gridDim.x) * kQkWarps, items = int64_t(A.T) * A.splits;
  Row dw[2];
#pragma unroll
  for (int i = 0; i < 8; ++i) dw[i / 4].v[i % 4] = pair(0.f, 0.f);
  for (int64_t item = int64_t(blockIdx.x) * kQkWarps + warp; item < items; item += nwarps) {
    const Item I = item_at(A, item);
    if (PAIR != kPairNone) make_angles(A, I.t, lane, cs);
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      const Part &P = A.p[part];
      const int first = part ? A.p[0].H : 0;
      const int h0 = max(I.r0 - first, 0), h1 = min(I.r1 - first, P.H);
      if (h0 >= h1) continue;
      Row C, S, W;
      factors<PAIR>(A, L, l, cs, one[part], -1.f, C, S);
      if (WEIGHTS) {
        const float4 wa = lds4(w_all[part] + L.a), wb = lds4(w_all[part] + L.b);
        W.v[0] = pair(wa.x, wa.y); W.v[1] = pair(wa.z, wa.w);
        W.v[2] = pair(wb.x, wb.y); W.v[3] = pair(wb.z, wb.w);
      }
      using Src = Source<T, PACKED, PAIR, ACC>;
      Src src(A, P, I.t, h0 + sub, R);
      const DT *dy = static_cast<const DT *>(P.dy) + I.t * P.dy_ts + (h0 + sub) * P.dy_hs;
      T *out = static_cast<T *>(P.out) + I.t * P.out_ts + (h0 + sub) * P.out_hs;
      const int64_t dy_step = R * P.dy_hs, out_step = R * P.out_hs;
      for (int h = h0 + sub; h - sub < h1; h += R * U) {
        typename Src::Data raw[U];
        Raw<DT> grad[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          src.load(L, h + u * R < h1, raw[u]);
          load8<PAIR, ACC>(dy, L, h + u * R < h1, grad[u]);
          dy += dy_step;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (h - sub + u * R >= h1) break;
          Row x, z;
          unpack8(raw[u], x);
          unpack8(grad[u], z);
          turn<PAIR>(A, L, row_buf, C, S, z);
          float r = 1.f, m = 0.f;
          Row dh = z;
          if (WEIGHTS) {
#pragma unroll
            for (int i = 0; i < 4; ++i) dh.v[i] = mul2(z.v[i], W.v[i]);
          }
          if (A.norm != GDN_NORM_NONE) {
            r = rnorm(A, group_sum(dot8(x, x), A.lg));
            m = group_sum(dot8(x, dh), A.lg) * r * A.inv_n;
          }
          const Pair rr = pair(r, r), mm = pair(-m, -m);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const Pair hx = mul2(x.v[i], rr);
            if (WEIGHTS) dw[part].v[i] = fma2(z.v[i], hx, dw[part].v[i]);
            x.v[i] = A.norm == GDN_NORM_NONE ? dh.v[i] : mul2(fma2(hx, mm, dh.v[i]), rr);
          }
          if (h + u * R < h1) store8<PAIR, ACC>(out, L, x);
          out += out_step;
        }
      }
    }
  }
  if (WEIGHTS) {    // the block's rows in a fixed order: warps 0..7, and in each its groups
#pragma unroll
    for (int part = 0; part < 2; ++part) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 f = unpair(dw[part].v[i / 2]);
        const int e = element(L, i);
        if (e < G * 8) row_buf[e] = i & 1 ? f.y : f.x;
      }
      __syncthreads();
      for (int e = threadIdx.x; e < A.d; e += kQkThreads) {
        float s = 0.f;
        for (int i = 0; i < kQkWarps * R; ++i) s += rows_all[i / R][(i % R) * G * 8 + e];
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

// The way the pairs are handled: halves go in chunks where they fall into them.
int pair_mode(const gdn_qk_params *p, int acc) {
  if (!p->rot) return kPairNone;
  if (p->interleaved) return kPairInterleaved;
  return acc >= 4 && p->rot % 8 == 0 ? kPairSplit : kPairShared;
}

constexpr int kFwdBlocksPerSm = 3, kBwdBlocksPerSm = 2;

// Rows an item and items a token: whole tokens, whose cosines then serve every
// head, where there are enough of them for all warps; else fewer rows, down to
// one step of a warp.
unsigned plan(QkArgs &A, int per_sm) {
  const int rows = A.p[0].H + A.p[1].H, step = 32 >> A.lg, sms = device_sms();
  const int64_t warps = int64_t(sms > 0 ? sms : 1) * per_sm * kQkWarps;
  int64_t want = (int64_t(A.T) * rows + warps - 1) / warps;          // rows a warp
  want = (want + step - 1) / step * step;
  A.rpi = int(want < 1 ? 1 : want < rows ? want : rows > 0 ? rows : 1);
  A.splits = (rows + A.rpi - 1) / A.rpi;
  const int64_t blocks = (int64_t(A.T) * A.splits + kQkWarps - 1) / kQkWarps;
  const int64_t most = int64_t(sms > 0 ? sms : 1) * per_sm;
  return unsigned(blocks < 1 ? 1 : blocks < most ? blocks : most);
}

// Turns the run-time choices into template arguments: a variant for each way
// the pairs lie, at the widest access (16 bytes of T where eight elements lie
// side by side) and narrower ones.
template <int V> struct Const { static constexpr int value = V; };
template <typename T, typename F>
void with_variant(int pair, int acc, F f) {
  auto pick = [&](auto a) {
    if (pair == kPairNone) f(Const<kPairNone>{}, a);
    else if (pair == kPairInterleaved) f(Const<kPairInterleaved>{}, a);
    else f(Const<kPairShared>{}, a);
  };
  if (pair == kPairSplit) f(Const<kPairSplit>{}, Const<4>{});
  else if (acc == 8 && sizeof(T) == 2) pick(Const<8>{});
  else if (acc >= 4) pick(Const<4>{});
  else pick(Const<1>{});
}

template <bool PACKED, bool PACK>
cudaError_t fwd_launch(const QkArgs &A, int dtype, int pair, int acc, unsigned grid, cudaStream_t s) {
  auto go = [&](auto type) {
    using T = decltype(type);
    with_variant<T>(pair, acc, [&](auto p, auto a) {
      gdn_qk_fwd_kernel<T, PACKED, PACK, decltype(p)::value, decltype(a)::value>
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
    with_variant<T>(pair, acc, [&](auto p, auto a) {
      gdn_qk_bwd_kernel<T, DT, PACKED, WEIGHTS, decltype(p)::value, decltype(a)::value>
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
  const unsigned grid = plan(A, kFwdBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, 2, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pair = pair_mode(p, acc);
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
  const unsigned grid = plan(A, kBwdBlocksPerSm);
  const int acc = access_width(A, p->dtype == GDN_BF16 ? 2 : 4, grad_dtype == GDN_BF16 ? 2 : 4, PACKED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!A.p[0].H && !A.p[1].H && !dw_q && !dw_k) return GDN_OK;
  const int pair = pair_mode(p, acc);
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
