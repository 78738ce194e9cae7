// The recurrent gated delta rule for serving: runs of new tokens of many
// sequences against a pool of states addressed by slot (gdn_recurrent_fwd).
//
// Run n covers tokens [t0, t1) and the state in slot slots[n]. Per value head
// (key head hk = h / (H_v / H_k)), with the state held transposed
// (st[j][i] = S_ij) and a_j = exp(g) (one value, or one per d_k channel j):
//   x_i = sum_j st[j][i] a_j k_j,  u_i = beta (v_i - x_i)
//   st[j][i] <- a_j st[j][i] + u_i k_j,  o_i = sum_j st[j][i] q_j
//
// Two tokens are taken together, so that a pass over the state serves both and
// the chain from token to token runs over a few scalars. With S the state
// before the two, c_m = a_0 .. a_m:
//   X_m = S^T k_m,  Y_m = S^T q_m                    (one pass, one reduction)
//   u_0 = beta_0 (v_0 - c_0 X_0),  u_1 = beta_1 (v_1 - c_1 X_1 - a_1 (k_0 . k_1) u_0)
//   o_0 = c_0 Y_0 + (k_0 . q_0) u_0,  o_1 = c_1 Y_1 + a_1 (k_0 . q_1) u_0 + (k_1 . q_1) u_1
//   S  <- c_1 S + a_1 u_0 k_0 + u_1 k_1              (one pass)
// With the channel gate the products of decays sit inside the dot products and
// in rows of k and q scaled by them. All of them are products of the tokens'
// own decays, never quotients, so a decay of zero is as good as any other.
//
// A warp owns 16 columns i and all rows j of one state; columns of st evolve
// independently, so warps exchange nothing of the state. Lane (rg, cg) =
// (lane / 4, lane % 4) holds columns 4 cg .. 4 cg + 3 of rows 32 p + 4 rg + r
// (r < 4, p < d_k / 32) in registers for the whole run: HBM sees one read and
// one write of the state however many tokens the run has. The partial sums are
// reduced over the eight rg lanes by halving (7 shuffles a token), after which
// one lane holds a column's X of every token and its neighbour the Y.
//
// (Four together take no fewer multiply-adds a token and half as many steps,
// but 64 more registers and twice the code: 63 us against 47 us for 64 runs of
// one to six tokens of 32 heads.)
//
// k, q, v and the decays of up to four tokens at a time come through shared
// memory in fp32, a token a warp: the rows of the group after next are on their
// way from HBM, those of the next are multiplied with each other, while this
// one is computed. k and q lie there twice over, k_j k_j, so that one 16-byte
// read gives the operands of paired multiply-adds for two rows.
#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kRecWarps = 4, kRecCols = 16 * kRecWarps;   // columns of d_v per CTA
constexpr int kGroup = 4;                                 // tokens staged together

struct RecArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  void *pool;
  const int32_t *slots, *cu, *keep;
  const uint8_t *reset;
  void *o;
  uint32_t *status;
  int64_t q_stride, k_stride, v_stride, num_slots;
  int N, T, L, Hk, Hv, dk, dv;      // L: tokens per run without cu
  int splits;                       // CTAs per state
  bool vec;                         // q, k, v rows can be read four elements at a time
};

// A group's tokens as they came, in fp32. Tokens past the group's end are zero
// with decay 1.
template <bool KDA>
struct alignas(16) RecRows {
  float k[kGroup][128], q[kGroup][128];
  float a[kGroup][KDA ? 128 : 4];
  float beta[kGroup];
};
// What the passes over the state take: rows twice over, and for each pair of
// tokens m = 0, 1 the scalars.
template <bool KDA>
struct alignas(16) RecCoef {
  float2 kx[kGroup][128], qx[kGroup][128];   // k and q (channel gate: c_m k_m, c_m q_m)
  float2 ku[KDA ? kGroup : 1][128];          // channel gate: the second of the two's decay times k_m
  float2 cu[KDA ? kGroup / 2 : 1][128];      // channel gate: c of the two, per row
  float4 s[kGroup];                          // c_m, beta_m, then d k_0 . k_1 and k_m . q_m
  float dq[kGroup], e[kGroup];               // d k_0 . q_1 (second tokens); decay after m in the two
};
template <bool KDA>
struct alignas(16) RecShared {
  RecRows<KDA> rows[2];              // of the next group; being fetched for the one after
  RecCoef<KDA> coef[2];              // of this group and of the next
  float v[3][kGroup][kRecCols];      // of all three
  float u[kRecWarps][2][16];
};
static_assert(sizeof(RecRows<false>) % 16 == 0 && sizeof(RecRows<true>) % 16 == 0 &&
              sizeof(RecCoef<false>) % 16 == 0 && sizeof(RecCoef<true>) % 16 == 0 &&
              offsetof(RecCoef<false>, s) % 16 == 0 && offsetof(RecRows<false>, a) % 16 == 0,
              "rows are read in 16-byte pieces");

template <typename T>
__device__ __forceinline__ float4 load4(const T *p, int n, bool vec) {
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (vec) {
    if (n > 0) r = ld4(p);
  } else {
    if (n > 0) r.x = to_f32(p[0]);
    if (n > 1) r.y = to_f32(p[1]);
    if (n > 2) r.z = to_f32(p[2]);
    if (n > 3) r.w = to_f32(p[3]);
  }
  return r;
}

__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ float4 lds4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ void sts4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }

__device__ __forceinline__ void copy_async(void *to, const void *from, int bytes) {
  const uint32_t p = uint32_t(__cvta_generic_to_shared(to));
  if (bytes == 16) asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(p), "l"(from) : "memory");
  else if (bytes == 8) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(p), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(p), "l"(from) : "memory");
}

// Starts the copy of token t's rows, as they are, to where land() turns them
// into fp32 in place; rows that cannot be copied in pieces are read here.
template <typename T, bool KDA>
__device__ __forceinline__ void fetch(const RecArgs &A, int64_t t, int h, int hk, int col0, int lane,
                                      RecRows<KDA> &R, float (*v)[kRecCols], int m) {
  const int c = lane * 4;
  const T *kp = static_cast<const T *>(A.k) + t * A.k_stride + int64_t(hk) * A.dk + c;
  const T *qp = static_cast<const T *>(A.q) + t * A.q_stride + int64_t(hk) * A.dk + c;
  const T *vp = static_cast<const T *>(A.v) + t * A.v_stride + int64_t(h) * A.dv + col0 + c;
  const float *gp = A.g + (t * A.Hv + h) * (KDA ? A.dk : 1);
  if (A.vec) {
    if (c < A.dk) {
      copy_async(reinterpret_cast<T *>(R.k[m]) + c, kp, 4 * sizeof(T));
      copy_async(reinterpret_cast<T *>(R.q[m]) + c, qp, 4 * sizeof(T));
      if (KDA) copy_async(&R.a[m][c], gp + c, 16);
    }
    if (c < kRecCols && col0 + c < A.dv) copy_async(reinterpret_cast<T *>(v[m]) + c, vp, 4 * sizeof(T));
  } else {
    sts4(&R.k[m][c], load4(kp, A.dk - c, false));
    sts4(&R.q[m][c], load4(qp, A.dk - c, false));
    if (KDA) sts4(&R.a[m][c], load4(gp + c, A.dk - c, false));
    if (c < kRecCols) sts4(&v[m][c], load4(vp, A.dv - col0 - c, false));
  }
  if (lane == 0) {
    if (!KDA) copy_async(&R.a[m][0], gp, 4);
    copy_async(&R.beta[m], A.beta + t * A.Hv + h, 4);
  }
}

template <typename T>
__device__ __forceinline__ float4 landed(const float *row, int lane, bool there, bool raw) {
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  if (!there) return zero;
  return raw ? ld4(reinterpret_cast<const T *>(row) + 4 * lane) : lds4(row + 4 * lane);
}
template <typename T, bool KDA>
__device__ __forceinline__ void land(const RecArgs &A, bool on, int col0, int lane, RecRows<KDA> &R,
                                     float (*v)[kRecCols], int m) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  const int c = lane * 4;
  const bool vc = c < kRecCols && col0 + c < A.dv;
  const float4 k4 = landed<T>(R.k[m], lane, on && c < A.dk, A.vec);
  const float4 q4 = landed<T>(R.q[m], lane, on && c < A.dk, A.vec);
  const float4 v4 = landed<T>(v[m], lane, on && vc, A.vec);
  float4 a4 = make_float4(1.f, 1.f, 1.f, 1.f);
  if (KDA && on && c < A.dk) {
    const float4 g = lds4(&R.a[m][c]);
    a4.x = expf(g.x);
    if (c + 1 < A.dk) a4.y = expf(g.y);
    if (c + 2 < A.dk) a4.z = expf(g.z);
    if (c + 3 < A.dk) a4.w = expf(g.w);
  }
  __syncwarp();                       // everything is read before anything is overwritten
  sts4(&R.k[m][c], k4);
  sts4(&R.q[m][c], q4);
  if (c < kRecCols) sts4(&v[m][c], v4);
  if (KDA) sts4(&R.a[m][c], a4);
  if (lane == 0) {
    if (!KDA) R.a[m][0] = on ? expf(R.a[m][0]) : 1.f;
    if (!on) R.beta[m] = 0.f;
  }
}

__device__ __forceinline__ void put_twice(float2 *p, float4 x) {
  *reinterpret_cast<float4 *>(p) = make_float4(x.x, x.x, x.y, x.y);
  *reinterpret_cast<float4 *>(p + 2) = make_float4(x.z, x.z, x.w, x.w);
}

// Warp m works out what token m has to do with the one before it. nb: tokens of
// the group.
template <bool KDA>
__device__ __forceinline__ void relate(const RecRows<KDA> &R, RecCoef<KDA> &C, int m, int nb, int lane) {
  const int c = lane * 4, f = m & ~1;                 // f: the first of the two
  if (f >= nb) return;
  const bool second = m & 1;
  const float4 km = lds4(&R.k[m][c]), qm = lds4(&R.q[m][c]), kf = lds4(&R.k[f][c]);
  float4 kd = km, qd = qm;                            // with the decay since the first
  float am = 1.f, a0 = 1.f, a1 = 1.f;
  if (KDA) {
    const float4 a = lds4(&R.a[m][c]);
    float4 x = a;                                     // c_m
    if (second) {
      kd = mul4(km, a);
      qd = mul4(qm, a);
      x = mul4(a, lds4(&R.a[f][c]));
    }
    put_twice(&C.kx[m][c], mul4(km, x));
    put_twice(&C.qx[m][c], mul4(qm, x));
    put_twice(&C.ku[m][c], second ? km : mul4(km, lds4(&R.a[f + 1][c])));
    if (second) put_twice(&C.cu[f / 2][c], x);
  } else {
    put_twice(&C.kx[m][c], km);
    put_twice(&C.qx[m][c], qm);
    a0 = R.a[f][0];
    a1 = R.a[f + 1][0];
    am = a1;
  }
  const float kk = warp_sum(second ? dot4(kf, kd) : 0.f), kq = warp_sum(dot4(km, qm));
  const float dq = warp_sum(second ? dot4(kf, qd) : 0.f);
  if (lane == 0) {
    C.s[m] = make_float4(KDA ? 1.f : second ? a0 * a1 : a0, R.beta[m], am * kk, kq);
    C.dq[m] = am * dq;
    C.e[m] = second ? 1.f : a1;
  }
}

// The tokens f, f + 1 of a group (B = 1: f alone) on a warp's columns; update:
// whether the state after them is wanted.
template <typename T, bool KDA, int NP, int B>
__device__ __forceinline__ void step(const float (*v)[kRecCols], const RecCoef<KDA> &C, int f, float (*us)[16],
                                     Pair (&S)[NP * 4][2], int lane, int wcol, T *o, int64_t o_stride,
                                     bool col_ok, bool update) {
  const int rg = lane >> 2, cg = lane & 3;
  Pair xy[2 * B][2];                  // X_0.., Y_0.. of two pairs of columns, this lane's rows
#pragma unroll
  for (int m = 0; m < 2 * B; ++m) xy[m][0] = xy[m][1] = pair(0.f, 0.f);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int m = 0; m < 2 * B; ++m) {
      const float2 *row = (m < B ? C.kx[f + m] : C.qx[f + m - B]) + 32 * p + 4 * rg;
#pragma unroll
      for (int r = 0; r < 4; r += 2) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(row + r);
        xy[m][0] = fma2(S[4 * p + r][0], w.x, xy[m][0]);
        xy[m][1] = fma2(S[4 * p + r][1], w.x, xy[m][1]);
        xy[m][0] = fma2(S[4 * p + r + 1][0], w.y, xy[m][0]);
        xy[m][1] = fma2(S[4 * p + r + 1][1], w.y, xy[m][1]);
      }
    }
  }
  // Halving: lane bit 4 picks columns 2, 3; bit 3 the odd one; bit 2 Y.
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float t1[2 * B], z[B];
#pragma unroll
  for (int m = 0; m < 2 * B; ++m) {
    const float2 lo2 = unpair(b4 ? xy[m][1] : xy[m][0]), give = unpair(b4 ? xy[m][0] : xy[m][1]);
    const float lo = lo2.x + __shfl_xor_sync(~0u, give.x, 16);
    const float hi = lo2.y + __shfl_xor_sync(~0u, give.y, 16);
    t1[m] = (b3 ? hi : lo) + __shfl_xor_sync(~0u, b3 ? lo : hi, 8);
  }
#pragma unroll
  for (int m = 0; m < B; ++m)
    z[m] = (b2 ? t1[B + m] : t1[m]) + __shfl_xor_sync(~0u, b2 ? t1[m] : t1[B + m], 4);
  const int c = cg * 4 + (b4 ? 2 : 0) + (b3 ? 1 : 0);     // this lane's column of the warp's 16
  // u in the X lanes; the Y lanes take it from there
  const float4 s0 = C.s[f], s1 = C.s[f + B - 1];
  const float z0 = KDA ? z[0] : s0.x * z[0], z1 = KDA ? z[B - 1] : s1.x * z[B - 1];
  const float u0x = s0.y * (v[f][wcol + c] - z0);
  const float u1x = B == 2 ? s1.y * (v[f + 1][wcol + c] - z1 - s1.z * u0x) : 0.f;
  const float u0o = __shfl_xor_sync(~0u, u0x, 4), u1o = B == 2 ? __shfl_xor_sync(~0u, u1x, 4) : 0.f;
  if (b2) {
    if (col_ok) {
      o[c] = from_f32<T>(z0 + s0.w * u0o);
      if (B == 2) o[o_stride + c] = from_f32<T>(z1 + C.dq[f + 1] * u0o + s1.w * u1o);
    }
  } else {
    us[0][c] = B == 2 && !KDA ? C.e[f] * u0x : u0x;
    if (B == 2) us[1][c] = u1x;
  }
  __syncwarp();
  if (!update) return;
  Pair w[B][2];
#pragma unroll
  for (int m = 0; m < B; ++m) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(&us[m][4 * cg]);
    w[m][0] = x.x;
    w[m][1] = x.y;
  }
  __syncwarp();                       // read before the next pair's are written
  const Pair cl = pair(s1.x, s1.x);
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = 32 * p + 4 * rg;
#pragma unroll
    for (int r = 0; r < 4; r += 2) {
      ulonglong2 a = make_ulonglong2(cl, cl);
      // with the channel gate a lone token's decay stands where the two's does
      if (KDA) a = *reinterpret_cast<const ulonglong2 *>(&C.cu[f / 2][at + r]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        S[4 * p + r][i] = mul2(S[4 * p + r][i], a.x);
        S[4 * p + r + 1][i] = mul2(S[4 * p + r + 1][i], a.y);
      }
#pragma unroll
      for (int m = 0; m < B; ++m) {
        const ulonglong2 k =
            *reinterpret_cast<const ulonglong2 *>((KDA ? C.ku[f + m] : C.kx[f + m]) + at + r);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          S[4 * p + r][i] = fma2(w[m][i], k.x, S[4 * p + r][i]);
          S[4 * p + r + 1][i] = fma2(w[m][i], k.y, S[4 * p + r + 1][i]);
        }
      }
    }
  }
}

// Four columns of a state row, as two pairs.
__device__ __forceinline__ void load_pairs(const float *p, Pair (&s)[2]) {
  const float4 v = ld4_stream(p);
  s[0] = pair(v.x, v.y);
  s[1] = pair(v.z, v.w);
}
__device__ __forceinline__ void load_pairs(const __nv_bfloat16 *p, Pair (&s)[2]) {
  const float4 v = ld4_stream(p);
  s[0] = pair(v.x, v.y);
  s[1] = pair(v.z, v.w);
}
template <typename ST>
__device__ __forceinline__ void store_pairs(ST *p, const Pair (&s)[2]) {
  const float2 a = unpair(s[0]), b = unpair(s[1]);
  st4_stream(p, make_float4(a.x, a.y, b.x, b.y));
}

// FULL: d_k = d_v = 128 (NP = 4), so that no row or column needs a check.
template <typename T, typename ST, bool KDA, int NP, bool FULL>
__global__ void __launch_bounds__(kRecWarps * 32, 4) gdn_recurrent_kernel(const __grid_constant__ RecArgs A) {
  __shared__ RecShared<KDA> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / A.splits, split = blockIdx.x % A.splits;
  const int n = unit / A.Hv, h = unit % A.Hv, hk = h / (A.Hv / A.Hk);
  const int dk = FULL ? 32 * NP : A.dk, dv = FULL ? 128 : A.dv;

  // The run. A bad one (tokens outside [0, T], keep outside its length, a slot
  // outside the pool, a slot that another run also names while one of the two
  // writes it) is refused as a whole; a negative slot is padding.
  const int slot = A.slots ? A.slots[n] : n;
  const int t0 = A.cu ? A.cu[n] : n * A.L, t1 = A.cu ? A.cu[n + 1] : t0 + A.L;
  const int kept = A.keep ? A.keep[n] : -2;
  const bool fresh = A.reset && A.reset[n];
  if (t0 < 0 || t1 < t0 || t1 > A.T) {
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    return;
  }
  const int len = t1 - t0;
  if (slot < 0 || len == 0) return;
  const int keep = A.keep ? kept : len;
  bool bad = slot >= A.num_slots || keep < 0 || keep > len;

  const int col0 = split * kRecCols, wcol = warp * 16, rg = lane >> 2, cg = lane & 3;
  const int col = col0 + wcol + 4 * cg;
  const bool col_ok = FULL || col < dv;
  ST *st = static_cast<ST *>(A.pool) + (int64_t(bad ? 0 : slot) * A.Hv + h) * dk * dv + col + 4 * rg * dv;
  Pair S[NP * 4][2];
  // d_v known: the rows lie at constant offsets. Otherwise the pointer steps
  // from row to row, kept from the compiler, which would hold them all.
  {
    const ST *src = st;
#pragma unroll
    for (int i = 0; i < NP * 4; ++i) {
      const int j = 32 * (i >> 2) + (i & 3);            // row less 4 rg
      S[i][0] = S[i][1] = pair(0.f, 0.f);
      if (!bad && !fresh && (FULL || (col_ok && j + 4 * rg < dk))) load_pairs(FULL ? st + j * dv : src, S[i]);
      if (!FULL) {
        src += ((i & 3) == 3 ? 29 : 1) * dv;
        asm volatile("" : "+l"(src));
      }
    }
  }

  // Groups of up to four tokens; none crosses the point after which the state is kept.
  auto group_len = [&](int p) { return min(kGroup, (p < keep ? keep : len) - p); };
  int p0 = 0, n0 = bad ? 0 : group_len(0), p1 = p0 + n0, n1 = bad ? 0 : group_len(p1);
  if (warp < n0) fetch<T, KDA>(A, t0 + int64_t(p0) + warp, h, hk, col0, lane, sm.rows[0], sm.v[0], warp);
  if (warp < n1) fetch<T, KDA>(A, t0 + int64_t(p1) + warp, h, hk, col0, lane, sm.rows[1], sm.v[1], warp);
  if (A.slots && !bad)
    for (int m = tid; m < A.N; m += kRecWarps * 32)
      if (A.slots[m] == slot && m != n) {
        const int lm = A.cu ? A.cu[m + 1] - A.cu[m] : A.L;
        const int km = A.keep ? A.keep[m] : lm;
        if (lm > 0 && (keep > 0 || km > 0)) bad = true;
      }
  land<T, KDA>(A, warp < n0, col0, lane, sm.rows[0], sm.v[0], warp);
  if (n1 > 0) land<T, KDA>(A, warp < n1, col0, lane, sm.rows[1], sm.v[1], warp);
  bad = __syncthreads_or(bad);

  const int64_t o_stride = int64_t(A.Hv) * dv;
  T *o = static_cast<T *>(A.o) + (int64_t(t0) * A.Hv + h) * dv + col0 + wcol;
  if (bad) {   // outputs that cannot be mistaken for results; the state is left alone
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    const float nan = __int_as_float(0x7fffffff);
    if (col_ok && rg == 0)
      for (int t = 0; t < len; ++t) st4(o + t * o_stride + 4 * cg, make_float4(nan, nan, nan, nan));
    return;
  }
  relate<KDA>(sm.rows[0], sm.coef[0], warp, n0, lane);
  __syncthreads();

  const bool idle = !FULL && col0 + wcol >= dv;         // warps behind the last column
  for (int b = 0, slot3 = 0;; ++b) {
    const int p2 = p1 + n1, n2 = group_len(p2);      // 0 at the run's end
    const int slot1 = slot3 == 2 ? 0 : slot3 + 1, slot2 = slot3 == 0 ? 2 : slot3 - 1;
    if (warp < n2)
      fetch<T, KDA>(A, t0 + int64_t(p2) + warp, h, hk, col0, lane, sm.rows[b & 1], sm.v[slot2], warp);
    if (n1 > 0) relate<KDA>(sm.rows[(b + 1) & 1], sm.coef[(b + 1) & 1], warp, n1, lane);
    const RecCoef<KDA> &C = sm.coef[b & 1];
    if (!idle) {
      const bool more = n1 > 0 || p1 == keep;        // the state after this group is wanted
      T *ob = o + p0 * o_stride;
      for (int f = 0; f < n0; f += 2) {
        const bool update = more || f + 2 < n0;
        if (f + 1 < n0)
          step<T, KDA, NP, 2>(sm.v[slot3], C, f, sm.u[warp], S, lane, wcol, ob + f * o_stride, o_stride, col_ok, update);
        else
          step<T, KDA, NP, 1>(sm.v[slot3], C, f, sm.u[warp], S, lane, wcol, ob + f * o_stride, o_stride, col_ok, update);
      }
      if (p1 == keep) {
        ST *dst = st;
#pragma unroll
        for (int i = 0; i < NP * 4; ++i) {
          const int j = 32 * (i >> 2) + (i & 3);
          if (FULL || (col_ok && j + 4 * rg < dk)) store_pairs(FULL ? st + j * dv : dst, S[i]);
          if (!FULL) {
            dst += ((i & 3) == 3 ? 29 : 1) * dv;
            asm volatile("" : "+l"(dst));
          }
        }
      }
    }
    if (n1 == 0) break;
    if (n2 > 0) land<T, KDA>(A, warp < n2, col0, lane, sm.rows[b & 1], sm.v[slot2], warp);
    __syncthreads();
    p0 = p1; n0 = n1; p1 = p2; n1 = n2;
    slot3 = slot1;
  }
}

// One token a run (a decoding batch): one CTA a state, the state in registers
// between one read and one write. A lane holds 16 bytes of each of its rows, so
// a warp reads whole rows; warp w has rows w, w + 8, ... (of a bf16 pool pairs
// of rows) and the warps' partial x and y meet in shared memory. The token's
// rows and gates do not depend on the slot and are under way while it is read;
// so is the search for a second run with the same slot while the state is.
// 16 pieces a lane either way: 8 warps for an fp32 state, 4 for a bf16 one (8
// there too where rows and columns are checked, which takes registers).
template <typename ST, bool FULL>
constexpr int kOneWarps = sizeof(ST) == 4 || !FULL ? 8 : 4;

template <typename ST>
struct Piece;                     // 16 bytes of a state row, as pairs of columns
template <>
struct Piece<float> {
  static constexpr int n = 4;
  float4 w;
  __device__ __forceinline__ void zero() { w = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float *p) { w = __ldcs(reinterpret_cast<const float4 *>(p)); }
  __device__ __forceinline__ Pair get(int i) const { return i ? pair(w.z, w.w) : pair(w.x, w.y); }
  __device__ __forceinline__ void hide() {}
  static __device__ __forceinline__ void store(float *p, const Pair (&x)[2]) {
    const float2 a = unpair(x[0]), b = unpair(x[1]);
    __stcs(reinterpret_cast<float4 *>(p), make_float4(a.x, a.y, b.x, b.y));
  }
};
template <>
struct Piece<__nv_bfloat16> {
  static constexpr int n = 8;
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = __ldcs(reinterpret_cast<const uint4 *>(p)); }
  __device__ __forceinline__ Pair get(int i) const {
    const uint32_t v = i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w;
    return pair(bf_lo(v), bf_hi(v));
  }
  // Keeps the compiler from holding all rows in fp32 from the first pass over
  // them to the second: twice the registers, and it spills.
  __device__ __forceinline__ void hide() {
    asm volatile("" : "+r"(w.x), "+r"(w.y), "+r"(w.z), "+r"(w.w));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const Pair (&x)[4]) {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpair(x[i]);
      v[i] = bf_pack(f.x, f.y);
    }
    __stcs(reinterpret_cast<uint4 *>(p), make_uint4(v[0], v[1], v[2], v[3]));
  }
};

template <typename T, typename ST, bool KDA, bool FULL>      // FULL: d_k = d_v = 128
__global__ void __launch_bounds__(32 * kOneWarps<ST, FULL>, 16 / kOneWarps<ST, FULL>)
    gdn_recurrent_one_kernel(const __grid_constant__ RecArgs A) {
  constexpr int V = Piece<ST>::n, LPR = 128 / V, RPW = 32 / LPR;   // lanes a row, rows a warp at once
  constexpr int W = kOneWarps<ST, FULL>, NR = 128 / (W * RPW);           // pieces a lane
  __shared__ float ks[128], qs[128], us[128], as[KDA ? 128 : 1], ka[KDA ? 128 : 1], qa[KDA ? 128 : 1];
  __shared__ __align__(16) float xpart[W][128], ypart[W][128];
  __shared__ float kq_s;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = blockIdx.x / A.Hv, h = blockIdx.x % A.Hv, hk = h / (A.Hv / A.Hk);
  const int dk = FULL ? 128 : A.dk, dv = FULL ? 128 : A.dv;

  const int slot = A.slots ? A.slots[n] : n;
  const int keep = A.keep ? A.keep[n] : 1;
  const bool fresh = A.reset && A.reset[n];
  float kv = 0.f, qv = 0.f, av = 1.f, vv = 0.f;    // thread c < 128: channel c
  if (tid < dk) {
    kv = to_f32(static_cast<const T *>(A.k)[n * A.k_stride + int64_t(hk) * dk + tid]);
    qv = to_f32(static_cast<const T *>(A.q)[n * A.q_stride + int64_t(hk) * dk + tid]);
    if (KDA) av = A.g[(int64_t(n) * A.Hv + h) * dk + tid];
  }
  if (tid < dv) vv = to_f32(static_cast<const T *>(A.v)[n * A.v_stride + int64_t(h) * dv + tid]);
  const float gate = KDA ? 0.f : A.g[int64_t(n) * A.Hv + h];
  const float beta = A.beta[int64_t(n) * A.Hv + h];
  if (slot < 0) return;
  bool bad = slot >= A.num_slots || keep < 0 || keep > 1;

  const int col = (lane % LPR) * V, sub = lane / LPR;
  const bool col_ok = FULL || col < dv;
  const int row0 = warp * RPW + sub;                // this lane's rows: row0 + r * W * RPW
  ST *st = static_cast<ST *>(A.pool) + (int64_t(bad ? 0 : slot) * A.Hv + h) * dk * dv + row0 * dv + col;
  Piece<ST> S[NR];
  // With d_v known the rows lie at constant offsets. Otherwise the pointer
  // steps from row to row, kept from the compiler, which would hold them all.
  const int step = W * RPW * dv;
  const ST *src = st;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    S[r].zero();
    if ((FULL || (col_ok && row0 + r * W * RPW < dk)) && !bad && !fresh)
      S[r].load(FULL ? st + r * step : src);
    if (!FULL) {
      src += step;
      asm volatile("" : "+l"(src));
    }
  }
  if (A.slots && !bad)
    for (int m = tid; m < A.N; m += 32 * W)
      if (A.slots[m] == slot && m != n && (keep > 0 || !A.keep || A.keep[m] > 0)) bad = true;
  if (tid < 128) {
    const float a = KDA && tid < dk ? expf(av) : 1.f;
    ks[tid] = kv;
    qs[tid] = qv;
    if (KDA) { as[tid] = a; ka[tid] = a * kv; qa[tid] = a * qv; }
  }
  bad = __syncthreads_or(bad);
  T *o = static_cast<T *>(A.o) + (int64_t(n) * A.Hv + h) * dv;
  if (bad) {
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    if (tid < dv) o[tid] = from_f32<T>(__int_as_float(0x7fffffff));
    return;
  }
  if (warp == 0) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s += ks[lane + 32 * i] * qs[lane + 32 * i];
    s = warp_sum(s);
    if (lane == 0) kq_s = s;
  }
  Pair x2[V / 2], y2[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) x2[i] = y2[i] = pair(0.f, 0.f);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    // a few rows of k and q at a time: read ahead for all rows they spill
    if (sizeof(ST) == 2 && r % 4 == 0) asm volatile("" ::: "memory");
    const int j = row0 + r * W * RPW;
    const float kj = KDA ? ka[j] : ks[j], qj = KDA ? qa[j] : qs[j];
    const Pair kk = pair(kj, kj), qq = pair(qj, qj);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const Pair sp = S[r].get(i);
      x2[i] = fma2(sp, kk, x2[i]);
      y2[i] = fma2(sp, qq, y2[i]);
    }
  }
  float x[V], y[V];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) {
    const float2 a = unpair(x2[i]), b = unpair(y2[i]);
    x[2 * i] = a.x; x[2 * i + 1] = a.y;
    y[2 * i] = b.x; y[2 * i + 1] = b.y;
  }
  if (RPW == 2) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      x[i] += __shfl_xor_sync(~0u, x[i], 16);
      y[i] += __shfl_xor_sync(~0u, y[i], 16);
    }
  }
  if (sub == 0) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      sts4(&xpart[warp][col + i], make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
      sts4(&ypart[warp][col + i], make_float4(y[i], y[i + 1], y[i + 2], y[i + 3]));
    }
  }
  __syncthreads();
  const float alpha = KDA ? 1.f : expf(gate);
  if (tid < 128) {
    float xs = 0.f, ys = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) { xs += xpart[w][tid]; ys += ypart[w][tid]; }
    const float u = beta * (vv - alpha * xs);
    us[tid] = u;
    if (tid < dv) o[tid] = from_f32<T>(alpha * ys + kq_s * u);
  }
  if (keep == 0) return;
  __syncthreads();
  ST *dst = st;
  Pair u2[V / 2];
#pragma unroll
  for (int i = 0; i < V / 2; ++i) u2[i] = pair(us[col + 2 * i], us[col + 2 * i + 1]);
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    if (sizeof(ST) == 2 && r % 4 == 0) asm volatile("" ::: "memory");
    const int j = row0 + r * W * RPW;
    const float kj = ks[j], a = KDA ? as[j] : alpha;
    const Pair kk = pair(kj, kj), aa = pair(a, a);
    S[r].hide();
    Pair s[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) s[i] = fma2(u2[i], kk, mul2(aa, S[r].get(i)));
    if (FULL || (col_ok && j < dk)) Piece<ST>::store(FULL ? st + r * step : dst, s);
    if (!FULL) {
      dst += step;
      asm volatile("" : "+l"(dst));
    }
  }
}

template <typename T, typename ST, bool KDA, int NP>
cudaError_t launch_np(RecArgs &A, cudaStream_t s) {
  A.splits = (A.dv + kRecCols - 1) / kRecCols;
  const unsigned grid = unsigned(A.N) * A.Hv * A.splits;
  if (NP == 4 && A.dk == 128 && A.dv == 128)
    gdn_recurrent_kernel<T, ST, KDA, 4, true><<<grid, kRecWarps * 32, 0, s>>>(A);
  else
    gdn_recurrent_kernel<T, ST, KDA, NP, false><<<grid, kRecWarps * 32, 0, s>>>(A);
  return cudaGetLastError();
}

template <typename T, typename ST, bool KDA>
cudaError_t launch_gate(RecArgs &A, cudaStream_t s) {
  // One token a run goes to its own kernel, where the rows come in whole pieces.
  if (!A.cu && A.L == 1 && A.dv % Piece<ST>::n == 0) {
    const unsigned units = unsigned(A.N) * A.Hv;
    if (A.dk == 128 && A.dv == 128)
      gdn_recurrent_one_kernel<T, ST, KDA, true><<<units, 32 * kOneWarps<ST, true>, 0, s>>>(A);
    else
      gdn_recurrent_one_kernel<T, ST, KDA, false><<<units, 32 * kOneWarps<ST, false>, 0, s>>>(A);
    return cudaGetLastError();
  }
  if (A.dk <= 64) return launch_np<T, ST, KDA, 2>(A, s);
  return A.dk <= 96 ? launch_np<T, ST, KDA, 3>(A, s) : launch_np<T, ST, KDA, 4>(A, s);
}

template <typename T, typename ST>
cudaError_t launch_types(RecArgs &A, bool kda, cudaStream_t s) {
  return kda ? launch_gate<T, ST, true>(A, s) : launch_gate<T, ST, false>(A, s);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace gdn

using namespace gdn;

extern "C" int gdn_recurrent_fwd(const void *q, const void *k, const void *v, const float *g,
                                 const float *beta, void *pool, const int32_t *slots,
                                 const int32_t *cu_seqlens, const int32_t *keep,
                                 const uint8_t *reset, int N, int T, int H_k, int H_v, int d_k,
                                 int d_v, int64_t num_slots, int64_t q_stride, int64_t k_stride,
                                 int64_t v_stride, int channel_gate, int dtype, int state_dtype,
                                 void *o, void *status, void *stream) {
  if ((dtype != GDN_BF16 && dtype != GDN_F32) ||
      (state_dtype != GDN_BF16 && state_dtype != GDN_F32))
    return GDN_ERR_INVALID_ARG;
  if (N < 0 || T < 0 || H_k < 1 || H_v < 1 || d_k < 1 || d_v < 1 || num_slots < 0)
    return GDN_ERR_INVALID_ARG;
  if (H_v % H_k) return GDN_ERR_INVALID_ARG;
  if (!cu_seqlens && N > 0 && T % N) return GDN_ERR_INVALID_ARG;
  if (!slots && N > num_slots) return GDN_ERR_INVALID_ARG;
  if (d_k > 128 || d_v > 128 || d_v % 4) return GDN_ERR_UNSUPPORTED;
  if (int64_t(N) * H_v >= (int64_t(1) << 30)) return GDN_ERR_UNSUPPORTED;
  if (q_stride < int64_t(H_k) * d_k || k_stride < int64_t(H_k) * d_k ||
      v_stride < int64_t(H_v) * d_v)
    return GDN_ERR_INVALID_ARG;
  if (N == 0 || T == 0) return GDN_OK;
  if (!q || !k || !v || !g || !beta || !pool || !o) return GDN_ERR_INVALID_ARG;
  const size_t e = dtype == GDN_BF16 ? 2 : 4;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(o, 4 * e) ||
      !aligned(pool, 16) || !aligned(g, 4) || !aligned(beta, 4) || !aligned(slots, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(keep, 4) || !aligned(status, 4))
    return GDN_ERR_INVALID_ARG;
  RecArgs A{};
  A.q = q; A.k = k; A.v = v; A.g = g; A.beta = beta; A.pool = pool;
  A.slots = slots; A.cu = cu_seqlens; A.keep = keep; A.reset = reset;
  A.o = o; A.status = static_cast<uint32_t *>(status);
  A.q_stride = q_stride; A.k_stride = k_stride; A.v_stride = v_stride;
  A.num_slots = num_slots;
  A.N = N; A.T = T; A.L = cu_seqlens ? 0 : T / N;
  A.Hk = H_k; A.Hv = H_v; A.dk = d_k; A.dv = d_v;
  A.vec = d_k % 4 == 0 && q_stride % 4 == 0 && k_stride % 4 == 0 && v_stride % 4 == 0 &&
          aligned(q, 4 * e) && aligned(k, 4 * e) && aligned(v, 4 * e) && (!channel_gate || aligned(g, 16));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (dtype == GDN_BF16)
    err = state_dtype == GDN_BF16 ? launch_types<__nv_bfloat16, __nv_bfloat16>(A, channel_gate, s)
                                  : launch_types<__nv_bfloat16, float>(A, channel_gate, s);
  else
    err = state_dtype == GDN_BF16 ? launch_types<float, __nv_bfloat16>(A, channel_gate, s)
                                  : launch_types<float, float>(A, channel_gate, s);
  return err == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}
