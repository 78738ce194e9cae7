// The recurrent gated delta rule for serving: runs of new tokens of many
// sequences against a pool of states addressed by slot (gdn_recurrent_fwd).
//
// Run n covers tokens [t0, t1) and the state in slot slots[n]. Per value head
// (key head hk = h / (H_v / H_k)), with the state held transposed
// (st[j][i] = S_ij) and a_j = exp(g) (one value, or one per d_k channel j):
//   x_i = sum_j st[j][i] a_j k_j,  u_i = beta (v_i - x_i)
//   st[j][i] <- a_j st[j][i] + u_i k_j,  o_i = sum_j st[j][i] q_j
//
// Up to four tokens are taken together, so that a pass over the state serves
// all of them and the chain from token to token runs over a few scalars. With
// S the state before the block, c_m = a_0 .. a_m, d_ml = a_(l+1) .. a_m:
//   X_m = S^T k_m,  Y_m = S^T q_m                    (one pass, one reduction)
//   u_m = beta_m (v_m - c_m X_m - sum_(l<m) d_ml (k_l . k_m) u_l)
//   o_m = c_m Y_m + sum_(l<=m) d_ml (k_l . q_m) u_l
//   S  <- c_last S + sum_l d_(last,l) u_l k_l         (one pass)
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
// k, q, v and the decays come through shared memory in fp32, a token a warp:
// the rows of block n + 2 are on their way from HBM, those of block n + 1 are
// multiplied with each other, while block n is computed.
#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kRecWarps = 4, kRecCols = 16 * kRecWarps;   // columns of d_v per CTA
constexpr int kBlock = 4;                                 // tokens taken together

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

// A block's tokens as they came, in fp32. Tokens past the block's end are zero
// with decay 1.
template <bool KDA>
struct alignas(16) RecRows {
  float k[kBlock][128], q[kBlock][128], v[kBlock][kRecCols];
  float a[kBlock][KDA ? 128 : 4];
  float beta[kBlock];
};
// What follows from them.
template <bool KDA>
struct alignas(16) RecCoef {
  float A[kBlock][kBlock], P[kBlock][kBlock];   // [m][l]: d_ml (k_l . k_m), d_ml (k_l . q_m)
  float c[kBlock], e[kBlock];                   // c_m and d_(last, l); 1 with the channel gate
  float ka[KDA ? kBlock : 1][128], qa[KDA ? kBlock : 1][128];   // c_m k_m, c_m q_m per channel
  float ke[KDA ? kBlock : 1][128], ce[KDA ? 128 : 1];           // d_(last, l) k_l, c_last
};
template <bool KDA>
struct alignas(16) RecShared {
  RecRows<KDA> rows[3];
  RecCoef<KDA> coef[2];
  float u[kRecWarps][kBlock][16];
};

static_assert(sizeof(RecRows<false>) % 16 == 0 && sizeof(RecRows<true>) % 16 == 0 &&
              sizeof(RecCoef<false>) % 16 == 0 && sizeof(RecCoef<true>) % 16 == 0 &&
              offsetof(RecCoef<false>, ka) % 16 == 0 && offsetof(RecRows<false>, a) % 16 == 0,
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

// One token's share of a lane.
template <bool KDA>
struct RecToken {
  float4 k, q, v, a;
  float beta;
};

template <typename T, bool KDA>
__device__ __forceinline__ void fetch(const RecArgs &A, int64_t t, bool on, int h, int hk, int col0,
                                      int lane, RecToken<KDA> &r) {
  const int c = lane * 4;
  r.k = r.q = r.v = make_float4(0.f, 0.f, 0.f, 0.f);
  r.a = make_float4(1.f, 1.f, 1.f, 1.f);
  r.beta = 0.f;
  if (!on) return;
  r.k = load4(static_cast<const T *>(A.k) + t * A.k_stride + int64_t(hk) * A.dk + c, A.dk - c, A.vec);
  r.q = load4(static_cast<const T *>(A.q) + t * A.q_stride + int64_t(hk) * A.dk + c, A.dk - c, A.vec);
  if (c < kRecCols)
    r.v = load4(static_cast<const T *>(A.v) + t * A.v_stride + int64_t(h) * A.dv + col0 + c,
                A.dv - col0 - c, A.vec);
  if (KDA) {
    const float *gp = A.g + (t * A.Hv + h) * A.dk + c;
    if (c + 0 < A.dk) r.a.x = gp[0];
    if (c + 1 < A.dk) r.a.y = gp[1];
    if (c + 2 < A.dk) r.a.z = gp[2];
    if (c + 3 < A.dk) r.a.w = gp[3];
  } else {
    r.a.x = A.g[t * A.Hv + h];
  }
  r.beta = A.beta[t * A.Hv + h];
}

template <bool KDA>
__device__ __forceinline__ void put(RecRows<KDA> &R, int m, bool on, int lane, int dk,
                                    const RecToken<KDA> &r) {
  const int c = lane * 4;
  sts4(&R.k[m][c], r.k);
  sts4(&R.q[m][c], r.q);
  if (c < kRecCols) sts4(&R.v[m][c], r.v);
  if (KDA) {
    float4 a = r.a;
    if (on) {
      a.x = c + 0 < dk ? expf(a.x) : 1.f;
      a.y = c + 1 < dk ? expf(a.y) : 1.f;
      a.z = c + 2 < dk ? expf(a.z) : 1.f;
      a.w = c + 3 < dk ? expf(a.w) : 1.f;
    }
    sts4(&R.a[m][c], a);
  } else if (lane == 0) {
    R.a[m][0] = on ? expf(r.a.x) : 1.f;
  }
  if (lane == 0) R.beta[m] = r.beta;
}

// Warp m works out what token m has to do with those before it.
template <bool KDA>
__device__ __forceinline__ void relate(const RecRows<KDA> &R, RecCoef<KDA> &C, int m, int nb, int lane) {
  const int c = lane * 4;
  if (m >= nb) {
    if (KDA) {      // a token of padding multiplies these by zero
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      sts4(&C.ka[m][c], zero);
      sts4(&C.qa[m][c], zero);
      sts4(&C.ke[m][c], zero);
    }
    return;
  }
  const float4 km = lds4(&R.k[m][c]), qm = lds4(&R.q[m][c]);
  float z[8];                         // k_l . k_m (l = 0..3), k_l . q_m
  float4 kd = km, qd = qm;            // with the decays since l
#pragma unroll
  for (int l = kBlock - 1; l >= 0; --l) {
    z[l] = z[4 + l] = 0.f;
    if (l > m) continue;
    const float4 kl = lds4(&R.k[l][c]);
    if (KDA && l < m) {
      const float4 a = lds4(&R.a[l + 1][c]);
      kd = mul4(kd, a);
      qd = mul4(qd, a);
    }
    z[l] = dot4(kl, kd);
    z[4 + l] = dot4(kl, qd);
  }
  if (KDA) {
    const float4 a0 = lds4(&R.a[0][c]);
    sts4(&C.ka[m][c], mul4(kd, a0));
    sts4(&C.qa[m][c], mul4(qd, a0));
    float4 e = make_float4(1.f, 1.f, 1.f, 1.f);
    for (int l = m + 1; l < nb; ++l) e = mul4(e, lds4(&R.a[l][c]));
    sts4(&C.ke[m][c], mul4(km, e));
    if (m == 0) sts4(&C.ce[c], mul4(a0, e));
  }
  // sum over the warp by halving: lane bits 4, 3, 2 pick one of the eight
  float y4[4], y2[2], y;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    y4[i] = (lane & 16 ? z[4 + i] : z[i]) + __shfl_xor_sync(~0u, lane & 16 ? z[i] : z[4 + i], 16);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    y2[i] = (lane & 8 ? y4[2 + i] : y4[i]) + __shfl_xor_sync(~0u, lane & 8 ? y4[i] : y4[2 + i], 8);
  y = (lane & 4 ? y2[1] : y2[0]) + __shfl_xor_sync(~0u, lane & 4 ? y2[0] : y2[1], 4);
  y += __shfl_xor_sync(~0u, y, 2);
  y += __shfl_xor_sync(~0u, y, 1);
  const int l = (lane >> 2) & 3;
  float d = 1.f, cm = 1.f, e = 1.f;
  if (!KDA) {
#pragma unroll
    for (int i = 0; i < kBlock; ++i) {
      const float a = R.a[i][0];
      if (i <= m) cm *= a;
      if (i <= m && i > l) d *= a;
      if (i > m && i < nb) e *= a;
    }
  }
  if ((lane & 3) == 0) (lane & 16 ? C.P : C.A)[m][l] = d * y;
  if (lane == 0) { C.c[m] = cm; C.e[m] = e; }
}

// One block of B tokens (the last may be padding) on a warp's columns.
template <typename T, bool KDA, int NP, int B>
__device__ __forceinline__ void block_step(const RecRows<KDA> &R, const RecCoef<KDA> &C, float (*us)[16],
                                           float4 (&S)[NP * 4], int nb, int lane, int wcol, T *o,
                                           int64_t o_stride, bool col_ok) {
  const int rg = lane >> 2, cg = lane & 3;
  float xy[2 * B][4];                 // X_0.., Y_0.. of four columns, this lane's rows
#pragma unroll
  for (int m = 0; m < 2 * B; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) xy[m][i] = 0.f;
#pragma unroll
  for (int p = 0; p < NP; ++p) {
#pragma unroll
    for (int m = 0; m < B; ++m) {
      const int at = 32 * p + 4 * rg;
      const float4 k4 = lds4(KDA ? &C.ka[m][at] : &R.k[m][at]);
      const float4 q4 = lds4(KDA ? &C.qa[m][at] : &R.q[m][at]);
      const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float4 s = S[4 * p + r];
        xy[m][0] += s.x * kk[r]; xy[m][1] += s.y * kk[r];
        xy[m][2] += s.z * kk[r]; xy[m][3] += s.w * kk[r];
        xy[B + m][0] += s.x * qq[r]; xy[B + m][1] += s.y * qq[r];
        xy[B + m][2] += s.z * qq[r]; xy[B + m][3] += s.w * qq[r];
      }
    }
  }
  // Halving: lane bit 4 picks columns 2, 3; bit 3 the odd one; bit 2 Y.
  const bool b4 = lane & 16, b3 = lane & 8, b2 = lane & 4;
  float t1[2 * B], z[B];
#pragma unroll
  for (int m = 0; m < 2 * B; ++m) {
    const float lo = (b4 ? xy[m][2] : xy[m][0]) + __shfl_xor_sync(~0u, b4 ? xy[m][0] : xy[m][2], 16);
    const float hi = (b4 ? xy[m][3] : xy[m][1]) + __shfl_xor_sync(~0u, b4 ? xy[m][1] : xy[m][3], 16);
    t1[m] = (b3 ? hi : lo) + __shfl_xor_sync(~0u, b3 ? lo : hi, 8);
  }
#pragma unroll
  for (int m = 0; m < B; ++m)
    z[m] = (b2 ? t1[B + m] : t1[m]) + __shfl_xor_sync(~0u, b2 ? t1[m] : t1[B + m], 4);
  const int c = cg * 4 + (b4 ? 2 : 0) + (b3 ? 1 : 0);     // this lane's column of the warp's 16
  float u[B];
#pragma unroll
  for (int m = 0; m < B; ++m) {       // right in the X lanes; the Y lanes take it from there
    float x = R.v[m][wcol + c] - (KDA ? z[m] : C.c[m] * z[m]);
#pragma unroll
    for (int l = 0; l < m; ++l) x -= C.A[m][l] * u[l];
    u[m] = m < nb ? R.beta[m] * x : 0.f;
  }
  __syncwarp();
  if (!b2)
#pragma unroll
    for (int m = 0; m < B; ++m) us[m][c] = KDA || m >= nb ? u[m] : C.e[m] * u[m];
#pragma unroll
  for (int m = 0; m < B; ++m) {
    const float other = __shfl_xor_sync(~0u, u[m], 4);
    u[m] = b2 ? other : u[m];
  }
  __syncwarp();
  if (b2 && col_ok)
#pragma unroll
    for (int m = 0; m < B; ++m)
      if (m < nb) {
        float y = KDA ? z[m] : C.c[m] * z[m];
#pragma unroll
        for (int l = 0; l <= m; ++l) y += C.P[m][l] * u[l];
        o[m * o_stride + c] = from_f32<T>(y);
      }
  float4 w[B];
#pragma unroll
  for (int m = 0; m < B; ++m) w[m] = lds4(&us[m][4 * cg]);
  const float cl = KDA ? 1.f : C.c[nb - 1];
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const int at = 32 * p + 4 * rg;
    float4 a4 = make_float4(cl, cl, cl, cl);
    if (KDA) a4 = lds4(&C.ce[at]);
    const float aa[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float4 &s = S[4 * p + r];
      s = make_float4(s.x * aa[r], s.y * aa[r], s.z * aa[r], s.w * aa[r]);
    }
#pragma unroll
    for (int m = 0; m < B; ++m) {
      const float4 k4 = lds4(KDA ? &C.ke[m][at] : &R.k[m][at]);
      const float kk[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float4 &s = S[4 * p + r];
        s.x += w[m].x * kk[r]; s.y += w[m].y * kk[r]; s.z += w[m].z * kk[r]; s.w += w[m].w * kk[r];
      }
    }
  }
}

// FULL: d_k = 32 NP and d_v = 128, so that no row or column needs a check.
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
  float4 S[NP * 4];
#pragma unroll
  for (int i = 0; i < NP * 4; ++i) {
    const int j = 32 * (i >> 2) + (i & 3);            // row less 4 rg
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!bad && !fresh && (FULL || (col_ok && j + 4 * rg < dk))) S[i] = ld4_stream(st + j * dv);
  }

  // Blocks of up to four tokens; none crosses the point after which the state is kept.
  auto block_len = [&](int p) { return min(kBlock, (p < keep ? keep : len) - p); };
  int p0 = 0, n0 = bad ? 0 : block_len(0), p1 = p0 + n0, n1 = bad ? 0 : block_len(p1);
  {
    RecToken<KDA> r;
    fetch<T, KDA>(A, t0 + int64_t(p0) + warp, warp < n0, h, hk, col0, lane, r);
    put<KDA>(sm.rows[0], warp, warp < n0, lane, dk, r);
    if (n1 > 0) {
      fetch<T, KDA>(A, t0 + int64_t(p1) + warp, warp < n1, h, hk, col0, lane, r);
      put<KDA>(sm.rows[1], warp, warp < n1, lane, dk, r);
    }
  }
  if (A.slots && !bad)
    for (int m = tid; m < A.N; m += kRecWarps * 32)
      if (A.slots[m] == slot && m != n) {
        const int lm = A.cu ? A.cu[m + 1] - A.cu[m] : A.L;
        const int km = A.keep ? A.keep[m] : lm;
        if (lm > 0 && (keep > 0 || km > 0)) bad = true;
      }
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

  for (int b = 0, slot3 = 0;; ++b) {
    const int p2 = p1 + n1, n2 = block_len(p2);      // 0 at the run's end
    RecToken<KDA> r;
    if (n2 > 0) fetch<T, KDA>(A, t0 + int64_t(p2) + warp, warp < n2, h, hk, col0, lane, r);
    const int slot1 = slot3 == 2 ? 0 : slot3 + 1, slot2 = slot3 == 0 ? 2 : slot3 - 1;
    if (n1 > 0) relate<KDA>(sm.rows[slot1], sm.coef[(b + 1) & 1], warp, n1, lane);
    const RecRows<KDA> &R = sm.rows[slot3];
    const RecCoef<KDA> &C = sm.coef[b & 1];
    T *ob = o + p0 * o_stride;
    if (n0 > 2)
      block_step<T, KDA, NP, 4>(R, C, sm.u[warp], S, n0, lane, wcol, ob, o_stride, col_ok);
    else if (n0 == 2)
      block_step<T, KDA, NP, 2>(R, C, sm.u[warp], S, n0, lane, wcol, ob, o_stride, col_ok);
    else
      block_step<T, KDA, NP, 1>(R, C, sm.u[warp], S, n0, lane, wcol, ob, o_stride, col_ok);
    if (p1 == keep) {
#pragma unroll
      for (int i = 0; i < NP * 4; ++i) {
        const int j = 32 * (i >> 2) + (i & 3);
        if (FULL || (col_ok && j + 4 * rg < dk)) st4_stream(st + j * dv, S[i]);
      }
    }
    if (n1 == 0) break;
    if (n2 > 0) put<KDA>(sm.rows[slot2], warp, warp < n2, lane, dk, r);
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
  // One token a run goes to its own kernel, where the rows come in whole pieces.
  if (!A.cu && A.L == 1 && A.dv % Piece<ST>::n == 0) {
    const unsigned units = unsigned(A.N) * A.Hv;
    if (A.dk == 128 && A.dv == 128)
      gdn_recurrent_one_kernel<T, ST, KDA, true><<<units, 32 * kOneWarps<ST, true>, 0, s>>>(A);
    else
      gdn_recurrent_one_kernel<T, ST, KDA, false><<<units, 32 * kOneWarps<ST, false>, 0, s>>>(A);
    return cudaGetLastError();
  }
  A.splits = (A.dv + kRecCols - 1) / kRecCols;
  const unsigned grid = unsigned(A.N) * A.Hv * A.splits;
  if (A.dk == 32 * NP && A.dv == 128)
    gdn_recurrent_kernel<T, ST, KDA, NP, true><<<grid, kRecWarps * 32, 0, s>>>(A);
  else
    gdn_recurrent_kernel<T, ST, KDA, NP, false><<<grid, kRecWarps * 32, 0, s>>>(A);
  return cudaGetLastError();
}

template <typename T, typename ST>
cudaError_t launch_types(RecArgs &A, bool kda, cudaStream_t s) {
  if (A.dk <= 64)
    return kda ? launch_np<T, ST, true, 2>(A, s) : launch_np<T, ST, false, 2>(A, s);
  return kda ? launch_np<T, ST, true, 4>(A, s) : launch_np<T, ST, false, 4>(A, s);
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
          aligned(q, 4 * e) && aligned(k, 4 * e) && aligned(v, 4 * e);
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
