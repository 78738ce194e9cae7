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
// S the state before the group, c_m = a_0 .. a_m, d_ml = a_(l+1) .. a_m:
//   X_m = S^T k_m,  Y_m = S^T q_m                    (one pass, one reduction)
//   u_m = beta_m (v_m - c_m X_m - sum_(l<m) d_ml (k_l . k_m) u_l)
//   o_m = c_m Y_m + sum_(l<=m) d_ml (k_l . q_m) u_l
//   S  <- c_last S + sum_l d_(last,l) u_l k_l         (one pass)
// With the channel gate the products of decays sit inside the dot products and
// in rows of k and q scaled by them. All of them are products of the tokens'
// own decays, never quotients, so a decay of zero is as good as any other.
//
// A CTA of four warps owns 64 columns i and all rows j of one state, in
// registers for the whole run: HBM sees one read and one write of the state
// however many tokens the run has. Lane (sub, cl) = (lane / 16, lane % 16) of a
// warp holds columns 4 cl .. 4 cl + 3 of rows 32 p + 4 g + r (g = 2 warp + sub,
// r < 4, p < d_k / 32). The two sub lanes add up their X and Y by a shuffle,
// the four warps through shared memory; then one thread has a column's X of
// every token and another its Y, which makes the chain over a group's tokens
// two barriers long. Measured (B200, 64 runs of 1 to 6 tokens, 32 heads, d =
// 128): 50 us, 64 % of the copy rate; with all rows of 16 columns in one warp,
// three shuffles and two tokens a pass instead, 56 us. One state's 64 tokens
// alone take 42 us (39 us that way): a warp then has its scheduler to itself
// and waits for its own operands. Short runs are bound by the chain from a
// CTA's slot to its rows to its state, which four CTAs an SM overlap; long ones
// by the multiply-adds and the instructions around them (313 a token and warp,
// 96 of them paired multiply-adds).
//
// k, q, v and the decays of a group come through shared memory in fp32, a token
// a warp: the rows of the group after next are on their way from HBM, those of
// the next are multiplied with each other, while this one is computed. k and q
// lie there twice over, k_j k_j, so that one 16-byte read gives the operands of
// paired multiply-adds for two rows (2.2 cycles for 64 products a scheduler,
// against 2.9 for two single ones).
#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kRecWarps = 4, kRecCols = 16 * kRecWarps;   // columns of d_v per CTA
constexpr int kGroup = 4;                                 // tokens taken together

struct RecArgs {
  const void *q, *k, *v;
  const float *g, *beta;
  void *pool;
  const int32_t *slots, *cu, *keep;
  const uint8_t *reset;
  void *o;
  uint32_t *status;
  int64_t q_stride, k_stride, v_stride, num_slots;
  int N, T, L, Hv, dk, dv;          // L: tokens per run without cu
  int splits;                       // CTAs per state: 1 or 2
  float per_k;                      // H_k / H_v
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
// What follows from them: rows of k and q twice over (channel gate: c_m k_m, c_m
// q_m), and the scalars of the chain.
template <bool KDA>
struct alignas(16) RecCoef {
  float2 kx[kGroup][128], qx[kGroup][128];
  float ku[KDA ? kGroup : 1][128];              // channel gate: d_(last, m) k_m
  float cu[KDA ? 128 : 4];                      // channel gate: c_last
  float A[kGroup][kGroup], P[kGroup][kGroup];   // [m][l]: d_ml (k_l . k_m), d_ml (k_l . q_m)
  float c[kGroup], e[kGroup], beta[kGroup];     // c_m and d_(last, m); 1 with the channel gate
};
template <bool KDA>
struct alignas(16) RecShared {
  RecRows<KDA> rows[2];              // of the next group; being fetched for the one after
  RecCoef<KDA> coef[2];              // of this group and of the next
  float v[3][kGroup][kRecCols];      // of all three
  float part[kRecWarps][2 * kGroup][kRecCols];   // the warps' X_0 .. X_3, Y_0 .. Y_3
  float u[kGroup][kRecCols], ue[kGroup][kRecCols];   // u_m; d_(last, m) u_m
};
static_assert(sizeof(RecRows<false>) % 16 == 0 && sizeof(RecRows<true>) % 16 == 0 &&
              sizeof(RecCoef<false>) % 16 == 0 && sizeof(RecCoef<true>) % 16 == 0 &&
              offsetof(RecCoef<false>, ku) % 16 == 0 && offsetof(RecCoef<true>, cu) % 16 == 0 &&
              offsetof(RecRows<false>, a) % 16 == 0,
              "rows are read in 16-byte pieces");

// Grid: x the CTAs of a run, y and z the runs.
constexpr int kGridY = 65535;
__device__ __forceinline__ int run_of(const RecArgs &A) { return blockIdx.y + blockIdx.z * kGridY; }
dim3 grid_of(const RecArgs &A, int per_run) {
  return dim3(unsigned(per_run), unsigned(A.N < kGridY ? A.N : kGridY), unsigned((A.N + kGridY - 1) / kGridY));
}
// h / (H_v / H_k): the middle of a head's interval, so that rounding of a few
// 2^-24 of h < 2^20 cannot reach the next whole number.
__device__ __forceinline__ int key_head(const RecArgs &A, int h) {
  return int((float(h) + 0.5f) * A.per_k);
}

// Bounds checks (GDN_CHECKS builds): n elements from p on, of a buffer of extent
// elements; what lies outside is skipped and recorded in the status block.
#define REC_IN_BOUNDS(base, p, n, extent) \
  GDN_IN_BOUNDS(A.status, (p) - (base), static_cast<long long>(extent) - (n) + 1)
#if GDN_CHECKS
__device__ __forceinline__ int64_t key_extent(const RecArgs &A, int64_t stride) {
  return int64_t(A.T - 1) * stride + int64_t(key_head(A, A.Hv - 1) + 1) * A.dk;
}
__device__ __forceinline__ int64_t value_extent(const RecArgs &A) {
  return int64_t(A.T - 1) * A.v_stride + int64_t(A.Hv) * A.dv;
}
__device__ __forceinline__ int64_t gate_extent(const RecArgs &A, bool kda) {
  return int64_t(A.T) * A.Hv * (kda ? A.dk : 1);
}
__device__ __forceinline__ int64_t pool_extent(const RecArgs &A) { return A.num_slots * A.Hv * A.dk * A.dv; }
__device__ __forceinline__ int64_t out_extent(const RecArgs &A) { return int64_t(A.T) * A.Hv * A.dv; }
#endif

// Up to four elements, one by one; zero past the n-th.
template <typename T>
__device__ __forceinline__ float4 load4(const T *p, int n) {
  float4 r = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n > 0) r.x = to_f32(p[0]);
  if (n > 1) r.y = to_f32(p[1]);
  if (n > 2) r.z = to_f32(p[2]);
  if (n > 3) r.w = to_f32(p[3]);
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
  const int kn = min(4, A.dk - c), vn = min(4, A.dv - col0 - c);      // what there is of the lane's four
  if (kn > 0 && !(REC_IN_BOUNDS(static_cast<const T *>(A.k), kp, kn, key_extent(A, A.k_stride)) &&
                  REC_IN_BOUNDS(static_cast<const T *>(A.q), qp, kn, key_extent(A, A.q_stride)) &&
                  (!KDA || REC_IN_BOUNDS(A.g, gp + c, kn, gate_extent(A, KDA)))))
    return;
  if (c < kRecCols && vn > 0 && !REC_IN_BOUNDS(static_cast<const T *>(A.v), vp, vn, value_extent(A))) return;
  if (!(KDA || REC_IN_BOUNDS(A.g, gp, 1, gate_extent(A, KDA))) ||
      !REC_IN_BOUNDS(A.beta, A.beta + t * A.Hv + h, 1, int64_t(A.T) * A.Hv))
    return;
  if (A.vec) {
    if (c < A.dk) {
      copy_async(reinterpret_cast<T *>(R.k[m]) + c, kp, 4 * sizeof(T));
      copy_async(reinterpret_cast<T *>(R.q[m]) + c, qp, 4 * sizeof(T));
      if (KDA) copy_async(&R.a[m][c], gp + c, 16);
    }
    if (c < kRecCols && col0 + c < A.dv) copy_async(reinterpret_cast<T *>(v[m]) + c, vp, 4 * sizeof(T));
  } else {
    sts4(&R.k[m][c], load4(kp, A.dk - c));
    sts4(&R.q[m][c], load4(qp, A.dk - c));
    if (KDA) sts4(&R.a[m][c], load4(gp + c, A.dk - c));
    if (c < kRecCols) sts4(&v[m][c], load4(vp, A.dv - col0 - c));
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

// One warp works out what token m has to do with those before it. nb: tokens of
// the group.
template <bool KDA>
__device__ __forceinline__ void relate(const RecRows<KDA> &R, RecCoef<KDA> &C, int m, int nb, int lane) {
  if (m >= nb) return;
  const int c = lane * 4;
  const float4 km = lds4(&R.k[m][c]), qm = lds4(&R.q[m][c]);
  float z[8];                         // k_l . k_m (l = 0..3), k_l . q_m
  float4 kd = km, qd = qm;            // with the decays since l
#pragma unroll
  for (int l = kGroup - 1; l >= 0; --l) {
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
    put_twice(&C.kx[m][c], mul4(kd, a0));
    put_twice(&C.qx[m][c], mul4(qd, a0));
    float4 e = make_float4(1.f, 1.f, 1.f, 1.f);
    for (int l = m + 1; l < nb; ++l) e = mul4(e, lds4(&R.a[l][c]));
    sts4(&C.ku[m][c], mul4(km, e));
    if (m == 0) sts4(&C.cu[c], mul4(a0, e));
  } else {
    put_twice(&C.kx[m][c], km);
    put_twice(&C.qx[m][c], qm);
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
    for (int i = 0; i < kGroup; ++i) {
      const float a = R.a[i][0];
      if (i <= m) cm *= a;
      if (i <= m && i > l) d *= a;
      if (i > m && i < nb) e *= a;
    }
  }
  if ((lane & 3) == 0) (lane & 16 ? C.P : C.A)[m][l] = d * y;
  if (lane == 0) { C.c[m] = cm; C.e[m] = e; C.beta[m] = R.beta[m]; }
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
  const int split = A.splits == 2 ? blockIdx.x & 1 : 0, h = A.splits == 2 ? blockIdx.x >> 1 : blockIdx.x;
  const int n = run_of(A);
  if (n >= A.N) return;
  const int hk = key_head(A, h);
  const int dk = FULL ? 32 * NP : A.dk, dv = FULL ? 128 : A.dv;

  // The run. A bad one (tokens outside [0, T], keep outside its length, a slot
  // outside the pool, a slot that another run also names while one of the two
  // writes it) is refused as a whole; a negative slot is padding, whatever its
  // boundaries say (a captured batch's unused runs may hold stale ones).
  const int slot = A.slots ? A.slots[n] : n;
  const int t0 = A.cu ? A.cu[n] : n * A.L, t1 = A.cu ? A.cu[n + 1] : t0 + A.L;
  const int kept = A.keep ? A.keep[n] : -2;
  const bool fresh = A.reset && A.reset[n];
  const bool outside = t0 < 0 || t1 < t0 || t1 > A.T;
  const int len = int(unsigned(t1) - unsigned(t0));
  if (outside || slot < 0 || len == 0) {
    if (outside && slot >= 0 && tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    return;
  }
  const int keep = A.keep ? kept : len;
  bool bad = slot >= A.num_slots || keep < 0 || keep > len;

  const int col0 = split * kRecCols, cl = 4 * (lane & 15), g4 = 4 * (2 * warp + (lane >> 4));
  const int col = col0 + cl;
  const bool col_ok = FULL || col < dv;
  ST *st = static_cast<ST *>(A.pool) + (int64_t(bad ? 0 : slot) * A.Hv + h) * dk * dv + col + g4 * dv;
  Pair S[NP * 4][2];
  // d_v known: the rows lie at constant offsets. Otherwise the pointer steps
  // from row to row, kept from the compiler, which would hold them all (with d_k
  // above 96 up to 16 bytes a thread are spilled all the same).
  if (bad || fresh) {
#pragma unroll
    for (int i = 0; i < NP * 4; ++i) S[i][0] = S[i][1] = pair(0.f, 0.f);
  } else {
    const ST *src = st;
#pragma unroll
    for (int i = 0; i < NP * 4; ++i) {
      const int j = 32 * (i >> 2) + (i & 3);            // row less g4
      if (!FULL) S[i][0] = S[i][1] = pair(0.f, 0.f);
      if ((FULL || (col_ok && j + g4 < dk)) &&
          REC_IN_BOUNDS(static_cast<ST *>(A.pool), FULL ? st + j * dv : src, 4, pool_extent(A)))
        load_pairs(FULL ? st + j * dv : src, S[i]);
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
  T *o = static_cast<T *>(A.o) + (int64_t(t0) * A.Hv + h) * dv + col0;
  if (bad) {   // outputs that cannot be mistaken for results; the state is left alone
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    const float nan = __int_as_float(0x7fffffff);
    if (col_ok && g4 == 0)
      for (int t = 0; t < len; ++t)
        if (REC_IN_BOUNDS(static_cast<T *>(A.o), o + t * o_stride + cl, 4, out_extent(A)))
          st4(o + t * o_stride + cl, make_float4(nan, nan, nan, nan));
    return;
  }
  relate<KDA>(sm.rows[0], sm.coef[0], warp, n0, lane);
  __syncthreads();

  // A bf16 state under fp32 activations takes its tokens one by one, products and
  // sum rounded each, as the definition writes them: the fp32 value that is then
  // rounded to 16 bits depends on how tokens fall into groups and calls only
  // through the sums' order. Grouped and fused, two to four times as many of the
  // stored values came out a step apart from those of the plain rule, which the
  // next call's fp32 outputs show (in single places by a thousandth of their
  // size); the error against 64 bits is the same either way. What it costs, in
  // instructions and in reads that start later: 42.6 us against 42.0 for 64 runs
  // of 1 to 6 tokens (32 heads, d = 128), 58 against 53 for 13 ragged runs of 0
  // to 64 (15 heads, d 96 and 80), 101 against 89 for 24 runs of 10 to 64 (16
  // heads, d = 128).
  constexpr bool kStep = sizeof(T) == 4 && sizeof(ST) == 2;
  const bool ylane = warp >= kRecWarps / 2;             // this thread's part of the chain: Y or X
  const int c = tid % kRecCols;                         // of this column
  const bool c_ok = FULL || col0 + c < dv;
  for (int b = 0, slot3 = 0;; ++b) {
    const int p2 = p1 + n1, n2 = group_len(p2);      // 0 at the run's end
    const int slot1 = slot3 == 2 ? 0 : slot3 + 1, slot2 = slot3 == 0 ? 2 : slot3 - 1;
    if (!kStep && warp < n2)
      fetch<T, KDA>(A, t0 + int64_t(p2) + warp, h, hk, col0, lane, sm.rows[b & 1], sm.v[slot2], warp);
    const RecCoef<KDA> &C = sm.coef[b & 1];
    if (b) __syncthreads();           // the next group's rows have landed
    if (n1 > 0) relate<KDA>(sm.rows[(b + 1) & 1], sm.coef[(b + 1) & 1], warp, n1, lane);

#pragma unroll 1
    for (int m = 0; m < n0; ++m) {
      Pair x[2] = {pair(0.f, 0.f), pair(0.f, 0.f)}, y[2] = {x[0], x[0]};
#pragma unroll
      for (int i = 0; i < NP * 4; i += 2) {
        const int j = 32 * (i >> 2) + (i & 3) + g4;
        const ulonglong2 k = *reinterpret_cast<const ulonglong2 *>(&C.kx[m][j]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2 *>(&C.qx[m][j]);
        x[0] = fma2(S[i][0], k.x, x[0]);
        x[1] = fma2(S[i][1], k.x, x[1]);
        y[0] = fma2(S[i][0], q.x, y[0]);
        y[1] = fma2(S[i][1], q.x, y[1]);
        x[0] = fma2(S[i + 1][0], k.y, x[0]);
        x[1] = fma2(S[i + 1][1], k.y, x[1]);
        y[0] = fma2(S[i + 1][0], q.y, y[0]);
        y[1] = fma2(S[i + 1][1], q.y, y[1]);
      }
      // the lower sixteen lanes take columns 0 and 1 of four, the upper ones 2 and 3
      const bool up = lane & 16;
      const float2 xk = unpair(up ? x[1] : x[0]), xg = unpair(up ? x[0] : x[1]);
      const float2 yk = unpair(up ? y[1] : y[0]), yg = unpair(up ? y[0] : y[1]);
      float2 xs, ys;
      xs.x = xk.x + __shfl_xor_sync(~0u, xg.x, 16);
      xs.y = xk.y + __shfl_xor_sync(~0u, xg.y, 16);
      ys.x = yk.x + __shfl_xor_sync(~0u, yg.x, 16);
      ys.y = yk.y + __shfl_xor_sync(~0u, yg.y, 16);
      const int at = cl + (up ? 2 : 0);
      *reinterpret_cast<float2 *>(&sm.part[warp][m][at]) = xs;
      *reinterpret_cast<float2 *>(&sm.part[warp][kGroup + m][at]) = ys;
    }
    __syncthreads();

    float z[kGroup];
#pragma unroll
    for (int m = 0; m < kGroup; ++m) {
      z[m] = 0.f;
      if (m < n0) {
        const int i = (ylane ? kGroup : 0) + m;
        z[m] = (sm.part[0][i][c] + sm.part[1][i][c]) + (sm.part[2][i][c] + sm.part[3][i][c]);
        if (!KDA) z[m] *= C.c[m];
      }
    }
    if (!ylane) {
      float u[kGroup];
#pragma unroll
      for (int m = 0; m < kGroup; ++m) {
        u[m] = 0.f;
        if (m < n0) {
          float x = sm.v[slot3][m][c] - z[m];
#pragma unroll
          for (int l = 0; l < m; ++l) x -= C.A[m][l] * u[l];
          u[m] = C.beta[m] * x;
          sm.u[m][c] = u[m];
          sm.ue[m][c] = KDA ? u[m] : C.e[m] * u[m];
        }
      }
    }
    __syncthreads();

    if (ylane && c_ok) {
#pragma unroll
      for (int m = 0; m < kGroup; ++m)
        if (m < n0) {
          float y = z[m];
#pragma unroll
          for (int l = 0; l <= m; ++l) y += C.P[m][l] * sm.u[l][c];
          if (REC_IN_BOUNDS(static_cast<T *>(A.o), o + (p0 + m) * o_stride + c, 1, out_extent(A)))
            o[(p0 + m) * o_stride + c] = from_f32<T>(y);
        }
    }
    if (kStep && (n1 > 0 || p1 == keep)) {
      const RecRows<KDA> &R = sm.rows[b & 1];
#pragma unroll 1
      for (int m = 0; m < n0; ++m) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sm.u[m][cl]);
#pragma unroll
        for (int i = 0; i < NP * 4; ++i) {
          const int j = 32 * (i >> 2) + (i & 3) + g4;
          const float k = R.k[m][j], a = R.a[m][KDA ? j : 0];
          const Pair k2 = pair(k, k), a2 = pair(a, a);
          S[i][0] = add2_apart(mul2(S[i][0], a2), mul2(w.x, k2));
          S[i][1] = add2_apart(mul2(S[i][1], a2), mul2(w.y, k2));
        }
      }
    } else if (n1 > 0 || p1 == keep) {   // the state after this group is wanted
      const Pair cl2 = KDA ? 0 : pair(C.c[n0 - 1], C.c[n0 - 1]);
#pragma unroll
      for (int i = 0; i < NP * 4; ++i) {
        const float a = KDA ? C.cu[32 * (i >> 2) + (i & 3) + g4] : 0.f;
        const Pair a2 = KDA ? pair(a, a) : cl2;
        S[i][0] = mul2(S[i][0], a2);
        S[i][1] = mul2(S[i][1], a2);
      }
#pragma unroll 1
      for (int m = 0; m < n0; ++m) {
        const ulonglong2 w = *reinterpret_cast<const ulonglong2 *>(&sm.ue[m][cl]);
#pragma unroll
        for (int i = 0; i < NP * 4; i += 2) {
          const int j = 32 * (i >> 2) + (i & 3) + g4;
          ulonglong2 k;
          if (KDA) {
            const float2 f = *reinterpret_cast<const float2 *>(&C.ku[m][j]);
            k = make_ulonglong2(pair(f.x, f.x), pair(f.y, f.y));
          } else {
            k = *reinterpret_cast<const ulonglong2 *>(&C.kx[m][j]);
          }
          S[i][0] = fma2(w.x, k.x, S[i][0]);
          S[i][1] = fma2(w.y, k.x, S[i][1]);
          S[i + 1][0] = fma2(w.x, k.y, S[i + 1][0]);
          S[i + 1][1] = fma2(w.y, k.y, S[i + 1][1]);
        }
      }
    }
    if (p1 == keep) {
      ST *dst = st;
#pragma unroll
      for (int i = 0; i < NP * 4; ++i) {
        const int j = 32 * (i >> 2) + (i & 3);
        if ((FULL || (col_ok && j + g4 < dk)) &&
            REC_IN_BOUNDS(static_cast<ST *>(A.pool), FULL ? st + j * dv : dst, 4, pool_extent(A)))
          store_pairs(FULL ? st + j * dv : dst, S[i]);
        if (!FULL) {
          dst += ((i & 3) == 3 ? 29 : 1) * dv;
          asm volatile("" : "+l"(dst));
        }
      }
    }
    if (n1 == 0) break;
    if (kStep && n2 > 0) {            // this group's rows were read up to here
      __syncthreads();
      if (warp < n2)
        fetch<T, KDA>(A, t0 + int64_t(p2) + warp, h, hk, col0, lane, sm.rows[b & 1], sm.v[slot2], warp);
    }
    if (n2 > 0) land<T, KDA>(A, warp < n2, col0, lane, sm.rows[b & 1], sm.v[slot2], warp);
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
// Bound by HBM: 256 states of 32 heads, d = 128, in 170 us = 97 % of the copy
// rate; 96 x 32 bf16 states with the channel gate in 34 us = 93 %.
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
  const int n = run_of(A), h = blockIdx.x;
  if (n >= A.N) return;
  const int hk = key_head(A, h);
  const int dk = FULL ? 128 : A.dk, dv = FULL ? 128 : A.dv;

  const int slot = A.slots ? A.slots[n] : n;
  const int keep = A.keep ? A.keep[n] : 1;
  const bool fresh = A.reset && A.reset[n];
  float kv = 0.f, qv = 0.f, av = 1.f, vv = 0.f;    // thread c < 128: channel c
  const int64_t head = int64_t(n) * A.Hv + h;
  if (tid < dk) {
    const int64_t ki = n * A.k_stride + int64_t(hk) * dk + tid, qi = n * A.q_stride + int64_t(hk) * dk + tid;
    if (GDN_IN_BOUNDS(A.status, ki, key_extent(A, A.k_stride))) kv = to_f32(static_cast<const T *>(A.k)[ki]);
    if (GDN_IN_BOUNDS(A.status, qi, key_extent(A, A.q_stride))) qv = to_f32(static_cast<const T *>(A.q)[qi]);
    if (KDA && GDN_IN_BOUNDS(A.status, head * dk + tid, gate_extent(A, KDA))) av = A.g[head * dk + tid];
  }
  if (tid < dv) {
    const int64_t vi = n * A.v_stride + int64_t(h) * dv + tid;
    if (GDN_IN_BOUNDS(A.status, vi, value_extent(A))) vv = to_f32(static_cast<const T *>(A.v)[vi]);
  }
  float gate = 0.f, beta = 0.f;
  if (GDN_IN_BOUNDS(A.status, head, int64_t(A.T) * A.Hv)) {
    if (!KDA) gate = A.g[head];
    beta = A.beta[head];
  }
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
    if ((FULL || (col_ok && row0 + r * W * RPW < dk)) && !bad && !fresh &&
        REC_IN_BOUNDS(static_cast<ST *>(A.pool), FULL ? st + r * step : src, V, pool_extent(A)))
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
  T *o = static_cast<T *>(A.o) + head * dv;
  const bool o_ok = tid < dv && GDN_IN_BOUNDS(A.status, head * dv + tid, out_extent(A));
  if (bad) {
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    if (o_ok) o[tid] = from_f32<T>(__int_as_float(0x7fffffff));
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
    if (o_ok) o[tid] = from_f32<T>(alpha * ys + kq_s * u);
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
    for (int i = 0; i < V / 2; ++i)   // products and sum rounded each: see kStep
      s[i] = add2_apart(mul2(aa, S[r].get(i)), mul2(u2[i], kk));
    if ((FULL || (col_ok && j < dk)) &&
        REC_IN_BOUNDS(static_cast<ST *>(A.pool), FULL ? st + r * step : dst, V, pool_extent(A)))
      Piece<ST>::store(FULL ? st + r * step : dst, s);
    if (!FULL) {
      dst += step;
      asm volatile("" : "+l"(dst));
    }
  }
}

template <typename T, typename ST, bool KDA, int NP>
cudaError_t launch_np(RecArgs &A, cudaStream_t s) {
  A.splits = (A.dv + kRecCols - 1) / kRecCols;
  const dim3 grid = grid_of(A, A.Hv * A.splits);
  if (NP == 4 && A.dk == 128 && A.dv == 128)
    gdn_recurrent_kernel<T, ST, KDA, 4, true><<<grid, kRecWarps * 32, 0, s>>>(A);
  else
    gdn_recurrent_kernel<T, ST, KDA, NP, false><<<grid, kRecWarps * 32, 0, s>>>(A);
  return cudaGetLastError();
}

template <typename T, typename ST, bool KDA>
cudaError_t launch_gate(RecArgs &A, cudaStream_t s) {
  // One token a run goes to its own kernel, where the rows come in whole pieces
  // (169 us against 179 us for 256 x 32 fp32 states, 34 us against 49 us for 96
  // x 32 bf16 ones by the kernel for runs). A call with boundaries never does: the
  // lengths are on the device.
  if (!A.cu && A.L == 1 && A.dv % Piece<ST>::n == 0) {
    const dim3 units = grid_of(A, A.Hv);
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
  if (H_v >= 1 << 20 || int64_t(N) * H_v >= (int64_t(1) << 30)) return GDN_ERR_UNSUPPORTED;
  // the search for a slot named twice: N reads a run and head (two seconds or so at the limit)
  if (slots && double(N) * N * H_v > 4398046511104.0) return GDN_ERR_UNSUPPORTED;   // 2^42
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
  A.per_k = float(H_k) / float(H_v);
  A.Hv = H_v; A.dk = d_k; A.dv = d_v;
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
