// The recurrent gated delta rule for serving: runs of new tokens of many
// sequences against a pool of states addressed by slot (gdn_recurrent_fwd).
//
// Run n covers tokens [t0, t1) and the state in slot slots[n]. Per value head
// (key head hk = h / (H_v / H_k)), with the state held transposed
// (st[j][i] = S_ij) and a_j = exp(g) (one value, or one per d_k channel j):
//   x_i = sum_j st[j][i] a_j k_j          y_i = sum_j st[j][i] a_j q_j
//   u_i = beta (v_i - x_i)                st[j][i] <- a_j st[j][i] + u_i k_j
//   o_i = y_i + (k . q) u_i               (= S_t q, read after the write)
// x and y come from the old state in one pass, so a token costs one reduction.
//
// A warp owns 16 columns i and all rows j of one state; columns of st evolve
// independently, so a run needs no exchange between warps. Lane (rg, cg) =
// (lane / 4, lane % 4) holds columns 4 cg .. 4 cg + 3 of rows 32 p + 4 rg + r
// (r < 4, p < d_k / 32) in registers for the whole run: HBM sees one read and
// one write of the state however many tokens the run has. The eight partial
// sums (x and y of four columns) are reduced over the eight rg lanes by
// halving: 7 shuffles, after which each lane holds one of the eight values.
//
// q, k, v and the gates of up to eight tokens at a time are staged in shared
// memory in fp32 by one warp per token (which also forms k . q).
#include "gdn_internal.cuh"
#include "rows.cuh"

namespace gdn {
namespace {

constexpr int kRecBatch = 8;        // tokens staged at a time

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

// Staged token: k (with the channel gate also a .* k, a .* q and a), q, v, and
// {a, beta, k . q}.
template <bool KDA>
struct RecStage {
  float k[kRecBatch][128], q[kRecBatch][128], v[kRecBatch][128];
  float ka[KDA ? kRecBatch : 1][128], a[KDA ? kRecBatch : 1][128];
  float gate[kRecBatch][4];
};

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

template <typename T, typename ST, bool KDA, int NP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, 16 / WARPS) gdn_recurrent_kernel(const RecArgs A) {
  __shared__ RecStage<KDA> sm;

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int unit = blockIdx.x / A.splits, split = blockIdx.x % A.splits;
  const int n = unit / A.Hv, h = unit % A.Hv, hk = h / (A.Hv / A.Hk);
  const int dk = A.dk, dv = A.dv;

  // The run. A bad one (tokens outside [0, T], keep outside its length, a slot
  // outside the pool, a slot that another run also names while one of the two
  // writes it) is refused as a whole; a negative slot is padding.
  const int t0 = A.cu ? A.cu[n] : n * A.L, t1 = A.cu ? A.cu[n + 1] : t0 + A.L;
  if (t0 < 0 || t1 < t0 || t1 > A.T) {
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    return;
  }
  const int len = t1 - t0;
  const int slot = A.slots ? A.slots[n] : n;
  if (slot < 0 || len == 0) return;
  const int keep = A.keep ? A.keep[n] : len;
  bool bad = slot >= A.num_slots || keep < 0 || keep > len;

  const int rg = lane >> 2, col = (split * WARPS + warp) * 16 + (lane & 3) * 4;
  const bool col_ok = col < dv;
  ST *st = static_cast<ST *>(A.pool) + (int64_t(bad ? 0 : slot) * A.Hv + h) * dk * dv + col;
  float4 S[NP * 4];
  const bool zero = bad || (A.reset && A.reset[n]);
#pragma unroll
  for (int i = 0; i < NP * 4; ++i) {
    const int j = 32 * (i >> 2) + 4 * rg + (i & 3);
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col_ok && j < dk && !zero) S[i] = ld4_stream(st + int64_t(j) * dv);
  }

  if (A.slots && !bad)
    for (int m = tid; m < A.N; m += WARPS * 32)
      if (A.slots[m] == slot && m != n) {
        const int lm = A.cu ? A.cu[m + 1] - A.cu[m] : A.L;
        const int km = A.keep ? A.keep[m] : lm;
        if (lm > 0 && (keep > 0 || km > 0)) bad = true;
      }
  bad = __syncthreads_or(bad);

  T *o = static_cast<T *>(A.o) + (int64_t(t0) * A.Hv + h) * dv + col;
  const int64_t o_stride = int64_t(A.Hv) * dv;
  if (bad) {   // outputs that cannot be mistaken for results; the state is left alone
    if (tid == 0 && A.status) atomicOr(A.status, kErrBadSeqlens);
    const float nan = __int_as_float(0x7fffffff);
    if (col_ok && rg == 0)
      for (int t = 0; t < len; ++t) st4(o + t * o_stride, make_float4(nan, nan, nan, nan));
    return;
  }

  for (int b0 = 0; b0 < len; b0 += kRecBatch) {
    const int nb = min(kRecBatch, len - b0);
    if (b0) __syncthreads();
    for (int b = warp; b < nb; b += WARPS) {
      const int64_t t = t0 + b0 + b;
      const int c = lane * 4;
      const float4 k4 = load4(static_cast<const T *>(A.k) + t * A.k_stride + int64_t(hk) * dk + c, dk - c, A.vec);
      const float4 q4 = load4(static_cast<const T *>(A.q) + t * A.q_stride + int64_t(hk) * dk + c, dk - c, A.vec);
      const float4 v4 = load4(static_cast<const T *>(A.v) + t * A.v_stride + int64_t(h) * dv + c, dv - c, A.vec);
      const float kq = warp_sum(k4.x * q4.x + k4.y * q4.y + k4.z * q4.z + k4.w * q4.w);
      *reinterpret_cast<float4 *>(&sm.k[b][c]) = k4;
      *reinterpret_cast<float4 *>(&sm.v[b][c]) = v4;
      float4 qa = q4;
      float a = 1.f;
      if (KDA) {
        const float *gp = A.g + (t * A.Hv + h) * dk + c;
        float4 a4 = make_float4(1.f, 1.f, 1.f, 1.f);
        if (c + 0 < dk) a4.x = expf(gp[0]);
        if (c + 1 < dk) a4.y = expf(gp[1]);
        if (c + 2 < dk) a4.z = expf(gp[2]);
        if (c + 3 < dk) a4.w = expf(gp[3]);
        qa = make_float4(q4.x * a4.x, q4.y * a4.y, q4.z * a4.z, q4.w * a4.w);
        *reinterpret_cast<float4 *>(&sm.ka[b][c]) =
            make_float4(k4.x * a4.x, k4.y * a4.y, k4.z * a4.z, k4.w * a4.w);
        *reinterpret_cast<float4 *>(&sm.a[b][c]) = a4;
      } else {
        a = expf(A.g[t * A.Hv + h]);
      }
      *reinterpret_cast<float4 *>(&sm.q[b][c]) = qa;
      if (lane == 0)
        *reinterpret_cast<float4 *>(sm.gate[b]) =
            make_float4(a, A.beta[t * A.Hv + h], kq, 0.f);
    }
    __syncthreads();

    for (int b = 0; b < nb; ++b) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const float4 k4 = *reinterpret_cast<const float4 *>(
            KDA ? &sm.ka[b][32 * p + 4 * rg] : &sm.k[b][32 * p + 4 * rg]);
        const float4 q4 = *reinterpret_cast<const float4 *>(&sm.q[b][32 * p + 4 * rg]);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, qq[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float4 s = S[4 * p + r];
          x.x += s.x * kk[r]; x.y += s.y * kk[r]; x.z += s.z * kk[r]; x.w += s.w * kk[r];
          y.x += s.x * qq[r]; y.y += s.y * qq[r]; y.z += s.z * qq[r]; y.w += s.w * qq[r];
        }
      }
      const float4 gate = *reinterpret_cast<const float4 *>(sm.gate[b]);   // a, beta, k . q
      // Halving: lanes with bit 4 of the lane number keep y, the others x ...
      const bool up = lane & 16;
      float4 w;
      {
        const float4 keep4 = up ? y : x, give = up ? x : y;
        w.x = keep4.x + __shfl_xor_sync(~0u, give.x, 16);
        w.y = keep4.y + __shfl_xor_sync(~0u, give.y, 16);
        w.z = keep4.z + __shfl_xor_sync(~0u, give.z, 16);
        w.w = keep4.w + __shfl_xor_sync(~0u, give.w, 16);
      }
      // ... bit 3 picks columns 2, 3 and bit 2 the odd one.
      const bool hi = lane & 8, odd = lane & 4;
      const float w0 = (hi ? w.z : w.x) + __shfl_xor_sync(~0u, hi ? w.x : w.z, 8);
      const float w1 = (hi ? w.w : w.y) + __shfl_xor_sync(~0u, hi ? w.y : w.w, 8);
      const float sum = (odd ? w1 : w0) + __shfl_xor_sync(~0u, odd ? w0 : w1, 4);
      const int c = (hi ? 2 : 0) + (odd ? 1 : 0);       // this lane's column of its four
      const float z = KDA ? sum : gate.x * sum;         // x (lower lanes) or y (upper lanes)
      float u = gate.y * (sm.v[b][(col + c) & 127] - z);
      u = __shfl_sync(~0u, u, lane & 15);               // the x lane of the same column
      const float out = z + gate.z * u;                 // upper lanes: o of column c
      float4 u4;
      u4.x = __shfl_sync(~0u, u, (lane & 3));
      u4.y = __shfl_sync(~0u, u, (lane & 3) + 4);
      u4.z = __shfl_sync(~0u, u, (lane & 3) + 8);
      u4.w = __shfl_sync(~0u, u, (lane & 3) + 12);
      if (up && col_ok) o[(b0 + b) * o_stride + c] = from_f32<T>(out);
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const float4 k4 = *reinterpret_cast<const float4 *>(&sm.k[b][32 * p + 4 * rg]);
        float4 a4 = make_float4(gate.x, gate.x, gate.x, gate.x);
        if (KDA) a4 = *reinterpret_cast<const float4 *>(&sm.a[b][32 * p + 4 * rg]);
        const float kk[4] = {k4.x, k4.y, k4.z, k4.w}, aa[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float4 &s = S[4 * p + r];
          s.x = aa[r] * s.x + u4.x * kk[r]; s.y = aa[r] * s.y + u4.y * kk[r];
          s.z = aa[r] * s.z + u4.z * kk[r]; s.w = aa[r] * s.w + u4.w * kk[r];
        }
      }
      if (b0 + b + 1 == keep && col_ok) {
#pragma unroll
        for (int i = 0; i < NP * 4; ++i) {
          const int j = 32 * (i >> 2) + 4 * rg + (i & 3);
          if (j < dk) st4_stream(st + int64_t(j) * dv, S[i]);
        }
      }
    }
  }
}

template <typename T, typename ST, bool KDA, int NP>
cudaError_t launch_np(RecArgs &A, cudaStream_t s) {
  const int warps = (A.dv + 15) / 16;
  A.splits = (warps + 7) / 8;
  const unsigned grid = unsigned(A.N) * A.Hv * A.splits;
  gdn_recurrent_kernel<T, ST, KDA, NP, 8><<<grid, 256, 0, s>>>(A);
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
