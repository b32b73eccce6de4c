// gdn_qk_norm.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their gradients (gdn_qk_norm.h).
//
// A head of D channels lies on D / 8 lanes, eight neighbouring channels each;
// its sum of squares is a sum over those eight in ascending order and a
// butterfly over the lanes, so a head's bits are its own.  A block takes a
// few tokens and all their heads: the angles' cosines and sines are computed
// once for a token into shared memory and serve every head.  A rotated pair
// (j, j + F) lies on two lanes F / 8 apart (one shuffle), an interleaved pair
// on one.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/gdn_qk_norm.h"
#include "gdn_common.cuh"

namespace gdn {

constexpr int kQkThreads = 256;
constexpr int kQkMaxTokens = 16;      // tokens of a block's angle table
constexpr int kQkWeightBlocks = 592;  // most partial sums of a weight's gradient

enum QkRot { kRotNone = 0, kRotHalves = 1, kRotPairs = 2 };

struct QkSide {
  const void* x;
  int64_t ldx;
  const float* w;
  void* y;
  int64_t ldy;
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  int H;
};

struct QkArgs {
  QkSide q, k;
  int64_t T;
  const int32_t* positions;
  const float* inv_freq;
  int F;            // rotated pairs
  int tokens;       // of one table
  int64_t span;     // tokens of one block
  float eps, inv_m;  // inv_m: 1 (l2) or 1 / D (rms)
  float* partial;   // [blocks][2][D] or nullptr
};

__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
  f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&f)[8]) {
  const uint4 r = *reinterpret_cast<const uint4*>(p);
  const unsigned u[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&f)[8]) {
  union {
    uint4 r;
    __nv_bfloat162 h[4];
  } u;
#pragma unroll
  for (int i = 0; i < 4; i++) u.h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = u.r;
}

// Cosine and sine of pos * f.  The angle is taken in quarter turns in fp64
// (an fp32 product has lost the angle from positions of a few thousand on)
// and the nearest quarter removed, so that the fp32 functions see at most an
// eighth of a turn.
__device__ __forceinline__ float2 angle(int pos, float f) {
  const double quarters = (double)pos * ((double)f * 0.63661977236758134308);  // 2 / pi
  const double whole = rint(quarters);
  float s, c;
  sincospif(0.5f * (float)(quarters - whole), &s, &c);
  const int turn = (int)((long long)whole & 3);
  if (turn & 1) {
    const float x = c;
    c = -s;
    s = x;
  }
  return turn & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

__device__ __forceinline__ void angle_table(const QkArgs& p, int64_t t0, int nt, float* cs,
                                            float* sn) {
  for (int e = threadIdx.x; e < nt * p.F; e += kQkThreads) {
    const int t = e / p.F, j = e - t * p.F;
    const float2 a = angle(p.positions[t0 + t], p.inv_freq[j]);
    cs[e] = a.x;
    sn[e] = a.y;
  }
}

// Rotate the eight channels from c0 on by the angles at cs, sn (SIGN = -1:
// back).  Every lane of the warp calls this.
template <int ROT, int SIGN>
__device__ __forceinline__ void rotate8(float (&n)[8], int c0, int F, const float* cs,
                                        const float* sn) {
  if (ROT == kRotHalves) {
    const bool first = c0 < F, in = c0 < 2 * F;
    const int lane = threadIdx.x & 31;
    const int src = in ? (first ? lane + F / 8 : lane - F / 8) : lane;
    const int j = first ? c0 : c0 - F;
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const float other = __shfl_sync(kFull, n[i], src);
      if (in) {
        const float s = (first ? -SIGN : SIGN) * sn[j + i];
        n[i] = __fmaf_rn(other, s, __fmul_rn(n[i], cs[j + i]));
      }
    }
  } else if (ROT == kRotPairs && c0 < 2 * F) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float c = cs[c0 / 2 + i], s = SIGN * sn[c0 / 2 + i];
      const float u = n[2 * i], v = n[2 * i + 1];
      n[2 * i] = __fmaf_rn(-v, s, __fmul_rn(u, c));
      n[2 * i + 1] = __fmaf_rn(u, s, __fmul_rn(v, c));
    }
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float s) {
#pragma unroll
  for (int m = 1; m < D / 8; m *= 2) s = __fadd_rn(s, __shfl_xor_sync(kFull, s, m));
  return s;
}

template <int D>
__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s = __fmul_rn(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 8; i++) s = __fmaf_rn(a[i], b[i], s);
  return head_sum<D>(s);
}

template <int D>
__device__ __forceinline__ void weights8(const float* w, int c0, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i++) f[i] = 1.f;
  if (w) load8(w + c0, f);
}

template <class IN, class OUT, int D, int ROT>
__global__ void __launch_bounds__(kQkThreads) k_qk_forward(const QkArgs p) {
  constexpr int kLanes = D / 8, kGroups = kQkThreads / kLanes;
  extern __shared__ float smem[];
  float *cs = smem, *sn = smem + p.tokens * p.F;
  const int64_t t0 = (int64_t)blockIdx.x * p.tokens;
  const int nt = (int)min((int64_t)p.tokens, p.T - t0);
  if (ROT != kRotNone) {
    angle_table(p, t0, nt, cs, sn);
    __syncthreads();
  }
  const int grp = threadIdx.x / kLanes, c0 = (threadIdx.x % kLanes) * 8;
  const int heads = p.q.H + p.k.H, items = nt * heads;
  float wq[8], wk[8];
  weights8<D>(p.q.w, c0, wq);
  weights8<D>(p.k.w, c0, wk);
  for (int first = 0; first < items; first += kGroups) {
    const int it = first + grp;
    const bool have = it < items;
    const int t = have ? it / heads : 0, hd = have ? it - t * heads : 0;
    const bool isq = hd < p.q.H;
    const QkSide& sd = isq ? p.q : p.k;
    const int64_t ch = (int64_t)(isq ? hd : hd - p.q.H) * D + c0;
    float n[8] = {};
    if (have) load8(static_cast<const IN*>(sd.x) + (t0 + t) * sd.ldx + ch, n);
    const float r =
        __frsqrt_rn(__fmaf_rn(dot8<D>(n, n), p.inv_m, p.eps));
#pragma unroll
    for (int i = 0; i < 8; i++) n[i] = __fmul_rn(__fmul_rn(n[i], r), isq ? wq[i] : wk[i]);
    rotate8<ROT, 1>(n, c0, p.F, cs + t * p.F, sn + t * p.F);
    if (have) store8(static_cast<OUT*>(sd.y) + (t0 + t) * sd.ldy + ch, n);
  }
}

template <class IN, class GR, int D, int ROT>
__device__ __forceinline__ void qk_backward_side(const QkArgs& p, const QkSide& sd, int64_t t0,
                                                 int nt, const float* cs, const float* sn,
                                                 float (&dw)[8]) {
  constexpr int kLanes = D / 8, kGroups = kQkThreads / kLanes;
  const int grp = threadIdx.x / kLanes, c0 = (threadIdx.x % kLanes) * 8;
  const int items = nt * sd.H;
  float w[8];
  weights8<D>(sd.w, c0, w);
  for (int first = 0; first < items; first += kGroups) {
    const int it = first + grp;
    const bool have = it < items;
    const int t = have ? it / sd.H : 0;
    const int64_t ch = (int64_t)(have ? it - t * sd.H : 0) * D + c0;
    float x[8] = {}, e[8] = {};
    if (have) {
      load8(static_cast<const IN*>(sd.x) + (t0 + t) * sd.ldx + ch, x);
      load8(static_cast<const GR*>(sd.dy) + (t0 + t) * sd.lddy + ch, e);
    }
    rotate8<ROT, -1>(e, c0, p.F, cs + t * p.F, sn + t * p.F);
    const float r = __frsqrt_rn(__fmaf_rn(dot8<D>(x, x), p.inv_m, p.eps));
#pragma unroll
    for (int i = 0; i < 8; i++) {
      dw[i] = __fmaf_rn(e[i], __fmul_rn(x[i], r), dw[i]);
      e[i] = __fmul_rn(e[i], w[i]);
    }
    const float m = __fmul_rn(dot8<D>(x, e), p.inv_m);
    const float z = __fmul_rn(__fmul_rn(r, r), m);
#pragma unroll
    for (int i = 0; i < 8; i++) e[i] = __fmul_rn(r, __fmaf_rn(-x[i], z, e[i]));
    if (have) store8(static_cast<IN*>(sd.dx) + (t0 + t) * sd.lddx + ch, e);
  }
}

// The block's sum of dw over its groups, in ascending order.
template <int D>
__device__ __forceinline__ void weight_partial(const float (&dw)[8], float* red, float* out) {
  constexpr int kLanes = D / 8, kGroups = kQkThreads / kLanes;
  const int grp = threadIdx.x / kLanes, c0 = (threadIdx.x % kLanes) * 8;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; i++) red[grp * D + c0 + i] = dw[i];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kQkThreads) {
    float s = 0.f;
    for (int j = 0; j < kGroups; j++) s = __fadd_rn(s, red[j * D + c]);
    out[c] = s;
  }
}

template <class IN, class GR, int D, int ROT>
__global__ void __launch_bounds__(kQkThreads) k_qk_backward(const QkArgs p) {
  extern __shared__ float smem[];
  float *cs = smem, *sn = smem + p.tokens * p.F;
  float dwq[8] = {}, dwk[8] = {};
  const int64_t begin = (int64_t)blockIdx.x * p.span, end = min(p.T, begin + p.span);
  for (int64_t t0 = begin; t0 < end; t0 += p.tokens) {
    const int nt = (int)min((int64_t)p.tokens, end - t0);
    if (ROT != kRotNone) {
      if (t0 != begin) __syncthreads();  // the last tokens' angles have been read
      angle_table(p, t0, nt, cs, sn);
      __syncthreads();
    }
    qk_backward_side<IN, GR, D, ROT>(p, p.q, t0, nt, cs, sn, dwq);
    qk_backward_side<IN, GR, D, ROT>(p, p.k, t0, nt, cs, sn, dwk);
  }
  if (p.partial) {
    __shared__ float red[kQkThreads * 8];
    float* out = p.partial + (int64_t)blockIdx.x * 2 * D;
    weight_partial<D>(dwq, red, out);
    weight_partial<D>(dwk, red, out + D);
  }
}

// d_w = sum of the blocks' partial sums: row group r of 8 adds the blocks
// r, r + 8, ... in order, then the groups are added in order.
__global__ void __launch_bounds__(256) k_qk_weight_sum(const float* partial, int blocks, int D,
                                                       float* d_wq, float* d_wk) {
  __shared__ float red[8][32];
  float* out = blockIdx.y == 0 ? d_wq : d_wk;
  if (!out) return;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  const float* col = partial + blockIdx.y * D + c;
  float s = 0.f;
  for (int b = r; b < blocks; b += 8) s = __fadd_rn(s, col[(int64_t)b * 2 * D]);
  red[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0) {
    for (int j = 1; j < 8; j++) s = __fadd_rn(s, red[j][threadIdx.x]);
    out[c] = s;
  }
}

// ----------------------------------------------------------------------------
// Launchers
// ----------------------------------------------------------------------------
struct QkPlan {
  int tokens;
  int64_t span, blocks;
};

// Tokens of a block: about four heads for each of its lane groups, fewer
// while the batch would leave multiprocessors idle.
static int qk_tokens(int64_t T, int heads, int d) {
  const int groups = kQkThreads / (d / 8);
  int n = 4 * groups / heads;
  n = n < 1 ? 1 : n > kQkMaxTokens ? kQkMaxTokens : n;
  while (n > 1 && (T + n - 1) / n < kQkWeightBlocks) n /= 2;
  return n;
}

static QkPlan qk_plan(int64_t T, int heads, int d, bool weights) {
  QkPlan pl;
  pl.tokens = qk_tokens(T, heads, d);
  pl.span = pl.tokens;
  if (weights) {
    const int64_t per = (T + kQkWeightBlocks - 1) / kQkWeightBlocks;
    pl.span = (per + pl.tokens - 1) / pl.tokens * pl.tokens;
  }
  pl.blocks = (T + pl.span - 1) / pl.span;
  return pl;
}

static size_t qk_smem(const QkArgs& p, int rot) {
  return rot == kRotNone ? 0 : (size_t)2 * p.tokens * p.F * sizeof(float);
}

template <class IN, class OTHER, int D, int ROT>
static cudaError_t qk_launch(bool backward, const QkArgs& p, int64_t blocks, cudaStream_t st) {
  if (backward)
    k_qk_backward<IN, OTHER, D, ROT><<<(unsigned)blocks, kQkThreads, qk_smem(p, ROT), st>>>(p);
  else
    k_qk_forward<IN, OTHER, D, ROT><<<(unsigned)blocks, kQkThreads, qk_smem(p, ROT), st>>>(p);
  return cudaGetLastError();
}

template <class IN, class OTHER, int D>
static cudaError_t qk_rot(bool bwd, const QkArgs& p, int rot, int64_t n, cudaStream_t st) {
  if (rot == kRotNone) return qk_launch<IN, OTHER, D, kRotNone>(bwd, p, n, st);
  if (rot == kRotHalves) return qk_launch<IN, OTHER, D, kRotHalves>(bwd, p, n, st);
  return qk_launch<IN, OTHER, D, kRotPairs>(bwd, p, n, st);
}

template <class IN, class OTHER>
static cudaError_t qk_dims(bool bwd, const QkArgs& p, int d, int rot, int64_t n,
                           cudaStream_t st) {
  if (d == 64) return qk_rot<IN, OTHER, 64>(bwd, p, rot, n, st);
  if (d == 128) return qk_rot<IN, OTHER, 128>(bwd, p, rot, n, st);
  return qk_rot<IN, OTHER, 256>(bwd, p, rot, n, st);
}

static cudaError_t qk_types(bool bwd, const QkArgs& p, bool ib, bool ob, int d, int rot,
                            int64_t n, cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  if (ib)
    return ob ? qk_dims<bf16, bf16>(bwd, p, d, rot, n, st)
              : qk_dims<bf16, float>(bwd, p, d, rot, n, st);
  return ob ? qk_dims<float, bf16>(bwd, p, d, rot, n, st)
            : qk_dims<float, float>(bwd, p, d, rot, n, st);
}

}  // namespace gdn

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == GDN_BF16 || d == GDN_F32; }

constexpr int64_t kMaxLd = (int64_t)1 << 40;

int check_shape(int64_t T, int Hq, int Hk, int d) {
  if (T < 0 || Hq < 0 || Hk < 0 || d <= 0 || (Hq == 0 && Hk == 0)) return GDN_ERR_INVALID_ARG;
  if (d != 64 && d != 128 && d != 256) return GDN_ERR_UNSUPPORTED;
  if (T > INT32_MAX || (int64_t)Hq + Hk > 65535) return GDN_ERR_UNSUPPORTED;
  return GDN_OK;
}

int check_common(int in_dtype, int other_dtype, int64_t T, int Hq, int Hk, int d, int norm,
                 float eps, const float* wq, const float* wk, const int32_t* positions,
                 const float* inv_freq, int rot_dim, int interleaved) {
  if (!valid_dtype(in_dtype) || !valid_dtype(other_dtype) || !(eps > 0.f) || !isfinite(eps) ||
      (norm != GDN_QK_NORM_L2 && norm != GDN_QK_NORM_RMS) || rot_dim < 0 ||
      (interleaved != 0 && interleaved != 1))
    return GDN_ERR_INVALID_ARG;
  const int rc = check_shape(T, Hq, Hk, d);
  if (rc != GDN_OK) return rc;
  if (rot_dim > d) return GDN_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0) return GDN_ERR_UNSUPPORTED;
  if (!aligned(wq, 16) || !aligned(wk, 16)) return GDN_ERR_INVALID_ARG;
  if (rot_dim > 0 && T > 0 &&
      (!positions || !inv_freq || !aligned(positions, 4) || !aligned(inv_freq, 4)))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

int check_heads(const void* p, int64_t ld, int dtype, int H, int d) {
  if (H == 0) return GDN_OK;
  const int per16 = dtype == GDN_BF16 ? 8 : 4;
  if (!p || !aligned(p, 16) || ld < (int64_t)H * d || ld % per16 != 0) return GDN_ERR_INVALID_ARG;
  return ld > kMaxLd ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

int rot_kind(int rot_dim, int interleaved) {
  return rot_dim == 0 ? gdn::kRotNone : interleaved ? gdn::kRotPairs : gdn::kRotHalves;
}

}  // namespace

extern "C" int gdn_qk_norm_forward(const void* q, int64_t ldq, const void* k, int64_t ldk,
                                   int in_dtype, int64_t T, int Hq, int Hk, int d, int norm,
                                   float eps, const float* wq, const float* wk,
                                   const int32_t* positions, const float* inv_freq, int rot_dim,
                                   int interleaved, void* oq, int64_t ldoq, void* ok,
                                   int64_t ldok, int out_dtype, void* stream) {
  int rc = check_common(in_dtype, out_dtype, T, Hq, Hk, d, norm, eps, wq, wk, positions,
                        inv_freq, rot_dim, interleaved);
  if (rc != GDN_OK || T == 0) return rc;
  if ((rc = check_heads(q, ldq, in_dtype, Hq, d)) != GDN_OK) return rc;
  if ((rc = check_heads(k, ldk, in_dtype, Hk, d)) != GDN_OK) return rc;
  if ((rc = check_heads(oq, ldoq, out_dtype, Hq, d)) != GDN_OK) return rc;
  if ((rc = check_heads(ok, ldok, out_dtype, Hk, d)) != GDN_OK) return rc;
  gdn::QkArgs p{};
  p.q.x = q, p.q.ldx = ldq, p.q.w = wq, p.q.y = oq, p.q.ldy = ldoq, p.q.H = Hq;
  p.k.x = k, p.k.ldx = ldk, p.k.w = wk, p.k.y = ok, p.k.ldy = ldok, p.k.H = Hk;
  p.T = T;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.F = rot_dim / 2;
  p.eps = eps;
  p.inv_m = norm == GDN_QK_NORM_RMS ? 1.f / (float)d : 1.f;
  const gdn::QkPlan pl = gdn::qk_plan(T, Hq + Hk, d, false);
  p.tokens = pl.tokens;
  p.span = pl.span;
  return gdn::qk_types(false, p, in_dtype == GDN_BF16, out_dtype == GDN_BF16, d,
                       rot_kind(rot_dim, interleaved), pl.blocks,
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

extern "C" size_t gdn_qk_norm_backward_workspace_bytes(int64_t T, int Hq, int Hk, int d) {
  if (check_shape(T, Hq, Hk, d) != GDN_OK || T == 0) return 0;
  return (size_t)gdn::qk_plan(T, Hq + Hk, d, true).blocks * 2 * d * sizeof(float);
}

extern "C" int gdn_qk_norm_backward(const void* q, int64_t ldq, const void* k, int64_t ldk,
                                    int in_dtype, int64_t T, int Hq, int Hk, int d, int norm,
                                    float eps, const float* wq, const float* wk,
                                    const int32_t* positions, const float* inv_freq, int rot_dim,
                                    int interleaved, const void* d_oq, int64_t lddoq,
                                    const void* d_ok, int64_t lddok, int grad_dtype, void* d_q,
                                    int64_t lddq, void* d_k, int64_t lddk, float* d_wq,
                                    float* d_wk, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  int rc = check_common(in_dtype, grad_dtype, T, Hq, Hk, d, norm, eps, wq, wk, positions,
                        inv_freq, rot_dim, interleaved);
  if (rc != GDN_OK) return rc;
  if ((d_wq && !wq) || (d_wk && !wk) || !aligned(d_wq, 16) || !aligned(d_wk, 16))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    for (float* dw : {d_wq, d_wk})
      if (dw && cudaMemsetAsync(dw, 0, (size_t)d * sizeof(float), st) != cudaSuccess)
        return GDN_ERR_CUDA;
    return GDN_OK;
  }
  if ((rc = check_heads(q, ldq, in_dtype, Hq, d)) != GDN_OK) return rc;
  if ((rc = check_heads(k, ldk, in_dtype, Hk, d)) != GDN_OK) return rc;
  if ((rc = check_heads(d_oq, lddoq, grad_dtype, Hq, d)) != GDN_OK) return rc;
  if ((rc = check_heads(d_ok, lddok, grad_dtype, Hk, d)) != GDN_OK) return rc;
  if ((rc = check_heads(d_q, lddq, in_dtype, Hq, d)) != GDN_OK) return rc;
  if ((rc = check_heads(d_k, lddk, in_dtype, Hk, d)) != GDN_OK) return rc;
  const bool weights = d_wq || d_wk;
  const gdn::QkPlan pl = gdn::qk_plan(T, Hq + Hk, d, weights);
  if (weights) {
    if (!workspace || workspace_bytes < gdn_qk_norm_backward_workspace_bytes(T, Hq, Hk, d))
      return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GDN_ERR_INVALID_ARG;
  }
  gdn::QkArgs p{};
  p.q.x = q, p.q.ldx = ldq, p.q.w = wq, p.q.dy = d_oq, p.q.lddy = lddoq, p.q.dx = d_q;
  p.q.lddx = lddq, p.q.H = Hq;
  p.k.x = k, p.k.ldx = ldk, p.k.w = wk, p.k.dy = d_ok, p.k.lddy = lddok, p.k.dx = d_k;
  p.k.lddx = lddk, p.k.H = Hk;
  p.T = T;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.F = rot_dim / 2;
  p.eps = eps;
  p.inv_m = norm == GDN_QK_NORM_RMS ? 1.f / (float)d : 1.f;
  p.tokens = pl.tokens;
  p.span = pl.span;
  p.partial = weights ? static_cast<float*>(workspace) : nullptr;
  if (gdn::qk_types(true, p, in_dtype == GDN_BF16, grad_dtype == GDN_BF16, d,
                    rot_kind(rot_dim, interleaved), pl.blocks, st) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (weights) {
    gdn::k_qk_weight_sum<<<dim3((unsigned)(d / 32), 2), 256, 0, st>>>(p.partial, (int)pl.blocks,
                                                                      d, d_wq, d_wk);
    if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  }
  return GDN_OK;
}
