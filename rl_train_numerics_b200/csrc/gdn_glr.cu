// gdn_glr.cu -- gated linear recurrence with a vector state (gdn_glr.h).
//
// h_t = a_t h_{t-1} + b_t per channel, a_t = exp(g_t).  One thread holds V
// neighbouring channels of one chunk of 16 tokens; a warp holds 32 V channels
// of a chunk, a block of 8 warps the 8 chunks of a tile of 128 tokens.  For
// every tile a thread
//   1. folds its chunk into (A, B) from A = 1, B = 0 (they do not depend on
//      the state that enters the chunk) and shares them,
//   2. runs the state over the tile's 8 chunks, H <- fma(A_i, H, B_i), and
//      keeps the H that enters its own,
//   3. walks its chunk again and writes h_t = fma(A, H, B).
// The last h of a chunk is the next chunk's H by the same operations, so the
// decode step, which keeps (H, A, B), has the forward's bits.  Every channel's
// operations are those of its own sequence in order, so nothing depends on
// the batch, on V or on how tiles are spread over blocks.
//
// Tokens behind a sequence's end are identity steps (a = 1, b = 0), which
// leave A, B and H as they are, bit for bit.
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/gdn_glr.h"
#include "gdn_common.cuh"

namespace gdn {

constexpr int kGlrChunk = GDN_GLR_CHUNK;
constexpr int kGlrWarps = 8;
constexpr int kGlrThreads = 32 * kGlrWarps;
constexpr int kGlrTile = kGlrChunk * kGlrWarps;
static_assert(kGlrTile == GDN_GLR_TILE, "carry rows are tile starts");

// V consecutive elements as loaded, all-zero bits for masked ones.
template <class T, int V>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 1> {
  using type = unsigned short;
};
template <>
struct Raw<__nv_bfloat16, 2> {
  using type = unsigned;
};
template <>
struct Raw<float, 1> {
  using type = float;
};
template <>
struct Raw<float, 2> {
  using type = float2;
};

__device__ __forceinline__ void raw_zero(unsigned short& r) { r = 0; }
__device__ __forceinline__ void raw_zero(unsigned& r) { r = 0u; }
__device__ __forceinline__ void raw_zero(float& r) { r = 0.f; }
__device__ __forceinline__ void raw_zero(float2& r) { r = make_float2(0.f, 0.f); }
__device__ __forceinline__ void widen(unsigned short r, float (&f)[1]) {
  f[0] = __uint_as_float((unsigned)r << 16);
}
__device__ __forceinline__ void widen(unsigned r, float (&f)[2]) {
  f[0] = __uint_as_float(r << 16);
  f[1] = __uint_as_float(r & 0xffff0000u);
}
__device__ __forceinline__ void widen(float r, float (&f)[1]) { f[0] = r; }
__device__ __forceinline__ void widen(float2 r, float (&f)[2]) {
  f[0] = r.x;
  f[1] = r.y;
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&f)[1]) {
  *p = __float2bfloat16_rn(f[0]);
}
__device__ __forceinline__ void put(__nv_bfloat16* p, const float (&f)[2]) {
  *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
}
__device__ __forceinline__ void put(float* p, const float (&f)[1]) { *p = f[0]; }
__device__ __forceinline__ void put(float* p, const float (&f)[2]) {
  *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
}
template <class T, int V>
__device__ __forceinline__ typename Raw<T, V>::type raw_load(const T* p) {
  return *reinterpret_cast<const typename Raw<T, V>::type*>(p);
}

// The gate of one token: a thread keeps one float `w` of it, from which the
// decay a and the input b come.  PLAIN: w = a.  COMPLEMENT needs a and 1 - a,
// each with its own relative accuracy: a decay below exp(-1/2) is kept as a
// (1 - a loses nothing there), the others as e = expm1(g), with a = 1 + e and
// 1 - a = -e; bit `i` of `low` says which.
template <int MODE>
__device__ __forceinline__ float gate_of(float g, unsigned& low, int i) {
  if (MODE == GDN_GLR_INPUT_PLAIN) return expf(g);
  const bool decayed = g < -0.5f;
  low |= (unsigned)decayed << i;
  return decayed ? expf(g) : expm1f(g);
}
template <int MODE>
__device__ __forceinline__ float gate_a(float w, unsigned low, int i) {
  if (MODE == GDN_GLR_INPUT_PLAIN) return w;
  return low >> i & 1 ? w : __fadd_rn(1.f, w);
}
template <int MODE>
__device__ __forceinline__ float gate_b(float w, unsigned low, int i, float x) {
  if (MODE == GDN_GLR_INPUT_PLAIN) return x;
  return __fmul_rn(low >> i & 1 ? __fsub_rn(1.f, w) : -w, x);
}

struct GlrArgs {
  const void* x;
  const void* g;
  int64_t ldx, ldg;
  const int32_t* cu;
  int N;
  int64_t T;
  int D, slabs;
  const float* h0;  // forward
  void* h;
  int64_t ldh;
  float* s_final;
  gdn_glr_state st;  // st.h == nullptr: none
  const int32_t* slot_idx;
  float* carry;
  const void* d_h;  // backward
  int64_t lddh;
  const float* ds_final;
  void* d_x;
  int64_t lddx;
  void* d_g;
  int64_t lddg;
  float* d_h0;
  int32_t* error;
};

__device__ __forceinline__ bool glr_seq_ok(const GlrArgs& p, int n) {
  return p.cu[0] == 0 && (int64_t)p.cu[p.N] == p.T && p.cu[n] >= 0 && p.cu[n + 1] >= p.cu[n] &&
         (int64_t)p.cu[n + 1] <= p.T;
}

// Slot of row n, or -1 when it is out of range or an earlier row has it too
// (the whole block calls this; every thread gets the answer).
__device__ __forceinline__ int glr_slot(const int32_t* slot_idx, int n, int n_slots) {
  if (!slot_idx) return n < n_slots ? n : -1;
  const int slot = slot_idx[n];
  int twice = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) twice |= slot_idx[i] == slot;
  twice = __syncthreads_or(twice);
  return slot >= 0 && slot < n_slots && !twice ? slot : -1;
}

template <int V>
__device__ __forceinline__ void row_get(const float* base, int64_t row, int D, int ch, bool live,
                                        float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; v++) f[v] = 0.f;
  if (base && live) {
#pragma unroll
    for (int v = 0; v < V; v++) f[v] = base[row * D + ch + v];
  }
}

// One block per (sequence, slab of 32 V channels).
template <class IN, class G, class OUT, int V, int MODE>
__global__ void __launch_bounds__(kGlrThreads) k_glr_forward(const GlrArgs p) {
  __shared__ float sA[2][kGlrWarps][32 * V], sB[2][kGlrWarps][32 * V];
  const int n = blockIdx.x / p.slabs, slab = blockIdx.x % p.slabs;
  if (!glr_seq_ok(p, n)) {
    if (threadIdx.x == 0 && p.error) atomicOr(p.error, kErrCuSeqlens);
    return;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ch = (slab * 32 + lane) * V;
  const bool live = ch < p.D;
  const int64_t L = (int64_t)p.cu[n + 1] - p.cu[n];
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)p.cu[n] * p.ldx + ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)p.cu[n] * p.ldg + ch;
  OUT* h = static_cast<OUT*>(p.h) + (int64_t)p.cu[n] * p.ldh + ch;
  float* carry = p.carry ? p.carry + ((int64_t)p.cu[n] / kGlrTile + n) * p.D + ch : nullptr;

  float H[V], Hm[V], A[V], B[V], hv[V];
  row_get<V>(p.h0, n, p.D, ch, live, H);
#pragma unroll
  for (int v = 0; v < V; v++) {
    Hm[v] = hv[v] = H[v];
    A[v] = 1.f;
    B[v] = 0.f;
  }
  const int64_t ntiles = (L + kGlrTile - 1) / kGlrTile;
  for (int64_t s = 0; s < ntiles; s++) {
    const int64_t t0 = s * kGlrTile + w * kGlrChunk;
    typename Raw<IN, V>::type rx[kGlrChunk];
    float ga[kGlrChunk][V];
    unsigned low = 0;
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      typename Raw<G, V>::type rg;
      raw_zero(rx[t]);
      raw_zero(rg);
      if (live && t0 + t < L) {
        rx[t] = raw_load<IN, V>(x + (t0 + t) * p.ldx);
        rg = raw_load<G, V>(g + (t0 + t) * p.ldg);
      }
      widen(rg, ga[t]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
      A[v] = 1.f;
      B[v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      float xv[V];
      widen(rx[t], xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        ga[t][v] = gate_of<MODE>(ga[t][v], low, t * V + v);
        const float a = gate_a<MODE>(ga[t][v], low, t * V + v);
        A[v] = __fmul_rn(a, A[v]);
        B[v] = __fmaf_rn(a, B[v], gate_b<MODE>(ga[t][v], low, t * V + v, xv[v]));
      }
    }
    // Two buffers: a thread writes one again only behind the other's barrier,
    // which every thread reaches after its reads of the first.
#pragma unroll
    for (int v = 0; v < V; v++) {
      sA[s & 1][w][lane * V + v] = A[v];
      sB[s & 1][w][lane * V + v] = B[v];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kGlrWarps; i++)
#pragma unroll
      for (int v = 0; v < V; v++) {
        if (i == w) Hm[v] = H[v];
        H[v] = __fmaf_rn(sA[s & 1][i][lane * V + v], H[v], sB[s & 1][i][lane * V + v]);
      }
    if (carry && live && w == 0) put(carry + s * p.D, Hm);
    if (!live || t0 >= L) continue;
#pragma unroll
    for (int v = 0; v < V; v++) {
      A[v] = 1.f;
      B[v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      float xv[V];
      widen(rx[t], xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        const float a = gate_a<MODE>(ga[t][v], low, t * V + v);
        A[v] = __fmul_rn(a, A[v]);
        B[v] = __fmaf_rn(a, B[v], gate_b<MODE>(ga[t][v], low, t * V + v, xv[v]));
        hv[v] = __fmaf_rn(A[v], Hm[v], B[v]);
      }
      if (t0 + t < L) put(h + (t0 + t) * p.ldh, hv);
    }
  }
  // The warp that holds the last token has its h and the chunk's (Hm, A, B).
  const int last_w = L > 0 ? (int)((L - 1) / kGlrChunk % kGlrWarps) : 0;
  if (p.s_final && live && w == last_w) put(p.s_final + (int64_t)n * p.D + ch, hv);
  if (p.st.h) {
    const int slot = glr_slot(p.slot_idx, n, p.st.n_slots);
    const int pos = (int)(L % kGlrChunk);
    if (slot < 0) {
      if (threadIdx.x == 0) atomicOr(p.st.error, kErrPos);
      return;
    }
    if (slab == 0 && threadIdx.x == 0) p.st.pos[slot] = pos;
    if (live && w == last_w) {
      const float one[2] = {1.f, 1.f}, zero[2] = {0.f, 0.f};
      const int64_t at = (int64_t)slot * p.D + ch;
#pragma unroll
      for (int v = 0; v < V; v++) {
        p.st.h[at + v] = pos ? Hm[v] : hv[v];
        p.st.a[at + v] = pos ? A[v] : one[v];
        p.st.b[at + v] = pos ? B[v] : zero[v];
      }
    }
  }
}

// Reverse mode: tiles from a sequence's last to its first.  A chunk's map of
// the adjoint mu is mu -> fma(A, mu, M) with the A of the forward and M its
// value from mu = 0, so the chunks of a tile are again evaluated side by
// side; h_{t-1} comes from the tile's carry row and the chunks' (A, B) by the
// forward's operations.
template <class IN, class G, class OUT, int V, int MODE>
__global__ void __launch_bounds__(kGlrThreads) k_glr_backward(const GlrArgs p) {
  __shared__ float sA[2][kGlrWarps][32 * V], sB[2][kGlrWarps][32 * V], sM[2][kGlrWarps][32 * V];
  const int n = blockIdx.x / p.slabs, slab = blockIdx.x % p.slabs;
  if (!glr_seq_ok(p, n)) {
    if (threadIdx.x == 0 && p.error) atomicOr(p.error, kErrCuSeqlens);
    return;
  }
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int ch = (slab * 32 + lane) * V;
  const bool live = ch < p.D;
  const int64_t L = (int64_t)p.cu[n + 1] - p.cu[n];
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)p.cu[n] * p.ldx + ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)p.cu[n] * p.ldg + ch;
  const OUT* dh = static_cast<const OUT*>(p.d_h) + (int64_t)p.cu[n] * p.lddh + ch;
  IN* dx = static_cast<IN*>(p.d_x) + (int64_t)p.cu[n] * p.lddx + ch;
  G* dg = static_cast<G*>(p.d_g) + (int64_t)p.cu[n] * p.lddg + ch;
  const int64_t row0 = (int64_t)p.cu[n] / kGlrTile + n;

  float mu[V];
  row_get<V>(p.ds_final, n, p.D, ch, live, mu);
  const int64_t ntiles = (L + kGlrTile - 1) / kGlrTile;
  for (int64_t s = ntiles - 1; s >= 0; s--) {
    const int64_t t0 = s * kGlrTile + w * kGlrChunk;
    typename Raw<IN, V>::type rx[kGlrChunk];
    typename Raw<OUT, V>::type rd[kGlrChunk];
    float ga[kGlrChunk][V], H[V], Hm[V], A[V], B[V], M[V];
    unsigned low = 0;
    row_get<V>(p.carry, row0 + s, p.D, ch, live, H);
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      typename Raw<G, V>::type rg;
      raw_zero(rx[t]);
      raw_zero(rd[t]);
      raw_zero(rg);
      if (live && t0 + t < L) {
        rx[t] = raw_load<IN, V>(x + (t0 + t) * p.ldx);
        rd[t] = raw_load<OUT, V>(dh + (t0 + t) * p.lddh);
        rg = raw_load<G, V>(g + (t0 + t) * p.ldg);
      }
      widen(rg, ga[t]);
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
      A[v] = 1.f;
      B[v] = M[v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      float xv[V];
      widen(rx[t], xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        ga[t][v] = gate_of<MODE>(ga[t][v], low, t * V + v);
        const float a = gate_a<MODE>(ga[t][v], low, t * V + v);
        A[v] = __fmul_rn(a, A[v]);
        B[v] = __fmaf_rn(a, B[v], gate_b<MODE>(ga[t][v], low, t * V + v, xv[v]));
      }
    }
#pragma unroll
    for (int t = kGlrChunk - 1; t >= 0; t--) {
      float dv[V];
      widen(rd[t], dv);
#pragma unroll
      for (int v = 0; v < V; v++)
        M[v] = __fmul_rn(gate_a<MODE>(ga[t][v], low, t * V + v), __fadd_rn(dv[v], M[v]));
    }
#pragma unroll
    for (int v = 0; v < V; v++) {
      sA[s & 1][w][lane * V + v] = A[v];
      sB[s & 1][w][lane * V + v] = B[v];
      sM[s & 1][w][lane * V + v] = M[v];
    }
    __syncthreads();
    float mm[V];
#pragma unroll
    for (int i = 0; i < kGlrWarps; i++)
#pragma unroll
      for (int v = 0; v < V; v++) {
        if (i == w) Hm[v] = H[v];
        H[v] = __fmaf_rn(sA[s & 1][i][lane * V + v], H[v], sB[s & 1][i][lane * V + v]);
      }
#pragma unroll
    for (int i = kGlrWarps - 1; i >= 0; i--)
#pragma unroll
      for (int v = 0; v < V; v++) {
        if (i == w) mm[v] = mu[v];
        mu[v] = __fmaf_rn(sA[s & 1][i][lane * V + v], mu[v], sM[s & 1][i][lane * V + v]);
      }
    if (!live || t0 >= L) continue;
    float hp[kGlrChunk][V];  // h_{t-1}
#pragma unroll
    for (int v = 0; v < V; v++) {
      A[v] = 1.f;
      B[v] = 0.f;
    }
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) {
      float xv[V];
      widen(rx[t], xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        hp[t][v] = __fmaf_rn(A[v], Hm[v], B[v]);
        const float a = gate_a<MODE>(ga[t][v], low, t * V + v);
        A[v] = __fmul_rn(a, A[v]);
        B[v] = __fmaf_rn(a, B[v], gate_b<MODE>(ga[t][v], low, t * V + v, xv[v]));
      }
    }
#pragma unroll
    for (int t = kGlrChunk - 1; t >= 0; t--) {
      float dv[V], xv[V], ox[V], og[V];
      widen(rd[t], dv);
      widen(rx[t], xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        const float lam = __fadd_rn(dv[v], mm[v]);
        mm[v] = __fmul_rn(gate_a<MODE>(ga[t][v], low, t * V + v), lam);
        ox[v] = gate_b<MODE>(ga[t][v], low, t * V + v, lam);
        og[v] = __fmul_rn(mm[v], MODE == GDN_GLR_INPUT_COMPLEMENT ? __fsub_rn(hp[t][v], xv[v])
                                                                  : hp[t][v]);
      }
      if (t0 + t < L) {
        put(dx + (t0 + t) * p.lddx, ox);
        put(dg + (t0 + t) * p.lddg, og);
      }
    }
  }
  if (p.d_h0 && live && w == 0) put(p.d_h0 + (int64_t)n * p.D + ch, mu);
}

// One block per row (a row's pos is read and written by one block).
constexpr int kGlrStepThreads = 1024;

template <class IN, class G, class OUT, int V, int MODE>
__global__ void __launch_bounds__(kGlrStepThreads) k_glr_step(const GlrArgs p) {
  const int b = blockIdx.x;
  const int slot = glr_slot(p.slot_idx, b, p.st.n_slots);
  const int pos = slot < 0 ? -1 : p.st.pos[slot];
  if (pos < 0 || pos >= kGlrChunk) {
    if (threadIdx.x == 0) atomicOr(p.st.error, kErrPos);
    return;
  }
  __syncthreads();  // every thread has read pos
  const bool full = pos == kGlrChunk - 1;
  if (threadIdx.x == 0) p.st.pos[slot] = full ? 0 : pos + 1;
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)b * p.ldx;
  const G* g = static_cast<const G*>(p.g) + (int64_t)b * p.ldg;
  OUT* h = static_cast<OUT*>(p.h) + (int64_t)b * p.ldh;
  const int64_t base = (int64_t)slot * p.D;
  for (int ch = threadIdx.x * V; ch < p.D; ch += kGlrStepThreads * V) {
    float xv[V], gv[V], H[V], A[V], B[V], hv[V];
    widen(raw_load<IN, V>(x + ch), xv);
    widen(raw_load<G, V>(g + ch), gv);
    widen(raw_load<float, V>(p.st.h + base + ch), H);
    widen(raw_load<float, V>(p.st.a + base + ch), A);
    widen(raw_load<float, V>(p.st.b + base + ch), B);
#pragma unroll
    for (int v = 0; v < V; v++) {
      unsigned low = 0;
      const float wv = gate_of<MODE>(gv[v], low, 0), a = gate_a<MODE>(wv, low, 0);
      A[v] = __fmul_rn(a, pos ? A[v] : 1.f);
      B[v] = __fmaf_rn(a, pos ? B[v] : 0.f, gate_b<MODE>(wv, low, 0, xv[v]));
      hv[v] = __fmaf_rn(A[v], H[v], B[v]);
      if (full) {
        A[v] = 1.f;
        B[v] = 0.f;
      }
    }
    put(h + ch, hv);
    if (full) put(p.st.h + base + ch, hv);
    put(p.st.a + base + ch, A);
    put(p.st.b + base + ch, B);
  }
}

// ----------------------------------------------------------------------------
// Launchers
// ----------------------------------------------------------------------------
enum GlrOp { kGlrFwd, kGlrBwd, kGlrStep };

template <class IN, class G, class OUT, int V, int MODE>
static cudaError_t glr_launch(GlrOp op, GlrArgs& p, cudaStream_t st) {
  p.slabs = (p.D + 32 * V - 1) / (32 * V);
  if (op == kGlrStep) {
    k_glr_step<IN, G, OUT, V, MODE><<<(unsigned)p.N, kGlrStepThreads, 0, st>>>(p);
  } else {
    const unsigned blocks = (unsigned)p.N * (unsigned)p.slabs;
    if (op == kGlrFwd)
      k_glr_forward<IN, G, OUT, V, MODE><<<blocks, kGlrThreads, 0, st>>>(p);
    else
      k_glr_backward<IN, G, OUT, V, MODE><<<blocks, kGlrThreads, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <class IN, class G, class OUT>
static cudaError_t glr_modes(GlrOp op, GlrArgs& p, bool pairs, int mode, cudaStream_t st) {
  if (mode == GDN_GLR_INPUT_PLAIN)
    return pairs ? glr_launch<IN, G, OUT, 2, GDN_GLR_INPUT_PLAIN>(op, p, st)
                 : glr_launch<IN, G, OUT, 1, GDN_GLR_INPUT_PLAIN>(op, p, st);
  return pairs ? glr_launch<IN, G, OUT, 2, GDN_GLR_INPUT_COMPLEMENT>(op, p, st)
               : glr_launch<IN, G, OUT, 1, GDN_GLR_INPUT_COMPLEMENT>(op, p, st);
}

static cudaError_t glr_types(GlrOp op, GlrArgs& p, bool ib, bool gb, bool ob, bool pairs,
                             int mode, cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  if (ib) {
    if (gb)
      return ob ? glr_modes<bf16, bf16, bf16>(op, p, pairs, mode, st)
                : glr_modes<bf16, bf16, float>(op, p, pairs, mode, st);
    return ob ? glr_modes<bf16, float, bf16>(op, p, pairs, mode, st)
              : glr_modes<bf16, float, float>(op, p, pairs, mode, st);
  }
  if (gb)
    return ob ? glr_modes<float, bf16, bf16>(op, p, pairs, mode, st)
              : glr_modes<float, bf16, float>(op, p, pairs, mode, st);
  return ob ? glr_modes<float, float, bf16>(op, p, pairs, mode, st)
            : glr_modes<float, float, float>(op, p, pairs, mode, st);
}

}  // namespace gdn

namespace {

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int d) { return d == GDN_BF16 || d == GDN_F32; }
size_t size_of(int dtype) { return dtype == GDN_BF16 ? 2 : 4; }

constexpr int kMaxD = 1 << 24;
constexpr int64_t kMaxLd = (int64_t)1 << 40;  // rows x stride stays far inside 64 bits

// One strided matrix: present, element-aligned, stride in range.
int check_rows(const void* p, int64_t ld, int dtype, int D) {
  if (!p || !aligned(p, size_of(dtype)) || ld < D) return GDN_ERR_INVALID_ARG;
  return ld > kMaxLd ? GDN_ERR_UNSUPPORTED : GDN_OK;
}
// Whether its rows can be read two elements at a time.
bool paired(const void* p, int64_t ld, int dtype) {
  return aligned(p, 2 * size_of(dtype)) && ld % 2 == 0;
}

int check_sizes(int in_dtype, int g_dtype, int other_dtype, int D, int mode) {
  if (!valid_dtype(in_dtype) || !valid_dtype(g_dtype) || !valid_dtype(other_dtype) || D <= 0 ||
      (mode != GDN_GLR_INPUT_PLAIN && mode != GDN_GLR_INPUT_COMPLEMENT))
    return GDN_ERR_INVALID_ARG;
  return D > kMaxD ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

int check_state(const gdn_glr_state& st) {
  if (st.n_slots <= 0 || !st.h || !st.a || !st.b || !st.pos || !st.error)
    return GDN_ERR_INVALID_ARG;
  if (!aligned(st.h, 16) || !aligned(st.a, 16) || !aligned(st.b, 16) || !aligned(st.pos, 4) ||
      !aligned(st.error, 4))
    return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

// Checks shared by forward and backward.
int check_batch(const int32_t* cu, int n_seqs, int64_t T, int D, const int32_t* error_word) {
  if (n_seqs < 0 || T < 0 || !aligned(error_word, 4)) return GDN_ERR_INVALID_ARG;
  if (T > INT32_MAX) return GDN_ERR_UNSUPPORTED;
  if (n_seqs == 0) return T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu || !aligned(cu, 4)) return GDN_ERR_INVALID_ARG;
  const int64_t blocks = (int64_t)n_seqs * ((D + 31) / 32);
  return blocks > INT32_MAX ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace

extern "C" int64_t gdn_glr_carry_rows(int n_seqs, int64_t total_tokens) {
  if (n_seqs < 0 || total_tokens < 0 || total_tokens > INT32_MAX) return 0;
  return total_tokens / GDN_GLR_TILE + n_seqs;
}

extern "C" int gdn_glr_forward(const void* x, int64_t ldx, int in_dtype, const void* g,
                               int64_t ldg, int g_dtype, const int32_t* cu_seqlens, int n_seqs,
                               int64_t total_tokens, int D, int input_mode, const float* h0,
                               void* h, int64_t ldh, int out_dtype, float* s_final,
                               const gdn_glr_state* state, const int32_t* slot_idx, float* carry,
                               int32_t* error_word, void* stream) {
  int rc = check_sizes(in_dtype, g_dtype, out_dtype, D, input_mode);
  if (rc == GDN_OK) rc = check_batch(cu_seqlens, n_seqs, total_tokens, D, error_word);
  if (rc != GDN_OK) return rc;
  bool pairs = D % 2 == 0;
  if (total_tokens > 0) {
    if ((rc = check_rows(x, ldx, in_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(g, ldg, g_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(h, ldh, out_dtype, D)) != GDN_OK) return rc;
    pairs = pairs && paired(x, ldx, in_dtype) && paired(g, ldg, g_dtype) &&
            paired(h, ldh, out_dtype);
  }
  if (!aligned(h0, 16) || !aligned(s_final, 16) || !aligned(carry, 16) || !aligned(slot_idx, 4))
    return GDN_ERR_INVALID_ARG;
  if (slot_idx && !state) return GDN_ERR_INVALID_ARG;
  if (state) {
    if ((rc = check_state(*state)) != GDN_OK) return rc;
    if (!slot_idx && n_seqs > state->n_slots) return GDN_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (error_word && cudaMemsetAsync(error_word, 0, sizeof(int32_t), st) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (n_seqs == 0) return GDN_OK;
  gdn::GlrArgs p{};
  p.x = x;
  p.g = g;
  p.ldx = ldx;
  p.ldg = ldg;
  p.cu = cu_seqlens;
  p.N = n_seqs;
  p.T = total_tokens;
  p.D = D;
  p.h0 = h0;
  p.h = h;
  p.ldh = ldh;
  p.s_final = s_final;
  if (state) p.st = *state;
  p.slot_idx = slot_idx;
  p.carry = carry;
  p.error = error_word;
  return gdn::glr_types(gdn::kGlrFwd, p, in_dtype == GDN_BF16, g_dtype == GDN_BF16,
                        out_dtype == GDN_BF16, pairs, input_mode, st) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

extern "C" int gdn_glr_backward(const void* x, int64_t ldx, int in_dtype, const void* g,
                                int64_t ldg, int g_dtype, const int32_t* cu_seqlens, int n_seqs,
                                int64_t total_tokens, int D, int input_mode, const float* carry,
                                const void* d_h, int64_t lddh, int dh_dtype,
                                const float* ds_final, void* d_x, int64_t lddx, void* d_g,
                                int64_t lddg, float* d_h0, int32_t* error_word, void* stream) {
  int rc = check_sizes(in_dtype, g_dtype, dh_dtype, D, input_mode);
  if (rc == GDN_OK) rc = check_batch(cu_seqlens, n_seqs, total_tokens, D, error_word);
  if (rc != GDN_OK) return rc;
  bool pairs = D % 2 == 0;
  if (total_tokens > 0) {
    if ((rc = check_rows(x, ldx, in_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(g, ldg, g_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(d_h, lddh, dh_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(d_x, lddx, in_dtype, D)) != GDN_OK) return rc;
    if ((rc = check_rows(d_g, lddg, g_dtype, D)) != GDN_OK) return rc;
    if (!carry) return GDN_ERR_INVALID_ARG;
    pairs = pairs && paired(x, ldx, in_dtype) && paired(g, ldg, g_dtype) &&
            paired(d_h, lddh, dh_dtype) && paired(d_x, lddx, in_dtype) &&
            paired(d_g, lddg, g_dtype);
  }
  if (!aligned(carry, 16) || !aligned(ds_final, 16) || !aligned(d_h0, 16))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (error_word && cudaMemsetAsync(error_word, 0, sizeof(int32_t), st) != cudaSuccess)
    return GDN_ERR_CUDA;
  if (n_seqs == 0) return GDN_OK;
  gdn::GlrArgs p{};
  p.x = x;
  p.g = g;
  p.ldx = ldx;
  p.ldg = ldg;
  p.cu = cu_seqlens;
  p.N = n_seqs;
  p.T = total_tokens;
  p.D = D;
  p.carry = const_cast<float*>(carry);
  p.d_h = d_h;
  p.lddh = lddh;
  p.ds_final = ds_final;
  p.d_x = d_x;
  p.lddx = lddx;
  p.d_g = d_g;
  p.lddg = lddg;
  p.d_h0 = d_h0;
  p.error = error_word;
  return gdn::glr_types(gdn::kGlrBwd, p, in_dtype == GDN_BF16, g_dtype == GDN_BF16,
                        dh_dtype == GDN_BF16, pairs, input_mode, st) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

extern "C" int gdn_glr_decode_step(const void* x, int64_t ldx, int in_dtype, const void* g,
                                   int64_t ldg, int g_dtype, const int32_t* slot_idx, int B,
                                   int D, int input_mode, gdn_glr_state state, void* h,
                                   int64_t ldh, int out_dtype, void* stream) {
  int rc = check_sizes(in_dtype, g_dtype, out_dtype, D, input_mode);
  if (rc != GDN_OK) return rc;
  if (B < 0) return GDN_ERR_INVALID_ARG;
  if (B == 0) return GDN_OK;
  if ((rc = check_state(state)) != GDN_OK) return rc;
  if ((rc = check_rows(x, ldx, in_dtype, D)) != GDN_OK) return rc;
  if ((rc = check_rows(g, ldg, g_dtype, D)) != GDN_OK) return rc;
  if ((rc = check_rows(h, ldh, out_dtype, D)) != GDN_OK) return rc;
  if (!aligned(slot_idx, 4)) return GDN_ERR_INVALID_ARG;
  if (!slot_idx && B > state.n_slots) return GDN_ERR_INVALID_ARG;
  const bool pairs = D % 2 == 0 && paired(x, ldx, in_dtype) && paired(g, ldg, g_dtype) &&
                     paired(h, ldh, out_dtype);
  gdn::GlrArgs p{};
  p.x = x;
  p.g = g;
  p.ldx = ldx;
  p.ldg = ldg;
  p.N = B;
  p.D = D;
  p.h = h;
  p.ldh = ldh;
  p.st = state;
  p.slot_idx = slot_idx;
  return gdn::glr_types(gdn::kGlrStep, p, in_dtype == GDN_BF16, g_dtype == GDN_BF16,
                        out_dtype == GDN_BF16, pairs, input_mode,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}
