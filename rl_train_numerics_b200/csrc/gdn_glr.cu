// gdn_glr.cu -- gated linear recurrence with a vector state (gdn_glr.h).
//
// h_t = a_t h_{t-1} + b_t per channel, a_t = exp(g_t).  A block takes a slab of
// 32 channels of one sequence and walks it in tiles of 128 tokens, 8 chunks of
// 16; one thread holds V neighbouring channels of one chunk.  For every tile
//   1. a thread folds its chunk into the maps (A_t, B_t) from A = 1, B = 0,
//      which do not depend on the state that enters the chunk, and shares the
//      last of them;
//   2. one warp runs the state over the chunks, H <- fma(A, H, B), a lane per
//      channel;
//   3. a thread writes h_t = fma(A_t, H, B_t) of its chunk.
// The last h of a chunk is the next chunk's H by the same operations, so the
// decode step, which keeps (H, A, B), has the forward's bits.  Every channel's
// operations are those of its own sequence in order, so nothing depends on
// the batch, on V or on how tiles are spread over blocks.  Tokens behind a
// sequence's end are identity steps (a = 1, b = -0), which leave A, B and H as
// they are, the sign of a zero included.
//
// Few sequences of few channels would leave most of the device idle: then a
// cluster of 2, 4 or 8 blocks takes as many neighbouring tiles at a time, every
// block writes its chunks' maps into all blocks' shared memory, and each runs
// the state over all of them.  The data are still read once.
//
// What bounds it is memory: 8 bytes an element forward (bf16 x and h, fp32 g) and
// 14 backward, for 21 and 33 instructions per 32 elements.  16384 x 2048 in 32
// sequences: 48 us (5.5 TB/s) and 78 us (6.0 TB/s, of 6.5 that a copy reaches);
// 57344 x 4096 in 64 uneven ones: 300 and 574 us (6.3 and 5.7 TB/s).  A sequence
// alone is bound by its steps, one after the other: 65536 x 2048 with bf16 gates
// takes 181 and 263 us (4.4 and 5.1 TB/s), 32768 x 1024 73 and 119.  Chunks of 16
// tokens keep the maps of two channels (64 floats) in a thread's registers from
// the fold to the write, at three blocks of a multiprocessor; slabs of 32
// channels make a token's row of a box a whole 128-byte line of fp32.
#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/gdn_glr.h"
#include "gdn_common.cuh"
#include "gdn_mma.cuh"
#include "gdn_tmap.h"
#include "gdn_umma.cuh"

namespace gdn {

namespace cg = cooperative_groups;

constexpr int kGlrChunk = GDN_GLR_CHUNK;
constexpr int kGlrChunks = 8;   // chunks of a tile
constexpr int kGlrTile = kGlrChunk * kGlrChunks;
constexpr int kGlrSlab = 32;    // channels of a block
constexpr int kGlrMaxStages = 8;
constexpr int kGlrPolls = 1 << 22;
// Blocks of a multiprocessor that a kernel's registers leave room for.
template <int V>
__host__ __device__ constexpr int glr_blocks(bool forward) {
  return V == 1 ? (forward ? 2 : 1) : 3;
}
template <int V>
constexpr int kGlrThreads = kGlrChunks * kGlrSlab / V;  // that compute
template <int V>
constexpr int kGlrBlock = kGlrThreads<V> + 32;  // and the service warp
static_assert(kGlrTile == GDN_GLR_TILE, "carry rows are tile starts");

// V consecutive elements as loaded, zeros for masked ones.
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

__device__ __forceinline__ void raw_zero(unsigned short& r, bool minus) { r = minus ? 0x8000 : 0; }
__device__ __forceinline__ void raw_zero(unsigned& r, bool minus) { r = minus ? 0x80008000u : 0u; }
__device__ __forceinline__ void raw_zero(float& r, bool minus) { r = minus ? -0.f : 0.f; }
__device__ __forceinline__ void raw_zero(float2& r, bool minus) {
  r.x = r.y = minus ? -0.f : 0.f;
}
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

// a = exp(g).  Far from 0 as 2^(g log2 e) by ex2.approx: a relative error of at
// most 2^-22 = 4 U (U = 2^-24), with |g| U for the rounded product and |g| U / 4
// for the rounded constant.  A state is a sum of inputs weighted by products of
// decays; where every |g| is at least 1/8, those errors change it by at most
// (4 U + 1.25 |g| U) / (1 - a) < 36 U.  -inf gives 0, a NaN stays one.
__device__ __forceinline__ float decay_far(float g) {
  float a;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(__fmul_rn(g, 1.4426950408889634f)));
  return a;
}
// a for |g| < 1/8: the Taylor series to g^5 / 5!.  A slow gate's error is not
// washed out by its own decay: a state that lives 1 / |g| tokens takes it up
// as often.  Here the rest of the series is 0.1 U of a, a product with |g| < 1/8
// scales down the roundings before the last, and the last is half a step: 0.8 U
// below 1 (1.4 U above), and half a step alone for g towards 0, without a bias
// (ex2.approx: 2.3 U and a bias of -0.3 U measured over [-1/2, 0], expf 2.3 and
// +0.2).  Two gates at a time, packed: forward and backward of 65536 x 2048
// alone 444 us (430 without it), of 10240 x 2048 in 5 uneven sequences 95 (92).
// expf, exact to 2 U everywhere, takes 490 and 98.
__device__ __forceinline__ float2 decay_near(float2 g) {
  float2 s = f2(1.f / 120.f, 1.f / 120.f);
  s = __ffma2_rn(s, g, f2(1.f / 24.f, 1.f / 24.f));
  s = __ffma2_rn(s, g, f2(1.f / 6.f, 1.f / 6.f));
  s = __ffma2_rn(s, g, f2(0.5f, 0.5f));
  s = __ffma2_rn(s, g, f2(1.f, 1.f));
  return __ffma2_rn(s, g, f2(1.f, 1.f));
}
// exp(g) - 1 for |g| <= 1/2: the Taylor series to g^8 / 8! (the rest is below
// 2^-26 of it).
__device__ __forceinline__ float2 decay_m1(float2 g) {
  float2 s = f2(1.f / 40320.f, 1.f / 40320.f);
  s = __ffma2_rn(s, g, f2(1.f / 5040.f, 1.f / 5040.f));
  s = __ffma2_rn(s, g, f2(1.f / 720.f, 1.f / 720.f));
  s = __ffma2_rn(s, g, f2(1.f / 120.f, 1.f / 120.f));
  s = __ffma2_rn(s, g, f2(1.f / 24.f, 1.f / 24.f));
  s = __ffma2_rn(s, g, f2(1.f / 6.f, 1.f / 6.f));
  s = __ffma2_rn(s, g, f2(0.5f, 0.5f));
  s = __ffma2_rn(s, g, f2(1.f, 1.f));
  return __fmul2_rn(s, g);
}

// Two gates: a thread keeps one float `w` of each, from which the decay a and
// the input b come.  PLAIN: w = a.  COMPLEMENT needs a and 1 - a, each with its
// own relative accuracy: for |g| < 1/2 it keeps e = exp(g) - 1, with a = 1 + e and
// 1 - a = -e, for the others a (1 - a loses little there); bits `i` and `i + 1` of
// `far` say which.  Both forms are computed: a branch for each gate costs far more.
template <int MODE>
__device__ __forceinline__ void gates_of(const float (&g)[2], float (&w)[2], unsigned& far,
                                         int i) {
  constexpr bool kPlain = MODE == GDN_GLR_INPUT_PLAIN;
  const float2 both = f2(g[0], g[1]), near2 = kPlain ? decay_near(both) : decay_m1(both);
  const float near[2] = {near2.x, near2.y};
#pragma unroll
  for (int v = 0; v < 2; v++) {
    const bool is_far = !(fabsf(g[v]) < (kPlain ? 0.125f : 0.5f));
    if (!kPlain) far |= (unsigned)is_far << (i + v);
    const float a = decay_far(g[v]);
    w[v] = is_far ? a : near[v];
  }
}
template <int MODE>
__device__ __forceinline__ float gate_a(float w, unsigned far, int i) {
  if (MODE == GDN_GLR_INPUT_PLAIN) return w;
  return far >> i & 1 ? w : __fadd_rn(1.f, w);
}
template <int MODE>
__device__ __forceinline__ float gate_b(float w, unsigned far, int i, float x) {
  if (MODE == GDN_GLR_INPUT_PLAIN) return x;
  return __fmul_rn(far >> i & 1 ? __fsub_rn(1.f, w) : -w, x);
}
// The two gates that token t of a chunk starts: its own and, with one channel a
// thread, the next token's.
template <int V, class S>
__device__ __forceinline__ void gate_pair(const S& sg, int t, float (&g)[2]) {
#pragma unroll
  for (int j = 0; j < 2; j += V) {
    float gv[V];
    widen(sg.get(t + j / V), gv);
#pragma unroll
    for (int v = 0; v < V; v++) g[j + v] = gv[v];
  }
}

// The zero x of an identity step, whose b is -0 (that of g is +0).
template <int MODE>
constexpr bool kGlrMinusX = MODE == GDN_GLR_INPUT_PLAIN;

struct GlrArgs {
  const void* x;
  const void* g;
  int ldx, ldg;
  const int32_t* cu;
  int N;
  int T, D, slabs, stages;
  bool longest_first;  // tile kernels: the grid's order of the sequences
  int longer;  // > 0: tile kernels take the sequences of more tokens, short ones the others
  const float* h0;  // forward
  void* h;
  int ldh;
  float* s_final;
  gdn_glr_state st;  // st.h == nullptr: none
  const int32_t* slot_idx;
  float* carry;
  const void* d_h;  // backward
  int lddh;
  const float* ds_final;
  void* d_x;
  int lddx;
  void* d_g;
  int lddg;
  float* d_h0;
  int32_t* error;
};

// Tensor maps of the staged kernels' inputs.
struct GlrBoxes {
  CUtensorMap x, g, dh;
};

// First token and length of sequence n; false when cu_seqlens does not start at
// 0, end at T and ascend here.  The four loads are independent of each other.
__device__ __forceinline__ bool glr_seq(const GlrArgs& p, int n, int& start, int& length) {
  const int zero = p.cu[0], total = p.cu[p.N], first = p.cu[n], end = p.cu[n + 1];
  start = first;
  length = end - first;
  return (zero == 0) & (total == p.T) & (first >= 0) & (end >= first) & (end <= p.T);
}

// The sequence with the r-th most tokens (the earlier of two as long as each
// other), for up to 32 of them: lane i of every warp finds the rank of sequence
// i.  Where blocks wait for a place, the longest then start first.  Any
// cu_seqlens give a permutation.
constexpr int kGlrOrder = 32;
__device__ __forceinline__ bool glr_seq_by_length(const GlrArgs& p, int r, int& n, int& start,
                                                  int& length) {
  const int i = threadIdx.x & 31, zero = p.cu[0], total = p.cu[p.N];
  const int first = i < p.N ? p.cu[i] : 0, end = i < p.N ? p.cu[i + 1] : 0;
  const int tokens = (int)((unsigned)end - (unsigned)first);
  int rank = 0;
  for (int j = 0; j < p.N; j++) {
    const int other = __shfl_sync(kFull, tokens, j);
    rank += other > tokens || (other == tokens && j < i);
  }
  n = __ffs(__ballot_sync(kFull, i < p.N && rank == r)) - 1;
  start = __shfl_sync(kFull, first, n);
  const int stop = __shfl_sync(kFull, end, n);
  length = stop - start;
  return (zero == 0) & (total == p.T) & (start >= 0) & (stop >= start) & (stop <= p.T);
}

// The sequence of more than p.longer tokens of which token j * p.longer is the first
// that is a multiple of p.longer; false when there is none.  So T / p.longer blocks
// of a slab find all of them, wherever they are.  A warp looks at 32 edges at a
// time; any cu_seqlens keep its reads inside.
__device__ __forceinline__ bool glr_seq_longer(const GlrArgs& p, int j, int& n, int& start,
                                               int& length) {
  const int token = j * p.longer;
  int width = p.N;
  n = 0;
  while (width > 1) {  // the sequence is one of n .. n + width - 1
    const int step = (width + 31) / 32, i = (threadIdx.x & 31) * step;
    const unsigned m = __ballot_sync(kFull, i < width && p.cu[n + i] <= token);
    const int first = m ? (31 - __clz(m)) * step : 0;
    n += first;
    width = min(step, width - first);
  }
  return glr_seq(p, n, start, length) && length > p.longer && start <= token &&
         token - start < p.longer;
}

// Slot of row n, or -1 when it is out of range or an earlier row has it too.
// Any threads call the first form, the whole block the second.
__device__ __forceinline__ int glr_slot(const int32_t* slot_idx, int n, int n_slots) {
  if (!slot_idx) return n < n_slots ? n : -1;
  const int slot = slot_idx[n];
  bool twice = false;
  for (int i = 0; i < n; i++) twice |= slot_idx[i] == slot;
  return slot >= 0 && slot < n_slots && !twice ? slot : -1;
}
__device__ __forceinline__ int glr_slot_block(const int32_t* slot_idx, int n, int n_slots) {
  if (!slot_idx) return n < n_slots ? n : -1;
  const int slot = slot_idx[n];
  int twice = 0;
  for (int i = threadIdx.x; i < n; i += blockDim.x) twice |= slot_idx[i] == slot;
  twice = __syncthreads_or(twice);
  return slot >= 0 && slot < n_slots && !twice ? slot : -1;
}

// Channels ch .. ch + V - 1 of a row of an fp32 [rows, D] array; zeros without
// one and from D on.
template <int V>
__device__ __forceinline__ void row_get(const float* base, int64_t row, int D, int ch,
                                        float (&f)[V]) {
#pragma unroll
  for (int v = 0; v < V; v++) f[v] = base && ch + v < D ? base[row * D + ch + v] : 0.f;
}

// The first block checks every entry of cu_seqlens and is the only one that
// clears the error word, so no launch is needed for it.
__device__ __forceinline__ void glr_report(const GlrArgs& p) {
  if (blockIdx.x != 0 || !p.error) return;
  int bad = p.cu[0] != 0 || p.cu[p.N] != p.T;
  for (int i = threadIdx.x; i < p.N; i += blockDim.x) bad |= p.cu[i + 1] < p.cu[i];
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) *p.error = bad ? kErrCuSeqlens : 0;
}

// Where a thread stands: its block takes tile rank, rank + cs, ... of slab
// `slab` of sequence n; the thread channels ch .. ch + V - 1 of chunk c.
struct GlrPlace {
  int n, slab, rank, cs, c, col, ch;
  bool live;
  int L, start, steps, tiles;  // steps of cs tiles; the block's own tiles
};

template <int V>
__device__ __forceinline__ bool glr_place(const GlrArgs& p, GlrPlace& at) {
  at.cs = (int)cg::this_cluster().num_blocks();
  at.rank = (int)cg::this_cluster().block_rank();
  const int unit = blockIdx.x / at.cs;
  const int turn = unit / p.slabs;
  at.slab = unit % p.slabs;
  if (p.longer == 0) {
    glr_report(p);
  } else if (unit == (int)(gridDim.x / at.cs) - 1) {
    pdl_wait();  // no sequence is left for the last blocks, which keep the grid from
    return false;  // ending before that of the short kernel
  }
  at.n = turn;
  const bool valid = p.longer > 0       ? glr_seq_longer(p, turn, at.n, at.start, at.L)
                     : p.longest_first ? glr_seq_by_length(p, turn, at.n, at.start, at.L)
                                       : glr_seq(p, at.n, at.start, at.L);
  if (!valid) return false;  // the same for a whole cluster
  at.c = threadIdx.x / (kGlrSlab / V);
  at.col = threadIdx.x % (kGlrSlab / V) * V;
  at.ch = at.slab * kGlrSlab + at.col;
  at.live = at.ch < p.D;
  const int tiles = at.L / kGlrTile + (at.L % kGlrTile != 0);
  at.steps = (tiles + at.cs - 1) / at.cs;
  at.tiles = (tiles + at.cs - 1 - at.rank) / at.cs;
  return true;
}

// Tokens of the chunk at t0 that exist.
__device__ __forceinline__ int chunk_tokens(const GlrPlace& at, int t0) {
  return min(kGlrChunk, max(0, at.L - t0));
}

// Row t of a chunk: one 32 x 32-bit product (strides are at most 2^27).
template <class T>
__device__ __forceinline__ T* row_at(T* row, int ld, int t) {
  return row + (int64_t)ld * t;
}

// The maps of one step's chunks, [cs * 8][32] pairs (multiplier, summand), from
// every block of the cluster.  The threads of a lone block store them and meet
// a block barrier.  Blocks of a cluster send them with st.async, whose bytes
// count on the receiver's mbarrier: a cluster barrier would have to wait for
// the h that each block has just written to global memory, too.
//
// Two maps are used in turn.  A thread sends step s + 2 behind its wait for
// s + 1, which needs what every thread of every block sends for s + 1, and
// that it sends behind its own reads of step s; so a map is not overwritten
// while it is read, and its barrier is in the right phase.
struct GlrMaps {
  float2* base;    // [2][cs * 8][32]
  uint64_t* full;  // [2]
  int cs;
  bool late;
  __device__ __forceinline__ void init(void* mem, uint64_t* bars, int blocks) {
    base = static_cast<float2*>(mem);
    full = bars;
    cs = blocks;
    late = false;
    if (cs == 1) return;
    if (threadIdx.x == 0) {
      mbar_init(smem_u32(&full[0]), 1);
      mbar_init(smem_u32(&full[1]), 1);
      fence_mbar_init();
    }
    cg::this_cluster().sync();  // every block has started and has its barriers
  }
  __device__ __forceinline__ float2* at(int s) const {
    return base + (s & 1) * cs * kGlrChunks * kGlrSlab;
  }
  // Bytes this block will receive for step s.
  __device__ __forceinline__ void expect(int s) {
    if (cs > 1 && threadIdx.x == 0)
      mbar_expect_tx(smem_u32(&full[s & 1]),
                     (uint32_t)(cs * kGlrChunks * kGlrSlab * sizeof(float2)));
  }
  // The maps of the other blocks (the block's own are there behind its barrier).
  __device__ __forceinline__ void wait(int s) {
    if (cs == 1) return;
    const uint32_t bar = smem_u32(&full[s & 1]), parity = (uint32_t)(s >> 1 & 1);
    for (int i = late ? kGlrPolls - (1 << 12) : 0; i < kGlrPolls; i++) {
      uint32_t done;  // acquires what other blocks sent
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}\n"
          : "=r"(done)
          : "r"(bar), "r"(parity)
          : "memory");
      if (done) return;
    }
    late = true;
  }
};

__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void send(uint32_t dst, uint32_t mbar, float x, float y) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::
          "r"(dst),
      "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void send(uint32_t dst, uint32_t mbar, float x, float y, float z,
                                     float w) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(dst),
      "r"(__float_as_uint(x)), "r"(__float_as_uint(y)), "r"(__float_as_uint(z)),
      "r"(__float_as_uint(w)), "r"(mbar)
      : "memory");
}

// Share (a, b) of this thread's chunk with every block of the cluster.
template <int V>
__device__ __forceinline__ void glr_share(const GlrMaps& m, int s, const GlrPlace& at,
                                          const float (&a)[V], const float (&b)[V]) {
  float2* to = m.at(s) + (at.rank * kGlrChunks + at.c) * kGlrSlab + at.col;
  if (m.cs == 1) {
    if (V == 1)
      *to = make_float2(a[0], b[0]);
    else
      *reinterpret_cast<float4*>(to) = make_float4(a[0], b[0], a[V - 1], b[V - 1]);
    return;
  }
  const uint32_t dst = smem_u32(to), bar = smem_u32(&m.full[s & 1]);
  for (int r = 0; r < m.cs; r++) {
    if (V == 1)
      send(remote(dst, r), remote(bar, r), a[0], b[0]);
    else
      send(remote(dst, r), remote(bar, r), a[0], b[0], a[V - 1], b[V - 1]);
  }
}

// Run the service warp's channel z over the maps of 8 chunks (REVERSE: last
// first) and, where they are the block's own, keep what enters each of them.
// All are loaded before the chain, so that its steps are dependent products
// alone.
template <bool REVERSE>
__device__ __forceinline__ float glr_chain(const float2* maps, float z, int lane, bool own,
                                           float (&enter)[kGlrChunks][kGlrSlab]) {
  float2 m[kGlrChunks];
#pragma unroll
  for (int i = 0; i < kGlrChunks; i++) m[i] = maps[i * kGlrSlab + lane];
#pragma unroll
  for (int k = 0; k < kGlrChunks; k++) {
    const int i = REVERSE ? kGlrChunks - 1 - k : k;
    if (own) enter[i][lane] = z;
    z = __fmaf_rn(m[i].x, z, m[i].y);
  }
  return z;
}

// How a thread gets V neighbouring elements of its chunk's tokens.
//
// Staged: the block's tile (128 tokens x 32 channels) is copied by one tensor
// map box into shared memory, two steps ahead; a thread reads its own slots.
// Rows behind the sequence's end hold the next sequence's tokens and are
// cleared by the threads that own them.
//
// Direct (rows that a tensor map cannot describe: a base or stride off 16
// bytes, an odd width): loads from global memory, all of the chunk's at once,
// one element a thread (20000 x 999 in 9 sequences: 58 and 104 us; the same of
// 1000 channels, staged: 40 and 60).
template <class T, int V, bool STAGED>
struct GlrSource;

template <class T, int V>
struct GlrSource<T, V, true> {
  using R = typename Raw<T, V>::type;
  T* tile;  // this thread's column of its chunk's first token in the stage
  __device__ __forceinline__ void set(T* stage, const GlrPlace& at) {
    tile = stage + at.c * kGlrChunk * kGlrSlab + at.col;
  }
  __device__ __forceinline__ R get(int t) const { return raw_load<T, V>(tile + t * kGlrSlab); }
  __device__ __forceinline__ void clear_from(int have, bool minus = false) {
    R zero;
    raw_zero(zero, minus);
    for (int t = have; t < kGlrChunk; t++) *reinterpret_cast<R*>(tile + t * kGlrSlab) = zero;
  }
};

template <class T, int V>
struct GlrSource<T, V, false> {
  using R = typename Raw<T, V>::type;
  R r[kGlrChunk], next[kGlrChunk];
  // The loads of the chunk that the step after this one folds.
  __device__ __forceinline__ void load(const T* row, int ld, int have, bool minus = false) {
    if (have == kGlrChunk) {
#pragma unroll
      for (int t = 0; t < kGlrChunk; t++) next[t] = raw_load<T, V>(row_at(row, ld, t));
    } else {
#pragma unroll
      for (int t = 0; t < kGlrChunk; t++) {
        raw_zero(next[t], minus);
        if (t < have) next[t] = raw_load<T, V>(row_at(row, ld, t));
      }
    }
  }
  __device__ __forceinline__ void take() {
#pragma unroll
    for (int t = 0; t < kGlrChunk; t++) r[t] = next[t];
  }
  __device__ __forceinline__ R get(int t) const { return r[t]; }
};

__device__ __forceinline__ void glr_prefetch(const GlrBoxes& box, bool backward) {
  for (const CUtensorMap* m : {&box.g, &box.x, backward ? &box.dh : &box.x})
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// 2-D tensor-map load of one box into shared memory (x * the element size is
// a multiple of 16 bytes: slabs are 32 channels).
__device__ __forceinline__ void glr_box(void* dst, const CUtensorMap* map, int x, int y,
                                        uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(mbar)
      : "memory");
}

// The next place in a ring of stages, and the parity of its wait.
struct GlrRing {
  int n, slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ explicit GlrRing(int stages) : n(stages) {}
  __device__ __forceinline__ void next() {
    if (++slot == n) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

// The ring's barriers, which count the copies' bytes, and the place of the
// next tile to take.  A wait gives up after kGlrPolls polls, and then the
// kernel goes on without waiting (every block still meets every barrier) and
// reports.
struct GlrPipe : GlrRing {
  uint64_t* full;  // [kGlrMaxStages]
  bool late = false;
  using GlrRing::GlrRing;
  __device__ __forceinline__ void init(uint64_t* bars) {
    full = bars;
    if (threadIdx.x == 0) {
      for (int i = 0; i < n; i++) mbar_init(smem_u32(&full[i]), 1);
      fence_mbar_init();
    }
    __syncthreads();
  }
  __device__ __forceinline__ void wait() {
    if (!mbar_wait(smem_u32(&full[slot]), parity, late ? 1 << 12 : kGlrPolls)) late = true;
  }
};

template <class IN, class G>
struct GlrForwardStage {
  alignas(128) G g[kGlrTile * kGlrSlab];
  alignas(128) IN x[kGlrTile * kGlrSlab];
};

__device__ __forceinline__ unsigned char* align128(unsigned char* p) {
  return p + ((128u - (smem_u32(p) & 127u)) & 127u);
}

template <class IN, class G, class OUT, int V, int MODE, bool STAGED>
__global__ void __launch_bounds__((kGlrBlock<V>), glr_blocks<V>(true))
    k_glr_forward(const GlrArgs p, const __grid_constant__ GlrBoxes box) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) float enter[kGlrChunks][kGlrSlab];
  __shared__ uint64_t bars[2 + kGlrMaxStages];
  using Stage = GlrForwardStage<IN, G>;
  unsigned char* smem = align128(smem_raw);
  Stage* stage = reinterpret_cast<Stage*>(smem);
  GlrPlace at;
  if (STAGED && threadIdx.x == 0) glr_prefetch(box, false);
  if (!glr_place<V>(p, at)) return;
  const int step_tokens = at.cs * kGlrTile;
  GlrMaps maps;
  maps.init(smem + (STAGED ? p.stages * sizeof(Stage) : 0), bars, at.cs);
  GlrPipe pipe(p.stages);
  if (STAGED) pipe.init(bars + 2);
  if (threadIdx.x >= kGlrThreads<V>) {
    // The service warp copies the block's tiles in order into the ring of stages
    // and runs the state over the chunks.
    const int lane = threadIdx.x & 31, ch = at.slab * kGlrSlab + lane;
    int copied = 0;
    auto issue = [&]() {
      if (!STAGED || copied >= at.tiles) return;
      if (lane == 0) {
        Stage& d = stage[pipe.slot];
        const int row = at.start + copied * step_tokens + at.rank * kGlrTile;
        const uint32_t bar = smem_u32(&pipe.full[pipe.slot]);
        mbar_expect_tx(bar, kGlrTile * kGlrSlab * (uint32_t)(sizeof(IN) + sizeof(G)));
        glr_box(d.g, &box.g, at.slab * kGlrSlab, row, bar);
        glr_box(d.x, &box.x, at.slab * kGlrSlab, row, bar);
      }
      copied++;
      pipe.next();
    };
    for (int j = 0; j < p.stages; j++) issue();
    float H[1];
    row_get<1>(p.h0, at.n, p.D, ch, H);
    for (int s = 0; s < at.steps; s++) {
      __syncthreads();  // every warp has folded its chunks of the step
      maps.wait(s);
      for (int r = 0; r < at.cs; r++)
        H[0] = glr_chain<false>(maps.at(s) + r * kGlrChunks * kGlrSlab, H[0], lane, r == at.rank,
                                enter);
      __syncthreads();
      issue();
      if (p.carry && s < at.tiles && ch < p.D)
        p.carry[(int64_t)(at.start / kGlrTile + at.n + s * at.cs + at.rank) * p.D + ch] =
            enter[0][lane];
    }
    if (maps.late && p.error) atomicOr(p.error, kErrTimeout);
    __syncwarp();
    if (at.cs > 1) cg::this_cluster().sync();
    return;
  }
  float Hm[V], hv[V], A[kGlrChunk][V], B[kGlrChunk][V];
  row_get<V>(p.h0, at.n, p.D, at.ch, hv);
#pragma unroll
  for (int v = 0; v < V; v++) {
    Hm[v] = hv[v];
    A[kGlrChunk - 1][v] = 1.f;
    B[kGlrChunk - 1][v] = 0.f;
  }
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)at.start * p.ldx + at.ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)at.start * p.ldg + at.ch;
  OUT* h = static_cast<OUT*>(p.h) + (int64_t)at.start * p.ldh + at.ch;
  int t0 = at.rank * kGlrTile + at.c * kGlrChunk;
  GlrSource<IN, V, STAGED> sx;
  GlrSource<G, V, STAGED> sg;
  auto load = [&](int t) {  // direct: the chunk at token t, ahead of its fold
    if constexpr (!STAGED) {
      const int have = at.live ? chunk_tokens(at, t) : 0;
      sx.load(x + (int64_t)t * p.ldx, p.ldx, have, kGlrMinusX<MODE>);
      sg.load(g + (int64_t)t * p.ldg, p.ldg, have);
    }
  };
  load(t0);
  for (int s = 0; s < at.steps; s++, t0 += step_tokens) {
    const int tokens = chunk_tokens(at, t0), have = at.live ? tokens : 0;
    if (s < at.tiles) {
      if constexpr (STAGED) {
        sx.set(stage[pipe.slot].x, at);
        sg.set(stage[pipe.slot].g, at);
        pipe.wait();
        if (tokens < kGlrChunk) {
          sx.clear_from(tokens, kGlrMinusX<MODE>);
          sg.clear_from(tokens);
        }
      } else {
        sx.take();
        sg.take();
      }
#pragma unroll
      for (int i = 0; i < kGlrChunk * V; i += 2) {
        float gv[2], w[2], xv[V];
        unsigned far = 0;
        gate_pair<V>(sg, i / V, gv);
        gates_of<MODE>(gv, w, far, 0);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int t = (i + j) / V, v = (i + j) % V;
          if (v == 0) widen(sx.get(t), xv);
          const float a = gate_a<MODE>(w[j], far, j), b = gate_b<MODE>(w[j], far, j, xv[v]);
          A[t][v] = t ? __fmul_rn(a, A[t ? t - 1 : 0][v]) : a;
          B[t][v] = t ? __fmaf_rn(a, B[t ? t - 1 : 0][v], b) : __fmaf_rn(a, 0.f, b);
        }
      }
    } else {  // only in a cluster's last step: this block's tile is behind the end
#pragma unroll
      for (int v = 0; v < V; v++) {
        A[kGlrChunk - 1][v] = 1.f;
        B[kGlrChunk - 1][v] = 0.f;
      }
    }
    load(t0 + step_tokens);
    maps.expect(s);
    glr_share<V>(maps, s, at, A[kGlrChunk - 1], B[kGlrChunk - 1]);
    __syncthreads();
    if (STAGED) pipe.next();
    __syncthreads();  // the service warp has handed over
    if (have == 0) continue;
#pragma unroll
    for (int v = 0; v < V; v++) Hm[v] = enter[at.c][at.col + v];
    OUT* out = h + (int64_t)t0 * p.ldh;
    if (have == kGlrChunk) {
#pragma unroll
      for (int t = 0; t < kGlrChunk; t++) {
#pragma unroll
        for (int v = 0; v < V; v++) hv[v] = __fmaf_rn(A[t][v], Hm[v], B[t][v]);
        put(row_at(out, p.ldh, t), hv);
      }
    } else {
#pragma unroll
      for (int t = 0; t < kGlrChunk; t++) {
#pragma unroll
        for (int v = 0; v < V; v++) hv[v] = __fmaf_rn(A[t][v], Hm[v], B[t][v]);
        if (t < have) put(row_at(out, p.ldh, t), hv);
      }
    }
  }
  if (pipe.late && p.error) atomicOr(p.error, kErrTimeout);
  if (at.cs > 1) {  // nothing is on its way to a block that ends
    __syncwarp();
    cg::this_cluster().sync();
  }
  // The thread that holds the last token has its h and the chunk's (Hm, A, B):
  // the identity steps behind the last token have left them.
  const int tail = at.L > 0 ? (at.L - 1) / kGlrChunk % (at.cs * kGlrChunks) : 0;
  const bool mine = at.live && at.rank * kGlrChunks + at.c == tail;
  if (p.s_final && mine) put(p.s_final + (int64_t)at.n * p.D + at.ch, hv);
  if (p.st.h) {
    if (!mine && !(at.slab == 0 && at.rank == 0 && threadIdx.x == 0)) return;
    const int slot = glr_slot(p.slot_idx, at.n, p.st.n_slots);
    const int pos = (int)(at.L % kGlrChunk);
    if (slot < 0) {
      atomicOr(p.st.error, kErrPos);
      return;
    }
    if (at.slab == 0 && at.rank == 0 && threadIdx.x == 0) p.st.pos[slot] = pos;
    if (mine) {
      const int64_t to = (int64_t)slot * p.D + at.ch;
#pragma unroll
      for (int v = 0; v < V; v++) {
        p.st.h[to + v] = pos ? Hm[v] : hv[v];
        p.st.a[to + v] = pos ? A[kGlrChunk - 1][v] : 1.f;
        p.st.b[to + v] = pos ? B[kGlrChunk - 1][v] : 0.f;
      }
    }
  }
}

// Reverse mode: steps from a sequence's last to its first.  A chunk's map of
// the adjoint mu is mu -> fma(A, mu, M) with the A of the forward and
// M = sum A_t dh_t over the chunk, so the chunks of a step are again evaluated side by
// side; h_{t-1} comes from the tile's carry row and the chunks' (A, B) by the
// forward's operations.
template <class IN, class G, class OUT>
struct GlrBackwardStage {
  alignas(128) G g[kGlrTile * kGlrSlab];
  alignas(128) IN x[kGlrTile * kGlrSlab];
  alignas(128) OUT dh[kGlrTile * kGlrSlab];
};

template <class IN, class G, class OUT, int V, int MODE, bool STAGED>
__global__ void __launch_bounds__((kGlrBlock<V>), glr_blocks<V>(false))
    k_glr_backward(const GlrArgs p, const __grid_constant__ GlrBoxes box) {
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(16) float enter[kGlrChunks][kGlrSlab];
  __shared__ __align__(16) float enter_mu[kGlrChunks][kGlrSlab];
  __shared__ __align__(16) float2 own[kGlrChunks][kGlrSlab];  // (A, B) of the block's chunks
  __shared__ uint64_t bars[2 + kGlrMaxStages];
  using Stage = GlrBackwardStage<IN, G, OUT>;
  unsigned char* smem = align128(smem_raw);
  Stage* stage = reinterpret_cast<Stage*>(smem);
  GlrPlace at;
  if (STAGED && threadIdx.x == 0) glr_prefetch(box, true);
  if (!glr_place<V>(p, at)) return;
  const int step_tokens = at.cs * kGlrTile;
  GlrMaps maps;
  maps.init(smem + (STAGED ? p.stages * sizeof(Stage) : 0), bars, at.cs);
  GlrPipe pipe(p.stages);
  // A block without a tile in the last step starts one step later than the others.
  const int skip = at.steps - at.tiles;
  if (STAGED) pipe.init(bars + 2);
  if (threadIdx.x >= kGlrThreads<V>) {
    // The service warp copies the block's tiles, last first, and runs mu over the
    // cluster's chunks and the state over the block's own.
    const int lane = threadIdx.x & 31, ch = at.slab * kGlrSlab + lane;
    int left = at.tiles;
    auto issue = [&]() {
      if (!STAGED || left <= 0) return;
      left--;
      if (lane == 0) {
        Stage& d = stage[pipe.slot];
        const int row = at.start + left * step_tokens + at.rank * kGlrTile;
        const uint32_t bar = smem_u32(&pipe.full[pipe.slot]);
        mbar_expect_tx(bar,
                       kGlrTile * kGlrSlab * (uint32_t)(sizeof(IN) + sizeof(G) + sizeof(OUT)));
        glr_box(d.g, &box.g, at.slab * kGlrSlab, row, bar);
        glr_box(d.x, &box.x, at.slab * kGlrSlab, row, bar);
        glr_box(d.dh, &box.dh, at.slab * kGlrSlab, row, bar);
      }
      pipe.next();
    };
    for (int j = 0; j < p.stages; j++) issue();
    const float* carry = p.carry + (int64_t)(at.start / kGlrTile + at.n) * p.D;
    auto entering = [&](int i) {  // the state that enters the block's tile of step i
      float h[1];
      const int tile = (at.steps - 1 - i) * at.cs + at.rank;
      row_get<1>(i >= skip && i < at.steps ? carry : nullptr, tile, p.D, ch, h);
      return h[0];
    };
    float mu[1], H = entering(0);
    row_get<1>(p.ds_final, at.n, p.D, ch, mu);
    for (int i = 0; i < at.steps; i++) {
      const float next = entering(i + 1);
      __syncthreads();  // every warp has folded its chunks of the step
      glr_chain<false>(&own[0][0], H, lane, true, enter);  // (other blocks' maps are on their way)
      maps.wait(i);
      for (int r = at.cs - 1; r >= 0; r--)
        mu[0] = glr_chain<true>(maps.at(i) + r * kGlrChunks * kGlrSlab, mu[0], lane,
                                r == at.rank, enter_mu);
      __syncthreads();
      if (i > skip) issue();  // every warp is done with the stage of step i - 1
      H = next;
    }
    if (p.d_h0 && at.rank == 0 && ch < p.D) p.d_h0[(int64_t)at.n * p.D + ch] = mu[0];
    if (maps.late && p.error) atomicOr(p.error, kErrTimeout);
    __syncwarp();
    if (at.cs > 1) cg::this_cluster().sync();
    return;
  }
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)at.start * p.ldx + at.ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)at.start * p.ldg + at.ch;
  const OUT* dh = static_cast<const OUT*>(p.d_h) + (int64_t)at.start * p.lddh + at.ch;
  IN* dx = static_cast<IN*>(p.d_x) + (int64_t)at.start * p.lddx + at.ch;
  G* dg = static_cast<G*>(p.d_g) + (int64_t)at.start * p.lddg + at.ch;
  GlrSource<IN, V, STAGED> sx;
  GlrSource<G, V, STAGED> sg;
  GlrSource<OUT, V, STAGED> sd;
  auto load = [&](int t) {  // direct: the chunk at token t, ahead of its fold
    if constexpr (!STAGED) {
      const int have = at.live && t >= 0 ? chunk_tokens(at, t) : 0;
      sg.load(g + (int64_t)t * p.ldg, p.ldg, have);
      sx.load(x + (int64_t)t * p.ldx, p.ldx, have);
      sd.load(dh + (int64_t)t * p.lddh, p.lddh, have);
    }
  };
  load(((at.steps - 1) * at.cs + at.rank) * kGlrTile + at.c * kGlrChunk);
  for (int i = 0; i < at.steps; i++) {
    const int tile = (at.steps - 1 - i) * at.cs + at.rank;
    const int t0 = tile * kGlrTile + at.c * kGlrChunk;
    const int tokens = chunk_tokens(at, t0), have = at.live ? tokens : 0;
    float ga[kGlrChunk][V], A[kGlrChunk][V], B[kGlrChunk][V], M[V], mm[V], Hm[V];
    unsigned far = 0;
    if (i >= skip) {
      if constexpr (STAGED) {
        sx.set(stage[pipe.slot].x, at);
        sg.set(stage[pipe.slot].g, at);
        sd.set(stage[pipe.slot].dh, at);
        pipe.wait();
        pipe.next();
        if (tokens < kGlrChunk) {
          sx.clear_from(tokens);
          sg.clear_from(tokens);
          sd.clear_from(tokens);
          fence_async_smem();  // the stage is copied into again
        }
      } else {
        sg.take();
        sx.take();
        sd.take();
      }
#pragma unroll
      for (int i = 0; i < kGlrChunk * V; i += 2) {
        float gv[2], w[2], xv[V], dv[V];
        gate_pair<V>(sg, i / V, gv);
        gates_of<MODE>(gv, w, far, i);
#pragma unroll
        for (int j = 0; j < 2; j++) {
          const int t = (i + j) / V, v = (i + j) % V;
          if (v == 0) {
            widen(sx.get(t), xv);
            widen(sd.get(t), dv);
          }
          ga[t][v] = w[j];
          const float a = gate_a<MODE>(w[j], far, i + j);
          const float b = gate_b<MODE>(w[j], far, i + j, xv[v]);
          A[t][v] = t ? __fmul_rn(a, A[t ? t - 1 : 0][v]) : a;
          B[t][v] = t ? __fmaf_rn(a, B[t ? t - 1 : 0][v], b) : __fmaf_rn(a, 0.f, b);
          M[v] = t ? __fmaf_rn(A[t][v], dv[v], M[v]) : __fmul_rn(a, dv[v]);
        }
      }
    } else {  // only in a cluster's first step: this block's tile is behind the end
#pragma unroll
      for (int v = 0; v < V; v++) {
        A[kGlrChunk - 1][v] = 1.f;
        B[kGlrChunk - 1][v] = M[v] = 0.f;
      }
    }
    load(t0 - step_tokens);
    maps.expect(i);
    glr_share<V>(maps, i, at, A[kGlrChunk - 1], M);
#pragma unroll
    for (int v = 0; v < V; v++)
      own[at.c][at.col + v] = make_float2(A[kGlrChunk - 1][v], B[kGlrChunk - 1][v]);
    __syncthreads();
    __syncthreads();  // the service warp has handed over
    if (have == 0) continue;
#pragma unroll
    for (int v = 0; v < V; v++) {
      Hm[v] = enter[at.c][at.col + v];
      mm[v] = enter_mu[at.c][at.col + v];
    }
    IN* ox = dx + (int64_t)t0 * p.lddx;
    G* og = dg + (int64_t)t0 * p.lddg;
    auto back = [&](int t, bool write) {
      float dv[V], xv[V], fx[V], fg[V];
      widen(sd.get(t), dv);
      widen(sx.get(t), xv);
#pragma unroll
      for (int v = 0; v < V; v++) {
        const float before = t ? __fmaf_rn(A[t ? t - 1 : 0][v], Hm[v], B[t ? t - 1 : 0][v]) : Hm[v];
        const float lam = __fadd_rn(dv[v], mm[v]);
        mm[v] = __fmul_rn(gate_a<MODE>(ga[t][v], far, t * V + v), lam);
        fx[v] = gate_b<MODE>(ga[t][v], far, t * V + v, lam);
        fg[v] = __fmul_rn(mm[v], MODE == GDN_GLR_INPUT_COMPLEMENT ? __fsub_rn(before, xv[v])
                                                                  : before);
      }
      if (write) {
        put(row_at(ox, p.lddx, t), fx);
        put(row_at(og, p.lddg, t), fg);
      }
    };
    if (have == kGlrChunk) {
#pragma unroll
      for (int t = kGlrChunk - 1; t >= 0; t--) back(t, true);
    } else {
#pragma unroll
      for (int t = kGlrChunk - 1; t >= 0; t--) back(t, t < have);
    }
  }
  if (pipe.late && p.error) atomicOr(p.error, kErrTimeout);
  if (at.cs > 1) {  // nothing is on its way to a block that ends
    __syncwarp();
    cg::this_cluster().sync();
  }
}

// Short sequences: a thread takes one channel of a whole sequence, chunk by
// chunk, with the operations of the kernels above in the same order.  There is
// no tile, no hand-over and no ring to set up, which is most of what a block
// spends on a sequence of a few tokens.
constexpr int kGlrShortThreads = 128;

// Sequence n of a block of the short kernels; false when it is not for it.  Where
// the call has longer ones (p.longer), their tile kernel is the next and shares the
// device with this one.
__device__ __forceinline__ bool glr_short_seq(const GlrArgs& p, int n, int& start, int& L) {
  if (p.longer > 0) pdl_trigger();
  glr_report(p);
  return glr_seq(p, n, start, L) && (p.longer == 0 || L <= p.longer);
}

template <class IN, class G, class OUT, int MODE>
__global__ void __launch_bounds__(kGlrShortThreads) k_glr_short_forward(const GlrArgs p) {
  const int n = blockIdx.x / p.slabs, ch = blockIdx.x % p.slabs * kGlrShortThreads + threadIdx.x;
  int start, L;
  if (!glr_short_seq(p, n, start, L)) return;
  const bool live = ch < p.D;
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)start * p.ldx + ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)start * p.ldg + ch;
  OUT* h = static_cast<OUT*>(p.h) + (int64_t)start * p.ldh + ch;
  float H[1], hv[1], A = 1.f, B = 0.f;
  row_get<1>(p.h0, n, p.D, ch, H);
  hv[0] = H[0];
  float Hm = H[0];
  GlrSource<IN, 1, false> sx;
  GlrSource<G, 1, false> sg;
  auto load = [&](int t) {
    const int have = live && t < L ? min(kGlrChunk, L - t) : 0;
    sx.load(x + (int64_t)t * p.ldx, p.ldx, have, kGlrMinusX<MODE>);
    sg.load(g + (int64_t)t * p.ldg, p.ldg, have);
  };
  load(0);
  for (int t0 = 0; live && t0 < L; t0 += kGlrChunk) {
    sx.take();
    sg.take();
    load(t0 + kGlrChunk);
    if (p.carry && t0 % kGlrTile == 0)
      p.carry[(int64_t)(start / kGlrTile + n + t0 / kGlrTile) * p.D + ch] = H[0];
    Hm = H[0];
    const int have = min(kGlrChunk, L - t0);
    OUT* out = h + (int64_t)t0 * p.ldh;
#pragma unroll
    for (int i = 0; i < kGlrChunk; i += 2) {
      float gv[2], w[2], xv[1];
      unsigned far = 0;
      gate_pair<1>(sg, i, gv);
      gates_of<MODE>(gv, w, far, 0);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int t = i + j;
        widen(sx.get(t), xv);
        const float a = gate_a<MODE>(w[j], far, j), b = gate_b<MODE>(w[j], far, j, xv[0]);
        A = t ? __fmul_rn(a, A) : a;
        B = t ? __fmaf_rn(a, B, b) : __fmaf_rn(a, 0.f, b);
        hv[0] = __fmaf_rn(A, Hm, B);
        if (t < have) put(row_at(out, p.ldh, t), hv);
      }
    }
    H[0] = hv[0];
  }
  if (p.s_final && live) put(p.s_final + (int64_t)n * p.D + ch, hv);
  if (p.st.h) {
    const int slot = glr_slot_block(p.slot_idx, n, p.st.n_slots);
    const int pos = L % kGlrChunk;
    if (slot < 0) {
      if (threadIdx.x == 0) atomicOr(p.st.error, kErrPos);
      return;
    }
    if (ch == 0) p.st.pos[slot] = pos;
    if (live) {
      const int64_t to = (int64_t)slot * p.D + ch;
      p.st.h[to] = pos ? Hm : hv[0];
      p.st.a[to] = pos ? A : 1.f;
      p.st.b[to] = pos ? B : 0.f;
    }
  }
}

template <class IN, class G, class OUT, int MODE>
__global__ void __launch_bounds__(kGlrShortThreads) k_glr_short_backward(const GlrArgs p) {
  __shared__ float enter[kGlrChunks][kGlrShortThreads];  // a thread's own column
  const int n = blockIdx.x / p.slabs, ch = blockIdx.x % p.slabs * kGlrShortThreads + threadIdx.x;
  int start, L;
  if (!glr_short_seq(p, n, start, L)) return;
  if (ch >= p.D) return;
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)start * p.ldx + ch;
  const G* g = static_cast<const G*>(p.g) + (int64_t)start * p.ldg + ch;
  const OUT* dh = static_cast<const OUT*>(p.d_h) + (int64_t)start * p.lddh + ch;
  IN* dx = static_cast<IN*>(p.d_x) + (int64_t)start * p.lddx + ch;
  G* dg = static_cast<G*>(p.d_g) + (int64_t)start * p.lddg + ch;
  float mu[1];
  row_get<1>(p.ds_final, n, p.D, ch, mu);
  float w[kGlrChunk], A[kGlrChunk], B[kGlrChunk];
  unsigned far;
  GlrSource<IN, 1, false> sx;
  GlrSource<G, 1, false> sg;
  GlrSource<OUT, 1, false> sd;
  auto fold = [&](int t0, int have) {  // the chunk's gates and maps
    sx.load(x + (int64_t)t0 * p.ldx, p.ldx, have);
    sg.load(g + (int64_t)t0 * p.ldg, p.ldg, have);
    sx.take();
    sg.take();
    far = 0;
#pragma unroll
    for (int i = 0; i < kGlrChunk; i += 2) {
      float gv[2], k[2], xv[1];
      gate_pair<1>(sg, i, gv);
      gates_of<MODE>(gv, k, far, i);
#pragma unroll
      for (int j = 0; j < 2; j++) {
        const int t = i + j;
        widen(sx.get(t), xv);
        w[t] = k[j];
        const float a = gate_a<MODE>(k[j], far, t), b = gate_b<MODE>(k[j], far, t, xv[0]);
        A[t] = t ? __fmul_rn(a, A[t ? t - 1 : 0]) : a;
        B[t] = t ? __fmaf_rn(a, B[t ? t - 1 : 0], b) : __fmaf_rn(a, 0.f, b);
      }
    }
  };
  for (int tile = (L - 1) / kGlrTile; L > 0 && tile >= 0; tile--) {
    const int first = tile * kGlrTile;
    const int chunks = min(kGlrChunks, (L - first + kGlrChunk - 1) / kGlrChunk);
    // The states that enter the tile's chunks, from its carry row.
    float H = p.carry[(int64_t)(start / kGlrTile + n + tile) * p.D + ch];
    enter[0][threadIdx.x] = H;
#pragma unroll 1
    for (int c = 1; c < chunks; c++) {
      fold(first + (c - 1) * kGlrChunk, kGlrChunk);
      H = __fmaf_rn(A[kGlrChunk - 1], H, B[kGlrChunk - 1]);
      enter[c][threadIdx.x] = H;
    }
#pragma unroll 1
    for (int c = chunks - 1; c >= 0; c--) {
      const float Hm = enter[c][threadIdx.x];
      const int t0 = first + c * kGlrChunk, have = min(kGlrChunk, L - t0);
      sd.load(dh + (int64_t)t0 * p.lddh, p.lddh, have);
      sd.take();
      fold(t0, have);
      IN* ox = dx + (int64_t)t0 * p.lddx;
      G* og = dg + (int64_t)t0 * p.lddg;
      float M = 0.f, mm = mu[0];
#pragma unroll
      for (int t = 0; t < kGlrChunk; t++) {
        float dv[1];
        widen(sd.get(t), dv);
        M = t ? __fmaf_rn(A[t], dv[0], M) : __fmul_rn(A[0], dv[0]);
      }
#pragma unroll
      for (int t = kGlrChunk - 1; t >= 0; t--) {
        float dv[1], xv[1], fx[1], fg[1];
        widen(sd.get(t), dv);
        widen(sx.get(t), xv);
        const float before = t ? __fmaf_rn(A[t ? t - 1 : 0], Hm, B[t ? t - 1 : 0]) : Hm;
        const float lam = __fadd_rn(dv[0], mm);
        mm = __fmul_rn(gate_a<MODE>(w[t], far, t), lam);
        fx[0] = gate_b<MODE>(w[t], far, t, lam);
        fg[0] = __fmul_rn(mm, MODE == GDN_GLR_INPUT_COMPLEMENT ? __fsub_rn(before, xv[0])
                                                               : before);
        if (t < have) {
          put(row_at(ox, p.lddx, t), fx);
          put(row_at(og, p.lddg, t), fg);
        }
      }
      mu[0] = __fmaf_rn(A[kGlrChunk - 1], mu[0], M);
    }
  }
  if (p.d_h0) put(p.d_h0 + (int64_t)n * p.D + ch, mu);
}

// One block per row (a row's pos is read and written by one block).  A row's
// first channels are loaded beside its pos, not behind it.  256 rows of 4096
// channels take 5.2 us a step in a graph of steps (their 29 MB stay in the L2), one
// of 2048 1.9.
constexpr int kGlrStepThreads = 1024;

template <class IN, class G, class OUT, int V, int MODE>
__global__ void __launch_bounds__(kGlrStepThreads) k_glr_step(const GlrArgs p) {
  const int b = blockIdx.x;
  const int slot = glr_slot_block(p.slot_idx, b, p.st.n_slots);
  if (slot < 0) {
    if (threadIdx.x == 0) atomicOr(p.st.error, kErrPos);
    return;
  }
  const IN* x = static_cast<const IN*>(p.x) + (int64_t)b * p.ldx;
  const G* g = static_cast<const G*>(p.g) + (int64_t)b * p.ldg;
  OUT* h = static_cast<OUT*>(p.h) + (int64_t)b * p.ldh;
  const int64_t base = (int64_t)slot * p.D;
  float xv[V], gv[V], H[V], A[V], B[V];
  auto load = [&](int ch) {
    if (ch >= p.D) return;
    widen(raw_load<IN, V>(x + ch), xv);
    widen(raw_load<G, V>(g + ch), gv);
    widen(raw_load<float, V>(p.st.h + base + ch), H);
    widen(raw_load<float, V>(p.st.a + base + ch), A);
    widen(raw_load<float, V>(p.st.b + base + ch), B);
  };
  load(threadIdx.x * V);
  const int pos = p.st.pos[slot];
  if (pos < 0 || pos >= kGlrChunk) {
    if (threadIdx.x == 0) atomicOr(p.st.error, kErrPos);
    return;
  }
  __syncthreads();  // every thread has read pos
  const bool full = pos == kGlrChunk - 1;
  if (threadIdx.x == 0) p.st.pos[slot] = full ? 0 : pos + 1;
  for (int ch = threadIdx.x * V; ch < p.D; ch += blockDim.x * V) {
    float hv[V], w[2];
    const float pair[2] = {gv[0], gv[V - 1]};
    unsigned far = 0;
    gates_of<MODE>(pair, w, far, 0);
#pragma unroll
    for (int v = 0; v < V; v++) {
      const float a = gate_a<MODE>(w[v], far, v);
      A[v] = __fmul_rn(a, pos ? A[v] : 1.f);
      B[v] = __fmaf_rn(a, pos ? B[v] : 0.f, gate_b<MODE>(w[v], far, v, xv[v]));
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
    load(ch + blockDim.x * V);
  }
}

template <int V>
static unsigned glr_step_threads(int D) {
  const int n = (D / V + 31) / 32 * 32;
  return (unsigned)(n < 32 ? 32 : n > kGlrStepThreads ? kGlrStepThreads : n);
}

// ----------------------------------------------------------------------------
// Launchers
// ----------------------------------------------------------------------------
enum GlrOp { kGlrFwd, kGlrBwd, kGlrStep };

constexpr size_t kGlrStatic = 4608;  // shared memory of a block that its launch does not size

// Launch shape.  Blocks of a cluster: doubled while every block of the grid
// still has a place on the device and a sequence has tiles for them on average
// (65536 x 2048 alone, forward: 387, 256, 183 us with 1, 2 and 4; 8 have no
// place and take 307).  A backward step of 8 blocks is slower than two of 4
// (32768 x 1024: 212 against 119 us).
//
// Stages: as many as the shared memory of a multiprocessor holds for the blocks
// that it gets, and at least two.  A backward cluster would rather have three
// and fewer blocks: with two its copies start only behind the last step (20000
// x 1000 in 9 sequences with bf16 gates: 72 against 55 us, 10240 x 2048 in 5 61
// against 55; of fp32 data the latter takes 81 against 89, and with fp32 gates
// two blocks are all that fit in either case).  Where blocks are many the others
// cover that, and three blocks with two stages win (16384 x 2048 in 32: 78
// against 84 us, of the complement form 86 against 100).
//
// Longest sequences first where some blocks have to wait for a place: 10240
// tokens of 2048 channels in sequences of 531, 793, 1762, 2136 and 5018, forward
// and backward: 95 us (without it 102); where it gains nothing, 16384 x 2048 in
// 32 equal ones: 129 (125).  With 64 sequences every block's search for its own
// costs more than the order gains.
struct GlrShape {
  int cs, stages;
  bool longest_first;
  size_t smem;
};

static GlrShape glr_shape(const GlrArgs& p, size_t stage, int most, bool backward) {
  constexpr int64_t kSms = 148;
  constexpr size_t kSmem = 228 * 1024, kBlock = 1024 + kGlrStatic;  // of an SM; fixed per block
  auto maps = [](int cs) { return (size_t)2 * cs * kGlrChunks * kGlrSlab * sizeof(float2) + 128; };
  auto places = [&](int cs) {
    const int64_t n = kSmem / (kBlock + maps(cs) + 2 * stage);
    return kSms * (n < most ? n : most);
  };
  // (there may be one sequence longer than p.longer; two blocks for each: 4 take 269
  // us where 2 take 402 above, but 8 such sequences of 2040 tokens 86 forward, not
  // 68, and where there are none the clusters to start are the cost)
  const int seqs = p.longer > 0 ? 1 : p.N;
  const int64_t units = (int64_t)seqs * p.slabs;
  const int max_cluster = p.longer > 0 ? 2 : backward ? 4 : 8;
  GlrShape sh{1, 0, false, 0};
  while (sh.cs < max_cluster && units * 2 * sh.cs <= places(2 * sh.cs) &&
         p.T > (int64_t)seqs * kGlrTile * sh.cs)
    sh.cs *= 2;
  // Sequences of unequal length keep the device waiting for the longest: two
  // blocks for each then gain more than a second wave of blocks costs (10240
  // tokens of 2048 channels in 5 sequences, forward and backward: 95 against 148
  // us where they are uneven, 103 against 86 us where they are equal), for a
  // backward from a few more units on (20000 x 2048 in 9, uneven: 104 against 134
  // us, 18432 in 9 equal ones: 95 against 104; the forward the same within 2 us).
  const int waves = backward && stage > 0 ? 4 : most;
  if (sh.cs == 1 && seqs > 1 && units <= waves * kSms && p.T > (int64_t)seqs * kGlrTile)
    sh.cs = 2;
  int64_t here = (units * sh.cs + kSms - 1) / kSms;  // blocks of a multiprocessor
  here = here < most && p.longer == 0 ? here : most;
  if (stage > 0) {
    const size_t fixed = kBlock + maps(sh.cs), least = backward && sh.cs > 1 ? 3 : 2;
    while (here > 1 && kSmem / here < fixed + least * stage) here--;
    sh.stages = (int)((kSmem / here - fixed) / stage);
    if (sh.stages > kGlrMaxStages) sh.stages = kGlrMaxStages;
  }
  sh.longest_first = seqs > 1 && seqs <= kGlrOrder && units * sh.cs > here * kSms;
  sh.smem = sh.stages * stage + maps(sh.cs);
  return sh;
}

template <class K>
static cudaError_t glr_run(K kernel, int threads, size_t stage, int most, bool backward,
                           GlrArgs& p, const GlrBoxes& box, cudaStream_t st) {
  const GlrShape sh = glr_shape(p, stage, most, backward);
  p.stages = sh.stages;
  p.longest_first = sh.longest_first;
  // The kernel's limit, not this call's size: two host threads may be here at once.
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       227 * 1024 - (int)kGlrStatic);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)sh.cs;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // behind the short kernel
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  const unsigned turns = p.longer > 0 ? (unsigned)((p.T + p.longer - 1) / p.longer) : p.N;
  cfg.gridDim = dim3((turns * (unsigned)p.slabs + (p.longer > 0)) * (unsigned)sh.cs);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = sh.smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = p.longer > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p, box);
}

// A map over [T][D] rows of stride ld whose boxes are one tile of one slab;
// columns past D and tokens past T read as zeros.
template <class T>
static bool glr_encode(CUtensorMap* map, const void* base, int64_t tokens, int D, int ld) {
  EncodeTiledFn fn = encode_fn();
  if (!fn || (reinterpret_cast<uintptr_t>(base) & 15) || (size_t)ld * sizeof(T) % 16) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)D, (cuuint64_t)tokens};
  const cuuint64_t stride[1] = {(cuuint64_t)ld * sizeof(T)};
  const cuuint32_t box[2] = {kGlrSlab, kGlrTile}, one[2] = {1, 1};
  return fn(map,
            sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
            2, const_cast<void*>(base), dims, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class IN, class G, class OUT, int MODE>
static cudaError_t glr_tiles(GlrOp op, GlrArgs& p, bool pairs, cudaStream_t st) {
  GlrBoxes box{};
  // pairs: the rows that are written take two elements at a time
  const bool staged = pairs && p.T > 0 && glr_encode<IN>(&box.x, p.x, p.T, p.D, p.ldx) &&
                      glr_encode<G>(&box.g, p.g, p.T, p.D, p.ldg) &&
                      (op == kGlrFwd || glr_encode<OUT>(&box.dh, p.d_h, p.T, p.D, p.lddh));
  if (op == kGlrFwd) {
    if (staged)
      return glr_run(k_glr_forward<IN, G, OUT, 2, MODE, true>, kGlrBlock<2>,
                     sizeof(GlrForwardStage<IN, G>), glr_blocks<2>(true), false, p, box, st);
    return glr_run(k_glr_forward<IN, G, OUT, 1, MODE, false>, kGlrBlock<1>, 0,
                   glr_blocks<1>(true), false, p, box, st);
  }
  if (staged)
    return glr_run(k_glr_backward<IN, G, OUT, 2, MODE, true>, kGlrBlock<2>,
                   sizeof(GlrBackwardStage<IN, G, OUT>), glr_blocks<2>(false), true, p, box, st);
  return glr_run(k_glr_backward<IN, G, OUT, 1, MODE, false>, kGlrBlock<1>, 0,
                 glr_blocks<1>(false), true, p, box, st);
}

template <class IN, class G, class OUT, int MODE>
static cudaError_t glr_launch(GlrOp op, GlrArgs& p, bool pairs, cudaStream_t st) {
  p.slabs = (p.D + kGlrSlab - 1) / kGlrSlab;
  if (op == kGlrStep) {
    if (pairs)
      k_glr_step<IN, G, OUT, 2, MODE><<<(unsigned)p.N, glr_step_threads<2>(p.D), 0, st>>>(p);
    else
      k_glr_step<IN, G, OUT, 1, MODE><<<(unsigned)p.N, glr_step_threads<1>(p.D), 0, st>>>(p);
    return cudaGetLastError();
  }
  // Sequences of up to 64 tokens on average, and more of them than one wave of
  // tile blocks takes: 64 sequences of 4096 channels, forward and backward, 300
  // tokens: 33 us (tiles: 133), 4096: 132 (166), 8192: 249 (213).
  if (p.T > (int64_t)64 * p.N || (int64_t)p.N * p.slabs <= 3 * 148)
    return glr_tiles<IN, G, OUT, MODE>(op, p, pairs, st);
  // The average says nothing of the longest, and a thread that walks thousands of
  // tokens alone would keep the device waiting: sequences of more than p.longer
  // tokens go to tile blocks, which share the device with the short kernel's.  63
  // sequences of one token and one of 3968, of 4096 channels: 43 us forward and 55
  // backward (219 and 700 by the short kernel alone; the long one alone 29 and 41);
  // 600 tokens in 999 and 60000 in one, 2048 channels: 402 and 512 (3052 and 10093).
  //
  // Since only the device knows the lengths, there are blocks for each sequence
  // that might be so long, T / p.longer of them, and those that find none cost
  // some time: 1000 sequences of 60 tokens of 2048 channels 203 and 395 us (without
  // them 191 and 383), 64 of 64 tokens of 4096 33 and 61 (31 and 57).  That grows
  // with their number, so they are kept to some for the work there is.  Up to the
  // least length it is worth no second launch (1024 tokens forward: 66 us, 512
  // backward: 97), and calls of so few tokens in all have none.
  const int least = op == kGlrFwd ? 1024 : 512;
  const int64_t turns = 1 + (512 + (int64_t)p.T * p.D / 65536) / p.slabs;
  const int64_t share = (p.T + turns - 1) / turns;
  p.longer = share > least ? (int)share : least;
  if (p.T <= p.longer) p.longer = 0;
  p.slabs = (p.D + kGlrShortThreads - 1) / kGlrShortThreads;
  const unsigned blocks = (unsigned)p.N * (unsigned)p.slabs;
  if (op == kGlrFwd)
    k_glr_short_forward<IN, G, OUT, MODE><<<blocks, kGlrShortThreads, 0, st>>>(p);
  else
    k_glr_short_backward<IN, G, OUT, MODE><<<blocks, kGlrShortThreads, 0, st>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || p.longer == 0) return e;
  p.slabs = (p.D + kGlrSlab - 1) / kGlrSlab;
  return glr_tiles<IN, G, OUT, MODE>(op, p, pairs, st);
}

template <class IN, class G, class OUT>
static cudaError_t glr_modes(GlrOp op, GlrArgs& p, bool pairs, int mode, cudaStream_t st) {
  if (mode == GDN_GLR_INPUT_PLAIN)
    return glr_launch<IN, G, OUT, GDN_GLR_INPUT_PLAIN>(op, p, pairs, st);
  return glr_launch<IN, G, OUT, GDN_GLR_INPUT_COMPLEMENT>(op, p, pairs, st);
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
constexpr int64_t kMaxTokens = INT32_MAX - (1 << 12);  // a last step's tiles stay in 32 bits
constexpr int64_t kMaxLd = (int64_t)1 << 27;  // a chunk's offsets fit 32 bits

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
  if (T > kMaxTokens) return GDN_ERR_UNSUPPORTED;
  if (n_seqs == 0) return T == 0 ? GDN_OK : GDN_ERR_INVALID_ARG;
  if (!cu || !aligned(cu, 4)) return GDN_ERR_INVALID_ARG;
  const int64_t blocks = (int64_t)n_seqs * ((D + 31) / 32);  // clusters of up to 8
  return blocks * 8 > INT32_MAX ? GDN_ERR_UNSUPPORTED : GDN_OK;
}

}  // namespace

extern "C" int64_t gdn_glr_carry_rows(int n_seqs, int64_t total_tokens) {
  if (n_seqs < 0 || total_tokens < 0 || total_tokens > kMaxTokens) return 0;
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
  if (!aligned(h0, 4) || !aligned(s_final, 4) || !aligned(carry, 4) || !aligned(slot_idx, 4))
    return GDN_ERR_INVALID_ARG;
  pairs = pairs && aligned(s_final, 8);  // (the others are read or written one at a time)
  if (slot_idx && !state) return GDN_ERR_INVALID_ARG;
  if (state) {
    if ((rc = check_state(*state)) != GDN_OK) return rc;
    if (!slot_idx && n_seqs > state->n_slots) return GDN_ERR_INVALID_ARG;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n_seqs == 0)
    return !error_word || cudaMemsetAsync(error_word, 0, sizeof(int32_t), st) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  gdn::GlrArgs p{};
  p.x = x;
  p.g = g;
  p.ldx = (int)ldx;
  p.ldg = (int)ldg;
  p.cu = cu_seqlens;
  p.N = n_seqs;
  p.T = (int)total_tokens;
  p.D = D;
  p.h0 = h0;
  p.h = h;
  p.ldh = (int)ldh;
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
  if (!aligned(carry, 4) || !aligned(ds_final, 4) || !aligned(d_h0, 4))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (n_seqs == 0)
    return !error_word || cudaMemsetAsync(error_word, 0, sizeof(int32_t), st) == cudaSuccess
               ? GDN_OK
               : GDN_ERR_CUDA;
  gdn::GlrArgs p{};
  p.x = x;
  p.g = g;
  p.ldx = (int)ldx;
  p.ldg = (int)ldg;
  p.cu = cu_seqlens;
  p.N = n_seqs;
  p.T = (int)total_tokens;
  p.D = D;
  p.carry = const_cast<float*>(carry);
  p.d_h = d_h;
  p.lddh = (int)lddh;
  p.ds_final = ds_final;
  p.d_x = d_x;
  p.lddx = (int)lddx;
  p.d_g = d_g;
  p.lddg = (int)lddg;
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
  p.ldx = (int)ldx;
  p.ldg = (int)ldg;
  p.N = B;
  p.D = D;
  p.h = h;
  p.ldh = (int)ldh;
  p.st = state;
  p.slot_idx = slot_idx;
  return gdn::glr_types(gdn::kGlrStep, p, in_dtype == GDN_BF16, g_dtype == GDN_BF16,
                        out_dtype == GDN_BF16, pairs, input_mode,
                        static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}
