// gdn_qk_norm.cu -- norms of queries and keys for each head with the position
// rotation in the same pass, and their gradients (gdn_qk_norm.h).
//
// A group of D / 8 lanes has a head's D channels, each lane two pieces of four
// neighbouring ones.  With pairs (j, j + F) the pieces of a lane are a rotated
// pair, so that the rotation needs no exchange; the lanes behind the rotated
// channels, and all lanes otherwise, have eight neighbours.  Sums over a head
// are the lane's two packed partial sums, added, and a butterfly over the
// group: a head's bits are its own.
//
// A group takes some heads of one token at a time: the token's cosines and
// sines, computed once by the group's lanes and exchanged, stay in registers
// with the weights, and the loads of several heads are under way together.
//
// Memory bounds it: each head is read once and written once (backward: two reads
// and a write).  32768 x (16 + 16) bf16 heads of 128: 85 us forward, 169 with an
// fp32 gradient backward, 6.3 TB/s each of 6.5 that a copy reaches.  A rotation with
// weights adds instructions (62 a head forward, 79 backward): 16384 x (32 + 8)
// takes 60 us (5.6 TB/s) and 100 us (5.0 TB/s).
#include <cuda_runtime.h>
#include <math.h>

#include "../../include/gdn_qk_norm.h"
#include "gdn_common.cuh"
#include "gdn_mma.cuh"

namespace gdn {

constexpr int kQkThreads = 256;

enum QkRot { kRotNone = 0, kRotHalves = 1, kRotPairs = 2 };

struct QkSide {
  const void* x;
  const void* dy;
  const float* w;
  void* out;  // y, or dx
  int64_t ldx, lddy, ldout;
  int H;
  int heads;   // of a unit: one token's heads that a group takes at a time
  int chunks;  // units of a token
  int64_t blocks;  // that the grid has for this side (q's first)
  int64_t span;    // units of one block
};

struct QkArgs {
  QkSide q, k;
  int64_t T;
  const int32_t* positions;
  const float* inv_freq;
  int F;             // rotated pairs
  float eps, inv_m;  // inv_m: 1 (l2) or 1 / D (rms)
  float* partial;    // [blocks][D] or nullptr
};

// Four neighbouring channels as loaded.
template <class T>
struct Four;
template <>
struct Four<float> {
  using type = float4;
};
template <>
struct Four<__nv_bfloat16> {
  using type = uint2;
};

// A lane's eight channels as packed pairs.
struct Eight {
  float2 v[4];
};
__device__ __forceinline__ void widen4(const float4& r, float2* v) {
  v[0] = f2(r.x, r.y);
  v[1] = f2(r.z, r.w);
}
__device__ __forceinline__ void widen4(const uint2& r, float2* v) {
  v[0] = f2(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u));
  v[1] = f2(__uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, const float2* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float2* v) {
  union {
    uint2 r;
    __nv_bfloat162 h[2];
  } u;
  u.h[0] = __floats2bfloat162_rn(v[0].x, v[0].y);
  u.h[1] = __floats2bfloat162_rn(v[1].x, v[1].y);
  *reinterpret_cast<uint2*>(p) = u.r;
}

// Angles are counted in turns, as fractions of 2^64: pos times a frequency wraps
// around by itself, which is the reduction that a far position needs (an fp32
// product has lost the angle from positions of a few thousand on).  The
// frequency comes from an fp64 product, the upper 32 bits of the angle are
// kept, and the nearest quarter turn is taken off, so that the fp32 functions
// see at most an eighth of a turn.
__device__ __forceinline__ uint64_t frequency(float f) {
  double turns = (double)f * 0.15915494309189533577;  // 1 / 2 pi
  turns -= floor(turns);
  return (uint64_t)(turns * 18446744073709551616.0);  // 2^64
}
__device__ __forceinline__ float2 angle(int pos, uint64_t f) {
  const uint32_t t = (uint32_t)(((uint64_t)(int64_t)pos * f) >> 32);
  const uint32_t quarter = (t + (1u << 29)) >> 30;
  float s, c;
  sincospif((float)(int32_t)(t - (quarter << 30)) * 4.656612873077393e-10f, &s, &c);  // 2^-31
  const float x = quarter & 1 ? -s : c, y = quarter & 1 ? c : s;
  return quarter & 2 ? f2(-x, -y) : f2(x, y);
}

// (sum x^2 [/ d] + eps)^(-1/2), off by at most two units in the last place: the
// correctly rounded function takes 66 us forward and 107 backward at 16384 x (32 +
// 8) rotated heads (59 and 100), and would take 3 U (U = 2^-24) off the 17 U that
// bound an fp32 y.
__device__ __forceinline__ float inverse_norm(float sum, const QkArgs& p) {
  return rsqrtf(__fmaf_rn(sum, p.inv_m, p.eps));
}

// Where a lane stands in its head: its pieces' first channels, and the first of
// its angles (-1: its channels are not rotated).
struct QkLane {
  int lane;  // in the group
  int a, b;
  int angle;
};
template <int D, int ROT>
__device__ __forceinline__ QkLane qk_lane(int F) {
  QkLane l;
  l.lane = threadIdx.x % (D / 8);
  l.a = 8 * l.lane;
  l.angle = -1;
  if (ROT == kRotHalves && l.lane < F / 4) {
    l.a = l.angle = 4 * l.lane;
    l.b = l.a + F;
  } else {
    l.b = l.a + 4;
    if (ROT == kRotPairs && l.a < 2 * F) l.angle = l.a / 2;
  }
  return l;
}

// A lane's four angles: cosines, sines and the sines' negatives as packed pairs.
struct Turn {
  float2 c[2], s[2], m[2];
};

// The angles of a token for a group: its lanes share the work, and each reads
// its four (SIGN = -1: to turn back).  All lanes of a warp call it (`have`: the
// group has a token).
template <int D, int ROT, int SIGN>
__device__ __forceinline__ void qk_angles(const QkArgs& p, const QkLane& l, bool have, int64_t t,
                                          const uint64_t* freq, float2* table, Turn& turn) {
  if (ROT == kRotNone) return;
  __syncwarp();  // the last token's have been read
  if (have) {
    const int pos = p.positions[t];
    for (int j = l.lane; j < p.F; j += D / 8) table[j] = angle(pos, freq[j]);
  }
  __syncwarp();
  // A group without a token has no table: it must not turn its zeros by what an
  // earlier kernel left there.
  float2 a[4];
#pragma unroll
  for (int i = 0; i < 4; i++) a[i] = have && l.angle >= 0 ? table[l.angle + i] : f2(1.f, 0.f);
#pragma unroll
  for (int i = 0; i < 2; i++) {
    turn.c[i] = f2(a[2 * i].x, a[2 * i + 1].x);
    turn.s[i] = f2(SIGN * a[2 * i].y, SIGN * a[2 * i + 1].y);
    turn.m[i] = f2(-turn.s[i].x, -turn.s[i].y);
  }
}

// Rotate a lane's channels.
template <int ROT>
__device__ __forceinline__ void rotate8(Eight& n, const QkLane& l, const Turn& turn) {
  if (ROT == kRotNone || l.angle < 0) return;
  if (ROT == kRotHalves) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const float2 u = n.v[i], v = n.v[2 + i];
      n.v[i] = __ffma2_rn(v, turn.m[i], __fmul2_rn(u, turn.c[i]));
      n.v[2 + i] = __ffma2_rn(u, turn.s[i], __fmul2_rn(v, turn.c[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float u = n.v[i].x, v = n.v[i].y;
      const float c = i & 1 ? turn.c[i / 2].y : turn.c[i / 2].x;
      const float s = i & 1 ? turn.s[i / 2].y : turn.s[i / 2].x;
      n.v[i].x = __fmaf_rn(-v, s, __fmul_rn(u, c));
      n.v[i].y = __fmaf_rn(u, s, __fmul_rn(v, c));
    }
  }
}

template <int D>
__device__ __forceinline__ float dot8(const Eight& a, const Eight& b) {
  float2 s = __fmul2_rn(a.v[0], b.v[0]);
#pragma unroll
  for (int i = 1; i < 4; i++) s = __ffma2_rn(a.v[i], b.v[i], s);
  float t = __fadd_rn(s.x, s.y);
#pragma unroll
  for (int m = 1; m < D / 8; m *= 2) t = __fadd_rn(t, __shfl_xor_sync(kFull, t, m));
  return t;
}
__device__ __forceinline__ void scale8(Eight& n, float r) {
#pragma unroll
  for (int i = 0; i < 4; i++) n.v[i] = __fmul2_rn(n.v[i], f2(r, r));
}
__device__ __forceinline__ void times8(Eight& n, const Eight& w) {
#pragma unroll
  for (int i = 0; i < 4; i++) n.v[i] = __fmul2_rn(n.v[i], w.v[i]);
}
__device__ __forceinline__ void weights8(const float* w, const QkLane& l, Eight& f) {
  widen4(*reinterpret_cast<const float4*>(w + l.a), f.v);
  widen4(*reinterpret_cast<const float4*>(w + l.b), f.v + 2);
}

// The unit (token, first head) of a group in one pass of its block.
struct QkUnit {
  bool have;
  int64_t t;
  int h0, heads;
};
__device__ __forceinline__ QkUnit qk_unit(const QkSide& sd, int64_t u, int64_t end) {
  QkUnit q;
  q.have = u < end;
  q.t = q.have ? u / sd.chunks : 0;
  q.h0 = q.have ? (int)(u - q.t * sd.chunks) * sd.heads : 0;
  q.heads = q.have ? min(sd.heads, sd.H - q.h0) : 0;
  return q;
}

// Heads whose loads are under way together, and the blocks of a multiprocessor
// that their registers are kept to.  10240 x (16 + 16) heads of 128, no
// rotation: forward 29 us with 4 heads and 5 blocks (2 heads: 31), backward 53 us
// with 2 heads and 3 blocks (4 heads and 2 blocks: 64, 1 and 4: 68).  16384 x
// (32 + 8) rotated with weights: forward 60 us (78 without the bound).  8192 x
// (8 + 2) heads of 256: backward 37 us with 2 and 3 (4 and 2: 53).  fp32 heads are
// twice the registers: forward of 16384 x (32 + 8) without rotation 100 us with 3
// blocks (1.0 of the copy rate; 5: 144, they spill), 8192 x (16 + 16) to bf16 33
// (52), 16384 x (16 + 8) of 64 31 (50).
//
// A rotation's backward has registers for 2 blocks only, whose warps do not
// cover each other's loads: it has the next batch under way while it works on
// one (16384 x (32 + 8): 100 us, without it 104; fp32, 8192 x (16 + 4): 47, 49).
// Two batches of 4 heads fit where all elements are bf16 (2 heads: 103), else 2
// (8192 x (16 + 16) heads of 64 with fp32 gradients: 30 us, 4 heads 42).  Without
// a rotation, and with heads of 256, 3 blocks do better (53 against 61 us, 37
// against 42).
constexpr int kQkForwardBatch = 4;
__host__ __device__ constexpr int qk_forward_blocks(int rot, size_t element) {
  return element == 4 ? 3 : rot == kRotNone ? 5 : 4;
}
__host__ __device__ constexpr bool qk_backward_ahead(int rot, int d) {
  return rot != kRotNone && d != 256;
}
__host__ __device__ constexpr int qk_backward_batch(int rot, int d, size_t elements) {
  return qk_backward_ahead(rot, d) && elements == 4 ? 4 : 2;
}
__host__ __device__ constexpr int qk_backward_blocks(int rot, int d) {
  return qk_backward_ahead(rot, d) ? 2 : 3;
}

template <class IN, class OUT, int D, int ROT>
__global__ void __launch_bounds__(kQkThreads, qk_forward_blocks(ROT, sizeof(IN)))
    k_qk_forward(const QkArgs p) {
  constexpr int kLanes = D / 8, kGroups = kQkThreads / kLanes, kBatch = kQkForwardBatch;
  extern __shared__ uint64_t freq[];  // [F], and each group's [F] cosines and sines
  const bool isq = blockIdx.x < p.q.blocks;
  const QkSide& sd = isq ? p.q : p.k;
  const int64_t first = (isq ? blockIdx.x : blockIdx.x - p.q.blocks) * sd.span;
  const int64_t end = min(first + sd.span, p.T * sd.chunks);
  const int grp = threadIdx.x / kLanes;
  const QkLane l = qk_lane<D, ROT>(p.F);
  float2* table = reinterpret_cast<float2*>(freq + p.F) + grp * p.F;
  if (ROT != kRotNone) {
    for (int j = threadIdx.x; j < p.F; j += kQkThreads) freq[j] = frequency(p.inv_freq[j]);
    __syncthreads();
  }
  Eight w;
  if (sd.w) weights8(sd.w, l, w);
  using Raw4 = typename Four<IN>::type;
  for (int64_t base = first; base < end; base += kGroups) {
    const QkUnit u = qk_unit(sd, base + grp, end);
    const IN* x = static_cast<const IN*>(sd.x) + u.t * sd.ldx + (int64_t)u.h0 * D;
    OUT* y = static_cast<OUT*>(sd.out) + u.t * sd.ldout + (int64_t)u.h0 * D;
    const IN *xa = x + l.a, *xb = x + l.b;
    OUT *ya = y + l.a, *yb = y + l.b;
    Turn turn;
    Raw4 ra[kBatch], rb[kBatch];
    // FULL: all of the batch's heads exist in all of the warp's groups, and
    // their chains of operations can be interleaved.
    auto load = [&](int left, bool full) {
#pragma unroll
      for (int i = 0; i < kBatch; i++) {
        if (full || i < left) {
          ra[i] = *reinterpret_cast<const Raw4*>(xa + i * D);
          rb[i] = *reinterpret_cast<const Raw4*>(xb + i * D);
        } else {
          ra[i] = rb[i] = Raw4{};
        }
      }
    };
    auto head = [&](int i, bool write) {
      Eight n;
      widen4(ra[i], n.v);
      widen4(rb[i], n.v + 2);
      scale8(n, inverse_norm(dot8<D>(n, n), p));
      if (sd.w) times8(n, w);
      rotate8<ROT>(n, l, turn);
      if (write) {
        store4(ya + i * D, n.v);
        store4(yb + i * D, n.v + 2);
      }
    };
    // The warp's groups go through as many heads as the one with most.
    bool full = __all_sync(kFull, u.heads >= kBatch);
    load(u.heads, full);  // under way while the angles are computed
    qk_angles<D, ROT, 1>(p, l, u.have, u.t, freq, table, turn);
    for (int h = 0; h < sd.heads; h += kBatch) {
      if (full) {
#pragma unroll
        for (int i = 0; i < kBatch; i++) head(i, true);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; i++) head(i, h + i < u.heads);
      }
      xa += kBatch * D, xb += kBatch * D, ya += kBatch * D, yb += kBatch * D;
      if (h + kBatch < sd.heads) {
        full = __all_sync(kFull, u.heads >= h + 2 * kBatch);
        load(u.heads - h - kBatch, full);
      }
    }
  }
}

template <class IN, class GR, int D, int ROT>
__global__ void __launch_bounds__(kQkThreads, qk_backward_blocks(ROT, D))
    k_qk_backward(const QkArgs p) {
  constexpr int kLanes = D / 8, kGroups = kQkThreads / kLanes;
  constexpr int kBatch = qk_backward_batch(ROT, D, sizeof(IN) + sizeof(GR));
  constexpr bool kAhead = qk_backward_ahead(ROT, D);
  extern __shared__ uint64_t freq[];  // [F], and each group's [F] cosines and sines
  const bool isq = blockIdx.x < p.q.blocks;
  const QkSide& sd = isq ? p.q : p.k;
  const int64_t first = (isq ? blockIdx.x : blockIdx.x - p.q.blocks) * sd.span;
  const int64_t end = min(first + sd.span, p.T * sd.chunks);
  const int grp = threadIdx.x / kLanes;
  const QkLane l = qk_lane<D, ROT>(p.F);
  float2* table = reinterpret_cast<float2*>(freq + p.F) + grp * p.F;
  if (ROT != kRotNone) {
    for (int j = threadIdx.x; j < p.F; j += kQkThreads) freq[j] = frequency(p.inv_freq[j]);
    __syncthreads();
  }
  Eight w, dw;
#pragma unroll
  for (int i = 0; i < 4; i++) dw.v[i] = f2(0.f, 0.f);
  if (sd.w) weights8(sd.w, l, w);
  using RawX = typename Four<IN>::type;
  using RawG = typename Four<GR>::type;
  struct Batch {  // of a unit's heads, as loaded
    RawX xa[kBatch], xb[kBatch];
    RawG ga[kBatch], gb[kBatch];
  };
  Batch cur;
  Turn turn;
  QkUnit u = qk_unit(sd, first + grp, end);
  const IN* x = static_cast<const IN*>(sd.x) + u.t * sd.ldx + (int64_t)u.h0 * D;
  const GR* dy = static_cast<const GR*>(sd.dy) + u.t * sd.lddy + (int64_t)u.h0 * D;
  auto load = [&](Batch& b, const IN* x, const GR* dy, int left, bool full) {
    const IN *px = x + l.a, *qx = x + l.b;
    const GR *pg = dy + l.a, *qg = dy + l.b;
#pragma unroll
    for (int i = 0; i < kBatch; i++) {
      if (full || i < left) {
        b.xa[i] = *reinterpret_cast<const RawX*>(px + i * D);
        b.xb[i] = *reinterpret_cast<const RawX*>(qx + i * D);
        b.ga[i] = *reinterpret_cast<const RawG*>(pg + i * D);
        b.gb[i] = *reinterpret_cast<const RawG*>(qg + i * D);
      } else {  // zeros: nothing for dw
        b.xa[i] = b.xb[i] = RawX{};
        b.ga[i] = b.gb[i] = RawG{};
      }
    }
  };
  bool full = __all_sync(kFull, u.heads >= kBatch);
  load(cur, x, dy, u.heads, full);
  for (int64_t base = first; base < end; base += kGroups) {
    IN* dx = static_cast<IN*>(sd.out) + u.t * sd.ldout + (int64_t)u.h0 * D;
    IN *pd = dx + l.a, *qd = dx + l.b;
    auto head = [&](int i, bool write) {
      Eight n, e;  // the head and its gradient
      widen4(cur.xa[i], n.v);
      widen4(cur.xb[i], n.v + 2);
      widen4(cur.ga[i], e.v);
      widen4(cur.gb[i], e.v + 2);
      rotate8<ROT>(e, l, turn);
      const float r = inverse_norm(dot8<D>(n, n), p);
      if (sd.w) {
        const float2 rr = f2(r, r);
#pragma unroll
        for (int j = 0; j < 4; j++)
          dw.v[j] = __ffma2_rn(e.v[j], __fmul2_rn(n.v[j], rr), dw.v[j]);
        times8(e, w);
      }
      const float m = __fmul_rn(dot8<D>(n, e), p.inv_m);
      const float z = -__fmul_rn(r, __fmul_rn(r, m));  // (r^2 may be out of range)
#pragma unroll
      for (int j = 0; j < 4; j++) e.v[j] = __ffma2_rn(n.v[j], f2(z, z), e.v[j]);
      scale8(e, r);
      if (write) {
        store4(pd + i * D, e.v);
        store4(qd + i * D, e.v + 2);
      }
    };
    qk_angles<D, ROT, -1>(p, l, u.have, u.t, freq, table, turn);
    const int heads = u.heads;
    for (int h = 0; h < sd.heads; h += kBatch) {
      const bool now = full;
      auto load_next = [&](Batch& b) {  // the unit's next batch, or the next unit's first
        int left = heads - h - kBatch;
        x += kBatch * D, dy += kBatch * D;
        if (h + kBatch >= sd.heads) {
          u = qk_unit(sd, base + kGroups + grp, end);
          left = u.heads;
          x = static_cast<const IN*>(sd.x) + u.t * sd.ldx + (int64_t)u.h0 * D;
          dy = static_cast<const GR*>(sd.dy) + u.t * sd.lddy + (int64_t)u.h0 * D;
        }
        full = __all_sync(kFull, left >= kBatch);
        load(b, x, dy, left, full);
      };
      Batch next;
      if (kAhead) load_next(next);
      if (now) {
#pragma unroll
        for (int i = 0; i < kBatch; i++) head(i, true);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; i++) head(i, h + i < heads);
      }
      pd += kBatch * D, qd += kBatch * D;
      if (kAhead)
        cur = next;
      else
        load_next(cur);
    }
  }
  if (p.partial && sd.w) {  // the block's sum of dw over its groups, in ascending order
    __shared__ float red[kGroups][D];
    store4(&red[grp][l.a], dw.v);
    store4(&red[grp][l.b], dw.v + 2);
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += kQkThreads) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < kGroups; j++) s = __fadd_rn(s, red[j][c]);
      p.partial[(int64_t)blockIdx.x * D + c] = s;
    }
  }
}

// d_w = sum of the blocks' partial sums (y: the side): row group r of 32 adds
// the blocks r, r + 32, ... in order, then the groups are added in order.
__global__ void __launch_bounds__(1024)
    k_qk_weight_sum(const float* partial, int q_blocks, int k_blocks, int D, float* d_wq,
                    float* d_wk) {
  __shared__ float red[32][32];
  float* out = blockIdx.y == 0 ? d_wq : d_wk;
  if (!out) return;
  pdl_wait();
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), r = threadIdx.x >> 5;
  const int blocks = blockIdx.y == 0 ? q_blocks : k_blocks;
  const float* col = partial + (blockIdx.y == 0 ? 0 : (int64_t)q_blocks * D) + c;
  float s = 0.f;
  for (int b = r; b < blocks; b += 32) s = __fadd_rn(s, col[(int64_t)b * D]);
  red[r][threadIdx.x & 31] = s;
  __syncthreads();
  if (r == 0) {
    for (int j = 1; j < 32; j++) s = __fadd_rn(s, red[j][threadIdx.x]);
    out[c] = s;
  }
}

// ----------------------------------------------------------------------------
// Launchers
// ----------------------------------------------------------------------------
// Heads of a unit and blocks of each side.  A unit has up to 32 heads (what it
// spends on the angles is shared by them), fewer while the units would not fill
// the device (kQkFill lane groups).  A block takes one unit for each of its
// groups; where it keeps a partial sum of a weight's gradient (`sums`: about
// how many there are to be) it takes its share of its side, so that all blocks
// run at once.  The plan depends on sizes alone, so the sums' order does not
// change from device to device.  False when the grid would be too large.
constexpr int kQkUnitHeads = 32;
constexpr int kQkFill = 148 * 4 * 8;

static int qk_sums(int rot, int d) { return 148 * qk_backward_blocks(rot, d); }

static bool qk_plan(QkArgs& p, int64_t T, int Hq, int Hk, int d, int sums) {
  p.T = T;
  p.q.H = Hq;
  p.k.H = Hk;
  const int groups = kQkThreads / (d / 8);
  int heads = kQkUnitHeads;
  while (heads > 1 && T * (Hq + Hk) / heads < kQkFill) heads /= 2;
  for (QkSide* s : {&p.q, &p.k}) {
    s->chunks = (s->H + heads - 1) / heads;
    s->heads = s->chunks > 0 ? (s->H + s->chunks - 1) / s->chunks : 0;  // even shares
    const int64_t units = T * s->chunks;
    int64_t passes = 1;
    if (sums) {
      const int64_t share = sums * (int64_t)s->H / (Hq + Hk);
      const int64_t blocks = (units + groups - 1) / groups;
      passes = share > 0 ? (blocks + share - 1) / share : blocks;
      if (passes < 1) passes = 1;
    }
    s->span = passes * groups;
    s->blocks = (units + s->span - 1) / s->span;
  }
  return p.q.blocks + p.k.blocks <= INT32_MAX;
}

static size_t qk_smem(const QkArgs& p, int d, int rot) {
  return rot == kRotNone ? 0 : (size_t)(kQkThreads / (d / 8) + 1) * p.F * sizeof(float2);
}

template <class IN, class OTHER, int D, int ROT>
static cudaError_t qk_launch(bool backward, const QkArgs& p, cudaStream_t st) {
  const unsigned blocks = (unsigned)(p.q.blocks + p.k.blocks);
  const size_t smem = qk_smem(p, D, ROT);
  if (backward)
    k_qk_backward<IN, OTHER, D, ROT><<<blocks, kQkThreads, smem, st>>>(p);
  else
    k_qk_forward<IN, OTHER, D, ROT><<<blocks, kQkThreads, smem, st>>>(p);
  return cudaGetLastError();
}

template <class IN, class OTHER, int D>
static cudaError_t qk_rot(bool bwd, const QkArgs& p, int rot, cudaStream_t st) {
  if (rot == kRotNone) return qk_launch<IN, OTHER, D, kRotNone>(bwd, p, st);
  if (rot == kRotHalves) return qk_launch<IN, OTHER, D, kRotHalves>(bwd, p, st);
  return qk_launch<IN, OTHER, D, kRotPairs>(bwd, p, st);
}

template <class IN, class OTHER>
static cudaError_t qk_dims(bool bwd, const QkArgs& p, int d, int rot,
                           cudaStream_t st) {
  if (d == 64) return qk_rot<IN, OTHER, 64>(bwd, p, rot, st);
  if (d == 128) return qk_rot<IN, OTHER, 128>(bwd, p, rot, st);
  return qk_rot<IN, OTHER, 256>(bwd, p, rot, st);
}

static cudaError_t qk_types(bool bwd, const QkArgs& p, bool ib, bool ob, int d, int rot,
                            cudaStream_t st) {
  using bf16 = __nv_bfloat16;
  if (ib)
    return ob ? qk_dims<bf16, bf16>(bwd, p, d, rot, st)
              : qk_dims<bf16, float>(bwd, p, d, rot, st);
  return ob ? qk_dims<float, bf16>(bwd, p, d, rot, st)
            : qk_dims<float, float>(bwd, p, d, rot, st);
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
  if (!gdn::qk_plan(p, T, Hq, Hk, d, 0)) return GDN_ERR_UNSUPPORTED;
  p.q.x = q, p.q.ldx = ldq, p.q.w = wq, p.q.out = oq, p.q.ldout = ldoq;
  p.k.x = k, p.k.ldx = ldk, p.k.w = wk, p.k.out = ok, p.k.ldout = ldok;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.F = rot_dim / 2;
  p.eps = eps;
  p.inv_m = norm == GDN_QK_NORM_RMS ? 1.f / (float)d : 1.f;
  return gdn::qk_types(false, p, in_dtype == GDN_BF16, out_dtype == GDN_BF16, d,
                       rot_kind(rot_dim, interleaved),
                       static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? GDN_OK
             : GDN_ERR_CUDA;
}

extern "C" size_t gdn_qk_norm_backward_workspace_bytes(int64_t T, int Hq, int Hk, int d) {
  if (check_shape(T, Hq, Hk, d) != GDN_OK || T == 0) return 0;
  gdn::QkArgs p{};
  // (the plan with more sums; a rotation's backward keeps fewer)
  if (!gdn::qk_plan(p, T, Hq, Hk, d, gdn::qk_sums(gdn::kRotNone, d))) return 0;
  return (size_t)(p.q.blocks + p.k.blocks) * d * sizeof(float);
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
  if (weights) {
    if (!workspace || workspace_bytes < gdn_qk_norm_backward_workspace_bytes(T, Hq, Hk, d))
      return GDN_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return GDN_ERR_INVALID_ARG;
  }
  gdn::QkArgs p{};
  const int rot = rot_kind(rot_dim, interleaved);
  if (!gdn::qk_plan(p, T, Hq, Hk, d, weights ? gdn::qk_sums(rot, d) : 0))
    return GDN_ERR_UNSUPPORTED;
  p.q.x = q, p.q.ldx = ldq, p.q.w = wq, p.q.dy = d_oq, p.q.lddy = lddoq, p.q.out = d_q;
  p.q.ldout = lddq;
  p.k.x = k, p.k.ldx = ldk, p.k.w = wk, p.k.dy = d_ok, p.k.lddy = lddok, p.k.out = d_k;
  p.k.ldout = lddk;
  p.positions = positions;
  p.inv_freq = inv_freq;
  p.F = rot_dim / 2;
  p.eps = eps;
  p.inv_m = norm == GDN_QK_NORM_RMS ? 1.f / (float)d : 1.f;
  p.partial = weights ? static_cast<float*>(workspace) : nullptr;
  if (gdn::qk_types(true, p, in_dtype == GDN_BF16, grad_dtype == GDN_BF16, d, rot, st) !=
      cudaSuccess)
    return GDN_ERR_CUDA;
  if (weights) {
    if (gdn::launch_dependent(gdn::k_qk_weight_sum, dim3((unsigned)(d / 32), 2), dim3(1024), 0,
                              st, (const float*)p.partial, (int)p.q.blocks, (int)p.k.blocks, d,
                              d_wq, d_wk) != cudaSuccess)
      return GDN_ERR_CUDA;
  }
  return GDN_OK;
}
