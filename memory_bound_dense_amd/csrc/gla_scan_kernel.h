// Gated linear attention over whole sequences for gfx950, forward and
// backward: per (sequence, head), with the state S (DK x DV) in float32,
//
//     S_t = diag(exp(g_t)) S_{t-1} + k_t v_t^T        o_t = scale S_t^T q_t
//
// The backward pass runs the same recurrence from the end,
//
//     D_t = diag(exp(g_{t+1})) D_{t+1} + (scale q_t) do_t^T   (D beyond the
//     last token is dS_T),  dv_t = D_t^T k_t,  dk_t = D_t v_t,
//     dq_t = scale S_t do_t,  dg_t = dg_{t+1} + q_t dq_t - k_t dk_t
//
// (the last because rowsum(S_t D_t) = dg_t + k_t dk_t = dg_{t+1} + q_t dq_t; the
// token's own term, the same in both, is left out of them).
// Reversed, a recurrence differs from the forward one only in its order and
// in that a token's gate acts after the token instead of before it, so the same
// kernels serve both:
//   scan_state_kernel  a segment's own state
//   scan_out_kernel    out_i  = X_i^T S     o  (K k, V v, X q), dv (K q, V do, X k)
//   scan_grad_kernel   out_i  = S W_i       dq (K k, V v, W do), dk (K q, V do, W v)
//
// A chunk of 32 tokens is one step.  With G the running sum of the gates in
// the chunk and r its value at the middle, the chunk is matrix products of
// x e^{G-r} and k e^{r-G}: their product is the decay e^{G_i - G_j} of every
// pair, and |G - r| <= kRange keeps each factor far from overflow.  Where that
// does not hold (very strong gates, gates of -inf that clear the state) or a
// value is huge or not finite, the same code takes the chunk 8 tokens at a time, and
// where it still does not, one token at a time, whose decay acts as a whole on
// the state: no pair of factors is formed, so any gate will do and nothing
// leaks from a later token into an earlier one.
//
// Precision: the products run on bf16 matrix instructions with fp32 sums, and
// every fp32 factor enters as a sum of bf16 terms -- two (2^-17 relative) where
// the result is rounded to 16 bits right after, three (2^-25) where it goes
// into the fp32 state or the gradient of the gates, which is a running sum (two
// there too if it and the tensors are bf16: see scan_grad_kernel).  q, k, v and do
// are exact in one term (bf16) or two (f16).
//
// Layout.  16x16x32 matrix instructions: an operand's lane (n = lane & 15,
// g = lane >> 4) holds row/column n and the 8 depth positions 8g..8g+7; a
// result's lane holds column n and rows 4g..4g+3.  Rows of two result tiles
// are numbered 8g + 4*tile + r, so that a lane's rows of both tiles are the 8
// depth positions it must supply when the result is the next product's
// operand: the state and the score matrix go from result to operand in
// registers.  Columns come in pairs, tile 0 the even ones and tile 1 the odd
// ones, so a lane loads and stores 4 bytes per token.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gemv_kernel.h"

namespace mbd {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kScanC = 32;               // tokens per chunk
constexpr float kRange = 40.0f;          // largest |G - r| of a chunk done as products
constexpr float kBig = 1e37f;            // larger factors are taken by the recurrence
// Steps with larger factors (x e^{G-r}, k e^{r-G}) or values are made smaller: a
// factor may be e^kRange times what its terms come to in the result, and the largest
// sum before that is undone, of 32 tokens' factors times a score of two values over
// 256 columns, is then at most 2^(66 + 5 + 23 + 23 + 8).  fp16 values are all smaller.
constexpr float kFactor = 0x1p66f;
constexpr uint32_t kValue = (127 + 23) << 7;   // 2^23 as the bits of a bf16 value

// A (sequence, token, head, channel) tensor: element strides, channels dense.
struct ScanTensor {
  const void* p;
  int64_t sb, sh;
  int32_t st;     // <= 2^24
  int32_t vec;    // channel pairs may be moved as one access
  uint32_t step;  // bytes of a token's stride
  uint32_t full;  // bytes from a chunk's first to behind its last element
};

// A factor m 2^e, m in [0.5, 1) (or 0, infinite or NaN): a segment's decay may be
// far beyond float32 in either direction and its product with a state still be in
// range (128 gates of 0.9 over 1e-15, -120 and then 120 over 1e25).
struct Decay {
  float m;
  int32_t e;
};

struct ScanArgs {
  ScanTensor K, V, G;      // the state's own inputs
  ScanTensor X;            // out: the side multiplied with the state; grad: q (forward) or k
  ScanTensor W;            // grad: do (forward) or v
  ScanTensor O;            // the output
  ScanTensor DG;           // grad, reversed: the gates' gradient
  const int32_t* offsets;  // packed sequences, or null
  int64_t total;           // rows of a packed tensor
  const float* S0;         // state before the first chunk (user layout), or null: zeros
  float* ST;               // state after the last chunk (user layout), or null
  float* slots;            // per segment: its start state, [dkp][dvp]; null: one segment
  Decay* decays;           // state-only: a segment's whole decay, [dkp]
  const float* others;     // grad, forward: the slots of the reversed recurrence, or null
  const float* dST;        // grad, forward: dS_T or null
  float* ends;             // grad: rowsum(S D) at the end of each segment, [dkp]
  float* qdq;              // grad: q dq, (rows, H, dkp) float32
  int64_t t;               // tokens per sequence (the longest, if packed)
  int32_t H, dk, dv, dkp, dvp, nseg, L, nblk, cols;
  int32_t ecol;            // state-only: first of the dv columns that V holds, in the slots
  float kscale, oscale;
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// The bits of x0 and x1 rounded to bf16, packed.
__device__ __forceinline__ uint32_t pack_bf16(float x0, float x1) {
  f32x2 x = {x0, x1};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2));
}
__device__ __forceinline__ float lo16(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
__device__ __forceinline__ float hi16(uint32_t w) { return __builtin_bit_cast(float, w & 0xffff0000u); }

// x0, x1 as N bf16 terms each, packed pairwise.
template <int N>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t (&w)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    w[i] = pack_bf16(x0, x1);
    if (i + 1 < N) {
      x0 -= lo16(w[i]);
      x1 -= hi16(w[i]);
    }
  }
}

// Eight fp32 values as N bf16 operands.
template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[N]) {
  u32x4 w[N];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    uint32_t t[N];
    split2<N>(x[2 * p], x[2 * p + 1], t);
#pragma unroll
    for (int i = 0; i < N; ++i) w[i][p] = t[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = __builtin_bit_cast(bf16x8, w[i]);
}

// One element of a packed 16-bit pair as fp32.
template <int DT>
__device__ __forceinline__ float pair_lo(uint32_t w) {
  if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(f16x2, w).x;
  else return lo16(w);
}
template <int DT>
__device__ __forceinline__ float pair_hi(uint32_t w) {
  if constexpr (DT == DT_F16) return (float)__builtin_bit_cast(f16x2, w).y;
  else return hi16(w);
}
template <int DT>
__device__ __forceinline__ uint32_t pair_round(float x0, float x1) {
  if constexpr (DT == DT_F16) {
    f16x2 h = {(_Float16)x0, (_Float16)x1};
    return __builtin_bit_cast(uint32_t, h);
  } else {
    return pack_bf16(x0, x1);
  }
}

// An operand of 8 values of the tensors' type as bf16 terms: itself (bf16),
// or two terms that hold its 11 bits exactly (f16).
template <int DT> constexpr int kTerms = DT == DT_F16 ? 2 : 1;
template <int DT>
__device__ __forceinline__ void exact_terms(u32x4 raw, bf16x8 (&out)[kTerms<DT>]) {
  if constexpr (DT == DT_F16) {
    float x[8];
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t w = raw[p];
      x[2 * p] = pair_lo<DT>(w);
      x[2 * p + 1] = pair_hi<DT>(w);
    }
    split8<2>(x, out);
  } else {
    out[0] = __builtin_bit_cast(bf16x8, raw);
  }
}

// The same for pairs: a word as one word per term.
template <int DT>
__device__ __forceinline__ void exact_pair(uint32_t w, uint32_t (&out)[kTerms<DT>]) {
  if constexpr (DT == DT_F16) split2<2>(pair_lo<DT>(w), pair_hi<DT>(w), out);
  else out[0] = w;
}

// c += a b, a of NA terms and b of NB terms (largest first): the products of
// terms i and j with i + j < max(NA, NB); the others are below the last one kept.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mfma_terms(const bf16x8 (&a)[NA], const bf16x8 (&b)[NB], f32x4 c) {
  constexpr int M = NA > NB ? NA : NB;
#pragma unroll
  for (int d = M - 1; d >= 0; --d) {
#pragma unroll
    for (int i = 0; i < NA; ++i) {
      const int j = d - i;
      if (j >= 0 && j < NB) c = mfma(a[i], b[j], c);
    }
  }
  return c;
}

// What a lane moves of a tensor: two channels of its 8 tokens, as offsets
// from the chunk's first token.  Offsets behind the chunk's last valid token
// fall out of the descriptor's range: loads give 0, stores do nothing.
struct Lane {
  uint32_t off0, step;   // bytes: channel 0 of the lane's lowest token, token stride
  bool lone;             // channel 1 is behind the last one
};
template <int BYTES>
__device__ __forceinline__ uint32_t off1_of(const Lane& l) {
  return l.lone ? kOffsetOutOfRange : l.off0 + BYTES;   // beyond the range where off0 is
}
template <bool REV>
__device__ __forceinline__ Lane lane_of(const ScanTensor& x, int g, int c0, int width, int bytes) {
  const uint32_t row = (uint32_t)(REV ? 24 - 8 * g : 8 * g) * (uint32_t)x.st;
  Lane l;
  l.off0 = c0 < width ? (row + (uint32_t)c0) * bytes : kOffsetOutOfRange;
  l.lone = c0 + 1 == width;
  l.step = x.step;
  return l;
}
// The first n (at least 1) of the 32 tokens at `at`.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const ScanTensor& x, const char* at, int n) {
  return make_rsrc(at, x.full - (uint32_t)(kScanC - n) * x.step);
}
// To the next chunk in the order of the recurrence.
template <bool REV>
__device__ __forceinline__ void walk(const ScanTensor& x, const char*& at) {
  const uint64_t by = (uint64_t)x.step * kScanC;
  at = REV ? at - by : at + by;
}
// The lane's offsets as the loop's own values: the 8 tokens' offsets are then
// formed where they are used, not kept in 8 registers per tensor over the loop.
__device__ __forceinline__ Lane fresh(Lane l) {
  asm volatile("" : "+v"(l.off0));
  return l;
}
// Token j (0..7) of the lane, in the order of the recurrence.
template <bool REV>
__device__ __forceinline__ uint32_t tok_off(const Lane& l, int j) {
  return (uint32_t)(REV ? 7 - j : j) * l.step;
}
template <bool REV>
__device__ __forceinline__ void load16(__amdgpu_buffer_rsrc_t r, const Lane& kept, int vec, uint32_t (&w)[8]) {
  const Lane l = fresh(kept);
  if (vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, l.off0 + tok_off<REV>(l, j), 0, 0);
  } else {
    const uint32_t off1 = off1_of<2>(l);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = __builtin_amdgcn_raw_buffer_load_b16(r, l.off0 + tok_off<REV>(l, j), 0, 0);
      const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(r, off1 + tok_off<REV>(l, j), 0, 0);
      w[j] = (a & 0xffffu) | (b << 16);
    }
  }
}
template <bool REV>
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, const Lane& l, int vec, int j, uint32_t w) {
  if (vec) {
    __builtin_amdgcn_raw_buffer_store_b32(w, r, l.off0 + tok_off<REV>(l, j), 0, 0);
  } else {
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)w, r, l.off0 + tok_off<REV>(l, j), 0, 0);
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w >> 16), r, off1_of<2>(l) + tok_off<REV>(l, j), 0, 0);
  }
}
// The gates of the lane's two channels: raw words, 8 (16-bit) or 16 (float32).
template <bool G32> constexpr int kGateWords = G32 ? 16 : 8;
template <bool REV, bool G32>
__device__ __forceinline__ void load_gates(__amdgpu_buffer_rsrc_t r, const Lane& kept, int vec,
                                           uint32_t (&w)[kGateWords<G32>]) {
  const Lane l = fresh(kept);
  if constexpr (G32) {
    const uint32_t off1 = off1_of<4>(l);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[2 * j] = __builtin_amdgcn_raw_buffer_load_b32(r, l.off0 + tok_off<REV>(l, j), 0, 0);
      w[2 * j + 1] = __builtin_amdgcn_raw_buffer_load_b32(r, off1 + tok_off<REV>(l, j), 0, 0);
    }
  } else {
    load16<REV>(r, l, vec, w);
  }
}
// Channel c of token j.
template <int DT, bool G32>
__device__ __forceinline__ float gate_value(const uint32_t (&w)[kGateWords<G32>], int c, int j) {
  if constexpr (G32) return __builtin_bit_cast(float, w[2 * j + c]);
  else return c ? pair_hi<DT>(w[j]) : pair_lo<DT>(w[j]);
}

// A chunk's gates for the lane's two channels and 8 tokens.
struct Gates {
  float up[2][8];     // e^{G - r}
  float down[2][8];   // e^{r - G}
  float a[2], b[2];   // e^{r}, e^{end - r}: the whole chunk's decay, in two halves
  bool hard;
};
// Decays are products of the gates' exponentials, from the middle of the chunk
// outwards: an element costs one exponential, one reciprocal and three products.
// A token's factor is within (1.3 |g| + 3) 2^-24: its argument g log2(e) is rounded
// once (and the constant is off by 0.23 2^-24), the exponential is within one unit,
// its product rounds once.  Over the tokens of a decay these add up, for equal
// gates linearly, as in the recurrence itself; a gate of 0 is exact.
template <int DT, bool G32, bool REV>
__device__ __forceinline__ void make_gates(const uint32_t (&w)[kGateWords<G32>], int lane, Gates& q) {
  const int g = lane >> 4;
  float total = 0.0f;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float run = 1.0f, size = 0.0f, P[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x = gate_value<DT, G32>(w, c, j);
      size += __builtin_fabsf(x);
      const float e = __builtin_amdgcn_exp2f(x * 1.44269504f);
      if (REV) P[j] = run;
      run = j == 0 ? e : run * e;
      if (!REV) P[j] = run;
    }
    // the lane groups' products: 0 and 1 before the middle, 2 and 3 behind it
    const float next = __shfl_xor(run, 16, 64), both = run * next;
    const float other = __shfl_xor(both, 32, 64);
    q.a[c] = g < 2 ? both : other;
    q.b[c] = g < 2 ? other : both;
    const float inv = __builtin_amdgcn_rcpf(g == 0 ? both : run);
    const float f = g == 2 ? 1.0f : g == 3 ? next : inv;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      q.up[c][j] = P[j] * f;
      q.down[c][j] = __builtin_amdgcn_rcpf(q.up[c][j]);
    }
    total = __builtin_fmaxf(total, size);
    if (!(size <= kRange)) total = __builtin_inff();   // NaN too
  }
  // |G - r| <= the sum of |g| over one half of the chunk (two lane groups)
  total += __shfl_xor(total, 16, 64);
  q.hard = !(total <= kRange);
}

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// The larger magnitudes of two pairs of 16-bit values, by their bits (NaN the
// largest), and whether a pair holds one that is too large for products or not finite.
__device__ __forceinline__ uint32_t pair_max(uint32_t m, uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, m),
                                                                __builtin_bit_cast(u16x2, w & 0x7fff7fffu)));
}
template <int DT>
__device__ __forceinline__ bool pair_wild(uint32_t m) {
  constexpr uint32_t e = DT == DT_F16 ? 0x7c00u : kValue;
  return (m & 0xffffu) >= e || (m >> 16) >= e;
}

// Two channels' columns (token-major pairs) as channel-major operands.
__device__ __forceinline__ void columns_of(const uint32_t (&w)[8], u32x4& c0, u32x4& c1) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    c0[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x05040100u);
    c1[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x07060302u);
  }
}

// xcd_unit for grids below 2^31.
__device__ __forceinline__ uint32_t xcd_unit32(uint32_t b, uint32_t G) {
  const uint32_t x = b % kXcds, q = G / kXcds, r = G % kXcds;
  return x * q + min(x, r) + b / kXcds;
}

// The sequence, head, segment and block of a workgroup.  Workgroups that read
// the same rows (a segment's blocks) are neighbours on one XCD.
struct Place {
  int seq, h, seg, blk;
  int64_t row0;       // first row of the sequence (packed), else 0
  int64_t b;          // batch index (0 if packed)
  int64_t len;        // tokens of the sequence
  int64_t slot;
  int64_t lo, hi;     // tokens of the segment
  bool last;          // the sequence's last segment
};
__device__ __forceinline__ bool place_of(const ScanArgs& a, Place& p) {
  uint32_t u = (uint32_t)xcd_unit32(blockIdx.x, gridDim.x);
  p.blk = (int)(u % (uint32_t)a.nblk);
  u /= (uint32_t)a.nblk;
  p.slot = u;
  p.seg = (int)(u % (uint32_t)a.nseg);
  u /= (uint32_t)a.nseg;
  p.h = (int)(u % (uint32_t)a.H);
  p.seq = (int)(u / (uint32_t)a.H);
  p.row0 = 0;
  p.b = p.seq;
  p.len = a.t;
  if (a.offsets) {
    // rows outside the tensor are never touched, whatever the offsets say
    const int64_t s = min(max((int64_t)a.offsets[p.seq], (int64_t)0), a.total);
    const int64_t e = min(max((int64_t)a.offsets[p.seq + 1], s), a.total);
    p.row0 = s;
    p.b = 0;
    p.len = min(e - s, a.t);
  }
  p.lo = (int64_t)p.seg * a.L;
  p.hi = min(p.len, p.lo + a.L);
  p.last = p.len <= p.lo + a.L;
  return p.seg == 0 || p.lo < p.len;
}
// The first chunk of the segment in the order of the recurrence.
template <bool REV>
__device__ __forceinline__ const char* base_of(const ScanTensor& x, const Place& p, int bytes) {
  const int64_t tok = p.lo + (REV && p.hi > p.lo ? (p.hi - p.lo - 1) / kScanC * kScanC : 0);
  return (const char*)x.p + (p.b * x.sb + p.h * x.sh + (p.row0 + tok) * (int64_t)x.st) * bytes;
}
// Row `m` of tile `tile` of a result: the token or channel 8 (m / 4) + 4 tile + m % 4.
__device__ __forceinline__ int row_of(int m, int tile) { return 8 * (m >> 2) + 4 * tile + (m & 3); }

constexpr int kPadRow = 8;              // 16-bit elements behind each row of a staged tile
constexpr int kTokRow = kScanC + 8;     // tokens per row of a transposed tile, padded

// The tokens [pos, pos + width) that a step takes: the whole chunk (32), or, where
// the gates or values do not allow it, 8 (those of one lane group) or 1.  A step
// scales the state by its own first half's decay and what the step before left, in
// one product; of a token's decay, which may be anything, that product could leave
// float32's range where the state does not.  A step of one token has all its decay
// before it (forward) or leaves all of it (reversed); where its neighbour there has
// another half of its own, a step of no tokens goes between them.
// `then` of a step of several tokens is the width of the step to be taken first if it
// is refused (forward), or whether a token's decay is left for it (reversed); of a
// step of none the width behind it.
struct Step {
  int pos, width, then;
};
__device__ __forceinline__ bool takes(const Step& t, int g, int j) {
  return (uint32_t)(8 * g + j - t.pos) < (uint32_t)t.width;
}
// What is taken instead of a step of several tokens, the step after `t`, and the
// next chunk's first one.
template <bool REV>
__device__ __forceinline__ void smaller(Step& t, bool refused) {
  if (REV && !refused) t = Step{t.pos, 0, t.width};
  else if (t.width == 32) t.width = 8;
  else t = REV ? Step{t.pos, 1, 0} : Step{t.pos, t.then, 1};
}
template <bool REV>
__device__ __forceinline__ void advance(Step& t) {
  t.pos += t.width;
  if (t.width == 0) t = Step{t.pos, t.then, 0};
  else if ((t.pos & 7) == 0 && t.width == 1) t = Step{t.pos, 8, 1};
  else t.then = 0;
}
__device__ __forceinline__ Step first_step(const Step& before) { return Step{0, 32, before.width == 1 ? 1 : 0}; }
// The words of the step's tokens; others read as 0.
__device__ __forceinline__ void take(const Step& t, int g, const uint32_t (&from)[8], uint32_t (&to)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) to[j] = from[j];
  if (t.width != 32) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!takes(t, g, j)) to[j] = 0u;
  }
}
// d times f.
__device__ __forceinline__ void times(Decay& d, float f) {
  const float m = d.m * f;
  d.m = __builtin_amdgcn_frexp_mantf(m);
  d.e = min(max(d.e + __builtin_amdgcn_frexp_expf(m), -(1 << 28)), 1 << 28);
}
__device__ __forceinline__ void times(Decay& d, Decay f) {
  d.e = min(max(d.e + f.e, -(1 << 28)), 1 << 28);
  times(d, f.m);
}
// x times d.
__device__ __forceinline__ float scaled(float x, Decay d) {
  return d.e > 0 && d.m > 0.0f ? ldexpf(x, d.e - 1) * (2.0f * d.m) : ldexpf(x * d.m, d.e);
}

// Gates of a step: of the chunk, of 8 tokens or none (the others' are 0), or of one
// token, whose decay acts as a whole before it (forward) or after it (reversed)
// and needs no pair of factors -- so it may be 0, infinite or NaN.
template <int DT, bool G32, bool REV>
__device__ __forceinline__ void step_gates(const Step& t, const uint32_t (&gw)[kGateWords<G32>], int lane, Gates& q) {
  const int g = lane >> 4;
  if (t.width == 1) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float x = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        q.up[c][j] = q.down[c][j] = 1.0f;
        x = (t.pos & 7) == j ? gate_value<DT, G32>(gw, c, j) : x;
      }
      x = __shfl(x, 2 * (t.pos & ~7) + (lane & 15), 64);
      q.a[c] = REV ? 1.0f : expf(x);
      q.b[c] = REV ? expf(x) : 1.0f;
    }
    q.hard = false;
    return;
  }
  uint32_t w[kGateWords<G32>];
#pragma unroll
  for (int j = 0; j < kGateWords<G32>; ++j) w[j] = gw[j];
  if (t.width < 32 && (t.width == 0 || g != t.pos >> 3)) {
#pragma unroll
    for (int j = 0; j < kGateWords<G32>; ++j) w[j] = 0u;
  }
  make_gates<DT, G32, REV>(w, lane, q);
}

// The scores of a step are shared: each of the NW waves computes 4 / NW of the
// four 16 x 16 tiles (rows j of tile jt, columns i of tile it), drops what lies
// behind the diagonal and leaves its bf16 terms where the product over j reads
// them: [it][term][lane], a lane's 8 positions j being rows 4g..4g+3 of both jt.
template <int NW> constexpr int kMine = 4 / NW;
template <int NW>
__device__ __forceinline__ void score_tile(int wave, int i, int& jt, int& it) {
  jt = NW == 4 ? wave & 1 : i;
  it = NW == 4 ? wave >> 1 : wave;
}
template <int TERMS>
__device__ __forceinline__ void put_scores(uint8_t* ps, f32x4 x, int jt, int it, int lane) {
  const int n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) x[r] = 8 * g + 4 * jt + r <= row_of(n, it) ? x[r] : 0.0f;
  uint32_t a[TERMS], b[TERMS];
  split2<TERMS>(x[0], x[1], a);
  split2<TERMS>(x[2], x[3], b);
#pragma unroll
  for (int m = 0; m < TERMS; ++m) *(u32x2*)(ps + ((it * TERMS + m) * 64 + lane) * 16 + 8 * jt) = u32x2{a[m], b[m]};
}
template <int TERMS>
__device__ __forceinline__ void get_scores(const uint8_t* ps, int it, int lane, bf16x8 (&x)[TERMS]) {
#pragma unroll
  for (int m = 0; m < TERMS; ++m) x[m] = *(const bf16x8*)(ps + ((it * TERMS + m) * 64 + lane) * 16);
}

// Scores without those of a token with itself.
template <int TERMS>
__device__ __forceinline__ void drop_own(bf16x8 (&x)[TERMS], int it, int lane) {
  const int n = lane & 15, g = lane >> 4;   // token row_of(n, it) is position 4 it + n % 4 of group n / 4
  const uint32_t keep = g != n >> 2 ? 0xffffffffu : n & 1 ? 0x0000ffffu : 0xffff0000u;
#pragma unroll
  for (int m = 0; m < TERMS; ++m) {
    u32x4 w = __builtin_bit_cast(u32x4, x[m]);
    w[2 * it] &= n & 2 ? 0xffffffffu : keep;
    w[2 * it + 1] &= n & 2 ? keep : 0xffffffffu;
    x[m] = __builtin_bit_cast(bf16x8, w);
  }
}

// ---- out_i = X_i^T S ---------------------------------------------------------
// With S the state before the chunk, in units of e^{-r}:
//     out = X' S + tril(X' K'^T) V,  S <- S + K'^T V,  X' = X e^{G-r}, K' = K e^{r-G}
// (reversed the diagonal of the decays belongs to the pair's later token).  A
// wave owns 32 columns of the state (64 VGPRs at DK 128) and of the output; X'
// and K' are computed once per workgroup, 32 channels per wave, and shared
// through LDS as bf16 terms, K' also transposed for the state's update.  Two
// barriers a chunk, the next chunk's loads in flight between them.
//
// Bound by issue and latency at two waves a SIMD: 4 x 2048 tokens, 16 heads of
// 128 x 128 in 8 segments take 75 us (168 MB: 2.2 TB/s; 7.4 us per further chunk
// of all 512 workgroups: 2.8 TB/s), vector units busy half of the time, matrix
// units a quarter.  Three workgroups a CU spill (154 us for 122 in all), and
// transposing LDS reads, rows without bank conflicts and operands read ahead
// change nothing: no part of a chunk's work weighs more than 10 us.  One lone
// workgroup takes 4.4 us a chunk, which bounds short sequences of few heads.

template <int NS>
constexpr size_t scan_out_lds() {
  return (size_t)4 * kScanC * (NS * 32 + kPadRow) * 2 + (size_t)3 * NS * 32 * kTokRow * 2 +
         (size_t)NS * 32 * 4 + 4096 + 64;
}

template <int DT, bool G32, int NS, int NW, bool REV>
__global__ __launch_bounds__(NW * 64, NS > 4 ? 1 : 2) void scan_out_kernel(const ScanArgs a) {
  constexpr int DKP = NS * 32, RS = DKP + kPadRow;
  constexpr int gb = G32 ? 4 : 2;
  constexpr int SL = (NS + NW - 1) / NW;              // slabs of 32 channels a wave stages
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint16_t* xs = (uint16_t*)smem;                     // X e^{G-r}: 2 terms of [32][RS]
  uint16_t* ks = xs + 2 * kScanC * RS;                // K e^{r-G}: 2 terms of [32][RS]
  uint16_t* kt = ks + 2 * kScanC * RS;                // the same, 3 terms of [DKP][kTokRow]
  float* dec = (float*)(kt + 3 * DKP * kTokRow);      // the state's decay before the step, [DKP]
  uint8_t* sc = (uint8_t*)(dec + DKP);                // the scores' terms
  int* wild = (int*)(sc + 4096);                      // one flag per wave

  Place p;
  if (!place_of(a, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int col = p.blk * a.cols + wave * 32 + 2 * n;     // the lane's output columns col, col + 1
  const int vwidth = min(a.dv, (p.blk + 1) * a.cols);

  f32x4 S[NS][2][2];
  if (!a.slots) {
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int d = 32 * s + 8 * g + 4 * tl + r;
            const bool in = a.S0 && d < a.dk && col + nt < vwidth;
            S[s][tl][nt][r] = in ? a.S0[(((int64_t)p.seq * a.H + p.h) * a.dk + d) * a.dv + col + nt] : 0.0f;
          }
  } else {
    const float* slot = a.slots + p.slot * (int64_t)a.dkp * a.dvp;
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int d = 32 * s + 8 * g + 4 * tl + r;
          f32x2 x = {0.0f, 0.0f};
          if (d < a.dkp && col < a.dvp) x = *(const f32x2*)(slot + (int64_t)d * a.dvp + col);
          S[s][tl][0][r] = x[0];
          S[s][tl][1][r] = x[1];
        }
  }

  const char *kb = base_of<REV>(a.K, p, 2), *vb = base_of<REV>(a.V, p, 2), *xb = base_of<REV>(a.X, p, 2),
             *gbp = base_of<REV>(a.G, p, gb), *ob = base_of<REV>(a.O, p, 2);
  const Lane vl = lane_of<REV>(a.V, g, col, vwidth, 2), ol = lane_of<REV>(a.O, g, col, vwidth, 2);
  Lane xl[SL], kl[SL], gl[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int d0 = 32 * (wave + i * NW) + 2 * n;     // beyond dk: nothing is loaded
    xl[i] = lane_of<REV>(a.X, g, d0, a.dk, 2);
    kl[i] = lane_of<REV>(a.K, g, d0, a.dk, 2);
    gl[i] = lane_of<REV>(a.G, g, d0, a.dk, gb);
  }
  const int nch = (int)((p.hi - p.lo + kScanC - 1) / kScanC);
  uint32_t vw[8], xw[SL][8], kw[SL][8], gw[SL][kGateWords<G32>];
  auto fetch = [&](int c) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    const auto gr = chunk_rsrc(a.G, gbp, nv), kr = chunk_rsrc(a.K, kb, nv),
               xr = chunk_rsrc(a.X, xb, nv);
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      load_gates<REV, G32>(gr, gl[i], a.G.vec, gw[i]);
      load16<REV>(kr, kl[i], a.K.vec, kw[i]);
      load16<REV>(xr, xl[i], a.X.vec, xw[i]);
    }
    load16<REV>(chunk_rsrc(a.V, vb, nv), vl, a.V.vec, vw);
    walk<REV>(a.G, gbp);
    walk<REV>(a.K, kb);
    walk<REV>(a.X, xb);
    walk<REV>(a.V, vb);
  };
  if (nch > 0) fetch(0);
  // a step's second half e^{end-r} is left to the next step, which scales the
  // state by both at once
  float left[SL][2], half[SL][2];
#pragma unroll
  for (int i = 0; i < SL; ++i) left[i][0] = left[i][1] = half[i][0] = half[i][1] = 1.0f;
  Step st = {0, 32, REV ? 0 : 1};
  for (int c = 0; c < nch;) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    bool hard = false;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int s = wave + i * NW, d0 = 32 * s + 2 * n;
      if (NS % NW != 0 && s >= NS) break;
      Gates q;
      step_gates<DT, G32, REV>(st, gw[i], lane, q);
      uint32_t xt[8], kv[8], kt3[3][8];
      take(st, g, xw[i], xt);
      take(st, g, kw[i], kv);
      float big = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 8 * g + j;
        const float x0 = pair_lo<DT>(xt[j]) * q.up[0][j], x1 = pair_hi<DT>(xt[j]) * q.up[1][j];
        float k0 = pair_lo<DT>(kv[j]) * q.down[0][j], k1 = pair_hi<DT>(kv[j]) * q.down[1][j];
        if (REV) {
          k0 *= a.kscale;
          k1 *= a.kscale;
        }
        big += (__builtin_fabsf(x0) + __builtin_fabsf(x1)) + (__builtin_fabsf(k0) + __builtin_fabsf(k1));
        uint32_t t[2], u[3];
        split2<2>(x0, x1, t);
        *(uint32_t*)(xs + row * RS + d0) = t[0];
        *(uint32_t*)(xs + (kScanC + row) * RS + d0) = t[1];
        split2<3>(k0, k1, u);
        *(uint32_t*)(ks + row * RS + d0) = u[0];
        *(uint32_t*)(ks + (kScanC + row) * RS + d0) = u[1];
#pragma unroll
        for (int m = 0; m < 3; ++m) kt3[m][j] = u[m];
      }
#pragma unroll
      for (int m = 0; m < 3; ++m) {
        u32x4 c0, c1;
        columns_of(kt3[m], c0, c1);
        *(u32x4*)(kt + (m * DKP + d0) * kTokRow + 8 * g) = c0;
        *(u32x4*)(kt + (m * DKP + d0 + 1) * kTokRow + 8 * g) = c1;
      }
      if (g == 0) {
        // what the step before leaves to be done, and this step's first half
        *(f32x2*)(dec + d0) = f32x2{q.a[0] * left[i][0], q.a[1] * left[i][1]};
      }
      half[i][0] = q.b[0];
      half[i][1] = q.b[1];
      hard |= q.hard || !(big <= kFactor);   // NaN too
    }
    uint32_t vv[8], rawv = 0;
    take(st, g, vw, vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) rawv = pair_max(rawv, vv[j]);
    hard |= pair_wild<DT>(rawv);
    const bool any = __ballot(hard) != 0;
    if (lane == 0) wild[wave] = any;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) all |= wild[w];
    all = __builtin_amdgcn_readfirstlane(all);
    if (st.width > 1 && (all | (REV ? st.then : 0))) {
      smaller<REV>(st, all != 0);
      __syncthreads();
      continue;
    }

#pragma unroll
    for (int i = 0; i < SL; ++i) {
      left[i][0] = half[i][0];
      left[i][1] = half[i][1];
    }
    u32x4 vc[2];
    columns_of(vv, vc[0], vc[1]);
    const Step now = st;
    advance<REV>(st);
    const int next = st.pos == kScanC ? c + 1 : c;
    if (next != c) {
      st = first_step(now);
      if (next < nch) fetch(next);   // in flight during the products
    }
    f32x4 o[2][2] = {};
    f32x4 pt[kMine<NW>] = {};   // this wave's scores, transposed: rows j, columns i
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      bf16x8 xx[2][2];
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          xx[tl][i] = *(const bf16x8*)(xs + (i * kScanC + row_of(n, tl)) * RS + 32 * s + 8 * g);
#pragma unroll
      for (int m = 0; m < kMine<NW>; ++m) {
        int jt, it;
        score_tile<NW>(wave, m, jt, it);
        bf16x8 kk[2], xo[2];   // xo: one of xx again, rather than a choice between registers
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          kk[i] = *(const bf16x8*)(ks + (i * kScanC + row_of(n, jt)) * RS + 32 * s + 8 * g);
          xo[i] = *(const bf16x8*)(xs + (i * kScanC + row_of(n, it)) * RS + 32 * s + 8 * g);
        }
        pt[m] = mfma_terms<2, 2>(kk, xo, pt[m]);
      }
      f32x4 d0 = *(const f32x4*)(dec + 32 * s + 8 * g), d1 = *(const f32x4*)(dec + 32 * s + 8 * g + 4);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        S[s][0][nt] *= d0;
        S[s][1][nt] *= d1;
        float x[8];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = S[s][0][nt][r];
          x[4 + r] = S[s][1][nt][r];
        }
        bf16x8 sx[2];
        split8<2>(x, sx);
#pragma unroll
        for (int it = 0; it < 2; ++it) o[it][nt] = mfma_terms<2, 2>(xx[it], sx, o[it][nt]);
      }
    }
#pragma unroll
    for (int m = 0; m < kMine<NW>; ++m) {
      int jt, it;
      score_tile<NW>(wave, m, jt, it);
      put_scores<2>(sc, pt[m], jt, it, lane);
    }
    bf16x8 vt[2][kTerms<DT>];
    exact_terms<DT>(vc[0], vt[0]);
    exact_terms<DT>(vc[1], vt[1]);
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        bf16x8 kk[3];
#pragma unroll
        for (int i = 0; i < 3; ++i)
          kk[i] = *(const bf16x8*)(kt + (i * DKP + 32 * s + row_of(n, tl)) * kTokRow + 8 * g);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] = mfma_terms(kk, vt[nt], S[s][tl][nt]);
      }
    // from here on the next step may be staged: only the scores are still read,
    // and they are written again behind its own barrier
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      bf16x8 ps[2];
      get_scores<2>(sc, it, lane, ps);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) o[it][nt] = mfma_terms(ps, vt[nt], o[it][nt]);
    }
    const __amdgpu_buffer_rsrc_t orsrc = chunk_rsrc(a.O, ob, nv);
    const Lane ot = fresh(ol);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (now.width == 32 || takes(now, g, j))
        store16<REV>(orsrc, ot, a.O.vec, j,
                     pair_round<DT>(o[j >> 2][0][j & 3] * a.oscale, o[j >> 2][1][j & 3] * a.oscale));
    if (next != c) walk<REV>(a.O, ob);
    c = next;
  }

  if (a.ST && (REV ? p.seg == 0 : p.last)) {
    // the last step's second half
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int s = wave + i * NW;
      if (NS % NW != 0 && s >= NS) break;
      if (g == 0) *(f32x2*)(dec + 32 * s + 2 * n) = f32x2{left[i][0], left[i][1]};
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            const int d = 32 * s + 8 * g + 4 * tl + r;
            if (d < a.dk && col + nt < vwidth)
              a.ST[(((int64_t)p.seq * a.H + p.h) * a.dk + d) * a.dv + col + nt] = S[s][tl][nt][r] * dec[d];
          }
  }
}

// ---- out_i = S W_i ------------------------------------------------------------
// out_i = e^{G_i - r} (S W_i + sum_j tril(W_i . V_j) K'_j), and with it dg.  A token's
// own term (j = i) is the same in q dq and in k dk: it is left out of both and added
// to the output alone.  Under strong gates it is nearly all of them, and the
// rounding that it left behind when it cancelled outweighed dg (gates of -10 to
// -7, 4096 tokens: 0.44 of dg in bf16, 0.010 in float32).
// A wave owns 32 channels (columns of the transposed state, 64 VGPRs at DV
// 128) and their part of the output; K e^{r-G} of its channels never leaves
// its registers.  V and W go through LDS, row-major for the products over DV
// and V also transposed for the state's update.  At the sizes above: dq 88 us
// with q dq left in float32 for the gates' gradient (235 MB: 2.7 TB/s), dk with
// dg 101 us (270 MB), bound as above, and by registers: 10 and 15 a lane are spilled
// in bf16 at four waves of 128 columns, 20..40 with fp16 or float32 gates or two waves
// (the 64-column forms none).

template <int DT, int NV>
constexpr size_t scan_grad_lds() {
  return (size_t)(kTerms<DT> == 1 ? 2 : 4) * kScanC * (NV * 32 + kPadRow) * 2 +
         (size_t)kTerms<DT> * NV * 32 * kTokRow * 2 + 6144 + 64;
}

template <int DT, bool G32, int NV, int NW, bool REV>
__global__ __launch_bounds__(NW * 64, NV > 4 ? 1 : 2) void scan_grad_kernel(const ScanArgs a) {
  constexpr int DVP = NV * 32, RS = DVP + kPadRow;
  constexpr int gb = G32 ? 4 : 2;
  constexpr int SL = (NV + NW - 1) / NW;        // slabs of 32 columns a wave stages
  // terms of the state and the scores: three, as the gates' gradient is a running
  // sum over the segment, and with two its errors show in an fp16 result (256 tokens
  // and more) and in a float32 one at once.  bf16 tensors and gates take two: a
  // term's error is below 2^-17 of it, so over t tokens sqrt(t) 2^-17, half a bf16
  // step only after some 10^5 tokens of one segment (16384 tokens, gates of -5 to -3:
  // 0.00173 of dg, bf16's rounding alone 0.00167; three: 356 for 333 us of
  // gradients of 4 x 2048 tokens, 16 heads of 128 x 128).
  constexpr int TP = G32 || DT == DT_F16 ? 3 : 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint16_t* vs = (uint16_t*)smem;               // V [32][RS]
  uint16_t* ws = vs + kScanC * RS;              // W [32][RS]
  // W as terms of [32][RS]: f16 is converted once a workgroup, not by every wave
  uint16_t* wt2 = kTerms<DT> == 1 ? ws : ws + kScanC * RS;
  uint16_t* vt = wt2 + kTerms<DT> * kScanC * RS;   // V transposed: terms of [DVP][kTokRow]
  uint8_t* sc = (uint8_t*)(vt + kTerms<DT> * DVP * kTokRow);   // the scores' terms
  int* wild = (int*)(sc + 6144);

  Place p;
  if (!place_of(a, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int col = (p.blk * NW + wave) * 32 + 2 * n;       // the lane's channels col, col + 1
  const int64_t head = (int64_t)p.seq * a.H + p.h;
  float* slot = a.slots ? a.slots + p.slot * (int64_t)a.dkp * a.dvp : nullptr;

  f32x4 S[NV][2][2];   // rows: DV, columns: the lane's channels
  auto load_state = [&] {
#pragma unroll
    for (int s = 0; s < NV; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int e = 32 * s + 8 * g + 4 * tl;
          f32x4 x = {};
          if (slot) {
            if (col + nt < a.dkp && e < a.dvp) x = *(const f32x4*)(slot + (int64_t)(col + nt) * a.dvp + e);
          } else if (a.S0 && col + nt < a.dk) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (e + r < a.dv) x[r] = a.S0[(head * a.dk + col + nt) * a.dv + e + r];
          }
          S[s][tl][nt] = x;
        }
  };
  // Behind the first chunk, which is needed before it (forward), or before it (reversed): 15 heads
  // of 64 x 96, 1001 tokens 28.4 us for 30.8, and 32.7 for 36.2.
  if (REV) load_state();

  const char *kb = base_of<REV>(a.K, p, 2), *vb = base_of<REV>(a.V, p, 2), *gbp = base_of<REV>(a.G, p, gb);
  const char *xb = base_of<REV>(a.X, p, 2), *wb = base_of<REV>(a.W, p, 2), *ob = base_of<REV>(a.O, p, 2), *dgb = nullptr;
  // rows of all sequences in one run: (b t + token, h, dkp)
  float* qdq = a.qdq + ((p.b * a.t + p.row0) * a.H + p.h) * a.dkp;
  float carry[2] = {0.0f, 0.0f};
  if (REV) {
    dgb = base_of<REV>(a.DG, p, gb);
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
      if (col + nt < a.dkp) carry[nt] = a.ends[p.slot * a.dkp + col + nt];
  }
  const Lane kl = lane_of<REV>(a.K, g, col, a.dk, 2), gl = lane_of<REV>(a.G, g, col, a.dk, gb);
  const Lane xl = lane_of<REV>(a.X, g, col, a.dk, 2), ol = lane_of<REV>(a.O, g, col, a.dk, 2);
  Lane dl = kl, wl[SL], vl[SL];
  if (REV) dl = lane_of<REV>(a.DG, g, col, a.dk, gb);
#pragma unroll
  for (int i = 0; i < SL; ++i) {
    const int e0 = 32 * (wave + i * NW) + 2 * n;
    vl[i] = lane_of<REV>(a.V, g, e0, a.dv, 2);
    wl[i] = lane_of<REV>(a.W, g, e0, a.dv, 2);
  }

  const int nch = (int)((p.hi - p.lo + kScanC - 1) / kScanC);
  uint32_t kw[8], gw[kGateWords<G32>], vw[SL][8], ww[SL][8];
  auto fetch = [&](int c) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    const auto vr = chunk_rsrc(a.V, vb, nv);
#pragma unroll
    for (int i = 0; i < SL; ++i) load16<REV>(vr, vl[i], a.V.vec, vw[i]);
    const auto wr = chunk_rsrc(a.W, wb, nv);
#pragma unroll
    for (int i = 0; i < SL; ++i) load16<REV>(wr, wl[i], a.W.vec, ww[i]);
    walk<REV>(a.W, wb);
    load_gates<REV, G32>(chunk_rsrc(a.G, gbp, nv), gl, a.G.vec, gw);
    load16<REV>(chunk_rsrc(a.K, kb, nv), kl, a.K.vec, kw);
    walk<REV>(a.V, vb);
    walk<REV>(a.G, gbp);
    walk<REV>(a.K, kb);
  };
  if (nch > 0) fetch(0);
  if (!REV) load_state();
  float left[2] = {1.0f, 1.0f};   // a step's second half e^{end-r}, done with the next step's first
  Step st = {0, 32, REV ? 0 : 1};
  for (int c = 0; c < nch;) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    bool hard = false;
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int s = wave + i * NW, e0 = 32 * s + 2 * n;
      if (NV % NW != 0 && s >= NV) break;
      uint32_t v[8], raw = 0;
      take(st, g, vw[i], v);
      u32x4 c0, c1;
      columns_of(v, c0, c1);
      bf16x8 t0[kTerms<DT>], t1[kTerms<DT>];
      exact_terms<DT>(c0, t0);
      exact_terms<DT>(c1, t1);
#pragma unroll
      for (int m = 0; m < kTerms<DT>; ++m) {
        *(bf16x8*)(vt + (m * DVP + e0) * kTokRow + 8 * g) = t0[m];
        *(bf16x8*)(vt + (m * DVP + e0 + 1) * kTokRow + 8 * g) = t1[m];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        raw = pair_max(raw, v[j]);
        *(uint32_t*)(vs + (8 * g + j) * RS + e0) = v[j];
      }
      take(st, g, ww[i], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        raw = pair_max(raw, v[j]);
        *(uint32_t*)(ws + (8 * g + j) * RS + e0) = v[j];
        if constexpr (kTerms<DT> > 1) {
          uint32_t t[kTerms<DT>];
          exact_pair<DT>(v[j], t);
#pragma unroll
          for (int m = 0; m < kTerms<DT>; ++m) *(uint32_t*)(wt2 + (m * kScanC + 8 * g + j) * RS + e0) = t[m];
        }
      }
      hard |= pair_wild<DT>(raw);
    }
    Gates q;
    step_gates<DT, G32, REV>(st, gw, lane, q);
    bf16x8 kk[2][3];
    {
      uint32_t kv[8];
      float big = 0.0f;
      take(st, g, kw, kv);
      float kf[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        kf[0][j] = pair_lo<DT>(kv[j]) * q.down[0][j];
        kf[1][j] = pair_hi<DT>(kv[j]) * q.down[1][j];
        if (REV) {
          kf[0][j] *= a.kscale;
          kf[1][j] *= a.kscale;
        }
        big += __builtin_fabsf(kf[0][j]) + __builtin_fabsf(kf[1][j]);
      }
      hard |= q.hard || !(big <= kFactor);   // NaN too
      split8<3>(kf[0], kk[0]);
      split8<3>(kf[1], kk[1]);
    }
    const bool any = __ballot(hard) != 0;
    if (lane == 0) wild[wave] = any;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) all |= wild[w];
    all = __builtin_amdgcn_readfirstlane(all);
    if (st.width > 1 && (all | (REV ? st.then : 0))) {
      smaller<REV>(st, all != 0);
      __syncthreads();
      continue;
    }

#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      q.a[nt] *= left[nt];
      left[nt] = q.b[nt];
    }
    uint32_t xw[8];
    load16<REV>(chunk_rsrc(a.X, xb, nv), xl, a.X.vec, xw);
    const Step now = st;
    advance<REV>(st);
    const int next = st.pos == kScanC ? c + 1 : c;
    if (next != c) {
      st = first_step(now);
      if (next < nch) fetch(next);   // in flight during the products
    }
    f32x4 o[2][2] = {};
    f32x4 pt[kMine<NW>] = {};   // this wave's W_i . V_j: rows j, columns i
#pragma unroll
    for (int s = 0; s < NV; ++s) {
      bf16x8 wt[2][kTerms<DT>];
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int m = 0; m < kTerms<DT>; ++m)
          wt[tl][m] = *(const bf16x8*)(wt2 + (m * kScanC + row_of(n, tl)) * RS + 32 * s + 8 * g);
#pragma unroll
      for (int m = 0; m < kMine<NW>; ++m) {
        int jt, it;
        score_tile<NW>(wave, m, jt, it);
        const u32x4 vv = *(const u32x4*)(vs + row_of(n, jt) * RS + 32 * s + 8 * g);
        const u32x4 wv = *(const u32x4*)(ws + row_of(n, it) * RS + 32 * s + 8 * g);
        if constexpr (DT == DT_F16)
          pt[m] = mfma(__builtin_bit_cast(f16x8, vv), __builtin_bit_cast(f16x8, wv), pt[m]);
        else
          pt[m] = mfma(__builtin_bit_cast(bf16x8, vv), __builtin_bit_cast(bf16x8, wv), pt[m]);
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float x[8];
        S[s][0][nt] *= q.a[nt];
        S[s][1][nt] *= q.a[nt];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[r] = S[s][0][nt][r];
          x[4 + r] = S[s][1][nt][r];
        }
        bf16x8 sx[TP];
        split8<TP>(x, sx);
#pragma unroll
        for (int it = 0; it < 2; ++it) o[it][nt] = mfma_terms(wt[it], sx, o[it][nt]);
      }
    }
#pragma unroll
    for (int m = 0; m < kMine<NW>; ++m) {
      int jt, it;
      score_tile<NW>(wave, m, jt, it);
      put_scores<TP>(sc, pt[m], jt, it, lane);
    }
#pragma unroll
    for (int s = 0; s < NV; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        bf16x8 vv[kTerms<DT>];
#pragma unroll
        for (int m = 0; m < kTerms<DT>; ++m)
          vv[m] = *(const bf16x8*)(vt + (m * DVP + 32 * s + row_of(n, tl)) * kTokRow + 8 * g);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] = mfma_terms(vv, kk[nt], S[s][tl][nt]);
      }
    // from here on the next step may be staged: only the scores are still read,
    // and they are written again behind its own barrier
    __syncthreads();
    f32x4 all_o[2][2];   // with a token's own term; o is without
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      bf16x8 ps[TP];
      get_scores<TP>(sc, it, lane, ps);
      const bf16x8 p2[2] = {ps[0], ps[1]};
      drop_own(ps, it, lane);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const bf16x8 k2[2] = {kk[nt][0], kk[nt][1]};
        all_o[it][nt] = mfma_terms(p2, k2, o[it][nt]);
        if constexpr (TP == 3) o[it][nt] = mfma_terms(ps, kk[nt], o[it][nt]);
        else o[it][nt] = mfma_terms(ps, k2, o[it][nt]);
      }
    }
    const __amdgpu_buffer_rsrc_t orsrc = chunk_rsrc(a.O, ob, nv);
    const Lane ot = fresh(ol);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (now.width == 32 || takes(now, g, j))
        store16<REV>(orsrc, ot, a.O.vec, j,
                     pair_round<DT>(all_o[j >> 2][0][j & 3] * q.up[0][j] * a.oscale,
                                    all_o[j >> 2][1][j & 3] * q.up[1][j] * a.oscale));
    float y[2][8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool mine = now.width == 32 || takes(now, g, j);
      y[0][j] = mine ? pair_lo<DT>(xw[j]) * (o[j >> 2][0][j & 3] * q.up[0][j] * a.oscale) : 0.0f;
      y[1][j] = mine ? pair_hi<DT>(xw[j]) * (o[j >> 2][1][j & 3] * q.up[1][j] * a.oscale) : 0.0f;
    }
    // the workspace's rows of this chunk: the lane's tokens are rows of H dkp floats
    float* qr = qdq + tok * a.H * a.dkp + col;
    const int64_t qs = (int64_t)a.H * a.dkp;
    if (!REV) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 8 * g + j;
        if ((now.width == 32 || takes(now, g, j)) && i < nv && col < a.dkp)
          *(f32x2*)(qr + i * qs) = f32x2{y[0][j], y[1][j]};
      }
    } else {
      // dg_t = (the value behind the step) + sum over this and the later tokens of q dq - k dk
      float run[2] = {0.0f, 0.0f}, d[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = 31 - 8 * g - j;
        f32x2 u = {0.0f, 0.0f};
        if ((now.width == 32 || takes(now, g, j)) && i < nv && col < a.dkp) u = *(const f32x2*)(qr + i * qs);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          run[nt] += u[nt] - y[nt][j];
          d[nt][j] = run[nt];
        }
      }
      const __amdgpu_buffer_rsrc_t drsrc = chunk_rsrc(a.DG, dgb, nv);
      const Lane dt = fresh(dl);
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        float s = run[nt];
        const float u = __shfl_up(s, 16, 64);
        if (g >= 1) s += u;
        const float v = __shfl_up(s, 32, 64);
        if (g >= 2) s += v;
        const float before = __shfl_up(s, 16, 64);
        const float base = (g >= 1 ? before : 0.0f) + carry[nt];
        carry[nt] += __shfl(s, 48 + n, 64);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[nt][j] += base;
        // A gate whose factor is 0 has no gradient; the sum's error of the tokens behind it
        // stays there too.  (A NaN goes on.)
        if (now.width == 1 && left[nt] == 0.0f) {
          carry[nt] *= 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) d[nt][j] *= 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (!(now.width == 32 || takes(now, g, j))) continue;
        if constexpr (G32) {
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, d[0][j]), drsrc,
                                                dt.off0 + tok_off<REV>(dt, j), 0, 0);
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, d[1][j]), drsrc,
                                                off1_of<4>(dt) + tok_off<REV>(dt, j), 0, 0);
        } else {
          store16<REV>(drsrc, dt, a.DG.vec, j, pair_round<DT>(d[0][j], d[1][j]));
        }
      }
    }
    if (next != c) {
      walk<REV>(a.X, xb);
      walk<REV>(a.O, ob);
      if (REV) walk<REV>(a.DG, dgb);
    }
    c = next;
  }

  // the last step's second half
#pragma unroll
  for (int s = 0; s < NV; ++s)
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] *= left[nt];
  if (REV) {
    if (a.ST && p.seg == 0) {
#pragma unroll
      for (int s = 0; s < NV; ++s)
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int e = 32 * s + 8 * g + 4 * tl + r;
              if (col + nt < a.dk && e < a.dv) a.ST[(head * a.dk + col + nt) * a.dv + e] = S[s][tl][nt][r];
            }
    }
  } else {
    // rowsum(S D) at the end of the segment
    float w[2] = {0.0f, 0.0f};
    const float* other = a.others ? a.others + p.slot * (int64_t)a.dkp * a.dvp : nullptr;
#pragma unroll
    for (int s = 0; s < NV; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const int e = 32 * s + 8 * g + 4 * tl;
          f32x4 x = {};
          if (other) {
            if (col + nt < a.dkp && e < a.dvp) x = *(const f32x4*)(other + (int64_t)(col + nt) * a.dvp + e);
          } else if (a.dST && col + nt < a.dk) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (e + r < a.dv) x[r] = a.dST[(head * a.dk + col + nt) * a.dv + e + r];
          }
#pragma unroll
          for (int r = 0; r < 4; ++r) w[nt] = __builtin_fmaf(x[r], S[s][tl][nt][r], w[nt]);
        }
#pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      w[nt] += __shfl_xor(w[nt], 16, 64);
      w[nt] += __shfl_xor(w[nt], 32, 64);
      if (g == 0 && col + nt < a.dkp) a.ends[p.slot * a.dkp + col + nt] = w[nt];
    }
  }
}

// ---- a segment's own state ----------------------------------------------------
// From zero, S = sum_t k_t e^{the gates behind t} v_t^T (reversed: q_t do_t^T and
// the gates before it and its own).  The tokens are walked against the order of
// the recurrence, so a token's factor is the running product of what has been
// walked and the sums are never rescaled: no chunk is cut for its gates' sake,
// and a factor that underflows belongs to a contribution that has decayed.
// Where that does not hold -- factors or values beyond kBig, or factors that
// rise again after they were tiny -- the wave does its channels over again as
// the recurrence itself.  The segment's whole decay, for the state at its start,
// is kept with an exponent of its own.  K and its factors stay in a wave's registers, V is
// shared through LDS in two buffers of its terms (f16 is converted once a
// workgroup: 73 us for 83 at 32768 tokens, 8 heads), one barrier a chunk.  Bound
// by HBM: at the sizes above 27 us (88 MB read, 29 MB written: 4.3 TB/s; further
// chunks at 5.1).

template <int DT, int NV>
constexpr size_t scan_state_lds() {
  return (size_t)2 * kTerms<DT> * NV * 32 * kTokRow * 2;
}
constexpr float kTiny = 0x1p-110f;  // factors that get close to float32's end lose bits
constexpr float kRise = 20.0f;      // which matter if they can rise by e^kRise (2^29) again

template <int DT, bool G32, int NV, int NW, bool REV>
__device__ __forceinline__ void own_state(const ScanArgs& a) {
  constexpr int DVP = NV * 32;
  constexpr int gb = G32 ? 4 : 2;
  constexpr int SL = (NV + NW - 1) / NW;        // slabs of 32 columns a wave stages
  constexpr bool DIR = !REV;                    // the order of the walk
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  Place p;
  if (!place_of(a, p)) return;
  // the state at the far end is not a start of any segment
  if (REV ? p.seg == 0 : p.last) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int col = (p.blk * NW + wave) * 32 + 2 * n;       // the lane's channels col, col + 1

  const char *kb = base_of<DIR>(a.K, p, 2), *vb = base_of<DIR>(a.V, p, 2), *gbp = base_of<DIR>(a.G, p, gb);
  const Lane kl = lane_of<DIR>(a.K, g, col, a.dk, 2), gl = lane_of<DIR>(a.G, g, col, a.dk, gb);
  Lane vl[SL];
#pragma unroll
  for (int i = 0; i < SL; ++i) vl[i] = lane_of<DIR>(a.V, g, 32 * (wave + i * NW) + 2 * n, a.dv, 2);
  const int nch = (int)((p.hi - p.lo + kScanC - 1) / kScanC);
  uint32_t kw[8], gw[kGateWords<G32>], vw[SL][8];
  auto fetch = [&](int c) {
    const int64_t tok = p.lo + (int64_t)(DIR ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    const auto vr = chunk_rsrc(a.V, vb, nv);
#pragma unroll
    for (int i = 0; i < SL; ++i) load16<DIR>(vr, vl[i], a.V.vec, vw[i]);
    load_gates<DIR, G32>(chunk_rsrc(a.G, gbp, nv), gl, a.G.vec, gw);
    load16<DIR>(chunk_rsrc(a.K, kb, nv), kl, a.K.vec, kw);
    walk<DIR>(a.V, vb);
    walk<DIR>(a.G, gbp);
    walk<DIR>(a.K, kb);
  };
  if (nch > 0) fetch(0);
  f32x4 S[NV][2][2] = {};               // rows: DV, columns: the lane's channels
  float run[2] = {1.0f, 1.0f};          // the walked gates' decay
  float low = 1.0f, rise = 0.0f, big = 0.0f;
  Decay whole[2] = {{0.5f, 1}, {0.5f, 1}};   // of the lane's tokens
  for (int c = 0; c < nch; ++c) {
    uint16_t* vt = (uint16_t*)smem + (c & 1) * kTerms<DT> * DVP * kTokRow;   // V transposed: terms of [DVP][kTokRow]
#pragma unroll
    for (int i = 0; i < SL; ++i) {
      const int s = wave + i * NW, e0 = 32 * s + 2 * n;
      if (NV % NW != 0 && s >= NV) break;
      u32x4 c0, c1;
      columns_of(vw[i], c0, c1);
      bf16x8 t0[kTerms<DT>], t1[kTerms<DT>];
      exact_terms<DT>(c0, t0);
      exact_terms<DT>(c1, t1);
#pragma unroll
      for (int m = 0; m < kTerms<DT>; ++m) {
        *(bf16x8*)(vt + (m * DVP + e0) * kTokRow + 8 * g) = t0[m];
        *(bf16x8*)(vt + (m * DVP + e0 + 1) * kTokRow + 8 * g) = t1[m];
      }
    }
    bf16x8 kk[2][3];
    float top = 0.0f;
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
      float P[8], of = 1.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = gate_value<DT, G32>(gw, ch, j);
        top = __builtin_fmaxf(top, x);
        const float e = __builtin_amdgcn_exp2f(x * 1.44269504f);
        if (DIR) P[j] = of;
        of = j == 0 ? e : of * e;
        if (!DIR) P[j] = of;
      }
      if (of >= 0x1p-120f) {
        times(whole[ch], of);
      } else {   // (or NaN) the product has lost bits, the factors have not
#pragma unroll
        for (int j = 0; j < 8; ++j) times(whole[ch], expf(gate_value<DT, G32>(gw, ch, j)));
      }
      // times the groups walked before this one, and the chunks before
      const float next = __shfl_xor(of, 16, 64), both = of * next;
      const float other = __shfl_xor(both, 32, 64);
      const float f = run[ch] * ((g & 1 ? next : 1.0f) * (g & 2 ? other : 1.0f));
      run[ch] *= both * other;
      float kf[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = P[j] * f;
        low = __builtin_fminf(low, x);
        kf[j] = (ch ? pair_hi<DT>(kw[j]) : pair_lo<DT>(kw[j])) * x;
        if (REV) kf[j] *= a.kscale;
        big += __builtin_fabsf(kf[j]);
      }
      split8<3>(kf, kk[ch]);
      if (!(run[ch] <= kBig)) big = __builtin_inff();   // NaN too
    }
    rise += 8.0f * top;
    // one buffer is staged while the other is read: its last readers are behind
    // the barrier before this one
    __syncthreads();
    if (c + 1 < nch) fetch(c + 1);   // in flight during the products
#pragma unroll
    for (int s = 0; s < NV; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) {
        bf16x8 vv[kTerms<DT>];
#pragma unroll
        for (int m = 0; m < kTerms<DT>; ++m)
          vv[m] = *(const bf16x8*)(vt + (m * DVP + 32 * s + row_of(n, tl)) * kTokRow + 8 * g);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] = mfma_terms(vv, kk[nt], S[s][tl][nt]);
      }
  }

  rise += __shfl_xor(rise, 16, 64);   // of all the chunk's tokens
  rise += __shfl_xor(rise, 32, 64);
  low = __builtin_fminf(low, __shfl_xor(low, 16, 64));
  low = __builtin_fminf(low, __shfl_xor(low, 32, 64));
#pragma unroll
  for (int ch = 0; ch < 2; ++ch)
#pragma unroll
    for (int x = 16; x <= 32; x *= 2) times(whole[ch], Decay{__shfl_xor(whole[ch].m, x, 64), __shfl_xor(whole[ch].e, x, 64)});
  if (__ballot(!(big <= kBig) || (rise > kRise && low < kTiny))) {
    const char *k1 = (const char*)a.K.p, *v1 = (const char*)a.V.p, *g1 = (const char*)a.G.p;
    whole[0] = whole[1] = Decay{0.5f, 1};
#pragma unroll
    for (int s = 0; s < NV; ++s)
#pragma unroll
      for (int tl = 0; tl < 2; ++tl) S[s][tl][0] = S[s][tl][1] = f32x4{};
    for (int64_t i = 0; i < p.hi - p.lo; ++i) {
      const int64_t tok = p.row0 + (REV ? p.hi - 1 - i : p.lo + i);
      const uint16_t* kr = (const uint16_t*)k1 + (p.b * a.K.sb + p.h * a.K.sh + tok * a.K.st);
      const uint16_t* vr = (const uint16_t*)v1 + (p.b * a.V.sb + p.h * a.V.sh + tok * a.V.st);
      const char* gr = g1 + (p.b * a.G.sb + p.h * a.G.sh + tok * a.G.st) * gb;
      float ex[2], k[2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        ex[nt] = 1.0f;
        k[nt] = 0.0f;
        if (col + nt < a.dk) {
          k[nt] = widen<DT>(kr[col + nt]) * (REV ? a.kscale : 1.0f);
          ex[nt] = expf(G32 ? ((const float*)gr)[col + nt] : widen<DT>(((const uint16_t*)gr)[col + nt]));
        }
        times(whole[nt], ex[nt]);
      }
#pragma unroll
      for (int s = 0; s < NV; ++s)
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int e = 32 * s + 8 * g + 4 * tl + r;
            const float v = e < a.dv ? widen<DT>(vr[e]) : 0.0f;
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const float x = S[s][tl][nt][r];
              S[s][tl][nt][r] = REV ? __builtin_fmaf(k[nt], v, x) * ex[nt] : __builtin_fmaf(k[nt], v, x * ex[nt]);
            }
          }
    }
  }

  float* slot = a.slots + p.slot * (int64_t)a.dkp * a.dvp;
#pragma unroll
  for (int s = 0; s < NV; ++s)
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int e = 32 * s + 8 * g + 4 * tl;
        if (col + nt < a.dkp && a.ecol + e < a.dvp)
          *(f32x4*)(slot + (int64_t)(col + nt) * a.dvp + a.ecol + e) = S[s][tl][nt];
      }
  if (g == 0)
#pragma unroll
    for (int nt = 0; nt < 2; ++nt)
      if (col + nt < a.dkp) a.decays[p.slot * a.dkp + col + nt] = whole[nt];
}

// The two recurrences of a backward pass side by side (grid y), or the forward one alone.
struct StateArgs {
  ScanArgs fwd, rev;
};
template <int DT, bool G32, int NV, int NW>
__global__ __launch_bounds__(NW * 64, 2) void scan_state_kernel(const StateArgs a) {
  if (blockIdx.y == 0) own_state<DT, G32, NV, NW, false>(a.fwd);
  else own_state<DT, G32, NV, NW, true>(a.rev);
}

}  // namespace mbd
