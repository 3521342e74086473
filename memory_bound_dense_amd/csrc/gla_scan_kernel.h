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
// (the last because rowsum(S_t D_t) = dg_t + k_t dk_t = dg_{t+1} + q_t dq_t).
// Reversed, a recurrence differs from the forward one only in its order and
// in that a token's gate acts after the token instead of before it, so two
// kernels serve everything:
//   scan_out_kernel    out_i  = X_i^T S     o  (K k, V v, X q), dv (K q, V do, X k)
//   scan_grad_kernel   out_i  = S W_i       dq (K k, V v, W do), dk (K q, V do, W v)
//
// A chunk of 32 tokens is one step.  With G the running sum of the gates in
// the chunk and r its value at the middle, the chunk is matrix products of
// x e^{G-r} and k e^{r-G}: their product is the decay e^{G_i - G_j} of every
// pair, and |G - r| <= kRange keeps each factor far from overflow.  Chunks
// where it does not hold (very strong gates, gates of -inf that clear the
// state) and chunks with values that are not finite take the recurrence
// itself, token by token, in the same registers; there a masked pair is
// never formed, so nothing leaks from a later token into an earlier one.
//
// Precision: the products run on bf16 matrix instructions with fp32 sums, and
// every fp32 factor enters as a sum of bf16 terms -- two (2^-17 relative) where
// the result is rounded to 16 bits right after, three (2^-25) where it goes
// into the fp32 state or the gates' gradient, which is a difference of sums.
// q, k, v and do are exact in one term (bf16) or two (f16).
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
constexpr uint32_t kBigBits = 0x7cf0bdc2u;   // 1e37f: larger factors (and NaN) are left to the recurrence

// A (sequence, token, head, channel) tensor: element strides, channels dense.
struct ScanTensor {
  const void* p;
  int64_t sb, sh;
  int32_t st;     // <= 2^24
  int32_t vec;    // channel pairs may be moved as one access
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
  float* sums;             // state-only: sum of the gates of a segment, [dkp]
  const float* others;     // grad, forward: the slots of the reversed recurrence, or null
  const float* dST;        // grad, forward: dS_T or null
  float* ends;             // grad: rowsum(S D) at the end of each segment, [dkp]
  float* qdq;              // grad: q dq, (rows, H, dkp) float32
  int64_t t;               // tokens per sequence (the longest, if packed)
  int32_t H, dk, dv, dkp, dvp, nseg, L, nblk, cols, g32, go32;
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
  uint32_t off0, off1, step;   // bytes: channel 0, channel 1 (of the lane's lowest token), token stride
};
template <bool REV>
__device__ __forceinline__ Lane lane_of(const ScanTensor& x, int g, int c0, int width, int bytes) {
  const uint32_t row = (uint32_t)(REV ? 24 - 8 * g : 8 * g) * (uint32_t)x.st;
  Lane l;
  l.off0 = c0 < width ? (row + (uint32_t)c0) * bytes : kOffsetOutOfRange;
  l.off1 = c0 + 1 < width ? (row + (uint32_t)c0 + 1u) * bytes : kOffsetOutOfRange;
  l.step = (uint32_t)x.st * bytes;
  return l;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rsrc(const ScanTensor& x, const char* base, int64_t tok,
                                                             int n, int width, int bytes) {
  // n valid tokens from tok on (none: an empty range)
  const uint32_t len = n > 0 ? ((uint32_t)(n - 1) * (uint32_t)x.st + (uint32_t)width) * bytes : 0u;
  return make_rsrc(base + tok * (int64_t)x.st * bytes, len);
}
// Token j (0..7) of the lane, in the order of the recurrence.
template <bool REV>
__device__ __forceinline__ uint32_t tok_off(const Lane& l, int j) {
  return (uint32_t)(REV ? 7 - j : j) * l.step;
}
template <bool REV>
__device__ __forceinline__ void load16(__amdgpu_buffer_rsrc_t r, const Lane& l, int vec, uint32_t (&w)[8]) {
  if (vec) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = __builtin_amdgcn_raw_buffer_load_b32(r, l.off0 + tok_off<REV>(l, j), 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t a = __builtin_amdgcn_raw_buffer_load_b16(r, l.off0 + tok_off<REV>(l, j), 0, 0);
      const uint32_t b = __builtin_amdgcn_raw_buffer_load_b16(r, l.off1 + tok_off<REV>(l, j), 0, 0);
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
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)(w >> 16), r, l.off1 + tok_off<REV>(l, j), 0, 0);
  }
}
// The gates of the lane's two channels: raw words, 8 (16-bit) or 16 (float32).
template <bool REV>
__device__ __forceinline__ void load_gates(__amdgpu_buffer_rsrc_t r, const Lane& l, int vec, int g32,
                                           uint32_t (&w)[16]) {
  if (g32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[2 * j] = __builtin_amdgcn_raw_buffer_load_b32(r, l.off0 + tok_off<REV>(l, j), 0, 0);
      w[2 * j + 1] = __builtin_amdgcn_raw_buffer_load_b32(r, l.off1 + tok_off<REV>(l, j), 0, 0);
    }
  } else {
    uint32_t p[8];
    load16<REV>(r, l, vec, p);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = p[j];
  }
}

// A chunk's gates for the lane's two channels and 8 tokens.
struct Gates {
  float up[2][8];     // e^{G - r}
  float down[2][8];   // e^{r - G}
  float a[2], b[2];   // e^{r}, e^{end - r}: the whole chunk's decay, in two halves
  float sum[2];       // end
  bool hard;
};
template <int DT>
__device__ __forceinline__ void gate_values(const uint32_t (&w)[16], int g32, float (&x)[2][8]) {
  if (g32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[0][j] = __builtin_bit_cast(float, w[2 * j]);
      x[1][j] = __builtin_bit_cast(float, w[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[0][j] = pair_lo<DT>(w[j]);
      x[1][j] = pair_hi<DT>(w[j]);
    }
  }
}
// e^x to fp32 rounding for |x| <= kRange: the product x log2(e) in two parts.
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * 1.44269502f;
  const float lo = __builtin_fmaf(x, 1.44269502f, -y) + x * 1.92596299e-8f;
  const float p = __builtin_amdgcn_exp2f(y);
  return __builtin_fmaf(p, lo * 0.693147182f, p);
}
template <bool REV>
__device__ __forceinline__ void make_gates(const float (&x)[2][8], int lane, Gates& q) {
  const int g = lane >> 4;
  q.hard = false;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float run = 0.0f, G[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (REV) G[j] = run;
      run += x[c][j];
      if (!REV) G[j] = run;
    }
    float a = run;
    const float u = __shfl_up(a, 16, 64);
    if (g >= 1) a += u;
    const float v = __shfl_up(a, 32, 64);
    if (g >= 2) a += v;
    const float before = __shfl_up(a, 16, 64);
    const float mid = __shfl(a, 16 + (lane & 15), 64);
    const float end = __shfl(a, 48 + (lane & 15), 64);
    const float base = g >= 1 ? before : 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = (base + G[j]) - mid;
      q.hard |= !(__builtin_fabsf(d) <= kRange);
      q.up[c][j] = exp_of(d);
      q.down[c][j] = exp_of(-d);
    }
    q.hard |= !(mid <= kRange) || !(end - mid <= kRange);
    q.a[c] = expf(mid);
    q.b[c] = expf(end - mid);
    q.sum[c] = end;
  }
}

__device__ __forceinline__ uint32_t mag(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
// Whether a pair of 16-bit values holds one that is not finite.
template <int DT>
__device__ __forceinline__ bool pair_wild(uint32_t w) {
  constexpr uint32_t e = DT == DT_F16 ? 0x7c00u : 0x7f80u;
  return (w & e) == e || ((w >> 16) & e) == e;
}

// Two channels' columns (token-major pairs) as channel-major operands.
__device__ __forceinline__ void columns_of(const uint32_t (&w)[8], u32x4& c0, u32x4& c1) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    c0[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x05040100u);
    c1[p] = __builtin_amdgcn_perm(w[2 * p + 1], w[2 * p], 0x07060302u);
  }
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
  int64_t u = xcd_unit(blockIdx.x, gridDim.x);
  p.blk = (int)(u % a.nblk);
  u /= a.nblk;
  p.slot = u;
  p.seg = (int)(u % a.nseg);
  u /= a.nseg;
  p.h = (int)(u % a.H);
  p.seq = (int)(u / a.H);
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
__device__ __forceinline__ const char* base_of(const ScanTensor& x, const Place& p, int bytes) {
  return (const char*)x.p + (p.b * x.sb + p.h * x.sh + p.row0 * (int64_t)x.st) * bytes;
}
// Row `m` of tile `tile` of a result: the token or channel 8 (m / 4) + 4 tile + m % 4.
__device__ __forceinline__ int row_of(int m, int tile) { return 8 * (m >> 2) + 4 * tile + (m & 3); }

constexpr int kPadRow = 8;              // 16-bit elements behind each row of a staged tile
constexpr int kTokRow = kScanC + 8;     // tokens per row of a transposed tile, padded

// ---- out_i = X_i^T S ---------------------------------------------------------
// A wave owns 32 columns of the state (64 VGPRs at DK 128) and of the output;
// X e^{G-r} and K e^{r-G} are computed once per workgroup, 32 channels per
// wave, and shared through LDS as bf16 terms.

template <int NS>
constexpr size_t scan_out_lds() {
  return (size_t)4 * kScanC * (NS * 32 + kPadRow) * 2 + (size_t)3 * NS * 32 * kTokRow * 2 +
         (size_t)2 * NS * 32 * 4 + 64;
}

template <int DT, int NS, int NW, bool REV>
__global__ __launch_bounds__(NW * 64, 2) void scan_out_kernel(const ScanArgs a) {
  constexpr int DKP = NS * 32, RS = DKP + kPadRow;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint16_t* xs = (uint16_t*)smem;                     // X e^{G-r}: 2 terms of [32][RS]
  uint16_t* ks = xs + 2 * kScanC * RS;                // K e^{r-G}: 2 terms of [32][RS]
  uint16_t* kt = ks + 2 * kScanC * RS;                // the same, 3 terms of [DKP][kTokRow]
  float* dec = (float*)(kt + 3 * DKP * kTokRow);      // e^{r} [DKP], e^{end-r} [DKP]
  int* wild = (int*)(dec + 2 * DKP);                  // one flag per wave
  float* seqx = (float*)smem;                         // token by token: X, K, e^g as [32][DKP] each

  Place p;
  if (!place_of(a, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int col = p.blk * a.cols + wave * 32 + 2 * n;     // the lane's output columns col, col + 1
  const int vwidth = min(a.dv, (p.blk + 1) * a.cols);
  const int gb = a.g32 ? 4 : 2;

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

  const char *kb = base_of(a.K, p, 2), *vb = base_of(a.V, p, 2), *xb = base_of(a.X, p, 2),
             *gbp = base_of(a.G, p, gb), *ob = base_of(a.O, p, 2);
  const Lane vl = lane_of<REV>(a.V, g, col, vwidth, 2), ol = lane_of<REV>(a.O, g, col, vwidth, 2);

  const int nch = (int)((p.hi - p.lo + kScanC - 1) / kScanC);
  for (int c = 0; c < nch; ++c) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    bool hard = false;
    uint32_t vw[8];
    load16<REV>(chunk_rsrc(a.V, vb, tok, nv, a.dv, 2), vl, a.V.vec, vw);
    // the staged slabs of 32 channels
    for (int s = wave; s < NS; s += NW) {
      const int d0 = 32 * s + 2 * n;
      uint32_t xw[8], kw[8], gw[16];
      const Lane xl = lane_of<REV>(a.X, g, d0, a.dk, 2), kl = lane_of<REV>(a.K, g, d0, a.dk, 2),
                 gl = lane_of<REV>(a.G, g, d0, a.dk, gb);
      load_gates<REV>(chunk_rsrc(a.G, gbp, tok, nv, a.dk, gb), gl, a.G.vec, a.g32, gw);
      load16<REV>(chunk_rsrc(a.K, kb, tok, nv, a.dk, 2), kl, a.K.vec, kw);
      load16<REV>(chunk_rsrc(a.X, xb, tok, nv, a.dk, 2), xl, a.X.vec, xw);
      float gv[2][8];
      gate_values<DT>(gw, a.g32, gv);
      Gates q;
      make_gates<REV>(gv, lane, q);
      float kf[2][8];
      uint32_t big = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int row = 8 * g + j;
        const float x0 = pair_lo<DT>(xw[j]) * q.up[0][j], x1 = pair_hi<DT>(xw[j]) * q.up[1][j];
        kf[0][j] = pair_lo<DT>(kw[j]) * a.kscale * q.down[0][j];
        kf[1][j] = pair_hi<DT>(kw[j]) * a.kscale * q.down[1][j];
        big = max(max(big, max(mag(x0), mag(x1))), max(mag(kf[0][j]), mag(kf[1][j])));
        uint32_t t[2];
        split2<2>(x0, x1, t);
        *(uint32_t*)(xs + row * RS + d0) = t[0];
        *(uint32_t*)(xs + (kScanC + row) * RS + d0) = t[1];
        split2<2>(kf[0][j], kf[1][j], t);
        *(uint32_t*)(ks + row * RS + d0) = t[0];
        *(uint32_t*)(ks + (kScanC + row) * RS + d0) = t[1];
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        bf16x8 t[3];
        split8<3>(kf[nt], t);
#pragma unroll
        for (int i = 0; i < 3; ++i) *(bf16x8*)(kt + (i * DKP + d0 + nt) * kTokRow + 8 * g) = t[i];
        if (g == 0) {
          dec[d0 + nt] = q.a[nt];
          dec[DKP + d0 + nt] = q.b[nt];
        }
      }
      hard |= q.hard || big > kBigBits;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) hard |= pair_wild<DT>(vw[j]);
    const bool any = __ballot(hard) != 0;
    if (lane == 0) wild[wave] = any;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) all |= wild[w];

    f32x4 o[2][2] = {};
    if (!__builtin_amdgcn_readfirstlane(all)) {
      f32x4 pt[2][2] = {};   // scores, transposed: rows j, columns i
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        bf16x8 kk[2][2], xx[2][2];
#pragma unroll
        for (int tl = 0; tl < 2; ++tl)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            kk[tl][i] = *(const bf16x8*)(ks + (i * kScanC + row_of(n, tl)) * RS + 32 * s + 8 * g);
            xx[tl][i] = *(const bf16x8*)(xs + (i * kScanC + row_of(n, tl)) * RS + 32 * s + 8 * g);
          }
#pragma unroll
        for (int jt = 0; jt < 2; ++jt)
#pragma unroll
          for (int it = 0; it < 2; ++it) pt[jt][it] = mfma_terms<2, 2>(kk[jt], xx[it], pt[jt][it]);
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
          bf16x8 st[2];
          split8<2>(x, st);
#pragma unroll
          for (int it = 0; it < 2; ++it) o[it][nt] = mfma_terms<2, 2>(xx[it], st, o[it][nt]);
        }
      }
      u32x4 vc[2];
      columns_of(vw, vc[0], vc[1]);
      bf16x8 vt[2][kTerms<DT>];
      exact_terms<DT>(vc[0], vt[0]);
      exact_terms<DT>(vc[1], vt[1]);
#pragma unroll
      for (int it = 0; it < 2; ++it) {
        float x[8];
#pragma unroll
        for (int jt = 0; jt < 2; ++jt)
#pragma unroll
          for (int r = 0; r < 4; ++r) x[4 * jt + r] = 8 * g + 4 * jt + r <= row_of(n, it) ? pt[jt][it][r] : 0.0f;
        bf16x8 ps[2];
        split8<2>(x, ps);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) o[it][nt] = mfma_terms(ps, vt[nt], o[it][nt]);
      }
#pragma unroll
      for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
          bf16x8 kk[3];
#pragma unroll
          for (int i = 0; i < 3; ++i)
            kk[i] = *(const bf16x8*)(kt + (i * DKP + 32 * s + row_of(n, tl)) * kTokRow + 8 * g);
          const f32x4 d = *(const f32x4*)(dec + DKP + 32 * s + 8 * g + 4 * tl);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] = mfma_terms(kk, vt[nt], S[s][tl][nt]) * d;
        }
    } else {
      // the recurrence itself: X, K and e^g of the chunk in fp32 through LDS
      __syncthreads();
      for (int s = wave; s < NS; s += NW) {
        const int d0 = 32 * s + 2 * n;
        uint32_t xw[8], kw[8], gw[16];
        const Lane xl = lane_of<REV>(a.X, g, d0, a.dk, 2), kl = lane_of<REV>(a.K, g, d0, a.dk, 2),
                   gl = lane_of<REV>(a.G, g, d0, a.dk, gb);
        load_gates<REV>(chunk_rsrc(a.G, gbp, tok, nv, a.dk, gb), gl, a.G.vec, a.g32, gw);
        load16<REV>(chunk_rsrc(a.K, kb, tok, nv, a.dk, 2), kl, a.K.vec, kw);
        load16<REV>(chunk_rsrc(a.X, xb, tok, nv, a.dk, 2), xl, a.X.vec, xw);
        float gv[2][8];
        gate_values<DT>(gw, a.g32, gv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float* to = seqx + (8 * g + j) * DKP + d0;
          *(f32x2*)to = f32x2{pair_lo<DT>(xw[j]), pair_hi<DT>(xw[j])};
          *(f32x2*)(to + kScanC * DKP) = f32x2{pair_lo<DT>(kw[j]) * a.kscale, pair_hi<DT>(kw[j]) * a.kscale};
          *(f32x2*)(to + 2 * kScanC * DKP) = f32x2{expf(gv[0][j]), expf(gv[1][j])};
        }
      }
      __syncthreads();
      for (int tg = 0; tg < 4; ++tg) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float* from = seqx + (8 * tg + j) * DKP;
          const uint32_t w = __shfl(vw[j], 16 * tg + n, 64);
          const float v0 = pair_lo<DT>(w), v1 = pair_hi<DT>(w);
          // a token behind the end changes nothing (its gate and k are 0)
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
              const int d = 32 * s + 8 * g + 4 * tl;
              const f32x4 x = *(const f32x4*)(from + d), k = *(const f32x4*)(from + kScanC * DKP + d),
                          e = *(const f32x4*)(from + 2 * kScanC * DKP + d);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                float y0 = S[s][tl][0][r], y1 = S[s][tl][1][r];
                if (!REV) {
                  y0 *= e[r];
                  y1 *= e[r];
                }
                y0 = __builtin_fmaf(k[r], v0, y0);
                y1 = __builtin_fmaf(k[r], v1, y1);
                s0 = __builtin_fmaf(x[r], y0, s0);
                s1 = __builtin_fmaf(x[r], y1, s1);
                if (REV) {
                  y0 *= e[r];
                  y1 *= e[r];
                }
                S[s][tl][0][r] = y0;
                S[s][tl][1][r] = y1;
              }
            }
          s0 += __shfl_xor(s0, 16, 64);
          s1 += __shfl_xor(s1, 16, 64);
          s0 += __shfl_xor(s0, 32, 64);
          s1 += __shfl_xor(s1, 32, 64);
          if (g == tg) {
            o[j >> 2][0][j & 3] = s0;
            o[j >> 2][1][j & 3] = s1;
          }
        }
      }
    }
    const __amdgpu_buffer_rsrc_t orsrc = chunk_rsrc(a.O, ob, tok, nv, a.dv, 2);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      store16<REV>(orsrc, ol, a.O.vec, j,
                   pair_round<DT>(o[j >> 2][0][j & 3] * a.oscale, o[j >> 2][1][j & 3] * a.oscale));
    __syncthreads();
  }

  if (a.ST && (REV ? p.seg == 0 : p.last)) {
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
              a.ST[(((int64_t)p.seq * a.H + p.h) * a.dk + d) * a.dv + col + nt] = S[s][tl][nt][r];
          }
  }
}

// ---- out_i = S W_i, and a segment's own state -------------------------------
// A wave owns 32 channels (columns of the transposed state, 64 VGPRs at DV
// 128) and their part of the output; K e^{r-G} of its channels never leaves
// its registers.  V and W go through LDS, row-major for the products over DV
// and V also transposed for the state's update.

template <int NV>
constexpr size_t scan_grad_lds() {
  return (size_t)2 * kScanC * (NV * 32 + kPadRow) * 2 + (size_t)NV * 32 * kTokRow * 2 + 64;
}

template <int DT, int NV, int NW, bool REV, bool GRAD>
__global__ __launch_bounds__(NW * 64, 2) void scan_grad_kernel(const ScanArgs a) {
  constexpr int DVP = NV * 32, RS = DVP + kPadRow;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  uint16_t* vs = (uint16_t*)smem;               // V [32][RS]
  uint16_t* ws = vs + kScanC * RS;              // W [32][RS]
  uint16_t* vt = ws + kScanC * RS;              // V transposed [DVP][kTokRow]
  int* wild = (int*)(vt + DVP * kTokRow);

  Place p;
  if (!place_of(a, p)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n = lane & 15, g = lane >> 4;
  const int col = (p.blk * NW + wave) * 32 + 2 * n;       // the lane's channels col, col + 1
  const int gb = a.g32 ? 4 : 2, gob = a.go32 ? 4 : 2;
  const int64_t head = (int64_t)p.seq * a.H + p.h;
  float* slot = a.slots ? a.slots + p.slot * (int64_t)a.dkp * a.dvp : nullptr;

  f32x4 S[NV][2][2];   // rows: DV, columns: the lane's channels
#pragma unroll
  for (int s = 0; s < NV; ++s)
#pragma unroll
    for (int tl = 0; tl < 2; ++tl)
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const int e = 32 * s + 8 * g + 4 * tl;
        f32x4 x = {};
        if (GRAD) {
          if (slot) {
            if (col + nt < a.dkp && e < a.dvp) x = *(const f32x4*)(slot + (int64_t)(col + nt) * a.dvp + e);
          } else if (a.S0 && col + nt < a.dk) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (e + r < a.dv) x[r] = a.S0[(head * a.dk + col + nt) * a.dv + e + r];
          }
        }
        S[s][tl][nt] = x;
      }

  const char *kb = base_of(a.K, p, 2), *vb = base_of(a.V, p, 2), *gbp = base_of(a.G, p, gb);
  const char *xb = nullptr, *wb = nullptr, *ob = nullptr, *dgb = nullptr;
  float* qdq = nullptr;
  float carry[2] = {0.0f, 0.0f}, gsum[2] = {0.0f, 0.0f};
  if (GRAD) {
    xb = base_of(a.X, p, 2);
    wb = base_of(a.W, p, 2);
    ob = base_of(a.O, p, 2);
    if (REV) dgb = base_of(a.DG, p, gob);
    // rows of all sequences in one run: (b t + token, h, dkp)
    qdq = a.qdq + ((p.b * a.t + p.row0) * a.H + p.h) * a.dkp;
    if (REV) {
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        if (col + nt < a.dkp) carry[nt] = a.ends[p.slot * a.dkp + col + nt];
    }
  }
  const Lane kl = lane_of<REV>(a.K, g, col, a.dk, 2), gl = lane_of<REV>(a.G, g, col, a.dk, gb);

  const int nch = (int)((p.hi - p.lo + kScanC - 1) / kScanC);
  for (int c = 0; c < nch; ++c) {
    const int64_t tok = p.lo + (int64_t)(REV ? nch - 1 - c : c) * kScanC;
    const int nv = (int)min((int64_t)kScanC, p.hi - tok);
    uint32_t kw[8], gw[16], xw[8];
    load_gates<REV>(chunk_rsrc(a.G, gbp, tok, nv, a.dk, gb), gl, a.G.vec, a.g32, gw);
    load16<REV>(chunk_rsrc(a.K, kb, tok, nv, a.dk, 2), kl, a.K.vec, kw);
    if (GRAD) load16<REV>(chunk_rsrc(a.X, xb, tok, nv, a.dk, 2), lane_of<REV>(a.X, g, col, a.dk, 2), a.X.vec, xw);
    bool wildv = false;
    for (int s = wave; s < NV; s += NW) {
      const int e0 = 32 * s + 2 * n;
      uint32_t w[8];
      load16<REV>(chunk_rsrc(a.V, vb, tok, nv, a.dv, 2), lane_of<REV>(a.V, g, e0, a.dv, 2), a.V.vec, w);
      u32x4 c0, c1;
      columns_of(w, c0, c1);
      *(u32x4*)(vt + e0 * kTokRow + 8 * g) = c0;
      *(u32x4*)(vt + (e0 + 1) * kTokRow + 8 * g) = c1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        wildv |= pair_wild<DT>(w[j]);
        *(uint32_t*)(vs + (8 * g + j) * RS + e0) = w[j];
      }
      if (GRAD) {
        load16<REV>(chunk_rsrc(a.W, wb, tok, nv, a.dv, 2), lane_of<REV>(a.W, g, e0, a.dv, 2), a.W.vec, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          wildv |= pair_wild<DT>(w[j]);
          *(uint32_t*)(ws + (8 * g + j) * RS + e0) = w[j];
        }
      }
    }
    const bool anyv = __ballot(wildv) != 0;
    if (lane == 0) wild[wave] = anyv;
    float gv[2][8];
    gate_values<DT>(gw, a.g32, gv);
    Gates q;
    make_gates<REV>(gv, lane, q);
    float kf[2][8];
    uint32_t big = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      kf[0][j] = pair_lo<DT>(kw[j]) * a.kscale * q.down[0][j];
      kf[1][j] = pair_hi<DT>(kw[j]) * a.kscale * q.down[1][j];
      big = max(big, max(mag(kf[0][j]), mag(kf[1][j])));
    }
    gsum[0] += q.sum[0];
    gsum[1] += q.sum[1];
    int hard = __ballot(q.hard || big > kBigBits) != 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) hard |= wild[w];

    f32x4 o[2][2] = {};
    if (!__builtin_amdgcn_readfirstlane(hard)) {
      bf16x8 kk[2][3];
      split8<3>(kf[0], kk[0]);
      split8<3>(kf[1], kk[1]);
      if (GRAD) {
        f32x4 pt[2][2] = {};   // W_i . V_j, rows j, columns i
#pragma unroll
        for (int s = 0; s < NV; ++s) {
          u32x4 vv[2], wr[2];
          bf16x8 ww[2][kTerms<DT>];
#pragma unroll
          for (int tl = 0; tl < 2; ++tl) {
            vv[tl] = *(const u32x4*)(vs + row_of(n, tl) * RS + 32 * s + 8 * g);
            wr[tl] = *(const u32x4*)(ws + row_of(n, tl) * RS + 32 * s + 8 * g);
            exact_terms<DT>(wr[tl], ww[tl]);
          }
#pragma unroll
          for (int jt = 0; jt < 2; ++jt)
#pragma unroll
            for (int it = 0; it < 2; ++it) {
              if constexpr (DT == DT_F16)
                pt[jt][it] = mfma(__builtin_bit_cast(f16x8, vv[jt]), __builtin_bit_cast(f16x8, wr[it]), pt[jt][it]);
              else
                pt[jt][it] = mfma(__builtin_bit_cast(bf16x8, vv[jt]), ww[it][0], pt[jt][it]);
            }
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            float x[8];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[r] = S[s][0][nt][r] *= q.a[nt];
              x[4 + r] = S[s][1][nt][r] *= q.a[nt];
            }
            bf16x8 st[3];
            split8<3>(x, st);
#pragma unroll
            for (int it = 0; it < 2; ++it) o[it][nt] = mfma_terms(ww[it], st, o[it][nt]);
          }
        }
#pragma unroll
        for (int it = 0; it < 2; ++it) {
          float x[8];
#pragma unroll
          for (int jt = 0; jt < 2; ++jt)
#pragma unroll
            for (int r = 0; r < 4; ++r) x[4 * jt + r] = 8 * g + 4 * jt + r <= row_of(n, it) ? pt[jt][it][r] : 0.0f;
          bf16x8 ps[3];
          split8<3>(x, ps);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) o[it][nt] = mfma_terms(ps, kk[nt], o[it][nt]);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) o[j >> 2][nt][j & 3] *= q.up[nt][j];
      } else {
#pragma unroll
        for (int s = 0; s < NV; ++s)
#pragma unroll
          for (int tl = 0; tl < 2; ++tl)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] *= q.a[nt];
      }
#pragma unroll
      for (int s = 0; s < NV; ++s)
#pragma unroll
        for (int tl = 0; tl < 2; ++tl) {
          bf16x8 vv[kTerms<DT>];
          exact_terms<DT>(*(const u32x4*)(vt + (32 * s + row_of(n, tl)) * kTokRow + 8 * g), vv);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) S[s][tl][nt] = mfma_terms(vv, kk[nt], S[s][tl][nt]) * q.b[nt];
        }
    } else {
      for (int tg = 0; tg < 4; ++tg) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t kraw = __shfl(kw[j], 16 * tg + n, 64);
          const float k0 = pair_lo<DT>(kraw) * a.kscale, k1 = pair_hi<DT>(kraw) * a.kscale;
          const float e0 = expf(__shfl(gv[0][j], 16 * tg + n, 64)), e1 = expf(__shfl(gv[1][j], 16 * tg + n, 64));
          const uint16_t *vr = vs + (8 * tg + j) * RS, *wr = ws + (8 * tg + j) * RS;
          float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
          for (int s = 0; s < NV; ++s)
#pragma unroll
            for (int tl = 0; tl < 2; ++tl) {
              const u32x2 v = *(const u32x2*)(vr + 32 * s + 8 * g + 4 * tl);
              u32x2 w = {};
              if (GRAD) w = *(const u32x2*)(wr + 32 * s + 8 * g + 4 * tl);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const uint32_t vw = v[r >> 1], ww = w[r >> 1];
                const float vx = r & 1 ? pair_hi<DT>(vw) : pair_lo<DT>(vw);
                float y0 = S[s][tl][0][r], y1 = S[s][tl][1][r];
                if (!REV) {
                  y0 *= e0;
                  y1 *= e1;
                }
                y0 = __builtin_fmaf(k0, vx, y0);
                y1 = __builtin_fmaf(k1, vx, y1);
                if (GRAD) {
                  const float wx = r & 1 ? pair_hi<DT>(ww) : pair_lo<DT>(ww);
                  s0 = __builtin_fmaf(wx, y0, s0);
                  s1 = __builtin_fmaf(wx, y1, s1);
                }
                if (REV) {
                  y0 *= e0;
                  y1 *= e1;
                }
                S[s][tl][0][r] = y0;
                S[s][tl][1][r] = y1;
              }
            }
          if (GRAD) {
            s0 += __shfl_xor(s0, 16, 64);
            s1 += __shfl_xor(s1, 16, 64);
            s0 += __shfl_xor(s0, 32, 64);
            s1 += __shfl_xor(s1, 32, 64);
            if (g == tg) {
              o[j >> 2][0][j & 3] = s0;
              o[j >> 2][1][j & 3] = s1;
            }
          }
        }
      }
    }
    if (GRAD) {
      const __amdgpu_buffer_rsrc_t orsrc = chunk_rsrc(a.O, ob, tok, nv, a.dk, 2);
      const Lane ol = lane_of<REV>(a.O, g, col, a.dk, 2);
      float y[2][8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float o0 = o[j >> 2][0][j & 3] * a.oscale, o1 = o[j >> 2][1][j & 3] * a.oscale;
        store16<REV>(orsrc, ol, a.O.vec, j, pair_round<DT>(o0, o1));
        y[0][j] = pair_lo<DT>(xw[j]) * o0;
        y[1][j] = pair_hi<DT>(xw[j]) * o1;
      }
      // the workspace's rows of this chunk: the lane's tokens are rows of H dkp floats
      float* qr = qdq + tok * a.H * a.dkp + col;
      const int64_t qs = (int64_t)a.H * a.dkp;
      if (!REV) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 8 * g + j;
          if (i < nv && col < a.dkp) *(f32x2*)(qr + i * qs) = f32x2{y[0][j], y[1][j]};
        }
      } else {
        // dg_t = (the value behind the chunk) + sum over this and the later tokens of q dq - k dk
        float run[2] = {0.0f, 0.0f}, d[2][8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int i = 31 - 8 * g - j;
          f32x2 u = {0.0f, 0.0f};
          if (i < nv && col < a.dkp) u = *(const f32x2*)(qr + i * qs);
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) {
            run[nt] += u[nt] - y[nt][j];
            d[nt][j] = run[nt];
          }
        }
        const __amdgpu_buffer_rsrc_t drsrc = chunk_rsrc(a.DG, dgb, tok, nv, a.dk, gob);
        const Lane dl = lane_of<REV>(a.DG, g, col, a.dk, gob);
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
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (a.go32) {
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, d[0][j]), drsrc,
                                                  dl.off0 + tok_off<REV>(dl, j), 0, 0);
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, d[1][j]), drsrc,
                                                  dl.off1 + tok_off<REV>(dl, j), 0, 0);
          } else {
            store16<REV>(drsrc, dl, a.DG.vec, j, pair_round<DT>(d[0][j], d[1][j]));
          }
        }
      }
    }
    __syncthreads();
  }

  if (!GRAD) {
    // this segment's own state, from zero
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
        if (col + nt < a.dkp) a.sums[p.slot * a.dkp + col + nt] = gsum[nt];
    return;
  }
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

}  // namespace mbd
