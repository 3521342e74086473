// libmbd_operators.so: gated linear attention over whole sequences
// (include/gla_scan.h) over the kernels of gla_scan_kernel.h.
#include "gla_scan.h"

#include "gla_scan_kernel.h"
#include "gla_scan_table.h"
#include "operand.h"
#include "operators.h"

namespace mbd {

// ---- segments' states from their own states ----------------------------------
// slots[s] holds segment s's own state (from zero; the last segment's in the
// order of the recurrence is not there, and not needed) and becomes its start
// state: one thread per 4 elements walks the sequence's segments.  Bound by HBM
// (64 heads of 128 x 128, 8 segments: 63 MB in 10.6 us, 5.9 TB/s) and, for few
// heads, by the walk (15 heads of 64 x 96, 32 segments, both sides: 12 us, 15 with
// 4 segments fetched at once).
struct Join {
  float* slots;
  const Decay* decays;
  const float* S0;          // user layout, or null
  const int32_t* offsets;
  int64_t total, t;
  int32_t H, dk, dv, dkp, dvp, nseg, L, rev;
};
struct JoinArgs {
  Join side[2];             // by grid y: a backward pass has two
};
__global__ __launch_bounds__(256) void scan_join_kernel(const JoinArgs both) {
  const Join& a = both.side[blockIdx.y];
  const int per = a.dkp * (a.dvp / 4), nx = (per + 255) / 256;
  const int64_t head = blockIdx.x / nx;            // seq * H + h
  const int seq = (int)(head / a.H);
  const int i = (int)(blockIdx.x - head * nx) * 256 + threadIdx.x;
  if (i >= per) return;
  int64_t len = a.t;
  if (a.offsets) {
    const int64_t s = min(max((int64_t)a.offsets[seq], (int64_t)0), a.total);
    len = min(min(max((int64_t)a.offsets[seq + 1], s), a.total) - s, a.t);
  }
  const int ns = max((int)((len + a.L - 1) / a.L), 1);
  const int d = i / (a.dvp / 4), e = (i - d * (a.dvp / 4)) * 4;
  f32x4 x = {};
  if (a.S0 && d < a.dk) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (e + r < a.dv) x[r] = a.S0[(head * a.dk + d) * a.dv + e + r];
  }
  const int64_t size = (int64_t)a.dkp * a.dvp;
  float* slot = a.slots + head * a.nseg * size + (int64_t)d * a.dvp + e;
  const Decay* decay = a.decays + head * a.nseg * a.dkp + d;
  constexpr int AHEAD = 8;   // segments fetched at once
  for (int s0 = 0; s0 + 1 < ns; s0 += AHEAD) {
    f32x4 u[AHEAD];
    Decay f[AHEAD];
#pragma unroll
    for (int m = 0; m < AHEAD; ++m)
      if (s0 + m + 1 < ns) {
        const int64_t at = a.rev ? ns - 1 - s0 - m : s0 + m;
        u[m] = *(const f32x4*)(slot + at * size);
        f[m] = decay[at * a.dkp];
      }
#pragma unroll
    for (int m = 0; m < AHEAD; ++m)
      if (s0 + m + 1 < ns) {
        const int64_t at = a.rev ? ns - 1 - s0 - m : s0 + m;
        *(f32x4*)(slot + at * size) = x;
#pragma unroll
        for (int r = 0; r < 4; ++r) x[r] = scaled(x[r], f[m]) + u[m][r];
      }
  }
  *(f32x4*)(slot + (a.rev ? 0 : ns - 1) * size) = x;
}

}  // namespace mbd

using mbd_host::kMagic;
using mbd_host::Region;

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 24;

struct Shape {
  int64_t batch, tokens, heads, dk, dv, rows;
  int g_bytes;
};

// Where a call's scratch lies, in bytes; see scan_plan.
struct ScanPlan {
  int nseg, L;
  int32_t dkp, dvp;
  int64_t heads;            // sequences x heads
  size_t slots, slots2, decays, decays2, ends, qdq, bytes;
};

int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }
// Waves of a workgroup: two for at most 64 columns, else four.
int waves_of(int64_t width) { return width <= 64 ? 2 : 4; }
int out_cols(int64_t dv) {   // output columns per workgroup: even shares of at most 128
  const int64_t nblk = (dv + 127) / 128, slabs = (dv + 31) / 32;
  return (int)(32 * ((slabs + nblk - 1) / nblk));
}

// Sequences are cut into segments that run side by side when the heads alone
// leave the GPU idle: as many as fit it in one round (two workgroups of four
// waves a CU, or four of two; a few more than that take a second round: 156
// heads and blocks in 4 segments of 400 tokens 173 us, in 3 127), of at least
// 64 tokens, or 32 where that leaves most of the round free (forward three
// quarters, backward half); short sequences stay whole, since the segments' own
// states are passes of their own.  Measured, heads of 128 x 128, in us (whole /
// segments of 32 / of 64):
//   forward   8 heads   129 tokens 28 / 29 / 33    255 41 / 31 / 34    512 77 / 38 / 37
//            32 heads   192        32 / 38 / 37    255 41 / 39 / 39    512 78 / 45 / 43
//   backward  8 heads    96        64 / 47 / 62   1001 517 / 79 / 85  1500 753 / 99 / 91
//            32 heads    64        48 / 50 / 49    255 144 / 74 / 82   512 284 / 106 / 95
ScanPlan scan_plan(const gla_scan_t* p, bool backward) {
  ScanPlan s = {};
  s.dkp = (int32_t)up(p->dk, 32);
  s.dvp = (int32_t)up(p->dv, 32);
  s.heads = p->batch * p->heads;
  const int64_t width = backward ? p->dk : out_cols(p->dv);
  const int waves = waves_of(width);
  const int64_t blocks = backward ? (p->dk + 32 * waves - 1) / (32 * waves) : (p->dv + width - 1) / width;
  const int64_t slots = 2048 / waves, units = std::max(s.heads * blocks, (int64_t)1);
  const bool fine = units * ((p->tokens + 31) / 32) <= slots / (backward ? 2 : 4);
  const int64_t least = fine ? 32 : 64;
  int64_t nseg = std::min(slots / units, (p->tokens + least - 1) / least);
  if (p->tokens < (backward ? 96 : fine ? 160 : 224)) nseg = 1;
  nseg = std::max(nseg, (int64_t)1);
  const int64_t L = std::max(up((p->tokens + nseg - 1) / nseg, mbd::kScanC), (int64_t)mbd::kScanC);
  s.L = (int)L;
  s.nseg = (int)std::max((p->tokens + L - 1) / L, (int64_t)1);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t r = at;
    at += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t states = (size_t)s.heads * s.nseg * s.dkp * s.dvp * 4, chans = (size_t)s.heads * s.nseg * s.dkp * 4;
  if (s.nseg > 1) {
    s.slots = take(states);
    s.decays = take(chans / sizeof(float) * sizeof(mbd::Decay));
    if (backward) {
      s.slots2 = take(states);
      s.decays2 = take(chans / sizeof(float) * sizeof(mbd::Decay));
    }
  }
  if (backward) {
    s.ends = take(chans);
    s.qdq = take((size_t)(p->offsets ? p->rows : p->batch * p->tokens) * p->heads * s.dkp * 4);
  }
  s.bytes = at;
  return s;
}

Region region(const gla_scan_t* p, const void* x, const gla_stride_t& s, int64_t d, int64_t bytes) {
  const int64_t b = p->offsets ? 1 : p->batch, t = p->offsets ? p->rows : p->tokens;
  return Region{(uintptr_t)x, bytes, {b, t, p->heads}, {s.batch, s.token, s.head}, d};
}

bool strides_fit(const gla_scan_t* p, const gla_stride_t& s, int64_t d) {
  const int64_t t = p->offsets ? p->rows : p->tokens;
  if (s.head < 0 || s.head > ((int64_t)1 << 40)) return false;
  if (!p->offsets && (s.batch < 0 || s.batch > ((int64_t)1 << 40))) return false;
  return t <= 1 || (s.token >= d && s.token <= kMaxStride);   // one token's stride is not used
}

// Sizes and scalars; *idle: nothing to do.
gemv_status_t check_sizes(const gla_scan_t* p, bool backward, bool* idle) {
  *idle = false;
  if (!p) return GEMV_ERR_INVALID_ARG;
  if (p->dtype != GEMV_F16 && p->dtype != GEMV_BF16) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->gate_f32 != 0 && p->gate_f32 != 1) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->batch < 0 || p->tokens < 0 || p->heads < 0 || p->dk < 0 || p->dv < 0) return GEMV_ERR_INVALID_ARG;
  if (p->offsets && p->rows < 0) return GEMV_ERR_INVALID_ARG;
  if (p->batch == 0 || p->heads == 0 || p->dk == 0 || p->dv == 0) {
    *idle = true;
    return GEMV_OK;
  }
  const int64_t lim = (int64_t)1 << 30;
  if (p->dk > 256 || p->dv > (backward ? 256 : 65536) || p->tokens > lim || (p->offsets && p->rows > lim) ||
      p->batch > ((int64_t)1 << 20) || p->heads > ((int64_t)1 << 20) ||
      p->batch * p->heads > ((int64_t)1 << 20))
    return GEMV_ERR_TOO_LARGE;
  if (!p->offsets && p->batch * p->tokens > ((int64_t)1 << 34)) return GEMV_ERR_TOO_LARGE;
  if (p->offsets && ((uintptr_t)p->offsets & 3u)) return GEMV_ERR_MISALIGNED;
  return GEMV_OK;
}

gemv_status_t check_inputs(const gla_scan_t* p, const void* q, const void* k, const void* v, const void* gk,
                           const void* o) {
  const int64_t rows = p->offsets ? p->rows : p->tokens;
  if (rows > 0 && p->tokens > 0 && (!q || !k || !v || !gk || !o)) return GEMV_ERR_INVALID_ARG;
  if (!strides_fit(p, p->q, p->dk) || !strides_fit(p, p->k, p->dk) || !strides_fit(p, p->v, p->dv) ||
      !strides_fit(p, p->gk, p->dk) || !strides_fit(p, p->o, p->dv))
    return GEMV_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o) & 1u) return GEMV_ERR_MISALIGNED;
  if ((uintptr_t)gk & (p->gate_f32 ? 3u : 1u)) return GEMV_ERR_MISALIGNED;
  return GEMV_OK;
}

gemv_status_t check_scratch(const ScanPlan& s, const void* workspace, size_t bytes) {
  if (s.bytes == 0) return GEMV_OK;
  if (!workspace || bytes < s.bytes) return GEMV_ERR_INVALID_ARG;
  if ((uintptr_t)workspace & 15u) return GEMV_ERR_MISALIGNED;
  return GEMV_OK;
}

// A grid's work-items along x (a 32-bit field of the dispatch) are kept at most 2^31.
bool grid_fits(int64_t grid, int threads) { return grid <= ((int64_t)1 << 31) / threads; }

// Workgroups of the outputs, and of the gradients over the key channels.
int64_t out_grid(const gla_scan_t* p, const ScanPlan& s) {
  return s.heads * s.nseg * ((p->dv + out_cols(p->dv) - 1) / out_cols(p->dv));
}
int64_t grad_grid(const gla_scan_t* p, const ScanPlan& s) {
  const int64_t cols = 32 * waves_of(p->dk);
  return s.heads * s.nseg * ((p->dk + cols - 1) / cols);
}

// Outputs against each other and against the inputs.
bool clash(const Region* out, int no, const Region* in, int ni) {
  for (int i = 0; i < no; ++i) {
    if (out[i].empty()) continue;
    if (!mbd_host::distinct(out[i])) return true;
    for (int j = i + 1; j < no; ++j)
      if (mbd_host::share(out[i], out[j])) return true;
    for (int j = 0; j < ni; ++j)
      if (mbd_host::share(out[i], in[j])) return true;
  }
  return false;
}

gemv_status_t check_forward(const gla_scan_t* p, const void* q, const void* k, const void* v, const void* gk,
                            const float* S0, const float* ST, const void* o, const void* workspace,
                            size_t workspace_bytes, bool* idle) {
  gemv_status_t st = check_sizes(p, false, idle);
  if (st != GEMV_OK || *idle) return st;
  st = check_inputs(p, q, k, v, gk, o);
  if (st != GEMV_OK) return st;
  if (((uintptr_t)S0 | (uintptr_t)ST) & 3u) return GEMV_ERR_MISALIGNED;
  const ScanPlan s = scan_plan(p, false);
  if (!grid_fits(out_grid(p, s), 256)) return GEMV_ERR_TOO_LARGE;
  st = check_scratch(s, workspace, workspace_bytes);
  if (st != GEMV_OK) return st;
  const int64_t state = s.heads * p->dk * p->dv, gb = p->gate_f32 ? 4 : 2;
  const Region in[] = {region(p, q, p->q, p->dk, 2), region(p, k, p->k, p->dk, 2), region(p, v, p->v, p->dv, 2),
                       region(p, gk, p->gk, p->dk, gb),
                       mbd_host::dense_region(p->offsets, p->batch + 1, 4),
                       mbd_host::dense_region(S0 == ST ? nullptr : S0, state, 4)};
  const Region out[] = {region(p, o, p->o, p->dv, 2), mbd_host::dense_region(ST, state, 4),
                        mbd_host::dense_region(s.bytes ? workspace : nullptr, (int64_t)s.bytes, 1)};
  if (clash(out, 3, in, 6)) return GEMV_ERR_ALIASING;
  return GEMV_OK;
}

gemv_status_t check_backward(const gla_scan_t* p, const gla_scan_grad_t* gr, const void* q, const void* k,
                             const void* v, const void* gk, const float* S0, const void* dout, const float* dST,
                             const void* dq, const void* dk, const void* dv, const void* dgk, const float* dS0,
                             const void* workspace, size_t workspace_bytes, bool* idle) {
  gemv_status_t st = check_sizes(p, true, idle);
  if (st != GEMV_OK || *idle) return st;
  if (!gr) return GEMV_ERR_INVALID_ARG;
  st = check_inputs(p, q, k, v, gk, dout);
  if (st != GEMV_OK) return st;
  const int64_t rows = p->offsets ? p->rows : p->tokens;
  if (rows > 0 && p->tokens > 0 && (!dq || !dk || !dv || !dgk)) return GEMV_ERR_INVALID_ARG;
  if (!strides_fit(p, gr->dq, p->dk) || !strides_fit(p, gr->dk, p->dk) || !strides_fit(p, gr->dv, p->dv) ||
      !strides_fit(p, gr->dgk, p->dk))
    return GEMV_ERR_INVALID_ARG;
  if (((uintptr_t)dq | (uintptr_t)dk | (uintptr_t)dv) & 1u) return GEMV_ERR_MISALIGNED;
  if (((uintptr_t)dgk & (p->gate_f32 ? 3u : 1u)) || (((uintptr_t)S0 | (uintptr_t)dST | (uintptr_t)dS0) & 3u))
    return GEMV_ERR_MISALIGNED;
  const ScanPlan s = scan_plan(p, true);
  if (!grid_fits(out_grid(p, s), 256) || !grid_fits(grad_grid(p, s), 256)) return GEMV_ERR_TOO_LARGE;
  st = check_scratch(s, workspace, workspace_bytes);
  if (st != GEMV_OK) return st;
  const int64_t state = s.heads * p->dk * p->dv, gb = p->gate_f32 ? 4 : 2;
  const Region in[] = {region(p, q, p->q, p->dk, 2),     region(p, k, p->k, p->dk, 2),
                       region(p, v, p->v, p->dv, 2),     region(p, gk, p->gk, p->dk, gb),
                       region(p, dout, p->o, p->dv, 2),  mbd_host::dense_region(p->offsets, p->batch + 1, 4),
                       mbd_host::dense_region(S0, state, 4), mbd_host::dense_region(dST, state, 4)};
  const Region out[] = {region(p, dq, gr->dq, p->dk, 2),   region(p, dk, gr->dk, p->dk, 2),
                        region(p, dv, gr->dv, p->dv, 2),   region(p, dgk, gr->dgk, p->dk, gb),
                        mbd_host::dense_region(dS0, state, 4),
                        mbd_host::dense_region(s.bytes ? workspace : nullptr, (int64_t)s.bytes, 1)};
  if (clash(out, 6, in, 8)) return GEMV_ERR_ALIASING;
  return GEMV_OK;
}

// ---- launches ------------------------------------------------------------------

using mbd::ScanFn;
using mbd::ScanForms;
const ScanForms* const kScanOut[2] = {&mbd::kScanOutF16, &mbd::kScanOutBf16};
const ScanForms* const kScanGrad[2] = {&mbd::kScanGradF16, &mbd::kScanGradBf16};
const mbd::StateForms* const kScanState[2] = {&mbd::kScanStateF16, &mbd::kScanStateBf16};
ScanFn scan_form(const ScanForms* const (&forms)[2], const gla_scan_t* p, int rev, int tier, bool four) {
  return (*forms[p->dtype])[p->gate_f32][rev][tier][four];
}
const size_t kOutLds[3] = {mbd::scan_out_lds<2>(), mbd::scan_out_lds<4>(), mbd::scan_out_lds<8>()};
template <int DT> constexpr size_t kStateLdsOf[3] = {mbd::scan_state_lds<DT, 2>(), mbd::scan_state_lds<DT, 4>(), mbd::scan_state_lds<DT, 8>()};
template <int DT> constexpr size_t kGradLdsOf[3] = {mbd::scan_grad_lds<DT, 2>(), mbd::scan_grad_lds<DT, 4>(), mbd::scan_grad_lds<DT, 8>()};
size_t state_lds(int dtype, int t) { return dtype == GEMV_F16 ? kStateLdsOf<mbd::DT_F16>[t] : kStateLdsOf<mbd::DT_BF16>[t]; }
size_t grad_lds(int dtype, int t) { return dtype == GEMV_F16 ? kGradLdsOf<mbd::DT_F16>[t] : kGradLdsOf<mbd::DT_BF16>[t]; }

// 64, 128 or 256 channels, by index.
int tier(int64_t d) { return d <= 64 ? 0 : d <= 128 ? 1 : 2; }

int gate_bytes(const gla_scan_t* p) { return p->gate_f32 ? 4 : 2; }
mbd::ScanTensor tensor(const gla_scan_t* p, const void* x, const gla_stride_t& s, int64_t d, int bytes = 2) {
  mbd::ScanTensor t;
  t.p = x;
  t.sb = p->offsets ? 0 : s.batch;
  t.sh = s.head;
  // one token's stride says nothing, but tells tokens behind it from it
  t.st = (int32_t)((p->offsets ? p->rows : p->tokens) > 1 ? s.token : up(d, 2));
  // 4-byte accesses: even channels, strides and a 4-byte aligned start
  t.vec = d % 2 == 0 && (s.batch % 2 == 0 || p->offsets || p->batch == 1) && (s.head % 2 == 0 || p->heads == 1) &&
          t.st % 2 == 0 && ((uintptr_t)x & 3u) == 0;
  t.step = (uint32_t)t.st * (uint32_t)bytes;
  t.full = (uint32_t)((mbd::kScanC - 1) * (uint64_t)t.step + (uint64_t)d * bytes);   // < 2^31
  return t;
}

mbd::ScanArgs common(const gla_scan_t* p, const ScanPlan& s) {
  mbd::ScanArgs a = {};
  a.offsets = p->offsets;
  a.total = p->rows;
  a.t = p->tokens;
  a.H = (int32_t)p->heads;
  a.dk = (int32_t)p->dk;
  a.dv = (int32_t)p->dv;
  a.dkp = s.dkp;
  a.dvp = s.dvp;
  a.nseg = s.nseg;
  a.L = s.L;
  return a;
}

hipError_t launch(ScanFn fn, int64_t grid, int waves, size_t lds, const mbd::ScanArgs& a, hipStream_t stream) {
  void* args[] = {(void*)&a};
  return hipLaunchKernel((const void*)fn, dim3((unsigned)grid), dim3((unsigned)waves * 64u), args, lds, stream);
}

// Own states of the segments, over `dv` columns; `sides` 2: of both recurrences
// (15 heads of 64 x 96, 1001 tokens: 19 us one after the other).
hipError_t launch_state(const gla_scan_t* p, int64_t grid, int waves, int64_t dv, const mbd::StateArgs& a, int sides,
                        hipStream_t stream) {
  const int t = tier(dv);
  void* args[] = {(void*)&a};
  return hipLaunchKernel((const void*)(*kScanState[p->dtype])[p->gate_f32][t][waves == 4],
                         dim3((unsigned)grid, (unsigned)sides), dim3((unsigned)waves * 64u), args, state_lds(p->dtype, t), stream);
}

mbd::Join join_of(const gla_scan_t* p, const ScanPlan& s, float* slots, const mbd::Decay* decays, const float* S0, int rev) {
  return mbd::Join{slots, decays, S0, p->offsets, p->rows, p->tokens, (int32_t)p->heads, (int32_t)p->dk,
                   (int32_t)p->dv, s.dkp, s.dvp, s.nseg, s.L, rev};
}
hipError_t launch_join(const ScanPlan& s, const mbd::JoinArgs& j, int sides, hipStream_t stream) {
  void* args[] = {(void*)&j};
  const int64_t nx = ((int64_t)s.dkp * (s.dvp / 4) + 255) / 256;
  return hipLaunchKernel((const void*)&mbd::scan_join_kernel, dim3((unsigned)(nx * s.heads), (unsigned)sides),
                         dim3(256), args, 0, stream);
}

}  // namespace

bool mbd_host::scan_set_attributes() {
  const auto set = [](const void* fn, size_t lds) {
    return lds <= 65536 || hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds) == hipSuccess;
  };
  for (int d = 0; d < 2; ++d)
    for (int g = 0; g < 2; ++g)
      for (int r = 0; r < 2; ++r)
        for (int t = 0; t < 3; ++t)
          for (int w = 0; w < 2; ++w)
            if (!set((const void*)(*kScanOut[d])[g][r][t][w], kOutLds[t]) ||
                !set((const void*)(*kScanGrad[d])[g][r][t][w], grad_lds(d, t)) ||
                (r == 0 && !set((const void*)(*kScanState[d])[g][t][w], state_lds(d, t))))
              return false;
  return true;
}

extern "C" size_t gla_scan_workspace_bytes(const gla_scan_t* p, int32_t backward) {
  bool idle = false;
  if (check_sizes(p, backward != 0, &idle) != GEMV_OK || idle) return 0;
  return scan_plan(p, backward != 0).bytes;
}

extern "C" gemv_status_t gla_scan_check_args(const gla_scan_t* p, const void* q, const void* k, const void* v,
                                             const void* gk, const float* S0, const float* ST, const void* o,
                                             const void* workspace, size_t workspace_bytes) {
  bool idle;
  return check_forward(p, q, k, v, gk, S0, ST, o, workspace, workspace_bytes, &idle);
}

extern "C" gemv_status_t gla_scan_grad_check_args(const gla_scan_t* p, const gla_scan_grad_t* grad, const void* q,
                                                  const void* k, const void* v, const void* gk, const float* S0,
                                                  const void* dout, const float* dST, const void* dq,
                                                  const void* dk, const void* dv, const void* dgk,
                                                  const float* dS0, const void* workspace,
                                                  size_t workspace_bytes) {
  bool idle;
  return check_backward(p, grad, q, k, v, gk, S0, dout, dST, dq, dk, dv, dgk, dS0, workspace, workspace_bytes, &idle);
}

extern "C" gemv_status_t gla_scan_forward(gemv_handle_t h, const gla_scan_t* p, const void* q, const void* k,
                                          const void* v, const void* gk, const float* S0, float* ST, void* o,
                                          void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!h || h->magic != kMagic) return report(nullptr, GEMV_ERR_NULL_HANDLE, "gla_scan_forward");
  bool idle = false;
  gemv_status_t st = check_forward(p, q, k, v, gk, S0, ST, o, workspace, workspace_bytes, &idle);
  if (st != GEMV_OK) return report(h, st, "gla_scan_forward arguments");
  if (idle || (p->tokens == 0 && !ST)) return GEMV_OK;
  if ((st = mbd_host::ready(h, "gla_scan_forward")) != GEMV_OK) return st;
  const ScanPlan s = scan_plan(p, false);
  const int64_t bh = s.heads;
  mbd::ScanArgs a = common(p, s);
  a.K = tensor(p, k, p->k, p->dk);
  a.V = tensor(p, v, p->v, p->dv);
  a.G = tensor(p, gk, p->gk, p->dk, gate_bytes(p));
  a.X = tensor(p, q, p->q, p->dk);
  a.O = tensor(p, o, p->o, p->dv);
  a.kscale = 1.0f;
  a.oscale = p->scale;
  a.S0 = S0;
  a.ST = ST;
  a.cols = out_cols(p->dv);
  a.nblk = (int32_t)((p->dv + a.cols - 1) / a.cols);
  hipError_t e = hipSuccess;
  if (s.nseg > 1) {
    char* w = (char*)workspace;
    a.slots = (float*)(w + s.slots);
    a.decays = (mbd::Decay*)(w + s.decays);
    // a segment's own state: columns in blocks of at most 256, channels in blocks of a workgroup's
    mbd::StateArgs sides = {a, {}};
    mbd::ScanArgs& b = sides.fwd;
    const int kw = waves_of(p->dk);
    b.nblk = (int32_t)((p->dk + 32 * kw - 1) / (32 * kw));
    for (int64_t c0 = 0; c0 < p->dv && e == hipSuccess; c0 += 256) {
      const int64_t c = std::min(p->dv - c0, (int64_t)256);
      b.V.p = (const char*)a.V.p + c0 * 2;
      b.dv = (int32_t)c;
      b.ecol = (int32_t)c0;
      e = launch_state(p, bh * s.nseg * b.nblk, kw, c, sides, 1, stream);
    }
    if (e == hipSuccess) e = launch_join(s, {{join_of(p, s, a.slots, a.decays, S0, 0), {}}}, 1, stream);
  }
  const int ow = waves_of(a.cols);
  if (e == hipSuccess) e = launch(scan_form(kScanOut, p, 0, tier(p->dk), ow == 4), out_grid(p, s), ow, kOutLds[tier(p->dk)], a, stream);
  return e == hipSuccess ? GEMV_OK : report(h, GEMV_ERR_HIP, hipGetErrorString(e));
}

extern "C" gemv_status_t gla_scan_backward(gemv_handle_t h, const gla_scan_t* p, const gla_scan_grad_t* grad,
                                           const void* q, const void* k, const void* v, const void* gk,
                                           const float* S0, const void* dout, const float* dST, void* dq, void* dk,
                                           void* dv, void* dgk, float* dS0, void* workspace, size_t workspace_bytes,
                                           hipStream_t stream) {
  if (!h || h->magic != kMagic) return report(nullptr, GEMV_ERR_NULL_HANDLE, "gla_scan_backward");
  bool idle = false;
  gemv_status_t st = check_backward(p, grad, q, k, v, gk, S0, dout, dST, dq, dk, dv, dgk, dS0, workspace,
                                    workspace_bytes, &idle);
  if (st != GEMV_OK) return report(h, st, "gla_scan_backward arguments");
  if (idle || (p->tokens == 0 && !dS0)) return GEMV_OK;
  if ((st = mbd_host::ready(h, "gla_scan_backward")) != GEMV_OK) return st;
  const ScanPlan s = scan_plan(p, true);
  char* w = (char*)workspace;
  const mbd::ScanTensor tq = tensor(p, q, p->q, p->dk), tk = tensor(p, k, p->k, p->dk),
                        tv = tensor(p, v, p->v, p->dv), tg = tensor(p, gk, p->gk, p->dk, gate_bytes(p)),
                        tdo = tensor(p, dout, p->o, p->dv);
  const int kw = waves_of(p->dk), cols = out_cols(p->dv), ow = waves_of(cols);
  const int kt = tier(p->dk), vt = tier(p->dv);
  mbd::ScanArgs f = common(p, s), r = common(p, s);
  f.G = r.G = tg;
  f.nblk = r.nblk = (int32_t)((p->dk + 32 * kw - 1) / (32 * kw));
  f.ends = r.ends = (float*)(w + s.ends);
  f.qdq = r.qdq = (float*)(w + s.qdq);
  f.K = tk;   // dq_i = scale S do_i
  f.V = tv;
  f.W = tdo;
  f.X = tq;
  f.O = tensor(p, dq, grad->dq, p->dk);
  f.kscale = 1.0f;
  f.oscale = p->scale;
  f.S0 = S0;
  f.dST = dST;
  r.K = tq;   // dk_j = D v_j, with the scale in D
  r.V = tdo;
  r.W = tv;
  r.X = tk;
  r.O = tensor(p, dk, grad->dk, p->dk);
  r.DG = tensor(p, dgk, grad->dgk, p->dk, gate_bytes(p));
  r.kscale = p->scale;
  r.oscale = 1.0f;
  r.S0 = dST;
  r.ST = dS0;
  mbd::ScanArgs o = r;   // dv_j = k_j^T D
  o.X = tk;
  o.O = tensor(p, dv, grad->dv, p->dv);
  o.ST = nullptr;
  o.cols = cols;
  o.nblk = (int32_t)((p->dv + cols - 1) / cols);
  const int64_t gk_grid = grad_grid(p, s), gv_grid = out_grid(p, s);
  hipError_t e = hipSuccess;
  if (s.nseg > 1) {
    f.slots = (float*)(w + s.slots);
    f.decays = (mbd::Decay*)(w + s.decays);
    r.slots = o.slots = (float*)(w + s.slots2);
    r.decays = o.decays = (mbd::Decay*)(w + s.decays2);
    f.others = r.slots;
    e = launch_state(p, gk_grid, kw, p->dv, {f, r}, 2, stream);
    if (e == hipSuccess)
      e = launch_join(s, {{join_of(p, s, f.slots, f.decays, S0, 0), join_of(p, s, r.slots, r.decays, dST, 1)}}, 2, stream);
  }
  if (e == hipSuccess) e = launch(scan_form(kScanGrad, p, 0, vt, kw == 4), gk_grid, kw, grad_lds(p->dtype, vt), f, stream);
  if (e == hipSuccess) e = launch(scan_form(kScanGrad, p, 1, vt, kw == 4), gk_grid, kw, grad_lds(p->dtype, vt), r, stream);
  if (e == hipSuccess) e = launch(scan_form(kScanOut, p, 1, kt, ow == 4), gv_grid, ow, kOutLds[kt], o, stream);
  return e == hipSuccess ? GEMV_OK : report(h, GEMV_ERR_HIP, hipGetErrorString(e));
}
