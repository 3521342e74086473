// libmbd_operators.so: root-mean-square norm with residual addition and
// 16-bit or scaled 8-bit output (include/rmsnorm.h).
//
// Bound by HBM: x and residual are read once, s and y written once.  A
// workgroup owns a row and keeps it in registers, so the sum of squares and
// the maximum are one pass and one reduction: with u_j = s_j w_j and the row's
// r = rsqrt(mean s^2 + eps), max |y| = r max |u| and y_j / scale = u_j * 448 /
// max |u|, so the codes do not wait for r.  16384 rows of 7168 with residual, to
// e4m3: 143 us (822 MB, 5.7 TB/s; a large copy reaches 5.05); one row 3.4 us, which
// is launch and two trips to memory.
#include "rmsnorm.h"

#include "gemv_kernel.h"
#include "operand.h"
#include "operators.h"

using mbd_host::kMagic;
using mbd_host::Region;

namespace mbd {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct NormArgs {
  const uint16_t *x, *res, *w;
  uint16_t* sum;
  void* y;
  float* scales;
  int64_t ldx, ldres, ldsum, ldy;
  int32_t n;
  float eps;
};

template <int DT>
__device__ __forceinline__ float norm_lo(uint32_t w) {
  return widen<DT>((uint16_t)w);
}
template <int DT>
__device__ __forceinline__ float norm_hi(uint32_t w) {
  return widen<DT>((uint16_t)(w >> 16));
}

__device__ __forceinline__ float wave_max(float v) {
  v = fmaxf(v, dpp_get<0xB1>(v));
  v = fmaxf(v, dpp_get<0x4E>(v));
  v = fmaxf(v, dpp_get<0x141>(v));
  v = fmaxf(v, dpp_get<0x140>(v));
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
// |u| where it is finite, else 0.
__device__ __forceinline__ float finite_mag(float u) {
  const float a = __builtin_fabsf(u);
  return a < __builtin_inff() ? a : 0.0f;
}

// Sum and maximum over the workgroup, in wave order; every thread gets both.
template <int T>
__device__ __forceinline__ void reduce(float& ss, float& mx) {
  __shared__ float part[2][T / 64];
  ss = wave_sum(ss);
  mx = wave_max(mx);
  if constexpr (T > 64) {
    if ((threadIdx.x & 63) == 0) {
      part[0][threadIdx.x >> 6] = ss;
      part[1][threadIdx.x >> 6] = mx;
    }
    __syncthreads();
    ss = 0.0f;
    mx = 0.0f;
#pragma unroll
    for (int i = 0; i < T / 64; ++i) {
      ss += part[0][i];
      mx = fmaxf(mx, part[1][i]);
    }
  }
}

// Four values as e4m3 codes.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// A row's factors.  inv = 448 / max |u| leaves fp32's range below 2^-119; rows of
// so small values are raised by `up` first.
struct RowScale {
  float r, scale, up, inv;
};
__device__ __forceinline__ RowScale row_scale(const NormArgs& p, float ss, float mx) {
  RowScale s;
  s.r = 1.0f / sqrtf(ss / (float)p.n + p.eps);
  s.scale = ss == 0.0f && mx == 0.0f ? 0.0f : s.r * mx / 448.0f;   // r is infinite if eps is 0 too
  s.up = mx < 0x1p-100f ? 0x1p100f : 1.0f;
  s.inv = mx > 0.0f ? 448.0f / (mx * s.up) : 0.0f;
  return s;
}

// Rows of whole 16-byte vectors, V of them per thread.
template <int DT, int T, int V, bool E4M3>
__global__ __launch_bounds__(T) void norm_kernel(const NormArgs p) {
  const int64_t row = blockIdx.x;
  const int nv = p.n >> 3;
  const uint16_t *xr = p.x + row * p.ldx, *rr = p.res ? p.res + row * p.ldres : nullptr;
  u32x4 s[V], w[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * T;
    s[i] = u32x4{};
    w[i] = u32x4{};
    if (v < nv) {
      s[i] = *(const u32x4*)(xr + 8 * v);
      w[i] = *(const u32x4*)(p.w + 8 * v);
    }
  }
  if (rr) {
    u32x4 t[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int v = threadIdx.x + i * T;
      t[i] = u32x4{};
      if (v < nv) t[i] = *(const u32x4*)(rr + 8 * v);
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t a = s[i][c], b = t[i][c];
        s[i][c] = (uint32_t)to_bits<DT>(norm_lo<DT>(a) + norm_lo<DT>(b)) |
                  (uint32_t)to_bits<DT>(norm_hi<DT>(a) + norm_hi<DT>(b)) << 16;
      }
    if (p.sum) {
      uint16_t* sr = p.sum + row * p.ldsum;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int v = threadIdx.x + i * T;
        if (v < nv) *(u32x4*)(sr + 8 * v) = s[i];
      }
    }
  }
  float ss = 0.0f, mx = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t a = s[i][c], b = w[i][c];
      const float s0 = norm_lo<DT>(a), s1 = norm_hi<DT>(a);
      ss = __builtin_fmaf(s0, s0, ss);
      ss = __builtin_fmaf(s1, s1, ss);
      if (E4M3) mx = fmaxf(mx, fmaxf(finite_mag(s0 * norm_lo<DT>(b)), finite_mag(s1 * norm_hi<DT>(b))));
    }
  reduce<T>(ss, mx);
  const RowScale k = row_scale(p, ss, mx);
  if (E4M3 && threadIdx.x == 0) p.scales[row] = k.scale;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int v = threadIdx.x + i * T;
    if (v >= nv) continue;
    float u[8];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t a = s[i][c], b = w[i][c];
      if (E4M3) {
        u[2 * c] = norm_lo<DT>(a) * norm_lo<DT>(b) * k.up;
        u[2 * c + 1] = norm_hi<DT>(a) * norm_hi<DT>(b) * k.up;
      } else {
        u[2 * c] = norm_lo<DT>(a) * k.r * norm_lo<DT>(b);
        u[2 * c + 1] = norm_hi<DT>(a) * k.r * norm_hi<DT>(b);
      }
    }
    if (E4M3) {
      u32x2 o;
      o[0] = codes4(u[0] * k.inv, u[1] * k.inv, u[2] * k.inv, u[3] * k.inv);
      o[1] = codes4(u[4] * k.inv, u[5] * k.inv, u[6] * k.inv, u[7] * k.inv);
      *(u32x2*)((uint8_t*)p.y + row * p.ldy + 8 * v) = o;
    } else {
      u32x4 o;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        o[c] = (uint32_t)to_bits<DT>(u[2 * c]) | (uint32_t)to_bits<DT>(u[2 * c + 1]) << 16;
      *(u32x4*)((uint16_t*)p.y + row * p.ldy + 8 * v) = o;
    }
  }
}

// Any row: element by element, twice over the row (the second time from the
// caches).  s is formed again from x and residual unless it was stored; where
// sum_out is one of them, each element is read by the thread that writes it.
template <int DT, bool E4M3>
__global__ __launch_bounds__(256) void norm_any_kernel(const NormArgs p) {
  const int64_t row = blockIdx.x;
  const uint16_t *xr = p.x + row * p.ldx, *rr = p.res ? p.res + row * p.ldres : nullptr;
  uint16_t* sr = p.sum ? p.sum + row * p.ldsum : nullptr;
  float ss = 0.0f, mx = 0.0f;
  for (int j = threadIdx.x; j < p.n; j += 256) {
    uint16_t b = xr[j];
    if (rr) b = to_bits<DT>(widen<DT>(b) + widen<DT>(rr[j]));
    if (sr) sr[j] = b;
    const float s = widen<DT>(b);
    ss = __builtin_fmaf(s, s, ss);
    if (E4M3) mx = fmaxf(mx, finite_mag(s * widen<DT>(p.w[j])));
  }
  reduce<256>(ss, mx);
  const RowScale k = row_scale(p, ss, mx);
  if (E4M3 && threadIdx.x == 0) p.scales[row] = k.scale;
  for (int j = threadIdx.x; j < p.n; j += 256) {
    uint16_t b = sr ? sr[j] : xr[j];
    if (rr && !sr) b = to_bits<DT>(widen<DT>(b) + widen<DT>(rr[j]));
    const float s = widen<DT>(b), w = widen<DT>(p.w[j]);
    if (E4M3) ((uint8_t*)p.y)[row * p.ldy + j] = (uint8_t)codes4(s * w * k.up * k.inv, 0.0f, 0.0f, 0.0f);
    else ((uint16_t*)p.y)[row * p.ldy + j] = to_bits<DT>(s * k.r * w);
  }
}

}  // namespace mbd

namespace {

using NormFn = void (*)(const mbd::NormArgs);
struct Form {
  int threads, vectors;   // per thread
  NormFn fn[2][2];        // [dtype][e4m3]
};
#define FORM(T, V)                                                                             \
  {T, V, {{&mbd::norm_kernel<0, T, V, false>, &mbd::norm_kernel<0, T, V, true>},               \
          {&mbd::norm_kernel<1, T, V, false>, &mbd::norm_kernel<1, T, V, true>}}}
const Form kForms[] = {FORM(64, 1), FORM(64, 2), FORM(256, 1), FORM(256, 2), FORM(256, 4), FORM(512, 4), FORM(1024, 4)};
const NormFn kAny[2][2] = {{&mbd::norm_any_kernel<0, false>, &mbd::norm_any_kernel<0, true>},
                           {&mbd::norm_any_kernel<1, false>, &mbd::norm_any_kernel<1, true>}};

// A lone row's leading dimensions are never used: replaced by ones that keep
// 16-byte boundaries.
rmsnorm_t lone_row(rmsnorm_t p) {
  if (p.m == 1) p.ldx = p.ldres = p.ldsum = p.ldy = (p.n + 7) / 8 * 8;
  return p;
}

Region rows_of(const void* x, const rmsnorm_t* p, int64_t ld, int64_t bytes) {
  return Region{(uintptr_t)x, bytes, {p->m, 1, 1}, {ld, 0, 0}, p->n};
}

}  // namespace

extern "C" gemv_status_t rmsnorm_check_args(const rmsnorm_t* given, const void* x, const void* residual, const void* w,
                                            const void* sum_out, const void* y, const float* scales) {
  const rmsnorm_t* p = given;
  if (!p) return GEMV_ERR_INVALID_ARG;
  if (p->dtype != GEMV_F16 && p->dtype != GEMV_BF16) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->out_e4m3 != 0 && p->out_e4m3 != 1) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->m < 0 || p->n < 0) return GEMV_ERR_INVALID_ARG;
  if (p->m == 0 || p->n == 0) return GEMV_OK;
  const int64_t lim = (int64_t)1 << 30;
  if (p->m > ((int64_t)1 << 21) || p->n > ((int64_t)1 << 24)) return GEMV_ERR_TOO_LARGE;
  if (p->m > 1 && (p->ldx > lim || p->ldy > lim || (residual && p->ldres > lim) || (sum_out && p->ldsum > lim)))
    return GEMV_ERR_TOO_LARGE;
  if (p->ldx < p->n || p->ldy < p->n || (residual && p->ldres < p->n) || (sum_out && p->ldsum < p->n))
    return GEMV_ERR_INVALID_ARG;
  const rmsnorm_t q = lone_row(*given);
  p = &q;
  if (!x || !w || !y || (sum_out && !residual) || (p->out_e4m3 != 0) != (scales != nullptr))
    return GEMV_ERR_INVALID_ARG;
  if ((((uintptr_t)x | (uintptr_t)residual | (uintptr_t)w | (uintptr_t)sum_out) & 1u) ||
      (!p->out_e4m3 && ((uintptr_t)y & 1u)) || ((uintptr_t)scales & 3u))
    return GEMV_ERR_MISALIGNED;
  const bool sum_x = sum_out == x && p->ldsum == p->ldx, sum_r = sum_out == residual && p->ldsum == p->ldres;
  const bool y_x = !p->out_e4m3 && y == x && p->ldy == p->ldx && !sum_x;
  const Region sum = rows_of(sum_out, p, p->ldsum, 2), out = rows_of(y, p, p->ldy, p->out_e4m3 ? 1 : 2),
               rx = rows_of(x, p, p->ldx, 2), rr = rows_of(residual, p, p->ldres, 2),
               rw = mbd_host::dense_region(w, p->n, 2), rs = mbd_host::dense_region(scales, p->m, 4);
  using mbd_host::share;
  if (share(sum, out) || share(sum, rs) || share(out, rs)) return GEMV_ERR_ALIASING;
  if (share(sum, rw) || share(out, rw) || share(rs, rw) || share(rs, rx) || share(rs, rr)) return GEMV_ERR_ALIASING;
  if ((!sum_x && share(sum, rx)) || (!sum_r && share(sum, rr))) return GEMV_ERR_ALIASING;
  if ((!y_x && share(out, rx)) || share(out, rr)) return GEMV_ERR_ALIASING;
  return GEMV_OK;
}

extern "C" gemv_status_t rmsnorm_run(gemv_handle_t h, const rmsnorm_t* given, const void* x, const void* residual,
                                     const void* w, void* sum_out, void* y, float* scales, hipStream_t stream) {
  if (!h || h->magic != kMagic) return report(nullptr, GEMV_ERR_NULL_HANDLE, "rmsnorm_run");
  gemv_status_t st = rmsnorm_check_args(given, x, residual, w, sum_out, y, scales);
  if (st != GEMV_OK) return report(h, st, "rmsnorm_run arguments");
  if (given->m == 0 || given->n == 0) return GEMV_OK;
  const rmsnorm_t q = lone_row(*given), *p = &q;
  if ((st = mbd_host::ready(h, "rmsnorm_run")) != GEMV_OK) return st;
  mbd::NormArgs a = {(const uint16_t*)x, (const uint16_t*)residual, (const uint16_t*)w, (uint16_t*)sum_out, y, scales,
                     p->ldx, p->ldres, p->ldsum, p->ldy, (int32_t)p->n, p->eps};
  const auto whole = [&](const void* q, int64_t ld) { return !q || (((uintptr_t)q & 15u) == 0 && ld % 8 == 0); };
  const bool yok = p->out_e4m3 ? (((uintptr_t)y & 7u) == 0 && p->ldy % 8 == 0) : whole(y, p->ldy);
  NormFn fn = kAny[p->dtype][p->out_e4m3];
  int threads = 256;
  if (p->n % 8 == 0 && whole(x, p->ldx) && whole(residual, p->ldres) && whole(sum_out, p->ldsum) && whole(w, 8) && yok) {
    for (const Form& f : kForms) {
      if ((int64_t)f.threads * f.vectors * 8 >= p->n) {
        fn = f.fn[p->dtype][p->out_e4m3];
        threads = f.threads;
        break;
      }
    }
  }
  void* args[] = {(void*)&a};
  hipError_t e = hipLaunchKernel((const void*)fn, dim3((unsigned)p->m), dim3((unsigned)threads), args, 0, stream);
  return e == hipSuccess ? GEMV_OK : report(h, GEMV_ERR_HIP, hipGetErrorString(e));
}
