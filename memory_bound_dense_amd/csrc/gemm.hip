// libmbd_operators.so: the dense product of many rows with its epilogue
// (include/gemm.h) over the kernels of gemm_kernel.h.
#include "gemm.h"

#include "gemm_kernel.h"
#include "operand.h"
#include "operators.h"

using mbd_host::kMagic;
using mbd_host::Region;

namespace {

int64_t in_bytes(int32_t type) { return type == GEMM_E4M3 ? 1 : 2; }
int64_t up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

using GemmFn = void (*)(const mbd::GemmArgs);

// Tiles: rows of B x tokens, and what a slab costs, in ns: `alone` for one
// workgroup on a CU, `shared` per workgroup where the CU has more to do.
// Measured (bf16, and used for every type): the tile's time over whole rounds,
// e.g. aligned 256 x 256 94 us for 64 slabs on 86 CUs and 98 us on 256; 128 x 128 52 us for 64 slabs
// on 256 CUs, 116 us for 4 workgroups a CU; 64 x 64 30 us for 64 slabs, 190 us
// for 16 a CU.
struct Tile {
  int bn, bm, threads;
  bool direct;       // loads straight into LDS
  size_t lds;        // dynamic
  int alone, shared;
  GemmFn fn[3];
};
#define TILE(BN, BM, WN, WM, ALONE, SHARED)                                                         \
  {BN, BM, WN * WM * 64, false, mbd::gemm_tile_lds<BN, BM>(), ALONE, SHARED,                               \
   {&mbd::gemm_tile_kernel<0, BN, BM, WN, WM>, &mbd::gemm_tile_kernel<1, BN, BM, WN, WM>,           \
    &mbd::gemm_tile_kernel<2, BN, BM, WN, WM>}}
#define DIRECT(BN, BM, WN, WM, WK, WN8, WM8, ST, ALONE, SHARED)                                                 \
  {BN, BM, WN * WM * WK * 64, true, 0, ALONE, SHARED,                                                                 \
   {&mbd::gemm_direct_kernel<0, BN, BM, WN, WM, WK, ST>, &mbd::gemm_direct_kernel<1, BN, BM, WN, WM, WK, ST>,   \
    &mbd::gemm_direct_kernel<2, BN, BM, WN8, WM8, 1, ST>}}
// [1]: rows on 16-byte boundaries
const Tile kTiles[2][5] = {
    {TILE(256, 256, 2, 4, 2300, 2300), TILE(128, 128, 2, 2, 1070, 750), TILE(64, 128, 2, 2, 850, 500),
     TILE(64, 64, 2, 2, 520, 330), {}},
    {DIRECT(256, 256, 2, 4, 1, 2, 4, 2, 1470, 1470), DIRECT(256, 128, 2, 2, 2, 4, 2, 3, 920, 920),
     DIRECT(128, 128, 1, 2, 2, 2, 2, 2, 810, 470), TILE(64, 128, 2, 2, 580, 350), TILE(64, 64, 2, 2, 470, 190)}};

// Few tokens: [row tiles 1..4][token tiles 1, 2, 4][type].
constexpr int kSkinnyWaves = 8;
#define SKINNY(RT, MT, U) \
  {&mbd::gemm_skinny_kernel<0, RT, MT, 8, U>, &mbd::gemm_skinny_kernel<1, RT, MT, 8, U>, &mbd::gemm_skinny_kernel<2, RT, MT, 8, U>}
const GemmFn kSkinny[4][3][3] = {{SKINNY(1, 1, 2), SKINNY(1, 2, 2), SKINNY(1, 4, 1)},
                                 {SKINNY(2, 1, 2), SKINNY(2, 2, 2), SKINNY(2, 4, 1)},
                                 {SKINNY(3, 1, 2), SKINNY(3, 2, 2), SKINNY(3, 4, 1)},
                                 {SKINNY(4, 1, 1), SKINNY(4, 2, 1), SKINNY(4, 4, 1)}};

struct GemmPlan {
  const Tile* tile;  // null: skinny
  int rt, mt;        // skinny: row tiles, token tiles (by index)
  int64_t tiles_m, tiles_n, nsplit, npad;
  size_t bytes;
};

// `whole`: rows of A and B on 16-byte boundaries.
GemmPlan gemm_plan(const gemm_t* p, bool whole) {
  GemmPlan g = {};
  const int64_t slabs = (p->k * in_bytes(p->in_type) + 127) / 128;
  g.nsplit = 1;
  if (p->m <= 64) {
    // Row tiles per workgroup: whole rounds over the 256 CUs, each as long as
    // its rows and (about 0.3 of a row tile per token tile) its tokens take.
    // Measured, 16 tokens, 1 / 2 / 3 / 4 row tiles: n = 11008, k = 4096 19.4 /
    // 20.4 / 17.2 / 18.0 us; n = 14336 25.4 / 22.9 / 29.0 / 22.2; n = 4096, k =
    // 11008 20.9 / 27.0 / 32.5 / 38.8.
    g.mt = p->m <= 16 ? 0 : p->m <= 32 ? 1 : 2;
    const int64_t t16 = (p->n + 15) / 16;
    int64_t best = 0;
    for (int rt = 1; rt <= 4; ++rt) {
      const int64_t groups = (t16 + rt - 1) / rt, cost = (groups + 255) / 256 * (10 * rt + (3 << g.mt));
      if (rt == 1 || cost < best) {
        best = cost;
        g.rt = rt - 1;
        g.tiles_n = groups;
      }
    }
    g.tiles_m = 1;
    const int64_t want = 256 / g.tiles_n;
    g.nsplit = std::max(std::min(want, slabs / (kSkinnyWaves * 2)), (int64_t)1);
  } else {
    // The tile and the split of k with the least modelled time: a CU's share of
    // the slabs, and for a split the partial sums' way through memory (4 TB/s)
    // and a second launch (4 us).
    int64_t best = 0;
    for (const Tile& t : kTiles[whole]) {
      if (!t.bn) continue;
      const int64_t tm = (p->m + t.bm - 1) / t.bm, tn = (p->n + t.bn - 1) / t.bn;
      for (int64_t ns = 1; ns <= 8; ++ns) {
        if (ns > 1 && slabs / ns < 4) break;
        const int64_t rounds = (tm * tn * ns + 255) / 256;
        int64_t cost = (slabs + ns - 1) / ns * std::max((int64_t)t.alone, rounds * t.shared);
        if (ns > 1) cost += 4000 + ns * p->m * p->n / 500;
        if (!g.tile || cost < best) {
          best = cost;
          g.tile = &t;
          g.tiles_m = tm;
          g.tiles_n = tn;
          g.nsplit = ns;
        }
      }
    }
  }
  g.npad = up(p->n, 4);
  if (!g.tile) g.npad = up(p->n, 16);
  if (g.nsplit > 1) g.bytes = (size_t)g.nsplit * p->m * g.npad * 4;
  return g;
}

// Workgroups of the product and of the join.
int64_t grid_of(const GemmPlan& g) { return g.tiles_m * g.tiles_n * g.nsplit; }
int64_t join_grid_of(const gemm_t* p, const GemmPlan& g) { return g.nsplit > 1 ? (p->m * (g.npad / 4) + 255) / 256 : 0; }
int threads_of(const GemmPlan& g) { return g.tile ? g.tile->threads : kSkinnyWaves * 64; }
// A grid's work-items along x (a 32-bit field of the dispatch) are kept at most 2^31.
bool launchable(const gemm_t* p, const GemmPlan& g) {
  return grid_of(g) <= ((int64_t)1 << 31) / threads_of(g) && join_grid_of(p, g) <= ((int64_t)1 << 23);
}

// A lone row's leading dimension is never used (a row of a long sequence's last
// token may have any): replaced by one that keeps 16-byte boundaries.
gemm_t lone_rows(gemm_t p) {
  const int64_t e = in_bytes(p.in_type), ld = up(p.k * e, 16) / e;
  if (p.m == 1) {
    p.lda = ld;
    p.ldc = p.ldr = up(p.n, 8);
  }
  if (p.n == 1) p.ldb = ld;
  return p;
}

bool whole_rows(const gemm_t* p, const void* A, const void* B) {
  const int64_t e = in_bytes(p->in_type);
  return ((((uintptr_t)A | (uintptr_t)B) & 15u) | ((p->lda * e) & 15) | ((p->ldb * e) & 15)) == 0;
}

Region matrix(const void* x, int64_t rows, int64_t cols, int64_t ld, int64_t bytes) {
  return Region{(uintptr_t)x, bytes, {rows, 1, 1}, {ld, 0, 0}, cols};
}

gemv_status_t check(const gemm_t* given, const void* A, const void* B, const void* C, const void* workspace,
                    size_t workspace_bytes, bool sizes_only) {
  const gemm_t* p = given;
  if (!p) return GEMV_ERR_INVALID_ARG;
  if (p->in_type < GEMM_F16 || p->in_type > GEMM_E4M3) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->dtype != GEMV_F16 && p->dtype != GEMV_BF16) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->in_type != GEMM_E4M3 && p->in_type != (int32_t)p->dtype) return GEMV_ERR_UNSUPPORTED_DTYPE;
  if (p->act < GEMM_ACT_NONE || p->act > GEMM_ACT_SILU) return GEMV_ERR_INVALID_ARG;
  if (p->m < 0 || p->n < 0 || p->k < 0) return GEMV_ERR_INVALID_ARG;
  if (p->m == 0 || p->n == 0) return GEMV_OK;
  const int64_t e = in_bytes(p->in_type), lim = (int64_t)1 << 30;
  if (p->m > lim || p->n > lim || p->k > lim) return GEMV_ERR_TOO_LARGE;
  // more than 2^22 of the largest tiles (512 threads each) are no launch; what the plan works out stays below 2^63
  if (p->m * p->n > (int64_t)1 << 38) return GEMV_ERR_TOO_LARGE;
  if (p->lda < p->k || p->ldb < p->k || p->ldc < p->n || (p->residual && p->ldr < p->n)) return GEMV_ERR_INVALID_ARG;
  const gemm_t q = lone_rows(*given);
  p = &q;
  if (p->lda > ((int64_t)1 << 23) / e || p->ldb > ((int64_t)1 << 23) / e || p->ldc > lim ||
      (p->residual && p->ldr > lim))
    return GEMV_ERR_TOO_LARGE;
  if (sizes_only) return GEMV_OK;
  if (!C || (p->k > 0 && (!A || !B))) return GEMV_ERR_INVALID_ARG;
  uintptr_t two = (uintptr_t)C | (uintptr_t)p->bias | (uintptr_t)p->residual;
  if (e == 2 && p->k > 0) two |= (uintptr_t)A | (uintptr_t)B;
  if ((two & 1u) || (((uintptr_t)p->scale_a | (uintptr_t)p->scale_b) & 3u)) return GEMV_ERR_MISALIGNED;
  const GemmPlan g = gemm_plan(p, whole_rows(p, A, B));
  if (!launchable(p, g)) return GEMV_ERR_TOO_LARGE;
  if (g.bytes) {
    if (!workspace || workspace_bytes < g.bytes) return GEMV_ERR_INVALID_ARG;
    if ((uintptr_t)workspace & 15u) return GEMV_ERR_MISALIGNED;
  }
  const bool in_place = p->residual == C && p->ldr == p->ldc;
  const Region in[] = {matrix(p->k > 0 ? A : nullptr, p->m, p->k, p->lda, e),
                       matrix(p->k > 0 ? B : nullptr, p->n, p->k, p->ldb, e),
                       mbd_host::dense_region(p->scale_a, p->m, 4), mbd_host::dense_region(p->scale_b, p->n, 4),
                       mbd_host::dense_region(p->bias, p->n, 2),
                       matrix(in_place ? nullptr : p->residual, p->m, p->n, p->ldr, 2)};
  const Region out[] = {matrix(C, p->m, p->n, p->ldc, 2),
                        mbd_host::dense_region(g.bytes ? workspace : nullptr, (int64_t)g.bytes, 1)};
  for (const Region& o : out) {
    for (const Region& i : in)
      if (mbd_host::share(o, i)) return GEMV_ERR_ALIASING;
  }
  if (mbd_host::share(out[0], out[1])) return GEMV_ERR_ALIASING;
  return GEMV_OK;
}

}  // namespace

bool mbd_host::gemm_set_attributes() {
  for (const auto& set : kTiles)
    for (const Tile& t : set)
      for (GemmFn f : t.fn)
        if (f && t.lds > 65536 &&
            hipFuncSetAttribute((const void*)f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)t.lds) != hipSuccess)
          return false;
  return true;
}

extern "C" size_t gemm_workspace_bytes(const gemm_t* p) {
  if (check(p, nullptr, nullptr, nullptr, nullptr, 0, true) != GEMV_OK || p->m == 0 || p->n == 0) return 0;
  // the pointers are not known here: what either kind of rows needs
  return std::max(gemm_plan(p, false).bytes, gemm_plan(p, true).bytes);
}

extern "C" gemv_status_t gemm_plan_config(const gemm_t* p, const void* A, const void* B, gemm_config_t* out) {
  if (!out) return GEMV_ERR_INVALID_ARG;
  *out = gemm_config_t{};
  const gemv_status_t st = check(p, nullptr, nullptr, nullptr, nullptr, 0, true);
  if (st != GEMV_OK || p->m == 0 || p->n == 0) return st;
  const gemm_t q = lone_rows(*p);
  const GemmPlan g = gemm_plan(&q, whole_rows(&q, A, B));
  if (!launchable(&q, g)) return GEMV_ERR_TOO_LARGE;
  if (g.tile) *out = gemm_config_t{g.tile->bn, g.tile->bm, g.tile->direct ? 2 : 1, (int32_t)g.nsplit};
  else *out = gemm_config_t{16 * (g.rt + 1), 16 << g.mt, 0, (int32_t)g.nsplit};
  return GEMV_OK;
}

extern "C" gemv_status_t gemm_check_args(const gemm_t* p, const void* A, const void* B, const void* C,
                                         const void* workspace, size_t workspace_bytes) {
  return check(p, A, B, C, workspace, workspace_bytes, false);
}

extern "C" gemv_status_t gemm_run(gemv_handle_t h, const gemm_t* given, const void* A, const void* B, void* C,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (!h || h->magic != kMagic) return report(nullptr, GEMV_ERR_NULL_HANDLE, "gemm_run");
  gemv_status_t st = check(given, A, B, C, workspace, workspace_bytes, false);
  if (st != GEMV_OK) return report(h, st, "gemm_run arguments");
  if (given->m == 0 || given->n == 0) return GEMV_OK;
  const gemm_t q = lone_rows(*given), *p = &q;
  if ((st = mbd_host::ready(h, "gemm_run")) != GEMV_OK) return st;
  const GemmPlan g = gemm_plan(p, whole_rows(p, A, B));
  const int64_t e = in_bytes(p->in_type);
  mbd::GemmArgs a = {};
  a.A = (const uint8_t*)A;
  a.B = (const uint8_t*)B;
  a.C = (uint16_t*)C;
  a.sa = p->scale_a;
  a.sb = p->scale_b;
  a.bias = (const uint16_t*)p->bias;
  a.res = (const uint16_t*)p->residual;
  a.part = (float*)workspace;
  a.lda = p->lda * e;
  a.ldb = p->ldb * e;
  a.ldc = p->ldc;
  a.ldr = p->residual ? p->ldr : 0;
  a.m = (int32_t)p->m;
  a.n = (int32_t)p->n;
  a.kbytes = (int32_t)(p->k * e);
  a.act = p->act;
  a.out = p->dtype;
  a.vec = p->ldc % 4 == 0 && ((uintptr_t)C & 7u) == 0 &&
          (!p->residual || (p->ldr % 4 == 0 && ((uintptr_t)p->residual & 7u) == 0));
  a.tiles_m = (int32_t)g.tiles_m;
  a.tiles_n = (int32_t)g.tiles_n;
  a.nsplit = (int32_t)g.nsplit;
  a.npad = (int32_t)g.npad;
  a.once = (((uintptr_t)B | (uint64_t)a.ldb) & 127u) == 0;
  a.alpha = p->alpha;
  void* args[] = {(void*)&a};
  const void* fn = (const void*)(g.tile ? g.tile->fn[p->in_type] : kSkinny[g.rt][g.mt][p->in_type]);
  hipError_t err = hipLaunchKernel(fn, dim3((unsigned)grid_of(g)), dim3((unsigned)threads_of(g)), args,
                                   g.tile ? g.tile->lds : 0, stream);
  if (err == hipSuccess && g.nsplit > 1)
    err = hipLaunchKernel((const void*)&mbd::gemm_join_kernel, dim3((unsigned)join_grid_of(p, g)), dim3(256), args, 0, stream);
  return err == hipSuccess ? GEMV_OK : report(h, GEMV_ERR_HIP, hipGetErrorString(err));
}
