// C ABI of libqwha: argument checks, workspace carving and launch sequencing.
// Every entry point validates on the host and launches nothing on failure.

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "kernels.h"

namespace qwha {

namespace {
thread_local char g_msg[512] = "";
}

qwha_status fail(qwha_status s, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return s;
}

namespace {
std::atomic<uint64_t> g_ring_wait_ns{2000000000ull};
std::atomic<int32_t> g_injected_failures{0};
}  // namespace

uint64_t ring_wait_ns() { return g_ring_wait_ns.load(std::memory_order_relaxed); }

qwha_status cuda_status(cudaError_t e, const char *what) {
  if (e == cudaSuccess) {
    // test hook: report an armed number of successful results as failures
    int32_t n = g_injected_failures.load();
    while (n > 0 && !g_injected_failures.compare_exchange_weak(n, n - 1)) {
    }
    if (n <= 0) return QWHA_OK;
    return fail(QWHA_ERR_CUDA, "%s: injected failure (qwha_debug_fail_cuda_checks)", what);
  }
  return fail(QWHA_ERR_CUDA, "%s: %s (cudaError %d)", what, cudaGetErrorString(e), (int)e);
}

int sm_count() {
  static int counts[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  if (counts[dev] == 0) {
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    counts[dev] = n;
  }
  return counts[dev];
}

cudaError_t allow_smem(const void *kernel, size_t bytes, std::atomic<size_t> (&allowed)[64]) {
  static std::mutex raising;  // the record follows the attribute
  std::atomic<size_t> &most = allowed[device_slot()];
  if (bytes <= 32 * 1024 || bytes <= most.load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(raising);
  if (bytes <= most.load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) most.store(bytes, std::memory_order_release);
  return e;
}

int device_slot() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  return dev;
}

}  // namespace qwha

using namespace qwha;

namespace {

const char *dtype_name(qwha_dtype d) { return d == QWHA_F32 ? "f32" : d == QWHA_BF16 ? "bf16" : "?"; }

bool valid_dtype(qwha_dtype d) { return d == QWHA_F32 || d == QWHA_BF16; }

// A second stream per device on which the dense forward computes Z = X H while
// the caller's stream builds W_eff and runs the GEMM (they do not depend on each
// other). Fork and join go through events, so the work stays ordered with the
// caller's stream and is captured with it in a CUDA graph.
struct Fork {
  cudaStream_t aux = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
};

std::mutex g_fork_mu;
Fork g_fork[64];

cudaError_t get_fork(Fork **out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  Fork &f = g_fork[dev];
  if (!f.aux) {
    e = cudaStreamCreateWithFlags(&f.aux, cudaStreamNonBlocking);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&f.fork, cudaEventDisableTiming);
    if (e == cudaSuccess) e = cudaEventCreateWithFlags(&f.join, cudaEventDisableTiming);
    if (e != cudaSuccess) return e;
  }
  *out = &f;
  return cudaSuccess;
}

qwha_status check_hadamard(int32_t n, int32_t had_block) {
  if (n <= 0) return fail(QWHA_ERR_INVALID_ARG, "row length %d must be positive", n);
  if (had_block < 2 || had_block > 32768 || !is_pow2(had_block))
    return fail(QWHA_ERR_INVALID_ARG, "had_block %d must be a power of two in [2, 32768]", had_block);
  if (n % had_block)
    return fail(QWHA_ERR_INVALID_ARG, "had_block %d does not divide the row length %d", had_block, n);
  return QWHA_OK;
}

#define QWHA_CHECK_PTR(p, name)                                                        \
  do {                                                                                 \
    if (!(p)) return fail(QWHA_ERR_INVALID_ARG, "%s is NULL", name);                   \
    if (!aligned16(p)) return fail(QWHA_ERR_MISALIGNED, "%s is not 16-byte aligned", name); \
  } while (0)

}  // namespace

// ---------------------------------------------------------------- stage timing

namespace {

enum Stage {
  ST_FWHT_FWD,
  ST_SPMM_FWD,
  ST_DEQUANT,
  ST_GEMM_FWD,
  ST_SDDMM,
  ST_GATHER_BWD,
  ST_FWHT_BWD,
  ST_GEMM_BWD,
  ST_INIT,
  ST_PLAN,
  ST_FWHT,
  ST_WEFF,
  ST_GEMM_DC,
  ST_DECODE_PREPARE,
  ST_DECODE_ENTRIES,
  ST_GEMV,
  ST_CACHE_WRITE,
  ST_CACHE_READ,
  ST_ROTARY,
  ST_ATTENTION,
  ST_PAGES,
  ST_CACHE_MOVE,
  ST_COUNT
};
const char *kStageNames[ST_COUNT] = {"fwht_fwd",   "spmm_fwd",   "dequant",  "gemm_fwd",  "sddmm_dc",
                                     "gather_bwd", "fwht_bwd",   "gemm_bwd", "init_alloc",
                                     "plan_build", "fwht",       "weff",      "gemm_dc",
                                     "decode_prepare", "decode_entries", "gemv",      "cache_write", "cache_read",
                                     "rotary", "cache_attention", "page_table", "cache_move"};

struct StageRec {
  int stage, kernels;
  cudaEvent_t a, b;
};

std::mutex g_prof_mu;
bool g_prof_on = false;
std::vector<StageRec> g_pending;
std::vector<cudaEvent_t> g_pool;
int64_t g_calls[ST_COUNT], g_launches[ST_COUNT];
double g_ms[ST_COUNT];

cudaEvent_t take_event() {
  if (!g_pool.empty()) {
    cudaEvent_t e = g_pool.back();
    g_pool.pop_back();
    return e;
  }
  cudaEvent_t e = nullptr;
  if (cudaEventCreate(&e) != cudaSuccess) return nullptr;
  return e;
}

// Brackets one stage with events when timing is on; counts launches always-on cheaply.
struct StageScope {
  int stage, kernels;
  cudaStream_t s;
  cudaEvent_t a = nullptr;
  StageScope(int st, int k, cudaStream_t str) : stage(st), kernels(k), s(str) {
    std::lock_guard<std::mutex> g(g_prof_mu);
    if (!g_prof_on) return;
    a = take_event();
    if (a) cudaEventRecord(a, s);
  }
  ~StageScope() {
    std::lock_guard<std::mutex> g(g_prof_mu);
    if (!g_prof_on || !a) return;
    cudaEvent_t b = take_event();
    if (!b) return;
    cudaEventRecord(b, s);
    g_pending.push_back({stage, kernels, a, b});
  }
};

}  // namespace

extern "C" {

void qwha_stage_timing(int32_t enable) {
  std::lock_guard<std::mutex> g(g_prof_mu);
  g_prof_on = enable != 0;
}

int32_t qwha_stage_count(void) { return ST_COUNT; }

const char *qwha_stage_name(int32_t i) { return (i >= 0 && i < ST_COUNT) ? kStageNames[i] : ""; }

qwha_status qwha_stage_report(int64_t *calls, int64_t *launches, double *ms) {
  std::lock_guard<std::mutex> g(g_prof_mu);
  qwha_status st = QWHA_OK;
  for (const StageRec &r : g_pending) {
    float t = 0.f;
    cudaError_t e = cudaEventSynchronize(r.b);
    if (e == cudaSuccess) e = cudaEventElapsedTime(&t, r.a, r.b);
    if (e != cudaSuccess && st == QWHA_OK) st = cuda_status(e, "stage events");
    g_calls[r.stage] += 1;
    g_launches[r.stage] += r.kernels;
    g_ms[r.stage] += t;
    g_pool.push_back(r.a);
    g_pool.push_back(r.b);
  }
  g_pending.clear();
  for (int i = 0; i < ST_COUNT; ++i) {
    if (calls) calls[i] = g_calls[i];
    if (launches) launches[i] = g_launches[i];
    if (ms) ms[i] = g_ms[i];
    g_calls[i] = g_launches[i] = 0;
    g_ms[i] = 0.0;
  }
  return st;
}

}  // extern "C"

extern "C" {

const char *qwha_status_string(qwha_status s) {
  switch (s) {
    case QWHA_OK: return "ok";
    case QWHA_ERR_INVALID_ARG: return "invalid argument";
    case QWHA_ERR_MISALIGNED: return "misaligned buffer";
    case QWHA_ERR_UNSUPPORTED: return "unsupported";
    case QWHA_ERR_WORKSPACE: return "workspace too small";
    case QWHA_ERR_CUDA: return "CUDA error";
    case QWHA_ERR_TIMEOUT: return "device wait timed out";
  }
  return "unknown status";
}

const char *qwha_last_error(void) { return g_msg; }

uint64_t qwha_debug_wait_limit_ns(uint64_t ns) { return g_ring_wait_ns.exchange(ns); }

void qwha_debug_fail_cuda_checks(int32_t n) { g_injected_failures.store(n > 0 ? n : 0); }

const char *qwha_version(void) { return "qwha-b200 0.1 (sm_100a)"; }

qwha_status qwha_fwht(qwha_dtype dt, const void *x, void *z, int64_t rows, int32_t n,
                      int32_t had_block, void *stream) {
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  qwha_status st = check_hadamard(n, had_block);
  if (st != QWHA_OK) return st;
  if (rows < 0) return fail(QWHA_ERR_INVALID_ARG, "rows %lld < 0", (long long)rows);
  if (rows == 0) return QWHA_OK;
  QWHA_CHECK_PTR(x, "x");
  QWHA_CHECK_PTR(z, "z");
  const size_t esz = dt == QWHA_F32 ? 4 : 2;
  const char *xb = static_cast<const char *>(x), *zb = static_cast<const char *>(z);
  const size_t bytes = (size_t)rows * n * esz;
  if (xb < zb + bytes && zb < xb + bytes) return fail(QWHA_ERR_INVALID_ARG, "x and z overlap");
  const int logn = ilog2(had_block);
  const float scale = (float)(1.0 / sqrt((double)had_block));
  (void)dtype_name;
  StageScope sc(ST_FWHT, 1, (cudaStream_t)stream);
  return cuda_status(launch_fwht(dt, dt, x, z, rows * (n / had_block), logn, scale, (cudaStream_t)stream),
                     "fwht launch");
}

}  // extern "C"

// ---------------------------------------------------------------- adapter

namespace {

struct Carver {  // hands out 256-byte aligned slices of the caller's workspace
  char *base;
  size_t off = 0;
  explicit Carver(void *b) : base(static_cast<char *>(b)) {}
  void *take(size_t bytes) {
    void *p = base ? base + off : nullptr;
    off += align_up(bytes, 256);
    return p;
  }
};


qwha_status check_adapter_shape(const qwha_adapter *a) {
  if (!a) return fail(QWHA_ERR_INVALID_ARG, "adapter is NULL");
  if (a->d_in <= 0 || a->d_out <= 0 || a->d_in % 8 || a->d_out % 8)
    return fail(QWHA_ERR_INVALID_ARG, "d_in %d and d_out %d must be positive multiples of 8", a->d_in, a->d_out);
  qwha_status st = check_hadamard(a->d_in, a->had_block);
  if (st != QWHA_OK) return st;
  if (a->p < 0 || a->p > (int64_t)a->d_in * a->d_out || a->p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld out of range", (long long)a->p);
  if (a->algo != QWHA_ALGO_SPARSE && a->algo != QWHA_ALGO_DENSE)
    return fail(QWHA_ERR_INVALID_ARG, "algo %d", (int)a->algo);
  if (a->algo == QWHA_ALGO_DENSE && weff_smem(a->d_in) > 200 * 1024)
    return fail(QWHA_ERR_UNSUPPORTED, "dense algorithm: d_in %d above 51200", a->d_in);
  if (a->weff && !aligned16(a->weff)) return fail(QWHA_ERR_MISALIGNED, "weff is not 16-byte aligned");
  QWHA_CHECK_PTR(a->row_ptr, "row_ptr");
  if (a->p > 0) {
    QWHA_CHECK_PTR(a->col_idx, "col_idx");
    QWHA_CHECK_PTR(a->coef, "coef");
  }
  return QWHA_OK;
}

qwha_status check_views(const qwha_adapter *a) {
  QWHA_CHECK_PTR(a->col_ptr, "col_ptr");
  QWHA_CHECK_PTR(a->tile_ptr, "tile_ptr");
  if (a->p > 0) {
    QWHA_CHECK_PTR(a->row_idx, "row_idx");
    QWHA_CHECK_PTR(a->perm, "perm");
    QWHA_CHECK_PTR(a->tile_pos, "tile_pos");
    QWHA_CHECK_PTR(a->tile_rk, "tile_rk");
  }
  if (cdiv(a->d_out, QWHA_TILE) > plan_max_row_blocks())
    return fail(QWHA_ERR_UNSUPPORTED, "d_out %d above %d", a->d_out, plan_max_row_blocks() * QWHA_TILE);
  return QWHA_OK;
}

qwha_status check_codes(const qwha_qweight *wq, int32_t d_in) {
  if (wq->bits < 2 || wq->bits > 4) return fail(QWHA_ERR_INVALID_ARG, "bits %d not in {2,3,4}", wq->bits);
  if (wq->group <= 0 || wq->group % 8 || d_in % wq->group)
    return fail(QWHA_ERR_INVALID_ARG, "group %d must be a multiple of 8 dividing d_in %d", wq->group, d_in);
  QWHA_CHECK_PTR(wq->qweight, "qweight");
  QWHA_CHECK_PTR(wq->scales, "scales");
  QWHA_CHECK_PTR(wq->zeros, "zeros");
  return QWHA_OK;
}

qwha_status check_qweight(const qwha_qweight *wq, int32_t d_out, int32_t d_in, qwha_dtype dt) {
  if (!wq) return QWHA_OK;
  if (dt != QWHA_BF16) return fail(QWHA_ERR_UNSUPPORTED, "the base GEMM needs dtype bf16");
  (void)d_out;
  return check_codes(wq, d_in);
}

qwha_status check_ws(void *ws, size_t ws_bytes, size_t need) {
  if (need == 0) return QWHA_OK;
  if (!ws || ws_bytes < need)
    return fail(QWHA_ERR_WORKSPACE, "workspace %zu bytes, need %zu", ws ? ws_bytes : (size_t)0, need);
  if (reinterpret_cast<uintptr_t>(ws) & 255) return fail(QWHA_ERR_MISALIGNED, "workspace not 256-byte aligned");
  return QWHA_OK;
}

// packed (index, value) entries of the SpMM in gather order
// Scratch of the SpMM for both directions: the forward over rows (segments
// d_out, width d_in) and the backward gather over columns.
size_t ent_bytes(int64_t p, int32_t d_out, int32_t d_in) {
  return std::max(spmm_scratch_bytes(p, d_out, d_in), spmm_scratch_bytes(p, d_in, d_out));
}

size_t fwd_ws(int32_t d_out, int32_t d_in, int64_t p, int64_t T, bool base) {
  const size_t n = ent_bytes(p, d_out, d_in);
  if (!base) return n;
  return n + align_up((size_t)T * d_out * 4, 256) + align_up(wdeq_bytes(d_out, d_in), 256);
}

size_t fwd_dense_ws(int32_t d_out, int32_t d_in) { return align_up((size_t)d_out * d_in * 2, 256); }


size_t bwd_dense_ws(int32_t d_out, int32_t d_in, int64_t T) {
  (void)T;
  return align_up((size_t)d_out * d_in * 2, 256);  // W_eff (unless the adapter carries one)
}

// The sparse backward's dZ buffer, which first holds the transposed dY and Z
// of the coefficient gradient (the gather writes dZ after the gradient has run).
size_t dz_region(int32_t d_out, int32_t d_in, int64_t T) {
  return std::max(align_up((size_t)T * d_in * 4, 256), sddmm_transposed_bytes(T, d_out, d_in));
}

size_t bwd_ws(int32_t d_out, int32_t d_in, int64_t p, int64_t T, bool base) {
  size_t n = align_up((size_t)kSddmmMaxChunks * (size_t)(p > 0 ? p : 1) * 4, 256);
  n += dz_region(d_out, d_in, T);  // dZ, and before it the transposed dY and Z of the gradient
  n += ent_bytes(p, d_out, d_in);  // CSC entries in gather order
  if (base) n += align_up((size_t)T * d_in * 4, 256) + align_up(wdeq_bytes(d_out, d_in), 256);
  return n;
}

// The tokens as the tensor-core product reads them, then Z in fp32 and the
// entries' sums.
size_t qgemv_ws(int32_t d_in, int64_t T, bool f32) {
  return gemv_own_x(d_in, T, f32) ? 0 : gemv_x_bytes(d_in, std::min<int64_t>(T, QWHA_DECODE_MAX_T), f32);
}
size_t decode_ws(int32_t d_out, int32_t d_in, int64_t p, int64_t T, bool base, bool f32) {
  const int64_t n = std::min<int64_t>(T, QWHA_DECODE_MAX_T);
  return (base ? gemv_x_bytes(d_in, n, f32) : 0) + (p > 0 ? gemv_z_bytes(d_out, d_in, n) : 0);
}

// Dense backward: W_eff, dX = dY W_eff (W_eff read MN-major), and dc = alpha *
// (dY^T Z) sampled at E by the GEMM epilogue (both operands read MN-major as
// stored).
qwha_status dense_bwd(const qwha_adapter *a, const qwha_qweight *wq, const void *dY, const void *Z, int64_t T,
                      float alpha, float *dc, void *dX, void *ws, cudaStream_t s) {
  Carver cv(ws);
  void *weff = a->weff ? a->weff : cv.take((size_t)a->d_out * a->d_in * 2);
  cudaError_t e = cudaSuccess;
  if (dX && T > 0) {
    if (!a->weff) {  // otherwise the forward's W_eff is used as it stands
      StageScope sc(ST_WEFF, 1, s);
      e = launch_weff(a, wq, alpha, weff, s);
    }
    if (e != cudaSuccess) return cuda_status(e, "W_eff");
    {
      StageScope sc(ST_GEMM_BWD, 1, s);
      e = launch_gemm_any(dY, false, weff, true, nullptr, dX, false, T, a->d_in, a->d_out, s);
    }
    if (e != cudaSuccess) return cuda_status(e, "GEMM dX");
  }
  if (a->p == 0 || !dc) return QWHA_OK;
  if (T == 0) return cuda_status(cudaMemsetAsync(dc, 0, (size_t)a->p * 4, s), "dc = 0");
  // the coefficient gradient as a sampled dense product: the tcgen05 GEMM's
  // epilogue writes alpha * (dY^T Z)[r_j, k_j] for the entries of E only
  StageScope sc(ST_GEMM_DC, 1, s);
  return cuda_status(launch_gemm_sampled(dY, true, Z, true, a->d_out, a->d_in, T, a->row_ptr, a->col_idx, a->p, alpha,
                                         dc, s),
                     "sampled GEMM dY^T Z");
}

}  // namespace

extern "C" {

int64_t qwha_plan_tiles(int32_t d_out, int32_t d_in) {
  if (d_out <= 0 || d_in <= 0) return 0;
  return cdiv(d_out, QWHA_TILE) * cdiv(d_in, QWHA_TILE);
}

size_t qwha_workspace_size(qwha_op op, int32_t d_out, int32_t d_in, int64_t p, int64_t T, int32_t with_base) {
  if (d_out <= 0 || d_in <= 0 || T < 0 || p < 0) return 0;
  switch (op) {
    case QWHA_OP_FWD: return fwd_ws(d_out, d_in, p, T, with_base != 0);
    case QWHA_OP_BWD: return bwd_ws(d_out, d_in, p, T, with_base != 0);
    case QWHA_OP_INIT: return init_workspace(d_out, d_in);
    case QWHA_OP_PLAN: return plan_workspace(d_out, d_in);
    case QWHA_OP_FWD_DENSE: return fwd_dense_ws(d_out, d_in);
    case QWHA_OP_BWD_DENSE: return bwd_dense_ws(d_out, d_in, T);
    case QWHA_OP_SELECT_GLOBAL: return select_global_workspace(d_out, d_in);
    case QWHA_OP_REFINE: return refine_workspace(d_out, d_in);
    case QWHA_OP_ENERGY: return energy_stats_workspace(d_out, d_in);
    case QWHA_OP_PATTERN: return pattern_stats_workspace(d_in);
    case QWHA_OP_DECODE: return decode_ws(d_out, d_in, p, T, with_base != 0, with_base == 2);
    case QWHA_OP_QGEMV: return qgemv_ws(d_in, T, with_base == 2);
    case QWHA_OP_SLOTS: return check_slots_bytes(p);
    case QWHA_OP_ATTENTION:
      return p > 0 && p <= 65535 ? attention_workspace(d_out, d_in, (int32_t)p, T, with_base == 2) : 0;
    case QWHA_OP_PAGES: return pages_workspace(d_out, p, T);
  }
  return 0;
}

qwha_status qwha_adapter_fwd(const qwha_adapter *a, const qwha_qweight *wq, qwha_dtype dt, const void *X,
                             int64_t T, float alpha, void *Z_out, void *Y, void *ws, size_t ws_bytes,
                             void *stream) {
  qwha_status st = check_adapter_shape(a);
  if (st != QWHA_OK) return st;
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if ((st = check_qweight(wq, a->d_out, a->d_in, dt)) != QWHA_OK) return st;
  if (T < 0) return fail(QWHA_ERR_INVALID_ARG, "T %lld < 0", (long long)T);
  if (T == 0) return QWHA_OK;
  QWHA_CHECK_PTR(X, "X");
  QWHA_CHECK_PTR(Z_out, "Z_out");
  QWHA_CHECK_PTR(Y, "Y");
  const bool dense = a->algo == QWHA_ALGO_DENSE;
  if (dense && dt != QWHA_BF16) return fail(QWHA_ERR_UNSUPPORTED, "the dense algorithm needs dtype bf16");
  const size_t need = dense ? fwd_dense_ws(a->d_out, a->d_in) : fwd_ws(a->d_out, a->d_in, a->p, T, wq != nullptr);
  if ((st = check_ws(ws, ws_bytes, need)) != QWHA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  const int logn = ilog2(a->had_block);
  const float inv = (float)(1.0 / sqrt((double)a->had_block));
  cudaError_t e = cudaSuccess;
  if (dense && a->z_given) {  // Z_out is an input: W_eff and the GEMM only
    void *weff = a->weff ? a->weff : ws;
    {
      StageScope sc(ST_WEFF, 1, s);
      e = launch_weff(a, wq, alpha, weff, s);
    }
    if (e != cudaSuccess) return cuda_status(e, "W_eff");
    StageScope sc(ST_GEMM_FWD, 1, s);
    return cuda_status(launch_gemm_nt(X, weff, nullptr, Y, false, T, a->d_out, a->d_in, s), "GEMM");
  }
  if (dense && gemm_fused_fwht_supported(T, logn)) {
    // W_eff, then one launch for Y = X W_eff^T whose extra warps write Z = X H
    // (kept for the backward) while the tensor cores run the GEMM.
    void *weff = a->weff ? a->weff : ws;
    {
      StageScope sc(ST_WEFF, 1, s);
      e = launch_weff(a, wq, alpha, weff, s);
    }
    if (e != cudaSuccess) return cuda_status(e, "W_eff");
    StageScope sc(ST_GEMM_FWD, 1, s);
    return cuda_status(launch_gemm_fwd_fused(X, weff, Y, T, a->d_out, a->d_in, Z_out, logn, inv, s),
                       "GEMM + transform");
  }
  if (dense) {
    // Z = X H (kept for the backward) on the auxiliary stream, concurrently
    // with W_eff and Y = X W_eff^T on the caller's stream.
    std::lock_guard<std::mutex> g(g_fork_mu);
    Fork *f = nullptr;
    e = get_fork(&f);
    if (e == cudaSuccess) e = cudaEventRecord(f->fork, s);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(f->aux, f->fork, 0);
    if (e != cudaSuccess) return cuda_status(e, "fork");
    {
      StageScope sc(ST_FWHT_FWD, 1, f->aux);
      e = launch_fwht(dt, dt, X, Z_out, T * (a->d_in / a->had_block), logn, inv, f->aux);
    }
    if (e == cudaSuccess) e = cudaEventRecord(f->join, f->aux);
    if (e != cudaSuccess) return cuda_status(e, "fwht");
    void *weff = a->weff ? a->weff : ws;
    {
      StageScope sc(ST_WEFF, 1, s);
      e = launch_weff(a, wq, alpha, weff, s);
    }
    if (e == cudaSuccess) {
      StageScope sc(ST_GEMM_FWD, 1, s);
      e = launch_gemm_nt(X, weff, nullptr, Y, false, T, a->d_out, a->d_in, s);
    }
    const cudaError_t ej = cudaStreamWaitEvent(s, f->join, 0);  // join even after a failed launch
    if (e != cudaSuccess) return cuda_status(e, "W_eff / GEMM");
    return cuda_status(ej, "join");
  }
  if (!a->z_given) {
    StageScope sc(ST_FWHT_FWD, 1, s);
    e = launch_fwht(dt, dt, X, Z_out, T * (a->d_in / a->had_block), logn, inv, s);
  }
  if (e != cudaSuccess) return cuda_status(e, "fwht");
  Carver cv(ws);
  const size_t ent_n = ent_bytes(a->p, a->d_out, a->d_in);
  void *ent = cv.take(ent_n);
  if (!wq) {
    StageScope sc(ST_SPMM_FWD, 0, s);
    e = launch_seg_spmm(dt, dt, Z_out, T, a->d_in, a->row_ptr, a->col_idx, a->coef, nullptr, a->p, a->d_out, alpha,
                        ent, ent_n, Y, s, &sc.kernels);
    return cuda_status(e, "spmm");
  }
  float *y_ad = static_cast<float *>(cv.take((size_t)T * a->d_out * 4));
  void *wdeq = cv.take(wdeq_bytes(a->d_out, a->d_in));
  {
    StageScope sc(ST_SPMM_FWD, 0, s);
    e = launch_seg_spmm(dt, QWHA_F32, Z_out, T, a->d_in, a->row_ptr, a->col_idx, a->coef, nullptr, a->p, a->d_out,
                        alpha, ent, ent_n, y_ad, s, &sc.kernels);
  }
  if (e != cudaSuccess) return cuda_status(e, "spmm");
  {
    StageScope sc(ST_DEQUANT, 1, s);
    e = launch_dequant(wq->bits, wq->group, a->d_out, a->d_in, wq->qweight, wq->scales, wq->zeros, wdeq, s);
  }
  if (e != cudaSuccess) return cuda_status(e, "dequant");
  StageScope sc(ST_GEMM_FWD, 1, s);
  return cuda_status(launch_gemm_fwd(X, wdeq, y_ad, Y, T, a->d_out, a->d_in, s), "base GEMM");
}

qwha_status qwha_adapter_bwd(const qwha_adapter *a, const qwha_qweight *wq, qwha_dtype dt, const void *dY,
                             const void *Z, int64_t T, float alpha, float *dc, void *dX, void *ws,
                             size_t ws_bytes, void *stream) {
  qwha_status st = check_adapter_shape(a);
  if (st != QWHA_OK) return st;
  const bool dense = a->algo == QWHA_ALGO_DENSE;
  if (!dense && (st = check_views(a)) != QWHA_OK) return st;
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (dense && dt != QWHA_BF16) return fail(QWHA_ERR_UNSUPPORTED, "the dense algorithm needs dtype bf16");
  if ((st = check_qweight(wq, a->d_out, a->d_in, dt)) != QWHA_OK) return st;
  if (T < 0) return fail(QWHA_ERR_INVALID_ARG, "T %lld < 0", (long long)T);
  if (a->p > 0 && dc) QWHA_CHECK_PTR(dc, "dc");
  if (T > 0) {
    QWHA_CHECK_PTR(dY, "dY");
    QWHA_CHECK_PTR(Z, "Z");
    if (dX) QWHA_CHECK_PTR(dX, "dX");
  }
  const size_t need = dense ? bwd_dense_ws(a->d_out, a->d_in, T) : bwd_ws(a->d_out, a->d_in, a->p, T, wq != nullptr);
  if ((st = check_ws(ws, ws_bytes, need)) != QWHA_OK) return st;
  cudaStream_t s = (cudaStream_t)stream;
  if (dense) return dense_bwd(a, wq, dY, Z, T, alpha, dc, dX, ws, s);
  Carver cv(ws);
  float *partial = static_cast<float *>(cv.take((size_t)kSddmmMaxChunks * (size_t)(a->p > 0 ? a->p : 1) * 4));
  float *dz = static_cast<float *>(cv.take(dz_region(a->d_out, a->d_in, T)));
  const size_t ent_n = ent_bytes(a->p, a->d_out, a->d_in);
  void *ent = cv.take(ent_n);
  cudaError_t e = cudaSuccess;
  if (dc) {
    StageScope sc(ST_SDDMM, 0, s);
    e = launch_sddmm(dt, dY, Z, T, a->d_out, a->d_in, a->tile_ptr, a->tile_pos, a->tile_rk, a->p, alpha, partial, dc,
                     s, dz, &sc.kernels);
  }
  if (e != cudaSuccess) return cuda_status(e, "sddmm");
  if (!dX || T == 0) return QWHA_OK;
  {
    StageScope sc(ST_GATHER_BWD, 0, s);
    e = launch_seg_spmm(dt, QWHA_F32, dY, T, a->d_out, a->col_ptr, a->row_idx, a->coef, a->perm, a->p, a->d_in, alpha,
                        ent, ent_n, dz, s, &sc.kernels);
  }
  if (e != cudaSuccess) return cuda_status(e, "gather");
  const int logn = ilog2(a->had_block);
  const float inv = (float)(1.0 / sqrt((double)a->had_block));
  const int64_t blocks = T * (a->d_in / a->had_block);
  if (!wq) {
    StageScope sc(ST_FWHT_BWD, 1, s);
    return cuda_status(launch_fwht(QWHA_F32, dt, dz, dX, blocks, logn, inv, s), "fwht");
  }
  float *dx_ad = static_cast<float *>(cv.take((size_t)T * a->d_in * 4));
  void *wdeq = cv.take(wdeq_bytes(a->d_out, a->d_in));
  {
    StageScope sc(ST_FWHT_BWD, 1, s);
    e = launch_fwht(QWHA_F32, QWHA_F32, dz, dx_ad, blocks, logn, inv, s);
  }
  if (e != cudaSuccess) return cuda_status(e, "fwht");
  {
    StageScope sc(ST_DEQUANT, 1, s);
    e = launch_dequant(wq->bits, wq->group, a->d_out, a->d_in, wq->qweight, wq->scales, wq->zeros, wdeq, s);
  }
  if (e != cudaSuccess) return cuda_status(e, "dequant");
  StageScope sc(ST_GEMM_BWD, 1, s);
  // dX = dY W_Q + dX_adapter: W_Q [d_out, d_in] is the MN-major B operand as stored
  return cuda_status(launch_gemm_any(dY, false, wdeq, true, dx_ad, dX, false, T, a->d_in, a->d_out, s),
                     "base GEMM (dX)");
}

qwha_status qwha_plan_build(int32_t d_out, int32_t d_in, int64_t p, const int32_t *row_ptr, const int32_t *col_idx,
                            int32_t *col_ptr, int32_t *row_idx, int32_t *perm, int32_t *tile_ptr,
                            int32_t *tile_pos, int32_t *tile_rk, void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  if (cdiv(d_out, QWHA_TILE) > plan_max_row_blocks())
    return fail(QWHA_ERR_UNSUPPORTED, "d_out %d above %d", d_out, plan_max_row_blocks() * QWHA_TILE);
  if (p < 0 || p > (int64_t)d_in * d_out || p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld out of range", (long long)p);
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  QWHA_CHECK_PTR(col_ptr, "col_ptr");
  QWHA_CHECK_PTR(tile_ptr, "tile_ptr");
  if (p > 0) {
    QWHA_CHECK_PTR(col_idx, "col_idx");
    QWHA_CHECK_PTR(row_idx, "row_idx");
    QWHA_CHECK_PTR(perm, "perm");
    QWHA_CHECK_PTR(tile_pos, "tile_pos");
    QWHA_CHECK_PTR(tile_rk, "tile_rk");
  }
  qwha_status st = check_ws(ws, ws_bytes, plan_workspace(d_out, d_in));
  if (st != QWHA_OK) return st;
  StageScope sc(ST_PLAN, 5, (cudaStream_t)stream);
  return cuda_status(launch_plan_build(d_out, d_in, p, row_ptr, col_idx, col_ptr, row_idx, perm, tile_ptr, tile_pos,
                                       tile_rk, ws, (cudaStream_t)stream),
                     "plan_build");
}

qwha_status qwha_validate_plan(const qwha_adapter *a, void *stream) {
  qwha_status st = check_adapter_shape(a);
  if (st != QWHA_OK) return st;
  uint32_t code = 0;
  int64_t where = 0;
  cudaError_t e = launch_validate(a, (cudaStream_t)stream, &code, &where);
  if (e != cudaSuccess) return cuda_status(e, "validate");
  if (code) return fail(QWHA_ERR_INVALID_ARG, "%s (at %lld)", validate_message(code), (long long)where);
  return QWHA_OK;
}

qwha_status qwha_check_stream_status(void *stream) {
  cudaError_t e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e, "stream");
  unsigned int word = 0;
  e = read_and_clear_error_word(&word, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e, "error word");
  if (word && !(word & ~(kErrSlot | kErrPage | kErrTable)))
    return fail(QWHA_ERR_INVALID_ARG, "cache: %s%s%s%s%s", word & kErrSlot ? "a slot outside the cache" : "",
                word & kErrSlot && word & (kErrPage | kErrTable) ? ", " : "",
                word & kErrPage ? "a page outside the cache or its page table" : "",
                word & kErrPage && word & kErrTable ? ", " : "",
                word & kErrTable ? "a row that contradicts the page table or would write to a shared page, or kept tokens that do not ascend" : "");
  if (word) return fail(QWHA_ERR_TIMEOUT, "device wait gave up (code 0x%x)", word);
  return QWHA_OK;
}

qwha_status qwha_init_alloc(const float *dWq, int32_t d_out, int32_t d_in, int32_t had_block, int64_t p,
                            int32_t min_per_row, qwha_remainder mode, int32_t *budgets, int32_t *row_ptr,
                            int32_t *col_idx, float *coef, void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  qwha_status st = check_hadamard(d_in, had_block);
  if (st != QWHA_OK) return st;
  if (d_in > init_max_din()) return fail(QWHA_ERR_UNSUPPORTED, "d_in %d above %d", d_in, init_max_din());
  if (min_per_row < 0 || min_per_row > d_in) return fail(QWHA_ERR_INVALID_ARG, "min_per_row %d", min_per_row);
  if (p < (int64_t)min_per_row * d_out || p > (int64_t)d_in * d_out || p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld outside [%lld, %lld]", (long long)p,
                (long long)min_per_row * d_out, (long long)d_in * d_out);
  if (mode != QWHA_REM_FEWEST_ALLOC && mode != QWHA_REM_LARGEST_ERROR)
    return fail(QWHA_ERR_INVALID_ARG, "remainder mode %d", (int)mode);
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(budgets, "budgets");
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  if (p > 0) {
    QWHA_CHECK_PTR(col_idx, "col_idx");
    QWHA_CHECK_PTR(coef, "coef");
  }
  if ((st = check_ws(ws, ws_bytes, init_workspace(d_out, d_in))) != QWHA_OK) return st;
  StageScope sc(ST_INIT, 3, (cudaStream_t)stream);
  return cuda_status(launch_init_alloc(dWq, d_out, d_in, had_block, p, min_per_row, (int)mode, budgets, row_ptr,
                                       col_idx, coef, ws, (cudaStream_t)stream),
                     "init_alloc");
}

qwha_status qwha_init_select_global(const float *dWq, int32_t d_out, int32_t d_in, int32_t had_block, int64_t p,
                                    qwha_selection sel, uint64_t seed, int32_t *budgets, int32_t *row_ptr,
                                    int32_t *col_idx, float *coef, void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  qwha_status st = check_hadamard(d_in, had_block);
  if (st != QWHA_OK) return st;
  if (d_in > init_max_din()) return fail(QWHA_ERR_UNSUPPORTED, "d_in %d above %d", d_in, init_max_din());
  if (p < 0 || p > (int64_t)d_in * d_out || p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld outside [0, %lld]", (long long)p, (long long)d_in * d_out);
  if (sel != QWHA_SEL_MAGNITUDE && sel != QWHA_SEL_RANDOM) return fail(QWHA_ERR_INVALID_ARG, "selection %d", (int)sel);
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(budgets, "budgets");
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  if (p > 0) {
    QWHA_CHECK_PTR(col_idx, "col_idx");
    QWHA_CHECK_PTR(coef, "coef");
  }
  if ((st = check_ws(ws, ws_bytes, select_global_workspace(d_out, d_in))) != QWHA_OK) return st;
  StageScope sc(ST_INIT, 21, (cudaStream_t)stream);
  return cuda_status(launch_select_global(dWq, d_out, d_in, had_block, p, (int)sel, seed, budgets, row_ptr, col_idx,
                                          coef, ws, (cudaStream_t)stream),
                     "init_select_global");
}

qwha_status qwha_energy_stats(const float *dWq, int32_t d_out, int32_t d_in, int32_t had_block, int64_t k,
                              double *stats, void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  qwha_status st = check_hadamard(d_in, had_block);
  if (st != QWHA_OK) return st;
  if (d_in > init_max_din()) return fail(QWHA_ERR_UNSUPPORTED, "d_in %d above %d", d_in, init_max_din());
  if (k < 1 || k >= (int64_t)d_in * d_out || k >= 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "k = %lld outside [1, %lld)", (long long)k, (long long)d_in * d_out);
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(stats, "stats");
  if ((st = check_ws(ws, ws_bytes, energy_stats_workspace(d_out, d_in))) != QWHA_OK) return st;
  StageScope sc(ST_INIT, 20, (cudaStream_t)stream);
  return cuda_status(launch_energy_stats(dWq, d_out, d_in, had_block, k, stats, ws, (cudaStream_t)stream),
                     "energy_stats");
}

qwha_status qwha_pattern_stats(int32_t d_out, int32_t d_in, int64_t p, const int32_t *row_ptr, const int32_t *col_idx,
                               int32_t *col_counts, int64_t *stats, void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  if (p < 0 || p > (int64_t)d_in * d_out || p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld outside [0, %lld]", (long long)p, (long long)d_in * d_out);
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  if (p > 0) QWHA_CHECK_PTR(col_idx, "col_idx");
  QWHA_CHECK_PTR(col_counts, "col_counts");
  QWHA_CHECK_PTR(stats, "stats");
  qwha_status st = check_ws(ws, ws_bytes, pattern_stats_workspace(d_in));
  if (st != QWHA_OK) return st;
  StageScope sc(ST_INIT, 4, (cudaStream_t)stream);
  return cuda_status(launch_pattern_stats(d_out, d_in, p, row_ptr, col_idx, col_counts, stats, ws,
                                          (cudaStream_t)stream),
                     "pattern_stats");
}

qwha_status qwha_calib_hessian(const void *X, int64_t T, int32_t d_in, float *S, void *stream) {
  if (T < 1 || d_in <= 0 || d_in % 8) return fail(QWHA_ERR_INVALID_ARG, "T %lld, d_in %d (a multiple of 8)", (long long)T, d_in);
  QWHA_CHECK_PTR(X, "X");
  QWHA_CHECK_PTR(S, "S");
  if ((uintptr_t)X % 16 || (uintptr_t)S % 16) return fail(QWHA_ERR_MISALIGNED, "X and S must be 16-byte aligned");
  StageScope sc(ST_INIT, 1, (cudaStream_t)stream);
  return cuda_status(launch_calib_hessian(X, T, d_in, S, (cudaStream_t)stream), "calib_hessian");
}

qwha_status qwha_refine_values(const float *dWq, int32_t d_out, int32_t d_in, int32_t had_block, const float *S,
                               float damp, const int32_t *row_ptr, const int32_t *col_idx, int64_t p, float *coef,
                               void *ws, size_t ws_bytes, void *stream) {
  if (d_out <= 0 || d_in <= 0 || d_in % 8) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d (a multiple of 8)", d_out, d_in);
  qwha_status st = check_hadamard(d_in, had_block);
  if (st != QWHA_OK) return st;
  if (!(damp >= 0.0f)) return fail(QWHA_ERR_INVALID_ARG, "damp %g", (double)damp);
  if (p < 0 || p > (int64_t)d_in * d_out || p > 2147483647LL) return fail(QWHA_ERR_INVALID_ARG, "p %lld", (long long)p);
  if (p == 0) return QWHA_OK;
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(S, "S");
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  QWHA_CHECK_PTR(col_idx, "col_idx");
  QWHA_CHECK_PTR(coef, "coef");
  if ((uintptr_t)dWq % 16 || (uintptr_t)S % 16) return fail(QWHA_ERR_MISALIGNED, "dWq and S must be 16-byte aligned");
  if ((st = check_ws(ws, ws_bytes, refine_workspace(d_out, d_in))) != QWHA_OK) return st;
  StageScope sc(ST_INIT, 14, (cudaStream_t)stream);
  return cuda_status(launch_refine(dWq, d_out, d_in, had_block, S, damp, row_ptr, col_idx, p, coef, ws,
                                   (cudaStream_t)stream),
                     "refine_values");
}

qwha_status qwha_init_norms(const float *dWq, int32_t rows, int32_t d_in, double *e, void *stream) {
  if (rows < 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "rows %d, d_in %d", rows, d_in);
  if (rows == 0) return QWHA_OK;
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(e, "e");
  StageScope sc(ST_INIT, 1, (cudaStream_t)stream);
  return cuda_status(launch_init_norms(dWq, rows, d_in, e, (cudaStream_t)stream), "init_norms");
}

qwha_status qwha_init_budgets(const double *e, int32_t d_out, int32_t d_in, int64_t p, int32_t min_per_row,
                              qwha_remainder mode, int32_t *budgets, int32_t *row_ptr, void *ws, size_t ws_bytes,
                              void *stream) {
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  if (min_per_row < 0 || min_per_row > d_in) return fail(QWHA_ERR_INVALID_ARG, "min_per_row %d", min_per_row);
  if (p < (int64_t)min_per_row * d_out || p > (int64_t)d_in * d_out || p > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "p = %lld outside [%lld, %lld]", (long long)p,
                (long long)min_per_row * d_out, (long long)d_in * d_out);
  if (mode != QWHA_REM_FEWEST_ALLOC && mode != QWHA_REM_LARGEST_ERROR)
    return fail(QWHA_ERR_INVALID_ARG, "remainder mode %d", (int)mode);
  QWHA_CHECK_PTR(e, "e");
  QWHA_CHECK_PTR(budgets, "budgets");
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  qwha_status st = check_ws(ws, ws_bytes, init_workspace(d_out, d_in));
  if (st != QWHA_OK) return st;
  StageScope sc(ST_INIT, 1, (cudaStream_t)stream);
  return cuda_status(launch_init_budgets(e, d_out, d_in, p, min_per_row, (int)mode, budgets, row_ptr, ws,
                                         (cudaStream_t)stream),
                     "init_budgets");
}

qwha_status qwha_init_select(const float *dWq, int32_t rows, int32_t d_in, int32_t had_block, const int32_t *budgets,
                             const int32_t *row_ptr, int64_t p_local, int32_t *col_idx, float *coef, void *stream) {
  if (rows < 0) return fail(QWHA_ERR_INVALID_ARG, "rows %d", rows);
  qwha_status st = check_hadamard(d_in, had_block);
  if (st != QWHA_OK) return st;
  if (d_in > init_max_din()) return fail(QWHA_ERR_UNSUPPORTED, "d_in %d above %d", d_in, init_max_din());
  if (p_local < 0 || p_local > 2147483647LL) return fail(QWHA_ERR_INVALID_ARG, "p_local %lld", (long long)p_local);
  if (rows == 0 || p_local == 0) return QWHA_OK;
  QWHA_CHECK_PTR(dWq, "dWq");
  QWHA_CHECK_PTR(budgets, "budgets");
  QWHA_CHECK_PTR(row_ptr, "row_ptr");
  QWHA_CHECK_PTR(col_idx, "col_idx");
  QWHA_CHECK_PTR(coef, "coef");
  StageScope sc(ST_INIT, 1, (cudaStream_t)stream);
  return cuda_status(launch_init_select(dWq, rows, d_in, had_block, budgets, row_ptr, p_local, col_idx, coef,
                                        (cudaStream_t)stream),
                     "init_select");
}

}  // extern "C"

// ---------------------------------------------------------------- serving

namespace {

qwha_status check_tokens(int64_t T) {
  if (T < 0) return fail(QWHA_ERR_INVALID_ARG, "T %lld < 0", (long long)T);
  if (T > QWHA_DECODE_MAX_T)
    return fail(QWHA_ERR_UNSUPPORTED, "T %lld above %d: use qwha_adapter_fwd", (long long)T, QWHA_DECODE_MAX_T);
  return QWHA_OK;
}

// A product's CTAs store their outputs while others still read the tokens.
qwha_status check_apart(const char *names, const void *p, size_t p_bytes, const void *q, size_t q_bytes) {
  const char *a = static_cast<const char *>(p), *b = static_cast<const char *>(q);
  if (a < b + q_bytes && b < a + p_bytes) return fail(QWHA_ERR_INVALID_ARG, "%s overlap", names);
  return QWHA_OK;
}

// The launches of a checked qwha_qgemv (a NULL) or qwha_adapter_decode call.
qwha_status decode_call(const qwha_adapter *a, const qwha_qweight *wq, qwha_dtype dt, const void *X, int64_t T,
                        int32_t d_out, int32_t d_in, float alpha, void *Z_out, void *Y, void *ws, cudaStream_t s) {
  GemvArgs g = {};
  if (wq) {
    g.qw = wq->qweight, g.scales = wq->scales, g.zeros = wq->zeros;
    g.bits = wq->bits, g.group = wq->group;
  }
  g.d_out = d_out, g.d_in = d_in, g.x = X, g.T = (int)T, g.f32 = dt == QWHA_F32, g.y = Y;
  const bool tensor = gemv_on_tensor_cores(g.qw, g.group);
  if (tensor) gemv_place_x(&g, ws);
  if (!a && gemv_own_x(d_in, T, g.f32)) g.xpieces = nullptr;
  if (!(g.err = device_error_word())) return fail(QWHA_ERR_CUDA, "no error word");
  if (a && a->p > 0) {
    g.row_ptr = a->row_ptr, g.col_idx = a->col_idx, g.coef = a->coef, g.p = a->p, g.alpha = alpha;
    gemv_place_z(&g, static_cast<char *>(ws) + (wq ? gemv_x_bytes(d_in, T, g.f32) : 0));
  }
  g.prepared = g.xpieces || g.zt || Z_out;
  if (g.prepared) {
    StageScope sc(ST_DECODE_PREPARE, 1, s);
    qwha_status st = cuda_status(launch_decode_prepare(g, a ? ilog2(a->had_block) : 0, Z_out, s), "decode preparation");
    if (st != QWHA_OK) return st;
  }
  if (g.zt) {
    StageScope sc(ST_DECODE_ENTRIES, 1, s);
    qwha_status st = cuda_status(launch_decode_entries(g, s), "decode entries");
    if (st != QWHA_OK) return st;
  }
  StageScope sc(ST_GEMV, 1, s);
  return cuda_status(launch_gemv(g, s), "matrix-vector product");
}

qwha_status check_cache(const qwha_cache *c) {
  if (c->bits != 2 && c->bits != 3 && c->bits != 4 && c->bits != 8)
    return fail(QWHA_ERR_INVALID_ARG, "cache bits %d not in {2,3,4,8}", c->bits);
  if (c->heads < 1 || c->heads > 65535) return fail(QWHA_ERR_INVALID_ARG, "cache heads %d", c->heads);
  if (c->head_dim < 8 || c->head_dim % 8)
    return fail(QWHA_ERR_INVALID_ARG, "cache head_dim %d must be a positive multiple of 8", c->head_dim);
  if (c->head_dim > cache_max_head_dim())
    return fail(QWHA_ERR_UNSUPPORTED, "cache head_dim %d above %d", c->head_dim, cache_max_head_dim());
  if (c->group <= 0 || c->group % 8 || c->head_dim % c->group)
    return fail(QWHA_ERR_INVALID_ARG, "cache group %d must be a multiple of 8 dividing head_dim %d", c->group,
                c->head_dim);
  if (c->had_block) {
    qwha_status st = check_hadamard(c->head_dim, c->had_block);
    if (st != QWHA_OK) return st;
  }
  if (c->page_size < 1 || c->n_pages < 0 || c->n_pages > 2147483647LL)
    return fail(QWHA_ERR_INVALID_ARG, "cache page_size %d, n_pages %lld", c->page_size, (long long)c->n_pages);
  if (c->n_pages > 0) {
    QWHA_CHECK_PTR(c->codes, "cache codes");
    QWHA_CHECK_PTR(c->scales, "cache scales");
    QWHA_CHECK_PTR(c->zeros, "cache zeros");
  }
  return QWHA_OK;
}

qwha_status check_caches(const qwha_cache *caches, int32_t n_caches, qwha_dtype dt, const void *const *rows,
                         int64_t n) {
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (n_caches < 1 || n_caches > 2) return fail(QWHA_ERR_INVALID_ARG, "n_caches %d not 1 or 2", n_caches);
  if (!caches || !rows) return fail(QWHA_ERR_INVALID_ARG, "%s is NULL", caches ? "rows" : "caches");
  if (n < 0 || n > (1LL << 40)) return fail(QWHA_ERR_INVALID_ARG, "n %lld out of range", (long long)n);
  for (int i = 0; i < n_caches; ++i) {
    qwha_status st = check_cache(caches + i);
    if (st != QWHA_OK) return st;
    if (n > 0) QWHA_CHECK_PTR(rows[i], "rows");
  }
  return QWHA_OK;
}

CachePair cache_pair(const qwha_cache *caches, int32_t n_caches, const void *const *rows) {
  CachePair c = {};
  for (int i = 0; i < n_caches; ++i) {
    c.cache[i] = caches[i];
    c.rows[i] = rows[i];
    c.unit[i] = caches[i].had_block ? 1.0 / sqrt((double)caches[i].had_block) : 1.0;
  }
  return c;
}

}  // namespace

extern "C" {

qwha_status qwha_qgemv(const qwha_qweight *wq, int32_t d_out, int32_t d_in, qwha_dtype dt, const void *X, int64_t T,
                       void *Y, void *ws, size_t ws_bytes, void *stream) {
  if (!wq) return fail(QWHA_ERR_INVALID_ARG, "wq is NULL");
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (d_out <= 0 || d_in <= 0) return fail(QWHA_ERR_INVALID_ARG, "d_out %d, d_in %d", d_out, d_in);
  qwha_status st = check_codes(wq, d_in);
  if (st != QWHA_OK || (st = check_tokens(T)) != QWHA_OK) return st;
  if (T == 0) return QWHA_OK;
  QWHA_CHECK_PTR(X, "X");
  QWHA_CHECK_PTR(Y, "Y");
  if ((st = check_ws(ws, ws_bytes, qgemv_ws(d_in, T, dt == QWHA_F32))) != QWHA_OK) return st;
  const size_t row = (size_t)T * (dt == QWHA_F32 ? 4 : 2);
  if ((st = check_apart("X and Y", X, row * d_in, Y, row * d_out)) != QWHA_OK) return st;
  return decode_call(nullptr, wq, dt, X, T, d_out, d_in, 0.f, nullptr, Y, ws, (cudaStream_t)stream);
}

qwha_status qwha_adapter_decode(const qwha_adapter *a, const qwha_qweight *wq, qwha_dtype dt, const void *X,
                                int64_t T, float alpha, void *Z_out, void *Y, void *ws, size_t ws_bytes,
                                void *stream) {
  qwha_status st = check_adapter_shape(a);
  if (st != QWHA_OK) return st;
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (wq && (st = check_codes(wq, a->d_in)) != QWHA_OK) return st;
  if ((st = check_tokens(T)) != QWHA_OK) return st;
  if (a->p > 2147483647LL - 4096) return fail(QWHA_ERR_UNSUPPORTED, "decode: p = %lld", (long long)a->p);
  if (a->z_given) return fail(QWHA_ERR_UNSUPPORTED, "a decode call computes its own transform (z_given must be 0)");
  if (T == 0) return QWHA_OK;
  QWHA_CHECK_PTR(X, "X");
  QWHA_CHECK_PTR(Y, "Y");
  if (Z_out) QWHA_CHECK_PTR(Z_out, "Z_out");
  if ((st = check_ws(ws, ws_bytes, decode_ws(a->d_out, a->d_in, a->p, T, wq != nullptr, dt == QWHA_F32))) != QWHA_OK) return st;
  const size_t row = (size_t)T * (dt == QWHA_F32 ? 4 : 2), x_bytes = row * a->d_in, y_bytes = row * a->d_out;
  if ((st = check_apart("X and Y", X, x_bytes, Y, y_bytes)) != QWHA_OK) return st;
  if (Z_out && ((st = check_apart("X and Z_out", X, x_bytes, Z_out, x_bytes)) != QWHA_OK ||
                (st = check_apart("Y and Z_out", Y, y_bytes, Z_out, x_bytes)) != QWHA_OK))
    return st;
  return decode_call(a, wq, dt, X, T, a->d_out, a->d_in, alpha, Z_out, Y, ws, (cudaStream_t)stream);
}

qwha_status qwha_cache_write(const qwha_cache *caches, int32_t n_caches, qwha_dtype dt, const void *const *rows,
                             const int64_t *slots, int64_t n, void *stream) {
  qwha_status st = check_caches(caches, n_caches, dt, rows, n);
  if (st != QWHA_OK) return st;
  if (n == 0) return QWHA_OK;
  QWHA_CHECK_PTR(slots, "slots");
  const CachePair c = cache_pair(caches, n_caches, rows);
  StageScope sc(ST_CACHE_WRITE, cache_write_launches(dt, c, n_caches), (cudaStream_t)stream);
  return cuda_status(launch_cache_write(dt, c, n_caches, slots, n, (cudaStream_t)stream), "cache_write");
}

qwha_status qwha_cache_read(const qwha_cache *caches, int32_t n_caches, qwha_dtype dt, const int32_t *pages,
                            int32_t max_pages, const int64_t *row_start, const int64_t *first, int32_t n_seqs,
                            void *const *rows, int64_t n, void *stream) {
  qwha_status st = check_caches(caches, n_caches, dt, rows, n);
  if (st != QWHA_OK) return st;
  if (n_seqs < 0 || max_pages < 0) return fail(QWHA_ERR_INVALID_ARG, "n_seqs %d, max_pages %d", n_seqs, max_pages);
  if (n == 0 || n_seqs == 0) return QWHA_OK;
  if (max_pages > 0) QWHA_CHECK_PTR(pages, "pages");
  QWHA_CHECK_PTR(row_start, "row_start");
  if (first) QWHA_CHECK_PTR(first, "first");
  const CachePair c = cache_pair(caches, n_caches, rows);
  StageScope sc(ST_CACHE_READ, cache_read_launches(c, n_caches), (cudaStream_t)stream);
  const ReadArgs r = {pages, max_pages, n_seqs, row_start, first};
  return cuda_status(launch_cache_read(dt, c, n_caches, r, n, (cudaStream_t)stream), "cache_read");
}

qwha_status qwha_validate_slots(const qwha_cache *cache, const int64_t *slots, int64_t n, void *ws, size_t ws_bytes,
                                void *stream) {
  if (!cache) return fail(QWHA_ERR_INVALID_ARG, "cache is NULL");
  qwha_status st = check_cache(cache);
  if (st != QWHA_OK) return st;
  if (n < 0 || n > (1LL << 40)) return fail(QWHA_ERR_INVALID_ARG, "n %lld out of range", (long long)n);
  if (n == 0) return QWHA_OK;
  QWHA_CHECK_PTR(slots, "slots");
  const int64_t n_slots = cache->n_pages * cache->page_size;
  if ((st = check_ws(ws, ws_bytes, check_slots_bytes(n_slots))) != QWHA_OK) return st;
  unsigned long long bad = 0;
  cudaError_t e = launch_check_slots(slots, n, n_slots, ws, &bad, (cudaStream_t)stream);
  if (e != cudaSuccess) return cuda_status(e, "validate_slots");
  if (bad != ~0ull)
    return fail(QWHA_ERR_INVALID_ARG, "%s (at %llu)", bad & 1 ? "a slot named twice" : "a slot outside the cache",
                bad >> 1);
  return QWHA_OK;
}

}  // extern "C"

namespace {

// n rows of `width` elements, `stride` apart, of two blocks: whether one writes
// what the other holds. Blocks with one stride may interleave.
bool rows_apart(const void *x, int64_t xs, int64_t xw, const void *y, int64_t ys, int64_t yw, int64_t n, int64_t esz) {
  const int64_t a = (int64_t)(uintptr_t)x, b = (int64_t)(uintptr_t)y;
  const int64_t a1 = a + ((n - 1) * xs + xw) * esz, b1 = b + ((n - 1) * ys + yw) * esz;
  if (a1 <= b || b1 <= a) return true;
  if (xs != ys) return false;
  const int64_t step = xs * esz, off = ((b - a) % step + step) % step;  // of a row of y behind one of x
  return off >= xw * esz && off + yw * esz <= step;
}

// Index arrays, which the kernels read one element at a time, need only the
// alignment of their elements: rows of a table or parts of a batch are passed as
// they lie.
#define QWHA_CHECK_INDEX(p, name)                                                                                \
  do {                                                                                                           \
    if (!(p)) return fail(QWHA_ERR_INVALID_ARG, "%s is NULL", name);                                             \
    if ((uintptr_t)(p) % sizeof(*(p))) return fail(QWHA_ERR_MISALIGNED, "%s is not aligned to its elements", name); \
  } while (0)

qwha_status check_table(const qwha_page_table *t) {
  if (!t) return fail(QWHA_ERR_INVALID_ARG, "the page table is NULL");
  if (t->page_size < 1 || t->max_pages < 0 || t->n_seqs < 0 || t->n_pages < 0)
    return fail(QWHA_ERR_INVALID_ARG, "page_size %d, max_pages %d, n_seqs %d, n_pages %d", t->page_size, t->max_pages,
                t->n_seqs, t->n_pages);
  if (t->n_pages > 0) QWHA_CHECK_INDEX(t->refs, "refs");
  if (t->n_seqs > 0 && t->max_pages > 0) QWHA_CHECK_INDEX(t->pages, "pages");
  if (t->n_seqs > 0) QWHA_CHECK_INDEX(t->held, "held");
  return QWHA_OK;
}

qwha_status check_moved(const qwha_cache *caches, int32_t n_caches) {
  if (n_caches < 1 || n_caches > 2) return fail(QWHA_ERR_INVALID_ARG, "n_caches %d not 1 or 2", n_caches);
  if (!caches) return fail(QWHA_ERR_INVALID_ARG, "caches is NULL");
  for (int i = 0; i < n_caches; ++i) {
    const qwha_status st = check_cache(caches + i);
    if (st != QWHA_OK) return st;
  }
  return QWHA_OK;
}

qwha_status resize(const qwha_page_table &t, const int64_t *want, int32_t *from, int32_t *to, void *ws, size_t ws_bytes,
                   void *stream) {
  QWHA_CHECK_INDEX(want, "want");
  const qwha_status st = check_ws(ws, ws_bytes, pages_workspace(t.n_seqs, t.n_pages, 0));
  if (st != QWHA_OK) return st;
  StageScope sc(ST_PAGES, 1, (cudaStream_t)stream);
  return cuda_status(launch_pages_resize(t, want, from, to, ws, (cudaStream_t)stream), "pages_resize");
}

qwha_status attend(const qwha_cache *k, const qwha_cache *v, qwha_dtype dt, const void *q, int64_t n,
                   int32_t q_heads, int64_t q_stride, const int32_t *pages, int32_t max_pages,
                   const int64_t *q_start, const int64_t *past, int32_t n_seqs, const int64_t *tree, float scale,
                   int64_t longest, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (!k || !v) return fail(QWHA_ERR_INVALID_ARG, "%s is NULL", k ? "v" : "k");
  qwha_status st = check_cache(k);
  if (st != QWHA_OK || (st = check_cache(v)) != QWHA_OK) return st;
  if (k->heads != v->heads || k->head_dim != v->head_dim || k->page_size != v->page_size || k->n_pages != v->n_pages)
    return fail(QWHA_ERR_INVALID_ARG, "the caches of keys and values differ in heads, head_dim, page_size or n_pages");
  if (q_heads < 1 || q_heads > 65535 || q_heads % k->heads)
    return fail(QWHA_ERR_INVALID_ARG, "q_heads %d must be a multiple of the cache's heads %d", q_heads, k->heads);
  if (n < 0 || n > 2147483647LL) return fail(QWHA_ERR_INVALID_ARG, "n %lld out of range", (long long)n);
  if (n_seqs < 0 || max_pages < 0) return fail(QWHA_ERR_INVALID_ARG, "n_seqs %d, max_pages %d", n_seqs, max_pages);
  if (!isfinite(scale)) return fail(QWHA_ERR_INVALID_ARG, "scale is not finite");
  const int64_t esz = dt == QWHA_F32 ? 4 : 2, row = (int64_t)q_heads * k->head_dim;
  if (q_stride < row || q_stride > (1LL << 32))
    return fail(QWHA_ERR_INVALID_ARG, "q_stride %lld of tokens of %lld elements", (long long)q_stride, (long long)row);
  if (q_stride * esz % 16) return fail(QWHA_ERR_MISALIGNED, "q_stride must be a multiple of 16 bytes");
  if (n == 0 || n_seqs == 0) return QWHA_OK;
  QWHA_CHECK_PTR(q, "q");
  QWHA_CHECK_PTR(out, "out");
  if (max_pages > 0) QWHA_CHECK_INDEX(pages, "pages");
  QWHA_CHECK_INDEX(q_start, "q_start");
  QWHA_CHECK_INDEX(past, "past");
  if (tree) QWHA_CHECK_INDEX(tree, "tree");
  if (lse) QWHA_CHECK_PTR(lse, "lse");
  if ((st = check_ws(ws, ws_bytes, attention_workspace(q_heads, k->head_dim, k->heads, n, dt == QWHA_F32))) != QWHA_OK)
    return st;
  const size_t q_bytes = (size_t)(((n - 1) * q_stride + row) * esz), out_bytes = (size_t)(n * row * esz);
  if ((st = check_apart("q and out", q, q_bytes, out, out_bytes)) != QWHA_OK) return st;
  if (lse && ((st = check_apart("q and lse", q, q_bytes, lse, (size_t)n * q_heads * 4)) != QWHA_OK ||
              (st = check_apart("out and lse", out, out_bytes, lse, (size_t)n * q_heads * 4)) != QWHA_OK))
    return st;
  AttnArgs a = {};
  a.k = *k, a.v = *v;
  a.unit_k = k->had_block ? (float)(1.0 / sqrt((double)k->had_block)) : 1.f;
  a.unit_v = v->had_block ? (float)(1.0 / sqrt((double)v->had_block)) : 1.f;
  a.q = q, a.q_stride = q_stride, a.n = n, a.q_heads = q_heads, a.grp = q_heads / k->heads;
  a.pages = pages, a.max_pages = max_pages;
  a.cap = (int)std::min<int64_t>((int64_t)max_pages * k->page_size, 1 << 30);
  a.longest = (int)std::min<int64_t>(a.cap, longest);
  const int lg = ilog2(k->page_size);  // 2^lg >= page_size: the product of 31 and 32 bits is exact where it counts
  a.page_shift = 31 + lg, a.page_mul = (unsigned int)(((1ull << a.page_shift) + k->page_size - 1) / k->page_size);
  a.q_start = q_start, a.past = past, a.n_seqs = n_seqs, a.tree = tree;
  a.scale2 = (float)(scale * 1.4426950408889634), a.out = out, a.lse = lse, a.f32 = dt == QWHA_F32;
  StageScope sc(ST_ATTENTION, attention_launches(a), (cudaStream_t)stream);
  return cuda_status(launch_attention(a, ws, (cudaStream_t)stream), "cache_attention");
}

CachePair moved_pair(const qwha_cache *caches, int32_t n_caches) {
  CachePair c = {};
  for (int i = 0; i < n_caches; ++i) c.cache[i] = caches[i];
  return c;
}

}  // namespace

extern "C" {

qwha_status qwha_rotary(qwha_dtype dt, int32_t n_x, const void *const *x, const int64_t *x_stride, void *const *y,
                        const int64_t *y_stride, const int32_t *heads, int32_t head_dim, int64_t n,
                        const int64_t *positions, const double *freq, int32_t rot, qwha_rotary_layout layout,
                        float factor, int32_t inverse, void *stream) {
  if (!valid_dtype(dt)) return fail(QWHA_ERR_INVALID_ARG, "dtype %d", (int)dt);
  if (n_x < 1 || n_x > 2) return fail(QWHA_ERR_INVALID_ARG, "n_x %d not 1 or 2", n_x);
  if (!x || !y || !x_stride || !y_stride || !heads) return fail(QWHA_ERR_INVALID_ARG, "x, y, strides or heads is NULL");
  if (head_dim < 8 || head_dim % 8 || head_dim > 32768)
    return fail(QWHA_ERR_INVALID_ARG, "head_dim %d must be a positive multiple of 8", head_dim);
  if (head_dim > cache_max_head_dim())
    return fail(QWHA_ERR_UNSUPPORTED, "head_dim %d above %d", head_dim, cache_max_head_dim());
  if (rot < 0 || rot % 2 || rot > head_dim)
    return fail(QWHA_ERR_INVALID_ARG, "rot %d must be even and at most head_dim %d", rot, head_dim);
  if (layout != QWHA_ROTARY_HALF && layout != QWHA_ROTARY_PAIRS) return fail(QWHA_ERR_INVALID_ARG, "layout %d", (int)layout);
  if (n < 0 || n > (1LL << 40)) return fail(QWHA_ERR_INVALID_ARG, "n %lld out of range", (long long)n);
  if (!isfinite(factor)) return fail(QWHA_ERR_INVALID_ARG, "factor is not finite");
  const int64_t esz = dt == QWHA_F32 ? 4 : 2;
  for (int i = 0; i < n_x; ++i) {
    if (heads[i] < 1 || heads[i] > 65535) return fail(QWHA_ERR_INVALID_ARG, "heads %d", heads[i]);
    const int64_t w = (int64_t)heads[i] * head_dim;
    if (x_stride[i] < w || y_stride[i] < w || x_stride[i] > (1LL << 32) || y_stride[i] > (1LL << 32))
      return fail(QWHA_ERR_INVALID_ARG, "strides %lld and %lld of tokens of %lld elements", (long long)x_stride[i],
                  (long long)y_stride[i], (long long)w);
    if (x_stride[i] * esz % 16 || y_stride[i] * esz % 16)
      return fail(QWHA_ERR_MISALIGNED, "the strides of tokens must be multiples of 16 bytes");
  }
  if (n == 0) return QWHA_OK;
  RotaryArgs r = {};
  for (int i = 0; i < n_x; ++i) {
    QWHA_CHECK_PTR(x[i], "x");
    QWHA_CHECK_PTR(y[i], "y");
    r.x[i] = x[i], r.y[i] = y[i], r.x_stride[i] = x_stride[i], r.y_stride[i] = y_stride[i], r.heads[i] = heads[i];
  }
  QWHA_CHECK_INDEX(positions, "positions");
  if (rot > 0) QWHA_CHECK_INDEX(freq, "freq");
  for (int i = 0; i < n_x; ++i)
    for (int j = 0; j < n_x; ++j) {
      const int64_t xw = (int64_t)heads[i] * head_dim, yw = (int64_t)heads[j] * head_dim;
      if (i == j && x[i] == y[i] && x_stride[i] == y_stride[i]) continue;  // in place
      if (!rows_apart(x[i], x_stride[i], xw, y[j], y_stride[j], yw, n, esz))
        return fail(QWHA_ERR_INVALID_ARG, "x and y overlap (in place is x itself, with its stride)");
    }
  if (n_x == 2 && !rows_apart(y[0], y_stride[0], (int64_t)heads[0] * head_dim, y[1], y_stride[1],
                              (int64_t)heads[1] * head_dim, n, esz))
    return fail(QWHA_ERR_INVALID_ARG, "the two outputs overlap");
  r.head_dim = head_dim, r.rot = rot, r.n = n, r.positions = positions, r.freq = freq, r.factor = factor;
  r.pairs = layout == QWHA_ROTARY_PAIRS, r.inverse = inverse != 0;
  StageScope sc(ST_ROTARY, 1, (cudaStream_t)stream);
  return cuda_status(launch_rotary(dt, r, (cudaStream_t)stream), "rotary");
}

qwha_status qwha_cache_attention(const qwha_cache *k, const qwha_cache *v, qwha_dtype dt, const void *q, int64_t n,
                                 int32_t q_heads, int64_t q_stride, const int32_t *pages, int32_t max_pages,
                                 const int64_t *q_start, const int64_t *past, int32_t n_seqs, const int64_t *tree,
                                 float scale, void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
  return attend(k, v, dt, q, n, q_heads, q_stride, pages, max_pages, q_start, past, n_seqs, tree, scale, INT64_MAX, out, lse, ws,
                ws_bytes, stream);
}

qwha_status qwha_cache_attention_upto(const qwha_cache *k, const qwha_cache *v, qwha_dtype dt, const void *q, int64_t n,
                                      int32_t q_heads, int64_t q_stride, const int32_t *pages, int32_t max_pages,
                                      const int64_t *q_start, const int64_t *past, int32_t n_seqs, const int64_t *tree,
                                      float scale, int64_t longest, void *out, float *lse, void *ws, size_t ws_bytes,
                                      void *stream) {
  if (longest < 0) return fail(QWHA_ERR_INVALID_ARG, "longest %lld is negative", (long long)longest);
  return attend(k, v, dt, q, n, q_heads, q_stride, pages, max_pages, q_start, past, n_seqs, tree, scale, longest, out, lse, ws,
                ws_bytes, stream);
}

qwha_status qwha_pages_resize(const qwha_page_table *t, const int64_t *want, void *ws, size_t ws_bytes, void *stream) {
  qwha_status st = check_table(t);
  if (st != QWHA_OK || t->n_seqs == 0) return st;
  return resize(*t, want, nullptr, nullptr, ws, ws_bytes, stream);
}

qwha_status qwha_pages_resize_copies(const qwha_page_table *t, const int64_t *want, int32_t *from, int32_t *to, void *ws,
                                     size_t ws_bytes, void *stream) {
  qwha_status st = check_table(t);
  if (st != QWHA_OK || t->n_seqs == 0) return st;
  QWHA_CHECK_INDEX(from, "from");
  QWHA_CHECK_INDEX(to, "to");
  if ((st = check_apart("from and to", from, (size_t)t->n_seqs * 4, to, (size_t)t->n_seqs * 4)) != QWHA_OK) return st;
  return resize(*t, want, from, to, ws, ws_bytes, stream);
}

qwha_status qwha_pages_fork(const qwha_page_table *t, const int64_t *src, const int64_t *dst, int32_t m, int32_t *from,
                            int32_t *to, void *ws, size_t ws_bytes, void *stream) {
  qwha_status st = check_table(t);
  if (st != QWHA_OK) return st;
  if (m < 0) return fail(QWHA_ERR_INVALID_ARG, "m %d", m);
  if (m == 0) return QWHA_OK;
  QWHA_CHECK_INDEX(src, "src");
  QWHA_CHECK_INDEX(dst, "dst");
  QWHA_CHECK_INDEX(from, "from");
  QWHA_CHECK_INDEX(to, "to");
  if ((st = check_ws(ws, ws_bytes, pages_workspace(t->n_seqs, t->n_pages, m))) != QWHA_OK) return st;
  StageScope sc(ST_PAGES, 1, (cudaStream_t)stream);
  return cuda_status(launch_pages_fork(*t, src, dst, m, from, to, ws, (cudaStream_t)stream), "pages_fork");
}

qwha_status qwha_cache_copy_pages(const qwha_cache *caches, int32_t n_caches, const int32_t *from, const int32_t *to,
                                  int32_t m, void *stream) {
  const qwha_status st = check_moved(caches, n_caches);
  if (st != QWHA_OK) return st;
  if (m < 0) return fail(QWHA_ERR_INVALID_ARG, "m %d", m);
  if (m == 0) return QWHA_OK;
  QWHA_CHECK_INDEX(from, "from");
  QWHA_CHECK_INDEX(to, "to");
  StageScope sc(ST_CACHE_MOVE, 1, (cudaStream_t)stream);
  return cuda_status(launch_copy_pages(moved_pair(caches, n_caches), n_caches, from, to, m, (cudaStream_t)stream),
                     "cache_copy_pages");
}

qwha_status qwha_cache_compact(const qwha_cache *caches, int32_t n_caches, const int32_t *pages, int32_t max_pages,
                               const int64_t *first, const int32_t *keep, int32_t width, int32_t n_seqs, void *stream) {
  const qwha_status st = check_moved(caches, n_caches);
  if (st != QWHA_OK) return st;
  if (n_seqs < 0 || max_pages < 0 || width < 0)
    return fail(QWHA_ERR_INVALID_ARG, "n_seqs %d, max_pages %d, width %d", n_seqs, max_pages, width);
  if (n_seqs == 0 || width == 0) return QWHA_OK;
  if (max_pages > 0) QWHA_CHECK_INDEX(pages, "pages");
  QWHA_CHECK_INDEX(first, "first");
  QWHA_CHECK_INDEX(keep, "keep");
  StageScope sc(ST_CACHE_MOVE, (int)cdiv(n_seqs, 65535), (cudaStream_t)stream);
  return cuda_status(launch_compact(moved_pair(caches, n_caches), n_caches, pages, max_pages, first, keep, width, n_seqs,
                                    (cudaStream_t)stream),
                     "cache_compact");
}

}  // extern "C"
