// C ABI of libonebit: host-side validation, workspace carving, launches.
// Every check runs before the first HIP call, so invalid calls touch nothing.
#include <math.h>

#include <algorithm>
#include <initializer_list>
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "attention.h"
#include "common.h"
#include "train.h"

using namespace onebit;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

constexpr int32_t kMaxWorkers = 64;

int check_rows(int64_t N, int32_t n) {
    if (n < 1 || n > kMaxWorkers) return ONEBIT_E_SIZE;
    if (N < 0) return ONEBIT_E_SIZE;
    if (N % (64 * (int64_t)n)) return ONEBIT_E_SIZE;
    // chunk length below 2^31: keeps the fp64 sums' addition depth (about
    // L / 2^18 + 21) within the finalize's certified bound
    if (N / n >= (int64_t)1 << 31) return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

// Segment tables live in device memory; the host can check only what it sees.
int check_segments(const int64_t* seg_off, const float* seg_k, int32_t n_seg, bool need_k) {
    if (seg_off == nullptr && seg_k == nullptr && n_seg == 0) return ONEBIT_OK;
    if (seg_off == nullptr || (need_k && seg_k == nullptr)) return ONEBIT_E_NULL;
    if (n_seg < 1) return ONEBIT_E_ARG;
    if (!aligned(seg_off, 8) || (seg_k && !aligned(seg_k, 4))) return ONEBIT_E_ALIGN;
    return ONEBIT_OK;
}

size_t round_up(size_t x) { return (x + 255) & ~(size_t)255; }

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A dispatch counts its grid in work-items with 32 bits: a launch takes at
// most 2^32 - 1 work-items along x, i.e. 16,777,215 workgroups of 256.
// Larger requests would be cut short without an error, so they are refused.
bool groups_ok(int64_t groups) {
    return groups >= 0 && groups <= (int64_t)(0xFFFFFFFFu / kThreads);
}

// LAMB step: the layer keys, then one slot per workgroup of the pass
size_t lamb_ws_bytes(int64_t N, int32_t n_seg) {
    return round_up((size_t)n_seg * sizeof(uint32_t)) +
           round_up((size_t)lamb_workgroups(N) * sizeof(uint32_t));
}

// Warmup layer passes: plan table, per-workgroup binary64 pairs, layer RMS.
WarmupWs split_warmup_ws(void* ws, int64_t N, int32_t n_seg) {
    char* p = static_cast<char*>(ws);
    WarmupWs w;
    w.wg_first = reinterpret_cast<int64_t*>(p);
    p += round_up((size_t)(n_seg + 1) * sizeof(int64_t));
    w.part = reinterpret_cast<double2*>(p);
    p += round_up((size_t)layer_grid(N, n_seg) * 2 * sizeof(double));
    w.rms = reinterpret_cast<double*>(p);
    p += round_up((size_t)n_seg * sizeof(double));
    w.need = reinterpret_cast<int32_t*>(p);
    p += round_up((size_t)(n_seg + 1) * sizeof(int32_t));
    w.rms_exact = reinterpret_cast<double*>(p);
    p += round_up((size_t)n_seg * sizeof(double));
    w.slots = reinterpret_cast<uint64_t*>(p);
    return w;
}

size_t partial_bytes(int64_t N, int32_t n) {
    const int64_t L = N / n;
    const ChunkPlan pw = make_plan(L, (int64_t)n * n, kCompressIters);
    const ChunkPlan ps = server_plan(L, n);
    const int64_t w = pw.bpc * n * n;
    const int64_t s = ps.bpc * n;
    return round_up((size_t)(w > s ? w : s) * sizeof(double));
}

int hip_status(hipError_t e) { return e == hipSuccess ? ONEBIT_OK : ONEBIT_E_HIP; }

// The launch helpers return hipGetLastError after their launches, which
// reports the last error of any HIP call on this thread.  An entry point
// therefore drops an error an earlier call left behind (a caller's stream
// or event query that returned hipErrorNotReady, say) before its first
// launch, so that its status reflects only its own launches.
void drop_stale_error() { (void)hipGetLastError(); }

// Scratch of onebit_server_reduce_noalloc: the fp64 partial sums of the
// server's chunk means (one per workgroup), in a file-scope device array.
// Every device the library runs on holds its own copy until the process
// ends.  Host code never passes the array's name to a kernel (on the host it
// is only a stand-in symbol): the device address comes from
// hipGetSymbolAddress, looked up once per device with that device current.
constexpr size_t kNoAllocDoubles = (size_t)1 << 20;  // 8 MiB
__device__ __align__(256) double scratch[kNoAllocDoubles];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
double* g_scratch[kMaxDevices];  // device address of `scratch`, per device

int scratch_of_current_device(double** out) {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return ONEBIT_E_HIP;
    if (dev < 0 || dev >= kMaxDevices) return ONEBIT_E_ARG;
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (g_scratch[dev] == nullptr) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr)
            return ONEBIT_E_HIP;
        g_scratch[dev] = static_cast<double*>(p);
    }
    *out = g_scratch[dev];
    return ONEBIT_OK;
}

}  // namespace

namespace onebit {
// the chunk-mean finalize that first copies each scale it will overwrite to
// prev (finalize.hip); ONEBIT_KEEP_PREV passes the second half of sv_scales
hipError_t launch_mean_finalize_keep(const double* partials, const ChunkPlan& plan,
                                     int64_t pairs, MeanTarget tgt, float* prev, hipStream_t st);
}  // namespace onebit

extern "C" {

const char* onebit_strerror(int status) {
    switch (status) {
        case ONEBIT_OK: return "ok";
        case ONEBIT_E_NULL: return "required pointer is NULL";
        case ONEBIT_E_SIZE: return "invalid size (N must be a multiple of 64*n, 1 <= n <= 64, N/n < 2^31; block and N must agree; grids within 2^32 work-items)";
        case ONEBIT_E_ALIGN: return "pointer misaligned (streamed float buffers need 16 bytes)";
        case ONEBIT_E_WORKSPACE: return "workspace missing or smaller than onebit_workspace_bytes()";
        case ONEBIT_E_ARG: return "invalid argument";
        case ONEBIT_E_HIP: return "HIP runtime error on launch";
        default: return "unknown status";
    }
}

size_t onebit_workspace_bytes(int64_t N, int32_t n, int32_t n_seg) {
    if (check_rows(N, n) != ONEBIT_OK || n_seg < 0) return 0;
    if (N == 0) return 256;
    return partial_bytes(N, n) + round_up((size_t)(n_seg > 0 ? n_seg : 1) * sizeof(uint32_t));
}

size_t frozen_v_workspace_bytes(int64_t N, int32_t n_seg) {
    if (N < 0 || (N % 4) || n_seg < 1) return 0;
    return lamb_ws_bytes(N, n_seg);
}

int onebit_compress_ex(const float* m, const uint32_t* mb_bits, const float* mb_scales, float beta1,
                       float* ef, float* scales, uint32_t* bits, int64_t N, int32_t n, float clip,
                       int32_t reset, const int64_t* seg_off, const float* seg_k,
                       const float* seg_err_ratio, int32_t n_seg, uint32_t flags, void* ws,
                       size_t ws_bytes, hipStream_t stream) {
    int st = check_rows(N, n);
    if (st) return st;
    if (!m || !ef || !scales || !bits) return ONEBIT_E_NULL;
    if ((mb_bits == nullptr) != (mb_scales == nullptr)) return ONEBIT_E_NULL;
    if ((st = check_segments(seg_off, seg_k, n_seg, true))) return st;
    if (seg_err_ratio && !seg_off) return ONEBIT_E_ARG;
    if (!aligned(m, 16) || !aligned(ef, 16) || !aligned(scales, 4) || !aligned(bits, 4) ||
        (mb_bits && !aligned(mb_bits, 4)) || (mb_scales && !aligned(mb_scales, 4)) ||
        (seg_err_ratio && !aligned(seg_err_ratio, 4)))
        return ONEBIT_E_ALIGN;
    if (clip != clip || beta1 != beta1 || (flags & ~ONEBIT_UNIT_SCALE)) return ONEBIT_E_ARG;
    if (N == 0) return ONEBIT_OK;
    const size_t need = onebit_workspace_bytes(N, n, n_seg);
    if (!ws || ws_bytes < need) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;

    const ChunkPlan plan = make_plan(N / n, (int64_t)n * n, kCompressIters);
    if (sum_depth(plan) > kMaxSumDepth || !groups_ok(plan.bpc)) return ONEBIT_E_SIZE;
    const bool clamp_on = clip > 0.0f && !isinf(clip);
    double* partials = static_cast<double*>(ws);
    CompressArgs a{m, ef, scales, bits, partials, N, n, clip, clamp_on, reset != 0,
                   seg_off, seg_k, n_seg, mb_bits, mb_scales, beta1, seg_err_ratio};
    drop_stale_error();
    hipError_t e = launch_compress(a, plan, stream);
    if (e != hipSuccess) return ONEBIT_E_HIP;
    MeanTarget tgt{ef, N, n, scales, (flags & ONEBIT_UNIT_SCALE) != 0};
    return hip_status(launch_mean_finalize(partials, plan, (int64_t)n * n, tgt, stream));
}

int onebit_compress(const float* m, float* ef, float* scales, uint32_t* bits, int64_t N, int32_t n,
                    float clip, int32_t reset, const int64_t* seg_off, const float* seg_k,
                    int32_t n_seg, void* ws, size_t ws_bytes, hipStream_t stream) {
    return onebit_compress_ex(m, nullptr, nullptr, 0.0f, ef, scales, bits, N, n, clip, reset,
                              seg_off, seg_k, nullptr, n_seg, 0u, ws, ws_bytes, stream);
}

int onebit_compress_grad(const float* g, const uint32_t* mb_bits, const float* mb_scales,
                         float beta1, float* ef, float* scales, uint32_t* bits, int64_t N,
                         int32_t n, float clip, int32_t reset, const int64_t* seg_off,
                         const float* seg_k, int32_t n_seg, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
    if (!mb_bits || !mb_scales) return ONEBIT_E_NULL;
    return onebit_compress_ex(g, mb_bits, mb_scales, beta1, ef, scales, bits, N, n, clip, reset,
                              seg_off, seg_k, nullptr, n_seg, 0u, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// Argument checks of the server calls (everything but the scratch).
int check_server(const uint32_t* bits, const float* scales, float* ef, float* sv_scales,
                 uint32_t* sv_bits, float* m_out, const int64_t* seg_off, const float* seg_k,
                 const float* seg_err_ratio, int32_t n_seg, int64_t N, int32_t n,
                 uint32_t flags) {
    int st = check_rows(N, n);
    if (st) return st;
    if (!bits || !scales || !ef || !sv_scales || !sv_bits) return ONEBIT_E_NULL;
    if ((st = check_segments(seg_off, seg_k, n_seg, true))) return st;
    if (seg_err_ratio && !seg_off) return ONEBIT_E_ARG;
    if (!aligned(bits, 4) || !aligned(scales, 4) || !aligned(ef, 16) || !aligned(sv_scales, 4) ||
        !aligned(sv_bits, 4) || (m_out && !aligned(m_out, 16)) ||
        (seg_err_ratio && !aligned(seg_err_ratio, 4)))
        return ONEBIT_E_ALIGN;
    if (flags & ~(ONEBIT_UNIT_SCALE | ONEBIT_KEEP_PREV)) return ONEBIT_E_ARG;
    if (N == 0) return ONEBIT_OK;
    const ChunkPlan plan = server_plan(N / n, n);
    if (sum_depth(plan) > kMaxSumDepth || !groups_ok(plan.bpc)) return ONEBIT_E_SIZE;
    if (m_out && !groups_ok(ceil_div(N, (int64_t)kDecompressTiles * kTile))) return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

// The server's launches on validated arguments, with the partial sums in
// `partials` (server_plan(N / n, n).bpc * n doubles).
int server_launch(const uint32_t* bits, const float* scales, float* ef, float* sv_scales,
                  uint32_t* sv_bits, float* m_out, const int64_t* seg_off, const float* seg_k,
                  const float* seg_err_ratio, int32_t n_seg, int64_t N, int32_t n,
                  int32_t reset, uint32_t flags, double* partials, hipStream_t stream) {
    const ChunkPlan plan = server_plan(N / n, n);
    drop_stale_error();
    hipError_t e = launch_server(bits, scales, ef, sv_scales, sv_bits, partials, N, n, plan,
                                 reset != 0, seg_off, seg_err_ratio, n_seg, stream);
    if (e != hipSuccess) return ONEBIT_E_HIP;
    MeanTarget tgt{ef, N, n, sv_scales, (flags & ONEBIT_UNIT_SCALE) != 0};
    // ONEBIT_KEEP_PREV: the finalize copies the scales it replaces to [n, 2n)
    e = launch_mean_finalize_keep(partials, plan, n, tgt,
                                  (flags & ONEBIT_KEEP_PREV) ? sv_scales + n : nullptr, stream);
    if (e != hipSuccess) return ONEBIT_E_HIP;
    if (m_out)
        return hip_status(
            launch_decompress(sv_bits, sv_scales, m_out, seg_off, seg_k, n_seg, N, n, stream));
    return ONEBIT_OK;
}

}  // namespace

extern "C" {

int onebit_server_reduce_ex(const uint32_t* bits, const float* scales, float* ef,
                            float* sv_scales, uint32_t* sv_bits, float* m_out,
                            const int64_t* seg_off, const float* seg_k,
                            const float* seg_err_ratio, int32_t n_seg, int64_t N, int32_t n,
                            int32_t reset, uint32_t flags, void* ws, size_t ws_bytes,
                            hipStream_t stream) {
    int st = check_server(bits, scales, ef, sv_scales, sv_bits, m_out, seg_off, seg_k,
                          seg_err_ratio, n_seg, N, n, flags);
    if (st || N == 0) return st;
    const size_t need = onebit_workspace_bytes(N, n, n_seg);
    if (!ws || ws_bytes < need) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    return server_launch(bits, scales, ef, sv_scales, sv_bits, m_out, seg_off, seg_k,
                         seg_err_ratio, n_seg, N, n, reset, flags, static_cast<double*>(ws),
                         stream);
}

int onebit_server_reduce_noalloc(const uint32_t* bits, const float* scales, float* ef,
                                 float* sv_scales, uint32_t* sv_bits, float* m_out,
                                 const int64_t* seg_off, const float* seg_k,
                                 const float* seg_err_ratio, int32_t n_seg, int64_t N, int32_t n,
                                 int32_t reset, uint32_t flags, hipStream_t stream) {
    int st = check_server(bits, scales, ef, sv_scales, sv_bits, m_out, seg_off, seg_k,
                          seg_err_ratio, n_seg, N, n, flags);
    if (st || N == 0) return st;
    const ChunkPlan plan = server_plan(N / n, n);
    if ((size_t)(plan.bpc * n) > kNoAllocDoubles) return ONEBIT_E_WORKSPACE;
    double* partials = nullptr;
    if ((st = scratch_of_current_device(&partials))) return st;
    // every partial the finalize reads is written by this call's server
    // kernel first, so the scratch needs no clearing
    return server_launch(bits, scales, ef, sv_scales, sv_bits, m_out, seg_off, seg_k,
                         seg_err_ratio, n_seg, N, n, reset, flags, partials, stream);
}

int onebit_server_reduce(const uint32_t* bits, const float* scales, float* ef, float* sv_scales,
                         uint32_t* sv_bits, float* m_out, const int64_t* seg_off,
                         const float* seg_k, int32_t n_seg, int64_t N, int32_t n, int32_t reset,
                         void* ws, size_t ws_bytes, hipStream_t stream) {
    return onebit_server_reduce_ex(bits, scales, ef, sv_scales, sv_bits, m_out, seg_off, seg_k,
                                   nullptr, n_seg, N, n, reset, 0u, ws, ws_bytes, stream);
}

int onebit_decompress(const uint32_t* sv_bits, const float* sv_scales, float* m_out,
                      const int64_t* seg_off, const float* seg_k, int32_t n_seg, int64_t N,
                      int32_t n, hipStream_t stream) {
    int st = check_rows(N, n);
    if (st) return st;
    if (!sv_bits || !sv_scales || !m_out) return ONEBIT_E_NULL;
    if ((st = check_segments(seg_off, seg_k, n_seg, true))) return st;
    if (!aligned(sv_bits, 4) || !aligned(sv_scales, 4) || !aligned(m_out, 16)) return ONEBIT_E_ALIGN;
    if (N == 0) return ONEBIT_OK;
    if (!groups_ok(ceil_div(N, (int64_t)kDecompressTiles * kTile))) return ONEBIT_E_SIZE;
    drop_stale_error();
    return hip_status(
        launch_decompress(sv_bits, sv_scales, m_out, seg_off, seg_k, n_seg, N, n, stream));
}

int onebit_error_materialize(const float* ef, const float* scales, float* e_out, int64_t N,
                             int32_t rows, int32_t n, hipStream_t stream) {
    int st = check_rows(N, n);
    if (st) return st;
    if (rows < 1 || rows > kMaxWorkers) return ONEBIT_E_SIZE;
    if (!ef || !scales || !e_out) return ONEBIT_E_NULL;
    if (!aligned(ef, 16) || !aligned(e_out, 16) || !aligned(scales, 4)) return ONEBIT_E_ALIGN;
    if (N == 0) return ONEBIT_OK;
    if (!groups_ok(ceil_div(N, kTile))) return ONEBIT_E_SIZE;
    drop_stale_error();
    return hip_status(launch_materialize(ef, scales, e_out, N, rows, n, stream));
}

int lamb_layer_scale(float* buf, int64_t N, int32_t batch, const int64_t* seg_off,
                     const float* seg_k, int32_t n_seg, int32_t divide, hipStream_t stream) {
    if (N < 0 || (N % 4) || batch < 1) return ONEBIT_E_SIZE;
    if (!buf || !seg_off || !seg_k) return ONEBIT_E_NULL;
    if (n_seg < 1) return ONEBIT_E_ARG;
    if (!aligned(buf, 16) || !aligned(seg_off, 8) || !aligned(seg_k, 4)) return ONEBIT_E_ALIGN;
    if (N == 0) return ONEBIT_OK;
    if (batch > 65535 || !groups_ok(ceil_div(ceil_div(N, kTile), 8))) return ONEBIT_E_SIZE;
    drop_stale_error();
    return hip_status(launch_layer_scale(buf, N, batch, seg_off, seg_k, n_seg, divide != 0, stream));
}

int frozen_v_step(const onebit_frozen_v_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (!a) return ONEBIT_E_NULL;
    if (a->N < 0 || (a->N % 4)) return ONEBIT_E_SIZE;
    if (!groups_ok(ceil_div(a->N, (int64_t)kMaxIters * kTile)) || !groups_ok(lamb_workgroups(a->N)))
        return ONEBIT_E_SIZE;
    const bool packed_m = a->mode == 2 || a->mode == 3;  // momentum given as sign words
    if (!a->x || (!a->m && !packed_m) || !a->v) return ONEBIT_E_NULL;
    if (!aligned(a->x, 16) || !aligned(a->m, 16) || !aligned(a->v, 16)) return ONEBIT_E_ALIGN;
    if (a->mode == 0) {
        if (a->N == 0) return ONEBIT_OK;
        drop_stale_error();
        return hip_status(launch_adam(a->x, a->m, a->v, a->N, a->lr, a->eps, stream));
    }
    if (a->mode == 2) {
        if (!a->m_bits || !a->m_scales) return ONEBIT_E_NULL;
        if (a->m_chunks < 1 || a->m_chunks > kMaxWorkers || (a->N % (64 * (int64_t)a->m_chunks)))
            return ONEBIT_E_SIZE;
        if (!aligned(a->m_bits, 4) || !aligned(a->m_scales, 4) || !aligned(a->m_out, 16))
            return ONEBIT_E_ALIGN;
        if (a->N == 0) return ONEBIT_OK;
        drop_stale_error();
        return hip_status(launch_adam_packed(a->x, a->m_bits, a->m_scales, a->v, a->m_out, a->N,
                                             a->m_chunks, a->lr, a->eps, stream));
    }
    if (a->mode != 1 && a->mode != 3) return ONEBIT_E_ARG;
    // mode 3 may take the previous momentum packed instead of m_prev
    const bool prev_packed = a->mode == 3 && a->mp_bits != nullptr;
    if ((!a->m_prev && !prev_packed) || !a->v_fresh || !a->seg_off || !a->c_avg || !a->r_prev ||
        !a->c_prev)
        return ONEBIT_E_NULL;
    if (a->mode == 3) {
        if (!a->m_bits || !a->m_scales || !a->m_seg_k || (a->use_c_t && !a->m_out))
            return ONEBIT_E_NULL;
        if ((a->mp_bits == nullptr) != (a->mp_scales == nullptr)) return ONEBIT_E_NULL;
        if (a->m_chunks < 1 || a->m_chunks > kMaxWorkers || (a->N % (64 * (int64_t)a->m_chunks)))
            return ONEBIT_E_SIZE;
        if (!aligned(a->m_bits, 4) || !aligned(a->m_scales, 4) || !aligned(a->m_seg_k, 4) ||
            !aligned(a->m_out, 16) || !aligned(a->mp_bits, 4) || !aligned(a->mp_scales, 4))
            return ONEBIT_E_ALIGN;
        if (a->m_out && !prev_packed) {  // m_out must not overlap m_prev, which is read
            const uintptr_t o = (uintptr_t)a->m_out, p = (uintptr_t)a->m_prev;
            const uintptr_t bytes = (uintptr_t)a->N * sizeof(float);
            if (o < p + bytes && p < o + bytes) return ONEBIT_E_ARG;
        }
    }
    if (a->n_seg < 1) return ONEBIT_E_ARG;
    if (!groups_ok(a->n_seg)) return ONEBIT_E_SIZE;
    if (!aligned(a->m_prev, 16) || !aligned(a->v_fresh, 16) || !aligned(a->seg_off, 8) ||
        !aligned(a->c_avg, 4) || !aligned(a->r_prev, 4) || !aligned(a->c_prev, 4) ||
        (a->ratio_max && !aligned(a->ratio_max, 4)) || (a->err_ratio && !aligned(a->err_ratio, 4)))
        return ONEBIT_E_ALIGN;
    if (a->N == 0) return ONEBIT_OK;
    const size_t need = lamb_ws_bytes(a->N, a->n_seg);
    if (!ws || ws_bytes < need) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    uint32_t* keys = static_cast<uint32_t*>(ws);
    uint32_t* wg_max = keys + round_up((size_t)a->n_seg * sizeof(uint32_t)) / sizeof(uint32_t);
    drop_stale_error();
    return hip_status(launch_lamb(*a, keys, wg_max, stream));
}

int int8_quantize(const float* g, float* err, int8_t* codes, float* block_scales, float* deq,
                  int64_t N, int32_t block, int32_t rounding, uint64_t seed, uint32_t step,
                  void* ws, size_t ws_bytes, hipStream_t stream) {
    if (block != 0 && block != 64 && block != 128 && block != 256 && block != 512 && block != 1024)
        return ONEBIT_E_SIZE;
    if (N < 0 || (N % 4) || (block && (N % block))) return ONEBIT_E_SIZE;
    if (!groups_ok(ceil_div(N, (int64_t)kInt8Tiles * kTile))) return ONEBIT_E_SIZE;
    if (rounding != 0 && rounding != 1) return ONEBIT_E_ARG;
    if (!g || !codes || !block_scales) return ONEBIT_E_NULL;
    if (!aligned(g, 16) || (err && !aligned(err, 16)) || !aligned(codes, 4) ||
        !aligned(block_scales, 4) || (deq && !aligned(deq, 16)))
        return ONEBIT_E_ALIGN;
    if (N == 0) return ONEBIT_OK;
    if (block == 0) {
        if (!ws || ws_bytes < 256) return ONEBIT_E_WORKSPACE;
        if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    }
    drop_stale_error();
    return hip_status(launch_int8(g, err, codes, block_scales, deq, N, block, seed, step,
                                  rounding == 1, static_cast<uint32_t*>(ws), stream));
}

int int8_sr_quantize(const float* g, float* err, int8_t* codes, float* block_scales, float* deq,
                     int64_t N, int32_t block, uint64_t seed, uint32_t step, hipStream_t stream) {
    if (block == 0) return ONEBIT_E_SIZE;  // the per-tensor variant needs a workspace
    return int8_quantize(g, err, codes, block_scales, deq, N, block, 0, seed, step, nullptr, 0,
                         stream);
}

// ---------------------------------------------------------------- warmup

size_t warmup_workspace_bytes(int64_t N, int32_t n_seg) {
    if (N < 0 || (N % 4) || n_seg < 1) return 0;
    return round_up((size_t)(n_seg + 1) * sizeof(int64_t)) +
           round_up((size_t)layer_grid(N, n_seg) * 2 * sizeof(double)) +
           round_up((size_t)n_seg * sizeof(double)) +
           round_up((size_t)(n_seg + 1) * sizeof(int32_t)) +
           round_up((size_t)n_seg * sizeof(double)) +
           round_up((size_t)layer_grid(N, n_seg) * 2 * kExactLimbs * sizeof(uint64_t));
}

int warmup_adam_step(float* x, float* m, float* v, const float* g, int64_t N, float lr, float eps,
                     float beta1, float beta2, hipStream_t stream) {
    if (N < 0 || (N % 4) || !groups_ok(ceil_div(N, (int64_t)kMaxIters * kTile)))
        return ONEBIT_E_SIZE;
    if (N == 0) return ONEBIT_OK;
    if (!x || !m || !v || !g) return ONEBIT_E_NULL;
    if (!aligned(x, 16) || !aligned(m, 16) || !aligned(v, 16) || !aligned(g, 16))
        return ONEBIT_E_ALIGN;
    drop_stale_error();
    return hip_status(launch_warmup_adam(x, m, v, g, N, lr, eps, beta1, beta2, stream));
}

int warmup_lamb_step(float* x, float* m, float* v, const float* g, int64_t N,
                     const int64_t* seg_off, int32_t n_seg, float lr, float eps, float beta1,
                     float beta2, float beta_c, int32_t first, float* c, float* c_avg, void* ws,
                     size_t ws_bytes, hipStream_t stream) {
    if (N < 0 || (N % 4)) return ONEBIT_E_SIZE;
    if ((N > 0 && (!x || !m || !v || !g)) || !seg_off || !c || !c_avg) return ONEBIT_E_NULL;
    if (n_seg < 1 || (first != 0 && first != 1)) return ONEBIT_E_ARG;
    if (!groups_ok(layer_grid(N, n_seg)) || !groups_ok(n_seg)) return ONEBIT_E_SIZE;
    if (!aligned(x, 16) || !aligned(m, 16) || !aligned(v, 16) || !aligned(g, 16) ||
        !aligned(seg_off, 8) || !aligned(c, 4) || !aligned(c_avg, 4))
        return ONEBIT_E_ALIGN;
    if (!ws || ws_bytes < warmup_workspace_bytes(N, n_seg)) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    WarmupLambArgs a;
    a.x = x;
    a.m = m;
    a.v = v;
    a.g = g;
    a.seg_off = seg_off;
    a.n_seg = n_seg;
    a.N = N;
    a.lr = lr;
    a.eps = eps;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.beta_c = beta_c;
    a.first = first;
    a.c = c;
    a.c_avg = c_avg;
    // N == 0: every layer is empty, c = 1 (the coefficient of a zero norm)
    drop_stale_error();
    return hip_status(launch_warmup_lamb(a, split_warmup_ws(ws, N, n_seg), stream));
}

int lamb_momentum_scale(const float* m, int64_t N, const int64_t* seg_off, int32_t n_seg,
                        float* k, void* ws, size_t ws_bytes, hipStream_t stream) {
    if (N < 0 || (N % 4)) return ONEBIT_E_SIZE;
    if ((N > 0 && !m) || !seg_off || !k) return ONEBIT_E_NULL;
    if (n_seg < 1) return ONEBIT_E_ARG;
    if (!groups_ok(layer_grid(N, n_seg)) || !groups_ok(n_seg)) return ONEBIT_E_SIZE;
    if (!aligned(m, 16) || !aligned(seg_off, 8) || !aligned(k, 4)) return ONEBIT_E_ALIGN;
    if (!ws || ws_bytes < warmup_workspace_bytes(N, n_seg)) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    drop_stale_error();
    return hip_status(
        launch_momentum_scale(m, N, seg_off, n_seg, k, split_warmup_ws(ws, N, n_seg), stream));
}

}  // extern "C"

// ---------------------------------------------------------------- training operators

namespace {

constexpr int64_t kMaxPositions = (int64_t)1 << 29;  // lengths and positions: 32-bit differences
constexpr int64_t kMaxLd = (int64_t)1 << 40;         // strides: more than any memory spans
constexpr int64_t kMaxTokenStride = (int64_t)1 << 23;  // 64 rows: a buffer below 2^31 bytes

// bytes of an element, 0 for an unknown type
size_t type_size(int32_t dtype) {
    return dtype == ONEBIT_F32 ? 4 : dtype == ONEBIT_BF16 || dtype == ONEBIT_F16 ? 2 : 0;
}

// rows of `cols` elements in groups of 8 columns, as the row kernels count
// them: below 2^31
bool row_groups_ok(int64_t rows, int64_t cols) {
    const int64_t per_row = ceil_div(cols, 8);
    return rows <= INT32_MAX && per_row <= INT32_MAX && rows * per_row <= INT32_MAX;
}

// Whether y's rows lie over p's without being them, as far as strides show: of
// one stride, or from one address on.
bool rows_cross(const void* y, int64_t ld_y, const void* p, int64_t ld_p, int64_t rows,
                int64_t cols, size_t size) {
    if (y == p) return ld_y != ld_p && rows > 1;
    if (!p || ld_y != ld_p) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(y), b = reinterpret_cast<uintptr_t>(p);
    const uint64_t apart = a < b ? b - a : a - b;  // bytes
    const uint64_t pitch = (uint64_t)ld_y * size, width = (uint64_t)cols * size;
    const uint64_t down = apart / pitch, right = apart % pitch, last = (uint64_t)rows - 1;
    return (down <= last && right < width) || (down < last && pitch - right < width);
}

int check_lengths(int32_t Tq, int32_t Tk) {
    return Tq < 0 || Tk < 0 || Tq > kMaxPositions || Tk > kMaxPositions ? ONEBIT_E_SIZE : ONEBIT_OK;
}

int check_bias_sizes(int32_t H, int32_t n_buckets, int32_t radius) {
    if (H < 1 || H > 65535) return ONEBIT_E_SIZE;
    if (n_buckets < 1 || n_buckets > kMaxBuckets || radius < 1 || radius > kMaxRadius)
        return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

bool position_ok(int32_t q_pos) { return q_pos >= -kMaxPositions && q_pos <= kMaxPositions; }

// distances' sums of every part of every head
size_t bias_grad_ws_bytes(int64_t parts, int32_t H, int32_t radius) {
    return round_up((size_t)parts * H * (2 * (size_t)radius + 1) * sizeof(float));
}

}  // namespace

extern "C" {

int dropout_apply(const void* x, const void* residual, void* y, int32_t dtype, int64_t rows,
                  int64_t cols, int64_t ld_x, int64_t ld_r, int64_t ld_y, float p, uint64_t seed,
                  uint32_t step, const uint32_t* step_dev, int64_t row0, hipStream_t stream) {
    const size_t size = type_size(dtype);
    if (!size) return ONEBIT_E_ARG;
    if (rows < 0 || cols < 0 || row0 < 0) return ONEBIT_E_SIZE;
    if (!(p >= 0.0f && p < 1.0f)) return ONEBIT_E_ARG;
    if (rows == 0 || cols == 0) return ONEBIT_OK;
    if (!x || !y) return ONEBIT_E_NULL;
    if (!row_groups_ok(rows, cols)) return ONEBIT_E_SIZE;
    if (ld_x < cols || ld_y < cols || (residual && ld_r < cols) || ld_x > kMaxLd || ld_y > kMaxLd ||
        (residual && ld_r > kMaxLd))
        return ONEBIT_E_SIZE;
    if (!aligned(x, size) || !aligned(y, size) || !aligned(residual, size)) return ONEBIT_E_ALIGN;
    if (rows_cross(y, ld_y, x, ld_x, rows, cols, size) ||
        rows_cross(y, ld_y, residual, ld_r, rows, cols, size))
        return ONEBIT_E_ARG;
    if (!aligned(step_dev, 4)) return ONEBIT_E_ALIGN;
    drop_stale_error();
    return hip_status(launch_dropout(x, residual, y, dtype, rows, cols, ld_x, ld_r, ld_y, row0, p,
                                     seed, step, step_dev, stream));
}

int rel_bias_expand(const float* table, const int32_t* map, void* out, int32_t dtype, int32_t H,
                    int32_t n_buckets, int32_t radius, int32_t Tq, int32_t Tk, int32_t q_pos,
                    hipStream_t stream) {
    const size_t size = type_size(dtype);
    if (!size || !position_ok(q_pos)) return ONEBIT_E_ARG;
    int st = check_lengths(Tq, Tk);
    if (st || (st = check_bias_sizes(H, n_buckets, radius))) return st;
    if (Tq == 0 || Tk == 0) return ONEBIT_OK;
    if (!table || !map || !out) return ONEBIT_E_NULL;
    if (!row_groups_ok(Tq, Tk)) return ONEBIT_E_SIZE;
    if (!aligned(table, 4) || !aligned(map, 4) || !aligned(out, size)) return ONEBIT_E_ALIGN;
    drop_stale_error();
    return hip_status(launch_rel_bias(RelBias{table, map, n_buckets, radius, H}, out, dtype, Tq, Tk,
                                      q_pos, stream));
}

size_t rel_bias_workspace_bytes(int32_t B, int32_t H, int32_t Tq, int32_t Tk, int32_t radius) {
    if (B < 0 || check_lengths(Tq, Tk) || check_bias_sizes(H, 1, radius)) return 0;
    if (B == 0 || Tq == 0 || Tk == 0) return 256;
    // of either width of element
    const int64_t wide = bias_grad_plan(B, H, Tq, Tk, ONEBIT_F32).parts();
    const int64_t narrow = bias_grad_plan(B, H, Tq, Tk, ONEBIT_BF16).parts();
    return bias_grad_ws_bytes(wide > narrow ? wide : narrow, H, radius);
}

int rel_bias_grad(const void* ds, int32_t dtype, const int32_t* map, float* dtable, int32_t B,
                  int32_t H, int32_t n_buckets, int32_t radius, int32_t Tq, int32_t Tk,
                  int32_t q_pos, int32_t accumulate, void* ws, size_t ws_bytes,
                  hipStream_t stream) {
    const size_t size = type_size(dtype);
    if (!size || !position_ok(q_pos) || (accumulate != 0 && accumulate != 1)) return ONEBIT_E_ARG;
    int st = B < 0 ? ONEBIT_E_SIZE : check_lengths(Tq, Tk);
    if (st || (st = check_bias_sizes(H, n_buckets, radius))) return st;
    const bool empty = B == 0 || Tq == 0 || Tk == 0;
    if (!map || !dtable || (!ds && !empty)) return ONEBIT_E_NULL;
    if (!aligned(ds, size) || !aligned(map, 4) || !aligned(dtable, 4)) return ONEBIT_E_ALIGN;
    if (!empty && !groups_ok(2 * bias_grad_plan(B, H, Tq, Tk, dtype).parts())) return ONEBIT_E_SIZE;
    if (!ws || ws_bytes < rel_bias_workspace_bytes(B, H, Tq, Tk, radius)) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    drop_stale_error();
    if (empty)  // sums over nothing
        return hip_status(launch_bias_join(static_cast<float*>(ws), map, dtable, H, 0, n_buckets,
                                           radius, accumulate != 0, stream));
    return hip_status(launch_rel_bias_grad(ds, dtype, map, dtable, B, H, n_buckets, radius, Tq, Tk,
                                           q_pos, accumulate != 0, static_cast<float*>(ws),
                                           stream));
}

}  // extern "C"

namespace {

// Strides of a tensor of T tokens of heads * D elements per sequence.  What is
// written must not overlap itself: each dimension steps over all that the ones
// of smaller strides span, as every slice or reordering of a whole tensor does.
int check_heads(const void* p, const int64_t s[3], int32_t B, int32_t T, int32_t heads, int32_t D,
                bool written) {
    if (B == 0 || T == 0) return ONEBIT_OK;
    if (!p) return ONEBIT_E_NULL;
    for (int k = 0; k < 3; ++k)
        if (s[k] < 0 || s[k] > (k == 1 ? kMaxTokenStride : kMaxLd) || s[k] % 8)
            return ONEBIT_E_SIZE;
    int64_t dim[3][2] = {{s[0], B}, {s[1], T}, {s[2], heads}};  // stride, count
    for (int k = 0; k < 3; ++k)
        for (int m = 0; m + 1 < 3; ++m)
            if (dim[m][0] > dim[m + 1][0]) {
                std::swap(dim[m][0], dim[m + 1][0]);
                std::swap(dim[m][1], dim[m + 1][1]);
            }
    int64_t span = D;
    for (int k = 0; k < 3 && written; ++k) {
        if (dim[k][1] == 1) continue;
        if (dim[k][0] < span) return ONEBIT_E_SIZE;
        if (dim[k][0] > (INT64_MAX - span) / dim[k][1]) return ONEBIT_E_SIZE;  // past any memory
        span += dim[k][0] * (dim[k][1] - 1);
    }
    return aligned(p, 16) ? ONEBIT_OK : ONEBIT_E_ALIGN;
}

// An output over a tensor of the call (empty ones are passed as they come).
bool written_over(const void* out, int32_t T, std::initializer_list<const void*> others) {
    for (const void* x : others)
        if (out == x && out && T > 0) return true;
    return false;
}

Strides strides_of(const int64_t s[3]) { return Strides{s[0], s[1], s[2]}; }

int check_attention_sizes(int32_t B, int32_t H, int32_t Hkv, int32_t Tq, int32_t Tk, int32_t D,
                          int32_t radius) {
    const int st = check_lengths(Tq, Tk);
    if (st) return st;
    if (B < 0 || H < 1 || H > 65535 || Hkv < 1 || H % Hkv) return ONEBIT_E_SIZE;
    if (D < 8 || D > 128 || D % 8 || radius < 0 || radius > kMaxRadius) return ONEBIT_E_SIZE;
    const int64_t heads = (int64_t)B * H;  // below 2^47
    // rows of a launch, and query tiles that one key head goes through
    if (heads > INT32_MAX || heads * Tq > (int64_t)INT32_MAX * 16 ||
        (int64_t)(Tq / kStep + 1) * (H / Hkv) > INT32_MAX)
        return ONEBIT_E_SIZE;
    if (!groups_ok((heads + 7) * attn_tiles(Tq) * attn_splits(B, H, Hkv, Tq, Tk).splits) ||
        !groups_ok((heads + 7) * attn_tiles(Tk)) || !groups_ok(heads * Tq))
        return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

// Workspace of the two directions, in the order it is carved.
struct AttnSizes {
    size_t split_o, split_ml;   // forward
    size_t delta, partials;     // backward; delta and norm together
};

AttnSizes attn_sizes(int32_t B, int32_t H, int32_t Hkv, int32_t Tq, int32_t Tk, int32_t D,
                     int32_t radius) {
    AttnSizes z = {};
    const size_t rows = (size_t)B * H * Tq;
    const int32_t splits = attn_splits(B, H, Hkv, Tq, Tk).splits;
    if (splits > 1) {
        z.split_o = round_up(rows * splits * D * sizeof(float));
        z.split_ml = round_up(rows * splits * sizeof(f4));
    }
    z.delta = round_up(2 * rows * sizeof(float));
    if (radius > 0)
        z.partials = round_up((size_t)B * attn_tiles(Tk) * H * (2 * (size_t)radius + 1) *
                              sizeof(float));
    return z;
}

int check_attention(const rel_attention_args* a) {
    if (!a) return ONEBIT_E_NULL;
    if (a->dtype != ONEBIT_BF16 && a->dtype != ONEBIT_F16) return ONEBIT_E_ARG;
    const bool bias = a->radius != 0 || a->n_buckets != 0 || a->table || a->map;
    int st = check_attention_sizes(a->B, a->H, a->Hkv, a->Tq, a->Tk, a->D, a->radius);
    if (st) return st;
    if (bias) {
        if (!a->table || !a->map) return ONEBIT_E_NULL;
        if ((st = check_bias_sizes(a->H, a->n_buckets, a->radius))) return st;
    }
    // the bias divided by the scale, and the scale times log2 e, stay in range
    if (!(a->scale >= 0x1p-64f && a->scale <= 0x1p64f)) return ONEBIT_E_ARG;
    if (!(a->p >= 0.0f && a->p < 1.0f) || !position_ok(a->q_pos) ||
        (a->causal != 0 && a->causal != 1))
        return ONEBIT_E_ARG;
    if (!aligned(a->table, 4) || !aligned(a->map, 4) || !aligned(a->q_pos_of, 4) ||
        !aligned(a->k_len, 4) || !aligned(a->step_dev, 4) || !aligned(a->lse, 4))
        return ONEBIT_E_ALIGN;
    if ((st = check_heads(a->q, a->q_stride, a->B, a->Tq, a->H, a->D, false)) ||
        (st = check_heads(a->k, a->k_stride, a->B, a->Tk, a->Hkv, a->D, false)) ||
        (st = check_heads(a->v, a->v_stride, a->B, a->Tk, a->Hkv, a->D, false)))
        return st;
    return check_heads(a->o, a->o_stride, a->B, a->Tq, a->H, a->D, true);
}

AttnArgs attn_args(const rel_attention_args* a) {
    AttnArgs k = {};
    k.q = a->q;
    k.k = a->k;
    k.v = a->v;
    k.o = a->o;
    k.o_in = a->o;
    k.sq = strides_of(a->q_stride);
    k.sk = strides_of(a->k_stride);
    k.sv = strides_of(a->v_stride);
    k.so = strides_of(a->o_stride);
    k.lse = a->lse;
    k.q_pos_dev = a->q_pos_of;
    k.k_len = a->k_len;
    k.bias = RelBias{a->table, a->map, a->n_buckets, a->radius, a->H};
    k.drop = drop_args(a->p, a->seed, a->step, a->step_dev);
    k.B = a->B;
    k.H = a->H;
    k.Hkv = a->Hkv;
    k.Tq = a->Tq;
    k.Tk = a->Tk;
    k.D = a->D;
    k.q_pos = a->q_pos;
    k.causal = a->causal;
    k.splits = 1;
    k.scale = a->scale;
    return k;
}

}  // namespace

extern "C" {

size_t rel_attention_workspace_bytes(int32_t B, int32_t H, int32_t Hkv, int32_t Tq, int32_t Tk,
                                     int32_t D, int32_t radius, int32_t backward) {
    if (check_attention_sizes(B, H, Hkv, Tq, Tk, D, radius)) return 0;
    const AttnSizes z = attn_sizes(B, H, Hkv, Tq, Tk, D, radius);
    const size_t fwd = z.split_o + z.split_ml;
    const size_t bwd = z.delta + z.partials;
    const size_t need = backward && bwd > fwd ? bwd : fwd;
    return need ? need : 256;
}

int rel_attention_forward(const rel_attention_args* a, void* ws, size_t ws_bytes,
                          hipStream_t stream) {
    const int st = check_attention(a);
    if (st) return st;
    if (a->B == 0 || a->Tq == 0) return ONEBIT_OK;
    AttnArgs k = attn_args(a);
    const AttnSplits plan = attn_splits(a->B, a->H, a->Hkv, a->Tq, a->Tk);
    k.few = plan.few;
    k.splits = plan.splits;
    if (k.splits > 1) {
        const AttnSizes z = attn_sizes(a->B, a->H, a->Hkv, a->Tq, a->Tk, a->D, a->radius);
        if (!ws || ws_bytes < z.split_o + z.split_ml) return ONEBIT_E_WORKSPACE;
        if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
        const int32_t tiles = (a->Tk + kStep - 1) / kStep;
        k.split_tiles = (tiles + k.splits - 1) / k.splits;
        k.split_o = static_cast<float*>(ws);
        k.split_ml = reinterpret_cast<f4*>(static_cast<char*>(ws) + z.split_o);
    }
    if (written_over(a->o, a->Tq, {a->q, a->k, a->v})) return ONEBIT_E_ARG;
    drop_stale_error();
    return hip_status(launch_attn_forward(k, a->dtype, stream));
}

int rel_attention_backward(const rel_attention_args* a, void* ws, size_t ws_bytes,
                           hipStream_t stream) {
    int st = check_attention(a);
    if (st) return st;
    if ((st = check_heads(a->d_o, a->do_stride, a->B, a->Tq, a->H, a->D, false)) ||
        (st = check_heads(a->dq, a->dq_stride, a->B, a->Tq, a->H, a->D, true)) ||
        (st = check_heads(a->dk, a->dk_stride, a->B, a->Tk, a->Hkv, a->D, true)) ||
        (st = check_heads(a->dv, a->dv_stride, a->B, a->Tk, a->Hkv, a->D, true)))
        return st;
    if (!a->lse && a->B > 0 && a->Tq > 0) return ONEBIT_E_NULL;
    if ((a->dtable && !a->table) || (a->accumulate != 0 && a->accumulate != 1))
        return ONEBIT_E_ARG;
    if (!aligned(a->dtable, 4)) return ONEBIT_E_ALIGN;
    const AttnSizes z =
        attn_sizes(a->B, a->H, a->Hkv, a->Tq, a->Tk, a->D, a->dtable ? a->radius : 0);
    if (!ws || ws_bytes < z.delta + z.partials) return ONEBIT_E_WORKSPACE;
    if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    if (a->B > 0 && (written_over(a->dq, a->Tq, {a->q, a->k, a->v, a->o, a->d_o}) ||
                     written_over(a->dk, a->Tk, {a->q, a->k, a->v, a->o, a->d_o, a->dq}) ||
                     written_over(a->dv, a->Tk, {a->q, a->k, a->v, a->o, a->d_o, a->dq, a->dk})))
        return ONEBIT_E_ARG;
    AttnArgs k = attn_args(a);
    k.d_o = a->d_o;
    k.dq = a->dq;
    k.dk = a->dk;
    k.dv = a->dv;
    k.sdo = strides_of(a->do_stride);
    k.sdq = strides_of(a->dq_stride);
    k.sdk = strides_of(a->dk_stride);
    k.sdv = strides_of(a->dv_stride);
    k.delta = static_cast<float*>(ws);
    k.norm = k.delta + (size_t)a->B * a->H * a->Tq;
    k.partials = reinterpret_cast<float*>(static_cast<char*>(ws) + z.delta);
    drop_stale_error();
    return hip_status(launch_attn_backward(k, a->dtype, a->dtable, a->accumulate != 0, stream));
}

}  // extern "C"

// ---------------------------------------------------------------- layer norm

namespace {

constexpr int64_t kMaxNormCols = (int64_t)1 << 29;
constexpr int64_t kMaxRows = (int64_t)1 << 40;

int check_norm(int32_t dtype, int32_t w_dtype, int64_t rows, int64_t cols) {
    if (!type_size(dtype) || (w_dtype != dtype && w_dtype != ONEBIT_F32)) return ONEBIT_E_ARG;
    if (rows < 0 || rows > kMaxRows || cols < 0 || cols > kMaxNormCols) return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

bool ld_ok(int64_t ld, int64_t cols) { return ld >= cols && ld <= kMaxLd; }

struct Matrix {
    const void* p;
    int64_t ld, rows, cols;
    size_t size;
};

// An output's rows over another matrix's, as far as strides show: from one address
// on, of one stride in bytes, or starting inside a matrix without gaps.
bool lies_over(const Matrix& out, const Matrix& in) {
    if (!out.p || !in.p || out.rows == 0 || out.cols == 0 || in.rows == 0 || in.cols == 0)
        return false;
    const bool after = (uintptr_t)out.p > (uintptr_t)in.p;
    const Matrix& first = after ? in : out;
    const Matrix& second = after ? out : in;
    const uint64_t apart = (uintptr_t)second.p - (uintptr_t)first.p;
    if (apart == 0) return true;
    const uint64_t width = (uint64_t)first.cols * first.size;
    const uint64_t pitch = (uint64_t)first.ld * first.size;
    if (first.rows == 1 || first.ld == first.cols) return apart < width * (uint64_t)first.rows;
    if (pitch != (uint64_t)second.ld * second.size && second.rows > 1) return false;
    const uint64_t down = apart / pitch, right = apart % pitch;
    return (down < (uint64_t)first.rows && right < width) ||
           (down + 1 < (uint64_t)first.rows && pitch - right < (uint64_t)second.cols * second.size);
}

}  // namespace

extern "C" {

int layer_norm_forward(const void* x, void* y, int32_t dtype, int64_t rows, int64_t cols,
                       int64_t ld_x, int64_t ld_y, const void* weight, const void* bias,
                       int32_t w_dtype, float eps, float* mean, float* rstd, hipStream_t stream) {
    const int st = check_norm(dtype, w_dtype, rows, cols);
    if (st) return st;
    if (!(eps >= 0.0f && eps < INFINITY)) return ONEBIT_E_ARG;
    if (rows == 0 || cols == 0) return ONEBIT_OK;
    if (!x || !y) return ONEBIT_E_NULL;
    if (!ld_ok(ld_x, cols) || !ld_ok(ld_y, cols)) return ONEBIT_E_SIZE;
    const size_t size = type_size(dtype), w_size = type_size(w_dtype);
    if (!aligned(x, size) || !aligned(y, size) || !aligned(weight, w_size) ||
        !aligned(bias, w_size) || !aligned(mean, 4) || !aligned(rstd, 4))
        return ONEBIT_E_ALIGN;
    const Matrix xs{x, ld_x, rows, cols, size}, ys{y, ld_y, rows, cols, size},
        w{weight, cols, 1, cols, w_size}, b{bias, cols, 1, cols, w_size},
        means{mean, rows, 1, rows, 4}, rstds{rstd, rows, 1, rows, 4};
    if (lies_over(ys, xs) && !(y == x && (ld_y == ld_x || rows == 1))) return ONEBIT_E_ARG;
    for (const Matrix& in : {w, b})
        if (lies_over(ys, in)) return ONEBIT_E_ARG;
    for (const Matrix& out : {means, rstds})
        for (const Matrix& other : {xs, ys, w, b})
            if (lies_over(out, other)) return ONEBIT_E_ARG;
    if (lies_over(means, rstds)) return ONEBIT_E_ARG;
    NormArgs a = {};
    a.x = x;
    a.y = y;
    a.weight = weight;
    a.bias = bias;
    a.mean = mean;
    a.rstd = rstd;
    a.rows = rows;
    a.cols = cols;
    a.ld_x = ld_x;
    a.ld_y = ld_y;
    a.eps = eps;
    a.dtype = dtype;
    a.w_wide = w_dtype == ONEBIT_F32;
    drop_stale_error();
    return hip_status(launch_layer_norm(a, stream));
}

size_t layer_norm_workspace_bytes(int64_t rows, int64_t cols) {
    if (check_norm(ONEBIT_F32, ONEBIT_F32, rows, cols)) return 0;
    const size_t need = round_up((size_t)norm_parts(rows, cols) * 2 * cols * sizeof(float));
    return need ? need : 256;
}

int layer_norm_backward(const void* dy, const void* x, const float* mean, const float* rstd,
                        void* dx, int32_t dtype, int64_t rows, int64_t cols, int64_t ld_dy,
                        int64_t ld_x, int64_t ld_dx, const void* weight, int32_t w_dtype,
                        float* dweight, float* dbias, int32_t accumulate, void* ws,
                        size_t ws_bytes, hipStream_t stream) {
    const int st = check_norm(dtype, w_dtype, rows, cols);
    if (st) return st;
    if (accumulate != 0 && accumulate != 1) return ONEBIT_E_ARG;
    if (cols == 0) return ONEBIT_OK;
    const bool sums = dweight || dbias;
    const size_t size = type_size(dtype);
    if (rows > 0) {
        if (!dy || !x || !mean || !rstd) return ONEBIT_E_NULL;
        if (!ld_ok(ld_dy, cols) || !ld_ok(ld_x, cols) || (dx && !ld_ok(ld_dx, cols)))
            return ONEBIT_E_SIZE;
    }
    if (!aligned(dy, size) || !aligned(x, size) || !aligned(dx, size) ||
        !aligned(weight, type_size(w_dtype)) || !aligned(mean, 4) || !aligned(rstd, 4) ||
        !aligned(dweight, 4) || !aligned(dbias, 4))
        return ONEBIT_E_ALIGN;
    const size_t w_size = type_size(w_dtype);
    const Matrix dys{dy, ld_dy, rows, cols, size}, xs{x, ld_x, rows, cols, size},
        dxs{dx, ld_dx, rows, cols, size}, w{weight, cols, 1, cols, w_size},
        means{mean, rows, 1, rows, 4}, rstds{rstd, rows, 1, rows, 4},
        dws{dweight, cols, 1, cols, 4}, dbs{dbias, cols, 1, cols, 4};
    for (const Matrix& in : {dys, xs})
        if (lies_over(dxs, in) && !(dx == in.p && (ld_dx == in.ld || rows == 1)))
            return ONEBIT_E_ARG;
    for (const Matrix& in : {w, means, rstds})
        if (lies_over(dxs, in)) return ONEBIT_E_ARG;
    for (const Matrix& out : {dws, dbs})
        for (const Matrix& other : {dys, xs, dxs, w, means, rstds})
            if (lies_over(out, other)) return ONEBIT_E_ARG;
    if (lies_over(dws, dbs)) return ONEBIT_E_ARG;
    if (sums) {
        if (!ws || ws_bytes < layer_norm_workspace_bytes(rows, cols)) return ONEBIT_E_WORKSPACE;
        if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    }
    if (!sums && (rows == 0 || !dx)) return ONEBIT_OK;
    NormArgs a = {};
    a.x = x;
    a.dy = dy;
    a.dx = dx;
    a.weight = weight;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.partials = sums ? static_cast<float*>(ws) : nullptr;
    a.rows = rows;
    a.cols = cols;
    a.ld_x = ld_x;
    a.ld_dy = ld_dy;
    a.ld_dx = ld_dx;
    a.dtype = dtype;
    a.w_wide = w_dtype == ONEBIT_F32;
    drop_stale_error();
    return hip_status(launch_layer_norm_grad(a, dweight, dbias, accumulate != 0, stream));
}

}  // extern "C"

// ---------------------------------------------------------------- linear layer

namespace {

int check_linear_sizes(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 0 || K < 0 || M > INT32_MAX || N > kMaxFeatures || K > kMaxFeatures)
        return ONEBIT_E_SIZE;
    // tiles of a launch (their threads counted in 32 bits), also of dw [N][K]
    const int64_t rows = M > N ? M : N, cols = N > K ? N : K;
    if (ceil_div(rows, 128) * ceil_div(cols, 128) > ((int64_t)1 << 22)) return ONEBIT_E_SIZE;
    return ONEBIT_OK;
}

// Workspace in the order it is carved: operands laid out anew, dz's parts, the partial
// sums of dbias, the parts of a divided product.
struct LinearSizes {
    size_t x, w, dz, sums, parts;
    size_t all() const { return x + w + dz + sums + parts; }
};

LinearSizes linear_sizes(int64_t M, int64_t N, int64_t K, bool backward) {
    LinearSizes z = {};
    z.x = round_up((size_t)M * padded(K) * 2);
    z.w = round_up((size_t)N * padded(K) * 2);
    if (!backward) {
        if (product_few(M)) return LinearSizes{};
        z.parts = round_up(product_plan(M, N, K, true, true).bytes);
        return z;
    }
    z.dz = round_up((size_t)M * padded(N) * 2 * 2);
    z.sums = round_up((size_t)slope_parts(M, N) * N * sizeof(float));
    for (const bool two : {false, true}) {
        const size_t dx = product_plan(M, K, product_depth(N, two), false, true).bytes,
                     dw = product_plan(N, K, product_depth(M, two), false, false).bytes;
        z.parts = std::max(z.parts, round_up(std::max(dx, dw)));
    }
    return z;
}

int check_linear(const linear_args* a) {
    if (!a) return ONEBIT_E_NULL;
    if (a->dtype != ONEBIT_BF16 && a->dtype != ONEBIT_F16) return ONEBIT_E_ARG;
    if (a->activation < ONEBIT_NONE || a->activation > ONEBIT_SILU) return ONEBIT_E_ARG;
    return check_linear_sizes(a->M, a->N, a->K);
}

// A matrix argument: NULL where nothing is read or written of it.
int check_matrix(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t size) {
    if (rows == 0 || cols == 0) return ONEBIT_OK;
    if (!p) return ONEBIT_E_NULL;
    if (!ld_ok(ld, cols)) return ONEBIT_E_SIZE;
    return aligned(p, size) ? ONEBIT_OK : ONEBIT_E_ALIGN;
}

}  // namespace

extern "C" {

size_t linear_workspace_bytes(int64_t M, int64_t N, int64_t K, int32_t backward) {
    if (check_linear_sizes(M, N, K)) return 0;
    const size_t need = linear_sizes(M, N, K, backward != 0).all();
    return need ? need : 256;
}

int linear_forward(const linear_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
    int st = check_linear(a);
    if (st) return st;
    const int64_t M = a->M, N = a->N, K = a->K;
    if (M == 0 || N == 0) return ONEBIT_OK;
    if (a->bias && a->bias_dtype != ONEBIT_F32 && a->bias_dtype != a->dtype) return ONEBIT_E_ARG;
    if ((st = check_matrix(a->x, a->ld_x, M, K, 2)) || (st = check_matrix(a->w, a->ld_w, N, K, 2)) ||
        (st = check_matrix(a->y, a->ld_y, M, N, 2)) ||
        (a->pre && (st = check_matrix(a->pre, a->ld_pre, M, N, 2))) ||
        (a->residual && (st = check_matrix(a->residual, a->ld_residual, M, N, 2))))
        return st;
    if (a->bias && !aligned(a->bias, type_size(a->bias_dtype))) return ONEBIT_E_ALIGN;
    const Matrix x{a->x, a->ld_x, M, K, 2}, w{a->w, a->ld_w, N, K, 2}, y{a->y, a->ld_y, M, N, 2},
        pre{a->pre, a->ld_pre, M, N, 2}, r{a->residual, a->ld_residual, M, N, 2},
        b{a->bias, N, 1, N, a->bias ? type_size(a->bias_dtype) : 2};
    const bool in_place = a->residual && a->y == a->residual && a->ld_y == a->ld_residual;
    for (const Matrix& in : {x, w, b})
        if (lies_over(y, in) || lies_over(pre, in)) return ONEBIT_E_ARG;
    if (lies_over(y, pre) || lies_over(pre, r) || (!in_place && lies_over(y, r)))
        return ONEBIT_E_ARG;
    const LinearSizes z = linear_sizes(M, N, K, false);
    if (z.all()) {
        if (!ws || ws_bytes < z.all()) return ONEBIT_E_WORKSPACE;
        if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    }
    char* room = static_cast<char*>(ws);
    drop_stale_error();
    ProductOut o = {};
    o.out = a->y;
    o.bias = a->bias;
    o.residual = a->residual;
    o.pre = a->pre;
    o.rows = M;
    o.cols = N;
    o.ld = a->ld_y;
    o.ld_r = a->ld_residual;
    o.ld_pre = a->ld_pre;
    o.type = a->dtype;
    o.act = a->activation;
    o.bias_wide = a->bias_dtype == ONEBIT_F32;
    if (product_few(M))
        return hip_status(launch_product_few(a->dtype, ProductIn{a->w, a->ld_w, K, 0},
                                             ProductIn{a->x, a->ld_x, K, 0}, K, o, stream));
    const bool takes_any = product_any(product_plan(M, N, K, true, true));
    PadRows x_anew, w_anew;
    bool any = false;
    const ProductIn xs = operand(a->x, a->ld_x, M, K, room, takes_any, x_anew, any);
    const ProductIn wi = operand(a->w, a->ld_w, N, K, room + z.x, takes_any, w_anew, any);
    if (launch_pad_rows(x_anew, w_anew, stream) != hipSuccess) return ONEBIT_E_HIP;
    return hip_status(launch_product(a->dtype, wi, true, xs, true, K, o, any,
                                     reinterpret_cast<float*>(room + z.x + z.w), stream));
}

int linear_backward(const linear_args* a, void* ws, size_t ws_bytes, hipStream_t stream) {
    int st = check_linear(a);
    if (st) return st;
    const int64_t M = a->M, N = a->N, K = a->K;
    if (a->accumulate != 0 && a->accumulate != 1) return ONEBIT_E_ARG;
    if (a->round_dz != 0 && a->round_dz != 1) return ONEBIT_E_ARG;
    if (a->dw && a->dw_dtype != ONEBIT_F32 && a->dw_dtype != a->dtype) return ONEBIT_E_ARG;
    const size_t dw_size = a->dw ? type_size(a->dw_dtype) : 2;
    const bool act = a->activation != ONEBIT_NONE;
    if ((st = check_matrix(a->dy, a->ld_dy, M, N, 2)) ||
        (act && (st = check_matrix(a->pre, a->ld_pre, M, N, 2))) ||
        (a->dw && ((st = check_matrix(a->x, a->ld_x, M, K, 2)) ||
                   (st = check_matrix(a->dw, a->ld_dw, N, K, dw_size)))) ||
        (a->dx && ((st = check_matrix(a->w, a->ld_w, N, K, 2)) ||
                   (st = check_matrix(a->dx, a->ld_dx, M, K, 2)))))
        return st;
    if (!aligned(a->dbias, 4)) return ONEBIT_E_ALIGN;
    // what is not read may be anything, its ld too
    const Matrix dy{a->dy, a->ld_dy, M, N, 2}, pre{act ? a->pre : nullptr, a->ld_pre, M, N, 2},
        x{a->dw ? a->x : nullptr, a->ld_x, M, K, 2}, w{a->dx ? a->w : nullptr, a->ld_w, N, K, 2}, dx{a->dx, a->ld_dx, M, K, 2},
        dw{a->dw, a->ld_dw, N, K, dw_size}, db{a->dbias, N, 1, N, 4};
    for (const Matrix& in : {dy, pre, x, w})
        if (lies_over(dx, in) || lies_over(dw, in) || lies_over(db, in)) return ONEBIT_E_ARG;
    if (lies_over(dx, dw) || lies_over(dx, db) || lies_over(dw, db)) return ONEBIT_E_ARG;
    const LinearSizes z = linear_sizes(M, N, K, true);
    if (z.all()) {
        if (!ws || ws_bytes < z.all()) return ONEBIT_E_WORKSPACE;
        if (!aligned(ws, 256)) return ONEBIT_E_ALIGN;
    }
    char* x_room = static_cast<char*>(ws);
    char* w_room = x_room + z.x;
    char* dz_room = w_room + z.w;
    float* sums = reinterpret_cast<float*>(dz_room + z.dz);
    float* parts = reinterpret_cast<float*>(dz_room + z.dz + z.sums);
    drop_stale_error();
    hipError_t e = hipSuccess;
    const bool want_dx = a->dx && M > 0 && K > 0, want_dw = a->dw && N > 0 && K > 0;
    const bool two = !a->round_dz && !slope_exact(a->activation);
    const GradIn g = grad_operands(GradShape{
        a->dy, a->x, a->w, M, N, K, a->ld_dy, a->ld_x, a->ld_w, act, two, want_dx, want_dw,
        product_any(product_plan(M, K, product_depth(N, two), false, true)),
        product_any(product_plan(N, K, product_depth(M, two), false, false)), x_room, w_room,
        dz_room});
    if (N > 0) {
        if (M > 0 && (g.dz_anew || a->dbias)) {
            SlopeArgs s = {};
            s.dy = a->dy;
            s.pre = a->pre;
            s.dz = g.dz_anew ? dz_room : nullptr;
            s.partials = a->dbias ? sums : nullptr;
            s.rows = M;
            s.cols = N;
            s.ld_dy = a->ld_dy;
            s.ld_pre = a->ld_pre;
            s.padded = padded(N);
            s.rest = g.dz.rest;
            s.act = a->activation;
            s.dtype = a->dtype;
            e = launch_slope(s, stream);
        }
        if (e == hipSuccess && a->dbias)
            e = launch_column_join(sums, M > 0 ? slope_parts(M, N) : 0, N, N, a->dbias, nullptr,
                                   a->accumulate != 0, stream);
    }
    if (e == hipSuccess) e = launch_pad_rows(g.x_anew, g.w_anew, stream);
    if (e == hipSuccess && want_dx) {
        ProductOut o = {};
        o.out = a->dx;
        o.rows = M;
        o.cols = K;
        o.ld = a->ld_dx;
        o.type = a->dtype;
        e = launch_product(a->dtype, g.w, false, g.dz, true, N, o, g.dx_any, parts, stream);
    }
    if (e == hipSuccess && want_dw) {
        ProductOut o = {};
        o.out = a->dw;
        o.rows = N;
        o.cols = K;
        o.ld = a->ld_dw;
        o.type = a->dw_dtype;
        o.accumulate = a->accumulate != 0;
        e = launch_product(a->dtype, g.x, false, g.dz, false, M, o, g.dw_any, parts, stream);
    }
    return hip_status(e);
}

}  // extern "C"

// ---------------------------------------------------------------- AdamW

namespace {

constexpr int64_t kMaxTensor = (int64_t)1 << 34;

size_t plan_tensors_bytes(int32_t n_tensors) {
    return round_up((size_t)n_tensors * sizeof(AdamWTensor));
}

struct Range {
    uintptr_t begin, end;
    bool written;
};

void add_range(std::vector<Range>& all, const void* p, int64_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    if (bytes > 0) all.push_back(Range{at, at + (uintptr_t)bytes, written});
}

// Whether something written lies over another range.
bool overlapping(std::vector<Range>& all) {
    std::sort(all.begin(), all.end(),
              [](const Range& a, const Range& b) { return a.begin < b.begin; });
    uintptr_t end = 0, written_end = 0;  // of the ranges before
    for (const Range& r : all) {
        if (r.begin < written_end || (r.written && r.begin < end)) return true;
        if (r.end > end) end = r.end;
        if (r.written && r.end > written_end) written_end = r.end;
    }
    return false;
}

int check_adamw_types(int32_t state_bits, int32_t g_dtype, int32_t copy_dtype) {
    return (state_bits != 8 && state_bits != 32) || !type_size(g_dtype) || !type_size(copy_dtype)
               ? ONEBIT_E_ARG
               : ONEBIT_OK;
}

}  // namespace

extern "C" {

size_t adamw_plan_bytes(const adamw_tensor* tensors, int32_t n_tensors, int64_t* tiles) {
    if (n_tensors < 0 || (n_tensors > 0 && !tensors)) return 0;
    int64_t all = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        if (tensors[i].n < 0 || tensors[i].n > kMaxTensor) return 0;
        all += ceil_div(tensors[i].n, kAdamWTile);
        if (!groups_ok(all)) return 0;
    }
    if (tiles) *tiles = all;
    const size_t need = plan_tensors_bytes(n_tensors) + (size_t)all * sizeof(int32_t);
    return need ? round_up(need) : 256;
}

int adamw_plan(const adamw_tensor* tensors, int32_t n_tensors, int32_t state_bits,
               int32_t g_dtype, int32_t copy_dtype, void* plan, size_t plan_bytes) {
    if (check_adamw_types(state_bits, g_dtype, copy_dtype)) return ONEBIT_E_ARG;
    if (n_tensors < 0) return ONEBIT_E_SIZE;
    if ((n_tensors > 0 && !tensors) || !plan) return ONEBIT_E_NULL;
    const size_t need = adamw_plan_bytes(tensors, n_tensors, nullptr);
    if (!need) return ONEBIT_E_SIZE;
    if (plan_bytes < need) return ONEBIT_E_WORKSPACE;
    if (!aligned(plan, 8)) return ONEBIT_E_ALIGN;
    const bool eight = state_bits == 8;
    const size_t g_size = type_size(g_dtype), c_size = type_size(copy_dtype);
    for (int32_t i = 0; i < n_tensors; ++i) {
        const adamw_tensor& t = tensors[i];
        if (!isfinite(t.lr_scale) || !isfinite(t.weight_decay)) return ONEBIT_E_ARG;
        if (t.n == 0) continue;
        if (!t.x || !t.g || !t.m || !t.v || (c_size == 2 && !t.copy) ||
            (eight && (!t.m_scale || !t.v_scale)))
            return ONEBIT_E_NULL;
        if (!aligned(t.x, 4) || !aligned(t.g, g_size) || (c_size == 2 && !aligned(t.copy, 2)) ||
            (!eight && (!aligned(t.m, 4) || !aligned(t.v, 4))) ||
            (eight && (!aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))))
            return ONEBIT_E_ALIGN;
    }
    try {
        std::vector<Range> all;
        all.reserve((size_t)n_tensors * 7);
        for (int32_t i = 0; i < n_tensors; ++i) {
            const adamw_tensor& t = tensors[i];
            const int64_t blocks = ceil_div(t.n, kStateBlock);
            add_range(all, t.x, 4 * t.n, true);
            add_range(all, t.g, (int64_t)g_size * t.n, false);
            if (c_size == 2) add_range(all, t.copy, 2 * t.n, true);
            add_range(all, t.m, (eight ? 1 : 4) * t.n, true);
            add_range(all, t.v, (eight ? 1 : 4) * t.n, true);
            if (eight) {
                add_range(all, t.m_scale, 4 * blocks, true);
                add_range(all, t.v_scale, 4 * blocks, true);
            }
        }
        if (overlapping(all)) return ONEBIT_E_ARG;
    } catch (const std::bad_alloc&) {
        return ONEBIT_E_WORKSPACE;
    }
    AdamWTensor* to = static_cast<AdamWTensor*>(plan);
    int32_t* tensor_of =
        reinterpret_cast<int32_t*>(static_cast<char*>(plan) + plan_tensors_bytes(n_tensors));
    int64_t tile = 0;
    for (int32_t i = 0; i < n_tensors; ++i) {
        const adamw_tensor& t = tensors[i];
        to[i] = AdamWTensor{t.x,       t.g,       t.copy, t.m,  t.v,        t.m_scale,
                            t.v_scale, t.n,       tile,   t.lr_scale, t.weight_decay};
        for (int64_t k = ceil_div(t.n, kAdamWTile); k > 0; --k) tensor_of[tile++] = i;
    }
    return ONEBIT_OK;
}

int adamw_step(const void* plan, int32_t n_tensors, int64_t tiles, int32_t state_bits,
               int32_t g_dtype, int32_t copy_dtype, float lr, float beta1, float beta2, float eps,
               uint32_t step, uint64_t seed, const float* g_scale, hipStream_t stream) {
    if (check_adamw_types(state_bits, g_dtype, copy_dtype) || step < 1) return ONEBIT_E_ARG;
    if (!(beta1 >= 0.0f && beta1 < 1.0f) || !(beta2 >= 0.0f && beta2 < 1.0f) ||
        !(eps >= 0.0f && eps < INFINITY) || !isfinite(lr))
        return ONEBIT_E_ARG;
    if (n_tensors < 0 || !groups_ok(tiles)) return ONEBIT_E_SIZE;
    if (tiles == 0) return ONEBIT_OK;
    if (n_tensors == 0) return ONEBIT_E_SIZE;
    if (!plan) return ONEBIT_E_NULL;
    if (!aligned(plan, 256) || !aligned(g_scale, 4)) return ONEBIT_E_ALIGN;
    AdamWArgs a = {};
    a.tensors = static_cast<const AdamWTensor*>(plan);
    a.tensor_of = reinterpret_cast<const int32_t*>(static_cast<const char*>(plan) +
                                                   plan_tensors_bytes(n_tensors));
    a.tiles = tiles;
    a.g_scale = g_scale;
    a.lr = lr;
    a.beta1 = beta1;
    a.beta2 = beta2;
    a.eps = eps;
    a.rate = (float)(1.0 / (1.0 - pow((double)beta1, (double)step)));
    a.root = (float)(1.0 / sqrt(1.0 - pow((double)beta2, (double)step)));
    a.k0 = (uint32_t)seed;
    a.k1 = (uint32_t)(seed >> 32);
    a.step = step;
    drop_stale_error();
    return hip_status(launch_adamw(a, state_bits, g_dtype, copy_dtype, stream));
}

}  // extern "C"
