// C ABI of libonebit: host-side validation, workspace carving, launches.
// Every check runs before the first HIP call, so invalid calls touch nothing.
#include <math.h>

#include <initializer_list>
#include <mutex>
#include <utility>

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
