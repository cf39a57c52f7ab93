// C ABI of the operators beside the convolution: argument checks and dispatch.
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include "../../include/wino.h"
#include "common.cuh"
#include "ops.h"
#include "sm100.cuh"

namespace {

using namespace wino;

thread_local int t_last_cuda = 0;   // last CUDA error of this thread's plan-less calls

int status(cudaError_t e) {
    if (e == cudaSuccess) return WINO_OK;
    t_last_cuda = (int)e;
    return WINO_ERR_CUDA;
}

constexpr int kMaxDevices = 64;

// SMs of the current device (148 when it cannot be read).
int sms() {
    static int cached[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
    if (cached[dev] == 0) {
        int v = 0;
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || v <= 0) v = 148;
        cached[dev] = v;
    }
    return cached[dev];
}

// Which kernel: few rows or outputs, the tensor cores where TMA can read the operands, the CUDA cores otherwise.
// Against the tensor cores (bf16) the row kernel wins up to 8 rows, which read w once (8 x 1280 -> 5120: 8.2 us against 11.4),
// and up to 32 rows for about 45000 outputs (32 x 512 -> 1000: 3.7 against 5.1; 48 x 1280 -> 1280: 9.3 against 7.5; more
// rows stay on the tensor cores, where a row's sums do not depend on how many there are).  Against the tiles of the
// CUDA cores (fp32) it wins while the tiles are few: they take about 0.07 us per column of K whatever their number up to two
// per SM, and it takes 9e-8 us per product and 3e-5 per output (512 x 640 -> 640: 28 us against 40; 1024 x 640 -> 640: 53 against
// 50; 8192 x 64 -> 64: 18 against 7).
cudaError_t launch_matmul(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    const bool tma = matmul_tma_operands(a);
    const double outputs = (double)a.M * a.N, K = (double)a.K0 + a.K1;
    const bool few = tma ? a.M <= 8 || (a.M <= 32 && outputs <= 45000.0) : a.M <= 16 || outputs * (K + 330.0) <= 780000.0 * K;
    if (few && a.M <= kMaxRowsM) return launch_matmul_rows(a, num_sms, st);
    return tma ? launch_matmul_tc(a, num_sms, st) : launch_matmul_simt(a, num_sms, st);
}

bool natural(const void* p, size_t size) { return (reinterpret_cast<uintptr_t>(p) & (size - 1)) == 0; }
bool dtype_ok(int t) { return t == WINO_F32 || t == WINO_BF16; }
size_t size_of(int t) { return t == WINO_BF16 ? 2 : 4; }

constexpr int64_t kMaxPitch = (int64_t)1 << 31;
constexpr int kMaxSize = 2147483647 - 1024;        // a size rounded up to a tile stays an int
constexpr double kMaxElements = 1099511627776.0;   // 2^40

// A matrix in device memory, for the overlap check: `rows` rows of `width` bytes, `pitch` bytes apart.
struct Region {
    uintptr_t p;
    size_t rows, width, pitch;
};
Region region(const void* p, size_t rows, size_t cols, int64_t pitch, size_t es) {
    return {reinterpret_cast<uintptr_t>(p), rows, cols * es, (size_t)pitch * es};
}
// Whether the two share a byte.  Column ranges of one wider buffer (equal pitches) are told apart;
// otherwise overlapping address ranges count as sharing.  A single row's pitch may be anything, 0 too: it is not looked at.
bool overlap(const Region& a, const Region& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t ae = a.p + (a.rows - 1) * a.pitch + a.width, be = b.p + (b.rows - 1) * b.pitch + b.width;
    if (ae <= b.p || be <= a.p) return false;
    if (a.rows == 1 && b.rows == 1) return true;
    const size_t pitch = a.rows == 1 ? b.pitch : a.pitch;
    if (b.rows > 1 && b.pitch != pitch) return true;
    const size_t d = b.p >= a.p ? (b.p - a.p) % pitch : (pitch - (a.p - b.p) % pitch) % pitch;
    return !(d >= a.width && d + b.width <= pitch);
}
// Exactly the same matrix: an operator may update it in place.
bool same(const Region& a, const Region& b) { return a.p == b.p && a.width == b.width && (a.pitch == b.pitch || a.rows == 1); }

bool pitch_ok(int64_t pitch, int cols, size_t rows) {
    return pitch <= kMaxPitch && (pitch >= cols || (rows == 1 && pitch >= 0));
}

}  // namespace

namespace wino {
int ops_last_cuda_error() { return t_last_cuda; }
}  // namespace wino

extern "C" {

int wino_group_norm(const wino_group_norm_args* g, void* stream) {
    if (!g || !g->x || !g->y || g->N <= 0 || g->H <= 0 || g->W <= 0 || g->C <= 0 || g->C2 < 0 || g->groups <= 0)
        return WINO_ERR_INVALID_ARG;
    if ((g->C2 > 0) != (g->x2 != nullptr) || !dtype_ok(g->x_dtype) || !dtype_ok(g->y_dtype)) return WINO_ERR_INVALID_ARG;
    if (g->act < WINO_ACT_NONE || g->act > WINO_ACT_GELU || !(g->eps >= 0.0f) || g->eps > 3e38f) return WINO_ERR_INVALID_ARG;
    const int64_t C = (int64_t)g->C + g->C2;
    if (C % g->groups != 0) return WINO_ERR_INVALID_ARG;
    const double hw = (double)g->H * g->W;
    if (hw > 1073741824.0 || hw * g->N > kMaxElements || hw * g->N * C > kMaxElements) return WINO_ERR_INVALID_ARG;
    const size_t rows = (size_t)g->N * g->H * g->W, xs = size_of(g->x_dtype), ys = size_of(g->y_dtype);
    if (!pitch_ok(g->x_pitch, g->C, rows) || (g->C2 && !pitch_ok(g->x2_pitch, g->C2, rows)) ||
        !pitch_ok(g->y_pitch, (int)C, rows))
        return WINO_ERR_INVALID_ARG;
    if (!natural(g->x, xs) || !natural(g->x2, xs) || !natural(g->y, ys) || !natural(g->add, 4) || !natural(g->gamma, 4) ||
        !natural(g->beta, 4))
        return WINO_ERR_INVALID_ARG;
    const Region y = region(g->y, rows, (size_t)C, g->y_pitch, ys), x = region(g->x, rows, g->C, g->x_pitch, xs);
    const bool in_place = !g->C2 && xs == ys && same(x, y);
    if ((!in_place && overlap(x, y)) || overlap(region(g->x2, rows, g->C2, g->x2_pitch, xs), y) ||
        overlap(region(g->add, (size_t)g->N, (size_t)C, C, 4), y) || overlap(region(g->gamma, 1, (size_t)C, C, 4), y) ||
        overlap(region(g->beta, 1, (size_t)C, C, 4), y))
        return WINO_ERR_INVALID_ARG;
    if (C > WINO_GROUP_NORM_MAX_CHANNELS || g->N > WINO_GROUP_NORM_MAX_IMAGES) return WINO_ERR_UNSUPPORTED;
    GroupNormArgs a = {};
    a.x = g->x;
    a.x2 = g->x2;
    a.add = g->add;
    a.gamma = g->gamma;
    a.beta = g->beta;
    a.y = g->y;
    a.ld0 = (long)g->x_pitch;
    a.ld1 = (long)g->x2_pitch;
    a.ldy = (long)g->y_pitch;
    a.HW = (long)g->H * g->W;
    a.N = g->N;
    a.C0 = g->C;
    a.C1 = g->C2;
    a.groups = g->groups;
    a.act = g->act;
    a.eps = g->eps;
    a.x_bf16 = g->x_dtype == WINO_BF16;
    a.y_bf16 = g->y_dtype == WINO_BF16;
    nvtxRangePushA("wino: group norm");
    const cudaError_t e = launch_group_norm(a, sms(), static_cast<cudaStream_t>(stream));
    nvtxRangePop();
    return status(e);
}

int wino_matmul(const wino_matmul_args* g, void* stream) {
    if (!g || !g->a || !g->w || !g->out || g->M <= 0 || g->N <= 0 || g->K <= 0 || g->K2 < 0) return WINO_ERR_INVALID_ARG;
    if ((g->K2 > 0) != (g->a2 != nullptr) || !dtype_ok(g->dtype) || !dtype_ok(g->out_dtype)) return WINO_ERR_INVALID_ARG;
    if (g->act < WINO_ACT_NONE || g->act > WINO_ACT_GELU) return WINO_ERR_INVALID_ARG;
    const int64_t K = (int64_t)g->K + g->K2;
    if (K > kMaxSize || g->M > kMaxSize || g->N > kMaxSize || (double)g->M * K > kMaxElements || (double)g->N * K > kMaxElements ||
        (double)g->M * g->N > kMaxElements)
        return WINO_ERR_INVALID_ARG;
    const size_t M = (size_t)g->M, N = (size_t)g->N, s = size_of(g->dtype), so = size_of(g->out_dtype);
    if (!pitch_ok(g->a_pitch, g->K, M) || (g->K2 && !pitch_ok(g->a2_pitch, g->K2, M)) || !pitch_ok(g->w_pitch, (int)K, N) ||
        (g->residual && !pitch_ok(g->residual_pitch, g->N, M)) || !pitch_ok(g->out_pitch, g->N, M))
        return WINO_ERR_INVALID_ARG;
    if (!natural(g->a, s) || !natural(g->a2, s) || !natural(g->w, s) || !natural(g->bias, 4) || !natural(g->residual, so) ||
        !natural(g->out, so))
        return WINO_ERR_INVALID_ARG;
    const Region out = region(g->out, M, N, g->out_pitch, so), res = region(g->residual, M, N, g->residual_pitch, so);
    if (overlap(region(g->a, M, g->K, g->a_pitch, s), out) || overlap(region(g->a2, M, g->K2, g->a2_pitch, s), out) ||
        overlap(region(g->w, N, (size_t)K, g->w_pitch, s), out) || overlap(region(g->bias, 1, N, g->N, 4), out) ||
        (g->residual && !same(res, out) && overlap(res, out)))
        return WINO_ERR_INVALID_ARG;
    MatmulArgs a = {};
    a.a = g->a;
    a.a2 = g->a2;
    a.w = g->w;
    a.bias = g->bias;
    a.res = g->residual;
    a.out = g->out;
    a.lda = (long)g->a_pitch;
    a.lda2 = (long)g->a2_pitch;
    a.ldw = (long)g->w_pitch;
    a.ldr = (long)g->residual_pitch;
    a.ldo = (long)g->out_pitch;
    a.M = g->M;
    a.N = g->N;
    a.K0 = g->K;
    a.K1 = g->K2;
    a.act = g->act;
    a.bf16 = g->dtype == WINO_BF16;
    a.out_bf16 = g->out_dtype == WINO_BF16;
    a.force_timeout = g->reserved == WINO_DEBUG_FORCE_TIMEOUT;
    nvtxRangePushA("wino: matmul");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = launch_matmul(a, sms(), st);
    nvtxRangePop();
    return status(e);
}

int wino_check_device_error_ops(void* stream) {
    cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return status(e);
    int first = 0;
    for (auto take : {group_norm_take_error, matmul_simt_take_error, matmul_rows_take_error, matmul_tc_take_error}) {
        int v = 0;
        if ((e = take(&v)) != cudaSuccess) return status(e);
        if (first == 0) first = v;
    }
    if (first == 0) return WINO_OK;
    return first == kDevErrBounds ? WINO_ERR_DEVICE_BOUNDS : WINO_ERR_DEVICE_TIMEOUT;
}

}  // extern "C"
