// Matrix product with bias, activation and residual on the CUDA cores: every
// type, size, pitch and alignment.  A 64x64 tile of the output per CTA, 16 of K
// at a time through shared memory, 4x4 outputs per thread, fp32 sums.
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace wino {
namespace {

__device__ int g_err;   // first failed index check since matmul_simt_take_error (debug build)

constexpr int kTile = 64, kStep = 16, kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}

template <typename T, typename TO>
__global__ void __launch_bounds__(kThreads) matmul_simt_kernel(const MatmulArgs p) {
    __shared__ float sa[kStep][kTile + 4], sw[kStep][kTile + 4];
    const int K = p.K0 + p.K1;
    const int tiles_n = (p.N + kTile - 1) / kTile;
    const int m0 = (int)(blockIdx.x / tiles_n) * kTile, n0 = (int)(blockIdx.x % tiles_n) * kTile;
    const int tid = threadIdx.x, tm = tid / 16 * 4, tn = tid % 16 * 4;
    grid_dependents_launch();
    grid_dependency_wait();
    float acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += kStep) {
#pragma unroll
        for (int i = 0; i < kTile * kStep / kThreads; ++i) {
            const int e = tid + i * kThreads, r = e / kStep, kk = e % kStep, k = k0 + kk;
            float va = 0.0f, vw = 0.0f;
            if (k < K && m0 + r < p.M) {
                const bool second = k >= p.K0;
                const size_t at = second ? (size_t)(m0 + r) * p.lda2 + (k - p.K0) : (size_t)(m0 + r) * p.lda + k;
                const size_t n = second ? (size_t)(p.M - 1) * p.lda2 + p.K1 : (size_t)(p.M - 1) * p.lda + p.K0;
                if (in_bounds(at, n, &g_err)) va = to_f32(static_cast<const T*>(second ? p.a2 : p.a)[at]);
            }
            if (k < K && n0 + r < p.N) {
                const size_t at = (size_t)(n0 + r) * p.ldw + k;
                if (in_bounds(at, (size_t)(p.N - 1) * p.ldw + K, &g_err)) vw = to_f32(static_cast<const T*>(p.w)[at]);
            }
            sa[kk][r] = va;
            sw[kk][r] = vw;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kStep; ++kk) {
            const float4 av = *reinterpret_cast<const float4*>(&sa[kk][tm]);
            const float4 wv = *reinterpret_cast<const float4*>(&sw[kk][tn]);
            const float am[4] = {av.x, av.y, av.z, av.w}, wn[4] = {wv.x, wv.y, wv.z, wv.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(am[i], wn[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + tm + i, n = n0 + tn + j;
            if (m >= p.M || n >= p.N) continue;
            float v = acc[i][j] + (p.bias ? p.bias[n] : 0.0f);
            if (p.act == WINO_ACT_SILU) v = activate<WINO_ACT_SILU, sizeof(TO) == 2>(v);
            if (p.act == WINO_ACT_GELU) v = activate<WINO_ACT_GELU, sizeof(TO) == 2>(v);
            const size_t at = (size_t)m * p.ldo + n;
            if (!in_bounds(at, (size_t)(p.M - 1) * p.ldo + p.N, &g_err)) continue;
            if (p.res) v += to_f32(static_cast<const TO*>(p.res)[(size_t)m * p.ldr + n]);
            if constexpr (sizeof(TO) == 2) static_cast<TO*>(p.out)[at] = __float2bfloat16_rn(v);
            else static_cast<TO*>(p.out)[at] = v;
        }
}

}  // namespace

cudaError_t launch_matmul_simt(const MatmulArgs& a, cudaStream_t st) {
    const long tiles = (long)((a.M + (long)kTile - 1) / kTile) * ((a.N + (long)kTile - 1) / kTile);
    if (tiles > 2147483647L) return cudaErrorInvalidConfiguration;
    const dim3 grid((unsigned)tiles), block(kThreads);
    using B = __nv_bfloat16;
    if (a.bf16)
        return a.out_bf16 ? launch_dependent(matmul_simt_kernel<B, B>, grid, block, 0, st, a)
                          : launch_dependent(matmul_simt_kernel<B, float>, grid, block, 0, st, a);
    return a.out_bf16 ? launch_dependent(matmul_simt_kernel<float, B>, grid, block, 0, st, a)
                      : launch_dependent(matmul_simt_kernel<float, float>, grid, block, 0, st, a);
}

cudaError_t matmul_simt_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
