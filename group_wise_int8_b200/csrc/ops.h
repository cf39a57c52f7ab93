// Kernels of the operators beside the convolution (internal header): group
// normalisation with an activation on NHWC activations, and the matrix product
// with bias, activation and residual in its epilogue.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

#include "../../include/wino.h"
#include "common.cuh"

namespace wino {

// ------------------------------------------------------------ activations
// SiLU v / (1 + exp(-v)) and GELU v Phi(v) in fp32.  FAST: the result is rounded to bf16 next, so the hardware's
// exponential and reciprocal (relative error below 2^-20, bf16's rounding is up to 2^-8) serve; otherwise the
// accurate expf (2 ulp) and a reciprocal to 1 ulp: below 2^-21 in all (SiLU over |v| <= 80: 2.2e-7 at most, 3.4e-8 on
// average; with a rounded division 1.9e-7 and 2.9e-8, and a group norm of 7 x 48 x 61 x 352 fp32 26 us, not 23).
// exp(-v) beyond fp32's range, or its inverse flushed to zero, makes SiLU below v = -88.7 (FAST: -87.3) zero, where it
// is smaller than 1e-36 in magnitude.
__device__ __forceinline__ float exp2_fast(float v) {   // results below 2^-126 become 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float reciprocal_full(float v) {   // to 1 ulp, subnormal results too
    float r;
    asm("rcp.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

template <bool FAST>
__device__ __forceinline__ float silu(float v) {
    // exp(-v) = inf (v below about -88) gives v * (1 / inf) = -0
    if (FAST) return reciprocal(1.0f + exp2_fast(v * -1.4426950408889634f)) * v;
    return v * reciprocal_full(1.0f + expf(-v));
}

// FAST GELU.  The tail q(a) = Phi(-a) = erfc(a / sqrt 2) / 2, a = |v|, is exp(-a^2 / 2) t P(t) with t = 1 / (1 + 0.3 a)
// and P the degree-7 polynomial of least relative error (2^-23, a least-squares fit reweighted towards the
// minimax one) to erfc(a / sqrt 2) exp(a^2 / 2) / (2t) on 0 <= a <= 13.2; beyond, q is below 2^-126 and v q, below
// 6e-39, comes out as zero.  v Phi(v) is v q for negative v and v (1 - q) otherwise, so that the left tail keeps its relative error: with fp32
// arithmetic below 2^-20, plus a^2 2^-24 through the exponential's argument.  Two values go through one reciprocal.
__device__ __forceinline__ void gelu_pair(float& v0, float& v1) {
    constexpr float P[8] = {0.1196245402097702f,  0.12082631886005402f, 0.09946505725383759f, 0.13003262877464294f,
                            -0.056450121104717255f, 0.20934641361236572f, -0.15893374383449554f, 0.036088839173316956f};
    const float a0 = fminf(fabsf(v0), 16.0f), a1 = fminf(fabsf(v1), 16.0f);   // (a NaN stays in the last product)
    const uint64_t a = f2_pack(a0, a1);
    float d0, d1, x0, x1;
    f2_unpack(f2_fma(a, f2_pack(0.3f, 0.3f), f2_pack(1.0f, 1.0f)), d0, d1);
    const float r = reciprocal(d0 * d1);
    const uint64_t t = f2_pack(r * d1, r * d0);
    uint64_t p = f2_pack(P[7], P[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) p = f2_fma(p, t, f2_pack(P[i], P[i]));
    f2_unpack(f2_mul(f2_mul(a, a), f2_pack(-0.72134752044448170f, -0.72134752044448170f)), x0, x1);   // -a^2 / 2 log2(e)
    float q0, q1;
    f2_unpack(f2_mul(f2_pack(exp2_fast(x0), exp2_fast(x1)), f2_mul(t, p)), q0, q1);
    v0 *= v0 < 0.0f ? q0 : 1.0f - q0;
    v1 *= v1 < 0.0f ? q1 : 1.0f - q1;
}

template <int ACT, bool FAST>
__device__ __forceinline__ float activate(float v) {
    if (ACT == WINO_ACT_SILU) return silu<FAST>(v);
    if (ACT == WINO_ACT_GELU && FAST) {
        float other = 0.0f;
        gelu_pair(v, other);
        return v;
    }
    if (ACT == WINO_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    return v;
}

// FAST SiLU of four values with one reciprocal, since the special-function unit is its bound (1.25 operations there per
// value instead of 2).  With e = exp(-|v|) and d = 1 + e, at most 2, v sigmoid(v) is v / d for v >= 0 and v e / d
// otherwise; X = (d0 d2, d1 d3) and r = 1 / (X0 X1) give the reciprocals of (d0, d1) as (r X1, r X0) (d2, d3) and those of
// (d2, d3) as the same pair times (d0, d1).  (min drops a NaN, which would reach its neighbours through r; the last
// product restores it.)
__device__ __forceinline__ void silu_quad(float& v0, float& v1, float& v2, float& v3) {
    const uint64_t scale = f2_pack(-1.4426950408889634f, -1.4426950408889634f), one = f2_pack(1.0f, 1.0f);
    float t0, t1, t2, t3, x0, x1;
    f2_unpack(f2_mul(f2_pack(fminf(fabsf(v0), 128.0f), fminf(fabsf(v1), 128.0f)), scale), t0, t1);
    f2_unpack(f2_mul(f2_pack(fminf(fabsf(v2), 128.0f), fminf(fabsf(v3), 128.0f)), scale), t2, t3);
    const float e0 = exp2_fast(t0), e1 = exp2_fast(t1), e2 = exp2_fast(t2), e3 = exp2_fast(t3);
    const uint64_t da = f2_add(f2_pack(e0, e1), one), db = f2_add(f2_pack(e2, e3), one);
    f2_unpack(f2_mul(da, db), x0, x1);
    const float r = reciprocal(x0 * x1);
    const uint64_t y = f2_pack(r * x1, r * x0);
    const uint64_t na = f2_pack(v0 < 0.0f ? e0 : 1.0f, v1 < 0.0f ? e1 : 1.0f);
    const uint64_t nb = f2_pack(v2 < 0.0f ? e2 : 1.0f, v3 < 0.0f ? e3 : 1.0f);
    const uint64_t sa = f2_mul(f2_mul(y, db), na), sb = f2_mul(f2_mul(y, da), nb);   // the sigmoids
    f2_unpack(f2_mul(f2_pack(v0, v1), sa), v0, v1);
    f2_unpack(f2_mul(f2_pack(v2, v3), sb), v2, v3);
}

// Activates N values.
template <int ACT, bool FAST, int N>
__device__ __forceinline__ void activate_all(float (&v)[N]) {
    if constexpr (ACT == WINO_ACT_SILU && FAST && N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) silu_quad(v[i], v[i + 1], v[i + 2], v[i + 3]);
        return;
    }
    if constexpr (ACT == WINO_ACT_GELU && FAST && N % 2 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 2) gelu_pair(v[i], v[i + 1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = activate<ACT, FAST>(v[i]);
}

// ------------------------------------------------------------ group norm
struct GroupNormArgs {
    const void* x;         // [N][HW] pixels, C0 channels, pitch ld0 elements
    const void* x2;        // the channels after C0 (C1 of them), pitch ld1; null when C1 == 0
    const float* add;      // [N][C] or null
    const float* gamma;    // [C] or null (1)
    const float* beta;     // [C] or null (0)
    void* y;               // [N][HW] pixels, C channels, pitch ldy
    long ld0, ld1, ldy;
    long HW;
    int N, C0, C1, groups, act;
    float eps;
    bool x_bf16, y_bf16;
};

cudaError_t launch_group_norm(const GroupNormArgs& a, int num_sms, cudaStream_t st);

// --------------------------------------------------------- matrix product
struct MatmulArgs {
    const void* a;         // [M][K0], pitch lda
    const void* a2;        // [M][K1], pitch lda2 (null when K1 == 0)
    const void* w;         // [N][K0 + K1], pitch ldw
    const float* bias;     // [N] or null
    const void* res;       // [M][N] of the output's type, pitch ldr, or null
    void* out;             // [M][N], pitch ldo
    long lda, lda2, ldw, ldr, ldo;
    int M, N, K0, K1, act;
    bool bf16;             // operand type: bf16 or fp32
    bool out_bf16;
    bool force_timeout;    // test hook of the tensor-core kernel: one of its bounded waits runs out
};
// The CUDA-core kernel: any type, size, pitch and alignment.
cudaError_t launch_matmul_simt(const MatmulArgs& a, int num_sms, cudaStream_t st);

// For a few rows (at most 65535 blocks of 8): any type, size, pitch and alignment.
constexpr int kMaxRowsM = 8 * 65535;   // rows that the row kernel's grid holds
cudaError_t launch_matmul_rows(const MatmulArgs& a, int num_sms, cudaStream_t st);

// The tensor-core kernel takes bf16 operands that TMA can read (16-byte aligned bases and pitches).
bool matmul_tma_operands(const MatmulArgs& a);
cudaError_t launch_matmul_tc(const MatmulArgs& a, int num_sms, cudaStream_t st);

// Device error words of the kernels above on the current device: the first error recorded since
// the last call of the function, which clears it (0: none).
cudaError_t group_norm_take_error(int* err);
cudaError_t matmul_simt_take_error(int* err);
cudaError_t matmul_rows_take_error(int* err);
cudaError_t matmul_tc_take_error(int* err);

// Last CUDA error of the calling thread's calls without a plan.
int ops_last_cuda_error();

// Sets a kernel's dynamic shared memory limit once per device (the attribute holds until exit).
template <typename F>
cudaError_t allow_smem(F* kern, size_t bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev >= 0 && dev < 64) done[dev] = true;
    return e;
}

}  // namespace wino
