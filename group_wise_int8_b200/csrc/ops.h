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

namespace wino {

// ------------------------------------------------------------ activations
// SiLU and GELU (erf form) in fp32.  FAST: the result is rounded to bf16 next, so the approximate
// exponential and reciprocal (relative error below 2^-20, bf16 rounds at 2^-9) serve; otherwise the
// accurate expf and an IEEE division.
template <bool FAST>
__device__ __forceinline__ float silu(float v) {
    // exp(-v) = inf (v below about -88) gives v * (1 / inf) = -0
    if (FAST) return __fdividef(1.0f, 1.0f + __expf(-v)) * v;
    return v / (1.0f + expf(-v));
}

template <bool FAST>
__device__ __forceinline__ float activate(float v, int act) {
    if (act == WINO_ACT_SILU) return silu<FAST>(v);
    if (act == WINO_ACT_GELU) return 0.5f * v * erfcf(v * -0.70710678118654752f);
    return v;
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
    // set by the launcher
    int cg;                // channels per group
    int gps;               // groups per slab
    int slabs;             // slabs per image
    int vec_y;             // 1: rows of y take whole-vector stores
    int res_rows;          // rows of a CTA kept in shared memory
};

// How a call is cut: a cluster of `cluster` CTAs per (image, slab of `gps` groups).
struct GroupNormSplit {
    int gps, cluster;
};
GroupNormSplit group_norm_split(const GroupNormArgs& a, int vec, int num_sms);
// split: null for the rule's choice.
cudaError_t launch_group_norm(GroupNormArgs a, int num_sms, const GroupNormSplit* split, cudaStream_t st);

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
};
// The CUDA-core kernel: any type, size, pitch and alignment.
cudaError_t launch_matmul_simt(const MatmulArgs& a, cudaStream_t st);

// The tensor-core kernels take bf16 operands that TMA can read (16-byte aligned bases and pitches).
bool matmul_tma_operands(const MatmulArgs& a);
bool matmul_operand_maps(const MatmulArgs& a, int w_rows, CUtensorMap (&map)[4]);   // a, a2, w for a, w for a2
// Persistent pair kernel for outputs of many tiles; bn: tile width (a multiple of 32 up to 256), 0: by the rule.
int matmul_tc_width(const MatmulArgs& a, int num_sms);
cudaError_t launch_matmul_tc(const MatmulArgs& a, int bn, int num_sms, cudaStream_t st);

// Device error words of the kernels above on the current device: the first error recorded since
// the last call of the function, which clears it (0: none).
cudaError_t group_norm_take_error(int* err);
cudaError_t matmul_simt_take_error(int* err);
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
