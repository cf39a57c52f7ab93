// Matrix product with bias, activation and residual for few rows or outputs (the projection of a batch's
// embeddings, a classifier): out = act([a | a2] w^T + bias) + residual; up to 8 rows per CTA.
//
// Bound: reading w once (M rows of a are small); at these sizes the latency of a launch and of one trip to memory
// (1 x 1280 -> 1280 bf16: 2.3 us for 3.3 MB; 8 x 320 -> 1280 fp32: 3.1 us; 16 x 1280 -> 1280 fp32: 6.0 us).
//
// A warp takes COLS consecutive output columns: its lanes stride over K in 16-byte vectors of w, several loads of each
// in flight at once, and multiply them with the rows of a (which all warps share
// through L1).  fp32 sums in every lane, as packed pairs, joined by shuffles in a fixed order.  bf16 products are exact in
// fp32.  Eight rows at most, so that the sums leave four CTAs per SM their registers (16 rows: 16 x 1280 -> 1280 fp32 10.4
// us, 6.0 as two blocks of eight).
// Where a base, a pitch or K's split is not a multiple of 16 bytes, one value at a time.
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace wino {
namespace {

__device__ int g_err;   // first failed index check since matmul_rows_take_error (debug build)

constexpr int kWarps = 4;

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(T) == 2) v[0] = __bfloat162float(*p);
        else v[0] = *p;
    } else {
        const uint4 r = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                v[2 * i] = __uint_as_float(w[i] << 16);
                v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            } else {
                v[i] = __uint_as_float(w[i]);
            }
        }
    }
}

// ROWS: rows of a per warp (M rounded up); COLS: output columns per warp.
template <typename T, typename TO, int VEC, int ROWS, int COLS>
__global__ void __launch_bounds__(32 * kWarps, 4) matmul_rows_kernel(const MatmulArgs p) {
    const int lane = threadIdx.x & 31;
    const int m0 = (int)blockIdx.y * ROWS;
    const int n0 = ((int)blockIdx.x * kWarps + (int)(threadIdx.x >> 5)) * COLS;
    const T *w = static_cast<const T*>(p.w), *a0 = static_cast<const T*>(p.a), *a1 = static_cast<const T*>(p.a2);
    grid_dependents_launch();
    grid_dependency_wait();
    if (n0 >= p.N) return;
    uint64_t acc[ROWS][COLS];   // packed pairs: the sums of even and of odd columns of K
#pragma unroll
    for (int m = 0; m < ROWS; ++m)
#pragma unroll
        for (int c = 0; c < COLS; ++c) acc[m][c] = 0ull;
    const size_t w_end = (size_t)(p.N - 1) * p.ldw + p.K0 + p.K1;
    auto source = [&](const T* a, long lda, int K, int k_off) {
        const size_t a_end = (size_t)(p.M - 1) * lda + K;
#pragma unroll 2
        for (int k = lane * VEC; k < K; k += 32 * VEC) {
            float wv[COLS][VEC];
#pragma unroll
            for (int c = 0; c < COLS; ++c) {
                const size_t at = (size_t)min(n0 + c, p.N - 1) * p.ldw + k_off + k;
#pragma unroll
                for (int i = 0; i < VEC; ++i) wv[c][i] = 0.0f;
                if (in_bounds(at + VEC - 1, w_end, &g_err)) load_vec<T, VEC>(w + at, wv[c]);
            }
#pragma unroll
            for (int m = 0; m < ROWS; ++m) {
                const size_t at = (size_t)min(m0 + m, p.M - 1) * lda + k;
                float av[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) av[i] = 0.0f;
                if (in_bounds(at + VEC - 1, a_end, &g_err)) load_vec<T, VEC>(a + at, av);
#pragma unroll
                for (int c = 0; c < COLS; ++c)
#pragma unroll
                    for (int i = 0; i < VEC; i += 2) {
                        const int j = i + 1 < VEC ? i + 1 : i;   // (one value at a time: both sums hold it)
                        acc[m][c] = f2_fma(f2_pack(av[i], av[j]), f2_pack(wv[c][i], wv[c][j]), acc[m][c]);
                    }
            }
        }
    };
    source(a0, p.lda, p.K0, 0);
    if (p.K1) source(a1, p.lda2, p.K1, p.K0);
    // the warp's sums: at each step a lane keeps half of its outputs and sends the other half, so that all of them take
    // about as many shuffles as there are outputs, and a lane ends with one (column fastest)
    constexpr int P = ROWS * COLS, kLanes = 32 / P;   // lanes that end with the same output
    float sum[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float even, odd;
        f2_unpack(acc[i / COLS][i % COLS], even, odd);
        sum[i] = VEC > 1 ? even + odd : even;
    }
#pragma unroll
    for (int n = P / 2, o = 16; o > 0; n >>= 1, o >>= 1) {
        if (n > 0) {
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float mine = lane & o ? sum[i + n] : sum[i], other = lane & o ? sum[i] : sum[i + n];
                sum[i] = mine + __shfl_xor_sync(0xffffffffu, other, o);
            }
        } else {
            sum[0] += __shfl_xor_sync(0xffffffffu, sum[0], o);
        }
    }
    {
        float v = sum[0];
        const int i = lane / kLanes, m = m0 + i / COLS, n = n0 + i % COLS;
        if (lane % kLanes != 0 || m >= p.M || n >= p.N) return;
        v += p.bias ? p.bias[n] : 0.0f;
        if (p.act == WINO_ACT_SILU) v = activate<WINO_ACT_SILU, sizeof(TO) == 2>(v);
        if (p.act == WINO_ACT_GELU) v = activate<WINO_ACT_GELU, sizeof(TO) == 2>(v);
        const size_t at = (size_t)m * p.ldo + n;
        if (!in_bounds(at, (size_t)(p.M - 1) * p.ldo + p.N, &g_err)) return;
        if constexpr (sizeof(TO) == 2) {
            if (p.res) v += __bfloat162float(static_cast<const TO*>(p.res)[(size_t)m * p.ldr + n]);
            static_cast<TO*>(p.out)[at] = __float2bfloat16_rn(v);
        } else {
            if (p.res) v += static_cast<const TO*>(p.res)[(size_t)m * p.ldr + n];
            static_cast<TO*>(p.out)[at] = v;
        }
    }
}

bool aligned16(const void* p, long pitch, int rows, size_t es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows == 1 || (size_t)pitch * es % 16 == 0);
}

template <typename T, typename TO, int VEC, int ROWS>
cudaError_t launch_cols(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    // two columns per warp halve the reads of a, but only while they leave every SM a block
    const bool two = ROWS > 1 && (long)a.N * ((a.M + ROWS - 1) / ROWS) >= 2L * kWarps * num_sms;
    const int per = kWarps * (two ? 2 : 1);
    const dim3 grid((unsigned)((a.N + per - 1) / per), (unsigned)((a.M + ROWS - 1) / ROWS)), block(32 * kWarps);
    return two ? launch_dependent(matmul_rows_kernel<T, TO, VEC, ROWS, 2>, grid, block, 0, st, a)
               : launch_dependent(matmul_rows_kernel<T, TO, VEC, ROWS, 1>, grid, block, 0, st, a);
}

template <typename T, typename TO, int VEC>
cudaError_t launch_rows(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    if (a.M == 1) return launch_cols<T, TO, VEC, 1>(a, num_sms, st);
    if (a.M <= 4) return launch_cols<T, TO, VEC, 4>(a, num_sms, st);
    return launch_cols<T, TO, VEC, 8>(a, num_sms, st);
}

template <typename T, typename TO>
cudaError_t launch_vec(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(T);
    const bool vec = aligned16(a.a, a.lda, a.M, sizeof(T)) && aligned16(a.w, a.ldw, a.N, sizeof(T)) && a.K0 % VEC == 0 &&
                     (a.K1 == 0 || (aligned16(a.a2, a.lda2, a.M, sizeof(T)) && a.K1 % VEC == 0));
    return vec ? launch_rows<T, TO, VEC>(a, num_sms, st) : launch_rows<T, TO, 1>(a, num_sms, st);
}

}  // namespace

cudaError_t launch_matmul_rows(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    if (a.M > kMaxRowsM) return cudaErrorInvalidValue;
    using B = __nv_bfloat16;
    if (a.bf16) return a.out_bf16 ? launch_vec<B, B>(a, num_sms, st) : launch_vec<B, float>(a, num_sms, st);
    return a.out_bf16 ? launch_vec<float, B>(a, num_sms, st) : launch_vec<float, float>(a, num_sms, st);
}

cudaError_t matmul_rows_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
