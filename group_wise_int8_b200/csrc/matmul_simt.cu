// Matrix product with bias, activation and residual on the CUDA cores: every
// type, size, pitch and alignment (fp32 operands, and bf16 ones that TMA cannot
// read).
//
// Bound: the fp32 pipes, 2 M N K operations at 74 TFLOP/s.  8192 x 1280 -> 1280 runs at 44 (the installed library: 58), and fewer tiles than SMs
// at less (512 x 1280 -> 1280: 17; the library 31).
//
// A 128 x 128 or 64 x 64 tile of the output per CTA of 256 threads, 8 x 8 or 4 x 4
// outputs per thread.  16 columns of K at a time go through shared memory, transposed so that a
// thread's rows and columns are 16-byte reads; the next 16 are on their way from
// memory in registers meanwhile, into the other of two buffers.  Sums are packed
// fp32 pairs.
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace wino {
namespace {

__device__ int g_err;   // first failed index check since matmul_simt_take_error (debug build)

constexpr int kStep = 16, kThreads = 256;

template <typename T>
__device__ __forceinline__ float to_f32(T v) {
    if constexpr (sizeof(T) == 2) return __bfloat162float(v);
    else return v;
}

// TILE / 16 consecutive values of K of one row of an operand, from column k0 (zero past its end).
template <typename T, int PER>
struct Fetch {
    float v[PER];
    // `vec`: the row starts at, and every PER columns keep, 16-byte (or PER-value) alignment
    __device__ __forceinline__ void load(const T* base, long ld, int row, int rows, int k, int K, bool vec) {
        const size_t end = (size_t)(rows - 1) * ld + K, at = (size_t)row * ld + k;
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i] = 0.0f;
        if (row >= rows) return;
        if (vec && k + PER <= K) {
            if (!in_bounds(at + PER - 1, end, &g_err)) return;
            if constexpr (sizeof(T) == 4) {
#pragma unroll
                for (int i = 0; i < PER; i += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(base + at + i);
                    v[i] = f.x;
                    v[i + 1] = f.y;
                    v[i + 2] = f.z;
                    v[i + 3] = f.w;
                }
            } else {
                uint32_t w[PER / 2];
                if constexpr (PER == 8) *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(base + at);
                else *reinterpret_cast<uint2*>(w) = *reinterpret_cast<const uint2*>(base + at);
#pragma unroll
                for (int i = 0; i < PER / 2; ++i) {
                    v[2 * i] = __uint_as_float(w[i] << 16);
                    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (k + i < K && in_bounds(at + i, end, &g_err)) v[i] = to_f32(base[at + i]);
        }
    }
};

template <typename T, typename TO, int TILE>
__global__ void __launch_bounds__(kThreads, 2) matmul_simt_kernel(const MatmulArgs p, const int vec) {
    constexpr int PER = TILE / 16, PITCH = TILE + 4;   // outputs per thread and side; also values fetched per thread
    __shared__ __align__(16) float sa[2][kStep][PITCH], sw[2][kStep][PITCH];
    const int tiles_n = (p.N + TILE - 1) / TILE;
    const int m0 = (int)(blockIdx.x / tiles_n) * TILE, n0 = (int)(blockIdx.x % tiles_n) * TILE;
    const int tid = threadIdx.x, tm = tid / 16 * 4, tn = tid % 16 * 4;
    const int fr = tid / (kStep / PER), fk = tid % (kStep / PER) * PER;   // the row and column this thread fetches
    grid_dependents_launch();
    grid_dependency_wait();

    const int steps0 = (p.K0 + kStep - 1) / kStep, steps = steps0 + (p.K1 + kStep - 1) / kStep;
    Fetch<T, PER> fa, fw;
    auto fetch = [&](int s) {
        const bool second = s >= steps0;
        const int k = (second ? s - steps0 : s) * kStep + fk;
        if (second) {
            fa.load(static_cast<const T*>(p.a2), p.lda2, m0 + fr, p.M, k, p.K1, vec != 0);
            fw.load(static_cast<const T*>(p.w) + p.K0, p.ldw, n0 + fr, p.N, k, p.K1, vec != 0);
        } else {
            fa.load(static_cast<const T*>(p.a), p.lda, m0 + fr, p.M, k, p.K0, vec != 0);
            fw.load(static_cast<const T*>(p.w), p.ldw, n0 + fr, p.N, k, p.K0, vec != 0);
        }
    };
    auto put = [&](int b) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            sa[b][fk + i][fr] = fa.v[i];
            sw[b][fk + i][fr] = fw.v[i];
        }
    };
    uint64_t acc[PER][PER / 2];
#pragma unroll
    for (int i = 0; i < PER; ++i)
#pragma unroll
        for (int j = 0; j < PER / 2; ++j) acc[i][j] = 0ull;
    fetch(0);
    put(0);
    __syncthreads();
    for (int s = 0; s < steps; ++s) {
        const int b = s & 1;
        if (s + 1 < steps) fetch(s + 1);
#pragma unroll
        for (int kk = 0; kk < kStep; ++kk) {
            float a[PER];
            uint64_t w[PER / 2];
#pragma unroll
            for (int i = 0; i < PER; i += 4) {   // rows tm.. and, in the larger tile, 64 further
                const float4 av = *reinterpret_cast<const float4*>(&sa[b][kk][tm + 16 * i]);
                const float4 wv = *reinterpret_cast<const float4*>(&sw[b][kk][tn + 16 * i]);
                a[i] = av.x;
                a[i + 1] = av.y;
                a[i + 2] = av.z;
                a[i + 3] = av.w;
                w[i / 2] = f2_pack(wv.x, wv.y);
                w[i / 2 + 1] = f2_pack(wv.z, wv.w);
            }
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint64_t aa = f2_pack(a[i], a[i]);
#pragma unroll
                for (int j = 0; j < PER / 2; ++j) acc[i][j] = f2_fma(aa, w[j], acc[i][j]);
            }
        }
        if (s + 1 < steps) {
            put(b ^ 1);
            __syncthreads();
        }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int m = m0 + tm + i % 4 + i / 4 * 64;
        if (m >= p.M) continue;
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int n = n0 + tn + j % 4 + j / 4 * 64;
            if (n >= p.N) continue;
            float lo, hi;
            f2_unpack(acc[i][j / 2], lo, hi);
            float v = (j & 1 ? hi : lo) + (p.bias ? p.bias[n] : 0.0f);
            if (p.act == WINO_ACT_SILU) v = activate<WINO_ACT_SILU, sizeof(TO) == 2>(v);
            if (p.act == WINO_ACT_GELU) v = activate<WINO_ACT_GELU, sizeof(TO) == 2>(v);
            const size_t at = (size_t)m * p.ldo + n;
            if (!in_bounds(at, (size_t)(p.M - 1) * p.ldo + p.N, &g_err)) continue;
            if (p.res) v += to_f32(static_cast<const TO*>(p.res)[(size_t)m * p.ldr + n]);
            if constexpr (sizeof(TO) == 2) static_cast<TO*>(p.out)[at] = __float2bfloat16_rn(v);
            else static_cast<TO*>(p.out)[at] = v;
        }
    }
}

template <typename T, typename TO, int TILE>
cudaError_t launch(const MatmulArgs& a, cudaStream_t st) {
    const long tiles = (long)((a.M + (long)TILE - 1) / TILE) * ((a.N + (long)TILE - 1) / TILE);
    if (tiles > 2147483647L) return cudaErrorInvalidConfiguration;
    const size_t es = sizeof(T), to = TILE / 16 * es < 16 ? TILE / 16 * es : 16;   // bytes of one load
    auto ok = [&](const void* p, long ld) { return reinterpret_cast<uintptr_t>(p) % to == 0 && (size_t)ld * es % to == 0; };
    const int vec = ok(a.a, a.lda) && ok(a.w, a.ldw) && (a.K1 == 0 || (ok(a.a2, a.lda2) && (size_t)a.K0 * es % to == 0));
    return launch_dependent(matmul_simt_kernel<T, TO, TILE>, dim3((unsigned)tiles), dim3(kThreads), 0, st, a, vec);
}

template <typename T, typename TO>
cudaError_t launch_tile(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    // the larger tile reads each operand half as often, but only where its tiles fill the SMs
    const long large = (long)((a.M + 127L) / 128) * ((a.N + 127L) / 128);
    return large >= num_sms ? launch<T, TO, 128>(a, st) : launch<T, TO, 64>(a, st);
}

}  // namespace

cudaError_t launch_matmul_simt(const MatmulArgs& a, int num_sms, cudaStream_t st) {
    using B = __nv_bfloat16;
    if (a.bf16) return a.out_bf16 ? launch_tile<B, B>(a, num_sms, st) : launch_tile<B, float>(a, num_sms, st);
    return a.out_bf16 ? launch_tile<float, B>(a, num_sms, st) : launch_tile<float, float>(a, num_sms, st);
}

cudaError_t matmul_simt_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
