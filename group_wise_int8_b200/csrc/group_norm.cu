// Group normalisation with an activation on NHWC activations, in one pass over
// device memory:
//   v = x + add[n][c],  mean and variance of v over the pixels and channels of
//   a group,  y = act((v - mean) / sqrt(var + eps) * gamma[c] + beta[c]).
// The channels may come from two tensors (a block input concatenated with a
// skip tensor), which are never joined in memory; a group may straddle them.
//
// Bound: device memory (x read once, y written once); per value about 10 fp32
// operations and, with SiLU, two special-function operations.
//
// Split: an image's channels are cut into slabs of whole groups, and a
// thread-block cluster of up to 16 CTAs takes one (image, slab), each CTA a
// contiguous range of pixels.  A CTA loads its part once into shared memory
// while it accumulates statistics, the cluster exchanges one (mean, M2) pair per
// group and CTA through distributed shared memory, and the CTA normalises from
// shared memory.  No workspace, no atomics, one launch; the order of every
// sum is fixed by the shape, so results repeat bit for bit.  A part that does
// not fit is kept as far as it fits and the rest is read again (mostly from L2).
//
// Statistics: a thread owns one vector of channels and strides over pixels.
// Per channel it sums d and d*d with d = x - p, p the first value it sees, so
// that a mean far from zero costs no digits, and (mean, M2) pairs are joined by
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + sum n_i (mean_i - mean)^2,
// again around one of the means.  All of it is fp32.
#include <algorithm>
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace wino {
namespace {

__device__ int g_err;   // first failed index check since group_norm_take_error (debug build)

constexpr int kThreads = 256;
constexpr int kMaxCluster = 16;
constexpr int kResBytes = 56 * 1024;   // a CTA's share kept in shared memory (three CTAs per SM)

template <typename T, int VEC>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
    using Raw = uint4;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[8]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};
template <>
struct Vec<float, 4> {
    using Raw = uint4;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[4]) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    }
};
template <>
struct Vec<__nv_bfloat16, 1> {
    using Raw = uint16_t;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[1]) { v[0] = __uint_as_float((uint32_t)r << 16); }
};
template <>
struct Vec<float, 1> {
    using Raw = uint32_t;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[1]) { v[0] = __uint_as_float(r); }
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Stores VEC values of y (vec: the address is aligned for one whole store).
template <typename TO, int VEC>
__device__ __forceinline__ void store(TO* p, const float (&v)[VEC], bool vec) {
    if constexpr (VEC == 1) {
        if constexpr (sizeof(TO) == 2) *p = __float2bfloat16_rn(v[0]);
        else *p = v[0];
    } else if (vec) {
        if constexpr (sizeof(TO) == 2) {
            if constexpr (VEC == 8)
                *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                          pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
            else
                *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
        } else {
#pragma unroll
            for (int i = 0; i < VEC; i += 4)
                *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            if constexpr (sizeof(TO) == 2) p[i] = __float2bfloat16_rn(v[i]);
            else p[i] = v[i];
        }
    }
}

// Layout of a CTA's shared memory (bytes): kept rows | per-thread (mean, M2) table | per-group
// (mean, M2) of this CTA | per-group (mean, 1/std) of the cluster.
struct Shape {
    int nv, RP, TV, nvp;
    __host__ __device__ Shape(int channels, int vec) {
        nv = channels / vec;                    // vectors per row of the slab
        TV = nv < kThreads ? nv : kThreads;     // vectors taken at a time
        RP = kThreads / TV;                     // rows taken at a time
        nvp = nv | 1;                           // table pitch: odd, so that a column read has no bank conflicts
    }
    __host__ __device__ size_t table() const { return (size_t)RP * nvp; }   // entries per vector lane
};

__device__ __forceinline__ float2 ld_cluster(const float2* p, int rank) {
    namespace cg = cooperative_groups;
    return *cg::this_cluster().map_shared_rank(p, rank);
}

template <typename TI, typename TO, int VEC>
__global__ void __launch_bounds__(kThreads) group_norm_kernel(const GroupNormArgs a) {
    namespace cg = cooperative_groups;
    using V = Vec<TI, VEC>;
    using Raw = typename V::Raw;
    constexpr bool FAST = sizeof(TO) == 2;
    extern __shared__ __align__(16) unsigned char smem[];
    const int C = a.C0 + a.C1;
    const int CS = (int)cg::this_cluster().num_blocks(), rank = (int)cg::this_cluster().block_rank();
    const long unit = (long)blockIdx.x / CS;
    const int n = (int)(unit / a.slabs), slab = (int)(unit - (long)n * a.slabs);
    const int g0 = slab * a.gps, ng = min(a.gps, a.groups - g0);
    const int ch0 = g0 * a.cg, nch = ng * a.cg;
    const Shape sh(nch, VEC);
    const int nv = sh.nv, TV = sh.TV, RP = sh.RP;
    const long row0 = a.HW * rank / CS;
    const int rows = (int)(a.HW * (rank + 1) / CS - row0);
    const int res = min(rows, a.res_rows);

    // the widest slab's sizes place the regions, so that they agree within a cluster and a launch
    const Shape full(a.gps * a.cg, VEC);
    const size_t keep_bytes = ((size_t)a.res_rows * full.nv * sizeof(Raw) + 15) / 16 * 16;
    Raw* keep = reinterpret_cast<Raw*>(smem);
    float2* table = reinterpret_cast<float2*>(smem + keep_bytes);
    float2* part = table + (size_t)VEC * max(full.table(), sh.table());
    float2* stat = part + a.gps;

    const int tid = threadIdx.x, tr = tid / TV, tv = tid - tr * TV;
    const bool active = tr < RP;
    grid_dependents_launch();
    grid_dependency_wait();

    // ---- load, keep, accumulate
    for (int vb = 0; vb < nv; vb += TV) {
        const int v = vb + tv;
        if (!active || v >= nv) continue;
        const int ch = ch0 + v * VEC;
        const bool second = ch >= a.C0;
        const long ld = second ? a.ld1 : a.ld0;
        const TI* src = (second ? static_cast<const TI*>(a.x2) + (ch - a.C0) : static_cast<const TI*>(a.x) + ch) +
                        ((long)n * a.HW + row0) * ld;
        const size_t limit = (size_t)((long)a.N * a.HW - 1) * ld + (second ? a.C1 : a.C0);   // elements of the source
        const size_t base = (size_t)((long)n * a.HW + row0) * ld + (second ? ch - a.C0 : ch);
        float p[VEC], s[VEC], q[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) p[i] = s[i] = q[i] = 0.0f;
        constexpr int U = 4;   // rows in flight per thread
        bool first = true;
        int r = tr;
        for (; r + (U - 1) * RP < rows; r += U * RP) {
            Raw raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u] = Raw{};
                if (in_bounds(base + (size_t)(r + u * RP) * ld + VEC - 1, limit, &g_err))
                    raw[u] = *reinterpret_cast<const Raw*>(src + (long)(r + u * RP) * ld);
            }
            if (first) {
                V::load(raw[0], p);
                first = false;
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float x[VEC];
                V::load(raw[u], x);
                if (r + u * RP < res) keep[(size_t)(r + u * RP) * nv + v] = raw[u];
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float d = x[i] - p[i];
                    s[i] += d;
                    q[i] = fmaf(d, d, q[i]);
                }
            }
        }
        for (; r < rows; r += RP) {
            Raw raw = Raw{};
            if (in_bounds(base + (size_t)r * ld + VEC - 1, limit, &g_err))
                raw = *reinterpret_cast<const Raw*>(src + (long)r * ld);
            float x[VEC];
            V::load(raw, x);
            if (first) {
#pragma unroll
                for (int i = 0; i < VEC; ++i) p[i] = x[i];
                first = false;
            }
            if (r < res) keep[(size_t)r * nv + v] = raw;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                const float d = x[i] - p[i];
                s[i] += d;
                q[i] = fmaf(d, d, q[i]);
            }
        }
        const int cnt = tr < rows ? (rows - tr + RP - 1) / RP : 0;
        const float inv = cnt ? 1.0f / (float)cnt : 0.0f;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float add = a.add ? a.add[(size_t)n * C + ch + i] : 0.0f;
            const float dm = s[i] * inv;
            table[(size_t)i * sh.table() + (size_t)tr * sh.nvp + v] =
                make_float2(p[i] + dm + add, fmaf(-s[i], dm, q[i]));
        }
    }
    __syncthreads();

    // ---- one warp per group: join the (mean, M2) pairs of its channels and row offsets
    const int warp = tid >> 5, lane = tid & 31;
    for (int g = warp; g < ng; g += kThreads / 32) {
        auto entry = [&](int ch, int ro) {   // channel within the slab
            return table[(size_t)(ch % VEC) * sh.table() + (size_t)ro * sh.nvp + ch / VEC];
        };
        const float pivot = entry(g * a.cg, 0).x;
        const int used = min(RP, rows);   // row offsets with at least one row
        float S = 0.0f, Q = 0.0f;
        for (int e = lane; e < a.cg * used; e += 32) {
            const int c = e / used, ro = e - c * used;
            const float2 m = entry(g * a.cg + c, ro);
            const float cnt = (float)((rows - ro + RP - 1) / RP), d = m.x - pivot;
            S = fmaf(cnt, d, S);
            Q += fmaf(cnt * d, d, m.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            S += __shfl_xor_sync(0xffffffffu, S, o);
            Q += __shfl_xor_sync(0xffffffffu, Q, o);
        }
        if (lane == 0) {
            const float cnt = (float)rows * (float)a.cg, dm = rows ? S / cnt : 0.0f;
            part[g] = make_float2(rows ? pivot + dm : 0.0f, fmaf(-S, dm, Q));
        }
    }
    if (CS > 1) cg::this_cluster().sync();
    else __syncthreads();

    // ---- join the CTAs' pairs in rank order
    for (int g = tid; g < ng; g += kThreads) {
        const float pivot = (CS > 1 ? ld_cluster(&part[g], 0) : part[g]).x;
        float S = 0.0f, Q = 0.0f;
        for (int k = 0; k < CS; ++k) {
            const float2 m = CS > 1 ? ld_cluster(&part[g], k) : part[g];
            const float cnt = (float)(a.HW * (k + 1) / CS - a.HW * k / CS) * (float)a.cg, d = m.x - pivot;
            S = fmaf(cnt, d, S);
            Q += fmaf(cnt * d, d, m.y);
        }
        const float cnt = (float)a.HW * (float)a.cg, dm = S / cnt;
        float var = fmaf(-S, dm, Q) / cnt;
        var = var < 0.0f ? 0.0f : var;   // rounding only; a NaN stays
        stat[g] = make_float2(pivot + dm, 1.0f / sqrtf(var + a.eps));
    }
    __syncthreads();
    // this CTA has read the others' pairs; it leaves only when they have read its own (waited for at the end)
    if (CS > 1) asm volatile("barrier.cluster.arrive.release;" ::: "memory");

    // ---- normalise, activate, store
    TO* y = static_cast<TO*>(a.y);
    for (int vb = 0; vb < nv; vb += TV) {
        const int v = vb + tv;
        if (!active || v >= nv) continue;
        const int ch = ch0 + v * VEC;
        const bool second = ch >= a.C0;
        const long ld = second ? a.ld1 : a.ld0;
        const TI* src = (second ? static_cast<const TI*>(a.x2) + (ch - a.C0) : static_cast<const TI*>(a.x) + ch) +
                        ((long)n * a.HW + row0) * ld;
        float m[VEC], A[VEC], B[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float2 st = stat[(v * VEC + i) / a.cg];
            m[i] = a.add ? st.x - a.add[(size_t)n * C + ch + i] : st.x;
            A[i] = st.y * (a.gamma ? a.gamma[ch + i] : 1.0f);
            B[i] = a.beta ? a.beta[ch + i] : 0.0f;
        }
        const size_t ybase = (size_t)((long)n * a.HW + row0) * a.ldy + ch;
        const size_t ylimit = (size_t)((long)a.N * a.HW - 1) * a.ldy + C;
#pragma unroll 2
        for (int r = tr; r < rows; r += RP) {
            const Raw raw = r < res ? keep[(size_t)r * nv + v] : *reinterpret_cast<const Raw*>(src + (long)r * ld);
            float x[VEC], o[VEC];
            V::load(raw, x);
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = activate<FAST>(fmaf(x[i] - m[i], A[i], B[i]), a.act);
            const size_t yi = ybase + (size_t)r * a.ldy;
            if (in_bounds(yi + VEC - 1, ylimit, &g_err)) store<TO, VEC>(y + yi, o, a.vec_y != 0);
        }
    }
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Shared memory of a CTA beside its kept rows.
size_t table_bytes(int groups, int cg, int gps, int vec) {
    // a narrower last slab has more row offsets, so its table can be larger
    const int last = groups - (groups - 1) / gps * gps;
    const size_t table = std::max(Shape(gps * cg, vec).table(), Shape(last * cg, vec).table());
    return sizeof(float2) * (vec * table + 2 * (size_t)gps);
}

size_t smem_bytes(const GroupNormArgs& a, int vec, int es) {
    return ((size_t)a.res_rows * a.gps * a.cg * es + 15) / 16 * 16 + table_bytes(a.groups, a.cg, a.gps, vec);
}

template <typename TI, typename TO, int VEC>
cudaError_t launch(const GroupNormArgs& a, int cluster, cudaStream_t st) {
    static bool done[64], done_cluster[64];
    auto kern = group_norm_kernel<TI, TO, VEC>;
    const size_t smem = smem_bytes(a, VEC, (int)sizeof(TI));
    cudaError_t e = allow_smem(kern, 227 * 1024, done);
    if (e != cudaSuccess) return e;
    if (cluster > 8) {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64 || !done_cluster[dev]) {
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) done_cluster[dev] = true;
        }
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((long)a.N * a.slabs * cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kern, a);
}

template <typename TI, typename TO>
cudaError_t launch_vec(const GroupNormArgs& a, bool vec, int cluster, cudaStream_t st) {
    constexpr int VEC = 16 / (int)sizeof(TI);
    return vec ? launch<TI, TO, VEC>(a, cluster, st) : launch<TI, TO, 1>(a, cluster, st);
}

bool aligned(const void* p, long ld_bytes, size_t to) {
    return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (size_t)ld_bytes % to == 0;
}

}  // namespace

// The widest slab (long contiguous runs) and the smallest cluster whose CTAs' shares fit in shared
// memory and that make two CTAs per SM; when no split does both, the one with the smallest share.
GroupNormSplit group_norm_split(const GroupNormArgs& a, int vec, int num_sms) {
    const int cg = (a.C0 + a.C1) / a.groups, es = a.x_bf16 ? 2 : 4;
    const int unit = std::min(a.groups, vec / gcd(cg, vec));   // groups of the narrowest slab of whole vectors
    const int units = (a.groups + unit - 1) / unit;
    GroupNormSplit best = {a.groups, 1};
    double best_bytes = 0;
    for (int s = 1; s <= units; ++s) {
        const int per = (units + s - 1) / s;
        if (s > 1 && per == (units + s - 2) / (s - 1)) continue;   // the same slabs
        const int gps = std::min(a.groups, per * unit);
        if (gps > unit && table_bytes(a.groups, cg, gps, vec) > 64 * 1024) continue;
        for (int c = 1; c <= kMaxCluster; c *= 2) {
            if (c > 1 && c > a.HW) break;
            const double bytes = (double)((a.HW + c - 1) / c) * gps * cg * es;
            const long ctas = (long)a.N * ((a.groups + gps - 1) / gps) * c;
            if (bytes <= kResBytes && (ctas >= 2 * num_sms || bytes <= 8 * 1024)) return {gps, c};
            if (best_bytes == 0 || bytes < best_bytes) {
                best_bytes = bytes;
                best = {gps, c};
            }
        }
    }
    return best;
}

cudaError_t launch_group_norm(GroupNormArgs a, int num_sms, const GroupNormSplit* split, cudaStream_t st) {
    const int C = a.C0 + a.C1, es = a.x_bf16 ? 2 : 4, eo = a.y_bf16 ? 2 : 4, VEC = 16 / es;
    a.cg = C / a.groups;
    const bool vec = C % VEC == 0 && a.C0 % VEC == 0 && aligned(a.x, a.ld0 * es, 16) &&
                     (a.C1 == 0 || aligned(a.x2, a.ld1 * es, 16));
    const size_t out_vec = (size_t)std::min(16, VEC * eo);
    a.vec_y = aligned(a.y, a.ldy * eo, out_vec) ? 1 : 0;
    const GroupNormSplit s = split ? *split : group_norm_split(a, vec ? VEC : 1, num_sms);
    a.gps = s.gps;
    a.slabs = (a.groups + s.gps - 1) / s.gps;
    const long share = (a.HW + s.cluster - 1) / s.cluster;
    a.res_rows = (int)std::min<long>(share, kResBytes / ((long)a.gps * a.cg * es));
    if (smem_bytes(a, vec ? VEC : 1, es) > 227 * 1024 || (double)a.N * a.slabs * s.cluster > 2147483647.0)
        return cudaErrorInvalidConfiguration;
    if (a.x_bf16)
        return a.y_bf16 ? launch_vec<__nv_bfloat16, __nv_bfloat16>(a, vec, s.cluster, st)
                        : launch_vec<__nv_bfloat16, float>(a, vec, s.cluster, st);
    return a.y_bf16 ? launch_vec<float, __nv_bfloat16>(a, vec, s.cluster, st)
                    : launch_vec<float, float>(a, vec, s.cluster, st);
}

cudaError_t group_norm_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
