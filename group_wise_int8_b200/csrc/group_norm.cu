// Group normalisation with an activation on NHWC activations, in one pass over
// device memory:
//   v = x + add[n][c],  mean and variance of v over the pixels and channels of
//   a group,  y = act((v - mean) / sqrt(var + eps) * gamma[c] + beta[c]).
// The channels may come from two tensors (a block input concatenated with a
// skip tensor), which are never joined in memory; a group may straddle them.
//
// Bound: device memory (x read once, y written once); per value about 10 fp32
// operations and, with SiLU, 1.25 special-function operations.  As built, 8 x 64 x 64 x 320 bf16 with SiLU takes 14.9 us
// where its 42 MB take 6.4 at the copy rate: 8.5 us of issue slots on the 128 SMs that the split uses (26 instructions
// per value, 19 of them in the two row loops), and as much again of latency between the phases, in which the schedulers
// issue nothing half of the time.  8 x 64 x 64 x 960 48.8 (19.2); 2 x 32 x 32 x 640 fp32 6.1 (1.6).
//
// Split: an image's channels are cut into slabs of whole groups, and a
// thread-block cluster of up to 16 CTAs takes one (image, slab), each CTA a
// contiguous range of pixels.  A CTA loads its part once into shared memory
// while it accumulates statistics, the cluster exchanges one (mean, M2) pair per
// group and CTA by writing it into every CTA's shared memory, and the CTA normalises from
// shared memory.  No workspace, no atomics, one launch; the order of every
// sum is fixed by the shape, so results repeat bit for bit.  A part that does
// not fit is kept as far as it fits and the rest is read again (mostly from L2).
//
// Statistics: a thread owns one vector of channels and strides over pixels.
// Per channel it sums d and d*d with d = x - p, p the first value it sees, so
// that a mean far from zero costs no digits.  Every kBlock rows (more than are kept) the pivot moves to the mean of the
// rows so far: around a first value far from the rest, thousands of equal squares would be summed, of
// which M2 is the small difference.  (mean, M2) pairs are joined by
//   mean = sum n_i mean_i / n,  M2 = sum M2_i + sum n_i (mean_i - mean)^2:
// a channel's pairs around one of their means, the channels of a group and the CTAs of a cluster (whose
// means may lie far apart) with the joint mean first.  All of it is fp32; M2 never falls below zero but by rounding.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "group_norm_split.h"
#include "kernels.h"
#include "ops.h"
#include "sm100.cuh"

namespace wino {
namespace {

using namespace group_norm;

__device__ int g_err;   // first failed index check since group_norm_take_error (debug build)

constexpr int kBlock = 64;   // rows between two recentrings of a thread's sums (more than are ever kept)

// A thread's VEC consecutive values: 16 bytes, or one value where alignment allows no more.
template <typename T, int VEC>
struct Vec {
    using Raw = uint4;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[VEC]) {
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
};
template <typename T>
struct Vec<T, 1> {
    using Raw = typename std::conditional<sizeof(T) == 2, uint16_t, uint32_t>::type;
    static __device__ __forceinline__ void load(const Raw& r, float (&v)[1]) {
        v[0] = __uint_as_float(sizeof(T) == 2 ? (uint32_t)r << 16 : (uint32_t)r);
    }
};

// Running sums of d and d * d, d = x - p, of VEC channels (packed pairs where VEC is even).
template <int VEC>
struct Sums {
    static constexpr int kPairs = VEC / 2;
    using Part = uint64_t;
    uint64_t p[kPairs], s[kPairs], q[kPairs];
    __device__ __forceinline__ void start(const float (&x)[VEC]) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            p[i] = f2_pack(x[2 * i], x[2 * i + 1]);
            s[i] = q[i] = 0ull;
        }
    }
    __device__ __forceinline__ void add(const float (&x)[VEC]) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint64_t d = f2_sub(f2_pack(x[2 * i], x[2 * i + 1]), p[i]);
            s[i] = f2_add(s[i], d);
            q[i] = f2_fma(d, d, q[i]);
        }
    }
    // Moves the pivot to the mean of the `rows` values so far; their squares go to `whole`.  (The sums follow the
    // pivot's actual step, so neither its rounding nor 1 / rows needs to be exact.)
    __device__ __forceinline__ void recentre(float rows, uint64_t (&whole)[kPairs]) {
        const uint64_t n = f2_pack(-rows, -rows), r = f2_pack(reciprocal(rows), reciprocal(rows));
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const uint64_t to = f2_fma(s[i], r, p[i]), step = f2_sub(to, p[i]), left = f2_fma(n, step, s[i]);
            whole[i] = f2_add(whole[i], f2_sub(q[i], f2_mul(step, f2_add(s[i], left))));
            p[i] = to;
            s[i] = left;
            q[i] = 0ull;
        }
    }
    __device__ __forceinline__ void join(const uint64_t (&whole)[kPairs]) {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) q[i] = f2_add(q[i], whole[i]);
    }
    __device__ __forceinline__ void get(float (&pv)[VEC], float (&sv)[VEC], float (&qv)[VEC]) const {
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            f2_unpack(p[i], pv[2 * i], pv[2 * i + 1]);
            f2_unpack(s[i], sv[2 * i], sv[2 * i + 1]);
            f2_unpack(q[i], qv[2 * i], qv[2 * i + 1]);
        }
    }
};
template <>
struct Sums<1> {
    static constexpr int kPairs = 1;
    using Part = float;
    float p, s, q;
    __device__ __forceinline__ void start(const float (&x)[1]) {
        p = x[0];
        s = q = 0.0f;
    }
    __device__ __forceinline__ void add(const float (&x)[1]) {
        const float d = x[0] - p;
        s += d;
        q = fmaf(d, d, q);
    }
    __device__ __forceinline__ void recentre(float rows, float (&whole)[kPairs]) {
        const float to = fmaf(s, reciprocal(rows), p), step = to - p, left = fmaf(-rows, step, s);
        whole[0] += q - step * (s + left);
        p = to;
        s = left;
        q = 0.0f;
    }
    __device__ __forceinline__ void join(const float (&whole)[kPairs]) { q += whole[0]; }
    __device__ __forceinline__ void get(float (&pv)[1], float (&sv)[1], float (&qv)[1]) const {
        pv[0] = p;
        sv[0] = s;
        qv[0] = q;
    }
};

// 16 bytes global -> shared without a register (counted in this thread's cp.async groups).
__device__ __forceinline__ void copy_async(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy_async4(float* dst, const float* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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

// A thread's vector of a pixel: where it starts in its source, and the source's end (in elements).
template <typename TI>
struct Source {
    const TI* p;
    long ld;
    size_t base, limit;
    __device__ __forceinline__ Source(const GroupNormArgs& a, long pixel, int ch) {
        const bool second = ch >= a.C0;
        ld = second ? a.ld1 : a.ld0;
        base = (size_t)pixel * ld + (second ? ch - a.C0 : ch);
        limit = (size_t)((long)a.N * a.HW - 1) * ld + (second ? a.C1 : a.C0);
        p = static_cast<const TI*>(second ? a.x2 : a.x) + base;
    }
};

// Stores to the same shared variable of another CTA of the cluster.
__device__ __forceinline__ void st_cluster(float2* p, int rank, float2 v) {
    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(sm100::map_rank(p, (uint32_t)rank)), "f"(v.x), "f"(v.y)
                 : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

template <typename TI, typename TO, int VEC, int ACT>
__global__ void __launch_bounds__(kThreads, 2) group_norm_kernel(const GroupNormArgs a, const Split k) {
    using V = Vec<TI, VEC>;
    using Raw = typename V::Raw;
    constexpr bool FAST = sizeof(TO) == 2;
    extern __shared__ __align__(16) unsigned char smem[];
    const int C = a.C0 + a.C1;
    const int CS = k.cluster, rank = (int)blockIdx.x & (CS - 1), slab = (int)(blockIdx.x >> k.log_cluster);
    const int n = (int)(blockIdx.z * gridDim.y + blockIdx.y);
    if (n >= a.N) return;   // (a whole cluster)
    if (CS > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");   // (waited for before the exchange)
    const int ch0 = slab * k.nch, nv = k.nv, RP = k.RP, entries = k.entries;
    const int x = rank < k.extra ? 1 : 0;
    const int rows = k.share + x;
    const long row0 = (long)n * a.HW + (long)rank * k.share + min(rank, k.extra);   // first pixel, over all images
    // (selected, not indexed: an index would put the parameters in local memory)
    const int fewer = x ? k.fewer[1] : k.fewer[0], more = x ? k.more[1] : k.more[0];
    const float inv0 = x ? k.inv0[1] : k.inv0[0], inv1 = x ? k.inv1[1] : k.inv1[0];
    const float inv_rows = x ? k.inv_rows[1] : k.inv_rows[0];
    const float cnt0 = (float)fewer, cnt1 = (float)(fewer + 1);
    const bool whole = rows <= k.res_rows;

    // kept rows | (mean, M2) of each row offset and channel | of each CTA and group | (mean, 1/std) of each group
    // | the slab's parameters
    Raw* keep = reinterpret_cast<Raw*>(smem);
    float2* table = reinterpret_cast<float2*>(smem + k.keep_bytes);
    float2* part = table + VEC * entries;
    float2* stat = part + CS * k.gps;
    float* prm = reinterpret_cast<float*>(smem + k.prm_at);

    const int tid = threadIdx.x, tr = (int)(((uint32_t)tid * k.inv_tv) >> 20), tv = tid - tr * k.TV;
    const bool active = tr < RP;
    const int mine = tr < more ? fewer + 1 : fewer;          // this thread's rows per vector
    const int kept = VEC > 1 ? (whole ? mine : k.res_per) : 0;   // of them kept by an asynchronous copy
    grid_dependents_launch();
    grid_dependency_wait();

    // ---- load, keep, accumulate
    // the slab's parameters, as [add, gamma, beta][channel]; later [mean - add, gamma / std, beta]
    // (a slab too wide for that reads them where they are)
    for (int c = tid; c < k.nprm; c += kThreads) {
        if (a.add) copy_async4(prm + c, a.add + (size_t)n * C + ch0 + c);
        else prm[c] = 0.0f;
        if (a.gamma) copy_async4(prm + k.nch + c, a.gamma + ch0 + c);
        else prm[k.nch + c] = 1.0f;
        if (a.beta) copy_async4(prm + 2 * k.nch + c, a.beta + ch0 + c);
        else prm[2 * k.nch + c] = 0.0f;
    }
    for (int vb = 0; vb < nv; vb += k.TV) {
        const int v = vb + tv;
        if (!active || v >= nv) continue;
        const Source<TI> src(a, row0 + tr, ch0 + v * VEC);
        const long step = (long)RP * src.ld;
        Sums<VEC> sums;
        float e[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) e[i] = 0.0f;
        sums.start(e);
        const TI* from = src.p;
        if constexpr (VEC > 1) {
            // every kept row's copy is under way before the first is read; a thread reads only what it copied
            constexpr int kParts = 4;
            const int per = (kept + kParts - 1) / kParts;
            Raw* to = keep + tr * nv + v;
            int i = 0;
#pragma unroll
            for (int q = 0; q < kParts; ++q) {
                for (const int end = min(kept, (q + 1) * per); i < end; ++i) {
                    if (in_bounds(src.base + (size_t)i * step + VEC - 1, src.limit, &g_err)) copy_async(to, from);
                    from += step;
                    to += RP * nv;
                }
                copy_commit();
            }
        }
        if constexpr (VEC > 1) {
            constexpr int kParts = 4;
            const int per = (kept + kParts - 1) / kParts;
            const Raw* own = keep + tr * nv + v;
            int i = 0;
            auto take = [&](int q) {
                const int end = min(kept, (q + 1) * per);
                if (q == 0 && kept > 0) {
                    V::load(*own, e);
                    sums.start(e);
                }
#pragma unroll 4
                for (; i < end; ++i) {
                    V::load(*own, e);
                    sums.add(e);
                    own += RP * nv;
                }
            };
            copy_wait<3>();
            take(0);
            copy_wait<2>();
            take(1);
            copy_wait<1>();
            take(2);
            copy_wait<0>();
            take(3);
        }
        // rows that are not kept (or, one value at a time, every row)
        auto fetch = [&](int i) {
            Raw raw = Raw{};
            if (in_bounds(src.base + (size_t)i * step + VEC - 1, src.limit, &g_err))
                raw = *reinterpret_cast<const Raw*>(src.p + (long)i * step);
            return raw;
        };
        if (kept == 0 && mine > 0) {
            V::load(fetch(0), e);
            sums.start(e);
        }
        auto read = [&](int i) {
            const Raw raw = fetch(i);
            if (VEC == 1 && (whole || i < k.res_per)) keep[(tr + i * RP) * nv + v] = raw;
            V::load(raw, e);
            sums.add(e);
        };
#pragma unroll 4
        for (int i = kept; i < min(mine, kBlock); ++i) read(i);
        if (mine > kBlock) {
            typename Sums<VEC>::Part squares[Sums<VEC>::kPairs] = {};   // of the rows before the last recentring
            for (int i = kBlock; i < mine;) {
                sums.recentre((float)i, squares);
                const int end = min(i + kBlock, mine);
#pragma unroll 4
                for (; i < end; ++i) read(i);
            }
            sums.join(squares);
        }
        const float inv = tr < more ? inv1 : inv0;
        float p[VEC], sum[VEC], q[VEC];
        sums.get(p, sum, q);
        float2* t = table + tr * k.nvp + v;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const float dm = sum[i] * inv;
            t[i * entries] = make_float2(p[i] + dm, fmaf(-sum[i], dm, q[i]));
        }
    }
    sm100::copy_wait_all();   // (a thread without rows, or of the one-value path, has copied parameters outside any group)
    __syncthreads();

    // ---- join the row offsets of each channel: `lanes` lanes of a warp per channel
    const int warp = tid >> 5, lane = tid & 31;
    {
        const int P = 1 << k.log_lanes, used = min(RP, rows);   // row offsets with at least one row
        for (int base = 0; base < k.nch; base += kThreads >> k.log_lanes) {
            const int c = base + (tid >> k.log_lanes), sub = tid & (P - 1);
            float2* col = table + (int)((unsigned)c % VEC) * entries + (int)((unsigned)c / VEC);
            float S = 0.0f, Q = 0.0f, pivot = 0.0f;
            if (c < k.nch) {
                pivot = col->x;
#pragma unroll 4
                for (int ro = sub; ro < used; ro += P) {
                    const float2 m = col[ro * k.nvp];
                    const float cnt = ro < more ? cnt1 : cnt0, d = m.x - pivot;
                    S = fmaf(cnt, d, S);
                    Q += fmaf(cnt * d, d, m.y);
                }
            }
            for (int o = P >> 1; o > 0; o >>= 1) {
                S += __shfl_xor_sync(0xffffffffu, S, o);
                Q += __shfl_xor_sync(0xffffffffu, Q, o);
            }
            if (c < k.nch && sub == 0) {   // into the channel's first entry, which its lanes have read
                const float dm = S * inv_rows;
                const float add = k.nprm ? prm[c] : (a.add ? a.add[(size_t)n * C + ch0 + c] : 0.0f);
                *col = make_float2(pivot + dm + add, fmaf(-S, dm, Q));   // (the addend moves the mean alone)
            }
        }
    }
    __syncthreads();

    // every CTA of the cluster has started: its shared memory may be written
    if (CS > 1) asm volatile("barrier.cluster.wait.acquire;" ::: "memory");

    // ---- join the channels of each group, each with `rows` values: one warp per group, the mean first
    for (int g = warp; g < k.gps; g += kThreads / 32) {
        auto channel = [&](int c) {
            c += g * k.cg;
            return table[(int)((unsigned)c % VEC) * entries + (int)((unsigned)c / VEC)];
        };
        const float2 own = lane < k.cg ? channel(lane) : make_float2(0.0f, 0.0f);
        const float pivot = __shfl_sync(0xffffffffu, own.x, 0);
        float S = lane < k.cg ? own.x - pivot : 0.0f;
        for (int c = lane + 32; c < k.cg; c += 32) S += channel(c).x - pivot;
        const float m = pivot + warp_sum(S) * k.inv_cg_f;
        float d = own.x - m, Q = lane < k.cg ? fmaf((float)rows * d, d, own.y) : 0.0f;
        for (int c = lane + 32; c < k.cg; c += 32) {
            const float2 o = channel(c);
            d = o.x - m;
            Q += fmaf((float)rows * d, d, o.y);
        }
        Q = warp_sum(Q);
        // to every CTA of the cluster
        if (lane < CS) st_cluster(&part[rank * k.gps + g], lane, rows ? make_float2(m, Q) : make_float2(0.0f, 0.0f));
    }
    if (CS > 1) sm100::cluster_sync();
    else __syncthreads();

    // ---- join the CTAs' pairs: one lane per (group, CTA)
    for (int base = 0; base < k.gps; base += kThreads >> k.log_cluster) {
        const int g = base + (tid >> k.log_cluster), r = tid & (CS - 1);
        const bool on = g < k.gps;
        float2 m = make_float2(0.0f, 0.0f);
        if (on) m = part[r * k.gps + g];
        const float pivot = __shfl_sync(0xffffffffu, m.x, lane & ~(CS - 1));   // the first CTA's mean
        const float cnt = (float)(k.share + (r < k.extra ? 1 : 0)) * (float)k.cg;
        float S = cnt * (m.x - pivot);
        for (int o = CS >> 1; o > 0; o >>= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
        const float mean = fmaf(S, k.inv_all, pivot), d = m.x - mean;
        float Q = fmaf(cnt * d, d, m.y);
        for (int o = CS >> 1; o > 0; o >>= 1) Q += __shfl_xor_sync(0xffffffffu, Q, o);
        if (on && r == 0) stat[g] = make_float2(mean, 1.0f / sqrtf(fmaf(Q, k.inv_all, a.eps)));
    }
    __syncthreads();
    for (int c = tid; c < k.nprm; c += kThreads) {
        const float2 st = stat[k.inv_cg ? (int)__umulhi((uint32_t)c, k.inv_cg) : c];
        prm[c] = st.x - prm[c];
        prm[k.nch + c] *= st.y;
    }
    __syncthreads();

    // ---- normalise, activate, store
    TO* y = static_cast<TO*>(a.y);
    for (int vb = 0; vb < nv; vb += k.TV) {
        const int v = vb + tv;
        if (!active || v >= nv) continue;
        const int ch = ch0 + v * VEC;
        float m[VEC], gamma[VEC], beta[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            const int c = v * VEC + i;
            if (k.nprm) {
                m[i] = prm[c];
                gamma[i] = prm[k.nch + c];
                beta[i] = prm[2 * k.nch + c];
            } else {
                const float2 st = stat[k.inv_cg ? (int)__umulhi((uint32_t)c, k.inv_cg) : c];
                m[i] = a.add ? st.x - a.add[(size_t)n * C + ch + i] : st.x;
                gamma[i] = a.gamma ? a.gamma[ch + i] * st.y : st.y;
                beta[i] = a.beta ? a.beta[ch + i] : 0.0f;
            }
        }
        const size_t ybase = (size_t)(row0 + tr) * a.ldy + ch, ystep = (size_t)RP * a.ldy;
        const size_t ylimit = (size_t)((long)a.N * a.HW - 1) * a.ldy + C;
        auto finish = [&](const Raw& raw, int i) {
            float o[VEC];
            V::load(raw, o);
            if constexpr (VEC > 1) {
#pragma unroll
                for (int j = 0; j < VEC; j += 2)
                    f2_unpack(f2_fma(f2_sub(f2_pack(o[j], o[j + 1]), f2_pack(m[j], m[j + 1])), f2_pack(gamma[j], gamma[j + 1]),
                                     f2_pack(beta[j], beta[j + 1])),
                              o[j], o[j + 1]);
            } else {
                o[0] = fmaf(o[0] - m[0], gamma[0], beta[0]);
            }
            activate_all<ACT, FAST>(o);
            const size_t yi = ybase + (size_t)i * ystep;
            if (in_bounds(yi + VEC - 1, ylimit, &g_err)) store<TO, VEC>(y + yi, o, k.vec_y);
        };
        const int held = whole ? mine : k.res_per;
        const Raw* own = keep + tr * nv + v;
        int i = 0;
#pragma unroll 1   // (a row's eight values are independent work enough; two rows would not fit in registers)
        for (; i < held; ++i) finish(own[i * RP * nv], i);
        if (held < mine) {
            const Source<TI> src(a, row0 + tr, ch);
            const long step = (long)RP * src.ld;
#pragma unroll 4
            for (i = held; i < mine; ++i) finish(*reinterpret_cast<const Raw*>(src.p + (long)i * step), i);
        }
    }
}

template <typename TI, typename TO, int VEC, int ACT>
cudaError_t launch(const GroupNormArgs& a, const Split& k, size_t smem, cudaStream_t st) {
    static bool done[64], done_cluster[64];
    auto kern = group_norm_kernel<TI, TO, VEC, ACT>;
    cudaError_t e = allow_smem(kern, kMaxSmem, done);
    if (e != cudaSuccess) return e;
    if (k.cluster > 8) {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64 || !done_cluster[dev]) {
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
            if (dev >= 0 && dev < 64) done_cluster[dev] = true;
        }
    }
    constexpr int kMaxY = 65535;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(k.slabs * k.cluster), (unsigned)std::min(a.N, kMaxY), (unsigned)((a.N + (long)kMaxY - 1) / kMaxY));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)k.cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = k.cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, a, k);
}

template <typename TI, typename TO, int VEC>
cudaError_t launch_act(const GroupNormArgs& a, const Split& k, size_t smem, cudaStream_t st) {
    switch (a.act) {
        case WINO_ACT_SILU: return launch<TI, TO, VEC, WINO_ACT_SILU>(a, k, smem, st);
        case WINO_ACT_GELU: return launch<TI, TO, VEC, WINO_ACT_GELU>(a, k, smem, st);
        default: return launch<TI, TO, VEC, WINO_ACT_NONE>(a, k, smem, st);
    }
}

template <typename TI, typename TO>
cudaError_t launch_vec(const GroupNormArgs& a, bool vec, const Split& k, size_t smem, cudaStream_t st) {
    return vec ? launch_act<TI, TO, 16 / (int)sizeof(TI)>(a, k, smem, st) : launch_act<TI, TO, 1>(a, k, smem, st);
}

bool aligned(const void* p, long ld_bytes, size_t to) {
    return (reinterpret_cast<uintptr_t>(p) % to) == 0 && (size_t)ld_bytes % to == 0;
}

}  // namespace

cudaError_t launch_group_norm(const GroupNormArgs& a, int num_sms, cudaStream_t st) {
    const int C = a.C0 + a.C1, es = a.x_bf16 ? 2 : 4, eo = a.y_bf16 ? 2 : 4, VEC = 16 / es;
    const bool vec = C % VEC == 0 && a.C0 % VEC == 0 && aligned(a.x, a.ld0 * es, 16) &&
                     (a.C1 == 0 || aligned(a.x2, a.ld1 * es, 16));
    const GroupNormShape shape = {a.HW, a.N, C, a.groups, es};
    const GroupNormSplit s = choose(shape, vec ? VEC : 1, num_sms);
    Split k;
    const size_t smem = make_split(shape, vec ? VEC : 1, s, &k);
    if (smem > kMaxSmem || a.N > 1000000000) return cudaErrorInvalidConfiguration;
    k.vec_y = aligned(a.y, a.ldy * eo, (size_t)std::min(16, VEC * eo));
    if (a.x_bf16)
        return a.y_bf16 ? launch_vec<__nv_bfloat16, __nv_bfloat16>(a, vec, k, smem, st)
                        : launch_vec<__nv_bfloat16, float>(a, vec, k, smem, st);
    return a.y_bf16 ? launch_vec<float, __nv_bfloat16>(a, vec, k, smem, st)
                    : launch_vec<float, float>(a, vec, k, smem, st);
}

cudaError_t group_norm_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
