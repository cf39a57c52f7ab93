// How a group norm call is cut into thread-block clusters: plain host arithmetic, apart from the kernel so that CPU tests
// reach it.
#pragma once
#include <algorithm>
#include <cstddef>
#include <cstdint>

namespace wino {

// What the split depends on.
struct GroupNormShape {
    long HW;
    int N, C, groups, es;   // es: bytes of an input value
};

// How a call is cut: a cluster of `cluster` CTAs per (image, slab of `gps` groups).
struct GroupNormSplit {
    int gps, cluster;
};

namespace group_norm {

constexpr int kThreads = 256;          // two CTAs per SM, with registers for a vector's parameters
constexpr int kMaxCluster = 16;
constexpr int kMaxParams = 2048;       // channels whose parameters fit in shared memory
constexpr int kResBytes = 90 * 1024;   // a CTA's share of the input kept in shared memory
constexpr size_t kMaxSmem = 227 * 1024;   // of a CTA

// What the kernel needs to know of its split, worked out once on the host.  A row offset is a thread's first row
// within its CTA's pixels; it takes every RP-th row from there.  Index 1 of a pair: the first `extra` CTAs of a
// cluster, which take one row more.
struct Split {
    int cluster, slabs, gps;      // CTAs per (image, slab); slabs per image; groups per slab
    int nch, nv;                  // channels and vectors of a slab's row
    int TV, RP;                   // vectors taken at a time; row offsets
    int nvp, entries;             // table pitch (odd: no bank conflicts down a column); table entries per lane of a vector
    uint32_t inv_tv;              // ceil(2^20 / TV): tid / TV = tid * inv_tv >> 20 for tid < 512
    uint32_t inv_cg;              // ceil(2^32 / cg): channel / cg = umulhi(channel, inv_cg) for channel < 2^14 (0: cg = 1)
    int cg;
    int log_cluster, log_lanes;   // log2 of cluster and of the lanes of a warp that join one channel
    int share, extra;             // rows per CTA
    int res_rows, res_per;        // rows kept in shared memory when not all are (a multiple of RP); those of one offset
    int fewer[2], more[2];        // an offset has `fewer` rows, the first `more` offsets one more
    float inv0[2], inv1[2];       // 1 / fewer (0 when none), 1 / (fewer + 1)
    float inv_rows[2];            // 1 / rows (0 when none)
    float inv_cg_f, inv_all;      // 1 / cg, 1 / (HW cg)
    int keep_bytes, prm_at, nprm; // bytes of the kept rows; where the parameters start; their channels (0: not kept)
    bool vec_y;                   // y takes whole-vector stores
};

inline int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Fills in what does not depend on pointers; the shared memory that the split needs.
inline size_t make_split(const GroupNormShape& a, int vec, const GroupNormSplit& s, Split* out) {
    Split k = {};
    k.cg = a.C / a.groups;
    k.gps = s.gps;
    k.cluster = s.cluster;
    k.slabs = a.groups / s.gps;
    k.nch = k.gps * k.cg;
    k.nv = k.nch / vec;
    k.TV = std::min(k.nv, kThreads);
    k.RP = kThreads / k.TV;
    k.nvp = k.nv | 1;
    k.entries = k.RP * k.nvp;
    k.inv_tv = ((1u << 20) + k.TV - 1) / k.TV;
    k.inv_cg = k.cg == 1 ? 0u : (uint32_t)(((1ull << 32) + k.cg - 1) / k.cg);
    while ((1 << k.log_cluster) < s.cluster) ++k.log_cluster;
    while (k.log_lanes < 5 && (2 << k.log_lanes) * (long)k.nch <= kThreads && (2 << k.log_lanes) <= k.RP) ++k.log_lanes;
    k.share = (int)(a.HW / s.cluster);
    k.extra = (int)(a.HW - (long)k.share * s.cluster);
    const int most = k.share + (k.extra ? 1 : 0);
    for (int x = 0; x < 2; ++x) {
        const int rows = k.share + x;
        k.fewer[x] = rows / k.RP;
        k.more[x] = rows - k.fewer[x] * k.RP;
        k.inv0[x] = k.fewer[x] ? 1.0f / (float)k.fewer[x] : 0.0f;
        k.inv1[x] = 1.0f / (float)(k.fewer[x] + 1);
        k.inv_rows[x] = rows ? 1.0f / (float)rows : 0.0f;
    }
    k.inv_cg_f = 1.0f / (float)k.cg;
    k.inv_all = (float)(1.0 / ((double)a.HW * k.cg));
    const long row_bytes = (long)k.nch * a.es;
    if (most * row_bytes <= kResBytes) {
        k.res_rows = most;
    } else {
        k.res_per = (int)(kResBytes / row_bytes / k.RP);
        k.res_rows = k.res_per * k.RP;
    }
    k.keep_bytes = (int)((k.res_rows * row_bytes + 15) / 16 * 16);
    const size_t prm_at =
        ((size_t)k.keep_bytes + 2 * sizeof(float) * ((size_t)vec * k.entries + (size_t)(s.cluster + 1) * k.gps) + 15) / 16 * 16;
    k.prm_at = (int)prm_at;
    k.nprm = k.nch <= kMaxParams ? k.nch : 0;
    if (out) *out = k;
    return prm_at + 3 * sizeof(float) * (size_t)k.nprm;
}

// The split with the least estimated time, in us: rounds of two CTAs per SM, each a fixed part (launch, joins, exchange)
// plus its share of the input.  The constants are a fit to every split of 75 shapes (8 x 8 to 256 x 256 pixels, 32 to 2560
// channels, batches of 1 to 16): its choice took 0.9 % more time than the best split on average and 6 % at most.  8 x 64 x 64 x 320
// bf16 with SiLU, for one, took 16.4 there in clusters of 8 CTAs of 82 KiB, 17.3 in clusters of 4 of as many bytes (rows of
// 80 bytes, not 160) and 21.0 as 512 CTAs of 41 KiB; 8 x 32 x 32 x 640 took 9.6 in clusters of 4 and 10.2 in clusters of 8.
inline GroupNormSplit choose(const GroupNormShape& a, int vec, int num_sms) {
    const int cg = a.C / a.groups, es = a.es;
    const int unit = vec / gcd(cg, vec);   // groups of the narrowest slab of whole vectors
    GroupNormSplit best = {a.groups, 1};
    double best_cost = 1e30;
    for (int slabs = 1; slabs <= a.groups; ++slabs) {
        if (a.groups % slabs != 0) continue;
        const int gps = a.groups / slabs;
        if (gps != a.groups && gps % unit != 0) continue;
        for (int c = 1; c <= kMaxCluster; c *= 2) {
            if (c > 1 && c > a.HW) break;
            const double kb = (double)((a.HW + c - 1) / c) * gps * cg * es / 1024.0;
            const double ctas = (double)a.N * slabs * c, full = 2.0 * num_sms, fill = std::min(1.0, ctas / full);
            const double row = (double)gps * cg * es, sectors = (gps * cg * es) % 32 ? 1.0 + 6.4 / row : 1.0;   // split ones
            double cost = 4.0 + 0.06 * kb * sectors * (0.6 + 0.4 * fill) + 0.05 * ((gps + 7) / 8);
            if (kb > kResBytes / 1024) cost += 0.04 * (kb - kResBytes / 1024);   // read twice
            if (c > 1) cost += c > 8 ? 1.3 : (c > 4 ? 0.4 : 0.2);
            if (c > 8 && ctas > num_sms) cost *= 2.0;   // clusters of 16 leave SMs idle
            cost *= std::max(1.0, ctas / full);
            if (cost >= best_cost) continue;
            // Up to kMaxParams channels, the kept rows (90 KiB), table (24 KiB: 384 entries of 8 channels) and parameters
            // (24 KiB) leave the exchange 11000 pairs.
            if ((gps * cg > kMaxParams || (c + 1) * gps > 10000) && make_split(a, vec, {gps, c}, nullptr) > kMaxSmem) continue;
            best_cost = cost;
            best = {gps, c};
        }
    }
    return best;
}

}  // namespace group_norm
}  // namespace wino
