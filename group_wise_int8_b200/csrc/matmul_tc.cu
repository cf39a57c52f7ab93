// Matrix product with bias, activation and residual on the sm_100a tensor cores,
// for outputs of many tiles: out = act([a | a2] w^T + bias) + residual in bf16
// operands and fp32 sums.  (The tensor cores truncate a partial sum where fp32 arithmetic rounds it, once every 16
// columns of K: up to about K 2^-28 of the terms' magnitudes, 1.9e-5 measured for 5120 terms of one sign.)
//
// Bound: the tensor cores when K is long, device memory (activations in, residual
// in, output out) for the 1x1 convolutions of an image network.  8192 x 1280 -> 5120 with GELU takes 83 us, 1290 TFLOP/s;
// 32768 x 960 -> 320 with residual 26.3 us where its 106 MB take 16.1 at the copy rate (the operands' way from L2 into the
// SMs comes first: 205 MB); 32768 x 320 -> 1280 30 us.
//
// Kernel structure (persistent; a cluster of two CTAs, one pair per two SMs, walks
// tiles of 256 rows x BN columns, BN a multiple of 32 up to 256):
//   The pair's MMA (tcgen05 cta_group::2, M = 256) reads A's 128 rows and half
//   of W's BN rows from each CTA's shared memory, so that a CTA loads (128 + BN/2)
//   rows per K step instead of 128 + BN: the L2-to-SM traffic of a lone CTA's
//   128 x 256 tiles would exceed what the SMs' ports carry at the tensor
//   cores' rate.
//   warp 0    = TMA producer: one or two blocks of 64 columns of K (128 bytes, 128-byte
//               swizzle) of a or a2 and of w per stage; both CTAs' loads complete on the
//               leader's barrier; columns past K read zeros.
//   warp 1    = TMEM allocator; in the leader the MMA issuer; two accumulators of BN columns,
//               so that the next tile's MMAs run under this tile's epilogue.
//   warps 2, 3 = the chunk buffers of one epilogue group each: residual chunks in
//               (TMA, two to four buffers a group), finished chunks out (TMA store).
//   warps 4-11 = epilogue, two groups of four warps (the four TMEM lane
//               quadrants) that take the tile's 64-column (fp32 output: 32) chunks in turn: fp32
//               accumulator + bias, activation, + residual, rounded once into a chunk
//               buffer (64- or 128-byte swizzle) that holds the residual chunk.
// Outputs or residuals whose base, pitch or row length is no multiple of 16 bytes (an odd
// number of columns) cannot go through TMA: there (DIRECT) each warp moves its own 32 rows, in 16-byte
// units as they lie in memory.  A row starts anywhere in a unit: the thread that holds the row shifts its
// packed values by that much (a few selects and byte permutes), the part of a unit that a chunk leaves
// over goes in front of the next chunk (an epilogue group takes consecutive chunks for that), and only the
// ends of a group's part of a row are stored value by value.  Residual units come in by
// asynchronous copies a chunk ahead and are shifted back.
// Every mbarrier wait is bounded.  On expiry the warp records the error and raises its CTA's abort flag, every role
// leaves its loop, in the other CTA too, and the pair waits (with a limit again) for the loads and MMAs under way before it
// frees its TMEM and returns.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "ops.h"
#include "sm100.cuh"

namespace wino {
namespace {

using namespace sm100;

__device__ int g_err;   // first error since matmul_tc_take_error

constexpr int kThreads = 384;
constexpr int kBK = 64;               // K per stage
constexpr int kMaxStages = 8;
constexpr int kARows = 128;           // rows of A per CTA
constexpr uint32_t kABytes = kARows * kBK * 2;
constexpr size_t kSmemBudget = 226 * 1024;

struct TcArgs {
    MatmulArgs m;   // m.force_timeout: before the pair's last tile the MMA issuer waits 1 ms on a barrier nothing completes
    int BN, kb, stages, buffers, tiles_m, tiles_n, steps0, steps1;   // kb: K blocks of 64 per stage (1 or 2)
};

// Epilogue chunks: 128 rows of 128 bytes (64 bf16 or 32 fp32 columns) in the 128-byte swizzle; where a tile's width
// leaves half a bf16 chunk, 32 columns.
constexpr int kChunkBytes = kARows * 128;
constexpr int kMaxBuffers = 4;   // per epilogue group
// DIRECT: a warp's 32 rows of a chunk's units and the one that it shares with its neighbour; 144 bytes apart, so that neither a
// row's owner nor the copies between a row and memory meet bank conflicts.
constexpr int kRowPitch = 128 + 16;
constexpr int kRowsBytes = 32 * kRowPitch;
// Byte offset of 16-byte unit j of a row of ROW bytes (64 or 128: the TMA swizzle of that width).
template <int ROW>
__device__ __forceinline__ uint32_t chunk_unit(int row, int j) {
    return (uint32_t)(row * ROW + ((j ^ (ROW == 64 ? (row >> 1) & 3 : row & 7)) << 4));
}

// p[j] = the word `elems` values of SIZE bytes (fewer than 16 bytes) behind word j, in place.
template <int SIZE, int N>
__device__ __forceinline__ void shift_words(uint32_t (&p)[N], int elems) {
    const int f = elems * SIZE / 4;
#pragma unroll
    for (int j = 0; j + 2 < N; ++j) p[j] = f & 2 ? p[j + 2] : p[j];
#pragma unroll
    for (int j = 0; j + 1 < N; ++j) p[j] = f & 1 ? p[j + 1] : p[j];
    if constexpr (SIZE == 2) {
        const uint32_t sel = elems & 1 ? 0x5432u : 0x3210u;
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = __byte_perm(p[j], j + 1 < N ? p[j + 1] : 0u, sel);
    }
}

// Bytes of a 16-byte unit of values of SIZE bytes of which `values` (one at least) lie before the row's end.  (Clamped
// before it is multiplied: a row has up to 2^31 values, and their bytes would pass an int.)
template <int SIZE>
__host__ __device__ constexpr int unit_bytes(int values) {
    return (values < 16 / SIZE ? values : 16 / SIZE) * SIZE;
}
static_assert(unit_bytes<2>(3) == 6 && unit_bytes<2>((1 << 30) + 1) == 16 && unit_bytes<4>((1 << 29) + 1) == 16 &&
                  unit_bytes<4>(2147483647) == 16,
              "a unit has at most 16 bytes however long its row is");

struct Tail {
    uint64_t full[kMaxStages];     // leader: both CTAs' operands of the stage have landed
    uint64_t empty[kMaxStages];    // the pair's MMAs have read the stage
    uint64_t acc_full[2];
    uint64_t acc_empty[2];         // leader: both CTAs' epilogues have read the accumulator
    uint64_t buf_full[2][kMaxBuffers];       // a group's chunk buffer is free to use, its residual (if any) landed
    uint64_t buf_ready[2][kMaxBuffers];      // ... and holds the output chunk: the group's four warps have written it
    uint64_t done;                   // after an expiry: the pair's MMAs have completed
    uint64_t never;                  // completed by nobody: the forced expiry waits on it
    alignas(16) float bias[8][64];   // per epilogue warp
    uint32_t tmem_base;
    uint32_t issued;                 // stages that this CTA's producer has loaded
    int abort_flag;
};

// Warp-uniform bounded wait: every lane polls, the loop exits for all lanes together.  (The timer is read only once a
// few polls have failed: reading it costs more than most waits.)
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                          unsigned long long limit_ns = kWaitLimitNs) {
    unsigned long long t0 = 0;
    for (uint32_t it = 0;; ++it) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
        if ((it & 63u) == 63u) {
            bool stop = *abort_flag != 0;
            if (it == 63u) {
                t0 = globaltimer();
            } else if (!stop && globaltimer() - t0 > limit_ns) {
                stop = true;
                *abort_flag = 1;
                atomicCAS(&g_err, 0, kDevErrTimeout);
            }
            if (__any_sync(0xffffffffu, stop)) return false;
        }
    }
}

// A ring's current barrier, asked for its phase one turn ahead: the answer is there when the turn comes.
struct Peek {
    int st = 0;
    uint32_t phase;
    bool ready = false;
    __device__ __forceinline__ Peek(uint64_t* bars, uint32_t first_phase) : phase(first_phase) { ready = mbar_test(bars, phase); }
    __device__ __forceinline__ bool wait(uint64_t* bars, volatile int* abort_flag) const {
        return __all_sync(0xffffffffu, ready) || warp_wait(&bars[st], phase, abort_flag);
    }
    __device__ __forceinline__ void next(uint64_t* bars, int stages) {
        if (++st == stages) {
            st = 0;
            phase ^= 1u;
        }
        ready = mbar_test(&bars[st], phase);
    }
};

// A pair's tiles, in steps of the grid's pairs (no division on the way).
struct Tile {
    int t, m, n;             // index, row of tiles, column of tiles
    int step, step_m, step_n;
    __device__ __forceinline__ Tile(const TcArgs& p, int first, int grid_pairs) {
        t = first;
        m = first / p.tiles_n;
        n = first - m * p.tiles_n;
        step = grid_pairs;
        step_m = step / p.tiles_n;
        step_n = step - step_m * p.tiles_n;
    }
    __device__ __forceinline__ void next(const TcArgs& p) {
        t += step;
        m += step_m;
        n += step_n;
        if (n >= p.tiles_n) {
            n -= p.tiles_n;
            ++m;
        }
    }
    __device__ __forceinline__ bool valid(const TcArgs& p) const { return t < p.tiles_m * p.tiles_n; }
};

// Chunks of COLS columns in a tile.
template <int COLS>
__device__ __forceinline__ int chunks_of(const TcArgs& p, const Tile& t) {
    return (min(p.BN, p.m.N - t.n * p.BN) + COLS - 1) / COLS;
}

// The chunks of one epilogue group, tile after tile: chunk c of each tile, c = g, g + 2, ...
template <int COLS>
struct Cursor {
    Tile tile;
    int c, g;
    __device__ __forceinline__ Cursor(const Tile& first, int group, const TcArgs& p) : tile(first), c(group), g(group) { settle(p); }
    __device__ __forceinline__ bool valid(const TcArgs& p) const { return tile.valid(p); }
    __device__ __forceinline__ void settle(const TcArgs& p) {   // to the next existing chunk
        while (tile.valid(p) && c >= chunks_of<COLS>(p, tile)) {
            tile.next(p);
            c = g;
        }
    }
    __device__ __forceinline__ void next(const TcArgs& p) {
        c += 2;
        settle(p);
    }
};

// All chunk buffers of a CTA.
__host__ __device__ constexpr int chunk_bytes(bool direct, bool res, int buffers) {
    return direct ? (res ? 2 : 1) * 8 * kRowsBytes : 2 * buffers * kChunkBytes;
}

template <typename TO, bool DIRECT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    matmul_tc_kernel(const __grid_constant__ CUtensorMap tmA0, const __grid_constant__ CUtensorMap tmA1,
                     const __grid_constant__ CUtensorMap tmW0, const __grid_constant__ CUtensorMap tmW1,
                     const __grid_constant__ CUtensorMap tmOut, const __grid_constant__ CUtensorMap tmRes,
                     const __grid_constant__ CUtensorMap tmOutHalf, const __grid_constant__ CUtensorMap tmResHalf,
                     const TcArgs p) {
    constexpr int CW = 128 / (int)sizeof(TO);
    const int NB = p.buffers;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t block_bytes = kABytes + (uint32_t)(p.BN / 2) * kBK * 2;   // one K block of A, then of W
    const uint32_t stage_bytes = (uint32_t)p.kb * block_bytes;
    // [2 groups][NB][kChunkBytes], or [output, residual if any][8 warps][kRowsBytes]
    unsigned char* chunks = smem + (size_t)p.stages * stage_bytes;
    Tail* tail = reinterpret_cast<Tail*>(chunks + chunk_bytes(DIRECT, p.m.res != nullptr, p.buffers));
    volatile int* abort_flag = &tail->abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t half = cluster_rank() & 1u;   // 0: the pair's leader, rows 0..127 of its tiles
    const uint16_t mask = 3;
    const Tile first(p, (int)(blockIdx.x / 2), (int)(gridDim.x / 2));
    const int steps = p.steps0 + p.steps1;
    grid_dependents_launch();

    if (threadIdx.x == 0) {
        for (int s = 0; s < p.stages; ++s) {
            mbar_init(&tail->full[s], 1);
            mbar_init(&tail->empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tail->acc_full[b], 1);
            mbar_init(&tail->acc_empty[b], 16);   // the epilogue warps of both CTAs
            for (int i = 0; i < NB; ++i) {
                mbar_init(&tail->buf_full[b][i], 1);
                mbar_init(&tail->buf_ready[b][i], 4);
            }
        }
        if (p.m.force_timeout) mbar_init(&tail->never, 1);
        tail->abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        prefetch_tensormap(&tmA0);
        prefetch_tensormap(&tmW0);
        if (!DIRECT) prefetch_tensormap(&tmOut);
    }
    if (warp == 1) tmem_alloc_pair(&tail->tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers exist before either signals the other's
    tc_fence_after();
    grid_dependency_wait();   // (the setup above overlaps the previous kernel's tail)
    const uint32_t tmem_base = tail->tmem_base;
    const bool has_res = p.m.res != nullptr;
    auto origin_m = [&](const Tile& t) { return t.m * 256 + (int)half * kARows; };
    auto origin_n = [&](const Tile& t, int c) { return t.n * p.BN + c * CW; };
    auto half_chunk = [&](int c) { return CW == 64 && c * CW + CW > p.BN; };   // the tile ends in its middle

    bool ok = true;   // no wait of this warp has run out, and none has been called off
    if (warp == 0) {
        // ------------------------------------------------------- TMA producer
        Peek ring_at(tail->empty, 1u);
        uint32_t issued = 0;
        const uint32_t full0 = map_rank(&tail->full[0], 0);
        for (Tile t = first; ok && t.valid(p); t.next(p)) {
            const int m0 = origin_m(t), n0 = t.n * p.BN + (int)half * (p.BN / 2);
            for (int s = 0; s < steps; s += p.kb) {
                if (!ring_at.wait(tail->empty, abort_flag)) {
                    ok = false;
                    break;
                }
                const int st = ring_at.st, blocks = min(p.kb, steps - s);
                ring_at.next(tail->empty, p.stages);
                const uint32_t bar = full0 + 8u * (uint32_t)st;
                unsigned char* dst = smem + (size_t)st * stage_bytes;
                if (elect_one()) {
                    if (half == 0) mbar_arrive_expect_tx(&tail->full[st], 2u * (uint32_t)blocks * block_bytes);
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        if (j < blocks) {
                            const bool second = s + j >= p.steps0;
                            const int k = (second ? s + j - p.steps0 : s + j) * kBK;
                            tma_load_2d_pair(dst + j * block_bytes, second ? &tmA1 : &tmA0, bar, k, m0);
                            tma_load_2d_pair(dst + j * block_bytes + kABytes, second ? &tmW1 : &tmW0, bar, k, n0);
                        }
                }
                ++issued;
            }
        }
        if (lane == 0) tail->issued = issued;
    } else if (warp == 1) {
        // --------------------------------------------------------- MMA issuer
        if (half == 0) {
            const uint32_t idesc = idesc_bf16(256, p.BN);
            const uint64_t a_desc = smem_desc_kmajor(smem_u32(smem), 128);
            const uint64_t w_desc = smem_desc_kmajor(smem_u32(smem) + kABytes, 128);
            const int last0 = (p.m.K0 - (p.steps0 - 1) * kBK + 15) / 16;                 // K-steps of 16 in a source's
            const int last1 = p.steps1 ? (p.m.K1 - (p.steps1 - 1) * kBK + 15) / 16 : 0;  // last block
            Peek ring_at(tail->full, 0u);
            int it = 0;
            for (Tile t = first; ok && t.valid(p); t.next(p), ++it) {
                const int b = it & 1;
                if (p.m.force_timeout && t.t + t.step >= p.tiles_m * p.tiles_n) ok = warp_wait(&tail->never, 0u, abort_flag, 1000000ull);
                ok = ok && warp_wait(&tail->acc_empty[b], (uint32_t)((it >> 1) & 1) ^ 1u, abort_flag);
                if (!ok) break;
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)b * 256u;
                for (int s = 0; s < steps; s += p.kb) {
                    if (!ring_at.wait(tail->full, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const int st = ring_at.st, blocks = min(p.kb, steps - s);
                    ring_at.next(tail->full, p.stages);
                    tc_fence_after();
                    const uint32_t off = (uint32_t)st * (stage_bytes >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            if (j < blocks) {
                                const int kn = s + j == p.steps0 - 1 ? last0 : (s + j == steps - 1 ? last1 : kBK / 16);
                                const uint64_t at = off + j * (block_bytes >> 4);
#pragma unroll
                                for (int kk = 0; kk < kBK / 16; ++kk)
                                    if (kk < kn) mma_bf16_pair(d, a_desc + at + 2 * kk, w_desc + at + 2 * kk, idesc, (s | j | kk) != 0);
                            }
                        mma_commit_pair(&tail->empty[st], mask);
                        if (s + p.kb >= steps) mma_commit_pair(&tail->acc_full[b], mask);
                    }
                }
            }
        }
    } else if (warp < 4) {
        // -------------------------------------- chunk buffers of one epilogue group
        if constexpr (!DIRECT) {
            const int g = warp - 2;
            unsigned char* ring = chunks + (size_t)g * NB * kChunkBytes;
            Cursor<CW> cur(first, g, p), ahead = cur;
            int loads = 0;                   // residual chunks asked for: the i-th into buffer i % NB
            auto hand_out = [&](int buf) {   // a free buffer, for the chunk at `ahead`
                if (!has_res) {
                    mbar_arrive(&tail->buf_full[g][buf]);
                } else if (ahead.valid(p)) {
                    const bool hc = half_chunk(ahead.c);
                    mbar_arrive_expect_tx(&tail->buf_full[g][buf], hc ? kChunkBytes / 2 : kChunkBytes);
                    tma_load_2d(ring + buf * kChunkBytes, hc ? &tmResHalf : &tmRes, &tail->buf_full[g][buf],
                                origin_n(ahead.tile, ahead.c), origin_m(ahead.tile));
                    ahead.next(p);
                    ++loads;
                }
            };
            if (lane == 0)
                for (int i = 0; i < NB; ++i) hand_out(i);
            __syncwarp();
            int buf = 0;
            uint32_t phase = 0;
            for (int i = 0; cur.valid(p); cur.next(p), ++i) {
                ok = warp_wait(&tail->buf_ready[g][buf], phase, abort_flag);
                if (!ok) break;
                if (lane == 0) {
                    const int m0 = origin_m(cur.tile);
                    if (m0 < p.m.M)
                        tma_store_2d(half_chunk(cur.c) ? &tmOutHalf : &tmOut, ring + buf * kChunkBytes, origin_n(cur.tile, cur.c), m0);
                    bulk_commit();
                    bulk_wait_read<1>();   // the store before this one has read its buffer, which is handed out again
                    if (i > 0) hand_out(buf ? buf - 1 : NB - 1);
                }
                __syncwarp();
                if (++buf == NB) {
                    buf = 0;
                    phase ^= 1u;
                }
            }
            if (lane == 0) {
                bulk_wait_read<0>();
                if (!ok)   // (otherwise the epilogue has waited for every residual chunk)
                    for (int i = max(0, loads - NB); i < loads; ++i) mbar_wait_teardown(&tail->buf_full[g][i % NB], (uint32_t)(i / NB) & 1u);
            }
        }
    } else {
        // ----------------------------------------------------------- epilogue
        const int g = (warp - 4) >> 2, quad = warp & 3, row = 32 * quad + lane;
        const uint32_t t_lane = tmem_base + ((uint32_t)(32 * quad) << 16);
        unsigned char* ring = chunks + (size_t)g * NB * kChunkBytes;
        float* bias_s = tail->bias[warp - 4];
        const uint32_t release = map_rank(&tail->acc_empty[0], 0);
        int it = 0, buf = 0;
        uint32_t rphase = 0;
        // DIRECT: the values of a unit; this warp's rows of the output and of the residual
        constexpr int E = 16 / (int)sizeof(TO);
        unsigned char* out_rows = chunks + (size_t)(warp - 4) * kRowsBytes;
        unsigned char* res_rows = out_rows + 8 * kRowsBytes;
        uint32_t carry[4] = {0u, 0u, 0u, 0u};   // this row's last unit of the chunk before
        // a group's chunks of a tile: every other one, or half of them
        auto first_chunk = [&](const Tile& t) { return DIRECT ? (g ? (chunks_of<CW>(p, t) + 1) / 2 : 0) : g; };
        auto end_chunk = [&](const Tile& t) { return DIRECT && g == 0 ? (chunks_of<CW>(p, t) + 1) / 2 : chunks_of<CW>(p, t); };
        constexpr int kChunkStep = DIRECT ? 1 : 2;
        // DIRECT: the units that hold the residual's chunk c of the warp's rows
        auto fetch_res = [&](const Tile& t, int c) {
            if constexpr (DIRECT) {
                if (has_res && t.valid(p) && c < end_chunk(t)) {
                    const TO* res = static_cast<const TO*>(p.m.res);
                    const int n0 = origin_n(t, c), left = p.m.N - n0, rows = p.m.M - origin_m(t) - 32 * quad, u = lane & 7;
                    const TO* at = res + (size_t)(p.m.M - rows + (lane >> 3)) * p.m.ldr + n0;
                    unsigned char* dst = res_rows + (lane >> 3) * kRowPitch + 16 * u;
                    const TO* res_end = res + (size_t)(p.m.M - 1) * p.m.ldr + p.m.N;   // (of the debug build's check)
                    auto copy = [&](unsigned char* to, const TO* from, int values) {   // (zeros behind the row's end)
                        const int bytes = unit_bytes<(int)sizeof(TO)>(values);
                        if (in_bounds((size_t)(from - res) + (size_t)bytes / sizeof(TO) - 1, (size_t)(res_end - res), &g_err))
                            copy_async16(to, from, bytes);
                    };
#pragma unroll 2
                    for (int r = lane >> 3; r < min(32, rows); r += 4, at += 4 * p.m.ldr, dst += 4 * kRowPitch) {
                        const int d = E * u - ((int)(reinterpret_cast<uintptr_t>(at) / sizeof(TO)) & (E - 1));
                        if (d < left) {
                            if (at + d >= res) {
                                copy(dst, at + d, left - d);
                            } else {   // the tensor starts inside the unit
                                for (int e = (int)(res - at) - d; e < E && d + e < left; ++e) reinterpret_cast<TO*>(dst)[e] = at[d + e];
                            }
                        }
                        if (u == 0 && d < 0 && d + 8 * E < left) copy(dst + 128, at + d + 8 * E, left - d - 8 * E);
                    }
                }
            }
        };
        // One chunk of W columns at column n0 of the output, from TMEM column `tcol`; `last`: this warp's last read of
        // accumulator b; the group's part of the tile's columns: lo to hi.
        auto chunk = [&](auto width, int n0, int m0, uint32_t tcol, int b, bool last, int lo, int hi, auto prefetch) {
            constexpr int W = decltype(width)::value, ROW = W * (int)sizeof(TO), UP = ROW / 16;
            unsigned char* cb = ring + (size_t)buf * kChunkBytes;
            uint32_t r[W];
#pragma unroll
            for (int j = 0; j < W; j += 32) tmem_ld<32>(t_lane + tcol + (uint32_t)j, *reinterpret_cast<uint32_t(*)[32]>(r + j));
            __syncwarp();
            tmem_ld_wait();
            tmem_regs_ready(r);
            if (last) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(release + 8u * (uint32_t)b);
            }
            float v[W];
#pragma unroll
            for (int j = 0; j < W; j += 4) {
                const float4 bb = *reinterpret_cast<const float4*>(bias_s + j);
                v[j] = __uint_as_float(r[j]) + bb.x;
                v[j + 1] = __uint_as_float(r[j + 1]) + bb.y;
                v[j + 2] = __uint_as_float(r[j + 2]) + bb.z;
                v[j + 3] = __uint_as_float(r[j + 3]) + bb.w;
            }
            if (p.m.act == WINO_ACT_SILU) activate_all<WINO_ACT_SILU, sizeof(TO) == 2>(v);
            if (p.m.act == WINO_ACT_GELU) activate_all<WINO_ACT_GELU, sizeof(TO) == 2>(v);
            if (!DIRECT && !warp_wait(&tail->buf_full[g][buf], rphase, abort_flag)) {
                ok = false;
                return;
            }
            if (!DIRECT && has_res) {
#pragma unroll
                for (int j = 0; j < ROW / 16; ++j) {
                    const uint4 w = *reinterpret_cast<const uint4*>(cb + chunk_unit<ROW>(row, j));
                    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if constexpr (sizeof(TO) == 2) {
                            v[8 * j + 2 * i] += __uint_as_float(x[i] << 16);
                            v[8 * j + 2 * i + 1] += __uint_as_float(x[i] & 0xffff0000u);
                        } else {
                            v[4 * j + i] += __uint_as_float(x[i]);
                        }
                    }
                }
            }
            if constexpr (DIRECT) {
                const int m = m0 + row;
                if (has_res) {
                    copy_wait_all();
                    __syncwarp();
                    uint32_t x[4 + ROW / 4];
#pragma unroll
                    for (int j = 0; j <= UP; ++j)
                        *reinterpret_cast<uint4*>(x + 4 * j) = *reinterpret_cast<const uint4*>(res_rows + lane * kRowPitch + 16 * j);
                    const TO* at = static_cast<const TO*>(p.m.res) + (size_t)m * p.m.ldr + n0;
                    shift_words<sizeof(TO)>(x, (int)(reinterpret_cast<uintptr_t>(at) / sizeof(TO)) & (E - 1));
#pragma unroll
                    for (int j = 0; j < ROW / 4; ++j) {
                        if constexpr (sizeof(TO) == 2) {
                            v[2 * j] += __uint_as_float(x[j] << 16);
                            v[2 * j + 1] += __uint_as_float(x[j] & 0xffff0000u);
                        } else {
                            v[j] += __uint_as_float(x[j]);
                        }
                    }
                    __syncwarp();
                    prefetch();
                }
                // unit j of the row in memory: `t` values behind unit j - 1 of the chunk
                TO* out = static_cast<TO*>(p.m.out);
                auto ahead = [&](const TO* at) { return (0 - (int)(reinterpret_cast<uintptr_t>(at) / sizeof(TO))) & (E - 1); };
                uint32_t x[4 + ROW / 4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = carry[j];
#pragma unroll
                for (int j = 0; j < ROW / 4; ++j) {
                    if constexpr (sizeof(TO) == 2) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
                        x[4 + j] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        x[4 + j] = __float_as_uint(v[j]);
                    }
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) carry[j] = x[ROW / 4 + j];
                shift_words<sizeof(TO)>(x, ahead(out + (size_t)m * p.m.ldo + n0));
#pragma unroll
                for (int j = 0; j <= UP; ++j)
                    *reinterpret_cast<uint4*>(out_rows + lane * kRowPitch + 16 * j) =
                        make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
                __syncwarp();
                // four rows at a time: whole units, and value by value the ends of the group's part of a row
                const int rows = min(32, p.m.M - m0 - 32 * quad), u = lane & 7, from = lo - n0, to = hi - n0;
                const unsigned char* src = out_rows + (lane >> 3) * kRowPitch;
                TO* at = out + (size_t)(m0 + 32 * quad + (lane >> 3)) * p.m.ldo + n0;
                const TO* end = out + (size_t)(p.m.M - 1) * p.m.ldo + p.m.N;   // (of the debug build's check)
#pragma unroll 2
                for (int r = lane >> 3; r < rows; r += 4, at += 4 * p.m.ldo, src += 4 * kRowPitch) {
                    const int d0 = ahead(at) - E, d = d0 + E * u;   // columns from n0 of the row's first unit and of unit u
                    if (u < UP && d >= from && d + E <= to && in_bounds((size_t)(at + d + E - 1 - out), (size_t)(end - out), &g_err))
                        *reinterpret_cast<uint4*>(at + d) = *reinterpret_cast<const uint4*>(src + 16 * u);
                    auto value = [&](int unit) {
                        const int x = d0 + E * unit + u;
                        if (u < E && x >= from && x < to && in_bounds((size_t)(at + x - out), (size_t)(end - out), &g_err))
                            at[x] = reinterpret_cast<const TO*>(src + 16 * unit)[u];
                    };
                    if (from == 0) value(0);
                    if (W >= to) value(min((to - d0) / E, UP));
                }
                __syncwarp();
                return;
            }
#pragma unroll
            for (int j = 0; j < ROW / 16; ++j) {
                uint4 w;
                if constexpr (sizeof(TO) == 2) {
                    uint32_t x[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
                        x[i] = *reinterpret_cast<const uint32_t*>(&h);
                    }
                    w = make_uint4(x[0], x[1], x[2], x[3]);
                } else {
                    w = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                                   __float_as_uint(v[4 * j + 3]));
                }
                *reinterpret_cast<uint4*>(cb + chunk_unit<ROW>(row, j)) = w;
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&tail->buf_ready[g][buf]);
            if (++buf == NB) {
                buf = 0;
                rphase ^= 1u;
            }
            __syncwarp();
        };
        float bias_next[CW / 32];   // this lane's columns of the next chunk, on their way before it starts
        auto fetch_bias = [&](const Tile& t, int c) {
#pragma unroll
            for (int j = 0; j < CW / 32; ++j) {
                const int n = origin_n(t, c) + 32 * j + lane;
                bias_next[j] = p.m.bias && n < p.m.N ? p.m.bias[n] : 0.0f;
            }
        };
        fetch_bias(first, first_chunk(first));
        fetch_res(first, first_chunk(first));
        Tile following = first;
        for (Tile t = first; ok && t.valid(p); t = following, ++it) {
            const int b = it & 1;
            const int c0 = first_chunk(t), end = end_chunk(t), m0 = origin_m(t);
            const int lo = origin_n(t, c0), hi = min(min(origin_n(t, end), origin_n(t, 0) + p.BN), p.m.N);
            following.next(p);
            ok = warp_wait(&tail->acc_full[b], (uint32_t)((it >> 1) & 1), abort_flag);
            if (!ok) break;
            tc_fence_after();
            for (int c = c0; ok && c < end; c += kChunkStep) {
                const bool last = c + kChunkStep >= end;
#pragma unroll
                for (int j = 0; j < CW / 32; ++j) bias_s[32 * j + lane] = bias_next[j];
                if (!last) fetch_bias(t, c + kChunkStep);
                else fetch_bias(following, first_chunk(following));
                auto prefetch = [&]() {
                    if (!last) fetch_res(t, c + kChunkStep);
                    else fetch_res(following, first_chunk(following));
                };
                const uint32_t tcol = (uint32_t)(b * 256 + c * CW);
                if (half_chunk(c)) chunk(std::integral_constant<int, 32>(), origin_n(t, c), m0, tcol, b, last, lo, hi, prefetch);
                else chunk(std::integral_constant<int, CW>(), origin_n(t, c), m0, tcol, b, last, lo, hi, prefetch);
            }
            if (c0 >= end) {   // a tile of one chunk leaves the second group nothing to read
                fetch_bias(following, first_chunk(following));
                fetch_res(following, first_chunk(following));
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(release + 8u * (uint32_t)b);
            }
        }
        if (DIRECT) copy_wait_all();
    }

    // Every role of both CTAs is done: the MMAs that read either CTA's shared memory have completed (both epilogues
    // waited for the last accumulator), and no arrival is under way to a CTA that has left.
    if (!ok && lane == 0) st_cluster_u32(map_rank(&tail->abort_flag, half ^ 1u), 1u);   // (an expiry ends the other CTA's roles, too)
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    if (__builtin_expect(*abort_flag, 0)) {   // (of both CTAs.)  Not so after an expiry: wait for what is under way
        if (threadIdx.x == 0) {
            mbar_init(&tail->done, 1);
            fence_mbar_init();
        }
        __syncthreads();
        cluster_sync();
        if (warp == 0 && half == 0 && lane == 0) {
            // the newest loads of each stage, by whichever CTA got further: a stage that only one of them has loaded
            // does not complete, and its loads have landed when the limit has passed
            const uint32_t n = max(tail->issued, ld_cluster_u32(map_rank(&tail->issued, 1))), S = (uint32_t)p.stages;
            const unsigned long long t0 = globaltimer();
            for (uint32_t i = n > S ? n - S : 0u; i < n; ++i)
                while (!mbar_try_wait(&tail->full[i % S], (i / S) & 1u) && globaltimer() - t0 <= kWaitLimitNs) {}
        } else if (warp == 1) {
            if (half == 0 && elect_one()) mma_commit_pair(&tail->done, mask);
            __syncwarp();
            if (lane == 0) mbar_wait_teardown(&tail->done, 0u);
        }
        tc_fence_before();
        __syncthreads();
        cluster_sync();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
}

size_t smem_bytes(const TcArgs& a, bool direct) {
    return 1024 + (size_t)a.stages * a.kb * (kABytes + a.BN / 2 * kBK * 2) + chunk_bytes(direct, a.m.res != nullptr, a.buffers) + sizeof(Tail);
}

bool tma_ok(const void* p, long pitch, int rows, size_t es) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (rows == 1 || (size_t)pitch * es % 16 == 0);
}

bool map_2d(CUtensorMap* map, bool bf16, const void* base, int cols, int rows, long pitch, int box_cols, int box_rows) {
    const size_t es = bf16 ? 2 : 4;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(rows == 1 ? ((size_t)cols * es + 15) / 16 * 16 : (size_t)pitch * es)};
    const cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    return make_tensor_map(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base, dims,
                           strides, box, box_cols * es == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Operand tensor maps: boxes of 64 columns x 128 rows of a and a2, x w_rows rows of w.
bool operand_maps(const MatmulArgs& a, int w_rows, CUtensorMap (&map)[4]) {
    const void* w1 = static_cast<const __nv_bfloat16*>(a.w) + a.K0;
    if (!map_2d(&map[0], true, a.a, a.K0, a.M, a.lda, kBK, kARows) || !map_2d(&map[2], true, a.w, a.K0, a.N, a.ldw, kBK, w_rows))
        return false;
    if (a.K1 == 0) {
        map[1] = map[0];
        map[3] = map[2];
        return true;
    }
    return map_2d(&map[1], true, a.a2, a.K1, a.M, a.lda2, kBK, kARows) && map_2d(&map[3], true, w1, a.K1, a.N, a.ldw, kBK, w_rows);
}

// The tile width: as few rounds of tiles over the SM pairs as possible, weighing a round by its width
// and a fixed part (filling the pipeline and the accumulator hand-over).  The fixed part is a fit to every width of 110
// products (16 to 33000 rows, K of 64 to 4096): the choice took 1.1 % more time than the best width on average and 15 % at
// most (19022 x 544 -> 695 takes 68 us in tiles of 64 columns and 48 in tiles of 128; 271 x 512 -> 128 6.5 in tiles of 64 and
// 5.4 in tiles of 32).  With fewer than 64 rows, many pairs at a time read the same few lines of a, which takes longer
// (1280 -> 1280 on 40 pairs: 8.7 us for 16 rows, 6.5 for 64; on 20 pairs 6.7 for both).
int tile_width(const MatmulArgs& a, int num_sms) {
    const long rows = (a.M + 255L) / 256, pairs = num_sms / 2;
    int best = 256;
    double best_cost = 0;
    for (int bn = 256; bn >= 32; bn -= 32) {
        const long tiles = rows * ((a.N + (long)bn - 1) / bn);
        double cost = (double)((tiles + pairs - 1) / pairs) * (bn + 48);
        if (a.M < 64) cost += 2.5 * std::max(0L, std::min(tiles, pairs) - 24);
        if (best_cost == 0 || cost < best_cost) {
            best_cost = cost;
            best = bn;
        }
    }
    return best;
}

}  // namespace

bool matmul_tma_operands(const MatmulArgs& a) {
    return a.bf16 && tma_ok(a.a, a.lda, a.M, 2) && tma_ok(a.w, a.ldw, a.N, 2) &&
           (a.K1 == 0 || (tma_ok(a.a2, a.lda2, a.M, 2) && a.K0 % 8 == 0));
}

cudaError_t launch_matmul_tc(const MatmulArgs& m, int num_sms, cudaStream_t st) {
    TcArgs a = {};
    a.m = m;
    a.BN = tile_width(m, num_sms);
    const long tiles_m = (m.M + 255L) / 256, tiles_n = (m.N + (long)a.BN - 1) / a.BN;
    if (tiles_m * tiles_n > 1073741824L) return cudaErrorInvalidConfiguration;
    a.tiles_m = (int)tiles_m;
    a.tiles_n = (int)tiles_n;
    a.steps0 = (m.K0 + kBK - 1) / kBK;
    a.steps1 = (m.K1 + kBK - 1) / kBK;
    const size_t so = m.out_bf16 ? 2 : 4;
    // (a TMA store writes whole 16-byte units: a row that ends inside one would have zeros written behind it)
    const bool direct = (size_t)m.N * so % 16 != 0 || !tma_ok(m.out, m.ldo, m.M, so) || (m.res && !tma_ok(m.res, m.ldr, m.M, so));
    CUtensorMap map[4], out, res, out_half, res_half;
    if (!operand_maps(m, a.BN / 2, map)) return cudaErrorInvalidValue;
    out = res = out_half = res_half = map[0];
    if (!direct) {
        const int cols = 128 / (int)so;
        bool ok = map_2d(&out, m.out_bf16, m.out, m.N, m.M, m.ldo, cols, kARows);
        if (m.res) ok = ok && map_2d(&res, m.out_bf16, m.res, m.N, m.M, m.ldr, cols, kARows);
        if (m.out_bf16 && a.BN % 64 != 0) {
            ok = ok && map_2d(&out_half, true, m.out, m.N, m.M, m.ldo, 32, kARows);
            if (m.res) ok = ok && map_2d(&res_half, true, m.res, m.N, m.M, m.ldr, 32, kARows);
        }
        if (!ok) return cudaErrorInvalidValue;
    }
    // two K blocks per stage where their MMAs take less time than the issue loops' turn (about 340 cycles; a block
    // takes 2 BN), as long as three stages fit
    a.kb = a.BN <= 128 ? 2 : 1;
    // Residual chunks wait in the buffers, so that tiles of few K blocks, whose time is the residual's way in, want more of
    // them, and others more stages (32768 x 320 -> 1280 with residual: 52 us with two buffers, 41 with three; 14778 x 128
    // -> 2624: 51, 35 and 31 with four; 32768 x 512 -> 640: 30 with two, 33 with three; without a residual two do)
    const int steps = a.steps0 + a.steps1;
    a.buffers = !m.res || steps > 6 ? 2 : (steps > 2 ? 3 : kMaxBuffers);
    a.stages = 2;
    while (a.buffers > 2 && smem_bytes(a, direct) > kSmemBudget) --a.buffers;
    a.stages = kMaxStages;
    while (a.stages > 2 && smem_bytes(a, direct) > kSmemBudget) --a.stages;
    const size_t smem = smem_bytes(a, direct);
    const long pairs = std::min<long>(tiles_m * tiles_n, std::max(1, num_sms / 2));
    static bool done[4][64];
    auto go = [&](auto kern, bool (&d)[64]) -> cudaError_t {
        const cudaError_t e = allow_smem(kern, kSmemBudget, d);
        if (e != cudaSuccess) return e;
        return launch_dependent(kern, dim3((unsigned)(2 * pairs)), dim3(kThreads), smem, st, map[0], map[1], map[2], map[3],
                                out, res, out_half, res_half, a);
    };
    if (m.out_bf16)
        return direct ? go(matmul_tc_kernel<__nv_bfloat16, true>, done[0]) : go(matmul_tc_kernel<__nv_bfloat16, false>, done[1]);
    return direct ? go(matmul_tc_kernel<float, true>, done[2]) : go(matmul_tc_kernel<float, false>, done[3]);
}

cudaError_t matmul_tc_take_error(int* err) {
    cudaError_t e = cudaMemcpyFromSymbol(err, g_err, sizeof(int));
    const int zero = 0;
    if (e == cudaSuccess && *err) e = cudaMemcpyToSymbol(g_err, &zero, sizeof(int));
    return e;
}

}  // namespace wino
