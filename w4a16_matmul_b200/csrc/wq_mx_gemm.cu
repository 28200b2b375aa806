// wq_mx_gemm.cu -- products of two MXFP4 matrices on the block-scaled tensor cores, dense and
// grouped by expert.
//
//   y[t, r] = sum over blocks b of 32 columns of  2^(sx[t, b] - 127) 2^(sw[r, b] - 127)
//             sum_{c in b} x4[t, c] w4[r, c]
//
// tcgen05.mma kind::mxf4.block_scale takes the packed 4-bit codes of both operands from shared
// memory and their scale bytes from tensor memory, and accumulates in fp32. One CTA computes a
// 128 (weight rows) x BN (activation rows) tile over a K range:
//   warp 0     TMA producer: per stage of 256 columns the codes of the weight tile [128 x 128
//              bytes] and of the activation tile [BN x 128 bytes], 128-byte swizzle; per 512
//              columns the scale bytes of both [128 + BN rows x 16 bytes];
//   warp 1     allocates tensor memory, and one lane issues the MMAs (K = 64 each);
//   warps 2-5  move the scale bytes into tensor memory: the MMA wants the four bytes of row r's
//              128 columns in lane r % 32 of column r / 32, in each of the four lane quarters,
//              so each warp fills its own quarter; afterwards they drain the accumulator. For few
//              rows they quantise the activations, too (XQ below).
// Few activation rows run this way; more, and most products of experts, run on pairs of CTAs, the
// second kernel below (launch_gemm_mxfp4 says when).
// Grouped by expert, a CTA finds its expert and its rows from the offsets on the device: the
// host reads nothing back, and launches as many row tiles as the worst distribution needs.
// Rows of the activation tile past the expert's range belong to the next expert (or lie behind
// the matrix, where TMA fills zeros): they fill accumulator columns that are not stored.
// Where the row tiles alone leave SMs idle (few activation rows), a cluster of CL CTAs splits K
// and meets in distributed shared memory; the partial sums are added in rank order.
// Every wait on an mbarrier is bounded; a wait that expires records an error word on the device
// (see wq_device_error) and the CTA skips the rest of its work, still releasing its tensor
// memory.
#include <algorithm>
#include <atomic>

#include "wq_tcgen05.cuh"

namespace wq {

__device__ int g_mx_error;          // 0, or the code of the first expired device wait

namespace {

constexpr int BM = 128;             // weight rows per CTA (MMA M)
constexpr int KB = 256;             // columns per stage: one 128-byte swizzle row of codes
constexpr int kThreads = 192;

template <int BN>
struct Cfg {
    static constexpr int A_BYTES = BM * KB / 2, B_BYTES = BN * KB / 2;
    static constexpr int STAGE = A_BYTES + B_BYTES;              // a multiple of 1024
    static constexpr int SC_BYTES = (BM + BN) * 16;
    static constexpr int STAGES = BN == 128 ? 3 : 4;             // room for two CTAs on an SM
    static constexpr int SSTAGES = STAGES / 2 + 1;
    // tensor memory: the accumulator, then TSLOTS slots of the scale bytes of 512 columns, per
    // 128 columns CH columns: 4 for the weight rows and BN / 32, rounded up to 4, for the
    // activation rows
    static constexpr int ACC_COLS = BN < 32 ? 32 : BN;
    static constexpr int XC = BN / 32 > 0 ? BN / 32 : 1;
    static constexpr int CH = 4 + (XC + 3) / 4 * 4;
    static constexpr int SLOT_COLS = 4 * CH;
    static constexpr int TSLOTS = BN <= 32 ? 3 : 4;
    static constexpr int USED_COLS = ACC_COLS + TSLOTS * SLOT_COLS;
    static constexpr uint32_t TMEM_COLS = USED_COLS <= 128 ? 128 : 256;
    static_assert(USED_COLS <= 256, "tensor memory of two CTAs");
    static constexpr int BARS = 2 * STAGES + 2 * SSTAGES + 2 * TSLOTS + 1;
    static constexpr int TOTAL = STAGES * STAGE + SSTAGES * SC_BYTES + BARS * 8 + 32 + 1024;   // + alignment slack
    static_assert(2 * (TOTAL + 1024) <= 228 * 1024, "shared memory of two CTAs");
};

// D[128 x BN] (+)= A B^T over 64 columns: codes through descriptors, scale bytes at the
// tensor-memory columns sfa / sfb (the byte pair of these columns is named in idesc).
__device__ __forceinline__ void umma_mxf4(uint32_t tmem_d, uint64_t da, uint64_t db, uint32_t idesc, uint32_t sfa,
                                          uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %6, 0; "
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p; }"
        ::"r"(tmem_d), "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The barrier alone, for CTAs whose memory needs no order (no fence behind pending stores).
__device__ __forceinline__ void cluster_sync_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_v4(uint32_t saddr, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

struct MxTile {
    int expert, t0, tend;            // expert (-1: none), first activation row, end of its rows
};

// Where a walk over the experts stands: those before e0 have `before` row tiles.
struct MxScan {
    int e0 = 0, before = 0;
};

// The row tile `mt` of all experts' tiles in order (warp-collective): expert e has
// ceil(rows / bn) tiles. Calls with one `at` ask for ascending mt. Offsets are clamped to
// [0, M], so no access leaves the buffers whatever they hold.
__device__ __forceinline__ MxTile find_tile(const int32_t* __restrict__ offsets, int experts, int M, int mt, int bn,
                                            MxScan& at) {
    const int lane = threadIdx.x & 31;
    for (; at.e0 < experts; at.e0 += 32) {
        const int e = at.e0 + lane;
        int lo = 0, hi = 0;
        if (e < experts) {
            lo = min(max(__ldg(offsets + e), 0), M);
            hi = min(max(__ldg(offsets + e + 1), lo), M);
        }
        const int tiles = (hi - lo + bn - 1) / bn;
        int incl = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += o;
        }
        const int total = __shfl_sync(0xFFFFFFFFu, incl, 31);
        if (mt < at.before + total) {
            const int f = max(0, __ffs(__ballot_sync(0xFFFFFFFFu, at.before + incl > mt)) - 1);
            const int t0 = __shfl_sync(0xFFFFFFFFu, lo + (mt - (at.before + incl - tiles)) * bn, f);
            lo = __shfl_sync(0xFFFFFFFFu, lo, f);
            hi = __shfl_sync(0xFFFFFFFFu, hi, f);
            return MxTile{t0 >= lo && t0 < hi ? at.e0 + f : -1, t0, hi};
        }
        at.before += total;
    }
    return MxTile{-1, 0, 0};
}

// Moves `at` to the group of consecutive experts, one of 32, that holds row tile `mt`: every lane
// adds up the tiles of its group, its loads independent of one another, where the walk would meet
// the memory's latency once every 32 experts.
__device__ __forceinline__ void skip_experts(const int32_t* __restrict__ offsets, int experts, int M, int mt, int bn,
                                             MxScan& at) {
    const int lane = threadIdx.x & 31, group = (experts + 31) / 32;
    const int e0 = min(experts, lane * group), e1 = min(experts, e0 + group);
    int tiles = 0;
#pragma unroll 8
    for (int e = e0; e < e1; ++e) {
        const int lo = min(max(__ldg(offsets + e), 0), M), hi = min(max(__ldg(offsets + e + 1), lo), M);
        tiles += (hi - lo + bn - 1) / bn;
    }
    int incl = tiles;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
        if (lane >= d) incl += o;
    }
    const int f = __ffs(__ballot_sync(0xFFFFFFFFu, incl > mt)) - 1;
    if (f < 0) {                                                 // there is no such tile
        at.e0 = experts;
        return;
    }
    at.e0 = f * group;
    at.before = __shfl_sync(0xFFFFFFFFu, incl - tiles, f);
}

// Activations as they come, for few rows (XQ): warps 2-5 quantise them on the way into the stage,
// a block of 32 columns a thread at a time, one or two scale stages ahead in registers. Every CTA
// of a row tile repeats that work; it saves the kernel in front, its workspace, and the wait for
// it (mx_quantises_itself says up to how many rows that pays).
struct XBlocks {
    static constexpr int PER = 2;                // blocks of 32 a thread has in 16 rows x 512 columns
    uint4 v[PER][4];
};
// Block j of thread m (0..127): activation row 8 j + m / 16, columns 32 (m % 16) .. + 31. Rows
// from `rows` on are left out: what their accumulator columns hold is not stored.
__device__ __forceinline__ void load_x_blocks(XBlocks& xb, const uint16_t* __restrict__ x, int m, int t0, int rows,
                                              int col0, int K) {
    const int col = col0 + 32 * (m % 16);
#pragma unroll
    for (int j = 0; j < XBlocks::PER; ++j) {
        const int row = 8 * j + m / 16;
        const uint16_t* p = x + (size_t)(t0 + row) * K + col;
#pragma unroll
        for (int i = 0; i < 4; ++i) xb.v[j][i] = row < rows && col < K ? ldg_v4(p + 8 * i) : make_uint4(0, 0, 0, 0);
    }
}
// 32 bf16 values -> their codes and scale byte, as the quantisation kernel makes them.
__device__ __forceinline__ uint32_t quantise32(const uint4 (&v)[4], uint4& codes) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        top = max_u16x2(top, max_u16x2(max_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                                       max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu)));
    const uint32_t s = mx_scale_byte(max(top & 0xFFFFu, top >> 16) >> 7);
    const float inv = mx_inverse_scale(s);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        float f[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[2 * j] = __uint_as_float(w[j] << 16) * inv;
            f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u) * inv;
        }
        c[i] = s == 255 ? 0u : e2m1x8(f);
    }
    codes = make_uint4(c[0], c[1], c[2], c[3]);
    return s;
}
// Barrier `id` of `threads` threads (whole warps) that also tells whether all of them are well.
__device__ __forceinline__ bool bar_all(int id, int threads, bool ok) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %3, 0; barrier.cta.red.and.pred q, %1, %2, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r) : "r"(id), "r"(threads), "r"((uint32_t)ok) : "memory");
    return r != 0;
}

template <int BN, int CL, bool EXPERTS, bool XQ>
__global__ void __launch_bounds__(kThreads, 2)
mx_gemm_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_ws,
               const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_xs,
               const uint16_t* __restrict__ x16, const int32_t* __restrict__ offsets, int experts,
               uint16_t* __restrict__ y, int M, int N, int K, int grid_n, int kt_per_split) {
    static_assert(!XQ || BN == 16, "few rows");
    static_assert(!EXPERTS || XQ, "experts otherwise run in pairs; so a CTA without a tile overlaps no kernel before it");
    // scale stages the activations are loaded ahead: two where a CTA walks all of K (28672 x 8192 at
    // 8 rows: 29.0 us one ahead, 25.0 two), one for experts (64 rows on 64 of 1408 x 2048: 19.4 / 21.2)
    constexpr int AHEAD = EXPERTS ? 1 : 2;
    using C = Cfg<BN>;
    constexpr uint32_t kScTx = XQ ? BM * 16 : C::SC_BYTES, kCodeTx = XQ ? C::A_BYTES : C::STAGE;
    constexpr int STAGES = C::STAGES, SS = C::SSTAGES, TS = C::TSLOTS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* sc_smem = smem + STAGES * C::STAGE;
    uint64_t* full = (uint64_t*)(sc_smem + SS * C::SC_BYTES);   // codes of a stage landed
    uint64_t* empty = full + STAGES;                             // ... and read by their MMAs
    uint64_t* sfull = empty + STAGES;                            // scale bytes of 512 columns landed
    uint64_t* sempty = sfull + SS;                               // ... and read by the movers
    uint64_t* tfull = sempty + SS;                               // scale bytes in tensor memory
    uint64_t* tfree = tfull + TS;                                // ... and read by their MMAs
    uint64_t* acc_full = tfree + TS;
    uint32_t* s_tmem = (uint32_t*)(acc_full + 1);
    int* s_abort = (int*)(s_tmem + 1);
    int* s_tile = s_abort + 1;                                   // expert, t0, tend

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lin = (int)blockIdx.x;
    const int n0 = (lin % grid_n) * BM;
    const int crank = CL > 1 ? (int)cluster_rank() : 0;
    if (threadIdx.x == 32) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < SS; ++s) { mbar_init(&sfull[s], 1); mbar_init(&sempty[s], 4); }
        for (int s = 0; s < TS; ++s) { mbar_init(&tfull[s], 4); mbar_init(&tfree[s], 1); }
        mbar_init(acc_full, 1);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        prefetch_map(&map_w); prefetch_map(&map_ws);
        if (!XQ) { prefetch_map(&map_x); prefetch_map(&map_xs); }
    }
    MxTile tile{0, (lin / grid_n) * BN, M};
    if (EXPERTS) {
        if (warp == 0) {
            MxScan at;
            // (64 experts, 25 with rows: 11.8 us by the walk alone, 13.4 with this in front)
            if (experts > 64) skip_experts(offsets, experts, M, lin / grid_n, BN, at);
            tile = find_tile(offsets, experts, M, lin / grid_n, BN, at);
            if (lane == 0) { s_tile[0] = tile.expert; s_tile[1] = tile.t0; s_tile[2] = tile.tend; }
        }
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(s_tmem)), "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;");
    }
    __syncthreads();
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = *s_tmem;
    if (EXPERTS) {
        tile = MxTile{s_tile[0], s_tile[1], s_tile[2]};
        if (tile.expert < 0) {                                   // (clusters are not used here)
            if (warp == 1)
                asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
            return;
        }
    }
    const int KT = (K + KB - 1) / KB;
    const int kt0 = crank * kt_per_split;                        // even: scale stages do not straddle splits
    const int nk = max(0, min(KT, kt0 + kt_per_split) - kt0);
    const int t0 = tile.t0, tend = tile.tend;
    const int w0 = tile.expert * N + n0;                         // first weight row of the tile in the stack
    XBlocks xb0, xb1;                                            // of the scale stages in turn
    if (XQ && warp >= 2) {
        load_x_blocks(xb0, x16, (int)threadIdx.x - 64, t0, tend - t0, kt0 * KB, K);
        if (AHEAD == 2 && nk > 2) load_x_blocks(xb1, x16, (int)threadIdx.x - 64, t0, tend - t0, (kt0 + 2) * KB, K);
    }

    auto stage_a = [&](int s) { return smem + s * C::STAGE; };
    auto stage_b = [&](int s) { return smem + s * C::STAGE + C::A_BYTES; };
    auto stage_sc = [&](int s) { return sc_smem + s * C::SC_BYTES; };
    auto dead = [&](int code) {
        *(volatile int*)s_abort = 1;
        atomicCAS(&g_mx_error, 0, code);
    };

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        const bool one = elect_one();
        // the weights of the first stages: they do not depend on the kernel before this one
        const int pre = min(nk, STAGES);
        if (one) {
            for (int i = 0; i < pre; ++i) {
                if ((i & 1) == 0) {
                    mbar_expect_tx(&sfull[i >> 1], kScTx);
                    tma_load_2d(stage_sc(i >> 1), &map_ws, ((kt0 + i) >> 1) * 16, w0, &sfull[i >> 1]);
                }
                mbar_expect_tx(&full[i], kCodeTx);
                tma_load_2d(stage_a(i), &map_w, (kt0 + i) * (KB / 2), w0, &full[i]);
            }
            asm volatile("griddepcontrol.wait;" ::: "memory");
            for (int i = 0; !XQ && i < pre; ++i) {
                if ((i & 1) == 0)
                    tma_load_2d(stage_sc(i >> 1) + BM * 16, &map_xs, ((kt0 + i) >> 1) * 16, t0, &sfull[i >> 1]);
                tma_load_2d(stage_b(i), &map_x, (kt0 + i) * (KB / 2), t0, &full[i]);
            }
        }
        __syncwarp();
        int s = 0, ss = ((STAGES + 1) / 2) % SS;
        uint32_t ph = 1, sph = (STAGES + 1) / 2 >= SS ? 1 : 0;    // parity of the stage's use
        int i = pre, sdone = (pre + 1) / 2;                       // stages and scale stages asked for
        for (; i < nk; ++i) {
            if ((i & 1) == 0) {
                if (!warp_wait(&sempty[ss], sph ^ 1, s_abort)) { dead(2201); break; }
                if (one) {
                    mbar_expect_tx(&sfull[ss], kScTx);
                    tma_load_2d(stage_sc(ss), &map_ws, ((kt0 + i) >> 1) * 16, w0, &sfull[ss]);
                    if (!XQ) tma_load_2d(stage_sc(ss) + BM * 16, &map_xs, ((kt0 + i) >> 1) * 16, t0, &sfull[ss]);
                }
                __syncwarp();
                ++sdone;
                if (++ss == SS) { ss = 0; sph ^= 1; }
            }
            if (!warp_wait(&empty[s], ph ^ 1, s_abort)) { dead(2202); break; }
            if (one) {
                mbar_expect_tx(&full[s], kCodeTx);
                tma_load_2d(stage_a(s), &map_w, (kt0 + i) * (KB / 2), w0, &full[s]);
                if (!XQ) tma_load_2d(stage_b(s), &map_x, (kt0 + i) * (KB / 2), t0, &full[s]);
            }
            __syncwarp();
            if (++s == STAGES) { s = 0; ph ^= 1; }
        }
        if (i < nk) {
            // gave up: the copies in flight must land before the CTA may end
            for (int j = max(0, i - STAGES); j < i; ++j) mbar_wait(&full[j % STAGES], (j / STAGES) & 1);
            for (int j = max(0, sdone - SS); j < sdone; ++j) mbar_wait(&sfull[j % SS], (j / SS) & 1);
        }
    } else if (warp == 1) {
        // ---------------- MMA issuer ----------------
        // E2M1 codes (format 1) in both operands, E8M0 scales, fp32 accumulator
        constexpr uint32_t idesc0 = (1u << 7) | (1u << 10) | ((uint32_t)(BN >> 3) << 17) | (1u << 23) |
                                    ((uint32_t)(BM >> 4) << 24);
        const bool one = elect_one();
        int s = 0, t = 0;
        uint32_t ph = 0, tph = 0;
        for (int i = 0; i < nk; ++i) {
            if ((i & 1) == 0 && !warp_wait(&tfull[t], tph, s_abort)) { dead(2203); break; }
            if (!warp_wait(&full[s], ph, s_abort)) { dead(2204); break; }
            asm volatile("tcgen05.fence::after_thread_sync;");
            const uint64_t da = sw128_desc(smem_u32(stage_a(s))), db = sw128_desc(smem_u32(stage_b(s)));
            const uint32_t sf = tmem + (uint32_t)(C::ACC_COLS + t * C::SLOT_COLS + (i & 1) * 2 * C::CH);
            const int left = (K - (kt0 + i) * KB) / 64;           // K is a multiple of 64
            // 64 codes are 32 bytes of the swizzle row: + 2 in descriptor units; bytes 0-1 or 2-3 of
            // the scale words
            auto mma = [&](int j) {
                const uint32_t id = (uint32_t)(j & 1) * 2u, sfa = sf + (uint32_t)((j >> 1) * C::CH);
                umma_mxf4(tmem, da + 2 * j, db + 2 * j, idesc0 | id << 4 | id << 29, sfa, sfa + 4,
                          (i > 0 || j > 0) ? 1u : 0u);
            };
            if (one) {
                if (left >= 4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) mma(j);
                } else {
                    for (int j = 0; j < left; ++j) mma(j);
                }
                umma_commit(&empty[s]);                           // fire once these MMAs are done
                if ((i & 1) || i + 1 == nk) umma_commit(&tfree[t]);
            }
            __syncwarp();
            if (++s == STAGES) { s = 0; ph ^= 1; }
            if ((i & 1) && ++t == TS) { t = 0; tph ^= 1; }
        }
        // a commit also after giving up: it fires once every MMA issued so far is done, so tensor
        // memory is never freed under a running MMA
        if (one) umma_commit(acc_full);
        __syncwarp();
    } else {
        // ---------------- scale bytes into tensor memory, then the epilogue ----------------
        const int q = warp & 3;                                   // this warp's lane quarter
        const uint32_t lane_base = tmem + ((uint32_t)(32 * q) << 16);
        int ss = 0, t = 0, cs = 0;                                // scale stage, slot, code stage (XQ)
        uint32_t sph = 0, tph = 0, cph = 0;
        const int nt = (nk + 1) / 2;
        auto move = [&](int it, XBlocks& xb) {
            bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&sfull[ss], sph, s_abort) &&
                                              (it < TS || mbar_wait(&tfree[t], tph ^ 1, s_abort)));
            if (XQ) {
                const int m = (int)threadIdx.x - 64, b = m % 16;  // (b: block of the scale stage)
                // the scale stage's code stages, each free again
                const bool two = 2 * it + 1 < nk;
                ok = ok && warp_wait(&empty[cs], cph ^ 1, s_abort);
                int cs1 = cs + 1;
                uint32_t cph1 = cph;
                if (cs1 == STAGES) { cs1 = 0; cph1 ^= 1; }
                if (two) ok = ok && warp_wait(&empty[cs1], cph1 ^ 1, s_abort);
                if (ok && (b < 8 || two)) {
                    uint8_t* tile_b = stage_b(b < 8 ? cs : cs1);
#pragma unroll
                    for (int j = 0; j < XBlocks::PER; ++j) {
                        const int row = 8 * j + m / 16;
                        if (t0 + row < tend) {
                            uint4 codes;
                            const uint32_t sb = quantise32(xb.v[j], codes);
                            // the 128-byte swizzle of the tile's rows
                            *(uint4*)(tile_b + row * 128 + (((b & 7) ^ (row & 7)) * 16)) = codes;
                            stage_sc(ss)[BM * 16 + row * 16 + b] = (uint8_t)sb;
                        }
                    }
                }
                cs = cs1 + 1;
                cph = cph1;
                if (cs == STAGES) { cs = 0; cph ^= 1; }
                if (it + AHEAD < nt)
                    load_x_blocks(xb, x16, m, t0, tend - t0, (kt0 + 2 * (it + AHEAD)) * KB, K);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // the MMAs read the codes
                ok = bar_all(1, 128, ok);                         // warps 2-5
            }
            if (!ok) { dead(2205); return false; }
            const uint4* sc = (const uint4*)stage_sc(ss);
            uint32_t v[C::SLOT_COLS];
#pragma unroll
            for (int j = 0; j < C::SLOT_COLS; ++j) v[j] = 0;
#pragma unroll
            for (int j = 0; j < 4 + C::XC; ++j) {                 // 32 rows each: the weights', then the activations'
                uint4 r = make_uint4(0, 0, 0, 0);
                if (BN >= 32 || j < 4 || lane < BN) r = sc[32 * j + lane];
                v[j] = r.x; v[C::CH + j] = r.y; v[2 * C::CH + j] = r.z; v[3 * C::CH + j] = r.w;
            }
            const uint32_t dst = lane_base + (uint32_t)(C::ACC_COLS + t * C::SLOT_COLS);
            tmem_st_part<C::SLOT_COLS>(dst, v);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) { mbar_arrive(&sempty[ss]); mbar_arrive(&tfull[t]); }
            if (++ss == SS) { ss = 0; sph ^= 1; }
            if (++t == TS) { t = 0; tph ^= 1; }
            return true;
        };
        for (int it = 0; it < nt; ++it) {
            if (!move(it, xb0)) break;
            if (XQ && AHEAD == 2 && (++it == nt || !move(it, xb1))) break;
        }
        const bool drain = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, 0)) &&
                           !__any_sync(0xFFFFFFFFu, *(volatile int*)s_abort != 0);
        if (drain) {
            asm volatile("tcgen05.fence::after_thread_sync;");
            const int i = 32 * q + lane, n = n0 + i;
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 16) {
                uint32_t v[16];
                if (CL == 1 && t0 + c0 >= tend) break;            // (the same for the whole CTA)
                tmem_ld16(lane_base + (uint32_t)c0, v);
                asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    if (CL > 1)                                   // the stages are free: partial sums [BN][BM]
                        ((float*)smem)[(c0 + j) * BM + i] = nk > 0 ? __uint_as_float(v[j]) : 0.f;
                    else if (n < N && t0 + c0 + j < tend)
                        y[(size_t)(t0 + c0 + j) * N + n] = (uint16_t)float_to_bf16_bits(__uint_as_float(v[j]));
                }
            }
        } else {
            dead(2206);
        }
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncwarp();
    if (CL > 1) {
        cluster_sync();                                           // every rank's partial sums are in place
        if (warp >= 2) {
            // rank r adds the activation rows r, r + CL, ...: one of them a warp, 4 weight rows a lane
            const int n = n0 + 4 * lane;
            const uint32_t base = smem_u32(smem) + 16u * (uint32_t)lane;
#pragma unroll 2
            for (int c = crank + CL * (warp - 2); c < BN; c += 4 * CL) {
                if (t0 + c >= tend) break;
                float4 v[CL];
#pragma unroll
                for (int r = 0; r < CL; ++r) v[r] = ld_cluster_v4(base + (uint32_t)(c * BM * 4), r);
                float4 sum = v[0];
#pragma unroll
                for (int r = 1; r < CL; ++r) { sum.x += v[r].x; sum.y += v[r].y; sum.z += v[r].z; sum.w += v[r].w; }
                uint16_t* yr = y + (size_t)(t0 + c) * N;
                const uint2 o = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                if ((N & 3) == 0) {
                    if (n < N) *(uint2*)(yr + n) = o;
                } else {
                    if (n < N) yr[n] = (uint16_t)o.x;
                    if (n + 1 < N) yr[n + 1] = (uint16_t)(o.x >> 16);
                    if (n + 2 < N) yr[n + 2] = (uint16_t)o.y;
                    if (n + 3 < N) yr[n + 3] = (uint16_t)(o.y >> 16);
                }
            }
        }
        __syncwarp();
        cluster_sync_relaxed();                                   // ... and read
    }
    __syncthreads();
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
    }
}

// ---------------------------------------------------------------------------------------
// Many activation rows: pairs of CTAs (cta_group::2) on tiles of 256 weight rows x bn <= 256
// activation rows, walked by a persistent grid. Each CTA of a pair holds half of the weight
// rows and half of the activation rows in shared memory and accumulates its 128 weight rows x
// bn: per MMA of 64 columns it reads (128 + bn / 2) x 32 bytes where a single CTA reads (128 + bn)
// x 32. At 256 x 256 that is 64 bytes a clock, and the copies into shared memory take as many
// again, of the 128 there are; a single CTA's 128 x 256 tile would want 192. There the MMAs bound
// the main loop: by their rate a stage of four takes 0.27 us at 1.9 GHz (128 clocks each), measured
// 0.29. Narrower tiles' stages take less, down to a floor that is not the MMAs': 0.26 us at 192
// wide, 0.20 from 160 down to 32 (9728 weight rows in L2, K 8192 less K 4096). 5.4 PFLOP/s over
// 4096 x 4096 x 11008 again and again (5.2 on three sets of inputs in turn), at the power limit.
// With short K the way from tile to tile counts: 8192 x 5632 x 2048 takes 4.4 us a tile, 2.3 of them
// its eight stages, as the one accumulator is taken out before the next tile's first MMA.
//   warp 0      TMA producer of its CTA's codes (both CTAs signal the leader's barrier);
//   warp 1      MMA issuer (the leader's CTA only), commits to both CTAs;
//   warps 2-5   scale bytes into tensor memory: the CTA's 128 weight rows and all activation rows;
//   warps 6-13  epilogue: the accumulator into registers as bf16, which frees it for the next
//               tile, then transposed (stmatrix) into rows of 64 weight rows, which TMA stores;
//   warp 14     TMA producer of the scale bytes, on rings of its own: a stage's codes take about
//               1.3 us to come, its scales longer, through two hands, so they start earlier.
// ---------------------------------------------------------------------------------------
struct Pair {
    static constexpr int THREADS = 480;
    static constexpr int TILE_A = BM * 128;                      // 128 weight rows x 256 columns of codes
    static constexpr int CODE_BYTES = 5 * 2 * TILE_A;            // 5 stages of 256 rows, more of fewer
    static constexpr int MAX_STAGES = 10;
    static constexpr int SS = 4, TS = 4;                         // scale stages (512 columns) in shared / tensor memory
    static constexpr int SC_BYTES = (BM + 256) * 16;
    // tensor memory: the accumulator, then per scale stage the bytes of 4 x 128 columns, 4
    // columns for the weight rows and 8 for the activation rows each
    static constexpr int CH = 12, SLOT_COLS = 4 * CH, ACC_COLS = 256;
    static constexpr int EPI_TILE = 32 * 128;                    // 32 activation rows x 64 weight rows of bf16
    static constexpr int BARS = 2 * MAX_STAGES + 2 * SS + 2 * TS + 2;
    static constexpr int TOTAL = CODE_BYTES + 8 * EPI_TILE + SS * SC_BYTES + BARS * 8 + 16 + 1024;
    static_assert(ACC_COLS + TS * SLOT_COLS <= 512, "tensor memory");
    static_assert(TOTAL <= 227 * 1024, "shared memory");
};

__device__ __forceinline__ uint32_t leader_addr(const void* p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
// (A release at cluster scope would stand here too, and cost a fence a time: measured 0.17 us a
// stage. What crosses CTAs is ordered by the tcgen05 fences around the arrival.)
__device__ __forceinline__ void mbar_arrive_leader(const uint64_t* b) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(leader_addr(b)) : "memory");
}
// A tile into this CTA's shared memory, its bytes counted on the leader's barrier `bar`.
__device__ __forceinline__ void tma_load_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(c0), "r"(c1), "r"(bar) : "memory");
}
__device__ __forceinline__ void umma_commit_pair(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}
// da, db: the low words of descriptors whose high word is `hi`.
__device__ __forceinline__ void umma_mxf4_pair(uint32_t tmem_d, uint32_t da, uint32_t db, uint32_t hi, uint32_t idesc,
                                               uint32_t sfa, uint32_t sfb, uint32_t accumulate) {
    asm volatile(
        "{ .reg .pred p; .reg .b64 a, b; mov.b64 a, {%1, %3}; mov.b64 b, {%2, %3}; setp.ne.b32 p, %7, 0; "
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%5], [%6], p; }"
        ::"r"(tmem_d), "r"(da), "r"(db), "r"(hi), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate));
}
// Whether the three phases are complete, by the whole warp and without waiting.
__device__ __forceinline__ bool warp_test3(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb, uint64_t* c, uint32_t pc) {
    uint32_t done;
    asm volatile(
        "{ .reg .pred p, q, r; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; "
        "mbarrier.test_wait.parity.shared::cta.b64 q, [%3], %4; mbarrier.test_wait.parity.shared::cta.b64 r, [%5], %6; "
        "and.pred p, p, q; and.pred p, p, r; selp.u32 %0, 1, 0, p; }"
        : "=r"(done)
        : "r"(smem_u32(a)), "r"(pa), "r"(smem_u32(b)), "r"(pb), "r"(smem_u32(c)), "r"(pc) : "memory");
    return __all_sync(0xFFFFFFFFu, done != 0);
}

template <bool EXPERTS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Pair::THREADS, 1)
mx_gemm_pair_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_ws,
                    const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_xs,
                    const __grid_constant__ CUtensorMap map_y,
                    const int32_t* __restrict__ offsets, int experts, uint16_t* __restrict__ y, int M, int N, int K,
                    int grid_n, int grid_m, int bn) {
    using C = Pair;
    constexpr int SS = C::SS, TS = C::TS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* epi_smem = smem + C::CODE_BYTES;
    uint8_t* sc_smem = epi_smem + 8 * C::EPI_TILE;
    uint64_t* full = (uint64_t*)(sc_smem + SS * C::SC_BYTES);   // (leader's) codes of both CTAs' stage landed
    uint64_t* empty = full + C::MAX_STAGES;                      // stage read by its MMAs
    uint64_t* sfull = empty + C::MAX_STAGES;                     // scale bytes of 512 columns landed
    uint64_t* sempty = sfull + SS;                               // ... and read by the movers
    uint64_t* tfull = sempty + SS;                               // (leader's) both CTAs' scales in tensor memory
    uint64_t* tfree = tfull + TS;                                // ... and read by their MMAs
    uint64_t* acc_full = tfree + TS;
    uint64_t* acc_free = acc_full + 1;                           // (leader's) both accumulators read
    uint32_t* s_tmem = (uint32_t*)(acc_free + 1);
    int* s_abort = (int*)(s_tmem + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    if (threadIdx.x == 32) {
        for (int s = 0; s < C::MAX_STAGES; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
        for (int s = 0; s < SS; ++s) { mbar_init(&sfull[s], 1); mbar_init(&sempty[s], 4); }
        for (int s = 0; s < TS; ++s) { mbar_init(&tfull[s], 8); mbar_init(&tfree[s], 1); }
        mbar_init(acc_full, 1);
        mbar_init(acc_free, 16);
        *s_abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (threadIdx.x == 0) {
        prefetch_map(&map_w); prefetch_map(&map_ws); prefetch_map(&map_x); prefetch_map(&map_xs); prefetch_map(&map_y);
    }
    __syncwarp();
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s_tmem)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.fence::before_thread_sync;");
    }
    __syncthreads();
    cluster_sync_relaxed();                                      // the peer's barriers are ready too
    asm volatile("tcgen05.fence::after_thread_sync;");
    const uint32_t tmem = *s_tmem;
    const int nk = (K + KB - 1) / KB, nsk = (nk + 1) / 2;        // stages and scale stages of a tile
    const int step = (int)gridDim.x / 2;
    const uint32_t b_bytes = (uint32_t)bn * 64, stage_bytes = C::TILE_A + b_bytes;   // bn / 2 rows of 128 bytes
    const int stages = min(C::MAX_STAGES, (int)(C::CODE_BYTES / stage_bytes));

    auto stage_a = [&](int s) { return smem + s * stage_bytes; };
    auto stage_b = [&](int s) { return smem + s * stage_bytes + C::TILE_A; };
    auto stage_sc = [&](int s) { return sc_smem + s * C::SC_BYTES; };
    auto dead = [&](int code) {
        *(volatile int*)s_abort = 1;
        atomicCAS(&g_mx_error, 0, code);
    };
    MxScan at;
    if (EXPERTS && experts > 64) skip_experts(offsets, experts, M, (int)blockIdx.x / 2 / grid_n, bn, at);
    // tile number `lin`: its weight-row tile nt (fastest) and its activation rows; false: none
    auto get = [&](int lin, int& n0, MxTile& t) {
        n0 = (lin % grid_n) * 256 + rank * BM;
        const int mt = lin / grid_n;
        if (EXPERTS) {
            t = find_tile(offsets, experts, M, mt, bn, at);
            return t.expert >= 0;
        }
        t = MxTile{0, mt * bn, M};
        return mt < grid_m;
    };

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        const bool one = elect_one();
        int s = 0, done = 0;                                     // stages asked for
        uint32_t ph = 0;
        bool ok = true;
        int n0;
        MxTile t;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int lin = (int)blockIdx.x / 2; ok && get(lin, n0, t); lin += step) {
            const int w0 = t.expert * N + n0, x0 = t.t0 + rank * (bn / 2);
            for (int i = 0; i < nk; ++i) {
                if (!warp_wait(&empty[s], ph ^ 1, s_abort)) { dead(2211); ok = false; break; }
                if (one) {
                    if (rank == 0) mbar_expect_tx(&full[s], 2 * stage_bytes);
                    const uint32_t bar = leader_addr(&full[s]);
                    tma_load_pair(stage_a(s), &map_w, i * (KB / 2), w0, bar);
                    tma_load_pair(stage_b(s), &map_x, i * (KB / 2), x0, bar);
                }
                __syncwarp();
                ++done;
                if (++s == stages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok && rank == 0)                                     // gave up: the copies in flight must land first
            for (int j = max(0, done - stages); j < done; ++j) mbar_wait(&full[j % stages], (j / stages) & 1);
    } else if (warp == 14) {
        // ---------------- TMA producer of the scale bytes ----------------
        const bool one = elect_one();
        int ss = 0, done = 0, n0;
        uint32_t ph = 0;
        bool ok = true;
        MxTile t;
        asm volatile("griddepcontrol.wait;" ::: "memory");
        for (int lin = (int)blockIdx.x / 2; ok && get(lin, n0, t); lin += step) {
            for (int i = 0; i < nsk; ++i) {
                if (!warp_wait(&sempty[ss], ph ^ 1, s_abort)) { dead(2212); ok = false; break; }
                if (one) {
                    mbar_expect_tx(&sfull[ss], (uint32_t)(BM + bn) * 16);
                    tma_load_2d(stage_sc(ss), &map_ws, i * 16, t.expert * N + n0, &sfull[ss]);
                    tma_load_2d(stage_sc(ss) + BM * 16, &map_xs, i * 16, t.t0, &sfull[ss]);
                }
                __syncwarp();
                ++done;
                if (++ss == SS) { ss = 0; ph ^= 1; }
            }
        }
        if (!ok)
            for (int j = max(0, done - SS); j < done; ++j) mbar_wait(&sfull[j % SS], (j / SS) & 1);
    } else if (warp == 1) {
        // ---------------- MMA issuer (leader) ----------------
        if (rank == 0) {
            const uint32_t idesc0 = (1u << 7) | (1u << 10) | ((uint32_t)(bn >> 3) << 17) | (1u << 23) |
                                    ((uint32_t)(256 >> 4) << 24);
            int s = 0, ts = 0;
            uint32_t ph = 0, tph = 0, aph = 1;
            bool ok = true;
            int n0;
            MxTile t;
            const bool one = elect_one();
            const uint64_t desc = sw128_desc(smem_u32(smem));
            const uint32_t desc_lo = (uint32_t)desc, desc_hi = (uint32_t)(desc >> 32);
            for (int lin = (int)blockIdx.x / 2; ok && get(lin, n0, t); lin += step) {
                if (!warp_wait(acc_free, aph, s_abort)) { dead(2213); ok = false; }
                // two stages a turn (the columns of one scale stage): the issuing thread's own time is
                // what a stage must not exceed, and each wait, ready or not, takes it 140 clocks
                for (int i = 0; ok && i < nk; i += 2) {
                    const bool two = i + 1 < nk;
                    const int s1 = !two ? s : s + 1 == stages ? 0 : s + 1;
                    const uint32_t ph1 = s1 < s ? ph ^ 1 : ph;
                    const bool ready = warp_test3(&tfull[ts], tph, &full[s], ph, &full[s1], ph1);
                    if (!ready) {
                        if (!warp_wait(&tfull[ts], tph, s_abort)) { dead(2214); ok = false; break; }
                        if (!warp_wait(&full[s], ph, s_abort)) { dead(2215); ok = false; break; }
                    }
                    asm volatile("tcgen05.fence::after_thread_sync;");
                    const uint32_t sf = tmem + (uint32_t)(C::ACC_COLS + ts * C::SLOT_COLS);
                    const int left = (K - i * KB) / 64;           // K is a multiple of 64
                    // 64 columns: j / 4 picks the stage (d: its descriptor words), j / 2 the scale words,
                    // j % 2 their bytes
                    auto mma = [&](int j, uint32_t d) {
                        const uint32_t id = (uint32_t)(j & 1) * 2u, sfa = sf + (uint32_t)((j >> 1) * C::CH);
                        umma_mxf4_pair(tmem, d + 2 * (j & 3), d + C::TILE_A / 16 + 2 * (j & 3), desc_hi,
                                       idesc0 | id << 4 | id << 29, sfa, sfa + 4, (i > 0 || j > 0) ? 1u : 0u);
                    };
                    const uint32_t d0 = desc_lo + (uint32_t)s * (stage_bytes / 16);
                    if (one) {
                        if (left >= 4) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) mma(j, d0);
                        } else {
                            for (int j = 0; j < left; ++j) mma(j, d0);
                        }
                        umma_commit_pair(&empty[s]);
                    }
                    __syncwarp();
                    if (two) {
                        if (!ready && !warp_wait(&full[s1], ph1, s_abort)) { dead(2215); ok = false; break; }
                        const uint32_t d1 = desc_lo + (uint32_t)s1 * (stage_bytes / 16);
                        if (one) {
                            if (left >= 8) {
#pragma unroll
                                for (int j = 4; j < 8; ++j) mma(j, d1);
                            } else {
                                for (int j = 4; j < left; ++j) mma(j, d1);
                            }
                            umma_commit_pair(&empty[s1]);
                        }
                        __syncwarp();
                    }
                    if (one) umma_commit_pair(&tfree[ts]);
                    __syncwarp();
                    ph = ph1;
                    s = s1 + 1;
                    if (s == stages) { s = 0; ph ^= 1; }
                    if (++ts == TS) { ts = 0; tph ^= 1; }
                }
                // (also after giving up, and then waited for: tensor memory is not freed under a
                // running MMA)
                if (one) umma_commit_pair(acc_full);
                __syncwarp();
                if (!ok) mbar_wait(acc_full, aph ^ 1);
                aph ^= 1;
            }
        }
    } else if (warp < 6) {
        // ---------------- scale bytes into tensor memory ----------------
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        int ss = 0, ts = 0, n0;
        uint32_t sph = 0, tph = 1;
        bool ok = true;
        MxTile t;
        for (int lin = (int)blockIdx.x / 2; ok && get(lin, n0, t); lin += step) {
            for (int i = 0; i < nsk; ++i) {
                ok = warp_wait(&sfull[ss], sph, s_abort) && warp_wait(&tfree[ts], tph, s_abort);
                if (!ok) { dead(2216); break; }
                const uint4* sc = (const uint4*)stage_sc(ss);
                uint32_t v[C::SLOT_COLS];
#pragma unroll
                for (int j = 0; j < C::CH; ++j) {                 // (rows past bn: columns that no MMA reads)
                    const uint4 r = sc[32 * j + lane];
                    v[j] = r.x; v[C::CH + j] = r.y; v[2 * C::CH + j] = r.z; v[3 * C::CH + j] = r.w;
                }
                const uint32_t dst = lane_base + (uint32_t)(C::ACC_COLS + ts * C::SLOT_COLS);
                tmem_st_part<32>(dst, v);
                tmem_st_part<16>(dst + 32, v + 32);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
                __syncwarp();
                if (lane == 0) { mbar_arrive(&sempty[ss]); mbar_arrive_leader(&tfull[ts]); }
                if (++ss == SS) { ss = 0; sph ^= 1; }
                if (++ts == TS) { ts = 0; tph ^= 1; }
            }
        }
    } else {
        // ---------------- epilogue ----------------
        const int q = warp & 3, h = (warp - 6) >> 2;              // lane quarter; columns 128 h .. 128 h + 127
        const uint32_t src = tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)(128 * h);
        // two warps of neighbouring quarters fill a store tile together (barrier `id`), in two
        // buffers in turn; its first warp's lane 0 issues the stores
        const int team = 2 * h + (q >> 1), id = 1 + team;
        const bool issuer = (q & 1) == 0 && lane == 0;
        uint8_t* bufs = epi_smem + 2 * team * C::EPI_TILE;
        const bool wide = (N & 7) == 0;                           // rows of y are then 16-byte aligned
        uint32_t aph = 0, flip = 0;
        bool ok = true;
        int n0;
        MxTile t;
        for (int lin = (int)blockIdx.x / 2; ok && get(lin, n0, t); lin += step, aph ^= 1) {
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(acc_full, aph, s_abort)) &&
                 !__any_sync(0xFFFFFFFFu, *(volatile int*)s_abort != 0);
            if (!bar_all(id, 64, ok)) { ok = false; dead(2217); break; }
            asm volatile("tcgen05.fence::after_thread_sync;");
            // activation rows of this tile that this warp holds
            const int rows = min(min(bn - 128 * h, 128), t.tend - t.t0 - 128 * h);
            // p[16 c + 4 g + 2 l + r]: weight rows 16 l + 8 r .. + 7 of the quarter, activation rows 32 c +
            // 8 g .. + 7, as the 8 x 8 fragments that stmatrix takes
            uint32_t p[64];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (32 * c < rows) {
                    uint32_t v[2][16];
                    tmem_ld_16x256b_x4(src + 32u * (uint32_t)c, v[0]);
                    tmem_ld_16x256b_x4(src + 32u * (uint32_t)c + (16u << 16), v[1]);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int g = 0; g < 4; ++g)
#pragma unroll
                        for (int l = 0; l < 2; ++l)
#pragma unroll
                            for (int r = 0; r < 2; ++r)
                                p[16 * c + 4 * g + 2 * l + r] =
                                    pack_bf16x2(__uint_as_float(v[l][4 * g + 2 * r]), __uint_as_float(v[l][4 * g + 2 * r + 1]));
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive_leader(acc_free);
            const int nt = n0 + 64 * (q >> 1);                    // the store tile's first weight row
            const int r0 = t.t0 + 128 * h;                        // ... and activation row
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (32 * c >= rows) break;
                uint8_t* buf = bufs + flip * C::EPI_TILE;
                flip ^= 1;
                // 128-byte rows in the swizzle that the store undoes, free of bank conflicts
#pragma unroll
                for (int g = 0; g < 2; ++g)
#pragma unroll
                    for (int l = 0; l < 2; ++l) {
                        const int row = 16 * g + 8 * (lane >> 4) + (lane & 7), col = 4 * (q & 1) + 2 * l + ((lane >> 3) & 1);
                        const uint32_t* f = p + 16 * c + 8 * g + 2 * l;
                        stmatrix_x4_trans(smem_u32(buf) + (uint32_t)(row * 128 + ((col ^ (row & 7)) * 16)), f[0], f[1], f[4], f[5]);
                    }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                // the other buffer's store has been read out by the time anyone passes
                if (issuer) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                bar_all(id, 64, true);
                if (wide && 32 * c + 32 <= rows) {
                    if (issuer && nt < N) {
                        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];"
                                     ::"l"(&map_y), "r"(nt), "r"(r0 + 32 * c), "r"(smem_u32(buf)) : "memory");
                        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                    }
                    __syncwarp();
                } else {
                    // the last rows of an expert (or of all), or rows of y that are not aligned
                    const int m = 32 * (q & 1) + lane;
                    const int left = min(32, rows - 32 * c);
                    uint16_t* yt = y + (size_t)(r0 + 32 * c) * N + nt;
                    if (wide) {
                        for (int row = m >> 3; row < left; row += 8)
                            if (nt + 8 * (m & 7) < N)
                                *(uint4*)(yt + (size_t)row * N + 8 * (m & 7)) =
                                    *(const uint4*)(buf + row * 128 + (((m & 7) ^ (row & 7)) * 16));
                    } else if (nt + m < N) {
                        for (int row = 0; row < left; ++row)
                            yt[(size_t)row * N + m] =
                                *(const uint16_t*)(buf + row * 128 + (((m >> 3) ^ (row & 7)) * 16) + 2 * (m & 7));
                    }
                    __syncwarp();
                }
            }
        }
        if (issuer) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    asm volatile("tcgen05.fence::before_thread_sync;");
    __syncwarp();
    cluster_sync_relaxed();                                      // no signal is under way to either CTA
    if (warp == 1) {
        asm volatile("tcgen05.fence::after_thread_sync;");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------

struct Maps {
    CUtensorMap w, ws, x, xs, y;
};

wq_status encode(CUtensorMap* map, CUtensorMapDataType type, int size, const void* base, int64_t cols, int64_t rows,
                 int box_cols, int box_rows, bool swizzle, const char* what) {
    auto enc = tensor_map_encoder();
    if (!enc) return fail(WQ_ECUDA, "cuTensorMapEncodeTiled is unavailable from the driver");
    cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)cols * (cuuint64_t)size};
    cuuint32_t box[2] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows};
    cuuint32_t es[2] = {1, 1};
    const CUresult r = enc(map, type, 2, (void*)base, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(WQ_ECUDA, "tensor map for %s failed (%d)", what, (int)r);
    return WQ_OK;
}
wq_status encode_u8(CUtensorMap* map, const void* base, int64_t row_bytes, int64_t rows, int box_bytes, int box_rows,
                    bool swizzle, const char* what) {
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, base, row_bytes, rows, box_bytes, box_rows, swizzle, what);
}

// Opts the kernel in to `bytes` of shared memory on the current device, once for each device
// (`raised`: one bit a device, per kernel).
template <typename Kernel>
void raise_smem(Kernel k, int bytes, std::atomic<uint64_t>& raised) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev > 63) dev = 63;
    const uint64_t bit = (uint64_t)1 << dev;
    if ((raised.load(std::memory_order_relaxed) & bit) && dev != 63) return;
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess)
        raised.fetch_or(bit, std::memory_order_relaxed);
}

template <int BN, int CL, bool EXPERTS, bool XQ>
wq_status launch_one(const Maps& mp, const uint16_t* x16, const int32_t* offsets, int experts, uint16_t* y, int M, int N, int K,
                     int grid_n, int64_t grid_m, int kt_per_split, bool overlap, cudaStream_t s) {
    auto k = mx_gemm_kernel<BN, CL, EXPERTS, XQ>;
    constexpr int smem = Cfg<BN>::TOTAL;
    static std::atomic<uint64_t> raised{0};
    raise_smem(k, smem, raised);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid_n * grid_m), CL, 1);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int na = 0;
    if (CL > 1) {
        attr[na].id = cudaLaunchAttributeClusterDimension;
        attr[na].val.clusterDim.x = 1;
        attr[na].val.clusterDim.y = CL;
        attr[na].val.clusterDim.z = 1;
        ++na;
    }
    if (overlap) {
        attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[na].val.programmaticStreamSerializationAllowed = 1;
        ++na;
    }
    cfg.attrs = attr;
    cfg.numAttrs = na;
    cudaLaunchKernelEx(&cfg, k, mp.w, mp.ws, mp.x, mp.xs, x16, offsets, experts, y, M, N, K, grid_n, kt_per_split);
    return check_launch("mxfp4 gemm");
}

// Activation rows a tile of the pair kernel: the grid runs in rounds of `pairs` tiles, and the
// fewest rounds times (bn + 400) wins. The 400 stand for what does not grow with bn: a tile's fill
// and way out and the floor of its stages. It is a ranking fitted to the launches below, not the
// kernel's time (1024 rows: 1.16 times by the clock, 1.6 by the rule). `rows`: of one expert;
// `columns`: weight tiles of all. Measured at 4096 x 4096 weights: 256 rows 11.3 us in 16 tiles of
// 256, 8.6 in 64 of 64; 512 rows 11.7 in 32 of 256, 9.8 in 64 of 128; 1024 rows 12.1 in 64 of 256,
// 14.0 in 128 of 128; 512 rows of 11008 x 4096 17.5 / 15.8 / 18.6 at 256 / 192 / 128.
int pair_width(int64_t rows, int64_t columns, int64_t pairs) {
    int best = 256;
    int64_t least = -1;
    for (int bn = 256; bn >= 32; bn -= 16) {
        const int64_t tiles = columns * ((rows + bn - 1) / bn), cost = (tiles + pairs - 1) / pairs * (bn + 400);
        if (least < 0 || cost < least) { least = cost; best = bn; }
    }
    return best;
}

template <bool EXPERTS>
wq_status launch_pair(const Maps& mp, const int32_t* offsets, int experts, uint16_t* y, int M, int N, int K,
                      int grid_n, int grid_m, int bn, bool overlap, cudaStream_t s) {
    auto k = mx_gemm_pair_kernel<EXPERTS>;
    static std::atomic<uint64_t> raised{0};
    raise_smem(k, Pair::TOTAL, raised);
    cudaLaunchConfig_t cfg = {};
    const int64_t tiles = (int64_t)grid_n * grid_m;
    cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(tiles, sm_count() / 2)), 1, 1);
    cfg.blockDim = dim3(Pair::THREADS);
    cfg.dynamicSmemBytes = Pair::TOTAL;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = overlap ? 1 : 0;
    cudaLaunchKernelEx(&cfg, k, mp.w, mp.ws, mp.x, mp.xs, mp.y, offsets, experts, y, M, N, K, grid_n, grid_m, bn);
    return check_launch("mxfp4 gemm (pairs)");
}

}  // namespace

// Few rows are quantised by the product (XQ), more by a kernel in front, which costs 0.5 to 0.9 us
// (and 4 us of host time) once, where XQ repeats the work in every tile. XQ / kernel in front:
//   4096 x 4096 at 1, 8, 16, 32 rows: 5.7 / 6.6, 5.9 / 6.6, 6.9 / 6.6, 8.8 / 7.6 us; 28672 x 8192
//   at 1, 8, 16, 32: 23.7 / 25.5, 25.0 / 24.6, 31.9 / 24.8, 45.8 / 25.5; 64 experts of 1408 x 2048
//   at 1/2, 3/4, 1 rows each: 12.0 / 13.5, 17.8 / 16.1, 19.5 / 18.3
bool mx_quantises_itself(int64_t m, int experts) { return m <= std::max(8, experts / 2); }

wq_status launch_gemm_mxfp4(const uint8_t* wp, const uint8_t* wsc, const uint8_t* xp, const uint8_t* xsc,
                            const uint16_t* x16, int64_t m, int64_t n, int64_t k, int experts, const int32_t* offsets,
                            uint16_t* y, bool overlap, cudaStream_t s) {
    const int M = (int)m, N = (int)n, K = (int)k;
    const int grid_n = (N + BM - 1) / BM;
    const int KT = (K + KB - 1) / KB;
    const int sms = sm_count();
    // activation rows a tile should hold: all of them, or the rows of a typical expert
    const int64_t rows = offsets ? (m + experts - 1) / experts : m;
    Maps mp;
    const int64_t pitch = mx_pitch(k);
    wq_status st;
    const int bn = rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : 128;
    // row tiles: with experts the most that any distribution of the rows needs
    const int64_t grid_m = offsets ? m / bn + std::min<int64_t>(experts, m) : (m + bn - 1) / bn;
    if (grid_m * grid_n > 0x7FFFFFFF) return fail(WQ_EUNSUPPORTED, "more than 2^31 - 1 tiles");
    // K split over a cluster: one CTA an SM as long as each keeps 512 columns, two while each
    // keeps 1024 (4096 x 4096 at one row, 32 tiles: 9.0 / 6.8 / 6.0 / 6.7 us at 1 / 2 / 4 / 8 ranks)
    int cl = 1;
    if (!offsets)
        while (cl < 8) {
            const int64_t ctas = grid_m * grid_n * cl * 2;
            const int stages = KT / (cl * 2);
            if (!((ctas <= sms && stages >= 2) || (ctas <= 2 * (int64_t)sms && stages >= 4))) break;
            cl *= 2;
        }
    // Pairs for many rows, and for experts unless the kernel quantises x: their persistent grid walks
    // the tiles that there are, and takes wide tiles at little cost (32 experts of 5632 x 2048 at 2 /
    // 8 / 32 / 128 rows each: 42.9 / 51.4 / 69.2 / 88.9 us one CTA a tile of the average's width,
    // 40.2 / 41.0 / 41.8 / 51.9 in pairs). Experts have more or fewer rows than the average: room for
    // half as many again, which spares most of them a second tile (at 32 / 64 / 128 rows: 46.6 /
    // 48.8 / 55.9 us without, 41.9 / 44.5 / 55.5 with as many again). From 33 rows on also where K is
    // short or cannot be split, as a pair takes all of K in turn: one CTA a tile / pairs, 128 rows of
    // 5632 x 2048 9.9 / 7.6 us (64 rows 7.6 / 6.7, 33: 6.8 / 6.5), of 11008 x 4096 13.1 / 9.6 (64:
    // 10.4 / 8.6), of 4096 x 4096 8.6 / 8.2 (64: 7.1 / 8.1), of 4096 x 11008 13.0 / 13.9; 77 rows of
    // 28672 x 8192 31.6 / 27.6 (64: 25.5 / 26.9), 33 of 20000 x 192 6.1 / 7.7 (77: 7.9 / 8.4; 77 of
    // 1024 x 1024 7.4 / 5.8).
    const bool pairs = offsets || rows > 128 || (rows > 64 && (cl == 1 || K <= 4096)) ||
                       (rows > 32 && cl <= 2 && K > 512 && K <= 4096);
    if (!x16 && pairs) {
        const int gn = (N + 255) / 256;
        const int64_t room = offsets ? std::max(rows, std::min<int64_t>(rows + rows / 2, 256)) : rows;
        const int bn = pair_width(room, (int64_t)gn * experts, sms / 2);
        const int64_t gm = offsets ? m / bn + std::min<int64_t>(experts, m) : (m + bn - 1) / bn;
        if (gm * gn > 0x3FFFFFFF) return fail(WQ_EUNSUPPORTED, "more than 2^30 - 1 tiles");
        if ((st = encode_u8(&mp.w, wp, k / 2, n * experts, KB / 2, BM, true, "the weight codes"))) return st;
        if ((st = encode_u8(&mp.ws, wsc, pitch, n * experts, 16, BM, false, "the weight scales"))) return st;
        if ((st = encode_u8(&mp.x, xp, k / 2, m, 128, bn / 2, true, "the activation codes"))) return st;
        if ((st = encode_u8(&mp.xs, xsc, pitch, m, 16, bn, false, "the activation scales"))) return st;
        mp.y = mp.w;                                             // not used where y's rows are not aligned
        if (n % 8 == 0 &&
            (st = encode(&mp.y, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, y, n, m, 64, 32, true, "the products")))
            return st;
        return offsets ? launch_pair<true>(mp, offsets, experts, y, M, N, K, gn, (int)gm, bn, overlap, s)
                       : launch_pair<false>(mp, offsets, experts, y, M, N, K, gn, (int)gm, bn, overlap, s);
    }
    int per = (KT + cl - 1) / cl;
    per += per & 1;
    if ((st = encode_u8(&mp.w, wp, k / 2, n * experts, KB / 2, BM, true, "the weight codes"))) return st;
    if ((st = encode_u8(&mp.ws, wsc, pitch, n * experts, 16, BM, false, "the weight scales"))) return st;
    if (!x16) {
        if ((st = encode_u8(&mp.x, xp, k / 2, m, KB / 2, bn, true, "the activation codes"))) return st;
        if ((st = encode_u8(&mp.xs, xsc, pitch, m, 16, bn, false, "the activation scales"))) return st;
    } else {
        mp.x = mp.xs = mp.w;                                     // not used
    }
#define WQ_MX(BN, CL, EX, XQ) \
    launch_one<BN, CL, EX, XQ>(mp, x16, offsets, experts, y, M, N, K, grid_n, grid_m, per, overlap, s)
#define WQ_MX_CL(BN, XQ)                                                         \
    (cl == 8 ? WQ_MX(BN, 8, false, XQ) : cl == 4 ? WQ_MX(BN, 4, false, XQ)       \
             : cl == 2 ? WQ_MX(BN, 2, false, XQ) : WQ_MX(BN, 1, false, XQ))
    if (offsets) return WQ_MX(16, 1, true, true);                // at most 8 rows an expert on average
    switch (bn) {
        case 16: return x16 ? WQ_MX_CL(16, true) : WQ_MX_CL(16, false);
        case 32: return WQ_MX_CL(32, false);
        case 64: return WQ_MX_CL(64, false);
        default:                                                 // (unsplit: pairs)
            return cl == 8 ? WQ_MX(128, 8, false, false) : cl == 4 ? WQ_MX(128, 4, false, false)
                                                                   : WQ_MX(128, 2, false, false);
    }
#undef WQ_MX_CL
#undef WQ_MX
}

wq_status read_mx_error(int32_t* code) {
    int v = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(&v, g_mx_error, sizeof v);
    if (e != cudaSuccess) return fail(WQ_ECUDA, "reading the device error word: %s", cudaGetErrorString(e));
    if (v != 0) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_mx_error, &zero, sizeof zero);
    }
    *code = v;
    return WQ_OK;
}

}  // namespace wq
