// ffn.cu -- the gated feed-forward product, forward and backward (hc_gated_ffn_*), on the
// 5th-generation tensor cores.
//
// Five products over bf16 or fp16 tiles, accumulated in fp32 in tensor memory, by one
// persistent kernel (128 output rows a tile, 64 k-values a ring stage):
//   IN    a | u = x [w_gate | w_up]: the same 128 (or 64) columns of both lie side by
//         side in one accumulator, so that h = act(a) * u is taken where they are drained
//   OUT   y = h w_out
//   MID   a | u again, and gh = gy w_out^T beside them; the drain takes h, ga = gh u act'(a)
//         and gu = gh act(a), none of which is rounded before that
//   GX    gx = [ga | gu] w_in^T
//   GW    gw_in = x^T [ga | gu], gw_out = h^T gy
// a and u are not kept between the passes: taking them again costs 2 products of 11 and
// reads C values a row, where keeping them in fp32 would move 16 F bytes, and 16-bit
// copies would round them a second time (an error of 1.7e-3 in gx and gw_in becomes
// 3.3e-3).
//
// Operands come by TMA in 128-byte swizzled tiles, K-major or MN-major as the arrays lie,
// so that nothing is transposed or copied; edges are the copy engine's zero fill.
// Large products take pairs of CTAs (256 x 256 outputs a tile, the two SMs of a cluster): each holds
// its 128 rows of A and accumulators, and half of B's columns (32768 rows, 1024 x 2816 SiLU, forward and
// backward, from rest : after seconds of load, which hold the clock near 1.5 GHz: 1361 : 1504 us a CTA a
// tile, 1215 : 1395 in pairs; the products that are run would take 1097 : 1216 at the rates of the
// library's largest).  Bound by the tensor pipe: it is busy 76 to 86 % of the cycles of the
// products, 68 % of MID's, whose gh is a product of half the width, and 61 % of IN's with GELU at C = 512,
// which the drain's instructions hold up.
// Warp roles (576 threads, one CTA an SM): warp 0 loads, warp 1 issues the MMAs, warps 2-17
// drain finished accumulators (four per TMEM lane quarter, 32 columns at a time: with two
// the activations' latency was longer than a tile's products at C = 512) and store through TMA.
// Every wait is bounded, as in tc.cu.
#include "rows.cuh"
#include "tcgen.cuh"

namespace hc {
namespace {

constexpr int FF_BM = 128, FF_BK = 64;
constexpr uint32_t FF_A_BYTES = FF_BM * FF_BK * 2;  // 16 KB
// One CTA a tile: 32 KB of B beside it, four stages; a pair: 16 KB in each CTA, six stages.
constexpr int FF_MAX_STAGES = 6;
__host__ __device__ constexpr int ff_stages(int ctas) { return ctas == 2 ? 6 : 4; }
__host__ __device__ constexpr uint32_t ff_stage(int ctas) { return FF_A_BYTES + 256 / ctas * FF_BK * 2; }
constexpr uint32_t FF_MN_BLOCK = FF_BK * 128;              // 64 MN values x 64 k-values
constexpr int FF_BOX = 32 * 64;                            // 32 rows x 32 values: an output box
constexpr int FF_EPI = 16;
constexpr int FF_THREADS = 32 * (2 + FF_EPI);
constexpr int FF_SMEM = 1024 + 192 * 1024 + FF_EPI * FF_BOX;
static_assert(ff_stages(1) * ff_stage(1) == 192 * 1024 && ff_stages(2) * ff_stage(2) == 192 * 1024, "");

enum FfnMode { FF_IN, FF_MID, FF_MM };

__device__ int g_ffn_status;

struct FfnParams {
    // Tiles 0 .. full - 1 are one unit each.  The `rest` that would leave SMs idle in the last
    // round are cut into `splits` runs of `per` k-chunks, a unit each, and joined afterwards.
    int units, tiles_n, full, rest, splits;
    int chunks, per;  // k-chunks of a product, of a split
    int bn;           // accumulator columns a tile
    int amn, bmn;     // operand majors (FF_MM)
    int M, N, F;      // output rows and columns; F for IN and MID
    int ctas;         // CTAs a tile: 128 rows each
    float* part;      // [split][rest][ctas][128][bn]
};
// Products that one launch runs one after another (FF_MM: up to three that do not read one
// another's results; else one).
constexpr int FF_GROUP = 3;
struct FfnGroup {
    FfnParams p[FF_GROUP];
    int n, units;
};
struct Maps {
    CUtensorMap a[FF_GROUP], b[FF_GROUP], o[FF_GROUP];  // operands and outputs; MID: x, gy; w_in, w_out; h, [ga | gu]
};
struct FfnUnit {
    int i, m0, n0, c0, c1;
    long long slot;  // of `part`, or -1: a whole tile
};
template <int CTAS, int MODE> __device__ __forceinline__ FfnUnit ffn_unit(const FfnGroup& g, int u) {
    int i = 0;
    if (MODE == FF_MM)
        while (u >= g.p[i].units) u -= g.p[i++].units;
    const FfnParams& p = g.p[i];
    const int rank = CTAS == 2 ? blockIdx.x & 1 : 0, width = MODE == FF_MM ? p.bn : p.bn / 2;
    FfnUnit r;
    int tile = u;
    r.i = i;
    r.c0 = 0;
    r.c1 = p.chunks;
    r.slot = -1;
    if (u >= p.full) {
        r.slot = (long long)(u - p.full) * CTAS + rank;
        const int split = (u - p.full) / p.rest;
        tile = p.full + (u - p.full) - split * p.rest;
        r.c0 = split * p.per;
        r.c1 = min(p.chunks, r.c0 + p.per);
    }
    r.m0 = (tile / p.tiles_n * CTAS + rank) * FF_BM;
    r.n0 = tile % p.tiles_n * width;
    return r;
}

struct FfnSmem {
    uint64_t full[FF_MAX_STAGES], empty[FF_MAX_STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ bool ff_wait(uint64_t* b, unsigned parity, volatile int* abort_flag) {
    return mbar_wait(b, parity, abort_flag, &g_ffn_status);
}

// act(x) and act'(x) of pairs, as act_f and act_d of rows.cuh (the drain of a tile has as many
// instructions to issue as its products take cycles at C = 512: 114688 rows, 512 x 2048, GELU forward
// from rest : under load 521 : 561 us a value at a time, 480 : 541 in pairs).
template <int ACT, bool SLOPE> __device__ __forceinline__ void act_pair(f32x2 x, f32x2& f, f32x2& d) {
    const f32x2 one = pk2(1.0f, 1.0f), minus = pk2(-1.0f, -1.0f);
    const auto all = [](float v) { return pk2(v, v); };
    float lo, hi;
    if constexpr (ACT == HC_PW_SILU) {
        unpk2(mul2(x, all(-kLog2e)), lo, hi);
        unpk2(add2(pk2(ex2f(lo), ex2f(hi)), one), lo, hi);
        const f32x2 s = pk2(rcpf(lo), rcpf(hi));
        f = mul2(x, s);
        if constexpr (SLOPE) d = mul2(s, fma2(x, fma2(s, minus, one), one));
    } else if constexpr (ACT == HC_PW_GELU) {
        // normal_tail with n = -|x| and -s
        float x0, x1;
        unpk2(x, x0, x1);
        const f32x2 n = pk2(fmaxf(-fabsf(x0), -14.0f), fmaxf(-fabsf(x1), -14.0f));
        unpk2(fma2(n, all(-0.33f), one), lo, hi);
        const f32x2 s = mul2(n, pk2(rcpf(lo), rcpf(hi)));
        unpk2(mul2(mul2(x, all(-0.5f * kLog2e)), x), lo, hi);
        const f32x2 e = pk2(ex2f(lo), ex2f(hi));
        f32x2 p = fma2(s, all(1.96299188e-05f), all(0.000127479288f));
        p = fma2(s, p, all(-0.000140480028f));
        p = fma2(s, p, all(-0.0017548654f));
        p = fma2(s, p, all(0.0114476355f));
        p = fma2(s, p, all(0.118352972f));
        p = fma2(s, p, all(0.3989425f));
        const f32x2 r = fma2(s, p, all(0.5f));
        f = fma2(n, mul2(r, e), pk2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
        if constexpr (SLOPE) {
            const f32x2 g = mul2(e, fma2(n, all(0.39894228040143268f), r));
            float g0, g1;
            unpk2(g, g0, g1);
            unpk2(fma2(g, minus, one), lo, hi);
            d = pk2(x0 >= 0.0f ? lo : g0, x1 >= 0.0f ? hi : g1);
        }
    } else {
        f = x;
        if constexpr (SLOPE) d = one;
    }
}

template <typename T> __device__ __forceinline__ uint32_t pack_pair(f32x2 v) {
    float a, b;
    uint32_t r;
    unpk2(v, a, b);
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// One warp's output box: 32 rows (a lane each) x 32 values, 64-byte swizzle.
__device__ __forceinline__ void box_free(int lane) {  // the store before has read it
    if (lane == 0) bulk_wait_read();
    __syncwarp();
}
// 16 values of the lane's row, columns 16 half ..
template <typename T>
__device__ __forceinline__ void box_put(unsigned char* box, const uint32_t (&v)[8], int half, int lane) {
#pragma unroll
    for (int j = 0; j < 2; j++)
        *reinterpret_cast<uint4*>(box + lane * 64 + (((2 * half + j) ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
}
__device__ __forceinline__ void box_store(const unsigned char* box, const CUtensorMap* map, int lane, int col, int part,
                                          int row, int cols, int rows) {
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (col < cols && row < rows) tma_store_3d(map, box, col, part, row);
        bulk_commit();
    }
}
template <typename T, int MODE, int ACT, int CTAS>
__global__ void __launch_bounds__(FF_THREADS, 1)
    ffn_kernel(const __grid_constant__ Maps maps, const __grid_constant__ FfnGroup group) {
    grid_begin();
    extern __shared__ __align__(1024) unsigned char dsmem[];
    unsigned char* ring = (unsigned char*)(((uintptr_t)dsmem + 1023) & ~(uintptr_t)1023);
    constexpr int STAGES = ff_stages(CTAS);
    constexpr uint32_t STAGE = ff_stage(CTAS);
    unsigned char* boxes = ring + STAGES * STAGE;
    __shared__ FfnSmem sh;
    const int rank = CTAS == 2 ? blockIdx.x & 1 : 0;  // of a pair; 0 leads
    const int first = blockIdx.x / CTAS, step = gridDim.x / CTAS;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;  // see elect_one
    volatile int* abort_flag = &sh.abort_flag;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; s++) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], FF_EPI * CTAS);
        }
        mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) {
        if constexpr (CTAS == 2)
            tc_alloc_pair(&sh.tmem_base, 512);
        else
            tc_alloc(&sh.tmem_base, 512);
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) cluster_sync();  // the other's barriers are there
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const int hw = group.p[0].bn / 2;  // IN, MID: columns of each of a and u

    if (warp == 0 && elect_one()) {
        // ---------------- loads ----------------
        long long it = 0;
        bool ok = true;
        for (int t = first; t < group.units && ok; t += step) {
            const FfnUnit un = ffn_unit<CTAS, MODE>(group, t);
            const FfnParams& p = group.p[un.i];
            const int m0 = un.m0, n0 = un.n0;
            for (int second = 0; second < (MODE == FF_MID ? 2 : 1) && ok; second++)
                for (int c = un.c0; c < un.c1; c++, it++) {
                    const int s = (int)(it % STAGES), k = c * FF_BK;
                    if (it >= STAGES && !ff_wait(&sh.empty[s], (unsigned)((it / STAGES - 1) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    unsigned char *sa = ring + s * STAGE, *sb = sa + FF_A_BYTES;
                    // the copies of both CTAs of a pair count on the leader's barrier; each brings
                    // its own rows of A and half of B's columns
                    const bool gh = MODE == FF_MID && !second;  // gh first
                    const int bn = (gh ? 128 : p.bn) / CTAS;    // columns of B here
                    if (rank == 0) mbar_expect_tx(&sh.full[s], CTAS * (FF_A_BYTES + (uint32_t)bn * FF_BK * 2));
                    const uint32_t bar = CTAS == 2 ? peer_addr(su32(&sh.full[s]), 0) : 0;
                    const auto copy = [&](unsigned char* dst, const CUtensorMap* m, int x, int y) {
                        if constexpr (CTAS == 2)
                            tma_2d_pair(dst, m, x, y, bar);
                        else
                            tma_2d(dst, m, x, y, &sh.full[s]);
                    };
                    if (gh) {
                        copy(sa, &maps.a[1], k, m0);
                        copy(sb, &maps.b[1], k, n0 + rank * bn);
                    } else if (MODE != FF_MM) {
                        copy(sa, &maps.a[un.i], k, m0);
                        for (int i = 0; i < bn / 64; i++) {
                            const int j = rank * (bn / 64) + i;  // 64-column block of a | u
                            const int col = j < hw / 64 ? n0 + 64 * j : p.F + n0 + 64 * (j - hw / 64);
                            copy(sb + i * FF_MN_BLOCK, &maps.b[un.i], col, k);
                        }
                    } else {
                        if (p.amn) {
                            copy(sa, &maps.a[un.i], m0, k);
                            copy(sa + FF_MN_BLOCK, &maps.a[un.i], m0 + 64, k);
                        } else {
                            copy(sa, &maps.a[un.i], k, m0);
                        }
                        if (p.bmn)
                            for (int i = 0; i < bn / 64; i++)
                                copy(sb + i * FF_MN_BLOCK, &maps.b[un.i], n0 + rank * bn + 64 * i, k);
                        else
                            copy(sb, &maps.b[un.i], k, n0 + rank * bn);
                    }
                }
        }
        if (rank == 0 && *abort_flag) {
            // wait (bounded, ignoring the abort flag) for the last copies issued into each stage
            int zero = 0;
            for (long long k = it > STAGES ? it - STAGES : 0; k < it; k++)
                ff_wait(&sh.full[k % STAGES], (unsigned)((k / STAGES) & 1), &zero);
        }
    } else if (warp == 1 && rank == 0 && elect_one()) {
        // ---------------- MMAs ----------------
        // IN, MM: tile t accumulates in half t & 1 of the 512 columns.  MID: a | u in the first
        // half and gh in 128 columns of the second, in turn: the next tile's gh is multiplied
        // while this one is drained.
        const uint32_t fmt = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
        const auto idesc = [&](int n, int amn, int bmn) {
            return (1u << 4) | fmt | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16) | ((uint32_t)(n >> 3) << 17) |
                   ((uint32_t)(FF_BM * CTAS >> 4) << 24);
        };
        long long it = 0;
        int tile = 0;
        bool ok = true;
        const auto commit = [&](uint64_t* b) {
            if constexpr (CTAS == 2)
                tc_commit_pair(b);
            else
                tc_commit(b);
        };
        const auto drained = [&](int b, unsigned parity) {  // by both CTAs
            uint64_t* bar = &sh.acc_empty[b];
            return mbar_wait_on([&] { return CTAS == 2 ? mbar_try_cluster(bar, parity) : mbar_try(bar, parity); }, abort_flag,
                                &g_ffn_status);
        };
        const auto product = [&](uint32_t d, uint32_t id, int c0, int c1, int amn, int bmn) {
            for (int c = c0; c < c1; c++, it++) {
                const int s = (int)(it % STAGES);
                if (!ff_wait(&sh.full[s], (unsigned)((it / STAGES) & 1), abort_flag)) return false;
                tc_fence_after();
                unsigned char* sa = ring + s * STAGE;
                const uint64_t a0 = sdesc(sa, amn ? FF_MN_BLOCK : 16, 1024);
                const uint64_t b0 = sdesc(sa + FF_A_BYTES, bmn ? FF_MN_BLOCK : 16, 1024);
                const uint32_t ak = amn ? 2048 >> 4 : 32 >> 4, bk = bmn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                for (int k = 0; k < FF_BK / 16; k++) {
                    if constexpr (CTAS == 2)
                        tc_mma_pair(d, a0 + k * ak, b0 + k * bk, id, c > c0 || k > 0 ? 1u : 0u);
                    else
                        tc_mma_bf16(d, a0 + k * ak, b0 + k * bk, id, c > c0 || k > 0 ? 1u : 0u);
                }
                commit(&sh.empty[s]);
            }
            return true;
        };
        for (int t = first; t < group.units && ok; t += step, tile++) {
            const FfnUnit un = ffn_unit<CTAS, MODE>(group, t);
            const FfnParams& p = group.p[un.i];
            const int b = tile & 1;
            if (MODE == FF_MID) {
                // (the tile before last was drained before a | u of the last)
                ok = product(tmem + 256 + b * 128, idesc(128, 0, 0), un.c0, un.c1, 0, 0);
                if (!ok || (tile > 0 && !drained(0, (unsigned)((tile - 1) & 1)))) break;
                tc_fence_after();
                ok = product(tmem, idesc(p.bn, 0, 1), un.c0, un.c1, 0, 1);
                if (ok) commit(&sh.acc_full[0]);
            } else {
                if (tile >= 2 && !drained(b, (unsigned)((tile / 2 - 1) & 1))) break;
                tc_fence_after();
                if (MODE == FF_IN)
                    ok = product(tmem + b * 256, idesc(p.bn, 0, 1), un.c0, un.c1, 0, 1);
                else
                    ok = product(tmem + b * 256, idesc(p.bn, p.amn, p.bmn), un.c0, un.c1, p.amn, p.bmn);
                if (ok) commit(&sh.acc_full[b]);
            }
        }
        // every MMA issued has completed before tensor memory is released
        commit(&sh.drain);
        int zero = 0;
        ff_wait(&sh.drain, 0, &zero);
    } else if (warp >= 2) {
        // ---------------- drain ----------------
        const int ew = warp - 2, q = warp & 3, part = ew >> 2;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        unsigned char* box = boxes + ew * FF_BOX;
        const auto release = [&](int b) {
            if constexpr (CTAS == 2)
                peer_arrive(peer_addr(su32(&sh.acc_empty[b]), 0));
            else
                mbar_arrive(&sh.acc_empty[b]);
        };
        int tile = 0;
        for (int t = first; t < group.units; t += step, tile++) {
            const FfnUnit un = ffn_unit<CTAS, MODE>(group, t);
            const FfnParams& p = group.p[un.i];
            const int b = MODE == FF_MID ? 0 : tile & 1, row = un.m0 + 32 * q;
            if (!ff_wait(&sh.acc_full[b], (unsigned)((MODE == FF_MID ? tile : tile >> 1) & 1), abort_flag)) break;
            __syncwarp();
            tc_fence_after();
            const uint32_t base = tmem + lanes + b * 256;
            if (MODE == FF_MID) {
                const uint32_t gbase = tmem + lanes + 256 + (tile & 1) * 128 + 32 * part;
                uint32_t ga[2][8], gu[2][8];
                box_free(lane);
#pragma unroll
                for (int cc = 0; cc < 2; cc++) {
                    float g[16], a[16], u[16];
                    tc_ld16_async(gbase + 16 * cc, g);
                    tc_ld16_async(base + 32 * part + 16 * cc, a);
                    tc_ld16_async(base + 128 + 32 * part + 16 * cc, u);
                    tc_wait_ld(g);
                    tc_wait_ld(a);
                    tc_wait_ld(u);
                    if (cc == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) release(0);
                    }
                    uint32_t h[8];
#pragma unroll
                    for (int i = 0; i < 8; i++) {
                        const f32x2 gg = pk2(g[2 * i], g[2 * i + 1]), uu = pk2(u[2 * i], u[2 * i + 1]);
                        f32x2 f, d;
                        act_pair<ACT, true>(pk2(a[2 * i], a[2 * i + 1]), f, d);
                        h[i] = pack_pair<T>(mul2(f, uu));
                        ga[cc][i] = pack_pair<T>(mul2(mul2(gg, uu), d));
                        gu[cc][i] = pack_pair<T>(mul2(gg, f));
                    }
                    box_put<T>(box, h, cc, lane);
                }
                const int col = un.n0 + 32 * part;
                box_store(box, &maps.o[un.i], lane, col, 0, row, p.F, p.M);
                box_free(lane);
                box_put<T>(box, ga[0], 0, lane);
                box_put<T>(box, ga[1], 1, lane);
                box_store(box, &maps.o[1], lane, col, 0, row, p.F, p.M);
                box_free(lane);
                box_put<T>(box, gu[0], 0, lane);
                box_put<T>(box, gu[1], 1, lane);
                box_store(box, &maps.o[1], lane, col, 1, row, p.F, p.M);
                continue;
            }
            for (int bx = part; bx < (MODE == FF_IN ? hw : p.bn) / 32; bx += 4) {
                const int col = un.n0 + 32 * bx;
                const bool whole = MODE != FF_MM || un.slot < 0;
                if (whole) box_free(lane);
#pragma unroll
                for (int cc = 0; cc < 2; cc++) {
                    float v[16];
                    f32x2 o[8];
                    tc_ld16_async(base + 32 * bx + 16 * cc, v);
                    if (MODE == FF_IN) {
                        float u[16];
                        tc_ld16_async(base + hw + 32 * bx + 16 * cc, u);
                        tc_wait_ld(v);
                        tc_wait_ld(u);
#pragma unroll
                        for (int i = 0; i < 8; i++) {
                            f32x2 f, d;
                            act_pair<ACT, false>(pk2(v[2 * i], v[2 * i + 1]), f, d);
                            o[i] = mul2(f, pk2(u[2 * i], u[2 * i + 1]));
                        }
                    } else {
                        tc_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 8; i++) o[i] = pk2(v[2 * i], v[2 * i + 1]);
                    }
                    if (whole) {
                        uint32_t h[8];
#pragma unroll
                        for (int i = 0; i < 8; i++) h[i] = pack_pair<T>(o[i]);
                        box_put<T>(box, h, cc, lane);
                    } else {
                        float* to = p.part + (un.slot * FF_BM + 32 * q + lane) * p.bn + 32 * bx + 16 * cc;
#pragma unroll
                        for (int i = 0; i < 16; i += 4)
                            *reinterpret_cast<float4*>(to + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                }
                if (whole) box_store(box, &maps.o[un.i], lane, col, 0, row, p.N, p.M);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) release(b);
        }
        if (lane == 0) bulk_wait_all();  // output boxes written out
    }
    tc_fence_before();
    __syncthreads();
    if constexpr (CTAS == 2) {
        cluster_sync();  // the leader's products are done, and nobody arrives here any more
        tc_fence_after();
        if (warp == 0) tc_dealloc_pair(tmem, 512);
    } else {
        tc_fence_after();
        if (warp == 0) tc_dealloc(tmem, 512);
    }
}

// Few rows (one token of some streams): every tile's product is cut along k over the CTAs of a
// cluster, so that all SMs read weights at once; each leaves its fp32 tile in its own shared memory
// and then takes a share of the rows from everyone's, summed in the order of the ranks.  MODE
// FF_IN (out: h) or FF_MM (out: y).  Warps: 0 loads, 1 multiplies, all eight add up.
constexpr int FS_THREADS = 256;
// CTAs of a cluster at most.  Of eight, the sixteen clusters of 16 tiles ran in two rounds; at most 4 : 6 : 8, us
// of 64 rows, forward: 4096 x 64 (1 and 64 tiles) 14.8 : 13.5 : 12.9, 4096 x 256 (4 and 64) 14.8 : 13.5 : 13.0,
// 4096 x 1024 (16 and 64) 16.1 : 15.0 : 20.9, 1024 x 2816 (44 and 16) 14.2 : 13.5 : 18.5, 2560 x 2560 (40 and 40)
// 17.4 : 17.3 : 17.5.
constexpr int FS_SPLITS = 6;
constexpr int FS_STAGES = 6;
constexpr uint32_t FS_STAGE = FF_A_BYTES + 128 * FF_BK * 2;  // 128 accumulator columns at most
constexpr int FS_SMEM = FS_STAGES * FS_STAGE;                // and the tile in fp32 (64 KB) over it

struct FfnFewParams {
    int chunks, per, bn, tiles_n, splits;
    int M, N, F;  // rows and columns out; F of FF_IN
    void* out;
    long long row;
};

__device__ __forceinline__ float4 peer_load(uint32_t addr, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(peer_addr(addr, rank)));
    return v;
}

template <typename T, int MODE, int ACT>
__global__ void __launch_bounds__(FS_THREADS, 1)
    ffn_few_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap, FfnFewParams p) {
    grid_begin();
    extern __shared__ __align__(1024) unsigned char ring[];
    __shared__ uint64_t full[FS_STAGES], empty[FS_STAGES], done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_word;
    volatile int* abort_flag = &abort_word;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = blockIdx.x % p.splits, tile = blockIdx.x / p.splits;
    const int hw = p.bn / 2, n0 = tile % p.tiles_n * (MODE == FF_IN ? hw : p.bn), m0 = tile / p.tiles_n * FF_BM;
    const int c0 = min(p.chunks, rank * p.per), c1 = min(p.chunks, c0 + p.per);
    if (threadIdx.x == 0) {
        for (int s = 0; s < FS_STAGES; s++) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(&done, 1);
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) tc_alloc(&tmem_base, 128);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    if (warp == 0 && elect_one()) {
        int it = 0;
        for (int c = c0; c < c1; c++, it++) {
            const int s = it % FS_STAGES, k = c * FF_BK;
            if (it >= FS_STAGES && !ff_wait(&empty[s], (unsigned)((it / FS_STAGES - 1) & 1), abort_flag)) break;
            unsigned char *sa = ring + s * FS_STAGE, *sb = sa + FF_A_BYTES;
            mbar_expect_tx(&full[s], FF_A_BYTES + (uint32_t)p.bn * FF_BK * 2);
            tma_2d(sa, &amap, k, m0, &full[s]);
            for (int i = 0; i < p.bn / 64; i++)
                tma_2d(sb + i * FF_MN_BLOCK, &bmap,
                       MODE == FF_IN ? (i < hw / 64 ? n0 + 64 * i : p.F + n0 + 64 * (i - hw / 64)) : n0 + 64 * i, k, &full[s]);
        }
        if (*abort_flag) {  // the last copy issued into each stage lands before the tile takes its place
            int zero = 0;
            for (int k = it > FS_STAGES ? it - FS_STAGES : 0; k < it; k++)
                ff_wait(&full[k % FS_STAGES], (unsigned)((k / FS_STAGES) & 1), &zero);
        }
    } else if (warp == 1 && elect_one()) {
        const uint32_t fmt = std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
        const uint32_t id = (1u << 4) | fmt | (1u << 16) | ((uint32_t)(p.bn >> 3) << 17) | ((uint32_t)(FF_BM >> 4) << 24);
        for (int c = c0; c < c1; c++) {
            const int it = c - c0, s = it % FS_STAGES;
            if (!ff_wait(&full[s], (unsigned)((it / FS_STAGES) & 1), abort_flag)) break;
            tc_fence_after();
            const uint64_t a0 = sdesc(ring + s * FS_STAGE, 16, 1024);
            const uint64_t b0 = sdesc(ring + s * FS_STAGE + FF_A_BYTES, FF_MN_BLOCK, 1024);
#pragma unroll
            for (int k = 0; k < FF_BK / 16; k++) tc_mma_bf16(tmem, a0 + 2 * k, b0 + 128 * k, id, it > 0 || k > 0);
            tc_commit(&empty[s]);
        }
        tc_commit(&done);
    }
    __syncwarp();
    int zero = 0;
    ff_wait(&done, 0, &zero);  // every copy has landed and every product has read it
    __syncwarp();
    tc_fence_after();
    __syncthreads();
    // ---- the tile to shared memory, 16-byte chunks of a row rotated by the row
    float* own = reinterpret_cast<float*>(ring);
    const int row = 32 * (warp & 3) + lane, quads = p.bn / 4;
    for (int cc = (warp >> 2) * (p.bn / 2); cc < ((warp >> 2) + 1) * (p.bn / 2); cc += 16) {
        float v[16];
        tc_ld16_async(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + cc, v);
        tc_wait_ld(v);
#pragma unroll
        for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(own + row * p.bn + ((((cc + i) >> 2) + row) % quads) * 4) =
                c0 < c1 ? make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem, 128);
    // ---- rows rank, rank + splits, ... of everyone's tile
    const int rows = min(FF_BM, p.M - m0), cols = MODE == FF_IN ? hw : p.bn;
    const uint32_t base = su32(own);
    for (int e = threadIdx.x; e < (rows - rank + p.splits - 1) / p.splits * (cols / 4); e += FS_THREADS) {
        const int r = rank + e / (cols / 4) * p.splits, c = e % (cols / 4);
        const uint32_t fa = base + (uint32_t)(r * p.bn + (c + r) % quads * 4) * 4;
        const uint32_t ga = base + (uint32_t)(r * p.bn + (c + hw / 4 + r) % quads * 4) * 4;
        float4 v[FS_SPLITS], w[FS_SPLITS];  // (all under way at once)
#pragma unroll
        for (int k = 0; k < FS_SPLITS; k++)
            if (k < p.splits) {
                v[k] = peer_load(fa, k);
                if (MODE == FF_IN) w[k] = peer_load(ga, k);
            }
        float f[4] = {}, g[4] = {};
#pragma unroll
        for (int k = 0; k < FS_SPLITS; k++)
            if (k < p.splits) {
                f[0] += v[k].x;
                f[1] += v[k].y;
                f[2] += v[k].z;
                f[3] += v[k].w;
                if (MODE == FF_IN) {
                    g[0] += w[k].x;
                    g[1] += w[k].y;
                    g[2] += w[k].z;
                    g[3] += w[k].w;
                }
            }
        if (MODE == FF_IN) {
#pragma unroll
            for (int i = 0; i < 4; i++) f[i] = act_f<ACT>(f[i]) * g[i];
        }
        if (n0 + 4 * c < p.N) store_pack<T, 4>(static_cast<T*>(p.out) + (long long)(m0 + r) * p.row + n0 + 4 * c, f);
    }
    __syncwarp();
    cluster_sync();  // nobody's tile goes while it is read
}

// The tiles that were cut: out = sum over splits, in order.  Grid: (cut tiles of all products,
// groups of 8 rows of a tile's ctas * 128).
struct FfnOut {
    void* p[FF_GROUP];
    long long row[FF_GROUP];
};
template <typename T>
__global__ void __launch_bounds__(256) ffn_join_kernel(const __grid_constant__ FfnGroup g, FfnOut out) {
    grid_begin();
    int i = 0, cut = blockIdx.x;
    while (cut >= g.p[i].rest) cut -= g.p[i++].rest;
    const FfnParams& p = g.p[i];
    const int tile = p.full + cut, rows = FF_BM * p.ctas, m0 = tile / p.tiles_n * rows + blockIdx.y * 8;
    const int n0 = tile % p.tiles_n * p.bn;
    const long long stride = (long long)p.rest * rows * p.bn;
    T* o = static_cast<T*>(out.p[i]);
    for (int e = threadIdx.x; e < 8 * p.bn / 4; e += 256) {
        const int r = e / (p.bn / 4), c = (e - r * (p.bn / 4)) * 4;
        if (m0 + r >= p.M || n0 + c >= p.N) continue;
        const float* in = p.part + ((long long)cut * rows + blockIdx.y * 8 + r) * p.bn + c;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
        for (int s = 0; s < p.splits; s++) {
            const float4 v = *reinterpret_cast<const float4*>(in + s * stride);
            f[0] += v.x;
            f[1] += v.y;
            f[2] += v.z;
            f[3] += v.w;
        }
        store_pack<T, 4>(o + (m0 + r) * out.row[i] + n0 + c, f);
    }
}
template <typename T> __global__ void __launch_bounds__(256) ffn_zero_kernel(T* out, long long n) {
    grid_begin();
    for (long long e = blockIdx.x * 256LL + threadIdx.x; e < n; e += gridDim.x * 256LL) out[e] = from_f<T>(0.0f);
}

// ---------------------------------------------------------------------------
// The shape and cut of a product: M x N outputs over K, tiles of 128 ctas x bn.
FfnParams ffn_plan(int M, int N, int K, int bn, int ctas) {
    FfnParams p = {};
    p.bn = bn;
    p.ctas = ctas;
    p.M = M;
    p.N = N;
    p.tiles_n = (int)cdiv(N, bn);
    p.chunks = (int)cdiv(K, FF_BK);
    p.per = p.chunks;
    p.splits = 1;
    p.units = p.full = (int)cdiv(M, FF_BM * ctas) * p.tiles_n;
    return p;
}
// Microseconds of a k-chunk, measured: a pair reads half of B a CTA, which takes 16 KB instead
// of 32 out of L2 a chunk and an MMA's operands twice as fast out of shared memory.
double ffn_chunk_us(int bn, int ctas) { return ctas == 2 ? bn > 128 ? 0.3 : 0.2 : bn > 128 ? 0.4 : bn > 64 ? 0.27 : 0.2; }
// The same for FF_MM.  What whole rounds over the SMs leave is cut in the way that takes the
// least time, at 0.04 us to write and read a partial tile of 128 rows: 176 tiles of 512
// chunks (gw_in of 32768 rows, 1024 x 5632; one CTA a tile) run in 1.17 rounds, not 2.
FfnParams ffn_mm_plan(int M, int N, int K) {
    FfnParams best = {};
    double least = 1e30;
    for (int ctas = 1; ctas <= 2; ctas++) {
        const int bn = N > 128 ? 256 : N > 64 || ctas == 2 ? 128 : 64, sms = device_sm_count() / ctas;
        if (ctas == 2 && (N <= 64 || M <= FF_BM || sms < 1)) continue;
        FfnParams p = ffn_plan(M, N, K, bn, ctas);
        const int all = p.full, rest = all % sms;
        const double chunk = ffn_chunk_us(bn, ctas), rounds = chunk * p.chunks * (all / sms);
        for (int s = 1; s <= 32; s++) {
            if (s > 1 && (rest == 0 || p.chunks / s < 4)) break;
            const int per = (p.chunks + s - 1) / s, n = per > 0 ? (p.chunks + per - 1) / per : 1;
            const double join = n > 1 ? 4.0 + 0.04 * ctas * rest * n : 0.0;
            const double t = rounds + chunk * per * ((rest * n + sms - 1) / sms) + join;
            if (t < least) {
                least = t;
                p.per = per;
                p.splits = n;
                p.rest = n > 1 ? rest : 0;
                p.full = all - p.rest;
                p.units = p.full + p.rest * n;
                best = p;
            }
        }
    }
    return best;
}
// Whether pairs take the least time for whole tiles of 256 columns.
bool ffn_pairs(int M, int tiles_n) {
    const int sms = device_sm_count();
    if (M <= FF_BM || sms < 2) return false;
    const long long one = (long long)cdiv(M, FF_BM) * tiles_n, two = (long long)cdiv(M, 2 * FF_BM) * tiles_n;
    return ffn_chunk_us(256, 2) * ((two + sms / 2 - 1) / (sms / 2)) <= ffn_chunk_us(256, 1) * ((one + sms - 1) / sms);
}
size_t part_bytes(const FfnParams& p) { return sizeof(float) * p.rest * p.splits * p.ctas * FF_BM * (size_t)p.bn; }
size_t pad16(size_t n) { return (n + 15) / 16 * 16; }

// The three products of the backward pass (gx, gw_in, gw_out) in one launch, where each alone
// would be a round or two of the GPU: tiles are cut so that a unit takes about half of what
// the whole takes of an SM.  False: longer than that, and they run one by one (whole tiles of unequal
// length would not fill it).  One by one : in one launch, us of the backward pass, rows, C x F: 1000, 128 x
// 512 37 : 22; 2000, 256 x 704 49 : 25; 7685, 328 x 872 92 : 75; 16384, 256 x 704 87 : 73; 4096, 512 x 1024
// 70 : 61; 2048, 1024 x 1024 59 : 60; 32768, 128 x 512 89 : 73.  Beyond the limit 8192, 512 x 2048 134 : 138, but
// 16384, 512 x 1024 136 : 126 and 4096, 1024 x 2816 149 : 130.  A quarter : half : all of the whole a unit:
// 7685, 328 x 872 98 : 75 : 93; 16384, 256 x 704 100 : 73 : 70; 4096, 512 x 1024 68 : 61 : 51.
bool ffn_group_plan(int M, int C, int F, FfnParams (&p)[3]) {
    const int dims[3][3] = {{M, C, 2 * F}, {C, 2 * F, M}, {F, C, M}}, sms = device_sm_count();
    double us[3], all = 0.0;
    for (int i = 0; i < 3; i++) {
        const int N = dims[i][1], bn = N > 128 ? 256 : N > 64 ? 128 : 64;
        p[i] = ffn_plan(dims[i][0], N, dims[i][2], bn, 1);
        us[i] = ffn_chunk_us(bn, 1);
        all += us[i] * p[i].chunks * p[i].full / sms;
    }
    if (all > 48.0) return false;
    for (int i = 0; i < 3; i++) {
        const double s = us[i] * p[i].chunks / (all / 2 > 4.0 ? all / 2 : 4.0);
        int n = s < 1.5 ? 1 : s > 32.0 ? 32 : (int)(s + 0.5);
        if (n > p[i].chunks / 4) n = p[i].chunks / 4;
        if (n <= 1) continue;
        p[i].per = (p[i].chunks + n - 1) / n;
        p[i].splits = (p[i].chunks + p[i].per - 1) / p[i].per;
        p[i].rest = p[i].full;
        p[i].full = 0;
        p[i].units = p[i].rest * p[i].splits;
    }
    return true;
}

struct Mat {
    const void* p;
    long long row;  // elements
    int cols, rows;
};
// Boxes of `rows` rows x 64 columns, 128-byte swizzle.
hc_status in_map(CUtensorMap* m, const Mat& t, uint32_t rows) {
    const uint64_t dims[2] = {(uint64_t)t.cols, (uint64_t)t.rows}, st[1] = {(uint64_t)t.row * 2};
    const uint32_t box[2] = {64, rows};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, t.p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// Output boxes of 32 rows x 32 columns; `parts` runs of `cols` columns lie side by side in a row.
hc_status out_map(CUtensorMap* m, const void* p, long long row, int cols, int parts, int rows) {
    const uint64_t dims[3] = {(uint64_t)cols, (uint64_t)parts, (uint64_t)rows};
    const uint64_t st[2] = {(uint64_t)cols * 2, (uint64_t)row * 2};
    const uint32_t box[3] = {32, 1, 32};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

template <typename T, int MODE, int ACT, int CTAS>
hc_status ffn_launch_ctas(const Maps& m, const FfnGroup& g, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    const auto kernel = ffn_kernel<T, MODE, ACT, CTAS>;
    once_per_device(done, [&] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, FF_SMEM) == cudaSuccess;
    });
    const int groups = device_sm_count() / CTAS;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CTAS * (g.units < groups ? g.units : groups));
    cfg.blockDim = dim3(FF_THREADS);
    cfg.dynamicSmemBytes = FF_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = CTAS;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = CTAS == 2 ? 2 : 1;
    cudaLaunchKernelEx(&cfg, kernel, m, g);
    return launched(MODE == FF_IN ? "ffn_in_kernel" : MODE == FF_MID ? "ffn_mid_kernel" : "ffn_mm_kernel", st);
}
template <typename T, int MODE, int ACT> hc_status ffn_launch(const Maps& m, const FfnGroup& g, cudaStream_t st) {
    return g.p[0].ctas == 2 ? ffn_launch_ctas<T, MODE, ACT, 2>(m, g, st) : ffn_launch_ctas<T, MODE, ACT, 1>(m, g, st);
}
template <typename T, int MODE> hc_status ffn_act(int act, const Maps& m, const FfnParams& p, cudaStream_t st) {
    const FfnGroup g = {{p}, 1, p.units};
    if (act == HC_PW_SILU) return ffn_launch<T, MODE, HC_PW_SILU>(m, g, st);
    if (act == HC_PW_GELU) return ffn_launch<T, MODE, HC_PW_GELU>(m, g, st);
    return ffn_launch<T, MODE, HC_PW_NONE>(m, g, st);
}

// out (M x N) = A B over K.  A: [M][K] rows, or with amn [K][M]; B: [N][K] rows, or with bmn [K][N].
struct Product {
    Mat A;
    bool amn;
    Mat B;
    bool bmn;
    int M, N, K;
    void* out;  // NULL: not wanted
    long long row;
};
// Runs products cut as `plan` says in one launch, and joins what was cut; `part` in turn.
template <typename T>
hc_status ffn_products(const Product* pr, const FfnParams* plan, int n, float* part, cudaStream_t st) {
    FfnGroup g = {};
    FfnOut out = {};
    Maps m;
    hc_status e;
    int cut = 0;
    for (int k = 0; k < n; k++) {
        const Product& q = pr[k];
        if (!q.out) continue;
        FfnParams& p = g.p[g.n];
        p = plan[k];
        p.amn = q.amn;
        p.bmn = q.bmn;
        p.part = part;
        part += part_bytes(p) / sizeof(float);
        if ((e = in_map(&m.a[g.n], q.A, q.amn ? FF_BK : FF_BM)) ||
            (e = in_map(&m.b[g.n], q.B, q.bmn ? FF_BK : p.bn / p.ctas)) ||
            (e = out_map(&m.o[g.n], q.out, q.row, q.N, 1, q.M)))
            return e;
        out.p[g.n] = q.out;
        out.row[g.n] = q.row;
        g.units += p.units;
        cut += p.rest;
        g.n++;
    }
    if (g.n == 0) return HC_OK;
    for (int k = g.n; k < FF_GROUP; k++) {
        m.a[k] = m.a[0];
        m.b[k] = m.b[0];
        m.o[k] = m.o[0];
    }
    if ((e = ffn_launch<T, FF_MM, HC_PW_NONE>(m, g, st)) || cut == 0) return e;
    launch_next(ffn_join_kernel<T>, dim3(cut, FF_BM * g.p[0].ctas / 8), dim3(256), 0, st, g, out);
    return launched("ffn_join_kernel", st);
}
template <typename T> hc_status ffn_mm(const Product& p, float* part, cudaStream_t st) {
    const FfnParams plan = ffn_mm_plan(p.M, p.N, p.K);
    return ffn_products<T>(&p, &plan, 1, part, st);
}

// The cut of a product with few rows: columns a tile and CTAs a cluster, or splits = 0 where the
// tiles alone fill the GPU.
struct FewPlan {
    int bn, tiles_n, splits, per, chunks;
};
FewPlan ffn_few_plan(int M, int N, int K, bool gated) {
    FewPlan p = {gated ? 128 : 64, 0, 0, 0, (int)cdiv(K, FF_BK)};
    p.tiles_n = (int)cdiv(N, 64);
    const long long tiles = (long long)cdiv(M, FF_BM) * p.tiles_n, sms = device_sm_count();
    if (tiles * 2 > sms) return p;
    long long s = sms / tiles;
    if (s > FS_SPLITS) s = FS_SPLITS;
    if (s > p.chunks) s = p.chunks;
    p.splits = (int)s;
    p.per = (int)cdiv(p.chunks, s);
    return p;
}
template <typename T, int MODE, int ACT>
hc_status ffn_few(const FewPlan& pl, const Mat& A, const Mat& B, int M, int N, int F, T* out, long long row,
                  cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    once_per_device(done, [] {
        return cudaFuncSetAttribute(ffn_few_kernel<T, MODE, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, FS_SMEM) ==
               cudaSuccess;
    });
    CUtensorMap a, b;
    hc_status e;
    if ((e = in_map(&a, A, FF_BM)) || (e = in_map(&b, B, FF_BK))) return e;
    const FfnFewParams p = {pl.chunks, pl.per, pl.bn, pl.tiles_n, pl.splits, M, N, F, out, row};
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(cdiv(M, FF_BM) * pl.tiles_n * pl.splits);
    cfg.blockDim = dim3(FS_THREADS);
    cfg.dynamicSmemBytes = FS_SMEM;
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = pl.splits;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, ffn_few_kernel<T, MODE, ACT>, a, b, p);
    return launched("ffn_few_kernel", st);
}
template <typename T>
hc_status ffn_few_in(int act, const FewPlan& pl, const Mat& A, const Mat& B, int M, int F, T* out, cudaStream_t st) {
    if (act == HC_PW_SILU) return ffn_few<T, FF_IN, HC_PW_SILU>(pl, A, B, M, F, F, out, F, st);
    if (act == HC_PW_GELU) return ffn_few<T, FF_IN, HC_PW_GELU>(pl, A, B, M, F, F, out, F, st);
    return ffn_few<T, FF_IN, HC_PW_NONE>(pl, A, B, M, F, F, out, F, st);
}

bool ffn_desc_ok(const hc_gated_ffn_desc* d) {
    return d && d->M >= 0 && d->C >= 1 && d->F >= 1 && d->act >= HC_PW_NONE && d->act <= HC_PW_GELU && dtype_ok(d->dtype);
}
bool ffn_size_ok(const hc_gated_ffn_desc* d) {
    return d->dtype != HC_DTYPE_F32 && d->C % 8 == 0 && d->F % 8 == 0 && d->C <= 1 << 16 && d->F <= 1 << 16 &&
           d->M < 0x7fffffff - 256 && (long long)d->M * (d->C > d->F ? d->C : d->F) <= 1LL << 38;  // (tiles fit an int)
}
// Rows of the copy engine: every one on a 16-byte boundary, and no stride of 0.
bool ffn_rows_ok(const hc_rows* r, int M) {
    return !r->p || (ptr_al(r->p, 16) && (M <= 1 || (r->row > 0 && r->row % 8 == 0)));
}
// Whether [p, p + n) shares an element with another such run, or with the M rows of r (elements of two bytes).
bool runs_meet(const void* p, long long n, const void* q, long long m) {
    const char *a = (const char*)p, *b = (const char*)q;
    return a && b && a < b + 2 * m && b < a + 2 * n;
}
bool run_meets_rows(const void* p, long long n, const hc_rows* r, const hc_gated_ffn_desc* d) {
    if (!p || !r || !r->p || d->M == 0) return false;
    const long long row = d->M > 1 ? r->row : d->C, from = ((const char*)p - (const char*)r->p) / 2;  // (both on 16 bytes)
    const long long first = from < d->C ? 0 : (from - d->C) / row + 1;  // that ends behind the run's start
    return first < d->M && first * row < from + n;
}
long long row_of(const hc_rows* r, const hc_gated_ffn_desc* d) { return d->M > 1 ? r->row : d->C; }

struct Space {
    size_t h, pre, part;  // h [M][F], [ga | gu] [M][2 F], partial sums
    size_t total() const { return h + pre + part; }
};
Space ffn_space(const hc_gated_ffn_desc* d, int pass) {
    const size_t m = (size_t)d->M;
    Space s = {pad16(m * d->F * 2), 0, 0};
    const auto part = [&](int M, int N, int K) {
        const size_t b = part_bytes(ffn_mm_plan(M, N, K));
        if (b > s.part) s.part = b;
    };
    if (pass == 0) {
        part(d->M, d->C, d->F);
        return s;
    }
    s.pre = pad16(2 * m * d->F * 2);
    FfnParams g[3];
    if (d->M > 0 && ffn_group_plan(d->M, d->C, d->F, g)) {
        s.part = part_bytes(g[0]) + part_bytes(g[1]) + part_bytes(g[2]);
    } else {
        part(d->M, d->C, 2 * d->F);
        part(d->C, 2 * d->F, d->M);
        part(d->F, d->C, d->M);
    }
    return s;
}

template <typename T>
hc_status ffn_fwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out, const hc_rows* y,
                  char* ws, cudaStream_t st) {
    const int M = d->M, C = d->C, F = d->F;
    void* h = ws;
    // columns of a and u each a tile: 64 where 128 would leave SMs without one
    const int ctas = ffn_pairs(M, cdiv(F, 128)) ? 2 : 1;
    const int hw = ctas == 2 || (long long)cdiv(M, FF_BM) * cdiv(F, 128) >= device_sm_count() ? 128 : 64;
    FfnParams p = ffn_plan(M, F, C, hw, ctas);
    p.bn = 2 * hw;
    p.F = F;
    const Mat xm = {x->p, row_of(x, d), C, M}, wi = {w_in, 2LL * F, 2 * F, C}, hm = {h, F, F, M}, wo = {w_out, C, C, F};
    Maps m;
    hc_status e;
    const FewPlan few = ffn_few_plan(M, F, C, true), few_out = ffn_few_plan(M, C, F, false);
    if (few.splits > 0) {
        if ((e = ffn_few_in<T>(d->act, few, xm, wi, M, F, (T*)h, st))) return e;
        if (few_out.splits > 0)
            return ffn_few<T, FF_MM, HC_PW_NONE>(few_out, hm, wo, M, C, 0, (T*)y->p, row_of(y, d), st);
        return ffn_mm<T>({hm, false, wo, true, M, C, F, y->p, row_of(y, d)}, (float*)(ws + ffn_space(d, 0).h), st);
    }
    if ((e = in_map(&m.a[0], xm, FF_BM)) || (e = in_map(&m.b[0], wi, FF_BK)) || (e = out_map(&m.o[0], h, F, F, 1, M)))
        return e;
    for (int k = 1; k < FF_GROUP; k++) {
        m.a[k] = m.a[0];
        m.b[k] = m.b[0];
        m.o[k] = m.o[0];
    }
    if ((e = ffn_act<T, FF_IN>(d->act, m, p, st))) return e;
    if (few_out.splits > 0) return ffn_few<T, FF_MM, HC_PW_NONE>(few_out, hm, wo, M, C, 0, (T*)y->p, row_of(y, d), st);
    return ffn_mm<T>({hm, false, wo, true, M, C, F, y->p, row_of(y, d)}, (float*)(ws + ffn_space(d, 0).h), st);
}

template <typename T>
hc_status ffn_bwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out, const hc_rows* gy,
                  const hc_rows* gx, T* gw_in, T* gw_out, char* ws, cudaStream_t st) {
    const int M = d->M, C = d->C, F = d->F;
    const Space sp = ffn_space(d, 1);
    void *h = ws, *pre = ws + sp.h;
    float* part = (float*)(ws + sp.h + sp.pre);
    if (M == 0) {  // no rows: the weights' gradients are zeros
        for (int k = 0; k < 2; k++) {
            T* out = k ? gw_out : gw_in;
            const long long n = (long long)C * F * (k ? 1 : 2), want = (n + 255) / 256, most = 16LL * device_sm_count();
            if (!out) continue;
            launch_next(ffn_zero_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, out, n);
            const hc_status e = launched("ffn_zero_kernel", st);
            if (e) return e;
        }
        return HC_OK;
    }
    const Mat xm = {x->p, row_of(x, d), C, M}, gym = {gy->p, row_of(gy, d), C, M}, wi = {w_in, 2LL * F, 2 * F, C};
    const Mat wo = {w_out, C, C, F}, hm = {h, F, F, M}, prem = {pre, 2LL * F, 2 * F, M};
    FfnParams p = ffn_plan(M, F, C, 128, ffn_pairs(M, cdiv(F, 128)) ? 2 : 1);
    p.bn = 256;
    p.F = F;
    Maps m;
    hc_status e;
    if ((e = in_map(&m.a[0], xm, FF_BM)) || (e = in_map(&m.b[0], wi, FF_BK)) || (e = in_map(&m.a[1], gym, FF_BM)) ||
        (e = in_map(&m.b[1], wo, 128 / p.ctas)) || (e = out_map(&m.o[0], h, F, F, 1, M)) ||
        (e = out_map(&m.o[1], pre, 2LL * F, F, 2, M)))
        return e;
    m.a[2] = m.a[0];
    m.b[2] = m.b[0];
    m.o[2] = m.o[0];
    if ((e = ffn_act<T, FF_MID>(d->act, m, p, st))) return e;
    const Product pr[3] = {{prem, false, wi, false, M, C, 2 * F, gx ? gx->p : nullptr, gx ? row_of(gx, d) : 0},
                           {xm, true, prem, true, C, 2 * F, M, gw_in, 2LL * F},
                           {hm, true, gym, true, F, C, M, gw_out, C}};
    FfnParams g[3];
    if (ffn_group_plan(M, C, F, g)) return ffn_products<T>(pr, g, 3, part, st);
    for (int k = 0; k < 3; k++)
        if (pr[k].out && (e = ffn_mm<T>(pr[k], part, st))) return e;
    return HC_OK;
}

}  // namespace

hc_status ffn_take_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_ffn_status, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return HC_ERR_CUDA;
    }
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_ffn_status, &zero, sizeof(int));
    }
    return (hc_status)v;
}

}  // namespace hc

using namespace hc;

extern "C" {

// Workspace: h [M][F], then (backward) [ga | gu] [M][2 F], then the partial sums of the
// products that are cut along k.
hc_status hc_gated_ffn_workspace_size(const hc_gated_ffn_desc* d, int pass, size_t* bytes) {
    if (!ffn_desc_ok(d) || pass < 0 || pass > 1 || !bytes) return HC_ERR_INVALID_ARG;
    if (!ffn_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = ffn_space(d, 0).total();
    if (pass == 1) {
        const size_t b = ffn_space(d, 1).total();
        if (b > *bytes) *bytes = b;
    }
    return HC_OK;
}

hc_status hc_gated_ffn_fwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out,
                           const hc_rows* y, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    const hc_status e = hc_gated_ffn_workspace_size(d, 0, &need);
    if (e) return e;
    if (!rows_in_ok(x, d->dtype, d->M) || !rows_out_ok(y, d->dtype, 1, d->M, d->C) || rows_same(x, y) || !f32_ok(w_in) ||
        !f32_ok(w_out))
        return HC_ERR_INVALID_ARG;
    if (!ffn_rows_ok(x, d->M) || !ffn_rows_ok(y, d->M)) return HC_ERR_UNSUPPORTED;
    const long long n_in = 2LL * d->C * d->F, n_out = n_in / 2;
    if (run_meets_rows(w_in, n_in, y, d) || run_meets_rows(w_out, n_out, y, d)) return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    if (d->M == 0) return HC_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    if (d->dtype == HC_DTYPE_BF16) return ffn_fwd<__nv_bfloat16>(d, x, w_in, w_out, y, (char*)ws, st);
    return ffn_fwd<__half>(d, x, w_in, w_out, y, (char*)ws, st);
}

hc_status hc_gated_ffn_bwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out,
                           const hc_rows* gy, const hc_rows* gx, void* gw_in, void* gw_out, void* ws, size_t ws_bytes,
                           void* stream) {
    size_t need = 0;
    const hc_status e = hc_gated_ffn_workspace_size(d, 1, &need);
    if (e) return e;
    if (!rows_in_ok(x, d->dtype, d->M) || !rows_in_ok(gy, d->dtype, d->M) ||
        (gx && gx->p && (!rows_out_ok(gx, d->dtype, 1, d->M, d->C) || rows_same(gx, x) || rows_same(gx, gy))) ||
        !f32_ok(w_in) || !f32_ok(w_out) || !f32_opt_ok(gw_in) || !f32_opt_ok(gw_out))
        return HC_ERR_INVALID_ARG;
    if (!ffn_rows_ok(x, d->M) || !ffn_rows_ok(gy, d->M) || (gx && !ffn_rows_ok(gx, d->M))) return HC_ERR_UNSUPPORTED;
    // the launch that writes one gradient reads what the others are taken from
    const long long n_in = 2LL * d->C * d->F, n_out = n_in / 2;
    if (runs_meet(gw_in, n_in, w_in, n_in) || runs_meet(gw_in, n_in, w_out, n_out) || runs_meet(gw_out, n_out, w_in, n_in) ||
        runs_meet(gw_out, n_out, w_out, n_out) || runs_meet(gw_in, n_in, gw_out, n_out) || run_meets_rows(w_in, n_in, gx, d) ||
        run_meets_rows(w_out, n_out, gx, d))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* r : {x, gy, gx})
        if (run_meets_rows(gw_in, n_in, r, d) || run_meets_rows(gw_out, n_out, r, d)) return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    if (d->dtype == HC_DTYPE_BF16)
        return ffn_bwd<__nv_bfloat16>(d, x, w_in, w_out, gy, gx, (__nv_bfloat16*)gw_in, (__nv_bfloat16*)gw_out, (char*)ws,
                                      st);
    return ffn_bwd<__half>(d, x, w_in, w_out, gy, gx, (__half*)gw_in, (__half*)gw_out, (char*)ws, st);
}

}  // extern "C"
