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
// Warp roles (320 threads, one CTA an SM): warp 0 loads, warp 1 issues the MMAs, warps 2-9
// drain finished accumulators (two per TMEM lane quarter, half of the columns each) and
// store through TMA.  Every wait is bounded, as in tc.cu.
#include "rows.cuh"
#include "tcgen.cuh"

namespace hc {
namespace {

constexpr int FF_BM = 128, FF_BK = 64;
constexpr int FF_STAGES = 4;
constexpr uint32_t FF_A_BYTES = FF_BM * FF_BK * 2;         // 16 KB
constexpr uint32_t FF_STAGE = FF_A_BYTES + 256 * FF_BK * 2;  // and 32 KB of B
constexpr uint32_t FF_MN_BLOCK = FF_BK * 128;              // 64 MN values x 64 k-values
constexpr int FF_BOX = 32 * 64;                            // 32 rows x 32 values: an output box
constexpr int FF_EPI = 8;
constexpr int FF_THREADS = 32 * (2 + FF_EPI);
constexpr int FF_SMEM = 1024 + FF_STAGES * FF_STAGE + FF_EPI * 2 * FF_BOX;

enum FfnMode { FF_IN, FF_MID, FF_MM };

__device__ int g_ffn_status;

struct FfnParams {
    int units, tiles_m, tiles_n, splits;
    int chunks;     // k-chunks of a product
    int per;        // k-chunks of a split
    int bn;         // accumulator columns a tile
    int amn, bmn;   // operand majors (FF_MM)
    int M, N, F;    // output rows and columns; F for IN and MID
    float* part;    // splits > 1: [split][M][N]
};

struct FfnSmem {
    uint64_t full[FF_STAGES], empty[FF_STAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ bool ff_wait(uint64_t* b, unsigned parity, volatile int* abort_flag) {
    return mbar_wait(b, parity, abort_flag, &g_ffn_status);
}

// act(a) and act'(a)
template <int ACT> __device__ __forceinline__ void act_both(float a, float& f, float& d) {
    if constexpr (ACT == HC_PW_SILU) {
        const float s = sigmoid_f(a);
        f = a * s;
        d = s * fmaf(a, 1.0f - s, 1.0f);
    } else if constexpr (ACT == HC_PW_GELU) {
        float t, e;
        const float r = normal_tail(a, t, e), g = e * fmaf(-0.39894228040143268f, t, r);
        f = fmaf(-t, r * e, fmaxf(a, 0.0f));
        d = a >= 0.0f ? 1.0f - g : g;
    } else {
        f = a;
        d = 1.0f;
    }
}

template <typename T> __device__ __forceinline__ uint32_t pack_pair(float a, float b) {
    Pack<T, 2> p;
    p.v[0] = from_f<T>(a);
    p.v[1] = from_f<T>(b);
    return *reinterpret_cast<const uint32_t*>(&p);
}

// One warp's output boxes: 32 rows (a lane each) x 32 values, 64-byte swizzle, in two
// buffers in turn.
struct BoxOut {
    unsigned char* buf;
    int turn;
};
template <typename T>
__device__ __forceinline__ void box_store(BoxOut& o, const CUtensorMap* map, const float (&v)[32], int lane, int col,
                                          int part, int row, int cols, int rows) {
    unsigned char* box = o.buf + o.turn * FF_BOX;
    o.turn ^= 1;
    if (lane == 0) bulk_wait_read1();  // the store before the last one has read this buffer
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 4; j++)
        *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
            make_uint4(pack_pair<T>(v[8 * j], v[8 * j + 1]), pack_pair<T>(v[8 * j + 2], v[8 * j + 3]),
                       pack_pair<T>(v[8 * j + 4], v[8 * j + 5]), pack_pair<T>(v[8 * j + 6], v[8 * j + 7]));
    fence_async_smem();
    __syncwarp();
    if (lane == 0) {
        if (col < cols && row < rows) tma_store_3d(map, box, col, part, row);
        bulk_commit();
    }
}

// amap, bmap: operands; a2map, b2map: gy and w_out of MID; omap: y, h or a gradient; o2map:
// [ga | gu] of MID.
template <typename T, int MODE, int ACT>
__global__ void __launch_bounds__(FF_THREADS, 1)
    ffn_kernel(const __grid_constant__ CUtensorMap amap, const __grid_constant__ CUtensorMap bmap,
               const __grid_constant__ CUtensorMap a2map, const __grid_constant__ CUtensorMap b2map,
               const __grid_constant__ CUtensorMap omap, const __grid_constant__ CUtensorMap o2map, FfnParams p) {
    grid_begin();
    extern __shared__ __align__(1024) unsigned char dsmem[];
    unsigned char* ring = (unsigned char*)(((uintptr_t)dsmem + 1023) & ~(uintptr_t)1023);
    unsigned char* boxes = ring + FF_STAGES * FF_STAGE;
    __shared__ FfnSmem sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    volatile int* abort_flag = &sh.abort_flag;
    if (threadIdx.x == 0) {
        for (int s = 0; s < FF_STAGES; s++) {
            mbar_init(&sh.full[s], 1);
            mbar_init(&sh.empty[s], 1);
        }
        for (int b = 0; b < 2; b++) {
            mbar_init(&sh.acc_full[b], 1);
            mbar_init(&sh.acc_empty[b], FF_EPI);
        }
        mbar_init(&sh.drain, 1);
        sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) tc_alloc(&sh.tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base;
    const int hw = p.bn / 2;  // IN, MID: columns of each of a and u

    if (warp == 0 && lane == 0) {
        // ---------------- loads ----------------
        long long it = 0;
        bool ok = true;
        for (int t = blockIdx.x; t < p.units && ok; t += gridDim.x) {
            const int n0 = (t % p.tiles_n) * (MODE == FF_MM ? p.bn : hw);
            const int rest = t / p.tiles_n, m0 = (rest % p.tiles_m) * FF_BM, split = rest / p.tiles_m;
            const int c0 = split * p.per, c1 = min(p.chunks, c0 + p.per);
            for (int second = 0; second < (MODE == FF_MID ? 2 : 1) && ok; second++)
                for (int c = c0; c < c1; c++, it++) {
                    const int s = (int)(it % FF_STAGES), k = c * FF_BK;
                    if (it >= FF_STAGES && !ff_wait(&sh.empty[s], (unsigned)((it / FF_STAGES - 1) & 1), abort_flag)) {
                        ok = false;
                        break;
                    }
                    unsigned char *sa = ring + s * FF_STAGE, *sb = sa + FF_A_BYTES;
                    if (MODE == FF_MID && second) {
                        mbar_expect_tx(&sh.full[s], FF_A_BYTES + 128 * FF_BK * 2);
                        tma_2d(sa, &a2map, k, m0, &sh.full[s]);
                        tma_2d(sb, &b2map, k, n0, &sh.full[s]);
                        continue;
                    }
                    mbar_expect_tx(&sh.full[s], FF_A_BYTES + (uint32_t)p.bn * FF_BK * 2);
                    if (MODE != FF_MM) {
                        tma_2d(sa, &amap, k, m0, &sh.full[s]);
                        for (int i = 0; i < hw / 64; i++) {
                            tma_2d(sb + i * FF_MN_BLOCK, &bmap, n0 + 64 * i, k, &sh.full[s]);
                            tma_2d(sb + (hw / 64 + i) * FF_MN_BLOCK, &bmap, p.F + n0 + 64 * i, k, &sh.full[s]);
                        }
                    } else {
                        if (p.amn) {
                            tma_2d(sa, &amap, m0, k, &sh.full[s]);
                            tma_2d(sa + FF_MN_BLOCK, &amap, m0 + 64, k, &sh.full[s]);
                        } else {
                            tma_2d(sa, &amap, k, m0, &sh.full[s]);
                        }
                        if (p.bmn)
                            for (int i = 0; i < p.bn / 64; i++)
                                tma_2d(sb + i * FF_MN_BLOCK, &bmap, n0 + 64 * i, k, &sh.full[s]);
                        else
                            tma_2d(sb, &bmap, k, n0, &sh.full[s]);
                    }
                }
        }
        if (*abort_flag) {
            // wait (bounded, ignoring the abort flag) for the last copy issued into each stage
            int zero = 0;
            for (long long k = it > FF_STAGES ? it - FF_STAGES : 0; k < it; k++)
                ff_wait(&sh.full[k % FF_STAGES], (unsigned)((k / FF_STAGES) & 1), &zero);
        }
    } else if (warp == 1 && lane == 0) {
        // ---------------- MMAs ----------------
        // IN, MM: tile t accumulates in half t & 1 of the 512 columns.  MID: a | u in half
        // t & 1 and gh in the first 128 columns of the other one, which the drain of the
        // tile before frees in the order gh, then a | u.
        const uint32_t fmt = sizeof(T) == 2 && std::is_same<T, __half>::value ? 0u : (1u << 7) | (1u << 10);
        const auto idesc = [&](int n, int amn, int bmn) {
            return (1u << 4) | fmt | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16) | ((uint32_t)(n >> 3) << 17) |
                   ((uint32_t)(FF_BM >> 4) << 24);
        };
        long long it = 0;
        int tile = 0;
        bool ok = true;
        const auto product = [&](uint32_t d, uint32_t id, int c0, int c1, int amn, int bmn) {
            for (int c = c0; c < c1; c++, it++) {
                const int s = (int)(it % FF_STAGES);
                if (!ff_wait(&sh.full[s], (unsigned)((it / FF_STAGES) & 1), abort_flag)) return false;
                tc_fence_after();
                unsigned char* sa = ring + s * FF_STAGE;
                const uint64_t a0 = sdesc(sa, amn ? FF_MN_BLOCK : 16, 1024);
                const uint64_t b0 = sdesc(sa + FF_A_BYTES, bmn ? FF_MN_BLOCK : 16, 1024);
                const uint32_t ak = amn ? 2048 >> 4 : 32 >> 4, bk = bmn ? 2048 >> 4 : 32 >> 4;
#pragma unroll
                for (int k = 0; k < FF_BK / 16; k++)
                    tc_mma_bf16(d, a0 + k * ak, b0 + k * bk, id, c > c0 || k > 0 ? 1u : 0u);
                tc_commit(&sh.empty[s]);
            }
            return true;
        };
        for (int t = blockIdx.x; t < p.units && ok; t += gridDim.x, tile++) {
            const int split = t / p.tiles_n / p.tiles_m;
            const int c0 = split * p.per, c1 = min(p.chunks, c0 + p.per);
            const int b = tile & 1;
            if (MODE == FF_MID) {
                // acc_empty[0]: gh drained, acc_empty[1]: a | u drained
                if (tile > 0 && !ff_wait(&sh.acc_empty[0], (unsigned)((tile - 1) & 1), abort_flag)) break;
                tc_fence_after();
                ok = product(tmem + b * 256, idesc(p.bn, 0, 1), c0, c1, 0, 1);
                if (!ok || (tile > 0 && !ff_wait(&sh.acc_empty[1], (unsigned)((tile - 1) & 1), abort_flag))) break;
                tc_fence_after();
                ok = product(tmem + (b ^ 1) * 256, idesc(128, 0, 0), c0, c1, 0, 0);
                if (ok) tc_commit(&sh.acc_full[0]);
            } else {
                if (tile >= 2 && !ff_wait(&sh.acc_empty[b], (unsigned)((tile / 2 - 1) & 1), abort_flag)) break;
                tc_fence_after();
                if (MODE == FF_IN)
                    ok = product(tmem + b * 256, idesc(p.bn, 0, 1), c0, c1, 0, 1);
                else
                    ok = product(tmem + b * 256, idesc(p.bn, p.amn, p.bmn), c0, c1, p.amn, p.bmn);
                if (ok) tc_commit(&sh.acc_full[b]);
            }
        }
        // every MMA issued has completed before tensor memory is released
        tc_commit(&sh.drain);
        int zero = 0;
        ff_wait(&sh.drain, 0, &zero);
    } else if (warp >= 2) {
        // ---------------- drain ----------------
        const int ew = warp - 2, q = warp & 3, half = ew >> 2;
        const uint32_t lanes = (uint32_t)(32 * q) << 16;
        BoxOut box{boxes + ew * 2 * FF_BOX, 0};
        int tile = 0;
        for (int t = blockIdx.x; t < p.units; t += gridDim.x, tile++) {
            const int n0 = (t % p.tiles_n) * (MODE == FF_MM ? p.bn : hw);
            const int rest = t / p.tiles_n, m0 = (rest % p.tiles_m) * FF_BM, split = rest / p.tiles_m;
            const int b = tile & 1, row = m0 + 32 * q;
            if (MODE == FF_MID) {
                if (!ff_wait(&sh.acc_full[0], (unsigned)(tile & 1), abort_flag)) break;
                tc_fence_after();
                float g[2][32];
                const uint32_t gbase = tmem + lanes + (b ^ 1) * 256 + half * 64, base = tmem + lanes + b * 256 + half * 64;
                tc_ld32(gbase, g[0]);
                tc_ld32(gbase + 32, g[1]);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh.acc_empty[0]);
#pragma unroll
                for (int cc = 0; cc < 2; cc++) {
                    float a[32], u[32];
                    tc_ld32(base + 32 * cc, a);
                    tc_ld32(base + 128 + 32 * cc, u);
                    if (cc == 1) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sh.acc_empty[1]);
                    }
#pragma unroll
                    for (int i = 0; i < 32; i++) {
                        float f, s;
                        act_both<ACT>(a[i], f, s);
                        const float gh = g[cc][i];
                        a[i] = gh * u[i] * s;
                        u[i] *= f;
                        g[cc][i] = gh * f;
                    }
                    const int col = n0 + 64 * half + 32 * cc;
                    box_store<T>(box, &omap, u, lane, col, 0, row, p.F, p.M);
                    box_store<T>(box, &o2map, a, lane, col, 0, row, p.F, p.M);
                    box_store<T>(box, &o2map, g[cc], lane, col, 1, row, p.F, p.M);
                }
                continue;
            }
            if (!ff_wait(&sh.acc_full[b], (unsigned)((tile >> 1) & 1), abort_flag)) break;
            tc_fence_after();
            const uint32_t base = tmem + lanes + b * 256;
            const int own = (MODE == FF_IN ? hw : p.bn) / 2;  // columns of this warp
            for (int cc = half * own; cc < (half + 1) * own; cc += 32) {
                float v[32];
                tc_ld32(base + cc, v);
                if (MODE == FF_IN) {
                    float u[32];
                    tc_ld32(base + hw + cc, u);
#pragma unroll
                    for (int i = 0; i < 32; i++) v[i] = act_f<ACT>(v[i]) * u[i];
                }
                if (MODE == FF_MM && p.splits > 1) {
                    const int r = row + lane;
                    if (r < p.M) {
                        float* o = p.part + ((long long)split * p.M + r) * p.N + n0 + cc;
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            if (n0 + cc + i < p.N)
                                *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    }
                } else {
                    box_store<T>(box, &omap, v, lane, n0 + cc, 0, row, p.N, p.M);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[b]);
        }
        if (lane == 0) bulk_wait_all();  // output boxes written out
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem, 512);
}

// out[r][c] = sum over splits, in order, of part[split][r][c]; four values a thread.
template <typename T>
__global__ void __launch_bounds__(256) ffn_join_kernel(const float* part, int splits, int M, int N, T* out,
                                                       long long row) {
    grid_begin();
    const long long total = (long long)M * (N / 4);
    for (long long e = blockIdx.x * 256LL + threadIdx.x; e < total; e += gridDim.x * 256LL) {
        const long long r = e / (N / 4), c = (e - r * (N / 4)) * 4;
        float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < splits; s++) {
            const float4 v = *reinterpret_cast<const float4*>(part + ((long long)s * M + r) * N + c);
            f[0] += v.x;
            f[1] += v.y;
            f[2] += v.z;
            f[3] += v.w;
        }
        store_pack<T, 4>(out + r * row + c, f);
    }
}

// ---------------------------------------------------------------------------
// A product's shape: M x N outputs over K.
struct MmPlan {
    int bn, tiles_m, tiles_n, chunks, splits, per;
};
MmPlan ffn_plan(int M, int N, int K, bool may_split) {
    MmPlan p;
    p.bn = N > 128 ? 256 : N > 64 ? 128 : 64;
    p.tiles_m = (int)cdiv(M, FF_BM);
    p.tiles_n = (int)cdiv(N, p.bn);
    p.chunks = (int)cdiv(K, FF_BK);
    const long long tiles = (long long)p.tiles_m * p.tiles_n, sms = device_sm_count();
    long long s = may_split && tiles > 0 && tiles < sms ? sms / tiles : 1;
    if (s > p.chunks / 4) s = p.chunks / 4;  // four chunks a split at least
    if (s < 1) s = 1;
    p.per = (int)((p.chunks + s - 1) / s);
    p.splits = p.per > 0 ? (p.chunks + p.per - 1) / p.per : 1;
    return p;
}
size_t part_bytes(const MmPlan& p, int M, int N) { return p.splits > 1 ? sizeof(float) * p.splits * (size_t)M * N : 0; }
size_t pad16(size_t n) { return (n + 15) / 16 * 16; }

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

struct Maps {
    CUtensorMap a, b, a2, b2, o, o2;
};

template <typename T, int MODE, int ACT> hc_status ffn_launch(const Maps& m, const FfnParams& p, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    once_per_device(done, [] {
        return cudaFuncSetAttribute(ffn_kernel<T, MODE, ACT>, cudaFuncAttributeMaxDynamicSharedMemorySize, FF_SMEM) ==
               cudaSuccess;
    });
    const int sms = device_sm_count();
    launch_next(ffn_kernel<T, MODE, ACT>, dim3(p.units < sms ? p.units : sms), dim3(FF_THREADS), FF_SMEM, st, m.a, m.b,
                m.a2, m.b2, m.o, m.o2, p);
    return launched(MODE == FF_IN ? "ffn_in_kernel" : MODE == FF_MID ? "ffn_mid_kernel" : "ffn_mm_kernel", st);
}
template <typename T, int MODE> hc_status ffn_act(int act, const Maps& m, const FfnParams& p, cudaStream_t st) {
    if (act == HC_PW_SILU) return ffn_launch<T, MODE, HC_PW_SILU>(m, p, st);
    if (act == HC_PW_GELU) return ffn_launch<T, MODE, HC_PW_GELU>(m, p, st);
    return ffn_launch<T, MODE, HC_PW_NONE>(m, p, st);
}

FfnParams params(const MmPlan& p, int M, int N, int F) {
    FfnParams q = {};
    q.units = p.tiles_m * p.tiles_n * p.splits;
    q.tiles_m = p.tiles_m;
    q.tiles_n = p.tiles_n;
    q.splits = p.splits;
    q.chunks = p.chunks;
    q.per = p.per;
    q.bn = p.bn;
    q.M = M;
    q.N = N;
    q.F = F;
    return q;
}

// out (M x N, T) = A B over K.  A: [M][K] rows, or with amn [K][M]; B: [N][K] rows, or with bmn [K][N].
template <typename T>
hc_status ffn_mm(const Mat& A, bool amn, const Mat& B, bool bmn, int M, int N, int K, T* out, long long row, float* part,
                 cudaStream_t st) {
    const MmPlan pl = ffn_plan(M, N, K, true);
    FfnParams p = params(pl, M, N, 0);
    p.amn = amn;
    p.bmn = bmn;
    p.part = part;
    hc_status e = HC_OK;
    if (K > 0) {
        Maps m;
        if ((e = in_map(&m.a, A, amn ? FF_BK : FF_BM)) || (e = in_map(&m.b, B, bmn ? FF_BK : pl.bn)) ||
            (e = out_map(&m.o, out, row, N, 1, M)))
            return e;
        m.a2 = m.a;
        m.b2 = m.b;
        m.o2 = m.o;
        if ((e = ffn_launch<T, FF_MM, HC_PW_NONE>(m, p, st)) || p.splits == 1) return e;
    }
    const long long want = cdiv((long long)M * (N / 4), 256), most = 16LL * device_sm_count();
    launch_next(ffn_join_kernel<T>, dim3((unsigned)(want < most ? want : most)), dim3(256), 0, st, (const float*)part,
                K > 0 ? p.splits : 0, M, N, out, row);
    return launched("ffn_join_kernel", st);
}

bool ffn_desc_ok(const hc_gated_ffn_desc* d) {
    return d && d->M >= 0 && d->C >= 1 && d->F >= 1 && d->act >= HC_PW_NONE && d->act <= HC_PW_GELU && dtype_ok(d->dtype);
}
bool ffn_size_ok(const hc_gated_ffn_desc* d) {
    return d->dtype != HC_DTYPE_F32 && d->C % 8 == 0 && d->F % 8 == 0 && d->C <= 1 << 16 && d->F <= 1 << 16 &&
           d->M < 0x7fffffff - 256;
}
// Rows of the copy engine: every one on a 16-byte boundary.
bool ffn_rows_ok(const hc_rows* r, int M) { return !r->p || (ptr_al(r->p, 16) && (M <= 1 || r->row % 8 == 0)); }
long long row_of(const hc_rows* r, const hc_gated_ffn_desc* d) { return d->M > 1 ? r->row : d->C; }

struct Space {
    size_t h, pre, part;  // h [M][F], [ga | gu] [M][2 F], partial sums
    size_t total() const { return h + pre + part; }
};
Space ffn_space(const hc_gated_ffn_desc* d, int pass) {
    const size_t m = (size_t)d->M;
    Space s = {pad16(m * d->F * 2), 0, 0};
    const auto part = [&](int M, int N, int K) {
        const size_t b = part_bytes(ffn_plan(M, N, K, true), M, N);
        if (b > s.part) s.part = b;
    };
    if (pass == 0) {
        part(d->M, d->C, d->F);
    } else {
        s.pre = pad16(2 * m * d->F * 2);
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
    MmPlan pl = ffn_plan(M, 2 * F, C, false);
    // columns of a and u each a tile: 64 where 128 would leave SMs without one
    const int hw = (long long)pl.tiles_m * cdiv(F, 128) >= device_sm_count() ? 128 : 64;
    pl.bn = 2 * hw;
    pl.tiles_n = (int)cdiv(F, hw);
    Maps m;
    hc_status e;
    if ((e = in_map(&m.a, {x->p, row_of(x, d), C, M}, FF_BM)) || (e = in_map(&m.b, {w_in, 2LL * F, 2 * F, C}, FF_BK)) ||
        (e = out_map(&m.o, h, F, F, 1, M)))
        return e;
    m.a2 = m.a;
    m.b2 = m.b;
    m.o2 = m.o;
    if ((e = ffn_act<T, FF_IN>(d->act, m, params(pl, M, F, F), st))) return e;
    return ffn_mm<T>({h, F, F, M}, false, {w_out, C, C, F}, true, M, C, F, (T*)y->p, row_of(y, d),
                     (float*)(ws + ffn_space(d, 0).h), st);
}

template <typename T>
hc_status ffn_bwd(const hc_gated_ffn_desc* d, const hc_rows* x, const void* w_in, const void* w_out, const hc_rows* gy,
                  const hc_rows* gx, T* gw_in, T* gw_out, char* ws, cudaStream_t st) {
    const int M = d->M, C = d->C, F = d->F;
    const Space sp = ffn_space(d, 1);
    void *h = ws, *pre = ws + sp.h;
    float* part = (float*)(ws + sp.h + sp.pre);
    const Mat xm = {x->p, row_of(x, d), C, M}, gym = {gy->p, row_of(gy, d), C, M};
    hc_status e = HC_OK;
    if (M > 0) {
        MmPlan pl = ffn_plan(M, 2 * F, C, false);
        pl.bn = 256;
        pl.tiles_n = (int)cdiv(F, 128);
        Maps m;
        if ((e = in_map(&m.a, xm, FF_BM)) || (e = in_map(&m.b, {w_in, 2LL * F, 2 * F, C}, FF_BK)) ||
            (e = in_map(&m.a2, gym, FF_BM)) || (e = in_map(&m.b2, {w_out, C, C, F}, 128)) ||
            (e = out_map(&m.o, h, F, F, 1, M)) || (e = out_map(&m.o2, pre, 2LL * F, F, 2, M)))
            return e;
        if ((e = ffn_act<T, FF_MID>(d->act, m, params(pl, M, F, F), st))) return e;
        if (gx && gx->p &&
            (e = ffn_mm<T>({pre, 2LL * F, 2 * F, M}, false, {w_in, 2LL * F, 2 * F, C}, false, M, C, 2 * F, (T*)gx->p,
                           row_of(gx, d), part, st)))
            return e;
    }
    if (gw_in && (e = ffn_mm<T>(xm, true, {pre, 2LL * F, 2 * F, M}, true, C, 2 * F, M, gw_in, 2LL * F, part, st))) return e;
    if (gw_out) return ffn_mm<T>({h, F, F, M}, true, gym, true, F, C, M, gw_out, C, part, st);
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
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    if (d->dtype == HC_DTYPE_BF16)
        return ffn_bwd<__nv_bfloat16>(d, x, w_in, w_out, gy, gx, (__nv_bfloat16*)gw_in, (__nv_bfloat16*)gw_out, (char*)ws,
                                      st);
    return ffn_bwd<__half>(d, x, w_in, w_out, gy, gx, (__half*)gw_in, (__half*)gw_out, (char*)ws, st);
}

}  // extern "C"
