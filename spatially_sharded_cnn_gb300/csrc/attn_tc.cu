// attn_tc.cu -- linear attention passes (attn.cuh) on the 5th-generation tensor cores, for
// bf16 rows, head sizes that are multiples of 8, rows on 16-byte boundaries.
//
// A block walks over one segment of one (sequence, head) in chunks of 128 rows, four
// products a chunk, all accumulated in fp32 in tensor memory:
//   1  scores = q k^T                             [128 x 128 x DK]
//   2  rows on the state: q Z                     [128 x DV x DK]
//   3  (scores * powers of lambda) v              [128 x DV x 128], scores in tensor memory
//   4  the state's part: k^T (weights * v)        [DK x DV x 128], three times
// The state stays in registers in fp32: a thread holds a row of it (half of the columns),
// adds product 4 to it and leaves a copy rounded to bf16 in shared memory for product 2.
// Roundings: scores and that copy once each to bf16 (y, whose terms have random
// signs, is then off by 2.3e-3 instead of the 1.7e-3 of its own rounding).  v times its
// weight goes into the state as three bf16 pieces (24 bits): states are fp32 outputs, which
// one rounding would leave 1.7e-3 off and two pieces 2.4e-6.
//
// All 256 threads work on every step and one of warp 0 issues copies and products, so that a
// block of 64-wide heads has 128 registers a thread, 112 KB of shared memory and 256
// columns of tensor memory, and two run on an SM, one computing while the other waits.
// Chunks end at the sequence's end: rows past it are never read, and those ahead of its
// first row are the copy engine's zero fill (negative row coordinates).  Every wait is
// bounded, and the threads agree on giving up at the next barrier.
#include "attn.cuh"
#include "tcgen.cuh"

namespace hc {
namespace {

constexpr int TT = 128;  // rows of a chunk
constexpr uint32_t TBLOCK = TT * 128;  // 128 rows x 64 values, 128-byte swizzle

__device__ int g_attn_status;

template <int DK, int DV> struct Shape {
    static constexpr uint32_t q = DK / 64 * TBLOCK, v = DV / 64 * TBLOCK;
    static constexpr uint32_t stage = 2 * q + v;                  // [q][k][v]
    // the state in bf16 (DK rows x DV), and between its reads the third piece of v
    static constexpr uint32_t z = DV / 64 * DK * 128 > v ? DV / 64 * DK * 128 : v;
    static constexpr uint32_t lo = DK < DV ? v : 0;               // second pieces of v (else over q)
    static constexpr uint32_t smem = 2 * stage + z + lo;
    static constexpr uint32_t cols = DV == 128 ? 512 : 256;
    // tensor memory columns: scores 0 .. 127 (as bf16: 0 .. 63), then rows on the chunk, rows on
    // the state; the state's part over the scores' upper half, or behind
    static constexpr uint32_t o1 = 128, o2 = 128 + DV, kv = DV == 128 ? 384 : 64;
    static constexpr int per_sm = DK == 64 && DV == 64 ? 2 : 1;
};

struct TcMaps {
    CUtensorMap q[3], k[3], v[3];
};

struct AttnSh {
    uint64_t full[2];
    uint64_t scores, rows, part;
    uint32_t tmem_base;
    int abort_flag;
    float pw[64];                  // lambda^n at 31 + n, n = 0 .. 31, and zeros ahead of it
    alignas(16) float col[32];     // a score block's columns: lambda^(31 - j), backwards lambda^j
};

// The two warps of a lane quarter.
__device__ __forceinline__ void pair_sync(int quarter) {
    switch (quarter) {
        case 0: asm volatile("bar.sync 1, 64;\n" ::: "memory"); break;
        case 1: asm volatile("bar.sync 2, 64;\n" ::: "memory"); break;
        case 2: asm volatile("bar.sync 3, 64;\n" ::: "memory"); break;
        default: asm volatile("bar.sync 4, 64;\n" ::: "memory");
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two bf16 values times w as three pieces each: 24 bits.
__device__ __forceinline__ void split_pair(uint32_t v, float w, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    float a = __uint_as_float(v << 16) * w, b = __uint_as_float(v & 0xffff0000u) * w;
    p0 = bf2(a, b);
    a -= __uint_as_float(p0 << 16);
    b -= __uint_as_float(p0 & 0xffff0000u);
    p1 = bf2(a, b);
    p2 = bf2(a - __uint_as_float(p1 << 16), b - __uint_as_float(p1 & 0xffff0000u));
}
// 16 bf16 values: a whole 32-byte sector where the address allows.
__device__ __forceinline__ void store16(__nv_bfloat16* p, const uint32_t (&v)[8], bool whole, int left) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};\n" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        if (left > 0) *reinterpret_cast<uint4*>(p) = make_uint4(v[0], v[1], v[2], v[3]);
        if (left > 8) *reinterpret_cast<uint4*>(p + 8) = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

template <int DK, int DV, bool CARRY>
__global__ void __launch_bounds__(256, (Shape<DK, DV>::per_sm))
    attn_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ AttnArgs a) {
    grid_begin();
    using S = Shape<DK, DV>;
    extern __shared__ __align__(1024) unsigned char ring[];  // swizzle atoms are 1 KB
    unsigned char *zop = ring + 2 * S::stage, *lobuf = zop + S::z;
    __shared__ AttnSh sh;
    volatile int* abort_flag = &sh.abort_flag;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: see elect_one
    const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane;

    const int ip = blockIdx.x % a.passes, rest = blockIdx.x / a.passes;
    const int seg = rest % a.segs, pair = rest / a.segs, b = pair / a.H, h = pair - b * a.H;
    const AttnPass& p = a.p[ip];
    const int len = attn_len(a.lens, b, a.L), chunks = (len + TT - 1) / TT;
    const int c0 = min(chunks, seg * a.per), c1 = min(chunks, c0 + a.per), count = c1 - c0;
    const float l2 = attn_log2_decay(a.decay, h);
    const int Dk = p.Dk, Dv = p.Dv, back = p.back;
    const long long zsize = (long long)Dk * Dv;

    if (tid == 0) {
        mbar_init(&sh.full[0], 1);
        mbar_init(&sh.full[1], 1);
        mbar_init(&sh.scores, 1);
        mbar_init(&sh.rows, 1);
        mbar_init(&sh.part, 1);
        sh.abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 0) tc_alloc(&sh.tmem_base, S::cols);
    if (warp == 1) {
        sh.pw[31 + lane] = ex2f(l2 * (float)lane);
        if (lane < 31) sh.pw[lane] = 0.0f;
        sh.col[lane] = ex2f(l2 * (float)(back ? lane : 31 - lane));
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base, lanes = (uint32_t)(32 * quarter) << 16;

    const auto first_row = [&](int it) { return len - (back ? c0 + it + 1 : chunks - c0 - it) * TT; };
    const auto load = [&](int it) {
        unsigned char* st = ring + (it & 1) * S::stage;
        const int t0 = first_row(it);
        mbar_expect_tx(&sh.full[it & 1], CARRY ? S::q + S::v : S::stage);
        for (int i = 0; i < (int)(S::q / TBLOCK); i++) {
            if (!CARRY) tma_4d(st + i * TBLOCK, &maps.q[ip], 64 * i, h, t0, b, &sh.full[it & 1]);
            tma_4d(st + S::q + i * TBLOCK, &maps.k[ip], 64 * i, h, t0, b, &sh.full[it & 1]);
        }
        for (int i = 0; i < (int)(S::v / TBLOCK); i++)
            tma_4d(st + 2 * S::q + i * TBLOCK, &maps.v[ip], 64 * i, h, t0, b, &sh.full[it & 1]);
    };
    int issued = count < 2 ? count : 2;  // chunks whose copies were issued
    if (warp == 0 && elect_one())
        for (int it = 0; it < issued; it++) load(it);
    __syncwarp();

    // ---- the state: row `row`, columns half * DV / 2 ..
    constexpr int ZC = DV / 2;
    const bool zrow = row < DK;
    float z[ZC];
    {
        const float* z0 = CARRY ? nullptr : p.carry ? p.carry + ((long long)pair * a.segs + seg) * zsize
                                          : p.z0    ? p.z0 + pair * zsize
                                                    : nullptr;
#pragma unroll
        for (int i = 0; i < ZC; i++) {
            const int n = half * ZC + i;
            z[i] = z0 && row < Dk && n < Dv ? z0[(long long)row * p.zm + (long long)n * p.zn] : 0.0f;
        }
    }
    const auto put_state = [&] {
        if (CARRY || !zrow) return;
#pragma unroll
        for (int i = 0; i < ZC; i += 8) {
            const int n = half * ZC + i, ch = (n & 63) >> 3;
            *reinterpret_cast<uint4*>(zop + (n >> 6) * (DK * 128) + row * 128 + ((ch ^ (row & 7)) << 4)) =
                make_uint4(bf2(z[i], z[i + 1]), bf2(z[i + 2], z[i + 3]), bf2(z[i + 4], z[i + 5]), bf2(z[i + 6], z[i + 7]));
        }
    };
    put_state();
    fence_async_smem();

    const bool whole = Dv % 16 == 0 && ((uintptr_t)p.y.p & 31) == 0 && p.y.row % 16 == 0 && p.y.batch % 16 == 0;
    constexpr uint32_t id_scores = idesc_bf16(TT, TT, 0, 0), id_rows = idesc_bf16(TT, DV, 0, 1),
                       id_part = idesc_bf16(TT, DV, 1, 1);
    const int ksteps = (Dk + 15) / 16;
    bool fail = false;
    const auto wait = [&](uint64_t* bar, unsigned parity) {
        if (!fail && !mbar_wait(bar, parity, abort_flag, &g_attn_status)) fail = true;
    };
    const auto wait_all = [&](uint64_t* bar, unsigned parity) {  // every thread of the warp
        wait(bar, parity);
        __syncwarp();
    };
    for (int it = 0; it < count; it++) {
        unsigned char* st = ring + (it & 1) * S::stage;
        unsigned char *sq = st, *sk = st + S::q, *sv = st + 2 * S::q, *slo = S::lo ? lobuf : sq;
        const unsigned full_ph = (it >> 1) & 1, ph = it & 1;
        const int t0 = first_row(it), lo = t0 < 0 ? -t0 : 0;
        if (!CARRY) {
            // the state's copy is there and the last chunk's results were read
            tc_fence_before();
            if (__syncthreads_or(fail)) break;
            wait_all(&sh.full[it & 1], full_ph);
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                const uint64_t dq = sdesc(sq, 16, 1024), dk = sdesc(sk, 16, 1024), dz = sdesc(zop, DK * 128, 1024);
#pragma unroll
                for (int k = 0; k < DK / 16; k++)
                    if (k < ksteps) {
                        const uint32_t off = (k >> 2) * (TBLOCK >> 4) + (k & 3) * 2;
                        tc_mma_bf16(tmem, dq + off, dk + off, id_scores, k > 0);
                    }
                tc_commit(&sh.scores);
#pragma unroll
                for (int k = 0; k < DK / 16; k++)
                    if (k < ksteps)
                        tc_mma_bf16(tmem + S::o2, dq + (k >> 2) * (TBLOCK >> 4) + (k & 3) * 2, dz + k * 128, id_rows,
                                    k > 0);
            }
            __syncwarp();
            // ---- scores times powers of lambda, in bf16, back to tensor memory.  This warp
            // takes column blocks half and half + 2 of its rows' four.
            wait_all(&sh.scores, ph);
            tc_fence_after();
            uint32_t pk[2][16];
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int cb = half + 2 * u;
                const bool diag = cb == quarter;
                if (diag) {
                    float s[32];
                    tc_ld32(tmem + lanes + 32 * cb, s);
                    // (a factor of 0 beside a score that is not finite would not do)
#pragma unroll
                    for (int j = 0; j < 32; j++) {
                        const float f = s[j] * sh.pw[31 + (back ? j - lane : lane - j)];
                        s[j] = (back ? j >= lane : j <= lane) ? f : 0.0f;
                    }
#pragma unroll
                    for (int j = 0; j < 16; j++) pk[u][j] = bf2(s[2 * j], s[2 * j + 1]);
                } else if (back ? cb > quarter : cb < quarter) {
                    // lambda^(rows apart) = one power of the row's, 1 at least, and one of the column's
                    float s[32];
                    tc_ld32(tmem + lanes + 32 * cb, s);
                    const float f = ex2f(l2 * (float)(back ? 32 * cb - row : row - 32 * cb - 31));
                    const f32x2 ff = pk2(f, f);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(&sh.col[j]);
                        unpk2(mul2(mul2(pk2(s[j], s[j + 1]), ff), pk2(c.x, c.y)), s[j], s[j + 1]);
                        unpk2(mul2(mul2(pk2(s[j + 2], s[j + 3]), ff), pk2(c.z, c.w)), s[j + 2], s[j + 3]);
                    }
#pragma unroll
                    for (int j = 0; j < 16; j++) pk[u][j] = bf2(s[2 * j], s[2 * j + 1]);
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j++) pk[u][j] = 0;
                }
            }
            // the rows' other warp has read its scores too
            tc_fence_before();
            pair_sync(quarter);
            tc_fence_after();
            tc_st16(tmem + lanes + 16 * half, pk[0]);
            tc_st16(tmem + lanes + 16 * (half + 2), pk[1]);
            tc_wait_st();
            tc_fence_before();
            if (__syncthreads_or(fail)) break;
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                const uint64_t dv = sdesc(sv, TBLOCK, 1024);
#pragma unroll
                for (int k = 0; k < TT / 16; k++) tc_mma_ts(tmem + S::o1, tmem + 8 * k, dv + k * 128, id_rows, k > 0);
                tc_commit(&sh.rows);
            }
            __syncwarp();
        }
        // ---- v times its weight in the state, as three pieces, over v, q and the state's copy:
        // taken while product 3 runs, stored behind it.  16 bytes a time, all of one row; rows
        // (tid >> 3) + 32 i of each 64-column block.
        wait_all(&sh.full[it & 1], full_ph);
        {
            constexpr int NB = DV / 64;
            uint4 p0[4 * NB], p1[4 * NB], p2[4 * NB];
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const int j = (tid >> 3) + 32 * i;
                w[i] = j < lo ? 0.0f : p.su * ex2f(l2 * (float)(back ? j - lo + 1 : TT - 1 - j));
            }
#pragma unroll
            for (int i = 0; i < 4 * NB; i++) p0[i] = *reinterpret_cast<const uint4*>(sv + 16 * (tid + 256 * i));
#pragma unroll
            for (int i = 0; i < 4 * NB; i++) {
                split_pair(p0[i].x, w[i & 3], p0[i].x, p1[i].x, p2[i].x);
                split_pair(p0[i].y, w[i & 3], p0[i].y, p1[i].y, p2[i].y);
                split_pair(p0[i].z, w[i & 3], p0[i].z, p1[i].z, p2[i].z);
                split_pair(p0[i].w, w[i & 3], p0[i].w, p1[i].w, p2[i].w);
            }
            if (!CARRY) {
                wait_all(&sh.rows, ph);
                tc_fence_after();
            }
#pragma unroll
            for (int i = 0; i < 4 * NB; i++) {
                const uint32_t at = 16 * (tid + 256 * i);
                *reinterpret_cast<uint4*>(sv + at) = p0[i];
                *reinterpret_cast<uint4*>(slo + at) = p1[i];
                *reinterpret_cast<uint4*>(zop + at) = p2[i];
            }
        }
        fence_async_smem();
        if (__syncthreads_or(fail)) break;
        if (warp == 0 && elect_one()) {
            tc_fence_after();
            const uint64_t dk = sdesc(sk, TBLOCK, 1024);
#pragma unroll
            for (int u = 0; u < 3; u++) {
                const uint64_t dv = sdesc(u == 2 ? zop : u ? slo : sv, TBLOCK, 1024);
#pragma unroll
                for (int k = 0; k < TT / 16; k++)
                    tc_mma_bf16(tmem + S::kv, dk + k * 128, dv + k * 128, id_part, u > 0 || k > 0);
            }
            tc_commit(&sh.part);
        }
        __syncwarp();
        if (!CARRY) {
            // ---- rows out, while the state's part is multiplied
            tc_fence_after();
            const float w = p.sx * ex2f(l2 * (float)(back ? TT - 1 - row : row >= lo ? row - lo + 1 : 0));
            __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y.p) + b * p.y.batch + (long long)(t0 + row) * p.y.row +
                               (long long)h * Dv;
#pragma unroll
            for (int cc = 0; cc < ZC; cc += 32) {
                float o[32], r[32];
                tc_ld32(tmem + lanes + S::o1 + half * ZC + cc, o);
                tc_ld32(tmem + lanes + S::o2 + half * ZC + cc, r);
                if (row >= lo) {
#pragma unroll
                    for (int i = 0; i < 32; i++) o[i] = fmaf(w, r[i], p.si * o[i]);
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        uint32_t v[8];
#pragma unroll
                        for (int j = 0; j < 8; j++) v[j] = bf2(o[i + 2 * j], o[i + 2 * j + 1]);
                        const int n = half * ZC + cc + i;
                        store16(y + n, v, whole && n < Dv, Dv - n);
                    }
                }
            }
        }
        wait_all(&sh.part, ph);
        tc_fence_after();
        if (issued < count && !fail) {
            if (warp == 0 && elect_one()) load(issued);
            __syncwarp();
            issued++;
        }
        // ---- the state behind the chunk
        const float wz = ex2f(l2 * (float)(TT - lo));
        if (32 * quarter < DK) {
#pragma unroll
            for (int cc = 0; cc < ZC; cc += 32) {
                float s[32];
                tc_ld32(tmem + lanes + S::kv + half * ZC + cc, s);
#pragma unroll
                for (int i = 0; i < 32; i++) z[cc + i] = fmaf(z[cc + i], wz, s[i]);
            }
        }
        if (it + 1 < count) {
            put_state();
            fence_async_smem();
        }
        if (CARRY) {
            tc_fence_before();
            if (__syncthreads_or(fail)) break;
        }
    }

    float* z1 = CARRY ? p.carry + ((long long)pair * a.segs + seg) * zsize
                      : p.z1 && a.segs == 1 ? p.z1 + pair * zsize
                                            : nullptr;
    if (z1 && row < Dk) {
#pragma unroll
        for (int i = 0; i < ZC; i++) {
            const int n = half * ZC + i;
            if (n < Dv) z1[(long long)row * p.zm + (long long)n * p.zn] = z[i];
        }
    }
    if (!CARRY) attn_blank<__nv_bfloat16>(p, b, h, len, a.L, seg, a.segs);
    // copies and products under way end before their memory is given back (after a wait that
    // ran out; otherwise every one of them has been waited for)
    if (tid == 0 && *abort_flag) {
        int zero = 0;
        for (int k = issued > 2 ? issued - 2 : 0; k < issued; k++)
            mbar_wait(&sh.full[k & 1], (unsigned)((k >> 1) & 1), &zero, &g_attn_status);
        tc_commit(&sh.rows);
        for (int i = 0; i < 2; i++) mbar_wait(&sh.rows, (unsigned)i, &zero, &g_attn_status);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tc_dealloc(tmem, S::cols);
}

// Rows of H heads of D values: boxes of 128 rows x 64 values of one head.
hc_status rows_map(CUtensorMap* m, const hc_rows& r, int D, const AttnArgs& a) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)a.H, (uint64_t)a.L, (uint64_t)a.B};
    const uint64_t row = a.L > 1 ? r.row : (long long)a.H * D;
    const uint64_t st[3] = {(uint64_t)D * 2, row * 2, (a.B > 1 ? (uint64_t)r.batch : row * a.L) * 2};
    const uint32_t box[4] = {64, 1, TT, 1};
    return make_tmap(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r.p, dims, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int DK, int DV> hc_status launch_shape(const AttnArgs& a, bool carry, cudaStream_t st) {
    using S = Shape<DK, DV>;
    static std::atomic<unsigned long long> done{0};
    once_per_device(done, [] {
        return cudaFuncSetAttribute(attn_tc_kernel<DK, DV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::smem) == cudaSuccess &&
               cudaFuncSetAttribute(attn_tc_kernel<DK, DV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    S::smem) == cudaSuccess;
    });
    TcMaps m;
    for (int i = 0; i < a.passes; i++) {
        hc_status e;
        if ((e = rows_map(&m.q[i], a.p[i].q, a.p[i].Dk, a)) || (e = rows_map(&m.k[i], a.p[i].k, a.p[i].Dk, a)) ||
            (e = rows_map(&m.v[i], a.p[i].v, a.p[i].Dv, a)))
            return e;
    }
    const dim3 grid((unsigned)((long long)a.B * a.H * a.segs * a.passes));
    if (carry)
        launch_next(attn_tc_kernel<DK, DV, true>, grid, dim3(256), S::smem, st, m, a);
    else
        launch_next(attn_tc_kernel<DK, DV, false>, grid, dim3(256), S::smem, st, m, a);
    return launched(carry ? "attn_tc_carry_kernel" : "attn_tc_kernel", st);
}

}  // namespace

hc_status launch_attn_tc(const AttnArgs& all, bool carry, cudaStream_t st) {
    return attn_by_shape(all, carry, [&](const AttnArgs& a) {
        const bool k = a.p[0].Dk > 64, v = a.p[0].Dv > 64;
        return k ? v ? launch_shape<128, 128>(a, carry, st) : launch_shape<128, 64>(a, carry, st)
                 : v ? launch_shape<64, 128>(a, carry, st) : launch_shape<64, 64>(a, carry, st);
    });
}

hc_status attn_take_status() {
    int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_attn_status, sizeof(int)) != cudaSuccess) {
        cudaGetLastError();
        return HC_ERR_CUDA;
    }
    if (v) {
        const int zero = 0;
        cudaMemcpyToSymbol(g_attn_status, &zero, sizeof(int));
    }
    return (hc_status)v;
}

}  // namespace hc
