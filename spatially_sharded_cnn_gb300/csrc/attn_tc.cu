// attn_tc.cu -- linear attention passes (attn.cuh) on the 5th-generation tensor cores, for
// bf16 rows, head sizes that are multiples of 8, rows on 16-byte boundaries.
//
// A block walks over one segment of one (sequence, head) in chunks of 128 rows, four
// products a chunk, all accumulated in fp32 in tensor memory:
//   1  scores = q k^T                                    [128 x 128 x DK]
//   2  rows on the state: q Z                            [128 x DV x DK]
//   3  (scores * powers of lambda) v                     [128 x DV x 128], scores in tensor memory
//   4  the state's part, transposed: v^T (weights * k)   [DV x DK x 128], three times
// The state stays in registers in fp32, transposed: a thread holds a column n of Z (a half
// or a quarter of the DK values), adds product 4 to it and leaves a copy rounded to bf16 in
// shared memory for product 2.
// Roundings: scores and that copy once each to bf16 (y, whose terms have random
// signs, is then off by 2.3e-3 instead of the 1.7e-3 of its own rounding).  k times its
// weight goes into the state as three bf16 pieces (24 bits): states are fp32 outputs, which
// one rounding would leave 1.7e-3 off and two pieces 2.4e-6.
//
// What a product of M = 128, K = 16 costs, measured: 42 + 0.46 N cycles with A in shared
// memory, 12 + 0.46 N with A in tensor memory.  So products that share A are issued as one
// wider one where the buffers can lie side by side.
//   64-wide heads (Shape::pair): two blocks an SM, one computing while the other waits, with
// 113 KB of shared memory, 256 columns of tensor memory and 128 registers a thread each.
// Products 1 and 2 are one (N = 192: the copy of Z lies behind or ahead of k's rows),
// and so are the three of 4 (the pieces go over q, over k and into the copy's place, next to one
// another), which takes the columns of 1 and 2 once everything has been read from them.
//   Wider heads: one block an SM, and product 4 runs while the scores are read and scaled
// (its pieces only replace what products 1 and 2 have read), product 3 while the state is
// added up, products 1 and 2 while the rows before are stored.  (Product 1 of the next chunk
// behind product 4, before the state is there: 94 us for 86 of this kernel alone, 8 x 4096 x 8
// heads, whose call with its carry pass takes 105: the thread that issues it is held up behind 4, few
// products wait in line.)
// All threads work on every step and one of warp 0 issues copies and products.
//
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
    static constexpr bool pair = DK == 64 && DV == 64;
    static constexpr uint32_t q = DK / 64 * TBLOCK, v = DV / 64 * TBLOCK;
    // x: the state's copy in bf16 (DV rows x DK), and between its reads the third piece of k
    static constexpr uint32_t zblock = DV * 128, z = DK / 64 * zblock, x = z > q ? z : q;
    // shared memory: v1 v0 q0 k0 x k1 q1 (the digit is the stage)
    static constexpr uint32_t smem = 2 * v + 4 * q + x;
    static constexpr uint32_t stage = 2 * q + v;  // bytes of a stage's copies
    // tensor memory columns.  pair: products 1 and 2 and product 4 0 .. 191, product 3 behind.
    // Else scores 0 .. 127, rows on the chunk, rows on the state, the state's part.
    // The scores go back as bf16 over their own first 64 columns.
    static constexpr uint32_t cols = pair ? 256 : 512;
    static constexpr uint32_t o1 = pair ? 192 : 128, o2 = pair ? 0 : 128 + DV, part = pair ? 0 : 384;
    static constexpr int per_sm = pair ? 2 : 1;
    // 16 warps an SM either way: with 8, the steps between the products took twice as long
    static constexpr int threads = pair ? 256 : 512, groups = threads / 128;  // warps of a lane quarter
};

struct TcMaps {
    CUtensorMap q[3], k[3], v[3], y[3];
};

struct AttnSh {
    uint64_t full[2];
    uint64_t scores, rows, part;
    uint32_t tmem_base;
    int abort_flag;
    // si times: lambda^n at 31 + n, n = 0 .. 31, and zeros ahead of it; a score block's columns,
    // lambda^(31 - j), backwards lambda^j
    float pw[64];
    alignas(16) float col[32];
};

// The warps of a lane quarter.
template <int THREADS> __device__ __forceinline__ void quarter_sync(int quarter) {
    switch (quarter) {
        case 0: asm volatile("bar.sync 1, %0;\n" ::"n"(THREADS) : "memory"); break;
        case 1: asm volatile("bar.sync 2, %0;\n" ::"n"(THREADS) : "memory"); break;
        case 2: asm volatile("bar.sync 3, %0;\n" ::"n"(THREADS) : "memory"); break;
        default: asm volatile("bar.sync 4, %0;\n" ::"n"(THREADS) : "memory");
    }
    __syncwarp();
}

__device__ __forceinline__ uint32_t bf2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two bf16 values times w as three pieces each: 24 bits.
__device__ __forceinline__ f32x2 widen(uint32_t v) { return pk2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
__device__ __forceinline__ uint32_t narrow(f32x2 v) {
    float a, b;
    unpk2(v, a, b);
    return bf2(a, b);
}
__device__ __forceinline__ void split_pair(uint32_t v, f32x2 w, uint32_t& p0, uint32_t& p1, uint32_t& p2) {
    const f32x2 minus = pk2(-1.0f, -1.0f);
    f32x2 f = mul2(widen(v), w);
    p0 = narrow(f);
    f = fma2(widen(p0), minus, f);
    p1 = narrow(f);
    p2 = narrow(fma2(widen(p1), minus, f));
}

struct Unit {  // a segment (or, carrying, a cell) of one (sequence, head) of one pass
    int ip, seg, run, pair, b, h, len, chunks, c0, count;
};
template <bool CARRY> __device__ __forceinline__ Unit unit_of(const AttnArgs& a, long long u) {
    Unit r;
    r.ip = (int)(u % a.passes);
    const int rest = (int)(u / a.passes);
    const int runs = CARRY ? a.cells() : a.segs;
    r.run = rest % runs;
    r.seg = CARRY ? r.run / a.split : r.run;
    r.pair = rest / runs;
    r.b = r.pair / a.H;
    r.h = r.pair - r.b * a.H;
    r.len = attn_len(a.lens, r.b, a.L);
    r.chunks = (r.len + TT - 1) / TT;
    r.c0 = min(r.chunks, r.seg * a.per + (CARRY ? r.run - r.seg * a.split : 0) * a.cell_per);
    r.count = min(r.chunks, min(CARRY ? r.c0 + a.cell_per : 0x7fffffff, (r.seg + 1) * a.per)) - r.c0;
    if (r.count < 0) r.count = 0;
    return r;
}

template <int DK, int DV, bool CARRY>
__global__ void __launch_bounds__((Shape<DK, DV>::threads), (Shape<DK, DV>::per_sm))
    attn_tc_kernel(const __grid_constant__ TcMaps maps, const __grid_constant__ AttnArgs a) {
    grid_begin();
    using S = Shape<DK, DV>;
    extern __shared__ __align__(1024) unsigned char smem[];  // swizzle atoms are 1 KB
    __shared__ AttnSh sh;
    volatile int* abort_flag = &sh.abort_flag;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform: see elect_one
    constexpr int THREADS = S::threads, GROUPS = S::groups;
    const int quarter = warp & 3, group = warp >> 2, row = 32 * quarter + lane;

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
    if (warp == 1 && lane < 31) sh.pw[lane] = 0.0f;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem_base, lanes = (uint32_t)(32 * quarter) << 16;

    unsigned char* const sx = smem + 2 * S::v + 2 * S::q;
    const auto buf_v = [&](int s) { return smem + (s ? 0 : S::v); };
    const auto buf_q = [&](int s) { return s ? sx + S::x + S::q : sx - 2 * S::q; };
    const auto buf_k = [&](int s) { return s ? sx + S::x : sx - S::q; };
    // pair: the copy of Z lies behind k's rows in stage 0, ahead of them in stage 1
    const auto buf_z = [&](int s) { return S::pair && s ? sx + S::x - S::z : sx; };

    // ---- copies, two chunks ahead, over the ends of units, by warp `mover`
    const long long units = (long long)a.B * a.H * (CARRY ? a.cells() : a.segs) * a.passes;
    long long lu = blockIdx.x;  // the unit and chunk to load next, and how many were loaded
    int lit = 0, loaded = 0;
    Unit ln = unit_of<CARRY>(a, lu < units ? lu : 0);
    const auto load_next = [&](int mover) {
        while (lu < units && lit >= ln.count) {
            lu += gridDim.x;
            lit = 0;
            if (lu < units) ln = unit_of<CARRY>(a, lu);
        }
        if (lu < units) {
            if (warp == mover && elect_one()) {
                if constexpr (!CARRY) bulk_wait_read();  // the stage's rows out have been read, too
                const AttnPass& lp = a.p[ln.ip];
                const int s = loaded & 1, t0 = ln.len - (lp.back ? ln.c0 + lit + 1 : ln.chunks - ln.c0 - lit) * TT;
                mbar_expect_tx(&sh.full[s], CARRY ? S::q + S::v : S::stage);
                for (int i = 0; i < (int)(S::q / TBLOCK); i++) {
                    if constexpr (!CARRY) tma_4d(buf_q(s) + i * TBLOCK, &maps.q[ln.ip], 64 * i, ln.h, t0, ln.b, &sh.full[s]);
                    tma_4d(buf_k(s) + i * TBLOCK, &maps.k[ln.ip], 64 * i, ln.h, t0, ln.b, &sh.full[s]);
                }
                for (int i = 0; i < (int)(S::v / TBLOCK); i++)
                    tma_4d(buf_v(s) + i * TBLOCK, &maps.v[ln.ip], 64 * i, ln.h, t0, ln.b, &sh.full[s]);
            }
            lit++;
            loaded++;
        }
        __syncwarp();
    };
    load_next(0);
    load_next(0);

    bool fail = false, stop = false;
    const auto wait_all = [&](uint64_t* bar, unsigned parity) {  // every thread of the warp
        if (!fail && !mbar_wait(bar, parity, abort_flag, &g_attn_status)) fail = true;
        __syncwarp();
    };
    int g = 0;  // chunks walked over
    for (long long un = blockIdx.x; un < units && !stop; un += gridDim.x) {
        const Unit u = unit_of<CARRY>(a, un);
        const int pair = u.pair, seg = u.seg, b = u.b, h = u.h, len = u.len, count = u.count;
        const AttnPass& p = a.p[u.ip];
        const int Dk = p.Dk, Dv = p.Dv, back = p.back;
        const float ld = attn_log_decay(a.decay, h), l2 = ld * kLog2e;
        const long long zsize = (long long)Dk * Dv;
        // the warp whose rows have no scores in its column blocks moves data meanwhile
        const int mover = back ? 3 : 4;
        if (!CARRY && warp == 1) {
            // (every warp is past a barrier behind its last read of these)
            sh.pw[31 + lane] = p.si * ex2f(l2 * (float)lane);
            sh.col[lane] = p.si * ex2f(l2 * (float)(back ? lane : 31 - lane));
        }
        const auto first_row = [&](int it) { return len - (back ? u.c0 + it + 1 : u.chunks - u.c0 - it) * TT; };

        // ---- the state: column zn of Z, rows zm ..  With DV = 64 product 4 gives every column
        // twice (lanes 0 .. 63 and 64 .. 127), and twice as many threads share one.
        constexpr int ZC = DK * DV / THREADS;
        const int zn = row % DV, zm = (DV == 64 ? group + GROUPS * (quarter >> 1) : group) * ZC;
        f32x2 z[ZC / 2];
        {
            float z0[ZC] = {};
            const auto place = [&](int i) { return zm + i < Dk && zn < Dv ? (zm + i) * p.zm + zn * p.zn : -1; };
            if (!CARRY)
                attn_state_ahead<ZC>(p, a, pair, seg, ld, u.chunks, TT, u.chunks * TT - len, place, z0);
#pragma unroll
            for (int i = 0; i < ZC; i += 2) z[i / 2] = pk2(z0[i], z0[i + 1]);
        }
        const auto put_state = [&](int s) {
            if (CARRY) return;
#pragma unroll
            for (int i = 0; i < ZC; i += 8) {
                const int m = zm + i, ch = (m & 63) >> 3;
                *reinterpret_cast<uint4*>(buf_z(s) + (m >> 6) * S::zblock + zn * 128 + ((ch ^ (zn & 7)) << 4)) =
                    make_uint4(narrow(z[i / 2]), narrow(z[i / 2 + 1]), narrow(z[i / 2 + 2]), narrow(z[i / 2 + 3]));
            }
        };
        put_state(g & 1);
        fence_async_smem();

        constexpr uint32_t id_scores = idesc_bf16(TT, S::pair ? 192 : TT, 0, 0), id_state = idesc_bf16(TT, DV, 0, 0),
                           id_rows = idesc_bf16(TT, DV, 0, 1), id_part = idesc_bf16(TT, S::pair ? 192 : DK, 1, 1);
        const int ksteps = (Dk + 15) / 16;
        // The steps of a chunk (s its stage, ph its parity, lo the rows that it lacks).
        const auto issue_scores = [&](int s) {  // products 1 and 2
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                const uint64_t dq = sdesc(buf_q(s), 16, 1024), dz = sdesc(buf_z(s), 16, 1024);
                const uint64_t dk = S::pair && s ? dz : sdesc(buf_k(s), 16, 1024);
#pragma unroll
                for (int k = 0; k < DK / 16; k++)
                    if (k < ksteps) {
                        const uint32_t off = (k >> 2) * (TBLOCK >> 4) + (k & 3) * 2;
                        tc_mma_bf16(tmem, dq + off, dk + off, id_scores, k > 0);
                    }
                if constexpr (!S::pair) {
#pragma unroll
                    for (int k = 0; k < DK / 16; k++)
                        if (k < ksteps)
                            tc_mma_bf16(tmem + S::o2, dq + (k >> 2) * (TBLOCK >> 4) + (k & 3) * 2,
                                        dz + (k >> 2) * (S::zblock >> 4) + (k & 3) * 2, id_state, k > 0);
                }
                tc_commit(&sh.scores);
            }
            __syncwarp();
        };
        const auto scale_scores = [&](uint32_t at) {
            // scores times powers of lambda, in bf16, back over themselves.  This warp takes column
            // blocks group, group + GROUPS, .. of its rows' four.
            constexpr int BLOCKS = 4 / GROUPS;
            uint32_t pk[BLOCKS][16];
#pragma unroll
            for (int u = 0; u < BLOCKS; u++) {
                const int cb = group + GROUPS * u;
                if (cb == quarter) {
                    float s[32];
                    tc_ld32(at + 32 * cb, s);
#pragma unroll
                    for (int j = 0; j < 32; j++) s[j] *= sh.pw[31 + (back ? j - lane : lane - j)];
#pragma unroll
                    for (int j = 0; j < 16; j++) pk[u][j] = bf2(s[2 * j], s[2 * j + 1]);
                } else if (back ? cb > quarter : cb < quarter) {
                    // lambda^(rows apart) = one power of the row's, 1 at least, and one of the column's
                    float s[32];
                    tc_ld32(at + 32 * cb, s);
                    const float f = ex2f(l2 * (float)(back ? 32 * cb - row : row - 32 * cb - 31));
                    const f32x2 ff = pk2(f, f);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        const float4 c = *reinterpret_cast<const float4*>(&sh.col[j]);
                        pk[u][j / 2] = narrow(mul2(mul2(pk2(s[j], s[j + 1]), ff), pk2(c.x, c.y)));
                        pk[u][j / 2 + 1] = narrow(mul2(mul2(pk2(s[j + 2], s[j + 3]), ff), pk2(c.z, c.w)));
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; j++) pk[u][j] = 0;
                }
            }
            // the rows' other warps have read their scores too
            tc_fence_before();
            quarter_sync<32 * GROUPS>(quarter);
            tc_fence_after();
#pragma unroll
            for (int u = 0; u < BLOCKS; u++) tc_st16(at + 16 * (group + GROUPS * u), pk[u]);
            tc_wait_st();
        };
        const auto issue_rows = [&](int s, uint32_t at) {  // product 3
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                const uint64_t dv = sdesc(buf_v(s), TBLOCK, 1024);
#pragma unroll
                for (int k = 0; k < TT / 16; k++) tc_mma_ts(tmem + S::o1, at + 8 * k, dv + k * 128, id_rows, k > 0);
                tc_commit(&sh.rows);
            }
            __syncwarp();
        };
        // k times its weight in the state as three pieces, p0 over k, p1 over q, p2 over the
        // state's copy: 16 bytes a time, all of one row; rows (tid >> 3) + THREADS / 8 * i of each
        // 64-column block
        constexpr int NP = TT * DK / 8 / THREADS, NW = TT * 8 / THREADS;
        uint4 p0[NP], p1[NP], p2[NP];
        const auto split_k = [&](int s, int lo) {
            f32x2 w[NW];
#pragma unroll
            for (int i = 0; i < NW; i++) {
                const int j = (tid >> 3) + THREADS / 8 * i;
                const float f = j < lo ? 0.0f : p.su * ex2f(l2 * (float)(back ? j - lo + 1 : TT - 1 - j));
                w[i] = pk2(f, f);
            }
#pragma unroll
            for (int i = 0; i < NP; i++) p0[i] = *reinterpret_cast<const uint4*>(buf_k(s) + 16 * (tid + THREADS * i));
#pragma unroll
            for (int i = 0; i < NP; i++) {
                split_pair(p0[i].x, w[i % NW], p0[i].x, p1[i].x, p2[i].x);
                split_pair(p0[i].y, w[i % NW], p0[i].y, p1[i].y, p2[i].y);
                split_pair(p0[i].z, w[i % NW], p0[i].z, p1[i].z, p2[i].z);
                split_pair(p0[i].w, w[i % NW], p0[i].w, p1[i].w, p2[i].w);
            }
        };
        const auto put_pieces = [&](int s) {
#pragma unroll
            for (int i = 0; i < NP; i++) {
                const uint32_t at = 16 * (tid + THREADS * i);
                *reinterpret_cast<uint4*>(buf_k(s) + at) = p0[i];
                *reinterpret_cast<uint4*>(buf_q(s) + at) = p1[i];
                *reinterpret_cast<uint4*>(sx + at) = p2[i];
            }
            fence_async_smem();
        };
        const auto issue_part = [&](int s) {  // product 4
            if (warp == 0 && elect_one()) {
                tc_fence_after();
                // (DV = 64: both 64-row blocks of v^T are the one there is)
                const uint64_t dv = sdesc(buf_v(s), DV == 64 ? 0 : TBLOCK, 1024);
                if constexpr (S::pair) {
                    const uint64_t dp = sdesc(s ? sx : buf_q(s), TBLOCK, 1024);
#pragma unroll
                    for (int k = 0; k < TT / 16; k++) tc_mma_bf16(tmem + S::part, dv + k * 128, dp + k * 128, id_part, k > 0);
                } else {
#pragma unroll
                    for (int u = 0; u < 3; u++) {
                        const uint64_t dp = sdesc(u == 0 ? sx : u == 1 ? buf_q(s) : buf_k(s), TBLOCK, 1024);
#pragma unroll
                        for (int k = 0; k < TT / 16; k++)
                            tc_mma_bf16(tmem + S::part, dv + k * 128, dp + k * 128, id_part, u > 0 || k > 0);
                    }
                }
                tc_commit(&sh.part);
            }
            __syncwarp();
        };
        const auto fade = [&](int lo) { return attn_fade(ld * (float)(TT - lo)); };  // while product 4 runs
        // the state behind the chunk (attn_faded: z by a rounded lambda^128 took 1.4 % less time and left
        // slow states 1e-5 off after 98341 rows)
        const auto add_part = [&](const AttnFade& f) {
            const f32x2 mm = pk2(f.m, f.m), keep = f.keep ? pk2(1.0f, 1.0f) : pk2(0.0f, 0.0f);
            constexpr int PARTS = S::pair ? 3 : 1;
#pragma unroll
            for (int cc = 0; cc < ZC; cc += 16) {
                float s[PARTS][16];
#pragma unroll
                for (int u = 0; u < PARTS; u++) tc_ld16_async(tmem + lanes + S::part + 64 * u + zm + cc, s[u]);
#pragma unroll
                for (int u = 0; u < PARTS; u++) tc_wait_ld(s[u]);
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    f32x2 t = pk2(s[PARTS - 1][2 * i], s[PARTS - 1][2 * i + 1]);  // the smallest first
#pragma unroll
                    for (int u = PARTS - 2; u >= 0; u--) t = add2(t, pk2(s[u][2 * i], s[u][2 * i + 1]));
                    f32x2& zz = z[cc / 2 + i];
                    zz = fma2(zz, keep, fma2(zz, mm, t));
                }
            }
        };
        constexpr int OC = DV / GROUPS;  // output columns of a thread
        uint32_t out[OC / 2];
        const auto read_rows = [&](int lo, uint32_t o2) {
            const float w = p.sx * ex2f(l2 * (float)(back ? TT - 1 - row : row >= lo ? row - lo + 1 : 0));
            const f32x2 ww = pk2(w, w);
#pragma unroll
            for (int cc = 0; cc < OC; cc += 16) {
                float o[16], r[16];
                tc_ld16_async(tmem + lanes + S::o1 + group * OC + cc, o);
                tc_ld16_async(o2 + lanes + group * OC + cc, r);
                tc_wait_ld(o);
                tc_wait_ld(r);
#pragma unroll
                for (int i = 0; i < 8; i++)
                    out[cc / 2 + i] = narrow(fma2(ww, pk2(r[2 * i], r[2 * i + 1]), pk2(o[2 * i], o[2 * i + 1])));
            }
        };
        // Rows out: over v's buffer, which every product has read, and from there by the copy
        // engine; a chunk that begins before the sequence straight from the registers (a copy
        // may not start at a negative row).
        const auto put_rows = [&](int s, int lo, int t0) {
            if (lo == 0) {
#pragma unroll
                for (int i = 0; i < OC; i += 8) {
                    const int n = group * OC + i, ch = (n & 63) >> 3;
                    *reinterpret_cast<uint4*>(buf_v(s) + (n >> 6) * TBLOCK + row * 128 + ((ch ^ (row & 7)) << 4)) =
                        make_uint4(out[i / 2], out[i / 2 + 1], out[i / 2 + 2], out[i / 2 + 3]);
                }
                fence_async_smem();
            } else if (row >= lo) {
                __nv_bfloat16* y = static_cast<__nv_bfloat16*>(p.y.p) + b * p.y.batch + (long long)(t0 + row) * p.y.row +
                                   (long long)h * Dv;
#pragma unroll
                for (int i = 0; i < OC; i += 8)
                    if (group * OC + i < Dv)
                        *reinterpret_cast<uint4*>(y + group * OC + i) =
                            make_uint4(out[i / 2], out[i / 2 + 1], out[i / 2 + 2], out[i / 2 + 3]);
            }
        };
        const auto store_rows = [&](int it, int s) {  // behind a barrier; warp 0's elected thread
            const int t0 = first_row(it);
            if (t0 < 0) return;
            for (int i = 0; i < (int)(S::v / TBLOCK); i++)
                if (64 * i < Dv) tma_store_4d(&maps.y[u.ip], buf_v(s) + i * TBLOCK, 64 * i, h, t0, b);
            bulk_commit();
        };

        for (int it = 0; it < count; it++, g++) {
            const int s = g & 1, t0 = first_row(it), lo = t0 < 0 ? -t0 : 0;
            const unsigned full_ph = (g >> 1) & 1, ph = g & 1;
            stop = true;
            if constexpr (CARRY) {
                wait_all(&sh.full[s], full_ph);
                split_k(s, lo);
                put_pieces(s);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;
                issue_part(s);
                const AttnFade f = fade(lo);
                wait_all(&sh.part, ph);
                tc_fence_after();
                load_next(mover);  // this chunk's stage is free
                add_part(f);
            } else if constexpr (S::pair) {
                const uint32_t scores = tmem + (s ? 64 : 0), o2 = tmem + (s ? 0 : 128);
                wait_all(&sh.full[s], full_ph);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;  // the state's copy is there, the last chunk's results were read
                if (it > 0 && warp == mover && elect_one()) store_rows(it - 1, s ^ 1);
                __syncwarp();
                issue_scores(s);
                split_k(s, lo);
                wait_all(&sh.scores, ph);
                tc_fence_after();
                put_pieces(s);
                if (g > 0) load_next(mover);
                scale_scores(scores + lanes);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;
                issue_rows(s, scores);
                wait_all(&sh.rows, ph);
                tc_fence_after();
                read_rows(lo, o2);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;
                issue_part(s);
                const AttnFade f = fade(lo);
                wait_all(&sh.part, ph);
                tc_fence_after();
                put_rows(s, lo, t0);
                add_part(f);
                if (it + 1 < count) {
                    put_state(s ^ 1);
                    fence_async_smem();
                }
            } else {
                wait_all(&sh.full[s], full_ph);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;
                if (it > 0 && warp == mover && elect_one()) store_rows(it - 1, s ^ 1);
                __syncwarp();
                issue_scores(s);
                split_k(s, lo);
                wait_all(&sh.scores, ph);
                tc_fence_after();
                put_pieces(s);
                if (__syncthreads_or(fail)) break;
                issue_part(s);
                if (g > 0) load_next(mover);
                scale_scores(tmem + lanes);
                tc_fence_before();
                if (__syncthreads_or(fail)) break;
                issue_rows(s, tmem);
                const AttnFade f = fade(lo);
                wait_all(&sh.part, ph);
                tc_fence_after();
                add_part(f);
                if (it + 1 < count) {
                    put_state(s ^ 1);
                    fence_async_smem();
                }
                wait_all(&sh.rows, ph);
                tc_fence_after();
                read_rows(lo, tmem + S::o2);
                put_rows(s, lo, t0);
            }
            stop = false;
        }
        if (stop) break;
        if (!CARRY && count > 0) {
            if (__syncthreads_or(fail)) break;
            if (warp == mover && elect_one()) {
                store_rows(count - 1, (g - 1) & 1);
                bulk_wait_read();  // the next unit's mover may be another one
            }
            __syncwarp();
        }

        float* z1 = CARRY ? p.carry + ((long long)pair * a.cells() + u.run) * zsize
                          : p.z1 && seg == a.segs - 1 ? p.z1 + pair * zsize
                                                : nullptr;
        if (z1 && zn < Dv) {
            const bool quads = attn_quads(p);
#pragma unroll
            for (int i = 0; i < ZC; i += 4) {
                const int m = zm + i;
                float* zp = z1 + m * p.zm + zn * p.zn;
                float f[4];
                unpk2(z[i / 2], f[0], f[1]);
                unpk2(z[i / 2 + 1], f[2], f[3]);
                if (m >= Dk) continue;
                if (quads) {
                    *reinterpret_cast<float4*>(zp) = make_float4(f[0], f[1], f[2], f[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; k++) zp[k * p.zm] = f[k];
                }
            }
        }
        if constexpr (!CARRY) attn_blank<__nv_bfloat16>(p, b, h, len, a.L, seg, a.segs);
    }
    if (!CARRY && (warp == 3 || warp == 4) && elect_one()) bulk_wait_all();
    __syncwarp();
    // copies and products under way end before their memory is given back (after a wait that
    // ran out; otherwise every one of them has been waited for)
    if (tid == 0 && *abort_flag) {
        int zero = 0;
        for (int k = loaded > 2 ? loaded - 2 : 0; k < loaded; k++)
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
        if ((e = rows_map(&m.y[i], a.p[i].y, a.p[i].Dv, a)) || (e = rows_map(&m.q[i], a.p[i].q, a.p[i].Dk, a)) ||
            (e = rows_map(&m.k[i], a.p[i].k, a.p[i].Dk, a)) ||
            (e = rows_map(&m.v[i], a.p[i].v, a.p[i].Dv, a)))
            return e;
    }
    const long long units = (long long)a.B * a.H * (carry ? a.cells() : a.segs) * a.passes;
    const long long most = (long long)S::per_sm * device_sm_count();
    const dim3 grid((unsigned)(units < most ? units : most));
    if (carry)
        launch_next(attn_tc_kernel<DK, DV, true>, grid, dim3(S::threads), S::smem, st, m, a);
    else
        launch_next(attn_tc_kernel<DK, DV, false>, grid, dim3(S::threads), S::smem, st, m, a);
    return launched(carry ? "attn_tc_carry_kernel" : "attn_tc_kernel", st);
}

}  // namespace

hc_status launch_attn_tc(const AttnArgs& all, bool carry, cudaStream_t st) {
    return attn_by_kernel(all, carry, [&](const AttnArgs& a) {
        const bool k = attn_wide(a.p[0].Dk), v = attn_wide(a.p[0].Dv);
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
