// scan.cu -- selective state-space scan on channels-last sequences, forward,
// backward and one token (formulas: hc_mixer.h).
//
// A state h[d][n] belongs to one (sequence, channel, state index).  A warp
// spreads d_state over NL lanes of four states each (d_state rounded up to 4,
// 8, 16, 32 or 64 with states whose B and C are zero) and its 32 / NL lane
// groups over channels: a value of B or C read from shared memory then serves
// several channels of a thread, a step size serves four states, and both sums
// the scan needs -- y over states, the gradients of B and C over channels --
// are partly in-thread and take few shuffles.
//
// The recurrence is sequential in the rows.  Where sequences and channels alone
// do not fill the GPU, a sequence is cut into segments of whole tiles: one pass
// takes every segment from a zero state, the segments' results are joined
// (h_out = exp(A * sum of steps) * h_in + h_local), and the full pass then runs
// every segment from its own first state.  The extra pass costs its
// exponentials again and buys a factor of `segs` in parallelism.
#include "rows.cuh"

namespace hc {
namespace {

constexpr int SC_T = 8;  // rows a tile; the backward pass keeps a tile's states in registers

struct ScanArgs {
    hc_rows u, dt, Bm, Cm, z, y;         // forward
    hc_rows gy, gu, gdt, gB, gC, gz;     // backward
    const float *A, *D, *bias, *h0, *ghT;
    const int* lens;
    float *hT, *saved, *gh0;
    float* part;  // backward: [B][segs][D * N | D | D] sums of gA, gD, gdt_bias
    float* gbc;   // backward, several channel tiles a group: [tile][B][L][G][2][N]
    int B, L, Dm, G, Dg, N;
    int dtype, softplus, vec;
    int ctiles;  // channel tiles per group
    int tiles;   // row tiles per sequence
    int segs, seg_tiles;  // segments a sequence is cut into, row tiles in each
    float* carry;         // [B][segs][D][NP]: a segment's state from a zero state, then the state it starts from
    float* dsum;          // [B][segs][D]: its sum of step sizes
};

__device__ __forceinline__ float ld1(const void* p, long long i, int dt) {
    if (dt == HC_DTYPE_F32) return static_cast<const float*>(p)[i];
    if (dt == HC_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
    return __half2float(static_cast<const __half*>(p)[i]);
}
__device__ __forceinline__ void st1(void* p, long long i, int dt, float v) {
    if (dt == HC_DTYPE_F32)
        static_cast<float*>(p)[i] = v;
    else if (dt == HC_DTYPE_BF16)
        static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
    else
        static_cast<__half*>(p)[i] = __float2half_rn(v);
}
// Channels c .. c + 3 of a row, those at or past n left alone; vec: aligned to
// four elements, and then n is a multiple of 4.
__device__ __forceinline__ void st4(void* p, long long i, int dt, int c, int n, bool vec, const float (&f)[4]) {
    if (vec && c < n) {
        if (dt == HC_DTYPE_F32)
            store_pack<float, 4>(static_cast<float*>(p) + i + c, f);
        else if (dt == HC_DTYPE_BF16)
            store_pack<__nv_bfloat16, 4>(static_cast<__nv_bfloat16*>(p) + i + c, f);
        else
            store_pack<__half, 4>(static_cast<__half*>(p) + i + c, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (c + k < n) st1(p, i + c + k, dt, f[k]);
}

// States n0 .. n0 + 3 of a [..][N] fp32 row (past N: zeros / not written).
__device__ __forceinline__ void ld_states(const float* p, int n0, int N, float (&f)[4]) {
    if (N % 4 == 0 && n0 < N) {
        load_pack<float, 4>(p + n0, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) f[k] = n0 + k < N ? p[n0 + k] : 0.0f;
}
__device__ __forceinline__ void st_states(float* p, int n0, int N, const float (&f)[4]) {
    if (N % 4 == 0 && n0 < N) {
        store_pack<float, 4>(p + n0, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (n0 + k < N) p[n0 + k] = f[k];
}

__device__ __forceinline__ int scan_len(const ScanArgs& a, int b) {
    return a.lens ? min(max(a.lens[b], 0), a.L) : a.L;
}

// Sums over the NL lanes of a group of each lane's v[0 .. M): the halving steps
// leave lane n with value `own` (the first of M / min(M, NL) it keeps at v[0..]).
template <int M, int NL>
__device__ __forceinline__ int lanes_sum(float (&v)[M], int n) {
    int first = 0, left = M;
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) {
        if (left > 1) {
            const int half = left / 2;
            const bool up = (n & o) != 0;
#pragma unroll
            for (int i = 0; i < M / 2; i++) {
                if (i < half) {
                    const float send = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
            first += up ? half : 0;
            left = half;
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
        }
    }
    return first;
}

// Two fp32 values in one 64-bit register pair: one instruction for two
// multiply-adds.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pk2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 ex2x2(f32x2 v) {
    float a, b;
    unpk2(v, a, b);
    return pk2(ex2f(a), ex2f(b));
}

__device__ __forceinline__ void cp_async(unsigned dst, const void* src, int bytes, bool on) {
    const int n = on ? bytes : 0;  // the rest of the destination is zeroed
    if (bytes == 16)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The layout the three kernels share.  A thread holds states 4n .. 4n + 3 of
// four channels as two channel pairs; a block's CT channels times a tile's rows
// are also walked elementwise, every thread at four fixed channels.
template <int NL> struct Tile {
    static constexpr int NP = 4 * NL, CG = 32 / NL;
    static constexpr int W = NL == 1 ? 1 : NL == 2 ? 2 : 4;  // warps
    static constexpr int WC = 4 * CG;                        // channels a warp
    static constexpr int CT = W * WC;                        // channels a block
    static constexpr int THREADS = W * 32;
    static constexpr int ROWS = THREADS / (CT / 4) < SC_T ? THREADS / (CT / 4) : SC_T;  // rows walked at once
    static constexpr int PLANE = SC_T * CT;                                             // values of a tile
    static constexpr int BC = 2 * SC_T * NP / THREADS;  // values of B and C a thread fetches
};

// Where a block works: CT channels of one group of one segment.
struct Where {
    int b, seg, bs, g, c0, cn, d0, len, tile0, tile1;
    __device__ __forceinline__ Where(const ScanArgs& a, int CT) {
        const int ct = blockIdx.x % (a.G * a.ctiles);
        bs = blockIdx.x / (a.G * a.ctiles);
        b = bs / a.segs;
        seg = bs % a.segs;
        g = ct / a.ctiles;
        c0 = (ct % a.ctiles) * CT;  // first channel inside the group
        cn = min(CT, a.Dg - c0);
        d0 = g * a.Dg + c0;
        len = scan_len(a, b);
        tile0 = seg * a.seg_tiles;
        tile1 = min(tile0 + a.seg_tiles, a.tiles);
    }
    // one past the last tile with a row of the sequence
    __device__ __forceinline__ int live1() const { return max(tile0, min(tile1, (len + SC_T - 1) / SC_T)); }
};

// A thread's place in the elementwise walk.  Read anew for every tile, so that
// the addresses made from it are not kept in registers across the recurrence.
template <int NL> struct Walk {
    int ec, er;  // four channels from ec, rows er, er + ROWS, ...
    __device__ __forceinline__ Walk() {
        int tid = threadIdx.x;
        asm volatile("" : "+r"(tid));
        ec = tid % (Tile<NL>::CT / 4) * 4;
        er = tid / (Tile<NL>::CT / 4);
    }
};

// Starts the copy of a tile's rows of one tensor to plane k of the raw buffer.
template <int NL>
__device__ __forceinline__ void fetch(const ScanArgs& a, const hc_rows& r, const Where& w, const Walk<NL>& at, int t0,
                                      int k, char* raw) {
    using S = Tile<NL>;
    const int sh = a.dtype == HC_DTYPE_F32 ? 2 : 1;
    const char* p = static_cast<const char*>(r.p) + ((w.b * r.batch + w.d0 + at.ec) << sh);
    for (int t = at.er; t < SC_T; t += S::ROWS) {  // none for er >= ROWS = SC_T
        const bool on = t0 + t < w.len && at.ec < w.cn;
        char* dst = raw + ((k * S::PLANE + t * S::CT + at.ec) << sh);
        const char* q = on ? p + (((t0 + t) * r.row) << sh) : p;
        if (a.vec) {
            cp_async((unsigned)__cvta_generic_to_shared(dst), q, 4 << sh, on);
            continue;
        }
        for (int i = 0; i < 4; i++) {
            const bool in = on && at.ec + i < w.cn;
            if (sh == 2)
                reinterpret_cast<unsigned*>(dst)[i] = in ? reinterpret_cast<const unsigned*>(q)[i] : 0u;
            else
                reinterpret_cast<unsigned short*>(dst)[i] =
                    in ? reinterpret_cast<const unsigned short*>(q)[i] : (unsigned short)0;
        }
    }
}
// Four channels of row t of plane k.
template <int NL>
__device__ __forceinline__ void get(const ScanArgs& a, const char* raw, int k, int t, int ec, float (&f)[4]) {
    const int at = k * Tile<NL>::PLANE + t * Tile<NL>::CT + ec;
    if (a.dtype == HC_DTYPE_F32)
        load_pack<float, 4>(reinterpret_cast<const float*>(raw) + at, f);
    else if (a.dtype == HC_DTYPE_BF16)
        load_pack<__nv_bfloat16, 4>(reinterpret_cast<const __nv_bfloat16*>(raw) + at, f);
    else
        load_pack<__half, 4>(reinterpret_cast<const __half*>(raw) + at, f);
}
// A tile's B and C, a few values a thread, held as loaded until put_bc.
template <int NL>
__device__ __forceinline__ void fetch_bc(const ScanArgs& a, const Where& w, int t0, unsigned (&bc)[Tile<NL>::BC]) {
    using S = Tile<NL>;
    const int sh = a.dtype == HC_DTYPE_F32 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < S::BC; i++) {
        const int q = threadIdx.x + i * S::THREADS;
        const int t = q / S::NP % SC_T, n = q % S::NP;
        const hc_rows& r = q / (SC_T * S::NP) ? a.Cm : a.Bm;
        bc[i] = 0;
        if (t0 + t < w.len && n < a.N) {
            const char* p = static_cast<const char*>(r.p) + ((w.b * r.batch + (t0 + t) * r.row + w.g * a.N + n) << sh);
            bc[i] = sh == 2 ? *reinterpret_cast<const unsigned*>(p) : *reinterpret_cast<const unsigned short*>(p);
        }
    }
}
// To bc2[2][T][NP], each value twice (a pair for the packed multiply-adds).
template <int NL>
__device__ __forceinline__ void put_bc(const ScanArgs& a, const unsigned (&bc)[Tile<NL>::BC], f32x2* bc2) {
#pragma unroll
    for (int i = 0; i < Tile<NL>::BC; i++) {
        const float v = a.dtype == HC_DTYPE_F32    ? __uint_as_float(bc[i])
                        : a.dtype == HC_DTYPE_BF16 ? __uint_as_float(bc[i] << 16)
                                                   : __half2float(__ushort_as_half((unsigned short)bc[i]));
        bc2[threadIdx.x + i * Tile<NL>::THREADS] = pk2(v, v);
    }
}

__device__ __forceinline__ void ld_pairs(const float* p, f32x2 (&v)[2]) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p);
    v[0] = q.x;
    v[1] = q.y;
}
__device__ __forceinline__ void ld_dup(const f32x2* p, f32x2 (&v)[4]) {
    const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(p), r = *reinterpret_cast<const ulonglong2*>(p + 2);
    v[0] = q.x;
    v[1] = q.y;
    v[2] = r.x;
    v[3] = r.y;
}
// The four channels' four states each as channel pairs, from rows of fp32
// states (`padded`: rows of NP with every state there, else rows of N).
template <int NL>
__device__ __forceinline__ void ld_tile(const float* p, long long step, int n, int N, bool padded, int tc, int cn,
                                        f32x2 (&v)[2][4]) {
    float f[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
        for (int j = 0; j < 4; j++) f[i][j] = 0.0f;
        if (p && tc + i < cn) {
            if (padded)
                load_pack<float, 4>(p + i * step + 4 * n, f[i]);
            else
                ld_states(p + i * step, 4 * n, N, f[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) v[i][j] = pk2(f[2 * i][j], f[2 * i + 1][j]);
}
template <int NL>
__device__ __forceinline__ void st_tile(float* p, long long step, int n, int N, bool padded, int tc, int cn,
                                        const f32x2 (&v)[2][4]) {
    float f[4][4];
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) unpk2(v[i][j], f[2 * i][j], f[2 * i + 1][j]);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (tc + i >= cn) continue;
        if (padded)
            store_pack<float, 4>(p + i * step + 4 * n, f[i]);
        else
            st_states(p + i * step, 4 * n, N, f[i]);
    }
}
template <int NL>
__device__ __forceinline__ void ld_rates(const ScanArgs& a, int d, int n, int tc, int cn, f32x2 (&A2)[2][4]) {
    ld_tile<NL>(a.A + (long long)d * a.N, a.N, n, a.N, false, tc, cn, A2);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] = mul2(A2[i][j], pk2(kLog2e, kLog2e));
}

// Sums y over a channel group's NL lanes and writes the channels' totals to row[0 .. 4).
template <int NL> __device__ __forceinline__ void put_lanes_sum(f32x2 a, f32x2 b, int n, float* row) {
    float y[4];
    unpk2(a, y[0], y[1]);
    unpk2(b, y[2], y[3]);
    const int first = lanes_sum<4, NL>(y, n);
    constexpr int KEEP = NL >= 4 ? 1 : 4 / NL;
    if (NL <= 4 || n < 4) {
#pragma unroll
        for (int i = 0; i < KEEP; i++) row[first + i] = y[i];
    }
}
// Sums v over a warp's channel groups (lanes n, n + NL, ...) and writes the four states' totals to out[0 .. 4).
template <int NL> __device__ __forceinline__ void put_groups_sum(const f32x2 (&v)[4], int lane, float* out) {
    constexpr int CG = 32 / NL;
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float lo, hi;
        unpk2(v[j], lo, hi);
        f[j] = lo + hi;
    }
    int at = 0, left = 4;
#pragma unroll
    for (int o = NL; o < 32; o <<= 1) {
        if (left > 1) {
            const int half = left / 2;
            const bool up = (lane & o) != 0;
#pragma unroll
            for (int i = 0; i < 2; i++) {
                if (i < half) {
                    const float send = up ? f[i] : f[i + half], keep = up ? f[i + half] : f[i];
                    f[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                }
            }
            at += up ? half : 0;
            left = half;
        } else {
            f[0] += __shfl_xor_sync(0xffffffffu, f[0], o);
        }
    }
    constexpr int KEEP = CG >= 4 ? 1 : 4 / CG;
    if (CG <= 4 || lane / NL < 4) {
#pragma unroll
        for (int i = 0; i < KEEP; i++) out[at + i] = f[i];
    }
}

// dt_bias and D of a block's channels to shared memory: bD[2][CT].
template <int NL> __device__ __forceinline__ void put_params(const ScanArgs& a, const Where& w, float* bD) {
    for (int c = threadIdx.x; c < Tile<NL>::CT; c += Tile<NL>::THREADS) {
        bD[c] = a.bias && c < w.cn ? a.bias[w.d0 + c] : 0.0f;
        bD[Tile<NL>::CT + c] = a.D && c < w.cn ? a.D[w.d0 + c] : 0.0f;
    }
}
// The step sizes of four channels, from dt + dt_bias.
__device__ __forceinline__ void steps(const ScanArgs& a, bool on, float (&s)[4]) {
#pragma unroll
    for (int k = 0; k < 4; k++) s[k] = on ? (a.softplus ? softplus_f(s[k]) : s[k]) : 0.0f;
}
__device__ __forceinline__ void add4(float (&a)[4], const float* p) {
    float b[4];
    load_pack<float, 4>(p, b);
#pragma unroll
    for (int k = 0; k < 4; k++) a[k] += b[k];
}

template <int NL> constexpr size_t fwd_smem() {
    using S = Tile<NL>;
    return sizeof(float) * (5 * S::PLANE + 2 * S::CT + 4 * SC_T * S::NP + 3 * S::PLANE);
}
template <int NL> __global__ void __launch_bounds__(Tile<NL>::THREADS) scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = Tile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // step sizes
    float* xs = dl + S::PLANE;                  // step * u
    float* us = xs + S::PLANE;                  // D * u
    float* gs = us + S::PLANE;                  // silu(z)
    float* ys = gs + S::PLANE;                  // C . h
    float* bD = ys + S::PLANE;                             // dt_bias, D
    f32x2* bc2 = reinterpret_cast<f32x2*>(bD + 2 * S::CT);  // [B, C][T][NP], twice each
    char* raw = reinterpret_cast<char*>(bc2 + 2 * SC_T * S::NP);
    const int lane = threadIdx.x & 31, n = lane % NL, tc = (threadIdx.x >> 5) * S::WC + lane / NL * 4;
    const Where w(a, S::CT);
    const bool gate = a.z.p != nullptr;
    f32x2 A2[2][4], h[2][4];
    ld_rates<NL>(a, w.d0 + tc, n, tc, w.cn, A2);
    if (a.segs > 1)
        ld_tile<NL>(a.carry + ((long long)w.bs * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc, w.cn, h);
    else
        ld_tile<NL>(a.h0 ? a.h0 + ((long long)w.b * a.Dm + w.d0 + tc) * a.N : nullptr, a.N, n, a.N, false, tc, w.cn, h);
    put_params<NL>(a, w, bD);
    unsigned bc[S::BC];
    const auto start = [&](int t0) {
        const Walk<NL> at;
        fetch<NL>(a, a.dt, w, at, t0, 0, raw);
        fetch<NL>(a, a.u, w, at, t0, 1, raw);
        if (gate) fetch<NL>(a, a.z, w, at, t0, 2, raw);
        fetch_bc<NL>(a, w, t0, bc);
    };
    const int live1 = w.live1();
    if (w.tile0 < live1) start(w.tile0 * SC_T);
    for (int tile = w.tile0; tile < live1; tile++) {
        const int t0 = tile * SC_T;
        cp_async_wait();
        __syncthreads();
        for (Walk<NL> at; at.er < SC_T; at.er += S::ROWS) {
            const int t = at.er, q = t * S::CT + at.ec;
            float s[4], x[4], D[4];
            get<NL>(a, raw, 0, t, at.ec, s);
            get<NL>(a, raw, 1, t, at.ec, x);
            load_pack<float, 4>(bD + S::CT + at.ec, D);
            add4(s, bD + at.ec);
            steps(a, t0 + t < w.len, s);
            store_pack<float, 4>(dl + q, s);
#pragma unroll
            for (int k = 0; k < 4; k++) {
                D[k] *= x[k];
                x[k] *= s[k];
            }
            store_pack<float, 4>(xs + q, x);
            store_pack<float, 4>(us + q, D);
            if (gate) {
                get<NL>(a, raw, 2, t, at.ec, s);
#pragma unroll
                for (int k = 0; k < 4; k++) s[k] = silu_f(s[k]);
                store_pack<float, 4>(gs + q, s);
            }
        }
        put_bc<NL>(a, bc, bc2);
        __syncthreads();
        if (tile + 1 < live1) start(t0 + SC_T);
        if (a.saved)
            st_tile<NL>(a.saved + (((long long)w.b * a.tiles + tile) * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc,
                        w.cn, h);
#pragma unroll 4
        for (int t = 0; t < SC_T; t++) {
            f32x2 s[2], x[2], B[4], C[4], y[2];
            ld_pairs(dl + t * S::CT + tc, s);
            ld_pairs(xs + t * S::CT + tc, x);
            ld_dup(bc2 + t * S::NP + 4 * n, B);
            ld_dup(bc2 + (SC_T + t) * S::NP + 4 * n, C);
#pragma unroll
            for (int i = 0; i < 2; i++) {
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    h[i][j] = fma2(ex2x2(mul2(s[i], A2[i][j])), h[i][j], mul2(x[i], B[j]));
                    y[i] = j ? fma2(C[j], h[i][j], y[i]) : mul2(C[j], h[i][j]);
                }
            }
            put_lanes_sum<NL>(y[0], y[1], n, ys + t * S::CT + tc);
        }
        __syncthreads();
        const int rows = min(SC_T, a.L - t0);
        for (Walk<NL> at; at.er < rows; at.er += S::ROWS) {
            const int t = at.er, q = t * S::CT + at.ec;
            float o[4], z[4];
            load_pack<float, 4>(ys + q, o);
            add4(o, us + q);
            if (gate) {
                load_pack<float, 4>(gs + q, z);
#pragma unroll
                for (int k = 0; k < 4; k++) o[k] *= z[k];
            }
            if (t0 + t >= w.len) o[0] = o[1] = o[2] = o[3] = 0.0f;
            st4(a.y.p, w.b * a.y.batch + (t0 + t) * a.y.row + w.d0, a.dtype, at.ec, w.cn, a.vec, o);
        }
    }
    // rows past the sequence's last tile
    const int end = min(w.tile1 * SC_T, a.L);
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const Walk<NL> at;
    for (int t = live1 * SC_T + at.er; t < end && at.er < S::ROWS; t += S::ROWS)
        st4(a.y.p, w.b * a.y.batch + t * a.y.row + w.d0, a.dtype, at.ec, w.cn, a.vec, zero);
    if (a.hT && w.seg == a.segs - 1)
        st_tile<NL>(a.hT + ((long long)w.b * a.Dm + w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, h);
}

// A segment's state from a zero state.  REV false: the state itself, over
// x = step * u and B, rows upwards.  REV true: the state's gradient, over
// q = gy * silu(z) and C, rows downwards: G_{t-1} = exp(step_t A) (G_t + q_t C_t).
template <int NL> constexpr size_t carry_smem() {
    using S = Tile<NL>;
    return sizeof(float) * (2 * S::PLANE + 2 * S::CT + 4 * SC_T * S::NP + 3 * S::PLANE);
}
template <int NL, bool REV>
__global__ void __launch_bounds__(Tile<NL>::THREADS) scan_carry_kernel(const __grid_constant__ ScanArgs a) {
    using S = Tile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);
    float* xs = dl + S::PLANE;
    float* bD = xs + S::PLANE;
    f32x2* bc2 = reinterpret_cast<f32x2*>(bD + 2 * S::CT);
    char* raw = reinterpret_cast<char*>(bc2 + 2 * SC_T * S::NP);
    const int lane = threadIdx.x & 31, n = lane % NL, tc = (threadIdx.x >> 5) * S::WC + lane / NL * 4;
    const Where w(a, S::CT);
    f32x2 A2[2][4], h[2][4], sum[2];
    ld_rates<NL>(a, w.d0 + tc, n, tc, w.cn, A2);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        sum[i] = pk2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; j++) h[i][j] = sum[i];
    }
    put_params<NL>(a, w, bD);
    unsigned bc[S::BC];
    const bool gate = REV && a.z.p;
    const auto start = [&](int t0) {
        const Walk<NL> at;
        fetch<NL>(a, a.dt, w, at, t0, 0, raw);
        fetch<NL>(a, REV ? a.gy : a.u, w, at, t0, 1, raw);
        if (gate) fetch<NL>(a, a.z, w, at, t0, 2, raw);
        fetch_bc<NL>(a, w, t0, bc);
    };
    const int tiles = w.live1() - w.tile0;
    const int first = REV ? w.tile0 + tiles - 1 : w.tile0, dir = REV ? -1 : 1;
    if (tiles > 0) start(first * SC_T);
    for (int k = 0; k < tiles; k++) {
        const int t0 = (first + dir * k) * SC_T;
        cp_async_wait();
        __syncthreads();
        for (Walk<NL> at; at.er < SC_T; at.er += S::ROWS) {
            const int t = at.er, q = t * S::CT + at.ec;
            float s[4], x[4], z[4];
            get<NL>(a, raw, 0, t, at.ec, s);
            get<NL>(a, raw, 1, t, at.ec, x);
            add4(s, bD + at.ec);
            steps(a, t0 + t < w.len, s);
            if (!REV) {
#pragma unroll
                for (int i = 0; i < 4; i++) x[i] *= s[i];
            } else if (gate) {
                get<NL>(a, raw, 2, t, at.ec, z);
#pragma unroll
                for (int i = 0; i < 4; i++) x[i] *= silu_f(z[i]);
            }
            store_pack<float, 4>(dl + q, s);
            store_pack<float, 4>(xs + q, x);
        }
        put_bc<NL>(a, bc, bc2);
        __syncthreads();
        if (k + 1 < tiles) start(t0 + dir * SC_T);
#pragma unroll 4
        for (int v = 0; v < SC_T; v++) {
            const int t = REV ? SC_T - 1 - v : v;
            f32x2 s[2], x[2], B[4];
            ld_pairs(dl + t * S::CT + tc, s);
            ld_pairs(xs + t * S::CT + tc, x);
            ld_dup(bc2 + ((REV ? SC_T : 0) + t) * S::NP + 4 * n, B);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                sum[i] = add2(sum[i], s[i]);
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const f32x2 e = ex2x2(mul2(s[i], A2[i][j]));
                    h[i][j] = REV ? mul2(e, fma2(x[i], B[j], h[i][j])) : fma2(e, h[i][j], mul2(x[i], B[j]));
                }
            }
        }
        __syncthreads();
    }
    const long long d = (long long)w.bs * a.Dm + w.d0 + tc;
    st_tile<NL>(a.carry + d * S::NP, S::NP, n, a.N, true, tc, w.cn, h);
    if (n == 0) {
        float t[4];
        unpk2(sum[0], t[0], t[1]);
        unpk2(sum[1], t[2], t[3]);
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (tc + i < w.cn) a.dsum[d + i] = t[i];
    }
}

// Replaces every segment's local result by the state it starts from.  A block
// takes SJ_STATES adjacent states of a sequence, its 32 rows of threads equal
// runs of segments: each run is joined, the runs' results are joined in order
// through shared memory, and each run is gone through again.
constexpr int SJ_STATES = 32;
template <bool REV>
__global__ void __launch_bounds__(1024) scan_join_kernel(const __grid_constant__ ScanArgs a, int NP) {
    __shared__ float hs[32][SJ_STATES + 1], as[32][SJ_STATES + 1];
    const int col = threadIdx.x % SJ_STATES, r = threadIdx.x / SJ_STATES;
    const int b = blockIdx.y;
    const long long q = (long long)blockIdx.x * SJ_STATES + col;
    const bool on = q < (long long)a.Dm * NP;
    const int d = on ? (int)(q / NP) : 0, n = on ? (int)(q % NP) : 0;
    const float A2 = on && n < a.N ? a.A[(long long)d * a.N + n] * kLog2e : 0.0f;
    const int per = (a.segs + 31) / 32, s0 = r * per, s1 = min(s0 + per, a.segs);
    float* cp = a.carry + (long long)b * a.segs * a.Dm * NP + (on ? q : 0);
    const float* dp = a.dsum + (long long)b * a.segs * a.Dm + d;
    const long long hstep = (long long)a.Dm * NP;
    float h = 0.0f, total = 0.0f;
#pragma unroll 4
    for (int k = s0; k < s1; k++) {
        const int s = REV ? a.segs - 1 - k : k;
        const float w = dp[(long long)s * a.Dm];
        h = fmaf(ex2f(w * A2), h, cp[s * hstep]);
        total += w;
    }
    hs[r][col] = h;
    as[r][col] = total;
    __syncthreads();
    const float* first = REV ? a.ghT : a.h0;
    h = first && on && n < a.N ? first[((long long)b * a.Dm + d) * a.N + n] : 0.0f;
    for (int k = 0; k < r; k++) h = fmaf(ex2f(as[k][col] * A2), h, hs[k][col]);
    if (!on) return;
#pragma unroll 4
    for (int k = s0; k < s1; k++) {
        const int s = REV ? a.segs - 1 - k : k;
        const float v = cp[s * hstep], w = dp[(long long)s * a.Dm];
        cp[s * hstep] = h;
        h = fmaf(ex2f(w * A2), h, v);
    }
}

// A block's tiles from the last to the first.  A tile's states are recomputed
// from its saved first state and kept in registers (H), with y and gC on the
// way, then the state's gradient runs back through them.
template <int NL> constexpr size_t bwd_smem() {
    using S = Tile<NL>;
    return sizeof(float) * (9 * S::PLANE + 2 * S::CT + 2 * S::ROWS * S::CT + 4 * SC_T * S::NP + S::W * SC_T * 2 * S::NP +
                            4 * S::PLANE);
}
template <int NL>
__global__ void __launch_bounds__(Tile<NL>::THREADS) scan_bwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = Tile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // step sizes
    float* us = dl + S::PLANE;                  // u
    float* xs = us + S::PLANE;                  // step * u
    float* qs = xs + S::PLANE;                  // gy * silu(z)
    float* ps = qs + S::PLANE;                  // slope of the step size
    float* ws = ps + S::PLANE;                  // gy * silu'(z)
    float* ys = ws + S::PLANE;                  // C . h
    float* GB = ys + S::PLANE;                  // G . B
    float* EA = GB + S::PLANE;                  // E . A / ln 2
    float* bD = EA + S::PLANE;                  // dt_bias, D
    float* sums = bD + 2 * S::CT;               // [ROWS][2][CT], each thread's gD and gdt_bias
    f32x2* bc2 = reinterpret_cast<f32x2*>(sums + 2 * S::ROWS * S::CT);
    float* red = reinterpret_cast<float*>(bc2 + 2 * SC_T * S::NP);  // [W][T][2][NP], the warps' gB and gC
    char* raw = reinterpret_cast<char*>(red + S::W * SC_T * 2 * S::NP);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane % NL, tc = warp * S::WC + lane / NL * 4;
    const Where w(a, S::CT);
    const bool gate = a.z.p != nullptr;
    f32x2 A2[2][4], G[2][4], gA[2][4];
    ld_rates<NL>(a, w.d0 + tc, n, tc, w.cn, A2);
    if (a.segs > 1)
        ld_tile<NL>(a.carry + ((long long)w.bs * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc, w.cn, G);
    else
        ld_tile<NL>(a.ghT ? a.ghT + ((long long)w.b * a.Dm + w.d0 + tc) * a.N : nullptr, a.N, n, a.N, false, tc, w.cn,
                    G);
#pragma unroll
    for (int i = 0; i < 2; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) gA[i][j] = pk2(0.0f, 0.0f);
    put_params<NL>(a, w, bD);
    for (int q = tid; q < 2 * S::ROWS * S::CT; q += S::THREADS) sums[q] = 0.0f;
    unsigned bc[S::BC];
    const auto start = [&](int t0) {
        const Walk<NL> at;
        fetch<NL>(a, a.dt, w, at, t0, 0, raw);
        fetch<NL>(a, a.u, w, at, t0, 1, raw);
        fetch<NL>(a, a.gy, w, at, t0, 2, raw);
        if (gate) fetch<NL>(a, a.z, w, at, t0, 3, raw);
        fetch_bc<NL>(a, w, t0, bc);
    };
    const int live1 = w.live1();
    __syncthreads();
    if (w.tile0 < live1) start((live1 - 1) * SC_T);
    for (int tile = w.tile1 - 1; tile >= w.tile0; tile--) {
        const int t0 = tile * SC_T, rows = min(SC_T, a.L - t0);
        const bool live = tile < live1;
        if (live) {
            cp_async_wait();
            __syncthreads();
            for (Walk<NL> at; at.er < SC_T; at.er += S::ROWS) {
                const int t = at.er, c = t * S::CT + at.ec;
                float s[4], u[4], q[4], p[4];
                get<NL>(a, raw, 0, t, at.ec, s);
                get<NL>(a, raw, 1, t, at.ec, u);
                get<NL>(a, raw, 2, t, at.ec, q);
                add4(s, bD + at.ec);
#pragma unroll
                for (int k = 0; k < 4; k++) p[k] = a.softplus ? sigmoid_f(s[k]) : 1.0f;
                steps(a, t0 + t < w.len, s);
                store_pack<float, 4>(dl + c, s);
                store_pack<float, 4>(us + c, u);
                store_pack<float, 4>(ps + c, p);
#pragma unroll
                for (int k = 0; k < 4; k++) u[k] *= s[k];
                store_pack<float, 4>(xs + c, u);
                if (gate) {
                    get<NL>(a, raw, 3, t, at.ec, u);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float r = sigmoid_f(u[k]);
                        p[k] = q[k] * r * fmaf(u[k], 1.0f - r, 1.0f);
                        q[k] *= u[k] * r;
                    }
                    store_pack<float, 4>(ws + c, p);
                }
                store_pack<float, 4>(qs + c, q);
            }
            put_bc<NL>(a, bc, bc2);
            __syncthreads();
            if (tile > w.tile0) start(t0 - SC_T);
            const float* first =
                a.saved + (((long long)w.b * a.tiles + tile) * a.Dm + w.d0 + tc) * S::NP;
            // H[t] is the state before row t (H[0] is read again where it is needed again)
            f32x2 H[SC_T][2][4], h[2][4];
            ld_tile<NL>(first, S::NP, n, a.N, true, tc, w.cn, h);
#pragma unroll
            for (int t = 0; t < SC_T; t++) {
                f32x2 s[2], x[2], q[2], B[4], C[4], y[2], gc[4];
                ld_pairs(dl + t * S::CT + tc, s);
                ld_pairs(xs + t * S::CT + tc, x);
                ld_pairs(qs + t * S::CT + tc, q);
                ld_dup(bc2 + t * S::NP + 4 * n, B);
                ld_dup(bc2 + (SC_T + t) * S::NP + 4 * n, C);
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        if (t) H[t][i][j] = h[i][j];
                        h[i][j] = fma2(ex2x2(mul2(s[i], A2[i][j])), h[i][j], mul2(x[i], B[j]));
                        y[i] = j ? fma2(C[j], h[i][j], y[i]) : mul2(C[j], h[i][j]);
                        gc[j] = i ? fma2(q[i], h[i][j], gc[j]) : mul2(q[i], h[i][j]);
                    }
                }
                if (gate) put_lanes_sum<NL>(y[0], y[1], n, ys + t * S::CT + tc);
                put_groups_sum<NL>(gc, lane, red + ((warp * SC_T + t) * 2 + 1) * S::NP + 4 * n);
            }
            // nothing of the way up is kept for the way down but H: the exponentials are taken again
            asm volatile("" ::: "memory");
            // gA summed tile by tile: one running sum over all rows would lose more
            f32x2 ga[2][4];
#pragma unroll
            for (int t = SC_T - 1; t >= 0; t--) {
                f32x2 s[2], x[2], q[2], B[4], C[4], gb[2], ea[2], gB[4];
                ld_pairs(dl + t * S::CT + tc, s);
                ld_pairs(xs + t * S::CT + tc, x);
                ld_pairs(qs + t * S::CT + tc, q);
                ld_dup(bc2 + t * S::NP + 4 * n, B);
                ld_dup(bc2 + (SC_T + t) * S::NP + 4 * n, C);
                if (t == 0) ld_tile<NL>(first, S::NP, n, a.N, true, tc, w.cn, H[0]);
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const f32x2 g = fma2(q[i], C[j], G[i][j]);
                        gB[j] = i ? fma2(g, x[i], gB[j]) : mul2(g, x[i]);
                        gb[i] = j ? fma2(g, B[j], gb[i]) : mul2(g, B[j]);
                        G[i][j] = mul2(g, ex2x2(mul2(s[i], A2[i][j])));
                        const f32x2 E = mul2(G[i][j], H[t][i][j]);
                        ea[i] = j ? fma2(E, A2[i][j], ea[i]) : mul2(E, A2[i][j]);
                        ga[i][j] = t == SC_T - 1 ? mul2(E, s[i]) : fma2(E, s[i], ga[i][j]);
                    }
                }
                put_lanes_sum<NL>(gb[0], gb[1], n, GB + t * S::CT + tc);
                put_lanes_sum<NL>(ea[0], ea[1], n, EA + t * S::CT + tc);
                put_groups_sum<NL>(gB, lane, red + (warp * SC_T + t) * 2 * S::NP + 4 * n);
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) gA[i][j] = add2(gA[i][j], ga[i][j]);
            __syncthreads();
        }
        for (Walk<NL> at; at.er < rows; at.er += S::ROWS) {
            const int t = at.er, c = t * S::CT + at.ec;
            float gu[4] = {0, 0, 0, 0}, gd[4] = {0, 0, 0, 0}, gz[4] = {0, 0, 0, 0};
            if (t0 + t < w.len) {
                float b[4], e[4], u[4], q[4], D[4], v[4];
                float* sum = sums + (t % S::ROWS) * 2 * S::CT + at.ec;
                load_pack<float, 4>(GB + c, b);
                load_pack<float, 4>(us + c, u);
                load_pack<float, 4>(qs + c, q);
                load_pack<float, 4>(bD + S::CT + at.ec, D);
                load_pack<float, 4>(dl + c, v);
#pragma unroll
                for (int k = 0; k < 4; k++) gu[k] = fmaf(b[k], v[k], D[k] * q[k]);
                load_pack<float, 4>(EA + c, e);
                load_pack<float, 4>(ps + c, v);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    gd[k] = fmaf(b[k], u[k], e[k] * kLn2) * v[k];
                    b[k] = gd[k];
                    q[k] *= u[k];
                }
                add4(q, sum);
                store_pack<float, 4>(sum, q);
                add4(b, sum + S::CT);
                store_pack<float, 4>(sum + S::CT, b);
                if (gate) {
                    load_pack<float, 4>(ys + c, e);
                    load_pack<float, 4>(ws + c, v);
#pragma unroll
                    for (int k = 0; k < 4; k++) gz[k] = v[k] * fmaf(D[k], u[k], e[k]);
                }
            }
            st4(a.gu.p, w.b * a.gu.batch + (t0 + t) * a.gu.row + w.d0, a.dtype, at.ec, w.cn, a.vec, gu);
            st4(a.gdt.p, w.b * a.gdt.batch + (t0 + t) * a.gdt.row + w.d0, a.dtype, at.ec, w.cn, a.vec, gd);
            if (gate) st4(a.gz.p, w.b * a.gz.batch + (t0 + t) * a.gz.row + w.d0, a.dtype, at.ec, w.cn, a.vec, gz);
        }
        for (int q = tid; q < rows * 2 * S::NP; q += S::THREADS) {
            const int t = q / (2 * S::NP), c = (q / S::NP) & 1, k = q % S::NP;
            if (k >= a.N) continue;
            float v = 0.0f;
            if (t0 + t < w.len) {
#pragma unroll
                for (int m = 0; m < S::W; m++) v += red[(m * SC_T + t) * 2 * S::NP + c * S::NP + k];
            }
            if (a.gbc) {
                a.gbc[((((long long)(w.c0 / S::CT) * a.B + w.b) * a.L + t0 + t) * a.G + w.g) * 2 * a.N + c * a.N + k] = v;
            } else {
                const hc_rows& o = c ? a.gC : a.gB;
                st1(o.p, w.b * o.batch + (t0 + t) * o.row + w.g * a.N + k, a.dtype, v);
            }
        }
    }
    float* pb = a.part + (long long)w.bs * (a.N + 2) * a.Dm;
    st_tile<NL>(pb + (long long)(w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, gA);
    if (a.gh0 && w.seg == 0)
        st_tile<NL>(a.gh0 + ((long long)w.b * a.Dm + w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, G);
    // gD and gdt_bias over the rows of threads, in order
    __syncthreads();
    for (int c = tid; c < w.cn; c += S::THREADS) {
        float x = 0.0f, y = 0.0f;
        for (int r = 0; r < S::ROWS; r++) {
            x += sums[r * 2 * S::CT + c];
            y += sums[(r * 2 + 1) * S::CT + c];
        }
        pb[(long long)a.N * a.Dm + w.d0 + c] = x;
        pb[(long long)(a.N + 1) * a.Dm + w.d0 + c] = y;
    }
}

// gB and gC: the channel tiles' sums in tile order.
__global__ void __launch_bounds__(256) scan_bc_kernel(const __grid_constant__ ScanArgs a) {
    const long long per = (long long)a.B * a.L * a.G * 2 * a.N;
    for (long long q = blockIdx.x * 256LL + threadIdx.x; q < per; q += gridDim.x * 256LL) {
        float v = 0.0f;
        for (int m = 0; m < a.ctiles; m++) v += a.gbc[m * per + q];
        const int k = (int)(q % a.N), w = (int)(q / a.N % 2), g = (int)(q / (2 * a.N) % a.G);
        const long long t = q / (2LL * a.N * a.G);
        const hc_rows& o = w ? a.gC : a.gB;
        st1(o.p, t / a.L * o.batch + t % a.L * o.row + g * a.N + k, a.dtype, v);
    }
}

// One token: NL lanes a channel, 32 / NL channels a warp.
template <int NL>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanArgs a, float* __restrict__ state) {
    const int lane = threadIdx.x & 31, n = lane % NL;
    const long long q = (blockIdx.x * 4LL + (threadIdx.x >> 5)) * (32 / NL) + lane / NL;
    const bool on = q < (long long)a.B * a.Dm;
    const int b = on ? (int)(q / a.Dm) : 0, d = on ? (int)(q % a.Dm) : 0, g = d / a.Dg;
    float* hp = state + ((long long)b * a.Dm + d) * a.N;
    float h[4], A[4], B[4], C[4];
    ld_states(hp, 4 * n, a.N, h);
    ld_states(a.A + (long long)d * a.N, 4 * n, a.N, A);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const bool in = 4 * n + k < a.N;
        B[k] = in ? ld1(a.Bm.p, b * a.Bm.batch + g * a.N + 4 * n + k, a.dtype) : 0.0f;
        C[k] = in ? ld1(a.Cm.p, b * a.Cm.batch + g * a.N + 4 * n + k, a.dtype) : 0.0f;
    }
    const float u = ld1(a.u.p, b * a.u.batch + d, a.dtype);
    float s = ld1(a.dt.p, b * a.dt.batch + d, a.dtype) + (a.bias ? a.bias[d] : 0.0f);
    if (a.softplus) s = softplus_f(s);
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        h[k] = fmaf(ex2f(s * (A[k] * kLog2e)), h[k], s * u * B[k]);
        y = fmaf(C[k], h[k], y);
    }
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!on) return;
    st_states(hp, 4 * n, a.N, h);
    if (n == 0) {
        if (a.D) y = fmaf(a.D[d], u, y);
        if (a.z.p) y *= silu_f(ld1(a.z.p, b * a.z.batch + d, a.dtype));
        st1(a.y.p, b * a.y.batch + d, a.dtype, y);
    }
}

bool scan_desc_ok(const hc_selective_scan_desc* d) {
    return d && d->B > 0 && d->L >= 0 && d->D > 0 && d->groups > 0 && d->D % d->groups == 0 && d->d_state > 0 &&
           (d->softplus == 0 || d->softplus == 1) && dtype_ok(d->dtype);
}
// Launch limits: (sequence, segment, channel tile) on grid x, sequences on grid y.
bool scan_size_ok(const hc_selective_scan_desc* d) {
    return d->d_state <= 64 && d->D <= (1 << 20) && d->B <= 65535 && (long long)d->B * d->D < (1LL << 31) &&
           d->L <= 0x7fffffff - 64;
}
int scan_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

template <typename F> hc_status scan_dispatch(int N, F&& f) {
    switch (scan_lanes(N)) {
        case 1: return f.template operator()<1>();
        case 2: return f.template operator()<2>();
        case 4: return f.template operator()<4>();
        case 8: return f.template operator()<8>();
    }
    return f.template operator()<16>();
}

// Channel tiles a group (Tile<NL>::CT channels each).
int scan_ctiles(const hc_selective_scan_desc* d) {
    const int nl = scan_lanes(d->d_state);
    return (int)cdiv(d->D / d->groups, nl <= 4 ? 128 : 512 / nl);
}

// Segments: none where (sequence, channel tile) blocks give every SM `want` of
// them, else as many as make up for it, of two tiles at least.
struct Segs {
    int n, tiles;
};
Segs scan_segs(const hc_selective_scan_desc* d, int want) {
    const int tiles = (int)cdiv(d->L, SC_T);
    const long long blocks = (long long)d->B * d->groups * scan_ctiles(d), full = (long long)want * device_sm_count();
    if (blocks * 2 > full || tiles < 4) return {1, tiles > 0 ? tiles : 1};
    long long n = full / blocks;
    if (n > tiles / 2) n = tiles / 2;
    const int per = (int)cdiv(tiles, n);
    return {(int)cdiv(tiles, per), per};
}
Segs fwd_segs(const hc_selective_scan_desc* d) { return scan_segs(d, 4); }
Segs bwd_segs(const hc_selective_scan_desc* d) { return scan_segs(d, 2); }

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
size_t carry_floats(const hc_selective_scan_desc* d, int segs) {
    return segs > 1 ? (size_t)d->B * segs * d->D * 4 * scan_lanes(d->d_state) : 0;
}
size_t carry_bytes(const hc_selective_scan_desc* d, int segs) {
    return up256(4 * carry_floats(d, segs)) + up256(segs > 1 ? 4 * (size_t)d->B * segs * d->D : 0);
}
size_t part_bytes(const hc_selective_scan_desc* d) {
    return up256(sizeof(float) * d->B * bwd_segs(d).n * (size_t)(d->d_state + 2) * d->D);
}
void set_segs(ScanArgs& a, const hc_selective_scan_desc* d, Segs s, void* ws) {
    a.segs = s.n;
    a.seg_tiles = s.tiles;
    a.carry = (float*)ws;
    a.dsum = (float*)((char*)ws + up256(4 * carry_floats(d, s.n)));
}

ScanArgs scan_args(const hc_selective_scan_desc* d, const hc_scan_in* in) {
    ScanArgs a = {};
    a.u = in->u;
    a.dt = in->dt;
    a.Bm = in->Bm;
    a.Cm = in->Cm;
    a.z = in->z;
    a.A = in->A;
    a.D = in->D;
    a.bias = in->dt_bias;
    a.B = d->B;
    a.L = d->L;
    a.Dm = d->D;
    a.G = d->groups;
    a.Dg = d->D / d->groups;
    a.N = d->d_state;
    a.dtype = d->dtype;
    a.softplus = d->softplus;
    a.tiles = (int)cdiv(d->L, SC_T);
    a.ctiles = scan_ctiles(d);
    return a;
}

bool scan_in_ok(const hc_selective_scan_desc* d, const hc_scan_in* in, long long rows) {
    return in && rows_in_ok(&in->u, d->dtype, rows) && rows_in_ok(&in->dt, d->dtype, rows) &&
           rows_in_ok(&in->Bm, d->dtype, rows) && rows_in_ok(&in->Cm, d->dtype, rows) &&
           (!in->z.p || rows_in_ok(&in->z, d->dtype, rows)) && f32_ok(in->A) && f32_opt_ok(in->D) &&
           f32_opt_ok(in->dt_bias);
}

// The first states of the segments (REV: of the gradient, from the last row up).
template <int NL, bool REV> hc_status launch_scan_carry(ScanArgs a, cudaStream_t st) {
    using S = Tile<NL>;
    static std::atomic<unsigned long long> attr{0};
    once_per_device(attr, [] {
        return cudaFuncSetAttribute(scan_carry_kernel<NL, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)carry_smem<NL>()) == cudaSuccess;
    });
    scan_carry_kernel<NL, REV><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, carry_smem<NL>(), st>>>(a);
    hc_status e = launched("scan_carry_kernel", st);
    if (e) return e;
    scan_join_kernel<REV><<<dim3(cdiv((long long)a.Dm * S::NP, SJ_STATES), a.B), 1024, 0, st>>>(a, S::NP);
    return launched("scan_join_kernel", st);
}

struct ScanFwd {
    ScanArgs a;
    cudaStream_t st;
    template <int NL> hc_status operator()() {
        using S = Tile<NL>;
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_fwd_kernel<NL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)fwd_smem<NL>()) == cudaSuccess;
        });
        if (a.segs > 1) {
            const hc_status e = launch_scan_carry<NL, false>(a, st);
            if (e) return e;
        }
        scan_fwd_kernel<NL><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, fwd_smem<NL>(), st>>>(a);
        return launched("scan_fwd_kernel", st);
    }
};

struct ScanBwd {
    ScanArgs a;
    const hc_scan_grad* g;
    cudaStream_t st;
    template <int NL> hc_status operator()() {
        using S = Tile<NL>;
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_bwd_kernel<NL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)bwd_smem<NL>()) == cudaSuccess;
        });
        if (a.segs > 1) {
            const hc_status e = launch_scan_carry<NL, true>(a, st);
            if (e) return e;
        }
        scan_bwd_kernel<NL><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, bwd_smem<NL>(), st>>>(a);
        hc_status e = launched("scan_bwd_kernel", st);
        if (e) return e;
        const long long bc = (long long)a.B * a.L * a.G * 2 * a.N;
        if (a.gbc && bc > 0) {
            const long long blocks = (bc + 255) / 256, most = 16LL * device_sm_count();
            scan_bc_kernel<<<(unsigned)(blocks < most ? blocks : most), 256, 0, st>>>(a);
            if ((e = launched("scan_bc_kernel", st))) return e;
        }
        return launch_column_totals(a.part, (long long)a.B * a.segs, g->gA, a.Dm * a.N, g->gD, a.Dm, g->gdt_bias, a.Dm, st);
    }
};

struct ScanStep {
    ScanArgs a;
    float* state;
    cudaStream_t st;
    template <int NL> hc_status operator()() {
        scan_step_kernel<NL><<<cdiv((long long)a.B * a.Dm, 4 * (32 / NL)), 128, 0, st>>>(a, state);
        return launched("scan_step_kernel", st);
    }
};

bool vec4(const ScanArgs& a) {
    for (const hc_rows* r : {&a.u, &a.dt, &a.z, &a.y, &a.gy, &a.gu, &a.gdt, &a.gz})
        if (!rows_vec(r, 4)) return false;
    return a.Dg % 4 == 0;
}

}  // namespace
}  // namespace hc

using namespace hc;

extern "C" {

// Workspace: forward [segment states][segment step sums]; backward the same two,
// [gA, gD, gdt_bias sums][gB, gC sums of each channel tile, where a group has
// several].
hc_status hc_selective_scan_workspace_size(const hc_selective_scan_desc* d, int pass, size_t* bytes) {
    if (!scan_desc_ok(d) || pass < 0 || pass > 1 || !bytes) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = carry_bytes(d, fwd_segs(d).n);
    if (pass == 1) {
        const int tiles = scan_ctiles(d);
        size_t b = carry_bytes(d, bwd_segs(d).n) + part_bytes(d);
        if (tiles > 1) b += sizeof(float) * tiles * (size_t)d->B * d->L * d->groups * 2 * d->d_state;
        if (b > *bytes) *bytes = b;
    }
    return HC_OK;
}

hc_status hc_selective_scan_saved_size(const hc_selective_scan_desc* d, size_t* bytes) {
    if (!scan_desc_ok(d) || !bytes) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = sizeof(float) * (size_t)d->B * cdiv(d->L, SC_T) * d->D * 4 * scan_lanes(d->d_state);
    return HC_OK;
}

hc_status hc_selective_scan_fwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const hc_rows* y, float* hT, void* saved, void* ws, size_t ws_bytes,
                                void* stream) {
    size_t need = 0;
    hc_status e = hc_selective_scan_workspace_size(d, 0, &need);
    if (e) return e;
    if (!scan_in_ok(d, in, d->L) || !rows_out_ok(y, d->dtype, d->B, d->L, d->D) || !f32_opt_ok(h0) ||
        !f32_opt_ok(hT) || (h0 && h0 == hT) || !f32_opt_ok(saved) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z})
        if (rows_same(y, r)) return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    ScanFwd f{scan_args(d, in), (cudaStream_t)stream};
    f.a.y = *y;
    f.a.h0 = h0;
    f.a.hT = hT;
    f.a.lens = lens;
    f.a.saved = (float*)saved;
    f.a.vec = vec4(f.a);
    set_segs(f.a, d, fwd_segs(d), ws);
    return scan_dispatch(d->d_state, f);
}

hc_status hc_selective_scan_bwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const void* saved, const hc_rows* gy, const float* ghT,
                                const hc_scan_grad* g, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    hc_status e = hc_selective_scan_workspace_size(d, 1, &need);
    if (e) return e;
    if (!scan_in_ok(d, in, d->L) || !g || !rows_in_ok(gy, d->dtype, d->L) || (d->L > 0 && !f32_ok(saved)) ||
        !f32_opt_ok(h0) || !f32_opt_ok(ghT) || !f32_ok(g->gA) || !f32_opt_ok(g->gD) || !f32_opt_ok(g->gdt_bias) ||
        !f32_opt_ok(g->gh0) || (ghT && ghT == g->gh0) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    const long long shared = (long long)d->groups * d->d_state;
    if (!rows_out_ok(&g->gu, d->dtype, d->B, d->L, d->D) || !rows_out_ok(&g->gdt, d->dtype, d->B, d->L, d->D) ||
        !rows_out_ok(&g->gB, d->dtype, d->B, d->L, shared) || !rows_out_ok(&g->gC, d->dtype, d->B, d->L, shared) ||
        (d->L > 0 && (in->z.p != nullptr) != (g->gz.p != nullptr)) ||
        (g->gz.p && !rows_out_ok(&g->gz, d->dtype, d->B, d->L, d->D)))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* o : {&g->gu, &g->gdt, &g->gB, &g->gC, &g->gz})
        for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z, gy})
            if (rows_same(o, r)) return HC_ERR_INVALID_ARG;
    if (!f32_ok(ws) || ws_bytes < need) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    ScanBwd f{scan_args(d, in), g, (cudaStream_t)stream};
    f.a.gy = *gy;
    f.a.gu = g->gu;
    f.a.gdt = g->gdt;
    f.a.gB = g->gB;
    f.a.gC = g->gC;
    f.a.gz = g->gz;
    f.a.ghT = ghT;
    f.a.gh0 = g->gh0;
    f.a.lens = lens;
    f.a.saved = (float*)saved;
    set_segs(f.a, d, bwd_segs(d), ws);
    const size_t carried = carry_bytes(d, f.a.segs);
    f.a.part = (float*)((char*)ws + carried);
    f.a.gbc = f.a.ctiles > 1 ? (float*)((char*)ws + carried + part_bytes(d)) : nullptr;
    f.a.vec = vec4(f.a);
    return scan_dispatch(d->d_state, f);
}

hc_status hc_selective_scan_step(const hc_selective_scan_desc* d, const hc_scan_in* in, float* state, const hc_rows* y,
                                 void* stream) {
    if (!scan_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!scan_in_ok(d, in, 1) || !rows_out_ok(y, d->dtype, d->B, 1, d->D) || !f32_ok(state)) return HC_ERR_INVALID_ARG;
    for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z})
        if (rows_same(y, r)) return HC_ERR_INVALID_ARG;
    traced_begin((cudaStream_t)stream);
    ScanStep f{scan_args(d, in), state, (cudaStream_t)stream};
    f.a.y = *y;
    return scan_dispatch(d->d_state, f);
}

}  // extern "C"
