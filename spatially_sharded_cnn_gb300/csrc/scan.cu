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

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr int SC_T = 16;  // rows a tile; the backward pass keeps a tile's states in registers

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
// Channels c .. c + 3 of a row, those at or past n as zeros; vec: aligned to
// four elements, and then n is a multiple of 4.
__device__ __forceinline__ void ld4(const void* p, long long i, int dt, int c, int n, bool vec, float (&f)[4]) {
    if (vec && c < n) {
        if (dt == HC_DTYPE_F32)
            load_pack<float, 4>(static_cast<const float*>(p) + i + c, f);
        else if (dt == HC_DTYPE_BF16)
            load_pack<__nv_bfloat16, 4>(static_cast<const __nv_bfloat16*>(p) + i + c, f);
        else
            load_pack<__half, 4>(static_cast<const __half*>(p) + i + c, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) f[k] = c + k < n ? ld1(p, i + c + k, dt) : 0.0f;
}
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

__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// log(1 + exp(x)); above 20 it is x to fp32 precision.
__device__ __forceinline__ float softplus_f(float x) { return x > 20.0f ? x : log1pf(expf(x)); }

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

template <int NL> struct FwdTile {
    static constexpr int NP = 4 * NL, CG = 32 / NL;
    static constexpr int W = NL == 1 ? 2 : 4;  // warps
    static constexpr int WC = 4 * CG;          // channels a warp
    static constexpr int CT = W * WC;          // channels a block
    static constexpr int THREADS = W * 32;
    static constexpr size_t SMEM = sizeof(float) * SC_T * (3 * CT + 2 * NP);
};

// One block: CT channels of one group of one segment.
template <int NL>
__global__ void __launch_bounds__(FwdTile<NL>::THREADS) scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = FwdTile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // [T][CT] step sizes
    float* du = dl + SC_T * S::CT;              // [T][CT] step * u
    float* ys = du + SC_T * S::CT;              // [T][CT] C . h
    float* Bs = ys + SC_T * S::CT;              // [T][NP]
    float* Cs = Bs + SC_T * S::NP;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ct = blockIdx.x % (a.G * a.ctiles), bs = blockIdx.x / (a.G * a.ctiles);
    const int b = bs / a.segs, seg = bs % a.segs;
    const int g = ct / a.ctiles, c0 = (ct % a.ctiles) * S::CT;  // first channel inside the group
    const int cn = min(S::CT, a.Dg - c0);                       // channels of this block
    const int d0 = g * a.Dg + c0;
    const int n = lane % NL, tc = warp * S::WC + (lane / NL) * 4;  // this thread's states and channels
    const int len = scan_len(a, b);
    float A2[4][4], h[4][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] = h[i][j] = 0.0f;
        if (tc + i < cn) {
            ld_states(a.A + (long long)(d0 + tc + i) * a.N, 4 * n, a.N, A2[i]);
            if (a.segs > 1)
                load_pack<float, 4>(a.carry + ((long long)bs * a.Dm + d0 + tc + i) * S::NP + 4 * n, h[i]);
            else if (a.h0)
                ld_states(a.h0 + ((long long)b * a.Dm + d0 + tc + i) * a.N, 4 * n, a.N, h[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] *= kLog2e;
    }
    const int tile1 = min((seg + 1) * a.seg_tiles, a.tiles);
    for (int tile = seg * a.seg_tiles; tile < tile1; tile++) {
        const int t0 = tile * SC_T, rows = min(SC_T, a.L - t0);
        if (t0 < len) {
            for (int q = tid; q < SC_T * (S::CT / 4); q += S::THREADS) {
                const int t = q / (S::CT / 4), c = (q % (S::CT / 4)) * 4;
                float x[4] = {0, 0, 0, 0}, s[4] = {0, 0, 0, 0};
                if (t0 + t < len && c < cn) {
                    ld4(a.u.p, b * a.u.batch + (t0 + t) * a.u.row + d0, a.dtype, c, cn, a.vec, x);
                    ld4(a.dt.p, b * a.dt.batch + (t0 + t) * a.dt.row + d0, a.dtype, c, cn, a.vec, s);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        if (a.bias && c + k < cn) s[k] += a.bias[d0 + c + k];
                        if (a.softplus) s[k] = softplus_f(s[k]);
                        x[k] *= s[k];
                    }
                }
                store_pack<float, 4>(dl + t * S::CT + c, s);
                store_pack<float, 4>(du + t * S::CT + c, x);
            }
            for (int q = tid; q < SC_T * S::NP; q += S::THREADS) {
                const int t = q / S::NP, k = q % S::NP;
                const bool on = t0 + t < len && k < a.N;
                Bs[q] = on ? ld1(a.Bm.p, b * a.Bm.batch + (t0 + t) * a.Bm.row + g * a.N + k, a.dtype) : 0.0f;
                Cs[q] = on ? ld1(a.Cm.p, b * a.Cm.batch + (t0 + t) * a.Cm.row + g * a.N + k, a.dtype) : 0.0f;
            }
            if (a.saved) {
#pragma unroll
                for (int i = 0; i < 4; i++)
                    if (tc + i < cn)
                        store_pack<float, 4>(a.saved + (((long long)b * a.tiles + tile) * a.Dm + d0 + tc + i) * S::NP +
                                                 4 * n,
                                             h[i]);
            }
            __syncthreads();
#pragma unroll 2
            for (int t = 0; t < SC_T; t++) {
                float s[4], x[4], B[4], C[4], y[4];
                load_pack<float, 4>(dl + t * S::CT + tc, s);
                load_pack<float, 4>(du + t * S::CT + tc, x);
                load_pack<float, 4>(Bs + t * S::NP + 4 * n, B);
                load_pack<float, 4>(Cs + t * S::NP + 4 * n, C);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    y[i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        h[i][j] = fmaf(ex2f(s[i] * A2[i][j]), h[i][j], x[i] * B[j]);
                        y[i] = fmaf(C[j], h[i][j], y[i]);
                    }
                }
                const int first = lanes_sum<4, NL>(y, n);
                constexpr int KEEP = NL >= 4 ? 1 : 4 / NL;
                if (NL <= 4 || n < 4) {
#pragma unroll
                    for (int i = 0; i < KEEP; i++) ys[t * S::CT + tc + first + i] = y[i];
                }
            }
            __syncthreads();
        }
        for (int q = tid; q < rows * (S::CT / 4); q += S::THREADS) {
            const int t = q / (S::CT / 4), c = (q % (S::CT / 4)) * 4;
            if (c >= cn) continue;
            float o[4] = {0, 0, 0, 0};
            if (t0 + t < len) {
                float x[4], zz[4];
                load_pack<float, 4>(ys + t * S::CT + c, o);
                if (a.D) {
                    ld4(a.u.p, b * a.u.batch + (t0 + t) * a.u.row + d0, a.dtype, c, cn, a.vec, x);
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (c + k < cn) o[k] = fmaf(a.D[d0 + c + k], x[k], o[k]);
                }
                if (a.z.p) {
                    ld4(a.z.p, b * a.z.batch + (t0 + t) * a.z.row + d0, a.dtype, c, cn, a.vec, zz);
#pragma unroll
                    for (int k = 0; k < 4; k++) o[k] *= silu_f(zz[k]);
                }
            }
            st4(a.y.p, b * a.y.batch + (t0 + t) * a.y.row + d0, a.dtype, c, cn, a.vec, o);
        }
        __syncthreads();
    }
    if (a.hT && seg == a.segs - 1) {
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (tc + i < cn) st_states(a.hT + ((long long)b * a.Dm + d0 + tc + i) * a.N, 4 * n, a.N, h[i]);
    }
}

// A segment's state from a zero state.  REV false: the state itself, over
// x = step * u and B, rows upwards.  REV true: the state's gradient, over
// q = gy * silu(z) and C, rows downwards: G_{t-1} = exp(step_t A) (G_t + q_t C_t).
template <int NL, bool REV>
__global__ void __launch_bounds__(FwdTile<NL>::THREADS) scan_carry_kernel(const __grid_constant__ ScanArgs a) {
    using S = FwdTile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // [T][CT] step sizes
    float* xs = dl + SC_T * S::CT;              // [T][CT] step * u, or q
    float* Bs = xs + SC_T * S::CT;              // [T][NP]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ct = blockIdx.x % (a.G * a.ctiles), bs = blockIdx.x / (a.G * a.ctiles);
    const int b = bs / a.segs, seg = bs % a.segs;
    const int g = ct / a.ctiles, c0 = (ct % a.ctiles) * S::CT;
    const int cn = min(S::CT, a.Dg - c0);
    const int d0 = g * a.Dg + c0;
    const int n = lane % NL, tc = warp * S::WC + (lane / NL) * 4;
    const int len = scan_len(a, b);
    float A2[4][4], h[4][4], sum[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        sum[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] = h[i][j] = 0.0f;
        if (tc + i < cn) ld_states(a.A + (long long)(d0 + tc + i) * a.N, 4 * n, a.N, A2[i]);
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] *= kLog2e;
    }
    const int tile0 = seg * a.seg_tiles, tile1 = min(tile0 + a.seg_tiles, a.tiles);
    for (int k = tile0; k < tile1; k++) {
        const int t0 = (REV ? tile1 - 1 - (k - tile0) : k) * SC_T;
        if (t0 >= len) continue;
        for (int q = tid; q < SC_T * (S::CT / 4); q += S::THREADS) {
            const int t = q / (S::CT / 4), c = (q % (S::CT / 4)) * 4;
            float x[4] = {0, 0, 0, 0}, s[4] = {0, 0, 0, 0};
            if (t0 + t < len && c < cn) {
                const hc_rows& in = REV ? a.gy : a.u;
                ld4(in.p, b * in.batch + (t0 + t) * in.row + d0, a.dtype, c, cn, a.vec, x);
                ld4(a.dt.p, b * a.dt.batch + (t0 + t) * a.dt.row + d0, a.dtype, c, cn, a.vec, s);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    if (a.bias && c + i < cn) s[i] += a.bias[d0 + c + i];
                    if (a.softplus) s[i] = softplus_f(s[i]);
                    if (!REV) x[i] *= s[i];
                }
                if (REV && a.z.p) {
                    float zz[4];
                    ld4(a.z.p, b * a.z.batch + (t0 + t) * a.z.row + d0, a.dtype, c, cn, a.vec, zz);
#pragma unroll
                    for (int i = 0; i < 4; i++) x[i] *= silu_f(zz[i]);
                }
            }
            store_pack<float, 4>(dl + t * S::CT + c, s);
            store_pack<float, 4>(xs + t * S::CT + c, x);
        }
        for (int q = tid; q < SC_T * S::NP; q += S::THREADS) {
            const int t = q / S::NP, j = q % S::NP;
            const hc_rows& in = REV ? a.Cm : a.Bm;
            Bs[q] = t0 + t < len && j < a.N ? ld1(in.p, b * in.batch + (t0 + t) * in.row + g * a.N + j, a.dtype) : 0.0f;
        }
        __syncthreads();
#pragma unroll 4
        for (int v = 0; v < SC_T; v++) {
            const int t = REV ? SC_T - 1 - v : v;
            float s[4], x[4], B[4];
            load_pack<float, 4>(dl + t * S::CT + tc, s);
            load_pack<float, 4>(xs + t * S::CT + tc, x);
            load_pack<float, 4>(Bs + t * S::NP + 4 * n, B);
#pragma unroll
            for (int i = 0; i < 4; i++) {
                sum[i] += s[i];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float e = ex2f(s[i] * A2[i][j]);
                    h[i][j] = REV ? e * fmaf(x[i], B[j], h[i][j]) : fmaf(e, h[i][j], x[i] * B[j]);
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if (tc + i >= cn) continue;
        const long long d = (long long)bs * a.Dm + d0 + tc + i;
        store_pack<float, 4>(a.carry + d * S::NP + 4 * n, h[i]);
        if (n == 0) a.dsum[d] = sum[i];
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

template <int NL> struct BwdTile {
    static constexpr int NP = 4 * NL, CG = 32 / NL;
    static constexpr int W = 4;
    static constexpr int WC = 2 * CG;  // channels a warp, two a thread
    static constexpr int CT = W * WC;
    static constexpr int THREADS = W * 32;
    // tile rows the elementwise parts cover at once
    static constexpr int RROWS = THREADS / (CT / 4) < SC_T ? THREADS / (CT / 4) : SC_T;
    // step, u, q, C . h, G . B, E . A; B, C; the warps' gB and gC
    static constexpr size_t SMEM = sizeof(float) * SC_T * (6 * CT + 2 * NP + 2 * NP * W);
};

// One block: CT channels of one group of one segment, its tiles from the last
// to the first.  A tile's states are recomputed from its saved first state and
// kept in registers, then the state's gradient runs back through them.
template <int NL>
__global__ void __launch_bounds__(BwdTile<NL>::THREADS) scan_bwd_kernel(const __grid_constant__ ScanArgs a) {
    using S = BwdTile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);
    float* us = dl + SC_T * S::CT;
    float* qs = us + SC_T * S::CT;
    float* ys = qs + SC_T * S::CT;
    float* GBs = ys + SC_T * S::CT;
    float* EAs = GBs + SC_T * S::CT;
    float* Bs = EAs + SC_T * S::CT;
    float* Cs = Bs + SC_T * S::NP;
    float* red = Cs + SC_T * S::NP;  // [W][T][2][NP]
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ct = blockIdx.x % (a.G * a.ctiles), bs = blockIdx.x / (a.G * a.ctiles);
    const int b = bs / a.segs, seg = bs % a.segs;
    const int g = ct / a.ctiles, c0 = (ct % a.ctiles) * S::CT;
    const int cn = min(S::CT, a.Dg - c0);
    const int d0 = g * a.Dg + c0;
    const int n = lane % NL, cg = lane / NL, tc = warp * S::WC + cg * 2;
    const int len = scan_len(a, b);
    float A2[2][4], G[2][4], gA[2][4];
#pragma unroll
    for (int i = 0; i < 2; i++) {
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] = G[i][j] = gA[i][j] = 0.0f;
        if (tc + i < cn) {
            ld_states(a.A + (long long)(d0 + tc + i) * a.N, 4 * n, a.N, A2[i]);
            if (a.segs > 1)
                load_pack<float, 4>(a.carry + ((long long)bs * a.Dm + d0 + tc + i) * S::NP + 4 * n, G[i]);
            else if (a.ghT)
                ld_states(a.ghT + ((long long)b * a.Dm + d0 + tc + i) * a.N, 4 * n, a.N, G[i]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) A2[i][j] *= kLog2e;
    }
    // the elementwise parts: four fixed channels a thread
    const int ec = (tid % (S::CT / 4)) * 4, er = tid / (S::CT / 4);
    float Dv[4], bv[4], sD[4], sb[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        Dv[k] = a.D && ec + k < cn ? a.D[d0 + ec + k] : 0.0f;
        bv[k] = a.bias && ec + k < cn ? a.bias[d0 + ec + k] : 0.0f;
        sD[k] = sb[k] = 0.0f;
    }
    for (int tile = min((seg + 1) * a.seg_tiles, a.tiles) - 1; tile >= seg * a.seg_tiles; tile--) {
        const int t0 = tile * SC_T, rows = min(SC_T, a.L - t0);
        const bool live = t0 < len;
        if (live) {
            for (int t = er; t < SC_T; t += S::RROWS) {  // none for er >= RROWS = SC_T
                float x[4] = {0, 0, 0, 0}, s[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
                if (t0 + t < len && ec < cn) {
                    ld4(a.u.p, b * a.u.batch + (t0 + t) * a.u.row + d0, a.dtype, ec, cn, a.vec, x);
                    ld4(a.dt.p, b * a.dt.batch + (t0 + t) * a.dt.row + d0, a.dtype, ec, cn, a.vec, s);
                    ld4(a.gy.p, b * a.gy.batch + (t0 + t) * a.gy.row + d0, a.dtype, ec, cn, a.vec, q);
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        s[k] += bv[k];
                        if (a.softplus) s[k] = softplus_f(s[k]);
                    }
                    if (a.z.p) {
                        float zz[4];
                        ld4(a.z.p, b * a.z.batch + (t0 + t) * a.z.row + d0, a.dtype, ec, cn, a.vec, zz);
#pragma unroll
                        for (int k = 0; k < 4; k++) q[k] *= silu_f(zz[k]);
                    }
                }
                store_pack<float, 4>(dl + t * S::CT + ec, s);
                store_pack<float, 4>(us + t * S::CT + ec, x);
                store_pack<float, 4>(qs + t * S::CT + ec, q);
            }
            for (int q = tid; q < SC_T * S::NP; q += S::THREADS) {
                const int t = q / S::NP, k = q % S::NP;
                const bool on = t0 + t < len && k < a.N;
                Bs[q] = on ? ld1(a.Bm.p, b * a.Bm.batch + (t0 + t) * a.Bm.row + g * a.N + k, a.dtype) : 0.0f;
                Cs[q] = on ? ld1(a.Cm.p, b * a.Cm.batch + (t0 + t) * a.Cm.row + g * a.N + k, a.dtype) : 0.0f;
            }
            // H[t] is the state before the tile's row t
            float H[SC_T + 1][2][4];
#pragma unroll
            for (int i = 0; i < 2; i++) {
#pragma unroll
                for (int j = 0; j < 4; j++) H[0][i][j] = 0.0f;
                if (tc + i < cn)
                    load_pack<float, 4>(
                        a.saved + (((long long)b * a.tiles + tile) * a.Dm + d0 + tc + i) * S::NP + 4 * n, H[0][i]);
            }
            __syncthreads();
#pragma unroll
            for (int t = 0; t < SC_T; t++) {
                float B[4], C[4], y[2];
                const float2 s = *reinterpret_cast<const float2*>(dl + t * S::CT + tc);
                const float2 x = *reinterpret_cast<const float2*>(us + t * S::CT + tc);
                const float sv[2] = {s.x, s.y}, xv[2] = {s.x * x.x, s.y * x.y};
                load_pack<float, 4>(Bs + t * S::NP + 4 * n, B);
                load_pack<float, 4>(Cs + t * S::NP + 4 * n, C);
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    y[i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        H[t + 1][i][j] = fmaf(ex2f(sv[i] * A2[i][j]), H[t][i][j], xv[i] * B[j]);
                        y[i] = fmaf(C[j], H[t + 1][i][j], y[i]);
                    }
                }
                if (a.z.p) {
                    const int first = lanes_sum<2, NL>(y, n);
                    if (NL <= 2 || n < 2) {
                        ys[t * S::CT + tc + first] = y[0];
                        if (NL == 1) ys[t * S::CT + tc + 1] = y[1];
                    }
                }
            }
            // gA summed tile by tile: a running sum over all rows would lose an ulp a row
            float ga_tile[2][4] = {};
#pragma unroll
            for (int t = SC_T - 1; t >= 0; t--) {
                float B[4], C[4], bc[8], gb[2] = {0, 0}, ea[2] = {0, 0};
                const float2 s = *reinterpret_cast<const float2*>(dl + t * S::CT + tc);
                const float2 x = *reinterpret_cast<const float2*>(us + t * S::CT + tc);
                const float2 q = *reinterpret_cast<const float2*>(qs + t * S::CT + tc);
                const float sv[2] = {s.x, s.y}, xv[2] = {s.x * x.x, s.y * x.y}, qv[2] = {q.x, q.y};
                load_pack<float, 4>(Bs + t * S::NP + 4 * n, B);
                load_pack<float, 4>(Cs + t * S::NP + 4 * n, C);
#pragma unroll
                for (int j = 0; j < 8; j++) bc[j] = 0.0f;
#pragma unroll
                for (int i = 0; i < 2; i++) {
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const float gg = fmaf(qv[i], C[j], G[i][j]);
                        bc[j] = fmaf(gg, xv[i], bc[j]);
                        bc[4 + j] = fmaf(qv[i], H[t + 1][i][j], bc[4 + j]);
                        gb[i] = fmaf(gg, B[j], gb[i]);
                        const float ga = gg * ex2f(sv[i] * A2[i][j]);
                        const float E = ga * H[t][i][j];
                        ea[i] = fmaf(E, A2[i][j], ea[i]);
                        ga_tile[i][j] = fmaf(E, sv[i], ga_tile[i][j]);
                        G[i][j] = ga;
                    }
                }
                const int first = lanes_sum<2, NL>(gb, n);
                lanes_sum<2, NL>(ea, n);
                if (NL <= 2 || n < 2) {
                    GBs[t * S::CT + tc + first] = gb[0];
                    EAs[t * S::CT + tc + first] = ea[0] * kLn2;
                    if (NL == 1) {
                        GBs[t * S::CT + tc + 1] = gb[1];
                        EAs[t * S::CT + tc + 1] = ea[1] * kLn2;
                    }
                }
                // over the channels: lanes n, n + NL, ... of the warp
                int at = 0, left = 8;
#pragma unroll
                for (int o = NL; o < 32; o <<= 1) {
                    if (left > 1) {
                        const int half = left / 2;
                        const bool up = (lane & o) != 0;
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            if (i < half) {
                                const float send = up ? bc[i] : bc[i + half], keep = up ? bc[i + half] : bc[i];
                                bc[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                            }
                        }
                        at += up ? half : 0;
                        left = half;
                    } else {
                        bc[0] += __shfl_xor_sync(0xffffffffu, bc[0], o);
                    }
                }
                constexpr int KEEP = S::CG >= 8 ? 1 : 8 / S::CG;
                if (S::CG <= 8 || cg < 8) {
                    float* r = red + (warp * SC_T + t) * 2 * S::NP + (at / 4) * S::NP + 4 * n + at % 4;
#pragma unroll
                    for (int i = 0; i < KEEP; i++) r[i] = bc[i];
                }
            }
#pragma unroll
            for (int i = 0; i < 2; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) gA[i][j] += ga_tile[i][j];
            __syncthreads();
        }
        for (int t = er; t < rows; t += S::RROWS) {
            if (ec >= cn) continue;
            float gu[4] = {0, 0, 0, 0}, gd[4] = {0, 0, 0, 0}, gz[4] = {0, 0, 0, 0};
            if (t0 + t < len) {
                float GB[4], EA[4], x[4], s[4], q[4];
                load_pack<float, 4>(GBs + t * S::CT + ec, GB);
                load_pack<float, 4>(EAs + t * S::CT + ec, EA);
                load_pack<float, 4>(us + t * S::CT + ec, x);
                load_pack<float, 4>(dl + t * S::CT + ec, s);
                load_pack<float, 4>(qs + t * S::CT + ec, q);
                float raw[4];
                ld4(a.dt.p, b * a.dt.batch + (t0 + t) * a.dt.row + d0, a.dtype, ec, cn, a.vec, raw);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    gu[k] = fmaf(GB[k], s[k], Dv[k] * q[k]);
                    gd[k] = fmaf(GB[k], x[k], EA[k]);
                    if (a.softplus) gd[k] *= sigmoid_f(raw[k] + bv[k]);
                    sb[k] += gd[k];
                    sD[k] = fmaf(q[k], x[k], sD[k]);
                }
                if (a.gz.p) {
                    float zz[4], w[4], y[4];
                    ld4(a.z.p, b * a.z.batch + (t0 + t) * a.z.row + d0, a.dtype, ec, cn, a.vec, zz);
                    ld4(a.gy.p, b * a.gy.batch + (t0 + t) * a.gy.row + d0, a.dtype, ec, cn, a.vec, w);
                    load_pack<float, 4>(ys + t * S::CT + ec, y);
#pragma unroll
                    for (int k = 0; k < 4; k++) gz[k] = w[k] * fmaf(Dv[k], x[k], y[k]) * silu_d(zz[k]);
                }
            }
            st4(a.gu.p, b * a.gu.batch + (t0 + t) * a.gu.row + d0, a.dtype, ec, cn, a.vec, gu);
            st4(a.gdt.p, b * a.gdt.batch + (t0 + t) * a.gdt.row + d0, a.dtype, ec, cn, a.vec, gd);
            if (a.gz.p) st4(a.gz.p, b * a.gz.batch + (t0 + t) * a.gz.row + d0, a.dtype, ec, cn, a.vec, gz);
        }
        for (int q = tid; q < rows * 2 * S::NP; q += S::THREADS) {
            const int t = q / (2 * S::NP), w = (q / S::NP) & 1, k = q % S::NP;
            if (k >= a.N) continue;
            float v = 0.0f;
            if (t0 + t < len) {
#pragma unroll
                for (int m = 0; m < S::W; m++) v += red[(m * SC_T + t) * 2 * S::NP + w * S::NP + k];
            }
            if (a.gbc) {
                a.gbc[((((long long)(ct % a.ctiles) * a.B + b) * a.L + t0 + t) * a.G + g) * 2 * a.N + w * a.N + k] = v;
            } else {
                const hc_rows& o = w ? a.gC : a.gB;
                st1(o.p, b * o.batch + (t0 + t) * o.row + g * a.N + k, a.dtype, v);
            }
        }
        __syncthreads();
    }
    float* pb = a.part + (long long)bs * (a.N + 2) * a.Dm;
#pragma unroll
    for (int i = 0; i < 2; i++) {
        if (tc + i < cn) {
            const long long d = d0 + tc + i;
#pragma unroll
            for (int j = 0; j < 4; j++)
                if (4 * n + j < a.N) pb[d * a.N + 4 * n + j] = gA[i][j];
            if (a.gh0 && seg == 0) st_states(a.gh0 + ((long long)b * a.Dm + d) * a.N, 4 * n, a.N, G[i]);
        }
    }
    // gD and gdt_bias over the epilogue's row lanes, in order
    if (er < S::RROWS) {
        store_pack<float, 4>(dl + er * S::CT + ec, sD);
        store_pack<float, 4>(us + er * S::CT + ec, sb);
    }
    __syncthreads();
    for (int c = tid; c < cn; c += S::THREADS) {
        float x = 0.0f, y = 0.0f;
        for (int r = 0; r < S::RROWS; r++) {
            x += dl[r * S::CT + c];
            y += us[r * S::CT + c];
        }
        pb[(long long)a.N * a.Dm + d0 + c] = x;
        pb[(long long)(a.N + 1) * a.Dm + d0 + c] = y;
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

// Channel tiles a group in a kernel whose warps take `per_lane` channels a lane group.
int scan_ctiles(const hc_selective_scan_desc* d, int warps, int per_lane) {
    return (int)cdiv(d->D / d->groups, warps * per_lane * 32 / scan_lanes(d->d_state));
}
int fwd_ctiles(const hc_selective_scan_desc* d) { return scan_ctiles(d, scan_lanes(d->d_state) == 1 ? 2 : 4, 4); }
int bwd_ctiles(const hc_selective_scan_desc* d) { return scan_ctiles(d, 4, 2); }

// Segments: none where (sequence, channel tile) blocks give every SM `want` of
// them, else as many as make up for it, of two tiles at least.
struct Segs {
    int n, tiles;
};
Segs scan_segs(const hc_selective_scan_desc* d, int ctiles, int want) {
    const int tiles = (int)cdiv(d->L, SC_T);
    const long long blocks = (long long)d->B * d->groups * ctiles, full = (long long)want * device_sm_count();
    if (blocks * 2 > full || tiles < 4) return {1, tiles > 0 ? tiles : 1};
    long long n = full / blocks;
    if (n > tiles / 2) n = tiles / 2;
    const int per = (int)cdiv(tiles, n);
    return {(int)cdiv(tiles, per), per};
}
Segs fwd_segs(const hc_selective_scan_desc* d) { return scan_segs(d, fwd_ctiles(d), 6); }
Segs bwd_segs(const hc_selective_scan_desc* d) { return scan_segs(d, bwd_ctiles(d), 2); }

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
    using S = FwdTile<NL>;
    static std::atomic<unsigned long long> attr{0};
    once_per_device(attr, [] {
        return cudaFuncSetAttribute(scan_carry_kernel<NL, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)S::SMEM) == cudaSuccess;
    });
    a.ctiles = (int)cdiv(a.Dg, S::CT);
    scan_carry_kernel<NL, REV><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, S::SMEM, st>>>(a);
    hc_status e = launched("scan_carry_kernel", st);
    if (e) return e;
    scan_join_kernel<REV><<<dim3(cdiv((long long)a.Dm * S::NP, SJ_STATES), a.B), 1024, 0, st>>>(a, S::NP);
    return launched("scan_join_kernel", st);
}

struct ScanFwd {
    ScanArgs a;
    cudaStream_t st;
    template <int NL> hc_status operator()() {
        using S = FwdTile<NL>;
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_fwd_kernel<NL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)S::SMEM) == cudaSuccess;
        });
        if (a.segs > 1) {
            const hc_status e = launch_scan_carry<NL, false>(a, st);
            if (e) return e;
        }
        a.ctiles = (int)cdiv(a.Dg, S::CT);
        scan_fwd_kernel<NL><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, S::SMEM, st>>>(a);
        return launched("scan_fwd_kernel", st);
    }
};

struct ScanBwd {
    ScanArgs a;
    const hc_scan_grad* g;
    cudaStream_t st;
    template <int NL> hc_status operator()() {
        using S = BwdTile<NL>;
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_bwd_kernel<NL>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)S::SMEM) == cudaSuccess;
        });
        if (a.segs > 1) {
            const hc_status e = launch_scan_carry<NL, true>(a, st);
            if (e) return e;
        }
        scan_bwd_kernel<NL><<<(unsigned)a.B * a.segs * a.G * a.ctiles, S::THREADS, S::SMEM, st>>>(a);
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
        const int tiles = bwd_ctiles(d);
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
    f.a.ctiles = bwd_ctiles(d);
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
