// scan.cuh -- what the selective-scan kernels share (scan_fwd.cu, scan_carry.cu,
// scan_bwd.cu, scan.cu).
#pragma once

#include "rows.cuh"

namespace hc {

constexpr int SC_T = 8;  // rows a tile; the forward pass saves the state before each tile for the backward pass

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
    float* dsum;          // [B][segs][D]: its sum of step sizes * log2 e
};

// States n0 .. n0 + 3 of a [..][N] fp32 row (past N: zeros / not written): 16 bytes
// at once where the row allows it -- a row of partial sums, (N + 2) * D floats
// after the one before it, need not start on 16 bytes even if N is a multiple of 4.
__device__ __forceinline__ bool states_vec(const float* p, int N) {
    return N % 4 == 0 && ((uintptr_t)p & 15u) == 0;
}
__device__ __forceinline__ void ld_states(const float* p, int n0, int N, float (&f)[4]) {
    if (states_vec(p, N) && n0 < N) {
        load_pack<float, 4>(p + n0, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++) f[k] = n0 + k < N ? p[n0 + k] : 0.0f;
}
__device__ __forceinline__ void st_states(float* p, int n0, int N, const float (&f)[4]) {
    if (states_vec(p, N) && n0 < N) {
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

// 2^(s * A).  The special function unit's 2^x is low on average, the same way in
// every row, which a state with a memory of hundreds of rows adds up: gA of 1024 rows
// was 1.4e-6 off.  The multiply-add that forms the argument adds a mean back before it
// rounds.  Mean error over 2^20 arguments from a third of x to x, without it and with
// it, in 1e-8: x = -0.3 -1.9, +0.1; -0.1 -1.8, -0.2; -0.03 -2.6, -1.0; -0.01 -2.1, -0.5;
// slower states, whose result comes to a few spacings (6e-8) below 1: -1e-3 -0.5, +1.1;
// -1e-4 -0.7, +0.9; -1e-5 -1.0, +0.6; -1e-6 -1.2, +0.4; -3e-7 -0.7, +1.8 (rms 3 to 4 for
// all; correctly rounded results 1.7).  An argument of 0 gives 1, and one below -1 takes
// no part of it (-5.0).
constexpr float kEx2Mean = 2.3e-8f;  // 1.6e-8 / ln 2
__device__ __forceinline__ f32x2 decay2(f32x2 s, f32x2 A) {
    float a, b;
    unpk2(fma2(s, A, pk2(kEx2Mean, kEx2Mean)), a, b);
    return pk2(ex2f(a), ex2f(b));
}

template <int BYTES> __device__ __forceinline__ void cp_async(unsigned dst, const void* src, bool on) {
    // BYTES are written: those of src, or zeros
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(on ? BYTES : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// The layout the kernels share.  A thread holds states 4n .. 4n + 3 of P channel
// pairs; a block's CT channels times a tile's rows are also walked elementwise,
// every thread at four fixed channels.
template <int NL_, int P_> struct Tile {
    static constexpr int NL = NL_, P = P_, NP = 4 * NL, CG = 32 / NL;
    static constexpr int WC = 2 * P * CG;                     // channels a warp
    static constexpr int W = WC >= 128 ? 1 : WC >= 64 ? 2 : 4;  // warps
    static constexpr int CT = W * WC;                         // channels a block
    static constexpr int THREADS = W * 32;
    static constexpr int ROWS = THREADS / (CT / 4) < SC_T ? THREADS / (CT / 4) : SC_T;  // rows walked at once
    static constexpr int STEPS = SC_T / ROWS;
    static constexpr int PLANE = SC_T * CT;  // values of a tile
    static constexpr int BC = 2 * SC_T * NP / THREADS;  // values of B and C a thread fetches
};

template <int NL> using FwdTile = Tile<NL, 2>;
template <int NL> using BwdTile = Tile<NL, 2>;

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
template <typename S> struct Walk {
    int ec, er;  // four channels from ec, rows er, er + ROWS, ... (STEPS of them)
    bool on;     // false for threads past the tile's rows
    __device__ __forceinline__ Walk() {
        int tid = threadIdx.x;
        asm volatile("" : "+r"(tid));
        ec = tid % (S::CT / 4) * 4;
        er = tid / (S::CT / 4);
        on = S::THREADS <= S::ROWS * (S::CT / 4) || er < S::ROWS;
    }
};

// Starts the copy of a tile's rows of one tensor to plane k of the raw buffer.
template <typename S, int DT>
__device__ __forceinline__ void fetch(const ScanArgs& a, const hc_rows& r, const Where& w, const Walk<S>& at, int t0,
                                      int k, char* raw) {
    using T = typename EltOf<DT>::type;
    // the tile's corner is the same for every thread of the block
    const T* p = static_cast<const T*>(r.p) + (w.b * r.batch + t0 * r.row + w.d0) + at.ec;
    T* dst = reinterpret_cast<T*>(raw) + k * S::PLANE + at.ec;
    if (!at.on) return;
#pragma unroll
    for (int i = 0; i < S::STEPS; i++) {
        const int t = at.er + i * S::ROWS;
        const bool on = t0 + t < w.len && at.ec < w.cn;
        const T* q = p + (on ? t * r.row : 0);
        if (a.vec) {
            cp_async<4 * sizeof(T)>((unsigned)__cvta_generic_to_shared(dst + t * S::CT), on ? q : r.p, on);
            continue;
        }
        for (int c = 0; c < 4; c++) dst[t * S::CT + c] = on && at.ec + c < w.cn ? q[c] : from_f<T>(0.0f);
    }
}
// Four channels of row t of plane k.
template <typename S, int DT>
__device__ __forceinline__ void get(const char* raw, int k, int t, int ec, float (&f)[4]) {
    using T = typename EltOf<DT>::type;
    load_pack<T, 4>(reinterpret_cast<const T*>(raw) + k * S::PLANE + t * S::CT + ec, f);
}
// Four channels from c of a row's channels below n; vec: n is a multiple of 4 and the row aligned to four elements.
template <int DT>
__device__ __forceinline__ void put(typename EltOf<DT>::type* row, int c, int n, bool vec, const float (&f)[4]) {
    using T = typename EltOf<DT>::type;
    if (vec) {
        if (c < n) store_pack<T, 4>(row + c, f);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (c + k < n) row[c + k] = from_f<T>(f[k]);
}
template <int DT>
__device__ __forceinline__ typename EltOf<DT>::type* out_row(const hc_rows& r, const Where& w, int t0, int t) {
    return static_cast<typename EltOf<DT>::type*>(r.p) + (w.b * r.batch + t0 * r.row + w.d0) + t * r.row;
}
// A tile's B and C, a few values a thread, held as loaded until put_bc.
template <typename S, int DT>
__device__ __forceinline__ void fetch_bc(const ScanArgs& a, const Where& w, int t0,
                                         typename EltOf<DT>::type (&bc)[S::BC]) {
    using T = typename EltOf<DT>::type;
#pragma unroll
    for (int i = 0; i < S::BC; i++) {
        const int q = threadIdx.x + i * S::THREADS;
        const int t = q / S::NP % SC_T, n = q % S::NP;
        const hc_rows& r = q / (SC_T * S::NP) ? a.Cm : a.Bm;
        bc[i] = from_f<T>(0.0f);
        if (t0 + t < w.len && n < a.N)
            bc[i] = (static_cast<const T*>(r.p) + (w.b * r.batch + t0 * r.row + w.g * a.N))[t * r.row + n];
    }
}
// To bc2[2][T][NP], each value twice (a pair for the packed multiply-adds).
template <typename S, int DT>
__device__ __forceinline__ void put_bc(const typename EltOf<DT>::type (&bc)[S::BC], f32x2* bc2) {
#pragma unroll
    for (int i = 0; i < S::BC; i++) {
        const float v = to_f(bc[i]);
        bc2[threadIdx.x + i * S::THREADS] = pk2(v, v);
    }
}

__device__ __forceinline__ void ld_pairs(const float* p, f32x2 (&v)[1]) { v[0] = *reinterpret_cast<const f32x2*>(p); }
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
// A thread's channels' four states each as channel pairs, from rows of fp32
// states (`padded`: rows of NP with every state there, else rows of N).
template <int P>
__device__ __forceinline__ void ld_tile(const float* p, long long step, int n, int N, bool padded, int tc, int cn,
                                        f32x2 (&v)[P][4]) {
    float f[2 * P][4];
#pragma unroll
    for (int i = 0; i < 2 * P; i++) {
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
    for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) v[i][j] = pk2(f[2 * i][j], f[2 * i + 1][j]);
}
template <int P>
__device__ __forceinline__ void st_tile(float* p, long long step, int n, int N, bool padded, int tc, int cn,
                                        const f32x2 (&v)[P][4]) {
    float f[2 * P][4];
#pragma unroll
    for (int i = 0; i < P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) unpk2(v[i][j], f[2 * i][j], f[2 * i + 1][j]);
#pragma unroll
    for (int i = 0; i < 2 * P; i++) {
        if (tc + i >= cn) continue;
        if (padded)
            store_pack<float, 4>(p + i * step + 4 * n, f[i]);
        else
            st_states(p + i * step, 4 * n, N, f[i]);
    }
}
template <int P>
__device__ __forceinline__ void ld_rates(const ScanArgs& a, int d, int n, int tc, int cn, f32x2 (&A)[P][4]) {
    ld_tile(a.A + (long long)d * a.N, a.N, n, a.N, false, tc, cn, A);
}

// Sums v over a channel group's NL lanes and writes the channels' totals to row[0 .. 2P).
template <int NL, int P> __device__ __forceinline__ void put_lanes_sum(const f32x2 (&v)[P], int n, float* row) {
    float y[2 * P];
#pragma unroll
    for (int i = 0; i < P; i++) unpk2(v[i], y[2 * i], y[2 * i + 1]);
    const int first = lanes_sum<2 * P, NL>(y, n);
    constexpr int KEEP = NL >= 2 * P ? 1 : 2 * P / NL;
    if (NL <= 2 * P || n < 2 * P) {
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
template <typename S> __device__ __forceinline__ void put_params(const ScanArgs& a, const Where& w, float* bD) {
    for (int c = threadIdx.x; c < S::CT; c += S::THREADS) {
        bD[c] = a.bias && c < w.cn ? a.bias[w.d0 + c] : 0.0f;
        bD[S::CT + c] = a.D && c < w.cn ? a.D[w.d0 + c] : 0.0f;
    }
}
// The step sizes of four channels, from dt and dt_bias; and to `dl` those times
// log2 e, so that exp(step * A) is 2^(dl * A).
__device__ __forceinline__ void steps(const ScanArgs& a, bool on, float (&s)[4], const float (&bias)[4], float* dl) {
    float t[4];
#pragma unroll
    for (int k = 0; k < 4; k++) {
        s[k] += bias[k];
        if (a.softplus) s[k] = softplus_f(s[k]);
        if (!on) s[k] = 0.0f;
        t[k] = s[k] * kLog2e;
    }
    store_pack<float, 4>(dl, t);
}
__device__ __forceinline__ void add4(float (&a)[4], const float* p) {
    float b[4];
    load_pack<float, 4>(p, b);
#pragma unroll
    for (int k = 0; k < 4; k++) a[k] += b[k];
}

inline int scan_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// Calls f with the lanes and element type of a call.
template <int NL, typename F> hc_status scan_dispatch_type(int dt, F& f) {
    if (dt == HC_DTYPE_F32) return f.template run<NL, HC_DTYPE_F32>();
    if (dt == HC_DTYPE_BF16) return f.template run<NL, HC_DTYPE_BF16>();
    return f.template run<NL, HC_DTYPE_F16>();
}
template <typename F> hc_status scan_dispatch(int N, int dt, F& f) {
    switch (scan_lanes(N)) {
        case 1: return scan_dispatch_type<1>(dt, f);
        case 2: return scan_dispatch_type<2>(dt, f);
        case 4: return scan_dispatch_type<4>(dt, f);
        case 8: return scan_dispatch_type<8>(dt, f);
    }
    return scan_dispatch_type<16>(dt, f);
}

hc_status launch_scan_fwd(const ScanArgs& a, cudaStream_t st);
hc_status launch_scan_bwd(const ScanArgs& a, cudaStream_t st);
// The first states of the segments in a.carry (rev: of the gradient, from the last row up).
hc_status launch_scan_carry(const ScanArgs& a, bool rev, cudaStream_t st);

}  // namespace hc
