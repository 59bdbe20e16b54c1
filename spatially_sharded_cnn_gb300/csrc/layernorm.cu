// layernorm.cu -- layer norm over the channels of each row, forward and backward
// (hc_layernorm_*).
//
// TPR threads hold one row in registers: its values are read once, the mean and then
// the squared deviations from it are summed from registers (two passes over values
// that do not move, so no cancellation), and the row is written.  Bound by memory:
// x in and y out, and for the backward pass x and gy in and gx out: 224 x 1024 x 512 bf16 take
// 82 us forward, 135 backward (69 and 104 at the rate of a copy).
#include "rows.cuh"

namespace hc {
namespace {

constexpr int LN_THREADS = 256;

struct LnShape {
    int L, C;
    int rows;    // B * L
    float eps;
    const int* lens;
    bool flat;   // rows at one stride throughout, all of them there
};

// Threads of a block: rows of up to a warp share one, a longer row has its own.
__host__ __device__ constexpr int ln_block(int tpr) { return tpr > 32 ? tpr : LN_THREADS; }

// V parameters; their array is aligned to 16 bytes.
template <int V> __device__ __forceinline__ void ln_param(const float* p, float (&f)[V]) {
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(p + i);
            f[i] = q.x;
            f[i + 1] = q.y;
            f[i + 2] = q.z;
            f[i + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) f[i] = p[i];
    }
}

// Sum over the TPR threads of a row; every one of them gets it, added in the same
// order.  red: a slot for each warp of the block, for rows that take several warps.
template <int TPR> __device__ __forceinline__ float ln_sum(float v, float* red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if constexpr (TPR > 32) {
        const int w = threadIdx.x >> 5;
        __syncthreads();  // the sum before has been read
        if ((threadIdx.x & 31) == 0) red[w] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int k = 0; k < TPR / 32; k++) v += red[k];
    }
    return v;
}

// Two at a time.
template <int TPR> __device__ __forceinline__ void ln_sums(float& a, float& b, float* red) {
#pragma unroll
    for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (TPR > 32) {
        const int w = threadIdx.x >> 5;
        __syncthreads();
        if ((threadIdx.x & 31) == 0) {
            red[2 * w] = a;
            red[2 * w + 1] = b;
        }
        __syncthreads();
        a = b = 0.0f;
#pragma unroll
        for (int k = 0; k < TPR / 32; k++) {
            a += red[2 * k];
            b += red[2 * k + 1];
        }
    }
}

__device__ __forceinline__ bool ln_live(const LnShape& s, int b, int l) { return !s.lens || l < s.lens[b]; }

// FLAT: one run of rows at one stride, all of them there.  FULL: threads that all have NV whole
// packs of channels.  Else a thread without channels reads the row's first pack and does not use
// it: no load of a flat row is behind a branch, and those of two rows go out together (224 x 1024 x
// 512 bf16 forward: 140 us with branches, 82 without; 768 channels 155 and 126).  Rows of ragged
// batches stay behind one (5 x 1537 x 330 fp32, training: 19.2 us, 21.2 where they read another's).
struct LnRow {
    long long r;
    int b, l;
    bool in, live;
};
template <bool FLAT> __device__ __forceinline__ LnRow ln_row(const LnShape& s, long long r) {
    if constexpr (FLAT) {
        const bool in = r < s.rows;
        r = in ? r : s.rows - 1;
        return {r, 0, (int)r, in, true};
    } else {
        LnRow w{r, 0, 0, r < s.rows, false};
        if (s.flat) {  // (of accesses that are no whole 16 bytes)
            w.l = (int)r;
            w.live = w.in;
        } else if (w.in) {
            w.b = (int)r / s.L;
            w.l = (int)r - w.b * s.L;
            w.live = ln_live(s, w.b, w.l);
        }
        return w;
    }
}
template <bool FLAT, typename T> __device__ __forceinline__ T* ln_ptr(const View<T>& v, const LnRow& w) {
    return FLAT ? v.p + w.r * v.row : v.p + w.b * v.batch + w.l * v.row;
}

// NV packs of V values a thread: channels (i * TPR + lane) * V of pack i.  Blocks
// walk over the rows, ROWS at a time.
template <typename T, int V, int TPR, int NV, bool FLAT, bool FULL>
__global__ void __launch_bounds__(ln_block(TPR))
    ln_fwd_kernel(View<const T> x, const float* gamma, const float* beta, View<T> y, float* mean, float* rstd,
                  LnShape s) {
    grid_begin();
    constexpr int ROWS = ln_block(TPR) / TPR;
    __shared__ float red[32];
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const float inv = 1.0f / s.C;
    // two rows at once where registers allow: the loads of one are under way while the sums of
    // the other wait for their shuffles (224 x 1024 x 512 bf16: 91 -> 82 us)
    constexpr int U = NV * V <= 16 ? 2 : 1;
    // every thread takes every turn: the sums are of whole warps
    for (long long r0 = (long long)blockIdx.x * ROWS * U; r0 < s.rows; r0 += (long long)gridDim.x * ROWS * U) {
        LnRow w[U];
        Pack<T, V> q[U][NV];
#pragma unroll
        for (int u = 0; u < U; u++) {
            w[u] = ln_row<FLAT>(s, r0 + u * ROWS + sub);
            const T* xr = ln_ptr<FLAT>(x, w[u]);
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const int c = (i * TPR + lane) * V;
                if (FLAT || w[u].live) q[u][i] = load_raw<T, V>(FULL || c < s.C ? xr + c : xr);
            }
        }
        float v[U][NV][V], m[U], rs[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            m[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                unpack(q[u][i], v[u][i]);
                const bool on = FULL || (i * TPR + lane) * V < s.C;
#pragma unroll
                for (int k = 0; k < V; k++) m[u] += on ? v[u][i][k] : 0.0f;
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) m[u] = __fmul_rn(ln_sum<TPR>(m[u], red), inv);  // rounded alike wherever it is used
#pragma unroll
        for (int u = 0; u < U; u++) {
            rs[u] = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; i++) {
                const bool on = FULL || (i * TPR + lane) * V < s.C;
#pragma unroll
                for (int k = 0; k < V; k++) {
                    v[u][i][k] = on ? v[u][i][k] - m[u] : 0.0f;
                    rs[u] = fmaf(v[u][i][k], v[u][i][k], rs[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; u++) rs[u] = __frcp_rn(__fsqrt_rn(ln_sum<TPR>(rs[u], red) * inv + s.eps));
        if (lane == 0) {
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (!w[u].in) continue;
                if (mean) mean[w[u].r] = w[u].live ? m[u] : 0.0f;
                if (rstd) rstd[w[u].r] = w[u].live ? rs[u] : 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * V;
            if (!FULL && c >= s.C) continue;
            float g[V], bt[V];
            ln_param<V>(gamma + c, g);
            ln_param<V>(beta + c, bt);
#pragma unroll
            for (int u = 0; u < U; u++) {
                if (!w[u].in) continue;
                float o[V];
#pragma unroll
                for (int k = 0; k < V; k++) o[k] = w[u].live ? fmaf(v[u][i][k] * rs[u], g[k], bt[k]) : 0.0f;
                store_pack<T, V>(ln_ptr<FLAT>(y, w[u]) + c, o);
            }
        }
    }
}

// A block of LN_THREADS a row that no variant above holds: read three times (7 x 1024 x
// 20480 bf16: 300 us, 87 at the rate of a copy).
template <typename T>
__global__ void __launch_bounds__(LN_THREADS) ln_fwd_long_kernel(View<const T> x, const float* gamma, const float* beta,
                                                                 View<T> y, float* mean, float* rstd, LnShape s) {
    grid_begin();
    __shared__ float red[32];
    for (long long r = blockIdx.x; r < s.rows; r += gridDim.x) {
        const int b = (int)(r / s.L), l = (int)(r - (long long)b * s.L);
        const bool live = ln_live(s, b, l);
        const T* xr = x.p + b * x.batch + l * x.row;
        float sum = 0.0f, sq = 0.0f;
        if (live)
            for (int c = threadIdx.x; c < s.C; c += LN_THREADS) sum += to_f(xr[c]);
        const float m = ln_sum<LN_THREADS>(sum, red) / s.C;
        if (live)
            for (int c = threadIdx.x; c < s.C; c += LN_THREADS) {
                const float d = to_f(xr[c]) - m;
                sq = fmaf(d, d, sq);
            }
        const float rs = __frcp_rn(__fsqrt_rn(ln_sum<LN_THREADS>(sq, red) / s.C + s.eps));
        if (threadIdx.x == 0) {
            if (mean) mean[r] = live ? m : 0.0f;
            if (rstd) rstd[r] = live ? rs : 0.0f;
        }
        T* yr = y.p + b * y.batch + l * y.row;
        for (int c = threadIdx.x; c < s.C; c += LN_THREADS)
            yr[c] = from_f<T>(live ? fmaf((to_f(xr[c]) - m) * rs, gamma[c], beta[c]) : 0.0f);
    }
}

// Backward: a thread keeps the sums for gamma and beta of its channels over the rows
// that its block walks; the block's row groups are then added in order into
// part[block][ggamma C | gbeta C].  gy * gamma is rounded before its mean is taken
// from it, as it was in that mean: where a row's gradient cancels to zero, it is zero.
template <typename T, int V, int TPR, int NV, bool FLAT, bool FULL>
__global__ void __launch_bounds__(ln_block(TPR))
    ln_bwd_kernel(View<const T> x, const float* gamma, const float* mean, const float* rstd, View<const T> gy,
                  View<T> gx, float* part, LnShape s) {
    grid_begin();
    constexpr int ROWS = ln_block(TPR) / TPR;
    __shared__ float red[32];  // two for each of 16 warps
    extern __shared__ float own[];  // [ROWS][2][C], rows of several groups
    const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    const float inv = 1.0f / s.C;
    constexpr int W = (V + 1) / 2;  // values in pairs; a single one has a zero beside it
    f32x2 gg[NV][W], gb[NV][W];
#pragma unroll
    for (int i = 0; i < NV; i++)
#pragma unroll
        for (int k = 0; k < W; k++) gg[i][k] = gb[i][k] = pk2(0.0f, 0.0f);
    // AHEAD: the next row is under way while this one is taken, where the registers for it cost no
    // block (224 x 1024 x 512 bf16: 151 us without, 134 with; x 256, a pack a thread: 73 and 94)
    constexpr bool AHEAD = sizeof(T) == 2 && V == 8 && NV == 2;
    struct Row {
        Pack<T, V> x[NV], g[NV];
        float rs, m;
    };
    const auto fetch = [&](const LnRow& w, Row& o) {
        const T *xr = ln_ptr<FLAT>(x, w), *gr = ln_ptr<FLAT>(gy, w);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * V;
            if (!FLAT && !w.live) continue;
            o.x[i] = load_raw<T, V>(FULL || c < s.C ? xr + c : xr);
            o.g[i] = load_raw<T, V>(FULL || c < s.C ? gr + c : gr);
        }
        o.rs = FLAT || w.live ? rstd[w.r] : 0.0f;
        o.m = FLAT || w.live ? -mean[w.r] : 0.0f;
    };
    const long long step = (long long)gridDim.x * ROWS;
    Row ahead;
    if constexpr (AHEAD) fetch(ln_row<FLAT>(s, blockIdx.x * (long long)ROWS + sub), ahead);
    for (long long r0 = (long long)blockIdx.x * ROWS; r0 < s.rows; r0 += step) {
        const LnRow w = ln_row<FLAT>(s, r0 + sub);
        const bool live = FLAT ? w.in : w.live;
        Row row;
        if constexpr (AHEAD) {
            row = ahead;
            fetch(ln_row<FLAT>(s, r0 + step + sub), ahead);
        } else {
            fetch(w, row);
        }
        Pack<T, V>(&xq)[NV] = row.x;
        Pack<T, V>(&gq)[NV] = row.g;
        const f32x2 rs2 = pk2(row.rs, row.rs), mm = pk2(row.m, row.m);
        // xhat and gamma * gy of pair k of pack i
        const auto pair = [&](int i, int k, const float(&ga)[V], f32x2& xh, f32x2& g, f32x2& q) {
            float xv[V], gv[V];
            unpack(xq[i], xv);
            unpack(gq[i], gv);
            const int o = V > 1 ? 2 * k + 1 : 0;
            xh = mul2(add2(pk2(xv[2 * k], V > 1 ? xv[o] : 0.0f), mm), rs2);
            g = pk2(gv[2 * k], V > 1 ? gv[o] : 0.0f);
            // (a packed product would be fused with the addition that follows)
            q = pk2(__fmul_rn(gv[2 * k], ga[2 * k]), V > 1 ? __fmul_rn(gv[o], ga[o]) : 0.0f);
        };
        f32x2 a1 = pk2(0.0f, 0.0f), a2 = a1;
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * V;
            if (!live || (!FULL && c >= s.C)) continue;
            float ga[V];
            ln_param<V>(gamma + c, ga);
#pragma unroll
            for (int k = 0; k < W; k++) {
                f32x2 xh, g, q;
                pair(i, k, ga, xh, g, q);
                gg[i][k] = fma2(g, xh, gg[i][k]);
                gb[i][k] = add2(gb[i][k], g);
                a1 = add2(a1, q);
                a2 = fma2(q, xh, a2);
            }
        }
        float s1, s2, t;
        unpk2(a1, s1, t);
        s1 += t;
        unpk2(a2, s2, t);
        s2 += t;
        ln_sums<TPR>(s1, s2, red);
        s1 = -__fmul_rn(s1, inv);
        s2 = -__fmul_rn(s2, inv);
        if (!w.in) continue;
        const f32x2 m1 = pk2(s1, s1), m2 = pk2(s2, s2);
        T* out = ln_ptr<FLAT>(gx, w);
#pragma unroll
        for (int i = 0; i < NV; i++) {
            const int c = (i * TPR + lane) * V;
            if (!FULL && c >= s.C) continue;
            float o[V];
            if (live) {
                float ga[V];
                ln_param<V>(gamma + c, ga);
#pragma unroll
                for (int k = 0; k < W; k++) {
                    f32x2 xh, g, q;
                    pair(i, k, ga, xh, g, q);
                    float lo, hi;
                    unpk2(mul2(rs2, fma2(xh, m2, add2(q, m1))), lo, hi);
                    o[2 * k] = lo;
                    if (V > 1) o[V > 1 ? 2 * k + 1 : 0] = hi;
                }
            } else {
#pragma unroll
                for (int k = 0; k < V; k++) o[k] = 0.0f;
            }
            store_pack<T, V>(out + c, o);
        }
    }
    if (!part) return;
    float* p = part + (long long)blockIdx.x * 2 * s.C;
    float* o = ROWS == 1 ? p : own + sub * 2 * s.C;
#pragma unroll
    for (int i = 0; i < NV; i++) {
        const int c = (i * TPR + lane) * V;
        if (c >= s.C) continue;
#pragma unroll
        for (int k = 0; k < W; k++) {
            float lo, hi;
            unpk2(gg[i][k], lo, hi);
            o[c + 2 * k] = lo;
            if (V > 1) o[c + 2 * k + 1] = hi;
            unpk2(gb[i][k], lo, hi);
            o[s.C + c + 2 * k] = lo;
            if (V > 1) o[s.C + c + 2 * k + 1] = hi;
        }
    }
    if constexpr (ROWS > 1) {
        __syncthreads();
        for (int c = threadIdx.x; c < 2 * s.C; c += LN_THREADS) {
            float t = own[c];
#pragma unroll 4
            for (int k = 1; k < ROWS; k++) t += own[k * 2 * s.C + c];
            p[c] = t;
        }
    }
}

// Rows that no variant above holds: a block's sums stay in its row of `part`, read and written for every
// row (28 x 1024 x 12288 bf16: 3300 us, 312 at the rate of a copy).
template <typename T>
__global__ void __launch_bounds__(LN_THREADS)
    ln_bwd_long_kernel(View<const T> x, const float* gamma, const float* mean, const float* rstd, View<const T> gy,
                       View<T> gx, float* part, LnShape s) {
    grid_begin();
    __shared__ float red[32];
    float* p = part ? part + (long long)blockIdx.x * 2 * s.C : nullptr;
    if (p)
        for (int c = threadIdx.x; c < s.C; c += LN_THREADS) p[c] = p[s.C + c] = 0.0f;
    for (long long r = blockIdx.x; r < s.rows; r += gridDim.x) {
        const int b = (int)(r / s.L), l = (int)(r - (long long)b * s.L);
        const bool live = ln_live(s, b, l);
        const T* xr = x.p + b * x.batch + l * x.row;
        const T* gr = gy.p + b * gy.batch + l * gy.row;
        const float m = live ? mean[r] : 0.0f, rs = live ? rstd[r] : 0.0f;
        float s1 = 0.0f, s2 = 0.0f;
        if (live)
            for (int c = threadIdx.x; c < s.C; c += LN_THREADS) {
                const float xh = (to_f(xr[c]) - m) * rs, g = to_f(gr[c]), q = __fmul_rn(g, gamma[c]);
                if (p) {
                    p[c] = fmaf(g, xh, p[c]);
                    p[s.C + c] += g;
                }
                s1 += q;
                s2 = fmaf(q, xh, s2);
            }
        const float m1 = ln_sum<LN_THREADS>(s1, red) / s.C, m2 = ln_sum<LN_THREADS>(s2, red) / s.C;
        T* o = gx.p + b * gx.batch + l * gx.row;
        for (int c = threadIdx.x; c < s.C; c += LN_THREADS)
            o[c] = from_f<T>(live ? rs * (__fmul_rn(to_f(gr[c]), gamma[c]) - m1 - (to_f(xr[c]) - m) * rs * m2) : 0.0f);
    }
}

// The threads of a row and the packs a thread, MOST values or fewer: the first that hold C
// channels (a variant that holds no more than one with fewer threads is left out: 224 x 1024 x 333 bf16
// forward takes 180 us with 128 threads a row of four values each, 135 with a warp).  False: none does.
template <int V, int MOST, int TPR, int NV, typename F> bool ln_try(int C, F& f) {
    constexpr int packs = MOST / V < 16 ? MOST / V : 16, warp = 32 * packs, two = warp > 128 ? warp : 128;
    constexpr int less = TPR == 64 ? warp : TPR == 128 ? two : TPR == 512 ? 128 * packs : 0;
    if constexpr (NV * V <= MOST && TPR * NV > less)
        if (C <= TPR * NV * V) {
            f.template run<V, TPR, NV>();
            return true;
        }
    return false;
}
template <int V, int MOST, typename F> bool ln_dispatch(int C, F& f) {
    return ln_try<V, MOST, 8, 1>(C, f) || ln_try<V, MOST, 8, 2>(C, f) || ln_try<V, MOST, 32, 1>(C, f) ||
           ln_try<V, MOST, 32, 2>(C, f) || ln_try<V, MOST, 32, 3>(C, f) || ln_try<V, MOST, 32, 4>(C, f) ||
           ln_try<V, MOST, 32, 8>(C, f) || ln_try<V, MOST, 32, 16>(C, f) || ln_try<V, MOST, 64, 2>(C, f) ||
           ln_try<V, MOST, 128, 2>(C, f) || ln_try<V, MOST, 128, 4>(C, f) || ln_try<V, MOST, 128, 8>(C, f) ||
           ln_try<V, MOST, 128, 16>(C, f) || ln_try<V, MOST, 512, 1>(C, f) || ln_try<V, MOST, 512, 2>(C, f) ||
           ln_try<V, MOST, 512, 4>(C, f) || ln_try<V, MOST, 512, 8>(C, f) || ln_try<V, MOST, 512, 16>(C, f);
}

// Blocks of the backward pass: each leaves a row of sums.
long long ln_blocks(const hc_layernorm_desc* d) {
    // (rows of 513 to 2048 channels take blocks of 64 or 128 threads)
    const long long rows = (long long)d->B * d->L, most = (d->C > 512 && d->C <= 2048 ? 8LL : 4LL) * device_sm_count();
    return rows < most ? rows : most;
}

bool ln_desc_ok(const hc_layernorm_desc* d) {
    return d && d->B >= 1 && d->L >= 0 && d->C >= 1 && d->eps >= 0.0f && dtype_ok(d->dtype);
}
bool ln_size_ok(const hc_layernorm_desc* d) { return d->C <= 1 << 20 && (long long)d->B * d->L < 1LL << 31; }

template <typename T> struct LnFwd {
    const hc_rows *x, *y;
    const float *gamma, *beta;
    float *mean, *rstd;
    LnShape s;
    cudaStream_t st;
    template <int V, int TPR, int NV> void run() {
        if constexpr (sizeof(T) * V == 16)
            if (s.flat) return s.C == TPR * NV * V ? go<V, TPR, NV, true, true>() : go<V, TPR, NV, true, false>();
        go<V, TPR, NV, false, false>();
    }
    template <int V, int TPR, int NV, bool FLAT, bool FULL> void go() {
        constexpr int threads = ln_block(TPR), rows = threads / TPR;
        const long long want = cdiv(s.rows, rows * (NV * V <= 16 ? 2 : 1)), most = 32LL * device_sm_count();
        const dim3 grid((unsigned)(want < most ? want : most));
        launch_next(ln_fwd_kernel<T, V, TPR, NV, FLAT, FULL>, grid, dim3(threads), 0, st,
                    view<const T>(x), gamma, beta, view<T>(y), mean, rstd, s);
    }
};

template <typename T> struct LnBwd {
    const hc_rows *x, *gy, *gx;
    const float *gamma, *mean, *rstd;
    float* part;
    LnShape s;
    long long blocks;
    cudaStream_t st;
    template <int V, int TPR, int NV> void run() {
        if constexpr (sizeof(T) * V == 16)
            if (s.flat) return s.C == TPR * NV * V ? go<V, TPR, NV, true, true>() : go<V, TPR, NV, true, false>();
        go<V, TPR, NV, false, false>();
    }
    template <int V, int TPR, int NV, bool FLAT, bool FULL> void go() {
        constexpr int threads = ln_block(TPR);
        const size_t smem = threads > TPR ? (size_t)(threads / TPR) * 2 * s.C * sizeof(float) : 0;
        launch_next(ln_bwd_kernel<T, V, TPR, NV, FLAT, FULL>, dim3((unsigned)blocks), dim3(threads), smem, st,
                    view<const T>(x), gamma, mean, rstd, view<const T>(gy), view<T>(gx), part, s);
    }
};

// Accesses of V elements (16 bytes, or two): whole packs in a row, every row on such a boundary
// (224 x 1024 x 330 bf16, training: 321 us in twos, 668 one by one).
template <int V> bool ln_wide(int C, const hc_rows* a, const hc_rows* b, const hc_rows* c) {
    return C % V == 0 && rows_vec(a, V) && rows_vec(b, V) && (!c || rows_vec(c, V));
}

// Rows at one stride throughout.
bool ln_flat(const hc_layernorm_desc* d, const hc_rows* r) { return d->B == 1 || r->batch == d->L * r->row; }

template <typename T>
hc_status ln_fwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* beta, const hc_rows* y,
                 float* mean, float* rstd, const int* lens, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    LnFwd<T> f{x, y, gamma, beta, mean, rstd, 
               {d->L, d->C, d->B * d->L, d->eps, lens, !lens && ln_flat(d, x) && ln_flat(d, y)}, st};
    if (!(ln_wide<W>(d->C, x, y, nullptr)   ? ln_dispatch<W, 32>(d->C, f)
          : ln_wide<2>(d->C, x, y, nullptr) ? ln_dispatch<2, 16>(d->C, f)
                                            : ln_dispatch<1, 16>(d->C, f))) {
        const long long most = 8LL * device_sm_count();
        launch_next(ln_fwd_long_kernel<T>, dim3((unsigned)(f.s.rows < most ? f.s.rows : most)), dim3(LN_THREADS), 0, st,
                    view<const T>(x), gamma, beta, view<T>(y), mean, rstd, f.s);
    }
    return launched("ln_fwd_kernel", st);
}

template <typename T>
hc_status ln_bwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* mean, const float* rstd,
                 const hc_rows* gy, const hc_rows* gx, float* part, const int* lens, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    LnBwd<T> f{x, gy, gx, gamma, mean, rstd, part,
               {d->L, d->C, d->B * d->L, d->eps, lens, !lens && ln_flat(d, x) && ln_flat(d, gy) && ln_flat(d, gx)},
               ln_blocks(d), st};
    if (!(ln_wide<W>(d->C, x, gy, gx)   ? ln_dispatch<W, 16>(d->C, f)
          : ln_wide<2>(d->C, x, gy, gx) ? ln_dispatch<2, 16>(d->C, f)
                                        : ln_dispatch<1, 16>(d->C, f)))
        launch_next(ln_bwd_long_kernel<T>, dim3((unsigned)f.blocks), dim3(LN_THREADS), 0, st, view<const T>(x), gamma,
                    mean, rstd, view<const T>(gy), view<T>(gx), part, f.s);
    return launched("ln_bwd_kernel", st);
}

}  // namespace
}  // namespace hc

using namespace hc;

extern "C" {

hc_status hc_layernorm_fwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const hc_rows* y, float* mean, float* rstd, const int* lens, void* stream) {
    if (!ln_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!ln_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!rows_in_ok(x, d->dtype, d->L) || !rows_out_ok(y, d->dtype, d->B, d->L, d->C) || rows_same(x, y) ||
        !f32_ok(gamma) || !f32_ok(beta) || !f32_opt_ok(mean) || !f32_opt_ok(rstd) || (mean && mean == rstd) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    if (d->L == 0) return HC_OK;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    if (d->dtype == HC_DTYPE_F32) return ln_fwd<float>(d, x, gamma, beta, y, mean, rstd, lens, st);
    if (d->dtype == HC_DTYPE_BF16) return ln_fwd<__nv_bfloat16>(d, x, gamma, beta, y, mean, rstd, lens, st);
    return ln_fwd<__half>(d, x, gamma, beta, y, mean, rstd, lens, st);
}

// [blocks][ggamma C | gbeta C]
hc_status hc_layernorm_workspace_size(const hc_layernorm_desc* d, size_t* bytes) {
    if (!ln_desc_ok(d) || !bytes) return HC_ERR_INVALID_ARG;
    if (!ln_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = (size_t)ln_blocks(d) * 2 * d->C * sizeof(float);
    return HC_OK;
}

hc_status hc_layernorm_bwd(const hc_layernorm_desc* d, const hc_rows* x, const float* gamma, const float* mean,
                           const float* rstd, const hc_rows* gy, const hc_rows* gx, float* ggamma, float* gbeta,
                           const int* lens, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    hc_status e = hc_layernorm_workspace_size(d, &need);
    if (e) return e;
    if (!rows_in_ok(x, d->dtype, d->L) || !rows_in_ok(gy, d->dtype, d->L) ||
        !rows_out_ok(gx, d->dtype, d->B, d->L, d->C) || rows_same(gx, x) || rows_same(gx, gy) || !f32_ok(gamma) ||
        (d->L > 0 && (!f32_ok(mean) || !f32_ok(rstd))) || !f32_opt_ok(ggamma) || !f32_opt_ok(gbeta) ||
        (ggamma && ggamma == gbeta) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    const bool sums = ggamma || gbeta;
    if (sums && need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    float* part = sums ? (float*)ws : nullptr;
    if (d->L > 0) {
        if (d->dtype == HC_DTYPE_F32)
            e = ln_bwd<float>(d, x, gamma, mean, rstd, gy, gx, part, lens, st);
        else if (d->dtype == HC_DTYPE_BF16)
            e = ln_bwd<__nv_bfloat16>(d, x, gamma, mean, rstd, gy, gx, part, lens, st);
        else
            e = ln_bwd<__half>(d, x, gamma, mean, rstd, gy, gx, part, lens, st);
        if (e) return e;
    }
    if (!sums) return HC_OK;
    return launch_column_totals(part, d->L > 0 ? ln_blocks(d) : 0, ggamma, d->C, gbeta, d->C, nullptr, 0, st);
}

}  // extern "C"
