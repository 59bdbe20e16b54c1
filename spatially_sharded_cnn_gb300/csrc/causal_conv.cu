// causal_conv.cu -- short causal depthwise convolution along channels-last
// sequences [B][L][D], forward, backward and one token (formulas:
// hc_mixer.h).  The K - 1 rows before a sequence come from a carried state:
// the left halo of a sequence cut into blocks.
//
// Bound by memory: a thread takes V adjacent channels and a run of rows, slides
// a K-row window in registers (two channels a register pair, packed
// multiply-adds) and reads each row once; only the K - 1 rows where two runs meet
// are read twice (from L1 or L2).  The next few rows are loaded while the last
// ones are worked on, which is what keeps enough bytes in flight.
#include "rows.cuh"

namespace hc {
namespace {

constexpr int CC_THREADS = 128;
constexpr int CC_RUN = 64;  // rows a thread takes at most
// Channels a thread where the rows allow it, and rows loaded ahead.  Forward on 8 x
// 4096 x 1024 bf16: 4 channels and 8 rows 35 us, 4 and 4 40, 8 and 4 39; backward
// on 56 x 1023 x 264 fp32: 4 rows 63 us, 8 rows 84 (two windows and two tensors fill
// its registers).
constexpr int CC_V = 4, CC_FWD_U = 8, CC_BWD_U = 4;

// Thread (col, r) of a block: channel vector blockIdx.y * ncol + col, run
// (blockIdx.x % blocks) * R + r of sequence blockIdx.x / blocks.
struct CcShape {
    int B, L, D;
    int cv, ncol, R;  // channel vectors; of them and runs per block
    int run;          // rows a run
    int blocks;       // blocks along a sequence
};

template <typename T, int V>
__device__ __forceinline__ void load_or_zero(const T* p, bool on, float (&f)[V]) {
    if (on) {
        load_pack<T, V>(p, f);
    } else {
#pragma unroll
        for (int i = 0; i < V; i++) f[i] = 0.0f;
    }
}
// V channels as pairs (the second of a lone channel's is zero).
template <int V> struct Pairs {
    static constexpr int N = (V + 1) / 2;
    f32x2 v[N];
    __device__ __forceinline__ void set(const float (&f)[V]) {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = pk2(f[2 * i], 2 * i + 1 < V ? f[2 * i + 1 < V ? 2 * i + 1 : 0] : 0.0f);
    }
    __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
        for (int i = 0; i < N; i++) {
            float lo, hi;
            unpk2(v[i], lo, hi);
            f[2 * i] = lo;
            if (2 * i + 1 < V) f[2 * i + 1 < V ? 2 * i + 1 : 0] = hi;
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < N; i++) v[i] = 0;
    }
};
// The weights and bias of a thread's channels: V * K adjacent floats, by 16 bytes
// (single loads at a stride of K floats cost more than a run's rows).
template <int V, int K>
__device__ __forceinline__ void load_taps(const float* w, const float* bias, int c0, Pairs<V> (&wk)[K], Pairs<V>& b) {
    float t[V * K], f[V];
    constexpr int Q = V % 4 == 0 ? 4 : 1;
#pragma unroll
    for (int q = 0; q < V * K; q += Q) {
        float v[Q];
        load_pack<float, Q>(w + (long long)c0 * K + q, v);
#pragma unroll
        for (int i = 0; i < Q; i++) t[q + i] = v[i];
    }
#pragma unroll
    for (int k = 0; k < K; k++) {
#pragma unroll
        for (int i = 0; i < V; i++) f[i] = t[i * K + k];
        wk[k].set(f);
    }
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = 0.0f;
    if (bias) {
#pragma unroll
        for (int q = 0; q < V; q += Q) {
            float v[Q];
            load_pack<float, Q>(bias + c0 + q, v);
#pragma unroll
            for (int i = 0; i < Q; i++) f[q + i] = v[i];
        }
    }
    b.set(f);
}
// Rows t .. t + U - 1 of those below end, as stored.
template <typename T, int V, int U>
__device__ __forceinline__ void load_rows(const T* p, long long row, int t, int end, Pack<T, V> (&q)[U]) {
#pragma unroll
    for (int u = 0; u < U; u++)
        if (t + u < end) q[u] = load_raw<T, V>(p + (t + u) * row);
}

__device__ __forceinline__ int seq_len(const int* lens, int b, int L) {
    return lens ? min(max(lens[b], 0), L) : L;
}

// Row t >= -(K-1) of the sequence whose rows before 0 are `state`.
template <typename T, int V, int K>
__device__ __forceinline__ void load_row(const T* xb, long long row, const T* state, long long D, int t, bool on,
                                         float (&f)[V]) {
    if (t >= 0)
        load_or_zero<T, V>(xb + t * row, on, f);
    else
        load_or_zero<T, V>(state + (t + K - 1) * D, on && state != nullptr, f);
}

// 8 x 4096 x 1024 bf16, K = 4, SiLU (134 MB): 30 us a call, 4.5 TB/s; bound by the bytes
// it has in flight: its rows ahead are in registers, and 122 of those leave four blocks
// an SM, 32 KB of loads (1216 blocks, two full waves).
template <typename T, int V, int K, int ACT>
__global__ void __launch_bounds__(CC_THREADS) cc_fwd_kernel(View<const T> x, View<T> y, const float* w,
                                                            const float* bias,
                                                            const T* state_in, T* state_out,
                                                            const int* lens, CcShape s) {
    grid_begin();
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.y * s.ncol + col;
    if (r >= s.R || cvec >= s.cv) return;
    const int b = blockIdx.x / s.blocks, blk = blockIdx.x % s.blocks;
    const int len = seq_len(lens, b, s.L);
    const long long t0l = ((long long)blk * s.R + r) * s.run;
    const int c0 = cvec * V;
    const T* xb = x.p + b * x.batch + c0;
    const T* si = state_in ? state_in + (long long)b * (K - 1) * s.D + c0 : nullptr;
    if (t0l == 0 && state_out) {
        T* so = state_out + (long long)b * (K - 1) * s.D + c0;
#pragma unroll
        for (int j = 0; j < K - 1; j++) {
            float v[V];
            load_row<T, V, K>(xb, x.row, si, s.D, len - (K - 1) + j, true, v);
            store_pack<T, V>(so + (long long)j * s.D, v);
        }
    }
    if (t0l >= s.L) return;
    const int t0 = (int)t0l, t1 = min(t0 + s.run, s.L), live = min(t1, len);
    T* yb = y.p + b * y.batch + c0;
    if (t0 < live) {
        Pack<T, V> now[CC_FWD_U], next[CC_FWD_U];
        load_rows<T, V>(xb, x.row, t0, live, now);
        Pairs<V> wk[K], bb, win[K];
        load_taps<V, K>(w, bias, c0, wk, bb);
#pragma unroll
        for (int k = 0; k < K - 1; k++) {
            float f[V];
            load_row<T, V, K>(xb, x.row, si, s.D, t0 - (K - 1) + k, true, f);
            win[k].set(f);
        }
        for (int t = t0; t < live; t += CC_FWD_U) {
            load_rows<T, V>(xb, x.row, t + CC_FWD_U, live, next);
#pragma unroll
            for (int u = 0; u < CC_FWD_U; u++) {
                if (t + u < live) {
                    float f[V];
                    unpack(now[u], f);
                    win[K - 1].set(f);
                    Pairs<V> o;
#pragma unroll
                    for (int i = 0; i < Pairs<V>::N; i++) {
                        o.v[i] = bb.v[i];
#pragma unroll
                        for (int k = 0; k < K; k++) o.v[i] = fma2(wk[k].v[i], win[k].v[i], o.v[i]);
                    }
                    o.get(f);
#pragma unroll
                    for (int i = 0; i < V; i++) f[i] = act_f<ACT>(f[i]);
                    store_pack<T, V>(yb + (t + u) * y.row, f);
                }
#pragma unroll
                for (int k = 0; k < K - 1; k++) win[k] = win[k + 1];
            }
#pragma unroll
            for (int u = 0; u < CC_FWD_U; u++) now[u] = next[u];
        }
    }
    float zero[V];
#pragma unroll
    for (int i = 0; i < V; i++) zero[i] = 0.0f;
    for (int t = max(t0, live); t < t1; t++) store_pack<T, V>(yb + t * y.row, zero);
}

// A run's rows [t0, t1): g_t for t in [t0, t1 + K - 1) recomputed, gx_t from
// the K-row window of g, gw and gb summed over its own rows; the block's sums
// go to part[block][(K + 1) * D]: K weights a channel, then the bias sums.
// 56 x 1023 x 264 fp32, ragged: 50 us (121 MB with half of the rows there), 166
// registers, three blocks an SM; bound by the bytes in flight as the forward kernel is.
template <typename T, int V, int K, int ACT>
__global__ void __launch_bounds__(CC_THREADS) cc_bwd_kernel(View<const T> x, View<const T> gy, View<T> gx,
                                                            const float* w, const float* bias,
                                                            const T* state_in,
                                                            const T* gstate_out,
                                                            T* gstate_in, float* part,
                                                            const int* lens, CcShape s) {
    grid_begin();
    __shared__ float sm[CC_THREADS * V];
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.y * s.ncol + col;
    const bool on = r < s.R && cvec < s.cv;
    const int b = blockIdx.x / s.blocks, blk = blockIdx.x % s.blocks;
    const int len = seq_len(lens, b, s.L);
    const long long t0l = ((long long)blk * s.R + r) * s.run;
    const int c0 = cvec * V;
    Pairs<V> gw[K], gb;
    gb.zero();
#pragma unroll
    for (int k = 0; k < K; k++) gw[k].zero();
    if (on && (t0l < s.L || t0l == 0)) {
        const int t0 = (int)t0l, t1 = min(t0 + s.run, s.L);
        const T* xb = x.p + b * x.batch + c0;
        const T* gyb = gy.p + b * gy.batch + c0;
        T* gxb = gx.p ? gx.p + b * gx.batch + c0 : nullptr;
        const long long cs = (long long)b * (K - 1) * s.D + c0;
        const T* si = state_in ? state_in + cs : nullptr;
        const int end = t1 + K - 1;  // one past the last row whose g this run needs
        const int live = min(end, len);
        Pack<T, V> xn[CC_BWD_U], gn[CC_BWD_U], xq[CC_BWD_U], gq[CC_BWD_U];
        load_rows<T, V>(xb, x.row, t0, live, xn);
        load_rows<T, V>(gyb, gy.row, t0, live, gn);
        Pairs<V> wk[K], bb, win[K], gwin[K];
        load_taps<V, K>(w, bias, c0, wk, bb);
#pragma unroll
        for (int k = 0; k < K; k++) gwin[k].zero();
#pragma unroll
        for (int k = 0; k < K - 1; k++) {
            float f[V];
            load_row<T, V, K>(xb, x.row, si, s.D, t0 - (K - 1) + k, t0 <= len, f);
            win[k].set(f);
        }
        // gwin[K - 1] = g_t; the row finished at t is t - (K - 1)
        for (int t = t0; t < end; t += CC_BWD_U) {
            load_rows<T, V>(xb, x.row, t + CC_BWD_U, live, xq);
            load_rows<T, V>(gyb, gy.row, t + CC_BWD_U, live, gq);
#pragma unroll
            for (int u = 0; u < CC_BWD_U; u++) {
                const int tt = t + u;
                float f[V], g[V];
                if (tt < live) {
                    unpack(xn[u], f);
                    win[K - 1].set(f);
                    Pairs<V> o;
#pragma unroll
                    for (int i = 0; i < Pairs<V>::N; i++) {
                        o.v[i] = bb.v[i];
#pragma unroll
                        for (int k = 0; k < K; k++) o.v[i] = fma2(wk[k].v[i], win[k].v[i], o.v[i]);
                    }
                    o.get(f);
                    unpack(gn[u], g);
#pragma unroll
                    for (int i = 0; i < V; i++) f[i] = g[i] * act_d<ACT>(f[i]);
                    gwin[K - 1].set(f);
                    if (tt < t1) {  // its own row
#pragma unroll
                        for (int i = 0; i < Pairs<V>::N; i++) {
                            gb.v[i] = add2(gb.v[i], gwin[K - 1].v[i]);
#pragma unroll
                            for (int k = 0; k < K; k++)
                                gw[k].v[i] = fma2(gwin[K - 1].v[i], win[k].v[i], gw[k].v[i]);
                        }
                    }
                } else {
                    win[K - 1].zero();
                    gwin[K - 1].zero();
                }
                const int row = tt - (K - 1);
                if (tt < end && (row >= t0 ? gxb != nullptr : t0 == 0 && gstate_in != nullptr)) {
                    Pairs<V> o;
#pragma unroll
                    for (int i = 0; i < Pairs<V>::N; i++) {
                        o.v[i] = mul2(wk[0].v[i], gwin[K - 1].v[i]);
#pragma unroll
                        for (int k = 1; k < K; k++) o.v[i] = fma2(wk[k].v[i], gwin[K - 1 - k].v[i], o.v[i]);
                    }
                    o.get(f);
                    const int j = row - (len - (K - 1));  // its row of state_out, if any
                    if (row >= len) {
#pragma unroll
                        for (int i = 0; i < V; i++) f[i] = 0.0f;
                    } else if (gstate_out && j >= 0) {
                        load_pack<T, V>(gstate_out + cs + (long long)j * s.D, g);
#pragma unroll
                        for (int i = 0; i < V; i++) f[i] += g[i];
                    }
                    if (row >= t0)
                        store_pack<T, V>(gxb + row * gx.row, f);
                    else
                        store_pack<T, V>(gstate_in + cs + (long long)(row + K - 1) * s.D, f);
                }
#pragma unroll
                for (int k = 0; k < K - 1; k++) {
                    win[k] = win[k + 1];
                    gwin[k] = gwin[k + 1];
                }
            }
#pragma unroll
            for (int u = 0; u < CC_BWD_U; u++) {
                xn[u] = xq[u];
                gn[u] = gq[u];
            }
        }
    }
    if (!part) return;
    // the runs' sums in run order
    const int wd = s.ncol * V;
    float* pb = part + (long long)blockIdx.x * (K + 1) * s.D;
#pragma unroll
    for (int k = 0; k <= K; k++) {
        if (on) {
            float f[V];
            (k < K ? gw[k < K ? k : 0] : gb).get(f);
#pragma unroll
            for (int i = 0; i < V; i++) sm[r * wd + col * V + i] = f[i];
        }
        __syncthreads();
        for (int q = threadIdx.x; q < wd; q += CC_THREADS) {
            const int c = blockIdx.y * wd + q;
            if (c < s.D) {
                float a = 0.0f;
                for (int m = 0; m < s.R; m++) a += sm[m * wd + q];
                pb[k < K ? (long long)c * K + k : (long long)K * s.D + c] = a;
            }
        }
        __syncthreads();
    }
}

// One token: y from the carried rows and x, and the carried rows moved on.  64 x
// 2048 bf16: 5.5 to 5.9 us a call from Python, most of it the call; replayed from a graph
// with the carried rows in DRAM 3.0 us.
template <typename T, int V, int K, int ACT>
__global__ void __launch_bounds__(128) cc_step_kernel(View<const T> x, View<T> y, const float* w,
                                                      const float* bias, T* state, int B,
                                                      int D, int cv) {
    grid_begin();
    const long long q = blockIdx.x * 128LL + threadIdx.x;
    if (q >= (long long)B * cv) return;
    const int b = (int)(q / cv), c0 = (int)(q % cv) * V;
    T* sb = state + (long long)b * (K - 1) * D + c0;
    float win[K][V], o[V];
#pragma unroll
    for (int k = 0; k < K - 1; k++) load_pack<T, V>(sb + (long long)k * D, win[k]);
    load_pack<T, V>(x.p + b * x.batch + c0, win[K - 1]);
#pragma unroll
    for (int i = 0; i < V; i++) {
        float a = bias ? bias[c0 + i] : 0.0f;
#pragma unroll
        for (int k = 0; k < K; k++) a = fmaf(w[(long long)(c0 + i) * K + k], win[k][i], a);
        o[i] = act_f<ACT>(a);
    }
    store_pack<T, V>(y.p + b * y.batch + c0, o);
#pragma unroll
    for (int k = 0; k < K - 1; k++) store_pack<T, V>(sb + (long long)k * D, win[k + 1]);
}

// Channel vectors a block: the split of a row into equal parts (of 128 bytes or
// more, and whole 32-byte sectors) that leaves the fewest threads without one.
// (264 fp32 channels: 66 of 128 threads busy with one part, 126 with five.)
int cc_columns(int cv) {
    int best = cv < CC_THREADS ? cv : CC_THREADS;
    double most = 0.0;
    for (int parts = 1; parts <= 16; parts++) {
        const int n = (int)cdiv(cv, parts);
        if (n > CC_THREADS || (parts > 1 && (n % 2 || n < 8))) continue;
        const double busy = (double)cv * (CC_THREADS / n) / cdiv(cv, n);
        if (busy > 1.05 * most) {
            most = busy;
            best = n;
        }
    }
    return best;
}

CcShape cc_shape(const hc_causal_conv_desc* d, int V) {
    CcShape s;
    s.B = d->B;
    s.L = d->L;
    s.D = d->D;
    s.cv = d->D / V;
    s.ncol = cc_columns(s.cv);
    s.R = CC_THREADS / s.ncol;
    // runs of CC_RUN rows, shorter where that leaves the launch under eight blocks an
    // SM, two rounds of the four (backward: three) that are resident (backward as above:
    // runs of 16, 32, 64 rows 82, 66, 61 us)
    const long long cols = cdiv(s.cv, s.ncol);
    long long runs = cdiv(s.L, CC_RUN);
    const long long want = cdiv(8LL * device_sm_count() * s.R, (long long)s.B * cols);
    if (runs < want) runs = want;
    const long long most = cdiv(s.L, 4);
    if (runs > most) runs = most;
    if (runs < 1) runs = 1;
    s.run = s.L > 0 ? (int)cdiv(s.L, runs) : 1;
    const long long r = s.L > 0 ? cdiv(s.L, s.run) : 1;
    s.blocks = (int)cdiv(r, s.R);
    return s;
}

size_t cc_part_bytes(const hc_causal_conv_desc* d) {
    size_t rows = 0;
    for (int v : {1, CC_V}) {
        if (d->D % v) continue;
        const CcShape s = cc_shape(d, v);
        const size_t n = (size_t)s.B * s.blocks;
        if (n > rows) rows = n;
    }
    return sizeof(float) * rows * (d->K + 1) * d->D;
}

bool cc_desc_ok(const hc_causal_conv_desc* d) {
    return d && d->B > 0 && d->L >= 0 && d->D > 0 && d->K >= 1 && (d->act == HC_PW_NONE || d->act == HC_PW_SILU) &&
           dtype_ok(d->dtype);
}
bool cc_size_ok(const hc_causal_conv_desc* d) {
    return d->K >= 2 && d->K <= 8 && d->D <= (1 << 20) && (long long)d->B * (d->L / 4 + 1) < (1LL << 31) &&
           d->L <= 0x7fffffff - 64;
}

template <typename T, int V, int K, typename F> hc_status cc_act(int act, F&& f) {
    return act == HC_PW_SILU ? f.template operator()<T, V, K, HC_PW_SILU>()
                             : f.template operator()<T, V, K, HC_PW_NONE>();
}
template <typename T, int K, typename F> hc_status cc_vec(bool vec, int act, F&& f) {
    return vec ? cc_act<T, CC_V, K>(act, f) : cc_act<T, 1, K>(act, f);
}
template <typename T, typename F> hc_status cc_k(int K, bool vec, int act, F&& f) {
    switch (K) {
        case 2: return cc_vec<T, 2>(vec, act, f);
        case 3: return cc_vec<T, 3>(vec, act, f);
        case 4: return cc_vec<T, 4>(vec, act, f);
        case 5: return cc_vec<T, 5>(vec, act, f);
        case 6: return cc_vec<T, 6>(vec, act, f);
        case 7: return cc_vec<T, 7>(vec, act, f);
        case 8: return cc_vec<T, 8>(vec, act, f);
    }
    return HC_ERR_UNSUPPORTED;
}
template <typename F> hc_status cc_dispatch(const hc_causal_conv_desc* d, bool vec, F&& f) {
    if (d->dtype == HC_DTYPE_F32) return cc_k<float>(d->K, vec, d->act, f);
    if (d->dtype == HC_DTYPE_BF16) return cc_k<__nv_bfloat16>(d->K, vec, d->act, f);
    return cc_k<__half>(d->K, vec, d->act, f);
}

struct CcFwd {
    const hc_causal_conv_desc* d;
    const hc_rows *x, *y;
    const float *w, *bias;
    const void* state_in;
    void* state_out;
    const int* lens;
    cudaStream_t st;
    template <typename T, int V, int K, int ACT> hc_status operator()() const {
        const CcShape s = cc_shape(d, V);
        launch_next(cc_fwd_kernel<T, V, K, ACT>, dim3((unsigned)(s.B * s.blocks), cdiv(s.cv, s.ncol)), CC_THREADS, 0, st,
                    view<const T>(x), view<T>(y), w, bias, (const T*)state_in, (T*)state_out, lens, s);
        return launched("cc_fwd_kernel", st);
    }
};

struct CcBwd {
    const hc_causal_conv_desc* d;
    const hc_rows *x, *gy, *gx;
    const float *w, *bias;
    float *gw, *gb;
    const void *state_in, *gstate_out;
    void* gstate_in;
    const int* lens;
    float* part;
    cudaStream_t st;
    template <typename T, int V, int K, int ACT> hc_status operator()() const {
        const CcShape s = cc_shape(d, V);
        const unsigned nb = (unsigned)(s.B * s.blocks);
        launch_next(cc_bwd_kernel<T, V, K, ACT>, dim3(nb, cdiv(s.cv, s.ncol)), CC_THREADS, 0, st,
                    view<const T>(x), view<const T>(gy), gx ? view<T>(gx) : View<T>{nullptr, 0, 0}, w, bias,
                    (const T*)state_in, (const T*)gstate_out, (T*)gstate_in, part, lens, s);
        hc_status e = launched("cc_bwd_kernel", st);
        if (e || !part) return e;
        const int kd = K * s.D;
        return launch_column_totals(part, nb, gw, kd, gb, s.D, nullptr, 0, st);
    }
};

struct CcStep {
    const hc_causal_conv_desc* d;
    const hc_rows *x, *y;
    const float *w, *bias;
    void* state;
    cudaStream_t st;
    template <typename T, int V, int K, int ACT> hc_status operator()() const {
        const int cv = d->D / V;
        launch_next(cc_step_kernel<T, V, K, ACT>, cdiv((long long)d->B * cv, 128), 128, 0, st, view<const T>(x),
                    view<T>(y), w, bias, (T*)state, d->B, d->D, cv);
        return launched("cc_step_kernel", st);
    }
};

}  // namespace

}  // namespace hc

using namespace hc;

extern "C" {

hc_status hc_causal_conv_fwd(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                             const hc_rows* y, const void* state_in, void* state_out, const int* lens, void* stream) {
    if (!cc_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!cc_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!rows_in_ok(x, d->dtype, d->L) || !rows_out_ok(y, d->dtype, d->B, d->L, d->D) || rows_same(x, y) ||
        !f32_ok(w) || !f32_opt_ok(bias) || !ptr_al(state_in, 16) || !ptr_al(state_out, 16) ||
        (state_in && state_in == state_out) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    traced_begin((cudaStream_t)stream);
    const int v = CC_V;
    const bool vec = d->D % v == 0 && rows_vec(x, v) && rows_vec(y, v);
    return cc_dispatch(d, vec, CcFwd{d, x, y, w, bias, state_in, state_out, lens, (cudaStream_t)stream});
}

hc_status hc_causal_conv_workspace_size(const hc_causal_conv_desc* d, size_t* bytes) {
    if (!cc_desc_ok(d) || !bytes) return HC_ERR_INVALID_ARG;
    if (!cc_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = cc_part_bytes(d);
    return HC_OK;
}

hc_status hc_causal_conv_bwd(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                             const hc_rows* gy, const hc_rows* gx, float* gw, float* gb, const void* state_in,
                             const void* gstate_out, void* gstate_in, const int* lens, void* ws, size_t ws_bytes,
                             void* stream) {
    size_t need = 0;
    hc_status e = hc_causal_conv_workspace_size(d, &need);
    if (e) return e;
    if (gx && !gx->p) gx = nullptr;
    if (!rows_in_ok(x, d->dtype, d->L) || !rows_in_ok(gy, d->dtype, d->L) ||
        (gx && (!rows_out_ok(gx, d->dtype, d->B, d->L, d->D) || rows_same(gx, x) || rows_same(gx, gy))) || !f32_ok(w) ||
        !f32_opt_ok(bias) || !f32_opt_ok(gw) || !f32_opt_ok(gb) || !ptr_al(state_in, 16) || !ptr_al(gstate_out, 16) ||
        !ptr_al(gstate_in, 16) || (gstate_in && (gstate_in == gstate_out || gstate_in == state_in)) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    const bool params = gw || gb;
    if (params && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    const int v = CC_V;
    const bool vec = d->D % v == 0 && rows_vec(x, v) && rows_vec(gy, v) && (!gx || rows_vec(gx, v));
    return cc_dispatch(d, vec, CcBwd{d, x, gy, gx, w, bias, gw, gb, state_in, gstate_out, gstate_in, lens,
                                     params ? (float*)ws : nullptr, (cudaStream_t)stream});
}

hc_status hc_causal_conv_step(const hc_causal_conv_desc* d, const hc_rows* x, const float* w, const float* bias,
                              void* state, const hc_rows* y, void* stream) {
    if (!cc_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!cc_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!rows_in_ok(x, d->dtype) || !rows_out_ok(y, d->dtype, d->B, 1, d->D) || x->p == y->p || !f32_ok(w) ||
        !f32_opt_ok(bias) || !f32_ok(state))
        return HC_ERR_INVALID_ARG;
    traced_begin((cudaStream_t)stream);
    const int v = CC_V;
    // a row stride that one token does not use does not decide the width
    const hc_rows x1{x->p, x->batch, 0, x->dtype}, y1{y->p, y->batch, 0, y->dtype};
    const bool vec = d->D % v == 0 && rows_vec(&x1, v) && rows_vec(&y1, v);
    return cc_dispatch(d, vec, CcStep{d, &x1, &y1, w, bias, state, (cudaStream_t)stream});
}

}  // extern "C"
