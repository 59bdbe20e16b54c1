// scan_bwd.cu -- the backward pass of the selective scan (scan.cu).
#include "scan.cuh"

namespace hc {
namespace {

// A block's tiles from the last to the first, each in two halves, the later one
// first.  A half's states are recomputed from its first state and kept in
// registers (H), with y and gC on the way, then the state's gradient runs back
// through them.  A tile's first state was saved; that of its later half is
// recomputed from it.  Half tiles keep a thread at 168 registers, three blocks an
// SM, with 28 to 112 bytes of it spilled; whole tiles take 255 and two.
//
// A state takes 5 fp32 operations and an exponential on the way up, 3 and one more
// in an earlier half's recomputation, 8 and one on the way down: 14.5 and 2.5 a row
// on average.  224 x 1024 x 256 fp32, 16 states: 1190 us, a third of the fp32 pipe
// and half of the issue slots; bound by the latency between dependent instructions
// with three warps a scheduler (a warp's 32 channels x 8 rows are about 3500
// instructions, a third of them the elementwise walks').
template <int NL> constexpr size_t bwd_smem() {
    using S = BwdTile<NL>;
    return sizeof(float) * (9 * S::PLANE + 2 * S::CT + 2 * S::ROWS * S::CT + 4 * SC_T * S::NP + S::W * SC_T * 2 * S::NP +
                            4 * S::PLANE + 8 * S::P * S::THREADS);
}
constexpr int HALF = SC_T / 2;
template <int NL, int DT>
__global__ void __launch_bounds__(BwdTile<NL>::THREADS, 384 / BwdTile<NL>::THREADS)
    scan_bwd_kernel(const __grid_constant__ ScanArgs a) {
    grid_begin();
    using S = BwdTile<NL>;
    using T = typename EltOf<DT>::type;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // step sizes * log2 e
    float* us = dl + S::PLANE;                  // u
    float* xs = us + S::PLANE;                  // step * u
    float* qs = xs + S::PLANE;                  // gy * silu(z)
    float* ps = qs + S::PLANE;                  // slope of the step size
    float* ws = ps + S::PLANE;                  // gy * silu'(z)
    float* ys = ws + S::PLANE;                  // C . h
    float* GB = ys + S::PLANE;                  // G . B
    float* EA = GB + S::PLANE;                  // E . A
    float* bD = EA + S::PLANE;                  // dt_bias, D
    float* sums = bD + 2 * S::CT;               // [ROWS][2][CT], each thread's gD and gdt_bias
    f32x2* bc2 = reinterpret_cast<f32x2*>(sums + 2 * S::ROWS * S::CT);
    float* red = reinterpret_cast<float*>(bc2 + 2 * SC_T * S::NP);  // [W][T][2][NP], the warps' gB and gC
    f32x2* gA = reinterpret_cast<f32x2*>(red + S::W * SC_T * 2 * S::NP);  // [P][4][threads], each thread's sums
    char* raw = reinterpret_cast<char*>(gA + 4 * S::P * S::THREADS);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int n = lane % NL, tc = warp * S::WC + lane / NL * 2 * S::P;
    const Where w(a, S::CT);
    const bool gate = a.z.p != nullptr;
    f32x2 A[S::P][4], G[S::P][4];
    ld_rates(a, w.d0 + tc, n, tc, w.cn, A);
    if (a.segs > 1)
        ld_tile(a.carry + ((long long)w.bs * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc, w.cn, G);
    else
        ld_tile(a.ghT ? a.ghT + ((long long)w.b * a.Dm + w.d0 + tc) * a.N : nullptr, a.N, n, a.N, false, tc, w.cn,
                    G);
#pragma unroll
    for (int i = 0; i < S::P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) gA[(4 * i + j) * S::THREADS + tid] = pk2(0.0f, 0.0f);
    put_params<S>(a, w, bD);
    for (int q = tid; q < 2 * S::ROWS * S::CT; q += S::THREADS) sums[q] = 0.0f;
    typename EltOf<DT>::type bc[S::BC];
    const auto start = [&](int t0) {
        const Walk<S> at;
        fetch<S, DT>(a, a.dt, w, at, t0, 0, raw);
        fetch<S, DT>(a, a.u, w, at, t0, 1, raw);
        fetch<S, DT>(a, a.gy, w, at, t0, 2, raw);
        if (gate) fetch<S, DT>(a, a.z, w, at, t0, 3, raw);
        fetch_bc<S, DT>(a, w, t0, bc);
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
            const Walk<S> at;
            if (at.on) {
                // every row's loads before the first row's stores
                float s[S::STEPS][4], u[S::STEPS][4], q[S::STEPS][4], z[S::STEPS][4], bias[4];
                load_pack<float, 4>(bD + at.ec, bias);
#pragma unroll
                for (int i = 0; i < S::STEPS; i++) {
                    const int t = at.er + i * S::ROWS;
                    get<S, DT>(raw, 0, t, at.ec, s[i]);
                    get<S, DT>(raw, 1, t, at.ec, u[i]);
                    get<S, DT>(raw, 2, t, at.ec, q[i]);
                    if (gate) get<S, DT>(raw, 3, t, at.ec, z[i]);
                }
#pragma unroll
                for (int i = 0; i < S::STEPS; i++) {
                    const int t = at.er + i * S::ROWS, c = t * S::CT + at.ec;
                    float p[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) p[k] = a.softplus ? sigmoid_f(s[i][k] + bias[k]) : 1.0f;
                    store_pack<float, 4>(ps + c, p);
                    steps(a, t0 + t < w.len, s[i], bias, dl + c);
                    store_pack<float, 4>(us + c, u[i]);
#pragma unroll
                    for (int k = 0; k < 4; k++) u[i][k] *= s[i][k];
                    store_pack<float, 4>(xs + c, u[i]);
                    if (gate) {
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float v = z[i][k], r = sigmoid_f(v);
                            p[k] = q[i][k] * r * fmaf(v, 1.0f - r, 1.0f);
                            q[i][k] *= v * r;
                        }
                        store_pack<float, 4>(ws + c, p);
                    }
                    store_pack<float, 4>(qs + c, q[i]);
                }
            }
            put_bc<S, DT>(bc, bc2);
            __syncthreads();
            if (tile > w.tile0) start(t0 - SC_T);
            const float* first = a.saved + (((long long)w.b * a.tiles + tile) * a.Dm + w.d0 + tc) * S::NP;
            if (tile > w.tile0) {  // the next tile's states on their way to L2
#pragma unroll
                for (int i = 0; i < 2 * S::P; i++)
                    if (tc + i < w.cn)
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(first - ((long long)a.Dm - i) * S::NP + 4 * n));
            }
            f32x2 h[S::P][4];
            ld_tile(first, S::NP, n, a.N, true, tc, w.cn, h);
#pragma unroll
            for (int t = 0; t < HALF; t++) {
                f32x2 s[S::P], x[S::P], B[4];
                ld_pairs(dl + t * S::CT + tc, s);
                ld_pairs(xs + t * S::CT + tc, x);
                ld_dup(bc2 + t * S::NP + 4 * n, B);
#pragma unroll
                for (int i = 0; i < S::P; i++)
#pragma unroll
                    for (int j = 0; j < 4; j++) h[i][j] = fma2(decay2(s[i], A[i][j]), h[i][j], mul2(x[i], B[j]));
            }
            // gA summed tile by tile: one running sum over all rows would lose more
            f32x2 ga[S::P][4];
#pragma unroll
            for (int i = 0; i < S::P; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) ga[i][j] = pk2(0.0f, 0.0f);
#pragma unroll 1
            for (int t1 = HALF; t1 >= 0; t1 -= HALF) {
                if (t1 == 0) ld_tile(first, S::NP, n, a.N, true, tc, w.cn, h);
                f32x2 H[HALF][S::P][4];  // the state before row t1 + t
                // a row's sums follow the next row's multiply-adds: their shuffles wait while there is other work,
                // and their stores do not hold up its loads
                f32x2 y[S::P], gc[4], y0[S::P], gc0[4];
#pragma unroll
                for (int t = 0; t < HALF; t++) {
                    const int r = t1 + t;
                    f32x2 s[S::P], x[S::P], q[S::P], B[4], C[4];
                    ld_pairs(dl + r * S::CT + tc, s);
                    ld_pairs(xs + r * S::CT + tc, x);
                    ld_pairs(qs + r * S::CT + tc, q);
                    ld_dup(bc2 + r * S::NP + 4 * n, B);
                    ld_dup(bc2 + (SC_T + r) * S::NP + 4 * n, C);
#pragma unroll
                    for (int i = 0; i < S::P; i++) {
                        y0[i] = y[i];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (!i) gc0[j] = gc[j];
                            H[t][i][j] = h[i][j];
                            h[i][j] = fma2(decay2(s[i], A[i][j]), h[i][j], mul2(x[i], B[j]));
                            y[i] = j ? fma2(C[j], h[i][j], y[i]) : mul2(C[j], h[i][j]);
                            gc[j] = i ? fma2(q[i], h[i][j], gc[j]) : mul2(q[i], h[i][j]);
                        }
                    }
                    if (t) {
                        put_lanes_sum<NL>(y0, n, ys + (r - 1) * S::CT + tc);
                        put_groups_sum<NL>(gc0, lane, red + ((warp * SC_T + r - 1) * 2 + 1) * S::NP + 4 * n);
                    }
                }
                put_lanes_sum<NL>(y, n, ys + (t1 + HALF - 1) * S::CT + tc);
                put_groups_sum<NL>(gc, lane, red + ((warp * SC_T + t1 + HALF - 1) * 2 + 1) * S::NP + 4 * n);
                // nothing of the way up is kept for the way down but H: the exponentials are taken again
                asm volatile("" ::: "memory");
                f32x2 gb[S::P], ea[S::P], gB[4], gb0[S::P], ea0[S::P], gB0[4];
#pragma unroll
                for (int t = HALF - 1; t >= 0; t--) {
                    const int r = t1 + t;
                    f32x2 s[S::P], x[S::P], q[S::P], B[4], C[4];
                    ld_pairs(dl + r * S::CT + tc, s);
                    ld_pairs(xs + r * S::CT + tc, x);
                    ld_pairs(qs + r * S::CT + tc, q);
                    ld_dup(bc2 + r * S::NP + 4 * n, B);
                    ld_dup(bc2 + (SC_T + r) * S::NP + 4 * n, C);
#pragma unroll
                    for (int i = 0; i < S::P; i++) {
                        gb0[i] = gb[i];
                        ea0[i] = ea[i];
#pragma unroll
                        for (int j = 0; j < 4; j++) {
                            if (!i) gB0[j] = gB[j];
                            const f32x2 g = fma2(q[i], C[j], G[i][j]);
                            gB[j] = i ? fma2(g, x[i], gB[j]) : mul2(g, x[i]);
                            gb[i] = j ? fma2(g, B[j], gb[i]) : mul2(g, B[j]);
                            G[i][j] = mul2(g, decay2(s[i], A[i][j]));
                            const f32x2 E = mul2(G[i][j], H[t][i][j]);
                            ea[i] = j ? fma2(E, A[i][j], ea[i]) : mul2(E, A[i][j]);
                            ga[i][j] = fma2(E, s[i], ga[i][j]);
                        }
                    }
                    if (t < HALF - 1) {
                        put_lanes_sum<NL>(gb0, n, GB + (r + 1) * S::CT + tc);
                        put_lanes_sum<NL>(ea0, n, EA + (r + 1) * S::CT + tc);
                        put_groups_sum<NL>(gB0, lane, red + (warp * SC_T + r + 1) * 2 * S::NP + 4 * n);
                    }
                }
                put_lanes_sum<NL>(gb, n, GB + t1 * S::CT + tc);
                put_lanes_sum<NL>(ea, n, EA + t1 * S::CT + tc);
                put_groups_sum<NL>(gB, lane, red + (warp * SC_T + t1) * 2 * S::NP + 4 * n);
            }
#pragma unroll
            for (int i = 0; i < S::P; i++)
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    f32x2* sum = gA + (4 * i + j) * S::THREADS + tid;
                    *sum = add2(ga[i][j], *sum);
                }
            __syncthreads();
        }
        const Walk<S> to;
#pragma unroll
        for (int i = 0; i < S::STEPS; i++) {
            const int t = to.er + i * S::ROWS, c = t * S::CT + to.ec;
            if (!to.on || t >= rows) break;
            float gu[4] = {0, 0, 0, 0}, gd[4] = {0, 0, 0, 0}, gz[4] = {0, 0, 0, 0};
            if (t0 + t < w.len) {
                float b[4], e[4], u[4], q[4], D[4], v[4];
                float* sum = sums + (t % S::ROWS) * 2 * S::CT + to.ec;
                load_pack<float, 4>(GB + c, b);
                load_pack<float, 4>(us + c, u);
                load_pack<float, 4>(qs + c, q);
                load_pack<float, 4>(bD + S::CT + to.ec, D);
                load_pack<float, 4>(dl + c, v);
#pragma unroll
                for (int k = 0; k < 4; k++) gu[k] = fmaf(b[k], v[k] * kLn2, D[k] * q[k]);
                load_pack<float, 4>(EA + c, e);
                load_pack<float, 4>(ps + c, v);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    gd[k] = fmaf(b[k], u[k], e[k]) * v[k];
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
            put<DT>(out_row<DT>(a.gu, w, t0, t), to.ec, w.cn, a.vec, gu);
            put<DT>(out_row<DT>(a.gdt, w, t0, t), to.ec, w.cn, a.vec, gd);
            if (gate) put<DT>(out_row<DT>(a.gz, w, t0, t), to.ec, w.cn, a.vec, gz);
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
                static_cast<T*>(o.p)[w.b * o.batch + (t0 + t) * o.row + w.g * a.N + k] = from_f<T>(v);
            }
        }
    }
    float* pb = a.part + (long long)w.bs * (a.N + 2) * a.Dm;
    f32x2 ga[S::P][4];
#pragma unroll
    for (int i = 0; i < S::P; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) ga[i][j] = mul2(gA[(4 * i + j) * S::THREADS + tid], pk2(kLn2, kLn2));
    st_tile(pb + (long long)(w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, ga);
    if (a.gh0 && w.seg == 0)
        st_tile(a.gh0 + ((long long)w.b * a.Dm + w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, G);
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

struct Launch {
    const ScanArgs& a;
    cudaStream_t st;
    template <int NL, int DT> hc_status run() {
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_bwd_kernel<NL, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)bwd_smem<NL>()) == cudaSuccess;
        });
        launch_next(scan_bwd_kernel<NL, DT>, (unsigned)a.B * a.segs * a.G * a.ctiles, BwdTile<NL>::THREADS,
                    bwd_smem<NL>(), st, a);
        return launched("scan_bwd_kernel", st);
    }
};

}  // namespace

hc_status launch_scan_bwd(const ScanArgs& a, cudaStream_t st) {
    Launch f{a, st};
    return scan_dispatch(a.N, a.dtype, f);
}

}  // namespace hc
