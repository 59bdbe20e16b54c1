// scan_fwd.cu -- the forward pass of the selective scan (scan.cu).
#include "scan.cuh"

namespace hc {
namespace {

// A tile's rows are copied to shared memory while the tile before it is computed;
// the walk over them makes step sizes, step * u, D * u and silu(z), the recurrence
// reads those as channel pairs, and a second walk writes y.  224 x 1024 x 256 fp32,
// 16 states, saving the states: 396 us, 3.6 TB/s (1.4 GB), a third of the fp32
// pipe; 16384 x 512 bf16 in segments 58 us.  Bound by instruction issue with four
// blocks an SM (123 to 128 registers): half of the 160 instructions a channel and row
// are the walks', which are not packed as the recurrence is.
template <int NL> constexpr size_t fwd_smem() {
    using S = FwdTile<NL>;
    return sizeof(float) * (5 * S::PLANE + 2 * S::CT + 4 * SC_T * S::NP + 3 * S::PLANE);
}
template <int NL, int DT>
__global__ void __launch_bounds__(FwdTile<NL>::THREADS) scan_fwd_kernel(const __grid_constant__ ScanArgs a) {
    grid_begin();
    using S = FwdTile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);  // step sizes * log2 e
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
    f32x2 A[2][4], h[2][4];
    ld_rates(a, w.d0 + tc, n, tc, w.cn, A);
    if (a.segs > 1)
        ld_tile(a.carry + ((long long)w.bs * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc, w.cn, h);
    else
        ld_tile(a.h0 ? a.h0 + ((long long)w.b * a.Dm + w.d0 + tc) * a.N : nullptr, a.N, n, a.N, false, tc, w.cn, h);
    put_params<S>(a, w, bD);
    typename EltOf<DT>::type bc[S::BC];
    const auto start = [&](int t0) {
        const Walk<S> at;
        fetch<S, DT>(a, a.dt, w, at, t0, 0, raw);
        fetch<S, DT>(a, a.u, w, at, t0, 1, raw);
        if (gate) fetch<S, DT>(a, a.z, w, at, t0, 2, raw);
        fetch_bc<S, DT>(a, w, t0, bc);
    };
    const int live1 = w.live1();
    if (w.tile0 < live1) start(w.tile0 * SC_T);
    for (int tile = w.tile0; tile < live1; tile++) {
        const int t0 = tile * SC_T;
        cp_async_wait();
        __syncthreads();
        const Walk<S> at;
        if (at.on) {
            // every row's loads before the first row's stores
            float s[S::STEPS][4], x[S::STEPS][4], z[S::STEPS][4], D[4], bias[4];
            load_pack<float, 4>(bD + at.ec, bias);
            load_pack<float, 4>(bD + S::CT + at.ec, D);
#pragma unroll
            for (int i = 0; i < S::STEPS; i++) {
                get<S, DT>(raw, 0, at.er + i * S::ROWS, at.ec, s[i]);
                get<S, DT>(raw, 1, at.er + i * S::ROWS, at.ec, x[i]);
                if (gate) get<S, DT>(raw, 2, at.er + i * S::ROWS, at.ec, z[i]);
            }
#pragma unroll
            for (int i = 0; i < S::STEPS; i++) {
                const int t = at.er + i * S::ROWS, q = t * S::CT + at.ec;
                steps(a, t0 + t < w.len, s[i], bias, dl + q);
                float o[4];
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    o[k] = D[k] * x[i][k];
                    x[i][k] *= s[i][k];
                }
                store_pack<float, 4>(xs + q, x[i]);
                store_pack<float, 4>(us + q, o);
                if (gate) {
#pragma unroll
                    for (int k = 0; k < 4; k++) z[i][k] = silu_f(z[i][k]);
                    store_pack<float, 4>(gs + q, z[i]);
                }
            }
        }
        put_bc<S, DT>(bc, bc2);
        __syncthreads();
        if (tile + 1 < live1) start(t0 + SC_T);
        if (a.saved)
            st_tile(a.saved + (((long long)w.b * a.tiles + tile) * a.Dm + w.d0 + tc) * S::NP, S::NP, n, a.N, true, tc,
                        w.cn, h);
        // a row's sum over states follows the next row's multiply-adds: its shuffles
        // wait while there is other work, and its store does not hold up their loads
        f32x2 y[2], before[2];
#pragma unroll
        for (int t = 0; t < SC_T; t++) {
            f32x2 s[2], x[2], B[4], C[4];
            ld_pairs(dl + t * S::CT + tc, s);
            ld_pairs(xs + t * S::CT + tc, x);
            ld_dup(bc2 + t * S::NP + 4 * n, B);
            ld_dup(bc2 + (SC_T + t) * S::NP + 4 * n, C);
#pragma unroll
            for (int i = 0; i < 2; i++) {
                before[i] = y[i];
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    h[i][j] = fma2(decay2(s[i], A[i][j]), h[i][j], mul2(x[i], B[j]));
                    y[i] = j ? fma2(C[j], h[i][j], y[i]) : mul2(C[j], h[i][j]);
                }
            }
            if (t) put_lanes_sum<NL>(before, n, ys + (t - 1) * S::CT + tc);
        }
        put_lanes_sum<NL>(y, n, ys + (SC_T - 1) * S::CT + tc);
        __syncthreads();
        const int rows = min(SC_T, a.L - t0);
        const Walk<S> to;
        float o[S::STEPS][4], skip[S::STEPS][4], open[S::STEPS][4];
        if (to.on) {
#pragma unroll
            for (int i = 0; i < S::STEPS; i++) {
                const int q = (to.er + i * S::ROWS) * S::CT + to.ec;
                load_pack<float, 4>(ys + q, o[i]);
                load_pack<float, 4>(us + q, skip[i]);
                if (gate) load_pack<float, 4>(gs + q, open[i]);
            }
#pragma unroll
            for (int i = 0; i < S::STEPS; i++) {
                const int t = to.er + i * S::ROWS;
                const bool on = t0 + t < w.len;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    o[i][k] += skip[i][k];
                    if (gate) o[i][k] *= open[i][k];
                    if (!on) o[i][k] = 0.0f;
                }
                if (t < rows) put<DT>(out_row<DT>(a.y, w, t0, t), to.ec, w.cn, a.vec, o[i]);
            }
        }
    }
    // rows past the sequence's last tile
    const int end = min(w.tile1 * SC_T, a.L);
    const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const Walk<S> at;
    for (int t = live1 * SC_T + at.er; t < end && at.on; t += S::ROWS)
        put<DT>(out_row<DT>(a.y, w, t, 0), at.ec, w.cn, a.vec, zero);
    if (a.hT && w.seg == a.segs - 1)
        st_tile(a.hT + ((long long)w.b * a.Dm + w.d0 + tc) * a.N, a.N, n, a.N, false, tc, w.cn, h);
}

struct Launch {
    const ScanArgs& a;
    cudaStream_t st;
    template <int NL, int DT> hc_status run() {
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_fwd_kernel<NL, DT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)fwd_smem<NL>()) == cudaSuccess;
        });
        launch_next(scan_fwd_kernel<NL, DT>, (unsigned)a.B * a.segs * a.G * a.ctiles, FwdTile<NL>::THREADS,
                    fwd_smem<NL>(), st, a);
        return launched("scan_fwd_kernel", st);
    }
};

}  // namespace

hc_status launch_scan_fwd(const ScanArgs& a, cudaStream_t st) {
    Launch f{a, st};
    return scan_dispatch(a.N, a.dtype, f);
}

}  // namespace hc
