// scan_carry.cu -- the segments of a selective scan (scan.cu): every segment
// from a zero state, and their results joined.
#include "scan.cuh"

namespace hc {
namespace {

// A segment's state from a zero state.  REV false: the state itself, over
// x = step * u and B, rows upwards.  REV true: the state's gradient, over
// q = gy * silu(z) and C, rows downwards: G_{t-1} = exp(step_t A) (G_t + q_t C_t).
// 16384 x 512 bf16: 41 us, two thirds of the full pass, whose exponentials it takes
// first; bound by instruction issue.
template <int NL> constexpr size_t carry_smem() {
    using S = FwdTile<NL>;
    return sizeof(float) * (2 * S::PLANE + 2 * S::CT + 4 * SC_T * S::NP + 3 * S::PLANE);
}
template <int NL, int DT, bool REV>
__global__ void __launch_bounds__(FwdTile<NL>::THREADS) scan_carry_kernel(const __grid_constant__ ScanArgs a) {
    grid_begin();
    using S = FwdTile<NL>;
    extern __shared__ float4 sm4[];
    float* dl = reinterpret_cast<float*>(sm4);
    float* xs = dl + S::PLANE;
    float* bD = xs + S::PLANE;
    f32x2* bc2 = reinterpret_cast<f32x2*>(bD + 2 * S::CT);
    char* raw = reinterpret_cast<char*>(bc2 + 2 * SC_T * S::NP);
    const int lane = threadIdx.x & 31, n = lane % NL, tc = (threadIdx.x >> 5) * S::WC + lane / NL * 4;
    const Where w(a, S::CT);
    f32x2 A[2][4], h[2][4], sum[2];
    ld_rates(a, w.d0 + tc, n, tc, w.cn, A);
#pragma unroll
    for (int i = 0; i < 2; i++) {
        sum[i] = pk2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; j++) h[i][j] = sum[i];
    }
    put_params<S>(a, w, bD);
    typename EltOf<DT>::type bc[S::BC];
    const bool gate = REV && a.z.p;
    const auto start = [&](int t0) {
        const Walk<S> at;
        fetch<S, DT>(a, a.dt, w, at, t0, 0, raw);
        fetch<S, DT>(a, REV ? a.gy : a.u, w, at, t0, 1, raw);
        if (gate) fetch<S, DT>(a, a.z, w, at, t0, 2, raw);
        fetch_bc<S, DT>(a, w, t0, bc);
    };
    const int tiles = w.live1() - w.tile0;
    const int first = REV ? w.tile0 + tiles - 1 : w.tile0, dir = REV ? -1 : 1;
    if (tiles > 0) start(first * SC_T);
    for (int k = 0; k < tiles; k++) {
        const int t0 = (first + dir * k) * SC_T;
        cp_async_wait();
        __syncthreads();
        const Walk<S> at;
        if (at.on) {
            float s[S::STEPS][4], x[S::STEPS][4], z[S::STEPS][4], bias[4];
            load_pack<float, 4>(bD + at.ec, bias);
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
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    if (!REV) x[i][k] *= s[i][k];
                    if (gate) x[i][k] *= silu_f(z[i][k]);
                }
                store_pack<float, 4>(xs + q, x[i]);
            }
        }
        put_bc<S, DT>(bc, bc2);
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
                    const f32x2 e = decay2(s[i], A[i][j]);
                    h[i][j] = REV ? mul2(e, fma2(x[i], B[j], h[i][j])) : fma2(e, h[i][j], mul2(x[i], B[j]));
                }
            }
        }
        __syncthreads();
    }
    const long long d = (long long)w.bs * a.Dm + w.d0 + tc;
    st_tile(a.carry + d * S::NP, S::NP, n, a.N, true, tc, w.cn, h);
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
// takes SJ_THREADS / R adjacent states of a sequence and R rows of threads, each
// with an equal run of segments: each run is joined, the runs' results are
// joined in order through shared memory, and each run is gone through again.
// Few segments take one row (no second walk's worth of work is saved), many as
// many rows as keep the walks short.
constexpr int SJ_THREADS = 256;  // 12 us for 228 segments of 512 channels x 16 states
template <bool REV, int R>
__global__ void __launch_bounds__(SJ_THREADS) scan_join_kernel(const __grid_constant__ ScanArgs a, int NP) {
    grid_begin();
    constexpr int S = SJ_THREADS / R;
    __shared__ float hs[R][S + 1], as[R][S + 1];
    const int col = threadIdx.x % S, r = threadIdx.x / S;
    const int b = blockIdx.y;
    const long long q = (long long)blockIdx.x * S + col;
    const bool on = q < (long long)a.Dm * NP;
    const int d = on ? (int)(q / NP) : 0, n = on ? (int)(q % NP) : 0;
    const float A = on && n < a.N ? a.A[(long long)d * a.N + n] : 0.0f;
    const int per = (a.segs + R - 1) / R, s0 = min(r * per, a.segs), s1 = min(s0 + per, a.segs);
    const long long hstep = REV ? -(long long)a.Dm * NP : (long long)a.Dm * NP, wstep = REV ? -a.Dm : a.Dm;
    const long long at = (long long)b * a.segs + (REV ? a.segs - 1 - s0 : s0);
    float* cp = a.carry + at * a.Dm * NP + (on ? q : 0);
    const float* dp = a.dsum + at * a.Dm + d;
    float h = 0.0f;
    if (R > 1) {
        float total = 0.0f;
#pragma unroll 4
        for (int k = 0; k < s1 - s0; k++) {
            const float w = dp[k * wstep];
            h = fmaf(ex2f(w * A), h, cp[k * hstep]);
            total += w;
        }
        hs[r][col] = h;
        as[r][col] = total;
        __syncthreads();
    }
    const float* first = REV ? a.ghT : a.h0;
    h = first && on && n < a.N ? first[((long long)b * a.Dm + d) * a.N + n] : 0.0f;
    if (R > 1)
        for (int k = 0; k < r; k++) h = fmaf(ex2f(as[k][col] * A), h, hs[k][col]);
    if (!on) return;
#pragma unroll 4
    for (int k = 0; k < s1 - s0; k++) {
        const float v = cp[k * hstep], w = dp[k * wstep];
        cp[k * hstep] = h;
        h = fmaf(ex2f(w * A), h, v);
    }
}
template <bool REV, int R> void join(const ScanArgs& a, int NP, cudaStream_t st) {
    launch_next(scan_join_kernel<REV, R>, dim3(cdiv((long long)a.Dm * NP, SJ_THREADS / R), a.B), SJ_THREADS, 0, st, a,
                NP);
}

template <bool REV> struct Launch {
    const ScanArgs& a;
    cudaStream_t st;
    template <int NL, int DT> hc_status run() {
        static std::atomic<unsigned long long> attr{0};
        once_per_device(attr, [] {
            return cudaFuncSetAttribute(scan_carry_kernel<NL, DT, REV>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)carry_smem<NL>()) == cudaSuccess;
        });
        launch_next(scan_carry_kernel<NL, DT, REV>, (unsigned)a.B * a.segs * a.G * a.ctiles, FwdTile<NL>::THREADS,
                    carry_smem<NL>(), st, a);
        const hc_status e = launched("scan_carry_kernel", st);
        if (e) return e;
        constexpr int NP = FwdTile<NL>::NP;
        if (a.segs <= 8)
            join<REV, 1>(a, NP, st);
        else
            join<REV, 8>(a, NP, st);
        return launched("scan_join_kernel", st);
    }
};

}  // namespace

hc_status launch_scan_carry(const ScanArgs& a, bool rev, cudaStream_t st) {
    Launch<false> up{a, st};
    Launch<true> down{a, st};
    return rev ? scan_dispatch(a.N, a.dtype, down) : scan_dispatch(a.N, a.dtype, up);
}

}  // namespace hc
