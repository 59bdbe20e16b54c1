// groupnorm.cu -- group norm with an activation on channels-last tensors
// [N][P][C], forward and backward (formulas: hc_mixer.h).
//
// Each pass is three launches: per-channel sums over chunks of pixels, the
// sums' combination per (image, group), and the elementwise result.  A thread
// keeps one vector of V channels for its whole chunk, so the parameters and
// sums of those channels stay in registers and every access is V adjacent
// elements.  The statistics of a chunk are a mean and a sum of squared
// deviations (deviations taken from the chunk's first pixel, so that a large
// common offset does not cancel), combined over chunks and channels in a
// fixed order.
#include "rows.cuh"

namespace hc {
namespace {

constexpr int GN_THREADS = 256;

// What a launch covers: thread (col, r) of a block takes channel vector
// blockIdx.z * ncol + col and pixels r, r + R, ... of chunk blockIdx.x.
struct GnShape {
    int N, P, C, Cg, G;
    int cv;      // channel vectors, C / V
    int ncol;    // of them per block
    int R;       // pixel rows per block
    int chunk;   // pixels per chunk
    int chunks;  // per image
};

// Sums the R per-thread values of each channel in row order.
template <int V>
__device__ __forceinline__ void gn_block_sum(float* sm, const GnShape& s, int col, int r, bool on, float (&a)[V]) {
    const int w = s.ncol * V;
    if (on) {
#pragma unroll
        for (int i = 0; i < V; i++) sm[r * w + col * V + i] = a[i];
    }
    __syncthreads();
    if (on && r == 0) {
        for (int k = 1; k < s.R; k++) {
#pragma unroll
            for (int i = 0; i < V; i++) a[i] += sm[k * w + col * V + i];
        }
    }
    __syncthreads();
}

// part[n][chunk][c] = (mean, sum of squared deviations) of the chunk's pixels.
template <typename T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_stats_kernel(View<const T> x, float2* __restrict__ part, GnShape s) {
    __shared__ float sm[GN_THREADS * V];
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = blockIdx.y;
    const bool on = r < s.R && cvec < s.cv;
    const long long p0 = (long long)blockIdx.x * s.chunk;
    const int cnt = (int)(s.P - p0 < s.chunk ? s.P - p0 : s.chunk);
    const T* xb = x.p + n * x.batch + p0 * x.row + (long long)cvec * V;
    float pivot[V], sum[V], sq[V];
#pragma unroll
    for (int i = 0; i < V; i++) pivot[i] = sum[i] = sq[i] = 0.0f;
    if (on) {
        load_pack<T, V>(xb, pivot);
#pragma unroll 4
        for (int p = r; p < cnt; p += s.R) {
            float v[V];
            load_pack<T, V>(xb + p * x.row, v);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float d = v[i] - pivot[i];
                sum[i] += d;
                sq[i] = fmaf(d, d, sq[i]);
            }
        }
    }
    gn_block_sum<V>(sm, s, col, r, on, sum);
    gn_block_sum<V>(sm, s, col, r, on, sq);
    if (on && r == 0) {
        float2* o = part + ((long long)n * s.chunks + blockIdx.x) * s.C + cvec * V;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float m = sum[i] / cnt;
            o[i] = make_float2(pivot[i] + m, fmaxf(0.0f, sq[i] - sum[i] * m));
        }
    }
}

__device__ __forceinline__ float gn_reduce(float v, float* red) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.0f;
    for (int k = 0; k < GN_THREADS / 32; k++) t += red[k];
    __syncthreads();
    return t;
}

// One block per (image, group): its chunks' and channels' means and squared
// deviations combined.
__global__ void __launch_bounds__(GN_THREADS) gn_combine_kernel(const float2* __restrict__ part, float eps,
                                                                float* __restrict__ mean, float* __restrict__ rstd,
                                                                GnShape s) {
    __shared__ float red[GN_THREADS / 32];
    const int n = blockIdx.x / s.G, g = blockIdx.x % s.G;
    const float2* pb = part + (long long)n * s.chunks * s.C + g * s.Cg;
    const int total = s.chunks * s.Cg;
    const int last = s.P - (s.chunks - 1) * s.chunk;  // pixels of the last chunk
    const float values = (float)s.P * s.Cg;
    float a = 0.0f;
    for (int q = threadIdx.x; q < total; q += GN_THREADS) {
        const int k = q / s.Cg;
        a += pb[(long long)k * s.C + (q - k * s.Cg)].x * (k == s.chunks - 1 ? last : s.chunk);
    }
    const float m = gn_reduce(a, red) / values;
    float b = 0.0f;
    for (int q = threadIdx.x; q < total; q += GN_THREADS) {
        const int k = q / s.Cg;
        const float2 e = pb[(long long)k * s.C + (q - k * s.Cg)];
        const float d = e.x - m;
        b += fmaf(d * d, (float)(k == s.chunks - 1 ? last : s.chunk), e.y);
    }
    b = gn_reduce(b, red);
    if (threadIdx.x == 0) {
        mean[blockIdx.x] = m;
        rstd[blockIdx.x] = 1.0f / sqrtf(b / values + eps);
    }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_apply_kernel(View<const T> x, View<T> y, const float* __restrict__ gamma,
                                                              const float* __restrict__ beta,
                                                              const float* __restrict__ mean,
                                                              const float* __restrict__ rstd, GnShape s) {
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = blockIdx.y;
    if (r >= s.R || cvec >= s.cv) return;
    const long long p0 = (long long)blockIdx.x * s.chunk;
    const int cnt = (int)(s.P - p0 < s.chunk ? s.P - p0 : s.chunk);
    const T* xb = x.p + n * x.batch + p0 * x.row + (long long)cvec * V;
    T* yb = y.p + n * y.batch + p0 * y.row + (long long)cvec * V;
    float m[V], a[V], b[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = cvec * V + i, g = n * s.G + c / s.Cg;
        m[i] = mean[g];
        a[i] = rstd[g] * gamma[c];
        b[i] = beta[c];
    }
#pragma unroll 4
    for (int p = r; p < cnt; p += s.R) {
        float v[V];
        load_pack<T, V>(xb + p * x.row, v);
#pragma unroll
        for (int i = 0; i < V; i++) v[i] = act_f<ACT>(fmaf(v[i] - m[i], a[i], b[i]));
        store_pack<T, V>(yb + p * y.row, v);
    }
}

// part[n][chunk][c] = (sum of g, sum of g * xhat) over the chunk's pixels,
// g = gy * act'(pre).
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_sums_kernel(View<const T> x, View<const T> gy,
                                                                 const float* __restrict__ gamma,
                                                                 const float* __restrict__ beta,
                                                                 const float* __restrict__ mean,
                                                                 const float* __restrict__ rstd,
                                                                 float2* __restrict__ part, GnShape s) {
    __shared__ float sm[GN_THREADS * V];
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = blockIdx.y;
    const bool on = r < s.R && cvec < s.cv;
    const long long p0 = (long long)blockIdx.x * s.chunk;
    const int cnt = (int)(s.P - p0 < s.chunk ? s.P - p0 : s.chunk);
    const T* xb = x.p + n * x.batch + p0 * x.row + (long long)cvec * V;
    const T* gb = gy.p + n * gy.batch + p0 * gy.row + (long long)cvec * V;
    float s1[V], s2[V];
#pragma unroll
    for (int i = 0; i < V; i++) s1[i] = s2[i] = 0.0f;
    if (on) {
        float m[V], rs[V], ga[V], be[V];
#pragma unroll
        for (int i = 0; i < V; i++) {
            const int c = cvec * V + i, g = n * s.G + c / s.Cg;
            m[i] = mean[g];
            rs[i] = rstd[g];
            ga[i] = gamma[c];
            be[i] = beta[c];
        }
#pragma unroll 2
        for (int p = r; p < cnt; p += s.R) {
            float v[V], w[V];
            load_pack<T, V>(xb + p * x.row, v);
            load_pack<T, V>(gb + p * gy.row, w);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float xh = (v[i] - m[i]) * rs[i];
                const float g = w[i] * act_d<ACT>(fmaf(xh, ga[i], be[i]));
                s1[i] += g;
                s2[i] = fmaf(g, xh, s2[i]);
            }
        }
    }
    gn_block_sum<V>(sm, s, col, r, on, s1);
    gn_block_sum<V>(sm, s, col, r, on, s2);
    if (on && r == 0) {
        float2* o = part + ((long long)n * s.chunks + blockIdx.x) * s.C + cvec * V;
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = make_float2(s1[i], s2[i]);
    }
}

// Blocks below N * G: the group's means of q and q * xhat (q = gamma * g).
// The others: 32 channels' parameter gradients over every image and chunk.
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_combine_kernel(const float2* __restrict__ part,
                                                                    const float* __restrict__ gamma,
                                                                    float2* __restrict__ gmean,
                                                                    float* __restrict__ ggamma,
                                                                    float* __restrict__ gbeta, GnShape s) {
    __shared__ float red[GN_THREADS / 32];
    __shared__ float2 col[GN_THREADS / 32][32];
    if ((int)blockIdx.x < s.N * s.G) {
        const int n = blockIdx.x / s.G, g = blockIdx.x % s.G;
        const float2* pb = part + (long long)n * s.chunks * s.C + g * s.Cg;
        const int total = s.chunks * s.Cg;
        float a = 0.0f, b = 0.0f;
        for (int q = threadIdx.x; q < total; q += GN_THREADS) {
            const int k = q / s.Cg, c = q - k * s.Cg;
            const float2 e = pb[(long long)k * s.C + c];
            const float ga = gamma[g * s.Cg + c];
            a = fmaf(ga, e.x, a);
            b = fmaf(ga, e.y, b);
        }
        a = gn_reduce(a, red);
        b = gn_reduce(b, red);
        const float values = (float)s.P * s.Cg;
        if (threadIdx.x == 0) gmean[blockIdx.x] = make_float2(a / values, b / values);
        return;
    }
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = (blockIdx.x - s.N * s.G) * 32 + lane;
    float2 t = make_float2(0.0f, 0.0f);
    if (c < s.C) {
        const long long rows = (long long)s.N * s.chunks;
#pragma unroll 4
        for (long long k = w; k < rows; k += GN_THREADS / 32) {
            const float2 e = part[k * s.C + c];
            t.x += e.x;
            t.y += e.y;
        }
    }
    col[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < s.C) {
        for (int k = 1; k < GN_THREADS / 32; k++) {
            t.x += col[k][lane].x;
            t.y += col[k][lane].y;
        }
        if (gbeta) gbeta[c] = t.x;
        if (ggamma) ggamma[c] = t.y;
    }
}

template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_apply_kernel(View<const T> x, View<const T> gy, View<T> gx,
                                                                  const float* __restrict__ gamma,
                                                                  const float* __restrict__ beta,
                                                                  const float* __restrict__ mean,
                                                                  const float* __restrict__ rstd,
                                                                  const float2* __restrict__ gmean, GnShape s) {
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = blockIdx.y;
    if (r >= s.R || cvec >= s.cv) return;
    const long long p0 = (long long)blockIdx.x * s.chunk;
    const int cnt = (int)(s.P - p0 < s.chunk ? s.P - p0 : s.chunk);
    const T* xb = x.p + n * x.batch + p0 * x.row + (long long)cvec * V;
    const T* gb = gy.p + n * gy.batch + p0 * gy.row + (long long)cvec * V;
    T* ob = gx.p + n * gx.batch + p0 * gx.row + (long long)cvec * V;
    float m[V], rs[V], ga[V], be[V], mq[V], mqx[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        const int c = cvec * V + i, g = n * s.G + c / s.Cg;
        m[i] = mean[g];
        rs[i] = rstd[g];
        ga[i] = gamma[c];
        be[i] = beta[c];
        mq[i] = gmean[g].x;
        mqx[i] = gmean[g].y;
    }
#pragma unroll 2
    for (int p = r; p < cnt; p += s.R) {
        float v[V], w[V];
        load_pack<T, V>(xb + p * x.row, v);
        load_pack<T, V>(gb + p * gy.row, w);
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float xh = (v[i] - m[i]) * rs[i];
            const float q = w[i] * act_d<ACT>(fmaf(xh, ga[i], be[i])) * ga[i];
            v[i] = rs[i] * (q - mq[i] - xh * mqx[i]);
        }
        store_pack<T, V>(ob + p * gx.row, v);
    }
}

// About eight blocks an SM over all images, at least eight pixels a thread.
GnShape gn_shape(const hc_groupnorm_desc* d, int V) {
    GnShape s;
    s.N = d->N;
    s.P = d->P;
    s.C = d->C;
    s.G = d->groups;
    s.Cg = d->C / d->groups;
    s.cv = d->C / V;
    s.ncol = s.cv < GN_THREADS ? s.cv : GN_THREADS;
    s.R = GN_THREADS / s.ncol;
    const long long ctiles = cdiv(s.cv, s.ncol);
    long long chunks = cdiv(8LL * device_sm_count(), (long long)s.N * ctiles);
    const long long most = cdiv(s.P, 8LL * s.R);
    if (chunks > most) chunks = most;
    s.chunk = (int)cdiv(s.P, chunks);
    s.chunks = (int)cdiv(s.P, s.chunk);
    return s;
}

// Chunks an image at most, whatever the vector width: what the workspace is
// sized for.
long long gn_max_chunks(const hc_groupnorm_desc* d) {
    const long long a = gn_shape(d, 1).chunks;
    long long b = a;
    if (d->C % 4 == 0) b = gn_shape(d, 4).chunks > b ? gn_shape(d, 4).chunks : b;
    if (d->C % 8 == 0) b = gn_shape(d, 8).chunks > b ? gn_shape(d, 8).chunks : b;
    return b;
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

bool gn_desc_ok(const hc_groupnorm_desc* d) {
    return d && d->N > 0 && d->P > 0 && d->C > 0 && d->groups > 0 && d->C % d->groups == 0 && d->eps >= 0.0f &&
           (d->act == HC_PW_NONE || d->act == HC_PW_SILU || d->act == HC_PW_GELU) && dtype_ok(d->dtype);
}
// Launch limits: images on grid y, (image, group) and channel blocks on grid x.
bool gn_size_ok(const hc_groupnorm_desc* d) {
    return d->N <= 65535 && (long long)d->N * d->groups < (1LL << 30) && d->C <= (1 << 20);
}

// Calls f with the element type, vector width and activation of the call.
template <typename T, int V, typename F> hc_status gn_act(int act, F&& f) {
    if (act == HC_PW_SILU) return f.template operator()<T, V, HC_PW_SILU>();
    if (act == HC_PW_GELU) return f.template operator()<T, V, HC_PW_GELU>();
    return f.template operator()<T, V, HC_PW_NONE>();
}
template <typename F> hc_status gn_dispatch(int dt, bool vec, int act, F&& f) {
    if (dt == HC_DTYPE_F32) return vec ? gn_act<float, 4>(act, f) : gn_act<float, 1>(act, f);
    if (dt == HC_DTYPE_BF16) return vec ? gn_act<__nv_bfloat16, 8>(act, f) : gn_act<__nv_bfloat16, 1>(act, f);
    return vec ? gn_act<__half, 8>(act, f) : gn_act<__half, 1>(act, f);
}

struct GnFwd {
    const hc_groupnorm_desc* d;
    const hc_rows *x, *y;
    const float *gamma, *beta;
    float *mean, *rstd;
    float2* part;
    cudaStream_t st;
    template <typename T, int V, int ACT> hc_status operator()() const {
        const GnShape s = gn_shape(d, V);
        const dim3 grid(s.chunks, s.N, cdiv(s.cv, s.ncol));
        gn_stats_kernel<T, V><<<grid, GN_THREADS, 0, st>>>(view<const T>(x), part, s);
        hc_status e = launched("gn_stats_kernel", st);
        if (e) return e;
        gn_combine_kernel<<<s.N * s.G, GN_THREADS, 0, st>>>(part, d->eps, mean, rstd, s);
        if ((e = launched("gn_combine_kernel", st))) return e;
        gn_apply_kernel<T, V, ACT>
            <<<grid, GN_THREADS, 0, st>>>(view<const T>(x), view<T>(y), gamma, beta, mean, rstd, s);
        return launched("gn_apply_kernel", st);
    }
};

struct GnBwd {
    const hc_groupnorm_desc* d;
    const hc_rows *x, *gy, *gx;
    const float *gamma, *beta, *mean, *rstd;
    float *ggamma, *gbeta;
    float2 *part, *gmean;
    cudaStream_t st;
    template <typename T, int V, int ACT> hc_status operator()() const {
        const GnShape s = gn_shape(d, V);
        const dim3 grid(s.chunks, s.N, cdiv(s.cv, s.ncol));
        gn_bwd_sums_kernel<T, V, ACT>
            <<<grid, GN_THREADS, 0, st>>>(view<const T>(x), view<const T>(gy), gamma, beta, mean, rstd, part, s);
        hc_status e = launched("gn_bwd_sums_kernel", st);
        if (e) return e;
        const unsigned params = ggamma || gbeta ? cdiv(s.C, 32) : 0;
        gn_bwd_combine_kernel<<<s.N * s.G + params, GN_THREADS, 0, st>>>(part, gamma, gmean, ggamma, gbeta, s);
        if ((e = launched("gn_bwd_combine_kernel", st))) return e;
        gn_bwd_apply_kernel<T, V, ACT><<<grid, GN_THREADS, 0, st>>>(view<const T>(x), view<const T>(gy), view<T>(gx),
                                                                   gamma, beta, mean, rstd, gmean, s);
        return launched("gn_bwd_apply_kernel", st);
    }
};

}  // namespace
}  // namespace hc

using namespace hc;

extern "C" {

// Workspace: [part][mean, rstd of a forward pass that keeps none, or the group
// means of a backward pass].
hc_status hc_groupnorm_workspace_size(const hc_groupnorm_desc* d, int pass, size_t* bytes) {
    if (!gn_desc_ok(d) || pass < 0 || pass > 1 || !bytes) return HC_ERR_INVALID_ARG;
    if (!gn_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = up256(sizeof(float2) * d->N * gn_max_chunks(d) * d->C) + sizeof(float2) * d->N * d->groups;
    return HC_OK;
}

hc_status hc_groupnorm_fwd(const hc_groupnorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const hc_rows* y, float* mean, float* rstd, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    hc_status e = hc_groupnorm_workspace_size(d, 0, &need);
    if (e) return e;
    if (!rows_in_ok(x, d->dtype) || !rows_out_ok(y, d->dtype, d->N, d->P, d->C) || x->p == y->p || !f32_ok(gamma) ||
        !f32_ok(beta) || !f32_opt_ok(mean) || !f32_opt_ok(rstd))
        return HC_ERR_INVALID_ARG;
    if (!f32_ok(ws) || ws_bytes < need) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    const int v = d->dtype == HC_DTYPE_F32 ? 4 : 8;
    const bool vec = d->C % v == 0 && rows_vec(x, v) && rows_vec(y, v);
    float* keep = (float*)((char*)ws + up256(sizeof(float2) * d->N * gn_max_chunks(d) * d->C));
    return gn_dispatch(d->dtype, vec, d->act,
                       GnFwd{d, x, y, gamma, beta, mean ? mean : keep, rstd ? rstd : keep + (size_t)d->N * d->groups,
                             (float2*)ws, (cudaStream_t)stream});
}

hc_status hc_groupnorm_bwd(const hc_groupnorm_desc* d, const hc_rows* x, const float* gamma, const float* beta,
                           const float* mean, const float* rstd, const hc_rows* gy, const hc_rows* gx, float* ggamma,
                           float* gbeta, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    hc_status e = hc_groupnorm_workspace_size(d, 1, &need);
    if (e) return e;
    if (!rows_in_ok(x, d->dtype) || !rows_in_ok(gy, d->dtype) || !rows_out_ok(gx, d->dtype, d->N, d->P, d->C) ||
        x->p == gx->p || gy->p == gx->p || !f32_ok(gamma) || !f32_ok(beta) || !f32_ok(mean) || !f32_ok(rstd) ||
        !f32_opt_ok(ggamma) || !f32_opt_ok(gbeta))
        return HC_ERR_INVALID_ARG;
    if (!f32_ok(ws) || ws_bytes < need) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    const int v = d->dtype == HC_DTYPE_F32 ? 4 : 8;
    const bool vec = d->C % v == 0 && rows_vec(x, v) && rows_vec(gy, v) && rows_vec(gx, v);
    float2* gmean = (float2*)((char*)ws + up256(sizeof(float2) * d->N * gn_max_chunks(d) * d->C));
    return gn_dispatch(d->dtype, vec, d->act,
                       GnBwd{d, x, gy, gx, gamma, beta, mean, rstd, ggamma, gbeta, (float2*)ws, gmean,
                             (cudaStream_t)stream});
}

}  // extern "C"
