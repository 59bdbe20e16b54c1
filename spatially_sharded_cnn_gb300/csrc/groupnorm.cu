// groupnorm.cu -- group norm with an activation on channels-last tensors
// [N][P][C], forward and backward (formulas: hc_mixer.h).
//
// Bound by memory: x once in and y once out is the floor, and the statistics
// need x before the first y.  Maps that stay in L2 take one launch:
// every block sums a run of whole groups over a chunk of pixels, the blocks meet
// (a cooperative grid, or clusters where a slice has few chunks), each block
// joins its groups' chunks and reads its own chunk again, last pixels first, from
// L2.  Larger ones take three: sums over chunks of pixels, their combination per
// (image, group), and the elementwise result.
// A thread keeps one vector of V channels throughout, so the parameters and sums
// of those channels stay in registers and every access is V adjacent elements.
// Statistics are a mean and a sum of squared deviations (deviations taken from a
// first pixel, so that a large common offset does not cancel), combined over
// threads, blocks and channels in a fixed order.
#include <cooperative_groups.h>

#include "rows.cuh"

namespace cg = cooperative_groups;

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

// Pixels r, r + R, ... below n, U of them loaded before the first is used.  In
// the last turn the places past n load the last pixel again and are used with
// `in` false: still U loads at once, and no branch around the work, which would
// be laid out U times.
template <int U, typename L, typename F>
__device__ __forceinline__ void gn_walk(int r, int n, int R, L&& load, F&& use) {
    int p = r;
    for (; p + (U - 1) * R < n; p += U * R) {
        decltype(load(0)) q[U];
#pragma unroll
        for (int k = 0; k < U; k++) q[k] = load(p + k * R);
#pragma unroll
        for (int k = 0; k < U; k++) use(p + k * R, q[k], true);
    }
    if (p < n) {
        decltype(load(0)) q[U];
#pragma unroll
        for (int k = 0; k < U; k++) q[k] = load(min(p + k * R, n - 1));
#pragma unroll
        for (int k = 0; k < U; k++) use(p + k * R, q[k], p + k * R < n);
    }
}
// The same as one loop of clamped turns: half the code, which a kernel that goes
// through it a few times waits for more than for the loads.
template <int U, typename L, typename F>
__device__ __forceinline__ void gn_walk_short(int r, int n, int R, L&& load, F&& use) {
#pragma unroll 1
    for (int p = r; p < n; p += U * R) {
        decltype(load(0)) q[U];
#pragma unroll
        for (int k = 0; k < U; k++) q[k] = load(min(p + k * R, n - 1));
#pragma unroll
        for (int k = 0; k < U; k++) use(p + k * R, q[k], p + k * R < n);
    }
}
template <typename T, int V> struct Two {
    Pack<T, V> a, b;
};

// Whether the elementwise pass, which goes through the map backwards, finds this
// chunk in L2: `tensors` tensors from here to the map's end are what L2 keeps.
// The other chunks are read past the caches, these are not (7 x 131072 x 256 bf16
// forward 254 -> 249 us; with all of them past the caches 262: the elementwise
// pass then takes 169 us where it takes 154).
template <typename T> __device__ __forceinline__ bool gn_kept(const GnShape& s, int n, long long p0, int tensors) {
    return ((s.N - n) * (double)s.P - p0) * s.C * (sizeof(T) * tensors) < 100e6;
}

// The R rows of threads' two sums of every channel, to tot[0 | 1][ncol * V]: rows
// in order, in as many runs as there are threads for but no more than sixteen, then
// the runs in order.  (256 runs of one row, which a single channel has threads for,
// would be one sum of 256 in order: three times the rounding error.)
template <int V>
__device__ __forceinline__ void gn_block_sum(float2* sm, float (*tot)[GN_THREADS * V], int ncol, int R, int col, int r,
                                             bool on, const float (&a)[V], const float (&b)[V]) {
    const int w = ncol * V, tid = threadIdx.x;
    if (on) {
#pragma unroll
        for (int i = 0; i < V; i++) sm[r * w + col * V + i] = make_float2(a[i], b[i]);
    }
    __syncthreads();
    int rows = R;
    const int parts = w < GN_THREADS ? min(min(GN_THREADS / w, 16), R) : 1;
    if (parts > 1) {
        const int c = tid % w, q = tid / w;
        float2 t = make_float2(0.0f, 0.0f);
        if (q < parts)
            for (int k = q; k < R; k += parts) {
                const float2 e = sm[k * w + c];
                t.x += e.x;
                t.y += e.y;
            }
        __syncthreads();
        if (q < parts) sm[q * w + c] = t;
        __syncthreads();
        rows = parts;
    }
    for (int c = tid; c < w; c += GN_THREADS) {
        float2 t = sm[c];
        for (int k = 1; k < rows; k++) {
            const float2 e = sm[k * w + c];
            t.x += e.x;
            t.y += e.y;
        }
        tot[0][c] = t.x;
        tot[1][c] = t.y;
    }
    __syncthreads();
}

// part[n][chunk][c] = (mean, sum of squared deviations) of the chunk's pixels.
// Reads x once: 7 x 131072 x 256 bf16 (470 MB) in 99 us, 4.7 TB/s.
template <typename T, int V>
__global__ void __launch_bounds__(GN_THREADS) gn_stats_kernel(View<const T> x, float2* part, GnShape s) {
    grid_begin();
    __shared__ float2 sm[GN_THREADS * V];
    __shared__ float tot[2][GN_THREADS * V];
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
        const auto add = [&](int, const Pack<T, V>& q, bool in) {
            float v[V];
            unpack(q, v);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float d = in ? v[i] - pivot[i] : 0.0f;
                sum[i] += d;
                sq[i] = fmaf(d, d, sq[i]);
            }
        };
        if (gn_kept<T>(s, n, p0, 1))
            gn_walk<8>(r, cnt, s.R, [&](int p) { return load_raw<T, V>(xb + p * x.row); }, add);
        else
            gn_walk<8>(r, cnt, s.R, [&](int p) { return load_raw_stream<T, V>(xb + p * x.row); }, add);
    }
    gn_block_sum<V>(sm, tot, s.ncol, s.R, col, r, on, sum, sq);
    if (on && r == 0) {
        float2* o = part + ((long long)n * s.chunks + blockIdx.x) * s.C + cvec * V;
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float t = tot[0][col * V + i], m = t / cnt;
            o[i] = make_float2(pivot[i] + m, fmaxf(0.0f, tot[1][col * V + i] - t * m));
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
// deviations combined.  The means are summed as offsets from the first one: sums of
// the means themselves lose up to three units in the mean's last place.
__global__ void __launch_bounds__(GN_THREADS) gn_combine_kernel(const float2* part, float eps,
                                                                float* mean, float* rstd,
                                                                GnShape s) {
    grid_begin();
    __shared__ float red[GN_THREADS / 32];
    const int n = blockIdx.x / s.G, g = blockIdx.x % s.G;
    const float2* pb = part + (long long)n * s.chunks * s.C + g * s.Cg;
    const int total = s.chunks * s.Cg;
    const int last = s.P - (s.chunks - 1) * s.chunk;  // pixels of the last chunk
    const float values = (float)s.P * s.Cg, pivot = pb[0].x;
    float a = 0.0f;
    for (int q = threadIdx.x; q < total; q += GN_THREADS) {
        const int k = q / s.Cg;
        a = fmaf(pb[(long long)k * s.C + (q - k * s.Cg)].x - pivot, (float)(k == s.chunks - 1 ? last : s.chunk), a);
    }
    const float m = pivot + gn_reduce(a, red) / values;
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

// y = act((x - mean) * (rstd * gamma) + beta): the same map read again and y
// written, 940 MB in 154 us, 6.1 TB/s; bound by memory.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_apply_kernel(View<const T> x, View<T> y, const float* gamma,
                                                              const float* beta,
                                                              const float* mean,
                                                              const float* rstd, GnShape s) {
    grid_begin();
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = s.N - 1 - blockIdx.y;
    if (r >= s.R || cvec >= s.cv) return;
    const long long p0 = (long long)(s.chunks - 1 - blockIdx.x) * s.chunk;  // what L2 still holds first
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
    gn_walk<4>(r, cnt, s.R, [&](int p) { return load_raw_last<T, V>(xb + p * x.row); },
               [&](int p, const Pack<T, V>& q, bool in) {
                   float v[V];
                   unpack(q, v);
#pragma unroll
                   for (int i = 0; i < V; i++) v[i] = act_f<ACT>(fmaf(v[i] - m[i], a[i], b[i]));
                   if (in) store_pack_last<T, V>(yb + p * y.row, v);
               });
}

// part[n][chunk][c] = (sum of g, sum of g * xhat) over the chunk's pixels,
// g = gy * act'(pre).  7 x 65536 x 256 fp32: x and gy, 940 MB, in 177 us, 5.3 TB/s.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_sums_kernel(View<const T> x, View<const T> gy,
                                                                 const float* gamma,
                                                                 const float* beta,
                                                                 const float* mean,
                                                                 const float* rstd,
                                                                 float2* part, GnShape s) {
    grid_begin();
    __shared__ float2 sm[GN_THREADS * V];
    __shared__ float tot[2][GN_THREADS * V];
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
        const auto add = [&](int, const Two<T, V>& q, bool in) {
            float v[V], w[V];
            unpack(q.a, v);
            unpack(q.b, w);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float xh = (v[i] - m[i]) * rs[i];
                const float g = (in ? w[i] : 0.0f) * act_d<ACT>(fmaf(xh, ga[i], be[i]));
                s1[i] += g;
                s2[i] = fmaf(g, xh, s2[i]);
            }
        };
        if (gn_kept<T>(s, n, p0, 2))
            gn_walk<4>(r, cnt, s.R, [&](int p) {
                return Two<T, V>{load_raw<T, V>(xb + p * x.row), load_raw<T, V>(gb + p * gy.row)};
            }, add);
        else
            gn_walk<4>(r, cnt, s.R, [&](int p) {
                return Two<T, V>{load_raw_stream<T, V>(xb + p * x.row), load_raw_stream<T, V>(gb + p * gy.row)};
            }, add);
    }
    gn_block_sum<V>(sm, tot, s.ncol, s.R, col, r, on, s1, s2);
    if (on && r == 0) {
        float2* o = part + ((long long)n * s.chunks + blockIdx.x) * s.C + cvec * V;
#pragma unroll
        for (int i = 0; i < V; i++) o[i] = make_float2(tot[0][col * V + i], tot[1][col * V + i]);
    }
}

// Blocks below nn * G: the group's means of q and q * xhat (q = gamma * g).
// The others: a few channels' parameter gradients over every image and chunk,
// thread rows taking every so many of them.
constexpr int GN_PARAM_CHANNELS = 8;
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_combine_kernel(const float2* part,
                                                                    const float* gamma,
                                                                    float2* gmean,
                                                                    float* ggamma,
                                                                    float* gbeta, GnShape s) {
    grid_begin();
    __shared__ float red[GN_THREADS / 32];
    __shared__ float2 col[GN_THREADS / GN_PARAM_CHANNELS][GN_PARAM_CHANNELS + 1];
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
    constexpr int CH = GN_PARAM_CHANNELS, ROWS = GN_THREADS / CH;
    const int lane = threadIdx.x % CH, w = threadIdx.x / CH;
    const int c = (blockIdx.x - s.N * s.G) * CH + lane;
    float2 t = make_float2(0.0f, 0.0f);
    if (c < s.C) {
        const long long rows = (long long)s.N * s.chunks;
#pragma unroll 8
        for (long long k = w; k < rows; k += ROWS) {
            const float2 e = part[k * s.C + c];
            t.x += e.x;
            t.y += e.y;
        }
    }
    col[w][lane] = t;
    __syncthreads();
    if (w == 0 && c < s.C) {
        for (int k = 1; k < ROWS; k++) {
            t.x += col[k][lane].x;
            t.y += col[k][lane].y;
        }
        if (gbeta) gbeta[c] = t.x;
        if (ggamma) ggamma[c] = t.y;
    }
}

// gx = rstd * (q - mean(q) - xhat * mean(q * xhat)), q = gamma * g: x and gy again
// and gx, 1410 MB at the same size in 215 us, 6.6 TB/s; bound by memory.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS) gn_bwd_apply_kernel(View<const T> x, View<const T> gy, View<T> gx,
                                                                  const float* gamma,
                                                                  const float* beta,
                                                                  const float* mean,
                                                                  const float* rstd,
                                                                  const float2* gmean, GnShape s) {
    grid_begin();
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const int cvec = blockIdx.z * s.ncol + col, n = s.N - 1 - blockIdx.y;
    if (r >= s.R || cvec >= s.cv) return;
    const long long p0 = (long long)(s.chunks - 1 - blockIdx.x) * s.chunk;  // what L2 still holds first
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
    gn_walk<4>(r, cnt, s.R,
               [&](int p) {
                   return Two<T, V>{load_raw_last<T, V>(xb + p * x.row), load_raw_last<T, V>(gb + p * gy.row)};
               },
               [&](int p, const Two<T, V>& q, bool in) {
                   float v[V], w[V];
                   unpack(q.a, v);
                   unpack(q.b, w);
#pragma unroll
                   for (int i = 0; i < V; i++) {
                       const float xh = (v[i] - m[i]) * rs[i];
                       const float e = w[i] * act_d<ACT>(fmaf(xh, ga[i], be[i])) * ga[i];
                       v[i] = rs[i] * (e - mq[i] - xh * mqx[i]);
                   }
                   if (in) store_pack_last<T, V>(ob + p * gx.row, v);
               });
}

// ---- one launch: every block at a (run of whole groups, chunk of pixels) ----

constexpr int GN_CLUSTER = 8;

struct GnGrid {
    int N, P, C, Cg, G;
    int cv;      // channel vectors of the map
    int ncol;    // of a slice (the last may have fewer)
    int R;       // pixel rows a block
    int slices;  // per image
    int chunk;   // pixels of a chunk
    int chunks;  // per image
};

// Where a block works: channels c0 .. c0 + chans of the slice, pixels p0 .. p0 + cnt.
struct GnWhere {
    int img, chunk, cols, c0, chans, groups, g0, p0, cnt;
    __device__ __forceinline__ GnWhere(const GnGrid& s, int V) {
        // the chunks of a slice are neighbours: they can be a cluster
        chunk = blockIdx.x % s.chunks;
        const int q = blockIdx.x / s.chunks, slice = q % s.slices;
        img = q / s.slices;
        const int v0 = slice * s.ncol;
        cols = min(s.ncol, s.cv - v0);
        c0 = v0 * V;
        chans = cols * V;
        g0 = c0 / s.Cg;
        groups = chans / s.Cg;
        p0 = chunk * s.chunk;
        cnt = pixels(s, chunk);
    }
    static __device__ __forceinline__ int pixels(const GnGrid& s, int k) { return min(s.chunk, s.P - k * s.chunk); }
};

// The blocks of a slice meet: a cluster, where they are few, else with the grid.
__device__ __forceinline__ void gn_meet(const GnGrid& s) {
    if (s.chunks <= GN_CLUSTER) {
        __threadfence();
        cg::this_cluster().sync();
    } else {
        cg::this_grid().sync();
    }
}

__device__ __forceinline__ float warp_sum(float v) {
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums f(chunk, group) over an image's chunks for each of `groups` groups, to
// out[group]: as many threads a group as the block has for it (each every so
// many chunks), then those in order.
template <typename F> __device__ __forceinline__ void gn_join(float2* sm, int groups, int chunks, float2* out, F&& f) {
    const int tid = threadIdx.x;
    const int parts = groups < GN_THREADS ? min(GN_THREADS / groups, chunks) : 1;
    for (int g0 = 0; g0 < groups; g0 += GN_THREADS) {
        const int n = min(groups - g0, GN_THREADS), g = g0 + tid % n, q = tid / n;
        float2 t = make_float2(0.0f, 0.0f);
        if (q < parts) {
#pragma unroll 8
            for (int k = q; k < chunks; k += parts) {
                const float2 e = f(k, g);
                t.x += e.x;
                t.y += e.y;
            }
        }
        if (q < parts) sm[q * n + g - g0] = t;
        __syncthreads();
        if (tid < n) {
            t = sm[tid];
            for (int k = 1; k < parts; k++) {
                t.x += sm[k * n + tid].x;
                t.y += sm[k * n + tid].y;
            }
            out[g0 + tid] = t;
        }
        __syncthreads();
    }
}
// Group of each of a vector's channels c .. c + V - 1.
template <int V, typename F> __device__ __forceinline__ void gn_groups(int c, int Cg, F&& f) {
    int g = c / Cg, left = Cg - (c - g * Cg);
#pragma unroll
    for (int i = 0; i < V; i++) {
        f(i, g);
        if (--left == 0) {
            g++;
            left = Cg;
        }
    }
}

// part[image][chunk][group] = (mean, squared deviations) of the chunk's pixels.
// 512 x 256 bf16: 6.5 us a call; bound by its launch, two dependent reads and the
// meeting (1.2 us for a cooperative grid).
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS, 3) gn_grid_kernel(View<const T> x, View<T> y, const float* gamma,
                                                                const float* beta, float eps,
                                                                float* mean, float* rstd,
                                                                float2* part, GnGrid s) {
    grid_begin();
    __shared__ float2 sm[GN_THREADS * V];
    __shared__ float tot[2][GN_THREADS * V];
    __shared__ float2 stat[GN_THREADS * V];
    float2* join = reinterpret_cast<float2*>(tot);  // free once the block's groups are joined
    const GnWhere w(s, V);
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const bool on = r < s.R && col < w.cols;
    const int c = col * V, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float ga[V], be[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        ga[i] = on ? gamma[w.c0 + c + i] : 0.0f;
        be[i] = on ? beta[w.c0 + c + i] : 0.0f;
    }
    const int n = w.img;
    const T* xb = x.p + n * x.batch + w.p0 * x.row + w.c0 + c;
    float pivot[V], sum[V], sq[V];
#pragma unroll
    for (int i = 0; i < V; i++) pivot[i] = sum[i] = sq[i] = 0.0f;
    if (on) {
        load_pack<T, V>(xb, pivot);
        gn_walk_short<2>(r, w.cnt, s.R, [&](int p) { return load_raw<T, V>(xb + p * x.row); },
                   [&](int, const Pack<T, V>& q, bool in) {
                       float v[V];
                       unpack(q, v);
#pragma unroll
                       for (int i = 0; i < V; i++) {
                           const float d = in ? v[i] - pivot[i] : 0.0f;
                           sum[i] += d;
                           sq[i] = fmaf(d, d, sq[i]);
                       }
                   });
    }
    gn_block_sum<V>(sm, tot, s.ncol, s.R, col, r, on, sum, sq);
    if (on && r == 0) {
#pragma unroll
        for (int i = 0; i < V; i++) {
            const float t = tot[0][c + i], m = t / w.cnt;
            tot[0][c + i] = pivot[i] + m;
            tot[1][c + i] = fmaxf(0.0f, tot[1][c + i] - t * m);
        }
    }
    __syncthreads();
    // a warp a group: its channels joined
    for (int g = warp; g < w.groups; g += GN_THREADS / 32) {
        float m = 0.0f, q = 0.0f;
        for (int k = lane; k < s.Cg; k += 32) m += tot[0][g * s.Cg + k];
        m = warp_sum(m) / s.Cg;
        for (int k = lane; k < s.Cg; k += 32) {
            const float d = tot[0][g * s.Cg + k] - m;
            q += fmaf(d * d, (float)w.cnt, tot[1][g * s.Cg + k]);
        }
        q = warp_sum(q);
        if (lane == 0) part[((long long)n * s.chunks + w.chunk) * s.G + w.g0 + g] = make_float2(m, q);
    }
    gn_meet(s);
    // its groups' chunks joined: the means (as offsets from the first chunk's, which keeps their last bits), then
    // the squared deviations from them
    const float2* p = part + (long long)n * s.chunks * s.G + w.g0;
    gn_join(sm, w.groups, s.chunks, stat, [&](int k, int g) {
        return make_float2((p[(long long)k * s.G + g].x - p[g].x) * w.pixels(s, k), 0.0f);
    });
    const float over = 1.0f / s.P, values = (float)s.P * s.Cg;
    gn_join(sm, w.groups, s.chunks, join, [&](int k, int g) {
        const float2 e = p[(long long)k * s.G + g];
        const float d = e.x - (p[g].x + stat[g].x * over);
        return make_float2(fmaf(d * d, (float)w.pixels(s, k) * s.Cg, e.y), 0.0f);
    });
    for (int g = threadIdx.x; g < w.groups; g += GN_THREADS) {
        const float m = p[g].x + stat[g].x * over, rs = 1.0f / sqrtf(join[g].x / values + eps);
        stat[g] = make_float2(m, rs);
        if (w.chunk == 0) {
            if (mean) mean[n * s.G + w.g0 + g] = m;
            if (rstd) rstd[n * s.G + w.g0 + g] = rs;
        }
    }
    __syncthreads();
    if (on) {
        float m[V], a[V];
        gn_groups<V>(c, s.Cg, [&](int i, int g) {
            m[i] = stat[g].x;
            a[i] = stat[g].y * ga[i];
        });
        T* yb = y.p + n * y.batch + w.p0 * y.row + w.c0 + c;
        // the pixels read last, which L2 still holds, first
        const int top = w.cnt - 1;
        gn_walk_short<2>(r, w.cnt, s.R, [&](int p) { return load_raw_last<T, V>(xb + (top - p) * x.row); },
                   [&](int p, const Pack<T, V>& q, bool in) {
                       float v[V];
                       unpack(q, v);
#pragma unroll
                       for (int i = 0; i < V; i++) v[i] = act_f<ACT>(fmaf(v[i] - m[i], a[i], be[i]));
                       if (in) store_pack_last<T, V>(yb + (top - p) * y.row, v);
                   });
    }
}

// part[image][chunk][group] = the chunk's sums of q and q * xhat;
// param[image][chunk][2][C] = those of g and g * xhat.  Forward and backward of
// 3 x 10961 x 120 bf16 with GELU: 37 us.
template <typename T, int V, int ACT>
__global__ void __launch_bounds__(GN_THREADS, 2) gn_bwd_grid_kernel(View<const T> x, View<const T> gy, View<T> gx,
                                                                    const float* gamma,
                                                                    const float* beta,
                                                                    const float* mean,
                                                                    const float* rstd, float2* part,
                                                                    float* param, GnGrid s) {
    grid_begin();
    __shared__ float2 sm[GN_THREADS * V];
    __shared__ float tot[2][GN_THREADS * V];
    float2* stat = reinterpret_cast<float2*>(tot);  // free once the block's groups are joined
    const GnWhere w(s, V);
    const int col = threadIdx.x % s.ncol, r = threadIdx.x / s.ncol;
    const bool on = r < s.R && col < w.cols;
    const int c = col * V, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float ga[V], be[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        ga[i] = on ? gamma[w.c0 + c + i] : 0.0f;
        be[i] = on ? beta[w.c0 + c + i] : 0.0f;
    }
    float* pb = param ? param + ((long long)w.img * s.chunks + w.chunk) * 2 * s.C + w.c0 : nullptr;
    const int n = w.img;
    const T* xb = x.p + n * x.batch + w.p0 * x.row + w.c0 + c;
    const T* gb = gy.p + n * gy.batch + w.p0 * gy.row + w.c0 + c;
    float m[V], rs[V];
    float s1[V], s2[V];
    gn_groups<V>(c, s.Cg, [&](int i, int g) {
        m[i] = on ? mean[n * s.G + w.g0 + g] : 0.0f;
        rs[i] = on ? rstd[n * s.G + w.g0 + g] : 0.0f;
        s1[i] = s2[i] = 0.0f;
    });
    if (on)
        gn_walk_short<2>(r, w.cnt, s.R,
                   [&](int p) {
                       return Two<T, V>{load_raw<T, V>(xb + p * x.row), load_raw<T, V>(gb + p * gy.row)};
                   },
                   [&](int, const Two<T, V>& q, bool in) {
                       float v[V], u[V];
                       unpack(q.a, v);
                       unpack(q.b, u);
#pragma unroll
                       for (int i = 0; i < V; i++) {
                           const float xh = (v[i] - m[i]) * rs[i];
                           const float g = (in ? u[i] : 0.0f) * act_d<ACT>(fmaf(xh, ga[i], be[i]));
                           s1[i] += g;
                           s2[i] = fmaf(g, xh, s2[i]);
                       }
                   });
    gn_block_sum<V>(sm, tot, s.ncol, s.R, col, r, on, s1, s2);
    for (int g = warp; g < w.groups; g += GN_THREADS / 32) {
        float a = 0.0f, b = 0.0f;
        for (int k = lane; k < s.Cg; k += 32) {
            const float ge = gamma[w.c0 + g * s.Cg + k];
            a = fmaf(ge, tot[0][g * s.Cg + k], a);
            b = fmaf(ge, tot[1][g * s.Cg + k], b);
        }
        a = warp_sum(a);
        b = warp_sum(b);
        if (lane == 0) part[((long long)n * s.chunks + w.chunk) * s.G + w.g0 + g] = make_float2(a, b);
    }
    if (pb)
        for (int k = threadIdx.x; k < w.chans; k += GN_THREADS) {
            pb[k] = tot[0][k];
            pb[s.C + k] = tot[1][k];
        }
    gn_meet(s);
    const float2* p = part + (long long)n * s.chunks * s.G + w.g0;
    gn_join(sm, w.groups, s.chunks, stat, [&](int k, int g) { return p[(long long)k * s.G + g]; });
    if (on) {
        const float over = 1.0f / ((float)s.P * s.Cg);
        float mq[V], mqx[V];
        gn_groups<V>(c, s.Cg, [&](int i, int g) {
            mq[i] = stat[g].x * over;
            mqx[i] = stat[g].y * over;
        });
        T* ob = gx.p + n * gx.batch + w.p0 * gx.row + w.c0 + c;
        const int top = w.cnt - 1;
        gn_walk_short<2>(r, w.cnt, s.R,
                   [&](int p) {
                       return Two<T, V>{load_raw_last<T, V>(xb + (top - p) * x.row),
                                        load_raw_last<T, V>(gb + (top - p) * gy.row)};
                   },
                   [&](int p, const Two<T, V>& q, bool in) {
                       float v[V], u[V];
                       unpack(q.a, v);
                       unpack(q.b, u);
#pragma unroll
                       for (int i = 0; i < V; i++) {
                           const float xh = (v[i] - m[i]) * rs[i];
                           const float e = u[i] * act_d<ACT>(fmaf(xh, ga[i], be[i])) * ga[i];
                           v[i] = rs[i] * (e - mq[i] - xh * mqx[i]);
                       }
                       if (in) store_pack_last<T, V>(ob + (top - p) * gx.row, v);
                   });
    }
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// SMs whose blocks can be there together: an imposed count (hc_set_sm_count) above
// the device's does not make more.
int gn_sms() {
    const int sms = device_sm_count();
    if (g_sm_override.load(std::memory_order_relaxed) <= 0) return sms;
    int dev = 0, there = 0;
    cudaGetDevice(&dev);
    if (cudaDeviceGetAttribute(&there, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) cudaGetLastError();
    return there > 0 && there < sms ? there : sms;
}

// The one-launch form's grid for kernels of `blocks` blocks an SM, or chunks = 0
// where the three launches take the call: maps that L2 does not keep between the
// two reads of `tensors` tensors (7 x 131072 x 256 bf16 image by image, a grid
// meeting each: 336 us, three launches 262), or a run of whole groups and whole
// vectors wider than a block's threads.  Slices of at least 64 bytes, a little
// wider where that makes them alike, and as many blocks as the GPU holds at once
// unless a thread would be left with under two pixels.  Up to GN_CLUSTER chunks a
// slice launch as clusters, which start 2 us sooner than a cooperative grid.
GnGrid gn_grid(const hc_groupnorm_desc* d, int V, int tensors, int blocks) {
    GnGrid s;
    s.N = d->N;
    s.P = d->P;
    s.C = d->C;
    s.G = d->groups;
    s.Cg = d->C / d->groups;
    s.cv = d->C / V;
    s.chunks = 0;
    const long long unit = s.Cg / gcd(s.Cg, V);  // vectors
    if (unit > GN_THREADS || (double)d->N * d->P * d->C * dtype_size(d->dtype) * tensors > 64e6) return s;
    const long long units = s.cv / unit;
    long long per = cdiv(64, unit * V * (long long)dtype_size(d->dtype));
    if (per > units) per = units;
    for (long long q = per; q <= 2 * per && q <= units; q++)
        if (units % q == 0) {
            per = q;
            break;
        }
    if (per * unit > GN_THREADS) per = GN_THREADS / unit;
    s.ncol = (int)(per * unit);
    s.R = GN_THREADS / s.ncol;
    s.slices = (int)cdiv(s.cv, s.ncol);
    const long long useful = cdiv(d->P, 2LL * s.R);
    long long chunks = (long long)blocks * gn_sms() / ((long long)s.slices * d->N);
    if (chunks > useful) chunks = useful;
    if (chunks < 1) return s;  // more (image, slice) pairs than blocks at once
    s.chunk = (int)cdiv(d->P, chunks);
    s.chunks = (int)cdiv(d->P, s.chunk);
    return s;
}
constexpr int GN_FWD_BLOCKS = 3, GN_BWD_BLOCKS = 2;  // the kernels' launch bounds

template <typename... P, typename... A>
void launch_grid(void (*k)(P...), const GnGrid& s, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)s.slices * s.chunks * s.N);
    cfg.blockDim = dim3(GN_THREADS);
    cfg.stream = st;
    cudaLaunchAttribute at[2] = {};
    if (s.chunks <= GN_CLUSTER) {
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = s.chunks;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[1].val.programmaticStreamSerializationAllowed = 1;
        cfg.numAttrs = 2;
    } else {
        at[0].id = cudaLaunchAttributeCooperative;
        at[0].val.cooperative = 1;
        cfg.numAttrs = 1;
    }
    cfg.attrs = at;
    cudaLaunchKernelEx(&cfg, k, P(args)...);
}

// About sixteen blocks an SM over all images, at least eight pixels a
// thread.  (7 x 65536 x 256 fp32 training step with 8, 12, 16, 24, 32 blocks: 697,
// 650, 654, 668, 677 us; 7 x 131072 x 256 bf16 forward: 269, 264, 261, 262, 269 us.)
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
    long long chunks = cdiv(16LL * device_sm_count(), s.N * ctiles);
    const long long most = cdiv(s.P, 8LL * s.R);
    if (chunks > most) chunks = most;
    s.chunk = (int)cdiv(s.P, chunks);
    s.chunks = (int)cdiv(s.P, s.chunk);
    return s;
}

// Bytes of the partial sums, the most that any vector width and pass takes.
size_t gn_part_bytes(const hc_groupnorm_desc* d) {
    size_t most = 0;
    for (int v : {1, 4, 8}) {
        if (d->C % v) continue;
        for (int tensors : {1, 2}) {
            const GnGrid g = gn_grid(d, v, tensors, tensors == 1 ? GN_FWD_BLOCKS : GN_BWD_BLOCKS);
            size_t b = sizeof(float2) * d->N * gn_shape(d, v).chunks * d->C;
            if (g.chunks) b = sizeof(float2) * (size_t)d->N * g.chunks * (d->groups + d->C);
            if (b > most) most = b;
        }
    }
    return most;
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
        const GnGrid one = gn_grid(d, V, 1, GN_FWD_BLOCKS);
        if (one.chunks) {
            launch_grid(gn_grid_kernel<T, V, ACT>, one, st, view<const T>(x), view<T>(y), gamma, beta, d->eps, mean, rstd,
                        part, one);
            return launched("gn_grid_kernel", st);
        }
        const GnShape s = gn_shape(d, V);
        const dim3 grid(s.chunks, s.N, cdiv(s.cv, s.ncol));
        launch_next(gn_stats_kernel<T, V>, grid, GN_THREADS, 0, st, view<const T>(x), part, s);
        hc_status e = launched("gn_stats_kernel", st);
        if (e) return e;
        launch_next(gn_combine_kernel, s.N * s.G, GN_THREADS, 0, st, part, d->eps, mean, rstd, s);
        if ((e = launched("gn_combine_kernel", st))) return e;
        launch_next(gn_apply_kernel<T, V, ACT>, grid, GN_THREADS, 0, st, view<const T>(x), view<T>(y), gamma, beta, mean,
                    rstd, s);
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
        const GnGrid one = gn_grid(d, V, 2, GN_BWD_BLOCKS);
        if (one.chunks) {
            float* param = ggamma || gbeta ? (float*)(part + (size_t)one.N * one.chunks * one.G) : nullptr;
            launch_grid(gn_bwd_grid_kernel<T, V, ACT>, one, st, view<const T>(x), view<const T>(gy), view<T>(gx), gamma,
                        beta, mean, rstd, part, param, one);
            const hc_status e = launched("gn_bwd_grid_kernel", st);
            if (e || !param) return e;
            return launch_column_totals(param, (long long)one.N * one.chunks, gbeta, one.C, ggamma, one.C, nullptr, 0,
                                        st);
        }
        const GnShape s = gn_shape(d, V);
        const dim3 grid(s.chunks, s.N, cdiv(s.cv, s.ncol));
        launch_next(gn_bwd_sums_kernel<T, V, ACT>, grid, GN_THREADS, 0, st, view<const T>(x), view<const T>(gy), gamma,
                    beta, mean, rstd, part, s);
        hc_status e = launched("gn_bwd_sums_kernel", st);
        if (e) return e;
        const unsigned params = ggamma || gbeta ? cdiv(s.C, GN_PARAM_CHANNELS) : 0;
        launch_next(gn_bwd_combine_kernel, s.N * s.G + params, GN_THREADS, 0, st, part, gamma, gmean, ggamma, gbeta, s);
        if ((e = launched("gn_bwd_combine_kernel", st))) return e;
        launch_next(gn_bwd_apply_kernel<T, V, ACT>, grid, GN_THREADS, 0, st, view<const T>(x), view<const T>(gy),
                    view<T>(gx), gamma, beta, mean, rstd, gmean, s);
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
    *bytes = up256(gn_part_bytes(d)) + sizeof(float2) * d->N * d->groups;
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
    float* keep = (float*)((char*)ws + up256(gn_part_bytes(d)));
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
    float2* gmean = (float2*)((char*)ws + up256(gn_part_bytes(d)));
    return gn_dispatch(d->dtype, vec, d->act,
                       GnBwd{d, x, gy, gx, gamma, beta, mean, rstd, ggamma, gbeta, (float2*)ws, gmean,
                             (cudaStream_t)stream});
}

}  // extern "C"
