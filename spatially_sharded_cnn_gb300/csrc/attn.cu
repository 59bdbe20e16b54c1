// attn.cu -- linear attention with a decay for each head: the join of segments, the form
// for one token, and the entry points (hc_linear_attn_*).
#include <math.h>

#include "attn.cuh"

namespace hc {
namespace {

// One thread an element of the state: carry[s - 1] becomes the state ahead of segment s.
// 32 cells' sums are read before the first is replaced (one after another, 32 segments took
// 16 us for a load's latency each).  Grid: (pairs, elements of a state, passes).
__global__ void __launch_bounds__(256) attn_join_kernel(AttnArgs a, int T) {
    grid_begin();
    const AttnPass& p = a.p[blockIdx.z];
    if (!p.keep) return;
    __shared__ AttnFade w[32];
    const int e = blockIdx.y * 256 + threadIdx.x, pair = blockIdx.x, size = p.Dk * p.Dv, cells = a.cells();
    const bool in = e < size;
    const int b = pair / a.H, h = pair - b * a.H;
    const int len = attn_len(a.lens, b, a.L), chunks = (len + T - 1) / T, part = chunks * T - len;
    const float ld = attn_log_decay(a.decay, h);
    float z = in && p.z0 ? p.z0[(long long)pair * size + e] : 0.0f;
    float* c = p.carry + (long long)pair * cells * size + e;
    int cell = 0, seg = 0;
    for (int s0 = 0; s0 < cells; s0 += 32) {
        float own[32];
#pragma unroll
        for (int i = 0; i < 32; i++) own[i] = in && s0 + i < cells ? c[(long long)(s0 + i) * size] : 0.0f;
        __syncthreads();
        if (threadIdx.x < 32 && s0 + (int)threadIdx.x < cells)
            w[threadIdx.x] = attn_cell_fade(ld, a, s0 + threadIdx.x, chunks, T, part, p.back);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 32; i++) {
            const int s = s0 + i;
            if (s >= cells) break;
            z = attn_faded(w[i], z, own[i]);
            if (++cell == a.split) {  // a segment ends
                cell = 0;
                if (in) c[(long long)seg++ * size] = z;
            }
        }
    }
}

// One token: a block a (sequence, head).  Thread (r, c) takes columns c * V .. of rows
// r, r + R, ...; bound by the states, read and written once.
template <typename T, int V>
__global__ void __launch_bounds__(256) attn_step_kernel(View<const T> q, View<const T> k, View<const T> v,
                                                        const float* decay, float* state, View<T> y, int H, int Dk,
                                                        int Dv, float scale) {
    grid_begin();
    __shared__ float sm[256 * V];
    const int pair = blockIdx.x, b = pair / H, h = pair - b * H;
    const int cols = (Dv + V - 1) / V, R = 256 / cols;
    const int r = threadIdx.x / cols, c = (threadIdx.x - r * cols) * V;
    const AttnFade w = attn_fade(attn_log_decay(decay, h));
    const T* qr = q.p + b * q.batch + (long long)h * Dk;
    const T* kr = k.p + b * k.batch + (long long)h * Dk;
    const T* vr = v.p + b * v.batch + (long long)h * Dv;
    float* z = state + (long long)pair * Dk * Dv + c;
    float acc[V], vf[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
        acc[i] = 0.0f;
        vf[i] = r < R ? to_f(vr[c + i]) : 0.0f;
    }
    if (r < R) {
#pragma unroll 4
        for (int d = r; d < Dk; d += R) {
            const float kf = to_f(kr[d]), qf = to_f(qr[d]);
            float s[V];
            load_pack<float, V>(z + (long long)d * Dv, s);
#pragma unroll
            for (int i = 0; i < V; i++) {
                s[i] = attn_faded(w, s[i], kf * vf[i]);
                acc[i] = fmaf(qf, s[i], acc[i]);
            }
            store_pack<float, V>(z + (long long)d * Dv, s);
        }
    }
#pragma unroll
    for (int i = 0; i < V; i++) sm[threadIdx.x * V + i] = acc[i];
    __syncthreads();
    for (int n = threadIdx.x; n < Dv; n += 256) {
        float t = 0.0f;
        for (int j = 0; j < R; j++) t += sm[j * cols * V + n];
        y.p[b * y.batch + (long long)h * Dv + n] = from_f<T>(scale * t);
    }
}

template <typename T>
hc_status attn_step(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                    const float* decay, float* state, const hc_rows* y, cudaStream_t st) {
    const dim3 grid((unsigned)((long long)d->B * d->H));
    if (d->Dv % 4 == 0)
        launch_next(attn_step_kernel<T, 4>, grid, dim3(256), 0, st, view<const T>(q), view<const T>(k),
                    view<const T>(v), decay, state, view<T>(y), d->H, d->Dk, d->Dv, d->scale);
    else
        launch_next(attn_step_kernel<T, 1>, grid, dim3(256), 0, st, view<const T>(q), view<const T>(k),
                    view<const T>(v), decay, state, view<T>(y), d->H, d->Dk, d->Dv, d->scale);
    return launched("attn_step_kernel", st);
}

bool attn_desc_ok(const hc_linear_attn_desc* d) {
    return d && d->B >= 1 && d->L >= 0 && d->H >= 1 && d->Dk >= 1 && d->Dv >= 1 && isfinite(d->scale) &&
           dtype_ok(d->dtype);
}
bool attn_size_ok(const hc_linear_attn_desc* d) {
    return d->Dk <= 128 && d->Dv <= 128 && d->L < 0x7fffffff - 256 && (long long)d->H * d->Dk <= 1 << 20 &&
           (long long)d->H * d->Dv <= 1 << 20 && (long long)d->B * d->H < 0x7fffffffLL / 3;
}

// Whether a call may run on the tensor cores, as far as its sizes say: where a chunk of 128
// rows costs less than the rows that there are in fp32.  Forward without states, us on the tensor
// cores : in fp32, 4096 sequences x 4 heads of 64: 337 : 296 of 8 rows, 339 : 375 of 16, 343 : 2143
// of 128; 1024 x 8 heads of 128: 413 : 647 of 8 rows; 64 x 4 heads of 32: 10.1 : 9.1 of 32 rows,
// 10.3 : 14.0 of 64.
bool attn_tc_sizes(const hc_linear_attn_desc* d) {
    const int D = d->Dk > d->Dv ? d->Dk : d->Dv;
    return d->dtype == HC_DTYPE_BF16 && d->Dk % 8 == 0 && d->Dv % 8 == 0 && d->L > (D > 64 ? 0 : D > 32 ? 8 : 32);
}
// And its rows: the copy engine wants 16-byte boundaries and strides that are not 0.
bool attn_tc_rows(const hc_linear_attn_desc* d, const hc_rows* r) {
    return ptr_al(r->p, 16) && (d->L <= 1 || (r->row > 0 && r->row % 8 == 0)) &&
           (d->B <= 1 || (r->batch > 0 && r->batch % 8 == 0));
}

struct Cut {
    int segs, per, split, cell_per;
};
// Segments of a sequence: as many as give the GPU enough blocks to fill it in launches of
// `passes` passes, two chunks each at least; then cells, so that the carry pass, which the last
// segments are no part of, fills it too.  In fp32 a batch with lengths is cut for twice the blocks,
// as those behind a sequence's end have nothing to do (once : twice, us; lengths evenly between 0
// and L; training of 5 x 1537 x 4 heads of 41 / 82 211 : 174, 8 x 1024 x 4 heads of 64 170 : 136, 5 x
// 1537 x 4 heads of 96 310 : 265; on the tensor cores 20 x 1500 x 4 heads of 64 109 : 135).
Cut attn_cut(const hc_linear_attn_desc* d, bool tc, bool bwd, bool ragged) {
    const int most = d->Dk > d->Dv ? d->Dk : d->Dv, least = d->Dk > d->Dv ? d->Dv : d->Dk;
    // (what registers and shared memory let an SM hold)
    const int per_sm = tc ? attn_wide(most) ? 1 : 2 : attn_fp32_per_sm(most, least), T = tc ? AT_TC : AT_T;
    // (on the tensor cores passes of another kernel are another launch)
    const int passes = bwd && (!tc || attn_wide(most) == attn_wide(least)) ? 3 : 1, kept = passes == 3 ? 2 : 1;
    const long long pairs = (long long)d->B * d->H, want = (long long)per_sm * device_sm_count();
    const int chunks = (int)(((long long)d->L + T - 1) / T);
    const long long blocks = ragged && !tc ? 2 * want : want;
    long long segs = pairs * passes < blocks ? blocks / (pairs * passes) : 1;
    if (segs > chunks / 2) segs = chunks / 2;
    if (segs < 1) segs = 1;
    const int per = (int)((chunks + segs - 1) / segs);
    Cut c = {per > 0 ? (chunks + per - 1) / per : 1, per, 1, per};
    if (c.segs > 1) {
        long long split = want / (pairs * kept * (c.segs - 1));
        if (split > per) split = per;
        if (split > 1) {
            c.cell_per = (int)((per + split - 1) / split);
            c.split = (per + c.cell_per - 1) / c.cell_per;
        }
    }
    return c;
}

size_t carry_floats(const hc_linear_attn_desc* d, const Cut& c) {
    return (size_t)d->B * d->H * (c.segs - 1) * c.split * d->Dk * d->Dv;
}

AttnArgs attn_args(const hc_linear_attn_desc* d, const float* decay, const int* lens, const Cut& c) {
    AttnArgs a = {};
    a.decay = decay;
    a.lens = lens;
    a.B = d->B;
    a.L = d->L;
    a.H = d->H;
    a.dtype = d->dtype;
    a.segs = c.segs;
    a.per = c.per;
    a.split = c.split;
    a.cell_per = c.cell_per;
    return a;
}

hc_status attn_run(const AttnArgs& a, bool tc, cudaStream_t st) {
    const auto launch = tc ? launch_attn_tc : launch_attn_fp32;
    hc_status e = HC_OK;
    if (a.segs > 1 && (e = launch(a, true, st))) return e;
    if (a.cells() > kFewCells && (e = launch_attn_join(a, tc ? AT_TC : AT_T, st))) return e;
    return launch(a, false, st);
}

}  // namespace

hc_status launch_attn_join(const AttnArgs& a, int T, cudaStream_t st) {
    const int size = a.p[0].Dk * a.p[0].Dv;  // the same for every pass
    launch_next(attn_join_kernel, dim3((unsigned)((long long)a.B * a.H), cdiv(size, 256), a.passes), dim3(256), 0, st, a,
                T);
    return launched("attn_join_kernel", st);
}

}  // namespace hc

using namespace hc;

extern "C" {

// Cells' sums: of S forward; of S and of G backward; whichever way the rows of the
// call let it run.
hc_status hc_linear_attn_workspace_size(const hc_linear_attn_desc* d, int pass, size_t* bytes) {
    if (!attn_desc_ok(d) || pass < 0 || pass > 1 || !bytes) return HC_ERR_INVALID_ARG;
    if (!attn_size_ok(d)) return HC_ERR_UNSUPPORTED;
    size_t n = 0;
    for (int way = 0; way < (attn_tc_sizes(d) ? 4 : 2); way++) {
        const bool tc = way > 1, ragged = way & 1;
        const size_t f = carry_floats(d, attn_cut(d, tc, false, ragged));
        const size_t b = pass ? 2 * carry_floats(d, attn_cut(d, tc, true, ragged)) : 0;
        n = n > f ? n : f;
        n = n > b ? n : b;
    }
    *bytes = n * sizeof(float);
    return HC_OK;
}

hc_status hc_linear_attn_fwd(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                             const float* log_decay, const hc_rows* y, const float* h0, float* hT, const int* lens,
                             void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    const hc_status e = hc_linear_attn_workspace_size(d, 0, &need);
    if (e) return e;
    if (!rows_in_ok(q, d->dtype, d->L) || !rows_in_ok(k, d->dtype, d->L) || !rows_in_ok(v, d->dtype, d->L) ||
        !rows_out_ok(y, d->dtype, d->B, d->L, (long long)d->H * d->Dv) || rows_same(y, q) || rows_same(y, k) ||
        rows_same(y, v) || !f32_opt_ok(log_decay) || !f32_opt_ok(h0) || !f32_opt_ok(hT) || (h0 && h0 == hT) ||
        !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    bool tc = attn_tc_sizes(d);
    for (const hc_rows* r : {q, k, v, y}) tc = tc && attn_tc_rows(d, r);
    AttnArgs a = attn_args(d, log_decay, lens, attn_cut(d, tc, false, lens));
    a.passes = 1;
    a.p[0] = {*q, *k, *v, *y, d->Dk, d->Dv, d->scale, d->scale, 1.0f, 0, h0, hT, d->Dv, 1,
              a.segs > 1 ? (float*)ws : nullptr, 1};
    return attn_run(a, tc, st);
}

hc_status hc_linear_attn_bwd(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                             const float* log_decay, const float* h0, const hc_rows* gy, const float* ghT,
                             const hc_rows* gq, const hc_rows* gk, const hc_rows* gv, float* gh0, const int* lens,
                             void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    const hc_status e = hc_linear_attn_workspace_size(d, 1, &need);
    if (e) return e;
    for (const hc_rows* r : {q, k, v, gy})
        if (!rows_in_ok(r, d->dtype, d->L)) return HC_ERR_INVALID_ARG;
    if (!rows_out_ok(gq, d->dtype, d->B, d->L, (long long)d->H * d->Dk) ||
        !rows_out_ok(gk, d->dtype, d->B, d->L, (long long)d->H * d->Dk) ||
        !rows_out_ok(gv, d->dtype, d->B, d->L, (long long)d->H * d->Dv) || !f32_opt_ok(log_decay) || !f32_opt_ok(h0) ||
        !f32_opt_ok(ghT) || !f32_opt_ok(gh0) || (ghT && ghT == gh0) || (h0 && h0 == gh0) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* o : {gq, gk, gv})
        for (const hc_rows* r : {q, k, v, gy})
            if (rows_same(o, r)) return HC_ERR_INVALID_ARG;
    if (rows_same(gq, gk) || rows_same(gq, gv) || rows_same(gk, gv)) return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    bool tc = attn_tc_sizes(d);
    for (const hc_rows* r : {q, k, v, gy, gq, gk, gv}) tc = tc && attn_tc_rows(d, r);
    const Cut cut = attn_cut(d, tc, true, lens);
    AttnArgs a = attn_args(d, log_decay, lens, cut);
    float *cs = nullptr, *cg = nullptr;
    if (a.segs > 1) {
        cs = (float*)ws;
        cg = cs + carry_floats(d, cut);
    }
    const float s = d->scale;
    // the states of gv's pass are those of gk's, transposed; S comes from k and v, whose
    // pass is not run: gq's takes S^T (v, k)
    const AttnPass pq = {*gy, *v, *k, *gq, d->Dv, d->Dk, s, s, 1.0f, 0, h0, nullptr, 1, d->Dv, cs, 1};
    const AttnPass pv = {*k, *q, *gy, *gv, d->Dk, d->Dv, s, 1.0f, s, 1, ghT, gh0, d->Dv, 1, cg, 1};
    const AttnPass pk = {*v, *gy, *q, *gk, d->Dv, d->Dk, s, 1.0f, s, 1, ghT, nullptr, 1, d->Dv, cg, 0};
    a.passes = 3;
    a.p[0] = pq;
    a.p[1] = pv;
    a.p[2] = pk;
    return attn_run(a, tc, st);
}

hc_status hc_linear_attn_step(const hc_linear_attn_desc* d, const hc_rows* q, const hc_rows* k, const hc_rows* v,
                              const float* log_decay, float* state, const hc_rows* y, void* stream) {
    if (!attn_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!attn_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!rows_in_ok(q, d->dtype) || !rows_in_ok(k, d->dtype) || !rows_in_ok(v, d->dtype) ||
        !rows_out_ok(y, d->dtype, d->B, 1, (long long)d->H * d->Dv) || rows_same(y, q) || rows_same(y, k) ||
        rows_same(y, v) || !f32_opt_ok(log_decay) || !f32_ok(state))
        return HC_ERR_INVALID_ARG;
    const cudaStream_t st = (cudaStream_t)stream;
    traced_begin(st);
    if (d->dtype == HC_DTYPE_F32) return attn_step<float>(d, q, k, v, log_decay, state, y, st);
    if (d->dtype == HC_DTYPE_BF16) return attn_step<__nv_bfloat16>(d, q, k, v, log_decay, state, y, st);
    return attn_step<__half>(d, q, k, v, log_decay, state, y, st);
}

}  // extern "C"
