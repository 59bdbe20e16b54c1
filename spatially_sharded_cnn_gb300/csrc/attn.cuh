// attn.cuh -- shared by the linear attention kernels (attn.cu, attn_fp32.cu, attn_tc.cu).
//
// One computation serves the forward pass and the three gradients.  A pass takes rows
// q, k ([Dk] a head) and v ([Dv]) and a state Z ([Dk][Dv]), and walks over the rows in
// chunks of T, forwards or backwards.  With w(n) = lambda^n, for rows i, j of a chunk
// whose first row that exists is lo (chunks end at the sequence's end, so the
// chunk with the first row may begin before it):
//   forwards   y_i = si sum_{j <= i} w(i-j) (q_i . k_j) v_j + sx w(i-lo+1) q_i Z
//              Z   <- w(T-lo) Z + su sum_j w(T-1-j) k_j v_j^T
//   backwards  y_i = si sum_{j >= i} w(j-i) (q_i . k_j) v_j + sx w(T-1-i) q_i Z
//              Z   <- w(T-lo) Z + su sum_j w(j-lo+1) k_j v_j^T
// Then, with the state S and the state's gradient G,
//   y  = forwards (q, k, v; S),              si = sx = scale, su = 1
//   gq = forwards (gy, v, k; S^T),           si = sx = scale, su = 1
//   gv = backwards(k, q, gy; G),             si = su = scale, sx = 1
//   gk = backwards(v, gy, q; G^T),           si = su = scale, sx = 1
// (a row j of the sum is then a later row, whose gradient it carries back).
//
// Where sequences times heads leave the GPU idle, a sequence's chunks are cut into
// segments, and the segments but the last into cells: every cell's own sum of k v^T (the
// carry pass), and then all segments at once, each from the state ahead of it, which it adds up
// from the cells, in order, where they are few, and finds joined (attn_join_kernel) where they
// are many.
#pragma once

#include "rows.cuh"

namespace hc {

constexpr float kLowDecay = -1e30f;  // stands for a log decay of minus infinity: 0 * it is 0

struct AttnPass {
    hc_rows q, k, v, y;
    int Dk, Dv;         // of this pass: the widths of q, k and of v, y
    float si, sx, su;
    int back;           // 1: backwards
    const float* z0;    // the state ahead of the first chunk, element (m, n) of pair p at p * Dk * Dv + m * zm + n * zn
    float* z1;          // where the state behind the last chunk goes, laid out so; NULL: nowhere
    int zm, zn;
    float* carry;       // cells' sums [pair][cell], laid out so; NULL: one segment
    int keep;           // the carry pass fills `carry` from this pass's k and v (su in them)
};
constexpr int kFewCells = 4;  // that a segment adds up itself (8 x 4096 x 8 heads of 128: a join of 2 took 20 us)

struct AttnArgs {
    AttnPass p[3];
    int passes;
    const float* decay;
    const int* lens;
    int B, L, H, dtype;
    int segs, per;         // segments of a sequence, chunks of a segment
    int split, cell_per;   // cells of a segment, chunks of a cell (split * cell_per = per)
    __host__ __device__ int cells() const { return (segs - 1) * split; }  // of a sequence
};

__host__ __device__ inline int attn_len(const int* lens, int b, int L) {
    if (!lens) return L;
    const int n = lens[b];
    return n < 0 ? 0 : n > L ? L : n;
}
__device__ __forceinline__ float attn_log_decay(const float* decay, int h) {
    if (!decay) return 0.0f;
    const float a = decay[h];
    return a < kLowDecay ? kLowDecay : a;
}

// A state z over rows whose log decays add up to x, with what they add to it, t: lambda z + t, for a
// lambda near 1 as z + ((lambda - 1) z + t).  A rounded lambda would be the same factor off each time
// (8192 tokens at a decay of -7e-5 ended 8e-5 off), and so would (lambda - 1) z added by itself,
// whose rounding repeats while z hardly moves.  Small lambdas are exact to a few 2^-24 themselves.
struct AttnFade {
    float m;    // lambda - 1, or lambda
    bool keep;
};
__device__ __forceinline__ AttnFade attn_fade(float x) {
    const bool keep = x > -0.5f;
    return {keep ? expm1f(x) : expf(x), keep};
}
__device__ __forceinline__ float attn_faded(const AttnFade& f, float z, float t) {
    return (f.keep ? z : 0.0f) + fmaf(z, f.m, t);
}

// What a state loses over cell c of a sequence of `chunks` chunks of T rows, at log decay ld a row.
// `part`: rows that the chunk with the first row lacks.
__device__ __forceinline__ AttnFade attn_cell_fade(float ld, const AttnArgs& a, int c, int chunks, int T, int part,
                                                   int back) {
    const int seg = c / a.split, c0 = min(chunks, seg * a.per + (c - seg * a.split) * a.cell_per);
    const int c1 = min(chunks, min(c0 + a.cell_per, (seg + 1) * a.per));
    const bool first = c1 > c0 && (back ? c1 == chunks : c0 == 0);
    return attn_fade(ld * (float)((c1 - c0) * T - (first ? part : 0)));
}
// Whether four rows m of a column are one 16-byte piece of the array (transposed states).
__device__ __forceinline__ bool attn_quads(const AttnPass& p) { return p.zm == 1 && p.zn % 4 == 0; }

// The state ahead of segment seg, N elements of it a thread: `at` gives element i's place in
// the array (below 0: none); four elements are rows m of a column.  The loads of all elements are
// under way at once: none is behind a branch (that took 40 us of 80 on 8 x 4096 x 8 heads of 128).
template <int N, typename F>
__device__ __forceinline__ void attn_state_ahead(const AttnPass& p, const AttnArgs& a, long long pair, int seg, float ld,
                                                 int chunks, int T, int part, F&& at, float (&z)[N]) {
    const long long size = (long long)p.Dk * p.Dv;
    const bool joined = seg > 0 && a.cells() > kFewCells;
    const float* from = joined ? p.carry + (pair * a.cells() + seg - 1) * size : p.z0 ? p.z0 + pair * size : nullptr;
    const bool quads = attn_quads(p);
    const auto load = [&](const float* s, float(&v)[N]) {
        if (quads) {
#pragma unroll
            for (int i = 0; i < N; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(s + max(at(i), 0));
                v[i] = f.x;
                v[i + 1] = f.y;
                v[i + 2] = f.z;
                v[i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < N; i++) v[i] = s[max(at(i), 0)];
        }
    };
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = 0.0f;
    if (from) load(from, z);
    if (joined) {
#pragma unroll
        for (int i = 0; i < N; i++) z[i] = at(i) >= 0 ? z[i] : 0.0f;
        return;
    }
    for (int c = 0; c < seg * a.split; c++) {
        const AttnFade w = attn_cell_fade(ld, a, c, chunks, T, part, p.back);
        const float* own = p.carry + (pair * a.cells() + c) * size;
        float v[N];
        load(own, v);
#pragma unroll
        for (int i = 0; i < N; i++) z[i] = attn_faded(w, z[i], v[i]);
    }
#pragma unroll
    for (int i = 0; i < N; i++) z[i] = at(i) >= 0 ? z[i] : 0.0f;
}

// Rows past the sequence's end: zeros, a share for each of `segs` blocks.
template <typename T>
__device__ __forceinline__ void attn_blank(const AttnPass& p, int b, int h, int len, int L, int seg, int segs) {
    const long long gone = (long long)(L - len), r0 = len + gone * seg / segs, r1 = len + gone * (seg + 1) / segs;
    T* y = static_cast<T*>(p.y.p) + b * p.y.batch + (long long)h * p.Dv;
    for (long long e = threadIdx.x; e < (r1 - r0) * p.Dv; e += blockDim.x) {
        const long long r = e / p.Dv;
        y[(r0 + r) * p.y.row + (e - r * p.Dv)] = from_f<T>(0.0f);
    }
}

// The tensor cores' kernels: head sizes up to 64, or up to 128.
__host__ __device__ constexpr bool attn_wide(int D) { return D > 64; }
// Runs f on the passes of each kernel together (gq's and gk's sizes are gv's the other way round); of a
// carry pass on those that fill one.
template <typename F> hc_status attn_by_kernel(const AttnArgs& all, bool carry, F&& f) {
    bool done[3] = {};
    for (int i = 0; i < all.passes; i++) {
        if (done[i] || (carry && !all.p[i].keep)) continue;
        AttnArgs a = all;
        a.passes = 0;
        for (int j = i; j < all.passes; j++)
            if (!done[j] && (!carry || all.p[j].keep) && attn_wide(all.p[j].Dk) == attn_wide(all.p[i].Dk) &&
                attn_wide(all.p[j].Dv) == attn_wide(all.p[i].Dv)) {
                a.p[a.passes++] = all.p[j];
                done[j] = true;
            }
        const hc_status e = f(a);
        if (e) return e;
    }
    return HC_OK;
}

// The kernels in fp32 (any type of row): 32-row chunks.  On the tensor cores (bf16): 128.
constexpr int AT_T = 32, AT_TC = 128;
// Blocks of the fp32 kernels that an SM holds, for pads (or head sizes) `most` >= `least`.  (Of 128 x 128 shared
// memory holds one; sequences are cut for two: 32 sequences x heads took 760 us so and 903 cut for one, 16 459 and 390.)
__host__ __device__ constexpr int attn_fp32_per_sm(int most, int least) { return least > (most > 96 ? 32 : 64) ? 2 : 3; }
hc_status launch_attn_fp32(const AttnArgs& a, bool carry, cudaStream_t st);
hc_status launch_attn_tc(const AttnArgs& a, bool carry, cudaStream_t st);
// Cells joined in order, in place: carry[s - 1] becomes the state ahead of segment s.
hc_status launch_attn_join(const AttnArgs& a, int T, cudaStream_t st);

}  // namespace hc
