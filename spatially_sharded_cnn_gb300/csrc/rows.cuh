// rows.cuh -- shared by the channels-last operators (groupnorm.cu,
// causal_conv.cu, scan.cu): element types, wide loads and stores, argument
// checks of hc_rows tensors.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace hc {

template <int DT> struct EltOf;
template <> struct EltOf<HC_DTYPE_F32> { using type = float; };
template <> struct EltOf<HC_DTYPE_BF16> { using type = __nv_bfloat16; };
template <> struct EltOf<HC_DTYPE_F16> { using type = __half; };

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <> __device__ __forceinline__ __half from_f<__half>(float v) { return __float2half_rn(v); }

// V adjacent elements; one aligned load or store of V * sizeof(T) <= 16 bytes.
template <typename T, int V> struct alignas(sizeof(T) * V) Pack {
    T v[V];
};
template <typename T, int V> __device__ __forceinline__ void load_pack(const T* p, float (&f)[V]) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = to_f(q.v[i]);
}
template <typename T, int V> __device__ __forceinline__ void store_pack(T* p, const float (&f)[V]) {
    Pack<T, V> q;
#pragma unroll
    for (int i = 0; i < V; i++) q.v[i] = from_f<T>(f[i]);
    *reinterpret_cast<Pack<T, V>*>(p) = q;
}

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

// 2^x and 1/x on the special function unit (2 and 1 ulp; results below the
// normal range are zero).
__device__ __forceinline__ float ex2f(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float rcpf(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_raw(const T* p) {
    return *reinterpret_cast<const Pack<T, V>*>(p);
}
// The same for data that is not read again soon: evicted first.
template <int BYTES> struct Word;
template <> struct Word<16> { using type = uint4; };
template <> struct Word<4> { using type = unsigned; };
template <> struct Word<2> { using type = unsigned short; };
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_raw_last(const T* p) {
    using W = typename Word<sizeof(T) * V>::type;
    union U {
        W w;
        Pack<T, V> q;
        __device__ U() {}
    } u;
    // volatile: never ahead of grid_begin
    if constexpr (sizeof(W) == 16)
        asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.w.x), "=r"(u.w.y), "=r"(u.w.z), "=r"(u.w.w)
                     : "l"(p));
    else if constexpr (sizeof(W) == 4)
        asm volatile("ld.global.cs.u32 %0, [%1];" : "=r"(u.w) : "l"(p));
    else
        asm volatile("ld.global.cs.u16 %0, [%1];" : "=h"(u.w) : "l"(p));
    return u.q;
}
// For rows that no cache holds until they are read again.
template <typename T, int V> __device__ __forceinline__ Pack<T, V> load_raw_stream(const T* p) {
    if constexpr (sizeof(T) * V == 16) {
        union U {
            uint4 w;
            Pack<T, V> q;
            __device__ U() {}
        } u;
        asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(u.w.x), "=r"(u.w.y), "=r"(u.w.z), "=r"(u.w.w)
                     : "l"(p));
        return u.q;
    } else {
        return load_raw<T, V>(p);
    }
}
template <typename T, int V> __device__ __forceinline__ void store_pack_last(T* p, const float (&f)[V]) {
    using W = typename Word<sizeof(T) * V>::type;
    union U {
        W w;
        Pack<T, V> q;
        __device__ U() {}
    } u;
#pragma unroll
    for (int i = 0; i < V; i++) u.q.v[i] = from_f<T>(f[i]);
    __stcs(reinterpret_cast<W*>(p), u.w);
}
template <typename T, int V> __device__ __forceinline__ void unpack(const Pack<T, V>& q, float (&f)[V]) {
#pragma unroll
    for (int i = 0; i < V; i++) f[i] = to_f(q.v[i]);
}

// SiLU x * s and its slope s * (1 + x * (1 - s)), s = 1 / (1 + exp(-x)): a few
// ulps from two special-function results, which the elementwise kernels would
// otherwise spend most of their instructions on.
__device__ __forceinline__ float sigmoid_f(float x) { return rcpf(1.0f + ex2f(-kLog2e * x)); }
__device__ __forceinline__ float silu_f(float x) { return x * sigmoid_f(x); }
__device__ __forceinline__ float silu_d(float x) {
    const float s = sigmoid_f(x);
    return s * fmaf(x, 1.0f - s, 1.0f);
}
// log(1 + exp(x)) = max(x, 0) + log(1 + e), e = exp(-|x|), with log(1 + e) =
// 2 atanh(v), v = e / (2 + e) <= 1/3, by the series of atanh up to v^13 (the
// next term is below 2^-25 of the sum): relative accuracy also where e is small,
// which a logarithm of the rounded 1 + e would not give.
__device__ __forceinline__ float softplus_f(float x) {
    const float e = ex2f(-kLog2e * fabsf(x));
    const float v = e * rcpf(2.0f + e), w = v * v;
    float p = fmaf(w, 1.0f / 13, 1.0f / 11);
    p = fmaf(w, p, 1.0f / 9);
    p = fmaf(w, p, 1.0f / 7);
    p = fmaf(w, p, 1.0f / 5);
    p = fmaf(w, p, 1.0f / 3);
    p = fmaf(w, p, 1.0f);
    return fmaf(2.0f * v, p, fmaxf(x, 0.0f));
}

// GELU x Phi(x) and its slope Phi(x) + x phi(x) from a = |x| (up to 14, where e ends),
// e = exp(-x^2 / 2) and R, Phi(-a) = e * R: the function R, a scaled complementary error
// function, falls from 1/2 like 1 / a.  It is a polynomial of degree 7 in
// s = a / (1 + 0.33 a), fitted here in 64 bits (least squares, reweighted until the
// largest error of e * R is level: 4e-9).  s = 0 at x = 0, so that the last addition
// alone rounds there, and the tail keeps its relative accuracy.
// GELU of normal values is 1.8e-8 off (rms; 2.4e-8 in the form with erff, which took
// 361 us where this takes 291 on 7 x 131072 x 256 bf16), its slope 2.4e-8 (2.7e-8).
__device__ __forceinline__ float normal_tail(float x, float& a, float& e) {
    a = fminf(fabsf(x), 14.0f);
    const float s = a * rcpf(fmaf(0.33f, a, 1.0f));
    e = ex2f(-0.5f * kLog2e * x * x);
    float p = fmaf(s, -1.96299188e-05f, 0.000127479288f);
    p = fmaf(s, p, 0.000140480028f);
    p = fmaf(s, p, -0.0017548654f);
    p = fmaf(s, p, -0.0114476355f);
    p = fmaf(s, p, 0.118352972f);
    p = fmaf(s, p, -0.3989425f);
    return fmaf(s, p, 0.5f);
}
// max(x, 0) - a Phi(-a)
__device__ __forceinline__ float pw_gelu_f(float x) {
    float a, e;
    const float r = normal_tail(x, a, e);
    return fmaf(-a, r * e, fmaxf(x, 0.0f));
}
// Phi(-a) - a phi(a), or 1 less that for x >= 0
__device__ __forceinline__ float pw_gelu_d(float x) {
    float a, e;
    const float r = normal_tail(x, a, e), g = e * fmaf(-0.39894228040143268f, a, r);
    return x >= 0.0f ? 1.0f - g : g;
}

template <int ACT> __device__ __forceinline__ float act_f(float x) {
    return ACT == HC_PW_SILU ? silu_f(x) : ACT == HC_PW_GELU ? pw_gelu_f(x) : x;
}
template <int ACT> __device__ __forceinline__ float act_d(float x) {
    return ACT == HC_PW_SILU ? silu_d(x) : ACT == HC_PW_GELU ? pw_gelu_d(x) : 1.0f;
}

// Column sums of in[rows][na + nb + nc] in a fixed order: the first na columns
// to `a`, the next nb to `b`, the last nc to `c` (each may be NULL).
hc_status launch_column_totals(const float* in, long long rows, float* a, int na, float* b, int nb, float* c, int nc,
                               cudaStream_t st);

// Two fp32 values in one 64-bit register pair: one instruction for two
// multiply-adds.
using f32x2 = unsigned long long;
__device__ __forceinline__ f32x2 pk2(float lo, float hi) {
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpk2(f32x2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
// These operators' kernels are launched so that one may start while the last
// blocks of the kernel before it in the stream are finishing: a kernel's first act
// is grid_begin, which waits until that kernel is complete and its writes are
// visible.  Hides most of a launch's latency (about 2 us), of which a short call
// has several: the ragged 5 x 1537 x 328 scan training took 148 us before and 130 after,
// 121 with later changes.  (Letting the next
// kernel's blocks in before this one's begin to end made the 224 x 1024 x 256 step
// 1.60 -> 1.74 ms: they take the shared memory that this one's later blocks want.)
// Everything is read through plain pointers or volatile loads, parameters too (an
// optimizer's kernel writes them just before the next call): loads through
// __restrict__ pointers or of the read-only path could be moved above the wait.
__device__ __forceinline__ void grid_begin() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
void launch_next(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute at = {};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

inline size_t dtype_size(int dt) { return dt == HC_DTYPE_F32 ? 4 : 2; }
inline bool dtype_ok(int dt) { return dt == HC_DTYPE_F32 || dt == HC_DTYPE_BF16 || dt == HC_DTYPE_F16; }
inline bool ptr_al(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// An input of the desc's type: present (unless it has no rows), aligned to its
// elements, strides >= 0.
inline bool rows_in_ok(const hc_rows* r, int dt, long long nr = 1) {
    return r && (r->p || nr == 0) && r->dtype == dt && ptr_al(r->p, dtype_size(dt)) && r->batch >= 0 && r->row >= 0;
}
// An output [nb][nr][C]: also no two of its rows overlap.
inline bool rows_out_ok(const hc_rows* r, int dt, long long nb, long long nr, long long C) {
    if (!rows_in_ok(r, dt, nr)) return false;
    if (nr == 0) return true;
    const long long b = r->batch, w = r->row;
    if (nr > 1 && w < C) return false;
    if (nb > 1 && b < C) return false;
    if (nb <= 1 || nr <= 1) return true;
    return b >= (nr - 1) * w + C || w >= (nb - 1) * b + C;
}
inline bool rows_same(const hc_rows* a, const hc_rows* b) { return a->p && a->p == b->p; }
// Whether every row starts on a boundary of `v` elements (given that the
// channel offsets used are multiples of v).
inline bool rows_vec(const hc_rows* r, int v) {
    return !r->p || (ptr_al(r->p, v * dtype_size((int)r->dtype)) && r->batch % v == 0 && r->row % v == 0);
}
// A tensor as the kernels take it.
template <typename T> struct View {
    T* p;
    long long batch, row;
};
template <typename T> View<T> view(const hc_rows* r) { return {static_cast<T*>(r->p), r->batch, r->row}; }

inline bool f32_ok(const void* p) { return p && ptr_al(p, 16); }
inline bool f32_opt_ok(const void* p) { return ptr_al(p, 16); }  // NULL passes

}  // namespace hc
