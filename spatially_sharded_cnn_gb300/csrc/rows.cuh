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

// SiLU x * s and its slope s * (1 + x * (1 - s)), s = 1 / (1 + exp(-x)).
__device__ __forceinline__ float sigmoid_f(float x) { return 1.0f / (1.0f + expf(-x)); }
__device__ __forceinline__ float silu_f(float x) { return x / (1.0f + expf(-x)); }
__device__ __forceinline__ float silu_d(float x) {
    const float s = sigmoid_f(x);
    return s * (1.0f + x * (1.0f - s));
}

template <int ACT> __device__ __forceinline__ float act_f(float x) {
    return ACT == HC_PW_SILU ? silu_f(x) : ACT == HC_PW_GELU ? gelu_f(x) : x;
}
template <int ACT> __device__ __forceinline__ float act_d(float x) {
    return ACT == HC_PW_SILU ? silu_d(x) : ACT == HC_PW_GELU ? gelu_d(x) : 1.0f;
}

// Column sums of in[rows][na + nb + nc] in a fixed order: the first na columns
// to `a`, the next nb to `b`, the last nc to `c` (each may be NULL).
hc_status launch_column_totals(const float* in, long long rows, float* a, int na, float* b, int nb, float* c, int nc,
                               cudaStream_t st);

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
