// attn_fp32.cu -- linear attention passes (attn.cuh) in fp32 multiply-adds, for rows of
// every type, head sizes up to 128 and any strides.
//
// A block walks over one segment of one (sequence, head): 32 rows of q, k and v go to
// shared memory, the state stays there, and 16 x 16 threads take each of the four
// products in register tiles.  Bound by the multiply-adds and the shared-memory reads
// that feed them.
#include "attn.cuh"

namespace hc {
namespace {

constexpr int TP = AT_T + 2;  // pitch of a transposed tile: pairs of rows stay aligned

template <int PK, int PV> struct AttnSmem {
    float qt[PK][TP], kt[PK][TP];  // transposed
    float k[AT_T][PK], v[AT_T][PV];
    float z[PK][PV];
    float pt[AT_T][TP];            // scores, transposed: [j][i]
    float wj[AT_T];                // what row j weighs in the state
};

// Four elements of a row from channel c on, zeros past D.
template <typename T> __device__ __forceinline__ void load4(const T* row, int c, int D, bool wide, float (&f)[4]) {
    if (wide && c + 4 <= D) {
        load_pack<T, 4>(row + c, f);
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = c + i < D ? to_f(row[c + i]) : 0.0f;
    }
}

template <typename T, int PK, int PV, bool CARRY>
__global__ void __launch_bounds__(256) attn_fp32_kernel(AttnArgs a) {
    grid_begin();
    extern __shared__ __align__(16) unsigned char raw[];
    AttnSmem<PK, PV>& sm = *reinterpret_cast<AttnSmem<PK, PV>*>(raw);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const AttnPass& p = a.p[blockIdx.y];
    const int seg = blockIdx.x % a.segs, pair = blockIdx.x / a.segs;
    const bool last = seg == a.segs - 1;
    if (CARRY && last) return;  // its state is the pass's own
    const int b = pair / a.H, h = pair - b * a.H;
    const int len = attn_len(a.lens, b, a.L), chunks = (len + AT_T - 1) / AT_T;
    const int c0 = min(chunks, seg * a.per), c1 = min(chunks, c0 + a.per);
    const float l2 = attn_log2_decay(a.decay, h);
    const int Dk = p.Dk, Dv = p.Dv;
    const long long zsize = (long long)Dk * Dv;
    const T* qb = static_cast<const T*>(p.q.p) + b * p.q.batch + (long long)h * Dk;
    const T* kb = static_cast<const T*>(p.k.p) + b * p.k.batch + (long long)h * Dk;
    const T* vb = static_cast<const T*>(p.v.p) + b * p.v.batch + (long long)h * Dv;
    T* yb = static_cast<T*>(p.y.p) + b * p.y.batch + (long long)h * Dv;
    const auto wide4 = [&](const hc_rows& r, int D) {
        return D % 4 == 0 && r.row % 4 == 0 && r.batch % 4 == 0 && ((uintptr_t)r.p & (4 * sizeof(T) - 1)) == 0;
    };
    const bool wq = wide4(p.q, Dk), wk = wide4(p.k, Dk), wv = wide4(p.v, Dv);

    // the state ahead of the segment
    const float* z0 = CARRY ? nullptr : p.carry ? p.carry + ((long long)pair * a.segs + seg) * zsize
                                      : p.z0    ? p.z0 + pair * zsize
                                                : nullptr;
    for (int e = tid; e < PK * PV; e += 256) {
        const int m = e / PV, n = e - m * PV;
        sm.z[m][n] = z0 && m < Dk && n < Dv ? z0[(long long)m * p.zm + (long long)n * p.zn] : 0.0f;
    }

    for (int idx = c0; idx < c1; idx++) {
        const int c = p.back ? chunks - 1 - idx : idx;
        const int t0 = len - (chunks - c) * AT_T, lo = t0 < 0 ? -t0 : 0;
        // ---- rows in; those ahead of the sequence are zeros
        for (int e = tid; e < AT_T * (PK / 4); e += 256) {
            const int i = e / (PK / 4), d = (e - i * (PK / 4)) * 4;
            float qf[4] = {0, 0, 0, 0}, kf[4] = {0, 0, 0, 0};
            if (i >= lo && d < Dk) {
                if (!CARRY) load4(qb + (long long)(t0 + i) * p.q.row, d, Dk, wq, qf);
                load4(kb + (long long)(t0 + i) * p.k.row, d, Dk, wk, kf);
            }
#pragma unroll
            for (int s = 0; s < 4; s++) {
                if (!CARRY) {
                    sm.qt[d + s][i] = qf[s];
                    sm.kt[d + s][i] = kf[s];
                }
                sm.k[i][d + s] = kf[s];
            }
        }
        for (int e = tid; e < AT_T * (PV / 4); e += 256) {
            const int i = e / (PV / 4), d = (e - i * (PV / 4)) * 4;
            float vf[4] = {0, 0, 0, 0};
            if (i >= lo && d < Dv) load4(vb + (long long)(t0 + i) * p.v.row, d, Dv, wv, vf);
#pragma unroll
            for (int s = 0; s < 4; s++) sm.v[i][d + s] = vf[s];
        }
        if (tid < AT_T) sm.wj[tid] = tid < lo ? 0.0f : p.su * exp2f(l2 * (p.back ? tid - lo + 1 : AT_T - 1 - tid));
        __syncthreads();
        if (!CARRY) {
            // ---- scores of rows 2 ty, + 1 on rows 2 tx, + 1
            float s[2][2] = {};
#pragma unroll 4
            for (int d = 0; d < Dk; d++) {
                const float2 q2 = *reinterpret_cast<const float2*>(&sm.qt[d][2 * ty]);
                const float2 k2 = *reinterpret_cast<const float2*>(&sm.kt[d][2 * tx]);
                s[0][0] = fmaf(q2.x, k2.x, s[0][0]);
                s[0][1] = fmaf(q2.x, k2.y, s[0][1]);
                s[1][0] = fmaf(q2.y, k2.x, s[1][0]);
                s[1][1] = fmaf(q2.y, k2.y, s[1][1]);
            }
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int w = 0; w < 2; w++) {
                    const int i = 2 * ty + u, j = 2 * tx + w, n = p.back ? j - i : i - j;
                    sm.pt[j][i] = n >= 0 ? s[u][w] * (p.si * exp2f(l2 * n)) : 0.0f;
                }
            // ---- rows on the state
            float o[2][PV / 16];
#pragma unroll
            for (int n = 0; n < PV / 16; n++) o[0][n] = o[1][n] = 0.0f;
#pragma unroll 2
            for (int d = 0; d < Dk; d++) {
                const float2 q2 = *reinterpret_cast<const float2*>(&sm.qt[d][2 * ty]);
#pragma unroll
                for (int n = 0; n < PV / 32; n++) {
                    const float2 z2 = *reinterpret_cast<const float2*>(&sm.z[d][2 * tx + 32 * n]);
                    o[0][2 * n] = fmaf(q2.x, z2.x, o[0][2 * n]);
                    o[0][2 * n + 1] = fmaf(q2.x, z2.y, o[0][2 * n + 1]);
                    o[1][2 * n] = fmaf(q2.y, z2.x, o[1][2 * n]);
                    o[1][2 * n + 1] = fmaf(q2.y, z2.y, o[1][2 * n + 1]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int i = 2 * ty + u;
                const float w = p.sx * exp2f(l2 * (p.back ? AT_T - 1 - i : i >= lo ? i - lo + 1 : 0));
#pragma unroll
                for (int n = 0; n < PV / 16; n++) o[u][n] *= w;
            }
            __syncthreads();
            // ---- and on the chunk's rows
#pragma unroll 2
            for (int j = 0; j < AT_T; j++) {
                const float2 p2 = *reinterpret_cast<const float2*>(&sm.pt[j][2 * ty]);
#pragma unroll
                for (int n = 0; n < PV / 32; n++) {
                    const float2 v2 = *reinterpret_cast<const float2*>(&sm.v[j][2 * tx + 32 * n]);
                    o[0][2 * n] = fmaf(p2.x, v2.x, o[0][2 * n]);
                    o[0][2 * n + 1] = fmaf(p2.x, v2.y, o[0][2 * n + 1]);
                    o[1][2 * n] = fmaf(p2.y, v2.x, o[1][2 * n]);
                    o[1][2 * n + 1] = fmaf(p2.y, v2.y, o[1][2 * n + 1]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int i = 2 * ty + u;
                if (i < lo) continue;
                T* yr = yb + (long long)(t0 + i) * p.y.row;
#pragma unroll
                for (int n = 0; n < PV / 32; n++) {
                    const int m = 2 * tx + 32 * n;
                    if (m < Dv) yr[m] = from_f<T>(o[u][2 * n]);
                    if (m + 1 < Dv) yr[m + 1] = from_f<T>(o[u][2 * n + 1]);
                }
            }
        }
        // ---- the state behind the chunk: rows 2 ty + 32 r, + 1, columns 2 tx + 32 n, + 1
        const float w = exp2f(l2 * (AT_T - lo));
#pragma unroll
        for (int r = 0; r < PK / 32; r++) {
            float z[2][PV / 16];
            const int m = 2 * ty + 32 * r;
#pragma unroll
            for (int n = 0; n < PV / 32; n++) {
                const float2 a0 = *reinterpret_cast<const float2*>(&sm.z[m][2 * tx + 32 * n]);
                const float2 a1 = *reinterpret_cast<const float2*>(&sm.z[m + 1][2 * tx + 32 * n]);
                z[0][2 * n] = w * a0.x;
                z[0][2 * n + 1] = w * a0.y;
                z[1][2 * n] = w * a1.x;
                z[1][2 * n + 1] = w * a1.y;
            }
#pragma unroll 2
            for (int j = 0; j < AT_T; j++) {
                const float f = sm.wj[j];
                const float2 k2 = *reinterpret_cast<const float2*>(&sm.k[j][m]);
                const float ka = k2.x * f, kc = k2.y * f;
#pragma unroll
                for (int n = 0; n < PV / 32; n++) {
                    const float2 v2 = *reinterpret_cast<const float2*>(&sm.v[j][2 * tx + 32 * n]);
                    z[0][2 * n] = fmaf(ka, v2.x, z[0][2 * n]);
                    z[0][2 * n + 1] = fmaf(ka, v2.y, z[0][2 * n + 1]);
                    z[1][2 * n] = fmaf(kc, v2.x, z[1][2 * n]);
                    z[1][2 * n + 1] = fmaf(kc, v2.y, z[1][2 * n + 1]);
                }
            }
            // (every row has read the state ahead of the barrier above)
#pragma unroll
            for (int n = 0; n < PV / 32; n++) {
                *reinterpret_cast<float2*>(&sm.z[m][2 * tx + 32 * n]) = make_float2(z[0][2 * n], z[0][2 * n + 1]);
                *reinterpret_cast<float2*>(&sm.z[m + 1][2 * tx + 32 * n]) = make_float2(z[1][2 * n], z[1][2 * n + 1]);
            }
        }
        __syncthreads();
    }
    if (c0 == c1) __syncthreads();  // the state as it was loaded
    float* z1 = CARRY ? p.carry + ((long long)pair * a.segs + seg) * zsize
                      : p.z1 && last ? p.z1 + pair * zsize
                                            : nullptr;
    if (z1)
        for (int e = tid; e < PK * PV; e += 256) {
            const int m = e / PV, n = e - m * PV;
            if (m < Dk && n < Dv) z1[(long long)m * p.zm + (long long)n * p.zn] = sm.z[m][n];
        }
    if (!CARRY) attn_blank<T>(p, b, h, len, a.L, seg, a.segs);
}

template <typename T, int PK, int PV> hc_status launch_pads(const AttnArgs& a, bool carry, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    constexpr int smem = (int)sizeof(AttnSmem<PK, PV>);
    once_per_device(done, [] {
        return cudaFuncSetAttribute(attn_fp32_kernel<T, PK, PV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem) == cudaSuccess &&
               cudaFuncSetAttribute(attn_fp32_kernel<T, PK, PV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem) == cudaSuccess;
    });
    const dim3 grid((unsigned)((long long)a.B * a.H * a.segs), a.passes);
    if (carry)
        launch_next(attn_fp32_kernel<T, PK, PV, true>, grid, dim3(256), smem, st, a);
    else
        launch_next(attn_fp32_kernel<T, PK, PV, false>, grid, dim3(256), smem, st, a);
    return launched(carry ? "attn_fp32_carry_kernel" : "attn_fp32_kernel", st);
}

template <typename T, int PK> hc_status launch_pk(const AttnArgs& a, bool carry, cudaStream_t st) {
    const int pv = (a.p[0].Dv + 31) / 32;
    return pv == 1   ? launch_pads<T, PK, 32>(a, carry, st)
           : pv == 2 ? launch_pads<T, PK, 64>(a, carry, st)
           : pv == 3 ? launch_pads<T, PK, 96>(a, carry, st)
                     : launch_pads<T, PK, 128>(a, carry, st);
}
template <typename T> hc_status launch_type(const AttnArgs& a, bool carry, cudaStream_t st) {
    const int pk = (a.p[0].Dk + 31) / 32;
    return pk == 1   ? launch_pk<T, 32>(a, carry, st)
           : pk == 2 ? launch_pk<T, 64>(a, carry, st)
           : pk == 3 ? launch_pk<T, 96>(a, carry, st)
                     : launch_pk<T, 128>(a, carry, st);
}

}  // namespace

hc_status launch_attn_fp32(const AttnArgs& all, bool carry, cudaStream_t st) {
    return attn_by_shape(all, carry, [&](const AttnArgs& a) {
        return a.dtype == HC_DTYPE_F32    ? launch_type<float>(a, carry, st)
               : a.dtype == HC_DTYPE_BF16 ? launch_type<__nv_bfloat16>(a, carry, st)
                                          : launch_type<__half>(a, carry, st);
    });
}

}  // namespace hc
