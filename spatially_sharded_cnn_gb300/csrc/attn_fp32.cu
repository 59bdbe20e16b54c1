// attn_fp32.cu -- linear attention passes (attn.cuh) in fp32 multiply-adds, for rows of
// every type, head sizes up to 128 and any strides.
//
// A block walks over one segment of one (sequence, head): 32 rows of q, k and v go to
// shared memory, the state stays there, and 16 x 16 threads take each of the four
// products in register tiles, two values an instruction.  Bound by the multiply-adds and the shared-memory reads
// that feed them.
#include "attn.cuh"

namespace hc {
namespace {

constexpr int TP = AT_T + 2;  // pitch of a transposed tile: pairs of rows stay aligned

template <int PK, int PV> struct AttnSmem {
    alignas(16) float k[AT_T][PK], v[AT_T][PV];
    float z[PK][PV];
    float qt[PK][TP], kt[PK][TP];  // transposed
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
    const int runs = CARRY ? a.cells() : a.segs, run = blockIdx.x % runs, pair = blockIdx.x / runs;  // a cell or a segment
    const int seg = CARRY ? run / a.split : run;
    const int b = pair / a.H, h = pair - b * a.H;
    const int len = attn_len(a.lens, b, a.L), chunks = (len + AT_T - 1) / AT_T;
    const int c0 = min(chunks, seg * a.per + (CARRY ? run - seg * a.split : 0) * a.cell_per);
    const int c1 = min(chunks, min(CARRY ? c0 + a.cell_per : 0x7fffffff, (seg + 1) * a.per));
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
    for (int e0 = 0; e0 < PK * PV; e0 += 256 * 16) {
        float z[16] = {};
        const auto place = [&](int i) {
            const int e = e0 + tid + 256 * i, m = e / PV, n = e - m * PV;
            return e < PK * PV && m < Dk && n < Dv ? m * p.zm + n * p.zn : -1;
        };
        if (!CARRY) attn_state_ahead<16>(p, a, pair, seg, l2, chunks, AT_T, chunks * AT_T - len, place, z);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int e = e0 + tid + 256 * i;
            if (e < PK * PV) sm.z[e / PV][e % PV] = z[i];
        }
    }

    // A chunk's rows wait in registers while the chunk before is multiplied: four values of row
    // (e / (P / 4)) each.
    constexpr int NK = PK / 32, NV = PV / 32;
    float qr[NK][4], kr[NK][4], vr[NV][4];
    const auto first_row = [&](int idx) { return len - (p.back ? idx + 1 : chunks - idx) * AT_T; };
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int u = 0; u < NK; u++) {
            const int e = tid + 256 * u, i = e / (PK / 4), d = (e - i * (PK / 4)) * 4;
            const bool in = t0 + i >= 0 && d < Dk;  // rows ahead of the sequence are zeros
#pragma unroll
            for (int s = 0; s < 4; s++) qr[u][s] = kr[u][s] = 0.0f;
            if (in && !CARRY) load4(qb + (long long)(t0 + i) * p.q.row, d, Dk, wq, qr[u]);
            if (in) load4(kb + (long long)(t0 + i) * p.k.row, d, Dk, wk, kr[u]);
        }
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int e = tid + 256 * u, i = e / (PV / 4), d = (e - i * (PV / 4)) * 4;
#pragma unroll
            for (int s = 0; s < 4; s++) vr[u][s] = 0.0f;
            if (t0 + i >= 0 && d < Dv) load4(vb + (long long)(t0 + i) * p.v.row, d, Dv, wv, vr[u]);
        }
    };
    if (c0 < c1) fetch(first_row(c0));

    for (int idx = c0; idx < c1; idx++) {
        const int t0 = first_row(idx), lo = t0 < 0 ? -t0 : 0;
#pragma unroll
        for (int u = 0; u < NK; u++) {
            const int e = tid + 256 * u, i = e / (PK / 4), d = (e - i * (PK / 4)) * 4;
            if (!CARRY) {
#pragma unroll
                for (int s = 0; s < 4; s++) {
                    sm.qt[d + s][i] = qr[u][s];
                    sm.kt[d + s][i] = kr[u][s];
                }
            }
            *reinterpret_cast<float4*>(&sm.k[i][d]) = make_float4(kr[u][0], kr[u][1], kr[u][2], kr[u][3]);
        }
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int e = tid + 256 * u, i = e / (PV / 4), d = (e - i * (PV / 4)) * 4;
            *reinterpret_cast<float4*>(&sm.v[i][d]) = make_float4(vr[u][0], vr[u][1], vr[u][2], vr[u][3]);
        }
        if (tid < AT_T) sm.wj[tid] = tid < lo ? 0.0f : p.su * exp2f(l2 * (p.back ? tid - lo + 1 : AT_T - 1 - tid));
        __syncthreads();
        if (idx + 1 < c1) fetch(first_row(idx + 1));
        if (!CARRY) {
            // ---- scores of rows 2 ty, + 1 on rows 2 tx, + 1
            f32x2 s[2] = {pk2(0.0f, 0.0f), pk2(0.0f, 0.0f)};
#pragma unroll 8
            for (int d = 0; d < Dk; d++) {
                const float2 q2 = *reinterpret_cast<const float2*>(&sm.qt[d][2 * ty]);
                const f32x2 k2 = *reinterpret_cast<const f32x2*>(&sm.kt[d][2 * tx]);
                s[0] = fma2(pk2(q2.x, q2.x), k2, s[0]);
                s[1] = fma2(pk2(q2.y, q2.y), k2, s[1]);
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                float sc[2];
                unpk2(s[u], sc[0], sc[1]);
#pragma unroll
                for (int w = 0; w < 2; w++) {
                    const int i = 2 * ty + u, j = 2 * tx + w, n = p.back ? j - i : i - j;
                    sm.pt[j][i] = n >= 0 ? sc[w] * (p.si * exp2f(l2 * n)) : 0.0f;
                }
            }
            // ---- rows on the state
            f32x2 o[2][NV];
#pragma unroll
            for (int n = 0; n < NV; n++) o[0][n] = o[1][n] = pk2(0.0f, 0.0f);
#pragma unroll 4
            for (int d = 0; d < Dk; d++) {
                const float2 q2 = *reinterpret_cast<const float2*>(&sm.qt[d][2 * ty]);
                const f32x2 qa = pk2(q2.x, q2.x), qc = pk2(q2.y, q2.y);
#pragma unroll
                for (int n = 0; n < NV; n++) {
                    const f32x2 z2 = *reinterpret_cast<const f32x2*>(&sm.z[d][2 * tx + 32 * n]);
                    o[0][n] = fma2(qa, z2, o[0][n]);
                    o[1][n] = fma2(qc, z2, o[1][n]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int i = 2 * ty + u;
                const float w = p.sx * exp2f(l2 * (p.back ? AT_T - 1 - i : i >= lo ? i - lo + 1 : 0));
#pragma unroll
                for (int n = 0; n < NV; n++) o[u][n] = mul2(o[u][n], pk2(w, w));
            }
            __syncthreads();
            // ---- and on the chunk's rows
#pragma unroll 4
            for (int j = 0; j < AT_T; j++) {
                const float2 p2 = *reinterpret_cast<const float2*>(&sm.pt[j][2 * ty]);
                const f32x2 pa = pk2(p2.x, p2.x), pc = pk2(p2.y, p2.y);
#pragma unroll
                for (int n = 0; n < NV; n++) {
                    const f32x2 v2 = *reinterpret_cast<const f32x2*>(&sm.v[j][2 * tx + 32 * n]);
                    o[0][n] = fma2(pa, v2, o[0][n]);
                    o[1][n] = fma2(pc, v2, o[1][n]);
                }
            }
#pragma unroll
            for (int u = 0; u < 2; u++) {
                const int i = 2 * ty + u;
                if (i < lo) continue;
                T* yr = yb + (long long)(t0 + i) * p.y.row;
#pragma unroll
                for (int n = 0; n < NV; n++) {
                    const int m = 2 * tx + 32 * n;
                    float f0, f1;
                    unpk2(o[u][n], f0, f1);
                    if (m < Dv) yr[m] = from_f<T>(f0);
                    if (m + 1 < Dv) yr[m + 1] = from_f<T>(f1);
                }
            }
        }
        // ---- the state behind the chunk: rows 2 ty + 32 r, + 1, columns 2 tx + 32 n, + 1
        // (every row has read the state ahead of the barrier above)
        const float w = exp2f(l2 * (AT_T - lo));
        const f32x2 ww = pk2(w, w);
#pragma unroll
        for (int r = 0; r < NK; r++) {
            f32x2 z[2][NV];
            const int m = 2 * ty + 32 * r;
#pragma unroll
            for (int n = 0; n < NV; n++) {
                z[0][n] = mul2(ww, *reinterpret_cast<const f32x2*>(&sm.z[m][2 * tx + 32 * n]));
                z[1][n] = mul2(ww, *reinterpret_cast<const f32x2*>(&sm.z[m + 1][2 * tx + 32 * n]));
            }
#pragma unroll 4
            for (int j = 0; j < AT_T; j++) {
                const float f = sm.wj[j];
                const float2 k2 = *reinterpret_cast<const float2*>(&sm.k[j][m]);
                const f32x2 ka = pk2(k2.x * f, k2.x * f), kc = pk2(k2.y * f, k2.y * f);
#pragma unroll
                for (int n = 0; n < NV; n++) {
                    const f32x2 v2 = *reinterpret_cast<const f32x2*>(&sm.v[j][2 * tx + 32 * n]);
                    z[0][n] = fma2(ka, v2, z[0][n]);
                    z[1][n] = fma2(kc, v2, z[1][n]);
                }
            }
#pragma unroll
            for (int n = 0; n < NV; n++) {
                *reinterpret_cast<f32x2*>(&sm.z[m][2 * tx + 32 * n]) = z[0][n];
                *reinterpret_cast<f32x2*>(&sm.z[m + 1][2 * tx + 32 * n]) = z[1][n];
            }
        }
        __syncthreads();
    }
    if (c0 == c1) __syncthreads();  // the state as it was loaded
    float* z1 = CARRY ? p.carry + ((long long)pair * runs + run) * zsize
                      : p.z1 && seg == a.segs - 1 ? p.z1 + pair * zsize
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
    const dim3 grid((unsigned)((long long)a.B * a.H * (carry ? a.cells() : a.segs)), a.passes);
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
