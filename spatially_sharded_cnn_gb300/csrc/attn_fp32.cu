// attn_fp32.cu -- linear attention passes (attn.cuh) in fp32 multiply-adds, for rows of
// every type, head sizes up to 128 and any strides.
//
// A block walks over one segment of one (sequence, head): 32 rows of q, k and v go to
// shared memory, the state stays there, and 8 x 16 threads take each of the four products in
// register tiles of 4 rows x pairs of columns, four steps of the sum at a time (one 16-byte read
// a row serves all of a thread's columns).  Bound by the multiply-adds, two an instruction, and the
// shared-memory reads that feed them, with three blocks of four warps an SM to hide their latency:
// 20 sequences of 512 rows x 4 heads of 41 / 82 take 74 us, 31 % of the issue slots, behind 29 of their cells.
#include "attn.cuh"

namespace hc {
namespace {

constexpr int FT = 128;  // threads of a block

// Pitches keep rows on 16 bytes and spread neighbours over the banks.
template <int PK, int PV> struct AttnSmem {
    alignas(16) float q[AT_T][PK + 4];
    float k[AT_T][PK + 4];
    float v[AT_T][PV];
    float z[PK][PV];
    float p[AT_T][AT_T + 4];  // scores
    float wj[AT_T];           // what row j weighs in the state
};

// acc[r][n] += a[r][0 .. 3] . b[0 .. 3][n]: rows of `a` in shared memory, `pitch` floats apart,
// four rows of `b` (`step` floats apart) of which a thread takes the pairs 32 columns apart.
template <int R, int N>
__device__ __forceinline__ void mul4(f32x2 (&acc)[R][N], const float* a, int pitch, const float* b, int step) {
    float4 x[R];
#pragma unroll
    for (int r = 0; r < R; r++) x[r] = *reinterpret_cast<const float4*>(a + r * pitch);
#pragma unroll
    for (int u = 0; u < 4; u++) {
        f32x2 y[N];
#pragma unroll
        for (int n = 0; n < N; n++) y[n] = *reinterpret_cast<const f32x2*>(b + u * step + 32 * n);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const float f = u == 0 ? x[r].x : u == 1 ? x[r].y : u == 2 ? x[r].z : x[r].w;
            const f32x2 ff = pk2(f, f);
#pragma unroll
            for (int n = 0; n < N; n++) acc[r][n] = fma2(ff, y[n], acc[r][n]);
        }
    }
}

// Rows of every type through one kernel: an element's type is a branch that all threads take
// alike, a few instructions of a chunk (and a third of the kernels to compile).
__device__ __forceinline__ const char* elem(const void* p, long long i, int dtype) {
    return static_cast<const char*>(p) + (dtype == HC_DTYPE_F32 ? 4 : 2) * i;
}
// 16 bits of an element as fp32.
__device__ __forceinline__ float half_of(unsigned v, int dtype) {
    return dtype == HC_DTYPE_BF16 ? __uint_as_float(v << 16) : __half2float(__ushort_as_half((unsigned short)v));
}
// Four elements of a row from channel c on, zeros past D.
__device__ __forceinline__ void load4(const char* row, int dtype, int c, int D, bool wide, float (&f)[4]) {
    if (dtype == HC_DTYPE_F32) {
        const float* p = reinterpret_cast<const float*>(row) + c;
        if (wide && c + 4 <= D) {
            load_pack<float, 4>(p, f);
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) f[i] = c + i < D ? p[i] : 0.0f;
        }
    } else {
        const unsigned short* p = reinterpret_cast<const unsigned short*>(row) + c;
        unsigned v[4];
        if (wide && c + 4 <= D) {
            const uint2 w = *reinterpret_cast<const uint2*>(p);
            v[0] = w.x & 0xffffu;
            v[1] = w.x >> 16;
            v[2] = w.y & 0xffffu;
            v[3] = w.y >> 16;
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++) v[i] = c + i < D ? p[i] : 0u;
        }
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = half_of(v[i], dtype);
    }
}
__device__ __forceinline__ void store1(char* p, int dtype, float v) {
    if (dtype == HC_DTYPE_F32)
        *reinterpret_cast<float*>(p) = v;
    else if (dtype == HC_DTYPE_BF16)
        *reinterpret_cast<__nv_bfloat16*>(p) = from_f<__nv_bfloat16>(v);
    else
        *reinterpret_cast<__half*>(p) = from_f<__half>(v);
}

template <int PK, int PV, bool CARRY>
__device__ __forceinline__ void attn_fp32_pass(const AttnArgs& a, const AttnPass& p, AttnSmem<PK, PV>& sm) {
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int runs = CARRY ? a.cells() : a.segs, run = blockIdx.x % runs, pair = blockIdx.x / runs;  // a cell or a segment
    const int seg = CARRY ? run / a.split : run;
    const int b = pair / a.H, h = pair - b * a.H;
    const int len = attn_len(a.lens, b, a.L), chunks = (len + AT_T - 1) / AT_T;
    const int c0 = min(chunks, seg * a.per + (CARRY ? run - seg * a.split : 0) * a.cell_per);
    const int c1 = min(chunks, min(CARRY ? c0 + a.cell_per : 0x7fffffff, (seg + 1) * a.per));
    const float ld = attn_log_decay(a.decay, h), l2 = ld * kLog2e;
    const int Dk = p.Dk, Dv = p.Dv;
    const long long zsize = (long long)Dk * Dv;
    const int dt = a.dtype, bytes = dt == HC_DTYPE_F32 ? 4 : 2;
    const char* qb = elem(p.q.p, b * p.q.batch + (long long)h * Dk, dt);
    const char* kb = elem(p.k.p, b * p.k.batch + (long long)h * Dk, dt);
    const char* vb = elem(p.v.p, b * p.v.batch + (long long)h * Dv, dt);
    char* yb = const_cast<char*>(elem(p.y.p, b * p.y.batch + (long long)h * Dv, dt));
    const auto wide4 = [&](const hc_rows& r, int D) {
        return D % 4 == 0 && r.row % 4 == 0 && r.batch % 4 == 0 && ((uintptr_t)r.p & (4 * bytes - 1)) == 0;
    };
    const bool wq = wide4(p.q, Dk), wk = wide4(p.k, Dk), wv = wide4(p.v, Dv);

    // the state ahead of the segment: four rows of a column at a time
    for (int e0 = tid; e0 < PK / 4 * PV; e0 += FT * 4) {
        float z[16] = {};
        const auto place = [&](int i) {
            const int e = e0 + FT * (i >> 2), m = e / PV * 4 + (i & 3), n = e % PV;
            return e < PK / 4 * PV && m < Dk && n < Dv ? m * p.zm + n * p.zn : -1;
        };
        if (!CARRY) attn_state_ahead<16>(p, a, pair, seg, ld, chunks, AT_T, chunks * AT_T - len, place, z);
#pragma unroll
        for (int i = 0; i < 16; i++) {
            const int e = e0 + FT * (i >> 2);
            if (e < PK / 4 * PV) sm.z[e / PV * 4 + (i & 3)][e % PV] = z[i];
        }
    }

    // A chunk's rows wait in registers while the chunk before is multiplied: four values of row
    // (e / (P / 4)) each.
    constexpr int NK = PK / 16, NV = PV / 16;
    float qr[NK][4], kr[NK][4], vr[NV][4];
    const auto first_row = [&](int idx) { return len - (p.back ? idx + 1 : chunks - idx) * AT_T; };
    const auto fetch = [&](int t0) {
#pragma unroll
        for (int u = 0; u < NK; u++) {
            const int e = tid + FT * u, i = e / (PK / 4), d = (e - i * (PK / 4)) * 4;
            const bool in = t0 + i >= 0 && d < Dk;  // rows ahead of the sequence are zeros
#pragma unroll
            for (int s = 0; s < 4; s++) qr[u][s] = kr[u][s] = 0.0f;
            if (in && !CARRY) load4(qb + (long long)(t0 + i) * p.q.row * bytes, dt, d, Dk, wq, qr[u]);
            if (in) load4(kb + (long long)(t0 + i) * p.k.row * bytes, dt, d, Dk, wk, kr[u]);
        }
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int e = tid + FT * u, i = e / (PV / 4), d = (e - i * (PV / 4)) * 4;
#pragma unroll
            for (int s = 0; s < 4; s++) vr[u][s] = 0.0f;
            if (t0 + i >= 0 && d < Dv) load4(vb + (long long)(t0 + i) * p.v.row * bytes, dt, d, Dv, wv, vr[u]);
        }
    };
    if (c0 < c1) fetch(first_row(c0));

    float* z1 = CARRY ? p.carry + ((long long)pair * runs + run) * zsize
                      : p.z1 && seg == a.segs - 1 ? p.z1 + pair * zsize
                                            : nullptr;
    constexpr int N = PV / 32;  // pairs of columns 2 tx + 32 n, + 1
    const f32x2 none = pk2(0.0f, 0.0f);
    for (int idx = c0; idx < c1; idx++) {
        const int t0 = first_row(idx), lo = t0 < 0 ? -t0 : 0;
#pragma unroll
        for (int u = 0; u < NK; u++) {
            const int e = tid + FT * u, i = e / (PK / 4), d = (e - i * (PK / 4)) * 4;
            if (!CARRY) *reinterpret_cast<float4*>(&sm.q[i][d]) = make_float4(qr[u][0], qr[u][1], qr[u][2], qr[u][3]);
            *reinterpret_cast<float4*>(&sm.k[i][d]) = make_float4(kr[u][0], kr[u][1], kr[u][2], kr[u][3]);
        }
#pragma unroll
        for (int u = 0; u < NV; u++) {
            const int e = tid + FT * u, i = e / (PV / 4), d = (e - i * (PV / 4)) * 4;
            *reinterpret_cast<float4*>(&sm.v[i][d]) = make_float4(vr[u][0], vr[u][1], vr[u][2], vr[u][3]);
        }
        if (tid < AT_T) sm.wj[tid] = tid < lo ? 0.0f : p.su * exp2f(l2 * (p.back ? tid - lo + 1 : AT_T - 1 - tid));
        __syncthreads();
        if (idx + 1 < c1) fetch(first_row(idx + 1));
        if (!CARRY) {
            // ---- scores of rows 4 ty .. on rows tx, tx + 16 (eight lanes' reads of k then meet every bank)
            float s[4][2] = {};
#pragma unroll 4
            for (int d = 0; d < Dk; d += 4) {
                float4 k2[2];
#pragma unroll
                for (int w = 0; w < 2; w++) k2[w] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * w][d]);
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const float4 q4 = *reinterpret_cast<const float4*>(&sm.q[4 * ty + u][d]);
#pragma unroll
                    for (int w = 0; w < 2; w++)
                        s[u][w] = fmaf(q4.x, k2[w].x, fmaf(q4.y, k2[w].y, fmaf(q4.z, k2[w].z, fmaf(q4.w, k2[w].w, s[u][w]))));
                }
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int i = 4 * ty + u;
#pragma unroll
                for (int w = 0; w < 2; w++) {
                    const int j = tx + 16 * w, n = p.back ? j - i : i - j;
                    sm.p[i][j] = n >= 0 ? s[u][w] * (p.si * exp2f(l2 * n)) : 0.0f;
                }
            }
            // ---- rows on the state
            f32x2 o[4][N];
#pragma unroll
            for (int u = 0; u < 4; u++)
#pragma unroll
                for (int n = 0; n < N; n++) o[u][n] = none;
            if (idx > 0 || p.z0) {  // else the state is zero
#pragma unroll 2
                for (int d = 0; d < Dk; d += 4) mul4<4, N>(o, &sm.q[4 * ty][d], PK + 4, &sm.z[d][2 * tx], PV);
            }
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int i = 4 * ty + u;
                const float w = p.sx * exp2f(l2 * (p.back ? AT_T - 1 - i : i >= lo ? i - lo + 1 : 0));
#pragma unroll
                for (int n = 0; n < N; n++) o[u][n] = mul2(o[u][n], pk2(w, w));
            }
            __syncthreads();
            // ---- and on the chunk's rows
#pragma unroll 2
            for (int j = 0; j < AT_T; j += 4) mul4<4, N>(o, &sm.p[4 * ty][j], AT_T + 4, &sm.v[j][2 * tx], PV);
#pragma unroll
            for (int u = 0; u < 4; u++) {
                const int i = 4 * ty + u;
                if (i < lo) continue;
                char* yr = yb + (long long)(t0 + i) * p.y.row * bytes;
#pragma unroll
                for (int n = 0; n < N; n++) {
                    const int m = 2 * tx + 32 * n;
                    float f0, f1;
                    unpk2(o[u][n], f0, f1);
                    if (m < Dv) store1(yr + m * bytes, dt, f0);
                    if (m + 1 < Dv) store1(yr + (m + 1) * bytes, dt, f1);
                }
            }
        }
        if (idx + 1 == c1 && !z1) break;
        // ---- the state behind the chunk: rows 4 ty .. + 32 r
        // (every row has read the state ahead of the barrier above)
        const AttnFade f = attn_fade(ld * (float)(AT_T - lo));
        const f32x2 mm = pk2(f.m, f.m), keep = f.keep ? pk2(1.0f, 1.0f) : none;
#pragma unroll
        for (int r = 0; r < PK / 32; r++) {
            f32x2 z[4][N];
            const int m = 4 * ty + 32 * r;
            if (m >= Dk) break;
#pragma unroll
            for (int u = 0; u < 4; u++)
#pragma unroll
                for (int n = 0; n < N; n++)
                    z[u][n] = mul2(*reinterpret_cast<const f32x2*>(&sm.z[m + u][2 * tx + 32 * n]), mm);
#pragma unroll 4
            for (int j = 0; j < AT_T; j++) {
                const float wj = sm.wj[j];
                const float4 k4 = *reinterpret_cast<const float4*>(&sm.k[j][m]);
                const float kw[4] = {k4.x * wj, k4.y * wj, k4.z * wj, k4.w * wj};
                f32x2 v2[N];
#pragma unroll
                for (int n = 0; n < N; n++) v2[n] = *reinterpret_cast<const f32x2*>(&sm.v[j][2 * tx + 32 * n]);
#pragma unroll
                for (int u = 0; u < 4; u++)
#pragma unroll
                    for (int n = 0; n < N; n++) z[u][n] = fma2(pk2(kw[u], kw[u]), v2[n], z[u][n]);
            }
#pragma unroll
            for (int u = 0; u < 4; u++)
#pragma unroll
                for (int n = 0; n < N; n++) {  // attn_faded
                    f32x2& to = *reinterpret_cast<f32x2*>(&sm.z[m + u][2 * tx + 32 * n]);
                    to = fma2(to, keep, z[u][n]);
                }
        }
        __syncthreads();
    }
    if (c0 == c1) __syncthreads();  // the state as it was loaded
    if (z1) {
        const bool quads = attn_quads(p);
        for (int e = tid; e < PK / 4 * PV; e += FT) {
            const int m = e / PV * 4, n = e % PV;
            if (m >= Dk || n >= Dv) continue;
            float* to = z1 + m * p.zm + n * p.zn;
            if (quads) {
                *reinterpret_cast<float4*>(to) = make_float4(sm.z[m][n], sm.z[m + 1][n], sm.z[m + 2][n], sm.z[m + 3][n]);
            } else {
                for (int i = 0; i < 4 && m + i < Dk; i++) to[i * p.zm] = sm.z[m + i][n];
            }
        }
    }
    if (!CARRY) {
        if (dt == HC_DTYPE_F32)
            attn_blank<float>(p, b, h, len, a.L, seg, a.segs);
        else  // (a zero is the same two bytes in either type)
            attn_blank<__half>(p, b, h, len, a.L, seg, a.segs);
    }
}

// Passes of Dk up to PK and Dv up to PV, or the other way round: those of one gradient call are one
// launch.
template <int PK, int PV, bool CARRY>
__global__ void __launch_bounds__(FT, (attn_fp32_per_sm(PK, PV))) attn_fp32_kernel(AttnArgs a) {
    grid_begin();
    extern __shared__ __align__(16) unsigned char raw[];
    const AttnPass& p = a.p[blockIdx.y];
    if (PK == PV || (p.Dk > PV && p.Dk <= PK))
        attn_fp32_pass<PK, PV, CARRY>(a, p, *reinterpret_cast<AttnSmem<PK, PV>*>(raw));
    else
        attn_fp32_pass<PV, PK, CARRY>(a, p, *reinterpret_cast<AttnSmem<PV, PK>*>(raw));
}

template <int PK, int PV> hc_status launch_pads(const AttnArgs& a, bool carry, cudaStream_t st) {
    static std::atomic<unsigned long long> done{0};
    constexpr int one = (int)sizeof(AttnSmem<PK, PV>), two = (int)sizeof(AttnSmem<PV, PK>), smem = one > two ? one : two;
    once_per_device(done, [] {
        return cudaFuncSetAttribute(attn_fp32_kernel<PK, PV, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
                   cudaSuccess &&
               cudaFuncSetAttribute(attn_fp32_kernel<PK, PV, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) ==
                   cudaSuccess;
    });
    const dim3 grid((unsigned)((long long)a.B * a.H * (carry ? a.cells() : a.segs)), a.passes);
    if (carry)
        launch_next(attn_fp32_kernel<PK, PV, true>, grid, dim3(FT), smem, st, a);
    else
        launch_next(attn_fp32_kernel<PK, PV, false>, grid, dim3(FT), smem, st, a);
    return launched(carry ? "attn_fp32_carry_kernel" : "attn_fp32_kernel", st);
}

}  // namespace

hc_status launch_attn_fp32(const AttnArgs& all, bool carry, cudaStream_t st) {
    AttnArgs a = all;
    if (carry) {  // the passes that fill one
        a.passes = 0;
        for (int i = 0; i < all.passes; i++)
            if (all.p[i].keep) a.p[a.passes++] = all.p[i];
    }
    const int k = cdiv(a.p[0].Dk, 32), v = cdiv(a.p[0].Dv, 32), most = k > v ? k : v, least = k > v ? v : k;
    switch (most * 4 + least) {
        case 5: return launch_pads<32, 32>(a, carry, st);
        case 9: return launch_pads<64, 32>(a, carry, st);
        case 10: return launch_pads<64, 64>(a, carry, st);
        case 13: return launch_pads<96, 32>(a, carry, st);
        case 14: return launch_pads<96, 64>(a, carry, st);
        case 15: return launch_pads<96, 96>(a, carry, st);
        case 17: return launch_pads<128, 32>(a, carry, st);
        case 18: return launch_pads<128, 64>(a, carry, st);
        case 19: return launch_pads<128, 96>(a, carry, st);
        default: return launch_pads<128, 128>(a, carry, st);
    }
}

}  // namespace hc
