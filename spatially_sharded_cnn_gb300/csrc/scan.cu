// scan.cu -- selective state-space scan on channels-last sequences, forward,
// backward and one token (formulas: hc_mixer.h).
//
// A state h[d][n] belongs to one (sequence, channel, state index).  A warp
// spreads d_state over NL lanes of four states each (d_state rounded up to 4,
// 8, 16, 32 or 64 with states whose B and C are zero) and its 32 / NL lane
// groups over channels: a value of B or C read from shared memory then serves
// several channels of a thread, a step size serves four states, and both sums
// the scan needs -- y over states, the gradients of B and C over channels --
// are partly in-thread and take few shuffles.
//
// The recurrence is sequential in the rows.  Where sequences and channels alone
// do not fill the GPU, a sequence is cut into segments of whole tiles: one pass
// takes every segment from a zero state, the segments' results are joined
// (h_out = exp(A * sum of steps) * h_in + h_local), and the full pass then runs
// every segment from its own first state.  The extra pass costs its
// exponentials again and buys a factor of `segs` in parallelism.
//
// scan_fwd.cu, scan_carry.cu and scan_bwd.cu hold the passes over a sequence,
// this file one token and the entry points.
#include "scan.cuh"

namespace hc {
namespace {

template <int DT> __device__ __forceinline__ float ld(const void* p, long long i) {
    return to_f(static_cast<const typename EltOf<DT>::type*>(p)[i]);
}
template <int DT> __device__ __forceinline__ void st(void* p, long long i, float v) {
    using T = typename EltOf<DT>::type;
    static_cast<T*>(p)[i] = from_f<T>(v);
}

// gB and gC: the channel tiles' sums in tile order, Q states a thread.  Bound by
// memory: 224 x 1024 rows of two tiles, 88 MB, in 19 us, 4.6 TB/s.
template <int DT, int Q> __global__ void __launch_bounds__(256) scan_bc_kernel(const __grid_constant__ ScanArgs a) {
    grid_begin();
    const unsigned width = (unsigned)(a.G * 2 * a.N) / Q;
    const long long rows = (long long)a.B * a.L, per = rows * width * Q;
    for (long long q = blockIdx.x * 256LL + threadIdx.x; q < rows * width; q += gridDim.x * 256LL) {
        const long long r = q < 0x7fffffffLL ? (unsigned)q / width : q / width;
        const unsigned j = (unsigned)(q - r * width) * Q;
        const long long b = r < 0x7fffffffLL ? (unsigned)r / (unsigned)a.L : r / a.L;
        const int t = (int)(r - b * a.L);
        float v[Q], e[Q];
        load_pack<float, Q>(a.gbc + q * Q, v);
#pragma unroll 4
        for (int m = 1; m < a.ctiles; m++) {
            load_pack<float, Q>(a.gbc + m * per + q * Q, e);
#pragma unroll
            for (int i = 0; i < Q; i++) v[i] += e[i];
        }
        const unsigned g = j / (2 * a.N), k = j - g * 2 * a.N, c = k >= (unsigned)a.N;
        const hc_rows& o = c ? a.gC : a.gB;
        const long long at = b * o.batch + t * o.row + g * a.N + k - c * a.N;
#pragma unroll
        for (int i = 0; i < Q; i++) st<DT>(o.p, at + i, v[i]);
    }
}
template <int DT> void sum_bc(const ScanArgs& a, cudaStream_t st) {
    const bool four = a.N % 4 == 0;
    const long long n = (long long)a.B * a.L * a.G * 2 * a.N / (four ? 4 : 1);
    const long long blocks = (n + 255) / 256, most = 64LL * device_sm_count();
    const unsigned grid = (unsigned)(blocks < most ? blocks : most);
    if (four)
        launch_next(scan_bc_kernel<DT, 4>, grid, 256, 0, st, a);
    else
        launch_next(scan_bc_kernel<DT, 1>, grid, 256, 0, st, a);
}

// One token: NL lanes a channel, 32 / NL channels a warp.  Reads and writes the
// states.  64 x 2048 x 16 (17 MB): replayed from a graph with the states in DRAM 7.3 us,
// 2.3 TB/s; called from Python with the states in L2 8.7 us, most of it the call.
// 2048 x 512 x 16 (134 MB): 48 us, 2.8 TB/s; bound by latency, one 16-byte load of states
// a thread in flight.
template <int NL, int DT>
__global__ void __launch_bounds__(128) scan_step_kernel(const __grid_constant__ ScanArgs a, float* state) {
    grid_begin();
    const int lane = threadIdx.x & 31, n = lane % NL;
    const long long q = (blockIdx.x * 4LL + (threadIdx.x >> 5)) * (32 / NL) + lane / NL;
    const bool on = q < (long long)a.B * a.Dm;
    const int b = on ? (int)(q / a.Dm) : 0, d = on ? (int)(q % a.Dm) : 0, g = d / a.Dg;
    float* hp = state + ((long long)b * a.Dm + d) * a.N;
    float h[4], A[4], B[4], C[4];
    ld_states(hp, 4 * n, a.N, h);
    ld_states(a.A + (long long)d * a.N, 4 * n, a.N, A);
#pragma unroll
    for (int k = 0; k < 4; k++) {
        const bool in = 4 * n + k < a.N;
        B[k] = in ? ld<DT>(a.Bm.p, b * a.Bm.batch + g * a.N + 4 * n + k) : 0.0f;
        C[k] = in ? ld<DT>(a.Cm.p, b * a.Cm.batch + g * a.N + 4 * n + k) : 0.0f;
    }
    const float u = ld<DT>(a.u.p, b * a.u.batch + d);
    float s = ld<DT>(a.dt.p, b * a.dt.batch + d) + (a.bias ? a.bias[d] : 0.0f);
    if (a.softplus) s = softplus_f(s);
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; k++) {
        h[k] = fmaf(ex2f(fmaf(s * kLog2e, A[k], kEx2Mean)), h[k], s * u * B[k]);
        y = fmaf(C[k], h[k], y);
    }
#pragma unroll
    for (int o = 1; o < NL; o <<= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (!on) return;
    st_states(hp, 4 * n, a.N, h);
    if (n == 0) {
        if (a.D) y = fmaf(a.D[d], u, y);
        if (a.z.p) y *= silu_f(ld<DT>(a.z.p, b * a.z.batch + d));
        st<DT>(a.y.p, b * a.y.batch + d, y);
    }
}

struct Step {
    const ScanArgs& a;
    float* state;
    cudaStream_t st;
    template <int NL, int DT> hc_status run() {
        launch_next(scan_step_kernel<NL, DT>, cdiv((long long)a.B * a.Dm, 4 * (32 / NL)), 128, 0, st, a, state);
        return launched("scan_step_kernel", st);
    }
};

hc_status launch_scan_bc(const ScanArgs& a, cudaStream_t st) {
    if (!a.gbc || a.L == 0) return HC_OK;
    if (a.dtype == HC_DTYPE_F32)
        sum_bc<HC_DTYPE_F32>(a, st);
    else if (a.dtype == HC_DTYPE_BF16)
        sum_bc<HC_DTYPE_BF16>(a, st);
    else
        sum_bc<HC_DTYPE_F16>(a, st);
    return launched("scan_bc_kernel", st);
}

bool scan_desc_ok(const hc_selective_scan_desc* d) {
    return d && d->B > 0 && d->L >= 0 && d->D > 0 && d->groups > 0 && d->D % d->groups == 0 && d->d_state > 0 &&
           (d->softplus == 0 || d->softplus == 1) && dtype_ok(d->dtype);
}
// Launch limits: (sequence, segment, channel tile) on grid x; segments are joined
// with sequences on grid y (scan_segs).
bool scan_size_ok(const hc_selective_scan_desc* d) {
    return d->d_state <= 64 && d->D <= (1 << 20) && (long long)d->B * d->D < (1LL << 31) && d->L <= 0x7fffffff - 64;
}
// Channel tiles a group in the forward and segment kernels, and in the backward kernel.
struct TileChannels {
    int fwd, bwd;
    template <int NL, int DT> hc_status run() {
        fwd = FwdTile<NL>::CT;
        bwd = BwdTile<NL>::CT;
        return HC_OK;
    }
};
int fwd_ctiles(const hc_selective_scan_desc* d) {
    TileChannels t;
    scan_dispatch(d->d_state, d->dtype, t);
    return (int)cdiv(d->D / d->groups, t.fwd);
}
int bwd_ctiles(const hc_selective_scan_desc* d) {
    TileChannels t;
    scan_dispatch(d->d_state, d->dtype, t);
    return (int)cdiv(d->D / d->groups, t.bwd);
}

// Segments: none where (sequence, channel tile) blocks give every SM a third of
// `want` of them or a sequence is short (a tile takes about a microsecond, the
// two extra launches as long as a dozen), else as many as make up for it, of two
// tiles at least.  Ragged sequences are cut twice as fine: blocks without rows end
// at once, and half of them have none where lengths are spread evenly.
// (16384 x 512 forward: cut for 4, 6, 8 blocks an SM 114, 105, 113 us; four of its blocks
// are resident at once, three of the backward kernel's.)
struct Segs {
    int n, tiles;
};
Segs scan_segs(const hc_selective_scan_desc* d, int ctiles, int want, bool ragged) {
    const int tiles = (int)cdiv(d->L, SC_T);
    const long long blocks = (long long)d->B * d->groups * ctiles;
    const long long full = (long long)want * device_sm_count() * (ragged ? 2 : 1);
    // (more than 65535 sequences, which the join's grid does not take, only an imposed SM count would cut)
    if (blocks * 3 > full || tiles < 16 || d->B > 65535) return {1, tiles > 0 ? tiles : 1};
    long long n = full / blocks;
    if (n > tiles / 2) n = tiles / 2;
    const int per = (int)cdiv(tiles, n);
    return {(int)cdiv(tiles, per), per};
}
Segs fwd_segs(const hc_selective_scan_desc* d, bool ragged) { return scan_segs(d, fwd_ctiles(d), 6, ragged); }
Segs bwd_segs(const hc_selective_scan_desc* d, bool ragged) { return scan_segs(d, bwd_ctiles(d), 3, ragged); }

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }
size_t carry_floats(const hc_selective_scan_desc* d, int segs) {
    return segs > 1 ? (size_t)d->B * segs * d->D * 4 * scan_lanes(d->d_state) : 0;
}
size_t carry_bytes(const hc_selective_scan_desc* d, int segs) {
    return up256(4 * carry_floats(d, segs)) + up256(segs > 1 ? 4 * (size_t)d->B * segs * d->D : 0);
}
size_t part_bytes(const hc_selective_scan_desc* d) {
    return up256(sizeof(float) * d->B * bwd_segs(d, true).n * (size_t)(d->d_state + 2) * d->D);
}
void set_segs(ScanArgs& a, const hc_selective_scan_desc* d, Segs s, void* ws) {
    a.segs = s.n;
    a.seg_tiles = s.tiles;
    a.carry = (float*)ws;
    a.dsum = (float*)((char*)ws + up256(4 * carry_floats(d, s.n)));
}

ScanArgs scan_args(const hc_selective_scan_desc* d, const hc_scan_in* in) {
    ScanArgs a = {};
    a.u = in->u;
    a.dt = in->dt;
    a.Bm = in->Bm;
    a.Cm = in->Cm;
    a.z = in->z;
    a.A = in->A;
    a.D = in->D;
    a.bias = in->dt_bias;
    a.B = d->B;
    a.L = d->L;
    a.Dm = d->D;
    a.G = d->groups;
    a.Dg = d->D / d->groups;
    a.N = d->d_state;
    a.dtype = d->dtype;
    a.softplus = d->softplus;
    a.tiles = (int)cdiv(d->L, SC_T);
    a.ctiles = fwd_ctiles(d);
    return a;
}

bool scan_in_ok(const hc_selective_scan_desc* d, const hc_scan_in* in, long long rows) {
    return in && rows_in_ok(&in->u, d->dtype, rows) && rows_in_ok(&in->dt, d->dtype, rows) &&
           rows_in_ok(&in->Bm, d->dtype, rows) && rows_in_ok(&in->Cm, d->dtype, rows) &&
           (!in->z.p || rows_in_ok(&in->z, d->dtype, rows)) && f32_ok(in->A) && f32_opt_ok(in->D) &&
           f32_opt_ok(in->dt_bias);
}

bool vec4(const ScanArgs& a) {
    for (const hc_rows* r : {&a.u, &a.dt, &a.z, &a.y, &a.gy, &a.gu, &a.gdt, &a.gz})
        if (!rows_vec(r, 4)) return false;
    return a.Dg % 4 == 0;
}

}  // namespace
}  // namespace hc

using namespace hc;

extern "C" {

// Workspace: forward [segment states][segment step sums]; backward the same two,
// [gA, gD, gdt_bias sums][gB, gC sums of each channel tile, where a group has
// several].
hc_status hc_selective_scan_workspace_size(const hc_selective_scan_desc* d, int pass, size_t* bytes) {
    if (!scan_desc_ok(d) || pass < 0 || pass > 1 || !bytes) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = carry_bytes(d, fwd_segs(d, true).n);  // the finer cut
    if (pass == 1) {
        const int tiles = bwd_ctiles(d);
        size_t b = carry_bytes(d, bwd_segs(d, true).n) + part_bytes(d);
        if (tiles > 1) b += sizeof(float) * tiles * (size_t)d->B * d->L * d->groups * 2 * d->d_state;
        if (b > *bytes) *bytes = b;
    }
    return HC_OK;
}

hc_status hc_selective_scan_saved_size(const hc_selective_scan_desc* d, size_t* bytes) {
    if (!scan_desc_ok(d) || !bytes) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    *bytes = sizeof(float) * (size_t)d->B * cdiv(d->L, SC_T) * d->D * 4 * scan_lanes(d->d_state);
    return HC_OK;
}

hc_status hc_selective_scan_fwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const hc_rows* y, float* hT, void* saved, void* ws, size_t ws_bytes,
                                void* stream) {
    size_t need = 0;
    hc_status e = hc_selective_scan_workspace_size(d, 0, &need);
    if (e) return e;
    if (!scan_in_ok(d, in, d->L) || !rows_out_ok(y, d->dtype, d->B, d->L, d->D) || !f32_opt_ok(h0) ||
        !f32_opt_ok(hT) || (h0 && h0 == hT) || !f32_opt_ok(saved) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z})
        if (rows_same(y, r)) return HC_ERR_INVALID_ARG;
    if (need && (!f32_ok(ws) || ws_bytes < need)) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    const cudaStream_t st = (cudaStream_t)stream;
    ScanArgs a = scan_args(d, in);
    a.y = *y;
    a.h0 = h0;
    a.hT = hT;
    a.lens = lens;
    a.saved = (float*)saved;
    a.vec = vec4(a);
    set_segs(a, d, fwd_segs(d, lens != nullptr), ws);
    if (a.segs > 1 && (e = launch_scan_carry(a, false, st))) return e;
    return launch_scan_fwd(a, st);
}

hc_status hc_selective_scan_bwd(const hc_selective_scan_desc* d, const hc_scan_in* in, const float* h0,
                                const int* lens, const void* saved, const hc_rows* gy, const float* ghT,
                                const hc_scan_grad* g, void* ws, size_t ws_bytes, void* stream) {
    size_t need = 0;
    hc_status e = hc_selective_scan_workspace_size(d, 1, &need);
    if (e) return e;
    if (!scan_in_ok(d, in, d->L) || !g || !rows_in_ok(gy, d->dtype, d->L) || (d->L > 0 && !f32_ok(saved)) ||
        !f32_opt_ok(h0) || !f32_opt_ok(ghT) || !f32_ok(g->gA) || !f32_opt_ok(g->gD) || !f32_opt_ok(g->gdt_bias) ||
        !f32_opt_ok(g->gh0) || (ghT && ghT == g->gh0) || !ptr_al(lens, 4))
        return HC_ERR_INVALID_ARG;
    const long long shared = (long long)d->groups * d->d_state;
    if (!rows_out_ok(&g->gu, d->dtype, d->B, d->L, d->D) || !rows_out_ok(&g->gdt, d->dtype, d->B, d->L, d->D) ||
        !rows_out_ok(&g->gB, d->dtype, d->B, d->L, shared) || !rows_out_ok(&g->gC, d->dtype, d->B, d->L, shared) ||
        (d->L > 0 && (in->z.p != nullptr) != (g->gz.p != nullptr)) ||
        (g->gz.p && !rows_out_ok(&g->gz, d->dtype, d->B, d->L, d->D)))
        return HC_ERR_INVALID_ARG;
    for (const hc_rows* o : {&g->gu, &g->gdt, &g->gB, &g->gC, &g->gz})
        for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z, gy})
            if (rows_same(o, r)) return HC_ERR_INVALID_ARG;
    if (!f32_ok(ws) || ws_bytes < need) return HC_ERR_WORKSPACE;
    traced_begin((cudaStream_t)stream);
    const cudaStream_t st = (cudaStream_t)stream;
    ScanArgs a = scan_args(d, in);
    a.gy = *gy;
    a.gu = g->gu;
    a.gdt = g->gdt;
    a.gB = g->gB;
    a.gC = g->gC;
    a.gz = g->gz;
    a.ghT = ghT;
    a.gh0 = g->gh0;
    a.lens = lens;
    a.saved = (float*)saved;
    a.vec = vec4(a);
    set_segs(a, d, bwd_segs(d, lens != nullptr), ws);
    const size_t carried = carry_bytes(d, bwd_segs(d, true).n);
    a.part = (float*)((char*)ws + carried);
    a.gbc = bwd_ctiles(d) > 1 ? (float*)((char*)ws + carried + part_bytes(d)) : nullptr;
    if (a.segs > 1 && (e = launch_scan_carry(a, true, st))) return e;
    a.ctiles = bwd_ctiles(d);
    if ((e = launch_scan_bwd(a, st)) || (e = launch_scan_bc(a, st))) return e;
    return launch_column_totals(a.part, (long long)a.B * a.segs, g->gA, a.Dm * a.N, g->gD, a.Dm, g->gdt_bias, a.Dm, st);
}

hc_status hc_selective_scan_step(const hc_selective_scan_desc* d, const hc_scan_in* in, float* state, const hc_rows* y,
                                 void* stream) {
    if (!scan_desc_ok(d)) return HC_ERR_INVALID_ARG;
    if (!scan_size_ok(d)) return HC_ERR_UNSUPPORTED;
    if (!scan_in_ok(d, in, 1) || !rows_out_ok(y, d->dtype, d->B, 1, d->D) || !f32_ok(state)) return HC_ERR_INVALID_ARG;
    for (const hc_rows* r : {&in->u, &in->dt, &in->Bm, &in->Cm, &in->z})
        if (rows_same(y, r)) return HC_ERR_INVALID_ARG;
    traced_begin((cudaStream_t)stream);
    ScanArgs a = scan_args(d, in);
    a.y = *y;
    Step f{a, state, (cudaStream_t)stream};
    return scan_dispatch(d->d_state, d->dtype, f);
}

}  // extern "C"
