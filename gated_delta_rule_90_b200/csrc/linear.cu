// Linear attention with a decay for each head: entry points, workspace, the
// cut of packed batches into blocks, the carry of the states over the blocks,
// and the sums over shared heads and over tokens.
#include "linear.cuh"

namespace gdr {
namespace lin {

// ------------------------------------------------------------ plan (packed batches)
// Exclusive block scan of x over 1024 threads (max or sum), plus the total.
template <bool MAX>
__device__ __forceinline__ int block_scan(int x, int *warp_tot, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc = MAX ? max(inc, y) : inc + y;
    }
    if (lane == 31) warp_tot[warp] = inc;
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < 32; ++w) {
        if (w == warp) before = all;
        all = MAX ? max(all, warp_tot[w]) : all + warp_tot[w];
    }
    __syncthreads();
    *total = all;
    int exc = __shfl_up_sync(0xffffffffu, inc, 1);
    if (lane == 0) exc = 0;
    return MAX ? max(before, exc) : before + exc;
}

// One CTA.  Offsets are taken as their running maximum inside [0, rows], so
// sequences never overlap and the slots always suffice.  `start` is scratch:
// the sequences' first rows.  The runs of the slots are filled in where there are any.
__global__ void __launch_bounds__(1024)
plan_kernel(const int32_t *cu, Geo geo, int4 *slot,
            int *blk_start, int *start, Runs runs) {
    stream_order();
    __shared__ int wt[32];
    const int tid = threadIdx.x;
    int hi = 0, nblk = 0;  // carried over tiles of 1024 sequences
    for (int base = 0; base < geo.n_seq; base += 1024) {
        const int s = base + tid;
        const int a = s < geo.n_seq ? min(max(cu[s], 0), geo.rows) : 0;
        const int b = s < geo.n_seq ? min(max(cu[s + 1], 0), geo.rows) : 0;
        int top, add;
        const int m = max(block_scan<true>(max(a, b), wt, &top), hi);
        const int t0 = max(m, a), t1 = max(t0, b);
        const int n = s < geo.n_seq ? max((t1 - t0 + geo.L - 1) / geo.L, geo.keep_empty) : 0;
        const int at = nblk + block_scan<false>(n, wt, &add);
        if (s < geo.n_seq) {
            blk_start[s] = at;
            start[2 * s] = t0;
            start[2 * s + 1] = t1;
        }
        hi = max(hi, top);
        nblk += add;
    }
    if (tid == 0) blk_start[geo.n_seq] = nblk;
    for (int i = tid; i < runs.count; i += 1024) runs.of[i] = make_int2(-1, 0);
    __syncthreads();  // read, and runs overwritten, by other threads of this CTA below
    for (int i = tid; i < geo.n_slots; i += 1024) {
        int4 r = make_int4(0, -1, 0, 0);
        if (i < nblk) {
            int lo = 0, up = geo.n_seq - 1;  // the last sequence with blk_start <= i
            while (lo < up) {
                const int mid = (lo + up + 1) >> 1;
                if (blk_start[mid] <= i) lo = mid; else up = mid - 1;
            }
            const int b = i - blk_start[lo], t0 = start[2 * lo] + b * geo.L;
            r = make_int4(t0, min(geo.L, start[2 * lo + 1] - t0), lo, b);
        }
        slot[i] = r;
        if (runs.count)
            for (int j = 0, u = run_of(geo, runs, r.x, i); j * kRunLen < r.y; ++j) runs.of[u + j] = make_int2(i, j);
    }
}

// ------------------------------------------------------------ carry over the blocks
// Elementwise in the state: S <- e^{gtot} S + X over the blocks of one
// (sequence, head), leaving in X the state that enters each block.  HBM-bound:
// X is read and written once.  A thread holds 4 elements; loads run 4 blocks
// ahead of the carry.
struct ScanArgs {
    float *X;
    const float *gtot, *init;
    float *fin;
};
template <bool REV>
__device__ __forceinline__ void scan(const ScanArgs &p, const Geo &geo, const Plan &plan, int nel,
                                     unsigned int *err) {
    float *__restrict__ X = p.X;
    const float *__restrict__ gtot = p.gtot, *__restrict__ init = p.init;
    float *__restrict__ fin = p.fin;
    const int s = blockIdx.x / geo.H, h = blockIdx.x - s * geo.H;
    const int el = (blockIdx.y * 256 + threadIdx.x) * 4;
    const int first = geo.varlen ? plan.blk_start[s] : s * geo.nb;
    const int nb = (geo.varlen ? plan.blk_start[s + 1] : first + geo.nb) - first;
    if (kChecked && !chk_span(first, nb, geo.n_slots, err)) return;
    if (el >= nel || (geo.skip_single && nb == 1)) return;
    const size_t so = ((size_t)s * geo.H + h) * nel + el;
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (init) S = *reinterpret_cast<const float4 *>(init + so);
    constexpr int kAhead = 4;
    for (int b0 = 0; b0 < nb; b0 += kAhead) {
        float4 x[kAhead];
        float a[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (b0 + u < nb) {
                const size_t sh = (size_t)(first + (REV ? nb - 1 - b0 - u : b0 + u)) * geo.H + h;
                x[u] = *reinterpret_cast<const float4 *>(X + sh * nel + el);
                a[u] = expf(gtot[sh]);
            }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (b0 + u < nb) {
                const size_t sh = (size_t)(first + (REV ? nb - 1 - b0 - u : b0 + u)) * geo.H + h;
                *reinterpret_cast<float4 *>(X + sh * nel + el) = S;
                S.x = fmaf(a[u], S.x, x[u].x);
                S.y = fmaf(a[u], S.y, x[u].y);
                S.z = fmaf(a[u], S.z, x[u].z);
                S.w = fmaf(a[u], S.w, x[u].w);
            }
    }
    if (fin) *reinterpret_cast<float4 *>(fin + so) = S;
}
// forward in time (blockIdx.z below nf), then backward
__global__ void __launch_bounds__(256)
scan_kernel(ScanArgs f, ScanArgs r, int nf, Geo geo, Plan plan, int nel, unsigned int *err) {
    stream_order();
    if ((int)blockIdx.z < nf)
        scan<false>(f, geo, plan, nel, err);
    else
        scan<true>(r, geo, plan, nel, err);
}

// ------------------------------------------------------------ sums
// The gradient of a shared query/key head: the sum over its value heads, fp32.
// A CTA takes 16 tokens of a slot at a time.
constexpr int kSumRows = 16;
template <typename T>
__global__ void __launch_bounds__(256)
group_sum_kernel(const float *x, T *out, Geo geo, Plan plan, int d) {
    stream_order();
    // slot by slot, so that rows of no sequence are left as they are
    const int4 sl = slot_of(geo, plan, blockIdx.x);
    const int r = geo.H / geo.Hk, per = geo.Hk * (d / 4);
    for (int j0 = blockIdx.y * kSumRows; j0 < sl.y; j0 += gridDim.y * kSumRows)
    for (int i = threadIdx.x; i < min(kSumRows, sl.y - j0) * per; i += 256) {
        const long row = sl.x + j0 + i / per;
        const int hk = (i % per) / (d / 4), d4 = (i % per) % (d / 4);
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = 0; j < r; ++j) {
            const float4 y = *reinterpret_cast<const float4 *>(
                x + ((size_t)row * geo.H + hk * r + j) * d + 4 * d4);
            s.x += y.x; s.y += y.y; s.z += y.z; s.w += y.w;
        }
        const size_t o = ((size_t)row * geo.Hk + hk) * d + 4 * d4;
        st_out(out, o, s.x);
        st_out(out, o + 1, s.y);
        st_out(out, o + 2, s.z);
        st_out(out, o + 3, s.w);
    }
}

// GDR_GATE_HEAD: dg of a head from its slots' sums, in a fixed order, 64 bits.
__global__ void __launch_bounds__(256)
dg_heads_kernel(const float *part, float *dg, Geo geo) {
    stream_order();
    __shared__ double red[256];
    double s = 0.0;
    for (int i = threadIdx.x; i < geo.n_slots; i += 256) s += part[(size_t)i * geo.H + blockIdx.x];
    red[threadIdx.x] = s;
    __syncthreads();
    for (int o = 128; o; o >>= 1) {
        if (threadIdx.x < o) red[threadIdx.x] += red[threadIdx.x + o];
        __syncthreads();
    }
    if (threadIdx.x == 0) dg[blockIdx.x] = (float)red[0];
}

// ------------------------------------------------------------ decode
// S <- a S + v k^T, o = S q for one token of each (sequence, head).  A row of S
// (d_k floats) needs only its own v_i, so LPR lanes take a row (VPL 16-byte
// vectors each), 32 / LPR rows a warp, and one shuffle reduction gives o_i.
// HBM-bound: the state is read and written once, kRows rows of a warp are in
// flight before any is used.
constexpr int kDecThreads = 128;

template <typename T, int VPL, int LPR>
__global__ void __launch_bounds__(kDecThreads)
decode_kernel(const T *__restrict__ q, const T *__restrict__ k, const T *__restrict__ v,
              const float *__restrict__ g, float *__restrict__ S, T *__restrict__ out, int H, int Hk,
              int dv, int rows, int gate_head, long long nheads, unsigned int *err) {
    constexpr int DK = 4 * VPL * LPR, RPW = 32 / LPR;  // rows a warp takes at a time
    constexpr int INF = VPL >= 4 ? 2 : VPL >= 2 ? 4 : 8;
    const size_t head = blockIdx.x;  // flattened (sequence, head)
    const size_t n = head / H;
    const int h = (int)(head - n * H);
    const size_t hq = n * Hk + h / (H / Hk);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sub = lane % LPR, rl = lane / LPR;
    const int r0 = blockIdx.y * rows, r1 = min(dv, r0 + rows);
    if (kChecked) {
        const long long hd = (long long)head;
        if (!(chk_span(hd, 1, nheads, err) && chk_span(r0, r1 - r0, dv, err))) return;
    }
    float4 kk[VPL], qq[VPL];
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        const size_t o = hq * DK + 4 * (sub + LPR * i);
        kk[i] = make_float4(ld_in(k, o), ld_in(k, o + 1), ld_in(k, o + 2), ld_in(k, o + 3));
        qq[i] = make_float4(ld_in(q, o), ld_in(q, o + 1), ld_in(q, o + 2), ld_in(q, o + 3));
    }
    const float a = expf(clamp_g(gate_head ? g[h] : g[head]));
    float *Sh = S + head * (size_t)dv * DK;
    const int step = RPW * (kDecThreads / 32);
    for (int rb = r0 + warp * RPW + rl; rb - rl < r1; rb += step * INF) {
        float4 x[INF][VPL];
        float vi[INF];
#pragma unroll
        for (int u = 0; u < INF; ++u) {
            const int r = rb + u * step;
            if (r < r1) {
                vi[u] = ld_in(v, head * dv + r);
#pragma unroll
                for (int i = 0; i < VPL; ++i)
                    x[u][i] = __ldcs(reinterpret_cast<const float4 *>(Sh + (size_t)r * DK) + sub + LPR * i);
            }
        }
#pragma unroll
        for (int u = 0; u < INF; ++u) {
            const int r = rb + u * step;
            float o = 0.f;
            if (r < r1) {
#pragma unroll
                for (int i = 0; i < VPL; ++i) {
                    float4 y = x[u][i];
                    y.x = fmaf(vi[u], kk[i].x, a * y.x);
                    y.y = fmaf(vi[u], kk[i].y, a * y.y);
                    y.z = fmaf(vi[u], kk[i].z, a * y.z);
                    y.w = fmaf(vi[u], kk[i].w, a * y.w);
                    o = fmaf(y.x, qq[i].x, fmaf(y.y, qq[i].y, fmaf(y.z, qq[i].z, fmaf(y.w, qq[i].w, o))));
                    __stcs(reinterpret_cast<float4 *>(Sh + (size_t)r * DK) + sub + LPR * i, y);
                }
            }
#pragma unroll
            for (int s = LPR / 2; s; s >>= 1) o += __shfl_xor_sync(0xffffffffu, o, s);
            if (r < r1 && sub == 0) st_out(out, head * dv + r, o);
        }
    }
}

}  // namespace lin
}  // namespace gdr

// ====================================================================== host side
using namespace gdr;
using namespace gdr::lin;
using gdr_host::LinCall;
using gdr_host::LinWs;

namespace {

bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
bool dim_ok(int d) { return d >= 16 && d <= 128 && d % 16 == 0; }

gdr_status check_types(int H, int Hk, int dk, int dv, gdr_dtype dtype, gdr_gate gate) {
    if ((dtype != GDR_F32 && dtype != GDR_BF16) || gate < GDR_GATE_SCALAR || gate > GDR_GATE_HEAD)
        return GDR_ERR_INVALID;
    if (H < 1 || Hk < 1 || H % Hk || dk < 1 || dv < 1) return GDR_ERR_INVALID;
    if (gate == GDR_GATE_PER_KEY_CHANNEL || !dim_ok(dk) || !dim_ok(dv) || H > 65535)
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

gdr_status check_shapes(int B, int T, int H, int Hk, int dk, int dv, int n_seq, bool varlen,
                        gdr_dtype dtype, gdr_gate gate, gdr_path path) {
    if (B < 1 || T < 0 || (varlen && (B != 1 || n_seq < 1))) return GDR_ERR_INVALID;
    if (path != GDR_PATH_AUTO && path != GDR_PATH_SIMT && path != GDR_PATH_TENSORCORE)
        return GDR_ERR_INVALID;
    const gdr_status st = check_types(H, Hk, dk, dv, dtype, gate);
    if (st != GDR_OK) return st;
    const double n = varlen ? n_seq : B;
    // rows, and walks (blocks of at least 128 tokens, heads, two column groups), are counted in 32 bits
    if ((double)B * T > 2.0e9 || n * H > 2.0e9 || ((double)B * T / 128 + n) * H * 2 > 2.1e9)
        return GDR_ERR_INVALID;
    return GDR_OK;
}

// Does the call run on the tensor cores?
gdr_status resolve(int T, gdr_dtype dtype, gdr_path path, bool *tc) {
    *tc = dtype == GDR_BF16 && path != GDR_PATH_SIMT && T > 0;
    return path == GDR_PATH_TENSORCORE && dtype != GDR_BF16 ? GDR_ERR_UNSUPPORTED : GDR_OK;
}

// What the size functions answer: 0 stands for a refused call, so a call of no tokens is given
// a size as well, though it takes NULL.
size_t ask(size_t need) { return need ? need : 256; }

template <typename T, int VPL, int LPR>
cudaError_t launch_decode(const LinCall &c) {
    // Rows of a head go to several CTAs while there are few heads: one CTA
    // takes 32 rows until the heads alone fill the GPU's 148 SMs four times.
    const long long nh = (long long)c.B * c.H;
    const int rows = nh < 4 * 148 ? 32 : c.dv_;
    decode_kernel<T, VPL, LPR><<<dim3((unsigned)nh, (c.dv_ + rows - 1) / rows), kDecThreads, 0, c.st>>>(
        (const T *)c.q, (const T *)c.k, (const T *)c.v, c.g, c.S_final, (T *)c.out, c.H, c.Hk, c.dv_,
        rows, c.gate == GDR_GATE_HEAD, nh, c.err);
    return cudaGetLastError();
}

template <typename T>
cudaError_t decode_t(const LinCall &c) {
    switch (c.dk_) {  // d_k = 4 VPL LPR
        case 16: return launch_decode<T, 1, 4>(c);
        case 32: return launch_decode<T, 1, 8>(c);
        case 48: return launch_decode<T, 3, 4>(c);
        case 64: return launch_decode<T, 1, 16>(c);
        case 80: return launch_decode<T, 5, 4>(c);
        case 96: return launch_decode<T, 3, 8>(c);
        case 112: return launch_decode<T, 7, 4>(c);
        default: return launch_decode<T, 1, 32>(c);
    }
}

}  // namespace

namespace gdr_host {

LinWs lin_ws(int B, int T, int H, int Hk, int dk, int dv, int n_seq, bool varlen, bool bwd, int L,
             int dot_cols) {
    LinWs w{};
    w.L = L;
    w.nb = (T + L - 1) / L;
    w.n_slots = varlen ? T / L + n_seq : B * w.nb;
    const size_t rows = (size_t)B * T, sh = (size_t)w.n_slots * H, nel = (size_t)dk * dv;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += up256(bytes);
        return at;
    };
    w.slot = take(varlen ? sizeof(int4) * w.n_slots : 0);
    w.blk_start = take(varlen ? sizeof(int) * ((size_t)3 * n_seq + 1) : 0);
    w.gtot = take(sh * 4);
    w.X = take(sh * nel * 4);
    if (bwd) {
        w.Y = take(sh * nel * 4);
        w.fin = take((size_t)(varlen ? n_seq : B) * H * nel * 4);
        w.rdot = take(rows * H * dot_cols * 4);
        w.cdot = take(rows * H * dot_cols * 4);
        w.dq32 = take(Hk < H ? rows * H * dk * 4 : 0);
        w.dk32 = take(Hk < H ? rows * H * dk * 4 : 0);
        w.part = take(sh * 4);
    }
    w.total = o;
    return w;
}

Geo lin_geo(const LinCall &c, const LinWs &w) {
    Geo g{};
    g.T = c.T; g.H = c.H; g.Hk = c.Hk; g.n_seq = c.cu ? c.n_seq : c.B; g.varlen = c.cu != nullptr;
    g.rows = c.B * c.T; g.L = w.L; g.nb = w.nb; g.n_slots = w.n_slots;
    g.gate_head = c.gate == GDR_GATE_HEAD;
    return g;
}

cudaError_t lin_plan(const LinCall &c, const Geo &geo, const LinWs &w, const Runs &runs) {
    if (!geo.varlen) return cudaSuccess;
    int *bs = (int *)(c.ws + w.blk_start);
    ProfToken tk = prof_begin(GDR_K_LIN_PLAN, c.st);
    const cudaError_t le = lin_launch(plan_kernel, dim3(1), 1024, 0, c.st, c.cu, geo, (int4 *)(c.ws + w.slot),
                                      bs, bs + geo.n_seq + 1, runs);
    prof_end(tk, c.st);
    return le;
}

cudaError_t lin_scan(const LinCall &c, const Geo &geo, const LinWs &w, const LinScan *f, const LinScan *r) {
    if (!geo.n_slots && !(f && f->fin) && !(r && r->fin)) return cudaSuccess;
    const int nel = c.dk_ * c.dv_;
    const Plan plan = {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
    const dim3 grid((unsigned)(geo.n_seq * geo.H), (unsigned)((nel / 4 + 255) / 256), f && r ? 2 : 1);
    ScanArgs a{}, b{};
    if (f) a = {f->X, f->gtot, f->init, f->fin};
    if (r) b = {r->X, r->gtot, r->init, r->fin};
    ProfToken tk = prof_begin(GDR_K_LIN_SCAN, c.st);
    const cudaError_t le = lin_launch(scan_kernel, grid, 256, 0, c.st, a, b, f ? 1 : 0, geo, plan, nel, c.err);
    prof_end(tk, c.st);
    return le;
}

cudaError_t lin_group_sum(const LinCall &c, const Geo &geo, const LinWs &w, const float *x, void *out,
                          int d) {
    if (!geo.n_slots) return cudaSuccess;
    const Plan plan = {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
    const int rounds = (geo.L + kSumRows - 1) / kSumRows;
    const dim3 grid(geo.n_slots, rounds < 4096 ? rounds : 4096);
    ProfToken tk = prof_begin(GDR_K_LIN_SUM, c.st);
    const cudaError_t le =
        c.dtype == GDR_BF16
            ? lin_launch(group_sum_kernel<__nv_bfloat16>, grid, 256, 0, c.st, x, (__nv_bfloat16 *)out, geo,
                         plan, d)
            : lin_launch(group_sum_kernel<float>, grid, 256, 0, c.st, x, (float *)out, geo, plan, d);
    prof_end(tk, c.st);
    return le;
}

cudaError_t lin_dg_heads(const LinCall &c, const Geo &geo, const float *part) {
    ProfToken tk = prof_begin(GDR_K_LIN_SUM, c.st);
    const cudaError_t le = lin_launch(dg_heads_kernel, dim3(c.H), 256, 0, c.st, part, c.dg, geo);
    prof_end(tk, c.st);
    return le;
}

}  // namespace gdr_host

extern "C" {

size_t gdr_fwd_linear_workspace_size(int B, int T, int H, int H_k, int d_k, int d_v, int n_seq,
                                     int varlen, gdr_dtype dtype, gdr_gate gate, gdr_path path) {
    bool tc;
    if (check_shapes(B, T, H, H_k, d_k, d_v, n_seq, varlen != 0, dtype, gate, path) != GDR_OK ||
        resolve(T, dtype, path, &tc) != GDR_OK)
        return 0;
    LinCall c{};
    static const int32_t packed = 0;  // only whether cu is NULL matters here
    c.cu = varlen ? &packed : nullptr;
    c.B = B; c.T = T; c.H = H; c.Hk = H_k; c.dk_ = d_k; c.dv_ = d_v; c.n_seq = n_seq;
    return ask(tc ? gdr_host::lin_tc_ws_bytes(c, false) : gdr_host::lin_simt_ws_bytes(c, false));
}

size_t gdr_bwd_linear_workspace_size(int B, int T, int H, int H_k, int d_k, int d_v, int n_seq,
                                     int varlen, gdr_dtype dtype, gdr_gate gate, gdr_path path) {
    bool tc;
    if (check_shapes(B, T, H, H_k, d_k, d_v, n_seq, varlen != 0, dtype, gate, path) != GDR_OK ||
        resolve(T, dtype, path, &tc) != GDR_OK)
        return 0;
    LinCall c{};
    static const int32_t packed = 0;
    c.cu = varlen ? &packed : nullptr;
    c.B = B; c.T = T; c.H = H; c.Hk = H_k; c.dk_ = d_k; c.dv_ = d_v; c.n_seq = n_seq;
    return ask(tc ? gdr_host::lin_tc_ws_bytes(c, true) : gdr_host::lin_simt_ws_bytes(c, true));
}

gdr_status gdr_fwd_linear(const void *q, const void *k, const void *v, const float *g,
                          const float *S0, void *out, float *S_final, int B, int T, int H, int H_k,
                          int d_k, int d_v, const int32_t *cu_seqlens, int n_seq, gdr_dtype dtype,
                          gdr_gate gate, gdr_path path, void *workspace, size_t workspace_bytes,
                          void *stream) {
    // With no tokens (B*T == 0) the token tensors are empty and may be NULL.
    if ((long long)B * T > 0 && (!q || !k || !v || !g || !out)) return GDR_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(S0) ||
        !aligned16(out) || !aligned16(S_final) || !aligned16(cu_seqlens))
        return GDR_ERR_INVALID;
    gdr_status st = check_shapes(B, T, H, H_k, d_k, d_v, n_seq, cu_seqlens != nullptr, dtype, gate,
                                 path);
    if (st != GDR_OK) return st;
    bool tc = false;
    if ((st = resolve(T, dtype, path, &tc)) != GDR_OK) return st;
    LinCall c{};
    c.q = q; c.k = k; c.v = v; c.g = g; c.S0 = S0; c.out = out; c.S_final = S_final;
    c.cu = cu_seqlens; c.B = B; c.T = T; c.H = H; c.Hk = H_k; c.dk_ = d_k; c.dv_ = d_v;
    c.n_seq = n_seq; c.dtype = dtype; c.gate = gate; c.ws = (uint8_t *)workspace;
    c.st = (cudaStream_t)stream;
    const size_t need = tc ? gdr_host::lin_tc_ws_bytes(c, false) : gdr_host::lin_simt_ws_bytes(c, false);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)))
        return GDR_ERR_INVALID;
    c.err = gdr_host::device_error_word();
    if (!c.err) return GDR_ERR_CUDA;
    return (tc ? gdr_host::lin_fwd_tc(c) : gdr_host::lin_fwd_simt(c)) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

gdr_status gdr_decode_step_linear(const void *q, const void *k, const void *v, const float *g,
                                  float *S_inout, void *out, int N, int H, int H_k, int d_k, int d_v,
                                  gdr_dtype dtype, gdr_gate gate, void *stream) {
    if (!q || !k || !v || !g || !S_inout || !out) return GDR_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(S_inout) ||
        !aligned16(out))
        return GDR_ERR_INVALID;
    if (N < 1 || (double)N * H > 2.0e9) return GDR_ERR_INVALID;
    const gdr_status st = check_types(H, H_k, d_k, d_v, dtype, gate);
    if (st != GDR_OK) return st;
    LinCall c{};
    c.q = q; c.k = k; c.v = v; c.g = g; c.S_final = S_inout; c.out = out; c.B = N; c.H = H; c.Hk = H_k;
    c.dk_ = d_k; c.dv_ = d_v; c.dtype = dtype; c.gate = gate; c.st = (cudaStream_t)stream;
    c.err = gdr::kChecked ? gdr_host::device_error_word() : nullptr;
    gdr_host::ProfToken tk = gdr_host::prof_begin(GDR_K_LIN_DECODE, c.st);
    const cudaError_t e = dtype == GDR_BF16 ? decode_t<__nv_bfloat16>(c) : decode_t<float>(c);
    gdr_host::prof_end(tk, c.st);
    return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

gdr_status gdr_bwd_linear(const void *q, const void *k, const void *v, const float *g,
                          const float *S0, const void *dout, const float *dS_final, void *dq,
                          void *dk, void *dv, float *dg, float *dS0, int B, int T, int H, int H_k,
                          int d_k, int d_v, const int32_t *cu_seqlens, int n_seq, gdr_dtype dtype,
                          gdr_gate gate, gdr_path path, void *workspace, size_t workspace_bytes,
                          void *stream) {
    if ((long long)B * T > 0 && (!q || !k || !v || !g || !dout || !dq || !dk || !dv || !dg))
        return GDR_ERR_INVALID;
    if (gate == GDR_GATE_HEAD && !dg) return GDR_ERR_INVALID;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(g) || !aligned16(S0) ||
        !aligned16(dout) || !aligned16(dS_final) || !aligned16(dq) || !aligned16(dk) ||
        !aligned16(dv) || !aligned16(dg) || !aligned16(dS0) || !aligned16(cu_seqlens))
        return GDR_ERR_INVALID;
    gdr_status st = check_shapes(B, T, H, H_k, d_k, d_v, n_seq, cu_seqlens != nullptr, dtype, gate,
                                 path);
    if (st != GDR_OK) return st;
    bool tc = false;
    if ((st = resolve(T, dtype, path, &tc)) != GDR_OK) return st;
    LinCall c{};
    c.q = q; c.k = k; c.v = v; c.g = g; c.S0 = S0; c.dout = dout; c.dS_final = dS_final;
    c.dq = dq; c.dk = dk; c.dv = dv; c.dg = dg; c.dS0 = dS0;
    c.cu = cu_seqlens; c.B = B; c.T = T; c.H = H; c.Hk = H_k; c.dk_ = d_k; c.dv_ = d_v;
    c.n_seq = n_seq; c.dtype = dtype; c.gate = gate; c.ws = (uint8_t *)workspace;
    c.st = (cudaStream_t)stream;
    const size_t need = tc ? gdr_host::lin_tc_ws_bytes(c, true) : gdr_host::lin_simt_ws_bytes(c, true);
    if (need && (!workspace || workspace_bytes < need || ((uintptr_t)workspace & 255u)))
        return GDR_ERR_INVALID;
    c.err = gdr_host::device_error_word();
    if (!c.err) return GDR_ERR_CUDA;
    return (tc ? gdr_host::lin_bwd_tc(c) : gdr_host::lin_bwd_simt(c)) == cudaSuccess ? GDR_OK : GDR_ERR_CUDA;
}

}  // extern "C"
