// Linear attention with a decay for each head on the CUDA cores, fp32: any
// token type, d_k and d_v multiples of 16 up to 128, forward and gradient.
//
// One operator serves all of it.  With roles a, b (d_b wide) and c (d_c wide),
//     out_i = sum_{j <= i} e^{G_i - G_j} (a_i . b_j) c_j + e^{G_i} X a_i,
//     X    <- e^{G_n} X + sum_j e^{G_n - G_j} c_j b_j^T
// (G: running sum of the log-decays) is the forward pass for (a, b, c) =
// (q, k, v), X = S, and gives dq for (dout, v, k), X = S^T.  Run backward in
// time (pairs j >= i, weights e^{G_j - G_i}, X the gradient of the state that
// leaves the block) it gives dv for (k, q, dout), X = dS, and dk for
// (v, dout, q), X = dS^T.
//
// The gradient of the log-decays: with R_t = q_t . dq_t and C_t = v_t . dv_t
// (= k_t . dk_t),
//     dg_t = sum_{s >= t, s in block} (R_s - C_s) + <S_end, dS_end>,
// S_end and dS_end the state after the block and its gradient.  Starting the
// sum again in each block of 256 keeps its rounding from growing with the
// sequence.
//
// Blocks of up to 256 tokens run in parallel: their own contribution to the state
// (state_kernel), the carry over the blocks (lin_scan), the outputs (out_kernel,
// grad_kernel, 32-token chunks in order).
#include "linear.cuh"

namespace gdr {
namespace lin {

constexpr int kThreads = 256;
constexpr int kC = 32;     // tokens of a chunk
constexpr int kNb = 32;    // columns of c (rows of X) of a CTA
constexpr int kBlk = gdr_host::kLinSimtL;

__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
    const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
    return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float s) {
    return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
}

// sG[i] = sum of the block's first i log-decays, in 64 bits: differences of
// far positions are rounded once, not at the size of the sums.
__device__ __forceinline__ void block_decays(const Geo &geo, const float *g, long t0, int len,
                                             int h, double *sG) {
    __shared__ double wsum[kThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    double x = tid < len ? (double)load_g(geo, g, t0 + tid, h) : 0.0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) wsum[warp] = x;
    __syncthreads();
    for (int w = 0; w < warp; ++w) x += wsum[w];
    sG[tid + 1] = x;
    if (tid == 0) sG[0] = 0.0;
    __syncthreads();
}

// ------------------------------------------------------------ block states
// X[slot, head] = sum_j w_j c_j b_j^T over the block, w_j = e^{G_n - G_j}
// (forward: b, c = k, v) or e^{G_j} (REV: b, c = q, dout); rows are value
// channels, columns key channels.  A thread holds a 4 x 4 tile; per token two
// 16-byte shared reads feed 16 FMAs.
template <typename T>
struct StateArgs {
    const T *b, *c;
    float *X;
};
template <typename T, bool REV>
__device__ __forceinline__ void block_state(const StateArgs<T> &p, int z, const float *g,
                                            float *gtot, const Geo &geo, const Plan &plan, int db,
                                            int dc, unsigned int *err) {
    const T *__restrict__ b = p.b, *__restrict__ c = p.c;
    float *__restrict__ X = p.X;
    __shared__ double sG[kBlk + 1];
    __shared__ __align__(16) float sb[kC * 128];
    __shared__ __align__(16) float sc[kC * kNb];
    const int slot = blockIdx.x, h = blockIdx.y, c0 = z * kNb, tid = threadIdx.x;
    const int4 sl = slot_of(geo, plan, slot);
    const long t0 = sl.x;
    const int len = sl.y;
    if (len <= 0) return;
    if (kChecked && !(chk_span(t0, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err) &&
                      chk_true(len <= kBlk && c0 < dc, err)))
        return;
    const int hb = h / (geo.H / geo.Hk);
    block_decays(geo, g, t0, len, h, sG);
    const int rg = tid >> 5, cg = tid & 31;
    float x[4][4] = {};
    for (int j0 = 0; j0 < len; j0 += kC) {
        const int n = min(kC, len - j0);
        for (int i = tid; i < n * (db / 4); i += kThreads) {
            const int j = i / (db / 4), d4 = i - j * (db / 4);
            reinterpret_cast<float4 *>(sb)[j * 32 + d4] =
                load4(b + ((t0 + j0 + j) * geo.Hk + hb) * db + 4 * d4);
        }
        for (int i = tid; i < n * (kNb / 4); i += kThreads) {
            const int j = i / (kNb / 4), q4 = i % (kNb / 4);
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (c0 + 4 * q4 < dc) {
                y = load4(c + ((t0 + j0 + j) * geo.H + h) * dc + c0 + 4 * q4);
                const float w = expf((float)(REV ? sG[j0 + j + 1] : sG[len] - sG[j0 + j + 1]));
                y.x *= w; y.y *= w; y.z *= w; y.w *= w;
            }
            reinterpret_cast<float4 *>(sc)[j * (kNb / 4) + q4] = y;
        }
        __syncthreads();
        if (4 * cg < db) {
            for (int j = 0; j < n; ++j) {
                const float4 cv = reinterpret_cast<const float4 *>(sc)[j * (kNb / 4) + rg];
                const float4 bv = reinterpret_cast<const float4 *>(sb)[j * 32 + cg];
                const float ca[4] = {cv.x, cv.y, cv.z, cv.w}, ba[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int s = 0; s < 4; ++s) x[r][s] = fmaf(ca[r], ba[s], x[r][s]);
            }
        }
        __syncthreads();
    }
    float *Xh = X + ((size_t)slot * geo.H + h) * dc * db;
    if (4 * cg < db) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int row = c0 + 4 * rg + r;
            if (row < dc)
                *reinterpret_cast<float4 *>(Xh + (size_t)row * db + 4 * cg) =
                    make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
        }
    }
    if (c0 == 0 && tid == 0 && gtot) gtot[(size_t)slot * geo.H + h] = (float)sG[len];
}

// forward (blockIdx.z below nz), then reverse
template <typename T>
__global__ void __launch_bounds__(kThreads)
state_kernel(StateArgs<T> f, StateArgs<T> r, int nz, const float *g, float *gtot,
             Geo geo, Plan plan, int db, int dc, unsigned int *err) {
    stream_order();
    const int z = blockIdx.z;
    if (z < nz)
        block_state<T, false>(f, z, g, gtot, geo, plan, db, dc, err);
    else
        block_state<T, true>(r, z - nz, g, nullptr, geo, plan, db, dc, err);
}

// ------------------------------------------------------------ outputs
template <typename T>
struct Roles {
    const T *a, *b, *c, *e;  // e: the rows that out is dotted with, or NULL
    int ha, hb, hc, he;      // their heads
    int db, dc;
    bool tr;                 // X is the transpose of the stored [d_v, d_k] state
    const float *X;
    void *out;
    float *dots;
};

template <typename T, typename To, bool REV>
__device__ __forceinline__ void outputs(const Roles<T> &ro, int z, const float *g, const Geo &geo,
                                        const Plan &plan, unsigned int *err) {
    const float *__restrict__ X = ro.X;
    To *__restrict__ out = (To *)ro.out;
    float *__restrict__ dots = ro.dots;
    extern __shared__ __align__(16) float sm[];
    __shared__ double sG[kBlk + 1];
    __shared__ float sInter[kC], sW[kC];
    const int db = ro.db, dc = ro.dc, lda = db + 4;
    constexpr int ldc = kC + 4;
    float *sa = sm, *sb = sa + kC * lda, *sX = sb + kC * lda;
    float *sP = sX + kNb * lda, *sc = sP + kC * ldc, *sct = sc + kC * ldc;
    const int slot = blockIdx.x, h = blockIdx.y, c0 = z * kNb, tid = threadIdx.x;
    const int4 sl = slot_of(geo, plan, slot);
    const long t0 = sl.x;
    const int len = sl.y;
    if (len <= 0) return;
    if (kChecked && !(chk_span(t0, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err) &&
                      chk_true(len <= kBlk && c0 < dc, err)))
        return;
    const int ha = h / (geo.H / ro.ha), hb = h / (geo.H / ro.hb), hc = h / (geo.H / ro.hc);
    block_decays(geo, g, t0, len, h, sG);
    const float *Xh = X + ((size_t)slot * geo.H + h) * dc * db;
    for (int i = tid; i < kNb * db; i += kThreads) {
        int r, d;
        if (ro.tr) {
            d = i / kNb;
            r = i % kNb;
        } else {
            r = i / db;
            d = i - r * db;
        }
        const int row = c0 + r;
        sX[r * lda + d] = row < dc ? Xh[ro.tr ? (size_t)d * dc + row : (size_t)row * db + d] : 0.f;
    }
    const int ti = tid >> 4, tj = tid & 15;
    const int nch = (len + kC - 1) / kC;
    for (int cc = 0; cc < nch; ++cc) {
        const int j0 = (REV ? nch - 1 - cc : cc) * kC, n = min(kC, len - j0);
        __syncthreads();
        // rows past the end are zero, whatever memory holds there
        for (int i = tid; i < kC * (db / 4); i += kThreads) {
            const int j = i / (db / 4), d4 = i - j * (db / 4);
            float4 xa = make_float4(0.f, 0.f, 0.f, 0.f), xb = xa;
            if (j < n) {
                xa = load4(ro.a + ((t0 + j0 + j) * ro.ha + ha) * db + 4 * d4);
                xb = load4(ro.b + ((t0 + j0 + j) * ro.hb + hb) * db + 4 * d4);
            }
            *reinterpret_cast<float4 *>(sa + j * lda + 4 * d4) = xa;
            *reinterpret_cast<float4 *>(sb + j * lda + 4 * d4) = xb;
        }
        if (tid < kC) {
            const double Gi = sG[min(j0 + tid + 1, len)];
            sInter[tid] = expf((float)(REV ? sG[j0 + n] - Gi : Gi - sG[j0]));
            sW[tid] = expf((float)(REV ? Gi - sG[j0] : sG[j0 + n] - Gi));
        }
        {
            const int j = tid >> 3, q4 = tid & 7;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (j < n && c0 + 4 * q4 < dc)
                y = load4(ro.c + ((t0 + j0 + j) * ro.hc + hc) * dc + c0 + 4 * q4);
            *reinterpret_cast<float4 *>(sc + j * ldc + 4 * q4) = y;
            sct[(4 * q4) * ldc + j] = y.x;
            sct[(4 * q4 + 1) * ldc + j] = y.y;
            sct[(4 * q4 + 2) * ldc + j] = y.z;
            sct[(4 * q4 + 3) * ldc + j] = y.w;
        }
        __syncthreads();
        // pair weights times (a_i . b_j), and X a_i: rows ti, ti + 16; columns tj, tj + 16
        float p[2][2] = {}, o[2][2] = {};
        for (int d = 0; d < db; d += 4) {
            float4 xa[2], xb[2], xx[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                xa[r] = *reinterpret_cast<const float4 *>(sa + (ti + 16 * r) * lda + d);
                xb[r] = *reinterpret_cast<const float4 *>(sb + (tj + 16 * r) * lda + d);
                xx[r] = *reinterpret_cast<const float4 *>(sX + (tj + 16 * r) * lda + d);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    p[r][s] = dot4(xa[r], xb[s], p[r][s]);
                    o[r][s] = dot4(xa[r], xx[s], o[r][s]);
                }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int i = ti + 16 * r, j = tj + 16 * s;
                float w = 0.f;
                if (i < n && j < n && (REV ? j >= i : j <= i)) {
                    const double Gi = sG[j0 + i + 1], Gj = sG[j0 + j + 1];
                    w = p[r][s] * expf((float)(REV ? Gj - Gi : Gi - Gj));
                }
                sP[i * ldc + j] = w;
                o[r][s] *= sInter[i];
            }
        __syncthreads();
        for (int j = 0; j < kC; j += 4) {
            float4 xp[2], xc[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                xp[r] = *reinterpret_cast<const float4 *>(sP + (ti + 16 * r) * ldc + j);
                xc[r] = *reinterpret_cast<const float4 *>(sct + (tj + 16 * r) * ldc + j);
            }
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int s = 0; s < 2; ++s) o[r][s] = dot4(xp[r], xc[s], o[r][s]);
        }
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int i = ti + 16 * r;
            const long row = t0 + j0 + i;
            float dot = 0.f;
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int col = c0 + tj + 16 * s;
                if (i < n && col < dc) {
                    st_out(out, ((size_t)row * geo.H + h) * dc + col, o[r][s]);
                    if (dots)
                        dot = fmaf(o[r][s],
                                   ld_in(ro.e, ((size_t)row * ro.he + h / (geo.H / ro.he)) * dc + col),
                                   dot);
                }
            }
            if (dots) {
#pragma unroll
                for (int k = 8; k; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
                if (tj == 0 && i < n)
                    dots[((size_t)z * geo.rows + row) * geo.H + h] = dot;
            }
        }
        if (cc == nch - 1) break;
        __syncthreads();  // all reads of X are done
        {
            const int rg = tid >> 5, cg = tid & 31;
            const float dec = expf((float)(sG[j0 + n] - sG[j0]));
            if (4 * cg < db) {
                float x[4][4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float4 y = *reinterpret_cast<const float4 *>(sX + (4 * rg + r) * lda + 4 * cg);
                    x[r][0] = dec * y.x; x[r][1] = dec * y.y; x[r][2] = dec * y.z; x[r][3] = dec * y.w;
                }
                for (int j = 0; j < n; ++j) {
                    const float4 cv = *reinterpret_cast<const float4 *>(sc + j * ldc + 4 * rg);
                    const float4 bv = *reinterpret_cast<const float4 *>(sb + j * lda + 4 * cg);
                    const float w = sW[j];
                    const float ca[4] = {w * cv.x, w * cv.y, w * cv.z, w * cv.w};
                    const float ba[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
                    for (int r = 0; r < 4; ++r)
#pragma unroll
                        for (int s = 0; s < 4; ++s) x[r][s] = fmaf(ca[r], ba[s], x[r][s]);
                }
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    *reinterpret_cast<float4 *>(sX + (4 * rg + r) * lda + 4 * cg) =
                        make_float4(x[r][0], x[r][1], x[r][2], x[r][3]);
            }
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
out_kernel(Roles<T> ro, const float *g, Geo geo, Plan plan, unsigned int *err) {
    stream_order();
    outputs<T, T, false>(ro, blockIdx.z, g, geo, plan, err);
}
// dq (blockIdx.z below nq), dk (below 2 nq), dv in one launch: a short step waited for each
// (T 100, H 4, d 64: 55 us with a launch each, 38 us so and with states and carries in pairs)
template <typename T, typename To>
__global__ void __launch_bounds__(kThreads)
grad_kernel(Roles<T> rq, Roles<T> rk, Roles<T> rv, int nq, const float *g, Geo geo, Plan plan,
            unsigned int *err) {
    stream_order();
    const int z = blockIdx.z;
    if (z < nq)
        outputs<T, To, false>(rq, z, g, geo, plan, err);
    else if (z < 2 * nq)
        outputs<T, To, true>(rk, z - nq, g, geo, plan, err);
    else
        outputs<T, T, true>(rv, z - 2 * nq, g, geo, plan, err);
}

// ------------------------------------------------------------ gradient of the decays
// One CTA per (slot, head): <S_end, dS_end>, then the reverse running sum of
// R - C over the block's tokens, in 64 bits.
__global__ void __launch_bounds__(kThreads)
dg_kernel(const float *rdot, int nr, const float *cdot, int nc,
          const float *X, const float *fin, const float *Y,
          float *dg, float *part, Geo geo, Plan plan, int nel,
          unsigned int *err) {
    stream_order();
    __shared__ double red[kThreads / 32], suf[kThreads / 32];
    const int slot = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int4 sl = slot_of(geo, plan, slot);
    const int len = sl.y;
    const size_t sh = (size_t)slot * geo.H + h;
    if (len <= 0) {
        if (part && tid == 0) part[sh] = 0.f;
        return;
    }
    if (kChecked && !(chk_span(sl.x, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err)))
        return;
    const int nb = geo.varlen ? plan.blk_start[sl.z + 1] - plan.blk_start[sl.z] : geo.nb;
    const float *Se = sl.w + 1 < nb ? X + (sh + geo.H) * nel
                                    : fin + ((size_t)sl.z * geo.H + h) * nel;
    const float *De = Y + sh * nel;
    float f = 0.f;
    for (int i = tid; i < nel / 4; i += kThreads)
        f = dot4(reinterpret_cast<const float4 *>(Se)[i], reinterpret_cast<const float4 *>(De)[i], f);
    double d = f;
#pragma unroll
    for (int o = 16; o; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (lane == 0) red[warp] = d;
    double x = 0.0;
    const long row = (long)sl.x + tid;
    if (tid < len) {
        for (int i = 0; i < nr; ++i) x += rdot[((size_t)i * geo.rows + row) * geo.H + h];
        for (int i = 0; i < nc; ++i) x -= cdot[((size_t)i * geo.rows + row) * geo.H + h];
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // inclusive sum from the warp's end
        const double y = __shfl_down_sync(0xffffffffu, x, o);
        if (lane + o < 32) x += y;
    }
    if (lane == 0) suf[warp] = x;
    __syncthreads();
    for (int w = kThreads / 32 - 1; w > warp; --w) x += suf[w];
    for (int w = 0; w < kThreads / 32; ++w) x += red[w];
    if (!part) {
        if (tid < len) dg[(size_t)row * geo.H + h] = (float)x;
        return;
    }
    x = tid < len ? x : 0.0;
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if (lane == 0) red[warp] = x;
    __syncthreads();
    if (tid == 0) {
        double s = 0.0;
        for (int w = 0; w < kThreads / 32; ++w) s += red[w];
        part[sh] = (float)s;
    }
}

}  // namespace lin
}  // namespace gdr

// ====================================================================== host side
using namespace gdr;
using namespace gdr::lin;

namespace {

int blocks_of(int d) { return (d + kNb - 1) / kNb; }
size_t out_smem(int db) { return sizeof(float) * (size_t)(3 * kC * (db + 4) + 3 * kC * (kC + 4)); }

Plan plan_of(const gdr_host::LinCall &c, const gdr_host::LinWs &w) {
    return {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
}

gdr_host::LinWs simt_ws(const gdr_host::LinCall &c, bool bwd) {
    // Blocks of up to 256 tokens; of fewer, down to one chunk, while the grid would leave SMs idle:
    // a block's chunks run one after another (gradients of T 100, H 4, d 64: 107 us in blocks of 256, 57 us of 32)
    int L = kBlk;
    while (L > kC) {
        const double slots = c.cu ? (double)c.T / L + c.n_seq : (double)c.B * ((c.T + L - 1) / L);
        if (slots * c.H * blocks_of(c.dv_) >= 2 * 148) break;
        L /= 2;
    }
    return gdr_host::lin_ws(c.B, c.T, c.H, c.Hk, c.dk_, c.dv_, c.n_seq, c.cu != nullptr, bwd, L,
                            blocks_of(c.dk_) > blocks_of(c.dv_) ? blocks_of(c.dk_) : blocks_of(c.dv_));
}

template <typename T>
cudaError_t launch_states(const gdr_host::LinCall &c, const Geo &geo, const Plan &plan, const StateArgs<T> &f,
                          const StateArgs<T> *r, float *gtot) {
    if (!geo.n_slots) return cudaSuccess;
    const int nz = blocks_of(c.dv_);
    gdr_host::ProfToken tk = gdr_host::prof_begin(GDR_K_LIN_STATE, c.st);
    const cudaError_t le = gdr_host::lin_launch(state_kernel<T>, dim3(geo.n_slots, c.H, r ? 2 * nz : nz),
                                                kThreads, 0, c.st, f, r ? *r : f, nz, c.g, gtot, geo, plan,
                                                c.dk_, c.dv_, c.err);
    gdr_host::prof_end(tk, c.st);
    return le;
}

template <typename T>
cudaError_t fwd_t(const gdr_host::LinCall &c) {
    const gdr_host::LinWs w = simt_ws(c, false);
    const Geo geo = gdr_host::lin_geo(c, w);
    const Plan plan = plan_of(c, w);
    float *X = (float *)(c.ws + w.X), *gtot = (float *)(c.ws + w.gtot);
    cudaError_t e;
    if ((e = gdr_host::lin_plan(c, geo, w)) != cudaSuccess) return e;
    if ((e = launch_states<T>(c, geo, plan, {(const T *)c.k, (const T *)c.v, X}, nullptr, gtot)) != cudaSuccess)
        return e;
    const gdr_host::LinScan f{X, gtot, c.S0, c.S_final};
    if ((e = gdr_host::lin_scan(c, geo, w, &f, nullptr)) != cudaSuccess) return e;
    if (!geo.n_slots) return cudaSuccess;
    const Roles<T> ro = {(const T *)c.q, (const T *)c.k, (const T *)c.v, nullptr, c.Hk, c.Hk, c.H, c.H,
                         c.dk_, c.dv_, false, X, c.out, nullptr};
    static gdr_host::SmemLimit limit;
    if ((e = limit.set((const void *)out_kernel<T>, (int)out_smem(128))) != cudaSuccess) return e;
    gdr_host::ProfToken tk = gdr_host::prof_begin(GDR_K_LIN_OUT, c.st);
    const cudaError_t le = gdr_host::lin_launch(out_kernel<T>, dim3(geo.n_slots, c.H, blocks_of(c.dv_)),
                                                kThreads, out_smem(c.dk_), c.st, ro, c.g, geo, plan, c.err);
    gdr_host::prof_end(tk, c.st);
    return le;
}

template <typename T, typename To>
cudaError_t launch_grads(const gdr_host::LinCall &c, const Geo &geo, const Plan &plan, const Roles<T> &rq,
                         const Roles<T> &rk, const Roles<T> &rv) {
    static gdr_host::SmemLimit limit;
    const cudaError_t e = limit.set((const void *)grad_kernel<T, To>, (int)out_smem(128));
    if (e != cudaSuccess) return e;
    const int nq = blocks_of(c.dk_);
    gdr_host::ProfToken tk = gdr_host::prof_begin(GDR_K_LIN_GRAD, c.st);
    const cudaError_t le = gdr_host::lin_launch(grad_kernel<T, To>, dim3(geo.n_slots, c.H,
                                                2 * nq + blocks_of(c.dv_)), kThreads,
                                                out_smem(c.dk_ > c.dv_ ? c.dk_ : c.dv_), c.st, rq, rk, rv, nq,
                                                c.g, geo, plan, c.err);
    gdr_host::prof_end(tk, c.st);
    return le;
}

template <typename T>
cudaError_t bwd_t(const gdr_host::LinCall &c) {
    const gdr_host::LinWs w = simt_ws(c, true);
    const Geo geo = gdr_host::lin_geo(c, w);
    const Plan plan = plan_of(c, w);
    float *X = (float *)(c.ws + w.X), *Y = (float *)(c.ws + w.Y);
    float *gtot = (float *)(c.ws + w.gtot), *fin = (float *)(c.ws + w.fin);
    float *rdot = (float *)(c.ws + w.rdot), *cdot = (float *)(c.ws + w.cdot);
    float *part = c.gate == GDR_GATE_HEAD ? (float *)(c.ws + w.part) : nullptr;
    const bool shared = c.Hk < c.H;
    const T *q = (const T *)c.q, *k = (const T *)c.k, *v = (const T *)c.v, *dy = (const T *)c.dout;
    cudaError_t e;
    if ((e = gdr_host::lin_plan(c, geo, w)) != cudaSuccess) return e;
    const StateArgs<T> back{q, dy, Y};
    if ((e = launch_states<T>(c, geo, plan, {k, v, X}, &back, gtot)) != cudaSuccess) return e;
    const gdr_host::LinScan f{X, gtot, c.S0, fin}, b{Y, gtot, c.dS_final, c.dS0};
    if ((e = gdr_host::lin_scan(c, geo, w, &f, &b)) != cudaSuccess) return e;
    if (geo.n_slots) {
        // of shared query/key heads per value head in fp32, then summed
        const Roles<T> rq = {dy, v, k, q, c.H, c.H, c.Hk, c.Hk, c.dv_, c.dk_, true, X,
                             shared ? (void *)(c.ws + w.dq32) : c.dq, rdot};
        const Roles<T> rk = {v, dy, q, nullptr, c.H, c.H, c.Hk, c.Hk, c.dv_, c.dk_, true, Y,
                             shared ? (void *)(c.ws + w.dk32) : c.dk, nullptr};
        const Roles<T> rv = {k, q, dy, v, c.Hk, c.Hk, c.H, c.H, c.dk_, c.dv_, false, Y, c.dv, cdot};
        e = shared ? launch_grads<T, float>(c, geo, plan, rq, rk, rv) : launch_grads<T, T>(c, geo, plan, rq, rk, rv);
        if (e == cudaSuccess && shared)
            e = gdr_host::lin_group_sum(c, geo, w, (const float *)(c.ws + w.dq32), c.dq, c.dk_);
        if (e == cudaSuccess && shared)
            e = gdr_host::lin_group_sum(c, geo, w, (const float *)(c.ws + w.dk32), c.dk, c.dk_);
        if (e != cudaSuccess) return e;
        gdr_host::ProfToken tk = gdr_host::prof_begin(GDR_K_LIN_GRAD, c.st);
        e = gdr_host::lin_launch(dg_kernel, dim3(geo.n_slots, c.H), kThreads, 0, c.st, rdot, blocks_of(c.dk_),
                                 cdot, blocks_of(c.dv_), X, fin, Y, c.dg, part, geo, plan, c.dk_ * c.dv_,
                                 c.err);
        gdr_host::prof_end(tk, c.st);
        if (e != cudaSuccess) return e;
    }
    return part ? gdr_host::lin_dg_heads(c, geo, part) : cudaSuccess;
}

}  // namespace

namespace gdr_host {
size_t lin_simt_ws_bytes(const LinCall &c, bool bwd) { return simt_ws(c, bwd).total; }
cudaError_t lin_fwd_simt(const LinCall &c) {
    return c.dtype == GDR_BF16 ? fwd_t<__nv_bfloat16>(c) : fwd_t<float>(c);
}
cudaError_t lin_bwd_simt(const LinCall &c) {
    return c.dtype == GDR_BF16 ? bwd_t<__nv_bfloat16>(c) : bwd_t<float>(c);
}
}  // namespace gdr_host
