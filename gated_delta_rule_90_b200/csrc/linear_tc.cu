// Linear attention with a decay for each head on the tensor cores (tcgen05):
// bf16 tokens, d_k and d_v multiples of 16 up to 128, forward and gradient.
//
// The operator of linear_simt.cu, roles a, b (d_b wide) and c (d_c wide), in
// chunks of 128 tokens, each chunk's sums started at the state X that the one
// before left:
//
//     P   = (A B^T) . Gamma,  Gamma_ij = e^{G_i - G_j} (j <= i)       [128, 128]
//     out = P C + e^{G} (A X^T)                                       [128, d_c]
//     X   = e^{G_n} X + (w C)^T B,  w_j = e^{G_n - G_j}               [d_c, d_b]
//
// (backward in time: j >= i, Gamma_ij = e^{G_j - G_i}, e^{G_n - G_i} in place of
// e^{G_i}, w_j = e^{G_j}).  One CTA walks a block of tokens of one sequence and
// head for 64 columns of c; A, B, C tiles come by TMA, all products run on
// tcgen05 with accumulators in tensor memory, and the carried state stays in
// registers, fp32.  The state's own chain is one multiply-add per element and
// chunk: (w C)^T B does not depend on X, so the chunks' products overlap.
//
// Precision.  bf16 operands are exact in every product of two inputs.  P is
// rounded to bf16 once (it multiplies C) and so is X where it multiplies A for
// an output that is stored in bf16: two independent roundings of 2^-9 relative,
// on disjoint parts of the output, next to the output's own.  w C is split into
// three bf16 terms by truncation, x = hi + mid + lo exactly (8 + 8 + 8 bits), so
// the state keeps fp32 accuracy; where the gradient of the decays needs the
// state's part of the output in fp32, X is split the same way.
#include "linear.cuh"
#include "sm100.cuh"
#include "tmap.cuh"

namespace gdr {
namespace lin {

using namespace sm100;

constexpr int kQ = 128;                  // tokens of a chunk
constexpr int kN = 64;                   // columns of c of a CTA
constexpr uint32_t kSpinTc = 1u << 24;   // poll limit of every mbarrier wait
constexpr int kTcThreads = 384;          // TMA, 2 MMA issuers, decays; 4 output warps; 4 state warps
constexpr uint32_t kAtom = kQ * 128;     // bytes of 128 rows of 64 bf16
constexpr float kLog2e = 1.4426950408889634f;

enum { kStateOnly = 0, kOut = 1, kOutDots = 2 };

// Shared memory of a CTA.  Buffers of the a, b, c tiles and terms of X by mode:
// 227 KB hold two of each tile with one term of X; with three terms (32 KB
// more) a and c have one buffer.
template <int MODE>
struct TcSmem {
    static constexpr int NA = MODE == kOutDots ? 1 : 2, NB = 2, NC = MODE == kOutDots ? 1 : 2;
    static constexpr int XT = MODE == kOutDots ? 3 : 1;
    static constexpr uint32_t A = 0;
    static constexpr uint32_t B = A + (MODE == kStateOnly ? 0 : NA * 2 * kAtom);
    static constexpr uint32_t Cc = B + NB * 2 * kAtom;
    static constexpr uint32_t CP = Cc + NC * kAtom;       // w C, three terms
    static constexpr uint32_t X = CP + 3 * kAtom;
    static constexpr uint32_t TAB = X + (MODE == kStateOnly ? 0 : XT * kAtom);
    // tables of a chunk's decays (floats)
    static constexpr int LC = 0, CF = 128, W = 256, EG = 384, RF = 512, DEC = 704;
    static constexpr uint32_t BARS = TAB + 712 * 4;
    static constexpr uint32_t TOTAL = BARS + 24 * 8 + 16;
};

// Tensor memory columns.  SD: (w C)^T B, one column block per split term where
// they fit, else the last two summed by the accumulator.
template <int MODE>
struct TcTmem {
    static constexpr int SDW = MODE == kOutDots ? 128 : 192, INW = MODE == kOutDots ? 128 : 64;
    static constexpr int SD = 0;
    static constexpr int P = SDW, PB = P + 128, O = PB + 64, OIN = O + 64;
    static constexpr uint32_t COLS = MODE == kStateOnly ? 256 : 512;
    static_assert(MODE == kStateOnly || OIN + INW <= 512, "tensor memory");
};

struct TcArgs {
    const float *g;
    const float *xin;    // state that enters: per (sequence, head), or per (slot, head) when `multi`
    float *xout;         // state that leaves (per sequence), or the blocks' own states (state only)
    float *gtot;         // state only: the blocks' sums of log-decays
    void *out;           // bf16, or fp32 with out32
    const __nv_bfloat16 *e;  // dots: rows that the state's part of out is multiplied with
    float *dots;         // [column groups, rows, H]
    int ha, hb, hc, he;  // heads of a, b, c, e
    int db, dc, ng;      // widths, column groups
    int tr;              // states are stored as the transpose of X
    int multi;           // more than one block per sequence
    int out32, wide;     // out is fp32; out is 32-byte aligned
};

__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int x, int y,
                                            int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void st32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// x0, x1 -> the bf16 pairs of the three truncated terms: x = hi + mid + lo, the
// differences exact.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
    hi = __byte_perm(u0, u1, 0x7632);
    const float r0 = x0 - __uint_as_float(u0 & 0xffff0000u), r1 = x1 - __uint_as_float(u1 & 0xffff0000u);
    const uint32_t m0 = __float_as_uint(r0), m1 = __float_as_uint(r1);
    mid = __byte_perm(m0, m1, 0x7632);
    const float l0 = r0 - __uint_as_float(m0 & 0xffff0000u), l1 = r1 - __uint_as_float(m1 & 0xffff0000u);
    lo = __byte_perm(__float_as_uint(l0), __float_as_uint(l1), 0x7632);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// The decays of one chunk (one warp; lane: 4 consecutive tokens), from 64-bit
// running sums so that differences are rounded once.  The pair weights of a
// 32 x 32 block off the diagonal are a product of a row factor and a column
// factor around the border of the column's block, both at most 1 for decays:
// no difference overflows; on the diagonal each is exponentiated (LC holds
// the sums inside the block in units of log 2).
template <bool REV, class SM>
__device__ __forceinline__ void decay_tables(float *tab, const float (&gv)[4], int n, int lane) {
    double p[4];
    p[0] = gv[0];
#pragma unroll
    for (int u = 1; u < 4; ++u) p[u] = p[u - 1] + gv[u];
    double inc = p[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const double y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
    }
    const double base = inc - p[3], Gn = __shfl_sync(0xffffffffu, inc, 31);
    double Gs[4];  // at the starts of the four 32-token blocks
#pragma unroll
    for (int b = 0; b < 4; ++b) Gs[b] = __shfl_sync(0xffffffffu, base, 8 * b);
    const int kb = lane >> 3;
    const double s0 = kb == 0 ? Gs[0] : kb == 1 ? Gs[1] : kb == 2 ? Gs[2] : Gs[3];
    const double s1 = kb == 0 ? Gs[1] : kb == 1 ? Gs[2] : kb == 2 ? Gs[3] : Gn;
    float lc[4], cf[4], w[4], eg[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const double G = base + p[u];
        const bool in = 4 * lane + u < n;
        lc[u] = (float)(G - s0) * kLog2e;
        cf[u] = expf((float)(REV ? G - s0 : s1 - G));
        w[u] = in ? expf((float)(REV ? G : Gn - G)) : 0.f;
        eg[u] = expf((float)(REV ? Gn - G : G));
    }
    float4 *t4 = reinterpret_cast<float4 *>(tab);
    t4[SM::LC / 4 + lane] = make_float4(lc[0], lc[1], lc[2], lc[3]);
    t4[SM::CF / 4 + lane] = make_float4(cf[0], cf[1], cf[2], cf[3]);
    t4[SM::W / 4 + lane] = make_float4(w[0], w[1], w[2], w[3]);
    t4[SM::EG / 4 + lane] = make_float4(eg[0], eg[1], eg[2], eg[3]);
    // row factors: forward, blocks before the row's own; reverse, blocks after it
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        if (REV ? b > kb : b < kb) {
            float r[4];
            const double e = REV ? Gs[b] : (b == 3 ? Gn : Gs[b + 1 < 4 ? b + 1 : 3]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const double G = base + p[u];
                r[u] = expf((float)(REV ? e - G : G - e));
            }
            // pair (row block kb, column block b) -> 32 entries at (pair index) * 32
            const int hiB = REV ? b : kb, loB = REV ? kb : b;
            t4[SM::RF / 4 + (hiB * (hiB - 1) / 2 + loB) * 8 + (lane & 7)] = make_float4(r[0], r[1], r[2], r[3]);
        }
    }
    if (lane == 0) tab[SM::DEC] = expf((float)Gn);
}

template <bool REV, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
chain_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
             const __grid_constant__ CUtensorMap tm_c, TcArgs p, Geo geo, Plan plan,
             unsigned int *err) {
    using SM = TcSmem<MODE>;
    using TM = TcTmem<MODE>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + SM::BARS);
    uint64_t *fullA = bars, *fullB = bars + 2, *fullC = bars + 4;      // tile loaded
    uint64_t *freeA = bars + 6, *freeB = bars + 8, *freeC = bars + 10; // its products are done
    uint64_t *pfull = bars + 12, *pfree = bars + 13, *pready = bars + 14, *ofull = bars + 15;
    uint64_t *ifull = bars + 16, *ifree = bars + 17, *cready = bars + 18, *sfull = bars + 19;
    uint64_t *xready = bars + 20, *tfull = bars + 21, *tfree = bars + 22;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 23);
    float *tab = reinterpret_cast<float *>(sm + SM::TAB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int ng = blockIdx.x % p.ng, sh = blockIdx.x / p.ng;
    const int slot = sh / geo.H, h = sh - slot * geo.H;
    const int4 sl = slot_of(geo, plan, slot);
    const int t0 = sl.x, len = sl.y, c0 = ng * kN;
    const int nch = (len + kQ - 1) / kQ;
    const int ha = h / (geo.H / p.ha), hb = h / (geo.H / p.hb), hc = h / (geo.H / p.hc);
    const size_t nel = (size_t)p.db * p.dc;
    // a slot of no sequence (an empty sequence has one block, which passes its state on)
    if (len < 0) return;
    // the walk's last block of the sequence: nothing enters after it
    const int nblk = geo.varlen ? plan.blk_start[sl.z + 1] - plan.blk_start[sl.z] : geo.nb;
    const bool last = REV ? sl.w == 0 : sl.w == nblk - 1;
    if (MODE == kStateOnly && last) return;
    if (kChecked && !(chk_span(t0, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err) &&
                      chk_tma(c0, 0, 2, p.dc, 1, err) &&
                      chk_true((smem_u32(sm) & 1023u) == 0 && len <= geo.L, err)))
        return;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&fullA[i], 1);
            mbar_init(&fullB[i], 1);
            mbar_init(&fullC[i], 1);
            mbar_init(&freeA[i], 2);
            mbar_init(&freeB[i], MODE == kStateOnly ? 1 : 2);
            mbar_init(&freeC[i], MODE == kStateOnly ? 1 : 5);  // O = P C; the 4 split warps
        }
        mbar_init(pfull, 1);
        mbar_init(pfree, 4);
        mbar_init(pready, 4);
        mbar_init(ofull, 1);
        mbar_init(ifull, 1);
        mbar_init(ifree, 4);
        mbar_init(cready, 4);
        mbar_init(sfull, 1);
        mbar_init(xready, 4);
        mbar_init(tfull, 1);
        mbar_init(tfree, MODE == kStateOnly ? 4 : 8);
        fence_mbar_init();
        prefetch_tmap(&tm_b);
        prefetch_tmap(&tm_c);
        if (MODE != kStateOnly) prefetch_tmap(&tm_a);
    }
    if (warp == 1) {
        tmem_alloc(tslot, TM::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int na = p.db > 64 ? 2 : 1;  // 64-wide column blocks of a and b
    bool ok = true;
    // chunk cc of the walk: first token and number of tokens
    auto chunk_at = [&](int cc) { return (REV ? nch - 1 - cc : cc) * kQ; };

    if (warp == 0) {
        // ===================== TMA loads =====================
        if (lane == 0) {
            for (int cc = 0; cc < nch && ok; ++cc) {
                const int y = t0 + chunk_at(cc);
                const int ib = cc % SM::NB, ic = cc % SM::NC, ia = cc % SM::NA;
                if (cc >= SM::NB) ok = mbar_wait_bounded(&freeB[ib], (cc / SM::NB - 1) & 1, kSpinTc, err);
                if (!ok) break;
                mbar_arrive_expect_tx(&fullB[ib], na * kAtom);
                for (int i = 0; i < na; ++i)
                    tma_load_3d(sm + SM::B + (ib * 2 + i) * kAtom, &tm_b, &fullB[ib], 64 * i, hb, y);
                if (MODE != kStateOnly) {
                    if (cc >= SM::NA) ok = mbar_wait_bounded(&freeA[ia], (cc / SM::NA - 1) & 1, kSpinTc, err);
                    if (!ok) break;
                    mbar_arrive_expect_tx(&fullA[ia], na * kAtom);
                    for (int i = 0; i < na; ++i)
                        tma_load_3d(sm + SM::A + (ia * 2 + i) * kAtom, &tm_a, &fullA[ia], 64 * i, ha, y);
                }
                if (cc >= SM::NC) ok = mbar_wait_bounded(&freeC[ic], (cc / SM::NC - 1) & 1, kSpinTc, err);
                if (!ok) break;
                mbar_arrive_expect_tx(&fullC[ic], kAtom);
                tma_load_3d(sm + SM::Cc + ic * kAtom, &tm_c, &fullC[ic], c0, hc, y);
            }
            // every load has landed and every product has read its tiles before the CTA ends:
            // free(i) follows full(i), so waiting for the last use of each buffer covers both
            for (int cc = nch - 1; cc >= 0 && cc >= nch - 2; --cc) {
                if (cc >= nch - SM::NB) mbar_wait_bounded(&freeB[cc % SM::NB], (cc / SM::NB) & 1, kSpinTc, err);
                if (MODE != kStateOnly && cc >= nch - SM::NA)
                    mbar_wait_bounded(&freeA[cc % SM::NA], (cc / SM::NA) & 1, kSpinTc, err);
                if (cc >= nch - SM::NC) mbar_wait_bounded(&freeC[cc % SM::NC], (cc / SM::NC) & 1, kSpinTc, err);
            }
        }
    } else if (warp == 1) {
        // ===================== MMA: P = A B^T, O = P C =====================
        if (MODE != kStateOnly && lane == 0) {
            const uint32_t idP = idesc_bf16(128, 128, 0, 0), idO = idesc_bf16(128, kN, 0, 1);
            const uint64_t dA = sdesc_sw128(smem_u32(sm + SM::A), 16, 1024);
            const uint64_t dB = sdesc_sw128(smem_u32(sm + SM::B), 16, 1024);
            const uint64_t dC = sdesc_sw128(smem_u32(sm + SM::Cc), kAtom, 1024);
            const int ks = p.db / 16;
            auto gram = [&](int cc) {
                const int ia = cc % SM::NA, ib = cc % SM::NB;
                ok = ok && mbar_wait_bounded(&fullA[ia], (cc / SM::NA) & 1, kSpinTc, err);
                ok = ok && mbar_wait_bounded(&fullB[ib], (cc / SM::NB) & 1, kSpinTc, err);
                // rows past the end are zeroed before they are multiplied (the short chunk is the
                // first or the last of the walk, so cready cannot be two phases ahead of this wait)
                if (len - chunk_at(cc) < kQ) ok = ok && mbar_wait_bounded(cready, cc & 1, kSpinTc, err);
                if (cc > 0) ok = ok && mbar_wait_bounded(pfree, (cc - 1) & 1, kSpinTc, err);
                if (!ok) return;
                tc_fence_after();
                for (int kk = 0; kk < ks; ++kk) {
                    const uint32_t o = (kk >> 2) * kAtom + (kk & 3) * 32;
                    mma_bf16_ss(tmem + TM::P, sdesc_add(dA, ia * 2 * kAtom + o),
                                sdesc_add(dB, ib * 2 * kAtom + o), idP, kk > 0);
                }
                mma_commit(&freeA[ia]);
                mma_commit(&freeB[ib]);
                mma_commit(pfull);
            };
            if (nch > 0) gram(0);
            for (int cc = 0; cc < nch && ok; ++cc) {
                const int ic = cc % SM::NC;
                ok = ok && mbar_wait_bounded(&fullC[ic], (cc / SM::NC) & 1, kSpinTc, err);
                ok = ok && mbar_wait_bounded(pready, cc & 1, kSpinTc, err);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ts(tmem + TM::O, tmem + TM::PB + kk * 8,
                                sdesc_add(dC, ic * kAtom + kk * 2048), idO, kk > 0);
                mma_commit(&freeC[ic]);
                mma_commit(ofull);
                if (cc + 1 < nch) gram(cc + 1);
            }
        }
    } else if (warp == 2) {
        // ===================== MMA: A X^T, (w C)^T B =====================
        if (lane == 0) {
            const uint64_t dA = sdesc_sw128(smem_u32(sm + SM::A), 16, 1024);
            const uint64_t dX = sdesc_sw128(smem_u32(sm + SM::X), kAtom, 1024);
            // b as [d_b, tokens]: with one 64-wide block the upper lanes repeat it (not read)
            const uint64_t dB = sdesc_sw128(smem_u32(sm + SM::B), na > 1 ? kAtom : 0, 1024);
            const uint64_t dP = sdesc_sw128(smem_u32(sm + SM::CP), kAtom, 1024);
            const int ks = p.db / 16;
            for (int cc = 0; cc < nch && ok; ++cc) {
                const int ia = cc % SM::NA, ib = cc % SM::NB;
                if (MODE != kStateOnly) {
                    ok = ok && mbar_wait_bounded(&fullA[ia], (cc / SM::NA) & 1, kSpinTc, err);
                    ok = ok && mbar_wait_bounded(xready, cc & 1, kSpinTc, err);
                    if (cc > 0) ok = ok && mbar_wait_bounded(ifree, (cc - 1) & 1, kSpinTc, err);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t idI = idesc_bf16(128, TM::INW, 0, 1), idL = idesc_bf16(128, kN, 0, 1);
                    for (int kk = 0; kk < ks; ++kk)
                        mma_bf16_ss(tmem + TM::OIN,
                                    sdesc_add(dA, ia * 2 * kAtom + (kk >> 2) * kAtom + (kk & 3) * 32),
                                    sdesc_add(dX, kk * 2048), idI, kk > 0);
                    if (MODE == kOutDots)
                        for (int kk = 0; kk < ks; ++kk)
                            mma_bf16_ss(tmem + TM::OIN + kN,
                                        sdesc_add(dA, ia * 2 * kAtom + (kk >> 2) * kAtom + (kk & 3) * 32),
                                        sdesc_add(dX, 2 * kAtom + kk * 2048), idL, 1);
                    mma_commit(&freeA[ia]);
                    mma_commit(ifull);
                }
                ok = ok && mbar_wait_bounded(&fullB[ib], (cc / SM::NB) & 1, kSpinTc, err);
                ok = ok && mbar_wait_bounded(cready, cc & 1, kSpinTc, err);
                if (!ok) break;
                tc_fence_after();
                const uint32_t idS = idesc_bf16(128, TM::SDW, 1, 1), idT = idesc_bf16(128, kN, 1, 1);
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)
                    mma_bf16_ss(tmem + TM::SD, sdesc_add(dB, ib * 2 * kAtom + kk * 2048),
                                sdesc_add(dP, kk * 2048), idS, kk > 0);
                if (TM::SDW == 128)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_bf16_ss(tmem + TM::SD + kN, sdesc_add(dB, ib * 2 * kAtom + kk * 2048),
                                    sdesc_add(dP, 2 * kAtom + kk * 2048), idT, 1);
                if (MODE == kStateOnly) mma_commit(&freeC[cc % SM::NC]);
                mma_commit(&freeB[ib]);
                mma_commit(sfull);
            }
        }
    } else if (warp == 3) {
        // ===================== decays =====================
        float gv[4], gt = 0.f;
        auto load = [&](int cc) {
            const int j0 = chunk_at(cc), n = min(kQ, len - j0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                gv[u] = 4 * lane + u < n ? load_g(geo, p.g, (long)t0 + j0 + 4 * lane + u, h) : 0.f;
        };
        double tot = 0.0;
        if (nch > 0) load(0);
        for (int cc = 0; cc < nch && ok; ++cc) {
            const int n = min(kQ, len - chunk_at(cc));
            if (cc > 0) ok = mbar_wait_bounded(tfree, (cc - 1) & 1, kSpinTc, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            decay_tables<REV, SM>(tab, gv, n, lane);
            if (MODE == kStateOnly) tot += (double)gv[0] + gv[1] + gv[2] + gv[3];
            __syncwarp();
            if (lane == 0) mbar_arrive(tfull);
            if (cc + 1 < nch) load(cc + 1);
        }
        if (MODE == kStateOnly && p.gtot && ng == 0) {
#pragma unroll
            for (int o = 16; o; o >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, o);
            gt = (float)tot;
            if (lane == 0) p.gtot[(size_t)slot * geo.H + h] = gt;
        }
    } else if (warp < 8) {
        // ===================== outputs: row i of the chunk =====================
        if (MODE != kStateOnly) {
            const int rb = warp & 3, i = rb * 32 + lane;
            const uint32_t lb = (uint32_t)(rb * 32) << 16;
            for (int cc = 0; cc < nch; ++cc) {
                const int j0 = chunk_at(cc), n = min(kQ, len - j0);
                ok = ok && mbar_wait_bounded(tfull, cc & 1, kSpinTc, err);
                ok = ok && mbar_wait_bounded(pfull, cc & 1, kSpinTc, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const float eg = tab[SM::EG + i], li = tab[SM::LC + i];
                // weights of the pairs, 32 columns at a time
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float w[32];
                    if (REV ? b < rb : b > rb) {
#pragma unroll
                        for (int u = 0; u < 16; ++u) w[u] = 0.f;
                    } else {
                        float x[32];
                        tmem_ld16(tmem + TM::P + lb + 32 * b, x);
                        tmem_ld16(tmem + TM::P + lb + 32 * b + 16, x + 16);
                        tmem_wait_ld();
                        if (b == rb) {
#pragma unroll
                            for (int u = 0; u < 32; ++u) {
                                const float lj = tab[SM::LC + 32 * b + u];
                                const bool in = REV ? u >= lane : u <= lane;
                                x[u] = in ? x[u] * ex2(REV ? lj - li : li - lj) : 0.f;
                            }
                        } else {
                            const int hiB = REV ? b : rb, loB = REV ? rb : b;
                            const float r = tab[SM::RF + (hiB * (hiB - 1) / 2 + loB) * 32 + lane];
#pragma unroll
                            for (int u4 = 0; u4 < 8; ++u4) {
                                const float4 c = *reinterpret_cast<const float4 *>(tab + SM::CF + 32 * b + 4 * u4);
                                x[4 * u4] *= r * c.x;
                                x[4 * u4 + 1] *= r * c.y;
                                x[4 * u4 + 2] *= r * c.z;
                                x[4 * u4 + 3] *= r * c.w;
                            }
                        }
#pragma unroll
                        for (int u = 0; u < 16; ++u) w[u] = __uint_as_float(pack2(x[2 * u], x[2 * u + 1]));
                    }
                    tmem_st16(tmem + TM::PB + lb + 16 * b, w);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(pready);
                    mbar_arrive(pfree);
                    mbar_arrive(tfree);
                }
                const size_t row = (size_t)t0 + j0 + i;
                ok = ok && mbar_wait_bounded(ifull, cc & 1, kSpinTc, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                float o[64];
#pragma unroll
                for (int b = 0; b < 4; ++b) tmem_ld16(tmem + TM::OIN + lb + 16 * b, o + 16 * b);
                if (MODE == kOutDots) {
                    float m[64];
#pragma unroll
                    for (int b = 0; b < 4; ++b) tmem_ld16(tmem + TM::OIN + kN + lb + 16 * b, m + 16 * b);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 64; ++u) o[u] = eg * (o[u] + m[u]);
                } else {
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 64; ++u) o[u] *= eg;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(ifree);
                if (MODE == kOutDots && i < n) {
                    float d = 0.f;
                    const __nv_bfloat16 *e = p.e + (row * p.he + h / (geo.H / p.he)) * p.dc + c0;
#pragma unroll
                    for (int b = 0; b < 8; ++b)
                        if (c0 + 8 * b < p.dc) {
                            float f[8];
                            unpack8(*reinterpret_cast<const uint4 *>(e + 8 * b), f);
#pragma unroll
                            for (int u = 0; u < 8; ++u) d = fmaf(o[8 * b + u], f[u], d);
                        }
                    p.dots[((size_t)ng * geo.rows + row) * geo.H + h] = d;
                }
                ok = ok && mbar_wait_bounded(ofull, cc & 1, kSpinTc, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    float x[16];
                    tmem_ld16(tmem + TM::O + lb + 16 * b, x);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 16; ++u) o[16 * b + u] += x[u];
                }
                tc_fence_before();
                if (i < n) {
                    const size_t at = (row * geo.H + h) * p.dc + c0;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (c0 + 16 * b >= p.dc) continue;
                        if (p.out32) {
                            float4 *q = reinterpret_cast<float4 *>((float *)p.out + at + 16 * b);
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                q[u] = make_float4(o[16 * b + 4 * u], o[16 * b + 4 * u + 1],
                                                   o[16 * b + 4 * u + 2], o[16 * b + 4 * u + 3]);
                        } else {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) w[u] = pack2(o[16 * b + 2 * u], o[16 * b + 2 * u + 1]);
                            __nv_bfloat16 *q = (__nv_bfloat16 *)p.out + at + 16 * b;
                            if (p.wide) {
                                st32(q, w);
                            } else {
                                reinterpret_cast<uint4 *>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                reinterpret_cast<uint4 *>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                    }
                }
            }
        }
    } else {
        // ===================== state: row k of X^T (d_b), 64 columns =====================
        const int rb = warp & 3, k = rb * 32 + lane;
        const uint32_t lb = (uint32_t)(rb * 32) << 16;
        float x[64];
#pragma unroll
        for (int u = 0; u < 64; ++u) x[u] = 0.f;
        const size_t unit = (size_t)(p.multi ? slot : sl.z) * geo.H + h;
        if (MODE != kStateOnly && p.xin && k < p.db) {
            const float *src = p.xin + unit * nel;
            if (p.tr) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (c0 + 4 * u < p.dc) {
                        const float4 y = *reinterpret_cast<const float4 *>(src + (size_t)k * p.dc + c0 + 4 * u);
                        x[4 * u] = y.x; x[4 * u + 1] = y.y; x[4 * u + 2] = y.z; x[4 * u + 3] = y.w;
                    }
            } else {
#pragma unroll
                for (int u = 0; u < 64; ++u)
                    if (c0 + u < p.dc) x[u] = src[(size_t)(c0 + u) * p.db + k];
            }
        }
        auto publish = [&]() {  // X as the B operand of A X^T: row k, swizzled
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                const uint32_t off = SM::X + k * 128 + ((b ^ (k & 7)) << 4);
                if (MODE == kOutDots) {
                    uint4 hi, mid, lo;
                    split3(x[8 * b], x[8 * b + 1], hi.x, mid.x, lo.x);
                    split3(x[8 * b + 2], x[8 * b + 3], hi.y, mid.y, lo.y);
                    split3(x[8 * b + 4], x[8 * b + 5], hi.z, mid.z, lo.z);
                    split3(x[8 * b + 6], x[8 * b + 7], hi.w, mid.w, lo.w);
                    *reinterpret_cast<uint4 *>(sm + off) = hi;
                    *reinterpret_cast<uint4 *>(sm + off + kAtom) = mid;
                    *reinterpret_cast<uint4 *>(sm + off + 2 * kAtom) = lo;
                } else {
                    *reinterpret_cast<uint4 *>(sm + off) = pack8(x + 8 * b);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(xready);
        };
        if (MODE != kStateOnly) publish();
        for (int cc = 0; cc < nch; ++cc) {
            const int n = min(kQ, len - chunk_at(cc)), ib = cc % SM::NB, ic = cc % SM::NC;
            ok = ok && mbar_wait_bounded(tfull, cc & 1, kSpinTc, err);
            ok = ok && mbar_wait_bounded(&fullC[ic], (cc / SM::NC) & 1, kSpinTc, err);
            if (n < kQ) ok = ok && mbar_wait_bounded(&fullB[ib], (cc / SM::NB) & 1, kSpinTc, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const float w = tab[SM::W + k], dec = tab[SM::DEC];
            __syncwarp();
            if (lane == 0) mbar_arrive(tfree);
            uint8_t *crow = sm + SM::Cc + ic * kAtom + k * 128;
            uint8_t *prow = sm + SM::CP + k * 128;
            if (k < n) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    float f[8];
                    unpack8(*reinterpret_cast<const uint4 *>(crow + ((b ^ (k & 7)) << 4)), f);
                    uint4 hi, mid, lo;
                    split3(w * f[0], w * f[1], hi.x, mid.x, lo.x);
                    split3(w * f[2], w * f[3], hi.y, mid.y, lo.y);
                    split3(w * f[4], w * f[5], hi.z, mid.z, lo.z);
                    split3(w * f[6], w * f[7], hi.w, mid.w, lo.w);
                    uint8_t *q = prow + ((b ^ (k & 7)) << 4);
                    *reinterpret_cast<uint4 *>(q) = hi;
                    *reinterpret_cast<uint4 *>(q + kAtom) = mid;
                    *reinterpret_cast<uint4 *>(q + 2 * kAtom) = lo;
                }
            } else {  // past the end: zero, whatever memory holds there
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    reinterpret_cast<uint4 *>(crow)[b] = z;
                    for (int t = 0; t < 3; ++t) reinterpret_cast<uint4 *>(prow + t * kAtom)[b] = z;
                    for (int t = 0; t < na; ++t)
                        reinterpret_cast<uint4 *>(sm + SM::B + (ib * 2 + t) * kAtom + k * 128)[b] = z;
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(cready);
                if (MODE != kStateOnly) mbar_arrive(&freeC[ic]);
            }
            ok = ok && mbar_wait_bounded(sfull, cc & 1, kSpinTc, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                float hi[16], mid[16];
                tmem_ld16(tmem + TM::SD + lb + 16 * b, hi);
                tmem_ld16(tmem + TM::SD + kN + lb + 16 * b, mid);
                if (TM::SDW == 192) {
                    float lo[16];
                    tmem_ld16(tmem + TM::SD + 2 * kN + lb + 16 * b, lo);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 16; ++u) mid[u] += lo[u];
                } else {
                    tmem_wait_ld();
                }
#pragma unroll
                for (int u = 0; u < 16; ++u) x[16 * b + u] = fmaf(dec, x[16 * b + u], hi[u] + mid[u]);
            }
            tc_fence_before();
            // the products with X of this chunk are done (issued before the state's)
            if (MODE != kStateOnly && cc + 1 < nch) publish();
        }
        if (ok && p.xout && k < p.db && (MODE == kStateOnly || last)) {
            float *dst = p.xout + (MODE == kStateOnly ? (size_t)slot * geo.H + h : (size_t)sl.z * geo.H + h) * nel;
            if (p.tr) {
#pragma unroll
                for (int u = 0; u < 16; ++u)
                    if (c0 + 4 * u < p.dc)
                        *reinterpret_cast<float4 *>(dst + (size_t)k * p.dc + c0 + 4 * u) =
                            make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
            } else {
#pragma unroll
                for (int u = 0; u < 64; ++u)
                    if (c0 + u < p.dc) dst[(size_t)(c0 + u) * p.db + k] = x[u];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, TM::COLS);
}


// ------------------------------------------------------------ pairs inside a chunk, for dg
// M = (Q K^T) . (dO V^T) . Gamma below the diagonal: row sums (the pairs' part of
// q_l . dq_l) and column sums (of k_m . dk_m), fp32.  Both factors are products
// of inputs, so no operand is rounded.  The column sums are the row sums of the
// transposed products, which the tensor cores form as well: 32 more MMAs cost
// less than summing over lanes.  Reads q, k, v, dout once: HBM-bound.
struct PairArgs {
    const float *g;
    float *rsum, *csum;  // [rows, H]
    int H_k, dk, dv;
};
constexpr int kPairTab = 704 + 8;
struct PairSmem {
    static constexpr uint32_t QK = 0, VO = 4 * kAtom, TAB = 8 * kAtom;
    static constexpr uint32_t BARS = TAB + 2 * kPairTab * 4, TOTAL = BARS + 8 * 8 + 16;
};

__global__ void __launch_bounds__(kTcThreads, 1)
pair_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
            PairArgs p, Geo geo, Plan plan, unsigned int *err) {
    using SM = TcSmem<kOut>;  // table layout
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + PairSmem::BARS);
    uint64_t *fullQ = bars, *fullV = bars + 1, *mdone = bars + 2, *tfull = bars + 3, *tfree = bars + 4;
    uint64_t *efree = bars + 5, *qdone = bars + 6;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = blockIdx.x / geo.H, h = blockIdx.x - slot * geo.H;
    const int4 sl = slot_of(geo, plan, slot);
    const int t0 = sl.x, len = sl.y, nch = (len + kQ - 1) / kQ, hk = h / (geo.H / geo.Hk);
    if (len <= 0 || (int)blockIdx.y >= nch) return;
    if (kChecked && !(chk_span(t0, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err) &&
                      chk_true((smem_u32(sm) & 1023u) == 0, err)))
        return;
    if (tid == 0) {
        mbar_init(fullQ, 1);
        mbar_init(fullV, 1);
        mbar_init(qdone, 1);
        mbar_init(mdone, 1);
        mbar_init(tfull, 2);
        mbar_init(tfree, 8);
        mbar_init(efree, 8);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int nk = p.dk > 64 ? 2 : 1, nv = p.dv > 64 ? 2 : 1;
    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            for (int cc = blockIdx.y; cc < nch; cc += gridDim.y, ++it) {
                const int y = t0 + cc * kQ;
                if (it) ok = mbar_wait_bounded(qdone, (it - 1) & 1, kSpinTc, err);
                if (!ok) break;
                mbar_arrive_expect_tx(fullQ, 2 * nk * kAtom);
                for (int i = 0; i < nk; ++i) {
                    tma_load_3d(sm + PairSmem::QK + i * kAtom, &tm_q, fullQ, 64 * i, hk, y);
                    tma_load_3d(sm + PairSmem::QK + (2 + i) * kAtom, &tm_k, fullQ, 64 * i, hk, y);
                }
                if (it) ok = mbar_wait_bounded(mdone, (it - 1) & 1, kSpinTc, err);
                if (!ok) break;
                mbar_arrive_expect_tx(fullV, 2 * nv * kAtom);
                for (int i = 0; i < nv; ++i) {
                    tma_load_3d(sm + PairSmem::VO + i * kAtom, &tm_o, fullV, 64 * i, h, y);
                    tma_load_3d(sm + PairSmem::VO + (2 + i) * kAtom, &tm_v, fullV, 64 * i, h, y);
                }
            }
            if (it) {  // the last loads have landed and been read
                mbar_wait_bounded(qdone, (it - 1) & 1, kSpinTc, err);
                mbar_wait_bounded(mdone, (it - 1) & 1, kSpinTc, err);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            const uint32_t id = idesc_bf16(128, 128, 0, 0);
            const uint64_t dq = sdesc_sw128(smem_u32(sm + PairSmem::QK), 16, 1024);
            const uint64_t dv = sdesc_sw128(smem_u32(sm + PairSmem::VO), 16, 1024);
            int it = 0;
            // columns: Q K^T 0, K Q^T 128, dO V^T 256, V dO^T 384
            auto both = [&](uint64_t d, int ks, uint32_t col) {
                for (int kk = 0; kk < ks; ++kk) {
                    const uint32_t o = (kk >> 2) * kAtom + (kk & 3) * 32;
                    mma_bf16_ss(tmem + col, sdesc_add(d, o), sdesc_add(d, 2 * kAtom + o), id, kk > 0);
                    mma_bf16_ss(tmem + col + 128, sdesc_add(d, 2 * kAtom + o), sdesc_add(d, o), id, kk > 0);
                }
            };
            for (int cc = blockIdx.y; cc < nch && ok; cc += gridDim.y, ++it) {
                if (it) ok = mbar_wait_bounded(efree, (it - 1) & 1, kSpinTc, err);
                ok = ok && mbar_wait_bounded(fullQ, it & 1, kSpinTc, err);
                if (!ok) break;
                tc_fence_after();
                both(dq, p.dk / 16, 0);
                mma_commit(qdone);
                ok = ok && mbar_wait_bounded(fullV, it & 1, kSpinTc, err);
                if (!ok) break;
                both(dv, p.dv / 16, 256);
                mma_commit(mdone);
            }
        }
    } else if (warp < 4) {  // decays: warp 2 for the rows, warp 3 for the columns
        float gv[4];
        int it = 0;
        auto load = [&](int cc) {
            const int n = min(kQ, len - cc * kQ);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                gv[u] = 4 * lane + u < n ? load_g(geo, p.g, (long)t0 + cc * kQ + 4 * lane + u, h) : 0.f;
        };
        load(blockIdx.y);
        for (int cc = blockIdx.y; cc < nch; cc += gridDim.y, ++it) {
            if (it) ok = mbar_wait_bounded(tfree, (it - 1) & 1, kSpinTc, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            float *tab = reinterpret_cast<float *>(sm + PairSmem::TAB) + (warp - 2) * kPairTab;
            if (warp == 2)
                decay_tables<false, SM>(tab, gv, min(kQ, len - cc * kQ), lane);
            else
                decay_tables<true, SM>(tab, gv, min(kQ, len - cc * kQ), lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(tfull);
            if (cc + (int)gridDim.y < nch) load(cc + gridDim.y);
        }
    } else {
        const bool rev = warp >= 8;
        const int rb = warp & 3, i = rb * 32 + lane;
        const uint32_t lb = (uint32_t)(rb * 32) << 16, col = rev ? 128 : 0;
        const float *tab = reinterpret_cast<const float *>(sm + PairSmem::TAB) + (rev ? kPairTab : 0);
        int it = 0;
        for (int cc = blockIdx.y; cc < nch; cc += gridDim.y, ++it) {
            const int n = min(kQ, len - cc * kQ);
            ok = ok && mbar_wait_bounded(tfull, it & 1, kSpinTc, err);
            ok = ok && mbar_wait_bounded(qdone, it & 1, kSpinTc, err);
            ok = ok && mbar_wait_bounded(mdone, it & 1, kSpinTc, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float li = tab[SM::LC + i];
            float s = 0.f;
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                if (rev ? b < rb : b > rb) continue;
                float x[32], y[32];
                tmem_ld16(tmem + col + lb + 32 * b, x);
                tmem_ld16(tmem + col + lb + 32 * b + 16, x + 16);
                tmem_ld16(tmem + 256 + col + lb + 32 * b, y);
                tmem_ld16(tmem + 256 + col + lb + 32 * b + 16, y + 16);
                tmem_wait_ld();
                float r = 0.f;
                if (b == rb) {
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        const float lj = tab[SM::LC + 32 * b + u];
                        const bool in = rev ? u > lane && 32 * b + u < n : u < lane;
                        r += in ? x[u] * y[u] * ex2(rev ? lj - li : li - lj) : 0.f;
                    }
                } else {
                    const int hiB = rev ? b : rb, loB = rev ? rb : b;
                    const float f = tab[SM::RF + (hiB * (hiB - 1) / 2 + loB) * 32 + lane];
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        const float z = x[u] * y[u] * tab[SM::CF + 32 * b + u];
                        r += 32 * b + u < n ? z : 0.f;
                    }
                    r *= f;
                }
                s += r;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(efree);
                mbar_arrive(tfree);
            }
            if (i < n) (rev ? p.csum : p.rsum)[((size_t)t0 + cc * kQ + i) * geo.H + h] = s;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ gradient of the decays
// One CTA per (sequence, head), chunks from the last to the first, 8 at a time
// (a warp group of 128 threads each), in 64 bits:
//     dg_t = sum_{l >= t in chunk} (R_l - C_l) + sum over later chunks (Ri - Ci) + <S_end, dS_end>,
// R = Ri + Rp, C = Ci + Cp: the state's part (dots of the chains) and the part of
// the chunk's own pairs, whose rows and columns sum to the same and so drop out
// of the carry.  S_end, dS_end at the end of the sequence.
struct DgArgs {
    const float *ri, *ci, *rp, *cp;
    int nri, nci;               // column groups of ri, ci
    const float *fin, *dfin;    // S_end, dS_end, or dfin NULL
    float *dg, *part;
    int nel;
};

__global__ void __launch_bounds__(1024)
dg_chunks_kernel(DgArgs p, const int32_t *__restrict__ cu, Geo geo, Plan plan) {
    __shared__ double tot[32], inter[32], red[32];
    const int s = blockIdx.x / geo.H, h = blockIdx.x - s * geo.H;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long t0;
    int len;
    if (geo.varlen) {
        const int a = plan.blk_start[s], b = plan.blk_start[s + 1];
        t0 = plan.slot[a].x;
        len = plan.slot[b - 1].x + plan.slot[b - 1].y - (int)t0;
    } else {
        t0 = (long)s * geo.T;
        len = geo.T;
    }
    double f = 0.0;
    if (p.dfin) {
        const size_t o = (size_t)blockIdx.x * p.nel;
        float acc = 0.f;
        for (int i = tid; i < p.nel / 4; i += 1024) {
            const float4 a = reinterpret_cast<const float4 *>(p.fin + o)[i];
            const float4 b = reinterpret_cast<const float4 *>(p.dfin + o)[i];
            acc = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc))));
        }
        f = acc;
#pragma unroll
        for (int o2 = 16; o2; o2 >>= 1) f += __shfl_xor_sync(0xffffffffu, f, o2);
        if (lane == 0) red[warp] = f;
        __syncthreads();
        f = 0.0;
        for (int w = 0; w < 32; ++w) f += red[w];
    }
    const int nch = (len + kQ - 1) / kQ, grp = tid >> 7, j = tid & 127;
    double all = 0.0, c0 = f;  // c0: the sum over the chunks behind
    for (int base = nch - 1; base >= 0; base -= 8) {
        const int cc = base - grp, i = cc * kQ + j;
        double x = 0.0, y = 0.0;  // everything; the state's part
        if (cc >= 0 && i < len) {
            const size_t at = ((size_t)t0 + i) * geo.H + h, pl = (size_t)geo.rows * geo.H;
            for (int u = 0; u < p.nri; ++u) y += p.ri[u * pl + at];
            for (int u = 0; u < p.nci; ++u) y -= p.ci[u * pl + at];
            x = y + ((double)p.rp[at] - (double)p.cp[at]);
        }
        double ys = y;
#pragma unroll
        for (int o = 16; o; o >>= 1) ys += __shfl_xor_sync(0xffffffffu, ys, o);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {  // inclusive sum from the warp's end
            const double z = __shfl_down_sync(0xffffffffu, x, o);
            if (lane + o < 32) x += z;
        }
        __syncthreads();  // the last round's readers are done
        if (lane == 0) {
            tot[warp] = x;
            inter[warp] = ys;
        }
        __syncthreads();
        double add = c0;
        for (int w = 0; w < 4 * grp; ++w) add += inter[w];  // groups behind this chunk
        for (int w = warp + 1; w < 4 * grp + 4; ++w) add += tot[w];
        x += add;
        for (int w = 0; w < 32; ++w) c0 += inter[w];
        if (cc >= 0 && i < len) {
            if (p.part)
                all += x;
            else
                p.dg[((size_t)t0 + i) * geo.H + h] = (float)x;
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int o = 16; o; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    __syncthreads();
    if (lane == 0) red[warp] = all;
    __syncthreads();
    if (tid == 0) {
        double r = 0.0;
        for (int w = 0; w < 32; ++w) r += red[w];
        p.part[blockIdx.x] = (float)r;
    }
}

}  // namespace lin
}  // namespace gdr

// ====================================================================== host side
using namespace gdr;
using namespace gdr::lin;
using gdr_host::LinCall;

namespace {

int groups(int d) { return (d + kN - 1) / kN; }
size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

// Tokens of a block: a whole sequence while the (sequence, head, column group)
// walks fill the GPU, else pieces of it.  Pieces cost a pass over k and v for
// their states and the carry, so equal sequences are cut where the estimate
// below says that it pays (about 1.5 us for a chunk of a walk, 0.9 us without
// outputs, 148 walks at a time), and packed ones, whose lengths the host does
// not know, into what one SM's share of all tokens is.
int block_len(int n_seq, bool varlen, int B, int T, int H, int ng, size_t nel) {
    const double sms = 148.0;
    if (varlen) {
        long L = (long)((double)T * H * ng / sms);
        if (L < 512) L = 512;
        if (L > T) L = T;
        return (int)((L + kQ - 1) / kQ * kQ);
    }
    const int ch = (T + kQ - 1) / kQ;
    int best = ch;
    double least = 1e30;
    for (int nb = 1; nb <= ch && nb <= 64; ++nb) {
        const int c = (ch + nb - 1) / nb;
        if (nb > 1 && c < 4) break;
        auto waves = [&](double units) { return (double)(long)((units + sms - 1) / sms); };
        double t = waves((double)n_seq * H * ng * nb) * (1.5 * c + 4);
        if (nb > 1)
            t += waves((double)n_seq * H * ng * (nb - 1)) * (0.9 * c + 4) + 6 +
                 (double)n_seq * nb * H * nel * 8 / 4e6;
        if (t < least * 0.97) {
            least = t;
            best = c;
        }
    }
    return best * kQ;
}

struct TcWs {
    size_t slot, blk_start, gtot, X, Y, fin, ri, ci, rp, cp, dq32, dk32, part, total;
    int L, nb, n_slots, multi;
};
TcWs tc_ws(const LinCall &c, bool bwd) {
    TcWs w{};
    const bool varlen = c.cu != nullptr;
    const int n_seq = varlen ? c.n_seq : c.B;
    const size_t nel = (size_t)c.dk_ * c.dv_, rows = (size_t)c.B * c.T;
    const int gk = groups(c.dk_), gv = groups(c.dv_);
    w.L = block_len(n_seq, varlen, c.B, c.T, c.H, bwd && gk > gv ? gk : gv, nel);
    if (w.L < kQ) w.L = kQ;
    w.nb = (c.T + w.L - 1) / w.L;
    w.n_slots = varlen ? c.T / w.L + n_seq : c.B * w.nb;
    w.multi = w.nb > 1;
    const size_t sh = (size_t)w.n_slots * c.H;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += up256(bytes);
        return at;
    };
    w.slot = take(varlen ? sizeof(int4) * w.n_slots : 0);
    w.blk_start = take(varlen ? sizeof(int) * ((size_t)3 * n_seq + 1) : 0);
    w.gtot = take(w.multi ? sh * 4 : 0);
    w.X = take(w.multi ? sh * nel * 4 : 0);
    if (bwd) {
        w.Y = take(w.multi ? sh * nel * 4 : 0);
        w.fin = take((size_t)n_seq * c.H * nel * 4);
        w.ri = take(rows * c.H * gk * 4);
        w.ci = take(rows * c.H * gk * 4);
        w.rp = take(rows * c.H * 4);
        w.cp = take(rows * c.H * 4);
        w.dq32 = take(c.Hk < c.H ? rows * c.H * c.dk_ * 4 : 0);
        w.dk32 = take(c.Hk < c.H ? rows * c.H * c.dk_ * 4 : 0);
        w.part = take((size_t)n_seq * c.H * 4);
    }
    w.total = o ? o : 256;  // 0 stands for a refused call
    return w;
}
// what the shared pieces (plan, carry, sums) need of it
gdr_host::LinWs common_ws(const TcWs &w) {
    gdr_host::LinWs l{};
    l.slot = w.slot;
    l.blk_start = w.blk_start;
    l.gtot = w.gtot;
    l.n_slots = w.n_slots;
    l.nb = w.nb;
    l.L = w.L;
    return l;
}

bool tile_map(CUtensorMap *m, const void *base, int d, int heads, size_t rows) {
    auto fn = gdr_host::tmap::encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * heads};
    cuuint32_t box[3] = {64, 1, kQ}, es[3] = {1, 1, 1};
    return fn(m, gdr_host::tmap::kBF, 3, const_cast<void *>(base), dims, strides, box, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Maps {
    CUtensorMap q, k, v, o;
};
bool make_maps(Maps *m, const LinCall &c) {
    const size_t rows = (size_t)c.B * c.T;
    return tile_map(&m->q, c.q, c.dk_, c.Hk, rows) && tile_map(&m->k, c.k, c.dk_, c.Hk, rows) &&
           tile_map(&m->v, c.v, c.dv_, c.H, rows) && (!c.dout || tile_map(&m->o, c.dout, c.dv_, c.H, rows));
}

template <bool REV, int MODE>
cudaError_t launch_chain(const LinCall &c, const Geo &geo, const Plan &plan, const CUtensorMap &a,
                         const CUtensorMap &b, const CUtensorMap &cc, TcArgs p, int id) {
    const size_t smem = TcSmem<MODE>::TOTAL;
    cudaError_t e = cudaFuncSetAttribute(chain_kernel<REV, MODE>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    p.g = c.g;
    p.ng = groups(p.dc);
    p.wide = ((uintptr_t)p.out & 31u) == 0;
    gdr_host::ProfToken tk = gdr_host::prof_begin(id, c.st);
    chain_kernel<REV, MODE><<<(unsigned)(geo.n_slots * geo.H * p.ng), kTcThreads, smem, c.st>>>(
        a, b, cc, p, geo, plan, c.err);
    gdr_host::prof_end(tk, c.st);
    return cudaGetLastError();
}

}  // namespace

namespace gdr_host {

size_t lin_tc_ws_bytes(const LinCall &c, bool bwd) { return tc_ws(c, bwd).total; }

cudaError_t lin_fwd_tc(const LinCall &c) {
    const TcWs w = tc_ws(c, false);
    const LinWs l = common_ws(w);
    Geo geo = lin_geo(c, l);
    geo.keep_empty = 1;
    const Plan plan = {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
    Maps m;
    if (!make_maps(&m, c)) return cudaErrorUnknown;
    cudaError_t e;
    if ((e = lin_plan(c, geo, l)) != cudaSuccess) return e;
    TcArgs p{};
    p.ha = p.hb = c.Hk; p.hc = c.H; p.he = c.H;
    p.db = c.dk_; p.dc = c.dv_;
    float *X = (float *)(c.ws + w.X);
    if (w.multi) {
        TcArgs s = p;
        s.xout = X;
        s.gtot = (float *)(c.ws + w.gtot);
        if ((e = launch_chain<false, kStateOnly>(c, geo, plan, m.k, m.k, m.v, s, GDR_K_LIN_STATE)) != cudaSuccess)
            return e;
        if ((e = lin_scan(c, geo, l, X, c.S0, nullptr, false)) != cudaSuccess) return e;
    }
    p.multi = w.multi;
    p.xin = w.multi ? X : c.S0;
    p.xout = c.S_final;
    p.out = c.out;
    return launch_chain<false, kOut>(c, geo, plan, m.q, m.k, m.v, p, GDR_K_LIN_OUT);
}

cudaError_t lin_bwd_tc(const LinCall &c) {
    const TcWs w = tc_ws(c, true);
    const LinWs l = common_ws(w);
    Geo geo = lin_geo(c, l);
    geo.keep_empty = 1;
    const Plan plan = {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
    Maps m;
    if (!make_maps(&m, c)) return cudaErrorUnknown;
    cudaError_t e;
    if ((e = lin_plan(c, geo, l)) != cudaSuccess) return e;
    const bool shared = c.Hk < c.H;
    float *X = (float *)(c.ws + w.X), *Y = (float *)(c.ws + w.Y), *fin = (float *)(c.ws + w.fin);
    float *ri = (float *)(c.ws + w.ri), *ci = (float *)(c.ws + w.ci);
    float *rp = (float *)(c.ws + w.rp), *cp = (float *)(c.ws + w.cp);
    float *part = c.gate == GDR_GATE_HEAD ? (float *)(c.ws + w.part) : nullptr;
    if (w.multi) {
        TcArgs s{};
        s.ha = s.hb = c.Hk; s.hc = c.H; s.he = c.H;
        s.db = c.dk_; s.dc = c.dv_;
        s.gtot = (float *)(c.ws + w.gtot);
        s.xout = X;
        if ((e = launch_chain<false, kStateOnly>(c, geo, plan, m.k, m.k, m.v, s, GDR_K_LIN_STATE)) != cudaSuccess)
            return e;
        if ((e = lin_scan(c, geo, l, X, c.S0, nullptr, false)) != cudaSuccess) return e;
        s.xout = Y;
        if ((e = launch_chain<true, kStateOnly>(c, geo, plan, m.q, m.q, m.o, s, GDR_K_LIN_STATE)) != cudaSuccess)
            return e;
        if ((e = lin_scan(c, geo, l, Y, c.dS_final, nullptr, true)) != cudaSuccess) return e;
    }
    // dq: (a, b, c) = (dout, v, k), the state transposed
    TcArgs p{};
    p.multi = w.multi;
    p.ha = p.hb = c.H; p.hc = p.he = c.Hk;
    p.db = c.dv_; p.dc = c.dk_; p.tr = 1;
    p.out32 = shared;
    p.xin = w.multi ? X : c.S0;
    p.xout = c.dS_final ? fin : nullptr;
    p.out = shared ? (void *)(c.ws + w.dq32) : c.dq;
    p.e = (const __nv_bfloat16 *)c.q;
    p.dots = ri;
    if ((e = launch_chain<false, kOutDots>(c, geo, plan, m.o, m.v, m.k, p, GDR_K_LIN_GRAD)) != cudaSuccess)
        return e;
    // dk: (v, dout, q), backward in time
    p.xin = w.multi ? Y : c.dS_final;
    p.xout = nullptr;
    p.out = shared ? (void *)(c.ws + w.dk32) : c.dk;
    p.e = (const __nv_bfloat16 *)c.k;
    p.dots = ci;
    if ((e = launch_chain<true, kOutDots>(c, geo, plan, m.v, m.o, m.q, p, GDR_K_LIN_GRAD)) != cudaSuccess)
        return e;
    // dv: (k, q, dout), backward in time
    TcArgs r{};
    r.multi = w.multi;
    r.ha = r.hb = c.Hk; r.hc = r.he = c.H;
    r.db = c.dk_; r.dc = c.dv_;
    r.xin = w.multi ? Y : c.dS_final;
    r.xout = c.dS0;
    r.out = c.dv;
    if ((e = launch_chain<true, kOut>(c, geo, plan, m.k, m.q, m.o, r, GDR_K_LIN_GRAD)) != cudaSuccess) return e;
    if (shared) {
        if ((e = lin_group_sum(c, geo, l, (const float *)(c.ws + w.dq32), c.dq, c.dk_)) != cudaSuccess) return e;
        if ((e = lin_group_sum(c, geo, l, (const float *)(c.ws + w.dk32), c.dk, c.dk_)) != cudaSuccess) return e;
    }
    if ((e = cudaFuncSetAttribute(pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)PairSmem::TOTAL)) != cudaSuccess)
        return e;
    const long units = (long)geo.n_slots * geo.H, most = w.L / kQ;
    long split = (4 * 148 + units - 1) / units;
    if (split > most) split = most;
    PairArgs pa{c.g, rp, cp, c.Hk, c.dk_, c.dv_};
    ProfToken tk = prof_begin(GDR_K_LIN_GRAD, c.st);
    pair_kernel<<<dim3((unsigned)units, (unsigned)split), kTcThreads, PairSmem::TOTAL, c.st>>>(
        m.q, m.k, m.v, m.o, pa, geo, plan, c.err);
    prof_end(tk, c.st);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    DgArgs d{ri, ci, rp, cp, groups(c.dk_), groups(c.dk_), fin, c.dS_final, c.dg, part, c.dk_ * c.dv_};
    tk = prof_begin(GDR_K_LIN_GRAD, c.st);
    dg_chunks_kernel<<<(unsigned)(geo.n_seq * geo.H), 1024, 0, c.st>>>(d, c.cu, geo, plan);
    prof_end(tk, c.st);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    if (!part) return cudaSuccess;
    Geo by_seq = geo;  // one sum per sequence and head
    by_seq.n_slots = geo.n_seq;
    return lin_dg_heads(c, by_seq, part);
}

}  // namespace gdr_host
