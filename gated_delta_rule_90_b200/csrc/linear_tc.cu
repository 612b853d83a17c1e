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
// chunk: (w C)^T B does not depend on X, so the chunks' products overlap.  64
// columns, not all of d_c: two walks of a head then share a and b through L2, and
// shared memory holds two buffers of each tile beside the split.
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
constexpr int kTcThreads = 640;          // 8 output warps, 8 state warps, TMA and decays, 3 MMA issuers
constexpr uint32_t kAtom = kQ * 128;     // bytes of 128 rows of 64 bf16
constexpr float kLog2e = 1.4426950408889634f;

enum { kStateOnly = 0, kOut = 1, kOutDots = 2 };
constexpr int kRun = kRunLen / kQ;  // chunks of a run

// Tables of a chunk's decays (floats): LC sums inside each 32-token block in
// units of log 2, CF column factors, then scalars by block (see decay_tables); for
// the pairs also LL, what LC leaves of its sums.
enum { kLC = 0, kCF = 128, kSS = 256, kSE = 260, kBB = 264, kDEC = 270, kTab = 272, kLL = 272, kPairTab = 400 };

// Shared memory of a CTA.  Two buffers of each tile, the three terms of w C, and
// X in one term; where X takes three, a has one buffer (it is free early: its two
// products come first).
template <int MODE>
struct TcSmem {
    static constexpr int NA = MODE == kOutDots ? 1 : 2, NB = 2, NC = 2;
    static constexpr int XT = MODE == kOutDots ? 3 : 1;
    static constexpr uint32_t A = 0;
    static constexpr uint32_t B = A + (MODE == kStateOnly ? 0 : NA * 2 * kAtom);
    static constexpr uint32_t Cc = B + NB * 2 * kAtom;
    static constexpr uint32_t CP = Cc + NC * kAtom;       // w C, three terms
    static constexpr uint32_t X = CP + 3 * kAtom;
    static constexpr uint32_t TAB = X + (MODE == kStateOnly ? 0 : XT * kAtom);
    static constexpr uint32_t BARS = TAB + 2 * kTab * 4;
    static constexpr uint32_t TOTAL = BARS + 34 * 8 + 16;
    static_assert(TOTAL <= 227 * 1024, "shared memory");
};

// Tensor memory columns.  SD = (w C)^T B, a block per split term, in one product
// 192 columns wide: an MMA took 74 cycles at up to 128 columns, 100 at 192, so three
// of 64 cost 240; and added into one block, the small terms' steps round at the size
// of the large one's sum (1.9e-7 of the state, against 6.5e-8 apart).  P is replaced
// in place by its bf16 form (8 columns of each 16).  O = P C has two buffers, so that
// a chunk's outputs are written after the next chunk's P, whose products run
// meanwhile (LAG).  With three terms of X, OIN = A X^T takes two blocks (the first
// term; the others) and O one buffer.
template <int MODE>
struct TcTmem {
    static constexpr bool DOTS = MODE == kOutDots;
    static constexpr int LAG = DOTS ? 0 : 1;
    static constexpr int SD = 0, P = 192, O = 320, OIN = DOTS ? 384 : 448;
    static constexpr uint32_t COLS = MODE == kStateOnly ? 256 : 512;
};

struct TcArgs {
    const float *g;
    const float *xin;    // state that enters a sequence, or NULL (zero)
    const float *xblk;   // state that enters a block of a sequence of several, per (slot, head)
    float *xout;         // state that leaves (per sequence), or the blocks' own states (state only)
    float *gtot;         // state only: the blocks' sums of log-decays
    void *out;           // bf16, or fp32 with out32
    const __nv_bfloat16 *e;  // dots: rows that the state's part of out is multiplied with
    float *dots;         // [2 x column groups, rows, H]
    // dots, forward: the state where a run starts, as the state's threads hold it; reverse: its
    // products with the gradient of that state, by warp
    float *bnd, *ydot;
    Runs runs;
    int ha, hb, hc, he;  // heads of a, b, c, e
    int db, dc, ng;      // widths, column groups
    int tr;              // states are stored as the transpose of X
    int out32, wide;     // out is fp32; out is 32-byte aligned
};

// Bounded wait: the loop rolled, for the kernels below are held back by the size
// of their code.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, unsigned int *err) {
#pragma unroll 1
    for (uint32_t i = 0; i < kSpinTc; ++i)
        if (mbar_try_wait(bar, parity)) return true;
    if (err) atomicOr(err, kErrTimeout);
    return false;
}
__device__ __forceinline__ void tma_load_3d(void *dst, const void *tmap, uint64_t *bar, int x, int y,
                                            int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
// MMAs and commits of one elected lane, in code that the whole warp runs: the
// descriptors then live in uniform registers.  Under a branch on the lane each
// MMA cost about ten instructions to move them there, which set its pace.
__device__ __forceinline__ void mma_ss(uint32_t el, uint32_t d, uint64_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc), "r"(el));
}
__device__ __forceinline__ void mma_ts(uint32_t el, uint32_t d, uint32_t a, uint64_t b, uint32_t id,
                                       uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "r"(acc), "r"(el));
}
__device__ __forceinline__ void commit(uint32_t el, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            smem_u32(bar)), "r"(el)
        : "memory");
}
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(e));
    return e;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
                 "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
                 "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
                 : "memory");
}
__device__ __forceinline__ void st32(void *p, const uint32_t *w) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}
// Packed pairs of fp32 (one instruction for two).
__device__ __forceinline__ uint64_t pk(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpk(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ void mul2(float &a, float &b, float x, float y) {  // a *= x, b *= y
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a, b)), "l"(pk(x, y)));
    unpk(r, a, b);
}
__device__ __forceinline__ void add2(float &a, float &b, float x, float y) {  // a += x, b += y
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pk(a, b)), "l"(pk(x, y)));
    unpk(r, a, b);
}
__device__ __forceinline__ void fma2(float &a, float &b, float m, float x, float y) {  // a += m x, b += m y
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pk(m, m)), "l"(pk(x, y)), "l"(pk(a, b)));
    unpk(r, a, b);
}
// x0, x1 -> the bf16 pairs of the three truncated terms: x = hi + mid + lo, the
// differences exact.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t &hi, uint32_t &mid, uint32_t &lo) {
    const uint32_t u0 = __float_as_uint(x0), u1 = __float_as_uint(x1);
    hi = __byte_perm(u0, u1, 0x7632);
    float r0 = x0, r1 = x1;
    add2(r0, r1, -__uint_as_float(u0 & 0xffff0000u), -__uint_as_float(u1 & 0xffff0000u));
    const uint32_t m0 = __float_as_uint(r0), m1 = __float_as_uint(r1);
    mid = __byte_perm(m0, m1, 0x7632);
    add2(r0, r1, -__uint_as_float(m0 & 0xffff0000u), -__uint_as_float(m1 & 0xffff0000u));
    lo = __byte_perm(__float_as_uint(r0), __float_as_uint(r1), 0x7632);
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// 16 bytes, asked for where this stands: a load that the compiler may move down to its
// use costs the gradients of a batch 9 % (467 us, 427 so), and one of the read-only kind
// may be moved above stream_order().
__device__ __forceinline__ uint4 load_row4(const void *p) {
    uint4 x;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                 : "l"(p));
    return x;
}

// A log-decay, unclamped: a clamp where it is loaded would make the warp wait for
// the load there (3300 cycles a chunk), not where the value is needed.
__device__ __forceinline__ float load_raw_g(const Geo &geo, const float *g, long row, int h) {
    float x;
    asm volatile("ld.global.f32 %0, [%1];" : "=f"(x) : "l"(geo.gate_head ? g + h : g + row * geo.H + h));
    return x;
}

// A number in two floats, hi + lo (about 48 bits): sums by Knuth's exact two-sum.
// The running sums of log-decays need it, for differences of far positions have to
// be rounded once, not at the size of the sums.  In fp64 the
// chunks waited for them (forward, B4 T4096 H16 d128: 106 us, 99 so).
struct Two {
    float h, l;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Two add(const Two &a, const Two &b) {
    const Two s = two_sum(a.h, b.h);
    const float l = s.l + (a.l + b.l), h = s.h + l;
    return {h, l - (h - s.h)};
}
__device__ __forceinline__ Two sub(const Two &a, const Two &b) { return add(a, {-b.h, -b.l}); }
__device__ __forceinline__ float diff(const Two &a, const Two &b) {
    const Two s = two_sum(a.h, -b.h);
    return s.h + (s.l + (a.l - b.l));
}
__device__ __forceinline__ Two shfl(const Two &a, int lane) {
    return {__shfl_sync(0xffffffffu, a.h, lane), __shfl_sync(0xffffffffu, a.l, lane)};
}

// The decays of one chunk (one warp; lane: 4 consecutive tokens), from running
// sums G.  All weights are products of factors around the borders s_b, e_b of the
// 32-token blocks, each at most 1 for decays, so nothing overflows:
//   pair (i, j) in different blocks: row factor(i) BB(blocks) column factor(j),
//     forward e^{G_i - s} and e^{e - G_j}, reverse e^{e - G_i} and e^{G_j - s};
//   pair in one block: 2^(difference of LC);
//   w_j = column factor(j) SE or SS(block), the state's weight = row factor(i) SS or SE,
// SS_b = e^{s_b}, SE_b = e^{G_n - e_b}, BB = e^{s_later - e_earlier}.  Returns G_n.
// LC is taken from the border of the row factor, s forward and e reverse, so that this
// factor is the power of a sum rounded once, at its own size.  A difference of two LC is
// rounded at the size of the sums: after decays of 0 earlier in the block (-104 each, 32 of
// them at most) by up to 2^-11, less than the rounding of P to bf16 (2^-8), which is all
// that the walks use it for.  The pairs, whose sums are fp32, need LL as well (their dg was
// off by 8.5e-5 of its norm where every 4th decay was 0, by 3.5e-7 so).
template <bool REV, bool LOW = false>
__device__ __forceinline__ Two decay_tables(float *tab, const float (&gv)[4], int lane) {
    Two p[4];
    p[0] = {gv[0], 0.f};
#pragma unroll
    for (int u = 1; u < 4; ++u) p[u] = add(p[u - 1], {gv[u], 0.f});
    Two inc = p[3];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Two y = {__shfl_up_sync(0xffffffffu, inc.h, o), __shfl_up_sync(0xffffffffu, inc.l, o)};
        const Two z = add(inc, y);
        if (lane >= o) inc = z;
    }
    Two base = {__shfl_up_sync(0xffffffffu, inc.h, 1), __shfl_up_sync(0xffffffffu, inc.l, 1)};
    if (lane == 0) base = {0.f, 0.f};
    const Two Gn = shfl(inc, 31);
    // the sum up to border b (0..4)
    auto border = [&](int b) {
        const Two y = shfl(base, 8 * (b & 3));
        return b == 4 ? Gn : y;
    };
    const int kb = lane >> 3;
    const Two s0 = border(kb), s1 = border(kb + 1);
    float lc[4], ll[4], cf[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const Two G = add(base, p[u]);
        const Two L = sub(G, REV ? s1 : s0);
        lc[u] = L.h * kLog2e;
        ll[u] = fmaf(L.h, kLog2e, -lc[u]) + L.l * kLog2e;
        cf[u] = expf(REV ? diff(G, s0) : diff(s1, G));
    }
    reinterpret_cast<float4 *>(tab + kLC)[lane] = make_float4(lc[0], lc[1], lc[2], lc[3]);
    if (LOW) reinterpret_cast<float4 *>(tab + kLL)[lane] = make_float4(ll[0], ll[1], ll[2], ll[3]);
    reinterpret_cast<float4 *>(tab + kCF)[lane] = make_float4(cf[0], cf[1], cf[2], cf[3]);
    // lanes 0-3 SS, 4-7 SE, 8-13 BB (pairs 10 20 21 30 31 32), 14 DEC
    int hi = lane & 3, lo = 0;
    if (lane >= 4 && lane < 8) { hi = 4; lo = lane - 3; }
    if (lane >= 8 && lane < 14) {
        hi = lane < 9 ? 1 : lane < 11 ? 2 : 3;
        lo = lane - 8 - hi * (hi - 1) / 2 + 1;
    }
    if (lane == 14) hi = 4;
    const Two bh = border(hi), bl = border(lo);
    if (lane < 15) tab[kSS + lane] = expf(diff(bh, bl));
    return Gn;
}
// row factor of a row from its LC
template <bool REV>
__device__ __forceinline__ float row_factor(float li) {
    return exp2f(REV ? -li : li);
}

// Roles of the 20 warps: 8 of outputs, 8 of the state; the decays; TMA with the MMAs
// of P; the MMAs of A X^T and P C; those of (w C)^T B.  Each role works a chunk
// ahead of the one that needs its results, over mbarriers; no wait lags a barrier
// by two phases (every phase needs an arrival of the waiter, or of one that
// follows it).
//
// Loops over columns are rolled where they can be: the five roles' unrolled code
// did not fit the instruction caches, and warps waited for instructions most of
// the time (forward, B4 T4096 H16 d128: 225 us unrolled, 151 us rolled; 88 to 95 us now).
// Bound by the latencies of the chain of hand-offs of a chunk (5,500 cycles), not by
// a pipe: issue slots 52 %, tensor 35 %, shared memory 45 %, DRAM 32 % busy at that size.
template <bool REV, int MODE>
__device__ __forceinline__ void walk(unsigned int bid, const CUtensorMap &tm_a, const CUtensorMap &tm_b,
                                     const CUtensorMap &tm_c, const TcArgs &p, const Geo &geo, const Plan &plan,
                                     unsigned int *err) {
    using SM = TcSmem<MODE>;
    using TM = TcTmem<MODE>;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + SM::BARS);
    uint64_t *fullA = bars, *fullB = bars + 2, *fullC = bars + 4;      // tile loaded
    uint64_t *freeA = bars + 6, *freeB = bars + 8, *freeC = bars + 10; // its readers are done
    uint64_t *pfull = bars + 12, *pready = bars + 14, *ofull = bars + 15;  // P and decays; its bf16 form; O
    uint64_t *ifull = bars + 16, *ifree = bars + 17;                   // OIN; O and OIN written out
    uint64_t *cready = bars + 20;                   // [2] w C, tokens 0-63 and 64-127
    uint64_t *sfree = bars + 22, *sfull = bars + 23, *sdfree = bars + 24;  // first half done; SD
    uint64_t *xready = bars + 25, *tfree = bars + 26, *zready = bars + 28;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 32);
    float *tabs = reinterpret_cast<float *>(sm + SM::TAB);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    const int ng = bid % p.ng, sh = bid / p.ng;
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
                      chk_true((smem_u32(sm) & 1023u) == 0 && len <= geo.L, err) &&
                      (MODE != kOutDots || chk_span(run_of(geo, p.runs, t0, slot),
                                                    (len + kRunLen - 1) / kRunLen, p.runs.count, err))))
        return;

    if (tid == 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            mbar_init(&fullA[i], 1);
            mbar_init(&fullB[i], 1);
            mbar_init(&fullC[i], 2);  // the tile and the chunk's decays
            mbar_init(&pfull[i], 2);
            mbar_init(&freeA[i], 2);
            mbar_init(&freeB[i], MODE == kStateOnly ? 1 : 2);
            mbar_init(&freeC[i], MODE == kStateOnly ? 8 : 9);  // the 8 split warps; O = P C
            mbar_init(&cready[i], 8);
            mbar_init(&tfree[i], MODE == kStateOnly ? 8 : 16);
        }
        mbar_init(pready, 8);
        mbar_init(ofull, 1);
        mbar_init(ifull, 1);
        mbar_init(ifree, 8);
        mbar_init(sfree, 1);
        mbar_init(sfull, 1);
        mbar_init(sdfree, 8);
        mbar_init(xready, 8);
        mbar_init(zready, 8);
        fence_mbar_init();
        prefetch_tmap(&tm_b);
        prefetch_tmap(&tm_c);
        if (MODE != kStateOnly) prefetch_tmap(&tm_a);
    }
    if (warp == 16) {
        tmem_alloc(tslot, TM::COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tslot;
    const int na = p.db > 64 ? 2 : 1;  // 64-wide column blocks of a and b
    bool ok = true;
    // first token of chunk cc of the walk
    auto chunk_at = [&](int cc) { return (REV ? nch - 1 - cc : cc) * kQ; };

    if (warp == 16) {
        // ===================== decays =====================
        float gv[4];
        auto load = [&](int cc) {
            const int j0 = chunk_at(cc), n = min(kQ, len - j0);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                gv[u] = 4 * lane + u < n ? load_raw_g(geo, p.g, (long)t0 + j0 + 4 * lane + u, h) : 0.f;
        };
        Two tot = {0.f, 0.f};
        if (nch > 0) load(0);
        for (int cc = 0; cc < nch; ++cc) {
            const int i2 = cc & 1;
            if (cc >= 2) ok = ok && wait(&tfree[i2], (cc / 2 - 1) & 1, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int u = 0; u < 4; ++u) gv[u] = clamp_g(gv[u]);
            tot = add(tot, decay_tables<REV>(tabs + i2 * kTab, gv, lane));
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&fullC[i2]);
                if (MODE != kStateOnly) mbar_arrive(&pfull[i2]);
            }
            __syncwarp();
            if (cc + 1 < nch) load(cc + 1);
        }
        if (MODE == kStateOnly && p.gtot && ng == 0) {
            if (lane == 0) p.gtot[(size_t)slot * geo.H + h] = tot.h;
        }
    } else if (warp == 17) {
        // ===================== TMA loads; MMA: P = A B^T =====================
        // the tiles of chunk cc, as their buffers fall free.  (The whole warp waits: under a branch
        // on the lane, the code after the waits ran apart for that lane and took several times as long.)
        auto issue = [&](int cc) {
            const int i2 = cc & 1, y = t0 + chunk_at(cc), ia = SM::NA == 2 ? i2 : 0;
            if (cc >= 2) ok = ok && wait(&freeB[i2], (cc / 2 - 1) & 1, err);
            if (ok && lane == 0) {
                mbar_arrive_expect_tx(&fullB[i2], na * kAtom);
                for (int i = 0; i < na; ++i)
                    tma_load_3d(sm + SM::B + (i2 * 2 + i) * kAtom, &tm_b, &fullB[i2], 64 * i, hb, y);
            }
            __syncwarp();
            if (cc >= 2) ok = ok && wait(&freeC[i2], (cc / 2 - 1) & 1, err);
            if (ok && lane == 0) {
                mbar_arrive_expect_tx(&fullC[i2], kAtom);
                tma_load_3d(sm + SM::Cc + i2 * kAtom, &tm_c, &fullC[i2], c0, hc, y);
            }
            __syncwarp();
            if (MODE != kStateOnly) {
                if (cc >= SM::NA) ok = ok && wait(&freeA[ia], (cc / SM::NA - 1) & 1, err);
                if (ok && lane == 0) {
                    mbar_arrive_expect_tx(&fullA[ia], na * kAtom);
                    for (int i = 0; i < na; ++i)
                        tma_load_3d(sm + SM::A + (ia * 2 + i) * kAtom, &tm_a, &fullA[ia], 64 * i, ha, y);
                }
                __syncwarp();
            }
        };
        const uint32_t el = elect_lane(), idP = idesc_bf16(128, 128, 0, 0);
        const uint64_t dA = sdesc_sw128(smem_u32(sm + SM::A), 16, 1024);
        const uint64_t dB = sdesc_sw128(smem_u32(sm + SM::B), 16, 1024);
        const int ks = p.db / 16;
        // ahead of the products as far as the buffers go
#pragma unroll 1
        for (int cc = 0; cc < min(nch, SM::NA); ++cc) issue(cc);
        for (int cc = 0; cc < nch; ++cc) {
            if (MODE != kStateOnly) {
                const int i2 = cc & 1, ia = SM::NA == 2 ? i2 : 0;
                ok = ok && wait(&fullA[ia], (cc / SM::NA) & 1, err);
                ok = ok && wait(&fullB[i2], (cc >> 1) & 1, err);
                // rows past the end are zeroed before they are multiplied (one chunk of the walk)
                if (len - chunk_at(cc) < kQ) ok = ok && wait(zready, 0, err);
                if (cc > 0) ok = ok && wait(ofull, (cc - 1) & 1, err);  // the last P is read
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const uint64_t da = sdesc_add(dA, ia * 2 * kAtom), db = sdesc_add(dB, i2 * 2 * kAtom);
#pragma unroll 1
                for (int kk = 0; kk < ks; ++kk) {
                    const uint32_t o = (kk >> 2) * kAtom + (kk & 3) * 32;
                    mma_ss(el, tmem + TM::P, sdesc_add(da, o), sdesc_add(db, o), idP, kk > 0);
                }
                commit(el, &freeA[ia]);
                commit(el, &freeB[i2]);
                commit(el, &pfull[i2]);
            }
            if (cc + 1 >= SM::NA && cc + 1 < nch) issue(cc + 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
        }
        // every load has landed and every product has read its tiles before the CTA ends:
        // free(i) follows full(i), so waiting for the last use of each buffer covers both
        for (int cc = max(nch - 2, 0); cc < nch; ++cc) {
            wait(&freeB[cc & 1], (cc / 2) & 1, err);
            wait(&freeC[cc & 1], (cc / 2) & 1, err);
            if (MODE != kStateOnly && cc >= nch - SM::NA)
                wait(&freeA[SM::NA == 2 ? cc & 1 : 0], (cc / SM::NA) & 1, err);
        }
        __syncwarp();
    } else if (warp == 18) {
        // ===================== MMA: OIN = A X^T, O = P C =====================
        if (MODE != kStateOnly) {
            const uint32_t el = elect_lane(), idN = idesc_bf16(128, kN, 0, 1);
            const uint64_t dA = sdesc_sw128(smem_u32(sm + SM::A), 16, 1024);
            const uint64_t dC = sdesc_sw128(smem_u32(sm + SM::Cc), kAtom, 1024);
            const uint64_t dX = sdesc_sw128(smem_u32(sm + SM::X), kAtom, 1024);
            const int ks = p.db / 16;
            for (int cc = 0; cc < nch; ++cc) {
                const int i2 = cc & 1, ia = SM::NA == 2 ? i2 : 0;
                // the product with X waits for the outputs of the chunk before: with LAG these come
                // after P of this chunk, so O goes first; else X does, which frees the a tile early
#pragma unroll
                for (int step = 0; step < 2; ++step) {
                    if (step == (TM::LAG ? 0 : 1)) {
                        ok = ok && wait(&fullC[i2], (cc >> 1) & 1, err);
                        ok = ok && wait(pready, cc & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t d = sdesc_add(dC, i2 * kAtom);
                        const uint32_t tO = tmem + TM::O + (TM::LAG ? i2 * kN : 0);
#pragma unroll 1
                        for (int kk = 0; kk < 8; ++kk)
                            mma_ts(el, tO, tmem + TM::P + kk * 16, sdesc_add(d, kk * 2048), idN, kk > 0);
                        commit(el, &freeC[i2]);
                        commit(el, ofull);
                    } else {
                        ok = ok && wait(&fullA[ia], (cc / SM::NA) & 1, err);
                        ok = ok && wait(xready, cc & 1, err);
                        if (cc > 0) ok = ok && wait(ifree, (cc - 1) & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        tc_fence_after();
                        const uint64_t da = sdesc_add(dA, ia * 2 * kAtom);
#pragma unroll 1
                        for (int kk = 0; kk < ks; ++kk) {
                            const uint64_t a = sdesc_add(da, (kk >> 2) * kAtom + (kk & 3) * 32);
                            const uint64_t b = sdesc_add(dX, kk * 2048);
                            mma_ss(el, tmem + TM::OIN, a, b, idN, kk > 0);
                            if (TM::DOTS) {
                                mma_ss(el, tmem + TM::OIN + kN, a, sdesc_add(b, kAtom), idN, kk > 0);
                                mma_ss(el, tmem + TM::OIN + kN, a, sdesc_add(b, 2 * kAtom), idN, 1);
                            }
                        }
                        commit(el, &freeA[ia]);
                        commit(el, ifull);
                    }
                }
                if (!ok) break;
            }
        }
    } else if (warp == 19) {
        // ===================== MMA: SD = (w C)^T B, half the tokens at a time =====================
        {
            const uint32_t el = elect_lane(), idS = idesc_bf16(128, 3 * kN, 1, 1);
            // b as [d_b, tokens]: with one 64-wide block the upper lanes repeat it (not read)
            const uint64_t dB = sdesc_sw128(smem_u32(sm + SM::B), na > 1 ? kAtom : 0, 1024);
            const uint64_t dP = sdesc_sw128(smem_u32(sm + SM::CP), kAtom, 1024);
            for (int cc = 0; cc < nch; ++cc) {
                const int i2 = cc & 1;
                ok = ok && wait(&fullB[i2], (cc >> 1) & 1, err);
                if (cc > 0) ok = ok && wait(sdfree, (cc - 1) & 1, err);
                const uint64_t db = sdesc_add(dB, i2 * 2 * kAtom);
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    ok = ok && wait(&cready[hf], cc & 1, err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll 1
                    for (int kk = 4 * hf; kk < 4 * hf + 4; ++kk)
                        mma_ss(el, tmem + TM::SD, sdesc_add(db, kk * 2048), sdesc_add(dP, kk * 2048), idS, kk > 0);
                    if (hf == 0) commit(el, sfree);
                }
                if (!ok) break;
                commit(el, &freeB[i2]);
                commit(el, sfull);
            }
        }
    } else if (warp < 8) {
        // ===================== outputs: row i of the chunk, half the columns =====================
        // P of chunk cc, then the outputs of chunk cc - LAG
        if (MODE != kStateOnly) {
            const int rb = warp & 3, hf = warp >> 2, i = rb * 32 + lane;
            const uint32_t lb = (uint32_t)(rb * 32) << 16;
            const int ncb = min(kN, p.dc - c0) >> 4;
            float eg = 0.f;  // weight of the state that entered chunk cc - 1
            uint4 ev[4];     // DOTS: this row's 32 columns of e, asked for before P
            for (int cc = 0; cc < nch + TM::LAG; ++cc) {
                float egn = 0.f;
                if (MODE == kOutDots) {
                    const int n = min(kQ, len - chunk_at(cc));
                    const size_t row = (size_t)t0 + chunk_at(cc) + i;
                    const __nv_bfloat16 *e = p.e + (row * p.he + h / (geo.H / p.he)) * p.dc + c0 + 32 * hf;
#pragma unroll
                    for (int u = 0; u < 4; ++u)
                        ev[u] = i < n && c0 + 32 * hf + 8 * u < p.dc
                                    ? load_row4(reinterpret_cast<const uint4 *>(e) + u)
                                    : make_uint4(0, 0, 0, 0);
                }
                if (cc < nch) {
                    const float *tab = tabs + (cc & 1) * kTab;
                    ok = ok && wait(&pfull[cc & 1], (cc >> 1) & 1, err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    const float li = tab[kLC + i], rf = row_factor<REV>(li);
                    egn = rf * tab[(REV ? kSE : kSS) + rb];
                    // weights of the pairs: this half's 16 columns of each block
#pragma unroll 1
                    for (int b = 0; b < 4; ++b) {
                        const int col = 32 * b + 16 * hf;
                        float w[8];
                        if (REV ? b < rb : b > rb) {
#pragma unroll
                            for (int u = 0; u < 8; ++u) w[u] = 0.f;
                        } else {
                            float x[16], f[16];
                            tmem_ld16(tmem + TM::P + lb + col, x);
#pragma unroll
                            for (int u4 = 0; u4 < 4; ++u4) {
                                const float4 l = *reinterpret_cast<const float4 *>(
                                    tab + (b == rb ? kLC : kCF) + col + 4 * u4);
                                f[4 * u4] = l.x; f[4 * u4 + 1] = l.y; f[4 * u4 + 2] = l.z; f[4 * u4 + 3] = l.w;
                            }
                            if (b == rb) {
#pragma unroll
                                for (int u = 0; u < 16; ++u) f[u] = ex2(REV ? f[u] - li : li - f[u]);
                            } else {
                                const int hiB = REV ? b : rb, loB = REV ? rb : b;
                                const float r = rf * tab[kBB + hiB * (hiB - 1) / 2 + loB];
#pragma unroll
                                for (int u = 0; u < 16; u += 2) mul2(f[u], f[u + 1], r, r);
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; u += 2) mul2(x[u], x[u + 1], f[u], f[u + 1]);
                            if (b == rb) {  // a select, so that what lies outside cannot matter
#pragma unroll
                                for (int u = 0; u < 16; ++u) {
                                    const bool in = REV ? u + 16 * hf >= lane : u + 16 * hf <= lane;
                                    x[u] = in ? x[u] : 0.f;
                                }
                            }
#pragma unroll
                            for (int u = 0; u < 8; ++u) w[u] = __uint_as_float(pack2(x[2 * u], x[2 * u + 1]));
                        }
                        tmem_st8(tmem + TM::P + lb + col, w);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(pready);
                        mbar_arrive(&tfree[cc & 1]);
                    }
                }
                if (cc >= TM::LAG) {
                    const int pc = cc - TM::LAG, j0 = chunk_at(pc), n = min(kQ, len - j0);
                    const size_t row = (size_t)t0 + j0 + i;
                    ok = ok && wait(ifull, pc & 1, err);
                    // (with LAG, P of chunk cc was formed after this product)
                    if (!TM::LAG || cc == nch) ok = ok && wait(ofull, pc & 1, err);
                    if (!TM::LAG) eg = egn;
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
                    float d = 0.f;
                    const size_t at = (row * geo.H + h) * p.dc + c0;
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int b = 2 * hf + v;
                        if (b >= ncb) break;
                        float o[16], y[16];
                        tmem_ld16(tmem + TM::OIN + lb + 16 * b, o);
                        tmem_ld16(tmem + TM::O + (TM::LAG ? (pc & 1) * kN : 0) + lb + 16 * b, y);
                        if (MODE == kOutDots) {
                            float m[16], f[16];
                            tmem_ld16(tmem + TM::OIN + kN + lb + 16 * b, m);
                            unpack8(ev[2 * v], f);
                            unpack8(ev[2 * v + 1], f + 8);
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; u += 2) {
                                add2(o[u], o[u + 1], m[u], m[u + 1]);
                                mul2(o[u], o[u + 1], eg, eg);
                            }
#pragma unroll
                            for (int u = 0; u < 16; ++u) d = fmaf(o[u], f[u], d);
#pragma unroll
                            for (int u = 0; u < 16; u += 2) add2(y[u], y[u + 1], o[u], o[u + 1]);
                        } else {
                            tmem_wait_ld();
#pragma unroll
                            for (int u = 0; u < 16; u += 2) fma2(y[u], y[u + 1], eg, o[u], o[u + 1]);
                        }
                        if (i < n && p.out32) {
                            float4 *q = reinterpret_cast<float4 *>((float *)p.out + at + 16 * b);
#pragma unroll
                            for (int u = 0; u < 4; ++u)
                                q[u] = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
                        } else if (i < n) {
                            uint32_t w[8];
#pragma unroll
                            for (int u = 0; u < 8; ++u) w[u] = pack2(y[2 * u], y[2 * u + 1]);
                            __nv_bfloat16 *q = (__nv_bfloat16 *)p.out + at + 16 * b;
                            if (p.wide) {
                                st32(q, w);
                            } else {
                                reinterpret_cast<uint4 *>(q)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                reinterpret_cast<uint4 *>(q)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                            }
                        }
                        __syncwarp();  // the loads above are warp-wide
                    }
                    if (MODE == kOutDots && i < n)
                        p.dots[((size_t)(2 * ng + hf) * geo.rows + row) * geo.H + h] = d;
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(ifree);
                }
                eg = egn;
            }
        }
    } else {
        // ===================== state: row k of X^T (d_b), half of the 64 columns =====================
        const int rb = warp & 3, hf = (warp >> 2) - 2, k = rb * 32 + lane;
        const int cx = c0 + 32 * hf;  // first column
        const uint32_t lb = (uint32_t)(rb * 32) << 16;
        float x[32];
#pragma unroll
        for (int u = 0; u < 32; ++u) x[u] = 0.f;
        const float *enter = nblk > 1 ? p.xblk : p.xin;
        if (MODE != kStateOnly && enter && k < p.db) {
            const float *src = enter + ((size_t)(nblk > 1 ? slot : sl.z) * geo.H + h) * nel;
            if (p.tr) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (cx + 4 * u < p.dc) {
                        const float4 y = *reinterpret_cast<const float4 *>(src + (size_t)k * p.dc + cx + 4 * u);
                        x[4 * u] = y.x; x[4 * u + 1] = y.y; x[4 * u + 2] = y.z; x[4 * u + 3] = y.w;
                    }
            } else {
#pragma unroll
                for (int u = 0; u < 32; ++u)
                    if (cx + u < p.dc) x[u] = src[(size_t)(cx + u) * p.db + k];
            }
        }
        // split of w C: row sr of a half's 64 tokens, 16 columns
        const int sw = warp - 8, sr = (sw & 1) * 32 + lane, sq = (sw >> 1) * 2;
        float dec = 0.f;  // decay over chunk cc - 1
        for (int cc = 0; cc <= nch; ++cc) {
            const int i2 = cc & 1, n = cc < nch ? min(kQ, len - chunk_at(cc)) : 0;
            const float *tab = tabs + i2 * kTab;
            float decn = 0.f;
            // kOut: split of the first half, the state of the chunk before, the second half, so that the
            // state's product runs meanwhile (95 us; the state first 103).  DOTS: the state first, for the
            // a tile's buffer waits for the product with it (119 us; between the halves 128).
#pragma unroll 1
            for (int step = 0; step < 3; ++step) {
                const bool update = step == (MODE == kOutDots ? 0 : 1);
                const int half = MODE == kOutDots ? step - 1 : step >> 1;
                if (!update && cc < nch) {
                    if (half == 0) {
                        ok = ok && wait(&fullC[i2], (cc >> 1) & 1, err);
                        if (n < kQ) ok = ok && wait(&fullB[i2], (cc >> 1) & 1, err);
                        if (cc > 0) ok = ok && wait(sfree, (cc - 1) & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
                    const int j = 64 * half + sr;
                    const float w = tab[kCF + j] * tab[(REV ? kSS : kSE) + (j >> 5)];
                    uint8_t *crow = sm + SM::Cc + i2 * kAtom + j * 128;
                    uint8_t *prow = sm + SM::CP + j * 128;
#pragma unroll 1
                    for (int b = sq; b < sq + 2; ++b) {
                        const int off = (b ^ (j & 7)) << 4;
                        uint4 hi, mid, lo;
                        hi = mid = lo = make_uint4(0, 0, 0, 0);
                        if (j < n) {
                            float f[8];
                            unpack8(*reinterpret_cast<const uint4 *>(crow + off), f);
#pragma unroll
                            for (int u = 0; u < 8; u += 2) mul2(f[u], f[u + 1], w, w);
                            split3(f[0], f[1], hi.x, mid.x, lo.x);
                            split3(f[2], f[3], hi.y, mid.y, lo.y);
                            split3(f[4], f[5], hi.z, mid.z, lo.z);
                            split3(f[6], f[7], hi.w, mid.w, lo.w);
                        } else {  // past the end: zero, whatever memory holds there
                            *reinterpret_cast<uint4 *>(crow + off) = hi;
                            for (int t = 0; t < na; ++t)
                                *reinterpret_cast<uint4 *>(sm + SM::B + (i2 * 2 + t) * kAtom + j * 128 + off) = hi;
                        }
                        *reinterpret_cast<uint4 *>(prow + off) = hi;
                        *reinterpret_cast<uint4 *>(prow + off + kAtom) = mid;
                        *reinterpret_cast<uint4 *>(prow + off + 2 * kAtom) = lo;
                    }
                    decn = tab[kDEC];
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&cready[half]);
                        if (half == 1) {
                            mbar_arrive(&freeC[i2]);
                            mbar_arrive(&tfree[i2]);
                            if (n < kQ) mbar_arrive(zready);
                        }
                    }
                }
                if (update && cc > 0) {  // X <- e^{G_n} X + SD of chunk cc - 1
                    ok = ok && wait(sfull, (cc - 1) & 1, err);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t col = tmem + TM::SD + lb + 32 * hf + 8 * b;
                        float hi[8], mid[8], lo[8];
                        tmem_ld8(col, hi);
                        tmem_ld8(col + kN, mid);
                        tmem_ld8(col + 2 * kN, lo);
                        tmem_wait_ld();
#pragma unroll
                        for (int u = 0; u < 8; u += 2) {
                            add2(mid[u], mid[u + 1], lo[u], lo[u + 1]);
                            add2(hi[u], hi[u + 1], mid[u], mid[u + 1]);
                            fma2(hi[u], hi[u + 1], dec, x[8 * b + u], x[8 * b + u + 1]);
                            x[8 * b + u] = hi[u];
                            x[8 * b + u + 1] = hi[u + 1];
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(sdfree);
                }
                if (update && cc < nch && MODE != kStateOnly) {
                    if (MODE == kOutDots) {
                        const int e = nch - cc;  // reverse: the chunk whose start this is
                        int at = -1;             // the run that starts there; at the block's end the next block's first
                        if (!REV) {
                            if (cc % kRun == 0) at = run_of(geo, p.runs, t0, slot) + cc / kRun;
                        } else if (cc > 0) {
                            if (e % kRun == 0) at = run_of(geo, p.runs, t0, slot) + e / kRun;
                        } else if (sl.w < nblk - 1) {
                            at = run_of(geo, p.runs, t0 + len, slot + 1);
                        }
                        if (at >= 0) {
                            const size_t u = ((size_t)at * geo.H + h) * p.ng + ng;
                            float4 *b4 = reinterpret_cast<float4 *>(p.bnd) + u * (8 * 256) + (tid - 256);
                            if (!REV) {
#pragma unroll
                                for (int v = 0; v < 8; ++v)
                                    b4[v * 256] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
                            } else {
                                float y = 0.f;
                                if (k < p.db)
#pragma unroll
                                    for (int v = 0; v < 8; ++v) {
                                        const float4 z = b4[v * 256];
                                        y = fmaf(x[4 * v], z.x, fmaf(x[4 * v + 1], z.y,
                                            fmaf(x[4 * v + 2], z.z, fmaf(x[4 * v + 3], z.w, y))));
                                    }
#pragma unroll
                                for (int o = 16; o; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
                                if (lane == 0) p.ydot[u * 8 + (warp - 8)] = y;
                            }
                        }
                    }
                    // X as the B operand of A X^T (row k, swizzled), once the last chunk's product is done
                    if (cc > 0) {
                        ok = ok && wait(ifull, (cc - 1) & 1, err);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                    }
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        const uint32_t off = SM::X + k * 128 + (((4 * hf + b) ^ (k & 7)) << 4);
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
                }
            }
            if (!ok) break;
            dec = decn;
        }
        if (ok && p.xout && k < p.db && (MODE == kStateOnly || last)) {
            float *dst = p.xout + (MODE == kStateOnly ? (size_t)slot * geo.H + h : (size_t)sl.z * geo.H + h) * nel;
            if (p.tr) {
#pragma unroll
                for (int u = 0; u < 8; ++u)
                    if (cx + 4 * u < p.dc)
                        *reinterpret_cast<float4 *>(dst + (size_t)k * p.dc + cx + 4 * u) =
                            make_float4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
            } else {
#pragma unroll
                for (int u = 0; u < 32; ++u)
                    if (cx + u < p.dc) dst[(size_t)(cx + u) * p.db + k] = x[u];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) tmem_dealloc(tmem, TM::COLS);
}

// ------------------------------------------------------------ pairs inside a chunk, for dg
// M = (Q K^T) . (dO V^T) . Gamma below the diagonal: row sums (the pairs' part of
// q_l . dq_l) and column sums (of k_m . dk_m), fp32.  Both factors are products
// of inputs, so no operand is rounded.  The column sums are the row sums of the
// transposed products, which the tensor cores form as well: 32 more MMAs cost
// less than summing over lanes.  Reads q, k, v, dout once.  B4 T4096 H16 d128, alone: 69 us
// (its bytes 41 us), with 8 warps for the sums 125.
struct PairArgs {
    const float *g;
    float *rsum, *csum;  // [2, rows, H]
    int dk, dv, split;
};
struct PairSmem {
    static constexpr uint32_t QK = 0, VO = 4 * kAtom, TAB = 8 * kAtom;
    static constexpr uint32_t BARS = TAB + 2 * kPairTab * 4, TOTAL = BARS + 8 * 8 + 16;
};

__device__ __forceinline__ void pairs(unsigned int bid, const CUtensorMap &tm_q, const CUtensorMap &tm_k,
                                      const CUtensorMap &tm_v, const CUtensorMap &tm_o, const PairArgs &p,
                                      const Geo &geo, const Plan &plan, unsigned int *err) {
    // chunks first, first + split, ... of a (slot, head)
    const int first = bid % p.split;
    bid /= p.split;
    extern __shared__ __align__(1024) uint8_t sm[];
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + PairSmem::BARS);
    uint64_t *fullQ = bars, *fullV = bars + 1, *mdone = bars + 2, *tfull = bars + 3, *tfree = bars + 4;
    uint64_t *efree = bars + 5, *qdone = bars + 6;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 8);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slot = bid / geo.H, h = bid - slot * geo.H;
    const int4 sl = slot_of(geo, plan, slot);
    const int t0 = sl.x, len = sl.y, nch = (len + kQ - 1) / kQ, hk = h / (geo.H / geo.Hk);
    if (len <= 0 || first >= nch) return;
    if (kChecked && !(chk_span(t0, len, geo.rows, err) && chk_span(slot, 1, geo.n_slots, err) &&
                      chk_true((smem_u32(sm) & 1023u) == 0, err)))
        return;
    if (tid == 0) {
        mbar_init(fullQ, 1);
        mbar_init(fullV, 1);
        mbar_init(qdone, 1);
        mbar_init(mdone, 1);
        mbar_init(tfull, 2);
        mbar_init(tfree, 16);
        mbar_init(efree, 16);
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
            for (int cc = first; cc < nch; cc += p.split, ++it) {
                const int y = t0 + cc * kQ;
                if (it) ok = wait(qdone, (it - 1) & 1, err);
                if (!ok) break;
                mbar_arrive_expect_tx(fullQ, 2 * nk * kAtom);
                for (int i = 0; i < nk; ++i) {
                    tma_load_3d(sm + PairSmem::QK + i * kAtom, &tm_q, fullQ, 64 * i, hk, y);
                    tma_load_3d(sm + PairSmem::QK + (2 + i) * kAtom, &tm_k, fullQ, 64 * i, hk, y);
                }
                if (it) ok = wait(mdone, (it - 1) & 1, err);
                if (!ok) break;
                mbar_arrive_expect_tx(fullV, 2 * nv * kAtom);
                for (int i = 0; i < nv; ++i) {
                    tma_load_3d(sm + PairSmem::VO + i * kAtom, &tm_o, fullV, 64 * i, h, y);
                    tma_load_3d(sm + PairSmem::VO + (2 + i) * kAtom, &tm_v, fullV, 64 * i, h, y);
                }
            }
            if (it) {  // the last loads have landed and been read
                wait(qdone, (it - 1) & 1, err);
                wait(mdone, (it - 1) & 1, err);
            }
        }
    } else if (warp == 1) {
        const uint32_t el = elect_lane(), id = idesc_bf16(128, 128, 0, 0);
        const uint64_t dq = sdesc_sw128(smem_u32(sm + PairSmem::QK), 16, 1024);
        const uint64_t dv = sdesc_sw128(smem_u32(sm + PairSmem::VO), 16, 1024);
        int it = 0;
        // columns: Q K^T 0, K Q^T 128, dO V^T 256, V dO^T 384
        for (int cc = first; cc < nch && ok; cc += p.split, ++it) {
            if (it) ok = wait(efree, (it - 1) & 1, err);
#pragma unroll 1
            for (int m = 0; m < 2 && ok; ++m) {
                ok = ok && wait(m ? fullV : fullQ, it & 1, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                const int ks = (m ? p.dv : p.dk) / 16;
                const uint64_t d = m ? dv : dq;
#pragma unroll 2
                for (int kk = 0; kk < ks; ++kk) {
                    const uint64_t x = sdesc_add(d, (kk >> 2) * kAtom + (kk & 3) * 32), y = sdesc_add(x, 2 * kAtom);
                    mma_ss(el, tmem + 256 * m, x, y, id, kk > 0);
                    mma_ss(el, tmem + 256 * m + 128, y, x, id, kk > 0);
                }
                commit(el, m ? mdone : qdone);
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
        load(first);
        for (int cc = first; cc < nch; cc += p.split, ++it) {
            if (it) ok = wait(tfree, (it - 1) & 1, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            float *tab = reinterpret_cast<float *>(sm + PairSmem::TAB) + (warp - 2) * kPairTab;
            if (warp == 2)
                decay_tables<false, true>(tab, gv, lane);
            else
                decay_tables<true, true>(tab, gv, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(tfull);
            if (cc + p.split < nch) load(cc + p.split);
        }
    } else {
        // rows (warps 4-11) or columns (12-19); two warps share a row's columns, 16 of each block each
        const bool rev = warp >= 12;
        const int rb = warp & 3, hf = ((warp - 4) >> 2) & 1, i = rb * 32 + lane;
        const uint32_t lb = (uint32_t)(rb * 32) << 16, col = rev ? 128 : 0;
        const float *tab = reinterpret_cast<const float *>(sm + PairSmem::TAB) + (rev ? kPairTab : 0);
        int it = 0;
        for (int cc = first; cc < nch; cc += p.split, ++it) {
            const int n = min(kQ, len - cc * kQ);
            ok = ok && wait(tfull, it & 1, err);
            ok = ok && wait(qdone, it & 1, err);
            ok = ok && wait(mdone, it & 1, err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            const float li = tab[kLC + i], ll = tab[kLL + i];
            const float rf = rev ? row_factor<true>(li) : row_factor<false>(li);
            float s = 0.f;
#pragma unroll 1
            for (int b = rev ? rb : 0; b <= (rev ? 3 : rb); ++b) {
                const int c = 32 * b + 16 * hf;
                float x[16], y[16], f[16];
                tmem_ld16(tmem + col + lb + c, x);
                tmem_ld16(tmem + 256 + col + lb + c, y);
#pragma unroll
                for (int u = 0; u < 16; u += 4) {
                    const float4 l = *reinterpret_cast<const float4 *>(tab + (b == rb ? kLC : kCF) + c + u);
                    f[u] = l.x; f[u + 1] = l.y; f[u + 2] = l.z; f[u + 3] = l.w;
                }
                tmem_wait_ld();
                float r0 = 0.f, r1 = 0.f;
#pragma unroll
                for (int u = 0; u < 16; u += 2) mul2(x[u], x[u + 1], y[u], y[u + 1]);
                if (b == rb) {
#pragma unroll
                    for (int u = 0; u < 16; u += 4) {
                        const float4 l = *reinterpret_cast<const float4 *>(tab + kLL + c + u);
                        const float d[4] = {l.x - ll, l.y - ll, l.z - ll, l.w - ll};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const float e = (f[u + w] - li) + d[w];
                            f[u + w] = ex2(rev ? e : -e);
                        }
                    }
                }
                if (b == rb || c + 16 > n) {  // selects: what lies outside cannot matter
#pragma unroll
                    for (int u = 0; u < 16; ++u) {
                        const int at = u + 16 * hf;
                        const bool in = c + u < n && (b != rb || (rev ? at > lane : at < lane));
                        x[u] = in ? x[u] * f[u] : 0.f;
                    }
#pragma unroll
                    for (int u = 0; u < 16; u += 2) add2(r0, r1, x[u], x[u + 1]);
                } else {
#pragma unroll
                    for (int u = 0; u < 16; u += 2) {
                        mul2(x[u], x[u + 1], f[u], f[u + 1]);
                        add2(r0, r1, x[u], x[u + 1]);
                    }
                }
                const float r = r0 + r1;
                const int hiB = rev ? b : rb, loB = rev ? rb : b;
                s = b == rb ? s + r : fmaf(r, rf * tab[kBB + hiB * (hiB - 1) / 2 + loB], s);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(efree);
                mbar_arrive(tfree);
            }
            if (i < n)
                (rev ? p.csum : p.rsum)[(size_t)hf * geo.rows * geo.H + ((size_t)t0 + cc * kQ + i) * geo.H + h] = s;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------ launches
// Walks of one kind.
template <bool REV, int MODE>
__global__ void __launch_bounds__(kTcThreads, 1)
chain_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
             const __grid_constant__ CUtensorMap tm_c, TcArgs p, Geo geo, Plan plan, unsigned int *err) {
    stream_order();
    walk<REV, MODE>(blockIdx.x, tm_a, tm_b, tm_c, p, geo, plan, err);
}
struct Maps {
    CUtensorMap q, k, v, o;
};
// Two kinds of work in one grid, so that the second's CTAs run on the SMs that the
// first leaves: the blocks' states of both directions; dq and the pairs; dk and dv.
// (Gradients of T 128, H 16, d 64: 37 us in a launch each, 24 us so; B 4, T 4096, d 128:
// 413 us for the walks and pairs apart, 409 us together.)
__global__ void __launch_bounds__(kTcThreads, 1)
states_kernel(const __grid_constant__ Maps m, TcArgs p, TcArgs r, unsigned int n, Geo geo, Plan plan,
              unsigned int *err) {
    stream_order();
    if (blockIdx.x < n)
        walk<false, kStateOnly>(blockIdx.x, m.k, m.k, m.v, p, geo, plan, err);
    else
        walk<true, kStateOnly>(blockIdx.x - n, m.q, m.q, m.o, r, geo, plan, err);
}
__global__ void __launch_bounds__(kTcThreads, 1)
dq_pairs_kernel(const __grid_constant__ Maps m, TcArgs p, PairArgs r, unsigned int n, Geo geo, Plan plan,
                unsigned int *err) {
    stream_order();
    if (blockIdx.x < n)
        walk<false, kOutDots>(blockIdx.x, m.o, m.v, m.k, p, geo, plan, err);
    else
        pairs(blockIdx.x - n, m.q, m.k, m.v, m.o, r, geo, plan, err);
}
__global__ void __launch_bounds__(kTcThreads, 1)
dk_dv_kernel(const __grid_constant__ Maps m, TcArgs p, TcArgs r, unsigned int n, Geo geo, Plan plan,
             unsigned int *err) {
    stream_order();
    if (blockIdx.x < n)
        walk<true, kOutDots>(blockIdx.x, m.v, m.o, m.q, p, geo, plan, err);
    else
        walk<true, kOut>(blockIdx.x - n, m.k, m.q, m.o, r, geo, plan, err);
}

// ------------------------------------------------------------ gradient of the decays
// A CTA takes a run of kRun chunks of a (block, head), in 64 bits:
//     dg_t = sum_{l >= t in chunk} (R_l - C_l) + sum over the run's later chunks (Ri - Ci) + <S, dS>,
// R = Ri + Rp, C = Ci + Cp: the state's part (dots of the chains) and the part of
// the chunk's own pairs, whose rows and columns sum to the same and so drop out
// of the carry; S, dS the state at the run's end and its gradient, whose product
// the chains form at every kRun-th chunk.  Carried on from the end of the sequence
// instead, the sum's error grew with the length (T 4096: 1.8e-6 to 6e-6 of dg).
struct DgArgs {
    const float *ri, *ci, *rp, *cp, *ydot;
    int nri, nci, ny;           // planes of ri, ci; products of a boundary
    const float *fin, *dfin;    // S, dS at the sequences' ends, or dfin NULL (zero)
    float *dg, *part;
    int nel;
    Runs runs;
};
__device__ __forceinline__ double warp_sum(double x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

__global__ void __launch_bounds__(kRunLen)
dg_runs_kernel(DgArgs p, Geo geo, Plan plan) {
    stream_order();
    constexpr int NW = kRunLen / 32;
    __shared__ double tot[NW], inter[NW], red[NW];
    const int no = blockIdx.x / geo.H, h = blockIdx.x - no * geo.H;  // number of the run
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = tid / kQ;
    const int2 at_run = geo.varlen ? p.runs.of[no] : make_int2(no / p.runs.block, no % p.runs.block);
    const int slot = at_run.x;
    const int4 sl = slot < 0 ? make_int4(0, -1, 0, 0) : slot_of(geo, plan, slot);
    const int first = at_run.y * kRunLen, len = sl.y - first;  // tokens from the run's start
    if (len <= 0) {
        if (p.part && tid == 0) p.part[(size_t)no * geo.H + h] = 0.f;
        return;
    }
    const int nblk = geo.varlen ? plan.blk_start[sl.z + 1] - plan.blk_start[sl.z] : geo.nb;
    const bool more = len > kRunLen;  // the block goes on after the run
    double f = 0.0;
    if (more || sl.w < nblk - 1) {
        const size_t u = (size_t)(more ? no + 1 : run_of(geo, p.runs, sl.x + sl.y, slot + 1)) * geo.H + h;
        if (tid < p.ny) f = p.ydot[u * p.ny + tid];
    } else if (p.dfin) {
        const size_t o = ((size_t)sl.z * geo.H + h) * p.nel;
        float acc = 0.f;
        for (int i = tid; i < p.nel / 4; i += kRunLen) {
            const float4 a = reinterpret_cast<const float4 *>(p.fin + o)[i];
            const float4 b = reinterpret_cast<const float4 *>(p.dfin + o)[i];
            acc = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, acc))));
        }
        f = acc;
    }
    double x = 0.0, y = 0.0;  // everything; the state's part
    const size_t at = ((size_t)sl.x + first + tid) * geo.H + h, pl = (size_t)geo.rows * geo.H;
    if (tid < len) {
        for (int u = 0; u < p.nri; ++u) y += p.ri[u * pl + at];
        for (int u = 0; u < p.nci; ++u) y -= p.ci[u * pl + at];
        x = y + (((double)p.rp[at] + p.rp[pl + at]) - ((double)p.cp[at] + p.cp[pl + at]));
    }
    f = warp_sum(f);
    const double ys = warp_sum(y);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {  // inclusive sum from the warp's end
        const double z = __shfl_down_sync(0xffffffffu, x, o);
        if (lane + o < 32) x += z;
    }
    if (lane == 0) {
        tot[warp] = x;
        inter[warp] = ys;
        red[warp] = f;
    }
    __syncthreads();
    // the boundary, the run's later chunks, and this chunk's later warps
    constexpr int WC = kQ / 32;
    double add = 0.0;
    if (lane < NW) {
        add = red[lane];
        if (lane >= WC * (grp + 1)) add += inter[lane];
        if (lane > warp && lane < WC * (grp + 1)) add += tot[lane];
    }
    x += warp_sum(add);
    if (!p.part) {
        if (tid < len) p.dg[at] = (float)x;
        return;
    }
    __syncthreads();
    x = warp_sum(tid < len ? x : 0.0);
    if (lane == 0) red[warp] = x;
    __syncthreads();
    if (warp == 0) {
        x = warp_sum(lane < NW ? red[lane] : 0.0);
        if (lane == 0) p.part[(size_t)no * geo.H + h] = (float)x;
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
// walks fill the GPU, else pieces of it.  Pieces cost a pass for their states and
// the carry, so equal sequences are cut where the estimate below says that it pays:
// one walk to an SM, a chunk of one 2.6 us and 5 us to start (three walks, 10 us and
// 15 us for the gradient), without outputs 1.9 us and 4 us (measured; T 8192, H 4,
// d 128 forward: 164 us in one piece, 35 us in 16; B 4, T 4096, H 16: 94 us in one,
// 146 us in two).  The constants are those of d 128; at d 64, where a chunk takes less,
// the pieces that they choose took (best of 1, 2, 4, 8, 16 pieces in brackets): forward
// T 8192, H 4 32 us (35), B 4, T 4096, H 16 87 us (87); gradients 78 us (65), 282 us
// (253), B 2, T 1500, H 8 70 us (56).  Of packed sequences the host does not know the
// lengths: those longer than one and a half times an SM's share of all tokens are cut.
// d 128, in us, at three quarters of a share, at one and a half, at three, and uncut: one
// sequence of 8,192 tokens, H 4, forward 59, 48, 67, 169, gradients 134, 127, 133, 464;
// 16 sequences of 65,536, H 16, forward 378, 377, 376, 366; gradients of 9 of 8,191,
// H 16 275, 270, 274, 260.  d 64: 37, 37, 46, 171; 83, 91, 86, 453; 285, 211, 211, 204;
// 193, 175, 168, 166.
int block_len(int n_seq, bool varlen, bool bwd, int T, int H, int ng, size_t nel) {
    const double sms = 148.0;
    const int ch = (T + kQ - 1) / kQ;
    if (varlen) {
        double L = 1.5 * T * H * ng / sms;
        if (L < 256) L = 256;
        if (L > T) L = T;
        return ((int)L + kQ - 1) / kQ * kQ;
    }
    int best = ch;
    double least = 1e30;
    for (int nb = 1; nb <= ch && nb <= 64; ++nb) {
        const int c = (ch + nb - 1) / nb;
        auto waves = [&](double units) { return (double)(long)((units + sms - 1) / sms); };
        const double walks = (double)n_seq * H * ng;
        double t = waves(walks * nb) * (bwd ? 10.0 * c + 15 : 2.6 * c + 5);
        if (nb > 1)
            t += (bwd ? 2 : 1) * (waves(walks * (nb - 1)) * (1.9 * c + 4) + 2 + 0.25 * nb +
                                  (double)n_seq * nb * H * nel * 8 / 4e6);
        if (t < least * 0.97) {
            least = t;
            best = c;
        }
    }
    return best * kQ;
}

struct TcWs {
    size_t slot, blk_start, run, gtot, gtot_rev, X, Y, fin, ri, ci, rp, cp, bnd, ydot, dq32, dk32, part, total;
    int L, nb, n_slots, multi, run_blk, n_runs;
};
TcWs tc_ws(const LinCall &c, bool bwd) {
    TcWs w{};
    const bool varlen = c.cu != nullptr;
    const int n_seq = varlen ? c.n_seq : c.B;
    const size_t nel = (size_t)c.dk_ * c.dv_, rows = (size_t)c.B * c.T;
    const int gk = groups(c.dk_), gv = groups(c.dv_);
    w.L = block_len(n_seq, varlen, bwd, c.T, c.H, bwd && gk > gv ? gk : gv, nel);
    if (w.L < kQ) w.L = kQ;
    w.nb = (c.T + w.L - 1) / w.L;
    w.n_slots = varlen ? c.T / w.L + n_seq : c.B * w.nb;
    w.multi = w.nb > 1;
    w.run_blk = (w.L + kRunLen - 1) / kRunLen;
    w.n_runs = !bwd ? 0 : varlen ? c.T / kRunLen + w.n_slots : w.n_slots * w.run_blk;  // run_of
    const size_t sh = (size_t)w.n_slots * c.H;
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o += up256(bytes);
        return at;
    };
    w.slot = take(varlen ? sizeof(int4) * w.n_slots : 0);
    w.blk_start = take(varlen ? sizeof(int) * ((size_t)3 * n_seq + 1) : 0);
    w.run = take(varlen ? sizeof(int2) * w.n_runs : 0);
    w.gtot = take(w.multi ? sh * 4 : 0);
    w.gtot_rev = take(bwd && w.multi ? sh * 4 : 0);
    w.X = take(w.multi ? sh * nel * 4 : 0);
    if (bwd) {
        w.Y = take(w.multi ? sh * nel * 4 : 0);
        w.fin = take((size_t)n_seq * c.H * nel * 4);
        w.ri = take(rows * c.H * 2 * gk * 4);
        w.ci = take(rows * c.H * 2 * gk * 4);
        w.rp = take(rows * c.H * 2 * 4);
        w.cp = take(rows * c.H * 2 * 4);
        w.dq32 = take(c.Hk < c.H ? rows * c.H * c.dk_ * 4 : 0);
        w.dk32 = take(c.Hk < c.H ? rows * c.H * c.dk_ * 4 : 0);
        const size_t runs = (size_t)w.n_runs * c.H;
        w.bnd = take(runs * gk * kN * 128 * 4);
        w.ydot = take(runs * gk * 8 * 4);
        w.part = take(runs * 4);
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

bool make_maps(Maps *m, const LinCall &c) {
    const size_t rows = (size_t)c.B * c.T;
    return tile_map(&m->q, c.q, c.dk_, c.Hk, rows) && tile_map(&m->k, c.k, c.dk_, c.Hk, rows) &&
           tile_map(&m->v, c.v, c.dv_, c.H, rows) && (!c.dout || tile_map(&m->o, c.dout, c.dv_, c.H, rows));
}

// the parts of a walk's arguments that follow from the others; its CTAs
unsigned int prepare(const LinCall &c, const Geo &geo, TcArgs *p) {
    p->g = c.g;
    p->ng = groups(p->dc);
    p->wide = ((uintptr_t)p->out & 31u) == 0;
    return (unsigned)(geo.n_slots * geo.H * p->ng);
}
template <typename K>
cudaError_t allow(gdr_host::SmemLimit *limit, K kernel) {
    constexpr int most = TcSmem<kOut>::TOTAL > TcSmem<kOutDots>::TOTAL ? TcSmem<kOut>::TOTAL : TcSmem<kOutDots>::TOTAL;
    static_assert(PairSmem::TOTAL <= most && TcSmem<kStateOnly>::TOTAL <= most, "shared memory");
    return limit->set((const void *)kernel, most);
}

template <bool REV, int MODE>
cudaError_t launch_chain(const LinCall &c, const Geo &geo, const Plan &plan, const CUtensorMap &a,
                         const CUtensorMap &b, const CUtensorMap &cc, TcArgs p, int id) {
    static gdr_host::SmemLimit limit;
    const cudaError_t e = allow(&limit, chain_kernel<REV, MODE>);
    if (e != cudaSuccess) return e;
    const unsigned int n = prepare(c, geo, &p);
    gdr_host::ProfToken tk = gdr_host::prof_begin(id, c.st);
    const cudaError_t le = gdr_host::lin_launch(chain_kernel<REV, MODE>, dim3(n), kTcThreads,
                                                TcSmem<MODE>::TOTAL, c.st, a, b, cc, p, geo, plan, c.err);
    gdr_host::prof_end(tk, c.st);
    return le;
}

}  // namespace

namespace gdr_host {

size_t lin_tc_ws_bytes(const LinCall &c, bool bwd) { return tc_ws(c, bwd).total; }

cudaError_t lin_fwd_tc(const LinCall &c) {
    const TcWs w = tc_ws(c, false);
    const LinWs l = common_ws(w);
    Geo geo = lin_geo(c, l);
    geo.keep_empty = geo.skip_single = 1;
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
        const LinScan f{X, s.gtot, c.S0, nullptr};
        if ((e = lin_scan(c, geo, l, &f, nullptr)) != cudaSuccess) return e;
    }
    p.xin = c.S0;
    p.xblk = X;
    p.xout = c.S_final;
    p.out = c.out;
    return launch_chain<false, kOut>(c, geo, plan, m.q, m.k, m.v, p, GDR_K_LIN_OUT);
}

cudaError_t lin_bwd_tc(const LinCall &c) {
    const TcWs w = tc_ws(c, true);
    const LinWs l = common_ws(w);
    Geo geo = lin_geo(c, l);
    geo.keep_empty = geo.skip_single = 1;
    const Plan plan = {(const int4 *)(c.ws + w.slot), (const int *)(c.ws + w.blk_start)};
    Maps m;
    if (!make_maps(&m, c)) return cudaErrorUnknown;
    cudaError_t e;
    const Runs runs{w.run_blk, w.n_runs, (int2 *)(c.ws + w.run)};
    if ((e = lin_plan(c, geo, l, runs)) != cudaSuccess) return e;
    const bool shared = c.Hk < c.H;
    const __nv_bfloat16 *q = (const __nv_bfloat16 *)c.q, *k = (const __nv_bfloat16 *)c.k;
    float *X = (float *)(c.ws + w.X), *Y = (float *)(c.ws + w.Y), *fin = (float *)(c.ws + w.fin);
    float *ri = (float *)(c.ws + w.ri), *ci = (float *)(c.ws + w.ci);
    float *rp = (float *)(c.ws + w.rp), *cp = (float *)(c.ws + w.cp);
    float *part = c.gate == GDR_GATE_HEAD ? (float *)(c.ws + w.part) : nullptr;
    static SmemLimit lim_s, lim_q, lim_k;
    ProfToken tk;
    if (w.multi) {
        TcArgs s{};
        s.ha = s.hb = c.Hk; s.hc = c.H; s.he = c.H;
        s.db = c.dk_; s.dc = c.dv_;
        TcArgs t = s;
        s.xout = X;
        t.xout = Y;
        s.gtot = (float *)(c.ws + w.gtot);
        t.gtot = (float *)(c.ws + w.gtot_rev);
        if ((e = allow(&lim_s, states_kernel)) != cudaSuccess) return e;
        const unsigned int n = prepare(c, geo, &s);
        prepare(c, geo, &t);
        tk = prof_begin(GDR_K_LIN_STATE, c.st);
        e = lin_launch(states_kernel, dim3(2 * n), kTcThreads, TcSmem<kStateOnly>::TOTAL, c.st, m, s, t, n, geo,
                       plan, c.err);
        prof_end(tk, c.st);
        if (e != cudaSuccess) return e;
        const LinScan f{X, s.gtot, c.S0, nullptr}, b{Y, t.gtot, c.dS_final, nullptr};
        if ((e = lin_scan(c, geo, l, &f, &b)) != cudaSuccess) return e;
    }
    // dq: (a, b, c) = (dout, v, k), the state transposed; beside it the pairs inside chunks
    TcArgs p{};
    p.ha = p.hb = c.H; p.hc = p.he = c.Hk;
    p.db = c.dv_; p.dc = c.dk_; p.tr = 1;
    p.out32 = shared;
    p.xin = c.S0;
    p.xblk = X;
    p.xout = c.dS_final ? fin : nullptr;
    p.out = shared ? (void *)(c.ws + w.dq32) : c.dq;
    p.e = q;
    p.dots = ri;
    p.bnd = (float *)(c.ws + w.bnd);
    p.ydot = (float *)(c.ws + w.ydot);
    p.runs = runs;
    // pairs: CTAs for a (slot, head), as many as end soonest on 148 SMs, a start costing about as
    // much as one and a half chunks (gradients of B4 T4096 H16 d128: one 463 us, two 410, four 414)
    const long units = (long)geo.n_slots * geo.H, most = w.L / kQ;
    long split = 1;
    double least = 1e30;
    for (long n = 1; n <= most && n <= 64; ++n) {
        const double t = (double)((units * n + 147) / 148) * ((double)((most + n - 1) / n) + 1.5);
        if (t < least) {
            least = t;
            split = n;
        }
    }
    const PairArgs pa{c.g, rp, cp, c.dk_, c.dv_, (int)split};
    if ((e = allow(&lim_q, dq_pairs_kernel)) != cudaSuccess) return e;
    unsigned int n = prepare(c, geo, &p);
    tk = prof_begin(GDR_K_LIN_GRAD, c.st);
    e = lin_launch(dq_pairs_kernel, dim3(n + (unsigned)(units * split)), kTcThreads, TcSmem<kOutDots>::TOTAL,
                   c.st, m, p, pa, n, geo, plan, c.err);
    prof_end(tk, c.st);
    if (e != cudaSuccess) return e;
    // dk: (v, dout, q), backward in time
    p.xin = c.dS_final;
    p.xblk = Y;
    p.xout = nullptr;
    p.out = shared ? (void *)(c.ws + w.dk32) : c.dk;
    p.e = k;
    p.dots = ci;
    // dv: (k, q, dout), backward in time; beside dk, unless dS0 is to be written over dS_final
    TcArgs r{};
    r.ha = r.hb = c.Hk; r.hc = r.he = c.H;
    r.db = c.dk_; r.dc = c.dv_;
    r.xin = c.dS_final;
    r.xblk = Y;
    r.xout = c.dS0;
    r.out = c.dv;
    const bool over = c.dS0 && c.dS0 == c.dS_final;
    if ((e = allow(&lim_k, dk_dv_kernel)) != cudaSuccess) return e;
    n = prepare(c, geo, &p);
    const unsigned int nv = prepare(c, geo, &r);
    static_assert(TcSmem<kOutDots>::TOTAL >= TcSmem<kOut>::TOTAL, "shared memory");
    tk = prof_begin(GDR_K_LIN_GRAD, c.st);
    e = lin_launch(dk_dv_kernel, dim3(n + (over ? 0 : nv)), kTcThreads, TcSmem<kOutDots>::TOTAL, c.st, m, p, r,
                   n, geo, plan, c.err);
    prof_end(tk, c.st);
    if (e != cudaSuccess) return e;
    if (shared) {
        if ((e = lin_group_sum(c, geo, l, (const float *)(c.ws + w.dq32), c.dq, c.dk_)) != cudaSuccess) return e;
        if ((e = lin_group_sum(c, geo, l, (const float *)(c.ws + w.dk32), c.dk, c.dk_)) != cudaSuccess) return e;
    }
    DgArgs d{ri, ci, rp, cp, (const float *)(c.ws + w.ydot), 2 * groups(c.dk_), 2 * groups(c.dk_),
             8 * groups(c.dk_), fin, c.dS_final, c.dg, part, c.dk_ * c.dv_, runs};
    tk = prof_begin(GDR_K_LIN_GRAD, c.st);
    e = lin_launch(dg_runs_kernel, dim3((unsigned)runs.count * geo.H), kRunLen, 0, c.st, d, geo, plan);
    prof_end(tk, c.st);
    if (e != cudaSuccess) return e;
    if (part) {
        Geo by_run = geo;  // one sum per run and head
        by_run.n_slots = runs.count;
        if ((e = lin_dg_heads(c, by_run, part)) != cudaSuccess) return e;
    }
    return over ? launch_chain<true, kOut>(c, geo, plan, m.k, m.q, m.o, r, GDR_K_LIN_GRAD) : cudaSuccess;
}

}  // namespace gdr_host
