// Shared pieces of the linear attention kernels (linear.cu, linear_simt.cu,
// linear_tc.cu): the cut of the sequences into blocks, and the decays.
//
// A sequence is cut into blocks of L tokens (the last may be shorter).  A slot
// is one (sequence, block) pair; the states that enter the blocks are held per
// (slot, head) as fp32 [d_v, d_k], like S itself.
#pragma once

#include <atomic>

#include "common.cuh"

namespace gdr {
namespace lin {

struct Geo {
    int T, H, Hk, n_seq, varlen, rows;  // rows: tokens of the whole batch
    int L, nb, n_slots;                 // nb: blocks per sequence (equal lengths)
    int gate_head;                      // g is [H]: one log-decay for all tokens
    int keep_empty;                     // an empty packed sequence has one block of no tokens
    int skip_single;                    // a sequence of one block takes its state from the caller's
};

// {first row, tokens, sequence, block}; a slot that no block fills has -1 tokens.
struct Plan {
    const int4 *slot;      // packed batches only
    const int *blk_start;  // [n_seq + 1]: first slot of each sequence
};

// Tokens of a run, the piece of a block over which the tensor-core path sums the
// gradient of the decays before it starts again.
constexpr int kRunLen = 512;

struct Runs {
    int block, count;  // of a full block; of the call
    int2 *of;          // packed batches, [count]: {slot, run of the slot}, slot -1 where there is none
};

// Number of the first run of a slot whose first row is t0.  In a packed batch a
// slot of n tokens has ceil(n / kRunLen) runs; consecutive slots start n rows and
// one slot later, and floor((t0 + n) / kRunLen) + 1 >= floor(t0 / kRunLen) +
// ceil(n / kRunLen), so the slots' runs are apart and there are at most
// floor(rows / kRunLen) + n_slots, however the tokens are shared out.  (A full
// block's runs for every slot took 12 GB for 256 sequences of 65,536 tokens, 16
// heads and d 128.)
__host__ __device__ __forceinline__ int run_of(const Geo &geo, const Runs &runs, int t0, int slot) {
    return geo.varlen ? t0 / kRunLen + slot : slot * runs.block;
}

__device__ __forceinline__ int4 slot_of(const Geo &geo, const Plan &plan, int slot) {
    if (geo.varlen) return plan.slot[slot];
    const int s = slot / geo.nb, b = slot - s * geo.nb;
    return make_int4(s * geo.T + b * geo.L, min(geo.L, geo.T - b * geo.L), s, b);
}

// First statement of every kernel of these calls but decode: the kernel is started
// (lin_launch) when the blocks of the one before it in the stream have ended, and waits
// here until that one's results are visible.  What is saved is the part of a launch
// before this point, 2 to 5 us at each kernel: measured in turn on one GPU, calls one after
// another on the same inputs, the gradients of 2 x 1,500 tokens with a decay for each head
// took 75 us in place of 89, the packed forward pass 357 in place of 368 (other GPUs and
// new inputs for each call: up to 12 % more on both sides).  To start the next kernel
// earlier, when this one's last blocks have begun (griddepcontrol.launch_dependents), takes
// more: waiting blocks hold the shared memory that this kernel's are still to use (gradients
// of a batch, in turn: 443 us, 430 with plain launches, 424 so).
// Pointers that reach a kernel's loads are not __restrict__ in its arguments, and no
// load is of the read-only kind: such a load may be moved up across the wait.
__device__ __forceinline__ void stream_order() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A decay of e^-104 is 0 in fp32 (the smallest subnormal is 2^-149 = e^-103.3),
// so clamping there changes no result and keeps sums of decays finite.
__device__ __forceinline__ float clamp_g(float g) { return g < -104.f ? -104.f : g; }

__device__ __forceinline__ float load_g(const Geo &geo, const float *g, long row, int h) {
    return clamp_g(geo.gate_head ? g[h] : g[row * geo.H + h]);
}

}  // namespace lin
}  // namespace gdr

namespace gdr_host {
// A kernel's dynamic shared memory limit, set once on each device (the call costs
// about as much as a launch).
class SmemLimit {
    std::atomic<unsigned long long> done_{0};

public:
    cudaError_t set(const void *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
        if (done_.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done_.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

// Launch of a kernel that begins with stream_order().
template <typename... P, typename... A>
cudaError_t lin_launch(void (*kernel)(P...), dim3 grid, unsigned int block, size_t smem, cudaStream_t st,
                       const A &...args) {
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    if (e != cudaSuccess) (void)cudaGetLastError();  // reported here, so not left for the caller
    return e;
}

// Arguments of one call, checked by the entry point.
struct LinCall {
    const void *q, *k, *v, *dout;
    const float *g, *S0, *dS_final;
    void *out, *dq, *dk, *dv;
    float *S_final, *dg, *dS0;
    const int32_t *cu;
    int B, T, H, Hk, dk_, dv_, n_seq;
    gdr_dtype dtype;
    gdr_gate gate;
    uint8_t *ws;
    unsigned int *err;
    cudaStream_t st;
};

// Byte offsets of the workspace (one layout for the forward and the backward call).
struct LinWs {
    size_t slot, blk_start, gtot, X, Y, fin, rdot, cdot, dq32, dk32, part, total;
    int n_slots, nb, L;
};
LinWs lin_ws(int B, int T, int H, int Hk, int dk, int dv, int n_seq, bool varlen, bool bwd, int L,
             int dot_cols);
gdr::lin::Geo lin_geo(const LinCall &c, const LinWs &w);
cudaError_t lin_plan(const LinCall &c, const gdr::lin::Geo &geo, const LinWs &w,
                     const gdr::lin::Runs &runs = {});
// States of the blocks carried over each sequence: X[slot] (the block's own
// contribution) becomes the state that enters the block, from `init` on; `fin` (may
// be NULL) receives the last state.  Forward in time (f), backward (r), or both in
// one launch.
struct LinScan {
    float *X;
    const float *gtot, *init;
    float *fin;
};
cudaError_t lin_scan(const LinCall &c, const gdr::lin::Geo &geo, const LinWs &w, const LinScan *f,
                     const LinScan *r);
cudaError_t lin_group_sum(const LinCall &c, const gdr::lin::Geo &geo, const LinWs &w,
                          const float *x, void *out, int d);
cudaError_t lin_dg_heads(const LinCall &c, const gdr::lin::Geo &geo, const float *part);

// CUDA-core path (linear_simt.cu)
constexpr int kLinSimtL = 256;
cudaError_t lin_fwd_simt(const LinCall &c);
cudaError_t lin_bwd_simt(const LinCall &c);
size_t lin_simt_ws_bytes(const LinCall &c, bool bwd);

// tensor-core path (linear_tc.cu)
cudaError_t lin_fwd_tc(const LinCall &c);
cudaError_t lin_bwd_tc(const LinCall &c);
size_t lin_tc_ws_bytes(const LinCall &c, bool bwd);
}  // namespace gdr_host
