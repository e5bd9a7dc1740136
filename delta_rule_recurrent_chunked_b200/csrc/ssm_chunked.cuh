// Chunked selective state space scan on sm_100a tensor cores (bf16 inputs).
//
// The tokens are cut into chunks of Q = 128. With l_t = delta_t A, g_i = l_1 + .. + l_i inside a
// chunk and S the state that enters it, the recurrence
//     S_t = exp(l_t) S_{t-1} + delta_t x_t B_t^T,   y_t = S_t C_t + D x_t
// is exactly
//     y_i = sum_{j<=i} (C_i . B_j) exp(g_i - g_j) delta_j x_j + exp(g_i) S C_i + D x_i
//     S'  = exp(g_Q) S + sum_j exp(g_Q - g_j) delta_j x_j B_j^T
// (every exponent is <= 0: no anchors and no range limits). One CTA runs one head's slice of 64
// value channels over its chunks, four products per chunk:
//     scores  C B^T             M=128 N=128 K=N     both from shared memory
//     inter   C S^T             M=128 N=64  K=N     S as bf16
//     intra   P x               M=128 N=64  K=128   P (bf16) in tensor memory, over its scores
//     state   B^T x1, x2, x3    M=128 N=64  K=128   x1 + x2 + x3 = exp(g_Q - g_j) delta_j x_j
// The state stays in the registers of one warpgroup in fp32 (a lane per row n of S^T).
//
// Roundings to bf16, each a choice: P and the copy of S that the outputs read (2^-8 of a
// product; the outputs are rounded to bf16 themselves). The state is carried on and returned in
// fp32, so the scaled x goes in three bf16 parts of 8 bits each (2^-24; two parts left 2.4e-6 in
// the state where its fp32 sums leave 2e-7). x, B and C are bf16 as they come.
//
// exp(g_i - g_j) for columns of an earlier 32-token block J of the chunk is taken as
// exp(g_i - g_end(J)) exp(g_end(J) - g_j), both <= 1: one exponential per row and block and one
// per token instead of one per element; only the diagonal 32 x 32 blocks take one per element.
//
// Roles (1024 threads): warps 0-7 weigh the scores (P), 8-15 scale x, 16-19 carry the state, 20-23
// write the outputs, warp 24 loads the tiles by TMA, warps 25-27 issue the MMAs of the state, the
// scores and the outputs, warps 28-31 prepare the per-token factors, up to four chunks ahead.
// Tiles are double-buffered, those of x apart from C and B, which are free as soon as the
// products have read them; scores run ahead. Every wait is bounded; a role whose wait runs out
// leaves its loop, and the loads and products that it started are waited for before the CTA ends.
//
// Three chains lead from chunk to chunk: state product -> registers -> S copy -> inter; the one set
// of output accumulators, since inter(c) waits until the output warps have drained both products of
// c - 1; and the S copy, which waits for the chunk's inter and intra products (SB_Y) though only
// inter reads it.
//
// Measured: 16 heads of P = N = 128, 8 x 4096 tokens (295 MB): 196 us; one sequence of 32768
// tokens, P = 64: 150 us in 9 segments. A chunk of 64 channels takes some 5,000 cycles, where its
// products take 1,500 on the tensor core and its shared memory traffic 2,700: bound by those chains
// and by the latency of the roles' instructions in them. With clocks in the waits (which slow a
// chunk to 6,800) the drain takes 3,000 cycles of a chunk; the outputs' MMA warp waits 2,250 for the
// S copy and 1,200 for the drain, 350 for the cleared tile of x and 180 for P; the state warps wait
// 2,100 for their product and 700 for SB_Y. The roles share the issue slots (52% busy) of four
// schedulers, rows r of P always those of the scheduler that owns their lanes of tensor memory; the
// weights of rows 96-127, with 4 of the 10 blocks, took 2,900 cycles a chunk. What was slower: weights
// of the diagonal blocks made before the scores come, on 8 warps (235 us) or on 12 with 4 left to
// scale x (242 us); the two warps of 32 rows at 64 columns each (193 us). 256 CTAs run in two waves on
// 148 SMs, 86% full.
#pragma once

#include <algorithm>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ssm_scan.cuh"

namespace drscan {

constexpr int SCK = 128;        // tokens per chunk
constexpr int SCV = 64;         // value channels per CTA
constexpr int SC_THREADS = 1024;
// Registers per thread: 64 at launch, then by role; the eight groups of four warps hold 2 x 56 (P)
// + 2 x 56 (scaled x) + 112 (state) + 80 (outputs) + 40 (loads and MMAs) + 48 (factors), not more
// than 8 x 64.
constexpr int SC_REG_P = 56, SC_REG_X = 56, SC_REG_STATE = 112, SC_REG_OUT = 80,
              SC_REG_ISSUE = 40, SC_REG_PAR = 48;
constexpr int SC_AHEAD = 2;     // chunks between a tile's prefetch into L2 and its load
constexpr int SC_NPAR = 4;      // chunks of per-token factors

// Shared memory (bytes). A tile row is 128 bytes (64 bf16) of a 128-byte-swizzled panel.
constexpr int SC_PANEL = SCK * 128;                      // 128 rows x 64 channels
constexpr int SC_C = 0;                                  // [stage] two panels
constexpr int SC_B = SC_C + 2 * SC_PANEL;                // two panels
constexpr int SC_X = SC_B + 2 * SC_PANEL;                // one panel
constexpr int SC_STAGE = SC_X + SC_PANEL;
constexpr int SC_NXS = 3;                                // slots of scaled x, 32 tokens each
constexpr int SC_XPART = 32 * 128;                       // .. of three parts
constexpr int SC_XS = 2 * SC_STAGE;
constexpr int SC_S = SC_XS + SC_NXS * 3 * SC_XPART;      // S^T rows n, 64 value channels
constexpr int SC_PAR = SC_S + SC_PANEL;                  // [SC_NPAR] SsmChunkPar
struct SsmChunkPar {
    float g2[SCK];     // (g_i - g before the token's block of 32) log2(e)
    float delta[SCK];
    float u[SCK];      // delta_j exp(g_end(J) - g_j), J the token's block of 32
    float w[SCK];      // delta_j exp(g_Q - g_j)
    float eg[SCK];     // exp(g_i)
    float between[16]; // [4 I + J] log2(e) times the steps of the blocks between J and I, J < I
    float gamma;       // exp(g_Q)
    float pad[3];
};
constexpr int SC_BAR = SC_PAR + SC_NPAR * (int)sizeof(SsmChunkPar);
// Barriers. One that is waited for by a role which may lag behind the next phase (its other
// waiters alone let that one complete) exists twice, for even and odd chunks: a wait by parity
// tells neighbouring phases apart, not a phase from the one after the next.
enum {
    SB_CB = 0,       // [2] tiles of C and B are there
    SB_CBFREE = 2,   // [2] .. have been read by their three products
    SB_X = 4,        // [2] the tile of x is there
    SB_XFREE = 6,    // [2] .. has been read
    SB_PAR = 8,      // [SC_NPAR] factors are there
    SB_PARFREE = 12, // [SC_NPAR]
    SB_SCORE = 16,   // [2] scores are in tensor memory
    SB_P = 18,       // [2] P is in tensor memory
    SB_CLEAR = 20,   // [2] the tile of x holds nothing behind the sequence
    SB_Y = 22,       // [2] inter and intra products are in tensor memory
    SB_DS = 24,      // the chunk's state product is in tensor memory
    SB_DSFREE = 25,  // .. has been read
    SB_ST = 26,      // the entering state's copy is in shared memory
    SB_YFREE = 27,   // inter and intra products have been read
    SB_XS = 28,      // [SC_NXS] scaled x of 32 tokens is in its slot
    SB_XSFREE = 31,  // [4] .. of the chunk's quarter has been read
    SB_DRAIN = 35,   // [3] all that an MMA warp issued is over
    SB_COUNT = 38
};
constexpr int SC_TOTAL = SC_BAR + 8 * SB_COUNT + 32;
// Tensor memory columns
constexpr uint32_t TC_SCORE = 0;   // [2] 128 columns; of each 16, P takes the first 8
constexpr uint32_t TC_INTRA = 256, TC_INTER = 320;
constexpr uint32_t TC_DS = 384;    // 64 columns of the first parts, 64 of the others

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// MMA and commit issued by one elected lane of a converged warp. With every operand the same in
// all lanes (and unrolled) the descriptors stay in uniform registers: an N = 128 product then
// issues every 64 cycles, the tensor core's rate; from a divergent lane, with descriptors formed
// in a loop, the same instruction measured about 190.
// D[tmem] (+)= A[smem] * B[smem]^T
__device__ __forceinline__ void mma_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T: A packs two bf16 of K in a 32-bit column.
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The product of K = kdim with A a tile along K (panels of 64, from shared address `a`) and B from
// descriptor `db`, which grows by `bstep` a K step and has `bpanel` from panel to panel.
__device__ __forceinline__ void mma_kmajor(uint32_t d_tmem, uint32_t a, uint64_t db,
                                           uint32_t bstep, uint32_t bpanel, int kdim,
                                           uint32_t idesc) {
    uint64_t da = smem_desc_sw128(a, 16, 1024);
    uint32_t acc = 0;
#pragma unroll 1
    for (int k = 0; k < kdim; k += 16) {
        mma_ss(d_tmem, da, db, idesc, acc);
        acc = 1;
        const bool turn = (k & 48) == 48;  // the panel's last step
        da += turn ? (SC_PANEL >> 4) - 6 : 2;
        db += turn ? bpanel - 3 * bstep : bstep;
    }
}

__device__ __forceinline__ void commit_elected(uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "elect.sync _|q, 0xffffffff;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
            bar)
        : "memory");
}

// The lower 32 bits of the timer in nanoseconds (they come round after 4.3 s).
__device__ __forceinline__ uint32_t timer_lo_ns() {
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}

// Whether the phase with the given parity is over. (mbar_test may suspend the thread for some
// microseconds until it is.)
__device__ __forceinline__ bool mbar_test_now(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cta.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

// Waits, as a whole warp, for the phase with the given parity: by a vote, since lanes that leave
// the polls at different times would run what follows one after another. Bounded by its polls: one
// that fails suspends the warp for 4 us (3.96 measured, from 10 to 300000 polls in a row), so that
// they last for DRSCAN_WAIT_LIMIT_NS. False (with the status latched) when they ran out: the caller
// leaves its loop, and whoever waits for it runs out too. (With a look at the clock in the loop, in
// whatever form, the scan of 8 x 16 heads and 4096 tokens took 183 to 223 us instead of 173.)
// TIMED, for tests: no suspension, and `limit` nanoseconds (0: one poll) instead.
template <bool TIMED>
__device__ __forceinline__ bool mbar_wait_warp(uint32_t bar, uint32_t parity, uint32_t limit) {
    if constexpr (TIMED) {
        const uint32_t t0 = timer_lo_ns();
#pragma unroll 1
        while (!__all_sync(0xffffffffu, mbar_test_now(bar, parity))) {
            if (__any_sync(0xffffffffu, timer_lo_ns() - t0 >= limit)) {
                raise_status(DR_ERR_TIMEOUT);
                return false;
            }
        }
    } else {
        int polls = (int)(DRSCAN_WAIT_LIMIT_NS / 4000);
#pragma unroll 1
        while (!__all_sync(0xffffffffu, mbar_test(bar, parity))) {
            if (--polls == 0) {
                raise_status(DR_ERR_TIMEOUT);
                return false;
            }
        }
    }
    return true;
}

// 8 consecutive columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float* r) {
    uint32_t* u = reinterpret_cast<uint32_t*>(r);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
          "=r"(u[7])
        : "r"(taddr));
}

// .. and stored.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* u) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "r"(u[0]), "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]),
                 "r"(u[7])
                 : "memory");
}

__device__ __forceinline__ void st_global_32(void* p, const uint32_t* u) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(u[0]), "r"(u[1]),
                 "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

// Bits of the pair of elements 0 and 1 of which those up to `top` count.
__device__ __forceinline__ uint32_t pair_mask(int top) {
    return top >= 1 ? 0xffffffffu : top == 0 ? 0xffffu : 0u;
}

template <int N>
__device__ __forceinline__ void regs_down() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// A box of a tensor map into L2 only.
__device__ __forceinline__ void tma_prefetch_4d(const void* map, int c0, int c1, int c2, int c3) {
    asm volatile("cp.async.bulk.prefetch.tensor.4d.L2.global.tile [%0, {%1, %2, %3, %4}];" ::"l"(map),
                 "r"(c0), "r"(c1), "r"(c2), "r"(c3)
                 : "memory");
}

struct SsmChunkArgs {
    SsmArgs s;
    // 1 where the tensor map's head / batch coordinate counts, 0 where the view repeats
    int xh, xb, bh, bb, ch, cb;
    int out32;  // the rows of out lie on 32-byte boundaries
    uint32_t wait_ns;  // limit of a wait of one role for another (TIMED)
};

// grid: (B * H * slices of SCV value channels, segments of this pass); block: SC_THREADS. TIMED:
// waits with a limit of the caller's, for tests of what happens when they run out.
template <int PASS, bool TIMED>
__global__ void __launch_bounds__(SC_THREADS, 1) ssm_chunked_kernel(
    const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmB,
    const __grid_constant__ CUtensorMap tmC, const __grid_constant__ SsmChunkArgs ca) {
    constexpr bool OUT = PASS == SSM_PASS_OUTPUTS;
    const SsmArgs& a = ca.s;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SC_BAR);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + SC_BAR + 8 * SB_COUNT + 8);
    float* sums = reinterpret_cast<float*>(sm + SC_BAR + 8 * SB_COUNT + 16);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto stage = [&](int s) { return sm + s * SC_STAGE; };
    auto par = [&](int s) {
        return reinterpret_cast<SsmChunkPar*>(sm + SC_PAR + s * (int)sizeof(SsmChunkPar));
    };
    // waits of chunk c
    auto wait2 = [&](int i, int c) {
        return mbar_wait_warp<TIMED>(bar(i + (c & 1)), (uint32_t)((c >> 1) & 1), ca.wait_ns);
    };
    auto wait1 = [&](int i, int c) {
        return mbar_wait_warp<TIMED>(bar(i), (uint32_t)(c & 1), ca.wait_ns);
    };
    auto wait_par = [&](int c) {
        return mbar_wait_warp<TIMED>(bar(SB_PAR + c % SC_NPAR), (uint32_t)((c / SC_NPAR) & 1),
                              ca.wait_ns);
    };
    // waits for async work that was started, whatever limit the others have
    auto drain = [&](int i, uint32_t parity) { mbar_wait_warp<false>(bar(i), parity, 0); };

    // (by a shuffle, so that the compiler knows the roles' branches to be uniform: without it the
    // two issuing warps' code is more than twice as long)
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int nsl = (a.P + SCV - 1) / SCV;
    const int v0 = (int)(blockIdx.x % nsl) * SCV;
    const long bh = blockIdx.x / nsl;
    const long b = bh / a.H;
    const int h = (int)(bh % a.H), g = h / (a.H / a.G);
    const int seg = (int)blockIdx.y;
    const int pv = min(SCV, a.P - v0);  // value channels of this slice
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int t0 = seg * a.seg_len;
    const int ntok = max(0, min(len - t0, min(a.seg_len, a.T - t0)));
    int nc = (ntok + SCK - 1) / SCK;
    auto valid = [&](int c) { return min(SCK, ntok - c * SCK); };

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(SB_CB + s), 1);
            mbar_init(bar(SB_CBFREE + s), OUT ? 3 : 1);  // the scores, the state's, the inter product
            mbar_init(bar(SB_X + s), 1);
            mbar_init(bar(SB_XFREE + s), OUT ? 5 : 8);  // the intra product and the output warps; the scaling warps
            mbar_init(bar(SB_SCORE + s), 1);
            mbar_init(bar(SB_P + s), 256);
            mbar_init(bar(SB_Y + s), 1);
            mbar_init(bar(SB_CLEAR + s), 8);
        }
        for (int s = 0; s < SC_NPAR; ++s) {
            mbar_init(bar(SB_PAR + s), 1);
            mbar_init(bar(SB_PARFREE + s), OUT ? 24 : 12);  // the warps that read factors
        }
        mbar_init(bar(SB_DS), 1);
        mbar_init(bar(SB_ST), 128);
        mbar_init(bar(SB_DSFREE), 128);
        for (int i = 0; i < SC_NXS; ++i) mbar_init(bar(SB_XS + i), 2);
        for (int i = 0; i < 4; ++i) mbar_init(bar(SB_XSFREE + i), 1);
        for (int i = 0; i < 3; ++i) mbar_init(bar(SB_DRAIN + i), 1);
        mbar_init(bar(SB_YFREE), 128);
        mbar_init_fence();
    }
    if (warp == 25) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are this CTA's, so they start at 0: as a constant, addresses of tensor
    // memory cost the issuing warps nothing
    constexpr uint32_t tmem = 0;
    if (*tmem_holder != tmem) {
        if (tid == 0) raise_status(DR_ERR_DEVICE_BOUNDS);
        nc = 0;
    }
    // a warp's 32 lanes of tensor memory
    const uint32_t trow = tmem + ((uint32_t)(warp & 3) << 21);
    auto release_par = [&](int c) {  // this warp has read the chunk's factors
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SB_PARFREE + c % SC_NPAR));
    };

    if (warp >= 28) {
        // ------------------------------------------------------------------ per-token factors
        // (warp 28 + k those of chunks k, k + 4, ..: one warp alone took 6,000 cycles a chunk,
        // twice what the products need)
        regs_down<SC_REG_PAR>();
        const float Ah = a.A[h] * 1.4426950408889634f;  // decays as powers of two
        float logsum = 0.f;
        static_assert(SC_NPAR == 4, "a slot of factors per warp");
        int c = warp - 28;
        for (; c < nc; c += SC_NPAR) {
            if (c >= SC_NPAR && !mbar_wait_warp<TIMED>(bar(SB_PARFREE + c % SC_NPAR),
                                                (uint32_t)((c / SC_NPAR - 1) & 1), ca.wait_ns))
                break;
            SsmChunkPar* pr = par(c % SC_NPAR);
#pragma unroll 1
            for (int t = lane; t < SCK; t += 32)  // a step of 0 behind the sequence keeps the state
                pr->delta[t] = c * SCK + t < ntok
                                   ? ssm_delta(a, h, ssm_dt(a, b, h, (long)t0 + c * SCK + t))
                                   : 0.f;
            __syncwarp();
            // four neighbouring tokens per lane, eight lanes a block of 32: sums from the block's
            // left (inclusive) and right (exclusive); those of whole blocks lead on to the chunk's
            // ends. Only weights inside a block are then differences of sums.
            const float4 d = *reinterpret_cast<const float4*>(&pr->delta[4 * lane]);
            // A decay below 2^-160 is none at all in fp32. Taken as 2^-160 it keeps the sums of a
            // block within 32 * 160, where an addition is off by 2^-12 at most and a difference of
            // two sums (some three additions of that size each) by 2^-9.4, 0.1 % of a weight: a
            // token that wipes the state may decay by far more, and would drown the steps behind
            // it.
            const auto step = [Ah](float dt) {
                const float l = dt * Ah;
                return l < -160.f ? -160.f : l;
            };
            const float l0 = step(d.x), l1 = step(d.y), l2 = step(d.z), l3 = step(d.w);
            const float q1 = l0 + l1, q2 = q1 + l2, q3 = q2 + l3;
            float left = q3, right = q3;
            const int at = lane & 7, block = lane >> 3;
#pragma unroll
            for (int off = 1; off < 8; off <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, left, off, 8);
                const float y = __shfl_down_sync(0xffffffffu, right, off, 8);
                if (at >= off) left += x;
                if (at + off < 8) right += y;
            }
            float lx = __shfl_up_sync(0xffffffffu, left, 1, 8);
            float rx = __shfl_down_sync(0xffffffffu, right, 1, 8);
            if (at == 0) lx = 0.f;
            if (at == 7) rx = 0.f;
            const float b0 = __shfl_sync(0xffffffffu, left, 7), b1 = __shfl_sync(0xffffffffu, left, 15),
                        b2 = __shfl_sync(0xffffffffu, left, 23), b3 = __shfl_sync(0xffffffffu, left, 31);
            const float before = block == 0 ? 0.f : block == 1 ? b0 : block == 2 ? b0 + b1 : b0 + b1 + b2;
            const float after = block == 3 ? 0.f : block == 2 ? b3 : block == 1 ? b2 + b3 : b1 + b2 + b3;
            const float total = (b0 + b1) + (b2 + b3);
            const float4 gp = make_float4(lx + l0, lx + q1, lx + q2, lx + q3);
            const float4 rp = make_float4(rx + l1 + l2 + l3, rx + l2 + l3, rx + l3, rx);
            *reinterpret_cast<float4*>(&pr->g2[4 * lane]) = gp;
            *reinterpret_cast<float4*>(&pr->u[4 * lane]) =
                make_float4(d.x * ex2(rp.x), d.y * ex2(rp.y), d.z * ex2(rp.z), d.w * ex2(rp.w));
            *reinterpret_cast<float4*>(&pr->w[4 * lane]) =
                make_float4(d.x * ex2(rp.x + after), d.y * ex2(rp.y + after),
                            d.z * ex2(rp.z + after), d.w * ex2(rp.w + after));
            *reinterpret_cast<float4*>(&pr->eg[4 * lane]) =
                make_float4(ex2(gp.x + before), ex2(gp.y + before), ex2(gp.z + before),
                            ex2(gp.w + before));
            if (lane < 16) {
                const int apart = (lane >> 2) - (lane & 3);
                pr->between[lane] = apart == 3 ? b1 + b2 : apart == 2 ? (lane & 3 ? b2 : b1) : 0.f;
            }
            if (lane == 0) pr->gamma = decay_f32(total * 0.6931471805599453f);
            logsum += total;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB_PAR + c % SC_NPAR));
        }
        // the warps' sums, in a fixed order, at the end of the kernel
        if (!OUT && lane == 0) sums[warp - 28] = logsum;
    } else if (warp >= 24) {
      // (registers are released by all four warps of a group, by the same instruction, and the
      // compiler holds what follows it to the rest: so one branch for the group)
      regs_down<SC_REG_ISSUE>();
      if (warp == 24) {
        // ------------------------------------------------------------------ tiles
        const int np = a.N > 64 ? 2 : 1;
        int c = 0, loaded_cb = 0;
        for (; c < nc; ++c) {
            const uint32_t fx = bar(SB_X + (c & 1)), fcb = bar(SB_CB + (c & 1));
            const uint32_t base = smem_u32(stage(c & 1));
            const int t = t0 + c * SCK, ta = t + SC_AHEAD * SCK;
            if (lane == 0 && c + SC_AHEAD < nc) {
                tma_prefetch_4d(&tmX, v0, ta, h * ca.xh, (int)b * ca.xb);
#pragma unroll 1
                for (int p = 0; p < np; ++p) {
                    tma_prefetch_4d(&tmB, 64 * p, ta, g * ca.bh, (int)b * ca.bb);
                    if (OUT) tma_prefetch_4d(&tmC, 64 * p, ta, g * ca.ch, (int)b * ca.cb);
                }
            }
            __syncwarp();
            if (c >= 2 && !wait2(SB_CBFREE, c - 2)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(fcb, (uint32_t)(OUT ? 2 * np : np) * SC_PANEL);
#pragma unroll 1
                for (int p = 0; p < np; ++p) {
                    tma_load_4d(base + SC_B + p * SC_PANEL, &tmB, fcb, 64 * p, t, g * ca.bh,
                                (int)b * ca.bb);
                    if (OUT)
                        tma_load_4d(base + SC_C + p * SC_PANEL, &tmC, fcb, 64 * p, t, g * ca.ch,
                                    (int)b * ca.cb);
                }
            }
            __syncwarp();
            loaded_cb = c + 1;
            if (c >= 2 && !wait2(SB_XFREE, c - 2)) break;
            if (lane == 0) {
                mbar_arrive_expect_tx(fx, SC_PANEL);
                tma_load_4d(base + SC_X, &tmX, fx, v0, t, h * ca.xh, (int)b * ca.xb);
            }
            __syncwarp();
        }
        // Nothing asynchronous may outlive the CTA: neither the commits that free the last tiles
        // (nobody else waits for them) nor, where a wait of any role ran out, the last loads
        if (c == nc) {
#pragma unroll 1
            for (int k = max(0, nc - 2); k < nc; ++k)
                if (!wait2(SB_CBFREE, k) || !wait2(SB_XFREE, k)) break;
        }
#pragma unroll 1
        for (int k = max(0, loaded_cb - 2); k < loaded_cb; ++k)
            drain(SB_CB + (k & 1), (uint32_t)((k >> 1) & 1));
#pragma unroll 1
        for (int k = max(0, c - 2); k < c; ++k)
            drain(SB_X + (k & 1), (uint32_t)((k >> 1) & 1));
      } else {
        // ------------------------------------------------------------------ MMAs
        // (whole warps, converged: see mma_ss. Three of them, so that no product waits for what
        // another waits for; each K step in a loop, whose few instructions stay in the first
        // instruction cache)
        const uint32_t base = smem_u32(sm);
        const int n = (int)__reduce_max_sync(0xffffffffu, (unsigned)nc);
        int c = 0;
        if (warp == 26) {
            // scores, as early as their tiles and the place of the P before last allow
            for (; OUT && c < n; ++c) {
                if (!wait2(SB_CB, c)) break;
                if (c >= 2 && !wait2(SB_Y, c - 2)) break;
                tc_fence_after();
                const uint32_t st = base + (c & 1) * SC_STAGE;
                mma_kmajor(tmem + TC_SCORE + 128 * (c & 1), st + SC_C,
                           smem_desc_sw128(st + SC_B, 16, 1024), 2, SC_PANEL >> 4, a.N,
                           idesc_bf16(128, 128, 0, 0));
                commit_elected(bar(SB_SCORE + (c & 1)));
                commit_elected(bar(SB_CBFREE + (c & 1)));
            }
        } else if (warp == 25) {
            // the state's
            uint32_t slot = 0, turn = 0;  // of the scaled x
            for (; c < n; ++c) {
                if (!wait2(SB_CB, c)) break;
                if (c > 0 && !wait1(SB_DSFREE, c - 1)) break;
                tc_fence_after();
                uint64_t da = smem_desc_sw128(base + (c & 1) * SC_STAGE + SC_B, SC_PANEL, 1024);
                bool ok = true;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {  // 32 tokens at a time
                    if (!(ok = mbar_wait_warp<TIMED>(bar(SB_XS + slot), turn, ca.wait_ns))) break;
                    uint64_t db =
                        smem_desc_sw128(base + SC_XS + slot * 3 * SC_XPART, SC_XPART, 1024);
#pragma unroll 1
                    for (uint32_t kk = 0; kk < 2; ++kk, da += 128, db += 128) {
                        // (one shape: only then does an accumulator's order hold)
                        constexpr uint32_t id = idesc_bf16(128, 64, 1, 1);
                        mma_ss(tmem + TC_DS, da, db, id, q | kk);
                        mma_ss(tmem + TC_DS + SCV, da, db + (SC_XPART >> 4), id, q | kk);
                        mma_ss(tmem + TC_DS + SCV, da, db + (2 * SC_XPART >> 4), id, 1);
                    }
                    commit_elected(bar(SB_XSFREE + q));
                    if (++slot == SC_NXS) slot = 0, turn ^= 1;
                }
                if (!ok) break;
                commit_elected(bar(SB_DS));
                commit_elected(bar(SB_CBFREE + (c & 1)));
            }
        } else {
            // the outputs'
            for (; OUT && c < n; ++c) {
                const uint32_t s = c & 1, st = base + s * SC_STAGE;
                if (!wait1(SB_ST, c)) break;
                if (!wait2(SB_CB, c)) break;
                if (c > 0 && !wait1(SB_YFREE, c - 1)) break;
                tc_fence_after();
                mma_kmajor(tmem + TC_INTER, st + SC_C,
                           smem_desc_sw128(base + SC_S, SC_PANEL, 1024), 128, 4 * 128, a.N,
                           idesc_bf16(128, 64, 0, 1));
                commit_elected(bar(SB_CBFREE + s));
                if (!wait2(SB_CLEAR, c)) break;
                if (!wait2(SB_P, c)) break;
                tc_fence_after();
                uint64_t dx = smem_desc_sw128(st + SC_X, SC_PANEL, 1024);
                uint32_t pa = tmem + TC_SCORE + 128 * s;
#pragma unroll 1
                for (uint32_t kk = 0; kk < 8; ++kk, dx += 128, pa += 16)
                    mma_ts(tmem + TC_INTRA, pa, dx, idesc_bf16(128, 64, 0, 1), kk);
                commit_elected(bar(SB_Y + s));
                commit_elected(bar(SB_XFREE + s));
            }
        }
        // products and commits in flight may not outlive the CTA's memory: those of a role whose
        // wait ran out, or whose results nobody took up since another's did
        if (n > 0 && (OUT || warp == 25)) {
            commit_elected(bar(SB_DRAIN + warp - 25));
            drain(SB_DRAIN + warp - 25, 0);
        }
      }
    } else if (warp < 8) {
        // ------------------------------------------------------------------ P from the scores
        // (two warps per 32 rows, which take turns at 16 columns, so that both have their part of the
        // diagonal block. The P of 16 columns goes over the first half of their scores, so no warp
        // writes what another reads.)
        regs_down<SC_REG_P>();
        if constexpr (OUT) {
            const int i = tid & 127, rw = warp & 3;
            for (int c = 0; c < nc; ++c) {
                const int s = c & 1, nv = valid(c);
                if (!wait_par(c)) break;
                const SsmChunkPar* pr = par(c % SC_NPAR);
                const float gi = pr->g2[i];
                if (!wait2(SB_SCORE, c)) break;
                tc_fence_after();
                const uint32_t tsc = trow + TC_SCORE + 128 * s;
                // 16 columns at a time, in a loop, whose code stays in the instruction cache
#pragma unroll 1
                for (int j0 = 16 * (warp >> 2); j0 < SCK; j0 += 32) {
                    const int J = j0 >> 5;
                    uint32_t pk[8];
                    if (J <= rw) {
                        float2 x[8];
                        tmem_ld16(tsc + j0, reinterpret_cast<float*>(x));
                        if (J < rw) {
                            const float r = ex2(gi + pr->between[4 * rw + J]);
                            const float4* u = reinterpret_cast<const float4*>(pr->u + j0);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 w = u[e];
                                x[2 * e] = mul2(mul2(make_float2(r, r), make_float2(w.x, w.y)),
                                                x[2 * e]);
                                x[2 * e + 1] = mul2(mul2(make_float2(r, r), make_float2(w.z, w.w)),
                                                    x[2 * e + 1]);
                            }
                        } else {
                            const float4* gq = reinterpret_cast<const float4*>(pr->g2 + j0);
                            const float4* dq = reinterpret_cast<const float4*>(pr->delta + j0);
                            float2 w[8];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const float4 gj = gq[e], dj = dq[e];
                                w[2 * e] = mul2(make_float2(dj.x, dj.y),
                                                make_float2(ex2(gi - gj.x), ex2(gi - gj.y)));
                                w[2 * e + 1] = mul2(make_float2(dj.z, dj.w),
                                                    make_float2(ex2(gi - gj.z), ex2(gi - gj.w)));
                            }
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 8; ++e) x[e] = mul2(x[e], w[e]);
                        }
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = pack2(x[e]);
                        if (J == rw || nv < SCK) {
                            // nothing above the diagonal, and nothing behind the sequence: by bits,
                            // as it may be infinite or NaN
                            const int top = min(i, nv - 1) - j0;
#pragma unroll
                            for (int e = 0; e < 8; ++e) pk[e] &= pair_mask(top - 2 * e);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e) pk[e] = 0;
                    }
                    tmem_st8(tsc + j0, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(SB_P + s));
                release_par(c);
            }
        }
    } else if (warp < 16) {
        // ------------------------------------------------------------------ scaled x
        // (a thread per token and 32 channels: warps 8 + q and 12 + q the tokens 32 q ..; each 32
        // tokens have a slot of their own, which the product frees)
        regs_down<SC_REG_X>();
        const int q = warp & 3, j = 32 * q + lane, half = (warp >> 2) & 1;
        // 16-byte pieces keep their swizzled places; each lane starts at another one, so that eight
        // lanes cover all banks
        const int at0 = 64 * half, swz = (j & 7) << 4;
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1;
            if (!wait_par(c)) break;
            const float w = par(c % SC_NPAR)->w[j];
            release_par(c);
            if (!wait2(SB_X, c)) break;
            uint8_t* xr = stage(s) + SC_X + j * 128;
            const bool live = j < valid(c);
            uint32_t x[16];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint4 v = *reinterpret_cast<const uint4*>(xr + ((at0 + 16 * k) ^ swz));
                x[4 * k] = v.x, x[4 * k + 1] = v.y, x[4 * k + 2] = v.z, x[4 * k + 3] = v.w;
            }
            if (valid(c) < SCK) {  // nothing behind the sequence may enter a product, not even as
                                   // 0 * NaN: it goes from the tiles of x and (once there) of B
                if (!wait2(SB_CB, c)) break;
                if (!live) {
                    uint8_t* br = stage(s) + SC_B + j * 128;
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] = 0;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int at = (at0 + 16 * k) ^ swz;
                        const uint4 z = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(xr + at) = z;
                        *reinterpret_cast<uint4*>(br + at) = z;
                        *reinterpret_cast<uint4*>(br + SC_PANEL + at) = z;
                    }
                }
                fence_async_smem();
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(SB_CLEAR + s));
                if (!OUT) mbar_arrive(bar(SB_XFREE + s));
            }
            // the slot's last use was three quarters ago. (Waited for by quarter, not by slot: that
            // quarter's use of a chunk before is known to be over, since this warp's last one
            // waited for it, so parity tells its phases apart.)
            const uint32_t use = 4 * c + q, slot = use % SC_NXS, last = use - SC_NXS;
            if (use >= SC_NXS &&
                !mbar_wait_warp<TIMED>(bar(SB_XSFREE + (last & 3)), (last >> 2) & 1, ca.wait_ns))
                break;
            uint8_t* to = sm + SC_XS + slot * 3 * SC_XPART + lane * 128;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                uint32_t p1[4], p2[4], p3[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 v = mul2(unpack2(x[4 * k + e]), make_float2(w, w));
                    p1[e] = pack2(v);
                    v = fma2(unpack2(p1[e]), make_float2(-1.f, -1.f), v);
                    p2[e] = pack2(v);
                    v = fma2(unpack2(p2[e]), make_float2(-1.f, -1.f), v);
                    p3[e] = pack2(v);
                }
                uint8_t* at = to + ((at0 + 16 * k) ^ swz);
                *reinterpret_cast<uint4*>(at) = make_uint4(p1[0], p1[1], p1[2], p1[3]);
                *reinterpret_cast<uint4*>(at + SC_XPART) = make_uint4(p2[0], p2[1], p2[2], p2[3]);
                *reinterpret_cast<uint4*>(at + 2 * SC_XPART) = make_uint4(p3[0], p3[1], p3[2], p3[3]);
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB_XS + slot));
        }
    } else if (warp < 20) {
        // ------------------------------------------------------------------ the state
        regs_up<SC_REG_STATE>();
        const int n = tid & 127;
        const long PN = (long)a.P * a.N;
        const bool row = n < a.N;
        float2 st[SCV / 2];
        const float* enter = nullptr;
        if (seg == 0)
            enter = a.S0 ? a.S0 + bh * PN : nullptr;
        else if (OUT)
            enter = a.seg_state + (bh * (a.nseg - 1) + seg - 1) * PN;
#pragma unroll
        for (int p = 0; p < SCV / 2; ++p) st[p] = make_float2(0.f, 0.f);
        if (enter && row) {
            const float* e = enter + (long)v0 * a.N + n;
#pragma unroll
            for (int p = 0; p < SCV / 2; ++p, e += 2 * a.N)
                if (p < 16 || pv == SCV) st[p] = make_float2(e[0], e[a.N]);
        }
        uint8_t* srow = sm + SC_S + n * 128;
        auto copy = [&]() {
            if (OUT) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(srow + ((k ^ (n & 7)) << 4)) =
                        make_uint4(pack2(st[4 * k]), pack2(st[4 * k + 1]), pack2(st[4 * k + 2]),
                                   pack2(st[4 * k + 3]));
                fence_async_smem();
                mbar_arrive(bar(SB_ST));
            }
        };
        copy();
        for (int c = 0; c < nc; ++c) {
            if (!wait_par(c)) break;
            const float gamma = par(c % SC_NPAR)->gamma;
            release_par(c);
            if (!wait1(SB_DS, c)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 0; p < SCV; p += 8) {
                float2 hi[4], lo[4];
                tmem_ld8(trow + TC_DS + p, reinterpret_cast<float*>(hi));
                tmem_ld8(trow + TC_DS + SCV + p, reinterpret_cast<float*>(lo));
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    st[p / 2 + k] =
                        fma2(make_float2(gamma, gamma), st[p / 2 + k], add2(hi[k], lo[k]));
            }
            tc_fence_before();
            mbar_arrive(bar(SB_DSFREE));
            if (c + 1 < nc) {  // the inter product has to have read the old copy
                if (OUT && !wait2(SB_Y, c)) break;
                copy();
            }
        }
        float* leave = !OUT ? a.seg_state + (bh * (a.nseg - 1) + seg) * PN
                       : seg == a.nseg - 1 && a.S_final ? a.S_final + bh * PN
                                                        : nullptr;
        if (leave && row) {
            float* e = leave + (long)v0 * a.N + n;
#pragma unroll
            for (int p = 0; p < SCV / 2; ++p, e += 2 * a.N)
                if (p < 16 || pv == SCV) e[0] = st[p].x, e[a.N] = st[p].y;
        }
    } else if (warp < 24) {
        // ------------------------------------------------------------------ outputs
        regs_up<SC_REG_OUT>();
        if constexpr (OUT) {
            const int i = tid & 127;
            const float Dh = a.D ? a.D[h] : 0.f;
            __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + b * a.osb + h * a.osh +
                                ((long)t0 + i) * a.ost + v0;
            for (int c = 0; c < nc; ++c, op += SCK * a.ost) {
                if (!wait_par(c)) break;
                const float eg = par(c % SC_NPAR)->eg[i];
                release_par(c);
                if (!wait2(SB_X, c)) break;
                // x into registers and its tile free before the products are there; outputs take
                // its place and leave once the products' columns are free
                const uint8_t* xr = stage(c & 1) + SC_X + i * 128;
                uint32_t y[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const uint4 v =
                        *reinterpret_cast<const uint4*>(xr + ((16 * k) ^ ((i & 7) << 4)));
                    y[4 * k] = v.x, y[4 * k + 1] = v.y, y[4 * k + 2] = v.z, y[4 * k + 3] = v.w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(SB_XFREE + (c & 1)));
                if (!wait2(SB_Y, c)) break;
                tc_fence_after();
#pragma unroll
                for (int k = 0; k < SCV; k += 8) {
                    float2 in[4], it[4];
                    tmem_ld8(trow + TC_INTRA + k, reinterpret_cast<float*>(in));
                    tmem_ld8(trow + TC_INTER + k, reinterpret_cast<float*>(it));
                    tmem_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[k / 2 + e] = pack2(fma2(make_float2(Dh, Dh), unpack2(y[k / 2 + e]),
                                                  fma2(make_float2(eg, eg), it[e], in[e])));
                }
                tc_fence_before();
                mbar_arrive(bar(SB_YFREE));
                if (i < valid(c)) {
                    // (a store costs a cycle per row, whatever its width)
#pragma unroll
                    for (int k = 0; k < SCV; k += 16)
                        if (k < 32 || pv == SCV) {
                            const uint32_t* u = y + k / 2;
                            if (ca.out32) {
                                st_global_32(op + k, u);
                            } else {
                                reinterpret_cast<uint4*>(op + k)[0] =
                                    make_uint4(u[0], u[1], u[2], u[3]);
                                reinterpret_cast<uint4*>(op + k)[1] =
                                    make_uint4(u[4], u[5], u[6], u[7]);
                            }
                        }
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (!OUT && tid == 0 && v0 == 0)
        a.seg_log[bh * (a.nseg - 1) + seg] =
            ((sums[0] + sums[1]) + (sums[2] + sums[3])) * 0.6931471805599453f;
    if (warp == 25) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------
// cuTensorMapEncodeTiled of the driver in use (looked up once).
inline PFN_cuTensorMapEncodeTiled_v12000 ssm_map_encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                                            cudaEnableDefault, &q) == cudaSuccess &&
                           q == cudaDriverEntryPointSuccess;
        return found ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p) : nullptr;
    }();
    return fn;
}

// Map over a view of nb x nh x T rows of `inner` bf16, box {64 channels, SCK tokens}; channels
// and tokens outside read as zero. *mh, *mb: whether the head and batch coordinates count (a
// dimension that repeats one row, or has size one, keeps coordinate 0).
inline bool ssm_map(CUtensorMap* m, const SsmView& v, int inner, int T, int nh, int nb, int* mh,
                    int* mb) {
    auto enc = ssm_map_encoder();
    if (!enc) return false;
    const cuuint64_t any = 16 * (cuuint64_t)((inner * 2 + 15) / 16);
    *mh = nh > 1 && v.sh > 0;
    *mb = nb > 1 && v.sb > 0;
    const cuuint64_t dims[4] = {(cuuint64_t)inner, (cuuint64_t)T, *mh ? (cuuint64_t)nh : 1,
                                *mb ? (cuuint64_t)nb : 1};
    const cuuint64_t strides[3] = {T > 1 ? (cuuint64_t)v.st * 2 : any,
                                   *mh ? (cuuint64_t)v.sh * 2 : any,
                                   *mb ? (cuuint64_t)v.sb * 2 : any};
    const cuuint32_t box[4] = {64, SCK, 1, 1}, estr[4] = {1, 1, 1, 1};
    return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(v.p), dims, strides, box,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Whether the tensor maps can describe the views: tokens that repeat one row, and strides of
// 2^40 bytes, they cannot.
inline bool ssm_chunked_fits(const SsmArgs& a) {
    const SsmView* views[3] = {&a.x, &a.Bm, &a.Cm};
    for (const SsmView* v : views) {
        if (a.T > 1 && (v->st <= 0 || v->st >= 1l << 39)) return false;
        if (v->sh >= 1l << 39 || v->sb >= 1l << 39) return false;
    }
    return true;
}

// Segments of a chunked scan: the count with the least time by a model in units of one chunk with
// outputs (2.9 us): a chunk without takes SC_STATES, a CTA SC_START to begin and to end, the two
// more launches SC_LAUNCHES and SC_CHAIN for each state that they chain. Fitted to 16 heads of 64
// channels and 256 chunks, where 9 segments (one wave of CTAs) took 147 us and 37 (four waves) 186;
// other shapes were not fitted.
constexpr float SC_STATES = 0.55f, SC_START = 1.5f, SC_LAUNCHES = 2.f, SC_CHAIN = 0.05f;

inline void plan_ssm_chunked(SsmArgs* a, int sms) {
    const long ctas = (long)a->B * a->H * ((a->P + SCV - 1) / SCV);
    const int nc = (int)(((long)a->T + SCK - 1) / SCK);
    auto waves = [&](int n) { return (float)((ctas * n + sms - 1) / sms); };
    float best = waves(1) * (nc + SC_START);
    int len = nc;
    const int most = (int)std::min<long>(nc, 4l * sms / ctas);
    for (int n = 2; n <= most; ++n) {
        const int l = (nc + n - 1) / n, m = (nc + l - 1) / l;
        const float t = waves(m) * (l + SC_START) + waves(m - 1) * (SC_STATES * l + SC_START) +
                        SC_LAUNCHES + SC_CHAIN * m;
        if (t < best) best = t, len = l;
    }
    a->seg_len = len * SCK;
    a->nseg = (nc + len - 1) / len;
}

template <int PASS, bool TIMED>
int launch_ssm_chunked_pass(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc,
                            const SsmChunkArgs& ca, long gx, int gy, cudaStream_t stream) {
    const int smem = SC_TOTAL + 1024;
    auto kern = ssm_chunked_kernel<PASS, TIMED>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return DR_ERR_CUDA;
    kern<<<dim3((unsigned)gx, (unsigned)gy), SC_THREADS, smem, stream>>>(mx, mb, mc, ca);
    return cudaGetLastError() == cudaSuccess ? DR_OK : DR_ERR_CUDA;
}

// The planned passes (a.nseg, a.seg_len and the scratch set).
template <bool TIMED>
int launch_ssm_chunked(const SsmArgs& a, uint32_t wait_ns, cudaStream_t stream) {
    SsmChunkArgs ca;
    ca.s = a;
    ca.wait_ns = wait_ns;
    CUtensorMap mx, mb, mc;
    if (!ssm_map(&mx, a.x, a.P, a.T, a.H, a.B, &ca.xh, &ca.xb) ||
        !ssm_map(&mb, a.Bm, a.N, a.T, a.G, a.B, &ca.bh, &ca.bb) ||
        !ssm_map(&mc, a.Cm, a.N, a.T, a.G, a.B, &ca.ch, &ca.cb))
        return DR_ERR_CUDA;
    const long ostrides = (a.B > 1 ? a.osb : 0) | (a.H > 1 ? a.osh : 0) | (a.T > 1 ? a.ost : 0);
    ca.out32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0 && (ostrides & 15) == 0;
    const long gx = (long)a.B * a.H * ((a.P + SCV - 1) / SCV);
    if (gx > 0x7fffffffl || a.nseg > 65535) return DR_ERR_UNSUPPORTED;
    if (a.nseg > 1) {
        int rc = launch_ssm_chunked_pass<SSM_PASS_STATES, TIMED>(mx, mb, mc, ca, gx,
                                                                 a.nseg - 1, stream);
        if (rc == DR_OK) rc = launch_ssm_chain(a, stream);
        if (rc != DR_OK) return rc;
    }
    return launch_ssm_chunked_pass<SSM_PASS_OUTPUTS, TIMED>(mx, mb, mc, ca, gx, a.nseg, stream);
}

}  // namespace drscan
