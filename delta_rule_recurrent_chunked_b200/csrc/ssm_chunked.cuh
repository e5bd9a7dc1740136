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
//     state   B^T [xh | xl]     M=128 N=128 K=128   xh + xl = exp(g_Q - g_j) delta_j x_j
// The state stays in the registers of one warpgroup in fp32 (a lane per row n of S^T).
//
// Roundings to bf16, each a choice: P and the copy of S that the outputs read (2^-8 of a
// product; the outputs are rounded to bf16 themselves), and the scaled x in two halves xh + xl
// (2^-16: one half alone would put 2^-8 into the state, which is carried on and returned in
// fp32). x, B and C are bf16 as they come.
//
// exp(g_i - g_j) for columns of an earlier 32-token block J of the chunk is taken as
// exp(g_i - g_end(J)) exp(g_end(J) - g_j), both <= 1: one exponential per row and block and one
// per token instead of one per element; only the diagonal 32 x 32 blocks take one per element.
//
// Roles (576 threads): warps 0-3 weigh the scores (P), 4-7 scale x, 8-11 carry the state, 12-15
// write the outputs, warp 16 loads tiles by TMA and prepares the per-token factors, warp 17
// issues the MMAs. Tiles are double-buffered; scores run one chunk ahead, so the only serial
// dependence between chunks is state -> registers -> S copy -> inter. Every wait is bounded.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>

#include "ssm_scan.cuh"

namespace drscan {

constexpr int SCK = 128;        // tokens per chunk
constexpr int SCV = 64;         // value channels per CTA
constexpr int SC_THREADS = 576;

// Shared memory (bytes). A tile row is 128 bytes (64 bf16) of a 128-byte-swizzled panel.
constexpr int SC_PANEL = SCK * 128;                      // 128 rows x 64 channels
constexpr int SC_C = 0;                                  // [stage] two panels
constexpr int SC_B = SC_C + 2 * SC_PANEL;                // two panels
constexpr int SC_X = SC_B + 2 * SC_PANEL;                // one panel
constexpr int SC_STAGE = SC_X + SC_PANEL;
constexpr int SC_XS = 2 * SC_STAGE;                      // xh, xl panels
constexpr int SC_S = SC_XS + 2 * SC_PANEL;               // S^T rows n, 64 value channels
constexpr int SC_PAR = SC_S + SC_PANEL;                  // [stage] SsmChunkPar
struct SsmChunkPar {
    float g2[SCK];     // g_i log2(e)
    float delta[SCK];
    float u[SCK];      // delta_j exp(g_end(J) - g_j), J the token's block of 32
    float w[SCK];      // delta_j exp(g_Q - g_j)
    float eg[SCK];     // exp(g_i)
    float gamma;       // exp(g_Q)
    float pad[3];
};
constexpr int SC_BAR = SC_PAR + 2 * (int)sizeof(SsmChunkPar);
enum {
    SB_FULL = 0,     // [2] tiles and factors of a stage are there
    SB_FREE = 2,     // [2] .. may be overwritten
    SB_SCORE = 4,    // [2] scores are in tensor memory
    SB_P = 6,        // [2] P is in tensor memory
    SB_XS = 8,       // scaled x is in shared memory
    SB_DS = 9,       // the chunk's state product is in tensor memory
    SB_ST = 10,      // the entering state's copy is in shared memory (and the product read)
    SB_Y = 11,       // inter and intra products are in tensor memory
    SB_YFREE = 12,   // .. have been read
    SB_COUNT = 13
};
constexpr int SC_TOTAL = SC_BAR + 8 * SB_COUNT + 24;
// Tensor memory columns
constexpr uint32_t TC_SCORE = 0;   // [2] 128 columns; P in the first 64
constexpr uint32_t TC_INTRA = 256, TC_INTER = 320, TC_DS = 384;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* map, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
        "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T: A packs two bf16 of K in a 32-bit column. One thread.
__device__ __forceinline__ void tc_mma_bf16_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                               uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// After an abort: waits (bounded) for the async work of a phase that was started.
__device__ __forceinline__ void mbar_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_test(bar, parity) && global_timer_ns() - t0 < DRSCAN_WAIT_LIMIT_NS) {
    }
}

struct SsmChunkArgs {
    SsmArgs s;
    // 1 where the tensor map's head / batch coordinate counts, 0 where the view repeats
    int xh, xb, bh, bb, ch, cb;
};

// grid: (B * H * slices of SCV value channels, segments of this pass); block: SC_THREADS.
template <int PASS>
__global__ void __launch_bounds__(SC_THREADS, 1) ssm_chunked_kernel(
    const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmB,
    const __grid_constant__ CUtensorMap tmC, const __grid_constant__ SsmChunkArgs ca) {
    constexpr bool OUT = PASS == SSM_PASS_OUTPUTS;
    const SsmArgs& a = ca.s;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + SC_BAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(sm + SC_BAR + 8 * SB_COUNT);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(sm + SC_BAR + 8 * SB_COUNT + 8);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto stage = [&](int s) { return sm + s * SC_STAGE; };
    auto par = [&](int s) {
        return reinterpret_cast<SsmChunkPar*>(sm + SC_PAR + s * (int)sizeof(SsmChunkPar));
    };

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
    const int nc = (ntok + SCK - 1) / SCK;
    auto valid = [&](int c) { return min(SCK, ntok - c * SCK); };

    if (tid == 0) {
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(SB_FULL + s), 2);
            mbar_init(bar(SB_FREE + s), OUT ? 16 : 8);  // warps of the roles that read a stage
            mbar_init(bar(SB_SCORE + s), 1);
            mbar_init(bar(SB_P + s), 128);
        }
        mbar_init(bar(SB_XS), 128);
        mbar_init(bar(SB_DS), 1);
        mbar_init(bar(SB_ST), 128);
        mbar_init(bar(SB_Y), 1);
        mbar_init(bar(SB_YFREE), 128);
        *abort_flag = 0;
        mbar_init_fence();
    }
    if (warp == 17) tmem_alloc(smem_u32(tmem_holder), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    // a warp's 32 lanes of tensor memory
    const uint32_t trow = tmem + ((uint32_t)(warp & 3) << 21);
    auto release = [&](int s) {  // this warp is done with the stage
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(SB_FREE + s));
    };

    if (warp == 16) {
        // ------------------------------------------------------------------ loads and factors
        const float l2e = 1.4426950408889634f;
        const float Ah = a.A[h];
        float logsum = 0.f;
        float dnext[4];
        auto fetch = [&](int c) {  // delta of this lane's four tokens, 0 behind the sequence
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = c * SCK + 4 * lane + k;
                dnext[k] = t < ntok ? ssm_delta(a, b, h, (long)t0 + t) : 0.f;
            }
        };
        if (nc > 0) fetch(0);
        int c = 0;
        for (; c < nc; ++c) {
            const int s = c & 1;
            if (c >= 2 && !mbar_wait(bar(SB_FREE + s), (uint32_t)(((c >> 1) - 1) & 1), abort_flag))
                break;
            if (lane == 0) {
                const uint32_t full = bar(SB_FULL + s), base = smem_u32(stage(s));
                const int np = a.N > 64 ? 2 : 1;
                mbar_arrive_expect_tx(full, (uint32_t)((OUT ? 2 * np : np) + 1) * SC_PANEL);
                for (int p = 0; p < np; ++p) {
                    tma_load_4d(base + SC_B + p * SC_PANEL, &tmB, full, 64 * p, t0 + c * SCK,
                                g * ca.bh, (int)b * ca.bb);
                    if (OUT)
                        tma_load_4d(base + SC_C + p * SC_PANEL, &tmC, full, 64 * p, t0 + c * SCK,
                                    g * ca.ch, (int)b * ca.cb);
                }
                tma_load_4d(base + SC_X, &tmX, full, v0, t0 + c * SCK, h * ca.xh, (int)b * ca.xb);
            }
            float d[4], l[4], pre[4], suf[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) d[k] = dnext[k], l[k] = d[k] * Ah * l2e;
            if (c + 1 < nc) fetch(c + 1);
            // inclusive sums from the left, exclusive from the right (short near the chunk's end,
            // where the weights of the state are largest)
            pre[0] = l[0], pre[1] = pre[0] + l[1], pre[2] = pre[1] + l[2], pre[3] = pre[2] + l[3];
            suf[3] = 0.f, suf[2] = l[3], suf[1] = suf[2] + l[2], suf[0] = suf[1] + l[1];
            float left = pre[3], right = pre[3];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float x = __shfl_up_sync(0xffffffffu, left, off);
                const float y = __shfl_down_sync(0xffffffffu, right, off);
                if (lane >= off) left += x;
                if (lane + off < 32) right += y;
            }
            const float total = __shfl_sync(0xffffffffu, left, 31);
            float lx = __shfl_up_sync(0xffffffffu, left, 1);
            float rx = __shfl_down_sync(0xffffffffu, right, 1);
            lx = lane == 0 ? 0.f : lx;
            rx = lane == 31 ? 0.f : rx;
#pragma unroll
            for (int k = 0; k < 4; ++k) pre[k] += lx, suf[k] += rx;
            const float end = __shfl_sync(0xffffffffu, pre[3], lane | 7);  // of the block of 32
            SsmChunkPar* pr = par(s);
            *reinterpret_cast<float4*>(&pr->g2[4 * lane]) = make_float4(pre[0], pre[1], pre[2], pre[3]);
            *reinterpret_cast<float4*>(&pr->delta[4 * lane]) = make_float4(d[0], d[1], d[2], d[3]);
            *reinterpret_cast<float4*>(&pr->u[4 * lane]) =
                make_float4(d[0] * ex2(end - pre[0]), d[1] * ex2(end - pre[1]),
                            d[2] * ex2(end - pre[2]), d[3] * ex2(end - pre[3]));
            *reinterpret_cast<float4*>(&pr->w[4 * lane]) =
                make_float4(d[0] * exp2f(suf[0]), d[1] * exp2f(suf[1]), d[2] * exp2f(suf[2]),
                            d[3] * exp2f(suf[3]));
            *reinterpret_cast<float4*>(&pr->eg[4 * lane]) =
                make_float4(ex2(pre[0]), ex2(pre[1]), ex2(pre[2]), ex2(pre[3]));
            if (lane == 0) pr->gamma = exp2f(total);
            logsum += total;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(SB_FULL + s));
        }
        if (!OUT && lane == 0 && v0 == 0)
            a.seg_log[bh * (a.nseg - 1) + seg] = logsum * 0.6931471805599453f;
        if (*abort_flag) {  // loads in flight may not outlive the CTA
            for (int k = max(0, c - 2); k < c; ++k)
                mbar_drain(bar(SB_FULL + (k & 1)), (uint32_t)((k >> 1) & 1));
        }
    } else if (warp == 17) {
        // ------------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            constexpr uint32_t id_score = idesc_bf16(128, 128, 0, 0);
            constexpr uint32_t id_val = idesc_bf16(128, 64, 0, 1);
            constexpr uint32_t id_state = idesc_bf16(128, 128, 1, 1);
            const int ksteps = a.N / 16;
            const uint32_t ss = smem_u32(sm + SC_S), xs = smem_u32(sm + SC_XS);
            auto scores = [&](int c) {
                const uint32_t st = smem_u32(stage(c & 1));
                for (int kk = 0; kk < ksteps; ++kk) {
                    const uint32_t o = (kk >> 2) * SC_PANEL + (kk & 3) * 32;
                    tc_mma_bf16(tmem + TC_SCORE + 128 * (c & 1),
                                smem_desc_sw128(st + SC_C + o, 16, 1024),
                                smem_desc_sw128(st + SC_B + o, 16, 1024), id_score, kk > 0);
                }
                tc_commit(bar(SB_SCORE + (c & 1)));
            };
            bool ok = true;
            int c = 0;
            if (OUT && nc > 0) {
                ok = mbar_wait(bar(SB_FULL), 0, abort_flag);
                if (ok) scores(0);
            }
            for (; ok && c < nc; ++c) {
                const int s = c & 1;
                const uint32_t st = smem_u32(stage(s));
                if (OUT && c + 1 < nc) {
                    // the next chunk's scores, where the chunk before had its P
                    ok = mbar_wait(bar(SB_FULL + (s ^ 1)), (uint32_t)(((c + 1) >> 1) & 1),
                                   abort_flag) &&
                         (c == 0 || mbar_wait(bar(SB_Y), (uint32_t)((c - 1) & 1), abort_flag));
                    if (!ok) break;
                    scores(c + 1);
                }
                if (!OUT && !(ok = mbar_wait(bar(SB_FULL + s), (uint32_t)((c >> 1) & 1), abort_flag)))
                    break;
                if (!(ok = mbar_wait(bar(SB_ST), (uint32_t)(c & 1), abort_flag))) break;
                tc_fence_after();
                if (OUT) {
                    if (c > 0 &&
                        !(ok = mbar_wait(bar(SB_YFREE), (uint32_t)((c - 1) & 1), abort_flag)))
                        break;
                    tc_fence_after();
                    for (int kk = 0; kk < ksteps; ++kk)
                        tc_mma_bf16(tmem + TC_INTER,
                                    smem_desc_sw128(st + SC_C + (kk >> 2) * SC_PANEL + (kk & 3) * 32,
                                                    16, 1024),
                                    smem_desc_sw128(ss + kk * 2048, SC_PANEL, 1024), id_val, kk > 0);
                }
                // scaled x is waited for before the intra product too: its writers clear the rows
                // of x and B behind a sequence
                ok = mbar_wait(bar(SB_XS), (uint32_t)(c & 1), abort_flag);
                if (!ok) break;
                if (OUT) {
                    if (!(ok = mbar_wait(bar(SB_P + s), (uint32_t)((c >> 1) & 1), abort_flag))) break;
                    tc_fence_after();
                    for (int kk = 0; kk < 8; ++kk)
                        tc_mma_bf16_ta(tmem + TC_INTRA, tmem + TC_SCORE + 128 * s + 8 * kk,
                                       smem_desc_sw128(st + SC_X + kk * 2048, SC_PANEL, 1024),
                                       id_val, kk > 0);
                    tc_commit(bar(SB_Y));
                }
                for (int kk = 0; kk < 8; ++kk)
                    tc_mma_bf16(tmem + TC_DS, smem_desc_sw128(st + SC_B + kk * 2048, SC_PANEL, 1024),
                                smem_desc_sw128(xs + kk * 2048, SC_PANEL, 1024), id_state, kk > 0);
                tc_commit(bar(SB_DS));
            }
            if (!ok) {  // products in flight may not outlive the CTA's memory
                tc_commit(bar(SB_DS));
                mbar_drain(bar(SB_DS), (uint32_t)(c & 1));
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------------------ P from the scores
        if constexpr (OUT) {
            const int i = tid;
            for (int c = 0; c < nc; ++c) {
                const int s = c & 1, nv = valid(c);
                if (!mbar_wait(bar(SB_FULL + s), (uint32_t)((c >> 1) & 1), abort_flag)) break;
                const SsmChunkPar* pr = par(s);
                const float gi = pr->g2[i];
                if (!mbar_wait(bar(SB_SCORE + s), (uint32_t)((c >> 1) & 1), abort_flag)) break;
                tc_fence_after();
                const uint32_t tsc = trow + TC_SCORE + 128 * s;
#pragma unroll 1
                for (int J = 0; J < 4; ++J) {
                    uint32_t pk[16];
                    if (J <= warp) {
                        float x[32];
                        tmem_ld16(tsc + 32 * J, x);
                        tmem_ld16(tsc + 32 * J + 16, x + 16);
                        tmem_wait_ld();
                        if (J < warp) {
                            const float r = ex2(gi - pr->g2[32 * J + 31]);
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 u = *reinterpret_cast<const float4*>(&pr->u[32 * J + j]);
                                x[j] *= r * u.x, x[j + 1] *= r * u.y;
                                x[j + 2] *= r * u.z, x[j + 3] *= r * u.w;
                            }
                        } else {
                            // every lane of the warp is in its diagonal block
#pragma unroll
                            for (int j = 0; j < 32; j += 4) {
                                const float4 gj = *reinterpret_cast<const float4*>(&pr->g2[32 * J + j]);
                                const float4 dj =
                                    *reinterpret_cast<const float4*>(&pr->delta[32 * J + j]);
                                x[j] = j <= lane ? x[j] * (dj.x * ex2(gi - gj.x)) : 0.f;
                                x[j + 1] = j + 1 <= lane ? x[j + 1] * (dj.y * ex2(gi - gj.y)) : 0.f;
                                x[j + 2] = j + 2 <= lane ? x[j + 2] * (dj.z * ex2(gi - gj.z)) : 0.f;
                                x[j + 3] = j + 3 <= lane ? x[j + 3] * (dj.w * ex2(gi - gj.w)) : 0.f;
                            }
                        }
                        if (nv < SCK) {  // whatever lies behind the sequence (NaN too) weighs nothing
#pragma unroll
                            for (int j = 0; j < 32; ++j) x[j] = 32 * J + j < nv ? x[j] : 0.f;
                        }
#pragma unroll
                        for (int j = 0; j < 16; ++j) pk[j] = pack_bf16(x[2 * j], x[2 * j + 1]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) pk[j] = 0;
                    }
                    // over the scores of columns 16 J ..: read already, by this very lane
                    tmem_st16(tsc + 16 * J, reinterpret_cast<const float*>(pk));
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(SB_P + s));
                release(s);
            }
        }
    } else if (warp < 8) {
        // ------------------------------------------------------------------ scaled x
        const int j = tid - 128;
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1;
            if (!mbar_wait(bar(SB_FULL + s), (uint32_t)((c >> 1) & 1), abort_flag)) break;
            const float w = par(s)->w[j];
            uint8_t* xr = stage(s) + SC_X + j * 128;
            uint8_t* br = stage(s) + SC_B + j * 128;
            uint8_t* hi = sm + SC_XS + j * 128;
            const bool live = j < valid(c);
            uint4 raw[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) raw[k] = *reinterpret_cast<const uint4*>(xr + k * 16);
            if (c > 0 && !mbar_wait(bar(SB_DS), (uint32_t)((c - 1) & 1), abort_flag)) break;
            if (live) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {  // 16-byte pieces keep their swizzled places
                    float x[8], rest[8];
                    Vec16<__nv_bfloat16>::unpack(raw[k], x);
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] *= w;
                    const uint4 top = Vec16<__nv_bfloat16>::pack(x);
                    Vec16<__nv_bfloat16>::unpack(top, rest);
#pragma unroll
                    for (int e = 0; e < 8; ++e) rest[e] = x[e] - rest[e];
                    *reinterpret_cast<uint4*>(hi + k * 16) = top;
                    *reinterpret_cast<uint4*>(hi + SC_PANEL + k * 16) =
                        Vec16<__nv_bfloat16>::pack(rest);
                }
            } else {  // nothing behind the sequence may enter a product, not even as 0 * NaN
                const uint4 z = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    *reinterpret_cast<uint4*>(hi + k * 16) = z;
                    *reinterpret_cast<uint4*>(hi + SC_PANEL + k * 16) = z;
                    *reinterpret_cast<uint4*>(xr + k * 16) = z;
                    *reinterpret_cast<uint4*>(br + k * 16) = z;
                    *reinterpret_cast<uint4*>(br + SC_PANEL + k * 16) = z;
                }
            }
            fence_async_smem();
            mbar_arrive(bar(SB_XS));
            release(s);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------------------ the state
        const int n = tid - 256;
        const long PN = (long)a.P * a.N;
        const bool row = n < a.N;
        float st[SCV];
        const float* enter = nullptr;
        if (seg == 0)
            enter = a.S0 ? a.S0 + bh * PN : nullptr;
        else if (OUT)
            enter = a.seg_state + (bh * (a.nseg - 1) + seg - 1) * PN;
#pragma unroll
        for (int p = 0; p < SCV; ++p)
            st[p] = enter && row && p < pv ? enter[(long)(v0 + p) * a.N + n] : 0.f;
        uint8_t* srow = sm + SC_S + n * 128;
        auto copy = [&]() {
            if (OUT) {
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    *reinterpret_cast<uint4*>(srow + ((k ^ (n & 7)) << 4)) =
                        Vec16<__nv_bfloat16>::pack(st + 8 * k);
                fence_async_smem();
            }
            mbar_arrive(bar(SB_ST));
        };
        copy();
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1;
            if (!mbar_wait(bar(SB_FULL + s), (uint32_t)((c >> 1) & 1), abort_flag)) break;
            const float gamma = par(s)->gamma;
            if (!mbar_wait(bar(SB_DS), (uint32_t)(c & 1), abort_flag)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 0; p < SCV; p += 16) {
                float hi[16], lo[16];
                tmem_ld16(trow + TC_DS + p, hi);
                tmem_ld16(trow + TC_DS + SCV + p, lo);
                tmem_wait_ld();
#pragma unroll
                for (int k = 0; k < 16; ++k) st[p + k] = fmaf(gamma, st[p + k], hi[k] + lo[k]);
            }
            tc_fence_before();
            if (c + 1 < nc) copy();  // the inter product has read the old copy before SB_DS
            release(s);
        }
        float* leave = !OUT ? a.seg_state + (bh * (a.nseg - 1) + seg) * PN
                       : seg == a.nseg - 1 && a.S_final ? a.S_final + bh * PN
                                                        : nullptr;
        if (leave && row) {
#pragma unroll
            for (int p = 0; p < SCV; ++p)
                if (p < pv) leave[(long)(v0 + p) * a.N + n] = st[p];
        }
    } else if (OUT) {
        // ------------------------------------------------------------------ outputs
        const int i = tid - 384;
        const float Dh = a.D ? a.D[h] : 0.f;
        __nv_bfloat16* op = static_cast<__nv_bfloat16*>(a.out) + b * a.osb + h * a.osh + v0;
        for (int c = 0; c < nc; ++c) {
            const int s = c & 1, nv = valid(c);
            if (!mbar_wait(bar(SB_FULL + s), (uint32_t)((c >> 1) & 1), abort_flag)) break;
            const float eg = par(s)->eg[i];
            uint8_t* xt = stage(s) + SC_X;
            uint8_t* xr = xt + i * 128;
            if (!mbar_wait(bar(SB_Y), (uint32_t)(c & 1), abort_flag)) break;
            tc_fence_after();
#pragma unroll
            for (int p = 0; p < SCV; p += 32) {
                float in[32], it[32];
                tmem_ld16(trow + TC_INTRA + p, in);
                tmem_ld16(trow + TC_INTRA + p + 16, in + 16);
                tmem_ld16(trow + TC_INTER + p, it);
                tmem_ld16(trow + TC_INTER + p + 16, it + 16);
                tmem_wait_ld();
                if (p + 32 >= SCV) {
                    tc_fence_before();
                    mbar_arrive(bar(SB_YFREE));
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint4* at = reinterpret_cast<uint4*>(xr + (((p / 8 + k) ^ (i & 7)) << 4));
                    float x[8];
                    Vec16<__nv_bfloat16>::unpack(*at, x);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        x[e] = fmaf(Dh, x[e], fmaf(eg, it[8 * k + e], in[8 * k + e]));
                    *at = Vec16<__nv_bfloat16>::pack(x);  // over x, which no one else reads now
                }
            }
            __syncwarp();
            // the warp's 32 rows, four at a time, eight lanes of 16 bytes each
            const int w0 = (warp & 3) * 32, k = lane & 7;
#pragma unroll
            for (int r = 0; r < 32; r += 4) {
                const int ii = w0 + r + (lane >> 3);
                const uint4 y = *reinterpret_cast<const uint4*>(xt + ii * 128 + ((k ^ (ii & 7)) << 4));
                if (ii < nv && 8 * k < pv)
                    *reinterpret_cast<uint4*>(op + ((long)t0 + c * SCK + ii) * a.ost + 8 * k) = y;
            }
            release(s);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 17) tmem_dealloc(tmem, 512);
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

// Segments of a chunked scan: the count with the least time by the model below, in units of one
// chunk with outputs; one without costs SC_STATES_COST, the two more launches SC_LAUNCHES.
constexpr float SC_STATES_COST = 0.5f;
constexpr float SC_LAUNCHES = 5.f;

inline void plan_ssm_chunked(SsmArgs* a, int sms) {
    const long ctas = (long)a->B * a->H * ((a->P + SCV - 1) / SCV);
    const int nc = (int)(((long)a->T + SCK - 1) / SCK);
    float best = (float)((ctas + sms - 1) / sms) * nc;
    int len = nc;
    const int most = (int)(nc < 4l * sms / ctas ? nc : 4l * sms / ctas);
    for (int n = 2; n <= most; ++n) {
        const int l = (nc + n - 1) / n, m = (nc + l - 1) / l;
        const float t = (float)((ctas * m + sms - 1) / sms) * l +
                        SC_STATES_COST * (float)((ctas * (m - 1) + sms - 1) / sms) * l + SC_LAUNCHES;
        if (t < best) best = t, len = l;
    }
    a->seg_len = len * SCK;
    a->nseg = (nc + len - 1) / len;
}

template <int PASS>
int launch_ssm_chunked_pass(const CUtensorMap& mx, const CUtensorMap& mb, const CUtensorMap& mc,
                            const SsmChunkArgs& ca, long gx, int gy, cudaStream_t stream) {
    const int smem = SC_TOTAL + 1024;
    auto kern = ssm_chunked_kernel<PASS>;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
        cudaSuccess)
        return DR_ERR_CUDA;
    kern<<<dim3((unsigned)gx, (unsigned)gy), SC_THREADS, smem, stream>>>(mx, mb, mc, ca);
    return cudaGetLastError() == cudaSuccess ? DR_OK : DR_ERR_CUDA;
}

// The planned passes (a.nseg, a.seg_len and the scratch set).
inline int launch_ssm_chunked(const SsmArgs& a, cudaStream_t stream) {
    SsmChunkArgs ca;
    ca.s = a;
    CUtensorMap mx, mb, mc;
    if (!ssm_map(&mx, a.x, a.P, a.T, a.H, a.B, &ca.xh, &ca.xb) ||
        !ssm_map(&mb, a.Bm, a.N, a.T, a.G, a.B, &ca.bh, &ca.bb) ||
        !ssm_map(&mc, a.Cm, a.N, a.T, a.G, a.B, &ca.ch, &ca.cb))
        return DR_ERR_CUDA;
    const long gx = (long)a.B * a.H * ((a.P + SCV - 1) / SCV);
    if (gx > 0x7fffffffl || a.nseg > 65535) return DR_ERR_UNSUPPORTED;
    if (a.nseg > 1) {
        int rc = launch_ssm_chunked_pass<SSM_PASS_STATES>(mx, mb, mc, ca, gx, a.nseg - 1, stream);
        if (rc == DR_OK) rc = launch_ssm_chain(a, stream);
        if (rc != DR_OK) return rc;
    }
    return launch_ssm_chunked_pass<SSM_PASS_OUTPUTS>(mx, mb, mc, ca, gx, a.nseg, stream);
}

}  // namespace drscan
