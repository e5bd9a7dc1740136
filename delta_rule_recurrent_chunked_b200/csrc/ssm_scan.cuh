// Selective state space scan, per token, fp32 state on CUDA cores (any input type), and the
// one-token step.
//
// Per head, with delta_t = dt_t (+ bias, through softplus) and a_t = exp(delta_t A):
//     S_t = a_t S_{t-1} + delta_t x_t B_t^T          S in R^{P x N}
//     y_t = S_t C_t + D x_t
// B and C are shared by the H / G heads of a group. It is the gated scan of this library
// without the delta rule's correction: decay, write delta x along B, read with C.
//
// The rows of S are independent given (a, delta, B, C). Eight neighbouring lanes hold two rows,
// N / 8 elements of each per lane in registers (elements 32 i + 4 q + 0..3 of lane q, so that the
// eight lanes' 16-byte reads of B and C from shared memory are one conflict-free access), a CTA
// of 128 threads 32 rows. A token costs a thread 3 N / 8 two-element FMA-type instructions, N / 16
// reads and three shuffles for the readout. Bound: those reads (4 cycles each per warp and SM; with
// one row per thread they took twice the time: 301 tokens of 128-element rows 79 us), or, with few
// rows, the latency of the chain of tokens; the entry point then cuts the tokens into segments. (2 x
// 4 ragged heads of 32 x 32 and 301 tokens, fp32: 12 us on the device in 10 segments.) Where the
// kernel and not its launches sets the time, fp32, heads of 128 x 128: 16 heads, 4096 tokens 306 us
// (floor 11), 8 x 16 heads 1817 us (90): 27 and 37 rows of S and tokens in a nanosecond.
//
// Segments (exact): the recurrence is affine in the state it enters with, S_out = (prod a) S_in
// + S_zero. A first launch runs every segment but the last from zero (the first from S0)
// without outputs, a second chains S_out over the segments, a third runs all of them from their
// entering states with outputs.
#pragma once

#include "dr_sequential.cuh"
#include "layer_common.cuh"

namespace drscan {

// Element strides of batch, head and token; channels are contiguous.
struct SsmView {
    const void* p;
    long sb, sh, st;
};

struct SsmArgs {
    SsmView x, dt, Bm, Cm;
    const float *A, *D, *dt_bias, *S0;
    const int* lengths;
    void* out;
    long osb, osh, ost;
    float* S_final;
    int B, H, G, T, P, N;
    bool softplus, dt_bf16;
    // segments: nseg per head of seg_len tokens each; seg_state [B,H,nseg-1,P,N] their end
    // states, seg_log [B,H,nseg-1] the logarithms of their decays
    int nseg, seg_len;
    float *seg_state, *seg_log;
};

// Whether a launch of a segmented scan writes the segments' end states (no outputs) or runs
// them from their entering states (all outputs).
enum { SSM_PASS_STATES = 0, SSM_PASS_OUTPUTS = 1 };

// dt of a token, and the step delta it makes.
__device__ __forceinline__ float ssm_dt(const SsmArgs& a, long b, int h, long t) {
    const long o = b * a.dt.sb + h * a.dt.sh + t * a.dt.st;
    return a.dt_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.dt.p)[o])
                     : static_cast<const float*>(a.dt.p)[o];
}

__device__ __forceinline__ float ssm_delta(const SsmArgs& a, int h, float dt) {
    const float d = a.dt_bias ? dt + a.dt_bias[h] : dt;
    return a.softplus ? softplus_f32(d) : d;
}

constexpr int SSM_TILE = 16;     // tokens staged in shared memory at a time (32: more registers in
                                 // flight than a third CTA per SM is worth)
constexpr int SSM_ROWS = 32;     // rows of S per CTA
constexpr int SSM_THREADS = 128;
constexpr int SSM_STEPS = SSM_THREADS;  // tokens whose steps and decays are made at a time, one a
                                        // thread (a tile's alone would take as long as its scan)

// grid: (B * H * (P / SSM_ROWS), segments of this pass); block: SSM_THREADS.
template <typename T, int N, int PASS>
__global__ void __launch_bounds__(SSM_THREADS) ssm_sequential_kernel(
    const __grid_constant__ SsmArgs a) {
    constexpr int EPT = N / 8;
    constexpr int VEC = Vec16<T>::N;
    __shared__ __align__(16) float sB[SSM_TILE][N];
    __shared__ __align__(16) float sC[PASS == SSM_PASS_OUTPUTS ? SSM_TILE : 1][N];
    __shared__ float sx[SSM_TILE][SSM_ROWS + 1];
    __shared__ float sy[PASS == SSM_PASS_OUTPUTS ? SSM_TILE : 1][SSM_ROWS + 1];
    __shared__ float sdelta[SSM_STEPS], sa[SSM_STEPS];

    const int tid = threadIdx.x, q = tid & 7, r = 2 * (tid >> 3);  // rows r and r + 1
    const int nrb = a.P / SSM_ROWS;
    const int rb = (int)(blockIdx.x % nrb);
    const long bh = blockIdx.x / nrb;
    const long b = bh / a.H;
    const int h = (int)(bh % a.H), g = h / (a.H / a.G);
    const int seg = (int)blockIdx.y;
    const int p0 = rb * SSM_ROWS;
    const long PN = (long)a.P * N;
    const long so = (long)(p0 + r) * N;  // this row within a state
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int t0 = seg * a.seg_len;  // below T: the entry point rounds nseg to what T needs
    const int t1 = min(len, t0 + min(a.seg_len, a.T - t0));

    float2 s[2][EPT / 2];
    const float* enter = nullptr;
    if (seg == 0)
        enter = a.S0 ? a.S0 + bh * PN + so : nullptr;
    else if (PASS == SSM_PASS_OUTPUTS)
        enter = a.seg_state + (bh * (a.nseg - 1) + seg - 1) * PN + so;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < EPT; i += 4) {
            const float4 v =
                enter ? *reinterpret_cast<const float4*>(enter + k * N + 8 * i + 4 * q)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
            s[k][i / 2] = make_float2(v.x, v.y), s[k][i / 2 + 1] = make_float2(v.z, v.w);
        }
    const float Ah = a.A[h], Dh = a.D ? a.D[h] : 0.f;
    const T* xp = static_cast<const T*>(a.x.p) + b * a.x.sb + h * a.x.sh + p0;
    const T* bp = static_cast<const T*>(a.Bm.p) + b * a.Bm.sb + g * a.Bm.sh;
    const T* cp = static_cast<const T*>(a.Cm.p) + b * a.Cm.sb + g * a.Cm.sh;
    T* op = static_cast<T*>(a.out) + b * a.osb + h * a.osh + p0;
    float logsum = 0.f;

    // a tile's loads wait in registers while the tile before is scanned
    constexpr int NV = (SSM_TILE * (N / VEC) + SSM_THREADS - 1) / SSM_THREADS;  // pieces of B and C
    constexpr int NX = (SSM_TILE * (SSM_ROWS / VEC) + SSM_THREADS - 1) / SSM_THREADS;
    uint4 nextB[NV], nextC[NV], nextx[NX];
    auto fetch = [&](int tt) {
        const int n = min(SSM_TILE, t1 - tt);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = tid + k * SSM_THREADS, t = e / (N / VEC), c = (e % (N / VEC)) * VEC;
            if (t < n) {
                nextB[k] = *reinterpret_cast<const uint4*>(bp + (long)(tt + t) * a.Bm.st + c);
                if constexpr (PASS == SSM_PASS_OUTPUTS)
                    nextC[k] = *reinterpret_cast<const uint4*>(cp + (long)(tt + t) * a.Cm.st + c);
            }
        }
#pragma unroll
        for (int k = 0; k < NX; ++k) {
            const int e = tid + k * SSM_THREADS;
            const int t = e / (SSM_ROWS / VEC), c = (e % (SSM_ROWS / VEC)) * VEC;
            if (t < n) nextx[k] = *reinterpret_cast<const uint4*>(xp + (long)(tt + t) * a.x.st + c);
        }
    };
    if (t0 < t1) fetch(t0);
    for (int tt = t0; tt < t1; tt += SSM_TILE) {
        const int n = min(SSM_TILE, t1 - tt);
        __syncthreads();  // the previous tile's readers are done
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int e = tid + k * SSM_THREADS, t = e / (N / VEC), c = (e % (N / VEC)) * VEC;
            if (t < n) {
                Vec16<T>::unpack(nextB[k], &sB[t][c]);
                if constexpr (PASS == SSM_PASS_OUTPUTS) Vec16<T>::unpack(nextC[k], &sC[t][c]);
            }
        }
#pragma unroll
        for (int k = 0; k < NX; ++k) {
            const int e = tid + k * SSM_THREADS;
            const int t = e / (SSM_ROWS / VEC), c = (e % (SSM_ROWS / VEC)) * VEC;
            if (t < n) {
                float v[VEC];
                Vec16<T>::unpack(nextx[k], v);
#pragma unroll
                for (int i = 0; i < VEC; ++i) sx[t][c + i] = v[i];
            }
        }
        const int step0 = (tt - t0) & (SSM_STEPS - 1);
        if (step0 == 0 && tt + tid < t1) {
            const float d = ssm_delta(a, h, ssm_dt(a, b, h, tt + tid));
            sdelta[tid] = d;
            sa[tid] = decay_f32(d * Ah);
            logsum += d * Ah;
        }
        if (tt + SSM_TILE < t1) fetch(tt + SSM_TILE);
        __syncthreads();
        // one token: the rows' new states, and this lane's part of their readouts
        auto token = [&](int t, float2* y) {
            const float at = sa[step0 + t], d = sdelta[step0 + t];
            const float2 a2 = make_float2(at, at);
            const float u[2] = {d * sx[t][r], d * sx[t][r + 1]};
            y[0] = y[1] = make_float2(0.f, 0.f);
#pragma unroll
            for (int i = 0; i < EPT; i += 4) {
                const float4 bv = *reinterpret_cast<const float4*>(&sB[t][8 * i + 4 * q]);
                float4 cv;
                if constexpr (PASS == SSM_PASS_OUTPUTS)
                    cv = *reinterpret_cast<const float4*>(&sC[t][8 * i + 4 * q]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 u2 = make_float2(u[k], u[k]);
                    float2& s0 = s[k][i / 2];
                    float2& s1 = s[k][i / 2 + 1];
                    s0 = fma2(a2, s0, mul2(u2, make_float2(bv.x, bv.y)));
                    s1 = fma2(a2, s1, mul2(u2, make_float2(bv.z, bv.w)));
                    if constexpr (PASS == SSM_PASS_OUTPUTS) {
                        y[k] = fma2(s0, make_float2(cv.x, cv.y), y[k]);
                        y[k] = fma2(s1, make_float2(cv.z, cv.w), y[k]);
                    }
                }
            }
        };
        // the parts of M tokens added up, their shuffles side by side; lanes 0-3 go on with the
        // first row, lanes 4-7 with the second
        auto readout = [&](int t, const float2 (*y)[2], auto count) {
            constexpr int M = decltype(count)::value;
            const bool second = q & 4;
            const int row = r + (q >> 2);
            float v[M];
#pragma unroll
            for (int m = 0; m < M; ++m) {
                const float f0 = y[m][0].x + y[m][0].y, f1 = y[m][1].x + y[m][1].y;
                v[m] = (second ? f1 : f0) + __shfl_xor_sync(0xffffffffu, second ? f0 : f1, 4);
            }
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], 2);
#pragma unroll
            for (int m = 0; m < M; ++m) v[m] += __shfl_xor_sync(0xffffffffu, v[m], 1);
            if ((q & 3) == 0) {
#pragma unroll
                for (int m = 0; m < M; ++m) sy[t + m][row] = fmaf(Dh, sx[t + m][row], v[m]);
            }
        };
        int t = 0;
        for (; t + 4 <= n; t += 4) {
            float2 y[4][2];
#pragma unroll
            for (int m = 0; m < 4; ++m) token(t + m, y[m]);
            if constexpr (PASS == SSM_PASS_OUTPUTS)
                readout(t, y, std::integral_constant<int, 4>());
        }
        for (; t < n; ++t) {
            float2 y[1][2];
            token(t, y[0]);
            if constexpr (PASS == SSM_PASS_OUTPUTS)
                readout(t, y, std::integral_constant<int, 1>());
        }
        if constexpr (PASS == SSM_PASS_OUTPUTS) {
            __syncthreads();
            for (int e = tid; e < n * (SSM_ROWS / VEC); e += SSM_THREADS) {
                const int t = e / (SSM_ROWS / VEC), c = (e % (SSM_ROWS / VEC)) * VEC;
                float v[VEC];
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[i] = sy[t][c + i];
                *reinterpret_cast<uint4*>(op + (long)(tt + t) * a.ost + c) = Vec16<T>::pack(v);
            }
        }
    }

    float* leave = nullptr;
    if (PASS == SSM_PASS_STATES) {
        leave = a.seg_state + (bh * (a.nseg - 1) + seg) * PN + so;
        if (rb == 0) {  // the threads' sums, in a fixed order
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                logsum += __shfl_xor_sync(0xffffffffu, logsum, off);
            __syncthreads();
            if ((tid & 31) == 0) sdelta[tid >> 5] = logsum;
            __syncthreads();
            if (tid == 0)
                a.seg_log[bh * (a.nseg - 1) + seg] =
                    (sdelta[0] + sdelta[1]) + (sdelta[2] + sdelta[3]);
        }
    } else if (seg == a.nseg - 1 && a.S_final) {
        leave = a.S_final + bh * PN + so;
    }
    if (leave) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < EPT; i += 4)
                *reinterpret_cast<float4*>(leave + k * N + 8 * i + 4 * q) =
                    make_float4(s[k][i / 2].x, s[k][i / 2].y, s[k][i / 2 + 1].x,
                                s[k][i / 2 + 1].y);
    }
}

// Chains the segments' end states in place: state s becomes the true one at the end of segment
// s. A thread per state element, eight segments' loads in flight; grid: B * H * P * N / block.
__global__ void __launch_bounds__(256) ssm_chain_kernel(float* state, const float* logs, long BH,
                                                        int nst, long PN) {
    const long e = blockIdx.x * 256l + threadIdx.x;
    if (e >= BH * PN) return;
    const long bh = e / PN;
    float* p = state + bh * nst * PN + e % PN;
    const float* lg = logs + bh * nst;
    float run = p[0];
    for (int s = 1; s < nst; s += 8) {
        float v[8], a[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = s + k < nst ? p[(s + k) * PN] : 0.f;
            a[k] = s + k < nst ? decay_f32(lg[s + k]) : 0.f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (s + k < nst) {
                run = fmaf(a[k], run, v[k]);
                p[(s + k) * PN] = run;
            }
    }
}

inline int launch_ssm_chain(const SsmArgs& a, cudaStream_t stream) {
    const long PN = (long)a.P * a.N, n = (long)a.B * a.H * PN;
    ssm_chain_kernel<<<(unsigned)((n + 255) / 256), 256, 0, stream>>>(
        a.seg_state, a.seg_log, (long)a.B * a.H, a.nseg - 1, PN);
    return cudaGetLastError() == cudaSuccess ? DR_OK : DR_ERR_CUDA;
}

// One token on a resident state: S is read and written once, which bounds the step (8 P N bytes
// a head). A row of S is N / 4 lanes of 16 bytes, so a warp's access covers 128 / N rows in one
// 512-byte piece; each warp owns SSM_STEP_U such pieces, all loaded before the first is used. 128
// sequences of 32 heads of 128 x 128 (539 MB): 87 us, 96% of the measured copy rate.
constexpr int SSM_STEP_U = 4;
constexpr int SSM_STEP_WARPS = 4;

template <typename T>
__device__ __forceinline__ float4 ld4(const T* p);
template <>
__device__ __forceinline__ float4 ld4<float>(const float* p) {
    return *reinterpret_cast<const float4*>(p);
}
template <>
__device__ __forceinline__ float4 ld4<__nv_bfloat16>(const __nv_bfloat16* p) {
    const uint2 r = *reinterpret_cast<const uint2*>(p);
    return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                       __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}

// grid: B * H * P rows over the rows of a CTA; block: 32 * SSM_STEP_WARPS.
template <typename T, int N>
__global__ void __launch_bounds__(32 * SSM_STEP_WARPS) ssm_step_kernel(
    const __grid_constant__ SsmArgs a, float* __restrict__ S) {
    constexpr int LPR = N / 4;        // lanes per row
    constexpr int RPA = 32 / LPR;     // rows per access
    constexpr int RPW = RPA * SSM_STEP_U;  // rows per warp (4, 8 or 16: one head)
    const int lane = threadIdx.x & 31;
    const long w = (long)blockIdx.x * SSM_STEP_WARPS + (threadIdx.x >> 5);
    const long row0 = w * RPW;
    if (row0 >= (long)a.B * a.H * a.P) return;
    float* sp = S + row0 * N + lane * 4;
    float4 s[SSM_STEP_U];
#pragma unroll
    for (int u = 0; u < SSM_STEP_U; ++u)
        s[u] = *reinterpret_cast<const float4*>(sp + u * 128);
    const long bh = row0 / a.P, b = bh / a.H;
    const int p0 = (int)(row0 % a.P), h = (int)(bh % a.H), g = h / (a.H / a.G);
    const int c = (lane % LPR) * 4, sub = lane / LPR;
    const float4 bv = ld4(static_cast<const T*>(a.Bm.p) + b * a.Bm.sb + g * a.Bm.sh + c);
    const float4 cv = ld4(static_cast<const T*>(a.Cm.p) + b * a.Cm.sb + g * a.Cm.sh + c);
    const T* xp = static_cast<const T*>(a.x.p) + b * a.x.sb + h * a.x.sh + p0 + sub;
    float x[SSM_STEP_U];
#pragma unroll
    for (int u = 0; u < SSM_STEP_U; ++u) x[u] = to_f32<T>(xp[u * RPA]);
    const float delta = ssm_delta(a, h, ssm_dt(a, b, h, 0));
    const float at = decay_f32(delta * a.A[h]), Dh = a.D ? a.D[h] : 0.f;
    T* op = static_cast<T*>(a.out) + b * a.osb + h * a.osh + p0 + sub;
#pragma unroll
    for (int u = 0; u < SSM_STEP_U; ++u) {
        const float dx = delta * x[u];
        float4 v = s[u];
        v.x = fmaf(at, v.x, dx * bv.x), v.y = fmaf(at, v.y, dx * bv.y);
        v.z = fmaf(at, v.z, dx * bv.z), v.w = fmaf(at, v.w, dx * bv.w);
        *reinterpret_cast<float4*>(sp + u * 128) = v;
        float y = fmaf(v.x, cv.x, fmaf(v.y, cv.y, fmaf(v.z, cv.z, v.w * cv.w)));
#pragma unroll
        for (int off = LPR / 2; off > 0; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (lane % LPR == 0) op[u * RPA] = from_f32<T>(fmaf(Dh, x[u], y));
    }
}

}  // namespace drscan
