// Selective state space scan, per token, fp32 state on CUDA cores (any input type), and the
// one-token step.
//
// Per head, with delta_t = dt_t (+ bias, through softplus) and a_t = exp(delta_t A):
//     S_t = a_t S_{t-1} + delta_t x_t B_t^T          S in R^{P x N}
//     y_t = S_t C_t + D x_t
// B and C are shared by the H / G heads of a group. It is the gated scan of this library
// without the delta rule's correction: decay, write delta x along B, read with C.
//
// The rows of S are independent given (a, delta, B, C). Four neighbouring lanes hold one row,
// N / 4 elements each in registers (elements 16 i + 4 q + 0..3 of lane q, so that the four
// lanes' 16-byte reads of B and C from shared memory are one conflict-free 64-byte access), a
// CTA of 128 threads 32 rows. A token costs 3 N / 4 FMA-type instructions per thread and two
// shuffles for the readout. Bound: FMA issue (3 P N per head and token), or, with few rows, the
// latency of the chain of tokens; the entry point then cuts the tokens into segments.
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

constexpr int SSM_TILE = 32;     // tokens staged in shared memory at a time
constexpr int SSM_ROWS = 32;     // rows of S per CTA
constexpr int SSM_THREADS = 128;

// grid: (B * H * (P / SSM_ROWS), segments of this pass); block: SSM_THREADS.
template <typename T, int N, int PASS>
__global__ void __launch_bounds__(SSM_THREADS) ssm_sequential_kernel(
    const __grid_constant__ SsmArgs a) {
    constexpr int EPT = N / 4;
    constexpr int VEC = Vec16<T>::N;
    __shared__ __align__(16) float sB[SSM_TILE][N];
    __shared__ __align__(16) float sC[PASS == SSM_PASS_OUTPUTS ? SSM_TILE : 1][N];
    __shared__ float sx[SSM_TILE][SSM_ROWS + 1];
    __shared__ float sy[PASS == SSM_PASS_OUTPUTS ? SSM_TILE : 1][SSM_ROWS + 1];
    __shared__ float sdelta[SSM_TILE], sa[SSM_TILE];

    const int tid = threadIdx.x, q = tid & 3, r = tid >> 2;
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

    float s[EPT];
    const float* enter = nullptr;
    if (seg == 0)
        enter = a.S0 ? a.S0 + bh * PN + so : nullptr;
    else if (PASS == SSM_PASS_OUTPUTS)
        enter = a.seg_state + (bh * (a.nseg - 1) + seg - 1) * PN + so;
#pragma unroll
    for (int i = 0; i < EPT; i += 4) {
        const float4 v = enter ? *reinterpret_cast<const float4*>(enter + 4 * i + 4 * q)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
        s[i] = v.x, s[i + 1] = v.y, s[i + 2] = v.z, s[i + 3] = v.w;
    }
    const float Ah = a.A[h], Dh = a.D ? a.D[h] : 0.f;
    const T* xp = static_cast<const T*>(a.x.p) + b * a.x.sb + h * a.x.sh + p0;
    const T* bp = static_cast<const T*>(a.Bm.p) + b * a.Bm.sb + g * a.Bm.sh;
    const T* cp = static_cast<const T*>(a.Cm.p) + b * a.Cm.sb + g * a.Cm.sh;
    T* op = static_cast<T*>(a.out) + b * a.osb + h * a.osh + p0;
    float logsum = 0.f;

    for (int tt = t0; tt < t1; tt += SSM_TILE) {
        const int n = min(SSM_TILE, t1 - tt);
        __syncthreads();  // the previous tile's readers are done
        for (int e = tid; e < n * (N / VEC); e += SSM_THREADS) {
            const int t = e / (N / VEC), c = (e % (N / VEC)) * VEC;
            Vec16<T>::unpack(*reinterpret_cast<const uint4*>(bp + (long)(tt + t) * a.Bm.st + c),
                             &sB[t][c]);
            if constexpr (PASS == SSM_PASS_OUTPUTS)
                Vec16<T>::unpack(
                    *reinterpret_cast<const uint4*>(cp + (long)(tt + t) * a.Cm.st + c), &sC[t][c]);
        }
        for (int e = tid; e < n * (SSM_ROWS / VEC); e += SSM_THREADS) {
            const int t = e / (SSM_ROWS / VEC), c = (e % (SSM_ROWS / VEC)) * VEC;
            float v[VEC];
            Vec16<T>::unpack(*reinterpret_cast<const uint4*>(xp + (long)(tt + t) * a.x.st + c), v);
#pragma unroll
            for (int i = 0; i < VEC; ++i) sx[t][c + i] = v[i];
        }
        if (tid < n) {
            const float d = ssm_delta(a, h, ssm_dt(a, b, h, tt + tid));
            sdelta[tid] = d;
            sa[tid] = decay_f32(d * Ah);
            logsum += d * Ah;
        }
        __syncthreads();
#pragma unroll 4
        for (int t = 0; t < n; ++t) {
            const float at = sa[t], u = sdelta[t] * sx[t][r];
            float y = 0.f;
#pragma unroll
            for (int i = 0; i < EPT; i += 4) {
                const float4 bv = *reinterpret_cast<const float4*>(&sB[t][4 * i + 4 * q]);
                s[i] = fmaf(at, s[i], u * bv.x);
                s[i + 1] = fmaf(at, s[i + 1], u * bv.y);
                s[i + 2] = fmaf(at, s[i + 2], u * bv.z);
                s[i + 3] = fmaf(at, s[i + 3], u * bv.w);
                if constexpr (PASS == SSM_PASS_OUTPUTS) {
                    const float4 cv = *reinterpret_cast<const float4*>(&sC[t][4 * i + 4 * q]);
                    y = fmaf(s[i], cv.x, y);
                    y = fmaf(s[i + 1], cv.y, y);
                    y = fmaf(s[i + 2], cv.z, y);
                    y = fmaf(s[i + 3], cv.w, y);
                }
            }
            if constexpr (PASS == SSM_PASS_OUTPUTS) {
                y += __shfl_xor_sync(0xffffffffu, y, 1);
                y += __shfl_xor_sync(0xffffffffu, y, 2);
                if (q == 0) sy[t][r] = fmaf(Dh, sx[t][r], y);
            }
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
        if (rb == 0 && tid < 32) {  // the tile's tokens are lanes of the first warp
#pragma unroll
            for (int off = 16; off > 0; off >>= 1)
                logsum += __shfl_xor_sync(0xffffffffu, logsum, off);
            if (tid == 0) a.seg_log[bh * (a.nseg - 1) + seg] = logsum;
        }
    } else if (seg == a.nseg - 1 && a.S_final) {
        leave = a.S_final + bh * PN + so;
    }
    if (leave) {
#pragma unroll
        for (int i = 0; i < EPT; i += 4)
            *reinterpret_cast<float4*>(leave + 4 * i + 4 * q) =
                make_float4(s[i], s[i + 1], s[i + 2], s[i + 3]);
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
// 512-byte piece; each warp owns SSM_STEP_U such pieces, all loaded before the first is used.
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
