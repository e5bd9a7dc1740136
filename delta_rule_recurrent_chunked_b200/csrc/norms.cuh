// RMS norms around a block.
//
// gated_norm, after a scan: over groups of neighbouring heads of a token, W = heads * d wide,
//     gate after:  out = y rsqrt(mean y^2 + eps) weight act(gate)
//     gate first:  v = y act(gate),  out = v rsqrt(mean v^2 + eps) weight
// y comes head-major or in any layout with contiguous channels; gate and out are rows of a
// token, [B, T, H d], as projections leave and read them.
//
// block_norm, between two blocks:
//     z = x, or x rsqrt(mean x^2 + eps) post_weight       the norm after a block
//     r = residual + scale z                              scale: a number or one per channel
//     out = r rsqrt(mean r^2 + eps) weight                the norm before the next block
//
// Bound: HBM; every tensor passes once. A row (group) is held in the registers of TPG threads,
// VPT 16-byte vectors each: the statistics are taken from the registers, the means in fp32.
// TPG = 4..32 lanes of a warp (several rows per warp, shuffles only), or 128..512 threads of a
// CTA (shuffles and one exchange through shared memory).
//
// Measured: gated_norm of 16 heads of 128 for 8 x 4096 tokens (bf16, silu, 403 MB) 80 us, 78% of the
// measured copy rate: issue slots 61% and special functions 45% busy on 20 warps per SM. block_norm
// of 32768 rows of 2048 (bf16 x, fp32 residual, 805 MB) 121 us, the copy rate (103%). For one token
// the host's call takes longer than the kernel: 128 sequences of 32 heads of 64 (fp32) 3.3 of 14 us,
// 128 rows of 4096 4.5 of 16.
#pragma once

#include "layer_common.cuh"

namespace drscan {

constexpr int NORM_BLOCK = 128;  // threads of a CTA that holds several rows

// Sum over the TPG threads of a row, in a fixed order.
template <int TPG>
__device__ __forceinline__ float row_sum(float v, float* smem) {
#pragma unroll
    for (int off = (TPG < 32 ? TPG : 32) / 2; off > 0; off >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, off);
    if constexpr (TPG > 32) {
        const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
        if (lane == 0) smem[warp] = v;
        __syncthreads();
        v = lane < TPG / 32 ? smem[lane] : 0.f;
#pragma unroll
        for (int off = TPG / 64; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        v = __shfl_sync(0xffffffffu, v, 0);
        __syncthreads();  // smem may be written again
    }
    return v;
}

// Division of 31-bit numbers by one known at launch: multiply by the upper bits of its reciprocal
// (Granlund and Montgomery 1994).
struct DivBy {
    unsigned d, mul, shift;
    DivBy() = default;
    explicit DivBy(unsigned d_) : d(d_), mul(0), shift(0) {
        while ((1ull << shift) < d) ++shift;
        mul = (unsigned)(((1ull << 32) * ((1ull << shift) - d)) / d + 1);
    }
    __device__ __forceinline__ unsigned operator()(unsigned n) const {
        return (__umulhi(n, mul) + n) >> shift;
    }
};

struct GatedNormArgs {
    const void* y;
    long ysb, ysh, yst;
    const void* gate;  // NULL: no gate
    long gsb, gst;
    const float* weight;
    void* out;
    long osb, ost;
    float eps, inv_w;   // 1 / (heads d)
    DivBy by_groups, by_T;
    int B, H, T, d;
    int heads;          // of a group
    int shared_weight;  // weight has d values, the same for every head (else H d)
    int sigmoid;        // act = sigmoid (else silu)
    int gate_first;
};

// block: NORM_BLOCK threads (TPG <= 32) or TPG; grid: rows * groups over the block's groups, R
// items each (all their loads before the first use: one 16-byte vector of y and of the gate in
// flight per thread does not cover the latency of HBM).
template <typename T, int TPG, int VPT, int R>
__global__ void __launch_bounds__(TPG <= 32 ? NORM_BLOCK : TPG) gated_norm_kernel(
    const __grid_constant__ GatedNormArgs a) {
    constexpr int VEC = Vec16<T>::N;
    constexpr int GPB = TPG <= 32 ? NORM_BLOCK / TPG : 1;
    __shared__ float smem[32];
    const unsigned ngr = a.H / a.heads;
    const unsigned total = (unsigned)a.B * a.T * ngr;  // below 2^31, as the entry point checks
    const int W = a.heads * a.d, nv = W / VEC, lt = threadIdx.x % TPG;
    const int dshift = __ffs(a.d) - 1;  // d is a power of two
    const T* gate = static_cast<const T*>(a.gate);

    uint4 yr[R][VPT], gr[R][VPT];
    T* op[R];
    unsigned gi[R];
    bool live[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const unsigned item = (blockIdx.x * R + r) * GPB + threadIdx.x / TPG;
        live[r] = item < total;
        const unsigned it = live[r] ? item : total - 1;  // an idle group repeats the last item
        const unsigned bt = a.by_groups(it), g = it - bt * ngr, ub = a.by_T(bt);
        const long b = ub, t = bt - ub * a.T;
        const T* yp =
            static_cast<const T*>(a.y) + b * a.ysb + t * a.yst + (long)g * a.heads * a.ysh;
        const T* gp = gate + b * a.gsb + t * a.gst + (long)g * W;
        op[r] = static_cast<T*>(a.out) + b * a.osb + t * a.ost + (long)g * W;
        gi[r] = g;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lt + i * TPG;
            yr[r][i] = gr[r][i] = make_uint4(0, 0, 0, 0);
            if (v < nv) {
                const int e = v * VEC, hh = e >> dshift;
                yr[r][i] = *reinterpret_cast<const uint4*>(yp + hh * a.ysh + (e & (a.d - 1)));
                if (gate) gr[r][i] = *reinterpret_cast<const uint4*>(gp + e);
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
        float2 y[VPT][VEC / 2], act[VPT][VEC / 2], ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            Vec16<T>::unpack(yr[r][i], reinterpret_cast<float*>(y[i]));
            if (gate) {
                Vec16<T>::unpack(gr[r][i], reinterpret_cast<float*>(act[i]));
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) {
                    const float2 s = sigmoid2(act[i][j]);
                    act[i][j] = a.sigmoid ? s : mul2(act[i][j], s);
                }
                if (a.gate_first) {
#pragma unroll
                    for (int j = 0; j < VEC / 2; ++j) y[i][j] = mul2(y[i][j], act[i][j]);
                }
            }
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) ss = fma2(y[i][j], y[i][j], ss);
        }
        const float rs = rsqrtf(fmaf(row_sum<TPG>(ss.x + ss.y, smem), a.inv_w, a.eps));
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = lt + i * TPG;
            if (!live[r] || v >= nv) continue;
            const int e = v * VEC;
            const float* wp = a.weight + (a.shared_weight ? e & (a.d - 1) : (int)gi[r] * W + e);
#pragma unroll
            for (int j = 0; j < VEC / 2; j += 2) {
                const float4 w = *reinterpret_cast<const float4*>(wp + 2 * j);
                y[i][j] = mul2(mul2(y[i][j], make_float2(rs, rs)), make_float2(w.x, w.y));
                y[i][j + 1] = mul2(mul2(y[i][j + 1], make_float2(rs, rs)), make_float2(w.z, w.w));
            }
            if (gate && !a.gate_first) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) y[i][j] = mul2(y[i][j], act[i][j]);
            }
            *reinterpret_cast<uint4*>(op[r] + e) = Vec16<T>::pack(reinterpret_cast<float*>(y[i]));
        }
    }
}

struct BlockNormArgs {
    const void* x;
    long xs;               // row pitch of x
    const void* residual;  // NULL: zeros
    const float *weight, *post_weight, *scale_v;  // post_weight, scale_v: may be NULL
    float scale, eps;
    void* out;
    void* residual_out;    // NULL: not stored
    long rows;
    int D;
};

// R: the type of residual and residual_out (T or fp32).
template <typename T, typename R, int TPG, int VPT>
__global__ void __launch_bounds__(TPG <= 32 ? NORM_BLOCK : TPG) block_norm_kernel(
    const __grid_constant__ BlockNormArgs a) {
    constexpr int VEC = Vec16<T>::N;
    constexpr int RV = VEC / Vec16<R>::N;  // 16-byte pieces of a residual vector
    constexpr int GPB = TPG <= 32 ? NORM_BLOCK / TPG : 1;
    __shared__ float smem[32];
    const long item = (long)blockIdx.x * GPB + threadIdx.x / TPG;
    const bool live = item < a.rows;
    const long row = live ? item : a.rows - 1;
    const int nv = a.D / VEC, lt = threadIdx.x % TPG;
    const T* xp = static_cast<const T*>(a.x) + row * a.xs;
    const R* rp = a.residual ? static_cast<const R*>(a.residual) + row * a.D : nullptr;

    uint4 xr[VPT], rr[VPT][RV];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lt + i * TPG;
        xr[i] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < RV; ++k) rr[i][k] = make_uint4(0, 0, 0, 0);
        if (v < nv) {
            xr[i] = *reinterpret_cast<const uint4*>(xp + (long)v * VEC);
            if (rp)
#pragma unroll
                for (int k = 0; k < RV; ++k)
                    rr[i][k] = *reinterpret_cast<const uint4*>(rp + (long)v * VEC +
                                                               k * Vec16<R>::N);
        }
    }
    float x[VPT][VEC], ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        Vec16<T>::unpack(xr[i], x[i]);
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(x[i][j], x[i][j], ss);
    }
    float post = 1.f;
    if (a.post_weight) post = rsqrtf(row_sum<TPG>(ss, smem) / (float)a.D + a.eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lt + i * TPG;
        const bool in = v < nv;
        float res[VEC];
#pragma unroll
        for (int k = 0; k < RV; ++k) Vec16<R>::unpack(rr[i][k], res + k * Vec16<R>::N);
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            float4 m = make_float4(post, post, post, post);
            if (a.post_weight && in) {
                const float4 w = *reinterpret_cast<const float4*>(a.post_weight + v * VEC + j);
                m.x *= w.x, m.y *= w.y, m.z *= w.z, m.w *= w.w;
            }
            float4 sc = make_float4(a.scale, a.scale, a.scale, a.scale);
            if (a.scale_v && in) sc = *reinterpret_cast<const float4*>(a.scale_v + v * VEC + j);
            x[i][j] = fmaf(x[i][j] * m.x, sc.x, res[j]);
            x[i][j + 1] = fmaf(x[i][j + 1] * m.y, sc.y, res[j + 1]);
            x[i][j + 2] = fmaf(x[i][j + 2] * m.z, sc.z, res[j + 2]);
            x[i][j + 3] = fmaf(x[i][j + 3] * m.w, sc.w, res[j + 3]);
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(x[i][j], x[i][j], ss);
        if (a.residual_out && live && in) {
            R* ro = static_cast<R*>(a.residual_out) + row * a.D + (long)v * VEC;
#pragma unroll
            for (int k = 0; k < RV; ++k)
                *reinterpret_cast<uint4*>(ro + k * Vec16<R>::N) =
                    Vec16<R>::pack(x[i] + k * Vec16<R>::N);
        }
    }
    const float rs = rsqrtf(row_sum<TPG>(ss, smem) / (float)a.D + a.eps);
    T* op = static_cast<T*>(a.out) + row * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = lt + i * TPG;
        if (!live || v >= nv) continue;
#pragma unroll
        for (int j = 0; j < VEC; j += 4) {
            const float4 w = *reinterpret_cast<const float4*>(a.weight + v * VEC + j);
            x[i][j] *= rs * w.x, x[i][j + 1] *= rs * w.y;
            x[i][j + 2] *= rs * w.z, x[i][j + 3] *= rs * w.w;
        }
        *reinterpret_cast<uint4*>(op + (long)v * VEC) = Vec16<T>::pack(x[i]);
    }
}

}  // namespace drscan
