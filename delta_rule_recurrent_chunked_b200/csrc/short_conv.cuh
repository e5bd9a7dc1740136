// Short causal convolution over tokens, one filter of K = 2..4 taps per channel, with SiLU, an
// optional L2 norm per head and the split of the channels into heads:
//
//     c_t[ch] = bias[ch] + sum_j w[ch][j] x_{t-K+1+j}[ch],    y = c sigmoid(c)
//     y_head <- y_head / sqrt(sum y_head^2 + eps)             (heads of a normalised split)
//
// x_{-1}, x_{-2}, .. come from state0, the K - 1 inputs before the sequence (zeros without it).
//
// Floor: HBM. Every input is read once and every output written once, at about K + 6 flops per
// 2 bytes. A warp owns 32 vectors of 16 bytes (256 bf16 channels) of one split and walks a tile
// of tokens; the last K - 1 rows stay in registers as the window, so a tile re-reads K - 1 rows
// of its neighbour only. The next rows are in flight while the last ones are summed. A head is 4 to 32
// neighbouring lanes, so its norm is a few shuffles and the head-major (or token-major) rows
// leave in 16-byte stores.
//
// Measured, q, k and v of 16 heads of 128 (6144 bf16 channels, q and k normalised) for 8 x 4096
// tokens, 805 MB: 170 us, 4.7 TB/s, 73% of the measured copy rate. The loads and stores alone take
// 137 us, without SiLU 158: the rest is the issue and latency of some hundred instructions per
// 16 bytes on the 16 warps that the window and the taps leave room for (issue slots 45%, special
// functions 56%, DRAM 48% busy under ncu). Tiles of 32 tokens 177 us, of 128 172; CTAs of 2 or 8
// warps 171 and 173. Vectors of 8 bytes leave room for 20 to 28 warps and take 174 to 179, more
// instructions and shuffles a byte. Fewer instructions saved no time: taps scaled for 2^x (172), one
// reciprocal for two sigmoids (171, and it loses saturated gates); the loop unrolled twice took 181.
#pragma once

#include "layer_common.cuh"

namespace drscan {

constexpr int CONV_MAX_SPLITS = 4;
constexpr int CONV_WARPS = 4;
constexpr int CONV_ROWS = 4;  // rows in flight per thread while four more are summed (8, with the
                              // registers of 3 CTAs per SM: 173 us)
constexpr int CONV_CTAS = 4;  // per SM, at 128 registers (5 spill)

struct ConvSplit {
    void* out;
    long sb, sh, st;
    int dim, normalise;
    int vec0;   // first 16-byte vector of the split within a row
    int nvec;   // vectors of the split
    int warp0;  // first warp column of the split
};

struct ConvArgs {
    const void* x;
    long xsb, xst;
    const float *weight, *bias;
    const void* state0;
    void* state_final;
    const int* lengths;
    ConvSplit split[CONV_MAX_SPLITS];
    int nsplit, ncols;  // ncols: warp columns of all splits
    float eps;
    int B, T, C, tile;
};

// The split that warp column `col` belongs to.
__device__ __forceinline__ int split_of(const ConvArgs& a, int col) {
    int si = 0;
    while (si + 1 < a.nsplit && col >= a.split[si + 1].warp0) ++si;
    return si;
}

// Sum over LANES neighbouring lanes.
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int off = LANES >> 1; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Runs `f` with the lanes of a normalised split's heads as a constant, 0 without the norm. (With the
// count at run time the sums of neighbouring rows' squares wait for one another: 178 us instead of
// 170.)
template <int VEC, typename F>
__device__ __forceinline__ void with_lanes(const ConvSplit& sp, F&& f) {
    if (!sp.normalise)
        f(std::integral_constant<int, 0>());
    else if (sp.dim == 32)
        f(std::integral_constant<int, 32 / VEC>());
    else if (sp.dim == 64)
        f(std::integral_constant<int, 64 / VEC>());
    else
        f(std::integral_constant<int, 128 / VEC>());
}

// The taps of one thread's channels, by pairs of channels (the sums run two to an instruction).
template <int VEC, int K>
struct ConvTaps {
    float2 w[K][VEC / 2], b[VEC / 2];
    __device__ __forceinline__ void load(const float* weight, const float* bias, int ch0) {
        // the taps of neighbouring channels lie together: whole 16-byte pieces
        float t[VEC * K], c[VEC];
#pragma unroll
        for (int i = 0; i < VEC * K; i += 4)
            *reinterpret_cast<float4*>(t + i) =
                *reinterpret_cast<const float4*>(weight + (long)ch0 * K + i);
#pragma unroll
        for (int i = 0; i < VEC; i += 4)
            *reinterpret_cast<float4*>(c + i) =
                bias ? *reinterpret_cast<const float4*>(bias + ch0 + i) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int v = 0; v < VEC / 2; ++v) {
            b[v] = make_float2(c[2 * v], c[2 * v + 1]);
#pragma unroll
            for (int j = 0; j < K; ++j) w[j][v] = make_float2(t[2 * v * K + j], t[(2 * v + 1) * K + j]);
        }
    }
};

// One row: window (oldest first) and the new row x -> the activated, normalised outputs.
template <int VEC, int K, bool SILU, int LANES>
__device__ __forceinline__ void conv_row(const ConvTaps<VEC, K>& f, float2 (&win)[K - 1][VEC / 2],
                                         const float2* x, float eps, float2* y) {
    float2 ss = make_float2(0.f, 0.f);
#pragma unroll
    for (int v = 0; v < VEC / 2; ++v) {
        float2 c = fma2(f.w[K - 1][v], x[v], f.b[v]);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) c = fma2(f.w[j][v], win[j][v], c);
        y[v] = SILU ? mul2(c, sigmoid2(c)) : c;
        if (LANES > 0) ss = fma2(y[v], y[v], ss);
    }
#pragma unroll
    for (int j = 0; j < K - 2; ++j)
#pragma unroll
        for (int v = 0; v < VEC / 2; ++v) win[j][v] = win[j + 1][v];
#pragma unroll
    for (int v = 0; v < VEC / 2; ++v) win[K - 2][v] = x[v];
    if (LANES > 0) {
        const float r = rsqrtf(group_sum<LANES>(ss.x + ss.y) + eps);
#pragma unroll
        for (int v = 0; v < VEC / 2; ++v) y[v] = mul2(y[v], make_float2(r, r));
    }
}

// grid: (warp columns * B, token tiles / CONV_WARPS); block: CONV_WARPS warps, one token tile
// each.
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * CONV_WARPS, CONV_CTAS) short_conv_kernel(
    const __grid_constant__ ConvArgs a) {
    constexpr int VEC = Vec16<T>::N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long b = blockIdx.x / a.ncols;
    const int col = (int)(blockIdx.x % a.ncols);
    const ConvSplit& sp = a.split[split_of(a, col)];
    const int v_in = (col - sp.warp0) * 32 + lane;  // vector within the split
    // lanes behind the split's last vector repeat it and store nothing: heads are whole powers
    // of two of lanes, so no head mixes live and idle lanes
    const bool live = v_in < sp.nvec;
    const int v = live ? v_in : sp.nvec - 1;
    const int ch0 = (sp.vec0 + v) * VEC;
    const int len = a.lengths ? min(max(a.lengths[b], 0), a.T) : a.T;
    const int tile = (int)blockIdx.y * CONV_WARPS + warp;
    const long t_begin = (long)tile * a.tile;
    const int t0 = (int)min(t_begin, (long)a.T);
    const int t1 = (int)min(t_begin + a.tile, (long)len);

    const T* xrow = static_cast<const T*>(a.x) + b * a.xsb + ch0;
    const T* prev = a.state0 ? static_cast<const T*>(a.state0) + b * (long)(K - 1) * a.C + ch0
                             : nullptr;
    // row i of the K - 1 earlier inputs followed by the sequence
    auto row = [&](long i) -> uint4 {
        if (i >= K - 1) return *reinterpret_cast<const uint4*>(xrow + (i - (K - 1)) * a.xst);
        if (prev) return *reinterpret_cast<const uint4*>(prev + i * a.C);
        return make_uint4(0, 0, 0, 0);
    };

    if (tile == 0 && a.state_final && live) {
        T* dst = static_cast<T*>(a.state_final) + b * (long)(K - 1) * a.C + ch0;
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            *reinterpret_cast<uint4*>(dst + (long)j * a.C) = row((long)len + j);
    }
    if (t0 >= t1) return;  // the whole warp

    ConvTaps<VEC, K> f;
    f.load(a.weight, a.bias, ch0);
    float2 win[K - 1][VEC / 2];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        Vec16<T>::unpack(row((long)t0 + j), reinterpret_cast<float*>(win[j]));

    const int lanes = sp.dim / VEC;
    const int head = v / lanes, within = v % lanes;
    T* dst = static_cast<T*>(sp.out) + b * sp.sb + head * sp.sh + within * VEC;
    const T* src = xrow + (long)t0 * a.xst;
    dst += (long)t0 * sp.st;
    // a group's rows are loaded while the group before is summed; rows behind the last are not read
    uint4 raw[CONV_ROWS];
    auto fetch = [&](int n) {
#pragma unroll
        for (int i = 0; i < CONV_ROWS; ++i) {
            if (i < n) raw[i] = *reinterpret_cast<const uint4*>(src);
            src += a.xst;
        }
    };
    fetch(t1 - t0);
    with_lanes<VEC>(sp, [&](auto lanes_of_head) {
        constexpr int LANES = decltype(lanes_of_head)::value;
        for (int t = t0; t < t1; t += CONV_ROWS) {
            const int n = t1 - t;  // rows left
            uint4 now[CONV_ROWS];
#pragma unroll
            for (int i = 0; i < CONV_ROWS; ++i) now[i] = raw[i];
            if (n > CONV_ROWS) fetch(n - CONV_ROWS);
#pragma unroll
            for (int i = 0; i < CONV_ROWS; ++i) {
                float2 x[VEC / 2], y[VEC / 2];
                Vec16<T>::unpack(now[i], reinterpret_cast<float*>(x));
                conv_row<VEC, K, SILU, LANES>(f, win, x, a.eps, y);
                if (live && i < n)
                    *reinterpret_cast<uint4*>(dst) = Vec16<T>::pack(reinterpret_cast<float*>(y));
                dst += sp.st;
            }
        }
    });
}

// One token per sequence on a resident state (the last K - 1 inputs, shifted in place). A warp
// per 32 vectors and sequence. grid: warp columns * ceil(B / CONV_WARPS).
template <typename T, int K, bool SILU>
__global__ void __launch_bounds__(32 * CONV_WARPS) short_conv_step_kernel(
    const __grid_constant__ ConvArgs a) {
    constexpr int VEC = Vec16<T>::N;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long b = (long)(blockIdx.x / a.ncols) * CONV_WARPS + warp;
    if (b >= a.B) return;  // the whole warp
    const int col = (int)(blockIdx.x % a.ncols);
    const ConvSplit& sp = a.split[split_of(a, col)];
    const int v_in = (col - sp.warp0) * 32 + lane;
    const bool live = v_in < sp.nvec;
    const int v = live ? v_in : sp.nvec - 1;
    const int ch0 = (sp.vec0 + v) * VEC;
    T* state = static_cast<T*>(a.state_final) + b * (long)(K - 1) * a.C + ch0;
    uint4 old[K - 1];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        old[j] = *reinterpret_cast<const uint4*>(state + (long)j * a.C);
    const uint4 now = *reinterpret_cast<const uint4*>(static_cast<const T*>(a.x) + b * a.xsb + ch0);
    ConvTaps<VEC, K> f;
    f.load(a.weight, a.bias, ch0);
    float2 win[K - 1][VEC / 2], x[VEC / 2], y[VEC / 2];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) Vec16<T>::unpack(old[j], reinterpret_cast<float*>(win[j]));
    Vec16<T>::unpack(now, reinterpret_cast<float*>(x));
    const int lanes = sp.dim / VEC;
    with_lanes<VEC>(sp, [&](auto lanes_of_head) {
        conv_row<VEC, K, SILU, decltype(lanes_of_head)::value>(f, win, x, a.eps, y);
    });
    __syncwarp();  // idle lanes have read the last vector's state before its owner shifts it
    if (live) {
#pragma unroll
        for (int j = 0; j < K - 2; ++j)
            *reinterpret_cast<uint4*>(state + (long)j * a.C) = old[j + 1];
        *reinterpret_cast<uint4*>(state + (long)(K - 2) * a.C) = now;
        T* dst = static_cast<T*>(sp.out) + b * sp.sb + (v / lanes) * sp.sh + (v % lanes) * VEC;
        *reinterpret_cast<uint4*>(dst) = Vec16<T>::pack(reinterpret_cast<float*>(y));
    }
}

}  // namespace drscan
