// C-ABI entry points of the operators around a scan: the short convolution, the selective
// state space scan and its one-token step, and the norms. Argument validation, kernel selection
// and launch; the declarations, with the meaning of every argument, are in drscan.h. Part of the
// translation unit of library.cu, behind drscan.cu: it shares that file's status word, checks of
// pointers, state copy and scratch pool.
#include <algorithm>
#include <climits>
#include <utility>

#include "norms.cuh"
#include "short_conv.cuh"
#include "ssm_chunked.cuh"
#include "ssm_scan.cuh"

using namespace drscan;

namespace {

// A view of at least one element per dimension of `nb` x `nh` x `nt` rows of `width` contiguous
// elements: aligned, with row strides of whole 16-byte pieces. The strides of dimensions of
// size one are never used and may be anything.
bool ok_view(const dr_view* v, long nb, long nh, long nt, int esize) {
    if (!v || !ok_ptr(v->data)) return false;
    const long long s[3] = {v->sb, v->sh, v->st};
    const long n[3] = {nb, nh, nt};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (s[i] < 0 || (s[i] * esize) % 16 != 0)) return false;
    return true;
}

// The same for a view that is written: no two rows may be the same memory. From the dimension of
// the smallest stride on, each steps over all that those before it span.
bool ok_out_view(const dr_view* v, long nb, long nh, long nt, int width, int esize) {
    if (!ok_view(v, nb, nh, nt, esize)) return false;
    std::pair<long long, long> dim[3] = {{v->sb, nb}, {v->sh, nh}, {v->st, nt}};
    std::sort(dim, dim + 3);
    double span = width;  // exact as far as memory reaches
    for (const auto& [stride, n] : dim) {
        if (n <= 1) continue;
        if ((double)stride < span) return false;
        span += (double)stride * (double)(n - 1);
    }
    return true;
}

// ------------------------------------------------------------------ short convolution

template <typename T, int K, bool SILU>
int launch_conv(const ConvArgs& a, bool step, cudaStream_t stream) {
    if (step) {
        const long blocks = (long)a.ncols * ((a.B + CONV_WARPS - 1) / CONV_WARPS);
        if (blocks > INT_MAX) return DR_ERR_UNSUPPORTED;
        short_conv_step_kernel<T, K, SILU><<<(unsigned)blocks, 32 * CONV_WARPS, 0, stream>>>(a);
        return launch_status();
    }
    ConvArgs c = a;
    // Tokens per warp: up to 64 as long as the launch still has 64 warps for each SM, since a tile
    // reads the taps and K - 1 rows of its neighbour again.
    c.tile = 2 * CONV_ROWS;
    while (c.tile < 64 &&
           (long)a.ncols * a.B * (((long)a.T + 2 * c.tile - 1) / (2 * c.tile)) >= 148 * 64)
        c.tile *= 2;
    const long tiles = ((long)a.T + c.tile - 1) / c.tile;  // of 64 for all that a grid cannot hold
    const long gy = (tiles + CONV_WARPS - 1) / CONV_WARPS, gx = (long)a.ncols * a.B;
    if (gx > INT_MAX || gy > 65535) return DR_ERR_UNSUPPORTED;
    short_conv_kernel<T, K, SILU>
        <<<dim3((unsigned)gx, (unsigned)gy), 32 * CONV_WARPS, 0, stream>>>(c);
    return launch_status();
}

template <typename T, int K>
int dispatch_conv_act(const ConvArgs& a, bool silu, bool step, cudaStream_t stream) {
    return silu ? launch_conv<T, K, true>(a, step, stream) : launch_conv<T, K, false>(a, step, stream);
}

template <typename T>
int dispatch_conv(const ConvArgs& a, int K, bool silu, bool step, cudaStream_t stream) {
    switch (K) {
        case 2:
            return dispatch_conv_act<T, 2>(a, silu, step, stream);
        case 3:
            return dispatch_conv_act<T, 3>(a, silu, step, stream);
        case 4:
            return dispatch_conv_act<T, 4>(a, silu, step, stream);
    }
    return DR_ERR_UNSUPPORTED;
}

// Checks what a prompt and a step share and fills the arguments; T = 1 for a step.
int conv_args(ConvArgs* a, const dr_view* x, const float* weight, const float* bias,
              const conv_split* splits, int nsplit, float eps, int B, int T, int C, int K,
              int mode) {
    if (mode & ~(DR_IN_BF16 | CONV_SILU)) return DR_ERR_INVALID_ARG;
    if (B < 0 || T < 0 || C <= 0 || K <= 0 || nsplit < 1 || !splits || !(eps >= 0.f))
        return DR_ERR_INVALID_ARG;
    const int esize = (mode & DR_IN_BF16) ? 2 : 4;
    const bool tokens = B > 0 && T > 0;
    if (!ok_opt(weight) || !ok_opt(bias)) return DR_ERR_INVALID_ARG;
    if (tokens && (!weight || !ok_view(x, B, 1, T, esize))) return DR_ERR_INVALID_ARG;
    if (tokens && T > 1 && x->st < C) return DR_ERR_INVALID_ARG;
    long sum = 0;
    for (int i = 0; i < nsplit; ++i) {
        if (splits[i].heads < 1 || splits[i].dim < 1) return DR_ERR_INVALID_ARG;
        sum += (long)splits[i].heads * splits[i].dim;
    }
    if (sum != C) return DR_ERR_INVALID_ARG;
    if (nsplit > CONV_MAX_SPLITS || K < 2 || K > 4) return DR_ERR_UNSUPPORTED;
    for (int i = 0; i < nsplit; ++i)
        if (!dim_supported(splits[i].dim)) return DR_ERR_UNSUPPORTED;
    *a = ConvArgs{};
    a->x = x ? x->data : nullptr;
    a->xsb = x ? x->sb : 0, a->xst = x ? x->st : 0;
    a->weight = weight, a->bias = bias;
    a->nsplit = nsplit, a->eps = eps;
    a->B = B, a->T = T, a->C = C;
    const int vec = 16 / esize;
    int vec0 = 0, col = 0;
    for (int i = 0; i < nsplit; ++i) {
        const conv_split& s = splits[i];
        if (tokens && !ok_out_view(&s.out, B, s.heads, T, s.dim, esize)) return DR_ERR_INVALID_ARG;
        ConvSplit& d = a->split[i];
        d.out = s.out.data;
        d.sb = s.out.sb, d.sh = s.out.sh, d.st = s.out.st;
        d.dim = s.dim, d.normalise = s.normalise != 0;
        d.vec0 = vec0, d.nvec = s.heads * s.dim / vec, d.warp0 = col;
        vec0 += d.nvec;
        col += (d.nvec + 31) / 32;
    }
    a->ncols = col;
    return DR_OK;
}

// ------------------------------------------------------------------ selective scan

template <typename T, int N>
int launch_ssm_sequential(const SsmArgs& a, cudaStream_t stream) {
    const long gx = (long)a.B * a.H * (a.P / SSM_ROWS);
    if (gx > INT_MAX || a.nseg > 65535) return DR_ERR_UNSUPPORTED;
    if (a.nseg > 1) {
        ssm_sequential_kernel<T, N, SSM_PASS_STATES>
            <<<dim3((unsigned)gx, (unsigned)(a.nseg - 1)), SSM_THREADS, 0, stream>>>(a);
        int rc = launch_status();
        if (rc != DR_OK) return rc;
        rc = launch_ssm_chain(a, stream);
        if (rc != DR_OK) return rc;
    }
    ssm_sequential_kernel<T, N, SSM_PASS_OUTPUTS>
        <<<dim3((unsigned)gx, (unsigned)a.nseg), SSM_THREADS, 0, stream>>>(a);
    return launch_status();
}

template <typename T>
int dispatch_ssm_sequential(const SsmArgs& a, cudaStream_t stream) {
    switch (a.N) {
        case 32:
            return launch_ssm_sequential<T, 32>(a, stream);
        case 64:
            return launch_ssm_sequential<T, 64>(a, stream);
        case 128:
            return launch_ssm_sequential<T, 128>(a, stream);
    }
    return DR_ERR_UNSUPPORTED;
}

// Segments of the per-token scan: of 32 tokens each, as far as four CTAs (of 32 rows) to an SM go,
// from three segments on, where one pass over all tokens takes 20 us or more: 192 tokens at N = 32, 96
// at N = 128. Two launches more and the scratch take the host 6 us. Measured on the device, fp32,
// whole and in segments: N = 32, 2 x 4 heads: 200 tokens 23 and 12 us, 301 tokens 34 and 12; N = 128,
// 4 heads: 100 tokens 25 and 16 us, 301 tokens 73 and 17; 32 heads of 128 x 128, 200 tokens 50 and
// 45. (301 tokens in segments of 48: 14 and 22 us; of 80: 18 and 31.)
void plan_ssm_sequential(SsmArgs* a) {
    a->nseg = 1;
    a->seg_len = a->T;
    const long ctas = (long)a->B * a->H * (a->P / SSM_ROWS);
    if ((long)a->T * (64 + a->N) < 192 * 96) return;
    const long most = std::min<long>(((long)a->T + 31) / 32, 592 / ctas);
    if (most > 2) {
        a->seg_len = (int)(((a->T + most - 1) / most + SSM_TILE - 1) / SSM_TILE * SSM_TILE);
        a->nseg = (a->T + a->seg_len - 1) / a->seg_len;
    }
}

template <typename T, int N>
int launch_ssm_step(const SsmArgs& a, float* S, cudaStream_t stream) {
    const long rows = (long)a.B * a.H * a.P;
    const long per = (128 / N) * SSM_STEP_U * (long)SSM_STEP_WARPS;
    const long blocks = (rows + per - 1) / per;
    if (blocks > INT_MAX) return DR_ERR_UNSUPPORTED;
    ssm_step_kernel<T, N><<<(unsigned)blocks, 32 * SSM_STEP_WARPS, 0, stream>>>(a, S);
    return launch_status();
}

template <typename T>
int dispatch_ssm_step(const SsmArgs& a, float* S, cudaStream_t stream) {
    switch (a.N) {
        case 32:
            return launch_ssm_step<T, 32>(a, S, stream);
        case 64:
            return launch_ssm_step<T, 64>(a, S, stream);
        case 128:
            return launch_ssm_step<T, 128>(a, S, stream);
    }
    return DR_ERR_UNSUPPORTED;
}

// SMs of the current device.
int sm_count() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1)
        return 148;
    return n;
}

// Limit of a wait inside the chunked scan's launches of this host thread, in nanoseconds, or -1 for
// the usual one (dr_debug_wait_limit).
thread_local long long g_wait_ns = -1;

SsmView as_view(const dr_view* v) {
    return v ? SsmView{v->data, (long)v->sb, (long)v->sh, (long)v->st} : SsmView{};
}

// Checks what the scan and the step share and fills the arguments; T = 1 for a step.
int ssm_args(SsmArgs* a, const dr_view* x, const dr_view* dt, const float* A, const dr_view* Bm,
             const dr_view* Cm, const float* D, const float* dt_bias, const dr_view* out, int B,
             int H, int G, int T, int P, int N, int mode) {
    if (B < 0 || H < 0 || G <= 0 || T < 0 || P <= 0 || N <= 0 || H % G != 0)
        return DR_ERR_INVALID_ARG;
    const long BH = (long)B * H;
    if (BH > INT_MAX) return DR_ERR_INVALID_ARG;
    const int esize = (mode & DR_IN_BF16) ? 2 : 4;
    if (!ok_opt(A) || !ok_opt(D) || !ok_opt(dt_bias)) return DR_ERR_INVALID_ARG;
    if (BH > 0 && T > 0) {
        if (!A || !dt || !dt->data) return DR_ERR_INVALID_ARG;
        if (reinterpret_cast<uintptr_t>(dt->data) % ((mode & SSM_DT_BF16) ? 2 : 4) != 0)
            return DR_ERR_INVALID_ARG;
        if (!ok_view(x, B, H, T, esize) || !ok_view(Bm, B, G, T, esize) ||
            !ok_view(Cm, B, G, T, esize) || !ok_out_view(out, B, H, T, P, esize))
            return DR_ERR_INVALID_ARG;
    }
    if (!dim_supported(P) || !dim_supported(N)) return DR_ERR_UNSUPPORTED;
    *a = SsmArgs{};
    a->x = as_view(x), a->dt = as_view(dt), a->Bm = as_view(Bm), a->Cm = as_view(Cm);
    a->A = A, a->D = D, a->dt_bias = dt_bias;
    if (out) a->out = out->data, a->osb = out->sb, a->osh = out->sh, a->ost = out->st;
    a->B = B, a->H = H, a->G = G, a->T = T, a->P = P, a->N = N;
    a->softplus = (mode & SSM_DT_SOFTPLUS) != 0;
    a->dt_bf16 = (mode & SSM_DT_BF16) != 0;
    a->nseg = 1;
    a->seg_len = T;
    return DR_OK;
}

// ------------------------------------------------------------------ norms

// Runs `launch` with the threads per row (TPG) and vectors per thread (VPT) for rows of nv
// 16-byte vectors: one vector a thread as long as a row fits a warp, whose sums need no barrier
// then; then up to four, what a thread can have in flight.
template <typename F>
int with_row_shape(int nv, F&& launch) {
    if (nv <= 4) return launch.template operator()<4, 1>();
    if (nv <= 8) return launch.template operator()<8, 1>();
    if (nv <= 16) return launch.template operator()<16, 1>();
    if (nv <= 32) return launch.template operator()<32, 1>();
    if (nv <= 64) return launch.template operator()<32, 2>();
    if (nv <= 128) return launch.template operator()<32, 4>();
    if (nv <= 256) return launch.template operator()<128, 2>();
    if (nv <= 512) return launch.template operator()<128, 4>();
    if (nv <= 1024) return launch.template operator()<256, 4>();
    return launch.template operator()<512, 4>();
}
constexpr int NORM_MAX_VECTORS = 2048;

long norm_blocks(long items, int tpg) {
    const int per = tpg <= 32 ? NORM_BLOCK / tpg : 1;
    return (items + per - 1) / per;
}

template <typename T>
struct GatedLaunch {
    const GatedNormArgs& a;
    cudaStream_t stream;
    template <int TPG, int VPT>
    int operator()() const {
        const double items = (double)a.B * a.T * (a.H / a.heads);
        if (items > INT_MAX) return DR_ERR_UNSUPPORTED;
        const long blocks = norm_blocks((long)items, TPG);
        const unsigned threads = TPG <= 32 ? NORM_BLOCK : TPG;
        // Several items per group once they fill the GPU (16 CTAs to an SM) all the same.
        constexpr int R = TPG <= 32 ? 4 / VPT : 1;
        if (R > 1 && blocks >= 148l * 16 * R) {
            gated_norm_kernel<T, TPG, VPT, R>
                <<<(unsigned)((blocks + R - 1) / R), threads, 0, stream>>>(a);
        } else {
            gated_norm_kernel<T, TPG, VPT, 1><<<(unsigned)blocks, threads, 0, stream>>>(a);
        }
        return launch_status();
    }
};

template <typename T, typename R>
struct BlockLaunch {
    const BlockNormArgs& a;
    cudaStream_t stream;
    template <int TPG, int VPT>
    int operator()() const {
        const long blocks = norm_blocks(a.rows, TPG);
        if (blocks > INT_MAX) return DR_ERR_UNSUPPORTED;
        block_norm_kernel<T, R, TPG, VPT>
            <<<(unsigned)blocks, TPG <= 32 ? NORM_BLOCK : TPG, 0, stream>>>(a);
        return launch_status();
    }
};

}  // namespace

extern "C" {

int short_conv_fwd(const dr_view* x, const float* weight, const float* bias, const void* state0,
                   const int* lengths, const conv_split* splits, int nsplit, void* state_final,
                   float eps, int B, int T, int C, int K, int mode, cudaStream_t stream) {
    ConvArgs a;
    const int rc = conv_args(&a, x, weight, bias, splits, nsplit, eps, B, T, C, K, mode);
    if (rc != DR_OK) return rc;
    if (!ok_opt(state0) || !ok_opt(state_final) || (reinterpret_cast<uintptr_t>(lengths) & 3))
        return DR_ERR_INVALID_ARG;
    if (state0 && state0 == state_final) return DR_ERR_INVALID_ARG;
    if (B == 0) return DR_OK;
    if (T == 0)
        return copy_state(static_cast<float*>(state_final), static_cast<const float*>(state0),
                          (size_t)B * (K - 1) * C * ((mode & DR_IN_BF16) ? 2 : 4) / sizeof(float),
                          stream);
    a.state0 = state0;
    a.state_final = state_final;
    a.lengths = lengths;
    const bool silu = (mode & CONV_SILU) != 0;
    return (mode & DR_IN_BF16) ? dispatch_conv<__nv_bfloat16>(a, K, silu, false, stream)
                               : dispatch_conv<float>(a, K, silu, false, stream);
}

int short_conv_step(const dr_view* x, const float* weight, const float* bias, void* state,
                    const conv_split* splits, int nsplit, float eps, int B, int C, int K, int mode,
                    cudaStream_t stream) {
    ConvArgs a;
    const int rc = conv_args(&a, x, weight, bias, splits, nsplit, eps, B, 1, C, K, mode);
    if (rc != DR_OK) return rc;
    if (!ok_opt(state) || (B > 0 && !state)) return DR_ERR_INVALID_ARG;
    if (B == 0) return DR_OK;
    a.state_final = state;
    const bool silu = (mode & CONV_SILU) != 0;
    return (mode & DR_IN_BF16) ? dispatch_conv<__nv_bfloat16>(a, K, silu, true, stream)
                               : dispatch_conv<float>(a, K, silu, true, stream);
}

int ssm_scan_fwd(const dr_view* x, const dr_view* dt, const float* A, const dr_view* Bm,
                 const dr_view* Cm, const float* D, const float* dt_bias, const float* S0,
                 const int* lengths, const dr_view* out, float* S_final, int B, int H, int G,
                 int T, int P, int N, int mode, cudaStream_t stream) {
    if (mode & ~(DR_IN_BF16 | DR_FORCE_SEQUENTIAL | SSM_DT_SOFTPLUS | SSM_DT_BF16))
        return DR_ERR_INVALID_ARG;
    SsmArgs a;
    int rc = ssm_args(&a, x, dt, A, Bm, Cm, D, dt_bias, out, B, H, G, T, P, N, mode);
    if (rc != DR_OK) return rc;
    if (!ok_opt(S0) || !ok_opt(S_final) || (reinterpret_cast<uintptr_t>(lengths) & 3))
        return DR_ERR_INVALID_ARG;
    if (S0 && S0 == S_final) return DR_ERR_INVALID_ARG;
    if (T > 1 << 30) return DR_ERR_UNSUPPORTED;  // tokens are counted in 32 bits, a chunk beyond T
    const long BH = (long)B * H;
    if (BH == 0) return DR_OK;
    const size_t PN = (size_t)P * N;
    if (T == 0) return copy_state(S_final, S0, BH * PN, stream);
    a.S0 = S0;
    a.S_final = S_final;
    a.lengths = lengths;
    // By the tokens alone, fitted to few heads. Device time (P 64) of the chunked kernel and the
    // per-token one: N = 128, 16 heads: 17 tokens 7.8 and 6.5 us, 33 tokens 8.0 and 9.9, 128 tokens
    // 8.7 and 17.4; N = 32: 65 tokens 8.2 and 9.4, 128 tokens 8.6 and 15.4. With more heads the two
    // meet later, and just above the limit the per-token kernel would be faster: 256 heads 15.6 and
    // 11.4 (17 tokens, N = 128), 16.2 and 15.4 (65, N = 32), 2048 heads 97 and 65, 101 and 82; from
    // twice the limit on the chunked kernel is (2048 heads: 100 and 113, 117 and 156).
    const bool chunked = (mode & DR_IN_BF16) && !(mode & DR_FORCE_SEQUENTIAL) &&
                         (long)T * N > 2048 && ssm_chunked_fits(a);
    if (chunked)
        plan_ssm_chunked(&a, sm_count());
    else
        plan_ssm_sequential(&a);
    void* scratch = nullptr;
    if (a.nseg > 1) {
        const size_t states = (size_t)BH * (a.nseg - 1);
        rc = scratch_alloc(&scratch, states * (PN + 1) * sizeof(float), stream);
        if (rc != DR_OK) return rc;
        a.seg_state = static_cast<float*>(scratch);
        a.seg_log = a.seg_state + states * PN;
    }
    rc = chunked && g_wait_ns < 0 ? launch_ssm_chunked<false>(a, 0, stream)
         : chunked                ? launch_ssm_chunked<true>(a, (uint32_t)g_wait_ns, stream)
         : (mode & DR_IN_BF16)    ? dispatch_ssm_sequential<__nv_bfloat16>(a, stream)
                                  : dispatch_ssm_sequential<float>(a, stream);
    if (scratch && cudaFreeAsync(scratch, stream) != cudaSuccess && rc == DR_OK) rc = DR_ERR_CUDA;
    return rc;
}

int dr_debug_wait_limit(long long limit_ns) {
    if (limit_ns < -1 || limit_ns > (long long)DRSCAN_WAIT_LIMIT_NS) return DR_ERR_INVALID_ARG;
    g_wait_ns = limit_ns;
    return DR_OK;
}

int ssm_step(const dr_view* x, const dr_view* dt, const float* A, const dr_view* Bm,
             const dr_view* Cm, const float* D, const float* dt_bias, float* S,
             const dr_view* out, int B, int H, int G, int P, int N, int mode,
             cudaStream_t stream) {
    if (mode & ~(DR_IN_BF16 | SSM_DT_SOFTPLUS | SSM_DT_BF16)) return DR_ERR_INVALID_ARG;
    SsmArgs a;
    const int rc = ssm_args(&a, x, dt, A, Bm, Cm, D, dt_bias, out, B, H, G, 1, P, N, mode);
    if (rc != DR_OK) return rc;
    if (!ok_opt(S) || ((long)B * H > 0 && !S)) return DR_ERR_INVALID_ARG;
    if ((long)B * H == 0) return DR_OK;
    return (mode & DR_IN_BF16) ? dispatch_ssm_step<__nv_bfloat16>(a, S, stream)
                               : dispatch_ssm_step<float>(a, S, stream);
}

int gated_norm_fwd(const dr_view* y, const dr_view* gate, const float* weight, const dr_view* out,
                   float eps, int B, int H, int T, int d, int norm_heads, int mode,
                   cudaStream_t stream) {
    if (mode & ~(DR_IN_BF16 | NORM_SIGMOID | NORM_GATE_FIRST | NORM_SHARED_WEIGHT))
        return DR_ERR_INVALID_ARG;
    if (B < 0 || H < 0 || T < 0 || d <= 0 || norm_heads <= 0 || H % norm_heads != 0 ||
        !(eps >= 0.f))
        return DR_ERR_INVALID_ARG;
    const int esize = (mode & DR_IN_BF16) ? 2 : 4;
    const bool tokens = B > 0 && H > 0 && T > 0;
    if (!ok_opt(weight)) return DR_ERR_INVALID_ARG;
    const bool gated = gate && gate->data;
    const long row = (long)H * d;
    if (row > INT_MAX) return DR_ERR_UNSUPPORTED;
    if (tokens && (!weight || !ok_view(y, B, H, T, esize) ||
                   (gated && !ok_view(gate, B, 1, T, esize)) ||
                   !ok_out_view(out, B, 1, T, (int)row, esize)))
        return DR_ERR_INVALID_ARG;
    if (!dim_supported(d) || (long)norm_heads * d > (long)NORM_MAX_VECTORS * (16 / esize))
        return DR_ERR_UNSUPPORTED;
    if (!tokens) return DR_OK;
    GatedNormArgs a{};
    a.y = y->data, a.ysb = y->sb, a.ysh = y->sh, a.yst = y->st;
    if (gated) a.gate = gate->data, a.gsb = gate->sb, a.gst = gate->st;
    a.weight = weight;
    a.out = out->data, a.osb = out->sb, a.ost = out->st;
    a.eps = eps;
    a.inv_w = 1.f / (float)(norm_heads * d);
    a.by_groups = DivBy((unsigned)(H / norm_heads));
    a.by_T = DivBy((unsigned)T);
    a.B = B, a.H = H, a.T = T, a.d = d, a.heads = norm_heads;
    a.shared_weight = (mode & NORM_SHARED_WEIGHT) != 0;
    a.sigmoid = (mode & NORM_SIGMOID) != 0;
    a.gate_first = (mode & NORM_GATE_FIRST) != 0;
    const int nv = norm_heads * d / (16 / esize);
    return (mode & DR_IN_BF16)
               ? with_row_shape(nv, GatedLaunch<__nv_bfloat16>{a, stream})
               : with_row_shape(nv, GatedLaunch<float>{a, stream});
}

int block_norm_fwd(const void* x, long long x_pitch, const void* residual, const float* weight,
                   const float* post_weight, const float* scale_v, float scale, void* out,
                   void* residual_out, float eps, long long rows, int D, int mode,
                   cudaStream_t stream) {
    if (mode & ~(DR_IN_BF16 | NORM_RESIDUAL_F32)) return DR_ERR_INVALID_ARG;
    if (rows < 0 || D <= 0 || !(eps >= 0.f)) return DR_ERR_INVALID_ARG;
    const int esize = (mode & DR_IN_BF16) ? 2 : 4;
    if (!ok_opt(x) || !ok_opt(residual) || !ok_opt(weight) || !ok_opt(post_weight) ||
        !ok_opt(scale_v) || !ok_opt(out) || !ok_opt(residual_out))
        return DR_ERR_INVALID_ARG;
    if (rows > 0 && (!x || !weight || !out)) return DR_ERR_INVALID_ARG;
    if (rows > 1 && (x_pitch < 0 || (x_pitch * esize) % 16 != 0)) return DR_ERR_INVALID_ARG;
    const int vec = 16 / esize;
    if (D % vec != 0 || D / vec > NORM_MAX_VECTORS) return DR_ERR_UNSUPPORTED;
    if (rows == 0) return DR_OK;
    BlockNormArgs a{x, (long)x_pitch, residual, weight, post_weight, scale_v, scale, eps, out,
                    residual_out, (long)rows, D};
    const int nv = D / vec;
    if (!(mode & DR_IN_BF16)) return with_row_shape(nv, BlockLaunch<float, float>{a, stream});
    return (mode & NORM_RESIDUAL_F32)
               ? with_row_shape(nv, BlockLaunch<__nv_bfloat16, float>{a, stream})
               : with_row_shape(nv, BlockLaunch<__nv_bfloat16, __nv_bfloat16>{a, stream});
}

}  // extern "C"
