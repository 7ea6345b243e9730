// group_norm.cu -- the channels-last group norm behind the C ABI of include/gtr_norm.h.
//
// Forward: z = (x - mean) rstd gamma + beta, out = act(z).  Backward, with dz = d_out act'(z), the
// per-channel sums P = sum dz, Q = sum dz xhat over the tokens of a batch entry and the M = N C / G
// elements of a group:
//     grad_x = rstd (gamma dz - (sum_group gamma P + xhat sum_group gamma Q) / M)
//     grad_gamma = sum_b Q,  grad_beta = sum_b P
// A few operations for 4 bytes moved (6 backward): HBM-bound, and what costs is reading the
// activations once for the sums and again for the result.
#include "../../include/gtr_norm.h"
#include "ops_common.cuh"

namespace gtr {
static __device__ unsigned int g_norm_error_word;
static __device__ __forceinline__ void set_error(unsigned e) { atomicOr(&g_norm_error_word, e); }

namespace gn {

using namespace ops;

struct Args {
    const uint16_t *x, *dy;
    const float *gamma, *beta, *stats;   // stats: backward
    uint16_t *out;                       // out or grad_x
    float *st, *part, *coef, *gg, *gb;
    float eps;
    int B, N, C, G, Cg, act;
    int splits, rows;                    // token ranges of a batch entry, tokens in each (the last: fewer)
    int cblocks;                         // blocks along the channels
};

// Welford pairs: the mean and the sum of squared deviations of n values.
struct Pair {
    float n, mean, m2;
};
__device__ __forceinline__ Pair merge(const Pair &a, const Pair &b) {
    const float n = a.n + b.n;
    if (n == 0.f) return a;
    const float d = b.mean - a.mean, f = b.n / n;
    return {n, fmaf(d, f, a.mean), a.m2 + b.m2 + d * d * a.n * f};
}

__device__ __forceinline__ float act_grad(float z) {   // silu'(z)
    const float s = sigmoid_f(z);
    return s * fmaf(z, 1.f - s, 1.f);
}

// ------------------------------------------------------------------ any shape: three launches
// 1. sums over the tokens of a range per channel; 2. the groups' figures from them; 3. the
// results.  The activations are read in 1 and again in 3 (from L2 where they fit).
constexpr int kRowLanes = 8;

// Sums of one token range: a block takes 32 V channels, its 8 rows of threads every eighth
// token.  Forward: per channel the mean and squared deviations, from sums shifted by the lane's
// first value (so that a large mean costs nothing); backward: P and Q.
template <typename T, int V, bool BWD>
__global__ void __launch_bounds__(32 * kRowLanes) group_norm_sums_kernel(const Args a) {
    __shared__ float red[kRowLanes][32][V][2];
    chain_wait();
    const int cb = blockIdx.x % a.cblocks, sb = blockIdx.x / a.cblocks;
    const int b = sb / a.splits, s = sb - b * a.splits;
    const int c = (cb * 32 + threadIdx.x) * V;
    const int r0 = s * a.rows, r1 = min(a.N, r0 + a.rows), rf = r0 + threadIdx.y;
    float s1[V], s2[V], mean[V], rstd[V], gam[V], bet[V];
#pragma unroll
    for (int v = 0; v < V; ++v) s1[v] = s2[v] = 0.f;
    const bool live = c < a.C;   // V divides C
    float n = 0.f;
    if (live && rf < r1) {
        const long long base = (long long)b * a.N * a.C + c;
        if (BWD) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float *st = a.stats + ((long long)b * a.G + (c + v) / a.Cg) * 2;
                mean[v] = __ldg(st), rstd[v] = __ldg(st + 1);
                gam[v] = a.gamma != nullptr ? __ldg(a.gamma + c + v) : 1.f;
                bet[v] = a.beta != nullptr ? __ldg(a.beta + c + v) : 0.f;
            }
        } else {
            unpack<T, V>(load_raw<V>(a.x + base + (long long)rf * a.C), mean);   // the shift
        }
#pragma unroll 4
        for (int r = rf; r < r1; r += kRowLanes) {
            float x[V];
            unpack<T, V>(load_raw<V>(a.x + base + (long long)r * a.C), x);
            if (BWD) {
                float dy[V];
                unpack<T, V>(load_raw<V>(a.dy + base + (long long)r * a.C), dy);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float xh = (x[v] - mean[v]) * rstd[v];
                    const float dz = a.act == GTR_ACT_SILU ? dy[v] * act_grad(fmaf(xh, gam[v], bet[v])) : dy[v];
                    s1[v] += dz;
                    s2[v] = fmaf(dz, xh, s2[v]);
                }
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float d = x[v] - mean[v];
                    s1[v] += d;
                    s2[v] = fmaf(d, d, s2[v]);
                }
                n += 1.f;
            }
        }
        if (!BWD) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float m = s1[v] / n;
                s2[v] = fmaxf(fmaf(-m, s1[v], s2[v]), 0.f) + 0.f * s2[v];   // a NaN stays one
                s1[v] = mean[v] + m;
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        red[threadIdx.y][threadIdx.x][v][0] = s1[v];
        red[threadIdx.y][threadIdx.x][v][1] = s2[v];
    }
    __syncthreads();
    for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * V; i += 32 * kRowLanes) {
        const int ch = cb * 32 * V + i;
        if (ch >= a.C) continue;
        float2 o;
        if (BWD) {
            o = make_float2(0.f, 0.f);
#pragma unroll
            for (int l = 0; l < kRowLanes; ++l) {
                o.x += red[l][i / V][i % V][0];
                o.y += red[l][i / V][i % V][1];
            }
        } else {
            Pair p{0.f, 0.f, 0.f};
#pragma unroll
            for (int l = 0; l < kRowLanes; ++l) {
                const int nl = (r1 - r0 - l + kRowLanes - 1) / kRowLanes;   // tokens of that row of threads
                if (nl > 0) p = merge(p, {(float)nl, red[l][i / V][i % V][0], red[l][i / V][i % V][1]});
            }
            o = make_float2(p.mean, p.m2);
        }
        reinterpret_cast<float2 *>(a.part)[((long long)b * a.splits + s) * a.C + ch] = o;
    }
}

__device__ __forceinline__ float block_sum(float v, float *red) {   // 256 threads; the sum in every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += red[w];
    return v;
}

// The figures of a group (one block each): forward mean and rstd, backward the two sums over M.
// Backward, further blocks add grad_gamma and grad_beta over batch entries and token ranges.
template <bool BWD>
__global__ void __launch_bounds__(256) group_norm_groups_kernel(const Args a) {
    __shared__ float red[3][8];
    __shared__ float cols[2][8][33];
    chain_wait();
    const float2 *part = reinterpret_cast<const float2 *>(a.part);
    const int tid = threadIdx.x;
    if ((long long)blockIdx.x < (long long)a.B * a.G) {
        const int b = blockIdx.x / a.G, g = blockIdx.x - b * a.G;
        const long long items = (long long)a.splits * a.Cg;
        const float m = (float)a.N * (float)a.Cg;
        if (BWD) {
            float p = 0.f, q = 0.f;
            for (long long i = tid; i < items; i += 256) {
                const int s = (int)(i / a.Cg), c = g * a.Cg + (int)(i - (long long)s * a.Cg);
                const float2 v = part[((long long)b * a.splits + s) * a.C + c];
                const float gam = a.gamma != nullptr ? __ldg(a.gamma + c) : 1.f;
                p = fmaf(gam, v.x, p);
                q = fmaf(gam, v.y, q);
            }
            p = block_sum(p, red[0]);
            q = block_sum(q, red[1]);
            if (tid == 0) {
                a.coef[2 * (long long)blockIdx.x] = p / m;
                a.coef[2 * (long long)blockIdx.x + 1] = q / m;
            }
        } else {
            Pair w{0.f, 0.f, 0.f};
            for (long long i = tid; i < items; i += 256) {
                const int s = (int)(i / a.Cg), c = g * a.Cg + (int)(i - (long long)s * a.Cg);
                const float2 v = part[((long long)b * a.splits + s) * a.C + c];
                w = merge(w, {(float)min(a.rows, a.N - s * a.rows), v.x, v.y});
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                w = merge(w, {__shfl_xor_sync(0xffffffffu, w.n, o), __shfl_xor_sync(0xffffffffu, w.mean, o),
                              __shfl_xor_sync(0xffffffffu, w.m2, o)});
            if (tid % 32 == 0) red[0][tid / 32] = w.n, red[1][tid / 32] = w.mean, red[2][tid / 32] = w.m2;
            __syncthreads();
            if (tid == 0) {
                Pair r{red[0][0], red[1][0], red[2][0]};
#pragma unroll
                for (int i = 1; i < 8; ++i) r = merge(r, {red[0][i], red[1][i], red[2][i]});
                a.st[2 * (long long)blockIdx.x] = r.mean;
                a.st[2 * (long long)blockIdx.x + 1] = 1.f / sqrtf(r.m2 / m + a.eps);
            }
        }
        return;
    }
    if (BWD) {
        const int x = tid % 32, y = tid / 32;
        const int c = (int)(blockIdx.x - (long long)a.B * a.G) * 32 + x;
        const long long rows = (long long)a.B * a.splits;
        float p = 0.f, q = 0.f;
        if (c < a.C)
            for (long long r = y; r < rows; r += 8) {
                const float2 v = part[r * a.C + c];
                p += v.x;
                q += v.y;
            }
        cols[0][y][x] = p;
        cols[1][y][x] = q;
        __syncthreads();
        if (y == 0 && c < a.C) {
#pragma unroll
            for (int l = 1; l < 8; ++l) p += cols[0][l][x], q += cols[1][l][x];
            if (a.gb != nullptr) a.gb[c] = p;
            if (a.gg != nullptr) a.gg[c] = q;
        }
    }
}

template <typename T, int V, bool BWD>
__global__ void __launch_bounds__(32 * kRowLanes) group_norm_apply_kernel(const Args a) {
    chain_wait();
    const int cb = blockIdx.x % a.cblocks, sb = blockIdx.x / a.cblocks;
    const int b = sb / a.splits, s = sb - b * a.splits;
    const int c = (cb * 32 + threadIdx.x) * V;
    if (c >= a.C) return;
    const int r0 = s * a.rows, r1 = min(a.N, r0 + a.rows);
    const long long base = (long long)b * a.N * a.C + c;
    const float *stats = BWD ? a.stats : a.st;
    float mean[V], rstd[V], gam[V], bet[V], k1[V], k2[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const long long g = (long long)b * a.G + (c + v) / a.Cg;
        mean[v] = stats[2 * g], rstd[v] = stats[2 * g + 1];
        gam[v] = a.gamma != nullptr ? __ldg(a.gamma + c + v) : 1.f;
        bet[v] = a.beta != nullptr ? __ldg(a.beta + c + v) : 0.f;
        if (BWD) k1[v] = a.coef[2 * g], k2[v] = a.coef[2 * g + 1];
    }
    bool bad = false;
#pragma unroll 4
    for (int r = r0 + threadIdx.y; r < r1; r += kRowLanes) {
        float x[V], y[V], dy[V];
        unpack<T, V>(load_raw<V>(a.x + base + (long long)r * a.C), x);
        if (BWD) unpack<T, V>(load_raw<V>(a.dy + base + (long long)r * a.C), dy);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float xh = (x[v] - mean[v]) * rstd[v], z = fmaf(xh, gam[v], bet[v]);
            if (BWD) {
                const float dz = a.act == GTR_ACT_SILU ? dy[v] * act_grad(z) : dy[v];
                y[v] = rstd[v] * (fmaf(gam[v], dz, -k1[v]) - xh * k2[v]);
            } else {
                y[v] = a.act == GTR_ACT_SILU ? z * sigmoid_f(z) : z;
            }
            bad |= Elem<T>::bad(y[v]);
        }
        store_raw<V>(a.out + base + (long long)r * a.C, pack<T, V>(y));
    }
    if (bad) set_error(kOpsErrRange);
}

}  // namespace gn

unsigned norm_take_errors() {
    unsigned word = 0;
    if (cudaMemcpyFromSymbol(&word, g_norm_error_word, sizeof(word)) != cudaSuccess) return kOpsErrCuda;
    if (word != 0) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_norm_error_word, &zero, sizeof(zero)) != cudaSuccess) return kOpsErrCuda;
    }
    return word;
}

// ------------------------------------------------------------------ host
using namespace ops;

static bool bad_sizes(int B, int N, int C, int G) {
    if (B < 0 || N < 0 || C <= 0 || G <= 0 || C % G != 0) return true;
    return N > kMaxTokens || (long long)B * N > kMaxElements / C || (long long)B * C > 0x7fffffffLL;
}

struct NormPlan {
    int splits, rows, cblocks;
};
// Token ranges of at least 64 tokens, enough of them for four blocks an SM.
static NormPlan norm_plan(int B, int N, int C, int V) {
    NormPlan p{};
    p.cblocks = (C + 32 * V - 1) / (32 * V);
    long long splits = (148 * 4 + (long long)B * p.cblocks - 1) / ((long long)B * p.cblocks);
    if (splits > (N + 63) / 64) splits = (N + 63) / 64;
    p.rows = (int)((N + splits - 1) / splits);
    p.splits = (N + p.rows - 1) / p.rows;
    return p;
}
static size_t norm_part_bytes(int B, int N, int C) {
    // the plan of single elements never has more ranges than the one of wide rows
    const int w = norm_plan(B, N, C, 8).splits, n = norm_plan(B, N, C, 1).splits;
    return align256((size_t)B * (w > n ? w : n) * C * 2 * sizeof(float));
}

template <typename T, int V, bool BWD>
static cudaError_t norm_launch(gn::Args a, cudaStream_t s) {
    const NormPlan p = norm_plan(a.B, a.N, a.C, V);
    a.splits = p.splits;
    a.rows = p.rows;
    a.cblocks = p.cblocks;
    const long long blocks = (long long)a.B * p.splits * p.cblocks;
    const long long groups = (long long)a.B * a.G + (BWD && (a.gg || a.gb) ? (a.C + 31) / 32 : 0);
    if (blocks > 0x7fffffffLL || groups > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 thr(32, gn::kRowLanes);
    cudaError_t e = launch_after(gn::group_norm_sums_kernel<T, V, BWD>, (unsigned)blocks, thr, 0, s, a);
    if (e == cudaSuccess) e = launch_after(gn::group_norm_groups_kernel<BWD>, (unsigned)groups, dim3(256), 0, s, a);
    if (e == cudaSuccess) e = launch_after(gn::group_norm_apply_kernel<T, V, BWD>, (unsigned)blocks, thr, 0, s, a);
    return e;
}
template <bool BWD>
static cudaError_t norm_dispatch(const gn::Args &a, int dtype, cudaStream_t s) {
    const bool wide = a.C % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.out, 16) && (!BWD || aligned_to(a.dy, 16));
    if (dtype == GTR_F16) return wide ? norm_launch<__half, 8, BWD>(a, s) : norm_launch<__half, 1, BWD>(a, s);
    return wide ? norm_launch<__nv_bfloat16, 8, BWD>(a, s) : norm_launch<__nv_bfloat16, 1, BWD>(a, s);
}
static bool bad_f32(const void *p, bool required) { return p == nullptr ? required : !aligned_to(p, 16); }

}  // namespace gtr

using namespace gtr;

extern "C" size_t gtr_group_norm_fwd_workspace_bytes(int B, int N, int C, int groups) {
    if (bad_sizes(B, N, C, groups) || B == 0 || N == 0) return 0;
    return norm_part_bytes(B, N, C) + align256((size_t)B * groups * 2 * sizeof(float));
}
extern "C" size_t gtr_group_norm_bwd_workspace_bytes(int B, int N, int C, int groups) {
    return gtr_group_norm_fwd_workspace_bytes(B, N, C, groups);
}

extern "C" gtr_status_t gtr_group_norm_fwd(const void *x, const float *gamma, const float *beta, int B, int N, int C,
                                           int groups, float eps, int dtype, int activation, void *out, float *stats,
                                           void *workspace, size_t workspace_bytes, void *stream) {
    NvtxRange nvtx_range("gtr_group_norm_fwd");
    if (bad_sizes(B, N, C, groups) || (dtype != GTR_F16 && dtype != GTR_BF16) ||
        (activation != GTR_ACT_NONE && activation != GTR_ACT_SILU) || !(eps >= 0.f && eps < 3.4e38f))
        return GTR_ERR_INVALID_ARG;
    const long long n = (long long)B * N * C;
    if (n == 0) return GTR_OK;
    if (!x || !out || !aligned_to(x, 2) || !aligned_to(out, 2) || bad_f32(gamma, false) || bad_f32(beta, false) ||
        bad_f32(stats, false))
        return GTR_ERR_INVALID_ARG;
    const size_t need = gtr_group_norm_fwd_workspace_bytes(B, N, C, groups);
    if (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need) return GTR_ERR_INVALID_ARG;
    const Span outs[] = {{out, n * 2}, {stats, (long long)B * groups * 8}, {workspace, (long long)need}};
    const Span ins[] = {{x, n * 2}, {gamma, (long long)C * 4}, {beta, (long long)C * 4}};
    for (int i = 0; i < 3; ++i) {
        for (int k = 0; k < 3; ++k)
            if (!(i == 0 && k == 0 && x == out) && overlap(outs[i], ins[k])) return GTR_ERR_INVALID_ARG;
        for (int k = i + 1; k < 3; ++k)
            if (overlap(outs[i], outs[k])) return GTR_ERR_INVALID_ARG;
    }
    gn::Args a{};
    a.x = static_cast<const uint16_t *>(x);
    a.gamma = gamma;
    a.beta = beta;
    a.out = static_cast<uint16_t *>(out);
    a.part = static_cast<float *>(workspace);
    a.st = stats != nullptr ? stats : a.part + norm_part_bytes(B, N, C) / sizeof(float);
    a.eps = eps;
    a.B = B;
    a.N = N;
    a.C = C;
    a.G = groups;
    a.Cg = C / groups;
    a.act = activation;
    return ops_cuda_status(norm_dispatch<false>(a, dtype, reinterpret_cast<cudaStream_t>(stream)));
}

extern "C" gtr_status_t gtr_group_norm_bwd(const void *x, const void *d_out, const float *stats, const float *gamma,
                                           const float *beta, int B, int N, int C, int groups, int dtype, int activation,
                                           void *grad_x, float *grad_gamma, float *grad_beta, void *workspace,
                                           size_t workspace_bytes, void *stream) {
    NvtxRange nvtx_range("gtr_group_norm_bwd");
    if (bad_sizes(B, N, C, groups) || (dtype != GTR_F16 && dtype != GTR_BF16) ||
        (activation != GTR_ACT_NONE && activation != GTR_ACT_SILU) || bad_f32(grad_gamma, false) || bad_f32(grad_beta, false))
        return GTR_ERR_INVALID_ARG;
    const long long n = (long long)B * N * C;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (n == 0) {
        if (overlap({grad_gamma, (long long)C * 4}, {grad_beta, (long long)C * 4})) return GTR_ERR_INVALID_ARG;
        cudaError_t e = grad_gamma ? cudaMemsetAsync(grad_gamma, 0, (size_t)C * 4, s) : cudaSuccess;
        if (e == cudaSuccess && grad_beta) e = cudaMemsetAsync(grad_beta, 0, (size_t)C * 4, s);
        return ops_cuda_status(e);
    }
    if (!x || !d_out || !grad_x || !aligned_to(x, 2) || !aligned_to(d_out, 2) || !aligned_to(grad_x, 2) ||
        bad_f32(stats, true) || bad_f32(gamma, false) || bad_f32(beta, false))
        return GTR_ERR_INVALID_ARG;
    const size_t need = gtr_group_norm_bwd_workspace_bytes(B, N, C, groups);
    if (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need) return GTR_ERR_INVALID_ARG;
    const Span outs[] = {{grad_x, n * 2}, {grad_gamma, (long long)C * 4}, {grad_beta, (long long)C * 4},
                         {workspace, (long long)need}};
    const Span ins[] = {{x, n * 2}, {d_out, n * 2}, {stats, (long long)B * groups * 8}, {gamma, (long long)C * 4},
                        {beta, (long long)C * 4}};
    for (int i = 0; i < 4; ++i) {
        for (int k = 0; k < 5; ++k)
            if (overlap(outs[i], ins[k])) return GTR_ERR_INVALID_ARG;
        for (int k = i + 1; k < 4; ++k)
            if (overlap(outs[i], outs[k])) return GTR_ERR_INVALID_ARG;
    }
    gn::Args a{};
    a.x = static_cast<const uint16_t *>(x);
    a.dy = static_cast<const uint16_t *>(d_out);
    a.stats = stats;
    a.gamma = gamma;
    a.beta = beta;
    a.out = static_cast<uint16_t *>(grad_x);
    a.gg = grad_gamma;
    a.gb = grad_beta;
    a.part = static_cast<float *>(workspace);
    a.coef = a.part + norm_part_bytes(B, N, C) / sizeof(float);
    a.B = B;
    a.N = N;
    a.C = C;
    a.G = groups;
    a.Cg = C / groups;
    a.act = activation;
    return ops_cuda_status(norm_dispatch<true>(a, dtype, s));
}
