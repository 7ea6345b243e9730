// group_norm.cu -- the channels-last group norm behind the C ABI of include/gtr_norm.h.
//
// Forward: z = (x - mean) rstd gamma + beta, out = act(z).  Backward, with dz = d_out act'(z), the
// per-channel sums P = sum dz, Q = sum dz xhat over the tokens of a batch entry and the M = N C / G
// elements of a group:
//     grad_x = rstd (gamma dz - (sum_group gamma P + xhat sum_group gamma Q) / M)
//     grad_gamma = sum_b Q,  grad_beta = sum_b P
// A few operations for 4 bytes moved (6 backward): HBM-bound, and what costs is reading the
// activations once for the sums and again for the result.
#include <type_traits>

#include "../../include/gtr_norm.h"
#include "ops_common.cuh"

namespace gtr {
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
    float *fig;                          // figures of the groups by token range
    int parts;                           // blocks along the channels that share a group
    int st_wanted;                       // forward: st is the caller's
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

// ------------------------------------------------------------------ groups of whole pieces: two launches
// Channels come in pieces of 8 (16 bytes), groups in whole pieces.  A block: a range of tokens by up to 32
// neighbouring pieces, whole groups of them (or a part of one group), a warp a token, so that a warp
// reads up to 512 consecutive bytes; each thread asks for several of its rows at once.  The first
// launch leaves every block's figures of its groups (forward: mean and deviations; backward: the sums of gamma P
// and gamma Q, and P and Q by channel); in the second launch every block joins its groups' figures
// over the token ranges itself, then writes the results.  The activations are read twice, the second
// time from L2 as far as they fit.  (Holding them on chip in between, the tokens shared out over a
// cluster's blocks, reads them once but took longer, the blocks of a cluster waiting for one another:
// 40 us for 26 at 16384 tokens of 1024 channels, 105 for 82 backward at 8 x 2304 of 2048.)  Those
// two sizes now: 25 us, and 83 us, 4.5 TB/s over both readings.
constexpr int kLanes = 8, kEntries = 4;   // tokens in step; entries of a group that a lane joins at most
struct Piece {
    int first, n, ngroups, cpg;   // the block's first piece, its pieces, its groups, pieces of a group in it
    int g0, entry;                // its first group, its first entry of a token range's figures
};
__device__ __forceinline__ Piece piece_of(const Args &a, int cb) {
    const int cpg = a.Cg / 8, all = a.C / 8;
    if (cpg <= 32) {
        const int gpb = 32 / cpg, g0 = cb * gpb;
        const int first = g0 * cpg, n = min(gpb * cpg, all - first);
        return {first, n, n / cpg, cpg, g0, g0};
    }
    const int g0 = cb / a.parts, q = cb - g0 * a.parts;
    return {g0 * cpg + q * 32, min(32, cpg - q * 32), 1, min(32, cpg - q * 32), g0, cb};
}
// Channels of entry q of a group.
__device__ __forceinline__ float entry_channels(const Args &a, int q) {
    return (float)(a.parts == 1 ? a.Cg : 8 * min(32, a.Cg / 8 - q * 32));
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Joins group g's figures over the token ranges (a warp): forward (mean, rstd), backward the two
// sums over M, in every lane.
template <bool BWD>
__device__ __forceinline__ float2 join(const Args &a, int b, int g, int lane) {
    const int items = a.splits * a.parts, E = a.G * a.parts;
    const float2 *src = reinterpret_cast<const float2 *>(a.fig) + (long long)b * a.splits * E + (long long)g * a.parts;
    const float m = (float)a.N * (float)a.Cg;
    float2 v[kEntries];
    float n[kEntries];
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        const int k = lane + 32 * i, s = k / a.parts, q = k - s * a.parts;
        n[i] = k < items ? (float)min(a.rows, a.N - s * a.rows) * entry_channels(a, q) : 0.f;
        v[i] = k < items ? src[(long long)s * E + q] : splat(0.f);
    }
    if (BWD) {
        float2 t = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
        return make_float2(warp_sum(t.x) / m, warp_sum(t.y) / m);
    }
    float t = 0.f, q = 0.f;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) t = fmaf(n[i], v[i].x, t);
    const float mean = warp_sum(t) / m;
#pragma unroll
    for (int i = 0; i < kEntries; ++i) {
        const float d = v[i].x - mean;
        q += fmaf(n[i] * d, d, v[i].y);
    }
    return make_float2(mean, 1.f / sqrtf(warp_sum(q) / m + a.eps));
}

template <typename T>
__device__ __forceinline__ void halves(const Raw<8> &r, float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = Elem<T>::get2(r.w[i]);
}
__device__ __forceinline__ void params4(const float *p, int c, float none, float2 (&f)[4]) {
    const float4 *q = reinterpret_cast<const float4 *>(p + c);
    const float4 lo = p != nullptr ? __ldg(q) : make_float4(none, none, none, none);
    const float4 hi = p != nullptr ? __ldg(q + 1) : lo;
    f[0] = make_float2(lo.x, lo.y), f[1] = make_float2(lo.z, lo.w), f[2] = make_float2(hi.x, hi.y), f[3] = make_float2(hi.z, hi.w);
}
// d_out times the activation's slope at z, in pairs.
__device__ __forceinline__ float2 slope(float2 dy, float2 z) {
    const float2 s = make_float2(sigmoid_f(z.x), sigmoid_f(z.y));
    const float2 one = __ffma2_rn(z, __fadd2_rn(splat(1.f), make_float2(-s.x, -s.y)), splat(1.f));
    return __fmul2_rn(dy, __fmul2_rn(s, one));
}

template <typename T, bool BWD, bool SILU>
__global__ void __launch_bounds__(32 * kLanes, 3) group_norm_figures_kernel(const Args a) {
    constexpr int AT = BWD ? 2 : 4;   // rows of a batch; the next batch is asked for before one is used
    __shared__ float red[kLanes][32][BWD ? 17 : 3];
    __shared__ float2 chan[32 * 8];
    chain_wait();
    const int cb = blockIdx.x % a.cblocks, sb = blockIdx.x / a.cblocks;
    const int b = sb / a.splits, s = sb - b * a.splits;
    const Piece pc = piece_of(a, cb);
    const int x = threadIdx.x, y = threadIdx.y, tid = y * 32 + x;
    const int c = (pc.first + x) * 8;
    const int r0 = s * a.rows, r1 = min(a.N, r0 + a.rows);
    const bool live = x < pc.n;
    const long long base = (long long)b * a.N * a.C + c;
    float mean = 0.f, rstd = 0.f;
    float2 gam[4], bet[4], P[4], Q[4];
    float tn = 0.f, tm = 0.f, tq = 0.f;
    if (BWD) {
#pragma unroll
        for (int v = 0; v < 4; ++v) P[v] = Q[v] = splat(0.f);
        if (live) {
            const float *st = a.stats + 2 * ((long long)b * a.G + c / a.Cg);
            mean = __ldg(st), rstd = __ldg(st + 1);
            params4(a.gamma, c, 1.f, gam);
            params4(a.beta, c, 0.f, bet);
        }
    }
    Raw<8> rx[AT], rd[AT], nx[AT], nd[AT];
    auto fetch = [&](int r) {
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            const bool in = live && r + u * kLanes < r1;
            nx[u] = in ? load_raw<8>(a.x + base + (long long)(r + u * kLanes) * a.C) : zero_raw<8>();
            if (BWD) nd[u] = in ? load_raw<8>(a.dy + base + (long long)(r + u * kLanes) * a.C) : zero_raw<8>();
        }
    };
    fetch(r0 + y);
    for (int r = r0 + y; live && r < r1; r += kLanes * AT) {
        const int k = min((r1 - r + kLanes - 1) / kLanes, AT);
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            rx[u] = nx[u];
            if (BWD) rd[u] = nd[u];
        }
        fetch(r + kLanes * AT);
        if (BWD) {
#pragma unroll
            for (int u = 0; u < AT; ++u) {
                if (u >= k) break;   // a whole warp
                float2 f[4], dz[4];
                halves<T>(rx[u], f);
                halves<T>(rd[u], dz);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float2 xh = __fmul2_rn(__fadd2_rn(f[v], splat(-mean)), splat(rstd));
                    if (SILU) dz[v] = slope(dz[v], __ffma2_rn(xh, gam[v], bet[v]));
                    P[v] = __fadd2_rn(P[v], dz[v]);
                    Q[v] = __ffma2_rn(dz[v], xh, Q[v]);
                }
            }
        } else {
            // the rows' mean and the deviations from it, merged into the running pair
            float2 t = splat(0.f), q2 = splat(0.f);
#pragma unroll
            for (int u = 0; u < AT; ++u) {   // the rows that are not there are zeros
                float2 f[4];
                halves<T>(rx[u], f);
                t = __fadd2_rn(t, __fadd2_rn(__fadd2_rn(f[0], f[1]), __fadd2_rn(f[2], f[3])));
            }
            const float n = (float)(8 * k), m = (t.x + t.y) / n;
#pragma unroll
            for (int u = 0; u < AT; ++u) {
                if (u >= k) break;
                float2 f[4];
                halves<T>(rx[u], f);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const float2 d = __fadd2_rn(f[v], splat(-m));
                    q2 = __ffma2_rn(d, d, q2);
                }
            }
            const float d = m - tm, w = n / (tn + n);
            tq += q2.x + q2.y + d * d * tn * w;
            tm = fmaf(d, w, tm);
            tn += n;
        }
    }
    if (BWD) {
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            red[y][x][2 * v] = P[v].x, red[y][x][2 * v + 1] = P[v].y;
            red[y][x][8 + 2 * v] = Q[v].x, red[y][x][8 + 2 * v + 1] = Q[v].y;
        }
        __syncthreads();
        {   // a channel a thread, over the tokens in step
            float2 t = splat(0.f);
#pragma unroll
            for (int l = 0; l < kLanes; ++l)
                t = __fadd2_rn(t, make_float2(red[l][tid / 8][tid % 8], red[l][tid / 8][8 + tid % 8]));
            const int ch = pc.first * 8 + tid;
            if (tid < pc.n * 8) {
                if (a.part != nullptr) reinterpret_cast<float2 *>(a.part)[((long long)b * a.splits + s) * a.C + ch] = t;
                chan[tid] = __fmul2_rn(t, splat(a.gamma != nullptr ? __ldg(a.gamma + ch) : 1.f));
            }
        }
        __syncthreads();
        for (int g = y; g < pc.ngroups; g += kLanes) {
            float2 t = splat(0.f);
            for (int i = x; i < pc.cpg * 8; i += 32) t = __fadd2_rn(t, chan[g * pc.cpg * 8 + i]);
            t = make_float2(warp_sum(t.x), warp_sum(t.y));
            if (x == 0) reinterpret_cast<float2 *>(a.fig)[((long long)b * a.splits + s) * a.G * a.parts + pc.entry + g] = t;
        }
        return;
    }
    red[y][x][0] = tn, red[y][x][1] = tm, red[y][x][2] = tq;
    __syncthreads();
    for (int g = y; g < pc.ngroups; g += kLanes) {   // a group a warp: the mean of the means, the deviations from it
        const int items = kLanes * pc.cpg;           // 256 at most
        float n = 0.f, m = 0.f, q = 0.f;
        for (int i = x; i < items; i += 32) {
            const float *e = red[i / pc.cpg][g * pc.cpg + i % pc.cpg];
            n += e[0];
            m = fmaf(e[0], e[1], m);
        }
        n = warp_sum(n);
        m = warp_sum(m) / n;
        for (int i = x; i < items; i += 32) {
            const float *e = red[i / pc.cpg][g * pc.cpg + i % pc.cpg];
            if (e[0] > 0.f) q += fmaf((e[1] - m) * (e[1] - m), e[0], e[2]);
        }
        q = warp_sum(q);
        if (x == 0)
            reinterpret_cast<float2 *>(a.fig)[((long long)b * a.splits + s) * a.G * a.parts + pc.entry + g] = make_float2(m, q);
    }
}

// The results.  Backward, the blocks behind `blocks` add up grad_gamma and grad_beta, 32 channels a
// block, over batch entries and token ranges in a fixed order.
template <typename T, bool BWD, bool SILU>
__global__ void __launch_bounds__(32 * kLanes, 3) group_norm_results_kernel(const Args a, int blocks) {
    constexpr int AT = 2;   // rows of a batch; the next batch is asked for before one is used
    __shared__ float2 fig[32];
    __shared__ float2 cols[kLanes][33];
    chain_wait();
    const int x = threadIdx.x, y = threadIdx.y;
    if (BWD && (int)blockIdx.x >= blocks) {
        const int c = ((int)blockIdx.x - blocks) * 32 + x;
        const int rows = a.B * a.splits;
        float2 t = splat(0.f);
        if (c < a.C)
#pragma unroll 8
            for (int r = y; r < rows; r += kLanes) t = __fadd2_rn(t, reinterpret_cast<const float2 *>(a.part)[(long long)r * a.C + c]);
        cols[y][x] = t;
        __syncthreads();
        if (y == 0 && c < a.C) {
#pragma unroll
            for (int l = 1; l < kLanes; ++l) t = __fadd2_rn(t, cols[l][x]);
            if (a.gb != nullptr) a.gb[c] = t.x;
            if (a.gg != nullptr) a.gg[c] = t.y;
        }
        return;
    }
    const int cb = blockIdx.x % a.cblocks, sb = blockIdx.x / a.cblocks;
    const int b = sb / a.splits, s = sb - b * a.splits;
    const Piece pc = piece_of(a, cb);
    const int c = (pc.first + x) * 8;
    const int r0 = s * a.rows, r1 = min(a.N, r0 + a.rows);
    const bool live = x < pc.n;
    const long long base = (long long)b * a.N * a.C + c;
    Raw<8> rx[AT], rd[AT], nx[AT], nd[AT];
    auto fetch = [&](int r) {   // x by plain loads: out may be x
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            const bool in = live && r + u * kLanes < r1;
            nx[u] = in ? load_plain<8>(a.x + base + (long long)(r + u * kLanes) * a.C) : zero_raw<8>();
            if (BWD) nd[u] = in ? load_raw<8>(a.dy + base + (long long)(r + u * kLanes) * a.C) : zero_raw<8>();
        }
    };
    fetch(r0 + y);
    for (int g = y; g < pc.ngroups; g += kLanes) {
        const float2 f = join<BWD>(a, b, pc.g0 + g, x);
        if (x == 0) {
            fig[g] = f;
            // one block a group writes the statistics: of the first token range, of the group's first part
            if (!BWD && s == 0 && a.st != nullptr && (a.parts == 1 || cb % a.parts == 0))
                reinterpret_cast<float2 *>(a.st)[(long long)b * a.G + pc.g0 + g] = f;
        }
    }
    __syncthreads();
    if (!live) return;
    const float2 f = fig[x / pc.cpg];
    float2 gam[4], bet[4];
    params4(a.gamma, c, 1.f, gam);
    params4(a.beta, c, 0.f, bet);
    float mean = f.x, rstd = f.y;
    if (BWD) {
        const float *st = a.stats + 2 * ((long long)b * a.G + c / a.Cg);
        mean = __ldg(st), rstd = __ldg(st + 1);
    }
    uint32_t worst = 0;
    for (int r = r0 + y; r < r1; r += kLanes * AT) {
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            rx[u] = nx[u];
            if (BWD) rd[u] = nd[u];
        }
        fetch(r + kLanes * AT);
        Raw<8> o[AT];
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            float2 h[4], dz[4];
            halves<T>(rx[u], h);
            if (BWD) halves<T>(rd[u], dz);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
                const float2 xh = __fmul2_rn(__fadd2_rn(h[v], splat(-mean)), splat(rstd));
                const float2 z = __ffma2_rn(xh, gam[v], bet[v]);
                float2 q = z;
                if (BWD) {
                    if (SILU) dz[v] = slope(dz[v], z);
                    q = __ffma2_rn(xh, splat(-f.y), __ffma2_rn(gam[v], dz[v], splat(-f.x)));
                    q = __fmul2_rn(splat(rstd), q);
                } else if (SILU) {
                    q = __fmul2_rn(z, make_float2(sigmoid_f(z.x), sigmoid_f(z.y)));
                }
                o[u].w[v] = Elem<T>::put2(q.x, q.y);
            }
        }
#pragma unroll
        for (int u = 0; u < AT; ++u)
            if (r + u * kLanes < r1) {
#pragma unroll
                for (int v = 0; v < 4; ++v) worst = Elem<T>::worst(worst, o[u].w[v]);
                store_raw<8>(a.out + base + (long long)(r + u * kLanes) * a.C, o[u]);
            }
    }
    if (Elem<T>::bad_raw(worst)) set_error(kOpsErrRange);
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
    __shared__ float red[2][8];
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
            // the mean of the means, then the deviations from it: no division in the loops
            auto each = [&](auto f) {
#pragma unroll 8
                for (long long i = tid; i < items; i += 256) {
                    const int s = (int)(i / a.Cg), c = g * a.Cg + (int)(i - (long long)s * a.Cg);
                    f((float)min(a.rows, a.N - s * a.rows), part[((long long)b * a.splits + s) * a.C + c]);
                }
            };
            float t = 0.f, q = 0.f;
            each([&](float n, float2 v) { t = fmaf(n, v.x, t); });
            const float mean = block_sum(t, red[0]) / m;
            each([&](float n, float2 v) {
                const float d = v.x - mean;
                q += fmaf(n * d, d, v.y);
            });
            q = block_sum(q, red[1]);
            if (tid == 0) {
                a.st[2 * (long long)blockIdx.x] = mean;
                a.st[2 * (long long)blockIdx.x + 1] = 1.f / sqrtf(q / m + a.eps);
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
    uint32_t worst = 0;
    // `count` rows from r on, asked for at once: x by plain loads, since out may be x forward, so that a load
    // stays ahead of the stores behind it
    auto rows = [&](auto count, int r) {
        constexpr int AT = decltype(count)::value;
        Raw<V> rx[AT], rd[AT];
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            const long long at = base + (long long)(r + u * kRowLanes) * a.C;
            rx[u] = load_plain<V>(a.x + at);
            if (BWD) rd[u] = load_raw<V>(a.dy + at);
        }
#pragma unroll
        for (int u = 0; u < AT; ++u) {
            float x[V], y[V], dy[V];
            unpack<T, V>(rx[u], x);
            if (BWD) unpack<T, V>(rd[u], dy);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float xh = (x[v] - mean[v]) * rstd[v], z = fmaf(xh, gam[v], bet[v]);
                if (BWD) {
                    const float dz = a.act == GTR_ACT_SILU ? dy[v] * act_grad(z) : dy[v];
                    y[v] = rstd[v] * (fmaf(gam[v], dz, -k1[v]) - xh * k2[v]);
                } else {
                    y[v] = a.act == GTR_ACT_SILU ? z * sigmoid_f(z) : z;
                }
            }
            const Raw<V> o = pack<T, V>(y);
#pragma unroll
            for (const uint32_t w : o.w) worst = Elem<T>::worst(worst, w);
            store_raw<V>(a.out + base + (long long)(r + u * kRowLanes) * a.C, o);
        }
    };
    int r = r0 + threadIdx.y;
    for (; r + 3 * kRowLanes < r1; r += 4 * kRowLanes) rows(std::integral_constant<int, 4>{}, r);
    for (; r < r1; r += kRowLanes) rows(std::integral_constant<int, 1>{}, r);
    if (Elem<T>::bad_raw(worst)) set_error(kOpsErrRange);
}

}  // namespace gn

unsigned *norm_error_word() { return error_word(); }

// ------------------------------------------------------------------ host
using namespace ops;

static bool bad_sizes(int B, int N, int C, int G) {
    if (B < 0 || N < 0 || C <= 0 || G <= 0 || C % G != 0) return true;
    return N > kMaxTokens || C > kMaxChannels || (long long)B * N > kMaxElements / C || (long long)B * C > 0x7fffffffLL;
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
static size_t piece_bytes(int B, int N, int C, int G);
static size_t norm_part_bytes(int B, int N, int C, int G) {   // whichever way the tensors' alignment leads
    const int w = norm_plan(B, N, C, 8).splits, n = norm_plan(B, N, C, 1).splits;
    const size_t any = align256((size_t)B * (w > n ? w : n) * C * 2 * sizeof(float)), pieces = piece_bytes(B, N, C, G);
    return any > pieces ? any : pieces;
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
struct PiecePlan {
    int parts, cblocks, splits, rows;
};
// Groups of whole pieces.  Token ranges: three blocks an SM in one wave, 32 tokens at least, and no
// more than a warp joins (kEntries a lane).
static bool piece_plan(int B, int N, int C, int G, PiecePlan *p) {
    const int Cg = C / G, cpg = Cg / 8;
    if (Cg % 8 != 0 || cpg > 32 * 32 * gn::kEntries) return false;
    p->parts = cpg <= 32 ? 1 : (cpg + 31) / 32;
    p->cblocks = cpg <= 32 ? (G + 32 / cpg - 1) / (32 / cpg) : G * p->parts;
    long long splits = 148 * 3 / ((long long)B * p->cblocks);
    const long long most = 32 * gn::kEntries / p->parts;
    if (splits > (N + 31) / 32) splits = (N + 31) / 32;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    p->rows = (int)((N + splits - 1) / splits);
    p->splits = (N + p->rows - 1) / p->rows;
    return true;
}
static size_t piece_fig_bytes(int B, int G, const PiecePlan &p) {
    return align256((size_t)B * p.splits * G * p.parts * 2 * sizeof(float));
}
static size_t piece_bytes(int B, int N, int C, int G) {
    PiecePlan p{};
    if (!piece_plan(B, N, C, G, &p)) return 0;
    return piece_fig_bytes(B, G, p) + align256((size_t)B * p.splits * C * 2 * sizeof(float));
}

template <typename T, bool BWD, bool SILU>
static cudaError_t piece_launch(gn::Args a, const PiecePlan &p, cudaStream_t s) {
    a.fig = a.part;
    a.part = BWD && (a.gg != nullptr || a.gb != nullptr) ? a.part + piece_fig_bytes(a.B, a.G, p) / sizeof(float) : nullptr;
    a.parts = p.parts;
    a.cblocks = p.cblocks;
    a.splits = p.splits;
    a.rows = p.rows;
    if (a.st_wanted == 0) a.st = nullptr;
    const long long blocks = (long long)a.B * p.splits * p.cblocks;
    const long long params = a.part != nullptr ? (a.C + 31) / 32 : 0;
    if (blocks + params > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    const dim3 thr(32, gn::kLanes);
    const cudaError_t e = launch_after(gn::group_norm_figures_kernel<T, BWD, SILU>, (unsigned)blocks, thr, 0, s, a);
    if (e != cudaSuccess) return e;
    return launch_after(gn::group_norm_results_kernel<T, BWD, SILU>, (unsigned)(blocks + params), thr, 0, s, a, (int)blocks);
}

template <bool BWD>
static cudaError_t norm_dispatch(const gn::Args &a, int dtype, cudaStream_t s) {
    const bool wide = a.C % 8 == 0 && aligned_to(a.x, 16) && aligned_to(a.out, 16) && (!BWD || aligned_to(a.dy, 16));
    PiecePlan pp{};
    if (wide && piece_plan(a.B, a.N, a.C, a.G, &pp)) {
        const bool silu = a.act == GTR_ACT_SILU;
        if (dtype == GTR_F16) return silu ? piece_launch<__half, BWD, true>(a, pp, s) : piece_launch<__half, BWD, false>(a, pp, s);
        return silu ? piece_launch<__nv_bfloat16, BWD, true>(a, pp, s) : piece_launch<__nv_bfloat16, BWD, false>(a, pp, s);
    }
    if (dtype == GTR_F16) return wide ? norm_launch<__half, 8, BWD>(a, s) : norm_launch<__half, 1, BWD>(a, s);
    return wide ? norm_launch<__nv_bfloat16, 8, BWD>(a, s) : norm_launch<__nv_bfloat16, 1, BWD>(a, s);
}

}  // namespace gtr

using namespace gtr;

extern "C" size_t gtr_group_norm_fwd_workspace_bytes(int B, int N, int C, int groups) {
    if (bad_sizes(B, N, C, groups) || B == 0 || N == 0) return 0;
    return norm_part_bytes(B, N, C, groups) + align256((size_t)B * groups * 2 * sizeof(float));
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
    a.st_wanted = stats != nullptr;
    a.st = stats != nullptr ? stats : a.part + norm_part_bytes(B, N, C, groups) / sizeof(float);
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
    a.coef = a.part + norm_part_bytes(B, N, C, groups) / sizeof(float);
    a.B = B;
    a.N = N;
    a.C = C;
    a.G = groups;
    a.Cg = C / groups;
    a.act = activation;
    return ops_cuda_status(norm_dispatch<true>(a, dtype, s));
}
