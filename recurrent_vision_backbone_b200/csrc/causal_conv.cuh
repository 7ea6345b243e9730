// causal_conv.cuh -- the short causal convolution over the scan order, forward and backward
// (included by ssm.cu, which holds the C entry points).
//
// Over scan positions p of one sequence, with X = [K - 1 earlier inputs ; x],
//     s_p = bias + sum_{j<K} w[j] X[p + j],   out_p = act(s_p)
// and, ds_p = d_out_p act'(s_p) (0 outside the sequence),
//     dX[r] = sum_j w[j] ds[r - j] (+ d_final on the last K - 1 rows),
//     dw[j] = sum_p ds_p X[p + j],   dbias = sum_p ds_p.
// K is 2 to 4: 2 K operations for 4 bytes moved (6 backward), so HBM-bound.
#pragma once

namespace gtr {
namespace cv {

using namespace ops;

constexpr int kThreads = 128;

struct Args {
    const uint16_t *x, *init, *dy, *dfin;
    const float *w, *bias;
    uint16_t *out, *fin;            // forward
    uint16_t *dx, *dinit;           // backward
    float *part;                    // [parts][K + 1][D] sums of ds X (K rows) and of ds
    long long ldx, lddy;
    int B, H, W, N, D, dir, act;
    int groups;                     // channel groups of V
    int tile, tiles;                // positions per thread, tiles per sequence
    int parts;                      // backward: blocks along the positions
};

// Row r of X (r counts from the K - 1 earlier inputs) at channels c .. c + V - 1.
template <int V>
__device__ __forceinline__ Raw<V> early_row(const Args &a, int b, int r, int K, int c) {
    return a.init != nullptr ? load_raw<V>(a.init + ((long long)b * (K - 1) + r) * a.D + c) : zero_raw<V>();
}

// One thread: V channels, `TP` consecutive scan positions; every row it needs (TP + K - 1) is
// requested before the first is used, so a thread waits for memory once.  Threads run along the
// channels, so a warp reads whole lines of each row whatever the scan order.
template <typename T, int V, int K, int TP>
__global__ void __launch_bounds__(kThreads) causal_conv_fwd_kernel(const Args a) {
    chain_wait();
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const int g = (int)(id % a.groups);
    const long long t = id / a.groups;
    const int b = (int)(t / a.tiles);
    if (b >= a.B) return;
    const int tile = (int)(t - (long long)b * a.tiles);
    const int c = g * V, p0 = tile * TP;
    const long long row0 = (long long)b * a.N;
    Raw<V> x[TP + K - 1];
    int tok[TP];
#pragma unroll
    for (int r = 0; r < K - 1; ++r) {
        const int p = p0 - (K - 1) + r;
        x[r] = p >= 0 ? load_raw<V>(a.x + (row0 + token_of(p, a.H, a.W, a.dir)) * a.ldx + c) : early_row<V>(a, b, r, K, c);
    }
    {
        Walk wk(p0, a.H, a.W, a.dir);
#pragma unroll
        for (int i = 0; i < TP; ++i) {
            tok[i] = wk.n;
            x[K - 1 + i] = p0 + i < a.N ? load_raw<V>(a.x + (row0 + tok[i]) * a.ldx + c) : zero_raw<V>();
            wk.next();
        }
    }
    // tile 0 also writes the carried rows: the last K - 1 of X.  The rows it needs of
    // init_state are in registers by then, so final_state may be init_state
    if (tile == 0 && a.fin != nullptr) {
        Raw<V> f[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            const int r = a.N + j;   // row of X
            f[j] = r >= K - 1 ? load_raw<V>(a.x + (row0 + token_of(r - (K - 1), a.H, a.W, a.dir)) * a.ldx + c)
                              : early_row<V>(a, b, r, K, c);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j) store_raw<V>(a.fin + ((long long)b * (K - 1) + j) * a.D + c, f[j]);
    }
    float w[V][K], bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < K; ++j) w[v][j] = __ldg(a.w + (long long)(c + v) * K + j);
        bias[v] = a.bias != nullptr ? __ldg(a.bias + c + v) : 0.f;
    }
    float win[K][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) unpack<T, V>(x[j], win[j]);
    bool bad = false;
#pragma unroll
    for (int i = 0; i < TP; ++i) {
        unpack<T, V>(x[K - 1 + i], win[K - 1]);
        float y[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            float s = bias[v];
#pragma unroll
            for (int j = 0; j < K; ++j) s = fmaf(w[v][j], win[j][v], s);
            y[v] = a.act == GTR_ACT_SILU ? s * sigmoid_f(s) : s;
            bad |= p0 + i < a.N && Elem<T>::bad(y[v]);
        }
        if (p0 + i < a.N) store_raw<V>(a.out + (row0 + tok[i]) * a.D + c, pack<T, V>(y));
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) win[j][v] = win[j + 1][v];
    }
    if (bad) set_error(kOpsErrRange);
}

// Backward.  A block: 32 channel groups (threadIdx.x) by kLanes position lanes (threadIdx.y);
// a lane walks `tile` positions and the K - 1 behind them (whose ds its last outputs need),
// keeping the last K rows of X and of ds in registers and its share of dw and dbias; the lanes'
// shares meet in shared memory and the block writes one partial row, so that the sum over
// tokens has a fixed order.  Rows are requested kAhead steps before they are used.
constexpr int kLanes = 8, kAhead = 4;
template <typename T, int V, int K>
__global__ void __launch_bounds__(32 * kLanes) causal_conv_bwd_kernel(const Args a) {
    __shared__ float red[kLanes][32][V];
    chain_wait();
    const int g = blockIdx.x % ((a.groups + 31) / 32) * 32 + threadIdx.x;
    const int part = blockIdx.x / ((a.groups + 31) / 32);
    const long long t = (long long)part * kLanes + threadIdx.y;
    const int b = (int)(t / a.tiles);
    const bool live = g < a.groups && b < a.B;
    const int c = g * V;
    float acc[K + 1][V];
#pragma unroll
    for (int j = 0; j <= K; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) acc[j][v] = 0.f;
    bool bad = false;
    if (live) {
        const int tile = (int)(t - (long long)b * a.tiles), p0 = tile * a.tile;
        const int p1 = min(p0 + a.tile, a.N);            // own positions: p0 .. p1 - 1
        const int pe = p1 + K - 1;                       // rows of dX reached at steps p0 .. pe - 1
        const long long row0 = (long long)b * a.N;
        float w[V][K], bias[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int j = 0; j < K; ++j) w[v][j] = __ldg(a.w + (long long)(c + v) * K + j);
            bias[v] = a.bias != nullptr ? __ldg(a.bias + c + v) : 0.f;
        }
        float xw[K][V], dw[K][V];   // rows p .. p + K - 1 of X; ds of positions p - K + 1 .. p
#pragma unroll
        for (int r = 0; r < K - 1; ++r) {
            const int p = p0 - (K - 1) + r;
            unpack<T, V>(p >= 0 ? load_raw<V>(a.x + (row0 + token_of(p, a.H, a.W, a.dir)) * a.ldx + c)
                                : early_row<V>(a, b, r, K, c), xw[r]);
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v) dw[j][v] = 0.f;
        Walk ahead(p0, a.H, a.W, a.dir), behind(max(p0 - (K - 1), 0), a.H, a.W, a.dir);
        Raw<V> qx[kAhead], qd[kAhead];
        auto fetch = [&](int p, int i) {
            const bool in = p < a.N && p < pe;
            qx[i] = in ? load_raw<V>(a.x + (row0 + ahead.n) * a.ldx + c) : zero_raw<V>();
            qd[i] = in ? load_raw<V>(a.dy + (row0 + ahead.n) * a.lddy + c) : zero_raw<V>();
            ahead.next();
        };
#pragma unroll
        for (int i = 0; i < kAhead; ++i) fetch(p0 + i, i);
        for (int pb = p0; pb < pe; pb += kAhead) {
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int p = pb + i;
                if (p >= pe) break;
                float dy[V];
                unpack<T, V>(qx[i], xw[K - 1]);
                unpack<T, V>(qd[i], dy);
                fetch(p + kAhead, i);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float d = dy[v];
                    if (a.act == GTR_ACT_SILU) {
                        float s = bias[v];
#pragma unroll
                        for (int j = 0; j < K; ++j) s = fmaf(w[v][j], xw[j][v], s);
                        const float sg = sigmoid_f(s);
                        d *= sg * fmaf(s, 1.f - sg, 1.f);
                    }
                    // behind the sequence there is no ds (not 0 times what the activation makes of X)
                    dw[K - 1][v] = p < a.N ? d : 0.f;
                }
                if (p < p1) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
#pragma unroll
                        for (int j = 0; j < K; ++j) acc[j][v] = fmaf(dw[K - 1][v], xw[j][v], acc[j][v]);
                        acc[K][v] += dw[K - 1][v];
                    }
                }
                // row p of dX: position p - (K - 1), or an earlier input where p < K - 1
                const bool own = p >= p0 + K - 1, first = p0 == 0 && p < K - 1;
                if (own || (first && a.dinit != nullptr)) {
                    float e[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        e[v] = 0.f;
#pragma unroll
                        for (int j = 0; j < K; ++j) e[v] = fmaf(w[v][j], dw[K - 1 - j][v], e[v]);
                    }
                    if (a.dfin != nullptr && p >= a.N) {
                        float f[V];
                        unpack<T, V>(load_raw<V>(a.dfin + ((long long)b * (K - 1) + p - a.N) * a.D + c), f);
#pragma unroll
                        for (int v = 0; v < V; ++v) e[v] += f[v];
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) bad |= Elem<T>::bad(e[v]);
                    if (own)
                        store_raw<V>(a.dx + (row0 + behind.n) * a.D + c, pack<T, V>(e));
                    else
                        store_raw<V>(a.dinit + ((long long)b * (K - 1) + p) * a.D + c, pack<T, V>(e));
                }
                if (p >= K - 1) behind.next();
#pragma unroll
                for (int j = 0; j < K - 1; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        xw[j][v] = xw[j + 1][v];
                        dw[j][v] = dw[j + 1][v];
                    }
            }
        }
    }
    if (bad) set_error(kOpsErrRange);
#pragma unroll
    for (int j = 0; j <= K; ++j) {
        __syncthreads();
#pragma unroll
        for (int v = 0; v < V; ++v) red[threadIdx.y][threadIdx.x][v] = acc[j][v];
        __syncthreads();
        for (int i = threadIdx.y * 32 + threadIdx.x; i < 32 * V; i += 32 * kLanes) {
            const int ch = (blockIdx.x % ((a.groups + 31) / 32)) * 32 * V + i;
            if (ch < a.D) {
                float s = 0.f;
#pragma unroll
                for (int l = 0; l < kLanes; ++l) s += red[l][i / V][i % V];
                a.part[((long long)part * (K + 1) + j) * a.D + ch] = s;
            }
        }
    }
}

// dw[d][j] and dbias[d]: the partial rows added in order.  A block: 32 columns of the
// [K + 1][D] sums by 8 row lanes.
template <int K>
__global__ void __launch_bounds__(256) causal_conv_sum_kernel(const float *part, int parts, int D, float *gw, float *gb) {
    __shared__ float red[8][33];
    chain_wait();
    const long long cols = (long long)(K + 1) * D, col = (long long)blockIdx.x * 32 + threadIdx.x;
    float s = 0.f;
    if (col < cols)
        for (int r = threadIdx.y; r < parts; r += 8) s += part[r * cols + col];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && col < cols) {
#pragma unroll
        for (int l = 1; l < 8; ++l) s += red[l][threadIdx.x];
        const int j = (int)(col / D), d = (int)(col - (long long)j * D);
        if (j < K)
            gw[(long long)d * K + j] = s;
        else if (gb != nullptr)
            gb[d] = s;
    }
}

}  // namespace cv
}  // namespace gtr
