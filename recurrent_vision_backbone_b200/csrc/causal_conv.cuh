// causal_conv.cuh -- the short causal convolution over the scan order, forward and backward
// (included by causal_conv.cu, which holds the C entry points).
//
// Over scan positions p of one sequence, with X = [K - 1 earlier inputs ; x],
//     s_p = bias + sum_{j<K} w[j] X[p + j],   out_p = act(s_p)
// and, ds_p = d_out_p act'(s_p) (0 outside the sequence),
//     dX[r] = sum_j w[j] ds[r - j] (+ d_final on the last K - 1 rows),
//     dw[j] = sum_p ds_p X[p + j],   dbias = sum_p ds_p.
// K is 2 to 4: 2 K operations for 4 bytes moved (6 backward), so HBM-bound.
#pragma once

#include <type_traits>

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
    int tile, tiles;                // positions of a thread or chunk, their number a sequence
};

// Row r < K - 1 of X, an earlier input, at channels c .. c + V - 1.  final_state may be init_state, so these
// are plain loads: each thread has the rows it needs before it writes any.
template <int V>
__device__ __forceinline__ Raw<V> early_row(const Args &a, int b, int r, int K, int c) {
    return a.init != nullptr ? load_plain<V>(a.init + ((long long)b * (K - 1) + r) * a.D + c) : zero_raw<V>();
}

// Few positions.  One thread: V channels, kDirect consecutive scan positions; every row it needs
// (kDirect + K - 1) is requested before the first is used, so a thread waits for memory once.  Threads
// run along the channels, so a warp reads whole lines of each row whatever the scan order.  1600
// tokens of 1024 channels: 9 us with cold caches, latency (6 us a call in a row).
constexpr int kDirect = 4;
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads, 4) causal_conv_fwd_kernel(const Args a) {
    constexpr int TP = kDirect;
    chain_wait();
    long long g, tile;
    const long long t = div_rem((long long)blockIdx.x * kThreads + threadIdx.x, a.groups, g);
    const int b = (int)div_rem(t, a.tiles, tile);
    if (b >= a.B) return;
    const int c = (int)g * V, p0 = (int)tile * TP;
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
    // the weights of V channels lie together: V K floats, in 16-byte pieces where they can be; channels
    // in pairs (V = 1: half of one)
    constexpr int NP = (V + 1) / 2;
    float2 w[K][NP], bias[NP];
    if constexpr (V % 4 == 0) {
        float4 q[V * K / 4];
#pragma unroll
        for (int i = 0; i < V * K / 4; ++i) q[i] = __ldg(reinterpret_cast<const float4 *>(a.w + (long long)c * K) + i);
#pragma unroll
        for (int i = 0; i < V * K; ++i) {
            const float4 f = q[i / 4];
            const float x1 = i % 4 == 0 ? f.x : i % 4 == 1 ? f.y : i % 4 == 2 ? f.z : f.w;
            const int v = i / K;
            if (v & 1)
                w[i % K][v / 2].y = x1;
            else
                w[i % K][v / 2].x = x1;
        }
    } else {
#pragma unroll
        for (int j = 0; j < K; ++j) w[j][0] = make_float2(__ldg(a.w + (long long)c * K + j), 0.f);
    }
#pragma unroll
    for (int v = 0; v < NP; ++v)
        bias[v] = a.bias != nullptr ? make_float2(__ldg(a.bias + c + 2 * v), V == 1 ? 0.f : __ldg(a.bias + c + 2 * v + (V > 1))) : splat(0.f);
    // tile 0 also writes the carried rows: the last K - 1 of X, after it has read what it needs of init_state
    // (which no other tile reads)
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
    float2 win[K][NP];
#pragma unroll
    for (int j = 0; j < K - 1; ++j) pairs_of<T, V>(x[j], win[j]);
    const bool silu = a.act == GTR_ACT_SILU;
    uint32_t worst = 0;
#pragma unroll
    for (int i = 0; i < TP; ++i) {
        pairs_of<T, V>(x[K - 1 + i], win[K - 1]);
        Raw<V> o;
#pragma unroll
        for (int v = 0; v < NP; ++v) {
            float2 s = bias[v];
#pragma unroll
            for (int j = 0; j < K; ++j) s = __ffma2_rn(w[j][v], win[j][v], s);
            const float2 y = __fmul2_rn(s, make_float2(sigmoid_f(s.x), sigmoid_f(s.y)));
            s = make_float2(silu ? y.x : s.x, silu ? y.y : s.y);
            o.w[v] = V == 1 ? Elem<T>::put(s.x) : Elem<T>::put2(s.x, s.y);
        }
        if (p0 + i < a.N) {
#pragma unroll
            for (const uint32_t q : o.w) worst = Elem<T>::worst(worst, q);
            store_raw<V>(a.out + (row0 + tok[i]) * a.D + c, o);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int v = 0; v < NP; ++v) win[j][v] = win[j + 1][v];
    }
    const bool bad = Elem<T>::bad_raw(worst);
    if (bad) set_error(kOpsErrRange);
}

// Rows in tiles through shared memory, for the walks below.  A block takes 128 channels, a pair a
// thread, of a chunk of positions; a thread stages and stores the rows tt and tt + 4 of every tile of
// kTok tokens, 8 channels of them, as 16-byte copies (element by element where rows do not line up).
constexpr int kWalkThreads = 64, kTok = 8, kStages = 3;
constexpr int kRowThreads = 2 * kWalkThreads / 8, kHalf = kTok / 2;   // threads of a row; the second row's distance
static_assert(kTok * kRowThreads == 2 * kWalkThreads, "two rows of a tile a thread");

// Eight channels of a finished row to memory, `left` of them inside the tensor.
template <typename T, bool WIDE>
__device__ __forceinline__ bool put_row(uint16_t *dst, const uint16_t *src, int left) {
    const Raw<8> v = load_plain<8>(src);
    if (WIDE) {
        store_raw<8>(dst, v);
        return Elem<T>::bad_raw(Elem<T>::worst(Elem<T>::worst(v.w[0], v.w[1]), Elem<T>::worst(v.w[2], v.w[3])));
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) {
            const uint16_t q = (uint16_t)(i & 1 ? v.w[i / 2] >> 16 : v.w[i / 2]);
            bad |= Elem<T>::bad_raw(q);
            dst[i] = q;
        }
    return bad;
}
__device__ __forceinline__ float2 param_pair(const float *p, int c, bool v0, bool v1, int j, int stride) {
    return make_float2(p != nullptr && v0 ? __ldg(p + (long long)c * stride + j) : 0.f,
                       p != nullptr && v1 ? __ldg(p + (long long)(c + 1) * stride + j) : 0.f);
}
// Row r of X at channels c, c + 1 (r counts from the K - 1 earlier inputs).
template <typename T, int K>
__device__ __forceinline__ float2 row_pair(const Args &a, int b, int r, int c, bool v0, bool v1) {
    if (r < K - 1) {   // plain loads, see early_row
        if (a.init == nullptr) return splat(0.f);
        const uint16_t *e = a.init + ((long long)b * (K - 1) + r) * a.D + c;
        return make_float2(v0 ? Elem<T>::get(e[0]) : 0.f, v1 ? Elem<T>::get(e[1]) : 0.f);
    }
    const uint16_t *src = a.x + ((long long)b * a.N + token_of(r - (K - 1), a.H, a.W, a.dir)) * a.ldx + c;
    return make_float2(Elem<T>::get(ld16(src, v0)), Elem<T>::get(ld16(src + 1, v1)));
}

// Many positions.  A thread walks its chunk with the last K rows of X in registers; rows come two
// tiles ahead of their use.  8 x 2304 tokens of 2048 channels: 43 us by itself with cold caches (a third of its
// writes leave the L2), 56 us a call in a row over inputs beyond L2, 2.7 TB/s (67 with the direct
// kernel, whose threads wait for memory without work of their own).
template <typename T, int K, bool WIDE>
__global__ void __launch_bounds__(kWalkThreads, 10) causal_conv_walk_kernel(const Args a) {
    constexpr int CH = 2 * kWalkThreads;
    __shared__ __align__(16) uint16_t rows[kStages][kTok][CH];
    __shared__ __align__(16) uint16_t outs[2][kTok][CH];
    chain_wait();
    const int tid = threadIdx.x, cb = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    const int b = part / a.tiles, chunk = part - b * a.tiles;
    const int p0 = chunk * a.tile, own = min(a.tile, a.N - p0);
    const long long row0 = (long long)b * a.N;
    const int c = cb * CH + 2 * tid;
    const bool v0 = c < a.D, v1 = c + 1 < a.D;
    const int tt = tid / kRowThreads, tc = tid % kRowThreads, c8 = cb * CH + tc * 8, left = a.D - c8;
    Walk in0(min(p0 + tt, a.N - 1), a.H, a.W, a.dir), in1(min(p0 + tt + kHalf, a.N - 1), a.H, a.W, a.dir);
    Walk out0 = in0, out1 = in1;
    auto stage = [&](int n0, int s) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const bool in = n0 + tt + kHalf * r < own;
            const long long row = row0 + (in ? (r ? in1.n : in0.n) : 0);
            stage_row<WIDE>(&rows[s][tt + kHalf * r][tc * 8], a.x + row * a.ldx + c8, in, left);
        }
        in0.advance(kTok);
        in1.advance(kTok);
        if (WIDE) copy_commit();
    };
    stage(0, 0);
    stage(kTok, 1);
    bool bad = false;
    auto flush = [&](int n0, int buf) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (n0 + tt + kHalf * r < own && left > 0)
                bad |= put_row<T, WIDE>(a.out + (row0 + (r ? out1.n : out0.n)) * a.D + c8, &outs[buf][tt + kHalf * r][tc * 8], left);
        out0.advance(kTok);
        out1.advance(kTok);
    };
    float2 w[K], xw[K];
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = param_pair(a.w, c, v0, v1, j, K);
    const float2 bias = param_pair(a.bias, c, v0, v1, 0, 1);
#pragma unroll
    for (int j = 0; j < K - 1; ++j) xw[j] = row_pair<T, K>(a, b, p0 + j, c, v0, v1);
    if (chunk == 0 && a.fin != nullptr) {   // the carried rows, after the thread's reads of init_state
        float2 f[K - 1];
#pragma unroll
        for (int j = 0; j < K - 1; ++j) f[j] = row_pair<T, K>(a, b, a.N + j, c, v0, v1);
#pragma unroll
        for (int j = 0; j < K - 1; ++j) {
            uint16_t *dst = a.fin + ((long long)b * (K - 1) + j) * a.D + c;
            if (v0) dst[0] = Elem<T>::put(f[j].x);
            if (v1) dst[1] = Elem<T>::put(f[j].y);
        }
    }
    const bool silu = a.act == GTR_ACT_SILU;
    int s = 0, buf = 0;
    for (int n0 = 0; n0 < own; n0 += kTok, buf ^= 1) {
        if (WIDE) copy_wait<kStages - 2>();
        __syncthreads();   // this tile's rows are here, the tile before has been computed
        stage(n0 + (kStages - 1) * kTok, s == 0 ? kStages - 1 : s - 1);
        if (n0 > 0) flush(n0 - kTok, buf ^ 1);
#pragma unroll
        for (int i = 0; i < kTok; ++i) {   // rows behind the chunk are zeros, and what they give is not stored
            xw[K - 1] = Elem<T>::get2(*reinterpret_cast<const uint32_t *>(&rows[s][i][2 * tid]));
            float2 z = bias;
#pragma unroll
            for (int j = 0; j < K; ++j) z = __ffma2_rn(w[j], xw[j], z);
            const float2 y = __fmul2_rn(z, make_float2(sigmoid_f(z.x), sigmoid_f(z.y)));
            *reinterpret_cast<uint32_t *>(&outs[buf][i][2 * tid]) = Elem<T>::put2(silu ? y.x : z.x, silu ? y.y : z.y);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) xw[j] = xw[j + 1];
        }
        s = s == kStages - 1 ? 0 : s + 1;
    }
    __syncthreads();
    flush((own - 1) / kTok * kTok, buf ^ 1);
    if (bad) set_error(kOpsErrRange);
}

// Backward.  A walk as well: the chunk's positions and the K - 1 behind it (whose ds its last
// outputs need).  A thread walks the chunk with the last K rows of X and of ds
// in registers and sums its channels' dw and dbias, one partial row a block, so that the sum over
// tokens has a fixed order.  Rows come in tiles of kTok tokens through shared memory, as 16-byte
// asynchronous copies two tiles ahead (element by element where rows do not line up), and leave
// through it as well: with rows read straight into registers the addresses were half of the
// instructions (114 us at 8 x 2304 tokens of 2048 channels; 66 so, 3.4 TB/s at 53 % issue).  A tile inside the chunk and the
// sequence runs without a branch; the first and the last test every step.
template <typename T, int K, bool WIDE>
__global__ void __launch_bounds__(kWalkThreads, 8) causal_conv_bwd_kernel(const Args a) {
    constexpr int CH = 2 * kWalkThreads;
    __shared__ __align__(16) uint16_t rows[kStages][2][kTok][CH];
    __shared__ __align__(16) uint16_t outs[2][kTok][CH];
    chain_wait();
    const int tid = threadIdx.x, cb = blockIdx.x % a.groups, part = blockIdx.x / a.groups;
    const int b = part / a.tiles, chunk = part - b * a.tiles;
    const int p0 = chunk * a.tile;
    const int own = min(a.tile, a.N - p0), steps = own + K - 1;   // steps n: position p0 + n
    const bool tail = p0 + steps > a.N;                           // some steps lie behind the sequence
    const long long row0 = (long long)b * a.N;
    const int c = cb * CH + 2 * tid;
    const bool v0 = c < a.D, v1 = c + 1 < a.D;

    const int tt = tid / kRowThreads, tc = tid % kRowThreads, c8 = cb * CH + tc * 8, left = a.D - c8;
    Walk in0(min(p0 + tt, a.N - 1), a.H, a.W, a.dir), in1(min(p0 + tt + kHalf, a.N - 1), a.H, a.W, a.dir);
    auto stage = [&](int n0, int s) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = n0 + tt + kHalf * r;
            const bool in = n < steps && p0 + n < a.N;
            const long long row = row0 + (in ? (r ? in1.n : in0.n) : 0);
            stage_row<WIDE>(&rows[s][0][tt + kHalf * r][tc * 8], a.x + row * a.ldx + c8, in, left);
            stage_row<WIDE>(&rows[s][1][tt + kHalf * r][tc * 8], a.dy + row * a.lddy + c8, in, left);
        }
        in0.advance(kTok);
        in1.advance(kTok);
        if (WIDE) copy_commit();
    };
    stage(0, 0);
    stage(kTok, 1);

    // rows leave as they came: row p = p0 + n of dX is position p - (K - 1), or an earlier input
    bool bad = false;
    Walk out0(max(p0 + tt - (K - 1), 0), a.H, a.W, a.dir), out1(max(p0 + tt + kHalf - (K - 1), 0), a.H, a.W, a.dir);
    auto flush = [&](int n0, int buf) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int n = n0 + tt + kHalf * r, p = p0 + n;
            const bool out = n >= K - 1;
            uint16_t *dst = out ? a.dx + (row0 + (r ? out1.n : out0.n)) * a.D + c8
                                : a.dinit != nullptr && p < K - 1 ? a.dinit + ((long long)b * (K - 1) + p) * a.D + c8 : nullptr;
            if (n < steps && left > 0 && dst != nullptr) {
                bad |= put_row<T, WIDE>(dst, &outs[buf][tt + kHalf * r][tc * 8], left);
            }
            // the next tile's row; a row ahead of the sequence (an earlier input) is followed by kTok - the rest
            Walk &w = r ? out1 : out0;
            const int q = p - (K - 1);
            w.advance(q < 0 ? kTok + q : kTok);
        }
    };

    float2 w[K], acc[K + 1];
#pragma unroll
    for (int j = 0; j < K; ++j) w[j] = param_pair(a.w, c, v0, v1, j, K);
    const float2 bias = param_pair(a.bias, c, v0, v1, 0, 1);
#pragma unroll
    for (int j = 0; j <= K; ++j) acc[j] = splat(0.f);
    float2 xw[K], dw[K];   // rows p .. p + K - 1 of X; ds of positions p - K + 1 .. p
#pragma unroll
    for (int j = 0; j < K - 1; ++j) xw[j] = row_pair<T, K>(a, b, p0 + j, c, v0, v1);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j] = splat(0.f);

    const bool silu = a.act == GTR_ACT_SILU;
    auto tile = [&](auto full, int n0, int s, int buf) {
        constexpr bool FULL = decltype(full)::value;   // every step the block's own and inside the sequence
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int n = n0 + i;
            if (!FULL && n >= steps) break;
            xw[K - 1] = Elem<T>::get2(*reinterpret_cast<const uint32_t *>(&rows[s][0][i][2 * tid]));
            const float2 dy = Elem<T>::get2(*reinterpret_cast<const uint32_t *>(&rows[s][1][i][2 * tid]));
            float2 z = bias;
#pragma unroll
            for (int j = 0; j < K; ++j) z = __ffma2_rn(w[j], xw[j], z);
            const float2 sg = make_float2(sigmoid_f(z.x), sigmoid_f(z.y));
            const float2 one = __ffma2_rn(z, __fadd2_rn(splat(1.f), make_float2(-sg.x, -sg.y)), splat(1.f));
            const float2 d = __fmul2_rn(dy, __fmul2_rn(sg, one));
            dw[K - 1] = make_float2(silu ? d.x : dy.x, silu ? d.y : dy.y);
            // behind the sequence there is no ds (not 0 times what the activation makes of X)
            if (!FULL && p0 + n >= a.N) dw[K - 1] = splat(0.f);
            if (FULL || n < own) {
#pragma unroll
                for (int j = 0; j < K; ++j) acc[j] = __ffma2_rn(dw[K - 1], xw[j], acc[j]);
                acc[K] = __fadd2_rn(acc[K], dw[K - 1]);
            }
            float2 e = __fmul2_rn(w[0], dw[K - 1]);
#pragma unroll
            for (int j = 1; j < K; ++j) e = __ffma2_rn(w[j], dw[K - 1 - j], e);
            if (!FULL && a.dfin != nullptr && p0 + n >= a.N) {
                const uint16_t *f = a.dfin + ((long long)b * (K - 1) + p0 + n - a.N) * a.D + c;
                e = __fadd2_rn(e, make_float2(v0 ? Elem<T>::get(__ldg(f)) : 0.f, v1 ? Elem<T>::get(__ldg(f + 1)) : 0.f));
            }
            *reinterpret_cast<uint32_t *>(&outs[buf][i][2 * tid]) = Elem<T>::put2(e.x, e.y);
#pragma unroll
            for (int j = 0; j < K - 1; ++j) xw[j] = xw[j + 1], dw[j] = dw[j + 1];
        }
    };
    int s = 0, buf = 0;
    for (int n0 = 0; n0 < steps; n0 += kTok, buf ^= 1) {
        if (WIDE) copy_wait<kStages - 2>();
        __syncthreads();   // this tile's rows are here, the tile before has been computed
        stage(n0 + (kStages - 1) * kTok, s == 0 ? kStages - 1 : s - 1);
        if (n0 > 0) flush(n0 - kTok, buf ^ 1);
        if (n0 + kTok <= own && !(tail && p0 + n0 + kTok > a.N))
            tile(std::true_type{}, n0, s, buf);
        else
            tile(std::false_type{}, n0, s, buf);
        s = s == kStages - 1 ? 0 : s + 1;
    }
    __syncthreads();
    flush((steps - 1) / kTok * kTok, buf ^ 1);
    if (bad) set_error(kOpsErrRange);
#pragma unroll
    for (int j = 0; j <= K; ++j) {
        float *dst = a.part + ((long long)part * (K + 1) + j) * a.D + c;
        if (v0) dst[0] = acc[j].x;
        if (v1) dst[1] = acc[j].y;
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
