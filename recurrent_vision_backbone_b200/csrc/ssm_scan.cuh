// ssm_scan.cuh -- the selective scan, forward, backward and for single tokens
// (included by ssm_scan.cu, which holds the C entry points).
//
// Per batch, channel d and state n over scan positions p (t_p the time step, x_p = t_p u_p):
//     h_p = a_p h_{p-1} + x_p B_p[n],  a_p = exp(t_p A[d][n]),   y_p[d] = sum_n C_p[n] h_p + D u_p
//
// What bounds it: one exponential and four multiply-adds for each state of each channel of each
// token, against 8 bytes for the token's channel: at 16 states the exponentials (16 a clock and
// SM) take twice the time of the memory traffic.  There is no matrix product in it: the decay
// differs in every (channel, state) pair.
//
// A position depends on all before it, and one sequence has too few (channel, state) pairs to
// fill the machine, so a sequence is cut into P chunks:
//   1. `local` walk: every chunk from a zero state; keeps the state it reaches and the sum of its
//      time steps (the product of its decays is exp(A times that sum): one number a channel).
//   2. fold: the states entering the chunks, in order, P steps.
//   3. `out` walk: every chunk again from its entering state, writing the outputs.
// The walk of step 1 costs as much as step 3, so P is 1 (step 3 alone) as soon as the channels
// alone keep the schedulers busy; else just large enough to do so.
//
// Walk layout: SL lanes a channel (one, or two that share its states), a block 128 / SL neighbouring
// channels.  Tiles of 8 SL tokens pass through shared memory: the channels' rows as 16-byte
// asynchronous copies, kStages tiles deep (or element by element where rows do not line up to 16
// bytes), B and C as float32, read as broadcasts, the outputs on their way back.  The time steps
// of two tokens are formed at once (packed arithmetic), and so are two states of a token.
// 16384 tokens of 1024 channels, 16 states, 74 chunks: 83 us the local walk, 104 the out walk (the
// exponentials' pipe busy 76 % and 69 % of the time), 10 the fold; the memory traffic alone is 21.
// 8 x 2304 tokens of 2048 channels in one walk with two lanes a channel: 289 us (52 %).
#pragma once

#include <type_traits>

namespace gtr {
namespace sc {

using namespace ops;

constexpr int kThreads = 128, kStages = 3;

struct Args {
    const uint16_t *u, *dt, *bm, *cm, *z, *dy;
    const float *A, *Dk, *dtb, *h0, *dfin;
    uint16_t *out;
    float *hf;
    long long ldu, lddt, ldb, ldc, ldz, lddy;
    int B, H, W, N, D, S, dir, softplus;
    int P, L, tiles;                // chunks a sequence, tokens a chunk, channel tiles
    int pairs;                      // backward: rows of channels start on 4 bytes and are even
    float *hs, *gs, *sdt;           // workspace: [B][P][D][SP], the same, [B][P][D]
    // backward
    uint16_t *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddtb, *dh0;
    float *pbc, *pd, *pt;           // workspace: [tiles][B N][2 SP], [B P][D], [B P][D]
};


enum { kLocal = 0, kOut = 1, kLocalBwd = 2 };

// States that only fill a kernel's, and how they stay out of the sums over states (their zeros times an
// infinite step, input or gradient would be no number there).  kFull: there are none.  kQuads: S is
// a multiple of four, whole groups of four are left out (backward up to 3 % of the time, forward none).
// kAny: values are selected one by one (backward 10 to 14 % at 5 states).
enum Pad { kFull = 0, kQuads = 1, kAny = 2 };

__host__ __device__ constexpr int left_of(int nv, int lanes) { return nv > lanes ? nv / lanes : 1; }

template <int MODE>
__host__ __device__ constexpr int walk_rows() { return MODE == kLocal ? 2 : MODE == kOut ? 3 : 4; }
// Blocks an SM that a walk's registers allow: four where the plan counts on them; two lanes a channel
// run when the channels alone are few blocks an SM.
template <int SP, int MODE, int SL>
__host__ __device__ constexpr int walk_blocks() { return SP > 16 ? 1 : MODE == kLocalBwd ? 3 : SL > 1 ? 2 : 4; }

// One walk over one chunk.  kLocal: hs[b][j] = the state reached from zero, sdt = the sum of the
// time steps.  kLocalBwd: also gs[b][j] = sum_p (prod_{r <= p} a_r) C_p e_p, the gradient that
// the chunk's outputs send to the state entering it.  kOut: outputs and the final state; the
// other modes keep every state to itself, so that only kOut has to leave padded ones out.
template <typename T, int SP, int MODE, bool WIDE, int SL, Pad PAD>
__global__ void __launch_bounds__(kThreads, walk_blocks<SP, MODE, SL>()) ssm_walk_kernel(const Args a) {
    static_assert(SL == 1 || (SL == 2 && MODE == kOut), "the local walks have chunks enough");
    static_assert(PAD == kFull || MODE == kOut, "only the outputs sum over states");
    constexpr int CH = kThreads / SL;           // channels of the block
    constexpr int TOK = 8 * SL;                 // tokens of a tile
    constexpr int NP = SP / SL / 2;             // pairs of states of a lane
    constexpr int R = walk_rows<MODE>();        // u, dt, z, dy
    constexpr int RT = 16 / SL;                 // threads that stage a token's row
    constexpr int NBC = 2 * SP / RT;            // B and C values a thread stages per tile
    __shared__ __align__(16) uint16_t rows[kStages][R][TOK][CH];
    __shared__ __align__(16) float bc[2][2][TOK][SP];
    __shared__ __align__(16) uint16_t outs[2][MODE == kOut ? TOK : 1][MODE == kOut ? CH : 8];
    chain_wait();
    const int tid = threadIdx.x;
    const int ct = blockIdx.x % a.tiles;
    const int cj = blockIdx.x / a.tiles;
    const int nj = MODE == kLocal ? a.P - 1 : a.P;   // the last chunk's reached state is not needed
    const int b = cj / nj, j = cj - b * nj;
    const int p0 = j * a.L, p1 = min(a.N, p0 + a.L);
    const int sl = tid % SL, cl = tid / SL, n0 = sl * 2 * NP;   // lane of the channel, channel, first state
    const int c = ct * CH + cl;
    const bool cv = c < a.D;
    const long long row0 = (long long)b * a.N;
    const bool gate = a.z != nullptr && MODE != kLocal, sp_on = a.softplus != 0;

    // staging: this thread's token of a tile, 8 of its channels, and some of its B and C
    const int tt = tid / RT, tc = tid % RT;
    const int c8 = ct * CH + tc * 8, left = a.D - c8;
    Walk wk(min(p0 + tt, a.N - 1), a.H, a.W, a.dir);
    uint16_t rb[NBC];
    auto stage = [&](int pb, int s) {   // request the rows of the tile at pb
        const bool in = pb + tt < p1;
        const long long row = row0 + (in ? wk.n : 0);
        stage_row<WIDE>(&rows[s][0][tt][tc * 8], a.u + row * a.ldu + c8, in, left);
        stage_row<WIDE>(&rows[s][1][tt][tc * 8], a.dt + row * a.lddt + c8, in, left);
        if (MODE != kLocal && gate) stage_row<WIDE>(&rows[s][MODE != kLocal ? 2 : 0][tt][tc * 8], a.z + row * a.ldz + c8, in, left);
        if (MODE == kLocalBwd) stage_row<WIDE>(&rows[s][MODE == kLocalBwd ? 3 : 0][tt][tc * 8], a.dy + row * a.lddy + c8, in, left);
        if (WIDE) copy_commit();
    };
    // values v = tc + RT i of a token's [B ; C]
    auto load_bc = [&](int pb, int n) {
        const bool in = pb + tt < p1;
        const long long row = row0 + (in ? n : 0);
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int v = tc + RT * i, k = v % SP;
            const bool isc = v >= SP;
            rb[i] = isc ? ld16(a.cm + row * a.ldc + k, in && k < a.S && MODE != kLocal) : ld16(a.bm + row * a.ldb + k, in && k < a.S);
        }
    };
    // the token of this thread in this tile and the next: rows are asked for kStages - 1 tiles
    // ahead, B and C one tile ahead
    int tok[kStages - 1];
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) {
        tok[s] = wk.n;
        stage(p0 + s * TOK, s);
        wk.advance(TOK);
    }
    load_bc(p0, tok[0]);
    // the outputs of a tile pass through shared memory, so that they leave as rows
    bool bad = false;
    auto flush = [&](int pb, int n, int buf) {
        if (pb + tt >= p1 || left <= 0) return;
        const Raw<8> r = load_plain<8>(&outs[buf][MODE == kOut ? tt : 0][MODE == kOut ? tc * 8 : 0]);
        uint16_t *dst = a.out + (row0 + n) * a.D + c8;
        if (WIDE) {   // whole pieces
            bad |= Elem<T>::bad_raw(Elem<T>::worst(Elem<T>::worst(r.w[0], r.w[1]), Elem<T>::worst(r.w[2], r.w[3])));
            store_raw<8>(dst, r);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) {
                    const uint16_t v = (uint16_t)(i & 1 ? r.w[i / 2] >> 16 : r.w[i / 2]);
                    bad |= Elem<T>::bad_raw(v);
                    dst[i] = v;
                }
        }
    };

    float2 A2[NP], h[NP], pr[NP], g[NP];   // pr, g: kLocalBwd
    const float *hin = nullptr;
    int hstride = SP;
    if (MODE == kOut) {
        if (j == 0) {
            // with several chunks the fold's copy of init_state: the last chunk may already have
            // written final_state over it
            hin = a.P > 1 ? a.hs + ((long long)b * a.P + a.P - 1) * a.D * SP
                          : a.h0 != nullptr ? a.h0 + (long long)b * a.D * a.S : nullptr;
            hstride = a.P > 1 ? SP : a.S;
        } else {
            hin = a.hs + ((long long)b * a.P + j - 1) * a.D * SP;
        }
    }
#pragma unroll
    for (int k = 0; k < 2 * NP; ++k) {
        const bool in = n0 + k < a.S && cv;
        const float av = in ? __ldg(a.A + (long long)c * a.S + n0 + k) * kLog2e : 0.f;
        const float hv = hin != nullptr && in ? hin[(long long)c * hstride + n0 + k] : 0.f;
        if (k & 1)
            A2[k / 2].y = av, h[k / 2].y = hv;
        else
            A2[k / 2].x = av, h[k / 2].x = hv;
    }
    if (MODE == kLocalBwd) {
#pragma unroll
        for (int k = 0; k < NP; ++k) pr[k] = splat(1.f), g[k] = splat(0.f);
    }
    const float dtb = a.dtb != nullptr && cv ? __ldg(a.dtb + c) : 0.f;
    const float Dk = MODE == kOut && a.Dk != nullptr && cv ? __ldg(a.Dk + c) : 0.f;
    float ssum = 0.f;

    // one token: t its step, x = t u, e (kLocalBwd); returns sum_n C h.  Each pair of states goes from
    // its product to its update before the next begins: with the exponentials of a token or two
    // ahead of the updates their pipe runs dry between bursts (the local walk took 97 us for 87)
    auto token = [&](int buf, int i, float t, float x, float e) -> float {
        const float4 *B4 = reinterpret_cast<const float4 *>(bc[buf][0][i] + n0);
        const float4 *C4 = reinterpret_cast<const float4 *>(bc[buf][1][i] + n0);
        const float2 t2 = splat(t), x2 = splat(x), e2 = splat(e);
        float2 y0 = splat(0.f), y1 = splat(0.f);
#pragma unroll
        for (int q = 0; q < NP / 2; ++q) {
            // with one lane a channel no state below the group's fewest is padded (of 16: 9, of 8: 4 or 1), and a
            // group of four is passed over; with two, where only the second lane would, it only leaves the
            // sum (passing over it: 378 us for 285 at 8 x 2304 tokens of 2048 channels, 12 states)
            constexpr int real = SL > 1 ? 0 : SP > 8 ? SP / 2 : PAD == kQuads ? 4 : 0;
            const bool maybe = 4 * q >= real, in = PAD != kQuads || !maybe || n0 + 4 * q < a.S;
            if (SL == 1 && !in) break;
            const float4 Bq = B4[q];
            const float4 Cq = MODE != kLocal ? C4[q] : Bq;
#pragma unroll
            for (int k = 2 * q; k < 2 * q + 2; ++k) {
                const float2 Bk = k & 1 ? make_float2(Bq.z, Bq.w) : make_float2(Bq.x, Bq.y);
                const float2 Ck = k & 1 ? make_float2(Cq.z, Cq.w) : make_float2(Cq.x, Cq.y);
                const float2 m = __fmul2_rn(t2, A2[k]);
                const float2 d = make_float2(ex2(m.x), ex2(m.y));
                h[k] = __ffma2_rn(d, h[k], __fmul2_rn(x2, Bk));
                if (PAD == kAny && maybe)
                    h[k] = make_float2(n0 + 2 * k < a.S ? h[k].x : 0.f, n0 + 2 * k + 1 < a.S ? h[k].y : 0.f);
                if (MODE == kOut && (SL == 1 || in)) (k & 1 ? y1 : y0) = __ffma2_rn(Ck, h[k], k & 1 ? y1 : y0);
                if (MODE == kLocalBwd) {
                    pr[k] = __fmul2_rn(pr[k], d);
                    g[k] = __ffma2_rn(pr[k], __fmul2_rn(e2, Ck), g[k]);
                }
            }
        }
        y0 = __fadd2_rn(y0, y1);
        return y0.x + y0.y;
    };

    // this lane's first token of a group (butterfly below leaves the sums of its two tokens here)
    const int own = 2 * sl;
    auto tile = [&](auto full, int pb, int buf, int s) {
        constexpr bool FULL = decltype(full)::value;
#pragma unroll
        for (int ig = 0; ig < TOK; ig += 2 * SL) {
            if (!FULL && pb + ig >= p1) break;   // the same for the whole block
            // the lanes of a channel each prepare two of 2 SL tokens
            const int i = ig + own;
            auto row2 = [&](int r) { return make_float2(Elem<T>::get(rows[s][r][i][cl]), Elem<T>::get(rows[s][r][i + 1][cl])); };
            const float2 u = row2(0);
            const float2 raw = __fadd2_rn(row2(1), splat(dtb));
            float2 ex, t = softplus_2(raw, ex);   // selected, not branched over: one block of code
            t = make_float2(sp_on ? t.x : raw.x, sp_on ? t.y : raw.y);
            const float2 x = __fmul2_rn(t, u);
            float2 sz = splat(1.f), e = splat(0.f);
            if (MODE != kLocal) {
                const float2 z = row2(MODE != kLocal ? 2 : 0);
                sz = make_float2(z.x * sigmoid_f(z.x), z.y * sigmoid_f(z.y));
                sz = make_float2(gate ? sz.x : 1.f, gate ? sz.y : 1.f);
            }
            if (MODE == kLocalBwd) e = __fmul2_rn(sz, row2(MODE == kLocalBwd ? 3 : 0));
            float y[2 * SL];
#pragma unroll
            for (int o = 0; o < 2 * SL; ++o) {
                y[o] = 0.f;
                if (!FULL && o > 0 && pb + ig + o >= p1) break;
                float to = o & 1 ? t.y : t.x, xo = o & 1 ? x.y : x.x;
                if constexpr (SL > 1) {
                    const int from = (tid & 31 & ~(SL - 1)) + o / 2;
                    to = __shfl_sync(0xffffffffu, to, from);
                    xo = __shfl_sync(0xffffffffu, xo, from);
                }
                if (MODE != kOut) ssum += to;
                y[o] = token(buf, ig + o, to, xo, o & 1 ? e.y : e.x);
            }
            if (MODE == kOut) {
                if constexpr (SL > 1) butterfly<1, SL, 2 * SL>(y, tid & 31);
                const float2 v = __fmul2_rn(__ffma2_rn(splat(Dk), u, make_float2(y[0], y[1])), sz);
                outs[buf][MODE == kOut ? i : 0][MODE == kOut ? cl : 0] = Elem<T>::put(v.x);
                outs[buf][MODE == kOut ? i + 1 : 0][MODE == kOut ? cl : 0] = Elem<T>::put(v.y);
            }
        }
    };

    int buf = 0, s = 0, before = 0;   // before: this thread's token of the tile before
    for (int pb = p0; pb < p1; pb += TOK, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < NBC; ++i) {
            const int v = tc + RT * i;
            bc[buf][v / SP][tt][v % SP] = Elem<T>::get(rb[i]);
        }
        if (WIDE) copy_wait<kStages - 2>();   // this tile's rows have landed
        // one barrier a tile: what is written behind it (the next buffers of B, C and the outputs, the
        // stage of the tile before) was last read ahead of it
        __syncthreads();
        load_bc(pb + TOK, tok[1]);
        static_assert(kStages == 3, "tok holds the tokens of two tiles");
        stage(pb + (kStages - 1) * TOK, s == 0 ? kStages - 1 : s - 1);
        if (MODE == kOut) {
            if (pb > p0) flush(pb - TOK, before, buf ^ 1);
            before = tok[0];
        }
        tok[0] = tok[1];
        tok[1] = wk.n;
        wk.advance(TOK);
        // whole tiles run without a branch, so that the scheduler can overlap their tokens
        if (pb + TOK <= p1)
            tile(std::true_type{}, pb, buf, s);
        else
            tile(std::false_type{}, pb, buf, s);
        s = s == kStages - 1 ? 0 : s + 1;
    }
    if (MODE == kOut) {
        __syncthreads();
        flush(p0 + (p1 - 1 - p0) / TOK * TOK, before, buf ^ 1);
        if (bad) set_error(kOpsErrRange);
        if (j != a.P - 1 || a.hf == nullptr) return;
    }
    if (!cv) return;
    if (MODE == kOut) {
        float *dst = a.hf + ((long long)b * a.D + c) * a.S + n0;
#pragma unroll
        for (int k = 0; k < 2 * NP; ++k)
            if (n0 + k < a.S) dst[k] = k & 1 ? h[k / 2].y : h[k / 2].x;
        return;
    }
    const long long at = ((long long)b * a.P + j) * a.D + c;
    float4 *dst = reinterpret_cast<float4 *>(a.hs + at * SP);
#pragma unroll
    for (int q = 0; q < SP / 4; ++q) dst[q] = make_float4(h[2 * q].x, h[2 * q].y, h[2 * q + 1].x, h[2 * q + 1].y);
    if (MODE == kLocalBwd) {
        float4 *gd = reinterpret_cast<float4 *>(a.gs + at * SP);
#pragma unroll
        for (int q = 0; q < SP / 4; ++q) gd[q] = make_float4(g[2 * q].x, g[2 * q].y, g[2 * q + 1].x, g[2 * q + 1].y);
    }
    a.sdt[at] = ssum;
}

// The chunks in order, one thread per (batch, channel, state).  Forward: hs[j] becomes the state
// leaving chunk j.  Backward (from the last chunk): gs[j] becomes the gradient of the state
// entering chunk j.  The chain itself is short; what costs are the loads, so those of kFold chunks
// are requested at once, ahead of the chain, and the blocks are small, so that a single sequence's
// reach every SM.  73 chunks of 16384 states: 10 us, most of it the latency of three batches.
constexpr int kFold = 32, kFoldThreads = 64;
template <bool REV>
__device__ __forceinline__ void fold_chain(float *v0, const float *s0, long long vs, long long ss, int m, float A2, float x) {
    // REV: j = m, m - 1, .., 1; else 0 .. m - 1
    for (int j0 = 0; j0 < m; j0 += kFold) {
        float v[kFold], s[kFold];
#pragma unroll
        for (int i = 0; i < kFold; ++i) {
            const int q = min(j0 + i, m - 1), j = REV ? m - q : q;
            v[i] = v0[j * vs];
            s[i] = s0[j * ss];
        }
#pragma unroll
        for (int i = 0; i < kFold; ++i)
            if (j0 + i < m) {
                x = fmaf(ex2(A2 * s[i]), x, v[i]);
                v0[(REV ? m - (j0 + i) : j0 + i) * vs] = x;
            }
    }
}
template <int SP, bool BWD>
__global__ void __launch_bounds__(kFoldThreads) ssm_fold_kernel(const Args a) {
    chain_wait();
    const long long per = (long long)a.D * SP;
    long long e;
    int b = (int)div_rem((long long)blockIdx.x * kFoldThreads + threadIdx.x, per, e), way = 0;
    if (BWD && b >= a.B) way = 1, b -= a.B;   // backward: the states, then the gradients
    if (b >= a.B) return;
    const int d = (int)(e / SP), n = (int)(e % SP);
    const bool in = n < a.S;
    const float A2 = in ? __ldg(a.A + (long long)d * a.S + n) * kLog2e : 0.f;
    const float *sd = a.sdt + (long long)b * a.P * a.D + d;
    const long long st = ((long long)b * a.D + d) * a.S + n;
    const int m = a.P - 1;
    if (way == 0) {
        float *hs = a.hs + (long long)b * a.P * per + e;
        const float h = a.h0 != nullptr && in ? a.h0[st] : 0.f;
        if (!BWD) hs[m * per] = h;   // the last slot is free: the entering state of chunk 0
        fold_chain<false>(hs, sd, per, a.D, m, A2, h);
    } else {
        fold_chain<true>(a.gs + (long long)b * a.P * per + e, sd, per, a.D, m, A2, a.dfin != nullptr && in ? a.dfin[st] : 0.f);
    }
}

// One token of every sequence: the states are the traffic (read and written once, 8 bytes a
// state against 8 bytes a channel), so lanes run along a channel's states, 16 bytes each: a
// warp reads and writes whole lines.  S / 4 lanes a channel (S = 4, 8, 16 or 32).  A thread takes NB
// neighbouring sequences, one or as many as lanes share the channel, whose states it asks for at once;
// each lane then prepares and finishes one of them.  BCW: B and C rows start on 8 bytes.
// 256 sequences of 2048 channels, 16 states: 17 us, 4.2 TB/s; one of 1024 channels: 4 us of latency.
template <typename T, int S, int NB, bool BCW>
__global__ void __launch_bounds__(256, NB <= 4 ? 4 : 2) ssm_token_kernel(const Args a) {
    constexpr int SL = S / 4;
    static_assert(NB == 1 || NB == SL, "a lane prepares one sequence");
    chain_wait();
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = (int)(id % SL), lane = threadIdx.x & 31;
    long long cc;
    const long long bg = div_rem(id / SL, a.D, cc);
    const int c = (int)cc;
    const long long b0 = bg * NB;
    // the sequence this lane prepares: the one whose sum butterfly leaves here (bits of q reversed)
    const int own = NB == 1 ? 0 : SL == 8 ? (q & 1) << 2 | (q & 2) | q >> 2 : SL == 4 ? (q & 1) << 1 | q >> 1 : q;
    float4 h[NB];
    uint2 rb[NB], rc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const bool in = b0 + i < a.B;
        const long long b = in ? b0 + i : 0;
        h[i] = in && a.h0 != nullptr ? *reinterpret_cast<const float4 *>(a.h0 + (b * a.D + c) * S + q * 4)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
        auto four = [&](const uint16_t *p) -> uint2 {
            if (BCW) return __ldg(reinterpret_cast<const uint2 *>(p));
            return make_uint2((uint32_t)__ldg(p) | (uint32_t)__ldg(p + 1) << 16, (uint32_t)__ldg(p + 2) | (uint32_t)__ldg(p + 3) << 16);
        };
        rb[i] = four(a.bm + b * a.ldb + q * 4);
        rc[i] = four(a.cm + b * a.ldc + q * 4);
    }
    const long long bo = b0 + own;
    const bool mine = bo < a.B;
    const float u = Elem<T>::get(ld16(a.u + bo * a.ldu + c, mine));
    const float raw = Elem<T>::get(ld16(a.dt + bo * a.lddt + c, mine)) + (a.dtb != nullptr ? __ldg(a.dtb + c) : 0.f);
    const float z = Elem<T>::get(ld16(a.z + bo * a.ldz + c, mine && a.z != nullptr));
    const float4 A = __ldg(reinterpret_cast<const float4 *>(a.A + (long long)c * S + q * 4));
    const float2 A0 = make_float2(A.x * kLog2e, A.y * kLog2e), A1 = make_float2(A.z * kLog2e, A.w * kLog2e);
    const float Dk = a.Dk != nullptr ? __ldg(a.Dk + c) : 0.f;
    const float t = a.softplus ? softplus_f(raw) : raw, x = t * u;
    float y[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        float ti = t, xi = x;
        if (NB > 1) {   // from the lane that prepared sequence i: the bits of i reversed
            const int from = (lane & ~(SL - 1)) + (SL == 8 ? (i & 1) << 2 | (i & 2) | i >> 2 : SL == 4 ? (i & 1) << 1 | i >> 1 : i);
            ti = __shfl_sync(0xffffffffu, t, from);
            xi = __shfl_sync(0xffffffffu, x, from);
        }
        const float2 m0 = __fmul2_rn(splat(ti), A0), m1 = __fmul2_rn(splat(ti), A1);
        const float2 h0 = __ffma2_rn(make_float2(ex2(m0.x), ex2(m0.y)), make_float2(h[i].x, h[i].y), __fmul2_rn(splat(xi), Elem<T>::get2(rb[i].x)));
        const float2 h1 = __ffma2_rn(make_float2(ex2(m1.x), ex2(m1.y)), make_float2(h[i].z, h[i].w), __fmul2_rn(splat(xi), Elem<T>::get2(rb[i].y)));
        if (b0 + i < a.B && a.hf != nullptr)
            *reinterpret_cast<float4 *>(a.hf + ((b0 + i) * a.D + c) * S + q * 4) = make_float4(h0.x, h0.y, h1.x, h1.y);
        const float2 y2 = __ffma2_rn(Elem<T>::get2(rc[i].x), h0, __fmul2_rn(Elem<T>::get2(rc[i].y), h1));
        y[i] = y2.x + y2.y;
    }
    butterfly<1, SL, NB>(y, lane);
    if (mine && (NB > 1 || q == 0)) {
        float o = fmaf(Dk, u, y[0]);
        if (a.z != nullptr) o *= z * sigmoid_f(z);
        const uint16_t r = Elem<T>::put(o);
        a.out[bo * a.D + c] = r;
        if (Elem<T>::bad_raw(r)) set_error(kOpsErrRange);
    }
}

}  // namespace sc
}  // namespace gtr
