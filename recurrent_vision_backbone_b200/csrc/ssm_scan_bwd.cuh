// ssm_scan_bwd.cuh -- gradients of the selective scan (included by ssm_scan_bwd.cu after ssm_scan.cuh).
//
// With h_p = a_p h_{p-1} + x_p B_p, x = t u, e_p = d_out_p silu(z_p) and G_p = dL/dh_p:
//     G_p = C_p e_p + a_{p+1} G_{p+1}   (+ d_final at the last position)
//     dC_p[n] = sum_d e_p h_p        dB_p[n] = sum_d G_p x_p       dA = sum_p (G_p a_p h_{p-1}) t_p
//     q_p = sum_n G_p B_p            r_p = sum_n (G_p a_p h_{p-1}) A
//     du = q t + D e      dt: (r + q u) sigmoid(raw)      dD = sum e u     dz = d_out y silu'(z)
//     d_init = a_0 G_0
// The states run forward and the gradients backward, so a sequence is cut into chunks of L
// tokens: one forward walk finds what each chunk does to a state entering it and to a gradient
// (ssm_walk_kernel<kLocalBwd>: both from the same exponentials), the fold runs over the chunks
// both ways, and ssm_grad_kernel does each chunk on its own:
//   * sweep: the states at every kSub-th token, kept in shared memory;
//   * from the last sub-chunk to the first: its kSub tokens forward again, decays and states in
//     registers, then backward.
// Each state element costs close to three exponentials and about 18 multiply-adds a token.  The
// division by a_p that would spare the states' second run is not open: decays may be 0.
// 4 x 1961 tokens of 1536 channels, 16 states: 406 us, of which ssm_grad_kernel 304 (257 instructions a
// token and 16 channels, issued 59 % of the time by 12 warps an SM: instruction issue and its
// latencies bound it, the exponentials' pipe is busy 32 %), the walk 85, the fold 22, the sums 13.
//
// Layout: a lane holds two neighbouring channels by four states.  The sums over channels (dB, dC:
// 8 values a token) and over states (q, r, y: 6 values) are butterflies that halve the number
// of values at every round, so that a token costs 7 + 5 exchanges at 16 states; four states by
// two channels is where the two together are least.  The scalars of a sub-chunk (t, x, e and
// what the gradients of u, dt, z need) are computed once per channel, spread over the warp.
#pragma once

namespace gtr {
namespace sc {

constexpr int kSub = 4, kMaxChunkBwd = 48, kAhead = 2;

template <int SP>
struct GradLayout {
    static constexpr int SL = SP / 4;            // lanes that share a channel pair
    static constexpr int CW = 64 / SL;           // channels of a warp
    static constexpr int CT = 4 * CW;            // channels of a block
    static constexpr int NE = (kSub * CW / 2 + 31) / 32;   // (token, channel pair) entries a lane prepares
    // shared memory, floats: B, C of the chunk; checkpoints; per warp t, x, e and q, r, y; dB, dC; zeros
    // for the lanes that hold nothing, 16 banks away from what the others read with them
    static constexpr int stage = 6 * kSub * CW;
    static constexpr int zeros = kSub * (3 * CW > SP ? 3 * CW : SP);
    static __host__ __device__ constexpr int floats(int L) {
        return 2 * L * SP + L / kSub * kThreads * 8 + 4 * stage + 2 * 4 * kSub * 2 * SP + 16 + zeros;
    }
};

// PAIRS: rows of channels start on 4 bytes and are even.  PAD also covers the channels that only fill a
// block's (the sums over channels take them in): a lane without a state or a channel of the
// call's reads zeros for t, x, e, B and C, the second channel of an odd row's last pair is left out
// of its lane's sums.
template <typename T, int SP, bool PAIRS, Pad PAD>
__global__ void __launch_bounds__(kThreads, 3) ssm_grad_kernel(const Args a) {
    using Lay = GradLayout<SP>;
    constexpr int SL = Lay::SL, CW = Lay::CW, NE = Lay::NE;
    extern __shared__ __align__(16) float sm[];
    chain_wait();
    __shared__ int stok[kMaxChunkBwd];                           // tokens of the chunk
    __shared__ uint32_t raw[kAhead + 1][4][NE][kThreads];        // u, dt, d_out, z entries on their way
    const int L = a.L;
    float *sB = sm, *sC = sB + L * SP;
    float4 *ck = reinterpret_cast<float4 *>(sC + L * SP);        // [L / kSub][2][kThreads]
    float *stage = reinterpret_cast<float *>(ck + L / kSub * 2 * kThreads);
    float *wsum = stage + 4 * Lay::stage;                        // [2][4 warps][kSub][2 SP]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *st = stage + warp * Lay::stage, *sx = st + kSub * CW, *se = sx + kSub * CW;
    float *rq = se + kSub * CW, *rr = rq + kSub * CW, *ry = rr + kSub * CW;
    const int sl = lane % SL, pr = lane / SL;
    const int ct = blockIdx.x % a.tiles;
    const int cj = blockIdx.x / a.tiles;
    const int b = cj / a.P, j = cj - b * a.P;
    const int p0 = j * L, p1 = min(a.N, p0 + L), nsub = (p1 - p0 + kSub - 1) / kSub;
    const long long row0 = (long long)b * a.N;
    const int cb = ct * Lay::CT + warp * CW;     // the warp's first channel
    const int c = cb + 2 * pr;                   // this lane's channels: c, c + 1
    const bool cv[2] = {c < a.D, c + 1 < a.D};
    const bool gate = a.z != nullptr, sp_on = a.softplus != 0;
    const bool live = PAD != kQuads || (cv[0] && sl * 4 < a.S);
    const bool two = PAD == kFull || PAIRS || cv[1];
    float *zeros = wsum + 2 * 4 * kSub * 2 * SP + 16;
    // what this lane reads of a token: its channels' t, x, e, its states' B and C (kQuads: from one place a lane,
    // chosen once)
    const float *lane_txe = live ? st + 2 * pr : zeros, *lane_B = live ? sB + sl * 4 : zeros, *lane_C = live ? sC + sl * 4 : zeros;
    const int lane_step = live ? kSub * SP : 0;
    auto pair_of = [&](const float *p, int tt) {
        if constexpr (PAD == kQuads)
            return *reinterpret_cast<const float2 *>(lane_txe + (p - st) + tt * CW);
        else
            return *reinterpret_cast<const float2 *>(p + tt * CW + 2 * pr);
    };
    auto quad_of = [&](const float *p, int s, int tt) {
        if constexpr (PAD == kQuads)
            return *reinterpret_cast<const float4 *>((p == sB ? lane_B : lane_C) + s * lane_step + tt * SP);
        else
            return *reinterpret_cast<const float4 *>(p + (s * kSub + tt) * SP + sl * 4);
    };
    if (PAD == kQuads)
        for (int i = tid; i < Lay::zeros; i += kThreads) zeros[i] = 0.f;
    if (tid < p1 - p0) stok[tid] = token_of(p0 + tid, a.H, a.W, a.dir);
    __syncthreads();
    for (int i = tid; i < (p1 - p0) * SP; i += kThreads) {
        const int n = i % SP;
        const long long row = row0 + stok[i / SP];
        sB[i] = Elem<T>::get(ld16(a.bm + row * a.ldb + n, n < a.S));
        sC[i] = Elem<T>::get(ld16(a.cm + row * a.ldc + n, n < a.S));
    }

    // states in pairs: [channel][pair]
    float2 A2[2][2], h[2][2], g[2][2], dA[2][2];
    {
        const float *hs = j > 0 ? a.hs + ((long long)b * a.P + j - 1) * a.D * SP
                                : a.h0 != nullptr ? a.h0 + (long long)b * a.D * a.S : nullptr;
        const int hst = j > 0 ? SP : a.S;
        const float *gs = j < a.P - 1 ? a.gs + ((long long)b * a.P + j + 1) * a.D * SP
                                      : a.dfin != nullptr ? a.dfin + (long long)b * a.D * a.S : nullptr;
        const int gst = j < a.P - 1 ? SP : a.S;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = sl * 4 + i;
                const bool in = cv[k] && n < a.S;
                const float av = in ? __ldg(a.A + (long long)(c + k) * a.S + n) * kLog2e : 0.f;
                const float hv = in && hs != nullptr ? hs[(long long)(c + k) * hst + n] : 0.f;
                const float gv = in && gs != nullptr ? gs[(long long)(c + k) * gst + n] : 0.f;
                if (i & 1)
                    A2[k][i / 2].y = av, h[k][i / 2].y = hv, g[k][i / 2].y = gv;
                else
                    A2[k][i / 2].x = av, h[k][i / 2].x = hv, g[k][i / 2].x = gv;
                dA[k][i / 2] = splat(0.f);
            }
    }
    // the entries (token, channel pair) of a sub-chunk that this lane prepares: pair lane % (CW / 2)
    // of tokens lane / (CW / 2) + (64 / CW) e; asked for one sub-chunk ahead
    const int el = 2 * (lane % (CW / 2)), ec = cb + el;
    const bool e0 = ec < a.D, e1 = ec + 1 < a.D;
    auto param = [&](const float *p) {
        return make_float2(p != nullptr && e0 ? __ldg(p + ec) : 0.f, p != nullptr && e1 ? __ldg(p + ec + 1) : 0.f);
    };
    const float2 dtb = param(a.dtb), Dk = param(a.Dk);
    float2 accD = splat(0.f), accT = splat(0.f);
    bool bad = false;
    auto put_entry = [&](uint32_t *dst, const uint16_t *p, long long at, bool in) {
        if (PAIRS)
            copy4_async(dst, p + at, in && e0 ? 4u : 0u);
        else
            *dst = (uint32_t)ld16(p + at, in && e0) | (uint32_t)ld16(p + at + 1, in && e1) << 16;
    };
    auto put_pair = [&](uint16_t *p, long long at, float2 v) {
        const uint32_t w = Elem<T>::put2(v.x, v.y);
        bad |= e1 ? Elem<T>::bad_raw(w) : Elem<T>::bad_raw(w & 0xffffu);
        if (PAIRS) {
            *reinterpret_cast<uint32_t *>(p + at) = w;
        } else {
            p[at] = (uint16_t)w;
            if (e1) p[at + 1] = (uint16_t)(w >> 16);
        }
    };
    auto entry = [&](int e) { return (lane + 32 * e) / (CW / 2); };   // token of the sub-chunk
    // The block's steps: the sweep over the sub-chunks but the last, then all from the last back.  A lane's
    // entries come through shared memory, each lane reading only its own, kAhead steps ahead.
    const int last_step = 2 * nsub - 2;
    auto fetch = [&](int k) {
        const int s = k < nsub - 1 ? k : last_step - k;
        uint32_t(*dst)[NE][kThreads] = raw[k % (kAhead + 1)];
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int q = s * kSub + entry(e);
            const bool in = k <= last_step && entry(e) < kSub && q < p1 - p0;
            const long long row = row0 + (in ? stok[q] : 0);
            put_entry(&dst[0][e][tid], a.u, row * a.ldu + ec, in);
            put_entry(&dst[1][e][tid], a.dt, row * a.lddt + ec, in);
            if (k >= nsub - 1) {
                put_entry(&dst[2][e][tid], a.dy, row * a.lddy + ec, in);
                if (gate) put_entry(&dst[3][e][tid], a.z, row * a.ldz + ec, in);
            }
        }
        if (PAIRS) copy_commit();
    };
    auto arrived = [&](int k) {   // the entries of step k
        if (PAIRS) copy_wait<kAhead - 1>();
        return raw[k % (kAhead + 1)];
    };
    auto real = [&](int k, int i, float2 v) {   // kAny: 0 where pair i of channel k only fills the lane
        if (PAD != kAny) return v;
        const int n = sl * 4 + 2 * i;
        return make_float2(cv[k] && n < a.S ? v.x : 0.f, cv[k] && n + 1 < a.S ? v.y : 0.f);
    };
    auto put2 = [](float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; };
    // a token forward: the decays, and the states after it
    auto forward = [&](int s, int tt, float2 (&d)[2][2]) {
        const float2 t = pair_of(st, tt);
        const float2 x = pair_of(sx, tt);
        const float4 B = quad_of(sB, s, tt);
        const float2 Bv[2] = {make_float2(B.x, B.y), make_float2(B.z, B.w)};
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 tk = splat(k ? t.y : t.x), xk = splat(k ? x.y : x.x);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float2 m = __fmul2_rn(tk, A2[k][i]);
                d[k][i] = real(k, i, make_float2(ex2(m.x), ex2(m.y)));
                h[k][i] = real(k, i, __ffma2_rn(d[k][i], h[k][i], __fmul2_rn(xk, Bv[i])));
            }
        }
    };
    __syncthreads();

    // sweep: checkpoints of the states entering the sub-chunks
#pragma unroll
    for (int k = 0; k < kAhead; ++k) fetch(k);
    for (int s = 0; s < nsub; ++s) {
        ck[(s * 2 + 0) * kThreads + tid] = make_float4(h[0][0].x, h[0][0].y, h[0][1].x, h[0][1].y);
        ck[(s * 2 + 1) * kThreads + tid] = make_float4(h[1][0].x, h[1][0].y, h[1][1].x, h[1][1].y);
        if (s == nsub - 1) break;
        __syncwarp();
        const auto *in = arrived(s);
#pragma unroll
        for (int e = 0; e < NE; ++e) {   // every sub-chunk but the last is whole
            if (entry(e) >= kSub) break;
            const int ix = entry(e) * CW + el;
            const float2 pre = __fadd2_rn(Elem<T>::get2(in[1][e][tid]), dtb);
            float2 x, t = softplus_2(pre, x);   // selected, not branched over
            t = make_float2(sp_on ? t.x : pre.x, sp_on ? t.y : pre.y);
            put2(st + ix, t);
            put2(sx + ix, __fmul2_rn(t, Elem<T>::get2(in[0][e][tid])));
        }
        __syncwarp();
        fetch(s + kAhead);
        float2 d[2][2];
#pragma unroll
        for (int tt = 0; tt < kSub; ++tt) forward(s, tt, d);
    }

    // sub-chunks from the last to the first
    // (whole ones without a branch inside, so that the scheduler can overlap their tokens)
    auto sub = [&](auto full, int s) {
        constexpr bool FULL = decltype(full)::value;
        const int q0 = s * kSub, m = FULL ? kSub : p1 - p0 - q0;
        float2 eu[NE], et[NE], ee[NE], esg[NE], ez[NE], esz[NE], ey[NE];   // u, t, e, dt / d raw, z, sigmoid(z), d_out
        __syncwarp();
        const auto *in = arrived(last_step - s);
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            if (entry(e) >= kSub) break;
            const int ix = entry(e) * CW + el;
            eu[e] = Elem<T>::get2(in[0][e][tid]);
            ey[e] = Elem<T>::get2(in[2][e][tid]);
            ez[e] = Elem<T>::get2(gate ? in[3][e][tid] : 0u);
            const float2 pre = __fadd2_rn(Elem<T>::get2(in[1][e][tid]), dtb);
            float2 x;
            const float2 t = softplus_2(pre, x);
            et[e] = make_float2(sp_on ? t.x : pre.x, sp_on ? t.y : pre.y);
            esg[e] = make_float2(sp_on ? sigmoid_of(pre.x, x.x) : 1.f, sp_on ? sigmoid_of(pre.y, x.y) : 1.f);
            esz[e] = make_float2(sigmoid_f(ez[e].x), sigmoid_f(ez[e].y));
            const float2 eg = __fmul2_rn(ey[e], __fmul2_rn(ez[e], esz[e]));
            ee[e] = make_float2(gate ? eg.x : ey[e].x, gate ? eg.y : ey[e].y);
            put2(st + ix, et[e]);
            put2(sx + ix, __fmul2_rn(et[e], eu[e]));
            put2(se + ix, ee[e]);
        }
        __syncwarp();
        fetch(last_step - s + kAhead);
        float2 d[kSub][2][2], hp[kSub][2][2];   // decays; states entering the tokens
        {
            const float4 c0 = ck[(s * 2 + 0) * kThreads + tid], c1 = ck[(s * 2 + 1) * kThreads + tid];
            h[0][0] = make_float2(c0.x, c0.y), h[0][1] = make_float2(c0.z, c0.w);
            h[1][0] = make_float2(c1.x, c1.y), h[1][1] = make_float2(c1.z, c1.w);
        }
#pragma unroll
        for (int tt = 0; tt < kSub; ++tt) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i) hp[tt][k][i] = h[k][i];   // behind the last token: the state after it
            if (FULL || tt < m) forward(s, tt, d[tt]);   // the same for the whole block
        }
        float *ws = wsum + (s & 1) * 4 * kSub * 2 * SP + warp * kSub * 2 * SP;
#pragma unroll
        for (int tt = kSub - 1; tt >= 0; --tt) {
            if (!FULL && tt >= m) continue;
            const float2 t = pair_of(st, tt);
            const float2 x = pair_of(sx, tt);
            const float2 e = pair_of(se, tt);
            const float4 B = quad_of(sB, s, tt);
            const float4 C = quad_of(sC, s, tt);
            const float2 Bv[2] = {make_float2(B.x, B.y), make_float2(B.z, B.w)};
            const float2 Cv[2] = {make_float2(C.x, C.y), make_float2(C.z, C.w)};
            float2 vb[2], vc[2];                           // dB, dC of this lane's channels
            float vs[4], vr[2];                            // q and y of both channels; r of both
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float2 tk = splat(k ? t.y : t.x), xk = splat(k ? x.y : x.x), ek = splat(k ? e.y : e.x);
                float2 q = splat(0.f), r = splat(0.f), y = splat(0.f);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 hn = tt + 1 < kSub ? hp[tt + 1 < kSub ? tt + 1 : tt][k][i] : h[k][i];   // after the token
                    const float2 G = real(k, i, __ffma2_rn(ek, Cv[i], g[k][i]));
                    const float2 Ga = __fmul2_rn(G, d[tt][k][i]), w = __fmul2_rn(Ga, hp[tt][k][i]);
                    q = __ffma2_rn(G, Bv[i], q);
                    r = __ffma2_rn(w, A2[k][i], r);
                    y = __ffma2_rn(Cv[i], hn, y);
                    dA[k][i] = __ffma2_rn(w, tk, dA[k][i]);
                    if (k == 0)
                        vb[i] = __fmul2_rn(G, xk), vc[i] = __fmul2_rn(ek, hn);
                    else if (two)
                        vb[i] = __ffma2_rn(G, xk, vb[i]), vc[i] = __ffma2_rn(ek, hn, vc[i]);
                    g[k][i] = Ga;
                }
                vs[k] = q.x + q.y;
                vs[2 + k] = y.x + y.y;
                vr[k] = r.x + r.y;
            }
            float vbc[8] = {vb[0].x, vb[0].y, vb[1].x, vb[1].y, vc[0].x, vc[0].y, vc[1].x, vc[1].y};
            const int ib = butterfly<SL, 32, 8>(vbc, lane);   // over the channels of the warp
            constexpr int lb = left_of(8, 32 / SL);
#pragma unroll
            for (int i = 0; i < lb; ++i) {
                const int v = ib + i;   // 0..3 dB, 4..7 dC of states sl * 4 + v % 4
                ws[tt * 2 * SP + (v >= 4 ? SP : 0) + sl * 4 + (v & 3)] = vbc[i];
            }
            // over the states of the channels: q and y halve from four values, r from two
            const int is = butterfly<1, SL, 4>(vs, lane), ir = butterfly<1, SL, 2>(vr, lane);
            constexpr int ls = left_of(4, SL), lr = left_of(2, SL);
#pragma unroll
            for (int i = 0; i < ls; ++i)   // q, q, y, y
                (is + i >= 2 ? ry : rq)[tt * CW + 2 * pr + ((is + i) & 1)] = vs[i];
#pragma unroll
            for (int i = 0; i < lr; ++i) rr[tt * CW + 2 * pr + ir + i] = vr[i];
        }
        __syncthreads();   // the warps' sums of dB, dC (two buffers: the next sub-chunk writes the other)
        for (int i = tid; i < m * 2 * SP; i += kThreads) {
            const float *w0 = wsum + (s & 1) * 4 * kSub * 2 * SP + i;
            const float v = (w0[0] + w0[kSub * 2 * SP]) + (w0[2 * kSub * 2 * SP] + w0[3 * kSub * 2 * SP]);
            const long long row = row0 + stok[q0 + i / (2 * SP)];
            a.pbc[((long long)ct * a.B * a.N + row) * 2 * SP + i % (2 * SP)] = v;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            if (!e0 || entry(e) >= m) continue;
            const int ix = entry(e) * CW + el;
            const float2 q = *reinterpret_cast<const float2 *>(rq + ix);
            const float2 r = __fmul2_rn(*reinterpret_cast<const float2 *>(rr + ix), splat(kLn2));   // A2 = A log2(e)
            const float2 dr = __fmul2_rn(__ffma2_rn(q, eu[e], r), esg[e]);
            accD = __ffma2_rn(ee[e], eu[e], accD);
            accT = __fadd2_rn(accT, dr);
            const long long o = (row0 + stok[q0 + entry(e)]) * a.D + ec;
            put_pair(a.du, o, __ffma2_rn(q, et[e], __fmul2_rn(Dk, ee[e])));
            put_pair(a.ddt, o, dr);
            if (gate) {
                const float2 y = __ffma2_rn(Dk, eu[e], *reinterpret_cast<const float2 *>(ry + ix)), sg = esz[e];
                const float2 one = __ffma2_rn(ez[e], __fadd2_rn(splat(1.f), make_float2(-sg.x, -sg.y)), splat(1.f));
                put_pair(a.dz, o, __fmul2_rn(__fmul2_rn(ey[e], y), __fmul2_rn(sg, one)));
            }
        }
    };
    if ((p1 - p0) % kSub != 0)
        sub(std::false_type{}, nsub - 1);
    else
        sub(std::true_type{}, nsub - 1);
    for (int s = nsub - 2; s >= 0; --s) sub(std::true_type{}, s);
    if (bad) set_error(kOpsErrRange);

    // the chunk's share of dA over the state slot that only this chunk reads (chunk 0: the last
    // slot, which nothing reads), of dD and of ddt_bias
    float *pa = a.hs + ((long long)b * a.P + (j > 0 ? j - 1 : a.P - 1)) * a.D * SP;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!cv[k]) continue;
        *reinterpret_cast<float4 *>(pa + (long long)(c + k) * SP + sl * 4) =
            make_float4(dA[k][0].x, dA[k][0].y, dA[k][1].x, dA[k][1].y);
        if (j == 0 && a.dh0 != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (sl * 4 + i < a.S)
                    a.dh0[((long long)b * a.D + c + k) * a.S + sl * 4 + i] = i & 1 ? g[k][i / 2].y : g[k][i / 2].x;
        }
    }
#pragma unroll
    for (int o = CW / 2; o < 32; o *= 2) {
        accD.x += __shfl_xor_sync(0xffffffffu, accD.x, o);
        accD.y += __shfl_xor_sync(0xffffffffu, accD.y, o);
        accT.x += __shfl_xor_sync(0xffffffffu, accT.x, o);
        accT.y += __shfl_xor_sync(0xffffffffu, accT.y, o);
    }
    if (lane < CW / 2) {
        const long long at = ((long long)b * a.P + j) * a.D + ec;
        if (e0) a.pd[at] = accD.x, a.pt[at] = accT.x;
        if (e1) a.pd[at + 1] = accD.y, a.pt[at + 1] = accT.y;
    }
}

// Adds the partial sums in a fixed order.  The first `bc_blocks` blocks: dB and dC, one thread a
// (token, state), over the channel tiles; the rest: dA, dD, ddt_bias over the chunks, 32 columns
// by 8 row lanes a block.
template <typename T, int SP>
__global__ void __launch_bounds__(256) ssm_grad_sum_kernel(const Args a, int bc_blocks) {
    __shared__ float red[8][33];
    chain_wait();
    if ((int)blockIdx.x < bc_blocks) {
        const long long id = (long long)blockIdx.x * 256 + threadIdx.x, rows = (long long)a.B * a.N;
        const long long row = id / (2 * SP);
        const int v = (int)(id % (2 * SP)), n = v % SP;
        if (row >= rows || n >= a.S) return;
        float s = 0.f;
#pragma unroll 8
        for (int k = 0; k < a.tiles; ++k) s += a.pbc[((long long)k * rows + row) * 2 * SP + v];
        const uint16_t r = Elem<T>::put(s);
        (v < SP ? a.dB : a.dC)[row * a.S + n] = r;
        if (Elem<T>::bad_raw(r)) set_error(kOpsErrRange);
        return;
    }
    const long long cols = (long long)a.D * (SP + 2);
    const long long col = (long long)(blockIdx.x - bc_blocks) * 32 + threadIdx.x % 32;
    const int lane = threadIdx.x / 32, rows = a.B * a.P;
    const long long na = (long long)a.D * SP;
    float s = 0.f;
    if (col < cols) {
        const float *src = col < na ? a.hs + col : col < na + a.D ? a.pd + (col - na) : a.pt + (col - na - a.D);
        const long long stride = col < na ? na : a.D;
#pragma unroll 8
        for (int r = lane; r < rows; r += 8) s += src[r * stride];
    }
    red[lane][threadIdx.x % 32] = s;
    __syncthreads();
    if (lane == 0 && col < cols) {
#pragma unroll
        for (int l = 1; l < 8; ++l) s += red[l][threadIdx.x];
        if (col < na) {
            const int d = (int)(col / SP), n = (int)(col % SP);
            if (n < a.S) a.dA[(long long)d * a.S + n] = s;
        } else if (col < na + a.D) {
            if (a.dD != nullptr) a.dD[col - na] = s;
        } else if (a.ddtb != nullptr) {
            a.ddtb[col - na - a.D] = s;
        }
    }
}

}  // namespace sc
}  // namespace gtr
