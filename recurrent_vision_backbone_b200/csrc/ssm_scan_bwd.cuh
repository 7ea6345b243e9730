// ssm_scan_bwd.cuh -- gradients of the selective scan (included by ssm.cu after ssm_scan.cuh).
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
//
// Layout: a lane holds two neighbouring channels by four states.  The sums over channels (dB, dC:
// 8 values a token) and over states (q, r, y: 6 values) are butterflies that halve the number
// of values at every round, so that a token costs 7 + 6 exchanges at 16 states; four states by
// two channels is where the two together are least.  The scalars of a sub-chunk (t, x, e and
// what the gradients of u, dt, z need) are computed once per channel, spread over the warp.
#pragma once

namespace gtr {
namespace sc {

constexpr int kSub = 4, kMaxChunkBwd = 64;

// Sums over lanes whose index differs in the bits [LO, HI): v[0 .. NV - 1] of every lane.  While
// a lane holds several values a round exchanges half of them; then whole values.  Lane l ends
// with the sums of the values [idx, idx + left) in v[0 .. left - 1], where idx is returned.
template <int LO, int HI, int NV>
__device__ __forceinline__ int butterfly(float *v, int lane) {
    if constexpr (LO >= HI) {
        return 0;
    } else if constexpr (NV > 1) {
        const bool up = lane & LO;
#pragma unroll
        for (int i = 0; i < NV / 2; ++i) {
            const float send = up ? v[i] : v[i + NV / 2], keep = up ? v[i + NV / 2] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, LO);
        }
        return (up ? NV / 2 : 0) + butterfly<LO * 2, HI, NV / 2>(v, lane);
    } else {
        v[0] += __shfl_xor_sync(0xffffffffu, v[0], LO);
        return butterfly<LO * 2, HI, 1>(v, lane);
    }
}
__host__ __device__ constexpr int left_of(int nv, int lanes) { return nv > lanes ? nv / lanes : 1; }

template <int SP>
struct GradLayout {
    static constexpr int SL = SP / 4;            // lanes that share a channel pair
    static constexpr int CW = 64 / SL;           // channels of a warp
    static constexpr int CT = 4 * CW;            // channels of a block
    static constexpr int NE = kSub * CW / 32;    // (token, channel) entries a lane prepares
    // shared memory, floats: B, C of the chunk; checkpoints; per warp t, x, e and q, r, y; dB, dC
    static constexpr int stage = 6 * kSub * CW;
    static __host__ __device__ constexpr int floats(int L) {
        return 2 * L * SP + L / kSub * kThreads * 8 + 4 * stage + 2 * 4 * kSub * 2 * SP;
    }
};

template <typename T, int SP>
__global__ void __launch_bounds__(kThreads) ssm_grad_kernel(const Args a) {
    using Lay = GradLayout<SP>;
    constexpr int SL = Lay::SL, CW = Lay::CW, NE = Lay::NE;
    extern __shared__ __align__(16) float sm[];
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
    const bool gate = a.z != nullptr;

    for (int i = tid; i < (p1 - p0) * SP; i += kThreads) {
        const int n = i % SP;
        const long long row = row0 + token_of(p0 + i / SP, a.H, a.W, a.dir);
        sB[i] = Elem<T>::get(ld16(a.bm + row * a.ldb + n, n < a.S));
        sC[i] = Elem<T>::get(ld16(a.cm + row * a.ldc + n, n < a.S));
    }

    float A2[2][4], h[2][4], g[2][4], dA[2][4];
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
                A2[k][i] = in ? __ldg(a.A + (long long)(c + k) * a.S + n) * kLog2e : 0.f;
                h[k][i] = in && hs != nullptr ? hs[(long long)(c + k) * hst + n] : 0.f;
                g[k][i] = in && gs != nullptr ? gs[(long long)(c + k) * gst + n] : 0.f;
                dA[k][i] = 0.f;
            }
    }
    // the entries (token, channel) of a sub-chunk that this lane prepares: channel lane % CW of
    // tokens lane / CW + (32 / CW) e
    const int ec = cb + lane % CW;
    const bool ecv = ec < a.D;
    const float dtb = a.dtb != nullptr && ecv ? __ldg(a.dtb + ec) : 0.f;
    const float Dk = a.Dk != nullptr && ecv ? __ldg(a.Dk + ec) : 0.f;
    float accD = 0.f, accT = 0.f;
    bool bad = false;
    __syncthreads();

    // sweep: checkpoints of the states entering the sub-chunks
    for (int s = 0; s < nsub; ++s) {
        ck[(s * 2 + 0) * kThreads + tid] = make_float4(h[0][0], h[0][1], h[0][2], h[0][3]);
        ck[(s * 2 + 1) * kThreads + tid] = make_float4(h[1][0], h[1][1], h[1][2], h[1][3]);
        if (s == nsub - 1) break;
        __syncwarp();
#pragma unroll
        for (int e = 0; e < NE; ++e) {   // every sub-chunk but the last is whole
            const int tt = (lane + 32 * e) / CW;
            const long long row = row0 + token_of(p0 + s * kSub + tt, a.H, a.W, a.dir);
            const float raw = Elem<T>::get(ld16(a.dt + row * a.lddt + ec, ecv)) + dtb;
            const float t = a.softplus ? softplus_f(raw) : raw;
            st[tt * CW + lane % CW] = t;
            sx[tt * CW + lane % CW] = t * Elem<T>::get(ld16(a.u + row * a.ldu + ec, ecv));
        }
        __syncwarp();
#pragma unroll
        for (int tt = 0; tt < kSub; ++tt) {
            const float2 t = *reinterpret_cast<const float2 *>(st + tt * CW + 2 * pr);
            const float2 x = *reinterpret_cast<const float2 *>(sx + tt * CW + 2 * pr);
            const float4 B = *reinterpret_cast<const float4 *>(sB + (s * kSub + tt) * SP + sl * 4);
            const float Bv[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[0][i] = fmaf(ex2(t.x * A2[0][i]), h[0][i], x.x * Bv[i]);
                h[1][i] = fmaf(ex2(t.y * A2[1][i]), h[1][i], x.y * Bv[i]);
            }
        }
    }

    // sub-chunks from the last to the first
    for (int s = nsub - 1; s >= 0; --s) {
        const int q0 = p0 + s * kSub, m = min(kSub, p1 - q0);
        float eu[NE], et[NE], ee[NE], esg[NE], ez[NE], ey[NE];   // u, t, e, sigmoid(raw), z, d_out
        long long er[NE];
        __syncwarp();
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int tt = (lane + 32 * e) / CW;
            const bool in = ecv && tt < m;
            er[e] = row0 + token_of(tt < m ? q0 + tt : q0, a.H, a.W, a.dir);
            eu[e] = Elem<T>::get(ld16(a.u + er[e] * a.ldu + ec, in));
            const float raw = Elem<T>::get(ld16(a.dt + er[e] * a.lddt + ec, in)) + dtb;
            ey[e] = Elem<T>::get(ld16(a.dy + er[e] * a.lddy + ec, in));
            ez[e] = Elem<T>::get(ld16(a.z + er[e] * a.ldz + ec, in && gate));
            et[e] = a.softplus ? softplus_f(raw) : raw;
            esg[e] = a.softplus ? sigmoid_f(raw) : 1.f;
            ee[e] = gate ? ey[e] * (ez[e] * sigmoid_f(ez[e])) : ey[e];
            st[tt * CW + lane % CW] = et[e];
            sx[tt * CW + lane % CW] = et[e] * eu[e];
            se[tt * CW + lane % CW] = ee[e];
        }
        __syncwarp();
        float d[kSub][2][4], hp[kSub][2][4];   // decays; states entering the tokens
        {
            const float4 c0 = ck[(s * 2 + 0) * kThreads + tid], c1 = ck[(s * 2 + 1) * kThreads + tid];
            h[0][0] = c0.x, h[0][1] = c0.y, h[0][2] = c0.z, h[0][3] = c0.w;
            h[1][0] = c1.x, h[1][1] = c1.y, h[1][2] = c1.z, h[1][3] = c1.w;
        }
#pragma unroll
        for (int tt = 0; tt < kSub; ++tt) {
            if (tt >= m) break;   // the same for the whole block
            const float2 t = *reinterpret_cast<const float2 *>(st + tt * CW + 2 * pr);
            const float2 x = *reinterpret_cast<const float2 *>(sx + tt * CW + 2 * pr);
            const float4 B = *reinterpret_cast<const float4 *>(sB + (s * kSub + tt) * SP + sl * 4);
            const float Bv[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hp[tt][0][i] = h[0][i];
                hp[tt][1][i] = h[1][i];
                d[tt][0][i] = ex2(t.x * A2[0][i]);
                d[tt][1][i] = ex2(t.y * A2[1][i]);
                h[0][i] = fmaf(d[tt][0][i], h[0][i], x.x * Bv[i]);
                h[1][i] = fmaf(d[tt][1][i], h[1][i], x.y * Bv[i]);
            }
        }
        float *ws = wsum + (s & 1) * 4 * kSub * 2 * SP + warp * kSub * 2 * SP;
#pragma unroll
        for (int tt = kSub - 1; tt >= 0; --tt) {
            if (tt >= m) continue;
            const float2 t = *reinterpret_cast<const float2 *>(st + tt * CW + 2 * pr);
            const float2 x = *reinterpret_cast<const float2 *>(sx + tt * CW + 2 * pr);
            const float2 e = *reinterpret_cast<const float2 *>(se + tt * CW + 2 * pr);
            const float4 B = *reinterpret_cast<const float4 *>(sB + (s * kSub + tt) * SP + sl * 4);
            const float4 C = *reinterpret_cast<const float4 *>(sC + (s * kSub + tt) * SP + sl * 4);
            const float Bv[4] = {B.x, B.y, B.z, B.w}, Cv[4] = {C.x, C.y, C.z, C.w};
            float vbc[8];                                  // dB[4], dC[4] of this lane's channels
            float vs[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};   // q, r, y of both, two unused
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float tk = k ? t.y : t.x, xk = k ? x.y : x.x, ek = k ? e.y : e.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // the state after the token: the next token's entering state, or the last
                    const float hn = tt + 1 < kSub ? (tt + 1 < m ? hp[tt + 1 < kSub ? tt + 1 : tt][k][i] : h[k][i]) : h[k][i];
                    const float G = fmaf(ek, Cv[i], g[k][i]);
                    const float Ga = G * d[tt][k][i], w = Ga * hp[tt][k][i];
                    vs[k] = fmaf(G, Bv[i], vs[k]);
                    vs[2 + k] = fmaf(w, A2[k][i], vs[2 + k]);
                    vs[4 + k] = fmaf(Cv[i], hn, vs[4 + k]);
                    dA[k][i] = fmaf(w, tk, dA[k][i]);
                    vbc[i] = k ? fmaf(G, xk, vbc[i]) : G * xk;
                    vbc[4 + i] = k ? fmaf(ek, hn, vbc[4 + i]) : ek * hn;
                    g[k][i] = Ga;
                }
            }
            const int ib = butterfly<SL, 32, 8>(vbc, lane);   // over the channels of the warp
            constexpr int lb = left_of(8, 32 / SL);
#pragma unroll
            for (int i = 0; i < lb; ++i) {
                const int v = ib + i;   // 0..3 dB, 4..7 dC of states sl * 4 + v % 4
                ws[tt * 2 * SP + (v >= 4 ? SP : 0) + sl * 4 + (v & 3)] = vbc[i];
            }
            const int is = butterfly<1, SL, 8>(vs, lane);     // over the states of the channels
            constexpr int ls = left_of(8, SL);
#pragma unroll
            for (int i = 0; i < ls; ++i) {
                const int v = is + i;   // q, q, r, r, y, y, -, -
                if (v < 6) rq[(v >> 1) * kSub * CW + tt * CW + 2 * pr + (v & 1)] = vs[i];
            }
        }
        __syncthreads();   // the warps' sums of dB, dC (two buffers: the next sub-chunk writes the other)
        for (int i = tid; i < m * 2 * SP; i += kThreads) {
            const float *w0 = wsum + (s & 1) * 4 * kSub * 2 * SP + i;
            const float v = w0[0] + w0[kSub * 2 * SP] + w0[2 * kSub * 2 * SP] + w0[3 * kSub * 2 * SP];
            const long long row = row0 + token_of(q0 + i / (2 * SP), a.H, a.W, a.dir);
            a.pbc[((long long)ct * a.B * a.N + row) * 2 * SP + i % (2 * SP)] = v;
        }
#pragma unroll
        for (int e = 0; e < NE; ++e) {
            const int tt = (lane + 32 * e) / CW, ix = tt * CW + lane % CW;
            if (!ecv || tt >= m) continue;
            const float q = rq[ix], r = rr[ix] * kLn2;   // A2 = A log2(e)
            const float du = fmaf(q, et[e], Dk * ee[e]);
            const float dr = fmaf(q, eu[e], r) * esg[e];
            accD = fmaf(ee[e], eu[e], accD);
            accT += dr;
            const long long o = er[e] * a.D + ec;
            a.du[o] = Elem<T>::put(du);
            a.ddt[o] = Elem<T>::put(dr);
            bad |= Elem<T>::bad(du) | Elem<T>::bad(dr);
            if (gate) {
                const float y = fmaf(Dk, eu[e], ry[ix]), sg = sigmoid_f(ez[e]);
                const float dz = ey[e] * y * (sg * fmaf(ez[e], 1.f - sg, 1.f));
                a.dz[o] = Elem<T>::put(dz);
                bad |= Elem<T>::bad(dz);
            }
        }
    }
    if (bad) set_error(kOpsErrRange);

    // the chunk's share of dA over the state slot that only this chunk reads (chunk 0: the last
    // slot, which nothing reads), of dD and of ddt_bias
    float *pa = a.hs + ((long long)b * a.P + (j > 0 ? j - 1 : a.P - 1)) * a.D * SP;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (!cv[k]) continue;
        *reinterpret_cast<float4 *>(pa + (long long)(c + k) * SP + sl * 4) =
            make_float4(dA[k][0], dA[k][1], dA[k][2], dA[k][3]);
        if (j == 0 && a.dh0 != nullptr) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (sl * 4 + i < a.S) a.dh0[((long long)b * a.D + c + k) * a.S + sl * 4 + i] = g[k][i];
        }
    }
#pragma unroll
    for (int o = CW; o < 32; o *= 2) {
        accD += __shfl_xor_sync(0xffffffffu, accD, o);
        accT += __shfl_xor_sync(0xffffffffu, accT, o);
    }
    if (lane < CW && ecv) {
        a.pd[((long long)b * a.P + j) * a.D + ec] = accD;
        a.pt[((long long)b * a.P + j) * a.D + ec] = accT;
    }
}

// Adds the partial sums in a fixed order.  The first `bc_blocks` blocks: dB and dC, one thread a
// (token, state), over the channel tiles; the rest: dA, dD, ddt_bias over the chunks, 32 columns
// by 8 row lanes a block.
template <typename T, int SP>
__global__ void __launch_bounds__(256) ssm_grad_sum_kernel(const Args a, int bc_blocks) {
    __shared__ float red[8][33];
    if ((int)blockIdx.x < bc_blocks) {
        const long long id = (long long)blockIdx.x * 256 + threadIdx.x, rows = (long long)a.B * a.N;
        const long long row = id / (2 * SP);
        const int v = (int)(id % (2 * SP)), n = v % SP;
        if (row >= rows || n >= a.S) return;
        float s = 0.f;
        for (int k = 0; k < a.tiles; ++k) s += a.pbc[((long long)k * rows + row) * 2 * SP + v];
        (v < SP ? a.dB : a.dC)[row * a.S + n] = Elem<T>::put(s);
        if (Elem<T>::bad(s)) set_error(kOpsErrRange);
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
