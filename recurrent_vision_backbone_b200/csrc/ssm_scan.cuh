// ssm_scan.cuh -- the selective scan, forward, backward and for single tokens
// (included by ssm.cu, which holds the C entry points).
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
// Walk layout: two neighbouring lanes share two neighbouring channels, each lane holding half
// of the states of both (NS states of its own channel and of its neighbour's).  A lane loads its
// own channel only; the time step and the input are exchanged by one shuffle each, the partial
// sums of y by another, and a warp reads 64 consecutive bytes of every row.  B and C of a tile of
// kTok tokens are staged in shared memory as float32 and read as broadcasts, each value serving
// two channels.  The next tile's rows are requested before a tile is computed.
#pragma once

namespace gtr {
namespace sc {

using namespace ops;

constexpr int kThreads = 128, kTok = 8;

struct Args {
    const uint16_t *u, *dt, *bm, *cm, *z, *dy;
    const float *A, *Dk, *dtb, *h0, *dfin;
    uint16_t *out;
    float *hf;
    long long ldu, lddt, ldb, ldc, ldz, lddy;
    int B, H, W, N, D, S, dir, softplus;
    int P, L, tiles;                // chunks a sequence, tokens a chunk, channel tiles
    float *hs, *gs, *sdt;           // workspace: [B][P][D][SP], the same, [B][P][D]
    // backward
    uint16_t *du, *ddt, *dz, *dB, *dC;
    float *dA, *dD, *ddtb, *dh0;
    float *pbc, *pd, *pt;           // workspace: [tiles][B N][2 SP], [B P][D], [B P][D]
};

__device__ __forceinline__ float2 f2(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint16_t ld16(const uint16_t *p, bool in) { return in ? __ldg(p) : (uint16_t)0; }

enum { kLocal = 0, kOut = 1, kLocalBwd = 2 };

// One walk over one chunk.  kLocal: hs[b][j] = the state reached from zero, sdt = the sum of the
// time steps.  kLocalBwd: also gs[b][j] = sum_p (prod_{r <= p} a_r) C_p dy_p, the gradient that
// the chunk's outputs send to the state entering it.  kOut: outputs and the final state.
template <typename T, int NS, int MODE>
__global__ void __launch_bounds__(kThreads) ssm_walk_kernel(const Args a) {
    constexpr int SP = 2 * NS;                  // states, padded with zero B and C
    constexpr int kStage = kTok * SP * 2 / kThreads;   // B and C values a thread stages per tile
    static_assert(kStage >= 1, "a tile of B and C has at least one value a thread");
    __shared__ __align__(16) float bc[2][2][kTok][SP];
    const int tid = threadIdx.x, lane = tid & 31, sl = lane & 1;
    const int ct = blockIdx.x % a.tiles;
    const int cj = blockIdx.x / a.tiles;
    const int nj = MODE == kLocal ? a.P - 1 : a.P;   // the last chunk's reached state is not needed
    const int b = cj / nj, j = cj - b * nj;
    const int p0 = j * a.L, p1 = min(a.N, p0 + a.L);
    const int c = ct * kThreads + tid, co = c ^ 1, n0 = sl * NS;
    const bool cv = c < a.D, cov = co < a.D;
    const long long row0 = (long long)b * a.N;

    float2 Ao[NS / 2], Ax[NS / 2], ho[NS / 2], hx[NS / 2];   // own channel, exchanged channel
    float2 po[NS / 2], px[NS / 2], go[NS / 2], gx[NS / 2];   // kLocalBwd only
    const float *hin = nullptr;
    long long hstride = SP;
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
    for (int k = 0; k < NS; ++k) {
        const int n = n0 + k;
        const bool in = n < a.S;
        float *A1 = k & 1 ? &Ao[k / 2].y : &Ao[k / 2].x, *A2 = k & 1 ? &Ax[k / 2].y : &Ax[k / 2].x;
        float *h1 = k & 1 ? &ho[k / 2].y : &ho[k / 2].x, *h2 = k & 1 ? &hx[k / 2].y : &hx[k / 2].x;
        *A1 = in && cv ? __ldg(a.A + (long long)c * a.S + n) * kLog2e : 0.f;
        *A2 = in && cov ? __ldg(a.A + (long long)co * a.S + n) * kLog2e : 0.f;
        *h1 = hin != nullptr && in && cv ? hin[(long long)c * hstride + n] : 0.f;
        *h2 = hin != nullptr && in && cov ? hin[(long long)co * hstride + n] : 0.f;
    }
    if (MODE == kLocalBwd) {
#pragma unroll
        for (int k = 0; k < NS / 2; ++k) po[k] = px[k] = f2(1.f), go[k] = gx[k] = f2(0.f);
    }
    const float dtb = a.dtb != nullptr && cv ? __ldg(a.dtb + c) : 0.f;
    const float Dk = MODE == kOut && a.Dk != nullptr && cv ? __ldg(a.Dk + c) : 0.f;
    const bool gate = a.z != nullptr && MODE != kLocal;
    float ssum = 0.f;
    bool bad = false;

    // requests of one tile: this thread's channel of kTok rows, its share of B and C
    Walk wk(p0, a.H, a.W, a.dir);
    uint16_t ru[kTok], rt[kTok], rz[kTok], ry[kTok], rb[kStage];
    auto fetch = [&](int pb) {
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const bool in = cv && pb + i < p1;
            const long long row = row0 + wk.n;
            ru[i] = ld16(a.u + row * a.ldu + c, in);
            rt[i] = ld16(a.dt + row * a.lddt + c, in);
            if (MODE != kLocal) rz[i] = ld16(a.z + row * a.ldz + c, in && gate);
            if (MODE == kLocalBwd) ry[i] = ld16(a.dy + row * a.lddy + c, in);
            wk.next();
        }
#pragma unroll
        for (int i = 0; i < kStage; ++i) {
            const int e = tid + i * kThreads, n = e % SP, p = pb + e / SP % kTok;
            const bool isc = e >= kTok * SP;
            const bool in = p < p1 && n < a.S;
            const long long row = row0 + token_of(in ? p : p0, a.H, a.W, a.dir);
            rb[i] = isc ? ld16(a.cm + row * a.ldc + n, in && MODE != kLocal) : ld16(a.bm + row * a.ldb + n, in);
        }
    };
    fetch(p0);
    Walk wo(p0, a.H, a.W, a.dir);
    int buf = 0;
    for (int pb = p0; pb < p1; pb += kTok, buf ^= 1) {
#pragma unroll
        for (int i = 0; i < kStage; ++i) {
            const int e = tid + i * kThreads;
            bc[buf][e / (kTok * SP)][e / SP % kTok][e % SP] = Elem<T>::get(rb[i]);
        }
        float u[kTok], t[kTok], z[kTok], y[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            u[i] = Elem<T>::get(ru[i]);
            const float raw = Elem<T>::get(rt[i]) + dtb;
            t[i] = a.softplus ? softplus_f(raw) : raw;
            if (MODE != kLocal) z[i] = Elem<T>::get(rz[i]);
            if (MODE == kLocalBwd) y[i] = Elem<T>::get(ry[i]) * (gate ? z[i] * sigmoid_f(z[i]) : 1.f);
        }
        // one barrier a tile: a thread that writes buffer b again has passed the barrier of the
        // tile between, which every thread reaches after its last read of b
        __syncthreads();
        fetch(pb + kTok);
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            if (pb + i >= p1) break;   // the same for the whole block
            const float x = t[i] * u[i];
            const float tx = __shfl_xor_sync(0xffffffffu, t[i], 1), xx = __shfl_xor_sync(0xffffffffu, x, 1);
            if (MODE != kOut) ssum += t[i];
            float yx = 0.f;
            if (MODE == kLocalBwd) yx = __shfl_xor_sync(0xffffffffu, y[i], 1);
            float2 so = f2(0.f), sx = f2(0.f);
            const float2 *B2 = reinterpret_cast<const float2 *>(&bc[buf][0][i][n0]);
            const float2 *C2 = reinterpret_cast<const float2 *>(&bc[buf][1][i][n0]);
#pragma unroll
            for (int k = 0; k < NS / 2; ++k) {
                const float2 Bk = B2[k];
                float2 e = __fmul2_rn(f2(t[i]), Ao[k]);
                float2 d = make_float2(ex2(e.x), ex2(e.y));
                float2 e2 = __fmul2_rn(f2(tx), Ax[k]);
                float2 d2 = make_float2(ex2(e2.x), ex2(e2.y));
                ho[k] = __ffma2_rn(d, ho[k], __fmul2_rn(f2(x), Bk));
                hx[k] = __ffma2_rn(d2, hx[k], __fmul2_rn(f2(xx), Bk));
                if (MODE == kOut) {
                    so = __ffma2_rn(C2[k], ho[k], so);
                    sx = __ffma2_rn(C2[k], hx[k], sx);
                }
                if (MODE == kLocalBwd) {
                    po[k] = __fmul2_rn(po[k], d);
                    px[k] = __fmul2_rn(px[k], d2);
                    go[k] = __ffma2_rn(po[k], __fmul2_rn(f2(y[i]), C2[k]), go[k]);
                    gx[k] = __ffma2_rn(px[k], __fmul2_rn(f2(yx), C2[k]), gx[k]);
                }
            }
            if (MODE == kOut) {
                float s = so.x + so.y + __shfl_xor_sync(0xffffffffu, sx.x + sx.y, 1);
                s = fmaf(Dk, u[i], s);
                if (gate) s *= z[i] * sigmoid_f(z[i]);
                if (cv) {
                    a.out[(row0 + wo.n) * a.D + c] = Elem<T>::put(s);
                    bad |= Elem<T>::bad(s);
                }
                wo.next();
            }
        }
    }
    if (MODE == kOut) {
        if (bad) set_error(kOpsErrRange);
        if (j != a.P - 1 || a.hf == nullptr) return;
    }
    float *dst = MODE == kOut ? a.hf + (long long)b * a.D * a.S : a.hs + ((long long)b * a.P + j) * a.D * SP;
    const int ds = MODE == kOut ? a.S : SP;
#pragma unroll
    for (int k = 0; k < NS; ++k) {
        const int n = n0 + k;
        if (MODE == kOut && n >= a.S) continue;
        const float h1 = k & 1 ? ho[k / 2].y : ho[k / 2].x, h2 = k & 1 ? hx[k / 2].y : hx[k / 2].x;
        if (cv) dst[(long long)c * ds + n] = h1;
        if (cov) dst[(long long)co * ds + n] = h2;
        if (MODE == kLocalBwd) {
            float *gd = a.gs + ((long long)b * a.P + j) * a.D * SP;
            if (cv) gd[(long long)c * SP + n] = k & 1 ? go[k / 2].y : go[k / 2].x;
            if (cov) gd[(long long)co * SP + n] = k & 1 ? gx[k / 2].y : gx[k / 2].x;
        }
    }
    if (MODE != kOut && cv) a.sdt[((long long)b * a.P + j) * a.D + c] = ssum;
}

// The chunks in order, one thread per (batch, channel, state).  Forward: hs[j] becomes the state
// leaving chunk j.  Backward (from the last chunk): gs[j] becomes the gradient of the state
// entering chunk j.  The loads of kFold chunks are issued before the chain uses the first.
constexpr int kFold = 8;
template <int SP, bool BWD>
__global__ void __launch_bounds__(256) ssm_fold_kernel(const Args a) {
    const long long per = (long long)a.D * SP;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int b = (int)(id / per);
    if (b >= a.B) return;
    const long long e = id - b * per;
    const int d = (int)(e / SP), n = (int)(e % SP);
    const float A2 = n < a.S ? __ldg(a.A + (long long)d * a.S + n) * kLog2e : 0.f;
    const float *sd = a.sdt + (long long)b * a.P * a.D + d;
    const int m = a.P - 1;
    {
        float *hs = a.hs + (long long)b * a.P * per + e;
        float h = a.h0 != nullptr && n < a.S ? a.h0[((long long)b * a.D + d) * a.S + n] : 0.f;
        if (!BWD) hs[m * per] = h;   // the last slot is free: the entering state of chunk 0
        for (int j0 = 0; j0 < m; j0 += kFold) {
            float v[kFold], s[kFold];
#pragma unroll
            for (int i = 0; i < kFold; ++i) {
                const int j = min(j0 + i, m - 1);
                v[i] = hs[j * per];
                s[i] = sd[(long long)j * a.D];
            }
#pragma unroll
            for (int i = 0; i < kFold; ++i)
                if (j0 + i < m) {
                    h = fmaf(ex2(A2 * s[i]), h, v[i]);
                    hs[(j0 + i) * per] = h;
                }
        }
    }
    if (BWD) {
        float *gs = a.gs + (long long)b * a.P * per + e;
        float g = a.dfin != nullptr && n < a.S ? a.dfin[((long long)b * a.D + d) * a.S + n] : 0.f;
        for (int j0 = m; j0 >= 1; j0 -= kFold) {
            float v[kFold], s[kFold];
#pragma unroll
            for (int i = 0; i < kFold; ++i) {
                const int j = max(j0 - i, 1);
                v[i] = gs[j * per];
                s[i] = sd[(long long)j * a.D];
            }
#pragma unroll
            for (int i = 0; i < kFold; ++i)
                if (j0 - i >= 1) {
                    g = fmaf(ex2(A2 * s[i]), g, v[i]);
                    gs[(j0 - i) * per] = g;
                }
        }
    }
}

// One token of every sequence: the states are the traffic (read and written once, 8 bytes a
// state against 8 bytes a channel), so lanes run along a channel's states, 16 bytes each: a
// warp reads and writes whole lines.  S / 4 lanes a channel (S = 4, 8, 16 or 32).
template <typename T, int S>
__global__ void __launch_bounds__(256) ssm_token_kernel(const Args a) {
    constexpr int SL = S / 4;
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int q = (int)(id % SL);
    const long long ch = id / SL;
    const bool live = ch < (long long)a.B * a.D;
    const int b = live ? (int)(ch / a.D) : 0, c = live ? (int)(ch - (long long)b * a.D) : 0;
    float4 h = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && a.h0 != nullptr) h = *reinterpret_cast<const float4 *>(a.h0 + ch * S + q * 4);
    const float4 A = __ldg(reinterpret_cast<const float4 *>(a.A + (long long)c * S + q * 4));
    const float u = Elem<T>::get(__ldg(a.u + b * a.ldu + c));
    const float raw = Elem<T>::get(__ldg(a.dt + b * a.lddt + c)) + (a.dtb != nullptr ? __ldg(a.dtb + c) : 0.f);
    float Bv[4], Cv[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        Bv[k] = Elem<T>::get(__ldg(a.bm + b * a.ldb + q * 4 + k));
        Cv[k] = Elem<T>::get(__ldg(a.cm + b * a.ldc + q * 4 + k));
    }
    const float zz = a.z != nullptr ? Elem<T>::get(__ldg(a.z + b * a.ldz + c)) : 0.f;
    const float t = a.softplus ? softplus_f(raw) : raw, x = t * u;
    h.x = fmaf(ex2(t * (A.x * kLog2e)), h.x, x * Bv[0]);
    h.y = fmaf(ex2(t * (A.y * kLog2e)), h.y, x * Bv[1]);
    h.z = fmaf(ex2(t * (A.z * kLog2e)), h.z, x * Bv[2]);
    h.w = fmaf(ex2(t * (A.w * kLog2e)), h.w, x * Bv[3]);
    if (live && a.hf != nullptr) *reinterpret_cast<float4 *>(a.hf + ch * S + q * 4) = h;
    float y = fmaf(Cv[0], h.x, fmaf(Cv[1], h.y, fmaf(Cv[2], h.z, Cv[3] * h.w)));
#pragma unroll
    for (int o = 1; o < SL; o *= 2) y += __shfl_xor_sync(0xffffffffu, y, o);
    if (live && q == 0) {
        if (a.Dk != nullptr) y = fmaf(__ldg(a.Dk + c), u, y);
        if (a.z != nullptr) y *= zz * sigmoid_f(zz);
        a.out[ch] = Elem<T>::put(y);
        if (Elem<T>::bad(y)) set_error(kOpsErrRange);
    }
}

}  // namespace sc
}  // namespace gtr
