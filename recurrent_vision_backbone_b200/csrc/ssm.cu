// ssm.cu -- the selective state-space mixer behind the C ABI of include/gtr_ssm.h: the short
// causal convolution (causal_conv.cuh) and the selective scan (ssm_scan.cuh, ssm_scan_bwd.cuh).
#include "../../include/gtr_ssm.h"
#include "ops_common.cuh"

namespace gtr {
static __device__ unsigned int g_ssm_error_word;
static __device__ __forceinline__ void set_error(unsigned e) { atomicOr(&g_ssm_error_word, e); }
}  // namespace gtr

#include "causal_conv.cuh"
#include "ssm_scan.cuh"
#include "ssm_scan_bwd.cuh"

namespace gtr {

unsigned ssm_take_errors() {
    unsigned word = 0;
    if (cudaMemcpyFromSymbol(&word, g_ssm_error_word, sizeof(word)) != cudaSuccess) return kOpsErrCuda;
    if (word != 0) {
        const unsigned zero = 0;
        if (cudaMemcpyToSymbol(g_ssm_error_word, &zero, sizeof(zero)) != cudaSuccess) return kOpsErrCuda;
    }
    return word;
}

using namespace ops;

static bool bad_common(int B, int H, int W, int D, int dir, int dtype) {
    if (B <= 0 || D <= 0 || H < 0 || W < 0 || dir < 0 || dir > 3) return true;
    if (dtype != GTR_F16 && dtype != GTR_BF16) return true;
    const long long N = (long long)H * W;
    return N > kMaxTokens || (long long)B * N > kMaxElements / D;
}
// A [B, N, cols] activation with rows ld apart: present, aligned, rows that do not overlap.
static bool bad_rows(const void *p, long long ld, int cols, long long rows) {
    if (rows == 0) return ld < 0;
    return p == nullptr || !aligned_to(p, 2) || (ld != 0 && ld < cols) || (ld > 0 && rows > (kMaxElements << 4) / ld);
}
static bool bad_f32(const void *p, bool required) { return p == nullptr ? required : !aligned_to(p, 16); }

static bool any_overlap(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int k = 0; k < ni; ++k)
            if (overlap(outs[i], ins[k])) return true;
        for (int k = i + 1; k < no; ++k)
            if (overlap(outs[i], outs[k])) return true;
    }
    return false;
}

constexpr long long kMaxGrid = 0x7fffffffLL;

// ------------------------------------------------------------------ convolution
struct ConvPlan {
    long long tiles;    // chunks of a sequence
    long long parts;    // chunks
    int tile;           // positions of a chunk
};
// Backward: chunks enough for one wave of eight blocks an SM (every block writes a partial row of the
// parameters' sums), of 32 positions at least (each recomputes K - 1 more).
static ConvPlan conv_bwd_plan(int B, long long N, int D) {
    ConvPlan p{};
    const long long blocks_c = (D + 127) / 128;
    long long tiles = 148 * 8 / (blocks_c * B);
    if (tiles < 1) tiles = 1;
    long long tile = (N + tiles - 1) / tiles;
    if (tile < 32) tile = 32;
    p.tile = (int)tile;
    p.tiles = (N + tile - 1) / tile;
    p.parts = (long long)B * p.tiles;
    return p;
}

static gtr_status_t check_conv(const gtr_conv_t *c) {
    if (c == nullptr || bad_common(c->B, c->Hgrid, c->Wgrid, c->D, c->direction, c->dtype)) return GTR_ERR_INVALID_ARG;
    if (c->activation != GTR_ACT_NONE && c->activation != GTR_ACT_SILU) return GTR_ERR_INVALID_ARG;
    if (c->K <= 0) return GTR_ERR_INVALID_ARG;
    if (c->K < 2 || c->K > 4) return GTR_ERR_UNSUPPORTED;
    const long long rows = (long long)c->B * c->Hgrid * c->Wgrid;
    if (bad_rows(c->x, c->ldx, c->D, rows) || bad_f32(c->w, rows > 0) || bad_f32(c->bias, false) ||
        (c->init_state && !aligned_to(c->init_state, 2)))
        return GTR_ERR_INVALID_ARG;
    return GTR_OK;
}

static cv::Args conv_args(const gtr_conv_t *c) {
    cv::Args a{};
    a.x = static_cast<const uint16_t *>(c->x);
    a.init = static_cast<const uint16_t *>(c->init_state);
    a.w = c->w;
    a.bias = c->bias;
    a.ldx = c->ldx ? c->ldx : c->D;
    a.B = c->B;
    a.H = c->Hgrid;
    a.W = c->Wgrid;
    a.N = c->Hgrid * c->Wgrid;
    a.D = c->D;
    a.dir = c->direction;
    a.act = c->activation;
    return a;
}

// Whether every row of every tensor starts on a `bytes` boundary and holds whole pieces of them.
static bool rows_on(int bytes, int D, const void *const *ps, int np, const long long *lds, int nl) {
    if (D * 2LL % bytes) return false;
    for (int i = 0; i < np; ++i)
        if (ps[i] && !aligned_to(ps[i], bytes)) return false;
    for (int i = 0; i < nl; ++i)
        if (lds[i] * 2 % bytes) return false;
    return true;
}

template <typename T, int V, int K, int TP>
static cudaError_t conv_fwd_launch(cv::Args a, cudaStream_t s) {
    a.groups = (a.D + V - 1) / V;
    a.tiles = (a.N + TP - 1) / TP;
    const long long blocks = ((long long)a.B * a.tiles * a.groups + cv::kThreads - 1) / cv::kThreads;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    return launch_after(cv::causal_conv_fwd_kernel<T, V, K, TP>, (unsigned)blocks, dim3(cv::kThreads), 0, s, a);
}
template <typename T, int V>
static cudaError_t conv_fwd_k(const cv::Args &a, int K, cudaStream_t s) {
    // four positions a thread instead of eight while eight make fewer than three blocks an SM
    const bool few = (long long)a.B * ((a.N + 7) / 8) * ((a.D + V - 1) / V) < 148LL * 3 * cv::kThreads;
    switch (K) {
    case 2: return few ? conv_fwd_launch<T, V, 2, 4>(a, s) : conv_fwd_launch<T, V, 2, 8>(a, s);
    case 3: return few ? conv_fwd_launch<T, V, 3, 4>(a, s) : conv_fwd_launch<T, V, 3, 8>(a, s);
    default: return few ? conv_fwd_launch<T, V, 4, 4>(a, s) : conv_fwd_launch<T, V, 4, 8>(a, s);
    }
}

template <typename T, int K>
static cudaError_t conv_bwd_launch(cv::Args a, const ConvPlan &p, bool wide, float *gw, float *gb, cudaStream_t s) {
    a.groups = (a.D + 2 * cv::kBwdThreads - 1) / (2 * cv::kBwdThreads);
    const long long blocks = p.parts * a.groups;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_after(wide ? cv::causal_conv_bwd_kernel<T, K, true> : cv::causal_conv_bwd_kernel<T, K, false>,
                                       (unsigned)blocks, dim3(cv::kBwdThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const long long cols = (long long)(K + 1) * a.D;
    return launch_after(cv::causal_conv_sum_kernel<K>, (unsigned)((cols + 31) / 32), dim3(32, 8), 0, s,
                        (const float *)a.part, (int)p.parts, a.D, gw, gb);
}
template <typename T>
static cudaError_t conv_bwd_k(const cv::Args &a, int K, const ConvPlan &p, bool wide, float *gw, float *gb, cudaStream_t s) {
    switch (K) {
    case 2: return conv_bwd_launch<T, 2>(a, p, wide, gw, gb, s);
    case 3: return conv_bwd_launch<T, 3>(a, p, wide, gw, gb, s);
    default: return conv_bwd_launch<T, 4>(a, p, wide, gw, gb, s);
    }
}

// dst = src, or zeros without src.
static gtr_status_t copy_or_zero(void *dst, const void *src, size_t bytes, cudaStream_t s) {
    if (dst == nullptr || dst == src || bytes == 0) return GTR_OK;
    return ops_cuda_status(src != nullptr ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                                          : cudaMemsetAsync(dst, 0, bytes, s));
}

// ------------------------------------------------------------------ scan
constexpr int kSmAim = 148 * 4;   // blocks of four warps that keep the schedulers busy

static int state_pad(int S) { return S <= 8 ? 8 : S <= 16 ? 16 : 32; }

struct ScanPlan {
    int P, L;
    int SL;   // lanes that share a channel in the walk that writes the outputs
};
// The walks of a forward scan.  With 96 blocks of 128 channels or more, one walk over whole
// sequences: two lanes a channel until the channels alone are three warps a scheduler, then one (8 x 2304
// tokens of 2048 channels, 128 blocks: 306 us with two lanes, 425 with one, 384 with four; 397 in four
// chunks).  Below that, as many chunks as make one wave of four blocks an SM, at least 32 tokens each
// (16384 tokens of 1024 channels, 8 blocks: 182 us with 74 chunks, 201 with 92, 250 with 37).
static ScanPlan scan_fwd_plan(int B, long long N, int D) {
    const long long base = (long long)B * ((D + sc::kThreads - 1) / sc::kThreads);
    const long long P = base >= 96 ? 1 : kSmAim / base;
    long long L = (N + P - 1) / P;
    L = (L + 7) / 8 * 8;
    if (L < 32) L = 32;
    if (L > N) L = N;
    ScanPlan r{};
    r.L = (int)L;
    r.P = (int)((N + L - 1) / L);
    r.SL = r.P == 1 && base < 148 * 3 ? 2 : 1;
    return r;
}
static size_t scan_fwd_bytes(int B, int D, int S, const ScanPlan &p) {
    if (p.P <= 1) return 0;
    const size_t rows = (size_t)B * p.P * D;
    return align256(rows * state_pad(S) * sizeof(float)) + align256(rows * sizeof(float));
}

static int grad_tile(int S) {
    const int sp = state_pad(S);
    return sp == 8 ? sc::GradLayout<8>::CT : sp == 16 ? sc::GradLayout<16>::CT : sc::GradLayout<32>::CT;
}
static ScanPlan scan_bwd_plan(int B, long long N, int D, int S) {
    const long long base = (long long)B * ((D + grad_tile(S) - 1) / grad_tile(S));
    // shorter chunks where whole ones would not fill the machine (three blocks an SM) twice
    const int L = base * ((N + sc::kMaxChunkBwd - 1) / sc::kMaxChunkBwd) < 148 * 3 * 2 ? 32 : sc::kMaxChunkBwd;
    ScanPlan r{};
    r.L = L;
    r.P = (int)((N + L - 1) / L);
    return r;
}
struct ScanBwdWs {
    size_t hs, gs, sdt, pbc, pd, pt, bytes;
};
static ScanBwdWs scan_bwd_ws(int B, long long N, int D, int S, const ScanPlan &p) {
    const size_t rows = (size_t)B * p.P * D, sp = (size_t)state_pad(S);
    const size_t tiles = ((size_t)D + grad_tile(S) - 1) / grad_tile(S);
    ScanBwdWs w{};
    w.hs = 0;
    w.gs = w.hs + align256(rows * sp * 4);
    w.sdt = w.gs + (p.P > 1 ? align256(rows * sp * 4) : 0);
    w.pd = w.sdt + (p.P > 1 ? align256(rows * 4) : 0);
    w.pt = w.pd + align256(rows * 4);
    w.pbc = w.pt + align256(rows * 4);
    w.bytes = w.pbc + align256(tiles * B * (size_t)N * 2 * sp * 4);
    return w;
}

static gtr_status_t check_ssm(const gtr_ssm_t *m) {
    if (m == nullptr || bad_common(m->B, m->Hgrid, m->Wgrid, m->D, m->direction, m->dtype)) return GTR_ERR_INVALID_ARG;
    if (m->S <= 0 || (m->dt_softplus != 0 && m->dt_softplus != 1)) return GTR_ERR_INVALID_ARG;
    if (m->S > 32) return GTR_ERR_UNSUPPORTED;
    const long long rows = (long long)m->B * m->Hgrid * m->Wgrid;
    if (bad_rows(m->u, m->ldu, m->D, rows) || bad_rows(m->dt, m->lddt, m->D, rows) ||
        bad_rows(m->Bm, m->ldb, m->S, rows) || bad_rows(m->Cm, m->ldc, m->S, rows) ||
        (m->z != nullptr && bad_rows(m->z, m->ldz, m->D, rows)) || bad_f32(m->A, rows > 0) ||
        bad_f32(m->Dskip, false) || bad_f32(m->dt_bias, false) || bad_f32(m->init_state, false))
        return GTR_ERR_INVALID_ARG;
    return GTR_OK;
}

static sc::Args ssm_args(const gtr_ssm_t *m) {
    sc::Args a{};
    a.u = static_cast<const uint16_t *>(m->u);
    a.dt = static_cast<const uint16_t *>(m->dt);
    a.bm = static_cast<const uint16_t *>(m->Bm);
    a.cm = static_cast<const uint16_t *>(m->Cm);
    a.z = static_cast<const uint16_t *>(m->z);
    a.A = m->A;
    a.Dk = m->Dskip;
    a.dtb = m->dt_bias;
    a.h0 = m->init_state;
    a.ldu = m->ldu ? m->ldu : m->D;
    a.lddt = m->lddt ? m->lddt : m->D;
    a.ldb = m->ldb ? m->ldb : m->S;
    a.ldc = m->ldc ? m->ldc : m->S;
    a.ldz = m->ldz ? m->ldz : m->D;
    a.B = m->B;
    a.H = m->Hgrid;
    a.W = m->Wgrid;
    a.N = m->Hgrid * m->Wgrid;
    a.D = m->D;
    a.S = m->S;
    a.dir = m->direction;
    a.softplus = m->dt_softplus;
    return a;
}
// The input tensors of a scan as byte ranges.
static int ssm_inputs(const gtr_ssm_t *m, const sc::Args &a, Span *s) {
    const long long rows = (long long)a.B * a.N, st = (long long)a.B * a.D * a.S * 4;
    int n = 0;
    s[n++] = {m->u, row_bytes(rows, a.ldu, a.D)};
    s[n++] = {m->dt, row_bytes(rows, a.lddt, a.D)};
    s[n++] = {m->Bm, row_bytes(rows, a.ldb, a.S)};
    s[n++] = {m->Cm, row_bytes(rows, a.ldc, a.S)};
    s[n++] = {m->z, row_bytes(rows, a.ldz, a.D)};
    s[n++] = {m->A, (long long)a.D * a.S * 4};
    s[n++] = {m->Dskip, (long long)a.D * 4};
    s[n++] = {m->dt_bias, (long long)a.D * 4};
    s[n++] = {m->init_state, st};
    return n;
}

template <typename T, int SP, int MODE, int SL>
static cudaError_t walk_launch(const sc::Args &a, bool wide, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)a.tiles * a.B * (MODE == sc::kLocal ? a.P - 1 : a.P));
    const auto kernel = wide ? sc::ssm_walk_kernel<T, SP, MODE, true, SL> : sc::ssm_walk_kernel<T, SP, MODE, false, SL>;
    // A walk that opens a call and covers many SMs starts plainly: blocks that wait on SMs where the
    // call ahead happens to have left room end up unevenly spread (468 us for 428 at 8 x 2304 tokens of
    // 2048 channels)
    if ((MODE != sc::kOut || a.P == 1) && grid > 148) {
        kernel<<<grid, sc::kThreads, 0, s>>>(a);
        return cudaGetLastError();
    }
    return launch_after(kernel, grid, dim3(sc::kThreads), 0, s, a);
}
template <int SP, bool BWD>
static cudaError_t fold_launch(const sc::Args &a, cudaStream_t s) {
    const long long n = (long long)a.B * a.D * SP * (BWD ? 2 : 1);
    return launch_after(sc::ssm_fold_kernel<SP, BWD>, (unsigned)((n + sc::kFoldThreads - 1) / sc::kFoldThreads),
                        dim3(sc::kFoldThreads), 0, s, a);
}
template <typename T, int SP>
static cudaError_t scan_fwd_launch(const sc::Args &a, int sl, bool wide, cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    if (a.P > 1) {
        e = walk_launch<T, SP, sc::kLocal, 1>(a, wide, s);
        if (e == cudaSuccess) e = fold_launch<SP, false>(a, s);
    }
    if (e != cudaSuccess) return e;
    sc::Args o = a;
    o.tiles = (a.D * (long long)sl + sc::kThreads - 1) / sc::kThreads;
    return sl == 1 ? walk_launch<T, SP, sc::kOut, 1>(o, wide, s) : walk_launch<T, SP, sc::kOut, 2>(o, wide, s);
}
template <typename T, int S, int NB>
static cudaError_t token_launch_nb(const sc::Args &a, cudaStream_t s) {
    const long long n = ((long long)a.B + NB - 1) / NB * a.D * (S / 4);
    const bool bcw = aligned_to(a.bm, 8) && aligned_to(a.cm, 8) && (a.B == 1 || (a.ldb % 4 == 0 && a.ldc % 4 == 0));
    return launch_after(bcw ? sc::ssm_token_kernel<T, S, NB, true> : sc::ssm_token_kernel<T, S, NB, false>,
                        (unsigned)((n + 255) / 256), dim3(256), 0, s, a);
}
// As many sequences a thread as lanes share a channel, once that leaves every SM eight blocks or more.
template <typename T, int S>
static cudaError_t token_launch(const sc::Args &a, cudaStream_t s) {
    return (long long)a.B * a.D / 256 >= 148 * 8 ? token_launch_nb<T, S, S / 4>(a, s) : token_launch_nb<T, S, 1>(a, s);
}
template <typename T>
static cudaError_t scan_fwd_dispatch(const sc::Args &a, int sl, bool wide, cudaStream_t s) {
    // one token: lanes along the states; other numbers of states take the walk
    if (a.N == 1) {
        switch (a.S) {
        case 4: return token_launch<T, 4>(a, s);
        case 8: return token_launch<T, 8>(a, s);
        case 16: return token_launch<T, 16>(a, s);
        case 32: return token_launch<T, 32>(a, s);
        }
    }
    switch (state_pad(a.S)) {
    case 8: return scan_fwd_launch<T, 8>(a, sl, wide, s);
    case 16: return scan_fwd_launch<T, 16>(a, sl, wide, s);
    default: return scan_fwd_launch<T, 32>(a, sl, wide, s);
    }
}

template <typename T, int SP>
static cudaError_t scan_bwd_launch(sc::Args a, bool wide, cudaStream_t s) {
    using Lay = sc::GradLayout<SP>;
    const size_t smem = (size_t)Lay::floats(a.L) * sizeof(float);
    const auto grad = a.pairs ? sc::ssm_grad_kernel<T, SP, true> : sc::ssm_grad_kernel<T, SP, false>;
    cudaError_t e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess && a.P > 1) {
        a.tiles = (a.D + sc::kThreads - 1) / sc::kThreads;
        e = walk_launch<T, SP, sc::kLocalBwd, 1>(a, wide, s);
        if (e == cudaSuccess) e = fold_launch<SP, true>(a, s);
    }
    if (e != cudaSuccess) return e;
    a.tiles = (a.D + Lay::CT - 1) / Lay::CT;
    e = launch_after(grad, (unsigned)((long long)a.tiles * a.B * a.P), dim3(sc::kThreads), smem, s, a);
    if (e != cudaSuccess) return e;
    const long long bc = ((long long)a.B * a.N * 2 * SP + 255) / 256, rest = ((long long)a.D * (SP + 2) + 31) / 32;
    return launch_after(sc::ssm_grad_sum_kernel<T, SP>, (unsigned)(bc + rest), dim3(256), 0, s, a, (int)bc);
}
template <typename T>
static cudaError_t scan_bwd_dispatch(const sc::Args &a, bool wide, cudaStream_t s) {
    switch (state_pad(a.S)) {
    case 8: return scan_bwd_launch<T, 8>(a, wide, s);
    case 16: return scan_bwd_launch<T, 16>(a, wide, s);
    default: return scan_bwd_launch<T, 32>(a, wide, s);
    }
}

// Whether the launches of a scan fit a grid (blocks along x only).
static bool grid_too_large(int B, long long N, int D, int S, long long P) {
    const long long sp = state_pad(S), tiles = (D + 31) / 32;
    return (long long)B * P > kMaxGrid || (long long)B * P * tiles > kMaxGrid || (long long)B * D > kMaxGrid * (sc::kFoldThreads / 2) / sp ||
           (long long)B * N > kMaxGrid * 8 / sp - (D * (sp + 2) + 31) / 32;
}

}  // namespace gtr

using namespace gtr;

extern "C" gtr_status_t gtr_causal_conv_fwd(const gtr_conv_t *conv, void *out, void *final_state, void *stream) {
    NvtxRange nvtx_range("gtr_causal_conv_fwd");
    gtr_status_t st = check_conv(conv);
    if (st != GTR_OK) return st;
    cv::Args a = conv_args(conv);
    const long long rows = (long long)a.B * a.N;
    const long long sb = (long long)a.B * (conv->K - 1) * a.D * 2;
    if ((rows > 0 && out == nullptr) || (out && !aligned_to(out, 2)) || (final_state && !aligned_to(final_state, 2)))
        return GTR_ERR_INVALID_ARG;
    const Span ins[] = {{conv->x, row_bytes(rows, a.ldx, a.D)}, {conv->w, (long long)a.D * conv->K * 4},
                        {conv->bias, (long long)a.D * 4},
                        {final_state == conv->init_state ? nullptr : conv->init_state, sb}};
    const Span outs[] = {{out, rows * a.D * 2}, {final_state, sb}};
    if (any_overlap(outs, 2, ins, 4) || (final_state == conv->init_state && overlap(outs[0], {conv->init_state, sb})))
        return GTR_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return copy_or_zero(final_state, conv->init_state, (size_t)sb, s);
    a.out = static_cast<uint16_t *>(out);
    a.fin = static_cast<uint16_t *>(final_state);
    // whole 16-byte pieces of rows where they line up, single elements elsewhere
    const void *ps[] = {a.x, a.out, a.fin, a.init};
    const long long lds[] = {a.ldx};
    const bool wide = rows_on(16, a.D, ps, 4, lds, 1);
    const bool h = conv->dtype == GTR_F16;
    return ops_cuda_status(wide ? (h ? conv_fwd_k<__half, 8>(a, conv->K, s) : conv_fwd_k<__nv_bfloat16, 8>(a, conv->K, s))
                                : (h ? conv_fwd_k<__half, 1>(a, conv->K, s) : conv_fwd_k<__nv_bfloat16, 1>(a, conv->K, s)));
}

extern "C" size_t gtr_causal_conv_bwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int K) {
    if (bad_common(B, Hgrid, Wgrid, D, 0, GTR_F16) || K < 2 || K > 4) return 0;
    const long long N = (long long)Hgrid * Wgrid;
    return N == 0 ? 0 : align256((size_t)conv_bwd_plan(B, N, D).parts * (K + 1) * D * sizeof(float));
}

extern "C" gtr_status_t gtr_causal_conv_bwd(const gtr_conv_t *conv, const void *d_out, long long ld_d_out,
                                            const void *d_final_state, void *grad_x, float *grad_w, float *grad_bias,
                                            void *grad_init_state, void *workspace, size_t workspace_bytes,
                                            void *stream) {
    NvtxRange nvtx_range("gtr_causal_conv_bwd");
    gtr_status_t st = check_conv(conv);
    if (st != GTR_OK) return st;
    cv::Args a = conv_args(conv);
    const long long rows = (long long)a.B * a.N;
    const long long sb = (long long)a.B * (conv->K - 1) * a.D * 2, wb = (long long)a.D * conv->K * 4;
    if (bad_rows(d_out, ld_d_out, a.D, rows) || (rows > 0 && grad_x == nullptr) || (grad_x && !aligned_to(grad_x, 2)) ||
        bad_f32(grad_w, true) || bad_f32(grad_bias, false) || (d_final_state && !aligned_to(d_final_state, 2)) ||
        (grad_init_state && !aligned_to(grad_init_state, 2)))
        return GTR_ERR_INVALID_ARG;
    a.lddy = ld_d_out ? ld_d_out : a.D;
    const size_t need = gtr_causal_conv_bwd_workspace_bytes(a.B, a.H, a.W, a.D, conv->K);
    if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need)) return GTR_ERR_INVALID_ARG;
    const Span ins[] = {{conv->x, row_bytes(rows, a.ldx, a.D)}, {conv->w, wb}, {conv->bias, (long long)a.D * 4},
                        {conv->init_state, sb}, {d_out, row_bytes(rows, a.lddy, a.D)}, {d_final_state, sb}};
    const Span outs[] = {{grad_x, rows * a.D * 2}, {grad_w, wb}, {grad_bias, (long long)a.D * 4}, {grad_init_state, sb},
                         {workspace, (long long)need}};
    if (any_overlap(outs, 5, ins, 6)) return GTR_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        st = copy_or_zero(grad_w, nullptr, (size_t)wb, s);
        if (st == GTR_OK) st = copy_or_zero(grad_bias, nullptr, (size_t)a.D * 4, s);
        return st != GTR_OK ? st : copy_or_zero(grad_init_state, d_final_state, (size_t)sb, s);
    }
    const ConvPlan p = conv_bwd_plan(a.B, a.N, a.D);
    if (p.parts > 0x7fffffffLL) return GTR_ERR_INVALID_ARG;
    a.dy = static_cast<const uint16_t *>(d_out);
    a.dfin = static_cast<const uint16_t *>(d_final_state);
    a.dx = static_cast<uint16_t *>(grad_x);
    a.dinit = static_cast<uint16_t *>(grad_init_state);
    a.part = static_cast<float *>(workspace);
    a.tile = p.tile;
    a.tiles = (int)p.tiles;
    const void *ps[] = {a.x, a.init, a.dy, a.dfin, a.dx, a.dinit};
    const long long lds[] = {a.ldx, a.lddy};
    const bool wide = rows_on(16, a.D, ps, 6, lds, 2);
    return ops_cuda_status(conv->dtype == GTR_F16 ? conv_bwd_k<__half>(a, conv->K, p, wide, grad_w, grad_bias, s)
                                                  : conv_bwd_k<__nv_bfloat16>(a, conv->K, p, wide, grad_w, grad_bias, s));
}

extern "C" size_t gtr_ssm_scan_fwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int S) {
    if (bad_common(B, Hgrid, Wgrid, D, 0, GTR_F16) || S < 1 || S > 32) return 0;
    const long long N = (long long)Hgrid * Wgrid;
    return N == 0 ? 0 : scan_fwd_bytes(B, D, S, scan_fwd_plan(B, N, D));
}

extern "C" gtr_status_t gtr_ssm_scan_fwd(const gtr_ssm_t *ssm, void *out, float *final_state, void *workspace,
                                         size_t workspace_bytes, void *stream) {
    NvtxRange nvtx_range("gtr_ssm_scan_fwd");
    const gtr_status_t st = check_ssm(ssm);
    if (st != GTR_OK) return st;
    sc::Args a = ssm_args(ssm);
    const long long rows = (long long)a.B * a.N, sb = (long long)a.B * a.D * a.S * 4;
    if ((rows > 0 && out == nullptr) || (out && !aligned_to(out, 2)) || bad_f32(final_state, false))
        return GTR_ERR_INVALID_ARG;
    const size_t need = gtr_ssm_scan_fwd_workspace_bytes(a.B, a.H, a.W, a.D, a.S);
    if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need)) return GTR_ERR_INVALID_ARG;
    Span ins[9];
    const int ni = ssm_inputs(ssm, a, ins);
    Span outs[] = {{out, rows * a.D * 2}, {need > 0 ? workspace : nullptr, (long long)need}, {final_state, sb}};
    if (any_overlap(outs, 2, ins, ni)) return GTR_ERR_INVALID_ARG;
    if (final_state == ssm->init_state) ins[ni - 1].p = nullptr;   // in-place carry
    if (any_overlap(outs, 3, ins, ni)) return GTR_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) return copy_or_zero(final_state, ssm->init_state, (size_t)sb, s);
    const ScanPlan p = scan_fwd_plan(a.B, a.N, a.D);
    if (grid_too_large(a.B, 0, a.D, a.S, p.P)) return GTR_ERR_INVALID_ARG;
    a.out = static_cast<uint16_t *>(out);
    a.hf = final_state;
    a.P = p.P;
    a.L = p.L;
    a.tiles = (a.D + sc::kThreads - 1) / sc::kThreads;
    a.hs = static_cast<float *>(workspace);
    a.sdt = a.hs + align256((size_t)a.B * a.P * a.D * state_pad(a.S) * sizeof(float)) / sizeof(float);
    const void *ps[] = {a.u, a.dt, a.z, a.out};
    const long long lds[] = {a.ldu, a.lddt, a.z ? a.ldz : 0};
    const bool wide = rows_on(16, a.D, ps, 4, lds, 3);
    return ops_cuda_status(ssm->dtype == GTR_F16 ? scan_fwd_dispatch<__half>(a, p.SL, wide, s)
                                                 : scan_fwd_dispatch<__nv_bfloat16>(a, p.SL, wide, s));
}

extern "C" size_t gtr_ssm_scan_bwd_workspace_bytes(int B, int Hgrid, int Wgrid, int D, int S) {
    if (bad_common(B, Hgrid, Wgrid, D, 0, GTR_F16) || S < 1 || S > 32) return 0;
    const long long N = (long long)Hgrid * Wgrid;
    return N == 0 ? 0 : scan_bwd_ws(B, N, D, S, scan_bwd_plan(B, N, D, S)).bytes;
}

extern "C" gtr_status_t gtr_ssm_scan_bwd(const gtr_ssm_t *ssm, const void *d_out, long long ld_d_out,
                                         const float *d_final_state, const gtr_ssm_grads_t *grads, void *workspace,
                                         size_t workspace_bytes, void *stream) {
    NvtxRange nvtx_range("gtr_ssm_scan_bwd");
    gtr_status_t st = check_ssm(ssm);
    if (st != GTR_OK) return st;
    if (grads == nullptr) return GTR_ERR_INVALID_ARG;
    sc::Args a = ssm_args(ssm);
    const long long rows = (long long)a.B * a.N, sb = (long long)a.B * a.D * a.S * 4;
    const long long ab = rows * a.D * 2, bb = rows * a.S * 2;
    const bool gate = ssm->z != nullptr;
    void *const act[] = {grads->u, grads->dt, grads->Bm, grads->Cm, gate ? grads->z : nullptr};
    for (int i = 0; i < 5; ++i)
        if ((rows > 0 && act[i] == nullptr && (i < 4 || gate)) || (act[i] && !aligned_to(act[i], 2)))
            return GTR_ERR_INVALID_ARG;
    if (bad_rows(d_out, ld_d_out, a.D, rows) || bad_f32(d_final_state, false) || bad_f32(grads->A, true) ||
        bad_f32(grads->Dskip, false) || bad_f32(grads->dt_bias, false) || bad_f32(grads->init_state, false))
        return GTR_ERR_INVALID_ARG;
    a.lddy = ld_d_out ? ld_d_out : a.D;
    const size_t need = gtr_ssm_scan_bwd_workspace_bytes(a.B, a.H, a.W, a.D, a.S);
    if (need > 0 && (workspace == nullptr || !aligned_to(workspace, 16) || workspace_bytes < need)) return GTR_ERR_INVALID_ARG;
    Span ins[11];
    int ni = ssm_inputs(ssm, a, ins);
    ins[ni++] = {d_out, row_bytes(rows, a.lddy, a.D)};
    ins[ni++] = {d_final_state, sb};
    const Span outs[] = {{act[0], ab}, {act[1], ab}, {act[2], bb}, {act[3], bb}, {act[4], ab},
                         {grads->A, (long long)a.D * a.S * 4}, {grads->Dskip, (long long)a.D * 4},
                         {grads->dt_bias, (long long)a.D * 4}, {grads->init_state, sb},
                         {need > 0 ? workspace : nullptr, (long long)need}};
    if (any_overlap(outs, 10, ins, ni)) return GTR_ERR_INVALID_ARG;
    cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
    if (rows == 0) {
        st = copy_or_zero(grads->A, nullptr, (size_t)a.D * a.S * 4, s);
        if (st == GTR_OK) st = copy_or_zero(grads->Dskip, nullptr, (size_t)a.D * 4, s);
        if (st == GTR_OK) st = copy_or_zero(grads->dt_bias, nullptr, (size_t)a.D * 4, s);
        return st != GTR_OK ? st : copy_or_zero(grads->init_state, d_final_state, (size_t)sb, s);
    }
    const ScanPlan p = scan_bwd_plan(a.B, a.N, a.D, a.S);
    if (grid_too_large(a.B, a.N, a.D, a.S, p.P)) return GTR_ERR_INVALID_ARG;
    const ScanBwdWs w = scan_bwd_ws(a.B, a.N, a.D, a.S, p);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.dy = static_cast<const uint16_t *>(d_out);
    a.dfin = d_final_state;
    a.du = static_cast<uint16_t *>(grads->u);
    a.ddt = static_cast<uint16_t *>(grads->dt);
    a.dB = static_cast<uint16_t *>(grads->Bm);
    a.dC = static_cast<uint16_t *>(grads->Cm);
    a.dz = static_cast<uint16_t *>(act[4]);
    a.dA = grads->A;
    a.dD = grads->Dskip;
    a.ddtb = grads->dt_bias;
    a.dh0 = grads->init_state;
    a.P = p.P;
    a.L = p.L;
    a.hs = reinterpret_cast<float *>(ws + w.hs);
    a.gs = reinterpret_cast<float *>(ws + w.gs);
    a.sdt = reinterpret_cast<float *>(ws + w.sdt);
    a.pbc = reinterpret_cast<float *>(ws + w.pbc);
    a.pd = reinterpret_cast<float *>(ws + w.pd);
    a.pt = reinterpret_cast<float *>(ws + w.pt);
    const void *ps[] = {a.u, a.dt, a.z, a.dy};
    const long long lds[] = {a.ldu, a.lddt, a.z ? a.ldz : 0, a.lddy};
    const bool wide = rows_on(16, a.D, ps, 4, lds, 4);
    const void *po[] = {a.du, a.ddt, a.dz};
    a.pairs = rows_on(4, a.D, ps, 4, lds, 4) && rows_on(4, a.D, po, 3, lds, 0);
    return ops_cuda_status(ssm->dtype == GTR_F16 ? scan_bwd_dispatch<__half>(a, wide, s)
                                                 : scan_bwd_dispatch<__nv_bfloat16>(a, wide, s));
}
