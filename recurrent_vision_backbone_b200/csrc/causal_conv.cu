// causal_conv.cu -- the short causal convolution behind the C ABI of include/gtr_ssm.h.
#include "../../include/gtr_ssm.h"
#include "ops_common.cuh"
#include "causal_conv.cuh"

namespace gtr {

unsigned *conv_error_word() { return error_word(); }

using namespace ops;

struct ConvPlan {
    long long tiles;    // chunks of a sequence
    long long parts;    // chunks
    int tile;           // positions of a chunk
};
// The walks: chunks enough for one wave of `blocks` blocks an SM (backward every block writes a partial
// row of the parameters' sums), of 32 positions at least (each begins with K - 1 more).
static ConvPlan conv_plan(int B, long long N, int D, int blocks) {
    ConvPlan p{};
    const long long blocks_c = (D + 127) / 128;
    long long tiles = 148LL * blocks / (blocks_c * B);
    if (tiles < 1) tiles = 1;
    long long tile = (N + tiles - 1) / tiles;
    if (tile < 32) tile = 32;
    p.tile = (int)tile;
    p.tiles = (N + tile - 1) / tile;
    p.parts = (long long)B * p.tiles;
    return p;
}
static ConvPlan conv_bwd_plan(int B, long long N, int D) { return conv_plan(B, N, D, 8); }

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

template <typename T, int V, int K>
static cudaError_t conv_direct(cv::Args a, cudaStream_t s) {
    a.groups = (a.D + V - 1) / V;
    a.tiles = (a.N + cv::kDirect - 1) / cv::kDirect;
    const long long blocks = ((long long)a.B * a.tiles * a.groups + cv::kThreads - 1) / cv::kThreads;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    return launch_after(cv::causal_conv_fwd_kernel<T, V, K>, (unsigned)blocks, dim3(cv::kThreads), 0, s, a);
}
template <typename T, int K>
static cudaError_t conv_walk(cv::Args a, const ConvPlan &p, bool wide, cudaStream_t s) {
    a.groups = (a.D + 2 * cv::kWalkThreads - 1) / (2 * cv::kWalkThreads);
    a.tile = p.tile;
    a.tiles = (int)p.tiles;
    if (p.parts * a.groups > kMaxGrid) return cudaErrorInvalidConfiguration;
    return launch_after(wide ? cv::causal_conv_walk_kernel<T, K, true> : cv::causal_conv_walk_kernel<T, K, false>,
                        (unsigned)(p.parts * a.groups), dim3(cv::kWalkThreads), 0, s, a);
}
template <typename T, int K>
static cudaError_t conv_fwd_launch(const cv::Args &a, bool wide, cudaStream_t s) {
    // the walk once there are chunks of 32 positions for eight blocks an SM.  us direct / walk, K = 4, inputs in
    // turn: 4736 x 1024, at the switch, 11.1 / 7.3; 2 x 2304 x 2048 19.2 / 17.0; 8 x 2304 x 2048 67 / 56; below the
    // switch 4096 x 1024 10.9 / 7.3, and 1600 x 1024 6.5 / 5.7, where the host's time for a call is near
    if ((long long)a.B * ((a.N + 31) / 32) * ((a.D + 127) / 128) >= 148 * 8)
        return conv_walk<T, K>(a, conv_plan(a.B, a.N, a.D, 10), wide, s);
    return wide ? conv_direct<T, 8, K>(a, s) : conv_direct<T, 1, K>(a, s);
}
template <typename T>
static cudaError_t conv_fwd_k(const cv::Args &a, int K, bool wide, cudaStream_t s) {
    switch (K) {
    case 2: return conv_fwd_launch<T, 2>(a, wide, s);
    case 3: return conv_fwd_launch<T, 3>(a, wide, s);
    default: return conv_fwd_launch<T, 4>(a, wide, s);
    }
}

template <typename T, int K>
static cudaError_t conv_bwd_launch(cv::Args a, const ConvPlan &p, bool wide, float *gw, float *gb, cudaStream_t s) {
    a.groups = (a.D + 2 * cv::kWalkThreads - 1) / (2 * cv::kWalkThreads);
    const long long blocks = p.parts * a.groups;
    if (blocks > kMaxGrid) return cudaErrorInvalidConfiguration;
    const cudaError_t e = launch_after(wide ? cv::causal_conv_bwd_kernel<T, K, true> : cv::causal_conv_bwd_kernel<T, K, false>,
                                       (unsigned)blocks, dim3(cv::kWalkThreads), 0, s, a);
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
    return ops_cuda_status(conv->dtype == GTR_F16 ? conv_fwd_k<__half>(a, conv->K, wide, s)
                                                  : conv_fwd_k<__nv_bfloat16>(a, conv->K, wide, s));
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
