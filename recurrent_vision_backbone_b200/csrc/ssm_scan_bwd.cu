// ssm_scan_bwd.cu -- the gradients of the selective scan behind the C ABI of include/gtr_ssm.h.
#include "../../include/gtr_ssm.h"
#include "ops_common.cuh"
#include "ssm_scan.cuh"
#include "ssm_scan_bwd.cuh"
#include "ssm_host.cuh"

namespace gtr {

unsigned *ssm_bwd_error_word() { return error_word(); }

static int grad_tile(int S) {
    const int sp = state_pad(S);
    return sp == 8 ? sc::GradLayout<8>::CT : sp == 16 ? sc::GradLayout<16>::CT : sc::GradLayout<32>::CT;
}
struct BwdPlan {
    int P, L;
};
static BwdPlan scan_bwd_plan(int B, long long N, int D, int S) {
    const long long base = (long long)B * ((D + grad_tile(S) - 1) / grad_tile(S));
    // shorter chunks where whole ones would not fill the machine (three blocks an SM) twice
    const int L = base * ((N + sc::kMaxChunkBwd - 1) / sc::kMaxChunkBwd) < 148 * 3 * 2 ? 32 : sc::kMaxChunkBwd;
    BwdPlan r{};
    r.L = L;
    r.P = (int)((N + L - 1) / L);
    return r;
}
struct ScanBwdWs {
    size_t hs, gs, sdt, pbc, pd, pt, bytes;
};
static ScanBwdWs scan_bwd_ws(int B, long long N, int D, int S, const BwdPlan &p) {
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

template <typename T, int SP, sc::Pad PAD>
static auto grad_kernel(bool pairs) {
    return pairs ? sc::ssm_grad_kernel<T, SP, true, PAD> : sc::ssm_grad_kernel<T, SP, false, PAD>;
}
template <typename T, int SP>
static cudaError_t scan_bwd_launch(sc::Args a, bool wide, cudaStream_t s) {
    using Lay = sc::GradLayout<SP>;
    const size_t smem = (size_t)Lay::floats(a.L) * sizeof(float);
    const sc::Pad pad = a.S % 4 != 0 ? sc::kAny : a.S == SP && a.D % Lay::CT == 0 ? sc::kFull : sc::kQuads;
    const auto grad = pad == sc::kFull ? grad_kernel<T, SP, sc::kFull>(a.pairs)
                      : pad == sc::kQuads ? grad_kernel<T, SP, sc::kQuads>(a.pairs) : grad_kernel<T, SP, sc::kAny>(a.pairs);
    // the largest any plan asks for: calls of different shapes may be on their way at once
    cudaError_t e = cudaFuncSetAttribute(grad, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)(Lay::floats(sc::kMaxChunkBwd) * sizeof(float)));
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

}  // namespace gtr

using namespace gtr;

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
    const BwdPlan p = scan_bwd_plan(a.B, a.N, a.D, a.S);
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
