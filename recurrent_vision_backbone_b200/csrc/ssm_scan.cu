// ssm_scan.cu -- the selective scan, forward and for single tokens, behind the C ABI of
// include/gtr_ssm.h.
#include "../../include/gtr_ssm.h"
#include "ops_common.cuh"
#include "ssm_scan.cuh"
#include "ssm_host.cuh"

namespace gtr {

unsigned *ssm_error_word() { return error_word(); }

constexpr int kSmAim = 148 * 4;   // blocks of four warps that keep the schedulers busy (one wave at up to 16 states)

struct ScanPlan {
    int P, L;
    int SL;   // lanes that share a channel in the walk that writes the outputs
};
// The walks of a forward scan.  With 96 blocks of 128 channels or more, one walk over whole sequences, with
// two lanes a channel until the channels alone are three warps a scheduler, then one.  2304 tokens, 16 states,
// us by blocks: one walk 201 and chunks 204 at 64, 285 and 297 at 90 and at 96, 285 and 355 at 112.  Two lanes
// and one: 285 and 348 at 96 to 144, 391 and 518 at 160 to 192, 546 and 518 at 224 to 288, 651 and 727 at
// 320, 766 and 727 at 384, 894 and 924 at 448 (steps where a wave of blocks is full; within 5 % of each
// other from 224 on but for 320).
// Fewer blocks: as many chunks as make one wave of four blocks an SM, at least 32 tokens each.  16384 tokens of
// 1024 channels (8 blocks), us with two, three, four, six blocks an SM: 16 states 230, 209, 182, 185; 8 states
// 156, 142, 119, 123.  With 17 to 32 states the registers leave two blocks an SM, and four are two waves: 325,
// 345, 339, 359 at 32 states; at 2048 channels 628, 648, 627, 646.
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

}  // namespace gtr

using namespace gtr;

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
