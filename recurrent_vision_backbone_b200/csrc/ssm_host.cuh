// ssm_host.cuh -- what the forward and the backward entry points of the selective scan share on the
// host: argument checks, kernel arguments, the launches of walks and folds (included by ssm_scan.cu
// and ssm_scan_bwd.cu after the kernels).
#pragma once

namespace gtr {

using namespace ops;

inline int state_pad(int S) { return S <= 8 ? 8 : S <= 16 ? 16 : 32; }

inline gtr_status_t check_ssm(const gtr_ssm_t *m) {
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

inline sc::Args ssm_args(const gtr_ssm_t *m) {
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
inline int ssm_inputs(const gtr_ssm_t *m, const sc::Args &a, Span *s) {
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

// How the states that a call lacks of SP are left out.
template <int SP>
inline sc::Pad state_padding(int S) { return S == SP ? sc::kFull : S % 4 == 0 ? sc::kQuads : sc::kAny; }
template <typename T, int SP, int MODE, int SL, sc::Pad PAD>
static auto walk_kernel(bool wide) {
    return wide ? sc::ssm_walk_kernel<T, SP, MODE, true, SL, PAD> : sc::ssm_walk_kernel<T, SP, MODE, false, SL, PAD>;
}
template <typename T, int SP, int MODE, int SL>
static cudaError_t walk_launch(const sc::Args &a, bool wide, cudaStream_t s) {
    const unsigned grid = (unsigned)((long long)a.tiles * a.B * (MODE == sc::kLocal ? a.P - 1 : a.P));
    auto kernel = walk_kernel<T, SP, MODE, SL, sc::kFull>(wide);
    if constexpr (MODE == sc::kOut) {
        const sc::Pad pad = state_padding<SP>(a.S);
        if (pad != sc::kFull) kernel = pad == sc::kQuads ? walk_kernel<T, SP, MODE, SL, sc::kQuads>(wide) : walk_kernel<T, SP, MODE, SL, sc::kAny>(wide);
    }
    // A walk that opens a call and covers many SMs starts plainly: blocks that wait on SMs where the
    // call ahead happens to have left room end up unevenly spread (381 us for 285 at 8 x 2304 tokens of
    // 2048 channels; no difference at 6 or 10 x 2304)
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
// Whether the launches of a scan fit a grid (blocks along x only).
inline bool grid_too_large(int B, long long N, int D, int S, long long P) {
    const long long sp = state_pad(S), tiles = (D + 31) / 32;
    return (long long)B * P > kMaxGrid || (long long)B * P * tiles > kMaxGrid || (long long)B * D > kMaxGrid * (sc::kFoldThreads / 2) / sp ||
           (long long)B * N > kMaxGrid * 8 / sp - (D * (sp + 2) + 31) / 32;
}

}  // namespace gtr
