// ops_common.cuh -- what the operators around the token mixer share (causal_conv.cu, ssm_scan.cu,
// ssm_scan_bwd.cu, group_norm.cu):
// 16-bit element access, scan walks, activations, and the host side of argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <nvtx3/nvToolsExt.h>

#include <cstdint>

#include "../../include/gtr_ops.h"
#include "ops_errors.h"

namespace gtr {

// The error word of this source file's kernels.
static __device__ unsigned int g_ops_error_word;
static __device__ __forceinline__ void set_error(unsigned e) { atomicOr(&g_ops_error_word, e); }
static inline unsigned *error_word() {   // its address on the current device; null: a CUDA error
    void *p = nullptr;
    return cudaGetSymbolAddress(&p, g_ops_error_word) == cudaSuccess ? static_cast<unsigned *>(p) : nullptr;
}

namespace ops {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

// ------------------------------------------------------------------ elements
template <typename T>
struct Elem;
template <>
struct Elem<__half> {
    static __device__ __forceinline__ float get(uint16_t r) { return __half2float(__ushort_as_half(r)); }
    static __device__ __forceinline__ uint16_t put(float f) { return __half_as_ushort(__float2half_rn(f)); }
    static __device__ __forceinline__ float2 get2(uint32_t r) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&r));
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    // whether a result left the type's range, tested on the rounded values, two to a word (or one): an
    // exponent of all ones, an infinity or NaN (so every kernel draws the line at the same value, 65520)
    static __device__ __forceinline__ bool bad_raw(uint32_t w) {
        return (w & 0x7c00u) == 0x7c00u || (w & 0x7c000000u) == 0x7c000000u;
    }
    // the larger magnitudes of two pairs (a NaN wins), to be tested once
    static __device__ __forceinline__ uint32_t worst(uint32_t a, uint32_t b) {
        const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2 *>(&a), __habs2(*reinterpret_cast<const __half2 *>(&b)));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
};
template <>
struct Elem<__nv_bfloat16> {
    static __device__ __forceinline__ float get(uint16_t r) { return __uint_as_float((uint32_t)r << 16); }
    static __device__ __forceinline__ uint16_t put(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
    static __device__ __forceinline__ float2 get2(uint32_t r) {
        return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t put2(float a, float b) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    static __device__ __forceinline__ bool bad_raw(uint32_t) { return false; }   // bf16 holds what float32 holds
    static __device__ __forceinline__ uint32_t worst(uint32_t, uint32_t) { return 0; }
};

// V consecutive elements as raw words: V = 8 is one 16-byte access, V = 1 two bytes.
template <int V>
struct Raw {
    uint32_t w[V >= 2 ? V / 2 : 1];
};
// load_raw goes through the read-only path: not for memory that the same kernel writes.  (What the launch
// ahead wrote may be read so: nothing of it is asked for before chain_wait, behind which all of
// that launch's writes are visible, and it does not change any more.)
template <int V>
__device__ __forceinline__ Raw<V> load_raw(const uint16_t *p) {
    Raw<V> r;
    if constexpr (V == 8) {
        const uint4 x = __ldg(reinterpret_cast<const uint4 *>(p));
        r.w[0] = x.x, r.w[1] = x.y, r.w[2] = x.z, r.w[3] = x.w;
    } else {
        static_assert(V == 1, "16 or 2 bytes");
        r.w[0] = __ldg(p);
    }
    return r;
}
template <int V>
__device__ __forceinline__ Raw<V> load_plain(const uint16_t *p) {
    if constexpr (V == 8) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        return {{x.x, x.y, x.z, x.w}};
    } else {
        static_assert(V == 1, "16 or 2 bytes");
        return {{*p}};
    }
}
template <int V>
__device__ __forceinline__ void store_raw(uint16_t *p, const Raw<V> &r) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
    else
        *p = (uint16_t)r.w[0];
}
template <int V>
__device__ __forceinline__ Raw<V> zero_raw() {
    Raw<V> r;
#pragma unroll
    for (auto &x : r.w) x = 0u;   // +0 in both types
    return r;
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Raw<V> &r, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = Elem<T>::get((uint16_t)r.w[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const float2 v = Elem<T>::get2(r.w[i]);
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
}
template <typename T, int V>
__device__ __forceinline__ Raw<V> pack(const float (&f)[V]) {
    Raw<V> r;
    if constexpr (V == 1) {
        r.w[0] = Elem<T>::put(f[0]);
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) r.w[i] = Elem<T>::put2(f[2 * i], f[2 * i + 1]);
    }
    return r;
}

// Elements as float32 in pairs (V = 1: the element and a zero).
template <typename T, int V>
__device__ __forceinline__ void pairs_of(const Raw<V> &r, float2 (&f)[(V + 1) / 2]) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i)
        f[i] = V == 1 ? make_float2(Elem<T>::get((uint16_t)r.w[0]), 0.f) : Elem<T>::get2(r.w[i]);
}

// ------------------------------------------------------------------ asynchronous copies
// 16 bytes to shared memory; `bytes` of them (0 or 16) are read, the rest becomes zeros.
__device__ __forceinline__ void copy16_async(void *dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy4_async(void *dst, const void *src, uint32_t bytes) {   // 4 or 0 of 4 bytes
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
                 "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>   // waits until at most N of this thread's groups are in flight
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint16_t ld16(const uint16_t *p, bool in) { return in ? __ldg(p) : (uint16_t)0; }
// Eight channels of a row to shared memory, `left` of them inside the tensor; zeros where !in.  WIDE:
// an asynchronous 16-byte copy (rows on 16 bytes, whole pieces); else element by element.
template <bool WIDE>
__device__ __forceinline__ void stage_row(uint16_t *dst, const uint16_t *src, bool in, int left) {
    if constexpr (WIDE) {
        copy16_async(dst, src, in && left > 0 ? 16u : 0u);   // 0 bytes: zeros
    } else {
        Raw<8> r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            r.w[i] = (uint32_t)ld16(src + 2 * i, in && 2 * i < left) | (uint32_t)ld16(src + 2 * i + 1, in && 2 * i + 1 < left) << 16;
        store_raw<8>(dst, r);
    }
}

// ------------------------------------------------------------------ functions
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {   // 2^x, about 2 ulp; 0 below 2^-126
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }
__device__ __forceinline__ float horner(float p, float e, float c) { return fmaf(p, e, c); }
__device__ __forceinline__ float2 horner(float2 p, float2 e, float c) { return __ffma2_rn(p, e, splat(c)); }
// log(1 + e) / e for e in [0, 1]: a polynomial of degree 10, interpolating at Chebyshev nodes (relative
// error 8.5e-10; 1.2e-7 evaluated in float32)
template <typename V>
__device__ __forceinline__ V log1p_over(V e, V first) {
    constexpr float c[] = {-0.013187826611101627f, 0.04100657254457474f,  -0.08188040554523468f, 0.12377995997667313f, -0.16087622940540314f,
                           0.19885820150375366f,   -0.24986496567726135f, 0.33332496881484985f,  -0.4999997913837433f, 1.0f};
    V p = first;   // the leading coefficient
#pragma unroll
    for (int i = 0; i < 10; ++i) p = horner(p, e, c[i]);
    return p;
}
constexpr float kLog1pLead = 0.001986696617677808f;
// max(x, 0) + log(1 + e^-|x|) of two values at once (packed arithmetic: half the instructions);
// relative error about |x| 2^-24 from the exponent's rounding, and a NaN stays one (fmaxf alone
// would drop it)
__device__ __forceinline__ float2 softplus_2(float2 x, float2 &e) {   // e: e^-|x|
    e = make_float2(ex2(fabsf(x.x) * -kLog2e), ex2(fabsf(x.y) * -kLog2e));
    return __ffma2_rn(log1p_over(e, splat(kLog1pLead)), e, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
}
__device__ __forceinline__ float rcp_f(float x) {   // 1 / x, about 1 ulp; 0 for infinities
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid_f(float x) { return rcp_f(1.f + ex2(x * -kLog2e)); }
// sigmoid(x), softplus's derivative, from e = e^-|x|: relative accuracy for either sign
__device__ __forceinline__ float sigmoid_of(float x, float e) {
    const float r = rcp_f(1.f + e);
    return x < 0.f ? e * r : r;
}
__device__ __forceinline__ float softplus_f(float x) {
    const float e = ex2(fabsf(x) * -kLog2e);
    return fmaxf(x, 0.f) + log1p_over(e, kLog1pLead) * e;
}

// ------------------------------------------------------------------ sums over lanes
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

// n / d with the remainder in r, n >= 0, d > 0: a 32-bit division wherever that will do (a 64-bit one
// takes several times as long, and what follows waits for it).
__device__ __forceinline__ long long div_rem(long long n, long long d, long long &r) {
    if (((n | d) >> 32) == 0) {
        const uint32_t q = (uint32_t)n / (uint32_t)d;
        r = (uint32_t)n - q * (uint32_t)d;
        return q;
    }
    const long long q = n / d;
    r = n - q * d;
    return q;
}

// ------------------------------------------------------------------ launches in a chain
// A kernel launched with launch_after may start while the one ahead of it in the stream drains;
// it waits here, before its first access to global memory, until that one has finished.
__device__ __forceinline__ void chain_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// ------------------------------------------------------------------ scan order
// Token of scan position p, and its successors without divisions: inside a row (or column)
// the token moves by `step`, at its end by `jump` more.
struct Walk {
    int n, i, inner, step, jump;
    __device__ __forceinline__ Walk(int p, int H, int W, int dir) {
        if (dir == GTR_L2R) {
            n = p, i = 0, inner = 0x7fffffff, step = 1, jump = 0;
        } else if (dir == GTR_R2L) {
            const int y = p / W, r = p - y * W;
            n = y * W + (W - 1 - r), i = r, inner = W, step = -1, jump = 2 * W;
        } else {
            const int x = p / H, r = p - x * H;
            i = r, inner = H;
            if (dir == GTR_T2B)
                n = r * W + x, step = W, jump = 1 - H * W;
            else
                n = (H - 1 - r) * W + x, step = -W, jump = H * W + 1;
        }
    }
    // (sums modulo 2^32: a step of several rows may pass 31 bits before the jumps bring it back)
    __device__ __forceinline__ void add(uint32_t d) { n = (int)((uint32_t)n + d); }
    __device__ __forceinline__ void next() {
        add((uint32_t)step);
        if (++i == inner) {
            i = 0;
            add((uint32_t)jump);
        }
    }
    __device__ __forceinline__ void advance(int k) {
        add((uint32_t)k * (uint32_t)step);
        i += k;
        while (i >= inner) {
            i -= inner;
            add((uint32_t)jump);
        }
    }
};
__device__ __forceinline__ int token_of(int p, int H, int W, int dir) {
    return dir == GTR_L2R ? p : Walk(p, H, W, dir).n;
}

// ------------------------------------------------------------------ host checks
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned_to(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Launches a kernel of one Args argument (and perhaps an int) that begins with chain_wait().
template <typename K, typename... A>
inline cudaError_t launch_after(K kernel, unsigned grid, dim3 block, size_t smem, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

struct Span {
    const void *p;
    long long bytes;
};
inline bool overlap(const Span &a, const Span &b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}
// bytes from the first to behind the last element of `rows` rows of `cols` 16-bit elements, `ld` apart
inline long long row_bytes(long long rows, long long ld, long long cols) {
    return rows <= 0 ? 0 : ((rows - 1) * ld + cols) * 2;
}
// (channels are counted in 32 bits, up to a block's width beyond the last)
constexpr long long kMaxTokens = (1LL << 30) - 1, kMaxChannels = (1LL << 30) - 1, kMaxElements = 1LL << 40, kMaxGrid = 0x7fffffffLL;

inline bool bad_common(int B, int H, int W, int D, int dir, int dtype) {
    if (B <= 0 || D <= 0 || D > kMaxChannels || H < 0 || W < 0 || dir < 0 || dir > 3) return true;
    if (dtype != GTR_F16 && dtype != GTR_BF16) return true;
    const long long N = (long long)H * W;
    return N > kMaxTokens || (long long)B * N > kMaxElements / D;
}
// A [B, N, cols] activation with rows ld apart: present, aligned, rows that do not overlap.
inline bool bad_rows(const void *p, long long ld, int cols, long long rows) {
    if (rows == 0) return ld < 0;
    return p == nullptr || !aligned_to(p, 2) || (ld != 0 && ld < cols) || (ld > 0 && rows > (kMaxElements << 4) / ld);
}
inline bool bad_f32(const void *p, bool required) { return p == nullptr ? required : !aligned_to(p, 16); }

inline bool any_overlap(const Span *outs, int no, const Span *ins, int ni) {
    for (int i = 0; i < no; ++i) {
        for (int k = 0; k < ni; ++k)
            if (overlap(outs[i], ins[k])) return true;
        for (int k = i + 1; k < no; ++k)
            if (overlap(outs[i], outs[k])) return true;
    }
    return false;
}

// Whether every row of every tensor starts on a `bytes` boundary and holds whole pieces of them.
inline bool rows_on(int bytes, int D, const void *const *ps, int np, const long long *lds, int nl) {
    if (D * 2LL % bytes) return false;
    for (int i = 0; i < np; ++i)
        if (ps[i] && !aligned_to(ps[i], bytes)) return false;
    for (int i = 0; i < nl; ++i)
        if (lds[i] * 2 % bytes) return false;
    return true;
}

// dst = src, or zeros without src.
inline gtr_status_t copy_or_zero(void *dst, const void *src, size_t bytes, cudaStream_t s) {
    if (dst == nullptr || dst == src || bytes == 0) return GTR_OK;
    return ops_cuda_status(src != nullptr ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, s)
                                          : cudaMemsetAsync(dst, 0, bytes, s));
}

}  // namespace ops
}  // namespace gtr
