// RMS norm of the residual stream in front of the layer, with the residual's addition and the
// rows in 8 bits beside the 16-bit ones, and its backward pass.
//
// Forward, per row:  s = rnd(x + residual), rstd = 1 / sqrt(mean(s^2) + eps), v = s * rstd * w,
//   y = rnd(v); e4m3: scale = max|v| / 448, code = e4m3(v / scale); block-scaled: per run of 32
//   the exponent of mx_exponent() and code = e4m3(v * 2^-e).
// s is rounded before it is normalised because the rounded s is what the next layers and the
// backward pass read.  y and the codes are each rounded once, from the fp32 v.
// Backward, per row: xhat = s * rstd, g = dy * w, c = mean(g * xhat),
//   dx = rstd * (g - xhat * c) + dsum;  over the rows: dweight = sum_t dy * xhat (fp32).
// Sums, statistics and gradients of the weight are fp32.  Both passes are bound by HBM: the row
// stays in registers between the reduction and the output, so every element is read once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int NORM_NATIVE = 0, NORM_E4M3 = 1, NORM_MX = 2;

// One thread's piece of a row: VEC elements of T in one load.
template <typename T, int VEC>
struct Pack;
template <>
struct Pack<__nv_bfloat16, 8> {
    uint4 r;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 4 ? (i < 2 ? r.x : r.y) : (i < 6 ? r.z : r.w);
        return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
    }
    __device__ __forceinline__ void set(const float* f) {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            o[i] = *reinterpret_cast<const uint32_t*>(&b);
        }
        r = make_uint4(o[0], o[1], o[2], o[3]);
    }
    __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
};
template <>
struct Pack<float, 4> {
    float4 r;
    __device__ __forceinline__ float get(int i) const { return i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w; }
    __device__ __forceinline__ void set(const float* f) { r = make_float4(f[0], f[1], f[2], f[3]); }
    __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Pack<float, 1> {
    float r;
    __device__ __forceinline__ float get(int) const { return r; }
    __device__ __forceinline__ void set(const float* f) { r = f[0]; }
    __device__ __forceinline__ void zero() { r = 0.f; }
};

// Sum or maximum of a over the row's threads: a warp (WARP) or the block.
template <bool WARP, bool MAX>
__device__ __forceinline__ void reduce_row(float& a, float* sm) {
    auto all = [&] {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float b = __shfl_xor_sync(0xffffffffu, a, o);
            a = MAX ? fmaxf(a, b) : a + b;
        }
    };
    all();
    if (WARP) return;
    const int lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    if (lane == 0) sm[threadIdx.x >> 5] = a;
    __syncthreads();
    a = lane < nw ? sm[lane] : 0.f;                            // 0: a maximum is one of magnitudes
    all();
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// f / sc as IEEE division rounds it, by Markstein's method: the product with the rounded reciprocal, corrected once by the
// exact remainder.  (Division itself takes its slow path's registers along: 232 us instead of 162 for 16384 rows of 7168.)
struct Divisor {
    float up, sc, inv;                                         // up: keeps the remainders of tiny rows above underflow
    __device__ __forceinline__ explicit Divisor(float s) {
        up = s < 0x1p-60f ? 0x1p64f : 1.f;
        inv = __frcp_rn(s * up);
        sc = s < INFINITY ? s * up : 0.f;                      // over infinity: 0, or NaN, without a remainder
    }
    __device__ __forceinline__ float divide(float f) const {    // of f * up
        const float q = f * inv;
        return fmaf(-fmaf(q, sc, -f), inv, q);                 // -0 stays -0
    }
};

// One row per block, or per warp (WARP) where a row is at most 32 * VPT vectors.  sum may be x or res
// itself: a thread reads its elements before it writes them.
template <typename T, int VEC, int VPT, bool WARP, int FMT, bool RES>
__global__ void __launch_bounds__(VPT <= 2 || VEC == 1 ? 1024 : 512)
    rmsnorm_kernel(const T* x, const T* res, const T* __restrict__ w, float eps, long long rows, int d, T* sum, T* y,
                   uint8_t* __restrict__ codes,
                   void* __restrict__ scales, float* __restrict__ rstd_out) {
    using P = Pack<T, VEC>;
    __shared__ float sm[FMT == NORM_E4M3 ? 64 : 32];
    const int nv = d / VEC;
    const int width = WARP ? 32 : blockDim.x;
    const int me = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const long long row = WARP ? (long long)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : (long long)blockIdx.x;
    if (row >= rows) return;                                   // WARP only: a whole warp leaves
    const P* xr = reinterpret_cast<const P*>(x + (size_t)row * d);
    const P* wr = reinterpret_cast<const P*>(w);
    P s[VPT], wv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = me + j * width;
        if (i < nv) s[j] = xr[i];
        else s[j].zero();
    }
    if (RES) {
        const P* rr = reinterpret_cast<const P*>(res + (size_t)row * d);
        P r[VPT];
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = me + j * width;
            if (i < nv) r[j] = rr[i];
            else r[j].zero();
        }
        P* sr = reinterpret_cast<P*>(sum + (size_t)row * d);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) f[e] = s[j].get(e) + r[j].get(e);
            s[j].set(f);
            const int i = me + j * width;
            if (i < nv) sr[i] = s[j];
        }
    }
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = me + j * width;
        if (i < nv) wv[j] = wr[i];
        else wv[j].zero();
    }
    float sq = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float f = s[j].get(e);
            sq = fmaf(f, f, sq);
        }
    reduce_row<WARP, false>(sq, sm);
    const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sq, (float)d), eps)));
    if (rstd_out && me == 0) rstd_out[row] = rstd;
    float sc = 1.f;
    if (FMT == NORM_E4M3) {
        // of the values themselves: s * w can leave fp32's range where s * rstd * w does not
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) mx = fmaxf(mx, fabsf(s[j].get(e) * rstd * wv[j].get(e)));
        reduce_row<WARP, true>(mx, sm + 32);
        sc = mx > 0.f ? fmaxf(__fdiv_rn(mx, 448.f), 1.17549435e-38f) : 1.f;      // at least 2^-126
        if (me == 0) static_cast<float*>(scales)[row] = sc;
    }
    const Divisor by(sc);
    P* yr = reinterpret_cast<P*>(y + (size_t)row * d);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = me + j * width;
        float f[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = s[j].get(e) * rstd * wv[j].get(e);
        if (i < nv) {
            P o;
            o.set(f);
            yr[i] = o;
        }
        if (FMT != NORM_NATIVE) {
            if (FMT == NORM_E4M3) {                            // the same value has the same code as in moe_quantize_rows_e4m3
                if (by.up != 1.f)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[e] *= by.up;
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] = by.divide(f[e]);
            } else {                                           // lanes 4q .. 4q + 3 hold a run of 32
                float m = 0.f;
#pragma unroll
                for (int e = 0; e < VEC; ++e) m = fmaxf(m, fabsf(f[e]));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int ex = mx_exponent(m);
                const float mul = __uint_as_float((uint32_t)(127 - ex) << 23);
                if ((me & 3) == 0 && i < nv)
                    static_cast<uint8_t*>(scales)[(size_t)row * ((d + 31) / 32) + (i >> 2)] = (uint8_t)(ex + 127);
#pragma unroll
                for (int e = 0; e < VEC; ++e) f[e] *= mul;
            }
            if (VEC == 8 && i < nv) {
                const uint2 c = make_uint2(codes2(f[0], f[1 % VEC]) | codes2(f[2 % VEC], f[3 % VEC]) << 16,
                                           codes2(f[4 % VEC], f[5 % VEC]) | codes2(f[6 % VEC], f[7 % VEC]) << 16);
                reinterpret_cast<uint2*>(codes + (size_t)row * d)[i] = c;
            }
        }
    }
}

// Backward.  Blocks (or, with WARP, the 8 warps of a block) walk the rows; each thread keeps its
// columns' share of dweight in registers, and a block writes one row of partial sums.
template <typename T, int VEC, int VPT, bool WARP, bool DSUM>
__global__ void __launch_bounds__(WARP ? 256 : VEC == 1 || VPT <= 2 ? 1024 : 512)
    rmsnorm_bwd_kernel(const T* dy, const T* __restrict__ s, const T* __restrict__ w,
                       const float* __restrict__ rstd, const T* dsum, long long rows, int d, T* dx,
                       float* __restrict__ partial) {
    using P = Pack<T, VEC>;
    extern __shared__ float smw[];                             // WARP: [warps][d] partial sums
    __shared__ float sm[2][32];
    const int nv = d / VEC;
    const int width = WARP ? 32 : blockDim.x;
    const int me = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int nw = blockDim.x >> 5, warp = threadIdx.x >> 5;
    const P* wr = reinterpret_cast<const P*>(w);
    float acc[VPT][VEC];
    P wv[VPT];
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
        const int i = me + j * width;
        if (i < nv) wv[j] = wr[i];
        else wv[j].zero();
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    }
    const long long step = WARP ? (long long)gridDim.x * nw : (long long)gridDim.x;
    const long long row0 = WARP ? (long long)blockIdx.x * nw + warp : (long long)blockIdx.x;
    // One vector a thread: a row is loaded while the one before is reduced and written, as otherwise the memory
    // idles during the reductions (16384 rows of 7168: 191 us with two vectors a thread and no loads ahead, 164 us so).
    constexpr bool AHEAD = VEC > 1 && VPT == 1;
    P na, nb, nc;
    float nr = 0.f;
    auto ahead = [&](long long row) {
        if (row >= rows || me >= nv) return;
        na = reinterpret_cast<const P*>(s + (size_t)row * d)[me];
        nb = reinterpret_cast<const P*>(dy + (size_t)row * d)[me];
        if (DSUM) nc = reinterpret_cast<const P*>(dsum + (size_t)row * d)[me];
        nr = rstd[row];
    };
    if (AHEAD) {
        na.zero(); nb.zero(); nc.zero();
        ahead(row0);
    }
    int turn = 0;
    for (long long row = row0; row < rows; row += step, turn ^= 1) {
        const P* sr = reinterpret_cast<const P*>(s + (size_t)row * d);
        const P* gr = reinterpret_cast<const P*>(dy + (size_t)row * d);
        P a[VPT], b[VPT], c[VPT];
        float r;
        if (AHEAD) {
            a[0] = na; b[0] = nb; c[0] = nc; r = nr;
            ahead(row + step);
        } else {
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int i = me + j * width;
                if (i < nv) { a[j] = sr[i]; b[j] = gr[i]; }
                else { a[j].zero(); b[j].zero(); }
            }
            if (DSUM) {
                const P* qr = reinterpret_cast<const P*>(dsum + (size_t)row * d);
#pragma unroll
                for (int j = 0; j < VPT; ++j) {
                    const int i = me + j * width;
                    if (i < nv) c[j] = qr[i];
                    else c[j].zero();
                }
            }
            r = rstd[row];
        }
        float dot = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xh = a[j].get(e) * r, g = b[j].get(e);
                dot = fmaf(g * wv[j].get(e), xh, dot);
                acc[j][e] = fmaf(g, xh, acc[j][e]);
            }
        reduce_row<WARP, false>(dot, sm[turn]);
        const float m = __fdiv_rn(dot, (float)d);
        P* dr = reinterpret_cast<P*>(dx + (size_t)row * d);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = me + j * width;
            float f[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                f[e] = r * (b[j].get(e) * wv[j].get(e) - a[j].get(e) * r * m);
                if (DSUM) f[e] += c[j].get(e);
            }
            if (i < nv) {
                P o;
                o.set(f);
                dr[i] = o;
            }
        }
    }
    if (WARP) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = me + j * 32;
            if (i < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) smw[warp * d + i * VEC + e] = acc[j][e];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < d; i += blockDim.x) {
            float t = 0.f;
            for (int q = 0; q < nw; ++q) t += smw[q * d + i];
            partial[(size_t)blockIdx.x * d + i] = t;
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int i = me + j * width;
            if (i < nv)
#pragma unroll
                for (int e = 0; e < VEC; ++e) partial[(size_t)blockIdx.x * d + (size_t)i * VEC + e] = acc[j][e];
        }
    }
}

// dweight[i] = sum over the partial rows, in a fixed order: 32 columns per block, 32 warps
// striding over the rows, then the warps' sums in order.
__global__ void __launch_bounds__(1024) colsum_partial_kernel(const float* __restrict__ partial, int n, int d,
                                                              float* __restrict__ out) {
    __shared__ float sm[32][33];
    const int c = blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    if (c < d)
        for (int r = threadIdx.y; r < n; r += 32) t += partial[(size_t)r * d + c];
    sm[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    t = sm[threadIdx.x][threadIdx.y];                          // warp y sums column y
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (threadIdx.x == 0 && blockIdx.x * 32 + threadIdx.y < d) out[blockIdx.x * 32 + threadIdx.y] = t;
}

struct NormArgs {
    const void *x, *res, *w;
    float eps;
    long long rows;
    int d;
    void *sum, *y;
    uint8_t* codes;
    void* scales;
    float* rstd;
};

template <typename T, int VEC, int VPT, bool WARP, int FMT, bool RES>
cudaError_t norm_launch(const NormArgs& a, int threads, cudaStream_t st) {
    const long long blocks = WARP ? (a.rows + threads / 32 - 1) / (threads / 32) : a.rows;
    rmsnorm_kernel<T, VEC, VPT, WARP, FMT, RES><<<(unsigned)blocks, threads, 0, st>>>(
        (const T*)a.x, (const T*)a.res, (const T*)a.w, a.eps, a.rows, a.d, (T*)a.sum, (T*)a.y, a.codes, a.scales, a.rstd);
    return cudaGetLastError();
}

template <typename T, int VEC, int VPT, bool WARP, int FMT>
cudaError_t norm_res(const NormArgs& a, int threads, cudaStream_t st) {
    return a.res ? norm_launch<T, VEC, VPT, WARP, FMT, true>(a, threads, st)
                 : norm_launch<T, VEC, VPT, WARP, FMT, false>(a, threads, st);
}

int round32(int v) { return (v + 31) / 32 * 32; }

template <typename T, int VEC, int FMT>
cudaError_t norm_shape(const NormArgs& a, cudaStream_t st) {
    const int nv = a.d / VEC;
    const bool few = a.rows <= 2 * num_sms();                  // not enough rows to fill the GPU: spread each
    if (!few && nv <= 32) return norm_res<T, VEC, 1, true, FMT>(a, 256, st);
    if (!few && nv <= 128) return norm_res<T, VEC, 4, true, FMT>(a, 256, st);
    if (few && nv <= 1024) return norm_res<T, VEC, 1, false, FMT>(a, round32(nv), st);
    if (VEC == 8 || nv <= 2048) return norm_res<T, VEC, 4, false, FMT>(a, round32((nv + 3) / 4), st);
    if constexpr (VEC < 8) {                                   // fp32: 16384 columns are 4096 vectors, or 16384 single ones
        if (VEC > 1 || nv <= 8192) return norm_res<T, VEC, 8, false, FMT>(a, round32((nv + 7) / 8), st);
        return norm_res<T, VEC, VEC == 1 ? 16 : 8, false, FMT>(a, round32((nv + 15) / 16), st);
    }
    return cudaErrorInvalidValue;
}

struct BwdArgs {
    const void *dy, *s, *w, *dsum;
    const float* rstd;
    long long rows;
    int d;
    void* dx;
    float* partial;
};

template <typename T, int VEC, int VPT, bool WARP>
cudaError_t bwd_launch(const BwdArgs& a, int threads, int blocks, cudaStream_t st) {
    const size_t smem = WARP ? (size_t)(threads / 32) * a.d * 4 : 0;
    auto k1 = rmsnorm_bwd_kernel<T, VEC, VPT, WARP, true>;
    auto k0 = rmsnorm_bwd_kernel<T, VEC, VPT, WARP, false>;
    (a.dsum ? k1 : k0)<<<blocks, threads, smem, st>>>((const T*)a.dy, (const T*)a.s, (const T*)a.w, a.rstd, (const T*)a.dsum,
                                                      a.rows, a.d, (T*)a.dx, a.partial);
    return cudaGetLastError();
}

template <typename T, int VEC>
cudaError_t bwd_shape(const BwdArgs& a, int* blocks, cudaStream_t st) {
    const int nv = a.d / VEC;
    const int cap = norm_bwd_partials(a.rows);
    *blocks = (int)(a.rows < cap ? a.rows : cap);
    if (nv <= 128) {                               // 8 warps of a block, a row each
        *blocks = (int)((a.rows + 7) / 8 < cap ? (a.rows + 7) / 8 : cap);
        return nv <= 32 ? bwd_launch<T, VEC, 1, true>(a, 256, *blocks, st)
                        : bwd_launch<T, VEC, 4, true>(a, 256, *blocks, st);
    }
    // As many blocks as fit with 64 registers a thread, but at most NORM_BWD_BLOCKS, which binds below 512 threads.  Twice as
    // many partial rows would suit many narrow rows (16384 of 1280: 47 us instead of 59, of 2048: 57 instead of 70) and
    // cost few rows, and the widest (700 of 2048: 18 instead of 14; 700 of 16384: 80 instead of 55).
    if (VEC > 1 && nv <= 1024) {
        const int threads = round32(nv), fit = num_sms() * (1024 / threads);
        if (*blocks > fit) *blocks = fit;
        return bwd_launch<T, VEC, 1, false>(a, threads, *blocks, st);
    }
    if (VEC == 8 || nv <= 2048) return bwd_launch<T, VEC, 2, false>(a, round32((nv + 1) / 2), *blocks, st);
    if constexpr (VEC < 8) {                                   // fp32: 16384 columns are 4096 vectors, or 16384 single ones
        if (VEC > 1 || nv <= 8192) return bwd_launch<T, VEC, 8, false>(a, round32((nv + 7) / 8), *blocks, st);
        return bwd_launch<T, VEC, VEC == 1 ? 16 : 8, false>(a, round32((nv + 15) / 16), *blocks, st);
    }
    return cudaErrorInvalidValue;
}

}  // namespace

int norm_bwd_partials(long long rows) { return (int)(rows < NORM_BWD_BLOCKS ? rows : NORM_BWD_BLOCKS); }

cudaError_t launch_rmsnorm(bool bf16, int fmt, const void* x, const void* res, const void* w, float eps, long long rows,
                           int d, void* sum, void* y, uint8_t* codes, void* scales, float* rstd, cudaStream_t st) {
    const NormArgs a = {x, res, w, eps, rows, d, sum, y, codes, scales, rstd};
    if (bf16) {
        if (fmt == NORM_E4M3) return norm_shape<__nv_bfloat16, 8, NORM_E4M3>(a, st);
        if (fmt == NORM_MX) return norm_shape<__nv_bfloat16, 8, NORM_MX>(a, st);
        return norm_shape<__nv_bfloat16, 8, NORM_NATIVE>(a, st);
    }
    const uintptr_t al = (uintptr_t)x | (uintptr_t)res | (uintptr_t)w | (uintptr_t)sum | (uintptr_t)y;
    if (d % 4 == 0 && al % 16 == 0) return norm_shape<float, 4, NORM_NATIVE>(a, st);
    return norm_shape<float, 1, NORM_NATIVE>(a, st);
}

cudaError_t launch_rmsnorm_bwd(bool bf16, const void* dy, const void* s, const void* w, const float* rstd, const void* dsum,
                               long long rows, int d, void* dx, float* dweight, float* partial, cudaStream_t st) {
    const BwdArgs a = {dy, s, w, dsum, rstd, rows, d, dx, partial};
    int blocks = 0;
    cudaError_t e;
    const uintptr_t al = (uintptr_t)dy | (uintptr_t)s | (uintptr_t)w | (uintptr_t)dsum | (uintptr_t)dx;
    if (bf16) e = bwd_shape<__nv_bfloat16, 8>(a, &blocks, st);
    else if (d % 4 == 0 && al % 16 == 0) e = bwd_shape<float, 4>(a, &blocks, st);
    else e = bwd_shape<float, 1>(a, &blocks, st);
    if (e != cudaSuccess) return e;
    colsum_partial_kernel<<<(d + 31) / 32, dim3(32, 32), 0, st>>>(partial, blocks, d, dweight);
    return cudaGetLastError();
}

}  // namespace moe
