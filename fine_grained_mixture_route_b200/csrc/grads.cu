// The global L2 norm over the gradients of a training step, and clipping by it:
//   norm = sqrt(sum over all tensors of g^2),  coef = min(1, max_norm / (norm + 1e-6)),
//   out = rnd(g * coef).
// Bound by HBM: the norm reads every gradient once; clipping has to know the norm before its first
// output, so it reads the gradients again, last ones first, which the L2 still holds.
//
// The tensors form one list of units of UNIT_BYTES; block b of the grid takes the units b, b + G, ...,
// keeps its sum in 64 bits and writes one partial; the last block of the last launch adds the partials
// in index order.  So the sums do not depend on timing.  Squares are taken in fp32 where the sum of a
// thread's 16 or 8 of them lies within 2^-80 .. 2^120, and in 64 bits otherwise: gradients of any
// size, down to the smallest subnormals, neither overflow nor vanish.
#include "common.cuh"
#include "launch.h"

namespace moe {
namespace {

constexpr int THREADS = 256;
constexpr int UNROLL = 4;                                       // 16-byte vectors of a thread in flight
constexpr int UNIT_VECS = THREADS * UNROLL;
constexpr int LIST = 160;                                       // tensors per launch (kernel parameters)

struct GradList {
    const void* src[LIST];
    void* dst[LIST];
    long long numel[LIST];
    long long first[LIST + 1];                                  // first unit of each tensor
    uint8_t bf16[LIST];
    int n;
};

struct GradState {                                              // head of the workspace, after the error word
    unsigned int done;
    float coef;
};

__device__ __forceinline__ int find(const GradList& L, long long u) {
    int lo = 0, hi = L.n;                                       // first[lo] <= u < first[hi]
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (L.first[m] <= u) lo = m;
        else hi = m;
    }
    return lo;
}

// A tensor's elements split into up to 16 / size - 1 before the first 16-byte boundary, whole
// vectors, and the rest.
struct Span {
    long long head, vecs, tail;
};
__host__ __device__ __forceinline__ Span span_of(const void* p, long long numel, int esz) {
    Span s;
    s.head = (long long)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / esz;
    if (s.head > numel) s.head = numel;
    s.vecs = (numel - s.head) * esz / 16;
    s.tail = numel - s.head - s.vecs * (16 / esz);
    return s;
}

__device__ __forceinline__ double square_sum_exact(const uint4& v, bool bf16) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double t = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const double a = __uint_as_float(w[i] << 16), b = __uint_as_float(w[i] & 0xFFFF0000u);
            t = fma(a, a, t);
            t = fma(b, b, t);
        } else {
            const double a = __uint_as_float(w[i]);
            t = fma(a, a, t);
        }
    }
    return t;
}

// Sum of the squares of two vectors.
template <bool BF16>
__device__ __forceinline__ double square_sum(const uint4& u, const uint4& v) {
    const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
    float a = 0.f, b = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (BF16) {
            const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
            a = fmaf(lo, lo, a);
            b = fmaf(hi, hi, b);
        } else {
            const float f = __uint_as_float(w[i]);
            if (i & 1) a = fmaf(f, f, a);
            else b = fmaf(f, f, b);
        }
    }
    const float q = a + b;
    if (q >= 8.2718061e-25f && q <= 1.3292280e36f) return (double)q;
    uint32_t any = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= w[i];
    if ((any & (BF16 ? 0x7FFF7FFFu : 0x7FFFFFFFu)) == 0u) return 0.0;      // experts without tokens: zeros
    return square_sum_exact(u, BF16) + square_sum_exact(v, BF16);
}

__device__ __forceinline__ float load1(const void* p, long long i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

__device__ __forceinline__ double block_sum(double t, double* sm) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if ((threadIdx.x & 31) == 0) sm[threadIdx.x >> 5] = t;
    __syncthreads();
    t = threadIdx.x < THREADS / 32 ? sm[threadIdx.x] : 0.0;
    if (threadIdx.x < 32)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    return t;                                                   // thread 0 holds the sum
}

template <bool BF16>
__device__ __forceinline__ double unit_sum(const uint4* p, long long v0, long long vecs) {
    uint4 v[UNROLL];
#pragma unroll
    for (int j = 0; j < UNROLL; ++j) {
        const long long i = v0 + threadIdx.x + j * THREADS;
        v[j] = i < vecs ? __ldg(p + i) : make_uint4(0, 0, 0, 0);
    }
    double t = 0.0;
#pragma unroll
    for (int j = 0; j < UNROLL; j += 2) t += square_sum<BF16>(v[j], v[j + 1]);
    return t;
}

__global__ void __launch_bounds__(THREADS) grad_norm_kernel(const __grid_constant__ GradList L, bool add, bool last,
                                                            float max_norm, float* __restrict__ norm, GradState* st,
                                                            double* partial) {
    __shared__ double sm[THREADS / 32];
    __shared__ bool finish;
    double t = 0.0;
    for (long long u = blockIdx.x; u < L.first[L.n]; u += gridDim.x) {
        const int k = find(L, u);
        const bool b = L.bf16[k];
        const int esz = b ? 2 : 4;
        const Span s = span_of(L.src[k], L.numel[k], esz);
        const long long v0 = (u - L.first[k]) * UNIT_VECS;
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(L.src[k]) + s.head * esz);
        t += b ? unit_sum<true>(p, v0, s.vecs) : unit_sum<false>(p, v0, s.vecs);
        if (u == L.first[k] && threadIdx.x < s.head + s.tail) {     // at most 14 elements
            const long long i = threadIdx.x < s.head ? threadIdx.x : L.numel[k] - s.tail + (threadIdx.x - s.head);
            const double g = load1(L.src[k], i, b);
            t = fma(g, g, t);
        }
    }
    t = block_sum(t, sm);
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = add ? partial[blockIdx.x] + t : t;
        __threadfence();
        finish = last && atomicAdd(&st->done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!finish) return;
    __threadfence();
    t = 0.0;
    for (int i = threadIdx.x; i < (int)gridDim.x; i += THREADS) t += __ldcg(partial + i);
    t = block_sum(t, sm);
    if (threadIdx.x == 0) {
        const float nrm = (float)sqrt(t);
        *norm = nrm;
        st->done = 0u;
        if (max_norm >= 0.f) {
            // an infinite max_norm clips no norm, not even an infinite one; a NaN norm stays NaN
            const float c = max_norm < INFINITY ? __fdiv_rn(max_norm, nrm + 1e-6f) : nrm >= 0.f ? 1.f : nrm;
            st->coef = c > 1.f ? 1.f : c;
        }
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 scaled(const uint4& v, float c) {
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(w[i] << 16) * c,
                                                           __uint_as_float(w[i] & 0xFFFF0000u) * c);
            w[i] = *reinterpret_cast<const uint32_t*>(&b);
        } else {
            w[i] = __float_as_uint(__uint_as_float(w[i]) * c);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void scale1(const void* src, void* dst, long long i, bool b, float c) {
    if (b) static_cast<__nv_bfloat16*>(dst)[i] = __float2bfloat16_rn(load1(src, i, true) * c);
    else static_cast<float*>(dst)[i] = load1(src, i, false) * c;
}

// Units from the last to the first: the norm's pass has left the last ones in the L2.
__global__ void __launch_bounds__(THREADS) grad_scale_kernel(const __grid_constant__ GradList L, bool in_place,
                                                             const GradState* st) {
    const float c = st->coef;
    if (in_place && c == 1.f) return;
    const long long units = L.first[L.n];
    for (long long q = blockIdx.x; q < units; q += gridDim.x) {
        const long long u = units - 1 - q;
        const int k = find(L, u);
        const bool b = L.bf16[k];
        const int esz = b ? 2 : 4;
        const Span s = span_of(L.src[k], L.numel[k], esz);
        const long long v0 = (u - L.first[k]) * UNIT_VECS;
        const char* src = static_cast<const char*>(L.src[k]) + s.head * esz;
        char* dst = static_cast<char*>(L.dst[k]) + s.head * esz;
        if ((reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
            const uint4* p = reinterpret_cast<const uint4*>(src);
            uint4* o = reinterpret_cast<uint4*>(dst);
            uint4 v[UNROLL];
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                const long long i = v0 + threadIdx.x + j * THREADS;
                if (i < s.vecs) v[j] = p[i];
            }
#pragma unroll
            for (int j = 0; j < UNROLL; ++j) {
                const long long i = v0 + threadIdx.x + j * THREADS;
                if (i < s.vecs) o[i] = b ? scaled<true>(v[j], c) : scaled<false>(v[j], c);
            }
        } else {                                                // source and target aligned differently
            const int per = 16 / esz;
            const long long e0 = s.head + v0 * per, all = s.head + s.vecs * per;
            for (long long i = e0 + threadIdx.x; i < all && i < e0 + (long long)UNIT_VECS * per; i += THREADS)
                scale1(L.src[k], L.dst[k], i, b, c);
        }
        if (u == L.first[k] && threadIdx.x < s.head + s.tail) {
            const long long i = threadIdx.x < s.head ? threadIdx.x : L.numel[k] - s.tail + (threadIdx.x - s.head);
            scale1(L.src[k], L.dst[k], i, b, c);
        }
    }
}

// Fills L with the tensors from `at` on that hold elements; returns the next index.
int fill(const moe_tensor_t* t, const moe_tensor_t* out, int n, int at, GradList* L) {
    L->n = 0;
    L->first[0] = 0;
    for (; at < n && L->n < LIST; ++at) {
        if (t[at].numel == 0) continue;
        const int k = L->n++;
        L->src[k] = t[at].data;
        L->dst[k] = out ? out[at].data : t[at].data;
        L->numel[k] = t[at].numel;
        L->bf16[k] = t[at].dtype == MOE_BF16;
        const Span s = span_of(t[at].data, t[at].numel, L->bf16[k] ? 2 : 4);
        const long long units = (s.vecs + UNIT_VECS - 1) / UNIT_VECS;
        L->first[k + 1] = L->first[k] + (units > 0 ? units : 1);
    }
    return at;
}

}  // namespace

size_t grad_workspace_bytes() { return 256 + (size_t)GRAD_BLOCKS * sizeof(double); }

// max_norm < 0: the norm alone.
cudaError_t launch_grad_norm(const moe_tensor_t* t, const moe_tensor_t* out, int n, float max_norm, float* norm, void* ws,
                             cudaStream_t stream) {
    GradState* st = reinterpret_cast<GradState*>(static_cast<char*>(ws) + GRAD_STATE_OFFSET);
    double* partial = reinterpret_cast<double*>(static_cast<char*>(ws) + 256);
    const int cap = num_sms() * 4 < GRAD_BLOCKS ? num_sms() * 4 : GRAD_BLOCKS;
    long long most = 0;                                         // every launch of a call has the same grid
    GradList L;
    for (int at = 0; at < n;) {
        at = fill(t, out, n, at, &L);
        if (L.first[L.n] > most) most = L.first[L.n];
    }
    const int grid = (int)(most < 1 ? 1 : (most < cap ? most : cap));
    int at = 0;
    bool add = false;
    do {
        at = fill(t, out, n, at, &L);
        grad_norm_kernel<<<grid, THREADS, 0, stream>>>(L, add, at >= n, max_norm, norm, st, partial);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
        add = true;
    } while (at < n);
    if (max_norm < 0.f) return cudaSuccess;
    // the launches of the scaling pass go backwards too: the lists are rebuilt from the front, so remember where each began
    int begins[GRAD_MAX_LAUNCHES];
    int launches = 0;
    for (at = 0; at < n;) {
        begins[launches++] = at;
        at = fill(t, out, n, at, &L);
    }
    for (int i = launches - 1; i >= 0; --i) {
        fill(t, out, n, begins[i], &L);
        if (L.n == 0) continue;
        const long long units = L.first[L.n];
        grad_scale_kernel<<<(int)(units < cap ? units : cap), THREADS, 0, stream>>>(L, out == nullptr, st);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace moe
