// The whole layer for a few tokens (T <= 16) in one cooperative kernel:
//   z = x C^T, picks and gates;  h[e,t] = gate * silu(w1_e x_t + b1) * (w3_e x_t + b3);
//   out[t] = sum over shared and picked experts of w2_e h[e,t], plus the gated b2.
// With so few rows every weight is used a handful of times, so the layer is bound by reading the
// matrices of the experts that some token picked, once.  One block per SM streams them through a
// shared-memory ring by bulk copies, and one producer warp keeps that ring full across all steps:
//   router scores (consumers) | shared experts' w1, w3 already arrive, they do not depend on the picks
//   -> all blocks have written their scores: every block ranks all tokens itself (router warps), while its
//      consumers work on the shared experts
//   -> picked experts' w1, w3
//   -> all blocks have written h: w2, whose first stages arrived while the block waited.
//
// Work is cut into units of 16 weight rows over the full contraction: 8 rows of w1 with the same 8 of w3
// (both halves of the SwiGLU in one thread's registers), or 16 rows of w2.  A unit's stages hold 16 x 2 KB;
// the 8 consumer warps split a stage's columns and add up at the end of the unit.  Up-projection units go
// round the blocks; the down-projection's units (output columns x expert) are cut into equal contiguous
// ranges, so a block may hold part of a column block's experts: it then writes partial sums, and the block
// that completes a column block adds them in block order.  Nothing depends on timing but who does that.
//
// Products: mma.sync m16n8k16 with the weights as the 16-row operand and the tokens as the 8 columns, fp32
// accumulators.  tcgen05's smallest tile is 64 or 128 weight rows, too coarse to spread a few experts evenly
// over 148 SMs, and takes 8-bit weights only against 8-bit activations; here the bound is HBM, the tensor
// pipe idles.  8-bit codes become bf16 exactly; scales are applied to fp32 sums (block scales: each run of
// 32 has its own sum).  Activations are not quantised: x is bf16 as given, and h is kept as the sum of two
// bf16 numbers (16 significant bits).  A thread's k-columns need only be the same for both operands, so
// every fragment is a plain 16- or 8-byte load, without ldmatrix.
// fp32 layers take the same route with FFMA.
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"
#include "pipe.cuh"
#include "route.cuh"

namespace moe {
namespace {

constexpr int CONS_WARPS = 8;
constexpr int CONS = CONS_WARPS * 32;
constexpr int ROUTE_WARPS = 3;                               // 12 warps in all: 168 registers a thread
constexpr int PRODUCER = CONS_WARPS;                            // warp index
constexpr int THREADS = CONS + 32 + ROUTE_WARPS * 32;
constexpr int ROW_BYTES = 2048;                                 // of one weight row in a stage
constexpr int ROWS = 16;
constexpr int STAGE_BYTES = ROWS * (ROW_BYTES + 64);
constexpr int MAX_STAGES = 6;
constexpr int SMEM_LIMIT = 232448;

enum { W_F32, W_BF16, W_E4M3, W_MX };

// esz: bytes of a weight.  PITCH: of a row in a stage, so that the fragment loads of 8 rows (16 bytes a
// thread) or 4 rows (8 bytes a thread) fall into different banks.  A slice is what the 8 warps take at
// once: 128 columns each (fp32: 64).
template <int F>
struct Fmt {
    static constexpr int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
    static constexpr int KS = ROW_BYTES / esz;
    static constexpr int PITCH = ROW_BYTES + (esz == 1 ? 32 : 64);
    static constexpr int PER_WARP = F == W_F32 ? 64 : 128;
    static constexpr int SLICE = PER_WARP * CONS_WARPS;
};

struct Params {
    const void *x, *cen;
    const float* rbias;
    FfnWeights R, Sh;
    void* out;
    int32_t* idx;
    float* gate;
    int32_t* counts;
    float* logits;                                              // [T][E]
    void* h;                                                    // bf16 [rows][2][Hs] (high, low part), fp32 [rows][Hs]
    float4* part;                                               // [blocks][2][NT][32]
    unsigned* cnt;                                              // [column blocks][NT]: units already added up
    uint32_t* err;
    unsigned long long* bar;                                    // two grid barriers (arrivals, ever growing)
    int T, d, E, I, k, Ks, Is, Hs, mode, nst;
    bool bias;
};

// Dynamic shared memory, in bytes from its start.
struct Smem {
    int ring, bars, red, mask, base, ge, gm, gb, gates, zl, pidx, pgate, misc, total;
    __host__ __device__ Smem(int nst, int NT, int T, int E, int k) {
        const int groups = E < T * k ? E : T * k;
        int o = 0;
        auto take = [&](int bytes) { const int at = o; o += (bytes + 15) / 16 * 16; return at; };
        ring = take(nst * STAGE_BYTES);
        bars = take((2 * MAX_STAGES + 1) * 8);
        red = take(2 * CONS_WARPS * NT * 32 * 16);
        mask = take(E * 4);
        base = take(E * 4);
        ge = take(groups * 4);
        gm = take(groups * 4);
        gb = take(groups * 4);
        gates = take(T * k * 4);
        zl = take(ROUTE_WARPS * E * 4);
        pidx = take(T * k * 4);
        pgate = take(T * k * 4);
        misc = take(16);
        total = o;
    }
};

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }
__device__ __forceinline__ void named_arrive(int id, int n) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory"); }

__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two bf16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ uint2 bf16_of_codes(uint32_t w) {
    uint32_t o[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hr));
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.x, f.y);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ float scale_of_byte(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

// Arrival number `old` (of G per round) on a barrier that only grows: the count that completes its round.
__device__ __forceinline__ unsigned long long round_end(unsigned long long old, unsigned G) { return (old / G + 1) * G; }

__device__ __forceinline__ bool grid_wait(unsigned long long* bar, unsigned long long target, volatile int* abort_flag,
                                          uint32_t* err) {
    unsigned long long v;
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(bar) : "memory");
        if (v >= target) return true;
        if ((i & 63u) == 0u) {
            if (*abort_flag) return false;
            if (globaltimer() - t0 > WAIT_NS || i >= WAIT_MAX_POLLS) {
                *abort_flag = 1;
                flag_error(err, ERR_PIPE_TIMEOUT);
                return false;
            }
        }
    }
}

// A block's place in the ring: the producer and the consumers count the same stages.
struct Ring {
    uint32_t base, bars;
    int nst, slot;
    uint32_t phase;
    __device__ __forceinline__ uint32_t full() const { return bars + slot * 8; }
    __device__ __forceinline__ uint32_t empty() const { return bars + (MAX_STAGES + slot) * 8; }
    __device__ __forceinline__ uint32_t at() const { return base + slot * STAGE_BYTES; }
    __device__ __forceinline__ void next() {
        if (++slot == nst) { slot = 0; phase ^= 1u; }
    }
};

// A thread's activation fragments of one slice: 4 steps of 32 columns, 8 columns a thread, for the token
// of its fragment column in each group of 8 tokens; HL = 2: high and low parts.  sf: the scale bytes of the
// warp's 4 runs for its two weight rows.
template <int NT, int HL>
struct Act {
    uint4 v[HL][NT][4];
    uint32_t sf[2];
};

template <int NT, int HL>
__device__ __forceinline__ void load_act(Act<NT, HL>& b, const __nv_bfloat16* const (&ptr)[NT], int low, int kb, int K,
                                         int lane) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const int k = kb + s * 32 + (lane & 3) * 8;
            const bool in = ptr[nt] != nullptr && k < K;
#pragma unroll
            for (int q = 0; q < HL; ++q)
                b.v[q][nt][s] = !in ? make_uint4(0, 0, 0, 0)
                                    : HL == 1 ? __ldg(reinterpret_cast<const uint4*>(ptr[nt] + k))
                                              : __ldcg(reinterpret_cast<const uint4*>(ptr[nt] + q * low + k));
        }
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}

// acc += 16 weight rows x up to 8 NT tokens over the warp's 128 columns kb .. of a slice that starts at byte
// `off` of each row in the stage.  Columns past K hold an earlier stage's bytes: both operands are zeroed.
template <int F, int NT, int HL>
__device__ __forceinline__ void mma_slice(float (&acc)[NT * 4], const Act<NT, HL>& b, uint32_t stage, int off, int kb,
                                          int K, uint32_t mask, int lane) {
    const int g = lane >> 2, c = (lane & 3) * 8;
    const uint32_t row = stage + g * Fmt<F>::PITCH + off;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        uint4 a0 = make_uint4(0, 0, 0, 0), a1 = make_uint4(0, 0, 0, 0);
        if (kb + s * 32 + c < K) {
            if (F == W_BF16) {
                a0 = lds128(row + (s * 32 + c) * 2);
                a1 = lds128(row + 8 * Fmt<F>::PITCH + (s * 32 + c) * 2);
            } else {
                const uint2 q0 = lds64(row + s * 32 + c), q1 = lds64(row + 8 * Fmt<F>::PITCH + s * 32 + c);
                const uint2 l0 = bf16_of_codes(q0.x), h0 = bf16_of_codes(q0.y);
                const uint2 l1 = bf16_of_codes(q1.x), h1 = bf16_of_codes(q1.y);
                a0 = make_uint4(l0.x, l0.y, h0.x, h0.y);
                a1 = make_uint4(l1.x, l1.y, h1.x, h1.y);
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (NT > 1 && ((mask >> (8 * nt)) & 0xFFu) == 0u) continue;
            if (F == W_MX) {                                    // a run's own sum, scaled in fp32
                float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int q = 0; q < HL; ++q) {
                    const uint4& v = b.v[q][nt][s];
                    mma_bf16(t, a0.x, a1.x, a0.y, a1.y, v.x, v.y);
                    mma_bf16(t, a0.z, a1.z, a0.w, a1.w, v.z, v.w);
                }
                const float f0 = scale_of_byte((b.sf[0] >> (8 * s)) & 0xFFu), f1 = scale_of_byte((b.sf[1] >> (8 * s)) & 0xFFu);
                acc[nt * 4] = fmaf(t[0], f0, acc[nt * 4]);
                acc[nt * 4 + 1] = fmaf(t[1], f0, acc[nt * 4 + 1]);
                acc[nt * 4 + 2] = fmaf(t[2], f1, acc[nt * 4 + 2]);
                acc[nt * 4 + 3] = fmaf(t[3], f1, acc[nt * 4 + 3]);
            } else {
#pragma unroll
                for (int q = 0; q < HL; ++q) {
                    const uint4& v = b.v[q][nt][s];
                    mma_bf16(acc + nt * 4, a0.x, a1.x, a0.y, a1.y, v.x, v.y);
                    mma_bf16(acc + nt * 4, a0.z, a1.z, a0.w, a1.w, v.z, v.w);
                }
            }
        }
    }
}

// What a consumer thread needs besides the unit itself.
struct Me {
    Ring ring;
    int warp, lane;
    volatile int* abort_flag;
    uint32_t* err;
};

__device__ __forceinline__ void wait_full(Me& me) { mbar_wait(me.ring.full(), me.ring.phase, me.abort_flag, me.err); }
__device__ __forceinline__ void release(Me& me) {
    __syncwarp();
    if (me.lane == 0) mbar_arrive(me.ring.empty());
    me.ring.next();
}

// One unit of 16 rows on the tensor cores.  ptr: the thread's tokens' activation rows (NULL: not among the
// unit's); sfw[q] (block scales): the words of the runs' scale bytes of the thread's two rows, one per 128
// columns, 1 KB apart.
template <int F, int NT, int HL>
__device__ __forceinline__ void unit_mma(float (&acc)[NT * 4], Me& me, const __nv_bfloat16* const (&ptr)[NT], int low, int K,
                                         uint32_t mask, const uint8_t* const (&sfw)[2]) {
    constexpr int SUBS = Fmt<F>::KS / Fmt<F>::SLICE;
    const int wk = me.warp * Fmt<F>::PER_WARP;
    Act<NT, HL> b;
    auto load = [&](int k0) {
        const int kb = k0 + wk;
        load_act<NT, HL>(b, ptr, low, kb, K, me.lane);
        if (F == W_MX && kb < K) {
            b.sf[0] = __ldg(reinterpret_cast<const uint32_t*>(sfw[0] + (size_t)(kb / 128) * 1024));
            b.sf[1] = __ldg(reinterpret_cast<const uint32_t*>(sfw[1] + (size_t)(kb / 128) * 1024));
        }
    };
    load(0);
    for (int k0 = 0; k0 < K;) {
        wait_full(me);
        const uint32_t stage = me.ring.at();
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            if (k0 >= K) break;
            if (k0 + wk < K)
                mma_slice<F, NT, HL>(acc, b, stage, (sub * Fmt<F>::SLICE + wk) * Fmt<F>::esz, k0 + wk, K, mask, me.lane);
            k0 += Fmt<F>::SLICE;
            if (k0 < K) load(k0);
        }
        release(me);
    }
}

// One unit of 16 rows in fp32: lane pairs share a row, each lane every other 16-byte piece of the warp's
// 64 columns, and acc[n] is token n's sum.
template <int NT>
__device__ __forceinline__ void unit_f32(float (&acc)[NT * 8], Me& me, const float* const (&ptr)[NT * 8], int K) {
    const int row = me.lane >> 1, half = me.lane & 1;
    for (int k0 = 0; k0 < K; k0 += Fmt<W_F32>::KS) {
        wait_full(me);
        const uint32_t a = me.ring.at() + row * Fmt<W_F32>::PITCH;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const int c = me.warp * 64 + (q * 2 + half) * 4;
            if (k0 + c >= K) continue;
            const uint4 u = lds128(a + c * 4);
            const float w0 = __uint_as_float(u.x), w1 = __uint_as_float(u.y), w2 = __uint_as_float(u.z),
                        w3 = __uint_as_float(u.w);
#pragma unroll
            for (int n = 0; n < NT * 8; ++n) {
                if (!ptr[n]) continue;
                const float4 v = __ldcg(reinterpret_cast<const float4*>(ptr[n] + k0 + c));
                acc[n] = fmaf(w0, v.x, fmaf(w1, v.y, fmaf(w2, v.z, fmaf(w3, v.w, acc[n]))));
            }
        }
        release(me);
    }
}

// The 8 warps' fragments of a unit to shared memory; after the barrier, warp (turn * NT + nt) % 8 holds the
// sums of token group nt in fragment order: c[0], c[1]: weight row lane / 4, tokens 2 (lane % 4) and + 1;
// c[2], c[3]: row lane / 4 + 8.  The two buffers alternate, so one barrier per unit is enough.
template <int NT>
__device__ __forceinline__ void put_frag(float4* red, const float (&acc)[NT * 4], const Me& me) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
        red[(me.warp * NT + nt) * 32 + me.lane] = make_float4(acc[nt * 4], acc[nt * 4 + 1], acc[nt * 4 + 2], acc[nt * 4 + 3]);
}
template <int NT>
__device__ __forceinline__ void put_f32(float4* red, float (&acc)[NT * 8], const Me& me) {
    const int row = me.lane >> 1;
#pragma unroll
    for (int n = 0; n < NT * 8; ++n) {
        const float t = acc[n] + __shfl_xor_sync(0xffffffffu, acc[n], 1);
        if ((me.lane & 1) == 0)
            reinterpret_cast<float*>(red + (me.warp * NT + n / 8) * 32 + (row & 7) * 4 + (n & 7) / 2)[(row >> 3) * 2 + (n & 1)] = t;
    }
}
template <int NT>
__device__ __forceinline__ float4 take_frag(const float4* red, int nt, int lane) {
    float4 t = red[nt * 32 + lane];
#pragma unroll
    for (int w = 1; w < CONS_WARPS; ++w) {
        const float4 v = red[(w * NT + nt) * 32 + lane];
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    return t;
}

// One expert as a unit sees it.
struct Group {
    int e;                                                      // index into its stack
    uint32_t mask;                                              // tokens
    int row;                                                    // of h: its first token's
    bool shared;
};

template <int FR, int NT>
struct Kernel {
    static constexpr int FS = FR == W_F32 ? W_F32 : W_BF16;
    using T = typename std::conditional<FR == W_F32, float, __nv_bfloat16>::type;

    const Params& p;
    char* sm;
    const Smem L;
    const int G;                                                // blocks

    __device__ Kernel(const Params& p_, char* sm_) : p(p_), sm(sm_), L(p_.nst, NT, p_.T, p_.E, p_.k), G((int)gridDim.x) {}
    template <typename U>
    __device__ __forceinline__ U* at(int off) const { return reinterpret_cast<U*>(sm + off); }
    __device__ __forceinline__ volatile int* abort_flag() const { return at<int>(L.misc); }
    __device__ __forceinline__ int n_routed() const { return at<volatile int>(L.misc)[1]; }
    __device__ __forceinline__ uint32_t route_bar() const { return smem_u32(sm + L.bars) + 2 * MAX_STAGES * 8; }
    __device__ __forceinline__ Ring ring() const { return Ring{smem_u32(sm + L.ring), smem_u32(sm + L.bars), p.nst, 0, 0}; }

    __device__ __forceinline__ Group group(int gi) const {      // shared experts first
        Group q;
        if (gi < p.Ks) {
            q.e = gi;
            q.mask = (1u << p.T) - 1u;
            q.row = p.T * p.k + gi * p.T;
            q.shared = true;
        } else {
            gi -= p.Ks;
            q.e = at<int>(L.ge)[gi];
            q.mask = at<uint32_t>(L.gm)[gi];
            q.row = at<int>(L.gb)[gi];
            q.shared = false;
        }
        return q;
    }
    // units of the up-projection: shared ones, then (picks known) the routed experts'
    __device__ __forceinline__ int shared_units() const { return p.Ks * ceil_div(p.Is, 8); }
    __device__ __forceinline__ void up_unit(int u, Group& q, int& r0) const {
        const int su = shared_units(), b = u < su ? ceil_div(p.Is, 8) : ceil_div(p.I, 8);
        const int v = u < su ? u : u - su;
        q = group((u < su ? 0 : p.Ks) + v / b);
        r0 = v % b * 8;
    }
    // the down-projection's range of block c among U units
    __device__ __forceinline__ int down_start(long long U, int c) const { return (int)(U * c / G); }

    // ------------------------------------------------------------------------------ producer
    __device__ void produce() {
        const int lane = threadIdx.x & 31;
        Ring ring = this->ring();
        long long issued = 0;
        bool ok = true;
        // copies the unit's rows (lane's row, or NULL) through the ring
        auto stream = [&](const char* row, int K, int esz, int pitch) {
            const int rows = __popc(__ballot_sync(0xffffffffu, row != nullptr));
            const int KS = ROW_BYTES / esz;
            for (int k0 = 0; k0 < K; k0 += KS) {
                ok = mbar_wait(ring.empty(), ring.phase ^ 1u, abort_flag(), p.err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                const uint32_t bytes = (uint32_t)(K - k0 < KS ? K - k0 : KS) * esz;
                if (lane == 0) mbar_expect_tx(ring.full(), rows * bytes);
                __syncwarp();
                if (row) bulk_load(ring.at() + lane * pitch, row + (size_t)k0 * esz, bytes, ring.full());
                ++issued;
                ring.next();
            }
        };
        const int su = shared_units();
        int units = su;
        bool routed = false;
        for (int u = blockIdx.x; ok; u += G) {
            if (u >= units && !routed) {
                ok = __all_sync(0xffffffffu, mbar_wait(route_bar(), 0, abort_flag(), p.err));
                routed = true;
                units = su + n_routed() * ceil_div(p.I, 8);
            }
            if (u >= units || !ok) break;
            Group q;
            int r0;
            up_unit(u, q, r0);
            const int F = q.shared ? FS : FR, I = q.shared ? p.Is : p.I;
            const int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
            const int r = r0 + (lane & 7);
            const void* w = q.shared ? (lane < 8 ? p.Sh.w1 : p.Sh.w3) : (lane < 8 ? p.R.w1 : p.R.w3);
            const char* row = lane < ROWS && r < I ? static_cast<const char*>(w) + ((size_t)q.e * I + r) * p.d * esz : nullptr;
            stream(row, p.d, esz, ROW_BYTES + (esz == 1 ? 32 : 64));
        }
        if (ok) {
            const int groups = p.Ks + n_routed();
            const long long U = (long long)ceil_div(p.d, ROWS) * groups;
            const int end = down_start(U, blockIdx.x + 1);
            for (int u = down_start(U, blockIdx.x); u < end && ok; ++u) {
                const Group q = group(u % groups);
                const int F = q.shared ? FS : FR, I = q.shared ? p.Is : p.I;
                const int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
                const int r = u / groups * ROWS + lane;
                const void* w = q.shared ? p.Sh.w2 : p.R.w2;
                const char* row = lane < ROWS && r < p.d ? static_cast<const char*>(w) + ((size_t)q.e * p.d + r) * I * esz : nullptr;
                stream(row, I, esz, ROW_BYTES + (esz == 1 ? 32 : 64));
            }
        }
        if (!ok) {                                              // given up: let the copies in flight land first
            const int n = (int)(issued < p.nst ? issued : p.nst);
            for (int i = 0; i < n; ++i) {
                const long long s = issued - 1 - i;
                mbar_wait(smem_u32(sm + L.bars) + (uint32_t)(s % p.nst) * 8, (uint32_t)(s / p.nst) & 1u, abort_flag(), p.err,
                          false);
            }
        }
    }

    // ------------------------------------------------------------------------------ router warps
    __device__ void rank() {
        const int tid = threadIdx.x - CONS - 32, warp = tid >> 5, lane = tid & 31;
        const int slots = p.T * p.k;
        if (warp == 0) {                                        // this block's scores are written: tell, and wait for all
            named_sync(2, CONS + 32);
            if (lane == 0) {
                __threadfence();
                const unsigned long long t = round_end(atomicAdd(p.bar, 1ull), G);
                at<volatile int>(L.misc)[2] = grid_wait(p.bar, t, abort_flag(), p.err) ? 1 : 0;
            }
        }
        named_sync(3, ROUTE_WARPS * 32);
        const bool ok = at<volatile int>(L.misc)[2] != 0;
        int32_t* pidx = at<int32_t>(L.pidx);
        float* pgate = at<float>(L.pgate);
        uint32_t* mask = at<uint32_t>(L.mask);
        int* base = at<int>(L.base);
        for (int e = tid; e < p.E; e += ROUTE_WARPS * 32) mask[e] = 0u;
        float* z = at<float>(L.zl) + warp * p.E;
        for (int t = warp; t < p.T && ok; t += ROUTE_WARPS) {
            for (int e = lane; e < p.E; e += 32) z[e] = __ldcg(p.logits + (size_t)t * p.E + e);
            __syncwarp();
            warp_route(z, p.E, p.k, p.mode, p.rbias, lane, pidx + t * p.k, pgate + t * p.k);
            __syncwarp();
        }
        named_sync(3, ROUTE_WARPS * 32);
        for (int s = tid; s < slots && ok; s += ROUTE_WARPS * 32) {
            if ((unsigned)pidx[s] < (unsigned)p.E) atomicOr(mask + pidx[s], 1u << (s / p.k));
            else if (blockIdx.x == 0) flag_error(p.err, ERR_EXPERT_RANGE);
        }
        named_sync(3, ROUTE_WARPS * 32);
        if (warp == 0) {                                        // experts met, in ascending order
            int groups = 0, rows = 0;
            for (int e0 = 0; e0 < p.E && ok; e0 += 32) {
                const uint32_t m = e0 + lane < p.E ? mask[e0 + lane] : 0u;
                const int n = __popc(m);
                int before = n;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, before, o);
                    if (lane >= o) before += v;
                }
                const int all = __shfl_sync(0xffffffffu, before, 31);
                const uint32_t met = __ballot_sync(0xffffffffu, n > 0);
                if (n > 0) {
                    const int gi = groups + __popc(met & ((1u << lane) - 1u));
                    at<int>(L.ge)[gi] = e0 + lane;
                    at<uint32_t>(L.gm)[gi] = m;
                    at<int>(L.gb)[gi] = rows + before - n;
                    base[e0 + lane] = rows + before - n;
                }
                groups += __popc(met);
                rows += all;
            }
            if (lane == 0) at<volatile int>(L.misc)[1] = groups;
        }
        named_sync(3, ROUTE_WARPS * 32);
        for (int s = tid; s < slots && ok; s += ROUTE_WARPS * 32) {
            const int e = pidx[s], t = s / p.k;
            if ((unsigned)e < (unsigned)p.E) at<float>(L.gates)[base[e] + __popc(mask[e] & ((1u << t) - 1u))] = pgate[s];
        }
        if (blockIdx.x == 0 && ok) {
            for (int s = tid; s < slots; s += ROUTE_WARPS * 32) {
                if (p.idx) p.idx[s] = pidx[s];
                if (p.gate) p.gate[s] = pgate[s];
            }
            if (p.counts)
                for (int e = tid; e < p.E; e += ROUTE_WARPS * 32) p.counts[e] = __popc(mask[e]);
        }
        named_sync(3, ROUTE_WARPS * 32);
        if (tid == 0) mbar_arrive(route_bar());
    }

    // ------------------------------------------------------------------------------ consumers
    // Router scores of this block's experts (rows blockIdx.x, + G, ...) for all tokens.
    __device__ void scores(float* red, const Me& me) {
        constexpr int VEC = FR == W_F32 ? 4 : 8;
        const int nv = p.d / VEC, tid = threadIdx.x;
        const uint4* x = static_cast<const uint4*>(p.x);
        const uint4* cen = static_cast<const uint4*>(p.cen);
        for (int e = blockIdx.x; e < p.E; e += G) {
            float acc[NT * 8];
#pragma unroll
            for (int t = 0; t < NT * 8; ++t) acc[t] = 0.f;
            for (int i = tid; i < nv; i += CONS) {
                const uint4 c = __ldg(cen + (size_t)e * nv + i);
                const uint32_t cw[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int t = 0; t < NT * 8; ++t) {
                    if (t >= p.T) break;
                    const uint4 v = __ldg(x + (size_t)t * nv + i);
                    const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        if (FR == W_F32) {
                            acc[t] = fmaf(__uint_as_float(vw[q]), __uint_as_float(cw[q]), acc[t]);
                        } else {
                            acc[t] = fmaf(__uint_as_float(vw[q] << 16), __uint_as_float(cw[q] << 16), acc[t]);
                            acc[t] = fmaf(__uint_as_float(vw[q] & 0xFFFF0000u), __uint_as_float(cw[q] & 0xFFFF0000u), acc[t]);
                        }
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT * 8; ++t) {
                if (t >= p.T) break;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
                if (me.lane == 0) red[me.warp * NT * 8 + t] = acc[t];
            }
            named_sync(1, CONS);
            if (tid < p.T) {
                float z = red[tid];
#pragma unroll
                for (int w = 1; w < CONS_WARPS; ++w) z += red[w * NT * 8 + tid];
                p.logits[(size_t)tid * p.E + e] = z;
            }
            named_sync(1, CONS);
        }
    }

    __device__ __forceinline__ float bias_at(const void* b, size_t i) const { return to_f32(static_cast<const T*>(b)[i]); }
    __device__ __forceinline__ float gate_of(const Group& q, int tok) const {
        return q.shared ? 1.f : at<float>(L.gates)[q.row + __popc(q.mask & ((1u << tok) - 1u))];
    }

    template <int F>
    __device__ __forceinline__ void up(Me& me, const Group& q, int r0, float4* red) {
        const int g = me.lane >> 2;
        if constexpr (F == W_F32) {
            const float* ptr[NT * 8];
            float acc[NT * 8];
#pragma unroll
            for (int n = 0; n < NT * 8; ++n) {
                ptr[n] = (q.mask >> n) & 1u ? static_cast<const float*>(p.x) + (size_t)n * p.d : nullptr;
                acc[n] = 0.f;
            }
            unit_f32<NT>(acc, me, ptr, p.d);
            put_f32<NT>(red, acc, me);
        } else {
            const __nv_bfloat16* ptr[NT];
            float acc[NT * 4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int n = nt * 8 + g;
                ptr[nt] = (q.mask >> n) & 1u ? static_cast<const __nv_bfloat16*>(p.x) + (size_t)n * p.d : nullptr;
            }
#pragma unroll
            for (int i = 0; i < NT * 4; ++i) acc[i] = 0.f;
            const uint8_t* sfw[2] = {nullptr, nullptr};
            if (F == W_MX) {                                    // w1's half of the tile, and w3's
                const int r = r0 + g;
                sfw[0] = p.R.sf13 + ((size_t)q.e * ceil_div(p.I, 128) + r / 128) * ceil_div(p.d, 128) * 1024 + (r & 31) * 16 +
                         ((r >> 5) & 3) * 4;
                sfw[1] = sfw[0] + 512;
            }
            unit_mma<F, NT, 1>(acc, me, ptr, 0, p.d, q.mask, sfw);
            put_frag<NT>(red, acc, me);
        }
    }

    // h of one unit from the summed fragments (token group nt).
    __device__ __forceinline__ void finish_up(const Group& q, int r0, float4 c, int nt, int lane) {
        const int I = q.shared ? p.Is : p.I, r = r0 + (lane >> 2);
        if (r >= I) return;
        const FfnWeights& W = q.shared ? p.Sh : p.R;
        const size_t at_row = (size_t)q.e * I + r;
        float s1 = 1.f, s3 = 1.f;
        if (FR == W_E4M3 && !q.shared) { s1 = W.s1[at_row]; s3 = W.s3[at_row]; }
        const float b1 = p.bias ? bias_at(W.b1, at_row) : 0.f, b3 = p.bias ? bias_at(W.b3, at_row) : 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = nt * 8 + (lane & 3) * 2 + i;
            if (!((q.mask >> tok) & 1u)) continue;
            const float a = (i ? c.y : c.x) * s1 + b1, b = (i ? c.w : c.z) * s3 + b3;
            const float h = silu_f32(a) * b * gate_of(q, tok);
            const size_t row = q.row + __popc(q.mask & ((1u << tok) - 1u));
            if (FR == W_F32) {
                static_cast<float*>(p.h)[row * p.Hs + r] = h;
            } else {
                const __nv_bfloat16 hi = __float2bfloat16_rn(h);
                const float rest = h - __bfloat162float(hi);
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.h) + row * 2 * p.Hs + r;
                o[0] = hi;
                o[p.Hs] = __float2bfloat16_rn(isfinite(rest) ? rest : 0.f);
            }
        }
    }

    template <int F>
    __device__ __forceinline__ void down(float (&acc)[FR == W_F32 ? NT * 8 : NT * 4], Me& me, const Group& q, int cb) {
        const int g = me.lane >> 2, K = q.shared ? p.Is : p.I;
        if constexpr (F == W_F32) {
            const float* ptr[NT * 8];
#pragma unroll
            for (int n = 0; n < NT * 8; ++n)
                ptr[n] = (q.mask >> n) & 1u
                             ? static_cast<const float*>(p.h) + (size_t)(q.row + __popc(q.mask & ((1u << n) - 1u))) * p.Hs
                             : nullptr;
            unit_f32<NT>(acc, me, ptr, K);
        } else {
            const __nv_bfloat16* ptr[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int n = nt * 8 + g;
                ptr[nt] = (q.mask >> n) & 1u ? static_cast<const __nv_bfloat16*>(p.h) +
                                                   (size_t)(q.row + __popc(q.mask & ((1u << n) - 1u))) * 2 * p.Hs
                                             : nullptr;
            }
            const uint8_t* sfw[2] = {nullptr, nullptr};
            if (F == W_MX) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = cb * ROWS + g + 8 * i;
                    sfw[i] = p.R.sf2 + ((size_t)q.e * ceil_div(p.d, 256) + r / 256) * ceil_div(p.I, 128) * 1024 +
                             ((r >> 7) & 1) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
                }
            }
            if (F == W_E4M3) {                                  // per-row scales differ from expert to expert
                float t[NT * 4];
#pragma unroll
                for (int i = 0; i < NT * 4; ++i) t[i] = 0.f;
                unit_mma<F, NT, 2>(t, me, ptr, p.Hs, K, q.mask, sfw);
                const int r = cb * ROWS + g;
                const float* s2 = p.R.s2 + (size_t)q.e * p.d;
                const float f0 = r < p.d ? s2[r] : 0.f, f1 = r + 8 < p.d ? s2[r + 8] : 0.f;
#pragma unroll
                for (int i = 0; i < NT * 4; ++i) acc[i] = fmaf(t[i], (i & 2) ? f1 : f0, acc[i]);
            } else {
                unit_mma<F, NT, 2>(acc, me, ptr, p.Hs, K, q.mask, sfw);
            }
        }
    }

    // A column block's sums over the block's groups [u0, u1) of `groups`: to the output when they are all,
    // else to the partial sums; the block that completes the count adds those of all blocks in order.
    __device__ __forceinline__ void finish_down(float4 c, int cb, int u0, int u1, int groups, long long U, int nt, int lane) {
        if (u1 - u0 != groups) {
            const int me = blockIdx.x;
            auto slot = [&](int b) { return p.part + (((size_t)b * 2 + (down_start(U, b) / groups == cb ? 0 : 1)) * NT + nt) * 32 + lane; };
            __stcg(slot(me), c);
            __threadfence();
            __syncwarp();
            unsigned old = 0;
            if (lane == 0) old = atomicAdd(p.cnt + cb * NT + nt, (unsigned)(u1 - u0));
            old = __shfl_sync(0xffffffffu, old, 0);
            if (old + (unsigned)(u1 - u0) != (unsigned)groups) return;
            __threadfence();
            const int first = cb * groups, last = first + groups;   // units of the column block (U < 2^31)
            int b = me;
            while (b > 0 && down_start(U, b) > first) --b;
            c = make_float4(0.f, 0.f, 0.f, 0.f);
            for (; b < G && down_start(U, b) < last; ++b) {
                if (down_start(U, b + 1) == down_start(U, b)) continue;
                const float4 v = __ldcg(slot(b));
                c.x += v.x; c.y += v.y; c.z += v.z; c.w += v.w;
            }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = cb * ROWS + (lane >> 2) + 8 * i;
            if (r >= p.d) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = nt * 8 + (lane & 3) * 2 + j;
                if (tok >= p.T) continue;
                float v = i ? (j ? c.w : c.z) : (j ? c.y : c.x);
                if (p.bias) {
                    for (int s = 0; s < p.Ks; ++s) v += bias_at(p.Sh.b2, (size_t)s * p.d + r);
                    for (int s = 0; s < p.k; ++s) {
                        const int e = at<int32_t>(L.pidx)[tok * p.k + s];
                        if ((unsigned)e < (unsigned)p.E) v = fmaf(at<float>(L.pgate)[tok * p.k + s], bias_at(p.R.b2, (size_t)e * p.d + r), v);
                    }
                }
                static_cast<T*>(p.out)[(size_t)tok * p.d + r] = from_f32<T>(v);
            }
        }
    }

    __device__ void consume() {
        Me me = {ring(), (int)(threadIdx.x >> 5), (int)(threadIdx.x & 31), abort_flag(), p.err};
        float4* red0 = at<float4>(L.red);
        const int cbs = ceil_div(p.d, ROWS);
        for (int i = blockIdx.x * CONS + threadIdx.x; i < cbs * NT; i += G * CONS) p.cnt[i] = 0u;
        scores(reinterpret_cast<float*>(red0), me);
        named_arrive(2, CONS + 32);

        int turn = 0;
        auto buffer = [&] { return red0 + (turn & 1) * CONS_WARPS * NT * 32; };
        const int su = shared_units();
        int units = su, met = 0;
        bool routed = false;
        for (int u = blockIdx.x;; u += G) {
            if (u >= units && !routed) {
                if (threadIdx.x == 0)                           // one thread decides, also when the wait gives up
                    at<volatile int>(L.misc)[3] = mbar_wait(route_bar(), 0, abort_flag(), p.err) ? n_routed() : 0;
                named_sync(1, CONS);
                met = at<volatile int>(L.misc)[3];
                routed = true;
                units = su + met * ceil_div(p.I, 8);
            }
            if (u >= units) break;
            Group q;
            int r0;
            up_unit(u, q, r0);
            if (FR != FS && !q.shared) up<FR>(me, q, r0, buffer());
            else up<FS>(me, q, r0, buffer());
            named_sync(1, CONS);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if ((turn * NT + nt) % CONS_WARPS == me.warp) finish_up(q, r0, take_frag<NT>(buffer(), nt, me.lane), nt, me.lane);
            ++turn;
        }
        named_sync(1, CONS);                                    // the block's h is written
        if (threadIdx.x == 0) {
            __threadfence();
            const unsigned long long t = round_end(atomicAdd(p.bar + 1, 1ull), G);
            grid_wait(p.bar + 1, t, abort_flag(), p.err);
        }
        named_sync(1, CONS);

        const int groups = p.Ks + met;
        if (groups == 0) {                                      // no shared expert, and no pick left
            for (size_t i = (size_t)blockIdx.x * CONS + threadIdx.x; i < (size_t)p.T * p.d; i += (size_t)G * CONS)
                static_cast<T*>(p.out)[i] = from_f32<T>(0.f);
            return;
        }
        const long long U = (long long)cbs * groups;
        const int end = down_start(U, blockIdx.x + 1);
        for (int u = down_start(U, blockIdx.x); u < end;) {
            const int cb = u / groups, u0 = u, u1 = (cb + 1) * groups < end ? (cb + 1) * groups : end;
            float acc[FR == W_F32 ? NT * 8 : NT * 4];
#pragma unroll
            for (float& a : acc) a = 0.f;
            for (; u < u1; ++u) {
                const Group q = group(u % groups);
                if (FR != FS && !q.shared) down<FR>(acc, me, q, cb);
                else down<FS>(acc, me, q, cb);
            }
            if constexpr (FR == W_F32) put_f32<NT>(buffer(), acc, me);
            else put_frag<NT>(buffer(), acc, me);
            named_sync(1, CONS);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if ((turn * NT + nt) % CONS_WARPS == me.warp)
                    finish_down(take_frag<NT>(buffer(), nt, me.lane), cb, u0, u1, groups, U, nt, me.lane);
            ++turn;
        }
    }
};

template <int FR, int NT>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(16) char sm[];
    Kernel<FR, NT> k(p, sm);
    if (threadIdx.x == 0) {
        const uint32_t bars = smem_u32(sm + k.L.bars);
        for (int s = 0; s < p.nst; ++s) {
            mbar_init(bars + s * 8, 1);
            mbar_init(bars + (MAX_STAGES + s) * 8, CONS_WARPS);
        }
        mbar_init(k.route_bar(), 1);
        int* misc = k.template at<int>(k.L.misc);
        misc[0] = misc[1] = misc[2] = misc[3] = 0;              // given up; experts met; scores complete; the consumers' view
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (warp < CONS_WARPS) k.consume();
    else if (warp == PRODUCER) k.produce();
    else k.rank();
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr int GRID_MAX = 256;

struct Layout {
    size_t logits, h, part, cnt, total;
    int Hs;
};
Layout few_layout(const Dims& D) {
    Layout L;
    const size_t T = D.T > 0 ? D.T : 1;
    const int widest = D.Ks > 0 && D.Is > D.I ? D.Is : D.I;
    L.Hs = (widest + 7) / 8 * 8;
    size_t o = 256;
    L.logits = o; o += al256(T * D.E * 4);
    L.h = o; o += al256(T * (D.k + D.Ks) * L.Hs * 4);           // two bf16 parts, or fp32
    L.part = o; o += al256((size_t)GRID_MAX * 2 * 2 * 32 * 16);
    L.cnt = o; o += al256((size_t)ceil_div(D.d, ROWS) * 2 * 4);
    L.total = o;
    return L;
}

template <int FR, int NT>
cudaError_t launch(Params& p, cudaStream_t st) {
    const Smem none(0, NT, p.T, p.E, p.k);
    int n = (SMEM_LIMIT - none.total) / STAGE_BYTES;
    p.nst = n > MAX_STAGES ? MAX_STAGES : n;
    const Smem L(p.nst, NT, p.T, p.E, p.k);
    auto kern = few_kernel<FR, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L.total);
    if (e != cudaSuccess) return e;
    const int grid = num_sms() < GRID_MAX ? num_sms() : GRID_MAX;
    void* args[] = {&p};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(THREADS), args, L.total, st);
}

template <int FR>
cudaError_t launch_t(Params& p, cudaStream_t st) {
    return p.T <= 8 ? launch<FR, 1>(p, st) : launch<FR, 2>(p, st);
}

}  // namespace

bool few_supported(const Dims& D) {
    if (D.T > MOE_FEW_MAX_TOKENS || D.d > FEW_MAX_D) return false;
    return D.bf16 || (D.d % 4 == 0 && D.I % 4 == 0 && (D.Ks == 0 || D.Is % 4 == 0));
}

size_t few_workspace_bytes(const Dims& D) { return few_layout(D).total; }

cudaError_t launch_few(const Dims& D, const void* x, const void* cen, const float* rbias, const FfnWeights& R,
                       const FfnWeights& Sh, void* out, int32_t* idx, float* gate, int32_t* counts, void* ws,
                       cudaStream_t st) {
    const Layout L = few_layout(D);
    char* w = static_cast<char*>(ws);
    Params p = {};
    p.x = x; p.cen = cen; p.rbias = rbias; p.R = R; p.Sh = Sh;
    p.out = out; p.idx = idx; p.gate = gate; p.counts = counts;
    p.logits = reinterpret_cast<float*>(w + L.logits);
    p.h = w + L.h;
    p.part = reinterpret_cast<float4*>(w + L.part);
    p.cnt = reinterpret_cast<unsigned*>(w + L.cnt);
    p.err = reinterpret_cast<uint32_t*>(w);
    p.bar = reinterpret_cast<unsigned long long*>(w + FEW_BARRIER_OFFSET);
    p.T = D.T; p.d = D.d; p.E = D.E; p.I = D.I; p.k = D.k; p.Ks = D.Ks; p.Is = D.Is; p.Hs = L.Hs;
    p.mode = D.gate_mode; p.bias = D.bias;
    if (!D.bf16) return launch_t<W_F32>(p, st);
    if (D.mx) return launch_t<W_MX>(p, st);
    if (D.q8) return launch_t<W_E4M3>(p, st);
    return launch_t<W_BF16>(p, st);
}

}  // namespace moe
