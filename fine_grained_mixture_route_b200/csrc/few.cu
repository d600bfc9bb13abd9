// The whole layer for a few tokens (T <= 16) in one cooperative kernel:
//   z = x C^T, picks and gates;  h[e,t] = gate * silu(w1_e x_t + b1) * (w3_e x_t + b3);
//   out[t] = sum over shared and picked experts of w2_e h[e,t], plus the gated b2.
// With so few rows every weight is used a handful of times, so the layer is bound by reading the
// matrices of the experts that some token picked, once.  One block per SM streams them through a
// shared-memory ring, and two producer warps keep that ring full across all steps:
//   router scores (consumers) | shared experts' w1, w3 already arrive, they do not depend on the picks
//   -> all blocks have written their scores: every block ranks all tokens itself (router warps), while its
//      consumers work on the shared experts
//   -> picked experts' w1, w3; the block's gates, ranked after the picks, are waited for before h and before b2
//   -> all blocks have written h: w2, whose first stages arrived while the block waited.
//
// Work is cut into units of 32 weight rows (fp32: 16) over the full contraction: in each row tile of 16, 8 rows of
// w1 with the same 8 of w3 (both halves of the SwiGLU in one thread's registers), or 16 rows of w2.  A unit's
// stages hold a slice of its columns, of the weights and of its tokens' activations alike; the 8 consumer warps
// split the slice and add up at the end of the unit.  Up-projection units go round the blocks; the
// down-projection's units (output columns x expert) are cut into equal contiguous ranges, so a block may hold
// part of a column block's experts: it then writes partial sums, and the block that completes a column block
// adds them in block order.  Nothing depends on timing but who does that.
//
// The ring is filled by cp.async, 16 bytes a thread: bulk copies cost about 30 ns each however short (rows of
// 1 KB: 3.7 TB/s, 2 KB: 5.2 TB/s; cp.async: 6.1 to 6.4 TB/s for either, measured with nothing else in the
// kernel).  Activations take the same way, as loads straight into registers would be waited for at every slice.
//
// Products: mma.sync m16n8k16 with the weights as the 16-row operand and the tokens as the 8 columns, fp32
// accumulators.  tcgen05's smallest tile is 64 or 128 weight rows, too coarse to spread a few experts evenly
// over 148 SMs, and takes 8-bit weights only against 8-bit activations; here the bound is HBM, the tensor
// pipe idles.  Scales are applied to fp32 sums (block scales: each run of 32 has its own sum).  Activations are
// not quantised: x is bf16 as given, and h is fp32, which the consumers cut into three bf16 parts of 8 bits each as they
// load it (exact): it costs no rounding, and no more bytes of the ring than two parts would.
// 8-bit codes become fp16, exactly and in one instruction a pair (bf16 takes four, and the conversions then
// bound the kernel: 185 us instead of 165 for w1, w3 of 22 block-scaled experts of 2048 x 7168).  Their
// activations are therefore fp16 too, each row times a power of two that brings its largest finite value into
// [2^14, 2^15), below 2^-112 times 2^126: x in one number, h in two (22 bits of its fp32 value).  fp16's smallest step is
// 2^-24, so a row is off by at most 2^-25 / 2^14 = 2^-39 of its largest value (below 2^-112: by 2^-151), and x keeps its
// 8 bits down to 2^-31 of it.  For h the rows' largest values have to be known: one grid barrier more, behind
// which the rows are converted, while the first weights of w2 arrive.
// A thread's k-columns need only be the same for both operands, so every fragment is a plain 16- or 8-byte
// load, without ldmatrix.
// fp32 layers take the same route with FFMA.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "launch.h"
#include "pipe.cuh"

namespace moe {
namespace {

constexpr int CONS_WARPS = 8;
constexpr int CONS = CONS_WARPS * 32;
constexpr int ROUTE_WARPS = 2, PRODUCERS = 2;                   // 12 warps in all: 168 registers a thread
constexpr int THREADS = CONS + (ROUTE_WARPS + PRODUCERS) * 32;
constexpr int MAX_STAGES = 8;
constexpr int RING_BYTES = 128 << 10;                           // of weights under way that are enough
constexpr int SMEM_LIMIT = 232448;

enum { W_F32, W_BF16, W_E4M3, W_MX };

// A stage: 16 R weight rows (R row tiles) over KS columns, the same columns of the unit's tokens, and with block
// scales the rows' scale bytes.  FR: format of the routed experts, F: of these weights.  The 8 consumer warps
// take KS / 8 columns each.  PITCH, ACT: of a weight row and an activation row, so that the fragment loads of 8
// rows (16 bytes a thread) or 4 rows (8 bytes a thread) fall into different banks.
template <int FR, int F>
struct Fmt {
    static constexpr int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
    static constexpr int ROWB = FR == W_F32 || FR == W_BF16 ? 1024 : 512;
    static constexpr int KS = ROWB / esz;
    static constexpr int PITCH = ROWB + (esz == 1 ? 32 : 64);
    static constexpr int PER_WARP = KS / CONS_WARPS;
};
constexpr int ACT = 1024 + 64;                                  // a row of x: 512 columns of 16 bits or 256 of 32
// A row of h: 4 bytes a column, fp32 or 8 fp16 high parts and their 8 low parts in turn.  A thread of the MMAs reads 32
// bytes at 4 places 32 bytes apart and 8 rows: 16 bytes more than a multiple of 128 keep those apart.
template <int FR, int F>
constexpr int hrow() { return FR == W_F32 ? ACT : Fmt<FR, F>::KS * 4 + 16; }
template <int FR, int R>
struct Stage {
    static constexpr int act = hrow<FR, FR>() > ACT ? hrow<FR, FR>() : ACT;      // of a token, at most
    static constexpr int acts = 16 * R * (Fmt<FR, FR>::ROWB + 64);
    static __host__ __device__ int scales(int T) { return acts + T * act; }
    // Weight rows at a multiple of 128 bytes in every stage: 16 bytes off, the copies are slower (one token on 256 experts
    // of 2048 x 7168: 142 us instead of 131)
    static __host__ __device__ int bytes(int T) { return (scales(T) + (FR == W_MX ? 16 * R * 16 : 0) + 127) / 128 * 128; }
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
    float* h;                                                   // [rows][Hs]; 8-bit experts' rows: see convert_h
    __half* x16;                                                // 8-bit experts: [T][d], row t times 1 / xf[t]
    float* xf;
    unsigned* hmax;                                             // their rows' largest finite |h|, as bits
    float4* part;                                               // [blocks][2][R NT][32]
    unsigned* cnt;                                              // [column blocks][R NT]: units already added up
    uint32_t* err;
    unsigned long long* bar;                                    // three grid barriers (arrivals, ever growing)
    int T, d, E, I, k, Ks, Is, Hs, mode, nst, stage;
    bool bias;
};

// Buffers of a unit's fragments: two that alternate save a barrier a unit; with 16 tokens on two row tiles one
// leaves room for a third stage.
__host__ __device__ constexpr int red_buffers(int frags) { return frags > 2 ? 1 : 2; }

// Dynamic shared memory, in bytes from its start.
constexpr int SPARE = ROUTE_WARPS * 4;                          // groups of 8 lanes that rank tokens
struct Smem {
    int ring, bars, turns, red, mask, base, ge, gm, gb, gates, pidx, pgate, misc, total;
    __host__ __device__ Smem(int ring_bytes, int frags, int T, int E, int k) {
        const int groups = E < T * k ? E : T * k;
        int o = 0;
        auto take = [&](int bytes) { const int at = o; o += (bytes + 15) / 16 * 16; return at; };
        ring = take(ring_bytes);
        bars = take((2 * MAX_STAGES + 3) * 8);
        turns = take(3 * 8);
        red = take(red_buffers(frags) * CONS_WARPS * frags * 32 * 16);
        mask = take(E * 4);
        base = take(E * 4);
        ge = take(groups * 4);
        gm = take(groups * 4);
        gb = take(groups * 4);
        gates = take(T * k * 4);
        pidx = take((T + SPARE) * k * 4);
        pgate = take((T + SPARE) * k * 4);
        misc = take(32);
        total = o;
    }
};

__device__ __forceinline__ void named_sync(int id, int n) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory"); }

// Asynchronous copies of 16 bytes past the L1, or of 4 (both addresses aligned to them), and the arrival of all
// of a thread's copies so far on a barrier that counts its threads.
template <int N>
__device__ __forceinline__ void async_load(uint32_t dst, const void* src) {
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void async_arrive(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ void mma_bf16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two fp16 pairs (exact; NaN stays NaN).
__device__ __forceinline__ uint2 f16_of_codes(uint32_t w) {
    const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3);
    const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// The power of two that brings m (finite, >= 0) into [2^14, 2^15), for m below 2^-112 less; its reciprocal is normal.
__device__ __forceinline__ float f16_scale(float m) {
    const int e = (int)(__float_as_uint(m) >> 23) - 127;        // subnormal or 0: -127
    return __uint_as_float((uint32_t)((14 - e > 126 ? 126 : 14 - e) + 127) << 23);
}

// 2^(b - 127) of the two low bytes of w (255: NaN), by way of bf16, which holds them all.
__device__ __forceinline__ float2 scales_of_bytes(uint32_t w) {
    const __nv_bfloat162_raw r = __nv_cvt_e8m0x2_to_bf162raw((__nv_fp8x2_storage_t)w);
    return make_float2(__uint_as_float((uint32_t)r.x << 16), __uint_as_float((uint32_t)r.y << 16));
}

// A grid barrier is a count of arrivals, G per round, that only grows: round_end is the count that completes the
// round in which it stands at `v`.
__device__ __forceinline__ unsigned long long load_acquire(const unsigned long long* p) {
    unsigned long long v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long round_end(unsigned long long v, unsigned G) { return (v / G + 1) * G; }
__device__ __forceinline__ void grid_arrive(unsigned long long* bar) {
    __threadfence();
    asm volatile("red.release.gpu.global.add.u64 [%0], 1;" ::"l"(bar) : "memory");
}

__device__ __forceinline__ bool grid_wait(unsigned long long* bar, unsigned long long target, volatile int* abort_flag,
                                          uint32_t* err) {
    const unsigned long long t0 = globaltimer();
    for (uint32_t i = 1;; ++i) {
        if (load_acquire(bar) >= target) return true;
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
    int nst, stage, slot;
    uint32_t phase;
    __device__ __forceinline__ uint32_t full() const { return bars + slot * 8; }
    __device__ __forceinline__ uint32_t empty() const { return bars + (MAX_STAGES + slot) * 8; }
    __device__ __forceinline__ uint32_t at() const { return base + slot * stage; }
    __device__ __forceinline__ void next() {
        if (++slot == nst) { slot = 0; phase ^= 1u; }
    }
};

__device__ __forceinline__ uint4 lds128(const char* a) { return *reinterpret_cast<const uint4*>(a); }

// With an infinite number or NaN among its columns a first part's sum is not finite, and stands alone.
__device__ __forceinline__ float add_parts(float first, float others) { return fabsf(first) < INFINITY ? first + others : first; }

// A thread's fragments of a stage: 16 R weight rows and up to 8 NT tokens over the warp's columns, wk from the
// stage's start and kb < K of all.  act[nt]: where the thread's token's row is in the stage (0: the token is not
// among the unit's); HL = 1: a row of x, HL = 2: one of h beside 8-bit weights.  Columns past K hold an earlier stage's bytes:
// both operands are zeroed.  sf: the scale bytes of the warp's 2 runs.
template <int FR, int F, int NT, int HL, int R>
struct Frag {
    using L = Fmt<FR, F>;
    static_assert(F != W_BF16 || HL == 1, "h beside 16-bit weights is unit_parts'");
    static constexpr int STEPS = L::PER_WARP / 32;
    using A = typename std::conditional<F == W_BF16, uint4, uint2>::type;
    A a[STEPS][R][2];
    uint4 b[STEPS][NT][HL];
    uint32_t sf[R][2];

    __device__ __forceinline__ void load(const char* stage, const int (&act)[NT], int sfs, int wk, int kb, int K, int lane) {
        const int g = lane >> 2, c = (lane & 3) * 8;
        const char* row = stage + g * L::PITCH;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
            const int k = wk + s * 32 + c;
            const bool in = kb + s * 32 + c < K;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int q = 0; q < HL; ++q)
                    b[s][nt][q] = in && act[nt] ? *reinterpret_cast<const uint4*>(stage + act[nt] + k * 2 * HL + q * 16) : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    a[s][i][h] = in ? *reinterpret_cast<const A*>(row + (i * 16 + h * 8) * L::PITCH + k * L::esz) : A{};
        }
        if (F == W_MX) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sf[i][h] = *reinterpret_cast<const uint32_t*>(stage + sfs + (i * 16 + h * 8 + g) * 16 + wk / 128 * 4) >> (wk / 64 % 2 * 16);
        }
    }

    // acc += weights x activations.  The tensor cores cut off what they add to a large sum instead of rounding it, always
    // towards zero: a stage (8-bit weights: a step of 32 columns, in which block scales are constant) has its own short
    // sum, and those are added in fp32.
    __device__ __forceinline__ void multiply(float (&acc)[R][NT * 4], uint32_t mask) const {
        if constexpr (F == W_BF16) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (NT > 1 && ((mask >> (8 * nt)) & 0xFFu) == 0u) continue;
                float t[R][4] = {};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const uint4 &a0 = a[s][i][0], &a1 = a[s][i][1], &v = b[s][nt][0];
                        mma_bf16(t[i], a0.x, a1.x, a0.y, a1.y, v.x, v.y);
                        mma_bf16(t[i], a0.z, a1.z, a0.w, a1.w, v.z, v.w);
                    }
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][nt * 4 + j] += t[i][j];
            }
        } else {
            float2 f[R][2];
            if (F == W_MX) {
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) f[i][h] = scales_of_bytes(sf[i][h]);
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s)
#pragma unroll
                for (int i = 0; i < R; ++i) {
                    const uint2 l0 = f16_of_codes(a[s][i][0].x), h0 = f16_of_codes(a[s][i][0].y);
                    const uint2 l1 = f16_of_codes(a[s][i][1].x), h1 = f16_of_codes(a[s][i][1].y);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if (NT > 1 && ((mask >> (8 * nt)) & 0xFFu) == 0u) continue;
                        float t[HL][4] = {};                    // high and low parts apart: half the chain of products
#pragma unroll
                        for (int q = 0; q < HL; ++q) {
                            const uint4& v = b[s][nt][q];
                            mma_f16(t[q], l0.x, l1.x, l0.y, l1.y, v.x, v.y);
                            mma_f16(t[q], h0.x, h1.x, h0.y, h1.y, v.z, v.w);
                        }
                        const float f0 = F != W_MX ? 1.f : s ? f[i][0].y : f[i][0].x, f1 = F != W_MX ? 1.f : s ? f[i][1].y : f[i][1].x;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float v = HL > 1 ? t[0][j] + t[HL - 1][j] : t[0][j];
                            acc[i][nt * 4 + j] = fmaf(v, j < 2 ? f0 : f1, acc[i][nt * 4 + j]);
                        }
                    }
                }
        }
    }
};

// What a consumer thread needs besides the unit itself.
struct Me {
    Ring ring;
    const char* sm;                                             // where the ring starts
    int warp, lane;
    volatile int* abort_flag;
    uint32_t* err;
};

__device__ __forceinline__ void wait_full(const Me& me, const Ring& r) {
    mbar_wait_limit(r.full(), r.phase, me.abort_flag, me.err, true, WAIT_NS);
}
__device__ __forceinline__ void release(Me& me) {
    __syncwarp();
    if (me.lane == 0) mbar_arrive(me.ring.empty());
    me.ring.next();
}

// One unit of 16 R rows on the tensor cores for the tokens of `mask`, whose activation rows stand in each stage
// in order, with HL parts each.
template <int FR, int F, int NT, int HL, int R>
__device__ __forceinline__ void unit_mma(float (&acc)[R][NT * 4], Me& me, int sfs, int K, uint32_t mask) {
    using L = Fmt<FR, F>;
    const int wk = me.warp * L::PER_WARP;
    int act[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int n = nt * 8 + (me.lane >> 2);
        act[nt] = (mask >> n) & 1u ? Stage<FR, R>::acts + __popc(mask & ((1u << n) - 1u)) * (HL > 1 ? hrow<FR, F>() : ACT) : 0;
    }
    // With 8-bit weights the latencies of a stage (shared memory, conversions, a chain of products), two warps a
    // scheduler, take longer than its bytes: where the registers allow it (one part an activation), a stage's
    // fragments are loaded while the one before is multiplied (126 us instead of 145 for the products of w1, w3
    // of 22 e4m3 experts of 2048 x 7168; with two parts, or 16-bit weights, it spills and loses).
    using Fr = Frag<FR, F, NT, HL, R>;
    Ring ahead = me.ring;
    auto fetch = [&](Fr& f, int k0) {
        wait_full(me, ahead);
        if (k0 + wk < K) f.load(me.sm + ahead.slot * ahead.stage, act, sfs, wk, k0 + wk, K, me.lane);
        ahead.next();
    };
    if constexpr (F == W_BF16 || HL > 1) {
        Fr f;
        for (int k0 = 0; k0 < K; k0 += L::KS) {
            fetch(f, k0);
            if (k0 + wk < K) f.multiply(acc, mask);
            release(me);
        }
    } else {
        Fr f[2];
        int k0 = 0;
        auto step = [&](const Fr& now, Fr& next) {
            if (k0 + L::KS < K) fetch(next, k0 + L::KS);
            if (k0 + wk < K) now.multiply(acc, mask);
            release(me);
            k0 += L::KS;
        };
        fetch(f[0], 0);
        while (true) {
            step(f[0], f[1]);
            if (k0 >= K) break;
            step(f[1], f[0]);
            if (k0 >= K) break;
        }
    }
}

// A unit of the down-projection with 16-bit weights and up to TOK tokens, t as unit_mma's.  Every fp32 number of h is the sum of
// three bf16 ones, exactly (down to bf16's smallest step, 2^-133): each part is the upper half of what the parts before leave, its
// top 8 bits.  (Of an infinite number or NaN the first part is one too, and the others mean nothing.)  The unit's tokens stand in order in the products' columns, so
// that 9 to 16 tokens of the layer take a second group of columns only in units that have as many.  With one or two tokens, as most
// units of routed experts have, the parts take the free columns: column 4 j + q is part q of token j, a third of the products;
// else column j is token j and each part has products of its own.  (16 tokens, alternating inputs: 64 experts of 1408 x 2048
// 178 us, 202 with products for every part and columns by the layer's tokens; 32 experts of 2048 x 7168 484 us, 555 with the
// columns by the layer's tokens.)
template <int FR, int NT, int R, int TOK>
__device__ __forceinline__ void unit_parts(float (&t)[R][NT * 4], Me& me, int K, uint32_t mask) {
    using L = Fmt<FR, W_BF16>;
    constexpr int STEPS = L::PER_WARP / 32, COLS = TOK == 2 ? 4 : 1, SETS = TOK == 2 ? 1 : 3, GROUPS = TOK > 8 ? 2 : 1;
    const int wk = me.warp * L::PER_WARP, g = me.lane >> 2, c = (me.lane & 3) * 8, q = g % COLS, n = __popc(mask);
    const char* row = me.sm + g * L::PITCH;
    const uint32_t up = 0xFFFF0000u, m1 = q > 0 ? up : 0u, m2 = q > 1 ? up : 0u;     // what the parts before a column's hold
    auto rest = [](uint32_t w, uint32_t m) { return __float_as_uint(__uint_as_float(w) - __uint_as_float(w & m)); };
    float acc[GROUPS][R][4] = {};
    for (int k0 = 0; k0 < K; k0 += L::KS) {
        wait_full(me, me.ring);
        if (k0 + wk < K) {
            const char* stage = me.sm + me.ring.slot * me.ring.stage + Stage<FR, R>::acts;
            const int at = me.ring.slot * me.ring.stage;
            uint4 a[STEPS][R][2], v[GROUPS][STEPS][2];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int k = wk + s * 32 + c;
                const bool in = k0 + k < K;
#pragma unroll
                for (int grp = 0; grp < GROUPS; ++grp) {
                    const int j = grp * 8 + g / COLS;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        v[grp][s][h] = in && j < n && q < 3 ? lds128(stage + j * hrow<FR, W_BF16>() + k * 4 + h * 16) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int h = 0; h < 2; ++h) a[s][i][h] = in ? lds128(row + at + (i * 16 + h * 8) * L::PITCH + k * 2) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int grp = 0; grp < GROUPS; ++grp) {
                float sum[SETS][R][4] = {};                     // short chains of products
#pragma unroll
                for (int s = 0; s < STEPS; ++s) {
                    const uint4 &lo = v[grp][s][0], &hi = v[grp][s][1];
                    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
                    uint32_t p[8];
#pragma unroll
                    for (int set = 0; set < SETS; ++set) {
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (TOK == 2) p[e] = rest(rest(w[e], m1), m2);
                            else p[e] = set == 0 ? w[e] : rest(p[e], up);
                        }
                        const uint32_t b0 = __byte_perm(p[0], p[1], 0x7632), b1 = __byte_perm(p[2], p[3], 0x7632);
                        const uint32_t b2 = __byte_perm(p[4], p[5], 0x7632), b3 = __byte_perm(p[6], p[7], 0x7632);
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const uint4 &a0 = a[s][i][0], &a1 = a[s][i][1];
                            mma_bf16(sum[set][i], a0.x, a1.x, a0.y, a1.y, b0, b1);
                            mma_bf16(sum[set][i], a0.z, a1.z, a0.w, a1.w, b2, b3);
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        acc[grp][i][e] += TOK == 2 ? sum[0][i][e] : add_parts(sum[0][i][e], sum[SETS > 1][i][e] + sum[SETS - 1][i][e]);
            }
        }
        release(me);
    }
    // A lane has columns 2 (lane % 4) and + 1, of the unit's tokens; t wants those of the layer's.
    const int quad = me.lane & ~3;
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float all = 0.f;                                    // two tokens: parts 0 and 1 here, part 2 in the next lane
            if (TOK == 2) all = add_parts(acc[0][i][2 * h], acc[0][i][2 * h + 1] + __shfl_down_sync(0xffffffffu, acc[0][i][2 * h], 1));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int tok = nt * 8 + (me.lane & 3) * 2 + e, j = __popc(mask & ((1u << tok) - 1u));
                    float y = 0.f;
                    if (TOK == 2) {
                        y = __shfl_sync(0xffffffffu, all, quad + (j * 2 & 3));
                    } else {
#pragma unroll
                        for (int grp = 0; grp < GROUPS; ++grp)
#pragma unroll
                            for (int o = 0; o < 2; ++o) {
                                const float z = __shfl_sync(0xffffffffu, acc[grp][i][2 * h + o], quad + (j >> 1 & 3));
                                if (j >> 3 == grp && (j & 1) == o) y = z;
                            }
                    }
                    t[i][nt * 4 + h * 2 + e] = (mask >> tok) & 1u ? y : 0.f;
                }
        }
}

// The same for the shared experts of layers with 8-bit ones, which are few: called, as the others need the registers (four
// tokens: e4m3 261 us instead of 266, block-scaled 282 instead of 286).
template <int FR, int NT, int R>
struct Called {
    float t[R][NT * 4];
    int slot;
    uint32_t phase;
};
template <int FR, int NT, int R>
__device__ __noinline__ Called<FR, NT, R> unit_parts_called(Me me, int K, uint32_t mask) {
    Called<FR, NT, R> o;
    unit_parts<FR, NT, R, NT * 8>(o.t, me, K, mask);
    o.slot = me.ring.slot;
    o.phase = me.ring.phase;
    return o;
}

// One unit of 16 rows in fp32: lane pairs share a row, each lane every other 16-byte piece of the warp's
// 32 columns, and acc[n] is token n's sum.
template <int NT>
__device__ __forceinline__ void unit_f32(float (&acc)[NT * 8], Me& me, int K, uint32_t mask) {
    using L = Fmt<W_F32, W_F32>;
    const int row = me.lane >> 1, half = me.lane & 1;
    for (int k0 = 0; k0 < K; k0 += L::KS) {
        wait_full(me, me.ring);
        const char* a = me.sm + me.ring.slot * me.ring.stage + row * L::PITCH;
        const char* x = me.sm + me.ring.slot * me.ring.stage + Stage<W_F32, 1>::acts;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int c = me.warp * L::PER_WARP + (q * 2 + half) * 4;
            if (k0 + c >= K) continue;
            const uint4 u = lds128(a + c * 4);
            const float w0 = __uint_as_float(u.x), w1 = __uint_as_float(u.y), w2 = __uint_as_float(u.z),
                        w3 = __uint_as_float(u.w);
            const char* at = x + c * 4;
#pragma unroll
            for (int n = 0; n < NT * 8; ++n) {
                if (!((mask >> n) & 1u)) continue;
                const uint4 v = lds128(at);
                at += ACT;
                acc[n] = fmaf(w0, __uint_as_float(v.x),
                              fmaf(w1, __uint_as_float(v.y), fmaf(w2, __uint_as_float(v.z), fmaf(w3, __uint_as_float(v.w), acc[n]))));
            }
        }
        release(me);
    }
}

// The 8 warps' fragments of a unit to shared memory.  Fragment f = row tile * NT + group of 8 tokens; after the
// barrier one warp adds up a fragment: c[0], c[1]: weight row lane / 4 of the tile, tokens 2 (lane % 4) and + 1;
// c[2], c[3]: row lane / 4 + 8.  Two buffers alternate, so that one barrier per unit is enough.
template <int NT, int R>
__device__ __forceinline__ void put_frag(float4* red, const float (&acc)[R][NT * 4], const Me& me) {
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            red[(me.warp * R * NT + i * NT + nt) * 32 + me.lane] =
                make_float4(acc[i][nt * 4], acc[i][nt * 4 + 1], acc[i][nt * 4 + 2], acc[i][nt * 4 + 3]);
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
template <int FRAGS>
__device__ __forceinline__ float4 take_frag(const float4* red, int f, int lane) {
    float4 t = red[f * 32 + lane];
#pragma unroll
    for (int w = 1; w < CONS_WARPS; ++w) {
        const float4 v = red[(w * FRAGS + f) * 32 + lane];
        t.x += v.x; t.y += v.y; t.z += v.z; t.w += v.w;
    }
    return t;
}

// Picks and gates of one token by W lanes (l: a lane's place among them) from its E <= W NPL logits zg: the rules
// of warp_route, made for latency.  A lane keeps the keys of its experts l + W i in registers, in an unsigned
// order (0: none left; taken, NaN or -infinity), and every round is one search of the lane's own keys and one
// reduction (largest key, lowest index that has it).  Gates wait: the picks are what the weights' copies need.
__device__ __forceinline__ float key_of(float z, int e, int mode, const float* __restrict__ bias) {
    const float b = bias ? bias[e] : 0.f;
    return mode == 2 ? 1.0f / (1.0f + expf(-z)) + b : z + b;
}
template <int W, int NPL>
__device__ __forceinline__ void few_pick(const float* zg, int E, int k, int mode, const float* __restrict__ bias, int l,
                                         int32_t* idx_row, float* key_row) {
    float v[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) v[i] = l + W * i < E ? __ldcg(zg + l + W * i) : 0.f;
    uint32_t key[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const float y = l + W * i < E ? key_of(v[i], l + W * i, mode, bias) : -INFINITY;
        const uint32_t b = __float_as_uint(y + 0.f);            // the two zeros are equal
        key[i] = y > -INFINITY ? (b >> 31 ? ~b : b | 0x80000000u) : 0u;
    }
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0u;
        int at = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (key[i] > best) { best = key[i]; at = l + W * i; }
        if (W == 32) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, best);
            at = __reduce_min_sync(0xffffffffu, best == top ? at : 0x7fffffff);
            best = top;
        } else {
#pragma unroll
            for (int o = W / 2; o > 0; o >>= 1) {
                const uint32_t ob = __shfl_xor_sync(0xffffffffu, best, o);
                const int oa = __shfl_xor_sync(0xffffffffu, at, o);
                if (ob > best || (ob == best && oa < at)) { best = ob; at = oa; }
            }
        }
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (l + W * i == at) key[i] = 0u;
        if (l == 0) {
            idx_row[j] = at;
            key_row[j] = best == 0u ? -INFINITY : __uint_as_float(best >> 31 ? best & 0x7FFFFFFFu : ~best);
        }
    }
    __syncwarp();
}
// gate_row: the picks' keys as few_pick left them, and in the end the gates.
template <int W, int NPL>
__device__ __forceinline__ void few_gate(const float* zg, int E, int k, int mode, const float* __restrict__ bias, int l,
                                         const int32_t* idx_row, float* gate_row) {
    auto sum = [](float v) {
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    };
    float m = -INFINITY, s = 0.f;
    if (mode == 0) {
        float v[NPL];
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            v[i] = l + W * i < E ? key_of(__ldcg(zg + l + W * i), l + W * i, 0, bias) : -INFINITY;
            m = fmaxf(m, v[i]);
        }
#pragma unroll
        for (int o = W / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int i = 0; i < NPL; ++i)
            if (l + W * i < E) s += expf(v[i] - m);
    } else if (mode == 1) {
        m = gate_row[0];
    }
    __syncwarp();
    for (int j = l; j < k; j += W) {
        const float g = mode == 2 ? 1.0f / (1.0f + expf(-__ldcg(zg + (idx_row[j] < E ? idx_row[j] : 0)))) : expf(gate_row[j] - m);
        gate_row[j] = g;
        if (mode != 0) s += g;
    }
    s = 1.0f / sum(s);
    for (int j = l; j < k; j += W) gate_row[j] *= s;
    __syncwarp();
}

// One expert as a unit sees it.
struct Group {
    int e;                                                      // index into its stack
    uint32_t mask;                                              // tokens
    int row;                                                    // of h: its first token's
    bool shared;
};

template <int FR, int NT, int R>
struct Kernel {
    static_assert(FR != W_F32 || R == 1, "fp32 units have one row tile");
    static constexpr int FRAGS = R * NT, UP = 8 * R, DOWN = 16 * R;    // fragments, rows of w1 (and w3) and of w2 of a unit
    static constexpr int FS = FR == W_F32 ? W_F32 : W_BF16;
    static constexpr bool Q8 = FR == W_E4M3 || FR == W_MX;
    using T = typename std::conditional<FR == W_F32, float, __nv_bfloat16>::type;

    const Params& p;
    char* sm;
    const Smem L;
    const int G;                                                // blocks

    __device__ Kernel(const Params& p_, char* sm_) : p(p_), sm(sm_), L(p_.nst * p_.stage, FRAGS, p_.T, p_.E, p_.k), G((int)gridDim.x) {}
    template <typename U>
    __device__ __forceinline__ U* at(int off) const { return reinterpret_cast<U*>(sm + off); }
    __device__ __forceinline__ volatile int* abort_flag() const { return at<int>(L.misc); }
    __device__ __forceinline__ int n_routed() const { return at<volatile int>(L.misc)[1]; }
    __device__ __forceinline__ int h_rows() const { return at<volatile int>(L.misc)[4]; }    // of picked experts
    __device__ __forceinline__ uint32_t route_bar() const { return smem_u32(sm + L.bars) + 2 * MAX_STAGES * 8; }
    __device__ __forceinline__ uint32_t h_bar() const { return route_bar() + 8; }
    __device__ __forceinline__ uint32_t gate_bar() const { return route_bar() + 16; }
    __device__ __forceinline__ Ring ring() const { return Ring{smem_u32(sm + L.ring), smem_u32(sm + L.bars), p.nst, p.stage, 0, 0}; }

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
    __device__ __forceinline__ int shared_units() const { return p.Ks * ceil_div(p.Is, UP); }
    __device__ __forceinline__ void up_unit(int u, Group& q, int& r0) const {
        const int su = shared_units(), b = u < su ? ceil_div(p.Is, UP) : ceil_div(p.I, UP);
        const int v = u < su ? u : u - su;
        q = group((u < su ? 0 : p.Ks) + v / b);
        r0 = v % b * UP;
    }
    // the down-projection's range of block c among U units (U G < 2^32: at most 2048 column blocks of 576 groups)
    __device__ __forceinline__ int down_start(uint32_t U, int c) const { return (int)(U * (uint32_t)c / (uint32_t)G); }
    // the block whose range holds unit u: the last c with U c < (u + 1) G
    __device__ __forceinline__ int down_block(uint32_t U, int u) const { return (int)(((uint32_t)(u + 1) * (uint32_t)G - 1u) / U); }

    // ------------------------------------------------------------------------------ producers
    // What a unit's stages bring, column by column: weights, then activations.  Warp w of the two copies the first
    // (0) or second 8 rows of each row tile (w1 and w3 of an up unit), and every other activation row; warp 0
    // copies the scale bytes.  A warp keeps its rows' addresses: 5 instructions a row and stage, as every one
    // delays the next copy.  Rows behind the matrix repeat its last one; their sums are not used.
    struct Source {
        const char* row[8 * R];                                 // this lane's 16 bytes of the first stage
        int bytes, esz;                                         // of a weight row, of a weight
        const char* act;                                        // activations of the unit's first token, this lane's part
        int act_row;                                            // bytes between tokens' rows
        uint32_t mask;
        bool down;                                              // rows of h, in order; else rows of x, by token
        const char* sf;                                         // this lane's row's scale word of the first 128 columns
        // row j of tile i: row i * tile + j of the matrix at `at`, of which `there` rows are left
        __device__ __forceinline__ void rows(const void* at, int tile, int there, int lane) {
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = i * tile + j < there ? i * tile + j : there - 1;
                    row[i * 8 + j] = static_cast<const char*>(at) + (long long)r * bytes + lane * 16;
                }
        }
    };
    __device__ __forceinline__ void copy_weights(const Source& q, const Ring& ring, int c, int w, int lane) const {
        constexpr int ROWB = Fmt<FR, FR>::ROWB;
        const int to = ROWB + (q.esz == 1 ? 32 : 64);
        uint32_t dst = ring.at() + w * 8 * to + lane * 16;
        const bool in0 = c + lane * 16 < q.bytes, in1 = ROWB > 512 && c + 512 + lane * 16 < q.bytes;
#pragma unroll
        for (int i = 0; i < R; ++i, dst += 8 * to)
#pragma unroll
            for (int j = 0; j < 8; ++j, dst += to) {
                const char* src = q.row[i * 8 + j] + c;
                if (in0) async_load<16>(dst, src);
                if (in1) async_load<16>(dst + 512, src + 512);
            }
        if (FR == W_MX && q.sf && w == 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (c + j * 128 < q.bytes)
                    async_load<4>(ring.at() + Stage<FR, R>::scales(p.T) + lane * 16 + j * 4, q.sf + (size_t)(c / 128 + j) * 1024);
        }
    }
    __device__ __forceinline__ void copy_acts(const Source& q, const Ring& ring, int c, int w, int lane) const {
        constexpr int ROWB = Fmt<FR, FR>::ROWB;
        const uint32_t to = ring.at() + Stage<FR, R>::acts + lane * 16;
        auto copy = [](uint32_t dst, const char* src, bool in0, bool in1) {
            if (in0) async_load<16>(dst, src);
            if (in1) async_load<16>(dst + 512, src + 512);
        };
        if (q.down) {                                           // this warp: one half (512 or 1024 bytes) of all rows
            const int up = q.esz == 1 ? 2 : q.esz == 2 ? 1 : 0; // 4 bytes a column
            const int half = (ROWB << up) / 2, c0 = (c << up) + w * half, end = q.bytes << up;
            const int pitch = FR == W_F32 ? ACT : 2 * half + 16;               // hrow
            const bool in0 = c0 + lane * 16 < end, in1 = half > 512 && c0 + 512 + lane * 16 < end;
            uint32_t dst = to + w * half;
            const char* a = q.act + c0;
            for (int n = __popc(q.mask); n > 0; --n, a += q.act_row, dst += pitch) copy(dst, a, in0, in1);
        } else {                                                // every other row
            const int up = q.esz == 1 ? 1 : 0, c0 = c << up, end = q.bytes << up;    // 8-bit weights have 16-bit x
            const bool in0 = c0 + lane * 16 < end, in1 = (ROWB << up) > 512 && c0 + 512 + lane * 16 < end;
            uint32_t dst = to + w * ACT, m = w ? q.mask & (q.mask - 1u) : q.mask;
            while (m) {
                copy(dst, q.act + c0 + (size_t)(__ffs(m) - 1) * q.act_row, in0, in1);
                dst += 2 * ACT;
                m &= m - 1u;
                m &= m - 1u;
            }
        }
    }
    __device__ __forceinline__ Source up_source(int u, int w, int lane) const {
        Group g;
        int r0;
        up_unit(u, g, r0);
        const int F = g.shared ? FS : FR, I = g.shared ? p.Is : p.I;
        const int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
        const void* m = g.shared ? (w ? p.Sh.w3 : p.Sh.w1) : (w ? p.R.w3 : p.R.w1);
        Source q;
        q.bytes = p.d * esz; q.esz = esz;
        q.rows(static_cast<const char*>(m) + ((size_t)g.e * I + r0) * q.bytes, 8, I - r0, lane);
        q.act = (Q8 && !g.shared ? reinterpret_cast<const char*>(p.x16) : static_cast<const char*>(p.x)) + lane * 16;
        q.act_row = p.d * (int)sizeof(T);
        q.mask = g.mask; q.down = false; q.sf = nullptr;
        const int r = r0 + (lane >> 4) * 8 + (lane & 7);        // of the lane's row in the stage
        if (FR == W_MX && !g.shared && lane < DOWN && r < I)
            q.sf = reinterpret_cast<const char*>(p.R.sf13) + ((size_t)g.e * ceil_div(I, 128) + r / 128) * ceil_div(p.d, 128) * 1024 +
                   (lane >> 3 & 1) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
        return q;
    }
    __device__ __forceinline__ Source down_source(int u, int groups, int w, int lane) const {
        const Group g = group(u % groups);
        const int F = g.shared ? FS : FR, I = g.shared ? p.Is : p.I;
        const int esz = F == W_F32 ? 4 : F == W_BF16 ? 2 : 1;
        const int r0 = u / groups * DOWN;
        const void* m = g.shared ? p.Sh.w2 : p.R.w2;
        Source q;
        q.bytes = I * esz; q.esz = esz;
        q.rows(static_cast<const char*>(m) + ((size_t)g.e * p.d + r0 + w * 8) * q.bytes, 16, p.d - r0 - w * 8, lane);
        q.act_row = p.Hs * 4;
        q.act = reinterpret_cast<const char*>(p.h) + (size_t)g.row * q.act_row + lane * 16;
        q.mask = g.mask; q.down = true; q.sf = nullptr;
        const int r = r0 + lane;
        if (FR == W_MX && !g.shared && lane < DOWN && r < p.d)
            q.sf = reinterpret_cast<const char*>(p.R.sf2) + ((size_t)g.e * ceil_div(p.d, 256) + r / 256) * ceil_div(I, 128) * 1024 +
                   ((r >> 7) & 1) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
        return q;
    }

    __device__ void produce(int w) {
        constexpr int ROWB = Fmt<FR, FR>::ROWB;
        const int lane = threadIdx.x & 31;
        Ring ring = this->ring();
        auto free_slot = [&](const Ring& r) {
            return __all_sync(0xffffffffu, mbar_try_wait(r.empty(), r.phase ^ 1u) ||
                                               mbar_wait(r.empty(), r.phase ^ 1u, abort_flag(), p.err)) != 0;
        };
        const int su = shared_units();
        int units = su;
        bool routed = false, ok = true;
        for (int u = blockIdx.x;; u += G) {
            if (u >= units && !routed) {
                ok = __all_sync(0xffffffffu, mbar_wait(route_bar(), 0, abort_flag(), p.err));
                routed = true;
                units = su + n_routed() * ceil_div(p.I, UP);
            }
            if (u >= units || !ok) break;
            const Source q = up_source(u, w, lane);
            for (int c = 0; c < q.bytes && (ok = free_slot(ring)); c += ROWB) {
                copy_weights(q, ring, c, w, lane);
                copy_acts(q, ring, c, w, lane);
                async_arrive(ring.full());
                ring.next();
            }
        }
        if (ok) {
            const int groups = p.Ks + n_routed();
            const uint32_t U = (uint32_t)(ceil_div(p.d, DOWN) * groups);
            const int begin = down_start(U, blockIdx.x), end = down_start(U, blockIdx.x + 1);
            // weights of as many stages as there are do not wait for h
            Ring early = ring;
            int left = p.nst;
            for (int u = begin; u < end && left > 0 && ok; ++u) {
                const Source q = down_source(u, groups, w, lane);
                for (int c = 0; c < q.bytes && left > 0 && (ok = free_slot(early)); c += ROWB, --left) {
                    copy_weights(q, early, c, w, lane);
                    early.next();
                }
            }
            ok = ok && __all_sync(0xffffffffu, mbar_wait(h_bar(), 0, abort_flag(), p.err));
            int done = p.nst - left;                            // stages whose weights are under way
            for (int u = begin; u < end && ok; ++u) {
                const Source q = down_source(u, groups, w, lane);
                for (int c = 0; c < q.bytes; c += ROWB) {
                    if (done > 0) {
                        --done;
                    } else {
                        if (!(ok = free_slot(ring))) break;
                        copy_weights(q, ring, c, w, lane);
                    }
                    copy_acts(q, ring, c, w, lane);
                    async_arrive(ring.full());
                    ring.next();
                }
            }
        }
        async_wait_all();                                       // also when a wait gave up
    }

    // ------------------------------------------------------------------------------ router warps
    // Picks of all tokens (and the experts' masks), or their gates.
    template <int W, int NPL>
    __device__ __forceinline__ void rank_tokens(int warp, int lane, bool gates) {
        constexpr int GROUPS = ROUTE_WARPS * 32 / W;
        const int l = lane % W;
        for (int t0 = 0; t0 < p.T; t0 += GROUPS) {
            const int mine = t0 + warp * (32 / W) + lane / W, t = mine < p.T ? mine : 0;
            // groups without a token of their own repeat the first, into rows behind the last
            const int row = mine < p.T ? mine : p.T + warp * (32 / W) + lane / W;
            int32_t* idx = at<int32_t>(L.pidx) + row * p.k;
            float* gate = at<float>(L.pgate) + row * p.k;
            if (gates) {
                few_gate<W, NPL>(p.logits + (size_t)t * p.E, p.E, p.k, p.mode, p.rbias, l, idx, gate);
                continue;
            }
            few_pick<W, NPL>(p.logits + (size_t)t * p.E, p.E, p.k, p.mode, p.rbias, l, idx, gate);
            for (int j = l; j < p.k && mine < p.T; j += W) {
                if ((unsigned)idx[j] < (unsigned)p.E) atomicOr(at<uint32_t>(L.mask) + idx[j], 1u << t);
                else if (blockIdx.x == 0) flag_error(p.err, ERR_EXPERT_RANGE);
            }
            __syncwarp();
        }
    }
    // few tokens: a warp each; many: 8 or 16 lanes each
    __device__ __forceinline__ void rank_tokens(int warp, int lane, bool gates) {
        if (p.T <= ROUTE_WARPS || p.E > 512) {
            if (p.E <= 64) rank_tokens<32, 2>(warp, lane, gates);
            else if (p.E <= 256) rank_tokens<32, 8>(warp, lane, gates);
            else rank_tokens<32, 32>(warp, lane, gates);
        } else if (p.E <= 64) {
            rank_tokens<8, 8>(warp, lane, gates);
        } else if (p.E <= 256) {
            rank_tokens<16, 16>(warp, lane, gates);
        } else {
            rank_tokens<16, 32>(warp, lane, gates);
        }
    }

    __device__ void rank() {
        const int tid = threadIdx.x - CONS - PRODUCERS * 32, warp = tid >> 5, lane = tid & 31;
        const int slots = p.T * p.k;
        const int32_t* pidx = at<int32_t>(L.pidx);
        const float* pgate = at<float>(L.pgate);
        uint32_t* mask = at<uint32_t>(L.mask);
        int* base = at<int>(L.base);
        for (int e = tid; e < p.E; e += ROUTE_WARPS * 32) mask[e] = 0u;
        if (tid == 0) at<volatile int>(L.misc)[2] = grid_wait(p.bar, at<unsigned long long>(L.turns)[0], abort_flag(), p.err);
        named_sync(3, ROUTE_WARPS * 32);
        const bool ok = at<volatile int>(L.misc)[2] != 0;
        if (ok) rank_tokens(warp, lane, false);
        named_sync(3, ROUTE_WARPS * 32);
        if (warp == 0) {                                        // experts met, in ascending order
            const int per = ceil_div(p.E, 32), e0 = lane * per, e1 = e0 + per < p.E ? e0 + per : p.E;
            int mine = 0;                                       // experts met << 16 | rows: at most 512 of either
            for (int e = e0; e < e1 && ok; ++e) {
                const int n = __popc(mask[e]);
                mine += n + (n > 0 ? 1 << 16 : 0);
            }
            int before = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o) before += v;
            }
            const int all = __shfl_sync(0xffffffffu, before, 31), groups = all >> 16;
            before -= mine;
            int gi = before >> 16, rows = before & 0xFFFF;
            for (int e = e0; e < e1 && ok; ++e) {
                const uint32_t m = mask[e];
                if (m == 0u) continue;
                at<int>(L.ge)[gi] = e;
                at<uint32_t>(L.gm)[gi] = m;
                at<int>(L.gb)[gi++] = rows;
                base[e] = rows;
                rows += __popc(m);
            }
            if (lane == 0) {
                at<volatile int>(L.misc)[1] = groups;
                at<volatile int>(L.misc)[4] = all & 0xFFFF;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(route_bar());
        }
        if (ok) rank_tokens(warp, lane, true);
        named_sync(3, ROUTE_WARPS * 32);
        for (int s = tid; s < slots && ok; s += ROUTE_WARPS * 32) {
            const int e = pidx[s], t = s / p.k;
            if ((unsigned)e < (unsigned)p.E) at<float>(L.gates)[base[e] + __popc(mask[e] & ((1u << t) - 1u))] = pgate[s];
        }
        named_sync(3, ROUTE_WARPS * 32);
        if (tid == 0) mbar_arrive(gate_bar());
        if (blockIdx.x == 0 && ok) {
            for (int s = tid; s < slots; s += ROUTE_WARPS * 32) {
                if (p.idx) p.idx[s] = pidx[s];
                if (p.gate) p.gate[s] = pgate[s];
            }
            if (p.counts)
                for (int e = tid; e < p.E; e += ROUTE_WARPS * 32) p.counts[e] = __popc(mask[e]);
        }
    }

    // ------------------------------------------------------------------------------ consumers
    // Router scores.  A task is one expert with TB tokens; 1, 2, 4 or 8 warps split its columns, as many as the
    // grid has warps for, so that with few experts and tokens a warp's loads are all under way at once.
    template <int TB>
    __device__ __forceinline__ void scores(float* red, const Me& me) {
        constexpr int VEC = FR == W_F32 ? 4 : 8;
        const int tbs = ceil_div(p.T, TB), tasks = p.E * tbs;
        int S = CONS_WARPS;
        while (S > 1 && (long long)tasks * S > (long long)G * CONS_WARPS) S >>= 1;
        const int per = CONS_WARPS / S, part = me.warp & (S - 1), sub = me.warp / S;
        const int nv = p.d / VEC, n = ceil_div(ceil_div(nv, 32), S) * 32;    // vectors of a warp
        const int v1 = (part + 1) * n < nv ? (part + 1) * n : nv;
        for (int t0 = blockIdx.x * per; t0 < tasks; t0 += G * per) {
            const int task = t0 + sub, e = task % p.E, tok = task / p.E * TB;
            float acc[TB] = {};
            if (task < tasks) {
                const uint4* c = static_cast<const uint4*>(p.cen) + (size_t)e * nv;
                const uint4* x[TB];
#pragma unroll
                for (int t = 0; t < TB; ++t)                    // tokens that are not there repeat the last one
                    x[t] = static_cast<const uint4*>(p.x) + (size_t)(tok + t < p.T ? tok + t : p.T - 1) * nv;
#pragma unroll 4
                for (int i = part * n + me.lane; i < v1; i += 32) {
                    const uint4 w = __ldg(c + i);
                    const uint32_t cw[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int t = 0; t < TB; ++t) {
                        const uint4 v = __ldg(x[t] + i);
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
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) acc[t] += __shfl_xor_sync(0xffffffffu, acc[t], o);
                if (me.lane == t) red[me.warp * TB + t] = acc[t];
            }
            named_sync(1, CONS);
            if ((int)threadIdx.x < per * TB) {
                const int q = threadIdx.x / TB, t = threadIdx.x % TB, mine = t0 + q;
                if (mine < tasks && mine / p.E * TB + t < p.T) {
                    float z = 0.f;
                    for (int w = 0; w < S; ++w) z += red[(q * S + w) * TB + t];
                    p.logits[(size_t)(mine / p.E * TB + t) * p.E + mine % p.E] = z;
                }
            }
            named_sync(1, CONS);
        }
    }

    // 8-bit experts' x: a task is 512 columns of a token, whose whole row it reads for the scale.  The last
    // blocks take them first, those which the scores leave idle.
    __device__ void convert_x(float* red, const Me& me) {
        const int parts = ceil_div(p.d, 512), nv = p.d / 8, tid = threadIdx.x;
        const uint4* x = static_cast<const uint4*>(p.x);
        for (int task = G - 1 - blockIdx.x; task < parts * p.T; task += G) {
            const int t = task / parts, j = task % parts;
            float m = 0.f;
            auto larger = [&](uint32_t w) {
                const float a = fabsf(__uint_as_float(w << 16)), b = fabsf(__uint_as_float(w & 0xFFFF0000u));
                if (a < INFINITY) m = fmaxf(m, a);              // neither infinity nor NaN
                if (b < INFINITY) m = fmaxf(m, b);
            };
            for (int i = tid; i < nv; i += CONS) {
                const uint4 v = __ldg(x + (size_t)t * nv + i);
                larger(v.x); larger(v.y); larger(v.z); larger(v.w);
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            if (me.lane == 0) red[me.warp] = m;
            named_sync(1, CONS);
            m = red[0];
#pragma unroll
            for (int w = 1; w < CONS_WARPS; ++w) m = fmaxf(m, red[w]);
            const float f = f16_scale(m);
            const int c = j * 512 + tid * 2;
            if (c < p.d) {
                const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.x) + (size_t)t * p.d + c));
                const __half2 h = __floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
                *reinterpret_cast<__half2*>(p.x16 + (size_t)t * p.d + c) = h;
            }
            if (j == 0 && tid == 0) p.xf[t] = 1.0f / f;
            named_sync(1, CONS);
        }
    }

    // The rows of h of the 8-bit experts, in place: 8 fp32 numbers -> the two fp16 parts of h * f16_scale(largest), 8 high
    // parts, then 8 low ones.
    __device__ void convert_h() {
        const int nv = p.I / 8, rows = h_rows();
        for (int i = blockIdx.x * CONS + threadIdx.x; i < rows * nv; i += G * CONS) {
            const int row = i / nv;
            uint4* hi = reinterpret_cast<uint4*>(p.h + (size_t)row * p.Hs) + i % nv * 2;
            uint4* lo = hi + 1;
            const float f = f16_scale(__uint_as_float(__ldcg(p.hmax + row)));
            const uint4 a = __ldcg(hi), b = __ldcg(lo);
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t ow[2][4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float v0 = __uint_as_float(w[2 * q]) * f, v1 = __uint_as_float(w[2 * q + 1]) * f;
                const __half2 h = __floats2half2_rn(v0, v1);
                const float2 g = __half22float2(h);
                const float r0 = v0 - g.x, r1 = v1 - g.y;       // infinite or NaN: no low part
                const __half2 l = __floats2half2_rn(fabsf(r0) < INFINITY ? r0 : 0.f, fabsf(r1) < INFINITY ? r1 : 0.f);
                ow[0][q] = *reinterpret_cast<const uint32_t*>(&h);
                ow[1][q] = *reinterpret_cast<const uint32_t*>(&l);
            }
            __stcg(hi, make_uint4(ow[0][0], ow[0][1], ow[0][2], ow[0][3]));
            __stcg(lo, make_uint4(ow[1][0], ow[1][1], ow[1][2], ow[1][3]));
        }
    }

    __device__ __forceinline__ float gate_of(const Group& q, int tok) const {
        return q.shared ? 1.f : at<float>(L.gates)[q.row + __popc(q.mask & ((1u << tok) - 1u))];
    }

    // The fragment of a unit that this warp finishes, or -1: they go round the warps.
    __device__ __forceinline__ int my_frag(const Me& me, int turn) const {
        const int f = (me.warp - turn * FRAGS) & (CONS_WARPS - 1);
        return f < FRAGS ? f : -1;
    }

    // One buffer: the last unit's fragments have been read.
    __device__ __forceinline__ void before_put() const {
        if (red_buffers(FRAGS) == 1) named_sync(1, CONS);
    }

    template <int F>
    __device__ __forceinline__ void up(Me& me, const Group& q, float4* red) {
        if constexpr (F == W_F32) {
            float acc[NT * 8];
#pragma unroll
            for (int n = 0; n < NT * 8; ++n) acc[n] = 0.f;
            unit_f32<NT>(acc, me, p.d, q.mask);
            before_put();
            put_f32<NT>(red, acc, me);
        } else {
            float acc[R][NT * 4];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int j = 0; j < NT * 4; ++j) acc[i][j] = 0.f;
            unit_mma<FR, F, NT, 1, R>(acc, me, Stage<FR, R>::scales(p.T), p.d, q.mask);
            before_put();
            put_frag<NT, R>(red, acc, me);
        }
    }

    // Scales and biases of a unit's fragment, for the lane's row of w1 and of w3: loaded before the unit, and as
    // they are, since the first use would wait for them (and every warp of the block for this one).
    struct Fin {
        float s1, s3, x[2];                                     // x: what undoes the scale of the lane's tokens' rows
        T b1, b3;
    };
    __device__ __forceinline__ Fin fin_of(const Group& q, int r, int nt, int lane) const {
        Fin f;
        f.s1 = f.s3 = f.x[0] = f.x[1] = 1.f;
        f.b1 = f.b3 = from_f32<T>(0.f);
        const int I = q.shared ? p.Is : p.I;
        if (r >= I) return f;
        const FfnWeights& W = q.shared ? p.Sh : p.R;
        const size_t at_row = (size_t)q.e * I + r;
        if (FR == W_E4M3 && !q.shared) { f.s1 = W.s1[at_row]; f.s3 = W.s3[at_row]; }
        if (Q8 && !q.shared)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int tok = nt * 8 + (lane & 3) * 2 + i;
                if (tok < p.T) f.x[i] = __ldcg(p.xf + tok);
            }
        if (p.bias) { f.b1 = static_cast<const T*>(W.b1)[at_row]; f.b3 = static_cast<const T*>(W.b3)[at_row]; }
        return f;
    }

    // h of one unit's row r from the summed fragment (token group nt).
    __device__ __forceinline__ void finish_up(const Group& q, int r, const Fin& f, float4 c, int nt, int lane) {
        const bool in = r < (q.shared ? p.Is : p.I);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int tok = nt * 8 + (lane & 3) * 2 + i;
            const bool mine = in && ((q.mask >> tok) & 1u);
            float h = 0.f;
            if (mine) {
                // the weights' scale first: codes times scaled rows may lie beyond fp32's range of the result
                const float a = (i ? c.y : c.x) * f.s1 * f.x[i] + to_f32(f.b1), b = (i ? c.w : c.z) * f.s3 * f.x[i] + to_f32(f.b3);
                h = silu_f32(a) * b * gate_of(q, tok);
            }
            if (Q8 && !q.shared) {                              // 8 rows of a token: lanes 4 apart
                float m = fabsf(h) < INFINITY ? fabsf(h) : 0.f;
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
                if (lane < 4 && m > 0.f) atomicMax(p.hmax + q.row + __popc(q.mask & ((1u << tok) - 1u)), __float_as_uint(m));
            }
            if (!mine) continue;
            const size_t row = q.row + __popc(q.mask & ((1u << tok) - 1u));
            p.h[row * p.Hs + r] = h;
        }
    }

    using Acc = float[R][FR == W_F32 ? NT * 8 : NT * 4];

    // acc (put_frag's order, fp32: put_f32's) += gate * b2 of the group's expert, for the rows b2_of has loaded.
    struct B2 {
        T b[R][2];
    };
    __device__ __forceinline__ B2 b2_of(const Me& me, const Group& q, int cb) const {
        const void* b2 = q.shared ? p.Sh.b2 : p.R.b2;
        B2 o;
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r = cb * DOWN + (FR == W_F32 ? me.lane >> 1 : i * 16 + h * 8 + (me.lane >> 2));
                o.b[i][h] = from_f32<T>(0.f);
                if (r < p.d) o.b[i][h] = static_cast<const T*>(b2)[(size_t)q.e * p.d + r];
            }
        return o;
    }
    __device__ __forceinline__ void add_b2(Acc& acc, const Me& me, const Group& q, const B2& b) const {
        if constexpr (FR == W_F32) {
            if (me.lane & 1) return;
#pragma unroll
            for (int n = 0; n < NT * 8; ++n)
                if ((q.mask >> n) & 1u) acc[0][n] = fmaf(gate_of(q, n), to_f32(b.b[0][0]), acc[0][n]);
        } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = nt * 8 + (me.lane & 3) * 2 + j;
                    if (!((q.mask >> tok) & 1u)) continue;
                    const float gate = gate_of(q, tok);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int h = 0; h < 2; ++h) acc[i][nt * 4 + h * 2 + j] = fmaf(gate, to_f32(b.b[i][h]), acc[i][nt * 4 + h * 2 + j]);
                }
        }
    }

    template <int F>
    __device__ __forceinline__ void down(Acc& acc, Me& me, const Group& q, int cb) {
        const int K = q.shared ? p.Is : p.I;
        const bool b2 = p.bias && me.warp == q.row % CONS_WARPS;    // one warp's: loaded before the unit, added after it
        B2 b;
        if (b2) b = b2_of(me, q, cb);
        if constexpr (F == W_F32) {
            unit_f32<NT>(acc[0], me, K, q.mask);
        } else {
            // (Loads before the unit are used after it, so that no warp waits for them.)
            // A unit has its own sums: scales differ from expert to expert, and a weight that is infinite or NaN
            // must not reach the tokens that did not pick the expert (0 times it is NaN).
            float t[R][NT * 4], f[R][2];
            unsigned m[NT][2];
#pragma unroll
            for (int i = 0; i < R; ++i) {
#pragma unroll
                for (int j = 0; j < NT * 4; ++j) t[i][j] = 0.f;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int r = cb * DOWN + i * 16 + h * 8 + (me.lane >> 2);
                    f[i][h] = F == W_E4M3 && r < p.d ? p.R.s2[(size_t)q.e * p.d + r] : 1.f;
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = nt * 8 + (me.lane & 3) * 2 + j;
                    const int row = q.row + __popc(q.mask & ((1u << tok) - 1u));
                    m[nt][j] = 0u;
                    if (F != W_BF16 && ((q.mask >> tok) & 1u)) m[nt][j] = __ldcg(p.hmax + row);
                }
            if constexpr (F == W_BF16) {
                if constexpr (FR != W_BF16) {
                    const Called<FR, NT, R> o = unit_parts_called<FR, NT, R>(me, K, q.mask);
#pragma unroll
                    for (int i = 0; i < R; ++i)
#pragma unroll
                        for (int j = 0; j < NT * 4; ++j) t[i][j] = o.t[i][j];
                    me.ring.slot = o.slot;
                    me.ring.phase = o.phase;
                } else {
                    const int n = __popc(q.mask);
                    if (n <= 2) unit_parts<FR, NT, R, 2>(t, me, K, q.mask);
                    else if (n <= 8) unit_parts<FR, NT, R, 8>(t, me, K, q.mask);
                    else unit_parts<FR, NT, R, NT * 8>(t, me, K, q.mask);
                }
            } else {
                unit_mma<FR, F, NT, 2, R>(t, me, Stage<FR, R>::scales(p.T), K, q.mask);
            }
#pragma unroll
            for (int j = 0; j < NT * 4; ++j) {
                const int tok = j / 4 * 8 + (me.lane & 3) * 2 + (j & 1);
                if (!((q.mask >> tok) & 1u)) continue;
                const float x = F == W_BF16 ? 1.f : 1.0f / f16_scale(__uint_as_float(m[j / 4][j & 1]));
#pragma unroll
                for (int i = 0; i < R; ++i) acc[i][j] = fmaf(t[i][j] * f[i][(j >> 1) & 1], x, acc[i][j]);
            }
        }
        if (b2) add_b2(acc, me, q, b);
    }

    // A column block's sums of fragment f over the block's groups [u0, u1) of `groups`: to the output when they
    // are all, else to the partial sums; the block that completes the count adds those of all blocks in order.
    __device__ __forceinline__ void finish_down(float4 c, int cb, int u0, int u1, int groups, uint32_t U, int f, int lane) {
        if (u1 - u0 != groups) {
            const int first = cb * groups;                      // a block's first partial column block, or its last
            auto slot = [&](int b, bool starts) { return p.part + (((size_t)b * 2 + (starts ? 0 : 1)) * FRAGS + f) * 32 + lane; };
            __stcg(slot(blockIdx.x, down_start(U, blockIdx.x) >= first), c);
            __threadfence();
            __syncwarp();
            unsigned old = 0;
            if (lane == 0) old = atomicAdd(p.cnt + cb * FRAGS + f, (unsigned)(u1 - u0));
            old = __shfl_sync(0xffffffffu, old, 0);
            if (old + (unsigned)(u1 - u0) != (unsigned)groups) return;
            __threadfence();
            c = make_float4(0.f, 0.f, 0.f, 0.f);
            const int b1 = down_block(U, first + groups - 1);
            for (int b = down_block(U, first); b <= b1; ++b) {
                const int at = down_start(U, b);
                if (down_start(U, b + 1) == at) continue;
                const float4 v = __ldcg(slot(b, at >= first));
                c.x += v.x; c.y += v.y; c.z += v.z; c.w += v.w;
            }
        }
        const int nt = f % NT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int r = cb * DOWN + f / NT * 16 + (lane >> 2) + 8 * h;
            if (r >= p.d) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int tok = nt * 8 + (lane & 3) * 2 + j;
                if (tok < p.T) static_cast<T*>(p.out)[(size_t)tok * p.d + r] = from_f32<T>(h ? (j ? c.w : c.z) : (j ? c.y : c.x));
            }
        }
    }

    __device__ void consume() {
        Me me = {ring(), sm + L.ring, (int)(threadIdx.x >> 5), (int)(threadIdx.x & 31), abort_flag(), p.err};
        float4* red0 = at<float4>(L.red);
        const int cbs = ceil_div(p.d, DOWN);
        for (int i = blockIdx.x * CONS + threadIdx.x; i < cbs * FRAGS; i += G * CONS) p.cnt[i] = 0u;
        if (p.T == 1) scores<1>(reinterpret_cast<float*>(red0), me);
        else scores<4>(reinterpret_cast<float*>(red0), me);
        if (Q8) {
            for (int i = blockIdx.x * CONS + threadIdx.x; i < p.T * p.k; i += G * CONS) p.hmax[i] = 0u;
            convert_x(reinterpret_cast<float*>(red0), me);
        }
        named_sync(1, CONS);                                    // the block's scores are written
        if (threadIdx.x == 0) grid_arrive(p.bar);

        int turn = 0;
        auto buffer = [&] { return red0 + (turn & (red_buffers(FRAGS) - 1)) * CONS_WARPS * FRAGS * 32; };
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
                units = su + met * ceil_div(p.I, UP);
            }
            if (u >= units) break;
            Group q;
            int r0;
            up_unit(u, q, r0);
            const int f = my_frag(me, turn), r = r0 + f / NT * 8 + (me.lane >> 2);
            Fin fin = {};
            if (f >= 0) fin = fin_of(q, r, f % NT, me.lane);
            if (FR != FS && !q.shared) up<FR>(me, q, buffer());
            else up<FS>(me, q, buffer());
            named_sync(1, CONS);
            if (f >= 0 && !q.shared) mbar_wait(gate_bar(), 0, abort_flag(), p.err);
            if (f >= 0) finish_up(q, r, fin, take_frag<FRAGS>(buffer(), f, me.lane), f % NT, me.lane);
            ++turn;
        }
        // add_b2 reads the block's own gates, also in a block that had no routed unit to wait for them
        mbar_wait(gate_bar(), 0, abort_flag(), p.err);
        named_sync(1, CONS);                                    // the block's h is written
        if (threadIdx.x == 0) {
            grid_arrive(p.bar + 1);
            const bool all = grid_wait(p.bar + 1, at<unsigned long long>(L.turns)[1], abort_flag(), p.err);
            if (all && !Q8) mbar_arrive(h_bar());
        }
        named_sync(1, CONS);
        if (Q8) {
            convert_h();
            named_sync(1, CONS);
            if (threadIdx.x == 0) {
                grid_arrive(p.bar + 2);
                if (grid_wait(p.bar + 2, at<unsigned long long>(L.turns)[2], abort_flag(), p.err)) mbar_arrive(h_bar());
            }
            named_sync(1, CONS);
        }

        const int groups = p.Ks + met;
        if (groups == 0) {                                      // no shared expert, and no pick left
            for (size_t i = (size_t)blockIdx.x * CONS + threadIdx.x; i < (size_t)p.T * p.d; i += (size_t)G * CONS)
                static_cast<T*>(p.out)[i] = from_f32<T>(0.f);
            return;
        }
        const uint32_t U = (uint32_t)(cbs * groups);
        const int end = down_start(U, blockIdx.x + 1);
        for (int u = down_start(U, blockIdx.x); u < end;) {
            const int cb = u / groups, u0 = u, u1 = (cb + 1) * groups < end ? (cb + 1) * groups : end;
            Acc acc;
#pragma unroll
            for (auto& row : acc)
#pragma unroll
                for (float& a : row) a = 0.f;
            for (; u < u1; ++u) {
                const Group q = group(u % groups);
                if (FR != FS && !q.shared) down<FR>(acc, me, q, cb);
                else down<FS>(acc, me, q, cb);
            }
            before_put();
            if constexpr (FR == W_F32) put_f32<NT>(buffer(), acc[0], me);
            else put_frag<NT, R>(buffer(), acc, me);
            named_sync(1, CONS);
            const int f = my_frag(me, turn);
            if (f >= 0) finish_down(take_frag<FRAGS>(buffer(), f, me.lane), cb, u0, u1, groups, U, f, me.lane);
            ++turn;
        }
    }
};

template <int FR, int NT, int R>
__global__ void __launch_bounds__(THREADS, 1) few_kernel(const __grid_constant__ Params p) {
    extern __shared__ __align__(128) char sm[];
    Kernel<FR, NT, R> k(p, sm);
    if (threadIdx.x == 0) {
        const uint32_t bars = smem_u32(sm + k.L.bars);
        for (int s = 0; s < p.nst; ++s) {
            mbar_init(bars + s * 8, PRODUCERS * 32);            // every producer thread's copies
            mbar_init(bars + (MAX_STAGES + s) * 8, CONS_WARPS);
        }
        mbar_init(k.route_bar(), 1);
        mbar_init(k.h_bar(), 1);
        mbar_init(k.gate_bar(), 1);
        // this block has not arrived yet, so that the barriers' rounds cannot end before it has read them
        for (int i = 0; i < 3; ++i) k.template at<unsigned long long>(k.L.turns)[i] = round_end(load_acquire(p.bar + i), gridDim.x);
        int* misc = k.template at<int>(k.L.misc);
        misc[0] = misc[1] = misc[2] = misc[3] = misc[4] = 0;    // given up; experts met; scores complete; the consumers' view; rows
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
    if (warp < CONS_WARPS) k.consume();
    else if (warp < CONS_WARPS + PRODUCERS) k.produce(warp - CONS_WARPS);
    else k.rank();
}

size_t al256(size_t x) { return (x + 255) & ~(size_t)255; }
constexpr int GRID_MAX = 256, MAX_FRAGS = 4;

struct Layout {
    size_t logits, h, x16, xf, hmax, part, cnt, total;
    int Hs;
};
Layout few_layout(const Dims& D) {
    Layout L;
    const size_t T = D.T > 0 ? D.T : 1;
    const int widest = D.Ks > 0 && D.Is > D.I ? D.Is : D.I;
    L.Hs = (widest + 7) / 8 * 8;
    size_t o = 256;
    L.logits = o; o += al256(T * D.E * 4);
    L.h = o; o += al256(T * (D.k + D.Ks) * L.Hs * 4);
    L.x16 = o; o += D.q8 ? al256(T * D.d * 2) : 0;
    L.xf = o; o += D.q8 ? al256(T * 4) : 0;
    L.hmax = o; o += D.q8 ? al256(T * D.k * 4) : 0;
    L.part = o; o += al256((size_t)GRID_MAX * 2 * MAX_FRAGS * 32 * 16);
    L.cnt = o; o += al256((size_t)ceil_div(D.d, 16) * MAX_FRAGS * 4);
    L.total = o;
    return L;
}

template <int FR, int NT, int R>
cudaError_t launch(Params& p, int grid, cudaStream_t st) {
    const int rest = Smem(0, R * NT, p.T, p.E, p.k).total, rows = 16 * R * Fmt<FR, FR>::ROWB;
    p.stage = Stage<FR, R>::bytes(p.T);
    int n = (SMEM_LIMIT - rest) / p.stage;
    n = n > MAX_STAGES ? MAX_STAGES : n;
    p.nst = n * rows > RING_BYTES ? RING_BYTES / rows : n;
    if (p.nst < 2) return cudaErrorInvalidValue;                // a consumer holds one stage while it waits for the next
    const Smem L(p.nst * p.stage, R * NT, p.T, p.E, p.k);
    auto kern = few_kernel<FR, NT, R>;
    // The limit is the function's, for all host threads: always the same one, so that no thread lowers it between another's
    // setting and launch.
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_LIMIT);
    if (e != cudaSuccess) return e;
    void* args[] = {&p};
    return cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3(grid), dim3(THREADS), args, L.total, st);
}

// Two row tiles use every activation fragment twice and halve the barriers, and are faster than one even where
// they leave a block only a unit or two (one token, 64 experts of 320 x 1280: 15.6 us on the device instead of
// 16.6; 8 tokens: 35 instead of 44; 256 experts of 2048 x 7168: 135 instead of 152).  fp32 units stay at one.
template <int FR>
cudaError_t launch_t(Params& p, cudaStream_t st) {
    constexpr int R = FR == W_F32 ? 1 : 2;
    const int grid = num_sms() < GRID_MAX ? num_sms() : GRID_MAX;
    return p.T <= 8 ? launch<FR, 1, R>(p, grid, st) : launch<FR, 2, R>(p, grid, st);
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
    p.h = reinterpret_cast<float*>(w + L.h);
    p.x16 = reinterpret_cast<__half*>(w + L.x16);
    p.xf = reinterpret_cast<float*>(w + L.xf);
    p.hmax = reinterpret_cast<unsigned*>(w + L.hmax);
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
