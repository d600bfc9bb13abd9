// Ranking of one token's router logits by one warp, for the CUDA-core router and the split-K router's last step.  (The
// few-token layer ranks by the same rules in a form of its own, made for latency.)
#pragma once

#include "common.cuh"

namespace moe {

// Picks and gates of one token by one warp from its E logits zr (shared memory, unchanged).
// The selection key is z + bias (gate modes 0 and 1) or sigmoid(z) + bias (mode 2); lane l owns
// experts l + 32 i and marks its picks in a bit mask.  k rounds of warp argmax on (key, -index)
// give the picks in descending key, equal keys to the lower index.  Gates: mode 0 the softmax of
// z + bias over all E experts read at the picks; mode 1 the softmax over the k picked keys;
// mode 2 sigmoid(z) at the picks divided by their sum.
__device__ __forceinline__ void warp_route(const float* zr, int E, int k, int mode, const float* __restrict__ bias, int lane,
                                           int32_t* idx_row, float* gate_row) {
    auto key_of = [&](int e) {
        const float z = zr[e];
        const float bb = bias ? bias[e] : 0.f;
        return mode == 2 ? 1.0f / (1.0f + expf(-z)) + bb : z + bb;
    };
    float m = -INFINITY, inv = 0.f;
    if (mode == 0) {
        for (int e = lane; e < E; e += 32) m = fmaxf(m, key_of(e));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        float s = 0.f;
        for (int e = lane; e < E; e += 32) s += expf(key_of(e) - m);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        inv = 1.0f / s;
    }
    uint32_t taken = 0;
    float first = 0.f, norm = 0.f;
    for (int j = 0; j < k; ++j) {
        float bv = -INFINITY;
        int bi = 0x7fffffff;
        for (int e = lane, i = 0; e < E; e += 32, ++i) {
            if (taken & (1u << i)) continue;
            const float v = key_of(e);
            if (v > bv) { bv = v; bi = e; }     // ascending e: equal keys keep the lower index
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ov = __shfl_xor_sync(0xffffffffu, bv, o);
            const int oi = __shfl_xor_sync(0xffffffffu, bi, o);
            if (ov > bv || (ov == bv && oi < bi)) { bv = ov; bi = oi; }
        }
        if (bi < E && (bi & 31) == lane) taken |= 1u << (bi >> 5);
        if (lane == 0) {
            idx_row[j] = bi;
            float g;
            if (mode == 0) {
                g = expf(bv - m) * inv;
            } else if (mode == 1) {
                if (j == 0) first = bv;
                g = expf(bv - first);
                norm += g;
            } else {
                g = 1.0f / (1.0f + expf(-zr[bi < E ? bi : 0]));     // no pick left (NaN or -inf keys): bi >= E
                norm += g;
            }
            gate_row[j] = g;
        }
        __syncwarp();
    }
    if (lane == 0 && mode != 0) {
        const float r = 1.0f / norm;
        for (int j = 0; j < k; ++j) gate_row[j] *= r;
    }
}

}  // namespace moe
