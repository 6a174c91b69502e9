// topk.cuh -- the router's selection (a1) by one warp, shared by the routing
// kernels and the few-token layer kernel, so that both pick the same experts
// and weights bit for bit.
#pragma once

#include "common.cuh"

namespace moe {

constexpr unsigned kFullWarp = 0xffffffffu;

// Selection order as one 64-bit key, larger first: an order-preserving map of
// the logit (-0 folded onto +0; NaN below every number) in the high word and
// the complement of the expert index in the low word (equal logits: the lower
// index wins).  Key 0 marks an expert already taken or past E.
__device__ __forceinline__ uint64_t select_key(float f, int e) {
    uint32_t b = __float_as_uint(f);
    if (b == 0x80000000u) b = 0u;
    const uint32_t ord = isnan(f) ? 0u : ((b & 0x80000000u) ? ~b : (b | 0x80000000u));
    return (static_cast<uint64_t>(ord) << 32) | (0xffffffffu - static_cast<uint32_t>(e));
}

// The logit of a key (exact, except -0 reads as +0 and a NaN as the canonical
// NaN; neither changes exp(l - m)).
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t ord = static_cast<uint32_t>(key >> 32);
    if (ord == 0u) return __uint_as_float(0x7fffffffu);
    return __uint_as_float((ord & 0x80000000u) ? (ord & 0x7fffffffu) : ~ord);
}

// Top-k of row[0..E) by one warp (row in global or shared memory).  Each lane
// keys its E/32 logits once; a selection round is a local max of the lane's
// keys and two warp-wide reductions, after which the owning lane clears the
// winner.  The j-th selection (id and logit) is kept in registers of lane
// j % 32, slot j / 32; the weights are a softmax over the selected logits,
// summed per lane in ascending j and then across the warp.  ids and w are
// written once at the end, lane j for entry j.
template <int EPL>
__device__ void warp_topk(const float* row, int E, int k, int32_t* ids, float* w,
                          int32_t* ids_copy = nullptr) {
    const int lane = threadIdx.x & 31;
    uint64_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < E ? select_key(row[e], e) : 0ull;
    }
    float sv[EPL];
    int si[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        sv[i] = 0.0f;
        si[i] = 0;
    }
    float m = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint64_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = key[i] > best ? key[i] : best;
        // the largest logit of the warp, then the lowest index that has it
        // (a cleared key has a zero low word, every other one's is above 0)
        const uint32_t top = __reduce_max_sync(kFullWarp, static_cast<uint32_t>(best >> 32));
        const uint32_t low = static_cast<uint32_t>(best);
        const uint32_t pick = __reduce_max_sync(
            kFullWarp, static_cast<uint32_t>(best >> 32) == top ? low : 0u);
        best = (static_cast<uint64_t>(top) << 32) | pick;
        const int bi = static_cast<int>(0xffffffffu - pick);
        const float bv = key_value(best);
        // selects, not indexed stores, so the arrays stay in registers
        const bool won = (bi & 31) == lane, keep = (j & 31) == lane;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            key[i] = (won && i == (bi >> 5)) ? 0ull : key[i];
            const bool here = keep && i == (j >> 5);
            sv[i] = here ? bv : sv[i];
            si[i] = here ? bi : si[i];
        }
        if (j == 0) m = bv;
    }
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (lane + 32 * i < k) z += expf(sv[i] - m);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kFullWarp, z, off);
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int j = lane + 32 * i;
        if (j < k) {
            ids[j] = si[i];
            if (ids_copy) ids_copy[j] = si[i];
            w[j] = expf(sv[i] - m) / z;
        }
    }
    __syncwarp();
}

}  // namespace moe
