// decode.cu -- the whole MoE layer for a few tokens (T <= 16) in one kernel:
// routing, the experts' gate/up and down products, the weighted combine and
// the residual.
//
//   ids, w  = top-k of the token's logits, softmax over the selected ones
//   h       = SiLU(x W_g[e]) * (x W_u[e])
//   out[t]  = residual[t] + sum_j w(t, j) * (h W_d[e])
//
// What bounds it is the stream of the active experts' packed weights, each
// read once; everything around the stream is latency.  One cooperative grid,
// one CTA per SM, runs the layer in three steps with two grid barriers:
//
//   1 every CTA routes the T tokens itself (the logits are a few KB), then the
//     gate/up tiles of all active experts, in (expert, row tile, k-block)
//     order, are cut into equal contiguous ranges, one per CTA.  A range ends
//     inside a row tile, so each CTA writes fp32 partial sums.
//   2 the down tiles in (expert, k-block, row tile) order are cut the same way.
//     A CTA then needs only the few k-blocks of h that its range covers: it
//     sums their partials, applies SiLU * up once, and keeps h in shared
//     memory.  (With the row tile outermost every CTA would need all of h.)
//     It writes fp32 partial sums of the output rows.
//   3 the partial sums of every output are added in a fixed order, with the
//     routing weights, over all CTAs, the residual added and rounded once.
//
// The weights arrive as 16 KB tiles (the packed layout of the grouped GEMMs)
// through a ring of bulk copies that one thread keeps full across the barriers:
// while the CTAs exchange partial sums the first down tiles land.  The products
// are m16n8k16 warp MMAs: at these sizes the tensor work is a fifth of the
// stream's time, and the register path lets the operands be widened.  bf16
// layers: tokens in M (16 at most), weight rows in N, and h as the sum of two
// bf16 values (16 bits), the low parts in the MMA's upper 8 rows while an expert
// has at most 8 tokens.  e4m3 layers: weights and x to f16, both exact, h to
// f16's 11 bits; nothing is quantised.  The only coarse rounding is out's.
//
// One tile is a chain of some 500 cycles of latency (barrier, loads, products),
// so four groups of four warps take the tiles in turn, 32 weight rows a warp;
// with all sixteen warps on each tile the stream stayed at 5.8 TB/s and every
// down tile of a small layer took 1000 cycles.
//
// Measured on one B200 (us; floor = the active experts' bytes at the copy's 6.53
// TB/s; then moe_forward on the same inputs, whose chain of kernels costs 6
// to 15 us more than this one's start and end, but whose tcgen05 stream is the
// faster one):
//   bf16 E=128 H=2048 I=768 top-8     T = 1: 27 (12; 40)      T = 8: 86 (74; 98)     T = 16: 130 (120; 142)
//   bf16 E=8 H=4096 I=14336 top-2     T = 1: 116 (108; 124)   T = 8: 375-405 (377; 360-377)
//   bf16 E=64 H=7168 I=2048 top-8     T = 1: 119 (108; 125)   T = 2: 204 (198; 205)  T = 8: 582-625 (578; 546-559)
//   e4m3 E=32 H=I=2880 top-4          T = 1: 31 (15; 46)      T = 8: 102 (81; 111)   T = 13: 131 (102; 133)
//                                     T = 16: 141 (109; 141)
// 18 warps leave 96 registers a thread: 20 to 152 bytes of spills by form, most
// where an expert may have more than 8 tokens.
// Where T = 1's 27 us go (the first of them): 3.2 us routing and tables in
// every CTA, 1.7 to the first tile, 7.4 of gate/up stream (9.6 in the last CTA),
// 1.7 for the first barrier under the down tiles' prefetch, 4.6 of h and down
// products, 1.2 for the second barrier, 2.3 of final sums, 2.5 between launches.
//
// All sums are in a fixed order: results do not depend on timing.
#include <cstdint>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "topk.cuh"

namespace moe {

namespace {

constexpr int kGroups = 4;
constexpr int kGroupWarps = 4;          // 32 weight rows of a tile each
constexpr int kConsumerWarps = kGroups * kGroupWarps;
constexpr int kConsumers = kConsumerWarps * 32;
// ... a warp that copies the weight tiles and one that copies the gate/up tiles'
// x slices (together the copies took longer than a tile's time)
constexpr int kWeightWarp = kConsumerWarps, kXWarp = kConsumerWarps + 1;
constexpr int kThreads = (kConsumerWarps + 2) * 32;
constexpr int kBarThread = 32;          // a consumer that stands at the grid barriers
constexpr int kMaxSlots = 12;           // a multiple of the groups: a slot stays with one
constexpr int kSmemBytes = 227 * 1024;
constexpr uint32_t kMagic = 0x4d6f4465u;

// h columns held at a time: 512 (8 k-blocks of bf16 tiles, 4 of e4m3 tiles)
template <bool FP8> __host__ __device__ constexpr int tile_k() { return FP8 ? 128 : 64; }
template <bool FP8> __host__ __device__ constexpr int chunk_kb() { return FP8 ? 4 : 8; }
// bytes of one token's row of a k-block of h (bf16: hi | lo; f16 for e4m3),
// plus 16 so that two rows start an odd number of 16-byte banks apart
template <bool FP8> __host__ __device__ constexpr int h_row_bytes() {
    return tile_k<FP8>() * (FP8 ? 2 : 4) + 16;
}
// a token's x of one gate/up tile, padded likewise, and a ring slot: a weight
// tile and the x slices of the tokens
template <bool FP8> __host__ __device__ constexpr int x_row_bytes() { return tile_k<FP8>() * 2 + 16; }
template <bool FP8> __host__ __device__ constexpr int slot_bytes(int rows) {
    return kTileBytes + rows * x_row_bytes<FP8>();
}
// the h buffer, before it the groups' exchange of gate/up sums [group][rows][128]
template <bool FP8> __host__ __device__ constexpr int h_bytes(int rows) {
    const int h = chunk_kb<FP8>() * rows * h_row_bytes<FP8>(), x = kGroups * rows * kTileRows * 4;
    return h > x ? h : x;
}
// slots beside it, a multiple of the groups (8 at 16 rows, 12 up to about 5);
// `rows` is the most tokens that one expert has, known after the routing
template <bool FP8> __host__ __device__ constexpr int slots_for(int rows, int smem) {
    const int n = (smem - h_bytes<FP8>(rows)) / slot_bytes<FP8>(rows) / kGroups * kGroups;
    return n < kMaxSlots ? n : kMaxSlots;
}

// Workspace header, made by moe_decode_workspace_init.
// The arrival counters only grow, by one per CTA and launch, so each launch
// finds them at a multiple of the grid (and they stay below the next one until
// its own CTA arrives), and no launch has to reset them.
struct Header {
    int32_t status;
    uint32_t magic;
    uint64_t pad0[7];
    uint64_t arrive[2][8];      // one 64-byte line per barrier
};

// Division of tile numbers (up to kDecodeMaxTiles = 2^24, so exact as floats) by
// a divisor known at the launch: the product with its reciprocal is off by less
// than one.  A third of the latency of an integer division, of which the way to
// the first tile and the way from a barrier to the next products have several.
struct Divisor {
    int d;
    float inv;
};
__host__ __device__ __forceinline__ int operator/(int x, const Divisor& v) {
    const int q = static_cast<int>(static_cast<float>(x) * v.inv), r = x - q * v.d;
    return q + (r >= v.d ? 1 : 0) - (r < 0 ? 1 : 0);
}
Divisor divisor(int d) { return Divisor{d, 1.0f / static_cast<float>(d)}; }

struct Args : SelfTest {
    int T, k, E, H, I;
    int mt_gu, kb_gu, mt_dn, kb_dn;
    Divisor by_mt_gu, by_kb_gu, by_mt_dn, by_S1, by_S2, by_G, by_hquads;
    const uint8_t* w_gu;
    const uint8_t* w_dn;
    const float* scales;         // [E][3], e4m3
    const __nv_bfloat16* x;
    const float* logits;
    const __nv_bfloat16* residual;
    __nv_bfloat16* out;
    int32_t* ids;
    float* w;
    int32_t* status;
    Header* hdr;
    float* p1;                   // gate/up partial columns of 128 rows
    float* p2;                   // down partial columns of 128 rows
    int smem;                    // dynamic shared memory past its alignment
};

// One chunk's share of a batch's h: the active expert, the first column of h, the
// first k-block of the h buffer, the first quad of the batch and the quads per
// token.
struct Piece {
    int i, col, slot, quad;
    Divisor quads;
};

struct Shared {
    uint64_t full[kMaxSlots];
    uint64_t empty[kMaxSlots];
    int abort;
    int ids[kDecodeMaxAssign];          // [T][k]
    float w[kDecodeMaxAssign];
    uint32_t mask[kMaxExperts];         // tokens that chose an expert
    int rank[kMaxExperts];              // index among the active experts
    int scan[kMaxExperts / 32];
    int most[kMaxExperts / 32];
    int expert[kDecodeMaxAssign];       // active experts, ascending
    int base[kDecodeMaxAssign + 1];     // first column of an active expert
    int tok[kDecodeMaxAssign];          // column -> token
    // an assignment's terms of the final sums: the first CTA with down tiles of
    // its expert and how many there are, the column of its first partial sum,
    // the expert's token count; the expert's first down tile, and the weight
    // (with e4m3's down scale)
    int4 term[kDecodeMaxAssign];
    int term_tile[kDecodeMaxAssign];
    float term_w[kDecodeMaxAssign];
    int start1[kMaxCtas + 1];           // first gate/up tile of each CTA
    int start2[kMaxCtas + 1];           // first down tile of each CTA
    int mod2[kMaxCtas];                 // its row tile
    uint32_t xmax[kDecodeMaxT];         // e4m3: a token's largest finite |x|
    float xmul[kDecodeMaxT];            // ... and its power-of-two scale
    uint32_t hmax[8][kDecodeMaxT];      // e4m3: largest |h| of a chunk's column
    Piece pieces[9];                    // of a batch, and the end
    int n_pieces;
};

__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kConsumers) : "memory");
}

__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n)
                 : "memory");
}

// The four warps of a group.
__device__ __forceinline__ void group_sync(int grp) {
    asm volatile("bar.sync %0, %1;" ::"r"(2 + grp), "n"(kGroupWarps * 32) : "memory");
}

__device__ __forceinline__ uint4 lds16(const uint8_t* p) {
    return *reinterpret_cast<const uint4*>(p);
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two pairs of f16 values: exact, NaN stays NaN.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t v, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(v));
}

__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// e4m3 layers multiply in f16, whose 11 bits hold every e4m3 and bf16 mantissa;
// its range is met by a power of two per token that brings the largest finite
// magnitude (`bits`) to [2^14, 2^15).  What that pushes below f16's normal
// range is off by 2^-25 there, 2^-39 of the largest: less than an fp32 ulp of
// the sums it enters.  scale_inv is the exact reciprocal.
__device__ __forceinline__ float f16_scale(uint32_t bits) {
    int e = 268 - static_cast<int>(bits >> 23);     // 127 + 14 - (exponent - 127)
    e = bits == 0 ? 127 : (e > 253 ? 253 : e);
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}
__device__ __forceinline__ float scale_inv(float s) {
    return __uint_as_float((254u << 23) - __float_as_uint(s));
}
// The down sums of e4m3 layers lack the matrix' scale (its largest weight / 448)
// until the end: this power of two in its place keeps them finite where out is.
constexpr float kSumScale = 1.0f / 16384.0f;
__device__ __forceinline__ uint32_t finite_mag(float v) {
    const uint32_t m = __float_as_uint(v) & 0x7fffffffu;
    return m < 0x7f800000u ? m : 0u;
}

// The CTA whose range of tiles holds tile X.
__device__ __forceinline__ int owner(const int* start, int G, int X, float tiles_per_cta_inv) {
    int c = static_cast<int>(static_cast<float>(X) * tiles_per_cta_inv);
    c = c < 0 ? 0 : (c > G - 1 ? G - 1 : c);
    while (start[c] > X) --c;
    while (start[c + 1] <= X) ++c;
    return c;
}

__device__ __forceinline__ void fault(Shared& s, int32_t* status) {
    report(status, MOE_ERR_TIMEOUT);
    *reinterpret_cast<volatile int*>(&s.abort) = 1;
}

// The bounded wait of this kernel's rings: the timer is read only now and then
// (a read takes longer than a tile's products).
__device__ __forceinline__ bool ring_wait(const Args& g, uint64_t* bar, uint32_t parity,
                                          volatile int* abort) {
    uint64_t t0 = 0;
    for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
        if ((i & 31u) != 31u) continue;
        if (*abort) return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0) t0 = now;
        else if (now - t0 > g.wait_limit()) return false;
    }
    return true;
}

// Arrival of this CTA at a grid barrier and the bounded wait until the counter
// reaches `target`.  Called by one thread, between two consumer_sync.
__device__ __forceinline__ bool grid_barrier(const Args& g, uint64_t* counter, uint64_t target) {
    asm volatile("fence.acq_rel.gpu;\n\tred.release.gpu.global.add.u64 [%0], 1;" ::"l"(counter)
                 : "memory");
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        uint64_t v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(counter) : "memory");
        if (v >= target) return true;
        if (globaltimer_ns() - t0 > g.wait_limit()) return false;
    }
}

// One lane's part of a tile: 32 weight rows of this warp by 16 tokens.  The K
// order inside a 128-byte row is permuted the same way for both operands: lane
// (g, t) takes 16-byte pieces 2t and 2t+1 of weight row g of each block of 8,
// whose swizzled places are conflict-free for a quarter warp, and the matching
// 32 (bf16) or 64 (f16, for 32 e4m3 codes) bytes of token rows g and g + 8.
struct Wts {
    uint4 v[4][2];
};
__device__ __forceinline__ void load_w(Wts& w, const uint8_t* rows, int g, int t) {
    const uint8_t* r = rows + g * kTileRowBytes;
    const int p0 = ((2 * t) ^ g) * 16, p1 = ((2 * t + 1) ^ g) * 16;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        w.v[b][0] = lds16(r + b * 8 * kTileRowBytes + p0);
        w.v[b][1] = lds16(r + b * 8 * kTileRowBytes + p1);
    }
}

// Token rows.  A lane whose row is past the expert's count reads row 0 with the
// lanes that own it (one broadcast); what it gives is never looked at.
template <bool FP8> struct Act {
    uint4 v[FP8 ? 4 : 2];
};
template <bool FP8>
__device__ __forceinline__ Act<FP8> load_act(const uint8_t* row, int t) {
    constexpr int N = FP8 ? 4 : 2;
    Act<FP8> a;
#pragma unroll
    for (int q = 0; q < N; ++q) a.v[q] = lds16(row + t * (N * 16) + q * 16);
    return a;
}

// bf16: D[16 tokens][32 weight rows of this warp] += act x W, four blocks of 8
// weight rows in N; a: token rows g, b: token rows g + 8 (or h's low parts).
__device__ __forceinline__ void tile_mma(float (&acc)[4][4], const Wts& w, const Act<false>& a,
                                         const Act<false>& b) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int n = 0; n < 4; ++n)
            mma_bf16(acc[n], a.v[p].x, b.v[p].x, a.v[p].y, b.v[p].y, w.v[n][p].x, w.v[n][p].y);
#pragma unroll
        for (int n = 0; n < 4; ++n)
            mma_bf16(acc[n], a.v[p].z, b.v[p].z, a.v[p].w, b.v[p].w, w.v[n][p].z, w.v[n][p].w);
    }
}

// e4m3: D[32 weight rows][8 tokens] += W x act, two blocks of 16 weight rows in M
// (the widened codes land in the registers that M wants), 8 tokens in N; acc[b]
// for tokens 0..7, acc[2 + b] for 8..15 (BOTH).  Word q of 4 codes meets 8 bytes
// of the token rows.
template <bool BOTH>
__device__ __forceinline__ void tile_mma(float (&acc)[4][4], const Wts& w, const Act<true>& a,
                                         const Act<true>& b) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const uint4 x = a.v[q >> 1], y = b.v[q >> 1];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const uint4 c0 = w.v[2 * m][q >> 2], c1 = w.v[2 * m + 1][q >> 2];
            uint32_t f0, f1, f2, f3;
            e4m3x4_to_f16x4((q & 3) == 0 ? c0.x : (q & 3) == 1 ? c0.y : (q & 3) == 2 ? c0.z : c0.w,
                            f0, f2);
            e4m3x4_to_f16x4((q & 3) == 0 ? c1.x : (q & 3) == 1 ? c1.y : (q & 3) == 2 ? c1.z : c1.w,
                            f1, f3);
            mma_f16(acc[m], f0, f1, f2, f3, (q & 1) ? x.z : x.x, (q & 1) ? x.w : x.y);
            if constexpr (BOTH)
                mma_f16(acc[2 + m], f0, f1, f2, f3, (q & 1) ? y.z : y.x, (q & 1) ? y.w : y.y);
        }
    }
}

// A lane's sums by (token, weight row of the warp's 32): calls f(token, row, v0,
// v1), bf16 with two weight rows (row, row + 1), e4m3 with one (v0).
template <bool FP8, bool MANY, class F>
__device__ __forceinline__ void each_sum(const float (&acc)[4][4], int g, int t, F f) {
    if constexpr (!FP8) {
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            f(g, 8 * n + 2 * t, acc[n][0], acc[n][1]);
            if (MANY) f(g + 8, 8 * n + 2 * t, acc[n][2], acc[n][3]);
        }
    } else {
#pragma unroll
        for (int n = 0; n < (MANY ? 4 : 2); ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f(8 * (n >> 1) + 2 * t + (i & 1), 16 * (n & 1) + g + 8 * (i >> 1), acc[n][i], 0.0f);
    }
}

// Few enough keys for one pass of the threads.
__device__ __forceinline__ bool routes_by_counting(const Args& g) {
    return g.T * ((g.E + 31) & ~31) <= kConsumers;
}

// Routing of all tokens by the consumer warps.  A few tokens' keys are ranked by
// counting: an expert's place is the number of keys above its own (keys are
// distinct), `parts` threads to a key; s.w gets the selected logits, and
// softmax_tokens makes them weights later, off the way to the first tiles.  The
// same order and the same sums as warp_topk, which takes larger batches a warp
// per token: ids and weights are its bits either way.
__device__ __forceinline__ void softmax_tokens(const Args& g, Shared& s, int warp, int lane) {
    for (int t = warp; t < g.T; t += kConsumerWarps) {
        float* w = s.w + t * g.k;
        const float m = w[0];
        __syncwarp();
        float z = 0.0f;
        for (int j = lane; j < g.k; j += 32) {
            const float v = expf(w[j] - m);
            w[j] = v;
            z += v;
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(kFullWarp, z, off);
        for (int j = lane; j < g.k; j += 32) w[j] = w[j] / z;
    }
}

template <bool FP8>
__device__ __forceinline__ void route_tokens(const Args& g, Shared& s, uint64_t* keys, int warp,
                                             int lane) {
    const int Ep = (g.E + 31) & ~31, n = g.T * Ep;
    const bool counting = routes_by_counting(g);
    if (counting && threadIdx.x < n) {
        const int t = threadIdx.x / Ep, e = threadIdx.x - t * Ep;
        keys[threadIdx.x] = e < g.E ? select_key(__ldg(g.logits + t * g.E + e), e) : 0ull;
    }
    if constexpr (FP8) {
        // each token's largest |x|, from the last warp down; a few tokens have
        // several warps each
        const int p2 = g.T == 1 ? 3 : g.T == 2 ? 2 : g.T <= 4 ? 1 : 0;
        const int u = kConsumerWarps - 1 - warp, tk = u >> p2, part = u & ((1 << p2) - 1);
        if (tk < g.T) {
            const uint4* xr = reinterpret_cast<const uint4*>(g.x + static_cast<size_t>(tk) * g.H);
            uint32_t m = 0;
#pragma unroll 8
            for (int v = part * 32 + lane; v < g.H / 8; v += 32 << p2) {
                const uint4 q = __ldg(xr + v);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    m = max(m, max(finite_mag(bf16_lo(w[j])), finite_mag(bf16_hi(w[j]))));
            }
            m = __reduce_max_sync(kFullWarp, m);
            if (lane == 0) atomicMax(&s.xmax[tk], m);
        }
    }
    if (!counting) {
        for (int t = warp; t < g.T; t += kConsumerWarps) {
            const float* row = g.logits + t * g.E;
            int* ids = s.ids + t * g.k;
            float* w = s.w + t * g.k;
            if (g.E <= 32) warp_topk<1>(row, g.E, g.k, ids, w);
            else if (g.E <= 128) warp_topk<4>(row, g.E, g.k, ids, w);
            else warp_topk<8>(row, g.E, g.k, ids, w);
            for (int j = lane; j < g.k; j += 32) atomicOr(&s.mask[ids[j]], 1u << t);
        }
        return;
    }
    consumer_sync();
    int parts = 1;
    while (parts < 16 && n * parts * 2 <= kConsumers) parts *= 2;
    {
        const int f = threadIdx.x / parts, part = threadIdx.x & (parts - 1);
        if (f < n) {                      // whole warps: n * parts is a multiple of 32
            const int t = f / Ep, e = f - t * Ep;
            const uint64_t own = keys[f];
            int place = 0;
            const ulonglong2* pairs = reinterpret_cast<const ulonglong2*>(keys + t * Ep);
#pragma unroll 4
            for (int i = part; i < Ep / 2; i += parts) {
                const ulonglong2 two = pairs[i];
                place += (two.x > own) + (two.y > own);
            }
            for (int off = 1; off < parts; off *= 2)
                place += __shfl_xor_sync(kFullWarp, place, off);
            if (part == 0 && e < g.E && place < g.k) {
                s.ids[t * g.k + place] = e;
                s.w[t * g.k + place] = key_value(own);
                atomicOr(&s.mask[e], 1u << t);
            }
        }
    }
    fence_proxy_async_smem();   // the ring's copies come after the keys
}

// Ring position shared by the copying and the product warps' loops.  The n-th
// tile of a CTA is in slot n % slots and belongs to group n % 4; a group only
// ever sees its own slots (slots is a multiple of 4), each use of them in turn.
struct Ring {
    int slot;
    uint32_t phase = 0;
    int slots;
    __device__ __forceinline__ explicit Ring(int n, int first = 0) : slot(first), slots(n) {}
    __device__ __forceinline__ void skip(int n) {       // n <= slots
        slot += n;
        if (slot >= slots) {
            slot -= slots;
            phase ^= 1u;
        }
    }
};

// A CTA's down tiles of one expert are a range of kb * MT + m, taken by chunks of
// whole k-blocks (the first and last may be partial): [a, b).  Within a chunk a
// row tile is visited once, for all its k-blocks: visit v takes tiles a + v,
// a + v + MT, ... below b.  Four visits at a time, one per group, their tiles
// interleaved in the ring; where a visit of the four has a tile less than the
// first, or there is no fourth visit, the place stays empty but is passed on.
struct Chunk {
    int i;               // active expert
    int a, b, kb0, kb1;  // tiles, k-blocks
    int kb, m, visits;   // the first visit's k-block and row tile, the visits
    int slot;            // the k-block of the h buffer where the chunk's begin
    bool first;          // of the expert's chunks in this CTA
};

// The chunks of a CTA in order, in batches that share the h buffer (CK
// k-blocks): as many whole experts' ranges as fit, or CK k-blocks of one.
struct Plan {
    int X, end, a2, CK, left;
    Divisor S2, MT;
    __device__ __forceinline__ Plan(int from, int to, const Args& g, int CK_)
        : X(from), end(to), a2(from), CK(CK_), left(CK_), S2(g.by_S2), MT(g.by_mt_dn) {}
    __device__ __forceinline__ bool done() const { return X >= end; }
    __device__ __forceinline__ void batch() { left = CK; }
    __device__ __forceinline__ bool take(Chunk& c) {
        if (X >= end) return false;
        c.i = X / S2;
        const int base = c.i * S2.d, to = min(end - base, S2.d);
        c.a = X - base;
        c.kb0 = c.a / MT;
        c.kb1 = (to - 1) / MT + 1;
        if (c.kb1 - c.kb0 > left) {
            if (left < CK) return false;
            c.kb1 = c.kb0 + CK;
        }
        c.b = min(c.kb1 * MT.d, to);
        c.kb = c.kb0;
        c.m = c.a - c.kb0 * MT.d;
        c.visits = min(c.b - c.a, MT.d);
        c.slot = CK - left;
        c.first = X == a2 || c.a == 0;
        left -= c.kb1 - c.kb0;
        X = base + c.b;
        return true;
    }
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
}

// Stores one (e4m3) or two sums, or adds to what this CTA stored for an earlier
// chunk of the expert: another group's warp may have, before the consumer_sync
// that ends each batch.
template <bool FP8>
__device__ __forceinline__ void put(float* d, float v0, float v1, bool first) {
    if constexpr (FP8) {
        __stcg(d, first ? v0 : __ldcg(d) + v0);
    } else {
        float2* p = reinterpret_cast<float2*>(d);
        if (!first) {
            const float2 o = __ldcg(p);
            v0 += o.x;
            v1 += o.y;
        }
        __stcg(p, make_float2(v0, v1));
    }
}

// What h's first bf16 value leaves for the second: 16 bits of mantissa
// together.  An infinite or NaN h is all in the first.
__device__ __forceinline__ float rest(float h, float hi) {
    return fabsf(h) < 3.0e38f ? h - hi : 0.0f;
}

// h of column c of active expert i, columns hc..hc+3: the gate/up partial sums
// of all CTAs that hold tiles of the row tile, in ascending order.
__device__ __forceinline__ float4 h_quad(const Args& g, const Shared& s, int i, int c0, int cnt,
                                         int c, int hc, int G1, float per1, float sg, float su) {
    const int m = hc >> 6, l = hc & 63;
    const int row = 32 * (l >> 4) + (l & 15);
    const int X0 = (i * g.mt_gu + m) * g.kb_gu;
    const int cf = owner(s.start1, G1, X0, per1);
    const float* q = g.p1 + ((static_cast<size_t>(c0) * g.mt_gu + m * cnt +
                              static_cast<size_t>(cf) * g.T) + c) * kTileRows + row;
    const size_t step = static_cast<size_t>(g.T) * kTileRows;
    float4 gt = make_float4(0.f, 0.f, 0.f, 0.f), up = gt;
    for (int cc = cf;; ++cc, q += step) {
        const float4 g0 = __ldcg(reinterpret_cast<const float4*>(q));
        const float4 u0 = __ldcg(reinterpret_cast<const float4*>(q + 16));
        gt.x += g0.x;
        gt.y += g0.y;
        gt.z += g0.z;
        gt.w += g0.w;
        up.x += u0.x;
        up.y += u0.y;
        up.z += u0.z;
        up.w += u0.w;
        if (s.start1[cc + 1] >= X0 + g.kb_gu) break;
    }
    auto act = [&](float a, float b) {
        return silu(a * sg) * (b * su);   // silu: ~1e-6, far below out's rounding
    };
    return make_float4(act(gt.x, up.x), act(gt.y, up.y), act(gt.z, up.z), act(gt.w, up.w));
}

// What the routing leaves for the three steps.
struct Run {
    uint8_t* smem;           // the ring
    uint8_t* hbuf;
    int rows, slots, slot_sz;
    int S1, S2, L1, L2, G1, G2;   // tiles per expert, in all; CTAs with tiles
    uint64_t seen[2];        // (kBarThread) the grid barriers' counters
};

// The three steps.  MANY: an expert has more than 8 tokens.
template <bool FP8, bool MANY>
__device__ __forceinline__ void run_steps(const Args& g, Shared& s, const Run& r_) {
    constexpr int BK = tile_k<FP8>();
    constexpr int CK = chunk_kb<FP8>();
    uint8_t* const smem = r_.smem;
    uint8_t* const hbuf = r_.hbuf;
    const int rows = r_.rows, slots = r_.slots, slot_sz = r_.slot_sz;
    const int S1 = r_.S1, S2 = r_.S2, L1 = r_.L1, L2 = r_.L2, G1 = r_.G1, G2 = r_.G2;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = gridDim.x, cta = blockIdx.x;
    const int a1 = s.start1[cta], b1 = s.start1[cta + 1];
    const int a2 = s.start2[cta], b2 = s.start2[cta + 1];

    if (warp == kWeightWarp) {
        // ---- one thread keeps the ring full of weight tiles through both
        // products
        Ring ring(slots);
        int it = 0;
        bool ok = true;
        bool withheld = false;
        for (int X = a1; lane == 0 && X < b1 && ok && !withheld;) {
            const int i = X / g.by_S1, end = (i + 1) * S1 < b1 ? (i + 1) * S1 : b1;
            const uint8_t* w =
                g.w_gu + (static_cast<size_t>(s.expert[i]) * S1 + (X - i * S1)) * kTileBytes;
            for (; X < end; ++X, w += kTileBytes) {
                if (g.withheld(cta, it)) {
                    withheld = true;
                    break;
                }
                if (it >= slots && !ring_wait(g, &s.empty[ring.slot], ring.phase ^ 1u, &s.abort)) {
                    ok = false;
                    break;
                }
                mbar_arrive_expect_tx(&s.full[ring.slot], kTileBytes);
                bulk_load(smem + ring.slot * slot_sz, w, kTileBytes, &s.full[ring.slot],
                          kEvictFirst);
                ring.skip(1);
                ++it;
            }
        }
        Plan plan(a2, b2, g, CK);
        Chunk ch;
        while (lane == 0 && ok && !withheld && !plan.done()) {
            plan.batch();
            while (ok && !withheld && plan.take(ch)) {
                const uint8_t* w = g.w_dn + static_cast<size_t>(s.expert[ch.i]) * S2 * kTileBytes;
                int m0 = ch.m, kb0 = ch.kb;                    // of visit v0
                for (int v0 = 0; v0 < ch.visits && ok && !withheld; v0 += kGroups) {
                    for (int L = ch.a + v0, d = 0; L < ch.b && ok && !withheld;
                         L += g.mt_dn, ++d) {
                        int m = m0, kb = kb0 + d;
                        for (int q = 0; q < kGroups; ++q) {
                            if (g.withheld(cta, it)) {
                                withheld = true;
                                break;
                            }
                            if (it >= slots &&
                                !ring_wait(g, &s.empty[ring.slot], ring.phase ^ 1u, &s.abort)) {
                                ok = false;
                                break;
                            }
                            if (v0 + q < ch.visits && L + q < ch.b) {
                                mbar_arrive_expect_tx(&s.full[ring.slot], kTileBytes);
                                mbar_arrive_n(&s.full[ring.slot], 32);   // (no x slice)
                                bulk_load(smem + ring.slot * slot_sz,
                                          w + (static_cast<size_t>(m) * g.kb_dn + kb) * kTileBytes,
                                          kTileBytes, &s.full[ring.slot], kEvictFirst);
                            } else {
                                mbar_arrive_n(&s.full[ring.slot], 33);
                            }
                            if (++m == g.mt_dn) {
                                m = 0;
                                ++kb;
                            }
                            ring.skip(1);
                            ++it;
                        }
                    }
                    for (m0 += kGroups; m0 >= g.mt_dn; m0 -= g.mt_dn) ++kb0;
                }
            }
        }
        if (!ok) fault(s, g.status);
        // this CTA's copies in flight (of the last `slots` tiles, or fewer) land
        // before its shared memory goes, also where a product warp gave up
        for (int j = it > slots ? it - slots : 0; j < it; ++j)
            mbar_wait(&s.full[j % slots], (j / slots) & 1u, nullptr, 10000000ull);
    } else if (warp == kXWarp) {
        // ---- the x slices of the gate/up tiles, in 16-byte pieces, one per lane
        // and turn (as bulk copies of a few hundred bytes each they kept the copy
        // engine from the weights)
        Ring ring(slots);
        int it = 0;
        constexpr int PIECES = BK / 8;                 // of a token's slice
        const int q = lane % PIECES;
        for (int X = a1; X < b1;) {
            const int i = X / g.by_S1, end = (i + 1) * S1 < b1 ? (i + 1) * S1 : b1;
            const int c0 = s.base[i], cnt = s.base[i + 1] - c0;
            int kb = X - X / g.by_kb_gu * g.kb_gu;
            for (; X < end; ++X) {
                if (it >= slots && !ring_wait(g, &s.empty[ring.slot], ring.phase ^ 1u, &s.abort)) {
                    fault(s, g.status);
                    cp_async_wait_all();
                    return;         // (a flag to leave the loops took 1% of the stream)
                }
                const uint32_t dst = smem_u32(smem + ring.slot * slot_sz + kTileBytes) + q * 16;
                // (the last e4m3 k-block may hold 64 of its 128 columns: the rest
                // is filled with zeros)
                const int col = kb * BK + q * 8;
                const bool in = col < g.H;
                for (int c = lane / PIECES; c < cnt; c += 32 / PIECES)
                    cp_async16(dst + c * x_row_bytes<FP8>(),
                               g.x + static_cast<size_t>(s.tok[c0 + c]) * g.H + (in ? col : 0),
                               in ? 16 : 0);
                cp_async_arrive_noinc(&s.full[ring.slot]);
                if (++kb == g.kb_gu) kb = 0;
                ring.skip(1);
                ++it;
            }
        }
        cp_async_wait_all();
    } else {
        // ---- consumers.  After a fault every wait returns soon, and the loops run
        // on to their ends, so all warps meet at the same barriers.  But a warp whose
        // wait ran out frees no slot any more: only a slot whose tile was there is
        // free, so the copying warps never arrive on a phase with arrivals of
        // another lap (with more than it has left the barrier is undefined), and
        // stop in turn.
        bool frees = lane == 0;
        const int gq = lane >> 2, t = lane & 3;
        const int grp = warp / kGroupWarps, wrow = warp % kGroupWarps * 32;  // first weight row
        Ring ring(slots, grp);
        float* exch = reinterpret_cast<float*>(hbuf);    // [group][rows][128]
        // while the first tiles are on their way: the weights, the optional
        // outputs, and what the final sums will need of each assignment
        if (routes_by_counting(g)) {
            softmax_tokens(g, s, warp, lane);
            consumer_sync();
        }
        const float per2 = static_cast<float>(G2) / static_cast<float>(L2);
        for (int f = kConsumers - 1 - static_cast<int>(threadIdx.x); f < g.T * g.k; f += kConsumers) {
            const int e = s.ids[f], tk = f / g.k, i = s.rank[e], c0 = s.base[i];
            const int cf = owner(s.start2, G2, i * S2, per2);
            s.term[f] = make_int4(cf, owner(s.start2, G2, (i + 1) * S2 - 1, per2) - cf + 1,
                                  (c0 + cf * g.T) * g.mt_dn +
                                      __popc(s.mask[e] & ((1u << tk) - 1u)),
                                  s.base[i + 1] - c0);
            s.term_tile[f] = i * S2;
            s.term_w[f] =
                FP8 ? s.w[f] * __ldg(g.scales + e * 3 + 2) * (1.0f / kSumScale) : s.w[f];
            if (cta == 0) {
                if (g.ids) g.ids[f] = e;
                if (g.w) g.w[f] = s.w[f];
            }
        }
        // the first batch's pieces of h, one per chunk, for the thread per four
        // columns (see step 2)
        Plan plan(a2, b2, g, CK);
        auto list_pieces = [&](Plan q) {
            if (threadIdx.x != 0) return;
            Chunk c;
            int n = 0, quad = 0;
            q.batch();
            for (; q.take(c); ++n) {
                const int quads = (c.kb1 - c.kb0) * (BK / 4);
                s.pieces[n] = Piece{c.i, c.kb0 * BK, c.slot, quad,
                                    Divisor{quads, __frcp_rn(static_cast<float>(quads))}};
                quad += quads * (s.base[c.i + 1] - s.base[c.i]);
            }
            s.pieces[n].quad = quad;
            s.n_pieces = n;
        };
        list_pieces(plan);
        // the barriers' targets: the next multiples of the grid
        uint64_t target[2] = {0, 0};
        if (threadIdx.x == kBarThread) {
#pragma unroll
            for (int i = 0; i < 2; ++i) target[i] = (r_.seen[i] / G + 1) * G;
        }
        // step 1: gate/up partial sums
        for (int X = a1; X < b1;) {
            const int r = X / g.by_kb_gu;               // row tile over all active experts
            const int i = r / g.by_mt_gu, m = r - i * g.mt_gu;
            const int end = (r + 1) * g.kb_gu < b1 ? (r + 1) * g.kb_gu : b1;
            const int c0 = s.base[i], cnt = s.base[i + 1] - c0;
            const int ra = gq < cnt ? gq : 0, rb = gq + 8 < cnt ? gq + 8 : 0;
            float acc[4][4] = {};
            for (; X < end; ++X) {
                if (((X - a1) & (kGroups - 1)) != grp) continue;
                if (!ring_wait(g, &s.full[ring.slot], ring.phase, &s.abort)) {
                    fault(s, g.status);
                    frees = false;
                }
                uint8_t* tile = smem + ring.slot * slot_sz;
                Wts w;
                load_w(w, tile + wrow * kTileRowBytes, gq, t);
                if constexpr (FP8) {
                    // x to scaled f16 in place, a warp of the group per token
                    for (int c = warp % kGroupWarps; c < cnt; c += kGroupWarps) {
                        const float mul = s.xmul[s.tok[c0 + c]];
                        uint2* v = reinterpret_cast<uint2*>(tile + kTileBytes +
                                                            c * x_row_bytes<FP8>()) + lane;
                        const uint2 b = *v;
                        *v = make_uint2(f16x2(bf16_lo(b.x) * mul, bf16_hi(b.x) * mul),
                                        f16x2(bf16_lo(b.y) * mul, bf16_hi(b.y) * mul));
                    }
                    group_sync(grp);
                }
                const uint8_t* xs = tile + kTileBytes;
                const Act<FP8> xa = load_act<FP8>(xs + ra * x_row_bytes<FP8>(), t);
                Act<FP8> xb = {};
                if (MANY && (!FP8 || cnt > 8))
                    xb = load_act<FP8>(xs + rb * x_row_bytes<FP8>(), t);
                __syncwarp();
                if (frees) mbar_arrive(&s.empty[ring.slot]);
                ring.skip(kGroups);
                if constexpr (!FP8) {
                    tile_mma(acc, w, xa, xb);
                } else {
                    if (MANY && cnt > 8) tile_mma<true>(acc, w, xa, xb);
                    else tile_mma<false>(acc, w, xa, xa);
                }
            }
            // the groups' sums of the row tile, added in group order
            each_sum<FP8, MANY>(acc, gq, t, [&](int tk, int r, float v0, float v1) {
                float* d = exch + (grp * rows + tk) * kTileRows + wrow + r;
                if (tk < cnt) {
                    if constexpr (FP8) *d = v0;
                    else *reinterpret_cast<float2*>(d) = make_float2(v0, v1);
                }
            });
            consumer_sync();
            // columns of 128 rows; segment (row tile r, CTA c) starts at column
            // sum of the counts before r + c * T: segments follow one another
            // with r or c or both growing, so no two overlap
            float* p = g.p1 + (static_cast<size_t>(c0) * g.mt_gu + m * cnt +
                               static_cast<size_t>(cta) * g.T) * kTileRows;
            for (int f = threadIdx.x; f < cnt * kTileRows; f += kConsumers) {
                float v = exch[f];
#pragma unroll
                for (int q = 1; q < kGroups; ++q) v += exch[q * rows * kTileRows + f];
                __stcg(p + f, v);
            }
            consumer_sync();
        }
        consumer_sync();
        if (threadIdx.x == kBarThread && !grid_barrier(g, &g.hdr->arrive[0][0], target[0]))
            fault(s, g.status);
        consumer_sync();

        // step 2: h of this CTA's k-blocks, and the down partial sums.  The ring
        // goes on where the gate/up tiles ended, so visit v0 + vq is this group's
        const int vq = (grp - (b1 - a1)) & (kGroups - 1);
        const float per1 = static_cast<float>(G1) / static_cast<float>(L1);
        Chunk ch;
        while (!plan.done()) {
            // the batch's h, four columns a thread and turn: all chunks' quads in
            // one sequence (a chunk's are a multiple of 16, of 32 for e4m3)
            const int quads_all = s.pieces[s.n_pieces].quad;
            constexpr int TURNS =
                CK * BK / 4 * (MANY ? kDecodeMaxT : 8) / kConsumers;
            float4 hq[TURNS];
            int hp[TURNS], hc[TURNS];      // where: piece, and column << 16 | quad
#pragma unroll
            for (int u = 0; u < TURNS; ++u) {
                const int idx = threadIdx.x + u * kConsumers;
                hq[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (idx >= quads_all) continue;
                int n = 0;
                while (s.pieces[n + 1].quad <= idx) ++n;
                const Piece pc = s.pieces[n];
                const int r = idx - pc.quad, c = r / pc.quads, j = r - c * pc.quads.d;
                hp[u] = n;
                hc[u] = c << 16 | j;
                if (pc.col + 4 * j < g.I) {
                    float sg = 1.0f, su = 1.0f;
                    const int c0 = s.base[pc.i];
                    if constexpr (FP8) {
                        const float inv = scale_inv(s.xmul[s.tok[c0 + c]]);
                        sg = __ldg(g.scales + s.expert[pc.i] * 3) * inv;
                        su = __ldg(g.scales + s.expert[pc.i] * 3 + 1) * inv;
                    }
                    hq[u] = h_quad(g, s, pc.i, c0, s.base[pc.i + 1] - c0, c, pc.col + 4 * j, G1,
                                   per1, sg, su);
                }
                if constexpr (FP8) {
                    // the largest |h| per column: a warp's quads are of one column
                    const uint32_t m = __reduce_max_sync(
                        kFullWarp, max(max(finite_mag(hq[u].x), finite_mag(hq[u].y)),
                                       max(finite_mag(hq[u].z), finite_mag(hq[u].w))));
                    if (lane == 0) atomicMax(&s.hmax[n][c], m);
                }
            }
            if constexpr (FP8) consumer_sync();
#pragma unroll
            for (int u = 0; u < TURNS; ++u) {
                if (static_cast<int>(threadIdx.x) + u * kConsumers >= quads_all) continue;
                const int c = hc[u] >> 16, j = (hc[u] & 0xffff) * 4;
                const int kl = s.pieces[hp[u]].slot + j / BK, jj = j % BK;
                uint8_t* d = hbuf + (kl * rows + c) * h_row_bytes<FP8>() + jj * 2;
                const float4 h = hq[u];
                if constexpr (FP8) {
                    const float mul = f16_scale(s.hmax[hp[u]][c]);
                    *reinterpret_cast<uint2*>(d) =
                        make_uint2(f16x2(h.x * mul, h.y * mul), f16x2(h.z * mul, h.w * mul));
                } else {
                    const uint32_t h0 = bf16x2(h.x, h.y), h1 = bf16x2(h.z, h.w);
                    *reinterpret_cast<uint2*>(d) = make_uint2(h0, h1);
                    *reinterpret_cast<uint2*>(d + BK * 2) =
                        make_uint2(bf16x2(rest(h.x, bf16_lo(h0)), rest(h.y, bf16_hi(h0))),
                                   bf16x2(rest(h.z, bf16_lo(h1)), rest(h.w, bf16_hi(h1))));
                }
            }
            consumer_sync();
            plan.batch();
            for (int n = 0; plan.take(ch); ++n) {
                const int c0 = s.base[ch.i], cnt = s.base[ch.i + 1] - c0;
                float* p = g.p2 + (static_cast<size_t>(c0) + static_cast<size_t>(cta) * g.T) *
                                      g.mt_dn * kTileRows +
                           wrow;
                const int ra = gq < cnt ? gq : 0, rb = gq + 8 < cnt ? gq + 8 : 0;
                // (e4m3) the unscaling of this lane's tokens
                float inv[4] = {1.0f, 1.0f, 1.0f, 1.0f};
                if constexpr (FP8) {
#pragma unroll
                    for (int q = 0; q < (MANY ? 4 : 2); ++q)
                        inv[q] = kSumScale *
                                 scale_inv(f16_scale(s.hmax[n][8 * (q >> 1) + 2 * t + (q & 1)]));
                }
                // this group's first visit's k-block (counted from the chunk's
                // first) and row tile
                int kb0 = 0, m = ch.m + vq;
                for (; m >= g.mt_dn; m -= g.mt_dn) ++kb0;
                for (int v0 = 0; v0 < ch.visits; v0 += kGroups) {
                    const bool visit = v0 + vq < ch.visits;
                    float acc[4][4] = {};
                    const uint8_t* hr = hbuf + (ch.slot + kb0) * rows * h_row_bytes<FP8>();
                    for (int L = ch.a + v0; L < ch.b;
                         L += g.mt_dn, hr += rows * h_row_bytes<FP8>()) {
                        if (!ring_wait(g, &s.full[ring.slot], ring.phase, &s.abort)) {
                            fault(s, g.status);
                            frees = false;
                        }
                        const bool real = visit && L + vq < ch.b;
                        Wts w;
                        if (real) load_w(w, smem + ring.slot * slot_sz + wrow * kTileRowBytes, gq, t);
                        __syncwarp();
                        if (frees) mbar_arrive(&s.empty[ring.slot]);
                        ring.skip(kGroups);
                        if (!real) continue;
                        const uint8_t* ha = hr + ra * h_row_bytes<FP8>();
                        const uint8_t* hb = hr + rb * h_row_bytes<FP8>();
                        const Act<FP8> xa = load_act<FP8>(ha, t);
                        if constexpr (FP8) {
                            if (MANY && cnt > 8) tile_mma<true>(acc, w, xa, load_act<FP8>(hb, t));
                            else tile_mma<false>(acc, w, xa, xa);
                        } else if (!(MANY && cnt > 8)) {
                            // hi in rows 0..7, lo in rows 8..15 of the same MMA
                            tile_mma(acc, w, xa, load_act<FP8>(ha + BK * 2, t));
                        } else {
                            tile_mma(acc, w, xa, load_act<FP8>(hb, t));
                            tile_mma(acc, w, load_act<FP8>(ha + BK * 2, t),
                                     load_act<FP8>(hb + BK * 2, t));
                        }
                    }
                    if (visit) {
                        float* d = p + static_cast<size_t>(m) * cnt * kTileRows;
                        if constexpr (FP8) {
#pragma unroll
                            for (int b = 0; b < (MANY ? 4 : 2); ++b)
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    acc[b][q] *= inv[(b >> 1) * 2 + (q & 1)];
                        } else if (!(MANY && cnt > 8)) {
#pragma unroll
                            for (int b = 0; b < 4; ++b) {       // hi + lo
                                acc[b][0] += acc[b][2];
                                acc[b][1] += acc[b][3];
                            }
                        }
                        // later chunks of an expert add to what this CTA wrote: of
                        // several the first has CK k-blocks, so every row tile
                        each_sum<FP8, MANY>(acc, gq, t, [&](int tk, int r, float v0s, float v1s) {
                            if (tk < cnt) put<FP8>(d + tk * kTileRows + r, v0s, v1s, ch.first);
                        });
                    }
                    for (m += kGroups; m >= g.mt_dn; m -= g.mt_dn) ++kb0;
                }
            }
            consumer_sync();   // hbuf is free, the batch's sums are written
            if constexpr (FP8) {
                for (int f = threadIdx.x; f < CK * kDecodeMaxT; f += kConsumers)
                    (&s.hmax[0][0])[f] = 0;
            }
            list_pieces(plan);
            consumer_sync();
        }
        // step 3: out[t] = residual[t] + sum over the token's assignments and
        // their CTAs; four columns a thread.  When there are few outputs `spl`
        // threads share one's terms: `sj` of them the assignments, sc = spl / sj
        // the CTAs of each; lanes first (ls, so that 8 lanes still read 128
        // consecutive bytes), then warps.
        const int hquads = g.H / 4, items = g.T * hquads;
        int spl2 = 0;                                  // powers of two, as exponents
        while ((1 << spl2) < 4 * kConsumerWarps && (items << (spl2 + 1)) <= G * kConsumers) ++spl2;
        const int sj2 = min(spl2, 31 - __clz(g.k)), ls2 = min(spl2, 2), lw2 = 5 - ls2;
        const int ws2 = spl2 - ls2, sj = 1 << sj2, sc = 1 << (spl2 - sj2);
        const int lw = 1 << lw2, ws = 1 << ws2, per_cta = kConsumers >> spl2;
        const int sub = ((warp & (ws - 1)) << ls2) + (lane >> lw2);
        const int jsub = sub & (sj - 1), csub = sub >> sj2;
        // the first item's residual is on its way while the CTA waits
        auto item_of = [&](int item0) {
            return item0 + ((warp >> ws2) << lw2) + (lane & (lw - 1));
        };
        auto residual_of = [&](int item) {
            return g.residual && sub == 0 && item < items
                       ? __ldcg(reinterpret_cast<const uint2*>(g.residual) + item)
                       : make_uint2(0u, 0u);
        };
        uint2 res = residual_of(item_of(cta * per_cta));
        if (threadIdx.x == kBarThread && !grid_barrier(g, &g.hdr->arrive[1][0], target[1]))
            fault(s, g.status);
        consumer_sync();

        float4* red = reinterpret_cast<float4*>(smem);   // the ring has run dry
        const size_t step = static_cast<size_t>(g.T) * g.mt_dn * kTileRows;
        for (int item0 = cta * per_cta; item0 < items; item0 += G * per_cta) {
            const int item = item_of(item0);
            if (item0 != cta * per_cta) res = residual_of(item);
            const int tk = item / g.by_hquads, col = (item - tk * hquads) * 4;
            float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
            if (item < items) {
                const int m = col / kTileRows, row = col - m * kTileRows;
                for (int j = jsub; j < g.k; j += sj) {
                    const int f = tk * g.k + j;
                    const int4 term = s.term[f];
                    const int tile0 = s.term_tile[f];
                    const float wt = s.term_w[f];
                    const int cf = term.x, n = term.y;
                    const float* q = g.p2 + (static_cast<size_t>(term.z) +
                                             static_cast<size_t>(m) * term.w) * kTileRows + row;
                    float4 part = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                    for (int cc = csub; cc < n; cc += sc) {
                        // does CTA cf + cc hold a tile of row tile m?  Its range
                        // within the expert starts at row tile `am` and has
                        // `len` tiles, the row tile fastest
                        const int st = s.start2[cf + cc] - tile0;
                        const int en = s.start2[cf + cc + 1] - tile0;
                        const int am = st < 0 ? 0 : s.mod2[cf + cc];
                        const int len = (en > S2 ? S2 : en) - (st < 0 ? 0 : st);
                        int d = m - am;
                        d += d < 0 ? g.mt_dn : 0;
                        if (d < len)
                            part = add4(part, __ldcg(reinterpret_cast<const float4*>(q + cc * step)));
                    }
                    sum.x += wt * part.x;
                    sum.y += wt * part.y;
                    sum.z += wt * part.z;
                    sum.w += wt * part.w;
                }
            }
            for (int off = lw; off < 32; off *= 2) {
                const float4 o = make_float4(__shfl_xor_sync(kFullWarp, sum.x, off),
                                             __shfl_xor_sync(kFullWarp, sum.y, off),
                                             __shfl_xor_sync(kFullWarp, sum.z, off),
                                             __shfl_xor_sync(kFullWarp, sum.w, off));
                sum = add4(sum, o);
            }
            if (ws > 1) {
                red[threadIdx.x] = sum;
                consumer_sync();
                if (sub == 0)
                    for (int q = 1; q < ws; ++q) sum = add4(sum, red[threadIdx.x + 32 * q]);
                consumer_sync();
            }
            if (sub == 0 && item < items) {
                const size_t o = static_cast<size_t>(tk) * g.H + col;
                if (g.residual)
                    sum = add4(sum, make_float4(bf16_lo(res.x), bf16_hi(res.x), bf16_lo(res.y),
                                                bf16_hi(res.y)));
                *reinterpret_cast<uint2*>(g.out + o) =
                    make_uint2(bf16x2(sum.x, sum.y), bf16x2(sum.z, sum.w));
            }
        }
    }
}

// MANY: the batch has more than 8 tokens, so that an expert may
template <bool FP8, bool MANY>
__global__ void __launch_bounds__(kThreads, 1) decode_kernel(const Args g) {
    extern __shared__ uint8_t dsmem_raw[];
    __shared__ Shared s;
    uint8_t* smem = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = gridDim.x;

    // (used below, so that the loads' latency hides behind the routing's)
    const uint32_t magic = __ldcg(&g.hdr->magic);
    uint64_t seen[2] = {0, 0};
    if (threadIdx.x == kBarThread) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            seen[i] = __ldcg(reinterpret_cast<const unsigned long long*>(&g.hdr->arrive[i][0]));
        s.abort = 0;
    }
    if (threadIdx.x < kDecodeMaxT) s.xmax[threadIdx.x] = 0;
    // a slot is full when its tile's bytes are there and, for the gate/up tiles,
    // the x slices that another warp's lanes copy
    if (threadIdx.x < kMaxSlots) {
        mbar_init(&s.full[threadIdx.x], 1 + 32);
        mbar_init(&s.empty[threadIdx.x], kGroupWarps);
        fence_mbar_init();
    }
    for (int e = threadIdx.x; e < kMaxExperts; e += kThreads) s.mask[e] = 0;
    __syncthreads();

    // ---- routing (every CTA, all tokens); keys in the ring's memory, no copy
    // is under way yet
    if (warp < kConsumerWarps) {
        route_tokens<FP8>(g, s, reinterpret_cast<uint64_t*>(smem), warp, lane);
    }
    // a workspace that was never initialised would hang the barriers: every
    // CTA sees the same word and leaves
    if (magic != kMagic) {
        if (threadIdx.x == 0) report(g.status, MOE_ERR_DEVICE);
        return;
    }
    __syncthreads();
    // active experts in ascending order with their first columns: one scan of
    // (active, count) pairs over the experts, a thread each
    const int e_own = threadIdx.x;
    const uint32_t mk = e_own < kMaxExperts ? s.mask[e_own] : 0u;
    const int own = mk ? (1 << 16) | __popc(mk) : 0;
    int inc = own;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(kFullWarp, inc, off);
        if (lane >= off) inc += o;
    }
    const int most_here = __reduce_max_sync(kFullWarp, own & 0xffff);
    if (lane == 31 && warp < kMaxExperts / 32) {
        s.scan[warp] = inc;
        s.most[warp] = most_here;
    }
    __syncthreads();
    int before = 0, all = 0, rows = 0;
#pragma unroll
    for (int i = 0; i < kMaxExperts / 32; ++i) {
        const int v = s.scan[i];
        if (i < warp) before += v;
        all += v;
        rows = max(rows, s.most[i]);
    }
    const int n_active = all >> 16;
    const int slot_sz = slot_bytes<FP8>(rows), slots = slots_for<FP8>(rows, g.smem);
    uint8_t* hbuf = smem + slots * slot_sz;
    if (mk) {
        const int ex = before + inc - own;
        const int i = ex >> 16, c0 = ex & 0xffff;
        s.rank[e_own] = i;
        s.expert[i] = e_own;
        s.base[i] = c0;
        int c = c0;
        for (uint32_t m = mk; m; m &= m - 1) s.tok[c++] = __ffs(m) - 1;
    }
    if (threadIdx.x == 0) s.base[n_active] = all & 0xffff;
    const int S1 = g.mt_gu * g.kb_gu, S2 = g.mt_dn * g.kb_dn;   // tiles per expert
    const int L1 = n_active * S1, L2 = n_active * S2;
    const int G1 = L1 < G ? L1 : G, G2 = L2 < G ? L2 : G;
    {
        // floor(L c / G) without 64-bit products: whole tiles, and the remainder's
        // (with fewer tiles than CTAs a tile each)
        const int q1 = L1 / g.by_G, r1 = L1 - q1 * G, q2 = L2 / g.by_G, r2 = L2 - q2 * G;
        for (int c = threadIdx.x; c <= G; c += kThreads) {
            s.start1[c] = c < G1 ? (L1 < G ? c : q1 * c + r1 * c / g.by_G) : L1;
            const int st = c < G2 ? (L2 < G ? c : q2 * c + r2 * c / g.by_G) : L2;
            s.start2[c] = st;
            if (c < G) s.mod2[c] = st - st / g.by_mt_dn * g.mt_dn;
        }
        if (FP8 && threadIdx.x < kDecodeMaxT)
            s.xmul[threadIdx.x] = f16_scale(s.xmax[threadIdx.x]);
        for (int f = threadIdx.x; f < 8 * kDecodeMaxT; f += kThreads) (&s.hmax[0][0])[f] = 0;
    }
    __syncthreads();
    const Run r{smem, hbuf, rows, slots, slot_sz, S1, S2, L1, L2, G1, G2,
                {seen[0], seen[1]}};
    if (MANY && rows > 8) run_steps<FP8, true>(g, s, r);
    else run_steps<FP8, false>(g, s, r);
}

__global__ void decode_ws_init_kernel(Header* h) {
    if (threadIdx.x == 0) {
        h->status = 0;
        h->arrive[0][0] = 0;
        h->arrive[1][0] = 0;
        h->magic = kMagic;
    }
}

// The opt-in to more than 48 KB of dynamic shared memory, once per device and
// instantiation.
constexpr int kMaxDevices = 64;
constexpr int kDynSmemMax = kSmemBytes - static_cast<int>(sizeof(Shared)) - 1024;

template <bool FP8, bool MANY>
cudaError_t opt_in_smem() {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [dev] {
        err[dev] = cudaFuncSetAttribute(decode_kernel<FP8, MANY>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize, kDynSmemMax);
    });
    return err[dev];
}

template <bool FP8, bool MANY>
cudaError_t launch(const Args& a, int grid, cudaStream_t s) {
    auto kern = decode_kernel<FP8, MANY>;
    const cudaError_t e = opt_in_smem<FP8, MANY>();
    if (e != cudaSuccess) return e;
    Args g = a;
    g.smem = kDynSmemMax - 128;
    static_assert(slots_for<FP8>(kDecodeMaxT, kDynSmemMax - 128) >= kGroups, "a slot per group");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kDynSmemMax;
    cfg.stream = s;
    // cooperative: the blocks wait on one another, so all must be resident
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeCooperative;
    at[0].val.cooperative = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, g);
}

struct Sizes {
    size_t p1, p2, total;
};

Sizes sizes(bool fp8, int T, int k, int E, int H, int I, int grid) {
    const PackedGeom geo = packed_geom(fp8, E, H, I);
    const size_t A = static_cast<size_t>(T) * k, col = kTileRows * sizeof(float);
    Sizes z;
    z.p1 = (A * geo.mt_gu + static_cast<size_t>(grid) * T) * col;
    z.p2 = (A + static_cast<size_t>(grid) * T) * geo.mt_dn * col;
    z.total = sizeof(Header) + z.p1 + z.p2;
    return z;
}

}  // namespace

size_t decode_ws_bytes(int fp8, int T, int k, int E, int H, int I) {
    return sizes(fp8 != 0, T, k, E, H, I, device_sm_count()).total;
}

cudaError_t launch_decode_ws_init(void* ws, cudaStream_t s) {
    static_assert(sizeof(Header) % 16 == 0, "partial sums stay 16-byte aligned");
    decode_ws_init_kernel<<<1, 32, 0, s>>>(static_cast<Header*>(ws));
    return cudaGetLastError();
}

cudaError_t launch_decode(const DecodeProblem& p, cudaStream_t s) {
    const bool fp8 = p.fp8 != 0;
    const PackedGeom geo = packed_geom(fp8, p.E, p.H, p.I);
    const int grid = device_sm_count();
    const Sizes z = sizes(fp8, p.T, p.k, p.E, p.H, p.I, grid);
    Args g{};
    static_cast<SelfTest&>(g) = self_test();
    g.T = p.T;
    g.k = p.k;
    g.E = p.E;
    g.H = p.H;
    g.I = p.I;
    g.mt_gu = geo.mt_gu;
    g.kb_gu = geo.kb_gu;
    g.mt_dn = geo.mt_dn;
    g.kb_dn = geo.kb_dn;
    g.by_mt_gu = divisor(g.mt_gu);
    g.by_kb_gu = divisor(g.kb_gu);
    g.by_mt_dn = divisor(g.mt_dn);
    g.by_S1 = divisor(g.mt_gu * g.kb_gu);
    g.by_S2 = divisor(g.mt_dn * g.kb_dn);
    g.by_G = divisor(grid);
    g.by_hquads = divisor(g.H / 4);
    g.w_gu = static_cast<const uint8_t*>(p.packed);
    g.w_dn = g.w_gu + geo.gu_bytes;
    g.scales = p.scales;
    g.x = static_cast<const __nv_bfloat16*>(p.x);
    g.logits = p.logits;
    g.residual = static_cast<const __nv_bfloat16*>(p.residual);
    g.out = static_cast<__nv_bfloat16*>(p.out);
    g.ids = p.ids;
    g.w = p.w;
    g.hdr = static_cast<Header*>(p.ws);
    g.status = p.status ? p.status : &g.hdr->status;
    g.p1 = reinterpret_cast<float*>(static_cast<char*>(p.ws) + sizeof(Header));
    g.p2 = reinterpret_cast<float*>(static_cast<char*>(p.ws) + sizeof(Header) + z.p1);
    if (p.T <= 8) return fp8 ? launch<true, false>(g, grid, s) : launch<false, false>(g, grid, s);
    return fp8 ? launch<true, true>(g, grid, s) : launch<false, true>(g, grid, s);
}

}  // namespace moe
