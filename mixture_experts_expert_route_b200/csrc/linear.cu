// linear.cu -- the dense products around the MoE layer, with everything that
// follows a product in its epilogue:
//
//   out = act(x W^T + bias) [* (x W_up^T + bias_up)] [+ residual]
//
// x [M,K] token rows, W [N,K] (or [2N,K]: gate rows, then up rows) as
// checkpoints keep them, both bf16 and K-major, so both operands come straight
// from the caller's tensors; sums, bias, activation and residual in fp32, one
// rounding to the output type.  The router's logits (fp32 out), a shared
// expert's two products, and the projections before and after the layer.
//
// Four kernels, by what bounds them:
//   few   M <= 16: the stream of W.  Warp MMAs fed by 16-byte loads from global
//         memory, no shared memory and no barrier in the way; K is split over
//         warps, and over the blocks of a cluster, until about 16 warps per SM
//         have loads in flight.
//   tile  one 128 x BN tcgen05 tile per block; when there are fewer tiles than
//         SMs, the blocks of a cluster split K and add their accumulators
//         through distributed shared memory.
//   pair  256 x 256 tiles on CTA pairs (cta_group::2), persistent, two TMEM
//         accumulators, so an epilogue runs under the next tile's products.
//   split such a tile on a cluster of two pairs, half of a long K each.
// No kernel needs a workspace, and no sum depends on timing.
//
// Measured on one B200 in a graph (us; floor at the measured copy and bf16 GEMM
// rates; cuBLAS = the plain product alone, no epilogue, in the same run):
//   few   M=1  K=7168 N=2x2048 gated    12.8  (floor 9.0 by bytes, cuBLAS 20.6)
//         M=13 K=2048 N=7168 residual   9.9   (4.6, 8.0)  224 blocks on 148 SMs
//         M=16 K=14336 N=4096 residual  23    (18, 24)
//   tile  M=77 K=N=2880                 10.1  (2.7, 7.5)  latency: ~6 us of first
//         copies, cluster sum and store around 11 k-blocks a block
//         M=4096 K=2048 N=128           8.9   (3.0, 5.3)
//         M=K=512 N=4096                7.5   (1.3, 5.0)
//         M=2500 K=2048 N=2041          39    (12.5, 218) rows that are not aligned
//   split M=512 K=7168 N=2x2048 gated   27-28 (18, 24)   128-wide tiles 34: they read
//         1.5x the shared memory that their MMAs take
//   pair  M=8192 K=7168 N=2x2048 gated  314-370 (288 at the burst rate; cuBLAS
//         321-378 in the same runs): the power cap; M=1024 K=N=4096 28 (21, 25.6);
//         M=1500 K=N=2048 16.5 (7.5, 11.5): 48 tiles on 74 pairs
#include <cstdint>
#include <cstring>
#include <mutex>

#include "common.cuh"
#include "kernels.h"

namespace moe {

namespace {

constexpr int kRowBytes = 128;           // one swizzle atom: 64 bf16 of K
constexpr int kBK = 64;
constexpr uint64_t kDrainLimitNs = 10000000ull;

// Where a wait that ran out is recorded when the call gives no status word: one
// per device, read by moe_linear_status.
__device__ int32_t own_status;

struct Args : SelfTest {
    int M, N, K;
    int act, gated;
    const __nv_bfloat16* x;
    const __nv_bfloat16* w;
    long long ldx, ldw, ldr, ldo;        // elements
    const void* bias;                    // bf16 or f32 [rows of W] or null
    int bias_f32;
    const void* residual;                // out's type, or null
    void* out;
    int out_f32;
    int vec;                             // bytes that out's and residual's rows are aligned to: 32, 16 or 0
    int32_t* status;
};

__device__ __forceinline__ void report_timeout(const Args& g) {
    report(g.status ? g.status : &own_status, MOE_ERR_TIMEOUT);
}

__device__ __forceinline__ float load_bias(const Args& g, int row) {
    if (!g.bias) return 0.0f;
    return g.bias_f32 ? __ldg(static_cast<const float*>(g.bias) + row)
                      : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(g.bias) + row));
}

// z / (1 + e^-y) with the fast exponential and division: off by a few fp32 ulp
// where it counts (the exponential's error grows with |y|, but then the factor
// is near 0 or 1), and a NaN, 0 or z at the ends as the exact form.
__device__ __forceinline__ float times_sigmoid(float z, float y) {
    return __fdividef(z, 1.0f + __expf(-y));
}

// (1 + erf(z / sqrt 2)) / 2, with its negative tail's relative accuracy, which the
// sum in fp32 loses (GELU was 6% off at z = -5 and 0 beyond -5.5):
//   Q(s) = erfc(s / sqrt 2) / 2 = e^(-s^2/2) t P(t),  t = 1 / (1 + 0.35 s),  s = |z|,
// and 1 - Q for z >= 0.  The form is Hastings' (Approximations for Digital
// Computers, 1955); P, of degree 8, is a least-squares fit, reweighted to an even
// error, to erfc in 64 bits over s <= 13.5: 3.2e-8 relative, 3.2e-7 evaluated in
// fp32; the exponential adds s^2 2^-24.  NaN stays NaN, t is 0 at infinity.
// (erfcf is as good, but M = K = 2048 N = 4096 went from 36 to 44 us with it; the
// last line as a choice of two values cost the CTA pairs' unaligned epilogue 10%
// in registers, with any activation.)
__device__ __forceinline__ float normal_cdf(float z) {
    const float s = fabsf(z), t = __fdividef(1.0f, fmaf(0.35f, s, 1.0f));
    float p = -0.0291258618f;
    p = fmaf(p, t, 0.143872216f);
    p = fmaf(p, t, -0.255504549f);
    p = fmaf(p, t, 0.158929288f);
    p = fmaf(p, t, -0.0229371469f);
    p = fmaf(p, t, 0.105432943f);
    p = fmaf(p, t, 0.119852431f);
    p = fmaf(p, t, 0.13985908f);
    p = fmaf(p, t, 0.139621571f);
    const float q = __expf(-0.5f * s * s) * (t * p);
    return fmaf(z < 0.0f ? 0.0f : 1.0f, fmaf(-2.0f, q, 1.0f), q);     // q or 1 - q
}

// The activations on fp32 (a NaN stays one).  GELU's tanh form is
// z (1 + tanh u) / 2 = z / (1 + e^-2u), which cancels nothing.  One branch for
// all of a thread's values: with a switch per value the 16 copies of five
// activations' code left a CTA pair's epilogue waiting for instructions, 19 us a
// tile with no activation at all; with IEEE divisions SiLU took 15 us a tile.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
    if (act == MOE_ACT_NONE) return;
    if (act == MOE_ACT_RELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = v[i] < 0.0f ? 0.0f : v[i];
    } else if (act == MOE_ACT_SILU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = times_sigmoid(v[i], v[i]);
    } else if (act == MOE_ACT_GELU) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] *= normal_cdf(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = times_sigmoid(
                v[i], 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
    }
}

__device__ __forceinline__ float load_res(const Args& g, long long row, int col) {
    const long long o = row * g.ldr + col;
    return g.out_f32 ? static_cast<const float*>(g.residual)[o]
                     : __bfloat162float(static_cast<const __nv_bfloat16*>(g.residual)[o]);
}

__device__ __forceinline__ void store_out(const Args& g, long long row, int col, float v) {
    const long long o = row * g.ldo + col;
    if (g.out_f32) static_cast<float*>(g.out)[o] = v;
    else static_cast<__nv_bfloat16*>(g.out)[o] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&b);
}

// 32 bytes of a row: a whole sector per access where rows are aligned to it, else
// two of 16 (vec: 32 or 16).
__device__ __forceinline__ void ld32(const void* p, uint32_t (&r)[8], int vec) {
    if (vec == 32) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                       "=r"(r[6]), "=r"(r[7])
                     : "l"(p)
                     : "memory");
    } else {
        const uint4 a = static_cast<const uint4*>(p)[0], b = static_cast<const uint4*>(p)[1];
        r[0] = a.x;
        r[1] = a.y;
        r[2] = a.z;
        r[3] = a.w;
        r[4] = b.x;
        r[5] = b.y;
        r[6] = b.z;
        r[7] = b.w;
    }
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&r)[8], int vec) {
    if (vec == 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p),
                     "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
                     "r"(r[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        static_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// 16 consecutive columns of one row, from column col (a multiple of 16); the
// arrays hold the residual's (see res16).
__device__ __forceinline__ bool wide16(const Args& g, int col) {
    return g.vec >= 16 && col + 16 <= g.N;
}
__device__ __forceinline__ void res16(const Args& g, long long row, int col, uint32_t (&a)[8],
                                      uint32_t (&b)[8]) {
    if (g.out_f32) {
        const float* p = static_cast<const float*>(g.residual) + row * g.ldr + col;
        ld32(p, a, g.vec);
        ld32(p + 8, b, g.vec);
    } else {
        ld32(static_cast<const __nv_bfloat16*>(g.residual) + row * g.ldr + col, a, g.vec);
    }
}
__device__ __forceinline__ void add_res16(const Args& g, float (&v)[16], const uint32_t (&a)[8],
                                          const uint32_t (&b)[8]) {
    if (g.out_f32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] += __uint_as_float(a[i]);
            v[8 + i] += __uint_as_float(b[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] += bf16_lo(a[i]);
            v[2 * i + 1] += bf16_hi(a[i]);
        }
    }
}
__device__ __forceinline__ void store16(const Args& g, long long row, int col, const float (&v)[16]) {
    uint32_t r[8];
    if (g.out_f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[8 * h + i]);
            st32(static_cast<float*>(g.out) + row * g.ldo + col + 8 * h, r, g.vec);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
        st32(static_cast<__nv_bfloat16*>(g.out) + row * g.ldo + col, r, g.vec);
    }
}

// Four consecutive columns (a multiple of 4): the residual's, and the store.
__device__ __forceinline__ float4 res4(const Args& g, long long row, int col) {
    const long long o = row * g.ldr + col;
    if (g.vec < 16 || col + 4 > g.N) {
        float a[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = col + i < g.N ? load_res(g, row, col + i) : 0.0f;
        return make_float4(a[0], a[1], a[2], a[3]);
    }
    if (g.out_f32) return *reinterpret_cast<const float4*>(static_cast<const float*>(g.residual) + o);
    const uint2 r =
        *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(g.residual) + o);
    return make_float4(bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y));
}
__device__ __forceinline__ void store4(const Args& g, long long row, int col, float4 v) {
    const long long o = row * g.ldo + col;
    if (g.vec < 16 || col + 4 > g.N) {
        const float a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (col + i >= g.N) break;
            store_out(g, row, col + i, a[i]);
        }
    } else if (g.out_f32) {
        *reinterpret_cast<float4*>(static_cast<float*>(g.out) + o) = v;
    } else {
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(g.out) + o) =
            make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
}

// The same of a warp's 32 rows where they are not aligned or end within: through
// a buffer of the warp, so that 16 lanes write 16 consecutive columns (with a
// row per lane every store touched 32 sectors: 78 us instead of 13 at M = 5000,
// K = 512, N = 1000).  row0 is lane 0's; all lanes take part.
constexpr int kBufFloats = 32 * 17;
template <class T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32(float v) { return v; }
template <> __device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
// every second row from p (and q, the residual's) on, n of them
template <class T>
__device__ __forceinline__ void rows16(T* p, long long ldo, const T* q, long long ldr,
                                       const float* buf, int n) {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        t[i] = buf[2 * 17 * i];
        if (q && i < n) t[i] += to_f32(q[2 * i * ldr]);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < n) p[2 * i * ldo] = from_f32<T>(t[i]);
}
__device__ __forceinline__ void some16(const Args& g, float* buf, long long row0, int col,
                                       const float (&v)[16]) {
    const int lane = threadIdx.x & 31, r = lane >> 4, c = lane & 15;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < 16; ++j) buf[lane * 17 + j] = v[j];
    __syncwarp();
    const int rows = static_cast<int>(min(32ll, g.M - row0));
    const int n = col + c < g.N ? (rows - r + 1) / 2 : 0;
    const long long o = (row0 + r) * g.ldo + col + c, d = (row0 + r) * g.ldr + col + c;
    if (g.out_f32)
        rows16(static_cast<float*>(g.out) + o, g.ldo,
               g.residual ? static_cast<const float*>(g.residual) + d : nullptr, g.ldr,
               buf + r * 17 + c, n);
    else
        rows16(static_cast<__nv_bfloat16*>(g.out) + o, g.ldo,
               g.residual ? static_cast<const __nv_bfloat16*>(g.residual) + d : nullptr, g.ldr,
               buf + r * 17 + c, n);
}

// What follows the sums (bias included) of 16 consecutive columns, a row per lane,
// and their store.  All lanes take part.
__device__ __forceinline__ void finish16(const Args& g, float* buf, long long row0, int col,
                                         float (&v)[16], const float (&u)[16]) {
    activate(v, g.act);
    if (g.gated) {
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] *= u[j];
    }
    if (!wide16(g, col)) {
        some16(g, buf, row0, col, v);
        return;
    }
    const long long row = row0 + (threadIdx.x & 31);
    if (row >= g.M) return;
    if (g.residual) {
        uint32_t qa[8], qb[8];
        res16(g, row, col, qa, qb);
        add_res16(g, v, qa, qb);
    }
    store16(g, row, col, v);
}

// ------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_addr(uint32_t smem, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem), "r"(rank));
    return a;
}
__device__ __forceinline__ float ld_cluster(uint32_t a) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
// Bulk copy into another block's shared memory, completing on its mbarrier (both
// shared::cluster addresses; 16-byte aligned, whole 16 bytes).
__device__ __forceinline__ void bulk_to_cluster(uint32_t dst, const void* src, uint32_t bytes,
                                                uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(dst), "r"(smem_u32(src)), "r"(bytes), "r"(bar)
        : "memory");
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}

// ================================================================= few
// A warp takes 16 weight rows (gated: 8 gate rows and their 8 up rows) and a
// range of 64-column steps of K.  m16n8k16 MMAs, tokens in M; the K order
// inside a step is permuted the same way for both operands: lane (g, t) reads
// 16-byte pieces t and t + 4 of its rows, so that each load of a warp covers
// whole 32-byte sectors.
constexpr int kFewThreads = 256;
constexpr int kFewWarps = kFewThreads / 32;

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Weights are read once: past L1.
__device__ __forceinline__ uint4 ld_stream(const uint4* p) {
    uint4 v;
    asm("ld.global.nc.L1::no_allocate.L2::256B.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <int MB>
struct Step {
    uint4 w[2][2];      // [block of 8 rows][16-byte piece]
    uint4 x[MB][2];     // [token row g, g + 8][piece]
};

// MB: blocks of 8 tokens.  wk: warps of a block that share rows and split K.
template <int MB>
__global__ void __launch_bounds__(kFewThreads, 2)
    linear_few_kernel(const Args g, int wk, int csize) {
    __shared__ float sums[kFewWarps][16][16];     // [warp][token][row]
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int gq = lane >> 2, t = lane & 3;
    const int wr = kFewWarps / wk;                // row groups of a block
    const uint32_t rank = csize > 1 ? cluster_ctarank() : 0;
    const int block = blockIdx.x / csize;
    const int per = g.gated ? 8 : 16;             // output columns of a row group
    const int col0 = (block * wr + warp / wk) * per;
    const int steps = (g.K + kBK - 1) / kBK, parts = wk * csize;
    const int part = static_cast<int>(rank) * wk + warp % wk;
    const int s0 = static_cast<int>(static_cast<long long>(steps) * part / parts);
    const int s1 = static_cast<int>(static_cast<long long>(steps) * (part + 1) / parts);

    // this lane's rows.  Rows and tokens past the end read row 0: what they give
    // is in columns and rows of the result that nobody looks at.
    const int c0 = col0 + gq, c1 = g.gated ? col0 + gq : col0 + 8 + gq;
    const __nv_bfloat16* w0 = g.w + (c0 < g.N ? c0 : 0) * g.ldw + 8 * t;
    const __nv_bfloat16* w1 =
        g.w + (c1 < g.N ? (g.gated ? static_cast<long long>(g.N) + c1 : c1) : 0) * g.ldw + 8 * t;
    const __nv_bfloat16* xr[MB];
#pragma unroll
    for (int m = 0; m < MB; ++m)
        xr[m] = g.x + (m * 8 + gq < g.M ? m * 8 + gq : 0) * g.ldx + 8 * t;
    auto load = [&](Step<MB>& st, int s) {
        const long long k = static_cast<long long>(s) * kBK;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            st.w[0][p] = ld_stream(reinterpret_cast<const uint4*>(w0 + k + 32 * p));
            st.w[1][p] = ld_stream(reinterpret_cast<const uint4*>(w1 + k + 32 * p));
#pragma unroll
            for (int m = 0; m < MB; ++m)
                st.x[m][p] = __ldg(reinterpret_cast<const uint4*>(xr[m] + k + 32 * p));
        }
    };
    const uint4 zero = make_uint4(0, 0, 0, 0);
    float acc[2][4] = {};
    auto mul = [&](const Step<MB>& st) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint4 a = st.x[0][p], b = MB > 1 ? st.x[MB - 1][p] : zero;
#pragma unroll
            for (int n = 0; n < 2; ++n)
                mma_bf16(acc[n], a.x, b.x, a.y, b.y, st.w[n][p].x, st.w[n][p].y);
#pragma unroll
            for (int n = 0; n < 2; ++n)
                mma_bf16(acc[n], a.z, b.z, a.w, b.w, st.w[n][p].z, st.w[n][p].w);
        }
    };
    // steps of loads in flight per warp: as many as the registers hold (one more
    // spilled, and took 27 us instead of 23 at M = 16, K = 14336, N = 4096)
    constexpr int DEPTH = MB == 1 ? 3 : 2;
    Step<MB> ring[DEPTH];
    const int full = min(s1, g.K / kBK);      // whole steps of this warp: [s0, full)
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        if (s0 + d < full) load(ring[d], s0 + d);
    for (int s = s0; s < full; s += DEPTH) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            if (s + d < full) mul(ring[d]);
            if (s + d + DEPTH < full) load(ring[d], s + d + DEPTH);
        }
    }
    if (s1 > full && s1 > s0) {
        // the last step has K % 64 columns, whole 16-byte pieces of them
        const long long k = static_cast<long long>(s1 - 1) * kBK;
        Step<MB> st;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const bool in = k + 32 * p + 8 * t < g.K;
            st.w[0][p] = in ? ld_stream(reinterpret_cast<const uint4*>(w0 + k + 32 * p)) : zero;
            st.w[1][p] = in ? ld_stream(reinterpret_cast<const uint4*>(w1 + k + 32 * p)) : zero;
#pragma unroll
            for (int m = 0; m < MB; ++m)
                st.x[m][p] = in ? __ldg(reinterpret_cast<const uint4*>(xr[m] + k + 32 * p)) : zero;
        }
        mul(st);
    }

    // sums over the warps that share the rows, in order, then over the cluster
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        *reinterpret_cast<float2*>(&sums[warp][gq][8 * n + 2 * t]) = make_float2(acc[n][0], acc[n][1]);
        *reinterpret_cast<float2*>(&sums[warp][gq + 8][8 * n + 2 * t]) =
            make_float2(acc[n][2], acc[n][3]);
    }
    __syncthreads();
    if (wk > 1) {
        for (int q = 0; q < wr; ++q) {     // 256 elements a row group, one a thread
            float v = 0.0f;
            for (int j = 0; j < wk; ++j) v += (&sums[q * wk + j][0][0])[threadIdx.x];
            (&sums[q * wk][0][0])[threadIdx.x] = v;
        }
        __syncthreads();
    }
    if (csize > 1) cluster_sync();
    // outputs of the block: wr row groups x M tokens x `per` columns, dealt over
    // the cluster's blocks
    const int total = wr * g.M * per;
    for (int f = static_cast<int>(rank) * kFewThreads + threadIdx.x; f < total;
         f += csize * kFewThreads) {
        const int c = f % per, m = f / per % g.M, q = f / (per * g.M);
        const int col = (block * wr + q) * per + c;
        if (col >= g.N) continue;
        const uint32_t a = smem_u32(&sums[q * wk][m][c]);
        float z = 0.0f, up = 0.0f;
        if (csize == 1) {
            z = sums[q * wk][m][c];
            if (g.gated) up = sums[q * wk][m][c + 8];
        } else {
            for (int r = 0; r < csize; ++r) {
                z += ld_cluster(cluster_addr(a, r));
                if (g.gated) up += ld_cluster(cluster_addr(a + 32, r));
            }
        }
        float v[1] = {z + load_bias(g, col)};
        activate(v, g.act);
        if (g.gated) v[0] *= up + load_bias(g, g.N + col);
        if (g.residual) v[0] += load_res(g, m, col);
        store_out(g, m, col, v[0]);
    }
    if (csize > 1) cluster_sync();     // peers may still be reading this block's sums
}

// ================================================================= tile
struct Maps {
    CUtensorMap x;     // box 64 x 128 rows
    CUtensorMap w;     // box 64 x rows of one weight copy
};

constexpr int kTileThreads = 256;
constexpr int kTileM = 128;
// two blocks fit on an SM
template <int BN> __host__ __device__ constexpr int tile_stages() { return BN == 64 ? 4 : 3; }

template <int BN>
__host__ __device__ constexpr int tile_stage_bytes() { return (kTileM + BN) * kRowBytes; }
template <int BN>
__host__ __device__ constexpr int tile_smem_bytes() {
    const int ring = tile_stages<BN>() * tile_stage_bytes<BN>(), acc = kTileM * (BN + 4) * 4;
    return 1024 + (ring > acc ? ring : acc);
}

struct TileCtl {
    uint64_t full[4];
    uint64_t empty[4];
    uint64_t done;
    uint32_t tmem;
    int abort;
    uint32_t issued;
    alignas(16) float bias[128];       // of the tile's accumulator columns
};

// The rows of a tile that this block of a cluster of CS finishes: four columns
// a thread, a row's threads side by side, each adding the blocks' sums in rank
// order.  All of an item's loads are in flight together, and those of a few
// items (one after the other an item took 1 us).
template <int BN, int CS>
__device__ __forceinline__ void finish_rows(const Args& g, const float* bias, const float* sacc,
                                            int m0, int n0, int rank) {
    constexpr int LD = BN + 4, U = 8 / CS;
    const int per = g.gated ? BN / 2 : BN, lq = 31 - __clz(per / 4);
    const int rows = min(kTileM, g.M - m0);
    const int r0 = rows * rank / CS, items = (rows * (rank + 1) / CS - r0) << lq;
    uint32_t from[CS];
#pragma unroll
    for (int q = 0; q < CS; ++q) from[q] = cluster_addr(smem_u32(sacc), q);
    for (int f0 = threadIdx.x; f0 < items; f0 += U * kTileThreads) {
        int r[U], c[U];
        bool in[U];
        float4 v[U][CS], w[U][CS], res[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int f = f0 + u * kTileThreads;
            r[u] = r0 + (f >> lq);
            c[u] = (f & ((1 << lq) - 1)) * 4;
            in[u] = f < items && n0 + c[u] < g.N;
            res[u] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (!in[u]) continue;
            const uint32_t o = (r[u] * LD + c[u]) * 4;
#pragma unroll
            for (int q = 0; q < CS; ++q) {
                v[u][q] = ld_cluster4(from[q] + o);
                if (g.gated) w[u][q] = ld_cluster4(from[q] + o + BN / 2 * 4);
            }
            if (g.residual) res[u] = res4(g, m0 + r[u], n0 + c[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!in[u]) continue;
            float z[4], up[4];
            const float4 b = *reinterpret_cast<const float4*>(bias + c[u]);
            float4 t = v[u][0];
#pragma unroll
            for (int q = 1; q < CS; ++q)
                t = make_float4(t.x + v[u][q].x, t.y + v[u][q].y, t.z + v[u][q].z, t.w + v[u][q].w);
            z[0] = t.x + b.x;
            z[1] = t.y + b.y;
            z[2] = t.z + b.z;
            z[3] = t.w + b.w;
            activate(z, g.act);
            if (g.gated) {
                const float4 d = *reinterpret_cast<const float4*>(bias + BN / 2 + c[u]);
                t = w[u][0];
#pragma unroll
                for (int q = 1; q < CS; ++q)
                    t = make_float4(t.x + w[u][q].x, t.y + w[u][q].y, t.z + w[u][q].z,
                                    t.w + w[u][q].w);
                up[0] = t.x + d.x;
                up[1] = t.y + d.y;
                up[2] = t.z + d.z;
                up[3] = t.w + d.w;
#pragma unroll
                for (int i = 0; i < 4; ++i) z[i] *= up[i];
            }
            store4(g, m0 + r[u], n0 + c[u],
                   make_float4(z[0] + res[u].x, z[1] + res[u].y, z[2] + res[u].z, z[3] + res[u].w));
        }
    }
}

template <int BN>
__global__ void __launch_bounds__(kTileThreads, 2)
    linear_tile_kernel(const __grid_constant__ Maps maps, const Args g, int csize) {
    extern __shared__ uint8_t dsmem_raw[];
    __shared__ TileCtl ctl;
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int STAGE = tile_stage_bytes<BN>(), S = tile_stages<BN>();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = csize > 1 ? cluster_ctarank() : 0;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        mbar_init(&ctl.done, 1);
        fence_mbar_init();
        ctl.abort = 0;
        ctl.issued = 0;
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 2) {
        tmem_alloc(&ctl.tmem, BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    pdl_wait();
    pdl_trigger();

    const int per = g.gated ? BN / 2 : BN;              // output columns of a tile
    const int tiles_n = (g.N + per - 1) / per;
    const int tile = blockIdx.x / csize;
    const int m0 = tile / tiles_n * kTileM, n0 = tile % tiles_n * per;
    const int KB = (g.K + kBK - 1) / kBK;
    const int kb0 = static_cast<int>(static_cast<long long>(KB) * rank / csize);
    const int kb1 = static_cast<int>(static_cast<long long>(KB) * (rank + 1) / csize);

    if (warp == 0 && lane == 0) {
        uint32_t issued = 0;
        for (int kb = kb0; kb < kb1; ++kb, ++issued) {
            if (g.withheld(rank, issued)) break;
            const uint32_t st = issued % S, use = issued / S;
            if (use > 0 &&
                !mbar_wait(&ctl.empty[st], (use - 1) & 1u, &ctl.abort, g.wait_limit())) {
                report_timeout(g);
                *reinterpret_cast<volatile int*>(&ctl.abort) = 1;
                break;
            }
            uint8_t* a = base + st * STAGE;
            mbar_arrive_expect_tx(&ctl.full[st], STAGE);
            tma_load_2d(a, &maps.x, &ctl.full[st], kb * kBK, m0, kEvictNormal);
            uint8_t* b = a + kTileM * kRowBytes;
            tma_load_2d(b, &maps.w, &ctl.full[st], kb * kBK, n0, kEvictNormal);
            if (g.gated)
                tma_load_2d(b + BN / 2 * kRowBytes, &maps.w, &ctl.full[st], kb * kBK, g.N + n0,
                            kEvictNormal);
        }
        ctl.issued = issued;
    } else if (warp == 1 && lane == 0) {
        const uint32_t idesc = make_idesc<false>(kTileM, BN);
        for (int kb = kb0; kb < kb1; ++kb) {
            const uint32_t i = kb - kb0, st = i % S;
            if (!mbar_wait(&ctl.full[st], (i / S) & 1u, &ctl.abort, g.wait_limit())) {
                report_timeout(g);
                *reinterpret_cast<volatile int*>(&ctl.abort) = 1;
                break;
            }
            tc_fence_after();
            const uint64_t ad = sw128_desc(smem_u32(base + st * STAGE));
            const uint64_t bd = sw128_desc(smem_u32(base + st * STAGE + kTileM * kRowBytes));
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
                umma<false>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (i | kk) ? 1u : 0u);
            umma_commit(&ctl.empty[st]);
        }
        umma_commit(&ctl.done);
    } else if (warp >= 4 && threadIdx.x - 128 < BN) {
        const int i = threadIdx.x - 128, c = n0 + (g.gated && i >= BN / 2 ? i - BN / 2 : i);
        ctl.bias[i] = c < g.N ? load_bias(g, g.gated && i >= BN / 2 ? g.N + c : c) : 0.0f;
    }
    __syncwarp();
    // the accumulator is whole (or the wait ran out): every thread, so that
    // none leaves while products read the ring
    if (!mbar_wait(&ctl.done, 0, nullptr, 2 * g.wait_limit())) report_timeout(g);
    tc_fence_after();
    __syncthreads();
    if (*reinterpret_cast<volatile int*>(&ctl.abort) && threadIdx.x == 0) {
        // copies in flight land before the ring is written over
        const uint32_t n = ctl.issued, first = n > S ? n - S : 0;
        for (uint32_t i = first; i < n; ++i)
            mbar_wait(&ctl.full[i % S], (i / S) & 1u, nullptr, kDrainLimitNs);
    }
    __syncthreads();

    const int q = warp & 3, half = warp >> 2;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16);
    if (csize == 1) {
        // out straight from the accumulator, a row per lane
        float* buf = reinterpret_cast<float*>(base) + warp * kBufFloats;    // (of the ring)
        const int span = per / 2;                      // this warp's output columns
        for (int c = half * span; c < (half + 1) * span && n0 + c < g.N; c += 16) {
            float v[16], u[16];
            tmem_ld16(ta + c, v);
            if (g.gated) tmem_ld16(ta + BN / 2 + c, u);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                v[i] += ctl.bias[c + i];
                if (g.gated) u[i] += ctl.bias[BN / 2 + c + i];
            }
            finish16(g, buf, m0 + 32 * q, n0 + c, v, u);
        }
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
        if (warp == 2) tmem_dealloc(tmem, BN);
        return;
    }
    // accumulator -> shared memory, rows of BN + 4 floats (a lane per row: the 4
    // keep 16-byte stores of 8 lanes on different banks)
    constexpr int LD = BN + 4;
    float* sacc = reinterpret_cast<float*>(base);
    {
        float* row = sacc + (32 * q + lane) * LD + half * (BN / 2);
#pragma unroll
        for (int c = 0; c < BN / 2; c += 16) {
            float v[16];
            tmem_ld16(ta + half * (BN / 2) + c, v);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(row + c + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    if (warp == 2) tmem_dealloc(tmem, BN);
    // the rows are dealt over the cluster's blocks
    if (csize == 2) finish_rows<BN, 2>(g, ctl.bias, sacc, m0, n0, rank);
    else if (csize == 4) finish_rows<BN, 4>(g, ctl.bias, sacc, m0, n0, rank);
    else finish_rows<BN, 8>(g, ctl.bias, sacc, m0, n0, rank);
    cluster_sync();                    // peers may still be reading this block's sums
}

// ================================================================= pair
constexpr int kPairThreads = 384;
constexpr int kEpiWarp0 = 4;                 // warps 4..11
constexpr int kEpiThreads = 256;

// 256 columns: 128-column tiles are bound by the shared memory that feeds the
// MMAs (581 us instead of 410 at M = 4096, K = 14336, N = 4096)
constexpr int kPairN = 256;
constexpr int kPairStageBytes = (128 + kPairN / 2) * kRowBytes;   // per CTA: 128 token rows,
                                                                  // half of the weight rows
constexpr int kPairStages = 6;
// behind the ring the epilogue warps' buffers for rows that are not aligned
constexpr int kPairSmemBytes = 1024 + kPairStages * kPairStageBytes + 8 * kBufFloats * 4;

struct PairCtl {
    uint64_t full[kPairStages];
    uint64_t empty[kPairStages];
    uint64_t tfull[2];
    uint64_t tempty[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    uint32_t prod_pos, mma_pos;        // stages filled (by this CTA), and read
    alignas(16) float bias[2][kPairN];
};

// A wait that ran out ends the cluster's work together: every CTA's waits return,
// and after the last cluster barrier all of them know.
template <int CTAS>
__device__ __forceinline__ void abort_cluster(const Args& g, PairCtl& ctl) {
    report_timeout(g);
#pragma unroll
    for (int r = 0; r < CTAS; ++r)
        asm volatile("st.shared::cluster.u32 [%0], 1;" ::"r"(cluster_addr(smem_u32(&ctl.abort), r))
                     : "memory");
}

// Then the products that a pair has issued end, and its copies land (bounded),
// before its memory goes.  Of the stages that the products have not read some may
// have been filled by one CTA only: the even one, on whose barriers both CTAs'
// copies complete, adds what the phase lacks of the other's.
__device__ __forceinline__ void drain_pair(PairCtl& ctl, int warp, int lane, int side, int rank) {
    if (side != 0 || lane != 0) return;
    if (warp == 1) {
        umma_commit_pair_local(&ctl.drain);
        mbar_wait(&ctl.drain, 0, nullptr, kDrainLimitNs);
    } else if (warp == 0) {
        const uint32_t own = ctl.prod_pos;
        uint32_t peer;
        asm volatile("ld.shared::cluster.u32 %0, [%1];"
                     : "=r"(peer)
                     : "r"(cluster_addr(smem_u32(&ctl.prod_pos), rank + 1))
                     : "memory");
        for (uint32_t it = ctl.mma_pos; it < max(own, peer); ++it) {
            uint64_t* bar = &ctl.full[it % kPairStages];
            if (it >= own)
                mbar_arrive_expect_tx(bar, kPairStageBytes);
            else if (it >= peer)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                                 smem_u32(bar)),
                             "r"(kPairStageBytes)
                             : "memory");
            mbar_wait(bar, (it / kPairStages) & 1u, nullptr, kDrainLimitNs);
        }
    }
}

// Tile t of the rasterised order: groups of 8 row tiles, in a group column tile
// by column tile, so that the tiles in flight share operands in L2.
__device__ __forceinline__ void pair_tile(int t, int tm, int tn, int& m, int& n) {
    const int per = 8 * tn, grp = t / per, first = grp * 8;
    const int h = min(8, tm - first);
    const int r = t - grp * per;
    m = first + r % h;
    n = r / h;
}

// WIDE: rows aligned to 16 bytes and N a multiple of 16.  The other form carries
// the code for what is not, which costs its epilogue a tenth (instruction fetch).
template <bool WIDE>
__global__ void __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ Maps maps, const Args g) {
    extern __shared__ uint8_t dsmem_raw[];
    __shared__ PairCtl ctl;
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int BN = kPairN, STAGE = kPairStageBytes, S = kPairStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl.tfull[i], 1);
            mbar_init(&ctl.tempty[i], 2 * (kEpiThreads / 32));
        }
        mbar_init(&ctl.drain, 1);
        fence_mbar_init();
        ctl.abort = 0;
        ctl.prod_pos = ctl.mma_pos = 0;
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 2) {
        tmem_alloc_pair(&ctl.tmem, 2 * BN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();          // the peer's barriers are initialised
    const uint32_t tmem = ctl.tmem;
    pdl_wait();
    pdl_trigger();

    const int per = g.gated ? BN / 2 : BN;
    const int tm = (g.M + 255) / 256, tn = (g.N + per - 1) / per, tiles = tm * tn;
    const int P = gridDim.x >> 1, p0 = blockIdx.x >> 1;
    const int KB = (g.K + kBK - 1) / kBK;
    auto raise = [&]() { abort_cluster<2>(g, ctl); };

    if (warp == 0) {
        if (lane == 0) {
            // both CTAs copy their own rows; the copies complete on the rank-0
            // CTA's barrier, which its thread arms for both.  Weight rows of a
            // gated tile: the gate rows on rank 0, the up rows on rank 1.
            uint32_t it = 0;
            int st = 0;
            uint32_t par = 1;
            bool ok = true;
            for (int t = p0; t < tiles && ok; t += P) {
                int m, n;
                pair_tile(t, tm, tn, m, n);
                const int xrow = m * 256 + rank * 128;
                const int wrow = g.gated ? rank * g.N + n * per : n * BN + rank * (BN / 2);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    if (g.withheld(rank, it)) {
                        ok = false;
                        break;
                    }
                    if (!mbar_wait(&ctl.empty[st], par, &ctl.abort, g.wait_limit())) {
                        raise();
                        ok = false;
                        break;
                    }
                    uint8_t* a = base + st * STAGE;
                    if (rank == 0) mbar_arrive_expect_tx(&ctl.full[st], 2 * STAGE);
                    tma_load_2d_pair(a, &maps.x, &ctl.full[st], kb * kBK, xrow, kEvictNormal);
                    tma_load_2d_pair(a + 128 * kRowBytes, &maps.w, &ctl.full[st], kb * kBK, wrow,
                                     kEvictNormal);
                    if (++st == S) {
                        st = 0;
                        par ^= 1u;
                    }
                }
            }
            ctl.prod_pos = it;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            const uint32_t idesc = make_idesc<false>(256, BN);
            const uint64_t a0 = sw128_desc(smem_u32(base));
            const uint64_t b0 = sw128_desc(smem_u32(base + 128 * kRowBytes));
            int st = 0;
            uint32_t ph = 0, it = 0, i = 0;
            bool ok = true;
            for (int t = p0; t < tiles && ok; t += P, ++i) {
                const int acc = i & 1;
                if (!mbar_wait(&ctl.tempty[acc], ((i >> 1) & 1u) ^ 1u, &ctl.abort,
                               g.wait_limit())) {
                    raise();
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem + acc * BN;
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    if (!mbar_wait(&ctl.full[st], ph, &ctl.abort, g.wait_limit())) {
                        raise();
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = a0 + static_cast<uint32_t>(st * (STAGE >> 4));
                    const uint64_t bd = b0 + static_cast<uint32_t>(st * (STAGE >> 4));
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        umma_pair<false>(d, ad + 2 * kk, bd + 2 * kk, idesc, (kb | kk) ? 1u : 0u);
                    umma_commit_pair(&ctl.empty[st]);
                    if (++st == S) {
                        st = 0;
                        ph ^= 1u;
                    }
                }
                if (ok) umma_commit_pair(&ctl.tfull[acc]);
            }
            ctl.mma_pos = it;
        }
        __syncwarp();
    } else if (warp >= kEpiWarp0) {
        const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const int et = threadIdx.x - kEpiWarp0 * 32;
        float* buf = reinterpret_cast<float*>(base + S * STAGE) + (warp - kEpiWarp0) * kBufFloats;
        uint32_t i = 0;
        for (int t = p0; t < tiles; t += P, ++i) {
            const int acc = i & 1;
            int m, n;
            pair_tile(t, tm, tn, m, n);
            const int n0 = n * per;
            // this tile's bias, in accumulator column order
            if (et < BN) {
                const int c = n0 + (g.gated && et >= BN / 2 ? et - BN / 2 : et);
                ctl.bias[acc][et] =
                    c < g.N ? load_bias(g, g.gated && et >= BN / 2 ? g.N + c : c) : 0.0f;
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            const long long row = static_cast<long long>(m) * 256 + rank * 128 + 32 * q + lane;
            const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + acc * BN;
            const float4* bias = reinterpret_cast<const float4*>(ctl.bias[acc]);
            const int span = per / 2;         // this warp's output columns
            const int cb = half * span, ce = min((half + 1) * span, g.N - n0);
            uint32_t qa[8], qb[8];
            const bool res = g.residual != nullptr && row < g.M;
            if (cb < ce && res && (WIDE || wide16(g, n0 + cb))) res16(g, row, n0 + cb, qa, qb);
            // (after a fault the waits return at once and the loop runs on, so
            // that all epilogue warps meet at the same barriers)
            if (!mbar_wait(&ctl.tfull[acc], (i >> 1) & 1u, &ctl.abort, g.wait_limit())) raise();
            tc_fence_after();
            // 16 columns at a time; the next ones' accumulators and residual are
            // on their way while these are worked on
            uint32_t r0[16], r1[16];
            if (cb < ce) {
                tmem_ld16_async(ta + cb, r0);
                if (g.gated) tmem_ld16_async(ta + BN / 2 + cb, r1);
            }
            for (int c = cb; c < ce; c += 16) {
                tmem_wait16(r0);
                if (g.gated) tmem_wait16(r1);
                float v[16], u[16], w[16];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 b = bias[c / 4 + j];
                    v[4 * j] = __uint_as_float(r0[4 * j]) + b.x;
                    v[4 * j + 1] = __uint_as_float(r0[4 * j + 1]) + b.y;
                    v[4 * j + 2] = __uint_as_float(r0[4 * j + 2]) + b.z;
                    v[4 * j + 3] = __uint_as_float(r0[4 * j + 3]) + b.w;
                }
                if (g.gated) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 b = bias[(BN / 2 + c) / 4 + j];
                        u[4 * j] = __uint_as_float(r1[4 * j]) + b.x;
                        u[4 * j + 1] = __uint_as_float(r1[4 * j + 1]) + b.y;
                        u[4 * j + 2] = __uint_as_float(r1[4 * j + 2]) + b.z;
                        u[4 * j + 3] = __uint_as_float(r1[4 * j + 3]) + b.w;
                    }
                }
                const bool wide = WIDE || wide16(g, n0 + c);
                if (res && wide) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) w[j] = 0.0f;
                    add_res16(g, w, qa, qb);
                }
                if (c + 16 < ce) {
                    tmem_ld16_async(ta + c + 16, r0);
                    if (g.gated) tmem_ld16_async(ta + BN / 2 + c + 16, r1);
                    if (res && (WIDE || wide16(g, n0 + c + 16))) res16(g, row, n0 + c + 16, qa, qb);
                }
                activate(v, g.act);
                if (g.gated) {
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] *= u[j];
                }
                if (!wide) {
                    if constexpr (!WIDE) some16(g, buf, row - lane, n0 + c, v);
                } else if (row < g.M) {
                    if (res) {
#pragma unroll
                        for (int j = 0; j < 16; ++j) v[j] += w[j];
                    }
                    store16(g, row, n0 + c, v);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_leader(&ctl.tempty[acc]);
        }
    }

    __syncthreads();
    cluster_sync();
    if (*reinterpret_cast<volatile int*>(&ctl.abort)) {        // in both CTAs or none
        drain_pair(ctl, warp, lane, rank, rank);
        __syncwarp();
        __syncthreads();
        cluster_sync();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 2 * BN);
    }
}

// ================================================================= split
// The pair kernel's 256 x 256 tile, one per cluster of two pairs that split K:
// for long products with too few such tiles for all pairs.  The CTAs of the same
// 128 rows then finish half of the columns each: either copies its sums of the
// other's half into that one's ring, which has run dry (as bulk copies; lane by
// lane, with 16-byte remote stores, it took 3 us).
constexpr int kSplitW = kPairN / 2;            // accumulator columns of a share
constexpr int kSplitLD = kSplitW + 4;          // the 4 keep 16-byte stores of 8 lanes on
                                               // different banks
constexpr int kShareBytes = 128 * kSplitLD * 4;
static_assert(2 * kShareBytes <= kPairStages * kPairStageBytes, "two shares fit into the ring");
__device__ __forceinline__ void umma_commit_pair_of(uint64_t* bar, int pair) {
    const uint16_t mask = static_cast<uint16_t>(0x3 << (2 * pair));
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)),
        "h"(mask)
        : "memory");
}

__global__ void __launch_bounds__(kPairThreads, 1)
    linear_split_kernel(const __grid_constant__ Maps maps, const Args g) {
    extern __shared__ uint8_t dsmem_raw[];
    __shared__ PairCtl ctl;
    __shared__ uint64_t arrived;              // the other pair's share
    uint8_t* base = reinterpret_cast<uint8_t*>(
        (reinterpret_cast<uintptr_t>(dsmem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    constexpr int BN = kPairN, STAGE = kPairStageBytes, S = kPairStages;
    constexpr int W = kSplitW, LD = kSplitLD;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank()), side = rank & 1, pair = rank >> 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&ctl.full[i], 1);
            mbar_init(&ctl.empty[i], 1);
        }
        mbar_init(&ctl.tfull[0], 1);
        mbar_init(&ctl.drain, 1);
        mbar_init(&arrived, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&arrived, kShareBytes);
        ctl.abort = 0;
        ctl.prod_pos = ctl.mma_pos = 0;
        tma_prefetch_desc(&maps.x);
        tma_prefetch_desc(&maps.w);
    }
    if (warp == 2) {
        tmem_alloc_pair(&ctl.tmem, BN);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();          // the peers' barriers are initialised
    const uint32_t tmem = ctl.tmem;
    pdl_wait();
    pdl_trigger();

    const int per = g.gated ? BN / 2 : BN;
    const int tm = (g.M + 255) / 256, t = blockIdx.x / 4;
    const int m = t % tm, n0 = t / tm * per;
    const int KB = (g.K + kBK - 1) / kBK;
    const int kb0 = pair ? KB / 2 : 0, kb1 = pair ? KB : KB / 2;
    auto raise = [&]() { abort_cluster<4>(g, ctl); };
    const int q = warp & 3, half = (warp - kEpiWarp0) >> 2;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16);

    if (warp == 0) {
        if (lane == 0) {
            // as in the pair kernel
            const int xrow = m * 256 + side * 128;
            const int wrow = g.gated ? side * g.N + n0 : n0 + side * (BN / 2);
            uint32_t it = 0;
            int st = 0;
            uint32_t par = 1;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (g.withheld(rank, it)) break;
                if (!mbar_wait(&ctl.empty[st], par, &ctl.abort, g.wait_limit())) {
                    raise();
                    break;
                }
                uint8_t* a = base + st * STAGE;
                if (side == 0) mbar_arrive_expect_tx(&ctl.full[st], 2 * STAGE);
                tma_load_2d_pair(a, &maps.x, &ctl.full[st], kb * kBK, xrow, kEvictNormal);
                tma_load_2d_pair(a + 128 * kRowBytes, &maps.w, &ctl.full[st], kb * kBK, wrow,
                                 kEvictNormal);
                if (++st == S) {
                    st = 0;
                    par ^= 1u;
                }
            }
            ctl.prod_pos = it;
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && side == 0) {
            const uint32_t idesc = make_idesc<false>(256, BN);
            const uint64_t a0 = sw128_desc(smem_u32(base));
            const uint64_t b0 = sw128_desc(smem_u32(base + 128 * kRowBytes));
            int st = 0;
            uint32_t ph = 0, it = 0;
            bool ok = true;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                if (!mbar_wait(&ctl.full[st], ph, &ctl.abort, g.wait_limit())) {
                    raise();
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t ad = a0 + static_cast<uint32_t>(st * (STAGE >> 4));
                const uint64_t bd = b0 + static_cast<uint32_t>(st * (STAGE >> 4));
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    umma_pair<false>(tmem, ad + 2 * kk, bd + 2 * kk, idesc, (it | kk) ? 1u : 0u);
                umma_commit_pair_of(&ctl.empty[st], pair);
                if (++st == S) {
                    st = 0;
                    ph ^= 1u;
                }
            }
            if (ok) umma_commit_pair_of(&ctl.tfull[0], pair);
            ctl.mma_pos = it;
        }
        __syncwarp();
    } else if (warp >= kEpiWarp0) {
        // the tile's bias, in accumulator column order
        const int et = threadIdx.x - kEpiWarp0 * 32;
        if (et < BN) {
            const int c = n0 + (g.gated && et >= BN / 2 ? et - BN / 2 : et);
            ctl.bias[0][et] = c < g.N ? load_bias(g, g.gated && et >= BN / 2 ? g.N + c : c) : 0.0f;
        }
        if (!mbar_wait(&ctl.tfull[0], 0, &ctl.abort, g.wait_limit())) raise();
        tc_fence_after();
    }
    __syncthreads();
    // this CTA's ring is idle (or, after a fault, what is in it is of no account)
    asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
    // accumulator column of column l of share j: a gated share's first half are
    // gate columns, its second half their up columns
    auto column = [&](int j, int l) {
        return g.gated ? (l < W / 2 ? j * (W / 2) + l : BN / 2 + j * (W / 2) + l - W / 2) : j * W + l;
    };
    const int srow = 32 * q + lane;
    const float* const share = reinterpret_cast<float*>(base) + srow * LD;   // what arrives
    float* const sent = reinterpret_cast<float*>(base + kShareBytes) + srow * LD;
    if (warp >= kEpiWarp0) {
#pragma unroll
        for (int c = 0; c < W / 2; c += 16) {
            const int l = half * (W / 2) + c;
            float v[16];
            tmem_ld16(ta + column(pair ^ 1, l), v);
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                *reinterpret_cast<float4*>(sent + l + i) =
                    make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        fence_proxy_async_smem();
    }
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");      // all rings are
    if (warp >= kEpiWarp0) {
        // 32 rows are whole once both their warps are here
        asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory");
        if (half == 0 && lane == 0)
            bulk_to_cluster(cluster_addr(smem_u32(share), rank ^ 2), sent, kShareBytes / 4,
                            cluster_addr(smem_u32(&arrived), rank ^ 2));
        if (!mbar_wait(&arrived, 0, nullptr, g.wait_limit())) raise();
    }
    if (warp >= kEpiWarp0) {
        const int outs = g.gated ? W / 2 : W;              // output columns of a share
        const long long row0 = static_cast<long long>(m) * 256 + side * 128 + 32 * q;
        float* buf = reinterpret_cast<float*>(base + S * STAGE) + (warp - kEpiWarp0) * kBufFloats;
        auto total = [&](int l, float (&v)[16]) {
            const int at = column(pair, l);
            tmem_ld16(ta + at, v);
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const float4 o = *reinterpret_cast<const float4*>(share + l + i);
                v[i] += o.x;
                v[i + 1] += o.y;
                v[i + 2] += o.z;
                v[i + 3] += o.w;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] += ctl.bias[0][at + i];
        };
        for (int l = half * (outs / 2); l < (half + 1) * (outs / 2); l += 16) {
            const int col = n0 + pair * outs + l;
            if (col >= g.N) break;
            float v[16], u[16];
            total(l, v);
            if (g.gated) total(l + W / 2, u);
            finish16(g, buf, row0, col, v, u);
        }
    }
    tc_fence_before();
    cluster_sync();          // both CTAs of a pair have read their accumulators
    if (*reinterpret_cast<volatile int*>(&ctl.abort)) {        // in all CTAs or none
        drain_pair(ctl, warp, lane, side, rank);
        __syncwarp();
        __syncthreads();
        cluster_sync();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, BN);
    }
}

// ---- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// [rows, K] bf16 with row stride ld, copied in boxes of 64 columns x box_rows,
// swizzled; columns past K and rows past the end read as zero.
bool make_map(CUtensorMap* m, const void* ptr, int K, long long rows, long long ld, int box_rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
    const cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
    const cuuint32_t estr[2] = {1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr int kMaxDevices = 64;

// More than 48 KB of dynamic shared memory, once per device and kernel.
template <class K>
cudaError_t opt_in(K kern, int bytes, std::once_flag* once, cudaError_t* err) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::call_once(once[dev], [&] {
        err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    return err[dev];
}

template <class... KArgs, class... A>
cudaError_t launch(void (*kern)(KArgs...), long long grid, int threads, int smem, int cluster,
                   cudaStream_t s, A... a) {
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cluster;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, static_cast<KArgs>(a)...);
}

cudaError_t launch_few(const Args& g, int sms, cudaStream_t s) {
    const int per = g.gated ? 8 : 16;
    const long long groups = (static_cast<long long>(g.N) + per - 1) / per;
    const int steps = (g.K + kBK - 1) / kBK;
    // K is split until there are 16 warps per SM, or 2 steps a warp
    int split = 1;
    while (split < 64 && groups * split * 2 <= 16LL * sms && steps >= split * 4) split *= 2;
    const int wk = split < kFewWarps ? split : kFewWarps, csize = split / wk;
    const long long grid = (groups + kFewWarps / wk - 1) / (kFewWarps / wk) * csize;
    return g.M <= 8 ? launch(linear_few_kernel<1>, grid, kFewThreads, 0, csize, s, g, wk, csize)
                    : launch(linear_few_kernel<2>, grid, kFewThreads, 0, csize, s, g, wk, csize);
}

template <int BN>
cudaError_t launch_tile(const Args& g, int sms, cudaStream_t s) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    cudaError_t e = opt_in(linear_tile_kernel<BN>, tile_smem_bytes<BN>(), once, err);
    if (e != cudaSuccess) return e;
    const int per = g.gated ? BN / 2 : BN;
    const long long tiles = (static_cast<long long>(g.M) + kTileM - 1) / kTileM *
                            ((static_cast<long long>(g.N) + per - 1) / per);
    const int KB = (g.K + kBK - 1) / kBK;
    // blocks of a cluster split K while all find room on the SMs and each keeps
    // at least 4 k-blocks; 6 where it shares its SM, and 12 where it would not
    // without the first split (us, more / fewer blocks: M = K = 512, N = 4096 10.0 /
    // 7.5; M = 512, K = 1024, N = 4096 11.7 / 10.2; M = 256, K = 2048, N = 768 8.0 /
    // 7.4; but M = 64, K = N = 2880, 180 blocks of 11 k-blocks, 9.4 / 11.5)
    int csize = 1;
    while (csize < 8 && tiles * csize * 2 <= 2 * sms &&
           KB >= (tiles * csize * 2 <= sms ? csize * 8 : csize == 1 ? 24 : csize * 12))
        csize *= 2;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (!make_map(&maps.x, g.x, g.K, g.M, g.ldx, kTileM) ||
        !make_map(&maps.w, g.w, g.K, g.gated ? 2LL * g.N : g.N, g.ldw, g.gated ? BN / 2 : BN))
        return cudaErrorInvalidValue;
    return launch(linear_tile_kernel<BN>, tiles * csize, kTileThreads, tile_smem_bytes<BN>(), csize,
                  s, maps, g, csize);
}

template <bool WIDE>
cudaError_t launch_pair(const Args& g, int sms, cudaStream_t s) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t err[kMaxDevices];
    cudaError_t e = opt_in(linear_pair_kernel<WIDE>, kPairSmemBytes, once, err);
    if (e != cudaSuccess) return e;
    const int per = g.gated ? kPairN / 2 : kPairN;
    const long long tiles = (static_cast<long long>(g.M) + 255) / 256 *
                            ((static_cast<long long>(g.N) + per - 1) / per);
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidConfiguration;
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (!make_map(&maps.x, g.x, g.K, g.M, g.ldx, 128) ||
        !make_map(&maps.w, g.w, g.K, g.gated ? 2LL * g.N : g.N, g.ldw, kPairN / 2))
        return cudaErrorInvalidValue;
    const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
    return launch(linear_pair_kernel<WIDE>, pairs * 2, kPairThreads, kPairSmemBytes, 2, s, maps,
                  g);
}

// Clusters of four CTAs of the split kernel that run at the same time, per device
// (0: none; 33 on a B200, whose GPCs are no multiples of four SMs).
int split_clusters() {
    static std::once_flag once[kMaxDevices];
    static int count[kMaxDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    std::call_once(once[dev], [&] {
        if (cudaFuncSetAttribute(linear_split_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kPairSmemBytes) != cudaSuccess)
            return;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(4);
        cfg.blockDim = dim3(kPairThreads);
        cfg.dynamicSmemBytes = kPairSmemBytes;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = 4;
        at[0].val.clusterDim.y = 1;
        at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, linear_split_kernel, &cfg) == cudaSuccess)
            count[dev] = n;
        else
            cudaGetLastError();     // (the other kernels take the product)
    });
    return count[dev];
}

cudaError_t launch_split(const Args& g, long long tiles, cudaStream_t s) {
    Maps maps;
    memset(&maps, 0, sizeof(maps));
    if (!make_map(&maps.x, g.x, g.K, g.M, g.ldx, 128) ||
        !make_map(&maps.w, g.w, g.K, g.gated ? 2LL * g.N : g.N, g.ldw, kPairN / 2))
        return cudaErrorInvalidValue;
    return launch(linear_split_kernel, tiles * 4, kPairThreads, kPairSmemBytes, 4, s, maps, g);
}

}  // namespace

cudaError_t launch_linear(const LinearProblem& p, cudaStream_t s) {
    Args g{};
    static_cast<SelfTest&>(g) = self_test();
    g.M = p.M;
    g.N = p.N;
    g.K = p.K;
    g.act = p.act;
    g.gated = p.gated;
    g.x = static_cast<const __nv_bfloat16*>(p.x);
    g.w = static_cast<const __nv_bfloat16*>(p.w);
    g.ldx = p.ldx;
    g.ldw = p.ldw;
    g.ldr = p.ldr;
    g.ldo = p.ldo;
    g.bias = p.bias;
    g.bias_f32 = p.bias_f32;
    g.residual = p.residual;
    g.out = p.out;
    g.out_f32 = p.out_f32;
    g.status = p.status;
    const uintptr_t es = p.out_f32 ? 4 : 2;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.out) | (p.ldo * es) |
                           (p.residual ? reinterpret_cast<uintptr_t>(p.residual) | (p.ldr * es) : 0);
    g.vec = bits % 32 == 0 ? 32 : bits % 16 == 0 ? 16 : 0;
    const int sms = device_sm_count();
    if (p.M <= 16) return launch_few(g, sms, s);
    // Measured on B200 (us, pair / 128-wide / 64-wide tiles): M = 1024, K = N =
    // 4096 (64 pair tiles) 28 / 34 / 45; M = 512, K = 7168, N = 2 x 2048 (32) 40 /
    // 34 / 40; M = 128, K = 4096, N = 2 x 14336 58 / 49 / 60; M = 300, K = N = 2880
    // (69 128-wide tiles) 19 / 14.0 / 13.3; M = 4096, K = 2048, N = 128 (32) 14.6 /
    // 8.6 / 8.9.  So: pairs once half of them have a tile and its 256 rows are not
    // half empty; else 128-wide tiles once there is one for every second SM.
    const int per = p.gated ? 128 : 256;
    const long long t256 = (static_cast<long long>(p.M) + 255) / 256 *
                           ((static_cast<long long>(p.N) + per - 1) / per);
    // Rows that are not aligned make the epilogue count, which twice the warps of
    // the 128-wide tiles hide better unless K is long (us, pair / 128-wide: M = 554,
    // K = 128, N = 6602 29 / 12; M = 5000, K = 512, N = 1001 32 / 22, K = 2048 41 /
    // 38; M = 2500, N = 2041, K = 2048 41 / 39, K = 4096 58 / 59; M = 3000, K = 2000,
    // N = 2 x 3001 62 / 91: half as many outputs of the same products).
    if (p.M > 128 && t256 * 4 >= sms && (g.vec || p.K > (p.gated ? 1024 : 2048)))
        return g.vec && p.N % 16 == 0 ? launch_pair<true>(g, sms, s) : launch_pair<false>(g, sms, s);
    // Fewer such tiles: two pairs to each, where all are resident, K is long enough
    // to pay for their exchange, and there are too many 128-wide tiles for two
    // blocks of each to have SMs of their own (us, split / 128-wide: M = 512, K =
    // 7168, N = 2 x 2048 28 / 34; M = 512, N = 4096, K = 4096 20 / 23, K = 2048 15.3 /
    // 16.7; with the last 256 rows half empty M = 300, K = N = 4096 19 / 22; but with
    // 69 128-wide tiles, M = 300, N = 2880, K = 4096 18 / 16, K = 14336 42 / 35, where
    // 64-wide ones take 16 and 43; with 16 pair tiles, M = 256, K = N = 4096 16.7 /
    // 16.6).
    const bool waste = (p.M - 1) % 256 < 128;
    const long long t128 = (static_cast<long long>(p.M) + 127) / 128 *
                           ((static_cast<long long>(p.N) + per / 2 - 1) / (per / 2));
    if (p.M > 128 && t256 > 16 && t128 * 2 > sms && p.K >= (waste ? 4096 : 2048) &&
        t256 < split_clusters())
        return launch_split(g, t256, s);
    if (t128 * 2 >= sms || (t256 > 16 && p.K >= 4096)) return launch_tile<128>(g, sms, s);
    return launch_tile<64>(g, sms, s);
}

cudaError_t read_linear_status(int32_t* code, cudaStream_t s) {
    void* word = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&word, own_status);
    if (e == cudaSuccess) e = cudaMemcpyAsync(code, word, sizeof(*code), cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
    if (e == cudaSuccess && *code != 0) e = cudaMemsetAsync(word, 0, sizeof(*code), s);
    return e;
}

}  // namespace moe
