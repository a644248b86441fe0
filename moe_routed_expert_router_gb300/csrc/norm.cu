// Residual addition and root-mean-square norm with an optional 8-bit output,
// and its gradients (see include/moe_nvfp4.h for the formulas).
//
// A block takes a row and keeps it in registers over the reduction, so every
// input is read once and every output written once.  Bound by HBM (4096 x 7168
// bf16 with residual and E4M3_128 output 32.4 us, 94 % of the measured copy
// bandwidth; without the residual, three bytes a value, 8192 x 7168 37.2 us, 71 %,
// with 69 % of the issue slots taken).  What keeps it there is that the loads of the next row do
// not wait for the reduction of the present one: other blocks' in the forward
// pass, a ring in shared memory in the backward pass.  (A ring in the forward
// pass too: 33.7 against 34.3 us at 4096 x 7168, 20.8 against 20.1 at 4096 x 4096.)
#include <math.h>

#include <algorithm>
#include <mutex>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kMaxH = 16384;
constexpr int kMaxPieces = 4;         // 16-bit rows: 16-byte pieces a thread holds
constexpr int kRowThreads = kMaxH / kChunk / kMaxPieces;
constexpr int kWarpRows = 8;          // rows a block takes where a row takes a warp
constexpr int kWarpPieces = 32 * kMaxPieces;
constexpr float kMinAmax = 7.888609052210118e-31f;   // 2^-100

struct NormArgs {
    const void *x, *r, *w;
    int64_t xs, rs;
    int H;
    float inv_h, eps;
    void *sum, *y;
    uint8_t *q;
    void *scales;
    float *rstd;
};

// Minimum and maximum that keep a NaN; the maximum of magnitudes, three at a time.
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Sum of the warps' sums (at most 16), on every lane of either half of a warp.
__device__ __forceinline__ float half_sum(const float *red) {
    const int i = threadIdx.x & 15;
    float v = i < (int)(blockDim.x >> 5) ? red[i] : 0.0f;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sum over the threads of a row (a warp, or the block), the same on every
// thread; `red` holds 32 words, and two calls in a row use different ones.
template <bool kWarp> __device__ __forceinline__ float row_sum(float v, float *red) {
    v = warp_sum(v);
    if constexpr (kWarp) return v;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return half_sum(red);
}

// The sum of one value and the maximum of another, with one barrier.
__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
template <bool kWarp> __device__ __forceinline__ void row_sum_max(float &sum, float &top, float (&red)[2][32]) {
    sum = warp_sum(sum);
    top = warp_max_nan(top);
    if constexpr (kWarp) return;
    if ((threadIdx.x & 31) == 0) {
        red[0][threadIdx.x >> 5] = sum;
        red[1][threadIdx.x >> 5] = top;
    }
    __syncthreads();
    sum = half_sum(red[0]);
    const int i = threadIdx.x & 15;
    top = i < (int)(blockDim.x >> 5) ? red[1][i] : 0.0f;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
}

// Four fp32 -> four E4M3 bytes, round to nearest even, saturating; NaN -> 0x7F.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t out;
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(out) : "f"(a), "f"(b), "f"(c), "f"(d));
    return out;
}

// 1 / sqrt(mean + eps).
__device__ __forceinline__ float row_rstd(float sumsq, float inv_h, float eps) {
    return __frsqrt_rn(fmaf(sumsq, inv_h, eps));
}

// p = s * weight of one piece, in fp32 (exact for 16-bit rows), from f = s.
template <int DT> __device__ __forceinline__ void product8(float (&f)[8], const Raw8<DT> &w) {
    float g[8];
    widen8<DT>(w, g);
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(f, e, g[e], g[e + 1]);
}

// A group's scale, and the factor that takes its products to its codes: with top
// = amax p * rstd and a = max(top, 2^-100) a code is that of p * rstd * 448 / a,
// which is p * (448 / amax p).  Groups with top or amax p at the bound or below it
// (or with a NaN) take their products times rstd first, and then 448 / a: rstd *
// 448 / 2^-100 may leave fp32, and so may 448 / amax p, from 2^-119.2 down, where
// rstd is large.  `low` is min(amax p, top).
__device__ __forceinline__ float e4m3_factor(float amax_p, float top, float low) {
    return __fdiv_rn(448.0f, low > kMinAmax ? amax_p : max_nan(top, kMinAmax));
}
__device__ __forceinline__ void at_the_bound(float (&p)[8], float low, float rstd) {
    if (low > kMinAmax) return;
#pragma unroll
    for (int e = 0; e < 8; e += 2) mul2(p, e, rstd, rstd);
}
__device__ __forceinline__ float e4m3_scale(float top) { return __fdiv_rn(max_nan(top, kMinAmax), 448.0f); }

__device__ __forceinline__ float amax8(const float (&n)[8], float m) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) m = amax3(m, n[e], n[e + 1]);
    return m;
}

// s = round(x + r) of one piece: the type's own addition, one rounding of the
// exact sum.
template <int DT> __device__ __forceinline__ uint32_t add_word(uint32_t x, uint32_t r) {
    uint32_t s;
    if constexpr (DT == MOE_DTYPE_F32) return __float_as_uint(__fadd_rn(__uint_as_float(x), __uint_as_float(r)));
    if constexpr (DT == MOE_DTYPE_BF16) asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(s) : "r"(x), "r"(r));
    if constexpr (DT == MOE_DTYPE_F16) asm("add.rn.f16x2 %0, %1, %2;" : "=r"(s) : "r"(x), "r"(r));
    return s;
}
template <int DT> __device__ __forceinline__ Raw8<DT> add8(const Raw8<DT> &x, const Raw8<DT> &r) {
    Raw8<DT> s;
    s.a = make_uint4(add_word<DT>(x.a.x, r.a.x), add_word<DT>(x.a.y, r.a.y), add_word<DT>(x.a.z, r.a.z), add_word<DT>(x.a.w, r.a.w));
    if constexpr (DT == MOE_DTYPE_F32)
        s.b = make_uint4(add_word<DT>(x.b.x, r.b.x), add_word<DT>(x.b.y, r.b.y), add_word<DT>(x.b.z, r.b.z), add_word<DT>(x.b.w, r.b.w));
    return s;
}

// A row a block, or (short rows) a row a warp and eight of them a
// block: no block barrier, and short rows fill an SM.  Thread i of a row's n (a
// multiple of 32) holds pieces i, i + n, ..., so a warp's accesses are 512
// consecutive bytes of a 16-bit row, a 128-value group is 16 neighbouring lanes
// and a 32-value group is four.  All of a thread's loads are issued before the
// first use; what it holds over the reduction is the products p = s * weight.
template <int DT, int Q, int V, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kRowThreads) k_rms_norm(const NormArgs a, int64_t rows) {
    using T = typename RowType<DT>::T;
    __shared__ float red[2][32];
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x;
    const int n8 = a.H / kChunk, n = kWarp ? 32 : blockDim.x;
    const int64_t t = kWarp ? (int64_t)blockIdx.x * kWarpRows + (threadIdx.x >> 5) : blockIdx.x;
    // whether piece i is inside the row.  A block's are, but the last: n <=
    // n8 / V + 32 and n8 >= 32 V (V - 1) in every row_shape, so (V - 1) n <= n8; so
    // is the first half of a warp's, which has V pieces from n8 > 16 V on
    auto inside = [&](int i) { return i < (kWarp ? V / 2 : V - 1) || tid + i * n < n8; };
    Raw8<DT> s[V], u[V], w[V];
    pdl_wait();
    pdl_trigger();
    if (kWarp && t >= rows) return;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * n;
        s[i] = u[i] = w[i] = Raw8<DT>{};
        if (inside(i)) {
            s[i] = load8<DT>(static_cast<const T *>(a.x) + t * a.xs + c * kChunk);
            if (a.r) u[i] = load8<DT>(static_cast<const T *>(a.r) + t * a.rs + c * kChunk);
        }
    }
    float p[V][8], s0 = 0.0f, s1 = 0.0f, row_mul = 0.0f, row_low = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * n;
        if (inside(i)) w[i] = load8_shared<DT>(static_cast<const T *>(a.w) + c * kChunk);
        if (a.r) {
            s[i] = add8<DT>(s[i], u[i]);
            if (a.sum && inside(i)) store8<DT>(static_cast<T *>(a.sum) + t * a.H + c * kChunk, s[i]);
        }
        widen8<DT>(s[i], p[i]);
#pragma unroll
        for (int e = 0; e < 8; e += 2) fma2(s0, s1, p[i][e], p[i][e + 1], p[i][e], p[i][e + 1]);
        product8<DT>(p[i], w[i]);
        if constexpr (Q == MOE_QUANT_E4M3_ROW) row_mul = amax8(p[i], row_mul);
    }
    float sum = s0 + s1;
    if constexpr (Q == MOE_QUANT_E4M3_ROW) row_sum_max<kWarp>(sum, row_mul, red);
    else sum = row_sum<kWarp>(sum, red[0]);
    const float rstd = row_rstd(sum, a.inv_h, a.eps);
    if (a.rstd && tid == 0) a.rstd[t] = rstd;
    if constexpr (Q == MOE_QUANT_E4M3_ROW) {
        const float top = __fmul_rn(row_mul, rstd);
        row_low = min_nan(row_mul, top);
        row_mul = e4m3_factor(row_mul, top, row_low);
        if (tid == 0) static_cast<float *>(a.scales)[t] = e4m3_scale(top);
    }
    constexpr int kLanes = Q == MOE_QUANT_MXFP8 ? 4 : 16;      // of a group
    const int64_t group0 = t * ((n8 + kLanes - 1) / kLanes);
    auto group_max = [&](float m) {
#pragma unroll
        for (int o = kLanes / 2; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        return m;
    };
    // E4M3_128: lane i of a group's 16 does the divisions of its piece i, all
    // pieces' at once
    float low[V], factor = row_mul;
    if constexpr (Q == MOE_QUANT_E4M3_128) {
        const int mine = threadIdx.x & 15;
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float amax_p = group_max(amax8(p[i], 0.0f));
            low[i] = min_nan(amax_p, __fmul_rn(amax_p, rstd));
            if (mine == i) m = amax_p;
        }
        const float own = __fmul_rn(m, rstd);
        factor = e4m3_factor(m, own, min_nan(m, own));
        const int c = (tid & ~15) + mine * n;
        if (mine < V && c < n8) static_cast<float *>(a.scales)[group0 + c / 16] = e4m3_scale(own);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = tid + i * n;
        if (Q == MOE_QUANT_NONE || a.y) {
            float f[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = p[i][e];
#pragma unroll
            for (int e = 0; e < 8; e += 2) mul2(f, e, rstd, rstd);
            if (inside(i)) store8<DT>(static_cast<T *>(a.y) + t * a.H + c * kChunk, narrow8<DT>(f));
        }
        if constexpr (Q == MOE_QUANT_NONE) continue;
        float mul = factor;
        if constexpr (Q == MOE_QUANT_E4M3_ROW) at_the_bound(p[i], row_low, rstd);
        if constexpr (Q == MOE_QUANT_E4M3_128) {
            mul = __shfl_sync(0xffffffffu, factor, (threadIdx.x & 16) + i);
            at_the_bound(p[i], low[i], rstd);
        }
        if constexpr (Q == MOE_QUANT_MXFP8) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) mul2(p[i], e, rstd, rstd);
            // floor(log2(amax)) + 127 is the exponent field of a normal amax;
            // E4M3's largest exponent is 8
            const int field = (int)((__float_as_uint(group_max(amax8(p[i], 0.0f))) >> 23) & 0xFFu);
            const int byte = field == 255 ? 255 : max(field - 8, 0);
            mul = field == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(254 - byte) << 23);
            if (c < n8 && c % kLanes == 0) static_cast<uint8_t *>(a.scales)[group0 + c / kLanes] = (uint8_t)byte;
        }
        if (inside(i)) {
#pragma unroll
            for (int e = 0; e < 8; e += 2) mul2(p[i], e, mul, mul);
            const uint2 o = make_uint2(e4m3x4(p[i][0], p[i][1], p[i][2], p[i][3]), e4m3x4(p[i][4], p[i][5], p[i][6], p[i][7]));
            *reinterpret_cast<uint2 *>(a.q + t * a.H + c * kChunk) = o;
        }
    }
}

struct NormGradArgs {
    const void *gy, *s, *w, *gs;
    const float *rstd;
    int T, H;
    void *gin;
    float *part;    // [blocks][H]
};

// Backward: block b takes rows b, b + blocks, ...; a thread keeps its columns'
// weight gradient in registers over all of them, so the column sums cost one
// [blocks][H] store at the end.  Bound by HBM (8192 x 4096 bf16 42 us of the
// pass's 44.4, whose floor is 39.7; the rest adds up the blocks' sums).  With
// R = 2 the next row is on its way into shared memory while one is worked on
// (cp.async; a thread copies the pieces that it will use itself and overwrites
// only what it has used, so its own copies are all that it waits for); R = 1 is
// for rows of which two do not fit.  Short rows take a warp each, as in the
// forward pass; the eight warps' sums are then added in order.
//
// Piece i of a thread is one 16-byte word of a 16-bit row or two of an fp32
// row, n words apart: neighbouring lanes copy neighbouring words (8192 fp32
// rows of 4096: 83 us, with a thread's two words side by side 141 us).  Words
// past an fp32 row are zeros; a 16-bit piece past the row is passed over.
template <int DT, int V, int R, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 32 * kWarpRows : kRowThreads) k_rms_norm_backward(const NormGradArgs a) {
    using T = typename RowType<DT>::T;
    extern __shared__ __align__(16) uint4 smem[];     // a row's [R][gy, s, gs][V][words][n]
    __shared__ float red[2][32];
    const int tid = kWarp ? threadIdx.x & 31 : threadIdx.x, group = kWarp ? threadIdx.x >> 5 : 0;
    const int n = kWarp ? 32 : blockDim.x;
    constexpr int kWords = sizeof(Raw8<DT>) / 16, kWord = 8 / kWords;   // values a word
    const int arr = V * kWords * n, stage = (a.gs ? 3 : 2) * arr;
    uint4 *ring = smem + group * R * stage;
    auto col = [&](int i, int h) { return ((i * kWords + h) * n + tid) * kWord; };
    auto past = [&](int i) { return kWords == 1 && col(i, 0) >= a.H; };
    float gw[V][8];
    Raw8<DT> w[V];
    pdl_wait();
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < V; ++i) {
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[i][e] = 0.0f;
        w[i] = Raw8<DT>{};
#pragma unroll
        for (int h = 0; h < kWords; ++h)
            if (col(i, h) < a.H)
                (&w[i].a)[h] = ld16_shared(static_cast<const T *>(a.w) + col(i, h));
    }
    auto fetch = [&](int64_t t, int slot) {
        if (t < a.T) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                if (past(i)) continue;
#pragma unroll
                for (int h = 0; h < kWords; ++h) {
                    const bool on = kWords == 1 || col(i, h) < a.H;
                    const int64_t from = t * a.H + (on ? col(i, h) : 0);
                    uint4 *at = ring + slot * stage + (i * kWords + h) * n + tid;
                    copy16(at, static_cast<const T *>(a.gy) + from, on);
                    copy16(at + arr, static_cast<const T *>(a.s) + from, on);
                    if (a.gs) copy16(at + 2 * arr, static_cast<const T *>(a.gs) + from, on);
                }
            }
        }
        copy_commit();
    };
    const int64_t step = (int64_t)gridDim.x * (kWarp ? kWarpRows : 1);
    int64_t t = (int64_t)blockIdx.x * (kWarp ? kWarpRows : 1) + group;
    if constexpr (R == 2) fetch(t, 0);
    int slot = 0;
    for (int par = 0; t < a.T; t += step, par ^= 1) {
        const float rstd = a.rstd[t];
        fetch(t + (R - 1) * step, R == 2 ? slot ^ 1 : 0);
        copy_wait<R - 1>();
        Raw8<DT> g[V], s[V];
        float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (past(i)) continue;
            const uint4 *at = ring + slot * stage + i * kWords * n + tid;
            g[i] = take8<DT>(at, n);
            s[i] = take8<DT>(at + arr, n);
            float f[8], m[8], wf[8];
            widen8<DT>(g[i], f);
            widen8<DT>(s[i], m);
            widen8<DT>(w[i], wf);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2(m, e, rstd, rstd);
                fma2(gw[i][e], gw[i][e + 1], f[e], f[e + 1], m[e], m[e + 1]);
                mul2(f, e, wf[e], wf[e + 1]);
                fma2(d0, d1, f[e], f[e + 1], m[e], m[e + 1]);
            }
        }
        const float c1 = -(row_sum<kWarp>(d0 + d1, red[par]) / (float)a.H);
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (past(i)) continue;
            float f[8], m[8], wf[8], o[8];
            Raw8<DT> q{};
            if (a.gs) q = take8<DT>(ring + slot * stage + 2 * arr + i * kWords * n + tid, n);
            widen8<DT>(g[i], f);
            widen8<DT>(s[i], m);
            widen8<DT>(w[i], wf);
            widen8<DT>(q, o);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                mul2(m, e, rstd, rstd);
                mul2(f, e, wf[e], wf[e + 1]);
                fma2(f[e], f[e + 1], m[e], m[e + 1], c1, c1);
                fma2(o[e], o[e + 1], f[e], f[e + 1], rstd, rstd);
            }
            const Raw8<DT> out = narrow8<DT>(o);
#pragma unroll
            for (int h = 0; h < kWords; ++h)
                if (col(i, h) < a.H) st16(static_cast<T *>(a.gin) + t * a.H + col(i, h), (&out.a)[h]);
        }
        if constexpr (R == 2) slot ^= 1;
    }
    float *sums = kWarp ? reinterpret_cast<float *>(smem) + group * a.H : a.part + (int64_t)blockIdx.x * a.H;
    const bool vectors = (reinterpret_cast<uintptr_t>(sums) & 15u) == 0;   // grad_w itself may be less aligned
    if constexpr (kWarp) {
        copy_wait<0>();
        __syncthreads();                              // the ring is free: the warps' sums, [8][H]
    }
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int h = 0; h < kWords; ++h) {
            if (col(i, h) >= a.H) continue;
#pragma unroll
            for (int e = 0; e < kWord; e += 4) {
                float *at = sums + col(i, h) + e, *v = &gw[i][h * kWord + e];
                if (kWarp || vectors) {
                    *reinterpret_cast<float4 *>(at) = make_float4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) at[k] = v[k];
                }
            }
        }
    if constexpr (kWarp) {
        __syncthreads();
        for (int h = threadIdx.x; h < a.H; h += blockDim.x) {
            float v = 0.0f;
#pragma unroll
            for (int g = 0; g < kWarpRows; ++g) v += reinterpret_cast<float *>(smem)[g * a.H + h];
            a.part[(int64_t)blockIdx.x * a.H + h] = v;
        }
    }
}

// grad_w[h] = sum of the blocks' partial sums: thread (i, j) adds every 64th
// block's from j on, four columns wide, then the 64 sums are added in order,
// eight by eight.  The partial sums come from L2 and the launch overlaps the end
// of the one before, so this is latency, 2 to 3 us: every thread's loads are one
// round (1216 rows of 2048: the pass 8.5 us; 32 groups of two rounds 9.5).
constexpr int kColumnGroups = 64;

__global__ void __launch_bounds__(8 * kColumnGroups) k_rms_norm_grad_w(const float *part, int blocks, int H, float *gw) {
    __shared__ float4 s[kColumnGroups][8];
    __shared__ float t[8][32];
    const int i = threadIdx.x & 7, j = threadIdx.x >> 3;
    const int h = blockIdx.x * 32 + i * 4;
    pdl_wait();
    pdl_trigger();
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h < H) {
#pragma unroll 5
        for (int b = j; b < blocks; b += kColumnGroups) {
            const float4 p = *reinterpret_cast<const float4 *>(part + (int64_t)b * H + h);
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
    }
    s[j][i] = v;
    __syncthreads();
    const float *c = reinterpret_cast<const float *>(s) + (threadIdx.x & 31);
    const int w = threadIdx.x >> 5;
    if (w < 8) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kColumnGroups / 8; ++k) sum += c[(w * (kColumnGroups / 8) + k) * 32];
        t[w][threadIdx.x & 31] = sum;
    }
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < H) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += t[k][threadIdx.x];
        gw[blockIdx.x * 32 + threadIdx.x] = sum;
    }
}

// Threads and pieces a thread for a row of n8 pieces.  Few rows: as many threads
// as there are, for the latency.  Many rows: 96 to 256 threads with two pieces,
// and four above `two` pieces a row.  Forward 400 (bf16, 8 bits out, 8192 rows of
// 4096 without residual 20.1 us against 23.8 with two pieces, with residual 4096
// rows 20.1 against 19.7; 2048 wide, one piece and 256 threads 39.5 us against
// 36.7 at 16384 rows), backward 512 (four pieces need the registers), in fp32
// 1024 (8192 rows of 4528 118 us against 140 us with four).
struct RowShape { int threads, v; };
RowShape row_shape(int n8, bool few, int two) {
    const int v = few ? (n8 <= 512 ? 1 : n8 <= 1024 ? 2 : 4) : (n8 <= 128 ? 1 : n8 <= two ? 2 : 4);
    return {((n8 + v - 1) / v + 31) / 32 * 32, v};
}

// Pieces a lane where a row takes a warp.
int warp_pieces(int n8) { return n8 <= 32 ? 1 : n8 <= 64 ? 2 : 4; }

constexpr int kSms = 152;
constexpr size_t kSmemSm = 227 * 1024;   // shared memory of an SM that its blocks share

// The kernel's dynamic shared-memory limit, set once a device.
template <auto Kernel> cudaError_t allow_smem() {
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemSm - 2048);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

template <int DT, int Q, bool kWarp>
cudaError_t launch_norm_v(const NormArgs &a, int T, int threads, int v, cudaStream_t st) {
    const dim3 grid(kWarp ? blocks_of(T, kWarpRows) : T), block(kWarp ? 32 * kWarpRows : threads);
    if (v == 1) return launch_pdl(k_rms_norm<DT, Q, 1, kWarp>, grid, block, 0, st, a, (int64_t)T);
    if (v == 2) return launch_pdl(k_rms_norm<DT, Q, 2, kWarp>, grid, block, 0, st, a, (int64_t)T);
    return launch_pdl(k_rms_norm<DT, Q, 4, kWarp>, grid, block, 0, st, a, (int64_t)T);
}

template <int DT, int Q> cudaError_t launch_norm_q(const NormArgs &a, int T, cudaStream_t st) {
    const int n8 = a.H / kChunk;
    const bool few = T <= 2 * kSms;
    // 16384 rows, bf16 with the residual: of 512 values 11.2 us against 17.1 us a
    // block a row, of 624 15.3 against 17.1, of 1024 20.8 against 20.2; without
    // it, of 1024 14.1 against 17.8 (one rule for both: the norm of a stored sum
    // has the bits of the norm that stored it).  1216 rows of 624: 3.2 against 2.7.
    const int most = T < 2048 ? kWarpPieces / 2 : kWarpPieces;
    if (n8 <= most && !few) return launch_norm_v<DT, Q, true>(a, T, 32, warp_pieces(n8), st);
    const RowShape s = row_shape(n8, few, 400);
    return launch_norm_v<DT, Q, false>(a, T, s.threads, s.v, st);
}

template <int DT> cudaError_t launch_norm(const NormArgs &a, int quant, int T, cudaStream_t st) {
    switch (quant) {
        case MOE_QUANT_NONE: return launch_norm_q<DT, MOE_QUANT_NONE>(a, T, st);
        case MOE_QUANT_E4M3_128: return launch_norm_q<DT, MOE_QUANT_E4M3_128>(a, T, st);
        case MOE_QUANT_E4M3_ROW: return launch_norm_q<DT, MOE_QUANT_E4M3_ROW>(a, T, st);
        default: return launch_norm_q<DT, MOE_QUANT_MXFP8>(a, T, st);
    }
}

// The backward pass's split.  Rows of up to 1024 values take a warp each (16384
// rows of 1024, bf16: 25.7 us against 65 us a block a row), longer ones a
// block.  Blocks an SM: 512 threads' worth, two to four (16384 rows: H = 2048
// 46.0 us with four, 58.1 with two; H = 6144 133 us with two, 171 with three,
// whose third waits), no more than its shared memory takes (1216 rows of 16384:
// 32.4 us with one, 36.8 with two); every block writes a row of partial sums.
// What one block does in two rounds is one block's, whose sums are the result:
// no workspace and no second launch (2 rows of 4096 3.1 us against 3.8, 4 rows
// would be 4.7; 16 rows of 512 2.8 against 3.2, 32 would be 4.4; host 7 us a call
// against 12).
constexpr int kOneBlockRounds = 2;
struct GradShape { RowShape row; bool warp; int blocks; };
GradShape grad_shape(int T, int H, int dtype) {
    const int n8 = H / kChunk;
    const bool f32 = dtype == MOE_DTYPE_F32;
    GradShape g;
    g.warp = n8 <= (f32 ? kWarpPieces / 2 : kWarpPieces);              // a warp's ring of fp32 rows is twice as large
    g.row = g.warp ? RowShape{32, warp_pieces(n8)} : row_shape(n8, false, f32 ? 1024 : 512);
    const int threads = g.warp ? 32 * kWarpRows : g.row.threads;
    const size_t rings = 2 * 3 * (f32 ? 32 : 16) * (size_t)g.row.v * threads;
    const int fit = (int)std::max<size_t>(1, kSmemSm / (rings + 2048));
    const int an_sm = std::min(fit, std::max(2, std::min(4, 512 / threads)));
    const int groups = g.warp ? blocks_of(T, kWarpRows) : T;          // rows, or eights of them
    g.blocks = groups <= kOneBlockRounds ? 1 : std::min(groups, an_sm * kSms);
    return g;
}

// Bytes of the blocks' partial sums; one block's are the result.
size_t grad_workspace(const GradShape &g, int H) { return g.blocks == 1 ? 0 : sizeof(float) * (size_t)g.blocks * (size_t)H; }

template <int DT, int V, int R, bool kWarp>
cudaError_t launch_norm_grad_v(const NormGradArgs &a, int blocks, int threads, size_t stage, cudaStream_t st) {
    const cudaError_t e = allow_smem<k_rms_norm_backward<DT, V, R, kWarp>>();
    if (e != cudaSuccess) return e;
    size_t smem = R * stage;
    if (kWarp) {
        smem = kWarpRows * std::max(smem, sizeof(float) * a.H);
        threads = 32 * kWarpRows;
    }
    return launch_pdl(k_rms_norm_backward<DT, V, R, kWarp>, dim3(blocks), dim3(threads), smem, st, a);
}

template <int DT> cudaError_t launch_norm_grad(const NormGradArgs &a, const GradShape &g, cudaStream_t st) {
    const int threads = g.row.threads, v = g.row.v, blocks = g.blocks;
    const size_t stage = (a.gs ? 3 : 2) * sizeof(Raw8<DT>) * v * threads;
    constexpr bool f32 = DT == MOE_DTYPE_F32;
    if (g.warp) {
        if (v == 1) return launch_norm_grad_v<DT, 1, 2, true>(a, blocks, threads, stage, st);
        if (v == 2 || f32) return launch_norm_grad_v<DT, 2, 2, true>(a, blocks, threads, stage, st);
        return launch_norm_grad_v<DT, f32 ? 2 : 4, 2, true>(a, blocks, threads, stage, st);
    }
    if constexpr (f32) {
        if (v == 1) return launch_norm_grad_v<DT, 1, 2, false>(a, blocks, threads, stage, st);
        if (2 * stage > kSmemSm - 2048) return launch_norm_grad_v<DT, 4, 1, false>(a, blocks, threads, stage, st);
    }
    if (v == 2) return launch_norm_grad_v<DT, 2, 2, false>(a, blocks, threads, stage, st);
    return launch_norm_grad_v<DT, 4, 2, false>(a, blocks, threads, stage, st);
}

moe_status check_rows(int32_t T, int32_t H, int32_t dtype) {
    if (T < 0 || !known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (H < kChunk || H > kMaxH || H % kChunk) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status moe_rms_norm(const void *x, int64_t x_stride, const void *residual, int64_t residual_stride,
                        const void *weight, int32_t T, int32_t H, int32_t dtype, float eps, int32_t quant,
                        void *sum, void *y, uint8_t *q, void *scales, float *rstd, void *stream) {
    moe_status st = check_rows(T, H, dtype);
    if (st != MOE_OK) return st;
    if (quant < MOE_QUANT_NONE || quant > MOE_QUANT_MXFP8) return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (x_stride < H || x_stride % kChunk) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (residual && (residual_stride < H || residual_stride % kChunk)) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (sum && !residual) return MOE_ERR_INVALID_ARG;
    if (quant == MOE_QUANT_NONE && (q || scales)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !weight) return MOE_ERR_INVALID_ARG;
    if (quant == MOE_QUANT_NONE ? !y : (!q || !scales)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(residual, 16) || !aligned_to(weight, 16) || !aligned_to(sum, 16) ||
        !aligned_to(y, 16) || !aligned_to(q, 16) || !aligned_to(scales, quant == MOE_QUANT_MXFP8 ? 1 : 4) ||
        !aligned_to(rstd, 4))
        return MOE_ERR_MISALIGNED;
    const NormArgs a{x, residual, weight, x_stride, residual_stride, H, 1.0f / (float)H, eps, sum, y, q, scales,
                     rstd};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MOE_DTYPE_F32: return cuda_status(launch_norm<MOE_DTYPE_F32>(a, quant, T, s));
        case MOE_DTYPE_BF16: return cuda_status(launch_norm<MOE_DTYPE_BF16>(a, quant, T, s));
        default: return cuda_status(launch_norm<MOE_DTYPE_F16>(a, quant, T, s));
    }
}

size_t moe_rms_norm_backward_workspace_for(int32_t T, int32_t H, int32_t dtype) {
    return T > 0 && H > 0 && known_dtype(dtype) ? grad_workspace(grad_shape(T, H, dtype), H) : 0;
}

size_t moe_rms_norm_backward_workspace(int32_t T, int32_t H) {
    return std::max(moe_rms_norm_backward_workspace_for(T, H, MOE_DTYPE_F32),
                    moe_rms_norm_backward_workspace_for(T, H, MOE_DTYPE_BF16));   // f16's is bf16's
}

moe_status moe_rms_norm_backward(const void *grad_y, const void *sum, const void *weight, const float *rstd,
                                 const void *grad_sum, int32_t T, int32_t H, int32_t dtype, void *grad_in,
                                 float *grad_w, void *workspace, size_t workspace_bytes, void *stream) {
    moe_status st = check_rows(T, H, dtype);
    if (st != MOE_OK) return st;
    if (!grad_w) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!grad_y || !sum || !weight || !rstd || !grad_in)) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_rms_norm_backward_workspace_for(T, H, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(grad_y, 16) || !aligned_to(sum, 16) || !aligned_to(weight, 16) || !aligned_to(rstd, 4) ||
        !aligned_to(grad_sum, 16) || !aligned_to(grad_in, 16) || !aligned_to(grad_w, 4) || !aligned_to(workspace, 16))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return cuda_status(cudaMemsetAsync(grad_w, 0, sizeof(float) * H, s));
    const GradShape g = grad_shape(T, H, dtype);
    const NormGradArgs a{grad_y, sum, weight, grad_sum, rstd, T, H, grad_in, g.blocks == 1 ? grad_w : static_cast<float *>(workspace)};
    cudaError_t e;
    switch (dtype) {
        case MOE_DTYPE_F32: e = launch_norm_grad<MOE_DTYPE_F32>(a, g, s); break;
        case MOE_DTYPE_BF16: e = launch_norm_grad<MOE_DTYPE_BF16>(a, g, s); break;
        default: e = launch_norm_grad<MOE_DTYPE_F16>(a, g, s); break;
    }
    if (e != cudaSuccess || g.blocks == 1) return cuda_status(e);
    return cuda_status(launch_pdl(k_rms_norm_grad_w, dim3((H + 31) / 32), dim3(8 * kColumnGroups), 0, s, (const float *)a.part, g.blocks,
                                  (int)H, grad_w));
}

}  // extern "C"
