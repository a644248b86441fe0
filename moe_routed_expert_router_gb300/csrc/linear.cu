// Products of a few tokens with a weight of 4-bit codes and group scales:
//   y[t][n] = round(x_scale[t] * ts * sum_k x[t][k] * E2M1(code[n][k]) * scale[n][k / G]),
// G = 16 with E4M3 scales and a tensor scale (NVFP4) or 32 with E8M0 scales (MXFP4).
//
// Bound by the weight's bytes, 4.5 or 4.25 bits a value, and close behind them by
// what widens a code: at the memory's rate an SM sub-partition has six issue
// slots for every two values.  So the products are warp MMAs (m16n8k16, f16
// operands, fp32 sums) with the weight's rows as the 16-row operand: a lane widens
// eight codes of a row with four conversion instructions and nothing is shared or
// shuffled.  f16 holds E2M1 * E4M3 exactly (six significant bits, 2^-10 to 2688);
// E8M0 scales go past f16, so MXFP4 multiplies the fp32 sum of every 32 values.
//
// bf16 tokens become f16 in a launch of their own, each row times a power of two
// that brings its largest magnitude to [2^7, 2^8): a bf16 value is exact in f16
// down to 2^-17, and what is smaller is off by at most 2^-25, that is 2^-32 of the
// row's largest.  f16 tokens are used where they lie.
//
// A block takes 16 * MT rows of the weight; its warps share K in stages of 256
// values, each with a cp.async ring of its own (no barriers between warps until
// the sums of a tile are joined).  The ring runs on into the block's next tile.
#include <algorithm>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kStageK = 256;               // values of K a stage
constexpr int kCodeBytes = kStageK / 2;    // a row's codes in a stage
constexpr int kScaleBytes = 16;            // a row's scales in a stage (MXFP4 uses 8)
constexpr int kRing = 4;
constexpr int kSms = 152;
constexpr int kMaxK = 1 << 16, kMaxTokens = 1 << 20;

struct LinearArgs {
    const uint8_t *codes, *scales;
    const float *ts;                       // tensor scale or null
    const __half *x;                       // [T] rows, x_stride apart
    const float *x_scale;                  // [T] or null for 1
    int64_t x_stride;
    void *out;
    int T, N, K, tiles, slices;            // tiles of rows; warps that share a tile's K
    int dtype, early;                      // out's type; whether the weight may be read before the launch before has ended
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// B bytes (4 or 8) into shared memory; zeros where not `on`.
template <int B> __device__ __forceinline__ void copy_small(void *dst, const void *src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_u32(dst)), "l"(src), "n"(B), "r"(on ? B : 0) : "memory");
}

__device__ __forceinline__ uint32_t lds32(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }

// Places for a tile's sums: with two, the next tile's need not wait for the reading of the last one's.
template <int MT, int NT> constexpr int join_buffers() { return MT * NT <= 4 ? 2 : 1; }

template <bool MX, int MT, int NT>
__global__ void __launch_bounds__(kThreads) k_linear(LinearArgs a) {
    constexpr int kRows = 16 * MT;
    constexpr int kStage = kRows * (kCodeBytes + kScaleBytes), kBufs = join_buffers<MT, NT>();
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wk = warp % a.slices, wm = warp / a.slices, groups = kWarps / a.slices;
    const int token0 = blockIdx.y * (8 * NT);
    uint8_t *ring = smem + warp * kRing * kStage;
    float4 *red = reinterpret_cast<float4 *>(smem + kWarps * kRing * kStage);   // [kBufs][warp][MT][NT][lane]
    const int stages = (a.K + kStageK - 1) / kStageK;
    const int64_t code_row = a.K / 2, scale_row = a.K / (MX ? 32 : 16);

    // one stage of the rows of a tile, into slot `slot`
    auto load = [&](int tile, int stage, int slot) {
        const int n0 = (tile * groups + wm) * kRows, k0 = stage * kStageK;
        uint8_t *to = ring + slot * kStage;
#pragma unroll
        for (int i = 0; i < 4 * MT; ++i) {
            const int id = i * 32 + lane, row = id >> 3, u = id & 7;
            const bool on = n0 + row < a.N && k0 + 32 * u < a.K;
            copy16(to + row * kCodeBytes + ((u ^ (row & 7)) << 4), a.codes + (on ? (n0 + row) * code_row + (k0 >> 1) + 16 * u : 0), on);
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int id = i * 32 + lane, row = id >> 1, half = id & 1;
            const bool on = n0 + row < a.N && k0 + 128 * half < a.K;
            constexpr int B = MX ? 4 : 8;
            copy_small<B>(to + kRows * kCodeBytes + row * kScaleBytes + half * B,
                          a.scales + (on ? (n0 + row) * scale_row + (int64_t)stage * (2 * B) + half * B : 0), on);
        }
    };
    // the stages of this warp, tile after tile
    int lt = blockIdx.x, ls = wk, slot = 0;
    auto load_next = [&](int to) {
        while (lt < a.tiles && ls >= stages) {
            lt += gridDim.x;
            ls = wk;
            if (wk >= stages) lt = a.tiles;
        }
        if (lt < a.tiles) {
            load(lt, ls, to);
            ls += a.slices;
        }
        copy_commit();
    };
    if (!a.early) pdl_wait();
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) load_next(i);
    if (a.early) pdl_wait();
    pdl_trigger();

    float ts = 1.0f;
    if (a.ts) ts = *a.ts;
    int buf = 0;
    for (int tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        float acc[MT][NT][4] = {};
        for (int stage = wk; stage < stages; stage += a.slices) {
            load_next((slot + kRing - 1) % kRing);
            copy_wait<kRing - 1>();
            __syncwarp();
            const uint8_t *from = ring + slot * kStage;
            uint4 sc[MT][2];               // the stage's scales of rows g and g + 8
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sc[m][h] = *reinterpret_cast<const uint4 *>(from + kRows * kCodeBytes + (16 * m + 8 * h + g) * kScaleBytes);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int k = stage * kStageK + 32 * u + 8 * t;
                uint4 xb[NT];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const int token = token0 + 8 * n + g;
                    xb[n] = make_uint4(0, 0, 0, 0);
                    if (token < a.T && k < a.K) xb[n] = ld16_shared(a.x + token * a.x_stride + k);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    uint32_t w[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        e2m1x8_to_f16x8(lds32(from + (16 * m + 8 * h + g) * kCodeBytes + ((u ^ g) << 4) + 4 * t), w[h]);
                        if constexpr (!MX) {
                            // the scale of values 8 t .. 8 t + 7 of the unit: byte 2 u + (t >> 1), twice
                            const uint32_t word = (&sc[m][h].x)[u >> 1];
                            const uint32_t two = __byte_perm(word, 0, (t >> 1) * 0x11 + ((u & 1) ? 0x22 : 0));
                            const uint32_t s = e4m3x2_to_f16x2(two & 0xFFFFu);
#pragma unroll
                            for (int j = 0; j < 4; ++j) w[h][j] = hmul2(w[h][j], s);
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if constexpr (MX) {
                            float d[4] = {};
                            mma16816(d, w[0][0], w[1][0], w[0][1], w[1][1], xb[n].x, xb[n].y);
                            mma16816(d, w[0][2], w[1][2], w[0][3], w[1][3], xb[n].z, xb[n].w);
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float s = e8m0_to_f32((&sc[m][h].x)[u >> 2] >> (8 * (u & 3)));
                                acc[m][n][2 * h] = fmaf(d[2 * h], s, acc[m][n][2 * h]);
                                acc[m][n][2 * h + 1] = fmaf(d[2 * h + 1], s, acc[m][n][2 * h + 1]);
                            }
                        } else {
                            mma16816(acc[m][n], w[0][0], w[1][0], w[0][1], w[1][1], xb[n].x, xb[n].y);
                            mma16816(acc[m][n], w[0][2], w[1][2], w[0][3], w[1][3], xb[n].z, xb[n].w);
                        }
                    }
                }
            }
            __syncwarp();
            slot = (slot + 1) % kRing;
        }
        // join the slices' sums in order
        float4 *mine = red + buf * (kWarps * MT * NT * 32);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
                mine[((warp * MT + m) * NT + n) * 32 + lane] = make_float4(acc[m][n][0], acc[m][n][1], acc[m][n][2], acc[m][n][3]);
        __syncthreads();
        const float *all = reinterpret_cast<const float *>(mine);
        const int outs = groups * kRows * 8 * NT;
        for (int i = threadIdx.x; i < outs; i += kThreads) {
            const int row = i % kRows, j = i / kRows, tok = j % (8 * NT), grp = j / (8 * NT);
            const int n = (tile * groups + grp) * kRows + row, token = token0 + tok;
            if (n >= a.N || token >= a.T) continue;
            const int from = ((((row >> 4) * NT + (tok >> 3)) * 32 + (row & 7) * 4 + ((tok & 7) >> 1)) << 2) + ((row >> 3) & 1) * 2 + (tok & 1);
            float s = 0.0f;
            for (int w = 0; w < a.slices; ++w) s += all[(grp * a.slices + w) * (MT * NT * 128) + from];
            s = s * ts;
            if (a.x_scale) s *= a.x_scale[token];
            const int64_t at = (int64_t)token * a.N + n;
            if (a.dtype == MOE_DTYPE_F32) static_cast<float *>(a.out)[at] = s;
            else if (a.dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(s);
            else static_cast<__half *>(a.out)[at] = __float2half_rn(s);
        }
        if constexpr (kBufs == 1) __syncthreads();
        else buf ^= 1;
    }
}

// bf16 rows as f16 times a power of two (see the top), and what undoes it.
constexpr int kXThreads = 256;
__global__ void __launch_bounds__(kXThreads) k_linear_x(const __nv_bfloat16 *x, int64_t stride, int K, __half *out, float *scale) {
    __shared__ float top[kXThreads / 32];
    const int64_t row = blockIdx.x;
    pdl_wait();
    pdl_trigger();
    float amax = 0.0f;
    for (int k = 8 * threadIdx.x; k < K; k += 8 * kXThreads) {
        float v[8];
        widen8<MOE_DTYPE_BF16>(load8_shared<MOE_DTYPE_BF16>(x + row * stride + k), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, isfinite(v[i]) ? fabsf(v[i]) : 0.0f);
    }
    amax = warp_max(amax);
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kXThreads / 32; ++i) amax = fmaxf(amax, top[i]);
    const int e = (int)(__float_as_uint(amax) >> 23) - 127;      // -127 for a row of subnormals or zeros
    const float up = ldexpf(1.0f, min(7 - e, 127)), more = ldexpf(1.0f, max(0, 7 - e - 127));   // 2^(7 - e) in two factors
    for (int k = 8 * threadIdx.x; k < K; k += 8 * kXThreads) {
        float v[8];
        widen8<MOE_DTYPE_BF16>(load8_shared<MOE_DTYPE_BF16>(x + row * stride + k), v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * up * more;
        store8<MOE_DTYPE_F16>(out + row * K + k, narrow8<MOE_DTYPE_F16>(v));
    }
    if (threadIdx.x == 0) scale[row] = ldexpf(1.0f, e - 7);
}

// ------------------------------------------------------------ host side

template <bool MX, int MT, int NT> cudaError_t launch(LinearArgs a, cudaStream_t st) {
    constexpr size_t smem = kWarps * (kRing * 16 * MT * (kCodeBytes + kScaleBytes) + join_buffers<MT, NT>() * MT * NT * 32 * sizeof(float4));
    static_assert(smem <= kSmemSm - 2048);
    const cudaError_t e = allow_smem<k_linear<MX, MT, NT>>();
    if (e != cudaSuccess) return e;
    const int stages = (a.K + kStageK - 1) / kStageK;
    a.slices = stages >= 8 ? 8 : stages >= 4 ? 4 : stages >= 2 ? 2 : 1;
    a.tiles = blocks_of(a.N, 16 * MT * (kWarps / a.slices));
    constexpr int an_sm = (int)std::max<size_t>(1, std::min<size_t>(2, 227 * 1024 / (smem + 1024)));
    const dim3 grid(std::min(a.tiles, kSms * an_sm), blocks_of(a.T, 8 * NT));
    return launch_pdl(k_linear<MX, MT, NT>, grid, dim3(kThreads), smem, st, a);
}

template <bool MX> cudaError_t launch_format(const LinearArgs &a, cudaStream_t st) {
    if (a.T <= 8) return launch<MX, 1, 1>(a, st);
    if (a.T <= 16) return launch<MX, 2, 2>(a, st);
    if (a.T <= 32) return launch<MX, 2, 4>(a, st);
    return launch<MX, 2, 8>(a, st);
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

size_t moe_linear_fp4_workspace(int32_t T, int32_t K, int32_t dtype) {
    if (T < 1 || K < 1 || dtype != MOE_DTYPE_BF16) return 0;
    return (size_t)T * K * sizeof(__half) + ((size_t)T * sizeof(float) + 15) / 16 * 16;
}

moe_status moe_linear_fp4(const void *x, int64_t x_stride, const moe_nvfp4 *weight, int32_t weight_format, int32_t T,
                          int32_t N, int32_t K, int32_t dtype, int32_t out_dtype, void *out, void *workspace,
                          size_t workspace_bytes, void *stream) {
    if (T < 0 || (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) || (out_dtype != dtype && out_dtype != MOE_DTYPE_F32) ||
        (weight_format != MOE_WEIGHTS_NVFP4 && weight_format != MOE_WEIGHTS_MXFP4) || !weight)
        return MOE_ERR_INVALID_ARG;
    if (N < 1 || K < 128 || K > kMaxK || K % 128 || x_stride < K || x_stride % kChunk || T > kMaxTokens || N > INT32_MAX - 1024)
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    const bool mx = weight_format == MOE_WEIGHTS_MXFP4;
    if (!x || !out || !weight->codes || !weight->scales || (!mx && !weight->tensor_scale)) return MOE_ERR_INVALID_ARG;
    const size_t need = moe_linear_fp4_workspace(T, K, dtype);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(weight->codes, 16) || !aligned_to(weight->scales, 16) ||
        !aligned_to(mx ? nullptr : weight->tensor_scale, 4) || !aligned_to(out, out_dtype == MOE_DTYPE_F32 ? 4 : 2) ||
        !aligned_to(workspace, 16))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    LinearArgs a{};
    a.codes = weight->codes;
    a.scales = weight->scales;
    a.ts = mx ? nullptr : weight->tensor_scale;
    a.out = out;
    a.T = T;
    a.N = N;
    a.K = K;
    a.dtype = out_dtype;
    if (dtype == MOE_DTYPE_BF16) {
        __half *x16 = static_cast<__half *>(workspace);
        float *scale = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + (size_t)T * K * sizeof(__half));
        const cudaError_t e = launch_pdl(k_linear_x, dim3(T), dim3(kXThreads), 0, s, static_cast<const __nv_bfloat16 *>(x), x_stride, (int)K,
                                         x16, scale);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
        a.x = x16;
        a.x_scale = scale;
        a.x_stride = K;
        a.early = 1;                       // k_linear_x starts no dependents before all that came before it has ended
    } else {
        a.x = static_cast<const __half *>(x);
        a.x_stride = x_stride;
    }
    return cuda_status(mx ? launch_format<true>(a, s) : launch_format<false>(a, s));
}

}  // extern "C"
