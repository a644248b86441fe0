// Residual addition and root-mean-square norm with an optional 8-bit output,
// and its gradients (see include/moe_nvfp4.h for the formulas).
//
// Forward: one block a row, the row in registers between its two uses (the sum
// of squares, then the products), so every input is read once and every output
// written once.  Bound by HBM.
#include <math.h>

#include <algorithm>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kMaxH = 16384;
constexpr int kMaxChunksThread = 4;   // 16-byte pieces of a row a thread holds
// Threads of a block whose threads hold v pieces (row_shape below).
constexpr int max_threads(int v) { return v < kMaxChunksThread ? 256 : kMaxH / kChunk / kMaxChunksThread; }
constexpr float kMinAmax = 7.888609052210118e-31f;   // 2^-100

struct NormArgs {
    const void *x, *r, *w;
    int64_t xs, rs;
    int H;
    float eps;
    void *sum, *y;
    uint8_t *q;
    void *scales;
    float *rstd;
};

// Maximum that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sum over the block, the same on every thread; `red` holds 33 words, and two
// calls in a row use different ones.
__device__ __forceinline__ float block_sum(float v, float *red) {
    v = warp_sum(v);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    return warp_sum(lane < nw ? red[lane] : 0.0f);
}

__device__ __forceinline__ float block_max_nan(float v, float *red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    v = lane < nw ? red[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
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

// 1 / sqrt(mean + eps): the IEEE square root and division, once a row.
__device__ __forceinline__ float row_rstd(float sumsq, int H, float eps) {
    return __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(sumsq, (float)H), eps)));
}

// Thread i holds pieces i, i + n, ... of the row (n threads, a multiple of 32),
// so a warp's loads are 512 consecutive bytes of a 16-bit row, a 128-value
// group is 16 neighbouring lanes and a 32-value group is four.
template <int DT, int Q, int V>
__global__ void __launch_bounds__(max_threads(V)) k_rms_norm(const NormArgs a) {
    using T = typename RowType<DT>::T;
    __shared__ float red[2][32];
    const int64_t t = blockIdx.x;
    const int n8 = a.H / kChunk, n = blockDim.x;
    const T *x = static_cast<const T *>(a.x) + t * a.xs;
    const T *r = a.r ? static_cast<const T *>(a.r) + t * a.rs : nullptr;
    float v[V][8];
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * n;
        if (c < n8) {
            widen8<DT>(load8<DT>(x + c * kChunk), v[i]);
            if (r) {
                float u[8];
                widen8<DT>(load8<DT>(r + c * kChunk), u);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = __fadd_rn(v[i][e], u[e]);
                const Raw8<DT> s = narrow8<DT>(v[i]);
                if (a.sum) store8<DT>(static_cast<T *>(a.sum) + t * a.H + c * kChunk, s);
                widen8<DT>(s, v[i]);   // the norm is the stored sum's
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(v[i][e], v[i][e], ss);
    }
    const float rstd = row_rstd(block_sum(ss, red[0]), a.H, a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = rstd;
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * n;
        if (c < n8) {
            float w[8];
            widen8<DT>(load8<DT>(static_cast<const T *>(a.w) + c * kChunk), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][e] = __fmul_rn(__fmul_rn(v[i][e], rstd), w[e]);
            if (a.y) store8<DT>(static_cast<T *>(a.y) + t * a.H + c * kChunk, narrow8<DT>(v[i]));
        }
        if constexpr (Q == MOE_QUANT_E4M3_ROW) {
#pragma unroll
            for (int e = 0; e < 8; ++e) amax = max_nan(amax, fabsf(v[i][e]));
        }
    }
    if constexpr (Q == MOE_QUANT_NONE) return;
    if constexpr (Q == MOE_QUANT_E4M3_ROW) {
        amax = max_nan(block_max_nan(amax, red[1]), kMinAmax);
        if (threadIdx.x == 0) static_cast<float *>(a.scales)[t] = __fdiv_rn(amax, 448.0f);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * n;
        float mul;
        if constexpr (Q == MOE_QUANT_E4M3_ROW) {
            mul = __fdiv_rn(448.0f, amax);
        } else {
            constexpr int kLanes = Q == MOE_QUANT_MXFP8 ? 4 : 16;
            float m = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(v[i][e]));
#pragma unroll
            for (int o = kLanes / 2; o >= 1; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
            const bool first = c < n8 && (c % kLanes) == 0;
            const int64_t at = t * ((n8 + kLanes - 1) / kLanes) + c / kLanes;
            if constexpr (Q == MOE_QUANT_E4M3_128) {
                m = max_nan(m, kMinAmax);
                mul = __fdiv_rn(448.0f, m);
                if (first) static_cast<float *>(a.scales)[at] = __fdiv_rn(m, 448.0f);
            } else {
                // floor(log2(amax)) + 127 is the exponent field of a normal amax;
                // E4M3's largest exponent is 8
                const int field = (int)((__float_as_uint(m) >> 23) & 0xFFu);
                const int byte = field == 255 ? 255 : max(field - 8, 0);
                mul = field == 255 ? __uint_as_float(0x7FC00000u) : __uint_as_float((uint32_t)(254 - byte) << 23);
                if (first) static_cast<uint8_t *>(a.scales)[at] = (uint8_t)byte;
            }
        }
        if (c < n8) {
            uint2 o;
            o.x = e4m3x4(__fmul_rn(v[i][0], mul), __fmul_rn(v[i][1], mul), __fmul_rn(v[i][2], mul), __fmul_rn(v[i][3], mul));
            o.y = e4m3x4(__fmul_rn(v[i][4], mul), __fmul_rn(v[i][5], mul), __fmul_rn(v[i][6], mul), __fmul_rn(v[i][7], mul));
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
// [blocks][H] store at the end.
template <int DT, int V>
__global__ void __launch_bounds__(max_threads(V)) k_rms_norm_backward(const NormGradArgs a) {
    using T = typename RowType<DT>::T;
    __shared__ float red[2][32];
    const int n8 = a.H / kChunk, n = blockDim.x;
    float gw[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) gw[i][e] = 0.0f;
    int par = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
        const float rstd = a.rstd[t];
        float g[V][8], nn[V][8];
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * n;
            if (c >= n8) continue;
            const int64_t at = t * a.H + c * kChunk;
            float w[8];
            widen8<DT>(load8<DT>(static_cast<const T *>(a.gy) + at), g[i]);
            widen8<DT>(load8<DT>(static_cast<const T *>(a.s) + at), nn[i]);
            widen8<DT>(load8<DT>(static_cast<const T *>(a.w) + c * kChunk), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                nn[i][e] *= rstd;
                gw[i][e] = fmaf(g[i][e], nn[i][e], gw[i][e]);
                g[i][e] *= w[e];
                dot = fmaf(g[i][e], nn[i][e], dot);
            }
        }
        const float c1 = block_sum(dot, red[par]) / (float)a.H;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = threadIdx.x + i * n;
            if (c >= n8) continue;
            const int64_t at = t * a.H + c * kChunk;
            float gs[8], o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) gs[e] = 0.0f;
            if (a.gs) widen8<DT>(load8<DT>(static_cast<const T *>(a.gs) + at), gs);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(rstd, fmaf(-nn[i][e], c1, g[i][e]), gs[e]);
            store8<DT>(static_cast<T *>(a.gin) + at, narrow8<DT>(o));
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = threadIdx.x + i * n;
        if (c >= n8) continue;
        store8<MOE_DTYPE_F32>(a.part + (int64_t)blockIdx.x * a.H + c * kChunk, narrow8<MOE_DTYPE_F32>(gw[i]));
    }
}

// grad_w[h] = sum over the blocks' partial sums, in block order within each of
// eight interleaved chains.
__global__ void __launch_bounds__(256) k_rms_norm_grad_w(const float *__restrict__ part, int blocks, int H,
                                                         float *__restrict__ gw) {
    __shared__ float s[8][33];
    const int h = blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (h < H)
        for (int b = threadIdx.y; b < blocks; b += 8) v += part[(int64_t)b * H + h];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && h < H) {
        for (int i = 1; i < 8; ++i) v += s[i][threadIdx.x];
        gw[h] = v;
    }
}

// Threads and pieces a thread for a row of n8 pieces.
struct RowShape { int threads, v; };
RowShape row_shape(int n8) {
    int v = 1;
    while (v < kMaxChunksThread && n8 > 256 * v) v *= 2;
    return {((n8 + v - 1) / v + 31) / 32 * 32, v};
}

template <int DT, int Q> cudaError_t launch_norm_q(const NormArgs &a, int T, cudaStream_t st) {
    const RowShape s = row_shape(a.H / kChunk);
    if (s.v == 1) k_rms_norm<DT, Q, 1><<<T, s.threads, 0, st>>>(a);
    else if (s.v == 2) k_rms_norm<DT, Q, 2><<<T, s.threads, 0, st>>>(a);
    else k_rms_norm<DT, Q, 4><<<T, s.threads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int DT> cudaError_t launch_norm(const NormArgs &a, int quant, int T, cudaStream_t st) {
    switch (quant) {
        case MOE_QUANT_NONE: return launch_norm_q<DT, MOE_QUANT_NONE>(a, T, st);
        case MOE_QUANT_E4M3_128: return launch_norm_q<DT, MOE_QUANT_E4M3_128>(a, T, st);
        case MOE_QUANT_E4M3_ROW: return launch_norm_q<DT, MOE_QUANT_E4M3_ROW>(a, T, st);
        default: return launch_norm_q<DT, MOE_QUANT_MXFP8>(a, T, st);
    }
}

template <int DT> cudaError_t launch_norm_grad(const NormGradArgs &a, int blocks, cudaStream_t st) {
    const RowShape s = row_shape(a.H / kChunk);
    if (s.v == 1) k_rms_norm_backward<DT, 1><<<blocks, s.threads, 0, st>>>(a);
    else if (s.v == 2) k_rms_norm_backward<DT, 2><<<blocks, s.threads, 0, st>>>(a);
    else k_rms_norm_backward<DT, 4><<<blocks, s.threads, 0, st>>>(a);
    return cudaGetLastError();
}

// Blocks of the backward pass: two for each of the GB300's 152 SMs.
constexpr int kGradBlocks = 304;
int grad_blocks(int T) { return std::min(T, kGradBlocks); }

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
    const NormArgs a{x, residual, weight, x_stride, residual_stride, H, eps, sum, y, q, scales, rstd};
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MOE_DTYPE_F32: return cuda_status(launch_norm<MOE_DTYPE_F32>(a, quant, T, s));
        case MOE_DTYPE_BF16: return cuda_status(launch_norm<MOE_DTYPE_BF16>(a, quant, T, s));
        default: return cuda_status(launch_norm<MOE_DTYPE_F16>(a, quant, T, s));
    }
}

size_t moe_rms_norm_backward_workspace(int32_t T, int32_t H) {
    if (T <= 0 || H <= 0) return 0;
    return sizeof(float) * (size_t)grad_blocks(T) * (size_t)H;
}

moe_status moe_rms_norm_backward(const void *grad_y, const void *sum, const void *weight, const float *rstd,
                                 const void *grad_sum, int32_t T, int32_t H, int32_t dtype, void *grad_in,
                                 float *grad_w, void *workspace, size_t workspace_bytes, void *stream) {
    moe_status st = check_rows(T, H, dtype);
    if (st != MOE_OK) return st;
    if (!grad_w) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!grad_y || !sum || !weight || !rstd || !grad_in || !workspace)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < moe_rms_norm_backward_workspace(T, H)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(grad_y, 16) || !aligned_to(sum, 16) || !aligned_to(weight, 16) || !aligned_to(rstd, 4) ||
        !aligned_to(grad_sum, 16) || !aligned_to(grad_in, 16) || !aligned_to(grad_w, 4) || !aligned_to(workspace, 16))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return cuda_status(cudaMemsetAsync(grad_w, 0, sizeof(float) * H, s));
    const int blocks = grad_blocks(T);
    const NormGradArgs a{grad_y, sum, weight, grad_sum, rstd, T, H, grad_in, static_cast<float *>(workspace)};
    cudaError_t e;
    switch (dtype) {
        case MOE_DTYPE_F32: e = launch_norm_grad<MOE_DTYPE_F32>(a, blocks, s); break;
        case MOE_DTYPE_BF16: e = launch_norm_grad<MOE_DTYPE_BF16>(a, blocks, s); break;
        default: e = launch_norm_grad<MOE_DTYPE_F16>(a, blocks, s); break;
    }
    if (e != cudaSuccess) return MOE_ERR_CUDA;
    k_rms_norm_grad_w<<<(H + 31) / 32, dim3(32, 8), 0, s>>>(a.part, blocks, H, grad_w);
    return cuda_status(cudaGetLastError());
}

}  // extern "C"
