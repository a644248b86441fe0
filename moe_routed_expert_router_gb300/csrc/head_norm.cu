// Root-mean-square norm of every query and key head with the position rotation
// behind it, and its gradients.
//
// A head row x of D values becomes n = x * rstd * w; then its first R values
// turn in R / 2 planes by angle_i = position * frequency_i:
//   (a, b) -> (a cos - b sin, b cos + a sin),
// a and b being the values i and i + R / 2, or 2i and 2i + 1 (interleaved).
// Backward, with g = grad turned back and n^ = x * rstd:
//   grad_w = sum over rows of g * n^,  grad_x = rstd * (g w - n^ mean(g w n^)).
//
// The angles of far positions: a frequency is given as a fraction of a turn in
// units of 2^-64, so position * fraction in 64-bit integers drops the whole turns
// exactly and what is left rounds to fp32 once (an error of 1e-7 radians at any
// position; an fp32 product would be off by 0.06 at position 10^6).
//
// Layout: 2^lg lanes a row, 16 values a lane in two 8-value pieces of which the
// second holds the partners of the first (half-split planes) or other whole
// planes (interleaved ones), so a rotation needs no other lane's values.  A block
// takes a tile of tokens of the queries or of the keys; the tile's sines and
// cosines are computed once into shared memory and serve every head.
#include <algorithm>
#include <cmath>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kMaxHeads = 1024, kMaxDim = 512;
constexpr int kSms = 152;
constexpr int kAngleBytes = 32 * 1024;     // of a tile's sines and cosines

// Queries or keys: rows [T][heads][D], `stride` values from token to token.
struct HeadTensor {
    const void *x, *w, *g;                 // g: the output's gradient (backward)
    void *out;
    int64_t stride, out_stride, g_stride;
    float *sums;                           // backward: [blocks][D] partial sums of grad_w
    int heads, inv;                        // inv = ceil(2^20 / heads): row / heads without a division
    int tokens, tiles, blocks;             // tokens a tile, tiles, blocks that share them
};

struct HeadArgs {
    HeadTensor q, k;
    const int32_t *pos;
    const uint64_t *turns;
    int T, D, R, lg;
    float eps, inv_d;
};

// What a thread is in its row.
struct Lane {
    int group, groups, c, p0, step;        // its row of a round, rows a round, its place, its pieces p0 and p0 + step
    bool on, turned;
};

__device__ __forceinline__ Lane lane_of(const HeadArgs &a) {
    Lane l;
    l.c = threadIdx.x & ((1 << a.lg) - 1);
    l.group = threadIdx.x >> a.lg;
    l.groups = blockDim.x >> a.lg;
    const int planes = a.R >> 4;           // lanes whose two pieces turn
    l.on = l.c < (a.D >> 4);
    l.turned = l.c < planes;
    l.p0 = l.turned ? l.c : l.c + planes;
    l.step = l.turned ? planes : (a.D - a.R) >> 4;
    return l;
}

// Sines and cosines of `n` tokens from t0 on: cos [n][R / 2], then sin.  The
// angles of a lane's pieces lie at 16-byte places c and c + R / 16 of a token.
template <bool kPairs>
__device__ __forceinline__ void fill_angles(const HeadArgs &a, int t0, int n, float *cs) {
    const int half = a.R >> 1, planes = a.R >> 4;
    if (half == 0) return;
    for (int j = threadIdx.x; j < n * half; j += blockDim.x) {
        const int t = j / half, i = j - t * half;
        const uint64_t turn = (uint64_t)(int64_t)a.pos[t0 + t] * a.turns[i];
        float s, c;
        sincospif((float)(int64_t)turn * 0x1p-63f, &s, &c);      // 2^63 is half a turn
        const int at = kPairs ? i : (((i >> 2) & 1) * planes + (i >> 3)) * 4 + (i & 3);
        cs[t * half + at] = c;
        cs[(n + t) * half + at] = s;
    }
}

struct Angles { float c[8], s[8]; };

__device__ __forceinline__ Angles angles_of(const HeadArgs &a, const Lane &l, const float *cs, int n, int t) {
    Angles r;
    if (l.turned) {
        const int half = a.R >> 1;
        const float4 *c = reinterpret_cast<const float4 *>(cs + t * half), *s = reinterpret_cast<const float4 *>(cs + (n + t) * half);
        *reinterpret_cast<float4 *>(r.c) = c[l.c];
        *reinterpret_cast<float4 *>(r.c + 4) = c[l.c + l.step];
        *reinterpret_cast<float4 *>(r.s) = s[l.c];
        *reinterpret_cast<float4 *>(r.s + 4) = s[l.c + l.step];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r.c[i] = 1.0f;
            r.s[i] = 0.0f;
        }
    }
    return r;
}

// v[0..7] and v[8..15], the lane's pieces, turned by the angles (kBack: by their opposites).
template <bool kPairs, bool kBack> __device__ __forceinline__ void turn16(float (&v)[16], const Angles &r) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float &a = kPairs ? v[2 * i] : v[i], &b = kPairs ? v[2 * i + 1] : v[i + 8];
        const float s = kBack ? -r.s[i] : r.s[i];
        const float u = fmaf(a, r.c[i], -(b * s)), w = fmaf(b, r.c[i], a * s);
        a = u;
        b = w;
    }
}

template <int DT> __device__ __forceinline__ void widen16(const Raw8<DT> (&r)[2], float (&v)[16]) {
    float a[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        widen8<DT>(r[h], a);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] = a[i];
    }
}

template <int DT> __device__ __forceinline__ void store16(typename RowType<DT>::T *p, const Lane &l, const float (&v)[16]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = v[8 * h + i];
        store8<DT>(p + 8 * (l.p0 + h * l.step), narrow8<DT>(a));
    }
}

template <int DT> __device__ __forceinline__ void fetch16(const typename RowType<DT>::T *p, const Lane &l, Raw8<DT> (&r)[2]) {
    r[0] = load8<DT>(p + 8 * l.p0);
    r[1] = load8<DT>(p + 8 * (l.p0 + l.step));
}

__device__ __forceinline__ float over_row(float v, int lg) {
    for (int o = 1 << lg >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// U rows a thread at once, all loads ahead of their use.
template <int DT, bool kPairs, int U>
__global__ void __launch_bounds__(kThreads) k_head_norm(HeadArgs a) {
    using T = typename RowType<DT>::T;
    extern __shared__ __align__(16) float cs[];
    const bool key = (int)blockIdx.x >= a.q.blocks;
    const HeadTensor h = key ? a.k : a.q;
    const int t0 = ((int)blockIdx.x - (key ? a.q.blocks : 0)) * h.tokens;
    const int n = min(h.tokens, a.T - t0), rows = n * h.heads;
    const Lane l = lane_of(a);
    pdl_wait();
    pdl_trigger();
    Raw8<DT> x[U][2], wr[2] = {};
    auto at = [&](int r, int64_t stride, int &t) {
        t = (int)((unsigned)(r * h.inv) >> 20);
        return (int64_t)(t0 + t) * stride + (int64_t)(r - t * h.heads) * a.D;
    };
    auto fetch = [&](int base) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * l.groups + l.group;
            int t;
            x[u][0] = x[u][1] = Raw8<DT>{};
            if (l.on && r < rows) fetch16<DT>(static_cast<const T *>(h.x) + at(r, h.stride, t), l, x[u]);
        }
    };
    fetch(0);
    if (l.on) {
        wr[0] = load8_shared<DT>(static_cast<const T *>(h.w) + 8 * l.p0);
        wr[1] = load8_shared<DT>(static_cast<const T *>(h.w) + 8 * (l.p0 + l.step));
    }
    fill_angles<kPairs>(a, t0, n, cs);
    __syncthreads();
    for (int base = 0; base < rows; base += U * l.groups) {
        if (base > 0) fetch(base);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int r = base + u * l.groups + l.group;
            float v[16], w[16], sum = 0.0f;
            widen16<DT>(x[u], v);
            widen16<DT>(wr, w);
#pragma unroll
            for (int i = 0; i < 16; ++i) sum = fmaf(v[i], v[i], sum);
            sum = over_row(sum, a.lg);
            if (l.on && r < rows) {
                const float rstd = __frsqrt_rn(fmaf(sum, a.inv_d, a.eps));
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = v[i] * w[i] * rstd;
                int t;
                T *to = static_cast<T *>(h.out) + at(r, h.out_stride, t);
                turn16<kPairs, false>(v, angles_of(a, l, cs, n, t));
                store16<DT>(to, l, v);
            }
        }
    }
}

// Blocks walk over tiles; a thread holds its 16 values' part of grad_w in
// registers until the end, so the order of the sums is fixed.
template <int DT, bool kPairs, int U>
__global__ void __launch_bounds__(kThreads) k_head_norm_backward(HeadArgs a) {
    using T = typename RowType<DT>::T;
    extern __shared__ __align__(16) float cs[];
    const bool key = (int)blockIdx.x >= a.q.blocks;
    const HeadTensor h = key ? a.k : a.q;
    const int block = (int)blockIdx.x - (key ? a.q.blocks : 0);
    const Lane l = lane_of(a);
    pdl_wait();
    pdl_trigger();
    float w[16] = {}, gw[16] = {};
    if (l.on) {
        Raw8<DT> wr[2];
        wr[0] = load8_shared<DT>(static_cast<const T *>(h.w) + 8 * l.p0);
        wr[1] = load8_shared<DT>(static_cast<const T *>(h.w) + 8 * (l.p0 + l.step));
        widen16<DT>(wr, w);
    }
    for (int tile = block; tile < h.tiles; tile += h.blocks) {
        const int t0 = tile * h.tokens, n = min(h.tokens, a.T - t0), rows = n * h.heads;
        Raw8<DT> x[U][2], g[U][2];
        auto at = [&](int r, int64_t stride, int &t) {
            t = (int)((unsigned)(r * h.inv) >> 20);
            return (int64_t)(t0 + t) * stride + (int64_t)(r - t * h.heads) * a.D;
        };
        auto fetch = [&](int base) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = base + u * l.groups + l.group;
                int t;
                x[u][0] = x[u][1] = g[u][0] = g[u][1] = Raw8<DT>{};
                if (l.on && r < rows) {
                    fetch16<DT>(static_cast<const T *>(h.x) + at(r, h.stride, t), l, x[u]);
                    fetch16<DT>(static_cast<const T *>(h.g) + at(r, h.g_stride, t), l, g[u]);
                }
            }
        };
        fetch(0);
        __syncthreads();                   // the tile before is done with the angles
        fill_angles<kPairs>(a, t0, n, cs);
        __syncthreads();
        for (int base = 0; base < rows; base += U * l.groups) {
            if (base > 0) fetch(base);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int r = base + u * l.groups + l.group;
                const bool mine = l.on && r < rows;
                int t = 0;
                const int64_t to = mine ? at(r, h.out_stride, t) : 0;
                float v[16], f[16], sum = 0.0f, dot = 0.0f;
                widen16<DT>(x[u], v);
                widen16<DT>(g[u], f);
                turn16<kPairs, true>(f, angles_of(a, l, cs, n, t));
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    sum = fmaf(v[i], v[i], sum);
                    dot = fmaf(f[i] * w[i], v[i], dot);
                }
                sum = over_row(sum, a.lg);
                dot = over_row(dot, a.lg);
                if (mine) {
                    const float rstd = __frsqrt_rn(fmaf(sum, a.inv_d, a.eps));
                    const float back = dot * rstd * a.inv_d * rstd;      // mean(g w n^) rstd
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        gw[i] = fmaf(f[i], v[i] * rstd, gw[i]);
                        f[i] = rstd * fmaf(-v[i], back, f[i] * w[i]);
                    }
                    store16<DT>(static_cast<T *>(h.out) + to, l, f);
                }
            }
        }
    }
    // the groups' sums, [groups][D], added in order
    __syncthreads();
    if (l.on) {
#pragma unroll
        for (int i = 0; i < 16; ++i) cs[l.group * a.D + 8 * (l.p0 + (i >> 3) * l.step) + (i & 7)] = gw[i];
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.D; d += blockDim.x) {
        float s = 0.0f;
        for (int i = 0; i < l.groups; ++i) s += cs[i * a.D + d];
        h.sums[(int64_t)block * a.D + d] = s;
    }
}

// grad_w of the queries (blockIdx.y 0) and keys: the blocks' sums in a fixed order.
__global__ void __launch_bounds__(8 * kColumnGroups) k_head_norm_grad_w(const float *q, int q_blocks, const float *k, int k_blocks, int D,
                                                                         float *gqw, float *gkw) {
    pdl_wait();
    pdl_trigger();
    if (blockIdx.y == 0) column_sums(q, q_blocks, D, gqw);
    else column_sums(k, k_blocks, D, gkw);
}

// ------------------------------------------------------------ host side

int lanes_log(int D) {
    int lg = 0;
    while (16 << lg < D) ++lg;
    return lg;
}

// The tile of one tensor: about `rounds` rows a group of lanes, as many tokens
// as their angles' shared memory allows, and no fewer tiles than fill the card
// while there are tokens to share.
void set_tiles(HeadTensor &t, int T, int heads, int R, int lg, int rounds) {
    const int groups = kThreads >> lg;
    t.heads = heads;
    t.inv = (1 << 20) / heads + ((1 << 20) % heads != 0);
    int n = std::max(1, groups * rounds / heads);
    n = std::min(n, std::max(1, T / (2 * kSms)));
    if (R > 0) n = std::min(n, std::max(1, kAngleBytes / (4 * R)));
    t.tokens = n;
    t.tiles = blocks_of(T, n);
    t.blocks = t.tiles;
}

size_t angle_bytes(const HeadArgs &a) { return sizeof(float) * (size_t)a.R * std::max(a.q.tokens, a.k.tokens); }

// Blocks of the backward pass: `most` in all, shared by rows.
constexpr int kBackBlocks = 3 * kSms;
void set_backward(HeadArgs &a, int T, int q_heads, int k_heads) {
    const int rounds = 4;
    set_tiles(a.q, T, q_heads, a.R, a.lg, rounds);
    set_tiles(a.k, T, k_heads, a.R, a.lg, rounds);
    const int for_q = std::max(1, std::min(kBackBlocks - 1, (int)((int64_t)kBackBlocks * q_heads / (q_heads + k_heads))));
    a.q.blocks = std::min(a.q.tiles, for_q);
    a.k.blocks = std::min(a.k.tiles, kBackBlocks - for_q);
}

bool one_each(const HeadArgs &a) { return a.q.blocks == 1 && a.k.blocks == 1; }   // whose sums are the result

template <int DT, bool kPairs> cudaError_t launch_forward(const HeadArgs &a, cudaStream_t st) {
    constexpr int U = DT == MOE_DTYPE_F32 ? 2 : 4;
    return launch_pdl(k_head_norm<DT, kPairs, U>, dim3(a.q.blocks + a.k.blocks), dim3(kThreads), angle_bytes(a), st, a);
}

template <int DT, bool kPairs> cudaError_t launch_backward(const HeadArgs &a, cudaStream_t st) {
    constexpr int U = DT == MOE_DTYPE_F32 ? 1 : 2;
    const size_t sums = sizeof(float) * (size_t)(kThreads >> a.lg) * a.D;
    return launch_pdl(k_head_norm_backward<DT, kPairs, U>, dim3(a.q.blocks + a.k.blocks), dim3(kThreads),
                      std::max(angle_bytes(a), sums), st, a);
}

moe_status check_heads(int32_t T, int32_t q_heads, int32_t k_heads, int32_t D, int32_t R, int32_t interleaved, int32_t dtype, float eps) {
    if (T < 0 || !known_dtype(dtype) || (interleaved & ~1)) return MOE_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
    if (q_heads < 1 || q_heads > kMaxHeads || k_heads < 1 || k_heads > kMaxHeads) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (D < 16 || D > kMaxDim || D % 16 || R < 0 || R > D || R % 16) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

bool good_stride(int64_t stride, int32_t heads, int32_t D) { return stride >= (int64_t)heads * D && stride % kChunk == 0; }

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

moe_status moe_head_norm(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *q_weight,
                         const void *k_weight, const int32_t *positions, const uint64_t *turns, int32_t T,
                         int32_t q_heads, int32_t k_heads, int32_t D, int32_t R, int32_t interleaved, int32_t dtype,
                         float eps, void *q_out, int64_t q_out_stride, void *k_out, int64_t k_out_stride, void *stream) {
    const moe_status st = check_heads(T, q_heads, k_heads, D, R, interleaved, dtype, eps);
    if (st != MOE_OK) return st;
    if (!good_stride(q_stride, q_heads, D) || !good_stride(k_stride, k_heads, D) || !good_stride(q_out_stride, q_heads, D) ||
        !good_stride(k_out_stride, k_heads, D))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!q || !k || !q_weight || !k_weight || !q_out || !k_out || (R > 0 && (!positions || !turns))) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(q_weight, 16) || !aligned_to(k_weight, 16) || !aligned_to(q_out, 16) ||
        !aligned_to(k_out, 16) || !aligned_to(positions, 4) || !aligned_to(turns, 8))
        return MOE_ERR_MISALIGNED;
    HeadArgs a{};
    a.q = HeadTensor{q, q_weight, nullptr, q_out, q_stride, q_out_stride};
    a.k = HeadTensor{k, k_weight, nullptr, k_out, k_stride, k_out_stride};
    a.pos = positions;
    a.turns = turns;
    a.T = T;
    a.D = D;
    a.R = R;
    a.lg = lanes_log(D);
    a.eps = eps;
    a.inv_d = 1.0f / (float)D;
    const int rounds = dtype == MOE_DTYPE_F32 ? 2 : 4;
    set_tiles(a.q, T, q_heads, R, a.lg, rounds);
    set_tiles(a.k, T, k_heads, R, a.lg, rounds);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MOE_DTYPE_F32:
            return cuda_status(interleaved ? launch_forward<MOE_DTYPE_F32, true>(a, s) : launch_forward<MOE_DTYPE_F32, false>(a, s));
        case MOE_DTYPE_BF16:
            return cuda_status(interleaved ? launch_forward<MOE_DTYPE_BF16, true>(a, s) : launch_forward<MOE_DTYPE_BF16, false>(a, s));
        default:
            return cuda_status(interleaved ? launch_forward<MOE_DTYPE_F16, true>(a, s) : launch_forward<MOE_DTYPE_F16, false>(a, s));
    }
}

size_t moe_head_norm_backward_workspace(int32_t T, int32_t q_heads, int32_t k_heads, int32_t D, int32_t R) {
    if (T < 1 || check_heads(T, q_heads, k_heads, D, R, 0, MOE_DTYPE_F32, 1.0f) != MOE_OK) return 0;
    HeadArgs a{};
    a.R = R;
    a.lg = lanes_log(D);
    set_backward(a, T, q_heads, k_heads);
    return one_each(a) ? 0 : sizeof(float) * (size_t)(a.q.blocks + a.k.blocks) * (size_t)D;
}

moe_status moe_head_norm_backward(const void *grad_q, int64_t grad_q_stride, const void *grad_k, int64_t grad_k_stride,
                                  const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                  const void *q_weight, const void *k_weight, const int32_t *positions,
                                  const uint64_t *turns, int32_t T, int32_t q_heads, int32_t k_heads, int32_t D,
                                  int32_t R, int32_t interleaved, int32_t dtype, float eps, void *grad_q_in,
                                  void *grad_k_in, float *grad_qw, float *grad_kw, void *workspace,
                                  size_t workspace_bytes, void *stream) {
    const moe_status st = check_heads(T, q_heads, k_heads, D, R, interleaved, dtype, eps);
    if (st != MOE_OK) return st;
    if (!good_stride(q_stride, q_heads, D) || !good_stride(k_stride, k_heads, D) || !good_stride(grad_q_stride, q_heads, D) ||
        !good_stride(grad_k_stride, k_heads, D))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (!grad_qw || !grad_kw) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!grad_q || !grad_k || !q || !k || !q_weight || !k_weight || !grad_q_in || !grad_k_in ||
                  (R > 0 && (!positions || !turns))))
        return MOE_ERR_INVALID_ARG;
    const size_t need = moe_head_norm_backward_workspace(T, q_heads, k_heads, D, R);
    if (need > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(grad_q, 16) || !aligned_to(grad_k, 16) || !aligned_to(q, 16) || !aligned_to(k, 16) || !aligned_to(q_weight, 16) ||
        !aligned_to(k_weight, 16) || !aligned_to(grad_q_in, 16) || !aligned_to(grad_k_in, 16) || !aligned_to(positions, 4) ||
        !aligned_to(turns, 8) || !aligned_to(grad_qw, 4) || !aligned_to(grad_kw, 4) || !aligned_to(workspace, 16))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        const cudaError_t e = cudaMemsetAsync(grad_qw, 0, sizeof(float) * D, s);
        return cuda_status(e != cudaSuccess ? e : cudaMemsetAsync(grad_kw, 0, sizeof(float) * D, s));
    }
    HeadArgs a{};
    a.q = HeadTensor{q, q_weight, grad_q, grad_q_in, q_stride, (int64_t)q_heads * D, grad_q_stride};
    a.k = HeadTensor{k, k_weight, grad_k, grad_k_in, k_stride, (int64_t)k_heads * D, grad_k_stride};
    a.pos = positions;
    a.turns = turns;
    a.T = T;
    a.D = D;
    a.R = R;
    a.lg = lanes_log(D);
    a.eps = eps;
    a.inv_d = 1.0f / (float)D;
    set_backward(a, T, q_heads, k_heads);
    const bool direct = one_each(a);
    a.q.sums = direct ? grad_qw : static_cast<float *>(workspace);
    a.k.sums = direct ? grad_kw : static_cast<float *>(workspace) + (size_t)a.q.blocks * D;
    cudaError_t e;
    switch (dtype) {
        case MOE_DTYPE_F32: e = interleaved ? launch_backward<MOE_DTYPE_F32, true>(a, s) : launch_backward<MOE_DTYPE_F32, false>(a, s); break;
        case MOE_DTYPE_BF16: e = interleaved ? launch_backward<MOE_DTYPE_BF16, true>(a, s) : launch_backward<MOE_DTYPE_BF16, false>(a, s); break;
        default: e = interleaved ? launch_backward<MOE_DTYPE_F16, true>(a, s) : launch_backward<MOE_DTYPE_F16, false>(a, s); break;
    }
    if (e != cudaSuccess || direct) return cuda_status(e);
    return cuda_status(launch_pdl(k_head_norm_grad_w, dim3((D + 31) / 32, 2), dim3(8 * kColumnGroups), 0, s, (const float *)a.q.sums,
                                  a.q.blocks, (const float *)a.k.sums, a.k.blocks, (int)D, grad_qw, grad_kw));
}

}  // extern "C"
