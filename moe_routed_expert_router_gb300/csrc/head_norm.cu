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
// Layout: 2^lg lanes a row, 16 values a lane in 16-byte words (two of 16-bit values,
// four of fp32 ones) a step apart, so that neighbouring lanes touch neighbouring
// words and the second half of a lane's words holds the partners of the first
// (half-split planes) or every word whole planes (interleaved ones): a rotation needs
// no other lane's values, and a lane has eight planes (a, b) either way.  A block takes a tile of tokens of the queries or
// of the keys; the tile's sines and cosines are computed once into shared memory.  A
// group of lanes stays with one token and walks over its heads, so what a token and
// a place in the row give (sines, cosines, weights, and in the forward pass their
// products) is in registers and a row costs its own arithmetic only, in packed fp32.
//
// Bound by HBM, reading and writing every row once: bf16 4096 x 72 heads of 128 26.2
// us (5.8 TB/s, 86 % of the copy bandwidth; with four rows a thread at once 30), fp32
// 8192 x 40 53 us (94 %); backward 8192 x 36 42.8 us (79 %), fp32 8192 x 40 82 us (91
// %).  Rows whose values are not a power of two leave lanes idle (28 + 4 heads of 80:
// 58 and 52 %).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kThreads = 256;
constexpr int kMaxHeads = 1024, kMaxDim = 512;
constexpr int kEach = 8;                   // heads that share what a group of lanes has of a token

// Queries or keys: rows [T][heads][D], `stride` values from token to token.
struct HeadTensor {
    const void *x, *w, *g;                 // g: the output's gradient (backward)
    void *out;
    int64_t stride, out_stride, g_stride;
    float *sums;                           // backward: [blocks][D] partial sums of grad_w
    int heads, split;                      // 2^split groups of lanes share a token's heads
    int tokens, tiles, blocks;             // tokens a tile (2^-split of the groups), tiles, blocks that share them
};

struct HeadArgs {
    HeadTensor q, k;
    const int32_t *pos;
    const uint64_t *turns;
    int T, D, R, lg;
    float eps, inv_d;
    int ring_at;                           // backward: of the ring in shared memory, in floats
};

// What a thread is in its row.
struct Lane {
    int groups, c, p0, step;               // rows of the block at once; its place in one, its words p0, p0 + step, ..
    int token, head, heads;                // of the tile; its first head, and heads from one to the next
    bool on, turned;
};

// A lane's words of a row, and values a word.
template <int DT> constexpr int kWords = DT == MOE_DTYPE_F32 ? 4 : 2;
template <int DT> struct Words { uint4 w[kWords<DT>]; };


template <int DT> __device__ __forceinline__ Lane lane_of(const HeadArgs &a, const HeadTensor &h) {
    Lane l;
    const int group = threadIdx.x >> a.lg;
    l.c = threadIdx.x & ((1 << a.lg) - 1);
    l.groups = blockDim.x >> a.lg;
    l.heads = 1 << h.split;
    l.head = group & (l.heads - 1);        // neighbouring groups have neighbouring heads
    l.token = group >> h.split;
    const int planes = a.R >> 4;           // lanes whose words turn
    l.on = l.c < (a.D >> 4);
    l.turned = l.c < planes;
    l.p0 = l.turned ? l.c : l.c - planes + a.R / kPieceValues<DT>;
    l.step = l.turned ? planes : (a.D - a.R) >> 4;
    return l;
}

// Sines and cosines of `n` tokens from t0 on: cos [n][R / 2], then sin, in the
// planes' order but for half-split planes of 16-bit values, whose lane c has planes
// 8 c .. 8 c + 7: these lie at 16-byte places c and c + R / 16 as well.
template <int DT, bool kPairs>
__device__ __forceinline__ void fill_angles(const HeadArgs &a, int t0, int n, float *cs) {
    const int half = a.R >> 1, planes = a.R >> 4;
    if (half == 0) return;
    int t = (int)threadIdx.x / half, i = (int)threadIdx.x - t * half;
    const int more_t = (int)blockDim.x / half, more_i = (int)blockDim.x - more_t * half;
    while (t < n) {
        const uint64_t turn = (uint64_t)(int64_t)a.pos[t0 + t] * a.turns[i];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 0x1p-31f, &s, &c);              // 2^63 is half a turn
        const int at = kPairs || DT == MOE_DTYPE_F32 ? i : (((i >> 2) & 1) * planes + (i >> 3)) * 4 + (i & 3);
        cs[t * half + at] = c;
        cs[(n + t) * half + at] = s;
        t += more_t;
        i += more_i;
        if (i >= half) {
            i -= half;
            ++t;
        }
    }
}

struct Angles { float c[8], s[8]; };

template <int DT, bool kPairs> __device__ __forceinline__ Angles angles_of(const HeadArgs &a, const Lane &l, const float *cs, int n) {
    Angles r;
    if (l.turned && l.token < n) {
        const int half = a.R >> 1;
        using F = std::conditional_t<kPairs && DT == MOE_DTYPE_F32, float2, float4>;      // the planes of a word, or of two
        constexpr int N = sizeof(F) / sizeof(float);
        const F *c = reinterpret_cast<const F *>(cs + l.token * half), *s = reinterpret_cast<const F *>(cs + (n + l.token) * half);
#pragma unroll
        for (int w = 0; w < 8 / N; ++w) {
            *reinterpret_cast<F *>(r.c + N * w) = c[l.c + w * l.step];
            *reinterpret_cast<F *>(r.s + N * w) = s[l.c + w * l.step];
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            r.c[i] = 1.0f;
            r.s[i] = 0.0f;
        }
    }
    return r;
}

// Where value a (b) of the lane's plane i is: its word, and its place in it.
template <int DT, bool kPairs> __device__ __forceinline__ constexpr int word_of(int i, int b) {
    return DT == MOE_DTYPE_F32 ? (kPairs ? i >> 1 : (i >> 2) + 2 * b) : (kPairs ? i >> 2 : b);
}
template <int DT, bool kPairs> __device__ __forceinline__ constexpr int place_of(int i, int b) {
    return DT == MOE_DTYPE_F32 ? (kPairs ? 2 * (i & 1) + b : i & 3) : (kPairs ? 2 * (i & 3) + b : i);
}

// The lane's words as eight planes (a, b), and back.
template <int DT, bool kPairs> __device__ __forceinline__ void to_planes(const Words<DT> &r, float (&a)[8], float (&b)[8]) {
    float v[kWords<DT>][kPieceValues<DT>];
#pragma unroll
    for (int w = 0; w < kWords<DT>; ++w) widen_piece<DT>(r.w[w], v[w]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a[i] = v[word_of<DT, kPairs>(i, 0)][place_of<DT, kPairs>(i, 0)];
        b[i] = v[word_of<DT, kPairs>(i, 1)][place_of<DT, kPairs>(i, 1)];
    }
}
template <int DT, bool kPairs>
__device__ __forceinline__ void store_planes(typename RowType<DT>::T *p, const Lane &l, const float (&a)[8], const float (&b)[8]) {
    float v[kWords<DT>][kPieceValues<DT>];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[word_of<DT, kPairs>(i, 0)][place_of<DT, kPairs>(i, 0)] = a[i];
        v[word_of<DT, kPairs>(i, 1)][place_of<DT, kPairs>(i, 1)] = b[i];
    }
#pragma unroll
    for (int w = 0; w < kWords<DT>; ++w) st16(p + kPieceValues<DT> * (l.p0 + w * l.step), narrow_piece<DT>(v[w]));
}

// r = x * y,  r += x * y  of eight values, two an instruction.
__device__ __forceinline__ void mul8(float (&r)[8], const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2)
        asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 z, x, y;\n\t"
            "mov.b64 {%0, %1}, z;\n\t}"
            : "=f"(r[i]), "=f"(r[i + 1]) : "f"(x[i]), "f"(x[i + 1]), "f"(y[i]), "f"(y[i + 1]));
}
__device__ __forceinline__ void mul8(float (&r)[8], const float (&x)[8], float y) {
    const float all[8] = {y, y, y, y, y, y, y, y};
    mul8(r, x, all);
}
__device__ __forceinline__ void fma8(float (&r)[8], const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) fma2(r[i], r[i + 1], x[i], x[i + 1], y[i], y[i + 1]);
}
__device__ __forceinline__ void fma8(float (&r)[8], const float (&x)[8], float y) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) fma2(r[i], r[i + 1], x[i], x[i + 1], y, y);
}
// The sum of x * y added to two halves s.
__device__ __forceinline__ void dot8(float (&s)[2], const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) fma2(s[0], s[1], x[i], x[i + 1], y[i], y[i + 1]);
}
__device__ __forceinline__ void scale8(float (&r)[8], float y) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(r, i, y, y);
}

template <int DT> __device__ __forceinline__ void fetch_row(const typename RowType<DT>::T *p, const Lane &l, Words<DT> &r) {
#pragma unroll
    for (int w = 0; w < kWords<DT>; ++w) r.w[w] = ld16(p + kPieceValues<DT> * (l.p0 + w * l.step));
}
template <int DT> __device__ __forceinline__ void fetch_weight(const void *from, const Lane &l, Words<DT> &r) {
    r = Words<DT>{};
    if (l.on) {
#pragma unroll
        for (int w = 0; w < kWords<DT>; ++w)
            r.w[w] = ld16_shared(static_cast<const typename RowType<DT>::T *>(from) + kPieceValues<DT> * (l.p0 + w * l.step));
    }
}

__device__ __forceinline__ void over_row(float &v, int lg) {
    for (int o = 1 << lg >> 1; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
}
__device__ __forceinline__ void over_row(float &v, float &w, int lg) {
    for (int o = 1 << lg >> 1; o >= 1; o >>= 1) {
        v += __shfl_xor_sync(0xffffffffu, v, o);
        w += __shfl_xor_sync(0xffffffffu, w, o);
    }
}

// U rows a thread at once, all loads ahead of their use.  kRest: R < D, some values are not rotated.
template <int DT, bool kPairs, int U, bool kRest>
__global__ void __launch_bounds__(kThreads) k_head_norm(HeadArgs a) {
    using T = typename RowType<DT>::T;
    extern __shared__ __align__(16) float cs[];
    const bool key = (int)blockIdx.x >= a.q.blocks;
    const HeadTensor h = key ? a.k : a.q;
    const int t0 = ((int)blockIdx.x - (key ? a.q.blocks : 0)) * h.tokens, n = min(h.tokens, a.T - t0);
    const Lane l = lane_of<DT>(a, h);
    const bool on = l.on && l.token < n;
    pdl_wait();
    pdl_trigger();
    Words<DT> x[U], wr;
    const int64_t pitch = (int64_t)l.heads * a.D;                   // from a row to the thread's next one
    const T *from = static_cast<const T *>(h.x) + (int64_t)(t0 + l.token) * h.stride + l.head * a.D;
    T *to = static_cast<T *>(h.out) + (int64_t)(t0 + l.token) * h.out_stride + l.head * a.D;
    int left = on ? (h.heads - l.head + l.heads - 1) >> h.split : 0;             // rows of this thread
    auto fetch = [&]() {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = Words<DT>{};
            if (u < left) fetch_row<DT>(from + u * pitch, l, x[u]);
        }
        from += U * pitch;
    };
    fetch();
    fetch_weight<DT>(h.w, l, wr);
    fill_angles<DT, kPairs>(a, t0, n, cs);
    __syncthreads();
    // a' = rstd (a (cos wa) - b (sin wb)),  b' = rstd (b (cos wb) + a (sin wa))
    float wa[8], wb[8], ca[8], cb[8], sa[8], sb[8];
    {
        const Angles r = angles_of<DT, kPairs>(a, l, cs, n);
        to_planes<DT, kPairs>(wr, wa, wb);
        mul8(ca, wa, r.c);
        mul8(cb, wb, r.c);
        if (!kRest || l.turned) {          // else nothing of the other value, whatever the weight is
            mul8(sa, wa, r.s);
            mul8(sb, wb, r.s);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) sa[i] = sb[i] = 0.0f;
        }
        scale8(sb, -1.0f);
    }
    for (int base = 0; base < h.heads; base += U * l.heads) {
        if (base > 0) fetch();
        float least = 1.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float va[8], vb[8], ya[8], yb[8], sum[2] = {};
            to_planes<DT, kPairs>(x[u], va, vb);
            dot8(sum, va, va);
            dot8(sum, vb, vb);
            float mean = sum[0] + sum[1];
            over_row(mean, a.lg);
            if (u < left) {
                const float rstd = rsqrtf(fmaf(mean, a.inv_d, a.eps));
                if constexpr (kRest) least = fminf(least, rstd);
                mul8(ya, va, ca);
                fma8(ya, vb, sb);
                mul8(yb, vb, cb);
                fma8(yb, va, sa);
                scale8(ya, rstd);
                scale8(yb, rstd);
                store_planes<DT, kPairs>(to + u * pitch, l, ya, yb);
            }
        }
        // A row with an infinity has an rstd of 0.  Where values are not rotated, 0 (a sine) times the infinity has reached
        // its place's other value above; they are written again, each by itself: 0, the infinity's own NaN.  (4096 x 40 heads
        // of 128, 64 turned: 16.8 us, without this 16.5; with a branch around the sines' products instead 18.8.  Rows that are
        // rotated whole have no such values.)
        if (kRest && least == 0.0f && !l.turned) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float va[8], vb[8];
#pragma unroll
                for (int w = 0; w < kWords<DT>; ++w)                // widened anew: kept from above they took 114 registers
                    asm volatile("" : "+r"(x[u].w[w].x), "+r"(x[u].w[w].y), "+r"(x[u].w[w].z), "+r"(x[u].w[w].w));
                to_planes<DT, kPairs>(x[u], va, vb);
                bool infinite = false;
#pragma unroll
                for (int i = 0; i < 8; ++i) infinite |= isinf(va[i]) || isinf(vb[i]);
                if (!infinite || u >= left) continue;
                scale8(va, 0.0f);
                scale8(vb, 0.0f);
                mul8(va, va, ca);
                mul8(vb, vb, cb);
                store_planes<DT, kPairs>(to + u * pitch, l, va, vb);
            }
        }
        to += U * pitch;
        left -= U;
    }
}

// Blocks walk over tiles; a thread holds its 16 values' part of grad_w in
// registers until the end, so the order of the sums is fixed.  Its rows come
// through a ring in shared memory, kRing rows deep, that runs on into the next tile
// (a thread reads what it copied itself: no barrier).  In registers, two rows at
// once, 8192 x 36 heads of 128 took 57.6 us.
template <int DT> constexpr int kRing = DT == MOE_DTYPE_F32 ? 3 : 4;
template <int DT> constexpr int kRowWords = 2 * kWords<DT>;                     // of x and of grad
template <int DT> constexpr int kRingBytes = kRing<DT> * kRowWords<DT> * 16 * kThreads;

template <int DT, bool kPairs>
__global__ void __launch_bounds__(kThreads, 2) k_head_norm_backward(HeadArgs a) {
    using T = typename RowType<DT>::T;
    constexpr int W = kWords<DT>, VW = kPieceValues<DT>;
    extern __shared__ __align__(16) float cs[];                     // angles, in the end sums; then the ring
    const bool key = (int)blockIdx.x < a.k.blocks;
    const HeadTensor h = key ? a.k : a.q;
    const int block = (int)blockIdx.x - (key ? 0 : a.k.blocks);
    const Lane l = lane_of<DT>(a, h);
    uint4 *ring = reinterpret_cast<uint4 *>(cs + a.ring_at) + threadIdx.x;
    const int rounds = (h.heads + l.heads - 1) >> h.split;          // rows a thread and tile
    const int64_t pitch = (int64_t)l.heads * a.D;                   // from a row to the thread's next one
    pdl_wait();
    pdl_trigger();
    // the copies: row `cr` of tile `ct` next
    int ct = block, cr = 0, fill = 0;
    const T *cx = nullptr, *cg = nullptr;
    auto tile_at = [&]() {
        const int64_t t = (int64_t)ct * h.tokens + l.token;
        cx = static_cast<const T *>(h.x) + t * h.stride + l.head * a.D + VW * l.p0;
        cg = static_cast<const T *>(h.g) + t * h.g_stride + l.head * a.D + VW * l.p0;
    };
    auto copy_row = [&]() {
        if (ct < h.tiles) {
            if (l.on && l.token < min(h.tokens, a.T - ct * h.tokens) && l.head + cr * l.heads < h.heads) {
                uint4 *to = ring + fill * (kRowWords<DT> * kThreads);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    copy16(to + w * kThreads, cx + VW * w * l.step, true);
                    copy16(to + (W + w) * kThreads, cg + VW * w * l.step, true);
                }
            }
            cx += pitch;
            cg += pitch;
            if (++cr == rounds) {
                cr = 0;
                ct += h.blocks;
                tile_at();
            }
        }
        copy_commit();
        if (++fill == kRing<DT>) fill = 0;
    };
    tile_at();
#pragma unroll
    for (int i = 0; i < kRing<DT> - 1; ++i) copy_row();
    int slot = 0;
    float wa[8], wb[8], gwa[8] = {}, gwb[8] = {};
    {
        Words<DT> wr;
        fetch_weight<DT>(h.w, l, wr);
        to_planes<DT, kPairs>(wr, wa, wb);
    }
    for (int tile = block; tile < h.tiles; tile += h.blocks) {
        const int t0 = tile * h.tokens, n = min(h.tokens, a.T - t0);
        const bool on = l.on && l.token < n;
        T *to = static_cast<T *>(h.out) + (int64_t)(t0 + l.token) * h.out_stride + l.head * a.D;
        __syncthreads();                   // the tile before is done with the angles
        fill_angles<DT, kPairs>(a, t0, n, cs);
        __syncthreads();
        const Angles r = angles_of<DT, kPairs>(a, l, cs, n);
        float minus[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) minus[i] = -r.s[i];
        for (int row = 0; row < rounds; ++row) {
            copy_row();
            copy_wait<kRing<DT> - 1>();
            const uint4 *at = ring + slot * (kRowWords<DT> * kThreads);
            if (++slot == kRing<DT>) slot = 0;
            const bool mine = on && l.head + row * l.heads < h.heads;
            Words<DT> x{}, g{};
            if (mine) {
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    x.w[w] = at[w * kThreads];
                    g.w[w] = at[(W + w) * kThreads];
                }
            }
            float va[8], vb[8], fa[8], fb[8], sum[2] = {}, dot[2] = {};
            {
                float ga[8], gb[8];
                to_planes<DT, kPairs>(g, ga, gb);
                mul8(fa, ga, r.c);         // turned back
                mul8(fb, gb, r.c);
                if (l.turned) {            // else a and b are no pair: 0 times an infinity would reach the other
                    fma8(fa, gb, r.s);
                    fma8(fb, ga, minus);
                }
            }
            to_planes<DT, kPairs>(x, va, vb);
            dot8(sum, va, va);
            dot8(sum, vb, vb);
            float pa[8], pb[8];            // g w
            mul8(pa, fa, wa);
            mul8(pb, fb, wb);
            dot8(dot, pa, va);
            dot8(dot, pb, vb);
            float mean = sum[0] + sum[1], both = dot[0] + dot[1];
            over_row(mean, both, a.lg);
            if (mine) {
                const float rstd = rsqrtf(fmaf(mean, a.inv_d, a.eps));
                const float back = -(both * rstd * a.inv_d) * rstd;              // - rstd mean(g w n^)
                float na[8], nb[8];
                mul8(na, va, rstd);
                mul8(nb, vb, rstd);
                fma8(gwa, fa, na);
                fma8(gwb, fb, nb);
                scale8(pa, rstd);
                scale8(pb, rstd);
                fma8(pa, na, back);
                fma8(pb, nb, back);
                store_planes<DT, kPairs>(to, l, pa, pb);
            }
            to += pitch;
        }
    }
    // the groups' sums, [groups][D], added in order
    __syncthreads();
    if (l.on) {
        float *mine = cs + (threadIdx.x >> a.lg) * a.D;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mine[VW * (l.p0 + word_of<DT, kPairs>(i, 0) * l.step) + place_of<DT, kPairs>(i, 0)] = gwa[i];
            mine[VW * (l.p0 + word_of<DT, kPairs>(i, 1) * l.step) + place_of<DT, kPairs>(i, 1)] = gwb[i];
        }
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

// The tile of one tensor: about `each` heads a group of lanes, fewer where tokens
// are so few that their tiles would not fill the card.
void set_tiles(HeadTensor &t, int T, int heads, int lg, int each) {
    int groups_log = 0;
    while ((kThreads >> lg) >> (groups_log + 1)) ++groups_log;
    t.heads = heads;
    t.split = 0;
    while (t.split < groups_log && (heads > each << t.split || T >> (groups_log - t.split) < 2 * kSms) && 1 << t.split < heads) ++t.split;
    t.tokens = 1 << (groups_log - t.split);
    while (t.tokens > 1 && t.tokens > T) t.tokens /= 2;
    t.tiles = blocks_of(T, t.tokens);
    t.blocks = t.tiles;
}

size_t angle_bytes(const HeadArgs &a) { return sizeof(float) * (size_t)a.R * std::max(a.q.tokens, a.k.tokens); }

// Blocks of the backward pass, shared by work: a row of a thread costs about three
// times a sine and cosine (a tile of few heads has many tokens: shared by rows, 8192
// tokens of 32 and 4 heads took 57 us, the keys' blocks half as long again).
constexpr int kBackBlocks = 2 * kSms;
int64_t work(const HeadTensor &t, int R) {
    return (int64_t)t.tiles * (3 * blocks_of(t.heads, 1 << t.split) + (t.tokens * (R / 2) + kThreads - 1) / kThreads);
}
void set_backward(HeadArgs &a, int T, int q_heads, int k_heads) {
    set_tiles(a.q, T, q_heads, a.lg, kEach);
    set_tiles(a.k, T, k_heads, a.lg, kEach);
    const int64_t for_q = kBackBlocks * work(a.q, a.R) / (work(a.q, a.R) + work(a.k, a.R));
    const int q = (int)std::max<int64_t>(1, std::min<int64_t>(kBackBlocks - 1, for_q));
    a.q.blocks = std::min(a.q.tiles, q);
    a.k.blocks = std::min(a.k.tiles, kBackBlocks - q);
}

bool one_each(const HeadArgs &a) { return a.q.blocks == 1 && a.k.blocks == 1; }   // whose sums are the result

template <int DT, bool kPairs> cudaError_t launch_forward(const HeadArgs &a, cudaStream_t st) {
    constexpr int U = DT == MOE_DTYPE_F32 ? 1 : 2;
    return launch_pdl(a.R < a.D ? k_head_norm<DT, kPairs, U, true> : k_head_norm<DT, kPairs, U, false>, dim3(a.q.blocks + a.k.blocks),
                      dim3(kThreads), angle_bytes(a), st, a);
}

template <int DT, bool kPairs> cudaError_t launch_backward(const HeadArgs &a, cudaStream_t st) {
    const cudaError_t e = allow_smem<k_head_norm_backward<DT, kPairs>>();
    if (e != cudaSuccess) return e;
    const size_t sums = sizeof(float) * (size_t)(kThreads >> a.lg) * a.D, front = std::max(angle_bytes(a), sums);
    HeadArgs b = a;
    b.ring_at = (int)(front / sizeof(float));
    return launch_pdl(k_head_norm_backward<DT, kPairs>, dim3(a.q.blocks + a.k.blocks), dim3(kThreads), front + kRingBytes<DT>, st, b);
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
    set_tiles(a.q, T, q_heads, a.lg, kEach);
    set_tiles(a.k, T, k_heads, a.lg, kEach);
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
