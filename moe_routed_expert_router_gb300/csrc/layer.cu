// The whole mixture-of-experts layer of up to 16 tokens with experts in bf16, f16
// or fp32, in two launches:
//   k_layer_logits  router logits in moe_route's order (route.cu), a block an expert;
//   k_layer         top-k and weights, then gate, up and SwiGLU of the chosen
//                   experts, then down, the sum over a token's experts, the shared
//                   expert and the base.
//
//   h[p] = w[p] * silu(gate_e x_t) * (up_e x_t),   out[t] = sum over p of down_e h[p]
//
// Bound by the bytes of the chosen experts' weights, each read once.  A few tokens
// an expert leave the tensor cores nothing to win: at the memory's rate an SM
// sub-partition has 88 issue slots for every 16 bytes a lane loads, and a token
// costs 4 packed FMAs of them, so the products are fp32 on the CUDA cores, exact
// in every type, and h stays in fp32.
//
// Every block chooses the experts itself (a microsecond, against a launch and its
// gap).  Gate and up rows are handed out by a ticket counter in small pieces, so
// the last piece is short and no block has to be resident for another's sake: a
// wait for the pieces is a wait for blocks that already run.  The rows of down are
// split evenly beforehand; a block sums its rows over all experts, so nothing is
// added through memory and equal inputs give equal bits.
#include <algorithm>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kSms = 152;
constexpr int kMaxTokens = 16, kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxWidth = 16384;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRows = 4;                   // weight rows a warp streams at once: two features' gate and up, or four rows of down

struct LayerArgs {
    const void *x, *router;
    const float *bias;
    const void *gate, *up, *down;          // [E][I][H], [E][I][H], [E][H][I]
    const void *sgate, *sup, *sdown;       // the shared expert's or null
    const void *base;
    void *out;
    int32_t *ids;
    float *wts;
    float *logits, *h;                     // [T][E]; [T * k][I], then [T][Is]
    int *count;                            // [0] pieces handed out, [1] pieces done
    int T, H, E, I, k, Is, kind, renorm;
};

// ------------------------------------------------------------ logits

constexpr int kLogitThreads = 256;

template <int RT> struct RouterWord { using T = float; };
template <> struct RouterWord<MOE_ROUTER_BF16> { using T = __nv_bfloat16; };
template <typename T> __device__ __forceinline__ float as_f32(T v) { return static_cast<float>(v); }

// Position p of H belongs to lane p mod 32, which adds its products in increasing p; then an xor butterfly and the bias:
// the order of moe_route, so both choose the same experts.
template <int DT, int RT>
__global__ void __launch_bounds__(kLogitThreads) k_layer_logits(LayerArgs a, int tokens) {
    using X = typename RowType<DT>::T;
    using W = typename RouterWord<RT>::T;
    extern __shared__ __align__(16) uint8_t smem[];
    W *w = reinterpret_cast<W *>(smem);                             // the router's row
    X *x = reinterpret_cast<X *>(smem + sizeof(W) * a.H);           // `tokens` rows of x
    const int e = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    if (e == 0 && threadIdx.x < 2) a.count[threadIdx.x] = 0;
    const uint8_t *from = reinterpret_cast<const uint8_t *>(static_cast<const W *>(a.router) + (int64_t)e * a.H);
    for (int i = 16 * threadIdx.x; i < (int)sizeof(W) * a.H; i += 16 * kLogitThreads) copy16(smem + i, from + i, true);
    for (int t0 = 0; t0 < a.T; t0 += tokens) {
        const int n = min(tokens, a.T - t0);
        const uint8_t *rows = reinterpret_cast<const uint8_t *>(static_cast<const X *>(a.x) + (int64_t)t0 * a.H);
        if (t0 > 0) __syncthreads();
        for (int i = 16 * threadIdx.x; i < (int)sizeof(X) * a.H * n; i += 16 * kLogitThreads)
            copy16(reinterpret_cast<uint8_t *>(x) + i, rows + i, true);
        copy_commit();
        copy_wait<0>();
        __syncthreads();
        for (int t = warp; t < n; t += kLogitThreads / 32) {
            float acc = 0.0f;
#pragma unroll 8
            for (int p = lane; p < a.H; p += 32) acc = fmaf(as_f32(x[t * a.H + p]), as_f32(w[p]), acc);
            acc = warp_sum(acc);
            if (lane == 0) a.logits[(t0 + t) * a.E + e] = a.bias ? acc + a.bias[e] : acc;
        }
    }
}

// ------------------------------------------------------------ choice of experts

// The block's view of the routing.
struct Routing {
    unsigned *mask;                        // [E] the tokens that chose an expert, a bit each
    int *first;                            // [E] its first pair
    int *expert, *start;                   // the chosen experts in increasing order (E: the shared one) and their first pairs
    int *token;                            // [pairs] token of a pair
    float *weight;                         // [pairs]
    int *n;                                // chosen experts, the shared one included
};

__host__ __device__ inline size_t routing_bytes(int E) { return sizeof(int) * (2 * (size_t)E + 4 * (kMaxPairs + kMaxTokens + 2) + 4); }

__device__ __forceinline__ Routing routing_at(uint8_t *smem, int E) {
    constexpr int P = kMaxPairs + kMaxTokens + 2;
    int *at = reinterpret_cast<int *>(smem);
    Routing r;
    r.mask = reinterpret_cast<unsigned *>(at);
    r.first = at + E;
    r.expert = r.first + E;
    r.start = r.expert + P;
    r.token = r.start + P;
    r.weight = reinterpret_cast<float *>(r.token + P);
    r.n = r.token + 2 * P;
    return r;
}

// Larger logit, larger key; a NaN lies below every other value and is chosen last.  0 is no key.
__device__ __forceinline__ uint32_t key_of(float v) {
    const uint32_t b = __float_as_uint(v);
    if (v != v) return 1u;
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

// Top-k and weights of token t by one warp, as moe_route's (ties to the lower id, the same sums); keys [E] in shared memory.
__device__ void choose(const LayerArgs &a, const Routing &r, int t, uint32_t *keys, int32_t *chosen, float *weights) {
    const int lane = threadIdx.x & 31;
    const float *logits = a.logits + t * a.E;
    float top = -INFINITY;
    for (int e = lane; e < a.E; e += 32) {
        const float v = logits[e];
        keys[e] = key_of(v);
        top = fmaxf(top, v);
    }
    float mine = 0.0f;
    int id = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = 0u;
        int at = 0x7fffffff;
        for (int e = lane; e < a.E; e += 32)
            if (keys[e] > best) { best = keys[e]; at = e; }
        const uint32_t k = __reduce_max_sync(0xffffffffu, best);
        const int e = (int)__reduce_min_sync(0xffffffffu, best == k ? (uint32_t)at : 0x7fffffffu);   // k <= E: there is one
        if ((e & 31) == lane) keys[e] = 0u;
        if (lane == j) {
            mine = logits[e];
            id = e;
        }
    }
    float num, den = 1.0f;
    if (a.kind == MOE_ROUTER_SOFTMAX) {
        top = warp_max(top);
        num = lane < a.k ? expf(mine - top) : 0.0f;
        if (a.renorm) {
            den = warp_sum(num);
        } else {
            float s = 0.0f;
            for (int e = lane; e < a.E; e += 32) s += expf(logits[e] - top);
            den = warp_sum(s);
        }
    } else {
        num = lane < a.k ? 1.0f / (1.0f + expf(-mine)) : 0.0f;
        if (a.renorm) den = warp_sum(num);
    }
    if (lane < a.k) {
        chosen[t * a.k + lane] = id;
        weights[t * a.k + lane] = num / den;
        atomicOr(&r.mask[id], 1u << t);
        if (blockIdx.x == 0) {
            a.ids[t * a.k + lane] = id;
            a.wts[t * a.k + lane] = num / den;
        }
    }
}

// `scratch`: keys [16 warps][E], then chosen and weights [T * k] each.
__device__ void route(const LayerArgs &a, const Routing &r, uint8_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t *keys = reinterpret_cast<uint32_t *>(scratch) + warp * a.E;
    int32_t *chosen = reinterpret_cast<int32_t *>(scratch) + kWarps * a.E;
    float *weights = reinterpret_cast<float *>(chosen + kMaxPairs);
    for (int e = threadIdx.x; e < a.E; e += kThreads) r.mask[e] = 0u;
    __syncthreads();
    if (warp < a.T) choose(a, r, warp, keys, chosen, weights);
    __syncthreads();
    if (warp == 0) {
        int n = 0, pairs = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, c = e < a.E ? __popc(r.mask[e]) : 0;
            const unsigned used = __ballot_sync(0xffffffffu, c > 0);
            int sum = c;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (c > 0) {
                const int i = n + __popc(used & ((1u << lane) - 1u));
                r.expert[i] = e;
                r.start[i] = r.first[e] = pairs + sum - c;
            }
            n += __popc(used);
            pairs += __shfl_sync(0xffffffffu, sum, 31);
        }
        if (a.Is > 0) {
            if (lane == 0) {
                r.expert[n] = a.E;
                r.start[n] = pairs;
            }
            if (lane < a.T) {
                r.token[pairs + lane] = lane;
                r.weight[pairs + lane] = 1.0f;
            }
            ++n;
            pairs += a.T;
        }
        if (lane == 0) {
            r.start[n] = pairs;
            *r.n = n;
        }
    }
    __syncthreads();
    for (int p = threadIdx.x; p < a.T * a.k; p += kThreads) {
        const int e = chosen[p], t = p / a.k;
        const int at = r.first[e] + __popc(r.mask[e] & ((1u << t) - 1u));
        r.token[at] = t;
        r.weight[at] = weights[p];
    }
    __syncthreads();
}

// ------------------------------------------------------------ products

// acc[i][j] = dot(row i, x_j) over the warp: every lane has every sum.  Eight values a lane and step, two steps' loads
// ahead of their use.
template <int DT, int XT, int M>
__device__ __forceinline__ void dots(const typename RowType<DT>::T *const (&row)[kRows], const typename RowType<XT>::T *const (&x)[M], int K,
                                     float (&sum)[kRows][M]) {
    const int lane = threadIdx.x & 31;
    float acc[kRows][M][2] = {};
    for (int k = 8 * lane; k < K; k += 512) {
        Raw8<DT> w[2][kRows];
        const bool second = k + 256 < K;
#pragma unroll
        for (int i = 0; i < kRows; ++i) w[0][i] = load8<DT>(row[i] + k);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
            w[1][i] = Raw8<DT>{};
            if (second) w[1][i] = load8<DT>(row[i] + k + 256);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            if (s == 1 && !second) break;
            float v[kRows][8];
#pragma unroll
            for (int i = 0; i < kRows; ++i) widen8<DT>(w[s][i], v[i]);
#pragma unroll
            for (int j = 0; j < M; ++j) {
                float y[8];
                widen8<XT>(load8_shared<XT>(x[j] + k + 256 * s), y);
#pragma unroll
                for (int i = 0; i < kRows; ++i)
#pragma unroll
                    for (int q = 0; q < 8; q += 2) fma2(acc[i][j][0], acc[i][j][1], v[i][q], v[i][q + 1], y[q], y[q + 1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
        for (int j = 0; j < M; ++j) sum[i][j] = warp_sum(acc[i][j][0] + acc[i][j][1]);
}

// Gate, up and SwiGLU of features f and f + 1 of an expert for its pairs from p on, M at most, into their rows h.
template <int DT, int M>
__device__ void gate_up(const LayerArgs &a, const Routing &r, const typename RowType<DT>::T *const (&row)[kRows], int p, int end, int f, int I, float *h) {
    using T = typename RowType<DT>::T;
    const int lane = threadIdx.x & 31;
    const T *x[M];
#pragma unroll
    for (int j = 0; j < M; ++j) x[j] = static_cast<const T *>(a.x) + r.token[min(p + j, end - 1)] * (int64_t)a.H;
    float s[kRows][M];
    dots<DT, DT, M>(row, x, a.H, s);
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (lane == 2 * j + i && p + j < end) {
                const float g = s[i][j];
                h[(int64_t)j * I + f + i] = g / (1.0f + expf(-g)) * s[2 + i][j] * r.weight[p + j];
            }
}

// Four rows of down of an expert for its pairs from p on, M at most, with rows h: added to the warp's sums [rows][kMaxTokens].
template <int DT, int M>
__device__ void down(const Routing &r, const typename RowType<DT>::T *const (&row)[kRows], const float *h, int p, int end, int I, float *sums) {
    const int lane = threadIdx.x & 31;
    const float *x[M];
#pragma unroll
    for (int j = 0; j < M; ++j) x[j] = h + (int64_t)min(j, end - 1 - p) * I;
    float s[kRows][M];
    dots<DT, MOE_DTYPE_F32, M>(row, x, I, s);
#pragma unroll
    for (int j = 0; j < M; ++j)
#pragma unroll
        for (int i = 0; i < kRows; ++i)
            if (lane == j * kRows + i && p + j < end) sums[i * kMaxTokens + r.token[p + j]] += s[i][j];
    __syncwarp();
}

template <int DT> __device__ __forceinline__ float load_f32(const void *p, int64_t i) { return as_f32(static_cast<const typename RowType<DT>::T *>(p)[i]); }
template <int DT> __device__ __forceinline__ void store_f32(void *p, int64_t i, float v) {
    if constexpr (DT == MOE_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (DT == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

template <int DT>
__global__ void __launch_bounds__(kThreads, 1) k_layer(LayerArgs a) {
    using T = typename RowType<DT>::T;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int ready;
    const Routing r = routing_at(smem, a.E);
    uint8_t *rest = smem + (routing_bytes(a.E) + 15) / 16 * 16;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_trigger();
    route(a, r, rest);
    const int n = *r.n, routed = a.Is > 0 ? n - 1 : n;
    const int each = a.I / 2, pieces = routed * each + a.Is / 2;
    const int routed_pairs = a.T * a.k;
    float *hs = a.h + (int64_t)routed_pairs * a.I;                  // the shared expert's rows

    // gate and up: two features a piece
    for (;;) {
        int piece = 0;
        if (lane == 0) piece = atomicAdd(a.count, 1);
        piece = __shfl_sync(0xffffffffu, piece, 0);
        if (piece >= pieces) break;
        const bool shared = piece >= routed * each;
        const int c = shared ? routed : piece / each;
        const int f = 2 * (shared ? piece - routed * each : piece - c * each);
        const int I = shared ? a.Is : a.I;
        const int64_t at = ((shared ? 0 : (int64_t)r.expert[c] * I) + f) * a.H;
        const T *g = static_cast<const T *>(shared ? a.sgate : a.gate) + at, *u = static_cast<const T *>(shared ? a.sup : a.up) + at;
        const T *const row[kRows] = {g, g + a.H, u, u + a.H};
        const int end = r.start[c + 1];
        for (int p = r.start[c]; p < end; p += 8) {
            const int m = end - p;
            float *h = shared ? hs + (int64_t)(p - routed_pairs) * I : a.h + (int64_t)p * I;
            if (m == 1) gate_up<DT, 1>(a, r, row, p, end, f, I, h);
            else if (m == 2) gate_up<DT, 2>(a, r, row, p, end, f, I, h);
            else if (m <= 4) gate_up<DT, 4>(a, r, row, p, end, f, I, h);
            else gate_up<DT, 8>(a, r, row, p, end, f, I, h);
        }
        __syncwarp();
        if (lane == 0) {
            __threadfence();
            atomicAdd(a.count + 1, 1);
        }
    }
    if (threadIdx.x == 0) {
        const uint64_t t0 = now_ns();
        int done;
        do {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(done) : "l"(a.count + 1) : "memory");
        } while (done < pieces && now_ns() - t0 < kWaitNs);
        ready = done >= pieces;
    }
    // this block's rows of down
    const int row0 = (int)((int64_t)blockIdx.x * a.H / gridDim.x), row1 = (int)((int64_t)(blockIdx.x + 1) * a.H / gridDim.x);
    const int groups = (row1 - row0 + kRows - 1) / kRows;
    float *sums = reinterpret_cast<float *>(rest) + warp * groups * kRows * kMaxTokens;
    for (int i = lane; i < groups * kRows * kMaxTokens; i += 32) sums[i] = 0.0f;
    __syncthreads();
    const bool good = ready;
    if (good) {
        for (int u = warp; u < groups * n; u += kWarps) {
            const int group = u / n, c = u - group * n;
            const bool shared = c == routed;
            const int I = shared ? a.Is : a.I;
            const T *d = static_cast<const T *>(shared ? a.sdown : a.down) + (shared ? 0 : (int64_t)r.expert[c] * a.H * I);
            const T *row[kRows];
#pragma unroll
            for (int i = 0; i < kRows; ++i) row[i] = d + (int64_t)min(row0 + group * kRows + i, row1 - 1) * I;
            const int end = r.start[c + 1];
            float *to = sums + group * kRows * kMaxTokens;
            for (int p = r.start[c]; p < end; p += 8) {
                const int m = end - p;
                const float *h = shared ? hs + (int64_t)(p - routed_pairs) * I : a.h + (int64_t)p * I;
                if (m == 1) down<DT, 1>(r, row, h, p, end, I, to);
                else if (m == 2) down<DT, 2>(r, row, h, p, end, I, to);
                else if (m <= 4) down<DT, 4>(r, row, h, p, end, I, to);
                else down<DT, 8>(r, row, h, p, end, I, to);
            }
        }
    }
    __syncthreads();
    const float *all = reinterpret_cast<const float *>(rest);
    const int rows = row1 - row0;
    for (int i = threadIdx.x; i < rows * a.T; i += kThreads) {
        const int t = i / rows, row = i - t * rows;
        float s = good ? 0.0f : __uint_as_float(0x7FC00000u);       // a wait that ran out
#pragma unroll 4
        for (int w = 0; w < kWarps; ++w) s += all[(w * groups * kRows + row) * kMaxTokens + t];
        const int64_t at = (int64_t)t * a.H + row0 + row;
        if (a.base) s += load_f32<DT>(a.base, at);
        store_f32<DT>(a.out, at, s);
    }
}

// ------------------------------------------------------------ host side

constexpr size_t kCountBytes = 128;

size_t logits_bytes(int T, int E) { return (sizeof(float) * (size_t)T * E + 15) / 16 * 16; }

template <int DT, int RT> cudaError_t launch_logits(const LayerArgs &a, cudaStream_t st) {
    cudaError_t e = allow_smem<k_layer_logits<DT, RT>>();
    if (e != cudaSuccess) return e;
    const size_t w = sizeof(typename RouterWord<RT>::T) * a.H, x = sizeof(typename RowType<DT>::T) * a.H;
    const int tokens = (int)std::min<size_t>(a.T, std::max<size_t>(1, (128 * 1024 - w) / x));
    return launch_pdl(k_layer_logits<DT, RT>, dim3(a.E), dim3(kLogitThreads), w + tokens * x, st, a, tokens);
}

template <int DT> cudaError_t launch_layer(const LayerArgs &a, int router_dtype, cudaStream_t st) {
    cudaError_t e = router_dtype == MOE_ROUTER_F32 ? launch_logits<DT, MOE_ROUTER_F32>(a, st) : launch_logits<DT, MOE_ROUTER_BF16>(a, st);
    if (e == cudaSuccess) e = allow_smem<k_layer<DT>>();
    if (e != cudaSuccess) return e;
    const size_t choice = sizeof(float) * ((size_t)kWarps * a.E + 2 * kMaxPairs);
    const int most = (a.H + kSms - 1) / kSms, groups = (most + kRows - 1) / kRows;
    const size_t sums = sizeof(float) * (size_t)kWarps * groups * kRows * kMaxTokens;
    return launch_pdl(k_layer<DT>, dim3(kSms), dim3(kThreads), (routing_bytes(a.E) + 15) / 16 * 16 + std::max(choice, sums), st, a);
}

bool good_width(int32_t v) { return v >= kChunk && v <= kMaxWidth && v % kChunk == 0; }

}  // namespace

extern "C" {

size_t moe_decode_layer_workspace(int32_t T, int32_t num_experts, int32_t inter, int32_t top_k, int32_t shared_inter) {
    if (T < 1 || T > kMaxTokens || num_experts < 1 || num_experts > kMaxExperts || inter < 1 || inter > kMaxWidth || top_k < 1 ||
        top_k > kMaxTopK || shared_inter < 0 || shared_inter > kMaxWidth)
        return 0;
    return kCountBytes + logits_bytes(T, num_experts) + sizeof(float) * ((size_t)T * top_k * inter + (size_t)T * shared_inter);
}

moe_status moe_decode_layer(const void *x, int32_t dtype, int32_t T, int32_t hidden, const void *router_w,
                            int32_t router_dtype, const float *router_bias, int32_t num_experts, int32_t top_k,
                            int32_t router, int32_t renormalize, const void *gate, const void *up, const void *down,
                            int32_t inter, const void *shared_gate, const void *shared_up, const void *shared_down,
                            int32_t shared_inter, const void *base, void *out, int32_t *topk_ids, float *topk_w,
                            void *workspace, size_t workspace_bytes, void *stream) {
    if (T < 0 || !known_dtype(dtype) || (router_dtype != MOE_ROUTER_F32 && router_dtype != MOE_ROUTER_BF16) ||
        (router != MOE_ROUTER_SOFTMAX && router != MOE_ROUTER_SIGMOID) || (renormalize & ~1))
        return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || !good_width(hidden) || !good_width(inter) || num_experts < 1 || num_experts > kMaxExperts || top_k < 1 ||
        top_k > kMaxTopK || top_k > num_experts || (shared_inter != 0 && !good_width(shared_inter)))
        return MOE_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return MOE_OK;
    if (!x || !router_w || !gate || !up || !down || !out || !topk_ids || !topk_w) return MOE_ERR_INVALID_ARG;
    if (shared_inter ? !shared_gate || !shared_up || !shared_down : shared_gate || shared_up || shared_down) return MOE_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < moe_decode_layer_workspace(T, num_experts, inter, top_k, shared_inter)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {x, router_w, gate, up, down, shared_gate, shared_up, shared_down, static_cast<const void *>(workspace)})
        if (!aligned_to(p, 16)) return MOE_ERR_MISALIGNED;
    const uintptr_t es = dtype == MOE_DTYPE_F32 ? 4 : 2;
    if (!aligned_to(base, es) || !aligned_to(out, es) || !aligned_to(router_bias, 4) || !aligned_to(topk_ids, 4) || !aligned_to(topk_w, 4))
        return MOE_ERR_MISALIGNED;
    LayerArgs a{};
    a.x = x;
    a.router = router_w;
    a.bias = router_bias;
    a.gate = gate;
    a.up = up;
    a.down = down;
    a.sgate = shared_gate;
    a.sup = shared_up;
    a.sdown = shared_down;
    a.base = base;
    a.out = out;
    a.ids = topk_ids;
    a.wts = topk_w;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.count = reinterpret_cast<int *>(ws);
    a.logits = reinterpret_cast<float *>(ws + kCountBytes);
    a.h = reinterpret_cast<float *>(ws + kCountBytes + logits_bytes(T, num_experts));
    a.T = T;
    a.H = hidden;
    a.E = num_experts;
    a.I = inter;
    a.k = top_k;
    a.Is = shared_inter;
    a.kind = router;
    a.renorm = renormalize;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case MOE_DTYPE_F32: e = launch_layer<MOE_DTYPE_F32>(a, router_dtype, s); break;
        case MOE_DTYPE_BF16: e = launch_layer<MOE_DTYPE_BF16>(a, router_dtype, s); break;
        default: e = launch_layer<MOE_DTYPE_F16>(a, router_dtype, s); break;
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
