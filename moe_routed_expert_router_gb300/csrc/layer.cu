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
// The weights stream through a ring of 2 KB stages in shared memory that every warp
// keeps for itself (four rows, 16 bytes a lane and row; a lane reads back only what
// it copied, so nothing is waited for but the copies).  The ring runs from piece to
// piece and on into the rows of down, which are on their way while the block waits
// for the last of h.
//
// Every block chooses the experts itself (a microsecond, against a launch and its
// gap).  Gate and up rows are handed out by a ticket counter, two features a piece,
// so the last piece is short and no block has to be resident for another's sake: a
// wait for the pieces is a wait for blocks that already run.  The rows of down are
// split evenly beforehand; a block's warps share the experts and slices of their
// widths and add over them in a fixed order, so nothing is added through memory and
// equal inputs give equal bits.
//
// Measured: 4 tokens, 128 experts of 4096 x 1536 and a shared one 186 us (6.1 TB/s, 92
// % of the copy bandwidth): logits 4 us, choice 3.6, gate and up 120 (6.1 TB/s, the
// last piece's wait 6 of them), down 55 (6.9 TB/s).  16 tokens of 2048 x 1024 f16 115
// us (83 %).  A fence behind every piece instead of one a warp: 213; chunks of eight
// features that all warps share, a barrier each: 232; stages of 4 KB: 224 against 222
// then; one feature a piece: 193.  Small layers are latency: logits, choice, two
// phases and the wait between them, 10 us.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace {

using namespace moe;

constexpr int kMaxTokens = 16, kMaxPairs = kMaxTokens * kMaxTopK;
constexpr int kMaxWidth = 16384;
constexpr int kWarps = 16, kThreads = 32 * kWarps;
constexpr int kRows = 4;                   // weight rows a stage: two features' gate and up, or four rows of down
constexpr int kStage = kRows * 512;        // its bytes: 16 a lane and row
constexpr int kMaxRing = 8;
constexpr int kQueue = 16;                 // pieces between a warp's copies and its products, more than kMaxRing
constexpr int kMostRows = 32;              // rows of down a block sums at once
constexpr int kMostPairs = 4;              // tokens that share a pass over an expert's weights: what registers hold sums for
constexpr int kLeastRing = 2, kLeastRows = 8;                     // what the tokens in shared memory have to leave room for

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
    int ring, pass_rows;                   // stages of a warp's ring; rows of down a block sums at once
};

// ------------------------------------------------------------ logits

constexpr int kLogitThreads = 512;

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
    int *expert, *start;                   // runs of up to kMostPairs pairs of one expert, experts increasing (E: the shared one):
                                           // the expert and the first pair
    int *token;                            // [pairs] token of a pair
    float *weight;                         // [pairs]
    int *runs;                             // [0] of chosen experts, [1] with the shared one's
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
    r.runs = r.token + 2 * P;
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
            const int own = (c + kMostPairs - 1) / kMostPairs << 16 | c;     // runs and pairs in one sum
            int sum = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += y;
            }
            if (c > 0) {
                const int before = sum - own, i = n + (before >> 16), p = pairs + (before & 0xFFFF);
                r.first[e] = p;
                for (int q = 0; q * kMostPairs < c; ++q) {
                    r.expert[i + q] = e;
                    r.start[i + q] = p + q * kMostPairs;
                }
            }
            sum = __shfl_sync(0xffffffffu, sum, 31);
            n += sum >> 16;
            pairs += sum & 0xFFFF;
        }
        if (lane == 0) r.runs[0] = n;
        if (a.Is > 0) {
            const int more = (a.T + kMostPairs - 1) / kMostPairs;
            if (lane < more) {
                r.expert[n + lane] = a.E;
                r.start[n + lane] = pairs + lane * kMostPairs;
            }
            if (lane < a.T) {
                r.token[pairs + lane] = lane;
                r.weight[pairs + lane] = 1.0f;
            }
            n += more;
            pairs += a.T;
        }
        if (lane == 0) {
            r.start[n] = pairs;
            r.runs[1] = n;
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

template <int N> constexpr int kLog = N <= 1 ? 0 : 1 + kLog<N / 2>;
template <> constexpr int kLog<1> = 0;

// Sums of v[0 .. N) over the warp: lane l returns that of v[l >> (5 - log2 N)].
template <int N> __device__ __forceinline__ float spread_sum(float (&v)[N], int lane) {
    int o = 16;
#pragma unroll
    for (int n = N / 2; n >= 1; n >>= 1, o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
    }
#pragma unroll
    for (int s = 16 >> kLog<N>; s >= 1; s >>= 1) v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
    return v[0];
}

template <int DT> __device__ __forceinline__ float load_f32(const void *p, int64_t i) { return as_f32(static_cast<const typename RowType<DT>::T *>(p)[i]); }
template <int DT> __device__ __forceinline__ void store_f32(void *p, int64_t i, float v) {
    if constexpr (DT == MOE_DTYPE_F32) static_cast<float *>(p)[i] = v;
    else if constexpr (DT == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else static_cast<__half *>(p)[i] = __float2half_rn(v);
}

// The expert of a run.
template <typename T> struct Expert {
    const T *gate, *up, *down;
    int I;
};
template <typename T> __device__ __forceinline__ Expert<T> expert_of(const LayerArgs &a, const Routing &r, int run) {
    const int e = r.expert[run];
    const bool shared = e == a.E;
    const int64_t at = shared ? 0 : (int64_t)e * a.I * a.H;
    return {static_cast<const T *>(shared ? a.sgate : a.gate) + at, static_cast<const T *>(shared ? a.sup : a.up) + at,
            static_cast<const T *>(shared ? a.sdown : a.down) + at, shared ? a.Is : a.I};
}

// h's row of pair p.
__device__ __forceinline__ float *h_row(const LayerArgs &a, int p) {
    const int routed = a.T * a.k;
    return p < routed ? a.h + (int64_t)p * a.I : a.h + (int64_t)routed * a.I + (int64_t)(p - routed) * a.Is;
}

// acc[i][j] += this lane's piece of the stage's row i times y_j, in fp32.
template <int DT, int M>
__device__ __forceinline__ void stage_dots(const uint8_t *stage, const float (&y)[M][kPieceValues<DT>], float (&acc)[kRows][M][2]) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float w[kPieceValues<DT>];
        widen_piece<DT>(*reinterpret_cast<const uint4 *>(stage + 512 * i), w);
#pragma unroll
        for (int j = 0; j < M; ++j)
#pragma unroll
            for (int q = 0; q < kPieceValues<DT>; q += 2) fma2(acc[i][j][0], acc[i][j][1], w[q], w[q + 1], y[j][q], y[j][q + 1]);
    }
}

// Calls f with the least of 1, 2, 4 that is at least n, as a constant.
template <typename F> __device__ __forceinline__ void by_pairs(int n, F f) {
    if (n == 1) f(std::integral_constant<int, 1>{});
    else if (n == 2) f(std::integral_constant<int, 2>{});
    else f(std::integral_constant<int, 4>{});
}

template <int DT, bool kXShared>
__global__ void __launch_bounds__(kThreads, 1) k_layer(LayerArgs a) {
    using T = typename RowType<DT>::T;
    constexpr int V = kPieceValues<DT>, kStep = 32 * V;             // values of a stage's row: a lane's, all
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int ready;
    __shared__ int queue[kWarps][kQueue];
    const Routing r = routing_at(smem, a.E);
    T *xs = reinterpret_cast<T *>(smem + (routing_bytes(a.E) + 15) / 16 * 16);
    uint8_t *rest = reinterpret_cast<uint8_t *>(xs) + (kXShared ? sizeof(T) * a.T * a.H : 0);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *sums = reinterpret_cast<float *>(rest) + warp * a.pass_rows * a.T;     // [rows of a pass][T], this warp's
    uint8_t *ring = rest + sizeof(float) * kWarps * a.pass_rows * a.T + warp * a.ring * kStage;
    pdl_wait();
    pdl_trigger();
    if constexpr (kXShared) {
        for (int i = threadIdx.x; i < a.T * a.H / V; i += kThreads) copy16(xs + V * i, static_cast<const T *>(a.x) + V * i, true);
        copy_commit();
    }
    route(a, r, rest);
    if constexpr (kXShared) {
        copy_wait<0>();
        __syncthreads();
    }
    const int routed = r.runs[0], runs = r.runs[1];
    // pieces of two features, units of kStep values of an expert's width; the shared expert's lie behind the others
    const int each = a.I / 2, shared_each = a.Is / 2, pieces = routed * each + (runs - routed) * shared_each;
    const int slices = (a.I + kStep - 1) / kStep, shared_slices = (a.Is + kStep - 1) / kStep;
    const int units = routed * slices + (runs - routed) * shared_slices;
    auto split = [&](int i, int of, int of_shared, int &run, int &part) {
        const bool shared = i >= routed * of;
        const int k = shared ? i - routed * of : i, n = shared ? of_shared : of;
        run = k / n;
        part = k - run * n;
        if (shared) run += routed;
    };
    const int row0 = (int)((int64_t)blockIdx.x * a.H / gridDim.x), row1 = (int)((int64_t)(blockIdx.x + 1) * a.H / gridDim.x);

    // The warp's copies: pieces of gate and up as its tickets give them, kStep values a stage; then its units of down,
    // pass after pass, kRows rows a stage.
    int ticket = 0;                        // of lane 0: the next piece
    if (lane == 0) ticket = atomicAdd(a.count, 1);
    int head = 0, fill = 0, steps = 0;     // pieces queued; the next stage; stages left of the piece or unit
    bool downs = false;
    int unit = warp, base = row0, rows_left = 0, values = 0;        // values of a row from this lane's on
    const T *p0 = nullptr, *p1 = nullptr;
    int64_t row_step = a.H;
    auto next_piece = [&]() {
        const int piece = __shfl_sync(0xffffffffu, ticket, 0);
        if (lane == 0) queue[warp][head % kQueue] = piece;
        ++head;
        if (piece >= pieces) {
            downs = true;
            return;
        }
        if (lane == 0) ticket = atomicAdd(a.count, 1);
        int run, part;
        split(piece, each, shared_each, run, part);
        const Expert<T> x = expert_of<T>(a, r, run);
        p0 = x.gate + (int64_t)(2 * part) * a.H + V * lane;
        p1 = x.up + (int64_t)(2 * part) * a.H + V * lane;
        values = a.H - V * lane;
        steps = (a.H + kStep - 1) / kStep;
    };
    auto next_unit = [&]() {
        while (unit >= units && base < row1) {
            unit = warp;
            base += a.pass_rows;
        }
        if (base >= row1) return;
        int run, part;
        split(unit, slices, shared_slices, run, part);
        const Expert<T> x = expert_of<T>(a, r, run);
        p0 = x.down + (int64_t)base * x.I + part * kStep + V * lane;
        values = x.I - part * kStep - V * lane;
        row_step = x.I;
        rows_left = min(a.pass_rows, row1 - base);
        steps = (rows_left + kRows - 1) / kRows;
        unit += kWarps;
    };
    auto copy_next = [&]() {
        if (steps == 0 && !downs) next_piece();
        if (steps == 0 && downs) next_unit();
        if (steps > 0) {
            uint8_t *to = ring + fill * kStage + 16 * lane;
            if (!downs) {
                if (values > 0) {
                    copy16(to, p0, true);
                    copy16(to + 512, p0 + a.H, true);
                    copy16(to + 1024, p1, true);
                    copy16(to + 1536, p1 + a.H, true);
                }
                p0 += kStep;
                p1 += kStep;
                values -= kStep;
            } else {
                if (values > 0) {
#pragma unroll
                    for (int i = 0; i < kRows; ++i)
                        if (i < rows_left) copy16(to + 512 * i, p0 + i * row_step, true);
                }
                p0 += kRows * row_step;
                rows_left -= kRows;
            }
            --steps;
        }
        copy_commit();
        if (++fill == a.ring) fill = 0;
    };
    int slot = 0;
    auto next_stage = [&]() {              // the oldest stage: all but the ring - 1 latest copies are there
        copy_next();
        switch (a.ring) {
            case 2: copy_wait<1>(); break;
            case 3: copy_wait<2>(); break;
            case 4: copy_wait<3>(); break;
            case 5: copy_wait<4>(); break;
            case 6: copy_wait<5>(); break;
            case 7: copy_wait<6>(); break;
            default: copy_wait<kMaxRing - 1>(); break;
        }
        const uint8_t *stage = ring + slot * kStage + 16 * lane;
        if (++slot == a.ring) slot = 0;
        return stage;
    };
    for (int i = 0; i < a.ring - 1; ++i) copy_next();

    // gate and up: h of a piece's two features for the pairs of its run
    int finished = 0;
    for (int tail = 0;; ++tail) {
        __syncwarp();
        const int piece = queue[warp][tail % kQueue];               // queued: the copies are a stage ahead at least
        if (piece >= pieces) break;
        int run, part;
        split(piece, each, shared_each, run, part);
        const int p = r.start[run], end = r.start[run + 1];
        by_pairs(end - p, [&](auto width) {
            constexpr int M = decltype(width)::value;
            const T *from[M];
#pragma unroll
            for (int j = 0; j < M; ++j)
                from[j] = (kXShared ? xs : static_cast<const T *>(a.x)) + r.token[min(p + j, end - 1)] * (int64_t)a.H + V * lane;
            float acc[kRows][M][2] = {};
            for (int k = 0; k < a.H; k += kStep) {
                const uint8_t *stage = next_stage();
                if (k + V * lane >= a.H) continue;
                float y[M][V];
#pragma unroll
                for (int j = 0; j < M; ++j) {
                    uint4 q;
                    if constexpr (kXShared) q = *reinterpret_cast<const uint4 *>(from[j] + k);
                    else q = ld16_shared(from[j] + k);
                    widen_piece<DT>(q, y[j]);
                }
                stage_dots<DT, M>(stage, y, acc);
            }
            float v[kRows * M];                                     // of a token: gate f, gate f + 1, up f, up f + 1
#pragma unroll
            for (int j = 0; j < M; ++j)
#pragma unroll
                for (int i = 0; i < kRows; ++i) v[j * kRows + i] = acc[i][j][0] + acc[i][j][1];
            constexpr int shift = 5 - kLog<kRows * M>;
            const float own = spread_sum<kRows * M>(v, lane), up = __shfl_down_sync(0xffffffffu, own, 2 << shift);
            const int j = lane >> shift >> 2, i = lane >> shift & 3;
            if ((lane & ((1 << shift) - 1)) == 0 && i < 2 && p + j < end)
                h_row(a, p + j)[2 * part + i] = own / (1.0f + expf(-own)) * up * r.weight[p + j];
        });
        ++finished;
    }
    // one release a warp: a fence behind every piece cost the stream a twentieth
    __syncwarp();
    if (lane == 0 && finished > 0) {
        __threadfence();
        atomicAdd(a.count + 1, finished);
    }
    if (threadIdx.x == 0) {
        const uint64_t t0 = now_ns();
        int done;
        do {
            asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(done) : "l"(a.count + 1) : "memory");
        } while (done < pieces && now_ns() - t0 < kWaitNs);
        ready = done >= pieces;
    }
    __syncthreads();
    const bool good = ready;
    if (!good) copy_wait<0>();

    // this block's rows of down
    for (int first = row0; first < row1; first += a.pass_rows) {
        const int rows = min(a.pass_rows, row1 - first);
        for (int i = lane; i < a.pass_rows * a.T; i += 32) sums[i] = 0.0f;
        __syncwarp();
        for (int u = warp; good && u < units; u += kWarps) {
            int run, part;
            split(u, slices, shared_slices, run, part);
            const int I = r.expert[run] == a.E ? a.Is : a.I;
            const int p = r.start[run], end = r.start[run + 1], k = part * kStep + V * lane;
            by_pairs(end - p, [&](auto width) {
                constexpr int M = decltype(width)::value;
                float y[M][V] = {};
                if (k < I) {
#pragma unroll
                    for (int j = 0; j < M; ++j) {
                        const float *from = h_row(a, min(p + j, end - 1)) + k;
#pragma unroll
                        for (int q = 0; q < V; q += 4) {
                            const uint4 v = ld16_shared(from + q);
                            y[j][q] = __uint_as_float(v.x);
                            y[j][q + 1] = __uint_as_float(v.y);
                            y[j][q + 2] = __uint_as_float(v.z);
                            y[j][q + 3] = __uint_as_float(v.w);
                        }
                    }
                }
                constexpr int shift = 5 - kLog<kRows * M>;
                const int j = lane >> shift >> 2, i = lane >> shift & 3;
                const bool writes = (lane & ((1 << shift) - 1)) == 0 && p + j < end;
                float *to = sums + i * a.T + (writes ? r.token[p + j] : 0);
                for (int row = 0; row < rows; row += kRows) {
                    const uint8_t *stage = next_stage();
                    float acc[kRows][M][2] = {};
                    if (k < I) stage_dots<DT, M>(stage, y, acc);
                    float v[kRows * M];
#pragma unroll
                    for (int b = 0; b < M; ++b)
#pragma unroll
                        for (int c = 0; c < kRows; ++c) v[b * kRows + c] = acc[c][b][0] + acc[c][b][1];
                    const float own = spread_sum<kRows * M>(v, lane);
                    if (writes) to[row * a.T] += own;
                }
            });
            __syncwarp();
        }
        __syncthreads();
        const float *all = reinterpret_cast<const float *>(rest);
        for (int i = threadIdx.x; i < rows * a.T; i += kThreads) {
            const int t = i / rows, row = i - t * rows;
            float s = good ? 0.0f : __uint_as_float(0x7FC00000u);   // a wait that ran out
#pragma unroll 4
            for (int w = 0; w < kWarps; ++w) s += all[(w * a.pass_rows + row) * a.T + t];
            const int64_t at = (int64_t)t * a.H + first + row;
            if (a.base) s += load_f32<DT>(a.base, at);
            store_f32<DT>(a.out, at, s);
        }
        __syncthreads();
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

// Shared memory of k_layer: the routing and the tokens, then the choice's scratch and, over it, sums and rings.
struct LayerShape { size_t front, choice; int pass_rows, ring; };

size_t sums_bytes(int T, int pass_rows) { return sizeof(float) * kWarps * pass_rows * T; }

LayerShape layer_shape(const LayerArgs &a, size_t x) {
    LayerShape s;
    s.front = (routing_bytes(a.E) + 15) / 16 * 16 + x;
    s.choice = sizeof(float) * ((size_t)kWarps * a.E + 2 * kMaxPairs);
    s.pass_rows = std::min(kMostRows, (blocks_of(a.H, kSms) + kRows - 1) / kRows * kRows);
    auto rings = [&]() { return ((int64_t)kSmemBlock - (int64_t)(s.front + sums_bytes(a.T, s.pass_rows))) / (kWarps * kStage); };
    while (rings() < kLeastRing && s.pass_rows > kLeastRows) s.pass_rows -= kRows;
    s.ring = (int)std::min<int64_t>(kMaxRing, rings());
    return s;
}

template <int DT, bool kXShared> cudaError_t launch_weights(LayerArgs a, const LayerShape &s, cudaStream_t st) {
    const cudaError_t e = allow_smem<k_layer<DT, kXShared>>();
    if (e != cudaSuccess) return e;
    a.pass_rows = s.pass_rows;
    a.ring = s.ring;
    return launch_pdl(k_layer<DT, kXShared>, dim3(kSms), dim3(kThreads),
                      s.front + std::max(s.choice, sums_bytes(a.T, s.pass_rows) + s.ring * kWarps * kStage), st, a);
}

// The tokens stay in shared memory where that leaves two stages a warp (16 tokens of 4096 bf16 values, 64 experts of 1536:
// 380 us, through the caches 416; 16 of 2048 115 against 138).
template <int DT> cudaError_t launch_layer(const LayerArgs &a, int router_dtype, cudaStream_t st) {
    const cudaError_t e = router_dtype == MOE_ROUTER_F32 ? launch_logits<DT, MOE_ROUTER_F32>(a, st) : launch_logits<DT, MOE_ROUTER_BF16>(a, st);
    if (e != cudaSuccess) return e;
    const LayerShape s = layer_shape(a, sizeof(typename RowType<DT>::T) * a.T * a.H);
    if (s.ring >= kLeastRing && s.front + s.choice <= kSmemBlock) return launch_weights<DT, true>(a, s, st);
    return launch_weights<DT, false>(a, layer_shape(a, 0), st);
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
