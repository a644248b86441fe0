// The (token, slot) pairs' way to the experts and back, for callers whose
// products are their own: stable sort by expert, rows to expert order, weighted
// rows back to token order, and the gradients (see include/moe_nvfp4.h).
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "rows.cuh"

namespace cg = cooperative_groups;

namespace {

using namespace moe;

constexpr int64_t kMaxRows = 0x7fffffff;   // rows, pairs and blocks of a launch
constexpr int kMaxCombineH = 65536;

// ------------------------------------------------------------------- sort

constexpr int kMaxAlign = 256;
constexpr int kSortMaxWarps = 32;
constexpr int kSortIds = 8;           // ids a lane has in flight
// Pairs a block of the cluster takes before there is another, up to 16 blocks
// (1024 tokens, k = 8: 4.4 us; with 1024 pairs a block 5.3 us, with 2048 6.0).
constexpr int kSortPairs = 512, kSortBlocks = 16;

// Inclusive scan over the block's threads; `red` holds 32 words.
__device__ __forceinline__ int block_scan(int v, int *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int w = lane < warps ? red[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        red[lane] = w;
    }
    __syncthreads();
    return warp ? v + red[warp - 1] : v;
}

// Shared memory of k_sort_pairs, in words: [warps][E] a warp's counts, then the
// index of its next pair in the block's run of an expert; [E] the block's
// counts; [E] an expert's first row for this block.
struct SortArgs {
    const int32_t *ids;
    int P, E, align, warps, run;   // `warps` of a block own `run` consecutive pairs each
    int64_t R;
    int32_t *offsets, *rows, *inv;
};

// Counting sort in one launch of one cluster (or one block).  Every warp owns a
// run of consecutive pairs and counts them per expert in shared memory; the
// blocks read each other's counts through distributed shared memory and scan
// them into the segments' first rows; the pairs are then placed in order, the
// ones of a warp that share an expert ranked by ballots of the expert's bits (by
// a match of the warp's ids 131072 pairs took 12.5 us, so 10.7).  All rows are
// set to -1 while the ids arrive; the barrier in between orders that before the
// placing.  Latency-bound: one read of the ids, one cluster barrier, one write
// (4 tokens, k = 8, E = 128: 2.3 us in a graph; 16384 tokens, E = 256: 10.6 us
// with 16 blocks, half of it the ranking, some 110 instructions for 32 pairs on
// 16 SMs; the scattered stores are 0.5 us, and placing through a sorted copy in
// shared memory, for neighbouring ones, measured no gain).  A cluster of 16 is more
// than every device has to hold; a whole GB300 does.
template <bool kCluster>
__global__ void __launch_bounds__(1024) k_sort_pairs(const SortArgs a) {
    extern __shared__ int smem[];
    const int E = a.E, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int *wc = smem, *tot = wc + a.warps * E, *first = tot + E;
    __shared__ int red[32];
    int nb = 1, rank = 0;
    if constexpr (kCluster) {
        nb = (int)cg::this_cluster().num_blocks();
        rank = (int)cg::this_cluster().block_rank();
    }
    for (int i = tid; i < a.warps * E; i += blockDim.x) wc[i] = 0;
    pdl_wait();
    pdl_trigger();
    const bool owns = warp < a.warps;
    const int64_t beg = owns ? min((int64_t)a.P, ((int64_t)rank * a.warps + warp) * a.run) : a.P;
    const int64_t end = min((int64_t)a.P, beg + a.run);
    int *mine = wc + warp * E;
    int id[kSortIds];
    auto load = [&](int64_t p0) {
#pragma unroll
        for (int i = 0; i < kSortIds; ++i) {
            const int64_t p = p0 + 32 * i + lane;
            id[i] = p < end ? a.ids[p] : -1;
            if (id[i] < 0 || id[i] >= E) id[i] = -1;
        }
    };
    load(beg);
    for (int64_t r = rank * (int64_t)blockDim.x + tid; r < a.R; r += nb * (int64_t)blockDim.x) a.rows[r] = -1;
    __syncthreads();
    for (int64_t p0 = beg; p0 < end; p0 += 32 * kSortIds) {
        if (p0 != beg) load(p0);
#pragma unroll
        for (int i = 0; i < kSortIds; ++i)
            if (id[i] >= 0) atomicAdd(mine + id[i], 1);
    }
    __syncthreads();
    int count = 0, before = 0;   // thread e: expert e's pairs in all blocks, and in those before this one
    if (tid < E) {
        for (int w = 0; w < a.warps; ++w) {
            const int c = wc[w * E + tid];
            wc[w * E + tid] = count;
            count += c;
        }
        if constexpr (kCluster) tot[tid] = count;
    }
    if constexpr (kCluster) {
        cg::this_cluster().sync();
        if (tid < E) {
            int c[kSortBlocks];
#pragma unroll
            for (int b = 0; b < kSortBlocks; ++b)
                c[b] = b < nb ? cg::this_cluster().map_shared_rank(tot, b)[tid] : 0;
            count = 0;
#pragma unroll
            for (int b = 0; b < kSortBlocks; ++b) {
                count += c[b];
                if (b < rank) before += c[b];
            }
        }
        cg::this_cluster().barrier_arrive();           // this block has read the others' counts
    }
    const int padded = (int)(((int64_t)count + a.align - 1) / a.align * a.align);
    const int segment = block_scan(padded, red);
    if (tid < E) {
        first[tid] = segment - padded + before;
        if (rank == 0) {
            a.offsets[tid] = segment - padded;
            if (tid == E - 1) a.offsets[E] = segment;
        }
    }
    __syncthreads();
    const int bits = 33 - __clz((E - 1) | 1);   // of an expert, and one that -1 has and no expert
    for (int64_t p0 = beg; p0 < end; p0 += 32 * kSortIds) {
        if (end - beg > 32 * kSortIds) load(p0);
#pragma unroll
        for (int i = 0; i < kSortIds; ++i) {
            const int64_t p = p0 + 32 * i + lane;
            if (p0 + 32 * i >= end) break;
            const int e = id[i];
            // the lanes with the same expert, bit by bit
            unsigned peers = 0xffffffffu;
            for (int b = 0; b < bits; ++b) {
                const bool on = e >> b & 1;
                const unsigned with = __ballot_sync(0xffffffffu, on);
                peers &= on ? with : ~with;
            }
            int row = -1;
            if (e >= 0) row = first[e] + mine[e] + __popc(peers & ((1u << lane) - 1u));
            __syncwarp();
            if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
            __syncwarp();
            if (p >= end) continue;
            if (row >= 0 && row < a.R) a.rows[row] = (int)p;   // ids that changed meanwhile write nothing out of range
            a.inv[p] = row;
        }
    }
    if constexpr (kCluster) cg::this_cluster().barrier_wait();   // the others have read this block's counts
}

size_t sort_smem(int warps, int E) { return sizeof(int) * ((size_t)warps + 2) * E; }

// The kernels' attributes, once a device: shared memory, and the cluster size.
cudaError_t configure_sort() {
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    for (auto kernel : {k_sort_pairs<false>, k_sort_pairs<true>}) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)sort_smem(kSortMaxWarps, kMaxExperts));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return e;
    }
    done[dev] = true;
    return cudaSuccess;
}

// --------------------------------------------------------------- dispatch

// Rows that a warp looks at for ones without a pair: a row of 512 pieces, up to
// 32 shorter ones (16384 x 256, bf16, no padding: 12.6 us for the dispatch,
// with one row a warp 25.8 us).
int zero_rows_a_warp(int pieces) { return std::max(1, std::min(32, 512 / pieces)); }

// Zeros for those of the `zero_rows` rows from r0 on that hold no pair, n words
// of each at `out`: a row at a time, or, where a row is shorter than a warp is
// wide, the lanes spread over all of them.
__device__ __forceinline__ void put_zero(uint4 *p) { st16(p, make_uint4(0, 0, 0, 0)); }
__device__ __forceinline__ void put_zero(uint32_t *p) { *p = 0; }
__device__ __forceinline__ void put_zero(uint8_t *p) { *p = 0; }

template <typename W>
__device__ __forceinline__ void zero_words(W *out, int n, int64_t r0, int zero_rows, unsigned none, int lane) {
    if (n >= 32) {
        for (unsigned m = none; m; m &= m - 1) {
            W *row = out + (r0 + __ffs(m) - 1) * n;
            for (int c = lane; c < n; c += 32) put_zero(row + c);
        }
    } else {
        for (int i = lane; i < zero_rows * n; i += 32)
            if (none >> (i / n) & 1) put_zero(out + r0 * n + i);
    }
}

__device__ __forceinline__ unsigned rows_without_pair(const int32_t *rows, int64_t r0, int zero_rows, int64_t R,
                                                      int64_t P, int lane) {
    bool none = false;
    if (lane < zero_rows && r0 + lane < R) {
        const int p = rows[r0 + lane];
        none = p < 0 || p >= P;
    }
    return __ballot_sync(0xffffffffu, none);
}

// Bound by the HBM writes, so nothing is read twice: a thread holds two 16-byte
// pieces of a token's row and stores them to each of the token's rows (4096 x
// 7168, 8 of 256 experts: 73 us in 8 bits with padding to 128 rows, 102 % of
// the measured copy bandwidth; a warp a row of out, which reads a token's row
// once a pair, 97 us).  A row of threads has a token and a part of its row; the
// blocks past the tokens' write zeros to the rows without a pair.
constexpr int kCopyPieces = 2;

template <typename W>
__global__ void __launch_bounds__(256) k_dispatch(const char *x, int64_t xs, int n, const char *scales, int scale_words,
                                                  int T, int k, const int32_t *rows,
                                                  const int32_t *inv, int64_t R, char *out,
                                                  char *out_scales, int token_blocks, int parts,
                                                  int zero_rows) {
    const int64_t row_bytes = (int64_t)n * 16;
    const int lane = threadIdx.x & 31;
    W *const oscale = reinterpret_cast<W *>(out_scales);
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= token_blocks) {
        const int warp = (threadIdx.y * blockDim.x + threadIdx.x) >> 5, warps = (blockDim.x * blockDim.y) >> 5;
        const int64_t r0 = (((int64_t)blockIdx.x - token_blocks) * warps + warp) * zero_rows;
        const unsigned none = rows_without_pair(rows, r0, zero_rows, R, T * (int64_t)k, lane);
        if (none == 0) return;
        zero_words(reinterpret_cast<uint4 *>(out), n, r0, zero_rows, none, lane);
        zero_words(oscale, scale_words, r0, zero_rows, none, lane);
        return;
    }
    const int part = blockIdx.x % parts;
    const int64_t t = (int64_t)(blockIdx.x / parts) * blockDim.y + threadIdx.y;
    if (t >= T) return;
    // every lane of a warp has the same token: lane j holds pair j's row
    int64_t mine = lane < k ? inv[t * k + lane] : -1;
    if (mine >= R) mine = -1;
    const int c0 = part * blockDim.x * kCopyPieces + threadIdx.x;
    uint4 v[kCopyPieces];
#pragma unroll
    for (int i = 0; i < kCopyPieces; ++i)
        if (c0 + i * (int)blockDim.x < n) v[i] = ld16(x + t * xs + (c0 + i * (int)blockDim.x) * 16);
    for (int j = 0; j < k; ++j) {
        const int64_t r = __shfl_sync(0xffffffffu, mine, j);
        if (r < 0) continue;
#pragma unroll
        for (int i = 0; i < kCopyPieces; ++i)
            if (c0 + i * (int)blockDim.x < n) st16(out + r * row_bytes + (c0 + i * (int)blockDim.x) * 16, v[i]);
    }
    // the scales, spread over the row's blocks
    for (int c = part * blockDim.x + threadIdx.x - lane; c < scale_words; c += parts * blockDim.x) {
        const bool on = c + lane < scale_words;
        const W s = on ? reinterpret_cast<const W *>(scales)[t * scale_words + c + lane] : W{};
        for (int j = 0; j < k; ++j) {
            const int64_t r = __shfl_sync(0xffffffffu, mine, j);
            if (r >= 0 && on) oscale[r * scale_words + c + lane] = s;
        }
    }
}

// ---------------------------------------------------------------- combine

// Bound by HBM: every pair's row read once, every token's written once.  A
// thread has up to eight 16-byte loads in flight: KB pairs' rows of PP pieces
// (KB x PP = 8), so that a token of two pairs asks for as much as one of eight
// (16384 tokens of 4096, k = 2, bf16: 59 us against 99 us with one piece).
// The registers are held to what lets an SM keep its blocks (4096 x 7168, k = 8,
// bf16: 77.1 us at 64 registers, 80.8 us at 66, with a block less; the rows passed
// between lanes by shuffles 87.9 us; over changing inputs 80 us, 98 % of the
// measured copy bandwidth).
// A piece is 16 bytes in every type: with eight fp32 values a thread a warp's
// access had holes (4096 x 4096, k = 10, fp32, backward: 208 us against 238).
constexpr int pair_pieces(int kb) { return kb == 5 ? 2 : 8 / kb; }
constexpr int kCombineThreads = 128;
constexpr int combine_blocks(int kb) { return kb == 2 || kb == 5 ? 6 : 8; }   // two or more pieces' sums take registers

template <int DT, int KB, int PP>
__global__ void __launch_bounds__(kCombineThreads, combine_blocks(KB))
k_combine(const typename RowType<DT>::T *y, int T, int k, int H, const int32_t *inv, int64_t R, const float *w,
          const typename RowType<DT>::T *base, typename RowType<DT>::T *out) {
    constexpr int N = kPieceValues<DT>;
    const int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    pdl_wait();
    pdl_trigger();
    if (t >= T) return;
    const int c0 = (blockIdx.y * PP * blockDim.x + threadIdx.x) * N, dc = blockDim.x * N;
    if (c0 >= H) return;
    float acc[PP][N] = {};
    for (int j0 = 0; j0 < k; j0 += KB) {
        uint4 v[KB][PP];
        int row[KB];
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            row[j] = j0 + j < k ? inv[t * k + j0 + j] : -1;
            if (row[j] >= R) row[j] = -1;
#pragma unroll
            for (int i = 0; i < PP; ++i)
                if (row[j] >= 0 && c0 + i * dc < H) v[j][i] = ld16(y + (int64_t)row[j] * H + c0 + i * dc);
        }
#pragma unroll
        for (int j = 0; j < KB; ++j) {
            if (row[j] < 0) continue;
            const float wj = w ? w[t * k + j0 + j] : 1.0f;
#pragma unroll
            for (int i = 0; i < PP; ++i) {
                if (c0 + i * dc >= H) continue;
                float f[N];
                widen_piece<DT>(v[j][i], f);
#pragma unroll
                for (int e = 0; e < N; e += 2) fma2(acc[i][e], acc[i][e + 1], f[e], f[e + 1], wj, wj);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < PP; ++i) {
        const int c = c0 + i * dc;
        if (c >= H) continue;
        if (base) {
            float f[N];
            widen_piece<DT>(ld16(base + t * H + c), f);
#pragma unroll
            for (int e = 0; e < N; ++e) acc[i][e] += f[e];
        }
        st16(out + t * H + c, narrow_piece<DT>(acc[i]));
    }
}

// Bound by HBM (8192 x 4096, k = 8, bf16, padded to 128 rows: 195 us, 97 % of
// the measured copy bandwidth).  Blocks (token, batch of kb pairs): the token's
// gradient row is read once a batch, every pair's row of y read and of grad_y
// written once, the dot products reduced over the block; or a token a warp and
// eight of them a block (short rows, no block barrier: 16384 x 256, k = 8 24.7 us
// against 105 us).  Later blocks write zeros to the rows without a pair.
template <int DT, int KB, int PP, bool kWarp>
__global__ void __launch_bounds__(256, 3)
k_combine_backward(const typename RowType<DT>::T *go, const typename RowType<DT>::T *y, int T, int k, int kb, int H,
                   const int32_t *rows, const int32_t *inv, int64_t R, const float *w, typename RowType<DT>::T *gy,
                   float *gw, int token_blocks, int parts, int zero_rows) {
    constexpr int N = kPieceValues<DT>;
    __shared__ float red[8][KB];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    pdl_wait();
    pdl_trigger();
    if ((int)blockIdx.x >= token_blocks) {
        const int64_t r0 = (((int64_t)blockIdx.x - token_blocks) * warps + warp) * zero_rows;
        const unsigned none = rows_without_pair(rows, r0, zero_rows, R, T * (int64_t)k, lane);
        if (none) zero_words(reinterpret_cast<uint4 *>(gy), H * (int)sizeof(*gy) / 16, r0, zero_rows, none, lane);
        return;
    }
    const int part = blockIdx.x % parts;
    const int64_t t = kWarp ? (int64_t)(blockIdx.x / parts) * 8 + warp : blockIdx.x / parts;
    if (kWarp && t >= T) return;
    const int tid = kWarp ? lane : threadIdx.x, dc = (kWarp ? 32 : blockDim.x) * N;
    const int j0 = part * kb;
    int row[KB];
    float wj[KB], dot[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        const bool on = j < kb && j0 + j < k;
        row[j] = on ? inv[t * k + j0 + j] : -1;
        if (row[j] >= R) row[j] = -1;
        wj[j] = row[j] >= 0 ? w[t * k + j0 + j] : 0.0f;
        dot[j] = 0.0f;
    }
    for (int c0 = tid * N; c0 < H; c0 += PP * dc) {
        uint4 g[PP], v[KB][PP];
#pragma unroll
        for (int i = 0; i < PP; ++i)
            if (c0 + i * dc < H) g[i] = ld16(go + t * H + c0 + i * dc);
#pragma unroll
        for (int j = 0; j < KB; ++j)
#pragma unroll
            for (int i = 0; i < PP; ++i)
                if (row[j] >= 0 && c0 + i * dc < H) v[j][i] = ld16(y + (int64_t)row[j] * H + c0 + i * dc);
#pragma unroll
        for (int i = 0; i < PP; ++i) {
            if (c0 + i * dc >= H) continue;
            float gf[N];
            widen_piece<DT>(g[i], gf);
#pragma unroll
            for (int j = 0; j < KB; ++j) {
                if (row[j] < 0) continue;
                float f[N], d1 = 0.0f;
                widen_piece<DT>(v[j][i], f);
#pragma unroll
                for (int e = 0; e < N; e += 2) {
                    fma2(dot[j], d1, f[e], f[e + 1], gf[e], gf[e + 1]);
                    f[e] = gf[e];
                    f[e + 1] = gf[e + 1];
                    mul2(f, e, wj[j], wj[j]);
                }
                dot[j] += d1;
                st16(gy + (int64_t)row[j] * H + c0 + i * dc, narrow_piece<DT>(f));
            }
        }
    }
#pragma unroll
    for (int j = 0; j < KB; ++j) {
        dot[j] = warp_sum(dot[j]);
        if (kWarp) {
            if (lane == j && j < kb && j0 + j < k) gw[t * k + j0 + j] = dot[j];
        } else if (lane == 0) {
            red[warp][j] = dot[j];
        }
    }
    if constexpr (kWarp) return;
    __syncthreads();
    if (threadIdx.x < kb && j0 + threadIdx.x < k) {
        float s = 0.0f;
        for (int i = 0; i < warps; ++i) s += red[i][threadIdx.x];
        gw[t * k + j0 + threadIdx.x] = s;
    }
}

// Pairs a thread loads together, of k: 8, 5 (two pieces: 5, 9 and 10 pairs; 4096 x
// 8192, k = 10, bf16: 109 us against 113 with 8 and 2), 4 or 2; few tokens have
// too few threads for more than one piece each.
int pair_batch(int k, bool few) {
    if (few) return 8;
    if (k <= 4) return k <= 2 ? 2 : 4;
    return k == 5 || k == 9 || k == 10 ? 5 : 8;
}
int even_batch(int k, int most) { const int n = (k + most - 1) / most; return (k + n - 1) / n; }
constexpr int kFewTokens = 2 * 152;
// Up to here the backward pass takes a block a pair (4096 wide, k = 8, bf16: 4
// tokens 2.3 us against 3.5 us, 128 tokens 5.7 against 6.2, 200 tokens 7.8 against 7.6).
constexpr int kFewBackward = 152;

template <int DT, int KB>
cudaError_t launch_combine_k(const void *y, int T, int k, int H, const int32_t *inv, int64_t R, const float *w,
                             const void *base, void *out, cudaStream_t st) {
    using E = typename RowType<DT>::T;
    constexpr int PP = pair_pieces(KB);
    const int n = (H / kPieceValues<DT> + PP - 1) / PP;                       // threads that a row can use
    const int tx = std::min(kCombineThreads, (n + 31) / 32 * 32), ty = kCombineThreads / tx;
    return launch_pdl(k_combine<DT, KB, PP>, dim3(blocks_of(T, ty), (n + tx - 1) / tx), dim3(tx, ty), 0, st,
                      static_cast<const E *>(y), T, k, H, inv, R, w, static_cast<const E *>(base),
                      static_cast<E *>(out));
}

template <int DT>
cudaError_t launch_combine(const void *y, int T, int k, int H, const int32_t *inv, int64_t R, const float *w,
                           const void *base, void *out, cudaStream_t st) {
    switch (pair_batch(k, T <= kFewTokens)) {
        case 2: return launch_combine_k<DT, 2>(y, T, k, H, inv, R, w, base, out, st);
        case 4: return launch_combine_k<DT, 4>(y, T, k, H, inv, R, w, base, out, st);
        case 5: return launch_combine_k<DT, 5>(y, T, k, H, inv, R, w, base, out, st);
        default: return launch_combine_k<DT, 8>(y, T, k, H, inv, R, w, base, out, st);
    }
}

template <int DT, int KB>
cudaError_t launch_combine_backward_k(const void *go, const void *y, int T, int k, int H, const int32_t *rows,
                                      const int32_t *inv, int64_t R, const float *w, void *gy, float *gw,
                                      cudaStream_t st) {
    using E = typename RowType<DT>::T;
    constexpr int PP = pair_pieces(KB);
    const bool few = T <= kFewBackward, warp = !few && H / kPieceValues<DT> <= 32 * (KB > 4 ? 4 : 8);
    const int kb = few ? 1 : even_batch(k, KB);
    const int pieces = (H / kPieceValues<DT> + PP - 1) / PP;                  // threads that a row can use
    const int threads = warp ? 256 : std::max(few ? 128 : 32, std::min(256, (pieces + 31) / 32 * 32));
    const int parts = (k + kb - 1) / kb;
    const int64_t token_blocks = (int64_t)(warp ? blocks_of(T, 8) : T) * parts;
    const int zero_rows = zero_rows_a_warp(H * (int)sizeof(E) / 16), block_rows = threads / 32 * zero_rows;
    const int64_t blocks = token_blocks + (R + block_rows - 1) / block_rows;
    if (blocks > kMaxRows) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)blocks);
    auto kernel = warp ? k_combine_backward<DT, KB, PP, true> : k_combine_backward<DT, KB, PP, false>;
    return launch_pdl(kernel, grid, dim3(threads), 0, st, static_cast<const E *>(go), static_cast<const E *>(y), T, k,
                      kb, H, rows, inv, R, w, static_cast<E *>(gy), gw, (int)token_blocks, parts, zero_rows);
}

template <int DT>
cudaError_t launch_combine_backward(const void *go, const void *y, int T, int k, int H, const int32_t *rows,
                                    const int32_t *inv, int64_t R, const float *w, void *gy, float *gw,
                                    cudaStream_t st) {
    switch (T <= kFewBackward ? 2 : pair_batch(k, false)) {
        case 2: return launch_combine_backward_k<DT, 2>(go, y, T, k, H, rows, inv, R, w, gy, gw, st);
        case 4: return launch_combine_backward_k<DT, 4>(go, y, T, k, H, rows, inv, R, w, gy, gw, st);
        case 5: return launch_combine_backward_k<DT, 5>(go, y, T, k, H, rows, inv, R, w, gy, gw, st);
        default: return launch_combine_backward_k<DT, 8>(go, y, T, k, H, rows, inv, R, w, gy, gw, st);
    }
}

// ----------------------------------------------------------------- checks

moe_status check_pairs(int32_t T, int32_t k, int64_t rows) {
    if (T < 0 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (k < 1 || k > kMaxTopK || (int64_t)T * k > kMaxRows || rows > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status check_values(int32_t dtype, int32_t H) {
    if (!known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (H < kChunk || H > kMaxCombineH || H % kChunk) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

int64_t moe_sorted_rows(int64_t pairs, int32_t num_experts, int32_t align) {
    if (pairs < 0 || pairs > kMaxRows || num_experts < 1 || num_experts > kMaxExperts) return -1;
    if (align < 1 || align > kMaxAlign || (align & (align - 1))) return -1;
    return (pairs + std::min<int64_t>(num_experts, pairs) * (align - 1)) / align * align;
}

moe_status moe_sort_pairs(const int32_t *topk_ids, int32_t T, int32_t k, int32_t num_experts, int32_t align,
                          int64_t rows, int32_t *expert_offsets, int32_t *sorted_rows, int32_t *pair_rows,
                          void *stream) {
    moe_status st = check_pairs(T, k, rows);
    if (st != MOE_OK) return st;
    const int64_t want = moe_sorted_rows((int64_t)T * k, num_experts, align);
    if (want < 0 || want > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (rows != want || !expert_offsets) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!topk_ids || !sorted_rows || !pair_rows)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(topk_ids, 4) || !aligned_to(expert_offsets, 4) || !aligned_to(sorted_rows, 4) ||
        !aligned_to(pair_rows, 4))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) return cuda_status(cudaMemsetAsync(expert_offsets, 0, sizeof(int32_t) * (num_experts + 1), s));
    if (configure_sort() != cudaSuccess) return MOE_ERR_CUDA;
    const int P = T * k, E = num_experts;
    int blocks = 1;
    while (blocks < kSortBlocks && (int64_t)blocks * kSortPairs < P) blocks *= 2;
    SortArgs a{topk_ids, P, E, align, 0, 0, rows, expert_offsets, sorted_rows, pair_rows};
    a.warps = (int)std::min<int64_t>(kSortMaxWarps, ((int64_t)P + 32 * blocks - 1) / (32 * blocks));
    a.run = (int)(((int64_t)P + 32LL * a.warps * blocks - 1) / (32LL * a.warps * blocks)) * 32;
    const int threads = std::max(32 * a.warps, (E + 31) / 32 * 32);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = sort_smem(a.warps, E);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = blocks;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 2 : 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, blocks > 1 ? k_sort_pairs<true> : k_sort_pairs<false>, a));
}

moe_status moe_dispatch(const void *x, int64_t x_stride_bytes, int64_t row_bytes, const void *scales,
                        int32_t scale_bytes, int32_t T, int32_t k, const int32_t *sorted_rows,
                        const int32_t *pair_rows, int64_t rows, void *out, void *out_scales, void *stream) {
    moe_status st = check_pairs(T, k, rows);
    if (st != MOE_OK) return st;
    if (row_bytes < 16 || row_bytes % 16 || row_bytes > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    if (x_stride_bytes < row_bytes || x_stride_bytes % 16 || scale_bytes < 0) return MOE_ERR_UNSUPPORTED_SHAPE;
    if ((scales != nullptr) != (out_scales != nullptr) || (scales != nullptr) != (scale_bytes > 0))
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if ((T > 0 && (!x || !pair_rows)) || !sorted_rows || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(out, 16) || !aligned_to(sorted_rows, 4) || !aligned_to(pair_rows, 4))
        return MOE_ERR_MISALIGNED;
    // a row's threads, the rows a block takes, and the blocks a row takes
    const int n = (int)(row_bytes / 16);
    const int tx = std::min(256, ((n + kCopyPieces - 1) / kCopyPieces + 31) / 32 * 32), ty = 256 / tx;
    const int parts = (n + tx * kCopyPieces - 1) / (tx * kCopyPieces);
    const int64_t token_blocks = (int64_t)blocks_of(T, ty) * parts;
    const int zero_rows = zero_rows_a_warp(n), block_rows = tx * ty / 32 * zero_rows;
    const int64_t blocks = token_blocks + (rows + block_rows - 1) / block_rows;
    if (blocks > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    const dim3 grid((unsigned)blocks);
    auto launch = [&](auto kernel, int word) {
        return cuda_status(launch_pdl(kernel, grid, dim3(tx, ty), 0, static_cast<cudaStream_t>(stream),
                                      static_cast<const char *>(x), x_stride_bytes, n,
                                      static_cast<const char *>(scales), (int)(scale_bytes / word), (int)T, (int)k,
                                      sorted_rows, pair_rows, rows, static_cast<char *>(out),
                                      static_cast<char *>(out_scales), (int)token_blocks, parts, zero_rows));
    };
    // scale rows are copied in words as wide as their length and addresses allow
    auto wide = [&](int a) { return scale_bytes % a == 0 && aligned_to(scales, a) && aligned_to(out_scales, a); };
    if (wide(16)) return launch(k_dispatch<uint4>, 16);
    if (wide(4)) return launch(k_dispatch<uint32_t>, 4);
    return launch(k_dispatch<uint8_t>, 1);
}

moe_status moe_combine(const void *y, int32_t dtype, int32_t T, int32_t k, int32_t H, const int32_t *pair_rows,
                       int64_t rows, const float *weights, const void *base, void *out, void *stream) {
    moe_status st = check_pairs(T, k, rows);
    if (st == MOE_OK) st = check_values(dtype, H);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if ((!y && rows > 0) || !pair_rows || !out) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(y, 16) || !aligned_to(base, 16) || !aligned_to(out, 16) || !aligned_to(pair_rows, 4) ||
        !aligned_to(weights, 4))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MOE_DTYPE_F32:
            return cuda_status(launch_combine<MOE_DTYPE_F32>(y, T, k, H, pair_rows, rows, weights, base, out, s));
        case MOE_DTYPE_BF16:
            return cuda_status(launch_combine<MOE_DTYPE_BF16>(y, T, k, H, pair_rows, rows, weights, base, out, s));
        default:
            return cuda_status(launch_combine<MOE_DTYPE_F16>(y, T, k, H, pair_rows, rows, weights, base, out, s));
    }
}

moe_status moe_combine_backward(const void *grad_out, const void *y, int32_t dtype, int32_t T, int32_t k, int32_t H,
                                const int32_t *sorted_rows, const int32_t *pair_rows, int64_t rows,
                                const float *weights, void *grad_y, float *grad_weights, void *stream) {
    moe_status st = check_pairs(T, k, rows);
    if (st == MOE_OK) st = check_values(dtype, H);
    if (st != MOE_OK) return st;
    if (T == 0) return MOE_OK;
    if (!grad_out || !pair_rows || !weights || !grad_weights) return MOE_ERR_INVALID_ARG;
    if (rows > 0 && (!y || !sorted_rows || !grad_y)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(grad_out, 16) || !aligned_to(y, 16) || !aligned_to(grad_y, 16) || !aligned_to(sorted_rows, 4) ||
        !aligned_to(pair_rows, 4) || !aligned_to(weights, 4) || !aligned_to(grad_weights, 4))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    switch (dtype) {
        case MOE_DTYPE_F32:
            return cuda_status(launch_combine_backward<MOE_DTYPE_F32>(grad_out, y, T, k, H, sorted_rows, pair_rows,
                                                                      rows, weights, grad_y, grad_weights, s));
        case MOE_DTYPE_BF16:
            return cuda_status(launch_combine_backward<MOE_DTYPE_BF16>(grad_out, y, T, k, H, sorted_rows, pair_rows,
                                                                       rows, weights, grad_y, grad_weights, s));
        default:
            return cuda_status(launch_combine_backward<MOE_DTYPE_F16>(grad_out, y, T, k, H, sorted_rows, pair_rows,
                                                                      rows, weights, grad_y, grad_weights, s));
    }
}

}  // extern "C"
