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

// ------------------------------------------------------------------- sort

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxAlign = 256;

// Inclusive scan over the block's 1024 threads; `red` holds 32 words.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t *red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    if (lane == 31) red[warp] = v;
    __syncthreads();
    if (warp == 0) {
        int64_t w = red[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += u;
        }
        red[lane] = w;
    }
    __syncthreads();
    return warp ? v + red[warp - 1] : v;
}

// Counting sort in one launch of one cluster.  Every warp owns a contiguous
// run of pairs: it counts them per expert in shared memory; the blocks read
// each other's per-expert totals through distributed shared memory (a cluster
// barrier on either side), scan them into the segments' first rows, and place
// the pairs in order.  Latency-bound: two passes over the ids and two barriers.
__global__ void __launch_bounds__(kSortThreads) k_sort_pairs(const int32_t *__restrict__ ids, int P, int E, int align,
                                                             int64_t R, int32_t *__restrict__ offsets,
                                                             int32_t *__restrict__ rows,
                                                             int32_t *__restrict__ inv) {
    cg::cluster_group cl = cg::this_cluster();
    extern __shared__ int smem[];
    int *wc = smem;                       // [32][E] a warp's counts, then its next rows
    int *tot = smem + kSortWarps * E;     // [E] this block's counts
    int *s_pad = tot + E;                 // [E][2] a segment's first row of padding and its end
    __shared__ int64_t red[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nb = (int)cl.num_blocks(), rank = (int)cl.block_rank();
    for (int i = tid; i < kSortWarps * E; i += kSortThreads) wc[i] = 0;
    __syncthreads();
    // this warp's run of pairs, a multiple of 32 long
    const int64_t seg = ((int64_t)P + (int64_t)nb * kSortThreads - 1) / ((int64_t)nb * kSortThreads) * 32;
    const int64_t beg = std::min<int64_t>(P, seg * (rank * kSortWarps + warp));
    const int64_t end = std::min<int64_t>(P, beg + seg);
    int *mine = wc + warp * E;
    for (int64_t p = beg + lane; p < end; p += 32) {
        const int e = ids[p];
        if (e >= 0 && e < E) atomicAdd(mine + e, 1);
    }
    __syncthreads();
    for (int e = tid; e < E; e += kSortThreads) {
        int c = 0;
        for (int w = 0; w < kSortWarps; ++w) c += wc[w * E + e];
        tot[e] = c;
    }
    cl.sync();
    int count = 0, before = 0;            // thread e: expert e's pairs, and those of the blocks before
    if (tid < E)
        for (int b = 0; b < nb; ++b) {
            const int c = cl.map_shared_rank(tot, b)[tid];
            count += c;
            if (b < rank) before += c;
        }
    const int64_t padded = ((int64_t)count + align - 1) / align * align;
    const int64_t last = block_scan(padded, red);   // E <= 1024 threads
    if (tid < E) {
        int run = (int)(last - padded);
        if (rank == 0) {
            offsets[tid] = run;
            if (tid == E - 1) offsets[E] = (int)last;
        }
        s_pad[2 * tid] = run + count;
        s_pad[2 * tid + 1] = (int)last;
        run += before;
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = wc[w * E + tid];
            wc[w * E + tid] = run;
            run += c;
        }
    }
    cl.sync();                            // the other blocks have read `tot`; this one's tables are written
    for (int64_t p0 = beg; p0 < end; p0 += 32) {
        const int64_t p = p0 + lane;
        int e = p < end ? ids[p] : -1;
        if (e >= E) e = -1;
        const unsigned peers = __match_any_sync(0xffffffffu, e);
        int row = -1;
        if (e >= 0) row = mine[e] + __popc(peers & ((1u << lane) - 1u));
        __syncwarp();
        if (e >= 0 && lane == __ffs(peers) - 1) mine[e] += __popc(peers);
        __syncwarp();
        if (p < end) {
            inv[p] = row;
            if (row >= 0 && row < R) rows[row] = (int)p;   // ids that changed meanwhile write nothing out of range
        }
    }
    // rows without a pair: every segment's padding, then what is past the last segment
    for (int e = rank * kSortWarps + warp; e < E; e += nb * kSortWarps)
        for (int r = s_pad[2 * e] + lane; r < s_pad[2 * e + 1]; r += 32) rows[r] = -1;
    for (int64_t r = (int64_t)s_pad[2 * E - 1] + rank * kSortThreads + tid; r < R; r += (int64_t)nb * kSortThreads)
        rows[r] = -1;
}

size_t sort_smem(int E) { return sizeof(int) * ((size_t)kSortWarps + 3) * E; }

// The kernel's shared-memory limit, once a device and for the largest E.
cudaError_t configure_sort() {
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(k_sort_pairs, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sort_smem(kMaxExperts));
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

// --------------------------------------------------------------- dispatch

// One warp a row of out: 16 bytes a lane and step.
__global__ void __launch_bounds__(256) k_dispatch(const char *x, int64_t xs, int64_t row_bytes, const char *scales,
                                                  int scale_bytes, int T, int k, const int32_t *__restrict__ rows,
                                                  int64_t R, char *out, char *out_scales) {
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (r >= R) return;
    const int p = rows[r];
    const int64_t t = (p >= 0 && p < T * (int64_t)k) ? p / k : -1;
    for (int64_t c = lane * 16; c < row_bytes; c += 512)
        st16(out + r * row_bytes + c, t < 0 ? make_uint4(0, 0, 0, 0) : ld16(x + t * xs + c));
    for (int c = lane; c < scale_bytes; c += 32)
        out_scales[r * scale_bytes + c] = t < 0 ? 0 : scales[t * scale_bytes + c];
}

// ---------------------------------------------------------------- combine

constexpr int kPairBatch = 8;   // rows of a token in flight together

template <int DT>
__global__ void k_combine(const typename RowType<DT>::T *y, int k, int H, const int32_t *__restrict__ inv, int64_t R,
                          const float *__restrict__ w, const typename RowType<DT>::T *base,
                          typename RowType<DT>::T *out) {
    const int64_t t = blockIdx.x;
    const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kChunk;
    if (c >= H) return;
    float acc[8] = {};
    for (int j0 = 0; j0 < k; j0 += kPairBatch) {
        Raw8<DT> v[kPairBatch];
        bool on[kPairBatch];
#pragma unroll
        for (int j = 0; j < kPairBatch; ++j) {
            const int row = j0 + j < k ? inv[t * k + j0 + j] : -1;
            on[j] = row >= 0 && row < R;
            if (on[j]) v[j] = load8<DT>(y + (int64_t)row * H + c);
        }
#pragma unroll
        for (int j = 0; j < kPairBatch; ++j) {
            if (!on[j]) continue;
            const float wj = w ? w[t * k + j0 + j] : 1.0f;
            float f[8];
            widen8<DT>(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(wj, f[e], acc[e]);
        }
    }
    if (base) {
        float f[8];
        widen8<DT>(load8<DT>(base + t * H + c), f);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] += f[e];
    }
    store8<DT>(out + t * H + c, narrow8<DT>(acc));
}

// Blocks 0..T-1: one token each, its gradient row read once, every pair's row
// of y read and of grad_y written once, the dot products reduced over the
// block.  Later blocks: zeros for the rows without a pair, 8 rows a block.
template <int DT>
__global__ void __launch_bounds__(256) k_combine_backward(const typename RowType<DT>::T *go,
                                                          const typename RowType<DT>::T *y, int T, int k, int H,
                                                          const int32_t *__restrict__ rows,
                                                          const int32_t *__restrict__ inv, int64_t R,
                                                          const float *__restrict__ w,
                                                          typename RowType<DT>::T *gy, float *__restrict__ gw) {
    __shared__ float red[8][kPairBatch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (blockIdx.x >= T) {
        const int64_t r = ((int64_t)blockIdx.x - T) * 8 + warp;
        if (r >= R) return;
        const int p = rows[r];
        if (p >= 0 && p < T * (int64_t)k) return;
        const float zero[8] = {};
        for (int c = lane * kChunk; c < H; c += 32 * kChunk) store8<DT>(gy + r * H + c, narrow8<DT>(zero));
        return;
    }
    const int64_t t = blockIdx.x;
    for (int j0 = 0; j0 < k; j0 += kPairBatch) {
        int64_t row[kPairBatch];
        float wj[kPairBatch], dot[kPairBatch];
#pragma unroll
        for (int j = 0; j < kPairBatch; ++j) {
            row[j] = j0 + j < k ? inv[t * k + j0 + j] : -1;
            if (row[j] >= R) row[j] = -1;
            wj[j] = row[j] >= 0 ? w[t * k + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = threadIdx.x * kChunk; c < H; c += blockDim.x * kChunk) {
            float g[8];
            widen8<DT>(load8<DT>(go + t * H + c), g);
            Raw8<DT> v[kPairBatch];
#pragma unroll
            for (int j = 0; j < kPairBatch; ++j)
                if (row[j] >= 0) v[j] = load8<DT>(y + row[j] * H + c);
#pragma unroll
            for (int j = 0; j < kPairBatch; ++j) {
                if (row[j] < 0) continue;
                float f[8], o[8];
                widen8<DT>(v[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dot[j] = fmaf(g[e], f[e], dot[j]);
                    o[e] = wj[j] * g[e];
                }
                store8<DT>(gy + row[j] * H + c, narrow8<DT>(o));
            }
        }
#pragma unroll
        for (int j = 0; j < kPairBatch; ++j) {
            const float s = warp_sum(dot[j]);
            if (lane == 0) red[warp][j] = s;
        }
        __syncthreads();
        if (threadIdx.x < kPairBatch && j0 + threadIdx.x < k) {
            float s = 0.0f;
            for (int i = 0; i < (int)blockDim.x / 32; ++i) s += red[i][threadIdx.x];
            gw[t * k + j0 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// Threads for a row of n8 pieces.
int row_threads(int n8) { return std::min(256, (n8 + 31) / 32 * 32); }

template <int DT>
cudaError_t launch_combine(const void *y, int T, int k, int H, const int32_t *inv, int64_t R, const float *w,
                           const void *base, void *out, cudaStream_t st) {
    using E = typename RowType<DT>::T;
    const int n8 = H / kChunk, th = row_threads(n8);
    k_combine<DT><<<dim3(T, (n8 + th - 1) / th), th, 0, st>>>(static_cast<const E *>(y), k, H, inv, R, w,
                                                             static_cast<const E *>(base), static_cast<E *>(out));
    return cudaGetLastError();
}

template <int DT>
cudaError_t launch_combine_backward(const void *go, const void *y, int T, int k, int H, const int32_t *rows,
                                    const int32_t *inv, int64_t R, const float *w, void *gy, float *gw,
                                    cudaStream_t st) {
    using E = typename RowType<DT>::T;
    k_combine_backward<DT><<<(unsigned)(T + (R + 7) / 8), 256, 0, st>>>(
        static_cast<const E *>(go), static_cast<const E *>(y), T, k, H, rows, inv, R, w, static_cast<E *>(gy), gw);
    return cudaGetLastError();
}

// ----------------------------------------------------------------- checks

constexpr int64_t kMaxRows = 0x7fffffff;

moe_status check_pairs(int32_t T, int32_t k, int64_t rows) {
    if (T < 0 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (k < 1 || k > kMaxTopK || (int64_t)T * k > kMaxRows || rows > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
    return MOE_OK;
}

moe_status check_values(int32_t dtype, int32_t H) {
    if (!known_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (H < kChunk || H % kChunk) return MOE_ERR_UNSUPPORTED_SHAPE;
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
    while (blocks < 8 && (int64_t)blocks * 2048 < P) blocks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_smem(E);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cuda_status(cudaLaunchKernelEx(&cfg, k_sort_pairs, topk_ids, P, E, (int)align, rows, expert_offsets,
                                          sorted_rows, pair_rows));
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
    k_dispatch<<<(unsigned)((rows + 7) / 8), 256, 0, static_cast<cudaStream_t>(stream)>>>(
        static_cast<const char *>(x), x_stride_bytes, row_bytes, static_cast<const char *>(scales), scale_bytes, T, k,
        sorted_rows, rows, static_cast<char *>(out), static_cast<char *>(out_scales));
    return cuda_status(cudaGetLastError());
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
