// The 4-bit product of more than a few tokens (see linear.cu for its formula) on the block-scaled FP4 tensor cores
// (tcgen05 kind::mxf4nvf4 and kind::mxf4), which take the weight's codes and scales as they lie in memory: no code is
// widened, and the warp MMAs that bound linear.cu from nine tokens on are gone.
//
// These MMAs want the tokens in 4 bits too.  A token's 16 (MXFP4: 32) values that share a scale are therefore written as
// integers of 23 bits in eight balanced octal digits,
//   x = 2^(e - 21) * (d0 * 8^7 + d1 * 8^6 + ... + d7),      -4 <= d <= 3,      largest |x| < 2^(e + 1),
// each of which E2M1 holds: what is dropped is at most 2^(e - 22).  Sixteen tokens are 128 columns of the MMA, a column a
// digit.  Adding octal 44444444 to the integer makes its digits d + 4, all from 0 to 7, so no digit waits for another's carry.
//   The columns' block scales give a block its power.  E4M3 holds 2^-9 to 2^8, so NVFP4 brings a token's largest value to
// [2^7, 2^8), gives a block's eight columns the one scale of 2^(e + 1), and the epilogue adds their sums with factors of 8^-i:
// a block whose largest value is below 2^-17 of the token's is written as if it were that, to 2^-39 of it.  (With the powers
// of eight in the scales as well that was 2^-30.)
//   E8M0 holds the powers of eight too, so MXFP4 has them in the scales and takes a token's values as they are; only a token
// below 2^-20 is brought there, so that its smallest digits have a power (a block below 2^-106 is written as if it were
// that).  A column's sum then passes fp32 only where the result does: 65536 values of 2^-20 times 6 * 2^127 stay below 2^127.
//   Infinities and NaNs count as zeros in the digits; the epilogue of a token that holds some adds their products.
//
// Two launches: k_linear_digits writes the digits and scales (8 x 4.5 bits a value), k_linear_tc multiplies; its blocks load
// weights while the digits are still being written.  An item is 256 weight rows (the M side, two accumulators of 128) x 16
// tokens x a part of K; the parts of an item are a cluster's blocks, each of which adds a share of the rows, in order.
//
// Bound by the weight's bytes where there are enough of them: 1 x 100003 x 4096 NVFP4 42.9 us (0.80 of the copy bandwidth),
// 16 x 100000 x 4096 45.5 (0.76), 16 x 38912 x 7168 37.9 (0.62), 16 x 16384 x 7168 MXFP4 21.9 (0.43; the warp MMAs of linear.cu
// 27.7).  About 8 us are outside the stream (digits, the first token tile, joining and storing), which itself runs at 4.5 TB/s
// (16 x 16384 x 7168) to 6.6 (1 x 100003 x 4096).  Every 16 tokens more read weights and digits from L2, 54 KB a stage in 0.53
// us, near what an SM takes from it: 64 x 38912 x 7168 67 us.  Tokens go in pieces of 256 (256 x 16384 x 7168 111 us, 1024 x
// 16384 x 7168 443), so this is not made for prompts.
// Tried, 16 x 16384 x 7168: digits made in the multiplying blocks by the warps of the epilogue 30 us (each block makes all of
// them again, 1.5 us a stage); rings of their own for weights, five stages, and digits, two, 22.2; groups of 216 rows that
// fill all SMs instead of 128 of them 25.0 (the next launch's blocks find no room beside the last ones).
#include <algorithm>

#include "linear.cuh"
#include "tc.cuh"

namespace {

using namespace moe;

constexpr int kDigits = 8, kTileTokens = 16;
constexpr int kStages = 4;
constexpr int kBK = 256;                       // K values a stage
constexpr int kRowBytes = kBK / 2;
constexpr int kTile = 128 * kRowBytes;         // codes of 128 rows
constexpr int kSf = 128 * 16;                  // their scales
constexpr int kStageBytes = 3 * kTile + 3 * kSf;
constexpr size_t kSmem = kStages * kStageBytes + 512 + 1024;
constexpr uint32_t kSfCol0 = 256;              // scales in tensor memory, behind the two accumulators
constexpr int kSfStride = 48;                  // columns of a stage's: A0, A1, B
constexpr int kThreads = 32 * 14;              // TMA, MMA, four scale warps, eight epilogue warps
constexpr int kEpiWarp0 = 6;
constexpr int kChunkTokens = 256;              // tokens a pair of launches
constexpr int kMaxParts = 8;
constexpr int kLeastMx = -20;                  // the least exponent of a token's largest value, MXFP4

static_assert(kSmem <= kSmemBlock, "the stages exceed a block's shared memory");

// Where a call's workspace holds what; tiles of 16 tokens, groups of 256 rows.
struct Layout {
    int tiles, groups, parts, stages, atoms;   // atoms: 512 bytes of token scales a tile and 64 (MXFP4: 128) values
    size_t codes, scales, partial, info, bytes;
};

struct TcArgs {
    CUtensorMap a, sa, b;
    const uint8_t *codes, *scales;             // the weight
    const float *ts;
    const uint8_t *b_scales;
    const void *x;
    int64_t x_stride;
    void *out;
    float *partial;                            // [part][T][N]
    const int2 *info;                          // a token's power of two, and 1 where it holds infinities or NaNs
    int T, N, K, bf16, dtype;
    int tiles, groups, parts, stages, atoms, rows;
};

struct DigitArgs {
    const void *x;
    int64_t x_stride;
    uint8_t *codes, *scales;
    int2 *info;
    int T, K, bf16, atoms;
};

// Eight values of a row in fp32.
__device__ __forceinline__ void row8(const void *x, int64_t at, int bf16, float (&v)[8]) {
    const uint4 raw = ld16_shared(static_cast<const uint16_t *>(x) + at);
    if (bf16) widen8<MOE_DTYPE_BF16>(Raw8<MOE_DTYPE_BF16>{raw}, v);
    else widen8<MOE_DTYPE_F16>(Raw8<MOE_DTYPE_F16>{raw}, v);
}

// A power of two as an E4M3 scale: 2^-9 to 2^8.
__device__ __forceinline__ uint32_t e4m3_power(int q) { return q >= -6 ? (uint32_t)(q + 7) << 3 : 1u << (q + 9); }

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
// Bits of a where the mask has ones, of b elsewhere.
__device__ __forceinline__ uint32_t choose(uint32_t mask, uint32_t a, uint32_t b) { return (a & mask) | (b & ~mask); }

// One block a token and 1024 of its values; a thread writes the digits of eight, lanes beside one another share a scale.
template <bool MX> __global__ void __launch_bounds__(128) k_linear_digits(DigitArgs a) {
    constexpr int kLanes = MX ? 4 : 2;         // of a scale block
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.y;
    const int64_t row = t * a.x_stride;
    const int at = blockIdx.x * 1024 + threadIdx.x * 8;
    float v[8] = {};
    if (at < a.K) row8(a.x, row + at, a.bf16, v);
    // the token's largest finite magnitude
    float m = 0.0f;
    int bad = 0;
#pragma unroll 8
    for (int i = threadIdx.x * 8; i < a.K; i += 128 * 8) {
        float w[8];
        row8(a.x, row + i, a.bf16, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = fabsf(w[j]);
            if (s < INFINITY) m = fmaxf(m, s);
            else bad = 1;
        }
    }
    __shared__ float most[4];
    m = warp_max(m);
    if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
    bad = __syncthreads_or(bad);
    const int E = exponent_of(fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])));
    const int lift = MX ? max(0, kLeastMx - E) : 0;
    const float up = MX ? power_of_two(lift) : scale_up(E), more = MX ? 1.0f : scale_more(E);
    // what undoes it; NVFP4's scales are twice a digit's weight
    if (blockIdx.x == 0 && threadIdx.x == 0) a.info[t] = make_int2(MX ? -lift : E - 8, bad);

    m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = fabsf(v[j]) < INFINITY ? v[j] * up * more : 0.0f;
        m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (at >= a.K) return;                     // K is a multiple of a warp's 256 values
    const int lane = threadIdx.x & 31;
    const int e = max(exponent_of(m), MX ? -106 : -10);    // at most 127, NVFP4 7
    const float fixed = power_of_two(21 - e);
    // digits of a value in the nibbles of a word: 24 bits spread to 32 in three steps (what strays into a nibble's fourth
    // bit is cleared at the end)
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        uint32_t y = (uint32_t)(__float2int_rn(v[j] * fixed) + 044444444);
        y = choose(0x00000FFFu, y, y << 4);
        y = choose(0x003F003Fu, y, y << 2);
        y = choose(0x07070707u, y, y << 1);
        r[j] = y & 0x77777777u;
    }
    // words of one digit of all eight: nibbles, then bytes change places; even values in the low half, odd ones in the high
    uint32_t low[4], high[4];                  // digits 8^0, 8^2, 8^4, 8^6 and 8^1, ... of values (0, 2), (4, 6), (1, 3), (5, 7)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t x = r[4 * (i & 1) + (i >> 1)], y = r[4 * (i & 1) + (i >> 1) + 2];
        low[i] = choose(0x0F0F0F0Fu, x, y << 4);
        high[i] = choose(0x0F0F0F0Fu, x >> 4, y);
    }
    const int tile = t / kTileTokens, r0 = (t % kTileTokens) * kDigits;
    uint8_t *codes = a.codes + ((int64_t)tile * 128 + r0) * (a.K / 2) + at / 2;
    auto store = [&](int power, uint32_t s) {
        // E2M1 codes of -4, -3, -2, -1, 0, 1, 2, 3
        const uint32_t even = prmt(0x0A0C0D0Eu, 0x05040200u, s), odd = prmt(0x0A0C0D0Eu, 0x05040200u, s >> 16);
        const int d = 7 - power;
        *reinterpret_cast<uint32_t *>(codes + (int64_t)d * (a.K / 2)) = even | odd << 4;
    };
    auto bytes = [&](const uint32_t (&w)[4], int odd) {
        const uint32_t t0 = prmt(w[0], w[1], 0x5140), t1 = prmt(w[2], w[3], 0x5140), t2 = prmt(w[0], w[1], 0x7362), t3 = prmt(w[2], w[3], 0x7362);
        store(odd, prmt(t0, t1, 0x5410));
        store(odd + 2, prmt(t0, t1, 0x7632));
        store(odd + 4, prmt(t2, t3, 0x5410));
        store(odd + 6, prmt(t2, t3, 0x7632));
    };
    bytes(low, 0);
    bytes(high, 1);
    // scales: a lane writes one digit's of four blocks
    const int d = lane & 7, from = lane & ~(4 * kLanes - 1);
    uint32_t word = 0u;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
        const int eb = __shfl_sync(0xffffffffu, e, from + kLanes * b);
        word |= (MX ? (uint32_t)(127 + eb - 3 * d) : e4m3_power(eb + 1)) << (8 * b);
    }
    uint8_t *scales = a.scales + ((int64_t)tile * a.atoms + at / (32 * kLanes)) * 512 + (r0 & 31) * 16 + (r0 >> 5) * 4;
    if (!MX || (lane & 8) == 0) *reinterpret_cast<uint32_t *>(scales + d * 16) = word;
}

struct Item {
    int tile, group;
};
__device__ __forceinline__ Item item_at(const TcArgs &a, int i) { return {i % a.tiles, i / a.tiles}; }   // tiles of the same weights run beside one another

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}
// Arrives at the barrier of the cluster's block `rank`, with what this block's threads wrote before.
__device__ __forceinline__ void arrive_at(uint64_t *bar, uint32_t rank) {
    asm volatile(
        "{\n\t.reg .b32 at;\n\tmapa.shared::cluster.u32 at, %0, %1;\n\t"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [at];\n\t}" ::"r"(smem_u32(bar)), "r"(rank)
        : "memory");
}

// Row n's share of the products of token t's infinities and NaNs, over the item's K.
template <bool MX> __device__ __noinline__ float beyond(const TcArgs &a, int t, int n, int k0, int k1) {
    float s = 0.0f;
    for (int k = k0; k < k1; k += 8) {
        float v[8];
        row8(a.x, t * a.x_stride + k, a.bf16, v);
        for (int j = 0; j < 8; ++j) {
            if (fabsf(v[j]) < INFINITY) continue;
            const int at = k + j;
            const uint32_t code = a.codes[(int64_t)n * (a.K / 2) + at / 2] >> (4 * (at & 1)) & 15u;
            const uint32_t scale = a.scales[(int64_t)n * (a.K / (MX ? 32 : 16)) + at / (MX ? 32 : 16)];
            const float w = f16x2_to_f32x2(e2m1x2_to_f16x2(code)).x;
            const float sv = MX ? (scale == 255u ? NAN : __uint_as_float(scale ? scale << 23 : 0x400000u)) : e4m3_to_f32(scale);
            s = fmaf(v[j], w * sv, s);
        }
    }
    return s;
}

// mbar_wait for what other blocks of the cluster wrote.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity, int *err) {
    auto test = [&]() {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
        return done != 0;
    };
    const uint64_t t0 = now_ns();
    while (!test())
        if (now_ns() - t0 > kWaitNs) {
            atomicOr(err, kErrTimeout);
            return false;
        }
    return true;
}

__device__ __forceinline__ void store_out(const TcArgs &a, int64_t at, float s) {
    if (a.dtype == MOE_DTYPE_F32) static_cast<float *>(a.out)[at] = s;
    else if (a.dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(s);
    else static_cast<__half *>(a.out)[at] = __float2half_rn(s);
}

// Every wait is bounded (about a second): where one runs out the results are NaN.
template <bool MX> __global__ void __launch_bounds__(kThreads, 1) k_linear_tc(const __grid_constant__ TcArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kStages * kStageBytes);
    uint64_t *sf_ready = full + kStages;
    uint64_t *empty = sf_ready + kStages;
    uint64_t *acc_full = empty + kStages;
    uint64_t *acc_empty = acc_full + 1;
    uint64_t *drain = acc_empty + 1;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(drain + 1);
    int *err = reinterpret_cast<int *>(tmem_slot + 1);   // this block's
    // Every part's sums of an item are there: two barriers in turn.  A part that is ahead may arrive for its next item before
    // another's arrival for this one has come to this block (it came to that part first), and would complete the phase in
    // its place.  An arrival for the item after next is behind the other's for the next one, which that issued behind all of
    // its arrivals for this.
    uint64_t *joined = drain + 2;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int items = a.tiles * a.groups, first = blockIdx.x / a.parts, step = gridDim.x / a.parts;
    const int part = blockIdx.x % a.parts;     // rank in the cluster
    const int k0 = part * a.stages / a.parts, k1 = (part + 1) * a.stages / a.parts;   // stages of K
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full + s, 1);
            mbar_init(sf_ready + s, 4);
            mbar_init(empty + s, 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 8);
        mbar_init(drain, 1);
        mbar_init(joined, a.parts);
        mbar_init(joined + 1, a.parts);
        *err = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    if (a.parts > 1) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, used = 0, last_ph = 0;
            bool ok = true;
            const uint32_t b_bytes = a.rows * kRowBytes;
            constexpr uint32_t kBSf = MX ? kSf / 2 : kSf;
            // the first stages' weights go out before the digits are there: the launch that writes those began after
            // every earlier one's end, and this one began after it had
            struct { int slot, tile, ks; } held[kStages];
            int n_held = 0, loads = 0;
            bool waited = false;
            auto load_tokens = [&](int slot, int tile, int ks) {
                uint8_t *st = smem + slot * kStageBytes;
                tma_2d(st + 2 * kTile, &a.b, full + slot, ks * kRowBytes, tile * 128);
                bulk_copy(st + 3 * kTile + 2 * kSf, a.b_scales + (size_t)tile * a.atoms * 512 + (size_t)ks * kBSf, kBSf, full + slot);
            };
            auto release = [&]() {
                pdl_wait();
                waited = true;
#pragma unroll
                for (int i = 0; i < kStages; ++i)
                    if (i < n_held) load_tokens(held[i].slot, held[i].tile, held[i].ks);
            };
            for (int i = first; ok && i < items; i += step) {
                const Item it = item_at(a, i);
                const int r0 = it.group * 256;
                for (int ks = k0; ks < k1; ++ks) {
                    if (!waited && loads == kStages) release();
                    if (!mbar_wait(empty + s, ph ^ 1, err)) { ok = false; break; }
                    uint8_t *st = smem + s * kStageBytes;
                    mbar_expect_tx(full + s, 2 * kTile + b_bytes + 2 * kSf + kBSf);
                    tma_2d(st, &a.a, full + s, ks * kRowBytes, r0);
                    tma_2d(st + kTile, &a.a, full + s, ks * kRowBytes, r0 + 128);
                    const int sx = MX ? (ks >> 1) * 16 : ks * 16;
                    tma_2d(st + 3 * kTile, &a.sa, full + s, sx, r0);
                    tma_2d(st + 3 * kTile + kSf, &a.sa, full + s, sx, r0 + 128);
                    if (waited) load_tokens(s, it.tile, ks);
                    else {
#pragma unroll
                        for (int q = 0; q < kStages; ++q)
                            if (q == n_held) held[q] = {s, it.tile, ks};
                        ++n_held;
                    }
                    ++loads;
                    used |= 1u << s;
                    last_ph = (last_ph & ~(1u << s)) | (ph << s);
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
            }
            if (!waited) release();
            pdl_trigger();
            // every load has landed before the block ends (true already unless a wait ran out)
            for (int t = 0; t < kStages; ++t)
                if (used & (1u << t)) mbar_wait(full + t, (last_ph >> t) & 1u, err);
        }
    } else if (warp == 1) {
        // ------------------------------------------------ MMA issue
        if (lane == 0) {
            int s = 0;
            uint32_t ph = 0, aph = 0;
            bool ok = true;
            for (int i = first; ok && i < items; i += step) {
                if (!mbar_wait(acc_empty, aph ^ 1, err)) break;
                aph ^= 1;
                tc_fence_after();
                for (int ks = k0; ks < k1; ++ks) {
                    if (!mbar_wait(sf_ready + s, ph, err)) { ok = false; break; }   // covers full
                    tc_fence_after();
                    const uint32_t base = smem_u32(smem + s * kStageBytes);
                    const uint64_t dA = desc_sw128(base), dB = desc_sw128(base + 2 * kTile);
                    const uint32_t sf = tmem + kSfCol0 + s * kSfStride;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk) {
                        const uint32_t accum = ks > k0 || kk ? 1u : 0u;
                        mma_blk<MX>(tmem, dA + 2 * kk, dB + 2 * kk, a.rows, kk, sf, sf + 32, accum);
                        mma_blk<MX>(tmem + 128, dA + (kTile >> 4) + 2 * kk, dB + 2 * kk, a.rows, kk, sf + 16, sf + 32, accum);
                    }
                    mma_commit(empty + s);
                    if (++s == kStages) { s = 0; ph ^= 1; }
                }
                if (!ok) break;
                mma_commit(acc_full);
            }
            mma_commit(drain);
            mbar_wait(drain, 0, err);
        }
    } else if (warp < kEpiWarp0) {
        // ------------------------------------------------ scales -> tensor memory
        // Lane l of a 32-lane quadrant, column 4 c + j of a chunk of 64 (MXFP4: 128) values: the four scale bytes of row
        // l + 32 j.  The MMA takes weight row r's from its own lane r, so the warp of quadrant q loads rows 32 q + l and
        // writes each word to the chunk's four columns; the tokens' atoms hold the columns as they are.
        const int quad = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(quad * 32) << 16) + kSfCol0;
        int s = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int i = first; ok && i < items; i += step) {
            for (int ks = k0; ks < k1; ++ks) {
                if (!mbar_wait(full + s, ph, err)) { ok = false; break; }
                tc_fence_after();
                const uint32_t from = smem_u32(smem + s * kStageBytes + 3 * kTile);
                uint32_t o[16];
#pragma unroll
                for (int op = 0; op < 2; ++op) {
                    const uint4 v = lds128(from + op * kSf + 16 * (lane + 32 * quad));
                    // MXFP4: a row's 16 bytes cover a pair of stages
                    const uint32_t c0 = (MX && (ks & 1)) ? v.z : v.x, c1 = (MX && (ks & 1)) ? v.w : v.y;
                    const uint32_t c2 = MX ? 0u : v.z, c3 = MX ? 0u : v.w;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        o[j] = c0;
                        o[4 + j] = c1;
                        o[8 + j] = c2;
                        o[12 + j] = c3;
                    }
                    tmem_st16(t_lane + s * kSfStride + 16 * op, o);
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const uint4 v = MX && c >= 2 ? make_uint4(0u, 0u, 0u, 0u) : lds128(from + 2 * kSf + 512 * c + 16 * lane);
                    o[4 * c] = v.x;
                    o[4 * c + 1] = v.y;
                    o[4 * c + 2] = v.z;
                    o[4 * c + 3] = v.w;
                }
                tmem_st16(t_lane + s * kSfStride + 32, o);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sf_ready + s);
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
        }
        mbar_wait(drain, 0, err);
    } else {
        // ------------------------------------------------ epilogue
        // A thread has one row of each accumulator and the 64 columns of eight tokens.
        const int quad = warp & 3, half = (warp - kEpiWarp0) >> 2;
        const uint32_t lane_base = tmem + ((uint32_t)(quad * 32) << 16) + 64 * half;
        const bool busy = 64 * half < a.rows;
        uint32_t aph = 0, turn = 0;
        bool ok = true;
        float ts = 1.0f;
        pdl_wait();
        int power = 0;                     // the tensor scale's
        if (a.ts) {
            const TensorScale split = split_scale(*a.ts);
            power = split.power;
            ts = split.rest;
        }
        for (int i = first; i < items; i += step) {
            const Item it = item_at(a, i);
            const int t0 = it.tile * kTileTokens + 8 * half, tokens = busy ? min(8, a.T - t0) : 0;
            const int n0 = it.group * 256 + quad * 32 + lane;
            int2 info = make_int2(0, 0);                           // lane j: token j's
            if (lane < tokens) info = a.info[t0 + lane];
            const float own_first = first_factor(info.x + power), own_second = second_factor(info.x + power);   // MXFP4: one is enough
            if (ok) ok = mbar_wait(acc_full, aph, err);
            aph ^= 1;
            tc_fence_after();
            float sum[2][8];
            if (busy) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        float v[16];
                        if (64 * half + 16 * c < a.rows) tmem_ld16_nowait(lane_base + 128 * h + 16 * c, v);
                        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const float *u = v + 8 * q;
                            float all = u[7];
#pragma unroll
                            for (int d = 6; d >= 0; --d) all = MX ? all + u[d] : fmaf(all, 0.125f, u[d]);
                            sum[h][2 * c + q] = all;
                        }
                    }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float first = __shfl_sync(0xffffffffu, own_first, j), second = MX ? 1.0f : __shfl_sync(0xffffffffu, own_second, j);
                const bool bad = __shfl_sync(0xffffffffu, info.y, j) != 0;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h][j] = ok ? sum[h][j] * first * second : NAN;
                    if (bad && j < tokens && n0 + 128 * h < a.N)
                        sum[h][j] += beyond<MX>(a, t0 + j, n0 + 128 * h, k0 * kBK, k1 * kBK);
                }
            }
            const int64_t at = (int64_t)t0 * a.N + n0;
            if (a.parts == 1) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (j < tokens && n0 + 128 * h < a.N) store_out(a, at + (int64_t)j * a.N + 128 * h, sum[h][j] * ts);
            } else {
                float *to = a.partial + (int64_t)part * a.T * a.N + at;
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (j < tokens && n0 + 128 * h < a.N) __stcg(to + (int64_t)j * a.N + 128 * h, sum[h][j]);
                asm volatile("bar.sync 1, 256;" ::: "memory");
                const int tid = threadIdx.x - 32 * kEpiWarp0;
                if (tid < a.parts) {
                    __threadfence();
                    arrive_at(joined + (turn & 1), tid);
                }
                if (!mbar_wait_cluster(joined + (turn & 1), turn >> 1 & 1, err)) ok = false;
                ++turn;
                // this block's rows of the 256 (parts is a power of two): element e is row e % rows of token e / rows, sixteen loads a thread
                const int lp = 31 - __clz(a.parts), rows = 256 >> lp, all = min(kTileTokens, a.T - it.tile * kTileTokens);
                const float *from = a.partial + (int64_t)it.tile * kTileTokens * a.N;
                const int64_t apart = (int64_t)a.T * a.N;
                float v[16];
#pragma unroll
                for (int f = 0; f < 16; ++f) {
                    const int e = tid + 256 * (f >> lp), tok = e >> (8 - lp), n = it.group * 256 + part * rows + (e & (rows - 1));
                    v[f] = tok < all && n < a.N ? __ldcg(from + (f & (a.parts - 1)) * apart + (int64_t)tok * a.N + n) : 0.0f;
                }
                float s = 0.0f;
#pragma unroll
                for (int f = 0; f < 16; ++f) {
                    s += v[f];
                    if ((f + 1) & (a.parts - 1)) continue;
                    const int e = tid + 256 * (f >> lp), tok = e >> (8 - lp), n = it.group * 256 + part * rows + (e & (rows - 1));
                    if (tok < all && n < a.N) store_out(a, (int64_t)(it.tile * kTileTokens + tok) * a.N + n, ok ? s * ts : NAN);
                    s = 0.0f;
                }
            }
        }
    }
    tc_fence_before();
    if (a.parts > 1) cluster_sync();           // no block leaves while another may arrive at its barrier
    else __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

// ------------------------------------------------------------ host side

// Clusters of as many blocks that fit on the GPU at once, as it reports.
int clusters_of(int blocks) { return blocks == 1 ? kSms : blocks == 2 ? 76 : blocks == 4 ? 36 : 15; }

Layout layout_of(bool mx, int T, int N, int K) {
    Layout l{};
    l.tiles = blocks_of(T, kTileTokens);
    l.groups = blocks_of(N, 256);
    l.stages = K / kBK;
    l.atoms = K / (mx ? 128 : 64);
    // parts of K, one to eight by powers of two: the fewest rounds of stages, with about two stages of filling an item and
    // two of joining it
    const int64_t items = (int64_t)l.tiles * l.groups;
    int64_t best = INT64_MAX;
    for (int p = 1; p <= std::min(l.stages, kMaxParts); p *= 2) {
        const int64_t at_once = clusters_of(p);
        const int64_t cost = (items + at_once - 1) / at_once * (blocks_of(l.stages, p) + (p > 1 ? 4 : 2));
        if (cost < best) {
            best = cost;
            l.parts = p;
        }
    }
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t from = at;
        at += (n + 255) / 256 * 256;
        return from;
    };
    l.codes = take((size_t)l.tiles * 128 * (K / 2));
    l.scales = take((size_t)l.tiles * l.atoms * 512);
    l.info = take((size_t)T * sizeof(int2));
    l.partial = take(l.parts > 1 ? (size_t)l.parts * T * N * sizeof(float) : 0);
    l.bytes = at;
    return l;
}

template <bool MX> cudaError_t launch_chunk(const LinearCall &c, cudaStream_t st) {
    const Layout l = layout_of(MX, c.T, c.N, c.K);
    uint8_t *ws = static_cast<uint8_t *>(c.workspace);
    DigitArgs t{};
    t.x = c.x;
    t.x_stride = c.x_stride;
    t.codes = ws + l.codes;
    t.scales = ws + l.scales;
    t.info = reinterpret_cast<int2 *>(ws + l.info);
    t.T = c.T;
    t.K = c.K;
    t.bf16 = c.dtype == MOE_DTYPE_BF16;
    t.atoms = l.atoms;
    TcArgs a{};
    a.rows = kDigits * (c.T <= 4 ? 4 : c.T <= 8 ? 8 : 16);
    constexpr int G = MX ? 32 : 16;
    if (!make_map(&a.a, c.codes, c.K / 2, c.N, c.K / 2, kRowBytes, 128, true) ||
        !make_map(&a.sa, c.scales, c.K / G, c.N, c.K / G, 16, 128, false) ||
        !make_map(&a.b, t.codes, c.K / 2, (uint64_t)l.tiles * 128, c.K / 2, kRowBytes, a.rows, true))
        return cudaErrorInvalidValue;
    cudaError_t e = allow_smem<k_linear_tc<MX>>();
    if (e != cudaSuccess) return e;
    e = launch_pdl(k_linear_digits<MX>, dim3(blocks_of(c.K, 1024), c.T), dim3(128), 0, st, t);
    if (e != cudaSuccess) return e;
    a.codes = c.codes;
    a.scales = c.scales;
    a.ts = c.ts;
    a.b_scales = t.scales;
    a.x = c.x;
    a.x_stride = c.x_stride;
    a.out = c.out;
    a.partial = reinterpret_cast<float *>(ws + l.partial);
    a.info = t.info;
    a.T = c.T;
    a.N = c.N;
    a.K = c.K;
    a.bf16 = t.bf16;
    a.dtype = c.out_dtype;
    a.tiles = l.tiles;
    a.groups = l.groups;
    a.parts = l.parts;
    a.stages = l.stages;
    a.atoms = l.atoms;
    cudaLaunchConfig_t cfg = {};
    // as few clusters as take the items in that many rounds: an SM that is free early takes the next launch's blocks
    const int64_t items = (int64_t)l.tiles * l.groups, at_once = clusters_of(l.parts), rounds = (items + at_once - 1) / at_once;
    cfg.gridDim = dim3(l.parts * (unsigned)((items + rounds - 1) / rounds));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = l.parts;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = l.parts > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k_linear_tc<MX>, a);
}

}  // namespace

namespace moe {

size_t linear_tc_workspace(bool mx, bool f16, int T, int N, int K) {
    // a stage is 256 values, and TMA wants rows of scales in whole 16 bytes
    if (T < 1 || N < 1 || K < 1 || K % (mx ? 512 : 256)) return 0;
    // What the two launches, the filling and the joining cost, 8 us, has to come back from the products.  The warp MMAs take
    // f16 rows as they are and bf16 ones behind a pass over them, so f16 rows want more work.  In graphs, us, warp MMAs against
    // here (which is the same for both types, and 0 to 3 % faster for MXFP4):
    //   tokens, weight        NVFP4 bf16   f16          MXFP4 bf16   f16
    //   1   16384 x 8192      20.3 22.8    18.7 22.8    18.4 22.3    16.8 22.3
    //   1   32768 x 8192      33.4 32.5    32.0 32.7    29.8 32.0    28.2 31.8
    //   1   100003 x 4096     49.5 42.4    48.8 42.3    43.6 40.5    42.9 40.5
    //   8   32768 x 8192      35.2 33.6    34.4 33.4    31.8 32.1    30.3 32.1
    //   16  4096 x 4096       9.8  12.7    7.8  12.7    9.6  12.7    7.5  12.7
    //   16  8192 x 4096       13.8 13.8    11.8 13.9    13.5 13.8    11.6 13.8
    //   16  8192 x 8192       20.8 18.1    17.7 18.1    20.8 17.8    18.0 17.8
    //   16  16384 x 7168      27.7 22.4    25.0 22.4    27.7 21.9    25.7 21.8
    //   17  4096 x 4096       13.6 13.0    9.1  13.0    14.2 13.0    9.7  13.0
    //   32  8192 x 4096       20.7 15.1    16.8 15.1    21.5 15.1    18.1 15.0
    //   32  11000 x 4096      23.7 15.3    19.8 15.3    24.8 15.3    21.4 15.2
    //   64  2048 x 4096       14.0 15.5    9.7  15.6    14.7 15.5    10.3 15.5
    //   64  7168 x 2048       17.1 11.7    14.8 11.7    18.3 11.7    16.1 11.7
    //   64  5800 x 4096       23.2 15.8    19.2 15.8    24.4 15.7    20.8 15.8
    // A call that no graph holds takes the host 4 us more than the other form's (two launches, three tensor maps, the
    // workspace): where the GPU is faster than the host, bf16 rows between the rule's borders and about twice the work lose them.
    const int64_t work = (int64_t)N * K * (T <= 16 ? 1 : blocks_of(T, 32));
    const int64_t least = T <= 8 ? (f16 && mx ? (int64_t)3 << 27 : (int64_t)1 << 28) : T <= 16 ? (f16 ? 3 << 25 : 1 << 25) : (f16 ? 5 << 23 : 1 << 24);
    if (work < least) return 0;
    size_t n = layout_of(mx, std::min(T, kChunkTokens), N, K).bytes;
    if (T % kChunkTokens) n = std::max(n, layout_of(mx, T % kChunkTokens, N, K).bytes);   // may have more parts
    return n;
}

cudaError_t launch_linear_tc(const LinearCall &call, cudaStream_t st) {
    LinearCall c = call;
    const size_t row = (size_t)call.N * (call.out_dtype == MOE_DTYPE_F32 ? 4 : 2);
    for (int t = 0; t < call.T; t += kChunkTokens) {
        c.T = std::min(kChunkTokens, call.T - t);
        c.x = static_cast<const uint16_t *>(call.x) + t * call.x_stride;
        c.out = static_cast<uint8_t *>(call.out) + t * row;
        const cudaError_t e = call.ts ? launch_chunk<false>(c, st) : launch_chunk<true>(c, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace moe
