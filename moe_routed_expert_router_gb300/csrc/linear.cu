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
// bf16 tokens become f16, times a power of two that brings the largest finite
// magnitude of a token's 256 values to [2^7, 2^8): a bf16 value is exact in f16
// down to 2^-17, and what is smaller is off by at most 2^-25, that is 2^-32 of the
// largest.  The power is taken back from the sum; with MXFP4 up to 2^20 of it, where the token was made larger, together
// with the scale of each 32 values: a sum of 256 values is below 2^19 and a scale at most 2^127, so nothing passes fp32
// that the result itself does not.  (What is left of the power is kept as a pair of bf16: as two floats it spilled at eight
// tokens, 1 x 16384 x 7168 MXFP4 17.6 us against 17.1.)
//
// One block an SM takes an even share of the weight's rows, so all SMs read
// equally much.  Its warps share K in stages of 256 values: a warp holds a stage's
// tokens in registers (turned into f16 there) and runs down the block's rows, 16 at
// a time, with a cp.async ring of its own, so that neither tokens nor weights pass
// between warps and no barrier stops the stream.  The warps' sums of a pass over
// the rows are joined in shared memory in a fixed order.  (Tokens in shared memory,
// whole or in chunks with a barrier each: 31 to 41 us against 27 at 16 x 16384 x 7168,
// before linear_tc.cu had that size.)
//
// Measured in graphs, us (share of the copy bandwidth): 4 x 4096 x 4096 NVFP4 bf16 6.3, f16 5.6, MXFP4 bf16 6.2, f16 5.3; 1 x
// 16384 x 7168 18.9 (0.52), 17.3, 17.1 (0.55), 15.6; 1 x 32760 x 8192 33.4 (0.67), 32.0, 29.8 (0.71), 28.3; 16 x 4096 x 4096
// 9.8, 7.8, 9.6, 7.5.  With all data in shared memory a sub-partition needs 39 cycles for 16 rows x 32 values and eight tokens
// (the eight code conversions 23 of them, the two MMAs 21 beside them; codes widened by shifts and masks instead 44), 16 us of
// the 33 that 1 x 32760 x 8192 takes: four warps do not hide each other's chains of load, conversion, product and MMA.  Each
// eight tokens more add two MMAs, so from 16 tokens on the warp MMAs are the limit, not the bytes: large products go to
// linear_tc.cu.
#include "linear.cuh"
#include "linear_split.cuh"

namespace {

using namespace moe;

template <int NT> constexpr int kStageK = linear_stage_k(NT);
template <int NT> constexpr int kWarps = linear_warps(NT);
template <int NT> constexpr int kStageBytes = linear_stage_bytes(NT);
constexpr int kRows = kLinearRows;
constexpr int kMaxK = 1 << 16, kMaxTokens = 1 << 20;
constexpr int kScaleShift = 20;            // MXFP4: how much of a token's power goes back together with the scales

struct LinearArgs : LinearSplit {
    const uint8_t *codes, *scales;
    const float *ts;                       // tensor scale or null
    const void *x;                         // [T] rows, x_stride values apart
    int64_t x_stride;
    void *out;
    int T, N, K, dtype;                    // out's type
    int bf16;                              // x's type
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Two scales of a word each: E4M3 bytes (a, a, b, b) as f16 pairs (a, a) and (b, b); E8M0 bytes (a, b, ., .) as the
// bf16 pair (a, b), exact: 2^-127 is one of its subnormals and byte 255 a NaN.
__device__ __forceinline__ void scales_e4m3(uint32_t w, uint32_t &first, uint32_t &second) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(first), "=r"(second) : "r"(w));
}
__device__ __forceinline__ void scales_e8m0(uint32_t w, uint32_t &first, uint32_t &second) {
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.bf16x2.ue8m0x2 %0, l;\n\tcvt.rn.bf16x2.ue8m0x2 %1, h;\n\t}"
        : "=r"(first), "=r"(second) : "r"(w));
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

// Largest magnitude of bf16 values, NaNs aside: pairs, then the larger of the two.
__device__ __forceinline__ uint32_t amax_pair(uint32_t m, uint32_t pair) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(m), "r"(pair & 0x7FFF7FFFu));
    return r;
}
__device__ __forceinline__ uint32_t amax8(const uint4 &p, uint32_t m) { return amax_pair(amax_pair(m, p.x), amax_pair(amax_pair(amax_pair(0u, p.y), p.z), p.w)); }
__device__ __forceinline__ float amax_of(uint32_t m) { return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)); }
// The same of the finite ones, where an infinity is among them.
__device__ __noinline__ float finite_amax8(uint4 p, float m) {
    const uint32_t u[4] = {p.x, p.y, p.z, p.w};
    for (int i = 0; i < 8; ++i) {
        const float v = fabsf(__uint_as_float(i & 1 ? u[i >> 1] & 0xFFFF0000u : u[i >> 1] << 16));
        if (v < INFINITY) m = fmaxf(m, v);
    }
    return m;
}
__device__ __forceinline__ uint4 scaled8(const uint4 &piece, float up, float more) {
    float v[8];
    widen8<MOE_DTYPE_BF16>(Raw8<MOE_DTYPE_BF16>{piece}, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) mul2(v, i, up, up);
    if (more != 1.0f) {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= more;
    }
    return narrow8<MOE_DTYPE_F16>(v).a;
}

// The warps that share a group's K wait for one another.
__device__ __forceinline__ void group_sync(int group, int warps) {
    if (warps == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(32 * warps) : "memory");
}

template <bool MX, int NT>
__global__ void __launch_bounds__(32 * kWarps<NT>, 1) k_linear(LinearArgs a) {
    constexpr int SK = kStageK<NT>;
    constexpr int kUnits = SK / 32, kCodePitch = SK / 2 + kCodePad, kStage = kStageBytes<NT>;   // a unit: 32 values of K
    constexpr int kChains = MX || NT == 4 ? 1 : 2;                  // of dependent MMAs a token group (MXFP4's are two long)
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int wm = warp / a.wk, wk = warp - wm * a.wk;
    const int token0 = blockIdx.y * (8 * NT), tokens = min(8 * NT, a.T - token0);
    const RowRange rows_here = linear_block_rows(a, blockIdx.x);
    uint8_t *ring = smem + warp * a.ring * kStage;
    float4 *red = reinterpret_cast<float4 *>(smem + a.wk * a.wm * a.ring * kStage);   // [warp][tile][NT][lane]
    const int stages = (a.K + SK - 1) / SK;
    const int64_t code_row = a.K / 2, scale_row = a.K / (MX ? 32 : 16);

    // The stream of this warp: pass, stage, tile.  A lane copies one 16-byte unit of every kLoadRows-th row and a piece of
    // a row's scales; rows that are not there are left out, for no result that is stored uses them.
    constexpr int kLoadRows = 32 / kUnits, kScalePiece = MX ? 4 : 8, kPieces = kUnits / 4;
    const int load_row = lane / kUnits, load_unit = lane % kUnits, scale_lane_row = lane / kPieces, scale_piece = lane % kPieces;
    const bool last_half = a.K % SK != 0;  // of the last stage
    const int64_t code_step = kLoadRows * code_row;
    int lp = 0, ls = wk, lj = 0, fill = 0, left = 0;                         // rows left in the warp's share of the pass
    const uint8_t *code_at = nullptr, *scale_at = nullptr;
    auto stream_at = [&]() {               // the first tile of pass lp and stage ls
        if (lp == a.passes) return;
        const RowRange pass = linear_pass_rows(a, rows_here, lp);
        const int n0 = linear_tile_rows(a, pass, wm * a.tiles).first;
        left = pass.end - n0;
        code_at = a.codes + (n0 + load_row) * code_row + ls * (SK / 2) + 16 * load_unit;
        scale_at = a.scales + (n0 + scale_lane_row) * scale_row + ls * (kPieces * kScalePiece) + scale_piece * kScalePiece;
    };
    auto load_next = [&]() {
        if (lp < a.passes) {
            uint8_t *to = ring + fill * kStage;
            uint8_t *code_to = to + load_row * kCodePitch + 16 * load_unit;
            uint8_t *scale_to = to + kRows * kCodePitch + scale_lane_row * kScaleBytes + scale_piece * kScalePiece;
            const int here = min(left, a.tile_rows), rows = here - load_row, scale_rows = scale_lane_row < kRows ? here - scale_lane_row : 0;
            if (last_half && ls == stages - 1) {                             // zeros behind K
                const bool code_on = load_unit < kUnits / 2, scale_on = scale_piece == 0;
#pragma unroll
                for (int i = 0; i < kRows / kLoadRows; ++i)
                    if (i * kLoadRows < rows) copy16(code_to + i * kLoadRows * kCodePitch, code_on ? code_at + i * code_step : a.codes, code_on);
                if (scale_rows > 0) copy_small<kScalePiece>(scale_to, scale_on ? scale_at : a.scales, scale_on);
            } else {
                const uint8_t *at = code_at;
#pragma unroll
                for (int i = 0; i < kRows / kLoadRows; ++i, at += code_step)
                    if (i * kLoadRows < rows) copy16(code_to + i * kLoadRows * kCodePitch, at, true);
                if (scale_rows > 0) copy_small<kScalePiece>(scale_to, scale_at, true);
            }
            if (++lj < a.tiles) {
                left -= a.tile_rows;
                code_at += a.tile_rows * code_row;
                scale_at += a.tile_rows * scale_row;
            } else {
                lj = 0;
                ls += a.wk;
                if (ls >= stages) {
                    ls = wk;
                    ++lp;
                }
                stream_at();
            }
        }
        copy_commit();
        if (++fill == a.ring) fill = 0;
    };
    auto wait_oldest = [&]() {             // all but the ring - 1 latest stages are there
        switch (a.ring) {
            case 2: copy_wait<1>(); break;
            case 3: copy_wait<2>(); break;
            case 4: copy_wait<3>(); break;
            case 5: copy_wait<4>(); break;
            default: copy_wait<kMostLinearRing - 1>(); break;
        }
        __syncwarp();
    };

    // A stage's tokens: unit u's values 8 t .. 8 t + 7 of token 8 n + g (a column without one takes the last: its sums are
    // not stored), and the scales of the sums' columns 2 t and 2 t + 1.
    uint4 x[NT][kUnits];
    // Of the power that gives a sum its size back, two factors: `undo`, which MXFP4 has with the scales, and what is left of it,
    // a pair of bf16 powers, with the sum.  NVFP4's bf16 tokens have the tensor scale's power in it too.
    float undo[NT][2], ts = 1.0f;
    uint32_t rest[NT];
    int more_power = 0;
    auto take_tokens = [&](int stage) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const uint16_t *row = static_cast<const uint16_t *>(a.x) + (token0 + min(8 * n + g, tokens - 1)) * a.x_stride + stage * SK + 8 * t;
#pragma unroll
            for (int u = 0; u < kUnits; ++u) x[n][u] = stage * SK + 32 * u < a.K ? ld16_shared(row + 32 * u) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            undo[n][0] = undo[n][1] = 1.0f;
            rest[n] = 0x3F803F80u;
            if (a.bf16) {
                uint32_t pairs = 0u;
#pragma unroll
                for (int u = 0; u < kUnits; ++u) pairs = amax8(x[n][u], pairs);
                float m = amax_of(pairs);
                if (m == INFINITY) {
                    m = 0.0f;
#pragma unroll
                    for (int u = 0; u < kUnits; ++u) m = finite_amax8(x[n][u], m);
                }
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
                const int e = exponent_of(m);
                const float up = scale_up(e), more = scale_more(e);
#pragma unroll
                for (int u = 0; u < kUnits; ++u) x[n][u] = scaled8(x[n][u], up, more);
                const int power = e - 7 + more_power, with_scale = max(-kScaleShift, min(0, power));
                const float first = MX ? power_of_two(with_scale) : first_factor(power);
                undo[n][0] = __shfl_sync(0xffffffffu, first, 8 * t);
                undo[n][1] = __shfl_sync(0xffffffffu, first, 8 * t + 4);
                const uint32_t second = __float_as_uint(MX ? power_of_two(power - with_scale) : second_factor(power));
                rest[n] = __shfl_sync(0xffffffffu, second, 8 * t) >> 16 | __shfl_sync(0xffffffffu, second, 8 * t + 4);
            }
        }
    };

    stream_at();
    pdl_wait();
    for (int i = 0; i < a.ring - 1; ++i) load_next();
    pdl_trigger();
    if (a.ts) ts = *a.ts;
    if (!MX && a.bf16) {
        const TensorScale split = split_scale(ts);
        more_power = split.power;
        ts = split.rest;
    }
    take_tokens(wk);
    const uint32_t scale_bytes = t >> 1 ? 0x3311 : 0x2200;
    float4 *mine = red + warp * a.tiles * (NT * 32) + lane;
    const bool one_stage = wk + a.wk >= stages;
    int slot = 0;
    for (int pass = 0; pass < a.passes; ++pass) {
        for (int stage = wk; stage < stages; stage += a.wk) {
            if (!one_stage && (pass > 0 || stage > wk)) take_tokens(stage);
            for (int j = 0; j < a.tiles; ++j) {
                load_next();
                wait_oldest();
                const uint8_t *from = ring + slot * kStage;
                if (++slot == a.ring) slot = 0;
                float acc[NT][kChains][4] = {};
                // the stage's scales of rows g and g + 8: per two units a word of E4M3 bytes, or a pair of bf16 values
                uint32_t sc[2][kUnits / 2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint8_t *p = from + kRows * kCodePitch + (8 * h + g) * kScaleBytes;
                    uint32_t raw[4];
                    if constexpr (MX && kUnits == 4) raw[0] = *reinterpret_cast<const uint32_t *>(p);
                    else if constexpr (MX || kUnits == 4) *reinterpret_cast<uint2 *>(raw) = *reinterpret_cast<const uint2 *>(p);
                    else *reinterpret_cast<uint4 *>(raw) = *reinterpret_cast<const uint4 *>(p);
                    if constexpr (MX) {
#pragma unroll
                        for (int i = 0; i < kUnits / 4; ++i) scales_e8m0(raw[i], sc[h][2 * i], sc[h][2 * i + 1]);
                    } else {
#pragma unroll
                        for (int i = 0; i < kUnits / 2; ++i) sc[h][i] = raw[i];
                    }
                }
                const uint8_t *codes = from + g * kCodePitch + 4 * t;
#pragma unroll
                for (int p = 0; p < kUnits / 2; ++p) { // two units
                    uint32_t w[2][2][4];               // [unit][row half]
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t s[2];
                        // the scale of values 8 t .. 8 t + 7 of a unit: byte t >> 1 of its two, twice
                        if constexpr (!MX) scales_e4m3(__byte_perm(sc[h][p], 0, scale_bytes), s[0], s[1]);
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            e2m1x8_to_f16x8(lds32(codes + 8 * h * kCodePitch + 16 * (2 * p + v)), w[v][h]);
                            if constexpr (!MX) {
#pragma unroll
                                for (int i = 0; i < 4; ++i) w[v][h][i] = hmul2(w[v][h][i], s[v]);
                            }
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const uint4 &b = x[n][2 * p + v];
                            if constexpr (MX) {
                                float d[4];
                                mma16816_zero(d, w[v][0][0], w[v][1][0], w[v][0][1], w[v][1][1], b.x, b.y);
                                mma16816(d, w[v][0][2], w[v][1][2], w[v][0][3], w[v][1][3], b.z, b.w);
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    const float s = __uint_as_float(v ? sc[h][p] & 0xFFFF0000u : sc[h][p] << 16);
                                    float f[2] = {undo[n][0], undo[n][1]};
                                    mul2(f, 0, s, s);
                                    acc[n][0][2 * h] = fmaf(d[2 * h], f[0], acc[n][0][2 * h]);
                                    acc[n][0][2 * h + 1] = fmaf(d[2 * h + 1], f[1], acc[n][0][2 * h + 1]);
                                }
                            } else {
                                mma16816(acc[n][v % kChains], w[v][0][0], w[v][1][0], w[v][0][1], w[v][1][1], b.x, b.y);
                                mma16816(acc[n][v % kChains], w[v][0][2], w[v][1][2], w[v][0][3], w[v][1][3], b.z, b.w);
                            }
                        }
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float4 *at = mine + (j * NT + n) * 32;
                    float4 s = stage > wk ? *at : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int c = 1; c < kChains; ++c)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][0][i] += acc[n][c][i];
                    const float u0 = __uint_as_float(rest[n] << 16), u1 = __uint_as_float(rest[n] & 0xFFFF0000u);
                    if constexpr (!MX) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[n][0][i] *= undo[n][i & 1];
                    }
                    s.x = fmaf(acc[n][0][0], u0, s.x);
                    s.y = fmaf(acc[n][0][1], u1, s.y);
                    s.z = fmaf(acc[n][0][2], u0, s.z);
                    s.w = fmaf(acc[n][0][3], u1, s.w);
                    *at = s;
                }
                __syncwarp();
            }
        }
        // join the sums of the group's warps in order
        group_sync(wm, a.wk);
        const RowRange there = linear_pass_rows(a, rows_here, pass);
        const float *all = reinterpret_cast<const float *>(red + wm * a.wk * a.tiles * (NT * 32));
        for (int i = wk * 32 + lane; i < a.tiles * kRows * tokens; i += 32 * a.wk) {
            const int row = i % kRows, tok = i / kRows % tokens, j = i / kRows / tokens;
            const RowRange tile = linear_tile_rows(a, there, wm * a.tiles + j);
            if (tile.first + row >= tile.end) continue;
            const float *p = all + ((j * NT + (tok >> 3)) * 32 + (row & 7) * 4 + ((tok & 7) >> 1)) * 4 + (row >> 3) * 2 + (tok & 1);
            float s = 0.0f;
#pragma unroll 4
            for (int w = 0; w < a.wk; ++w) s += p[w * a.tiles * (NT * 128)];
            s *= ts;
            const int64_t at = (int64_t)(token0 + tok) * a.N + tile.first + row;
            if (a.dtype == MOE_DTYPE_F32) static_cast<float *>(a.out)[at] = s;
            else if (a.dtype == MOE_DTYPE_BF16) static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(s);
            else static_cast<__half *>(a.out)[at] = __float2half_rn(s);
        }
        if (pass + 1 < a.passes) group_sync(wm, a.wk);
    }
}

// ------------------------------------------------------------ host side

template <bool MX, int NT> cudaError_t launch(LinearArgs a, cudaStream_t st) {
    const cudaError_t e = allow_smem<k_linear<MX, NT>>();
    if (e != cudaSuccess) return e;
    static_cast<LinearSplit &>(a) = linear_split(NT, a.T, a.N, a.K);
    return launch_pdl(k_linear<MX, NT>, dim3(a.blocks, a.groups), dim3(32 * a.wk * a.wm), a.smem, st, a);
}

template <bool MX> cudaError_t launch_format(const LinearArgs &a, cudaStream_t st) {
    switch (linear_tokens(a.T)) {
        case 1: return launch<MX, 1>(a, st);
        case 2: return launch<MX, 2>(a, st);
        default: return launch<MX, 4>(a, st);
    }
}

moe_status cuda_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

extern "C" {

size_t moe_linear_fp4_workspace_for(int32_t weight_format, int32_t dtype, int32_t T, int32_t N, int32_t K) {
    if (T < 1 || T > kMaxTokens || N < 1 || N > INT32_MAX - 1024 || K < 128 || K > kMaxK || K % 128) return 0;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return 0;
    return linear_tc_workspace(weight_format == MOE_WEIGHTS_MXFP4, dtype == MOE_DTYPE_F16, T, N, K);
}

size_t moe_linear_fp4_workspace(int32_t weight_format, int32_t T, int32_t N, int32_t K) {
    return std::max(moe_linear_fp4_workspace_for(weight_format, MOE_DTYPE_BF16, T, N, K),
                    moe_linear_fp4_workspace_for(weight_format, MOE_DTYPE_F16, T, N, K));
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
    const size_t ws = linear_tc_workspace(mx, dtype == MOE_DTYPE_F16, T, N, K);
    if (!x || !out || !weight->codes || !weight->scales || (!mx && !weight->tensor_scale) || (ws && !workspace) || workspace_bytes < ws)
        return MOE_ERR_INVALID_ARG;
    if (!aligned_to(x, 16) || !aligned_to(weight->codes, 16) || !aligned_to(weight->scales, 16) ||
        !aligned_to(mx ? nullptr : weight->tensor_scale, 4) || !aligned_to(out, out_dtype == MOE_DTYPE_F32 ? 4 : 2) ||
        (ws && !aligned_to(workspace, 256)))
        return MOE_ERR_MISALIGNED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ws) {
        const LinearCall c{x, x_stride, weight->codes, weight->scales, mx ? nullptr : weight->tensor_scale, T, N, K, dtype, out_dtype, out, workspace};
        return cuda_status(launch_linear_tc(c, s));
    }
    LinearArgs a{};
    a.codes = weight->codes;
    a.scales = weight->scales;
    a.ts = mx ? nullptr : weight->tensor_scale;
    a.x = x;
    a.x_stride = x_stride;
    a.out = out;
    a.T = T;
    a.N = N;
    a.K = K;
    a.dtype = out_dtype;
    a.bf16 = dtype == MOE_DTYPE_BF16;
    return cuda_status(mx ? launch_format<true>(a, s) : launch_format<false>(a, s));
}

}  // extern "C"
