// Rows of activations in 16-byte pieces, shared by the norm and the
// dispatch / combine kernels: eight values at a time, widened to fp32.
#pragma once

#include <mutex>

#include "card.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr int kChunk = 8;   // values a thread moves at once

template <int DT> struct RowType;
template <> struct RowType<MOE_DTYPE_F32> { using T = float; };
template <> struct RowType<MOE_DTYPE_BF16> { using T = __nv_bfloat16; };
template <> struct RowType<MOE_DTYPE_F16> { using T = __half; };

// Eight values as they are stored.
template <int DT> struct Raw8 { uint4 a; };
template <> struct Raw8<MOE_DTYPE_F32> { uint4 a, b; };

// Loads and stores of data touched once: no L1 allocation.  The loads are not
// the read-only kind, because an output may be an input's own memory.
__device__ __forceinline__ uint4 ld16(const void *p) {
    uint4 r;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
__device__ __forceinline__ void st16(void *p, uint4 v) {
    asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};"
                 ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 16 bytes from global into shared memory without registers (cp.async); a
// thread's copies since the last commit form a group.
// `on` false: zeros, and `src` (any valid address) is not read.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of the thread's latest groups are unfinished.
template <int N> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

template <int DT> __device__ __forceinline__ Raw8<DT> load8(const typename RowType<DT>::T *p) {
    Raw8<DT> r;
    r.a = ld16(p);
    if constexpr (DT == MOE_DTYPE_F32) r.b = ld16(p + 4);
    return r;
}

// Eight values from shared memory, `n` words apart where they take two.
template <int DT> __device__ __forceinline__ Raw8<DT> take8(const uint4 *at, int n) {
    Raw8<DT> v;
    v.a = at[0];
    if constexpr (DT == MOE_DTYPE_F32) v.b = at[n];
    return v;
}

// The same of a row that other blocks read too (a weight): kept in L1.  Not the
// read-only kind either: with dependent launches the kernel before may still be
// writing when this one's first blocks start.
__device__ __forceinline__ uint4 ld16_shared(const void *p) {
    uint4 r;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
    return r;
}
template <int DT> __device__ __forceinline__ Raw8<DT> load8_shared(const typename RowType<DT>::T *p) {
    Raw8<DT> r;
    r.a = ld16_shared(p);
    if constexpr (DT == MOE_DTYPE_F32) r.b = ld16_shared(p + 4);
    return r;
}

template <int DT> __device__ __forceinline__ void store8(typename RowType<DT>::T *p, const Raw8<DT> &r) {
    st16(p, r.a);
    if constexpr (DT == MOE_DTYPE_F32) st16(p + 4, r.b);
}

// Two fp32 operations in one instruction (f32x2), each rounded as the scalar
// one is: a *= b;  c += a * b.
template <int N> __device__ __forceinline__ void mul2(float (&a)[N], int i, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%0, %1};\n\tmov.b64 y, {%2, %3};\n\tmul.rn.f32x2 x, x, y;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(a[i]), "+f"(a[i + 1]) : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float &c0, float &c1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
        "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
        : "+f"(c0), "+f"(c1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

template <int DT> __device__ __forceinline__ void widen8(const Raw8<DT> &r, float (&v)[8]) {
    const uint32_t u[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    if constexpr (DT == MOE_DTYPE_F32) {
        const uint32_t w[4] = {r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = __uint_as_float(u[i]);
            v[4 + i] = __uint_as_float(w[i]);
        }
    } else if constexpr (DT == MOE_DTYPE_BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(u[i] << 16);
            v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = f16x2_to_f32x2(u[i]);
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
}

// Round to nearest even into the stored type.
template <int DT> __device__ __forceinline__ Raw8<DT> narrow8(const float (&v)[8]) {
    Raw8<DT> r;
    if constexpr (DT == MOE_DTYPE_F32) {
        r.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
        r.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
    } else {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (DT == MOE_DTYPE_BF16) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t *>(&h);
            } else {
                const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
                u[i] = *reinterpret_cast<const uint32_t *>(&h);
            }
        }
        r.a = make_uint4(u[0], u[1], u[2], u[3]);
    }
    return r;
}

// A 16-byte piece of a row: eight 16-bit values or four fp32 ones, so that
// neighbouring lanes always touch neighbouring 16 bytes.
template <int DT> constexpr int kPieceValues = DT == MOE_DTYPE_F32 ? 4 : 8;

template <int DT> __device__ __forceinline__ void widen_piece(const uint4 &r, float (&v)[kPieceValues<DT>]) {
    if constexpr (DT == MOE_DTYPE_F32) {
        v[0] = __uint_as_float(r.x);
        v[1] = __uint_as_float(r.y);
        v[2] = __uint_as_float(r.z);
        v[3] = __uint_as_float(r.w);
    } else {
        widen8<DT>(Raw8<DT>{r}, v);
    }
}

template <int DT> __device__ __forceinline__ uint4 narrow_piece(const float (&v)[kPieceValues<DT>]) {
    if constexpr (DT == MOE_DTYPE_F32)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        return narrow8<DT>(v).a;
}

// grad_w[h] = sum of the blocks' partial sums: thread (i, j) adds every 64th
// block's from j on, four columns wide, then the 64 sums are added in order,
// eight by eight.  The partial sums come from L2 and the launch overlaps the end
// of the one before, so this is latency, 2 to 3 us: every thread's loads are one
// round (1216 rows of 2048: the pass 8.5 us; 32 groups of two rounds 9.5).
constexpr int kColumnGroups = 64;

__device__ __forceinline__ void column_sums(const float *part, int blocks, int H, float *gw) {
    __shared__ float4 s[kColumnGroups][8];
    __shared__ float t[8][32];
    const int i = threadIdx.x & 7, j = threadIdx.x >> 3;
    const int h = blockIdx.x * 32 + i * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (h < H) {
#pragma unroll 5
        for (int b = j; b < blocks; b += kColumnGroups) {
            const float4 p = *reinterpret_cast<const float4 *>(part + (int64_t)b * H + h);
            v.x += p.x;
            v.y += p.y;
            v.z += p.z;
            v.w += p.w;
        }
    }
    s[j][i] = v;
    __syncthreads();
    const float *c = reinterpret_cast<const float *>(s) + (threadIdx.x & 31);
    const int w = threadIdx.x >> 5;
    if (w < 8) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < kColumnGroups / 8; ++k) sum += c[(w * (kColumnGroups / 8) + k) * 32];
        t[w][threadIdx.x & 31] = sum;
    }
    __syncthreads();
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < H) {
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 8; ++k) sum += t[k][threadIdx.x];
        gw[blockIdx.x * 32 + threadIdx.x] = sum;
    }
}

// The kernel's dynamic shared-memory limit, kSmemBlock, set once a device.
template <auto Kernel> cudaError_t allow_smem() {
    static std::mutex mu;
    static bool done[kMaxDevices] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(mu);
    if (done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBlock);
    if (e == cudaSuccess) done[dev] = true;
    return e;
}

inline bool aligned_to(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline bool known_dtype(int32_t d) { return d == MOE_DTYPE_F32 || d == MOE_DTYPE_BF16 || d == MOE_DTYPE_F16; }

}  // namespace moe
