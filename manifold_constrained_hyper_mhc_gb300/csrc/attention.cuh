// What the attention kernels and the 4-bit cache share: the packed batch, the cache's layout, and how a row of
// attention output is written.
#pragma once

#include <cuda_fp16.h>

#include <atomic>

#include "mhc_device.cuh"
#include "mhc_kernels.h"

namespace mhc {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {  // 2^x, hardware approximation (2 ulp; 2^-inf is 0)
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The kernel's dynamic shared memory, set once for each device (the call takes half a microsecond).
template <class Kernel>
inline cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t> &done) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev >= 0 && dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ---- the packed batch -------------------------------------------------------------

// A row's sequence and its first and last row; there is none where b < 0.
struct SeqOfRow {
    int b;
    int64_t begin, end;
};

__device__ __forceinline__ int64_t clamp_row(int32_t o, int64_t T) { return o < 0 ? 0 : (o > T ? T : (int64_t)o); }

// The sequence of packed row t, by one warp: the last b with offsets[b] <= t, if t < offsets[b + 1].  Each step
// narrows the range to a 32nd (one load a lane), so 1,024 sequences take two.  Offsets that decrease give some
// sequence or none, and read nothing outside [0, B].
__device__ __forceinline__ SeqOfRow find_sequence(const int32_t *__restrict__ offsets, int B, int64_t t, int64_t T) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = B;
    while (n > 32) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && __ldg(offsets + lo + lane * step) <= t;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        if (k == 0) return {-1, 0, 0};
        lo += (k - 1) * step;
        n = min(step, n - (k - 1) * step);
    }
    const bool le = lane < n && __ldg(offsets + lo + lane) <= t;
    const int b = lo + __popc(__ballot_sync(0xffffffffu, le)) - 1;
    if (b < 0) return {-1, 0, 0};
    const int64_t begin = clamp_row(__ldg(offsets + b), T), end = clamp_row(__ldg(offsets + b + 1), T);
    if (t < begin || t >= end) return {-1, 0, 0};
    return {b, begin, end};
}

// A block's exclusive sum; `total` the whole.  Two syncs; `scratch` 33 words.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t &total, int64_t *scratch) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
    for (int w = 0; w < NT / 32; ++w) {
        const int64_t y = scratch[w];
        if (w < warp) before += y;
        all += y;
    }
    __syncthreads();
    total = all;
    return before + x - v;
}

// ---- the cache ----------------------------------------------------------------------
// [pages][heads][page / 16 groups] of 17 * D bytes: K of the group's 16 tokens (8 * D bytes of E2M1 codes, then
// D / 2 bytes of scales), V the same way.  A row of codes is D / 2 bytes, two codes a byte (the even value in the
// low half), its 16-byte chunks (32 values: one scale block) in the order chunk ^ swizzle(row), so that eight rows'
// chunks of the same index lie in different shared memory banks once a group is copied there as it is.
template <int D>
struct CacheLayout {
    static constexpr int kGroup = 16;               // tokens
    static constexpr int kBlocks = D / 32;          // scale blocks of a row
    static constexpr int kRow = D / 2;              // bytes of a row's codes
    static constexpr int kPart = 17 * D / 2;        // bytes of K or V of a group
    static constexpr int kGroupBytes = 2 * kPart;
    static constexpr int kScales = 8 * D;           // the scales' place in a part
    __host__ __device__ static constexpr int swizzle(int row) { return (row >> (D == 128 ? 1 : 2)) & (kBlocks - 1); }
};

template <int D>
__device__ __forceinline__ int64_t cache_group(const CacheArgs &c, int page, int head, int group) {
    return (((int64_t)page * c.heads + head) * (c.page >> 4) + group) * CacheLayout<D>::kGroupBytes;
}

// The page of position p of sequence b, or -1 where the table or the cache has none.
__device__ __forceinline__ int cache_page(const CacheArgs &c, int b, int64_t p) {
    if (p < 0) return -1;
    const int64_t col = p >> c.page_log2;
    if (col >= c.width) return -1;
    const int page = __ldg(c.page_table + (int64_t)b * c.width + col);
    return page >= 0 && page < c.pages ? page : -1;
}

__device__ __forceinline__ float ue8m0(uint32_t byte) {  // 2^(byte - 127); 255 is NaN, 0 is 2^-127
    return __uint_as_float(byte == 255u ? 0x7fffffffu : byte == 0u ? 0x00400000u : byte << 23);
}

// Both E2M1 codes of the low byte of w (the low half's value in the low half), exact.
template <int BYTE>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t w) {
    uint32_t d;
    if constexpr (BYTE == 0) asm("{ .reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, a; }" : "=r"(d) : "r"(w));
    if constexpr (BYTE == 1) asm("{ .reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, b; }" : "=r"(d) : "r"(w));
    if constexpr (BYTE == 2) asm("{ .reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, c; }" : "=r"(d) : "r"(w));
    if constexpr (BYTE == 3) asm("{ .reg .b8 a,b,c,e; mov.b32 {a,b,c,e}, %1; cvt.rn.f16x2.e2m1x2 %0, e; }" : "=r"(d) : "r"(w));
    return d;
}
__device__ __forceinline__ float2 half2_to_float2(uint32_t h) { return __half22float2(*reinterpret_cast<__half2 *>(&h)); }

// ---- an output row ----------------------------------------------------------------------
// One head's row, a warp's: lane i holds values i * D/32 .. of it.  bf16, MXFP8 (quantized from fp32 in one rounding)
// and the log-sum, whichever are asked for.
template <int D>
__device__ __forceinline__ void write_head_row(const AttnOut &o, int64_t t, int head, const float (&v)[D / 32], float lse) {
    constexpr int N = D / 32;  // values a lane
    const int lane = threadIdx.x & 31;
    const int64_t at = (t * o.heads + head) * (int64_t)D + lane * N;
    if (o.out != nullptr) {
        uint32_t w[N / 2];
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = pack2_rn(v[2 * i], v[2 * i + 1]);
        if constexpr (N == 4) *reinterpret_cast<uint2 *>(o.out + at) = make_uint2(w[0], w[1]);
        else *reinterpret_cast<uint32_t *>(o.out + at) = w[0];
    }
    if (o.mx.q != nullptr) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) amax = fmaxf(amax, fabsf(v[i]));
#pragma unroll
        for (int m = 1; m < 32 / N; m <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
        const int E = mx_exp(amax, o.mx.mode);
        const float m = __uint_as_float((uint32_t)(127 - E) << 23);
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < N / 2; ++i)
            w |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2 * i] * m, v[2 * i + 1] * m), __NV_SATFINITE, __NV_E4M3) << (16 * i);
        if constexpr (N == 4) *reinterpret_cast<uint32_t *>(o.mx.q + at) = w;
        else *reinterpret_cast<uint16_t *>(o.mx.q + at) = (uint16_t)w;
        if (lane % (32 / N) == 0)
            o.mx.scale[mx_scale_offset(t, head * N + lane / (32 / N), o.heads * D)] = (uint8_t)(E + 127);
    }
    if (o.lse != nullptr && lane == 0) o.lse[t * o.heads + head] = lse;
}

// ---- a row of attention, plainly ----------------------------------------------------------
// One query's attention over n keys by one warp, in fp32: lane i holds values i * D/32 .. of the query, the keys and
// the result.  key(j, x) and value(j, x) fetch the lane's part.  One pass with the running maximum m of the scores and
// the sum l of their exponentials, both in base 2: what was summed before a new maximum is scaled by 2^(m_old - m).
// Eight keys at a time, their loads in flight together (a key alone takes a load's latency, 0.7 us).
template <int D, class Key, class Value>
__device__ __forceinline__ float attend_row(const float (&q)[D / 32], float scale_log2, int64_t n, Key key, Value value, float (&o)[D / 32]) {
    constexpr int N = D / 32, kBatch = 8;
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.f;
    for (int64_t j = 0; j < n; j += kBatch) {
        float x[kBatch][N], s[kBatch], m1 = m;
#pragma unroll
        for (int u = 0; u < kBatch; ++u) key(j + u < n ? j + u : n - 1, x[u]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            s[u] = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) s[u] = fmaf(q[i], x[u][i], s[u]);
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) value(j + u < n ? j + u : n - 1, x[u]);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            s[u] = warp_sum(s[u]) * scale_log2;
            if (j + u < n) m1 = fmaxf(m1, s[u]);
        }
        const float base = m1 == -INFINITY ? 0.f : m1, a = ex2(m - base);  // (scores of -inf alone add nothing; NaN stays)
        m = m1;
        l *= a;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= a;
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
            if (j + u < n) {
                const float p = ex2(s[u] - base);
                l += p;
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = fmaf(p, x[u][i], o[i]);
            }
    }
    const float r = n > 0 ? 1.f / l : 0.f;  // no key: 0; keys whose scores are all -inf: NaN, 0 * inf
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] *= r;
    return n > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace mhc
