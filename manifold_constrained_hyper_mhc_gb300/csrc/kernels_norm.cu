// Producers of the MXFP8 form besides the fused step: the residual addition with RMSNorm, and the SwiGLU.
//
//   add_rmsnorm  s = bf16(x + residual);  y = bf16(s / sqrt(mean_h s^2 + eps) * gamma);  MXFP8 of y
//   swiglu       MXFP8 of silu(gate) * up
//
// One scale per 32 values, or one per 128 (then written four times, so the scale tiles keep their layout and
// every consumer of them works unchanged).  Both are bound by HBM: each input is read once and each output
// written once.
//
// Roundings.  s and y are held in bf16 between sublayers, so they are rounded there, and the norm and the
// codes are taken from the rounded values, as in the fused step.  The products s * gamma are exact in fp32
// (8-bit significands); the reciprocal root is applied as a pair of fp32 values, so y before its rounding is
// the fp32 value nearest to the exact one, up to the square sum's error.  The SwiGLU's value goes from fp32
// to its code in one rounding; a value that fp32 cannot place (within a few ulp of a border between two
// codes, or a maximum at the border of two exponents) is computed again in fp64.
#include <algorithm>
#include <cstdint>

#include "mhc_device.cuh"
#include "mhc_kernels.h"

namespace mhc {

namespace {

// Packed bf16 arithmetic on the two halves of a word.
__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) { return *reinterpret_cast<__nv_bfloat162 *>(&w); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 b) { return *reinterpret_cast<uint32_t *>(&b); }
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b) { return as_u32(__hadd2_rn(as_bf162(a), as_bf162(b))); }
// The largest magnitude of 8 bf16 values (NaN counts as none).
__device__ __forceinline__ float absmax8(uint4 a) {
    const uint32_t w[4] = {a.x & 0x7FFF7FFFu, a.y & 0x7FFF7FFFu, a.z & 0x7FFF7FFFu, a.w & 0x7FFF7FFFu};
    const __nv_bfloat162 m = __hmax2(__hmax2(as_bf162(w[0]), as_bf162(w[1])), __hmax2(as_bf162(w[2]), as_bf162(w[3])));
    return fmaxf(__low2float(m), __high2float(m));
}

// The 16-byte vectors of one row are spread over the threads so that consecutive lanes hold consecutive
// vectors: 4 lanes hold a block of 32 values, 16 lanes one of 128.
template <int kLanes>
__device__ __forceinline__ float group_max(float a) {
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
    return a;
}

// 2^-E for E in [-127, 127] (2^-127 is subnormal).
__device__ __forceinline__ float inv_pow2(int E) {
    return __uint_as_float(E < 127 ? (uint32_t)(127 - E) << 23 : 0x400000u);
}

// E4M3 codes of 8 scaled values, as two words.
__device__ __forceinline__ uint2 e4m3_codes(const float2 (&u)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int p = 0; p < 4; ++p) w[p] = (uint32_t)__nv_cvt_float2_to_fp8x2(u[p], __NV_SATFINITE, __NV_E4M3);
    return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// The scale bytes w of the row's 128-value group k, by a lane that is `on` (a row's last group may be incomplete: then
// byte by byte, the padding is not written).
__device__ __forceinline__ void mx_store_scales(uint32_t w, bool on, uint8_t *scale, int k, int H) {
    if (on) {
        uint8_t *dst = scale + k * 512;  // mx_scale_col(4 k)
        const int left = H / 32 - 4 * k;
        if (left >= 4) {
            *reinterpret_cast<uint32_t *>(dst) = w;
        } else {
            for (int b = 0; b < left; ++b) dst[b] = (uint8_t)(w >> (8 * b));
        }
    }
}

// Stores vector v (8 scaled values of exponent E) of a row: its codes at `q`, and the scale bytes of 128 values as one
// word from the first of their 16 lanes.  Every lane of the warp calls it.
template <int kBlockLanes>
__device__ __forceinline__ void mx_store(const float2 (&u)[4], int E, bool on, uint8_t *q, uint8_t *scale, int v, int H) {
    if (on) __stcs(reinterpret_cast<uint2 *>(q), e4m3_codes(u));
    uint32_t w = (uint32_t)(E + 127);
    if (kBlockLanes == 16) {
        w *= 0x01010101u;
    } else {
        w |= __shfl_down_sync(0xffffffffu, w, 4) << 8;   // blocks k, k + 1
        w |= __shfl_down_sync(0xffffffffu, w, 8) << 16;  // and k + 2, k + 3
    }
    mx_store_scales(w, on && (v & 15) == 0, scale, v >> 4, H);
}

// ---- residual addition + RMSNorm ---------------------------------------------------------------------
// fp32 holds a row's squares, its root and the products s * gamma where v = mean s^2 + eps is in [2^-40, 2^60] (eps 1e-12 is;
// a product below fp32's range is off by 2^-150, times a root of at most 2^20).  A CTA that met a row beyond ("far": zeros, or
// next to nothing, with a smaller eps; magnitudes past 2^30; infinities, NaN) looks its rows over again at its end and computes
// the far ones in fp64, each thread over its own results.  The borders there lie a little outside those that send it there, so
// a row's result does not depend on the rows beside it.
// Kept out of the loop over the rows, without loops unrolled and without fp64's division and root (they are calls), this costs
// the other rows nothing up to 8192 values a row; longer ones, in 32 registers, up to 7 % (4096 x 8224 52.9 -> 55.7 us, 16384
// 86.5 -> 92.7; 1024 x 65536 nothing).  The same row taken again in the loop, in fp64 or scaled, cost every row up to 25 %.
constexpr uint32_t kMeanMinBits = (127u - 40u) << 23, kMeanMaxBits = (127u + 60u) << 23;
template <int kNT, int kBlockLanes>
__device__ __forceinline__ void norm_far_rows(const uint16_t *x, const uint16_t *residual, const uint16_t *gamma, int64_t T, int H,
                                              float eps, uint16_t *R_out, uint16_t *X_out, const MxOut &mx, double *parts) {
    const int tid = threadIdx.x, nvec = H / kVec;
    const double inv_0 = (double)(1.f / (float)H), inv_h = inv_0 * fma(-inv_0, (double)H, 2.0);
    const double inf = __hiloint2double(0x7FF00000, 0);
    auto two_to = [](int e) { return __hiloint2double((int)((uint32_t)(1023 + e) << 20), 0); };
#pragma unroll 1
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x) {
        const int64_t at = t * (int64_t)H;
        const uint16_t *p = (R_out != nullptr ? R_out : x) + at;  // s: R_out may have replaced the residual
        const uint16_t *q = R_out != nullptr || residual == nullptr ? nullptr : residual + at;
        auto row = [&](int v) {
            const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p) + v);
            if (q == nullptr) return a;
            const uint4 b = __ldcs(reinterpret_cast<const uint4 *>(q) + v);
            return make_uint4(add2(a.x, b.x), add2(a.y, b.y), add2(a.z, b.z), add2(a.w, b.w));
        };
        double sum = 0.0;
#pragma unroll 1
        for (int v = tid; v < nvec; v += kNT) {
            float f[8];
            unpack8(row(v), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fma((double)f[e], (double)f[e], sum);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        __syncthreads();  // `parts` has been read
        if ((tid & 31) == 0) parts[tid >> 5] = sum;
        __syncthreads();
        sum = 0.0;
#pragma unroll 1
        for (int w = 0; w < kNT / 32; ++w) sum += parts[w];
        const double v = fma(sum, inv_h, (double)eps);
        if (v > 0.99 * 9.094947017729282e-13 && v < 1.01 * 1.152921504606847e18) continue;
        // 1 / sqrt(v): v = m 4^k with m in [1, 4), an fp32 estimate of m's and one Newton step
        const int k = ((int)((uint32_t)__double2hiint(v) >> 20) - 1023) >> 1;
        const double m = v * two_to(-2 * k), r0 = (double)rsqrtf((float)m);
        double r = r0 * fma(-0.5 * m, r0 * r0, 1.5) * two_to(-k);
        if (!(v > 0.0 && v < inf)) r = v == 0.0 ? inf : v > 0.0 ? 0.0 : v;
        uint8_t *const scale = mx.q != nullptr ? mx.scale + mx_scale_row(t, H) : nullptr;
#pragma unroll 1
        for (int v0 = 0; v0 < nvec; v0 += kNT) {  // whole groups of lanes: the maxima are exchanged
            const int v = v0 + tid;
            const bool on = v < nvec;
            float f[8], g[8];
            unpack8(on ? row(v) : make_uint4(0u, 0u, 0u, 0u), f);
            unpack8(on ? ld_ro(gamma + v * kVec) : make_uint4(0u, 0u, 0u, 0u), g);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = (float)((double)f[e] * (double)g[e] * r);
            const uint4 y = pack8_rn(f);
            if (on && X_out != nullptr) st_stream(X_out + at + v * kVec, y);
            if (mx.q != nullptr) {
                unpack8(y, f);
                const int E = mx_exp(group_max<kBlockLanes>(on ? absmax8(y) : 0.f), mx.mode);
                const float sc = inv_pow2(E);
                float2 u[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) u[e / 2] = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(sc, sc));
                mx_store<kBlockLanes>(u, E, on, mx.q + at + v * kVec, scale, v, H);
            }
        }
    }
}

// A CTA takes rows in turn.  Rows of at most kNT * kV vectors stay in registers, and the next row's loads are in flight while
// a row's sum is awaited and its results are stored; longer ones (kV == 0: a CTA a row) are read again after the square sum,
// from L2.  8192 x 7168 with the residual (413 MB): 64.3 us, 6.4 TB/s, with 448 threads of two vectors, two CTAs an SM;
// without the loads ahead, four CTAs an SM, 75.5; three CTAs with the loads ahead spill: 86.
// CTAs an SM (8192 rows of 512 to 4096 with one vector a thread: 6.6 to 41.5 us with 1536 threads an SM, 7.9 to 42.1 with
// 1024, 7.4 to 40.9 with 2048, where 333 rows of 4096 take 4.2 us for 3.4).
constexpr int norm_ctas(int nt, int v) { return v == 0 ? 4 : v == 2 ? 2 : 1536 / nt; }
template <int kNT, int kV, int kBlockLanes>
__global__ void __launch_bounds__(kNT, norm_ctas(kNT, kV))
add_rmsnorm_kernel(const uint16_t *__restrict__ x, const uint16_t *residual, const uint16_t *__restrict__ gamma, int64_t T, int H,
                   float eps, uint16_t *R_out, uint16_t *__restrict__ X_out, MxOut mx) {
    __shared__ float sWarp[2][kNT / 32];
    __shared__ double sParts[kNT / 32];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int tid = threadIdx.x, nvec = H / kVec;
    constexpr int kRegs = kV > 0 ? kV : 1;
    uint4 a[kRegs], b[kRegs];
    // this thread's vectors of row t, of both inputs
    auto fetch = [&](int64_t t) {
        const int64_t at = t * (int64_t)H + tid * kVec;
#pragma unroll
        for (int k = 0; k < kRegs; ++k) {
            const bool on = tid + k * kNT < nvec;
            a[k] = on ? ld_stream(x + at + k * kNT * kVec) : make_uint4(0u, 0u, 0u, 0u);
            b[k] = on && residual != nullptr ? __ldcs(reinterpret_cast<const uint4 *>(residual + at + k * kNT * kVec)) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto added = [&](uint4 p, uint4 q) { return residual != nullptr ? make_uint4(add2(p.x, q.x), add2(p.y, q.y), add2(p.z, q.z), add2(p.w, q.w)) : p; };
    auto squares = [&](uint4 a) {
        float f[8];
        unpack8(a, f);
        float2 q = __fmul2_rn(make_float2(f[0], f[1]), make_float2(f[0], f[1]));
#pragma unroll
        for (int e = 2; e < 8; e += 2) q = __ffma2_rn(make_float2(f[e], f[e + 1]), make_float2(f[e], f[e + 1]), q);
        return q.x + q.y;
    };
    bool any_far = false;  // the same in the whole CTA
    if (kV > 0) fetch(blockIdx.x);
    int odd = 0;
    for (int64_t t = blockIdx.x; t < T; t += gridDim.x, odd ^= 1) {
        const int64_t at = t * (int64_t)H + (int64_t)tid * kVec;
        auto again = [&](int off) {  // (rows that do not stay in registers)
            const uint4 p = ld_stream(x + at + off);
            return added(p, residual != nullptr ? __ldcs(reinterpret_cast<const uint4 *>(residual + at + off)) : p);
        };
        uint4 s[kRegs];
        float sum = 0.f;
        if constexpr (kV > 0) {
#pragma unroll
            for (int k = 0; k < kV; ++k) s[k] = added(a[k], b[k]);
            if (t + gridDim.x < T) fetch(t + gridDim.x);
#pragma unroll
            for (int k = 0; k < kV; ++k) sum += squares(s[k]);
        } else {
            for (int v = tid; v < nvec; v += kNT) sum += squares(again((v - tid) * kVec));
        }
        sum = warp_sum(sum);
        if ((tid & 31) == 0) sWarp[odd][tid >> 5] = sum;
        __syncthreads();
        float hi = (tid & 31) < kNT / 32 ? sWarp[odd][tid & 31] : 0.f;
        hi = warp_sum(hi);
        // 1 / sqrt(v), v = sum / H + eps, as rh + rl: an approximation and one Newton step whose residual 1 - v rh^2 is taken
        // with exact products (fp64 here was what the prefill's time went to: 151 us)
        const float inv = 1.f / (float)H, inv_lo = fmaf(-inv, (float)H, 1.f) * inv;
        const float mh = hi * inv, ml = fmaf(hi, inv, -mh) + hi * inv_lo;
        const float vh = mh + eps, vz = vh - mh, vl = ((mh - (vh - vz)) + (eps - vz)) + ml;
        any_far |= __float_as_uint(vh) - kMeanMinBits > kMeanMaxBits - kMeanMinBits;  // (NaN too)
        const float rh = rsqrtf(vh);
        const float ph = rh * rh, pl = fmaf(rh, rh, -ph);
        const float res = fmaf(-vh, ph, 1.f) - fmaf(vh, pl, vl * ph);
        const float rl = 0.5f * rh * res;
        uint8_t *const scale = mx.q != nullptr ? mx.scale + mx_scale_row(t, H) : nullptr;
        const float2 rh2 = make_float2(rh, rh), rl2 = make_float2(rl, rl);
        auto finish = [&](uint4 a, int off) {
            const int v = tid + off / kVec;
            const bool on = v < nvec;
            float f[8], g[8];
            unpack8(a, f);
            unpack8(on ? ld_ro(gamma + tid * kVec + off) : make_uint4(0u, 0u, 0u, 0u), g);
            if (on && R_out != nullptr) st_stream(R_out + at + off, a);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
                const float2 q = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(g[e], g[e + 1]));  // exact
                const float2 o = __ffma2_rn(q, rh2, __fmul2_rn(q, rl2));
                f[e] = o.x;
                f[e + 1] = o.y;
            }
            const uint4 y = pack8_rn(f);
            if (on && X_out != nullptr) st_stream(X_out + at + off, y);
            if (mx.q != nullptr) {
                unpack8(y, f);
                const float amax = group_max<kBlockLanes>(on ? absmax8(y) : 0.f);
                const int E = mx_exp(amax, mx.mode);
                const float sc = inv_pow2(E);
                float2 u[4];
#pragma unroll
                for (int e = 0; e < 8; e += 2) u[e / 2] = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(sc, sc));
                mx_store<kBlockLanes>(u, E, on, mx.q + at + off, scale, v, H);
            }
        };
        if constexpr (kV > 0) {
#pragma unroll
            for (int k = 0; k < kV; ++k)
                if (k == 0 || k * kNT < nvec) finish(s[k], k * kNT * kVec);
        } else {
            for (int v0 = 0; v0 < nvec; v0 += kNT)  // whole groups of lanes: the maxima are exchanged
                finish(v0 + tid < nvec ? again(v0 * kVec) : make_uint4(0u, 0u, 0u, 0u), v0 * kVec);
        }
    }
    if (any_far) {
        // (what is known of these pointers is for the loop above, whose loads do not wait for its stores)
        const uint16_t *x_again = x, *gamma_again = gamma;
        uint16_t *X_again = X_out;
        asm volatile("" : "+l"(x_again), "+l"(gamma_again), "+l"(X_again)::"memory");
        norm_far_rows<kNT, kBlockLanes>(x_again, residual, gamma_again, T, H, eps, R_out, X_again, mx, sParts);
    }
}

// ---- SwiGLU ------------------------------------------------------------------------------------------
// a / (1 + exp(-a)) * b with the hardware's exponential and reciprocal, the exponential's argument as a pair (its rounding
// alone would cost |a| ulp).  For a >= kGateMin the relative error is at most 4.5 2^-23: the exponential 2^-22, the
// reciprocal 2^-23, three roundings 2^-24 each; twice that in units of the last place of a scaled value just below a
// power of two: within kNear.
constexpr float kGateMin = -80.f;  // below it the reciprocal's argument comes near fp32's largest values
constexpr uint32_t kNear = 12;
// (Above kGateMax the pair overflows.)
constexpr float kGateMax = 1e38f;
__device__ __forceinline__ bool gate_far(float a) { return a < kGateMin || a > kGateMax; }
__device__ __forceinline__ float2 silu_mul2(float2 a, float2 b) {
    constexpr float kL2E = 1.44269504f, kL2ELo = 1.92596303e-8f, kLn2 = 0.693147181f;  // log2(e) as a pair
    const float2 t = __fmul2_rn(a, make_float2(-kL2E, -kL2E));
    float2 tl = __ffma2_rn(a, make_float2(-kL2E, -kL2E), make_float2(-t.x, -t.y));
    tl = __ffma2_rn(a, make_float2(-kL2ELo, -kL2ELo), tl);
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    e = __ffma2_rn(e, __fmul2_rn(tl, make_float2(kLn2, kLn2)), e);
    const float2 d = __fadd2_rn(e, make_float2(1.f, 1.f));
    return __fmul2_rn(__fmul2_rn(a, make_float2(rcp_approx(d.x), rcp_approx(d.y))), b);
}
__device__ __noinline__ double silu_mul_f64(float a, float b) { return (double)a / (1.0 + exp(-(double)a)) * (double)b; }

// Whether u = x * 2^-E may lie on the other side of a border between two codes, being kNear units off: its 20 bits below
// E4M3's significand within that of one half, i.e. border_key(u) <= kNear << 13.  (Below E4M3's normal range the
// codes are fixed-point and the test is not exact there; a code off by one of 2^-9 in values of up to 448 is what fp32
// leaves.)
__device__ __forceinline__ uint32_t border_key(float u) { return (__float_as_uint(u) << 12) + ((0x80000u + kNear) << 12); }
// The same for a maximum: near a power of two (or past fp32's range), or near 1.75 times one (mode 1).
__device__ __forceinline__ bool near_exponent(float a, int mode) {
    if (a < 1.5046328e-36f) return false;  // 2^-119: up to 2^-118 (mode 1: 1.75 2^-119) the exponent is the smallest one
    const uint32_t m = __float_as_uint(a) & 0x7FFFFFu;
    return m + kNear > 0x7FFFFFu || m < kNear || (mode == 1 && m - (0x600000u - kNear) <= 2 * kNear);
}
// mx_exp of a value held in fp64 (products beyond fp32's range among them).
__device__ __noinline__ int mx_exp_f64(double amax, int mode) {
    if (isinf(amax)) return 120;  // as mx_exp
    if (!(amax >= 1.1754943508222875e-38)) return -127;  // 2^-126
    const int e = ilogb(amax);
    int E = e - 8;
    if (mode == 1 && amax > scalbn(1.75, e)) E += 1;
    return E < -127 ? -127 : (E > 127 ? 127 : E);
}

// 16 output values of a lane (consecutive lanes hold consecutive ones of a row; `on`: inside the row): their codes go to
// `q`, the row's scales are at `scale`.  kBlockLanes lanes share an exponent.
constexpr int kLaneVals = 16;
template <int kBlockLanes>
__device__ __forceinline__ void swiglu_vals(const uint4 (&ga)[2], const uint4 (&ub)[2], bool on, uint8_t *q, uint8_t *scale, int v,
                                            int F, int mode) {
    float a[kLaneVals], b[kLaneVals], f[kLaneVals];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        unpack8(ga[h], *reinterpret_cast<float (*)[8]>(&a[8 * h]));
        unpack8(ub[h], *reinterpret_cast<float (*)[8]>(&b[8 * h]));
    }
    float amax = 0.f;
#pragma unroll
    for (int e = 0; e < kLaneVals; e += 2) {
        const float2 y = silu_mul2(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
        f[e] = y.x;
        f[e + 1] = y.y;
        amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
    }
    __nv_bfloat162 lo2 = as_bf162(ga[0].x), hi2 = lo2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t w[4] = {ga[h].x, ga[h].y, ga[h].z, ga[h].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            lo2 = __hmin2(lo2, as_bf162(w[k]));
            hi2 = __hmax2(hi2, as_bf162(w[k]));
        }
    }
    bool far = on && (gate_far(fminf(__low2float(lo2), __high2float(lo2))) || gate_far(fmaxf(__low2float(hi2), __high2float(hi2))));
    amax = group_max<kBlockLanes>(amax);
    int E = mx_exp(amax, mode);
    if (__any_sync(0xffffffffu, far || (on && near_exponent(amax, mode)))) {
        // the block's maximum in fp64, from the values that can be it
        double m = 0.0;
        const float cut = amax * 0.99999f;
#pragma unroll
        for (int e = 0; e < kLaneVals; ++e) {
            if (on && (gate_far(a[e]) || !(fabsf(f[e]) < cut))) {
                const double d = fabs(silu_mul_f64(a[e], b[e]));
                m = d > m ? d : m;
            }
        }
#pragma unroll
        for (int o = 1; o < kBlockLanes; o <<= 1) {
            const double d = __shfl_xor_sync(0xffffffffu, m, o);
            m = d > m ? d : m;
        }
        E = mx_exp_f64(m, mode);
        far |= isinf(amax);  // products past fp32's range: infinite here, their codes are not
    }
    const float sc = inv_pow2(E);
    float2 u[kLaneVals / 2];
    uint32_t key = 0xFFFFFFFFu;
#pragma unroll
    for (int e = 0; e < kLaneVals; e += 2) {
        u[e / 2] = __fmul2_rn(make_float2(f[e], f[e + 1]), make_float2(sc, sc));
        key = min(key, min(border_key(u[e / 2].x), border_key(u[e / 2].y)));
    }
    if (on && (key <= kNear << 13 || far)) {
#pragma unroll
        for (int e = 0; e < kLaneVals; ++e) {
            float &w = e & 1 ? u[e / 2].y : u[e / 2].x;
            if (border_key(w) <= kNear << 13 || gate_far(a[e]) || isinf(w)) {
                // the fp64 value over 2^E, with whatever fp32 drops of it kept as a sticky last bit, rounds to the same code
                const double d = silu_mul_f64(a[e], b[e]) * (double)sc;
                w = __double2float_rz(d);
                if ((double)w != d) w = __uint_as_float(__float_as_uint(w) | 1u);
            }
        }
    }
    const uint2 c0 = e4m3_codes(*reinterpret_cast<const float2 (*)[4]>(&u[0])), c1 = e4m3_codes(*reinterpret_cast<const float2 (*)[4]>(&u[4]));
    if (on) __stcs(reinterpret_cast<uint4 *>(q), make_uint4(c0.x, c0.y, c1.x, c1.y));
    // the scale bytes of 128 values (8 lanes) as one word
    uint32_t w = (uint32_t)(E + 127);
    if (kBlockLanes == 8) {
        w *= 0x01010101u;
    } else {
        w |= __shfl_down_sync(0xffffffffu, w, 2) << 8;   // blocks k, k + 1
        w |= __shfl_down_sync(0xffffffffu, w, 4) << 16;  // and k + 2, k + 3
    }
    mx_store_scales(w, on && (v & 7) == 0, scale, v >> 3, F);
}

// A thread takes 16 values at a time (two vectors of gate, two of up: four loads of 16 bytes), the next ones' loads in
// flight; rows are padded to whole groups of 8 lanes (128 values: a word of scales).  16384 x 2048 (169 MB): 33.4 us with one
// CTA of 512 threads an SM, that is 5.0 TB/s; 39.8 with 8 values at a time and 768 threads (twice the votes, shuffles and
// scale stores a value, half the bytes in flight a thread); 34.0 with two CTAs of 256 threads, 39 with 384 threads, 41.6 with
// 768 (registers spill; 640 threads spill a little and take 33.0).  A call that does not fill one round of the large CTAs
// takes the small ones (48 x 2048: 3.2 us against 3.7; 2048 x 2048: 10.1 against 8.5).
template <int kNT, int kBlockLanes>
__global__ void __launch_bounds__(kNT)
swiglu_kernel(const uint16_t *__restrict__ gu, int64_t T, int F, int lanes_row, MxOut mx) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t step = (int64_t)gridDim.x * kNT, first = (int64_t)blockIdx.x * kNT + threadIdx.x;
    const int64_t dt = step / lanes_row;
    const int dv = (int)(step - dt * lanes_row);
    int64_t t = first / lanes_row;
    int v = (int)(first - t * lanes_row);
    uint4 g[2], u[2];
    bool on;
    auto load = [&]() {
        on = t < T && v * kLaneVals < F;
        const uint16_t *src = gu + t * 2 * (int64_t)F + (int64_t)v * kLaneVals;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            g[h] = on ? ld_stream(src + 8 * h) : make_uint4(0u, 0u, 0u, 0u);
            u[h] = on ? ld_stream(src + F + 8 * h) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    load();
    for (int64_t n = (int64_t)blockIdx.x * kNT; n < T * lanes_row; n += step) {  // the same for the whole block
        const uint4 g0[2] = {g[0], g[1]}, u0[2] = {u[0], u[1]};
        const bool on0 = on;
        const int64_t t0 = t;
        const int v0 = v;
        t += dt;
        v += dv;
        if (v >= lanes_row) {
            v -= lanes_row;
            ++t;
        }
        load();
        swiglu_vals<kBlockLanes>(g0, u0, on0, mx.q + t0 * F + (int64_t)v0 * kLaneVals, mx.scale + mx_scale_row(t0, F), v0, F, mx.mode);
    }
}

// A launch that may start while the launch before it drains (it waits for that one's results itself).
template <typename... P, typename... A>
cudaError_t launch_pdl(void (*kern)(P...), unsigned grid, unsigned block, cudaStream_t stream, A... args) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    mark_main_kernel(stream, true);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    mark_main_kernel(stream, false);
    return e;
}

template <int kNT, int kV>
cudaError_t launch_norm_nv(const uint16_t *x, const uint16_t *residual, const uint16_t *gamma, int64_t T, int H, float eps,
                           uint16_t *R_out, uint16_t *X_out, const MxOut &mx, int block, int num_sms, cudaStream_t stream) {
    auto kern = block == 128 ? add_rmsnorm_kernel<kNT, kV, 16> : add_rmsnorm_kernel<kNT, kV, 4>;
    return launch_pdl(kern, (unsigned)std::min<int64_t>(T, kV == 0 ? T : (int64_t)num_sms * norm_ctas(kNT, kV)), kNT, stream, x, residual, gamma, T, H, eps, R_out, X_out, mx);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const uint16_t *x, const uint16_t *residual, const uint16_t *gamma, int64_t T, int H,
                               float eps, uint16_t *R_out, uint16_t *X_out, const MxOut &mx, int block, int num_sms,
                               cudaStream_t stream) {
    const int nvec = H / kVec;
    // The fewest threads that hold the row with one vector each, from 513 vectors with two (us at 8192 rows with the
    // residual, a CTA a row: H = 512: 64 x 1 8.9, 256 x 1 15; 2048: 256 x 1 24.5, 128 x 2 24.1, 64 x 4 28.0; 4096: 512 x 1
    // 45.3, 256 x 2 47.8; 7168: 448 x 2 75, 512 threads reading the row twice 84.8; 8192: 512 x 2 85.6, 256 x 4 97, twice
    // 89.5.  With rows in turn 6.3, 21.9, 40.9, 64.3 and 75.9).
    if (nvec <= 64) return launch_norm_nv<64, 1>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    if (nvec <= 128) return launch_norm_nv<128, 1>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    if (nvec <= 256) return launch_norm_nv<256, 1>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    if (nvec <= 512) return launch_norm_nv<512, 1>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    if (nvec <= 896) return launch_norm_nv<448, 2>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    if (nvec <= 1024) return launch_norm_nv<512, 2>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
    return launch_norm_nv<512, 0>(x, residual, gamma, T, H, eps, R_out, X_out, mx, block, num_sms, stream);
}

cudaError_t launch_swiglu(const uint16_t *gate_up, int64_t T, int F, const MxOut &mx, int block, int num_sms,
                          cudaStream_t stream) {
    const int lanes_row = (F / kLaneVals + 7) / 8 * 8;
    const int64_t n = T * lanes_row;
    if (n >= (int64_t)num_sms * 512) {
        auto kern = block == 128 ? swiglu_kernel<512, 8> : swiglu_kernel<512, 2>;
        return launch_pdl(kern, (unsigned)num_sms, 512, stream, gate_up, T, F, lanes_row, mx);
    }
    auto kern = block == 128 ? swiglu_kernel<128, 8> : swiglu_kernel<128, 2>;
    return launch_pdl(kern, (unsigned)((n + 127) / 128), 128, stream, gate_up, T, F, lanes_row, mx);
}

}  // namespace mhc
