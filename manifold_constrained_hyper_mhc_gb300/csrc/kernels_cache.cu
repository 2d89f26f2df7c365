// The 4-bit cache of an attention's keys and values: tokens are quantized to MXFP4 as they are written, and read back
// as bf16.
//
// Per block of 32 values along the head (x_0 .. x_31): E = floor(log2 max|x|) - 2, or the smallest E with
// max|x| <= 6 * 2^E, in [-127, 127]; the scale byte is E + 127 and the codes are the E2M1 values (0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives) nearest to x * 2^-E, ties to the even code.
//
// Both are copies bound by memory.  A warp's rows (K and V of the heads) are one token's, so that its place in the cache
// (its sequence, then its page: dependent loads) is looked up once for all of them.
//
// Measured: 8,192 tokens of 8 heads of 128 written in 9.9 us from bf16 with the source in L2 (13.9 cold; 42 MB, 6.2 us at the
// copy rate) and in 17.3 from fp32 (76 MB, 11.2 us).  No pipe is full (ALU 50 %, issue 48 %, DRAM 31 % cold): a load
// instruction of a warp touches 32 separate pieces of 16 bytes, and the place of a token is two dependent loads.
// 100,798 tokens read back in 86.5 us, 89 % of the copy rate.
#include "attention.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 4;  // warp steps whose loads are in flight together

// Reading: a row (K or V of a head) takes D / 8 lanes of 8 values; a warp step takes kRows rows.
template <int D>
struct Rows {
    static constexpr int kLanes = D / 8, kRows = 32 / kLanes;
};

// E of a block from its largest magnitude (zero or subnormal: -127, infinite: 126).
__device__ __forceinline__ int mx4_exp(float amax, int mode) {
    const uint32_t u = __float_as_uint(amax);
    const int ef = (int)(u >> 23);
    if (ef == 0) return -127;
    int E = ef - 127 - 2;
    if (mode == 1 && (u & 0x7FFFFFu) > 0x400000u) E += 1;  // significand above 1.5
    return E < -127 ? -127 : E;
}

// A block of 32 values a lane (its largest magnitude and its 16 bytes of codes need no other lane): a token's blocks are
// K's of all heads, then V's.
template <int D, bool kF32>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(CacheArgs c, CacheWriteArgs a, int64_t T) {
    using L = CacheLayout<D>;
    const int lane = threadIdx.x & 31;
    const int blocks = c.heads * L::kBlocks, warps = (2 * blocks + 31) / 32;   // of K; warps a token
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / warps;
    if (t >= T) return;
    const int i = (int)(item % warps) * 32 + lane;
    const bool on = i < 2 * blocks;
    const int v = i >= blocks ? 1 : 0, j = on ? i - v * blocks : 0;
    // the values are on their way while the token's place is looked up
    const int64_t at = t * (v ? a.v_stride : a.k_stride) + j * 32;
    float x[32];
    if constexpr (kF32) {
        const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(v ? a.v : a.k) + at);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float4 f = __ldg(p + u);
            x[4 * u] = f.x; x[4 * u + 1] = f.y; x[4 * u + 2] = f.z; x[4 * u + 3] = f.w;
        }
    } else {
        const uint16_t *p = static_cast<const uint16_t *>(v ? a.v : a.k) + at;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            float f[8];
            unpack8(ld_ro(p + 8 * u), f);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * u + e] = f[e];
        }
    }
    const SeqOfRow s = find_sequence(c.offsets, c.B, t, T);
    if (s.b < 0) return;  // behind the last sequence
    const int64_t pos = (int64_t)__ldg(c.seq_lens + s.b) - (s.end - t);
    const int page = cache_page(c, s.b, pos);
    if (page < 0 || !on) return;
    uint32_t top = 0;   // as whole numbers magnitudes keep their order, and NaN is above infinity
#pragma unroll
    for (int e = 0; e < 32; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
    const bool nan = top > 0x7f800000u;
    const int E = mx4_exp(__uint_as_float(top), a.mode);
    const float m = __uint_as_float((uint32_t)(127 - E) << 23);  // 2^-E, E in [-127, 126]
    uint32_t w[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        w[q] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t b;
            asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(b) : "f"(x[8 * q + 2 * e + 1] * m), "f"(x[8 * q + 2 * e] * m));
            w[q] |= b << (8 * e);
        }
        if (nan) w[q] = 0;
    }
    const int place = (int)(pos & (c.page - 1)), row = place & 15, blk = j % L::kBlocks;
    uint8_t *part = c.data + cache_group<D>(c, page, j / L::kBlocks, place >> 4) + v * L::kPart;
    *reinterpret_cast<uint4 *>(part + row * L::kRow + (blk ^ L::swizzle(row)) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
    part[L::kScales + row * L::kBlocks + blk] = (uint8_t)(nan ? 255 : E + 127);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(CacheArgs c, uint16_t *__restrict__ k, uint16_t *__restrict__ v, int64_t T, int rows_per_warp) {
    using L = CacheLayout<D>;
    constexpr int kLanes = Rows<D>::kLanes, kRows = Rows<D>::kRows;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int rows = 2 * c.heads, runs = (rows + rows_per_warp - 1) / rows_per_warp;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / runs;
    if (t >= T) return;
    const int r0 = (int)(item % runs) * rows_per_warp, r1 = min(rows, r0 + rows_per_warp);
    const SeqOfRow s = find_sequence(c.offsets, c.B, t, T);
    if (s.b < 0) return;
    const int64_t pos = (int64_t)__ldg(c.seq_lens + s.b) - (s.end - t);
    const int page = cache_page(c, s.b, pos);
    const int at = (int)(pos & (c.page - 1)), row16 = at & 15;
    const int chunk = (sub >> 2) ^ L::swizzle(row16);
    for (int first = r0 + lane / kLanes; first < r1; first += kAhead * kRows) {
        uint32_t w[kAhead], byte[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = first + u * kRows;
            w[u] = 0, byte[u] = 255;  // no such place: NaN
            if (page >= 0 && r < r1) {
                const uint8_t *part = c.data + cache_group<D>(c, page, r >> 1, at >> 4) + (r & 1) * L::kPart;
                w[u] = __ldg(reinterpret_cast<const uint32_t *>(part + row16 * L::kRow + chunk * 16 + (sub & 3) * 4));
                byte[u] = __ldg(part + L::kScales + row16 * L::kBlocks + (sub >> 2));
            }
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int r = first + u * kRows;
            if (r >= r1) break;
            const float m = ue8m0(byte[u]);
            const uint32_t h[4] = {e2m1x2<0>(w[u]), e2m1x2<1>(w[u]), e2m1x2<2>(w[u]), e2m1x2<3>(w[u])};
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 f = half2_to_float2(h[i]);
                o[i] = pack2_rn(f.x * m, f.y * m);  // exact but where it leaves bf16's range
            }
            st_stream((r & 1 ? v : k) + (t * c.heads + (r >> 1)) * (int64_t)D + sub * 8, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

constexpr int kFill = 32;
// Rows of a token that one warp takes: all of them where the tokens alone fill the device (kFill warps an SM), else as
// few as fill it, a warp step's rows at least.
int rows_per_warp(int rows, int step, int64_t T, int num_sms) {
    const int64_t want = ((int64_t)num_sms * kFill + T - 1) / T;  // warps a token
    const int64_t steps = (rows + step - 1) / step;
    const int64_t each = steps / (want < 1 ? 1 : want);
    return (int)((each < 1 ? 1 : each) * step);
}

}  // namespace

cudaError_t launch_kv_write(const CacheArgs &c, const CacheWriteArgs &a, int64_t T, int D, cudaStream_t stream) {
    const int64_t warps = T * ((2 * c.heads * (D / 32) + 31) / 32);
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    mark_main_kernel(stream, true);
    if (D == 128) {
        if (a.f32) kv_write_kernel<128, true><<<grid, kThreads, 0, stream>>>(c, a, T);
        else kv_write_kernel<128, false><<<grid, kThreads, 0, stream>>>(c, a, T);
    } else {
        if (a.f32) kv_write_kernel<64, true><<<grid, kThreads, 0, stream>>>(c, a, T);
        else kv_write_kernel<64, false><<<grid, kThreads, 0, stream>>>(c, a, T);
    }
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

cudaError_t launch_kv_read(const CacheArgs &c, uint16_t *k, uint16_t *v, int64_t T, int D, int num_sms, cudaStream_t stream) {
    const int per = rows_per_warp(2 * c.heads, 256 / D, T, num_sms);
    const int64_t warps = T * ((2 * c.heads + per - 1) / per);
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    mark_main_kernel(stream, true);
    if (D == 128) kv_read_kernel<128><<<grid, kThreads, 0, stream>>>(c, k, v, T, per);
    else kv_read_kernel<64><<<grid, kThreads, 0, stream>>>(c, k, v, T, per);
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

}  // namespace mhc
