// The 4-bit cache of an attention's keys and values: tokens are quantized to MXFP4 as they are written, and read back
// as bf16.
//
// Per block of 32 values along the head (x_0 .. x_31): E = floor(log2 max|x|) - 2, or the smallest E with
// max|x| <= 6 * 2^E, in [-127, 127]; the scale byte is E + 127 and the codes are the E2M1 values (0, 0.5, 1, 1.5, 2,
// 3, 4, 6 and their negatives) nearest to x * 2^-E, ties to the even code.
//
// Both are copies bound by memory.  A warp takes one token and a run of its rows (K and V of each head), so that the
// token's place in the cache (its sequence, then its page: dependent loads) is looked up once for all of them.
#include "attention.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 128;

// A row (K or V of a head) takes D / 8 lanes of 8 values; a warp step takes kRows rows.
template <int D>
struct Rows {
    static constexpr int kLanes = D / 8, kRows = 32 / kLanes;
};

__device__ __forceinline__ void load8(const void *p, int64_t i, bool f32, float (&x)[8]) {
    if (f32) {
        const float4 a = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i));
        const float4 b = __ldcs(reinterpret_cast<const float4 *>(static_cast<const float *>(p) + i) + 1);
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    } else {
        unpack8(ld_stream(static_cast<const uint16_t *>(p) + i), x);
    }
}

// E of a block from its largest magnitude (zero or subnormal: -127, infinite: 126).
__device__ __forceinline__ int mx4_exp(float amax, int mode) {
    const uint32_t u = __float_as_uint(amax);
    const int ef = (int)(u >> 23);
    if (ef == 0) return -127;
    int E = ef - 127 - 2;
    if (mode == 1 && (u & 0x7FFFFFu) > 0x400000u) E += 1;  // significand above 1.5
    return E < -127 ? -127 : E;
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(CacheArgs c, CacheWriteArgs a, int64_t T, int rows_per_warp) {
    using L = CacheLayout<D>;
    constexpr int kLanes = Rows<D>::kLanes, kRows = Rows<D>::kRows;
    const int lane = threadIdx.x & 31, sub = lane % kLanes;
    const int rows = 2 * c.heads, runs = (rows + rows_per_warp - 1) / rows_per_warp;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / runs;
    if (t >= T) return;
    const int r0 = (int)(item % runs) * rows_per_warp, r1 = min(rows, r0 + rows_per_warp);
    const SeqOfRow s = find_sequence(c.offsets, c.B, t, T);
    if (s.b < 0) return;  // behind the last sequence
    const int64_t pos = (int64_t)__ldg(c.seq_lens + s.b) - (s.end - t);
    const int page = cache_page(c, s.b, pos);
    if (page < 0) return;
    const int at = (int)(pos & (c.page - 1)), row16 = at & 15;
    for (int r = r0 + lane / kLanes; r - lane / kLanes < r1; r += kRows) {  // (the whole warp: shuffles below)
        const bool on = r < r1;
        const int head = (on ? r : r0) >> 1, v = (on ? r : r0) & 1;
        float x[8];
        load8(v ? a.v : a.k, t * (v ? a.v_stride : a.k_stride) + head * D + sub * 8, a.f32, x);
        float amax = 0.f;
        bool nan = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            amax = fmaxf(amax, fabsf(x[i]));
            nan |= x[i] != x[i];
        }
        amax = nan ? __uint_as_float(0x7fffffffu) : amax;
        // the block's four lanes; as whole numbers magnitudes keep their order, and NaN is above infinity
        uint32_t u = __float_as_uint(amax);
        u = max(u, __shfl_xor_sync(0xffffffffu, u, 1));
        u = max(u, __shfl_xor_sync(0xffffffffu, u, 2));
        nan = u > 0x7f800000u;
        const int E = mx4_exp(__uint_as_float(u), a.mode);
        const float m = __uint_as_float((uint32_t)(127 - E) << 23);  // 2^-E, E in [-127, 126]
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t b;
            asm("{ .reg .b8 t; cvt.rn.satfinite.e2m1x2.f32 t, %1, %2; cvt.u32.u8 %0, t; }" : "=r"(b) : "f"(x[2 * i + 1] * m), "f"(x[2 * i] * m));
            w |= b << (8 * i);
        }
        const uint32_t byte = nan ? 255u : (uint32_t)(E + 127);
        if (!on) continue;
        uint8_t *part = c.data + cache_group<D>(c, page, head, at >> 4) + v * L::kPart;
        const int chunk = (sub >> 2) ^ L::swizzle(row16);
        *reinterpret_cast<uint32_t *>(part + row16 * L::kRow + chunk * 16 + (sub & 3) * 4) = nan ? 0u : w;
        if ((sub & 3) == 0) part[L::kScales + row16 * L::kBlocks + (sub >> 2)] = (uint8_t)byte;
    }
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
    for (int r = r0 + lane / kLanes; r < r1; r += kRows) {
        const int head = r >> 1, part_v = r & 1;
        uint32_t w = 0, byte = 255;  // no such place: NaN
        if (page >= 0) {
            const uint8_t *part = c.data + cache_group<D>(c, page, head, at >> 4) + part_v * L::kPart;
            const int chunk = (sub >> 2) ^ L::swizzle(row16);
            w = __ldg(reinterpret_cast<const uint32_t *>(part + row16 * L::kRow + chunk * 16 + (sub & 3) * 4));
            byte = __ldg(part + L::kScales + row16 * L::kBlocks + (sub >> 2));
        }
        const float m = ue8m0(byte);
        const uint32_t h[4] = {e2m1x2<0>(w), e2m1x2<1>(w), e2m1x2<2>(w), e2m1x2<3>(w)};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = half2_to_float2(h[i]);
            o[i] = pack2_rn(f.x * m, f.y * m);  // exact but where it leaves bf16's range
        }
        st_stream((part_v ? v : k) + (t * c.heads + head) * (int64_t)D + sub * 8, make_uint4(o[0], o[1], o[2], o[3]));
    }
}

// Rows of a token that one warp takes: all of them where the tokens alone fill the device (16 warps an SM), else as
// few as fill it, a warp step's rows at least.
int rows_per_warp(int rows, int step, int64_t T, int num_sms) {
    const int64_t want = ((int64_t)num_sms * 16 + T - 1) / T;  // warps a token
    const int64_t steps = (rows + step - 1) / step;
    const int64_t each = steps / (want < 1 ? 1 : want);
    return (int)((each < 1 ? 1 : each) * step);
}

}  // namespace

cudaError_t launch_kv_write(const CacheArgs &c, const CacheWriteArgs &a, int64_t T, int D, int num_sms, cudaStream_t stream) {
    const int per = rows_per_warp(2 * c.heads, 256 / D, T, num_sms);
    const int64_t warps = T * ((2 * c.heads + per - 1) / per);
    const unsigned grid = (unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32));
    mark_main_kernel(stream, true);
    if (D == 128) kv_write_kernel<128><<<grid, kThreads, 0, stream>>>(c, a, T, per);
    else kv_write_kernel<64><<<grid, kThreads, 0, stream>>>(c, a, T, per);
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
