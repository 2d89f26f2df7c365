// Attention of a sequence's last tokens (one, or the few of a speculative-verify block) over its 4-bit cache.
#include "attention.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) decode_rows_kernel(DecodeArgs a) {
    using L = CacheLayout<D>;
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / a.q_heads;
    if (t >= a.T) return;
    const int hq = (int)(item % a.q_heads), head = hq / (a.q_heads / a.c.heads);
    const SeqOfRow s = find_sequence(a.c.offsets, a.c.B, t, a.T);
    if (s.b < 0) return;
    // a length beyond the table's: positions from the table's end on are NaN, and one of them is enough
    const int64_t n = s.end - s.begin, room = (int64_t)a.c.width << a.c.page_log2;
    const int64_t len = min((int64_t)__ldg(a.c.seq_lens + s.b), room + n);
    const int64_t sees = max((int64_t)0, len - n + (t - s.begin) + 1);
    float q[N], o[N];
    const uint16_t *qp = a.q + t * a.q_stride + hq * D + lane * N;
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __uint_as_float((uint32_t)qp[i] << 16);
    auto fetch = [&](int64_t j, int part_v, float (&x)[N]) {
        const int page = cache_page(a.c, s.b, j);
        const int at = (int)(j & (a.c.page - 1)), row = at & 15, blk = lane * N / 32;
        if (page < 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) x[i] = __uint_as_float(0x7fffffffu);
            return;
        }
        const uint8_t *part = a.c.data + cache_group<D>(a.c, page, head, at >> 4) + part_v * L::kPart;
        const uint8_t *codes = part + row * L::kRow + (blk ^ L::swizzle(row)) * 16 + (lane * N % 32) / 2;
        const float m = ue8m0(part[L::kScales + row * L::kBlocks + blk]);
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            const float2 f = half2_to_float2(e2m1x2<0>(codes[i / 2]));
            x[i] = f.x * m;
            x[i + 1] = f.y * m;
        }
    };
    const float lse = attend_row<D>(
        q, a.sm_scale * kLog2e, sees, [&](int64_t j, float (&x)[N]) { fetch(j, 0, x); }, [&](int64_t j, float (&x)[N]) { fetch(j, 1, x); }, o);
    write_head_row<D>(a.o, t, hq, o, lse);
}

}  // namespace

size_t decode_workspace_bytes() { return kControlBytes; }

cudaError_t launch_decode(const DecodeArgs &a, int num_sms, cudaStream_t stream) {
    const unsigned grid = (unsigned)((a.T * a.q_heads + kThreads / 32 - 1) / (kThreads / 32));
    mark_main_kernel(stream, true);
    if (a.D == 128) decode_rows_kernel<128><<<grid, kThreads, 0, stream>>>(a);
    else decode_rows_kernel<64><<<grid, kThreads, 0, stream>>>(a);
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

}  // namespace mhc
