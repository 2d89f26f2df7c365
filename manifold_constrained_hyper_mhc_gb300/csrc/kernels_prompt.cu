// Causal attention over packed prompts, with grouped heads.
#include "attention.cuh"

namespace mhc {
namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) prompt_rows_kernel(PromptArgs a) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t t = item / a.q_heads;
    if (t >= a.Tq) return;
    const int hq = (int)(item % a.q_heads), head = hq / (a.q_heads / a.kv_heads);
    const SeqOfRow s = find_sequence(a.q_offsets, a.B, t, a.Tq);
    if (s.b < 0) return;
    const int64_t k0 = clamp_row(__ldg(a.k_offsets + s.b), a.Tk), k1 = clamp_row(__ldg(a.k_offsets + s.b + 1), a.Tk);
    const int64_t sees = max((int64_t)0, max((int64_t)0, k1 - k0) - (s.end - t) + 1);
    float q[N], o[N];
    const uint16_t *qp = a.q + t * a.q_stride + hq * D + lane * N;
    auto widen = [](const uint16_t *p, float (&x)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = __uint_as_float((uint32_t)__ldg(p + i) << 16);
    };
    widen(qp, q);
    const float lse = attend_row<D>(
        q, a.sm_scale * kLog2e, sees, [&](int64_t j, float (&x)[N]) { widen(a.k + (k0 + j) * a.k_stride + head * D + lane * N, x); },
        [&](int64_t j, float (&x)[N]) { widen(a.v + (k0 + j) * a.v_stride + head * D + lane * N, x); }, o);
    write_head_row<D>(a.o, t, hq, o, lse);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int num_sms, cudaStream_t stream) {
    const unsigned grid = (unsigned)((a.Tq * a.q_heads + kThreads / 32 - 1) / (kThreads / 32));
    mark_main_kernel(stream, true);
    if (a.D == 128) prompt_rows_kernel<128><<<grid, kThreads, 0, stream>>>(a);
    else prompt_rows_kernel<64><<<grid, kThreads, 0, stream>>>(a);
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

}  // namespace mhc
