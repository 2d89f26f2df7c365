// Causal attention over packed prompts, with grouped heads.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = sm_scale log2(e) <q, k_j>,  m near the largest s so far
//
// 4 D operations for each query head and visible key: the tensor cores are the floor.  The rows of one kv head are its
// tokens times the heads of the group, NT = 128 / G whole tokens to a tile of 128 rows, so that a tile's rows see nearly
// the same keys whatever G is.  A CTA takes two such tiles (A and B) over all their keys, 128 at a time, so that the
// tensor cores work for one while the other's exponentials are taken:
//   warps 0-3, 4-7  a row a thread: S from tensor memory, the row's maximum and sum, P as bf16 back over S (2^-8 of p: the
//                   products take it beside bf16 v); a maximum is raised only when a score is kLazy above it (p is then
//                   at most 2^kLazy), so the accumulators are rescaled a few times a row
//   warps 8, 9      A's and B's products: S = Q K^T from shared memory, O += P V with P from tensor memory.  They take
//                   turns, O and the next S of one tile at a time (products of both at once end together, and both tiles
//                   then wait for their exponentials together); the waits and commits of one are covered by the other's
//   warp 10         the copies: Q once, then K and V in turn into a ring (TMA, rows of a sequence in 128-byte swizzles).
//                   Then what else the last tiles of V hold: rows behind the sequence are zeroed, and the tiles that some
//                   row sees only in part are searched for values that are not finite (0 times such a value is not 0).
//                   One found, or scores beyond 2^28, sends the CTA's rows through a plain fp32 loop instead.
// Every mbarrier wait is bounded in time; one that gives up sets bit 0 of the status word.
#include <algorithm>
#include <cstring>

#include "attention.cuh"
#include "sm100_ptx.cuh"
#include "tma_encode.h"

namespace mhc {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                           // of a tile
constexpr float kLazy = 8.f;
constexpr float kFar = 268435456.f;                  // 2^28: from here on s - m rounded once may be off by 2^4
constexpr uint64_t kWaitLimitNs = 1000000000ull;     // 1 s per wait
constexpr int kMmaWarp = 8 /* and 9 */, kLoadWarp = 10, kThreads = 12 * 32;

template <int D>
struct Cfg {
    static constexpr int NH = D / 64;                // 128-byte wide halves of a row
    static constexpr int kHalf = 128 * 128;          // bytes of 128 such rows
    static constexpr int kTile = NH * kHalf;         // Q of a tile, or 128 keys' K or V
    static constexpr int ST = D == 128 ? 5 : 8;      // ring
    static constexpr int kSmem = 1024 + 2 * kTile + ST * kTile;
};

struct PromptMaps {
    CUtensorMap q, k, v;
};

struct Bars {
    uint64_t q_full, kv_full[8], kv_empty[8], s_full[2], p_full[2], o_full[2], turn[2], fixed, drained[2];
};

__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
// A wait by a whole warp, back-to-back tests; `dead` stays the same in all lanes.
__device__ __forceinline__ void wait(uint64_t *bar, uint32_t parity, bool &dead) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || dead) return;
    const uint64_t t0 = globaltimer_ns();
    do {
        for (int i = 0; i < 64; ++i)
            if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    } while (!__any_sync(0xffffffffu, globaltimer_ns() - t0 > kWaitLimitNs));
    dead = true;
}
template <int N>
__device__ __forceinline__ void more_registers() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
        "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};\n" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]),
        "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]),
        "r"(r[31])
        : "memory");
}
// D[tmem] (+)= A[smem] x B[smem], bf16.
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// V [keys][64] halves as the N x K operand: N contiguous (64-wide 128-byte swizzled atoms kHalf apart), groups of 8 keys
// 1,024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_v(uint32_t saddr, uint32_t half_bytes) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)((half_bytes >> 4) & 0x3FFFu) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

struct PromptSeq {
    int64_t begin, k0;   // first packed query, first packed key
    int n, len;          // queries and keys
};
__device__ __forceinline__ PromptSeq prompt_sequence(const PromptArgs &a, int b) {
    const int64_t lo = clamp_row(__ldg(a.q_offsets + b), a.Tq), hi = clamp_row(__ldg(a.q_offsets + b + 1), a.Tq);
    const int64_t k0 = clamp_row(__ldg(a.k_offsets + b), a.Tk), k1 = clamp_row(__ldg(a.k_offsets + b + 1), a.Tk);
    return {lo, k0, hi > lo ? (int)(hi - lo) : 0, k1 > k0 ? (int)(k1 - k0) : 0};
}

// One row by a warp, in fp32: the plain form.
template <int D>
__device__ __noinline__ void plain_row(const PromptArgs &a, const PromptSeq &s, int i, int head, int g) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31, hq = head * (a.q_heads / a.kv_heads) + g;
    auto widen = [](const uint16_t *p, float (&x)[N]) {
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = __uint_as_float((uint32_t)__ldg(p + e) << 16);
    };
    float q[N], o[N];
    widen(a.q + (s.begin + i) * a.q_stride + hq * D + lane * N, q);
    const float lse = attend_row<D>(
        q, a.sm_scale * kLog2e, max(0, s.len - s.n + i + 1), [&](int64_t j, float (&x)[N]) { widen(a.k + (s.k0 + j) * a.k_stride + head * D + lane * N, x); },
        [&](int64_t j, float (&x)[N]) { widen(a.v + (s.k0 + j) * a.v_stride + head * D + lane * N, x); }, o);
    write_head_row<D>(a.o, s.begin + i, hq, o, lse);
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptMaps maps, const __grid_constant__ PromptArgs a) {
    using C = Cfg<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem, *ring = smem + 2 * C::kTile;
    __shared__ Bars bar;
    __shared__ uint32_t tmem_base;
    __shared__ int found[2], redo;
    __shared__ int64_t scan[32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.q_heads / a.kv_heads, NT = 128 / G;
    const int head = (int)(blockIdx.x % (unsigned)a.kv_heads), place = (int)(blockIdx.x / (unsigned)a.kv_heads);

    // ---- which pair of tiles: from the last sequence's last (which sees most keys) on
    if (tid == 0) found[0] = -1, redo = 0;
    __syncthreads();
    int64_t before = 0;
    for (int base = 0; base < a.B; base += kThreads) {
        const int b = a.B - 1 - base - tid;
        const int pairs = b >= 0 ? (prompt_sequence(a, b).n + 2 * NT - 1) / (2 * NT) : 0;
        int64_t all;
        const int64_t mine = before + block_scan<kThreads>((int64_t)pairs, all, scan);
        if (place >= mine && place < mine + pairs) {
            found[0] = b;
            found[1] = pairs - 1 - (int)(place - mine);
        }
        before += all;
        if (place < before) break;
    }
    __syncthreads();
    if (found[0] < 0) return;
    const PromptSeq s = prompt_sequence(a, found[0]);
    const int q0 = found[1] * 2 * NT;
    int tokens[2], tiles[2];  // of tile A and B: tokens, and tiles of keys that the last of them sees
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        tokens[x] = min(NT, max(0, s.n - q0 - x * NT));
        const int end = tokens[x] > 0 ? max(0, s.len - s.n + q0 + x * NT + tokens[x]) : 0;
        tiles[x] = (end + kKeys - 1) / kKeys;
    }
    const int n_tiles = max(tiles[0], tiles[1]);

    if (tid == 0) {
        mbar_init(&bar.q_full, 1);
        for (int i = 0; i < C::ST; ++i) {
            mbar_init(&bar.kv_full[i], 1);
            mbar_init(&bar.kv_empty[i], 2);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(&bar.s_full[x], 1);
            mbar_init(&bar.p_full[x], 128);
            mbar_init(&bar.o_full[x], 1);
            mbar_init(&bar.turn[x], 1);
        }
        mbar_init(&bar.fixed, 1);
        for (int x = 0; x < 2; ++x) mbar_init(&bar.drained[x], 1);
        fence_mbar_init();
        fence_proxy_async_smem();
    }
    if (warp < 8 && (tid & 127) >= NT * G) {   // the rows that no token fills, once: nothing is copied there
        for (int h = 0; h < C::NH; ++h)
            for (int o = 0; o < 128; o += 16)
                *reinterpret_cast<uint4 *>(sQ + (warp >> 2) * C::kTile + h * C::kHalf + (tid & 127) * 128 + o) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    const uint32_t tm = tmem_base;            // columns: S of A, S of B (P over them), O of A, O of B
    bool dead = false;
    // The registers of the launch (168 a thread), split anew: 2 * 208 + 88 = 3 * 168.
    auto finish = [&]() {  // by every thread, at its role's end
        if (dead && lane == 0) atomicOr(a.status, 1u);
        tmem_fence_before();
        named_sync(2, kThreads);
    };

    if (warp < 8) {
        more_registers<208>();
        // ---- a row a thread
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + lanes + x * 128, tO = tm + lanes + 256 + x * 128;
        const int i = row / G, g = row - i * G, tok = q0 + x * NT + i;
        const bool on = i < tokens[x];
        const int vis = on ? max(0, s.len - s.n + tok + 1) : 0x7fffffff;   // (a row that is none has nothing to hide)
        const float f = a.sm_scale * kLog2e;
        float m = -INFINITY;
        float2 l2 = make_float2(0.f, 0.f);
        const int n = tiles[x];
        const float2 f2 = make_float2(f, f);
        uint32_t r[4][32];                    // the row's scores, 32 keys at a time
        float hi[4];
        auto maximum = [&](int c) {
            hi[c] = __uint_as_float(r[c][0]);
#pragma unroll
            for (int e = 1; e < 31; e += 2) hi[c] = fmaxf(hi[c], fmaxf(__uint_as_float(r[c][e]), __uint_as_float(r[c][e + 1])));
            hi[c] = fmaxf(hi[c], __uint_as_float(r[c][31]));
        };
        auto exponentials = [&](int c, float2 nb) {  // P of chunk c, over S's first columns (loaded by then)
            uint32_t p[16];
            float2 sum = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                float2 v = __ffma2_rn(make_float2(__uint_as_float(r[c][2 * e]), __uint_as_float(r[c][2 * e + 1])), f2, nb);
                v.x = ex2(v.x);
                v.y = ex2(v.y);
                sum = __fadd2_rn(sum, v);
                p[e] = pack2_rn(v.x, v.y);
            }
            l2 = __fadd2_rn(l2, sum);
            tmem_st16(tS + 16 * c, p);
        };
        for (int j = 0; j < n && !dead; ++j) {
            wait(&bar.s_full[x], j & 1, dead);
            if (dead) break;
            tmem_fence_after();
            const int lim = vis - j * kKeys;
            const float2 before_l = l2;
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, r[c]);
            tmem_wait_ld();
            if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int seen = lim - 32 * c;                           // of the chunk's keys, as bits
                    const uint32_t bits = seen >= 32 ? 0xffffffffu : seen <= 0 ? 0u : (1u << seen) - 1u;
#pragma unroll
                    for (int e = 0; e < 32; ++e) r[c][e] = bits >> e & 1u ? r[c][e] : 0xff800000u;
                }
            }
#pragma unroll
            for (int c = 0; c < 4; ++c) maximum(c);
            const float top = fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3])) * f;
            if (__any_sync(0xffffffffu, top > m + kLazy)) {
                const float m1 = fmaxf(m, top), al = m == -INFINITY ? 0.f : ex2(m - m1);
                if (on && fabsf(m1) > kFar && fabsf(m1) < INFINITY) redo = 1;
                m = m1;
                l2 = make_float2(before_l.x * al, before_l.y * al);
                if (j > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t o[32];
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                        tmem_st32(tO + 32 * c, o);
                    }
                }
            }
            const float base = m == -INFINITY ? 0.f : m;
#pragma unroll
            for (int c = 0; c < 4; ++c) exponentials(c, make_float2(-base, -base));
            tmem_wait_st();
            tmem_fence_before();
            mbar_arrive(&bar.p_full[x]);
        }
        if (n > 0) wait(&bar.o_full[x], 0, dead);
        tmem_fence_after();
        named_sync(1, 288);                   // (with the copies' warp: `redo` is known)
        if (redo) {
            for (int r = warp; r < (tokens[0] + tokens[1]) * G; r += 8) plain_row<D>(a, s, q0 + r / G, head, r % G);
        } else if (!dead) {
            const float l = l2.x + l2.y, inv = vis > 0 ? 1.f / l : 0.f;   // (scores that are all -inf: NaN, 0 * inf)
            const int64_t t = s.begin + tok;
            const int hq = head * G + g;
            uint32_t scales = 0;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                if (n > 0) {
                    tmem_ld32(tO + 32 * c, o);
                    tmem_wait_ld();
                }
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = vis > 0 ? __uint_as_float(o[e]) * inv : 0.f;
                const int64_t at = (t * a.q_heads + hq) * (int64_t)D + 32 * c;
                if (on && a.o.out != nullptr) {
#pragma unroll
                    for (int e = 0; e < 32; e += 8)
                        *reinterpret_cast<uint4 *>(a.o.out + at + e) =
                            make_uint4(pack2_rn(v[e], v[e + 1]), pack2_rn(v[e + 2], v[e + 3]), pack2_rn(v[e + 4], v[e + 5]), pack2_rn(v[e + 6], v[e + 7]));
                }
                if (on && a.o.mx.q != nullptr) {
                    float amax = 0.f;
#pragma unroll
                    for (int e = 0; e < 32; ++e) amax = fmaxf(amax, fabsf(v[e]));
                    const int E = mx_exp(amax, a.o.mx.mode);
                    const float k = __uint_as_float((uint32_t)(127 - E) << 23);
                    uint32_t w[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        w[e] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * e] * k, v[4 * e + 1] * k), __NV_SATFINITE, __NV_E4M3) |
                               (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * e + 2] * k, v[4 * e + 3] * k), __NV_SATFINITE, __NV_E4M3) << 16;
                    *reinterpret_cast<uint4 *>(a.o.mx.q + at) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4 *>(a.o.mx.q + at + 16) = make_uint4(w[4], w[5], w[6], w[7]);
                    scales |= (uint32_t)(E + 127) << (8 * c);
                }
                __syncwarp();
            }
            if (on && a.o.mx.q != nullptr) {  // the head's blocks lie next to each other in a scale tile
                uint8_t *p = a.o.mx.scale + mx_scale_offset(t, hq * (D / 32), a.q_heads * D);
                if constexpr (D == 128) *reinterpret_cast<uint32_t *>(p) = scales;
                else *reinterpret_cast<uint16_t *>(p) = (uint16_t)scales;
            }
            if (on && a.o.lse != nullptr) a.o.lse[t * a.q_heads + hq] = vis > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
        }
        finish();
        return;
    }
    fewer_registers<88>();
    if (warp == kMmaWarp || warp == kMmaWarp + 1) {
        // ---- products of tile A, of tile B: what one warp spends on waits and commits, the other's products cover
        constexpr uint32_t idS = idesc_bf16_f32(128, kKeys), idO = idesc_bf16_f32(128, D) | (1u << 16);   // (V: N contiguous)
        const int x = warp - kMmaWarp, n = tiles[x];
        const uint32_t tS = tm + x * 128, tO = tm + 256 + x * 128, q = smem_u32(sQ + x * C::kTile);
        auto scores = [&](int use) {  // S of the K that use number `use` of the ring holds; then K is done with
            const uint32_t k = smem_u32(ring + (use % C::ST) * C::kTile);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t o = (kk / 4) * C::kHalf + (kk % 4) * 32;
                    umma_ss(tS, sdesc_kmajor_sw128(q + o, 1024), sdesc_kmajor_sw128(k + o, 1024), idS, kk > 0);
                }
                umma_commit(&bar.s_full[x]);
                umma_commit(&bar.kv_empty[use % C::ST]);
            }
            __syncwarp();
        };
        if (n > 0) {
            wait(&bar.q_full, 0, dead);
            wait(&bar.kv_full[0], 0, dead);
            tmem_fence_after();
            if (!dead) scores(0);
        }
        for (int j = 0; j < n && !dead; ++j) {
            const int uv = 2 * j + 1, uk = 2 * j + 2;
            wait(&bar.kv_full[uv % C::ST], (uv / C::ST) & 1, dead);
            if (j == n_tiles - 1 && n_tiles * kKeys > s.len) wait(&bar.fixed, 0, dead);
            if (j + 1 < n) wait(&bar.kv_full[uk % C::ST], (uk / C::ST) & 1, dead);
            wait(&bar.p_full[x], j & 1, dead);
            if (x == 0 ? j > 0 && j - 1 < tiles[1] : j < tiles[0]) wait(&bar.turn[x], (x == 0 ? j - 1 : j) & 1, dead);
            if (dead) break;
            tmem_fence_after();
            const uint32_t v = smem_u32(ring + (uv % C::ST) * C::kTile);
            if (elect_one()) {
#pragma unroll
                for (int kk = 0; kk < kKeys / 16; ++kk) umma_tmemA(tO, tS + kk * 8, sdesc_v(v + kk * 2048, C::kHalf), idO, j > 0 || kk > 0);
                umma_commit(&bar.kv_empty[uv % C::ST]);
                if (j == n - 1) umma_commit(&bar.o_full[x]);
            }
            __syncwarp();
            if (j + 1 < n) scores(uk);
            if (lane == 0) mbar_arrive(&bar.turn[1 - x]);
            __syncwarp();
        }
        // (the ring is the other tile's too: what this one does not use)
        for (int use = 2 * n; use < 2 * n_tiles && !dead; ++use) {
            wait(&bar.kv_full[use % C::ST], (use / C::ST) & 1, dead);
            if (lane == 0) mbar_arrive(&bar.kv_empty[use % C::ST]);
            __syncwarp();
        }
        if (dead) {  // the products in flight must end before their operands and accumulators go
            if (elect_one()) umma_commit(&bar.drained[x]);
            __syncwarp();
            bool d = false;
            wait(&bar.drained[x], 0, d);
        }
    } else if (warp == kLoadWarp) {
        // ---- copies
        const int uses = 2 * n_tiles;
        int i = 0;
        if (n_tiles > 0) {
            if (elect_one()) {
                const uint32_t bytes = (uint32_t)(C::NH * NT * G * 128);
                mbar_arrive_expect_tx(&bar.q_full, 2 * bytes);
                for (int x = 0; x < 2; ++x)
                    for (int h = 0; h < C::NH; ++h)
                        tma_load_4d(sQ + x * C::kTile + h * C::kHalf, &maps.q, 64 * h, 0, head, (int)(s.begin + q0 + x * NT), &bar.q_full);
            }
            __syncwarp();
            for (; i < uses; ++i) {
                const int st = i % C::ST;
                wait(&bar.kv_empty[st], ((i / C::ST) & 1) ^ 1, dead);
                if (dead) break;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.kv_full[st], C::kTile);
                    for (int h = 0; h < C::NH; ++h)
                        tma_load_3d(ring + st * C::kTile + h * C::kHalf, i & 1 ? &maps.v : &maps.k, 64 * h, head, (int)(s.k0 + (i / 2) * kKeys), &bar.kv_full[st]);
                }
                __syncwarp();
            }
            // ---- what else the last tiles of V hold (those that some row sees only in part: the tokens of both tiles lie
            // in three of them at most, and nothing is copied over the last three)
            static_assert(C::ST >= 5, "");
            const int first = max(0, s.len - s.n + q0 + 1) / kKeys;
            for (int j = max(first, n_tiles - 3); j < n_tiles && !dead; ++j) {
                const int use = 2 * j + 1;
                wait(&bar.kv_full[use % C::ST], (use / C::ST) & 1, dead);
                uint8_t *v = ring + (use % C::ST) * C::kTile;
                const int rows = min(kKeys, s.len - j * kKeys);
                if (rows < kKeys) {   // rows behind the sequence
                    for (int h = 0; h < C::NH; ++h)
                        for (int o = rows * 128 + lane * 16; o < C::kHalf; o += 512) *reinterpret_cast<uint4 *>(v + h * C::kHalf + o) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.fixed);
                }
                uint32_t bad = 0;
                for (int h = 0; h < C::NH; ++h)
#pragma unroll 4
                    for (int o = lane * 16; o < rows * 128; o += 512) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(v + h * C::kHalf + o);
                        // an exponent of all ones carries into the sign's place
                        bad |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) | ((w.z & 0x7f807f80u) + 0x00800080u) |
                               ((w.w & 0x7f807f80u) + 0x00800080u);
                    }
                if (bad & 0x80008000u) redo = 1;
            }
            // every copy has to land before the CTA's shared memory goes (where nothing gave up, they have been used)
            for (int u = max(0, i - C::ST); u < i; ++u) {
                bool d = false;
                wait(&bar.kv_full[u % C::ST], (u / C::ST) & 1, d);
                dead |= d;
            }
        }
        __syncwarp();
        named_sync(1, 288);
    }
    finish();
    if (warp == kMmaWarp) {
        tmem_fence_after();
        tmem_dealloc(tm, 512);
    }
}

template <int D>
cudaError_t launch_one(const PromptArgs &a, cudaStream_t stream) {
    using C = Cfg<D>;
    tma::EncodeTiledFn fn;
    cudaError_t e = tma::encoder(fn);
    if (e != cudaSuccess) return e;
    const int G = a.q_heads / a.kv_heads, NT = 128 / G;
    PromptMaps maps;
    std::memset(&maps, 0, sizeof maps);
    {
        const cuuint64_t dq[4] = {D, (cuuint64_t)G, (cuuint64_t)a.kv_heads, (cuuint64_t)a.Tq}, sq[3] = {D * 2, (cuuint64_t)G * D * 2, (cuuint64_t)a.q_stride * 2};
        const cuuint32_t bq[4] = {64, (cuuint32_t)G, 1, (cuuint32_t)NT};
        if ((e = tma::encode_bf16(fn, &maps.q, 4, a.q, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
        const cuuint64_t dk[3] = {D, (cuuint64_t)a.kv_heads, (cuuint64_t)std::max<int64_t>(a.Tk, 1)};
        const cuuint32_t bk[3] = {64, 1, kKeys};
        // (without keys nothing is copied: any address does)
        const cuuint64_t sk[2] = {D * 2, (cuuint64_t)a.k_stride * 2}, sv[2] = {D * 2, (cuuint64_t)a.v_stride * 2};
        if ((e = tma::encode_bf16(fn, &maps.k, 3, a.Tk > 0 ? a.k : a.q, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
        if ((e = tma::encode_bf16(fn, &maps.v, 3, a.Tk > 0 ? a.v : a.q, dk, sv, bk, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    }
    auto kern = prompt_kernel<D>;
    static std::atomic<uint64_t> allowed{0};
    if ((e = allow_smem(kern, C::kSmem, allowed)) != cudaSuccess) return e;
    const int64_t pairs = a.Tq / (2 * NT) + std::min<int64_t>(a.B, a.Tq);   // at most: the lengths are on the device
    mark_main_kernel(stream, true);
    kern<<<(unsigned)(pairs * a.kv_heads), kThreads, C::kSmem, stream>>>(maps, a);
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    return a.D == 128 ? launch_one<128>(a, stream) : launch_one<64>(a, stream);
}

}  // namespace mhc
