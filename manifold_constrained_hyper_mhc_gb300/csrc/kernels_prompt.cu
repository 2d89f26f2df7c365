// Causal attention over packed prompts, with grouped heads.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = sm_scale log2(e) <q, k_j>,  m at or above the largest s so far
//
// 4 D operations for each query head and visible key: the tensor cores are the floor.  The rows of one kv head are its
// tokens times the heads of the group, NT = 128 / G whole tokens to a tile of 128 rows, so that a tile's rows see nearly
// the same keys whatever G is.  A CTA takes two such tiles (A and B) over all their keys, 128 at a time:
//   warps 0-3, 4-7  A's and B's rows, a row a thread: S from tensor memory, the row's maximum and sum, P as bf16 back to
//                   tensor memory (2^-8 of p: the products take it beside bf16 v); m is set kLazy above the largest score
//                   and raised when one passes it, so the accumulators are rescaled a few times a row and p is at most 1
//                   (sums of p v end where fp32 sums of weights and v do; p ends at 2^-126, 2^-118 of the largest)
//   warp 8          S = Q K^T from shared memory, A's and B's in turn into the same columns: S is in registers soon after
//                   it is there, so the next one is computed beside the exponentials of this one
//   warp 9          O += P V with P from tensor memory
//   warp 10         the copies: Q, then K and V in turn into a ring (TMA, rows of a sequence in 128-byte swizzles)
//   warp 11         what else the last tiles of V hold: rows that none of the pair sees are zeroed, and the tiles that some
//                   row sees only in part are searched for values that are not finite (0 times such a value is not 0).
//                   One that some rows of a tile do not see, or scores beyond 2^28, sends the tile's rows through a plain
//                   fp32 loop instead.
// The grid has a block for every pair of tiles; a CTA that has issued its pair's copies takes over a block that has not
// begun (cluster launch control), so that its next pair's copies and first products run beside the present one's end, and
// pairs of all lengths fill the device.
// Every mbarrier wait is bounded in time; one that gives up sets bit 0 of the status word.
//
// Measured: 8,192 tokens, 56 / 8 heads of 128: 660 us a call among calls, 1,457 TFLOP/s, 75 % of the measured bf16 rate (84 %
// of that of long runs: the power limit lowers the clock) and 620 us alone, 80 %; the tensor pipe is 67 % active.  2,000
// tokens after 30,001: 1,170 us, 79 %, and 1,120 alone.  8,192 tokens, 32 / 4 heads of 64: 247 us, 1,113 TFLOP/s, no pipe
// full (tensor 47 % active, exponentials 47 %, ALU 37 %, issue 53 %): the chain from S over the exponentials to P.  Short
// prompts (nine of 37 to 1,500 tokens, 32 / 8 heads: 85 us, 40 %, tensor pipe 40 %) have that chain, the last products and
// the result of a pair in a row, 14 us, of which the products take 6.4.
#include <algorithm>
#include <cstring>

#include "attention.cuh"
#include "sm100_ptx.cuh"
#include "tile_ring.h"
#include "tma_encode.h"

namespace mhc {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                           // of a tile
constexpr float kLazy = 8.f;
constexpr float kFar = 268435456.f;                  // 2^28: from here on s - m rounded once may be off by 2^4
constexpr uint64_t kWaitLimitNs = 20000000000ull;    // 20 s per wait: 32 rows of a warp over 2^20 keys, plainly, take 3 s
constexpr int kMmaWarp = 8 /* and 9 */, kLoadWarp = 10, kThreads = 12 * 32;

template <int D>
struct Cfg {
    static constexpr int NH = D / 64;                // 128-byte wide halves of a row
    static constexpr int kHalf = 128 * 128;          // bytes of 128 such rows
    static constexpr int kTile = NH * kHalf;         // Q of a tile, or 128 keys' K or V
    static constexpr int ST = D == 128 ? 5 : 8;      // ring
    static constexpr int kSmem = 1024 + 2 * kTile + ST * kTile;
    using Ring = TileRing<ST>;
    static_assert(Ring::kFull <= 10 && ST <= 8, "");   // (Bars)
};

struct PromptMaps {
    CUtensorMap q, k, v;
};

constexpr int kPart = 3;   // tiles of keys that a pair's rows see only in part: its tokens are at most 256 neighbours

// A wait by parity needs the phase before to be complete (tile_ring.h).  It is, at each of them: a waiter goes through every
// phase of item_full, item_empty, next, q_full, q_empty, kv_empty, s_full, s_taken, p_full, pv_done, rows_done and of its
// own kv_full (warp 8 K's, warp 9 V's).  Those that skip phases are warp 9 at `checked` and warp 11 at `go` (tiles of keys that an item
// does not have) and at kv_full: an item's slot is written anew only when every role has left it, and `checked` and `go` have
// completed their phases of it by then; `go` itself comes after kv_full's phase has begun.
struct Bars {
    uint64_t item_full[2], item_empty[2], next;
    uint64_t q_full, q_empty, kv_full[10], kv_empty[8], s_full[2], s_taken, p_full[2], pv_done[2];
    uint64_t go[2][kPart], checked[2][kPart], rows_done[2], drained[2];
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
// A pair of tiles of one kv head.
struct Item {
    PromptSeq s;
    int more, head, q0;      // whether there is one; its kv head, and its first token
    int tokens[2], tiles[2]; // of tile A and B: tokens, and tiles of keys that the last of them sees
    int first[2], seen;      // keys that the first token of each sees, and those that the pair's last one sees
    int n_tiles, part;       // tiles of keys, and the first that some row sees only in part
};

// Which pair is `place`, by one warp.  Sequence b's pairs are the places from floor(offset_b / X) + b on, X tokens to a pair: they
// never reach the next sequence's, and the range of places that holds the last b with floor(offset_b / X) + b <= place is
// narrowed to a 32nd a step.  Places without a pair are left over, one a sequence at most.  Places are taken from the
// last on, so that a sequence's longest pairs come first.
__device__ __forceinline__ Item locate(const PromptArgs &a, unsigned block, unsigned blocks, int NT) {
    const int lane = threadIdx.x & 31, X = 2 * NT;
    Item it{};
    it.more = 1;
    it.head = (int)(block % (unsigned)a.kv_heads);
    const int64_t place = (int64_t)(blocks / (unsigned)a.kv_heads) - 1 - (int64_t)(block / (unsigned)a.kv_heads);
    auto key = [&](int b) { return clamp_row(__ldg(a.q_offsets + b), a.Tq) / X + b; };
    int lo = 0, n = a.B;
    while (n > 32) {
        const int step = (n + 31) / 32;
        const bool le = lane * step < n && key(lo + lane * step) <= place;
        const int k = __popc(__ballot_sync(0xffffffffu, le));
        if (k == 0) return it;
        lo += (k - 1) * step;
        n = min(step, n - (k - 1) * step);
    }
    const bool le = lane < n && key(lo + lane) <= place;
    const int b = lo + __popc(__ballot_sync(0xffffffffu, le)) - 1;
    if (b < 0) return it;
    const int64_t begin = clamp_row(__ldg(a.q_offsets + b), a.Tq), end = clamp_row(__ldg(a.q_offsets + b + 1), a.Tq);
    const int64_t k0 = clamp_row(__ldg(a.k_offsets + b), a.Tk), k1 = clamp_row(__ldg(a.k_offsets + b + 1), a.Tk);
    const int64_t pair = place - (begin / X + b);
    if (end <= begin || pair * X >= end - begin) return it;
    it.s = {begin, k0, (int)(end - begin), k1 > k0 ? (int)(k1 - k0) : 0};
    it.q0 = (int)pair * X;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
        it.tokens[x] = min(NT, max(0, it.s.n - it.q0 - x * NT));
        const int last = it.tokens[x] > 0 ? max(0, it.s.len - it.s.n + it.q0 + x * NT + it.tokens[x]) : 0;
        it.tiles[x] = (last + kKeys - 1) / kKeys;
        it.first[x] = max(0, it.s.len - it.s.n + it.q0 + x * NT + 1);
        it.seen = max(it.seen, last);
    }
    it.n_tiles = max(it.tiles[0], it.tiles[1]);
    it.part = max(max(0, it.s.len - it.s.n + it.q0 + 1) / kKeys, it.n_tiles - kPart);
    return it;
}

// ---- a row's scores of 32 keys
__device__ __forceinline__ float largest(const uint32_t (&r)[32]) {
    float hi = __uint_as_float(r[0]);
#pragma unroll
    for (int e = 1; e < 31; e += 2) hi = fmaxf(hi, fmaxf(__uint_as_float(r[e]), __uint_as_float(r[e + 1])));
    return fmaxf(hi, __uint_as_float(r[31]));
}
// Their exponentials as bf16, and added to the row's sum.
__device__ __forceinline__ void exponentials(const uint32_t (&r)[32], float2 f2, float2 minus_m, float2 &l2, uint32_t *p) {
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        float2 v = __ffma2_rn(make_float2(__uint_as_float(r[2 * e]), __uint_as_float(r[2 * e + 1])), f2, minus_m);
        v.x = ex2(v.x);
        v.y = ex2(v.y);
        sum = __fadd2_rn(sum, v);
        p[e] = pack2_rn(v.x, v.y);
    }
    l2 = __fadd2_rn(l2, sum);
}

// Lane a of a group of four gives its units u[0..3] to the lanes of those numbers, and gets unit a of each.
template <int N>
__device__ __forceinline__ void transpose4(uint32_t (&u)[4][N]) {
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        const bool high = threadIdx.x & m;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            if (p & m) continue;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const uint32_t x = __shfl_xor_sync(0xffffffffu, high ? u[p][i] : u[p | m][i], m);
                if (high) u[p][i] = x;
                else u[p | m][i] = x;
            }
        }
    }
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
    using Ring = typename C::Ring;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t *sQ = smem, *ring = smem + 2 * C::kTile;
    __shared__ Bars bar;
    __shared__ Item items[2];
    __shared__ int redo[2][2], far[2][2];     // of an item's tiles
    __shared__ __align__(16) uint4 answer;    // which block was taken over
    __shared__ uint32_t tmem_base;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = a.q_heads / a.kv_heads, NT = 128 / G;

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], 11);   // every other warp
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.p_full[i], 128);
            mbar_init(&bar.pv_done[i], 1);
            mbar_init(&bar.rows_done[i], 4);   // its warps
            mbar_init(&bar.drained[i], 1);
            for (int k = 0; k < kPart; ++k) {
                mbar_init(&bar.go[i][k], 1);
                mbar_init(&bar.checked[i][k], 1);
            }
        }
        mbar_init(&bar.next, 1);
        mbar_init(&bar.s_taken, 128);
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, 1);
        for (uint32_t i = 0; i < Ring::kFull; ++i) mbar_init(&bar.kv_full[i], 1);
        for (int i = 0; i < C::ST; ++i) mbar_init(&bar.kv_empty[i], 1);
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
    const uint32_t tm = tmem_base;            // columns: S (of either tile), P of A, P of B, O of A, O of B
    bool dead = false, issued = false;        // a wait gave up; this warp has issued products
    auto finish = [&]() {  // by every thread, at its role's end
        if (dead && lane == 0) atomicOr(a.status, 1u);
        tmem_fence_before();
        named_sync(2, kThreads);
    };
    // Item t is in slot t % 2, the 1 + t / 2nd there.
    auto take = [&](int t) {
        wait(&bar.item_full[t & 1], (t >> 1) & 1, dead);
        return !dead && items[t & 1].more != 0;
    };
    auto leave = [&](int t) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[t & 1]);
    };

    // The registers of the launch (168 a thread), split anew: 2 * 208 + 88 = 3 * 168.
    if (warp < 8) {
        more_registers<208>();
        // ---- a row a thread
        const int x = warp >> 2, row = tid & 127;
        const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tm + lanes, tP = tS + 128 + x * 64, tO = tS + 256 + x * 128;
        const int i = row / G, g = row - i * G;
        const float f = a.sm_scale * kLog2e;
        const float2 f2 = make_float2(f, f);
        uint32_t n_s = 0, n_pv = 0;           // scores so far, products with V waited for
        for (int t = 0; take(t); ++t) {
            const Item &it = items[t & 1];
            const int tok = it.q0 + x * NT + i, n = it.tiles[x], slot = t & 1;
            const bool on = i < it.tokens[x];
            const int vis = on ? max(0, it.s.len - it.s.n + tok + 1) : 0x7fffffff;   // (a row that is none has nothing to hide)
            float m = -INFINITY;
            float2 l2 = make_float2(0.f, 0.f);
            for (int j = 0; j < n; ++j, ++n_s) {
                wait(&bar.s_full[x], n_s & 1, dead);
                if (dead) break;
                tmem_fence_after();
                uint32_t r[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + 32 * c, r[c]);
                tmem_wait_ld();
                tmem_fence_before();
                mbar_arrive(&bar.s_taken);    // (the next scores may come, the other tile's)
                const int lim = vis - j * kKeys;
                if (__any_sync(0xffffffffu, lim < kKeys)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int seen = lim - 32 * c;                           // of the chunk's keys, as bits
                        const uint32_t bits = seen >= 32 ? 0xffffffffu : seen <= 0 ? 0u : (1u << seen) - 1u;
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[c][e] = bits >> e & 1u ? r[c][e] : 0xff800000u;
                    }
                }
                const float top = fmaxf(fmaxf(largest(r[0]), largest(r[1])), fmaxf(largest(r[2]), largest(r[3]))) * f;
                bool idle = j == 0;           // the products with the P before are done
                auto pv_done = [&]() {
                    if (idle) return;
                    wait(&bar.pv_done[x], n_pv & 1, dead);
                    ++n_pv;
                    idle = true;
                    tmem_fence_after();
                };
                if (__any_sync(0xffffffffu, top > m)) {
                    const float m1 = fmaxf(m, top + kLazy), al = m == -INFINITY ? 0.f : ex2(m - m1);
                    if (on && fabsf(m1) > kFar && fabsf(m1) < INFINITY) far[slot][x] = 1;
                    m = m1;
                    l2 = make_float2(l2.x * al, l2.y * al);
                    if (j > 0) {   // (few columns at a time: the scores are in registers)
                        pv_done();
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(tO + 16 * c, o);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * al);
                            tmem_st16(tO + 16 * c, o);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.f : m;
                uint32_t p[2][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) exponentials(r[c], f2, make_float2(-base, -base), l2, &p[c / 2][c % 2 * 16]);
                pv_done();
                tmem_st32(tP, p[0]);
                tmem_st32(tP + 32, p[1]);
                tmem_wait_st();
                tmem_fence_before();
                mbar_arrive(&bar.p_full[x]);
            }
            if (dead) break;
            if (n > 0) {
                wait(&bar.pv_done[x], n_pv & 1, dead);
                ++n_pv;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.rows_done[x]);             // (`far` is known; not a barrier without a limit)
            wait(&bar.checked[slot][kPart - 1], (t >> 1) & 1, dead);   // (the last of them)
            wait(&bar.rows_done[x], t & 1, dead);
            if (dead) break;
            tmem_fence_after();
            if (redo[slot][x] | far[slot][x]) {
                for (int r = warp & 3; r < it.tokens[x] * G; r += 4) plain_row<D>(a, it.s, it.q0 + x * NT + r / G, it.head, r % G);
            } else {
                const float l = l2.x + l2.y, inv = vis > 0 ? 1.f / l : 0.f;   // (scores that are all -inf: NaN, 0 * inf)
                const int at_row = (int)((it.s.begin + tok) * a.q_heads + it.head * G + g);   // (below 2^30)
                // Rows go out by four lanes at a time, 64 or 32 bytes of a row together: a store by a lane for its own row
                // takes a cycle of the memory pipe for each of 32 lines (4,000 for both tiles).
                const unsigned rows_on = __ballot_sync(0xffffffffu, on) >> (lane & ~3);
                uint32_t scales = 0;
                // (a loop: unrolled, its instructions come from beyond the cache each time)
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    uint32_t o[32];
                    if (n > 0) {
                        tmem_ld32(tO + 32 * c, o);
                        tmem_wait_ld();
                    }
                    float v[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = n > 0 && vis > 0 ? __uint_as_float(o[e]) * inv : 0.f;
                    if (a.o.mx.q != nullptr) {
                        float amax = 0.f;
#pragma unroll
                        for (int e = 0; e < 32; ++e) amax = fmaxf(amax, fabsf(v[e]));
                        const int E = mx_exp(amax, a.o.mx.mode);
                        const float k = __uint_as_float((uint32_t)(127 - E) << 23);
                        uint32_t u[4][2];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            u[e / 2][e % 2] = (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * e] * k, v[4 * e + 1] * k), __NV_SATFINITE, __NV_E4M3) |
                                              (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[4 * e + 2] * k, v[4 * e + 3] * k), __NV_SATFINITE, __NV_E4M3) << 16;
                        scales |= (uint32_t)(E + 127) << (8 * c);
                        transpose4(u);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int at = __shfl_sync(0xffffffffu, at_row, (lane & ~3) | r);
                            if (rows_on >> r & 1u) *reinterpret_cast<uint2 *>(a.o.mx.q + at * (int64_t)D + 32 * c + (lane & 3) * 8) = make_uint2(u[r][0], u[r][1]);
                        }
                        __syncwarp();
                    }
                    if (a.o.out != nullptr) {
                        uint32_t u[4][4];
#pragma unroll
                        for (int e = 0; e < 16; ++e) u[e / 4][e % 4] = pack2_rn(v[2 * e], v[2 * e + 1]);
                        transpose4(u);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const int at = __shfl_sync(0xffffffffu, at_row, (lane & ~3) | r);
                            if (rows_on >> r & 1u)
                                *reinterpret_cast<uint4 *>(a.o.out + at * (int64_t)D + 32 * c + (lane & 3) * 8) = make_uint4(u[r][0], u[r][1], u[r][2], u[r][3]);
                        }
                        __syncwarp();
                    }
                }
                if (on && a.o.mx.q != nullptr) {  // the head's blocks lie next to each other in a scale tile
                    uint8_t *p = a.o.mx.scale + mx_scale_offset(it.s.begin + tok, (it.head * G + g) * (D / 32), a.q_heads * D);
                    if constexpr (D == 128) *reinterpret_cast<uint32_t *>(p) = scales;
                    else *reinterpret_cast<uint16_t *>(p) = (uint16_t)scales;
                }
                if (on && a.o.lse != nullptr) a.o.lse[at_row] = vis > 0 ? (m + log2f(l)) * kLn2 : -INFINITY;
            }
            tmem_fence_before();
            leave(t);
        }
        finish();
        return;
    }
    fewer_registers<88>();
    if (warp == kMmaWarp) {
        // ---- S = Q K^T: A's, B's, A's ... as soon as the one before has been taken
        constexpr uint32_t id = idesc_bf16_f32(128, kKeys);
        uint32_t use0 = 0, n_q = 0, n_s = 0;  // uses of the ring before this item; items with copies, scores so far
        for (int t = 0; take(t); leave(t), ++t) {
            const Item &it = items[t & 1];
            const int n_tiles = it.n_tiles, tiles[2] = {it.tiles[0], it.tiles[1]};
            if (n_tiles == 0) continue;
            wait(&bar.q_full, n_q & 1, dead);
            ++n_q;
            for (int j = 0; j < n_tiles; ++j) {
                const uint32_t use = use0 + 2 * j, k = smem_u32(ring + Ring::stage(use) * C::kTile);
                wait(&bar.kv_full[Ring::full(use)], Ring::full_parity(use), dead);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (j >= tiles[x]) continue;
                    if (n_s > 0) wait(&bar.s_taken, (n_s - 1) & 1, dead);
                    ++n_s;
                    if (dead) break;
                    tmem_fence_after();
                    const uint32_t q = smem_u32(sQ + x * C::kTile);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = (kk / 4) * C::kHalf + (kk % 4) * 32;
                            umma_ss(tm, sdesc_kmajor_sw128(q + o, 1024), sdesc_kmajor_sw128(k + o, 1024), id, kk > 0);
                        }
                        umma_commit(&bar.s_full[x]);
                    }
                    __syncwarp();
                    issued = true;
                }
                if (dead) break;
                if (elect_one()) {
                    umma_commit(&bar.kv_empty[Ring::stage(use)]);
                    if (j == n_tiles - 1) umma_commit(&bar.q_empty);
                }
                __syncwarp();
            }
            use0 += 2 * n_tiles;
            if (dead) break;
        }
    } else if (warp == kMmaWarp + 1) {
        // ---- O += P V
        constexpr uint32_t id = idesc_bf16_f32(128, D) | (1u << 16);   // (V: N contiguous)
        uint32_t use0 = 0, n_p[2] = {0, 0};
        for (int t = 0; take(t); leave(t), ++t) {
            const Item &it = items[t & 1];
            const int n_tiles = it.n_tiles, part = it.part, tiles[2] = {it.tiles[0], it.tiles[1]};
            for (int j = 0; j < n_tiles; ++j) {
                const uint32_t use = use0 + 2 * j + 1, v = smem_u32(ring + Ring::stage(use) * C::kTile);
                wait(&bar.kv_full[Ring::full(use)], Ring::full_parity(use), dead);
                if (j >= part) wait(&bar.checked[t & 1][j - part], (t >> 1) & 1, dead);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    if (j >= tiles[x]) continue;
                    wait(&bar.p_full[x], n_p[x] & 1, dead);
                    ++n_p[x];
                    if (dead) break;
                    tmem_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < kKeys / 16; ++kk)
                            umma_tmemA(tm + 256 + x * 128, tm + 128 + x * 64 + kk * 8, sdesc_v(v + kk * 2048, C::kHalf), id, j > 0 || kk > 0);
                        umma_commit(&bar.pv_done[x]);
                    }
                    __syncwarp();
                    issued = true;
                }
                if (dead) break;
                if (elect_one()) umma_commit(&bar.kv_empty[Ring::stage(use)]);
                __syncwarp();
            }
            use0 += 2 * n_tiles;
            if (dead) break;
        }
    } else if (warp == kLoadWarp) {
        // ---- copies, and the items
        unsigned block = blockIdx.x;
        bool more = true, asked = false;
        uint32_t use = 0, n_q = 0;
        int t = 0;
        for (;; ++t) {
            const int slot = t & 1;
            wait(&bar.item_empty[slot], ((t >> 1) & 1) ^ 1, dead);
            if (dead) break;
            Item it{};
            if (more) it = locate(a, block, gridDim.x, NT);
            if (lane == 0) {
                items[slot] = it;
                redo[slot][0] = redo[slot][1] = far[slot][0] = far[slot][1] = 0;
                mbar_arrive(&bar.item_full[slot]);
            }
            __syncwarp();
            if (!more) break;
            if (lane < kPart && it.part + lane >= it.n_tiles) mbar_arrive(&bar.go[slot][lane]);   // (a phase of each with every item)
            __syncwarp();
            if (elect_one()) {  // a block that has not begun is taken over, if there is one: the next item
                fence_proxy_async_smem();
                mbar_arrive_expect_tx(&bar.next, 16);
                asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(smem_u32(&answer)),
                             "r"(smem_u32(&bar.next))
                             : "memory");
            }
            __syncwarp();
            asked = true;
            if (it.n_tiles > 0) {
                wait(&bar.q_empty, (n_q & 1) ^ 1, dead);
                if (dead) break;
                ++n_q;
                if (elect_one()) {
                    mbar_arrive_expect_tx(&bar.q_full, (uint32_t)(2 * C::NH * NT * G * 128));
                    for (int x = 0; x < 2; ++x)
                        for (int h = 0; h < C::NH; ++h)
                            tma_load_4d(sQ + x * C::kTile + h * C::kHalf, &maps.q, 64 * h, 0, it.head, (int)(it.s.begin + it.q0 + x * NT), &bar.q_full);
                }
                __syncwarp();
                for (int i = 0; i < 2 * it.n_tiles; ++i, ++use) {
                    const uint32_t st = Ring::stage(use);
                    uint64_t *full = &bar.kv_full[Ring::full(use)];
                    wait(&bar.kv_empty[st], Ring::empty_parity(use) ^ 1, dead);   // (the release of the use ST before)
                    if (dead) break;
                    if (elect_one()) {
                        mbar_arrive_expect_tx(full, C::kTile);
                        for (int h = 0; h < C::NH; ++h)
                            tma_load_3d(ring + st * C::kTile + h * C::kHalf, i & 1 ? &maps.v : &maps.k, 64 * h, it.head, (int)(it.s.k0 + (i / 2) * kKeys), full);
                        if ((i & 1) && i / 2 >= it.part) mbar_arrive(&bar.go[slot][i / 2 - it.part]);
                    }
                    __syncwarp();
                }
                if (dead) break;
            }
            wait(&bar.next, t & 1, dead);
            if (dead) break;
            asked = false;
            uint32_t ok, first;
            asm volatile(
                "{\n .reg .b128 h;\n .reg .pred p;\n ld.shared.b128 h, [%2];\n"
                " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
                " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n}\n"
                : "=r"(ok), "=r"(first)
                : "r"(smem_u32(&answer))
                : "memory");
            more = ok != 0;
            block = first;
            __syncwarp();
        }
        // the last releases, which nobody else waits for, have to arrive before the CTA's shared memory goes
        for (uint32_t u = use > (uint32_t)C::ST ? use - C::ST : 0; u < use && !dead; ++u) wait(&bar.kv_empty[Ring::stage(u)], Ring::empty_parity(u), dead);
        if (n_q > 0 && !dead) wait(&bar.q_empty, (n_q - 1) & 1, dead);
        if (dead) {  // and what was asked for has to land
            bool d = false;
            for (uint32_t u = use > (uint32_t)C::ST ? use - C::ST : 0; u < use; ++u) wait(&bar.kv_full[Ring::full(u)], Ring::full_parity(u), d);
            if (n_q > 0) wait(&bar.q_full, (n_q - 1) & 1, d);
            if (asked) wait(&bar.next, t & 1, d);
        }
    } else {
        // ---- what else V's tiles hold that some row sees only in part
        uint32_t use0 = 0;
        for (int t = 0; take(t); leave(t), ++t) {
            const Item &it = items[t & 1];
            for (int k = 0; k < kPart; ++k) {
                const int j = it.part + k;
                if (j < it.n_tiles) {
                    const uint32_t use = use0 + 2 * j + 1;
                    wait(&bar.go[t & 1][k], (t >> 1) & 1, dead);   // (its copy is the barrier's present phase)
                    wait(&bar.kv_full[Ring::full(use)], Ring::full_parity(use), dead);
                    if (dead) break;
                    uint8_t *v = ring + Ring::stage(use) * C::kTile;
                    const int rows = min(kKeys, it.seen - j * kKeys);
                    if (rows < kKeys) {   // rows that none sees, or behind the sequence
                        for (int h = 0; h < C::NH; ++h)
                            for (int o = rows * 128 + lane * 16; o < C::kHalf; o += 512) *reinterpret_cast<uint4 *>(v + h * C::kHalf + o) = make_uint4(0, 0, 0, 0);
                        fence_proxy_async_smem();
                    }
                    auto not_finite = [&](int from) {   // of the rows from .. rows - 1, by each lane's part of them
                        uint32_t bad = 0;
                        for (int h = 0; h < C::NH; ++h)
#pragma unroll 4
                            for (int o = from * 128 + lane * 16; o < rows * 128; o += 512) {
                                const uint4 w = *reinterpret_cast<const uint4 *>(v + h * C::kHalf + o);
                                // an exponent of all ones carries into the sign's place
                                bad |= ((w.x & 0x7f807f80u) + 0x00800080u) | ((w.y & 0x7f807f80u) + 0x00800080u) | ((w.z & 0x7f807f80u) + 0x00800080u) |
                                       ((w.w & 0x7f807f80u) + 0x00800080u);
                            }
                        return (bad & 0x80008000u) != 0;
                    };
                    if (__any_sync(0xffffffffu, not_finite(0)))
                        for (int x = 0; x < 2; ++x)   // which tile has rows that do not see it
                            if (j < it.tiles[x] && not_finite(max(0, it.first[x] - j * kKeys))) redo[t & 1][x] = 1;
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&bar.checked[t & 1][k]);
                __syncwarp();
            }
            use0 += 2 * it.n_tiles;
            if (dead) break;
        }
    }
    if (dead && issued) {  // the products in flight must end before their operands and accumulators go
        if (elect_one()) umma_commit(&bar.drained[warp - kMmaWarp]);
        __syncwarp();
        bool d = false;
        wait(&bar.drained[warp - kMmaWarp], 0, d);
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
    const int64_t pairs = a.Tq / (2 * NT) + a.B;   // places (locate): the lengths are on the device
    mark_main_kernel(stream, true);
    kern<<<(unsigned)(pairs * a.kv_heads), kThreads, C::kSmem, stream>>>(maps, a);
    mark_main_kernel(stream, false);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, cudaStream_t stream) {
    return a.D == 128 ? launch_one<128>(a, stream) : launch_one<64>(a, stream);
}

}  // namespace mhc
