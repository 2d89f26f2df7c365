// Attention of a sequence's last tokens (one, or the few of a speculative-verify block) over its 4-bit cache.
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = 2^(s_j - m),  s_j = sm_scale log2(e) <q, k_j>,  m the largest s so far
//
// The cache is read once (17/32 byte a value): that is the floor, and what must not be in its way are the conversions,
// about three instructions for every four codes.  The keys of all (sequence, kv head) pairs are one long line of slices of
// 32 tokens, cut into equal shares whatever the lengths (the host knows none of them), a share for each warp of one CTA an
// SM.  A warp keeps its own running maximum, sum and accumulators, and its copies run ahead into its own ring in shared
// memory: no two warps wait for each other.  A pair that lies in one share is finished there; of the others each share
// leaves its part in the workspace, and a second kernel joins them.
//
// The rows of a pair are the tokens times the heads of the group, in tiles of 8, 16 or 24.  A warp computes, on the legacy
// tensor path (operands from registers: the codes are converted there and never written back),
//   S^T [32 tokens x rows] = K Q^T   m16n8k16, fp16: E2M1 codes are exact there, and so is q with its largest of 32 values
//                                    in [8, 16) down to 2^-20 of that (what lies lower is off by at most 2^-28 of it);
//                                    each 32 values' sum is multiplied by q's unit and K's scale in fp32, so that a small
//                                    block of q beside a large one of K counts in full (two sums at once: 64 sequences
//                                    below in 114.1 us, with one unit a row 114.6; head_dim 64 32.5 against 31.6)
//   O^T [D x rows] += V^T P'^T       with V's codes, and P' = p * 2^(scale - largest scale that the row saw so far) in fp16 (2^-11 of p, and
//                                    2^-36 of the largest p; scales below 2^-27 of the largest are lost, as they are in fp32
//                                    beside that largest)
// The k order of a product is free: a lane takes 8 neighbouring codes of K (ldmatrix), and 4 of V for two tokens
// (ldmatrix.trans), as they lie; q and the output follow that order.  P crosses from one product's layout to the other's
// by movmatrix.
//
// Measured (in a graph): 64 sequences of 100 to 16,000 tokens, 64 / 8 heads of 128: 110 us, 76 % of the copy rate (at 118 us
// the copies alone took 98, the arithmetic alone 103: about 600 instructions a slice, half of them on the ALU pipe, which is
// 64 % busy); 32,003 tokens, 6 queries of 56 / 8 heads: 38 us, the conversions, which each row tile does anew, by two warps
// a scheduler with no pipe full (ALU 39 %, tensor 30 %); 3 sequences of 60,001 to 131,000, 32 / 4 heads of 64: 29 us, 37 %,
// no pipe full either (ALU 53 %, issue 59 %, DRAM 36 %): the latency of 12 warps with half the bytes a slice, and the
// join behind them.
#include "attention.cuh"
#include "mhc.h"
#include "sm100_ptx.cuh"

namespace mhc {
namespace {

using namespace ptx;

constexpr int kMaxCtas = 160;
constexpr int kSlice = 32;        // tokens
// p = 2^(s - m) with m set kHead (log2) below the largest score, and raised when a score is kHead + kLazy above it (few
// rescales): p is at most 2^12, P' = p * 2^(scale - top + kGain) at most 2^15 (fp16 ends at 2^16).  p loses bits below
// 2^-14, that is 2^-25 of the largest, and is off by at most 2^-36 of it there.
constexpr float kHead = 11.f, kLazy = 1.f;
constexpr int kGain = 3;
// What a pair costs besides its slices, in slices (its q, its join): 100-token sequences beside long ones.
constexpr int kPairCost = 3;

// The workspace after its control block: where each sequence begins on the line and the line's length (int64 [B + 1]), then
// the parts, two for each share (of a pair that began in an earlier share, and of one that goes on in a later one): their
// sums [row][D], and each row's maximum and sum.
constexpr size_t kStartBytes = (MHC_MAX_SEQUENCES + 2) * 8;
constexpr int kFewRows = 1024;          // rows of a call up to which eight warps join one (of 1,824 parts and 8 to a pair's rows, 8 each)
constexpr size_t kPartFloats = 144 * (128 + 2);   // of all shares of a CTA: 144 rows of D = 128, 192 of D = 64

template <int D, int ROWS_, int NW_, int ST_>
struct Cfg {
    static constexpr int ROWS = ROWS_, NW = NW_, ST = ST_;         // rows of a warp, warps, ring stages of a warp
    static constexpr int NT = NW * 32, NB = D / 32, NTILE = ROWS / 8;
    static constexpr int kSliceBytes = 2 * CacheLayout<D>::kGroupBytes;
    static constexpr int kRing = NW * ST * kSliceBytes;
    static constexpr int kScale = NW * kSlice * NB * 6;            // a slice's scales, K's in fp32, V's in fp16: a warp's own
    static constexpr int kQ = ROWS > 8 ? NW * (D / 16) * NTILE * 32 * 8 : 0;   // q's fragments
    static constexpr int kUnits = NW * NB * ROWS * 4;              // the units of q's blocks
    static constexpr int kSmem = kRing + kScale + kQ + kUnits;
    static_assert(kSmem <= 226000 && NW * ROWS * (D + 2) <= kPartFloats, "");
};

// The parts of a launch.
struct Parts {
    int64_t *start;       // [B + 1]
    float *o, *ml;        // [2 * units][rows][D], [2 * units][rows][2]
};
template <int D, class C>
__host__ __device__ __forceinline__ Parts parts_of(unsigned int *ctrl, int ctas) {
    uint8_t *p = reinterpret_cast<uint8_t *>(ctrl) + kControlBytes;
    float *o = reinterpret_cast<float *>(p + kStartBytes);
    return {reinterpret_cast<int64_t *>(p), o, o + (size_t)2 * ctas * C::NW * C::ROWS * D};
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool kTrans, int kAt>
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
    if constexpr (kTrans)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4 + %5];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr), "n"(kAt));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4 + %5];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr), "n"(kAt));
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t d;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {  // of an 8 x 8 matrix of halves
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
    return d;
}
__device__ __forceinline__ uint32_t mul_half2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ float quad_max(float v) {   // over the lanes of a group of four
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float column_max(float v) { // over the lanes with the same place in their group of four
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ float column_sum(float v) {
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// Two scale bytes as fp32 (0 is 2^-127, 255 NaN): the hardware's conversion to bf16, widened.
__device__ __forceinline__ float2 ue8m0x2(uint32_t bytes) {
    uint32_t d;
    asm("{ .reg .b16 t; cvt.u16.u32 t, %1; cvt.rn.bf16x2.ue8m0x2 %0, t; }" : "=r"(d) : "r"(bytes));
    return make_float2(__uint_as_float(d << 16), __uint_as_float(d & 0xffff0000u));
}
constexpr uint32_t kNormal = 15 + kGain;   // scale bytes whose factor is a normal half: the largest one's exponent field
// 2^(byte - top + kGain) as fp16 bits, byte <= top: zero below 2^-24, NaN for 255.
__device__ __forceinline__ uint32_t v_scale(uint32_t byte, uint32_t top) {
    const int e = (int)byte - (int)top + 15 + kGain;
    return byte == 255u ? 0x7fffu : e >= 1 ? (uint32_t)e << 10 : e > -10 ? 0x400u >> (1 - e) : 0u;
}

// What is to be done: a sequence's geometry, and a CTA's place on the line.
struct Seq {
    int64_t begin;      // first packed row
    int n, len;         // packed rows; tokens in the cache (at most one past what the table holds for each packed row)
    int tiles, slices;  // row tiles of a kv head; slices of a pair
};

__device__ __forceinline__ Seq sequence(const DecodeArgs &a, int rows, int b) {
    Seq s;
    const int64_t lo = clamp_row(__ldg(a.c.offsets + b), a.T), hi = clamp_row(__ldg(a.c.offsets + b + 1), a.T);
    s.begin = lo;
    s.n = hi > lo ? (int)(hi - lo) : 0;
    // lengths beyond the table: positions from its end on are NaN, so no more of them are needed than rows
    const int64_t room = (int64_t)a.c.width << a.c.page_log2;
    s.len = (int)max((int64_t)0, min((int64_t)__ldg(a.c.seq_lens + b), room + s.n));
    s.tiles = (int)(((int64_t)s.n * (a.q_heads / a.c.heads) + rows - 1) / rows);
    s.slices = max(1, (s.len + kSlice - 1) / kSlice);
    return s;
}
// On the line a pair is kPairCost places, then its slices.
__device__ __forceinline__ int64_t cost(const DecodeArgs &a, const Seq &s) { return (int64_t)a.c.heads * s.tiles * (s.slices + kPairCost); }

// A share's length: at least two places.
__device__ __forceinline__ int64_t share_of(int64_t total, int64_t units) { return max((int64_t)2, (total + units - 1) / units); }

template <int D, class C>
struct Warp {                              // a warp's running state
    float o[C::NB][2][C::NTILE][4];        // O^T: per 32 values two tiles of 16, per 8 rows
    float m[C::NTILE][2], l[C::NTILE][2];  // rows 2 (lane % 4) and the next: reference maximum, sum of the lane's own tokens
    uint32_t top, low;                     // V's largest scale byte so far: o is in units of 2^(top - 127 - kGain), or of
                                           // what it was when a row saw its last token (own); the smallest byte whose
                                           // factor is a normal half
};

// 16 tokens' codes (half kHalf of a slice) of K or V (kPart): r0 the first 8 tokens', r1 the others', a block each.
// codes: the slice's address and lane_codes().
template <int D, int kPart, int kHalf>
__device__ __forceinline__ void fetch(uint32_t codes, uint32_t (&r0)[D / 32], uint32_t (&r1)[D / 32]) {
    using L = CacheLayout<D>;
    constexpr int kAt = kHalf * L::kGroupBytes + kPart * L::kPart;
    uint32_t r[4];
    ldsm4<kPart == 1, kAt>(r, codes);
    if constexpr (D == 128) {
#pragma unroll
        for (int b = 0; b < 4; ++b) r0[b] = r[b];
        ldsm4<kPart == 1, kAt + 8 * L::kRow>(r, codes);
#pragma unroll
        for (int b = 0; b < 4; ++b) r1[b] = r[b];
    } else {
        r0[0] = r[0]; r0[1] = r[1]; r1[0] = r[2]; r1[1] = r[3];
    }
}
// Where a lane's row of such a load lies: matrices are the blocks of 8 tokens, or of 8 and the next 8 for D = 64 (rows 8
// apart have the same chunk order).
template <int D>
__device__ __forceinline__ uint32_t lane_codes() {
    using L = CacheLayout<D>;
    const int lane = threadIdx.x & 31, mi = lane >> 3;
    const int row = (lane & 7) + (D == 128 ? 0 : (mi >> 1) * 8), blk = D == 128 ? mi : mi & 1;
    return row * L::kRow + (blk ^ L::swizzle(row)) * 16;
}

// V's scale bytes of a token (the lane's) of a slice.
template <int D, int NB>
__device__ __forceinline__ uint32_t v_scales(uint32_t base) {
    using L = CacheLayout<D>;
    const uint32_t at = base + ((threadIdx.x & 31) >> 4) * L::kGroupBytes + L::kScales + (threadIdx.x & 15) * NB;
    uint32_t vw;
    if constexpr (NB == 4) asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(vw) : "r"(at), "n"(L::kPart));
    else asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=r"(vw) : "r"(at), "n"(L::kPart));
    return vw;
}
// The largest of a lane's scale bytes that is a number.
template <int NB>
__device__ __forceinline__ uint32_t largest_scale(uint32_t vw) {
    uint32_t mine = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const uint32_t e = (vw >> (8 * b)) & 255u;
        mine = max(mine, e == 255u ? 0u : e);
    }
    return mine;
}
// Where a slice's next window ends: at the first token from lo on that not every row with tokens left sees.
template <int NTL>
__device__ __forceinline__ int window_end(const int (&vis_g)[NTL], int lo, int end) {
#pragma unroll
    for (int r = 0; r < NTL; ++r)
        if (vis_g[r] > lo) end = min(end, vis_g[r]);
    return __reduce_min_sync(0xffffffffu, end);
}
// Whether a slice holds a scale above all those that some row with tokens left sees: that row's p would lose bits to a V
// which is none of its own, so such a slice is gone through window by window.
template <int D, int NB, int NTL>
__device__ __forceinline__ bool needs_windows(uint32_t top, uint32_t base, int tok0, int len, uint32_t bad, const int (&vis_g)[NTL]) {
    const int lane = threadIdx.x & 31, all = window_end(vis_g, tok0, tok0 + kSlice);   // (seen by all of those rows)
    const bool on = tok0 + lane < len && !((bad >> (lane >> 4)) & 1u);
    const uint32_t mine = on ? largest_scale<NB>(v_scales<D, NB>(base)) : 0u;
    const uint32_t seen = max(top, __reduce_max_sync(0xffffffffu, tok0 + lane < all ? mine : 0u));
    return __any_sync(0xffffffffu, mine > seen);
}

// A slice of 32 tokens from shared memory.  units: of q's blocks, for rows 2 (lane % 4) and the next; tok0: its first
// token; vis: tokens that those rows see, vis_g: those that row lane / 4 sees; f: the factors of those rows' scores.  With
// kMask only tokens from .. to - 1.
template <int D, class C, bool kMask>
__device__ __forceinline__ void slice(Warp<D, C> &w, uint32_t base, const uint32_t (&q)[C::NB][2][C::NTILE * 2], const uint2 *sq, const float2 *units,
                                      float *sk, uint32_t *sv, uint8_t *own, int tok0, int from, int to, int len, uint32_t bad, const float (&f)[C::NTILE][2],
                                      const int (&vis)[C::NTILE][2], const int (&vis_g)[C::NTILE]) {
    using L = CacheLayout<D>;
    constexpr int NB = C::NB, NTL = C::NTILE;
    const int lane = threadIdx.x & 31, g4 = lane >> 2, t4 = lane & 3;
    const uint32_t codes = base + lane_codes<D>();
    // ---- scales, a token a lane
    uint32_t vw, v_hi, v_lo;   // V's scale bytes, the largest and the smallest of them
    {
        const uint32_t at = base + (lane >> 4) * L::kGroupBytes + L::kScales + (lane & 15) * NB;
        uint32_t kw;
        if constexpr (NB == 4) asm volatile("ld.shared.u32 %0, [%1];" : "=r"(kw) : "r"(at));
        else asm volatile("ld.shared.u16 %0, [%1];" : "=r"(kw) : "r"(at));
        vw = v_scales<D, NB>(base);
        if constexpr (kMask) {
            if ((bad >> (lane >> 4)) & 1u) kw = vw = 0xffffffffu;   // no such page: NaN
            if (tok0 + lane >= min(len, to) || tok0 + lane < from) kw = vw = 0u;   // (what the rest of a page holds; other windows)
        }
        const float2 k01 = ue8m0x2(kw);
        if constexpr (NB == 4) {
            const float2 k23 = ue8m0x2(kw >> 16);
            *reinterpret_cast<float4 *>(sk + lane * 4) = make_float4(k01.x, k01.y, k23.x, k23.y);
            const uint32_t even = vw & 0x00ff00ffu, odd = (vw >> 8) & 0x00ff00ffu, hi = __vmaxu2(even, odd), lo = __vminu2(even, odd);
            v_hi = max(hi & 0xffffu, hi >> 16);
            v_lo = min(lo & 0xffffu, lo >> 16);
        } else {
            *reinterpret_cast<float2 *>(sk + lane * 2) = k01;
            v_hi = max(vw & 255u, (vw >> 8) & 255u);
            v_lo = min(vw & 255u, (vw >> 8) & 255u);
        }
        __syncwarp();
    }
    // ---- scores: s[h][r] holds tokens 16 h + g4 (and + 8) x rows 8 r + 2 t4 (and + 1)
    float s[2][NTL][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t r0[NB], r1[NB];
        if (h == 0) fetch<D, 0, 0>(codes, r0, r1);
        else fetch<D, 0, 1>(codes, r0, r1);
        float sc0[NB], sc1[NB];
#pragma unroll
        for (int b = 0; b < NB; b += (NB == 4 ? 4 : 2)) {
            const float *p0 = sk + (16 * h + g4) * NB, *p1 = p0 + 8 * NB;
            if constexpr (NB == 4) {
                const float4 u = *reinterpret_cast<const float4 *>(p0), v = *reinterpret_cast<const float4 *>(p1);
                sc0[0] = u.x; sc0[1] = u.y; sc0[2] = u.z; sc0[3] = u.w;
                sc1[0] = v.x; sc1[1] = v.y; sc1[2] = v.z; sc1[3] = v.w;
            } else {
                const float2 u = *reinterpret_cast<const float2 *>(p0), v = *reinterpret_cast<const float2 *>(p1);
                sc0[0] = u.x; sc0[1] = u.y; sc1[0] = v.x; sc1[1] = v.y;
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            const uint32_t a0[4] = {e2m1x2<0>(r0[b]), e2m1x2<0>(r1[b]), e2m1x2<1>(r0[b]), e2m1x2<1>(r1[b])};
            const uint32_t a1[4] = {e2m1x2<2>(r0[b]), e2m1x2<2>(r1[b]), e2m1x2<3>(r0[b]), e2m1x2<3>(r1[b])};
            uint32_t qb[NTL][4];
            if constexpr (NTL == 1) {
                qb[0][0] = q[b][0][0]; qb[0][1] = q[b][0][1]; qb[0][2] = q[b][1][0]; qb[0][3] = q[b][1][1];
            } else {
#pragma unroll
                for (int r = 0; r < NTL; ++r)
#pragma unroll
                    for (int h2 = 0; h2 < 2; ++h2) {
                        const uint2 u = sq[((b * 2 + h2) * NTL + r) * 32 + lane];
                        qb[r][2 * h2] = u.x;
                        qb[r][2 * h2 + 1] = u.y;
                    }
            }
#pragma unroll
            for (int r = 0; r < NTL; ++r) {
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
                mma(acc, a0, qb[r][0], qb[r][1]);
                mma(acc, a1, qb[r][2], qb[r][3]);
                const float2 u = units[(b * NTL + r) * 4];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float k = j ? sc1[b] : sc0[b];
                    const float2 x = __fmul2_rn(make_float2(acc[2 * j], acc[2 * j + 1]), u);
                    const float2 y = b == 0 ? __fmul2_rn(x, make_float2(k, k)) : __ffma2_rn(x, make_float2(k, k), make_float2(s[h][r][2 * j], s[h][r][2 * j + 1]));
                    s[h][r][2 * j] = y.x;
                    s[h][r][2 * j + 1] = y.y;
                }
            }
        }
    }
    // ---- the running maximum
    float hi[NTL][2];
    bool raise = v_hi > w.top || v_lo < w.low;
    bool far = false;          // a V scale is NaN, or too far below the largest to be a normal half
#pragma unroll
    for (int r = 0; r < NTL; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float &x = s[h][r][2 * j + e];
                    x *= f[r][e];
                    if constexpr (kMask) {
                        const int tok = tok0 + 16 * h + 8 * j + g4;
                        if (tok < from || tok >= min(vis[r][e], to)) x = -INFINITY;
                    }
                }
            hi[r][e] = fmaxf(fmaxf(s[0][r][e], s[0][r][2 + e]), fmaxf(s[1][r][e], s[1][r][2 + e]));
            raise |= hi[r][e] > w.m[r][e] + (kHead + kLazy);
        }
    if (__any_sync(0xffffffffu, raise)) {
        const uint32_t top = max(w.top, __reduce_max_sync(0xffffffffu, largest_scale<NB>(vw)));
        w.low = max((int)top - (kNormal - 1), 0);
        far = __any_sync(0xffffffffu, v_hi == 255u || v_lo < w.low);
        const float rise = ex2((float)((int)w.top - (int)top));
        w.top = top;
#pragma unroll
        for (int r = 0; r < NTL; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float m = fmaxf(w.m[r][e], column_max(hi[r][e]) - kHead);
                const float al = w.m[r][e] == -INFINITY ? 0.f : ex2(w.m[r][e] - m);
                const bool on = !kMask || vis[r][e] > from;            // a row that has seen all of its own keeps its unit
                const float unit = on ? rise : 1.f;
                if (on) own[r * 8 + 2 * t4 + e] = (uint8_t)top;
                w.m[r][e] = m;
                w.l[r][e] *= al;
#pragma unroll
                for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        w.o[b][h][r][e] *= al * unit;
                        w.o[b][h][r][2 + e] *= al * unit;
                    }
            }
    }
    // ---- V's scales: word (token pair, block)
    {
        const uint32_t other = __shfl_xor_sync(0xffffffffu, vw, 1);
        const uint32_t even = lane & 1 ? other : vw, odd = lane & 1 ? vw : other;
        uint32_t x[NB / 2];
        if (far) {
#pragma unroll
            for (int i = 0; i < NB / 2; ++i) {   // an even lane writes the first half of the blocks, an odd one the second
                const int sh = 8 * ((lane & 1) * (NB / 2) + i);
                x[i] = v_scale((even >> sh) & 255u, w.top) | v_scale((odd >> sh) & 255u, w.top) << 16;
            }
        } else {  // the same for four bytes at once: each is top - kNormal + 1 .. top, its exponent field 1 .. kNormal
            const uint32_t down = (w.top - kNormal) * 0x01010101u, fe = even - down, fo = odd - down;
#pragma unroll
            for (int i = 0; i < NB / 2; ++i)     // the two bytes to bits 8 and 24, then up by two: a half's exponent
                x[i] = __byte_perm(fe, fo, lane & 1 ? (NB == 4 ? (i ? 0x7030 : 0x6020) : 0x5010) : (i ? 0x5010 : 0x4000)) << 2 & 0x7c007c00u;
        }
        if constexpr (NB == 4) *reinterpret_cast<uint2 *>(sv + (lane >> 1) * 4 + (lane & 1) * 2) = make_uint2(x[0], x[1]);
        else sv[(lane >> 1) * 2 + (lane & 1)] = x[0];
    }
    // ---- exponentials and their sums; p as halves, turned: p16[r][n] is row 8 r + g4, tokens 8 n + 2 t4 (and + 1)
    uint32_t p16[NTL][4];
#pragma unroll
    for (int r = 0; r < NTL; ++r) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float m = w.m[r][e] == -INFINITY ? 0.f : w.m[r][e];
            float sum = 0.f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    s[h][r][2 * j + e] = ex2(s[h][r][2 * j + e] - m);
                    sum += s[h][r][2 * j + e];
                }
            w.l[r][e] += sum;
        }
#pragma unroll
        for (int n = 0; n < 4; ++n) p16[r][n] = transpose8(pack_half(s[n >> 1][r][2 * (n & 1)], s[n >> 1][r][2 * (n & 1) + 1]));
    }
    __syncwarp();
    // ---- O^T += V^T P'^T, 16 tokens at a time
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t v0[NB], v1[NB];
        if (h == 0) fetch<D, 1, 0>(codes, v0, v1);
        else fetch<D, 1, 1>(codes, v0, v1);
        uint32_t sc[2][NB];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const uint32_t *p = sv + (4 * (2 * h + j) + t4) * NB;
            if constexpr (NB == 4) {
                const uint4 u = *reinterpret_cast<const uint4 *>(p);
                sc[j][0] = u.x; sc[j][1] = u.y; sc[j][2] = u.z; sc[j][3] = u.w;
            } else {
                const uint2 u = *reinterpret_cast<const uint2 *>(p);
                sc[j][0] = u.x; sc[j][1] = u.y;
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            uint32_t pb[NTL][2];
#pragma unroll
            for (int r = 0; r < NTL; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    pb[r][j] = mul_half2(p16[r][2 * h + j], sc[j][b]);
                    if constexpr (kMask) {  // (0 times a NaN scale is no part of what a row does not see)
                        const int tok = tok0 + 16 * h + 8 * j + 2 * t4;
                        const int end = min(vis_g[r], to);
                        pb[r][j] &= (tok >= from && tok < end ? 0xffffu : 0u) | (tok + 1 >= from && tok + 1 < end ? 0xffff0000u : 0u);
                    }
                }
            const uint32_t e0 = e2m1x2<0>(v0[b]), e1 = e2m1x2<2>(v0[b]), e2 = e2m1x2<0>(v1[b]), e3 = e2m1x2<2>(v1[b]);
            const uint32_t g0 = e2m1x2<1>(v0[b]), g1 = e2m1x2<3>(v0[b]), g2 = e2m1x2<1>(v1[b]), g3 = e2m1x2<3>(v1[b]);
            const uint32_t a0[4] = {__byte_perm(e0, e1, 0x5410), __byte_perm(e0, e1, 0x7632), __byte_perm(e2, e3, 0x5410), __byte_perm(e2, e3, 0x7632)};
            const uint32_t a1[4] = {__byte_perm(g0, g1, 0x5410), __byte_perm(g0, g1, 0x7632), __byte_perm(g2, g3, 0x5410), __byte_perm(g2, g3, 0x7632)};
#pragma unroll
            for (int r = 0; r < NTL; ++r) {
                mma(w.o[b][0][r], a0, pb[r][0], pb[r][1]);
                mma(w.o[b][1][r], a1, pb[r][0], pb[r][1]);
            }
        }
    }
}

struct Pair {
    Seq seq;
    int b, pair;             // sequence; head * tiles + row tile
    int s0, count;           // first place (slices from 0; below 0: the pair's own cost), places in this share
    int first, n, limit;     // first slice and number of slices; tokens up to the last
    const uint8_t *src;      // the head in page 0
};

template <int D, class C>
__global__ void __launch_bounds__(C::NT, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
    using L = CacheLayout<D>;
    constexpr int NB = C::NB, NTL = C::NTILE, NW = C::NW, ST = C::ST, NT = C::NT;
    extern __shared__ __align__(128) uint8_t smem[];
    uint8_t *ring = smem;
    float *scale = reinterpret_cast<float *>(smem + C::kRing);
    uint2 *sq = reinterpret_cast<uint2 *>(smem + C::kRing + C::kScale);
    __shared__ int64_t scan[34];
    __shared__ int64_t found[NW][2];
    __shared__ Pair pairs[C::NW][2];           // a warp's present pair and its next one (in registers they cost the slices theirs)
    __shared__ int2 look[C::NW][32];           // the next one's first pages
    __shared__ uint8_t own[C::NW][C::ROWS];    // the rows' units (Warp)
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g4 = lane >> 2, t4 = lane & 3;
    const int G = a.q_heads / a.c.heads;
    const int unit = (int)blockIdx.x * NW + warp;                      // which share
    const Parts parts = parts_of<D, C>(a.ctrl, gridDim.x);
    asm volatile("griddepcontrol.launch_dependents;");                 // (the second kernel waits for all of this one)

    // ---- the shares of the line: a sequence a thread, the sum of what is before each (for those beyond NT a second time,
    // once the line's length is known)
    int64_t total;
    const int64_t c0 = tid < a.c.B ? cost(a, sequence(a, C::ROWS, tid)) : 0, before0 = block_scan<NT>(c0, total, scan);
    for (int base = NT; base < a.c.B; base += NT) {
        int64_t all;
        block_scan<NT>(base + tid < a.c.B ? cost(a, sequence(a, C::ROWS, base + tid)) : 0, all, scan);
        total += all;
    }
    const int64_t share = share_of(total, (int64_t)gridDim.x * NW);
    {
        const int64_t first = share * blockIdx.x * NW;
        auto place = [&](int b, int64_t mine, int64_t c) {  // sequence b is on the line from `mine` on: whose shares begin there
            for (int w = 0; w < NW; ++w)
                if (first + w * share >= mine && first + w * share < mine + c) {
                    found[w][0] = b;
                    found[w][1] = first + w * share - mine;
                }
            if (blockIdx.x == 0 && b < a.c.B) parts.start[b] = mine;
        };
        place(tid, before0, c0);
        int64_t before = 0;
        for (int base = 0; base < a.c.B && a.c.B > NT; base += NT) {
            int64_t all;
            const int b = base + tid;
            const int64_t c = b < a.c.B ? cost(a, sequence(a, C::ROWS, b)) : 0, mine = before + block_scan<NT>(c, all, scan);
            if (base > 0) place(b, mine, c);
            before += all;
        }
        if (blockIdx.x == 0 && tid == 0) parts.start[a.c.B] = total;
    }
    __syncthreads();
    int64_t at = share * unit;
    const int64_t end = min(total, at + share);
    if (at >= end) return;
    // (from here on no barrier of the CTA)

    // ---- a pair, and a share's part of it
    auto part_of = [&](Pair &p, int64_t left) {
        p.count = (int)min((int64_t)(p.seq.slices - p.s0), left);
        p.first = max(p.s0, 0);
        p.n = max(0, p.s0 + p.count - p.first);
        p.limit = min(p.seq.len, (p.first + p.n) * kSlice);
        p.src = a.c.data + (int64_t)(p.pair / p.seq.tiles) * (a.c.page >> 4) * L::kGroupBytes;
    };
    auto pages_of = [&](const Pair &p, int k, int (&page)[2]) {  // of slice k of the part, a slice a lane
        const int64_t t0 = (int64_t)(p.first + k) * kSlice;
#pragma unroll
        for (int i = 0; i < 2; ++i) page[i] = k < p.n && t0 + 16 * i < p.limit ? cache_page(a.c, p.b, t0 + 16 * i) : -1;
    };

    // ---- the ring
    uint32_t put = 0, got = 0;                                         // slices copied to and taken from it
    int page_cur[2], page_next[2] = {-1, -1};                                     // pages of slices k0 + lane, and the 32 after
    int copied = 0;                                                    // slices of this part whose copy was started
    uint32_t bad_pages = 0;                                            // two bits a copied slice, the last one's lowest
    const int page_bytes = a.c.heads * (a.c.page >> 4) * L::kGroupBytes;
    auto copy = [&](const Pair &p) {  // starts the next slice's copy, or an empty group
        if (copied < p.n) {
            if ((copied & 31) == 0 && copied > 0) {
                page_cur[0] = page_next[0];
                page_cur[1] = page_next[1];
                pages_of(p, copied + 32 + lane, page_next);
            }
            const int t0 = (p.first + copied) * kSlice;
            const int p0 = __shfl_sync(0xffffffffu, page_cur[0], copied & 31), p1 = __shfl_sync(0xffffffffu, page_cur[1], copied & 31);
            constexpr int kChunks = L::kGroupBytes / 16, kRound = kChunks / 32 * 32;   // whole warps' rounds, then both groups' rest
            constexpr int kRest = kChunks - kRound;                                     // 8 or 4: lanes 0 .. for the first group, then the second
            static_assert(2 * kRest <= 32, "");
            const uint32_t dst = smem_u32(ring + (warp * ST + put % ST) * C::kSliceBytes) + lane * 16;
            const uint8_t *src0 = p.src + lane * 16 + (int64_t)p0 * page_bytes + ((t0 & (a.c.page - 1)) >> 4) * L::kGroupBytes;
            const uint8_t *src1 = p.src + lane * 16 + (int64_t)p1 * page_bytes + (((t0 + 16) & (a.c.page - 1)) >> 4) * L::kGroupBytes;
            bad_pages = bad_pages << 2 | (p0 < 0 ? 1u : 0u) | (p1 < 0 ? 2u : 0u);
            if ((p0 | p1) >= 0) {
#pragma unroll
                for (int i = 0; i < kRound * 16; i += 512) {
                    cp_async16(dst + i, src0 + i);
                    cp_async16(dst + i + L::kGroupBytes, src1 + i);
                }
                if (lane < 2 * kRest)
                    cp_async16(dst + kRound * 16 + (lane < kRest ? 0 : L::kGroupBytes - kRest * 16), (lane < kRest ? src0 : src1 - kRest * 16) + kRound * 16);
            } else if (p0 >= 0 || p1 >= 0) {
                const uint8_t *src = p0 >= 0 ? src0 : src1;
                for (int i = 0; i < L::kGroupBytes; i += 512)
                    if (i + lane * 16 < L::kGroupBytes) cp_async16(dst + i + (p0 >= 0 ? 0 : L::kGroupBytes), src + i);
            }
            ++put;
            ++copied;
        }
        cp_commit();
    };
    uint4 qw[NTL][NB];                                                 // q of the lane's rows, 8 values of each block
    auto load_q = [&](const Pair &p) {
        const int row0 = (p.pair % p.seq.tiles) * C::ROWS, rows = min(C::ROWS, p.seq.n * G - row0), head = p.pair / p.seq.tiles;
#pragma unroll
        for (int r = 0; r < NTL; ++r) {
            const int row = r * 8 + g4, i = (row0 + row) / G;
            const uint16_t *x = a.q + (p.seq.begin + i) * a.q_stride + (head * G + (row0 + row) % G) * D + t4 * 8;
#pragma unroll
            for (int k = 0; k < NB; ++k) qw[r][k] = row < rows ? __ldg(reinterpret_cast<const uint4 *>(x + k * 32)) : make_uint4(0, 0, 0, 0);
        }
    };
    auto begin = [&](const Pair &p) {  // its pages known (page_cur)
        copied = 0;
        pages_of(p, 32 + lane, page_next);
        if constexpr (NTL == 1) load_q(p);
#pragma unroll
        for (int i = 0; i < ST - 1; ++i) copy(p);
    };

    int now = 0;
    {
        Pair p;
        p.b = (int)found[warp][0];
        p.seq = sequence(a, C::ROWS, p.b);
        p.pair = (int)(found[warp][1] / (p.seq.slices + kPairCost));
        p.s0 = (int)(found[warp][1] % (p.seq.slices + kPairCost)) - kPairCost;
        part_of(p, end - at);
        pages_of(p, lane, page_cur);
        if (lane == 0) pairs[warp][0] = p;
        __syncwarp();
        begin(p);
    }
    while (true) {
        const Pair &cur = pairs[warp][now];
        // ---- what comes next, ahead of its use
        at += cur.count;
        const bool more = at < end;
        if (more) {
            Pair next = cur;
            next.s0 = -kPairCost;
            if (++next.pair == a.c.heads * next.seq.tiles) {
                next.pair = 0;
                do next.seq = sequence(a, C::ROWS, ++next.b);
                while (next.seq.n == 0);
            }
            part_of(next, end - at);
            int page_look[2];
            pages_of(next, lane, page_look);
            look[warp][lane] = make_int2(page_look[0], page_look[1]);
            if (lane == 0) pairs[warp][now ^ 1] = next;
            __syncwarp();
        }
        const int row0 = (cur.pair % cur.seq.tiles) * C::ROWS, rows = min(C::ROWS, cur.seq.n * G - row0), head = cur.pair / cur.seq.tiles;
        // ---- q: row lane / 4 (+ 8) as B fragments, each block scaled by a power of two of its own to at most 2^4; its unit is
        // relative to the row's, which the scores are multiplied by at the end
        if constexpr (NTL > 1) load_q(cur);
        float *su = reinterpret_cast<float *>(smem + C::kRing + C::kScale + C::kQ) + warp * (NB * C::ROWS);
        uint32_t q[NB][2][NTL * 2];
        float f[NTL][2];
        int vis[NTL][2], vis_g[NTL];
        int seen = 0x7fffffff;                                         // tokens that every row sees
#pragma unroll
        for (int r = 0; r < NTL; ++r) {
            const int row = r * 8 + g4;
            vis_g[r] = row < rows ? max(0, cur.seq.len - cur.seq.n + (row0 + row) / G + 1) : 0;
            seen = min(seen, row < rows ? vis_g[r] : 0x7fffffff);
            float x[NB][8], amax[NB], most = 0.f;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                unpack8(qw[r][k], x[k]);
                amax[k] = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) amax[k] = fmaxf(amax[k], fabsf(x[k][e]));
                amax[k] = quad_max(amax[k]);
                most = fmaxf(most, amax[k]);
            }
            const int up = min(126, 3 + 127 - (int)(__float_as_uint(most) >> 23));   // the largest * 2^up is in [8, 16)
            const float fg = a.sm_scale * kLog2e * __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                f[r][e] = __shfl_sync(0xffffffffu, fg, 8 * t4 + 4 * e);
                vis[r][e] = __shfl_sync(0xffffffffu, vis_g[r], 8 * t4 + 4 * e);
            }
#pragma unroll
            for (int k = 0; k < NB; ++k) {
                const int own_up = min(min(126, up + 126), 3 + 127 - (int)(__float_as_uint(amax[k]) >> 23));
                const float mul = __uint_as_float((uint32_t)(own_up + 127) << 23);
                if (t4 == k) su[(k * NTL + r) * 8 + g4] = __uint_as_float((uint32_t)(up - own_up + 127) << 23);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    q[k][h][r] = pack_half(x[k][4 * h] * mul, x[k][4 * h + 1] * mul);
                    q[k][h][NTL + r] = pack_half(x[k][4 * h + 2] * mul, x[k][4 * h + 3] * mul);
                }
            }
        }
        seen = __reduce_min_sync(0xffffffffu, seen);
        if constexpr (NTL > 1) {
#pragma unroll
            for (int k = 0; k < NB; ++k)
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int r = 0; r < NTL; ++r) sq[(((warp * NB + k) * 2 + h) * NTL + r) * 32 + lane] = make_uint2(q[k][h][r], q[k][h][NTL + r]);
        }
        __syncwarp();

        Warp<D, C> w;
#pragma unroll
        for (int k = 0; k < NB; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int r = 0; r < NTL; ++r)
#pragma unroll
                    for (int e = 0; e < 4; ++e) w.o[k][h][r][e] = 0.f;
#pragma unroll
        for (int r = 0; r < NTL; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) w.m[r][e] = -INFINITY, w.l[r][e] = 0.f;
        w.top = w.low = 0;
        if (lane < C::ROWS) own[warp][lane] = 0;                       // (a barrier follows before it is used)

        for (int k = 0; k < cur.n; ++k) {
            cp_wait<ST - 2>();
            __syncwarp();                                              // slice k is there for all lanes, and k - 1 is done with
            copy(cur);
            const int stage = warp * ST + got % ST;
            ++got;
            const int tok0 = (cur.first + k) * kSlice;
            const uint32_t base = smem_u32(ring + stage * C::kSliceBytes), bad = bad_pages >> (2 * (copied - 1 - k)) & 3u;
            float *sk = scale + warp * (kSlice * NB * 3 / 2);
            uint32_t *sv = reinterpret_cast<uint32_t *>(sk + kSlice * NB);
            const float2 *units = reinterpret_cast<const float2 *>(su) + t4;
            if (tok0 + kSlice <= seen && bad == 0)
                slice<D, C, false>(w, base, q, sq + warp * (NB * 2 * NTL * 32), units, sk, sv, own[warp], tok0, tok0, tok0 + kSlice, cur.seq.len, bad, f, vis, vis_g);
            else {
                const bool windows = needs_windows<D, NB, NTL>(w.top, base, tok0, cur.seq.len, bad, vis_g);
                for (int lo = tok0, hi; lo < tok0 + kSlice; lo = hi) {
                    hi = windows ? window_end(vis_g, lo, tok0 + kSlice) : tok0 + kSlice;
                    slice<D, C, true>(w, base, q, sq + warp * (NB * 2 * NTL * 32), units, sk, sv, own[warp], tok0, lo, hi, cur.seq.len, bad, f, vis, vis_g);
                    __syncwarp();                                      // (the scales are written anew)
                }
            }
            __syncwarp();
        }
        __syncwarp();                                                  // (every lane has read the last slice)
        // ---- the next pair's first copies run while this one is written
        if (more) {
            page_cur[0] = look[warp][lane].x;
            page_cur[1] = look[warp][lane].y;
            begin(pairs[warp][now ^ 1]);
        }
        const bool whole = cur.s0 == -kPairCost && cur.s0 + cur.count == cur.seq.slices;
        const int slot = 2 * unit + (cur.s0 == -kPairCost ? 1 : 0);
#pragma unroll
        for (int r = 0; r < NTL; ++r)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // row 8 r + 2 t4 + e, values 32 k + 4 g4 ..
                const float l = column_sum(w.l[r][e]);
                const int row = r * 8 + 2 * t4 + e;
                const bool on = row < rows;
                const int e_units = (int)own[warp][row] - kGain;         // 2^(own - 127 - kGain), below 2^-126 too
                const float units = __uint_as_float(e_units > 0 ? (uint32_t)e_units << 23 : 0x00800000u >> (1 - e_units));
                if (!whole) {                                          // divided: the sums may pass fp32's end where V does not
                    const float inv = l == 0.f ? 0.f : 1.f / l;
                    float *o = parts.o + ((size_t)slot * C::ROWS + row) * D + 4 * g4;
                    if (on) {
#pragma unroll
                        for (int k = 0; k < NB; ++k)
                            *reinterpret_cast<float4 *>(o + 32 * k) =
                                make_float4(w.o[k][0][r][e] * inv * units, w.o[k][0][r][2 + e] * inv * units, w.o[k][1][r][e] * inv * units, w.o[k][1][r][2 + e] * inv * units);
                        if (g4 == 0) *reinterpret_cast<float2 *>(parts.ml + ((size_t)slot * C::ROWS + row) * 2) = make_float2(w.m[r][e], l);
                    }
                    continue;
                }
                const int i = (row0 + row) / G, hq = head * G + (row0 + row) % G;
                const bool sees = cur.seq.len - cur.seq.n + i >= 0;    // what sees nothing gives zeros and -inf
                const int64_t t = cur.seq.begin + i;
                const float inv = 1.f / l;                             // (keys whose scores are all -inf: NaN, 0 * inf)
#pragma unroll
                for (int k = 0; k < NB; ++k) {
                    float v[4] = {w.o[k][0][r][e] * inv * units, w.o[k][0][r][2 + e] * inv * units, w.o[k][1][r][e] * inv * units, w.o[k][1][r][2 + e] * inv * units};
                    if (!sees) v[0] = v[1] = v[2] = v[3] = 0.f;
                    const int64_t o = (t * a.q_heads + hq) * (int64_t)D + 32 * k + 4 * g4;
                    if (on && a.o.out != nullptr) *reinterpret_cast<uint2 *>(a.o.out + o) = make_uint2(pack2_rn(v[0], v[1]), pack2_rn(v[2], v[3]));
                    if (a.o.mx.q != nullptr) {
                        const float amax = column_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
                        const int E = mx_exp(amax, a.o.mx.mode);
                        const float m = __uint_as_float((uint32_t)(127 - E) << 23);
                        if (on) {
                            *reinterpret_cast<uint32_t *>(a.o.mx.q + o) =
                                (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[0] * m, v[1] * m), __NV_SATFINITE, __NV_E4M3) |
                                (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2] * m, v[3] * m), __NV_SATFINITE, __NV_E4M3) << 16;
                            if (g4 == 0) a.o.mx.scale[mx_scale_offset(t, hq * NB + k, a.q_heads * D)] = (uint8_t)(E + 127);
                        }
                    }
                }
                if (on && g4 == 0 && a.o.lse != nullptr) a.o.lse[t * a.q_heads + hq] = sees ? (w.m[r][e] + log2f(l)) * kLn2 : -INFINITY;
            }
        if (!more) break;
        now ^= 1;
        __syncwarp();                                                  // (the one that was present is written over)
    }
    cp_wait<0>();
}

// A part's sum l at its maximum m, at the maximum `top` of several.  Where m is -inf the part has no weight, and l is 0, or
// NaN if all its scores are: that stays, in the result and in the log-sum.
__device__ __forceinline__ float sum_at(float l, float m, float top) { return m == -INFINITY ? l : l * ex2(m - top); }

// Joins the parts of the pairs that were cut: kWarps warps a row (token, q head), each a run of the parts, eight loads in
// flight.  The order is fixed by the lengths alone.
template <int D, class C, int kWarps>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32) join_kernel(const __grid_constant__ DecodeArgs a, int ctas) {
    constexpr int N = D / 32, kRows = kWarps == 1 ? 4 : 1;
    const int lane = threadIdx.x & 31, warp = kWarps == 1 ? 0 : threadIdx.x >> 5;
    const int64_t item = (int64_t)blockIdx.x * kRows + (kWarps == 1 ? threadIdx.x >> 5 : 0);
    const int64_t t = item / a.q_heads;
    const int hq = (int)(item % a.q_heads), G = a.q_heads / a.c.heads;
    SeqOfRow s{-1, 0, 0};
    Seq seq{};
    if (t < a.T) s = find_sequence(a.c.offsets, a.c.B, t, a.T);
    if (s.b >= 0) seq = sequence(a, C::ROWS, s.b);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (s.b < 0) return;
    const Parts parts = parts_of<D, C>(a.ctrl, ctas);
    const int64_t start = __ldcg(parts.start + s.b), share = share_of(__ldcg(parts.start + a.c.B), (int64_t)ctas * C::NW);
    const int r = (int)(t - s.begin) * G + hq % G, row = r % C::ROWS;
    const int64_t place = start + (int64_t)((hq / G) * seq.tiles + r / C::ROWS) * (seq.slices + kPairCost);
    const int u0 = (int)(place / share), u1 = (int)((place + seq.slices + kPairCost - 1) / share);
    if (u0 == u1) return;  // not cut (the same for all warps of a row)
    auto at = [&](int u) { return (size_t)(2 * u + (u == u0 ? 1 : 0)) * C::ROWS + row; };
    const int per = (u1 - u0 + kWarps) / kWarps, lo = u0 + warp * per, hi = min(u1 + 1, lo + per);   // this warp's parts
    float m = -INFINITY, l = 0.f, o[N] = {};
    for (int base = lo; base < hi; base += 32) {
        const float2 ml = base + lane < hi ? __ldcg(reinterpret_cast<const float2 *>(parts.ml + at(base + lane) * 2)) : make_float2(-INFINITY, 0.f);
        float top = ml.x;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, m);
        const float before = sum_at(l, m, top), mine = sum_at(ml.y, ml.x, top);
        m = top;
        l = before + warp_sum(mine);
        const float inv = l == 0.f ? 0.f : 1.f / l, old = before * inv, weight = mine * inv;   // o stays a mean
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] *= old;
        const int n = min(32, hi - base);
        for (int j = 0; j < n; j += 8) {
            float v[8][N];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float *p = parts.o + at(min(base + j + i, hi - 1)) * D + lane * N;
                if constexpr (N == 4) {
                    const float4 x = __ldcg(reinterpret_cast<const float4 *>(p));
                    v[i][0] = x.x; v[i][1] = x.y; v[i][2] = x.z; v[i][3] = x.w;
                } else {
                    const float2 x = __ldcg(reinterpret_cast<const float2 *>(p));
                    v[i][0] = x.x; v[i][1] = x.y;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float x = __shfl_sync(0xffffffffu, weight, (j + i) & 31);
#pragma unroll
                for (int e = 0; e < N; ++e) o[e] = j + i < n ? fmaf(v[i][e], x, o[e]) : o[e];
            }
        }
    }
    if constexpr (kWarps > 1) {
        __shared__ float so[kWarps][D], sm[kWarps], sl[kWarps];
#pragma unroll
        for (int i = 0; i < N; ++i) so[warp][lane * N + i] = o[i];
        if (lane == 0) {
            sm[warp] = m;
            sl[warp] = l;
        }
        __syncthreads();
        if (warp != 0) return;
        m = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm[w]);
        l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) l += sum_at(sl[w], sm[w], m);
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float x = sum_at(sl[w], sm[w], m) * inv;
#pragma unroll
            for (int i = 0; i < N; ++i) o[i] = fmaf(so[w][lane * N + i], x, o[i]);
        }
    }
    const bool sees = seq.len - seq.n + (int)(t - s.begin) >= 0;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = !sees ? 0.f : l == 0.f ? o[i] / l : o[i];   // (keys whose scores are all -inf: NaN)
    write_head_row<D>(a.o, t, hq, o, sees ? (m + log2f(l)) * kLn2 : -INFINITY);
}

template <int D, class C>
cudaError_t launch_one(const DecodeArgs &a, int num_sms, cudaStream_t stream) {
    auto kern = decode_kernel<D, C>;
    static std::atomic<uint64_t> allowed{0};
    cudaError_t e = allow_smem(kern, C::kSmem, allowed);
    if (e != cudaSuccess) return e;
    const int ctas = num_sms < kMaxCtas ? num_sms : kMaxCtas;
    mark_main_kernel(stream, true);
    kern<<<ctas, C::NT, C::kSmem, stream>>>(a);
    mark_main_kernel(stream, false);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // its prologue runs beside the first kernel's end
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // Few rows have many parts each: eight warps a row.
    if (a.T * a.q_heads <= kFewRows) {
        cfg.gridDim = dim3((unsigned)(a.T * a.q_heads));
        cfg.blockDim = dim3(256);
        return cudaLaunchKernelEx(&cfg, join_kernel<D, C, 8>, a, ctas);
    }
    cfg.gridDim = dim3((unsigned)((a.T * a.q_heads + 3) / 4));
    cfg.blockDim = dim3(128);
    return cudaLaunchKernelEx(&cfg, join_kernel<D, C, 1>, a, ctas);
}

// By the rows of an average sequence (its tokens times a group's heads): row tiles of 8, 16 or 24, whichever's tiles take
// least.  A tile of 24 takes as long as 1.2 of 16 for D = 64 and as 1.75 of them for D = 128, where six warps of it fill
// the registers and the workspace (64 sequences of 8,000 tokens, 48 rows: 252 against 310 us, and 503 against 446; 24 rows of
// one sequence of 32,003: 22.2 against 24.8, and 30.7 against 32.7); one of 16 as 1.7 of 8.  Warps that share a slice
// over more rows, and wait for each other at every slice, are slower than tiles that read it again (D = 128, 42 rows:
// 44.5 us against 39.3).
template <int D>
cudaError_t launch_rows(const DecodeArgs &a, int num_sms, cudaStream_t stream) {
    const int64_t rows = (a.T + a.c.B - 1) / a.c.B * (a.q_heads / a.c.heads);
    if (rows <= 8) return launch_one<D, Cfg<D, 8, 12, 3>>(a, num_sms, stream);
    if ((rows + 23) / 24 * (D == 64 ? 120 : 175) <= (rows + 15) / 16 * 100) return launch_one<D, Cfg<D, 24, D == 64 ? 8 : 6, 4>>(a, num_sms, stream);
    return launch_one<D, Cfg<D, 16, 8, 4>>(a, num_sms, stream);
}

}  // namespace

size_t decode_workspace_bytes() { return kControlBytes + kStartBytes + (size_t)2 * kMaxCtas * kPartFloats * 4; }

cudaError_t launch_decode(const DecodeArgs &a, int num_sms, cudaStream_t stream) {
    return a.D == 128 ? launch_rows<128>(a, num_sms, stream) : launch_rows<64>(a, num_sms, stream);
}

}  // namespace mhc
