// 8-bit matrix products on the 5th-generation tensor cores: out[m][n] = sum_k x[m][k] w[n][k] with x in
// MXFP8 (E4M3 codes, one UE8M0 scale byte per 32 values in the 128x4 tile layout) and w in E4M3 with one
// scale per 128 x 128 block, for one weight or for a weight per expert over ragged row groups.
//
// The weight is the MMA's M side (128 output channels per CTA), the tokens its N side, so a call of few
// tokens wastes no tensor work on padding: D[n][m] = W[n][k] X[m][k]^T, with the accumulator's lanes the
// output channels and its columns the tokens.  Both operands are K-major and come in by TMA as 128-byte
// swizzled boxes of 128 k values ("k block").  The tensor cores apply the UE8M0 scales themselves
// (kind::mxf8f6f4, one scale byte per row and 32 k values, read from tensor memory):
//   - the tokens' scale words (4 bytes: one k block of one token) are gathered into the layout that a
//     32x128b copy to tensor memory expects, so a tile may start at any row (ragged groups, gathered rows);
//   - UE8M0 weight scales fill the weight operand's scale block with one byte;
//   - fp32 weight scales (kWF32) are not representable there: the operand's scales are 1, every k block
//     gets its own accumulator, and the epilogue warps add it to fp32 registers times the block's scale.
//
// Roles of a CTA: warp 0 copies operands, warp 1 issues the MMAs, warp 2 (and 3) loads scales (2 also owns the
// tensor memory), the others are the epilogue (and copy gathered rows).  They hand work over through mbarriers: a
// ring of stages (two k blocks each), a ring of scale chunks, and two accumulators, so one tile's epilogue overlaps
// the next tile's products.
//
// Tiles.  A k block of a 128 x TN tile takes TN * 2 tensor cycles, and 16 KB + TN * 128 bytes of copies.  From L2 an SM
// gets about 50 bytes a cycle, so large calls are bound by copies: a pair of CTAs (cta_group::2) shares the token rows
// of a 256 x 224 tile, 31 KB an SM and k block.  Measured (UE8M0 scales): 8192 x 7168 x 7168 in 237-245 us, 3.4-3.5
// PFLOP/s, 90-93 % of twice the measured bf16 rate, the clock at 1.65 GHz under the power limit (275-280 us in runs of
// seconds, where it falls further); without the copies it would be 196 us, without the MMAs 211.  Few tokens are bound by the
// weight's bytes: 6 x 7168 x 7168 in 13.0 us; 48 rows over 64 experts, of which 25 to 35 get one (0.886 GB in the mean of
// six sets in turn), in 138 us, 6.4 TB/s.  fp32 scales: 2048 x 7168 x 4096 in 69 us, bound by
// the hand-over of one accumulator per k block (its load, sum and release are a chain of 700-800 cycles in the epilogue
// warps; the MMAs would take 320-400).
//
// Few tiles (decode) are split over k in a cluster: each CTA of the cluster sums its range, then the ranges
// are added in rank order through distributed shared memory, so the result is the same in every run.
//
// Every mbarrier wait is bounded in time.  A wait that gives up sets bit 0 of the status word; the role then
// issues nothing more, the CTA waits (bounded) for its copies and MMAs in flight, frees its tensor memory and
// returns; the call's output is then not to be trusted.
#include <cuda.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>

#include "mhc_device.cuh"
#include "mhc_kernels.h"
#include "sm100_ptx.cuh"
#include "tma_encode.h"

namespace mhc {

namespace {

using namespace ptx;

constexpr int kBM = 128;       // output channels per CTA (the MMA's M; one weight scale block)
constexpr int kBK = 128;       // k values per block (one 128-byte swizzled row; one weight scale block)
constexpr int kSB = 2;         // k blocks per stage: each has its own barriers, but the MMA warp tests and issues a stage at
                               // a time (its waits and loop cost about 350 cycles, nearly a block's MMAs of the largest tile)
constexpr int kSF = 4;         // k blocks per chunk of scales, and the chunks of their ring (a chunk takes a memory latency, a
constexpr int kSfSlots = 3;    // fence and an arrival at the pair's leader, about 2,000 cycles, whatever its size)
constexpr int kMaxSplit = 8;   // CTAs a tile's k range is split among (a portable cluster)
constexpr int kSplitStages = 4;  // and only beyond so many stages: a stage takes a CTA 0.41 us, the join 1.2 (one token) to
                                 // 2.6 us (128): K = 512 3.8 us whole, 4.6 in two; 1024 4.65 and 4.8; 2048 6.3 and 5.7
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per wait
constexpr int kSmemMax = 227 * 1024;
// More than half of an SM's shared memory, always: two CTAs that allocate tensor memory then never share an
// SM, so no allocation waits for another (clusters that wait for each other's columns could block forever).
constexpr int kSmemMin = kSmemMax / 2 + 1024;

template <int TN, int CG, bool kWF32, bool kGather>
struct Cfg {
    // Epilogue warps: SH of them share the columns of each lane quadrant.  With fp32 weight scales they read every
    // accumulator of one k block, so there are more of them, each with at most 64 columns (and sums in registers).
    static constexpr int SH = kWF32 ? (TN + 63) / 64 : TN >= 64 ? 2 : 1;
    static constexpr int EW = 4 * SH;
    static constexpr int SW = kWF32 ? 1 : 2;                   // warps that load scales
    static constexpr int W_EPI = 2 + SW, W_GATHER = W_EPI + EW;
    static constexpr int GW = !kGather ? 0 : kWF32 ? 1 : 3;    // extra warps that copy gathered rows, the last ones
    static constexpr int NT = 32 * (W_GATHER + GW);            // threads
    static constexpr int CC = !kWF32 || TN < 32 ? 16 : 32;     // columns per tensor-memory load
    static constexpr int OUT = CC * kBM * 2;                   // bytes of a share's staged results
    static constexpr int NB = (TN + 127) / 128;                // token scale atoms (128 rows x 4 bytes)
    static constexpr int TNC = TN / CG;                        // token rows this CTA copies
    static constexpr int A_BLOCK = kBM * kBK, B_BLOCK = TNC * kBK, SF_BLOCK = 512 * (1 + NB);  // bytes of one k block
    static constexpr int A_BYTES = kSB * A_BLOCK, B_BYTES = kSB * B_BLOCK, SF_BYTES = kSF * SF_BLOCK;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int FIXED = 1024 /*alignment*/ + 1024 /*barriers*/ + (kMaxExperts + 1) * 4 + kSfSlots * SF_BYTES + SH * OUT;
    static constexpr int NS_FIT = (kSmemMax - FIXED) / STAGE;
    static constexpr int NS = NS_FIT > 6 ? 6 : NS_FIT;         // ring stages
    // Accumulators: one being summed, one being stored; with fp32 weight scales one per k block in flight (the hand-over
    // to the epilogue and back takes longer than a k block's MMAs).
    static constexpr int NA = !kWF32 ? 2 : TN <= 64 ? 4 : TN > 160 ? 2 : 3;
    static constexpr int SFA_SETS = kWF32 ? 1 : kSB;           // (fp32 weight scales: the operand's are all ones)
    static constexpr int COL_SFA = NA * TN;                    // tensor memory columns: accumulators, scales (two sets)
    static constexpr int COL_SFB = COL_SFA + 4 * SFA_SETS;
    static constexpr int COLS_USED = COL_SFB + kSB * 4 * NB;
    static constexpr int COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int SMEM = FIXED + NS * STAGE;
    static_assert(COLS_USED <= 512, "tensor memory");
    static_assert(TN % (16 * CG) == 0 && TN <= 256 && TNC % 8 == 0, "MMA N");
    static_assert(NS >= 3 && 2 * kSB * NS + 2 * kSfSlots + 2 * NA + 2 <= 1024 / 8, "stages");
    static_assert(kSF % kSB == 0, "a stage's scales are in one chunk");
};

struct LinearMaps {
    CUtensorMap w, x, x16;  // x in boxes of a CTA's rows (one row for gathered rows), and of 16 rows
};

struct LinearParams {
    const uint8_t *x_scales;
    const void *w_scales;         // [E][nNB][nKB] UE8M0 bytes or fp32
    const int32_t *rows;          // [M] row of x of each output row (nullptr: the same row)
    const int32_t *offsets;       // [E + 1] (nullptr: one weight)
    void *out;
    int64_t M, R;                 // output rows, rows of x
    int N, K, E;
    int out_f32;
    int split;                    // CTAs of the cluster along k
    unsigned int *status;
};

__device__ __forceinline__ void bwait(uint64_t *bar, uint32_t parity, bool &dead) {
    mbar_wait_timed(bar, parity, dead, kWaitLimitNs);
}

// A wait by a whole warp: `dead` stays the same in all lanes.  kEager: back-to-back tests (each suspends for a while by
// itself), for the warps whose reaction the ring waits for; the others hand the issue slots on.
template <bool kEager>
__device__ __forceinline__ void wwait(uint64_t *bar, uint32_t parity, bool &dead) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || dead) return;
    if constexpr (kEager) {
        const uint64_t t0 = globaltimer_ns();
        do {
            for (int i = 0; i < 64; ++i)
                if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
        } while (globaltimer_ns() - t0 <= kWaitLimitNs);
        dead = true;
    } else {
        mbar_wait_timed(bar, parity, dead, kWaitLimitNs);
    }
    dead = __any_sync(0xffffffffu, dead);
}
// The waits for a stage's blocks, all tested before any is waited for.
__device__ __forceinline__ void wwait_blocks(uint64_t *blocks, uint32_t parity, bool &dead) {
    bool ok = true;
#pragma unroll
    for (int h = 0; h < kSB; ++h) ok &= mbar_try_wait(blocks + h, parity);
    if (__all_sync(0xffffffffu, ok) || dead) return;
    for (int h = 0; h < kSB; ++h) wwait<true>(blocks + h, parity, dead);
}
// One lane of the (converged) warp.  The tensor-core and copy instructions take their operands from uniform
// registers: loops around them run in the whole warp with values that are the same in every lane, and only the
// instructions themselves in the elected lane.  (With the loop in one lane each operand was moved there on its own:
// about 100 cycles per instruction, 1,100 per k block.)
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(ok));
    return ok != 0;
}
// Position in a ring of N slots: the slot and the parity of its current phase.
template <int N>
struct Ring {
    int s = 0;
    uint32_t ph = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) {
            s = 0;
            ph ^= 1u;
        }
    }
};

// Shared memory descriptor of a scale atom: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}
// One scale atom to four tensor-memory columns, the 32 rows repeated in the four lane quadrants (of both CTAs of
// a pair, each from its own shared memory).
template <int CG>
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
    else
        asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_take(uint32_t *dst_smem, uint32_t cols) {
    if constexpr (CG == 1) {
        tmem_alloc(dst_smem, cols);
        tmem_relinquish();
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(dst_smem)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_give(uint32_t taddr, uint32_t cols) {
    if constexpr (CG == 1) tmem_dealloc(taddr, cols);
    else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(cols) : "memory");
}
// Arrive on the mbarrier (of both CTAs of a pair) when all MMAs and copies issued so far by this thread are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if constexpr (CG == 1)
        umma_commit(bar);
    else
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                         smem_u32(bar)),
                     "h"((uint16_t)3)
                     : "memory");
}
// The pair leader's barrier at the same offset as `bar`; `bar` itself for a CTA alone.
template <int CG>
__device__ __forceinline__ uint32_t lead(uint64_t *bar) {
    return CG == 1 ? smem_u32(bar) : mapa(smem_u32(bar), 0);
}
// Arrival on the leader's barrier by its peer.  Releasing at cluster scope waits for the thread's earlier memory
// operations, about 1,000 cycles, so it is kept to arrivals that publish shared memory.
__device__ __forceinline__ void arrive_release_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// ... and this one tells only that this thread's tensor-memory loads have returned (it has waited for them).
__device__ __forceinline__ void arrive_relaxed_if(bool on, uint32_t bar) {
    asm volatile("{\n .reg .pred p;\n setp.ne.u32 p, %0, 0;\n @p mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%1];\n}\n" ::"r"(
                     (uint32_t)on),
                 "r"(bar)
                 : "memory");
}
// Instruction descriptor of kind::mxf8f6f4: E4M3 x E4M3, both K-major, UE8M0 scales, M x N.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
    return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= (A . scales) x (B . scales); the descriptor's scale ids pick the byte of the scale columns.
template <int CG>
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
            " tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
            : "memory");
}
// Operand copies that complete on a barrier of this CTA or, in a pair, of its leader.
template <int CG>
__device__ __forceinline__ void load_w(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];\n" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
            "%4}], [%5];\n" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void load_x(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
            "[%4];\n" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
// Four rows of a 2-D tensor (box one row high), 128 bytes each, to consecutive rows of shared memory.
template <int CG>
__device__ __forceinline__ void load_x_rows(void *dst, const CUtensorMap *map, int x, const int (&r)[4], uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
            "%4, %5, %6}], [%7];\n" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3, %4, %5, %6}], [%7];\n" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
            : "memory");
}
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

// 16 or 32 accumulator columns of this warp's lane quadrant.
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_load(uint32_t taddr, uint32_t (&r)[32]) {
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

// A tile of the schedule: weight e, token rows [m0, m0 + valid) (at most TN), output channels from n0 (this CTA's
// 128 of the pair's 256).  The MMA's N is what the tile has, in steps of 16 (32 for a pair, of which each CTA copies
// half the rows).
struct Tile {
    int e, n0, valid;
    int64_t m0;
    template <int CG>
    __device__ int width() const { return (valid + 16 * CG - 1) & ~(16 * CG - 1); }
};

// Tile r of nt token tiles x nN weight tiles: bands of kBand weight tiles, a band's weight tiles before the next token
// tile, so the tiles that run together are about as many token as weight tiles and share both in L2 (8192 x 7168 x 7168: 244
// us, 252 in bands of 1, 250 of 4, 242 of 16; 32768 gathered rows over 32 experts: 706, 722, 747, 740).
constexpr int kBand = 8;
__device__ __forceinline__ void tile_of(int64_t r, int64_t nt, int nN, int64_t &tt, int &tn) {
    const int64_t band = r / (nt * kBand);
    const int in_band = min(kBand, nN - (int)band * kBand);
    r -= band * nt * kBand;
    tt = r / in_band;
    tn = (int)band * kBand + (int)(r - tt * in_band);
}

// Tile `i` of the call (`pair`: the CTA of a pair).  Experts: `cum` holds the first token tile of each expert (cum[E]
// their number).
template <int TN, int CG>
__device__ __forceinline__ Tile tile_at(int64_t i, const LinearParams &p, const int *cum, int nN, int64_t nT, int pair) {
    Tile t;
    int64_t tt;
    int tn;
    if (p.offsets == nullptr) {
        tile_of(i, nT, nN, tt, tn);
        t.e = 0;
        t.n0 = (tn * CG + pair) * kBM;
        t.m0 = tt * TN;
        t.valid = (int)min((int64_t)TN, p.M - t.m0);
        return t;
    }
    int lo = 0, hi = p.E - 1;  // the last expert whose first tile is <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)cum[mid] * nN <= i) lo = mid;
        else hi = mid - 1;
    }
    tile_of(i - (int64_t)cum[lo] * nN, cum[lo + 1] - cum[lo], nN, tt, tn);
    t.e = lo;
    t.n0 = (tn * CG + pair) * kBM;
    const int64_t b = min(max((int64_t)__ldg(p.offsets + lo), (int64_t)0), p.M);
    const int64_t end = min((int64_t)__ldg(p.offsets + lo + 1), p.M);
    t.m0 = b + tt * TN;
    t.valid = (int)min((int64_t)TN, end - t.m0);
    return t;
}

// A barrier of 128 threads (number `id`), and one that also says whether any of them brought true.
__device__ __forceinline__ void sync_128(int id) {
    __syncwarp();
    asm volatile("bar.sync %0, 128;\n" ::"r"(id) : "memory");
}
__device__ __forceinline__ bool any_of_128(bool b, int id) {
    uint32_t r;
    __syncwarp();
    asm volatile("{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 128, p;\n selp.u32 %0, 1, 0, q;\n}\n"
                 : "=r"(r)
                 : "r"((uint32_t)b), "r"(id)
                 : "memory");
    return r != 0;
}

// Stores the tile's 128 channels (from n0 on) of tokens m, m + 1, ..., the first `count` of v's: warp q of the four that
// share these columns holds channels 32 q + lane.  The values pass through `buf` (NV x 256 bytes; barrier `id`), so a row
// leaves as whole lines, 16 bytes a lane (stored from registers, 64 bytes of a row at a time, a tile's results took 4,500 to
// 6,700 cycles: 6000 rows over 32 experts, K = 2048, 158 us against 150).  N % 8 == 0: those are inside a row or not.
template <int NV>
__device__ __forceinline__ void store_tokens(const LinearParams &p, int64_t m, int n0, int q, int lane, const float (&v)[NV], int count,
                                             unsigned char *buf, int id) {
    if (p.out_f32) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            sync_128(id);  // what was there has been read
#pragma unroll
            for (int j = 0; j < NV / 2; ++j) reinterpret_cast<float *>(buf)[j * kBM + 32 * q + lane] = v[h * (NV / 2) + j];
            sync_128(id);
            const int n = n0 + 4 * lane;
#pragma unroll
            for (int j = q; j < NV / 2; j += 4)
                if (h * (NV / 2) + j < count && n < p.N)
                    __stcs(reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + (m + h * (NV / 2) + j) * p.N + n),
                           *reinterpret_cast<const float4 *>(buf + j * 512 + lane * 16));
        }
    } else {
        sync_128(id);
#pragma unroll
        for (int j = 0; j < NV; ++j)
            reinterpret_cast<unsigned short *>(buf)[j * kBM + 32 * q + lane] = (unsigned short)pack2_rn(v[j], 0.f);
        sync_128(id);
        const int n = n0 + 8 * (lane & 15);
#pragma unroll
        for (int r = 0; r < NV / 8; ++r) {
            const int j = 8 * r + 2 * q + (lane >> 4);
            if (j < count && n < p.N)
                __stcs(reinterpret_cast<uint4 *>(reinterpret_cast<unsigned short *>(p.out) + (m + j) * p.N + n),
                       *reinterpret_cast<const uint4 *>(buf + j * 256 + (lane & 15) * 16));
        }
    }
}

__device__ __forceinline__ void store_out4(const LinearParams &p, int64_t m, int n, float4 v) {
    if (p.out_f32) __stcs(reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + m * p.N + n), v);
    else __stcs(reinterpret_cast<uint2 *>(reinterpret_cast<unsigned short *>(p.out) + m * p.N + n), make_uint2(pack2_rn(v.x, v.y), pack2_rn(v.z, v.w)));
}

template <int TN, int CG, bool kWF32, bool kGather>
__global__ void __launch_bounds__(Cfg<TN, CG, kWF32, kGather>::NT, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
    using C = Cfg<TN, CG, kWF32, kGather>;
    constexpr int NS = C::NS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *sA = smem, *sB = sA + NS * C::A_BYTES, *sSF = sB + NS * C::B_BYTES;
    unsigned char *sOut = sSF + kSfSlots * C::SF_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sOut + C::SH * C::OUT);
    uint64_t *full = bars, *empty = full + kSB * NS, *full_sf = empty + kSB * NS, *empty_sf = full_sf + kSfSlots,
             *acc_full = empty_sf + kSfSlots, *acc_empty = acc_full + C::NA, *drained = acc_empty + C::NA;
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(drained + 1);
    int *sCum = reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(bars) + 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = CG == 1 ? p.split : 1;
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0;
    const int pair = CG == 1 ? 0 : (int)(blockIdx.x & 1);  // 0: issues the pair's MMAs
    const int nN = (p.N + kBM * CG - 1) / (kBM * CG), nNB = (p.N + kBM - 1) / kBM, nKB = (p.K + kBK - 1) / kBK;
    const int64_t nT = (p.M + TN - 1) / TN;
    bool dead = false;

    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&maps.w)) : "memory");
        asm volatile("prefetch.tensormap [%0];\n" ::"l"(reinterpret_cast<uint64_t>(&maps.x)) : "memory");
    }
    if (warp == 1 && lane == 0) {
        for (int i = 0; i < kSB * NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSfSlots; ++i) {
            mbar_init(&full_sf[i], CG);
            mbar_init(&empty_sf[i], 1);
        }
        for (int i = 0; i < C::NA; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], CG * C::EW);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_take<CG>(sTmem, C::COLS);
    }
    // up to here only this CTA's own memory; from here on the previous launch's results
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;");
    if (p.offsets != nullptr && warp == 0) {
        // first token tile of each expert: a running sum over 32 experts at a time
        int base = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const int e = e0 + lane;
            int n = 0;
            if (e < p.E) {
                const int64_t b = min(max((int64_t)__ldg(p.offsets + e), (int64_t)0), p.M);
                const int64_t end = min((int64_t)__ldg(p.offsets + e + 1), p.M);
                n = end > b ? (int)((end - b + TN - 1) / TN) : 0;
            }
            int inc = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (e < p.E) sCum[e] = base + inc - n;
            base += __shfl_sync(0xffffffffu, inc, 31);
        }
        if (lane == 0) sCum[p.E] = base;
    }
    tmem_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync_all();  // the peer's barriers exist before anything arrives on them
    tmem_fence_after();
    const uint32_t tbase = *sTmem;
    const int64_t first = blockIdx.x / (S * CG), step = gridDim.x / (S * CG);
    int64_t ntiles = (p.offsets != nullptr ? (int64_t)sCum[p.E] : nT) * nN;
    if (S > 1) ntiles = min(ntiles, step);  // a split cluster takes one tile (only overlapping groups make more tiles)
    // this CTA's share of the stages, and of their k blocks
    const int nKS = (nKB + kSB - 1) / kSB;
    const int ks0 = (int)((int64_t)nKS * rank / S), ks1 = (int)((int64_t)nKS * (rank + 1) / S);
    const int kb0 = ks0 * kSB, kb1 = min(ks1 * kSB, nKB);

    if (warp == 0 || warp >= C::W_GATHER) {
        // ================================ operand copies (gathered rows: by the extra warps too)
        constexpr int kParts = kGather ? 1 + C::GW : 1;
        constexpr int kRows4 = C::TNC / 4;  // groups of four rows
        constexpr int kRows4Part = (kRows4 + kParts - 1) / kParts;
        const int part = warp == 0 ? 0 : warp - C::W_GATHER + 1;
        Ring<NS> st;
        int last_st = -1;  // the last block copied, and its phase
        uint32_t last_ph = 0;
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN, CG>(i, p, sCum, nN, nT, pair);
            // this CTA's part of the tile's rows: a multiple of 16, all that is copied (a group's last tile is half empty
            // on average, and the copies are what bounds a tile)
            const int rows = t.width<CG>() / CG, q0 = CG == 1 ? 0 : pair * rows;
            int r[kRows4Part][4];  // this warp's rows, the same in every lane
            if (kGather) {
                int mine[4] = {0, 0, 0, 0};
                if (lane < kRows4) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int q = q0 + 4 * lane + j;
                        const int v = q < t.valid ? __ldg(p.rows + t.m0 + q) : 0;
                        mine[j] = v >= 0 && v < p.R ? v : 0;  // a row outside x: its scales become NaN (below)
                    }
                }
#pragma unroll
                for (int g = 0; g < kRows4Part; ++g)
#pragma unroll
                    for (int j = 0; j < 4; ++j) r[g][j] = __shfl_sync(0xffffffffu, mine[j], (part + g * kParts) & 31);
            }
            for (int ks = ks0; ks < ks1 && !dead; ++ks, st.next()) {
#pragma unroll
                for (int h = 0; h < kSB; ++h) {
                    const int at = st.s * kSB + h, x = (ks * kSB + h) * kBK;
                    wwait<true>(&empty[at], st.ph ^ 1u, dead);
                    if (dead) break;
                    const uint32_t bar = lead<CG>(&full[at]);
                    if (x >= p.K) {  // no such block: nothing to copy
                        if (part == 0 && pair == 0 && elect_one()) mbar_arrive(&full[at]);
                        continue;
                    }
                    unsigned char *da = sA + st.s * C::A_BYTES + h * C::A_BLOCK, *db = sB + st.s * C::B_BYTES + h * C::B_BLOCK;
                    if (part == 0 && elect_one()) {
                        // the leader expects the pair's bytes (the peer's may land before: the phase waits for this arrival)
                        if (pair == 0) mbar_arrive_expect_tx(&full[at], CG * (C::A_BLOCK + rows * kBK));
                        load_w<CG>(da, &maps.w, x, t.n0, t.e, bar);
                        if (!kGather) {
                            if (rows == C::TNC) {
                                load_x<CG>(db, &maps.x, x, (int)t.m0 + q0, bar);
                            } else {
                                for (int g = 0; g < rows; g += 16) load_x<CG>(db + g * kBK, &maps.x16, x, (int)t.m0 + q0 + g, bar);
                            }
                        }
                    }
                    if (kGather && elect_one()) {
                        // (the whole tile apart: a test for every four rows costs the full tiles a fifth)
                        if (rows == C::TNC) {
#pragma unroll
                            for (int g = 0; g < kRows4Part; ++g)
                                if (part + g * kParts < kRows4) load_x_rows<CG>(db + (part + g * kParts) * 512, &maps.x, x, r[g], bar);
                        } else {
#pragma unroll
                            for (int g = 0; g < kRows4Part; ++g)
                                if (4 * (part + g * kParts) < rows) load_x_rows<CG>(db + (part + g * kParts) * 512, &maps.x, x, r[g], bar);
                        }
                    }
                    last_st = at;
                    last_ph = st.ph;
                }
            }
        }
        if (dead) {  // the copies in flight must land before the CTA's shared memory goes
            // (a pair's land on its leader's barriers; the cluster barrier below holds the peer).  Barrier by barrier, the
            // last phase that was armed; those of a phase that has long passed return at once.
            bool gave_up = false;
            for (int j = 0; j < kSB * NS && last_st >= 0 && pair == 0; ++j) bwait(&full[j], j <= last_st ? last_ph : last_ph ^ 1u, gave_up);
        }
    } else if (warp == 1) {
        // ================================ MMA issue
        if (pair == 0) {
            Ring<NS> st;
            Ring<C::NA> ac;
            Ring<kSfSlots> sc;
            bool have_sfa = false;
            const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(sA), 1024), db0 = sdesc_kmajor_sw128(smem_u32(sB), 1024),
                           ds0 = sdesc_scales(smem_u32(sSF));
            for (int64_t i = first; i < ntiles && !dead; i += step) {
                const uint32_t idesc = idesc_mxf8(kBM * CG, tile_at<TN, CG>(i, p, sCum, nN, nT, pair).template width<CG>());
                if (!kWF32) wwait<true>(&acc_empty[ac.s], ac.ph ^ 1u, dead);
                int in_chunk = 0;  // k blocks of the chunk of scales that are used
                for (int ks = ks0; ks < ks1; ++ks) {
                    if (in_chunk == 0) wwait<true>(full_sf + sc.s, sc.ph, dead);
                    wwait_blocks(full + st.s * kSB, st.ph, dead);
                    if (dead) break;
                    tmem_fence_after();
                    const bool last = ks + 1 == ks1, chunk_done = last || in_chunk + kSB == kSF;
                    const uint64_t ds = ds0 + (uint64_t)((sc.s * C::SF_BYTES + in_chunk * C::SF_BLOCK) >> 4), a = da0 + (uint64_t)((st.s * C::A_BYTES) >> 4),
                                   b = db0 + (uint64_t)((st.s * C::B_BYTES) >> 4);
                    // the stage's k steps of 32 inside K: past it the scale bytes are padding, so no MMA there
                    const int nk = min(4 * kSB, (p.K - ks * kSB * kBK) / 32);
                    // one k block: its scales to tensor memory, then its MMAs (in order in the tensor pipe)
                    auto block = [&](int h, uint32_t d, bool fresh) {
                        const uint32_t sfa = tbase + C::COL_SFA + (kWF32 ? 0 : 4 * h), sfb = tbase + C::COL_SFB + 4 * C::NB * h;
                        const uint64_t dsh = ds + (uint64_t)(h * C::SF_BLOCK >> 4);
                        if (!kWF32 || !have_sfa) tmem_cp_scales<CG>(sfa, dsh);  // fp32 weight scales: all ones, once
#pragma unroll
                        for (int n = 0; n < C::NB; ++n) tmem_cp_scales<CG>(sfb + 4 * n, dsh + 32 * (1 + n));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (4 * h + k < nk)
                                umma_mxf8<CG>(d, a + (uint64_t)((h * C::A_BLOCK >> 4) + 2 * k), b + (uint64_t)((h * C::B_BLOCK >> 4) + 2 * k),
                                              idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), sfa, sfb, (uint32_t)(!fresh || k > 0));
                    };
                    if constexpr (kWF32) {
#pragma unroll
                        for (int h = 0; h < kSB; ++h) {
                            if (4 * h >= nk) break;
                            wwait<true>(&acc_empty[ac.s], ac.ph ^ 1u, dead);
                            if (dead) break;
                            tmem_fence_after();
                            if (elect_one()) {
                                block(h, tbase + (uint32_t)(ac.s * TN), true);
                                commit<CG>(&acc_full[ac.s]);
                                commit<CG>(&empty[st.s * kSB + h]);
                                if (h + 1 < kSB && 4 * (h + 1) >= nk) commit<CG>(&empty[st.s * kSB + h + 1]);
                                if (chunk_done && (h + 1 == kSB || 4 * (h + 1) >= nk)) commit<CG>(&empty_sf[sc.s]);
                            }
                            __syncwarp();
                            have_sfa = true;
                            ac.next();
                        }
                    } else {
                        if (elect_one()) {
#pragma unroll
                            for (int h = 0; h < kSB; ++h) {
                                if (4 * h < nk) block(h, tbase + (uint32_t)(ac.s * TN), h == 0 && ks == ks0);
                                commit<CG>(&empty[st.s * kSB + h]);
                            }
                            if (chunk_done) commit<CG>(&empty_sf[sc.s]);
                            if (last) commit<CG>(&acc_full[ac.s]);
                        }
                    }
                    __syncwarp();
                    in_chunk += kSB;
                    if (chunk_done) {
                        in_chunk = 0;
                        sc.next();
                    }
                    st.next();
                }
                if (!kWF32) ac.next();
            }
            if (dead) {  // the MMAs in flight must end before their operands and accumulators go
                if (elect_one()) commit<CG>(drained);
                bool gave_up = false;
                bwait(drained, 0, gave_up);
            }
        }
        __syncwarp();
    } else if (warp < C::W_EPI) {
        // ================================ scales: each of the SW warps takes every SW-th chunk
        // A chunk's loads are all in flight in registers before its slot is waited for; then they are written to
        // shared memory and made visible to the copies with one fence (cp.async loads with a fence behind each k
        // block's cost a memory latency each: 0.7-1.1 us per k block).
        Ring<kSfSlots> sc;
        int turn = 0;
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN, CG>(i, p, sCum, nN, nT, pair);
            const int KT = (p.K / 32 + 3) / 4;
            const uint8_t *src[(TN + 31) / 32];
            int ok[(TN + 31) / 32];  // 1 load, 0 zeros (a row past the group), -1 NaN (a row index outside x)
#pragma unroll
            for (int j = 0; j < (TN + 31) / 32; ++j) {
                const int q = j * 32 + lane;
                int64_t m = t.m0 + q;
                ok[j] = q < t.valid ? 1 : 0;
                if (kGather && ok[j]) {
                    m = __ldg(p.rows + m);
                    if (m < 0 || m >= p.R) ok[j] = -1;
                }
                if (ok[j] != 1) m = 0;
                src[j] = p.x_scales + (m / 128) * KT * 512 + (m % 32) * 16 + (m % 128 / 32) * 4;
            }
            // (the second half of a pair's last tile may lie past N: any scale does, its rows are zeros)
            const uint8_t *ws = reinterpret_cast<const uint8_t *>(p.w_scales) + ((int64_t)t.e * nNB + min(t.n0 / kBM, nNB - 1)) * nKB;
            for (int kb = kb0; kb < kb1; kb += kSF, sc.next(), turn = turn + 1 == C::SW ? 0 : turn + 1) {
                if (turn != warp - 2) continue;
                uint32_t v[kSF][(TN + 31) / 32], w[kSF];
#pragma unroll
                for (int h = 0; h < kSF; ++h) {
                    const bool on = kb + h < kb1;
                    w[h] = kWF32 ? 0x7Fu /* 2^0 */ : on ? __ldg(ws + kb + h) : 0u;
#pragma unroll
                    for (int j = 0; j < (TN + 31) / 32; ++j) {
                        v[h][j] = ok[j] < 0 ? 0xFFFFFFFFu : 0u;
                        if (on && ok[j] > 0) v[h][j] = __ldg(reinterpret_cast<const uint32_t *>(src[j] + (int64_t)(kb + h) * 512));
                    }
                }
                wwait<true>(&empty_sf[sc.s], sc.ph ^ 1u, dead);
                if (dead) break;
#pragma unroll
                for (int h = 0; h < kSF; ++h) {
                    unsigned char *sf = sSF + sc.s * C::SF_BYTES + h * C::SF_BLOCK;
                    const uint32_t w4 = w[h] * 0x01010101u;
                    *reinterpret_cast<uint4 *>(sf + lane * 16) = make_uint4(w4, w4, w4, w4);
#pragma unroll
                    for (int j = 0; j < (TN + 31) / 32; ++j)
                        *reinterpret_cast<uint32_t *>(sf + 512 * (1 + j / 4) + lane * 16 + (j % 4) * 4) = v[h][j];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (pair == 0) mbar_arrive(&full_sf[sc.s]);
                    else arrive_release_at(lead<CG>(&full_sf[sc.s]));
                }
            }
        }
    } else {
        // ================================ epilogue: warp w holds the accumulator's lanes 32 (w % 4) ...
        const int q = warp & 3;
        const int share = (warp - C::W_EPI) >> 2;  // this warp's columns: loads share, share + SH, ...
        const uint32_t tq = tbase + ((uint32_t)(32 * q) << 16);
        Ring<C::NA> ac;
        float *red = reinterpret_cast<float *>(sA);  // split: this CTA's sums [token][128], in the stages (free by then)
        const uint32_t free_bar = lead<CG>(acc_empty);
        // Accumulator `acc` has been read: its loads are back in every lane, so there is nothing in memory to publish and the
        // arrival can be relaxed.  It is on the way to the next MMAs, and one predicated instruction for both CTAs of a pair: a
        // branch for lane 0 with an arrival per CTA took 200 cycles a k block (2048 x 7168 x 4096 with fp32 scales 84 us
        // against 77).
        auto release = [&](int acc) {
            tmem_fence_before();
            __syncwarp();
            arrive_relaxed_if(lane == 0, free_bar + 8 * acc);
        };
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN, CG>(i, p, sCum, nN, nT, pair);
            auto emit = [&](int tok, float (&v)[C::CC]) {  // tokens tok ... of the tile
                if (S > 1) {
#pragma unroll
                    for (int j = 0; j < C::CC; ++j) red[(tok + j) * kBM + 32 * q + lane] = v[j];
                } else {
                    store_tokens(p, t.m0 + tok, t.n0, q, lane, v, t.valid - tok, sOut + share * C::OUT, 1 + share);
                }
            };
            if constexpr (kWF32) {
                constexpr int kLoads = (TN / C::CC + C::SH - 1) / C::SH;
                float2 acc[kLoads][C::CC / 2];
#pragma unroll
                for (int c = 0; c < kLoads; ++c)
#pragma unroll
                    for (int j = 0; j < C::CC / 2; ++j) acc[c][j] = make_float2(0.f, 0.f);
                const float *ws = reinterpret_cast<const float *>(p.w_scales) + ((int64_t)t.e * nNB + min(t.n0 / kBM, nNB - 1)) * nKB;
                float next = __ldg(ws + kb0);
                for (int kb = kb0; kb < kb1; ++kb) {
                    const float2 s2 = make_float2(next, next);
                    next = __ldg(ws + min(kb + 1, kb1 - 1));
                    wwait<true>(&acc_full[ac.s], ac.ph, dead);
                    if (dead) break;
                    tmem_fence_after();
                    const uint32_t at = tq + (uint32_t)(ac.s * TN);
#pragma unroll
                    for (int c = 0; c < kLoads; ++c) {
                        const int col = (c * C::SH + share) * C::CC;
                        uint32_t v[C::CC];
                        if (col < t.valid) {
                            tmem_load(at + (uint32_t)col, v);
                            tmem_wait_ld();
                        }
                        if (c == kLoads - 1) {  // all loads are back
                            release(ac.s);
                            ac.next();
                        }
                        if (col < t.valid) {
#pragma unroll
                            for (int j = 0; j < C::CC / 2; ++j)
                                acc[c][j] = __ffma2_rn(make_float2(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), s2, acc[c][j]);
                        }
                    }
                }
                dead = any_of_128(dead, 1 + share);
                if (!dead) {
#pragma unroll
                    for (int c = 0; c < kLoads; ++c) {
                        const int tok = (c * C::SH + share) * C::CC;
                        float v[C::CC];
#pragma unroll
                        for (int j = 0; j < C::CC; ++j) v[j] = j & 1 ? acc[c][j / 2].y : acc[c][j / 2].x;
                        if (tok < t.valid) emit(tok, v);
                    }
                }
            } else {
                wwait<false>(&acc_full[ac.s], ac.ph, dead);
                dead = any_of_128(dead, 1 + share);
                if (dead) break;
                tmem_fence_after();
                for (int c = share * C::CC; c < t.valid; c += C::SH * C::CC) {
                    uint32_t u[C::CC];
                    tmem_load(tq + (uint32_t)(ac.s * TN + c), u);
                    tmem_wait_ld();
                    float v[C::CC];
#pragma unroll
                    for (int j = 0; j < C::CC; ++j) v[j] = __uint_as_float(u[j]);
                    emit(c, v);
                }
                release(ac.s);
                ac.next();
            }
        }
    }
    if (dead) atomicOr(p.status, 1u);
    if (S > 1) {
        // the cluster's ranges of k, added in rank order; this CTA takes every S-th token, a warp one at a time (a lane
        // four output channels)
        const bool gave_up = __syncthreads_or(dead) != 0;
        cluster_sync_all();
        if (first < ntiles && !gave_up) {
            const Tile t = tile_at<TN, CG>(first, p, sCum, nN, nT, pair);
            const int n = t.n0 + 4 * lane;
            const uint32_t mine = smem_u32(sA) + (uint32_t)lane * 16;
            for (int tok = rank + S * warp; tok < t.valid; tok += S * (C::NT / 32)) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int r = 0; r < S; ++r) {
                    const float4 a = ld_cluster_f32x4(mapa(mine, (uint32_t)r) + (uint32_t)tok * kBM * 4);
                    v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
                }
                if (n < p.N) store_out4(p, t.m0 + tok, n, v);  // N % 8 == 0: all four or none
            }
        }
        __syncwarp();
        cluster_sync_all();
    } else {
        __syncthreads();
        if (CG == 2) cluster_sync_all();  // nothing of the pair still reads or signals the other's memory
    }
    tmem_fence_after();
    if (warp == 2) tmem_give<CG>(tbase, C::COLS);
}

std::mutex g_mu;

cudaError_t encode_u8(tma::EncodeTiledFn fn, CUtensorMap *m, int rank, const void *ptr, const cuuint64_t *dims,
                      const cuuint64_t *strides, const cuuint32_t *box) {
    const cuuint32_t es[3] = {1, 1, 1};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, (cuuint32_t)rank, const_cast<void *>(ptr), dims, strides, box, es,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Token tiles of a call: their number for one weight, an upper bound for experts (the offsets are on the device).
int64_t token_tiles(const LinearArgs &a, int tn) {
    const int64_t n = (a.M + tn - 1) / tn;
    return a.offsets == nullptr ? n : std::min<int64_t>(a.M, n + std::min<int64_t>(a.E, a.M) - 1);
}

template <int TN, int CG, bool kWF32, bool kGather>
cudaError_t launch_one(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    using C = Cfg<TN, CG, kWF32, kGather>;
    tma::EncodeTiledFn fn;
    cudaError_t e = tma::encoder(fn);
    if (e != cudaSuccess) return e;
    LinearMaps maps;
    std::memset(&maps, 0, sizeof maps);
    {
        const cuuint64_t K = (cuuint64_t)a.K, N = (cuuint64_t)a.N;
        const cuuint64_t dims[3] = {K, N, (cuuint64_t)a.E}, strides[2] = {K, K * N};
        const cuuint32_t box[3] = {kBK, kBM, 1};
        if ((e = encode_u8(fn, &maps.w, 3, a.w, dims, strides, box)) != cudaSuccess) return e;
        const cuuint64_t dx[2] = {K, (cuuint64_t)a.R}, sx[1] = {K};
        const cuuint32_t bx[2] = {kBK, kGather ? 1u : (cuuint32_t)C::TNC};
        if ((e = encode_u8(fn, &maps.x, 2, a.x, dx, sx, bx)) != cudaSuccess) return e;
        const cuuint32_t b16[2] = {kBK, 16};
        if (!kGather && C::TNC > 16 && (e = encode_u8(fn, &maps.x16, 2, a.x, dx, sx, b16)) != cudaSuccess) return e;
    }
    auto kern = linear_kernel<TN, CG, kWF32, kGather>;
    constexpr int smem = C::SMEM > kSmemMin ? C::SMEM : kSmemMin;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = CG;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3(CG);
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const int64_t nN = (a.N + kBM * CG - 1) / (kBM * CG), nKS = (a.K + kSB * kBK - 1) / (kSB * kBK);
    const int64_t bound = token_tiles(a, TN) * nN;
    // Few tiles: each is split over k among the S CTAs of a cluster, as many as keep every cluster resident at once (a
    // second wave of clusters costs more than the larger share: 256 x 7168 x 1024, 16 clusters of 8: 26 us, of 4: 15).
    int S = 1, resident;
    {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        static int fits[64][kMaxSplit + 1];  // clusters of CG * S CTAs resident at once
        std::lock_guard<std::mutex> lock(g_mu);
        if (fits[dev][0] == 0) {  // once per device
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
            fits[dev][0] = 1;
        }
        const int64_t most = CG == 2 || nKS <= kSplitStages ? 1 : std::min<int64_t>(std::min<int64_t>(num_sms / bound, kMaxSplit), nKS);
        for (S = most < 1 ? 1 : (int)most;; --S) {
            int &n = fits[dev][S];
            if (n == 0) {
                attr[0].val.clusterDim.x = (unsigned)(CG * S);
                cfg.gridDim = dim3((unsigned)(CG * S));
                if (CG * S == 1) n = num_sms;
                else if ((e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
                if (n < 1) {
                    n = 0;
                    if (S == 1) return cudaErrorInvalidConfiguration;
                }
            }
            if (S == 1 || n >= bound) {
                resident = n;
                break;
            }
        }
    }
    LinearParams p{};
    p.x_scales = a.x_scales; p.w_scales = a.w_scales; p.rows = a.rows; p.offsets = a.offsets; p.out = a.out;
    p.M = a.M; p.R = a.R; p.N = a.N; p.K = a.K; p.E = a.E; p.out_f32 = a.out_f32; p.split = S;
    p.status = a.status;
    attr[0].val.clusterDim.x = (unsigned)(CG * S);
    cfg.gridDim = dim3((unsigned)(S > 1 ? bound * S : std::min<int64_t>(bound, resident) * CG));
    mark_main_kernel(stream, true);
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    mark_main_kernel(stream, false);
    return e;
}

template <int TN, int CG, bool kWF32>
cudaError_t launch_tn(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    return a.rows != nullptr ? launch_one<TN, CG, kWF32, true>(a, num_sms, stream) : launch_one<TN, CG, kWF32, false>(a, num_sms, stream);
}

// About how many rounds of tiles a call takes on `units` CTAs or pairs (experts: half a tile per expert is lost on
// average); fewer tiles than half the CTAs are split over k.
double rounds(const LinearArgs &a, int tn, int cg, int num_sms) {
    const double nt = a.offsets == nullptr ? (double)((a.M + tn - 1) / tn) : std::min((double)a.M, (double)a.M / tn + 0.5 * a.E);
    const double tiles = nt * (double)((a.N + kBM * cg - 1) / (kBM * cg)), units = num_sms / cg;
    if (tiles > units) return std::ceil(tiles / units);
    return cg == 2 || a.K <= kSplitStages * kSB * kBK ? 1.0 : 1.0 / std::min<double>(std::floor(units / tiles), kMaxSplit);
}

template <bool kWF32>
cudaError_t launch_scaled(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    // tokens a weight meets (experts' groups differ: half as many again as their mean).  Both sides, k = n = 7168, UE8M0 /
    // fp32 scales, us: 16 tokens in a tile of 16 13.8 / 15.5, of 32 13.8 / 15.6; 24 tokens 16.3 / 21.7 (two tiles), of 32
    // 14.3 / 15.8; 48 tokens 17.6 / 22.6 in tiles of 32, 14.8 / 17.6 in one of 64; 64 tokens 15.3 / 18.2 of 64, 15.6 / 18.1
    // of 128; 96 tokens 18.4 / 25.3 of 64, 16.5 / 19.0 of 128.  512 rows over 32 experts of 4096 x 7168 (24 by the rule):
    // 164 / 196 in tiles of 16, 147 / 156 of 32, 145 / 161 of 64.
    const int64_t per = a.offsets != nullptr ? (3 * a.M + 2 * a.E - 1) / (2 * a.E) : a.M;
    if (per <= 16) return launch_tn<16, 1, kWF32>(a, num_sms, stream);
    if (per <= 32) return launch_tn<32, 1, kWF32>(a, num_sms, stream);
    if (per <= 64) return launch_tn<64, 1, kWF32>(a, num_sms, stream);
    // Beyond, CTAs of 128 tokens, or pairs of 160, 192 or 224 (fp32 scales: up to 192, the sums are in registers): whichever's
    // rounds take least.  A k block's time in a full round, us: UE8M0 (the operands' copies) 0.275, 0.249, 0.268, 0.305;
    // fp32 (the accumulators' hand-over) 0.386, 0.41, 0.436.  Measured, CTAs / pairs of 160 / 192 / 224: 700 tokens, k = n =
    // 7168, 48.4 / 32.4 / 33.2 / 35.5, fp32 65.7 / 47.5 / 50.6; 4096 x 7168 x 4096 107.4 / 83.6 / 75.1 / 69.2, fp32 148.5 /
    // 148.7 / 118.7.  One round of CTAs stays one (200 tokens, k = 2048, n = 7168: 8.9 us, 9.5 in pairs).  Experts take the
    // widest pair (4096 tokens to 8 of 64 experts, 2048 -> 7168: 454 us against 475 in those of 192): their weights are read
    // once per tile.
    constexpr int kPair = kWF32 ? 192 : 224;
    const double r128 = rounds(a, 128, 1, num_sms), t128 = r128 * (kWF32 ? 0.386 : 0.275),
                 tpair = rounds(a, kPair, 2, num_sms) * (kWF32 ? 0.436 : 0.305);
    if (r128 > 1.0 && a.offsets == nullptr) {
        const double t160 = rounds(a, 160, 2, num_sms) * (kWF32 ? 0.41 : 0.249);
        if constexpr (!kWF32) {
            const double t192 = rounds(a, 192, 2, num_sms) * 0.268;
            if (t192 < std::min(tpair, std::min(t160, t128))) return launch_one<192, 2, kWF32, false>(a, num_sms, stream);
        }
        if (t160 < std::min(tpair, t128)) return launch_one<160, 2, kWF32, false>(a, num_sms, stream);
    }
    if (r128 > 1.0 && tpair < t128) return launch_tn<kPair, 2, kWF32>(a, num_sms, stream);
    return launch_tn<128, 1, kWF32>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    return a.w_scales_f32 ? launch_scaled<true>(a, num_sms, stream) : launch_scaled<false>(a, num_sms, stream);
}

}  // namespace mhc
