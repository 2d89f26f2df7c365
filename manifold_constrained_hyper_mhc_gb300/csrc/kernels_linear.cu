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
// Roles of a CTA: warp 0 copies operands, warp 1 issues the MMAs, warps 2 and 3 load scales (3 also owns the
// tensor memory), the others are the epilogue.  They hand work over through mbarriers: a ring of stages (one
// k block each) and two accumulators, so one tile's epilogue overlaps the next tile's products.
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
constexpr int kBK = 128;       // k values per stage (one 128-byte swizzled row; one weight scale block)
constexpr int kSfBlocks = 4;   // k blocks per chunk of scales
constexpr int kGatherWarps = 3;
constexpr int kSfSlots = 3;    // chunks in the scales' ring
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per wait
constexpr int kSmemMax = 227 * 1024;
// More than half of an SM's shared memory, always: two CTAs that allocate tensor memory then never share an
// SM, so no allocation waits for another (clusters that wait for each other's columns could block forever).
constexpr int kSmemMin = kSmemMax / 2 + 1024;

template <int TN, int CG, bool kGather>
struct Cfg {
    static constexpr int EW = 4 * CG;                          // epilogue warps
    static constexpr int GW = kGather ? kGatherWarps : 0;      // extra copy warps, the last ones
    static constexpr int W_GATHER = 4 + EW;
    static constexpr int NT = 32 * (W_GATHER + GW);            // threads
    static constexpr int NB = (TN + 127) / 128;                // token scale atoms (128 rows x 4 bytes)
    static constexpr int A_BYTES = kBM * kBK;
    static constexpr int TNC = TN / CG;                        // token rows this CTA copies
    static constexpr int B_BYTES = TNC * kBK;
    static constexpr int SF_BYTES = 512 * (1 + NB);            // weight atom, token atoms
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int SF_CHUNK = kSfBlocks * SF_BYTES;      // scales come in chunks of k blocks, in their own ring
    static constexpr int FIXED = 1024 /*alignment*/ + 1024 /*barriers*/ + (kMaxExperts + 1) * 4 + kSfSlots * SF_CHUNK;
    static constexpr int NS_FIT = (kSmemMax - FIXED) / STAGE;
    static constexpr int NS = NS_FIT > 10 ? 10 : NS_FIT;       // ring stages
    static constexpr int CW = (TN / 16 + CG - 1) / CG;         // 16-column chunks of a warp (CG warps share the columns)
    static constexpr int COL_SFA = 2 * TN;                     // tensor memory columns: accumulators, scales (two sets)
    static constexpr int COL_SFB = COL_SFA + 8;
    static constexpr int COLS_USED = COL_SFB + 8 * NB;
    static constexpr int COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int SMEM = FIXED + NS * STAGE;
    static_assert(COLS_USED <= 512, "tensor memory");
    static_assert(TN % (16 * CG) == 0 && TN <= 256 && TNC % 8 == 0, "MMA N");
    static_assert(NS >= 3, "stages");
};

struct LinearMaps {
    CUtensorMap w, x;
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

// A wait by a whole warp: `dead` stays the same in all lanes.
__device__ __forceinline__ void wwait(uint64_t *bar, uint32_t parity, bool &dead) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || dead) return;
    mbar_wait_timed(bar, parity, dead, kWaitLimitNs);
    dead = __any_sync(0xffffffffu, dead);
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
__device__ __forceinline__ void arrive_relaxed_at(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
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
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
    return v;
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
// tile, so the tiles that run together are about as many token as weight tiles and share both in L2.
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

__device__ __forceinline__ void store_out(const LinearParams &p, int64_t m, int n, float v) {
    if (p.out_f32) __stcs(reinterpret_cast<float *>(p.out) + m * p.N + n, v);
    else __stcs(reinterpret_cast<unsigned short *>(p.out) + m * p.N + n, __bfloat16_as_ushort(__float2bfloat16_rn(v)));
}

template <int TN, int CG, bool kWF32, bool kGather>
__global__ void __launch_bounds__(Cfg<TN, CG, kGather>::NT, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
    using C = Cfg<TN, CG, kGather>;
    constexpr int NS = C::NS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *sA = smem, *sB = sA + NS * C::A_BYTES, *sSF = sB + NS * C::B_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sSF + kSfSlots * C::SF_CHUNK);
    uint64_t *full = bars, *empty = full + NS, *full_sf = empty + NS, *empty_sf = full_sf + kSfSlots, *acc_full = empty_sf + kSfSlots,
             *acc_empty = acc_full + 2, *drained = acc_empty + 2;
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(drained + 1);
    int *sCum = reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(bars) + 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = CG == 1 ? p.split : 1;
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0;
    const int pair = CG == 1 ? 0 : (int)(blockIdx.x & 1);  // 0: issues the pair's MMAs
    const int nN = (p.N + kBM * CG - 1) / (kBM * CG), nNB = (p.N + kBM - 1) / kBM, nKB = (p.K + kBK - 1) / kBK;
    const int64_t nT = (p.M + TN - 1) / TN;
    bool dead = false;

    if (warp == 1 && lane == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < kSfSlots; ++i) {
            mbar_init(&full_sf[i], CG);
            mbar_init(&empty_sf[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], CG * C::EW);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
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
    const int64_t ntiles = (p.offsets != nullptr ? (int64_t)sCum[p.E] : nT) * nN;
    const int64_t first = blockIdx.x / (S * CG), step = gridDim.x / (S * CG);
    // this CTA's share of the k blocks
    const int kb0 = (int)((int64_t)nKB * rank / S), kb1 = (int)((int64_t)nKB * (rank + 1) / S);

    if (warp == 0 || warp >= C::W_GATHER) {
        // ================================ operand copies (gathered rows: by the extra warps too)
        constexpr int kParts = kGather ? 1 + C::GW : 1;
        constexpr int kRows4 = C::TNC / 4;  // groups of four rows
        constexpr int kRows4Part = (kRows4 + kParts - 1) / kParts;
        const int part = warp == 0 ? 0 : warp - C::W_GATHER + 1;
        Ring<NS> st;
        int it = 0;
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN, CG>(i, p, sCum, nN, nT, pair);
            const int q0 = CG == 1 ? 0 : pair * (t.width<CG>() / 2);  // this CTA's part of the tile's rows
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
            for (int kb = kb0; kb < kb1; ++kb, ++it, st.next()) {
                wwait(&empty[st.s], st.ph ^ 1u, dead);
                if (dead) break;
                const uint32_t bar = lead<CG>(&full[st.s]);
                unsigned char *da = sA + st.s * C::A_BYTES, *db = sB + st.s * C::B_BYTES;
                if (part == 0 && elect_one()) {
                    // the leader expects the pair's bytes (the peer's may land before: the phase waits for this arrival)
                    if (pair == 0) mbar_arrive_expect_tx(&full[st.s], CG * (C::A_BYTES + C::B_BYTES));
                    load_w<CG>(da, &maps.w, kb * kBK, t.n0, t.e, bar);
                    if (!kGather) load_x<CG>(db, &maps.x, kb * kBK, (int)t.m0 + q0, bar);
                }
                if (kGather && elect_one()) {
#pragma unroll
                    for (int g = 0; g < kRows4Part; ++g)
                        if (part + g * kParts < kRows4) load_x_rows<CG>(db + (part + g * kParts) * 512, &maps.x, kb * kBK, r[g], bar);
                }
            }
        }
        if (dead) {  // the copies in flight must land before the CTA's shared memory goes
            bool gave_up = false;  // (a pair's land on its leader's barriers; the cluster barrier below holds the peer)
            for (int j = it > NS ? it - NS : 0; j < it && pair == 0; ++j) bwait(&full[j % NS], (uint32_t)((j / NS) & 1), gave_up);
        }
    } else if (warp == 1) {
        // ================================ MMA issue
        if (pair == 0) {
            Ring<NS> st;
            Ring<2> ac;
            Ring<kSfSlots> sc;
            Ring<2> sf;  // the two sets of scale columns
            const uint64_t da0 = sdesc_kmajor_sw128(smem_u32(sA), 1024), db0 = sdesc_kmajor_sw128(smem_u32(sB), 1024),
                           ds0 = sdesc_scales(smem_u32(sSF));
            for (int64_t i = first; i < ntiles && !dead; i += step) {
                const uint32_t idesc = idesc_mxf8(kBM * CG, tile_at<TN, CG>(i, p, sCum, nN, nT, pair).template width<CG>());
                int left = kSfBlocks;  // k blocks left in the chunk of scales
                for (int kb = kb0; kb < kb1; ++kb) {
                    const bool fresh = kWF32 || kb == kb0;  // starts an accumulator
                    if (fresh) wwait(&acc_empty[ac.s], ac.ph ^ 1u, dead);
                    if (left == kSfBlocks) wwait(&full_sf[sc.s], sc.ph, dead);
                    wwait(&full[st.s], st.ph, dead);
                    if (dead) break;
                    tmem_fence_after();
                    const bool last = kb + 1 == kb1, chunk_done = last || left == 1;
                    const uint32_t sfa = tbase + C::COL_SFA + 4 * sf.s, sfb = tbase + C::COL_SFB + 4 * C::NB * sf.s;
                    const uint64_t ds = ds0 + (uint64_t)((sc.s * C::SF_CHUNK + (kSfBlocks - left) * C::SF_BYTES) >> 4);
                    const uint64_t a = da0 + (uint64_t)((st.s * C::A_BYTES) >> 4), b = db0 + (uint64_t)((st.s * C::B_BYTES) >> 4);
                    const uint32_t d = tbase + (uint32_t)(ac.s * TN);
                    const int nk = min(4, (p.K - kb * kBK) / 32);  // past K the scale bytes are padding: no MMA there
                    if (elect_one()) {
                        tmem_cp_scales<CG>(sfa, ds);
#pragma unroll
                        for (int n = 0; n < C::NB; ++n) tmem_cp_scales<CG>(sfb + 4 * n, ds + 32 * (1 + n));
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (k < nk)
                                umma_mxf8<CG>(d, a + 2 * k, b + 2 * k, idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), sfa, sfb,
                                              (uint32_t)(!fresh || k > 0));
                        commit<CG>(&empty[st.s]);
                        if (chunk_done) commit<CG>(&empty_sf[sc.s]);
                        if (kWF32 || last) commit<CG>(&acc_full[ac.s]);
                    }
                    __syncwarp();
                    if (kWF32 || last) ac.next();
                    if (--left == 0 || last) {
                        left = kSfBlocks;
                        sc.next();
                    }
                    sf.next();
                    st.next();
                }
            }
            if (dead) {  // the MMAs in flight must end before their operands and accumulators go
                if (elect_one()) commit<CG>(drained);
                bool gave_up = false;
                bwait(drained, 0, gave_up);
            }
        }
        __syncwarp();
    } else if (warp < 4) {
        // ================================ scales: the two warps take every other chunk
        // A chunk's loads are all in flight in registers before its slot is waited for; then they are written to
        // shared memory and made visible to the copies with one fence (a fence per k block, with cp.async loads
        // behind it, cost a memory latency each: 0.7-1.1 us per k block).
        int ch = 0;
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
            for (int kb = kb0; kb < kb1; kb += kSfBlocks, ++ch) {
                if ((ch & 1) != (warp & 1)) continue;
                uint32_t v[kSfBlocks][(TN + 31) / 32], w[kSfBlocks];
#pragma unroll
                for (int b = 0; b < kSfBlocks; ++b) {
                    const bool on = kb + b < kb1;
                    w[b] = kWF32 ? 0x7Fu /* 2^0 */ : on ? __ldg(ws + kb + b) : 0u;
#pragma unroll
                    for (int j = 0; j < (TN + 31) / 32; ++j) {
                        v[b][j] = ok[j] < 0 ? 0xFFFFFFFFu : 0u;
                        if (on && ok[j] > 0) v[b][j] = __ldg(reinterpret_cast<const uint32_t *>(src[j] + (int64_t)(kb + b) * 512));
                    }
                }
                const int sl = ch % kSfSlots;
                bwait(&empty_sf[sl], (uint32_t)((ch / kSfSlots) & 1) ^ 1u, dead);
                if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
#pragma unroll
                for (int b = 0; b < kSfBlocks; ++b) {
                    unsigned char *sf = sSF + sl * C::SF_CHUNK + b * C::SF_BYTES;
                    const uint32_t w4 = w[b] * 0x01010101u;
                    *reinterpret_cast<uint4 *>(sf + lane * 16) = make_uint4(w4, w4, w4, w4);
#pragma unroll
                    for (int j = 0; j < (TN + 31) / 32; ++j)
                        *reinterpret_cast<uint32_t *>(sf + 512 * (1 + j / 4) + lane * 16 + (j % 4) * 4) = v[b][j];
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (pair == 0) mbar_arrive(&full_sf[sl]);
                    else arrive_release_at(lead<CG>(&full_sf[sl]));
                }
            }
        }
    } else {
        // ================================ epilogue: warp w holds the accumulator's lanes 32 (w % 4) ...
        const int q = warp & 3;
        const int half = (warp - 4) >> 2;  // of a pair's CTA: the even or the odd 16-column chunks
        const uint32_t tq = tbase + ((uint32_t)(32 * q) << 16);
        int at = 0;
        float *red = reinterpret_cast<float *>(sA);  // split: this CTA's sums [token][128], in the stages (free by then)
        auto release = [&](uint64_t *bar) {
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (pair == 0) mbar_arrive(bar);
                else arrive_relaxed_at(lead<CG>(bar));
            }
        };
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN, CG>(i, p, sCum, nN, nT, pair);
            const int n = t.n0 + 32 * q + lane;
            auto emit = [&](int tok, float v) {
                if (S > 1) red[tok * kBM + 32 * q + lane] = v;
                else if (n < p.N) store_out(p, t.m0 + tok, n, v);
            };
            if constexpr (kWF32) {
                float acc[C::CW][16];
#pragma unroll
                for (int c = 0; c < C::CW; ++c)
#pragma unroll
                    for (int j = 0; j < 16; ++j) acc[c][j] = 0.f;
                const float *ws = reinterpret_cast<const float *>(p.w_scales) + ((int64_t)t.e * nNB + min(t.n0 / kBM, nNB - 1)) * nKB;
                float mine = 0.f;
                for (int kb = kb0; kb < kb1; ++kb, ++at) {
                    if (((kb - kb0) & 31) == 0) mine = kb + lane < kb1 ? __ldg(ws + kb + lane) : 0.f;
                    bwait(&acc_full[at & 1], (uint32_t)((at >> 1) & 1), dead);
                    if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                    tmem_fence_after();
                    const float sc = __shfl_sync(0xffffffffu, mine, (kb - kb0) & 31);
#pragma unroll
                    for (int c = 0; c < C::CW; ++c) {
                        const int col = (c * CG + half) * 16;
                        if (col < t.valid) {
                            uint32_t v[16];
                            tmem_ld16(tq + (uint32_t)((at & 1) * TN + col), v);
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) acc[c][j] = fmaf(__uint_as_float(v[j]), sc, acc[c][j]);
                        }
                    }
                    release(&acc_empty[at & 1]);
                }
                if (!dead) {
#pragma unroll
                    for (int c = 0; c < C::CW; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const int tok = (c * CG + half) * 16 + j;
                            if (tok < t.valid) emit(tok, acc[c][j]);
                        }
                }
            } else {
                bwait(&acc_full[at & 1], (uint32_t)((at >> 1) & 1), dead);
                if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                tmem_fence_after();
                for (int c = half * 16; c < t.valid; c += CG * 16) {
                    uint32_t v[16];
                    tmem_ld16(tq + (uint32_t)((at & 1) * TN + c), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < t.valid) emit(c + j, __uint_as_float(v[j]));
                }
                release(&acc_empty[at & 1]);
                ++at;
            }
        }
    }
    if (dead) atomicOr(p.status, 1u);
    if (S > 1) {
        // the cluster's ranges of k, added in rank order; this CTA takes every S-th token
        const bool gave_up = __syncthreads_or(dead) != 0;
        cluster_sync_all();
        if (first < ntiles && !gave_up) {
            const Tile t = tile_at<TN, CG>(first, p, sCum, nN, nT, pair);
            const int n = t.n0 + (tid & (kBM - 1));
            const uint32_t mine = smem_u32(sA) + (uint32_t)(tid & (kBM - 1)) * 4;
            for (int tok = rank + S * (tid / kBM); tok < t.valid && tid < C::NT / kBM * kBM; tok += S * (C::NT / kBM)) {
                float v = 0.f;
                for (int r = 0; r < S; ++r) v += ld_cluster_f32(mapa(mine, (uint32_t)r) + (uint32_t)tok * kBM * 4);
                if (n < p.N) store_out(p, t.m0 + tok, n, v);
            }
        }
        __syncwarp();
        cluster_sync_all();
    } else {
        __syncthreads();
        if (CG == 2) cluster_sync_all();  // nothing of the pair still reads or signals the other's memory
    }
    tmem_fence_after();
    if (warp == 3) tmem_give<CG>(tbase, C::COLS);
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
    using C = Cfg<TN, CG, kGather>;
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
    int resident = num_sms;  // CTAs, or pairs, at once
    {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        static int ready[64];
        std::lock_guard<std::mutex> lock(g_mu);
        if (ready[dev] == 0) {
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
            int n = num_sms;
            if (CG == 2 && (e = cudaOccupancyMaxActiveClusters(&n, kern, &cfg)) != cudaSuccess) return e;
            if (n < 1) return cudaErrorInvalidConfiguration;
            ready[dev] = n;
        }
        resident = ready[dev];
    }
    const int64_t nN = (a.N + kBM * CG - 1) / (kBM * CG), nKB = (a.K + kBK - 1) / kBK;
    const int64_t bound = token_tiles(a, TN) * nN;
    int64_t S = CG == 2 ? 1 : std::min<int64_t>(std::min<int64_t>(num_sms / bound, 8), nKB / 2);
    if (S < 1) S = 1;
    LinearParams p{};
    p.x_scales = a.x_scales; p.w_scales = a.w_scales; p.rows = a.rows; p.offsets = a.offsets; p.out = a.out;
    p.M = a.M; p.R = a.R; p.N = a.N; p.K = a.K; p.E = a.E; p.out_f32 = a.out_f32; p.split = (int)S;
    p.status = a.status;
    attr[0].val.clusterDim.x = (unsigned)(CG * S);
    cfg.gridDim = dim3((unsigned)(S > 1 ? bound * S : std::min<int64_t>(bound, resident) * CG));
    mark_main_kernel(stream, true);
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    mark_main_kernel(stream, false);
    return e;
}

template <int TN, int CG>
cudaError_t launch_tn(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    if (a.w_scales_f32)
        return a.rows != nullptr ? launch_one<TN, CG, true, true>(a, num_sms, stream) : launch_one<TN, CG, true, false>(a, num_sms, stream);
    return a.rows != nullptr ? launch_one<TN, CG, false, true>(a, num_sms, stream) : launch_one<TN, CG, false, false>(a, num_sms, stream);
}

constexpr int kPairTN = 224;  // two accumulators and the scales in 512 columns; a multiple of 32

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    const int64_t per = a.offsets != nullptr ? (a.M + a.E - 1) / a.E : a.M;  // tokens a weight meets
    if (per <= 16) return launch_tn<16, 1>(a, num_sms, stream);
    if (per <= 32) return launch_tn<32, 1>(a, num_sms, stream);
    if (per <= 64) return launch_tn<64, 1>(a, num_sms, stream);
    const int64_t pairs = token_tiles(a, kPairTN) * ((a.N + 2 * kBM - 1) / (2 * kBM));
    if (per <= 128 || pairs < num_sms / 2) return launch_tn<128, 1>(a, num_sms, stream);
    return launch_tn<kPairTN, 2>(a, num_sms, stream);
}

}  // namespace mhc
