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
// Roles of a CTA: warp 0 copies operands, warp 1 issues the MMAs, warp 2 loads scales, warp 3 owns the
// tensor memory, the others are the epilogue.  They hand work over through mbarriers: a ring of stages (one
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
constexpr uint64_t kWaitLimitNs = 1000000000ull;  // 1 s per wait
constexpr int kSmemMax = 227 * 1024;
// More than half of an SM's shared memory, always: two CTAs that allocate tensor memory then never share an
// SM, so no allocation waits for another (clusters that wait for each other's columns could block forever).
constexpr int kSmemMin = kSmemMax / 2 + 1024;

template <int TN, bool kWF32>
struct Cfg {
    static constexpr int EW = 4;                               // epilogue warps
    static constexpr int NT = 128 + 32 * EW;                   // threads
    static constexpr int NB = (TN + 127) / 128;                // token scale atoms (128 rows x 4 bytes)
    static constexpr int A_BYTES = kBM * kBK;
    static constexpr int B_BYTES = TN * kBK;
    static constexpr int SF_BYTES = 512 * (1 + NB);            // weight atom, token atoms
    static constexpr int STAGE = A_BYTES + B_BYTES + SF_BYTES;
    static constexpr int FIXED = 1024 /*alignment*/ + 1024 /*barriers*/ + (kMaxExperts + 1) * 4;
    static constexpr int NS_FIT = (kSmemMax - FIXED) / STAGE;
    static constexpr int NS = NS_FIT > 10 ? 10 : NS_FIT;       // ring stages
    static constexpr int SF_AHEAD = NS > 4 ? 4 : NS - 1;       // stages of scale loads in flight
    static constexpr int COL_SFA = 2 * TN;                     // tensor memory columns: accumulators, scales (two sets)
    static constexpr int COL_SFB = COL_SFA + 8;
    static constexpr int COLS_USED = COL_SFB + 8 * NB;
    static constexpr int COLS = COLS_USED <= 64 ? 64 : COLS_USED <= 128 ? 128 : COLS_USED <= 256 ? 256 : 512;
    static constexpr int SMEM = FIXED + NS * STAGE;
    static_assert(COLS_USED <= 512, "tensor memory");
    static_assert(TN % 16 == 0 && TN <= 256, "MMA N");
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

// Shared memory descriptor of a scale atom: 32 rows of 16 bytes, no swizzle, 8-row groups 128 bytes apart.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(128u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    return d;
}
// One scale atom to four tensor-memory columns, the 32 rows repeated in the four lane quadrants.
__device__ __forceinline__ void tmem_cp_scales(uint32_t taddr, uint64_t desc) {
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}
// Instruction descriptor of kind::mxf8f6f4: E4M3 x E4M3, both K-major, UE8M0 scales, M x N.
__host__ __device__ constexpr uint32_t idesc_mxf8(int M, int N) {
    return (1u << 23) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// D[tmem] (+)= (A . scales) x (B . scales); the descriptor's scale ids pick the byte of the scale columns.
__device__ __forceinline__ void umma_mxf8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// Four rows of a 2-D tensor (box one row high), 128 bytes each, to consecutive rows of shared memory.
__device__ __forceinline__ void tma_gather4(void *dst, const CUtensorMap *map, int x, int r0, int r1, int r2, int r3,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5, %6}], [%7];\n" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_u32(bar))
        : "memory");
}
// Four bytes global -> shared, asynchronously; zeros when !valid (nothing is read).
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory");
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];\n" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// A tile of the schedule: weight e, token rows [m0, m_end) (at most TN), output channels from n0.
struct Tile {
    int e, n0, valid;
    int64_t m0;
};

// Tile `i` of the call.  One weight: token tiles inside a weight tile.  Experts: `cum` holds the first token
// tile of each expert (cum[E] their number); a weight tile's token tiles are neighbours, so they share it in L2.
template <int TN>
__device__ __forceinline__ Tile tile_at(int64_t i, const LinearParams &p, const int *cum, int nN, int64_t nT) {
    Tile t;
    if (p.offsets == nullptr) {
        t.e = 0;
        t.n0 = (int)(i / nT) * kBM;
        t.m0 = (i % nT) * TN;
        t.valid = (int)min((int64_t)TN, p.M - t.m0);
        return t;
    }
    int lo = 0, hi = p.E - 1;  // the last expert whose first tile is <= i
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if ((int64_t)cum[mid] * nN <= i) lo = mid;
        else hi = mid - 1;
    }
    const int nt = cum[lo + 1] - cum[lo];
    const int r = (int)(i - (int64_t)cum[lo] * nN);
    t.e = lo;
    t.n0 = (r / nt) * kBM;
    const int64_t b = min(max((int64_t)__ldg(p.offsets + lo), (int64_t)0), p.M);
    const int64_t end = min((int64_t)__ldg(p.offsets + lo + 1), p.M);
    t.m0 = b + (int64_t)(r % nt) * TN;
    t.valid = (int)min((int64_t)TN, end - t.m0);
    return t;
}

__device__ __forceinline__ void store_out(const LinearParams &p, int64_t m, int n, float v) {
    if (p.out_f32) __stcs(reinterpret_cast<float *>(p.out) + m * p.N + n, v);
    else __stcs(reinterpret_cast<unsigned short *>(p.out) + m * p.N + n, __bfloat16_as_ushort(__float2bfloat16_rn(v)));
}

template <int TN, bool kWF32, bool kGather>
__global__ void __launch_bounds__(Cfg<TN, kWF32>::NT, 1)
linear_kernel(const __grid_constant__ LinearMaps maps, const LinearParams p) {
    using C = Cfg<TN, kWF32>;
    constexpr int NS = C::NS;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    unsigned char *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    unsigned char *sA = smem, *sB = sA + NS * C::A_BYTES, *sSF = sB + NS * C::B_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sSF + NS * C::SF_BYTES);
    uint64_t *full = bars, *full_sf = full + NS, *empty = full_sf + NS, *acc_full = empty + NS, *acc_empty = acc_full + 2,
             *drained = acc_empty + 2;
    uint32_t *sTmem = reinterpret_cast<uint32_t *>(drained + 1);
    int *sCum = reinterpret_cast<int *>(reinterpret_cast<unsigned char *>(bars) + 1024);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int S = p.split;
    const int rank = S > 1 ? (int)(blockIdx.x % S) : 0;
    const int nN = (p.N + kBM - 1) / kBM, nKB = (p.K + kBK - 1) / kBK;
    const int64_t nT = (p.M + TN - 1) / TN;
    bool dead = false;

    if (warp == 1 && lane == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&full_sf[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], C::EW);
        }
        mbar_init(drained, 1);
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(sTmem, C::COLS);
        tmem_relinquish();
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
    tmem_fence_after();
    const uint32_t tbase = *sTmem;
    const int64_t ntiles = (p.offsets != nullptr ? (int64_t)sCum[p.E] : nT) * nN;
    const int64_t first = blockIdx.x / S, step = gridDim.x / S;
    // this CTA's share of the k blocks
    const int kb0 = (int)((int64_t)nKB * rank / S), kb1 = (int)((int64_t)nKB * (rank + 1) / S);

    if (warp == 0) {
        // ================================ operand copies
        int it = 0;
        for (int64_t i = first; i < ntiles; i += step) {
            const Tile t = tile_at<TN>(i, p, sCum, nN, nT);
            int r[4] = {0, 0, 0, 0};
            if (kGather && lane < TN / 4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int q = 4 * lane + j;
                    const int v = q < t.valid ? __ldg(p.rows + t.m0 + q) : 0;
                    r[j] = v >= 0 && v < p.R ? v : 0;  // a row outside x: its scales become NaN (below)
                }
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % NS;
                bwait(&empty[s], (uint32_t)((it / NS) & 1) ^ 1u, dead);
                if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                if (lane == 0) {
                    mbar_arrive_expect_tx(&full[s], C::A_BYTES + C::B_BYTES);
                    tma_load_3d(sA + s * C::A_BYTES, &maps.w, kb * kBK, t.n0, t.e, &full[s]);
                    if (!kGather) tma_load_2d(sB + s * C::B_BYTES, &maps.x, kb * kBK, (int)t.m0, &full[s]);
                }
                if (kGather) {
                    __syncwarp();
                    if (lane < TN / 4)
                        tma_gather4(sB + s * C::B_BYTES + lane * 512, &maps.x, kb * kBK, r[0], r[1], r[2], r[3], &full[s]);
                }
            }
            if (dead) break;
        }
        if (dead) {  // the copies in flight must land before the CTA's shared memory goes
            bool gave_up = false;
            for (int j = it > NS ? it - NS : 0; j < it; ++j) bwait(&full[j % NS], (uint32_t)((j / NS) & 1), gave_up);
        }
    } else if (warp == 1) {
        // ================================ MMA issue (one thread)
        if (lane == 0) {
            constexpr uint32_t idesc = idesc_mxf8(kBM, TN);
            int it = 0, at = 0;  // k blocks; accumulators handed over
            for (int64_t i = first; i < ntiles && !dead; i += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const bool fresh = kWF32 || kb == kb0;  // starts an accumulator
                    if (fresh) {
                        bwait(&acc_empty[at & 1], (uint32_t)((at >> 1) & 1) ^ 1u, dead);
                        tmem_fence_after();
                    }
                    const int s = it % NS;
                    const uint32_t ph = (uint32_t)((it / NS) & 1);
                    bwait(&full[s], ph, dead);
                    bwait(&full_sf[s], ph, dead);
                    if (dead) break;
                    tmem_fence_after();
                    const uint32_t sfa = tbase + C::COL_SFA + 4 * (it & 1), sfb = tbase + C::COL_SFB + 4 * C::NB * (it & 1);
                    const uint32_t sf = smem_u32(sSF + s * C::SF_BYTES);
                    tmem_cp_scales(sfa, sdesc_scales(sf));
#pragma unroll
                    for (int b = 0; b < C::NB; ++b) tmem_cp_scales(sfb + 4 * b, sdesc_scales(sf + 512 * (1 + b)));
                    const uint64_t a = sdesc_kmajor_sw128(smem_u32(sA + s * C::A_BYTES), 1024);
                    const uint64_t b = sdesc_kmajor_sw128(smem_u32(sB + s * C::B_BYTES), 1024);
                    const uint32_t d = tbase + (uint32_t)((at & 1) * TN);
                    const int nk = min(4, (p.K - kb * kBK) / 32);  // past K the scale bytes are padding: no MMA there
                    for (int k = 0; k < nk; ++k)
                        umma_mxf8(d, a + 2 * k, b + 2 * k, idesc | ((uint32_t)k << 4) | ((uint32_t)k << 29), sfa, sfb,
                                  (uint32_t)(!fresh || k > 0));
                    umma_commit(&empty[s]);
                    if (kWF32 || kb + 1 == kb1) {
                        umma_commit(&acc_full[at & 1]);
                        ++at;
                    }
                }
            }
            if (dead) {  // the MMAs in flight must end before their operands and accumulators go
                umma_commit(drained);
                bool gave_up = false;
                bwait(drained, 0, gave_up);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ================================ scales
        int it = 0;
        const uint32_t ones = 0x7F7F7F7Fu;  // 2^0
        auto publish = [&](int j) {  // this warp's writes of stage j are visible to the copies that follow
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&full_sf[j % NS]);
        };
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN>(i, p, sCum, nN, nT);
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
            const uint8_t *ws = reinterpret_cast<const uint8_t *>(p.w_scales) + ((int64_t)t.e * nN + t.n0 / kBM) * nKB;
            uint32_t mine = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const int s = it % NS;
                if (!kWF32 && ((kb - kb0) & 31) == 0) mine = kb + lane < kb1 ? __ldg(ws + kb + lane) : 0;
                bwait(&empty[s], (uint32_t)((it / NS) & 1) ^ 1u, dead);
                if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                unsigned char *sf = sSF + s * C::SF_BYTES;
                const uint32_t w = kWF32 ? ones : __shfl_sync(0xffffffffu, mine, (kb - kb0) & 31) * 0x01010101u;
                *reinterpret_cast<uint4 *>(sf + lane * 16) = make_uint4(w, w, w, w);
#pragma unroll
                for (int j = 0; j < (TN + 31) / 32; ++j) {
                    unsigned char *dst = sf + 512 * (1 + j / 4) + lane * 16 + (j % 4) * 4;
                    if (ok[j] >= 0) cp_async4(smem_u32(dst), src[j] + (int64_t)kb * 512, ok[j] > 0);
                    else *reinterpret_cast<uint32_t *>(dst) = 0xFFFFFFFFu;
                }
                cp_async_commit();
                if (it >= C::SF_AHEAD - 1) {
                    cp_async_wait<C::SF_AHEAD - 1>();
                    publish(it - (C::SF_AHEAD - 1));
                }
            }
        }
        cp_async_wait<0>();
        if (!dead)
            for (int j = it >= C::SF_AHEAD - 1 ? it - (C::SF_AHEAD - 1) : 0; j < it; ++j) publish(j);
    } else if (warp >= 4) {
        // ================================ epilogue: warp w holds the accumulator's lanes 32 (w % 4) ...
        const int q = warp & 3;
        const uint32_t tq = tbase + ((uint32_t)(32 * q) << 16);
        int at = 0;
        float *red = reinterpret_cast<float *>(sA);  // split: this CTA's sums [token][128], in the stages (free by then)
        for (int64_t i = first; i < ntiles && !dead; i += step) {
            const Tile t = tile_at<TN>(i, p, sCum, nN, nT);
            const int n = t.n0 + 32 * q + lane;
            auto emit = [&](int tok, float v) {
                if (S > 1) red[tok * kBM + 32 * q + lane] = v;
                else if (n < p.N) store_out(p, t.m0 + tok, n, v);
            };
            if constexpr (kWF32) {
                float acc[TN];
#pragma unroll
                for (int c = 0; c < TN; ++c) acc[c] = 0.f;
                const float *ws = reinterpret_cast<const float *>(p.w_scales) + ((int64_t)t.e * nN + t.n0 / kBM) * nKB;
                float mine = 0.f;
                for (int kb = kb0; kb < kb1; ++kb, ++at) {
                    if (((kb - kb0) & 31) == 0) mine = kb + lane < kb1 ? __ldg(ws + kb + lane) : 0.f;
                    bwait(&acc_full[at & 1], (uint32_t)((at >> 1) & 1), dead);
                    if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                    tmem_fence_after();
                    const float sc = __shfl_sync(0xffffffffu, mine, (kb - kb0) & 31);
#pragma unroll
                    for (int c = 0; c < TN; c += 16) {
                        uint32_t v[16];
                        tmem_ld16(tq + (uint32_t)((at & 1) * TN + c), v);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 16; ++j) acc[c + j] = fmaf(__uint_as_float(v[j]), sc, acc[c + j]);
                    }
                    tmem_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_empty[at & 1]);
                }
                if (!dead) {
#pragma unroll
                    for (int c = 0; c < TN; ++c)
                        if (c < t.valid) emit(c, acc[c]);
                }
            } else {
                bwait(&acc_full[at & 1], (uint32_t)((at >> 1) & 1), dead);
                if (__any_sync(0xffffffffu, dead)) { dead = true; break; }
                tmem_fence_after();
                for (int c = 0; c < t.valid; c += 16) {
                    uint32_t v[16];
                    tmem_ld16(tq + (uint32_t)((at & 1) * TN + c), v);
                    tmem_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < t.valid) emit(c + j, __uint_as_float(v[j]));
                }
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[at & 1]);
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
            const Tile t = tile_at<TN>(first, p, sCum, nN, nT);
            const int n = t.n0 + (tid & (kBM - 1));
            const uint32_t mine = smem_u32(sA) + (uint32_t)(tid & (kBM - 1)) * 4;
            for (int tok = rank + S * (tid / kBM); tok < t.valid; tok += S * (C::NT / kBM)) {
                float v = 0.f;
                for (int r = 0; r < S; ++r) v += ld_cluster_f32(mapa(mine, (uint32_t)r) + (uint32_t)tok * kBM * 4);
                if (n < p.N) store_out(p, t.m0 + tok, n, v);
            }
        }
        __syncwarp();
        cluster_sync_all();
    } else {
        __syncthreads();
    }
    tmem_fence_after();
    if (warp == 3) tmem_dealloc(tbase, C::COLS);
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

template <int TN, bool kWF32, bool kGather>
cudaError_t launch_one(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    using C = Cfg<TN, kWF32>;
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
        const cuuint32_t bx[2] = {kBK, kGather ? 1u : (cuuint32_t)TN};
        if ((e = encode_u8(fn, &maps.x, 2, a.x, dx, sx, bx)) != cudaSuccess) return e;
    }
    auto kern = linear_kernel<TN, kWF32, kGather>;
    constexpr int smem = C::SMEM > kSmemMin ? C::SMEM : kSmemMin;
    {
        int dev = 0;
        if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
        if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
        static bool ready[64];
        std::lock_guard<std::mutex> lock(g_mu);
        if (!ready[dev]) {
            if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem)) != cudaSuccess) return e;
            ready[dev] = true;
        }
    }
    const int64_t nN = (a.N + kBM - 1) / kBM, nKB = (a.K + kBK - 1) / kBK;
    // token tiles: their number for one weight, an upper bound for experts (the offsets are on the device)
    int64_t nT = (a.M + TN - 1) / TN;
    if (a.offsets != nullptr) nT = std::min<int64_t>(a.M, nT + std::min<int64_t>(a.E, a.M) - 1);
    const int64_t bound = nT * nN;
    int64_t S = std::min<int64_t>(std::min<int64_t>(num_sms / bound, 8), nKB / 2);
    if (S < 1) S = 1;
    LinearParams p{};
    p.x_scales = a.x_scales; p.w_scales = a.w_scales; p.rows = a.rows; p.offsets = a.offsets; p.out = a.out;
    p.M = a.M; p.R = a.R; p.N = a.N; p.K = a.K; p.E = a.E; p.out_f32 = a.out_f32; p.split = (int)S;
    p.status = a.status;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = dim3((unsigned)(S > 1 ? bound * S : std::min<int64_t>(bound, num_sms)));
    cfg.blockDim = dim3(C::NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = S > 1 ? 2 : 1;
    mark_main_kernel(stream, true);
    e = cudaLaunchKernelEx(&cfg, kern, maps, p);
    mark_main_kernel(stream, false);
    return e;
}

template <int TN>
cudaError_t launch_tn(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    if (a.w_scales_f32)
        return a.rows != nullptr ? launch_one<TN, true, true>(a, num_sms, stream) : launch_one<TN, true, false>(a, num_sms, stream);
    return a.rows != nullptr ? launch_one<TN, false, true>(a, num_sms, stream) : launch_one<TN, false, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, int num_sms, cudaStream_t stream) {
    const int64_t per = a.offsets != nullptr ? (a.M + a.E - 1) / a.E : a.M;  // tokens a weight meets
    if (per <= 16) return launch_tn<16>(a, num_sms, stream);
    if (per <= 32) return launch_tn<32>(a, num_sms, stream);
    if (per <= 64) return launch_tn<64>(a, num_sms, stream);
    return launch_tn<128>(a, num_sms, stream);
}

}  // namespace mhc
