// Expert products of a mixture-of-experts layer on the 5th-generation tensor cores: for rows p grouped
// by expert (expert e owns rows offsets[e] .. offsets[e + 1]) and stacked weights W [E][N][K],
//
//   y[p][n] = sum_k W_e[n][k] x[rows[p]][k]
//
// with W and x in INT8 (per-token x per-channel scales), FP8 E4M3 (the same) or W packed INT4 with x in
// fp16 / bf16; optionally N = 2 I and y[p][i] = silu(gate) up of rows i and I + i of W.
//
// Swap-AB: the MMA's M dimension is weight rows (TMEM lanes), its N dimension the activation rows of one
// expert, so that a ragged group costs its own length rounded up to 16 or 32 and not to a 128-row tile.  An
// expert's rows are cut into blocks of nearly equal length; a tile is (expert, row block, weight rows), row
// blocks innermost so that the CTAs that run together share weight tiles in L2.  Every CTA derives the tile
// list from the offsets in device memory, so the host never waits for them.
//
// Two shapes (see choose_pair):
//   pair    two CTAs per tile of 256 weight rows and up to 256 activation rows (cta_group::2): each CTA
//           brings 128 weight rows and half of the activation rows, so a stage moves two thirds of the
//           bytes that a CTA of its own would move for the same MMA
//   single  one CTA per tile of 128 weight rows and up to 64 activation rows with a deeper ring: few rows
//           per expert, where the weights' bytes are all that counts
//
// Persistent warp-specialized CTA, one per SM:
//   warp 0      TMA: weight tiles (8-bit kinds) and, when the rows lie in order, activations
//   warp 1      an elected thread issues tcgen05.mma into one of two accumulators
//   warp 2      allocates tensor memory; in the pair's second CTA it and warp 1 tell the first that a stage is filled
//   warp 3      (INT4) packed weight tiles, 128 rows x 64 bytes (two stages), into a ring of their own
//   warps 4-7   epilogue of the previous tile: scales, SwiGLU, conversion, stores (4-11 for 8-bit pairs)
//   then        four warps that gather indexed activation rows by cp.async (TMA's gather of four rows a
//               request took 32 cycles for its 512 bytes, four times what the MMAs leave), and for INT4
//               three groups of four warps that dequantize every third packed tile each
//
// Measured on B200 (graphs of calls, short ones after a pause for full clocks and long ones for the clocks that the
// power cap leaves), 16384 rows over 32 experts of 4096 x 4096, 0.55 T products: INT8 with SwiGLU 225 and 266 us (2.4 and
// 2.1 POPS, 0.71 of twice the bf16 burst and of twice the sustained rate), INT4 with bf16 rows 497 and 571 us (1.11 and
// 0.96 PFLOP/s, 0.65 and 0.66 of those rates; 449 and 523 us where the rows already lie in order).  32 rows over 8 INT8
// experts of 4096 x 14336, 466 MB: 72 to 76 us (6.1 TB/s and more, 0.95 of the copy rate).
#include "grouped.cuh"

#include <algorithm>
#include <climits>

namespace wq {
namespace {

using namespace sm100;
using namespace grouped;

enum Kind { K_I8, K_FP8, K_W4H, K_W4B };  // INT8, E4M3, INT4 weights with fp16 / bf16 activations

constexpr int STAGE_K = 128;           // bytes of k per stage and row (128 INT8/FP8 or 64 16-bit values)
constexpr uint32_t A_BYTES = BM * STAGE_K;
constexpr int PK = 2;                  // stages per packed INT4 tile
constexpr int P_ROW = PK * 32;         // and bytes of a weight row (128 codes)
constexpr uint32_t P_BYTES = BM * P_ROW;
constexpr int EPI_WARP0 = 4, GATHER_WARPS = 4, DQ_GROUPS = 3;
constexpr int MAX_STAGES = 8, PSTAGES = DQ_GROUPS;   // packed slots: one per dequantizing group
constexpr unsigned SITE_PRODUCER = 0x1001, SITE_MMA = 0x1002, SITE_EPILOGUE = 0x1004, SITE_DRAIN = 0x1008,
                   SITE_DEQUANT = 0x1010, SITE_PACKED = 0x1020, SITE_GATHER = 0x1040;

struct Bars {
    uint64_t full[MAX_STAGES], empty[MAX_STAGES];  // TMA copies of a stage landed / its MMAs done
    uint64_t put[MAX_STAGES];  // what warps write of a stage: gathered rows (an arrival per thread, when its
                               // copies land), dequantized weights (one per warp) and, in a pair's first CTA,
                               // word that the second's share is there
    uint64_t pk_full[PSTAGES], pk_empty[PSTAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

__host__ __device__ constexpr bool is_w4(Kind k) { return k == K_W4H || k == K_W4B; }

template <Kind KIND, bool GATHER, bool PAIR>
struct Layout {
    static constexpr bool W4 = is_w4(KIND);
    static constexpr int BR = PAIR ? 256 : 64;               // activation rows of a tile, at most
    static constexpr int SR = PAIR ? BR / 2 : BR;            // of them in this CTA's shared memory
    static constexpr uint32_t B_BYTES = SR * STAGE_K;
    static constexpr int STAGES = PAIR ? 6 : 8;
    static constexpr int BOX = PAIR ? 64 : 16;               // rows per box when the activations lie in order
    static constexpr int EPI_WARPS = PAIR && !W4 ? 8 : 4;    // 8: two per 32 TMEM lanes, half the rows each
    static constexpr int GA_WARP0 = EPI_WARP0 + EPI_WARPS;
    static constexpr int DQ_WARP0 = GA_WARP0 + (GATHER ? GATHER_WARPS : 0);
    static constexpr int THREADS = 32 * (DQ_WARP0 + (W4 ? 4 * DQ_GROUPS : 0));
    static constexpr uint32_t OFF_B = STAGES * A_BYTES;
    static constexpr uint32_t OFF_P = OFF_B + STAGES * B_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_P + (W4 ? PSTAGES * P_BYTES : 0);
    static constexpr uint32_t OFF_SRC = OFF_BAR + 1024;                   // bits [2][BR]: rows whose index is bad
    static constexpr uint32_t OFF_SX = OFF_SRC + (GATHER ? 2 * BR / 8 : 0);  // float [2][BR] (8-bit kinds)
    static constexpr uint32_t OFF_TAB = OFF_SX + (W4 ? 0 : 2 * BR * 4);   // int offsets[E + 1], tiles[E + 1]
    static constexpr size_t smem(int E) { return 1024 + OFF_TAB + 2 * (size_t)(E + 1) * 4; }
    static_assert(PAIR || !W4, "INT4 with few rows has a kernel of its own");
    static_assert(smem(MAX_E) <= 232448, "fits the shared memory of a CTA");
    static_assert(STAGES <= MAX_STAGES && (!W4 || STAGES == PK * DQ_GROUPS), "ring: two stage slots per group");
};
static_assert(sizeof(Bars) <= 1024, "barriers fit their space");

template <Kind KIND, bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (PAIR) {
        if (KIND == K_I8) mma_i8_pair(d, a, b, idesc, acc);
        else if (KIND == K_FP8) mma_f8f6f4_pair(d, a, b, idesc, acc);
        else mma_f16_pair(d, a, b, idesc, acc);
    } else {   // INT4 comes in pairs only
        if (KIND == K_I8) mma_i8(d, a, b, idesc, acc);
        else mma_f8f6f4(d, a, b, idesc, acc);
    }
}

template <Kind KIND>
__host__ __device__ constexpr uint32_t idesc_rows(int m, int rows) {
    return KIND == K_I8 ? make_idesc(2, 1, 1, m, rows)
                        : make_idesc(1, KIND == K_W4B ? 1 : 0, KIND == K_W4B ? 1 : 0, m, rows);
}

__device__ __forceinline__ uint32_t bfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

// What a thread needs of a group's scale s and zero point z to dequantize its codes.
template <bool BF>
struct GroupConst {
    uint32_t zc, hi, lo;
    // fp16: -(1024 + z), -(64 + z) and s.  bf16: -(128 + z) twice, and s = hi + lo, two bf16 values that
    // hold the 11 bits of s (an infinite s: lo is zero).
    __device__ __forceinline__ void set(uint32_t s16, uint32_t z) {
        if (BF) {
            const float s = half_bits_to_float((uint16_t)s16);
            const uint32_t h = float_to_bf16_bits_rn(s);
            const uint32_t l = isinf(s) ? 0u : float_to_bf16_bits_rn(s - __uint_as_float(h << 16));
            zc = 0xC300C300u + z * 0x00010001u;
            hi = h * 0x00010001u;
            lo = l * 0x00010001u;
        } else {
            zc = 0xD400E400u + z * 0x00100001u;
            hi = s16 * 0x00010001u;
            lo = 0;
        }
    }
};

// One word of 8 codes -> 8 weights s (q - z) in k order, each rounded once to the activations' type (the
// tensor cores take both operands in one type).
// fp16: a byte's two nibbles become 1024 + q and 1024 + 16 q by one PRMT and one LOP3, an exact fma by
// (1, 1/16) with -(1024 + z), -(64 + z) leaves q - z, and one product rounds.
// bf16: 128 + q has 8 bits, so a nibble can only sit in the lowest bits: the odd codes come from the word
// shifted by 4.  (q - z) hi + (q - z) lo in one fma after a product whose own rounding is 2^-16 of the result.
template <bool BF>
__device__ __forceinline__ uint4 dequant_word(uint32_t w, uint32_t magic, const GroupConst<BF> &g) {
    uint32_t o[4];
    const uint32_t w4 = w >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF) {
            const uint32_t h = mask_or(prmt(w, w4, 0x4400u + 0x1111u * i), 0x000F000Fu, magic);
            const uint32_t d = bfma2(h, 0x3F803F80u, g.zc);
            o[i] = bfma2(d, g.hi, bfma2(d, g.lo, 0x80008000u));
        } else {
            const uint32_t h = mask_or(prmt(w, 0u, 0x4040u + 0x0101u * i), 0x00F0000Fu, magic);
            o[i] = hmul2(hfma2(h, 0x2C003C00u, g.zc), g.hi);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// SWIGLU: a CTA's 128 weight rows are, per 32 TMEM lanes, 16 gate rows and the 16 up rows that belong to
// them, so gate and up of one output meet by a shuffle inside a warp.
template <Kind KIND, bool GATHER, bool SWIGLU, bool PAIR>
__global__ void __launch_bounds__(Layout<KIND, GATHER, PAIR>::THREADS, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                        const Args a) {
    using L = Layout<KIND, GATHER, PAIR>;
    constexpr bool W4 = L::W4, TMA_STAGE = !W4 || !GATHER;  // the stage's barrier `full` is used
    constexpr int BR = L::BR, STEP = PAIR ? 32 : 16, STAGES = L::STAGES;
    constexpr int BNC = SWIGLU ? BM / 2 : BM;          // output columns of this CTA's share of a tile
    constexpr int BN = PAIR ? 2 * BNC : BNC;
    constexpr int KE = W4 ? STAGE_K / 2 : STAGE_K;     // k values per stage
    constexpr uint32_t TMEM_COLS = 2 * BR;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bar = reinterpret_cast<Bars *>(base + L::OFF_BAR);
    uint32_t *bad_tab = reinterpret_cast<uint32_t *>(base + L::OFF_SRC);
    float *sx_tab = reinterpret_cast<float *>(base + L::OFF_SX);
    int *off = reinterpret_cast<int *>(base + L::OFF_TAB), *tiles = off + a.E + 1;
    const uint32_t sA = smem_u32(base), sB = smem_u32(base + L::OFF_B), sP = smem_u32(base + L::OFF_P);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = PAIR ? (int)cluster_ctarank() : 0;
    const int first = PAIR ? (int)blockIdx.x >> 1 : (int)blockIdx.x, stride = PAIR ? (int)gridDim.x >> 1 : (int)gridDim.x;
    // Stages of a tile.  INT4: whole packed tiles; past the depth codes, scales and activations are zeros.
    const int packs = (a.K + PK * KE - 1) / (PK * KE), kst = W4 ? packs * PK : (a.K + KE - 1) / KE;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bar->full[s]), 1);
            mbar_init(smem_u32(&bar->empty[s]), 1);
            mbar_init(smem_u32(&bar->put[s]), max(1, (GATHER ? 32 * GATHER_WARPS : 0) + (W4 ? 4 : 0) + (PAIR && rank == 0)));
        }
        for (int p = 0; p < PSTAGES; ++p) {
            mbar_init(smem_u32(&bar->pk_full[p]), 1);
            mbar_init(smem_u32(&bar->pk_empty[p]), 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar->acc_full[i]), 1);
            mbar_init(smem_u32(&bar->acc_empty[i]), (PAIR ? 2 : 1) * L::EPI_WARPS);
        }
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        if (!GATHER) prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
    }
    if (warp == 1) build_table<BR>(a, off, tiles, lane);
    if (warp == 2) {
        if (PAIR) {
            tmem_alloc_pair(smem_u32(&bar->tmem_base), TMEM_COLS);
            tmem_relinquish_pair();
        } else {
            tmem_alloc(smem_u32(&bar->tmem_base), TMEM_COLS);
            tmem_relinquish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // the other CTA's barriers are set up before anything arrives on them
    tc_fence_after();
    const uint32_t tmem_base = bar->tmem_base;
    const WaitCtl ctl{&bar->abort, a.status, a.limit_ns};
    Tile w;

    // First weight row (of the stacked [E N] rows) of lane group i (16 lanes) of this CTA's share of tile t.
    auto weight_row = [&](const Tile &t, int i) {
        return t.e * a.N + t.n0 + rank * BNC + (SWIGLU ? (i & 1) * (a.N / 2) + (i >> 1) * 16 : i * 16);
    };
    constexpr int WB = W4 ? P_ROW : STAGE_K;
    // WB bytes of k (block kb) of this CTA's 128 weight rows of tile w.  SwiGLU with I % 16 == 0: one box of
    // the weights seen as [E][I / 16][2][16][K], whose rows come as 16 gate rows, their 16 up rows, ...
    auto load_weights = [&](uint32_t dst, uint32_t fb, int kb) {
        if (!SWIGLU) {
            tma_load_2d(dst, &tmap_w, fb, kb * WB, weight_row(w, 0));
        } else if (a.box) {
            tma_load_5d(dst, &tmap_w, fb, kb * WB, 0, 0, (w.n0 + rank * BNC) >> 4, w.e);
        } else {
            for (int i = 0; i < 8; ++i) tma_load_2d(dst + i * 16 * WB, &tmap_w, fb, kb * WB, weight_row(w, i));
        }
    };
    // Activation rows that this CTA holds of tile t, and the first of them.
    auto local_rows = [&](const Tile &t) { return (t.rows + STEP - 1) / STEP * STEP / (PAIR ? 2 : 1); };

    if (warp == 0) {
        // -------------------------------------------------------------------- TMA: weights (8-bit), ordered rows
        // The warp runs the loop together and one elected lane issues, so that the operands stay uniform.
        if (TMA_STAGE) {
            const bool leader = elect_one();
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; ok && get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride) {
                const int boxes = GATHER ? 0 : (local_rows(w) + L::BOX - 1) / L::BOX;
                const int x0 = w.r0 + rank * local_rows(w);
                const uint32_t bytes = boxes * L::BOX * STAGE_K + (W4 ? 0 : A_BYTES);
                for (int kb = 0; kb < kst; ++kb, ++it) {
                    const uint32_t s = it % STAGES, u = it / STAGES;
                    const uint32_t fb = smem_u32(&bar->full[s]);
                    ok = wait_parity_lean(smem_u32(&bar->empty[s]), (u & 1) ^ 1, ctl, SITE_PRODUCER);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    if (leader) {
                        mbar_arrive_expect_tx(fb, bytes);
                        if (!W4) load_weights(sA + s * A_BYTES, fb, kb);
                        for (int i = 0; i < boxes; ++i)
                            tma_load_2d(sB + s * L::B_BYTES + i * L::BOX * STAGE_K, &tmap_x, fb, kb * KE, x0 + i * L::BOX);
                    }
                    __syncwarp();
                }
            }
            // Every issued copy lands before the CTA leaves.
            for (uint32_t s = 0; s < STAGES; ++s) {
                const uint32_t issued = it > s ? (it - s - 1) / STAGES + 1 : 0;
                if (issued) drain_parity(smem_u32(&bar->full[s]), (issued - 1) & 1, DRAIN_NS, a.status, SITE_DRAIN);
            }
        }
        __syncwarp();
    } else if (PAIR && rank == 1 && (warp == 1 || warp == 2)) {
        // -------------------------------------------------------------------- the second CTA's stages are filled
        // Each warp tells the first CTA of every other stage, so that the fence of one overlaps the other's wait.
        const bool leader = elect_one();
        uint32_t it = warp - 1, end = 0;
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride) {
            for (end += kst; it < end; it += 2) {
                const uint32_t s = it % STAGES, ph = (it / STAGES) & 1;
                const uint32_t fb = smem_u32(&bar->full[s]), pb = smem_u32(&bar->put[s]);
                if (GATHER || W4)
                    ok = TMA_STAGE ? wait_parity2(fb, ph, pb, ph, ctl, SITE_MMA) : wait_parity_lean(pb, ph, ctl, SITE_MMA);
                else
                    ok = wait_parity_lean(fb, ph, ctl, SITE_MMA);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                if (GATHER) fence_proxy_async_smem();  // rows copied by cp.async, read by the tensor cores
                if (leader) {
                    fence_release_smem();
                    mbar_arrive_cluster(mapa_shared(pb, 0));
                }
                __syncwarp();
            }
        }
        // The first CTA's commits arrive on this one's barriers too: all of them have when the drain has.
        if (warp == 1 && leader) drain_parity(smem_u32(&bar->drain), 0, DRAIN_NS, a.status, SITE_DRAIN);
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------------------- MMA issuer
        const bool leader = elect_one();
        const uint64_t desc_a = umma_desc_sw128_kmajor(sA), desc_b = umma_desc_sw128_kmajor(sB);
        uint32_t s = 0, ph = 0, n = 0;
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride, ++n) {
            const uint32_t acc = n & 1, d = tmem_base + acc * BR;
            const uint32_t idesc = idesc_rows<KIND>(PAIR ? 2 * BM : BM, local_rows(w) * (PAIR ? 2 : 1));
            const uint32_t ae = smem_u32(&bar->acc_empty[acc]), ap = ((n >> 1) & 1) ^ 1;
            ok = PAIR ? wait_parity_cluster(ae, ap, ctl, SITE_MMA) : wait_parity_lean(ae, ap, ctl, SITE_MMA);
            if (!(ok = __all_sync(0xffffffffu, ok))) break;
            for (int kb = 0; kb < kst; ++kb) {
                const uint32_t fb = smem_u32(&bar->full[s]), pb = smem_u32(&bar->put[s]);
                if (PAIR)
                    ok = TMA_STAGE ? wait_parity_cluster(pb, ph, fb, ctl, SITE_MMA)
                                   : wait_parity_cluster(pb, ph, ctl, SITE_MMA);
                else
                    ok = GATHER ? wait_parity2(fb, ph, pb, ph, ctl, SITE_MMA) : wait_parity_lean(fb, ph, ctl, SITE_MMA);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                if (GATHER) fence_proxy_async_smem();  // rows copied by cp.async, read by the tensor cores
                if (leader) {
                    const uint64_t da = desc_a + s * (A_BYTES >> 4), db = desc_b + s * (L::B_BYTES >> 4);
#pragma unroll
                    for (int kk = 0; kk < STAGE_K / 32; ++kk)
                        mma_step<KIND, PAIR>(d, da + 2 * kk, db + 2 * kk, idesc, kb != 0 || kk != 0);
                    if (PAIR) tc_commit_pair_both(smem_u32(&bar->empty[s]));
                    else tc_commit(smem_u32(&bar->empty[s]));
                }
                __syncwarp();
                if (++s == STAGES) {
                    s = 0;
                    ph ^= 1;
                }
            }
            if (ok && leader) {
                if (PAIR) tc_commit_pair_both(smem_u32(&bar->acc_full[acc]));
                else tc_commit(smem_u32(&bar->acc_full[acc]));
            }
            __syncwarp();
        }
        if (leader) {
            if (PAIR) tc_commit_pair_both(smem_u32(&bar->drain));
            else tc_commit(smem_u32(&bar->drain));
            drain_parity(smem_u32(&bar->drain), 0, DRAIN_NS, a.status, SITE_DRAIN);
        }
        __syncwarp();
    } else if (W4 && warp == 3) {
        // -------------------------------------------------------------------- packed weight tiles
        const bool leader = elect_one();
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride) {
            for (int b = 0; b < packs; ++b, ++it) {
                const uint32_t p = it % PSTAGES, u = it / PSTAGES;
                ok = wait_parity_lean(smem_u32(&bar->pk_empty[p]), (u & 1) ^ 1, ctl, SITE_PACKED);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (leader) {
                    const uint32_t fb = smem_u32(&bar->pk_full[p]);
                    mbar_arrive_expect_tx(fb, P_BYTES);
                    load_weights(sP + p * P_BYTES, fb, b);
                }
                __syncwarp();
            }
        }
        for (uint32_t p = 0; p < PSTAGES; ++p) {
            const uint32_t issued = it > p ? (it - p - 1) / PSTAGES + 1 : 0;
            if (issued) drain_parity(smem_u32(&bar->pk_full[p]), (issued - 1) & 1, DRAIN_NS, a.status, SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp >= EPI_WARP0 && warp < EPI_WARP0 + L::EPI_WARPS) {
        // -------------------------------------------------------------------- epilogue
        const int q = warp & 3;                   // TMEM lanes 32 q .. 32 q + 31
        constexpr int PARTS = L::EPI_WARPS / 4, ET = 32 * L::EPI_WARPS;
        const int part = (warp - EPI_WARP0) >> 2; // takes every PARTS-th 32 rows
        const uint32_t t_row = tmem_base + ((uint32_t)(32 * q) << 16);
        uint32_t n = 0;
        bool ok = true;
        for (int t = first; get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride, ++n) {
            const uint32_t acc = n & 1, u = n >> 1;
            uint32_t *bad = bad_tab + acc * (BR / 32);
            float *sxs = sx_tab + acc * BR;
            if (GATHER || !W4) {
                for (int r0 = 32 * (warp - EPI_WARP0); r0 < w.rows; r0 += ET) {
                    const int r = r0 + lane;
                    int v = w.r0 + r;
                    bool out = false;
                    if (GATHER && r < w.rows) {
                        v = __ldg(a.rows + v);
                        out = (unsigned)v >= (unsigned)a.T;
                    }
                    if (GATHER) {
                        const uint32_t m = __ballot_sync(0xffffffffu, out);
                        if (lane == 0) bad[r0 / 32] = m;
                    }
                    if (!W4) sxs[r] = r < w.rows && !out ? __ldg(a.sx + (size_t)v * a.sx_stride) : 0.0f;
                }
                asm volatile("bar.sync 1, %0;" ::"n"(ET) : "memory");
            }
            const int col = w.n0 + rank * BNC + (SWIGLU ? 16 * q + (lane & 15) : 32 * q + lane);
            const bool col_ok = col < a.ldy, cols_ok = __all_sync(0xffffffffu, col_ok);
            float sw = 1.0f;
            if (!W4)
                sw = a.sw_per_row ? __ldg(a.sw + min((size_t)a.E * a.N - 1,
                                                     (size_t)weight_row(w, 2 * q + (lane >> 4)) + (lane & 15)))
                                  : __ldg(a.sw + w.e);
            // After a wait has run out the warps still walk the tiles, so that all meet at the barrier.
            ok = ok && wait_parity_lean(smem_u32(&bar->acc_full[acc]), u & 1, ctl, SITE_EPILOGUE);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            for (int c = 32 * part; c < w.rows; c += 32 * PARTS) {
                uint32_t r[32];
                tmem_ld_32x32b_x32(t_row + acc * BR + c, r);
                tmem_ld_wait();
                const uint32_t zero = GATHER ? bad[c / 32] : 0u;
                const int left = w.rows - c;
                uint16_t *yt = a.y + (size_t)(w.r0 + c) * a.ldy + col;
                const bool full = left >= 32 && cols_ok;
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; j += 4) {
                    float sv[4] = {1.0f, 1.0f, 1.0f, 1.0f};
                    if (!W4) *reinterpret_cast<float4 *>(sv) = *reinterpret_cast<const float4 *>(sxs + c + j);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float f = KIND == K_I8 ? (float)(int32_t)r[j + i] : __uint_as_float(r[j + i]);
                        v[j + i] = W4 ? f : __fmul_rn(__fmul_rn(f, sv[i]), sw);
                    }
                }
                if (SWIGLU) {
                    // Lanes 0-15 hold gate rows and keep the even rows of y, lanes 16-31 up rows and the odd ones.
                    const bool up = lane >= 16;
                    float o[16];
#pragma unroll
                    for (int j = 0; j < 32; j += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + 1], 16);
                        o[j / 2] = swiglu(up ? other : v[j], up ? v[j + 1] : other);
                    }
                    if (zero)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if ((zero >> (2 * j + (up ? 1 : 0))) & 1) o[j] = 0.0f;
                    store_column<KIND == K_W4B>(yt + (up ? a.ldy : 0), 2 * (size_t)a.ldy, o,
                                                col_ok ? (left + (up ? 0 : 1)) / 2 : 0, full);
                } else {
                    if (zero)
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if ((zero >> j) & 1) v[j] = 0.0f;
                    store_column<KIND == K_W4B>(yt, (size_t)a.ldy, v, col_ok ? left : 0, full);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) {
                    fence_release_smem();
                    mbar_arrive_cluster(mapa_shared(smem_u32(&bar->acc_empty[acc]), 0));
                } else {
                    mbar_arrive(smem_u32(&bar->acc_empty[acc]));
                }
            }
        }
    } else if (GATHER && warp >= L::GA_WARP0 && warp < L::GA_WARP0 + GATHER_WARPS) {
        // -------------------------------------------------------------------- gathered activations
        // Thread (16-byte chunk c of a row's 128 bytes, row rr of every 16): cp.async into the 128-byte
        // swizzle, whose completion arrives on the stage's barrier by itself.  Padding repeats the last row; an
        // index outside x reads row 0 (the epilogue writes zeros for it).
        constexpr int PASSES = L::SR / 16;
        const int gt = (int)threadIdx.x - 32 * L::GA_WARP0, c = gt & 7, rr = gt >> 3;
        const size_t pitch = (size_t)a.K * (W4 ? 2 : 1);
        const uint32_t dst0 = sB + rr * STAGE_K + ((c ^ (rr & 7)) << 4);
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, STEP>(a, off, tiles, t, w); t += stride) {
            const int mine = local_rows(w);
            const uint8_t *src[PASSES];
#pragma unroll
            for (int j = 0; j < PASSES; ++j) {
                const int v = __ldg(a.rows + w.r0 + min(rank * mine + 16 * j + rr, w.rows - 1));
                src[j] = a.x + ((unsigned)v < (unsigned)a.T ? (size_t)v : 0) * pitch + c * 16;
            }
            for (int kb = 0; kb < kst; ++kb, ++it) {
                const uint32_t s = it % STAGES, u = it / STAGES;
                ok = wait_parity_lean(smem_u32(&bar->empty[s]), (u & 1) ^ 1, ctl, SITE_GATHER);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t dst = dst0 + s * L::B_BYTES;
                const bool in = kb * STAGE_K + c * 16 < (int)pitch;   // false only past the end of the depth
#pragma unroll
                for (int j = 0; j < PASSES; ++j) {
                    if (16 * j < mine) cp_async16(dst + 16 * j * STAGE_K, in ? src[j] : a.x, in);
                    src[j] += STAGE_K;
                }
                cp_async_arrive(smem_u32(&bar->put[s]));
            }
        }
        cp_async_wait_all();
    } else if (W4 && warp >= L::DQ_WARP0) {
        // -------------------------------------------------------------------- dequantizers
        // Group d of four warps takes every third packed tile and fills stages 2 d and 2 d + 1 (packed and stage
        // slots belong to one group each); a thread takes one weight row, 128 codes.
        constexpr bool BF = KIND == K_W4B;
        const uint32_t magic = opaque_const(BF ? 0x43004300u : 0x64006400u);
        const int row = 32 * (warp & 3) + lane, d = (warp - L::DQ_WARP0) >> 2;
        const int lg = 31 - __clz(a.gs), groups = a.K >> lg, zwords = (groups + 7) / 8;
        const bool whole = a.K % (PK * KE) == 0;   // every packed tile is full, and its scales are aligned to their size
        const uint32_t pf = smem_u32(&bar->pk_full[d]), pe = smem_u32(&bar->pk_empty[d]);
        const uint32_t eb = smem_u32(&bar->empty[2 * d]), fb = smem_u32(&bar->put[2 * d]);
        const uint32_t src = sP + d * P_BYTES + row * P_ROW, s3 = (uint32_t)((row >> 1) & 3) << 4;  // 64-byte swizzle
        const uint32_t dst = sA + 2 * d * A_BYTES + row * STAGE_K, r7 = (uint32_t)(row & 7) << 4;   // 128-byte swizzle
        const uint16_t *srow = nullptr;
        const uint32_t *zrow = nullptr;
        uint2 ns = {}, cs = {};   // scales (up to four) and zeros of the group's next packed tile and of this one
        uint32_t nz = 0, cz = 0, pk0 = 0, ph = 0;
        auto load = [&](int b) {
            const int g = min(b * (PK * KE) >> lg, groups - 1);
            nz = __ldg(zrow + (g >> 3));
            const uint16_t *p = srow + g;
            if (lg >= 7) {
                ns.x = __ldg(p);
            } else if (!whole) {
                uint32_t v[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __ldg(srow + min(g + i, groups - 1));
                ns = make_uint2(v[0] | (v[1] << 16), v[2] | (v[3] << 16));
            } else if (lg == 6) {
                ns.x = __ldg(reinterpret_cast<const uint32_t *>(p));
            } else {
                ns = __ldg(reinterpret_cast<const uint2 *>(p));
            }
        };
        bool ok = true, have = true;
        auto tile_from = [&](int t, int b) {   // sets up tile t and requests the scales of its packed tile b
            have = get_tile<BN, BR, STEP>(a, off, tiles, t, w);
            if (!have) return;
            const size_t wr = min((size_t)weight_row(w, row >> 4) + (row & 15), (size_t)a.E * a.N - 1);
            srow = a.scales + wr * groups;
            zrow = a.qzeros + wr * zwords;
            if (b < packs) load(b);
        };
        auto first_of = [&](uint32_t pk) { return (int)((d + DQ_GROUPS - pk % DQ_GROUPS) % DQ_GROUPS); };
        tile_from(first, d);
        for (int t = first; ok && have; t += stride, pk0 += packs) {
            int b = first_of(pk0);
            if (b >= packs) {   // a short tile without a packed tile of this group's
                tile_from(t + stride, first_of(pk0 + packs));
                continue;
            }
            for (; b < packs; b += DQ_GROUPS, ph ^= 1) {
                cs = ns;
                cz = nz;
                const int k0 = b * (PK * KE);
                ok = wait_parity2(pf, ph, eb, ph ^ 1, ctl, SITE_DEQUANT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                uint4 v[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] = lds128(src + ((c << 4) ^ s3));
                // The codes are in registers: the slot goes back (the fence orders the reads before the next copy).
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(pe);
                if (b + DQ_GROUPS < packs) load(b + DQ_GROUPS);
                else tile_from(t + stride, first_of(pk0 + packs));
                GroupConst<BF> gc;
#pragma unroll
                for (int h = 0; h < 4; ++h) {   // 32 codes, all in one group; two of these make a stage
                    if (h == 0 || (h << 5 & (a.gs - 1)) == 0) {
                        const int g = min((k0 + 32 * h) >> lg, groups - 1), i = g - min(k0 >> lg, groups - 1);
                        const uint32_t s2 = i < 2 ? cs.x : cs.y;
                        // Past the depth weights are zero: codes (0 there) minus a zero point, times a large scale, would be
                        // infinities that the zeros of x turn into NaN.
                        const uint32_t s16 = (i & 1) ? s2 >> 16 : s2 & 0xFFFFu;
                        gc.set(k0 + 32 * h < a.K ? s16 : 0u, (cz >> (4 * (g & 7))) & 0xFu);
                    }
                    if (h == 2) {
                        ok = wait_parity_lean(eb + 8, ph ^ 1, ctl, SITE_DEQUANT);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    }
                    const uint32_t words[4] = {v[h].x, v[h].y, v[h].z, v[h].w};
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        sts128(dst + (h >> 1) * A_BYTES + (((4 * (h & 1) + j) << 4) ^ r7), dequant_word<BF>(words[j], magic, gc));
                    if (h & 1) {
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(fb + 8 * (h >> 1));
                    }
                }
                if (!ok) break;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (PAIR) cluster_sync();  // nothing of the other CTA's still arrives here
    if (warp == 2) {
        tc_fence_after();
        if (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
        else tmem_dealloc(tmem_base, TMEM_COLS);
    }
}

template <Kind KIND, bool GATHER, bool SWIGLU, bool PAIR>
wq_status launch(const CUtensorMap &tx, const CUtensorMap &tw, const Args &a, long long most_tiles, cudaStream_t st,
                 const char *who) {
    using L = Layout<KIND, GATHER, PAIR>;
    auto kern = grouped_gemm_kernel<KIND, GATHER, SWIGLU, PAIR>;
    const size_t smem = L::smem(a.E);
    static std::atomic<uint64_t> allowed{0};
    const wq_status ok = allow_smem(kern, L::smem(MAX_E), allowed, who);
    if (ok != WQ_OK) return ok;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(L::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = PAIR ? 2 : 1;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int units = PAIR ? num_sms() / 2 : num_sms();
    cfg.gridDim = dim3((unsigned)std::min<long long>(units, most_tiles) * (PAIR ? 2 : 1));
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tx, tw, a);
    if (e != cudaSuccess) return fail(WQ_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return WQ_OK;
}

// Pair tiles once the experts have rows enough to fill them, measured on B200 by rows per expert (drawn at random).
// INT4, the other side being grouped_few.cu with its tiles of 16 rows: 64 experts of 4096 x 2048, bf16, groups of 64,
// 12 rows 173 against 124 us, 18 rows 173 against 176, 22 rows 173 against 204; 8 experts of 4096 x 14336, fp16, 12 rows
// 148 against 90, 20 rows 149 against 157, 22 rows 149 against 146.  (The rounding of the weights changes here, so wq.h
// names the 22.)  8 bits, the other side being single tiles of up to 64 rows: 8 experts of 4096 x 14336, 32 rows 82
// against 77 us, 48 rows 83 against 79, 64 rows 84 against 96; 64 experts of 4096 x 2048, 32 rows 95 against 91, 48 rows
// 99 against 94, 64 rows 101 against 112: 36 gives up at most 5% up to about 50 rows.
template <Kind KIND>
bool choose_pair(const Args &a) {
    return (long long)a.R >= (is_w4(KIND) ? 22ll : 36ll) * std::min(a.E, a.R);
}

template <Kind KIND, bool PAIR>
wq_status dispatch(const void *w, Args a, bool swiglu, cudaStream_t st, const char *who) {
    constexpr bool W4 = is_w4(KIND);
    a.ldy = swiglu ? a.N / 2 : a.N;
    const int bn = (swiglu ? BM / 2 : BM) * (PAIR ? 2 : 1), br = Layout<KIND, false, PAIR>::BR;
    a.nb = (a.ldy + bn - 1) / bn;
    const long long most = ((long long)std::min(a.E, a.R) + a.R / br) * a.nb;  // tiles of any offsets
    WQ_REQUIRE(most < INT_MAX / 2, WQ_ERR_UNSUPPORTED, "%s: R (%d) x N (%d) gives too many tiles", who, a.R, a.N);
    const bool gather = a.rows != nullptr;
    constexpr int W_BYTES = W4 ? P_ROW : STAGE_K;   // of a weight row per copy
    CUtensorMap tx = {}, tw;   // tx: not used by gathered rows
    const CUtensorMapDataType xt = KIND == K_W4H ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : KIND == K_W4B ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int xb = W4 ? 2 : 1;
    if (!gather && !encode_tmap_2d(&tx, xt, xb, a.x, (uint64_t)a.K, (uint64_t)a.T, (uint64_t)a.K * xb, STAGE_K / xb,
                        Layout<KIND, false, PAIR>::BOX,
                        CU_TENSOR_MAP_SWIZZLE_128B))
        return WQ_ERR_CUDA;
    if (!encode_weights(&tw, w, W4 ? (uint64_t)a.K / 2 : (uint64_t)a.K, W_BYTES, a, swiglu)) return WQ_ERR_CUDA;
    if (gather)
        return swiglu ? launch<KIND, true, true, PAIR>(tx, tw, a, most, st, who)
                      : launch<KIND, true, false, PAIR>(tx, tw, a, most, st, who);
    return swiglu ? launch<KIND, false, true, PAIR>(tx, tw, a, most, st, who)
                  : launch<KIND, false, false, PAIR>(tx, tw, a, most, st, who);
}

// INT4 experts with fewer rows than this on average go to grouped_stream.cu, the rest to grouped_few.cu.  Measured on
// B200 by rows per expert: 8 experts of 28672 x 4096, 4 rows 109 against 152 us, 7 rows 148 against 154, 8 rows 160
// against 154 (every ninth row of an expert is another tile); 8 experts of 4096 x 14336, 6 rows 92 against 91; 64 uneven
// experts of 4096 x 2048, 6 rows 103 against 117 us, 12 rows 154 against 146.
constexpr long long STREAM_ROWS = 7;

template <Kind KIND>
wq_status run(const void *x, const void *w, Args a, bool swiglu, cudaStream_t st, const char *who) {
    a.x = static_cast<const uint8_t *>(x);
    a.status = device_status_word();
    if (!a.status) return WQ_ERR_CUDA;
    a.limit_ns = wait_limit();
    if (choose_pair<KIND>(a)) return dispatch<KIND, true>(w, a, swiglu, st, who);
    if constexpr (is_w4(KIND)) {
        if (a.R < STREAM_ROWS * std::min(a.E, a.R)) return stream_rows_w4(w, a, KIND == K_W4B, swiglu, st, who);
        return few_rows_w4(w, a, KIND == K_W4B, swiglu, st, who);
    } else return dispatch<KIND, false>(w, a, swiglu, st, who);
}

}  // namespace

bool grouped::encode_weights(CUtensorMap *map, const void *w, uint64_t row_bytes, int width, Args &a, bool swiglu) {
    const uint64_t half = (uint64_t)a.N / 2;
    const CUtensorMapSwizzle swizzle = width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
    a.box = swiglu && half % 16 == 0;
    if (!a.box)
        return encode_tmap_2d(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, row_bytes, (uint64_t)a.E * a.N, row_bytes, width,
                              swiglu ? 16 : BM, swizzle);
    const uint64_t dims[5] = {row_bytes, 16, 2, half / 16, (uint64_t)a.E};
    const uint64_t strides[4] = {row_bytes, half * row_bytes, 16 * row_bytes, (uint64_t)a.N * row_bytes};
    const uint32_t box[5] = {(uint32_t)width, 16, 2, 4, 1};
    return encode_tmap(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, w, dims, strides, box, swizzle);
}

namespace {

constexpr int MAX_SIZE = 1 << 29;   // row numbers and bytes of a row stay within 32 bits

// Checks that every grouped product makes of its sizes.
wq_status check_sizes(const char *who, int T, const int32_t *rows, const int32_t *offsets, int R, int E, int N, int K,
                      int swiglu) {
    WQ_REQUIRE_PTR(offsets, "offsets");
    WQ_REQUIRE(aligned16(rows), WQ_ERR_ALIGNMENT, "rows is not 16-byte aligned");
    WQ_REQUIRE(T > 0 && R > 0 && E > 0 && N > 0 && K > 0, WQ_ERR_INVALID_ARG,
               "%s: sizes must be positive (T=%d R=%d E=%d N=%d K=%d)", who, T, R, E, N, K);
    WQ_REQUIRE(E <= MAX_E, WQ_ERR_UNSUPPORTED, "%s: E (%d) must be at most %d", who, E, MAX_E);
    WQ_REQUIRE(T <= MAX_SIZE && R <= MAX_SIZE && K <= MAX_SIZE, WQ_ERR_UNSUPPORTED,
               "%s: T (%d), R (%d) and K (%d) must be at most %d", who, T, R, K, MAX_SIZE);
    WQ_REQUIRE(rows || R == T, WQ_ERR_INVALID_ARG, "%s: without rows, R (%d) must equal T (%d)", who, R, T);
    WQ_REQUIRE(!swiglu || N % 2 == 0, WQ_ERR_INVALID_ARG, "%s: N (%d) must be even with SwiGLU", who, N);
    WQ_REQUIRE((long long)E * N <= INT_MAX - 4 * BM, WQ_ERR_UNSUPPORTED, "%s: E * N must be below 2^31", who);
    return WQ_OK;
}

// y is written while the inputs are read.  `bits`: of a weight.
wq_status check_output(const char *who, const Args &a, const void *x, int x_bytes, const void *w, int bits, int swiglu) {
    const size_t y_bytes = (size_t)a.R * (swiglu ? a.N / 2 : a.N) * 2, weights = (size_t)a.E * a.N * a.K;
    const size_t groups = a.gs ? a.K / a.gs : 0, rows = (size_t)a.E * a.N;
    const bool bad = overlap(a.y, y_bytes, x, (size_t)a.T * a.K * x_bytes) || overlap(a.y, y_bytes, w, weights * bits / 8) ||
                     overlap(a.y, y_bytes, a.offsets, ((size_t)a.E + 1) * 4) ||
                     (a.rows && overlap(a.y, y_bytes, a.rows, (size_t)a.R * 4)) ||
                     (a.scales && overlap(a.y, y_bytes, a.scales, rows * groups * 2)) ||
                     (a.qzeros && overlap(a.y, y_bytes, a.qzeros, rows * ((groups + 7) / 8) * 4)) ||
                     (a.sx && overlap(a.y, y_bytes, a.sx, a.sx_stride ? (size_t)a.T * 4 : 4)) ||
                     (a.sw && overlap(a.y, y_bytes, a.sw, (a.sw_per_row ? rows : (size_t)a.E) * 4));
    WQ_REQUIRE(!bad, WQ_ERR_INVALID_ARG, "%s: y overlaps an input", who);
    return WQ_OK;
}

template <Kind KIND>
wq_status w4_entry(const uint16_t *x, int T, const int32_t *rows, const int32_t *offsets, int R,
                   const uint32_t *qweight, const uint16_t *scales, const uint32_t *qzeros, int E, int N, int K,
                   int group_size, int swiglu, uint16_t *y, void *stream, const char *who) {
    WQ_REQUIRE_PTR(x, "x");
    WQ_REQUIRE_PTR(qweight, "qweight");
    WQ_REQUIRE_PTR(scales, "scales");
    WQ_REQUIRE_PTR(qzeros, "qzeros");
    WQ_REQUIRE_PTR(y, "y");
    const wq_status e = check_sizes(who, T, rows, offsets, R, E, N, K, swiglu);
    if (e != WQ_OK) return e;
    WQ_REQUIRE(group_size == 32 || group_size == 64 || group_size == 128 || group_size == 256, WQ_ERR_UNSUPPORTED,
               "%s: group_size must be 32, 64, 128 or 256 (got %d)", who, group_size);
    WQ_REQUIRE(K % group_size == 0, WQ_ERR_INVALID_ARG, "%s: K (%d) must be a multiple of group_size (%d)", who, K,
               group_size);
    Args a = {};
    a.offsets = offsets;
    a.rows = rows;
    a.scales = scales;
    a.qzeros = qzeros;
    a.y = y;
    a.T = T; a.R = R; a.E = E; a.N = N; a.K = K; a.gs = group_size;
    const wq_status o = check_output(who, a, x, 2, qweight, 4, swiglu);
    if (o != WQ_OK) return o;
    return run<KIND>(x, qweight, a, swiglu != 0, as_stream(stream), who);
}

template <Kind KIND>
wq_status w8_entry(const void *xq, const float *sx, int sx_per_row, int T, const int32_t *rows, const int32_t *offsets,
                   int R, const void *wq_, const float *sw, int sw_per_row, int E, int N, int K, int swiglu,
                   uint16_t *y, void *stream, const char *who) {
    WQ_REQUIRE_PTR(xq, "xq");
    WQ_REQUIRE_PTR(sx, "sx");
    WQ_REQUIRE_PTR(wq_, "wq");
    WQ_REQUIRE_PTR(sw, "sw");
    WQ_REQUIRE_PTR(y, "y");
    const wq_status e = check_sizes(who, T, rows, offsets, R, E, N, K, swiglu);
    if (e != WQ_OK) return e;
    WQ_REQUIRE(K % 16 == 0, WQ_ERR_UNSUPPORTED, "%s: K (%d) must be a multiple of 16", who, K);
    WQ_REQUIRE(KIND != K_I8 || K <= 131056, WQ_ERR_UNSUPPORTED,
               "%s: K (%d) must be at most 131056 (int32 accumulators)", who, K);
    Args a = {};
    a.offsets = offsets;
    a.rows = rows;
    a.sx = sx;
    a.sw = sw;
    a.sx_stride = sx_per_row ? 1 : 0;
    a.sw_per_row = sw_per_row != 0;
    a.y = y;
    a.T = T; a.R = R; a.E = E; a.N = N; a.K = K;
    const wq_status o = check_output(who, a, xq, 1, wq_, 8, swiglu);
    if (o != WQ_OK) return o;
    return run<KIND>(xq, wq_, a, swiglu != 0, as_stream(stream), who);
}

}  // namespace
}  // namespace wq

extern "C" wq_status wq_grouped_gemm_w4a16(const uint16_t *x, int T, const int32_t *rows, const int32_t *offsets, int R,
                                           const uint32_t *qweight, const uint16_t *scales, const uint32_t *qzeros,
                                           int E, int N, int K, int group_size, int swiglu, uint16_t *y,
                                           void *stream) {
    return wq::w4_entry<wq::K_W4H>(x, T, rows, offsets, R, qweight, scales, qzeros, E, N, K, group_size, swiglu, y,
                                   stream, "wq_grouped_gemm_w4a16");
}

extern "C" wq_status wq_grouped_gemm_w4a16_bf16(const uint16_t *x, int T, const int32_t *rows, const int32_t *offsets,
                                                int R, const uint32_t *qweight, const uint16_t *scales,
                                                const uint32_t *qzeros, int E, int N, int K, int group_size, int swiglu,
                                                uint16_t *y, void *stream) {
    return wq::w4_entry<wq::K_W4B>(x, T, rows, offsets, R, qweight, scales, qzeros, E, N, K, group_size, swiglu, y,
                                   stream, "wq_grouped_gemm_w4a16_bf16");
}

extern "C" wq_status wq_grouped_gemm_w8a8(const int8_t *xq, const float *sx, int T, const int32_t *rows,
                                          const int32_t *offsets, int R, const int8_t *wq_, const float *sw, int E,
                                          int N, int K, int swiglu, uint16_t *y, void *stream) {
    return wq::w8_entry<wq::K_I8>(xq, sx, 1, T, rows, offsets, R, wq_, sw, 1, E, N, K, swiglu, y, stream,
                                  "wq_grouped_gemm_w8a8");
}

extern "C" wq_status wq_grouped_gemm_fp8(const uint8_t *xq, const float *sx, int sx_per_row, int T, const int32_t *rows,
                                         const int32_t *offsets, int R, const uint8_t *wq_, const float *sw,
                                         int sw_per_row, int E, int N, int K, int swiglu, uint16_t *y, void *stream) {
    return wq::w8_entry<wq::K_FP8>(xq, sx, sx_per_row, T, rows, offsets, R, wq_, sw, sw_per_row, E, N, K, swiglu, y,
                                   stream, "wq_grouped_gemm_fp8");
}
