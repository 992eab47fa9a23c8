// Expert products of a mixture-of-experts layer on the 5th-generation tensor cores: for rows p grouped
// by expert (expert e owns rows offsets[e] .. offsets[e + 1]) and stacked weights W [E][N][K],
//
//   y[p][n] = sum_k W_e[n][k] x[rows[p]][k]
//
// with W and x in INT8 (per-token x per-channel scales), FP8 E4M3 (the same) or W packed INT4 with x in
// fp16 / bf16; optionally N = 2 I and y[p][i] = silu(gate) up of rows i and I + i of W.
//
// Swap-AB: the MMA's M dimension is 128 weight rows (TMEM lanes), its N dimension the activation rows of
// one expert, so that a ragged group costs its own length rounded up to 16 and not to a 128-row tile.  An
// expert's rows are cut into blocks of at most 256 of nearly equal length; a tile is (expert, row block,
// 128 weight rows), row blocks innermost so that the CTAs that run together share weight tiles in L2.
// Every CTA derives the tile list from the offsets in device memory, so the host never waits for them.
//
// Persistent warp-specialized CTA, one per SM:
//   warp 0      activations into a shared-memory ring (128-byte swizzle): TMA gather of four indexed rows
//               per request (tile::gather4), the 32 lanes each issuing their share, or 32-row boxes when
//               the rows already lie in order; for 8-bit weights also the weight tile
//   warp 1      one thread issues tcgen05.mma into one of two 256-column fp32/int32 accumulators
//   warp 2      allocates tensor memory
//   warp 3      (INT4) packed weight tiles, 128 rows x 32 bytes, into a ring of their own
//   warps 4-7   epilogue of the previous tile: scales, SwiGLU, conversion, stores
//   warps 8-15  (INT4) dequantize packed tiles into the weight operand's shared-memory stage
#include "sm100.cuh"
#include "wq_device.cuh"
#include "wq_host.h"

#include <algorithm>
#include <climits>

namespace wq {
namespace {

using namespace sm100;

enum Kind { K_I8, K_FP8, K_W4H, K_W4B };  // INT8, E4M3, INT4 weights with fp16 / bf16 activations

constexpr int BM = 128;                // weight rows of a tile
constexpr int BR = 256;                // activation rows of a tile, at most
constexpr int STAGE_K = 128;           // bytes of k per stage and row (128 INT8/FP8 or 64 16-bit values)
constexpr int STAGES = 4;
constexpr int PSTAGES = 6;             // packed INT4 tiles
constexpr uint32_t A_BYTES = BM * STAGE_K, B_BYTES = BR * STAGE_K, P_BYTES = BM * 32;
constexpr int BOX_ROWS = 32;           // rows per box when the activations lie in order
constexpr int MAX_E = 512;
constexpr int EPI_WARP0 = 4, DQ_WARP0 = 8, DQ_WARPS = 8;
constexpr uint64_t DRAIN_NS = 2000000000ull;
constexpr unsigned SITE_PRODUCER = 0x1001, SITE_MMA = 0x1002, SITE_EPILOGUE = 0x1004, SITE_DRAIN = 0x1008,
                   SITE_DEQUANT = 0x1010, SITE_PACKED = 0x1020;

struct Bars {
    uint64_t full[STAGES], empty[STAGES];   // copies of a stage landed / its MMAs done
    uint64_t dq_full[STAGES];               // INT4: dequantized weight tile of the stage written
    uint64_t pk_full[PSTAGES], pk_empty[PSTAGES];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drain;
    uint32_t tmem_base;
    int abort;
};

__host__ __device__ constexpr bool is_w4(Kind k) { return k == K_W4H || k == K_W4B; }

template <Kind KIND>
struct Layout {
    static constexpr bool W4 = is_w4(KIND);
    static constexpr int THREADS = W4 ? 512 : 256;
    static constexpr uint32_t OFF_B = STAGES * A_BYTES;
    static constexpr uint32_t OFF_P = OFF_B + STAGES * B_BYTES;
    static constexpr uint32_t OFF_BAR = OFF_P + (W4 ? PSTAGES * P_BYTES : 0);
    static constexpr uint32_t OFF_SRC = OFF_BAR + 512;                    // int [2][BR]: token of each row
    static constexpr uint32_t OFF_SX = OFF_SRC + 2 * BR * 4;              // float [2][BR] (8-bit kinds)
    static constexpr uint32_t OFF_TAB = OFF_SX + (W4 ? 0 : 2 * BR * 4);   // int offsets[E + 1], tiles[E + 1]
    static size_t smem(int E) { return 1024 + OFF_TAB + 2 * (size_t)(E + 1) * 4; }
};
static_assert(sizeof(Bars) <= 512, "barriers fit their space");

struct Args {
    const int32_t *offsets, *rows;   // rows null: row p of x itself
    const float *sx, *sw;
    int sx_stride, sw_per_row;
    const uint16_t *scales;          // INT4: fp16 [E][N][K/gs]
    const uint32_t *qzeros;
    uint16_t *y;
    int T, R, E, N, K, gs;           // T: rows of x, R: grouped rows
    int nb;                          // weight-row blocks per expert
    int ldy;                         // columns of y (N, or N / 2 with SwiGLU)
    unsigned int *status;
    uint64_t limit_ns;
};

struct Tile {
    int e, n0;        // expert, first output column of the tile
    int r0, rows;     // first grouped row, number of rows
};

__device__ __forceinline__ int row_blocks(int n) { return (n + BR - 1) / BR; }

// Offsets clamped to [0, R] and made non-decreasing (a valid array is unchanged), and the exclusive
// prefix of the experts' tile counts; by one warp.
__device__ __forceinline__ void build_table(const Args &a, int *off, int *tiles, int lane) {
    int high = 0;
    for (int i0 = 0; i0 <= a.E; i0 += 32) {
        int v = i0 + lane <= a.E ? min(max(__ldg(a.offsets + i0 + lane), 0), a.R) : 0;
        v = max(v, high);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) v = max(v, __shfl_up_sync(0xffffffffu, v, o));
        if (i0 + lane <= a.E) off[i0 + lane] = v;
        high = __shfl_sync(0xffffffffu, v, 31);
    }
    __syncwarp();
    int run = 0;
    for (int i0 = 0; i0 < a.E; i0 += 32) {
        const int v = i0 + lane < a.E ? row_blocks(off[i0 + lane + 1] - off[i0 + lane]) * a.nb : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        if (i0 + lane < a.E) tiles[i0 + lane] = run + s - v;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) tiles[a.E] = run;
}

// Tile t of the list; false past its end.  BN: output columns per tile.
template <int BN>
__device__ __forceinline__ bool get_tile(const Args &a, const int *off, const int *tiles, int t, Tile &w) {
    if (t >= tiles[a.E]) return false;
    int lo = 0, hi = a.E;  // the expert e with tiles[e] <= t < tiles[e + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int first = off[lo], n = off[lo + 1] - first, rb = row_blocks(n);
    const int per = ((n + rb - 1) / rb + 15) & ~15;
    const int local = t - tiles[lo], b = local % rb;
    w.e = lo;
    w.n0 = (local / rb) * BN;
    w.r0 = first + b * per;
    w.rows = min(per, n - b * per);
    return true;
}

// Four rows of a 2-D tensor (row indices r0..r3, elements from c0) into 4 consecutive 128-byte lines.
__device__ __forceinline__ void tma_gather4(uint32_t dst, const CUtensorMap *map, uint32_t bar, int c0, int r0, int r1,
                                            int r2, int r3) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
        : "memory");
}

template <Kind KIND>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (KIND == K_I8) mma_i8(d, a, b, idesc, acc);
    else if (KIND == K_FP8) mma_f8f6f4(d, a, b, idesc, acc);
    else mma_f16(d, a, b, idesc, acc);
}

template <Kind KIND>
__host__ __device__ constexpr uint32_t idesc_rows(int rows) {
    return KIND == K_I8 ? make_idesc(2, 1, 1, BM, rows)
                        : make_idesc(1, KIND == K_W4B ? 1 : 0, KIND == K_W4B ? 1 : 0, BM, rows);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t d;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
    return d;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One word of 8 codes -> 8 weights s (q - z) in k order, each rounded once to the activations' type (the
// tensor cores take both operands in one type).  A byte's two nibbles become 1024 + q and 1024 + 16 q in
// one PRMT and one LOP3; an exact fma by (1, 1/16) with -(1024 + z), -(64 + z) leaves q - z.
template <bool BF>
__device__ __forceinline__ uint4 dequant_word(uint32_t w, uint32_t zc, uint32_t s2, float s) {
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t h = (prmt(w, 0u, 0x4040u + 0x0101u * i) & 0x00F0000Fu) | 0x64006400u;
        const uint32_t d = hfma2(h, 0x2C003C00u, zc);
        if (BF) {
            const float2 f = half2_bits_to_float2(d);
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(__fmul_rn(f.y, s)), "f"(__fmul_rn(f.x, s)));
        } else {
            o[i] = hmul2(d, s2);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// silu(g) u.  The fast exponential and division are off by a few fp32 units, far below the 16-bit
// rounding that follows.
__device__ __forceinline__ float swiglu(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

template <Kind KIND>
__device__ __forceinline__ uint16_t out_bits(float v) {
    return KIND == K_W4B ? float_to_bf16_bits_rn(v) : float_to_half_bits_rn(v);
}

// SWIGLU: a tile's 128 weight rows are, per 32 TMEM lanes, 16 gate rows and the 16 up rows that belong to
// them, so gate and up of one output meet by a shuffle inside a warp.
template <Kind KIND, bool GATHER, bool SWIGLU>
__global__ void __launch_bounds__(Layout<KIND>::THREADS, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tmap_x, const __grid_constant__ CUtensorMap tmap_w,
                        const Args a) {
    using L = Layout<KIND>;
    constexpr bool W4 = L::W4;
    constexpr int BN = SWIGLU ? BM / 2 : BM;           // output columns per tile
    constexpr int KE = W4 ? STAGE_K / 2 : STAGE_K;     // k values per stage
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars *bar = reinterpret_cast<Bars *>(base + L::OFF_BAR);
    int *src_tab = reinterpret_cast<int *>(base + L::OFF_SRC);
    float *sx_tab = reinterpret_cast<float *>(base + L::OFF_SX);
    int *off = reinterpret_cast<int *>(base + L::OFF_TAB), *tiles = off + a.E + 1;
    const uint32_t sA = smem_u32(base), sB = smem_u32(base + L::OFF_B), sP = smem_u32(base + L::OFF_P);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kst = (a.K + KE - 1) / KE;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&bar->full[s]), 1);
            mbar_init(smem_u32(&bar->dq_full[s]), DQ_WARPS);
            mbar_init(smem_u32(&bar->empty[s]), 1);
        }
        for (int p = 0; p < PSTAGES; ++p) {
            mbar_init(smem_u32(&bar->pk_full[p]), 1);
            mbar_init(smem_u32(&bar->pk_empty[p]), DQ_WARPS);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar->acc_full[i]), 1);
            mbar_init(smem_u32(&bar->acc_empty[i]), 4);
        }
        mbar_init(smem_u32(&bar->drain), 1);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&tmap_x);
        prefetch_tmap(&tmap_w);
    }
    if (warp == 1) build_table(a, off, tiles, lane);
    if (warp == 2) {
        tmem_alloc(smem_u32(&bar->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = bar->tmem_base;
    const WaitCtl ctl{&bar->abort, a.status, a.limit_ns};
    Tile w;

    // First weight row (of the stacked [E N] rows) of lane group i (16 lanes) of tile w.
    auto weight_row = [&](const Tile &t, int i) {
        return t.e * a.N + t.n0 + (SWIGLU ? (i & 1) * (a.N / 2) + (i >> 1) * 16 : i * 16);
    };

    if (warp == 0) {
        // -------------------------------------------------------------------- activations (8-bit: weights too)
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && get_tile<BN>(a, off, tiles, t, w); t += gridDim.x) {
            const int pad = (w.rows + 15) & ~15;
            // Rows this lane fetches: quads lane and lane + 32 of the tile.  Padding repeats the last
            // row; an index outside x is replaced by row 0 (the epilogue writes zeros for it).
            int idx[2][4];
            if (GATHER) {
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int r = min(4 * (lane + 32 * q) + j, w.rows - 1);
                        const int v = __ldg(a.rows + w.r0 + r);
                        idx[q][j] = (unsigned)v < (unsigned)a.T ? v : 0;
                    }
            }
            const int boxes = (pad + BOX_ROWS - 1) / BOX_ROWS;
            const uint32_t bytes = (GATHER ? pad : boxes * BOX_ROWS) * STAGE_K + (W4 ? 0 : A_BYTES);
            for (int kb = 0; kb < kst; ++kb, ++it) {
                const uint32_t s = it % STAGES, u = it / STAGES;
                const uint32_t fb = smem_u32(&bar->full[s]);
                if (lane == 0) {
                    ok = wait_parity(smem_u32(&bar->empty[s]), (u & 1) ^ 1, ctl, SITE_PRODUCER);
                    if (ok) {
                        mbar_arrive_expect_tx(fb, bytes);
                        if (!W4) {
                            if (SWIGLU) {
                                for (int i = 0; i < 8; ++i)
                                    tma_load_2d(sA + s * A_BYTES + i * 16 * STAGE_K, &tmap_w, fb, kb * KE,
                                                weight_row(w, i));
                            } else {
                                tma_load_2d(sA + s * A_BYTES, &tmap_w, fb, kb * KE, weight_row(w, 0));
                            }
                        }
                    }
                }
                ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
                if (!ok) break;
                const uint32_t dst = sB + s * B_BYTES;
                if (GATHER) {
#pragma unroll
                    for (int q = 0; q < 2; ++q)
                        if (4 * (lane + 32 * q) < pad)
                            tma_gather4(dst + 4 * (lane + 32 * q) * STAGE_K, &tmap_x, fb, kb * KE, idx[q][0], idx[q][1],
                                        idx[q][2], idx[q][3]);
                } else if (lane < boxes) {
                    tma_load_2d(dst + lane * BOX_ROWS * STAGE_K, &tmap_x, fb, kb * KE, w.r0 + lane * BOX_ROWS);
                }
                __syncwarp();
            }
        }
        // Every issued copy lands before the CTA leaves.
        if (lane == 0) {
            for (uint32_t s = 0; s < STAGES; ++s) {
                const uint32_t issued = it > s ? (it - s - 1) / STAGES + 1 : 0;
                if (issued) drain_parity(smem_u32(&bar->full[s]), (issued - 1) & 1, DRAIN_NS, a.status, SITE_DRAIN);
            }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            // ---------------------------------------------------------------- MMA issuer
            uint32_t it = 0, n = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && get_tile<BN>(a, off, tiles, t, w); t += gridDim.x, ++n) {
                const uint32_t acc = n & 1, u = n >> 1;
                if (!wait_parity(smem_u32(&bar->acc_empty[acc]), (u & 1) ^ 1, ctl, SITE_MMA)) break;
                tc_fence_after();
                const uint32_t d = tmem_base + acc * BR;
                const uint32_t idesc = idesc_rows<KIND>((w.rows + 15) & ~15);
                for (int kb = 0; kb < kst; ++kb, ++it) {
                    const uint32_t s = it % STAGES, us = it / STAGES;
                    if (!wait_parity(smem_u32(&bar->full[s]), us & 1, ctl, SITE_MMA) ||
                        (W4 && !wait_parity(smem_u32(&bar->dq_full[s]), us & 1, ctl, SITE_MMA))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < STAGE_K / 32; ++kk)
                        mma_step<KIND>(d, umma_desc_sw128_kmajor(sA + s * A_BYTES + kk * 32),
                                       umma_desc_sw128_kmajor(sB + s * B_BYTES + kk * 32), idesc, kb != 0 || kk != 0);
                    tc_commit(smem_u32(&bar->empty[s]));
                }
                if (ok) tc_commit(smem_u32(&bar->acc_full[acc]));
            }
            tc_commit(smem_u32(&bar->drain));
            drain_parity(smem_u32(&bar->drain), 0, DRAIN_NS, a.status, SITE_DRAIN);
        }
        __syncwarp();
    } else if (W4 && warp == 3) {
        if (lane == 0) {
            // ---------------------------------------------------------------- packed weight tiles
            uint32_t it = 0;
            bool ok = true;
            for (int t = blockIdx.x; ok && get_tile<BN>(a, off, tiles, t, w); t += gridDim.x) {
                for (int kb = 0; kb < kst; ++kb, ++it) {
                    const uint32_t p = it % PSTAGES, u = it / PSTAGES;
                    if (!wait_parity(smem_u32(&bar->pk_empty[p]), (u & 1) ^ 1, ctl, SITE_PACKED)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = smem_u32(&bar->pk_full[p]);
                    mbar_arrive_expect_tx(fb, P_BYTES);
                    if (SWIGLU) {
                        for (int i = 0; i < 8; ++i)
                            tma_load_2d(sP + p * P_BYTES + i * 16 * 32, &tmap_w, fb, kb * 32, weight_row(w, i));
                    } else {
                        tma_load_2d(sP + p * P_BYTES, &tmap_w, fb, kb * 32, weight_row(w, 0));
                    }
                }
            }
            for (uint32_t p = 0; p < PSTAGES; ++p) {
                const uint32_t issued = it > p ? (it - p - 1) / PSTAGES + 1 : 0;
                if (issued) drain_parity(smem_u32(&bar->pk_full[p]), (issued - 1) & 1, DRAIN_NS, a.status, SITE_DRAIN);
            }
        }
        __syncwarp();
    } else if (warp >= EPI_WARP0 && warp < EPI_WARP0 + 4) {
        // -------------------------------------------------------------------- epilogue
        const int q = warp & 3;                   // TMEM lanes 32 q .. 32 q + 31
        const int et = (int)threadIdx.x - 32 * EPI_WARP0;
        const uint32_t t_row = tmem_base + ((uint32_t)(32 * q) << 16);
        uint32_t n = 0;
        bool ok = true;
        for (int t = blockIdx.x; get_tile<BN>(a, off, tiles, t, w); t += gridDim.x, ++n) {
            const uint32_t acc = n & 1, u = n >> 1;
            int *src = src_tab + acc * BR;
            float *sxs = sx_tab + acc * BR;
            for (int r = et; r < w.rows; r += 128) {
                int v = w.r0 + r;
                if (GATHER) {
                    v = __ldg(a.rows + v);
                    if ((unsigned)v >= (unsigned)a.T) v = -1;
                }
                src[r] = v;
                if (!W4) sxs[r] = v >= 0 ? __ldg(a.sx + (size_t)v * a.sx_stride) : 0.0f;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            const int col = w.n0 + (SWIGLU ? 16 * q + (lane & 15) : 32 * q + lane);
            const bool col_ok = col < a.ldy;
            float sw = 1.0f;
            if (!W4)
                sw = a.sw_per_row ? __ldg(a.sw + min((size_t)a.E * a.N - 1,
                                                     (size_t)weight_row(w, 2 * q + (lane >> 4)) + (lane & 15)))
                                  : __ldg(a.sw + w.e);
            // After a wait has run out the warps still walk the tiles, so that all four meet at the barrier.
            ok = ok && wait_parity(smem_u32(&bar->acc_full[acc]), u & 1, ctl, SITE_EPILOGUE);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) continue;
            tc_fence_after();
            uint16_t *yt = a.y + (size_t)w.r0 * a.ldy;
            for (int c = 0; c < w.rows; c += 16) {
                uint32_t r[16];
                tmem_ld_32x32b_x16(t_row + acc * BR + c, r);
                tmem_ld_wait();
                float v[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float f = KIND == K_I8 ? (float)(int32_t)r[j] : __uint_as_float(r[j]);
                    v[j] = W4 ? f : __fmul_rn(__fmul_rn(f, sxs[min(c + j, w.rows - 1)]), sw);
                }
                if (SWIGLU) {
                    const bool up = lane >= 16;   // this lane's weight row is an up row
#pragma unroll
                    for (int j = 0; j < 16; j += 2) {
                        const float other = __shfl_xor_sync(0xffffffffu, up ? v[j] : v[j + 1], 16);
                        const float g = up ? other : v[j], l = up ? v[j + 1] : other;
                        const int row = c + j + (up ? 1 : 0);
                        if (row < w.rows && col_ok)
                            yt[(size_t)row * a.ldy + col] = src[row] >= 0 ? out_bits<KIND>(swiglu(g, l)) : (uint16_t)0;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < w.rows && col_ok)
                            yt[(size_t)(c + j) * a.ldy + col] = src[c + j] >= 0 ? out_bits<KIND>(v[j]) : (uint16_t)0;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar->acc_empty[acc]));
        }
    } else if (W4 && warp >= DQ_WARP0) {
        // -------------------------------------------------------------------- dequantizers
        // Thread (row of the tile, half of the stage's 64 codes).
        const int row = 32 * (warp & 3) + lane, half = (warp - DQ_WARP0) >> 2;
        const int groups = a.K / a.gs, zwords = (groups + 7) / 8;
        uint32_t it = 0;
        bool ok = true;
        for (int t = blockIdx.x; ok && get_tile<BN>(a, off, tiles, t, w); t += gridDim.x) {
            const size_t wr = min((size_t)weight_row(w, row >> 4) + (row & 15), (size_t)a.E * a.N - 1);
            const uint16_t *srow = a.scales + wr * groups;
            const uint32_t *zrow = a.qzeros + wr * zwords;
            // A thread's 32 codes of a stage lie in one group; its scale and zero are fetched a stage ahead.
            auto fetch = [&](int kb, uint32_t &sh, uint32_t &z) {
                const int g = min((kb * KE + half * 32) / a.gs, groups - 1);
                sh = __ldg(srow + g);
                z = (__ldg(zrow + (g >> 3)) >> (4 * (g & 7))) & 0xFu;
            };
            uint32_t sh, z;
            fetch(0, sh, z);
            for (int kb = 0; kb < kst; ++kb, ++it) {
                uint32_t shn = sh, zn = z;
                if (kb + 1 < kst) fetch(kb + 1, shn, zn);
                const uint32_t p = it % PSTAGES, up = it / PSTAGES, s = it % STAGES, us = it / STAGES;
                ok = wait_parity(smem_u32(&bar->pk_full[p]), up & 1, ctl, SITE_DEQUANT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                // 32-byte swizzle: half h of row r lies at h ^ ((r / 4) mod 2).
                const uint4 q = lds128(sP + p * P_BYTES + row * 32 + ((half ^ ((row >> 2) & 1)) << 4));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar->pk_empty[p]));
                ok = wait_parity(smem_u32(&bar->empty[s]), (us & 1) ^ 1, ctl, SITE_DEQUANT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                const uint32_t s2 = sh | (sh << 16), zc = 0xD400E400u + z * 0x00100001u;
                const float sf = half_bits_to_float((uint16_t)sh);
                const uint32_t ws[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts128(sA + s * A_BYTES + row * STAGE_K + (((4 * half + j) ^ (row & 7)) << 4),
                           dequant_word<KIND == K_W4B>(ws[j], zc, s2, sf));
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar->dq_full[s]));
                sh = shn;
                z = zn;
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem_base, 512);
    }
}

template <Kind KIND, bool GATHER, bool SWIGLU>
wq_status launch(const CUtensorMap &tx, const CUtensorMap &tw, const Args &a, int grid, cudaStream_t st,
                 const char *who) {
    auto kern = grouped_gemm_kernel<KIND, GATHER, SWIGLU>;
    const size_t smem = Layout<KIND>::smem(a.E);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(WQ_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
    kern<<<grid, Layout<KIND>::THREADS, smem, st>>>(tx, tw, a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail(WQ_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return WQ_OK;
}

// x: [T] rows of K values; w: [E N] rows (of K bytes, or K / 2 packed).
template <Kind KIND>
wq_status dispatch(const void *x, const void *w, Args a, bool swiglu, cudaStream_t st, const char *who) {
    constexpr bool W4 = is_w4(KIND);
    a.status = device_status_word();
    if (!a.status) return WQ_ERR_CUDA;
    a.limit_ns = wait_limit();
    a.ldy = swiglu ? a.N / 2 : a.N;
    const int bn = swiglu ? BM / 2 : BM;
    a.nb = (a.ldy + bn - 1) / bn;
    const long long most = ((long long)std::min(a.E, a.R) + a.R / BR) * a.nb;  // tiles of any offsets
    WQ_REQUIRE(most < INT_MAX / 2, WQ_ERR_UNSUPPORTED, "%s: R (%d) x N (%d) gives too many tiles", who, a.R, a.N);
    const bool gather = a.rows != nullptr;
    CUtensorMap tx, tw;
    const CUtensorMapDataType xt = KIND == K_W4H ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : KIND == K_W4B ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const int xb = W4 ? 2 : 1;
    if (!encode_tmap_2d(&tx, xt, xb, x, (uint64_t)a.K, (uint64_t)a.T, (uint64_t)a.K * xb, STAGE_K / xb,
                        gather ? 1 : BOX_ROWS, CU_TENSOR_MAP_SWIZZLE_128B))
        return WQ_ERR_CUDA;
    const uint64_t wbytes = W4 ? (uint64_t)a.K / 2 : (uint64_t)a.K;
    if (!encode_tmap_2d(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, wbytes, (uint64_t)a.E * a.N, wbytes,
                        W4 ? 32 : STAGE_K, swiglu ? 16 : BM,
                        W4 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_128B))
        return WQ_ERR_CUDA;
    const int grid = (int)std::min<long long>(num_sms(), most);
    if (gather)
        return swiglu ? launch<KIND, true, true>(tx, tw, a, grid, st, who)
                      : launch<KIND, true, false>(tx, tw, a, grid, st, who);
    return swiglu ? launch<KIND, false, true>(tx, tw, a, grid, st, who)
                  : launch<KIND, false, false>(tx, tw, a, grid, st, who);
}

// Checks that every grouped product makes of its sizes.
wq_status check_sizes(const char *who, int T, const int32_t *rows, const int32_t *offsets, int R, int E, int N, int K,
                      int swiglu) {
    WQ_REQUIRE_PTR(offsets, "offsets");
    WQ_REQUIRE(aligned16(rows), WQ_ERR_ALIGNMENT, "rows is not 16-byte aligned");
    WQ_REQUIRE(T > 0 && R > 0 && E > 0 && N > 0 && K > 0, WQ_ERR_INVALID_ARG,
               "%s: sizes must be positive (T=%d R=%d E=%d N=%d K=%d)", who, T, R, E, N, K);
    WQ_REQUIRE(E <= MAX_E, WQ_ERR_UNSUPPORTED, "%s: E (%d) must be at most %d", who, E, MAX_E);
    WQ_REQUIRE(rows || R == T, WQ_ERR_INVALID_ARG, "%s: without rows, R (%d) must equal T (%d)", who, R, T);
    WQ_REQUIRE(!swiglu || N % 2 == 0, WQ_ERR_INVALID_ARG, "%s: N (%d) must be even with SwiGLU", who, N);
    WQ_REQUIRE((long long)E * N <= INT_MAX - 4 * BM, WQ_ERR_UNSUPPORTED, "%s: E * N must be below 2^31", who);
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
    return dispatch<KIND>(x, qweight, a, swiglu != 0, as_stream(stream), who);
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
    return dispatch<KIND>(xq, wq_, a, swiglu != 0, as_stream(stream), who);
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
