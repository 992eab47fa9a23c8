// Expert products with INT4 weights for few rows per expert (decode batches, 7 to 22): the same products as
// grouped_gemm.cu's kernel, whose tiles these are, organised around the stream of packed weights.
//
//   y[p][n] = sum_j s[n][j] * ( sum_{k in group j} (q[n][k] - z[n][j]) x[rows[p]][k] )
//
// With up to 16 activation rows a weight takes part in so few products that turning it into an fp16 value
// s (q - z) would cost more than the tensor cores' work on it.  So the MMA's operand is q - z itself, an
// integer of 5 bits that fp16 and bf16 hold exactly, every group of codes has an accumulator of its own in
// tensor memory, and the group's scale multiplies the 128 x 16 sums in fp32 when the group is done: no
// weight is rounded, and a scale costs one fma per row of x instead of one product per code.
//
// Persistent CTA, one per SM; a tile is 128 weight rows times up to 16 rows of one expert, and the S CTAs
// of a cluster share a tile's depth, so that the last round of tiles is short:
//   warp 0       TMA: 128 rows x 128 bytes (a pack of 256 codes) of packed weights into a deep ring
//   warps 1, 2   an elected thread each issues tcgen05.mma for every other pack (A from tensor memory): a
//                wait takes a thread about 100 cycles even when it is over, an MMA 45 and a commit 50, so
//                one thread alone cannot issue 16 MMAs of 16 codes in the 710 cycles that a pack's bytes take
//   warp 3       allocates tensor memory
//   warps 4-7    scale: each pack's accumulators, times the scales of the lane's weight row, into registers;
//                at the end of a tile the cluster's parts meet in the first CTA's shared memory, which
//                applies SwiGLU, rounds and stores
//   warps 8-15   two groups of four warps, every other pack each: rows of x into shared memory, and codes ->
//                q - z into tensor memory.  A thread takes 256 codes at a time: with 128 (and twice the warps)
//                its waits, loads and addresses were 250 of 390 instructions
//
// Measured on B200: 8 experts of 28672 x 4096 for 64 rows, fp16, 492 MB, 149 us (3.3 TB/s, floor 76 us); 64 experts of
// 4096 x 2048 for 768 bf16 rows, groups of 64, 297 MB, 110 us where each has 12 rows and 120 us at random counts, of
// which those above 16 rows are another tile (2.7 and 2.5 TB/s, floor 46 us).  With the whole dequantization, the fmas,
// all but one MMA per stage and the loads of x and scales taken out, 440 MB of weights take 94 us against 148: no
// unit bounds it alone, the loop of a dequantizing group (two thirds of its 1290 cycles per pack are arithmetic
// at about 5 cycles an instruction) and the rest of the pipeline lie close together.
#include "grouped.cuh"

#include <algorithm>
#include <climits>

namespace wq {
namespace grouped {
namespace {

using namespace sm100;

constexpr int BR = 16;                      // rows of a tile, at most (the MMA's N)
constexpr int SK = 128;                     // codes per stage
constexpr int STAGES = 4, P_SLOTS = 8, MAX_ACCS = 8;
constexpr uint32_t X_ATOM = BR * 128, X_BYTES = 2 * X_ATOM;   // 64 values a row and atom
constexpr uint32_t P_BYTES = BM * 128;      // a pack: 256 codes of 128 rows, two stages
constexpr uint32_t A_COLS = SK / 2;         // tensor memory columns of a stage
constexpr int THREADS = 512, DQ_WARP0 = 8;
constexpr int MAX_SPLIT = 4;
constexpr uint32_t OFF_X = P_SLOTS * P_BYTES;
constexpr uint32_t OFF_RED = OFF_X + STAGES * X_BYTES;    // not used when the tile is not split
constexpr uint32_t RED_BYTES = BM * BR * 4;                   // one CTA's part of a tile
constexpr unsigned SITE_PACKED = 0x2001, SITE_MMA = 0x2002, SITE_SCALE = 0x2008, SITE_DEQUANT = 0x2010,
                   SITE_DRAIN = 0x2020, SITE_SPLIT = 0x2040;

// Tensor memory: four stages of 64 columns, then accumulators, 16 columns per group and 256 / gs groups per pack.
// Pack, stage and accumulator slots belong to one dequantizing group and one issuer each (an even number of
// packs, 4 stages, an even number of accumulators): a thread that waited for a slot that another one had not
// used yet could take an older phase of its barrier, of the same parity, for the one it waits for.
static_assert(STAGES * A_COLS + 256 * BR / 16 <= 512, "tensor memory");

struct Bars {
    uint64_t pk_full[P_SLOTS], pk_empty[P_SLOTS];
    uint64_t full[STAGES], empty[STAGES];       // rows of x and q - z of a stage
    uint64_t acc_full[MAX_ACCS], acc_empty[MAX_ACCS];   // accumulators of a pack
    uint64_t red_full[4], red_free[4];      // per scale warp: the other CTAs' parts are here / may be sent
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
};

constexpr size_t smem_bytes(int split, int E) {
    return 1024 + OFF_RED + (size_t)(split - 1) * RED_BYTES + 1024 + 2 * (size_t)(E + 1) * 4;
}

static_assert(smem_bytes(MAX_SPLIT, MAX_E) <= 232448 && sizeof(Bars) <= 1024, "shared memory");

// The part of a tile's depth that CTA `rank` of `split` takes: stages [s0, s1), in whole packed tiles.
struct Depth {
    int s0, s1;
    __device__ __forceinline__ Depth(int K, int rank, int split) {
        const int st = (K + SK - 1) / SK, packs = (st + 1) / 2;
        s0 = 2 * (int)((long long)packs * rank / split);
        s1 = min(st, 2 * (int)((long long)packs * (rank + 1) / split));
    }
};

template <bool BF, bool SWIGLU>
__global__ void __launch_bounds__(THREADS, 1)
    few_rows_kernel(const __grid_constant__ CUtensorMap tmap_w, const Args a, int split) {
    constexpr int BN = SWIGLU ? BM / 2 : BM;   // output columns per tile
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t off_bar = OFF_RED + (split - 1) * RED_BYTES;
    Bars *bar = reinterpret_cast<Bars *>(base + off_bar);
    int *off = reinterpret_cast<int *>(base + off_bar + 1024), *tiles = off + a.E + 1;
    const uint32_t sP = smem_u32(base), sX = smem_u32(base + OFF_X), sR = smem_u32(base + OFF_RED);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = split > 1 ? (int)cluster_ctarank() : 0;
    const int first = (int)blockIdx.x / split, stride = (int)gridDim.x / split;
    const Depth dep(a.K, rank, split);
    const int nst = dep.s1 - dep.s0, packs = (nst + 1) / 2;   // of a tile, in this CTA
    const int accs = min(a.gs / 16, MAX_ACCS), acc_cols = 256 / a.gs * BR;
    const int lg = 31 - __clz(a.gs), groups = a.K >> lg, zwords = (groups + 7) / 8;

    if (threadIdx.x == 0) {
        for (int i = 0; i < P_SLOTS; ++i) {
            mbar_init(smem_u32(&bar->pk_full[i]), 1);
            mbar_init(smem_u32(&bar->pk_empty[i]), 4);
        }
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(smem_u32(&bar->full[i]), 4);
            mbar_init(smem_u32(&bar->empty[i]), 1);
        }
        for (int i = 0; i < MAX_ACCS; ++i) {
            mbar_init(smem_u32(&bar->acc_full[i]), 1);
            mbar_init(smem_u32(&bar->acc_empty[i]), 4);
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(smem_u32(&bar->red_full[i]), max(1, split - 1));
            mbar_init(smem_u32(&bar->red_free[i]), 1);
        }
        mbar_init(smem_u32(&bar->drain[0]), 1);
        mbar_init(smem_u32(&bar->drain[1]), 1);
        bar->abort = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) prefetch_tmap(&tmap_w);
    if (warp == 1) build_table<BR>(a, off, tiles, lane);
    if (warp == 3) {
        tmem_alloc(smem_u32(&bar->tmem_base), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();  // every CTA's barriers are set up before another arrives on them
    tc_fence_after();
    const uint32_t tmem = bar->tmem_base;
    const WaitCtl ctl{&bar->abort, a.status, a.limit_ns};
    Tile w;

    // First weight row (of the stacked [E N] rows) of lane group i (16 lanes) of tile t.
    auto weight_row = [&](const Tile &t, int i) {
        return t.e * a.N + t.n0 + (SWIGLU ? (i & 1) * (a.N / 2) + (i >> 1) * 16 : i * 16);
    };

    if (warp == 0) {
        // -------------------------------------------------------------------- packed weights
        const bool leader = elect_one();
        uint32_t p = 0, ph = 1, it = 0;
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, BR>(a, off, tiles, t, w); t += stride) {
            for (int sb = dep.s0; sb < dep.s1; sb += 2, ++it) {
                ok = wait_parity_lean(smem_u32(&bar->pk_empty[p]), ph, ctl, SITE_PACKED);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                if (leader) {
                    const uint32_t fb = smem_u32(&bar->pk_full[p]), dst = sP + p * P_BYTES;
                    mbar_arrive_expect_tx(fb, P_BYTES);
                    if (!SWIGLU) {
                        tma_load_2d(dst, &tmap_w, fb, sb * 64, weight_row(w, 0));
                    } else if (a.box) {
                        tma_load_5d(dst, &tmap_w, fb, sb * 64, 0, 0, w.n0 >> 4, w.e);
                    } else {
                        for (int i = 0; i < 8; ++i)
                            tma_load_2d(dst + i * 16 * 128, &tmap_w, fb, sb * 64, weight_row(w, i));
                    }
                }
                __syncwarp();
                if (++p == P_SLOTS) {
                    p = 0;
                    ph ^= 1;
                }
            }
        }
        for (uint32_t i = 0; i < P_SLOTS; ++i) {  // every issued copy lands before the CTA leaves
            const uint32_t issued = it > i ? (it - i - 1) / P_SLOTS + 1 : 0;
            if (issued) drain_parity(smem_u32(&bar->pk_full[i]), (issued - 1) & 1, DRAIN_NS, a.status, SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp <= 2) {
        // -------------------------------------------------------------------- MMA issuers
        const bool leader = elect_one();
        const int me = warp - 1;
        const uint64_t desc_x = umma_desc_sw128_kmajor(sX);
        constexpr uint32_t IDESC = make_idesc(1, BF ? 1 : 0, BF ? 1 : 0, BM, BR);
        const int gmask = a.gs / 16 - 1;             // MMAs (16 codes) per group, less one
        uint32_t pk = 0;                             // packs before this tile
        bool ok = true;
        for (int t = first; ok && get_tile<BN, BR, BR>(a, off, tiles, t, w); t += stride, pk += packs) {
            for (int b = (int)((me - pk) & 1); b < packs; b += 2) {
                const uint32_t c = (pk + b) % accs, cu = (pk + b) / accs;
                const uint32_t acc = tmem + STAGES * A_COLS + c * acc_cols;
                const uint32_t ae = smem_u32(&bar->acc_empty[c]);
                for (int h = 0; h < 2; ++h) {   // the second stage of the last pack may be empty
                    const uint32_t it = 2 * (pk + b) + h, s = it % STAGES, u = it / STAGES;
                    const uint32_t fb = smem_u32(&bar->full[s]);
                    ok = h == 0 ? wait_parity2(ae, (cu & 1) ^ 1, fb, u & 1, ctl, SITE_MMA)
                                : wait_parity_lean(fb, u & 1, ctl, SITE_MMA);
                    if (!(ok = __all_sync(0xffffffffu, ok))) break;
                    tc_fence_after();
                    if (leader) {
                        const uint32_t a_tm = tmem + s * A_COLS;
                        const uint64_t db = desc_x + s * (X_BYTES >> 4);
                        const int steps = (a.K - (dep.s0 + 2 * b + h) * SK) / 16;
#pragma unroll
                        for (int k = 0; k < SK / 16; ++k)
                            if (k < steps)
                                mma_f16_tmem_a(acc + (((8 * h + k) * 16) >> lg) * BR, a_tm + k * 8,
                                               db + (k >> 2) * (X_ATOM >> 4) + (k & 3) * 2, IDESC,
                                               ((8 * h + k) & gmask) != 0);
                        tc_commit(smem_u32(&bar->empty[s]));
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (leader) tc_commit(smem_u32(&bar->acc_full[c]));
                __syncwarp();
            }
        }
        if (leader) {
            tc_commit(smem_u32(&bar->drain[me]));
            drain_parity(smem_u32(&bar->drain[me]), 0, DRAIN_NS, a.status, SITE_DRAIN);
        }
        __syncwarp();
    } else if (warp >= 4 && warp < DQ_WARP0) {
        // -------------------------------------------------------------------- scales, end of the tile
        const int q = warp & 3, trow = 32 * q + lane;   // TMEM lanes 32 q ..; this lane's row of the tile
        const uint32_t t_row = tmem + ((uint32_t)(32 * q) << 16);
        const int g_first = (dep.s0 * SK) >> lg, g_last = min(groups, (dep.s1 * SK + a.gs - 1) >> lg);
        const int gpp = max(1, 256 >> lg);       // groups per pack
        const bool whole = a.K % 256 == 0;       // every pack is full, and its scales are aligned to their size
        const uint16_t *srow = nullptr;
        uint4 ns = {};                           // scales of the next pack
        auto rows_of = [&](const Tile &t) {
            const size_t wr = min((size_t)weight_row(t, trow >> 4) + (trow & 15), (size_t)a.E * a.N - 1);
            srow = a.scales + wr * groups;
        };
        auto load = [&](int g) {
            const uint16_t *p = srow + g;
            if (!whole) {
                uint32_t v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = i < gpp ? __ldg(srow + min(g + i, groups - 1)) : 0u;
                ns = make_uint4(v[0] | (v[1] << 16), v[2] | (v[3] << 16), v[4] | (v[5] << 16), v[6] | (v[7] << 16));
            } else if (gpp == 1) {
                ns.x = __ldg(p);
            } else if (gpp == 2) {
                ns.x = __ldg(reinterpret_cast<const uint32_t *>(p));
            } else if (gpp == 4) {
                const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
                ns.x = v.x;
                ns.y = v.y;
            } else {
                ns = __ldg(reinterpret_cast<const uint4 *>(p));
            }
        };
        uint32_t pk = 0, n = 0;
        bool have = get_tile<BN, BR, BR>(a, off, tiles, first, w), ok = true;
        if (have) {
            rows_of(w);
            load(g_first);
        }
        for (int t = first; ok && have; t += stride, ++n) {
            const Tile cur = w;
            // Rows of the tile whose index lies outside x.
            bool out = false;
            if (a.rows && lane < cur.rows) out = (unsigned)__ldg(a.rows + cur.r0 + lane) >= (unsigned)a.T;
            const uint32_t zero_rows = __ballot_sync(0xffffffffu, out);
            float acc[BR];
#pragma unroll
            for (int i = 0; i < BR; ++i) acc[i] = 0.0f;
            int g = g_first;
            for (int b = 0; b < packs; ++b, ++pk) {
                const uint32_t c = pk % accs, cols = t_row + STAGES * A_COLS + c * acc_cols;
                const uint4 sc = ns;
                const int here = min(gpp, g_last - g);
                g += gpp;
                if (b + 1 < packs) {
                    load(g);
                } else {
                    have = get_tile<BN, BR, BR>(a, off, tiles, t + stride, w);
                    if (have) {
                        rows_of(w);
                        load(g_first);
                    }
                }
                ok = wait_parity_lean(smem_u32(&bar->acc_full[c]), (pk / accs) & 1, ctl, SITE_SCALE);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const uint32_t sp[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {   // two groups at a time; columns past `here` groups are not used
                    if (2 * i >= here) break;
                    const float2 s2 = half2_bits_to_float2(sp[i]);
                    uint32_t r[32];
                    if (gpp > 1) {
                        tmem_ld_32x32b_x32(cols + 2 * i * BR, r);
                    } else {
                        uint32_t r1[16];
                        tmem_ld_32x32b_x16(cols, r1);
#pragma unroll
                        for (int j = 0; j < 16; ++j) r[j] = r1[j];
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < BR; ++j) acc[j] = fmaf(s2.x, __uint_as_float(r[j]), acc[j]);
                    if (2 * i + 1 < here) {
#pragma unroll
                        for (int j = 0; j < BR; ++j) acc[j] = fmaf(s2.y, __uint_as_float(r[16 + j]), acc[j]);
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar->acc_empty[c]));
            }
            if (!ok) break;
            if (split > 1) {
                // Parts are added in rank order.  A lane's values lie 512 bytes apart, so that a warp's stores
                // and loads are contiguous.
                if (rank != 0) {
                    if (n > 0) {
                        ok = wait_parity_lean<true>(smem_u32(&bar->red_free[q]), (n - 1) & 1, ctl, SITE_SPLIT);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        fence_cluster();
                    }
                    const uint32_t dst = mapa_shared(sR + (rank - 1) * RED_BYTES + trow * 4, 0);
#pragma unroll
                    for (int j = 0; j < BR; ++j)
                        st_cluster_f32(dst + j * BM * 4, acc[j]);
                    __syncwarp();
                    if (lane == 0) {   // releases the whole warp's stores
                        fence_cluster();
                        mbar_arrive_cluster(mapa_shared(smem_u32(&bar->red_full[q]), 0));
                    }
                    continue;
                }
                ok = wait_parity_lean<true>(smem_u32(&bar->red_full[q]), n & 1, ctl, SITE_SPLIT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                fence_cluster();
                for (int c = 0; c < split - 1; ++c) {
                    const float *part = reinterpret_cast<const float *>(base + OFF_RED + c * RED_BYTES) + trow;
#pragma unroll
                    for (int j = 0; j < BR; ++j)
                        acc[j] += part[j * BM];
                }
                __syncwarp();
                if (lane > 0 && lane < split) {
                    fence_cluster();
                    mbar_arrive_cluster(mapa_shared(smem_u32(&bar->red_free[q]), lane));
                }
            }
            const int col = cur.n0 + (SWIGLU ? 16 * q + (lane & 15) : 32 * q + lane);
            const bool col_ok = col < a.ldy;
            uint16_t *yt = a.y + (size_t)cur.r0 * a.ldy + col;
            const bool full = cur.rows == BR && __all_sync(0xffffffffu, col_ok);
            if (SWIGLU) {
                const bool up = lane >= 16;   // this lane's weight row is an up row
                float o[BR / 2];
#pragma unroll
                for (int j = 0; j < BR; j += 2) {
                    const float other = __shfl_xor_sync(0xffffffffu, up ? acc[j] : acc[j + 1], 16);
                    o[j / 2] = swiglu(up ? other : acc[j], up ? acc[j + 1] : other);
                }
                if (zero_rows)
#pragma unroll
                    for (int j = 0; j < BR / 2; ++j)
                        if ((zero_rows >> (2 * j + (up ? 1 : 0))) & 1) o[j] = 0.0f;
                store_column<BF>(yt + (up ? a.ldy : 0), 2 * (size_t)a.ldy, o,
                                 col_ok ? (cur.rows + (up ? 0 : 1)) / 2 : 0, full);
            } else {
                if (zero_rows)
#pragma unroll
                    for (int j = 0; j < BR; ++j)
                        if ((zero_rows >> j) & 1) acc[j] = 0.0f;
                store_column<BF>(yt, (size_t)a.ldy, acc, col_ok ? cur.rows : 0, full);
            }
        }
    } else if (warp >= DQ_WARP0) {
        // -------------------------------------------------------------------- codes -> q - z
        // Group d takes every other pack and fills stages 2 d and 2 d + 1; a thread takes one weight row.
        const int q = warp & 3, trow = 32 * q + lane, d = (warp - DQ_WARP0) >> 2;
        const uint32_t t_a = tmem + ((uint32_t)(32 * q) << 16) + 2 * d * A_COLS, r7 = (uint32_t)(trow & 7) << 4;
        const uint32_t magic = opaque_const(BF ? 0x43004300u : 0x64006400u);
        const uint32_t fb = smem_u32(&bar->full[2 * d]), eb = smem_u32(&bar->empty[2 * d]);
        // Rows of x: warp q brings rows q, q + 4, q + 8, q + 12 of the tile, a lane 16 of the pack's 512 bytes.
        const size_t pitch = (size_t)a.K * 2;
        const uint32_t xd = sX + (2 * d + (lane >> 4)) * X_BYTES + ((lane >> 3) & 1) * X_ATOM;
        const uint8_t *xp[4] = {};
        const uint32_t *zrow = nullptr;
        uint4 nx[4] = {};                   // x and zeros of this thread's next pack
        uint32_t nz = 0;
        int rows = 0;                       // of the tile that they belong to
        auto load = [&](int b) {            // pack b of the tile whose pointers are set
            const int k0 = (dep.s0 + 2 * b) * SK;
            nz = __ldg(zrow + (min(k0 >> lg, groups - 1) >> 3));
            const size_t at = (size_t)k0 * 2 + lane * 16;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (q + 4 * i < rows)
                    nx[i] = at < pitch ? __ldg(reinterpret_cast<const uint4 *>(xp[i] + at)) : make_uint4(0, 0, 0, 0);
        };
        uint32_t pk0 = 0;                   // packs before this tile
        uint32_t p = d, pp = 0, ep = 1;     // slot and parities of this group's next pack
        bool ok = true, have = true;
        auto tile_from = [&](int t, int b) {   // sets up tile t and requests its pack b
            have = get_tile<BN, BR, BR>(a, off, tiles, t, w);
            if (!have) return;
            const size_t wr = min((size_t)weight_row(w, trow >> 4) + (trow & 15), (size_t)a.E * a.N - 1);
            zrow = a.qzeros + wr * zwords;
            rows = w.rows;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (q + 4 * i >= rows) continue;
                int v = w.r0 + q + 4 * i;
                if (a.rows) v = __ldg(a.rows + v);
                // An index outside x reads row 0 (zeros are stored for it).
                xp[i] = a.x + ((unsigned)v < (unsigned)a.T ? (size_t)v : 0) * pitch;
            }
            if (b < packs) load(b);
        };
        tile_from(first, d);
        for (int t = first; ok && have; t += stride, pk0 += packs) {
            const int b0 = (int)((d - pk0) & 1);
            if (b0 >= packs) {              // a tile of one pack, of the other group
                tile_from(t + stride, (int)((d - pk0 - packs) & 1));
                continue;
            }
            for (int b = b0; b < packs; b += 2) {
                const int here = rows;
                const uint32_t cz = nz;
                ok = wait_parity2(smem_u32(&bar->pk_full[p]), pp, eb, ep, ctl, SITE_DEQUANT);
                if (!(ok = __all_sync(0xffffffffu, ok))) break;
                tc_fence_after();
                const uint32_t src = sP + p * P_BYTES + trow * 128;
                const int k0 = (dep.s0 + 2 * b) * SK;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const bool real = 2 * b + h < nst;   // the second stage of a tile's last pack may be empty
                    if (real) {
                        // 128-byte swizzle: chunk c of row r lies at c ^ (r mod 8).
                        uint4 v[4];
#pragma unroll
                        for (int c = 0; c < 4; ++c) v[c] = lds128(src + (((4 * h + c) << 4) ^ r7));
                        Zero<BF> z((cz >> (4 * (((k0 + h * SK) >> lg) & 7))) & 0xFu);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {    // 32 codes, all in one group
                            if (c > 0 && a.gs < SK) z = Zero<BF>((cz >> (4 * (((k0 + h * SK + 32 * c) >> lg) & 7))) & 0xFu);
                            uint32_t o[16];
                            code_word<BF>(v[c].x, magic, z, o);
                            code_word<BF>(v[c].y, magic, z, o + 4);
                            code_word<BF>(v[c].z, magic, z, o + 8);
                            code_word<BF>(v[c].w, magic, z, o + 12);
                            tmem_st_32x32b_x16(t_a + h * A_COLS + c * 16, o);
                        }
                    }
                    if (h == 0) {
                        ok = wait_parity_lean(eb + 8, ep, ctl, SITE_DEQUANT);
                        if (!(ok = __all_sync(0xffffffffu, ok))) break;
                        tc_fence_after();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = q + 4 * i;
                            if (r < here) sts128(xd + r * 128 + (((lane ^ r) & 7) << 4), permute_x(nx[i]));
                        }
                        fence_proxy_async_smem();
                        if (b + 2 < packs) load(b + 2);
                        else tile_from(t + stride, (int)((d - pk0 - packs) & 1));
                    }
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) {
                        if (h == 1) mbar_arrive(smem_u32(&bar->pk_empty[p]));
                        mbar_arrive(fb + 8 * h);
                    }
                }
                if (!ok) break;
                p += 2;
                if (p >= P_SLOTS) {
                    p -= P_SLOTS;
                    pp ^= 1;
                }
                ep ^= 1;
            }
        }
        tmem_st_wait();   // after a wait that ran out, stores of half a pack may still be in flight
    }

    tc_fence_before();
    __syncthreads();
    if (split > 1) cluster_sync();  // nothing of another CTA's still arrives here
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// CTAs of a cluster that share a tile's depth: the number (1, 2 or 4) with the shortest schedule, where a
// round of tiles lasts its depth and, for the parts' exchange, as long as two packs (64 experts, N = 4096,
// K = 2048: 103 us unsplit, 144 us on pairs; 2 x 4096 x 14336: 31 us on pairs, 33 us on fours).
int choose_split(long long tiles, int K, const int (&clusters)[3]) {
    const int packs = ((K + SK - 1) / SK + 1) / 2;
    int best = 1;
    double best_t = 1e300;
    for (int i = 0; i < 3; ++i) {
        const int s = 1 << i;
        if (s > 1 && packs < 2 * s) break;
        const long long rounds = (tiles + clusters[i] - 1) / clusters[i];
        const double t = (double)rounds * ((double)packs / s + (s > 1 ? 2.0 : 0.0));
        if (t < 0.98 * best_t) {
            best_t = t;
            best = s;
        }
    }
    return best;
}

template <bool BF, bool SWIGLU>
wq_status launch(const CUtensorMap &tw, const Args &a, long long tiles, cudaStream_t st, const char *who) {
    auto kern = few_rows_kernel<BF, SWIGLU>;
    static std::atomic<uint64_t> allowed{0};
    const wq_status ok = allow_smem(kern, smem_bytes(MAX_SPLIT, MAX_E), allowed, who);
    if (ok != WQ_OK) return ok;
    // Looked up once: every device of the library's kind answers the same.
    static const int clusters[3] = {num_sms(), resident_clusters(kern, THREADS, smem_bytes(2, MAX_E), 2),
                                    resident_clusters(kern, THREADS, smem_bytes(4, MAX_E), 4)};
    const int split = choose_split(tiles, a.K, clusters);
    const size_t smem = smem_bytes(split, a.E);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)std::min<long long>(clusters[split / 2], tiles) * split);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = split;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tw, a, split);
    if (e != cudaSuccess) return fail(WQ_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
    return WQ_OK;
}

}  // namespace

wq_status few_rows_w4(const void *w, Args a, bool bf16, bool swiglu, cudaStream_t st, const char *who) {
    a.ldy = swiglu ? a.N / 2 : a.N;
    const int bn = swiglu ? BM / 2 : BM;
    a.nb = (a.ldy + bn - 1) / bn;
    const long long most = ((long long)std::min(a.E, a.R) + a.R / BR) * a.nb;  // tiles of any offsets
    WQ_REQUIRE(most < INT_MAX / 2, WQ_ERR_UNSUPPORTED, "%s: R (%d) x N (%d) gives too many tiles", who, a.R, a.N);
    CUtensorMap tw;
    if (!encode_weights(&tw, w, (uint64_t)a.K / 2, 128, a, swiglu)) return WQ_ERR_CUDA;
    if (bf16) return swiglu ? launch<true, true>(tw, a, most, st, who) : launch<true, false>(tw, a, most, st, who);
    return swiglu ? launch<false, true>(tw, a, most, st, who) : launch<false, false>(tw, a, most, st, who);
}

}  // namespace grouped
}  // namespace wq
