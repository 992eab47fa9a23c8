// Expert products with INT4 weights for a handful of rows per expert (single tokens and small decode batches):
//
//   y[p][n] = sum_j s[n][j] * ( sum_{k in group j} (q[n][k] - z[n][j]) x[rows[p]][k] )
//
// Nothing but the stream of packed weights counts here, and a tile of 16 tensor-core columns would be mostly
// padding; what has to be small is the number of instructions per code and the granularity of the work.  So every
// warp is on its own: it copies its codes into a ring of its own (cp.async, no barrier), turns them into q - z in
// registers (integers of 5 bits, exact in fp16 and bf16) straight in the order of an mma.sync fragment, and keeps
// the group sums and their scaled sums in fp32.  Warp-level MMAs rather than tcgen05: those take their
// operand from shared or tensor memory, and storing the converted codes there, with the hand-over between warps,
// is what bounds grouped_few.cu; at 8 columns the tensor work is a quarter of what the warp-level pipe does.
//
// Persistent CTAs of 4 or 8 warps, 16 warps an SM (see choose_tile); a tile is 16 RT weight rows times up to 8 rows
// of one expert.  The tile's depth is dealt to the CTA's warps in chunks of 128 codes, so that a weight row is read
// in contiguous pieces, and the warps' sums meet in shared memory in a fixed order.  A lane holds rows r and r + 8
// of each block of 16 (r = lane / 4) and a quarter (t = lane % 4) of a chunk's codes.
//
// Measured on B200, fp16, groups of 128: 2 of 8 experts of 28672 x 4096 for one token, 122 MB, 31 to 33 us (3.8 TB/s; 54
// us in grouped_few.cu), 8 experts for 32 rows, 485 MB, 104 to 113 us (4.5 TB/s; 152); 64 experts of 4096 x 2048 for 192
// rows, 268 MB, 65 us (4.1 TB/s; 90).  No unit is full (issue 0.59 of a slot a cycle and scheduler, integer pipe 53%, tensor
// pipe 28%, HBM 54%), and taking out one part gains little: the conversion 10%, the copies 3%, scales and zero points
// 7%, x 5%, half of the MMAs nothing.  The last round of tiles costs the rest: 896 tiles for one token are 1.5 rounds.
#include "grouped.cuh"

#include <algorithm>
#include <climits>
#include <type_traits>

namespace wq {
namespace grouped {
namespace {

using namespace sm100;

constexpr int BR = 8;          // rows of a tile, at most (the MMA's N)
constexpr int CHUNK = 128;     // codes of a weight row per step of a warp
constexpr int SM_WARPS = 16;   // of an SM: 128 registers a thread

template <int RT, int WARPS>
struct Layout {
    static constexpr uint32_t SLOT = RT * 16 * (CHUNK / 2);       // codes of a step
    static constexpr uint32_t RING = 2 * SLOT;
    // A warp's sums: [4 pairs of rows][16 RT weight rows], pitch chosen so that a half warp's stores of
    // fragments fall into different banks.
    static constexpr uint32_t PAIR = (RT * 16 + 4) * 8;
    static constexpr uint32_t PART = 4 * PAIR;
    static constexpr uint32_t OFF_RED = WARPS * RING;             // two buffers: one barrier per tile
    static constexpr uint32_t OFF_TAB = OFF_RED + 2 * WARPS * PART;
    static constexpr size_t bytes(int E) { return OFF_TAB + 2 * (size_t)(E + 1) * 4; }
};

// d = a b + c; the first product of a group starts from zeros, which take no register.
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1, bool first) {
    const float c0 = first ? 0.0f : d[0], c1 = first ? 0.0f : d[1], c2 = first ? 0.0f : d[2], c3 = first ? 0.0f : d[3];
    if (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
            "{%10,%11,%12,%13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Loads that stay where they are written: a prefetch that moved to its use would show its whole latency.
__device__ __forceinline__ uint4 load128(const void *p) {
    uint4 v;
    asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t load32(const void *p) {
    uint32_t v;
    asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t load16(const void *p) {
    uint16_t v;
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
    return v;
}

// Tile t of the list as get_tile finds it, by a whole warp: the lanes look at 32 experts at a time, and an expert
// with no more rows than a tile needs no division.
template <int BN>
__device__ __forceinline__ bool find_tile(const Args &a, const int *off, const int *tiles, int t, int lane, Tile &w) {
    if (t >= tiles[a.E]) return false;
    int e = -1;
    for (int i = lane; i - lane < a.E; i += 32) {
        const int n = __popc(__ballot_sync(0xffffffffu, i < a.E && tiles[i] <= t));
        e += n;
        if (n < 32) break;
    }
    const int first = off[e], n = off[e + 1] - first;
    int local = t - tiles[e];
    w.e = e;
    w.r0 = first;
    w.rows = n;
    if (n > BR) {
        const int rb = (n + BR - 1) / BR, b = local % rb;
        local /= rb;
        w.r0 += b * BR;
        w.rows = min(BR, n - b * BR);
    }
    w.n0 = local * BN;
    return true;
}

// SUB: groups of codes in a chunk, 1 (group size 128 or more), 2 (64) or 4 (32).
template <bool BF, bool SWIGLU, int SUB, int RT, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, SM_WARPS / WARPS)
    stream_rows_kernel(const uint8_t *__restrict__ weights, const Args a) {
    using L = Layout<RT, WARPS>;
    constexpr int BN = SWIGLU ? RT * 8 : RT * 16;   // output columns per tile
    constexpr int HALF = SWIGLU ? RT / 2 : RT;      // blocks of 16 rows before those of up rows
    constexpr int CPL = RT / 2;                     // of the 2 RT rows of a quad: those whose scales a lane loads
    extern __shared__ __align__(128) uint8_t smem[];
    int *off = reinterpret_cast<int *>(smem + L::OFF_TAB), *tiles = off + a.E + 1;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, t = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * L::RING;
    const int chunks = (a.K + CHUNK - 1) / CHUNK, lg = 31 - __clz(a.gs), groups = a.K >> lg, zwords = (groups + 7) / 8;
    const int pitch = a.K / 2;
    const uint32_t magic = opaque_const(BF ? 0x43004300u : 0x64006400u);

    if (warp == 0) build_table<BR>(a, off, tiles, lane);
    __syncthreads();

    // What is requested next: chunk c of tile nt.
    int nt = blockIdx.x, c = warp;
    Tile nw;
    int last = 0;                          // of the tile's rows (or gate rows) that exist, counted from r
    bool whole = false;                    // all of them do
    const uint8_t *gate = nullptr, *up = nullptr, *xp = nullptr;   // row r of the tile's gate, up and activation rows
    const uint16_t *srow[CPL];
    const uint32_t *zrow[CPL];
    auto enter = [&]() -> bool {
        if (!find_tile<BN>(a, off, tiles, nt, lane, nw)) return false;
        const size_t row0 = (size_t)nw.e * a.N + nw.n0;
        gate = weights + (row0 + r) * pitch + t * 16;
        up = gate + (size_t)(a.N / 2) * pitch;
        last = min(BN, a.ldy - nw.n0) - 1 - r;
        whole = last + r == BN - 1;
        // Past the tile's rows the last of them, for an index outside x row 0: their sums are not stored.
        int v = nw.r0 + min(r, nw.rows - 1);
        if (a.rows) v = __ldg(a.rows + v);
        xp = a.x + ((unsigned)v < (unsigned)a.T ? (size_t)v : 0) * ((size_t)a.K * 2) + (SUB == 1 ? t * 64 : t * 16);
#pragma unroll
        for (int u = 0; u < CPL; ++u) {
            const int q = t * CPL + u, i = q >> 1;
            const size_t row = row0 + (SWIGLU && i >= HALF ? a.N / 2 : 0) + (r + min(16 * (i % HALF) + 8 * (q & 1), last));
            srow[u] = a.scales + row * groups;
            zrow[u] = a.qzeros + row * zwords;
        }
        return true;
    };
    uint4 nx[4];
    uint32_t ns[CPL][SUB], nz[CPL];
    // `all`: every row and code of it exists.
    auto request_as = [&](uint32_t slot, auto all) {
        constexpr bool ALL = decltype(all)::value;
        const int k0 = c * CHUNK;
        const bool in = ALL || k0 + 32 * t < a.K;
        // Where a group is shorter than a chunk, a lane takes word t of every 16 bytes (see below): swizzled, so that
        // those reads fall into different banks.
        const uint32_t dst = ring + slot * L::SLOT + r * 64 + (SUB == 1 ? t : t ^ ((r >> 1) & 3)) * 16;
        const int at = in ? k0 / 2 : 0;
        const uint8_t *g = gate + at, *v = up + at;
#pragma unroll
        for (int i = 0; i < RT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // rows past the end: the last one
                const int row = 16 * (i % HALF) + 8 * h;
                cp_async16(dst + (2 * i + h) * 512,
                           (SWIGLU && i >= HALF ? v : g) + (long long)(ALL ? row : min(row, last)) * pitch, in);
            }
        const uint8_t *xk = xp + (size_t)(uint32_t)k0 * 2;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            nx[j] = ALL || (SUB == 1 ? in : k0 + 32 * j < a.K) ? load128(xk + (SUB == 1 ? 16 : 64) * j)
                                                               : make_uint4(0, 0, 0, 0);
        const int g0 = k0 >> lg;
#pragma unroll
        for (int u = 0; u < CPL; ++u) {
#pragma unroll
            for (int s = 0; s < SUB; ++s) ns[u][s] = ALL || g0 + s < groups ? load16(srow[u] + g0 + s) : 0u;
            nz[u] = load32(zrow[u] + (g0 >> 3)) >> (4 * (g0 & 7));
        }
    };
    auto request = [&](uint32_t slot) {
        if (whole && (c + 1) * CHUNK <= a.K) request_as(slot, std::true_type{});
        else request_as(slot, std::false_type{});
    };

    bool have = enter();
    const bool mine = c < chunks;          // some of a tile's depth is this warp's
    uint32_t slot = 0;
    if (have && mine) request(0);
    cp_async_commit();

    for (int buf = 0; have; buf ^= 1) {
        const Tile w = nw;                 // its first chunk of this warp has been requested
        if (!mine) {
            nt += gridDim.x;
            have = enter();
        }
        float acc[RT][4];
#pragma unroll
        for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.0f;
        for (int b = warp; b < chunks; b += WARPS) {
            uint4 x[4];
            uint32_t sz[CPL][SUB];   // scale and zero point of a row and group
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = permute_x(nx[j]);
#pragma unroll
            for (int u = 0; u < CPL; ++u)
#pragma unroll
                for (int s = 0; s < SUB; ++s) sz[u][s] = ns[u][s] | Zero<BF>::pack((nz[u] >> (4 * s)) & 0xFu);
            c += WARPS;
            if (c >= chunks) {
                c = warp;
                nt += gridDim.x;
                have = enter();
            }
            if (have) request(slot ^ 1);
            cp_async_commit();
            cp_async_wait<1>();
            __syncwarp();
            const uint32_t src = ring + slot * L::SLOT + (SUB == 1 ? lane * 16 : r * 64 + t * 4);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                uint32_t q[2][4];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (SUB == 1) {
                        const uint4 v = lds128(src + (2 * i + h) * 512);
                        q[h][0] = v.x, q[h][1] = v.y, q[h][2] = v.z, q[h][3] = v.w;
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            q[h][j] = lds32(src + (2 * i + h) * 512 + ((j ^ ((r >> 1) & 3)) << 4));
                    }
                }
#pragma unroll
                for (int s = 0; s < SUB; ++s) {
                    uint32_t p[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        p[h] = __shfl_sync(0xffffffffu, sz[(2 * i + h) % CPL][s], (lane & ~3) | ((2 * i + h) / CPL));
                    const Zero<BF> z0 = Zero<BF>::unpack(p[0]), z1 = Zero<BF>::unpack(p[1]);
                    float d[4];
#pragma unroll
                    for (int j = s * (4 / SUB); j < (s + 1) * (4 / SUB); ++j) {
                        uint32_t o0[4], o1[4];
                        code_word<BF>(q[0][j], magic, z0, o0);
                        code_word<BF>(q[1][j], magic, z1, o1);
                        mma<BF>(d, o0[0], o1[0], o0[1], o1[1], x[j].x, x[j].y, j == s * (4 / SUB));
                        mma<BF>(d, o0[2], o1[2], o0[3], o1[3], x[j].z, x[j].w, false);
                    }
                    const float s0 = half_bits_to_float((uint16_t)p[0]), s1 = half_bits_to_float((uint16_t)p[1]);
                    acc[i][0] = fmaf(s0, d[0], acc[i][0]);
                    acc[i][1] = fmaf(s0, d[1], acc[i][1]);
                    acc[i][2] = fmaf(s1, d[2], acc[i][2]);
                    acc[i][3] = fmaf(s1, d[3], acc[i][3]);
                }
            }
            __syncwarp();   // every lane has read the slot that the next request fills
            slot ^= 1;
        }
        uint8_t *part = smem + L::OFF_RED + (buf * WARPS + warp) * L::PART;
        if (2 * t < w.rows) {
#pragma unroll
            for (int i = 0; i < RT; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float2 *>(part + t * L::PAIR + (16 * i + 8 * h + r) * 8) =
                        make_float2(acc[i][2 * h], acc[i][2 * h + 1]);
        }
        __syncthreads();
        const int n = threadIdx.x % BN, col = w.n0 + n;
        if (col >= a.ldy) continue;
        for (int pair = threadIdx.x / BN; pair < 4 && 2 * pair < w.rows; pair += WARPS * 32 / BN) {
            const uint8_t *sum = smem + L::OFF_RED + buf * WARPS * L::PART + pair * L::PAIR + n * 8;
            float2 v = make_float2(0.0f, 0.0f), u = v;
#pragma unroll
            for (int i = 0; i < WARPS; ++i) {
                const float2 f = *reinterpret_cast<const float2 *>(sum + i * L::PART);
                v.x += f.x, v.y += f.y;
                if (SWIGLU) {
                    const float2 g = *reinterpret_cast<const float2 *>(sum + i * L::PART + BN * 8);
                    u.x += g.x, u.y += g.y;
                }
            }
            if (SWIGLU) v = make_float2(swiglu(v.x, u.x), swiglu(v.y, u.y));
            const int p = w.r0 + 2 * pair;
            const bool two = 2 * pair + 1 < w.rows;
            if (a.rows) {   // an index outside x: zeros, whatever the scales are
                if ((unsigned)__ldg(a.rows + p) >= (unsigned)a.T) v.x = 0.0f;
                if (two && (unsigned)__ldg(a.rows + p + 1) >= (unsigned)a.T) v.y = 0.0f;
            }
            const uint32_t o = round_pair<BF>(v.x, v.y);
            uint16_t *y = a.y + (size_t)p * a.ldy + col;
            *y = (uint16_t)o;
            if (two) y[a.ldy] = (uint16_t)(o >> 16);
        }
    }
}

template <bool BF, bool SWIGLU, int SUB, int RT, int WARPS>
wq_status launch(const void *w, Args a, cudaStream_t st, const char *who) {
    using L = Layout<RT, WARPS>;
    auto kern = stream_rows_kernel<BF, SWIGLU, SUB, RT, WARPS>;
    static std::atomic<uint64_t> allowed{0};
    const wq_status ok = allow_smem(kern, L::bytes(MAX_E), allowed, who);
    if (ok != WQ_OK) return ok;
    const int bn = SWIGLU ? RT * 8 : RT * 16;
    a.nb = (a.ldy + bn - 1) / bn;
    const long long most = ((long long)std::min(a.E, a.R) + a.R / BR) * a.nb;  // tiles of any offsets
    WQ_REQUIRE(most < INT_MAX / 2, WQ_ERR_UNSUPPORTED, "%s: R (%d) x N (%d) gives too many tiles", who, a.R, a.N);
    const int grid = (int)std::min<long long>((long long)num_sms() * (SM_WARPS / WARPS), most);
    kern<<<grid, WARPS * 32, L::bytes(a.E), st>>>(static_cast<const uint8_t *>(w), a);
    return check_launch(who);
}

// Tiles and warps by the number of tiles of 64 weight rows (if every row had an expert of its own): four warps a
// tile as soon as that leaves none without work, for a tile costs a warp its set-up and a barrier however short its
// share of the depth; eight warps below, and half as many rows where there are fewer tiles than SMs.  Measured on
// B200, fp16, four and eight warps: 64 experts of 4096 x 2048 for 192 rows (4032 tiles) 76 and 84 us; 8 experts of
// 4096 x 14336 for 16 rows (450 tiles) 74 and 70 us.  One expert of 4096 x 14336 (64 tiles), eight warps, tiles of
// 64 and 32 rows: 23 and 17 us; 8 experts of 28672 x 4096 (3100 tiles): 111 and 140 us.
template <bool BF, bool SWIGLU, int SUB>
wq_status choose_tile(const void *w, const Args &a, cudaStream_t st, const char *who) {
    const int bn = SWIGLU ? 32 : 64, sms = num_sms();
    const long long tiles = (long long)std::min(a.E, a.R) * ((a.ldy + bn - 1) / bn);
    if (tiles >= 4ll * sms) return launch<BF, SWIGLU, SUB, 4, 4>(w, a, st, who);
    if (tiles >= sms) return launch<BF, SWIGLU, SUB, 4, 8>(w, a, st, who);
    return launch<BF, SWIGLU, SUB, 2, 8>(w, a, st, who);
}

template <bool BF, bool SWIGLU>
wq_status choose_group(const void *w, const Args &a, cudaStream_t st, const char *who) {
    if (a.gs >= 128) return choose_tile<BF, SWIGLU, 1>(w, a, st, who);
    if (a.gs == 64) return choose_tile<BF, SWIGLU, 2>(w, a, st, who);
    return choose_tile<BF, SWIGLU, 4>(w, a, st, who);
}

}  // namespace

wq_status stream_rows_w4(const void *w, Args a, bool bf16, bool swiglu, cudaStream_t st, const char *who) {
    a.ldy = swiglu ? a.N / 2 : a.N;
    if (bf16) return swiglu ? choose_group<true, true>(w, a, st, who) : choose_group<true, false>(w, a, st, who);
    return swiglu ? choose_group<false, true>(w, a, st, who) : choose_group<false, false>(w, a, st, who);
}

}  // namespace grouped
}  // namespace wq
