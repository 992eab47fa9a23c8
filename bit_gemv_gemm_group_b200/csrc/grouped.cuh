// Shared by the kernels of the expert products: arguments, the tile list that every CTA derives from the
// offsets in device memory, and small device helpers.
#pragma once

#include <atomic>

#include "sm100.cuh"
#include "wq_device.cuh"
#include "wq_host.h"

namespace wq {
namespace grouped {

constexpr int BM = 128;                // weight rows of a CTA's share of a tile (TMEM lanes)
constexpr int MAX_E = 512;
constexpr uint64_t DRAIN_NS = 2000000000ull;

struct Args {
    const uint8_t *x;                // [T] rows
    const int32_t *offsets, *rows;   // rows null: row p of x itself
    const float *sx, *sw;
    int sx_stride, sw_per_row;
    const uint16_t *scales;          // INT4: fp16 [E][N][K/gs]
    const uint32_t *qzeros;
    uint16_t *y;
    int T, R, E, N, K, gs;           // T: rows of x, R: grouped rows
    int nb;                          // weight-row blocks per expert
    int box;                         // SwiGLU: the weight map is the 5-D one (see load_weights)
    int ldy;                         // columns of y (N, or N / 2 with SwiGLU)
    unsigned int *status;
    uint64_t limit_ns;
};

struct Tile {
    int e, n0;        // expert, first output column of the tile
    int r0, rows;     // first grouped row, number of rows
};

// Offsets clamped to [0, R] and made non-decreasing (a valid array is unchanged), and the exclusive
// prefix of the experts' tile counts; by one warp.
template <int BR>
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
        const int v = i0 + lane < a.E ? (off[i0 + lane + 1] - off[i0 + lane] + BR - 1) / BR * a.nb : 0;
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

// Tile t of the list; false past its end.  BN: output columns per tile, BR and STEP: most rows of a block
// and what its length is rounded up to.
template <int BN, int BR, int STEP>
__device__ __forceinline__ bool get_tile(const Args &a, const int *off, const int *tiles, int t, Tile &w) {
    if (t >= tiles[a.E]) return false;
    int lo = 0, hi = a.E;  // the expert e with tiles[e] <= t < tiles[e + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tiles[mid] <= t) lo = mid;
        else hi = mid;
    }
    const int first = off[lo], n = off[lo + 1] - first, rb = (n + BR - 1) / BR;
    const int per = ((n + rb - 1) / rb + STEP - 1) / STEP * STEP;
    const int local = t - tiles[lo], b = local % rb;
    w.e = lo;
    w.n0 = (local / rb) * BN;
    w.r0 = first + b * per;
    w.rows = min(per, n - b * per);
    return true;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// (w & mask) | magic in one LOP3: `magic` comes from opaque_const, which the compiler cannot fold into a second one.
__device__ __forceinline__ uint32_t mask_or(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(w), "r"(mask), "r"(magic));
    return d;
}

__device__ __forceinline__ uint32_t opaque_const(uint32_t v) {
    uint32_t m;
    asm volatile("mov.b32 %0, %1;" : "=r"(m) : "r"(v));
    return m;
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

__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}

// q - z of the 8 codes of a word as fp16 or bf16 pairs, in the order 0, 4, 1, 5, 2, 6, 3, 7 in which masks of
// the word leave them (x is taken in the same order, see permute_x): the integer pipe, which runs at half
// the issue rate, is the busiest one of the kernels that do this, and in k order each pair would take a byte permutation more.
// fp16: masked nibbles under the exponent of 1024 read 1024 + q (low nibbles) and 1024 + 16 q (high ones).
// bf16: 128 + q has 8 bits, so every nibble is shifted down first.
template <bool BF>
struct Zero {
    uint32_t lo, hi;   // fp16: -(1024 + z) and -(64 + z); bf16: -(128 + z)
    __device__ __forceinline__ explicit Zero(uint32_t z)
        : lo((BF ? 0xC300C300u : 0xE400E400u) + z * 0x00010001u), hi(0xD400D400u + z * 0x00100010u) {}
    // From 16 bits of a register whose lower half is free for something else.
    static __device__ __forceinline__ uint32_t pack(uint32_t z) { return ((BF ? 0xC300u : 0xE400u) + z) << 16; }
    static __device__ __forceinline__ Zero unpack(uint32_t v) {
        Zero r(0);
        r.lo = prmt(v, 0u, 0x3232u);
        r.hi = r.lo * 16u + (0xD400D400u - 0xE400E400u * 16u);
        return r;
    }
};

template <bool BF>
__device__ __forceinline__ void code_word(uint32_t w, uint32_t magic, const Zero<BF> &z, uint32_t *o) {
    if (BF) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(o[i]) : "r"(mask_or(w >> (4 * i), 0x000F000Fu, magic)), "r"(z.lo));
    } else {
        const uint32_t w8 = w >> 8;
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[0]) : "r"(mask_or(w, 0x000F000Fu, magic)), "r"(z.lo));
        o[1] = hfma2(mask_or(w, 0x00F000F0u, magic), 0x2C002C00u, z.hi);
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(o[2]) : "r"(mask_or(w8, 0x000F000Fu, magic)), "r"(z.lo));
        o[3] = hfma2(mask_or(w8, 0x00F000F0u, magic), 0x2C002C00u, z.hi);
    }
}

// Eight values of x in the order of code_word.
__device__ __forceinline__ uint4 permute_x(uint4 v) {
    return make_uint4(prmt(v.x, v.z, 0x5410u), prmt(v.x, v.z, 0x7632u), prmt(v.y, v.w, 0x5410u),
                      prmt(v.y, v.w, 0x7632u));
}

// silu(g) u.  With e = exp(-|g|) <= 1, silu(g) = g / (1 + e) or g e / (1 + e): nothing overflows, and a gate far below
// zero keeps its value until e itself is below fp32's subnormals (g = -103).  The fast exponential is off by at most
// 2 + 1.2 |g| units and the fast division (divisors of 1 to 2) by 2: less than 2^-16 for every g whose silu is not
// subnormal, far below the 16-bit rounding that follows.  An IEEE division costs 18.4 against 15.7 us in 903 rows of 20
// FP8 experts of 1000 x 1360.
__device__ __forceinline__ float swiglu(float g, float u) {
    const float e = __expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e) * u;
}

// Two values rounded to fp16 or bf16, the first in the low half: one instruction, where a conversion of a single
// value takes the quarter-rate pipe.
template <bool BF>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
    uint32_t d;
    if (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
    return d;
}

// Stores v[0 .. count) down a column of y: rows `step` elements apart.  `full` (the same in the whole warp): all of
// them, without a test per row.
template <bool BF, int N>
__device__ __forceinline__ void store_column(uint16_t *y, size_t step, const float (&v)[N], int count, bool full) {
    if (full) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const uint32_t h = round_pair<BF>(v[j], v[j + 1]);
            *y = (uint16_t)h;
            y += step;
            *y = (uint16_t)(h >> 16);
            y += step;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            const uint32_t h = round_pair<BF>(v[j], v[j + 1]);
            if (j < count) *y = (uint16_t)h;
            y += step;
            if (j + 1 < count) *y = (uint16_t)(h >> 16);
            y += step;
        }
    }
}

// Lets `kern` use `smem` bytes of shared memory, once per device (`done`: a bit each).
template <typename Kernel>
wq_status allow_smem(Kernel kern, size_t smem, std::atomic<uint64_t> &done, const char *who) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const uint64_t bit = 1ull << (dev & 63);
    if (e == cudaSuccess && (done.load(std::memory_order_acquire) & bit)) return WQ_OK;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return fail(WQ_ERR_CUDA, "%s: cudaFuncSetAttribute: %s", who, cudaGetErrorString(e));
    done.fetch_or(bit, std::memory_order_release);
    return WQ_OK;
}

// Clusters of `size` CTAs of a kernel that are resident at once (one CTA per SM; some GPCs have SMs left over), at
// least 1.  A persistent grid of more clusters would run the rest after the others have finished.
template <typename Kernel>
int resident_clusters(Kernel kern, int threads, size_t smem, int size) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(num_sms() / size * size);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess) {
        cudaGetLastError();
        n = num_sms() / size;
    }
    return n < 1 ? 1 : n;
}

// Map of the stacked weights for tiles of 128 rows x `width` bytes, 64 or 128, with the swizzle of that width
// (row_bytes: bytes of a weight row).  SwiGLU with I % 16 == 0: the 5-D view [E][I / 16][2][16][row] (a.box), whose box of
// 4 x 2 x 16 rows is 16 gate rows, their 16 up rows, and so on; otherwise boxes of 16 rows.
bool encode_weights(CUtensorMap *map, const void *w, uint64_t row_bytes, int width, Args &a, bool swiglu);

// INT4 weights and 7 to 22 rows per expert (grouped_few.cu); `bf16`: type of x and y.
wq_status few_rows_w4(const void *w, Args a, bool bf16, bool swiglu, cudaStream_t st, const char *who);

// INT4 weights and a handful of rows per expert (grouped_stream.cu).
wq_status stream_rows_w4(const void *w, Args a, bool bf16, bool swiglu, cudaStream_t st, const char *who);

}  // namespace grouped
}  // namespace wq
