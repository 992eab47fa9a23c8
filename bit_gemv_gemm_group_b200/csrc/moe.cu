// Router and combine of a mixture-of-experts layer (one feed-forward network split into E experts,
// each token sent to k of them).
//
// wq_moe_route: from logits l [T][E], per token the k selectable experts with the largest logits
// (a logit is selectable when it is neither NaN nor -inf; ties go to the lowest expert), their
// softmax weights, and the grouping by expert that the expert products read: a stable counting sort
// of the T k (token, choice) pairs by expert, so that the rows of an expert are in token order and the
// result never depends on the order in which blocks run.
//
// A warp takes one token: lane l holds E / 32 neighbouring logits as order-preserving 32-bit keys, and each of
// the k rounds is one warp maximum, a ballot whose lowest lane is the lowest expert that holds it, and a pop in
// that lane.  Up to 64 tokens one block does everything in one launch.  Above, the first launch writes ids,
// weights and each block's expert counts, and the second adds up the counts of the blocks before its own, ranks
// its tokens and writes rows and slots; ranks come from a bit per (expert, token) of the chunk, so no
// order-dependent atomic decides a position.
#include "wq_device.cuh"
#include "wq_host.h"

#include <algorithm>
#include <climits>

namespace wq {
namespace {

constexpr int CHUNK = 128;        // tokens ranked at a time: four 32-bit words per expert
// Device time in a graph of calls, top 8.  Tokens of a single block: 128 tokens, 64 experts take it 9.9 us, two launches
// 5.4 us; 64 tokens 5.8 us.
constexpr int ONE_T = 64;
// Of a block of the first and of the second launch: 16384 tokens, 128 experts 16.9 us; 512 in the first 17.9 (64 tokens
// in one block 7.6), 1024 in the second 22.3.
constexpr int CHOOSE_THREADS = 1024, THREADS = 512;
constexpr int MIN_PER_BLOCK = 16, MAX_BLOCKS = 256;  // the second launch reads every block's counts
constexpr int MAX_E = 512, MAX_K = 32, MAX_T = MAX_BLOCKS * 32768;  // counts are 16 bits wide
constexpr uint32_t KEY_NONE = 0x007FFFFFu;  // key of -inf; keys at or below it are not selectable

__device__ __forceinline__ float load_logit(const float *p) { return __ldg(p); }
__device__ __forceinline__ float load_logit(const __half *p) { return __half2float(__ldg(p)); }
__device__ __forceinline__ float load_logit(const __nv_bfloat16 *p) { return __bfloat162float(__ldg(p)); }

// Order-preserving key of a logit: larger floats have larger keys, -0 and +0 the same one.
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (v != v) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_logit(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? (k ^ 0x80000000u) : ~k);
}

// exp(v - top) for v <= top, 1 at the top itself (also when both are +inf).
__device__ __forceinline__ float exp_below(float v, float top) { return v == top ? 1.0f : expf(v - top); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Larger keys first; exchanges of neighbours leave equal ones in their order.
__device__ __forceinline__ void order2(uint32_t &ka, int &ia, uint32_t &kb, int &ib) {
    if (kb > ka) {
        const uint32_t k = ka;
        ka = kb;
        kb = k;
        const int i = ia;
        ia = ib;
        ib = i;
    }
}

// One token's choice by one warp: lane j < k returns the j-th expert (-1 where none is left) and its weight.
template <typename T, int EPL>
__device__ __forceinline__ void choose(const T *__restrict__ row, int E, int k, bool renorm, int lane, int &id,
                                       float &weight) {
    uint32_t key[EPL];
    int at[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        at[i] = lane * EPL + i;
        key[i] = at[i] < E ? logit_key(load_logit(row + at[i])) : 0u;
    }
    float all = 0.0f, top = 0.0f;
    if (!renorm) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
        best = __reduce_max_sync(0xffffffffu, best);
        if (best > KEY_NONE) {
            top = key_logit(best);
#pragma unroll
            for (int i = 0; i < EPL; ++i)
                if (key[i] > KEY_NONE) all += exp_below(key_logit(key[i]), top);
        }
        all = warp_sum(all);
    }
    // Up to four keys a lane are sorted once, and a round pops the winner's first.  With more, the winner's
    // largest is found again.
    constexpr bool SORTED = EPL <= 4;
    if (SORTED && EPL > 1) {
#pragma unroll
        for (int p = 0; p < EPL - 1; ++p)
#pragma unroll
            for (int i = 0; i + 1 < EPL - p; ++i) order2(key[i], at[i], key[i + 1], at[i + 1]);
    }
    id = -1;
    uint32_t mine_key = 0u;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        int where = at[0];
        if (!SORTED) {
#pragma unroll
            for (int i = 1; i < EPL; ++i)
                if (key[i] > best) {
                    best = key[i];
                    where = at[i];
                }
        }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m <= KEY_NONE) break;
        const int win = __ffs(__ballot_sync(0xffffffffu, best == m)) - 1;
        const int e = __shfl_sync(0xffffffffu, where, win);
        if (lane == j) {
            id = e;
            mine_key = m;
        }
        if (lane == win) {
            if (SORTED) {
#pragma unroll
                for (int i = 0; i + 1 < EPL; ++i) {
                    key[i] = key[i + 1];
                    at[i] = at[i + 1];
                }
                key[EPL - 1] = 0u;
            } else {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (at[i] == where) key[i] = 0u;
            }
        }
    }
    const uint32_t top_key = __shfl_sync(0xffffffffu, mine_key, 0);
    const float mine = id >= 0 ? exp_below(key_logit(mine_key), key_logit(top_key)) : 0.0f;
    if (renorm) all = warp_sum(mine);
    weight = id >= 0 ? __fdiv_rn(mine, all) : 0.0f;
}

// Exclusive prefix of cnt[0..E) into base[0..E), total into base[E]; by one warp.
__device__ __forceinline__ void scan_counts(const int *cnt, int *base, int E, int lane) {
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
        const int v = e0 + lane < E ? cnt[e0 + lane] : 0;
        int s = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int n = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += n;
        }
        if (e0 + lane < E) base[e0 + lane] = run + s - v;
        run += __shfl_sync(0xffffffffu, s, 31);
    }
    if (lane == 0) base[E] = run;
}

struct RouteArgs {
    int T, E, k, per_block;  // per_block: tokens of one block
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *slots;
    uint16_t *counts;        // [blocks][E rounded up to 8]
};

__host__ __device__ constexpr int pitch_of(int E) { return (E + 7) & ~7; }

// Positions of one chunk's pairs: bits[e][w] has bit t % 32 of word t / 32 set when token t of the
// chunk chose e; a pair's rank is the number of set bits below its own, after base[e].  `ids`: the chunk's.
__device__ __forceinline__ void mark(uint32_t *bits, const int32_t *ids, int pairs, int k) {
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int t = i / k, e = ids[i];
        if (e >= 0) atomicOr(&bits[4 * e + (t >> 5)], 1u << (t & 31));
    }
}

__device__ __forceinline__ void place(const uint32_t *bits, const int *base, const int32_t *ids, const RouteArgs &a,
                                      int t0, int pairs) {
    for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int t = i / a.k, e = ids[i];
        int p = -1;
        if (e >= 0) {
            p = base[e] + __popc(bits[4 * e + (t >> 5)] & ((1u << (t & 31)) - 1u));
            for (int w = 0; w < (t >> 5); ++w) p += __popc(bits[4 * e + w]);
            a.rows[p] = t0 + t;
        }
        a.slots[(size_t)t0 * a.k + i] = p;
    }
}

__device__ __forceinline__ int set_bits(const uint32_t *bits, int e) {
    return __popc(bits[4 * e]) + __popc(bits[4 * e + 1]) + __popc(bits[4 * e + 2]) + __popc(bits[4 * e + 3]);
}

// Choices of the block's tokens; ONE: the whole of T is this block's single chunk, ranked at once.
template <typename T, int EPL, bool ONE>
__global__ void __launch_bounds__(CHOOSE_THREADS) route_choose_kernel(const T *__restrict__ logits, RouteArgs a,
                                                                      bool renorm) {
    extern __shared__ int sh[];  // ONE: bits [E][4], counts [E], base [E + 1], ids [T k]; else counts [E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)blockIdx.x * a.per_block, t1 = ONE ? a.T : min(a.T, t0 + a.per_block);
    int *cnt = ONE ? sh + 4 * a.E : sh;
    int32_t *ids = ONE ? sh + 6 * a.E + 1 : nullptr;
    for (int i = threadIdx.x; i < (ONE ? 5 : 1) * a.E; i += blockDim.x) sh[i] = 0;
    if (!ONE) asm volatile("griddepcontrol.launch_dependents;");  // route_place_kernel waits for this grid itself
    __syncthreads();
    for (int t = t0 + warp; t < t1; t += (int)blockDim.x / 32) {
        int id;
        float w;
        choose<T, EPL>(logits + (size_t)t * a.E, a.E, a.k, renorm, lane, id, w);
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = id;
            a.weights[(size_t)t * a.k + lane] = w;
            if (ONE) ids[t * a.k + lane] = id;
            if (id >= 0) atomicAdd(&cnt[id], 1);
        }
    }
    __syncthreads();
    if (!ONE) {
        const int pitch = pitch_of(a.E);
        for (int e = threadIdx.x; e < pitch; e += blockDim.x)
            a.counts[(size_t)blockIdx.x * pitch + e] = (uint16_t)(e < a.E ? cnt[e] : 0);
        return;
    }
    uint32_t *bits = reinterpret_cast<uint32_t *>(sh);
    int *base = cnt + a.E;
    mark(bits, ids, a.T * a.k, a.k);
    if (warp == 0) scan_counts(cnt, base, a.E, lane);
    __syncthreads();
    place(bits, base, ids, a, 0, a.T * a.k);
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.offsets[e] = base[e];
    for (int p = base[a.E] + threadIdx.x; p < a.T * a.k; p += blockDim.x) a.rows[p] = -1;
}

__global__ void __launch_bounds__(THREADS) route_place_kernel(RouteArgs a) {
    extern __shared__ int sh[];  // bits [E][4], totals [E8], before [E8], base [E + 1]
    const int E = a.E, pitch = pitch_of(E);
    uint32_t *bits = reinterpret_cast<uint32_t *>(sh);
    int *total = sh + 4 * E, *before = total + pitch, *base = before + pitch;
    for (int i = threadIdx.x; i < 4 * E + 2 * pitch; i += THREADS) sh[i] = 0;
    __syncthreads();
    // Launched before route_choose_kernel is done: nothing above reads what that writes.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // A thread adds eight experts' counts over every parts-th block: sums of integers, the same in any order.
    const int cols = pitch / 8, parts = THREADS / cols, part = threadIdx.x / cols, e0 = 8 * (threadIdx.x % cols);
    if (part < parts) {
        int all[8] = {}, low[8] = {};
#pragma unroll 8
        for (int b = part; b < (int)gridDim.x; b += parts) {
            const uint4 v = __ldcg(reinterpret_cast<const uint4 *>(a.counts + (size_t)b * pitch + e0));
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
            const bool is_low = b < (int)blockIdx.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int n = (u[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
                all[i] += n;
                low[i] += is_low ? n : 0;
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (all[i]) atomicAdd(&total[e0 + i], all[i]);
            if (low[i]) atomicAdd(&before[e0 + i], low[i]);
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) scan_counts(total, base, E, threadIdx.x);
    __syncthreads();
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += THREADS) a.offsets[e] = base[e];
    for (long long p = base[E] + (long long)blockIdx.x * THREADS + threadIdx.x; p < (long long)a.T * a.k;
         p += (long long)gridDim.x * THREADS)
        a.rows[p] = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += THREADS) base[e] += before[e];
    const int t0 = (int)blockIdx.x * a.per_block, t1 = min(a.T, t0 + a.per_block);
    for (int t = t0; t < t1; t += CHUNK) {
        const int pairs = min(CHUNK, t1 - t) * a.k;
        const int32_t *ids = a.ids + (size_t)t * a.k;
        __syncthreads();
        mark(bits, ids, pairs, a.k);
        __syncthreads();
        place(bits, base, ids, a, t, pairs);
        if (t + CHUNK >= t1) break;
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += THREADS) {
            base[e] += set_bits(bits, e);
            bits[4 * e] = bits[4 * e + 1] = bits[4 * e + 2] = bits[4 * e + 3] = 0u;
        }
    }
}

// Tokens per block: a token per warp, doubled until MAX_BLOCKS blocks cover T.
int tokens_per_block(int T) {
    int per = MIN_PER_BLOCK;
    while ((long long)per * MAX_BLOCKS < T) per *= 2;
    return per;
}

template <typename T, int EPL>
wq_status route_launch(const T *logits, const RouteArgs &a, bool renorm, cudaStream_t st) {
    if (a.T <= ONE_T) {
        const size_t smem = (6 * a.E + 1 + a.T * a.k) * sizeof(int);
        route_choose_kernel<T, EPL, true><<<1, CHOOSE_THREADS, smem, st>>>(logits, a, renorm);
        return check_launch("wq_moe_route");
    }
    const int blocks = (a.T + a.per_block - 1) / a.per_block;
    route_choose_kernel<T, EPL, false><<<blocks, CHOOSE_THREADS, a.E * sizeof(int), st>>>(logits, a, renorm);
    const wq_status e = check_launch("wq_moe_route");
    if (e != WQ_OK) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = (5 * a.E + 1 + 2 * pitch_of(a.E)) * sizeof(int);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t le = cudaLaunchKernelEx(&cfg, route_place_kernel, a);
    if (le != cudaSuccess) return fail(WQ_ERR_CUDA, "wq_moe_route: launch failed: %s", cudaGetErrorString(le));
    return WQ_OK;
}

template <typename T>
wq_status route_dispatch(const void *logits, const RouteArgs &a, bool renorm, cudaStream_t st) {
    const T *l = static_cast<const T *>(logits);
    if (a.E <= 32) return route_launch<T, 1>(l, a, renorm, st);
    if (a.E <= 64) return route_launch<T, 2>(l, a, renorm, st);
    if (a.E <= 128) return route_launch<T, 4>(l, a, renorm, st);
    if (a.E <= 256) return route_launch<T, 8>(l, a, renorm, st);
    return route_launch<T, 16>(l, a, renorm, st);
}

// ---------------------------------------------------------------------------
// Combine: out[t] = sum_j weights[t][j] * y[slots[t][j]], summed in fp32 in the order of j and rounded
// once; a slot outside [0, R) adds nothing.  One pass over y: a thread owns VEC neighbouring columns of
// one token and requests up to eight of its rows before it adds the first.
// ---------------------------------------------------------------------------
template <int VEC>
struct Pack;
template <>
struct Pack<8> { using type = uint4; };
template <>
struct Pack<4> { using type = uint2; };
template <>
struct Pack<2> { using type = uint32_t; };
template <>
struct Pack<1> { using type = uint16_t; };

template <bool BF>
__device__ __forceinline__ float from_bits(uint16_t b) {
    return BF ? __uint_as_float((uint32_t)b << 16) : half_bits_to_float(b);
}

template <bool BF>
__device__ __forceinline__ uint16_t to_bits(float v) {
    return BF ? float_to_bf16_bits_rn(v) : float_to_half_bits_rn(v);
}

constexpr int COMBINE_THREADS = 128, COMBINE_AHEAD = 8;

template <bool BF, int VEC>
__global__ void __launch_bounds__(COMBINE_THREADS) combine_kernel(const uint16_t *__restrict__ y, int R,
                                                                  const float *__restrict__ weights,
                                                                  const int32_t *__restrict__ slots, int k, int N,
                                                                  int segs, uint16_t *__restrict__ out) {
    using P = typename Pack<VEC>::type;
    const int t = (int)(blockIdx.x / segs);
    const int c = ((int)(blockIdx.x % segs) * COMBINE_THREADS + (int)threadIdx.x) * VEC;
    if (c >= N) return;
    float acc[VEC];
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
    for (int j0 = 0; j0 < k; j0 += COMBINE_AHEAD) {
        P v[COMBINE_AHEAD];
        float w[COMBINE_AHEAD];
        bool in[COMBINE_AHEAD];
#pragma unroll
        for (int j = 0; j < COMBINE_AHEAD; ++j) {
            const size_t at = (size_t)t * k + j0 + j;
            const int p = j0 + j < k ? __ldg(slots + at) : -1;
            in[j] = (unsigned)p < (unsigned)R;
            if (in[j]) {
                w[j] = __ldg(weights + at);
                v[j] = __ldg(reinterpret_cast<const P *>(y + (size_t)p * N + c));
            }
        }
#pragma unroll
        for (int j = 0; j < COMBINE_AHEAD; ++j) {
            if (!in[j]) continue;
            const uint16_t *h = reinterpret_cast<const uint16_t *>(&v[j]);
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w[j], from_bits<BF>(h[i]), acc[i]);
        }
    }
    P o;
    uint16_t *h = reinterpret_cast<uint16_t *>(&o);
#pragma unroll
    for (int i = 0; i < VEC; ++i) h[i] = to_bits<BF>(acc[i]);
    *reinterpret_cast<P *>(out + (size_t)t * N + c) = o;
}

template <bool BF, int VEC>
wq_status combine_launch(const uint16_t *y, int R, const float *weights, const int32_t *slots, int T, int k, int N,
                         uint16_t *out, cudaStream_t st) {
    const int segs = (N / VEC + COMBINE_THREADS - 1) / COMBINE_THREADS;
    WQ_REQUIRE((long long)T * segs <= INT_MAX, WQ_ERR_UNSUPPORTED, "wq_moe_combine: T (%d) x N (%d) is too large", T, N);
    combine_kernel<BF, VEC><<<T * segs, COMBINE_THREADS, 0, st>>>(y, R, weights, slots, k, N, segs, out);
    return check_launch("wq_moe_combine");
}

template <bool BF>
wq_status combine_dispatch(const uint16_t *y, int R, const float *weights, const int32_t *slots, int T, int k, int N,
                           uint16_t *out, cudaStream_t st) {
    // Rows start 2 N bytes apart: the widest load that divides that keeps every row's loads aligned.
    if (N % 8 == 0) return combine_launch<BF, 8>(y, R, weights, slots, T, k, N, out, st);
    if (N % 4 == 0) return combine_launch<BF, 4>(y, R, weights, slots, T, k, N, out, st);
    if (N % 2 == 0) return combine_launch<BF, 2>(y, R, weights, slots, T, k, N, out, st);
    return combine_launch<BF, 1>(y, R, weights, slots, T, k, N, out, st);
}

}  // namespace
}  // namespace wq

extern "C" size_t wq_moe_route_workspace_bytes(int T, int E) {
    if (T <= wq::ONE_T || T > wq::MAX_T || E <= 0) return 0;
    const int per = wq::tokens_per_block(T);
    return (size_t)((T + per - 1) / per) * (size_t)wq::pitch_of(E) * sizeof(uint16_t);
}

extern "C" wq_status wq_moe_route(const void *logits, wq_dtype dtype, int T, int E, int top_k, int renormalize,
                                  int32_t *ids, float *weights, int32_t *offsets, int32_t *rows, int32_t *slots,
                                  void *workspace, void *stream) {
    using namespace wq;
    WQ_REQUIRE_PTR(logits, "logits");
    WQ_REQUIRE_PTR(ids, "ids");
    WQ_REQUIRE_PTR(weights, "weights");
    WQ_REQUIRE_PTR(offsets, "offsets");
    WQ_REQUIRE_PTR(rows, "rows");
    WQ_REQUIRE_PTR(slots, "slots");
    WQ_REQUIRE(T > 0 && E > 0 && top_k > 0, WQ_ERR_INVALID_ARG,
               "wq_moe_route: sizes must be positive (T=%d E=%d top_k=%d)", T, E, top_k);
    WQ_REQUIRE(dtype == WQ_F32 || dtype == WQ_F16 || dtype == WQ_BF16, WQ_ERR_INVALID_ARG,
               "wq_moe_route: unknown dtype %d", (int)dtype);
    WQ_REQUIRE(top_k <= E, WQ_ERR_INVALID_ARG, "wq_moe_route: top_k (%d) must be at most E (%d)", top_k, E);
    WQ_REQUIRE(E <= MAX_E && top_k <= MAX_K, WQ_ERR_UNSUPPORTED,
               "wq_moe_route: E (%d) must be at most %d and top_k (%d) at most %d", E, MAX_E, top_k, MAX_K);
    WQ_REQUIRE(T <= MAX_T && (long long)T * top_k <= INT_MAX, WQ_ERR_UNSUPPORTED,
               "wq_moe_route: T (%d) must be at most %d, and T * top_k below 2^31", T, MAX_T);
    const size_t ws_bytes = wq_moe_route_workspace_bytes(T, E), pairs = (size_t)T * top_k * 4;
    if (ws_bytes) WQ_REQUIRE_PTR(workspace, "workspace");
    // Blocks write while others still read, so no two of these may share memory.
    const struct { const void *p; size_t n; } part[] = {
        {logits, (size_t)T * E * (dtype == WQ_F32 ? 4 : 2)}, {ids, pairs}, {weights, pairs}, {rows, pairs}, {slots, pairs},
        {offsets, ((size_t)E + 1) * 4}, {workspace, ws_bytes}};
    for (int i = 0; i < 7; ++i)
        for (int j = 0; j < i; ++j)
            WQ_REQUIRE(!(part[i].n && overlap(part[i].p, part[i].n, part[j].p, part[j].n)), WQ_ERR_INVALID_ARG,
                       "wq_moe_route: an output or the workspace overlaps another argument");
    const RouteArgs a{T, E, top_k, tokens_per_block(T), ids, weights, offsets, rows, slots,
                      static_cast<uint16_t *>(workspace)};
    cudaStream_t st = as_stream(stream);
    if (dtype == WQ_F32) return route_dispatch<float>(logits, a, renormalize != 0, st);
    if (dtype == WQ_F16) return route_dispatch<__half>(logits, a, renormalize != 0, st);
    return route_dispatch<__nv_bfloat16>(logits, a, renormalize != 0, st);
}

extern "C" wq_status wq_moe_combine(const uint16_t *y, wq_dtype dtype, int R, const float *weights,
                                    const int32_t *slots, int T, int top_k, int N, uint16_t *out, void *stream) {
    using namespace wq;
    WQ_REQUIRE_PTR(y, "y");
    WQ_REQUIRE_PTR(weights, "weights");
    WQ_REQUIRE_PTR(slots, "slots");
    WQ_REQUIRE_PTR(out, "out");
    WQ_REQUIRE(R > 0 && T > 0 && top_k > 0 && N > 0, WQ_ERR_INVALID_ARG,
               "wq_moe_combine: sizes must be positive (R=%d T=%d top_k=%d N=%d)", R, T, top_k, N);
    WQ_REQUIRE(dtype == WQ_F16 || dtype == WQ_BF16, WQ_ERR_INVALID_ARG,
               "wq_moe_combine: dtype must be WQ_F16 or WQ_BF16 (got %d)", (int)dtype);
    const size_t bytes = (size_t)T * N * 2, pairs = (size_t)T * top_k * 4;
    WQ_REQUIRE(!overlap(out, bytes, y, (size_t)R * N * 2) && !overlap(out, bytes, weights, pairs) &&
                   !overlap(out, bytes, slots, pairs),
               WQ_ERR_INVALID_ARG, "wq_moe_combine: out overlaps an input");
    cudaStream_t st = as_stream(stream);
    if (dtype == WQ_BF16) return combine_dispatch<true>(y, R, weights, slots, T, top_k, N, out, st);
    return combine_dispatch<false>(y, R, weights, slots, T, top_k, N, out, st);
}
