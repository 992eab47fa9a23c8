// Router and combine of a mixture-of-experts layer (one feed-forward network split into E experts,
// each token sent to k of them).
//
// wq_moe_route: from logits l [T][E], per token the k selectable experts with the largest logits
// (a logit is selectable when it is neither NaN nor -inf; ties go to the lowest expert), their
// softmax weights, and the grouping by expert that the expert products read: a stable counting sort
// of the T k (token, choice) pairs by expert, so that the rows of an expert are in token order and the
// result never depends on the order in which blocks run.
//
// A warp takes one token: lane l holds logits l, l + 32, ... as order-preserving 32-bit keys, and each
// of the k rounds is a lane-local maximum, one warp maximum of the keys and one warp minimum of the
// indices that hold it.  A block of 32 warps takes chunks of 128 tokens.  Up to 128 tokens one block
// does everything in one launch.  Above, the first launch writes ids, weights and each block's expert
// counts, and the second adds up the counts of the blocks before its own, ranks its tokens and writes
// rows and slots; ranks come from a bit per (expert, token) of the chunk, so no order-dependent atomic
// decides a position.
#include "wq_device.cuh"
#include "wq_host.h"

#include <algorithm>
#include <climits>

namespace wq {
namespace {

constexpr int CHUNK = 128;        // tokens ranked at a time: four 32-bit words per expert
constexpr int ROUTE_WARPS = 32;
constexpr int ROUTE_THREADS = 32 * ROUTE_WARPS;
constexpr int MAX_BLOCKS = 256;   // the second launch reads every block's counts: few, larger blocks
constexpr int MAX_E = 512, MAX_K = 32;
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

// One token's choice by one warp: lane j < k returns the j-th expert (-1 where none is left) and its weight.
template <typename T, int EPL>
__device__ __forceinline__ void choose(const T *__restrict__ row, int E, int k, bool renorm, int lane, int &id,
                                       float &weight) {
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        const int e = lane + 32 * i;
        key[i] = e < E ? logit_key(load_logit(row + e)) : 0u;
    }
    id = -1;
    float mine = 0.0f, top = 0.0f, all = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = 0u;
        int at = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i;
            }
        const uint32_t m = __reduce_max_sync(0xffffffffu, best);
        if (m <= KEY_NONE) break;
        const unsigned e = __reduce_min_sync(0xffffffffu, best == m ? (unsigned)(lane + 32 * at) : UINT_MAX);
        if (j == 0) {
            top = key_logit(m);
            if (!renorm) {
#pragma unroll
                for (int i = 0; i < EPL; ++i)
                    if (key[i] > KEY_NONE) all += exp_below(key_logit(key[i]), top);
                all = warp_sum(all);
            }
        }
        if (lane == j) {
            id = (int)e;
            mine = exp_below(key_logit(m), top);
        }
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (e == (unsigned)(lane + 32 * i)) key[i] = 0u;
    }
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
    int T, E, k, per_block;  // per_block: tokens of one block, a multiple of CHUNK
    int32_t *ids;
    float *weights;
    int32_t *offsets, *rows, *slots;
    int *counts;             // [blocks][E]
};

// Positions of one chunk's pairs: bits[e][w] has bit t % 32 of word t / 32 set when token t of the
// chunk chose e; a pair's rank is the number of set bits below its own, after base[e].
__device__ __forceinline__ void mark(uint32_t *bits, const RouteArgs &a, int t0, int n) {
    for (int i = threadIdx.x; i < n * a.k; i += blockDim.x) {
        const int t = i / a.k, e = a.ids[(size_t)t0 * a.k + i];
        if (e >= 0) atomicOr(&bits[4 * e + (t >> 5)], 1u << (t & 31));
    }
}

__device__ __forceinline__ void place(const uint32_t *bits, const int *base, const RouteArgs &a, int t0, int n) {
    for (int i = threadIdx.x; i < n * a.k; i += blockDim.x) {
        const int t = i / a.k, e = a.ids[(size_t)t0 * a.k + i];
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
__global__ void __launch_bounds__(ROUTE_THREADS) route_choose_kernel(const T *__restrict__ logits, RouteArgs a,
                                                                     bool renorm) {
    extern __shared__ int sh[];  // ONE: bits [E][4], counts [E], base [E + 1]; else counts [E]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int t0 = (int)blockIdx.x * a.per_block, t1 = min(a.T, t0 + a.per_block);
    int *cnt = ONE ? sh + 4 * a.E : sh;
    for (int i = threadIdx.x; i < (ONE ? 5 : 1) * a.E; i += ROUTE_THREADS) sh[i] = 0;
    __syncthreads();
    for (int t = t0 + warp; t < t1; t += ROUTE_WARPS) {
        int id;
        float w;
        choose<T, EPL>(logits + (size_t)t * a.E, a.E, a.k, renorm, lane, id, w);
        if (lane < a.k) {
            a.ids[(size_t)t * a.k + lane] = id;
            a.weights[(size_t)t * a.k + lane] = w;
            if (id >= 0) atomicAdd(&cnt[id], 1);
        }
    }
    __syncthreads();
    if (!ONE) {
        for (int e = threadIdx.x; e < a.E; e += ROUTE_THREADS) a.counts[(size_t)blockIdx.x * a.E + e] = cnt[e];
        return;
    }
    uint32_t *bits = reinterpret_cast<uint32_t *>(sh);
    int *base = cnt + a.E;
    mark(bits, a, 0, a.T);
    if (warp == 0) scan_counts(cnt, base, a.E, lane);
    __syncthreads();
    place(bits, base, a, 0, a.T);
    for (int e = threadIdx.x; e <= a.E; e += ROUTE_THREADS) a.offsets[e] = base[e];
    for (int p = base[a.E] + threadIdx.x; p < a.T * a.k; p += ROUTE_THREADS) a.rows[p] = -1;
}

__global__ void __launch_bounds__(ROUTE_THREADS) route_place_kernel(RouteArgs a) {
    extern __shared__ int sh[];  // bits [E][4], totals [E], before [E], base [E + 1]
    const int E = a.E;
    uint32_t *bits = reinterpret_cast<uint32_t *>(sh);
    int *total = sh + 4 * E, *before = total + E, *base = before + E;
    const int lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < 6 * E; i += ROUTE_THREADS) sh[i] = 0;
    __syncthreads();
    // Every thread adds one expert's counts over every (ROUTE_THREADS / E)-th block: sums of integers,
    // the same in any order.
    const int parts = max(1, ROUTE_THREADS / E), part = threadIdx.x / E, e0 = threadIdx.x % E;
    if (part < parts) {
        int all = 0, low = 0;
#pragma unroll 4
        for (int b = part; b < (int)gridDim.x; b += parts) {
            const int v = a.counts[(size_t)b * E + e0];
            all += v;
            low += b < (int)blockIdx.x ? v : 0;
        }
        if (all) atomicAdd(&total[e0], all);
        if (low) atomicAdd(&before[e0], low);
    }
    __syncthreads();
    if (threadIdx.x < 32) scan_counts(total, base, E, lane);
    __syncthreads();
    const int last = base[E];
    if (blockIdx.x == 0)
        for (int e = threadIdx.x; e <= E; e += ROUTE_THREADS) a.offsets[e] = base[e];
    for (long long p = last + (long long)blockIdx.x * ROUTE_THREADS + threadIdx.x; p < (long long)a.T * a.k;
         p += (long long)gridDim.x * ROUTE_THREADS)
        a.rows[p] = -1;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) base[e] += before[e];
    const int t0 = (int)blockIdx.x * a.per_block, t1 = min(a.T, t0 + a.per_block);
    for (int t = t0; t < t1; t += CHUNK) {
        const int n = min(CHUNK, t1 - t);
        __syncthreads();
        mark(bits, a, t, n);
        __syncthreads();
        place(bits, base, a, t, n);
        __syncthreads();
        for (int e = threadIdx.x; e < E; e += ROUTE_THREADS) {
            base[e] += set_bits(bits, e);
            bits[4 * e] = bits[4 * e + 1] = bits[4 * e + 2] = bits[4 * e + 3] = 0u;
        }
    }
}

// Tokens per block: one chunk, doubled until MAX_BLOCKS blocks cover T.
int tokens_per_block(int T) {
    long long per = CHUNK;
    while (per * MAX_BLOCKS < T) per *= 2;
    return (int)per;
}

template <typename T, int EPL>
wq_status route_launch(const T *logits, RouteArgs a, bool renorm, cudaStream_t st) {
    if (a.T <= CHUNK) {
        route_choose_kernel<T, EPL, true><<<1, ROUTE_THREADS, (6 * a.E + 1) * sizeof(int), st>>>(logits, a, renorm);
        return check_launch("wq_moe_route");
    }
    const int blocks = (a.T + a.per_block - 1) / a.per_block;
    route_choose_kernel<T, EPL, false><<<blocks, ROUTE_THREADS, a.E * sizeof(int), st>>>(logits, a, renorm);
    const wq_status e = check_launch("wq_moe_route");
    if (e != WQ_OK) return e;
    route_place_kernel<<<blocks, ROUTE_THREADS, (7 * a.E + 1) * sizeof(int), st>>>(a);
    return check_launch("wq_moe_route");
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
    if (T <= wq::CHUNK || E <= 0) return 0;
    const int per = wq::tokens_per_block(T);
    return (size_t)((T + per - 1) / per) * (size_t)E * sizeof(int);
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
    WQ_REQUIRE((long long)T * top_k <= INT_MAX, WQ_ERR_UNSUPPORTED, "wq_moe_route: T * top_k must be below 2^31");
    if (wq_moe_route_workspace_bytes(T, E)) WQ_REQUIRE_PTR(workspace, "workspace");
    const RouteArgs a{T, E, top_k, tokens_per_block(T), ids, weights, offsets, rows, slots,
                      static_cast<int *>(workspace)};
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
    cudaStream_t st = as_stream(stream);
    if (dtype == WQ_BF16) return combine_dispatch<true>(y, R, weights, slots, T, top_k, N, out, st);
    return combine_dispatch<false>(y, R, weights, slots, T, top_k, N, out, st);
}
