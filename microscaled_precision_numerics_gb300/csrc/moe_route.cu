// moe_route.cu -- the router's choice of experts for each token, and the gradient of its logits.
//
//   ids = the top_k largest logits;  w = softmax over the chosen, or their entries of the softmax over all
//   dz[id_j] = w_j (dw_j - sum_i w_i dw_i)   or   dz[e] = p_e (dw_j where e = id_j, else 0, - sum_i w_i dw_i)
//
// A warp takes a token: its logits stay in registers, expert e in lane e % 32, and are read once.  A choice is a scan of the lane's
// keys and two warp reductions (the largest key, then the first place among the lanes that hold it).  Bound by the integer
// instructions of the scans: 8192 tokens, 8 of 128 experts (BF16) take 8.0 us, 8 of 512 (FP32, 17 MB) 12.7, 16 of 1024 24.7 (without
// thinning out 28 and 79, the loads of a row behind one another).
#include "../../include/mxnum.h"
#include "../../include/mxnum_layer.h"
#include "mx_internal.h"
#include "mx_chain.cuh"

namespace mxk {

namespace {

constexpr int ROUTE_WARPS = 4;

template <bool F32>
__device__ __forceinline__ float logit(const void* p, int64_t i) {
    if (F32) return load_global(static_cast<const float*>(p) + i);
    return __uint_as_float((uint32_t)load_global(static_cast<const uint16_t*>(p) + i) << 16);
}

// A row's logits, -inf beyond its end.  Every lane loads (its last one again there), so that all loads are on their way at once: behind
// branches they followed one another (8192 x 1024 took 64 us).
template <int EPL, bool F32>
__device__ __forceinline__ void load_row(const void* logits, int64_t at, int experts, float (&z)[EPL]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < EPL; ++i) z[i] = logit<F32>(logits, at + min(i * 32 + lane, experts - 1));
#pragma unroll
    for (int i = 0; i < EPL; ++i) z[i] = i * 32 + lane < experts ? z[i] : -INFINITY;
}

// Keys in the order of the logits: NaN above all, zeros of both signs alike, 0 for -inf and for what is taken already.
__device__ __forceinline__ uint32_t key_of(float z) {
    if (z != z) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(__fadd_rn(z, 0.0f));
    if (b == 0xFF800000u) return 0u;
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
    if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The top_k largest of a warp's keys, key[i] of lane l in place i * 32 + l, of equal ones the first place: number j to lane j
// (key 0: none left).
template <int N>
__device__ __forceinline__ void choose(uint32_t (&key)[N], int top_k, uint32_t& my_key, int& my_place) {
    const int lane = threadIdx.x & 31;
    my_key = 0u;
    my_place = 0;
    for (int j = 0; j < top_k; ++j) {
        uint32_t best = key[0];
        int at = lane;
#pragma unroll
        for (int i = 1; i < N; ++i)
            if (key[i] > best) {
                best = key[i];
                at = i * 32 + lane;
            }
        const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
        if (most == 0u) break;
        const int place = (int)__reduce_min_sync(0xFFFFFFFFu, best == most ? (uint32_t)at : 0xFFFFFFFFu);
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i * 32 + lane == place) key[i] = 0u;
        if (lane == j) {
            my_key = most;
            my_place = place;
        }
    }
}

constexpr int ROUTE_FEW = 64;                              // candidates that two keys a lane hold

// EPL: experts a lane.  From 256 experts on (EPL >= 8) the keys are thinned out first: the top_k-th largest of the lanes' maxima is
// a bound that top_k keys reach, and few others do; those that reach it, in the order of the experts, are the ones to choose
// from.  Should there be more than 64 (many equal logits), all are.
template <int EPL, bool F32>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
moe_route_kernel(const void* logits, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize, int32_t* ids, float* weights) {
    constexpr bool THIN = EPL >= 8;
    __shared__ uint2 s_few[THIN ? ROUTE_WARPS : 1][THIN ? ROUTE_FEW : 1];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + warp;
    if (t >= tokens) return;
    float z[EPL];
    load_row<EPL, F32>(logits, t * ldl, experts, z);
    uint32_t key[EPL], best = 0u;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
        key[i] = key_of(z[i]);
        best = max(best, key[i]);
    }
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
    const float top = value_of(most);                      // (no logit but -inf: not used)
    float all = 0.0f;
    if (!normalize) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) all += key[i] != 0u ? expf(value_of(key[i]) - top) : 0.0f;
        all = warp_add(all);
    }
    uint32_t my_key = 0u;                                  // of choice `lane`
    int my_id = 0, few = ROUTE_FEW + 1;
    if constexpr (THIN) {
        uint32_t bound = most, rest = best;
        for (int j = 0; j < top_k && bound != 0u; ++j) {
            bound = __reduce_max_sync(0xFFFFFFFFu, rest);
            if (lane == __ffs(__ballot_sync(0xFFFFFFFFu, rest == bound)) - 1) rest = 0u;
        }
        bound = max(bound, 1u);
        few = 0;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const unsigned reach = __ballot_sync(0xFFFFFFFFu, key[i] >= bound);
            const int at = few + __popc(reach & ((1u << lane) - 1u));
            if (key[i] >= bound && at < ROUTE_FEW) s_few[warp][at] = make_uint2(key[i], (uint32_t)(i * 32 + lane));
            few += __popc(reach);
        }
        __syncwarp();
        if (few <= ROUTE_FEW) {
            uint32_t two[2] = {lane < few ? s_few[warp][lane].x : 0u, lane + 32 < few ? s_few[warp][lane + 32].x : 0u};
            choose(two, top_k, my_key, my_id);
            my_id = (int)s_few[warp][my_id].y;
        }
    }
    if (few > ROUTE_FEW) choose(key, top_k, my_key, my_id);
    const float mine = my_key != 0u ? expf(value_of(my_key) - top) : 0.0f;
    const float total = normalize ? warp_add(mine) : all;
    if (lane < top_k) {
        ids[t * top_k + lane] = my_key != 0u ? my_id : -1;
        weights[t * top_k + lane] = my_key != 0u ? __fdiv_rn(mine, total) : 0.0f;
    }
}

template <int EPL, bool F32>
__global__ void __launch_bounds__(32 * ROUTE_WARPS)
moe_route_backward_kernel(const void* logits, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize, const int32_t* ids,
                          const float* dweights, void* dlogits, int64_t ldd) {
    chain_begin();
    const int lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * ROUTE_WARPS + (threadIdx.x >> 5);
    if (t >= tokens) return;
    int id = -1;
    float dw = 0.0f, z = -INFINITY;
    if (lane < top_k) {
        id = load_global(ids + t * top_k + lane);
        if (id < 0 || id >= experts) id = -1;
        else {
            dw = load_global(dweights + t * top_k + lane);
            z = logit<F32>(logits, t * ldl + id);
        }
    }
    float p[EPL];                                          // all logits, then the softmax over all, then the gradient
    if (!normalize) {
        load_row<EPL, F32>(logits, t * ldl, experts, p);
    } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i) p[i] = -INFINITY;
    }
    float top = z;
#pragma unroll
    for (int i = 0; i < EPL; ++i) top = fmaxf(top, p[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    float sum = 0.0f;
    float w = id >= 0 && (z != -INFINITY) ? expf(z - top) : 0.0f;
    if (normalize) sum = w;
    else
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            p[i] = p[i] == -INFINITY ? 0.0f : expf(p[i] - top);
            sum += p[i];
        }
    sum = warp_add(sum);                                   // a NaN passes the maximum and reaches the sum
    const bool none = sum == 0.0f;                         // nothing chosen, or nothing but -inf
    const bool is_nan = sum != sum;                        // a NaN or +inf: the softmax is NaN everywhere, where a term is 0 too
    w = none ? 0.0f : __fdiv_rn(w, sum);
    const float inner = warp_add(__fmul_rn(w, dw));
    const float share = none ? 0.0f : -__fdiv_rn(inner, sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = normalize || (p[i] == 0.0f && !is_nan) ? 0.0f : __fmul_rn(p[i], share);
    const float part = normalize ? __fmul_rn(w, __fsub_rn(dw, inner)) : __fmul_rn(w, dw);
    // what a chosen expert has besides, from all of its choices (one, unless an id is given twice); the first of them writes it
    float chosen = normalize || w == 0.0f ? 0.0f : -__fmul_rn(w, inner);
    bool mine = id >= 0;
    for (int j = 0; j < top_k; ++j) {
        const int e = __shfl_sync(0xFFFFFFFFu, id, j);
        const float d = __shfl_sync(0xFFFFFFFFu, part, j);
        if (e == id) {
            chosen += d;
            mine = mine && j >= lane;
        }
    }
    auto store = [&](int e, float v) {
        if (F32) static_cast<float*>(dlogits)[t * ldd + e] = v;
        else static_cast<uint16_t*>(dlogits)[t * ldd + e] = (uint16_t)pack_bf16x2(v, 0.0f);
    };
#pragma unroll
    for (int i = 0; i < EPL; ++i)
        if (i * 32 + lane < experts) store(i * 32 + lane, p[i]);
    __syncwarp();                                          // the row is written: the chosen ones over it
    if (mine) store(id, chosen);
}

}  // namespace

template <bool F32>
static cudaError_t route(const void* logits, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize, int32_t* ids,
                         float* weights, cudaStream_t stream) {
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3((unsigned)((tokens + ROUTE_WARPS - 1) / ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), 0, 0, stream,
                              logits, ldl, tokens, experts, top_k, normalize, ids, weights);
    };
    if (experts <= 64) return go(moe_route_kernel<2, F32>);
    if (experts <= 128) return go(moe_route_kernel<4, F32>);
    if (experts <= 256) return go(moe_route_kernel<8, F32>);
    if (experts <= 512) return go(moe_route_kernel<16, F32>);
    return go(moe_route_kernel<32, F32>);
}

template <bool F32>
static cudaError_t route_backward(const void* logits, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize,
                                  const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t stream) {
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3((unsigned)((tokens + ROUTE_WARPS - 1) / ROUTE_WARPS)), dim3(32 * ROUTE_WARPS), 0, 0, stream,
                              logits, ldl, tokens, experts, top_k, normalize, ids, dweights, dlogits, ldd);
    };
    if (experts <= 64) return go(moe_route_backward_kernel<2, F32>);
    if (experts <= 128) return go(moe_route_backward_kernel<4, F32>);
    if (experts <= 256) return go(moe_route_backward_kernel<8, F32>);
    if (experts <= 512) return go(moe_route_backward_kernel<16, F32>);
    return go(moe_route_backward_kernel<32, F32>);
}

cudaError_t launch_moe_route(const void* logits, bool f32, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize,
                             int32_t* ids, float* weights, cudaStream_t stream) {
    return f32 ? route<true>(logits, ldl, tokens, experts, top_k, normalize, ids, weights, stream)
               : route<false>(logits, ldl, tokens, experts, top_k, normalize, ids, weights, stream);
}

cudaError_t launch_moe_route_backward(const void* logits, bool f32, int64_t ldl, int64_t tokens, int experts, int top_k, int normalize,
                                      const int32_t* ids, const float* dweights, void* dlogits, int64_t ldd, cudaStream_t stream) {
    return f32 ? route_backward<true>(logits, ldl, tokens, experts, top_k, normalize, ids, dweights, dlogits, ldd, stream)
               : route_backward<false>(logits, ldl, tokens, experts, top_k, normalize, ids, dweights, dlogits, ldd, stream);
}

}  // namespace mxk
