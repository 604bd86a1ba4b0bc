// kv_cache.cu -- the NVFP4 key/value cache of a generation step: page and slot maps from the requests' lengths,
// the write of new keys and values, and the reading back of cached ones as BF16.
//
// 4-bit RL pages: rollout engines run on NVFP4 (Miles page), and a key/value cache in few bits has scales that are
// calibrated ahead (NeMo RL FP8 page, "FP8 KV cache"); here the second-level scale S is one FP32 per kv head.
#include "mx_internal.h"
#include "mx_kv.cuh"
#include "mx_chain.cuh"

namespace mxk {

namespace {

// ------------------------------------------------------------------------------------------------
// Page and slot maps.
//
// For request r with L_r cached and N_r new tokens and pages of P tokens: had_r = ceil(L_r / P), have_r =
// max(had_r, min(ceil((L_r + N_r) / P), W)), W the table's width.  The new pages, in request order, pop the free stack from
// its top: new page k is free[F - 1 - k], or -1 once the stack is empty.  New token t of request r (t counted
// over all requests) sits at position L_r + t - start_r in page table[r][position / P].
//
// Two exclusive sums over the requests (tokens and pages) and then independent look-ups: a few kilobytes, bound by
// latency (3.2 us for 64 requests of one token).  Every CTA of the one cluster sums all requests for itself (R / 1024 steps a
// thread) rather than wait for another launch; the outputs are shared out afterwards, each thread's look-ups side by side.
// One cluster of 8 CTAs, so that the tokens without a slot are counted in its shared memory, is also what a large step waits
// for: 8.6 us for 500 requests with 32 thousand tokens, four thousand look-ups a CTA of nine dependent steps each.
// ------------------------------------------------------------------------------------------------
constexpr int SLOT_THREADS = 1024;

struct SlotArgs {
    const int32_t* seq_lens;
    const int32_t* new_lens;
    int R;
    uint32_t page;
    DivU32 dv_page;
    int32_t* table;
    int64_t width, stride;
    const int32_t* free_pages;
    int64_t free_capacity;
    const int32_t* free_count;
    int32_t *q_start, *total_lens, *slots, *positions;
    int64_t max_tokens;
    int32_t *free_left, *unplaced;
};

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// For U values x: the largest i in [0, n) with v[i] <= x (v[0] = 0, v non-decreasing), the searches side by side.
template <int U>
__device__ __forceinline__ void last_not_above(const int* v, int n, const int (&x)[U], int (&at)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) at[u] = 0;
    for (int span = n > 1 ? 1 << (31 - __clz(n - 1)) : 0; span > 0; span >>= 1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int next = at[u] + span;
            if (next < n && v[next] <= x[u]) at[u] = next;
        }
    }
}

__global__ void __launch_bounds__(SLOT_THREADS) kv_slots_kernel(const SlotArgs a) {
    extern __shared__ int sm[];
    int* s_start = sm;                         // [R + 1] first new token of each request
    int* s_pages = s_start + a.R + 1;          // [R + 1] first new page of each request
    int* s_seq = s_pages + a.R + 1;            // [R] cached tokens
    __shared__ int2 s_warp[32];
    __shared__ int s_placed[32];
    __shared__ int s_total_placed;
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    const int per = (a.R + SLOT_THREADS - 1) / SLOT_THREADS, r0 = tid * per;
    const uint32_t P = a.page;
    chain_begin();
    const int64_t n_free = max64(0, min64(load_global(a.free_count), a.free_capacity));

    auto meet = [&]() {                        // of the cluster, or of the one CTA
        if (cluster_size() > 1) cluster_sync();
        else __syncthreads();
    };
    int2 sum = make_int2(0, 0);
    for (int r = r0; r < min(a.R, r0 + per); ++r) {
        const int seq = max(0, a.seq_lens[r]), fresh = max(0, a.new_lens[r]);
        const uint32_t had = divu32((uint32_t)seq + P - 1, a.dv_page), want = divu32((uint32_t)seq + (uint32_t)fresh + P - 1, a.dv_page);
        const int pages = (int)max64(0, min64(want, a.width) - had);
        s_seq[r] = seq;
        s_start[r] = fresh;                    // for the moment
        s_pages[r] = pages;
        sum.x += fresh;
        sum.y += pages;
    }
    int2 incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl.x, o), y = __shfl_up_sync(0xFFFFFFFFu, incl.y, o);
        if (lane >= o) {
            incl.x += x;
            incl.y += y;
        }
    }
    if (lane == 31) s_warp[wid] = incl;
    __syncthreads();
    // the warps' sums before this one's
    int2 before = lane < wid ? s_warp[lane] : make_int2(0, 0);
    before.x = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)before.x);
    before.y = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)before.y);
    int2 run = make_int2(before.x + incl.x - sum.x, before.y + incl.y - sum.y);
    for (int r = r0; r < min(a.R, r0 + per); ++r) {
        const int fresh = s_start[r], pages = s_pages[r];
        s_start[r] = run.x;
        s_pages[r] = run.y;
        run.x += fresh;
        run.y += pages;
        if (r == a.R - 1) {
            s_start[a.R] = run.x;
            s_pages[a.R] = run.y;
        }
    }
    // every read of seq_lens and free_count is done before any CTA writes total_lens or free_left, which
    // may be the same arrays
    meet();

    const int nthr = SLOT_THREADS * (int)cluster_size(), me = (int)cluster_rank() * SLOT_THREADS + tid;
    const int tokens = s_start[a.R], fresh_pages = s_pages[a.R];
    for (int r = me; r <= a.R; r += nthr) {
        a.q_start[r] = s_start[r];
        if (r < a.R) a.total_lens[r] = s_seq[r] + (s_start[r + 1] - s_start[r]);
    }
    auto had_of = [&](int r) { return divu32((uint32_t)s_seq[r] + P - 1, a.dv_page); };
    for (int k = me; k < fresh_pages; k += nthr) {
        const int x[1] = {k};
        int r[1];
        last_not_above(s_pages, a.R, x, r);
        const int64_t col = (int64_t)had_of(r[0]) + (k - s_pages[r[0]]);
        if (col < a.width) a.table[r[0] * a.stride + col] = k < n_free ? load_global(a.free_pages + (n_free - 1 - k)) : -1;
    }
    int placed = 0;
    constexpr int U = 4;                       // tokens of a thread looked up side by side
    for (int64_t t0 = me; t0 < a.max_tokens; t0 += (int64_t)U * nthr) {
        int x[U], r[U], pos[U], page[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = (int)min64(t0 + (int64_t)u * nthr, INT32_MAX);
        if (x[0] < tokens) last_not_above(s_start, a.R, x, r);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            pos[u] = page[u] = -1;
            if (x[u] < tokens) {
                pos[u] = s_seq[r[u]] + (x[u] - s_start[r[u]]);
                const uint32_t col = divu32((uint32_t)pos[u], a.dv_page), had = had_of(r[u]);
                if (pos[u] >= 0 && col < a.width) {
                    if (col < had) {
                        page[u] = a.table[r[u] * a.stride + col];       // an older page: not written by this call
                    } else {
                        const int64_t k = s_pages[r[u]] + (int64_t)(col - had);
                        if (k < n_free) page[u] = load_global(a.free_pages + (n_free - 1 - k));
                    }
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t t = t0 + (int64_t)u * nthr;
            if (t >= a.max_tokens) break;
            const uint32_t off = (uint32_t)pos[u] - divu32((uint32_t)pos[u], a.dv_page) * P;
            const int64_t s = (int64_t)page[u] * P + off;
            const int slot = page[u] >= 0 && s <= INT32_MAX ? (int)s : -1;
            placed += slot >= 0;
            a.slots[t] = slot;
            a.positions[t] = pos[u];
        }
    }
    placed = __reduce_add_sync(0xFFFFFFFFu, placed);
    if (lane == 0) s_placed[wid] = placed;
    __syncthreads();
    if (wid == 0) {
        placed = __reduce_add_sync(0xFFFFFFFFu, s_placed[lane]);
        if (lane == 0) s_total_placed = placed;
    }
    meet();                                                             // every CTA's count is in its shared memory
    if (me == 0) {
        int all = 0;
        const uint32_t mine = (uint32_t)__cvta_generic_to_shared(&s_total_placed);
        for (uint32_t c = 0; c < cluster_size(); ++c) {
            uint32_t there;
            int v;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(c));
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(there) : "memory");
            all += v;
        }
        *a.unplaced = tokens - all;
        *a.free_left = (int)max64(0, n_free - fresh_pages);
    }
    meet();                                                             // nobody leaves while CTA 0 reads its count
}

// ------------------------------------------------------------------------------------------------
// Write and read of cached tokens: one thread per 16-element block, as the quantizers and dequantizers of
// the framework, with the same arithmetic and S per head.  Both are bound by memory (2.5625 bytes a value).
// A warp holds the D / 16 blocks of neighbouring tokens of one head, so that the single bytes of the V scales, whose
// neighbours in memory are other tokens' of the same block, leave it merged by sectors (4 tokens a sector for D = 128
// instead of one).  Grid: tokens, heads; no index is divided, and K and V of a block share a thread's indexes.  16381
// tokens of 8 heads, D = 128: 30.0 us for both, 84 % of the measured copy rate (41.6 with one block a thread and divided
// indexes); the write is bound by issue (70 % of the slots), the reading by HBM.
// ------------------------------------------------------------------------------------------------

// The record of (slot, head), or null when the slot is outside the cache.
template <typename T>
__device__ __forceinline__ T* record_of(T* cache, int64_t slot, int h, const KvShape& c, int& token) {
    if (slot < 0 || slot >= c.pages * c.page) return nullptr;
    const uint32_t s = (uint32_t)slot, page = divu32(s, c.dv_page), off = s - page * (uint32_t)c.page;
    token = (int)(off & (KV_GROUP - 1));
    const int64_t rec = ((int64_t)page * c.heads + h) * (c.page / KV_GROUP) + off / KV_GROUP;
    return cache + rec * kv_record_bytes(c.dim);
}

// A 16-block of BF16 as codes and block scale byte under S.
__device__ __forceinline__ uint2 quantize_block(const uint4& x0, const uint4& x1, float S, uint32_t& bs) {
    const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
    uint32_t m2 = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m2 = absmax_bf16x2_int(m2, w[j]);     // integer maximum: a NaN is the largest
    bs = nvfp4_block_scale_fast(__uint_as_float(fold_halves(m2) << 16), S, nvfp4_fast_rs(S));
    const float r = nvfp4_block_recip(bs, S);
    uint2 out;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __fmul_rn(bf16_lo(w[j]), r);
        f[2 * j + 1] = __fmul_rn(bf16_hi(w[j]), r);
    }
    out.x = cvt_e2m1x8(f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = __fmul_rn(bf16_lo(w[4 + j]), r);
        f[2 * j + 1] = __fmul_rn(bf16_hi(w[4 + j]), r);
    }
    out.y = cvt_e2m1x8(f);
    if (r == 0.0f) {                                                  // zeros for infinities too (infinity * 0)
        out.x &= 0x88888888u;
        out.y &= 0x88888888u;
    }
    return out;
}

// The BF16 values of a 16-block.
__device__ __forceinline__ void dequantize_block(uint2 q, uint32_t bs, float S, uint4& y0, uint4& y1) {
    const float f = e4m3_to_f32(bs);
    const uint32_t w[2] = {q.x, q.y};
    uint32_t out[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t p = e2m1x2_to_f16x2((w[j >> 2] >> (8 * (j & 3))) & 0xFFu);
        // the product with the block scale is exact, so the value is rounded by S and once to BF16
        const float v0 = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(p & 0xFFFFu))), f);
        const float v1 = __fmul_rn(__half2float(__ushort_as_half((unsigned short)(p >> 16))), f);
        out[j] = pack_bf16x2(__fmul_rn(v0, S), __fmul_rn(v1, S));
    }
    y0 = make_uint4(out[0], out[1], out[2], out[3]);
    y1 = make_uint4(out[4], out[5], out[6], out[7]);
}

template <int D>
__global__ void __launch_bounds__(256)
kv_append_kernel(const uint16_t* k, const uint16_t* v, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                 const int32_t* slots, int64_t T, const float* s_k, const float* s_v, uint8_t* cache, KvShape c) {
    chain_begin();
    constexpr int nb = D / 16;
    const int64_t t = (int64_t)blockIdx.x * (256 / nb) + threadIdx.x / nb;
    const int h = blockIdx.y, b = threadIdx.x % nb;
    if (t >= T) return;
    const uint4* from_k = reinterpret_cast<const uint4*>(k + t * k_token + h * k_head + b * 16);
    const uint4* from_v = reinterpret_cast<const uint4*>(v + t * v_token + h * v_head + b * 16);
    const uint4 k0 = load_global(from_k), k1 = load_global(from_k + 1), v0 = load_global(from_v), v1 = load_global(from_v + 1);
    int token;
    uint8_t* rec = record_of(cache, load_global(slots + t), h, c, token);
    if (!rec) return;
    uint32_t bs;
    *reinterpret_cast<uint2*>(rec + token * (D / 2) + b * 8) = quantize_block(k0, k1, load_global(s_k + h), bs);
    rec[kv_k_scales(D) + token * nb + b] = (uint8_t)bs;
    *reinterpret_cast<uint2*>(rec + kv_v_codes(D) + token * (D / 2) + b * 8) = quantize_block(v0, v1, load_global(s_v + h), bs);
    rec[kv_v_scales(D) + b * 16 + kv_token_of_row(token)] = (uint8_t)bs;
}

template <int D>
__global__ void __launch_bounds__(256)
kv_gather_kernel(const uint8_t* cache, const int32_t* slots, int64_t T, const float* s_k, const float* s_v, uint16_t* k,
                 uint16_t* v, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, KvShape c) {
    chain_begin();
    constexpr int nb = D / 16;
    const int64_t t = (int64_t)blockIdx.x * (256 / nb) + threadIdx.x / nb;
    const int h = blockIdx.y, b = threadIdx.x % nb;
    if (t >= T) return;
    uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
    int token;
    const uint8_t* rec = record_of(cache, load_global(slots + t), h, c, token);
    if (rec) {
        const uint2 kq = load_global(reinterpret_cast<const uint2*>(rec + token * (D / 2) + b * 8));
        const uint2 vq = load_global(reinterpret_cast<const uint2*>(rec + kv_v_codes(D) + token * (D / 2) + b * 8));
        const uint32_t ks = load_global(rec + kv_k_scales(D) + token * nb + b);
        const uint32_t vs = load_global(rec + kv_v_scales(D) + b * 16 + kv_token_of_row(token));
        dequantize_block(kq, ks, load_global(s_k + h), k0, k1);
        dequantize_block(vq, vs, load_global(s_v + h), v0, v1);
    }
    uint4* to_k = reinterpret_cast<uint4*>(k + t * k_token + h * k_head + b * 16);
    uint4* to_v = reinterpret_cast<uint4*>(v + t * v_token + h * v_head + b * 16);
    stcs_32b(to_k, k0, k1);
    stcs_32b(to_v, v0, v1);
}

}  // namespace

cudaError_t launch_kv_slots(const int32_t* seq_lens, const int32_t* new_lens, int64_t R, int64_t page, int32_t* table,
                            int64_t width, int64_t stride, const int32_t* free_pages, int64_t free_capacity,
                            const int32_t* free_count, int32_t* q_start, int32_t* total_lens, int32_t* slots,
                            int32_t* positions, int64_t max_tokens, int32_t* free_left, int32_t* unplaced,
                            cudaStream_t stream) {
    static PerDevice pd;
    int unused = 0;
    cudaError_t e = per_device_once(pd, unused, [](int&) {
        return cudaFuncSetAttribute(kv_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (3 * (int)KV_MAX_REQUESTS + 2) * (int)sizeof(int));
    });
    if (e != cudaSuccess) return e;
    const SlotArgs a{seq_lens, new_lens, (int)R, (uint32_t)page, make_divu32((uint64_t)page), table, width, stride, free_pages, free_capacity,
                     free_count, q_start, total_lens, slots, positions, max_tokens, free_left, unplaced};
    const unsigned ctas = max_tokens > 4 * SLOT_THREADS ? 8 : 1;          // one CTA as long as it looks up once
    return launch_chained(kv_slots_kernel, dim3(ctas), SLOT_THREADS, (size_t)(3 * R + 2) * sizeof(int), ctas, stream, a);
}

cudaError_t launch_kv_append(const uint16_t* k, const uint16_t* v, int64_t k_token, int64_t k_head, int64_t v_token,
                             int64_t v_head, const int32_t* slots, int64_t T, const float* s_k, const float* s_v,
                             uint8_t* cache, const KvShape& c, cudaStream_t stream) {
    const dim3 grid((unsigned)((T + 256 / (c.dim / 16) - 1) / (256 / (c.dim / 16))), (unsigned)c.heads);
    return launch_chained(c.dim == 64 ? kv_append_kernel<64> : (c.dim == 128 ? kv_append_kernel<128> : kv_append_kernel<256>), grid, 256, 0, 0,
                          stream, k, v, k_token, k_head, v_token, v_head, slots, T, s_k, s_v, cache, c);
}

cudaError_t launch_kv_gather(const uint8_t* cache, const int32_t* slots, int64_t T, const float* s_k, const float* s_v,
                             uint16_t* k, uint16_t* v, int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head,
                             const KvShape& c, cudaStream_t stream) {
    const dim3 grid((unsigned)((T + 256 / (c.dim / 16) - 1) / (256 / (c.dim / 16))), (unsigned)c.heads);
    return launch_chained(c.dim == 64 ? kv_gather_kernel<64> : (c.dim == 128 ? kv_gather_kernel<128> : kv_gather_kernel<256>), grid, 256, 0, 0,
                          stream, cache, slots, T, s_k, s_v, k, v, k_token, k_head, v_token, v_head, c);
}

}  // namespace mxk
