// moe_rows.cu -- tokens sorted by expert, their rows taken there (BF16, or quantized already) and brought back with weights,
// and the gradients.
//
// A choice is one (token, expert) pair, number t * top_k + j; its row is its place in the order by expert, ties by number.
// Rows move by token: a token's row is read once and written to (or added up from) its top_k places, so dispatch reads each
// input once and combine writes each output once.  All are bound by memory; the sums follow j, not the order of arrival, so
// the results do not vary.
#include "../../include/mxnum.h"
#include "../../include/mxnum_layer.h"
#include "mx_internal.h"
#include "mx_chain.cuh"

namespace mxk {

namespace {

// ------------------------------------------------------------------------------------------------
// Sort: a stable counting sort.  The choices are cut into chunks, a CTA each.  A first kernel counts every chunk's choices of
// each expert; in the second each CTA adds up what the chunks before it hold, and places its own tile by tile: a warp finds
// the equal experts among its 32 choices by a match and ranks them behind its own count so far.
// ------------------------------------------------------------------------------------------------
constexpr int SORT_THREADS = 512, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ROUNDS = 8;                             // choices of a thread in a tile
constexpr int SORT_TILE = SORT_THREADS * SORT_ROUNDS;
constexpr int SORT_MAX_CHUNKS = 256;

struct SortArgs {
    const int32_t* ids;
    int64_t n, chunk;
    int experts, chunks;
    int64_t* offsets;
    int32_t *rows, *source, *counts;
};

__global__ void __launch_bounds__(SORT_THREADS) moe_count_kernel(const SortArgs a) {
    extern __shared__ int hist[];
    for (int g = threadIdx.x; g < a.experts; g += SORT_THREADS) hist[g] = 0;
    __syncthreads();
    chain_begin();
    const int64_t first = blockIdx.x * a.chunk, last = min64(a.n, first + a.chunk);
    for (int64_t i = first + threadIdx.x; i < last; i += SORT_THREADS) {
        const int id = load_global(a.ids + i);
        if (id >= 0 && id < a.experts) atomicAdd(&hist[id], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.experts; g += SORT_THREADS) a.counts[(int64_t)blockIdx.x * a.experts + g] = hist[g];
}

__global__ void __launch_bounds__(SORT_THREADS) moe_place_kernel(const SortArgs a) {
    extern __shared__ int sm[];
    int* s_next = sm;                                      // [experts] next row of each expert
    int* s_count = s_next + a.experts;                     // [warps][experts]
    __shared__ int s_warp[SORT_WARPS];
    chain_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.experts;
    const int64_t first = blockIdx.x * a.chunk, last = min64(a.n, first + a.chunk);
    if (a.chunks == 1) {                                   // no counts: made here
        for (int g = tid; g < G; g += SORT_THREADS) s_next[g] = 0;
        __syncthreads();
        for (int64_t i = first + tid; i < last; i += SORT_THREADS) {
            const int id = load_global(a.ids + i);
            if (id >= 0 && id < G) atomicAdd(&s_next[id], 1);
        }
        __syncthreads();
    }
    // exclusive sum of the experts' totals; a thread owns `per` neighbouring experts (at most two)
    const int per = (G + SORT_THREADS - 1) / SORT_THREADS;
    int total[2] = {0, 0}, before[2] = {0, 0}, sum = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = tid * per + k;
        if (k < per && g < G) {
            if (a.chunks == 1) total[k] = s_next[g];
            else
                for (int c = 0; c < a.chunks; ++c) {
                    const int v = load_global(a.counts + (int64_t)c * G + g);
                    total[k] += v;
                    if (c < (int)blockIdx.x) before[k] += v;
                }
            sum += total[k];
        }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += v;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const int ahead = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)(lane < warp ? s_warp[lane] : 0));
    const int placed = (int)__reduce_add_sync(0xFFFFFFFFu, (unsigned)(lane < SORT_WARPS ? s_warp[lane] : 0));
    int run = ahead + incl - sum;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int g = tid * per + k;
        if (k < per && g < G) {
            if (blockIdx.x == 0) a.offsets[g] = run;
            s_next[g] = run + before[k];
            run += total[k];
        }
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[G] = placed;
    if (a.source)
        for (int64_t r = placed + (int64_t)blockIdx.x * SORT_THREADS + tid; r < a.n; r += (int64_t)gridDim.x * SORT_THREADS) a.source[r] = -1;

    for (int64_t tile = first; tile < last; tile += SORT_TILE) {
        for (int i = tid; i < SORT_WARPS * G; i += SORT_THREADS) s_count[i] = 0;
        __syncthreads();
        int* mine = s_count + warp * G;
        int id[SORT_ROUNDS], rank[SORT_ROUNDS];
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) {
            const int64_t i = tile + (warp * SORT_ROUNDS + r) * 32 + lane;
            id[r] = i < last ? load_global(a.ids + i) : -1;
            if (id[r] >= G) id[r] = -1;
            id[r] = max(id[r], -1);
        }
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) {
            const unsigned peers = __match_any_sync(0xFFFFFFFFu, id[r]);
            const int at = __popc(peers & ((1u << lane) - 1u));
            const int so_far = id[r] >= 0 ? mine[id[r]] : 0;
            __syncwarp();
            if (id[r] >= 0 && at == 0) mine[id[r]] = so_far + __popc(peers);
            __syncwarp();
            rank[r] = so_far + at;
        }
        __syncthreads();
        for (int g = tid; g < G; g += SORT_THREADS) {      // counts to first rows of each warp
            int next = s_next[g];
            for (int w = 0; w < SORT_WARPS; ++w) {
                const int v = s_count[w * G + g];
                s_count[w * G + g] = next;
                next += v;
            }
            s_next[g] = next;
        }
        __syncthreads();
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) {
            const int64_t i = tile + (warp * SORT_ROUNDS + r) * 32 + lane;
            if (i >= last) continue;
            const int row = id[r] >= 0 ? mine[id[r]] + rank[r] : -1;
            a.rows[i] = row;
            if (a.source && row >= 0) a.source[row] = (int32_t)i;
        }
        __syncthreads();
    }
}

// ------------------------------------------------------------------------------------------------
// Dispatch: a warp takes 1 KB of a token's row (32 bytes a lane in two coalesced halves) to its top_k rows.
// ------------------------------------------------------------------------------------------------
constexpr int MOVE_TOKENS = 8;                             // tokens (warps) of a CTA
constexpr int MOVE_BYTES = 1024;

__global__ void __launch_bounds__(32 * MOVE_TOKENS)
moe_dispatch_kernel(const uint8_t* x, int64_t pitch, int64_t tokens, int64_t row_bytes, const int32_t* rows, int top_k, uint8_t* y,
                    int64_t y_pitch, int64_t total_rows) {
    chain_begin();
    const int lane = threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * MOVE_TOKENS + threadIdx.y;
    if (t >= tokens) return;
    const int64_t b0 = (int64_t)blockIdx.y * MOVE_BYTES + lane * 16, b1 = b0 + 512;
    const int row = lane < top_k ? load_global(rows + t * top_k + lane) : -1;
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
    if (b0 < row_bytes) v0 = load_global(reinterpret_cast<const uint4*>(x + t * pitch + b0));
    if (b1 < row_bytes) v1 = load_global(reinterpret_cast<const uint4*>(x + t * pitch + b1));
    for (int j = 0; j < top_k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, j);
        if (r < 0 || r >= total_rows) continue;
        if (b0 < row_bytes) *reinterpret_cast<uint4*>(y + r * y_pitch + b0) = v0;
        if (b1 < row_bytes) *reinterpret_cast<uint4*>(y + r * y_pitch + b1) = v1;
    }
}

struct ScaleArgs {
    const uint8_t* s;
    const float* s2;
    int64_t tokens, columns;                               // scale columns
    const int32_t* rows;
    int top_k, G;
    const int64_t* offsets;
    uint8_t* s_out;
    float* s2_out;
    int64_t total_rows;
};

// The scale bytes of the dispatched rows, by 4-byte words (four scale columns of a row), a warp a token.
__global__ void __launch_bounds__(256) moe_dispatch_scales_kernel(const ScaleArgs a) {
    extern __shared__ int64_t s_off[];                     // [G + 1], then the tiles before each group and a scan's scratch
    int* s_ptile = reinterpret_cast<int*>(s_off + a.G + 1);
    int* s_scratch = s_ptile + a.G + 1;
    chain_begin();
    for (int i = threadIdx.x; i <= a.G; i += blockDim.x) s_off[i] = load_global(a.offsets + i);
    __syncthreads();
    scan_group_tiles(s_off, a.G, s_ptile, s_scratch);
    const int lane = threadIdx.x & 31;
    const int64_t me = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * 8;
    const int64_t nct = (a.columns + 3) / 4, tile_bound = (a.total_rows + 127 * (int64_t)a.G + 127) / 128;
    const uint32_t last_mask = (a.columns & 3) ? (1u << (8 * (a.columns & 3))) - 1u : 0xFFFFFFFFu;
    for (int64_t t = me; t < a.tokens; t += warps) {
        int64_t place = -1;                                // row in the grouped layout of choice `lane`
        if (lane < a.top_k) {
            const int r = load_global(a.rows + t * a.top_k + lane);
            if (r >= 0 && r < a.total_rows) {
                const int64_t p = grouped_scale_row(s_off, s_ptile, a.G, r);
                if (p >= 0 && p < tile_bound * 128) place = p;
                if (a.s2_out) a.s2_out[r] = load_global(a.s2 + t);
            }
        }
        for (int64_t c = lane; c < ((nct + 31) & ~int64_t(31)); c += 32) {
            uint32_t word = 0u;
            if (c < nct) word = load_global(reinterpret_cast<const uint32_t*>(a.s + sf_offset(t, 4 * c, nct)));
            if (c == nct - 1) word &= last_mask;
            for (int j = 0; j < a.top_k; ++j) {
                const int64_t p = __shfl_sync(0xFFFFFFFFu, place, j);
                if (c < nct && p >= 0) *reinterpret_cast<uint32_t*>(a.s_out + sf_offset(p, 4 * c, nct)) = word;
            }
        }
    }
    zero_grouped_padding(a.s_out, s_off, s_ptile, a.G, nct, tile_bound, me, warps);
}

// ------------------------------------------------------------------------------------------------
// Combine: a warp takes 256 elements of a token, eight rows' loads in flight.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

constexpr int COMBINE_ROWS = 8;                            // rows fetched side by side

__global__ void __launch_bounds__(32 * MOVE_TOKENS)
moe_combine_kernel(const uint16_t* z, int64_t ldz, int64_t total_rows, int64_t hidden, const int32_t* rows, const float* weights,
                   int64_t tokens, int top_k, const uint16_t* residual, int64_t ldr, uint16_t* y, int64_t ldy) {
    chain_begin();
    const int lane = threadIdx.x;
    const int64_t t = (int64_t)blockIdx.x * MOVE_TOKENS + threadIdx.y;
    if (t >= tokens) return;
    const int64_t c = (int64_t)blockIdx.y * 256 + lane * 8;
    const bool in = c < hidden;
    int row = -1;
    float weight = 0.0f;
    if (lane < top_k) {
        row = load_global(rows + t * top_k + lane);
        if (row >= total_rows) row = -1;
        weight = weights ? load_global(weights + t * top_k + lane) : 1.0f;
    }
    uint4 res = make_uint4(0u, 0u, 0u, 0u);
    if (residual && in) res = load_global(reinterpret_cast<const uint4*>(residual + t * ldr + c));
    float acc[8] = {};
    for (int j0 = 0; j0 < top_k; j0 += COMBINE_ROWS) {
        uint4 v[COMBINE_ROWS];
#pragma unroll
        for (int j = 0; j < COMBINE_ROWS; ++j) {
            const int r = j0 + j < 32 ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (r >= 0 && in) v[j] = load_global(reinterpret_cast<const uint4*>(z + r * ldz + c));
        }
#pragma unroll
        for (int j = 0; j < COMBINE_ROWS; ++j) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, (j0 + j) & 31);
            const float w = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
            if (r < 0 || j0 + j >= top_k) continue;
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = __fmaf_rn(w, f[i], acc[i]);
        }
    }
    if (!in) return;
    if (residual) {
        float f[8];
        unpack8(res, f);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] = __fadd_rn(acc[i], f[i]);
    }
    *reinterpret_cast<uint4*>(y + t * ldy + c) = pack8(acc);
}

// A CTA a token; the products of the weights' gradient are summed per thread, by a butterfly and over the warps in order.
constexpr int CB_THREADS = 256;
__global__ void __launch_bounds__(CB_THREADS)
moe_combine_backward_kernel(const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldz, int64_t total_rows, int64_t hidden,
                            const int32_t* rows, const float* weights, int top_k, uint16_t* dz, int64_t lddz, float* dweights) {
    __shared__ float sm[CB_THREADS / 32][MX_MOE_MAX_TOP_K];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int64_t t = blockIdx.x;
    int row = -1;
    float weight = 0.0f;
    if (lane < top_k) {
        row = load_global(rows + t * top_k + lane);
        if (row >= total_rows) row = -1;
        weight = load_global(weights + t * top_k + lane);
    }
    for (int j0 = 0; j0 < top_k; j0 += COMBINE_ROWS) {
        float dot[COMBINE_ROWS] = {};
        for (int64_t c0 = 0; c0 < hidden; c0 += (int64_t)blockDim.x * 8) {
            const int64_t c = c0 + threadIdx.x * 8;
            const bool in = c < hidden;
            uint4 v[COMBINE_ROWS], g = make_uint4(0u, 0u, 0u, 0u);
            if (in) g = load_global(reinterpret_cast<const uint4*>(dy + t * lddy + c));
#pragma unroll
            for (int j = 0; j < COMBINE_ROWS; ++j) {
                const int r = j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= 0 && in) v[j] = load_global(reinterpret_cast<const uint4*>(z + r * ldz + c));
            }
            float d[8];
            unpack8(g, d);
#pragma unroll
            for (int j = 0; j < COMBINE_ROWS; ++j) {
                const int r = j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
                const float w = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
                if (r < 0) continue;
                float f[8];
                unpack8(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    dot[j] = __fmaf_rn(d[i], f[i], dot[j]);
                    f[i] = __fmul_rn(w, d[i]);
                }
                if (in) *reinterpret_cast<uint4*>(dz + r * lddz + c) = pack8(f);
            }
        }
#pragma unroll
        for (int j = 0; j < COMBINE_ROWS; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (lane == 0 && j0 + j < top_k) sm[warp][j0 + j] = dot[j];
        }
    }
    __syncthreads();
    if (warp == 0 && lane < top_k) {
        float s = sm[0][lane];
        for (int w = 1; w < warps; ++w) s += sm[w][lane];
        dweights[t * top_k + lane] = row >= 0 ? s : 0.0f;
    }
}

int64_t sort_chunk(int64_t choices) {
    const int64_t tiles = (choices + SORT_TILE - 1) / SORT_TILE;
    return (tiles + SORT_MAX_CHUNKS - 1) / SORT_MAX_CHUNKS * SORT_TILE;
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t choices, int64_t experts) {
    const int64_t chunk = sort_chunk(choices);
    return (size_t)((choices + chunk - 1) / chunk) * (size_t)experts * sizeof(int32_t);
}

cudaError_t launch_moe_sort(const int32_t* ids, int64_t choices, int experts, int64_t* offsets, int32_t* rows, int32_t* source,
                            void* workspace, cudaStream_t stream) {
    static PerDevice pd;
    int unused = 0;
    cudaError_t e = per_device_once(pd, unused, [](int&) {
        return cudaFuncSetAttribute(moe_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (SORT_WARPS + 1) * MX_MAX_GROUPS * (int)sizeof(int));
    });
    if (e != cudaSuccess) return e;
    SortArgs a{ids, choices, sort_chunk(choices), experts, 0, offsets, rows, source, static_cast<int32_t*>(workspace)};
    a.chunks = (int)((choices + a.chunk - 1) / a.chunk);
    if (a.chunks > 1) {
        e = launch_chained(moe_count_kernel, dim3(a.chunks), dim3(SORT_THREADS), (size_t)experts * sizeof(int), 0, stream, a);
        if (e != cudaSuccess) return e;
    }
    return launch_chained(moe_place_kernel, dim3(a.chunks), dim3(SORT_THREADS), (size_t)(SORT_WARPS + 1) * experts * sizeof(int), 0, stream, a);
}

static cudaError_t dispatch_bytes(const uint8_t* x, int64_t pitch, int64_t tokens, int64_t row_bytes, const int32_t* rows, int top_k,
                                  uint8_t* y, int64_t y_pitch, int64_t total_rows, cudaStream_t stream) {
    const dim3 grid((unsigned)((tokens + MOVE_TOKENS - 1) / MOVE_TOKENS), (unsigned)((row_bytes + MOVE_BYTES - 1) / MOVE_BYTES));
    return launch_chained(moe_dispatch_kernel, grid, dim3(32, MOVE_TOKENS), 0, 0, stream, x, pitch, tokens, row_bytes, rows, top_k, y,
                          y_pitch, total_rows);
}

cudaError_t launch_moe_dispatch(const uint16_t* x, int64_t ldx, int64_t tokens, int64_t hidden, const int32_t* rows, int top_k,
                                uint16_t* y, int64_t ldy, int64_t total_rows, cudaStream_t stream) {
    return dispatch_bytes(reinterpret_cast<const uint8_t*>(x), 2 * ldx, tokens, 2 * hidden, rows, top_k, reinterpret_cast<uint8_t*>(y),
                          2 * ldy, total_rows, stream);
}

cudaError_t launch_moe_dispatch_quantized(bool fp4, const uint8_t* q, const uint8_t* s, const float* s2, int64_t tokens, int64_t hidden,
                                          const int32_t* rows, int top_k, int G, const int64_t* offsets, uint8_t* q_out, uint8_t* s_out,
                                          float* s2_out, int64_t total_rows, cudaStream_t stream) {
    const int64_t bytes = fp4 ? hidden / 2 : hidden;
    const cudaError_t e = dispatch_bytes(q, bytes, tokens, bytes, rows, top_k, q_out, bytes, total_rows, stream);
    if (e != cudaSuccess) return e;
    const ScaleArgs a{s, s2, tokens, hidden / (fp4 ? 16 : 32), rows, top_k, G, offsets, s_out, s2_out, total_rows};
    const unsigned grid = (unsigned)min64((tokens + 7) / 8, 2 * device_sm_count());
    return launch_chained(moe_dispatch_scales_kernel, dim3(grid), dim3(256), (size_t)12 * (G + 1) + 128, 0, stream, a);
}

cudaError_t launch_moe_combine(const uint16_t* z, int64_t ldz, int64_t total_rows, int64_t hidden, const int32_t* rows,
                               const float* weights, int64_t tokens, int top_k, const uint16_t* residual, int64_t ldr, uint16_t* y,
                               int64_t ldy, cudaStream_t stream) {
    const dim3 grid((unsigned)((tokens + MOVE_TOKENS - 1) / MOVE_TOKENS), (unsigned)((hidden + 255) / 256));
    return launch_chained(moe_combine_kernel, grid, dim3(32, MOVE_TOKENS), 0, 0, stream, z, ldz, total_rows, hidden, rows, weights, tokens,
                          top_k, residual, ldr, y, ldy);
}

cudaError_t launch_moe_combine_backward(const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldz, int64_t total_rows,
                                        int64_t hidden, const int32_t* rows, const float* weights, int64_t tokens, int top_k,
                                        uint16_t* dz, int64_t lddz, float* dweights, cudaStream_t stream) {
    const int threads = (int)min64(CB_THREADS, (hidden / 8 + 31) / 32 * 32);
    return launch_chained(moe_combine_backward_kernel, dim3((unsigned)tokens), dim3(threads), 0, 0, stream, dy, lddy, z, ldz, total_rows,
                          hidden, rows, weights, top_k, dz, lddz, dweights);
}

}  // namespace mxk
