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

#include <type_traits>

namespace mxk {

namespace {

// ------------------------------------------------------------------------------------------------
// Sort: a stable counting sort.  A warp finds the equal experts among its 32 choices by a match and ranks them behind its own
// count so far; the warps' counts of an expert are summed in their order, then the CTAs', then the experts'.
//
// Up to SORT_CLUSTER_MAX choices one cluster does it all in one launch, the choices in registers and the CTAs' counts exchanged
// through shared memory: a chain of a few latencies (65536 choices 7.5 us; in two launches, as below, 13).  Beyond, the choices are
// cut into chunks, a CTA each: a first kernel counts every chunk's choices of each expert, in the second each CTA adds up what the
// chunks before it hold (131080 choices of 128 experts 12.3 us, 131072 in one launch 9.5; 524288 14.9, twenty million 219).
// ------------------------------------------------------------------------------------------------
constexpr int SORT_THREADS = 1024, SORT_WARPS = SORT_THREADS / 32;
constexpr int SORT_ROUNDS = 8;                             // most choices of a thread at once
constexpr int SORT_CTAS = 16;                              // most CTAs of the cluster
constexpr int64_t SORT_CLUSTER_MAX = (int64_t)SORT_CTAS * SORT_THREADS * SORT_ROUNDS;
constexpr int SORT_TILE = SORT_THREADS * SORT_ROUNDS;
constexpr int SORT_MAX_CHUNKS = 256;

struct SortArgs {
    const int32_t* ids;
    int64_t n, chunk;                                      // choices, choices of a CTA
    int experts, chunks;
    int64_t* offsets;
    int32_t *rows, *source, *counts;
};

// A choice's expert, -1 where it has none.
__device__ __forceinline__ int expert_of(const SortArgs& a, int64_t i, int64_t last) {
    const int id = i < last ? load_global(a.ids + i) : -1;
    return id >= 0 && id < a.experts ? id : -1;
}

// Ranks the choices of a warp (ROUNDS times 32 neighbouring ones) among its own of the same expert; `mine` counts them.  The lanes
// of the same expert are those whose numbers agree in every bit, by a vote a bit (65536 choices of 128 experts: 1.8 us less than
// with __match_any_sync).
template <int ROUNDS>
__device__ __forceinline__ void rank_in_warp(const int (&id)[ROUNDS], int (&rank)[ROUNDS], uint16_t* mine, int experts) {
    const unsigned before = (1u << (threadIdx.x & 31)) - 1u;
    unsigned same[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) same[r] = __ballot_sync(0xFFFFFFFFu, id[r] >= 0);
    for (int bit = 1; bit < experts; bit <<= 1)
#pragma unroll
        for (int r = 0; r < ROUNDS; ++r) {
            const unsigned set = __ballot_sync(0xFFFFFFFFu, (id[r] & bit) != 0);
            same[r] &= (id[r] & bit) ? set : ~set;
        }
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const unsigned peers = same[r];                    // (of a choice without an expert: not used)
        const int at = __popc(peers & before), so_far = id[r] >= 0 ? mine[id[r]] : 0;
        __syncwarp();
        if (id[r] >= 0 && at == 0) mine[id[r]] = (uint16_t)(so_far + __popc(peers));
        __syncwarp();
        rank[r] = so_far + at;
    }
}

// The counts of expert g by warp become the counts of the warps before; returns their total.
__device__ __forceinline__ int sum_over_warps(uint16_t* count, int experts, int g) {
    int run = 0;
#pragma unroll 1
    for (int w0 = 0; w0 < SORT_WARPS; w0 += 8) {           // eight loads side by side
        int v[8];
#pragma unroll
        for (int w = 0; w < 8; ++w) v[w] = count[(w0 + w) * experts + g];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            count[(w0 + w) * experts + g] = (uint16_t)run;
            run += v[w];
        }
    }
    return run;
}

// Exclusive sum over the threads of a CTA, and the total.
__device__ __forceinline__ int sum_before(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        if (lane >= o) incl += x;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    const unsigned w = (unsigned)s_warp[lane];
    total = (int)__reduce_add_sync(0xFFFFFFFFu, w);
    return (int)__reduce_add_sync(0xFFFFFFFFu, lane < warp ? w : 0u) + incl - v;
}

__device__ __forceinline__ void clear_counts(uint16_t* count, int experts) {
    for (int i = threadIdx.x; i < SORT_WARPS * experts / 2; i += SORT_THREADS) reinterpret_cast<uint32_t*>(count)[i] = 0u;
}

// Words of the tables of a CTA (an even number: staged choices of 8 bytes follow).
__host__ __device__ inline int sort_table_words(int ctas, int experts) { return ((1 + ctas + SORT_WARPS / 2) * experts + 1) & ~1; }

template <int ROUNDS>
__global__ void __launch_bounds__(SORT_THREADS) moe_sort_kernel(const SortArgs a) {
    extern __shared__ int sm[];
    int* s_next = sm;                                      // [experts] next row of each expert
    int* s_total = s_next + a.experts;                     // [CTAs][experts] counts of each CTA
    __shared__ int s_warp[32];
    uint32_t me, peers;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(me));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(peers));
    uint16_t* count = reinterpret_cast<uint16_t*>(s_total + peers * a.experts);       // [warps][experts]
    int2* staged = reinterpret_cast<int2*>(sm + sort_table_words(peers, a.experts));  // [choices of the CTA] row and choice, in row order
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");             // this CTA runs
    clear_counts(count, a.experts);
    chain_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.experts;
    const int64_t first = me * a.chunk, last = min64(a.n, first + a.chunk), at = first + (warp * ROUNDS) * 32 + lane;
    int id[ROUNDS], rank[ROUNDS];
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) id[r] = expert_of(a, at + r * 32, last);
    __syncthreads();
    rank_in_warp(id, rank, count + warp * G, G);
    __syncthreads();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (tid < G) {
        const int total = sum_over_warps(count, G, tid);
        const uint32_t mine = (uint32_t)__cvta_generic_to_shared(s_total + me * G + tid);
        for (uint32_t p = 0; p < peers; ++p) {
            uint32_t there;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(mine), "r"(p));
            asm volatile("st.shared::cluster.s32 [%0], %1;" :: "r"(there), "r"(total) : "memory");
        }
    }
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    int before = 0, total = 0, placed;
    if (tid < G)
        for (uint32_t p = 0; p < peers; ++p) {
            const int v = s_total[p * G + tid];
            total += v;
            if (p < me) before += v;
        }
    const int start = sum_before(total, s_warp, placed);
    int here = 0;
    if (tid < G) {
        here = s_total[me * G + tid];
        s_next[tid] = start + before;
        if (me == 0) a.offsets[tid] = start;
    }
    if (me == 0 && tid == 0) a.offsets[G] = placed;
    // the choices of this CTA in the order of their rows, so that those of an expert, neighbours in `source`, leave together (one by
    // one, each with a sector of its own, 65536 of them took 0.7 us more)
    __syncthreads();                                       // s_warp has been read
    int staged_choices;
    const int place = sum_before(here, s_warp, staged_choices);
    if (tid < G) s_total[me * G + tid] = place;            // (read by this thread alone so far)
    __syncthreads();
#pragma unroll
    for (int r = 0; r < ROUNDS; ++r) {
        const int64_t i = at + r * 32;
        if (i >= last) continue;
        int row = -1;
        if (id[r] >= 0) {
            const int nth = count[warp * G + id[r]] + rank[r];
            row = s_next[id[r]] + nth;
            if (a.source) staged[s_total[me * G + id[r]] + nth] = make_int2(row, (int)i);
        }
        a.rows[i] = row;
    }
    if (a.source) {
        __syncthreads();
        for (int p = tid; p < staged_choices; p += SORT_THREADS) a.source[staged[p].x] = staged[p].y;
    }
    if (a.source)
        for (int64_t r = placed + (int64_t)me * SORT_THREADS + tid; r < a.n; r += (int64_t)peers * SORT_THREADS) a.source[r] = -1;
}

__global__ void __launch_bounds__(SORT_THREADS) moe_count_kernel(const SortArgs a) {
    extern __shared__ int sm[];
    for (int g = threadIdx.x; g < a.experts; g += SORT_THREADS) sm[g] = 0;
    __syncthreads();
    chain_begin();
    const int64_t first = blockIdx.x * a.chunk, last = min64(a.n, first + a.chunk);
    for (int64_t i = first + threadIdx.x; i < last; i += SORT_THREADS) {
        const int id = expert_of(a, i, last);
        if (id >= 0) atomicAdd(&sm[id], 1);
    }
    __syncthreads();
    for (int g = threadIdx.x; g < a.experts; g += SORT_THREADS) a.counts[(int64_t)blockIdx.x * a.experts + g] = sm[g];
}

__global__ void __launch_bounds__(SORT_THREADS) moe_place_kernel(const SortArgs a) {
    extern __shared__ int sm[];
    int* s_next = sm;                                      // [experts] next row of each expert
    uint16_t* count = reinterpret_cast<uint16_t*>(s_next + a.experts);                // [warps][experts]
    __shared__ int s_warp[32];
    chain_begin();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.experts;
    const int64_t first = blockIdx.x * a.chunk, last = min64(a.n, first + a.chunk);
    int total = 0, before = 0, placed;
    if (tid < G)
        for (int c = 0; c < a.chunks; ++c) {
            const int v = load_global(a.counts + (int64_t)c * G + tid);
            total += v;
            if (c < (int)blockIdx.x) before += v;
        }
    const int start = sum_before(total, s_warp, placed);
    if (tid < G) {
        s_next[tid] = start + before;
        if (blockIdx.x == 0) a.offsets[tid] = start;
    }
    if (blockIdx.x == 0 && tid == 0) a.offsets[G] = placed;
    if (a.source)
        for (int64_t r = placed + (int64_t)blockIdx.x * SORT_THREADS + tid; r < a.n; r += (int64_t)gridDim.x * SORT_THREADS) a.source[r] = -1;
    for (int64_t tile = first; tile < last; tile += SORT_TILE) {
        clear_counts(count, G);
        const int64_t at = tile + (warp * SORT_ROUNDS) * 32 + lane;
        int id[SORT_ROUNDS], rank[SORT_ROUNDS];
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) id[r] = expert_of(a, at + r * 32, last);
        __syncthreads();
        rank_in_warp(id, rank, count + warp * G, G);
        __syncthreads();
        const int here = tid < G ? sum_over_warps(count, G, tid) : 0;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < SORT_ROUNDS; ++r) {
            const int64_t i = at + r * 32;
            if (i >= last) continue;
            const int row = id[r] >= 0 ? s_next[id[r]] + count[warp * G + id[r]] + rank[r] : -1;
            a.rows[i] = row;
            if (a.source && row >= 0) a.source[row] = (int32_t)i;
        }
        __syncthreads();
        if (tid < G) s_next[tid] += here;
    }
}

// ------------------------------------------------------------------------------------------------
// Dispatch: a warp takes 1 KB of a token's row (32 bytes a lane) to its top_k rows.  For rows in few
// bits the first CTAs of the launch move the scale bytes meanwhile, by words of four scale columns: a warp a token or several
// (one look-up for the choices of all: 5166 tokens to 3 of 256 experts 9.8 to 6.6 us), the groups' tables in shared memory, and zeros
// between the groups.  Bound by HBM: 8192 tokens to 65536 rows of 2048 codes take 27 us, 22 of
// them the rows (7.0 TB/s); the rest are a million scale words, a sector of their own each, since the rows that share one
// belong to different tokens.
// ------------------------------------------------------------------------------------------------
constexpr int MOVE_WARPS = 8, MOVE_THREADS = 32 * MOVE_WARPS;
constexpr int MOVE_BYTES = 1024;
// Most CTAs for the scales, two an SM of 152 (8192 tokens: 33 us with 152, 27 with 304 to 1024; the rows alone take 22).
constexpr int MOVE_SCALE_CTAS = 304;
// With five CTAs an SM (48 registers) the scales of 869 tokens of 6528 to 7 of 8 experts take 9.4 us, with six 13.4, with four those of
// 8192 tokens 28.1 in place of 27.0.
constexpr int MOVE_PER_SM = 5;

struct MoveArgs {
    const uint8_t* x; int64_t pitch;
    uint8_t* y; int64_t y_pitch;
    int64_t tokens, row_bytes, total_rows;
    const int32_t* rows;
    int top_k;
    unsigned scale_ctas;                                   // 0: rows alone
    DivU32 dv_top_k;
    int scale_tokens;                                      // of a warp in turn, whose choices are looked up at once
    uint32_t pieces;                                       // of MOVE_BYTES in a row
    DivU32 dv_pieces;
    const uint8_t* s;
    const float* s2;
    int64_t columns;                                       // scale columns
    int G;
    const int64_t* offsets;
    uint8_t* s_out;
    float* s2_out;
};

// Zeros the grouped layout's rows behind each group's last and its tiles behind the last group, 512 bytes (128 rows of four scale
// columns) a warp and step; lane l has the rows l, l + 32, l + 64 and l + 96 of a tile side by side.
__device__ __forceinline__ void zero_between_groups(uint8_t* s, const int64_t* s_off, const int* s_ptile, int G, int nct,
                                                    int64_t tile_bound, int64_t me, int64_t warps) {
    const int lane = threadIdx.x & 31;
    for (int i = (int)me; i < G * nct; i += (int)warps) {
        const int g = i / nct, c = i - g * nct;
        const int used = (int)((s_off[g + 1] - s_off[g]) & 127);
        const int64_t tile = (int64_t)s_ptile[g + 1] - 1;
        if (used == 0 || tile < 0 || tile >= tile_bound) continue;        // full or empty (offsets out of order: nothing outside)
        uint32_t* at = reinterpret_cast<uint32_t*>(s + (tile * nct + c) * 512 + lane * 16);
        if (lane >= used) {
            *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
        } else {
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (lane + 32 * q >= used) at[q] = 0u;
        }
    }
    const int64_t filled = min64(max64(0, (int64_t)s_ptile[G]), tile_bound);
    uint4* tail = reinterpret_cast<uint4*>(s + filled * nct * 512);
    for (int64_t i = me * 32 + lane; i < (tile_bound - filled) * nct * 32; i += warps * 32) tail[i] = make_uint4(0u, 0u, 0u, 0u);
}

__device__ __forceinline__ void move_scales(const MoveArgs& a) {
    extern __shared__ int64_t s_off[];                     // [G + 1], then the tiles before each group and a scan's scratch
    int* s_ptile = reinterpret_cast<int*>(s_off + a.G + 1);
    int* s_scratch = s_ptile + a.G + 1;
    const int lane = threadIdx.x & 31;
    const int64_t me = (int64_t)blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5), warps = (int64_t)a.scale_ctas * MOVE_WARPS;
    const int64_t nct = (a.columns + 3) / 4, tile_bound = (a.total_rows + 127 * (int64_t)a.G + 127) / 128;
    const uint32_t last_mask = (a.columns & 3) ? (1u << (8 * (a.columns & 3))) - 1u : 0xFFFFFFFFu;
    // `width` lanes (a power of two) a choice, 32 / width choices side by side
    const int width = nct >= 32 ? 32 : 1 << (32 - __clz((int)nct - 1)), mine = lane & (width - 1), j0 = lane / width, js = 32 / width;
    // `n` tokens in turn, whose choices are neighbours in `rows`, a lane each: one search for all of them
    const int n = a.scale_tokens, my_token = (int)divu32((uint32_t)lane, a.dv_top_k);
    auto row_of = [&](int64_t t) { return lane < n * a.top_k && t + my_token < a.tokens ? load_global(a.rows + t * a.top_k + lane) : -1; };
    auto word_of = [&](int64_t t, int64_t c) {
        return t < a.tokens && c < nct ? load_global(reinterpret_cast<const uint32_t*>(a.s + sf_offset(t, 4 * c, nct))) : 0u;
    };
    int row = row_of(me * n);                              // on their way while the tables are made
    uint32_t word = word_of(me * n, mine), word2 = word_of(me * n, mine + 32);        // (none beyond 32 where `width` is less)
    for (int i = threadIdx.x; i <= a.G; i += MOVE_THREADS) s_off[i] = load_global(a.offsets + i);
    __syncthreads();
    scan_group_tiles(s_off, a.G, s_ptile, s_scratch);
    for (int64_t t0 = me * n; t0 < a.tokens; t0 += warps * n) {
        const int r = row;
        row = row_of(t0 + warps * n);                      // the next tokens', on their way meanwhile
        int64_t place = -1;                                // row in the grouped layout of this lane's choice
        if (r >= 0 && r < a.total_rows) {
            const int64_t p = grouped_scale_row(s_off, s_ptile, a.G, r);
            if (p >= 0 && p < tile_bound * 128) place = p;
            if (a.s2_out) a.s2_out[r] = load_global(a.s2 + t0 + my_token);
        }
        for (int i = 0; i < n && t0 + i < a.tokens; ++i) {
            const int64_t t = t0 + i;
            uint32_t w = word, w2 = word2;
            const int64_t then = i + 1 < n ? t + 1 : t0 + warps * n;
            word = word_of(then, mine);
            word2 = word_of(then, mine + 32);
            for (int64_t c = mine; c - mine < nct; c += 64) {
                if (c - mine > 0) {
                    w = word_of(t, c);
                    w2 = word_of(t, c + 32);
                }
                if (c == nct - 1) w &= last_mask;
                if (c + 32 == nct - 1) w2 &= last_mask;
                for (int j = 0; j < a.top_k; j += js) {
                    const int64_t p = __shfl_sync(0xFFFFFFFFu, place, min(31, i * a.top_k + j + j0));
                    if (j + j0 >= a.top_k || p < 0) continue;
                    uint32_t* to = reinterpret_cast<uint32_t*>(a.s_out + sf_offset(p, 4 * c, nct));
                    if (c < nct) to[0] = w;
                    if (c + 32 < nct) to[32 * 128] = w2;
                }
            }
        }
    }
    zero_between_groups(a.s_out, s_off, s_ptile, a.G, (int)nct, tile_bound, me, warps);
}

__global__ void __launch_bounds__(MOVE_THREADS, MOVE_PER_SM) moe_dispatch_kernel(const MoveArgs a) {
    chain_begin();
    if (blockIdx.x < a.scale_ctas) {
        move_scales(a);
        return;
    }
    const int lane = threadIdx.x & 31;
    const uint32_t item = (blockIdx.x - a.scale_ctas) * MOVE_WARPS + (threadIdx.x >> 5);
    const int64_t t = divu32(item, a.dv_pieces);
    if (t >= a.tokens) return;
    const int64_t b0 = (int64_t)(item - (uint32_t)t * a.pieces) * MOVE_BYTES + lane * 32, b1 = b0 + 16;
    const int row = lane < a.top_k ? load_global(a.rows + t * a.top_k + lane) : -1;
    uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
    if (b0 < a.row_bytes) v0 = load_global(reinterpret_cast<const uint4*>(a.x + t * a.pitch + b0));
    if (b1 < a.row_bytes) v1 = load_global(reinterpret_cast<const uint4*>(a.x + t * a.pitch + b1));
    for (int j = 0; j < a.top_k; ++j) {
        const int r = __shfl_sync(0xFFFFFFFFu, row, j);
        if (r < 0 || r >= a.total_rows) continue;
        if (b1 < a.row_bytes) stcs_32b(a.y + r * a.y_pitch + b0, v0, v1);
        else if (b0 < a.row_bytes) *reinterpret_cast<uint4*>(a.y + r * a.y_pitch + b0) = v0;
    }
}

// ------------------------------------------------------------------------------------------------
// Combine: a warp takes 256 elements of a token, eight rows' loads in flight; neighbouring warps take neighbouring pieces of the
// same rows (46.5 us for 8192 x 8 rows of 2048, 96 % of the measured copy rate; 51 with the pieces of eight tokens in a CTA).
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

constexpr int COMBINE_ROWS = 8;                            // most rows fetched side by side

// ROWS: top_k up to COMBINE_ROWS, so that no slots without a row are gone through; MANY: top_k is larger, several passes.
template <int ROWS, bool MANY>
__global__ void __launch_bounds__(MOVE_THREADS)
moe_combine_kernel(const uint16_t* z, int64_t ldz, int64_t total_rows, int64_t hidden, const int32_t* rows, const float* weights,
                   int64_t tokens, int top_k, const uint16_t* residual, int64_t ldr, uint16_t* y, int64_t ldy, uint32_t pieces, DivU32 dv_pieces) {
    chain_begin();
    const int lane = threadIdx.x & 31;
    const uint32_t item = blockIdx.x * MOVE_WARPS + (threadIdx.x >> 5);
    const int64_t t = divu32(item, dv_pieces);
    if (t >= tokens) return;
    const int64_t c = (int64_t)(item - (uint32_t)t * pieces) * 256 + lane * 8;
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
    for (int j0 = 0; j0 < (MANY ? top_k : ROWS); j0 += ROWS) {
        uint4 v[ROWS];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int r = !MANY || j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
            v[j] = make_uint4(0u, 0u, 0u, 0u);
            if (r >= 0 && in) v[j] = load_global(reinterpret_cast<const uint4*>(z + r * ldz + c));
        }
#pragma unroll
        for (int j = 0; j < ROWS; ++j) {
            const int r = !MANY || j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
            const float w = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
            if (r < 0) continue;
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

// A CTA a token; the products of the weights' gradient are summed per thread, by a butterfly and over the warps in order.  8192 x 8
// rows of 2048 take 84 us, the measured copy rate.
constexpr int CB_THREADS = 256;
template <int ROWS, bool MANY>
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
    for (int j0 = 0; j0 < (MANY ? top_k : ROWS); j0 += ROWS) {
        float dot[ROWS] = {};
        for (int64_t c0 = 0; c0 < hidden; c0 += (int64_t)blockDim.x * 8) {
            const int64_t c = c0 + threadIdx.x * 8;
            const bool in = c < hidden;
            uint4 v[ROWS], g = make_uint4(0u, 0u, 0u, 0u);
            if (in) g = load_global(reinterpret_cast<const uint4*>(dy + t * lddy + c));
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const int r = !MANY || j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                if (r >= 0 && in) v[j] = load_global(reinterpret_cast<const uint4*>(z + r * ldz + c));
            }
            float d[8];
            unpack8(g, d);
#pragma unroll
            for (int j = 0; j < ROWS; ++j) {
                const int r = !MANY || j0 + j < top_k ? __shfl_sync(0xFFFFFFFFu, row, j0 + j) : -1;
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
        for (int j = 0; j < ROWS; ++j) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) dot[j] += __shfl_xor_sync(0xFFFFFFFFu, dot[j], o);
            if (lane == 0 && (!MANY || j0 + j < top_k)) sm[warp][j0 + j] = dot[j];
        }
    }
    __syncthreads();
    if (warp == 0 && lane < top_k) {
        float s = sm[0][lane];
        for (int w = 1; w < warps; ++w) s += sm[w][lane];
        dweights[t * top_k + lane] = row >= 0 ? s : 0.0f;
    }
}

// Choices of a chunk: whole tiles, at most SORT_MAX_CHUNKS chunks.
int64_t sort_chunk(int64_t choices) {
    const int64_t tiles = (choices + SORT_TILE - 1) / SORT_TILE;
    return (tiles + SORT_MAX_CHUNKS - 1) / SORT_MAX_CHUNKS * SORT_TILE;
}

template <int ROUNDS>
cudaError_t sort_in_cluster(SortArgs a, cudaStream_t stream) {
    auto kernel = moe_sort_kernel<ROUNDS>;
    static PerDevice pd;
    int unused = 0;
    const cudaError_t e = per_device_once(pd, unused, [kernel](int&) {
        const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   sort_table_words(SORT_CTAS, MX_MAX_GROUPS) * 4 + ROUNDS * SORT_THREADS * 8);
        return s != cudaSuccess ? s : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    a.chunk = ROUNDS * SORT_THREADS;
    const unsigned ctas = (unsigned)((a.n + a.chunk - 1) / a.chunk);
    const size_t smem = (size_t)sort_table_words((int)ctas, a.experts) * 4 + (size_t)a.chunk * 8;
    return launch_chained(kernel, dim3(ctas), dim3(SORT_THREADS), smem, ctas, stream, a);
}

}  // namespace

size_t moe_sort_workspace_bytes(int64_t choices, int64_t experts) {
    if (choices <= SORT_CLUSTER_MAX) return 16;
    const int64_t chunk = sort_chunk(choices);
    return (size_t)((choices + chunk - 1) / chunk) * (size_t)experts * sizeof(int32_t);
}

cudaError_t launch_moe_sort(const int32_t* ids, int64_t choices, int experts, int64_t* offsets, int32_t* rows, int32_t* source,
                            void* workspace, cudaStream_t stream) {
    SortArgs a{ids, choices, 0, experts, 0, offsets, rows, source, static_cast<int32_t*>(workspace)};
    // as few choices a thread as the cluster allows: each is a step of the chain
    if (choices <= SORT_CLUSTER_MAX / 8) return sort_in_cluster<1>(a, stream);
    if (choices <= SORT_CLUSTER_MAX / 4) return sort_in_cluster<2>(a, stream);
    if (choices <= SORT_CLUSTER_MAX / 2) return sort_in_cluster<4>(a, stream);
    if (choices <= SORT_CLUSTER_MAX) return sort_in_cluster<8>(a, stream);
    static PerDevice pd;
    int unused = 0;
    cudaError_t e = per_device_once(pd, unused, [](int&) {
        return cudaFuncSetAttribute(moe_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (1 + SORT_WARPS / 2) * MX_MAX_GROUPS * (int)sizeof(int));
    });
    if (e != cudaSuccess) return e;
    a.chunk = sort_chunk(choices);
    a.chunks = (int)((choices + a.chunk - 1) / a.chunk);
    e = launch_chained(moe_count_kernel, dim3(a.chunks), dim3(SORT_THREADS), (size_t)experts * sizeof(int), 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_chained(moe_place_kernel, dim3(a.chunks), dim3(SORT_THREADS), (size_t)(1 + SORT_WARPS / 2) * experts * sizeof(int), 0, stream, a);
}

static cudaError_t move_rows(MoveArgs a, cudaStream_t stream) {
    a.pieces = (uint32_t)((a.row_bytes + MOVE_BYTES - 1) / MOVE_BYTES);
    a.dv_pieces = make_divu32(a.pieces);
    const int64_t ctas = a.scale_ctas + (a.tokens * a.pieces + MOVE_WARPS - 1) / MOVE_WARPS;
    return launch_chained(moe_dispatch_kernel, dim3((unsigned)ctas), dim3(MOVE_THREADS), a.scale_ctas ? (size_t)12 * (a.G + 1) + 128 : 0, 0,
                          stream, a);
}

cudaError_t launch_moe_dispatch(const uint16_t* x, int64_t ldx, int64_t tokens, int64_t hidden, const int32_t* rows, int top_k,
                                uint16_t* y, int64_t ldy, int64_t total_rows, cudaStream_t stream) {
    MoveArgs a{};
    a.x = reinterpret_cast<const uint8_t*>(x); a.pitch = 2 * ldx;
    a.y = reinterpret_cast<uint8_t*>(y); a.y_pitch = 2 * ldy;
    a.tokens = tokens; a.row_bytes = 2 * hidden; a.total_rows = total_rows;
    a.rows = rows; a.top_k = top_k;
    return move_rows(a, stream);
}

cudaError_t launch_moe_dispatch_quantized(bool fp4, const uint8_t* q, const uint8_t* s, const float* s2, int64_t tokens, int64_t hidden,
                                          const int32_t* rows, int top_k, int G, const int64_t* offsets, uint8_t* q_out, uint8_t* s_out,
                                          float* s2_out, int64_t total_rows, cudaStream_t stream) {
    MoveArgs a{};
    a.x = q; a.y = q_out;
    a.pitch = a.y_pitch = a.row_bytes = fp4 ? hidden / 2 : hidden;
    a.tokens = tokens; a.total_rows = total_rows;
    a.rows = rows; a.top_k = top_k;
    a.s = s; a.s2 = s2; a.columns = hidden / (fp4 ? 16 : 32);
    a.G = G; a.offsets = offsets; a.s_out = s_out; a.s2_out = s2_out;
    // a warp a token and four of the pieces between groups, up to two CTAs an SM; with more tokens each has several
    const int64_t pieces = (int64_t)G * ((a.columns + 3) / 4);
    a.scale_ctas = (unsigned)min64(MOVE_SCALE_CTAS, (max64(tokens, pieces / 4) + MOVE_WARPS - 1) / MOVE_WARPS);
    const int64_t warps = (int64_t)a.scale_ctas * MOVE_WARPS;
    a.dv_top_k = make_divu32(top_k);
    a.scale_tokens = (int)min64(max(1, 32 / top_k), (tokens + warps - 1) / warps);
    return move_rows(a, stream);
}

// f of the rows that are fetched side by side and whether there are more, as constants.
template <typename F>
static cudaError_t for_rows(int top_k, F&& f) {
    switch (top_k) {
        case 1: return f(std::integral_constant<int, 1>{}, std::false_type{});
        case 2: return f(std::integral_constant<int, 2>{}, std::false_type{});
        case 3: return f(std::integral_constant<int, 3>{}, std::false_type{});
        case 4: return f(std::integral_constant<int, 4>{}, std::false_type{});
        case 5: return f(std::integral_constant<int, 5>{}, std::false_type{});
        case 6: return f(std::integral_constant<int, 6>{}, std::false_type{});
        case 7: return f(std::integral_constant<int, 7>{}, std::false_type{});
        case 8: return f(std::integral_constant<int, 8>{}, std::false_type{});
        default: return f(std::integral_constant<int, COMBINE_ROWS>{}, std::true_type{});
    }
}

cudaError_t launch_moe_combine(const uint16_t* z, int64_t ldz, int64_t total_rows, int64_t hidden, const int32_t* rows,
                               const float* weights, int64_t tokens, int top_k, const uint16_t* residual, int64_t ldr, uint16_t* y,
                               int64_t ldy, cudaStream_t stream) {
    const uint32_t pieces = (uint32_t)((hidden + 255) / 256);
    const unsigned ctas = (unsigned)((tokens * pieces + MOVE_WARPS - 1) / MOVE_WARPS);
    return for_rows(top_k, [&](auto n, auto many) {
        return launch_chained(moe_combine_kernel<n.value, many.value>, dim3(ctas), dim3(MOVE_THREADS), 0, 0, stream, z, ldz, total_rows, hidden, rows, weights,
                              tokens, top_k, residual, ldr, y, ldy, pieces, make_divu32(pieces));
    });
}

cudaError_t launch_moe_combine_backward(const uint16_t* dy, int64_t lddy, const uint16_t* z, int64_t ldz, int64_t total_rows,
                                        int64_t hidden, const int32_t* rows, const float* weights, int64_t tokens, int top_k,
                                        uint16_t* dz, int64_t lddz, float* dweights, cudaStream_t stream) {
    const int threads = (int)min64(CB_THREADS, (hidden / 8 + 31) / 32 * 32);
    return for_rows(top_k, [&](auto n, auto many) {
        return launch_chained(moe_combine_backward_kernel<n.value, many.value>, dim3((unsigned)tokens), dim3(threads), 0, 0, stream, dy, lddy, z, ldz,
                              total_rows, hidden, rows, weights, top_k, dz, lddz, dweights);
    });
}

}  // namespace mxk
