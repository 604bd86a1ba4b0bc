// kv_attention.cu -- attention of a generation step over the NVFP4 key/value cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c q_i . k_j - m_i),  c = scale * log2(e),
//   k_j = val(code) * val(block scale) * S_k, v_j alike with S_v,
// over the cached positions j in (pos_i - window, pos_i], pos_i = L - N + i for new token i of a request with L
// cached tokens of which N are new.
//
// Bound: the cache is read once, 1.125 D bytes a token and kv head, and with G q heads to a kv head every byte meets
// G query rows: 4 G D / (1.125 D) = 3.6 G operations a byte, far below the tensor cores' balance.  The work is
// turning 4-bit codes into matrix operands fast enough: a record of 16 tokens (2304 bytes for D = 128) may cost
// one quarter of an SM at most 396 clocks at the measured copy rate, and its 64 conversions and interleavings take the ALU
// about 160 of them, its 64 FP16 multiplications and 16 matrix instructions the pipe that they share 256.
//
// Tokens are the rows (M) of both products and query rows the columns (N = 8), so eight query rows fill a fragment:
//   scores  S^T[16 tokens, 8 NQ rows] = K[16, D] Q^T:  K's codes become the A fragment of mma.m16n8k16 in registers.  A
//           thread of the quad owns D / 4 contiguous elements of a token, a run of bytes; the contraction index may
//           be permuted freely as long as Q's fragment follows.  Block scales multiply the FP16 pairs exactly (2 + 4
//           significant bits), so the only roundings of a score are FP32 sums.
//   output  O^T[D, 8 NQ] += V^T[D, 16] P:  A is V with two neighbouring tokens in a register.  The nibbles of two tokens
//           are interleaved as packed codes (4 logic instructions for 32 codes), after which one conversion gives
//           the pair (token, next token) of a dimension.  P^T comes out of S^T's accumulators by one 8x8 transpose.
// Q enters as FP16, scaled by a power of two per row so that its largest element lies in [2^15, 2^16): every BF16 value
// down to 2^-29 of it stays exact.  P enters as FP16, relative to the running maximum and times 2^7, which FP16 has room for with
// a maximum that lags by 2^8: off by 2^-11 relatively at most, against 2^-8 of the BF16 output, and below 2^-21 by 2^-32
// absolutely (without the 2^7 by 2^-25: the tail beside one strong position came out up to a third off).  The sum of P that
// divides the output is FP32 and of P before this rounding.
//
// Split: all (request, kv head, column tile) items lie end to end, each as its tiles of 32 positions and a fixed cost of
// att_item_cost tiles (look-ups, queries, the join of the warps; without it eight requests with one very short among them
// took 32 us instead of 14), and every CTA takes an equal run of that line.  A run's first and last item may be shared
// with neighbours; those leave (maximum, sum, output) pieces in the workspace and a second kernel joins them in CTA order.
// Short contexts are not split so: a CTA takes an item, or a cluster of up to 8 CTAs divides it and joins its parts through
// distributed shared memory, in one launch and without the workspace.
// The four warps of a CTA take every fourth tile of 32 positions with statistics of their own, through two stages of
// cp.async each, four for D = 64 (for D = 128 three stages, or eight warps a CTA, were slower: 75.1 and 84.3 against 73.7 us).
//
// Measured on a GB300 (device us, share of the measured copy rate): 64 requests to 8192 tokens, 32 q heads over 8 kv heads, D =
// 128: 72.9 (75 %; of the scheduler slots 58 % issue, the ALU is busy 49 %, the pipe that HMUL2 and HMMA share 51 %: bound
// by latency with the 12 warps an SM that the registers leave); one request of 131071 tokens: 34.1 (65 %; about 8 us
// of it are fixed: launch, look-ups, joins); one of 777: 6.8 (latency; 10.0 without clusters).
// The host knows the table's width and max_q, not the lengths, and lays the work out for those: under a table of 131072
// positions the request of 777 takes 8.5 (the split and its second launch), 57 to 1000 tokens 19.9 instead of 16.6; with max_q = 64
// for one new token each, 64 to 8192 take 104 instead of 73 (two column fragments, one of them empty and the other half empty).
#include "mx_internal.h"
#include "mx_kv.cuh"
#include "mx_fragment.cuh"
#include "mx_chain.cuh"

namespace mxk {

namespace {

constexpr int ATT_WARPS = 4;
constexpr int ATT_THREADS = 32 * ATT_WARPS;
constexpr int ATT_TILE = 32;                 // tokens of a warp's step: two records
// What an item costs besides its tiles, in tiles: 3.5 us, in which a CTA does 12 tiles for D = 128 and more for 64 (24 requests with
// drafts 18.9 us with 16 and 19.9 with 12; for 256 12 as well, 8 was 1 % slower).
__host__ __device__ constexpr int att_item_cost(int D) { return D == 64 ? 16 : 12; }
constexpr int ATT_MIN_SHARE = 8;             // smallest share of a CTA: two steps a warp
// Tables beyond which items have a cluster where the GPU has room, and longest tables whose items are not split over the GPU:
// more items than CTAs, or clusters of 4 and 8 (for each CTA of the cluster), or else by the share of the GPU that the items fill.
constexpr int64_t ATT_CLUSTER_TOKENS = 384, ATT_WHOLE_TOKENS = 896, ATT_WHOLE_CLUSTER_TOKENS = 512, ATT_WHOLE_FULL_TOKENS = 1920;
constexpr float ATT_SLACK = 8.0f;            // the running maximum may lag by 2^8
constexpr float ATT_P_SHIFT = 7.0f;          // P is held times 2^7: at most 2^15 in FP16

__host__ __device__ constexpr int att_stages(int D) { return D == 64 ? 4 : 2; }
// Resident CTAs per SM: by registers (O holds D / 4 * NQ of them) and by shared memory.
__host__ __device__ constexpr int att_ctas(int D, int NQ) { return D == 64 && NQ == 1 ? 4 : (D == 256 && NQ == 2 ? 2 : 3); }
__host__ __device__ constexpr int att_ring_bytes(int D) { return ATT_WARPS * att_stages(D) * 2 * kv_record_bytes(D); }
constexpr int ATT_MAX_CTAS_PER_SM = 4;
constexpr int ATT_MAX_CLUSTER = 8;

// Workspace: partial results of the work items that several CTAs share.  Each CTA has two places: 0 for an item
// that began in an earlier CTA, 1 for one that goes on in the next.
struct Piece {
    int first_cta, count;                    // CTAs first_cta (place 1), first_cta + 1 .. (place 0); count 0: not shared
    int token0, kv_head, col0, cols;         // where its query rows go
};

struct AttParams {
    KvAttentionArgs a;
    DivU32 dv_group, dv_page_groups;         // q heads per kv head; records per page
    int page_groups;
    float* part_ml;                          // [CTAs][2][8 NQ][2]
    float* part_o;                           // [CTAs][2][8 NQ][D]
    Piece* pieces;
    int n_pieces;                            // entries of pieces
    bool by_item;                            // they are numbered by item (else by CTA)
    bool whole_items;                        // an item is not shared: a CTA or cluster takes those that begin in its share, or one each
    int cluster;                             // CTAs that divide the context of such an item (1: no cluster)
};

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The same place in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t there_u32(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 load_there4(uint32_t at) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float2 load_there2(uint32_t at) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
// Words of a thread's run of codes in shared memory.
template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    if constexpr (N == 1) {
        w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * i);
            w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
        }
    }
}

// What request r asks for: tiles of its context, items (kv head x column tile) and the first tile's position.
struct Request {
    int first, count, base, len, tile0, tiles, col_tiles, per_item;       // count: rows (max_q at most); base: position of new token 0; per_item: cost of an item
    __device__ int64_t cost(int kv_heads) const { return (int64_t)per_item * col_tiles * kv_heads; }
};
template <int D, int NQ>
__device__ __forceinline__ Request request_of(const KvAttentionArgs& a, int r, bool one_each) {
    Request q;
    q.first = load_global(a.q_start + r);
    // (offsets outside [0, T] are invalid input; the clamps keep every access inside q and out all the same)
    const int fresh = q.first < 0 ? 0 : (int)max64(0, min64(load_global(a.q_start + r + 1), a.T) - q.first);
    q.count = min(fresh, a.max_q);
    q.len = max(0, load_global(a.seq_lens + r));
    q.base = q.len - fresh;                                                // whatever max_q leaves of the rows
    const int64_t lo = a.window > 0 ? max64(0, (int64_t)q.base + 1 - a.window) : 0;
    q.tile0 = (int)(lo / ATT_TILE);
    const uint32_t held = (uint32_t)min64(q.len, a.width * a.page);       // positions that the table has pages for
    q.tiles = max(1, (int)((held + ATT_TILE - 1) / ATT_TILE) - q.tile0);
    q.col_tiles = (q.count * a.group + 8 * NQ - 1) / (8 * NQ);
    q.per_item = one_each ? 1 : q.tiles + att_item_cost(D);
    return q;
}

// CLUSTER: every item belongs to a cluster, which divides its context and joins it in shared memory.
template <int D, int NQ, bool CLUSTER>
__global__ void __launch_bounds__(ATT_THREADS, att_ctas(D, NQ)) kv_attention_kernel(const __grid_constant__ AttParams p) {
    constexpr int STAGES = att_stages(D), REC = kv_record_bytes(D), STAGE_BYTES = 2 * REC;
    constexpr int KS = D / 16;               // k-steps of the scores
    constexpr int MT = D / 16;               // 16-row tiles of the output
    constexpr int KW = D / 32, VW = D / 64;  // words of a thread's run of K and V codes
    constexpr int CHUNKS = REC / 16;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t s_warp_sum[ATT_WARPS];
    __shared__ int s_warp_items[ATT_WARPS];
    __shared__ int64_t s_off;
    __shared__ int s_r, s_item;
    __shared__ float s_m[ATT_WARPS][8 * NQ], s_l[ATT_WARPS][8 * NQ];
    __shared__ float2 s_ml[8 * NQ];          // of the CTA, for its cluster

    const KvAttentionArgs& a = p.a;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;

    // ---- the CTA's share: equal runs over (request, kv head, column tile, fixed cost and context tiles)
    chain_begin();
    const bool whole_items = CLUSTER || p.whole_items, one_each = CLUSTER || (p.whole_items && p.by_item);
    const int per = (a.R + ATT_THREADS - 1) / ATT_THREADS, r0 = tid * per;
    int64_t mine = 0;
    int my_items = 0;
    for (int r = r0; r < min(a.R, r0 + per); ++r) {
        const Request q = request_of<D, NQ>(a, r, one_each);
        mine += q.cost(a.kv_heads);
        my_items += q.col_tiles * a.kv_heads;
    }
    int64_t incl = mine;
    int incl_items = my_items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xFFFFFFFFu, incl, o);
        const int y = __shfl_up_sync(0xFFFFFFFFu, incl_items, o);
        if (lane >= o) {
            incl += x;
            incl_items += y;
        }
    }
    if (lane == 31) {
        s_warp_sum[warp] = incl;
        s_warp_items[warp] = incl_items;
    }
    __syncthreads();
    int64_t total = 0, excl = incl - mine;
    int excl_items = incl_items - my_items, items = 0;
    for (int w = 0; w < ATT_WARPS; ++w) {
        items += s_warp_items[w];
        if (w < warp) {
            excl += s_warp_sum[w];
            excl_items += s_warp_items[w];
        }
        total += s_warp_sum[w];
    }
    const uint32_t rank = CLUSTER ? blockIdx.x % p.cluster : 0u, taker = CLUSTER ? blockIdx.x / p.cluster : blockIdx.x;
    const uint32_t takers = CLUSTER ? gridDim.x / p.cluster : gridDim.x;
    const int64_t share = max64(whole_items ? 1 : ATT_MIN_SHARE, (total + takers - 1) / takers);
    const int64_t begin = min64(total, taker * share), end = min64(total, begin + share);
    if (mine > 0 && begin >= excl && begin < excl + mine && begin < end) {
        int64_t at = excl;
        int r = r0, it = excl_items;
        for (;; ++r) {
            const Request q = request_of<D, NQ>(a, r, one_each);
            const int64_t w = q.cost(a.kv_heads);
            if (begin < at + w) break;
            at += w;
            it += q.col_tiles * a.kv_heads;
        }
        s_r = r;
        s_off = begin - at;
        s_item = it;
    }
    // every entry is written in every call: by the item's first CTA, or here
    if (whole_items) {
    } else if (!p.by_item) {
        if (tid == 0) p.pieces[blockIdx.x].count = 0;
    } else {
        for (int i = items + blockIdx.x * ATT_THREADS + tid; i < p.n_pieces; i += gridDim.x * ATT_THREADS) p.pieces[i].count = 0;
    }
    __syncthreads();
    if (begin >= end) return;

    int r = s_r, item0 = s_item;             // request; number of its first item
    int64_t off = s_off;                     // place inside the request
    Request rq = request_of<D, NQ>(a, r, one_each);
    uint8_t* ring = smem + warp * (STAGES * STAGE_BYTES);
    const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);

    for (int64_t at = begin; at < end;) {
        while (off >= rq.cost(a.kv_heads)) {                               // next request with work
            off -= rq.cost(a.kv_heads);
            item0 += rq.col_tiles * a.kv_heads;
            rq = request_of<D, NQ>(a, ++r, one_each);
        }
        const int per_item = rq.per_item, item = (int)(off / per_item), in_item = (int)(off - (int64_t)item * per_item);
        if (whole_items && in_item > 0) {                                // the CTA before has it
            at += per_item - in_item;
            off += per_item - in_item;
            continue;
        }
        const int run = whole_items ? per_item : (int)min64(per_item - in_item, end - at);      // of the share inside this item
        int first_tile = whole_items ? 0 : max(0, in_item - att_item_cost(D)), n_tiles = whole_items ? rq.tiles : in_item + run - att_item_cost(D) - first_tile;
        if (n_tiles <= 0) {                                                // nothing but the fixed cost: the next CTA begins the item
            at += run;
            off += run;
            continue;
        }
        if (CLUSTER) {                                                     // the CTA's part of them, which may be none
            first_tile = rq.tiles * (int)rank / p.cluster;
            n_tiles = rq.tiles * (int)(rank + 1) / p.cluster - first_tile;
        }
        const int64_t item_at = at - in_item;                              // where the item begins
        const int h = item / rq.col_tiles, col0 = (item - h * rq.col_tiles) * 8 * NQ;
        const int cols = rq.count * a.group;                               // query rows of this kv head
        const int base_pos = rq.base;

        // ---- the warp's tiles: first_tile + warp, + 4, ...; lane i looks up record i & 1 of step 16 b + i / 2
        const int steps = n_tiles > warp ? (n_tiles - warp + ATT_WARPS - 1) / ATT_WARPS : 0;
        auto look_up = [&](int b) -> int64_t {
            const int k = 16 * b + (lane >> 1);
            if (k >= steps) return -1;
            const int64_t grp = 2 * (int64_t)(rq.tile0 + first_tile + warp + ATT_WARPS * k) + (lane & 1);
            if (grp * KV_GROUP >= rq.len) return -1;
            const uint32_t col = divu32((uint32_t)grp, p.dv_page_groups);
            if (col >= a.width) return -1;
            const int page = load_global(a.table + r * a.stride + col);
            if (page < 0 || page >= a.pages) return -1;
            return (((int64_t)page * a.kv_heads + h) * p.page_groups + ((uint32_t)grp - col * (uint32_t)p.page_groups)) * REC;
        };
        int64_t now = look_up(0), next = look_up(1);
        uint32_t there = 0;                                                // two bits a stage: its records hold data
        int in_slot = 0;
        auto issue = [&](int k) {
            if (k < steps) {
                if ((k & 15) == 0 && k > 0) {
                    now = next;
                    next = look_up((k >> 4) + 1);
                }
                const int64_t a0 = __shfl_sync(0xFFFFFFFFu, now, 2 * (k & 15)), a1 = __shfl_sync(0xFFFFFFFFu, now, 2 * (k & 15) + 1);
                const uint32_t got = (a0 >= 0 ? 1u : 0u) | (a1 >= 0 ? 2u : 0u);
                there = (there & ~(3u << (2 * in_slot))) | (got << (2 * in_slot));
                const uint32_t dst = ring_u32 + in_slot * STAGE_BYTES + 16 * lane;
                const uint8_t *p0 = a.cache + a0 + 16 * lane, *p1 = a.cache + a1 + 16 * (lane - CHUNKS);
                // 16-byte pieces lane + 32 i of the two records
                if (got == 3u) {
#pragma unroll
                    for (int i = 0; i < (2 * CHUNKS + 31) / 32; ++i) {
                        const uint8_t* from = 32 * i + 32 <= CHUNKS ? p0 : (32 * i >= CHUNKS || lane >= CHUNKS - 32 * i ? p1 : p0);
                        if (32 * i + 32 <= 2 * CHUNKS || lane < 2 * CHUNKS - 32 * i) copy_async_16(dst + 512 * i, from + 512 * i);
                    }
                } else if (got != 0u) {
                    for (int i = 0; 32 * i + lane < 2 * CHUNKS; ++i) {
                        const bool second = 32 * i + lane >= CHUNKS;
                        if (got & (second ? 2u : 1u)) copy_async_16(dst + 512 * i, (second ? p1 : p0) + 512 * i);
                    }
                }
            }
            copy_async_commit();
            in_slot = in_slot + 1 == STAGES ? 0 : in_slot + 1;
        };
        // the queries are fetched while the look-ups are on their way, and made into fragments behind the first copies (fetched
        // behind them too, 64 requests with D = 64 take 48.9 us instead of 47.4)
        uint32_t qw[NQ][D / 8];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            const int col = col0 + nq * 8 + g;
            const bool real = col < cols;
            const int i = real ? (int)divu32((uint32_t)col, p.dv_group) : 0;
            const int hq = real ? h * a.group + (col - i * a.group) : 0;
            const uint4* src = reinterpret_cast<const uint4*>(a.q + (int64_t)(rq.first + i) * a.q_token + (int64_t)hq * a.q_head + t4 * (D / 4));
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                uint4 v = make_uint4(0u, 0u, 0u, 0u);
                if (real) v = load_global(src + k);
                qw[nq][4 * k] = v.x; qw[nq][4 * k + 1] = v.y; qw[nq][4 * k + 2] = v.z; qw[nq][4 * k + 3] = v.w;
            }
        }
        const float S_k = load_global(a.s_k + h);
#pragma unroll
        for (int k = 0; k < STAGES - 1; ++k) issue(k);

        // ---- Q^T fragments: column g of each eight, elements [t4 * D / 4, + D / 4), as FP16 scaled by a power of two
        uint32_t qf[NQ][KS][2];
        float mul[NQ][2], slack[NQ][2];                                    // score -> exponent of two, columns 2 t4, 2 t4 + 1
        int pos[NQ][2];                                                    // last position they attend to (-1: none)
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq) {
            uint32_t (&w)[D / 8] = qw[nq], m2 = 0;
#pragma unroll
            for (int k = 0; k < D / 8; ++k) m2 = absmax_bf16x2_int(m2, w[k]);
            uint32_t amax = fold_halves(m2);
            if (amax >= 0x7F80u) {                                         // infinities and NaN go through as they are
                amax = 0;
#pragma unroll
                for (int k = 0; k < D / 8; ++k) {
                    const uint32_t lo = w[k] & 0x7FFFu, hi = (w[k] >> 16) & 0x7FFFu;
                    amax = max(amax, max(lo < 0x7F80u ? lo : 0u, hi < 0x7F80u ? hi : 0u));
                }
            }
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            // x * 2^(142 - e) with e the biased exponent of the largest element (27 at least: the factor stays finite)
            const int e = max((int)(amax >> 7), 27);
            const float c = a.scale * 1.4426950408889634f * S_k * __uint_as_float((uint32_t)(e - 15) << 23);
            // a negative factor goes into Q: scores are then compared before they are multiplied
            const float up = copysignf(__uint_as_float((uint32_t)(127 + 142 - e) << 23), c);
#pragma unroll
            for (int k = 0; k < D / 8; ++k) qf[nq][k >> 1][k & 1] = pack_f16x2(bf16_lo(w[k]) * up, bf16_hi(w[k]) * up);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                mul[nq][j] = __shfl_sync(0xFFFFFFFFu, c == 0.0f ? FLT_MIN : fabsf(c), 4 * (2 * t4 + j));      // not 0: 0 * -inf
                slack[nq][j] = fminf(ATT_SLACK / mul[nq][j], 1e30f);
                const int cj = col0 + nq * 8 + 2 * t4 + j;
                pos[nq][j] = cj < cols ? base_pos + (int)divu32((uint32_t)cj, p.dv_group) : -1;
            }
        }
        // positions that every column of the tile attends to
        const int last_col = min(cols, col0 + 8 * NQ) - 1;
        const int all_hi = base_pos + (int)divu32((uint32_t)col0, p.dv_group) + 1;
        const int all_lo = a.window > 0 ? max(0, base_pos + (int)divu32((uint32_t)last_col, p.dv_group) + 1 - a.window) : 0;

        float o[NQ][MT][4] = {};
        float m[NQ][2], l[NQ][2];
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                m[nq][j] = -INFINITY;
                l[nq][j] = 0.0f;
            }

        int slot = 0, tok0 = (rq.tile0 + first_tile + warp) * ATT_TILE;
        const uint8_t* const at_k = ring + kv_token_of_row(g) * (D / 2) + t4 * (D / 8);
        const uint8_t* const at_ks = ring + kv_k_scales(D) + kv_token_of_row(g) * (D / 16) + t4 * (D / 64);
        const uint8_t* const at_v = ring + kv_v_codes(D) + g * (D / 16);
        const uint8_t* const at_vs = ring + kv_v_scales(D) + (D == 64 ? g >> 1 : (D == 128 ? g : 2 * g)) * 16 + 2 * t4;
        const int v_row[2] = {kv_token_of_row(2 * t4) * (D / 2), kv_token_of_row(2 * t4 + 1) * (D / 2)};
        for (int k = 0; k < steps; ++k, tok0 += ATT_WARPS * ATT_TILE) {
            copy_async_wait<STAGES - 2>();
            __syncwarp();
            issue(k + STAGES - 1);
            const int st = slot * STAGE_BYTES;
            const uint32_t have = (there >> (2 * slot)) & 3u;
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            const bool full = have == 3u && tok0 <= all_hi - ATT_TILE && tok0 >= all_lo;

            // scores
            float s[2][NQ][4] = {};
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                uint32_t kw[2][KW], ksc[2][(D + 127) / 128];                  // scales in pairs of blocks
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    load_words<KW>(at_k + st + gr * REC + x * (8 * D / 2), kw[x]);
                    const uint8_t* sc = at_ks + st + gr * REC + x * (8 * D / 16);
                    if constexpr (D == 64) ksc[x][0] = e4m3x2_to_f16x2(*sc);
                    else if constexpr (D == 128) ksc[x][0] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(sc));
                    else {
                        const uint32_t four = *reinterpret_cast<const uint32_t*>(sc);
                        ksc[x][0] = e4m3x2_to_f16x2(four);
                        ksc[x][(D + 127) / 128 - 1] = e4m3x2_to_f16x2(four >> 16);
                    }
                }
#pragma unroll
                for (int w = 0; w < KW; ++w) {
                    uint32_t f[2][4];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        e2m1x8_to_f16(kw[x][w], f[x]);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            f[x][i] = ((w >> 1) & 1) ? mul_f16x2_hi(f[x][i], ksc[x][w >> 2]) : mul_f16x2_lo(f[x][i], ksc[x][w >> 2]);
                    }
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq) {
                        mma_16816(s[gr][nq], f[0][0], f[1][0], f[0][1], f[1][1], qf[nq][2 * w][0], qf[nq][2 * w][1]);
                        mma_16816(s[gr][nq], f[0][2], f[1][2], f[0][3], f[1][3], qf[nq][2 * w + 1][0], qf[nq][2 * w + 1][1]);
                    }
                }
            }

            // fragment row g of half x of record gr is token gr * 16 + 8 x + token_of_row(g)
            if (!full) {
#pragma unroll
                for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int tok = tok0 + gr * 16 + 8 * x + kv_token_of_row(g);
                        const bool there_is = (have >> gr) & 1u;
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                            for (int j = 0; j < 2; ++j) {
                                const bool in = there_is && tok <= pos[nq][j] && (a.window == 0 || tok > pos[nq][j] - a.window);
                                if (!in) s[gr][nq][2 * x + j] = -INFINITY;
                            }
                    }
            }
            // softmax
            float top[NQ][2];
            bool raise = false;
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                top[nq][0] = top[nq][1] = -INFINITY;
#pragma unroll
                for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            top[nq][j] = fmaxf(top[nq][j], s[gr][nq][2 * x + j]);
                        }
                raise |= top[nq][0] - m[nq][0] > slack[nq][0] || top[nq][1] - m[nq][1] > slack[nq][1];
            }
            if (__any_sync(0xFFFFFFFFu, raise)) {
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float v = fmaxf(top[nq][j], m[nq][j]);
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
                        v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
                        f[j] = m[nq][j] == -INFINITY ? 0.0f : ex2((m[nq][j] - v) * mul[nq][j]);
                        m[nq][j] = v;
                        l[nq][j] *= f[j];
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[nq][mt][e] *= f[e & 1];
                }
            }
            uint32_t pf[2][NQ][2];                                         // P as B fragments
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq) {
                // 2^(mul (s - m) + 7), the difference first: the products of large scores (2^31 and more) would be rounded by more than FP16
                // has room for.  A column with nothing so far has only -inf, from which 0 is taken.
                const float m0 = m[nq][0] == -INFINITY ? 0.0f : m[nq][0], m1 = m[nq][1] == -INFINITY ? 0.0f : m[nq][1];
#pragma unroll
                for (int gr = 0; gr < 2; ++gr)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float p0 = ex2(__fmaf_rn(s[gr][nq][2 * x] - m0, mul[nq][0], ATT_P_SHIFT)), p1 = ex2(__fmaf_rn(s[gr][nq][2 * x + 1] - m1, mul[nq][1], ATT_P_SHIFT));
                        l[nq][0] += p0;
                        l[nq][1] += p1;
                        pf[gr][nq][x] = transpose_8x8(pack_f16x2(p0, p1));
                    }
            }

            // output: dimensions [g * D / 8, + D / 8) of each pair of tokens; byte i of the interleaved words is a dimension
#pragma unroll
            for (int gr = 0; gr < 2; ++gr) {
                uint32_t vw[2][2][VW], vsc[2][(D + 127) / 128];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
#pragma unroll
                    for (int y = 0; y < 2; ++y)
                        load_words<VW>(at_v + v_row[y] + st + gr * REC + x * (8 * D / 2), vw[x][y]);
#pragma unroll
                    for (int b = 0; b < (D + 127) / 128; ++b)
                        vsc[x][b] = *reinterpret_cast<const uint16_t*>(at_vs + st + gr * REC + 16 * b + 8 * x);
                }
                if (!full) {
                    uint32_t nan[2][(D + 127) / 128], any = 0;             // 0x7F in the byte of a scale that is NaN
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int tok = tok0 + gr * 16 + 8 * x;
                        const bool hv = (have >> gr) & 1u;
                        // bytes beyond the context may be anything
                        const uint32_t keep = (hv && tok + kv_token_of_row(2 * t4) < rq.len ? 0x00FFu : 0u) |
                                              (hv && tok + kv_token_of_row(2 * t4 + 1) < rq.len ? 0xFF00u : 0u);
#pragma unroll
                        for (int b = 0; b < (D + 127) / 128; ++b) {
                            vsc[x][b] &= keep;
                            nan[x][b] = ((vsc[x][b] & 0x007Fu) == 0x007Fu ? 0x00FFu : 0u) | ((vsc[x][b] & 0x7F00u) == 0x7F00u ? 0xFF00u : 0u);
                            vsc[x][b] &= ~nan[x][b];
                            any |= nan[x][b];
                        }
                    }
                    // A NaN would reach the columns that mask its token, as 0 * NaN.  It goes instead, block by block, to the
                    // columns that attend to the token, however small their probability for it.
                    if (__any_sync(0xFFFFFFFFu, any != 0)) {
#pragma unroll 1
                        for (int q = 0; q < 8; ++q)
#pragma unroll
                            for (int nq = 0; nq < NQ; ++nq) {
                                const int hi = __shfl_sync(0xFFFFFFFFu, (q & 1) ? pos[nq][1] : pos[nq][0], q >> 1);      // of column q
                                uint32_t on[2] = {0u, 0u};
#pragma unroll
                                for (int x = 0; x < 2; ++x)
#pragma unroll
                                    for (int y = 0; y < 2; ++y) {
                                        const int tok = tok0 + gr * 16 + 8 * x + kv_token_of_row(2 * t4 + y);
                                        if (tok <= hi && (a.window == 0 || tok > hi - a.window)) on[x] |= 0xFFu << (8 * y);
                                    }
#pragma unroll
                                for (int b = 0; b < (D + 127) / 128; ++b) {
                                    uint32_t hit = (nan[0][b] & on[0]) | (nan[1][b] & on[1]);
                                    hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 1);
                                    hit |= __shfl_xor_sync(0xFFFFFFFFu, hit, 2);
                                    const float add = hit && (q >> 1) == t4 ? __int_as_float(0x7FC00000) : 0.0f;
#pragma unroll
                                    for (int w = 2 * b; w < VW && w < 2 * b + 2; ++w)
#pragma unroll
                                        for (int e = 0; e < 16; ++e)
                                            if ((e & 1) == (q & 1)) o[nq][4 * w + (e >> 2)][e & 3] += add;
                                }
                            }
                    }
                }
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int b = 0; b < (D + 127) / 128; ++b) vsc[x][b] = e4m3x2_to_f16x2(vsc[x][b]);
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    uint32_t f[2][2][4];                                   // [half][even / odd dimension][byte]
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t wa = vw[x][0][w], wb = vw[x][1][w];
                        e2m1x8_to_f16((wa & 0x0F0F0F0Fu) | ((wb << 4) & 0xF0F0F0F0u), f[x][0]);
                        e2m1x8_to_f16(((wa >> 4) & 0x0F0F0F0Fu) | (wb & 0xF0F0F0F0u), f[x][1]);
#pragma unroll
                        for (int y = 0; y < 2; ++y)
#pragma unroll
                            for (int i = 0; i < 4; ++i) f[x][y][i] = mul_f16x2(f[x][y][i], vsc[x][w >> 1]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq)
                            mma_16816(o[nq][4 * w + i], f[0][0][i], f[0][1][i], f[1][0][i], f[1][1][i], pf[gr][nq][0], pf[gr][nq][1]);
                }
            }
        }
        copy_async_wait<0>();

        // ---- join the four warps
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                if (m[nq][j] != -INFINITY) m[nq][j] = __fmaf_rn(m[nq][j], mul[nq][j], -ATT_P_SHIFT);       // from here on the exponent of two of l and o
                float v = l[nq][j];
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
                v += __shfl_xor_sync(0xFFFFFFFFu, v, 16);
                if (g == 0) {
                    s_m[warp][nq * 8 + 2 * t4 + j] = m[nq][j];
                    s_l[warp][nq * 8 + 2 * t4 + j] = v;
                }
            }
        const bool whole = first_tile == 0 && n_tiles == rq.tiles;
        const int place = first_tile > 0 ? 0 : 1;
        const int64_t part = ((int64_t)blockIdx.x * 2 + place) * (8 * NQ);
        float* buf = reinterpret_cast<float*>(smem);                       // [warp][8 NQ][D + 4]
        constexpr int LD = D + 4;
        static_assert(ATT_WARPS * 8 * NQ * LD * 4 <= att_ring_bytes(D), "the join fits in the ring");
        const float S_v = load_global(a.s_v + h);
        auto store = [&](int col, int d, float4 x, float M, float L) {
            if (col >= cols) return;
            const int i = (int)divu32((uint32_t)col, p.dv_group), hq = h * a.group + (col - i * a.group);
            const int64_t t = rq.first + i;
            const float f = L == 0.0f ? 0.0f : 1.0f / L;                   // (S_v / L may be too small for FP32 where x * S_v / L is not)
            *reinterpret_cast<uint2*>(a.out + t * a.o_token + (int64_t)hq * a.o_head + d) =
                make_uint2(pack_bf16x2(x.x * f * S_v, x.y * f * S_v), pack_bf16x2(x.z * f * S_v, x.w * f * S_v));
            if (a.lse && d == 0) a.lse[t * ((int64_t)a.kv_heads * a.group) + hq] = L == 0.0f ? -INFINITY : __fmaf_rn(M, 0.6931471805599453f, logf(L));
        };
        __syncthreads();                                                   // ring no longer read; s_m, s_l written
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int c = nq * 8 + 2 * t4 + j;
                float M = s_m[0][c];
#pragma unroll
                for (int w = 1; w < ATT_WARPS; ++w) M = fmaxf(M, s_m[w][c]);
                const float f = m[nq][j] == -INFINITY ? 0.0f : ex2(m[nq][j] - M);
                float* dst = buf + (warp * 8 * NQ + c) * LD + g * (D / 8);
#pragma unroll
                for (int mt = 0; mt < MT; mt += 2)
                    *reinterpret_cast<float4*>(dst + 2 * mt) = make_float4(o[nq][mt][j] * f, o[nq][mt][2 + j] * f, o[nq][mt + 1][j] * f, o[nq][mt + 1][2 + j] * f);
            }
        __syncthreads();
        for (int e = tid; e < 8 * NQ * (D / 4); e += ATT_THREADS) {
            const int c = e / (D / 4), d = (e - c * (D / 4)) * 4;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) M = fmaxf(M, s_m[w][c]);
#pragma unroll
            for (int w = 0; w < ATT_WARPS; ++w) {
                const float4 v = *reinterpret_cast<const float4*>(buf + (w * 8 * NQ + c) * LD + d);
                x.x += v.x; x.y += v.y; x.z += v.z; x.w += v.w;
                L = __fmaf_rn(s_l[w][c], s_m[w][c] == -INFINITY ? 0.0f : ex2(s_m[w][c] - M), L);
            }
            if (CLUSTER) {                                                 // in the first warp's place, for the others
                *reinterpret_cast<float4*>(buf + c * LD + d) = x;
                if (d == 0) s_ml[c] = make_float2(M, L);
            } else if (!whole) {
                *reinterpret_cast<float4*>(p.part_o + (part + c) * D + d) = x;
                if (d == 0) *reinterpret_cast<float2*>(p.part_ml + (part + c) * 2) = make_float2(M, L);
            } else {
                store(col0 + c, d, x, M, L);
            }
        }
        if (CLUSTER) {                                                     // join of the cluster, in the order of its CTAs
            cluster_barrier();
            for (int e = (int)rank * ATT_THREADS + tid; e < 8 * NQ * (D / 4); e += ATT_THREADS * p.cluster) {
                const int c = e / (D / 4), d = (e - c * (D / 4)) * 4;
                float2 ml[ATT_MAX_CLUSTER];
                float4 v[ATT_MAX_CLUSTER], x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int k = 0; k < ATT_MAX_CLUSTER; ++k) {                // beyond the last CTA its place again, with nothing in it
                    ml[k] = load_there2(there_u32(s_ml + c, min(k, p.cluster - 1)));
                    v[k] = load_there4(there_u32(buf + c * LD + d, min(k, p.cluster - 1)));
                    if (k >= p.cluster) {
                        ml[k] = make_float2(-INFINITY, 0.0f);
                        v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    }
                }
#pragma unroll
                for (int k = 0; k < ATT_MAX_CLUSTER; ++k) M = fmaxf(M, ml[k].x);
#pragma unroll
                for (int k = 0; k < ATT_MAX_CLUSTER; ++k) {
                    const float f = ml[k].x == -INFINITY ? 0.0f : ex2(ml[k].x - M);
                    L = __fmaf_rn(ml[k].y, f, L);
                    x.x = __fmaf_rn(v[k].x, f, x.x); x.y = __fmaf_rn(v[k].y, f, x.y);
                    x.z = __fmaf_rn(v[k].z, f, x.z); x.w = __fmaf_rn(v[k].w, f, x.w);
                }
                store(col0 + c, d, x, M, L);
            }
            cluster_barrier();                                             // before anybody writes its ring again, or leaves
        }
        if (first_tile == 0 && tid == 0 && !whole_items && (p.by_item || !whole)) {
            Piece pc{(int)blockIdx.x, 0, rq.first, h, col0, cols};
            if (!whole) pc.count = (int)((item_at + per_item - 1) / share) - (int)blockIdx.x + 1;
            p.pieces[p.by_item ? item0 + item : (int)blockIdx.x] = pc;
        }
        __syncthreads();                                                   // buffer free for the next item's ring
        at += run;
        off += run;
    }
}

// Join of the pieces of an item, in the order of the CTAs: a warp takes a column, or with SHARED (few items, many pieces) all
// warps of a CTA share a column's pieces.  A lane holds D / 32 neighbouring dimensions.
constexpr int JOIN_THREADS = 256;
template <int D, bool SHARED>
__global__ void __launch_bounds__(JOIN_THREADS) kv_attention_join_kernel(const __grid_constant__ AttParams p, int columns) {
    constexpr int V = D / 32, WARPS = JOIN_THREADS / 32, UB = 8;             // UB pieces in flight
    chain_begin();
    const Piece pc = p.pieces[blockIdx.x];
    if (pc.count <= 0) return;
    const KvAttentionArgs& a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = SHARED ? (int)blockIdx.y : (int)blockIdx.y * WARPS + warp, col = pc.col0 + c;
    if (col >= pc.cols) return;
    float M = -INFINITY, L = 0.0f, o[V] = {};
    constexpr int step = SHARED ? WARPS : 1;
    for (int k0 = SHARED ? warp : 0; k0 < pc.count; k0 += UB * step) {
        float x[UB][V], ml[UB][2];
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const int k = k0 + u * step;
            const int64_t at = ((int64_t)(pc.first_cta + k) * 2 + (k == 0 ? 1 : 0)) * columns + c;
            const bool in = k < pc.count;
            const float2 q = in ? *reinterpret_cast<const float2*>(p.part_ml + at * 2) : make_float2(-INFINITY, 0.0f);
            ml[u][0] = q.x;
            ml[u][1] = q.y;
            const float* src = p.part_o + at * D + lane * V;
#pragma unroll
            for (int v = 0; v < V; v += 2) {
                const float2 f = in ? *reinterpret_cast<const float2*>(src + v) : make_float2(0.0f, 0.0f);
                x[u][v] = f.x;
                x[u][v + 1] = f.y;
            }
        }
        float Mn = M;
#pragma unroll
        for (int u = 0; u < UB; ++u) Mn = fmaxf(Mn, ml[u][0]);
        const float f0 = M == -INFINITY ? 0.0f : ex2(M - Mn);
        L *= f0;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] *= f0;
#pragma unroll
        for (int u = 0; u < UB; ++u) {
            const float f = ml[u][0] == -INFINITY ? 0.0f : ex2(ml[u][0] - Mn);
            L = __fmaf_rn(ml[u][1], f, L);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = __fmaf_rn(x[u][v], f, o[v]);
        }
        M = Mn;
    }
    if constexpr (SHARED) {
        __shared__ float s_o[WARPS][D], s_ml[WARPS][2];
#pragma unroll
        for (int v = 0; v < V; ++v) s_o[warp][lane * V + v] = o[v];
        if (lane == 0) {
            s_ml[warp][0] = M;
            s_ml[warp][1] = L;
        }
        __syncthreads();
        if (warp != 0) return;
        M = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_ml[w][0]);
        L = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = s_ml[w][0] == -INFINITY ? 0.0f : ex2(s_ml[w][0] - M);
            L = __fmaf_rn(s_ml[w][1], f, L);
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] = __fmaf_rn(s_o[w][lane * V + v], f, o[v]);
        }
    }
    const int i = (int)divu32((uint32_t)col, p.dv_group), hq = pc.kv_head * a.group + (col - i * a.group);
    const int64_t t = pc.token0 + i;
    const float f = L == 0.0f ? 0.0f : 1.0f / L, S_v = load_global(a.s_v + pc.kv_head);
    uint32_t* out = reinterpret_cast<uint32_t*>(a.out + t * a.o_token + (int64_t)hq * a.o_head + lane * V);
#pragma unroll
    for (int v = 0; v < V; v += 2) out[v >> 1] = pack_bf16x2(o[v] * f * S_v, o[v + 1] * f * S_v);
    if (a.lse && lane == 0) a.lse[t * ((int64_t)a.kv_heads * a.group) + hq] = L == 0.0f ? -INFINITY : __fmaf_rn(M, 0.6931471805599453f, logf(L));
}

template <int D, int NQ>
cudaError_t launch_nq(AttParams& p, int num_sms, cudaStream_t stream) {
    static PerDevice pd;
    static int clusters[MX_MAX_DEVICES][ATT_MAX_CLUSTER + 1];                 // that the device runs at once, by their CTAs
    int dev = 0;
    cudaError_t e = per_device_once(pd, dev, [](int& value) {
        cudaError_t s = cudaGetDevice(&value);
        if (s == cudaSuccess) s = cudaFuncSetAttribute(kv_attention_kernel<D, NQ, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, att_ring_bytes(D));
        if (s == cudaSuccess) s = cudaFuncSetAttribute(kv_attention_kernel<D, NQ, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, att_ring_bytes(D));
        for (int c = 2; c <= ATT_MAX_CLUSTER && s == cudaSuccess; c *= 2) {
            cudaLaunchAttribute at{};
            at.id = cudaLaunchAttributeClusterDimension;
            at.val.clusterDim = {(unsigned)c, 1, 1};
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3((unsigned)c);
            cfg.blockDim = dim3(ATT_THREADS);
            cfg.dynamicSmemBytes = att_ring_bytes(D);
            cfg.attrs = &at;
            cfg.numAttrs = 1;
            s = cudaOccupancyMaxActiveClusters(&clusters[value][c], kv_attention_kernel<D, NQ, true>, &cfg);
        }
        return s;
    });
    if (e != cudaSuccess) return e;
    const KvAttentionArgs& a = p.a;
    const int64_t items = (int64_t)a.R * a.kv_heads * ((a.max_q * (int64_t)a.group + 8 * NQ - 1) / (8 * NQ)), table = a.width * a.page;
    // Few items: all warps of a CTA join one column's pieces, and four places for CTAs stay empty.  Behind the kernel before, whose
    // last CTAs still hold registers and shared memory, some SMs take one CTA less, and what waits for them begins when others
    // end (one request of 130944 tokens, 72 tiles for each of 456 CTAs: 41.7 us, with 452 CTAs 34.7).
    const int resident = num_sms * att_ctas(D, NQ);
    const bool shared = items * 8 <= resident;
    const int ctas = shared ? max(1, resident - 4) : resident;
    p.by_item = items <= ctas;
    // Short contexts (by the table's width) are not split over the GPU: one launch instead of two.  Where the items leave room,
    // each has a cluster of 2 to 8 CTAs, whose meeting takes 1.3 us: one request of 256 positions 6.9 us with one and 6.1
    // without, 512 6.7 and 7.6; 2048 7.9 and split over the GPU 9.0, 5000 10.6 and 10.4 (and 2 us more of the host's time).
    // Clusters that wait for room cost more than the split: 56 of 8 CTAs 16.5 us instead of 12.3.  The fuller the GPU with
    // unsplit items, the longer they may be: 320 items to 1000 positions 16.2 unsplit and 16.9 split, to 1700 23.5 and 20.7; 456
    // items 17.0 and 20.3, 23.5 and 24.8.  512 items, more than CTAs, to 512 positions 15.4 and 16.5, to 1000 22.9 and 22.1.
    p.cluster = 1;
    while (table > ATT_CLUSTER_TOKENS && p.cluster < ATT_MAX_CLUSTER && items <= clusters[dev][2 * p.cluster]) p.cluster *= 2;
    const int64_t limit = !p.by_item ? ATT_WHOLE_TOKENS
                        : p.cluster > 2 ? ATT_WHOLE_CLUSTER_TOKENS * p.cluster : max64(ATT_CLUSTER_TOKENS, ATT_WHOLE_FULL_TOKENS * items * p.cluster / ctas);
    p.whole_items = table <= limit;
    if (!p.whole_items) p.cluster = 1;
    p.n_pieces = (int)(p.by_item ? items : ctas);
    uint8_t* ws = static_cast<uint8_t*>(a.workspace);
    p.pieces = reinterpret_cast<Piece*>(ws);
    p.part_ml = reinterpret_cast<float*>(ws + (int64_t)num_sms * ATT_MAX_CTAS_PER_SM * sizeof(Piece));
    p.part_o = p.part_ml + (int64_t)ctas * 2 * (8 * NQ) * 2;
    if (p.cluster > 1)
        return launch_chained(kv_attention_kernel<D, NQ, true>, dim3((unsigned)(items * p.cluster)), ATT_THREADS, att_ring_bytes(D), (unsigned)p.cluster, stream, p);
    const int64_t grid_x = p.whole_items ? min64(items, ctas) : ctas;
    e = launch_chained(kv_attention_kernel<D, NQ, false>, dim3((unsigned)grid_x), ATT_THREADS, att_ring_bytes(D), 0, stream, p);
    if (e != cudaSuccess || p.whole_items) return e;
    const dim3 grid((unsigned)p.n_pieces, shared ? 8 * NQ : 8 * NQ * 32 / JOIN_THREADS);
    return shared ? launch_chained(kv_attention_join_kernel<D, true>, grid, JOIN_THREADS, 0, 0, stream, p, 8 * NQ)
                  : launch_chained(kv_attention_join_kernel<D, false>, grid, JOIN_THREADS, 0, 0, stream, p, 8 * NQ);
}

template <int D>
cudaError_t launch_d(AttParams& p, int num_sms, cudaStream_t stream) {
    const int64_t rows = (int64_t)p.a.max_q * p.a.group;
    // Two column fragments for more than eight query rows of a kv head; wider items of 32 (drafts, D = 64: 26.8 us instead of
    // 20.3) keep too few warps on an SM, and their registers spill for larger D.
    return rows <= 8 ? launch_nq<D, 1>(p, num_sms, stream) : launch_nq<D, 2>(p, num_sms, stream);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t D) {
    const int columns = 8 * (att_ctas((int)D, 1) > 2 * att_ctas((int)D, 2) ? att_ctas((int)D, 1) : 2 * att_ctas((int)D, 2));   // of an SM's CTAs
    return (size_t)((int64_t)device_sm_count() * (ATT_MAX_CTAS_PER_SM * (int64_t)sizeof(Piece) + 2 * columns * (D + 2) * 4));
}

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int num_sms, cudaStream_t stream) {
    AttParams p{};
    p.a = a;
    p.page_groups = a.page / KV_GROUP;
    p.dv_group = make_divu32((uint64_t)a.group);
    p.dv_page_groups = make_divu32((uint64_t)p.page_groups);
    if (a.dim == 64) return launch_d<64>(p, num_sms, stream);
    if (a.dim == 128) return launch_d<128>(p, num_sms, stream);
    return launch_d<256>(p, num_sms, stream);
}

}  // namespace mxk
