// matvec_nvfp4.cu -- products of a few tokens with NVFP4 weights (the linear layers of a generation step).
//
//   y[m, n] = s2[n or 0] * sum_k x[m, k] * val(q[n, k]) * val(bs[n, k / 16])
//
// Bound: the weights are read once, 0.5625 bytes a value, and each value meets M tokens; up to 16 tokens the HBM
// copy rate is the floor.  What has to keep up is the expansion of the codes: 128 values a thread cost 64
// conversions on the ALU and 64 multiplications by the block scale (2 clocks a warp each), inside the 396 clocks that the
// copy rate leaves a quarter of an SM for the 2304 bytes of a warp's step.  The multiplications share the FP16 pipe with the
// matrix instructions (8 clocks each): 254 clocks a step for up to 8 tokens, 381 for up to 16.
// (On tcgen05 with the expanded weights as A in tensor memory the same products were no faster, 40.6 us against 36.7 for
// 151937 x 2048: an M = 128, N = 16, K = 16 instruction costs about 50 clocks however few its columns are, and 16 of them
// a stage of 128 x 256 values fill the 790 clocks that the copy rate leaves.)
//
// Weight rows are the rows (M) of mma.m16n8k16 and tokens its columns, eight to a fragment.  val(q) * val(bs) has at
// most 6 significant bits and is exact in FP16.  x enters as FP16 scaled by a power of two per token and step, its largest
// element there in [2^15, 2^16): exact down to 2^-29 of that, an absolute error of 2^-40 of it below.  The product of
// a step is scaled back as it joins the sum.
//
// A warp takes 32 rows, 8 consecutive ones in each of the four 32-row bands of a 128-row scale tile: the 16 bytes that the
// GEMM scale layout holds for a row of the first band are the four bands' scales of the same four columns, so no
// scale sector is fetched for a quarter of its bytes.  In a step of 128 values a thread reads 16 bytes of codes from
// each of its four rows (a quad: 64 contiguous bytes) and one 16-byte piece of scales, through a cp.async
// ring of its warp's: what keeps HBM busy is bytes in flight, and the ring holds 74 to 110 KB an SM without registers.  It
// runs on across the rows that a CTA takes in turn, while x stays where it is.
// A CTA has 16 warps, WK of them along K for each group of 32 rows: 1 where there are rows enough for every warp of the
// GPU, which then never wait for each other, up to all 16 where there are few.  Partial sums meet in shared memory,
// and across the CTAs of a cluster, which split K further, through distributed shared memory; always in the same order,
// so a result does not depend on timing.
//
// Measured on a GB300 (device us, share of the measured copy rate): 1 x 151937 x 2048 31.9 (81 %: HBM, without loads 27.1).
// The others with weights that stay in L2 from call to call / with others than the last calls', from HBM: 5 x 12288 x 4096 11.0 /
// 11.5 (38 / 37 %: about 4 us fixed; four warps along K make 96 turns of the 384 row groups, for 96 of 152 SMs), 16 x 4096 x 14336 16.7 /
// 16.8 (30 %: about 10 us are launch, first loads, the staging of x (3.3) and the two meetings; the FP16 pipe is busy
// 32 % of the whole), 1 x 4096 x 4096 4.7 / 5.0 (29 / 28 %: latency).
#include "mx_internal.h"
#include "mx_fragment.cuh"
#include "mx_chain.cuh"

namespace mxk {

namespace {

constexpr int MV_ROWS = 32;                           // of a warp
constexpr int MV_STEP = 128;                          // values of K a step
// A warp's step in the ring: codes of four rows a lane, scales; where rows start on 8 bytes only, 8 bytes more of a row.
__host__ __device__ constexpr int mv_slot(bool A16) { return 4 * 512 + 256 + (A16 ? 0 : 256); }
constexpr int MV_MAX_SPLIT = 8;                       // CTAs of a cluster
constexpr int MV_SMEM = 225 * 1024;                   // dynamic shared memory of a CTA, which has its SM to itself
constexpr int MV_WARPS = 16;
__host__ __device__ constexpr int mv_stages(int NQ) { return NQ == 1 ? 3 : 2; }
__host__ __device__ constexpr int mv_ring(int NQ, bool A16) { return MV_WARPS * mv_stages(NQ) * mv_slot(A16); }
// Bytes of a staged token: a stretch of `steps` steps, and 64 so that odd and even tokens lie on both bank halves.
__host__ __device__ constexpr int mv_row_bytes(int steps) { return steps * MV_STEP * 2 + 64; }
// Partial sums, FP32 [warp][token][row]; staged x; its scales, FP32 [token][step].
__host__ __device__ constexpr int mv_sums(int M) { return MV_WARPS * M * MV_ROWS * 4; }
__host__ __device__ constexpr int mv_x(int M, int steps) { return M * (mv_row_bytes(steps) + steps * 4); }

struct MvPlan {
    int wk;                                           // warps along K (a power of two)
    int stretch;                                      // steps of x staged at once: all of the CTA's, or a multiple of wk
};

__device__ __forceinline__ void copy_async_16z(uint32_t dst, const void* src, int bytes) {      // the rest of 16 is zero
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_async_8z(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" :: "r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// TAIL: K is not a multiple of the step.  A16: rows start on 16 bytes (K % 32 == 0).  Where they do not, odd rows lie 8
// bytes into a 16-byte piece: a quad brings the pieces that cover them, its last lane the 8 bytes of the fifth, and a
// lane reads its 16 bytes from two neighbours.  All rows of a lane are odd or all even, as its g is.  4 x 57611 x 3152 takes
// 32 us so, and 43 with two copies of 8 bytes a lane (3200, a multiple of the step: 23).
template <int NQ, bool TAIL, bool A16>
__global__ void __launch_bounds__(32 * MV_WARPS, 1)
matvec_kernel(const __grid_constant__ MatvecArgs a, const MvPlan plan) {
    constexpr int WARPS = MV_WARPS, THREADS = 32 * WARPS, STAGES = mv_stages(NQ), SLOT = mv_slot(A16);
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int WK = plan.wk, wk = warp & (WK - 1), groups_cta = WARPS / WK, row_bytes = mv_row_bytes(plan.stretch);
    float* sums = reinterpret_cast<float*>(smem + mv_ring(NQ, A16));                 // [warp][M][MV_ROWS]
    float* xscale = sums + WARPS * a.M * MV_ROWS;                               // [M][stretch]
    uint8_t* xs = smem + (MV_SMEM - a.M * row_bytes) / 16 * 16;
    uint32_t rank, ranks;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    // row groups in the order of the scale tiles: group r is rows 128 (r / 4) + 8 (r % 4) + {0..7} + {0, 32, 64, 96}
    const int groups = (int)((a.N + 127) / 128 * 4), turns = (groups + groups_cta - 1) / groups_cta;
    const int turn0 = (int)(blockIdx.x / ranks), turn_step = (int)(gridDim.x / ranks);
    const int steps = (int)((a.K + MV_STEP - 1) / MV_STEP);
    const int cta0 = (int)((int64_t)steps * rank / ranks), cta1 = (int)((int64_t)steps * (rank + 1) / ranks);
    const int64_t nct = sf_col_tiles(a.K, 16);

    // ---- x of a stretch as FP16: a quad takes a (token, step) pair, 32 values a lane as the fragments have them, finds the largest
    // element and scales by it.  The loads of the first stretch go ahead of the weights'.
    uint4 x[4];
    auto load_x = [&](int c0, int n_steps, int task) {
        const int pair = task >> 2, m = pair / n_steps, st = pair - m * n_steps;
        const int64_t k = (int64_t)(c0 + st) * MV_STEP + t4 * 32;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            x[u] = make_uint4(0u, 0u, 0u, 0u);
            if (m < a.M && (!TAIL || k + u * 8 < a.K)) x[u] = load_global(reinterpret_cast<const uint4*>(a.x + m * a.ldx + k) + u);
        }
    };
    auto stage_x = [&](int c0, int n_steps, bool loaded) {
        for (int task = tid; task - lane < 4 * a.M * n_steps; task += THREADS) {
            if (!loaded) load_x(c0, n_steps, task);
            loaded = false;
            uint32_t m2 = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) m2 = absmax_bf16x2_int(absmax_bf16x2_int(absmax_bf16x2_int(absmax_bf16x2_int(m2, x[u].x), x[u].y), x[u].z), x[u].w);
            uint32_t amax = fold_halves(m2);
            if (amax >= 0x7F80u) {                    // infinities and NaN go through as they are: the largest finite element
                amax = 0;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const uint32_t h = (w[i >> 1] >> (16 * (i & 1))) & 0x7FFFu;
                        amax = max(amax, h < 0x7F80u ? h : 0u);
                    }
                }
            }
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
            amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
            // x * 2^(142 - e), e the biased exponent of the pair's largest element (27 at least: the factor stays finite)
            const int e = max((int)(amax >> 7), 27);
            const float up = __uint_as_float((uint32_t)(127 + 142 - e) << 23);
            const int pair = task >> 2, m = pair / n_steps, st = pair - m * n_steps;
            if (m < a.M) {
                // unit i of thread t4's four goes to place i * 4 + t4: a quad reads 64 contiguous bytes
                uint8_t* to = xs + m * row_bytes + st * (MV_STEP * 2) + t4 * 16;
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    *reinterpret_cast<uint4*>(to + u * 64) =
                        make_uint4(pack_f16x2(bf16_lo(x[u].x) * up, bf16_hi(x[u].x) * up), pack_f16x2(bf16_lo(x[u].y) * up, bf16_hi(x[u].y) * up),
                                   pack_f16x2(bf16_lo(x[u].z) * up, bf16_hi(x[u].z) * up), pack_f16x2(bf16_lo(x[u].w) * up, bf16_hi(x[u].w) * up));
                if (t4 == 0) xscale[m * plan.stretch + st] = __uint_as_float((uint32_t)(e - 15) << 23);
            }
        }
        __syncthreads();
    };
    chain_begin();
    load_x(cta0, min(plan.stretch, cta1 - cta0), tid);

    // ---- the warp's steps, cta0 + wk, + WK, ... of one row group after the other, enter the ring STAGES - 1 ahead
    uint8_t* ring = smem + warp * (STAGES * SLOT);
    const uint32_t ring_u32 = (uint32_t)__cvta_generic_to_shared(ring);
    int in_group = cta0 + wk < cta1 ? turn0 * groups_cta + warp / WK : groups;
    int in_step = cta0 + wk, in_slot = 0;
    const uint8_t *in_q[4], *in_s;                    // the thread's next bytes
    const int odd = A16 ? 0 : 8 * (g & 1);            // bytes that the thread's rows lie beyond a 16-byte boundary
    const bool beyond = odd && t4 == 3;               // the upper half of the thread's 16 bytes is of the fifth piece
    // rows beyond the last repeat it, or the one before it that starts as they do (-1: there is none, and nothing is read)
    const int64_t last_row = A16 ? a.N - 1 : a.N - 1 - ((a.N - 1 - g) & 1);
    const int inputs = (int)a.K;                      // 2^24 at most
    auto left_of = [&](int step) { return min(32, inputs - step * MV_STEP - t4 * 32); };     // valid values of the thread's 32
    auto aim = [&]() {                                // at the first step of in_group
        const int64_t band = in_group >> 2, r0 = band * 128 + 8 * (in_group & 3) + g;
#pragma unroll
        for (int b = 0; b < 4; ++b) in_q[b] = a.q + min64(last_row, r0 + 32 * b) * (a.K / 2) + (int64_t)in_step * (MV_STEP / 2) + t4 * 16 - odd;
        in_s = a.s + ((band * nct + 2 * (int64_t)in_step + (t4 >> 1)) << 9) + ((8 * (in_group & 3) + g) << 4);
    };
    if (in_group < groups) aim();
    auto issue = [&]() {
        if (in_group < groups) {
            const uint32_t slot_at = ring_u32 + in_slot * SLOT, dst = slot_at + lane * 16, dst_s = slot_at + 4 * 512 + (g * 2 + (t4 >> 1)) * 16;
            if (!TAIL) {
#pragma unroll
                for (int b = 0; b < 4; ++b) copy_async_16(dst + b * 512, in_q[b]);
                if ((t4 & 1) == 0) copy_async_16(dst_s, in_s);
            } else {                                  // beyond K zeros, from an address that is valid all the same
                const int left = max(0, left_of(in_step));
                // of an even row, or of one on 16 bytes, the piece may hold 16 values of the row; of an odd one 32, or none
                const int bytes = !A16 && last_row < 0 ? 0 : (left > 0 && odd ? 16 : left / 2);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    copy_async_16z(dst + b * 512, bytes > 0 ? in_q[b] : a.q, bytes);
                    if (beyond)
                        copy_async_8z(slot_at + 4 * 512 + 256 + b * 64 + g * 8, bytes > 0 && left > 16 ? in_q[b] + 16 : a.q, bytes > 0 && left > 16 ? 8 : 0);
                }
                if ((t4 & 1) == 0) copy_async_16z(dst_s, left > 0 ? in_s : a.s, left > 0 ? 16 : 0);
            }
            in_step += WK;
            if (in_step < cta1) {
#pragma unroll
                for (int b = 0; b < 4; ++b) in_q[b] += WK * (MV_STEP / 2);
                in_s += WK * 1024;
            } else {
                in_step = cta0 + wk;
                in_group += turn_step * groups_cta;
                if (in_group < groups) aim();
            }
        }
        copy_async_commit();
        in_slot = in_slot + 1 == STAGES ? 0 : in_slot + 1;
    };
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) issue();

    int slot = 0;
    const int sc_shift = 16 * (t4 & 1);
    const int hi_at = beyond ? 4 * 512 + 256 + g * 8 : lane * 16 + odd + 8, hi_step = beyond ? 64 : 512;
    const bool once = cta1 - cta0 <= plan.stretch;    // x is staged once for all rows
    for (int turn = turn0; turn < turns; turn += turn_step) {
        const int group = turn * groups_cta + warp / WK;
        float acc[2][NQ][4] = {};
        for (int c0 = cta0; c0 < cta1; c0 += plan.stretch) {
            const int c1 = min(cta1, c0 + plan.stretch);
            const bool start = turn == turn0 && c0 == cta0;
            if (start || !once) {
                if (!start) __syncthreads();          // the previous stretch is done with
                stage_x(c0, c1 - c0, start);
            }

            // ---- the products.  A stretch begins at a multiple of WK steps from cta0, so the warps' turns go on.
            // Columns beyond the last token repeat it and are not stored.
            if (group < groups) {
                const uint8_t* xr[NQ];
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) xr[nq] = xs + min(a.M - 1, nq * 8 + g) * row_bytes + t4 * 16;
                for (int step = c0 + wk; step < c1; step += WK) {
                    copy_async_wait<STAGES - 2>();
                    __syncwarp();                     // the scales come by other lanes; and the slot of the last step is free
                    const uint8_t* st = ring + slot * SLOT;
                    uint4 q[4], s;
#pragma unroll
                    for (int b = 0; b < 4; ++b) {
                        if (A16) {
                            q[b] = *reinterpret_cast<const uint4*>(st + b * 512 + lane * 16);
                        } else {
                            const uint2 lo = *reinterpret_cast<const uint2*>(st + b * 512 + lane * 16 + odd);
                            const uint2 hi = *reinterpret_cast<const uint2*>(st + hi_at + b * hi_step);
                            q[b] = make_uint4(lo.x, lo.y, hi.x, hi.y);
                        }
                    }
                    s = *reinterpret_cast<const uint4*>(st + 4 * 512 + (g * 2 + (t4 >> 1)) * 16);
                    if (TAIL && left_of(step) < 32) {  // scales beyond K are padding
                        const uint32_t keep = left_of(step) < 16 ? 0u : ((t4 & 1) ? 0x00FF0000u : 0x000000FFu);
                        s.x &= keep; s.y &= keep; s.z &= keep; s.w &= keep;
                    }
                    issue();
                    slot = slot + 1 == STAGES ? 0 : slot + 1;
                    const int x_at = (step - c0) * (MV_STEP * 2);
                    // the two block scales of the thread's run, columns 2 (t4 & 1) and + 1 of the four
                    const uint32_t sc[4] = {e4m3x2_to_f16x2(s.x >> sc_shift), e4m3x2_to_f16x2(s.y >> sc_shift),
                                            e4m3x2_to_f16x2(s.z >> sc_shift), e4m3x2_to_f16x2(s.w >> sc_shift)};
                    float part[2][NQ][4] = {};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {     // 8 of the thread's 32 values: two k-steps
                        uint4 xb[NQ];
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq) xb[nq] = *reinterpret_cast<const uint4*>(xr[nq] + x_at + i * 64);
                        uint32_t f[4][4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint32_t codes = i == 0 ? q[b].x : (i == 1 ? q[b].y : (i == 2 ? q[b].z : q[b].w));
                            e2m1x8_to_f16(codes, f[b]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) f[b][j] = i < 2 ? mul_f16x2_lo(f[b][j], sc[b]) : mul_f16x2_hi(f[b][j], sc[b]);
                        }
#pragma unroll
                        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                mma_16816(part[t][nq], f[2 * t][0], f[2 * t + 1][0], f[2 * t][1], f[2 * t + 1][1], xb[nq].x, xb[nq].y);
                                mma_16816(part[t][nq], f[2 * t][2], f[2 * t + 1][2], f[2 * t][3], f[2 * t + 1][3], xb[nq].z, xb[nq].w);
                            }
                    }
#pragma unroll
                    for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const float xsc = xscale[min(a.M - 1, nq * 8 + 2 * t4 + j) * plan.stretch + step - c0];
#pragma unroll
                            for (int t = 0; t < 2; ++t) {
                                acc[t][nq][j] = __fmaf_rn(part[t][nq][j], xsc, acc[t][nq][j]);
                                acc[t][nq][2 + j] = __fmaf_rn(part[t][nq][2 + j], xsc, acc[t][nq][2 + j]);
                            }
                        }
                }
            }
        }

        // ---- the results: row 32 b + r of the group's four runs of 8, token m
        auto store = [&](int group, int b, int r, int m, float v) {
            const int64_t n = (int64_t)(group >> 2) * 128 + 8 * (group & 3) + 32 * b + r;
            if (group >= groups || n >= a.N || m >= a.M) return;
            v *= load_global(a.s2 + (a.s2_per_row ? n : 0));
            if (a.y_fp32) static_cast<float*>(a.y)[m * a.ldy + n] = v;
            else static_cast<uint16_t*>(a.y)[m * a.ldy + n] = (uint16_t)pack_bf16x2(v, 0.0f);
        };
        if (WK == 1 && ranks == 1) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) store(group, 2 * t + (j >> 1), g, nq * 8 + 2 * t4 + (j & 1), acc[t][nq][j]);
            continue;
        }
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int m = nq * 8 + 2 * t4 + (j & 1);
                if (m < a.M) {
#pragma unroll
                    for (int t = 0; t < 2; ++t) sums[(warp * a.M + m) * MV_ROWS + 8 * (2 * t + (j >> 1)) + g] = acc[t][nq][j];
                }
            }
        __syncthreads();
        // the WK partial sums of an element lie M rows apart; with a cluster the CTA's sum takes the first one's place
        const int per_group = a.M * MV_ROWS;
        for (int i = tid; i < groups_cta * per_group; i += THREADS) {
            const int gi = i / per_group, e = i - gi * per_group;
            float* at = sums + gi * WK * per_group + e;
            float y = 0.0f;
#pragma unroll 4
            for (int w = 0; w < WK; ++w) y += at[w * per_group];
            if (ranks > 1) *at = y;
            else store(turn * groups_cta + gi, (e % MV_ROWS) >> 3, e & 7, e / MV_ROWS, y);
        }
        if (ranks == 1) {
            __syncthreads();                          // the sums are read before anybody writes them again
            continue;
        }
        cluster_barrier();
        for (int i = tid + (int)rank * THREADS; i < groups_cta * per_group; i += THREADS * (int)ranks) {
            const int gi = i / per_group, e = i - gi * per_group;
            const uint32_t at = (uint32_t)__cvta_generic_to_shared(sums + gi * WK * per_group + e);
            float v[MV_MAX_SPLIT];
#pragma unroll
            for (int c = 0; c < MV_MAX_SPLIT; ++c) {
                uint32_t there;
                asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(at), "r"(min(c, (int)ranks - 1)));
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[c]) : "r"(there) : "memory");
            }
            float y = v[0];
#pragma unroll
            for (int c = 1; c < MV_MAX_SPLIT; ++c)
                if (c < (int)ranks) y += v[c];
            store(turn * groups_cta + gi, (e % MV_ROWS) >> 3, e & 7, e / MV_ROWS, y);
        }
        cluster_barrier();                            // and before anybody leaves
    }
    copy_async_wait<0>();
}

// The split of the work: warps along K and CTAs of a cluster along K, for one CTA an SM, so that the costs below are least.
// In half steps of a warp: the busiest warp's steps (latency) and the mean of the CTA's warps (the pipes and the memory that
// they share), 2.5 for a meeting of the CTA's warps, 2.25 more for one of a cluster, the staging of x by its size.  Fitted to
// the times of all splits of 110 shapes, of which it chooses one that is 1 % slower than the best on average.
// clusters[c] is how many clusters of c CTAs the device runs at once (the SMs of a cluster share a GPC, so it is below SMs / c).
constexpr double MV_STAGING = 0.002, MV_MEET = 2.5, MV_MEET_CLUSTER = 2.25;
MvPlan mv_plan(int ring, const MatvecArgs& a, const int (&clusters)[MV_MAX_SPLIT + 1], int& ctas_k) {
    const int steps = (int)((a.K + MV_STEP - 1) / MV_STEP), warps = MV_WARPS;
    const int64_t groups = (a.N + 127) / 128 * 4;
    int fits = 0;                                     // steps of x that have room
    while (fits < steps && ring + mv_sums(a.M) + mv_x(a.M, fits + 1) + 16 <= MV_SMEM) ++fits;
    MvPlan best{1, 1};
    double least = 1e30;
    ctas_k = 1;
    for (int c = 1; c <= MV_MAX_SPLIT && c <= steps; ++c) {
        if (clusters[c] < 1) continue;
        for (int wk = 1; warps % wk == 0 && (c * wk <= steps || wk == 1); wk *= 2) {
            const int per_turn = warps / wk, mine = (steps + c - 1) / c;
            const int64_t turns = (groups + per_turn - 1) / per_turn, rounds = (turns + clusters[c] - 1) / clusters[c];
            const int stretch = mine <= fits ? mine : fits / wk * wk;
            if (stretch < 1) continue;
            const double staging = 0.5 + MV_STAGING * a.M * stretch;
            const int again = mine <= fits ? 0 : (mine + stretch - 1) / stretch;
            const double meeting = (c > 1 || wk > 1 ? MV_MEET : 0.0) + (c > 1 ? MV_MEET_CLUSTER : 0.0);
            const double cost = (double)rounds * ((mine + wk - 1) / wk + (double)mine / wk + meeting + staging * again) + staging;
            if (cost < least) {
                least = cost;
                best = MvPlan{wk, stretch};
                ctas_k = c;
            }
        }
    }
    return best;
}

template <int NQ, bool TAIL, bool A16>
cudaError_t launch_nq(const MatvecArgs& a, cudaStream_t stream) {
    static PerDevice pd;
    static int clusters[MX_MAX_DEVICES][MV_MAX_SPLIT + 1];
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(32 * MV_WARPS);
    cfg.dynamicSmemBytes = MV_SMEM;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int dev = 0;
    cudaError_t e = per_device_once(pd, dev, [&](int& value) {
        cudaError_t s = cudaGetDevice(&value);
        if (s == cudaSuccess) s = cudaFuncSetAttribute(matvec_kernel<NQ, TAIL, A16>, cudaFuncAttributeMaxDynamicSharedMemorySize, MV_SMEM);
        for (int c = 1; c <= MV_MAX_SPLIT && s == cudaSuccess; ++c) {
            at.val.clusterDim = {(unsigned)c, 1, 1};
            cfg.gridDim = dim3((unsigned)c);
            s = cudaOccupancyMaxActiveClusters(&clusters[value][c], matvec_kernel<NQ, TAIL, A16>, &cfg);
        }
        return s;
    });
    if (e != cudaSuccess) return e;
    int c = 1;
    const MvPlan plan = mv_plan(mv_ring(NQ, A16), a, clusters[dev], c);
    const int per_turn = MV_WARPS / plan.wk;
    const int64_t turns = ((a.N + 127) / 128 * 4 + per_turn - 1) / per_turn;
    return launch_chained(matvec_kernel<NQ, TAIL, A16>, dim3((unsigned)(min64(turns, max(1, clusters[dev][c])) * c)), 32 * MV_WARPS, MV_SMEM,
                          (unsigned)c, stream, a, plan);
}

template <int NQ>
cudaError_t launch_aligned(const MatvecArgs& a, cudaStream_t stream) {
    if (a.K % MV_STEP == 0) return launch_nq<NQ, false, true>(a, stream);
    return a.K % 32 == 0 ? launch_nq<NQ, true, true>(a, stream) : launch_nq<NQ, true, false>(a, stream);
}

}  // namespace

// Sixteen tokens a pass over the weights: a third and fourth fragment of eight columns would not fit the registers (32
// tokens in one pass 42 us, in two 37 at 12288 x 4096), and the weights of most layers stay in L2 for the next pass.
cudaError_t launch_matvec_nvfp4(const MatvecArgs& a, cudaStream_t stream) {
    for (int m = 0; m < a.M; m += 16) {
        MatvecArgs p = a;
        p.M = a.M - m < 16 ? a.M - m : 16;
        p.x = a.x + m * a.ldx;
        p.y = a.y_fp32 ? static_cast<void*>(static_cast<float*>(a.y) + m * a.ldy) : static_cast<void*>(static_cast<uint16_t*>(a.y) + m * a.ldy);
        const cudaError_t e = p.M <= 8 ? launch_aligned<1>(p, stream) : launch_aligned<2>(p, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace mxk
