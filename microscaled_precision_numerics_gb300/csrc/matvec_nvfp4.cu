// matvec_nvfp4.cu -- products of a few tokens with NVFP4 weights (the linear layers of a generation step).
//
//   y[m, n] = s2[n or 0] * sum_k x[m, k] * val(q[n, k]) * val(bs[n, k / 16])
//
// Bound: the weights are read once, 0.5625 bytes a value, and each value meets M tokens; up to 16 tokens the HBM
// copy rate is the floor.  What has to keep up is the expansion of the codes: 128 values a thread cost 64
// conversions and 64 multiplications by the block scale (2 clocks a warp each), inside the 396 clocks that the copy rate
// leaves a quarter of an SM for the 2304 bytes of a warp's step.
//
// Weight rows are the rows (M) of mma.m16n8k16 and tokens its columns, eight to a fragment.  val(q) * val(bs) has at
// most 6 significant bits and is exact in FP16.  x enters as FP16 scaled by a power of two per token (its largest
// element of the stretch in [2^15, 2^16)): exact down to 2^-29 of that, an absolute error of 2^-40 of it below.
//
// A warp takes 32 rows, 8 consecutive ones in each of the four 32-row bands of a 128-row scale tile: the 16 bytes that the
// GEMM scale layout holds for a row of the first band are the four bands' scales of the same four columns, so no
// scale sector is fetched for a quarter of its bytes.  In a step of 128 values a thread reads 16 bytes of codes from
// each of its four rows (a quad: 64 contiguous bytes) and one 16-byte piece of scales.
// CTA: 128 rows, four warps across them and two along K.  The CTAs of a cluster split K further and add up through
// distributed shared memory in rank order: no workspace, no second launch, and the sum does not depend on timing.
#include "mx_internal.h"
#include "mx_fragment.cuh"

namespace mxk {

namespace {

constexpr int MV_THREADS = 256;
constexpr int MV_ROWS = 128;
constexpr int MV_STEP = 128;                          // values of K a step
__host__ __device__ constexpr int mv_chunk(int NQ) { return NQ <= 2 ? 2048 : 4096 / NQ; }            // values of K staged at once
__host__ __device__ constexpr int mv_row_bytes(int NQ) { return mv_chunk(NQ) * 2 + 64; }            // 64: odd and even tokens on both bank halves
__host__ __device__ constexpr int mv_smem(int NQ) { return 8 * NQ * mv_row_bytes(NQ); }

struct Step {
    uint4 q[4];                                       // codes of the four rows
    uint4 s;                                          // scales: word b of band b, four columns
};

template <bool A16>
__device__ __forceinline__ uint4 load_codes(const uint8_t* p, int left) {
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (A16) {
        if (left > 0) v = __ldcs(reinterpret_cast<const uint4*>(p));
    } else {                                          // rows on 8 bytes only: K % 32 == 16
        uint2 a = make_uint2(0u, 0u), b = a;
        if (left > 0) a = __ldcs(reinterpret_cast<const uint2*>(p));
        if (left > 16) b = __ldcs(reinterpret_cast<const uint2*>(p) + 1);
        v = make_uint4(a.x, a.y, b.x, b.y);
    }
    return v;
}

template <int NQ, bool A16>
__global__ void __launch_bounds__(MV_THREADS, NQ <= 2 ? 2 : 1) matvec_kernel(const __grid_constant__ MatvecArgs a) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int s_e[8 * NQ];                       // biased exponent that the tokens are scaled by
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t4 = lane & 3;
    const int wr = warp & 3, wk = warp >> 2;
    uint32_t rank, ranks;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ranks));
    const int64_t band = blockIdx.x / ranks;
    const int steps = (int)((a.K + MV_STEP - 1) / MV_STEP);
    const int cta0 = (int)((int64_t)steps * rank / ranks), cta1 = (int)((int64_t)steps * (rank + 1) / ranks);
    const int64_t nct = sf_col_tiles(a.K, 16);

    const uint8_t* row[4];
#pragma unroll
    for (int b = 0; b < 4; ++b) row[b] = a.q + min64(a.N - 1, band * MV_ROWS + 32 * b + 8 * wr + g) * (a.K / 2) + t4 * 16;
    const uint8_t* scales = a.s + (band * nct << 9) + ((8 * wr + g) << 4);
    auto fetch = [&](int step, Step& st) {
        const int left = (int)(a.K - (int64_t)step * MV_STEP) - t4 * 32;         // valid values of the thread's 32
#pragma unroll
        for (int b = 0; b < 4; ++b) st.q[b] = load_codes<A16>(row[b] + (int64_t)step * (MV_STEP / 2), left);
        st.s = make_uint4(0u, 0u, 0u, 0u);
        if (left > 0) st.s = __ldcs(reinterpret_cast<const uint4*>(scales + ((2 * (int64_t)step + (t4 >> 1)) << 9)));
        if (left == 16) {                             // the second block's scale is padding
            const uint32_t keep = (t4 & 1) ? 0x00FF0000u : 0x000000FFu;
            st.s.x &= keep; st.s.y &= keep; st.s.z &= keep; st.s.w &= keep;
        }
    };

    float acc[2][NQ][4] = {};
    int scaled[NQ][2];                                // exponents that acc's columns carry
    constexpr int CH = mv_chunk(NQ) / MV_STEP;
    for (int c0 = cta0; c0 < cta1; c0 += CH) {
        const int c1 = min(cta1, c0 + CH), half = (c1 - c0 + 1) / 2;
        const int k0 = c0 + wk * half, k1 = min(c1, k0 + half);
        Step st[2];
        if (k0 < k1) fetch(k0, st[0]);                // on their way while x is staged
        if (k0 + 1 < k1) fetch(k0 + 1, st[1]);

        // ---- x of this stretch as FP16: a warp takes a token at a time
        if (c0 > cta0) __syncthreads();               // the previous stretch is done with
        constexpr int UNITS = mv_chunk(NQ) / 8 / 32;  // 8-value units a lane
        const int n_units = (c1 - c0) * (MV_STEP / 8);
        for (int m = warp; m < 8 * NQ; m += MV_THREADS / 32) {
            uint4 x[UNITS];
            uint32_t amax = 0;
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int unit = lane + 32 * u;
                const int64_t k = (int64_t)c0 * MV_STEP + unit * 8;
                x[u] = make_uint4(0u, 0u, 0u, 0u);
                if (m < a.M && unit < n_units && k < a.K) x[u] = __ldg(reinterpret_cast<const uint4*>(a.x + m * a.ldx + k));
            }
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
                    amax = max(amax, lo < 0x7F80u ? lo : 0u);                    // infinities and NaN go through as they are
                    amax = max(amax, hi < 0x7F80u ? hi : 0u);
                }
            }
            amax = __reduce_max_sync(0xFFFFFFFFu, amax);
            // x * 2^(142 - e); e never falls from one stretch to the next, so the sums only ever scale down
            const int e = max(max((int)(amax >> 7), 27), c0 > cta0 ? s_e[m] : 0);
            const float up = __uint_as_float((uint32_t)(127 + 142 - e) << 23);
#pragma unroll
            for (int u = 0; u < UNITS; ++u) {
                const int unit = lane + 32 * u;
                if (unit >= n_units) break;
                const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                uint32_t f[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) f[i] = pack_f16x2(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
                // unit i of thread t4's four inside a step goes to place i * 4 + t4: a quad reads 64 contiguous bytes
                const int place = (unit & ~15) + (unit & 3) * 4 + ((unit >> 2) & 3);
                *reinterpret_cast<uint4*>(smem + m * mv_row_bytes(NQ) + place * 16) = make_uint4(f[0], f[1], f[2], f[3]);
            }
            __syncwarp();
            if (lane == 0) s_e[m] = e;
        }
        __syncthreads();
#pragma unroll
        for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int e = s_e[nq * 8 + 2 * t4 + j];
                if (c0 > cta0) {
                    const float f = __uint_as_float((uint32_t)max(0, 127 + scaled[nq][j] - e) << 23);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        acc[t][nq][j] *= f;
                        acc[t][nq][2 + j] *= f;
                    }
                }
                scaled[nq][j] = e;
            }

        auto multiply = [&](int step, const Step& w) {
            const uint8_t* xs = smem + g * mv_row_bytes(NQ) + (step - c0) * (MV_STEP * 2) + t4 * 16;
            const uint32_t sw[4] = {w.s.x, w.s.y, w.s.z, w.s.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {             // 8 of the thread's 32 values: two k-steps
                uint4 xb[NQ];
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq) xb[nq] = *reinterpret_cast<const uint4*>(xs + nq * 8 * mv_row_bytes(NQ) + i * 64);
                uint32_t f[4][4];
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    const uint32_t codes = i == 0 ? w.q[b].x : (i == 1 ? w.q[b].y : (i == 2 ? w.q[b].z : w.q[b].w));
                    e2m1x8_to_f16(codes, f[b]);
                    // column 2 (t4 & 1) + i / 2 of the four, in both halves
                    const uint32_t sc = e4m3x2_to_f16x2(__byte_perm(sw[b], 0u, 0x1111u * (2 * (t4 & 1) + (i >> 1))));
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[b][j] = mul_f16x2(f[b][j], sc);
                }
#pragma unroll
                for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        mma_16816(acc[t][nq], f[2 * t][0], f[2 * t + 1][0], f[2 * t][1], f[2 * t + 1][1], xb[nq].x, xb[nq].y);
                        mma_16816(acc[t][nq], f[2 * t][2], f[2 * t + 1][2], f[2 * t][3], f[2 * t + 1][3], xb[nq].z, xb[nq].w);
                    }
            }
        };
        for (int k = k0; k < k1; k += 2) {
            multiply(k, st[0]);
            if (k + 2 < k1) fetch(k + 2, st[0]);
            if (k + 1 < k1) {
                multiply(k + 1, st[1]);
                if (k + 3 < k1) fetch(k + 3, st[1]);
            }
        }
    }

    // ---- the sums: two warps along K, then the cluster's CTAs, [token][row] in shared memory
    __syncthreads();
    float* sum = reinterpret_cast<float*>(smem);      // [8 NQ][MV_ROWS]
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
        if (wk == pass) {
#pragma unroll
            for (int nq = 0; nq < NQ; ++nq)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int m = nq * 8 + 2 * t4 + (j & 1);
                        float* d = sum + m * MV_ROWS + 32 * (2 * t + (j >> 1)) + 8 * wr + g;
                        const float v = acc[t][nq][j];
                        *d = pass == 0 ? v : (*d + v);
                    }
        }
        __syncthreads();
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
    const uint32_t sum_u32 = (uint32_t)__cvta_generic_to_shared(sum), e_u32 = (uint32_t)__cvta_generic_to_shared(s_e);
    for (int i = tid + (int)rank * MV_THREADS; i < a.M * MV_ROWS; i += MV_THREADS * (int)ranks) {
        const int m = i / MV_ROWS, rr = i % MV_ROWS;
        float y = 0.0f;
        for (uint32_t c = 0; c < ranks; ++c) {
            uint32_t at, at_e;
            float v;
            int e;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(sum_u32 + 4 * i), "r"(c));
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at_e) : "r"(e_u32 + 4 * m), "r"(c));
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(e) : "r"(at_e) : "memory");
            y += v * __uint_as_float((uint32_t)(e - 15) << 23);
        }
        const int64_t n = band * MV_ROWS + rr;
        if (n >= a.N) continue;
        y *= __ldg(a.s2 + (a.s2_per_row ? n : 0));
        if (a.y_fp32) static_cast<float*>(a.y)[m * a.ldy + n] = y;
        else static_cast<uint16_t*>(a.y)[m * a.ldy + n] = (uint16_t)pack_bf16x2(y, 0.0f);
    }
    asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// CTAs along K: the split whose slowest wave of CTAs is shortest, counting a CTA's fixed cost as four steps.
int mv_split(int64_t bands, int steps, int slots) {
    int best = 1;
    double least = 1e30;
    for (int c = 1; c <= 8 && 2 * c <= max(2, steps); ++c) {
        const double waves = (double)((bands * c + slots - 1) / slots);
        const double cost = waves * ((double)((steps + 2 * c - 1) / (2 * c)) + 4.0);
        if (cost < least) {
            least = cost;
            best = c;
        }
    }
    return best;
}

template <int NQ, bool A16>
cudaError_t launch_nq(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    static PerDevice pd;
    int resident = 0;
    cudaError_t e = per_device_once(pd, resident, [](int& value) {
        const cudaError_t s = cudaFuncSetAttribute(matvec_kernel<NQ, A16>, cudaFuncAttributeMaxDynamicSharedMemorySize, mv_smem(NQ));
        return s != cudaSuccess ? s : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&value, matvec_kernel<NQ, A16>, MV_THREADS, mv_smem(NQ));
    });
    if (e != cudaSuccess) return e;
    const int64_t bands = (a.N + MV_ROWS - 1) / MV_ROWS;
    const int c = mv_split(bands, (int)((a.K + MV_STEP - 1) / MV_STEP), num_sms * max(1, resident));
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(bands * c));
    cfg.blockDim = dim3(MV_THREADS);
    cfg.dynamicSmemBytes = mv_smem(NQ);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim = {(unsigned)c, 1, 1};
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, matvec_kernel<NQ, A16>, a);
}

template <int NQ>
cudaError_t launch_aligned(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    return a.K % 32 == 0 ? launch_nq<NQ, true>(a, num_sms, stream) : launch_nq<NQ, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_matvec_nvfp4(const MatvecArgs& a, int num_sms, cudaStream_t stream) {
    if (a.M <= 8) return launch_aligned<1>(a, num_sms, stream);
    if (a.M <= 16) return launch_aligned<2>(a, num_sms, stream);
    if (a.M <= 32) return launch_aligned<4>(a, num_sms, stream);
    return launch_aligned<8>(a, num_sms, stream);
}

}  // namespace mxk
