// matvec_nvfp4.cu -- products of a few tokens with NVFP4 weights (the linear layers of a generation step).
//
//   y[m, n] = s2[n or 0] * sum_k x[m, k] * val(q[n, k]) * val(bs[n, k / 16])
#include "mx_internal.h"

namespace mxk {

namespace {

// A warp for each output row: its lanes take the row's 16-blocks in turn, eight tokens at a time.
__global__ void __launch_bounds__(256) matvec_simple_kernel(const MatvecArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (n >= a.N) return;
    const int64_t nct = sf_col_tiles(a.K, 16);
    for (int m0 = 0; m0 < a.M; m0 += 8) {
        float acc[8] = {};
        for (int64_t b = lane; b < a.K / 16; b += 32) {
            const uint2 c = __ldg(reinterpret_cast<const uint2*>(a.q + n * (a.K / 2) + b * 8));
            const float bs = e4m3_to_f32(__ldg(a.s + sf_offset(n, b, nct)));
            float w[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const uint32_t p = e2m1x2_to_f16x2(((j < 4 ? c.x : c.y) >> (8 * (j & 3))) & 0xFFu);
                w[2 * j] = __half2float(__ushort_as_half((unsigned short)(p & 0xFFFFu))) * bs;
                w[2 * j + 1] = __half2float(__ushort_as_half((unsigned short)(p >> 16))) * bs;
            }
#pragma unroll
            for (int m = 0; m < 8; ++m) {
                if (m0 + m >= a.M) break;
                const uint16_t* x = a.x + (m0 + m) * a.ldx + b * 16;
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[m] = fmaf(__uint_as_float((uint32_t)__ldg(x + j) << 16), w[j], acc[m]);
            }
        }
        const float s2 = __ldg(a.s2 + (a.s2_per_row ? n : 0));
#pragma unroll
        for (int m = 0; m < 8; ++m) {
            for (int o = 16; o > 0; o >>= 1) acc[m] += __shfl_xor_sync(0xFFFFFFFFu, acc[m], o);
            if (lane != 0 || m0 + m >= a.M) continue;
            const float y = acc[m] * s2;
            if (a.y_fp32) static_cast<float*>(a.y)[(m0 + m) * a.ldy + n] = y;
            else static_cast<uint16_t*>(a.y)[(m0 + m) * a.ldy + n] = (uint16_t)pack_bf16x2(y, 0.0f);
        }
    }
}

}  // namespace

cudaError_t launch_matvec_nvfp4(const MatvecArgs& a, int, cudaStream_t stream) {
    matvec_simple_kernel<<<(unsigned)((a.N + 7) / 8), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace mxk
