// norm.cu -- root-mean-square norm with the residual's addition and its output in MXFP8, and its gradient.
//
//   h = BF16(x + residual),  y = BF16(h r w),  r = 1 / sqrt(mean(h^2) + eps),  codes and scales of y in 32-blocks
//   dx = r (dn - n mean(dn n)) + dsum,  dw = sum over rows of dy n,  with n = h r and dn = dy w
//
// Both are bound by HBM: a few operations for the 6 to 10 bytes of an element.  Every row is read once, kept in registers as
// packed BF16 and written from there.
//
// The sum of squares has one order that depends on the row's width alone, so that a row's values are the same whichever
// outputs are asked for and in whichever batch it stands (a product in training and one in generation read the same
// codes): S_i over the 256 elements of segment i, eight elements a lane in a chain and the 32 lanes by a butterfly; then the
// segments i and i + 32 in pairs and those by a butterfly again.  Where FP32's range does not hold the squares the row is
// summed once more in FP64.
#include "../../include/mxnum.h"
#include "../../include/mxnum_layer.h"
#include "mx_internal.h"
#include "mx_chain.cuh"

namespace mxk {

namespace {

constexpr int SEG = 256;                                  // elements of a segment: 32 lanes of 8
constexpr int MAX_SEGS = MX_RMSNORM_MAX_COLS / SEG;       // 64

struct RowNorm {                                          // 1 / sqrt(mean + eps) of a row
    float r;
    double wide;                                          // used in place of r where it is not zero
};

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

template <typename T>
__device__ __forceinline__ T butterfly(T v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// BF16(a + b) of eight pairs.
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
    float x[8], y[8];
    unpack8(a, x);
    unpack8(b, y);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fadd_rn(x[i], y[i]);
    return pack8(x);
}

__device__ __forceinline__ float squares8(const uint4& v) {
    float f[8], s = 0.0f;
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __fmaf_rn(f[i], f[i], s);
    return s;
}
__device__ __forceinline__ double squares8_wide(const uint4& v) {
    float f[8];
    double s = 0.0;
    unpack8(v, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) s = __fma_rn((double)f[i], (double)f[i], s);
    return s;
}

// Whether FP32 held the squares: none beyond its range, and what its subnormals lost (at most 2^-136 over a row) is nothing
// beside the sum or eps.
__device__ __forceinline__ bool fp32_holds(float ss, float eps) {
    return ss <= FLT_MAX && (ss >= 8.27180613e-25f || eps >= 8.67361738e-19f);        // 2^-80, 2^-60
}
__device__ __forceinline__ RowNorm norm_of(float ss, float inv_cols, float eps) {
    return RowNorm{__fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(ss, inv_cols), eps))), 0.0};
}
__device__ __forceinline__ RowNorm norm_of_wide(double ss, double cols, float eps) {
    return RowNorm{0.0f, 1.0 / sqrt(ss / cols + (double)eps)};
}
__device__ __forceinline__ float normed(float h, const RowNorm& n) {
    return n.wide == 0.0 ? __fmul_rn(h, n.r) : (float)((double)h * n.wide);
}

// Eight weights from column c on.
template <bool W32>
__device__ __forceinline__ void weights8(const void* w, int c, float (&f)[8]) {
    if (W32) {
        const float4 a = load_global(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c));
        const float4 b = load_global(reinterpret_cast<const float4*>(static_cast<const float*>(w) + c) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c)), f);
    }
}

// The threads of one row (a whole number of warps) meet; rows of a CTA are numbered from 0.
__device__ __forceinline__ void row_sync(int row, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(row + 1), "r"(threads) : "memory");
}

// The sum over a row of per-lane parts, part[i] of segment warp + i * warps: in shared memory sm[segments], in the fixed order.
template <int NV, typename T>
__device__ __forceinline__ T row_sum(const T (&part)[NV], T* sm, int row, int threads, int nseg) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = threads >> 5;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const T s = butterfly(part[i]);
        if (lane == 0 && warp + i * warps < nseg) sm[warp + i * warps] = s;
    }
    row_sync(row, threads);
    T v = lane < nseg ? sm[lane] : T(0);
    if (lane + 32 < nseg) v += sm[lane + 32];
    return butterfly(v);
}

struct NormArgs {
    const uint16_t* x; int64_t ldx;
    const uint16_t* residual; int64_t ldr;
    const void* w;
    float eps, inv_cols;
    int64_t rows; int cols;
    uint16_t* sum; int64_t lds;
    uint16_t* y; int64_t ldy;
    uint8_t *q_row, *s_row, *q_col, *s_col;
};

// One row a group of blockDim.x threads, blockDim.y rows a CTA; NV vectors of eight elements a thread.
template <int NV, bool W32>
__global__ void __launch_bounds__(1024) norm_rows_kernel(const NormArgs a) {
    __shared__ double sm_all[8][MAX_SEGS];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, ty = threadIdx.y;
    const int nseg = (a.cols + SEG - 1) / SEG;
    const int64_t nct = sf_col_tiles(a.cols, 32);
    if (a.q_row) {                                         // scale rows from a.rows up to a whole tile: zeros
        const int64_t words = (((a.rows + 127) & ~int64_t(127)) - a.rows) * nct;
        const int64_t me = ((int64_t)blockIdx.x * blockDim.y + ty) * blockDim.x + threadIdx.x;
        for (int64_t i = me; i < words; i += (int64_t)gridDim.x * blockDim.x * blockDim.y)
            *reinterpret_cast<uint32_t*>(a.s_row + sf_offset(a.rows + i / nct, 4 * (i % nct), nct)) = 0u;
    }
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + ty;
    if (row >= a.rows) return;
    uint4 h[NV];
    float part[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = ((warp + i * warps) * 32 + lane) * 8;
        h[i] = make_uint4(0u, 0u, 0u, 0u);
        if (c < a.cols) {
            h[i] = load_global(reinterpret_cast<const uint4*>(a.x + row * a.ldx + c));
            if (a.residual) h[i] = add8(h[i], load_global(reinterpret_cast<const uint4*>(a.residual + row * a.ldr + c)));
            if (a.sum) *reinterpret_cast<uint4*>(a.sum + row * a.lds + c) = h[i];
        }
        part[i] = squares8(h[i]);
    }
    const float ss = row_sum(part, reinterpret_cast<float*>(sm_all[ty]), ty, blockDim.x, nseg);
    RowNorm n = norm_of(ss, a.inv_cols, a.eps);
    if (!fp32_holds(ss, a.eps)) {                          // the same for all threads of the row
        double wide[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) wide[i] = squares8_wide(h[i]);
        row_sync(ty, blockDim.x);                          // the FP32 sums have been read
        n = norm_of_wide(row_sum(wide, sm_all[ty], ty, blockDim.x, nseg), a.cols, a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = ((warp + i * warps) * 32 + lane) * 8;
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (c < a.cols) {
            float f[8], w[8];
            unpack8(h[i], f);
            weights8<W32>(a.w, c, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(normed(f[j], n), w[j]);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
        }
        if (a.q_row) {
            // a block of 32 is four lanes'; those beyond the row's end hold zeros
            uint32_t m = absmax_bf16x2(absmax_bf16x2(y.x, y.y), absmax_bf16x2(y.z, y.w));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
            m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
            const uint32_t s = e8m0_from_amax_bits(fold_halves(m));
            const float inv = inv_scale_from_e8m0(s);
            if (c < a.cols) {
                float f[8];
                unpack8(y, f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], inv);
                *reinterpret_cast<uint2*>(a.q_row + row * a.cols + c) =
                    make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
            }
            if ((lane & 3) == 0 && (c >> 5) < 4 * nct) a.s_row[sf_offset(row, c >> 5, nct)] = c < a.cols ? (uint8_t)s : (uint8_t)0;
        }
    }
}

// Column-wise codes of 32 rows a CTA: a first pass over the rows for their sums, a warp a row, a second one for the codes.
constexpr int NC_THREADS = 256;
template <bool W32>
__global__ void __launch_bounds__(NC_THREADS) norm_cols_kernel(const NormArgs a) {
    __shared__ float sm_r[32];
    __shared__ double sm_wide[32];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t r0 = (int64_t)blockIdx.x * 32;
    auto load_h = [&](int64_t row, int c) {
        uint4 h = load_global(reinterpret_cast<const uint4*>(a.x + row * a.ldx + c));
        if (a.residual) h = add8(h, load_global(reinterpret_cast<const uint4*>(a.residual + row * a.ldr + c)));
        return h;
    };
    const int nseg = (a.cols + SEG - 1) / SEG;
    for (int r = warp; r < 32; r += NC_THREADS / 32) {
        float mine = 0.0f;
        for (int s = 0; s < nseg; ++s) {
            const int c = s * SEG + lane * 8;
            const float v = butterfly(c < a.cols ? squares8(load_h(r0 + r, c)) : 0.0f);
            if (lane == (s & 31)) mine += v;
        }
        const float ss = butterfly(mine);
        RowNorm n = norm_of(ss, a.inv_cols, a.eps);
        if (!fp32_holds(ss, a.eps)) {
            double wide = 0.0;
            for (int s = 0; s < nseg; ++s) {
                const int c = s * SEG + lane * 8;
                const double v = butterfly(c < a.cols ? squares8_wide(load_h(r0 + r, c)) : 0.0);
                if (lane == (s & 31)) wide += v;
            }
            n = norm_of_wide(butterfly(wide), a.cols, a.eps);
        }
        if (lane == 0) {
            sm_r[r] = n.r;
            sm_wide[r] = n.wide;
        }
    }
    __syncthreads();
    // a warp 64 columns: lane -> chunk of eight columns, quarter of eight rows
    const int chunk = lane & 7, q = lane >> 3;
    const int64_t nct = sf_col_tiles(a.rows, 32), padded_cols = (a.cols + 127) & ~127;
    for (int c0 = warp * 64; c0 < padded_cols; c0 += NC_THREADS * 2) {
        const int c = c0 + chunk * 8;
        const bool in = c < a.cols;
        uint4 v[8];
        float w[8];
        if (in) weights8<W32>(a.w, c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (in) {
                const RowNorm n{sm_r[q * 8 + i], sm_wide[q * 8 + i]};
                float f[8];
                unpack8(load_h(r0 + q * 8 + i, c), f);
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(normed(f[j], n), w[j]);
                v[i] = pack8(f);
            }
        }
        uint32_t m[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
        for (int i = 1; i < 8; ++i) {
            m[0] = absmax_bf16x2(m[0], v[i].x); m[1] = absmax_bf16x2(m[1], v[i].y);
            m[2] = absmax_bf16x2(m[2], v[i].z); m[3] = absmax_bf16x2(m[3], v[i].w);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            m[k] = absmax_bf16x2(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], 8));
            m[k] = abs_halves(absmax_bf16x2(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], 16)));
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t s = e8m0_from_amax_bits((j & 1) ? (m[j >> 1] >> 16) : (m[j >> 1] & 0xFFFFu));
            const float inv = inv_scale_from_e8m0(s);
            float f[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t word = (j >> 1) == 0 ? v[i].x : ((j >> 1) == 1 ? v[i].y : ((j >> 1) == 2 ? v[i].z : v[i].w));
                f[i] = __fmul_rn((j & 1) ? bf16_hi(word) : bf16_lo(word), inv);
            }
            if (in)
                *reinterpret_cast<uint2*>(a.q_col + (int64_t)(c + j) * a.rows + r0 + q * 8) =
                    make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
            if (q == 0) a.s_col[sf_offset(c + j, r0 / 32, nct)] = in ? (uint8_t)s : (uint8_t)0;
        }
        // scale columns from rows / 32 up to a whole word: zeros, from the last rows' CTA
        if (r0 + 32 == a.rows && q == 0)
            for (int64_t b = a.rows / 32; b < 4 * nct; ++b)
                for (int j = 0; j < 8; ++j) a.s_col[sf_offset(c + j, b, nct)] = 0;
    }
}

// ------------------------------------------------------------------------------------------------
// Gradient.  A CTA walks rows; each thread keeps the sums of dw for its columns in registers, and the CTAs' sums meet in the
// workspace, where a second kernel adds them in the order of the CTAs.
// ------------------------------------------------------------------------------------------------
struct NormBackwardArgs {
    const uint16_t* dy; int64_t lddy;
    const uint16_t* h; int64_t ldh;
    const void* w;
    float eps, inv_cols;
    int64_t rows; int cols;
    const uint16_t* dsum; int64_t ldds;
    uint16_t* dx; int64_t lddx;
    float *dw, *partial;
};

constexpr int NB_CTAS = 304;                               // most partial sums of a column

template <int NV, bool W32>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormBackwardArgs a) {
    __shared__ double sm_all[2][2][MAX_SEGS];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nseg = (a.cols + SEG - 1) / SEG;
    float dw[NV][8] = {};
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1) {
        uint4 h[NV], g[NV];
        float squares[NV], inner[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = ((warp + i * warps) * 32 + lane) * 8;
            h[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
            inner[i] = 0.0f;
            if (c < a.cols) {
                h[i] = load_global(reinterpret_cast<const uint4*>(a.h + row * a.ldh + c));
                g[i] = load_global(reinterpret_cast<const uint4*>(a.dy + row * a.lddy + c));
                float x[8], d[8], w[8];
                unpack8(h[i], x);
                unpack8(g[i], d);
                weights8<W32>(a.w, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) inner[i] = __fmaf_rn(__fmul_rn(d[j], w[j]), x[j], inner[i]);
            }
            squares[i] = squares8(h[i]);
        }
        float* sm_s = reinterpret_cast<float*>(sm_all[turn][0]);
        float* sm_c = reinterpret_cast<float*>(sm_all[turn][1]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float s = butterfly(squares[i]), c = butterfly(inner[i]);
            if (lane == 0 && warp + i * warps < nseg) {
                sm_s[warp + i * warps] = s;
                sm_c[warp + i * warps] = c;
            }
        }
        __syncthreads();
        float ss = lane < nseg ? sm_s[lane] : 0.0f, cc = lane < nseg ? sm_c[lane] : 0.0f;
        if (lane + 32 < nseg) {
            ss += sm_s[lane + 32];
            cc += sm_c[lane + 32];
        }
        ss = butterfly(ss);
        cc = butterfly(cc);
        RowNorm n = norm_of(ss, a.inv_cols, a.eps);
        float mean = __fmul_rn(__fmul_rn(cc, a.inv_cols), n.r);          // mean(dn n)
        // the products dn h likewise: too large, or so small that subnormals would decide (where eps does not)
        if (!fp32_holds(ss, a.eps) || !(fabsf(cc) <= FLT_MAX) || (fabsf(cc) < 7.88860905e-31f && a.eps < 9.09494702e-13f)) {
            double s_wide = 0.0, c_wide = 0.0;
            __syncthreads();                                             // the FP32 sums have been read
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = ((warp + i * warps) * 32 + lane) * 8;
                double inner_wide = 0.0;
                if (c < a.cols) {
                    float x[8], d[8], w[8];
                    unpack8(h[i], x);
                    unpack8(g[i], d);
                    weights8<W32>(a.w, c, w);
                    for (int j = 0; j < 8; ++j) inner_wide = __fma_rn((double)d[j] * (double)w[j], (double)x[j], inner_wide);
                }
                const double s = butterfly(squares8_wide(h[i])), cs = butterfly(inner_wide);
                if (lane == 0 && warp + i * warps < nseg) {
                    sm_all[turn][0][warp + i * warps] = s;
                    sm_all[turn][1][warp + i * warps] = cs;
                }
            }
            __syncthreads();
            for (int s = lane; s < nseg; s += 32) {
                s_wide += sm_all[turn][0][s];
                c_wide += sm_all[turn][1][s];
            }
            n = norm_of_wide(butterfly(s_wide), a.cols, a.eps);
            mean = (float)(butterfly(c_wide) * n.wide / a.cols);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = ((warp + i * warps) * 32 + lane) * 8;
            if (c < a.cols) {
                float x[8], d[8], w[8], o[8];
                unpack8(h[i], x);
                unpack8(g[i], d);
                weights8<W32>(a.w, c, w);
                if (a.dsum) unpack8(load_global(reinterpret_cast<const uint4*>(a.dsum + row * a.ldds + c)), o);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float nj = normed(x[j], n);
                    const float t = __fmaf_rn(-nj, mean, __fmul_rn(d[j], w[j]));
                    float v = n.wide == 0.0 ? __fmul_rn(n.r, t) : (float)(n.wide * (double)t);
                    if (a.dsum) v = __fadd_rn(v, o[j]);
                    o[j] = v;
                    dw[i][j] = __fmaf_rn(d[j], nj, dw[i][j]);
                }
                *reinterpret_cast<uint4*>(a.dx + row * a.lddx + c) = pack8(o);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = ((warp + i * warps) * 32 + lane) * 8;
        if (c < a.cols) {
            float4* p = reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.cols + c);
            p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dw[c] = the sum of `parts` partial sums: 32 columns a CTA, eight warps a share of the parts each.
__global__ void __launch_bounds__(256) norm_dweight_kernel(const float* partial, int parts, int cols, float* dw) {
    __shared__ float sm[8][32];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < cols)
        for (int p = warp; p < parts; p += 8) s += load_global(partial + (int64_t)p * cols + c);
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sm[i][lane];
        dw[c] = s;
    }
}

// Threads of a row: whole warps, eight elements a thread, two vectors a thread for the widest rows.
int row_threads(int64_t cols, int& nv) {
    const int64_t vectors = (cols + 7) / 8;
    nv = vectors > 1024 ? 2 : 1;
    return (int)(((vectors + nv - 1) / nv + 31) / 32 * 32);
}

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr, const void* w, bool w32,
                           float eps, int64_t rows, int64_t cols, uint16_t* sum, int64_t lds, uint16_t* y, int64_t ldy,
                           uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, cudaStream_t stream) {
    NormArgs a{x, ldx, residual, ldr, w, eps, (float)(1.0 / (double)cols), rows, (int)cols, sum, lds, y, ldy, q_row, s_row, q_col, s_col};
    if (q_row || y || sum) {
        int nv;
        const int threads = row_threads(cols, nv);
        const int per = threads >= 256 ? 1 : min(8, 256 / threads);
        void (*k)(const NormArgs) = nv == 1 ? (w32 ? norm_rows_kernel<1, true> : norm_rows_kernel<1, false>)
                                            : (w32 ? norm_rows_kernel<2, true> : norm_rows_kernel<2, false>);
        cudaError_t e = launch_chained(k, dim3((unsigned)((rows + per - 1) / per)), dim3(threads, per), 0, 0, stream, a);
        if (e != cudaSuccess) return e;
        if (sum) {                                         // it may have replaced x or the residual
            a.x = sum;
            a.ldx = lds;
            a.residual = nullptr;
        }
    }
    if (q_col)
        return launch_chained(w32 ? norm_cols_kernel<true> : norm_cols_kernel<false>, dim3((unsigned)(rows / 32)), dim3(NC_THREADS), 0, 0,
                              stream, a);
    return cudaSuccess;
}

size_t rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)min64(rows, NB_CTAS) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh, const void* w, bool w32,
                                    float eps, int64_t rows, int64_t cols, const uint16_t* dsum, int64_t ldds, uint16_t* dx,
                                    int64_t lddx, float* dweight, void* workspace, cudaStream_t stream) {
    const NormBackwardArgs a{dy, lddy, h, ldh, w, eps, (float)(1.0 / (double)cols), rows, (int)cols, dsum, ldds, dx, lddx, dweight,
                             static_cast<float*>(workspace)};
    int nv;
    const int threads = row_threads(cols, nv);
    const int ctas = (int)min64(rows, min(NB_CTAS, 2 * device_sm_count()));
    void (*k)(const NormBackwardArgs) = nv == 1 ? (w32 ? norm_backward_kernel<1, true> : norm_backward_kernel<1, false>)
                                                : (w32 ? norm_backward_kernel<2, true> : norm_backward_kernel<2, false>);
    const cudaError_t e = launch_chained(k, dim3(ctas), dim3(threads), 0, 0, stream, a);
    if (e != cudaSuccess) return e;
    return launch_chained(norm_dweight_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(256), 0, 0, stream,
                          static_cast<const float*>(workspace), ctas, (int)cols, dweight);
}

}  // namespace mxk
