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
// A call, so that FP64 stays behind a branch: as a selection between both products it cost 600 us of 8192 x 4096's 680.
__device__ __noinline__ float times_wide(float h, double r) { return (float)((double)h * r); }
__device__ __forceinline__ void normed8(float (&f)[8], const RowNorm& n) {
    if (n.wide == 0.0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], n.r);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = times_wide(f[j], n.wide);
    }
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

// The codes of eight neighbouring elements of a row as the four lanes of a 32-block hold them (zeros beyond the row's end), and
// the block's scale byte.  All lanes of the warp call it.
__device__ __forceinline__ void quantize_row8(const NormArgs& a, int64_t row, int c, int64_t nct, const uint4& y) {
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
    if ((c & 31) == 0 && (c >> 5) < 4 * nct) a.s_row[sf_offset(row, c >> 5, nct)] = c < a.cols ? (uint8_t)s : (uint8_t)0;
}

constexpr int NR_THREADS = 256;

// Without column-wise codes: one row a group of blockDim.x threads, blockDim.y rows a CTA; NV vectors of eight elements a thread.
template <int NV, bool W32>
__global__ void __launch_bounds__(NR_THREADS) norm_rows_kernel(const NormArgs a) {
    __shared__ double sm_all[8][MAX_SEGS];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, ty = threadIdx.y;
    const int nseg = (a.cols + SEG - 1) / SEG;
    const int64_t nct = sf_col_tiles(a.cols, 32);
    if (a.q_row) {                                         // scale rows from a.rows up to a whole tile: zeros
        const int words = (int)((((a.rows + 127) & ~int64_t(127)) - a.rows) * nct);
        const int64_t me = ((int64_t)blockIdx.x * blockDim.y + ty) * blockDim.x + threadIdx.x;
        if (me < words)
            for (int i = (int)me; i < words; i += gridDim.x * blockDim.x * blockDim.y)
                *reinterpret_cast<uint32_t*>(a.s_row + sf_offset(a.rows + i / (int)nct, 4 * (i % (int)nct), nct)) = 0u;
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
            normed8(f, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], w[j]);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
        }
        if (a.q_row) quantize_row8(a, row, c, nct, y);
    }
}

// With column-wise codes: a cluster takes 32 rows, its CTAs T_SEGS segments of them each.  A warp holds whole segments of rows
// in registers (eight a thread), so the sums of squares of a segment are one butterfly; the CTAs write theirs into each other's
// shared memory and meet once.  The output goes through shared memory, where a thread finds the 8 x 8 elements whose columns
// it quantizes.
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
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer_address(const void* mine, uint32_t peer) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(peer));
    return there;
}

constexpr int TILE_ROWS = 32;
template <int SEGS>
struct TileCfg {
    static constexpr int THREADS = 128 * SEGS;             // 4 * SEGS warps, each eight of the 32 * SEGS (row, segment) pairs
    static constexpr int COLS = SEG * SEGS;
    static constexpr int TILE = TILE_ROWS * COLS * 2;      // bytes; the FP64 sums of a slow tile lie there before it is written
    static constexpr int SMEM = TILE + TILE_ROWS * MAX_SEGS * 4;
    static_assert(TILE >= TILE_ROWS * MAX_SEGS * 8, "the FP64 sums fit the tile");
};

template <int SEGS, bool W32>
__global__ void __launch_bounds__(TileCfg<SEGS>::THREADS, SEGS == 2 ? 3 : 1) norm_tile_kernel(const NormArgs a) {
    using C = TileCfg<SEGS>;
    constexpr int WARPS = C::THREADS / 32, ITEMS = 8;
    extern __shared__ __align__(16) uint8_t sm_tile[];
    float* part = reinterpret_cast<float*>(sm_tile + C::TILE);            // [32][MAX_SEGS]
    double* part_wide = reinterpret_cast<double*>(sm_tile);               // the same in FP64
    __shared__ RowNorm s_norm[TILE_ROWS];
    cluster_arrive();                                      // this CTA runs: the others may write into its shared memory
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), peers = cluster_size();
    const int nseg = (a.cols + SEG - 1) / SEG;
    const int64_t r0 = (int64_t)(blockIdx.x / peers) * TILE_ROWS;
    const int c_cta = (int)rank * C::COLS;
    // item i of a warp: row (warp + i * WARPS) / SEGS, segment (warp + i * WARPS) % SEGS of the CTA; WARPS is a multiple of SEGS
    const int seg = warp % SEGS, c = c_cta + seg * SEG + lane * 8, gseg = (int)rank * SEGS + seg;
    const bool in = c < a.cols;
    auto row_of = [&](int i) { return (warp + i * WARPS) / SEGS; };
    uint4 h[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        h[i] = make_uint4(0u, 0u, 0u, 0u);
        if (in) h[i] = load_global(reinterpret_cast<const uint4*>(a.x + (r0 + row_of(i)) * a.ldx + c));
    }
    if (a.residual && in) {
        uint4 r[ITEMS];
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) r[i] = load_global(reinterpret_cast<const uint4*>(a.residual + (r0 + row_of(i)) * a.ldr + c));
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) h[i] = add8(h[i], r[i]);
        if (a.sum)
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) *reinterpret_cast<uint4*>(a.sum + (r0 + row_of(i)) * a.lds + c) = h[i];
    }
    cluster_wait();
    const uint32_t there = (uint32_t)lane < peers ? peer_address(part, lane) : 0u;
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const float s = butterfly(squares8(h[i]));
        if ((uint32_t)lane < peers && gseg < nseg)
            asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(there + (row_of(i) * MAX_SEGS + gseg) * 4), "f"(s) : "memory");
    }
    cluster_sync();
    bool fine = true;
    for (int r = warp; r < TILE_ROWS; r += WARPS) {
        float v = lane < nseg ? part[r * MAX_SEGS + lane] : 0.0f;
        if (lane + 32 < nseg) v += part[r * MAX_SEGS + lane + 32];
        const float ss = butterfly(v);
        fine = fine && fp32_holds(ss, a.eps);
        if (lane == 0) s_norm[r] = norm_of(ss, a.inv_cols, a.eps);
    }
    if (__syncthreads_or(!fine)) {                         // the same in every CTA of the cluster: all have the same sums
        const uint32_t wide_there = (uint32_t)lane < peers ? peer_address(part_wide, lane) : 0u;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const double s = butterfly(squares8_wide(h[i]));
            if ((uint32_t)lane < peers && gseg < nseg)
                asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(wide_there + (row_of(i) * MAX_SEGS + gseg) * 8), "d"(s) : "memory");
        }
        cluster_sync();
        for (int r = warp; r < TILE_ROWS; r += WARPS) {
            float v = lane < nseg ? part[r * MAX_SEGS + lane] : 0.0f;
            double w = lane < nseg ? part_wide[r * MAX_SEGS + lane] : 0.0;
            if (lane + 32 < nseg) {
                v += part[r * MAX_SEGS + lane + 32];
                w += part_wide[r * MAX_SEGS + lane + 32];
            }
            const bool row_fine = fp32_holds(butterfly(v), a.eps);
            const double ss = butterfly(w);
            if (lane == 0 && !row_fine) s_norm[r] = norm_of_wide(ss, a.cols, a.eps);
        }
        __syncthreads();
    }
    const int64_t nct_row = sf_col_tiles(a.cols, 32);
    float w[8];
    if (in) weights8<W32>(a.w, c, w);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int r = row_of(i);
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            float f[8];
            unpack8(h[i], f);
            normed8(f, s_norm[r]);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], w[j]);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(a.y + (r0 + r) * a.ldy + c) = y;
        }
        *reinterpret_cast<uint4*>(sm_tile + (r * C::COLS + seg * SEG + lane * 8) * 2) = y;
        if (a.q_row) quantize_row8(a, r0 + r, c, nct_row, y);
    }
    __syncthreads();
    if (a.q_row && r0 + TILE_ROWS == a.rows) {             // scale rows up to a whole tile: zeros, this CTA's columns
        const int pad = (int)(((a.rows + 127) & ~int64_t(127)) - a.rows), first = c_cta / 128, last = min((int)nct_row, first + C::COLS / 128);
        for (int i = threadIdx.x; i < pad * 8; i += C::THREADS)
            for (int k = first + i % 8; k < last; k += 8)
                *reinterpret_cast<uint32_t*>(a.s_row + sf_offset(a.rows + i / 8, 4 * k, nct_row)) = 0u;
    }
    // a warp 64 columns: lane -> chunk of eight columns, quarter of eight rows
    const int chunk = lane & 7, q = lane >> 3, cc = warp * 64 + chunk * 8, gc = c_cta + cc;
    const int64_t nct = sf_col_tiles(a.rows, 32);
    const int padded_cols = (a.cols + 127) & ~127;
    if (warp * 64 >= C::COLS || c_cta + warp * 64 >= padded_cols) return;
    const bool gin = gc < a.cols;
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const uint4*>(sm_tile + ((q * 8 + i) * C::COLS + cc) * 2);
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
        if (gin)
            *reinterpret_cast<uint2*>(a.q_col + (int64_t)(gc + j) * a.rows + r0 + q * 8) =
                make_uint2(cvt_e4m3x4(f[0], f[1], f[2], f[3]), cvt_e4m3x4(f[4], f[5], f[6], f[7]));
        if (q == 0) a.s_col[sf_offset(gc + j, r0 / 32, nct)] = gin ? (uint8_t)s : (uint8_t)0;
    }
    // scale columns from rows / 32 up to a whole word: zeros
    if (r0 + TILE_ROWS == a.rows && q == 0)
        for (int64_t b = a.rows / 32; b < 4 * nct; ++b)
            for (int j = 0; j < 8; ++j) a.s_col[sf_offset(gc + j, b, nct)] = 0;
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

constexpr int NB_THREADS = 256;
constexpr int NB_CTAS = 304;                               // most partial sums of a column
// Stages of the ring: two for wide rows (four vectors a thread and more), where three would leave room for one CTA or none.
template <int NV>
constexpr int NB_STAGES = NV <= 2 ? 3 : 2;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

// A thread fetches its own vectors of the rows to come into shared memory (nobody else reads them there, so no barrier guards
// them), one or two rows ahead: the loads wait in no registers, and a row's sums do not hold up the next row's.
template <int NV, bool W32>
__global__ void __launch_bounds__(NB_THREADS) norm_backward_kernel(const NormBackwardArgs a) {
    constexpr int STAGES = NB_STAGES<NV>;
    extern __shared__ __align__(16) uint8_t sm_rows[];     // [stage][dy, h, dsum][NV][thread] of 16 bytes
    __shared__ double sm_all[2][2][MAX_SEGS];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int nseg = (a.cols + SEG - 1) / SEG, tensors = a.dsum ? 3 : 2;
    const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(sm_rows) + threadIdx.x * 16;
    const uint32_t vector = blockDim.x * 16, tensor = NV * vector, stage_bytes = tensors * tensor;
    auto col = [&](int i) { return ((warp + i * warps) * 32 + lane) * 8; };
    auto fetch = [&](int64_t row, uint32_t stage) {
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = col(i);
                if (c >= a.cols) continue;
                const uint32_t at = sm0 + stage * stage_bytes + i * vector;
                copy16(at, a.dy + row * a.lddy + c);
                copy16(at + tensor, a.h + row * a.ldh + c);
                if (a.dsum) copy16(at + 2 * tensor, a.dsum + row * a.ldds + c);
            }
        }
        copies_commit();                                   // an empty group where there is no row, so that the count goes on
    };
    auto fetched = [&](uint32_t stage, int which, int i) {
        return *reinterpret_cast<const uint4*>(sm_rows + stage * stage_bytes + which * tensor + i * vector + threadIdx.x * 16);
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) fetch(blockIdx.x + (int64_t)s * gridDim.x, s);
    float dw[NV][8] = {};
    int turn = 0;
    uint32_t stage = 0;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, turn ^= 1, stage = stage + 1 == STAGES ? 0 : stage + 1) {
        // the stage that this fills was read in the turn before, by this thread
        fetch(row + (int64_t)(STAGES - 1) * gridDim.x, stage == 0 ? STAGES - 1 : stage - 1);
        copies_wait<STAGES - 1>();
        uint4 h[NV], g[NV];
        float* sm_s = reinterpret_cast<float*>(sm_all[turn][0]);
        float* sm_c = reinterpret_cast<float*>(sm_all[turn][1]);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            h[i] = g[i] = make_uint4(0u, 0u, 0u, 0u);
            float inner = 0.0f;
            if (c < a.cols) {
                g[i] = fetched(stage, 0, i);
                h[i] = fetched(stage, 1, i);
                float x[8], d[8], w[8];
                unpack8(h[i], x);
                unpack8(g[i], d);
                weights8<W32>(a.w, c, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) inner = __fmaf_rn(__fmul_rn(d[j], w[j]), x[j], inner);
            }
            const float s = butterfly(squares8(h[i]));
            inner = butterfly(inner);
            if (lane == 0 && warp + i * warps < nseg) {
                sm_s[warp + i * warps] = s;
                sm_c[warp + i * warps] = inner;
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
            __syncthreads();                                             // the FP32 sums have been read
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = col(i);
                double inner = 0.0;
                if (c < a.cols) {
                    float x[8], d[8], w[8];
                    unpack8(h[i], x);
                    unpack8(g[i], d);
                    weights8<W32>(a.w, c, w);
#pragma unroll
                    for (int j = 0; j < 8; ++j) inner = __fma_rn((double)d[j] * (double)w[j], (double)x[j], inner);
                }
                const double s = butterfly(squares8_wide(h[i]));
                inner = butterfly(inner);
                if (lane == 0 && warp + i * warps < nseg) {
                    sm_all[turn][0][warp + i * warps] = s;
                    sm_all[turn][1][warp + i * warps] = inner;
                }
            }
            __syncthreads();
            double s_wide = 0.0, c_wide = 0.0;
            for (int s = lane; s < nseg; s += 32) {
                s_wide += sm_all[turn][0][s];
                c_wide += sm_all[turn][1][s];
            }
            n = norm_of_wide(butterfly(s_wide), a.cols, a.eps);
            mean = (float)(butterfly(c_wide) * n.wide / a.cols);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = col(i);
            if (c >= a.cols) continue;
            float x[8], d[8], w[8], o[8];
            unpack8(h[i], x);
            unpack8(g[i], d);
            weights8<W32>(a.w, c, w);
            normed8(x, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                o[j] = __fmaf_rn(-x[j], mean, __fmul_rn(d[j], w[j]));
                dw[i][j] = __fmaf_rn(d[j], x[j], dw[i][j]);
            }
            normed8(o, n);
            if (a.dsum) {
                float s[8];
                unpack8(fetched(stage, 2, i), s);
#pragma unroll
                for (int j = 0; j < 8; ++j) o[j] = __fadd_rn(o[j], s[j]);
            }
            *reinterpret_cast<uint4*>(a.dx + row * a.lddx + c) = pack8(o);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = col(i);
        if (c < a.cols) {
            float4* p = reinterpret_cast<float4*>(a.partial + (int64_t)blockIdx.x * a.cols + c);
            p[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            p[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
}

// dw[c] = the sum of `parts` partial sums: 32 columns a CTA, 32 warps a share of the parts each.
constexpr int ND_WARPS = 32;
__global__ void __launch_bounds__(32 * ND_WARPS) norm_dweight_kernel(const float* partial, int parts, int cols, float* dw) {
    __shared__ float sm[ND_WARPS][33];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    if (c < cols)
        for (int p = warp; p < parts; p += ND_WARPS) s += load_global(partial + (int64_t)p * cols + c);
    sm[warp][lane] = s;
    __syncthreads();
    s = butterfly(sm[lane][warp]);                         // a warp a column
    if (lane == 0 && blockIdx.x * 32 + warp < cols) dw[blockIdx.x * 32 + warp] = s;
}

// Vectors of eight elements a thread (1, 2, 4 or 8) such that at most `threads` take a row, and whole warps of threads.
int row_threads(int64_t cols, int threads, int& nv) {
    const int64_t vectors = (cols + 7) / 8;
    nv = 1;
    while (nv * threads < vectors) nv *= 2;
    return (int)(((vectors + nv - 1) / nv + 31) / 32 * 32);
}

template <bool W32>
cudaError_t norm_rows(const NormArgs& a, cudaStream_t stream) {
    // many rows: four vectors a thread, so that more bytes are on their way for every row's meeting of its warps; few rows: as
    // many threads a row as have work
    const bool many = a.rows >= 4 * device_sm_count();
    int nv;
    const int threads = row_threads(a.cols, many ? max(32, (int)min64(NR_THREADS, (a.cols / 32 + 31) / 32 * 32)) : NR_THREADS, nv);
    const int per = NR_THREADS / threads > 8 ? 8 : max(1, NR_THREADS / threads);
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads, per), 0, 0, stream, a);
    };
    if (nv == 1) return go(norm_rows_kernel<1, W32>);
    if (nv == 2) return go(norm_rows_kernel<2, W32>);
    if (nv == 4) return go(norm_rows_kernel<4, W32>);
    return go(norm_rows_kernel<8, W32>);
}

template <int SEGS, bool W32>
cudaError_t norm_tile(const NormArgs& a, cudaStream_t stream) {
    using C = TileCfg<SEGS>;
    auto kernel = norm_tile_kernel<SEGS, W32>;
    static PerDevice pd;
    int unused = 0;
    const cudaError_t e = per_device_once(pd, unused, [kernel](int&) {
        const cudaError_t s = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        return s != cudaSuccess ? s : cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    });
    if (e != cudaSuccess) return e;
    const unsigned cluster = (unsigned)((a.cols + C::COLS - 1) / C::COLS);
    return launch_chained(kernel, dim3((unsigned)(a.rows / TILE_ROWS) * cluster), dim3(C::THREADS), C::SMEM, cluster, stream, a);
}

template <int NV, bool W32>
cudaError_t norm_backward(const NormBackwardArgs& a, int threads, cudaStream_t stream) {
    auto kernel = norm_backward_kernel<NV, W32>;
    static PerDevice pd;
    int unused = 0;
    const cudaError_t e = per_device_once(pd, unused, [kernel](int&) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NB_STAGES<NV> * 3 * NV * NB_THREADS * 16);
    });
    if (e != cudaSuccess) return e;
    const int ctas = (int)min64(a.rows, min(NB_CTAS, (NV == 8 ? 1 : 2) * device_sm_count()));   // that run at once
    const cudaError_t e2 = launch_chained(kernel, dim3(ctas), dim3(threads), (size_t)NB_STAGES<NV> * (a.dsum ? 3 : 2) * NV * threads * 16, 0,
                                          stream, a);
    if (e2 != cudaSuccess) return e2;
    return launch_chained(norm_dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(32 * ND_WARPS), 0, 0, stream,
                          static_cast<const float*>(a.partial), ctas, a.cols, a.dw);
}

template <bool W32>
cudaError_t norm_backward(const NormBackwardArgs& a, cudaStream_t stream) {
    int nv;
    const int threads = row_threads(a.cols, NB_THREADS, nv);
    if (nv == 1) return norm_backward<1, W32>(a, threads, stream);
    if (nv == 2) return norm_backward<2, W32>(a, threads, stream);
    if (nv == 4) return norm_backward<4, W32>(a, threads, stream);
    return norm_backward<8, W32>(a, threads, stream);
}

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t* x, int64_t ldx, const uint16_t* residual, int64_t ldr, const void* w, bool w32,
                           float eps, int64_t rows, int64_t cols, uint16_t* sum, int64_t lds, uint16_t* y, int64_t ldy,
                           uint8_t* q_row, uint8_t* s_row, uint8_t* q_col, uint8_t* s_col, cudaStream_t stream) {
    const NormArgs a{x, ldx, residual, ldr, w, eps, (float)(1.0 / (double)cols), rows, (int)cols, sum, lds, y, ldy, q_row, s_row, q_col, s_col};
    if (!q_col) return w32 ? norm_rows<true>(a, stream) : norm_rows<false>(a, stream);
    // clusters of up to eight CTAs of 512 columns, or sixteen of 1024
    if (cols <= 8 * TileCfg<2>::COLS) return w32 ? norm_tile<2, true>(a, stream) : norm_tile<2, false>(a, stream);
    return w32 ? norm_tile<4, true>(a, stream) : norm_tile<4, false>(a, stream);
}

size_t rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
    return (size_t)min64(rows, NB_CTAS) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh, const void* w, bool w32,
                                    float eps, int64_t rows, int64_t cols, const uint16_t* dsum, int64_t ldds, uint16_t* dx,
                                    int64_t lddx, float* dweight, void* workspace, cudaStream_t stream) {
    const NormBackwardArgs a{dy, lddy, h, ldh, w, eps, (float)(1.0 / (double)cols), rows, (int)cols, dsum, ldds, dx, lddx, dweight,
                             static_cast<float*>(workspace)};
    return w32 ? norm_backward<true>(a, stream) : norm_backward<false>(a, stream);
}

}  // namespace mxk
