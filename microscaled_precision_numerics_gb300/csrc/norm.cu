// norm.cu -- root-mean-square norm with the residual's addition and its output in MXFP8, and its gradient.
//
//   h = BF16(x + residual),  y = BF16(h w r),  r = 1 / sqrt(mean(h^2) + eps),  codes and scales of y in 32-blocks
//   dx = r (dn - n mean(dn n)) + dsum,  dw = sum over rows of dy n,  with n = h r and dn = dy w
//
// Both are close to HBM's rate and to the issue rate at once: 6 to 10 bytes of an element, and some twenty instructions.  Every
// element is read once and waits as packed BF16, in registers or shared memory.
//
// The sum of squares has one order that depends on the row's width alone, so that a row's values are the same whichever
// outputs are asked for and in whichever batch it stands (a product in training and one in generation read the same
// codes): S_i over the 256 elements of segment i, the even and the odd ones of a lane's eight in two chains and the 32 lanes by a
// butterfly; then the segments i and i + 32 in pairs and those by a butterfly again.  Where FP32's range does not hold the squares the row is
// summed once more in FP64.
#include "../../include/mxnum.h"
#include "../../include/mxnum_layer.h"
#include "mx_internal.h"
#include "mx_chain.cuh"

#include <type_traits>

namespace mxk {

namespace {

constexpr int SEG = 256;                                  // elements of a segment: 32 lanes of 8
constexpr int MAX_SEGS = MX_RMSNORM_MAX_COLS / SEG;       // 64

struct RowNorm {                                          // 1 / sqrt(mean + eps) of a row as p * r
    float p;                                              // a power of two, 1 unless the row was summed in FP64
    float r;
};

using Pairs = uint64_t[4];                                // eight FP32 values as packed pairs
__device__ __forceinline__ void unpack8(const uint4& v, Pairs& f) {
    f[0] = f2_pack(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = f2_pack(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = f2_pack(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = f2_pack(bf16_lo(v.w), bf16_hi(v.w));
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return pack_bf16x2(lo, hi);
}
__device__ __forceinline__ uint4 pack8(const Pairs& f) {
    return make_uint4(pack_pair(f[0]), pack_pair(f[1]), pack_pair(f[2]), pack_pair(f[3]));
}
__device__ __forceinline__ void times8(Pairs& f, float s) {
    const uint64_t ss = f2_pack(s, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = f2_mul(f[i], ss);
}
__device__ __forceinline__ uint32_t cvt_e4m3_pairs(uint64_t a, uint64_t b) {
    float a0, a1, b0, b1;
    f2_unpack(a, a0, a1);
    f2_unpack(b, b0, b1);
    return cvt_e4m3x4(a0, a1, b0, b1);
}

// The sum over the LANES neighbouring lanes of a group.
template <int LANES = 32, typename T>
__device__ __forceinline__ T butterfly(T v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

// The butterfly sums of N values of every lane at once (N = 1, 2, 4, 8): lane l gets that of value l / (32 / N).  As long as
// a lane has more than one it keeps half of them and gives the other half to its partner, so eight sums take 9 exchanges
// instead of 40, and each is added up in the butterfly's order.
template <int N>
__device__ __forceinline__ float butterfly_of(const float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = v[i];
    int o = 16;
#pragma unroll
    for (int n = N; n > 1; n >>= 1, o >>= 1) {
        const bool upper = (lane & o) != 0;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float keep = upper ? w[i + n / 2] : w[i], give = upper ? w[i] : w[i + n / 2];
            w[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
        }
    }
#pragma unroll
    for (; o > 0; o >>= 1) w[0] += __shfl_xor_sync(0xFFFFFFFFu, w[0], o);
    return w[0];
}
template <int N>
__device__ __forceinline__ int value_of_lane() { return (threadIdx.x & 31) / (32 / N); }
template <int N>
__device__ __forceinline__ bool first_of_value() { return (threadIdx.x & (32 / N - 1)) == 0; }

// BF16(a + b) of eight pairs: one rounding, the same as that of the FP32 sum (two BF16 values that are further apart than FP32 is
// wide do not come near a BF16 rounding boundary).
__device__ __forceinline__ uint32_t add_bf16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint4 add8(const uint4& a, const uint4& b) {
    return make_uint4(add_bf16x2(a.x, b.x), add_bf16x2(a.y, b.y), add_bf16x2(a.z, b.z), add_bf16x2(a.w, b.w));
}

__device__ __forceinline__ float sum_pair(uint64_t v) {
    float lo, hi;
    f2_unpack(v, lo, hi);
    return __fadd_rn(lo, hi);
}
__device__ __forceinline__ float squares8(const uint4& v) {
    Pairs f;
    unpack8(v, f);
    uint64_t s = f2_mul(f[0], f[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) s = f2_fma(f[i], f[i], s);
    return sum_pair(s);
}
__device__ __forceinline__ double squares8_wide(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        s = __fma_rn((double)bf16_lo(w[i]), (double)bf16_lo(w[i]), s);
        s = __fma_rn((double)bf16_hi(w[i]), (double)bf16_hi(w[i]), s);
    }
    return s;
}

// Whether FP32 held the squares: none beyond its range, and what its subnormals lost (at most 2^-136 over a row) is nothing
// beside the sum or eps.
__device__ __forceinline__ bool fp32_holds(float ss, float eps) {
    return ss <= FLT_MAX && (ss >= 8.27180613e-25f || eps >= 8.67361738e-19f);        // 2^-80, 2^-60
}
__device__ __forceinline__ RowNorm norm_of(float ss, float inv_cols, float eps) {
    return RowNorm{1.0f, __frsqrt_rn(__fadd_rn(__fmul_rn(ss, inv_cols), eps))};
}
// The same from FP64, split so that neither factor leaves FP32's normal range where the product does.
__device__ __forceinline__ RowNorm norm_of_wide(double ss, double cols, float eps) {
    const double r = 1.0 / sqrt(ss / cols + (double)eps);
    if (!(r > 0.0) || isinf(r)) return RowNorm{1.0f, (float)r};
    const int e = max(-126, min(127, ilogb(r)));
    return RowNorm{__uint_as_float((uint32_t)(e + 127) << 23), (float)(r * exp2(-(double)e))};
}
// h w r, the weight first: with BF16 weights that product is exact, so that a value is rounded once before its rounding to BF16
// and fewer fall on the other side of a BF16 boundary than in 64 bits.
__device__ __forceinline__ void normed8(Pairs& f, const Pairs& w, const RowNorm& n) {
    if (n.p != 1.0f) times8(f, n.p);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = f2_mul(f[j], w[j]);
    times8(f, n.r);
}

// Eight weights from column c on.
template <bool W32>
__device__ __forceinline__ void weights8(const void* w, int c, Pairs& f) {
    if (W32) {
        const ulonglong2 a = load_global(reinterpret_cast<const ulonglong2*>(static_cast<const float*>(w) + c));
        const ulonglong2 b = load_global(reinterpret_cast<const ulonglong2*>(static_cast<const float*>(w) + c) + 1);
        f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    } else {
        unpack8(load_global(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(w) + c)), f);
    }
}

// The threads of one row (a whole number of warps) meet; rows of a CTA are numbered from 0.
__device__ __forceinline__ void row_sync(int row, int threads) {
    asm volatile("bar.sync %0, %1;" :: "r"(row + 1), "r"(threads) : "memory");
}

// The sum over a row's segments in sm, in the fixed order.
template <typename T>
__device__ __forceinline__ T segments_sum(const T* sm, int nseg) {
    const int lane = threadIdx.x & 31;
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

// The codes of eight neighbouring elements of a row, to q where they lie inside it; returns the scale byte of the 32-block that four
// lanes hold, 0 beyond the row.  All lanes of the warp call it, with zeros where there are no elements.
__device__ __forceinline__ uint8_t quantize_row8(const uint4& y, uint8_t* q, bool in) {
    uint32_t m = absmax_bf16x2(absmax_bf16x2(y.x, y.y), absmax_bf16x2(y.z, y.w));
    m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = absmax_bf16x2(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t byte = e8m0_from_amax_bits(fold_halves(m));            // 0 for a block of zeros
    Pairs f;
    unpack8(y, f);
    times8(f, inv_scale_from_e8m0(byte));
    const uint2 codes = make_uint2(cvt_e4m3_pairs(f[0], f[1]), cvt_e4m3_pairs(f[2], f[3]));
    if (in) *reinterpret_cast<uint2*>(q) = codes;
    return in ? (uint8_t)byte : (uint8_t)0;
}
// Offset of (row, 32-block of column c) in the row-wise scale layout, split into the row's and the column's part.
__device__ __forceinline__ int64_t scale_row_offset(int64_t row, int64_t nct) {
    return ((row >> 7) * nct << 9) + ((row & 31) << 4) + ((row >> 5 & 3) << 2);
}
__device__ __forceinline__ int scale_col_offset(int c) { return (c >> 7 << 9) + (c >> 5 & 3); }

// Clears the scale rows from a.rows up to a whole tile; thread `me` of `all`.  16 bytes hold the rows l, l + 32, l + 64 and l + 96 of a
// tile (one row of 11840 takes 4.3 us, and 10.5 with a word at a time).
__device__ __forceinline__ void clear_scale_rows(const NormArgs& a, int64_t nct, int64_t me, int64_t all) {
    const int used = (int)(a.rows & 127);
    if (used == 0) return;
    for (int64_t i = me; i < nct * 32; i += all) {         // (in 64 bits: narrow rows take 2^32 threads and more)
        const int l = (int)i & 31;
        uint32_t* at = reinterpret_cast<uint32_t*>(a.s_row + ((a.rows >> 7) * nct + (i >> 5)) * 512 + l * 16);
        if (l >= used) {
            *reinterpret_cast<uint4*>(at) = make_uint4(0u, 0u, 0u, 0u);
        } else {
#pragma unroll
            for (int q = 1; q < 4; ++q)
                if (l + 32 * q >= used) at[q] = 0u;
        }
    }
}

// Rows of up to 256 elements, without column-wise codes: LANES lanes a row (8, 16 or 32), eight elements each, ROWS rows a lane with
// their loads side by side, the weights in registers.  The sums are those of a segment whose other lanes hold zeros.  With a residual
// and codes 262144 x 128 take 38.9 us, 90 % of the measured copy rate (a warp a row with eight rows a CTA: 102.8).
constexpr int NN_THREADS = 256;
// CTAs with a row a lane from which on a lane takes four (262144 x 256 71.5 us, and 90.4 with one; below, 65536 x 64 5.6 with one and 6.2
// with four).
constexpr int NN_MANY = 2432;
template <int LANES, int ROWS, bool W32>
__global__ void __launch_bounds__(NN_THREADS) norm_narrow_kernel(const NormArgs a) {
    constexpr int SIDE = 32 / LANES;
    chain_begin();
    const int lane = threadIdx.x & 31, c = lane % LANES * 8;
    const int64_t nct = sf_col_tiles(a.cols, 32), thread = (int64_t)blockIdx.x * NN_THREADS + threadIdx.x;
    if (a.q_row) clear_scale_rows(a, nct, thread, (int64_t)gridDim.x * NN_THREADS);
    const int64_t first = (thread >> 5) * (SIDE * ROWS) + lane / LANES;
    auto inside = [&](int i) { return c < a.cols && first + i * SIDE < a.rows; };
    uint4 h[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        h[i] = make_uint4(0u, 0u, 0u, 0u);
        if (inside(i)) h[i] = load_global(reinterpret_cast<const uint4*>(a.x + (first + i * SIDE) * a.ldx + c));
    }
    if (a.residual) {
        uint4 r[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (inside(i)) r[i] = load_global(reinterpret_cast<const uint4*>(a.residual + (first + i * SIDE) * a.ldr + c));
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (inside(i)) {
                h[i] = add8(h[i], r[i]);
                if (a.sum) *reinterpret_cast<uint4*>(a.sum + (first + i * SIDE) * a.lds + c) = h[i];
            }
    }
    Pairs w = {};
    if (c < a.cols) weights8<W32>(a.w, c, w);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const int64_t row = first + i * SIDE;
        const float ss = butterfly<LANES>(squares8(h[i]));
        RowNorm n = norm_of(ss, a.inv_cols, a.eps);
        const bool fine = fp32_holds(ss, a.eps);
        if (__any_sync(0xFFFFFFFFu, !fine)) {
            const double wide = butterfly<LANES>(squares8_wide(h[i]));
            if (!fine) n = norm_of_wide(wide, a.cols, a.eps);
        }
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (inside(i)) {
            Pairs f;
            unpack8(h[i], f);
            normed8(f, w, n);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(a.y + row * a.ldy + c) = y;
        }
        if (a.q_row) {
            uint32_t s = quantize_row8(y, a.q_row + row * a.cols + c, inside(i));
            // the scales of 128 columns (0 beyond the row), a word
            const uint32_t s1 = __shfl_down_sync(0xFFFFFFFFu, s, 4), s2 = __shfl_down_sync(0xFFFFFFFFu, s, 8), s3 = __shfl_down_sync(0xFFFFFFFFu, s, 12);
            s |= s1 << 8;
            if (LANES > 8) s |= s2 << 16 | s3 << 24;
            if (c % 128 == 0 && c < 128 * nct && row < a.rows)
                *reinterpret_cast<uint32_t*>(a.s_row + scale_row_offset(row, nct) + scale_col_offset(c)) = s;
        }
    }
}

// Without column-wise codes: one row a group of blockDim.x threads, blockDim.y rows a CTA; NV vectors of eight elements a thread.
// At most four a thread and 64 registers: with eight, one CTA an SM ran through 32 KB of straight-line code for every row
// (1003 x 14336 took 54 us, now 17: four turns of two CTAs an SM, each a row's loads, meeting and stores after one another, which wait for
// memory most of the time: half of the issue slots are taken).
// FULL: the threads' vectors are the row exactly, no comparisons (8192 x 4096 to codes 29.8 to 27.3 us).  With residual, sum and codes
// 8192 x 4096 takes 36.5 us on the same tensors again and again, 96 % of the measured copy rate, and 40.3 where they change.
constexpr int NR_THREADS = NORM_ROWS_THREADS;
template <int NV, bool W32, bool FULL>
__global__ void __launch_bounds__(NR_THREADS, 2) norm_rows_kernel(const NormArgs a) {
    __shared__ double sm_all[8][MAX_SEGS];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, ty = threadIdx.y;
    const int nseg = (a.cols + SEG - 1) / SEG;
    const int64_t nct = sf_col_tiles(a.cols, 32);
    if (a.q_row)
        clear_scale_rows(a, nct, ((int64_t)blockIdx.x * blockDim.y + ty) * blockDim.x + threadIdx.x, (int64_t)gridDim.x * blockDim.y * blockDim.x);
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + ty;
    if (row >= a.rows) return;
    const int c0 = (warp * 32 + lane) * 8, step = warps * SEG;
    auto inside = [&](int i) { return FULL || c0 + i * step < a.cols; };
    const uint16_t* x = a.x + row * a.ldx;
    uint4 h[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        h[i] = make_uint4(0u, 0u, 0u, 0u);
        if (inside(i)) h[i] = load_global(reinterpret_cast<const uint4*>(x + c0 + i * step));
    }
    if (a.residual) {
        const uint16_t* residual = a.residual + row * a.ldr;
        uint16_t* sum = a.sum + row * a.lds;
        uint4 r[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (inside(i)) r[i] = load_global(reinterpret_cast<const uint4*>(residual + c0 + i * step));
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (inside(i)) {
                h[i] = add8(h[i], r[i]);
                if (a.sum) *reinterpret_cast<uint4*>(sum + c0 + i * step) = h[i];
            }
    }
    float part[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) part[i] = squares8(h[i]);
    float* sm = reinterpret_cast<float*>(sm_all[ty]);
    const float mine = butterfly_of(part);
    const int my_seg = warp + value_of_lane<NV>() * warps;
    if (first_of_value<NV>() && my_seg < nseg) sm[my_seg] = mine;
    row_sync(ty, blockDim.x);
    const float ss = segments_sum(sm, nseg);
    RowNorm n = norm_of(ss, a.inv_cols, a.eps);
    if (!fp32_holds(ss, a.eps)) {                          // the same for all threads of the row
        row_sync(ty, blockDim.x);                          // the FP32 sums have been read
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const double s = butterfly(squares8_wide(h[i]));
            if (lane == 0 && warp + i * warps < nseg) sm_all[ty][warp + i * warps] = s;
        }
        row_sync(ty, blockDim.x);
        n = norm_of_wide(segments_sum(sm_all[ty], nseg), a.cols, a.eps);
    }
    uint16_t* to_y = a.y + row * a.ldy;
    uint8_t *q = a.q_row + row * a.cols, *s = a.s_row + scale_row_offset(row, nct);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * step;
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (inside(i)) {
            Pairs f, w;
            unpack8(h[i], f);
            weights8<W32>(a.w, c, w);
            normed8(f, w, n);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(to_y + c) = y;
        }
        if (a.q_row) {
            const uint8_t byte = quantize_row8(y, q + c, inside(i));
            if ((c & 31) == 0 && (FULL || c < 128 * nct)) s[scale_col_offset(c)] = byte;
        }
    }
}

// With column-wise codes: a cluster takes 32 rows, its CTAs T_SEGS segments of them each.  A warp takes whole segments of rows
// (eight a thread), so the sums of squares of a segment are one butterfly; the CTAs write theirs into each other's shared memory
// and meet once.  The tile waits in shared memory, where the output takes its place and a thread then finds the two columns
// that it quantizes.
// 8192 x 4096 with residual, sum and both orientations: 53 us, 76 % of the measured copy rate; 8192 x 8192 112, 72 %.  Some 7 us are the cluster: eight CTAs
// start and meet together, and 5 % of the SMs fit no cluster of eight.  The transposed codes leave in pieces of 32 bytes and their
// scales in single bytes.  No quicker: four CTAs of 1024 columns, five CTAs an SM with 48 registers (59), the sums sent
// asynchronously to a barrier in place of the meeting, all loads at once.
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
__device__ __forceinline__ void cluster_sync() {           // also orders the shared memory writes before it for the peers
    cluster_arrive();
    cluster_wait();
}
__device__ __forceinline__ uint32_t peer_address(const void* mine, uint32_t peer) {
    uint32_t there;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"((uint32_t)__cvta_generic_to_shared(mine)), "r"(peer));
    return there;
}

constexpr int TILE_ROWS = 32;
constexpr int PART = MAX_SEGS + 1;                         // pitch of the sums of a row, odd against bank conflicts
template <int SEGS>
struct TileCfg {
    static constexpr int THREADS = 128 * SEGS;             // 4 * SEGS warps, each eight of the 32 * SEGS (row, segment) pairs
    static constexpr int COLS = SEG * SEGS;
    static constexpr int TILE = TILE_ROWS * COLS * 2;      // bytes
    static constexpr int SMEM = TILE + TILE_ROWS * PART * 4;              // and the rows' sums by segments
};

// The rows of a tile that FP32 does not hold (their p is 0 so far).  Every CTA of the cluster calls it with all its threads; the
// FP64 sums of 16 rows at a time take the place of the FP32 ones.
template <int SEGS>
__device__ __noinline__ void slow_rows(const NormArgs& a, const uint8_t* sm_tile, float* part, RowNorm* s_norm, int gseg, int nseg,
                                       uint32_t peers) {
    constexpr int WARPS = TileCfg<SEGS>::THREADS / 32, HALF = TILE_ROWS / 2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, seg = warp % SEGS;
    double* wide = reinterpret_cast<double*>(part);        // [HALF][PART]
    for (int first = 0; first < TILE_ROWS; first += HALF) {
        cluster_sync();                                    // what stands there has been read
#pragma unroll 1
        for (int r = warp / SEGS; r < HALF; r += 4) {
            const double s = butterfly(squares8_wide(*reinterpret_cast<const uint4*>(
                sm_tile + ((first + r) * TileCfg<SEGS>::COLS + seg * SEG + lane * 8) * 2)));
            if ((uint32_t)lane < peers && gseg < nseg)
                asm volatile("st.shared::cluster.f64 [%0], %1;" :: "r"(peer_address(wide + r * PART + gseg, lane)), "d"(s) : "memory");
        }
        cluster_sync();
#pragma unroll 1
        for (int r = warp; r < HALF; r += WARPS) {
            const double s = segments_sum(wide + r * PART, nseg);
            if (lane == 0 && s_norm[first + r].p == 0.0f) s_norm[first + r] = norm_of_wide(s, a.cols, a.eps);
        }
    }
    __syncthreads();
}

template <int SEGS, bool W32>
__global__ void __launch_bounds__(TileCfg<SEGS>::THREADS, 8 / SEGS) norm_tile_kernel(const NormArgs a) {
    using C = TileCfg<SEGS>;
    constexpr int WARPS = C::THREADS / 32, ITEMS = 8, ROWS_A_WARP = TILE_ROWS / WARPS;
    extern __shared__ __align__(16) uint8_t sm_tile[];
    float* part = reinterpret_cast<float*>(sm_tile + C::TILE);            // [32][PART]
    __shared__ RowNorm s_norm[TILE_ROWS];
    __shared__ __align__(4) uint8_t s_scales[TILE_ROWS][8 * SEGS];        // the rows' block scales
    cluster_arrive();                                      // this CTA runs: the others may write into its shared memory
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank(), peers = cluster_size();
    const int nseg = (a.cols + SEG - 1) / SEG;
    const int64_t r0 = (int64_t)(blockIdx.x / peers) * TILE_ROWS;
    const int c_cta = (int)rank * C::COLS;
    // item i of a warp: row warp / SEGS + 4 i, segment warp % SEGS of the CTA
    const int seg = warp % SEGS, c = c_cta + seg * SEG + lane * 8, gseg = (int)rank * SEGS + seg, row0 = warp / SEGS;
    const bool in = c < a.cols;
    const uint16_t *x = a.x + (r0 + row0) * a.ldx + c, *residual = a.residual + (r0 + row0) * a.ldr + c;
    auto place = [&](int i) { return reinterpret_cast<uint4*>(sm_tile + ((row0 + 4 * i) * C::COLS + seg * SEG + lane * 8) * 2); };
    float sums[ITEMS];
#pragma unroll
    for (int half = 0; half < ITEMS; half += 4) {
        uint4 h[4], r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = r[i] = make_uint4(0u, 0u, 0u, 0u);
            if (in) h[i] = load_global(reinterpret_cast<const uint4*>(x));
            if (in && a.residual) r[i] = load_global(reinterpret_cast<const uint4*>(residual));
            x += 4 * a.ldx;
            residual += 4 * a.ldr;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (a.residual) h[i] = add8(h[i], r[i]);
            *place(half + i) = h[i];
            sums[half + i] = squares8(h[i]);
        }
    }
    const float mine = butterfly_of(sums);                 // that of row row0 + 4 * (lane / 4)
    cluster_wait();
    if (gseg < nseg) {
        const float* at = part + (row0 + 4 * value_of_lane<ITEMS>()) * PART + gseg;
        for (uint32_t p = lane & 3; p < peers; p += 4)
            asm volatile("st.shared::cluster.f32 [%0], %1;" :: "r"(peer_address(at, p)), "f"(mine) : "memory");
    }
    cluster_sync();
    float v[ROWS_A_WARP];
#pragma unroll
    for (int i = 0; i < ROWS_A_WARP; ++i) {
        const float* at = part + (warp + i * WARPS) * PART + lane;
        v[i] = lane < nseg ? at[0] : 0.0f;
        if (lane + 32 < nseg) v[i] += at[32];
    }
    const float ss = butterfly_of(v);
    const int my_row = warp + value_of_lane<ROWS_A_WARP>() * WARPS;
    const bool fine = fp32_holds(ss, a.eps);
    if (first_of_value<ROWS_A_WARP>()) s_norm[my_row] = fine ? norm_of(ss, a.inv_cols, a.eps) : RowNorm{0.0f, 0.0f};
    if (__syncthreads_or(!fine)) {
        // the same in every CTA of the cluster, as all have the same sums
        slow_rows<SEGS>(a, sm_tile, part, s_norm, gseg, nseg, peers);
    }
    const int64_t nct_row = sf_col_tiles(a.cols, 32);
    uint16_t *to_sum = a.sum + (r0 + row0) * a.lds + c, *to_y = a.y + (r0 + row0) * a.ldy + c;
    uint8_t* to_q = a.q_row + (r0 + row0) * a.cols + c;
    Pairs w;
    if (in) weights8<W32>(a.w, c, w);
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const int r = row0 + 4 * i;
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (in) {
            const uint4 h = *place(i);
            // (only now: the meeting of the cluster would have waited for earlier stores to reach memory)
            if (a.sum) *reinterpret_cast<uint4*>(to_sum) = h;
            Pairs f;
            unpack8(h, f);
            normed8(f, w, s_norm[r]);
            y = pack8(f);
            if (a.y) *reinterpret_cast<uint4*>(to_y) = y;
        }
        *place(i) = y;
        if (a.q_row) {
            const uint8_t byte = quantize_row8(y, to_q, in);
            if ((lane & 3) == 0) s_scales[row0 + 4 * i][seg * 8 + lane / 4] = byte;
        }
        to_sum += 4 * a.lds;
        to_y += 4 * a.ldy;
        to_q += 4 * (int64_t)a.cols;
    }
    __syncthreads();
    if (a.q_row && threadIdx.x < TILE_ROWS * 2 * SEGS) {   // words of four blocks, those of a row 512 bytes apart
        const int r = threadIdx.x / (2 * SEGS), k = threadIdx.x % (2 * SEGS), c4 = c_cta / 128 + k;
        if (c4 < nct_row)
            *reinterpret_cast<uint32_t*>(a.s_row + scale_row_offset(r0 + r, nct_row) + c4 * 512) = *reinterpret_cast<const uint32_t*>(&s_scales[r][4 * k]);
    }
    if (a.q_row && r0 + TILE_ROWS == a.rows) {             // scale rows up to a whole tile: zeros, this CTA's columns
        const int pad = (int)(((a.rows + 127) & ~int64_t(127)) - a.rows), first = c_cta / 128, last = min((int)nct_row, first + C::COLS / 128);
        for (int i = threadIdx.x; i < pad * 8; i += C::THREADS)
            for (int k = first + i % 8; k < last; k += 8)
                *reinterpret_cast<uint32_t*>(a.s_row + sf_offset(a.rows + i / 8, 4 * k, nct_row)) = 0u;
    }
    // a warp 64 columns, a lane two neighbours: both whole 32-blocks are its own
    const int cc = warp * 64 + lane * 2, gc = c_cta + cc;
    const int64_t nct = sf_col_tiles(a.rows, 32);
    const int padded_cols = (a.cols + 127) & ~127;
    if (warp * 64 >= C::COLS || c_cta + warp * 64 >= padded_cols) return;
    const bool gin = gc < a.cols;
    uint32_t t[TILE_ROWS], m = 0u;
#pragma unroll
    for (int i = 0; i < TILE_ROWS; ++i) {
        t[i] = *reinterpret_cast<const uint32_t*>(sm_tile + (i * C::COLS + cc) * 2);
        m = i == 0 ? t[0] : absmax_bf16x2(m, t[i]);
    }
    m = abs_halves(m);
    uint8_t* q_col = a.q_col + (int64_t)gc * a.rows + r0;
    uint8_t* s_col = a.s_col + sf_offset(gc, r0 / 32, nct);               // the next column's is 16 bytes on
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t s = e8m0_from_amax_bits(j ? m >> 16 : m & 0xFFFFu);
        const float inv = inv_scale_from_e8m0(s);
        uint32_t codes[TILE_ROWS / 4];
#pragma unroll
        for (int k = 0; k < TILE_ROWS / 4; ++k) {
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __fmul_rn(j ? bf16_hi(t[4 * k + i]) : bf16_lo(t[4 * k + i]), inv);
            codes[k] = cvt_e4m3x4(f[0], f[1], f[2], f[3]);
        }
        if (gin)
            stcs_32b(q_col + j * a.rows, make_uint4(codes[0], codes[1], codes[2], codes[3]), make_uint4(codes[4], codes[5], codes[6], codes[7]));
        s_col[j * 16] = gin ? (uint8_t)s : (uint8_t)0;
    }
    // scale columns from rows / 32 up to a whole word: zeros
    if (r0 + TILE_ROWS == a.rows)
        for (int64_t b = a.rows / 32; b < 4 * nct; ++b)
            for (int j = 0; j < 2; ++j) a.s_col[sf_offset(gc + j, b, nct)] = 0;
}

// ------------------------------------------------------------------------------------------------
// Eight FP32 values as they are: the gradient's kernel, whose values meet in more ways, is quicker without the pairs (45 us for
// 8192 x 4096, and 47.5 with them, which take more moves between registers).
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <bool W32>
__device__ __forceinline__ void weights8(const void* w, int c, float (&f)[8]) {
    Pairs p;
    weights8<W32>(w, c, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_unpack(p[i], f[2 * i], f[2 * i + 1]);
}

// Gradient.  A CTA walks rows; each thread keeps the sums of dw for its columns in registers.  The CTAs of a cluster add theirs
// up through shared memory, and a second kernel adds the clusters' sums in their order.
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

// A form of the kernel: CTAs of up to THREADS threads, PER_SM of those an SM (which sets the registers of a thread), NV vectors of eight
// elements a thread.  Every form keeps the weights in registers.
template <int THREADS_, int PER_SM_, int NV_>
struct BackwardForm {
    static constexpr int THREADS = THREADS_, PER_SM = PER_SM_, NV = NV_;
};
constexpr int NB_CLUSTER = 2;                              // wider clusters leave SMs idle (8192 x 4096 47 us, with four 63, with eight 65; 777 x 2048
                                                           // 8.7, 10.6 and 11.8)
constexpr int NB_PARTS = 304;                              // most partial sums of a column: two an SM of 152 (a pair of CTAs has one, four fit an SM)
constexpr int NB_STAGES = 2;

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" :: "n"(LEFT) : "memory");
}

// A lane's sums of h^2 and dn h over eight elements, even and odd ones apart as in the forward's sums.
__device__ __forceinline__ void products8(const float (&x)[8], const float (&d)[8], const float (&w)[8], float& squares, float& inner) {
    float s[2] = {0.0f, 0.0f}, c[2] = {0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        s[j & 1] = __fmaf_rn(x[j], x[j], s[j & 1]);
        c[j & 1] = __fmaf_rn(__fmul_rn(d[j], w[j]), x[j], c[j & 1]);
    }
    squares = __fadd_rn(s[0], s[1]);
    inner = __fadd_rn(c[0], c[1]);
}
__device__ __forceinline__ double inner8_wide(const float (&x)[8], const float (&d)[8], const float (&w)[8]) {
    double s = 0.0;
    for (int j = 0; j < 8; ++j) s = __fma_rn((double)d[j] * (double)w[j], (double)x[j], s);
    return s;
}
// Whether FP32 held both sums of a row: dn h likewise neither too large, nor so small that subnormals would decide (where eps
// does not).
__device__ __forceinline__ bool fp32_holds_both(float ss, float cc, float eps) {
    return fp32_holds(ss, eps) && fabsf(cc) <= FLT_MAX && (fabsf(cc) >= 7.88860905e-31f || eps >= 9.09494702e-13f);
}
// A factor far from 1 is split as a slow row's is, so that dy r keeps its bits where dy n has them.
__device__ __forceinline__ void split_far(RowNorm& n) {
    if (n.r < 9.53674316e-7f || n.r > 1048576.0f) {        // 2^-20, 2^20; neither for a slow row
        n.p = __uint_as_float(__float_as_uint(n.r) & 0x7F800000u);
        n.r = __uint_as_float((__float_as_uint(n.r) & 0x007FFFFFu) | 0x3F800000u);
    }
}
// With x = h p: o = p (r dy w - x r^2 mean), dw += (r dy) x.  SCALED false: p is 1 (its products would take a tenth of the
// instructions).
template <bool SCALED>
__device__ __forceinline__ void gradient8(float (&x)[8], float (&d)[8], const float (&w)[8], const RowNorm& n, float by_x, float (&dw)[8],
                                          float (&o)[8]) {
    if (SCALED)
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], n.p);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        d[j] = __fmul_rn(d[j], n.r);
        o[j] = __fmaf_rn(x[j], by_x, __fmul_rn(d[j], w[j]));
        dw[j] = __fmaf_rn(d[j], x[j], dw[j]);
    }
    if (SCALED)
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = __fmul_rn(o[j], n.p);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// A thread fetches its own vectors of the next row into shared memory (nobody else reads them there, so no barrier guards
// them) while it works on this one: the loads wait in no registers, and a row's sums do not hold up the next row's.
// FULL: every vector of every thread lies inside the row (its width is the threads' vectors exactly), which
// spares the comparisons: 2 of 45 us for 8192 x 4096.
template <typename F, bool W32, bool FULL>
__global__ void __launch_bounds__(F::THREADS, F::PER_SM) norm_backward_kernel(const NormBackwardArgs a) {
    constexpr int NV = F::NV;
    extern __shared__ __align__(16) uint8_t sm_rows[];     // [stage][dy, h, dsum][NV][thread] of 16 bytes
    __shared__ double sm_all[2][2][MAX_SEGS];              // [turn][sum][segment]
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, tid = threadIdx.x, threads = blockDim.x;
    const int nseg = (a.cols + SEG - 1) / SEG, tensors = a.dsum ? 3 : 2;
    const uint32_t vector = threads * 16, tensor = NV * vector, stage_bytes = tensors * tensor;
    const uint32_t sm0 = (uint32_t)__cvta_generic_to_shared(sm_rows) + tid * 16;
    const int c0 = (warp * 32 + lane) * 8, step = warps * SEG;
    auto outside = [&](int i) { return !FULL && c0 + i * step >= a.cols; };
    const int64_t first = blockIdx.x, next = gridDim.x;
    const uint16_t *dy = a.dy + first * a.lddy + c0, *from_h = a.h + first * a.ldh + c0, *dsum = a.dsum + first * a.ldds + c0;
    uint16_t* dx = a.dx + first * a.lddx + c0;
    auto fetch = [&](int64_t row, uint32_t stage) {        // rows in turn
        if (row < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (outside(i)) continue;
                const uint32_t at = sm0 + stage * stage_bytes + i * vector;
                copy16(at, dy + i * step);
                copy16(at + tensor, from_h + i * step);
                if (a.dsum) copy16(at + 2 * tensor, dsum + i * step);
            }
            dy += next * a.lddy;
            from_h += next * a.ldh;
            dsum += next * a.ldds;
        }
        copies_commit();                                   // an empty group where there is no row, so that the count goes on
    };
    auto fetched = [&](uint32_t stage, int which, int i) {
        return *reinterpret_cast<const uint4*>(sm_rows + stage * stage_bytes + which * tensor + i * vector + tid * 16);
    };
    fetch(first, 0);
    float dw[NV][8] = {}, weight[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (!outside(i)) weights8<W32>(a.w, c0 + i * step, weight[i]);
    uint32_t turn = 0;
    for (int64_t row = first; row < a.rows; row += next, turn ^= 1) {
        fetch(row + next, turn ^ 1);                  // into the stage that this thread read in the turn before
        copies_wait<1>();
        float parts[2 * NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            parts[i] = parts[NV + i] = 0.0f;
            if (outside(i)) continue;
            float x[8], d[8];
            unpack8(fetched(turn, 1, i), x);
            unpack8(fetched(turn, 0, i), d);
            products8(x, d, weight[i], parts[i], parts[NV + i]);
        }
        float* sm_s = reinterpret_cast<float*>(sm_all[turn][0]);
        float* sm_c = reinterpret_cast<float*>(sm_all[turn][1]);
        const float mine = butterfly_of(parts);
        const int value = value_of_lane<2 * NV>(), my_seg = warp + (value % NV) * warps;
        if (first_of_value<2 * NV>() && my_seg < nseg) (value < NV ? sm_s : sm_c)[my_seg] = mine;
        __syncthreads();
        float v[2] = {lane < nseg ? sm_s[lane] : 0.0f, lane < nseg ? sm_c[lane] : 0.0f};
        if (lane + 32 < nseg) {
            v[0] += sm_s[lane + 32];
            v[1] += sm_c[lane + 32];
        }
        const float both = butterfly_of(v);                              // of the first in the lower half of the warp
        const float ss = __shfl_sync(0xFFFFFFFFu, both, 0), cc = __shfl_sync(0xFFFFFFFFu, both, 16);
        RowNorm n = norm_of(ss, a.inv_cols, a.eps);
        float mean = __fmul_rn(__fmul_rn(cc, a.inv_cols), n.r);          // mean(dn n)
        if (!fp32_holds_both(ss, cc, a.eps)) {
            __syncthreads();                                                   // the FP32 sums have been read
#pragma unroll 1
            for (int i = 0; i < NV; ++i) {
                double inner = 0.0, squares = 0.0;
                if (!outside(i)) {
                    const uint4 h = fetched(turn, 1, i);
                    float x[8], d[8], w[8];
                    unpack8(h, x);
                    unpack8(fetched(turn, 0, i), d);
                    weights8<W32>(a.w, c0 + i * step, w);
                    inner = inner8_wide(x, d, w);
                    squares = squares8_wide(h);
                }
                squares = butterfly(squares);
                inner = butterfly(inner);
                if (lane == 0 && warp + i * warps < nseg) {
                    sm_all[turn][0][warp + i * warps] = squares;
                    sm_all[turn][1][warp + i * warps] = inner;
                }
            }
            __syncthreads();
            n = norm_of_wide(segments_sum(sm_all[turn][0], nseg), a.cols, a.eps);
            mean = (float)(segments_sum(sm_all[turn][1], nseg) / a.cols * n.p * n.r);
        }
        split_far(n);
        const float by_x = -__fmul_rn(__fmul_rn(mean, n.r), n.r);
        auto emit = [&](auto scaled) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (outside(i)) continue;
                float x[8], d[8], o[8];
                unpack8(fetched(turn, 1, i), x);
                unpack8(fetched(turn, 0, i), d);
                gradient8<decltype(scaled)::value>(x, d, weight[i], n, by_x, dw[i], o);
                if (a.dsum) {
                    unpack8(fetched(turn, 2, i), x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __fadd_rn(o[j], x[j]);
                }
                *reinterpret_cast<uint4*>(dx + i * step) = pack8(o);
            }
        };
        if (n.p != 1.0f) emit(std::true_type{});
        else emit(std::false_type{});
        dx += next * a.lddx;
    }
    // the cluster's sums: each CTA's in its shared memory (the ring is free: 8 bytes a column and more), a share of the columns each
    float* sm_dw = reinterpret_cast<float*>(sm_rows);
    __syncthreads();                                       // the last row has been read
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (!outside(i)) {
            const int c = c0 + i * step;
            reinterpret_cast<float4*>(sm_dw + c)[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            reinterpret_cast<float4*>(sm_dw + c)[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    }
    cluster_sync();
    const int peers = (int)cluster_size();
    for (int c = ((int)cluster_rank() * threads + tid) * 4; c < a.cols; c += peers * threads * 4) {
        uint64_t s0 = 0, s1 = 0;
        for (int p = 0; p < peers; ++p) {
            uint64_t v0, v1;
            asm volatile("ld.shared::cluster.v2.b64 {%0, %1}, [%2];" : "=l"(v0), "=l"(v1) : "r"(peer_address(sm_dw + c, p)) : "memory");
            s0 = f2_add(s0, v0);
            s1 = f2_add(s1, v1);
        }
        *reinterpret_cast<ulonglong2*>(a.partial + (int64_t)(blockIdx.x / peers) * a.cols + c) = make_ulonglong2(s0, s1);
    }
    cluster_sync();                                        // nobody leaves while the others read its sums
}

// Rows of up to 1024 elements, a warp or part of one each: LANES lanes (8, 16 or 32), NV vectors of eight elements a lane (more than one
// with 32 lanes only).  The warps walk the rows, each lane with a ring of its own vectors in shared memory, and a CTA adds its sums of dw
// up there at the end.  262144 x 128 with dsum take 39.7 us, the measured copy rate, and 32768 x 512 20.3 (89.5 and 25.9 with rows side by side in the
// form for wider rows); two CTAs of 256 threads an SM: with 384 (80 registers) 42.4, with 512 (64, which spill) 52.3.
constexpr int NBN_THREADS = 256;
template <int NV>
constexpr int NBN_STAGES = NV == 4 ? 2 : 4;

// The sum over a row's segments, whose sums are v, in the fixed order.
template <typename T, int NV>
__device__ __forceinline__ T few_segments_sum(const T (&v)[NV]) {
    if constexpr (NV == 1) return v[0];
    else if constexpr (NV == 2) return v[0] + v[1];
    else return (v[0] + v[2]) + (v[1] + v[3]);
}

// p, r and mean(dn n) of the warp's rows, summed in FP64 (out of line, so that it costs the others no registers).  dy and h: the lane's
// vectors, NBN_THREADS apart.
template <int LANES, int NV, bool W32>
__device__ __noinline__ float3 slow_narrow_row(const uint4* dy, const uint4* h, bool in, const void* weight, int c, int cols, float eps) {
    double squares[NV], inner[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        squares[i] = inner[i] = 0.0;
        if (in && c + i * SEG < cols) {
            float x[8], d[8], w[8];
            unpack8(h[i * NBN_THREADS], x);
            unpack8(dy[i * NBN_THREADS], d);
            weights8<W32>(weight, c + i * SEG, w);
            squares[i] = squares8_wide(h[i * NBN_THREADS]);
            inner[i] = inner8_wide(x, d, w);
        }
        squares[i] = butterfly<LANES>(squares[i]);
        inner[i] = butterfly<LANES>(inner[i]);
    }
    const RowNorm n = norm_of_wide(few_segments_sum(squares), cols, eps);
    return make_float3(n.p, n.r, (float)(few_segments_sum(inner) / cols * n.p * n.r));
}

template <int LANES, int NV, bool W32>
__global__ void __launch_bounds__(NBN_THREADS, 2) norm_backward_narrow_kernel(const NormBackwardArgs a) {
    static_assert(NV == 1 || LANES == 32, "several vectors a lane: a segment each");
    constexpr int SIDE = 32 / LANES, WARPS = NBN_THREADS / 32, STAGES = NBN_STAGES<NV>;
    constexpr uint32_t TENSOR = NV * NBN_THREADS * 16;
    extern __shared__ __align__(16) uint8_t sm_rows[];     // [stage][dy, h, dsum][NV][thread] of 16 bytes; then [warp][column] sums
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = lane % LANES * 8;
    const uint32_t stage_bytes = (a.dsum ? 3 : 2) * TENSOR, sm0 = (uint32_t)__cvta_generic_to_shared(sm_rows) + threadIdx.x * 16;
    const int64_t next = (int64_t)gridDim.x * (WARPS * SIDE), first = ((int64_t)blockIdx.x * WARPS + warp) * SIDE + lane / LANES;
    // the group's first row decides for the warp (its lanes stay together), the lane's own whether it has one
    const int64_t turns = first - lane / LANES < a.rows ? (a.rows - (first - lane / LANES) + next - 1) / next : 0;
    auto has = [&](int i) { return c + i * SEG < a.cols; };
    const uint16_t *dy = a.dy + first * a.lddy + c, *from_h = a.h + first * a.ldh + c, *dsum = a.dsum + first * a.ldds + c;
    uint16_t* dx = a.dx + first * a.lddx + c;
    auto fetch = [&](int64_t t, uint32_t stage) {          // turns in order
        if (first + t * next < a.rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has(i)) continue;
                const uint32_t at = sm0 + stage * stage_bytes + i * (NBN_THREADS * 16);
                copy16(at, dy + i * SEG);
                copy16(at + TENSOR, from_h + i * SEG);
                if (a.dsum) copy16(at + 2 * TENSOR, dsum + i * SEG);
            }
            dy += next * a.lddy;
            from_h += next * a.ldh;
            dsum += next * a.ldds;
        }
        copies_commit();                                   // an empty group where there is no row, so that the count goes on
    };
#pragma unroll
    for (int t = 0; t < STAGES - 1; ++t) fetch(t, t);
    float w[NV][8] = {}, dw[NV][8] = {};
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (has(i)) weights8<W32>(a.w, c + i * SEG, w[i]);
    uint32_t stage = 0;
    for (int64_t t = 0; t < turns; ++t) {
        fetch(t + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);      // into the stage that this lane read in the turn before
        copies_wait<STAGES - 1>();
        auto fetched = [&](int which) { return reinterpret_cast<const uint4*>(sm_rows + stage * stage_bytes + which * TENSOR) + threadIdx.x; };
        const bool row_in = first + t * next < a.rows;
        float parts[2 * NV];
        uint4 held[2];                                     // of one vector a lane, which need not be read again (2 of 41 us)
        auto vector = [&](int which, int i) { return NV == 1 ? held[which] : fetched(which)[i * NBN_THREADS]; };
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            parts[i] = parts[NV + i] = 0.0f;
            if (!row_in || !has(i)) continue;
            if (NV == 1)
                for (int k = 0; k < 2; ++k) held[k] = fetched(k)[0];
            float x[8], d[8];
            unpack8(vector(1, i), x);
            unpack8(vector(0, i), d);
            products8(x, d, w[i], parts[i], parts[NV + i]);
        }
        float ss, cc;
        if constexpr (NV == 1) {
            ss = butterfly<LANES>(parts[0]);
            cc = butterfly<LANES>(parts[1]);
        } else {                                           // value v to the lanes from v * 32 / (2 NV) on; then the segments in pairs
            float both = butterfly_of(parts);
#pragma unroll
            for (int o = 8; o >= 16 / NV; o >>= 1) both += __shfl_xor_sync(0xFFFFFFFFu, both, o);
            ss = __shfl_sync(0xFFFFFFFFu, both, 0);
            cc = __shfl_sync(0xFFFFFFFFu, both, 16);
        }
        RowNorm n = norm_of(ss, a.inv_cols, a.eps);
        float mean = __fmul_rn(__fmul_rn(cc, a.inv_cols), n.r);          // mean(dn n)
        const bool fine = fp32_holds_both(ss, cc, a.eps);
        if (__any_sync(0xFFFFFFFFu, !fine)) {
            const float3 wide = slow_narrow_row<LANES, NV, W32>(fetched(0), fetched(1), row_in, a.w, c, a.cols, a.eps);
            if (!fine) {
                n = RowNorm{wide.x, wide.y};
                mean = wide.z;
            }
        }
        split_far(n);
        const float by_x = -__fmul_rn(__fmul_rn(mean, n.r), n.r);
        auto emit = [&](auto scaled) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!has(i)) continue;
                float x[8], d[8], o[8];
                unpack8(vector(1, i), x);
                unpack8(vector(0, i), d);
                gradient8<decltype(scaled)::value>(x, d, w[i], n, by_x, dw[i], o);
                if (a.dsum) {
                    unpack8(fetched(2)[i * NBN_THREADS], x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = __fadd_rn(o[j], x[j]);
                }
                *reinterpret_cast<uint4*>(dx + i * SEG) = pack8(o);
            }
        };
        if (row_in) {
            if (n.p != 1.0f) emit(std::true_type{});
            else emit(std::false_type{});
        }
        dx += next * a.lddx;
        stage = stage == STAGES - 1 ? 0 : stage + 1;
    }
    if (LANES < 32)
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int o = 16; o >= LANES; o >>= 1) dw[0][j] += __shfl_xor_sync(0xFFFFFFFFu, dw[0][j], o);
    constexpr int WIDTH = NV * LANES * 8;                  // (half of the ring at most)
    float* sm_dw = reinterpret_cast<float*>(sm_rows);
    __syncthreads();                                       // the last rows have been read
    if (lane < LANES)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float4* at = reinterpret_cast<float4*>(sm_dw + warp * WIDTH + c + i * SEG);
            at[0] = make_float4(dw[i][0], dw[i][1], dw[i][2], dw[i][3]);
            at[1] = make_float4(dw[i][4], dw[i][5], dw[i][6], dw[i][7]);
        }
    __syncthreads();
    for (int at = threadIdx.x; at < a.cols; at += NBN_THREADS) {
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) s += sm_dw[k * WIDTH + at];
        a.partial[(int64_t)blockIdx.x * a.cols + at] = s;
    }
}

// dw[c] = the sum of `parts` partial sums: 32 columns a CTA, 32 warps a share of the parts each.
constexpr int ND_WARPS = 32;
__global__ void __launch_bounds__(32 * ND_WARPS) norm_dweight_kernel(const float* partial, int parts, int cols, float* dw) {
    __shared__ float sm[ND_WARPS][33];
    chain_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    constexpr int LOADS = (NB_PARTS + ND_WARPS - 1) / ND_WARPS;           // side by side
    float v[LOADS], s = 0.0f;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
        const int p = warp + i * ND_WARPS;
        v[i] = p < parts && c < cols ? load_global(partial + (int64_t)p * cols + c) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) s += v[i];
    sm[warp][lane] = s;
    __syncthreads();
    s = butterfly(sm[lane][warp]);                         // a warp a column
    if (lane == 0 && blockIdx.x * 32 + warp < cols) dw[blockIdx.x * 32 + warp] = s;
}

template <int LANES, bool W32>
cudaError_t norm_narrow(const NormArgs& a, cudaStream_t stream) {
    auto go = [&](auto kernel, int rows_a_cta) {
        return launch_chained(kernel, dim3((unsigned)((a.rows + rows_a_cta - 1) / rows_a_cta)), dim3(NN_THREADS), 0, 0, stream, a);
    };
    constexpr int side = NN_THREADS / LANES;
    if (a.rows >= (int64_t)NN_MANY * side) return go(norm_narrow_kernel<LANES, 4, W32>, 4 * side);
    return go(norm_narrow_kernel<LANES, 1, W32>, side);
}

template <bool W32>
cudaError_t norm_rows(const NormArgs& a, cudaStream_t stream) {
    if (a.cols <= 64) return norm_narrow<8, W32>(a, stream);
    if (a.cols <= 128) return norm_narrow<16, W32>(a, stream);
    if (a.cols <= 256) return norm_narrow<32, W32>(a, stream);
    const NormRowsForm form = norm_rows_form(a.rows, a.cols);
    const int threads = form.threads, nv = form.nv;
    if (nv > 4 || (int64_t)nv * threads * 8 < a.cols) return cudaErrorInvalidConfiguration;       // no form covers the row
    const int per = max(1, 256 / threads);
    auto go = [&](auto kernel) {
        return launch_chained(kernel, dim3((unsigned)((a.rows + per - 1) / per)), dim3(threads, per), 0, 0, stream, a);
    };
    const bool full = a.cols == nv * threads * 8;
    if (nv == 1) return full ? go(norm_rows_kernel<1, W32, true>) : go(norm_rows_kernel<1, W32, false>);
    if (nv == 2) return full ? go(norm_rows_kernel<2, W32, true>) : go(norm_rows_kernel<2, W32, false>);
    return full ? go(norm_rows_kernel<4, W32, true>) : go(norm_rows_kernel<4, W32, false>);
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

cudaError_t add_parts(const NormBackwardArgs& a, int parts, cudaStream_t stream) {
    return launch_chained(norm_dweight_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(32 * ND_WARPS), 0, 0, stream,
                          static_cast<const float*>(a.partial), parts, a.cols, a.dw);
}

template <typename F, bool W32, bool FULL>
cudaError_t norm_backward(const NormBackwardArgs& a, int threads, cudaStream_t stream) {
    auto kernel = norm_backward_kernel<F, W32, FULL>;
    static PerDevice pd;
    int sms = 0;
    const cudaError_t e = per_device_once(pd, sms, [kernel](int& n) {
        n = device_sm_count();
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NB_STAGES * 3 * F::NV * F::THREADS * 16);
    });
    if (e != cudaSuccess) return e;
    // as many CTAs an SM as the registers hold, up to four (8192 x 2880, 192 threads, takes 32.7 us, and 41.0 with three)
    const int per_sm = min(4, F::THREADS * F::PER_SM / threads);
    const int parts = (int)min64((a.rows + NB_CLUSTER - 1) / NB_CLUSTER, min(NB_PARTS, per_sm * sms / NB_CLUSTER));
    const cudaError_t e2 = launch_chained(kernel, dim3(parts * NB_CLUSTER), dim3(threads),
                                          (size_t)NB_STAGES * (a.dsum ? 3 : 2) * F::NV * threads * 16, NB_CLUSTER, stream, a);
    return e2 != cudaSuccess ? e2 : add_parts(a, parts, stream);
}

template <int LANES, int NV, bool W32>
cudaError_t norm_backward_narrow(const NormBackwardArgs& a, cudaStream_t stream) {
    auto kernel = norm_backward_narrow_kernel<LANES, NV, W32>;
    constexpr int tensor = NBN_STAGES<NV> * NV * NBN_THREADS * 16;
    static PerDevice pd;
    int sms = 0;
    const cudaError_t e = per_device_once(pd, sms, [kernel](int& n) {
        n = device_sm_count();
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 3 * tensor);
    });
    if (e != cudaSuccess) return e;
    constexpr int rows_a_cta = NBN_THREADS / LANES;
    const int parts = (int)min64((a.rows + rows_a_cta - 1) / rows_a_cta, min(NB_PARTS, 2 * sms));
    const cudaError_t e2 = launch_chained(kernel, dim3(parts), dim3(NBN_THREADS), (size_t)(a.dsum ? 3 : 2) * tensor, 0, stream, a);
    return e2 != cudaSuccess ? e2 : add_parts(a, parts, stream);
}

template <bool W32>
cudaError_t norm_backward(const NormBackwardArgs& a, cudaStream_t stream) {
    if (a.cols <= 64) return norm_backward_narrow<8, 1, W32>(a, stream);
    if (a.cols <= 128) return norm_backward_narrow<16, 1, W32>(a, stream);
    if (a.cols <= 256) return norm_backward_narrow<32, 1, W32>(a, stream);
    if (a.cols <= 512) return norm_backward_narrow<32, 2, W32>(a, stream);
    if (a.cols <= 1024) return norm_backward_narrow<32, 4, W32>(a, stream);
    auto go = [&](auto form) {
        using F = decltype(form);
        const int threads = (int)(((a.cols + 8 * F::NV - 1) / (8 * F::NV) + 31) / 32 * 32);
        return a.cols == F::NV * threads * 8 ? norm_backward<F, W32, true>(a, threads, stream) : norm_backward<F, W32, false>(a, threads, stream);
    };
    // 768 threads an SM with 80 registers as long as a row's threads come near them with two vectors each, else 512 with 128 and four:
    // 8192 x 5120 takes 47.3 us, 2000 x 12288 31.8, 3421 x 8192 32.6 and 2000 x 16384 38.7, where 1024 threads with 64 registers,
    // which do not hold the weights, took 56.4, 40.1, 42.7 and 53.9
    if (a.cols <= 2048) return go(BackwardForm<256, 3, 1>{});
    if (a.cols <= 4096) return go(BackwardForm<256, 3, 2>{});
    if (a.cols <= 6144) return go(BackwardForm<384, 2, 2>{});
    if (a.cols <= 8192) return go(BackwardForm<256, 2, 4>{});
    if (a.cols <= 12288) return go(BackwardForm<768, 1, 2>{});
    return go(BackwardForm<512, 1, 4>{});
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
    return (size_t)min64(rows, NB_PARTS) * (size_t)cols * sizeof(float);
}

cudaError_t launch_rmsnorm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* h, int64_t ldh, const void* w, bool w32,
                                    float eps, int64_t rows, int64_t cols, const uint16_t* dsum, int64_t ldds, uint16_t* dx,
                                    int64_t lddx, float* dweight, void* workspace, cudaStream_t stream) {
    const NormBackwardArgs a{dy, lddy, h, ldh, w, eps, (float)(1.0 / (double)cols), rows, (int)cols, dsum, ldds, dx, lddx, dweight,
                             static_cast<float*>(workspace)};
    return w32 ? norm_backward<true>(a, stream) : norm_backward<false>(a, stream);
}

}  // namespace mxk
