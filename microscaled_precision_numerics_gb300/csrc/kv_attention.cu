// kv_attention.cu -- attention of a generation step over the NVFP4 key/value cache.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j - m_i),  k_j = val(code) * val(block scale) * S_k
//
// over the cached positions j in (pos_i - window, pos_i], pos_i = L - N + i for new token i of a request with L
// cached tokens of which N are new.
#include "mx_internal.h"
#include "mx_kv.cuh"

namespace mxk {

namespace {

// One CTA for each (new token, q head): its four warps take every fourth cached token, a lane D / 32 elements
// of it, with a running maximum and sum each, and join at the end.
template <int D>
__global__ void __launch_bounds__(128) kv_attention_simple_kernel(const KvAttentionArgs a) {
    constexpr int E = D / 32;
    const int t = blockIdx.x, hq = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int lo = 0, hi = a.R;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.q_start + mid) <= t) lo = mid; else hi = mid;
    }
    const int r = lo, first = __ldg(a.q_start + r), count = __ldg(a.q_start + r + 1) - first, len = __ldg(a.seq_lens + r);
    const int pos = len - count + (t - first);
    const int begin = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int h = hq / a.group;
    const float S_k = __ldg(a.s_k + h), S_v = __ldg(a.s_v + h);
    float q[E], o[E] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const uint32_t b = __ldg(a.q + t * a.q_token + hq * a.q_head + lane * E + e);
        q[e] = __uint_as_float(b << 16) * S_k;
    }
    const int nb = D / 16, blk = lane * E / 16;
    for (int j = begin + warp; j <= pos; j += 4) {
        const int64_t col = j / a.page;
        const int page = col < a.width ? __ldg(a.table + r * a.stride + col) : -1;
        if (page < 0 || page >= a.pages) continue;
        const int off = j % a.page, tok = off & 15;
        const uint8_t* rec = a.cache + (((int64_t)page * a.kv_heads + h) * (a.page / KV_GROUP) + off / KV_GROUP) * kv_record_bytes(D);
        const float ks = e4m3_to_f32(rec[kv_k_scales(D) + tok * nb + blk]);
        const float vs = e4m3_to_f32(rec[kv_v_scales(D) + blk * 16 + kv_token_of_row(tok)]);
        float dot = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const int at = tok * (D / 2) + (lane * E + e) / 2;
            const uint32_t kw = e2m1x2_to_f16x2(rec[at]), vw = e2m1x2_to_f16x2(rec[kv_v_codes(D) + at]);
            const __half2 kp = *reinterpret_cast<const __half2*>(&kw), vp = *reinterpret_cast<const __half2*>(&vw);
            dot = fmaf(q[e], __low2float(kp) * ks, dot);
            dot = fmaf(q[e + 1], __high2float(kp) * ks, dot);
            v[e] = __low2float(vp) * vs;
            v[e + 1] = __high2float(vp) * vs;
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xFFFFFFFFu, dot, s);
        dot *= a.scale;
        const float mn = fmaxf(m, dot), c = expf(m - mn), p = expf(dot - mn);
        l = fmaf(l, c, p);
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(o[e], c, p * v[e]);
        m = mn;
    }
    __shared__ float s_m[4], s_l[4], s_o[4][D];
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][lane * E + e] = o[e];
    __syncthreads();
    float top = -INFINITY, sum = 0.0f;
    for (int w = 0; w < 4; ++w) top = fmaxf(top, s_m[w]);
    float c[4];
    for (int w = 0; w < 4; ++w) {
        c[w] = s_l[w] > 0.0f ? expf(s_m[w] - top) : (s_l[w] == 0.0f ? 0.0f : s_l[w]);
        sum += c[w] * s_l[w];
    }
    for (int d = threadIdx.x; d < D; d += 128) {
        float x = 0.0f;
        for (int w = 0; w < 4; ++w) x += c[w] * s_o[w][d];
        x = sum == 0.0f ? 0.0f : x * S_v / sum;
        a.out[t * a.o_token + hq * a.o_head + d] = (uint16_t)pack_bf16x2(x, 0.0f);
    }
    if (a.lse && threadIdx.x == 0) a.lse[(int64_t)t * gridDim.y + hq] = sum == 0.0f ? -INFINITY : top + logf(sum);
}

}  // namespace

size_t kv_attention_workspace_bytes(int64_t) { return 16; }

cudaError_t launch_kv_attention(const KvAttentionArgs& a, int, cudaStream_t stream) {
    const dim3 grid((unsigned)a.T, (unsigned)(a.kv_heads * a.group));
    if (a.dim == 64) kv_attention_simple_kernel<64><<<grid, 128, 0, stream>>>(a);
    else if (a.dim == 128) kv_attention_simple_kernel<128><<<grid, 128, 0, stream>>>(a);
    else kv_attention_simple_kernel<256><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace mxk
