// qkv_attn_step: attention of one new token per sequence over a paged cache
// (include/qkv.h has the contract).
//
// s_j = scale * q.K_j, online softmax (running maximum m and sum l), out = sum p_j V_j / l.
// Scores are kept in the log2 domain (scale * log2(e) folded into q), so p = 2^(s - m).
#include <math_constants.h>

#include "paged_common.cuh"

namespace {

using namespace qkv_paged;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ void put_out(const PagedAttnParams& p, int b, int h, int d, float v) {
    const int64_t at = b * p.out_stride + static_cast<int64_t>(h) * p.hd + d;
    if (p.out_bf16) {
        const uint32_t u = __float_as_uint(v);  // round to nearest even; NaN stays NaN
        const uint16_t r = (u & 0x7fffffffu) > 0x7f800000u ? static_cast<uint16_t>(0x7fffu)
                                                            : static_cast<uint16_t>((u + 0x7fffu + ((u >> 16) & 1u)) >> 16);
        static_cast<uint16_t*>(p.out)[at] = r;
    } else {
        static_cast<float*>(p.out)[at] = v;
    }
}

// lse of head h of sequence b from its maximum and sum (log2 domain); an empty row has sum 0.
__device__ __forceinline__ void put_lse(const PagedAttnParams& p, int b, int h, float m, float l, bool empty) {
    const float lse2 = empty ? -CUDART_INF_F : m + log2f(l);
    const int64_t at = static_cast<int64_t>(b) * p.nh + h;
    if (p.lse) p.lse[at] = lse2 * kLn2;
    if (p.add_weight) p.lse2[at] = lse2;
}

__device__ __forceinline__ float kv_get(const void* kv, int f16, int64_t i) {
    return f16 ? __half2float(static_cast<const __half*>(kv)[i]) : static_cast<const float*>(kv)[i];
}

// ---------------------------------------------------------------- any head_dim, any alignment

constexpr int kAnyThreads = 128, kAnyTile = 128;

// One CTA per (sequence, q head), tiles of 128 slots: a warp per slot for the dots, a thread per
// output column for the sum.
__global__ void __launch_bounds__(kAnyThreads) paged_attn_any_kernel(const __grid_constant__ PagedAttnParams p) {
    __shared__ float q_s[QKV_MAX_HEAD_DIM];
    __shared__ float s_s[kAnyTile];
    __shared__ int64_t row_s[kAnyTile];
    __shared__ float red_s[2 * kAnyThreads / 32];
    const int b = blockIdx.x / p.nh, h = blockIdx.x - b * p.nh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = h / (p.nh / p.nkv) * p.hd;
    const int n = checked_len(p.c, p.lens, b);
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    for (int d = tid; d < p.hd; d += kAnyThreads)
        q_s[d] = p.q[b * p.q_stride + static_cast<int64_t>(h) * p.hd + d] * (p.scale * kLog2e);
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    float* scores = p.add_weight ? p.scores + (static_cast<int64_t>(b) * p.nh + h) * cap : nullptr;
    float m = -CUDART_INF_F, l = 0.f, acc[QKV_MAX_HEAD_DIM / kAnyThreads] = {};
    for (int j = first; j < n; j += kAnyTile) {
        const int nj = min(kAnyTile, n - j);
        if (tid < nj) row_s[tid] = row_offset(p.c, b, j + tid);
        __syncthreads();
        for (int i = warp; i < nj; i += kAnyThreads / 32) {
            const int64_t row = row_s[i];
            float s = 0.f;
            if (row >= 0)
                for (int d = lane; d < p.hd; d += 32) s = fmaf(q_s[d], kv_get(p.c.k, p.kv_f16, row + j0 + d), s);
            for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
            if (lane == 0) {
                s_s[i] = row >= 0 ? s : -CUDART_INF_F;
                if (scores) scores[j + i] = s_s[i];
            }
        }
        __syncthreads();
        // a NaN score makes the maximum NaN (as max over the formula's scores) through the sum below
        const float s = tid < nj ? s_s[tid] : -CUDART_INF_F;
        float mt = s;
        for (int o = 16; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        if (lane == 0) red_s[warp] = mt;
        __syncthreads();
        mt = fmaxf(fmaxf(red_s[0], red_s[1]), fmaxf(red_s[2], red_s[3]));
        const float mn = fmaxf(m, mt);
        const float keep = m == mn ? 1.f : exp2f(m - mn);  // m == mn also where both are infinite
        const float pr = tid < nj ? (s == -CUDART_INF_F && mn == -CUDART_INF_F ? 0.f : exp2f(s - mn)) : 0.f;
        if (tid < nj) s_s[tid] = pr;
        float lt = pr;
        for (int o = 16; o; o >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, o);
        if (lane == 0) red_s[4 + warp] = lt;
        __syncthreads();
        l = l * keep + (red_s[4] + red_s[5] + red_s[6] + red_s[7]);
        m = mn;
        for (int k = 0; k < QKV_MAX_HEAD_DIM / kAnyThreads; ++k) {
            const int d = tid + k * kAnyThreads;
            if (d >= p.hd) break;
            float a = acc[k] * keep;
            for (int i = 0; i < nj; ++i)
                if (row_s[i] >= 0) a = fmaf(s_s[i], kv_get(p.c.v, p.kv_f16, row_s[i] + j0 + d), a);
            acc[k] = a;
        }
        __syncthreads();
    }
    for (int k = 0; k < QKV_MAX_HEAD_DIM / kAnyThreads; ++k) {
        const int d = tid + k * kAnyThreads;
        if (d < p.hd) put_out(p, b, h, d, first < n ? acc[k] / l : 0.f);
    }
    if (tid == 0) put_lse(p, b, h, m, l, first >= n);
}

// ---------------------------------------------------------------- running attention weights

constexpr int kWeightThreads = 256;

// slot_weight[b][kv head][j] += sum over the kv head's q heads of 2^(score - lse): one thread a slot.
__global__ void __launch_bounds__(kWeightThreads) paged_attn_weight_kernel(const __grid_constant__ PagedAttnParams p,
                                                                           int chunks) {
    const int item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
    const int b = item / p.nkv, hk = item - b * p.nkv, G = p.nh / p.nkv;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    int n = __ldg(p.lens + b);
    if (n < 0 || n > cap) n = 0;  // flagged by the attention kernel
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    const int64_t h0 = static_cast<int64_t>(b) * p.nh + static_cast<int64_t>(hk) * G;
    float* weight = p.c.slot_weight + static_cast<int64_t>(item) * cap;
    for (int64_t j = first + static_cast<int64_t>(chunk) * kWeightThreads + threadIdx.x; j < n;
         j += static_cast<int64_t>(chunks) * kWeightThreads) {
        float w = 0.f;
        for (int g = 0; g < G; ++g) w += exp2f(p.scores[(h0 + g) * cap + j] - p.lse2[h0 + g]);
        weight[j] += w;
    }
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, cudaStream_t stream) {
    paged_attn_any_kernel<<<p.c.n_seq * p.nh, kAnyThreads, 0, stream>>>(p);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || !p.add_weight) return e;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    const int chunks = static_cast<int>(cap / kWeightThreads / 8 + 1);
    paged_attn_weight_kernel<<<p.c.n_seq * p.nkv * chunks, kWeightThreads, 0, stream>>>(p, chunks);
    return cudaGetLastError();
}

cudaError_t paged_attn_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
