// qkv_paged_store_step: bias, per-head q / k RMSNorm, neox rotation and the store into the
// pages, in one pass over the projected rows (include/qkv.h has the contract).
//
// Per token and head of q or k:  z = y + b;  n_i = z_i * inv * w_i with
// inv = 1 / sqrt(sum z^2 / hd + eps);  (n_d, n_{d + hd/2}) rotated by the angle pos * inv_freq[d].
// Every value is read once and written once, so the pass is bound by memory (or, for a few
// tokens, by one trip through the latencies of position -> angle and page id -> row).
#include "epilogue_math.cuh"
#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace {

using namespace qkv_epi;
using namespace qkv_paged;

constexpr int kThreads = 256;
constexpr int kSms = 152;
constexpr int kMaxTokens = 4;  // tokens of one CTA: one sincosf a thread at hd = 128

// Four neighbouring values as loaded.  Plain loads, not read-only ones: q may be written over Y.
template <typename YT>
struct Raw4;
template <>
struct Raw4<float> {
    float4 v;
    __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    __device__ __forceinline__ float4 get() const { return v; }
};
template <>
struct Raw4<uint16_t> {  // bf16
    uint2 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ float4 get() const {
        return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                           __uint_as_float(v.y & 0xffff0000u));
    }
};
__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

__device__ __forceinline__ void kv_put4(void* kv, int f16, int64_t idx, float4 v) {
    if (f16) {
        __half2 h[2] = {__floats2half2_rn(v.x, v.y), __floats2half2_rn(v.z, v.w)};
        *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(kv) + idx) = *reinterpret_cast<uint2*>(h);
    } else {
        *reinterpret_cast<float4*>(reinterpret_cast<float*>(kv) + idx) = v;
    }
}

__device__ __forceinline__ float4 add4(float4 a, float4 b) {
    return make_float4(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y), __fadd_rn(a.z, b.z), __fadd_rn(a.w, b.w));
}
__device__ __forceinline__ float4 norm4(float4 a, float inv, float4 w) {
    return make_float4(__fmul_rn(__fmul_rn(a.x, inv), w.x), __fmul_rn(__fmul_rn(a.y, inv), w.y),
                       __fmul_rn(__fmul_rn(a.z, inv), w.z), __fmul_rn(__fmul_rn(a.w, inv), w.w));
}
__device__ __forceinline__ float sq4(float4 a, float s) {
    return __fmaf_rn(a.x, a.x, __fmaf_rn(a.y, a.y, __fmaf_rn(a.z, a.z, __fmaf_rn(a.w, a.w, s))));
}
// 1 / rms of a head from the sum of its squares.
__device__ __forceinline__ float head_inv(const PagedStoreParams& p, float ss) {
    return rsqrtf(__fadd_rn(__fmul_rn(ss, p.inv_hd), p.eps));
}

// Where the CTA's tokens go: row offsets (-1: not stored), sequences and slots.
struct Tokens {
    int64_t row[kMaxTokens];
    int seq[kMaxTokens], slot[kMaxTokens], pos[kMaxTokens];
};

// Look up the CTA's tokens and make the (cos, sin) of their pairs.
__device__ __forceinline__ void token_tables(const PagedStoreParams& p, int t0, int nt, Tokens& tk,
                                             float2 (*cs_s)[QKV_MAX_HEAD_DIM / 2]) {
    const int half = p.hd >> 1;
    if (threadIdx.x < nt) {
        const int t = t0 + threadIdx.x;
        const int pos = __ldg(p.positions + t);
        const int seq = p.seqs ? __ldg(p.seqs + t) : t;
        const int slot = p.slots ? __ldg(p.slots + t) : pos;
        int64_t row = -1;
        if (seq >= p.c.n_seq) {
            flag_bad(kFlagIndexRange, seq);
        } else if (seq >= 0) {
            if (slot < 0 || slot >= p.c.max_pages * p.c.page_size) flag_bad(kFlagSlotRange, slot);
            else row = row_offset(p.c, seq, slot);
        }
        tk.row[threadIdx.x] = row;
        tk.seq[threadIdx.x] = seq;
        tk.slot[threadIdx.x] = slot;
        tk.pos[threadIdx.x] = pos;
    }
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
        const int t = i / half, d = i - t * half;
        cs_s[t][d] = rope_cos_sin(__ldg(p.positions + t0 + t), p.inv_freq[d]);
    }
}

// A k head's slot starts with no weight.
__device__ __forceinline__ void track_slot(const PagedStoreParams& p, const Tokens& tk, int t, int kv_head) {
    const int64_t at = (static_cast<int64_t>(tk.seq[t]) * p.nkv + kv_head) * p.c.max_pages * p.c.page_size + tk.slot[t];
    if (p.c.slot_weight) p.c.slot_weight[at] = 0.f;
    if (p.c.slot_pos) p.c.slot_pos[at] = tk.pos[t];
}

// LP lanes work on one head, four neighbouring pairs a lane (LP: the power of two at or above hd / 8; the
// lanes beyond idle).  A group keeps its head for the CTA's T tokens, so bias, norm weight and addresses are
// made once, and the loads of all T (of the next head, as each is used) are in flight together.
template <typename YT, int T>
__global__ void __launch_bounds__(kThreads) paged_store_kernel(const __grid_constant__ PagedStoreParams p, int lp,
                                                               int heads_per_cta) {
    __shared__ __align__(16) float2 cs_s[T][QKV_MAX_HEAD_DIM / 2];
    __shared__ Tokens tk;
    qkv_ptx::griddep_wait();
    const int half = p.hd >> 1;
    const int t0 = blockIdx.x * T, nt = min(T, p.nt - t0);
    const int end = min(p.nh + 2 * p.nkv, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
    const int groups = kThreads / lp, g = threadIdx.x / lp, l = threadIdx.x % lp, d = 4 * l;
    int h = blockIdx.y * heads_per_cta + g;
    const YT* y = static_cast<const YT*>(p.y) + t0 * p.y_stride + static_cast<int64_t>(h) * p.hd + d;
    Raw4<YT> n0[T], n1[T];
    const bool wide = d < half;  // a lane that has pairs
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (wide && h < end && t < nt) {
            n0[t].load(y + t * p.y_stride);
            n1[t].load(y + t * p.y_stride + half);
        }
    token_tables(p, t0, nt, tk, cs_s);
    __syncthreads();
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    // every group makes the same number of rounds: the lanes of a warp meet in its shuffles
    for (int h_first = blockIdx.y * heads_per_cta; h_first < end; h_first += groups, h += groups) {
        const bool live = wide && h < end;
        const int sec = h < p.nh ? 0 : h < p.nh + p.nkv ? 1 : 2;
        const int j = (sec == 0 ? h : sec == 1 ? h - p.nh : h - p.nh - p.nkv) * p.hd + d;  // within the section
        const bool norm = p.norm_w[0] != nullptr;  // v heads then only join the shuffles
        float4 b0 = zero, b1 = zero, w0 = zero, w1 = zero;
        if (live && p.bias) {
            b0 = load4(p.bias + static_cast<int64_t>(h) * p.hd + d);
            b1 = load4(p.bias + static_cast<int64_t>(h) * p.hd + half + d);
        }
        if (live && norm && sec != 2) {
            w0 = load4(p.norm_w[sec] + d);
            w1 = load4(p.norm_w[sec] + half + d);
        }
        y += static_cast<int64_t>(groups) * p.hd;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            float4 a0 = zero, a1 = zero;
            if (live && t < nt) {
                a0 = n0[t].get();
                a1 = n1[t].get();
            }
            if (wide && h + groups < end && t < nt) {
                n0[t].load(y + t * p.y_stride);
                n1[t].load(y + t * p.y_stride + half);
            }
            if (p.bias) {
                a0 = add4(a0, b0);
                a1 = add4(a1, b1);
            }
            float inv = 0.f;
            if (norm) {
                float ss = sq4(a0, sq4(a1, 0.f));
                for (int o = lp >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                inv = head_inv(p, ss);
            }
            if (!live || t >= nt || tk.seq[t] < 0) continue;
            if (sec != 2) {
                if (norm) {
                    a0 = norm4(a0, inv, w0);
                    a1 = norm4(a1, inv, w1);
                }
                const float4 c0 = *reinterpret_cast<const float4*>(cs_s[t] + d);
                const float4 c1 = *reinterpret_cast<const float4*>(cs_s[t] + d + 2);
                float4 r0, r1;
                rope_rotate_cs(a0.x, a1.x, make_float2(c0.x, c0.y), r0.x, r1.x);
                rope_rotate_cs(a0.y, a1.y, make_float2(c0.z, c0.w), r0.y, r1.y);
                rope_rotate_cs(a0.z, a1.z, make_float2(c1.x, c1.y), r0.z, r1.z);
                rope_rotate_cs(a0.w, a1.w, make_float2(c1.z, c1.w), r0.w, r1.w);
                a0 = r0;
                a1 = r1;
            }
            const int64_t row = tk.row[t];
            if (sec == 0) {
                float* q = p.q + (t0 + t) * p.q_stride + j;
                *reinterpret_cast<float4*>(q) = a0;
                *reinterpret_cast<float4*>(q + half) = a1;
            } else if (row >= 0) {
                void* kv = sec == 1 ? p.c.k : p.c.v;
                kv_put4(kv, p.kv_f16, row + j, a0);
                kv_put4(kv, p.kv_f16, row + j + half, a1);
                if (sec == 1 && l == 0) track_slot(p, tk, t, h - p.nh);
            }
        }
    }
}

// Any even hd, any alignment: a warp strides over a head's pairs one by one; a token a CTA row.
template <typename YT>
__global__ void __launch_bounds__(kThreads) paged_store_any_kernel(const __grid_constant__ PagedStoreParams p,
                                                                   int heads_per_cta) {
    __shared__ float2 cs_s[1][QKV_MAX_HEAD_DIM / 2];
    __shared__ Tokens tk;
    qkv_ptx::griddep_wait();
    const int half = p.hd >> 1, t = blockIdx.x, lane = threadIdx.x & 31;
    const int end = min(p.nh + 2 * p.nkv, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
    token_tables(p, t, 1, tk, cs_s);
    __syncthreads();
    if (tk.seq[0] < 0) return;
    const int64_t row = tk.row[0];
    for (int h = blockIdx.y * heads_per_cta + (threadIdx.x >> 5); h < end; h += kThreads / 32) {
        const int sec = h < p.nh ? 0 : h < p.nh + p.nkv ? 1 : 2;
        const int j0 = (sec == 0 ? h : sec == 1 ? h - p.nh : h - p.nh - p.nkv) * p.hd;  // within the section
        const YT* y = static_cast<const YT*>(p.y) + t * p.y_stride + static_cast<int64_t>(h) * p.hd;
        const float* b = p.bias ? p.bias + static_cast<int64_t>(h) * p.hd : nullptr;
        const float* w = sec == 2 ? nullptr : p.norm_w[sec];
        float* q = p.q + t * p.q_stride + j0;
        void* kv = sec == 1 ? p.c.k : p.c.v;
        float inv = 0.f;
        if (w) {
            float ss = 0.f;
            for (int d = lane; d < p.hd; d += 32) {
                const float z = b ? __fadd_rn(load1(y + d), __ldg(b + d)) : load1(y + d);
                ss = __fmaf_rn(z, z, ss);
            }
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            inv = head_inv(p, ss);
        }
        for (int d = lane; d < half; d += 32) {
            float z0 = load1(y + d), z1 = load1(y + half + d);
            if (b) {
                z0 = __fadd_rn(z0, __ldg(b + d));
                z1 = __fadd_rn(z1, __ldg(b + half + d));
            }
            if (sec != 2) {
                if (w) {
                    z0 = __fmul_rn(__fmul_rn(z0, inv), __ldg(w + d));
                    z1 = __fmul_rn(__fmul_rn(z1, inv), __ldg(w + half + d));
                }
                float r0, r1;
                rope_rotate_cs(z0, z1, cs_s[0][d], r0, r1);
                z0 = r0;
                z1 = r1;
            }
            if (sec == 0) {
                q[d] = z0;
                q[half + d] = z1;
            } else if (row >= 0) {
                kv_put(kv, p.kv_f16, static_cast<size_t>(row + j0 + d), z0);
                kv_put(kv, p.kv_f16, static_cast<size_t>(row + j0 + half + d), z1);
            }
        }
        if (lane == 0 && sec == 1 && row >= 0) track_slot(p, tk, 0, h - p.nh);
    }
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename YT>
cudaError_t launch_t(const PagedStoreParams& p, cudaStream_t stream) {
    const int ys = sizeof(YT), es = p.kv_f16 ? 2 : 4;
    const bool vec = p.hd % 8 == 0 && aligned(p.y, 4 * ys) && p.y_stride % 4 == 0 && aligned(p.bias, 16) &&
                     aligned(p.norm_w[0], 16) && aligned(p.norm_w[1], 16) && aligned(p.q, 16) &&
                     p.q_stride % 4 == 0 && aligned(p.c.k, 4 * es) && aligned(p.c.v, 4 * es) &&
                     p.c.page_stride % 4 == 0;
    int lp = 1;
    while (lp < (vec ? p.hd / 8 : 32)) lp *= 2;
    // Tokens share a CTA (and what a head needs) once there are enough for every SM; before that the
    // heads of a token are spread over CTAs, down to one round each, at the price of more angles.
    const bool many = vec && p.nt >= kMaxTokens * 4 * kSms;
    const int heads = p.nh + 2 * p.nkv, tokens = many ? kMaxTokens : 1;
    int per = heads;
    while (!many && per > kThreads / lp && static_cast<int64_t>(p.nt) * ((heads + per - 1) / per) < kSms) per = (per + 1) / 2;
    const dim3 grid((p.nt + tokens - 1) / tokens, (heads + per - 1) / per);
    if (!vec) return launch_dependent(paged_store_any_kernel<YT>, grid, kThreads, 0, stream, p, per);
    return launch_dependent(many ? paged_store_kernel<YT, kMaxTokens> : paged_store_kernel<YT, 1>, grid, kThreads, 0,
                            stream, p, lp, per);
}

}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, int y_dtype, cudaStream_t stream) {
    return y_dtype == QKV_BF16 ? launch_t<uint16_t>(p, stream) : launch_t<float>(p, stream);
}

cudaError_t paged_store_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
