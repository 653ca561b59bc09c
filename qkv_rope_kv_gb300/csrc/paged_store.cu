// qkv_paged_store_step: bias, per-head q / k RMSNorm, neox rotation and the store into the
// pages, in one pass over the projected rows (include/qkv.h has the contract).
//
// Per token and head of q or k:  z = y + b;  n_i = z_i * inv * w_i with
// inv = 1 / sqrt(sum z^2 / hd + eps);  (n_d, n_{d + hd/2}) rotated by the angle pos * inv_freq[d].
// Every value is read once and written once, so the pass is bound by memory (or, for a few
// tokens, by one trip through the latencies of position -> angle and page id -> row).
// Measured (GPU time): one token 2.5 us, 64 of 40 + 2 x 8 heads of 128 with norms 3.1 us, 8191 of them 60.2 us
// (318.9 MB at 5.3 TB/s, 0.78 of the copy rate; issue slots are 72 % busy).  There, one token per CTA takes
// 73 us, four 64.5, loads without a branch 73, seven warps 61.7.
// With a qkv_rope, 32 tokens of 28 + 2 x 4 heads 2.9 us, 8191 of the above (halves, ramp) 68.8: its angles take a 64-bit product
// and a sine and cosine of turns instead of a table's factor.  (Issue slots are 58 % busy, DRAM at 0.68 of the copy rate: what
// bounds it is not established.)
#include "epilogue_math.cuh"
#include "paged_common.cuh"
#include "ptx_sync.cuh"
#include "rope_math.cuh"

namespace {

using namespace qkv_epi;
using namespace qkv_paged;
using namespace qkv_rope_math;

constexpr int kThreads = 256;
// Tokens of one CTA: what fits 64 registers, so four CTAs on an SM (bf16 rows 62; f32 rows spill 76 bytes).
constexpr int kMaxTokens = 3;

// Four neighbouring values of Y as loaded.  Plain loads, not read-only ones: q may be written over Y.
template <typename YT>
struct Raw4;
template <>
struct Raw4<float> {
    Quad v;
    __device__ __forceinline__ void load(const float* p) { v = quad(p); }
    __device__ __forceinline__ Quad get() const { return v; }
};
template <>
struct Raw4<uint16_t> {  // bf16
    uint2 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ Quad get() const {
        return {pack(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)),
                pack(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u))};
    }
};
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) {
    return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}

__device__ __forceinline__ void kv_put4(void* kv, int f16, int64_t idx, Quad v) {
    if (f16) {
        const float2 x = unpack(v.a), y = unpack(v.b);
        __half2 h[2] = {__floats2half2_rn(x.x, x.y), __floats2half2_rn(y.x, y.y)};
        *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(kv) + idx) = *reinterpret_cast<uint2*>(h);
    } else {
        *reinterpret_cast<ulonglong2*>(reinterpret_cast<float*>(kv) + idx) = make_ulonglong2(v.a, v.b);
    }
}

// 1 / rms of a head from the sum of its squares.
__device__ __forceinline__ float head_inv(const PagedStoreParams& p, float ss) {
    return rsqrtf(__fadd_rn(__fmul_rn(ss, p.inv_hd), p.eps));
}

// The rotation: the plan's, or a qkv_rope's with its pairs half a head apart or neighbours.
enum Form { kPlan, kHalves, kNeighbours };
template <Form F>
struct Rotation {  // what the parameters do not hold of it
    RopeTable table;
    __device__ __forceinline__ int rot(const PagedStoreParams&) const { return table.rot; }
    __device__ __forceinline__ float2 at(const PagedStoreParams&, int pos, int d) const { return cos_sin(table, pos, d); }
};
template <>
struct Rotation<kPlan> {
    __device__ __forceinline__ int rot(const PagedStoreParams& p) const { return p.hd; }
    __device__ __forceinline__ float2 at(const PagedStoreParams& p, int pos, int d) const {
        return rope_cos_sin(pos, p.inv_freq[d]);
    }
};

// Where the CTA's tokens go: row offsets (-1: not stored), sequences and slots.
struct Tokens {
    int64_t row[kMaxTokens];
    int seq[kMaxTokens], slot[kMaxTokens], pos[kMaxTokens];
};

// Look up the CTA's tokens and make the (cos, sin) of their pairs.
template <Form F>
__device__ __forceinline__ void token_tables(const PagedStoreParams& p, const Rotation<F>& r, int t0, int nt, Tokens& tk,
                                             float (*cos_s)[QKV_MAX_HEAD_DIM / 2],
                                             float (*sin_s)[QKV_MAX_HEAD_DIM / 2]) {
    const int half = r.rot(p) >> 1;
    if (threadIdx.x < nt) {
        const int t = t0 + threadIdx.x;
        const int pos = p.positions[t];
        const int seq = p.seqs ? p.seqs[t] : t;
        const int slot = p.slots ? p.slots[t] : pos;
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
        const float2 cs = r.at(p, p.positions[t0 + t], d);
        cos_s[t][d] = cs.x;
        sin_s[t][d] = cs.y;
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
// (Of a qkv_rope's halves, the values that pass go by eight neighbours a lane; so do all where pairs are neighbours.)
template <typename YT, int T, Form F>
__global__ void __launch_bounds__(kThreads, 4) paged_store_kernel(const __grid_constant__ PagedStoreParams p,
                                                               const __grid_constant__ Rotation<F> r, int lp,
                                                               int heads_per_cta) {
    __shared__ __align__(16) float cos_s[T][QKV_MAX_HEAD_DIM / 2], sin_s[T][QKV_MAX_HEAD_DIM / 2];
    __shared__ Tokens tk;
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int half = p.hd >> 1, rot = r.rot(p);
    const int t0 = blockIdx.x * T, nt = min(T, p.nt - t0);
    const int end = min(p.nh + 2 * p.nkv, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
    const int groups = kThreads / lp, g = threadIdx.x / lp, l = threadIdx.x % lp;
    int h = blockIdx.y * heads_per_cta + g;
    // a lane's two quads, and whether it has any
    int d0 = 4 * l, apart = half;
    bool wide = d0 < half;
    if constexpr (F != kPlan) {
        int d1;
        lane_quads<F == kNeighbours>(l, rot, d0, d1);
        apart = d1 - d0;
        wide = 8 * l < p.hd;
    }
    const YT* y = static_cast<const YT*>(p.y) + t0 * p.y_stride + static_cast<int64_t>(h) * p.hd + d0;
    Raw4<YT> n0[T], n1[T];
#pragma unroll
    for (int t = 0; t < T; ++t)
        if (wide && h < end && t < nt) {
            n0[t].load(y + t * p.y_stride);
            n1[t].load(y + t * p.y_stride + apart);
        }
    token_tables(p, r, t0, nt, tk, cos_s, sin_s);
    __syncthreads();
    int64_t rows[T];
    bool here[T];  // a token that is no padding
#pragma unroll
    for (int t = 0; t < T; ++t) {
        here[t] = t < nt && tk.seq[t] >= 0;
        rows[t] = here[t] ? tk.row[t] : -1;
    }
    const bool norm = p.norm_w[0] != nullptr;
    // every group makes the same number of rounds: the lanes of a warp meet in its shuffles
    for (int h_first = blockIdx.y * heads_per_cta; h_first < end; h_first += groups, h += groups) {
        const bool live = wide && h < end, ahead = wide && h + groups < end;
        const int sec = h < p.nh ? 0 : h < p.nh + p.nkv ? 1 : 2;
        const int j = (sec == 0 ? h : sec == 1 ? h - p.nh : h - p.nh - p.nkv) * p.hd + d0;  // within the section
        Quad b0 = {0, 0}, b1 = {0, 0}, w0 = {0, 0}, w1 = {0, 0};
        if (live && p.bias) {
            b0 = quad(p.bias + static_cast<int64_t>(h) * p.hd + d0);
            b1 = quad(p.bias + static_cast<int64_t>(h) * p.hd + apart + d0);
        }
        if (live && norm && sec != 2) {
            w0 = quad(p.norm_w[sec] + d0);
            w1 = quad(p.norm_w[sec] + apart + d0);
        }
        y += static_cast<int64_t>(groups) * p.hd;
        float* q = p.q + t0 * p.q_stride + j;
        void* kv = sec == 1 ? p.c.k : p.c.v;
#pragma unroll
        for (int t = 0; t < T; ++t) {
            Quad x0 = {0, 0}, x1 = {0, 0};
            if (live && t < nt) {
                x0 = n0[t].get();
                x1 = n1[t].get();
            }
            if (ahead && t < nt) {
                n0[t].load(y + t * p.y_stride);
                n1[t].load(y + t * p.y_stride + apart);
            }
            if (p.bias) {
                x0 = {add2(x0.a, b0.a), add2(x0.b, b0.b)};
                x1 = {add2(x1.a, b1.a), add2(x1.b, b1.b)};
            }
            if (norm) {  // v heads only join the shuffles
                const float2 sq = unpack(fma2(x0.a, x0.a, fma2(x0.b, x0.b, fma2(x1.a, x1.a, mul2(x1.b, x1.b)))));
                float ss = sq.x + sq.y;
                for (int o = lp >> 1; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
                if (sec != 2) {
                    const float inv = head_inv(p, ss);
                    const u64 i2 = pack(inv, inv);
                    x0 = {mul2(mul2(x0.a, i2), w0.a), mul2(mul2(x0.b, i2), w0.b)};
                    x1 = {mul2(mul2(x1.a, i2), w1.a), mul2(mul2(x1.b, i2), w1.b)};
                }
            }
            if (!live || !here[t]) continue;
            if (sec != 2 && (F == kPlan || 8 * l < rot)) {
                const Quad c = quad(cos_s[t] + 4 * l), s = quad(sin_s[t] + 4 * l);
                if (F == kNeighbours) {
                    rotate_neighbours(x0, x1, c, s);
                } else {
                    Quad r0, r1;
                    rotate2(x0.a, x1.a, c.a, s.a, r0.a, r1.a);
                    rotate2(x0.b, x1.b, c.b, s.b, r0.b, r1.b);
                    x0 = r0;
                    x1 = r1;
                }
            }
            if (sec == 0) {
                *reinterpret_cast<ulonglong2*>(q + t * p.q_stride) = make_ulonglong2(x0.a, x0.b);
                *reinterpret_cast<ulonglong2*>(q + t * p.q_stride + apart) = make_ulonglong2(x1.a, x1.b);
            } else if (rows[t] >= 0) {
                kv_put4(kv, p.kv_f16, rows[t] + j, x0);
                kv_put4(kv, p.kv_f16, rows[t] + j + apart, x1);
                if (sec == 1 && l == 0) track_slot(p, tk, t, h - p.nh);
            }
        }
    }
}

// Any even hd, any alignment: a warp strides over a head's pairs one by one; a token a CTA row.
template <typename YT, Form F>
__global__ void __launch_bounds__(kThreads) paged_store_any_kernel(const __grid_constant__ PagedStoreParams p,
                                                                   const __grid_constant__ Rotation<F> r,
                                                                   int heads_per_cta) {
    __shared__ float cos_s[1][QKV_MAX_HEAD_DIM / 2], sin_s[1][QKV_MAX_HEAD_DIM / 2];
    __shared__ Tokens tk;
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int half = p.hd >> 1, turn = r.rot(p) >> 1, t = blockIdx.x, lane = threadIdx.x & 31;
    const int end = min(p.nh + 2 * p.nkv, static_cast<int>(blockIdx.y + 1) * heads_per_cta);
    token_tables(p, r, t, 1, tk, cos_s, sin_s);
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
            // the pair's two values; behind the last pair, two that pass
            int d0 = d, d1 = turn + d;
            if (F == kNeighbours || (F == kHalves && d >= turn)) {
                d0 = 2 * d;
                d1 = 2 * d + 1;
            }
            float z0 = load1(y + d0), z1 = load1(y + d1);
            if (b) {
                z0 = __fadd_rn(z0, __ldg(b + d0));
                z1 = __fadd_rn(z1, __ldg(b + d1));
            }
            if (sec != 2) {
                if (w) {
                    z0 = __fmul_rn(__fmul_rn(z0, inv), __ldg(w + d0));
                    z1 = __fmul_rn(__fmul_rn(z1, inv), __ldg(w + d1));
                }
                if (F == kPlan || d < turn) {
                    float r0, r1;
                    rope_rotate_cs(z0, z1, make_float2(cos_s[0][d], sin_s[0][d]), r0, r1);
                    z0 = r0;
                    z1 = r1;
                }
            }
            if (sec == 0) {
                q[d0] = z0;
                q[d1] = z1;
            } else if (row >= 0) {
                kv_put(kv, p.kv_f16, static_cast<size_t>(row + j0 + d0), z0);
                kv_put(kv, p.kv_f16, static_cast<size_t>(row + j0 + d1), z1);
            }
        }
        if (lane == 0 && sec == 1 && row >= 0) track_slot(p, tk, 0, h - p.nh);
    }
}

bool aligned(const void* p, int n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename YT, Form F>
cudaError_t launch_t(const PagedStoreParams& p, const Rotation<F>& r, bool eights, cudaStream_t stream) {
    const int ys = sizeof(YT), es = p.kv_f16 ? 2 : 4;
    const bool vec = p.hd % 8 == 0 && eights && aligned(p.y, 4 * ys) && p.y_stride % 4 == 0 && aligned(p.bias, 16) &&
                     aligned(p.norm_w[0], 16) && aligned(p.norm_w[1], 16) && aligned(p.q, 16) &&
                     p.q_stride % 4 == 0 && aligned(p.c.k, 4 * es) && aligned(p.c.v, 4 * es) &&
                     p.c.page_stride % 4 == 0;
    int lp = 1;
    while (lp < (vec ? p.hd / 8 : 32)) lp *= 2;
    // Tokens share a CTA (and what a head needs) once there are enough for every SM; before that the
    // heads of a token are spread over CTAs, down to one round each, at the price of more angles.
    const bool many = vec && p.nt >= 16 * kSms;
    const int heads = p.nh + 2 * p.nkv, tokens = many ? kMaxTokens : 1;
    int per = heads;
    while (!many && per > kThreads / lp && static_cast<int64_t>(p.nt) * ((heads + per - 1) / per) < kSms) per = (per + 1) / 2;
    const dim3 grid((p.nt + tokens - 1) / tokens, (heads + per - 1) / per);
    if (!vec) return launch_dependent(paged_store_any_kernel<YT, F>, grid, kThreads, 0, stream, 1, p, r, per);
    return launch_dependent(many ? paged_store_kernel<YT, kMaxTokens, F> : paged_store_kernel<YT, 1, F>, grid, kThreads,
                            0, stream, 1, p, r, lp, per);
}

}  // namespace

cudaError_t launch_paged_store(const PagedStoreParams& p, const RopeTable* rope, int y_dtype, cudaStream_t stream) {
    const bool bf16 = y_dtype == QKV_BF16;
    if (!rope) return (bf16 ? launch_t<uint16_t, kPlan> : launch_t<float, kPlan>)(p, {}, true, stream);
    const bool eights = rope->rot % 8 == 0;  // a lane's eight values all turn or all pass
    if (rope->neighbours)
        return (bf16 ? launch_t<uint16_t, kNeighbours> : launch_t<float, kNeighbours>)(p, {*rope}, eights, stream);
    return (bf16 ? launch_t<uint16_t, kHalves> : launch_t<float, kHalves>)(p, {*rope}, eights, stream);
}

cudaError_t paged_store_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
