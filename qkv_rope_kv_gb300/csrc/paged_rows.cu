// Attention of many q rows over a paged cache (qkv_prompt_attn_step, and the prefix of qkv_prefix_attn_step; include/qkv.h
// has the contracts): any head size, cache type and alignment, in f32.
//
// s_j = scale * q.K_j, running maximum m and sum l of each row, out = sum p_j V_j / l, scores in log2 terms.  A tile of 64
// rows goes over blocks of 64 slots: both products are made by plain f32 multiply-adds from shared memory, each thread 4 x 4
// scores and 4 rows x hd / 16 columns of the sums.  Multiply-adds bound it (and their operands' reads from shared memory) where
// there are many rows; a few, 17 tokens of 14 heads over 2, take 17.5 us with the plan and the join: a chain of latencies.
#include "paged_rows.cuh"

namespace {

using namespace qkv_rows;
using qkv_ptx::griddep_launch_dependents;
using qkv_ptx::griddep_wait;

constexpr int kThreads = 256, kRows = 64, kBlock = 64;
constexpr int kPStride = kBlock + 4;

template <int HDP>
struct Shape {
    static constexpr int kStride = HDP + 4;  // floats of a row: sixteen rows' quads fall into different banks
    static constexpr int kCols = HDP / 64;   // quads of columns of a thread
    static constexpr int kSmem = 4 * (2 * 64 * kStride + kRows * kPStride);
    static constexpr int kCtas = HDP == 256 ? 1 : 2;  // an SM
};

__device__ __forceinline__ float get(const float* p) { return __ldg(p); }
__device__ __forceinline__ float get(const __half* p) { return __half2float(__ldg(p)); }

// A block of K or V on its way to shared memory: all 16-byte pieces of a thread in flight together.  Slots that are not
// there, and columns behind hd, are zeros.
template <typename KT, int HDP>
struct Block {
    static constexpr int kPer = 16 / sizeof(KT);                          // values of a piece
    static constexpr int kPieces = kBlock * HDP / (kPer * kThreads);      // of a thread
    static constexpr int kBatch = kPieces > 8 ? 8 : kPieces;
    uint4 v[kBatch];
    __device__ __forceinline__ void load(const PagedRowsParams& p, const void* pool, const int64_t* row_s, int from) {
        const KT* src = static_cast<const KT*>(pool);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int e = threadIdx.x + (from + k) * kThreads, r = e / (HDP / kPer), d = e % (HDP / kPer) * kPer;
            const int64_t at = row_s[r];
            v[k] = make_uint4(0u, 0u, 0u, 0u);
            if (at >= 0 && d < p.hd) v[k] = __ldg(reinterpret_cast<const uint4*>(src + at + d));
        }
    }
    __device__ __forceinline__ void store(float* to, int from) const {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int e = threadIdx.x + (from + k) * kThreads, r = e / (HDP / kPer), d = e % (HDP / kPer) * kPer;
            float4* dst = reinterpret_cast<float4*>(to + r * Shape<HDP>::kStride + d);
            if constexpr (kPer == 4) {
                *dst = *reinterpret_cast<const float4*>(&v[k]);
            } else {
                const __half2* h = reinterpret_cast<const __half2*>(&v[k]);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 x = __half22float2(h[2 * i]), y = __half22float2(h[2 * i + 1]);
                    dst[i] = make_float4(x.x, x.y, y.x, y.y);
                }
            }
        }
    }
};

// The same for rows that 16-byte loads cannot read (hd or addresses).
template <typename KT, int HDP>
__device__ __forceinline__ void load_any(const PagedRowsParams& p, const void* pool, const int64_t* row_s, float* to) {
    const KT* src = static_cast<const KT*>(pool);
#pragma unroll 8
    for (int e = threadIdx.x; e < kBlock * HDP; e += kThreads) {
        const int r = e / HDP, d = e % HDP;
        const int64_t at = row_s[r];
        to[r * Shape<HDP>::kStride + d] = at >= 0 && d < p.hd ? get(src + at + d) : 0.f;
    }
}

template <typename KT, int HDP>
__global__ void __launch_bounds__(kThreads, Shape<HDP>::kCtas) paged_rows_any_kernel(const __grid_constant__ PagedRowsParams p) {
    using S = Shape<HDP>;
    extern __shared__ __align__(16) float smem[];
    float *q_s = smem, *kv_s = q_s + kRows * S::kStride, *p_s = kv_s + kBlock * S::kStride;
    __shared__ int64_t row_s[kBlock];
    __shared__ int lo_s[kRows], hi_s[kRows];
    griddep_wait();
    griddep_launch_dependents();
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, G = p.nh / p.nkv;
    const bool vec = ((reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                       static_cast<uintptr_t>(p.c.page_stride * sizeof(KT)) | static_cast<uintptr_t>(p.hd * sizeof(KT))) & 15u) == 0;
    const bool q_vec = ((reinterpret_cast<uintptr_t>(p.q) | static_cast<uintptr_t>(p.q_stride * 4) | static_cast<uintptr_t>(p.hd * 4)) & 15u) == 0;
    using B = Block<KT, HDP>;
    constexpr bool kAhead = B::kPieces <= 4;  // there are registers for it
    Walk<> w;
    if (!w.begin(p)) return;
    if (tid == 0) note_none(p);
    Piece piece;
    while (w.next(p, piece)) {
        const RowTile& t = piece.t;
        const int kv = piece.head / p.blocks, g0 = (piece.head - kv * p.blocks) * p.per_block, heads = min(p.per_block, G - g0);
        const int rows = t.ntok * p.per_block;
        __syncthreads();  // the last piece's rows have been read
        if (tid == 0) note_piece(p, w, piece);
        if (tid < kRows) {
            int lo = 0, hi = 0;
            if (tid < rows) row_span(p, t, tid / p.per_block, lo, hi);
            lo_s[tid] = lo;
            hi_s[tid] = hi;
        }
        const float scale = p.scale * kLog2e;
#pragma unroll 4
        for (int e = tid; e < kRows * HDP / 4; e += kThreads) {
            const int r = e / (HDP / 4), d = e % (HDP / 4) * 4, i = r / p.per_block, g = r - i * p.per_block;
            float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows && g < heads && d < p.hd) {
                const float* src = p.q + (t.row0 + i) * p.q_stride + static_cast<int64_t>(kv * G + g0 + g) * p.hd + d;
                if (q_vec) y = __ldcg(reinterpret_cast<const float4*>(src));
                else y = make_float4(__ldcg(src), d + 1 < p.hd ? __ldcg(src + 1) : 0.f, d + 2 < p.hd ? __ldcg(src + 2) : 0.f,
                                     d + 3 < p.hd ? __ldcg(src + 3) : 0.f);
            }
            *reinterpret_cast<float4*>(q_s + r * S::kStride + d) = make_float4(y.x * scale, y.y * scale, y.z * scale, y.w * scale);
        }
        float m[4], l[4];
        float4 o[4][S::kCols];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            m[i] = -CUDART_INF_F;
            l[i] = 0.f;
#pragma unroll
            for (int c = 0; c < S::kCols; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        for (int u = piece.from; u < piece.to; ++u) {
            const int j0 = t.lo + u * kBlock;
            if (tid < kBlock) {
                const int64_t row = j0 + tid < t.hi ? row_offset(p.c, t.seq, j0 + tid) : -1;
                row_s[tid] = row < 0 ? -1 : row + static_cast<int64_t>(kv) * p.hd;
            }
            __syncthreads();
            B x;
            if (vec) {
#pragma unroll
                for (int k = 0; k < B::kPieces; k += B::kBatch) {
                    x.load(p, p.c.k, row_s, k);
                    x.store(kv_s, k);
                }
                if (kAhead) x.load(p, p.c.v, row_s, 0);  // V is on its way while the scores are made
            } else {
                load_any<KT, HDP>(p, p.c.k, row_s, kv_s);
            }
            __syncthreads();
            float s[4][4] = {};
#pragma unroll 4
            for (int d = 0; d < HDP; d += 4) {
                float4 a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    a[i] = *reinterpret_cast<const float4*>(q_s + (ty + 16 * i) * S::kStride + d);
                    b[i] = *reinterpret_cast<const float4*>(kv_s + (tx + 16 * i) * S::kStride + d);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        s[i][j] = fmaf(a[i].x, b[j].x, fmaf(a[i].y, b[j].y, fmaf(a[i].z, b[j].z, fmaf(a[i].w, b[j].w, s[i][j]))));
            }
            // a weight below zero marks a slot that the row does not see
            const bool mixed = j0 < t.all_lo || j0 + kBlock > t.all_hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = ty + 16 * i, lo = lo_s[r], hi = hi_s[r];
                bool in[4];
                float mt = m[i];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int slot = j0 + tx + 16 * j;
                    in[j] = row_s[tx + 16 * j] >= 0 && slot >= lo && slot < hi;
                    if (!in[j]) s[i][j] = -CUDART_INF_F;
                    mt = fmaxf(mt, s[i][j]);
                }
#pragma unroll
                for (int k = 1; k < 16; k <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, k));
                const float keep = m[i] == mt ? 1.f : exp2f(m[i] - mt), base = mt == -CUDART_INF_F ? 0.f : mt;
                m[i] = mt;
                l[i] *= keep;
#pragma unroll
                for (int c = 0; c < S::kCols; ++c)
                    o[i][c] = make_float4(o[i][c].x * keep, o[i][c].y * keep, o[i][c].z * keep, o[i][c].w * keep);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float e = exp2f(s[i][j] - base);
                    l[i] += e;
                    p_s[r * kPStride + tx + 16 * j] = mixed && !in[j] ? -1.f : e;
                }
            }
            __syncthreads();
            if (vec) {
#pragma unroll
                for (int k = 0; k < B::kPieces; k += B::kBatch) {
                    if (!kAhead) x.load(p, p.c.v, row_s, k);
                    x.store(kv_s, k);
                }
            } else {
                load_any<KT, HDP>(p, p.c.v, row_s, kv_s);
            }
            __syncthreads();
#pragma unroll 2
            for (int j = 0; j < kBlock; j += 4) {
                float4 e[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) e[i] = *reinterpret_cast<const float4*>(p_s + (ty + 16 * i) * kPStride + j);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int c = 0; c < S::kCols; ++c) {
                        const float4 v = *reinterpret_cast<const float4*>(kv_s + (j + k) * S::kStride + 4 * tx + 64 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f = k == 0 ? e[i].x : k == 1 ? e[i].y : k == 2 ? e[i].z : e[i].w;
                            if (mixed && f < 0.f) continue;  // whatever V holds there
                            o[i][c] = make_float4(fmaf(f, v.x, o[i][c].x), fmaf(f, v.y, o[i][c].y), fmaf(f, v.z, o[i][c].z),
                                                  fmaf(f, v.w, o[i][c].w));
                        }
                    }
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 1; k < 16; k <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], k);
            const int r = ty + 16 * i;
            const int row = t.row0 + r / p.per_block, g = r % p.per_block, h = kv * G + g0 + g;
            if (r >= rows || g >= heads) continue;
            if (w.whole(piece)) {
                const bool empty = lo_s[r] >= hi_s[r];
                const float inv = empty ? 0.f : 1.f / l[i];
                const int64_t at = p.first ? row * p.out_stride + static_cast<int64_t>(h) * p.hd
                                           : (static_cast<int64_t>(row) * p.nh + h) * p.hd;
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) {
                    const float v[4] = {o[i][c].x, o[i][c].y, o[i][c].z, o[i][c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int d = 4 * tx + 64 * c + k;
                        if (d >= p.hd) continue;
                        const float y = empty ? 0.f : v[k] * inv;
                        if (p.first) put_out(p, at + d, y);
                        else p.prefix_out[at + d] = y;
                    }
                }
                float* lse = p.first ? p.lse : p.prefix_lse;
                if (tx == 0 && lse) lse[static_cast<int64_t>(row) * p.nh + h] = lse_of(m[i], l[i], empty);
            } else {
                float* part = part_of(p, blockIdx.x, piece.first);
                float* to = part_o(p, part, r);
                if (tx == 0) *part_ml(part, r) = make_float2(m[i], l[i]);
#pragma unroll
                for (int c = 0; c < S::kCols; ++c) {
                    const float v[4] = {o[i][c].x, o[i][c].y, o[i][c].z, o[i][c].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 * tx + 64 * c + k < p.hd) to[4 * tx + 64 * c + k] = v[k];
                }
            }
        }
    }
}

template <typename KT, int HDP>
cudaError_t launch_t(const PagedRowsParams& p, cudaStream_t stream) {
    auto kernel = paged_rows_any_kernel<KT, HDP>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<HDP>::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(kSms * Shape<HDP>::kCtas), kThreads, Shape<HDP>::kSmem, stream, 1, p);
}

template <typename KT>
cudaError_t launch_any(const PagedRowsParams& p, cudaStream_t stream) {
    return p.hd <= 64 ? launch_t<KT, 64>(p, stream) : p.hd <= 128 ? launch_t<KT, 128>(p, stream) : launch_t<KT, 256>(p, stream);
}

}  // namespace

RowsShape paged_rows_any_shape(const PagedRowsParams& p) {
    return {kRows, kRows, kBlock, kSms * (p.hd <= 128 ? Shape<128>::kCtas : Shape<256>::kCtas), 1, false};
}

// f16 rows that 16-byte copies can read, of whole steps of 16 columns that fit tensor memory beside the scores.  (4 x 509
// tokens of 28 heads over 4: 94 us, and 2050 by f32 multiply-adds; 17 tokens of 14 over 2, the smallest, 19.5 and 23.6.)
bool paged_rows_on_tensor_cores(const PagedRowsParams& p) {
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * 2);
    return p.kv_f16 && p.hd <= 128 && p.hd % 16 == 0 && (bits & 15u) == 0;
}

RowsShape paged_rows_shape(const PagedRowsParams& p) {
    if (!paged_rows_on_tensor_cores(p)) return paged_rows_any_shape(p);
    return paged_rows_tc_shape(!p.out_bf16);
}

cudaError_t launch_paged_rows(const PagedRowsParams& p, cudaStream_t stream) {
    if (paged_rows_on_tensor_cores(p)) return launch_paged_rows_tc(p, stream);
    return p.kv_f16 ? launch_any<__half>(p, stream) : launch_any<float>(p, stream);
}

cudaError_t paged_rows_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
