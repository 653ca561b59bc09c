// Attention of many q rows over a paged cache: the plan before it (which rows go together, over which slots) and the
// joining of parts behind it.  Both are small next to the attention between them.
#include "paged_rows.cuh"

namespace {

using namespace qkv_rows;
using qkv_ptx::griddep_launch_dependents;
using qkv_ptx::griddep_wait;

constexpr int kPlanThreads = 512;

// Exclusive prefix sum over the CTA's threads, and the sum; all threads call.
template <typename T>
__device__ __forceinline__ T scan(T v, T& sum, T* warp_s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();  // the last call's sums have been read
    if (lane == 31) warp_s[warp] = incl;
    __syncthreads();
    T before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) before += warp_s[w];
        sum += warp_s[w];
    }
    return before + incl - v;
}

// For the tensor cores: q as f16, scaled by a power of two for each row into [2^13, 2^14) where the remainders are far from
// f16's subnormals, and the remainders; and by what scores are to be multiplied to be in log2 terms.  A warp a row, as
// many bytes as q has (or half as many again); rows that belong to no sequence too.
__device__ __forceinline__ void convert_q(const PagedRowsParams& p) {
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(p.nt) * p.nh, step = static_cast<int64_t>(gridDim.x - 1) * (kPlanThreads / 32);
    const float by = fabsf(p.scale) * kLog2e;
    for (int64_t r = static_cast<int64_t>(blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5); r < rows; r += step) {
        const int64_t tok = r / p.nh;
        const float* q = p.q + tok * p.q_stride + (r - tok * p.nh) * p.hd + 4 * lane;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (4 * lane < p.hd) {
            if ((reinterpret_cast<uintptr_t>(q) & 15u) == 0) {
                const float4 f = __ldcg(reinterpret_cast<const float4*>(q));
                v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
            } else {
#pragma unroll
                for (int k = 0; k < 4; ++k) v[k] = __ldcg(q + k);
            }
        }
        float big = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
        big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));  // not below zero
        // exponent of the largest |q|, kept where both 2^(13 - e) and 2^(e - 13) are normal
        int e = static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 127;
        e = e == 128 ? 13 : max(-113, min(e, 126));
        // scores are compared before they are multiplied: by a number above zero, the sign goes into q
        float sc = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
        if (p.scale < 0.f) sc = -sc;
        const float unscale = by == 0.f ? 1.f : fmaxf(by * __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23), 1.1754944e-38f);
        if (by == 0.f) sc = 0.f;
        if (4 * lane < p.hd) {
            __half2 h[2], l[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float a = v[2 * k] * sc, b = v[2 * k + 1] * sc;
                h[k] = __floats2half2_rn(a, b);
                const float2 f = __half22float2(h[k]);
                l[k] = __floats2half2_rn(a - f.x, b - f.y);
            }
            const int64_t at = r * p.hd + 4 * lane;
            *reinterpret_cast<uint2*>(p.q_high + at) = *reinterpret_cast<uint2*>(h);
            if (!p.out_bf16) *reinterpret_cast<uint2*>(p.q_low + at) = *reinterpret_cast<uint2*>(l);
        }
        if (lane == 0) p.q_unscale[r] = unscale;
    }
}

// Several new tokens of each sequence: tiles of neighbouring tokens.
__global__ void __launch_bounds__(kPlanThreads) plan_prompt_kernel(const __grid_constant__ PagedRowsParams p) {
    __shared__ int off_s[kPlanThreads + 1], first_s[kPlanThreads], n_s[kPlanThreads], len_s[kPlanThreads];
    __shared__ int64_t warp_s[kPlanThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x > 0) return convert_q(p);
    const int per_tile = p.tile_tokens;
    int64_t length = 0, tiles = 0;
    for (int b0 = 0; b0 < p.c.n_seq; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int count = 0;
        if (b < p.c.n_seq) {
            const int a = p.first[b], e = p.first[b + 1];
            int n = e - a;
            if (a < 0 || e < a || e > p.nt) {
                flag_bad(kFlagIndexRange, a < 0 ? a : e);
                n = 0;
            }
            first_s[threadIdx.x] = a;
            n_s[threadIdx.x] = n;
            len_s[threadIdx.x] = checked_len(p.c, p.lens, b);
            count = (n + per_tile - 1) / per_tile;
        }
        int64_t here;
        off_s[threadIdx.x] = static_cast<int>(scan<int64_t>(count, here, warp_s));
        if (threadIdx.x == 0) off_s[kPlanThreads] = static_cast<int>(here);
        __syncthreads();
        // d_first that goes up and down could name more tiles than rows: no more than there is room for
        if (here > p.max_tiles - tiles) {
            if (threadIdx.x == 0) flag_bad(kFlagIndexRange, p.first[b0]);
            here = p.max_tiles - tiles;
        }
        for (int64_t t0 = 0; t0 < here; t0 += kPlanThreads) {
            const int t = static_cast<int>(t0) + threadIdx.x;
            RowTile x = {};
            if (t < here) {
                int lo = 0, hi = kPlanThreads;  // the last sequence that begins at or before t and has tiles
                while (hi - lo > 1) {
                    const int mid = (lo + hi) / 2;
                    if (off_s[mid] <= t) lo = mid;
                    else hi = mid;
                }
                const int tok = (t - off_s[lo]) * per_tile;
                x.seq = b0 + lo;
                x.row0 = first_s[lo] + tok;
                x.ntok = min(per_tile, n_s[lo] - tok);
                x.base = len_s[lo] - n_s[lo] + tok + 1;
                x.hi = max(0, x.base + x.ntok - 1);
                const int see = p.window > 0 ? max(0, x.base - p.window) : 0;
                x.all_lo = p.window > 0 ? max(0, x.base + x.ntok - 1 - p.window) : 0;
                x.all_hi = max(0, x.base);
                x.lo = see < x.hi ? see / p.block * p.block : 0;
                x.units = max(1, (x.hi - x.lo + p.block - 1) / p.block);  // rows that see nothing are written too
            }
            int64_t sum;
            x.start = length + scan<int64_t>(x.units ? x.units + p.tile_cost : 0, sum, warp_s);
            if (t < here) p.tiles[tiles + t] = x;
            length += sum;
        }
        tiles += here;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.total[0] = length;
        p.total[1] = tiles;
    }
}

// One new token of each sequence, the beginnings shared: tiles of neighbouring sequences with the same d_share.
__global__ void __launch_bounds__(kPlanThreads) plan_prefix_kernel(const __grid_constant__ PagedRowsParams p) {
    __shared__ int hi_s[kPlanThreads], all_s[kPlanThreads], n_s[kPlanThreads], start_s[kPlanThreads], run_s[kPlanThreads];
    __shared__ int64_t warp_s[kPlanThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x > 0) return convert_q(p);
    const int per_tile = p.tile_tokens;
    int64_t length = 0, tiles = 0;
    // a tile ends where a round does
    for (int b0 = 0; b0 < p.c.n_seq; b0 += kPlanThreads) {
        const int i = threadIdx.x, b = b0 + i;
        int share = -1, begin = 0, seen = 0;
        bool edge = false;
        if (b < p.c.n_seq) {
            share = p.share[b];
            edge = i == 0 || p.share[b - 1] != share;
            begin = p.prefix_len[b];
            if (begin < 0 || begin > p.c.max_pages * p.c.page_size) {
                flag_bad(kFlagIndexRange, begin);
                begin = 0;
            }
            begin = seen = min(begin, checked_len(p.c, p.lens, b));
            if (share < 0 || share >= p.c.n_seq) {
                flag_bad(kFlagIndexRange, share);
                seen = 0;
            }
        }
        // where this one's run of equal d_share began
        int run = edge ? i : 0;
        const int lane = i & 31;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run = max(run, up);
        }
        __syncthreads();
        if (lane == 31) run_s[i >> 5] = run;
        hi_s[i] = 0;
        all_s[i] = 0x7fffffff;
        n_s[i] = 0;
        __syncthreads();
        for (int w = 0; w < i >> 5; ++w) run = max(run, run_s[w]);
        const bool head = b < p.c.n_seq && (i - run) % per_tile == 0;
        int64_t here;
        const int mine = static_cast<int>(scan<int64_t>(head, here, warp_s)) + head - 1;
        if (head) start_s[mine] = i;
        __syncthreads();
        if (b < p.c.n_seq) {
            atomicMax(&hi_s[mine], seen);
            atomicMin(&all_s[mine], seen);
            atomicAdd(&n_s[mine], 1);
        }
        __syncthreads();
        if (b < p.c.n_seq) {
            // a sequence alone in its tile that shares with nobody else's pages is read with its own slots
            const bool alone = n_s[mine] == 1 && share == b;
            p.starts[b] = alone ? 0 : begin;
            p.row_end[b] = alone ? 0 : seen;
            p.row_tile[b] = static_cast<int>(tiles) + mine;
        }
        RowTile x = {};
        if (i < here) {
            x.row0 = b0 + start_s[i];
            x.seq = p.share[x.row0];
            x.ntok = n_s[i];
            x.hi = x.ntok == 1 && x.seq == x.row0 ? 0 : hi_s[i];
            x.all_hi = all_s[i];
            x.units = (x.hi + p.block - 1) / p.block;
        }
        int64_t sum;
        x.start = length + scan<int64_t>(x.units ? x.units + p.tile_cost : 0, sum, warp_s);
        if (i < here) p.tiles[tiles + i] = x;
        length += sum;
        tiles += here;
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        p.total[0] = length;
        p.total[1] = tiles;
    }
}

constexpr int kJoinThreads = 256, kJoinRows = kJoinThreads / 32;
constexpr int kMaxCols = QKV_MAX_HEAD_DIM / 32;

// The parts of a row, in the order of its slots: the lane's columns lane, lane + 32, ...
struct Joined {
    float m, l, o[kMaxCols];
};
__device__ __forceinline__ void join_row(const PagedRowsParams& p, int64_t start, int64_t share, int c0, int parts, int row,
                                         Joined& j) {
    const int lane = threadIdx.x & 31;
    j.m = -CUDART_INF_F;
    j.l = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCols; ++k) j.o[k] = 0.f;
    const bool first = start == share * c0;  // the tile is the first of its first CTA
    for (int c = lane; c < parts; c += 32) j.m = fmaxf(j.m, __ldcg(part_ml(part_of(p, c0 + c, c > 0 || first), row)).x);
    for (int o = 16; o; o >>= 1) j.m = fmaxf(j.m, __shfl_xor_sync(0xffffffffu, j.m, o));
#pragma unroll 4
    for (int c = 0; c < parts; ++c) {
        float* part = part_of(p, c0 + c, c > 0 || first);
        const float2 ml = __ldcg(part_ml(part, row));
        const float k = ml.x == j.m ? 1.f : exp2f(ml.x - j.m);
        const float* o = part_o(p, part, row);
        j.l = fmaf(ml.y, k, j.l);
#pragma unroll
        for (int i = 0; i < kMaxCols; ++i)
            if (lane + 32 * i < p.hd) j.o[i] = fmaf(__ldcg(o + lane + 32 * i), k, j.o[i]);
    }
}

// Prompt: CTA x takes rows of the tile that CTA x of the attention began and others went on with; a warp a row.
__global__ void __launch_bounds__(kJoinThreads) join_prompt_kernel(const __grid_constant__ PagedRowsParams p, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t total = __ldcg(p.total) * p.nkv * p.blocks, share = share_of(total, ctas);
    if (share * blockIdx.x >= total) return;
    const RowPiece* s = p.pieces + blockIdx.x;
    const int parts = __ldcg(&s->parts);
    if (parts == 0) return;
    const int64_t start = __ldcg(&s->start);
    const int head = __ldcg(&s->head), kv = head / p.blocks, G = p.nh / p.nkv;
    const int g0 = (head - kv * p.blocks) * p.per_block, heads = min(p.per_block, G - g0);
    const RowTile t = load_tile(p, __ldcg(&s->tile));
    for (int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5); r < t.ntok * heads; r += gridDim.y * kJoinRows) {
        const int i = r / heads, g = r - i * heads, h = kv * G + g0 + g;
        Joined j;
        join_row(p, start, share, blockIdx.x, parts, row_of(p, i, g), j);
        int lo, hi;
        row_span(p, t, i, lo, hi);
        const bool empty = lo >= hi;
        const float inv = empty ? 0.f : 1.f / j.l;
        const int64_t at = (t.row0 + i) * p.out_stride + static_cast<int64_t>(h) * p.hd;
#pragma unroll
        for (int k = 0; k < kMaxCols; ++k) {
            const int d = (threadIdx.x & 31) + 32 * k;
            if (d < p.hd) put_out(p, at + d, empty ? 0.f : j.o[k] * inv);
        }
        if ((threadIdx.x & 31) == 0 && p.lse) p.lse[static_cast<int64_t>(t.row0 + i) * p.nh + h] = lse_of(j.m, j.l, empty);
    }
}

// Prefix: a warp for each sequence and q head joins the prefix's result, from parts or whole, and the own slots'.
__global__ void __launch_bounds__(kJoinThreads) join_prefix_kernel(const __grid_constant__ PagedRowsParams p, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t x = static_cast<int64_t>(blockIdx.x) * kJoinRows + (threadIdx.x >> 5);
    const int b = static_cast<int>(x / p.nh), h = static_cast<int>(x - static_cast<int64_t>(b) * p.nh);
    if (b >= p.c.n_seq) return;
    const int lane = threadIdx.x & 31, G = p.nh / p.nkv, kv = h / G;
    const bool prefix = __ldcg(p.row_end + b) > 0;
    const int64_t row = static_cast<int64_t>(b) * p.nh + h;
    const float own = __ldcg(p.own_lse + row);
    float theirs = -CUDART_INF_F;
    Joined j;
#pragma unroll
    for (int k = 0; k < kMaxCols; ++k) j.o[k] = 0.f;
    if (prefix) {
        const RowTile t = load_tile(p, __ldcg(p.row_tile + b));
        const int64_t per_head = __ldcg(p.total), share = share_of(per_head * p.nkv * p.blocks, ctas);
        const int blk = (h - kv * G) / p.per_block;
        const int64_t start = (static_cast<int64_t>(kv) * p.blocks + blk) * per_head + t.start;
        const int c0 = static_cast<int>(start / share), c1 = static_cast<int>((start + t.units - 1) / share);
        if (c0 < c1) {
            join_row(p, start, share, c0, c1 - c0 + 1, row_of(p, b - t.row0, h - kv * G - blk * p.per_block), j);
            const float inv = 1.f / j.l;
#pragma unroll
            for (int k = 0; k < kMaxCols; ++k) j.o[k] *= inv;
            theirs = lse_of(j.m, j.l, false);
        } else {
            theirs = __ldcg(p.prefix_lse + row);
#pragma unroll
            for (int k = 0; k < kMaxCols; ++k)
                if (lane + 32 * k < p.hd) j.o[k] = __ldcg(p.prefix_out + row * p.hd + lane + 32 * k);
        }
    }
    // One that is empty (-inf) leaves the other as it is.  A NaN, or +inf (whose own row is NaN already), stays.
    const bool none = own == -CUDART_INF_F, alone = !prefix;
    const float top = fmaxf(own, theirs);
    float a = alone ? 0.f : expf(theirs - top), z = none && !alone && theirs > -CUDART_INF_F ? 0.f : expf(own - top);
    if (alone) z = 1.f;
    const float inv = 1.f / (a + z);
    const int64_t at = b * p.out_stride + static_cast<int64_t>(h) * p.hd;
#pragma unroll
    for (int k = 0; k < kMaxCols; ++k) {
        const int d = lane + 32 * k;
        if (d >= p.hd) break;
        const float mine = __ldcg(p.own_out + row * p.hd + d);
        const float v = alone ? mine : z == 0.f ? j.o[k] : a == 0.f ? mine : (j.o[k] * a + mine * z) * inv;
        put_out(p, at + d, v);
    }
    if (lane == 0 && p.lse) p.lse[row] = alone || top == -CUDART_INF_F ? own : z == 0.f ? theirs : a == 0.f ? own : top + logf(a + z);
}

}  // namespace

cudaError_t launch_paged_rows_plan(const PagedRowsParams& p, cudaStream_t stream) {
    int converting = 0;
    if (paged_rows_shape(p).tensor) {  // a CTA for every 4 rows a warp, up to four on an SM
        const int64_t each = 4 * (kPlanThreads / 32), want = (static_cast<int64_t>(p.nt) * p.nh + each - 1) / each;
        converting = static_cast<int>(want < 4 * kSms ? want : 4 * kSms);
    }
    return launch_dependent(p.first ? plan_prompt_kernel : plan_prefix_kernel, dim3(1 + converting), kPlanThreads, 0, stream, 1, p);
}

cudaError_t launch_paged_rows_join(const PagedRowsParams& p, cudaStream_t stream) {
    const int ctas = paged_rows_shape(p).ctas;
    if (p.first) {
        const int each = (p.rows + 4 * kJoinRows - 1) / (4 * kJoinRows);  // four rows a warp
        return launch_dependent(join_prompt_kernel, dim3(ctas, each), kJoinThreads, 0, stream, 1, p, ctas);
    }
    const int64_t rows = static_cast<int64_t>(p.c.n_seq) * p.nh;
    return launch_dependent(join_prefix_kernel, dim3(static_cast<unsigned int>((rows + kJoinRows - 1) / kJoinRows)),
                            kJoinThreads, 0, stream, 1, p, ctas);
}

cudaError_t paged_rows_plan_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
