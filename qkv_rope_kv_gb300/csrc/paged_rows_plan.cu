// Attention of many q rows over a paged cache: the plan before it (which rows go together, over which slots) and the
// joining of parts behind it.  For 8191 new tokens of 40 heads of 128, 46 us of 580 go into q as f16 (252 MB, 0.80 of the copy
// rate) and 18 into the join of 36 MB of parts (each CTA of the attention but the first begins within a tile); for 17 tokens,
// six and four are their own latencies, the join's for nothing: no tile is split there.
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

// The largest value of the CTA's threads up to this one, and of all (in `all`); all threads call.
__device__ __forceinline__ int max_scan(int v, int& all, int* warp_s) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = max(v, up);
    }
    __syncthreads();  // the last call's values have been read
    if (lane == 31) warp_s[warp] = v;
    __syncthreads();
    all = warp_s[0];
    for (int w = 0; w < kPlanThreads / 32; ++w) {
        if (w < warp) v = max(v, warp_s[w]);
        all = max(all, warp_s[w]);
    }
    return v;
}

// For the tensor cores: q as f16, scaled by a power of two for each row into [2^13, 2^14) where the remainders are far from
// f16's subnormals, and the remainders; and by what scores are to be multiplied to be in log2 terms.  A warp a row, as
// many bytes as q has (or half as many again); rows that belong to no sequence too.
__device__ __forceinline__ void convert_q(const PagedRowsParams& p) {
    constexpr int kAhead = 4;  // rows of a warp in flight
    const int lane = threadIdx.x & 31;
    const int64_t rows = static_cast<int64_t>(p.nt) * p.nh;
    const int step = static_cast<int>(gridDim.x - 1) * (kPlanThreads / 32), step_tok = step / p.nh, step_head = step - step_tok * p.nh;
    const float by = fabsf(p.scale) * kLog2e;
    const bool quads = ((reinterpret_cast<uintptr_t>(p.q) | static_cast<uintptr_t>(p.q_stride * 4)) & 15u) == 0;
    const int begin = static_cast<int>(blockIdx.x - 1) * (kPlanThreads / 32) + (threadIdx.x >> 5);
    int tok = begin / p.nh, head = begin - tok * p.nh;  // (counted on: a division of 64 bits a row took as long as the copying)
    for (int64_t r0 = begin; r0 < rows; r0 += static_cast<int64_t>(kAhead) * step) {
        float v[kAhead][4];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t r = r0 + static_cast<int64_t>(j) * step;
            const float* q = p.q + tok * p.q_stride + head * p.hd + 4 * lane;
            tok += step_tok;
            head += step_head;
            if (head >= p.nh) {
                head -= p.nh;
                ++tok;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[j][k] = 0.f;
            if (r < rows && 4 * lane < p.hd) {
                if (quads) {
                    const float4 f = __ldcg(reinterpret_cast<const float4*>(q));
                    v[j][0] = f.x, v[j][1] = f.y, v[j][2] = f.z, v[j][3] = f.w;
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) v[j][k] = __ldcg(q + k);
                }
            }
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            const int64_t r = r0 + static_cast<int64_t>(j) * step;
            if (r >= rows) break;
            float big = fmaxf(fmaxf(fabsf(v[j][0]), fabsf(v[j][1])), fmaxf(fabsf(v[j][2]), fabsf(v[j][3])));
            big = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(big)));  // not below zero
            // exponent of the largest |q|, kept where both 2^(13 - e) and 2^(e - 13) are normal
            int e = static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 127;
            e = e == 128 ? 13 : max(-113, min(e, 126));
            // scores are compared before they are multiplied: by a number above zero, the sign goes into q
            float sc = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
            if (p.scale < 0.f) sc = -sc;
            if (by == 0.f) sc = 0.f;
            const float unscale =
                by == 0.f ? 1.f : fmaxf(by * __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23), 1.1754944e-38f);
            if (4 * lane < p.hd) {
                __half2 h[2], l[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float a = v[j][2 * k] * sc, b = v[j][2 * k + 1] * sc;
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
}

// Several new tokens of each sequence: tiles of neighbouring tokens.
__global__ void __launch_bounds__(kPlanThreads) plan_prompt_kernel(const __grid_constant__ PagedRowsParams p) {
    __shared__ int off_s[kPlanThreads + 1], first_s[kPlanThreads], n_s[kPlanThreads], len_s[kPlanThreads];
    __shared__ int64_t warp_s[kPlanThreads / 32];
    __shared__ int top_s[kPlanThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    if (blockIdx.x > 0) return convert_q(p);
    const int per_tile = p.tile_tokens;
    int64_t length = 0, tiles = 0;
    int top = 0;        // the largest of d_first before this round
    bool fell = false;  // whether it has decreased
    for (int b0 = 0; b0 < p.c.n_seq; b0 += kPlanThreads) {
        const int b = b0 + threadIdx.x;
        int count = 0, a = 0, e = 0;
        if (b < p.c.n_seq) {
            a = p.first[b];
            e = p.first[b + 1];
        }
        // Behind a decrease a pair may be in order and still begin below where another ended: two sequences with the same rows.
        // (Only looked for there: a prefix maximum of every call's d_first.)
        int over = a;
        if (__syncthreads_or(e < a && b < p.c.n_seq) || fell) {
            int all;
            over = max(max_scan(b < p.c.n_seq ? a : 0, all, top_s), top);
            top = max(top, all);
            fell = true;
        } else if (b0 + kPlanThreads < p.c.n_seq) {
            top = p.first[b0 + kPlanThreads - 1];
        }
        if (b < p.c.n_seq) {
            int n = e - a;
            if (a < 0 || e < a || e > p.nt || a < over) {
                flag_bad(kFlagIndexRange, a < 0 || a < over ? a : e);
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
            x.start = length + scan<int64_t>(x.units ? x.units + tile_cost(p, x) : 0, sum, warp_s);
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
        x.start = length + scan<int64_t>(x.units ? x.units + tile_cost(p, x) : 0, sum, warp_s);
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
// Q quads of columns of a lane: four from 4 * lane, and for heads above 128 from 128 + 4 * lane.  With one quad four CTAs fit on
// an SM, and a call's run all at once: 18 us for 36 MB, where one kernel for both kinds, of which two fitted, took 34.
static_assert(QKV_MAX_HEAD_DIM <= 256, "columns of a lane");
constexpr int kJoinCtas = 4;

// Columns [d, d + 4) of a row, as far as there are any.
__device__ __forceinline__ float4 get4(const float* row, int d, int hd) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (d + 4 <= hd && (reinterpret_cast<uintptr_t>(row + d) & 15u) == 0) return __ldcg(reinterpret_cast<const float4*>(row + d));
    if (d < hd) v.x = __ldcg(row + d);
    if (d + 1 < hd) v.y = __ldcg(row + d + 1);
    if (d + 2 < hd) v.z = __ldcg(row + d + 2);
    if (d + 3 < hd) v.w = __ldcg(row + d + 3);
    return v;
}
__device__ __forceinline__ void put4(const PagedRowsParams& p, int64_t at, int d, float4 v) {
    const float x[4] = {v.x, v.y, v.z, v.w};
    if (p.out_bf16) {
        uint16_t* o = static_cast<uint16_t*>(p.out) + at + d;
        uint32_t two[2];
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(two[0]) : "f"(v.y), "f"(v.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(two[1]) : "f"(v.w), "f"(v.z));
        if (d + 4 <= p.hd && (reinterpret_cast<uintptr_t>(o) & 7u) == 0) {
            *reinterpret_cast<uint2*>(o) = make_uint2(two[0], two[1]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (d + k < p.hd) o[k] = static_cast<uint16_t>(two[k >> 1] >> (16 * (k & 1)));
        }
    } else {
        float* o = static_cast<float*>(p.out) + at + d;
        if (d + 4 <= p.hd && (reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
            *reinterpret_cast<float4*>(o) = v;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (d + k < p.hd) o[k] = x[k];
        }
    }
}
__device__ __forceinline__ float4 fma4(float4 a, float k, float4 b) {
    return make_float4(fmaf(a.x, k, b.x), fmaf(a.y, k, b.y), fmaf(a.z, k, b.z), fmaf(a.w, k, b.w));
}

// The parts of a row, in the order of its slots, a few at a time, all of whose loads are in flight together.
template <int Q>
struct Joined {
    float m, l;
    float4 o[Q];
};
template <int Q>
__device__ __forceinline__ void join_row(const PagedRowsParams& p, int64_t start, int64_t share, int c0, int parts, int row,
                                         Joined<Q>& j) {
    constexpr int kAhead = 4;
    const int lane = threadIdx.x & 31;
    j.m = -CUDART_INF_F;
    j.l = 0.f;
#pragma unroll
    for (int k = 0; k < Q; ++k) j.o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool first = start == share * c0;  // the tile is the first of its first CTA
#pragma unroll 1
    for (int b = 0; b < parts; b += kAhead) {
        float2 ml[kAhead];
        float4 o[kAhead][Q];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (b + i >= parts) continue;
            float* part = part_of(p, c0 + b + i, b + i > 0 || first);
            ml[i] = __ldcg(part_ml(part, row));
#pragma unroll
            for (int k = 0; k < Q; ++k) o[i][k] = get4(part_o(p, part, row), 128 * k + 4 * lane, p.hd);
        }
        float top = j.m;
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (b + i < parts) top = fmaxf(top, ml[i].x);
        const float keep = j.m == top ? 1.f : exp2f(j.m - top);
        j.m = top;
        j.l *= keep;
#pragma unroll
        for (int k = 0; k < Q; ++k) j.o[k] = fma4(j.o[k], keep, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (b + i >= parts) continue;
            const float f = ml[i].x == top ? 1.f : exp2f(ml[i].x - top);
            j.l = fmaf(ml[i].y, f, j.l);
#pragma unroll
            for (int k = 0; k < Q; ++k) j.o[k] = fma4(o[i][k], f, j.o[k]);
        }
    }
}

// Prompt: CTA x takes rows of the tile that CTA x of the attention began and others went on with; a warp a row.
template <int Q>
__global__ void __launch_bounds__(kJoinThreads, Q == 1 ? kJoinCtas : 2) join_prompt_kernel(const __grid_constant__ PagedRowsParams p, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    const RowPiece* s = p.pieces + blockIdx.x;
    const int64_t total = __ldcg(p.total) * p.nkv * p.blocks, share = share_of(total, ctas);
    const int4 x = __ldcg(reinterpret_cast<const int4*>(s)), y = __ldcg(reinterpret_cast<const int4*>(s) + 1);
    if (share * blockIdx.x >= total || y.x == 0) return;  // (what was loaded is none)
    const int64_t start = static_cast<uint32_t>(x.x) | static_cast<int64_t>(x.y) << 32;
    const int parts = y.x, head = x.w, kv = head / p.blocks, G = p.nh / p.nkv;
    const int g0 = (head - kv * p.blocks) * p.per_block, heads = min(p.per_block, G - g0);
    const RowTile t = load_tile(p, x.z);
    for (int r = blockIdx.y * kJoinRows + (threadIdx.x >> 5); r < t.ntok * heads; r += gridDim.y * kJoinRows) {
        const int i = r / heads, g = r - i * heads, h = kv * G + g0 + g;
        Joined<Q> j;
        join_row(p, start, share, blockIdx.x, parts, row_of(p, i, g), j);
        int lo, hi;
        row_span(p, t, i, lo, hi);
        const bool empty = lo >= hi;
        const float inv = 1.f / j.l;
        const int64_t at = (t.row0 + i) * p.out_stride + static_cast<int64_t>(h) * p.hd;
        const int d = 4 * (threadIdx.x & 31);
#pragma unroll
        for (int k = 0; k < Q; ++k) {
            const float4 o = make_float4(j.o[k].x * inv, j.o[k].y * inv, j.o[k].z * inv, j.o[k].w * inv);
            put4(p, at, 128 * k + d, empty ? make_float4(0.f, 0.f, 0.f, 0.f) : o);
        }
        if (d == 0 && p.lse) p.lse[static_cast<int64_t>(t.row0 + i) * p.nh + h] = lse_of(j.m, j.l, empty);
    }
}

// Prefix: a warp for each sequence and q head joins the prefix's result, from parts or whole, and the own slots'.
template <int Q>
__global__ void __launch_bounds__(kJoinThreads, Q == 1 ? kJoinCtas : 2) join_prefix_kernel(const __grid_constant__ PagedRowsParams p, int ctas) {
    griddep_wait();
    griddep_launch_dependents();
    const int64_t x = static_cast<int64_t>(blockIdx.x) * kJoinRows + (threadIdx.x >> 5);
    const int b = static_cast<int>(x / p.nh), h = static_cast<int>(x - static_cast<int64_t>(b) * p.nh);
    if (b >= p.c.n_seq) return;
    const int d = 4 * (threadIdx.x & 31), G = p.nh / p.nkv, kv = h / G;
    const int64_t row = static_cast<int64_t>(b) * p.nh + h;
    // all that is needed whatever the case, in flight together
    const int seen = __ldcg(p.row_end + b), tile = __ldcg(p.row_tile + b);
    const int64_t per_head = __ldcg(p.total);
    const float own = __ldcg(p.own_lse + row);
    float4 mine[Q];
#pragma unroll
    for (int k = 0; k < Q; ++k) mine[k] = get4(p.own_out + row * p.hd, 128 * k + d, p.hd);
    const bool prefix = seen > 0;
    float theirs = -CUDART_INF_F;
    Joined<Q> j;
#pragma unroll
    for (int k = 0; k < Q; ++k) j.o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (prefix) {
        const RowTile t = load_tile(p, tile);
        const int64_t share = share_of(per_head * p.nkv * p.blocks, ctas);
        const int blk = (h - kv * G) / p.per_block;
        const int64_t start = (static_cast<int64_t>(kv) * p.blocks + blk) * per_head + t.start;
        const int c0 = static_cast<int>(start / share), c1 = static_cast<int>((start + t.units - 1) / share);
        if (c0 < c1) {
            join_row(p, start, share, c0, c1 - c0 + 1, row_of(p, b - t.row0, h - kv * G - blk * p.per_block), j);
            const float inv = 1.f / j.l;
#pragma unroll
            for (int k = 0; k < Q; ++k) j.o[k] = fma4(j.o[k], inv, make_float4(0.f, 0.f, 0.f, 0.f));
            theirs = lse_of(j.m, j.l, false);
        } else {
            theirs = __ldcg(p.prefix_lse + row);
#pragma unroll
            for (int k = 0; k < Q; ++k) j.o[k] = get4(p.prefix_out + row * p.hd, 128 * k + d, p.hd);
        }
    }
    // One that is empty (-inf) leaves the other as it is.  A NaN, or +inf (whose own row is NaN already), stays.
    const bool none = own == -CUDART_INF_F, alone = !prefix;
    const float top = fmaxf(own, theirs);
    const float a = alone ? 0.f : expf(theirs - top), z = alone ? 1.f : none && theirs > -CUDART_INF_F ? 0.f : expf(own - top);
    const float inv = 1.f / (a + z);
    const int64_t at = b * p.out_stride + static_cast<int64_t>(h) * p.hd;
#pragma unroll
    for (int k = 0; k < Q; ++k) {
        const float4 s = fma4(mine[k], z, fma4(j.o[k], a, make_float4(0.f, 0.f, 0.f, 0.f)));
        put4(p, at, 128 * k + d, alone || a == 0.f ? mine[k] : z == 0.f ? j.o[k] : fma4(s, inv, make_float4(0.f, 0.f, 0.f, 0.f)));
    }
    if (d == 0 && p.lse) p.lse[row] = alone || top == -CUDART_INF_F ? own : z == 0.f ? theirs : a == 0.f ? own : top + logf(a + z);
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
    const bool wide = p.hd > 128;
    if (p.first) {
        // four CTAs a tile: a row or two a warp where tiles are small
        return launch_dependent(wide ? join_prompt_kernel<2> : join_prompt_kernel<1>, dim3(ctas, 4), kJoinThreads, 0, stream, 1, p, ctas);
    }
    const int64_t rows = static_cast<int64_t>(p.c.n_seq) * p.nh;
    return launch_dependent(wide ? join_prefix_kernel<2> : join_prefix_kernel<1>,
                            dim3(static_cast<unsigned int>((rows + kJoinRows - 1) / kJoinRows)), kJoinThreads, 0, stream, 1, p, ctas);
}

cudaError_t paged_rows_plan_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
