// qkv_attn_step: attention of one new token per sequence over a paged cache
// (include/qkv.h has the contract).
//
// s_j = scale * q.K_j, online softmax (running maximum m and sum l), out = sum p_j V_j / l.
// Scores are kept in the log2 domain (scale * log2(e) folded into q), so p = 2^(s - m).
#include <math_constants.h>

#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace {

using namespace qkv_paged;
using qkv_ptx::griddep_wait;

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
    griddep_wait();
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

// ---------------------------------------------------------------- split over the length, tensor cores

// Work is counted in units of 16 (f16) or 8 (f32) neighbouring slots of one item, an item being
// (sequence, kv head, block of up to 8 of its q heads).  The units of all items, in order, are dealt
// to the CTAs in equal contiguous shares, whatever the lengths are; where a share ends inside an
// item, its part goes to the workspace and the last CTA to arrive joins the item's parts in order.
//
// Within a CTA unit f belongs to warp f % 4, and each warp is a stream of its own: it copies its
// units into its own ring of stages (cp.async, rows addressed through the page table, rows outside
// the sequence filled with zeros) and computes them, with no barrier but at the end of an item.
//
// The 8 q heads of an item take half of the 16 rows of an MMA.  The other half carries what the
// first loses: rows 0-7 hold q rounded to f16 (tf32), rows 8-15 the rounded remainder, and the same
// with the softmax weights, so both products keep about 22 bits at no extra MMA.  An f32 cache's own
// rows are split too (two MMAs).  Before the split q is scaled by a power of two into [2^13, 2^14),
// and the weights are 2^(s - m + 12) with m at most 3 below the running maximum (then O need not be
// rescaled for every new maximum), both far from f16's ends.

constexpr int kWarps = 4, kSplitThreads = 32 * kWarps;
constexpr float kPShift = 12.f;  // weights are kept times 2^12
constexpr int kMinShare = 8;     // units
constexpr float kLazy = 3.f;     // and may exceed that by 2^3 before the maximum moves

template <typename KT, int HD>
struct Split {
    static constexpr bool kF16 = sizeof(KT) == 2;
    static constexpr int UK = kF16 ? 16 : 8;                  // slots of a unit
    static constexpr int kRowBytes = HD * sizeof(KT);
    static constexpr int kTileBytes = UK * kRowBytes;         // K or V of a unit
    static constexpr int kStages = HD < 256 ? 24576 / (2 * kTileBytes) : kF16 ? 3 : 2;
    static constexpr int kRingBytes = kStages * 2 * kTileBytes;
    static constexpr int kORow = HD + 4;                      // floats; + 4 spreads the heads over the banks
    static constexpr int kWarpsFloats = kWarps * kAttnHeads * (kORow + 2);  // the warps' O, m and l
    static constexpr int kMergeFloats = kWarpsFloats > kAttnHeads * kAttnMaxCtas ? kWarpsFloats : kAttnHeads * kAttnMaxCtas;
    static constexpr int kNT = HD / 8;                        // output column tiles
    static constexpr int kQRegs = kF16 ? HD / 4 : HD / 2;     // A fragments of q
    static constexpr bool kQSmem = kQRegs > 64;               // too many beside O: kept in shared memory
    static constexpr int kSmem = kWarps * kRingBytes + kMergeFloats * 4 + (kQSmem ? kQRegs * 128 : 0) + kWarps * kStages * 4;
    static constexpr int kCtas = HD == 256 ? 1 : 2;           // per SM
    static_assert(kStages >= 2, "ring");
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldm4t(uint32_t a, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void lds4(uint32_t a, float (&r)[4]) {
    asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ unsigned int atom_add_acq_rel(unsigned int* p, unsigned int v) {
    unsigned int old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// Two values rounded to f16 in hi, and the remainders rounded to f16 in lo.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// The leading 11 bits of a value (a tf32 number) and the next 11.
__device__ __forceinline__ void split_tf32(float a, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(a) & 0xffffe000u;
    lo = __float_as_uint(a - __uint_as_float(hi)) & 0xffffe000u;
}
// The same for cache values: an infinite one has no remainder (inf - inf is NaN, which max drops).
__device__ __forceinline__ void split_tf32_kv(float a, uint32_t& hi, uint32_t& lo) {
    hi = __float_as_uint(a) & 0xffffe000u;
    lo = __float_as_uint(fmaxf(a - __uint_as_float(hi), -1e30f)) & 0xffffe000u;
}
// The sum of a product's two halves; an infinite or NaN first half stands alone (the second is
// then a product of the same infinity with a remainder of any sign).
__device__ __forceinline__ float join_halves(float hi, float lo) { return fabsf(hi) < CUDART_INF_F ? hi + lo : hi; }

// Byte offset of 16-byte chunk c of row r within a tile.  f16: eight rows of one chunk (ldmatrix)
// fall into eight different bank groups.  f32: K is read as 4 chunks of 2 neighbouring rows, V as 2
// chunks of the 4 even (odd) rows.
template <bool F16, bool V>
__device__ __forceinline__ int swz(int r, int c, int row_bytes) {
    const int x = F16 ? (r & 7) : V ? (r & 6) : ((r & 1) << 2);
    return r * row_bytes + ((c ^ x) << 4);
}

// A place in the order of units.
struct Walk {
    int b;         // sequence
    int lo, n;     // its first unit and its length
    int first;     // its first slot
    int units;     // units of one of its items
    int item, u;   // item, and unit within it
};

template <int UK>
__device__ __forceinline__ void seq_units(const PagedAttnParams& p, int b, bool flag, Walk& w) {
    int n = __ldg(p.lens + b);
    if (n < 0 || n > p.c.max_pages * p.c.page_size) {
        if (flag) flag_bad(kFlagIndexRange, n);
        n = 0;
    }
    w.b = b;
    w.n = n;
    w.first = p.window > 0 ? max(0, n - p.window) : 0;
    w.lo = w.first / UK;
    w.units = n > 0 ? (n + UK - 1) / UK - w.lo : 0;
}

template <typename KT, int HD>
__global__ void __launch_bounds__(kSplitThreads, Split<KT, HD>::kCtas)
    paged_attn_split_kernel(const __grid_constant__ PagedAttnParams p, int blocks_per_head, int min_share) {
    using S = Split<KT, HD>;
    constexpr int UK = S::UK;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int64_t red_s[kWarps];
    __shared__ int longest_s[kWarps];
    __shared__ int64_t start_s;
    __shared__ int b_s;
    __shared__ unsigned int last_s;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int B = p.c.n_seq, G = p.nh / p.nkv, items = p.nkv * blocks_per_head;
    unsigned char* ring = smem + warp * S::kRingBytes;
    float* merge = reinterpret_cast<float*>(smem + kWarps * S::kRingBytes);
    float* merge_m = merge + kWarps * kAttnHeads * S::kORow;
    float* merge_l = merge_m + kWarps * kAttnHeads;
    uint32_t* q_s = reinterpret_cast<uint32_t*>(merge + S::kMergeFloats);
    uint32_t* live_s = q_s + (S::kQSmem ? S::kQRegs * 32 : 0) + warp * S::kStages;

    griddep_wait();
    // Total number of units and the longest item; and the sequence in which this CTA's share begins.
    Walk mine;  // sequence tid of the first 128
    int64_t total = 0;
    int longest = 0;
    for (int b0 = 0; b0 < B; b0 += kSplitThreads) {
        Walk w;
        w.units = 0;
        if (b0 + tid < B) seq_units<UK>(p, b0 + tid, blockIdx.x == 0, w);
        if (b0 == 0) mine = w;
        total += w.units;
        longest = max(longest, w.units);
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (lane == 0) {
        red_s[warp] = total;
        longest_s[warp] = longest;
    }
    __syncthreads();
    for (int b = blockIdx.x; b < B; b += gridDim.x) {  // an empty sequence has no unit: its rows are written here
        Walk w;
        seq_units<UK>(p, b, false, w);
        if (w.units == 0) {
            for (int i = tid; i < p.nh * p.hd; i += kSplitThreads) put_out(p, b, 0, i, 0.f);
            for (int h = tid; h < p.nh; h += kSplitThreads) put_lse(p, b, h, 0.f, 0.f, true);
        }
    }
    total = (red_s[0] + red_s[1] + red_s[2] + red_s[3]) * items;
    // A share is at least kMinShare units (each part of an item costs a join), but short items are
    // not gathered in one CTA while others have none.
    longest = min(max(max(longest_s[0], longest_s[1]), max(longest_s[2], longest_s[3])), min_share);
    int64_t share = (total + gridDim.x - 1) / gridDim.x;
    share = share < longest ? longest : share;
    const int64_t f0 = share * blockIdx.x, f1 = f0 + share < total ? f0 + share : total;
    if (f0 >= f1) return;
    int64_t before = 0;  // units of the sequences before this round's
    for (int b0 = 0; b0 < B; b0 += kSplitThreads) {
        if (b0 > 0) {
            mine.units = 0;
            if (b0 + tid < B) seq_units<UK>(p, b0 + tid, false, mine);
        }
        const int64_t units = static_cast<int64_t>(mine.units) * items;
        int64_t incl = units;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        __syncthreads();
        if (lane == 31) red_s[warp] = incl;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i)
            if (i < warp) incl += red_s[i];
        incl += before;
        if (units > 0 && incl - units <= f0 && f0 < incl) {
            b_s = b0 + tid;
            start_s = incl - units;
        }
        before += red_s[0] + red_s[1] + red_s[2] + red_s[3];
        if (f0 < before) break;  // uniform: every thread has the same sums
    }
    // columns beyond hd are zeros for good: no copy writes there
    if (p.hd < HD)
        for (int i = lane * 16; i < S::kRingBytes; i += 512) *reinterpret_cast<uint4*>(ring + i) = make_uint4(0, 0, 0, 0);
    __syncthreads();

    Walk at;     // the segment being computed
    seq_units<UK>(p, b_s, false, at);
    at.item = static_cast<int>((f0 - start_s) / at.units);
    at.u = static_cast<int>((f0 - start_s) % at.units);
    auto next_item = [&](Walk& w) {
        if (++w.item < items) return;
        w.item = 0;
        do seq_units<UK>(p, w.b + 1, false, w);  // called only where more units follow
        while (w.units == 0);
    };
    Walk ahead = at;            // the unit to be copied next, fa in the flat order
    int64_t fa = f0 + warp;
    int skip = warp;            // how far ahead is behind fa
    const int hd_chunks = p.hd * static_cast<int>(sizeof(KT)) / 16;
    constexpr int kChunks = S::kRowBytes / 16;

    // Row offset (lane = slot of the unit; -1: not read) of unit fa, and the column of its kv head.
    int64_t row = -1;
    int head_col = 0;
    auto locate = [&]() {
        row = -1;
        if (fa >= f1) return;
        for (ahead.u += skip; ahead.u >= ahead.units;) {
            ahead.u -= ahead.units;
            next_item(ahead);
        }
        skip = kWarps;
        head_col = ahead.item / blocks_per_head * p.hd;
        const int slot = (ahead.lo + ahead.u) * UK + lane;
        if (lane < UK && slot >= ahead.first && slot < ahead.n) row = row_offset(p.c, ahead.b, slot);
    };
    int put = 0;  // stage that the next unit goes to
    auto copy = [&]() {
        if (fa < f1) {
            const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) live_s[put] = live;
            const uint32_t dst = smem_addr(ring + put * 2 * S::kTileBytes);
            const int64_t off = row >= 0 ? row + head_col : 0;
#pragma unroll
            for (int i = 0; i < UK * kChunks / 32; ++i) {
                const int ci = i * 32 + lane, r = ci / kChunks, c = ci % kChunks;
                const int64_t o = __shfl_sync(0xffffffffu, off, r);
                const uint32_t bytes = (live >> r) & 1u ? 16u : 0u;
                if (c < hd_chunks) {
                    cp_async16(dst + swz<S::kF16, false>(r, c, S::kRowBytes),
                               static_cast<const char*>(p.c.k) + (o * sizeof(KT) + c * 16), bytes);
                    cp_async16(dst + S::kTileBytes + swz<S::kF16, true>(r, c, S::kRowBytes),
                               static_cast<const char*>(p.c.v) + (o * sizeof(KT) + c * 16), bytes);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        put = put + 1 == S::kStages ? 0 : put + 1;
        fa += kWarps;
    };
    for (int i = 0; i < S::kStages - 1; ++i) {
        locate();
        copy();
    }
    locate();

    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    int get = 0;                 // stage of the next unit to compute
    int64_t f = f0 + warp;       // that unit
    for (int64_t fs = f0; fs < f1;) {
        // the segment: the CTA's units of one item
        const int64_t item_start = fs - at.u, item_end = item_start + at.units;
        const int64_t fe = item_end < f1 ? item_end : f1;
        const int item = at.item;
        const int hk = item / blocks_per_head, hb = item - hk * blocks_per_head;
        const int h0 = hk * G + hb * kAttnHeads, nheads = min(kAttnHeads, G - hb * kAttnHeads);

        // q of head g as A fragments
        uint32_t qa[S::kQRegs];
        float unscale = 1.f;
        {
            const float* q = p.q + at.b * p.q_stride + static_cast<int64_t>(h0 + g) * p.hd;
            float x[HD / 4];
            float big = 0.f;
            const float qs = p.scale * kLog2e;
#pragma unroll
            for (int i = 0; i < HD / 4; ++i) {
                // f16: 16 (i / 4) + 2t + (0, 1, 8, 9); f32: 4 (i / 4) of 16 a round: 16 (i / 4) + 4t + i % 4
                const int d = S::kF16 ? (i / 4) * 16 + 2 * t + (i & 1) + ((i >> 1) & 1) * 8 : (i / 4) * 16 + 4 * t + (i & 3);
                x[i] = g < nheads && d < p.hd ? __ldg(q + d) * qs : 0.f;
                big = fmaxf(big, fabsf(x[i]));
            }
            if constexpr (S::kF16) {
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                // exponent of the largest |q|, kept where both 2^(13 - e) and 2^(e - 13) are normal
                int e = static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 127;
                e = e == 128 ? 13 : max(-113, min(e, 126));
                const float s = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                unscale = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
#pragma unroll
                for (int i = 0; i < HD / 4; i += 2) split_f16(x[i] * s, x[i + 1] * s, qa[i], qa[i + 1]);
            } else {
#pragma unroll
                for (int i = 0; i < HD / 4; ++i) split_tf32(x[i], qa[2 * i], qa[2 * i + 1]);
            }
            if constexpr (S::kQSmem) {
                // every warp has the same fragments; each writes a quarter (the last segment's have
                // been read: its merge came after)
#pragma unroll
                for (int i = 0; i < S::kQRegs; i += 4)
                    if ((i / 4) % kWarps == warp)
                        *reinterpret_cast<uint4*>(q_s + (i / 4 * 32 + lane) * 4) = make_uint4(qa[i], qa[i + 1], qa[i + 2], qa[i + 3]);
                __syncthreads();
            }
        }

        float O[S::kNT][4] = {};
        float m = -CUDART_INF_F, l = 0.f;  // of head g; l over this lane's slots
        for (; f < fe; f += kWarps) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
            __syncwarp();  // unit f is there, and every lane is done with the one before it
            copy();        // into that one's stage
            locate();
            const uint32_t tile = smem_addr(ring + get * 2 * S::kTileBytes);
            const uint32_t live = live_s[get];
            constexpr int kST = UK / 8;
            float c[kST][4] = {};
            if constexpr (S::kF16) {
                const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    uint32_t r[4];
                    ldm4(tile + swz<true, false>(key, 2 * s + half, S::kRowBytes), r);
                    mma_f16(c[0], qa + 4 * s, r[0], r[1]);
                    mma_f16(c[kST - 1], qa + 4 * s, r[2], r[3]);
                }
            } else {
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    float r[4];
                    lds4(tile + swz<false, false>(g, 4 * s + t, S::kRowBytes), r);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) split_tf32_kv(r[i], hi[i], lo[i]);
                    uint32_t a[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) a[i] = S::kQSmem ? q_s[((2 * s + i / 4) * 32 + lane) * 4 + i % 4] : qa[8 * s + i];
                    mma_tf32(c[0], a, hi[0], hi[1]);
                    mma_tf32(c[0], a + 4, hi[2], hi[3]);
                    mma_tf32(c[0], a, lo[0], lo[1]);
                    mma_tf32(c[0], a + 4, lo[2], lo[3]);
                }
            }
            float sc[2 * kST];
            float mt = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < kST; ++j)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float v = join_halves(c[j][i], c[j][2 + i]) * unscale;
                    sc[2 * j + i] = (live >> (8 * j + 2 * t + i)) & 1u ? v : -CUDART_INF_F;
                    mt = fmaxf(mt, sc[2 * j + i]);
                }
            if (p.add_weight && g < nheads) {
                const int u = static_cast<int>(f - item_start) + at.lo;
                float* dst = p.scores + (static_cast<int64_t>(at.b) * p.nh + h0 + g) * cap + static_cast<int64_t>(u) * UK;
#pragma unroll
                for (int j = 0; j < kST; ++j)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int k = 8 * j + 2 * t + i, slot = u * UK + k;
                        if (slot >= at.first && slot < at.n) dst[k] = sc[2 * j + i];
                    }
            }
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 1));
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 2));
            if (__any_sync(0xffffffffu, mt > m + kLazy)) {
                const float mn = fmaxf(m, mt);
                const float keep = m == mn ? 1.f : ex2(m - mn);
                m = mn;
                l *= keep;
#pragma unroll
                for (int n = 0; n < S::kNT; ++n)
#pragma unroll
                    for (int i = 0; i < 4; ++i) O[n][i] *= keep;
            }
            const float base = (m == -CUDART_INF_F ? 0.f : m) - kPShift;
            uint32_t pa[4];
            float pr[2 * kST];
#pragma unroll
            for (int i = 0; i < 2 * kST; ++i) {
                pr[i] = ex2(sc[i] - base);
                l += pr[i];
            }
            if constexpr (S::kF16) {
                split_f16(pr[0], pr[1], pa[0], pa[1]);
                split_f16(pr[2 * kST - 2], pr[2 * kST - 1], pa[2], pa[3]);
                const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    uint32_t r[4];
                    ldm4t(tile + S::kTileBytes + swz<true, true>(key, 2 * s + half, S::kRowBytes), r);
                    mma_f16(O[2 * s], pa, r[0], r[1]);
                    mma_f16(O[2 * s + 1], pa, r[2], r[3]);
                }
            } else {
                split_tf32(pr[0], pa[0], pa[1]);
                split_tf32(pr[1], pa[2], pa[3]);
#pragma unroll
                for (int s = 0; s < HD / 32; ++s) {
                    // columns 4 (g + 8s) + i are column g of output tile 4s + i
                    float r0[4], r1[4];
                    lds4(tile + S::kTileBytes + swz<false, true>(2 * t, g + 8 * s, S::kRowBytes), r0);
                    lds4(tile + S::kTileBytes + swz<false, true>(2 * t + 1, g + 8 * s, S::kRowBytes), r1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t h0r, l0r, h1r, l1r;
                        split_tf32_kv(r0[i], h0r, l0r);
                        split_tf32_kv(r1[i], h1r, l1r);
                        mma_tf32(O[4 * s + i], pa, h0r, h1r);
                        mma_tf32(O[4 * s + i], pa, l0r, l1r);
                    }
                }
            }
            get = get + 1 == S::kStages ? 0 : get + 1;
        }

        // join the four warps
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        __syncthreads();  // the previous segment's merge has been read
        if (t == 0) {
            merge_m[warp * kAttnHeads + g] = m;
            merge_l[warp * kAttnHeads + g] = l;
        }
        float* mo = merge + (warp * kAttnHeads + g) * S::kORow;
        if constexpr (S::kF16) {
#pragma unroll
            for (int n = 0; n < S::kNT; ++n)
                *reinterpret_cast<float2*>(mo + 8 * n + 2 * t) =
                    make_float2(join_halves(O[n][0], O[n][2]), join_halves(O[n][1], O[n][3]));
        } else {
#pragma unroll
            for (int s = 0; s < HD / 32; ++s)
#pragma unroll
                for (int i = 0; i < 2; ++i)  // columns of tiles 4s .. 4s + 3: four neighbours
                    *reinterpret_cast<float4*>(mo + 4 * (2 * t + i + 8 * s)) = make_float4(
                        join_halves(O[4 * s][i], O[4 * s][2 + i]), join_halves(O[4 * s + 1][i], O[4 * s + 1][2 + i]),
                        join_halves(O[4 * s + 2][i], O[4 * s + 2][2 + i]),
                        join_halves(O[4 * s + 3][i], O[4 * s + 3][2 + i]));
        }
        __syncthreads();
        constexpr int kPer = HD / 64;  // float4 columns of a thread: 16 threads a head
        const int hh = tid >> 4, cc = (tid & 15) * 4;
        float M = -CUDART_INF_F, L = 0.f;
        float4 acc[kPer] = {};
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, merge_m[w * kAttnHeads + hh]);
        for (int w = 0; w < kWarps; ++w) {
            const float mw = merge_m[w * kAttnHeads + hh];
            const float k = mw == M ? 1.f : ex2(mw - M);
            L = fmaf(merge_l[w * kAttnHeads + hh], k, L);
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float4 o = *reinterpret_cast<const float4*>(merge + (w * kAttnHeads + hh) * S::kORow + cc + 64 * i);
                acc[i].x = fmaf(o.x, k, acc[i].x);
                acc[i].y = fmaf(o.y, k, acc[i].y);
                acc[i].z = fmaf(o.z, k, acc[i].z);
                acc[i].w = fmaf(o.w, k, acc[i].w);
            }
        }
        bool finish = fs == item_start && fe == item_end;
        if (!finish) {
            // this CTA's part; parts of an item are numbered by their CTAs
            const int c0 = static_cast<int>(item_start / share), c1 = static_cast<int>((item_end - 1) / share);
            const int part_floats = kAttnHeads * (HD + 2);
            auto part = [&](int c) { return p.part + static_cast<int64_t>(2 * c + (c == c0)) * part_floats; };
            float* mine = part(blockIdx.x);
#pragma unroll
            for (int i = 0; i < kPer; ++i) __stcg(reinterpret_cast<float4*>(mine + hh * HD + cc + 64 * i), acc[i]);
            if (cc == 0) __stcg(reinterpret_cast<float2*>(mine + kAttnHeads * HD + 2 * hh), make_float2(M, L));
            __syncthreads();
            // release this CTA's part (the barrier orders the other threads' writes before) and, in
            // the last CTA, acquire the others'
            if (tid == 0) last_s = atom_add_acq_rel(p.counters + c0, 1u);
            __syncthreads();
            const int n = c1 - c0 + 1;
            finish = last_s == static_cast<unsigned int>(n - 1);
            if (finish) {
                if (tid == 0) p.counters[c0] = 0u;
                // head hh's 16 threads: maximum, weights and sum over the parts; the weights go to shared memory
                M = -CUDART_INF_F;
                for (int i = tid & 15; i < n; i += 16)
                    M = fmaxf(M, __ldcg(reinterpret_cast<const float2*>(part(c0 + i) + kAttnHeads * HD + 2 * hh)).x);
                for (int o = 8; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
                L = 0.f;
                for (int i = tid & 15; i < n; i += 16) {
                    const float2 ml = __ldcg(reinterpret_cast<const float2*>(part(c0 + i) + kAttnHeads * HD + 2 * hh));
                    const float k = ml.x == M ? 1.f : ex2(ml.x - M);
                    merge[hh * kAttnMaxCtas + i] = k;
                    L = fmaf(ml.y, k, L);
                }
                for (int o = 8; o; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
                __syncwarp();
                for (int i = 0; i < kPer; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
                for (int c = 0; c < n; ++c) {
                    const float k = merge[hh * kAttnMaxCtas + c];
                    const float* src = part(c0 + c) + hh * HD + cc;
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const float4 o = __ldcg(reinterpret_cast<const float4*>(src + 64 * i));
                        acc[i].x = fmaf(o.x, k, acc[i].x);
                        acc[i].y = fmaf(o.y, k, acc[i].y);
                        acc[i].z = fmaf(o.z, k, acc[i].z);
                        acc[i].w = fmaf(o.w, k, acc[i].w);
                    }
                }
            }
        }
        if (finish && hh < nheads) {
            const float inv = 1.f / L;  // no weight at all (every score -inf) gives NaN, as the formula does
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int d = cc + 64 * i;
                const float v[4] = {acc[i].x, acc[i].y, acc[i].z, acc[i].w};
                for (int k = 0; k < 4; ++k)
                    if (d + k < p.hd) put_out(p, at.b, h0 + hh, d + k, v[k] * inv);
            }
            if (cc == 0) put_lse(p, at.b, h0 + hh, M - kPShift, L, false);
        }
        fs = fe;
        if (fs < f1) {
            at.u = 0;
            next_item(at);
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

// ---------------------------------------------------------------- running attention weights

constexpr int kWeightThreads = 128, kWeightSlots = 4;  // slots of a thread

// slot_weight[b][kv head][j] += sum over the kv head's q heads of 2^(score - lse).
__global__ void __launch_bounds__(kWeightThreads) paged_attn_weight_kernel(const __grid_constant__ PagedAttnParams p,
                                                                           int chunks) {
    griddep_wait();
    const int item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
    const int b = item / p.nkv, hk = item - b * p.nkv, G = p.nh / p.nkv;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    int n = __ldg(p.lens + b);
    if (n < 0 || n > cap) n = 0;  // flagged by the attention kernel
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    const int64_t h0 = static_cast<int64_t>(b) * p.nh + static_cast<int64_t>(hk) * G;
    float* weight = p.c.slot_weight + static_cast<int64_t>(item) * cap;
    constexpr int kSpan = kWeightThreads * kWeightSlots;
    for (int64_t j0 = first + static_cast<int64_t>(chunk) * kSpan + threadIdx.x; j0 < n;
         j0 += static_cast<int64_t>(chunks) * kSpan) {
        float w[kWeightSlots];
#pragma unroll
        for (int k = 0; k < kWeightSlots; ++k) w[k] = 0.f;
#pragma unroll 4
        for (int g = 0; g < G; ++g) {
            const float lse2 = __ldcg(p.lse2 + h0 + g);
            const float* s = p.scores + (h0 + g) * cap + j0;
#pragma unroll
            for (int k = 0; k < kWeightSlots; ++k)
                if (j0 + k * kWeightThreads < n) w[k] += exp2f(__ldcg(s + k * kWeightThreads) - lse2);
        }
#pragma unroll
        for (int k = 0; k < kWeightSlots; ++k)
            if (j0 + k * kWeightThreads < n) weight[j0 + k * kWeightThreads] += w[k];
    }
}

template <typename KT, int HD>
cudaError_t launch_split(const PagedAttnParams& p, cudaStream_t stream) {
    using S = Split<KT, HD>;
    auto kernel = paged_attn_split_kernel<KT, HD>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    int dev = 0, sms = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const int grid = sms * S::kCtas < kAttnMaxCtas ? sms * S::kCtas : kAttnMaxCtas;
    const int blocks_per_head = (p.nh / p.nkv + kAttnHeads - 1) / kAttnHeads;
    return launch_dependent(kernel, grid, kSplitThreads, S::kSmem, stream, p, blocks_per_head, kMinShare);
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnParams& p, cudaStream_t stream) {
    const int es = p.kv_f16 ? 2 : 4;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * es) | static_cast<uintptr_t>(p.hd * es);
    cudaError_t e;
    if ((bits & 15u) != 0) {  // rows that 16-byte copies cannot read
        e = launch_dependent(paged_attn_any_kernel, p.c.n_seq * p.nh, kAnyThreads, 0, stream, p);
    } else if (p.kv_f16) {
        e = p.hd <= 64 ? launch_split<uint16_t, 64>(p, stream)
                       : p.hd <= 128 ? launch_split<uint16_t, 128>(p, stream) : launch_split<uint16_t, 256>(p, stream);
    } else {
        e = p.hd <= 64 ? launch_split<float, 64>(p, stream)
                       : p.hd <= 128 ? launch_split<float, 128>(p, stream) : launch_split<float, 256>(p, stream);
    }
    if (e != cudaSuccess || !p.add_weight) return e;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    // up to two blocks for every resident one; longer sequences loop
    const int64_t spans = (cap + kWeightThreads * kWeightSlots - 1) / (kWeightThreads * kWeightSlots);
    const int64_t most = 4096 / (static_cast<int64_t>(p.c.n_seq) * p.nkv) + 1;
    const int chunks = static_cast<int>(spans < most ? spans : most);
    return launch_dependent(paged_attn_weight_kernel, p.c.n_seq * p.nkv * chunks, kWeightThreads, 0, stream, p, chunks);
}

cudaError_t paged_attn_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
