// qkv_attn_step: attention of one new token per sequence over a paged cache
// (include/qkv.h has the contract).
//
// s_j = scale * q.K_j, online softmax (running maximum m and sum l), out = sum p_j V_j / l.
// Scores are kept in the log2 domain (scale * log2(e) folded into q), so p = 2^(s - m).
#include <cuda_bf16.h>
#include <math_constants.h>

#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace {

using namespace qkv_paged;
using qkv_ptx::griddep_launch_dependents;
using qkv_ptx::griddep_wait;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Rounded to nearest even.
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __bfloat16_as_ushort(__float2bfloat16_rn(v)); }

__device__ __forceinline__ void put_out(const PagedAttnParams& p, int b, int h, int d, float v) {
    const int64_t at = b * p.out_stride + static_cast<int64_t>(h) * p.hd + d;
    if (p.out_bf16) {
        static_cast<uint16_t*>(p.out)[at] = bf16_bits(v);
    } else {
        static_cast<float*>(p.out)[at] = v;
    }
}

// Four neighbouring values, as one store where the row's address allows it.
__device__ __forceinline__ void put_out4(const PagedAttnParams& p, int64_t at, float4 v) {
    if (p.out_bf16) {
        const uint32_t lo = bf16_bits(v.x) | static_cast<uint32_t>(bf16_bits(v.y)) << 16;
        const uint32_t hi = bf16_bits(v.z) | static_cast<uint32_t>(bf16_bits(v.w)) << 16;
        uint16_t* o = static_cast<uint16_t*>(p.out) + at;
        if ((reinterpret_cast<uintptr_t>(o) & 7u) == 0) {
            *reinterpret_cast<uint2*>(o) = make_uint2(lo, hi);
        } else {
            o[0] = static_cast<uint16_t>(lo);
            o[1] = static_cast<uint16_t>(lo >> 16);
            o[2] = static_cast<uint16_t>(hi);
            o[3] = static_cast<uint16_t>(hi >> 16);
        }
    } else {
        float* o = static_cast<float*>(p.out) + at;
        if ((reinterpret_cast<uintptr_t>(o) & 15u) == 0) {
            *reinterpret_cast<float4*>(o) = v;
        } else {
            o[0] = v.x;
            o[1] = v.y;
            o[2] = v.z;
            o[3] = v.w;
        }
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
    griddep_launch_dependents();
    const int b = blockIdx.x / p.nh, h = blockIdx.x - b * p.nh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int j0 = h / (p.nh / p.nkv) * p.hd;
    const int n = checked_len(p.c, p.lens, b);
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    for (int d = tid; d < p.hd; d += kAnyThreads)
        q_s[d] = p.q[b * p.q_stride + static_cast<int64_t>(h) * p.hd + d] * (p.scale * kLog2e);
    float* scores = p.add_weight ? p.scores + (static_cast<int64_t>(b) * p.nh + h) * p.score_stride : nullptr;
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

// One new token has as many q rows as a kv head has q heads (5 to 8 here): each byte of the cache takes
// 5 to 8 flops, so memory bounds a batch, and latencies a short sequence.  Of M = 128 (the least of a
// tcgen05.mma, whose accumulators would also have to leave TMEM for every softmax step) 8 rows would be used;
// an mma.sync has 16, all in use here, and its pipe is 13 to 17 % busy.
// Measured (GPU time, of the copy rate): 64 sequences of 8 x 128 x f16 to 8192 slots 184 us, DRAM at 6.2 TB/s
// (0.92); one of 32749 slots 29 us (0.68: about 9 us of it are launch, lengths, first pages and the join);
// 32 to 4099 slots with weights 40.2 us; 14 x 64 x f32, 509 slots 5.9 us, all latency.
//
// Work is counted in units of 8 to 32 neighbouring slots of one item (8 KB of K and V as a rule), an item
// being (sequence, kv head, block of up to 8 of its q heads).  Lengths are on the device, so every CTA finds
// its own work from them.  Each item gets CTAs of its own, so that no CTA has two beginnings and ends on its
// path, unless the largest share is then more than kOwnUnits units above that of dealing all units in a row
// to the CTAs in equal contiguous shares (where an item counts kItemCost units more, for its q and its end).
// With more items than CTAs, whole items are dealt where that costs no more than kJoinCost units of joins
// (4 x 128 x f16: 128 sequences of 100 slots 14.6 us, 17.9 us in shares of units; of 400 27.6, 30.0; always whole
// items: the ragged 14B batch 299 us instead of 179).
// The part of an item that a CTA does not hold whole goes to the workspace, and the last CTA to arrive joins
// the item's parts in order (in a cluster: through shared memory).
//
// Within a CTA the units go to the four warps in turn, and each warp is a stream of its own: it copies its
// units into its own ring of stages (cp.async, rows addressed through the page table, rows outside
// the sequence filled with zeros) and computes them, with no barrier but at the end of an item.  Two CTAs of
// four warps on an SM: one of eight takes 188 to 194 us for the batch of 184; warps in step, by barriers, add
// 2.7 us to the 32749 slots; a ring of two stages takes the same.  Code runs few times in a call, so its size
// counts: the loops that fill the ring and join parts are kept rolled.
//
// The 8 q heads of an item take half of the 16 rows of an MMA.  The other half carries what the
// first loses: rows 0-7 hold q rounded to f16 (tf32), rows 8-15 the rounded remainder, and the same
// with the softmax weights, so both products keep 23 bits at no extra MMA.  An f32 cache's own
// rows are split too (two MMAs).  The weights are 2^(s - m + shift) with m at most 3 below the running
// maximum (then O need not be rescaled for every new maximum).  f16: before the split q is scaled by a power of
// two into [2^13, 2^14), and the shift is 12, both far from the type's ends.  f32: the shift is -3, so no weight
// is above 1 and O stays finite wherever sum p_j |V_j| does.  Sums over many MMAs are made outside of them,
// rounded to nearest (add4): 20 x 6000 slots x 8 x 128 x f32 come out 5e-7 off (2-norms) instead of 6.1e-6,
// f16 4e-7 instead of 2.3e-6, at the same times (an f32 batch: 3 % more).

constexpr int kMinShare = 8;     // units
constexpr int kItemCost = 8;     // units
constexpr int kJoinCost = 16;    // units
constexpr int kOwnUnits = 8;     // how much larger the largest share may be with CTAs of its own for each item
constexpr int kMaxAbreast = 8;   // blocks of q heads that go side by side
constexpr int kJoinParts = 40;   // more parts than this are joined in two levels
constexpr float kLazy = 3.f;     // a weight may be 2^3 above the running maximum's before the maximum moves

template <typename KT, int HD>
struct Split {
    using Type = KT;
    static constexpr int kHd = HD;
    static constexpr bool kF16 = sizeof(KT) == 2;
    static constexpr int kWarps = 4, kThreads = 32 * kWarps;
    static constexpr int kCtas = HD == 256 ? 1 : 2;        // per SM
    // slots of a unit: 8 KB of K and V, or the fewest that an MMA takes
    static constexpr int UK = kF16 ? (HD == 64 ? 32 : 16) : (HD == 64 ? 16 : 8);
    static constexpr int kRowBytes = HD * sizeof(KT);
    static constexpr int kTileBytes = UK * kRowBytes;      // K or V of a unit
    static constexpr int kStages = HD < 256 ? 24576 / (2 * kTileBytes) : kF16 ? 3 : 2;
    static constexpr int kRingBytes = kStages * 2 * kTileBytes;
    static constexpr int kNT = HD / 8;                     // output column tiles
    static constexpr int kQuads = HD / 16;                 // a lane's outputs of one head, in fours
    static constexpr int kQRow = HD + (kF16 ? 8 : 16);     // floats; spreads the heads' rows over the banks
    static constexpr int kQLoads = kAttnHeads * HD / kThreads;
    // q's fragments stay in registers beside O, and the next item's q is loaded ahead, where there is room (4 x 128 x
    // f32, 32000 slots, values split by masks: 37 us, with fragments in registers, and spilled, 64).  What the
    // compiler still spills: head size 256 without clusters 144 bytes (f32) and 132 (f16), in clusters 8 (f32); f32
    // of 128 without clusters 12.
    static constexpr bool kQRegs = kF16 && HD < 256;
    static constexpr bool kQAhead = kF16 ? HD < 256 : HD < 128;
    static constexpr float kPShift = kF16 ? 12.f : -kLazy;  // weights are kept times 2^kPShift
    static constexpr int kMergeFloats = (kWarps - 1) * kAttnHeads * HD;  // O of the warps but the first
    static constexpr int kPartFloats = kAttnHeads * (HD + 2);
    static constexpr int kSmem = kWarps * kRingBytes +
                                 4 * (kMergeFloats + 2 * kWarps * kAttnHeads + kAttnHeads * kQRow + kWarps * kStages);
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
// c += t with each sum rounded to nearest (an MMA's own accumulation drops bits, always towards zero, which adds
// up over a long row of MMAs).
__device__ __forceinline__ void add4(float (&c)[4], const float (&t)[4]) {
    unsigned long long x, y;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(c[i]), "f"(c[i + 1]));
        asm("mov.b64 %0, {%1, %2};" : "=l"(y) : "f"(t[i]), "f"(t[i + 1]));
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(x) : "l"(y));
        asm("mov.b64 {%0, %1}, %2;" : "=f"(c[i]), "=f"(c[i + 1]) : "l"(x));
    }
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

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// What CTA `rank` of the cluster has at the place of `p` in its shared memory.
__device__ __forceinline__ uint32_t peer_addr(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ float2 peer_float2(const float2* p, int rank) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_addr(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ float4 peer_float4(const float4* p, int rank) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(peer_addr(p, rank)) : "memory");
    return v;
}

// Two values rounded to f16 in hi, and the remainders rounded to f16 in lo.
__device__ __forceinline__ void split_f16(float a, float b, uint32_t& hi, uint32_t& lo) {
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    hi = *reinterpret_cast<const uint32_t*>(&h);
    lo = *reinterpret_cast<const uint32_t*>(&l);
}
// A value as the sum of two tf32 numbers of 11 bits: itself rounded to nearest, and what is left, rounded too.  Both
// together are off by 2^-23 of the value at most.
__device__ __forceinline__ void split_tf32(float a, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(hi) : "f"(a));
    asm("cvt.rn.tf32.f32 %0, %1;" : "=r"(lo) : "f"(a - __uint_as_float(hi)));
}
// The same for cache values, the rest cut off, which has the same bound and takes the least time (100 x 4000 slots
// of 28/4 x 128: 272 us; the rest rounded 276; both cut by a mask, which loses two bits, 297).  An infinite value
// becomes the largest number and an infinite rest, whose products have the same sign; a NaN becomes two.
__device__ __forceinline__ void split_tf32_kv(float a, uint32_t& hi, uint32_t& lo) {
    asm("cvt.rn.satfinite.tf32.f32 %0, %1;" : "=r"(hi) : "f"(a));
    lo = __float_as_uint(a - __uint_as_float(hi)) & 0xffffe000u;
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
    int b;          // sequence
    int lo, n;      // its first unit and its length
    int first;      // its first slot
    int units;      // units of one of its items
    int item, u;    // item, and unit within it
    int64_t start;  // where the item starts in the order (units and item costs)
};

// An item of which a CTA holds a part.
struct Pending {
    int b, h0, nheads;
    int c0, n;             // the first of its CTAs, and how many
    unsigned int counted;  // parts of the group that were counted before this one
};
__device__ __forceinline__ int join_fan(int n) {
    return n <= kJoinParts ? n : static_cast<int>(ceilf(sqrtf(static_cast<float>(n))));
}

template <int UK>
__device__ __forceinline__ void seq_units(const PagedAttnParams& p, int b, bool flag, Walk& w) {
    int n = p.lens[b];
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

// a / b of non-negative values; 32-bit division where both fit, as they do in all but huge batches.
__device__ __forceinline__ int64_t div_small(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// Column of value j of a lane's quad i (the layout of O's fragments; four neighbours in the f32 case).
template <bool F16>
__device__ __forceinline__ int quad_col(int i, int j, int t) {
    return F16 ? 8 * (2 * i + (j >> 1)) + 2 * t + (j & 1) : 4 * (2 * t + (i & 1) + 8 * (i >> 1)) + j;
}

__device__ __forceinline__ float4 fma4(float4 o, float k, float4 a) {
    return make_float4(fmaf(o.x, k, a.x), fmaf(o.y, k, a.y), fmaf(o.z, k, a.z), fmaf(o.w, k, a.w));
}

// C > 1: clusters of C CTAs, each with units of one item; the CTAs' parts are joined through
// their shared memory.
template <typename KT, int HD, int C>
__global__ void __launch_bounds__(Split<KT, HD>::kThreads, Split<KT, HD>::kCtas)
    paged_attn_split_kernel(const __grid_constant__ PagedAttnParams p, int abreast, int serial) {
    using S = Split<KT, HD>;
    constexpr int UK = S::UK;
    constexpr bool CLUSTERED = C > 1;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Pending pending_s[2];
    __shared__ unsigned int last_s;
    const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in all lanes, and known to be
    const int B = p.c.n_seq, G = p.nh / p.nkv, items = p.nkv * serial;
    // The CTAs (clusters) are dealt to the blocks of q heads that go abreast, which split up their own work alike.
    const int ctas = gridDim.x / abreast;
    const int me = blockIdx.x / C / abreast, blk = blockIdx.x / C - me * abreast;
    const int cta = me * C + blockIdx.x % C;
    float* const parts = p.part + static_cast<int64_t>(2 * blk * ctas) * S::kPartFloats;
    unsigned int* const counters = p.counters + 2 * blk * ctas;
    unsigned char* ring = smem + warp * S::kRingBytes;
    float* merge = reinterpret_cast<float*>(smem + S::kWarps * S::kRingBytes);
    float* merge_m = merge + S::kMergeFloats;
    float* merge_l = merge_m + S::kWarps * kAttnHeads;
    float* q_s = merge_l + S::kWarps * kAttnHeads;
    uint32_t* live_s = reinterpret_cast<uint32_t*>(q_s + kAttnHeads * S::kQRow) + warp * S::kStages;

    // columns beyond hd are zeros for good: no copy writes there
    if (p.hd < HD)
        for (int i = lane * 16; i < S::kRingBytes; i += 512) *reinterpret_cast<uint4*>(ring + i) = make_uint4(0, 0, 0, 0);

    // lengths and page ids on their way to L2 while the launch before this one ends
    const int64_t line = static_cast<int64_t>(blockIdx.x) * S::kThreads + tid;
    if (line * 32 < B) prefetch_l2(p.lens + line * 32);
    if (line * 32 < static_cast<int64_t>(B) * p.c.max_pages) prefetch_l2(p.c.table + line * 32);
    griddep_wait();
    griddep_launch_dependents();  // what follows may take the places of CTAs that are done, and wait there
    // How much there is: units, sequences that have any, and the longest item.  Every warp finds it for
    // itself (32 lengths at a time), which takes fewer latencies than a barrier would.
    int units0 = 0;  // of sequence `lane`
    int64_t total = 0;
    int longest = 0, nonempty = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
        Walk w;
        w.units = 0;
        if (b0 + lane < B) seq_units<UK>(p, b0 + lane, blockIdx.x == 0 && warp == 0, w);
        if (b0 == 0) units0 = w.units;
        total += w.units;
        longest = max(longest, w.units);
        nonempty += w.units > 0;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    nonempty = __reduce_add_sync(0xffffffffu, nonempty);
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
    if (nonempty < B)  // an empty sequence has no unit: its rows are written here
        for (int b = blockIdx.x; b < B; b += gridDim.x) {
            Walk w;
            seq_units<UK>(p, b, false, w);
            if (w.units == 0) {
                for (int i = tid; i < p.nh * p.hd; i += S::kThreads) put_out(p, b, 0, i, 0.f);
                for (int h = tid; h < p.nh; h += S::kThreads) put_lse(p, b, h, 0.f, 0.f, true);
            }
        }
    total *= items;
    const int64_t n_items = static_cast<int64_t>(nonempty) * items;
    // CTAs of their own for the items, ceil(units / share) each, which are no more than the grid; or equal
    // shares of everything, whatever the items, where that makes the largest share clearly smaller.
    // A share is at least kMinShare units (each part costs a join), but not above the longest item.
    const int64_t spare = static_cast<int64_t>(ctas) - C * n_items;
    const int64_t least = min(longest, kMinShare);
    int64_t alone = spare > 0 ? min(max(div_small(total + spare - 1, spare), least), static_cast<int64_t>(longest)) : longest;
    if (CLUSTERED && n_items > 0) {
        // as many clusters for every item as there are for one take less where lengths are alike, and one for
        // each saves a join
        const int64_t even = div_small(ctas / C, n_items) * C, single = max(div_small(longest + C - 1, C), least);
        if (even > 0) alone = min(alone, max(div_small(longest + even - 1, even), least));
        if (single <= alone + kOwnUnits) alone = max(alone, single);
    }
    const int64_t dealt = max(div_small(total + n_items * kItemCost + ctas - 1, ctas), least + kItemCost);
    const bool own = CLUSTERED || (spare >= 0 && alone <= dealt + kOwnUnits);
    // Not own: whole items, the same number for every CTA (each taking the room of the longest), where that makes
    // the largest share no more than dealing units does with its joins.
    const int64_t each = div_small(n_items + ctas - 1, ctas);
    const bool whole = !own && each * (longest + kItemCost) <= dealt + kJoinCost;
    const int cost = own || whole ? 0 : kItemCost;
    const int room = whole ? longest : 0;
    const int64_t share = own ? alone : whole ? each * room : dealt;
    // The order is counted in CTAs (own) or in units and item costs; this CTA starts at x.
    const int64_t x = own ? cta : share * cta;
    auto extent = [&](int units) -> int64_t {  // of one item
        if (units == 0 || !own) return units == 0 ? 0 : max(units + cost, room);
        const int n = (units + static_cast<int>(share) - 1) / static_cast<int>(share);
        return (n + C - 1) / C * C;
    };
    int64_t before = 0, start = 0;  // extent of the sequences before this round's; where x's sequence starts
    int b_at = -1;
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
        Walk w;
        w.units = units0;
        if (b0 > 0) {
            w.units = 0;
            if (b0 + lane < B) seq_units<UK>(p, b0 + lane, false, w);
        }
        const int64_t size = extent(w.units) * items;
        int64_t incl = size;
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        incl += before;
        const unsigned int here = __ballot_sync(0xffffffffu, size > 0 && incl - size <= x && x < incl);
        if (here) {
            b_at = b0 + __ffs(here) - 1;
            start = __shfl_sync(0xffffffffu, incl - size, __ffs(here) - 1);
            break;
        }
        before = __shfl_sync(0xffffffffu, incl, 31);
    }
    if (b_at < 0) return;  // nothing starts here or later

    auto next_item = [&](Walk& w) {  // called only where an item follows
        w.start += max(w.units + cost, room);
        w.u = 0;
        if (++w.item < items) return;
        w.item = 0;
        do seq_units<UK>(p, w.b + 1, false, w);
        while (w.units == 0);
    };
    Walk at;     // the segment being computed: the CTA's units of one item, from at.u
    seq_units<UK>(p, b_at, false, at);
    int64_t end;      // where this CTA's share ends in the order
    int c0 = 0, c1 = 0;  // first and last CTA (cluster) of the item (own)
    {
        const int64_t e = extent(at.units);
        at.item = static_cast<int>(div_small(x - start, e));
        const int64_t r = (x - start) - at.item * e;
        if (own) {  // chunk r of e: the order is the item's own units
            c0 = static_cast<int>(cta - r) / C;
            c1 = c0 + static_cast<int>(e) / C - 1;
            at.start = 0;
            const int n = static_cast<int>(e), each = at.units / n, left = at.units - each * n, i = static_cast<int>(r);
            at.u = i * each + min(i, left);
            end = at.u + each + (i < left ? 1 : 0);
        } else {
            at.start = start + at.item * e;
            at.u = static_cast<int>(r);
            end = min(x + share, whole ? n_items * room : total + n_items * cost);
            if (at.u >= at.units) {  // only the item's cost is left here
                if (at.start + at.units + cost >= end) return;  // (never of whole items)
                next_item(at);
            }
        }
    }

    // q of the item's heads, scaled to log2 terms: through registers into q_s, zeros where there is none
    float qx[S::kQLoads];
    auto load_q = [&](const Walk& w) {
        const int hk = w.item / serial, hb = w.item - hk * serial + blk;
        const int nheads = min(kAttnHeads, G - hb * kAttnHeads);
        const float* q = p.q + w.b * p.q_stride + static_cast<int64_t>(hk * G + hb * kAttnHeads) * p.hd;
#pragma unroll
        for (int i = 0; i < S::kQLoads; ++i) {
            const int e = tid + i * S::kThreads, h = e / HD, d = e % HD;
            qx[i] = h < nheads && d < p.hd ? __ldca(q + h * p.hd + d) : 0.f;  // (a plain load: +1.5 us at 32768 slots)
        }
    };
    auto keep_q = [&]() {
#pragma unroll
        for (int i = 0; i < S::kQLoads; ++i) {
            const int e = tid + i * S::kThreads;
            q_s[e / HD * S::kQRow + e % HD] = qx[i] * (p.scale * kLog2e);
        }
    };
    load_q(at);

    Walk ahead = at;  // the unit to be copied next
    int skip = warp;  // how many units it is behind that
    bool more = true;
    const int hd_chunks = p.hd * static_cast<int>(sizeof(KT)) / 16;
    constexpr int kChunks = S::kRowBytes / 16;
    // Move to the warp's next unit and ask the table for its pages (lane = slot of the unit); nothing waits
    // for the answer before place() makes it the offset of the slot's row (-1: not read).
    struct Asked {
        int id, in_page, col;
        bool in, there;
    };
    auto ask = [&]() {
        Asked a = {0, 0, 0, false, false};
        if (!more) return a;
        int u = ahead.u + skip;
        skip = S::kWarps;
        while (u >= ahead.units) {
            u -= ahead.units;
            if (ahead.start + max(ahead.units + cost, room) >= end) {
                more = false;
                return a;
            }
            next_item(ahead);
        }
        ahead.u = u;
        if (ahead.start + u >= end) {
            more = false;
            return a;
        }
        const int slot = (ahead.lo + u) * UK + lane;
        a.there = true;
        a.in = lane < UK && slot >= ahead.first && slot < ahead.n;
        a.col = ahead.item / serial * p.hd;
        if (a.in) {
            const int pg = slot / p.c.page_size;
            a.in_page = slot - pg * p.c.page_size;
            a.id = p.c.table[static_cast<int64_t>(ahead.b) * p.c.max_pages + pg];
        }
        return a;
    };
    auto place = [&](const Asked& a) -> int64_t {
        if (!a.in) return -1;
        if (static_cast<unsigned int>(a.id) >= static_cast<unsigned int>(p.c.n_pages)) {
            flag_bad(kFlagIndexRange, a.id);
            return -1;
        }
        return a.id * p.c.page_stride + static_cast<int64_t>(a.in_page) * p.c.nkt + a.col;
    };
    int put = S::kStages - 1;  // stage that the next unit goes to (the first copy is of no unit)
    auto copy = [&](const Asked& a) {
        if (a.there) {
            const int64_t row = place(a);
            const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
            if (lane == 0) live_s[put] = live;
            const uint32_t dst = smem_addr(ring + put * 2 * S::kTileBytes);
            const int64_t off = row >= 0 ? row : 0;
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
    };
    // Outputs of an item go through shared memory (the place of the warps' O) into its rows.
    auto keep_out = [&](int i, float4 o, float inv) {  // no weight at all (every score -inf) gives NaN, as the formula does
        const float v[4] = {o.x * inv, o.y * inv, o.z * inv, o.w * inv};
#pragma unroll
        for (int j = 0; j < 4; ++j) merge[g * HD + quad_col<S::kF16>(i, j, t)] = v[j];
    };
    auto put_rows = [&](int b, int h0, int nheads) {
        const int64_t to = b * p.out_stride + static_cast<int64_t>(h0) * p.hd;
#pragma unroll 1
        for (int e = lane * 4; e < nheads * p.hd; e += 128) {  // hd is a multiple of 4 here
            const int h = e / p.hd;
            put_out4(p, to + e, *reinterpret_cast<const float4*>(merge + h * HD + (e - h * p.hd)));
        }
    };
    auto part = [&](const Pending& e, int c) { return parts + static_cast<int64_t>(2 * c + (c == e.c0)) * S::kPartFloats; };
    int pendings = 0;  // segments that are not whole items

    int get = 0;             // stage of the next unit to compute
    int u = at.u + warp;     // that unit
    // The copies run kStages - 1 units ahead and the questions to the table one more (after the first, most
    // hit L1: a line of the table names 32 pages).  `warm` counts the rounds that only fill the ring; they
    // share the loop's code.
    Asked asked = {0, 0, 0, false, false};
    int warm = S::kStages;
    for (;;) {
        const int us = at.u, ue = end - at.start < at.units ? static_cast<int>(end - at.start) : at.units;
        const int hk = at.item / serial, hb = at.item - hk * serial + blk;
        const int h0 = hk * G + hb * kAttnHeads, nheads = min(kAttnHeads, G - hb * kAttnHeads);
        const bool follows = at.start + max(at.units + cost, room) < end;
        Walk next = at;
        if (follows) next_item(next);

        uint32_t qa[S::kQRegs ? HD / 4 : 8];  // q of head g as A fragments
        float unscale = 1.f;
        const float* qg = q_s + g * S::kQRow;
        float O[S::kNT][4];
        float m = -CUDART_INF_F, l = 0.f;  // of head g; l over this lane's slots
        for (bool fresh = true;;) {
            if (warm == 0) {
                if (fresh) {
                    fresh = false;
                    if constexpr (S::kF16) {
                        float big = 0.f;
#pragma unroll
                        for (int s = 0; s < HD / 8; ++s) {
                            const float2 v = *reinterpret_cast<const float2*>(qg + 8 * s + 2 * t);
                            big = fmaxf(big, fmaxf(fabsf(v.x), fabsf(v.y)));
                        }
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
                        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
                        // exponent of the largest |q|, kept where both 2^(13 - e) and 2^(e - 13) are normal
                        int e = static_cast<int>((__float_as_uint(big) >> 23) & 255u) - 127;
                        e = e == 128 ? 13 : max(-113, min(e, 126));
                        const float sc = __uint_as_float(static_cast<uint32_t>(13 - e + 127) << 23);
                        unscale = __uint_as_float(static_cast<uint32_t>(e - 13 + 127) << 23);
                        auto fragment = [&](int s, uint32_t* a) {  // of 16 columns
                            const float2 v = *reinterpret_cast<const float2*>(qg + 16 * s + 2 * t);
                            const float2 w = *reinterpret_cast<const float2*>(qg + 16 * s + 8 + 2 * t);
                            split_f16(v.x * sc, v.y * sc, a[0], a[1]);
                            split_f16(w.x * sc, w.y * sc, a[2], a[3]);
                        };
                        if constexpr (S::kQRegs) {
#pragma unroll
                            for (int s = 0; s < HD / 16; ++s) fragment(s, qa + 4 * s);
                        } else {  // the fragments take q's place; each warp makes a part of them
                            constexpr int kPart = HD / 16 / S::kWarps;
                            uint32_t a[4 * kPart];
#pragma unroll
                            for (int s = 0; s < kPart; ++s) fragment(warp * kPart + s, a + 4 * s);
                            __syncthreads();
#pragma unroll
                            for (int s = 0; s < kPart; ++s)
                                reinterpret_cast<uint4*>(q_s)[(warp * kPart + s) * 32 + lane] =
                                    make_uint4(a[4 * s], a[4 * s + 1], a[4 * s + 2], a[4 * s + 3]);
                            __syncthreads();
                        }
                    }
                    if (S::kQAhead && follows) load_q(next);  // waited for at this segment's end
#pragma unroll
                    for (int n = 0; n < S::kNT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i) O[n][i] = 0.f;
                }
                if (u >= ue) break;
                asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
                __syncwarp();  // unit u is there, and every lane is done with the one before it
            }
            copy(asked);  // into that one's stage
            asked = ask();
            if (warm > 0) {
                if (--warm == 0) {
                    keep_q();
                    __syncthreads();
                }
                continue;
            }
            const uint32_t tile = smem_addr(ring + get * 2 * S::kTileBytes);
            const uint32_t live = live_s[get];
            constexpr int kST = UK / 8;
            float c[kST][4] = {};
            if constexpr (S::kF16) {
                const int key = ((lane >> 4) << 3) + (lane & 7), half = (lane >> 3) & 1;
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    uint32_t* a = qa + (S::kQRegs ? 4 * s : 0);
                    if constexpr (!S::kQRegs) {
                        const uint4 v = reinterpret_cast<const uint4*>(q_s)[s * 32 + lane];
                        a[0] = v.x;
                        a[1] = v.y;
                        a[2] = v.z;
                        a[3] = v.w;
                    }
#pragma unroll
                    for (int j = 0; j < kST; j += 2) {
                        uint32_t r[4];
                        ldm4(tile + swz<true, false>(8 * j + key, 2 * s + half, S::kRowBytes), r);
                        float s0[4] = {}, s1[4] = {};
                        mma_f16(s0, a, r[0], r[1]);
                        mma_f16(s1, a, r[2], r[3]);
                        add4(c[j], s0);
                        add4(c[j + 1], s1);
                    }
                }
            } else {
#pragma unroll
                for (int s = 0; s < HD / 16; ++s) {
                    uint32_t* a = qa;
                    const float4 v = *reinterpret_cast<const float4*>(qg + 16 * s + 4 * t);
                    split_tf32(v.x, a[0], a[1]);
                    split_tf32(v.y, a[2], a[3]);
                    split_tf32(v.z, a[4], a[5]);
                    split_tf32(v.w, a[6], a[7]);
#pragma unroll
                    for (int j = 0; j < kST; ++j) {
                        float r[4];
                        lds4(tile + swz<false, false>(8 * j + g, 4 * s + t, S::kRowBytes), r);
                        uint32_t hi[4], lo[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) split_tf32_kv(r[i], hi[i], lo[i]);
                        float sum[4] = {};
                        mma_tf32(sum, a, lo[0], lo[1]);  // the small products first, as nothing is cut off them
                        mma_tf32(sum, a + 4, lo[2], lo[3]);
                        mma_tf32(sum, a, hi[0], hi[1]);
                        mma_tf32(sum, a + 4, hi[2], hi[3]);
                        add4(c[j], sum);
                    }
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
            if (p.add_weight && g < nheads) {  // whole units: the rows of scores are padded to them
                float* dst = p.scores + (static_cast<int64_t>(at.b) * p.nh + h0 + g) * p.score_stride + (at.lo + u) * UK + 2 * t;
#pragma unroll
                for (int j = 0; j < kST; ++j) *reinterpret_cast<float2*>(dst + 8 * j) = make_float2(sc[2 * j], sc[2 * j + 1]);
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
            const float base = (m == -CUDART_INF_F ? 0.f : m) - S::kPShift;
            float pr[2 * kST];
#pragma unroll
            for (int i = 0; i < 2 * kST; ++i) {
                pr[i] = ex2(sc[i] - base);
                l += pr[i];
            }
            if constexpr (S::kF16) {
                const int key = (((lane >> 3) & 1) << 3) + (lane & 7), half = lane >> 4;
#pragma unroll
                for (int j = 0; j < kST; j += 2) {  // 16 slots
                    uint32_t pa[4];
                    split_f16(pr[2 * j], pr[2 * j + 1], pa[0], pa[1]);
                    split_f16(pr[2 * j + 2], pr[2 * j + 3], pa[2], pa[3]);
#pragma unroll
                    for (int s = 0; s < HD / 16; ++s) {
                        uint32_t r[4];
                        ldm4t(tile + S::kTileBytes + swz<true, true>(8 * j + key, 2 * s + half, S::kRowBytes), r);
                        float t0[4] = {}, t1[4] = {};
                        mma_f16(t0, pa, r[0], r[1]);
                        mma_f16(t1, pa, r[2], r[3]);
                        add4(O[2 * s], t0);
                        add4(O[2 * s + 1], t1);
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < kST; ++j) {  // 8 slots
                    uint32_t pa[4];
                    split_tf32(pr[2 * j], pa[0], pa[1]);
                    split_tf32(pr[2 * j + 1], pa[2], pa[3]);
#pragma unroll
                    for (int s = 0; s < HD / 32; ++s) {
                        // columns 4 (g + 8s) + i are column g of output tile 4s + i
                        float r0[4], r1[4];
                        lds4(tile + S::kTileBytes + swz<false, true>(8 * j + 2 * t, g + 8 * s, S::kRowBytes), r0);
                        lds4(tile + S::kTileBytes + swz<false, true>(8 * j + 2 * t + 1, g + 8 * s, S::kRowBytes), r1);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t h0r, l0r, h1r, l1r;
                            split_tf32_kv(r0[i], h0r, l0r);
                            split_tf32_kv(r1[i], h1r, l1r);
                            float tile[4] = {};
                            mma_tf32(tile, pa, l0r, l1r);
                            mma_tf32(tile, pa, h0r, h1r);
                            add4(O[4 * s + i], tile);
                        }
                    }
                }
            }
            get = get + 1 == S::kStages ? 0 : get + 1;
            u += S::kWarps;
        }
        u -= ue;  // the warp's first unit of the next segment

        // The four warps' sums into warp 0, in lane-linear quads.
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (!S::kQAhead && follows) load_q(next);
        float4 acc[S::kQuads];
#pragma unroll
        for (int i = 0; i < S::kQuads; ++i) {
            if constexpr (S::kF16)
                acc[i] = make_float4(join_halves(O[2 * i][0], O[2 * i][2]), join_halves(O[2 * i][1], O[2 * i][3]),
                                     join_halves(O[2 * i + 1][0], O[2 * i + 1][2]),
                                     join_halves(O[2 * i + 1][1], O[2 * i + 1][3]));
            else  // tiles 4s .. 4s + 3, column 2t + (i & 1)
                acc[i] = make_float4(join_halves(O[4 * (i >> 1)][i & 1], O[4 * (i >> 1)][2 + (i & 1)]),
                                     join_halves(O[4 * (i >> 1) + 1][i & 1], O[4 * (i >> 1) + 1][2 + (i & 1)]),
                                     join_halves(O[4 * (i >> 1) + 2][i & 1], O[4 * (i >> 1) + 2][2 + (i & 1)]),
                                     join_halves(O[4 * (i >> 1) + 3][i & 1], O[4 * (i >> 1) + 3][2 + (i & 1)]));
        }
        if constexpr (CLUSTERED) {
            // All warps' sums to shared memory (the place of their units); then each CTA of the cluster joins its
            // share of the quads, and so do, where clusters share an item, the CTAs of its last cluster to arrive.
            // Four threads take a quad: a warp of each CTA one, then a quarter of the clusters.  (Warps joined first,
            // then CTAs by the cluster's first one: 0.7 us more for 28/4 x 128 x f16, 1641 slots.)
            constexpr int kPer = S::kQuads * 32 / C;  // quads of a CTA
            const int rank = blockIdx.x % C, w = tid & 3, clusters = c1 - c0 + 1;
            float2* ml = reinterpret_cast<float2*>(merge_m);
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
#pragma unroll
            for (int i = 0; i < S::kQuads; ++i) reinterpret_cast<float4*>(ring)[i * 32 + lane] = acc[i];
            if (t == 0) ml[warp * kAttnHeads + g] = make_float2(m, l);
            cluster_sync();
            auto part_of = [&](int c) {  // of the item's cluster c, this CTA's share
                return p.part + static_cast<int64_t>(2 * ((c * abreast + blk) * C + rank)) * S::kPartFloats;
            };
            auto join4 = [&](float& M, float& L, float4& v) {
                float top = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float k = M == top ? 1.f : ex2(M - top);
                M = top;
                L *= k;
                v = fma4(v, k, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    L += __shfl_xor_sync(0xffffffffu, L, x);
                    v.x += __shfl_xor_sync(0xffffffffu, v.x, x);
                    v.y += __shfl_xor_sync(0xffffffffu, v.y, x);
                    v.z += __shfl_xor_sync(0xffffffffu, v.z, x);
                    v.w += __shfl_xor_sync(0xffffffffu, v.w, x);
                }
            };
            auto emit = [&](int e, float M, float L, float4 v) {  // a column a thread
                const int h = (e & 31) >> 2, col = quad_col<S::kF16>(e >> 5, w, e & 3);
                const float mine = w < 2 ? (w == 0 ? v.x : v.y) : (w == 2 ? v.z : v.w);
                if (h >= nheads) return;
                if (col < p.hd) put_out(p, at.b, h0 + h, col, mine / L);
                if ((e & ~28) == 0 && w == 0) put_lse(p, at.b, h0 + h, M - S::kPShift, L, false);
            };
            const float4* theirs = reinterpret_cast<const float4*>(smem + w * S::kRingBytes);
#pragma unroll 1
            for (int f = tid >> 2; f < kPer; f += S::kThreads / 4) {
                const int e = rank * kPer + f;
                float2 v[C];
                float4 o[C];
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    v[r] = peer_float2(ml + w * kAttnHeads + ((e & 31) >> 2), r);
                    o[r] = peer_float4(theirs + e, r);
                }
                float M = v[0].x, L = 0.f;
                float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 1; r < C; ++r) M = fmaxf(M, v[r].x);
#pragma unroll
                for (int r = 0; r < C; ++r) {
                    const float k = v[r].x == M ? 1.f : ex2(v[r].x - M);
                    L = fmaf(v[r].y, k, L);
                    sum = fma4(o[r], k, sum);
                }
                join4(M, L, sum);
                if (clusters == 1) {
                    emit(e, M, L, sum);
                } else if (w == 0) {
                    float4* to = reinterpret_cast<float4*>(part_of(me));
                    __stcg(to + f, sum);
                    if ((f & 3) == 0) __stcg(reinterpret_cast<float2*>(to + kPer) + (f >> 2), make_float2(M, L));
                }
            }
            __syncwarp();
            asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
            if (clusters > 1) {
                unsigned int* counter = p.counters + (c0 * abreast + blk) * C + rank;
                __syncthreads();
                if (tid == 0) last_s = atom_add_acq_rel(counter, 1u);
                __syncthreads();
                if (last_s == static_cast<unsigned int>(clusters - 1)) {
                    if (tid == 0) *counter = 0u;
#pragma unroll 1
                    for (int f = tid >> 2; f < kPer; f += S::kThreads / 4) {
                        float M = -CUDART_INF_F, L = 0.f;
                        float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
                        for (int c = w; c < clusters; c += 16) {
                            float2 v[4];
                            float4 o[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4* from = reinterpret_cast<const float4*>(part_of(c0 + min(c + 4 * i, clusters - 1)));
                                v[i] = __ldcg(reinterpret_cast<const float2*>(from + kPer) + (f >> 2));
                                o[i] = __ldcg(from + f);
                            }
                            float top = M;
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (c + 4 * i < clusters) top = fmaxf(top, v[i].x);
                            const float keep = M == top ? 1.f : ex2(M - top);
                            M = top;
                            L *= keep;
                            sum = fma4(sum, keep, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (c + 4 * i < clusters) {
                                    const float k = v[i].x == M ? 1.f : ex2(v[i].x - M);
                                    L = fmaf(v[i].y, k, L);
                                    sum = fma4(o[i], k, sum);
                                }
                        }
                        join4(M, L, sum);
                        emit(rank * kPer + f, M, L, sum);
                    }
                }
            }
            __syncwarp();
            asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // no CTA leaves while its sums may be read
        } else {
            __syncthreads();  // the last segment's merge and this one's q have been read
            if (warp > 0) {
                if (t == 0) {
                    merge_m[warp * kAttnHeads + g] = m;
                    merge_l[warp * kAttnHeads + g] = l;
                }
                float4* mo = reinterpret_cast<float4*>(merge) + (warp - 1) * S::kQuads * 32 + lane;
#pragma unroll
                for (int i = 0; i < S::kQuads; ++i) mo[i * 32] = acc[i];
            }
            if (follows) keep_q();
            __syncthreads();
            float M = m, L = l;
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < S::kWarps; ++w) M = fmaxf(M, merge_m[w * kAttnHeads + g]);
                const float k0 = m == M ? 1.f : ex2(m - M);
                L = l * k0;
#pragma unroll
                for (int i = 0; i < S::kQuads; ++i) acc[i] = fma4(acc[i], k0, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll
                for (int w = 1; w < S::kWarps; ++w) {
                    const float mw = merge_m[w * kAttnHeads + g], k = mw == M ? 1.f : ex2(mw - M);
                    L = fmaf(merge_l[w * kAttnHeads + g], k, L);
                    const float4* mo = reinterpret_cast<const float4*>(merge) + (w - 1) * S::kQuads * 32 + lane;
#pragma unroll
                    for (int i = 0; i < S::kQuads; ++i) acc[i] = fma4(mo[i * 32], k, acc[i]);
                }
            }
            if (us == 0 && ue == at.units) {
                if (warp == 0) {
                    __syncwarp();  // the warps' O have been read: their place takes the rows
                    const float inv = 1.f / L;
#pragma unroll
                    for (int i = 0; i < S::kQuads; ++i) keep_out(i, acc[i], inv);
                    if (t == 0 && g < nheads) put_lse(p, at.b, h0 + g, M - S::kPShift, L, false);
                    __syncwarp();
                    put_rows(at.b, h0, nheads);
                }
            } else {
                // This CTA's part; an item's parts are those of its CTAs c0 .. c1, and the last of a group of
                // them to be counted will be joined by its CTA, at the end of all its units.  A CTA has two
                // such segments at most, its first and its last.
                if (!own) {
                    c0 = static_cast<int>(div_small(at.start, share));
                    c1 = static_cast<int>(div_small(at.start + at.units - 1, share));
                }
                if (warp == 0) {
                    const Pending e = {at.b, h0, nheads, c0, c1 - c0 + 1, 0u};
                    float* to = part(e, me);
                    if (g < nheads) {
#pragma unroll
                        for (int i = 0; i < S::kQuads; ++i) __stcg(reinterpret_cast<float4*>(to) + i * 32 + lane, acc[i]);
                        if (t == 0) __stcg(reinterpret_cast<float2*>(to + kAttnHeads * HD) + g, make_float2(M, L));
                    }
                    __syncwarp();
                    if (lane == 0) {
                        const int fan = join_fan(e.n), first = e.c0 + (me - e.c0) / fan * fan;
                        pending_s[pendings] = e;
                        // release the part (the warp's writes come before, by its barrier)
                        pending_s[pendings].counted = atom_add_acq_rel(counters + 2 * first + (first == e.c0), 1u);
                    }
                }
                ++pendings;
            }
        }
        if (CLUSTERED || !follows) break;  // a cluster has one item
        at = next;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");

    // Join what this CTA was the last to complete: groups of neighbouring parts first, then the groups
    // (one group where the parts are few).
#pragma unroll 1
    for (int k = 0; k < pendings; ++k) {
        __syncthreads();  // pending_s is written; the ring and the last join's rows have been read
        const Pending e = pending_s[k];
        const int fan = join_fan(e.n), groups = (e.n + fan - 1) / fan, group = (me - e.c0) / fan;
        int first = e.c0 + group * fan, count = min(fan, e.n - group * fan), stride = 1;
        unsigned int* counter = counters + 2 * first + (first == e.c0);
        unsigned int counted = e.counted;
        constexpr int kMine = 2 * HD / S::kThreads;  // fours of one head that a thread joins
        // Each thread copies its pieces of many parts into shared memory of its own (the ring's place), all
        // in flight together, then sums them with a short loop: code that runs once is fetched as it runs.
        constexpr int kPieces = S::kThreads * 16 * (kMine + 1);
        constexpr int kBatch = S::kWarps * S::kRingBytes / kPieces;
        float4 sum[kMine];
        float Mh, Lh;
#pragma unroll 1
        while (counted == static_cast<unsigned int>(count - 1)) {
            if (tid == 0) *counter = 0u;
#pragma unroll
            for (int i = 0; i < kMine; ++i) sum[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            Mh = -CUDART_INF_F;
            Lh = 0.f;
#pragma unroll 1
            for (int b0 = 0; b0 < count; b0 += kBatch) {
                const int nb = min(kBatch, count - b0);
                if (g < e.nheads) {
#pragma unroll 1
                    for (int c = 0; c < nb; ++c) {
                        const float4* from = reinterpret_cast<const float4*>(part(e, first + (b0 + c) * stride));
                        const uint32_t to = smem_addr(smem + c * kPieces);
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            cp_async16(to + (i * S::kThreads + tid) * 16, from + i * S::kThreads + tid, 16u);
                        // maximum and sum of heads 2i and 2i + 1
                        cp_async16(to + (kMine * S::kThreads + tid) * 16, from + S::kQuads * 32 + (g >> 1), 16u);
                    }
                    asm volatile("cp.async.wait_all;" ::: "memory");
                    const float2* ml = reinterpret_cast<const float2*>(smem) + 2 * (kMine * S::kThreads + tid) + (g & 1);
                    float mb = Mh;
#pragma unroll 4
                    for (int c = 0; c < nb; ++c) mb = fmaxf(mb, ml[c * (kPieces / 8)].x);
                    const float keep = Mh == mb ? 1.f : ex2(Mh - mb);
                    Mh = mb;
                    Lh *= keep;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) sum[i] = fma4(sum[i], keep, make_float4(0.f, 0.f, 0.f, 0.f));
#pragma unroll 4
                    for (int c = 0; c < nb; ++c) {
                        const float2 v = ml[c * (kPieces / 8)];
                        const float k = v.x == Mh ? 1.f : ex2(v.x - Mh);
                        Lh = fmaf(v.y, k, Lh);
#pragma unroll
                        for (int i = 0; i < kMine; ++i)
                            sum[i] = fma4(reinterpret_cast<const float4*>(smem + c * kPieces)[i * S::kThreads + tid], k, sum[i]);
                    }
                }
            }
            if (stride > 1 || groups == 1) {
                if (g < e.nheads) {
                    const float inv = 1.f / Lh;
#pragma unroll
                    for (int i = 0; i < kMine; ++i) keep_out(i * S::kWarps + warp, sum[i], inv);
                    if (warp == 0 && t == 0) put_lse(p, e.b, e.h0 + g, Mh - S::kPShift, Lh, false);
                }
                __syncthreads();
                if (warp == 0) put_rows(e.b, e.h0, e.nheads);
                break;
            }
            __syncthreads();  // the parts have been read: the first one's place takes the group's
            if (g < e.nheads) {
                float4* to = reinterpret_cast<float4*>(part(e, first));
#pragma unroll
                for (int i = 0; i < kMine; ++i) __stcg(to + i * S::kThreads + tid, sum[i]);
                if (warp == 0 && t == 0) __stcg(reinterpret_cast<float2*>(to + S::kQuads * 32) + g, make_float2(Mh, Lh));
            }
            first = e.c0;
            count = groups;
            stride = fan;
            counter = p.counters + 2 * kAttnMaxCtas + blk * ctas + e.c0;
            __syncthreads();
            if (tid == 0) last_s = atom_add_acq_rel(counter, 1u);
            __syncthreads();
            counted = last_s;
        }
    }
}

// ---------------------------------------------------------------- running attention weights

constexpr int kWeightThreads = 128, kWeightSpan = 4 * kWeightThreads;  // slots of a CTA

// slot_weight[b][kv head][j] += sum over the kv head's q heads of 2^(score - lse): four neighbouring slots a
// thread, the rows of all heads in flight together.  A second pass over 4 bytes a score, since no weight is
// known before the whole row's sum; 6 us more for 32 x 28 heads to 4099 slots, 8.9 us alone with cold caches
// (8.9 MB, 1.0 TB/s: bound by two loads' latency, which the attention's end hides in part).
__global__ void __launch_bounds__(kWeightThreads) paged_attn_weight_kernel(const __grid_constant__ PagedAttnParams p,
                                                                           int chunks) {
    // Lengths and old weights do not come from the attention kernel, and what comes before that one was done
    // when it began: they are read while it ends.
    const int item = blockIdx.x / chunks, chunk = blockIdx.x - item * chunks;
    const int b = item / p.nkv, hk = item - b * p.nkv, G = p.nh / p.nkv;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    int n = __ldcg(p.lens + b);
    if (n < 0 || n > cap) n = 0;  // flagged by the attention kernel
    const int first = p.window > 0 ? max(0, n - p.window) : 0;
    const int64_t h0 = static_cast<int64_t>(b) * p.nh + static_cast<int64_t>(hk) * G;
    float* weight = p.c.slot_weight + static_cast<int64_t>(item) * cap;
    bool waited = false;
    for (int64_t j = (first & ~3) + static_cast<int64_t>(chunk) * kWeightSpan + threadIdx.x * 4; j < n;
         j += static_cast<int64_t>(chunks) * kWeightSpan) {
        float old[4], w[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int k = 0; k < 4; ++k) old[k] = j + k >= first && j + k < n ? __ldcg(weight + j + k) : 0.f;
        if (!waited) {
            griddep_wait();
            waited = true;
        }
#pragma unroll 8
        for (int g = 0; g < G; ++g) {
            const float lse2 = __ldcg(p.lse2 + h0 + g);
            const float4 s = __ldcg(reinterpret_cast<const float4*>(p.scores + (h0 + g) * p.score_stride + j));
            w[0] += ex2(s.x - lse2);
            w[1] += ex2(s.y - lse2);
            w[2] += ex2(s.z - lse2);
            w[3] += ex2(s.w - lse2);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (j + k >= first && j + k < n) weight[j + k] = old[k] + w[k];
    }
    if (!waited) griddep_wait();
    griddep_launch_dependents();
}

// How many clusters of the split kernel are launched at most: by the kernel's CTAs on an SM and the cluster's size.
// Clusters need neighbouring SMs, and only a perfect packing holds as many as the occupancy query says: of 36
// clusters of 8, a launch behind another kernel had 33 to 36 running at once, the rest after them (28/4 x 128 x f16,
// 24000 slots: 25.7 us on 36 clusters, 18.5 on 32).  So these are 8/9 of what a GB300 holds (36, 74 and 152; with one
// CTA an SM 15, 36 and 76), and constants: the split of the sums follows from them, and what the query says depends on
// the device's layout and the process's limits.
constexpr int sure_clusters(int ctas_per_sm, int size) {
    return ctas_per_sm == 2 ? (size == 8 ? 32 : size == 4 ? 65 : 135) : (size == 8 ? 13 : size == 4 ? 32 : 67);
}

struct Grid {
    int ctas, cluster;    // CTAs in all, and of a cluster
    int abreast, serial;  // blocks of q heads of a kv head: side by side, and one after another
};

// Clusters of C where every item can have two of them (C = 8), or one if sequences are short, and sequences can
// be longer than what one CTA does as fast (6 units).  No more clusters than can have work.  28/4 x 128 x f16
// without and with: one sequence of 64 slots 6.1 and 6.4 us, 500 10.1 and 6.8, 24000 21.1 and 18.5; six of 500
// (C = 8) 10.6 and 8.1, ten of 400 (C = 4) 10.6 and 8.4, 25 of 400 (C = 2) 12.4 and 10.9; beyond the limits one
// cluster an item loses: ragged 80 items to 1000 slots (C = 2) 12.4 and 15.4, 24 of 24000 (C = 8) 55 and 60.
template <typename S>
Grid split_grid(const PagedAttnParams& p) {
    // Blocks of q heads that read the same rows go abreast, so that all but the first find them in L2 (12 q heads
    // to each of 8 kv heads of 128 x f16, 64 sequences of 8192 slots: 642 us as items of their own, 503 us abreast).
    // Above 64 q heads a kv head's blocks are items one after another.
    const int blocks = (p.nh / p.nkv + kAttnHeads - 1) / kAttnHeads;
    const int abreast = blocks <= kMaxAbreast ? blocks : 1, serial = blocks / abreast;
    const int64_t units = static_cast<int64_t>(p.c.max_pages) * p.c.page_size / S::UK;  // of a full sequence
    const int64_t items = static_cast<int64_t>(p.c.n_seq) * p.nkv * blocks;
    for (int C = 8; C > 1 && units >= 6; C /= 2) {
        const int clusters = sure_clusters(S::kCtas, C);
        if (!((units <= (C == 8 ? 256 : 16 * C) && items <= clusters) || (C == 8 && items * 2 <= clusters))) continue;
        const int64_t useful = items * (units / (kMinShare * C) + 1);
        const int most = static_cast<int>(useful < clusters ? useful : clusters);
        return {most / abreast * abreast * C, C, abreast, serial};
    }
    return {kSms * S::kCtas / abreast * abreast, 1, abreast, serial};
}

template <typename S, int C>
cudaError_t launch_split_t(const PagedAttnParams& p, const Grid& g, cudaStream_t stream) {
    auto kernel = paged_attn_split_kernel<typename S::Type, S::kHd, C>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(g.ctas), S::kThreads, S::kSmem, stream, C, p, g.abreast, g.serial);
}

template <typename S>
cudaError_t launch_split(const PagedAttnParams& p, cudaStream_t stream) {
    const Grid g = split_grid<S>(p);
    switch (g.cluster) {
        case 8: return launch_split_t<S, 8>(p, g, stream);
        case 4: return launch_split_t<S, 4>(p, g, stream);
        case 2: return launch_split_t<S, 2>(p, g, stream);
        default: return launch_split_t<S, 1>(p, g, stream);
    }
}

// fn of the split kernel's instance for the cache.
template <typename Fn>
auto with_split(const PagedAttnParams& p, Fn fn) {
    if (p.kv_f16)
        return p.hd <= 64 ? fn(Split<uint16_t, 64>()) : p.hd <= 128 ? fn(Split<uint16_t, 128>()) : fn(Split<uint16_t, 256>());
    return p.hd <= 64 ? fn(Split<float, 64>()) : p.hd <= 128 ? fn(Split<float, 128>()) : fn(Split<float, 256>());
}

// Whether 16-byte copies can read the rows.
bool rows_of_16(const PagedAttnParams& p) {
    const int es = p.kv_f16 ? 2 : 4;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * es) | static_cast<uintptr_t>(p.hd * es);
    return (bits & 15u) == 0;
}

}  // namespace

void paged_attn_grid(const PagedAttnParams& p, int* ctas, int* cluster) {
    const Grid g = rows_of_16(p) ? with_split(p, [&](auto s) { return split_grid<decltype(s)>(p); })
                                 : Grid{p.c.n_seq * p.nh, 1, 1, 1};
    *ctas = g.ctas;
    *cluster = g.cluster;
}

cudaError_t launch_paged_attn(const PagedAttnParams& p, cudaStream_t stream) {
    const cudaError_t e =
        rows_of_16(p) ? with_split(p, [&](auto s) { return launch_split<decltype(s)>(p, stream); })
                      : launch_dependent(paged_attn_any_kernel, dim3(p.c.n_seq * p.nh), kAnyThreads, 0, stream, 1, p);
    if (e != cudaSuccess || !p.add_weight) return e;
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    // a span for each CTA, up to 4096 CTAs or so; longer sequences loop
    const int64_t spans = (cap + kWeightSpan - 1) / kWeightSpan + 1;  // + 1: a window may begin inside one
    const int64_t most = 4096 / (static_cast<int64_t>(p.c.n_seq) * p.nkv) + 1;
    const int chunks = static_cast<int>(spans < most ? spans : most);
    return launch_dependent(paged_attn_weight_kernel, dim3(p.c.n_seq * p.nkv * chunks), kWeightThreads, 0, stream, 1, p, chunks);
}

cudaError_t paged_attn_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
