// Attention of many q rows over a paged f16 cache on the 5th-generation tensor cores (qkv_prompt_attn_step, and the prefix of
// qkv_prefix_attn_step; include/qkv.h has the contracts).
//
// s_j = scale * q.K_j, running maximum m and sum l of each row, out = sum p_j V_j / l, scores in log2 terms.  128 q rows (the
// rows of a tcgen05.mma) go over blocks of 128 slots: S = Q K^T and O += P V with both accumulators in tensor memory, 128
// columns each.  P, in f16, takes the place of S there and is the second product's A operand.  While the softmax is at one
// block, the tensor cores work on another:
//   out BF16          a tile has 256 rows in two streams of 128, each with S and O of its own; K and V are read once for both
//   out F32, "SPLIT"  a tile has 128 rows, one stream, whose S is there twice: a block's scores are made during the softmax of
//                     the last one's
// SPLIT, q is kept as the sum of two f16 (rounded, and the remainder rounded), so are the weights, both
// products are made twice, and 22 bits of each are kept.  For out BF16 everything is rounded once, by 2^-11 at most, which adds
// 4e-4 to the 1.7e-3 that out's rounding takes (scores of standard deviation 2) and halves the time (8191 tokens of 10 heads over 2:
// 168 us and 316).  q is scaled by a power of two for each row, into [2^13, 2^14); the weights are 2^(s - m + kShift), m
// being the maximum or up to some 2^9 below it.
//   warps 0-3, 4-7   softmax: S out of tensor memory, P back into it, O rescaled where the maximum has to move; at the end O / l
//                    to memory.  A row a thread of a stream each, P in two halves so that its product begins early; SPLIT: a
//                    row is two threads', of warps w and w + 4 and of 64 columns each, which meet at barriers of their own.
//   warp 8           issues the MMAs; 9 copies q; 10 and 11 only fill up the warpgroup
//   warps 12-15      copy K and V into a ring of chunks of 128 slots x 64 columns in the 128-byte swizzle that the MMA reads.
//                    Pages of a multiple of 8 slots: 12 asks for boxes of a page's rows by TMA, 13-15 hand them on and
//                    look at V where that is needed.  Others: all four by cp.async, a row at a time.
// An MMA of 128 x 128 x 16 takes 64 cycles, so a block of 128 rows takes 1024, and 2048 SPLIT.  What it takes in fact: 1800 for
// 8191 new tokens of 40 heads over 8 (507 us; the tensor pipe is busy for 59 % of them), by the chain of a stream's S, softmax
// (of which twice 230 cycles bring the scores, 600 make the weights, 270 hand them on) and products; SPLIT about 3800 for 96
// rows over 32704 slots (80 us, 49 %), by the same chain and the warp that asks for copies.  A CTA's first piece begins some
// 20000 cycles late: its instructions are in no cache yet.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cstring>

#include "paged_rows.cuh"

namespace {

using namespace qkv_rows;
using namespace qkv_ptx;

constexpr int kHalf = 128, kBlock = 128;
constexpr int kSoftWarps = 8, kMmaWarp = 8, kLoadWarp = 12, kLoadWarps = 4, kThreads = 32 * (kLoadWarp + kLoadWarps);
// Registers: 128 a thread at launch, of which the copying and issuing warpgroups give up what the two with a row of scores
// in registers take: 2 * 128 * (72 + 184) = 512 * 128.
constexpr int kLaunchRegs = 128, kFewRegs = 72, kManyRegs = 184;
static_assert(2 * 128 * (kFewRegs + kManyRegs) <= kThreads * kLaunchRegs, "registers");
constexpr int kChunkBytes = kBlock * 128;  // 128 slots (or q rows) x 64 columns
constexpr unsigned int kFlagTimeout = 2u;
// Named barriers: 1 to 4 of pairs of warps, then one for each stream's warps that have rows, and one for all of its warps.
constexpr int kStreamBarrier = 5, kEndBarrier = 7;
constexpr int kFailEnd = 1, kFailOneOfTwo = 2;  // p.fail
constexpr int kControlBytes = 2560;  // barriers and small tables, behind the chunks
// Weights are kept times 2^kShift; the maximum moves where 64 of a row are together above kMostWeight (64 times the
// largest are not).
constexpr float kMostWeight = 60000.f;
constexpr int kFold = 2;       // SPLIT: blocks that are summed in one accumulator before it is added to the others' sum
// out BF16: blocks of a piece, whose sums are added to those of the tile's pieces before it.  One accumulator for 262144
// slots of values above zero made results 1e-3 too small, as much as the rounding to bf16 is off; 32768 slots lose 1.3e-4.
constexpr int kMostBlocks = 256;
// Units that a tile's beginning and end take for 128 rows.  (0, 3 and 6 gave 71, 60 and 65 us for 32 sequences of four tokens;
// 0, 3 and 5 of them 679, 550 and 566 for 8191 tokens, whose tiles have twice as many rows.)
constexpr int kTileCost = 3;
constexpr int kMaxStages = 12, kPoisonRing = 16, kLiveRing = 8;

template <bool SPLIT, int NCH>  // NCH chunks of 64 columns a head
struct Shape {
    static constexpr int kQChunks = 2 * NCH;  // two streams, or two parts
    // (even: a head's chunks are neighbours)
    static constexpr int kStages = 14 - kQChunks < kMaxStages ? 14 - kQChunks : kMaxStages;
    // Copies in flight ahead of the one that is waited for (cp.async).  The MMAs free a block's V only after the next
    // block's K is there, so that many chunks must fit behind those in flight.
    static constexpr int kLag = kStages - 2 * NCH > 5 ? 5 : kStages - 2 * NCH;
    static constexpr float kShift = SPLIT ? 9.f : 6.f;  // SPLIT: remainders of weights 2^-10 of the largest keep 23 bits
    static constexpr int kControlAt = (kQChunks + kStages) * kChunkBytes, kSmem = kControlAt + kControlBytes;
    static_assert(kSmem <= 227 * 1024 && kStages % 2 == 0 && kStages % NCH == 0, "shared memory");
};

// ---------------------------------------------------------------- tcgen05

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// One lane of a warp whose lanes are all here.  The warp that issues MMAs runs as a whole and elects for each instruction, so
// that the compiler knows all operands to be the same in its lanes, as the instructions want them (issued by `if (lane == 0)`,
// an MMA took about 100 cycles to issue instead of the 64 that it runs).
__device__ __forceinline__ bool elect() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
    if (elect())
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Shared-memory descriptors of chunks of 128-byte rows in the 128-byte swizzle (eight rows, 1024 bytes, an atom; version 1,
// layout type 2).  K-major (Q, K): the stride offset leads to the next eight rows, the leading one is not used.
// MN-major (V: rows are slots, the summed dimension): the stride offset leads to the next eight slots, the leading one
// to the next 64 columns, a chunk further.
// The upper halves are the same; these are the lower ones, which grow by 1 for 16 bytes.
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr & 0x3FFFFu) >> 4 | 1u << 16; }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) {
    return (addr & 0x3FFFFu) >> 4 | static_cast<uint32_t>(kChunkBytes >> 4) << 16;
}
// kind::f16, D f32, A and B f16, M = 128; bit 16: B is MN-major.
__device__ __forceinline__ uint32_t idesc(int n, bool b_mn) {
    return 1u << 4 | (b_mn ? 1u << 16 : 0u) | static_cast<uint32_t>(n >> 3) << 17 | static_cast<uint32_t>(kHalf >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accumulate) {
    if (elect())
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(accumulate),
                     "r"(kDescHigh)
                     : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t id, uint32_t accumulate) {
    if (elect())
        asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
                     "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(id), "r"(accumulate),
                     "r"(kDescHigh)
                     : "memory");
}
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap* map, int col, int row, int page, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(row), "r"(page), "r"(smem_u32(bar))
        : "memory");
}

// N consecutive columns of this warp's 32 lanes: thread l has lane l's.
__device__ __forceinline__ void tm_ld32(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
          "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}
__device__ __forceinline__ void tm_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
          "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
__device__ __forceinline__ void tm_st16(uint32_t a, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(a),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tm_st32(uint32_t a, const uint32_t (&r)[32]) {
    uint32_t x[16];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] = r[16 * i + k];
        tm_st16(a + 16 * i, x);
    }
}
__device__ __forceinline__ uint32_t tm_ld1(uint32_t a) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(a));
    tc_wait_ld();
    return r;
}
__device__ __forceinline__ void tm_st1(uint32_t a, uint32_t r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(a), "r"(r) : "memory");
}

// As mbar_wait_bounded, without asking to be suspended: these waits are short, and there are many.  Some last for a whole
// piece or, where a stream has no rows in the pieces before, for several; so the limit counts from when the CTA last asked
// for a block, which *moved holds (and blocks come to an end).  Nothing is kept of a wait's own beginning: code that is
// inlined at every wait costs time (noting when it began and what *moved was then: 2.5 % of all calls).
__device__ __forceinline__ uint32_t now_ns() { return static_cast<uint32_t>(globaltimer_ns()); }
__device__ __forceinline__ bool wait_moving(uint64_t* bar, uint32_t parity, const uint32_t* moved, int32_t limit_ns) {
    const uint32_t at = smem_u32(bar);
    for (int i = 0;; ++i) {
        uint32_t ok;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(ok) : "r"(at), "r"(parity) : "memory");
        if (ok) return true;
        if ((i & 63) == 63) {
            const uint32_t now = now_ns();  // (what is read after it may be later)
            if (static_cast<int32_t>(now - *static_cast<const volatile uint32_t*>(moved)) > limit_ns) return false;
        }
    }
}

// ---------------------------------------------------------------- arithmetic

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
using u64 = unsigned long long;
__device__ __forceinline__ u64 pack2(float x, float y) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack2(u64 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ u64 fma2(u64 x, u64 y, u64 z) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
__device__ __forceinline__ u64 add2(u64 x, u64 y) {
    u64 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ u64 mul2(u64 x, u64 y) {
    u64 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
    return r;
}
__device__ __forceinline__ void scale16(uint32_t at, float by) {
    uint32_t o[16];
    tm_ld16(at, o);
    tc_wait_ld();
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * by);
    tm_st16(at, o);
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
// Two values rounded to f16, and the remainders rounded to f16.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    hi = f16x2(a, b);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    lo = f16x2(a - f.x, b - f.y);
}
// Byte offset of 16 bytes of a 128-byte row within a chunk.
__device__ __forceinline__ uint32_t swz(int row, int c16) { return row * 128 + ((c16 ^ (row & 7)) << 4); }

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool finite_f16x2(uint32_t w) {
    return (w & 0x7c00u) != 0x7c00u && (w & 0x7c000000u) != 0x7c000000u;
}

__device__ __forceinline__ bool finite_f16x8(const uint4& v) {
    return finite_f16x2(v.x) && finite_f16x2(v.y) && finite_f16x2(v.z) && finite_f16x2(v.w);
}
// The kinds of eight values of f16: bit j of the low byte for +inf in value j, of the next -inf, of the third NaN.
__device__ __forceinline__ uint32_t kinds_of(const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t r = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t h = w[j >> 1] >> (16 * (j & 1));
        if ((h & 0x7c00u) == 0x7c00u) r |= ((h & 0x3ffu) != 0 ? 0x10000u : (h & 0x8000u) != 0 ? 0x100u : 1u) << j;
    }
    return r;
}

// SPLIT: scores of 64 slots from `slot0` on, in tensor memory at `at`, of which some are NaN in some rows.  For K with infinities
// the products with the two parts of q need not be those with q (0 * inf where the remainder is zero), so those
// scores are made anew: an infinity of that sign, or NaN where K or q have one, signs differ or q has a zero there.  A
// warp reads K of all slots together, 8 bytes a lane; a lane looks at its own row's q only where K is infinite.  q_row:
// null for rows that have no say; seen: slots that the row sees.  (One such slot costs next to nothing, an infinity in
// every slot of 40000 20 to 30 times the call's time; each score by its own thread from memory took a millisecond a block.)
__device__ __noinline__ void mend_scores(const PagedRowsParams& p, uint32_t at, const float* q_row, int seq, int kv, int slot0,
                                         uint32_t seen0, uint32_t seen1) {
    const int lane = threadIdx.x & 31;
    const bool mine = q_row != nullptr;
    const uint32_t any0 = __reduce_or_sync(0xffffffffu, mine ? seen0 : 0u), any1 = __reduce_or_sync(0xffffffffu, mine ? seen1 : 0u);
    const int64_t off0 = (any0 >> lane) & 1u ? row_offset(p.c, seq, slot0 + lane) : -1;
    const int64_t off1 = (any1 >> lane) & 1u ? row_offset(p.c, seq, slot0 + 32 + lane) : -1;
    const __half* pool = static_cast<const __half*>(p.c.k) + static_cast<int64_t>(kv) * p.hd + 4 * lane;
#pragma unroll 1
    for (int k0 = 0; k0 < 64; k0 += 8) {
        uint2 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int64_t o = __shfl_sync(0xffffffffu, k0 < 32 ? off0 : off1, (k0 + k) & 31);
            w[k] = make_uint2(0u, 0u);
            if (o >= 0 && 4 * lane < p.hd) w[k] = __ldg(reinterpret_cast<const uint2*>(pool + o));
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            uint32_t lanes = __ballot_sync(0xffffffffu, !finite_f16x2(w[k].x) || !finite_f16x2(w[k].y));
            if (!lanes) continue;  // q is at fault
            float f = __uint_as_float(tm_ld1(at + k0 + k));
            const bool need = mine && f != f && (((k0 < 32 ? seen0 : seen1) >> ((k0 + k) & 31)) & 1u);
            bool plus = false, minus = false, nan = false;
            for (; lanes; lanes &= lanes - 1) {
                const int l = __ffs(lanes) - 1;
                const uint32_t x = __shfl_sync(0xffffffffu, w[k].x, l), y = __shfl_sync(0xffffffffu, w[k].y, l);
                for (int j = 0; j < 4; ++j) {
                    const uint32_t h = (j < 2 ? x : y) >> (16 * (j & 1));
                    if (!need || (h & 0x7c00u) != 0x7c00u) continue;
                    const float q = __ldcg(q_row + 4 * l + j);
                    if ((h & 0x3ffu) != 0 || !(fabsf(q) > 0.f) || p.scale == 0.f) nan = true;
                    else if ((q < 0.f) != (p.scale < 0.f) != ((h & 0x8000u) != 0)) minus = true;
                    else plus = true;
                }
                if (__all_sync(0xffffffffu, !need || nan || (plus && minus))) break;
            }
            if (need && !nan && plus != minus) f = plus ? CUDART_INF_F : -CUDART_INF_F;
            __syncwarp();
            tm_st1(at + k0 + k, __float_as_uint(f));
        }
    }
}

// 16 bytes of values of es bytes, to any address of such values.
__device__ __noinline__ void store_any(char* to, uint4 v, int es) {
    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
    for (int j = 0; j < 16; j += es) {
        const uint32_t x = j < 4 ? e[0] : j < 8 ? e[1] : j < 12 ? e[2] : e[3];
        if (es == 2) *reinterpret_cast<uint16_t*>(to + j) = static_cast<uint16_t>(x >> (8 * (j & 3)));
        else *reinterpret_cast<uint32_t*>(to + j) = x;
    }
}
__device__ __forceinline__ void store16(char* to, uint4 v, int es) {
    if ((reinterpret_cast<uintptr_t>(to) & 15u) == 0) *reinterpret_cast<uint4*>(to) = v;
    else store_any(to, v, es);
}

// Whether `yes` holds in any lane of the two softmax warps that have the same rows; they meet here.
__device__ __forceinline__ bool pair_any(int quarter, bool yes) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(static_cast<uint32_t>(yes)), "r"(1 + quarter) : "memory");
    return any != 0;
}

// Whether `yes` holds in any lane of `warps` warps, which meet here.
__device__ __forceinline__ bool stream_any(int barrier, int warps, bool yes) {
    uint32_t any;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, %2, %3, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(any) : "r"(static_cast<uint32_t>(yes)), "r"(barrier), "r"(32 * warps) : "memory");
    return any != 0;
}

struct Control {
    uint64_t landed[kMaxStages], full[kMaxStages], empty[kMaxStages];
    uint64_t q_ready[2], q_free[2], s_full[2], p_half[2], half_done[2], p_ready[2], o_full[2], pv_done, o_free, drained;
    uint32_t live[kLiveRing][4];   // slots of a block that are there
    uint32_t poison[kPoisonRing];  // n: in piece n, V had infinities or NaN that were replaced
    float top[2][kHalf];           // SPLIT: of the rows, by side
    bool grow[2][kHalf];           // whether a row's maximum is to be looked for
    uint32_t moved;                // when a block was last asked for, in ns
    uint32_t tmem;
};
static_assert(sizeof(Control) <= kControlBytes, "control");

// 16 bytes of V, zeros in the place of infinities and NaN.
__device__ __forceinline__ void keep_finite(uint32_t at, uint32_t (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if ((v[j] & 0x7c00u) == 0x7c00u) v[j] &= 0xffff0000u;
        if ((v[j] & 0x7c000000u) == 0x7c000000u) v[j] &= 0x0000ffffu;
    }
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}
__device__ __forceinline__ bool clean16(uint32_t at) {
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(at) : "memory");
    if (finite_f16x2(v[0]) && finite_f16x2(v[1]) && finite_f16x2(v[2]) && finite_f16x2(v[3])) return false;
    keep_finite(at, v);
    return true;
}

// What the infinities and NaN of V that a row sees in slots [lo, hi) make of its result.  The products do not tell: a
// weight of zero (of a slot that the row does not see; or rounded, or a remainder) times them is NaN.  So blocks with
// slots that only some rows see get zeros in their place, and where any row of a stream came out infinite or NaN, or had
// such zeros, the stream's `warps` warps that have rows look here, together: each reads every warps-th 32 slots of V, 16 bytes a
// lane, and notes kind and column of what it finds, once for all rows where all see the slot and else for each row that
// does; then every row takes its own.  A row's span is empty where it takes no part; SPLIT, a row's two threads have the
// columns of every other 16.  8191 tokens of 10 heads over 2 with one infinity in an early slot take 0.36 ms instead of 0.17, out
// F32 0.57 instead of 0.32.  (A search by each row for itself, a value at a time, would take a second for 32768 slots.)
constexpr int kKindWords = 3 * 128 / 32, kCommon = kHalf;  // of a row: a bit for each kind and column
constexpr int kSpansAt = 4 * (kHalf + 1) * kKindWords;
static_assert(kSpansAt % 16 == 0 && kSpansAt + kHalf * sizeof(int2) <= kChunkBytes, "what the rows' warps leave each other");
template <bool SPLIT, int NCH>
__device__ __noinline__ void mend_rows(const PagedRowsParams& p, int warps, int seq, int kv, int lo, int hi, char* to, int es) {
    extern __shared__ __align__(1024) unsigned char smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = SPLIT ? 0 : warp >> 2, side = SPLIT ? warp >> 2 : -1, row = 32 * (warp & 3) + lane;
    const int rows = SPLIT ? 16 * warps : 32 * warps, rank = SPLIT ? (warp & 3) + side * (warps / 2) : warp & 3;
    const int barrier = kStreamBarrier + t;
    unsigned char* scratch = smem + t * NCH * kChunkBytes;  // q's place
    uint32_t* kinds = reinterpret_cast<uint32_t*>(scratch);
    int2* spans = reinterpret_cast<int2*>(scratch + kSpansAt);
    volatile uint32_t* moved = &reinterpret_cast<Control*>(smem + Shape<SPLIT, NCH>::kControlAt)->moved;
    const bool live = lo < hi;
    if (side <= 0) {  // (a row's two sides see the same)
        spans[row] = make_int2(lo, hi);
        for (int k = 0; k < kKindWords; ++k) kinds[row * kKindWords + k] = 0;
        if (row < kKindWords) kinds[kCommon * kKindWords + row] = 0;
    }
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
    int from = 0x7fffffff, to_all = 0x7fffffff, from_all = 0, end = 0;  // slots that any row sees, and that all do
    for (int r = lane; r < rows; r += 32) {
        const int2 s = spans[r];
        if (s.x >= s.y) continue;
        from = min(from, s.x), from_all = max(from_all, s.x), to_all = min(to_all, s.y), end = max(end, s.y);
    }
    from = __reduce_min_sync(0xffffffffu, from), from_all = __reduce_max_sync(0xffffffffu, from_all);
    to_all = __reduce_min_sync(0xffffffffu, to_all), end = __reduce_max_sync(0xffffffffu, end);
    constexpr int kLanes = 8 * NCH, kSlots = 32 / kLanes, kLoads = 32 / kSlots;  // of a slot; slots of a load; loads of 32 slots
    const int c = lane % kLanes, which = lane / kLanes;
    const bool has = 8 * c < p.hd;
    const uint4* v0 = reinterpret_cast<const uint4*>(static_cast<const __half*>(p.c.v) + static_cast<int64_t>(kv) * p.hd + (has ? 8 * c : 0));
    auto ask = [&](int at) { return at + lane < end ? page_ref(p.c, seq, at + lane) : PageRef{0, -1}; };
    uint32_t common = 0;
    if (end > 0) {
        from += 32 * rank;
        PageRef asked = ask(from);
        for (; from < end; from += 32 * warps) {
            const int64_t off = asked.in_page >= 0 ? row_offset(p.c, asked) : -1;
            asked = ask(min(from, end) + 32 * warps);
            if (lane == 0) *moved = now_ns();
            uint4 v[kLoads];
            bool clean = true;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int64_t o = __shfl_sync(0xffffffffu, off, kSlots * k + which);
                v[k] = make_uint4(0u, 0u, 0u, 0u);
                if (o >= 0 && has) v[k] = __ldg(v0 + o / 8);
            }
#pragma unroll
            for (int k = 0; k < kLoads; ++k) clean = clean && finite_f16x8(v[k]);
            if (__all_sync(0xffffffffu, clean)) continue;
#pragma unroll
            for (int k = 0; k < kLoads; ++k) {
                const int slot = from + kSlots * k + which;
                uint32_t found = finite_f16x8(v[k]) ? 0u : kinds_of(v[k]);
                if (slot >= from_all && slot < to_all) {
                    common |= found;
                    found = 0;
                }
                for (uint32_t lanes = __ballot_sync(0xffffffffu, found != 0); lanes; lanes &= lanes - 1) {
                    const int l = __ffs(lanes) - 1, at = l % kLanes, s = from + kSlots * k + l / kLanes;
                    const uint32_t f = __shfl_sync(0xffffffffu, found, l);
                    for (int r = lane; r < rows; r += 32) {
                        const int2 see = spans[r];
                        if (s < see.x || s >= see.y) continue;
                        for (int kind = 0; kind < 3; ++kind)
                            if ((f >> (8 * kind)) & 255u)
                                atomicOr(&kinds[r * kKindWords + 4 * kind + (at >> 2)], ((f >> (8 * kind)) & 255u) << (8 * (at & 3)));
                    }
                }
            }
        }
    }
    for (int kind = 0; kind < 3; ++kind)
        if ((common >> (8 * kind)) & 255u)
            atomicOr(&kinds[kCommon * kKindWords + 4 * kind + (c >> 2)], ((common >> (8 * kind)) & 255u) << (8 * (c & 3)));
    asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(32 * warps) : "memory");
    if (!live) return;
    for (int w = 0; 32 * w < p.hd; ++w) {
        uint32_t any[3];
        for (int kind = 0; kind < 3; ++kind) any[kind] = kinds[row * kKindWords + 4 * kind + w] | kinds[kCommon * kKindWords + 4 * kind + w];
        for (uint32_t left = any[0] | any[1] | any[2]; left; left &= left - 1) {
            const int b = __ffs(left) - 1, d = 32 * w + b;
            if (side >= 0 && ((d >> 4) & 1) != side) continue;
            const bool plus = (any[0] >> b) & 1u, minus = (any[1] >> b) & 1u, nan = ((any[2] >> b) & 1u) || (plus && minus);
            const uint32_t bits = nan ? 0x7fc00000u : plus ? 0x7f800000u : 0xff800000u;
            if (es == 2) reinterpret_cast<uint16_t*>(to)[d] = static_cast<uint16_t>(bits >> 16);
            else reinterpret_cast<uint32_t*>(to)[d] = bits;
        }
    }
}

// out BF16: to a row's sums (of V in tensor memory, l) and maximum, those of the tile's pieces before this one, which are where
// its part would be.  The warp's lanes together.
__device__ __noinline__ float2 add_before(const PagedRowsParams& p, float* part, int row, uint32_t o_at, float m, float l, bool mine) {
    const float2 ml = mine ? *part_ml(part, row) : make_float2(-CUDART_INF_F, 0.f);
    const float4* sum = reinterpret_cast<const float4*>(part_o(p, part, row));
    const float top = fmaxf(m, ml.x), keep = m == top ? 1.f : ex2(m - top), f = ml.x == top ? 1.f : ex2(ml.x - top);
    for (int c = 0; c < p.hd; c += 16) {
        uint32_t v[16];
        tm_ld16(o_at + c, v);
        tc_wait_ld();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float4 y = mine ? sum[c / 4 + k] : make_float4(0.f, 0.f, 0.f, 0.f);
            v[4 * k] = __float_as_uint(fmaf(y.x, f, __uint_as_float(v[4 * k]) * keep));
            v[4 * k + 1] = __float_as_uint(fmaf(y.y, f, __uint_as_float(v[4 * k + 1]) * keep));
            v[4 * k + 2] = __float_as_uint(fmaf(y.z, f, __uint_as_float(v[4 * k + 2]) * keep));
            v[4 * k + 3] = __float_as_uint(fmaf(y.w, f, __uint_as_float(v[4 * k + 3]) * keep));
        }
        tm_st16(o_at + c, v);
    }
    tc_wait_st();
    return make_float2(top, fmaf(ml.y, f, l * keep));
}

template <bool SPLIT, int NCH>
__global__ void __launch_bounds__(kThreads, 1)
    paged_rows_tc_kernel(const __grid_constant__ PagedRowsParams p, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_ql, int box) {
    using S = Shape<SPLIT, NCH>;
    constexpr float kShift = S::kShift;
    extern __shared__ __align__(1024) unsigned char smem[];  // atoms of the swizzle: no other shared memory before it
    Control& ctl = *reinterpret_cast<Control*>(smem + S::kControlAt);
    const uint32_t q_at = smem_u32(smem), ring_at = q_at + S::kQChunks * kChunkBytes;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    constexpr int kParts = SPLIT ? 2 : 1;
    // chunk c of part `part` (0: rounded, 1: remainder) of stream t's q
    auto q_chunk = [&](int t, int part, int c) { return q_at + (((SPLIT ? 0 : t) * kParts + part) * NCH + c) * kChunkBytes; };
    auto chunk_at = [&](uint32_t n) { return ring_at + n % S::kStages * kChunkBytes; };
    auto wait_for = [&](uint64_t* bar, uint32_t parity) { return wait_moving(bar, parity, &ctl.moved, p.wait_limit_ns); };
    auto note_moved = [&]() { *static_cast<volatile uint32_t*>(&ctl.moved) = now_ns(); };

    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&ctl.tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    if (tid < kPoisonRing) ctl.poison[tid] = 0;
    if (tid == 0) {
        ctl.moved = now_ns();
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(&ctl.landed[s], 1);
            mbar_init(&ctl.full[s], box ? kLoadWarps - 1 : kLoadWarps);
            mbar_init(&ctl.empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            mbar_init(&ctl.q_ready[t], 1);
            mbar_init(&ctl.q_free[t], SPLIT ? 8 : 4);
            mbar_init(&ctl.s_full[t], 1);
            mbar_init(&ctl.p_half[t], 4);
            mbar_init(&ctl.half_done[t], 1);
            mbar_init(&ctl.p_ready[t], 4);
            mbar_init(&ctl.o_full[t], 1);
        }
        mbar_init(&ctl.pv_done, 1);
        mbar_init(&ctl.o_free, 8);
        mbar_init(&ctl.drained, 1);
        mbar_fence_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ctl.tmem;
    griddep_wait();
    griddep_launch_dependents();
    if (tid == 0) note_moved();  // (what came before may have taken long)

    const int G = p.nh / p.nkv;
    Walk<SPLIT ? 0x7fffffff : kMostBlocks> w;
    Piece x;
    const bool work = w.begin(p);
    if (work && tid == 0) note_none(p);
    if (work) {
        if (warp < kSoftWarps) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        else asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    }
    if (work && warp < kSoftWarps) {
      if constexpr (SPLIT) {
        // ---- softmax, SPLIT: thread `lane` of warp w has row 32 (w % 4) + lane and columns 64 (w / 4) .. + 63 of every block; the
        // warps of a pair, w and w + 4, have the same rows
        const int quarter = warp & 3, side = warp >> 2;
        const uint32_t lanes_at = tmem + (static_cast<uint32_t>(32 * quarter) << 16), o_at = lanes_at + 256, sum_at = lanes_at + 384;
        uint32_t s_phase = 0, o_phase = 0;  // s_phase: bit t
        int piece = 0, block0 = 0;
        bool ok = true;
        // Block number `block`'s weights are in O; those of the block before it are known to be.
        auto wait_pv = [&](int block) {
            const bool there = __all_sync(0xffffffffu, wait_for(&ctl.pv_done, block & 1)) && (p.fail != kFailOneOfTwo || warp != 0);
            tc_fence_after();
            return there;
        };
        while (ok && w.next(p, x)) {
            const RowTile& tile = x.t;
            const int kv = x.head / p.blocks, g0 = (x.head - kv * p.blocks) * p.per_block, heads = min(p.per_block, G - g0);
            const int first_block = block0, n = x.to - x.from;
            block0 += n;
            ++piece;
            if (tid == 0) note_piece(p, w, x);
            const int r = 32 * quarter + lane, i = r / p.per_block, g = r - i * p.per_block;
            const int h_row = kv * G + g0 + g;
            const int64_t row = tile.row0 + i;
            const bool mine = i < tile.ntok && g < heads;
            const int busy_pairs = (tile.ntok * p.per_block + 31) / 32;
            const bool busy = quarter < busy_pairs;
            // The tensor cores cut bits off a score's sums too, each towards zero: 2^-23 of it are missing on average, and given
            // back here.  (Log sum exp over 4096 slots of normal numbers, heads of 16 to 128 columns: off by -0.8 to -1.4 times
            // 2^-23 of itself without, by -0.4 to 0.2 with it; where all products have one sign, by up to -2.2.)
            const float unscale = mine ? __ldcg(p.q_unscale + row * p.nh + h_row) * (1.f + 1.1920929e-7f) : 1.f;
            int see_lo = 0, see_hi = 0;
            if (mine) row_span(p, tile, i, see_lo, see_hi);
            float m = -CUDART_INF_F, l = 0.f;  // l: of this side's columns
            bool live_row = mine;              // a row that has come to NaN has no say any more
#pragma unroll 1
            for (int b = 0; b < n; ++b) {
                const int t = b & 1;
                ok = __all_sync(0xffffffffu, wait_for(&ctl.s_full[t], (s_phase >> t) & 1)) && ok;
                s_phase ^= 1u << t;
                tc_fence_after();
                if (busy) {
                    const uint32_t at = lanes_at + 128 * t + 64 * side;
                    const int j0 = tile.lo + (x.from + b) * kBlock;
                    const uint32_t* live = ctl.live[(first_block + b) % kLiveRing];
                    const bool mixed = j0 < tile.all_lo || j0 + kBlock > tile.all_hi ||
                                       (live[0] & live[1] & live[2] & live[3]) != 0xffffffffu;
                    // the slots of columns 32 c .. 32 c + 31 that the row sees
                    auto seen = [&](int c) {
                        const int a = see_lo - j0 - 32 * c, e = see_hi - j0 - 32 * c;
                        const uint32_t below = e >= 32 ? 0xffffffffu : e <= 0 ? 0u : (1u << e) - 1u;
                        const uint32_t from = a <= 0 ? 0xffffffffu : a >= 32 ? 0u : 0xffffffffu << a;
                        return below & from & live[c];
                    };
                    uint32_t v[2][32];
                    tm_ld32(at, v[0]);
                    tm_ld32(at + 32, v[1]);
                    tc_wait_ld();
                    float total;
                    // The weights are made with the maximum as it was.  Their sum tells whether that will do (none is then above
                    // f16's largest): the maximum itself is looked for only at first and where the sum has grown, by both
                    // warps of the pair.  Rows that are none (what is in q's place there varies) have no say.
#pragma unroll 1
                    for (int round = 0;; ++round) {
                        if (mixed) {
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                const uint32_t in = seen(2 * side + c);
#pragma unroll
                                for (int k = 0; k < 32; ++k)
                                    if (!((in >> k) & 1u)) v[c][k] = 0xff800000u;
                            }
                        }
                        // 2^(s - m) first: its argument is small where it counts, and so is its rounding
                        const float base = m == -CUDART_INF_F ? 0.f : m;
                        const u64 by = pack2(unscale, unscale), minus = pack2(-base, -base);
                        constexpr float kTimes = 512.f;  // 2^kShift
                        const u64 up = pack2(kTimes, kTimes);
                        u64 sum[2] = {0, 0};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t h[16], low[16];
#pragma unroll
                            for (int k = 0; k < 32; k += 2) {
                                const float2 y =
                                    unpack2(fma2(pack2(__uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1])), by, minus));
                                const u64 e = mul2(pack2(ex2(y.x), ex2(y.y)), up);
                                sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], e);
                                const float2 f = unpack2(e);
                                split2(f.x, f.y, h[k / 2], low[k / 2]);
                            }
                            tm_st16(at + 32 * c, h);
                            tm_st16(at + 32 * c + 16, low);
                        }
                        const float2 s2 = unpack2(add2(sum[0], sum[1]));
                        total = s2.x + s2.y;
                        const bool grow = live_row && (m == -CUDART_INF_F || !(total <= kMostWeight));
                        if (round == 2 || !pair_any(quarter, !ok || grow)) break;
                        if (pair_any(quarter, !ok)) {  // a wait ran out: both leave
                            ok = false;
                            break;
                        }
                        if (round == 0) {
                            const bool odd = __any_sync(0xffffffffu, live_row && total != total);
                            if (odd) {  // K with infinities, or NaN
                                const float* q_row = p.q + row * p.q_stride + static_cast<int64_t>(h_row) * p.hd;
#pragma unroll
                                for (int c = 0; c < 2; ++c) tm_st32(at + 32 * c, v[c]);
                                tc_wait_st();
                                mend_scores(p, at, live_row ? q_row : nullptr, tile.seq, kv, j0 + 64 * side, seen(2 * side), seen(2 * side + 1));
                                tc_wait_st();
                                tm_ld32(at, v[0]);
                                tm_ld32(at + 32, v[1]);
                                tc_wait_ld();
                            }
                            if (pair_any(quarter, odd)) continue;
                        }
                        float tops[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                        for (int k = 0; k < 32; k += 2)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                tops[c] = max3(tops[c], __uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1]));
                        const float top = fmaxf(tops[0], tops[1]) * unscale;
                        // (moved only where the row's own sums ask for it: its bits do not depend on what other rows see)
                        ctl.top[side][r] = top;
                        ctl.grow[side][r] = grow;
                        pair_any(quarter, false);
                        const float next = grow || ctl.grow[side ^ 1][r] ? fmaxf(m, fmaxf(top, ctl.top[side ^ 1][r])) : m;
                        const float keep = m == next ? 1.f : ex2(m - next);
                        m = next;
                        l *= keep;
                        if (b > 0) {
                            ok = wait_pv(first_block + b - 1) && ok;  // the weights before these are in O
#pragma unroll 1
                            for (int c = 16 * side; c < p.hd; c += 32) {
                                scale16(o_at + c, keep);
                                if (b > kFold) scale16(sum_at + c, keep);
                            }
                        }
                        tc_wait_st();
                        tc_fence_before();
                        // all of O is as it is to be before either side's weights go into it; and where one's wait ran out both
                        // leave, or the other would stay at the next barrier
                        ok = !pair_any(quarter, !ok);
                        round = 1;                 // the next one is the last
                    }
                    l += total;
                    live_row = live_row && total == total;
                    tc_wait_st();
                }
                if (!ok) break;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(side ? &ctl.p_ready[t] : &ctl.p_half[t]);
                // The tensor cores cut bits off every sum, always towards zero: 5e-6 of 4096 slots' sums in one accumulator
                // were lost.  So the sums of kFold blocks are added to the others' here, rounded to nearest.
                if (b > 0 && b % kFold == 0) {
                    if (busy) {
                        ok = wait_pv(first_block + b - 1);
#pragma unroll 1
                        for (int c = 16 * side; c < p.hd; c += 32) {
                            uint32_t o[16], y[16];
                            tm_ld16(o_at + c, o);
                            if (b > kFold) tm_ld16(sum_at + c, y);
                            tc_wait_ld();
                            if (b > kFold) {
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) + __uint_as_float(y[k]));
                            }
                            tm_st16(sum_at + c, o);
                        }
                        tc_wait_st();
                        tc_fence_before();
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl.o_free);
                }
            }
            // (not by pv_done, whose last phase but one may be under way or over: a barrier tells a phase only from the next)
            const bool there = ok && __all_sync(0xffffffffu, wait_for(&ctl.o_full[0], o_phase));
            o_phase ^= 1u;
            ok = !pair_any(quarter, !there);
            tc_fence_after();
            if (busy) {
                const bool put = mine && ok;  // (nothing is written where a wait ran out)
                float* to;
                const bool both = n > kFold;
                ctl.top[side][r] = l;
                pair_any(quarter, false);
                l += ctl.top[side ^ 1][r];
                const bool poison = ctl.poison[piece % kPoisonRing] == static_cast<uint32_t>(piece);
                const bool whole = w.whole(x), empty = see_lo >= see_hi;
                const float inv = !whole ? 1.f : empty ? 0.f : 1.f / l;  // (a row that sees nothing has sums of zero)
                float* part = part_of(p, blockIdx.x, x.first);
                if (!whole) to = part_o(p, part, r);
                else if (!p.first) to = p.prefix_out + (row * p.nh + h_row) * p.hd;
                else to = static_cast<float*>(p.out) + row * p.out_stride + static_cast<int64_t>(h_row) * p.hd;
                // through q's place, by rows of a warp; the sides take 16 columns in turn
                constexpr int kRowBytes = 64;  // of 32 rows: a round's
                const uint32_t stage = q_chunk(0, 0, 0) + warp * 32 * kRowBytes;
                float odd = 0.f;
#pragma unroll 1
                for (int c = 16 * side; c < p.hd; c += 32) {
                    uint32_t v[16], y[16];
                    tm_ld16(o_at + c, v);
                    if (both) tm_ld16(sum_at + c, y);
                    tc_wait_ld();
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        float o = __uint_as_float(v[k]);
                        if (both) o += __uint_as_float(y[k]);
                        o *= inv;
                        odd = fmaf(o, 0.f, odd);
                        v[k] = __float_as_uint(o);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * kRowBytes +
                                                                                      ((k ^ ((lane >> 1) & 3)) << 4)),
                                     "r"(v[4 * k]), "r"(v[4 * k + 1]), "r"(v[4 * k + 2]), "r"(v[4 * k + 3])
                                     : "memory");
                    __syncwarp();
                    // four lanes a row
#pragma unroll
                    for (int k = 0; k < 32; k += 8) {
                        const int from = k + (lane >> 2);
                        char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<u64>(to), from)) + 4 * c +
                                    16 * (lane & 3);
                        const bool has = __shfl_sync(0xffffffffu, put, from);
                        uint4 w4;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w4.x), "=r"(w4.y), "=r"(w4.z), "=r"(w4.w)
                                     : "r"(stage + from * kRowBytes + (((lane & 3) ^ ((from >> 1) & 3)) << 4))
                                     : "memory");
                        if (has) store16(dst, w4, 4);
                    }
                    __syncwarp();
                }
                if (put && side == 0) {
                    float* lse = p.first ? p.lse : p.prefix_lse;
                    if (!whole) *part_ml(part, r) = make_float2(m - kShift, l);
                    else if (lse) lse[row * p.nh + h_row] = lse_of(m - kShift, l, empty);
                }
                const bool live = put && l > 0.f;
                // (a sum of weights that is NaN makes all of the row NaN already)
                if (stream_any(kStreamBarrier, 2 * busy_pairs, live && (poison || !(odd == 0.f))))
                    mend_rows<SPLIT, NCH>(p, 2 * busy_pairs, tile.seq, kv, live ? max(see_lo, tile.lo + x.from * kBlock) : 0,
                                          live ? min(see_hi, tile.lo + x.to * kBlock) : 0, reinterpret_cast<char*>(to), 4);
                tc_fence_before();
            }
            // all warps come here, whatever became of their waits, and leave together
            if (stream_any(kEndBarrier, kSoftWarps, !ok)) {
                ok = false;
                break;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_free[0]);
        }
        if (!ok && lane == 0) flag_bad(kFlagTimeout, 0);
      } else {
        // ---- softmax: thread `lane` of warp w has row 32 (w % 4) + lane of stream w / 4
        const int t = warp >> 2, quarter = warp & 3;
        const uint32_t s_at = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + 128 * t, o_at = s_at + 256;
        uint32_t s_phase = 0, o_phase = 0;
        int piece = 0, block0 = 0;
        bool ok = true;
        while (ok && w.next(p, x)) {
            const RowTile& tile = x.t;
            const int kv = x.head / p.blocks, g0 = (x.head - kv * p.blocks) * p.per_block, heads = min(p.per_block, G - g0);
            const int first_block = block0;
            block0 += x.to - x.from;
            ++piece;
            if (tid == 0) note_piece(p, w, x);
            const int token0 = t * p.part_tokens;  // the stream's first
            if (token0 >= tile.ntok) continue;                  // nothing for this stream
            const int r = 32 * quarter + lane, in_part = r / p.per_block, g = r - in_part * p.per_block;
            const int i = token0 + in_part, row = tile.row0 + i, h_row = kv * G + g0 + g;
            const bool mine = in_part < p.part_tokens && i < tile.ntok && g < heads;
            const int busy_warps = (min(p.part_tokens, tile.ntok - token0) * p.per_block + 31) / 32;
            const bool busy = quarter < busy_warps;
            const float unscale = mine ? __ldcg(p.q_unscale + static_cast<int64_t>(row) * p.nh + h_row) : 1.f;
            int see_lo = 0, see_hi = 0;
            if (mine) row_span(p, tile, i, see_lo, see_hi);
            float m = -CUDART_INF_F, l = 0.f;
            bool live_row = mine;  // a row that has come to NaN has no say any more
            for (int u = x.from; u < x.to; ++u) {
                ok = __all_sync(0xffffffffu, wait_for(&ctl.s_full[t], s_phase));
                s_phase ^= 1;
                if (!ok) break;
                tc_fence_after();
                const int j0 = tile.lo + u * kBlock;
                const uint32_t* live = ctl.live[(first_block + u - x.from) % kLiveRing];
                const bool mixed = j0 < tile.all_lo || j0 + kBlock > tile.all_hi ||
                                   (live[0] & live[1] & live[2] & live[3]) != 0xffffffffu;
                // the slots of columns 32 c .. 32 c + 31 that the row sees
                auto seen = [&](int c) {
                    const int a = see_lo - j0 - 32 * c, b = see_hi - j0 - 32 * c;
                    const uint32_t below = b >= 32 ? 0xffffffffu : b <= 0 ? 0u : (1u << b) - 1u;
                    const uint32_t from = a <= 0 ? 0xffffffffu : a >= 32 ? 0u : 0xffffffffu << a;
                    return below & from & live[c];
                };
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    if (busy) {
                        const uint32_t at = s_at + 64 * half;
                        float total;
                        uint32_t v[2][32];
                        tm_ld32(at, v[0]);
                        tm_ld32(at + 32, v[1]);
                        tc_wait_ld();
                        // The weights are made with the maximum as it was.  Their sum tells whether that will do (none is then
                        // above f16's largest): the maximum itself is looked for only at first and where the sum has grown.
                        // Rows that are none (what is in q's place there varies) have no say in the warp's votes.
#pragma unroll 1
                        for (int round = 0;; ++round) {
                            if (mixed) {
#pragma unroll
                                for (int c = 0; c < 2; ++c) {
                                    const uint32_t in = seen(2 * half + c);
#pragma unroll
                                    for (int k = 0; k < 32; ++k)
                                        if (!((in >> k) & 1u)) v[c][k] = 0xff800000u;
                                }
                            }
                            const float base = (m == -CUDART_INF_F ? 0.f : m) - kShift;
                            const u64 by = pack2(unscale, unscale), minus = pack2(-base, -base);
                            u64 sum[2] = {0, 0};
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                uint32_t h[16];
#pragma unroll
                                for (int k = 0; k < 32; k += 2) {
                                    const float2 y =
                                        unpack2(fma2(pack2(__uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1])), by, minus));
                                    const float a = ex2(y.x), b = ex2(y.y);
                                    sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pack2(a, b));
                                    h[k / 2] = f16x2(a, b);
                                }
                                tm_st16(at + 32 * c, h);
                            }
                            const float2 s2 = unpack2(add2(sum[0], sum[1]));
                            total = s2.x + s2.y;
                            const bool grow = live_row && (m == -CUDART_INF_F || !(total <= kMostWeight));
                            if (round == 2 || !__any_sync(0xffffffffu, grow)) break;
                            float tops[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
                            for (int k = 0; k < 32; k += 2)
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    tops[c] = max3(tops[c], __uint_as_float(v[c][k]), __uint_as_float(v[c][k + 1]));
                            // (moved only where the row's own sum asks for it: its bits do not depend on what other rows see)
                            const float next = grow ? fmaxf(m, fmaxf(tops[0], tops[1]) * unscale) : m;
                            const float keep = m == next ? 1.f : ex2(m - next);
                            m = next;
                            l *= keep;
                            round = 1;  // the next one is the last
                            if (half == 1) {  // the first half's weights are on their way into O
                                ok = __all_sync(0xffffffffu, wait_for(&ctl.half_done[t], s_phase ^ 1));
                                tc_fence_after();
                            }
                            if (half == 1 || u > x.from)
#pragma unroll 1
                                for (int c = 0; c < p.hd; c += 16) {
                                    uint32_t o[16];
                                    tm_ld16(o_at + c, o);
                                    tc_wait_ld();
#pragma unroll
                                    for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * keep);
                                    tm_st16(o_at + c, o);
                                }
                        }
                        l += total;
                        live_row = live_row && total == total;
                        tc_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(half ? &ctl.p_ready[t] : &ctl.p_half[t]);
                }
                if (!ok) break;
            }
            ok = ok && __all_sync(0xffffffffu, wait_for(&ctl.o_full[t], o_phase));
            o_phase ^= 1u;
            tc_fence_after();
            if (busy) {
                const bool put = mine && ok;  // (nothing is written where a wait ran out)
                const bool poison = ctl.poison[piece % kPoisonRing] == static_cast<uint32_t>(piece);
                const bool whole = w.whole(x), empty = see_lo >= see_hi;
                float* part = part_of(p, blockIdx.x, x.first);
                m -= kShift;
                if (!x.begin) {
                    const float2 ml = add_before(p, part, t * kHalf + r, o_at, m, l, mine);
                    m = ml.x;
                    l = ml.y;
                }
                const float inv = !whole ? 1.f : empty ? 0.f : 1.f / l;  // (a row that sees nothing has sums of zero)
                // Results go to memory through q's place, by rows of a warp: 16 bytes a lane of neighbouring lanes instead of a
                // row a lane, which took 7000 cycles of a tile.
                const int es = whole && p.first && p.out_bf16 ? 2 : 4;
                char* to;
                if (!whole) to = reinterpret_cast<char*>(part_o(p, part, t * kHalf + r));
                else if (!p.first) to = reinterpret_cast<char*>(p.prefix_out + (static_cast<int64_t>(row) * p.nh + h_row) * p.hd);
                else to = static_cast<char*>(p.out) + (row * p.out_stride + static_cast<int64_t>(h_row) * p.hd) * es;
                constexpr int kRowBytes = 128;  // of 32 rows: a round's
                const uint32_t stage = q_chunk(t, 0, 0) + quarter * 32 * kRowBytes;
                const int columns = kRowBytes / es;
                float odd = 0.f;
#pragma unroll 1
                for (int c0 = 0; c0 < p.hd; c0 += columns) {
#pragma unroll 1
                    for (int c = c0; c < min(p.hd, c0 + columns); c += 16) {
                        uint32_t v[16];
                        tm_ld16(o_at + c, v);
                        tc_wait_ld();
                        uint32_t d[16];
                        float o[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            o[k] = __uint_as_float(v[k]) * inv;
                            odd = fmaf(o[k], 0.f, odd);
                            d[k] = __float_as_uint(o[k]);
                        }
                        if (es == 2) {
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d[k]) : "f"(o[2 * k + 1]), "f"(o[2 * k]));
                        }
                        const uint32_t dst = stage + lane * kRowBytes, first = (c - c0) * es / 16;  // 16-byte piece of the row
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            if (es == 4 || k < 2)
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + (((first + k) ^ (lane & 7)) << 4)),
                                             "r"(d[4 * k]), "r"(d[4 * k + 1]), "r"(d[4 * k + 2]), "r"(d[4 * k + 3])
                                             : "memory");
                    }
                    __syncwarp();
                    // eight lanes a row
                    const int skip = c0 * es + 16 * (lane & 7);
#pragma unroll
                    for (int k = 0; k < 32; k += 4) {
                        const int from = k + (lane >> 3);
                        char* dst = reinterpret_cast<char*>(__shfl_sync(0xffffffffu, reinterpret_cast<u64>(to), from)) + skip;
                        const bool has = __shfl_sync(0xffffffffu, put, from);
                        uint4 w4;
                        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(w4.x), "=r"(w4.y), "=r"(w4.z), "=r"(w4.w)
                                     : "r"(stage + from * kRowBytes + (((lane & 7) ^ (from & 7)) << 4))
                                     : "memory");
                        if (has && skip < p.hd * es) store16(dst, w4, es);
                    }
                    __syncwarp();
                }
                // (a sum of weights that is NaN makes all of the row NaN already)
                const bool live = put && l > 0.f;
                // (a sum of weights that is NaN makes all of the row NaN already)
                if (stream_any(kStreamBarrier + t, busy_warps, live && (poison || !(odd == 0.f))))
                    mend_rows<SPLIT, NCH>(p, busy_warps, tile.seq, kv, live ? max(see_lo, tile.lo + x.from * kBlock) : 0,
                                          live ? min(see_hi, tile.lo + x.to * kBlock) : 0, to, es);
                if (put) {
                    float* lse = p.first ? p.lse : p.prefix_lse;
                    if (!whole) *part_ml(part, t * kHalf + r) = make_float2(m, l);
                    else if (lse) lse[static_cast<int64_t>(row) * p.nh + h_row] = lse_of(m, l, empty);
                }
                tc_fence_before();
            }
            // all warps of the stream come here, whatever became of their waits
            // all warps of the stream come here, whatever became of their waits, and leave together
            if (stream_any(kEndBarrier + t, 4, !ok)) {
                ok = false;
                break;
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.q_free[t]);
        }
        if (!ok && lane == 0) flag_bad(kFlagTimeout, 0);
      }
    } else if (work && warp == kMmaWarp) {
        // ---- MMAs
        const int steps = p.hd / 16;
        const uint32_t id_s = idesc(kBlock, false), id_o = idesc(p.hd, true);
        // The next block's K and V: stages of their first chunks, and the phases that they wait for.
        uint32_t k_at = 0, k_phase = 0, v_at = NCH, v_phase = 0;
        uint32_t q_phase = 0, h_phase = 0, p_phase = 0, o_phase = 0;  // bit t
        bool ok = true;
        auto wait = [&](uint64_t* bar, uint32_t phase) {
            if (ok) ok = __all_sync(0xffffffffu, wait_for(bar, phase));
            tc_fence_after();
        };
        auto wait_full = [&](uint32_t at, uint32_t phase) {  // a block's chunks of K or V
#pragma unroll
            for (int c = 0; c < NCH; ++c) wait(&ctl.full[at + c], phase);
        };
        // (one commit for a head's chunks: each takes the issuing thread 65 to 115 cycles)
        auto release = [&](uint32_t at) { tc_commit(&ctl.empty[at]); };
        auto next_block = [&](uint32_t& at, uint32_t& phase) {
            at += 2 * NCH;
            if (at >= S::kStages) {
                at -= S::kStages;
                phase ^= 1u;
            }
        };
        const uint32_t ring = desc_k(ring_at), ring_v = desc_mn(ring_at);
        auto scores = [&](int t) {  // of stream t and the next block
            uint32_t acc = 0;
#pragma unroll
            for (int part = kParts - 1; part >= 0; --part)  // the small products first
#pragma unroll
                for (int c = 0; c < NCH; ++c) {
                    const uint32_t a = desc_k(q_chunk(t, part, c)), b = ring + (k_at + c) * (kChunkBytes >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)  // 16 columns are 32 bytes
                        if (4 * c + k < steps) {
                            mma_ss(tmem + 128 * t, a + 2 * k, b + 2 * k, id_s, acc);
                            acc = 1;
                        }
                }
            tc_commit(&ctl.s_full[t]);
        };
        // O of stream t: the first half of the slots as soon as their weights are there
        auto sums = [&](int t, uint32_t acc) {
            const uint32_t v = ring_v + v_at * (kChunkBytes >> 4), o = tmem + 256 + (SPLIT ? 0 : 128 * t), w0 = tmem + 128 * t;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (half == 0) {
                    wait(&ctl.p_half[t], (h_phase >> t) & 1);
                    h_phase ^= 1u << t;
                } else {
                    wait(&ctl.p_ready[t], (p_phase >> t) & 1);
                    p_phase ^= 1u << t;
                }
                if (!ok) return;
#pragma unroll
                for (int k = half * kBlock / 32; k < (half + 1) * kBlock / 32; ++k)  // 16 slots are 2048 bytes
#pragma unroll
                    for (int part = kParts - 1; part >= 0; --part) {
                        mma_ts(o, w0 + 32 * (k >> 1) + 16 * part + 8 * (k & 1), v + 128 * k, id_o, acc);
                        acc = 1;
                    }
                if (!SPLIT && half == 0) tc_commit(&ctl.half_done[t]);
            }
        };
        while (ok && w.next(p, x)) {
            const int n = x.to - x.from;
            if (SPLIT) {
                wait(&ctl.q_ready[0], q_phase);
                q_phase ^= 1u;
                for (int b = 0; b < min(n, 2) && ok; ++b) {
                    wait_full(k_at, k_phase);
                    if (!ok) break;
                    scores(b);
                    release(k_at);
                    next_block(k_at, k_phase);
                }
                for (int b = 0; b < n && ok; ++b) {
                    const int t = b & 1;
                    wait_full(v_at, v_phase);
                    if (b > 0 && b % kFold == 0) {  // the accumulator's sums have been added to the others
                        wait(&ctl.o_free, o_phase);
                        o_phase ^= 1u;
                    }
                    if (ok) sums(t, b % kFold != 0);
                    if (!ok) break;
                    tc_commit(&ctl.pv_done);
                    release(v_at);
                    next_block(v_at, v_phase);
                    if (b + 1 == n && p.fail != kFailEnd) tc_commit(&ctl.o_full[0]);
                    if (b + 2 >= n) continue;
                    wait_full(k_at, k_phase);
                    if (!ok) break;
                    scores(t);
                    release(k_at);
                    next_block(k_at, k_phase);
                }
            } else {
                const int halves = x.t.ntok > p.part_tokens ? 2 : 1;
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if (t >= halves || !ok) break;
                    wait(&ctl.q_ready[t], (q_phase >> t) & 1);
                    q_phase ^= 1u << t;
                    if (t == 0) wait_full(k_at, k_phase);
                    if (ok) scores(t);
                }
                if (!ok) break;
                release(k_at);
                next_block(k_at, k_phase);
                for (int b = 0; b < n && ok; ++b) {
                    const bool last = b + 1 == n;
                    if (!last) wait_full(k_at, k_phase);  // (here rather than between weights that are there and scores)
                    wait_full(v_at, v_phase);
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (t >= halves) break;
                        if (ok) sums(t, b > 0);
                        if (!ok) break;
                        if (t + 1 == halves) release(v_at);
                        if (!last) scores(t);
                        else if (p.fail != kFailEnd) tc_commit(&ctl.o_full[t]);
                    }
                    if (!ok) break;
                    next_block(v_at, v_phase);
                    if (!last) {
                        release(k_at);
                        next_block(k_at, k_phase);
                    }
                }
            }
        }
        if (!ok) {  // what was issued ends before tensor memory is freed
            tc_commit(&ctl.drained);
            wait_for(&ctl.drained, 0);
            if (lane == 0) flag_bad(kFlagTimeout, 0);
        }
        __syncwarp();
    } else if (work && warp == kMmaWarp + 1) {
        // ---- q of the next piece, as soon as the last one's results have left its place
        uint32_t phase = 3;  // bit t: nothing to wait for at first
        bool ok = true;
        const uint32_t bytes = kParts * NCH * 128 * p.per_block * p.part_tokens;
        while (ok && w.next(p, x)) {
            const int kv = x.head / p.blocks, h0 = kv * G + (x.head - kv * p.blocks) * p.per_block;
            for (int t = 0; t < (SPLIT ? 1 : 2); ++t) {
                const int token = t * p.part_tokens;
                if (!ok || token >= x.t.ntok) break;
                ok = __all_sync(0xffffffffu, wait_for(&ctl.q_free[t], (phase >> t) & 1));
                phase ^= 1u << t;
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&ctl.q_ready[t], bytes);
                    for (int c = 0; c < NCH; ++c) {
                        tma_box(q_chunk(t, 0, c), &map_q, 64 * c, h0, x.t.row0 + token, &ctl.q_ready[t]);
                        if (SPLIT) tma_box(q_chunk(t, kParts - 1, c), &map_ql, 64 * c, h0, x.t.row0 + token, &ctl.q_ready[t]);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) flag_bad(kFlagTimeout, 0);
    } else if (work && warp >= kLoadWarp && box) {
        // ---- copies by TMA: boxes of `box` rows of a page, lane b of warp 12 the b-th of a block
        uint32_t item = 0;
        int piece = 0, block = 0;
        bool ok = true;
        if (warp == kLoadWarp) {
            while (ok && w.next(p, x)) {
                const RowTile& tile = x.t;
                const int col = x.head / p.blocks * p.hd, per = kBlock / box;
                // page ids are asked for a block ahead
                auto ask = [&](int u) {
                    const int slot = tile.lo + u * kBlock + lane * box;
                    return u < x.to && lane < per && slot < tile.hi ? page_ref(p.c, tile.seq, slot) : PageRef{0, -1};
                };
                PageRef asked = ask(x.from);
                for (int u = x.from; ok && u < x.to; ++u, ++block) {
                    const PageRef at = asked;
                    asked = ask(u + 1);
                    bool valid = at.in_page >= 0;
                    if (valid && static_cast<unsigned int>(at.id) >= static_cast<unsigned int>(p.c.n_pages)) {
                        flag_bad(kFlagIndexRange, at.id);
                        valid = false;
                    }
                    const uint32_t boxes = __ballot_sync(0xffffffffu, valid);
                    const int j0 = tile.lo + u * kBlock;
#pragma unroll
                    for (int kc = 0; kc < 2 * NCH; ++kc) {  // K's chunks, then V's
                        const uint32_t n = item;
                        if (ok && n >= S::kStages && kc % NCH == 0)  // a head's chunks are freed together
                            ok = __all_sync(0xffffffffu, wait_for(&ctl.empty[n % S::kStages], (n / S::kStages - 1) & 1));
                        if (!ok) break;
                        ++item;
                        if (kc == 0) {
                            if (lane == 0) note_moved();
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int s = 32 * c + lane;
                                const uint32_t there = __ballot_sync(0xffffffffu, j0 + s < tile.hi && ((boxes >> (s / box)) & 1u));
                                if (lane == 0) ctl.live[block % kLiveRing][c] = there;
                            }
                        }
                        if (lane == 0) mbar_arrive_expect_tx(&ctl.landed[n % S::kStages], __popc(boxes) * box * 128);
                        __syncwarp();
                        if (valid)
                            tma_box(chunk_at(n) + lane * box * 128, kc < NCH ? &map_k : &map_v, col + 64 * (kc % NCH), at.in_page,
                                    at.id, &ctl.landed[n % S::kStages]);
                    }
                }
            }
            if (!ok) {  // no copy is in flight when the CTA ends
                for (uint32_t n = item > S::kStages ? item - S::kStages : 0; n < item; ++n)
                    wait_for(&ctl.landed[n % S::kStages], (n / S::kStages) & 1);
                if (lane == 0) flag_bad(kFlagTimeout, 0);
            }
        } else {
            const int chunks16 = p.hd / 8, me = (warp - kLoadWarp - 1) * 32 + lane;
            while (ok && w.next(p, x)) {
                ++piece;
                for (int u = x.from; ok && u < x.to; ++u, ++block) {
                    const int j0 = x.t.lo + u * kBlock;
                    const bool check = j0 < x.t.all_lo || j0 + kBlock > x.t.all_hi;
#pragma unroll 1
                    for (int kc = 0; kc < 2 * NCH; ++kc) {
                        const uint32_t n = item++;
                        ok = __all_sync(0xffffffffu, wait_for(&ctl.landed[n % S::kStages], (n / S::kStages) & 1));
                        if (!ok) break;
                        const uint32_t* live = ctl.live[block % kLiveRing];
                        if (kc >= NCH && (check || (live[0] & live[1] & live[2] & live[3]) != 0xffffffffu)) {
                            const int width = min(8, chunks16 - 8 * (kc - NCH));  // 16-byte pieces of a row here
                            bool bad = false;
                            constexpr int kSkip = 32 * (kLoadWarps - 1) / 8, kBatch = 4;  // rows from one piece of a thread to the next
                            const uint32_t col = me & 7;
#pragma unroll 1
                            for (int r0 = me >> 3; r0 < kBlock; r0 += kBatch * kSkip) {
                                uint32_t v[kBatch][4], at[kBatch];
                                bool there[kBatch];
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    const int row = min(r0 + k * kSkip, kBlock - 1);
                                    at[k] = chunk_at(n) + swz(row, col);
                                    there[k] = (live[row >> 5] >> (row & 31)) & 1u;
                                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                                 : "=r"(v[k][0]), "=r"(v[k][1]), "=r"(v[k][2]), "=r"(v[k][3]) : "r"(at[k]) : "memory");
                                }
#pragma unroll
                                for (int k = 0; k < kBatch; ++k) {
                                    if (static_cast<int>(col) >= width || r0 + k * kSkip >= kBlock) continue;
                                    // slots that are not there: whatever the page, or the ring before, holds
                                    if (!there[k]) v[k][0] = v[k][1] = v[k][2] = v[k][3] = 0;
                                    else if (finite_f16x2(v[k][0]) && finite_f16x2(v[k][1]) && finite_f16x2(v[k][2]) &&
                                             finite_f16x2(v[k][3]))
                                        continue;
                                    else bad = true;
                                    keep_finite(at[k], v[k]);
                                }
                            }
                            if (bad) ctl.poison[piece % kPoisonRing] = piece;
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&ctl.full[n % S::kStages]);
                    }
                }
            }
            if (!ok && lane == 0) flag_bad(kFlagTimeout, 0);
        }
    } else if (work && warp >= kLoadWarp) {
        // ---- copies by cp.async: warp i of four has slots 32 i .. 32 i + 31 of a block
        const int i = warp - kLoadWarp;
        uint32_t item = 0, done = 0;  // chunks asked for, chunks handed over
        int piece = 0, block = 0;
        bool ok = true;
        const int chunks16 = p.hd / 8;  // 16-byte pieces of a row
        // of the chunks in flight: which hold V to be looked at (bit n % 32 of chunk n), and their pieces (four bits each)
        uint32_t look = 0;
        u64 pieces = 0;
        auto hand_over = [&]() {
            const uint32_t n = done++;
            if ((look >> (n % 32)) & 1u) {
                bool bad = false;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (static_cast<int>(n % NCH) * 8 + (lane & 7) < chunks16)
                        bad |= clean16(chunk_at(n) + swz(32 * i + 4 * k + (lane >> 3), lane & 7));
                // pieces in flight are few: the number's last four bits tell which
                if (bad) {
                    const uint32_t low = static_cast<uint32_t>(pieces >> (4 * (n % 16))) & 15u;
                    ctl.poison[low] = piece - ((piece - low) & 15u);
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl.full[n % S::kStages]);
        };
        while (ok && w.next(p, x)) {
            const RowTile& tile = x.t;
            const int kv = x.head / p.blocks;
            ++piece;
            auto ask = [&](int u) {
                const int slot = tile.lo + u * kBlock + 32 * i + lane;
                return u < x.to && slot < tile.hi ? page_ref(p.c, tile.seq, slot) : PageRef{0, -1};
            };
            PageRef asked = ask(x.from);
            for (int u = x.from; ok && u < x.to; ++u, ++block) {
                const int j0 = tile.lo + u * kBlock;
                const int64_t at = asked.in_page >= 0 ? row_offset(p.c, asked) : -1;
                asked = ask(u + 1);
                const uint32_t there = __ballot_sync(0xffffffffu, at >= 0);
                const int64_t base = at >= 0 ? at + static_cast<int64_t>(kv) * p.hd : 0;
                const bool check = j0 < tile.all_lo || j0 + kBlock > tile.all_hi;
                int64_t off[8];
#pragma unroll
                for (int k = 0; k < 8; ++k) off[k] = __shfl_sync(0xffffffffu, base, 4 * k + (lane >> 3));
#pragma unroll
                for (int kc = 0; kc < 2 * NCH; ++kc) {  // K's chunks, then V's
                    const bool is_v = kc >= NCH;
                    const int c = kc % NCH;
                    const __half* pool = static_cast<const __half*>(is_v ? p.c.v : p.c.k);
                    const uint32_t n = item;
                    if (ok && n >= S::kStages && c == 0)  // a head's chunks are freed together
                        ok = __all_sync(0xffffffffu, wait_for(&ctl.empty[n % S::kStages], (n / S::kStages - 1) & 1));
                    if (!ok) break;
                    ++item;
                    if (kc == 0 && lane == 0) {
                        if (i == 0) note_moved();
                        ctl.live[block % kLiveRing][i] = there;
                    }
                    pieces = (pieces & ~(15ull << (4 * (n % 16)))) | static_cast<u64>(piece & 15) << (4 * (n % 16));
                    look = is_v && check ? look | 1u << (n % 32) : look & ~(1u << (n % 32));
                    if (8 * c + (lane & 7) < chunks16) {
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            const int row = 4 * k + (lane >> 3);
                            cp_async16(chunk_at(n) + swz(32 * i + row, lane & 7), pool + off[k] + 64 * c + 8 * (lane & 7),
                                       (there >> row) & 1u ? 16u : 0u);
                        }
                    }
                    asm volatile("cp.async.commit_group;" ::: "memory");
                    if (item > S::kLag) {
                        asm volatile("cp.async.wait_group %0;" ::"n"(S::kLag) : "memory");
                        hand_over();
                    }
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (ok) {
            while (done < item) hand_over();
        } else if (lane == 0) {
            flag_bad(kFlagTimeout, 0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kMmaWarp)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f) : nullptr;
    }();
    return fn;
}

// Three dimensions of f16 values, read in boxes of 64 values of the first.
bool encode(CUtensorMap* map, const void* base, int64_t n0, int64_t n1, int64_t n2, int64_t stride1, int64_t stride2, int box1,
            int box2) {
    if (!encoder()) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(n0), static_cast<cuuint64_t>(n1), static_cast<cuuint64_t>(n2)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(stride1) * 2, static_cast<cuuint64_t>(stride2) * 2};
    const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(box1), static_cast<cuuint32_t>(box2)}, steps[3] = {1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(base), dims, strides, boxes, steps,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool SPLIT, int NCH>
cudaError_t launch_t(const PagedRowsParams& p, cudaStream_t stream) {
    auto kernel = paged_rows_tc_kernel<SPLIT, NCH>;
    constexpr int smem = Shape<SPLIT, NCH>::kSmem;
    // fewer registers at launch than the warpgroups share out would leave some of them waiting for ever
    static const bool enough = [&] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, kernel) == cudaSuccess && a.numRegs >= kLaunchRegs;
    }();
    if (!enough) return cudaErrorInvalidKernelImage;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    // Boxes of as many rows, a power of two, as divide a page and a block; eight rows are an atom of the swizzle.
    int box = 1;
    while (box < kBlock && p.c.page_size % (2 * box) == 0) box *= 2;
    CUtensorMap maps[4];  // pools as columns x rows of a page x pages, q as columns x heads x tokens
    std::memset(maps, 0, sizeof maps);
    for (int i = 0; i < 2 && box; ++i)
        if (box < 8 || p.c.nkt < 64 ||
            !encode(&maps[i], i ? p.c.v : p.c.k, p.c.nkt, p.c.page_size, p.c.n_pages, p.c.nkt, p.c.page_stride, box, 1))
            box = 0;
    const int64_t nqt = static_cast<int64_t>(p.nh) * p.hd;
    for (int i = 0; i < (SPLIT ? 2 : 1); ++i)
        if (!encode(&maps[2 + i], i ? p.q_low : p.q_high, p.hd, p.nh, p.nt, p.hd, nqt, p.per_block, p.part_tokens))
            return cudaErrorInvalidValue;
    return launch_dependent(kernel, dim3(kSms), kThreads, smem, stream, 1, p, maps[0], maps[1], maps[2], maps[3], box);
}

}  // namespace

RowsShape paged_rows_tc_shape(bool split) {
    return {split ? kHalf : 2 * kHalf, kHalf, kBlock, kSms, kTileCost, true};
}

cudaError_t launch_paged_rows_tc(const PagedRowsParams& p, cudaStream_t stream) {
    if (p.out_bf16) return p.hd <= 64 ? launch_t<false, 1>(p, stream) : launch_t<false, 2>(p, stream);
    return p.hd <= 64 ? launch_t<true, 1>(p, stream) : launch_t<true, 2>(p, stream);
}

cudaError_t paged_rows_tc_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
