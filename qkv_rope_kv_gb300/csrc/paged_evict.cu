// qkv_evict_step: cut every (sequence, kv head) down to the slots with the largest running
// attention weight and the newest ones (include/qkv.h has the contract).
//
// Each slot gets a 32-bit key that orders as (protected, weight); the budget-th largest key is
// found by a radix select, equal keys are taken from the lowest slot up.  Only rows move that
// have to: the i-th dropped slot below the budget takes the i-th kept slot above it.  Sources
// (>= budget) and destinations (< budget) are disjoint, so the copies need no order.
//
// Two launches: one finds the moves (one or more CTAs per item, bound by their chain of barriers and
// cluster exchanges), one makes them with the whole GPU (bound by the latency of list, table and
// row, or by memory); a single one where items have little to move.  Measured (GPU time): 8 sequences x 8
// heads, 2112 -> 2048 slots 9.9 us; 1 x 4, 32749 -> 8192 22.6 us; 32 x 2, to 4099 -> 1000 18.5 us (the bytes
// would take 0.9, 4.0 and 5.6 us).  256 threads instead of 1024: 14.8 us for the first kernel where 1024 take
// 9.3; both in one launch for the prompt: 30 us.
#include <algorithm>

#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace {

using namespace qkv_paged;

constexpr int kThreads = 1024;
constexpr int kBins = 2048, kPasses = 3;               // digits of 11, 11 and 10 bits
constexpr int kFixedSmem = (kPasses + 1) * kBins * 4;  // a histogram a digit and the cluster's sum of one
constexpr int kMaxCluster = 16;
constexpr int64_t kOwnMoveBytes = 128 * 1024;
constexpr int64_t kPrefetchBytes = 4 * 1024 * 1024;
constexpr uint32_t kCountEverywhere = 4096;            // keys left from which on a digit needs no exchange (24.9 -> 24.1 us)
constexpr int64_t kMaxSlots = 48 * 1024;               // slots of a CTA whose keys fit in shared memory
constexpr int64_t kClusterSlots = 4096;                // slots of a CTA of a cluster
static_assert(2 * kClusterSlots <= kMaxSlots, "a CTA that is alone holds its keys");
static_assert(kFixedSmem >= kThreads * 16, "a batch of moves fits the histograms' place");

// Slots of a CTA that is alone, as its keys are kept: whole rounds of its threads.
__host__ __device__ constexpr int64_t cap_slots(int64_t cap) { return (cap + kThreads - 1) / kThreads * kThreads; }

// Order-preserving key of a slot: protected slots above everything, NaN above every number.
__device__ __forceinline__ uint32_t slot_key(float w, int pos, int64_t protect_from) {
    if (pos >= protect_from) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void cluster_sync(int size) {
    if (size == 1) {
        __syncthreads();
    } else {
        __syncwarp();
        asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
}

__device__ __forceinline__ uint32_t peer_address(const void* p, int rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(qkv_ptx::smem_u32(p)), "r"(rank));
    return a;
}

// A 32-bit word of CTA `rank` of a cluster of `size`, at the place of `p` in its shared memory.
__device__ __forceinline__ uint32_t peer_word(const uint32_t* p, int rank, int size) {
    if (size == 1) return *p;
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(peer_address(p, rank)) : "memory");
    return v;
}

// Add to a counter of the first `to` CTAs of the cluster (1: this CTA's own).
__device__ __forceinline__ void add_count(uint32_t* counter, uint32_t n, int to) {
    if (to == 1) {
        atomicAdd(counter, n);
        return;
    }
    for (int r = 0; r < to; ++r)
        asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(peer_address(counter, r)), "r"(n) : "memory");
}

// Count one key's bin: one addition for the whole warp where its lanes agree (equal weights would
// otherwise serialise on one address).
__device__ __forceinline__ void count_bin(uint32_t* hist, uint32_t bin, bool in, int to) {
    const unsigned int active = __ballot_sync(0xffffffffu, in);
    if (active == 0u) return;
    const int leader = __ffs(active) - 1;
    const uint32_t first = __shfl_sync(0xffffffffu, bin, leader);
    if (__all_sync(0xffffffffu, !in || bin == first)) {
        if (static_cast<int>(threadIdx.x & 31) == leader) add_count(hist + first, static_cast<uint32_t>(__popc(active)), to);
    } else if (in) {
        add_count(hist + bin, 1u, to);
    }
}

// Make an item's moves chunk, chunk + chunks, ... (which they are does not depend on how many there are, so the
// list is read together with its length; LISTED: it is in shared memory, `known` long).  A thread looks up a move's rows and carries its weight and position;
// then all threads copy the rows of K and V, CT by CT, kUnroll of them in flight.  to_s and from_s: THREADS
// entries of shared memory.
template <typename CT, int THREADS, int kUnroll, bool LISTED>
__device__ __forceinline__ void make_moves(const PagedEvictParams& p, int item, int chunk, int chunks, int64_t* to_s,
                                           int64_t* from_s, const int32_t* holes, const int32_t* movers, int known) {
    const int b = item / p.nkv, h = item - b * p.nkv, tid = threadIdx.x;
    const int cap = p.c.max_pages * p.c.page_size;
    const int64_t base = static_cast<int64_t>(item) * cap;
    const int row_units = p.hd * (p.kv_f16 ? 2 : 4) / static_cast<int>(sizeof(CT));
    const int elem_per_unit = static_cast<int>(sizeof(CT)) / (p.kv_f16 ? 2 : 4);
    const int i0 = tid / (2 * row_units), c0 = tid - i0 * 2 * row_units;
    const int step_i = THREADS / (2 * row_units), step_c = THREADS - step_i * 2 * row_units;
    CT* kp = static_cast<CT*>(p.c.k);
    CT* vp = static_cast<CT*>(p.c.v);
#pragma unroll 1
    for (int64_t p0 = chunk;; p0 += static_cast<int64_t>(THREADS) * chunks) {
        const int64_t at = p0 + static_cast<int64_t>(tid) * chunks;
        const bool could = at < (LISTED ? known : cap / 2);
        const int to = could ? (LISTED ? holes[at] : __ldcg(holes + at)) : 0;
        const int from = could ? (LISTED ? movers[at] : __ldcg(movers + at)) : 0;
        const int pairs = LISTED ? known : __ldcg(p.moves + item);
        if (p0 >= pairs) break;
        const int n = static_cast<int>(min(static_cast<int64_t>(THREADS), (pairs - p0 + chunks - 1) / chunks));
        if (tid < n) {
            // everything the two slots name is asked for before any of it is looked at
            const float w = p.c.slot_weight[base + from];
            const int pos = p.c.slot_pos[base + from];
            const PageRef rt = page_ref(p.c, b, to), rf = page_ref(p.c, b, from);
            const int64_t ot = row_offset(p.c, rt), of = row_offset(p.c, rf);
            const bool can = ot >= 0 && of >= 0;  // else the slot stays as it is
            to_s[tid] = can ? (ot + h * p.hd) / elem_per_unit : -1;
            from_s[tid] = (of + h * p.hd) / elem_per_unit;
            p.weight_out[base + to] = can ? w : p.c.slot_weight[base + to];
            p.pos_out[base + to] = can ? pos : p.c.slot_pos[base + to];
        }
        __syncthreads();
        // unit c of move i, and on by THREADS units a step
        int i = i0, c = c0;
#pragma unroll 1
        while (i < n) {
            CT v[kUnroll];
            CT* dst[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                dst[u] = nullptr;
                if (i < n && to_s[i] >= 0) {
                    CT* pool = c < row_units ? kp + c : vp + (c - row_units);
                    dst[u] = pool + to_s[i];
                    v[u] = pool[from_s[i]];
                }
                i += step_i;
                c += step_c;
                if (c >= 2 * row_units) {
                    c -= 2 * row_units;
                    ++i;
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (dst[u]) *dst[u] = v[u];
        }
        __syncthreads();
    }
}

// A cluster of `size` CTAs per (sequence, kv head); each holds a contiguous run of the slots.  CACHED: their
// keys are kept in shared memory; otherwise they are made again each time.  ALONE: a cluster is one CTA
// (11.0 us; 11.8 us where the kernel has to ask).  MOVES (alone, rows of whole 16 bytes): it makes its
// moves too.
template <bool CACHED, bool MOVES, bool ALONE, int T>
__global__ void __launch_bounds__(T, kThreads / T) paged_evict_select_kernel(const __grid_constant__ PagedEvictParams p,
                                                                      int cluster) {
    static_assert(ALONE || !MOVES, "a cluster's moves are made by the second kernel");
    const int size = ALONE ? 1 : cluster;
    constexpr int W = T / 32;
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem);
    uint32_t* sum = hist + kPasses * kBins;
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kFixedSmem);
    __shared__ uint32_t warp_s[W], warp2_s[W];
    __shared__ uint32_t found_s[3];  // bin, keys still wanted from it, keys in it
    __shared__ uint32_t publish_s[3];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = blockIdx.x / size, rank = blockIdx.x - item * size;
    const int b = item / p.nkv, h = item - b * p.nkv;
    const int cap = p.c.max_pages * p.c.page_size;
    for (int i = tid; i < kPasses * kBins / 4; i += T) reinterpret_cast<uint4*>(hist)[i] = make_uint4(0, 0, 0, 0);
    const int64_t base = static_cast<int64_t>(item) * cap;
    // Lengths, weights and positions on their way to L2 while the launch before this one ends: of all slots, or if
    // that is much (0.6 us of bandwidth), of those likely to be in use.  32 sequences x 2 heads to 4099 slots
    // 20.9 -> 19.8 us, with the likely ones alone 20.6.
    const bool few = static_cast<int64_t>(p.c.n_seq) * p.nkv * cap * 8 <= kPrefetchBytes;
    const int64_t likely = few ? cap : min(static_cast<int64_t>(cap), 2 * static_cast<int64_t>(p.budget));
    if (rank == 0 && tid == 0) prefetch_l2(p.lens + b);
    if (rank == 0 && tid == 32) prefetch_l2(p.next_pos + b);
    for (int64_t s = (rank * T + tid) * 32; s < likely; s += size * T * 32) {
        prefetch_l2(p.c.slot_weight + base + s);
        prefetch_l2(p.c.slot_pos + base + s);
    }
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int len = p.lens[b];
    const int next_pos = p.next_pos[b];
    const bool sane = len >= 0 && len <= cap;
    if (rank == 0 && tid == 0) {
        if (h == 0) {
            if (!sane) flag_bad(kFlagIndexRange, len);
            p.lens_out[b] = sane ? min(len, p.budget) : len;
        }
        if (!MOVES && (!sane || len <= p.budget)) p.moves[item] = 0;
    }
    if (!sane) return;
    const float* w_in = p.c.slot_weight + base;
    const int32_t* pos_in = p.c.slot_pos + base;
    float* w_out = p.weight_out + base;
    int32_t* pos_out = p.pos_out + base;
    if (len <= p.budget) {
        for (int s = rank * T + tid; s < len; s += size * T) {
            w_out[s] = w_in[s];
            pos_out[s] = pos_in[s];
        }
        return;
    }
    const int64_t protect_from = static_cast<int64_t>(next_pos) - p.recent;
    const int run = (len + size * T - 1) / (size * T) * 32;  // slots of a warp
    const int s0 = (rank * W + warp) * run;
    const int mine = max(0, min(run, len - s0));
    uint32_t* my_keys = keys + warp * run;
    auto key_of = [&](int i) -> uint32_t {  // i-th slot of this warp
        if (CACHED) return my_keys[i];
        return slot_key(__ldcg(w_in + s0 + i), __ldcg(pos_in + s0 + i), protect_from);
    };
    if (CACHED) {
#pragma unroll 8
        for (int i = lane; i < mine; i += 32) my_keys[i] = slot_key(w_in[s0 + i], pos_in[s0 + i], protect_from);
    }
    __syncthreads();  // the histograms are clear

    // The budget-th largest key, digit by digit: after a digit, `low` is the smallest key with the
    // digits found so far, and `want` how many of the keys with those digits are kept.
    uint32_t low = 0u, want = static_cast<uint32_t>(p.budget), in_bin = 0u;
    int shift = 32;
#pragma unroll 1
    for (int pass = 0; pass < kPasses; ++pass) {
        const int above = shift;
        shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
        uint32_t* my_hist = hist + pass * kBins;
        // few keys are left: each is counted in every CTA at once, and no exchange of sums has to follow
        const bool everywhere = size > 1 && pass > 0 && in_bin <= kCountEverywhere;
#pragma unroll 4
        for (int i = lane; i < run; i += 32) {
            const bool there = i < mine;
            const uint32_t k = there ? key_of(i) : 0u;
            count_bin(my_hist, (k >> shift) & (pass == 2 ? 1023u : 2047u), there && (pass == 0 || k >> above == low >> above),
                      everywhere ? size : 1);
        }
        const uint32_t* bins = my_hist;
        if (size == 1) {
            __syncthreads();
        } else if (everywhere) {
            cluster_sync(size);
        } else if constexpr (!ALONE) {
            // each CTA adds up its share of the bins over the cluster and hands the sums to every CTA
            cluster_sync(size);
            const int each = kBins / size, per = T / each;  // bins of a CTA; threads of a bin
            const int bin = rank * each + tid / per, part = tid % per;
            uint32_t c = 0u;
            for (int r = part; r < size; r += per) c += peer_word(my_hist + bin, r, size);
            for (int o = per >> 1; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            for (int r = part; r < size; r += per)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_address(sum + bin, r)), "r"(c) : "memory");
            cluster_sync(size);
            bins = sum;
        }
        // thread t: its share of the bins from the top one down, so that a scan runs from the largest key down
        constexpr int kMine = kBins / T;
        static_assert(kMine == 2 || kMine == 4, "one load a thread");
        uint32_t c[kMine], incl = 0u;
        if constexpr (kMine == 2) {
            const uint2 v = *reinterpret_cast<const uint2*>(bins + kBins - 2 - 2 * tid);
            c[0] = v.y;
            c[1] = v.x;
        } else {
            const uint4 v = *reinterpret_cast<const uint4*>(bins + kBins - 4 - 4 * tid);
            c[0] = v.w;
            c[1] = v.z;
            c[2] = v.y;
            c[3] = v.x;
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) incl += c[i];
        const uint32_t total = incl;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) warp_s[warp] = incl;
        __syncthreads();
        incl += __reduce_add_sync(0xffffffffu, lane < warp ? warp_s[lane] : 0u);
        uint32_t excl = incl - total;
        if (excl < want && want <= incl) {
#pragma unroll
            for (int i = 0; i < kMine; ++i) {
                if (excl < want && want <= excl + c[i]) {
                    found_s[0] = kBins - 1 - kMine * tid - i;
                    found_s[1] = want - excl;
                    found_s[2] = c[i];
                }
                excl += c[i];
            }
        }
        __syncthreads();
        low |= found_s[0] << shift;
        want = found_s[1];
        in_bin = found_s[2];
        if (want == in_bin) break;  // all keys from `low` up are kept
        __syncthreads();            // found_s and (before the next cluster barrier) sum have been read
    }
    // kept: keys above the found digits, and of those with them all, or (whole keys) the first `want`
    const bool ranked = want != in_bin;
    uint32_t tie0 = 0u;
    if (ranked) {
        uint32_t n = 0u;
        for (int i = lane; i < run; i += 32) n += __popc(__ballot_sync(0xffffffffu, i < mine && key_of(i) == low));
        if (lane == 0) warp2_s[warp] = n;
        __syncthreads();
        if (warp == 0) {
            n = __reduce_add_sync(0xffffffffu, lane < W ? warp2_s[lane] : 0u);
            if (lane == 0) publish_s[0] = n;
        }
        cluster_sync(size);
        tie0 = __reduce_add_sync(0xffffffffu, (lane < rank ? peer_word(publish_s, lane, size) : 0u) +
                                                  (lane < warp ? warp2_s[lane] : 0u));
        __syncthreads();
    }
    // MOVES: the lists stay here, behind the place of make_moves' rows
    int32_t* holes = MOVES ? reinterpret_cast<int32_t*>(keys + cap_slots(cap)) : p.lists + static_cast<int64_t>(item) * 2 * (cap / 2);
    int32_t* movers = holes + cap / 2;
    int pairs = 0;
    uint32_t hole0 = 0u, mover0 = 0u;
    const bool copy_meta = w_out != w_in || pos_out != pos_in;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // count, then write the lists
        uint32_t tie_at = tie0, hole_at = hole0, mover_at = mover0;
#pragma unroll 1
        for (int i = lane; i < run; i += 32) {
            const bool in = i < mine;
            const int s = s0 + i;
            const uint32_t k = in ? key_of(i) : 0u;
            const unsigned int below = (1u << lane) - 1u;
            bool kept = in && k >= low;
            if (ranked) {
                const unsigned int tied = __ballot_sync(0xffffffffu, in && k == low);
                kept = in && (k > low || (k == low && tie_at + __popc(tied & below) < want));
                tie_at += __popc(tied);
            }
            const bool hole = in && !kept && s < p.budget, mover = kept && s >= p.budget;
            const unsigned int hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
            if (pass) {
                if (hole) holes[hole_at + __popc(hm & below)] = s;
                if (mover) movers[mover_at + __popc(mm & below)] = s;
                if (copy_meta && kept && s < p.budget) {
                    w_out[s] = w_in[s];
                    pos_out[s] = pos_in[s];
                }
            }
            hole_at += __popc(hm);
            mover_at += __popc(mm);
        }
        if (pass == 0) {
            if (lane == 0) {
                warp_s[warp] = hole_at;
                warp2_s[warp] = mover_at;
            }
            __syncthreads();
            if (warp == 0) {
                const uint32_t h_all = __reduce_add_sync(0xffffffffu, lane < W ? warp_s[lane] : 0u);
                const uint32_t m_all = __reduce_add_sync(0xffffffffu, lane < W ? warp2_s[lane] : 0u);
                if (lane == 0) {
                    publish_s[1] = h_all;
                    publish_s[2] = m_all;
                }
            }
            cluster_sync(size);
            const uint32_t nh = lane < size ? peer_word(publish_s + 1, lane, size) : 0u;
            const uint32_t nm = lane < size ? peer_word(publish_s + 2, lane, size) : 0u;
            const uint32_t all = __reduce_add_sync(0xffffffffu, nh);
            pairs = static_cast<int>(all);
            if (!MOVES && rank == 0 && tid == 0) p.moves[item] = pairs;
            hole0 = __reduce_add_sync(0xffffffffu, (lane < rank ? nh : 0u) + (lane < warp ? warp_s[lane] : 0u));
            mover0 = __reduce_add_sync(0xffffffffu, (lane < rank ? nm : 0u) + (lane < warp ? warp2_s[lane] : 0u));
        }
    }
    if constexpr (MOVES) {
        __syncthreads();  // the list is written, and the histograms have been read
        int64_t* to_s = reinterpret_cast<int64_t*>(smem);
        make_moves<uint4, T, T == kThreads ? 2 : 4, true>(p, item, 0, 1, to_s, to_s + T, holes, movers, pairs);
    } else {
        if (size > 1) cluster_sync(size);  // no CTA leaves while another may read its shared memory
    }
}

// The moves, `chunks` CTAs per item.
constexpr int kMoveThreads = 256;

template <typename CT>
__global__ void __launch_bounds__(kMoveThreads) paged_evict_move_kernel(const __grid_constant__ PagedEvictParams p,
                                                                        int chunks) {
    __shared__ int64_t to_s[kMoveThreads], from_s[kMoveThreads];
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int item = blockIdx.x / chunks, half = p.c.max_pages * p.c.page_size / 2;
    const int32_t* holes = p.lists + static_cast<int64_t>(item) * 2 * half;
    make_moves<CT, kMoveThreads, 8, false>(p, item, blockIdx.x - item * chunks, chunks, to_s, from_s, holes, holes + half, 0);
}

template <typename CT>
cudaError_t launch_move(const PagedEvictParams& p, int64_t most, cudaStream_t stream) {
    // enough CTAs for every SM to have four, but none for fewer than 16 of the moves there can be
    const int64_t items = static_cast<int64_t>(p.c.n_seq) * p.nkv;
    int64_t chunks = (4 * kSms + items - 1) / items;
    if (chunks > (most + 15) / 16) chunks = (most + 15) / 16;
    return launch_dependent(paged_evict_move_kernel<CT>, dim3(static_cast<unsigned int>(items * chunks)), kMoveThreads, 0,
                            stream, 1, p, static_cast<int>(chunks));
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    const int items = p.c.n_seq * p.nkv, es = p.kv_f16 ? 2 : 4;
    // CTAs of a (sequence, kv head): one up to 2 kClusterSlots slots of capacity (the cluster's exchanges cost
    // 3 us: 8.8 us alone, 11.7 us in twos at 4128 slots), then one for each kClusterSlots (32768 slots in
    // clusters of 4, 8, 16: 18.1, 15.5, 17.4 us), while that leaves no more than two per SM
    int size = cap > 2 * kClusterSlots ? 2 : 1;
    while (size > 1 && size < kMaxCluster && cap > kClusterSlots * size && static_cast<int64_t>(items) * size < 2 * kSms)
        size *= 2;
    const int64_t slots = (cap + static_cast<int64_t>(size) * kThreads - 1) / (static_cast<int64_t>(size) * kThreads) * kThreads;
    const bool cached = slots <= kMaxSlots;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * es) | static_cast<uintptr_t>(p.hd * es);
    const bool whole16 = (bits & 15u) == 0;
    // One launch where no item can have more than kOwnMoveBytes to move (its CTA then takes about as long as
    // a second launch would), or no item has anything to move.
    const int64_t most = std::max<int64_t>(0, std::min<int64_t>(p.budget, cap - p.budget));
    const bool moves = size == 1 && cached && whole16 && most * 2 * p.hd * es <= kOwnMoveBytes;
    // A CTA of 1024 threads has an SM to itself: with more items than SMs, half the threads (8 heads x 128 x f16,
    // 32 sequences 600 -> 550 slots 14.5 us with 1024, 9.6 us with 512; 2112 -> 2048 22.0 and 16.7 us).
    const bool halves = items > kSms;
    const int threads = size == 1 && halves ? kThreads / 2 : kThreads;
    const size_t smem = kFixedSmem + (cached ? static_cast<size_t>(slots) * 4 : 0) + (moves ? static_cast<size_t>(cap / 2) * 8 : 0);
    // A kernel, and the most shared memory that a call of it can need.  That limit belongs to the kernel, not to the
    // launch: were it set to what this call needs, a call of another thread could lower it before this one's launch.
    struct Select {
        void (*kernel)(PagedEvictParams, int);
        int64_t most_smem;
    };
    const Select select =
        moves       ? Select{halves ? paged_evict_select_kernel<true, true, true, kThreads / 2>
                                    : paged_evict_select_kernel<true, true, true, kThreads>,
                             kFixedSmem + 2 * kClusterSlots * (4 + 4)}
        : size == 1 ? Select{halves ? paged_evict_select_kernel<true, false, true, kThreads / 2>
                                    : paged_evict_select_kernel<true, false, true, kThreads>,
                             kFixedSmem + 2 * kClusterSlots * 4}
        : cached    ? Select{paged_evict_select_kernel<true, false, false, kThreads>, kFixedSmem + kMaxSlots * 4}
                    : Select{paged_evict_select_kernel<false, false, false, kThreads>, kFixedSmem};
    auto kernel = select.kernel;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(select.most_smem));
    if (e == cudaSuccess && size > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess)
        e = launch_dependent(kernel, dim3(static_cast<unsigned int>(items) * size), threads, smem, stream, size, p, size);
    if (e != cudaSuccess || moves || most == 0) return e;
    if (whole16) return launch_move<uint4>(p, most, stream);
    return p.kv_f16 ? launch_move<uint16_t>(p, most, stream) : launch_move<uint32_t>(p, most, stream);
}

cudaError_t paged_evict_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
