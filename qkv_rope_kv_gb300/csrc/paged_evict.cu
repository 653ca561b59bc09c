// qkv_evict_step: cut every (sequence, kv head) down to the slots with the largest running
// attention weight and the newest ones (include/qkv.h has the contract).
//
// Each slot gets a 32-bit key that orders as (protected, weight); the budget-th largest key is
// found by a radix select, equal keys are taken from the lowest slot up.  Only rows move that
// have to: the i-th dropped slot below the budget takes the i-th kept slot above it.  Sources
// (>= budget) and destinations (< budget) are disjoint, so the copies need no order.
#include "paged_common.cuh"
#include "ptx_sync.cuh"

namespace {

using namespace qkv_paged;

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// Order-preserving key of a slot: protected slots above everything, NaN above every number.
__device__ __forceinline__ uint32_t slot_key(float w, int pos, int64_t protect_from) {
    if (pos >= protect_from) return 0xffffffffu;
    if (w != w) return 0xfffffffeu;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 counts as +0
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kBins = 2048, kPasses = 3;           // digits of 11, 11 and 10 bits
constexpr int kBatch = 1024;                       // moves whose rows are looked up at a time
constexpr int kFixedSmem = (kPasses + 1) * kBins * 4;  // a histogram a digit and the cluster's sum of one; later
                                                       // the batch's row offsets
constexpr int kMaxCluster = 16;
constexpr int kSms = 152;
constexpr int64_t kClusterSlots = 4096;            // slots of a CTA before another joins it
constexpr int64_t kMaxSlots = 32768;               // slots of a CTA whose keys (and list entries) fit in shared memory
static_assert(kFixedSmem >= kBatch * 16, "row offsets fit the histograms' place");

__device__ __forceinline__ void cluster_sync(int size) {
    if (size == 1) {
        __syncthreads();
    } else {
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

// Entry i of a list of 16-bit slots in the shared memory of CTA `rank`.
__device__ __forceinline__ int peer_entry(const uint16_t* list, int i, int rank, int size) {
    if (size == 1) return list[i];
    uint16_t v;
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(peer_address(list + i, rank)) : "memory");
    return v;
}

// Count one key's bin: one atomic for the whole warp where its lanes agree (equal weights would
// otherwise serialise on one address).
__device__ __forceinline__ void count_bin(uint32_t* hist, uint32_t bin, bool in) {
    const unsigned int active = __ballot_sync(0xffffffffu, in);
    if (active == 0u) return;
    const int leader = __ffs(active) - 1;
    const uint32_t first = __shfl_sync(0xffffffffu, bin, leader);
    if (__all_sync(0xffffffffu, !in || bin == first)) {
        if (static_cast<int>(threadIdx.x & 31) == leader) atomicAdd(hist + first, static_cast<uint32_t>(__popc(active)));
    } else if (in) {
        atomicAdd(hist + bin, 1u);
    }
}

// A cluster of `size` CTAs per (sequence, kv head); each holds a contiguous run of the slots.  CACHED: their
// keys are kept in shared memory, and so are the lists of what moves; otherwise the keys are made again each
// time and the lists are in the workspace.  CT is the unit of the row copies.
template <typename CT, bool CACHED>
__global__ void __launch_bounds__(kThreads) paged_evict_kernel(const __grid_constant__ PagedEvictParams p, int size) {
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t* hist = reinterpret_cast<uint32_t*>(smem);
    uint32_t* sum = hist + kPasses * kBins;
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem + kFixedSmem);
    __shared__ uint32_t warp_s[kWarps], warp2_s[kWarps];
    __shared__ uint32_t found_s[3];  // bin, keys still wanted from it, keys in it
    __shared__ uint32_t publish_s[3];
    __shared__ int hole_s[kMaxCluster + 1], mover_s[kMaxCluster + 1];  // where each CTA's lists begin
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = blockIdx.x / size, rank = blockIdx.x - item * size;
    const int b = item / p.nkv, h = item - b * p.nkv;
    const int cap = p.c.max_pages * p.c.page_size;
    for (int i = tid; i < kPasses * kBins; i += kThreads) hist[i] = 0u;
    qkv_ptx::griddep_wait();
    const int len = __ldg(p.lens + b);
    const int next_pos = __ldg(p.next_pos + b);
    const bool sane = len >= 0 && len <= cap;
    if (h == 0 && rank == 0 && tid == 0) {
        if (!sane) flag_bad(kFlagIndexRange, len);
        p.lens_out[b] = sane ? min(len, p.budget) : len;
    }
    if (!sane) return;
    const int64_t base = static_cast<int64_t>(item) * cap;
    const float* w_in = p.c.slot_weight + base;
    const int32_t* pos_in = p.c.slot_pos + base;
    float* w_out = p.weight_out + base;
    int32_t* pos_out = p.pos_out + base;
    if (len <= p.budget) {
        for (int s = rank * kThreads + tid; s < len; s += size * kThreads) {
            w_out[s] = w_in[s];
            pos_out[s] = pos_in[s];
        }
        return;
    }
    const int64_t protect_from = static_cast<int64_t>(next_pos) - p.recent;
    const int run = (len + size * kThreads - 1) / (size * kThreads) * 32;  // slots of a warp
    const int cta0 = rank * kWarps * run;                                  // this CTA's first slot
    const int s0 = cta0 + warp * run;
    const int mine = max(0, min(run, len - s0));
    uint32_t* my_keys = keys + warp * run;
    uint16_t* list = reinterpret_cast<uint16_t*>(keys + kWarps * run);  // holes from the front, movers from the back
    auto key_of = [&](int i) -> uint32_t {  // i-th slot of this warp
        if (CACHED) return my_keys[i];
        return slot_key(__ldcg(w_in + s0 + i), __ldcg(pos_in + s0 + i), protect_from);
    };
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
        if (CACHED && pass == 0) {
#pragma unroll 4
            for (int i = lane; i < mine; i += 32) my_keys[i] = slot_key(w_in[s0 + i], pos_in[s0 + i], protect_from);
            __syncwarp();
        }
#pragma unroll 1
        for (int i = lane; i < run; i += 32) {
            const bool there = i < mine;
            const uint32_t k = there ? key_of(i) : 0u;
            count_bin(my_hist, (k >> shift) & (pass == 2 ? 1023u : 2047u), there && (pass == 0 || k >> above == low >> above));
        }
        const uint32_t* bins = my_hist;
        if (size == 1) {
            __syncthreads();
        } else {
            // each CTA adds up its share of the bins over the cluster and hands the sums to every CTA
            cluster_sync(size);
            const int each = kBins / size, per = kThreads / each;  // bins of a CTA; threads of a bin
            const int bin = rank * each + tid / per, part = tid % per;
            uint32_t c = 0u;
            for (int r = part; r < size; r += per) c += peer_word(my_hist + bin, r, size);
            for (int o = per >> 1; o; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
            for (int r = part; r < size; r += per)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_address(sum + bin, r)), "r"(c) : "memory");
            cluster_sync(size);
            bins = sum;
        }
        // thread t: bins 2047 - 2t and 2046 - 2t, so that a scan runs from the largest key down
        const uint32_t c0 = bins[kBins - 1 - 2 * tid], c1 = bins[kBins - 2 - 2 * tid];
        uint32_t incl = c0 + c1;
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) warp_s[warp] = incl;
        __syncthreads();
        incl += __reduce_add_sync(0xffffffffu, lane < warp ? warp_s[lane] : 0u);
        const uint32_t excl = incl - c0 - c1;
        if (excl < want && want <= incl) {
            const bool second = excl + c0 < want;
            found_s[0] = kBins - 1 - 2 * tid - second;
            found_s[1] = want - excl - (second ? c0 : 0u);
            found_s[2] = second ? c1 : c0;
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
            n = __reduce_add_sync(0xffffffffu, warp2_s[lane]);
            if (lane == 0) publish_s[0] = n;
        }
        cluster_sync(size);
        tie0 = __reduce_add_sync(0xffffffffu, (lane < rank ? peer_word(publish_s, lane, size) : 0u) +
                                                  (lane < warp ? warp2_s[lane] : 0u));
        __syncthreads();
    }
    int32_t* g_holes = p.lists + static_cast<int64_t>(item) * 2 * (cap / 2);
    int32_t* g_movers = g_holes + cap / 2;
    const int slots = kWarps * run;
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
                const int at = hole ? hole_at + __popc(hm & below) : mover_at + __popc(mm & below);
                if (CACHED) {
                    if (hole || mover) list[hole ? at : slots - 1 - at] = static_cast<uint16_t>(s - cta0);
                } else {
                    if (hole) g_holes[at] = s;
                    if (mover) g_movers[at] = s;
                }
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
            const uint32_t nh = warp_s[lane], nm = warp2_s[lane];
            hole0 = __reduce_add_sync(0xffffffffu, lane < warp ? nh : 0u);
            mover0 = __reduce_add_sync(0xffffffffu, lane < warp ? nm : 0u);
            if (warp == 0) {
                const uint32_t h_all = __reduce_add_sync(0xffffffffu, nh), m_all = __reduce_add_sync(0xffffffffu, nm);
                if (lane == 0) {
                    publish_s[1] = h_all;
                    publish_s[2] = m_all;
                }
            }
            if (!CACHED) {  // the workspace's lists are the whole item's
                cluster_sync(size);
                hole0 += __reduce_add_sync(0xffffffffu, lane < rank ? peer_word(publish_s + 1, lane, size) : 0u);
                mover0 += __reduce_add_sync(0xffffffffu, lane < rank ? peer_word(publish_s + 2, lane, size) : 0u);
            }
        }
    }
    // The lists are there, and no CTA will read a weight or position below the budget any more.
    cluster_sync(size);
    if (warp < 2) {  // begins of the CTAs' lists: holes by warp 0, movers by warp 1
        int c = lane < size ? static_cast<int>(peer_word(publish_s + 1 + warp, lane, size)) : 0, incl = c;
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane <= size) (warp ? mover_s : hole_s)[lane] = incl - c;
    }
    __syncthreads();
    const int pairs = hole_s[size];

    // This CTA's share of the moves, a batch at a time: a thread looks up a move's rows and carries its
    // weight and position; then all threads copy the rows of K and V.
    int64_t* to_s = reinterpret_cast<int64_t*>(smem);
    int64_t* from_s = to_s + kBatch;
    const int share = (pairs + size - 1) / size;
    const int p1 = min(pairs, (rank + 1) * share);
    const int row_units = p.hd * (p.kv_f16 ? 2 : 4) / static_cast<int>(sizeof(CT));
    const int elem_per_unit = static_cast<int>(sizeof(CT)) / (p.kv_f16 ? 2 : 4);
    CT* kp = static_cast<CT*>(p.c.k);
    CT* vp = static_cast<CT*>(p.c.v);
#pragma unroll 1
    for (int p0 = rank * share; p0 < p1; p0 += kBatch) {
        const int n = min(kBatch, p1 - p0);
        for (int i = tid; i < n; i += kThreads) {
            int to, from;
            if (CACHED) {
                int rh = 0, rm = 0;  // whose lists hold move p0 + i
                for (int r = 1; r < size; ++r) {
                    rh += hole_s[r] <= p0 + i;
                    rm += mover_s[r] <= p0 + i;
                }
                to = rh * slots + peer_entry(list, p0 + i - hole_s[rh], rh, size);
                from = rm * slots + peer_entry(list, slots - 1 - (p0 + i - mover_s[rm]), rm, size);
            } else {
                to = __ldcg(g_holes + p0 + i);
                from = __ldcg(g_movers + p0 + i);
            }
            const float w = w_in[from];
            const int pos = pos_in[from];
            const int64_t rt = row_offset(p.c, b, to), rf = row_offset(p.c, b, from);
            to_s[i] = rt >= 0 && rf >= 0 ? (rt + h * p.hd) / elem_per_unit : -1;
            from_s[i] = (rf + h * p.hd) / elem_per_unit;
            w_out[to] = w;
            pos_out[to] = pos;
        }
        __syncthreads();
        const int total = n * 2 * row_units;
        constexpr int kUnroll = 4;
#pragma unroll 1
        for (int e0 = tid; e0 < total; e0 += kThreads * kUnroll) {
            CT v[kUnroll];
            CT* dst[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int e = e0 + u * kThreads, i = e / (2 * row_units), c = e - i * 2 * row_units;
                dst[u] = nullptr;
                if (e < total && to_s[i] >= 0) {
                    CT* pool = c < row_units ? kp + c : vp + (c - row_units);
                    dst[u] = pool + to_s[i];
                    v[u] = pool[from_s[i]];
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (dst[u]) *dst[u] = v[u];
        }
        __syncthreads();
    }
    if (CACHED) cluster_sync(size);  // the other CTAs have read this one's lists
}

template <typename CT>
cudaError_t launch_t(const PagedEvictParams& p, cudaStream_t stream) {
    // CTAs of a (sequence, kv head): one for 4096 slots of capacity, while that leaves no more than
    // two per SM
    const int64_t cap = static_cast<int64_t>(p.c.max_pages) * p.c.page_size;
    const int items = p.c.n_seq * p.nkv;
    int size = 1;
    while (size < kMaxCluster && cap > kClusterSlots * size && static_cast<int64_t>(items) * size < 2 * kSms) size *= 2;
    const int64_t slots = (cap + static_cast<int64_t>(size) * kThreads - 1) / (static_cast<int64_t>(size) * kThreads) * kThreads;
    const bool cached = slots <= kMaxSlots;
    const int64_t key_bytes = slots * 6;  // keys and list entries
    auto kernel = cached ? paged_evict_kernel<CT, true> : paged_evict_kernel<CT, false>;
    const size_t smem = kFixedSmem + (cached ? static_cast<size_t>(key_bytes) : 0);
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e == cudaSuccess && size > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned int>(items) * size);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = size;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = size > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p, size);
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
    const int es = p.kv_f16 ? 2 : 4;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * es) | static_cast<uintptr_t>(p.hd * es);
    if ((bits & 15u) == 0) return launch_t<uint4>(p, stream);
    return p.kv_f16 ? launch_t<uint16_t>(p, stream) : launch_t<uint32_t>(p, stream);
}

cudaError_t paged_evict_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
