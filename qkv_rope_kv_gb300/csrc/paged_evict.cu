// qkv_evict_step: cut every (sequence, kv head) down to the slots with the largest running
// attention weight and the newest ones (include/qkv.h has the contract).
//
// Each slot gets a 32-bit key that orders as (protected, weight); the budget-th largest key is
// found by a radix select, equal keys are taken from the lowest slot up.  Only rows move that
// have to: the i-th dropped slot below the budget takes the i-th kept slot above it.  Sources
// (>= budget) and destinations (< budget) are disjoint, so the copies need no order.
#include "paged_common.cuh"

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

// Exclusive prefix over the warps of one value per warp (all threads get their warp's).
__device__ __forceinline__ int warp_prefix(int mine, int* buf, int warp, int lane) {
    if (lane == 0) buf[warp] = mine;
    __syncthreads();
    int v = lane < warp ? buf[lane] : 0;
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    return v;
}

template <bool VEC>
__device__ __forceinline__ void copy_row(char* base, int64_t to, int64_t from, int bytes, int lane) {
    if constexpr (VEC) {
        for (int i = lane * 16; i < bytes; i += 512)
            *reinterpret_cast<uint4*>(base + to + i) = *reinterpret_cast<const uint4*>(base + from + i);
    } else {
        for (int i = lane * 2; i < bytes; i += 64)
            *reinterpret_cast<uint16_t*>(base + to + i) = *reinterpret_cast<const uint16_t*>(base + from + i);
    }
}

// One CTA per (sequence, kv head).
template <bool VEC>
__global__ void __launch_bounds__(kThreads) paged_evict_kernel(const __grid_constant__ PagedEvictParams p) {
    __shared__ unsigned int hist_s[256];
    __shared__ int buf_s[kWarps];
    __shared__ unsigned int prefix_s;
    __shared__ int want_s;
    const int b = blockIdx.x / p.nkv, h = blockIdx.x - b * p.nkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cap = p.c.max_pages * p.c.page_size;
    const int len = __ldg(p.lens + b);
    const bool sane = len >= 0 && len <= cap;
    if (h == 0 && tid == 0) {
        if (!sane) flag_bad(kFlagIndexRange, len);
        p.lens_out[b] = sane ? min(len, p.budget) : len;
    }
    if (!sane) return;
    const int64_t base = static_cast<int64_t>(blockIdx.x) * cap;
    const float* w_in = p.c.slot_weight + base;
    const int32_t* pos_in = p.c.slot_pos + base;
    float* w_out = p.weight_out + base;
    int32_t* pos_out = p.pos_out + base;
    if (len <= p.budget) {
        for (int s = tid; s < len; s += kThreads) {
            w_out[s] = w_in[s];
            pos_out[s] = pos_in[s];
        }
        return;
    }
    const int64_t protect_from = static_cast<int64_t>(__ldg(p.next_pos + b)) - p.recent;

    // The budget-th largest key, byte by byte from the top: after a byte, prefix holds the key's
    // bytes so far and `want` how many of the keys with that prefix are still to be taken.
    if (tid == 0) {
        prefix_s = 0u;
        want_s = p.budget;
    }
    for (int shift = 24; shift >= 0; shift -= 8) {
        if (tid < 256) hist_s[tid] = 0u;
        __syncthreads();
        const uint32_t prefix = prefix_s, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
        for (int s = tid; s < len; s += kThreads) {
            const uint32_t k = slot_key(w_in[s], pos_in[s], protect_from);
            if ((k & mask) == prefix) atomicAdd(&hist_s[(k >> shift) & 255u], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane i holds the bytes 255 - 8i .. 248 - 8i, from the largest down
            unsigned int c[8], sum = 0u;
            for (int i = 0; i < 8; ++i) sum += c[i] = hist_s[255 - 8 * lane - i];
            unsigned int incl = sum;
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned int up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const unsigned int want = static_cast<unsigned int>(want_s);
            unsigned int above = incl - sum;
            __syncwarp();
            if (above < want && want <= incl)
                for (int i = 0; i < 8; ++i) {
                    if (above + c[i] >= want) {
                        prefix_s = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
                        want_s = static_cast<int>(want - above);
                        break;
                    }
                    above += c[i];
                }
        }
        __syncthreads();
    }
    const uint32_t T = prefix_s;
    const int ties = want_s;  // how many slots with key T are kept, lowest first

    // Each warp owns a contiguous run of slots, so ranks follow the slots' order.
    const int run = (len + kThreads - 1) / kThreads * 32;
    const int s0 = warp * run, s1 = min(len, s0 + run);
    int n_tie = 0;
    for (int s = s0 + lane; s < s0 + run; s += 32) {
        const bool tie = s < s1 && slot_key(w_in[s], pos_in[s], protect_from) == T;
        n_tie += __popc(__ballot_sync(0xffffffffu, tie));
    }
    const int tie0 = warp_prefix(n_tie, buf_s, warp, lane);
    int32_t* holes = p.lists + static_cast<int64_t>(blockIdx.x) * 2 * (cap / 2);
    int32_t* movers = holes + cap / 2;
    int hole0 = 0, mover0 = 0, n_pairs = 0;
    for (int pass = 0; pass < 2; ++pass) {  // count, then write the lists
        int tie_at = tie0, hole_at = hole0, mover_at = mover0;
        for (int s = s0 + lane; s < s0 + run; s += 32) {
            const bool in = s < s1;
            const uint32_t k = in ? slot_key(w_in[s], pos_in[s], protect_from) : 0u;
            const unsigned int tied = __ballot_sync(0xffffffffu, in && k == T);
            const unsigned int below = (1u << lane) - 1u;
            const bool kept = in && (k > T || (k == T && tie_at + __popc(tied & below) < ties));
            tie_at += __popc(tied);
            const bool hole = in && !kept && s < p.budget, mover = kept && s >= p.budget;
            const unsigned int hm = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
            if (pass && hole) holes[hole_at + __popc(hm & below)] = s;
            if (pass && mover) movers[mover_at + __popc(mm & below)] = s;
            hole_at += __popc(hm);
            mover_at += __popc(mm);
        }
        if (pass == 0) {
            hole0 = warp_prefix(hole_at, buf_s, warp, lane);
            mover0 = warp_prefix(mover_at, buf_s, warp, lane);
        } else if (warp == kWarps - 1 && lane == 0) {
            want_s = hole_at;  // the total
        }
    }
    __syncthreads();
    n_pairs = want_s;

    // Kept slots below the budget keep their weight and position; then the moves overwrite the
    // freed slots (their old values are not needed: sources lie at or above the budget).
    if (w_out != w_in || pos_out != pos_in)
        for (int s = tid; s < p.budget; s += kThreads) {
            w_out[s] = w_in[s];
            pos_out[s] = pos_in[s];
        }
    __syncthreads();
    const int es = p.kv_f16 ? 2 : 4, bytes = p.hd * es;
    for (int i = warp; i < n_pairs; i += kWarps) {
        const int to = holes[i], from = movers[i];
        const int64_t rt = row_offset(p.c, b, to), rf = row_offset(p.c, b, from);
        if (rt >= 0 && rf >= 0) {
            const int64_t bt = (rt + h * p.hd) * es, bf = (rf + h * p.hd) * es;
            copy_row<VEC>(static_cast<char*>(p.c.k), bt, bf, bytes, lane);
            copy_row<VEC>(static_cast<char*>(p.c.v), bt, bf, bytes, lane);
        }
        if (lane == 0) {
            w_out[to] = w_in[from];
            pos_out[to] = pos_in[from];
        }
    }
}

}  // namespace

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
    const int es = p.kv_f16 ? 2 : 4;
    const uintptr_t bits = reinterpret_cast<uintptr_t>(p.c.k) | reinterpret_cast<uintptr_t>(p.c.v) |
                           static_cast<uintptr_t>(p.c.page_stride * es) | static_cast<uintptr_t>(p.hd * es);
    const int grid = p.c.n_seq * p.nkv;
    if ((bits & 15u) == 0) paged_evict_kernel<true><<<grid, kThreads, 0, stream>>>(p);
    else paged_evict_kernel<false><<<grid, kThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

cudaError_t paged_evict_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad) {
    return status_read(stream, flags, bad);
}
