// qkv_rope_step: rows of heads turned by their positions (include/qkv.h has the contract).
//
// Pairs (x0, x1) -> (x0 c - x1 s, x0 s + x1 c), every value read and written once, so memory bounds all but a few
// rows.  A thread takes eight neighbouring values of a head, or four pairs whose halves are apart, and the same ones of
// several heads of its row: the angles are made once for them, and all its loads are in flight together.
// Measured (GPU time in a graph): one token of 14 + 2 heads of 64 1.6 us (one trip through position and angle; a call takes the
// host 5), 1641 tokens of 32 heads of 128 f16, half of each turned, 5.2 us (26.9 MB, in part from L2), 8191 of 48 bf16 heads 33.7
// us (201 MB at 6.0 TB/s, 0.88 of the copy rate; issue slots are 58 % busy).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "paged_common.cuh"
#include "ptx_sync.cuh"
#include "rope_math.cuh"

namespace {

using namespace qkv_rope_math;
using qkv_paged::kSms;
using qkv_paged::launch_dependent;

constexpr int kThreads = 256;
constexpr int kMaxHeads = 4;  // of a thread

template <typename T>
struct Four;  // four neighbouring values as stored
template <>
struct Four<float> {
    Quad v;
    __device__ __forceinline__ void load(const float* p) { v = quad(p); }
    __device__ __forceinline__ Quad get() const { return v; }
    static __device__ __forceinline__ void store(float* p, Quad q) {
        *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(q.a, q.b);
    }
};
template <>
struct Four<__nv_bfloat16> {
    uint2 v;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ Quad get() const {
        return {pack(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)),
                pack(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u))};
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, Quad q) {
        const float2 x = unpack(q.a), y = unpack(q.b);
        __nv_bfloat162 h[2] = {__floats2bfloat162_rn(x.x, x.y), __floats2bfloat162_rn(y.x, y.y)};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
    }
};
template <>
struct Four<__half> {
    uint2 v;
    __device__ __forceinline__ void load(const __half* p) { v = *reinterpret_cast<const uint2*>(p); }
    __device__ __forceinline__ Quad get() const {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
        const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
        return {pack(x.x, x.y), pack(y.x, y.y)};
    }
    static __device__ __forceinline__ void store(__half* p, Quad q) {
        const float2 x = unpack(q.a), y = unpack(q.b);
        __half2 h[2] = {__floats2half2_rn(x.x, x.y), __floats2half2_rn(y.x, y.y)};
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
    }
};

// Work item: (row, HEADS neighbouring heads, lane l of hd / 8); items in that order, a thread each.
template <typename T, bool NEIGHBOURS, int HEADS>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int lanes = p.hd >> 3, blocks = (p.n_heads + HEADS - 1) / HEADS;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t unit = item / lanes;
    const int l = static_cast<int>(item - unit * lanes);
    const int64_t row = unit / blocks;
    if (row >= p.nt) return;
    const int h0 = static_cast<int>(unit - row * blocks) * HEADS;
    const bool turned = 8 * l < p.rope.rot;
    int a, b;
    lane_quads<NEIGHBOURS>(l, p.rope.rot, a, b);
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride + static_cast<int64_t>(h0) * p.hd;
    T* out = static_cast<T*>(p.out) + row * p.out_stride + static_cast<int64_t>(h0) * p.hd;
    Four<T> v0[HEADS], v1[HEADS];
#pragma unroll
    for (int k = 0; k < HEADS; ++k)
        if (HEADS == 1 || h0 + k < p.n_heads) {
            v0[k].load(x + k * p.hd + a);
            v1[k].load(x + k * p.hd + b);
        }
    Quad c = {0, 0}, s = {0, 0};
    if (turned) {
        const int pos = p.positions[row];
        float2 t[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = cos_sin(p.rope, pos, 4 * l + i);
        c = {pack(t[0].x, t[1].x), pack(t[2].x, t[3].x)};
        s = {pack(t[0].y, t[1].y), pack(t[2].y, t[3].y)};
        if (p.inverse) {
            s.a ^= 0x8000000080000000ull;
            s.b ^= 0x8000000080000000ull;
        }
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
        if (HEADS > 1 && h0 + k >= p.n_heads) break;
        Quad x0 = v0[k].get(), x1 = v1[k].get();
        if (turned) {
            if (NEIGHBOURS) {
                rotate_neighbours(x0, x1, c, s);
            } else {
                Quad r0, r1;
                rotate2(x0.a, x1.a, c.a, s.a, r0.a, r1.a);
                rotate2(x0.b, x1.b, c.b, s.b, r0.b, r1.b);
                x0 = r0;
                x1 = r1;
            }
        }
        Four<T>::store(out + k * p.hd + a, x0);
        Four<T>::store(out + k * p.hd + b, x1);
    }
}

__device__ __forceinline__ float get1(const float* p) { return *p; }
__device__ __forceinline__ float get1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float get1(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ void put1(float* p, float v) { *p = v; }
__device__ __forceinline__ void put1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put1(__half* p, float v) { *p = __float2half_rn(v); }

// Any head size and alignment: a thread takes one pair, or one value that passes.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_any_kernel(const __grid_constant__ RopeParams p) {
    qkv_ptx::griddep_wait();
    qkv_ptx::griddep_launch_dependents();
    const int half = p.rope.rot >> 1, units = p.hd - half;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t head = item / units;
    const int u = static_cast<int>(item - head * units);
    const int64_t row = head / p.n_heads;
    if (row >= p.nt) return;
    const int h = static_cast<int>(head - row * p.n_heads);
    const T* x = static_cast<const T*>(p.x) + row * p.x_stride + static_cast<int64_t>(h) * p.hd;
    T* out = static_cast<T*>(p.out) + row * p.out_stride + static_cast<int64_t>(h) * p.hd;
    if (u >= half) {
        out[half + u] = x[half + u];
        return;
    }
    const int a = p.rope.neighbours ? 2 * u : u, b = p.rope.neighbours ? 2 * u + 1 : half + u;
    float2 cs = cos_sin(p.rope, p.positions[row], u);
    if (p.inverse) cs.y = -cs.y;
    const float x0 = get1(x + a), x1 = get1(x + b);
    put1(out + a, __fsub_rn(__fmul_rn(x0, cs.x), __fmul_rn(x1, cs.y)));
    put1(out + b, __fadd_rn(__fmul_rn(x0, cs.y), __fmul_rn(x1, cs.x)));
}

template <typename T>
cudaError_t launch_t(const RopeParams& p, cudaStream_t stream) {
    const uintptr_t n = 4 * sizeof(T);
    const bool vec = p.hd % 8 == 0 && p.rope.rot % 8 == 0 && reinterpret_cast<uintptr_t>(p.x) % n == 0 &&
                     reinterpret_cast<uintptr_t>(p.out) % n == 0 && p.x_stride % 4 == 0 && p.out_stride % 4 == 0;
    const int64_t heads = static_cast<int64_t>(p.nt) * p.n_heads;
    const auto grid = [](int64_t items) { return dim3(static_cast<unsigned int>((items + kThreads - 1) / kThreads)); };
    if (!vec) return launch_dependent(rope_any_kernel<T>, grid(heads * (p.hd - p.rope.rot / 2)), kThreads, 0, stream, 1, p);
    const int lanes = p.hd / 8;
    // Several heads a thread once that still leaves every SM two CTAs: 8191 tokens of 48 heads take 39 us and not 102 (one head
    // a thread, whose angles are then most of the work), 1641 of 32 10.2 and not 14.3, 200 of 32 6.1 either way (with a launch).
    const bool many = heads * lanes >= static_cast<int64_t>(2 * kSms) * kThreads * kMaxHeads;
    const int per = many ? kMaxHeads : 1;
    const dim3 g = grid(static_cast<int64_t>(p.nt) * ((p.n_heads + per - 1) / per) * lanes);
    if (p.rope.neighbours)
        return launch_dependent(many ? rope_kernel<T, true, kMaxHeads> : rope_kernel<T, true, 1>, g, kThreads, 0, stream, 1, p);
    return launch_dependent(many ? rope_kernel<T, false, kMaxHeads> : rope_kernel<T, false, 1>, g, kThreads, 0, stream, 1, p);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t stream) {
    switch (dtype) {
        case QKV_F32: return launch_t<float>(p, stream);
        case QKV_BF16: return launch_t<__nv_bfloat16>(p, stream);
        default: return launch_t<__half>(p, stream);
    }
}
