// Rotary positions of a qkv_rope (include/qkv.h): frequencies as turns a position, in units of 2^-64 turn.
#pragma once

#include <cuda_runtime.h>

#include "qkv_internal.h"

namespace qkv_rope_math {

// (cos, sin) of pair d at position pos, times the magnitude.  The product keeps its low 64 bits, so whole turns
// fall away exactly, and the upper half, signed, is the angle in 2^-31 half turns, |x| <= 1: one rounding to f32
// (2^-25 half turns) and sincospif, which has no large arguments to reduce.
__device__ __forceinline__ float2 cos_sin(const RopeTable& r, int pos, int d) {
    const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(pos)) * r.turns[d];
    const int top = static_cast<int>(static_cast<unsigned int>((turn + 0x80000000ull) >> 32));
    float s, c;
    sincospif(__fmul_rn(__int2float_rn(top), 4.656612873077393e-10f), &s, &c);  // 2^-31
    return make_float2(__fmul_rn(c, r.magnitude), __fmul_rn(s, r.magnitude));
}

// Four neighbouring values as two packed f32 pairs: one instruction works on both of a pair, with each
// result rounded as its scalar form is.
using u64 = unsigned long long;
struct Quad {
    u64 a, b;
};
__device__ __forceinline__ u64 pack(float x, float y) {
    u64 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 unpack(u64 v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
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
__device__ __forceinline__ u64 fma2(u64 x, u64 y, u64 z) {
    u64 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
    return r;
}
// (x0 c - x1 s, x0 s + x1 c) of two pairs, each product and the sum rounded.  Both sums are written as
// x - y = fma(y, -1, x): the assembler joins a packed add with the product before it into one fma.
__device__ __forceinline__ void rotate2(u64 x0, u64 x1, u64 c, u64 s, u64& r0, u64& r1) {
    const u64 minus = pack(-1.f, -1.f), neg_s = s ^ 0x8000000080000000ull;
    r0 = fma2(mul2(x1, s), minus, mul2(x0, c));
    r1 = fma2(mul2(x0, neg_s), minus, mul2(x1, c));
}
__device__ __forceinline__ Quad quad(const float* p) {  // 16-byte aligned
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p);
    return {v.x, v.y};
}
// Eight neighbouring values x0 | x1, pairs of neighbours, turned by the four angles of c and s.
__device__ __forceinline__ void rotate_neighbours(Quad& x0, Quad& x1, Quad c, Quad s) {
    const float2 p0 = unpack(x0.a), p1 = unpack(x0.b), p2 = unpack(x1.a), p3 = unpack(x1.b);
    u64 e0, o0, e1, o1;
    rotate2(pack(p0.x, p1.x), pack(p0.y, p1.y), c.a, s.a, e0, o0);
    rotate2(pack(p2.x, p3.x), pack(p2.y, p3.y), c.b, s.b, e1, o1);
    const float2 a = unpack(e0), b = unpack(o0), g = unpack(e1), h = unpack(o1);
    x0 = {pack(a.x, b.x), pack(a.y, b.y)};
    x1 = {pack(g.x, h.x), pack(g.y, h.y)};
}

// Where a lane's two quads of a head are, lanes taking eight values each: of turned values four pairs.
template <bool NEIGHBOURS>
__device__ __forceinline__ void lane_quads(int l, int rot, int& a, int& b) {
    if (!NEIGHBOURS && 8 * l < rot) {
        a = 4 * l;
        b = rot / 2 + 4 * l;
    } else {
        a = 8 * l;
        b = 8 * l + 4;
    }
}

}  // namespace qkv_rope_math
