// C-ABI layer of the rotations of include/qkv.h that are not the plan's: frequencies (host, 64 bits) and
// argument validation; the kernels are in rope.cu.
#include <cmath>
#include <cstring>
#include <new>

#include "qkv_internal.h"

namespace {

#define REQUIRE(cond, ...)                                              \
    do {                                                                \
        if (!(cond)) return api_fail(QKV_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

bool positive(double v) { return std::isfinite(v) && v > 0.0; }

constexpr double kTwoPi = 6.283185307179586;

// f of pair d, as include/qkv.h defines it.
double frequency(const qkv_rope_desc& c, int d) {
    const double rot = c.rot_dim;
    const double theta = c.scaling == QKV_ROPE_SCALE_BASE ? c.theta * std::pow(c.factor, rot / (rot - 2.0)) : c.theta;
    const double f = std::pow(theta, -2.0 * d / rot);
    switch (c.scaling) {
        case QKV_ROPE_SCALE_LINEAR: return f / c.factor;
        case QKV_ROPE_SCALE_RAMP: {
            const auto at = [&](double turns) { return rot * std::log(c.orig_ctx / (kTwoPi * turns)) / (2.0 * std::log(c.theta)); };
            const double lo = std::fmax(0.0, std::floor(at(c.high))), hi = std::fmin(rot - 1.0, std::ceil(at(c.low)));
            const double g = std::fmin(1.0, std::fmax(0.0, (d - lo) / std::fmax(hi - lo, 0.001)));
            return f / c.factor * g + f * (1.0 - g);
        }
        case QKV_ROPE_SCALE_BANDS: {
            const double g = std::fmin(1.0, std::fmax(0.0, (c.orig_ctx * f / kTwoPi - c.low) / (c.high - c.low)));
            return (1.0 - g) * f / c.factor + g * f;
        }
        case QKV_ROPE_SCALE_TABLE: return f / c.divisors[d];
        default: return f;
    }
}

// f / (2 pi) without its whole turns, in 2^-64 turn: 1 / (2 pi) in two parts, so that nothing of a double is lost.
unsigned long long turns(double f) {
    constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;
    const double q = f * hi, rest = std::fma(f, hi, -q) + f * lo;
    const double part = q - std::floor(q), more = std::ldexp(rest, 64);
    unsigned long long t = static_cast<unsigned long long>(std::ldexp(part, 64));  // part < 1
    return t + static_cast<unsigned long long>(static_cast<long long>(std::nearbyint(more)));
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

extern "C" qkv_status qkv_rope_create(const qkv_rope_desc* d, qkv_rope** out) {
    REQUIRE(out, "out is null");
    *out = nullptr;
    REQUIRE(d, "desc is null");
    REQUIRE(d->head_dim >= 2 && d->head_dim <= QKV_MAX_HEAD_DIM, "head_dim must be in [2, %d] (got %d)", QKV_MAX_HEAD_DIM,
            d->head_dim);
    REQUIRE(d->rot_dim >= 2 && d->rot_dim <= d->head_dim && d->rot_dim % 2 == 0,
            "rot_dim must be even and in [2, head_dim = %d] (got %d)", d->head_dim, d->rot_dim);
    REQUIRE(d->layout == QKV_ROPE_NEOX || d->layout == QKV_ROPE_INTERLEAVED, "unknown rope layout %d", d->layout);
    REQUIRE(positive(d->theta), "theta must be finite and > 0");
    REQUIRE(positive(d->magnitude) && positive(static_cast<float>(d->magnitude)),
            "magnitude must be a finite f32 number > 0");
    const int s = d->scaling;
    REQUIRE(s >= QKV_ROPE_SCALE_NONE && s <= QKV_ROPE_SCALE_TABLE, "unknown rope scaling %d", s);
    const bool parts = s == QKV_ROPE_SCALE_RAMP || s == QKV_ROPE_SCALE_BANDS;
    if (s == QKV_ROPE_SCALE_LINEAR || s == QKV_ROPE_SCALE_BASE || parts)
        REQUIRE(positive(d->factor), "factor must be finite and > 0");
    if (s == QKV_ROPE_SCALE_BASE) REQUIRE(d->rot_dim >= 4, "BASE scaling needs rot_dim >= 4");
    if (parts) {
        REQUIRE(positive(d->orig_ctx), "orig_ctx must be finite and > 0");
        REQUIRE(positive(d->low) && std::isfinite(d->high) && d->high > d->low, "0 < low < high must hold");
    }
    if (s == QKV_ROPE_SCALE_RAMP) REQUIRE(d->theta > 1.0, "RAMP scaling needs theta > 1");
    if (s == QKV_ROPE_SCALE_TABLE) {
        REQUIRE(d->divisors, "divisors is null");
        for (int i = 0; i < d->rot_dim / 2; ++i) REQUIRE(positive(d->divisors[i]), "divisors[%d] must be finite and > 0", i);
    }
    qkv_rope* r = new (std::nothrow) qkv_rope;
    if (!r) return api_fail(QKV_ERR_INVALID_ARG, "out of host memory");
    std::memset(r, 0, sizeof *r);
    r->head_dim = d->head_dim;
    r->table.rot = d->rot_dim;
    r->table.neighbours = d->layout == QKV_ROPE_INTERLEAVED;
    r->table.magnitude = static_cast<float>(d->magnitude);
    for (int i = 0; i < d->rot_dim / 2; ++i) {
        const double f = frequency(*d, i);
        // beyond 2^52 radians a position no fraction of a turn is left of a double
        if (!(f >= 0.0 && f <= 4503599627370496.0)) {
            delete r;
            return api_fail(QKV_ERR_INVALID_ARG, "the frequency of pair %d is out of range", i);
        }
        r->freq[i] = f;
        r->table.turns[i] = turns(f);
    }
    *out = r;
    return QKV_OK;
}

extern "C" void qkv_rope_destroy(qkv_rope* r) { delete r; }

extern "C" qkv_status qkv_rope_freqs(const qkv_rope* r, double* out_host, int32_t n) {
    REQUIRE(r, "rope is null");
    REQUIRE(out_host, "out_host is null");
    REQUIRE(n == r->table.rot / 2, "n must be rot_dim/2 = %d (got %d)", r->table.rot / 2, n);
    std::memcpy(out_host, r->freq, sizeof(double) * n);
    return QKV_OK;
}

extern "C" qkv_status qkv_rope_step(const qkv_rope* rope, const qkv_rope_args* a, void* stream) {
    REQUIRE(rope, "rope is null");
    REQUIRE(a, "args is null");
    REQUIRE(a->nt >= 0, "nt must be >= 0");
    REQUIRE(a->n_heads >= 1, "n_heads must be >= 1");
    if (a->dtype != QKV_F32 && a->dtype != QKV_BF16 && a->dtype != QKV_F16)
        return api_fail(QKV_ERR_UNSUPPORTED, "dtype %d not supported (F32, BF16 or F16)", a->dtype);
    const int64_t row = static_cast<int64_t>(a->n_heads) * rope->head_dim;
    REQUIRE(a->x_stride >= row && a->out_stride >= row, "x_stride and out_stride must be >= n_heads * head_dim = %lld",
            static_cast<long long>(row));
    if (a->nt == 0) return QKV_OK;
    REQUIRE(a->x && a->out && a->d_positions, "x, out or d_positions is null");
    REQUIRE(a->nt <= (int64_t(1) << 38) / row, "nt * n_heads * head_dim must be at most 2^38");
    const size_t es = a->dtype == QKV_F32 ? 4 : 2;
    REQUIRE(reinterpret_cast<uintptr_t>(a->x) % es == 0 && reinterpret_cast<uintptr_t>(a->out) % es == 0 &&
                reinterpret_cast<uintptr_t>(a->d_positions) % 4 == 0,
            "a pointer is not aligned to its elements");
    const size_t xb = ((a->nt - 1) * static_cast<size_t>(a->x_stride) + row) * es;
    const size_t ob = ((a->nt - 1) * static_cast<size_t>(a->out_stride) + row) * es;
    REQUIRE((a->x == a->out && (a->x_stride == a->out_stride || a->nt == 1)) || !overlap(a->x, xb, a->out, ob),
            "out must be x itself (the same stride where there are rows to step over) or not overlap it");
    REQUIRE(!overlap(a->d_positions, 4 * static_cast<size_t>(a->nt), a->out, ob), "out must not overlap d_positions");
    RopeParams p;
    std::memset(&p, 0, sizeof p);
    p.rope = rope->table;
    p.x = a->x;
    p.out = a->out;
    p.x_stride = a->x_stride;
    p.out_stride = a->out_stride;
    p.positions = a->d_positions;
    p.nt = a->nt;
    p.n_heads = a->n_heads;
    p.hd = rope->head_dim;
    p.inverse = a->inverse != 0;
    const cudaError_t e = launch_rope(p, a->dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess)
        return api_fail(QKV_ERR_CUDA, "rope kernel launch: %s (%s)", cudaGetErrorName(e), cudaGetErrorString(e));
    return QKV_OK;
}
