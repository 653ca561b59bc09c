// C-ABI layer of the paged-cache entry points: argument validation and workspace layout
// (include/qkv.h has the contracts; the kernels are in paged_store.cu, paged_attn.cu and
// paged_evict.cu).
#include <cmath>
#include <cstring>

#include "qkv_internal.h"
#include "qkv_test.h"

namespace {

#define REQUIRE(cond, ...)                                              \
    do {                                                                \
        if (!(cond)) return api_fail(QKV_ERR_INVALID_ARG, __VA_ARGS__); \
    } while (0)

qkv_status cuda_fail(cudaError_t e, const char* what) {
    return api_fail(QKV_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int64_t capacity(const qkv_paged_kv* c) { return static_cast<int64_t>(c->max_pages) * c->page_size; }

constexpr int64_t kMaxCapacity = int64_t(1) << 30;  // slots and what kernels round up from them stay in 32 bits

// Sizes only (what the workspace queries need).
qkv_status check_shape(const qkv_plan* plan, const qkv_paged_kv* c) {
    REQUIRE(plan, "plan is null");
    REQUIRE(c, "cache is null");
    REQUIRE(c->n_pages >= 1 && c->page_size >= 1 && c->n_seq >= 1 && c->max_pages >= 1,
            "n_pages, page_size, n_seq and max_pages must be >= 1 (got %d, %d, %d, %d)", c->n_pages, c->page_size,
            c->n_seq, c->max_pages);
    REQUIRE(capacity(c) <= kMaxCapacity, "max_pages * page_size must be at most 2^30");
    REQUIRE(static_cast<int64_t>(c->n_seq) * (plan->d.n_head + plan->d.n_head_kv) <= (int64_t(1) << 24),
            "n_seq * heads must be at most 2^24");
    const int64_t page = static_cast<int64_t>(c->page_size) * plan->nkt;
    REQUIRE(c->page_stride == 0 || c->page_stride >= page, "page_stride must be 0 or >= page_size * nkt = %lld",
            static_cast<long long>(page));
    return QKV_OK;
}

qkv_status view(const qkv_plan* plan, const qkv_paged_kv* c, PagedView* v) {
    qkv_status st = check_shape(plan, c);
    if (st != QKV_OK) return st;
    REQUIRE(c->k && c->v, "a page pool pointer is null");
    REQUIRE(c->page_table, "page_table is null");
    const uintptr_t es = plan->d.kv_dtype == QKV_F16 ? 2 : 4;
    REQUIRE(aligned(c->k, es) && aligned(c->v, es), "the page pools must be aligned to their elements");
    REQUIRE(aligned(c->page_table, 4) && aligned(c->slot_weight, 4) && aligned(c->slot_pos, 4),
            "page_table, slot_weight and slot_pos must be 4-byte aligned");
    v->k = c->k;
    v->v = c->v;
    v->table = c->page_table;
    v->n_pages = c->n_pages;
    v->page_size = c->page_size;
    v->n_seq = c->n_seq;
    v->max_pages = c->max_pages;
    v->page_stride = c->page_stride ? c->page_stride : static_cast<int64_t>(c->page_size) * plan->nkt;
    v->slot_weight = c->slot_weight;
    v->slot_pos = c->slot_pos;
    v->nkt = static_cast<int32_t>(plan->nkt);
    return QKV_OK;
}

size_t up256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Floats of a row of scores: whole units of slots, 16-byte aligned rows.
int64_t score_stride(const qkv_paged_kv* c) { return (capacity(c) + 31) & ~static_cast<int64_t>(31); }

// Byte offsets of the parts of qkv_attn_step's workspace.
struct AttnLayout {
    size_t part, lse2, scores, total;
};
AttnLayout attn_layout(const qkv_plan* plan, const qkv_paged_kv* c, bool weights) {
    AttnLayout l;
    const size_t rows = static_cast<size_t>(c->n_seq) * plan->d.n_head;
    const size_t hd = plan->d.head_dim <= 64 ? 64 : plan->d.head_dim <= 128 ? 128 : 256;  // as the kernels pad it
    l.part = up256(3 * kAttnMaxCtas * sizeof(uint32_t));
    static_assert(3 * kAttnMaxCtas * sizeof(uint32_t) <= 4096, "the counters are in what a caller has to zero");
    l.lse2 = l.part + up256(sizeof(float) * 2 * kAttnMaxCtas * kAttnHeads * (hd + 2));
    l.scores = l.lse2 + (weights ? up256(sizeof(float) * rows) : 0);
    l.total = l.scores + (weights ? up256(sizeof(float) * rows * score_stride(c)) : 0);
    return l;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

}  // namespace

extern "C" qkv_status qkv_paged_store_step(const qkv_plan* plan, const qkv_paged_kv* cache,
                                           const qkv_paged_store_args* a, void* stream) {
    PagedStoreParams p;
    std::memset(&p, 0, sizeof p);
    qkv_status st = view(plan, cache, &p.c);
    if (st != QKV_OK) return st;
    REQUIRE(a, "args is null");
    REQUIRE(a->nt >= 0, "nt must be >= 0");
    if (a->y_dtype != QKV_F32 && a->y_dtype != QKV_BF16)
        return api_fail(QKV_ERR_UNSUPPORTED, "y_dtype %d not supported (F32 or BF16)", a->y_dtype);
    REQUIRE(a->nt == 0 || (a->Y && a->q && a->d_positions), "Y, q or d_positions is null");
    REQUIRE(a->y_stride >= plan->rows, "y_stride must be >= R = %lld", static_cast<long long>(plan->rows));
    REQUIRE(a->q_stride >= plan->nqt, "q_stride must be >= nqt = %lld", static_cast<long long>(plan->nqt));
    REQUIRE((a->q_norm_w == nullptr) == (a->k_norm_w == nullptr), "q_norm_w and k_norm_w: both or neither");
    if (a->q_norm_w) REQUIRE(a->eps >= 0.f && std::isfinite(a->eps), "eps must be finite and >= 0");
    REQUIRE(a->d_seqs || a->nt <= cache->n_seq, "without d_seqs, nt must be <= n_seq");
    const int ys = a->y_dtype == QKV_F32 ? 4 : 2;
    REQUIRE(aligned(a->Y, ys) && aligned(a->q, 4) && aligned(a->bias, 4) && aligned(a->q_norm_w, 4) &&
                aligned(a->k_norm_w, 4) && aligned(a->d_positions, 4) && aligned(a->d_seqs, 4) && aligned(a->d_slots, 4),
            "a pointer is not aligned to its elements");
    const size_t ybytes = a->nt ? ((a->nt - 1) * static_cast<size_t>(a->y_stride) + plan->rows) * ys : 0;
    const size_t qbytes = a->nt ? ((a->nt - 1) * static_cast<size_t>(a->q_stride) + plan->nqt) * 4 : 0;
    const bool in_place = a->Y == a->q && a->y_dtype == QKV_F32 && (a->y_stride == a->q_stride || a->nt == 1);
    REQUIRE(in_place || !overlap(a->Y, ybytes, a->q, qbytes),
            "q must be Y itself (F32, the same stride where there are rows to step over) or not overlap it");
    if (a->nt == 0) return QKV_OK;
    p.y = a->Y;
    p.y_stride = a->y_stride;
    p.bias = a->bias;
    p.norm_w[0] = a->q_norm_w;
    p.norm_w[1] = a->k_norm_w;
    p.eps = a->eps;
    p.positions = a->d_positions;
    p.seqs = a->d_seqs;
    p.slots = a->d_slots;
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.nt = a->nt;
    p.nh = plan->d.n_head;
    p.nkv = plan->d.n_head_kv;
    p.hd = plan->d.head_dim;
    p.kv_f16 = plan->d.kv_dtype == QKV_F16 ? 1 : 0;
    p.inv_hd = 1.f / static_cast<float>(p.hd);
    std::memcpy(p.inv_freq, plan->inv_freq, sizeof p.inv_freq);
    const cudaError_t e = launch_paged_store(p, a->y_dtype, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged store kernel launch");
    return QKV_OK;
}

extern "C" qkv_status qkv_attn_workspace_bytes(const qkv_plan* plan, const qkv_paged_kv* cache, size_t* out) {
    qkv_status st = check_shape(plan, cache);
    if (st != QKV_OK) return st;
    REQUIRE(out, "out is null");
    *out = attn_layout(plan, cache, cache->slot_weight != nullptr).total;
    return QKV_OK;
}

extern "C" qkv_status qkv_attn_step(const qkv_plan* plan, const qkv_paged_kv* cache, const qkv_attn_args* a,
                                    void* stream) {
    PagedAttnParams p;
    std::memset(&p, 0, sizeof p);
    qkv_status st = view(plan, cache, &p.c);
    if (st != QKV_OK) return st;
    REQUIRE(a, "args is null");
    if (plan->d.n_head % plan->d.n_head_kv != 0)
        return api_fail(QKV_ERR_UNSUPPORTED, "n_head %d is not a multiple of n_head_kv %d", plan->d.n_head,
                        plan->d.n_head_kv);
    if (a->out_dtype != QKV_F32 && a->out_dtype != QKV_BF16)
        return api_fail(QKV_ERR_UNSUPPORTED, "out_dtype %d not supported (F32 or BF16)", a->out_dtype);
    REQUIRE(a->q && a->d_lens && a->out, "q, d_lens or out is null");
    REQUIRE(a->q_stride >= plan->nqt && a->out_stride >= plan->nqt, "q_stride and out_stride must be >= nqt = %lld",
            static_cast<long long>(plan->nqt));
    REQUIRE(std::isfinite(a->scale), "scale must be finite");
    REQUIRE(a->window >= 0, "window must be >= 0");
    REQUIRE(!a->add_weight || cache->slot_weight, "add_weight needs a cache with slot_weight");
    const int os = a->out_dtype == QKV_F32 ? 4 : 2;
    REQUIRE(aligned(a->q, 4) && aligned(a->d_lens, 4) && aligned(a->lse, 4) && aligned(a->out, os),
            "a pointer is not aligned to its elements");
    const size_t rows = static_cast<size_t>(cache->n_seq);
    REQUIRE(!overlap(a->q, ((rows - 1) * a->q_stride + plan->nqt) * 4, a->out,
                     ((rows - 1) * a->out_stride + plan->nqt) * os),
            "out must not overlap q");
    const AttnLayout l = attn_layout(plan, cache, a->add_weight != 0);
    REQUIRE(a->d_workspace && aligned(a->d_workspace, 16), "d_workspace must be a 16-byte aligned pointer");
    REQUIRE(a->workspace_bytes >= l.total, "the workspace has %zu bytes, %zu are needed", a->workspace_bytes, l.total);
    char* ws = static_cast<char*>(a->d_workspace);
    p.q = a->q;
    p.q_stride = a->q_stride;
    p.lens = a->d_lens;
    p.scale = a->scale;
    p.window = a->window;
    p.out = a->out;
    p.out_bf16 = a->out_dtype == QKV_BF16;
    p.out_stride = a->out_stride;
    p.lse = a->lse;
    p.add_weight = a->add_weight != 0;
    p.counters = reinterpret_cast<unsigned int*>(ws);
    p.part = reinterpret_cast<float*>(ws + l.part);
    p.lse2 = reinterpret_cast<float*>(ws + l.lse2);
    p.scores = reinterpret_cast<float*>(ws + l.scores);
    p.score_stride = score_stride(cache);
    p.nh = plan->d.n_head;
    p.nkv = plan->d.n_head_kv;
    p.hd = plan->d.head_dim;
    p.kv_f16 = plan->d.kv_dtype == QKV_F16 ? 1 : 0;
    const cudaError_t e = launch_paged_attn(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "paged attention kernel launch");
    return QKV_OK;
}

// Test hook (include/qkv_test.h).
extern "C" qkv_status qkv_test_attn_grid(const qkv_plan* plan, const qkv_paged_kv* cache, int32_t* ctas,
                                         int32_t* cluster) {
    PagedAttnParams p;
    std::memset(&p, 0, sizeof p);
    qkv_status st = view(plan, cache, &p.c);
    if (st != QKV_OK) return st;
    if (plan->d.n_head % plan->d.n_head_kv != 0) return api_fail(QKV_ERR_UNSUPPORTED, "uneven groups of q heads");
    REQUIRE(ctas && cluster, "ctas or cluster is null");
    p.nh = plan->d.n_head;
    p.nkv = plan->d.n_head_kv;
    p.hd = plan->d.head_dim;
    p.kv_f16 = plan->d.kv_dtype == QKV_F16 ? 1 : 0;
    paged_attn_grid(p, ctas, cluster);
    return QKV_OK;
}

extern "C" qkv_status qkv_evict_workspace_bytes(const qkv_plan* plan, const qkv_paged_kv* cache, size_t* out) {
    qkv_status st = check_shape(plan, cache);
    if (st != QKV_OK) return st;
    REQUIRE(out, "out is null");
    *out = sizeof(int32_t) * (1 + 2 * static_cast<size_t>(capacity(cache) / 2)) * cache->n_seq * plan->d.n_head_kv;
    return QKV_OK;
}

extern "C" qkv_status qkv_evict_step(const qkv_plan* plan, const qkv_paged_kv* cache, const qkv_evict_args* a,
                                     void* stream) {
    PagedEvictParams p;
    std::memset(&p, 0, sizeof p);
    qkv_status st = view(plan, cache, &p.c);
    if (st != QKV_OK) return st;
    REQUIRE(a, "args is null");
    REQUIRE(cache->slot_weight && cache->slot_pos, "the cache must have slot_weight and slot_pos");
    REQUIRE(a->d_lens && a->d_next_pos && a->lens_out && a->weight_out && a->pos_out, "null pointer");
    REQUIRE(a->budget >= 1, "budget must be >= 1");
    REQUIRE(a->recent >= 0 && a->recent <= a->budget, "recent must be in [0, budget]");
    REQUIRE(aligned(a->d_lens, 4) && aligned(a->d_next_pos, 4) && aligned(a->lens_out, 4) && aligned(a->weight_out, 4) &&
                aligned(a->pos_out, 4),
            "a pointer is not 4-byte aligned");
    const size_t nb = sizeof(int32_t) * cache->n_seq;
    REQUIRE(!overlap(a->d_lens, nb, a->lens_out, nb) && !overlap(a->d_next_pos, nb, a->lens_out, nb),
            "lens_out must not overlap d_lens or d_next_pos");
    const size_t sb = 4 * static_cast<size_t>(capacity(cache)) * cache->n_seq * plan->d.n_head_kv;
    REQUIRE((a->weight_out == cache->slot_weight || !overlap(a->weight_out, sb, cache->slot_weight, sb)) &&
                (a->pos_out == cache->slot_pos || !overlap(a->pos_out, sb, cache->slot_pos, sb)),
            "weight_out and pos_out must be slot_weight and slot_pos themselves or not overlap them");
    REQUIRE(!overlap(a->weight_out, sb, a->pos_out, sb) && !overlap(a->weight_out, sb, cache->slot_pos, sb) &&
                !overlap(a->pos_out, sb, cache->slot_weight, sb),
            "weight_out must not overlap pos_out or slot_pos, nor pos_out slot_weight");
    size_t need = 0;
    st = qkv_evict_workspace_bytes(plan, cache, &need);
    if (st != QKV_OK) return st;
    REQUIRE(a->workspace_bytes >= need && a->d_workspace, "the workspace has %zu bytes, %zu are needed",
            a->workspace_bytes, need);
    REQUIRE(aligned(a->d_workspace, 4), "d_workspace must be 4-byte aligned");
    p.lens = a->d_lens;
    p.next_pos = a->d_next_pos;
    p.budget = a->budget;
    p.recent = a->recent;
    p.lens_out = a->lens_out;
    p.weight_out = a->weight_out;
    p.pos_out = a->pos_out;
    p.moves = static_cast<int32_t*>(a->d_workspace);
    p.lists = p.moves + static_cast<size_t>(cache->n_seq) * plan->d.n_head_kv;
    p.nkv = plan->d.n_head_kv;
    p.hd = plan->d.head_dim;
    p.kv_f16 = plan->d.kv_dtype == QKV_F16 ? 1 : 0;
    const cudaError_t e = launch_paged_evict(p, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "eviction kernel launch");
    return QKV_OK;
}
