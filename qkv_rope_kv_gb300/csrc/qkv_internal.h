// Internal declarations shared by the C-ABI layer and the kernel files of
// libqkv.so.  Not part of the public interface (include/qkv.h is).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "qkv.h"

struct qkv_plan {
    qkv_plan_desc d;
    int64_t nqt, nkt, rows, half;
    int vec;  // rows can be streamed as aligned 16-byte vectors (H * elem % 16 == 0)
    float inv_freq[QKV_MAX_HEAD_DIM / 2];
};

// A qkv_rope as a launch carries it.
struct RopeTable {
    unsigned long long turns[QKV_MAX_HEAD_DIM / 2];  // of each pair a position, in 2^-64 turn
    float magnitude;
    int32_t rot;         // values of a head that are turned, from the first on
    int32_t neighbours;  // pairs (2d, 2d + 1), else (d, d + rot / 2)
};
struct qkv_rope {
    RopeTable table;
    int32_t head_dim;
    double freq[QKV_MAX_HEAD_DIM / 2];
};

// Everything one decode-layer launch needs, passed by value (__grid_constant__),
// so a captured graph node carries its own copy.
struct DecodeParams {
    const float* x;         // [H] hidden vector
    const void* w[3];       // q / k / v weight sections, row-major [rows x H]
    const float* bias[3];   // q / k / v bias sections (fused and epilogue modes)
    float* out[3];          // q / k / v outputs (in-place epilogue operands)
    void* kv_k;             // K region [n_ctx x nkt]
    void* kv_v;             // V region [n_ctx x nkt]
    const int32_t* pos;     // device position
    int32_t H, nqt, nkt, hd, n_ctx, kv_f16;
    int32_t nf;             // FusedFFN: rows per half of the gate|up weight (0 for the QKV stage)
    const float* norm_w;    // RMSNorm weight [H]: x is then the hidden state h, normalised in-kernel
    float norm_eps;         // RMSNorm epsilon
    const float* qk_norm_w[2];  // FusedQkvNorm: per-head norm weights of q and k [hd] each
    float qk_eps;               // FusedQkvNorm epsilon
    unsigned int* head_cnt;     // FusedQkvNorm: per-head completion counters [nh + nkv], zero between launches
    // Weight sections of the next layer of a model graph when it has this layer's shape, else
    // null: a read-only L2 prefetch hint (the pair ring brings its first items into L2 while
    // this layer finishes); no result depends on it.
    const void* next_w[3];
    // Test hook of the bounded waits (zero in every product call): a non-zero wait limit
    // replaces the default, and withhold_last_copy makes the ring producers skip each
    // CTA's last weight copy, so the wait for it runs out.
    unsigned long long wait_limit_ns;
    int32_t withhold_last_copy;
    float inv_freq[QKV_MAX_HEAD_DIM / 2];
};

enum DecodeMode { kProjectOnly = 0, kFused = 1 };

// decode_kernels.cu
cudaError_t launch_decode(const DecodeParams& p, int w_dtype, int vec, DecodeMode mode, bool pdl,
                          cudaStream_t stream);
cudaError_t launch_epilogue(const DecodeParams& p, cudaStream_t stream);
cudaError_t launch_chain_add_bias(float* y, const float* b, int64_t n, cudaStream_t stream);
cudaError_t launch_chain_rope(const DecodeParams& p, float* y, int n_heads, cudaStream_t stream);
cudaError_t launch_chain_store(const DecodeParams& p, const float* src, void* cache,
                               cudaStream_t stream);
cudaError_t device_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad_pos);
// FusedFFN decode: out[i] = silu((W x)[i]) * (W x)[nf + i] over the concat gate|up
// weight p.w[0] [2 nf x H] into p.out[0] [nf]; rows must be 16-byte aligned.
// Returns cudaErrorNotSupported when no ring shape fits the hidden size.
cudaError_t launch_ffn(const DecodeParams& p, int w_dtype, bool pdl, cudaStream_t stream);
// FusedQkvNorm decode: the fused stage with each q and k head RMS-normalised (weights
// p.qk_norm_w, epsilon p.qk_eps) after its bias and before its rotation; p.head_cnt is a
// zeroed workspace of nh + nkv counters, left zeroed.  Rows must be 16-byte aligned.
// Returns cudaErrorNotSupported when no ring shape fits the hidden size.
cudaError_t launch_qknorm(const DecodeParams& p, int w_dtype, bool pdl, cudaStream_t stream);
// The library's own FusedQkvNorm counters (a fixed device array of kQknormStaticHeads
// entries): their device address on the current device, looked up on first use there.
constexpr int kQknormStaticHeads = 1024;
constexpr int kQknormMaxDevices = 64;
cudaError_t qknorm_static_workspace(unsigned int** out);

// prefill_tcgen05.cu
struct PrefillParams {
    const uint16_t* X;      // [nt x H] bf16
    const uint16_t* W;      // [R x H] bf16
    const float* bias;      // [R]
    const int32_t* positions;
    float* Y;               // [nt x R]
    void* kv_k;
    void* kv_v;
    int32_t nt, H, nqt, nkt, hd, n_ctx, kv_f16;
    // Test hook of the bounded waits (zero in every product call): a non-zero wait limit
    // replaces the default, and withhold_xchg makes each CTA of a cluster of 2 skip sending its
    // partial sums to the peer, so the peer's wait for them runs out.
    unsigned long long wait_limit_ns;
    int32_t withhold_xchg;
    float inv_freq[QKV_MAX_HEAD_DIM / 2];
};
qkv_status launch_prefill(const PrefillParams& p, bool pdl, cudaStream_t stream, const char** why);
cudaError_t prefill_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad_pos);

// rope.cu
struct RopeParams {
    RopeTable rope;
    const void* x;
    void* out;
    int64_t x_stride, out_stride;
    const int32_t* positions;
    int32_t nt, n_heads, hd, inverse;
};
cudaError_t launch_rope(const RopeParams& p, int dtype, cudaStream_t stream);

// ---- paged cache (paged_store.cu, paged_attn.cu, paged_evict.cu)

// qkv_paged_kv as a launch carries it, with the plan's row width.
struct PagedView {
    void* k;
    void* v;
    const int32_t* table;  // [n_seq x max_pages]
    int32_t n_pages, page_size, n_seq, max_pages;
    int64_t page_stride;   // elements from page to page
    float* slot_weight;    // [n_seq x nkv x capacity] or null
    int32_t* slot_pos;     // the same
    int32_t nkt;
};

struct PagedStoreParams {
    PagedView c;
    const void* y;
    int64_t y_stride;
    const float* bias;       // [R] or null
    const float* norm_w[2];  // q, k norm weights [hd], or both null
    float eps;
    const int32_t* positions;
    const int32_t* seqs;   // or null: token t belongs to sequence t
    const int32_t* slots;  // or null: the slot is the position
    float* q;
    int64_t q_stride;
    int32_t nt, nh, nkv, hd, kv_f16;
    float inv_hd;  // 1 / hd
    float inv_freq[QKV_MAX_HEAD_DIM / 2];
};
// With `rope` (or null) in place of the plan's rotation.
cudaError_t launch_paged_store(const PagedStoreParams& p, const RopeTable* rope, int y_dtype, cudaStream_t stream);
cudaError_t paged_store_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);

// Workspace of qkv_attn_step.  The counters come first, in a place that no shape moves, so one
// workspace serves calls of different shapes.
constexpr int kAttnMaxCtas = 320;  // upper bound of the split grid (two CTAs on each of 152 SMs)
constexpr int kAttnHeads = 8;      // q heads of one work item
struct PagedAttnParams {
    PagedView c;
    const float* q;
    int64_t q_stride;
    const int32_t* lens;
    float scale;
    int32_t window;          // -1: each sequence's first slot is in starts (and no weights)
    void* out;
    int32_t out_bf16;
    int64_t out_stride;
    float* lse;              // [n_seq x nh] or null
    int32_t add_weight;
    unsigned int* counters;  // [3 * kAttnMaxCtas], zero between calls
    float* part;             // [2 * kAttnMaxCtas][kAttnHeads][hd padded to 64, 128 or 256, + 2]
    float* lse2;             // [n_seq x nh], log2 domain (add_weight)
    float* scores;           // [n_seq x nh x score_stride], log2 domain (add_weight)
    int64_t score_stride;    // the capacity, rounded up to whole units (32)
    int32_t nh, nkv, hd, kv_f16;
    const int32_t* starts;   // [n_seq], >= 0
};
cudaError_t launch_paged_attn(const PagedAttnParams& p, cudaStream_t stream);
// The main kernel's grid for these sizes (and pointers' alignment): CTAs, and CTAs of a cluster.
void paged_attn_grid(const PagedAttnParams& p, int* ctas, int* cluster);
cudaError_t paged_attn_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);

// Attention of many q rows over the same slots (paged_rows*.cu).  The rows (tokens x q heads of a kv head) go in tiles; the
// slots that any of a tile's rows sees, in blocks, are its units.  A kernel's CTAs get equal shares of all tiles in
// a row, kv head by kv head, each tile as long as its units and a constant for its beginning and end; so a tile's blocks can
// be spread over several CTAs, and their parts are joined afterwards.
struct alignas(16) RowTile {
    int64_t start;  // where it begins, within its kv head
    int32_t units;
    int32_t seq;    // whose row of the page table
    int32_t row0, ntok;  // q rows
    int32_t lo, hi;      // slots that are read: lo a multiple of the block
    int32_t base;        // row i sees [max(0, base + i - window), base + i); prefix: [0, row_end[row0 + i])
    int32_t all_lo, all_hi;  // slots that every row sees
};
struct alignas(16) RowPiece {  // for each CTA, the tile that begins in it and goes on in others
    int64_t start;  // of the tile, over all heads
    int32_t tile, head;
    int32_t parts;  // 0: none
};
constexpr int kRowsMaxCtas = 304;
struct PagedRowsParams {
    PagedView c;
    const float* q;
    int64_t q_stride;
    const int32_t* first;       // prompt: [n_seq + 1]; prefix: null
    const int32_t* lens;
    const int32_t* share;       // prefix: [n_seq] each
    const int32_t* prefix_len;
    float scale;
    int32_t window;
    void* out;
    int32_t out_bf16;
    int64_t out_stride;
    float* lse;
    int32_t nt, nh, nkv, hd, kv_f16;
    // the plan, made on the device
    int32_t rows, block;        // of a tile, of a unit
    int32_t per_block, blocks;  // q heads of a kv head in a tile, and how many such blocks it has
    int32_t part_rows, part_tokens;  // a tile's rows come in one or two parts, of whole tokens each (see row_of)
    int32_t tile_tokens, tile_cost, max_tiles;
    int64_t* total;             // [0] how long the tiles of one block of q heads are, [1] tiles
    RowTile* tiles;
    int32_t* starts;            // prefix: [n_seq] each: where the rows' own slots begin, ...
    int32_t* row_end;           // ... how many of the prefix are seen, ...
    int32_t* row_tile;          // ... and in which tile
    // tensor cores: q in f16 as [nt][nqt] rounded values times a power of two, the remainders, and what gives scores back
    uint16_t* q_high;
    uint16_t* q_low;            // (out F32)
    float* q_unscale;           // [nt][nh]
    RowPiece* pieces;           // [kRowsMaxCtas]
    float* part;                // [2 * kRowsMaxCtas][rows][hd + 2]
    float* prefix_out;          // prefix: [n_seq][nqt] and [n_seq][nh]: of whole tiles
    float* prefix_lse;
    const float* own_out;       // the same of the rows' own slots
    const float* own_lse;
    int32_t wait_limit_ns;      // of the tensor cores' bounded waits
    // Test hook (zero in every product call): 1 makes no piece's end known to the warps that wait for it, 2 (out F32) takes one
    // warp's waits for a block's sums for run out.
    int32_t fail;
};
cudaError_t launch_paged_rows_plan(const PagedRowsParams& p, cudaStream_t stream);
cudaError_t launch_paged_rows(const PagedRowsParams& p, cudaStream_t stream);
cudaError_t launch_paged_rows_join(const PagedRowsParams& p, cudaStream_t stream);
// Rows of a tile, slots of a block and CTAs of the kernel that these sizes and addresses get.
struct RowsShape {
    int32_t rows, part_rows, block, ctas, tile_cost;
    bool tensor;  // the kernel on the tensor cores
};
RowsShape paged_rows_shape(const PagedRowsParams& p);
RowsShape paged_rows_tc_shape(bool split);
RowsShape paged_rows_any_shape(const PagedRowsParams& p);
bool paged_rows_on_tensor_cores(const PagedRowsParams& p);
cudaError_t launch_paged_rows_tc(const PagedRowsParams& p, cudaStream_t stream);
cudaError_t paged_rows_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);
cudaError_t paged_rows_tc_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);
cudaError_t paged_rows_plan_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);

struct PagedEvictParams {
    PagedView c;
    const int32_t* lens;
    const int32_t* next_pos;
    int32_t budget, recent;
    int32_t* lens_out;
    float* weight_out;
    int32_t* pos_out;
    int32_t* moves;  // [n_seq x nkv]: how many moves an item has
    int32_t* lists;  // [n_seq x nkv][2][capacity / 2]: slots freed, slots moved
    int32_t nkv, hd, kv_f16;
};
cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream);
cudaError_t paged_evict_status_read(cudaStream_t stream, uint32_t* flags, int32_t* bad);

// qkv_api.cu: record the message of a failing call and return its status.
qkv_status api_fail(qkv_status s, const char* fmt, ...);
