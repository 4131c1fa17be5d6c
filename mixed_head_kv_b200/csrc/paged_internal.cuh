// paged_internal.cuh — the paged mixed-head cache (include/duo.h, duo_paged_*):
// its host object, the parameter blocks of its kernels and their launches.
#pragma once

#include <vector>

#include "duo_internal.cuh"

namespace duo {

constexpr int kPagedMaxBatch = DUO_PAGED_MAX_BATCH;
constexpr int kPagedMaxSeqs = DUO_PAGED_MAX_SEQS;

// Error-word bits (DUO_ERR_BIT_PAGED_* in duo.h).
constexpr uint32_t kErrPagedArgument = DUO_ERR_BIT_PAGED_ARGUMENT;
constexpr uint32_t kErrPagedCapacity = DUO_ERR_BIT_PAGED_CAPACITY;
constexpr uint32_t kErrPagedShared = DUO_ERR_BIT_PAGED_SHARED;
constexpr uint32_t kErrPagedWait = DUO_ERR_BIT_PAGED_WAIT;

// Decode CTAs that can hold partial results at a time (the workspace is sized
// before the device is known: 160 SMs x 2).
constexpr int kPagedMaxCtas = 320;

// Device addresses and sizes that every kernel of a paged cache needs.
struct PagedView {
    uint8_t* k_pages;  // [num_pages][R][P][D], R = retrieval heads of all layers
    uint8_t* v_pages;
    bf16* k_window;    // [max_seqs][S][W][D], S = streaming heads of all layers
    bf16* v_window;
    int32_t* table;    // [max_seqs][max_pages]
    int32_t* seq_len;  // [max_seqs]
    int32_t* ref;      // [num_pages]
    uint32_t* err;
    int32_t max_seqs, max_pages, num_pages, P, D, S, R, W;  // S, R: sink and recent; W = S + R
    int32_t r_all, s_all;  // retrieval / streaming heads of all layers
    int32_t elem;          // bytes per element of the pages
    int32_t P_log2;        // P is a power of two
};

// KV heads of one layer: retrieval heads first, then streaming heads, each with
// its index in the pages or the windows (consecutive within a layer).
struct PagedHeads {
    int32_t n_retr, n_strm;
    int32_t r0, s0;  // index of the layer's first retrieval / streaming head
    int16_t head[DUO_MAX_KV_HEADS];
};

// ------------------------------------------------------------------ page upkeep
struct PagePlan {           // what a planning kernel leaves for the copy kernel
    int32_t n_pages;        // page pairs to copy
    int32_t n_seqs;         // window pairs to copy (entries with src < 0 are skipped)
    int32_t used;           // compact: pages in use (0: leave the table alone)
    int32_t pad;
    int2 seq[kPagedMaxBatch];  // (src, dst) windows
    uint32_t arrived[kPagedMaxBatch];  // fork: CTAs of the entry that have looked at it; 0 between calls
};
struct PageOps {
    PagedView v;
    PagePlan* plan;
    int2* pair;     // [num_pages] (src, dst) pages
    int32_t* list;  // [num_pages] free pages in ascending order / new page numbers
    int32_t n;
    const int32_t* a;  // seqs or src
    const int32_t* b;  // n_tok or dst
};
cudaError_t launch_paged_extend(const PageOps& p, int num_sms, cudaStream_t s);
cudaError_t launch_paged_fork(const PageOps& p, int num_sms, cudaStream_t s);
cudaError_t launch_paged_copy(const PageOps& p, int num_sms, cudaStream_t s);
cudaError_t launch_paged_release(const PageOps& p, cudaStream_t s);
cudaError_t launch_paged_compact(const PageOps& p, int num_sms, cudaStream_t s);

// E4M3 scales of one layer: [Hkv][k_scale, v_scale, 1/k_scale, 1/v_scale]. They
// travel in the launch, so nothing on the host has to outlive the call.
struct PagedScales {
    float value[DUO_MAX_KV_HEADS * 4];
};
cudaError_t launch_paged_set_scales(float* dst, const PagedScales& x, int n, cudaStream_t s);
cudaError_t launch_paged_unit_scales(float* dst, int n, cudaStream_t s);

// ------------------------------------------------------------------ append
struct PagedAppendParams {
    PagedView v;
    PagedHeads h;
    const bf16* k;
    const bf16* v_rows;
    int64_t n_rows, kv_stride;
    const int32_t* seqs;
    const int32_t* row_start;
    int32_t n, fp8;
    const float* kv_scale;  // fp8: [Hkv][k_scale, v_scale, 1/k_scale, 1/v_scale]
};
cudaError_t launch_paged_append(const PagedAppendParams& p, int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ decode
struct PagedDecodeParams {
    PagedView v;
    PagedHeads h;
    const bf16* q;
    const bf16* k_new;
    const bf16* v_new;
    bf16* out;
    int64_t q_stride, kv_stride, out_stride;
    const int32_t* seqs;
    int32_t n, Hq, Hkv, G;
    float scale_log2;
    const float* kv_scale;
    float* part_o;       // [kPagedMaxCtas][2][G][D]
    float* part_ml;      // [kPagedMaxCtas][2][G][2] running maximum and sum
    uint32_t* counters;  // [kPagedMaxBatch * Hkv], zero between launches
    int32_t test_withhold;  // 1: a test of the bounded waits (duo_paged_test_wait_timeout)
};
struct PagedMaps {
    CUtensorMap k, v;    // pages (D, P, num_pages * R)
    CUtensorMap wk, wv;  // windows (D, W, max_seqs * S), box of 64 rows
};
cudaError_t launch_paged_decode(const PagedDecodeParams& p, const PagedMaps& m, int fp8, int num_sms, cudaStream_t s);

// ------------------------------------------------------------------ packed prompts
struct PackedPrefillParams {
    bf16* out;
    const bf16* v;
    int64_t kv_stride;
    const int32_t* row_start;
    uint32_t* err;
    uint32_t* work;  // [0] next work item, [1] CTAs done; zero between launches
    int64_t n_rows, out_stride;
    int32_t n, Hq, Hkv, G, D, S, R;
    float scale_log2;
    int32_t test_withhold;  // 1: a test of the bounded waits (duo_paged_test_wait_timeout)
    PagedHeads h;
};
struct PackedMaps {
    CUtensorMap q, k, v;  // (D, heads, rows), box (64, 1, 128)
};
cudaError_t launch_prefill_packed(const PackedPrefillParams& p, const PackedMaps& m, int num_sms, cudaStream_t s);

// Tensor-map encoding (duo_abi.cu): bf16 or one-byte elements, `rank` dimensions
// innermost first, byte strides of dimensions 1 .. rank - 1.
bool encode_map(CUtensorMap* m, bool bytes, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                const uint32_t* box, CUtensorMapSwizzle swizzle);

}  // namespace duo

// Host object behind the opaque duo_paged handle.
struct duo_paged {
    duo_paged_layout lay;
    int32_t G = 1;
    float scale = 0.f;
    int device = 0;
    int num_sms = 148;
    bool fp8 = false;
    int32_t test_wait = 0;               // duo_paged_test_wait_timeout: launch kinds still to withhold tiles
    duo::PagedView view{};
    std::vector<duo::PagedHeads> heads;  // [layers]
    duo::PagedMaps maps{};
    duo::PagePlan* plan = nullptr;
    int2* pair = nullptr;
    int32_t* list = nullptr;
    float* part_o = nullptr;
    float* part_ml = nullptr;
    uint32_t* counters = nullptr;
    uint32_t* work = nullptr;
    float* kv_scales = nullptr;          // device [layers][Hkv][4]
};
