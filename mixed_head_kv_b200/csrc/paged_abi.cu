// paged_abi.cu — the C ABI of the paged cache (include/duo.h, duo_paged_*):
// argument checks, workspace carving, tensor maps and launches. No device memory
// is allocated and no call waits for the device, but duo_paged_error.
#include <cmath>
#include <cstring>
#include <new>

#include "paged_internal.cuh"

using namespace duo;

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }

struct Workspace {
    size_t err, plan, pair, list, part_o, part_ml, counters, scales, total;
};

Workspace workspace_for(const duo_paged_layout& L) {
    Workspace w{};
    const size_t G = static_cast<size_t>(L.num_q_heads / L.num_kv_heads);
    w.err = kAlign;  // error word, then the packed prefill's two counters
    w.plan = align_up(sizeof(PagePlan));
    w.pair = align_up(static_cast<size_t>(L.num_pages) * sizeof(int2));
    w.list = align_up(static_cast<size_t>(L.num_pages) * sizeof(int32_t));
    w.part_o = align_up(static_cast<size_t>(kPagedMaxCtas) * 2 * G * L.head_dim * sizeof(float));
    w.part_ml = align_up(static_cast<size_t>(kPagedMaxCtas) * 2 * G * 2 * sizeof(float));
    w.counters = align_up(static_cast<size_t>(kPagedMaxBatch) * L.num_kv_heads * sizeof(uint32_t));
    w.scales = align_up(static_cast<size_t>(L.num_layers) * L.num_kv_heads * 4 * sizeof(float));
    w.total = w.err + w.plan + w.pair + w.list + w.part_o + w.part_ml + w.counters + w.scales;
    return w;
}

duo_status check_layout(const duo_paged_layout* L, const uint8_t* mask, int64_t* n_retr, int64_t* n_strm) {
    if (!L || !mask) return DUO_ERR_INVALID_ARG;
    if (L->num_layers < 1 || L->num_layers > (1 << 16)) return DUO_ERR_INVALID_ARG;
    if (L->max_seqs < 1 || L->max_seqs > DUO_PAGED_MAX_SEQS) return DUO_ERR_INVALID_ARG;
    if (L->num_kv_heads < 1 || L->num_kv_heads > DUO_MAX_KV_HEADS) return DUO_ERR_INVALID_ARG;
    if (L->num_q_heads < 1 || L->num_q_heads > DUO_MAX_Q_HEADS) return DUO_ERR_INVALID_ARG;
    if (L->num_q_heads % L->num_kv_heads != 0) return DUO_ERR_INVALID_ARG;
    if (L->num_q_heads / L->num_kv_heads > DUO_PAGED_MAX_GROUP) return DUO_ERR_INVALID_ARG;
    if (L->head_dim != 64 && L->head_dim != 128) return DUO_ERR_INVALID_ARG;
    if (L->sink < 0 || L->recent < 1) return DUO_ERR_INVALID_ARG;
    if (static_cast<int64_t>(L->sink) + L->recent > (1 << 24)) return DUO_ERR_INVALID_ARG;
    if (L->kv_format != DUO_KV_BF16 && L->kv_format != DUO_KV_E4M3) return DUO_ERR_INVALID_ARG;
    if (L->page_size != 16 && L->page_size != 32 && L->page_size != 64 && L->page_size != 128)
        return DUO_ERR_INVALID_ARG;
    if (L->num_pages < 1 || L->num_pages > DUO_PAGED_MAX_PAGES) return DUO_ERR_INVALID_ARG;
    if (L->max_pages < 1 || static_cast<int64_t>(L->max_pages) * L->page_size > (1 << 27)) return DUO_ERR_INVALID_ARG;
    if (!(L->softmax_scale >= 0.f) || !std::isfinite(L->softmax_scale)) return DUO_ERR_INVALID_ARG;
    const int64_t n = static_cast<int64_t>(L->num_layers) * L->num_kv_heads;
    int64_t r = 0;
    for (int64_t i = 0; i < n; ++i) {
        if (mask[i] > 1) return DUO_ERR_INVALID_ARG;
        r += mask[i];
    }
    // Tensor-map coordinates (page, head) and (sequence, head) are 32 bits wide.
    if (static_cast<int64_t>(L->num_pages) * r > INT32_MAX) return DUO_ERR_INVALID_ARG;
    if (static_cast<int64_t>(L->max_seqs) * (n - r) > INT32_MAX) return DUO_ERR_INVALID_ARG;
    *n_retr = r;
    *n_strm = n - r;
    return DUO_OK;
}

duo_paged_sizes sizes_for(const duo_paged_layout& L, int64_t n_retr, int64_t n_strm) {
    duo_paged_sizes s{};
    const size_t elem = L.kv_format == DUO_KV_E4M3 ? 1 : 2;
    s.pages = static_cast<size_t>(L.num_pages) * n_retr * L.page_size * L.head_dim * elem;
    s.windows = static_cast<size_t>(L.max_seqs) * n_strm * (static_cast<size_t>(L.sink) + L.recent) * L.head_dim * 2;
    s.page_table = static_cast<size_t>(L.max_seqs) * L.max_pages * sizeof(int32_t);
    s.seq_len = static_cast<size_t>(L.max_seqs) * sizeof(int32_t);
    s.page_ref = static_cast<size_t>(L.num_pages) * sizeof(int32_t);
    s.workspace = workspace_for(L).total;
    return s;
}

duo_status check_device(const duo_paged* c) {
    if (!c) return DUO_ERR_INVALID_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess) return DUO_ERR_CUDA;
    return dev == c->device ? DUO_OK : DUO_ERR_STATE;
}

// n entries, with the device arrays they need.
duo_status check_entries(const duo_paged* c, int32_t n, const void* a, const void* b) {
    if (!c || n < 0 || n > DUO_PAGED_MAX_BATCH) return DUO_ERR_INVALID_ARG;
    if (n > 0 && (!a || !b)) return DUO_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(a) & 3u) != 0 || (reinterpret_cast<uintptr_t>(b) & 3u) != 0)
        return DUO_ERR_ALIGNMENT;
    return check_device(c);
}

// A row stride in elements: 0 selects dense rows.
bool row_stride(int64_t given, int64_t heads, int64_t D, int64_t* out) {
    const int64_t dense = heads * D;
    *out = given == 0 ? dense : given;
    return given == 0 || (given >= dense && given % 8 == 0 && given <= INT32_MAX);
}

bool layer_ok(const duo_paged* c, int32_t layer) { return c && layer >= 0 && layer < c->lay.num_layers; }

const float* scales_of(const duo_paged* c, int32_t layer) {
    return c->kv_scales + static_cast<size_t>(layer) * c->lay.num_kv_heads * 4;
}

PageOps page_ops(const duo_paged* c, int32_t n, const int32_t* a, const int32_t* b) {
    PageOps p{};
    p.v = c->view;
    p.plan = c->plan;
    p.pair = c->pair;
    p.list = c->list;
    p.n = n;
    p.a = a;
    p.b = b;
    return p;
}

bool packed_map(CUtensorMap* m, const void* base, int64_t D, int64_t heads, int64_t rows, int64_t stride) {
    const uint64_t dims[3] = {static_cast<uint64_t>(D), static_cast<uint64_t>(heads), static_cast<uint64_t>(rows)};
    const uint64_t strides[2] = {static_cast<uint64_t>(D * 2), static_cast<uint64_t>(stride * 2)};
    const uint32_t box[3] = {64, 1, static_cast<uint32_t>(kTileQ)};
    return encode_map(m, false, base, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace

extern "C" {

duo_status duo_paged_size(const duo_paged_layout* layout, const uint8_t* is_retrieval, duo_paged_sizes* sizes) {
    int64_t r = 0, s = 0;
    const duo_status st = check_layout(layout, is_retrieval, &r, &s);
    if (st != DUO_OK) return st;
    if (!sizes) return DUO_ERR_INVALID_ARG;
    *sizes = sizes_for(*layout, r, s);
    return DUO_OK;
}

duo_status duo_paged_alloc(const duo_paged_layout* layout, const uint8_t* is_retrieval,
                           const duo_paged_buffers* buffers, void* stream, duo_paged** out) {
    int64_t nr = 0, ns = 0;
    const duo_status st = check_layout(layout, is_retrieval, &nr, &ns);
    if (st != DUO_OK) return st;
    if (!buffers || !out) return DUO_ERR_INVALID_ARG;
    const duo_paged_layout& L = *layout;
    const duo_paged_buffers& b = *buffers;
    if ((nr > 0 && (!b.k_pages || !b.v_pages)) || (ns > 0 && (!b.k_window || !b.v_window)) || !b.page_table ||
        !b.seq_len || !b.page_ref || !b.workspace)
        return DUO_ERR_INVALID_ARG;
    const void* every[] = {b.k_pages, b.v_pages, b.k_window, b.v_window, b.page_table, b.seq_len, b.page_ref, b.workspace};
    for (const void* p : every)
        if (!aligned256(p)) return DUO_ERR_ALIGNMENT;

    duo_paged* c = nullptr;
    try {
        c = new duo_paged();
        c->heads.resize(static_cast<size_t>(L.num_layers));
    } catch (...) {
        delete c;
        return DUO_ERR_HOST_MEMORY;
    }
    c->lay = L;
    c->G = L.num_q_heads / L.num_kv_heads;
    c->scale = L.softmax_scale > 0.f ? L.softmax_scale : 1.0f / std::sqrt(static_cast<float>(L.head_dim));
    c->fp8 = L.kv_format == DUO_KV_E4M3;
    if (cudaGetDevice(&c->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&c->num_sms, cudaDevAttrMultiProcessorCount, c->device) != cudaSuccess) {
        delete c;
        return DUO_ERR_CUDA;
    }
    const Workspace w = workspace_for(L);
    uint8_t* p = static_cast<uint8_t*>(b.workspace);
    PagedView& v = c->view;
    v.err = reinterpret_cast<uint32_t*>(p);
    c->work = v.err + 1;
    p += w.err;
    c->plan = reinterpret_cast<PagePlan*>(p); p += w.plan;
    c->pair = reinterpret_cast<int2*>(p); p += w.pair;
    c->list = reinterpret_cast<int32_t*>(p); p += w.list;
    c->part_o = reinterpret_cast<float*>(p); p += w.part_o;
    c->part_ml = reinterpret_cast<float*>(p); p += w.part_ml;
    c->counters = reinterpret_cast<uint32_t*>(p); p += w.counters;
    c->kv_scales = reinterpret_cast<float*>(p);
    v.k_pages = static_cast<uint8_t*>(b.k_pages);
    v.v_pages = static_cast<uint8_t*>(b.v_pages);
    v.k_window = static_cast<bf16*>(b.k_window);
    v.v_window = static_cast<bf16*>(b.v_window);
    v.table = b.page_table;
    v.seq_len = b.seq_len;
    v.ref = b.page_ref;
    v.max_seqs = L.max_seqs;
    v.max_pages = L.max_pages;
    v.num_pages = L.num_pages;
    v.P = L.page_size;
    v.D = L.head_dim;
    v.S = L.sink;
    v.R = L.recent;
    v.W = L.sink + L.recent;
    v.r_all = static_cast<int32_t>(nr);
    v.s_all = static_cast<int32_t>(ns);
    v.elem = c->fp8 ? 1 : 2;
    for (v.P_log2 = 4; (1 << v.P_log2) < v.P;) ++v.P_log2;
    int32_t r0 = 0, s0 = 0;
    for (int32_t l = 0; l < L.num_layers; ++l) {
        PagedHeads& h = c->heads[l];
        std::memset(&h, 0, sizeof(h));
        h.r0 = r0;
        h.s0 = s0;
        int n = 0;
        for (int pass = 0; pass < 2; ++pass) {
            for (int32_t g = 0; g < L.num_kv_heads; ++g)
                if ((is_retrieval[static_cast<int64_t>(l) * L.num_kv_heads + g] != 0) == (pass == 0))
                    h.head[n++] = static_cast<int16_t>(g);
            if (pass == 0) h.n_retr = n;
        }
        h.n_strm = n - h.n_retr;
        r0 += h.n_retr;
        s0 += h.n_strm;
    }

    // Tensor maps of the pools. A pool without heads has none and is never read.
    const uint64_t D = static_cast<uint64_t>(L.head_dim);
    bool good = true;
    if (nr > 0) {
        const uint64_t e = c->fp8 ? 1 : 2;
        const uint64_t dims[3] = {D, static_cast<uint64_t>(L.page_size), static_cast<uint64_t>(L.num_pages) * nr};
        const uint64_t strides[2] = {D * e, D * e * L.page_size};
        const uint32_t tile = c->fp8 ? 128 : 64;  // rows of a decode tile
        const uint32_t rows = static_cast<uint32_t>(L.page_size) < tile ? L.page_size : tile;
        const uint32_t box[3] = {c->fp8 ? static_cast<uint32_t>(D) : 64u, rows, 1};
        const CUtensorMapSwizzle sw = c->fp8 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
        good = encode_map(&c->maps.k, c->fp8, b.k_pages, 3, dims, strides, box, sw) &&
               encode_map(&c->maps.v, c->fp8, b.v_pages, 3, dims, strides, box, sw);
    }
    if (good && ns > 0) {
        const uint64_t dims[3] = {D, static_cast<uint64_t>(v.W), static_cast<uint64_t>(L.max_seqs) * ns};
        const uint64_t strides[2] = {D * 2, D * 2 * v.W};
        const uint32_t box[3] = {64, 64, 1};
        good = encode_map(&c->maps.wk, false, b.k_window, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) &&
               encode_map(&c->maps.wv, false, b.v_window, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    good = good && cudaMemsetAsync(b.workspace, 0, w.total, s) == cudaSuccess;
    good = good && launch_paged_unit_scales(c->kv_scales, L.num_layers * L.num_kv_heads * 4, s) == cudaSuccess;
    if (!good) {
        delete c;
        return DUO_ERR_CUDA;
    }
    *out = c;
    return DUO_OK;
}

duo_status duo_paged_free(duo_paged* cache) {
    delete cache;
    return DUO_OK;
}

duo_status duo_paged_set_kv_scales(duo_paged* c, int32_t layer, const float* k_scale, const float* v_scale,
                                   void* stream) {
    if (!layer_ok(c, layer) || !k_scale || !v_scale) return DUO_ERR_INVALID_ARG;
    if (!c->fp8) return DUO_ERR_STATE;
    PagedScales x{};
    const int32_t H = c->lay.num_kv_heads;
    for (int32_t g = 0; g < H; ++g) {
        const float pair[2] = {k_scale[g], v_scale[g]};
        for (float f : pair)
            if (!(f > 0.f) || !std::isfinite(f) || !std::isfinite(1.0f / f)) return DUO_ERR_INVALID_ARG;
        x.value[g * 4 + 0] = pair[0];
        x.value[g * 4 + 1] = pair[1];
        x.value[g * 4 + 2] = 1.0f / pair[0];  // the quantizer multiplies by the 32-bit reciprocals
        x.value[g * 4 + 3] = 1.0f / pair[1];
    }
    const duo_status st = check_device(c);
    if (st != DUO_OK) return st;
    float* dst = c->kv_scales + static_cast<size_t>(layer) * H * 4;
    return launch_paged_set_scales(dst, x, H * 4, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DUO_OK : DUO_ERR_CUDA;
}

duo_status duo_paged_extend(duo_paged* c, int32_t n, const int32_t* seqs, const int32_t* n_tok, void* stream) {
    const duo_status st = check_entries(c, n, seqs, n_tok ? n_tok : seqs);
    if (st != DUO_OK || n == 0) return st;
    return launch_paged_extend(page_ops(c, n, seqs, n_tok), c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_fork(duo_paged* c, int32_t n, const int32_t* src, const int32_t* dst, void* stream) {
    const duo_status st = check_entries(c, n, src, dst);
    if (st != DUO_OK || n == 0) return st;
    return launch_paged_fork(page_ops(c, n, src, dst), c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_copy(duo_paged* c, int32_t n, const int32_t* src, const int32_t* dst, void* stream) {
    const duo_status st = check_entries(c, n, src, dst);
    if (st != DUO_OK || n == 0) return st;
    return launch_paged_copy(page_ops(c, n, src, dst), c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_release(duo_paged* c, int32_t n, const int32_t* seqs, void* stream) {
    const duo_status st = check_entries(c, n, seqs, seqs);
    if (st != DUO_OK || n == 0) return st;
    return launch_paged_release(page_ops(c, n, seqs, nullptr), static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_compact(duo_paged* c, void* stream) {
    const duo_status st = check_device(c);
    if (st != DUO_OK) return st;
    return launch_paged_compact(page_ops(c, 0, nullptr, nullptr), c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_append(duo_paged* c, int32_t layer, int32_t n, const int32_t* seqs, const int32_t* row_start,
                            const void* k, const void* v, int64_t n_rows, int64_t kv_stride, void* stream) {
    if (!layer_ok(c, layer) || n_rows < 0 || n_rows >= (1 << 30)) return DUO_ERR_INVALID_ARG;
    const duo_paged_layout& L = c->lay;
    PagedAppendParams p{};
    if (!row_stride(kv_stride, L.num_kv_heads, L.head_dim, &p.kv_stride)) return DUO_ERR_INVALID_ARG;
    const duo_status st = check_entries(c, n, seqs, row_start);
    if (st != DUO_OK || n == 0 || n_rows == 0) return st;
    if (!k || !v) return DUO_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v)) return DUO_ERR_ALIGNMENT;
    p.v = c->view;
    p.h = c->heads[layer];
    p.k = static_cast<const bf16*>(k);
    p.v_rows = static_cast<const bf16*>(v);
    p.n_rows = n_rows;
    p.seqs = seqs;
    p.row_start = row_start;
    p.n = n;
    p.fp8 = c->fp8 ? 1 : 0;
    p.kv_scale = scales_of(c, layer);
    return launch_paged_append(p, c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DUO_OK : DUO_ERR_CUDA;
}

duo_status duo_paged_prefill(duo_paged* c, int32_t layer, int32_t n, const int32_t* row_start, const void* q,
                             const void* k, const void* v, void* out, int64_t n_rows, int64_t q_stride,
                             int64_t kv_stride, int64_t out_stride, void* stream) {
    if (!layer_ok(c, layer) || n_rows < 0 || n_rows >= (1 << 30)) return DUO_ERR_INVALID_ARG;
    const duo_paged_layout& L = c->lay;
    int64_t qs = 0, ks = 0, os = 0;
    if (!row_stride(q_stride, L.num_q_heads, L.head_dim, &qs) || !row_stride(kv_stride, L.num_kv_heads, L.head_dim, &ks) ||
        !row_stride(out_stride, L.num_q_heads, L.head_dim, &os))
        return DUO_ERR_INVALID_ARG;
    const duo_status st = check_entries(c, n, row_start, row_start);
    if (st != DUO_OK || n == 0 || n_rows == 0) return st;
    if (!q || !k || !v || !out) return DUO_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return DUO_ERR_ALIGNMENT;
    PackedMaps m;
    if (!packed_map(&m.q, q, L.head_dim, L.num_q_heads, n_rows, qs) ||
        !packed_map(&m.k, k, L.head_dim, L.num_kv_heads, n_rows, ks) ||
        !packed_map(&m.v, v, L.head_dim, L.num_kv_heads, n_rows, ks))
        return DUO_ERR_CUDA;
    PackedPrefillParams p{};
    p.out = static_cast<bf16*>(out);
    p.v = static_cast<const bf16*>(v);
    p.kv_stride = ks;
    p.row_start = row_start;
    p.err = c->view.err;
    p.work = c->work;
    p.n_rows = n_rows;
    p.out_stride = os;
    p.n = n;
    p.Hq = L.num_q_heads;
    p.Hkv = L.num_kv_heads;
    p.G = c->G;
    p.D = L.head_dim;
    p.S = L.sink;
    p.R = L.recent;
    p.scale_log2 = c->scale * 1.4426950408889634f;
    p.h = c->heads[layer];
    p.test_withhold = (c->test_wait & DUO_TEST_WAIT_PREFILL) ? 1 : 0;  // one launch only
    c->test_wait &= ~DUO_TEST_WAIT_PREFILL;
    return launch_prefill_packed(p, m, c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DUO_OK : DUO_ERR_CUDA;
}

duo_status duo_paged_decode(duo_paged* c, int32_t layer, int32_t n, const int32_t* seqs, const void* q,
                            const void* k_new, const void* v_new, void* out, int64_t q_stride, int64_t kv_stride,
                            int64_t out_stride, void* stream) {
    if (!layer_ok(c, layer)) return DUO_ERR_INVALID_ARG;
    const duo_paged_layout& L = c->lay;
    PagedDecodeParams p{};
    if (!row_stride(q_stride, L.num_q_heads, L.head_dim, &p.q_stride) ||
        !row_stride(kv_stride, L.num_kv_heads, L.head_dim, &p.kv_stride) ||
        !row_stride(out_stride, L.num_q_heads, L.head_dim, &p.out_stride))
        return DUO_ERR_INVALID_ARG;
    const duo_status st = check_entries(c, n, seqs, seqs);
    if (st != DUO_OK || n == 0) return st;
    if (!q || !k_new || !v_new || !out) return DUO_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(out)) return DUO_ERR_ALIGNMENT;
    p.v = c->view;
    p.h = c->heads[layer];
    p.q = static_cast<const bf16*>(q);
    p.k_new = static_cast<const bf16*>(k_new);
    p.v_new = static_cast<const bf16*>(v_new);
    p.out = static_cast<bf16*>(out);
    p.seqs = seqs;
    p.n = n;
    p.Hq = L.num_q_heads;
    p.Hkv = L.num_kv_heads;
    p.G = c->G;
    p.scale_log2 = c->scale * 1.4426950408889634f;
    p.kv_scale = scales_of(c, layer);
    p.part_o = c->part_o;
    p.part_ml = c->part_ml;
    p.counters = c->counters;
    p.test_withhold = (c->test_wait & DUO_TEST_WAIT_DECODE) ? 1 : 0;  // one launch only
    c->test_wait &= ~DUO_TEST_WAIT_DECODE;
    return launch_paged_decode(p, c->maps, c->fp8 ? 1 : 0, c->num_sms, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DUO_OK
               : DUO_ERR_CUDA;
}

duo_status duo_paged_test_wait_timeout(duo_paged* c, int32_t launches) {
    if (!c || (launches & ~(DUO_TEST_WAIT_DECODE | DUO_TEST_WAIT_PREFILL)) != 0) return DUO_ERR_INVALID_ARG;
    c->test_wait = launches;
    return DUO_OK;
}

duo_status duo_paged_error(duo_paged* c, void* stream, uint32_t* flags) {
    if (!c || !flags) return DUO_ERR_INVALID_ARG;
    const duo_status st = check_device(c);
    if (st != DUO_OK) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    uint32_t v = 0;
    if (cudaMemcpyAsync(&v, c->view.err, sizeof(v), cudaMemcpyDeviceToHost, s) != cudaSuccess) return DUO_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return DUO_ERR_CUDA;
    if (v != 0 && cudaMemsetAsync(c->view.err, 0, sizeof(uint32_t), s) != cudaSuccess) return DUO_ERR_CUDA;
    *flags = v;
    return DUO_OK;
}

}  // extern "C"
