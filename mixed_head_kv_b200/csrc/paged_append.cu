// paged_append.cu — packed rows of new tokens into a paged cache: retrieval
// heads' rows into the sequence's pages, streaming heads' rows into its window
// (slot rules of append.cu).
//
// CTA (x, i) takes tokens x, x + gridDim.x, .. of entry i, so no search over the
// entries is needed and any row_start is safe. A token's K and V rows of all
// heads are contiguous in the input: they are read coalesced, 16 bytes of K and
// of V per thread and head with two heads in flight, and written as whole
// 16-byte pieces. Bound by HBM (rows read once, written once); below about 2000
// tokens by the latency of the chain seqs -> length -> page number -> row.
#include "paged_internal.cuh"
#include "sm100.cuh"

namespace duo {

namespace {

constexpr int kThreads = 128;

template <int D>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const PagedView& v = p.v;
    const int e = blockIdx.y;
    const int seq = p.seqs[e];
    if (seq < 0 || seq >= v.max_seqs) return;
    bool hit = false;
    for (int j = threadIdx.x; j < p.n; j += kThreads) hit |= j != e && p.seqs[j] == seq;
    bool bad = __syncthreads_or(hit) != 0;
    const int64_t r0 = p.row_start[e], r1 = p.row_start[e + 1];
    const int64_t len = v.seq_len[seq];
    bad = bad || r0 < 0 || r1 < r0 || r1 > p.n_rows || r1 - r0 > len ||
          len > static_cast<int64_t>(v.max_pages) * v.P;
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(v.err, kErrPagedArgument);
        return;
    }
    const int64_t n_tok = r1 - r0, pos0 = len - n_tok;
    constexpr int LPR = D / 8;  // threads per row
    const int c = threadIdx.x % LPR;
    const int n_heads = p.h.n_retr + p.h.n_strm;
    for (int64_t t = blockIdx.x; t < n_tok; t += gridDim.x) {
        const int64_t pos = pos0 + t;
        // Window slot, or -1 when a later token of the call takes it over.
        int64_t slot = -1;
        if (pos < v.S) slot = pos;
        else if (pos >= len - v.R) slot = v.S + (pos - v.S) % v.R;
        int64_t row = -1;  // (page, head 0, row in page) as a row of the pages
        if (p.h.n_retr > 0) {
            const int page = v.table[static_cast<int64_t>(seq) * v.max_pages + pos / v.P];
            uint32_t wrong = 0;
            if (page < 0 || page >= v.num_pages) wrong = kErrPagedArgument;
            else if (v.ref[page] > 1) wrong = kErrPagedShared;
            else row = static_cast<int64_t>(page) * v.r_all * v.P + pos % v.P;
            if (wrong && threadIdx.x == 0) atomicOr(v.err, wrong);
        }
        const int64_t src = (r0 + t) * p.kv_stride + c * 8;
        const int first = row < 0 ? p.h.n_retr : 0;
        const int last = slot < 0 ? p.h.n_retr : n_heads;
#pragma unroll 2
        for (int i = first + threadIdx.x / LPR; i < last; i += kThreads / LPR) {
            const int g = p.h.head[i];
            const uint4 kx = ld_nc_v4(p.k + src + g * D);
            const uint4 vx = ld_nc_v4(p.v_rows + src + g * D);
            if (i >= p.h.n_retr) {
                const int64_t dst =
                    ((static_cast<int64_t>(seq) * v.s_all + p.h.s0 + i - p.h.n_retr) * v.W + slot) * D + c * 8;
                *reinterpret_cast<uint4*>(v.k_window + dst) = kx;
                *reinterpret_cast<uint4*>(v.v_window + dst) = vx;
                continue;
            }
            const int64_t dst = (row + static_cast<int64_t>(p.h.r0 + i) * v.P) * D + c * 8;
            if (p.fp8) {
                *reinterpret_cast<uint2*>(v.k_pages + dst) = e4m3x8_from_bf16x8(kx, p.kv_scale[g * 4 + 2]);
                *reinterpret_cast<uint2*>(v.v_pages + dst) = e4m3x8_from_bf16x8(vx, p.kv_scale[g * 4 + 3]);
            } else {
                *reinterpret_cast<uint4*>(v.k_pages + dst * 2) = kx;
                *reinterpret_cast<uint4*>(v.v_pages + dst * 2) = vx;
            }
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
    const int64_t cap = 2368 / p.n > 16 ? 2368 / p.n : 16;  // 16 CTAs per SM over the entries
    const dim3 grid(static_cast<unsigned>(p.n_rows < cap ? p.n_rows : cap), static_cast<unsigned>(p.n));
    if (p.v.D == 128) return launch_pdl(paged_append_kernel<128>, grid, dim3(kThreads), 0, s, p);
    return launch_pdl(paged_append_kernel<64>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace duo
