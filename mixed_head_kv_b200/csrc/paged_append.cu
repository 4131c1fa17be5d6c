// paged_append.cu — packed rows of new tokens into a paged cache: retrieval
// heads' rows into the sequence's pages, streaming heads' rows into its window
// (slot rules of append.cu).
//
// CTA (x, i) works on entry i, so no search over the entries is needed and any
// row_start is safe; its warps take two tokens of the entry at a time. A token's K
// and V rows of all heads are contiguous in the input: they are read coalesced,
// 16 bytes per lane, two pieces of K and of V of both tokens in flight, and written
// as whole 16-byte pieces. Bound by HBM (rows read once, written once) from some
// 10,000 tokens on, below by the chain entry -> length -> page number -> count ->
// row -> store, about five memory latencies.
#include "paged_internal.cuh"
#include "sm100.cuh"

namespace duo {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 2;  // of a warp at a time
constexpr int kPieces = 2;  // 16-byte pieces of a lane at a time, of K and of V

template <int D>
__global__ void __launch_bounds__(kThreads, 4) paged_append_kernel(const __grid_constant__ PagedAppendParams p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const PagedView& v = p.v;
    const int e = blockIdx.y;
    const int seq = p.seqs[e];
    if (seq < 0 || seq >= v.max_seqs) return;
    const int64_t r0 = p.row_start[e], r1 = p.row_start[e + 1];
    const int64_t len = v.seq_len[seq];
    bool hit = false;
    for (int j = threadIdx.x; j < p.n; j += kThreads) hit |= j != e && p.seqs[j] == seq;
    bool bad = __syncthreads_or(hit) != 0;
    bad = bad || r0 < 0 || r1 < r0 || r1 > p.n_rows || r1 - r0 > len ||
          len > static_cast<int64_t>(v.max_pages) * v.P;
    if (bad) {
        if (threadIdx.x == 0 && blockIdx.x == 0) atomicOr(v.err, kErrPagedArgument);
        return;
    }
    const int n_tok = static_cast<int>(r1 - r0), pos0 = static_cast<int>(len - n_tok);  // lengths are below 2^27
    constexpr int kRowLanes = D / 8;  // lanes per row
    const int lane = threadIdx.x & 31;
    const int c = lane % kRowLanes, h0 = lane / kRowLanes;
    const int n_heads = p.h.n_retr + p.h.n_strm;
    const int stride = gridDim.x * kWarps;
    for (int t0 = blockIdx.x * kWarps + (threadIdx.x >> 5); t0 < n_tok; t0 += kTokens * stride) {
        int first[kTokens], last[kTokens], slot[kTokens];  // heads [first, last) of the layer's list are stored
        int64_t row[kTokens], src[kTokens];                // (page, head 0, row in the page); the input's row
        int page[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const int t = t0 + u * stride, pos = pos0 + t;
            page[u] = -1;
            if (t < n_tok && p.h.n_retr > 0)
                page[u] = v.table[static_cast<int64_t>(seq) * v.max_pages + (pos >> v.P_log2)];
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const int t = t0 + u * stride, pos = pos0 + t;
            first[u] = last[u] = 0;
            row[u] = src[u] = 0;
            slot[u] = -1;
            if (t >= n_tok) continue;
            // Window slot, or -1 when a later token of the call takes it over.
            if (pos < v.S) slot[u] = pos;
            else if (pos >= len - v.R) slot[u] = v.S + (pos - v.S) % v.R;
            uint32_t wrong = 0;
            if (p.h.n_retr > 0) {
                if (page[u] < 0 || page[u] >= v.num_pages) wrong = kErrPagedArgument;
                else if (v.ref[page[u]] > 1) wrong = kErrPagedShared;
                if (wrong && lane == 0) atomicOr(v.err, wrong);
            }
            row[u] = static_cast<int64_t>(page[u]) * v.r_all * v.P + (pos & (v.P - 1));
            src[u] = (r0 + t) * p.kv_stride + c * 8;
            first[u] = wrong ? p.h.n_retr : 0;
            last[u] = slot[u] < 0 ? p.h.n_retr : n_heads;
        }
        const int most = last[0] > last[1] ? last[0] : last[1];
        constexpr int kStep = 32 / kRowLanes;  // heads per pass of the warp
        for (int i0 = h0; i0 < most; i0 += kPieces * kStep) {
            uint4 kx[kTokens][kPieces], vx[kTokens][kPieces];
#pragma unroll
            for (int u = 0; u < kTokens; ++u)
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const int i = i0 + j * kStep;
                    if (i < first[u] || i >= last[u]) continue;
                    const int64_t at = src[u] + p.h.head[i] * D;
                    kx[u][j] = ld_nc_v4(p.k + at);
                    vx[u][j] = ld_nc_v4(p.v_rows + at);
                }
#pragma unroll
            for (int u = 0; u < kTokens; ++u)
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const int i = i0 + j * kStep;
                    if (i < first[u] || i >= last[u]) continue;
                    if (i >= p.h.n_retr) {
                        const int64_t dst =
                            ((static_cast<int64_t>(seq) * v.s_all + p.h.s0 + i - p.h.n_retr) * v.W + slot[u]) * D + c * 8;
                        *reinterpret_cast<uint4*>(v.k_window + dst) = kx[u][j];
                        *reinterpret_cast<uint4*>(v.v_window + dst) = vx[u][j];
                        continue;
                    }
                    const int64_t dst = (row[u] + static_cast<int64_t>(p.h.r0 + i) * v.P) * D + c * 8;
                    if (p.fp8) {
                        const float* sc = p.kv_scale + p.h.head[i] * 4;
                        *reinterpret_cast<uint2*>(v.k_pages + dst) = e4m3x8_from_bf16x8(kx[u][j], sc[2]);
                        *reinterpret_cast<uint2*>(v.v_pages + dst) = e4m3x8_from_bf16x8(vx[u][j], sc[3]);
                    } else {
                        *reinterpret_cast<uint4*>(v.k_pages + dst * 2) = kx[u][j];
                        *reinterpret_cast<uint4*>(v.v_pages + dst * 2) = vx[u][j];
                    }
                }
        }
    }
}

}  // namespace

cudaError_t launch_paged_append(const PagedAppendParams& p, cudaStream_t s) {
    // Eight CTAs per SM over all entries, twice what is resident (at 6000 rows of 12
    // entries 10.2 us; half as many 12.7, four times as many 11.0), and no more than the
    // rows need.
    int64_t x = (1184 + p.n - 1) / p.n;
    const int64_t need = (p.n_rows + kWarps - 1) / kWarps;
    if (x > need) x = need;
    const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(p.n));
    if (p.v.D == 128) return launch_pdl(paged_append_kernel<128>, grid, dim3(kThreads), 0, s, p);
    return launch_pdl(paged_append_kernel<64>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace duo
