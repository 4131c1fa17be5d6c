// paged_append.cu — packed rows of new tokens into a paged cache: retrieval
// heads' rows into the sequence's pages, streaming heads' rows into its window
// (slot rules of append.cu).
//
// The work is cut by rows, not by entries. A sum over the entries' tokens, which every
// CTA makes for itself, numbers the usable entries' tokens 0 .. T - 1; warp w of all
// takes numbers w, w + warps, .. two at a time and looks each one's entry up. (With CTAs
// dealt out to the entries alike, a prompt of 32768 tokens among 511 entries of one token
// had 3 CTAs: 1090 us, now 28; on their own the two take 23 and 6.)
// A token's K and V rows of all heads are contiguous in the input: they are read
// coalesced, 16 bytes per lane, two pieces of K and of V of both tokens in flight, and
// written as whole 16-byte pieces. Bound by HBM (rows read once, written once) from some
// 10,000 tokens on, below by the chain entry -> length -> page number -> count ->
// row -> store, about five memory latencies, and 1 us for the numbering.
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
    const int tid = threadIdx.x;
    // Of the usable entries: tokens before each; number of the input's row and position
    // in the sequence of token x, less x; the sequence and its length.
    __shared__ int before[kPagedMaxBatch + 1], row_less[kPagedMaxBatch], pos_less[kPagedMaxBatch];
    __shared__ int seq_of[kPagedMaxBatch], len_of[kPagedMaxBatch];
    __shared__ uint32_t once[kPagedMaxSeqs / 32], twice[kPagedMaxSeqs / 32];  // sequences named
    __shared__ int2 of_warp[kWarps];
    if (p.n > 1) {
        for (int i = tid; i < kPagedMaxSeqs / 32; i += kThreads) once[i] = twice[i] = 0;
        __syncthreads();
    }
    grid_dependency_wait();
    grid_launch_dependents();
    const PagedView& v = p.v;
    // Two entries in a row per thread.
    constexpr int kOwn = 2;
    static_assert(kOwn * kThreads >= kPagedMaxBatch, "every entry has a thread");
    const int i0 = tid * kOwn;
    int own_seq[kOwn], own[kOwn], r0[kOwn], len[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        own_seq[j] = i0 + j < p.n ? p.seqs[i0 + j] : -1;
        if (own_seq[j] >= v.max_seqs) own_seq[j] = -1;
        own[j] = 0;
        if (own_seq[j] < 0) continue;
        r0[j] = p.row_start[i0 + j];
        len[j] = v.seq_len[own_seq[j]];
        const int64_t n = static_cast<int64_t>(p.row_start[i0 + j + 1]) - r0[j];
        const bool bad = r0[j] < 0 || n < 0 || r0[j] + n > p.n_rows || n > len[j] || len[j] > v.max_pages << v.P_log2;
        own[j] = bad ? -1 : static_cast<int>(n);
    }
    if (p.n > 1) {
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int seq = own_seq[j];
            const uint32_t bit = 1u << (seq & 31);
            if (seq >= 0 && (atomicOr(&once[seq >> 5], bit) & bit) != 0u) atomicOr(&twice[seq >> 5], bit);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kOwn; ++j) {
            const int seq = own_seq[j];
            if (seq >= 0 && ((twice[seq >> 5] >> (seq & 31)) & 1u) != 0u) own[j] = -1;
        }
    }
    const bool wrong_entry = own[0] < 0 || own[1] < 0;
    own[0] = max(own[0], 0);
    own[1] = max(own[1], 0);
    int at = 0;
    if (p.n > 1) {
        int sum = own[0] + own[1];
        // Ranges that overlap, behind one that runs backwards, could have more tokens than 32
        // bits hold; all others have fewer than there are rows, 2^30. Thousands tell.
        const int thousands = __reduce_add_sync(0xffffffffu, (own[0] >> 10) + (own[1] >> 10));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, sum, o);
            sum += (tid & 31) >= o ? x : 0;
        }
        if ((tid & 31) == 31) of_warp[tid >> 5] = make_int2(sum, thousands);
        __syncthreads();
        at = sum - own[0] - own[1];
        int all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int2 x = of_warp[w];
            at += w < (tid >> 5) ? x.x : 0;
            all += x.y;
        }
        if (all >= 1 << 20) {
            if (tid == 0 && blockIdx.x == 0) atomicOr(v.err, kErrPagedArgument);
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        if (i0 + j < p.n) {
            before[i0 + j] = at;
            if (own[j] > 0) {
                row_less[i0 + j] = r0[j] - at;
                pos_less[i0 + j] = len[j] - own[j] - at;
                seq_of[i0 + j] = own_seq[j];
                len_of[i0 + j] = len[j];
            }
            if (i0 + j + 1 == p.n) before[p.n] = at + own[j];
        }
        at += own[j];
    }
    if (wrong_entry && blockIdx.x == 0) atomicOr(v.err, kErrPagedArgument);
    __syncthreads();
    const uint32_t total = static_cast<uint32_t>(before[p.n]);
    constexpr int kRowLanes = D / 8;  // lanes per row
    const int lane = threadIdx.x & 31;
    const int c = lane % kRowLanes, h0 = lane / kRowLanes;
    const int n_heads = p.h.n_retr + p.h.n_strm;
    const uint32_t stride = gridDim.x * kWarps;
    for (uint32_t u0 = blockIdx.x * kWarps + (tid >> 5); u0 < total; u0 += kTokens * stride) {
        int first[kTokens], last[kTokens], slot[kTokens];  // heads [first, last) of the layer's list are stored
        int64_t row[kTokens], src[kTokens];                // (page, head 0, row in the page); the input's row
        int page[kTokens], seq[kTokens];
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            const uint32_t x = u0 + u * stride;
            page[u] = seq[u] = slot[u] = -1;
            if (x >= total) continue;
            int lo = 0, up = p.n - 1;  // the last entry with no more than x tokens before it
            while (lo < up) {
                const int mid = (lo + up + 1) >> 1;
                if (static_cast<uint32_t>(before[mid]) <= x) lo = mid;
                else up = mid - 1;
            }
            seq[u] = seq_of[lo];
            const int pos = pos_less[lo] + static_cast<int>(x);
            if (p.h.n_retr > 0) page[u] = v.table[static_cast<int64_t>(seq[u]) * v.max_pages + (pos >> v.P_log2)];
            src[u] = static_cast<int64_t>(row_less[lo] + static_cast<int>(x)) * p.kv_stride + c * 8;
            row[u] = pos & (v.P - 1);
            // Window slot, or -1 when a later token of the call takes it over.
            if (pos < v.S) slot[u] = pos;
            else if (pos >= len_of[lo] - v.R) slot[u] = v.S + (pos - v.S) % v.R;
        }
#pragma unroll
        for (int u = 0; u < kTokens; ++u) {
            first[u] = last[u] = 0;
            if (seq[u] < 0) continue;
            uint32_t wrong = 0;
            if (p.h.n_retr > 0) {
                if (page[u] < 0 || page[u] >= v.num_pages) wrong = kErrPagedArgument;
                else if (v.ref[page[u]] > 1) wrong = kErrPagedShared;
                if (wrong && lane == 0) atomicOr(v.err, wrong);
            }
            row[u] += static_cast<int64_t>(page[u]) * v.r_all * v.P;
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
                    const int64_t from = src[u] + p.h.head[i] * D;
                    kx[u][j] = ld_nc_v4(p.k + from);
                    vx[u][j] = ld_nc_v4(p.v_rows + from);
                }
#pragma unroll
            for (int u = 0; u < kTokens; ++u)
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    const int i = i0 + j * kStep;
                    if (i < first[u] || i >= last[u]) continue;
                    if (i >= p.h.n_retr) {
                        const int64_t dst =
                            ((static_cast<int64_t>(seq[u]) * v.s_all + p.h.s0 + i - p.h.n_retr) * v.W + slot[u]) * D + c * 8;
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

cudaError_t launch_paged_append(const PagedAppendParams& p, int num_sms, cudaStream_t s) {
    // Eight CTAs per SM, twice what is resident (7000 rows 9.4 us; with half as many a
    // quarter more, with four times as many a twelfth), and no more than the rows need.
    int64_t x = static_cast<int64_t>(num_sms) * 8;
    const int64_t need = (p.n_rows + kWarps - 1) / kWarps;
    if (x > need) x = need;
    const dim3 grid(static_cast<unsigned>(x));
    if (p.v.D == 128) return launch_pdl(paged_append_kernel<128>, grid, dim3(kThreads), 0, s, p);
    return launch_pdl(paged_append_kernel<64>, grid, dim3(kThreads), 0, s, p);
}

}  // namespace duo
