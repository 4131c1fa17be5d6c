// paged_pages.cu — upkeep of a paged cache: reserving tokens, forking, copying,
// releasing and compacting. The bookkeeping (page table, lengths, reference
// counts) lives on the device, so a call is one or two launches and no host
// round trip:
//   - a planning kernel of one CTA validates the call, ranks the free pages and
//     updates table, lengths and counts. The k-th page a call asks for is the
//     k-th free page in ascending order: two prefix sums, over the entries'
//     needs and over the pool's free flags. One CTA is enough up to some 20,000 pages
//     (a 180 GB pool of 8 MB pages), where the flags are 80 KB and latency bounds it, a
//     chain of about six dependent memory accesses and block scans. Larger pools take
//     longer, each thread going through pages of its own: an extend that needs pages 5.0
//     us of 1000 pages, 6.7 of 20,000, 18 of 100,000, 188 of 2^20 (3.8 of any pool when no
//     sequence needs one); a compact with nothing to move 3.4, 6.7, 32, 428.
//   - the copy kernel moves the pages and windows that the plan lists, all heads
//     of all layers. It is bound by HBM, read plus write, when there is
//     something to copy, and a bare launch otherwise.
// Fork and release need no plan and are one launch each.
// Measured: forking 16 sequences into 64, extending those and releasing them (3.2 GB
// of windows and last pages, the sources' counted for every fork, of which L2 serves
// some) 0.36 ms, 8.9 TB/s; copying 12 sequences, releasing the originals and compacting
// (5.5 GB) 0.85 ms, 6.5 TB/s, of a copy rate of 6.57; with nothing to copy 1 to 2 us
// for release, 5 for the others.
#include "paged_internal.cuh"
#include "sm100.cuh"

namespace duo {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
// CTAs per SM at most. Three or four are resident, and a CTA's stores and its next loads
// do not overlap: more CTAs than that, one behind the other, keep more in flight (copying
// 12 sequences and compacting: 890 us with 8 for both, 850 with 64 and 8, 845 with 64
// and 16; 16 forks into 64: 400 with 6, 365 with 24). Empty CTAs cost about 0.6 us per
// eight and SM, so a call that often has nothing to copy has few. More of them resident,
// with fewer registers: 885 us.
constexpr int kExtendCtas = 6;
constexpr int kCompactCtas = 8;
constexpr int kForkCtas = 24;
constexpr int kCopyCtas = 64;
constexpr int kCopyUnroll = 8;                                 // 16-byte loads in flight per thread
constexpr int kCopyChunk = kCopyThreads * kCopyUnroll * 16;    // bytes a CTA moves at a time

__device__ __forceinline__ int pages_of(int32_t len, int32_t P) { return (len + P - 1) / P; }

// Pages an entry asks for, as a summand: what no pool has stays more than any pool
// has, and 512 of them still fit 32 bits.
constexpr int kTooMany = DUO_PAGED_MAX_PAGES + 1;
__device__ __forceinline__ int summand(int pages) { return pages < kTooMany ? pages : kTooMany; }

// A length the table can hold; anything else is treated as damaged.
__device__ __forceinline__ bool len_ok(const PagedView& v, int32_t len) {
    return len >= 0 && static_cast<int64_t>(len) <= static_cast<int64_t>(v.max_pages) * v.P;
}

// Exclusive prefix sum over the CTA's threads (kPlanThreads); `total` for all.
// `warp_sum` holds kPlanThreads / 32 ints.
__device__ __forceinline__ int block_scan(int x, int* warp_sum, int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += y;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sum[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warp_sum[lane] = w;
    }
    __syncthreads();
    total = warp_sum[31];
    const int before = (warp ? warp_sum[warp - 1] : 0) + s - x;
    __syncthreads();  // warp_sum may be written again
    return before;
}

// The thread's share of the pool: pages [lo, hi), consecutive, in thread order.
struct Share {
    int lo, hi;
};
__device__ __forceinline__ Share my_pages(int num_pages) {
    const int per = ((num_pages + kPlanThreads - 1) / kPlanThreads + 3) & ~3;  // whole int4 loads
    Share s;
    s.lo = min(static_cast<int>(threadIdx.x) * per, num_pages);
    s.hi = min(s.lo + per, num_pages);
    return s;
}

// Calls f(page, ref) for the thread's pages, the loads four pages wide.
template <typename F>
__device__ __forceinline__ void each_page(const int32_t* ref, Share s, F f) {
    int p = s.lo;
    for (; p + 4 <= s.hi; p += 4) {
        const int4 r = *reinterpret_cast<const int4*>(ref + p);
        f(p, r.x);
        f(p + 1, r.y);
        f(p + 2, r.z);
        f(p + 3, r.w);
    }
    for (; p < s.hi; ++p) f(p, ref[p]);
}

// Writes the first `need` free pages, ascending, to `list`; returns how many
// pages are free. Ends with a barrier that makes the list visible.
__device__ __forceinline__ int rank_free(const PagedView& v, int need, int32_t* list, int* warp_sum) {
    const Share s = my_pages(v.num_pages);
    int mine = 0, total;
    each_page(v.ref, s, [&](int, int r) { mine += r == 0; });
    int at = block_scan(mine, warp_sum, total);
    if (need <= total && at < need && mine > 0)
        each_page(v.ref, s, [&](int p, int r) {
            if (r == 0 && at < need) list[at++] = p;
        });
    __syncthreads();
    return total;
}

// Last i with off[i] <= k (off ascending, off[0] = 0, i < n).
__device__ __forceinline__ int find_entry(const int* off, int n, int k) {
    int lo = 0, hi = n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

struct PlanShared {
    int seq[kPagedMaxBatch];   // the entry's sequence, -1: skipped
    int other[kPagedMaxBatch]; // copy: the source; extend: the shared last page, -1: none
    int off[kPagedMaxBatch];   // exclusive prefix sum of the pages needed
    int first[kPagedMaxBatch]; // extend: table index of the entry's first new page; copy: pages
    uint32_t once[kPagedMaxSeqs / 32];
    uint32_t twice[kPagedMaxSeqs / 32];
    uint32_t source[kPagedMaxSeqs / 32];
    int warp_sum[kPlanThreads / 32];
    uint32_t flags;
};

__device__ __forceinline__ void clear_marks(PlanShared& sh) {
    for (int i = threadIdx.x; i < kPagedMaxSeqs / 32; i += kPlanThreads) sh.once[i] = sh.twice[i] = sh.source[i] = 0;
    if (threadIdx.x == 0) sh.flags = 0;
    __syncthreads();
}
__device__ __forceinline__ void mark(PlanShared& sh, int seq) {
    const uint32_t bit = 1u << (seq & 31);
    if (atomicOr(&sh.once[seq >> 5], bit) & bit) atomicOr(&sh.twice[seq >> 5], bit);
}
__device__ __forceinline__ bool marked(const uint32_t* set, int seq) { return (set[seq >> 5] >> (seq & 31)) & 1u; }

// Reserve tokens (duo_paged_extend). Entry i, one thread each: its sequence's
// length, whether its last page has to be copied, the pages it needs.
__global__ void __launch_bounds__(kPlanThreads, 1) extend_plan_kernel(const PageOps p) {
    __shared__ PlanShared sh;
    grid_dependency_wait();
    const PagedView& v = p.v;
    const int i = threadIdx.x;
    clear_marks(sh);
    int seq = i < p.n ? p.a[i] : -1;
    if (seq < 0 || seq >= v.max_seqs) seq = -1;
    int len = 0, add = 0, tail = -1;
    if (seq >= 0) {
        mark(sh, seq);
        len = v.seq_len[seq];
        add = p.b ? p.b[i] : 1;
        const int64_t room = static_cast<int64_t>(v.max_pages) * v.P;
        if (!len_ok(v, len) || add < 0) {
            atomicOr(&sh.flags, kErrPagedArgument);
            len = add = 0;
        } else if (static_cast<int64_t>(len) + add > room) {
            atomicOr(&sh.flags, kErrPagedCapacity);
            add = 0;
        }
        if (add > 0 && len % v.P != 0) {
            tail = v.table[static_cast<int64_t>(seq) * v.max_pages + len / v.P];
            if (tail < 0 || tail >= v.num_pages) {
                atomicOr(&sh.flags, kErrPagedArgument);
                tail = -1;
            } else if (v.ref[tail] <= 1) {
                tail = -1;  // its own: no copy
            }
        }
    }
    if (i < kPagedMaxBatch) sh.other[i] = tail;
    __syncthreads();
    if (seq >= 0 && marked(sh.twice, seq)) atomicOr(&sh.flags, kErrPagedArgument);
    bool cow = false;
    if (tail >= 0) {
        // Sharers of the page named earlier in this call leave it before this one.
        int before = 0;
        for (int j = 0; j < i; ++j) before += sh.other[j] == tail;
        cow = v.ref[tail] - before > 1;
    }
    const int had = pages_of(len, v.P);
    const int need = summand(pages_of(len + add, v.P) - had + (cow ? 1 : 0));
    int total, n_cow;
    const int off = block_scan(need, sh.warp_sum, total);
    const int at = block_scan(cow ? 1 : 0, sh.warp_sum, n_cow);
    if (i < kPagedMaxBatch) {
        sh.seq[i] = seq;
        sh.off[i] = off;
        sh.first[i] = had - (cow ? 1 : 0);
    }
    const uint32_t flags = sh.flags;
    int n_free = 0;
    if (flags == 0 && total > 0) n_free = rank_free(v, total, p.list, sh.warp_sum);
    const bool ok = flags == 0 && total <= n_free;
    if (i == 0) {
        p.plan->n_pages = ok ? n_cow : 0;
        p.plan->n_seqs = 0;
        p.plan->used = 0;
        const uint32_t e = flags | (flags == 0 && total > n_free ? kErrPagedCapacity : 0u);
        if (e) atomicOr(v.err, e);
    }
    if (ok) {
        for (int k = i; k < total; k += kPlanThreads) {
            const int e = find_entry(sh.off, p.n, k);
            const int page = p.list[k];
            v.table[static_cast<int64_t>(sh.seq[e]) * v.max_pages + sh.first[e] + (k - sh.off[e])] = page;
            v.ref[page] = 1;
        }
        if (cow) {
            p.pair[at] = make_int2(tail, p.list[off]);
            atomicSub(&v.ref[tail], 1);
        }
        if (seq >= 0 && add > 0) v.seq_len[seq] = len + add;
    }
    __syncthreads();
    grid_launch_dependents();
}

// Copy sequences (duo_paged_copy): the entries' checks as in fork, then pages of
// their own for all of them.
__global__ void __launch_bounds__(kPlanThreads, 1) copy_plan_kernel(const PageOps p) {
    __shared__ PlanShared sh;
    grid_dependency_wait();
    const PagedView& v = p.v;
    const int i = threadIdx.x;
    clear_marks(sh);
    int src = i < p.n ? p.a[i] : -1, dst = i < p.n ? p.b[i] : -1;
    if (src < 0 || src >= v.max_seqs || dst < 0 || dst >= v.max_seqs) src = dst = -1;
    if (dst >= 0) {
        mark(sh, dst);
        atomicOr(&sh.source[src >> 5], 1u << (src & 31));
    }
    __syncthreads();
    int len = 0;
    if (dst >= 0) {
        len = v.seq_len[src];
        if (marked(sh.twice, dst) || marked(sh.source, dst) || v.seq_len[dst] != 0 || !len_ok(v, len)) {
            atomicOr(&sh.flags, kErrPagedArgument);
            dst = -1;
            len = 0;
        }
    }
    const int need = dst >= 0 ? summand(pages_of(len, v.P)) : 0;
    int total;
    const int off = block_scan(need, sh.warp_sum, total);
    if (i < kPagedMaxBatch) {
        sh.seq[i] = dst;
        sh.other[i] = src;
        sh.off[i] = off;
    }
    const int n_free = rank_free(v, total, p.list, sh.warp_sum);
    const bool ok = total <= n_free;
    if (ok) {
        for (int k = i; k < total; k += kPlanThreads) {
            const int e = find_entry(sh.off, p.n, k);
            const int page = p.list[k], j = k - sh.off[e];
            const int old = v.table[static_cast<int64_t>(sh.other[e]) * v.max_pages + j];
            const bool good = old >= 0 && old < v.num_pages;
            if (!good) atomicOr(&sh.flags, kErrPagedArgument);
            v.table[static_cast<int64_t>(sh.seq[e]) * v.max_pages + j] = page;
            v.ref[page] = 1;
            p.pair[k] = make_int2(good ? old : page, page);
        }
        if (dst >= 0) v.seq_len[dst] = len;
    }
    if (i < p.n) p.plan->seq[i] = make_int2(ok && dst >= 0 ? src : -1, dst);
    __syncthreads();
    if (i == 0) {
        p.plan->n_pages = ok ? total : 0;
        p.plan->n_seqs = ok ? p.n : 0;
        p.plan->used = 0;
        const uint32_t e = sh.flags | (ok ? 0u : kErrPagedCapacity);
        if (e) atomicOr(v.err, e);
    }
    __syncthreads();
    grid_launch_dependents();
}

// Compact (duo_paged_compact): holes below `used` in ascending order take the
// used pages at `used` and above in ascending order. Both ranks come out of one
// prefix sum over the free flags: a free page's rank is the number of free pages
// before it, a used page's its number minus that.
__global__ void __launch_bounds__(kPlanThreads, 1) compact_plan_kernel(const PageOps p) {
    __shared__ PlanShared sh;
    __shared__ int holes_shared;
    grid_dependency_wait();
    const PagedView& v = p.v;
    const Share s = my_pages(v.num_pages);
    if (threadIdx.x == 0) holes_shared = 0;
    int mine = 0, n_free;
    each_page(v.ref, s, [&](int, int r) { mine += r == 0; });
    int at = block_scan(mine, sh.warp_sum, n_free);
    const int used = v.num_pages - n_free;
    {
        int f = at, holes = 0;
        each_page(v.ref, s, [&](int pg, int r) {
            if (r == 0) {
                if (pg < used) {
                    p.pair[f].y = pg;
                    ++holes;
                }
                ++f;
            }
        });
        if (holes) atomicAdd(&holes_shared, holes);
    }
    __syncthreads();
    const int holes = holes_shared;  // as many as used pages at `used` and above
    {
        int f = at;
        each_page(v.ref, s, [&](int pg, int r) {
            if (r == 0) {
                ++f;
                return;
            }
            if (pg >= used) {
                const int k = (pg - f) - (used - holes);
                p.pair[k].x = pg;
                p.list[pg] = p.pair[k].y;  // the page's new number
            }
        });
    }
    __syncthreads();
    for (int k = threadIdx.x; k < holes; k += kPlanThreads) {
        const int2 m = p.pair[k];
        v.ref[m.y] = v.ref[m.x];
        v.ref[m.x] = 0;
    }
    if (threadIdx.x == 0) {
        p.plan->n_pages = holes;
        p.plan->n_seqs = 0;
        p.plan->used = holes > 0 ? used : 0;
    }
    __syncthreads();
    grid_launch_dependents();
}

// Copies `bytes` (a multiple of 16) at from + at .. of one chunk.
__device__ __forceinline__ void copy_chunk(const uint8_t* from, uint8_t* to, int64_t at, int64_t bytes) {
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
        const int64_t o = at + j * (kCopyThreads * 16);
        if (o < bytes) x[j] = ld_nc_v4(from + o);
    }
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j) {
        const int64_t o = at + j * (kCopyThreads * 16);
        if (o < bytes) __stcs(reinterpret_cast<uint4*>(to + o), x[j]);  // leaves L2 first: 474 -> 406 us for the forks
    }
}

// Fork (duo_paged_fork), some CTAs per entry: its table row, the counts, the windows.
// All of them look at the entry; the last to have done so writes the length, which
// the others' checks read. (With the windows in a launch of their own, as the
// other calls have it, a small fork took two latencies instead of one.)
__global__ void __launch_bounds__(kCopyThreads) fork_kernel(const PageOps p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const PagedView& v = p.v;
    const int e = blockIdx.y;
    const int src = p.a[e], dst = p.b[e];
    if (src < 0 || src >= v.max_seqs || dst < 0 || dst >= v.max_seqs) return;  // padding
    // Refused without reading what another entry may be writing: an entry whose
    // dst stands elsewhere in the call. The others are the only writers of
    // their dst, and no dst is a src.
    bool hit = false;
    for (int j = threadIdx.x; j < p.n; j += kCopyThreads) {
        const int sj = p.a[j], dj = p.b[j];
        if (sj < 0 || sj >= v.max_seqs || dj < 0 || dj >= v.max_seqs) continue;  // padding
        hit |= sj == dst || (j != e && dj == dst);
    }
    bool bad = __syncthreads_or(hit) != 0;
    int len = 0;
    if (!bad) {
        len = v.seq_len[src];
        bad = v.seq_len[dst] != 0 || !len_ok(v, len);
    }
    __syncthreads();  // every thread has read the lengths
    if (threadIdx.x == 0) {
        __threadfence();
        if (atomicAdd(&p.plan->arrived[e], 1u) == gridDim.x - 1) {
            p.plan->arrived[e] = 0;
            if (bad) atomicOr(v.err, kErrPagedArgument);
            else v.seq_len[dst] = len;
        }
    }
    if (bad) return;
    const int n = pages_of(len, v.P);
    for (int j = blockIdx.x * kCopyThreads + threadIdx.x; j < n; j += gridDim.x * kCopyThreads) {
        const int page = v.table[static_cast<int64_t>(src) * v.max_pages + j];
        v.table[static_cast<int64_t>(dst) * v.max_pages + j] = page;
        if (page >= 0 && page < v.num_pages) atomicAdd(&v.ref[page], 1);
        else atomicOr(v.err, kErrPagedArgument);
    }
    const int64_t bytes = static_cast<int64_t>(v.s_all) * v.W * v.D * 2;
    const int64_t chunks = (bytes + kCopyChunk - 1) / kCopyChunk * 2;
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        uint8_t* base = reinterpret_cast<uint8_t*>((c & 1) ? v.v_window : v.k_window);
        copy_chunk(base + src * bytes, base + dst * bytes, (c >> 1) * kCopyChunk + threadIdx.x * 16, bytes);
    }
}

constexpr int kEntryThreads = 128;

// Release (duo_paged_release), one CTA per entry.
__global__ void __launch_bounds__(kEntryThreads) release_kernel(const PageOps p) {
    grid_dependency_wait();
    const PagedView& v = p.v;
    const int e = blockIdx.x;
    const int seq = p.a[e];
    if (seq >= 0 && seq < v.max_seqs) {
        bool hit = false;
        for (int j = threadIdx.x; j < p.n; j += kEntryThreads) hit |= j != e && p.a[j] == seq;
        bool bad = __syncthreads_or(hit) != 0;
        const int len = bad ? 0 : v.seq_len[seq];  // a sequence named twice is left alone by both
        bad |= !len_ok(v, len);
        __syncthreads();
        if (threadIdx.x == 0) {
            if (bad) atomicOr(v.err, kErrPagedArgument);
            else v.seq_len[seq] = 0;
        }
        if (!bad) {
            const int n = pages_of(len, v.P);
            for (int j = threadIdx.x; j < n; j += kEntryThreads) {
                const int page = v.table[static_cast<int64_t>(seq) * v.max_pages + j];
                if (page >= 0 && page < v.num_pages) atomicSub(&v.ref[page], 1);
                else atomicOr(v.err, kErrPagedArgument);
            }
        }
    }
    grid_launch_dependents();
}

// Copies the planned pages and windows, chunk by chunk; for a compaction also
// renumbers the page table (nothing here reads both).
__global__ void __launch_bounds__(kCopyThreads) paged_copy_kernel(const PageOps p) {
    grid_dependency_wait();
    grid_launch_dependents();
    const PagedView& v = p.v;
    const int n_pages = p.plan->n_pages, n_seqs = p.plan->n_seqs, used = p.plan->used;
    const int64_t page_bytes = static_cast<int64_t>(v.r_all) * v.P * v.D * v.elem;
    const int64_t win_bytes = static_cast<int64_t>(v.s_all) * v.W * v.D * 2;
    const int64_t page_chunks = (page_bytes + kCopyChunk - 1) / kCopyChunk;
    const int64_t win_chunks = (win_bytes + kCopyChunk - 1) / kCopyChunk;
    const int64_t of_pages = n_pages * page_chunks * 2;
    const int64_t total = of_pages + n_seqs * win_chunks * 2;
    for (int64_t c = blockIdx.x; c < total; c += gridDim.x) {
        const bool page = c < of_pages;
        const int64_t per = 2 * (page ? page_chunks : win_chunks);
        const int64_t u = page ? c : c - of_pages;
        const int64_t k = u / per, r = u - k * per;
        const int2 m = page ? p.pair[k] : p.plan->seq[k];
        if (m.x < 0) continue;
        const int64_t bytes = page ? page_bytes : win_bytes;
        uint8_t* base = page ? ((r & 1) ? v.v_pages : v.k_pages)
                             : reinterpret_cast<uint8_t*>((r & 1) ? v.v_window : v.k_window);
        const int64_t at = (r >> 1) * kCopyChunk + threadIdx.x * 16;
        const uint8_t* from = base + m.x * bytes;
        uint8_t* to = base + m.y * bytes;
        copy_chunk(from, to, at, bytes);
    }
    if (used > 0) {
        for (int s = blockIdx.x; s < v.max_seqs; s += gridDim.x) {
            const int len = v.seq_len[s];
            const int n = len_ok(v, len) ? pages_of(len, v.P) : 0;
            int32_t* row = v.table + static_cast<int64_t>(s) * v.max_pages;
            for (int j = threadIdx.x; j < n; j += kCopyThreads) {
                const int page = row[j];
                if (page >= used && page < v.num_pages) row[j] = p.list[page];
            }
        }
    }
}

__global__ void set_scales_kernel(float* dst, const __grid_constant__ PagedScales x, int n) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) dst[i] = x.value[i];
}
__global__ void unit_scales_kernel(float* dst, int n) {
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n; i += gridDim.x * blockDim.x) dst[i] = 1.0f;
}

// `per_sm` CTAs per SM, and no more than there can be pieces: `pages` page pairs,
// `windows` window pairs, the rows of the table.
cudaError_t launch_copies(const PageOps& p, int num_sms, int64_t pages, int64_t windows, int64_t rows, int per_sm,
                          cudaStream_t s) {
    const PagedView& v = p.v;
    const int64_t page_bytes = static_cast<int64_t>(v.r_all) * v.P * v.D * v.elem;
    const int64_t win_bytes = static_cast<int64_t>(v.s_all) * v.W * v.D * 2;
    int64_t grid = 2 * (pages * ((page_bytes + kCopyChunk - 1) / kCopyChunk) +
                        windows * ((win_bytes + kCopyChunk - 1) / kCopyChunk));
    if (grid < rows) grid = rows;
    if (grid < 1) grid = 1;
    if (grid > num_sms * per_sm) grid = num_sms * per_sm;
    return launch_pdl(paged_copy_kernel, dim3(static_cast<unsigned>(grid)), dim3(kCopyThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_paged_set_scales(float* dst, const PagedScales& x, int n, cudaStream_t s) {
    set_scales_kernel<<<1, 128, 0, s>>>(dst, x, n);
    return cudaGetLastError();
}
cudaError_t launch_paged_unit_scales(float* dst, int n, cudaStream_t s) {
    unit_scales_kernel<<<(n + 255) / 256 < 64 ? (n + 255) / 256 : 64, 256, 0, s>>>(dst, n);
    return cudaGetLastError();
}

cudaError_t launch_paged_extend(const PageOps& p, int num_sms, cudaStream_t s) {
    const cudaError_t e = launch_pdl(extend_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    return e != cudaSuccess ? e : launch_copies(p, num_sms, p.n, 0, 0, kExtendCtas, s);
}
cudaError_t launch_paged_fork(const PageOps& p, int num_sms, cudaStream_t s) {
    // Over all entries, and no more than their windows' chunks.
    const int64_t bytes = static_cast<int64_t>(p.v.s_all) * p.v.W * p.v.D * 2;
    int64_t parts = (static_cast<int64_t>(num_sms) * kForkCtas + p.n - 1) / p.n;
    const int64_t chunks = (bytes + kCopyChunk - 1) / kCopyChunk * 2;
    if (parts > chunks) parts = chunks;
    if (parts < 1) parts = 1;
    return launch_pdl(fork_kernel, dim3(static_cast<unsigned>(parts), static_cast<unsigned>(p.n)), dim3(kCopyThreads), 0, s, p);
}
cudaError_t launch_paged_copy(const PageOps& p, int num_sms, cudaStream_t s) {
    const cudaError_t e = launch_pdl(copy_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    return e != cudaSuccess ? e : launch_copies(p, num_sms, p.v.num_pages, p.n, 0, kCopyCtas, s);
}
cudaError_t launch_paged_release(const PageOps& p, cudaStream_t s) {
    return launch_pdl(release_kernel, dim3(static_cast<unsigned>(p.n)), dim3(kEntryThreads), 0, s, p);
}
cudaError_t launch_paged_compact(const PageOps& p, int num_sms, cudaStream_t s) {
    const cudaError_t e = launch_pdl(compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p);
    return e != cudaSuccess ? e : launch_copies(p, num_sms, p.v.num_pages / 2, 0, p.v.max_seqs, kCompactCtas, s);
}

}  // namespace duo
