// paged_decode.cu — one decoding step of one layer over a paged cache.
//
// out_h = sum_j softmax_j(scale q_h . k_j) v_j over the rows j the new token
// attends to: all `len` rows of the sequence's pages (retrieval heads) or the
// first min(len, W) rows of its window (streaming heads; their order does not
// matter). The new token's row is part of both and is written on the way.
//
// Bound by HBM: every cache row is read once for G query heads, 2 G flops per
// byte, so the work is laid out as one long list of equal tiles of 32 KB and cut
// into equal shares:
//   - a tile is 64 bf16 rows (128 rows of E4M3 codes) of K and V of one (entry,
//     KV head); D = 64 tiles are half that. The tiles of all retrieval (entry,
//     head) pairs, then of all streaming pairs, form one sequence of T tiles;
//     CTA c of C takes tiles [T c / C, T (c + 1) / C). Ragged batches, one long
//     sequence and many short ones balance alike, and the lengths are read on
//     the device: a captured launch stays right as the sequences grow;
//   - a pair cut by a share boundary is joined by the last of its CTAs to
//     finish: each leaves its unnormalised sums, maximum and weight in the
//     workspace, at most two per CTA. The joining order is the CTA order, so
//     results do not depend on which CTA is last.
// Two CTAs per SM: 4 warps compute, 1 warp loads.
//   - the loading warp streams tiles through a ring of 96 KB by TMA (page-sized
//     boxes, 128-byte swizzle; page numbers are fetched 32 at a time, one load
//     ahead) and the group's queries and the new rows through a 2-slot ring;
//   - every computing warp owns 16 (32) rows of each tile and runs on its own: no
//     barrier inside a pair. S^T = K Q^T and O^T = V^T P^T with m16n8k16: the
//     rows are the M side, so the group's heads fill the N side up to 8 and the
//     cost does not depend on G; P^T changes from accumulator to operand layout
//     in registers. K and V come out of shared memory with ldmatrix; E4M3 codes
//     are converted to f16 in registers (exact; the queries are scaled by a power
//     of two per head to fit f16, and K's order along D is permuted the same way
//     on both sides so that a thread converts whole 16-byte words).
//   - softmax in the exp2 domain, 32-bit statistics and sums; the maximum is
//     moved only when a score exceeds it by more than 2^8 (exact: all terms stay
//     relative to the same maximum). P is rounded to bf16 (f16 with E4M3): the
//     operand type, relative error 2^-9 (2^-12) per term.
// Rows behind the last one in a page hold anything: their scores are replaced,
// and their V rows are zeroed in shared memory (0 x NaN would not be 0).
#include "paged_internal.cuh"
#include "sm100.cuh"

namespace duo {

namespace {

constexpr int kWarps = 4;                 // computing warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kCtasPerSm = 2;
constexpr int kRingBytes = 96 * 1024;
constexpr int kMaxG = DUO_PAGED_MAX_GROUP;
// A pair is cut into at most about this many parts: joining reads G x D floats
// of each part in one CTA.
constexpr int kPartsPerPair = 48;

template <int D>
struct Smem {
    static constexpr int kStage = D * 256;  // K and V of a tile
    static constexpr int kStages = kRingBytes / kStage;
    static constexpr int kRing = 0;
    static constexpr int kQSlot = (kMaxG + 2) * D * 2;  // queries, new K row, new V row
    static constexpr int kQ = kRing + kRingBytes;
    static constexpr int kMerge = kQ + 2 * kQSlot;      // one warp's O
    static constexpr int kStat = kMerge + kMaxG * D * 4;  // maximum and sum of a warp's heads
    static constexpr int kBar = kStat + kWarps * kMaxG * 2 * 4;
    static constexpr int kMisc = kBar + 32 * 8;
    static constexpr int kPrefix = kMisc + 32;  // per entry: length, tiles before (retrieval, streaming), sequence
};
__host__ __device__ constexpr int smem_bytes(int D, int n) {
    return (D == 128 ? Smem<128>::kPrefix : Smem<64>::kPrefix) + (n + 1) * 8 + n * 4 + n * 2 + 8;
}
static_assert(smem_bytes(128, kPagedMaxBatch) <= 113 * 1024, "two CTAs per SM");

constexpr int kFull = 0;     // + stage (up to 6)
constexpr int kEmpty = 6;    // + stage
constexpr int kQFull = 12;   // + slot
constexpr int kQEmpty = 14;  // + slot

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// acc += A (16 x 16) B (16 x 8)
template <bool F16>
__device__ __forceinline__ void mma16816(float (&acc)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2_of_codes(uint32_t two) {  // low 16 bits: two E4M3 codes
    uint32_t r;
    asm("{\n\t.reg .b16 c;\n\tcvt.u16.u32 c, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, c;\n\t}" : "=r"(r) : "r"(two));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& x) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// The computing warps' barrier.
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// One stretch of tiles of one (entry, KV head) pair inside a CTA's share.
struct Segment {
    int e, seq, len;     // entry, sequence, its tokens
    int idx;             // index of the head in the layer's list (retrieval first)
    int retr;            // 1: pages, 0: window
    int t0, t1, tiles;   // tiles [t0, t1) of `tiles`
    int64_t first;       // number of the pair's first tile in the whole list
};

struct Work {
    const int* len;
    const int* before_r;  // [n + 1] retrieval tiles of one head before entry i
    const int* before_s;
    const uint16_t* seq;
    int n, n_retr, n_strm;
    int64_t of_retr, total;

    // The segment that starts at tile u and ends at `hi` at the latest.
    __device__ __forceinline__ Segment at(int64_t u, int64_t hi) const {
        Segment s;
        s.retr = u < of_retr;
        const int* before = s.retr ? before_r : before_s;
        const int heads = s.retr ? n_retr : n_strm;
        const int64_t x = s.retr ? u : u - of_retr;
        int lo = 0, up = n - 1;
        while (lo < up) {
            const int mid = (lo + up + 1) >> 1;
            if (static_cast<int64_t>(before[mid]) * heads <= x) lo = mid;
            else up = mid - 1;
        }
        s.e = lo;
        s.tiles = before[lo + 1] - before[lo];
        const int64_t y = x - static_cast<int64_t>(before[lo]) * heads;
        const int h = static_cast<int>(y / s.tiles);
        s.t0 = static_cast<int>(y - static_cast<int64_t>(h) * s.tiles);
        s.first = u - s.t0;
        const int64_t left = hi - u;
        s.t1 = left < s.tiles - s.t0 ? s.t0 + static_cast<int>(left) : s.tiles;
        s.idx = s.retr ? h : n_retr + h;
        s.seq = seq[lo];
        s.len = len[lo];
        return s;
    }
};

__device__ __forceinline__ int64_t share_start(int64_t total, int c, int n) { return total * c / n; }
__device__ __forceinline__ int share_of(int64_t total, int64_t u, int n) {
    return static_cast<int>(((u + 1) * n - 1) / total);
}

__device__ __forceinline__ void report(uint32_t* err, uint32_t bit) { atomicOr(err, bit); }

// The window row of position pos.
__device__ __forceinline__ int window_slot(const PagedView& v, int pos) {
    return pos < v.S ? pos : v.S + (pos - v.S) % v.R;
}

template <int D, bool FP8>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    paged_decode_kernel(const __grid_constant__ PagedDecodeParams p, const __grid_constant__ PagedMaps maps) {
    using L = Smem<D>;
    constexpr int kPageTile = FP8 ? 128 : 64;  // rows of a page tile
    constexpr int kWinTile = 64;
    constexpr int kHalf = L::kStage / 2;       // V behind K
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    auto bar = [&](int i) { return base + L::kBar + 8u * i; };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::kMisc);
    uint32_t* last_flag = reinterpret_cast<uint32_t*>(smem + L::kMisc + 4);
    int* before_r = reinterpret_cast<int*>(smem + L::kPrefix);
    int* before_s = before_r + p.n + 1;
    int* len_of = before_s + p.n + 1;
    uint16_t* seq_of = reinterpret_cast<uint16_t*>(len_of + p.n);
    const PagedView& v = p.v;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < L::kStages; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), kWarps);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kQFull + s), 1);
            mbar_init(bar(kQEmpty + s), kWarps);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    // Marks of the sequences named once and twice, in the ring before its first tile.
    uint32_t* once = reinterpret_cast<uint32_t*>(smem + L::kRing);
    uint32_t* twice = once + kPagedMaxSeqs / 32;
    for (int i = tid; i < kPagedMaxSeqs / 32; i += kThreads) once[i] = twice[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    for (int i = tid; i < p.n; i += kThreads) {
        const int s = p.seqs[i];
        const bool in = s >= 0 && s < v.max_seqs;
        int len = in ? v.seq_len[s] : -1;
        if (in) {
            const uint32_t bit = 1u << (s & 31);
            if (atomicOr(&once[s >> 5], bit) & bit) atomicOr(&twice[s >> 5], bit);
            if (len < 0 || static_cast<int64_t>(len) > static_cast<int64_t>(v.max_pages) * v.P) {
                if (blockIdx.x == 0) report(v.err, kErrPagedArgument);
                len = -1;
            }
        }
        len_of[i] = len;
        seq_of[i] = static_cast<uint16_t>(in ? s : 0);
    }
    __syncthreads();
    if (warp == 0) {  // lengths of entries named twice dropped, tiles counted
        int sum_r = 0, sum_s = 0;
        for (int i0 = 0; i0 < p.n; i0 += 32) {
            const int i = i0 + lane;
            int len = i < p.n ? len_of[i] : -1;
            if (len >= 0) {
                const int s = seq_of[i];
                if ((twice[s >> 5] >> (s & 31)) & 1u) {
                    if (blockIdx.x == 0) report(v.err, kErrPagedArgument);
                    len_of[i] = len = -1;
                }
            }
            const int rows = len > 0 ? len : 0;
            int r = (rows + kPageTile - 1) / kPageTile;
            int w = ((rows < v.W ? rows : v.W) + kWinTile - 1) / kWinTile;
            const int r_own = r, w_own = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, r, o), b = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) {
                    r += a;
                    w += b;
                }
            }
            if (i < p.n) {
                before_r[i] = sum_r + r - r_own;
                before_s[i] = sum_s + w - w_own;
            }
            sum_r += __shfl_sync(0xffffffffu, r, 31);
            sum_s += __shfl_sync(0xffffffffu, w, 31);
        }
        if (lane == 0) {
            before_r[p.n] = sum_r;
            before_s[p.n] = sum_s;
            fence_proxy_async_smem();  // the marks' words become TMA destinations
        }
    }
    __syncthreads();
    // Rows of empty sequences are zero.
    for (int e = blockIdx.x; e < p.n; e += gridDim.x)
        if (len_of[e] == 0)
            for (int i = tid; i < p.Hq * D / 8; i += kThreads)
                *reinterpret_cast<uint4*>(p.out + e * p.out_stride + i * 8) = make_uint4(0, 0, 0, 0);

    Work work;
    work.len = len_of;
    work.before_r = before_r;
    work.before_s = before_s;
    work.seq = seq_of;
    work.n = p.n;
    work.n_retr = p.h.n_retr;
    work.n_strm = p.h.n_strm;
    work.of_retr = static_cast<int64_t>(before_r[p.n]) * p.h.n_retr;
    work.total = work.of_retr + static_cast<int64_t>(before_s[p.n]) * p.h.n_strm;
    const int64_t pairs = static_cast<int64_t>(p.n) * (p.h.n_retr + p.h.n_strm);
    int n_cta = gridDim.x;
    if (n_cta > work.total) n_cta = static_cast<int>(work.total);
    if (n_cta > pairs * kPartsPerPair) n_cta = static_cast<int>(pairs * kPartsPerPair);
    const int c = blockIdx.x;
    if (c >= n_cta) return;
    const int64_t lo = share_start(work.total, c, n_cta), hi = share_start(work.total, c + 1, n_cta);

    if (warp == kWarps) {
        // ------------------------------------------------------------ loads
        int64_t tile = 0;  // of this CTA
        int n_seg = 0;
        bool ok = true;
        for (int64_t u = lo; ok && u < hi; ++n_seg) {
            const Segment s = work.at(u, hi);
            const int g = p.h.head[s.idx];
            const int slot = n_seg & 1;
            if (n_seg >= 2 && !mbar_wait(bar(kQEmpty + slot), ((n_seg >> 1) - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                const uint32_t q = base + L::kQ + slot * L::kQSlot;
                mbar_arrive_expect_tx(bar(kQFull + slot), (p.G + 2) * D * 2);
                bulk_load(q, p.q + s.e * p.q_stride + g * p.G * D, p.G * D * 2, bar(kQFull + slot));
                bulk_load(q + kMaxG * D * 2, p.k_new + s.e * p.kv_stride + g * D, D * 2, bar(kQFull + slot));
                bulk_load(q + (kMaxG + 1) * D * 2, p.v_new + s.e * p.kv_stride + g * D, D * 2, bar(kQFull + slot));
            }
            const int rows = s.retr ? s.len : (s.len < v.W ? s.len : v.W);
            const int* row_table = v.table + static_cast<int64_t>(s.seq) * v.max_pages;
            const int n_pages = (s.len + v.P - 1) / v.P;
            // Page numbers, 32 at a time: `have` covers [win, win + 32), `next` the 32 behind.
            int win = 0, have = 0, next = 0;
            if (s.retr) {
                win = static_cast<int>(static_cast<int64_t>(s.t0) * kPageTile / v.P);
                have = win + lane < n_pages ? row_table[win + lane] : -1;
                next = win + 32 + lane < n_pages ? row_table[win + 32 + lane] : -1;
            }
            for (int t = s.t0; t < s.t1; ++t, ++tile) {
                const int st = static_cast<int>(tile % L::kStages);
                const int64_t round = tile / L::kStages;
                if (round > 0 && !mbar_wait(bar(kEmpty + st), (round - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = base + L::kRing + st * L::kStage;
                if (s.retr) {
                    const int row0 = t * kPageTile;
                    const int valid = rows - row0 < kPageTile ? rows - row0 : kPageTile;
                    const int box = v.P < kPageTile ? v.P : kPageTile;  // rows of one copy
                    const int n_box = (valid + box - 1) / box;
                    const int pg0 = row0 / v.P;
                    while (pg0 >= win + 32) {
                        win += 32;
                        have = next;
                        next = win + 32 + lane < n_pages ? row_table[win + 32 + lane] : -1;
                    }
                    // A tile's boxes: at most 8 pages, all in [pg0, pg0 + 8). Lane b copies box b.
                    const int pg = pg0 + (lane & 7);
                    const int a0 = __shfl_sync(0xffffffffu, have, (pg - win) & 31);
                    const int a1 = __shfl_sync(0xffffffffu, next, (pg - win) & 31);
                    int page = pg - win < 32 ? a0 : a1;
                    const bool mine = lane < n_box;
                    if (mine && (page < 0 || page >= v.num_pages)) {
                        report(v.err, kErrPagedArgument);
                        page = -1;
                    }
                    constexpr int kRowBytes = FP8 ? D : 128;       // of a swizzled box
                    constexpr int kCols = FP8 ? 1 : D / 64;
                    const int box_bytes = box * D * (FP8 ? 1 : 2);
                    if (lane == 0) mbar_arrive_expect_tx(bar(kFull + st), 2 * n_box * box_bytes);
                    __syncwarp();
                    if (mine) {
                        // An unusable page number loads zeros (a coordinate outside the map).
                        const int z = page < 0 ? -1 : page * v.r_all + p.h.r0 + s.idx;
                        const int y = row0 % v.P;
#pragma unroll
                        for (int cb = 0; cb < kCols; ++cb) {
                            const uint32_t d = dst + cb * (kPageTile * kRowBytes) + lane * box * kRowBytes;
                            tma_load_3d(d, &maps.k, bar(kFull + st), cb * 64, y, z);
                            tma_load_3d(d + kHalf, &maps.v, bar(kFull + st), cb * 64, y, z);
                        }
                    }
                } else if (lane == 0) {
                    const int z = s.seq * v.s_all + p.h.s0 + (s.idx - p.h.n_retr);
                    mbar_arrive_expect_tx(bar(kFull + st), 2 * kWinTile * D * 2);
#pragma unroll
                    for (int cb = 0; cb < D / 64; ++cb) {
                        const uint32_t d = dst + cb * (kWinTile * 128);
                        tma_load_3d(d, &maps.wk, bar(kFull + st), cb * 64, t * kWinTile, z);
                        tma_load_3d(d + kHalf, &maps.wv, bar(kFull + st), cb * 64, t * kWinTile, z);
                    }
                }
                __syncwarp();
            }
            u += s.t1 - s.t0;
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            report(v.err, kErrPagedWait);
        }
        // Every copy issued lands before the CTA may exit.
        const int64_t from = tile > L::kStages ? tile - L::kStages : 0;
        for (int64_t t = from; t < tile; ++t)
            mbar_wait(bar(kFull + static_cast<int>(t % L::kStages)), (t / L::kStages) & 1, nullptr);
        for (int i = n_seg > 2 ? n_seg - 2 : 0; i < n_seg; ++i) mbar_wait(bar(kQFull + (i & 1)), (i >> 1) & 1, nullptr);
        return;
    }

    // ---------------------------------------------------------------- computing warps
    const int gq = lane >> 2;  // row of an accumulator, column of an operand: key / head
    const int cq = lane & 3;
    constexpr int kSteps = D / 16;
    int64_t tile = 0;
    int n_seg = 0;
    bool ok = true;
    float* merge = reinterpret_cast<float*>(smem + L::kMerge);
    float* stat = reinterpret_cast<float*>(smem + L::kStat);  // [warp][head][2]
    for (int64_t u = lo; u < hi; ++n_seg) {
        const Segment s = work.at(u, hi);
        const int g = p.h.head[s.idx];
        const int slot = n_seg & 1;
        const uint32_t q = base + L::kQ + slot * L::kQSlot;
        if (ok && !mbar_wait(bar(kQFull + slot), (n_seg >> 1) & 1, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abort_flag = 1;
        const bool codes = FP8 && s.retr;  // operands are f16 made of codes
        // The queries as the B operand: head gq, this thread's part of D.
        uint32_t b[kSteps][2];
        float scale0 = p.scale_log2, scale1 = p.scale_log2;  // of heads 2 cq and 2 cq + 1
        if (!codes) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const uint32_t a = q + gq * D * 2 + k * 32 + cq * 4;
                b[k][0] = b[k][1] = 0u;
                if (gq < p.G) {
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b[k][0]) : "r"(a));
                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(b[k][1]) : "r"(a + 16));
                }
            }
        } else {
            // K's codes 16 w + 64 o + 4 j + i (w = cq, o = j / 4 block) stand for the
            // operand's positions 2 cq + {0, 1, 8, 9} of step j: the same for Q.
            uint32_t x[kSteps][2];
            float mx = 0.f;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const uint32_t a = q + gq * D * 2 + (k >> 2) * 128 + cq * 32 + (k & 3) * 8;
                x[k][0] = x[k][1] = 0u;
                if (gq < p.G) {
                    const uint2 w = lds64(a);
                    x[k][0] = w.x;
                    x[k][1] = w.y;
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    mx = fmaxf(mx, fmaxf(fabsf(bf16lo_to_f32(x[k][i])), fabsf(bf16hi_to_f32(x[k][i]))));
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            // A power of two that brings the largest element to [2^12, 2^13): f16 then
            // loses only what is 2^26 times smaller.
            int ex = mx > 0.f && mx < INFINITY ? ilogbf(mx) - 12 : 0;
            if (ex < -100) ex = -100;
            const float up = exp2f(static_cast<float>(-ex));
#pragma unroll
            for (int k = 0; k < kSteps; ++k)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    b[k][i] = pack_f16x2(bf16lo_to_f32(x[k][i]) * up, bf16hi_to_f32(x[k][i]) * up);
            const float back = exp2f(static_cast<float>(ex)) * p.scale_log2 * p.kv_scale[g * 4];
            scale0 = __shfl_sync(0xffffffffu, back, (2 * cq) * 4);
            scale1 = __shfl_sync(0xffffffffu, back, (2 * cq + 1) * 4);
        }
        float o[kSteps][4];
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
        const int rows = s.retr ? s.len : (s.len < v.W ? s.len : v.W);
        const int new_row = s.retr ? s.len - 1 : window_slot(v, s.len - 1);
        const int tile_rows = s.retr ? kPageTile : kWinTile;
        for (int t = s.t0; t < s.t1; ++t, ++tile) {
            const int st = static_cast<int>(tile % L::kStages);
            const uint32_t kt = base + L::kRing + st * L::kStage, vt = kt + kHalf;
            if (ok && !mbar_wait(bar(kFull + st), (tile / L::kStages) & 1, abort_flag)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) *abort_flag = 1;
            const int per = tile_rows / kWarps;  // this warp's rows of the tile
            const int w0 = warp * per;
            const int valid = rows - t * tile_rows - w0;  // of them, rows to attend to
            bool touched = false;
            if (ok && valid > 0) {
                // The new token's row: into the tile, and into the cache.
                const int nr = new_row - t * tile_rows - w0;
                if (nr >= 0 && nr < per) {
                    touched = true;
                    const int row = w0 + nr;
                    const int which = lane >> 4, ch = lane & 15;  // K or V, 16 bytes of bf16
                    if (ch < D / 8) {
                        const uint4 x = lds128(q + (kMaxG + which) * D * 2 + ch * 16);
                        if (codes) {
                            const uint2 y = e4m3x8_from_bf16x8(x, p.kv_scale[g * 4 + 2 + which]);
                            const uint32_t a = (which ? vt : kt) + row * D +
                                               (((ch >> 1) ^ (D == 128 ? row & 7 : (row >> 1) & 3)) << 4) + (ch & 1) * 8;
                            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(a), "r"(y.x), "r"(y.y) : "memory");
                        } else {
                            sts128((which ? vt : kt) + (ch >> 3) * (tile_rows * 128) + row * 128 + (((ch & 7) ^ (row & 7)) << 4), x);
                        }
                        if (!s.retr) {
                            bf16* dst = (which ? v.v_window : v.k_window) +
                                        ((static_cast<int64_t>(s.seq) * v.s_all + p.h.s0 + s.idx - p.h.n_retr) * v.W + new_row) * D + ch * 8;
                            *reinterpret_cast<uint4*>(dst) = x;
                        } else {
                            const int page = v.table[static_cast<int64_t>(s.seq) * v.max_pages + new_row / v.P];
                            const bool in = page >= 0 && page < v.num_pages;  // else the loads reported it
                            if (in && v.ref[page] > 1) {
                                report(v.err, kErrPagedShared);
                            } else if (in) {
                                const int64_t at = ((static_cast<int64_t>(page) * v.r_all + p.h.r0 + s.idx) * v.P + new_row % v.P) * D + ch * 8;
                                uint8_t* pool = which ? v.v_pages : v.k_pages;
                                if (FP8) *reinterpret_cast<uint2*>(pool + at) = e4m3x8_from_bf16x8(x, p.kv_scale[g * 4 + 2 + which]);
                                else *reinterpret_cast<uint4*>(pool + at * 2) = x;
                            }
                        }
                    }
                }
                if (valid < per) {  // V rows behind the last one
                    touched = true;
                    for (int r = w0 + valid; r < w0 + per; ++r) {
                        if (codes) {
                            if (lane < D / 16) sts128(vt + r * D + lane * 16, make_uint4(0, 0, 0, 0));
                        } else if (lane < D / 8) {
                            sts128(vt + (lane >> 3) * (tile_rows * 128) + r * 128 + (lane & 7) * 16, make_uint4(0, 0, 0, 0));
                        }
                    }
                }
                __syncwarp();
                const int parts = per / 16;  // 1, or 2 with codes
                for (int part = 0; part < parts; ++part) {
                    const int r0 = w0 + part * 16;
                    const int left = valid - part * 16;
                    if (left <= 0) break;
                    // S^T = K Q^T
                    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
                    if (!codes) {
                        const int r = r0 + (lane & 15);
#pragma unroll
                        for (int k = 0; k < kSteps; ++k) {
                            const int ch = (k & 3) * 2 + (lane >> 4);
                            uint32_t a[4];
                            ldsm4(kt + (k >> 2) * (tile_rows * 128) + r * 128 + ((ch ^ (r & 7)) << 4), a);
                            mma16816<false>(acc[k & 1], a, b[k][0], b[k][1]);
                        }
                    } else if (FP8) {
#pragma unroll
                        for (int o4 = 0; o4 < D / 64; ++o4) {
                            const int ra = r0 + gq, rb = ra + 8;
                            const int ch = o4 * 4 + cq;
                            const uint4 xa = lds128(kt + ra * D + ((ch ^ (D == 128 ? ra & 7 : (ra >> 1) & 3)) << 4));
                            const uint4 xb = lds128(kt + rb * D + ((ch ^ (D == 128 ? rb & 7 : (rb >> 1) & 3)) << 4));
                            const uint32_t wa[4] = {xa.x, xa.y, xa.z, xa.w}, wb[4] = {xb.x, xb.y, xb.z, xb.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t a[4] = {f16x2_of_codes(wa[j]), f16x2_of_codes(wb[j]),
                                                       f16x2_of_codes(wa[j] >> 16), f16x2_of_codes(wb[j] >> 16)};
                                mma16816<true>(acc[j & 1], a, b[o4 * 4 + j][0], b[o4 * 4 + j][1]);
                            }
                        }
                    }
                    // Rows gq and gq + 8, heads 2 cq and 2 cq + 1.
                    float x[4];
                    x[0] = gq < left ? (acc[0][0] + acc[1][0]) * scale0 : -INFINITY;
                    x[1] = gq < left ? (acc[0][1] + acc[1][1]) * scale1 : -INFINITY;
                    x[2] = gq + 8 < left ? (acc[0][2] + acc[1][2]) * scale0 : -INFINITY;
                    x[3] = gq + 8 < left ? (acc[0][3] + acc[1][3]) * scale1 : -INFINITY;
                    float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
                    if (__any_sync(0xffffffffu, t0 > m0 + 8.f || t1 > m1 + 8.f)) {
#pragma unroll
                        for (int d = 4; d < 32; d <<= 1) {
                            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
                            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
                        }
                        const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
                        const float f0 = n0 == -INFINITY ? 1.f : fast_exp2(m0 - n0);
                        const float f1 = n1 == -INFINITY ? 1.f : fast_exp2(m1 - n1);
                        m0 = n0;
                        m1 = n1;
                        l0 *= f0;
                        l1 *= f1;
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            o[i][0] *= f0;
                            o[i][1] *= f1;
                            o[i][2] *= f0;
                            o[i][3] *= f1;
                        }
                    }
                    const float u0 = m0 == -INFINITY ? 0.f : m0, u1 = m1 == -INFINITY ? 0.f : m1;
                    x[0] = fast_exp2(x[0] - u0);
                    x[1] = fast_exp2(x[1] - u1);
                    x[2] = fast_exp2(x[2] - u0);
                    x[3] = fast_exp2(x[3] - u1);
                    l0 += x[0] + x[2];
                    l1 += x[1] + x[3];
                    // P^T from accumulator to operand layout.
                    const uint32_t p0 = transpose8x8(codes ? pack_f16x2(x[0], x[1]) : pack_bf16x2(x[0], x[1]));
                    const uint32_t p1 = transpose8x8(codes ? pack_f16x2(x[2], x[3]) : pack_bf16x2(x[2], x[3]));
                    // O^T += V^T P^T
                    if (!codes) {
                        const int r = r0 + (lane & 7) + ((lane >> 4) << 3);
#pragma unroll
                        for (int i = 0; i < kSteps; ++i) {
                            const int ch = (i & 3) * 2 + ((lane >> 3) & 1);
                            uint32_t a[4];
                            ldsm4t(vt + (i >> 2) * (tile_rows * 128) + r * 128 + ((ch ^ (r & 7)) << 4), a);
                            mma16816<false>(o[i], a, p0, p1);
                        }
                    } else if (FP8) {
                        // Columns gq D / 8 .. of rows 2 cq, 2 cq + 1, 2 cq + 8, 2 cq + 9;
                        // the columns 2 i and 2 i + 1 of them are rows gq and gq + 8 of step i.
                        uint32_t w[4][D / 32];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int r = r0 + 2 * cq + (k & 1) + (k >> 1) * 8;
                            if (D == 128) {
                                const uint4 y = lds128(vt + r * D + ((gq ^ (r & 7)) << 4));
                                w[k][0] = y.x;
                                w[k][1] = y.y;
                                w[k][D / 32 - 2] = y.z;
                                w[k][D / 32 - 1] = y.w;
                            } else {
                                const uint2 y = lds64(vt + r * D + (((gq >> 1) ^ ((r >> 1) & 3)) << 4) + (gq & 1) * 8);
                                w[k][0] = y.x;
                                w[k][1] = y.y;
                            }
                        }
#pragma unroll
                        for (int i4 = 0; i4 < D / 32; ++i4) {
                            const uint32_t lo01 = __byte_perm(w[0][i4], w[1][i4], 0x5140);
                            const uint32_t hi01 = __byte_perm(w[0][i4], w[1][i4], 0x7362);
                            const uint32_t lo89 = __byte_perm(w[2][i4], w[3][i4], 0x5140);
                            const uint32_t hi89 = __byte_perm(w[2][i4], w[3][i4], 0x7362);
                            const uint32_t a0[4] = {f16x2_of_codes(lo01), f16x2_of_codes(lo01 >> 16),
                                                    f16x2_of_codes(lo89), f16x2_of_codes(lo89 >> 16)};
                            const uint32_t a1[4] = {f16x2_of_codes(hi01), f16x2_of_codes(hi01 >> 16),
                                                    f16x2_of_codes(hi89), f16x2_of_codes(hi89 >> 16)};
                            mma16816<true>(o[2 * i4], a0, p0, p1);
                            mma16816<true>(o[2 * i4 + 1], a1, p0, p1);
                        }
                    }
                }
            }
            if (touched) fence_proxy_async_smem();  // before TMA writes the stage again
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(kEmpty + st));
        }
        if (lane == 0) mbar_arrive(bar(kQEmpty + slot));
        // ------------------------------------------------------------ end of the segment
        // Join the four warps: maxima and sums first, then O warp by warp into warp 0.
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, d);
            l1 += __shfl_xor_sync(0xffffffffu, l1, d);
        }
        if (gq == 0) {
            stat[(warp * kMaxG + 2 * cq) * 2] = m0;
            stat[(warp * kMaxG + 2 * cq) * 2 + 1] = l0;
            stat[(warp * kMaxG + 2 * cq + 1) * 2] = m1;
            stat[(warp * kMaxG + 2 * cq + 1) * 2 + 1] = l1;
        }
        group_sync();
        float mj[2], lj[2];
        float f[2];  // this warp's factor to the joint maximum
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int h = 2 * cq + i;
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stat[(w * kMaxG + h) * 2]);
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = stat[(w * kMaxG + h) * 2], lw = stat[(w * kMaxG + h) * 2 + 1];
                // lw is not 0 with mw = -inf only for scores of -inf or NaN: kept as they are.
                sum += lw * (mw == m ? 1.f : fast_exp2(mw - m));
            }
            mj[i] = m;
            lj[i] = sum;
            const float own = i ? m1 : m0;
            f[i] = own == m ? 1.f : fast_exp2(own - m);
        }
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            o[i][0] *= f[0];
            o[i][1] *= f[1];
            o[i][2] *= f[0];
            o[i][3] *= f[1];
        }
        // Row of D that accumulator i holds in its first (half 0) or second pair.
        auto col = [&](int i, int half) { return codes ? gq * (D / 8) + 2 * i + half : i * 16 + half * 8 + gq; };
        for (int w = 1; w < kWarps; ++w) {
            if (warp == w) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (2 * cq + (j & 1) < p.G) merge[(i * 4 + j) * 32 + lane] = o[i][j];
            }
            group_sync();
            if (warp == 0) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (2 * cq + (j & 1) < p.G) o[i][j] += merge[(i * 4 + j) * 32 + lane];
            }
            group_sync();
        }
        const bool whole = s.t0 == 0 && s.t1 == s.tiles;
        const float v_scale = codes ? p.kv_scale[g * 4 + 1] : 1.f;
        if (whole) {
            if (warp == 0 && ok) {
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int h = 2 * cq + (j & 1);
                        if (h < p.G)
                            p.out[s.e * p.out_stride + (g * p.G + h) * D + col(i, j >> 1)] =
                                __float2bfloat16(o[i][j] * (v_scale / lj[j & 1]));
                    }
            }
        } else {
            const int part = c * 2 + (u == lo ? 0 : 1);
            if (warp == 0) {
                float* po = p.part_o + static_cast<int64_t>(part) * p.G * D;
                float* pm = p.part_ml + static_cast<int64_t>(part) * p.G * 2;
#pragma unroll
                for (int i = 0; i < kSteps; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int h = 2 * cq + (j & 1);
                        if (h < p.G) po[h * D + col(i, j >> 1)] = o[i][j];
                    }
                if (gq == 0) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (2 * cq + i < p.G) {
                            pm[(2 * cq + i) * 2] = mj[i];
                            pm[(2 * cq + i) * 2 + 1] = lj[i];
                        }
                }
                __threadfence();
                __syncwarp();
                if (lane == 0) {
                    const int c0 = share_of(work.total, s.first, n_cta);
                    const int c1 = share_of(work.total, s.first + s.tiles - 1, n_cta);
                    uint32_t* counter = p.counters + s.e * p.Hkv + s.idx;
                    const uint32_t done = atomicAdd(counter, 1u);
                    const bool last = done == static_cast<uint32_t>(c1 - c0);
                    if (last) *counter = 0u;  // for the next launch
                    *last_flag = last ? 1u : 0u;
                }
            }
            group_sync();
            const bool last = *last_flag != 0u;
            group_sync();
            if (last) {
                __threadfence();
                const int c0 = share_of(work.total, s.first, n_cta);
                const int c1 = share_of(work.total, s.first + s.tiles - 1, n_cta);
                // Part of CTA k: its first segment unless the pair starts inside its share.
                auto part_of = [&](int k) { return k * 2 + (s.first <= share_start(work.total, k, n_cta) ? 0 : 1); };
                for (int i = tid; i < p.G * D; i += kWarps * 32) {
                    const int h = i / D;
                    float m = -INFINITY;
                    for (int k = c0; k <= c1; ++k) m = fmaxf(m, __ldcg(p.part_ml + (static_cast<int64_t>(part_of(k)) * p.G + h) * 2));
                    float sum = 0.f, acc = 0.f;
                    for (int k = c0; k <= c1; ++k) {
                        const int64_t a = static_cast<int64_t>(part_of(k)) * p.G + h;
                        const float mk = __ldcg(p.part_ml + a * 2), lk = __ldcg(p.part_ml + a * 2 + 1);
                        const float w = mk == m ? 1.f : fast_exp2(mk - m);
                        sum += lk * w;
                        acc += __ldcg(p.part_o + a * D + i % D) * w;
                    }
                    p.out[s.e * p.out_stride + g * p.G * D + i] = __float2bfloat16(acc * (v_scale / sum));
                }
            }
        }
        u += s.t1 - s.t0;
    }
    if (!ok && lane == 0) report(v.err, kErrPagedWait);
}

template <int D, bool FP8>
cudaError_t launch_one(const PagedDecodeParams& p, const PagedMaps& m, int num_sms, cudaStream_t s) {
    const int smem = smem_bytes(D, p.n);
    static SmemLimitOnce limit;
    const cudaError_t e = limit.apply(reinterpret_cast<const void*>(&paged_decode_kernel<D, FP8>), 113 * 1024);
    if (e != cudaSuccess) return e;
    int ctas = num_sms * kCtasPerSm;
    if (ctas > kPagedMaxCtas) ctas = kPagedMaxCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &paged_decode_kernel<D, FP8>, p, m);
}

}  // namespace

cudaError_t launch_paged_decode(const PagedDecodeParams& p, const PagedMaps& m, int fp8, int num_sms, cudaStream_t s) {
    if (p.v.D == 128) return fp8 ? launch_one<128, true>(p, m, num_sms, s) : launch_one<128, false>(p, m, num_sms, s);
    return fp8 ? launch_one<64, true>(p, m, num_sms, s) : launch_one<64, false>(p, m, num_sms, s);
}

}  // namespace duo
