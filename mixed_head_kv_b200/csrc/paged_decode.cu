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
//     head) pairs, then of all streaming pairs, form one list, and every pair has
//     one unit more, for the work at its end, which takes about as long as a tile.
//     CTA c takes the c-th equal share of the units. Ragged batches, one long
//     sequence and many short ones balance alike, and the lengths are read on
//     the device: a captured launch stays right as the sequences grow;
//   - a pair cut by a share boundary is joined by the last of its CTAs to
//     finish: each leaves its unnormalised sums, maximum and weight in the
//     workspace, at most two per CTA, and counts itself once all its tiles are
//     done (counting and joining between tiles cost 2 to 6 us of streaming each).
//     The joining order is the CTA order, so results do not depend on which CTA
//     is last.
// Two CTAs per SM: 4 warps compute, 1 warp loads.
//   - the loading warp finds the pairs of the share, publishes each through a
//     2-slot ring together with the group's queries and the new rows, and streams
//     tiles through a ring of 96 KB by TMA (boxes of page or tile size, 128-byte
//     swizzle; page numbers are fetched 32 at a time);
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
//     relative to the same maximum). P is rounded to the operand type: bf16, relative
//     error at most 2^-8 per term; with E4M3 f16, 2^-11, of weights times 2^7, the most
//     that f16 holds when they reach 2^8: what is below 2^-21 of the maximum so far
//     has an absolute error of 2^-32 of it instead (without the factor 2^-14 and 2^-25:
//     beside one large key, thousands of rows weighed nothing in O and something in the sum).
//     Groups of up to four leave half of the N side free: with bf16 its columns 4 .. 7 hold
//     the same heads again and take what the rounding left of each weight, rounded in
//     turn. The two sums are added at the segment's end, and these groups lose 2^-16 per
//     term, as little as the contiguous caches' groups of one and two, which multiply in
//     32 bits (4 x 131072 tokens 165.0 us instead of 164.7, 529 tokens 7.6 instead of 7.5; for
//     codes, whose weights lose 2^-11, the same cost 5 % and is not done).
// Measured (captured launches): 4 x 131072 tokens, groups of 4, half of 8 KV heads
// retrieval: 165 us, 6.53 TB/s, the copy rate. 32769 tokens, 8 of 32 heads
// retrieval: 30.5 us, 4.5 TB/s; 48 ragged sequences of E4M3 codes 22 us; 200 of
// groups of 8 23.5 us; 529 tokens 7.7 us. What the smaller ones take beyond the
// bytes is fixed: about 3 us until the first tiles arrive (lengths, the sums over
// the entries, page numbers, rows: a chain of loads), 2 us at each pair's end and
// 4 us for counting and joining.
// Rows behind the last one in a page hold anything: their scores are replaced,
// and their V rows are zeroed in shared memory (0 x NaN would not be 0).
#include "paged_internal.cuh"
#include "paged_shares.cuh"
#include "sm100.cuh"

namespace duo {

namespace {

constexpr int kWarps = 4;                 // computing warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kCtasPerSm = 2;
constexpr int kRingBytes = 96 * 1024;
constexpr int kMaxG = DUO_PAGED_MAX_GROUP;
// Units of work at the end of a pair. (48 and 200 ragged sequences, outside a captured
// launch: 24.3 and 27.2 us; with 2 units 24.5 and 26.7, with 3 25.5 and 28.0.)
constexpr int kEndUnits = 1;
// Weights that become f16 are 2^kLift times what they are: 2^8 x 2^7 at most, of 2^16.
constexpr float kLift = 7.f;

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
// What rounding x0 and x1 to the two numbers of `w` left, rounded too.
__device__ __forceinline__ uint32_t bf16x2_rest(uint32_t w, float x0, float x1) {
    return pack_bf16x2(x0 - bf16lo_to_f32(w), x1 - bf16hi_to_f32(w));
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint4& x) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w) : "memory");
}

// The computing warps' barrier.
__device__ __forceinline__ void group_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

__device__ __forceinline__ bool group_any(bool x) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0u;
}

// The sums over the warps of accumulators [W n, W n + n), n = steps / 4, in warp W.
// In round i a warp hands its part of quarter W + i over: 4 KB serve all.
template <int W, int kSteps>
__device__ __forceinline__ void gather_quarter(const float (&o)[kSteps][4], float (&r)[kSteps / kWarps][4], float* merge,
                                               int lane) {
    constexpr int n = kSteps / kWarps;
#pragma unroll
    for (int i = 0; i < n; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = o[W * n + i][j];
#pragma unroll
    for (int t = 1; t < kWarps; ++t) {
        constexpr int mask = kWarps - 1;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const int k = ((W + t) & mask) * n + i;
            *reinterpret_cast<float4*>(merge + (k * 32 + lane) * 4) = make_float4(o[k][0], o[k][1], o[k][2], o[k][3]);
        }
        group_sync();
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float4 y = *reinterpret_cast<const float4*>(merge + ((W * n + i) * 32 + lane) * 4);
            r[i][0] += y.x;
            r[i][1] += y.y;
            r[i][2] += y.z;
            r[i][3] += y.w;
        }
        if (t + 1 < kWarps) group_sync();
    }
}

// One stretch of tiles of one (entry, KV head) pair inside a CTA's share.
struct Segment {
    int e, seq, len;     // entry, sequence, its tokens
    int idx;             // index of the head in the layer's list (retrieval first)
    int retr;            // 1: pages, 0: window
    int t0, t1, tiles;   // tiles [t0, t1) of `tiles`
    int units;           // units of the list it takes up
    int new_row;         // the new token's row in the pages' list or the window
    int parts;           // shares that hold tiles of the pair
    int part0;           // slot of the first share's part; those of the others follow, two apart from 2 (share + 1)
};

template <int D>
struct Smem {
    static constexpr int kStage = D * 256;  // K and V of a tile
    static constexpr int kStages = kRingBytes / kStage;
    static constexpr int kRing = 0;
    static constexpr int kQSlot = (kMaxG + 2) * D * 2;  // queries, new K row, new V row
    static constexpr int kQ = kRing + kRingBytes;
    static constexpr int kMerge = kQ + 2 * kQSlot;      // one warp's O
    static constexpr int kStat = kMerge + kMaxG * D * 4;  // maximum and sum of a warp's heads
    static_assert(kStat % 16 == 0, "read as int4 at first");
    static constexpr int kBar = kStat + kWarps * kMaxG * 2 * 4;
    static constexpr int kMisc = kBar + 32 * 8;
    static constexpr int kSeg = kMisc + 16;     // the two segments in flight, and two cut pairs to be joined
    static constexpr int kHeads = kSeg + 4 * static_cast<int>(sizeof(Segment));  // the layer's KV heads
    static constexpr int kPrefix = kHeads + DUO_MAX_KV_HEADS * 2;  // per entry: length, tiles before (retrieval, streaming), sequence
};
__host__ __device__ constexpr int smem_bytes(int D, int n) {
    return (D == 128 ? Smem<128>::kPrefix : Smem<64>::kPrefix) + (n + 1) * 8 + n * 4 + n * 2 + 8;
}
static_assert(smem_bytes(128, kPagedMaxBatch) <= 113 * 1024, "two CTAs per SM");

// Division, one copy for the whole kernel: most of its code is run once per CTA, and
// what runs once waits for the instruction cache line by line.
__device__ __noinline__ int64_t divide(int64_t a, int64_t b) {  // both >= 0, b > 0
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// T units over n CTAs: the first `more` shares hold `base` + 1 units, the others `base`.
struct Shares {
    int64_t base;
    int more;
    __device__ __forceinline__ int64_t start(int c) const { return base * c + (c < more ? c : more); }
    __device__ __forceinline__ int of(int64_t u) const {
        const int64_t large = (base + 1) * more;
        return u < large ? static_cast<int>(divide(u, base + 1)) : more + static_cast<int>(divide(u - large, base));
    }
};

// The list of work: units are the tiles of a pair and kEndUnits for its end (joining
// the warps and writing the result takes about as long as a tile), so that shares
// of many short pairs weigh as much as shares of long ones.
struct Work {
    const int* len;
    const int* before_r;  // [n + 1] units of one retrieval head before entry i
    const int* before_s;
    const uint16_t* seq;
    int n, n_retr, n_strm;
    int64_t of_retr;
    Shares shares;
    int c;                // this CTA's share

    // Unit `at` of the pair is unit u of the list; `n` units in the pair.
    __device__ __forceinline__ void fill(Segment& s, int n, int at, int64_t u, int64_t hi) const {
        const int64_t left = hi - u;
        const int end = left < n - at ? at + static_cast<int>(left) : n;
        s.tiles = n - kEndUnits;
        s.units = end - at;
        s.t0 = at < s.tiles ? at : s.tiles;
        s.t1 = end < s.tiles ? end : s.tiles;
        s.seq = seq[s.e];
        s.len = len[s.e];
    }
    // Where the parts of the pair are, for a segment that starts at unit u and has tiles.
    __device__ __forceinline__ void find_parts(Segment& s, int64_t u) const {
        s.parts = 1;
        s.part0 = 0;
        if (s.t1 - s.t0 < s.tiles) {
            const int64_t first = u - s.t0;
            const int c0 = s.t0 == 0 ? c : shares.of(first);
            const int c1 = s.t1 == s.tiles ? c : shares.of(first + s.tiles - 1);
            s.parts = c1 - c0 + 1;
            // A share has two slots: 2 c for the pair that it begins in, 2 c + 1 for the one that it ends in.
            s.part0 = 2 * c0 + (first > shares.start(c0) ? 1 : 0);
        }
    }
    // The segment that starts at unit u and ends at `hi` at the latest.
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
        const int units = before[lo + 1] - before[lo];
        const int64_t y = x - static_cast<int64_t>(before[lo]) * heads;
        const int h = static_cast<int>(divide(y, units));
        s.idx = s.retr ? h : n_retr + h;
        fill(s, units, static_cast<int>(y - static_cast<int64_t>(h) * units), u, hi);
        return s;
    }
    // The one behind it, which starts at unit u: the next head, or the next entry
    // with rows, or the first of the windows.
    __device__ __forceinline__ void next(Segment& s, int64_t u, int64_t hi) const {
        int units = s.tiles + kEndUnits;
        ++s.idx;
        if (s.idx == (s.retr ? n_retr : n_retr + n_strm)) {
            if (u == of_retr) {
                s.retr = 0;
                s.e = -1;
            }
            const int* before = s.retr ? before_r : before_s;
            do {
                ++s.e;
                units = before[s.e + 1] - before[s.e];
            } while (units == 0);
            s.idx = s.retr ? 0 : n_retr;
        }
        fill(s, units, 0, u, hi);
    }
};

__device__ __forceinline__ void report(uint32_t* err, uint32_t bit) { atomicOr(err, bit); }

// The window row of position pos.
__device__ __forceinline__ int window_slot(const PagedView& v, int pos) {
    return pos < v.S ? pos : v.S + (pos - v.S) % v.R;
}

// Joins the parts of a cut pair into its G output rows. A warp takes a head (with
// fewer than four heads, the parts of a head are shared out between warps): its
// lanes read the parts' statistics at once, D / 32 columns each of eight parts at a
// time. The first eight are on their way before the statistics that weigh them.
template <int D>
__device__ __forceinline__ void join_parts(const PagedDecodeParams& p, const Segment& s, int g, float v_scale, float* merge,
                                           int warp, int lane) {
    constexpr int V = D / 32, B = 8;  // columns per lane, parts per batch
    const int n = s.parts;
    const int split = p.G == 1 ? kWarps : p.G == 2 ? kWarps / 2 : 1;  // warps per head
    const int sub = warp & (split - 1);
    // Part k is in slot part0 for k = 0, else in slot 2 (c0 + k).
    const int even = s.part0 & ~1;
    for (int h0 = 0; h0 < p.G; h0 += kWarps / split) {
        const int h = h0 + warp / split;
        const bool on = h < p.G;  // else the warp works on head 0 and keeps it to itself
        const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + (on ? h : 0);
        const float* po = p.part_o + (on ? h : 0) * D + lane * V;
        float m = -INFINITY, sum = 0.f, w = 0.f, acc[V];
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 1
        for (int c = 0; c < n; c += 32) {  // 32 parts with their weights one per lane
#pragma unroll 1
            for (int k0 = c + sub; k0 < n && k0 < c + 32; k0 += B * split) {
                float x[B][V];
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int k = k0 + j * split;
                    const float* src = po + static_cast<int64_t>((k == 0 || k >= n ? s.part0 : even + 2 * k) * p.G) * D;
                    if (V == 4) *reinterpret_cast<float4*>(x[j]) = __ldcg(reinterpret_cast<const float4*>(src));
                    else *reinterpret_cast<float2*>(x[j]) = __ldcg(reinterpret_cast<const float2*>(src));
                }
                if (k0 == c + sub) {
                    auto stat_of = [&](int k) {
                        return k < n ? __ldcg(ml + (k == 0 ? s.part0 : even + 2 * k) * p.G) : make_float2(-INFINITY, 0.f);
                    };
                    if (c == 0) {  // the joint maximum
#pragma unroll 1
                        for (int k = 0; k < n; k += 32) m = fmaxf(m, stat_of(k + lane).x);
#pragma unroll
                        for (int d = 1; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
                    }
                    const float2 y = stat_of(c + lane);
                    w = y.x == m ? 1.f : fast_exp2(y.x - m);
                    sum += y.y * w;  // (used by the head's first warp, which has a part of every batch)
                }
#pragma unroll
                for (int j = 0; j < B; ++j) {
                    const int k = k0 + j * split;
                    const float f = __shfl_sync(0xffffffffu, w, k & 31);
                    if (k < n && k < c + 32)
#pragma unroll
                        for (int v = 0; v < V; ++v) acc[v] += x[j][v] * f;
                }
            }
        }
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (split > 1) {
#pragma unroll
            for (int v = 0; v < V; ++v) merge[(warp * V + v) * 32 + lane] = acc[v];
            group_sync();
            if (sub == 0)
#pragma unroll 1
                for (int o = 1; o < split; ++o)
#pragma unroll
                    for (int v = 0; v < V; ++v) acc[v] += merge[((warp + o) * V + v) * 32 + lane];
        }
        if (on && sub == 0) {
            const float f = v_scale / sum;
            bf16* dst = p.out + s.e * p.out_stride + (g * p.G + h) * D + lane * V;
#pragma unroll
            for (int v = 0; v < V; v += 2) *reinterpret_cast<uint32_t*>(dst + v) = pack_bf16x2(acc[v] * f, acc[v + 1] * f);
        }
    }
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
    int16_t* heads = reinterpret_cast<int16_t*>(smem + L::kHeads);
    if (tid < p.h.n_retr + p.h.n_strm) heads[tid] = p.h.head[tid];
    if (warp == kWarps && lane < 4 && (lane < 2 ? p.v.r_all : p.v.s_all) > 0)  // a pool without heads has no map
        tma_prefetch_desc(lane == 0 ? &maps.k : lane == 1 ? &maps.v : lane == 2 ? &maps.wk : &maps.wv);
    // Marks of the sequences named once and twice, in the ring before its first tile.
    uint32_t* once = reinterpret_cast<uint32_t*>(smem + L::kRing);
    uint32_t* twice = once + kPagedMaxSeqs / 32;
    for (int i = tid; i < kPagedMaxSeqs / 32; i += kThreads) once[i] = twice[i] = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    __syncthreads();
    // The entries, four in a row per thread: lengths, then the units before each by a
    // scan over the CTA. Entries named twice count as skipped.
    constexpr int kOwn = 4;
    static_assert(kOwn * kThreads >= kPagedMaxBatch, "every entry has a thread");
    const int i0 = tid * kOwn;
    int my_seq[kOwn], my_len[kOwn];
#pragma unroll
    for (int j = 0; j < kOwn; ++j) my_seq[j] = i0 + j < p.n ? p.seqs[i0 + j] : -1;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        if (my_seq[j] >= v.max_seqs) my_seq[j] = -1;
        my_len[j] = my_seq[j] >= 0 ? v.seq_len[my_seq[j]] : -1;
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int s = my_seq[j];
        if (s >= 0) {
            const uint32_t bit = 1u << (s & 31);
            if (atomicOr(&once[s >> 5], bit) & bit) atomicOr(&twice[s >> 5], bit);
        }
    }
    __syncthreads();
    int sum_r = 0, sum_s = 0, longest = 0;  // units; of the longest pair
    bool wrong = false;
#pragma unroll
    for (int j = 0; j < kOwn; ++j) {
        const int s = my_seq[j];
        if (s >= 0) {
            const bool bad = ((twice[s >> 5] >> (s & 31)) & 1u) != 0u || my_len[j] < 0 ||
                             my_len[j] > v.max_pages << v.P_log2;  // the table holds at most 2^27 tokens
            wrong |= bad;
            my_len[j] = bad ? -1 : my_len[j];
        }
        if (i0 + j < p.n) {
            before_r[i0 + j] = sum_r;
            before_s[i0 + j] = sum_s;
            len_of[i0 + j] = my_len[j];
            seq_of[i0 + j] = static_cast<uint16_t>(s < 0 ? 0 : s);
        }
        if (my_len[j] > 0) {  // tiles, and the end of the pair
            const int units_r = (my_len[j] + kPageTile - 1) / kPageTile + kEndUnits;
            const int units_s = ((my_len[j] < v.W ? my_len[j] : v.W) + kWinTile - 1) / kWinTile + kEndUnits;
            sum_r += units_r;
            sum_s += units_s;
            if (p.h.n_retr > 0) longest = max(longest, units_r);
            if (p.h.n_strm > 0) longest = max(longest, units_s);
        }
    }
    if (wrong && blockIdx.x == 0) report(v.err, kErrPagedArgument);
    __syncwarp();
    const int own_r = sum_r, own_s = sum_s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum_r, o), y = __shfl_up_sync(0xffffffffu, sum_s, o);
        sum_r += lane >= o ? x : 0;
        sum_s += lane >= o ? y : 0;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    int4* const of_warp = reinterpret_cast<int4*>(smem + L::kStat);
    if (lane == 31) of_warp[warp] = make_int4(sum_r, sum_s, longest, 0);
    fence_proxy_async_smem();  // the marks' words become TMA destinations
    __syncthreads();
    int total_r = 0, total_s = 0, off_r = sum_r - own_r, off_s = sum_s - own_s;
#pragma unroll
    for (int w = 0; w <= kWarps; ++w) {
        const int4 x = of_warp[w];
        longest = max(longest, x.z);
        off_r += w < warp ? x.x : 0;
        off_s += w < warp ? x.y : 0;
        total_r += x.x;
        total_s += x.y;
    }
#pragma unroll
    for (int j = 0; j < kOwn; ++j)
        if (i0 + j < p.n) {
            before_r[i0 + j] += off_r;
            before_s[i0 + j] += off_s;
        }
    if (tid == 0) {
        before_r[p.n] = total_r;
        before_s[p.n] = total_s;
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
    work.of_retr = static_cast<int64_t>(total_r) * p.h.n_retr;
    const int64_t total = work.of_retr + static_cast<int64_t>(total_s) * p.h.n_strm;
    const int n_cta = share_count(total, longest, gridDim.x);
    const int c = blockIdx.x;
    if (c >= n_cta) return;
    Segment* const slots = reinterpret_cast<Segment*>(smem + L::kSeg);

    if (warp == kWarps) {
        // ------------------------------------------------------------ loads
        work.c = c;
        work.shares.base = divide(total, n_cta);
        work.shares.more = static_cast<int>(total - work.shares.base * n_cta);
        const int64_t lo = work.shares.start(c), hi = work.shares.start(c + 1);
        int st = 0, round = 0;  // ring position
        int n_seg = 0;
        bool ok = true;
        Segment s = work.at(lo, hi);
        for (int64_t u = lo; ok && u < hi;) {
            if (s.t0 == s.t1) {  // only the end of a pair whose tiles other shares hold
                u += s.units;
                if (u < hi) work.next(s, u, hi);
                continue;
            }
            const int g = heads[s.idx];
            const int slot = n_seg & 1;
            if (n_seg >= 2 && !mbar_wait(bar(kQEmpty + slot), ((n_seg >> 1) - 1) & 1, abort_flag)) {
                ok = false;
                break;
            }
            if (lane == 0) {
                const uint32_t q = base + L::kQ + slot * L::kQSlot;
                mbar_expect_tx(bar(kQFull + slot), (p.G + 2) * D * 2);
                bulk_load(q, p.q + s.e * p.q_stride + g * p.G * D, p.G * D * 2, bar(kQFull + slot));
                bulk_load(q + kMaxG * D * 2, p.k_new + s.e * p.kv_stride + g * D, D * 2, bar(kQFull + slot));
                bulk_load(q + (kMaxG + 1) * D * 2, p.v_new + s.e * p.kv_stride + g * D, D * 2, bar(kQFull + slot));
            }
            const int rows = s.retr ? s.len : (s.len < v.W ? s.len : v.W);
            const int* row_table = v.table + static_cast<int64_t>(s.seq) * v.max_pages;
            const int n_pages = (s.len + v.P - 1) >> v.P_log2;
            // Page numbers, 32 at a time: `have` covers [win, win + 32), `next` the 32 behind.
            int win = 0, have = 0, next = 0;
            if (s.retr) {
                win = s.t0 * kPageTile >> v.P_log2;  // a sequence has at most 2^27 tokens
                have = win + lane < n_pages ? row_table[win + lane] : -1;
                next = win + 32 + lane < n_pages ? row_table[win + 32 + lane] : -1;
            }
            // The new token's row goes into the cache here, off the computing warps' path:
            // lanes 0-15 K, 16-31 V, 16 bytes each. Its loads are issued now and used
            // behind the segment's tiles.
            const int new_row = s.new_row = s.retr ? s.len - 1 : window_slot(v, s.len - 1);
            const int new_tile = new_row / (s.retr ? kPageTile : kWinTile);
            const int which = lane >> 4, ch = lane & 15;
            const bool owner = new_tile >= s.t0 && new_tile < s.t1 && ch < D / 8;
            uint4 fresh = make_uint4(0, 0, 0, 0);
            int new_page = -1, new_ref = 0;
            float inv_scale = 1.f;
            if (owner) {
                fresh = ld_nc_v4((which ? p.v_new : p.k_new) + s.e * p.kv_stride + g * D + ch * 8);
                if (s.retr) new_page = row_table[new_row >> v.P_log2];
                if (FP8) inv_scale = p.kv_scale[g * 4 + 2 + which];
            }
            work.find_parts(s, u);  // while the loads above are on their way
            if (lane == 0) {
                slots[slot] = s;
                mbar_arrive(bar(kQFull + slot));  // releases the segment
            }
            if (p.test_withhold != 0 && c == 0) {  // a test of the waits for these tiles: none is loaded
                mbar_wait(bar(kEmpty), 0, abort_flag, 2 * kWaitTimeoutNs);
                ok = false;
            }
            for (int t = s.t0; ok && t < s.t1; ++t) {
                if (round > 0 && !mbar_wait(bar(kEmpty + st), (round - 1) & 1, abort_flag)) {
                    ok = false;
                    break;
                }
                const uint32_t dst = base + L::kRing + st * L::kStage;
                if (s.retr) {
                    const int row0 = t * kPageTile;
                    const int valid = rows - row0 < kPageTile ? rows - row0 : kPageTile;
                    const int box = v.P < kPageTile ? v.P : kPageTile;  // rows of one copy
                    const int n_box = (valid + box - 1) >> (v.P < kPageTile ? v.P_log2 : kPageTile == 64 ? 6 : 7);
                    const int pg0 = row0 >> v.P_log2;
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
                        const int y = row0 & (v.P - 1);
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
                if (t == s.t0 && new_page >= 0 && new_page < v.num_pages) new_ref = v.ref[new_page];
                if (++st == L::kStages) {
                    st = 0;
                    ++round;
                }
            }
            if (owner) {
                if (!ok && new_page >= 0 && new_page < v.num_pages) new_ref = v.ref[new_page];  // perhaps not looked at yet
                if (!s.retr) {
                    bf16* dst = (which ? v.v_window : v.k_window) +
                                ((static_cast<int64_t>(s.seq) * v.s_all + p.h.s0 + s.idx - p.h.n_retr) * v.W + new_row) * D + ch * 8;
                    *reinterpret_cast<uint4*>(dst) = fresh;
                } else if (new_ref > 1) {
                    report(v.err, kErrPagedShared);
                } else if (new_page >= 0 && new_page < v.num_pages) {  // else the loads reported it
                    const int64_t at = ((static_cast<int64_t>(new_page) * v.r_all + p.h.r0 + s.idx) * v.P + (new_row & (v.P - 1))) * D + ch * 8;
                    uint8_t* pool = which ? v.v_pages : v.k_pages;
                    if (FP8) *reinterpret_cast<uint2*>(pool + at) = e4m3x8_from_bf16x8(fresh, inv_scale);
                    else *reinterpret_cast<uint4*>(pool + at * 2) = fresh;
                }
            }
            ++n_seg;
            u += s.units;
            if (u < hi) work.next(s, u, hi);
        }
        if (!ok && lane == 0) {
            *abort_flag = 1;
            report(v.err, kErrPagedWait);
        }
        // The end: a segment without tiles.
        if (n_seg >= 2) ok = mbar_wait(bar(kQEmpty + (n_seg & 1)), ((n_seg >> 1) - 1) & 1, abort_flag) && ok;
        if (lane == 0) {
            slots[n_seg & 1].tiles = 0;
            mbar_arrive(bar(kQFull + (n_seg & 1)));
        }
        // Every copy issued lands before the CTA may exit.
        for (int i = 0; i < L::kStages; ++i) {
            const int rounds = round + (i < st ? 1 : 0);  // times stage i was filled
            if (rounds > 0) mbar_wait(bar(kFull + i), (rounds - 1) & 1, nullptr);
        }
        if (n_seg >= 1) mbar_wait(bar(kQFull + ((n_seg - 1) & 1)), ((n_seg - 1) >> 1) & 1, nullptr);
        return;
    }

    // ---------------------------------------------------------------- computing warps
    const int gq = lane >> 2;  // row of an accumulator, column of an operand: key / head
    const int cq = lane & 3;
    constexpr int kSteps = D / 16;
    int st = 0, round = 0;
    int n_seg = 0;
    bool ok = true;
    float* merge = reinterpret_cast<float*>(smem + L::kMerge);
    float* stat = reinterpret_cast<float*>(smem + L::kStat);  // [warp][head][2]
    Segment* const pending = slots + 2;
    int n_pending = 0;
    for (;; ++n_seg) {
        const int slot = n_seg & 1;
        const uint32_t q = base + L::kQ + slot * L::kQSlot;
        if (ok && !mbar_wait(bar(kQFull + slot), (n_seg >> 1) & 1, abort_flag)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abort_flag = 1;
        const Segment s = slots[slot];
        if (group_any(!ok) || s.tiles == 0) break;  // the same for all four warps
        const int g = heads[s.idx];
        const bool codes = FP8 && s.retr;  // operands are f16 made of codes
        const bool two_parts = p.G <= 4 && !codes;   // of each weight
        const int head_q = two_parts ? gq & 3 : gq;  // column gq's head
        // The queries as the B operand: column gq, this thread's part of D.
        uint32_t b[kSteps][2];
        float scale0 = p.scale_log2, scale1 = p.scale_log2;  // of columns 2 cq and 2 cq + 1
        if (!codes) {
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const uint32_t a = q + head_q * D * 2 + k * 32 + cq * 4;
                b[k][0] = b[k][1] = 0u;
                if (head_q < p.G) {
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
        const int new_row = s.new_row;
        const int tile_rows = s.retr ? kPageTile : kWinTile;
        for (int t = s.t0; t < s.t1; ++t) {
            const uint32_t kt = base + L::kRing + st * L::kStage, vt = kt + kHalf;
            if (ok && !mbar_wait(bar(kFull + st), round & 1, abort_flag)) ok = false;
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) *abort_flag = 1;
            const int per = tile_rows / kWarps;  // this warp's rows of the tile
            const int w0 = warp * per;
            const int valid = rows - t * tile_rows - w0;  // of them, rows to attend to
            bool touched = false;
            if (ok && valid > 0) {
                // The new token's row goes over what the cache held in its place.
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
                    }
                }
                if (valid < per) {  // V rows behind the last one
                    touched = true;
                    constexpr int kPieces = D / 8;  // 16 bytes each of a bf16 row; half as many of codes
                    if (codes) {
                        for (int i = lane; i < (per - valid) * (kPieces / 2); i += 32)
                            sts128(vt + (w0 + valid) * D + i * 16, make_uint4(0, 0, 0, 0));
                    } else {
                        for (int i = lane; i < (per - valid) * kPieces; i += 32) {
                            const int r = w0 + valid + i / kPieces, ch = i % kPieces;
                            sts128(vt + (ch >> 3) * (tile_rows * 128) + r * 128 + (ch & 7) * 16, make_uint4(0, 0, 0, 0));
                        }
                    }
                }
                __syncwarp();
                const int parts = per / 16;  // 1, or 2 with codes
#pragma unroll 1
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
                    // Rows gq and gq + 8, columns 2 cq and 2 cq + 1.
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
                    x[0] -= u0;
                    x[1] -= u1;
                    x[2] -= u0;
                    x[3] -= u1;
                    if (codes) {  // to the difference: a large maximum less kLift would be rounded
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] += kLift;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = fast_exp2(x[i]);
                    l0 += x[0] + x[2];
                    l1 += x[1] + x[3];
                    // P^T from accumulator to operand layout.
                    uint32_t w01 = codes ? pack_f16x2(x[0], x[1]) : pack_bf16x2(x[0], x[1]);
                    uint32_t w23 = codes ? pack_f16x2(x[2], x[3]) : pack_bf16x2(x[2], x[3]);
                    if (two_parts) {
                        const uint32_t rest01 = bf16x2_rest(w01, x[0], x[1]), rest23 = bf16x2_rest(w23, x[2], x[3]);
                        w01 = cq >= 2 ? rest01 : w01;
                        w23 = cq >= 2 ? rest23 : w23;
                    }
                    const uint32_t p0 = transpose8x8(w01), p1 = transpose8x8(w23);
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
            if (++st == L::kStages) {
                st = 0;
                ++round;
            }
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
        // O: warp w ends up with the sums of quarter w of the accumulators.
        float r[kSteps / kWarps][4];
        if (warp == 0) gather_quarter<0, kSteps>(o, r, merge, lane);
        else if (warp == 1) gather_quarter<1, kSteps>(o, r, merge, lane);
        else if (warp == 2) gather_quarter<2, kSteps>(o, r, merge, lane);
        else gather_quarter<3, kSteps>(o, r, merge, lane);
        if (two_parts) {
            // Columns 0 .. 3 take the second parts' sums from columns 4 .. 7. Where a value row
            // has an infinity the first sum is the answer: a second part may be zero or negative.
#pragma unroll
            for (int i = 0; i < kSteps / kWarps; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float rest = __shfl_down_sync(0xffffffffu, r[i][j], 2);
                    r[i][j] += isfinite(r[i][j]) ? rest : 0.f;
                }
        }
        const int i0 = warp * (kSteps / kWarps);
        // Column of D that accumulator i holds in its first (half 0) or second pair.
        auto col = [&](int i, int half) { return codes ? gq * (D / 8) + 2 * i + half : i * 16 + half * 8 + gq; };
        const bool whole = s.t0 == 0 && s.t1 == s.tiles;
        if (whole) {
            const float v_scale = codes ? p.kv_scale[g * 4 + 1] : 1.f;
            const float inv[2] = {v_scale / lj[0], v_scale / lj[1]};
            bf16* dst = p.out + s.e * p.out_stride + (g * p.G + 2 * cq) * D;
            if (ok) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (2 * cq + h < p.G)
#pragma unroll
                        for (int i = 0; i < kSteps / kWarps; ++i)
#pragma unroll
                            for (int j = 0; j < 2; ++j)
                                dst[h * D + col(i0 + i, j)] = __float2bfloat16(r[i][2 * j + h] * inv[h]);
            }
        } else {
            const int part = 2 * c + (s.t0 == 0 && s.part0 == 2 * c + 1 ? 1 : 0);
            float* po = p.part_o + (static_cast<int64_t>(part) * p.G + 2 * cq) * D;
            float* pm = p.part_ml + static_cast<int64_t>(part) * p.G * 2;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (2 * cq + h < p.G)
#pragma unroll
                    for (int i = 0; i < kSteps / kWarps; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j) po[h * D + col(i0 + i, j)] = r[i][2 * j + h];
            if (warp == 0 && gq == 0) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (2 * cq + i < p.G) {
                        pm[(2 * cq + i) * 2] = mj[i];
                        pm[(2 * cq + i) * 2 + 1] = lj[i];
                    }
            }
            if (tid == 0) pending[n_pending] = s;
            ++n_pending;
        }
        // The next segment's group_any() is the barrier behind the last reads of stat and merge.
    }
    if (!ok && lane == 0) report(v.err, kErrPagedWait);
    // ---------------------------------------------------------------- cut pairs
    // A share cuts at most two pairs, at its ends. They are counted here, behind all
    // tiles: each step of the chain (writes out, count, other parts in) takes a
    // memory latency, which is several times longer while the tiles stream.
    if (n_pending > 0) {
        group_sync();
        if (tid == 0) {
            // Releases the CTA's writes (ordered before by the barrier), then acquires
            // the other parts' of the pairs that it is the last to finish.
            asm volatile("fence.acq_rel.gpu;" ::: "memory");
            uint32_t* const c0 = p.counters + pending[0].e * p.Hkv + pending[0].idx;
            uint32_t* const c1 = p.counters + pending[1].e * p.Hkv + pending[1].idx;
            const uint32_t b0 = atomicAdd(c0, 1u);
            const uint32_t b1 = n_pending > 1 ? atomicAdd(c1, 1u) : 0u;
            uint32_t last = 0;
            if (b0 + 1u == static_cast<uint32_t>(pending[0].parts)) {
                last |= 1u;
                *c0 = 0u;  // for the next launch
            }
            if (n_pending > 1 && b1 + 1u == static_cast<uint32_t>(pending[1].parts)) {
                last |= 2u;
                *c1 = 0u;
            }
            asm volatile("fence.acq_rel.gpu;" ::: "memory");
            *last_flag = ok ? last : 0u;
        }
        group_sync();
        for (int i = 0; i < n_pending; ++i)
            if ((*last_flag >> i) & 1u) {
                const Segment s = pending[i];
                const int g = heads[s.idx];
                join_parts<D>(p, s, g, FP8 && s.retr ? p.kv_scale[g * 4 + 1] : 1.f, merge, warp, lane);
                group_sync();  // the joining buffer is free again
            }
    }
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
