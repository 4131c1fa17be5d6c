// prefill_packed.cu — causal attention of whole prompts packed one behind the
// other (duo_paged_prefill), on tcgen05.
//
// out_i = sum_{j <= i, seen} softmax_j(scale q_i . k_j) v_j within each prompt;
// a streaming head's query sees j < sink or i - j < recent only.
//
// Work item = two tiles A and B of 128 query rows that read the same K and V
// tiles: two query heads of one KV head over the same rows (even query groups),
// or 256 rows of one query head (odd groups). Sharing halves the K/V traffic into
// shared memory, and the two tiles' softmax run half a step apart: while the
// tensor core works on one tile the other's exponentials are computed. Per pair
// of tiles and 128 keys the tensor core needs 2048 cycles (4 products of
// 128 x 128 x D) and the 16-lane exponential unit of an SM as many, so the two
// pipes bound the kernel together.
//
// One persistent CTA per SM takes items from a counter, retrieval heads first,
// longest prompts first, last query tiles first: the long items start early and
// the short ones fill the end. Which prompts there are is read on the device by
// every CTA (at most 512 lengths, ranked in shared memory). Key tiles that no
// row of the item sees are never listed: a streaming item has its sink tiles and
// the band of its window.
//
// Warp roles (384 threads; registers moved from the last group to the others):
//   warps 0-3  softmax of tile A, one thread per row    warps 4-7  of tile B
//   warp 8     takes the items, loads Q, the K and the V tiles (2 stages each)
//   warp 9     issues the products (the whole warp runs the loop, one lane issues),
//              owns TMEM
//   warps 10-11 clear the V tiles that are seen in part of what a weight of zero
//              must not meet
// TMEM (512 columns): S of A and B, 128 columns each, P (bf16) written over the S
// it was made from, O of A and of B at 256.
// Softmax in the exp2 domain; the running maximum moves when a score exceeds it by more
// than 2^8, and to any higher score once 64 weights have added up to more than 2^10
// (exact: all terms stay relative to the same maximum), sums in 32 bits; P rounded to
// bf16, the operand type (relative 2^-8 at most per term). Every mbarrier wait is bounded;
// on timeout the CTA records kErrPagedWait and unwinds.
//
// Measured: 32768 rows, D = 128: 8 retrieval heads 1.68 ms, 1310 TFLOP/s; 24
// streaming heads (sink 64, recent 256) 0.28 ms, 460 TFLOP/s of unmasked pairs, of
// which a 128 x 128 tile holds about half. 12 prompts of 40 to 2500 rows, 16 query
// heads on retrieval KV heads 75 us; 160 prompts of up to 150 rows 21.6 us; one of 37
// rows 6.4 us, a chain of launch, plan, loads, two products and the output.
// A pair of tiles takes about 3200 cycles per 128 keys, where either pipe needs 2048.
// What is left is the chain of one tile (scores out of TMEM 300, weights 1950 with the
// other tile on the same unit half of the time, handing over, 768 of products, 130
// until the scores are seen) and the issuing warp, which cannot run ahead of the
// tensor core and stands still between two products at each of its three waits.
// Slower by 3 to 20 %: two or four threads per row in 16 softmax warps, output warps
// of their own, an issuing warp per tile (the tiles then run in step instead of in
// turn), all waits before one run of products; a polynomial for part of the
// exponentials gained 1 % at most.
#include <type_traits>

#include "item_queue.cuh"
#include "paged_internal.cuh"
#include "prefill_common.cuh"

namespace duo {

namespace {

constexpr int kPackThreads = 384;
constexpr int kSoftmaxRegs = 216;
constexpr int kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "registers of a 384-thread launch");

// A row's 64 weights against the maximum so far may add up to this much; with more, the
// maximum moves to the highest score there is, however little that is above it, and the
// tiles behind are taken in one pass again. (64 weights of 1 for a row of equal scores,
// 16 times that for scores that grow; far from what 32 bits cannot hold. A maximum that
// stayed 2^4 to 2^8 below the scores sent every later tile through the second pass:
// 16384 rows, 8 heads 696 us instead of 415.)
constexpr float kMaxHalfSum = 1024.f;

// Scores (exp2 domain) from here on lose whole units when the product with the scale is
// rounded. The weights come out of a fused product and difference, so it is the maximum
// alone that is rounded: a common factor of 2^0.5 at most below this size, but from 2^31
// on one that 32 bits do not hold. From this size on what the maximum lost is kept and
// subtracted too. (160 short prompts 21.6 us instead of 21.4, 12 ragged ones 75.0 instead
// of 74.8; a pass of their own for rows with such scores: 21.8.)
constexpr float kLargeScore = 16777216.f;  // 2^24

// One work item, as the roles read it from the queue.
struct PackItem {
    int idx;            // -1: no more
    int retr, g;        // KV head
    int head_a, head_b; // query heads
    int start, n;       // the group's first row and its rows
    int p0, p1;         // its prompts [p0, p1)
    int qa, qb;         // first query row of the tiles, in the group
    int na, nb;         // key tiles of A (a prefix of B's list when B exists) and B (0: no tile B)
    int sink_tiles, band0;  // key tile j is tile j < sink_tiles ? j : band0 + j - sink_tiles
};

__device__ __forceinline__ int key_row(const PackItem& it, int j) {
    return (j < it.sink_tiles ? j : it.band0 + j - it.sink_tiles) * kTileK;
}

// The call's prompts, in shared memory. Neighbouring prompts that fit into one tile
// of 128 rows together form a group and share its work items: a tile of thirty-row
// prompts then holds four of them, each row seeing its own prompt's keys only.
struct Prompts {
    int* row;           // [n + 1] first rows
    int* tiles_before;  // [groups + 1] query tiles of the groups before, by rank
    int* len;           // [groups] rows
    uint16_t* next;     // [n] first prompt behind the group that would start here
    uint16_t* first;    // [groups + 1] first prompt
    uint16_t* by_rank;  // [groups] longest first
    int n_groups;
    static __host__ __device__ int bytes(int n) { return (n + 1) * 8 + n * 4 + n * 2 + (n + 1) * 2 + n * 2; }
};

template <int D>
struct Layout {
    static constexpr int kColBlocks = D / 64;
    static constexpr int kTile = kColBlocks * kTileBytesPerColBlock;
    static constexpr int kQ = 0;  // tiles A and B
    static constexpr int kK = kQ + 2 * kTile;
    static constexpr int kV = kK + 2 * kTile;
    static constexpr int kBar = kV + 2 * kTile;
    static constexpr int kQueue = kBar + 48 * 8;
    static constexpr int kMisc = kQueue + 4 * static_cast<int>(sizeof(PackItem));
    static constexpr int kStage = (kMisc + 112 + 127) / 128 * 128;  // output rows, 2 KB per softmax warp
    static constexpr int kSeqs = kStage + 8 * 2048;  // the arrays of struct Prompts
    static int bytes(int n) { return kSeqs + Prompts::bytes(n); }
};
constexpr int kMaxSmem = 227 * 1024;

constexpr int kQFull = 0;
constexpr int kQEmpty = 1;
constexpr int kKFull = 2;     // + stage
constexpr int kKEmpty = 4;    // + stage
constexpr int kVFull = 6;     // + stage
constexpr int kVEmpty = 8;    // + stage
constexpr int kVRaw = 30;     // + parity: a V tile that the V warps still have to go through
constexpr int kSFull = 11;    // + tile (A, B)
constexpr int kPFull = 13;    // + 2 tile + half: P of 64 keys written (4 arrivals)
constexpr int kODone = 17;    // + tile, one phase per product PV
constexpr int kOEmpty = 19;   // + tile, O read out (4 arrivals)
constexpr int kItemFull = 21;   // + slot
constexpr int kItemEmpty = 25;  // + slot
constexpr int kDrain = 29;
constexpr int kHalfDone = 32;  // + tile, one phase per first half of a product PV
constexpr int kConsumers = 11;  // 8 softmax warps, the issuer, 2 V warps

// Whether some row of the item's tiles sees a part only of the key tile from row0.
__device__ __forceinline__ bool seen_in_part(const PackedPrefillParams& p, const PackItem& it, int row0) {
    const int last_row = (it.nb > 0 ? it.qb : it.qa) + kTileQ - 1;
    return row0 + kTileK > it.qa || (!it.retr && row0 + kTileK > p.S && row0 <= last_row - p.R);
}

// Query tiles of a prompt of `len` rows.
__device__ __forceinline__ int query_tiles(int len, int rows) { return (len + rows - 1) / rows; }

// One copy, as it is long and two places need it. Item numbers fit 32 bits: at most
// 2^23 + 512 query tiles of 256 heads.
__device__ __noinline__ PackItem pack_item(const PackedPrefillParams& p, const Prompts& pr, uint32_t idx) {
    PackItem it;
    const bool by_heads = (p.G & 1) == 0;       // tile pair = two heads of a group, or 256 rows of one
    const int rows = by_heads ? kTileQ : 2 * kTileQ;
    const uint32_t per_kv = by_heads ? p.G / 2 : p.G;
    const uint32_t of_retr = pr.tiles_before[pr.n_groups] * p.h.n_retr * per_kv;
    it.retr = idx < of_retr;
    const uint32_t units = (it.retr ? p.h.n_retr : p.h.n_strm) * per_kv;
    const uint32_t x = it.retr ? idx : idx - of_retr;
    const uint32_t tile = x / units, unit = x - tile * units;
    int lo = 0, up = pr.n_groups - 1;
    while (lo < up) {
        const int mid = (lo + up + 1) >> 1;
        if (static_cast<uint32_t>(pr.tiles_before[mid]) <= tile) lo = mid;
        else up = mid - 1;
    }
    const int qt = pr.tiles_before[lo + 1] - 1 - static_cast<int>(tile);  // the group's last tile first
    const int e = pr.by_rank[lo];
    it.idx = 0;
    it.g = p.h.head[(it.retr ? 0 : p.h.n_retr) + unit / per_kv];
    it.head_a = it.g * p.G + (by_heads ? 2 * (unit % per_kv) : unit % per_kv);
    it.head_b = by_heads ? it.head_a + 1 : it.head_a;
    it.p0 = pr.first[e];
    it.p1 = pr.first[e + 1];
    it.start = pr.row[it.p0];
    it.n = pr.len[e];
    it.qa = qt * rows;
    it.qb = by_heads ? it.qa : it.qa + kTileQ;
    const bool has_b = it.qb < it.n;
    const int last_a = it.qa / kTileQ, last_b = it.qb / kTileQ;  // diagonal key tiles
    if (it.retr) {
        it.sink_tiles = 0;
        it.band0 = 0;
    } else {
        int a = (p.S + kTileK - 1) / kTileK;
        if (a > last_a) a = last_a;  // the band covers the rest
        const int low = it.qa - p.R + 1;
        const int tb = low > 0 ? low / kTileK : 0;
        it.sink_tiles = a < tb ? a : tb;
        it.band0 = tb;
    }
    it.na = it.sink_tiles + last_a - it.band0 + 1;
    it.nb = has_b ? it.sink_tiles + last_b - it.band0 + 1 : 0;
    return it;
}

__device__ __forceinline__ void give_up(uint32_t* err, volatile int* abort_flag) {
    *abort_flag = 1;
    atomicOr(err, kErrPagedWait);
}

// 1 in one lane of the warp, the same in every call.
__device__ __forceinline__ uint32_t elect_lane() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}
// Several products in one piece of assembly, issued by one lane: the issuing warp has 64
// cycles per product. Descriptors advance by the operand's bytes / 16.
//
// D[tmem] = A[smem] * B[smem]^T over four steps of 16 (one 64-column block).
__device__ __forceinline__ void tc_mma_ss4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %3, q;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem] over four steps of 16 (64 rows of V).
__device__ __forceinline__ void tc_mma_ts4(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b64 b1, b2, b3;\n\t.reg .b32 a1, a2, a3;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.eq.b32 q, 0, 0;\n\t"
        "add.s32 a1, %1, 8;\n\tadd.s32 a2, %1, 16;\n\tadd.s32 a3, %1, 24;\n\t"
        "add.s64 b1, %2, 128;\n\tadd.s64 b2, %2, 256;\n\tadd.s64 b3, %2, 384;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b1, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b2, %3, q;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b3, %3, q;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// An arrival without a branch around it, which would end the block that the compiler
// schedules.
__device__ __forceinline__ void mbar_arrive_if(bool yes, uint32_t bar) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(bar),
                 "r"(static_cast<uint32_t>(yes))
                 : "memory");
}

template <int N>
__device__ __forceinline__ void regs_inc() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The keys that a row of the item sees.
struct RowKeys {
    RowVis vis;
    int own0;  // first row of the row's prompt, in the group
    __device__ __forceinline__ uint32_t bits(int k0) const { return chunk_bits_row(vis, k0) & ~bits_below32(own0 - k0); }
};
__device__ __forceinline__ RowKeys row_keys(const PackedPrefillParams& p, const PackItem& it, const int* first_row, int q) {
    RowKeys r;
    r.vis = row_visible(it.retr, 0, it.n, p.S, p.R, q);
    r.own0 = 0;
    if (it.p1 - it.p0 > 1) {
        int lo = it.p0, up = it.p1 - 1;
        while (lo < up) {
            const int mid = (lo + up + 1) >> 1;
            if (first_row[mid] <= it.start + q) lo = mid;
            else up = mid - 1;
        }
        __syncwarp();
        r.own0 = first_row[lo] - it.start;
        r.vis.c_sink = it.retr ? 0 : r.own0 + p.S;
    }
    return r;
}

// Adds to 16 columns of a row, from `col`, the infinities and NaN of the value rows
// that it sees among the tiles that were cleared of them: a visible row has a
// positive weight, so the sum is that value whatever the weight is.
template <typename Seen>
__device__ __forceinline__ void add_odd_values(const PackedPrefillParams& p, const PackItem& it, int n, int col, Seen seen,
                                               uint32_t (&r)[16]) {
    const bf16* const v = p.v + static_cast<int64_t>(it.start) * p.kv_stride + it.g * p.D + col;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int row0 = key_row(it, j);
        if (!seen_in_part(p, it, row0)) continue;
#pragma unroll 1
        for (int k0 = row0; k0 < row0 + kTileK && k0 < it.n; k0 += 32)
#pragma unroll 1
            for (uint32_t bits = seen(k0); bits; bits &= bits - 1) {
                const bf16* const row = v + (k0 + __ffs(bits) - 1) * p.kv_stride;  // seen keys are rows of the group
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float x = __bfloat162float(row[i]);
                    if (!isfinite(x)) r[i] = __float_as_uint(__uint_as_float(r[i]) + x);
                }
            }
    }
}

// Groups of neighbouring prompts, their ranks by length and the query tiles before
// each. The whole CTA; `scratch`: 16 KB that nobody uses yet.
__device__ __forceinline__ void group_prompts(const PackedPrefillParams& p, Prompts& pr, const uint32_t* wrong,
                                              volatile int* n_groups, uint8_t* scratch, int rows_per_tile) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
#pragma unroll 1
    for (int i = tid; i < p.n; i += kPackThreads) {
        // The first unusable prompt at i or behind; up to there the rows ascend.
        int stop = p.n;
#pragma unroll 1
        for (int w = i >> 5; w <= (p.n - 1) >> 5; ++w) {
            const uint32_t bits = w == i >> 5 ? wrong[w] & (0xFFFFFFFFu << (i & 31)) : wrong[w];
            if (bits) {
                stop = w * 32 + __ffs(bits) - 1;
                break;
            }
        }
        // The last j with all of [i, j) in one tile.
        int lo = i < stop ? i : stop, up = stop;
        while (lo < up) {
            const int mid = (lo + up + 1) >> 1;
            if (pr.row[mid] - pr.row[i] <= kTileQ) lo = mid;
            else up = mid - 1;
        }
        pr.next[i] = static_cast<uint16_t>(lo > i ? lo : i + 1);
    }
    __syncthreads();
    // The groups are what following `next` from prompt 0 meets. One thread takes jumps
    // of eight groups, then each place that it met is followed for eight groups by a
    // thread of its own: a chain of up to 512 reads becomes one of 64.
    const int n1 = p.n + 1;
    uint16_t* const jump[2] = {reinterpret_cast<uint16_t*>(scratch), reinterpret_cast<uint16_t*>(scratch) + n1};
    uint16_t* const met = jump[1] + n1;  // [65]
    volatile int* const n_met = reinterpret_cast<volatile int*>(scratch + 8 * 1024);
    volatile int* const n_long = n_met + 1;
    uint32_t* const is_long = reinterpret_cast<uint32_t*>(scratch + 8 * 1024 + 64);   // a bit per group
    uint32_t* const is_short = is_long + kPagedMaxBatch / 32;
#pragma unroll 1
    for (int i = tid; i <= p.n; i += kPackThreads) {  // two groups on
        const int k = i < p.n ? pr.next[i] : p.n;
        jump[0][i] = k < p.n ? pr.next[k] : static_cast<uint16_t>(p.n);
    }
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i <= p.n; i += kPackThreads) jump[1][i] = jump[0][jump[0][i]];
    __syncthreads();
#pragma unroll 1
    for (int i = tid; i <= p.n; i += kPackThreads) jump[0][i] = jump[1][jump[1][i]];
    __syncthreads();
    if (tid == 0) {
        int m = 0;
#pragma unroll 1
        for (int i = 0; i < p.n; i = jump[0][i]) met[m++] = static_cast<uint16_t>(i);
        *n_met = m;
    }
    __syncthreads();
    if (tid < *n_met) {
        int g = tid * 8, i = met[tid];
#pragma unroll 1
        for (int k = 0; k < 8 && i < p.n; ++k, ++g) {
            pr.first[g] = static_cast<uint16_t>(i);
            i = pr.next[i];
        }
        if (i >= p.n) {  // the last of them
            pr.first[g] = static_cast<uint16_t>(p.n);
            *n_groups = g;
        }
    }
    __syncthreads();
    pr.n_groups = *n_groups;
    // Groups of more than one tile come first, longest first; those of one tile and empty
    // ones follow in order.
#pragma unroll 1
    for (int i0 = 0; i0 < pr.n_groups; i0 += kPackThreads) {
        const int i = i0 + tid;
        int len = 0;
        if (i < pr.n_groups) {
            const int f = pr.first[i];
            len = (wrong[f >> 5] >> (f & 31)) & 1u ? 0 : pr.row[pr.first[i + 1]] - pr.row[f];
            pr.len[i] = len;
        }
        const uint32_t l = __ballot_sync(0xffffffffu, len > kTileQ), s = __ballot_sync(0xffffffffu, len > 0 && len <= kTileQ);
        if (lane == 0 && i / 32 < kPagedMaxBatch / 32) {
            is_long[i / 32] = l;
            is_short[i / 32] = s;
        }
    }
    __syncthreads();
    int longs = 0, shorts = 0;
#pragma unroll 1
    for (int w = 0; w <= (pr.n_groups - 1) >> 5; ++w) {
        longs += __popc(is_long[w]);
        shorts += __popc(is_short[w]);
    }
#pragma unroll 1
    for (int i = tid; i < pr.n_groups; i += kPackThreads) {
        const uint32_t below = (1u << (i & 31)) - 1u;
        int long_before = __popc(is_long[i >> 5] & below), short_before = __popc(is_short[i >> 5] & below);
#pragma unroll 1
        for (int w = 0; w < i >> 5; ++w) {
            long_before += __popc(is_long[w]);
            short_before += __popc(is_short[w]);
        }
        if ((is_long[i >> 5] >> (i & 31)) & 1u) jump[0][long_before] = static_cast<uint16_t>(i);  // the list of long ones
        else if ((is_short[i >> 5] >> (i & 31)) & 1u) pr.by_rank[longs + short_before] = static_cast<uint16_t>(i);
        else pr.by_rank[longs + shorts + (i - long_before - short_before)] = static_cast<uint16_t>(i);
    }
    __syncthreads();
#pragma unroll 1
    for (int k = tid; k < longs; k += kPackThreads) {
        const int len = pr.len[jump[0][k]];
        int rank = 0;
#pragma unroll 4
        for (int j = 0; j < longs; ++j) {
            const int other = pr.len[jump[0][j]];
            rank += other > len || (other == len && j < k);
        }
        pr.by_rank[rank] = jump[0][k];
    }
    __syncthreads();
    if (warp == 0) {
        int sum = 0;
#pragma unroll 1
        for (int i0 = 0; i0 < longs; i0 += 32) {
            const int i = i0 + lane;
            const int own = i < longs ? query_tiles(pr.len[pr.by_rank[i]], rows_per_tile) : 0;
            int t = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, t, o);
                t += lane >= o ? a : 0;
            }
            if (i < longs) pr.tiles_before[i] = sum + t - own;
            sum += __shfl_sync(0xffffffffu, t, 31);
        }
        if (lane == 0) *n_long = sum;  // tiles of the long groups
    }
    __syncthreads();
#pragma unroll 1
    for (int r = longs + tid; r <= pr.n_groups; r += kPackThreads)
        pr.tiles_before[r] = *n_long + min(r - longs, shorts);
}

template <int D>
__global__ void __launch_bounds__(kPackThreads, 1)
    prefill_packed_kernel(const __grid_constant__ PackedPrefillParams p, const __grid_constant__ PackedMaps maps) {
    using Lay = Layout<D>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const uint32_t base = smem_u32(smem);
    const uint32_t sQ = base + Lay::kQ, sK = base + Lay::kK, sV = base + Lay::kV;
    auto bar = [&](int i) { return base + Lay::kBar + 8u * i; };
    PackItem* queue = reinterpret_cast<PackItem*>(smem + Lay::kQueue);
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem + Lay::kMisc);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Lay::kMisc + 4);
    // Marks (item_queue.cuh): a V tile that some rows of the item see in part held an
    // infinity or NaN.
    volatile int* const marked_odd = reinterpret_cast<volatile int*>(smem + Lay::kMisc + 80);
    static_assert(80 + kItemMarks * 4 <= 112, "the marks end where the output rows begin");
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        mbar_init(bar(kQFull), 1);
        mbar_init(bar(kQEmpty), 1);
        mbar_init(bar(kDrain), 1);
        for (int s = 0; s < 2; ++s) {
            mbar_init(bar(kKFull + s), 1);
            mbar_init(bar(kKEmpty + s), 1);
            mbar_init(bar(kVFull + s), 2);
            mbar_init(bar(kVRaw + s), 1);
            mbar_init(bar(kVEmpty + s), 1);
            mbar_init(bar(kSFull + s), 1);
            mbar_init(bar(kODone + s), 1);
            mbar_init(bar(kHalfDone + s), 1);
            mbar_init(bar(kOEmpty + s), 4);
            mbar_init(bar(kPFull + 2 * s), 4);
            mbar_init(bar(kPFull + 2 * s + 1), 4);
        }
        for (int s = 0; s < kQueueSlots; ++s) {
            mbar_init(bar(kItemFull + s), 1);
            mbar_init(bar(kItemEmpty + s), kConsumers);
        }
        *abort_flag = 0;
        for (int i = 0; i < kItemMarks; ++i) marked_odd[i] = kNoItem;
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 9) {
        tmem_alloc(base + Lay::kMisc, kTmemCols);
        tmem_relinquish();
    }
    Prompts pr;
    pr.row = reinterpret_cast<int*>(smem + Lay::kSeqs);
    pr.tiles_before = pr.row + p.n + 1;
    pr.len = pr.tiles_before + p.n + 1;
    pr.next = reinterpret_cast<uint16_t*>(pr.len + p.n);
    pr.first = pr.next + p.n;
    pr.by_rank = pr.first + p.n + 1;
    uint32_t* const wrong = reinterpret_cast<uint32_t*>(smem + Lay::kMisc + 16);  // one bit per prompt: range not usable
    volatile int* const n_groups = reinterpret_cast<volatile int*>(smem + Lay::kMisc + 8);
    static_assert(kPagedMaxBatch <= 512, "16 words of bits");
    grid_dependency_wait();
    grid_launch_dependents();
#pragma unroll 1
    for (int i0 = 0; i0 <= p.n; i0 += kPackThreads) {
        const int i = i0 + tid;
        bool bad = false;
        if (i <= p.n) {
            const int r = p.row_start[i];
            pr.row[i] = r;
            if (i < p.n) {
                const int end = p.row_start[i + 1];
                bad = r < 0 || end < r || end > p.n_rows;
            }
        }
        const uint32_t bits = __ballot_sync(0xffffffffu, bad);
        if (lane == 0 && i / 32 < kPagedMaxBatch / 32) wrong[i / 32] = bits;
        if (bits != 0 && lane == 0 && blockIdx.x == 0) atomicOr(p.err, kErrPagedArgument);
    }
    __syncthreads();
    const int rows_per_tile = (p.G & 1) ? 2 * kTileQ : kTileQ;
    if (p.n == 1) {  // one prompt: none of the below
        pr.n_groups = 1;
        if (tid == 0) {
            pr.len[0] = (wrong[0] & 1u) ? 0 : pr.row[1] - pr.row[0];
            pr.first[0] = 0;
            pr.first[1] = 1;
            pr.by_rank[0] = 0;
            pr.tiles_before[0] = 0;
            pr.tiles_before[1] = query_tiles(pr.len[0], rows_per_tile);
        }
    } else {
        group_prompts(p, pr, wrong, n_groups, smem + Lay::kStage, rows_per_tile);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t n_items =
        static_cast<uint32_t>(pr.tiles_before[pr.n_groups]) * (p.h.n_retr + p.h.n_strm) * ((p.G & 1) ? p.G : p.G / 2);

    // Item number `ord` of this CTA; false: none left, or a wait ran out.
    auto take_item = [&](int ord, PackItem& it) -> bool {
        const int slot = ord % kQueueSlots;
        if (!mbar_wait(bar(kItemFull + slot), (ord / kQueueSlots) & 1, abort_flag)) {
            give_up(p.err, abort_flag);
            return false;
        }
        it = queue[slot];
        return it.idx >= 0;
    };
    auto free_item = [&](int ord) { mbar_arrive(bar(kItemEmpty + ord % kQueueSlots)); };

    if (warp >= 8) {
        regs_dec<kOtherRegs>();
        if (warp == 8 && lane == 0) {
            // -------------------------------------------------------- items, Q and K
            // The next item is taken and published behind the loads of this one's first key
            // tile: nobody waits for the counter then, the first loads least of all.
            tma_prefetch_desc(&maps.q);
            int published = 0;
            auto publish = [&](PackItem& it) -> bool {
                // The first item is the CTA's own number; the counter hands out the ones behind.
                const uint32_t i = published == 0 ? blockIdx.x
                                   : *abort_flag == 0 ? gridDim.x + atomicAdd(p.work, 1u) : 0xFFFFFFFFu;
                it.idx = -1;
                if (i < n_items) it = pack_item(p, pr, i);
                const int slot = published % kQueueSlots;
                if (published >= kQueueSlots &&
                    !mbar_wait_compact(bar(kItemEmpty + slot), ((published / kQueueSlots) - 1) & 1, abort_flag))
                    return false;
                queue[slot] = it;
                mbar_arrive(bar(kItemFull + slot));
                ++published;
                return true;
            };
            int g = 0;                // K and V tiles of the items before
            int q_loads = 0, k_loads = 0;
            int raw0 = 0, raw1 = 0;   // V tiles that the V warps go through, by stage
            PackItem it, after;
            bool ok = publish(it);
            while (ok && it.idx >= 0) {
                if (q_loads >= 1) ok = mbar_wait_compact(bar(kQEmpty), (q_loads - 1) & 1, abort_flag);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(kQFull), (it.nb > 0 ? 2 : 1) * Lay::kTile);
#pragma unroll 1
                for (int kb = 0; kb < Lay::kColBlocks; ++kb) {
                    tma_load_3d(sQ + kb * kTileBytesPerColBlock, &maps.q, bar(kQFull), kb * 64, it.head_a, it.start + it.qa);
                    if (it.nb > 0)
                        tma_load_3d(sQ + Lay::kTile + kb * kTileBytesPerColBlock, &maps.q, bar(kQFull), kb * 64, it.head_b,
                                    it.start + it.qb);
                }
                ++q_loads;
                if (p.test_withhold != 0 && blockIdx.x == 0) {  // a test of the waits for the tiles: none is loaded
                    mbar_wait(bar(kKEmpty), 0, abort_flag, 2 * kWaitTimeoutNs);
                    ok = false;
                    break;
                }
                // K and V tiles in turn: by the time a K stage is free the V stage before it is.
                const int n = it.na > it.nb ? it.na : it.nb;
#pragma unroll 1
                for (int j = 0; ok && j < n; ++j, ++g) {
                    const int st = g & 1;
                    const int row0 = key_row(it, j);
                    if (g >= 2) ok = mbar_wait_compact(bar(kKEmpty + st), ((g >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                    mbar_arrive_expect_tx(bar(kKFull + st), Lay::kTile);
#pragma unroll 1
                    for (int kb = 0; kb < Lay::kColBlocks; ++kb)
                        tma_load_3d(sK + st * Lay::kTile + kb * kTileBytesPerColBlock, &maps.k, bar(kKFull + st), kb * 64,
                                    it.g, it.start + row0);
                    ++k_loads;
                    if (g >= 2) ok = mbar_wait_compact(bar(kVEmpty + st), ((g >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                    const bool part = seen_in_part(p, it, row0);
                    const uint32_t full = bar((part ? kVRaw : kVFull) + st);
                    mbar_arrive_expect_tx(full, Lay::kTile);
#pragma unroll 1
                    for (int kb = 0; kb < Lay::kColBlocks; ++kb)
                        tma_load_3d(sV + st * Lay::kTile + kb * kTileBytesPerColBlock, &maps.v, full, kb * 64, it.g,
                                    it.start + row0);
                    if (part) ++(st ? raw1 : raw0);
                    else mbar_arrive(full);  // for the second of the V warps
                    if (j == 0) ok = publish(after);
                }
                it = after;
            }
            if (!ok) give_up(p.err, abort_flag);
            // Every load issued lands before the CTA may exit.
            for (int j = k_loads > 2 ? k_loads - 2 : 0; j < k_loads; ++j) mbar_wait_compact(bar(kKFull + (j & 1)), (j >> 1) & 1, nullptr);
            for (int st = 0; st < 2; ++st) {
                const int raw = st ? raw1 : raw0;
                if (raw > 0) mbar_wait_compact(bar(kVRaw + st), (raw - 1) & 1, nullptr);
            }
            for (int j = g > 2 ? g - 2 : 0; j < g; ++j) mbar_wait_compact(bar(kVFull + (j & 1)), (j >> 1) & 1, abort_flag);
            if (q_loads > 0) mbar_wait_compact(bar(kQFull), (q_loads - 1) & 1, nullptr);
        } else if (warp >= 10) {
            // -------------------------------------------------------- V tiles seen in part
            // A V tile that some row of the item sees only in part (the diagonal, the window's
            // edges, a group of prompts) is gone through by both warps, 64 rows each, before
            // the products may read it: a weight of zero must not meet an infinity or a NaN.
            // Rows behind the group's end, which belong to other prompts or to nobody, become
            // zero; a non-finite element becomes zero too and is counted for the rows that
            // see it at the item's end.
            const int half = warp - 10;
            int g = 0;
            int raw0 = 0, raw1 = 0;  // such tiles so far, by stage
            bool ok = true;
            for (int ord = 0; ok; ++ord) {
                PackItem it;
                const bool more = take_item(ord, it);
                __syncwarp();
                if (lane == 0) free_item(ord);
                if (!__all_sync(0xffffffffu, more)) break;
                const int n = it.na > it.nb ? it.na : it.nb;
                for (int j = 0; j < n; ++j, ++g) {
                    const int st = g & 1;
                    const int row0 = key_row(it, j);
                    if (!seen_in_part(p, it, row0)) continue;
                    const int turn = st ? raw1++ : raw0++;
                    ok = __all_sync(0xffffffffu, mbar_wait_compact(bar(kVRaw + st), turn & 1, abort_flag));
                    if (!ok) break;
                    const int valid = it.n - row0;
                    bool odd = false;
#pragma unroll 1
                    for (int kb = 0; kb < Lay::kColBlocks; ++kb) {
                        const uint32_t tile = sV + st * Lay::kTile + kb * kTileBytesPerColBlock + half * (64 * 128);
                        // 0 x w summed up: NaN in the end if any w was not finite.
                        __nv_bfloat162 sum[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) sum[i] = __floats2bfloat162_rn(0.f, 0.f);
                        const __nv_bfloat162 zero = sum[0];
#pragma unroll 4
                        for (int i = 0; i < 64 * 8 / 32; ++i) {
                            const int row = half * 64 + i * 4 + (lane >> 3);
                            const uint32_t a = tile + (i * 32 + lane) * 16;
                            uint4 w = lds128(a);
                            if (row >= valid) {
                                w = make_uint4(0, 0, 0, 0);
                                asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0u) : "memory");
                            }
                            const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                sum[k] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&words[k]), zero, sum[k]);
                        }
                        sum[0] = __hadd2(__hadd2(sum[0], sum[1]), __hadd2(sum[2], sum[3]));
                        const float check = __low2float(sum[0]) + __high2float(sum[0]);
                        if (__any_sync(0xffffffffu, !(check == 0.f))) {
                            odd = true;
#pragma unroll 1
                            for (int i = lane; i < 64 * 32; i += 32) {
                                uint32_t w;
                                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(tile + i * 4));
                                if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
                                if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
                                asm volatile("st.shared.u32 [%0], %1;" ::"r"(tile + i * 4), "r"(w) : "memory");
                            }
                            __syncwarp();
                        }
                    }
                    if (odd && lane == 0) marked_odd[mark_place(ord)] = ord;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kVFull + st));
                }
            }
            if (!ok && lane == 0) give_up(p.err, abort_flag);
        } else if (warp == 9) {
            // -------------------------------------------------------- products
            // The whole warp walks the loop and one elected lane issues: control flow and
            // descriptors stay uniform over the warp. One lane on its own took 4100 cycles
            // per pair of tiles to issue what the tensor core computes in 2048.
            constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTileK, 0, 0);
            constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 0, 1);
            const uint32_t lead = elect_lane();
            const uint64_t dq = smem_desc_sw128(sQ, 16, 1024), dk = smem_desc_sw128(sK, 16, 1024);
            const uint64_t dv = smem_desc_sw128(sV, kTileBytesPerColBlock, 1024);
            int g = -1;              // key tile that the item starts with; the first is 0
            int count_a = 0, count_b = 0;  // products PV of each tile so far
            int items_a = 0, items_b = 0;  // items that had the tile so far
            bool ok = true;
            // S(x) = Q(x) K(t)^T for the CTA's key tile t; `last`: the last product to read it,
            // `last_q`: and the last to read Q.
            auto qk = [&](auto x_, int t, bool wait, bool last, bool last_q) {
                constexpr int x = decltype(x_)::value;
                const int st = t & 1;
                if (wait && !__all_sync(0xffffffffu, mbar_wait_compact(bar(kKFull + st), (t >> 1) & 1, abort_flag))) return false;
                tc_fence_after();
                const uint64_t q = dq + x * (Lay::kTile >> 4), k = dk + st * (Lay::kTile >> 4);
                if (lead) {
#pragma unroll
                    for (int kb = 0; kb < D / 64; ++kb)
                        tc_mma_ss4(tmem + x * kTileK, q + kb * (kTileBytesPerColBlock >> 4),
                                   k + kb * (kTileBytesPerColBlock >> 4), idesc_qk, kb);
                    tc_commit(bar(kSFull + x));
                    if (last) tc_commit(bar(kKEmpty + st));
                    if (last && last_q) tc_commit(bar(kQEmpty));
                }
                __syncwarp();
                return true;
            };
            // O(x) += P(x) V(t); `first`: of the item.
            auto pv = [&](auto x_, int t, bool wait, bool last, bool first, int count, int items) {
                constexpr int x = decltype(x_)::value;
                const int st = t & 1;
                if (wait && !__all_sync(0xffffffffu, mbar_wait_compact(bar(kVFull + st), (t >> 1) & 1, abort_flag))) return false;
                if (first && items > 0 &&
                    !__all_sync(0xffffffffu, mbar_wait_compact(bar(kOEmpty + x), (items - 1) & 1, abort_flag)))
                    return false;
                const uint64_t vt = dv + st * (Lay::kTile >> 4);
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!__all_sync(0xffffffffu, mbar_wait_compact(bar(kPFull + 2 * x + half), count & 1, abort_flag))) return false;
                    tc_fence_after();
                    if (lead) {
                        tc_mma_ts4(tmem + kTmemO + x * 128, tmem + x * kTileK + half * 32, vt + half * 4 * (2048 >> 4), idesc_pv,
                                   first && half == 0 ? 0u : 1u);
                        if (half == 0) tc_commit(bar(kHalfDone + x));
                        if (half == 1) tc_commit(bar(kODone + x));
                        if (half == 1 && last) tc_commit(bar(kVEmpty + st));
                    }
                    __syncwarp();
                }
                return true;
            };
            constexpr std::integral_constant<int, 0> A{};
            constexpr std::integral_constant<int, 1> B{};
            int ord = 0, na = 0, nb = 0;
            // The next item's tile counts (0: none left), its queries waited for.
            auto next_item = [&](int& a, int& b) {
                PackItem it;
                const bool more = take_item(ord, it);
                __syncwarp();
                if (lead) free_item(ord);
                a = b = 0;
                if (!__all_sync(0xffffffffu, more)) return;
                a = __shfl_sync(0xffffffffu, it.na, 0);
                b = __shfl_sync(0xffffffffu, it.nb, 0);
                ok = __all_sync(0xffffffffu, mbar_wait_compact(bar(kQFull), ord & 1, abort_flag));
                ++ord;
            };
            // Per key tile PV(A), QK(A) of the next tile, PV(B), QK(B): the next tile behind an
            // item's last is the next item's first, so that its scores are there when the
            // softmax has written the item's rows. Every QK of the item is issued by then, and
            // its queries have been replaced. A's list is B's without its last tile, or as
            // long; there may be no B. Before the first item: one tile of nothing.
            int n = 1;
            while (ok && n > 0) {
                int next_a = na, next_b = nb, next_n = n;
#pragma unroll 1
                for (int j = 0; ok && j < n; ++j) {
                    const int t = g + j;
                    const bool turn = j + 1 == n;  // the next tile is the next item's
                    if (j < na) ok = pv(A, t, true, j >= nb, j == 0, count_a++, items_a);
                    if (ok && turn) {
                        next_item(next_a, next_b);
                        next_n = next_a > next_b ? next_a : next_b;
                    }
                    const int k = turn ? 0 : j + 1;  // the next tile's number in its item
                    if (ok && k < next_a && (turn || k < na)) ok = qk(A, t + 1, true, k >= next_b, k + 1 == next_n);
                    if (ok && j < nb) ok = pv(B, t, j >= na, true, j == 0, count_b++, items_b);
                    if (ok && k < next_b && (turn || k < nb)) ok = qk(B, t + 1, k >= next_a, true, k + 1 == next_n);
                }
                items_a += na > 0;
                items_b += nb > 0;
                g += n;
                na = next_a;
                nb = next_b;
                n = next_n;
            }
            if (!ok && lead) give_up(p.err, abort_flag);
            if (lead) tc_commit(bar(kDrain));  // every product issued has completed before TMEM is released
            mbar_wait_compact(bar(kDrain), 0, nullptr);
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------ softmax
        regs_inc<kSoftmaxRegs>();
        const int x = warp >> 2;  // tile
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        const uint32_t tS = tmem + lane_base + x * kTileK;
        const uint32_t tO = tmem + lane_base + kTmemO + x * 128;
        const uint64_t scale2 = f2pack(p.scale_log2, p.scale_log2);
        int count = 0;  // key tiles so far
        bool ok = true;
        for (int ord = 0; ok; ++ord) {
            PackItem it;
            const bool more = take_item(ord, it);
            __syncwarp();
            if (lane == 0) free_item(ord);
            if (!__all_sync(0xffffffffu, more)) break;
            const int n = x ? it.nb : it.na;
            if (n == 0) continue;
            const int q0 = x ? it.qb : it.qa;
            const int head = x ? it.head_b : it.head_a;
            const bool single = it.p1 - it.p0 == 1;
            const RowKeys keys = row_keys(p, it, pr.row, q0 + row);
            auto seen_bits = [&](int k0) { return keys.bits(k0); };
            // The first key tiles, which all rows of the warp see whole (a streaming item's few
            // tiles are looked at one by one).
            const int whole_tiles = single && it.retr ? (q0 + quarter * 32 + 1) / kTileK : 0;
            float m_run = -INFINITY, l_run = 0.f;
            float m_low = 0.f;     // the exact maximum minus m_run where that is large, else 0
            bool settled = false;  // every row of the warp has a maximum, and none a large one
            for (int j = 0; j < n; ++j, ++count) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar(kSFull + x), count & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int row0 = key_row(it, j);
                // The tile in four runs of 32 keys: what the warp's 32 rows [r0, r0 + 31] see
                // of each is all of it, nothing, or a part: one bit per run, the same for the
                // whole warp. Only parts are masked element by element; a run that no row sees
                // costs nothing but a zero P.
                uint32_t none = 0u, all = 15u;
                if (j >= whole_tiles) {
                    auto below = [](int x) { return (1u << (x < 0 ? 0 : x > 4 ? 4 : x)) - 1u; };
                    const int d = (q0 + quarter * 32 - row0) >> 5;  // the diagonal's run
                    none = ~below(d + 1);
                    all = single ? below(d) : 0u;
                    if (single && !it.retr) {
                        const int e = q0 + quarter * 32 - p.R - row0;  // keys <= e are outside all rows' windows,
                        const int sk = p.S - row0;                     // keys > e + 31 inside all; keys < sk are sinks
                        all &= ~below(((e + 31) >> 5) + 1) | below(sk >> 5);
                        none |= below((e + 1) >> 5) & ~below((sk + 31) >> 5);
                    }
                    all = __shfl_sync(0xffffffffu, all, 0);
                    none = __shfl_sync(0xffffffffu, none, 0);
                }
                // Two versions of what follows.
                //
                // A tile seen whole, once every row of the warp has a maximum, is taken at that
                // maximum at once, in halves of 64 keys, unrolled: a half's sum of weights shows
                // whether a score outgrew it. Looking for the maximum first took a quarter of
                // the time from the scores to their weights, a chain that the other tile's work
                // does not hide.
                //
                // Any other tile, and a half whose sum is too large (or NaN), is handled run by
                // run, each run read from TMEM twice (for the maximum, for the weights), in a
                // quarter of the code: the roles' loops have to fit the instruction cache
                // together. Weights go over S columns that have been read (run c's over 16 c ..)
                // and only when no second look at S can be needed.
                auto exps_of = [&](uint32_t (&run)[32], uint64_t negm, auto two_parts, uint64_t neglow) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float e0, e1;
                        uint64_t e = ffma2(f2pack(__uint_as_float(run[i]), __uint_as_float(run[i + 1])), scale2, negm);
                        if (decltype(two_parts)::value) e = fadd2(e, neglow);
                        f2unpack(e, e0, e1);
                        run[i] = __float_as_uint(fast_exp2(e0));
                        run[i + 1] = __float_as_uint(fast_exp2(e1));
                    }
                };
                auto pack_weights = [&](const uint32_t (&run)[32], uint32_t (&pk)[16], uint64_t (&acc)[2]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        const float p0 = __uint_as_float(run[i]), p1 = __uint_as_float(run[i + 1]);
                        acc[(i >> 1) & 1] = fadd2(acc[(i >> 1) & 1], f2pack(p0, p1));
                        pk[i >> 1] = pack_bf16x2(p0, p1);
                    }
                };
                auto sum_of = [&](const uint64_t (&acc)[2]) {
                    float a0, a1;
                    f2unpack(fadd2(acc[0], acc[1]), a0, a1);
                    return a0 + a1;
                };
                auto hand_over = [&](int half) {  // 64 keys' weights are written
                    tc_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    mbar_arrive_if(lane == 0, bar(kPFull + 2 * x + half));
                };
                int c_slow = 0;  // runs from here on are handled one by one
                const bool outgrown = all == 15u && settled;  // (if any are) by a half's sum
                if (outgrown) {
                    uint32_t s[4][32], pk[2][16];
                    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
                    const uint64_t negm = f2pack(-m_run, -m_run);
                    tmem_ld32(tS, s[0]);
                    tmem_ld32(tS + 32, s[1]);
                    tc_wait_ld();
                    tmem_ld32(tS + 64, s[2]);
                    tmem_ld32(tS + 96, s[3]);
                    // The exponentials of a run are on their way while the run before is summed
                    // and packed: with both in one loop a warp on its own took 455 cycles per
                    // run, of which its exponentials need 256.
                    exps_of(s[0], negm, std::false_type{}, 0);
                    exps_of(s[1], negm, std::false_type{}, 0);
                    pack_weights(s[0], pk[0], acc);
                    tc_wait_ld();
                    exps_of(s[2], negm, std::false_type{}, 0);
                    pack_weights(s[1], pk[1], acc);
                    float sum = sum_of(acc);
                    if (__all_sync(0xffffffffu, sum <= kMaxHalfSum)) {
                        tmem_st16(tS, pk[0]);
                        tmem_st16(tS + 16, pk[1]);
                        l_run += sum;
                        acc[0] = acc[1] = f2pack(0.f, 0.f);
                        exps_of(s[3], negm, std::false_type{}, 0);
                        hand_over(0);
                        pack_weights(s[2], pk[0], acc);
                        pack_weights(s[3], pk[1], acc);
                        sum = sum_of(acc);
                        c_slow = 2;
                        if (__all_sync(0xffffffffu, sum <= kMaxHalfSum)) {
                            tmem_st16(tS + 32, pk[0]);
                            tmem_st16(tS + 48, pk[1]);
                            l_run += sum;
                            hand_over(1);
                            c_slow = 4;
                        }
                    }
                }
                if (c_slow < 4) {
                    float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
                    for (int c = c_slow; c < 4; ++c) {
                        if ((none >> c) & 1u) continue;
                        uint32_t run[32];
                        tmem_ld32(tS + c * 32, run);
                        tc_wait_ld();
                        if (!((all >> c) & 1u)) {
                            const uint32_t bits = seen_bits(row0 + 32 * c);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((bits >> k) & 1u)) run[k] = 0xFF800000u;  // -inf
                            tmem_st32(tS + c * 32, run);  // for the second pass
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], __uint_as_float(run[i]), __uint_as_float(run[i + 1]));
                    }
                    tc_wait_st();
                    const float top = fmax3(fmaxf(m[0], m[1]), m[2], m[3]);
                    const float mt = top * p.scale_log2;
                    const bool large = fabsf(mt) >= kLargeScore && fabsf(mt) < INFINITY;
                    const float low = large ? fmaf(top, p.scale_log2, -mt) : 0.f;
                    const float gain = (mt - m_run) + (low - m_low);  // (NaN where both are the same infinity)
                    const float least = outgrown ? 0.f : kRescaleThreshold;
                    if (__any_sync(0xffffffffu, gain > least)) {
                        float factor = 1.f;
                        if (gain > least) {
                            factor = fast_exp2(-gain);
                            m_run = mt;
                            m_low = low;
                        }
                        l_run *= factor;
                        settled = __all_sync(0xffffffffu, m_run > -INFINITY && fabsf(m_run) < kLargeScore);
                        if (j >= 1) {
                            // The last product that wrote O: PV(j-1), or PV(j) of the half before.
                            const bool ready = c_slow == 0 ? mbar_wait(bar(kODone + x), (count - 1) & 1, abort_flag)
                                                           : mbar_wait(bar(kHalfDone + x), count & 1, abort_flag);
                            if (!__all_sync(0xffffffffu, ready)) {
                                ok = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 16; ++c) {
                                uint32_t r[16];
                                tmem_ld16(tO + c * 16, r);
                                tc_wait_ld();
#pragma unroll
                                for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * factor);
                                tmem_st16(tO + c * 16, r);
                            }
                        }
                    }
                    const float m_use = m_run == -INFINITY ? 0.f : m_run;
                    const uint64_t negm = f2pack(-m_use, -m_use), neglow = f2pack(-m_low, -m_low);
                    uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
#pragma unroll 1
                    for (int c = c_slow; c < 4; ++c) {
                        uint32_t pk[16];
                        if ((none >> c) & 1u) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        } else {
                            uint32_t run[32];
                            tmem_ld32(tS + c * 32, run);
                            tc_wait_ld();
                            exps_of(run, negm, std::true_type{}, neglow);
                            pack_weights(run, pk, acc);
                        }
                        tmem_st16(tS + c * 16, pk);
                        if (c & 1) hand_over(c >> 1);
                    }
                    l_run += sum_of(acc);
                }
            }
            if (!ok) break;
            if (!__all_sync(0xffffffffu, mbar_wait(bar(kODone + x), (count - 1) & 1, abort_flag))) {
                ok = false;
                break;
            }
            tc_fence_after();
            const float inv = 1.f / l_run;
            // 32 columns at a time through 2 KB of the warp's own shared memory: a thread
            // has a whole row, and rows written straight from registers would cost 32
            // memory transactions per instruction instead of 8.
            const uint32_t stage = base + Lay::kStage + warp * 2048;
            const int rows = it.n - (q0 + quarter * 32);  // of the warp that exist
            bf16* const o = p.out + (static_cast<int64_t>(it.start) + q0 + quarter * 32) * p.out_stride + head * D;
            if (marked_odd[mark_place(ord)] == ord) {
#pragma unroll 1
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t r[16];
                    tmem_ld16(tO + c * 16, r);
                    tc_wait_ld();
                    add_odd_values(p, it, n, c * 16, seen_bits, r);
                    tmem_st16(tO + c * 16, r);
                }
                tc_wait_st();
            }
            const uint32_t put = stage + lane * 64, swz = (lane >> 1) & 3;
            const uint32_t get = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
            bf16* dst = o + (lane >> 2) * p.out_stride + (lane & 3) * 8;
            const int64_t step = 8 * p.out_stride;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c, dst += 32) {
                uint32_t r[32];
                tmem_ld32(tO + c * 32, r);
                tc_wait_ld();
                if (c + 1 == D / 32) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kOEmpty + x));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = put + ((i ^ swz) << 4);
                    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a),
                                 "r"(pack_bf16x2(__uint_as_float(r[8 * i]) * inv, __uint_as_float(r[8 * i + 1]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(r[8 * i + 2]) * inv, __uint_as_float(r[8 * i + 3]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(r[8 * i + 4]) * inv, __uint_as_float(r[8 * i + 5]) * inv)),
                                 "r"(pack_bf16x2(__uint_as_float(r[8 * i + 6]) * inv, __uint_as_float(r[8 * i + 7]) * inv))
                                 : "memory");
                }
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 w = lds128(get + i * 512);  // rows lane / 4, 8 apart: the same swizzle
                    if ((lane >> 2) + i * 8 < rows) *reinterpret_cast<uint4*>(dst + i * step) = w;
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) give_up(p.err, abort_flag);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 9) tmem_dealloc(tmem, kTmemCols);
    if (tid == 0) {  // the last CTA leaves the counters at zero for the next launch
        const uint32_t done = atomicAdd(p.work + 1, 1u);
        if (done == gridDim.x - 1) {
            p.work[0] = 0u;
            p.work[1] = 0u;
        }
    }
}

template <int D>
cudaError_t launch_d(const PackedPrefillParams& p, const PackedMaps& m, int num_sms, cudaStream_t s) {
    static SmemLimitOnce limit;
    const cudaError_t e = limit.apply(reinterpret_cast<const void*>(&prefill_packed_kernel<D>), kMaxSmem);
    if (e != cudaSuccess) return e;
    // No more CTAs than there can be items; the whole shared memory for every D: one CTA
    // per SM, so none waits for TMEM.
    const int64_t units = (p.h.n_retr + p.h.n_strm) * ((p.G & 1) ? p.G : p.G / 2);
    const int64_t items = ((p.n_rows + kTileQ - 1) / kTileQ + p.n) * units;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(items < num_sms ? items : num_sms));
    cfg.blockDim = dim3(kPackThreads);
    cfg.dynamicSmemBytes = kMaxSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, &prefill_packed_kernel<D>, p, m);
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedPrefillParams& p, const PackedMaps& m, int num_sms, cudaStream_t s) {
    if (Layout<128>::bytes(p.n) > kMaxSmem) return cudaErrorInvalidValue;
    return p.D == 128 ? launch_d<128>(p, m, num_sms, s) : launch_d<64>(p, m, num_sms, s);
}

}  // namespace duo
