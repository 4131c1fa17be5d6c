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
//   warp 8     takes the items, loads Q and the K tiles (2 stages)
//   warp 9     issues the products (one thread), owns TMEM
//   warp 10    loads the V tiles (2 stages); warps 10 and 11 clear the tiles that
//              are seen in part of what a weight of zero must not meet
// TMEM (512 columns): S of A and B, 128 columns each, P (bf16) written over the S
// it was made from, O of A and of B at 256.
// Softmax in the exp2 domain; the running maximum moves only when it grows by
// more than 2^8 (exact), sums in 32 bits; P rounded to bf16, the operand type
// (relative 2^-9 per term). Every mbarrier wait is bounded; on timeout the CTA
// records kErrPagedWait and unwinds.
#include <type_traits>

#include "paged_internal.cuh"
#include "prefill_common.cuh"

namespace duo {

namespace {

constexpr int kPackThreads = 384;
constexpr int kSoftmaxRegs = 216;
constexpr int kOtherRegs = 72;
static_assert(2 * kSoftmaxRegs + kOtherRegs <= 3 * 168, "registers of a 384-thread launch");

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
constexpr int kQueueSlots = 4;
constexpr int kConsumers = 11;  // 8 softmax warps, the issuer, 2 V warps

// Query tiles of a prompt of `len` rows.
__device__ __forceinline__ int query_tiles(int len, int rows) { return (len + rows - 1) / rows; }

__device__ __forceinline__ PackItem pack_item(const PackedPrefillParams& p, const Prompts& pr, int64_t idx) {
    PackItem it;
    const bool by_heads = (p.G & 1) == 0;       // tile pair = two heads of a group, or 256 rows of one
    const int rows = by_heads ? kTileQ : 2 * kTileQ;
    const int per_kv = by_heads ? p.G / 2 : p.G;
    const int64_t n_tiles = pr.tiles_before[pr.n_groups];
    const int64_t of_retr = n_tiles * p.h.n_retr * per_kv;
    it.retr = idx < of_retr;
    const int units = (it.retr ? p.h.n_retr : p.h.n_strm) * per_kv;
    const int64_t x = it.retr ? idx : idx - of_retr;
    int lo = 0, up = pr.n_groups - 1;
    while (lo < up) {
        const int mid = (lo + up + 1) >> 1;
        if (static_cast<int64_t>(pr.tiles_before[mid]) * units <= x) lo = mid;
        else up = mid - 1;
    }
    const int64_t y = x - static_cast<int64_t>(pr.tiles_before[lo]) * units;
    const int nt = pr.tiles_before[lo + 1] - pr.tiles_before[lo];
    const int qt = nt - 1 - static_cast<int>(y / units);
    const int unit = static_cast<int>(y % units);
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
// The products and commits of sm100.cuh, issued by the lanes with `lead` set only.
__device__ __forceinline__ void tc_mma_ss_by(uint32_t lead, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tc_mma_ts_by(uint32_t lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                             uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\t"
        "setp.ne.b32 e, %5, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead)
        : "memory");
}
__device__ __forceinline__ void tc_commit_by(uint32_t lead, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.b32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
        "r"(lead)
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

// Adds to 32 columns of a row, from `col`, the infinities and NaN of the value rows
// that it sees among the tiles that were cleared of them: a visible row has a
// positive weight, so the sum is that value whatever the weight is.
template <typename Seen>
__device__ __forceinline__ void add_odd_values(const PackedPrefillParams& p, const PackItem& it, int n, int col, Seen seen,
                                               uint32_t (&r)[32]) {
    const int last_row = (it.nb > 0 ? it.qb : it.qa) + kTileQ - 1;
    const bf16* const v = p.v + static_cast<int64_t>(it.start) * p.kv_stride + it.g * p.D + col;
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
        const int row0 = key_row(it, j);
        if (!(row0 + kTileK > it.qa || (!it.retr && row0 + kTileK > p.S && row0 <= last_row - p.R))) continue;
#pragma unroll 1
        for (int k0 = row0; k0 < row0 + kTileK && k0 < it.n; k0 += 32)
#pragma unroll 1
            for (uint32_t bits = seen(k0); bits; bits &= bits - 1) {
                const bf16* const row = v + (k0 + __ffs(bits) - 1) * p.kv_stride;  // seen keys are rows of the group
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = __bfloat162float(row[i]);
                    if (!isfinite(x)) r[i] = __float_as_uint(__uint_as_float(r[i]) + x);
                }
            }
    }
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
    // By item (modulo 8): a V tile that some rows see in part held an infinity or NaN.
    volatile int* const odd_values = reinterpret_cast<volatile int*>(smem + Lay::kMisc + 80);
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
            mbar_init(bar(kOEmpty + s), 4);
            mbar_init(bar(kPFull + 2 * s), 4);
            mbar_init(bar(kPFull + 2 * s + 1), 4);
        }
        for (int s = 0; s < kQueueSlots; ++s) {
            mbar_init(bar(kItemFull + s), 1);
            mbar_init(bar(kItemEmpty + s), kConsumers);
        }
        *abort_flag = 0;
        for (int i = 0; i < 8; ++i) odd_values[i] = 0;
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
    for (int i = tid; i < p.n; i += kPackThreads) {
        // The first unusable prompt at i or behind; up to there the rows ascend.
        int stop = p.n;
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
    if (tid == 0) {
        int g = 0;
        for (int i = 0; i < p.n; i = pr.next[i]) pr.first[g++] = static_cast<uint16_t>(i);
        pr.first[g] = static_cast<uint16_t>(p.n);
        *n_groups = g;
    }
    __syncthreads();
    pr.n_groups = *n_groups;
    for (int i = tid; i < pr.n_groups; i += kPackThreads) {
        const int f = pr.first[i];
        pr.len[i] = (wrong[f >> 5] >> (f & 31)) & 1u ? 0 : pr.row[pr.first[i + 1]] - pr.row[f];
    }
    __syncthreads();
    for (int i = tid; i < pr.n_groups; i += kPackThreads) {
        const int len = pr.len[i];
        int rank = 0;
        for (int j = 0; j < pr.n_groups; ++j) rank += pr.len[j] > len || (pr.len[j] == len && j < i);
        pr.by_rank[rank] = static_cast<uint16_t>(i);
    }
    __syncthreads();
    if (warp == 0) {
        const int rows = (p.G & 1) ? 2 * kTileQ : kTileQ;
        int sum = 0;
        for (int i0 = 0; i0 < pr.n_groups; i0 += 32) {
            const int i = i0 + lane;
            const int own = i < pr.n_groups ? query_tiles(pr.len[pr.by_rank[i]], rows) : 0;
            int t = own;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int a = __shfl_up_sync(0xffffffffu, t, o);
                if (lane >= o) t += a;
            }
            if (i < pr.n_groups) pr.tiles_before[i] = sum + t - own;
            sum += __shfl_sync(0xffffffffu, t, 31);
        }
        if (lane == 0) pr.tiles_before[pr.n_groups] = sum;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int64_t n_items =
        static_cast<int64_t>(pr.tiles_before[pr.n_groups]) * (p.h.n_retr + p.h.n_strm) * ((p.G & 1) ? p.G : p.G / 2);

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
            // The next item is taken and published before this one's K tiles are loaded,
            // so that nobody waits for the counter.
            tma_prefetch_desc(&maps.q);
            int published = 0;
            auto publish = [&](PackItem& it) -> bool {
                const unsigned i = *abort_flag == 0 ? atomicAdd(p.work, 1u) : 0xFFFFFFFFu;
                it.idx = -1;
                if (i < n_items) it = pack_item(p, pr, i);
                const int slot = published % kQueueSlots;
                if (published >= kQueueSlots &&
                    !mbar_wait(bar(kItemEmpty + slot), ((published / kQueueSlots) - 1) & 1, abort_flag))
                    return false;
                queue[slot] = it;
                mbar_arrive(bar(kItemFull + slot));
                ++published;
                return true;
            };
            int g = 0;  // K tiles issued
            int q_loads = 0;
            PackItem it, after;
            bool ok = publish(it);
            while (ok && it.idx >= 0) {
                ok = publish(after);
                if (ok && q_loads >= 1) ok = mbar_wait(bar(kQEmpty), (q_loads - 1) & 1, abort_flag);
                if (!ok) break;
                mbar_arrive_expect_tx(bar(kQFull), (it.nb > 0 ? 2 : 1) * Lay::kTile);
                for (int kb = 0; kb < Lay::kColBlocks; ++kb) {
                    tma_load_3d(sQ + kb * kTileBytesPerColBlock, &maps.q, bar(kQFull), kb * 64, it.head_a, it.start + it.qa);
                    if (it.nb > 0)
                        tma_load_3d(sQ + Lay::kTile + kb * kTileBytesPerColBlock, &maps.q, bar(kQFull), kb * 64, it.head_b,
                                    it.start + it.qb);
                }
                ++q_loads;
                const int n = it.na > it.nb ? it.na : it.nb;
                for (int j = 0; j < n; ++j, ++g) {
                    const int st = g & 1;
                    if (g >= 2 && !mbar_wait(bar(kKEmpty + st), ((g >> 1) - 1) & 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    mbar_arrive_expect_tx(bar(kKFull + st), Lay::kTile);
                    for (int kb = 0; kb < Lay::kColBlocks; ++kb)
                        tma_load_3d(sK + st * Lay::kTile + kb * kTileBytesPerColBlock, &maps.k, bar(kKFull + st), kb * 64,
                                    it.g, it.start + key_row(it, j));
                }
                it = after;
            }
            if (!ok) give_up(p.err, abort_flag);
            // Every load issued lands before the CTA may exit.
            for (int j = g > 2 ? g - 2 : 0; j < g; ++j) mbar_wait(bar(kKFull + (j & 1)), (j >> 1) & 1, nullptr);
            if (q_loads > 0) mbar_wait(bar(kQFull), (q_loads - 1) & 1, nullptr);
        } else if (warp >= 10) {
            // -------------------------------------------------------- V
            // Warp 10 loads. A tile that some row of the item sees only in part (the
            // diagonal, the window's edges, a group of prompts) is then gone through by
            // both warps, half each, before the products may read it: a weight of zero
            // must not meet an infinity or a NaN. Rows behind the group's end, which
            // belong to other prompts or to nobody, become zero; a non-finite element
            // becomes zero too and is counted for the rows that see it at the item's end.
            const int half = warp - 10;
            int g = 0, raw = 0;
            for (int ord = 0;; ++ord) {
                PackItem it;
                const bool more = take_item(ord, it);
                __syncwarp();
                if (lane == 0) free_item(ord);
                if (!__all_sync(0xffffffffu, more)) break;
                // The flag of four items ago, whose rows have long been written.
                if (half == 0 && lane == 0) odd_values[(ord + 4) & 7] = 0;
                const int n = it.na > it.nb ? it.na : it.nb;
                const int last_row = (it.nb > 0 ? it.qb : it.qa) + kTileQ - 1;
                bool ok = true;
                for (int j = 0; j < n; ++j, ++g) {
                    const int st = g & 1;
                    if (g >= 2 && !mbar_wait(bar(kVEmpty + st), ((g >> 1) - 1) & 1, abort_flag)) ok = false;
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const int row0 = key_row(it, j);
                    const bool part =
                        row0 + kTileK > it.qa || (!it.retr && row0 + kTileK > p.S && row0 <= last_row - p.R);
                    const uint32_t full = part ? bar(kVRaw + (raw & 1)) : bar(kVFull + st);
                    if (half == 0 && lane == 0) {
                        mbar_arrive_expect_tx(full, Lay::kTile);
                        for (int kb = 0; kb < Lay::kColBlocks; ++kb)
                            tma_load_3d(sV + st * Lay::kTile + kb * kTileBytesPerColBlock, &maps.v, full, kb * 64, it.g,
                                        it.start + row0);
                        if (!part) mbar_arrive(full);  // for the other warp
                    }
                    if (part) {
                        ok = __all_sync(0xffffffffu, mbar_wait(bar(kVRaw + (raw & 1)), (raw >> 1) & 1, nullptr));
                        ++raw;
                        const int valid = it.n - row0;
                        bool odd = false;
#pragma unroll
                        for (int kb = 0; kb < Lay::kColBlocks; ++kb) {
                            const uint32_t tile = sV + st * Lay::kTile + kb * kTileBytesPerColBlock + half * (64 * 128);
                            uint32_t seen = 0;
#pragma unroll 4
                            for (int i = 0; i < 64 * 8 / 32; ++i) {
                                const int row = half * 64 + i * 4 + (lane >> 3);
                                const uint32_t a = tile + (i * 32 + lane) * 16;
                                if (row < valid) {
                                    const uint4 w = lds128(a);
                                    // Bit 15 of a half word: its exponent bits are all ones.
                                    seen |= ((w.x & 0x7F807F80u) + 0x00800080u) | ((w.y & 0x7F807F80u) + 0x00800080u) |
                                            ((w.z & 0x7F807F80u) + 0x00800080u) | ((w.w & 0x7F807F80u) + 0x00800080u);
                                } else {
                                    asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(a), "r"(0u) : "memory");
                                }
                            }
                            if (__any_sync(0xffffffffu, (seen & 0x80008000u) != 0u)) {
                                odd = true;
#pragma unroll 1
                                for (int i = lane; i < 64 * 32; i += 32) {
                                    uint32_t w;
                                    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(tile + i * 4));
                                    if ((w & 0x7F80u) == 0x7F80u) w &= 0xFFFF0000u;
                                    if ((w & 0x7F800000u) == 0x7F800000u) w &= 0x0000FFFFu;
                                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(tile + i * 4), "r"(w) : "memory");
                                }
                            }
                        }
                        if (odd && lane == 0) odd_values[ord & 7] = 1;
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(kVFull + st));
                    }
                }
                if (!ok) {
                    if (lane == 0) give_up(p.err, abort_flag);
                    break;
                }
            }
            for (int j = g > 2 ? g - 2 : 0; j < g; ++j) mbar_wait(bar(kVFull + (j & 1)), (j >> 1) & 1, abort_flag);
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
            int g = 0;               // K/V tiles of the items before
            int count_a = 0, count_b = 0;  // products PV of each tile so far
            int items_a = 0, items_b = 0;  // items that had the tile so far
            bool ok = true;
            for (int ord = 0; ok; ++ord) {
                PackItem it;
                const bool more = take_item(ord, it);
                __syncwarp();
                if (lead) free_item(ord);
                if (!__all_sync(0xffffffffu, more)) break;
                const int na = __shfl_sync(0xffffffffu, it.na, 0), nb = __shfl_sync(0xffffffffu, it.nb, 0);
                const int n = na > nb ? na : nb;
                ok = __all_sync(0xffffffffu, mbar_wait(bar(kQFull), ord & 1, abort_flag));
                // S(x) = Q(x) K(j)^T; `last`: the last to read the K tile.
                auto qk = [&](auto x_, int j, bool wait, bool last) {
                    constexpr int x = decltype(x_)::value;
                    const int st = (g + j) & 1;
                    if (wait && !__all_sync(0xffffffffu, mbar_wait(bar(kKFull + st), ((g + j) >> 1) & 1, abort_flag))) return false;
                    tc_fence_after();
                    const uint64_t q = dq + x * (Lay::kTile >> 4), k = dk + st * (Lay::kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * kTileBytesPerColBlock + (kk & 3) * 32) >> 4;
                        tc_mma_ss_by(lead, tmem + x * kTileK, q + off, k + off, idesc_qk, kk > 0 ? 1u : 0u);
                    }
                    tc_commit_by(lead, bar(kSFull + x));
                    if (last) {
                        tc_commit_by(lead, bar(kKEmpty + st));
                        if (j + 1 == n) tc_commit_by(lead, bar(kQEmpty));
                    }
                    return true;
                };
                // O(x) += P(x) V(j); `last`: the last to read the V tile.
                auto pv = [&](auto x_, int j, bool wait, bool last, int count, int items) {
                    constexpr int x = decltype(x_)::value;
                    const int st = (g + j) & 1;
                    if (wait && !__all_sync(0xffffffffu, mbar_wait(bar(kVFull + st), ((g + j) >> 1) & 1, abort_flag))) return false;
                    if (j == 0 && items > 0 &&
                        !__all_sync(0xffffffffu, mbar_wait(bar(kOEmpty + x), (items - 1) & 1, abort_flag)))
                        return false;
                    const uint64_t vt = dv + st * (Lay::kTile >> 4);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        if (!__all_sync(0xffffffffu, mbar_wait(bar(kPFull + 2 * x + half), count & 1, abort_flag))) return false;
                        tc_fence_after();
#pragma unroll
                        for (int k4 = 0; k4 < 4; ++k4) {
                            const int kk = half * 4 + k4;
                            tc_mma_ts_by(lead, tmem + kTmemO + x * 128, tmem + x * kTileK + kk * 8, vt + kk * (2048 >> 4),
                                         idesc_pv, (j > 0 || kk > 0) ? 1u : 0u);
                        }
                    }
                    tc_commit_by(lead, bar(kODone + x));
                    if (last) tc_commit_by(lead, bar(kVEmpty + st));
                    return true;
                };
                constexpr std::integral_constant<int, 0> A{};
                constexpr std::integral_constant<int, 1> B{};
                // The tiles' lists differ by one tile at most, or one is empty.
                if (ok && na > 0) ok = qk(A, 0, true, nb == 0);
                if (ok && nb > 0) ok = qk(B, 0, na == 0, true);
                for (int j = 0; ok && j < n; ++j) {
                    if (j < na) {
                        ok = pv(A, j, true, j >= nb, count_a, items_a);
                        ++count_a;
                        if (ok && j + 1 < na) ok = qk(A, j + 1, true, j + 1 >= nb);
                    }
                    if (ok && j < nb) {
                        ok = pv(B, j, j >= na, true, count_b, items_b);
                        ++count_b;
                        if (ok && j + 1 < nb) ok = qk(B, j + 1, j + 1 >= na, true);
                    }
                }
                items_a += na > 0;
                items_b += nb > 0;
                g += n;
            }
            if (!ok && lead) give_up(p.err, abort_flag);
            tc_commit_by(lead, bar(kDrain));  // every product issued has completed before TMEM is released
            mbar_wait(bar(kDrain), 0, nullptr);
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
            RowVis vis = row_visible(it.retr, 0, it.n, p.S, p.R, q0 + row);
            int own0 = 0;  // first row of this row's prompt, in the group
            const bool single = it.p1 - it.p0 == 1;
            if (!single) {
                int lo = it.p0, up = it.p1 - 1;
                while (lo < up) {
                    const int mid = (lo + up + 1) >> 1;
                    if (pr.row[mid] <= it.start + row) lo = mid;
                    else up = mid - 1;
                }
                __syncwarp();
                own0 = pr.row[lo] - it.start;
                vis.c_sink = it.retr ? 0 : own0 + p.S;
            }
            // The 32 keys from k0 that this row sees.
            auto seen_bits = [&](int k0) { return chunk_bits_row(vis, k0) & ~bits_below32(own0 - k0); };
            float m_run = -INFINITY, l_run = 0.f;
            for (int j = 0; j < n; ++j, ++count) {
                if (!__all_sync(0xffffffffu, mbar_wait(bar(kSFull + x), count & 1, abort_flag))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t s[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, s[c]);
                tc_wait_ld();
                const int row0 = key_row(it, j);
                // The tile in four runs of 32 keys: what the warp's 32 rows [r0, r0 + 31] see
                // of each is all of it, nothing, or a part, by comparisons that are the same
                // for the whole warp. Only parts are masked element by element; a run that
                // no row sees costs nothing but a zero P.
                const int r0 = q0 + quarter * 32;
                uint32_t none = 0;  // bit c: nothing of run c is seen
                float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto max_of = [&](const uint32_t (&run)[32]) {
#pragma unroll
                    for (int i = 0; i < 32; i += 2)
                        m[(i >> 1) & 3] = fmax3(m[(i >> 1) & 3], __uint_as_float(run[i]), __uint_as_float(run[i + 1]));
                };
                if (row0 + kTileK <= q0 && (it.retr || row0 + kTileK <= p.S || row0 > q0 + kTileQ - 1 - p.R)) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) max_of(s[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int k0 = row0 + 32 * c, k1 = k0 + 31;
                        if (k0 > r0 + 31 || (!it.retr && single && k0 >= p.S && k1 <= r0 - p.R)) {
                            none |= 1u << c;
                            continue;
                        }
                        if (!(k1 <= r0 && single && (it.retr || k1 < p.S || k0 > r0 + 31 - p.R))) {
                            const uint32_t bits = seen_bits(k0);
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (!((bits >> k) & 1u)) s[c][k] = 0xFF800000u;  // -inf
                        }
                        max_of(s[c]);
                    }
                }
                const float mt = fmax3(fmaxf(m[0], m[1]), m[2], m[3]) * p.scale_log2;
                float factor = 1.f;
                if (mt > m_run + kRescaleThreshold) {
                    factor = fast_exp2(m_run - mt);
                    m_run = mt;
                }
                // PV(j-1) is the last product that wrote O.
                if (j >= 1 && __any_sync(0xffffffffu, factor != 1.f)) {
                    if (!__all_sync(0xffffffffu, mbar_wait(bar(kODone + x), (count - 1) & 1, abort_flag))) {
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
                const float m_use = m_run == -INFINITY ? 0.f : m_run;
                const uint64_t negm = f2pack(-m_use, -m_use);
                uint64_t acc[2] = {f2pack(0.f, 0.f), f2pack(0.f, 0.f)};
                // Weights, in two versions: with a test per run the compiler cannot overlap
                // the runs, which costs a fully seen tile 8 %.
                auto weights = [&](auto some_) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t pk[16];
                        if (decltype(some_)::value && ((none >> c) & 1u)) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) pk[i] = 0u;
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; i += 2) {
                                float e0, e1;
                                f2unpack(ffma2(f2pack(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])), scale2, negm),
                                         e0, e1);
                                const float p0 = fast_exp2(e0), p1 = fast_exp2(e1);
                                acc[(i >> 1) & 1] = fadd2(acc[(i >> 1) & 1], f2pack(p0, p1));
                                pk[i >> 1] = pack_bf16x2(p0, p1);
                            }
                        }
                        tmem_st16(tS + c * 16, pk);  // every S column has been read
                        if (c & 1) {
                            tc_wait_st();
                            tc_fence_before();
                            __syncwarp();
                            if (lane == 0) mbar_arrive(bar(kPFull + 2 * x + (c >> 1)));
                        }
                    }
                };
                if (none == 0) weights(std::false_type{});
                else weights(std::true_type{});
                float a0, a1;
                f2unpack(fadd2(acc[0], acc[1]), a0, a1);
                l_run = l_run * factor + (a0 + a1);
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
            const bool odd = odd_values[ord & 7] != 0;
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t r[32];
                tmem_ld32(tO + c * 32, r);
                tc_wait_ld();
                if (odd) add_odd_values(p, it, n, c * 32, seen_bits, r);
                if (c + 1 == D / 32) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(kOEmpty + x));
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t a = stage + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4);
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
                    const int rr = i * 8 + (lane >> 2), ch = lane & 3;
                    const uint4 w = lds128(stage + rr * 64 + ((ch ^ ((rr >> 1) & 3)) << 4));
                    if (rr < rows) *reinterpret_cast<uint4*>(o + rr * p.out_stride + c * 32 + ch * 8) = w;
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
    // The whole shared memory for every D: one CTA per SM, so none waits for TMEM.
    prefill_packed_kernel<D><<<static_cast<unsigned>(num_sms), kPackThreads, kMaxSmem, s>>>(p, m);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill_packed(const PackedPrefillParams& p, const PackedMaps& m, int num_sms, cudaStream_t s) {
    if (Layout<128>::bytes(p.n) > kMaxSmem) return cudaErrorInvalidValue;
    return p.D == 128 ? launch_d<128>(p, m, num_sms, s) : launch_d<64>(p, m, num_sms, s);
}

}  // namespace duo
