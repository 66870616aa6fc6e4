// chunk_attention, bfloat16 path on the 5th-generation tensor cores.
//
// The online softmax over 128-key tiles: S = Q K^T, m = running row maximum, P =
// 2^(S c - m), O += P V, O / sum(P) at the end.  Bound by the tensor core for
// long chunks (4 d operations per row and key) and by the K/V stream for a few
// rows per sequence (plain decoding).
//
// Rows are packed: token-major, then the G = Hq / Hkv query heads of a kv head,
// so every K/V byte is read once for all of them.  A row tile holds npt =
// floor(128 / G) whole tokens; an item is (sequence, kv head, up to two
// consecutive row tiles) with its range of keys.  One CTA per SM keeps two
// streams of products going, so that the tensor core works on one while the
// softmax of the other runs:
//   two row tiles  stream i is row tile i, both over the same key tiles (each
//                  K/V tile in shared memory serves 256 rows);
//   one row tile   (at most npt tokens left) stream i takes the key tiles t with
//                  t % 2 == i, and the two results are joined at the end.
//
// Balance: an item costs its keys plus a fixed C0 (in keys).  The items of all
// sequences, laid end to end, are cut into one run of equal cost per CTA, so
// every CTA has the same work whatever the lengths; the run's borders follow
// from closed forms, so nothing is precomputed and the schedule is made on the
// device from the lengths (a captured graph serves any of them).  An item cut by
// a border leaves one partial result (unnormalised O, maximum, sum, float32)
// per run in the workspace, and a second kernel joins them in order.
//
// CTA roles (384 threads)
//   warps 0-3, 4-7  softmax of stream 0 and 1: thread r owns row r (tensor-memory
//            lane r).  P (bfloat16 pairs) takes the place of S in tensor memory.
//            The running maximum is raised (and O rescaled) only when a row grows
//            by more than 2^8.
//   warp 8   issues every product, alternating the streams: PV(i, t - 1), then
//            S(i, t).  The tensor core works in issue order, so S(i, t) may
//            overwrite P(i, t - 1), and S(i, t)'s completion implies that O holds
//            every earlier product (a rescale waits for nothing else).
//   warp 9   K/V producer: 16-key pages by TMA into a ring of slots, in the order
//            in which warp 8 consumes them.
//   warp 10  loads the items' Q tiles, and clears what must not reach O (zero weight
//            times NaN is NaN) in the V tiles that not every row sees whole: rows that
//            no row of the item attends to (past its last key, or before its first
//            in the same page), and rows with NaN or infinity that some attend to; these
//            are noted, and the rows that do attend to them add them in their
//            epilogue.  Such tiles land on a barrier of their own (vraw), and warp 10
//            passes them on to warp 8.
//   warp 11  scheduler: walks the run, checks each new sequence's blocks, and
//            publishes the items a few ahead.
// Measured: 4,096 rows after 12,281 keys (28/4 heads of 128) 547 us = 1,539 TFLOP/s by
// themselves, 574-584 us called for seconds under the power cap; one row of each of 64
// sequences of 512-8,192 keys 121 us = 5.8 TB/s; chunks of 1-1,500 rows 89 us (four to five us
// per item beside its tiles); one row after 300 keys 14 us (captured 12).  A pair of
// tiles of two full row tiles takes 1.65 us, of which the softmax is the longer half; an
// exponential by polynomial for a part of the scores is slower (573-680 us), as are four
// softmax warpgroups.
// Every wait is bounded; one that runs out sets the abort flag, which ends the other
// roles' waits, and the roles leave after their copies and products in flight are done.
// The CTA's records then name the sequences of its run, and the second kernel, behind
// every TV_OK, gives them TV_ERR_TIMEOUT.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "tv_chunk.cuh"
#include "tv_internal.h"
#include "tv_tc.cuh"

namespace tv {

namespace {

constexpr int KT = 128;            // keys per tile
constexpr int MT = 128;            // rows per row tile
constexpr int THREADS = 384;
constexpr int MMA_WARP = 8, LOAD_WARP = 9, FIX_WARP = 10, SCHED_WARP = 11;
constexpr int GQ = 4;              // items published ahead
constexpr int FIX_TILES = 6;       // key tiles of an item that only some of its rows see
constexpr int FIX_BUFS = 4;        // items whose V notes may be live (see warp 10)
// Rows up to which the epilogue of a single row tile goes through shared memory row by
// row (both streams' rows of D + 4 floats fit the second Q tile): one warp would write
// them out alone otherwise.
constexpr int FEW = 30;
static_assert(2 * FEW * (128 + 4) * 4 <= MT * 128 * 2 && 2 * FEW * (64 + 4) * 4 <= MT * 64 * 2, "xo");
// a border this close to an item's end (in tiles) moves there: a cut costs more than the
// imbalance
constexpr int SNAP = 2;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float RESCALE_LOG2 = 8.0f;
// fixed cost of an item, in keys: Q load, pipeline fill and drain, epilogue
constexpr int64_t C0 = 512;
// cost of a run, in keys, below which cutting further costs more to join than it saves
constexpr int64_t RUN_MIN = 768;

struct alignas(16) Item {      // moved as four 16-byte words
    int b, g, P, i0;        // sequence, kv head, prefix, first token
    int ntok, row0, kbase, hi;  // tokens; row of the first; first key (multiple of 16), key end
    int t_lo, t_hi, fa, fb; // key tiles of this piece; tiles < fa or >= fb need masks
    int flags, slot, n, pad;  // slot: partial result, or -1; n: tiles to do (0: bad sequence)
};
// A slot's record: it holds a piece, and the piece is the item's last one; or a wait of the CTA
// ran out (then the record is: first and last sequence of its run).
constexpr int PIECE = 1, PIECE_LAST = 2, PIECE_LATE = 4;
constexpr int ITEM_END = 1, ITEM_TWO = 2, ITEM_BAD = 4, ITEM_STATUS = 8;
static_assert(sizeof(Item) == 64 && alignof(Item) == 16, "four 16-byte words");

template <int D>
struct Lay {
    static constexpr int HALVES = D / 64;
    static constexpr int PAGE_BYTES = 16 * D * 2;
    static constexpr int SLOT_BYTES = KT * D * 2;
    static constexpr int SLOTS = D == 128 ? 5 : 10;
    static constexpr int Q_BYTES = MT * D * 2;             // one row tile
    static constexpr int OFF_RING = 0;
    static constexpr int OFF_Q = SLOTS * SLOT_BYTES;       // two row tiles
    static constexpr int OFF_X = OFF_Q + Q_BYTES;          // epilogue of one row tile: the second Q tile
    static constexpr int OFF_ITEMS = OFF_Q + 2 * Q_BYTES;  // [GQ]
    static constexpr int OFF_MISC = OFF_ITEMS + GQ * 64;   // tensor memory's address, abort flag
    static constexpr int OFF_BARS = OFF_MISC + 16;
    static constexpr int NBARS = 3 * SLOTS + 8 + 4 + 2 * GQ + 2;
    static constexpr int OFF_BAD = OFF_BARS + (NBARS * 8 + 15) / 16 * 16;  // [FIX_BUFS][FIX_TILES][4]
    static constexpr int OFF_ML = OFF_BAD + FIX_BUFS * FIX_TILES * 16;  // join: maximum, sum per row
    static constexpr int BYTES = OFF_ML + 2 * MT * 4 + 1024;   // + alignment slack
    static_assert(OFF_ITEMS % 1024 == 0 && OFF_BAD - OFF_ITEMS <= 1024, "the barriers beside the abort flag");
};
static_assert(Lay<128>::BYTES <= 232448 && Lay<64>::BYTES <= 232448, "shared memory of one SM");

struct Params {
    ChunkView c;
    __nv_bfloat16* out;
    int64_t o_stride;
    const __nv_bfloat16* q;      // for the rows that see a V row with NaN or infinity
    int64_t q_stride;
    const __nv_bfloat16* k;
    const __nv_bfloat16* v;
    int32_t* status;
    int4* rec;                   // what the slots hold: (first row, tokens, kv head, PIECE_*)
    float* part;                 // partial results, two slots per CTA
    int Hkv, G, npt, window;
    int prows;                   // rows of a partial result: 128 or 256
    float scale_log2;            // scale * log2(e); with a cap: 2 log2(e) scale / cap
    float cap_log2;              // cap * log2(e)
    float cap_x, cap_small;      // scale / cap; products with s^2 < cap_small take the polynomial
    float cap_c[3];              // its coefficients in s^2: scale * log2(e) * (scale / cap)^(2e) * TANH_C[e]
    LateWait late;               // test-only
};

// tanh(x) / x as a polynomial in x^2 for |x| <= 0.35: interpolated at the Chebyshev nodes of
// [0, 0.35^2] (its nearest pole is at x^2 = -pi^2 / 4), off by at most 2.9e-6 of itself: of a
// score of 100 that is a fourteenth of a weight's rounding (2^-8).  The error changes slowly with
// the score, and what the scores near a row's maximum share cancels in the softmax.
// One term more costs 2.6 us of 41 (2,100 tokens of 16 heads of 64, window 1024).
constexpr double TANH_SMALL = 0.35;
constexpr double TANH_C[3] = {0.9999971183259196, -0.3329087359461761, 0.12394375936950675};

// ------------------------------------------------------------ the run space
// Sequence of n rows after P keys: items of m = 2 npt tokens, item k costing C0 +
// min(P + (k + 1) m, window + m) keys, the last one C0 + min(P + n, window + m).
struct Seq {
    int P, n, m, items;          // m: tokens per item
    int64_t w;                   // window + m, or no limit
    bool shape;                  // P and n fit the block table
};
constexpr int64_t NO_WINDOW = 1ll << 40;

__device__ __forceinline__ Seq seq_of(const Params& p, int P, int n) {
    Seq s;
    s.P = P;
    s.n = n;
    s.shape = chunk_shape_ok(p.c, P, n);
    s.m = 2 * p.npt;
    s.w = p.window > 0 ? (int64_t)p.window + s.m : NO_WINDOW;
    s.items = (int)(((unsigned)n + (unsigned)s.m - 1) / (unsigned)s.m);
    return s;
}
// Cost of item k, and of the first k items.
__device__ __forceinline__ int64_t item_cost(const Seq& s, int k) {
    if (!s.shape) return C0;
    return C0 + min((int64_t)s.P + min((int64_t)s.n, (int64_t)(k + 1) * s.m), s.w);
}
__device__ __noinline__ int64_t seq_cost(Seq s, int k) {
    if (!s.shape || k == 0) return k * C0;
    const int64_t full = min(k, s.items - 1);                    // items of m tokens
    int64_t lin = full;                                          // of them below the window's limit
    if (s.w != NO_WINDOW) lin = s.w > s.P ? min(full, (int64_t)((unsigned)(s.w - s.P) / (unsigned)s.m)) : 0;
    int64_t c = lin * s.P + s.m * (lin * (lin + 1) / 2) + full * C0;
    if (lin < full) c += (full - lin) * s.w;
    return k == s.items ? c + item_cost(s, k - 1) : c;
}
__device__ __forceinline__ int64_t seq_units(const Params& p, int P, int n) {
    const Seq s = seq_of(p, P, n);
    return s.items == 0 ? 0 : seq_cost(s, s.items) * p.Hkv;
}
// Keys of item k: from kbase (multiple of 16) to hi, in tiles of KT.
__device__ __forceinline__ void item_keys(const Params& p, const Seq& s, int k, int& i0, int& i1,
                                          int& kbase, int& hi, int& tiles) {
    i0 = k * s.m;
    i1 = min(s.n, i0 + s.m);
    if (!s.shape) {
        kbase = hi = tiles = 0;
        return;
    }
    hi = s.P + i1;
    kbase = chunk_first_key(s.P + i0, p.window) & ~15;
    tiles = (hi - kbase + KT - 1) / KT;
}
// Tile at which a border y units into an item of the given cost cuts it (both runs
// beside the border compute it; non-decreasing in y).
__device__ __noinline__ int cut_tile(int64_t y, int64_t cost, int tiles) {
    if (y <= C0) return 0;
    if (y >= cost) return tiles;
    const float per = __fdiv_rn((float)tiles, (float)(cost - C0));
    const int t = (int)ceilf(__fmul_rn((float)(y - C0), per));
    return t <= SNAP ? 0 : (t >= tiles - SNAP ? tiles : t);
}
// Item at unit y of a sequence (Hkv equal stretches): kv head, item, its first unit.
__device__ __forceinline__ void item_at(const Params& p, const Seq& s, int64_t y, int& g, int& k,
                                        int64_t& start) {
    const int64_t per = seq_cost(s, s.items);
    g = min(p.Hkv - 1, (int)__fdiv_rn((float)y, (float)per));
    while (g * per > y) --g;                                     // the quotient, made exact
    while ((g + 1) * per <= y) ++g;
    const int64_t r = y - g * per;
    int lo = 0, hi = s.items;                                    // cost(lo) <= r < cost(hi)
#pragma unroll 1
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq_cost(s, mid) <= r) lo = mid;
        else hi = mid;
    }
    k = lo;
    start = g * per + seq_cost(s, lo);
}
// Runs of equal length over the units: as many as there are CTAs; fewer when they
// would be short and every (sequence, kv head) has one.  The length is rounded up, so
// the last run may be shorter.
struct Runs {
    int64_t total, len;
    int count;
};
__device__ __forceinline__ Runs runs_of(const Params& p, int64_t total, int ctas) {
    Runs r;
    r.total = total;
    r.count = (int)min((int64_t)ctas, max(total / RUN_MIN, (int64_t)p.c.B * p.Hkv));
    r.len = __float2ll_ru(__fdiv_ru(__ll2float_ru(total), (float)r.count));
    return r;
}
__device__ __forceinline__ int64_t run_start(const Runs& r, int i) {
    return i < r.count ? min(i * r.len, r.total) : r.total;
}

// The bounded wait of tv_device.cuh with its slow path out of line (this kernel has
// some forty waits, and its instructions have to stay in the cache beside each
// other).  TRIES polls, each of which may suspend the warp, come before it: the
// waits of the products and of the softmax are on the critical path, and reading
// the clock costs more than a poll.
// The abort flag ends a wait early, but not one for the role's own copies or products (`own`).
// It lies in the 1,024 bytes that hold the barriers, so that its address needs no register.
constexpr uint32_t ABORT_AT = GQ * 64 + 4;
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, bool own) {
    const uint64_t t0 = globaltimer_ns();
#pragma unroll 1
    while (!mbar_try_wait(bar, parity)) {
        uint32_t late;
        asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(late) : "r"((smem_u32(bar) & ~1023u) + ABORT_AT));
        if ((late != 0 && !own) || globaltimer_ns() - t0 > TV_WAIT_NS) return false;
    }
    return true;
}
template <int TRIES = 1>
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, bool own = false) {
    bool ok = mbar_try_wait(bar, parity);
#pragma unroll 1
    for (int k = 1; k < TRIES && !ok; ++k) ok = mbar_try_wait(bar, parity);
    if (!ok) ok = wait_slow(bar, parity, own);
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void wait_own(uint64_t* bar, uint32_t parity) { wait_all(bar, parity, true); }

// The same for warp 8, which has nothing to spare: it polls, and leaves the loop only
// to look at the clock.
__device__ __forceinline__ bool wait_mma(uint64_t* bar, uint32_t parity) {
    bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
#pragma unroll 1
    for (int k = 0; k < 256 && !ok; ++k) ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
    return ok || wait_all(bar, parity);
}

// After a wait ran out, by one thread: the sequences with units in this CTA's run get
// TV_ERR_TIMEOUT, and the CTA's records their range, for the second kernel to repeat it (the
// first CTA of a sequence may write its TV_OK later).  The run is found again, so that nothing
// about it is kept in registers for this.
__device__ __noinline__ void report_late(const Params& p) {
    int64_t total = 0;
    for (int b = 0; b < p.c.B; ++b) {
        const int lo = p.c.q_start[b], hi = p.c.q_start[b + 1];
        if (lo < 0 || lo > hi || hi > p.c.T) return;       // (every sequence has its status)
        total += seq_units(p, p.c.prefix[b], hi - lo);
    }
    const Runs runs = runs_of(p, total, gridDim.x);
    const int64_t x_lo = run_start(runs, blockIdx.x), x_hi = run_start(runs, blockIdx.x + 1);
    int first = 0, last = -1;
    int64_t at = 0;
    for (int b = 0; b < p.c.B && at < x_hi; ++b) {
        const int64_t end = at + seq_units(p, p.c.prefix[b], p.c.q_start[b + 1] - p.c.q_start[b]);
        if (end > at && end > x_lo) {
            if (last < 0) first = b;
            last = b;
            p.status[b] = TV_ERR_TIMEOUT;
        }
        at = end;
    }
    p.rec[2 * blockIdx.x] = p.rec[2 * blockIdx.x + 1] = make_int4(first, last, 0, PIECE_LATE);
}

// S = Q K^T of one tile (M = N = 128), then a commit to `bar`: one elected lane of the
// converged warp issues all of it (an elect per instruction costs more than the
// instruction).  Descriptors advance 32 bytes per K = 16 step; the second half of the
// head is 16 KB on in Q and 1 KB on in K.
template <int D>
__device__ __forceinline__ void mma_s(uint32_t d, uint64_t a, uint64_t b, uint64_t* bar) {
    constexpr uint32_t IDESC = idesc_bf16(MT, KT, false);
    if constexpr (D == 128) {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 1024;\n\tadd.u64 b, %2, 64;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 1026;\n\tadd.u64 b, %2, 66;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 1028;\n\tadd.u64 b, %2, 68;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 1030;\n\tadd.u64 b, %2, 70;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(IDESC), "r"(smem_u32(bar))
            : "memory");
    } else {
        asm volatile(
            "{\n\t.reg .pred e, f, t;\n\t.reg .b64 a, b;\n\t"
            "elect.sync _|e, 0xffffffff;\n\t"
            "setp.ne.b32 f, 0, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, f;\n\t"
            "add.u64 a, %1, 2;\n\tadd.u64 b, %2, 2;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 4;\n\tadd.u64 b, %2, 4;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "add.u64 a, %1, 6;\n\tadd.u64 b, %2, 6;\n\t"
            "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
            "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%4];\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(IDESC), "r"(smem_u32(bar))
            : "memory");
    }
}
// O (+)= P V of one tile: P in tensor memory (8 columns per K = 16 step), V a page per step.
template <int D>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint64_t b, uint32_t accumulate) {
    constexpr uint32_t IDESC = idesc_bf16(MT, D, true);
    asm volatile(
        "{\n\t.reg .pred e, f, t;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.ne.b32 f, %4, 0;\n\tsetp.eq.b32 t, 0, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, f;\n\t"
        "add.u32 a, %1, 8;\n\tadd.u64 b, %2, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
        "add.u32 a, a, 8;\n\tadd.u64 b, b, %5;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(IDESC), "r"(accumulate), "n"(16 * D * 2 / 16)
        : "memory");
}

// Tiles of an item that warp 10 goes through: t < fa (some rows' windows start
// later) and t >= fb (some rows end earlier, or the tile reaches past hi).
__device__ __forceinline__ void item_edges(const Params& p, Item& it) {
    it.fb = (it.P + it.i0 + 1 - it.kbase) / KT;
    const int first_all = p.window > 0 ? it.P + it.i0 + it.ntok - p.window : 0;  // seen by every row
    it.fa = first_all > it.kbase ? (first_all - it.kbase + KT - 1) / KT : 0;
}
__device__ __forceinline__ int fix_index(const Item& it, int t) {  // 0 .. FIX_TILES - 1
    return t < it.fa ? t : max(it.fa, 0) + (t - max(it.fa, it.fb));
}

// Adds to O (tensor memory, this warp's lanes) the V rows that warp 10 took out
// although some rows attend to them: weight 2^(s - m), the score from global
// memory.  Rare (V rows with NaN or infinity), so out of line.  t0, step: the
// stream's tiles; first .. self: the lane's keys (none: self < first).
template <int D, bool CAP>
__device__ __noinline__ void add_noted(const Params& p, const Item& it, const uint32_t* notes, int t0,
                                       int step, uint32_t tO, int first, int self,
                                       const __nv_bfloat16* q, float m) {
#pragma unroll 1
    for (int t = t0; t < it.t_hi; t += step) {
        if (t >= it.fa && t < it.fb) continue;
#pragma unroll 1
        for (int e = 0; e < KT; ++e) {
            if (!((notes[fix_index(it, t) * 4 + (e >> 5)] >> (e & 31)) & 1u)) continue;
            const int key = it.kbase + t * KT + e;
            const int64_t blk = p.c.table[(int64_t)it.b * p.c.max_blocks + key / p.c.bs];
            const int64_t krow = ((blk * p.Hkv + it.g) * p.c.bs + key % p.c.bs) * D;
            const bool seen = key >= first && key <= self;
            float w = 0.f;
            if (seen) {
                float s = 0.f;
#pragma unroll 1
                for (int c = 0; c < D; ++c) s = fmaf(__bfloat162float(q[c]), __bfloat162float(p.k[krow + c]), s);
                s = CAP ? p.cap_log2 * tanhf(s * p.cap_x) : s * p.scale_log2;
                w = exp2f(s - m);
            }
            __syncwarp();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
                uint32_t r[16];
                tmem_ld16(tO + c, r);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float o = __uint_as_float(r[x]);
                    r[x] = __float_as_uint(seen ? fmaf(w, __bfloat162float(p.v[krow + c + x]), o) : o);
                }
                tmem_st16(tO + c, r);
                tmem_wait_st();
            }
        }
    }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(THREADS, 1)
chunk_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
    using L = Lay<D>;
    constexpr uint32_t TMEM_O = 256;                       // S at 0 and 128, O at 256 and 256 + D
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~uintptr_t(1023));
    Item* items = reinterpret_cast<Item*>(smem + L::OFF_ITEMS);
    uint32_t* bad = reinterpret_cast<uint32_t*>(smem + L::OFF_BAD);
    uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::OFF_BARS);
    uint64_t* empty = full + L::SLOTS;
    uint64_t* sfull = empty + L::SLOTS;   // [2] S(i, t) done (and all products before it)
    uint64_t* pfull = sfull + 2;          // [2] P(i, t) written
    uint64_t* ofull = pfull + 2;          // [2] the item's last PV(i) done
    uint64_t* ofree = ofull + 2;          // [2] O(i) read by the epilogue
    uint64_t* qfull = ofree + 2;
    uint64_t* qempty = qfull + 1;
    uint64_t* xdone = qempty + 1;         // an epilogue's use of the second Q tile is over
    uint64_t* drain = xdone + 1;
    uint64_t* gq_full = drain + 1;        // [GQ]
    uint64_t* gq_empty = gq_full + GQ;    // [GQ]
    uint64_t* vraw = gq_empty + GQ;       // [SLOTS] a V tile that warp 10 goes through has landed
    uint64_t* xall = vraw + L::SLOTS;     // [2] every softmax warp has written xo, has read xo
    auto* tmp = reinterpret_cast<ChunkLocateTmp<THREADS>*>(smem + L::OFF_RING);  // before the first copy
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::OFF_MISC);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::OFF_ITEMS + ABORT_AT);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t sbase = smem_u32(smem);
    if (tid == 0) {
        for (int s = 0; s < L::SLOTS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&vraw[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sfull[i], 1);
            mbar_init(&pfull[i], 4);
            mbar_init(&ofull[i], 1);
            mbar_init(&ofree[i], 4);
        }
        mbar_init(qfull, 1);
        mbar_init(qempty, 1);
        mbar_init(xdone, 1);
        mbar_init(drain, 1);
        mbar_init(&xall[0], 8);
        mbar_init(&xall[1], 8);
        for (int s = 0; s < GQ; ++s) {
            mbar_init(&gq_full[s], 1);
            mbar_init(&gq_empty[s], 11);  // 8 softmax warps, MMA, producer, warp 10
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == MMA_WARP) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    {
        // rows of a Q tile past npt * G are never loaded: zero, so that their scores are finite
        const int used = p.npt * p.G;
        for (int e = tid; e < 2 * L::HALVES * (MT - used) * 8; e += THREADS) {
            const int t = e / ((MT - used) * 8), r = e % ((MT - used) * 8);
            *reinterpret_cast<uint4*>(smem + L::OFF_Q + t * (MT * 128) + used * 128 + r * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
    pdl_wait();  // everything above touched only shared memory and tensor memory
    pdl_launch_dependents();

    // ---- this CTA's run
    Runs runs;
    int64_t x_lo = 0, x_hi = 0;
    auto where = [&](int64_t total) {
        runs = runs_of(p, total, gridDim.x);
        x_lo = run_start(runs, blockIdx.x);
        x_hi = run_start(runs, blockIdx.x + 1);
        return x_lo < x_hi ? x_lo : total;
    };
    auto units = [&](int P, int n) { return seq_units(p, P, n); };
    const ChunkPlace at = p.c.B <= 32 ? chunk_locate_warp(p.c, where, units)
                                      : chunk_locate<THREADS>(tmp, p.c, where, units);
    if (blockIdx.x == 0)
        for (int b = tid; b < p.c.B; b += THREADS)
            if (!at.valid || p.c.q_start[b] == p.c.q_start[b + 1])
                p.status[b] = (at.valid && chunk_shape_ok(p.c, p.c.prefix[b], 0)) ? TV_OK : TV_ERR_OUT_OF_RANGE;
    Seq s0{};
    bool ok0 = false;
    if (at.b < p.c.B) {
        // the first sequence's blocks, by every thread at once
        s0 = seq_of(p, at.P, at.n);
        ok0 = s0.shape && chunk_blocks_ok(p.c, at.b, chunk_first_key(s0.P, p.window), (int64_t)s0.P + s0.n, tid, THREADS);
    }
    fence_proxy_async_smem();  // the ring's first bytes held the search's scratch
    ok0 = __syncthreads_and(ok0 ? 1 : 0) != 0;

    // (test-only: this warp's first wait for work counts as run out)
    bool alive = !(p.late.warp == warp && (p.late.cta < 0 || p.late.cta == (int)blockIdx.x));
    // Work item k, from the queue; false at the end, or (alive false) after a timeout.
    auto take = [&](uint32_t k, Item& it) -> bool {
        const int s = k % GQ;
        alive = wait_all(&gq_full[s], (k / GQ) & 1u);
        const int4* src = reinterpret_cast<const int4*>(&items[s]);
        int4* dst = reinterpret_cast<int4*>(&it);
#pragma unroll
        for (int u = 0; u < 4; ++u) dst[u] = lds_v4_volatile(src + u);
        __syncwarp();
        // "slot read": no release needed, and a release would wait for the epilogue's stores
        if (lane == 0) remote_arrive_relaxed_after(&gq_empty[s], 0, it.b | it.row0 | it.t_lo | it.n);
        return alive && !(it.flags & ITEM_END);
    };

    if (warp == SCHED_WARP) {
        // ============================== scheduler ==============================
        uint32_t k = 0;
        // the slots' records: empty until a piece is published
        int4 rec0 = make_int4(0, 0, 0, 0), rec1 = rec0;
        auto publish = [&](const Item& it) -> bool {
            const int s = k % GQ;
            if (!wait_all(&gq_empty[s], ((k / GQ) & 1u) ^ 1u)) return false;
            if (lane == 0) {
                const int4* src = reinterpret_cast<const int4*>(&it);
#pragma unroll
                for (int u = 0; u < 4; ++u) reinterpret_cast<int4*>(&items[s])[u] = src[u];
                mbar_arrive(&gq_full[s]);
            }
            __syncwarp();
            ++k;
            return true;
        };
        if (alive && at.b < p.c.B) {
            int b = at.b, g, qk;
            Seq s = s0;
            bool ok = ok0;
            int row = at.row;
            int64_t start, x = x_lo;
            item_at(p, s, x_lo - at.base, g, qk, start);
            start += at.base;
#pragma unroll 1
            while (true) {
                Item it;
                int i1, tiles;
                const int64_t cost = item_cost(s, qk);
                item_keys(p, s, qk, it.i0, i1, it.kbase, it.hi, tiles);
                it.t_lo = cut_tile(x - start, cost, tiles);
                it.t_hi = cut_tile(min(x_hi - start, cost), cost, tiles);
                // a sequence that does not fit has items without tiles: the run with the first
                // unit writes them
                if (tiles == 0 ? x == start : it.t_lo < it.t_hi) {
                    const bool whole = it.t_lo == 0 && it.t_hi == tiles;
                    it.b = b;
                    it.g = g;
                    it.P = s.P;
                    it.ntok = i1 - it.i0;
                    it.row0 = row + it.i0;
                    it.slot = whole ? -1 : 2 * (int)blockIdx.x + (it.t_lo == 0 ? 1 : 0);
                    it.n = ok ? it.t_hi - it.t_lo : 0;
                    it.flags = (it.ntok > p.npt ? ITEM_TWO : 0) | (ok ? 0 : ITEM_BAD) |
                               (g == 0 && it.i0 == 0 && it.t_lo == 0 ? ITEM_STATUS : 0);
                    it.pad = 0;
                    item_edges(p, it);
                    if (!whole) {
                        const int4 rec = make_int4(it.row0, it.ntok, g, PIECE | (it.t_hi == tiles ? PIECE_LAST : 0));
                        if (it.t_lo == 0) rec1 = rec;
                        else rec0 = rec;
                    }
                    alive = publish(it);
                }
                start += cost;
                x = start;
                if (!alive || x >= x_hi) break;
                if (++qk < s.items) continue;
                qk = 0;
                if (++g < p.Hkv) continue;
                g = 0;
                // the next sequence with rows: there is one, since x < x_hi
                int n = 0;
                do {
                    ++b;
                    row = p.c.q_start[b];
                    n = p.c.q_start[b + 1] - row;
                } while (n == 0 && b + 1 < p.c.B);
                s = seq_of(p, p.c.prefix[b], n);
                ok = s.shape && chunk_blocks_ok(p.c, b, chunk_first_key(s.P, p.window),
                                                (int64_t)s.P + s.n, lane, 32);
                ok = __all_sync(0xffffffffu, ok);
            }
        }
        if (lane == 0) {
            p.rec[2 * blockIdx.x] = rec0;
            p.rec[2 * blockIdx.x + 1] = rec1;
        }
        if (alive) {
            Item it{};
            it.flags = ITEM_END;
            alive = publish(it);
        }
        if (!alive && lane == 0) *abort_flag = 1;
    } else if (warp == LOAD_WARP) {
        // ============================ K/V producer ============================
        if (lane == 0) {
            tma_prefetch_desc(&kmap);
            tma_prefetch_desc(&vmap);
        }
        uint32_t ld = 0, slot = 0, ph = 0; // slots filled so far; the next one, its round's parity
        uint32_t raw = 0, raw_ph = 0;      // per slot: last filled through vraw, and vraw's next parity
        Item it;
        for (uint32_t k = 0; alive && take(k, it); ++k) {
            if (it.n == 0) continue;
            const bool two = (it.flags & ITEM_TWO) != 0;
            // K/V of one token's rows are read once; longer chunks come back to them
            const uint64_t policy = it.ntok == 1 ? l2_policy_evict_first() : l2_policy_evict_normal();
            // cache rows of the pages, 32 (four tiles) per window: lane l holds page l.  K runs
            // at most two tiles ahead of V, so two windows are enough; the block ids of the
            // window after are loaded early.
            constexpr int WT = 32 / (KT / 16);
            const int32_t* table = p.c.table + (int64_t)it.b * p.c.max_blocks;
            int nxt_blk = 0, nxt_off = 0;
            auto fetch = [&](int w) {
                const int key = it.kbase + (it.t_lo + w * WT) * KT + lane * 16;
                nxt_blk = key < it.hi ? __ldg(table + key / p.c.bs) : 0;
                nxt_off = key % p.c.bs;
            };
            auto rows = [&]() -> int { return (nxt_blk * p.Hkv + it.g) * p.c.bs + nxt_off; };
            fetch(0);
            int cur = rows(), prev = 0, wk = 0;
            if (it.n > WT) fetch(1);
            // the order in which the products take them: V(x / 2 - lag), K(x / 2)
            const int lag = two ? 1 : 2;
#pragma unroll 1
            for (int x = 0; x < 2 * (it.n + lag); ++x) {
                const bool is_v = (x & 1) == 0;
                const int j = (x >> 1) - (is_v ? lag : 0);        // tile of the piece
                if (j < 0 || j >= it.n) continue;
                // everything but the copies comes before the wait for the slot
                const int w = j / WT;
                if (!is_v && w > wk) {
                    prev = cur;
                    cur = rows();
                    wk = w;
                    if (it.n > (w + 1) * WT) fetch(w + 1);
                }
                const int t = it.t_lo + j;
                const int pages = min(KT / 16, (it.hi - it.kbase - t * KT + 15) >> 4);
                const int y = __shfl_sync(0xffffffffu, w == wk ? cur : prev, (j % WT) * (KT / 16) + (lane & 7));
                uint8_t* dst = smem + L::OFF_RING + slot * L::SLOT_BYTES + (lane & 7) * L::PAGE_BYTES;
                // a V tile at the edges goes through warp 10, which passes it on
                const uint32_t edge = is_v && (t < it.fa || t >= it.fb) ? 1u : 0u;
                uint64_t* bar = edge ? &vraw[slot] : &full[slot];
                alive = wait_all<64>(&empty[slot], ph ^ 1u);
                if (!alive) break;
                raw = (raw & ~(1u << slot)) | (edge << slot);
                raw_ph ^= edge << slot;
                mbar_arrive_expect_tx_relaxed_elect(bar, (uint32_t)pages * L::PAGE_BYTES);
                if (lane < pages) {
                    if constexpr (D == 128) {
                        if (is_v) tma_load_3d_hint(dst, &vmap, bar, 0, y, 0, policy);
                        else tma_load_4d_hint(dst, &kmap, bar, 0, 0, 0, y >> 3, policy);
                    } else {
                        tma_load_2d(dst, is_v ? &vmap : &kmap, bar, 0, y, policy);
                    }
                }
                __syncwarp();
                ++ld;
                if (++slot == L::SLOTS) {
                    slot = 0;
                    ph ^= 1u;
                }
            }
        }
        if (!alive && lane == 0) *abort_flag = 1;
        // copies in flight end before the CTA does
        for (uint32_t u = ld > (uint32_t)L::SLOTS ? ld - L::SLOTS : 0; u < ld; ++u) {
            const uint32_t s = u % L::SLOTS;
            if ((raw >> s) & 1u) wait_own(&vraw[s], ((raw_ph >> s) & 1u) ^ 1u);
            else wait_own(&full[s], (u / L::SLOTS) & 1u);
        }
    } else if (warp == MMA_WARP) {
        // ============================== products ==============================
        uint32_t slot = 0, par = 0;                    // next ring position: slot, parity of its round
        uint32_t qi = 0, ppar = 0, opar = 3;           // ppar, opar: parity bit per stream
        Item it;
        const uint32_t ring = sbase + L::OFF_RING;
        const uint64_t qd = smem_desc_sw128(sbase + L::OFF_Q, 16, 1024);
        // d = 128: K is [page][row group][half][8 rows][128 bytes], 8-key groups 2 KB apart;
        // V is [page][half][16 rows][128 bytes]
        const uint64_t kd = smem_desc_sw128(ring, 16, D == 128 ? 2048 : 1024), vd = smem_desc_sw128(ring, 2048, 1024);
        auto next = [&](uint32_t& s, uint32_t& ph) {
            if (++s == L::SLOTS) {
                s = 0;
                ph ^= 1u;
            }
        };
        auto issue_s = [&](int i, int qt, uint32_t s) {
            mma_s<D>(tmem + i * KT, qd + qt * (L::Q_BYTES / 16), kd + s * (L::SLOT_BYTES / 16), &sfull[i]);
        };
        auto issue_pv = [&](int i, uint32_t s, bool first) {
            mma_pv<D>(tmem + TMEM_O + i * D, tmem + i * KT, vd + s * (L::SLOT_BYTES / 16), first ? 0u : 1u);
        };
        // P of stream i is there, and (first product of an item) O(i) has been read
        auto wait_p = [&](int i, bool first) -> bool {
            bool ok = wait_mma(&pfull[i], (ppar >> i) & 1u);
            if (first) {
                ok = ok && wait_mma(&ofree[i], (opar >> i) & 1u);
                opar ^= 1u << i;
            }
            ppar ^= 1u << i;
            tc_fence_after();
            return ok;
        };
#pragma unroll 1
        for (uint32_t k = 0; alive && take(k, it); ++k) {
            if (it.n == 0) continue;
            const int n = it.n;
            alive = wait_mma(qfull, qi & 1u);
            ++qi;
            if (it.flags & ITEM_TWO) {
                // ring order K(0) V(0) K(1) V(1) ...; both streams read every tile
                alive = alive && wait_mma(&full[slot], par);
                if (!alive) break;
                tc_fence_after();
                issue_s(0, 0, slot);
                issue_s(1, 1, slot);
                tc_commit_elect(&empty[slot]);
                if (n == 1) tc_commit_elect(qempty);
#pragma unroll 1
                for (int j = 1; j <= n; ++j) {
                    next(slot, par);
                    const uint32_t vs = slot;
                    alive = wait_mma(&full[vs], par);              // V(j - 1)
                    if (j < n) {
                        next(slot, par);
                        alive = alive && wait_mma(&full[slot], par);   // K(j)
                    }
                    alive = alive && wait_p(0, j == 1);
                    if (!alive) break;
                    issue_pv(0, vs, j == 1);
                    if (j < n) issue_s(0, 0, slot);
                    else tc_commit_elect(&ofull[0]);
                    alive = wait_p(1, j == 1);
                    if (!alive) break;
                    issue_pv(1, vs, j == 1);
                    if (j < n) {
                        issue_s(1, 1, slot);
                        tc_commit_elect(&empty[vs]);
                        tc_commit_elect(&empty[slot]);
                        if (j == n - 1) tc_commit_elect(qempty);
                    } else {
                        tc_commit_elect(&ofull[1]);
                        tc_commit_elect(&empty[vs]);
                    }
                }
                next(slot, par);
            } else {
                // ring order K(0) K(1) V(0) K(2) V(1) ... V(n - 1); stream j % 2 reads tile j
#pragma unroll 1
                for (int j = 0; j < n + 2; ++j) {
                    const int i = j & 1;
                    if (j >= 2 && j - 2 < n) {
                        alive = wait_mma(&full[slot], par) && wait_p(i, j < 4);
                        if (!alive) break;
                        issue_pv(i, slot, j < 4);
                        tc_commit_elect(&empty[slot]);
                        if (j >= n) tc_commit_elect(&ofull[i]);
                        next(slot, par);
                    }
                    if (j < n) {
                        alive = wait_mma(&full[slot], par);
                        if (!alive) break;
                        tc_fence_after();
                        issue_s(i, 0, slot);
                        tc_commit_elect(&empty[slot]);
                        if (j == n - 1) tc_commit_elect(qempty);
                        next(slot, par);
                    }
                }
            }
        }
        if (!alive && lane == 0) *abort_flag = 1;
        // products in flight end before the tensor memory is freed
        tc_commit_elect(drain);
        wait_own(drain, 0);
    } else if (warp == FIX_WARP) {
        // ==================== Q tiles, V rows that must not reach O ====================
        if (lane == 0) tma_prefetch_desc(&qmap);
        const uint64_t qpol = l2_policy_evict_first();
        uint32_t ld = 0, qi = 0, xi = 0, ph = 0;             // ph: vraw's parity per slot
        Item it;
        for (uint32_t k = 0; alive && take(k, it); ++k) {
            if (it.n == 0) continue;
            const int n = it.n;
            const bool two = (it.flags & ITEM_TWO) != 0;
            alive = wait_all(qempty, (qi & 1u) ^ 1u);
            // the second Q tile also serves the epilogues of single row tiles before
            if (alive && two && xi > 0) alive = wait_all(xdone, (xi - 1) & 1u);
            if (!alive) break;
            ++qi;
            const int nq = two ? 2 : 1;
            mbar_arrive_expect_tx_relaxed_elect(qfull, (uint32_t)(nq * L::HALVES * 128 * p.G * p.npt));
            for (int t = 0; t < nq; ++t)
                for (int hf = 0; hf < L::HALVES; ++hf)
                    tma_load_3d_elect(smem + L::OFF_Q + t * L::Q_BYTES + hf * (MT * 128), &qmap, qfull, hf * 64,
                                      it.g * p.G, it.row0 + t * p.npt, qpol);
            if (!two) {
                // one use outstanding at most, or the barrier's phases could not be told apart
                if (xi > 0) alive = wait_all(xdone, (xi - 1) & 1u);
                if (!alive) break;
                ++xi;
            }
            // ring position of V(j): two row tiles K0 V0 K1 V1 ..., one K0 K1 V0 K2 V1 ... V(n-1)
            auto v_at = [&](int j) -> uint32_t { return ld + (two || j == n - 1 ? 2 * j + 1 : 2 * j + 2); };
            // notes of live item qi - 1: its Q buffer is free, so every S of the item before is done,
            // and with it the epilogue of the item three before
            uint32_t* notes = bad + ((qi - 1) % FIX_BUFS) * FIX_TILES * 4;
            for (int e = lane; e < FIX_TILES * 4; e += 32) notes[e] = 0u;
            __syncwarp();
            for (int j = 0; alive && j < n; ++j) {
                const int t = it.t_lo + j;
                if (t >= it.fa && t < it.fb) {
                    j = min(n, it.fb - it.t_lo) - 1;       // on to the tiles at the far end
                    continue;
                }
                // (a slot is filled through vraw again only after its tile was passed on and used)
                const uint32_t slot = v_at(j) % L::SLOTS;
                alive = wait_all(&vraw[slot], (ph >> slot) & 1u);
                if (!alive) break;
                ph ^= 1u << slot;
                uint8_t* vt = smem + L::OFF_RING + slot * L::SLOT_BYTES;
                const int nv = it.hi - (it.kbase + t * KT);          // keys the item has in this tile
                // rows before the first token's window, in the first page
                const int lead = chunk_first_key(it.P + it.i0, p.window) - (it.kbase + t * KT);
                // one token: no key is seen by some of its rows only
                const int scan = it.ntok > 1 ? min(nv, KT) : 0;
#pragma unroll 1
                for (int q = 0; q < KT / 32; ++q) {
                    const int r = q * 32 + lane;
                    uint8_t* row = vt + (r >> 4) * L::PAGE_BYTES + (r & 15) * 128;
                    bool clear = r >= nv || r < lead, odd = false;
                    if (r < scan && !clear) {
                        // bfloat16 with all exponent bits set, two per word
                        uint32_t acc = 0;
#pragma unroll
                        for (int hf = 0; hf < L::HALVES; ++hf)
#pragma unroll
                            for (int c = 0; c < 8; ++c) {
                                const uint4 x = *reinterpret_cast<const uint4*>(row + hf * 2048 + ((c ^ (lane & 7)) << 4));
                                acc |= ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                                       ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
                            }
                        odd = (acc & 0x80008000u) != 0;
                        clear = odd;
                    }
                    const uint32_t m = __ballot_sync(0xffffffffu, odd);
                    if (m != 0 && lane == 0) notes[fix_index(it, t) * 4 + q] = m;
                    if (clear)
#pragma unroll
                        for (int hf = 0; hf < L::HALVES; ++hf)
#pragma unroll
                            for (int c = 0; c < 8; ++c)
                                *reinterpret_cast<uint4*>(row + hf * 2048 + ((c ^ (lane & 7)) << 4)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();  // the tensor core reads V through the async proxy
                __syncwarp();
                if (lane == 0) mbar_arrive(&full[slot]);
            }
            ld += 2 * n;
        }
        if (!alive && lane == 0) *abort_flag = 1;
        if (qi > 0) wait_own(qfull, (qi - 1) & 1u);          // its own copies in flight
    } else {
        // ============================== softmax ==============================
        const int i = warp >> 2;                              // stream
        const int row = tid & 127;                            // tensor-memory lane
        const uint32_t lane_off = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tS = tmem + lane_off + i * KT, tO = tmem + lane_off + TMEM_O + i * D;
        float* xo = reinterpret_cast<float*>(smem + L::OFF_X);  // [columns][rows]
        float* ml = reinterpret_cast<float*>(smem + L::OFF_ML);
        uint32_t sc = 0, oc = 0, live = 0, xc = 0;
        // every softmax warp has written xo (0), has read it (1): with a bounded wait, unlike
        // bar.sync
        auto all_x = [&](int which) {
            __syncwarp();
            if (lane == 0) {
                if (which == 0) mbar_arrive(&xall[0]);
                else mbar_arrive_relaxed(&xall[1]);   // reads only: nothing to release
            }
            alive = alive && wait_all(&xall[which], xc & 1u);
            xc += which;
        };
        for (uint32_t k = 0; alive; ++k) {
            // the item stays in its slot, which is given back at its end: its fields in registers
            // would be spilled beside the scores, and L1 is too small to hold what is spilled
            const Item& it = items[k % GQ];
            alive = wait_all(&gq_full[k % GQ], (k / GQ) & 1u);
            if (!alive || (it.flags & ITEM_END)) break;
            const bool two = (it.flags & ITEM_TWO) != 0;
            const int n = it.n, ja = it.fa - it.t_lo, jb = it.fb - it.t_lo;
            if ((it.flags & ITEM_STATUS) && tid == 0)
                p.status[it.b] = (it.flags & ITEM_BAD) ? TV_ERR_OUT_OF_RANGE : TV_OK;
            int row_ = row;
            asm volatile("" : "+r"(row_));                  // (per item, not kept over the tiles)
            const int tok_l = row_ / p.G, head = row_ - tok_l * p.G;
            const int tok = tok_l + (two ? i * p.npt : 0);    // token within the item
            const bool mine = tok_l < p.npt && tok < it.ntok;
            // keys of the row, from the first key of the piece's tiles on
            const int self = it.P + it.i0 + min(tok, it.ntok - 1);
            const int first = p.window > 0 ? max(0, self - p.window + 1) : 0;
            const int step = two ? 1 : 2, j0 = two ? 0 : i;
            const bool have = n > j0;                      // O(i) will hold this item
            const int rows = p.G * min(it.ntok, p.npt);       // rows of the item in a row tile
            const bool wrows = (warp & 3) * 32 < rows;        // some of them in this warp
            // (a bad sequence has no tiles: 0 / 1.  A row whose every score is -infinity ends as 0 / 0.)
            float m_used = n > 0 ? -INFINITY : 0.f, l = n > 0 ? 0.f : 1.f;
            for (int j = j0; j < n; j += step) {
                if (!wait_all<64>(&sfull[i], sc & 1u)) {
                    alive = false;
                    break;
                }
                ++sc;
                tc_fence_after();
                if (!wrows) {
                    // nothing of the item in this warp: its rows of P may hold anything (a row of
                    // the product reads its own row of P only)
                    if (lane == 0) mbar_arrive_relaxed(&pfull[i]);
                    continue;
                }
                float sv[KT];
                auto load_s = [&]() {
                    uint32_t r[KT / 32][32];
#pragma unroll
                    for (int c = 0; c < KT / 32; ++c) tmem_ld32(tS + c * 32, r[c]);
                    tmem_wait_ld();
#pragma unroll
                    for (int c = 0; c < KT; ++c) sv[c] = __uint_as_float(r[c / 32][c % 32]);
                };
                load_s();
                if constexpr (CAP) {
                    // cap tanh(scale s / cap), in units of log 2.  An exponential and a reciprocal
                    // more per score would bind on the special function unit, so arguments up to
                    // 0.35 take a polynomial, two scores per instruction; S is read again where it
                    // turns out that one of the warp's is larger.
                    float big[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < KT; c += 2) {
                        const uint64_t x = f2_pack(sv[c], sv[c + 1]), u = f2_mul(x, x);
                        uint64_t y = f2_pack(p.cap_c[2], p.cap_c[2]);
#pragma unroll
                        for (int e = 1; e >= 0; --e) y = f2_fma(y, u, f2_pack(p.cap_c[e], p.cap_c[e]));
                        f2_unpack(f2_mul(x, y), sv[c], sv[c + 1]);
                        float ua, ub;
                        f2_unpack(u, ua, ub);
                        big[(c >> 1) & 3] = fmax3(big[(c >> 1) & 3], ua, ub);
                    }
                    if (__any_sync(0xffffffffu, mine && !(fmaxf(fmax3(big[0], big[1], big[2]), big[3]) < p.cap_small))) {
                        // cap (1 - 2 / (1 + e^(2x))) for those that are, in place and rolled: the
                        // instruction cache is for the other path
#pragma unroll 1
                        for (int c = 0; c < KT; c += 16) {
                            uint32_t r[16];
                            tmem_ld16(tS + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float x = __uint_as_float(r[e]), u = x * x;
                                const float w = ex2_approx(x * p.scale_log2);
                                const float y = fmaf(-2.f * p.cap_log2, rcp_approx(1.f + w), p.cap_log2);
                                r[e] = __float_as_uint(
                                    u < p.cap_small ? x * fmaf(fmaf(p.cap_c[2], u, p.cap_c[1]), u, p.cap_c[0]) : y);
                            }
                            tmem_st16(tS + c, r);
                        }
                        tmem_wait_st();
                        load_s();
                    }
                }
                if (j < ja || j >= jb) {
                    // visible keys of the tile: bits a .. z, a word for 32 columns
                    const int k0 = it.kbase + (it.t_lo + j) * KT;
                    const int a = first - k0, z = self - k0;
#pragma unroll
                    for (int h = 0; h < KT; h += 32) {
                        const int lo = min(max(a - h, 0), 32), hi = min(max(z - h + 1, 0), 32);
                        const uint32_t vis = hi > lo ? (0xffffffffu >> (32 - (hi - lo))) << lo : 0u;
#pragma unroll
                        for (int c = 0; c < 32; ++c) sv[h + c] = ((vis >> c) & 1u) ? sv[h + c] : -INFINITY;
                    }
                }
                const float csc = CAP ? 1.f : p.scale_log2;
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int c = 0; c < KT; c += 8)
#pragma unroll
                    for (int u = 0; u < 4; ++u) mx[u] = fmax3(mx[u], sv[c + u], sv[c + 4 + u]);
                const float tmax = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * csc;
                const bool need = (m_used == -INFINITY) ? (tmax > -INFINITY) : (tmax > m_used + RESCALE_LOG2);
                if (__any_sync(0xffffffffu, need)) {
                    const float f = (need && m_used > -INFINITY) ? exp2f(m_used - tmax) : 1.f;
                    if (j > j0) {
                        // O holds every product before this S: rescale it
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t r[16];
                            tmem_ld16(tO + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                            tmem_st16(tO + c, r);
                        }
                        // (the wait below covers these stores too)
                    }
                    l *= f;
                    if (need) m_used = tmax;
                }
                const float nbase = (m_used == -INFINITY) ? 0.f : -m_used;
                const uint64_t sc2 = f2_pack(csc, csc), nb2 = f2_pack(nbase, nbase);
                uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                for (int h = 0; h < KT; h += 64) {
                    uint32_t pk[32];
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        float xa, xb;
                        f2_unpack(f2_fma(f2_pack(sv[h + c], sv[h + c + 1]), sc2, nb2), xa, xb);
                        const float a = ex2_approx(xa), b2 = ex2_approx(xb);
                        acc[(c >> 1) & 3] = f2_add(acc[(c >> 1) & 3], f2_pack(a, b2));
                        // weights to bfloat16, the products' input type: at most 2^-8 of each
                        pk[c / 2] = pack_bf16x2(a, b2);
                    }
                    tmem_st32(tS + h / 2, pk);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(&pfull[i]);
                float lo, hi;
                f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), lo, hi);
                l += lo + hi;
            }
            if (!alive) break;
            // ---- epilogue.  Two streams of one row tile are joined: weights 2^(m_i - max).
            const bool join = !two && it.n > 1;
            // partial result: [D / 4][rows] x 4 columns, then the maxima and the sums
            float* pslot = it.slot >= 0 ? p.part + (int64_t)it.slot * p.prows * (D + 2) : nullptr;
            const uint32_t* notes = bad + (live % FIX_BUFS) * FIX_TILES * 4;
            if (it.n > 0) ++live;
            if (have) {
                if (!wait_all(&ofull[i], (oc++) & 1u)) {
                    alive = false;
                    break;
                }
                tc_fence_after();
                // V rows that warp 10 took out although some rows attend to them
                if (it.ntok > 1 && (it.fa > it.t_lo || it.fb < it.t_hi) &&
                    __any_sync(0xffffffffu, lane < FIX_TILES * 4 && notes[lane] != 0u))
                    add_noted<D, CAP>(p, it, notes, it.t_lo + j0, step, tO, first, mine ? self : -1,
                                      p.q + (int64_t)(it.row0 + tok) * p.q_stride + (int64_t)(it.g * p.G + head) * D,
                                      m_used);
            }
            auto o_read = [&]() {                             // O may be overwritten by the next item
                if (!have) return;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_relaxed(&ofree[i]);
            };
            if (!two && rows <= FEW) {
                // few rows: both streams leave theirs in shared memory, then all 256 threads join
                // and write 8 columns each
                constexpr int PITCH = D + 4;
                if (wrows && have) {
                    float* xr = xo + (i * FEW + row) * PITCH;
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t r[16];
                        tmem_ld16(tO + c, r);
                        tmem_wait_ld();
                        if (row < rows)
#pragma unroll
                            for (int e = 0; e < 16; e += 4)
                                *reinterpret_cast<uint4*>(xr + c + e) = make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
                    }
                }
                o_read();
                if (wrows) {
                    ml[i * 64 + row] = m_used;
                    ml[i * 64 + 32 + row] = l;
                }
                all_x(0);
#pragma unroll 1
                for (int e = tid; e < rows * (D / 8); e += 256) {
                    const int r = e / (D / 8), c = e % (D / 8) * 8;
                    float m = ml[r], sum = ml[32 + r], w0 = 1.f, w1 = 0.f;
                    float f[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) f[x] = it.n > 0 ? xo[r * PITCH + c + x] : 0.f;
                    if (join) {
                        const float m1 = ml[64 + r], mm = fmaxf(m, m1), bz = mm == -INFINITY ? 0.f : mm;
                        w0 = exp2f(m - bz);
                        w1 = exp2f(m1 - bz);
                        sum = w0 * sum + w1 * ml[96 + r];
                        m = mm;
#pragma unroll
                        for (int x = 0; x < 8; ++x) f[x] = fmaf(w1, xo[(FEW + r) * PITCH + c + x], w0 * f[x]);
                    }
                    if (pslot) {
                        float4* dst = reinterpret_cast<float4*>(pslot) + c / 4 * p.prows + r;
                        dst[0] = make_float4(f[0], f[1], f[2], f[3]);
                        dst[p.prows] = make_float4(f[4], f[5], f[6], f[7]);
                        if (c == 0) {
                            pslot[p.prows * D + r] = m;
                            pslot[p.prows * (D + 1) + r] = sum;
                        }
                    } else {
                        const float inv = 1.f / sum;
                        const int t = r / p.G;
                        uint4 v;
                        v.x = pack_bf16x2(f[0] * inv, f[1] * inv);
                        v.y = pack_bf16x2(f[2] * inv, f[3] * inv);
                        v.z = pack_bf16x2(f[4] * inv, f[5] * inv);
                        v.w = pack_bf16x2(f[6] * inv, f[7] * inv);
                        *reinterpret_cast<uint4*>(p.out + (int64_t)(it.row0 + t) * p.o_stride +
                                                  (int64_t)(it.g * p.G + r - t * p.G) * D + c) = v;
                    }
                }
                fence_proxy_async_smem();  // the next Q tile may land where xo was
                all_x(1);
            } else {
                // a thread per row; stream 1 of a single row tile hands its rows over, 32 columns at
                // a time (xo: [column][row])
                const int prow = (two ? i * MT : 0) + row;
                const bool writes = (two || i == 0) && wrows;
                // Four lanes exchange their rows' 16-byte pieces, so that they write 64 bytes of one
                // row together: a store of 16 bytes of 32 rows takes 32 cycles, of 64 bytes of 8 rows 8.
                const uint64_t orow = reinterpret_cast<uint64_t>(p.out + (int64_t)(it.row0 + tok) * p.o_stride +
                                                                 (int64_t)(it.g * p.G + head) * D + (lane & 3) * 8);
                uint64_t prow4[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) prow4[x] = __shfl_sync(0xffffffffu, orow, (lane & ~3) + x) + 16 * ((lane & 3) - x);
                const uint32_t valid = __ballot_sync(0xffffffffu, mine) >> (lane & ~3);
                float w0 = 1.f, w1 = 0.f, inv = 0.f;
#pragma unroll 1
                for (int c = 0; c < D; c += 32) {
                    uint32_t r[32];
                    if (join) {
                        if (i == 1 && wrows) {
                            if (c == 0) {
                                ml[row] = m_used;
                                ml[MT + row] = l;
                            }
                            tmem_ld32(tO + c, r);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) xo[e * MT + row] = __uint_as_float(r[e]);
                        }
                        all_x(0);
                    }
                    if (writes) {
                        if (c == 0) {
                            if (join) {
                                const float m1 = ml[row], l1 = ml[MT + row];
                                const float mm = fmaxf(m_used, m1), bz = mm == -INFINITY ? 0.f : mm;
                                w0 = exp2f(m_used - bz);
                                w1 = exp2f(m1 - bz);
                                l = w0 * l + w1 * l1;
                                m_used = mm;
                            }
                            inv = 1.f / l;
                            if (mine && pslot) {
                                pslot[p.prows * D + prow] = m_used;
                                pslot[p.prows * (D + 1) + prow] = l;
                            }
                        }
                        if (have) {
                            tmem_ld32(tO + c, r);
                            tmem_wait_ld();
                        } else {
#pragma unroll
                            for (int e = 0; e < 32; ++e) r[e] = 0u;
                        }
                        if (join)
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                r[e] = __float_as_uint(fmaf(w1, xo[e * MT + row], w0 * __uint_as_float(r[e])));
                        if (pslot) {
                            if (mine)
#pragma unroll
                                for (int e = 0; e < 32; e += 4)
                                    reinterpret_cast<uint4*>(pslot)[(c + e) / 4 * p.prows + prow] =
                                        make_uint4(r[e], r[e + 1], r[e + 2], r[e + 3]);
                        } else {
                            uint32_t u[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                u[e] = pack_bf16x2(__uint_as_float(r[2 * e]) * inv, __uint_as_float(r[2 * e + 1]) * inv);
                            // 4 x 4 transpose of 16-byte pieces over four lanes
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if ((e & 4) == 0) {
                                    const uint32_t y = __shfl_xor_sync(0xffffffffu, (lane & 1) ? u[e] : u[e + 4], 1);
                                    if (lane & 1) u[e] = y;
                                    else u[e + 4] = y;
                                }
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint32_t y = __shfl_xor_sync(0xffffffffu, (lane & 2) ? u[e] : u[e + 8], 2);
                                if (lane & 2) u[e] = y;
                                else u[e + 8] = y;
                            }
#pragma unroll
                            for (int x = 0; x < 4; ++x)
                                if ((valid >> x) & 1u)
                                    *reinterpret_cast<uint4*>(prow4[x] + 2 * c) =
                                        make_uint4(u[4 * x], u[4 * x + 1], u[4 * x + 2], u[4 * x + 3]);
                        }
                    }
                    if (join) {
                        fence_proxy_async_smem();
                        all_x(1);
                    }
                }
                o_read();
            }
            if (!two && it.n > 0 && tid == 0) mbar_arrive(xdone);
            __syncwarp();
            if (lane == 0) remote_arrive_relaxed_after(&gq_empty[k % GQ], 0, it.b);
        }
        if (!alive && lane == 0) *abort_flag = 1;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == MMA_WARP) tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort_flag != 0) report_late(p);
}

// Joins the pieces of the items that run borders cut: the CTA of slot 2 r + 1 (an item
// that starts in run r and goes on) and 32 columns.  The pieces that follow are in the
// slots 2 (r + 1), 2 (r + 2), ... up to the last one; weights 2^(m_k - max) on the
// unnormalised rows, in run order.  A run with a wait that ran out: its sequences' statuses,
// again; an item that it cut gives zeros.
constexpr int JOIN_THREADS = 256;

template <int D>
__global__ void __launch_bounds__(JOIN_THREADS)
chunk_tc_join_kernel(const __grid_constant__ Params p, int ctas) {
    const int row = threadIdx.x, t = row / MT, tok_l = (row % MT) / p.G, head = (row % MT) % p.G;
    const int tok = tok_l + t * p.npt, c0 = blockIdx.y * 32;
    pdl_wait();
    pdl_launch_dependents();
    int slot = 2 * blockIdx.x + 1;
    int4 rec = __ldcg(&p.rec[slot]);
    if ((rec.w & PIECE_LATE) && c0 == 0)
        for (int b = rec.x + (int)threadIdx.x; b <= rec.y; b += JOIN_THREADS)
            if (p.c.q_start[b] != p.c.q_start[b + 1]) p.status[b] = TV_ERR_TIMEOUT;
    if (!(rec.w & PIECE) || tok_l >= p.npt || tok >= rec.y || row >= p.prows) return;
    const int row0 = rec.x, g = rec.z;
    float mx = -INFINITY, den = 0.f, acc[32];
#pragma unroll
    for (int e = 0; e < 32; ++e) acc[e] = 0.f;
#pragma unroll 1
    while (true) {
        const float* sl = p.part + (int64_t)slot * p.prows * (D + 2);
        // the next slot's record, early
        const int ahead = slot + (slot & 1 ? 1 : 2);
        const bool more = !(rec.w & PIECE_LAST) && ahead < 2 * ctas;
        const int4 nrec = more ? __ldcg(&p.rec[ahead]) : rec;
        if (rec.w & PIECE_LATE) {
            den = 1.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) acc[e] = 0.f;
            break;
        }
        if (rec.w & PIECE) {
            const float mk = __ldcg(sl + p.prows * D + row), lk = __ldcg(sl + p.prows * (D + 1) + row);
            float4 v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = __ldcg(reinterpret_cast<const float4*>(sl) + (c0 / 4 + e) * p.prows + row);
            const float mm = fmaxf(mx, mk), bz = mm == -INFINITY ? 0.f : mm;
            const float f = exp2f(mx - bz), w = exp2f(mk - bz);
            mx = mm;
            den = fmaf(w, lk, den * f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                acc[4 * e] = fmaf(w, v[e].x, acc[4 * e] * f);
                acc[4 * e + 1] = fmaf(w, v[e].y, acc[4 * e + 1] * f);
                acc[4 * e + 2] = fmaf(w, v[e].z, acc[4 * e + 2] * f);
                acc[4 * e + 3] = fmaf(w, v[e].w, acc[4 * e + 3] * f);
            }
        }
        if (!more) break;
        slot = ahead;
        rec = nrec;
    }
    const float inv = 1.f / den;
    __nv_bfloat16* dst = p.out + (int64_t)(row0 + tok) * p.o_stride + (int64_t)(g * p.G + head) * D + c0;
#pragma unroll
    for (int e = 0; e < 32; e += 8) {
        uint4 v;
        v.x = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
        v.y = pack_bf16x2(acc[e + 2] * inv, acc[e + 3] * inv);
        v.z = pack_bf16x2(acc[e + 4] * inv, acc[e + 5] * inv);
        v.w = pack_bf16x2(acc[e + 6] * inv, acc[e + 7] * inv);
        *reinterpret_cast<uint4*>(dst + e) = v;
    }
}

// ---------------------------------------------------------------- host side
int partial_rows(int T, int G) { return T <= MT / G ? MT : 2 * MT; }

template <int D, bool CAP>
tv_status launch(const ChunkAttnArgs& a, const Params& p, const CUtensorMap& qm, const CUtensorMap& km,
                 const CUtensorMap& vm, int ctas) {
    static std::atomic<bool> set[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TV_ERR_CUDA;
    if (!set[dev]) {
        if (cudaFuncSetAttribute(chunk_tc_kernel<D, CAP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Lay<D>::BYTES) != cudaSuccess) {
            cudaGetLastError();
            return TV_ERR_CUDA;
        }
        set[dev] = true;
    }
    LaunchCfg lc(dim3((unsigned)ctas), dim3(THREADS), Lay<D>::BYTES, a.stream);
    if (cudaLaunchKernelEx(&lc.cfg, chunk_tc_kernel<D, CAP>, qm, km, vm, p) != cudaSuccess) return TV_ERR_CUDA;
    if (ctas == 1) return TV_OK;                               // nothing is cut
    LaunchCfg lj(dim3((unsigned)ctas, D / 32), dim3(JOIN_THREADS), 0, a.stream);
    return cudaLaunchKernelEx(&lj.cfg, chunk_tc_join_kernel<D>, p, ctas) == cudaSuccess ? TV_OK : TV_ERR_CUDA;
}

}  // namespace

bool chunk_attn_tc_applicable(int Hq, int Hkv, int d, tv_dtype dt) {
    return dt == TV_BF16 && (d == 64 || d == 128) && Hq / Hkv <= MT;
}

size_t chunk_attn_tc_workspace(int T, int B, int Hq, int Hkv, int d) {
    (void)B;
    return (size_t)2 * device_sm_count() * (partial_rows(T, Hq / Hkv) * (d + 2) * sizeof(float) + sizeof(int4));
}

tv_status launch_chunk_attn_tc(const ChunkAttnArgs& a) {
    const int G = a.Hq / a.Hkv, npt = MT / G;
    const int64_t rows = (int64_t)a.num_blocks * a.Hkv * a.bs;
    if (rows >= (1ll << 31)) return TV_ERR_UNSUPPORTED;
    CUtensorMap qm, km, vm;
    if (!make_q_rows_map(&qm, a.q, a.d, a.Hq, a.T, a.q_stride, G, npt)) return TV_ERR_CUDA;
    const bool maps = a.d == 128 ? make_kpage_map(&km, a.k_cache, rows) && make_page_map(&vm, a.v_cache, rows)
                                 : make_cache_map(&km, a.k_cache, 64, rows) && make_cache_map(&vm, a.v_cache, 64, rows);
    if (!maps) return TV_ERR_CUDA;
    Params p{};
    p.c = ChunkView{a.q_start, a.prefix_lens, a.block_table, a.T, a.B, a.max_blocks, a.bs, a.num_blocks};
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.o_stride = a.out_stride;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.q_stride = a.q_stride;
    p.k = static_cast<const __nv_bfloat16*>(a.k_cache);
    p.v = static_cast<const __nv_bfloat16*>(a.v_cache);
    p.status = a.status;
    p.rec = static_cast<int4*>(a.ws);
    p.part = reinterpret_cast<float*>(p.rec + 2 * device_sm_count());
    p.Hkv = a.Hkv;
    p.G = G;
    p.npt = npt;
    p.window = a.window;
    p.late = test_late_wait();
    p.prows = partial_rows(a.T, G);
    // (finite: a score of 0 stays 0)
    p.scale_log2 = a.softcap > 0.f ? fminf(2.f * LOG2E * a.scale / a.softcap, 3e38f) : a.scale * LOG2E;
    p.cap_log2 = a.softcap * LOG2E;
    if (a.softcap > 0.f) {
        const double k = (double)a.scale / a.softcap;
        p.cap_x = (float)std::min(k, 3e38);
        for (int e = 0; e < 3; ++e) p.cap_c[e] = (float)(TANH_C[e] * a.scale * 1.4426950408889634 * pow(k, 2 * e));
        // Beyond the polynomial's range a score is a difference of numbers of the cap's size, off by
        // 2^-23 of the cap: so the range is left only at 0.35 caps, whatever the cap, until the last
        // coefficient is no float32 any more (k^4 below 2^-149) and x has to be small enough not to
        // need it.  s^2 has to be finite.
        const double small = k > 1e5 ? 0.0 : std::min((k < 1e-10 ? 0.05 : TANH_SMALL) / k, 1e18);
        p.cap_small = (float)(small * small);
    }
    // one CTA per SM; fewer when even the longest sequences that fit give fewer runs
    const int64_t items = (int64_t)a.Hkv * (a.T / (2 * npt) + std::min(a.T, a.B));
    const int64_t units = items * std::min<int64_t>((int64_t)a.max_blocks * a.bs + C0, 1ll << 31);
    const int ctas = (int)std::clamp<int64_t>(std::max(units / RUN_MIN, (int64_t)a.B * a.Hkv), 1, device_sm_count());
    if (a.d == 128)
        return a.softcap > 0.f ? launch<128, true>(a, p, qm, km, vm, ctas) : launch<128, false>(a, p, qm, km, vm, ctas);
    return a.softcap > 0.f ? launch<64, true>(a, p, qm, km, vm, ctas) : launch<64, false>(a, p, qm, km, vm, ctas);
}

}  // namespace tv
