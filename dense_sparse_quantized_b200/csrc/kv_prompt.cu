// kv_prompt.cu -- attention over the 4-bit cache for many query rows per
// sequence (prompts, drafts checked at once): bound by matrix products and
// exponentials, so both products run on tcgen05.
//
// Work.  A job is (sequence, kv head, tile of R query rows), a row being one
// (query token, query head of the group) pair.  Its tokens are cut into units
// of 128, of which only those that some row sees count.  A job costs its units
// and kPieceCost more; the costs of all jobs, in order, are dealt to the CTAs
// in equal runs, wherever jobs begin and end.  What a job's pieces leave is
// joined through the workspace, in order.
//
// A CTA works on two row tiles of 128 at once (one at 256 dimensions), so that
// one tile's products run under the other's softmax; a job of one row tile is
// worked on twice, in every other unit, and put together at its end:
//   warps 0-3, 4-7  softmax of row tile 0, 1: thread = row.  Reads its 128
//                   scores from tensor memory, raises the running maximum if
//                   one exceeds it by more than 2^8 in the numerator (then the
//                   output so far is rescaled in tensor memory), writes the
//                   numerators back as fp16 over the scores.
//   warps 8-11      bring K and V: codes by cp.async into each warp's own
//                   place in shared memory a unit ahead, unpacked from there
//                   exactly to fp16 (kv_device.h) into the 128-byte-swizzled
//                   tiles of a ring.  Eight dimensions come out as 0 4 1 5 2 6 3 7; the queries are
//                   stored in that order, the output's columns renamed.
//   warp 14         works out the run and its pieces, ahead of the others.
//   warps 12, 13    issue the products of row tile 0, 1: S = Q K^T (K-major),
//                   then O += P V with P from tensor memory and V token-major
//                   (MN-major B).
// Unit t + 1's scores of a row tile are issued after unit t's output product
// of the same tile, so the commit that announces them also says that this
// product is done, and the output may be rescaled.
//
// Tokens that no row of the job sees get scale 0, whatever the cache holds
// there.  A NaN among the values would reach every row of the unit through
// the product, so its scale becomes 0 too and the rows that see the token get
// a NaN numerator; which tokens these are, and pages that do not exist, goes
// beside the tiles in `flags`.
//
// Measured on one B200, among other calls (bench.py --op kv): a prompt of 6000
// tokens, 32 query heads on 8 kv heads of 128, bf16, takes 370 to 376 us, 784 to
// 797 TFLOP/s of the scores that are seen (0.47 to 0.48 of a burst bf16 product's
// rate; 385 to 390 us apart).  A unit takes a pair about 4400 cycles: 1024 each
// for its two products (64 for each of 16 instructions, measured alone and
// beside everything else), 1500 for 128 exponentials a thread (1024 at the
// pipe's rate), 600 for the scores and their maximum, the rest waiting for one
// another.  What the steps brought, in runs too short for the power cap: products issued by one thread each from
// unrolled loops, not through local memory, 890 -> 764 us; loops rolled and
// unpacking by cp.async from shared memory, 708 -> 621; a product warp for each
// pair and numerators handed over by halves, 621 -> 527; pieces' own cost dealt
// too, 527 -> 468; no 64-bit division, 474 -> 427; turns at the exponentials,
// 444 -> 402 (in step, both pairs wait for the same pipe); pieces worked out by
// a warp of its own, 402 -> 387; the first half's numerators handed over while the
// second's are worked out, 387 -> 382; parts joined a row a warp, 382 -> 355
// (355 us at 1965 MHz are the 376 at the 1867 of a longer run).
//
// Every mbarrier wait is bounded (ptx.h).  One that runs out sets the device's
// status word, which dsq_kv_check reports, and ends its role; the others' waits
// run out in turn; what the product warps have issued is waited for (again with
// a limit), and the CTA frees its tensor memory and returns.
#include <algorithm>

#include "kv_device.h"
#include "ptx.h"

namespace dsq {

namespace {

constexpr int kN = 128;          // tokens of a unit
constexpr int kBlk = 128 * 128;  // bytes of 128 rows x 64 dimensions, swizzled
constexpr int kThreads = 512;
constexpr int kFlags = 4;        // units whose flags are kept
constexpr int kPieceCost = 3;    // units' time that a piece takes besides its units: queries in, outputs out
constexpr int kMinRun = 6;       // least cost of a CTA's run: shorter ones cost more to join than they save

template <int D_>
struct Shape {
    static constexpr int D = D_;
    static constexpr int A = D == 256 ? 1 : 2;       // row tiles at once: 128 (A + D / 128) columns of tensor memory each
    static constexpr int R = 128 * A;
    static constexpr int kStages = D == 256 ? 1 : 2; // K and V tiles in the ring
    static constexpr int kTile = D / 64 * kBlk;      // bytes of 128 rows
    // Of a loading warp: the codes and key words of its two tiles, and twice
    // their value words.  At 256 dimensions key and value codes take turns in
    // one place; there is no room for two.
    static constexpr bool kTurns = D == 256;
    static constexpr int kRawTile = (kTurns ? 1 : 2) * kKvTile * D / 2 + D, kRaw = 2 * kRawTile + 4 * D;
    __host__ __device__ static constexpr int raw_codes(int which) { return kTurns ? 0 : which * kKvTile * D / 2; }
    static constexpr int kRawWords = kRawTile - D;
    static constexpr int kSmem = (A + 2 * kStages) * kTile + 4 * kRaw + 1024;
    static_assert(kSmem + 512 <= 227 * 1024, "shared memory of a CTA");
    static constexpr int kO = A * 128;               // first column of the outputs
};

struct PromptParams {
    KvAttend a;
    float *parts;
    KvCarry *carries;
    int one_each;  // a job a CTA
};

// What the r-th pair of softmax and product warps does of a piece: rows
// [first, end) of the job's kv head, units x, x + step, ... below y (none: y =
// x).  A job of 128 rows or fewer is shared by units, else by row tiles.
struct Share {
    int first, end, x, y, step, shared;
};

// A piece of a CTA's run: units [t0, t1) of one job.
struct Piece {
    KvSeq s;
    int b, head, qt, t0, t1, rest;  // rest: the job's cost behind t1
    int begins, valid;
    int lo, hi;                     // tokens that some row of the job sees
    Share share[2];
};

constexpr int kPieces = 4;  // worked out ahead
struct Shared {
    uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], pfull[2][2], qfull[2], ofull[2], turn[2], other, joined;
    uint64_t piece_full[kPieces], piece_empty[kPieces];
    uint64_t drained[2];                // products issued by a warp that gave up a wait
    Piece piece[kPieces];
    uint4 nans[kFlags], holes[kFlags];  // by loading warp: NaN tokens; sub-tiles without a page
    float other_m[128], other_l[128];   // of a shared job, the second pair's maxima and sums
    uint32_t tmem;
    int64_t run, end;                   // cost of every CTA's run; where this one ends among all
};

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ void commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t at, float *v) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, float *v) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at)
        : "memory");
#pragma unroll
    for (int i = 0; i < 16; i++) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Shared-memory operand of 128-byte rows, 128-byte swizzle, groups of eight
// rows 1024 bytes apart: the descriptor's low word (address and leading
// dimension) and its high word, which all operands here have in common.
// K-major: a row is one of M or N, 64 elements of k.  MN-major: a row is one k,
// 64 elements of N, the next 64 of N kBlk bytes on.
__device__ __forceinline__ uint32_t operand(uint32_t at, uint32_t leading) { return at >> 4 | (leading >> 4) << 16; }
constexpr uint32_t kOperandHigh = 64u | 1u << 14 | 2u << 29;
constexpr uint32_t instruction(int n, bool b_mn_major) {
    return (1u << 4) | ((uint32_t)b_mn_major << 16) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// Set when a wait ran out, until dsq_kv_check reads it; one on each device.
__device__ int g_status;

// A warp's wait, all lanes testing; the same answer for all.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; i++) {
        if (__all_sync(kFull, mbar_try_wait(bar, parity))) return true;
        if ((i & 63u) == 0 && __any_sync(kFull, global_ns() - t0 > kWaitNs)) return false;
    }
}
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// D[tmem] (+)= A B, fp16, fp32 accumulator; A from shared or tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 y, {%2, %5};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(add), "n"(kOperandHigh)
        : "memory");
}

// Units [x, y) of a row tile's job: at least one, so that every row is written.
template <int R>
__device__ __forceinline__ int2 units_of(const KvAttend &a, const KvSeq &s, int qt) {
    const int last = min((qt + 1) * R, s.rows * a.share) - 1;
    const int lo = seen_by(a, s, qt * R).x / kN, hi = (max(seen_by(a, s, last).y, 0) + kN - 1) / kN;
    return make_int2(lo, max(hi, lo + 1));
}
template <int R>
__device__ __forceinline__ int tiles_of(const KvAttend &a, const KvSeq &s) {
    return (int)(((uint32_t)(s.rows * a.share) + R - 1) / R);
}

template <int R>
__device__ __forceinline__ Share share_of(const KvAttend &a, const Piece &p, int r) {
    Share w;
    const int rows = min((p.qt + 1) * R, p.s.rows * a.share);
    w.shared = R > 128 && rows - p.qt * R <= 128;
    w.step = w.shared ? 2 : 1;
    w.first = p.qt * R + (w.shared ? 0 : 128 * r);
    w.end = min(w.first + 128, rows);
    w.x = w.y = p.t0;
    if (w.first < w.end) {
        w.x = max(p.t0, seen_by(a, p.s, w.first).x / kN);
        w.y = max(w.x, min(p.t1, (max(seen_by(a, p.s, w.end - 1).y, 0) + kN - 1) / kN));
        if (w.shared) w.x = min(w.x + r, w.y);
    }
    return w;
}

// ----------------------------------------------------------------- warp 14
// Where a CTA's run begins -- a job, and how much of its cost lies before --
// and its cost.
struct Start {
    int b, head, qt, first, left;
};
template <int R>
__device__ __forceinline__ Start find_run(const KvAttend &a, bool one_each, Shared &sh) {
    const int lane = threadIdx.x & 31;
    auto cost = [&](const KvSeq &s, int qt) {
        const int2 u = units_of<R>(a, s, qt);
        return one_each ? 1 : kPieceCost + u.y - u.x;
    };
    auto head_cost = [&](int b) -> int64_t {  // of one kv head of sequence b
        const KvSeq s = kv_seq(a, b);
        const int tiles = tiles_of<R>(a, s);
        if (one_each) return tiles;
        int64_t n = 0;
#pragma unroll 1
        for (int qt = 0; qt < tiles; qt++) n += cost(s, qt);
        return n;
    };
    auto scan = [&](int64_t w) {
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int64_t up = __shfl_up_sync(kFull, w, m);
            if (lane >= m) w += up;
        }
        return w;
    };
    int64_t run = 1, u0 = blockIdx.x, u1 = u0 + 1;
    if (!one_each) {
        int64_t total = 0;
        if (a.batch < 8) {  // few sequences: the lanes take row tiles, else sequences
#pragma unroll 1
            for (int b = 0; b < a.batch; b++) {
                const KvSeq s = kv_seq(a, b);
                const int tiles = tiles_of<R>(a, s);
#pragma unroll 1
                for (int qt = lane; qt < tiles; qt += 32) total += (int64_t)cost(s, qt) * a.c.kv_heads;
            }
        } else
#pragma unroll 1
            for (int b = lane; b < a.batch; b += 32) total += head_cost(b) * a.c.kv_heads;
#pragma unroll
        for (int m = 16; m; m >>= 1) total += __shfl_xor_sync(kFull, total, m);
        run = max(divide(total + gridDim.x - 1, gridDim.x), (int64_t)kMinRun);
        u0 = min(total, run * blockIdx.x);
        u1 = min(total, u0 + run);
    }
    int64_t before = 0;
    Start at = {a.batch, 0, 0, 0, (int)(u1 - u0)};
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch && u0 < u1; b0 += 32) {
        const int64_t w = b0 + lane < a.batch ? head_cost(b0 + lane) : 0, sum = scan(w * a.c.kv_heads);
        const uint32_t past = __ballot_sync(kFull, before + sum > u0);
        if (past) {
            const int l = __ffs(past) - 1;
            at.b = b0 + l;
            before += __shfl_sync(kFull, sum - w * a.c.kv_heads, l);
            const int64_t per_head = max((int64_t)1, __shfl_sync(kFull, w, l));
            at.head = (int)divide(u0 - before, (int)min(per_head, (int64_t)0x7fffffff));
            before += at.head * per_head;
            break;
        }
        before += __shfl_sync(kFull, sum, 31);
    }
    if (at.b < a.batch) {
        const KvSeq s = kv_seq(a, at.b);
        const int tiles = tiles_of<R>(a, s);
#pragma unroll 1
        for (int q0 = 0; q0 < tiles; q0 += 32) {
            const int w = q0 + lane < tiles ? cost(s, q0 + lane) : 0;
            const int64_t sum = scan(w);
            const uint32_t past = __ballot_sync(kFull, before + sum > u0);
            if (past) {
                const int l = __ffs(past) - 1;
                at.qt = q0 + l;
                at.first = (int)(u0 - before - __shfl_sync(kFull, sum - w, l));
                break;
            }
            before += __shfl_sync(kFull, sum, 31);
        }
        if (one_each) {
            const int2 u = units_of<R>(a, s, at.qt);
            at.left = kPieceCost + u.y - u.x;
        }
    }
    if (lane == 0) {
        sh.run = run;
        sh.end = u1;
    }
    return at;
}

// Finds the run and works its pieces out, ahead of the warps that use them.
// This role and the others: false if a wait ran out.
template <int D, typename T>
__device__ __forceinline__ bool piece_role(const KvAttend &a, bool one_each, Shared &sh) {
    using S = Shape<D>;
    constexpr int R = S::R;
    const int lane = threadIdx.x & 31;
    Start at = find_run<R>(a, one_each, sh);
    for (uint32_t n = 0;; n++) {
        Piece p = {};
#pragma unroll 1
        while (at.left > 0 && at.b < a.batch) {
            p.s = kv_seq(a, at.b);
            const int tiles = tiles_of<R>(a, p.s);
            if (at.qt >= tiles) {
                at.qt = 0;
                if (tiles == 0 || ++at.head >= a.c.kv_heads) {
                    at.head = 0;
                    at.b++;
                }
                continue;
            }
            // [first, end) of the job's cost, kPieceCost of it before its units
            const int2 u = units_of<R>(a, p.s, at.qt);
            const int cost = kPieceCost + u.y - u.x, end = min(cost, at.first + at.left);
            p.b = at.b;
            p.head = at.head;
            p.qt = at.qt;
            p.t0 = u.x + max(0, at.first - kPieceCost);
            p.t1 = u.x + max(0, end - kPieceCost);
            p.rest = cost - end;
            p.begins = at.first <= kPieceCost;
            at.left -= end - at.first;
            at.first = 0;
            at.qt++;
            if (p.t0 < p.t1) {
                p.valid = 1;
                break;
            }
        }
        const int last = min((p.qt + 1) * R, p.s.rows * a.share) - 1;
        if (p.valid) {
            p.lo = seen_by(a, p.s, p.qt * R).x;
            p.hi = seen_by(a, p.s, last).y;
            p.share[0] = share_of<R>(a, p, 0);
            p.share[1] = share_of<R>(a, p, 1);
        }
        if (!warp_wait(&sh.piece_empty[n % kPieces], (n / kPieces & 1) ^ 1)) return false;
        if (lane == 0) {
            sh.piece[n % kPieces] = p;
            mbar_arrive(&sh.piece_full[n % kPieces]);
        }
        __syncwarp();
        if (!p.valid) return true;
        for (int rho = p.qt * R + lane; rho <= last; rho += 32) {  // its queries come to L2 meanwhile
            const T *q = (const T *)a.q + row_at(a, p.s, p.head, rho, a.q_token, a.q_head);
#pragma unroll
            for (int i = 0; i < D; i += 64) asm volatile("prefetch.global.L2 [%0];" ::"l"(q + i));
        }
    }
}

// The pieces, for a warp of the other roles.
struct Pieces {
    uint32_t n = 0;
    bool ok = true;      // no wait for one ran out
    Share mine, theirs;  // the r-th pair's, and the other's
    __device__ __forceinline__ bool next(Shared &sh, Piece &p, int r) {
        const uint32_t at = n % kPieces;
        if (!warp_wait(&sh.piece_full[at], n / kPieces & 1)) return ok = false;
        p = sh.piece[at];
        mine = sh.piece[at].share[r];
        theirs = sh.piece[at].share[r ^ 1];
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(&sh.piece_empty[at]);
        n++;
        return p.valid;
    }
};

// ------------------------------------------------------------ warps 8-11
// Each warp brings tiles 2 w and 2 w + 1 of a unit's eight: by cp.async as they
// are into its own `raw`, keys and values apart so that one's copy runs while
// the other is unpacked, and from there unpacked into the operand.  The value
// words come with the keys, so that their NaNs are known when the keys are
// handed over; they are kept for two units.  The loops are kept rolled: four
// roles' code has to fit the instruction caches.
template <int D>
struct Loader {
    using S = Shape<D>;
    const KvAttend &a;
    Shared &sh;
    Pieces pieces;
    Piece p;
    int t;
    bool more;
    const int lane, warp;

    // A unit on its way: the pages of the warp's tiles, and which tokens of
    // the unit some row sees.
    struct Unit {
        int lo, hi, page[2], in_page[2], head;
        bool there;
    };
    __device__ __forceinline__ Loader(const KvAttend &a_, Shared &sh_)
        : a(a_), sh(sh_), lane(threadIdx.x & 31), warp((threadIdx.x >> 5) & 3) {
        more = pieces.next(sh, p, 0);
        t = p.t0;
    }
    __device__ __forceinline__ Unit next() {
        Unit u = {};
        u.there = more;
        u.page[0] = u.page[1] = -1;
        if (!more) return u;
        u.lo = p.lo - t * kN;
        u.hi = p.hi - t * kN;
        u.head = p.head;
        const int32_t *row = a.page_table + (int64_t)p.b * a.table_pages;
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const int tile = t * (kN / kKvTile) + 2 * warp + i, col = a.tiles_by.div(tile);
            u.in_page[i] = tile - col * a.c.page_tiles;
            if (col < a.table_pages && u.hi > (2 * warp + i) * kKvTile) u.page[i] = row[col];
        }
        if (++t == p.t1) {
            more = pieces.next(sh, p, 0);
            t = p.t0;
        }
        return u;
    }
    __device__ __forceinline__ bool there(const Unit &u, int i) const {
        return (uint32_t)(i ? u.page[1] : u.page[0]) < (uint32_t)a.c.pages;
    }
    // Starts the copy of both tiles' keys or values; a tile without a page is
    // not copied, and not used.
    __device__ __forceinline__ void copy(const Unit &u, int which, uint32_t raw, uint32_t value_words) const {
#pragma unroll
        for (int i = 0; i < 2; i++)
            if (there(u, i)) {
                const uint8_t *src =
                    a.c.cache + (((int64_t)u.page[i] * a.c.kv_heads + u.head) * a.c.page_tiles + u.in_page[i]) * kv_tile_bytes(D);
                const uint32_t dst = raw + i * S::kRawTile;
#pragma unroll
                for (int k = 0; k < D / 64; k++)
                    cp_async16(dst + S::raw_codes(which) + k * 512 + lane * 16, src + kv_codes(D, which) + k * 512 + lane * 16);
                if (which == 0 && lane < D / 8)  // D / 16 chunks of key words, then as many of value words
                    cp_async16(lane < D / 16 ? dst + S::kRawWords + lane * 16 : value_words + i * D + (lane - D / 16) * 16,
                               src + kv_words(D, 0) + lane * 16);
            }
        cp_async_commit();
    }
    // Which of this lane's value words are NaN, by tile (bits 0, 1).
    __device__ __forceinline__ uint32_t nans(const Unit &u, uint32_t value_words) const {
        const int tok = lane >> 1, pair = lane & 1;
        uint32_t bad = 0;
#pragma unroll 1
        for (int i = 0; i < 2; i++) {
            const int at = (2 * warp + i) * kKvTile + tok;
            const bool use = there(u, i) && at >= u.lo && at < u.hi;
#pragma unroll
            for (int g = 0; g < D / 64; g++) {
                uint16_t word;
                asm volatile("ld.shared.u16 %0, [%1];"
                             : "=h"(word)
                             : "r"(value_words + i * D + g * 4 * kKvTile + (pair * kKvTile + tok) * 2));
                if (use && (word & 0x7c00u) == 0x7c00u) bad |= 1u << i;
            }
        }
        return bad;
    }
    // Unpacks them into the operand at `tile`.  Lane: token lane / 2, groups of
    // 32 dimensions lane % 2, + 2, ...; four of them at a time.
    __device__ __forceinline__ void unpack(const Unit &u, int which, uint32_t raw, uint32_t value_words, uint32_t tile) const {
        const int tok = lane >> 1, pair = lane & 1;
        constexpr int G = D / 64, N = G < 2 ? 2 : 4;  // groups of a lane's token; groups at a time
        const uint32_t codes = raw + S::raw_codes(which) + tok * (D / 2) + pair * 16;
        const uint32_t words = (which ? value_words : raw + S::kRawWords) + (pair * kKvTile + tok) * 2;
        const uint32_t words_tile = which ? D : S::kRawTile, to = tile + (2 * warp * kKvTile + tok) * 128;
        uint32_t swizzle[4];
#pragma unroll
        for (int k = 0; k < 4; k++) swizzle[k] = ((pair * 4 + k) ^ (tok & 7)) << 4;
#pragma unroll 1
        for (int c0 = 0; c0 < 2 * G; c0 += N) {
            uint4 x[N];
            uint32_t w[N];
#pragma unroll
            for (int c = 0; c < N; c++) {
                const int i = (c0 + c) / G, g = (c0 + c) % G, at = (2 * warp + i) * kKvTile + tok;
                uint16_t word;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(word) : "r"(words + i * words_tile + g * 4 * kKvTile));
                x[c] = lds128(codes + i * S::kRawTile + g * 32);
                const bool use = there(u, i) && at >= u.lo && at < u.hi && !(which == 1 && (word & 0x7c00u) == 0x7c00u);
                w[c] = use ? word : 0u;
            }
#pragma unroll
            for (int c = 0; c < N; c++) {
                const int i = (c0 + c) / G, g = (c0 + c) % G;
                const Decode d(prmt(w[c], w[c], 0x1010));
                const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w}, row = to + i * kKvTile * 128 + g * kBlk;
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const uint32_t y = v[k] >> 8;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + swizzle[k]), "r"(d.low(v[k])),
                                 "r"(d.high(v[k])), "r"(d.low(y)), "r"(d.high(y))
                                 : "memory");
                }
            }
        }
    }
};

template <int D>
__device__ __forceinline__ bool load_role(const KvAttend &a, Shared &sh, uint32_t kbuf, uint32_t vbuf, uint32_t raw0) {
    using S = Shape<D>;
    using L = Loader<D>;
    L ld(a, sh);
    const uint32_t raw = raw0 + ld.warp * S::kRaw, words = raw + 2 * S::kRawTile;
    typename L::Unit u = ld.next(), u1 = ld.next();
    ld.copy(u, 0, raw, words);
    if (!S::kTurns) ld.copy(u, 1, raw, words);
    for (uint32_t it = 0; u.there; it++) {
        const typename L::Unit u2 = ld.next();
        const uint32_t stage = it % S::kStages, phase = it / S::kStages & 1;
        const uint32_t words0 = words + (it & 1) * 2 * D, words1 = words + (~it & 1) * 2 * D;
#pragma unroll 1
        for (int which = 0; which < 2; which++) {
            if (!warp_wait(which ? &sh.vempty[stage] : &sh.kempty[stage], phase ^ 1)) {
                cp_async_wait<0>();
                return false;
            }
            cp_async_wait<S::kTurns ? 0 : 1>();  // all copies but the other half's, the last started
            __syncwarp();
            if (which == 0) {
                const uint32_t nan = ld.nans(u, words0);
                uint32_t bad = 0;
                if (__any_sync(kFull, nan)) {
#pragma unroll 1
                    for (int i = 0; i < 32; i++) {  // lane i: token i / 2 of both tiles
                        const uint32_t of = __shfl_sync(kFull, nan, i);
                        bad |= (of & 1u) << (i >> 1) | (of >> 1) << (16 + (i >> 1));
                    }
                }
                if (ld.lane == 0) {
                    reinterpret_cast<uint32_t *>(&sh.nans[it % kFlags])[ld.warp] = bad;
                    reinterpret_cast<uint32_t *>(&sh.holes[it % kFlags])[ld.warp] = (uint32_t)!ld.there(u, 0) | (uint32_t)!ld.there(u, 1) << 1;
                }
            }
            ld.unpack(u, which, raw, words0, (which ? vbuf : kbuf) + stage * S::kTile);
            fence_async();
            __syncwarp();
            if (ld.lane == 0) mbar_arrive(which ? &sh.vfull[stage] : &sh.kfull[stage]);
            if (!S::kTurns) ld.copy(u1, which, raw, words1);
            else if (which == 0) ld.copy(u, 1, raw, words0);
            else ld.copy(u1, 0, raw, words1);
        }
        u = u1;
        u1 = u2;
    }
    cp_async_wait<0>();
    return ld.pieces.ok;
}

// ----------------------------------------------------------- warps 12, 13
// One for each row tile, so that neither waits for the other's softmax.  All
// lanes walk, one issues.  `it`: units worked on.
template <int D>
__device__ __forceinline__ bool issue_products(Shared &sh, uint32_t qbuf, uint32_t kbuf, uint32_t vbuf, int r, bool lead, uint32_t &it) {
    using S = Shape<D>;
    constexpr uint32_t kScores = instruction(kN, false), kOut = instruction(D, true);
    const uint32_t st = sh.tmem + 128 * r, ot = sh.tmem + S::kO + D * r;
    const uint32_t q0 = operand(qbuf + r * S::kTile, 16), k0 = operand(kbuf, 16), v0 = operand(vbuf, kBlk);
    Pieces pieces;
    Piece p;
    uint32_t done = 0, queries = 0;
    while (pieces.next(sh, p, r)) {
        const Share &mine = pieces.mine;
        for (int t = p.t0; t < p.t1; t++, it++) {
            const uint32_t stage = it % S::kStages, phase = it / S::kStages & 1;
            const bool on = t >= mine.x && t < mine.y && !((t - mine.x) & (mine.step - 1));
            if (!warp_wait(&sh.kfull[stage], phase)) return false;
            if (t == mine.x && on && !warp_wait(&sh.qfull[r], queries++ & 1)) return false;
            fence_after();
            if (lead) {
                if (on) {
                    const uint32_t k = k0 + stage * (S::kTile >> 4);
#pragma unroll
                    for (int i = 0; i < D / 16; i++) {
                        const uint32_t at = (i / 4 * kBlk + i % 4 * 32) >> 4;
                        mma_ss(st, q0 + at, k + at, kScores, i);
                    }
                    commit(&sh.sfull[r]);
                }
                commit(&sh.kempty[stage]);
            }
            __syncwarp();
            if (!warp_wait(&sh.vfull[stage], phase)) return false;
#pragma unroll
            for (int half = 0; half < 2; half++) {
                if (on && !warp_wait(&sh.pfull[r][half], done & 1)) return false;
                fence_after();
                if (lead) {
                    if (on) {
                        const uint32_t v = v0 + stage * (S::kTile >> 4);
#pragma unroll
                        for (int i = 4 * half; i < 4 * half + 4; i++) mma_ts(ot, st + 8 * i, v + i * (2048 >> 4), kOut, i + (t - mine.x));
                        if (half && t + mine.step >= mine.y) commit(&sh.ofull[r]);
                    }
                    if (half) commit(&sh.vempty[stage]);
                }
                __syncwarp();
            }
            done += on;
        }
    }
    return pieces.ok;
}

template <int D>
__device__ __forceinline__ bool product_role(Shared &sh, uint32_t qbuf, uint32_t kbuf, uint32_t vbuf, int r) {
    constexpr uint32_t kStages = Shape<D>::kStages;
    const bool lead = elect_one();  // one thread throughout: a commit speaks for its own thread's products
    uint32_t it = 0;
    if (!issue_products<D>(sh, qbuf, kbuf, vbuf, r, lead, it)) {
        if (lead) commit(&sh.drained[r]);
        __syncwarp();
        warp_wait(&sh.drained[r], 0);
        return false;
    }
    // The last releases of the ring, which nobody else waits for: none is to
    // arrive when the CTA's shared memory is another's.
    for (uint32_t i = it > kStages ? it - kStages : 0; i < it; i++)
        if (!warp_wait(&sh.kempty[i % kStages], i / kStages & 1) || !warp_wait(&sh.vempty[i % kStages], i / kStages & 1)) return false;
    return true;
}

// ------------------------------------------------------------- warps 0-7
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The lowest n bits, none for n <= 0, all for n >= 32.
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Two at once: a * b + c, and a + b.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}

// A warp's 32 rows of a row tile between global and shared memory, where they
// lie as the operand does: LANES lanes take a row's 16-byte chunks, so that a
// row's bytes go together.
template <int D>
struct Rows {
    static constexpr int LANES = D / 8, AT_ONCE = 32 / LANES;
    const int lane = threadIdx.x & 31, chunk = lane % LANES, sub = lane / LANES;
    __device__ __forceinline__ uint32_t at(uint32_t tile, int row) const {  // of this lane's chunk
        return tile + chunk / 8 * kBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4);
    }
};

// The queries, into the row tile; returns what the scores of this thread's
// row are to be multiplied by.  A negative scale becomes the queries' sign, so
// that the largest score stays the largest.
template <int D, typename T>
__device__ __forceinline__ float load_queries(const KvAttend &a, const Piece &p, int first, int end, int row0, uint32_t tile) {
    using W = Rows<D>;
    constexpr int N = D == 64 ? 8 : 16;  // loads under way
    const W w;
    const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
    int up = 0;
#pragma unroll 1
    for (int i0 = 0; i0 < 32; i0 += N * W::AT_ONCE) {
        uint4 x[N];
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int rho = min(first + row0 + i0 + i * W::AT_ONCE + w.sub, end - 1);
            x[i] = reinterpret_cast<const uint4 *>((const T *)a.q + row_at(a, p.s, p.head, rho, a.q_token, a.q_head))[w.chunk];
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            int e = 0;
            if constexpr (!std::is_same<T, __half>::value) {
                uint32_t top = top_bits(x[i], 0);
#pragma unroll
                for (int m = 1; m < W::LANES; m <<= 1) top = max(top, __shfl_xor_sync(kFull, top, m));
                e = up_of(top);
                const int of = __shfl_sync(kFull, e, w.lane % W::AT_ONCE * W::LANES);
                if (w.lane / W::AT_ONCE == i0 / W::AT_ONCE + i) up = of;
            }
            uint4 y[1] = {x[i]};
            query_codes_order<T, 1>(y, e);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(w.at(tile, row0 + i0 + i * W::AT_ONCE + w.sub)),
                         "r"(y[0].x ^ sign), "r"(y[0].y ^ sign), "r"(y[0].z ^ sign), "r"(y[0].w ^ sign)
                         : "memory");
        }
    }
    // not 0: a masked score times it is to stay -inf
    return fmaxf(fabsf(a.scale_log2) * exponent(-up), 1.17549435e-38f);
}

template <int D, typename T>
__device__ __forceinline__ bool softmax_role(const PromptParams &pp, Shared &sh, uint32_t qbuf, int r) {
    using S = Shape<D>;
    const KvAttend &a = pp.a;
    const int row = threadIdx.x & 127, row0 = row & 96;
    const uint32_t lanes = (uint32_t)row0 << 16;  // this warp's quarter of tensor memory
    const uint32_t st = sh.tmem + 128 * r + lanes, ot = sh.tmem + S::kO + D * r + lanes, tile = qbuf + r * S::kTile;
    const bool lead = (threadIdx.x & 31) == 0;
    Pieces pieces;
    Piece p;
    uint32_t it0 = 0, sn = 0, on = 0, joins = 0, turns = 0;
    while (pieces.next(sh, p, r)) {
        const Share &mine = pieces.mine;
        const int first = mine.first, end = mine.end, rho = first + row;
        const bool idle = first + row0 >= end;  // no rows for this warp
        // Units that both pairs work on: they take turns at the exponentials.
        int2 both = make_int2(0, 0);
        if (S::A == 2 && !mine.shared) {
            const Share &theirs = pieces.theirs;
            both = make_int2(max(mine.x, theirs.x), min(mine.y, theirs.y));
        }
        float m = kNoMax, l = 0.0f;
        if (mine.x < mine.y) {
            const int2 seen = seen_by(a, p.s, min(rho, end - 1));
            const int all_lo = seen_by(a, p.s, end - 1).x, all_hi = seen_by(a, p.s, first).y;
            const float f = load_queries<D, T>(a, p, first, end, row0, tile);
            fence_async();
            fence_before();
            __syncwarp();
            if (lead) mbar_arrive(&sh.qfull[r]);
            for (int t = mine.x; t < mine.y; t += mine.step) {
                if (!warp_wait(&sh.sfull[r], sn++ & 1)) return false;
                fence_after();
                const bool in_turn = t >= both.x && t < both.y;
                if (idle) {
                    if (in_turn) {
                        if (!warp_wait(&sh.turn[r], (turns ^ r ^ 1) & 1)) return false;
                        turns++;
                    }
                    if (lead) {
                        if (in_turn) mbar_arrive(&sh.turn[r ^ 1]);
                        mbar_arrive(&sh.pfull[r][0]);
                        mbar_arrive(&sh.pfull[r][1]);
                    }
                    continue;
                }
                const uint32_t flag = (it0 + t - p.t0) % kFlags;
                const uint4 nans = sh.nans[flag], holes = sh.holes[flag];
                if (all_lo > t * kN || all_hi < (t + 1) * kN || (nans.x | nans.y | nans.z | nans.w | holes.x | holes.y | holes.z | holes.w)) {
                    // some row sees part of the unit: its scores go back masked
                    const uint32_t hole = holes.x | holes.y << 2 | holes.z << 4 | holes.w << 6;
                    const int lo = seen.x - t * kN, hi = seen.y - t * kN;
#pragma unroll 1
                    for (int i = 0; i < 4; i++) {
                        float s[32];
                        tmem_ld32(st + 32 * i, s);
                        wait_ld();
                        const uint32_t nan = i == 0 ? nans.x : i == 1 ? nans.y : i == 2 ? nans.z : nans.w;
                        // bits of the 32 tokens that this row does not see
                        uint32_t off = below(lo - 32 * i) | ~below(hi - 32 * i);
                        off |= (hole >> (2 * i) & 1u ? 0x0000ffffu : 0u) | (hole >> (2 * i) & 2u ? 0xffff0000u : 0u);
#pragma unroll
                        for (int k = 0; k < 32; k++) {
                            if (nan >> k & 1u) s[k] = NAN;
                            if (off >> k & 1u) s[k] = -INFINITY;
                        }
                        tmem_st32(st + 32 * i, reinterpret_cast<const uint32_t *>(s));
                    }
                    wait_st();
                }
                float s[kN];
#pragma unroll
                for (int i = 0; i < kN; i += 32) tmem_ld32(st + i, s + i);
                wait_ld();
                float top[4] = {max3(s[0], s[1], s[2]), max3(s[32], s[33], s[34]), max3(s[64], s[65], s[66]), max3(s[96], s[97], s[98])};
#pragma unroll
                for (int i = 3; i < 31; i += 2)
#pragma unroll
                    for (int k = 0; k < 4; k++) top[k] = max3(top[k], s[32 * k + i], s[32 * k + i + 1]);
                const float x = max3(max3(top[0], top[1], top[2]), max3(top[3], s[31], s[63]), fmaxf(s[95], s[127])) * f;
                if (__any_sync(kFull, x > m + (kLift + kLazy))) {
                    const float next = fmaxf(m, x - kLift), keep = ex2(m - next);
                    m = next;
                    l *= keep;
                    if (t > mine.x) {
#pragma unroll 1
                        for (int i = 0; i < D; i += 16) {
                            float o[16];
                            tmem_ld16(ot + i, o);
                            wait_ld();
#pragma unroll
                            for (int k = 0; k < 16; k++) o[k] *= keep;
                            tmem_st16(ot + i, reinterpret_cast<const uint32_t *>(o));
                        }
                    }
                }
                // The first pair's first turn is there from the start.
                if (in_turn) {
                    if (!warp_wait(&sh.turn[r], (turns ^ r ^ 1) & 1)) return false;
                    turns++;
                }
                float2 sum[2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
                auto hand_over = [&](int half) {  // the product over 64 tokens starts while the others are worked on
                    wait_st();
                    fence_before();
                    __syncwarp();
                    if (lead) mbar_arrive(&sh.pfull[r][half]);
                };
#pragma unroll
                for (int half = 0; half < 2; half++) {
                    uint32_t ph[32];
#pragma unroll
                    for (int k = 0; k < 32; k++) {
                        const float2 y =
                            fma2(make_float2(s[64 * half + 2 * k], s[64 * half + 2 * k + 1]), make_float2(f, f), make_float2(-m, -m));
                        const float2 e = make_float2(ex2(y.x), ex2(y.y));
                        sum[k & 1] = add2(sum[k & 1], e);
                        ph[k] = pack_h2(e.x, e.y);
                        if (half == 1 && k == 7) hand_over(0);  // its store has had time to end
                    }
                    if (half == 1 && in_turn && lead) mbar_arrive(&sh.turn[r ^ 1]);
                    tmem_st32(st + 32 * half, ph);
                }
                hand_over(1);
                sum[0] = add2(sum[0], sum[1]);
                l += sum[0].x + sum[0].y;
            }
            if (!warp_wait(&sh.ofull[r], on++ & 1)) return false;
            fence_after();
        }
        it0 += p.t1 - p.t0;

        // A shared job: the first pair takes in what the second found.
        float f0 = 1.0f, f1 = 0.0f;
        bool two = false;
        if (mine.shared) {
            if (r == 1) {
                sh.other_m[row] = m;
                sh.other_l[row] = l;
                fence_before();
                __syncwarp();
                if (lead) mbar_arrive(&sh.other);
                if (!warp_wait(&sh.joined, joins++ & 1)) return false;
                continue;
            }
            if (!warp_wait(&sh.other, joins++ & 1)) return false;
            fence_after();
            const Share &theirs = pieces.theirs;
            two = theirs.x < theirs.y;
            if (two) {
                const float m1 = sh.other_m[row], top = fmaxf(m, m1);
                f0 = ex2(m - top);
                f1 = ex2(m1 - top);
                l = l * f0 + sh.other_l[row] * f1;
                m = top;
            }
        }

        // The rows' outputs, by way of the queries' place, or the piece's
        // partial result.
        const bool whole = p.begins && p.rest == 0;
        float *part = pp.parts + (2 * blockIdx.x + (p.begins ? 1 : 0)) * kv_part_floats<D, S::R>();
        const int part_row = first - p.qt * S::R + row;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll 1
        for (int i = 0; i < D && !idle; i += 16) {
            float o[16];
            if (mine.x < mine.y) {
                tmem_ld16(ot + i, o);
                wait_ld();
            } else {
#pragma unroll
                for (int k = 0; k < 16; k++) o[k] = 0.0f;
            }
            if (two) {
                float o1[16];
                tmem_ld16(ot + D + i, o1);
                wait_ld();
#pragma unroll
                for (int k = 0; k < 16; k++) o[k] = o[k] * f0 + o1[k] * f1;
            }
#pragma unroll
            for (int k = 0; k < 16; k += 8) {
                // columns k .. k + 7 are dimensions 0 4 1 5 2 6 3 7
                if (whole) {
                    const int chunk = (i + k) / 8;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     tile + chunk / 8 * kBlk + row * 128 + (((chunk & 7) ^ (row & 7)) << 4)),
                                 "r"(pack_out<T>(o[k] * inv, o[k + 2] * inv)), "r"(pack_out<T>(o[k + 4] * inv, o[k + 6] * inv)),
                                 "r"(pack_out<T>(o[k + 1] * inv, o[k + 3] * inv)), "r"(pack_out<T>(o[k + 5] * inv, o[k + 7] * inv))
                                 : "memory");
                } else {
                    float4 *to = reinterpret_cast<float4 *>(part + part_row * D + i + k);
                    to[0] = make_float4(o[k], o[k + 2], o[k + 4], o[k + 6]);
                    to[1] = make_float4(o[k + 1], o[k + 3], o[k + 5], o[k + 7]);
                }
            }
        }
        if (whole) {
            using W = Rows<D>;
            const W w;
            __syncwarp();
#pragma unroll 4
            for (int i = 0; i < 32; i += W::AT_ONCE) {
                const int of = row0 + i + w.sub;
                const uint4 x = lds128(w.at(tile, of));
                if (first + of < end)
                    reinterpret_cast<uint4 *>((T *)a.out + row_at(a, p.s, p.head, first + of, a.out_token, a.out_head))[w.chunk] = x;
            }
            __syncwarp();
            if (a.lse && rho < end) a.lse[row_at(a, p.s, p.head, rho, a.q_heads, 1)] = lse_of(m, l);
        } else if (!idle) {
            part[S::R * D + part_row] = m;
            part[S::R * D + S::R + part_row] = l;
            if (p.begins && r == 0 && row == 0) {
                const KvCarry c = {1, (int)divide(sh.end + p.rest - 1, (int)sh.run) - (int)blockIdx.x, p.b, p.head, p.qt, {}};
                pp.carries[blockIdx.x] = c;
            }
        }
        fence_before();
        if (mine.shared) {
            __syncwarp();
            if (lead) mbar_arrive(&sh.joined);
        }
    }
    return pieces.ok;
}

template <int D, typename T>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ PromptParams pp) {
    using S = Shape<D>;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Shared sh;
    const uint32_t qbuf = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t kbuf = qbuf + S::A * S::kTile, vbuf = kbuf + S::kStages * S::kTile;
    const int warp = threadIdx.x >> 5;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; i++) {
            mbar_init(&sh.kfull[i], 4);
            mbar_init(&sh.vfull[i], 4);
            mbar_init(&sh.kempty[i], S::A);
            mbar_init(&sh.vempty[i], S::A);
            mbar_init(&sh.sfull[i], 1);
            mbar_init(&sh.ofull[i], 1);
            mbar_init(&sh.pfull[i][0], 4);
            mbar_init(&sh.pfull[i][1], 4);
            mbar_init(&sh.qfull[i], 4);
            mbar_init(&sh.turn[i], 4);
            mbar_init(&sh.drained[i], 1);
        }
        for (int i = 0; i < kPieces; i++) {
            mbar_init(&sh.piece_full[i], 1);
            mbar_init(&sh.piece_empty[i], 4 * S::A + 4 + S::A);  // all warps but this one's
        }
        mbar_init(&sh.other, 4);
        mbar_init(&sh.joined, 4);
        fence_mbar_init();
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh.tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    kv_after_previous();
    if (threadIdx.x == 0 && !pp.one_each) pp.carries[blockIdx.x].valid = 0;
    fence_before();
    __syncthreads();
    fence_after();

    // 512 threads x 128 registers: 2 x 184 + 88 + 56 for the four warpgroups.
    bool ok = true;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
        if (warp < 4 * S::A) ok = softmax_role<D, T>(pp, sh, qbuf, warp >> 2);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
        ok = load_role<D>(pp.a, sh, kbuf, vbuf, vbuf + S::kStages * S::kTile);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 14) ok = piece_role<D, T>(pp.a, pp.one_each, sh);
        else if (warp < 12 + S::A) ok = product_role<D>(sh, qbuf, kbuf, vbuf, warp - 12);
    }
    if (!ok && (threadIdx.x & 31) == 0) report(&g_status, kStatusTimeout);
    fence_before();
    __syncthreads();
    if (warp == 12) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(sh.tmem), "r"(512) : "memory");
    }
}

template <int D, typename T>
int launch_prompt(const KvAttend &a, void *workspace, int sms, cudaStream_t st) {
    using S = Shape<D>;
    // A job a CTA where every job has an SM and six units at most: no joining,
    // one launch.
    const int64_t jobs = a.c.kv_heads * (a.q_start ? a.batch + (int64_t)a.q_tokens * a.share / S::R
                                                    : a.batch * (((int64_t)a.rows_each * a.share + S::R - 1) / S::R));
    int64_t tokens = a.most_tokens;
    if (a.window) tokens = std::min<int64_t>(tokens, (int64_t)a.window + S::R / a.share + 1);
    const bool one_each = jobs <= sms && tokens / kN + 2 <= 6;
    const PromptParams p = {a, (float *)workspace, kv_carries<D, S::R>(workspace), one_each};
    auto kernel = prompt_kernel<D, T>;
    static KvOnce once;
    if (!once.set_smem((const void *)kernel, S::kSmem)) return DSQ_ERR_CUDA;
    const int grid = one_each ? (int)jobs : std::min(sms, kMaxCtas);
    const int rc = kv_launch(kernel, grid, kThreads, S::kSmem, st, p);
    return rc != DSQ_OK || one_each ? rc : launch_join<D, S::R, T>(a, p.parts, p.carries, grid, jobs, st);
}

// A wait that nothing ends, through the wait of the roles above.
__global__ void __launch_bounds__(32) wait_timeout_kernel() {
    __shared__ uint64_t bar;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        fence_mbar_init();
    }
    __syncthreads();
    if (!warp_wait(&bar, 0) && threadIdx.x == 0) report(&g_status, kStatusTimeout);
}

template <typename T>
int launch_of(const KvAttend &a, int head_dim, void *workspace, int sms, cudaStream_t st) {
    if (head_dim == 64) return launch_prompt<64, T>(a, workspace, sms, st);
    if (head_dim == 128) return launch_prompt<128, T>(a, workspace, sms, st);
    return launch_prompt<256, T>(a, workspace, sms, st);
}

}  // namespace

size_t kv_prompt_workspace(int head_dim) {
    return head_dim == 64 ? kv_parts_bytes<64, Shape<64>::R>() : head_dim == 128 ? kv_parts_bytes<128, Shape<128>::R>()
                                                                                 : kv_parts_bytes<256, Shape<256>::R>();
}

int launch_kv_prompt(const KvAttend &a, int head_dim, int dtype, void *workspace, int sms, cudaStream_t st) {
    if (dtype == DSQ_DTYPE_F16) return launch_of<__half>(a, head_dim, workspace, sms, st);
    return launch_of<__nv_bfloat16>(a, head_dim, workspace, sms, st);
}

int launch_kv_wait_timeout(cudaStream_t st) {
    wait_timeout_kernel<<<1, 32, 0, st>>>();
    return cudaGetLastError() == cudaSuccess ? DSQ_OK : DSQ_ERR_CUDA;
}

int kv_take_status(int *word) {
    *word = 0;
    const int zero = 0;
    if (cudaDeviceSynchronize() == cudaSuccess && cudaMemcpyFromSymbol(word, g_status, sizeof(int)) == cudaSuccess &&
        (*word == 0 || cudaMemcpyToSymbol(g_status, &zero, sizeof(int)) == cudaSuccess))
        return DSQ_OK;
    cudaGetLastError();
    return DSQ_ERR_CUDA;
}

}  // namespace dsq
