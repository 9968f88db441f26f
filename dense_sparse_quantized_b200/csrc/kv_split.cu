// kv_split.cu -- attention over the 4-bit cache for few query rows per
// sequence: bound by the cache's bytes, so everything here serves to stream
// them.
//
// Work.  A job is (sequence, kv head, tile of R query rows), a row being one
// (query token, query head of the group) pair, so the heads that share a kv
// head share its bytes.  A job's tokens are cut into units of 32; the units of
// all jobs, in order, are dealt to the CTAs in equal runs, and a CTA's run to
// its warps in equal runs, wherever the jobs begin and end: long and short
// sequences and any number of heads fill the GPU alike.  Each CTA finds its
// place from kv_lens and q_start itself, so nothing is planned on the host
// and a captured call follows the lengths.
//
// A warp runs through its units alone, with a running maximum and sum.  A job
// inside one warp's run is written at once.  What spans warps of a CTA is
// merged in shared memory at the end, what spans CTAs through the workspace by
// join_kernel, always in the same order.
//
// A unit.  Two tiles of 16 tokens, brought to the warp's own ring in shared
// memory by cp.async of whole tiles.  Scores: mma.sync m16n8k16 with the 16
// tokens of a tile as M and the rows as N = 8 (a group of eight heads fills
// it; the cache's codes are unpacked once for all rows).  The order of the 16
// tokens along M and k and that of the dimensions along k and M is free, so
// it is chosen such that a lane's fragment is what it can load whole:
//   keys: lane (r, j) holds D/4 consecutive dimensions of tokens tok(r) and
//     tok(r) + 2, tok(r) = 4 (r / 2) + r % 2;
//   values: D/8 consecutive dimensions, from r D/8 on, of tokens 4j .. 4j+3.
// Codes become fp16 exactly: LOP3 places two in the halves of 1024 (or 64),
// HADD2 takes off 1024 + zero, HMUL2 multiplies by the scale -- 4 bits times 7
// bits, no rounding.  The scores' fragment, rounded to fp16 and transposed by
// movmatrix, is the B operand of the second product, out^T = V^T P^T.
//
// The running maximum is raised only when some score exceeds it by more than
// 2^8 in the numerator (one vote a unit); until then numerators up to 2^15 are
// as exact as ones up to 2^7, which they are at the maximum (kLift).
//
// Measured on one B200, among other calls (bench.py --op kv): four sequences of
// 100000 to 131072 tokens, 64 query heads on 8 kv heads of 128, 558 MB of cache,
// take 137 to 141 us, 4.0 TB/s (0.60 of a copy's rate; 147 to 157 us apart); 48
// uneven ones up to 4096, 115 MB, 43 us (49 apart).  Bound by issue: about
// 400 instructions a tile of 2304 bytes, 13 for every eight codes (3 for a pair
// in both halves of a register, and a shift), at three quarters of the issue
// rate inside the loop; about 8 us of a call go to finding the run, the first
// loads and joining.  A loop with the ring's slots in variables took a tenth more
// for the first, partial results in rows (whose stores meet the same banks) 5 us
// more, and a run found by every warp in 64-bit numbers 4 us more.
#include <algorithm>

#include "kv_device.h"
#include "ptx.h"

namespace dsq {

namespace {

// A tiling: head dimension, tiles of eight query rows, warps of a CTA, tiles
// of a warp's ring.  Shared memory of a warp: the ring, whose space takes the
// warp's last partial result when it is done, and its first partial result.
template <int D_, int NT_, int NW_, int RING_>
struct Split {
    static constexpr int D = D_, NT = NT_, NW = NW_, RING = RING_;
    static constexpr int R = 8 * NT;
    static constexpr int kTile = kv_tile_bytes(D);
    static constexpr int kPart = (R * (D + 2) * 4 + 127) / 128 * 128;  // the swizzles count on 128-byte rings
    static constexpr int kWarp = RING * kTile + kPart;
    static constexpr int kSmem = NW * kWarp;
    static_assert(RING * kTile >= kPart && RING % 2 == 0 && kSmem <= 224 * 1024, "shared memory of a CTA");
};

struct SplitParams {
    KvAttend a;
    float *parts;
    KvCarry *carries;
    int min_run;  // least units of a CTA's run; 0: a job a CTA
    int shift;    // units of 32 << shift tokens: 0 unless their number could pass 31 bits
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
// Where 16-byte chunk c of a token's row of codes goes in a ring tile, such
// that the fragment loads below meet no bank twice.  Keys: the rows in the
// order of M; values: rows t at t / 4 + 4 (t % 4).
template <int D>
__device__ __forceinline__ int key_at(int t, int c) {
    const int row = (t >> 2) * 2 + (t & 1) + ((t & 2) << 2);
    return row * (D / 2) + (D == 256 ? c ^ (row & 1) : c) * 16;
}
template <int D>
__device__ __forceinline__ int value_at(int t, int c) {
    const int row = (t >> 2) + 4 * (t & 3);
    return kv_codes(D, 1) + row * (D / 2) + (D == 256 ? c ^ (2 * (t >> 2)) : D == 128 ? c ^ (2 * (t >> 3)) : c) * 16;
}

// A lane's part in copying tiles to the ring, 16-byte chunk `lane` of every 512
// bytes: where it goes in a tile.
template <int D>
struct Copy {
    static constexpr int kRow = D / 32, N = D / 64;  // chunks of a token's row; of a lane's in K, and in V
    uint32_t key[N], value[N], words;
    __device__ __forceinline__ Copy(uint32_t ring, int lane) {
#pragma unroll
        for (int i = 0; i < N; i++) {
            key[i] = ring + key_at<D>((lane + 32 * i) / kRow, lane % kRow);
            value[i] = ring + value_at<D>((lane + 32 * i) / kRow, lane % kRow);
        }
        words = ring + kv_words(D, 0) + lane * 16;
    }
    __device__ __forceinline__ void start(uint32_t at, const uint8_t *src, int lane) const {
#pragma unroll
        for (int i = 0; i < N; i++) {
            cp_async16(key[i] + at, src + i * 512);
            cp_async16(value[i] + at, src + kv_codes(D, 1) + i * 512);
        }
        if (lane < D / 8) cp_async16(words + at, src + kv_words(D, 0));
    }
};

// The jobs of a sequence.
struct Jobs : KvSeq {
    int lo, units, tiles;  // first token any query sees, units of a job, row tiles
    int weight;            // units of all of the sequence's jobs
};
template <int R>
__device__ __forceinline__ Jobs jobs_of(const KvAttend &a, int b, int shift) {
    Jobs j;
    static_cast<KvSeq &>(j) = kv_seq(a, b);
    j.lo = a.window ? max(0, j.len - j.rows - a.window + 1) : 0;
    j.units = max(1, ((j.len + (32 << shift) - 1) >> (5 + shift)) - (j.lo >> (5 + shift)));
    j.tiles = (int)(((uint32_t)(j.rows * a.share) + R - 1) / R);
    j.weight = a.c.kv_heads * j.tiles * j.units;
    return j;
}

// A CTA's run: `size` units from unit `first` on, in or behind sequence b, the
// units before which are `before`; all runs but the last are `of` units long.
struct Run {
    int first, before, of, b, size;
};

// Finds it (one warp).  Where a CTA takes one job, job numbers are searched
// instead of unit numbers, and units counted from the sequence's first.
template <int R>
__device__ __forceinline__ void find_run(const SplitParams &p, Run &run) {
    const KvAttend &a = p.a;
    const int lane = threadIdx.x & 31;
    auto weight = [&](int b) {
        if (b >= a.batch) return 0;
        const Jobs j = jobs_of<R>(a, b, p.shift);
        return p.min_run ? j.weight : a.c.kv_heads * j.tiles;
    };
    const int w0 = weight(lane);  // of the first 32 sequences, for both passes
    int first = blockIdx.x, of = 1, total = 0;
    if (p.min_run) {
        total = w0;
#pragma unroll 1
        for (int b = lane + 32; b < a.batch; b += 32) total += weight(b);
        total = (int)__reduce_add_sync(kFull, (uint32_t)total);
        of = max((int)(((uint32_t)total + gridDim.x - 1) / gridDim.x), p.min_run);
        first = (int)min((uint32_t)total, (uint32_t)first * (uint32_t)of);
    }
    int b = a.batch, before = 0;
#pragma unroll 1
    for (int b0 = 0; b0 < a.batch; b0 += 32) {
        const int w = b0 == 0 ? w0 : weight(b0 + lane);
        int sum = w;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int up = __shfl_up_sync(kFull, sum, m);
            if (lane >= m) sum += up;
        }
        const uint32_t past = __ballot_sync(kFull, before + sum > first);
        if (past) {
            const int l = __ffs(past) - 1;
            b = b0 + l;
            before += __shfl_sync(kFull, sum - w, l);
            // A q_start out of order can have more units than 31 bits count:
            // no place in the sequence is taken that is not in it.
            if (a.q_start && (uint32_t)first - (uint32_t)before >= (uint32_t)__shfl_sync(kFull, w, l)) b = a.batch;
            break;
        }
        before += __shfl_sync(kFull, sum, 31);
    }
    int size = 0;
    if (b < a.batch) {
        size = min(of, total - first);
        if (!p.min_run) {
            size = jobs_of<R>(a, b, p.shift).units;
            first = (first - before) * size;
            before = 0;
        }
    }
    if (lane == 0) run = {first, before, of, b, size};
}

// A partial result in shared memory: a warp's accumulators as they are, two
// floats a lane, then the rows' maxima and sums.
template <int D>
__device__ __forceinline__ int part_at(int nc, int i, int lane) { return ((nc * (D / 16) + i) * 32 + lane) * 2; }

template <typename S, typename T>
__global__ void __launch_bounds__(S::NW * 32, 1) split_kernel(const __grid_constant__ SplitParams p) {
    constexpr int D = S::D, NT = S::NT, NW = S::NW, RING = S::RING, R = S::R;
    constexpr int KW = D / 32;   // 8-code words of a lane's key dimensions
    constexpr int VW = D / 64;   // and of its value dimensions
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int head_valid[NW], head_ended[NW], tail_valid[NW];
    __shared__ int job_id[NW][3];      // (b, kv head, row tile) of each warp's last job
    __shared__ Run run;
    __shared__ int job_end[NW];        // unit behind the last job's last
    const KvAttend &a = p.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, jj = lane & 3;
    const uint32_t ring = smem_u32(smem) + warp * S::kWarp;
    float *const head_part = reinterpret_cast<float *>(smem + warp * S::kWarp + RING * S::kTile);
    const Copy<D> copy(ring, lane);
    // This lane's fragments in a ring tile.
    const uint32_t key_row = ring + r * (D / 2) + (D == 256 ? 2 * jj ^ (r & 1) : jj) * (D == 64 ? 8 : 16);
    const uint32_t key_word = ring + kv_words(D, 0) + jj * (D / 4) / kKvGroup * 32 + (4 * (r >> 1) + (r & 1)) * 2;
    const uint32_t value_row = ring + kv_codes(D, 1) + jj * (D / 2) +
                               (D == 64 ? r * 4 : D == 128 ? ((r >> 1) ^ (2 * (jj >> 1))) * 16 + (r & 1) * 8 : (r ^ (2 * jj)) * 16);
    const uint32_t value_word = ring + kv_words(D, 1) + r * (D / 8) / kKvGroup * 32 + jj * 8;
    float *const tail_part = reinterpret_cast<float *>(smem + warp * S::kWarp);

    kv_after_previous();

    if (threadIdx.x == 0 && p.min_run) p.carries[blockIdx.x].valid = 0;
    if (warp == 0) find_run<R>(p, run);
    if (lane == 0) head_valid[warp] = head_ended[warp] = tail_valid[warp] = 0;
    __syncthreads();

    // This warp's run [u, u_end) of the units of all jobs; `before` of them are
    // those of the sequences before b.
    int b = run.b, before = run.before;
    const int mine = (run.size + NW - 1) / NW, skip = min(run.size, warp * mine);
    int u = run.first + skip;
    const int u_end = u + min(mine, run.size - skip);
    while (u < u_end && b < a.batch) {
        const Jobs j = jobs_of<R>(a, b, p.shift);
        if ((uint32_t)u - (uint32_t)before >= (uint32_t)j.weight) {
            before = (int)((uint32_t)before + (uint32_t)j.weight);
            b++;
            continue;
        }
        // The job, and the units of it that are in this run.
        const int rel = u - before, job = (int)((uint32_t)rel / (uint32_t)j.units);
        const int head = j.tiles == 1 ? job : (int)((uint32_t)job / (uint32_t)j.tiles), qt = job - head * j.tiles;
        const int first = rel - job * j.units;
        const int last = min(j.units, first + (u_end - u));  // units [first, last) of the job
        const int rho0 = qt * R, rho1 = min(rho0 + R, j.rows * a.share) - 1;
        const int2 seen0 = seen_by(a, j, rho0), seen1 = seen_by(a, j, rho1);
        const int lo_any = seen0.x, hi_any = seen1.y, lo_all = seen1.x, hi_all = seen0.y;
        // Tiles of 16 tokens: those of the units, less what no row sees.
        const int unit0 = j.lo >> (5 + p.shift);
        const int tile0 = max((unit0 + first) << (1 + p.shift), lo_any / 32 * 2);
        const int tile1 = min((unit0 + last) << (1 + p.shift), (max(hi_any, 0) + 15) / 16);

        // Page numbers of the next 64 table columns, one per lane and register.
        int col = a.tiles_by.div(tile0), col0 = col, in_page = tile0 - col * a.c.page_tiles;
        const int32_t *row = a.page_table + (int64_t)b * a.table_pages;
        auto pages_from = [&](int c) { return c + lane < a.table_pages ? row[c + lane] : -1; };
        int pages = pages_from(col0), pages_next = pages_from(col0 + 32);
        uint4 raw[NT][KW];
#pragma unroll
        for (int n = 0; n < NT; n++) {
            const uint4 *from = reinterpret_cast<const uint4 *>(
                (const T *)a.q + row_at(a, j, head, min(rho0 + 8 * n + r, rho1), a.q_token, a.q_head) + jj * (D / 4));
#pragma unroll
            for (int w = 0; w < KW; w++) raw[n][w] = from[w];
        }
        const uint8_t *const base = a.c.cache + (int64_t)head * a.c.page_tiles * S::kTile + lane * 16;
        const uint8_t *src = nullptr;     // this lane's chunk of the next tile
        int left = tile1 - tile0, rest = 0;  // tiles to copy; of them on this page
        bool exists = false;              // the page
        auto turn = [&] {
            const int page = __shfl_sync(kFull, pages, col - col0);
            exists = (uint32_t)page < (uint32_t)a.c.pages;
            if (exists) src = base + ((int64_t)page * a.c.kv_heads * a.c.page_tiles + in_page) * S::kTile;
            rest = a.c.page_tiles - in_page;
            in_page = 0;
            if (++col - col0 == 32) {
                col0 += 32;
                pages = pages_next;
                pages_next = pages_from(col0 + 32);
            }
        };
        bool there[RING];  // whether a ring tile holds a tile of the cache
        auto issue = [&](int slot) {
            if (rest == 0 && left > 0) turn();
            there[slot] = exists && left > 0;
            if (there[slot]) copy.start(slot * S::kTile, src, lane);
            cp_async_commit();
            src += S::kTile;
            rest--;
            left--;
        };
#pragma unroll
        for (int i = 0; i < RING; i++) issue(i);

        // Queries: the B operand of the scores, column n = r.
        uint32_t q[D / 16][NT][2];
        float scale[NT][2];  // of the accumulator's columns 2 jj, 2 jj + 1; positive, the sign is the queries'
        const uint32_t sign = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
#pragma unroll
        for (int n = 0; n < NT; n++) {
            uint4(&x)[KW] = raw[n];
            int up = 0;
            if constexpr (!std::is_same<T, __half>::value) {  // four lanes share the row
                uint32_t top = 0;
#pragma unroll
                for (int w = 0; w < KW; w++) top = top_bits(x[w], top);
                top = max(top, __shfl_xor_sync(kFull, top, 1));
                up = up_of(max(top, __shfl_xor_sync(kFull, top, 2)));
            }
            query_codes_order<T, KW>(x, up);
            const float factor = fmaxf(fabsf(a.scale_log2) * exponent(-up), 1.17549435e-38f);  // not 0: -inf times it is -inf
#pragma unroll
            for (int w = 0; w < KW; w++) {
                q[2 * w][n][0] = x[w].x ^ sign;
                q[2 * w][n][1] = x[w].y ^ sign;
                q[2 * w + 1][n][0] = x[w].z ^ sign;
                q[2 * w + 1][n][1] = x[w].w ^ sign;
            }
#pragma unroll
            for (int c = 0; c < 2; c++) {
                scale[n][c] = __shfl_sync(kFull, factor, (2 * jj + c) * 4);
            }
        }

        float o[D / 16][NT][4], m[NT][2], l[NT][2];
#pragma unroll
        for (int i = 0; i < D / 16; i++)
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int k = 0; k < 4; k++) o[i][n][k] = 0.0f;
#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                m[n][c] = kNoMax;
                l[n][c] = 0.0f;
            }

        auto unit = [&](int tile, int at) {  // tiles `tile`, + 1, in the ring from `at` on
            cp_async_wait<RING - 2>();
            __syncwarp();
            const int t0 = tile * 16;
            const bool masked = t0 < lo_all || t0 + 32 > hi_all || !there[at] || !there[at + 1];
            float s[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const uint32_t buf = (at + h) * S::kTile;
                uint32_t kw[2][KW];
#pragma unroll
                for (int e = 0; e < 2; e++) {
                    const uint32_t at_row = key_row + buf + 8 * e * (D / 2);
                    if constexpr (D == 64)
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(kw[e][0]), "=r"(kw[e][1]) : "r"(at_row));
                    else {
#pragma unroll
                        for (int c = 0; c < KW / 4; c++) {  // at 256 dimensions chunk 2 jj + c, in odd rows 2 jj + 1 - c
                            const uint4 v = lds128(c == 0 ? at_row : (at_row ^ 16));
                            kw[e][4 * c] = v.x;
                            kw[e][4 * c + 1] = v.y;
                            kw[e][4 * c + 2] = v.z;
                            kw[e][4 * c + 3] = v.w;
                        }
                    }
                }
                constexpr int G = D == 256 ? 2 : 1;  // groups of a lane's key dimensions
#pragma unroll
                for (int g = 0; g < G; g++) {
                    uint16_t p0, p1;
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p0) : "r"(key_word + buf + g * 32));
                    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(p1) : "r"(key_word + buf + g * 32 + 4));
                    const Decode d0(prmt(p0, p0, 0x1010)), d1(prmt(p1, p1, 0x1010));
#pragma unroll
                    for (int w = g * (KW / G); w < (g + 1) * (KW / G); w++) {
                        const uint32_t x = kw[0][w], y = kw[1][w];
                        const uint32_t f0[4] = {d0.low(x), d1.low(y), d0.high(x), d1.high(y)};
                        const uint32_t f1[4] = {d0.low(x >> 8), d1.low(y >> 8), d0.high(x >> 8), d1.high(y >> 8)};
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            if (w == 0) mma16816_zero(s[h][n], f0, q[0][n][0], q[0][n][1]);
                            else mma16816(s[h][n], f0, q[2 * w][n][0], q[2 * w][n][1]);
                            mma16816(s[h][n], f1, q[2 * w + 1][n][0], q[2 * w + 1][n][1]);
                        }
                    }
                }
            }
            uint2 vp[2];
#pragma unroll
            for (int h = 0; h < 2; h++)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                             : "=r"(vp[h].x), "=r"(vp[h].y)
                             : "r"(value_word + (at + h) * S::kTile));
            if (masked) {
                // Column c of s is k % 2, its token tok + 2 (k / 2).  A NaN
                // value must reach the rows that see it alone: its scale
                // becomes 0 and those rows' scores NaN.  Tokens that no row
                // sees, which may be anything, get scale 0.
                int2 seen[NT][2];
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int c = 0; c < 2; c++) seen[n][c] = seen_by(a, j, min(rho0 + 8 * n + 2 * jj + c, rho1));
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    uint32_t bad = 0;
                    uint32_t w[2] = {vp[h].x, vp[h].y};
#pragma unroll
                    for (int i = 0; i < 4; i++) {
                        const int t = t0 + 16 * h + 4 * jj + i;
                        const bool use = there[at + h] && t >= lo_any && t < hi_any;
                        const bool nan = ((w[i / 2] >> (16 * (i % 2))) & 0x7c00u) == 0x7c00u;
                        if (!use || nan) w[i / 2] &= i % 2 ? 0x0000ffffu : 0xffff0000u;
                        if (use && nan) bad |= 1u << (4 * jj + i);
                    }
                    vp[h] = make_uint2(w[0], w[1]);
                    bad = __reduce_or_sync(kFull, bad);
#pragma unroll
                    for (int n = 0; n < NT; n++)
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const int i = 4 * (r >> 1) + (r & 1) + (k & 2), t = t0 + 16 * h + i;
                            if (!there[at + h] || t < seen[n][k & 1].x || t >= seen[n][k & 1].y) s[h][n][k] = -INFINITY;
                            else if (bad >> i & 1u) s[h][n][k] = NAN;
                        }
                }
            }
            bool raise = false;
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    top[n][c] = scale[n][c] * fmaxf(fmaxf(s[0][n][c], s[0][n][2 + c]), fmaxf(s[1][n][c], s[1][n][2 + c]));
                    raise |= top[n][c] > m[n][c] + (kLift + kLazy);
                }
            if (__any_sync(kFull, raise)) {
#pragma unroll
                for (int n = 0; n < NT; n++)
#pragma unroll
                    for (int c = 0; c < 2; c++) {
                        float x = top[n][c];
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 4));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 8));
                        x = fmaxf(x, __shfl_xor_sync(kFull, x, 16));
                        x = fmaxf(x - kLift, m[n][c]);
                        const float keep = ex2(m[n][c] - x);
                        m[n][c] = x;
                        l[n][c] *= keep;
#pragma unroll
                        for (int i = 0; i < D / 16; i++) {
                            o[i][n][c] *= keep;
                            o[i][n][2 + c] *= keep;
                        }
                    }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int h = 0; h < 2; h++)
#pragma unroll
                for (int n = 0; n < NT; n++) {
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        s[h][n][k] = ex2(fmaf(s[h][n][k], scale[n][k & 1], -m[n][k & 1]));
                        l[n][k & 1] += s[h][n][k];
                    }
                    pb[h][n][0] = movmatrix_t(pack_h2(s[h][n][0], s[h][n][1]));
                    pb[h][n][1] = movmatrix_t(pack_h2(s[h][n][2], s[h][n][3]));
                }
#pragma unroll
            for (int h = 0; h < 2; h++) {
                uint32_t vw[4][VW];
#pragma unroll
                for (int i = 0; i < 4; i++) {  // token 4 jj + i: row jj + 4 i
                    const uint32_t at_row = value_row + (at + h) * S::kTile + 4 * i * (D / 2);
                    if constexpr (D == 64)
                        vw[i][0] = lds32(at_row);
                    else if constexpr (D == 128)
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(vw[i][0]), "=r"(vw[i][1]) : "r"(at_row));
                    else {
                        const uint4 v = lds128(at_row);
                        vw[i][0] = v.x;
                        vw[i][1] = v.y;
                        vw[i][2] = v.z;
                        vw[i][3] = v.w;
                    }
                }
                const Decode d0(vp[h].x), d1(vp[h].y);
#pragma unroll
                for (int w = 0; w < VW; w++) {
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        const uint32_t sel = half ? 0x7632u : 0x5410u;
                        const uint32_t x = prmt(vw[0][w], vw[1][w], sel), y = prmt(vw[2][w], vw[3][w], sel);
                        const uint32_t f0[4] = {d0.low(x), d0.high(x), d1.low(y), d1.high(y)};
                        const uint32_t f1[4] = {d0.low(x >> 8), d0.high(x >> 8), d1.low(y >> 8), d1.high(y >> 8)};
#pragma unroll
                        for (int n = 0; n < NT; n++) {
                            mma16816(o[4 * w + 2 * half][n], f0, pb[h][n][0], pb[h][n][1]);
                            mma16816(o[4 * w + 2 * half + 1][n], f1, pb[h][n][0], pb[h][n][1]);
                        }
                    }
                }
            }
            __syncwarp();
            issue(at);
            issue(at + 1);
        };
        for (int tile = tile0; tile < tile1; tile += RING) {
#pragma unroll
            for (int i = 0; i < RING; i += 2)
                if (tile + i < tile1) unit(tile + i, i);
        }
        cp_async_wait<0>();
        __syncwarp();

#pragma unroll
        for (int n = 0; n < NT; n++)
#pragma unroll
            for (int c = 0; c < 2; c++) {
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 4);
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 8);
                l[n][c] += __shfl_xor_sync(kFull, l[n][c], 16);
            }
        const bool begins = first == 0, ends = last == j.units;
        if (begins && ends) {
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const int rho = rho0 + 8 * n + 2 * jj + c;
                    if (rho > rho1) continue;
                    const float inv = l[n][c] == 0.0f ? 0.0f : 1.0f / l[n][c];
                    T *dst = (T *)a.out + row_at(a, j, head, rho, a.out_token, a.out_head) + r * (D / 8);
#pragma unroll
                    for (int i = 0; i < D / 16; i += 4)
                        *reinterpret_cast<uint4 *>(dst + 2 * i) =
                            make_uint4(pack_out<T>(o[i][n][c] * inv, o[i][n][2 + c] * inv),
                                       pack_out<T>(o[i + 1][n][c] * inv, o[i + 1][n][2 + c] * inv),
                                       pack_out<T>(o[i + 2][n][c] * inv, o[i + 2][n][2 + c] * inv),
                                       pack_out<T>(o[i + 3][n][c] * inv, o[i + 3][n][2 + c] * inv));
                    if (a.lse && r == 0)
                        a.lse[row_at(a, j, head, rho, a.q_heads, 1)] =
                            lse_of(m[n][c], l[n][c]);
                }
        } else {
            float *dst = begins ? tail_part : head_part;
#pragma unroll
            for (int n = 0; n < NT; n++)
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const int row_n = 8 * n + 2 * jj + c;
#pragma unroll
                    for (int i = 0; i < D / 16; i++)
                        *reinterpret_cast<float2 *>(dst + part_at<D>(2 * n + c, i, lane)) = make_float2(o[i][n][c], o[i][n][2 + c]);
                    if (r == 0) {
                        dst[R * D + row_n] = m[n][c];
                        dst[R * D + R + row_n] = l[n][c];
                    }
                }
            if (lane == 0) {
                if (begins) {
                    tail_valid[warp] = 1;
                    job_id[warp][0] = b;
                    job_id[warp][1] = head;
                    job_id[warp][2] = qt;
                    job_end[warp] = before + (job + 1) * j.units;
                } else {
                    head_valid[warp] = 1;
                    head_ended[warp] = ends;
                }
            }
        }
        u += last - first;
    }
    __syncthreads();

    // What spans warps: chains of partial results, a warp's last (or the CTA's
    // very first) and the first ones of the warps behind it.  The warps share
    // out the chains.
    const uint32_t hv = __ballot_sync(kFull, lane < NW && head_valid[lane % NW]);
    const uint32_t he = __ballot_sync(kFull, lane < NW && head_ended[lane % NW]);
    const uint32_t tv = __ballot_sync(kFull, lane < NW && tail_valid[lane % NW]);
    const int chains = (int)(hv & 1u) + __popc(tv), group = max(1, NW / max(1, chains));
#pragma unroll 1
    for (int c = warp / group; c < chains; c += (NW + group - 1) / group) {
        uint32_t later = tv;
        for (int i = (int)(hv & 1u); i < c; i++) later &= later - 1;
        const int w = (hv & 1u) && c == 0 ? -1 : __ffs(later) - 1;
        const uint32_t heads = hv >> (w + 1), ends = he >> (w + 1);
        const int run_of = __ffs(~heads) - 1, end = __ffs(ends & heads) - 1;
        const bool ended = end >= 0 && end < run_of;
        const int n = (w < 0 ? 0 : 1) + (ended ? end + 1 : run_of);
        auto part = [&](int i) {
            const bool tail = w >= 0 && i == 0;
            const int of = w < 0 ? i : w + i;
            return reinterpret_cast<const float *>(smem + of * S::kWarp + (tail ? 0 : RING * S::kTile));
        };
        const bool whole = w >= 0 && ended;
        KvSeq j = {};
        int head = 0, rho0 = 0;
        float *const to = p.parts + (2 * blockIdx.x + (w < 0 ? 0 : 1)) * kv_part_floats<D, R>();
        if (whole) {
            j = kv_seq(a, job_id[w][0]);
            head = job_id[w][1];
            rho0 = job_id[w][2] * R;
        } else if (w >= 0 && warp % group == 0 && lane == 0) {
            const uint32_t last = min((uint32_t)(job_end[w] - 1) / (uint32_t)run.of, gridDim.x - 1);  // of a q_start out of order it may be anything
            const KvCarry mt = {1, (int)last - (int)blockIdx.x, job_id[w][0], job_id[w][1], job_id[w][2], {}};
            p.carries[blockIdx.x] = mt;
        }
        // Accumulators 4 i0 .. 4 i0 + 3 of row group nc at a time: they share
        // the rows' factors.
        constexpr int kSub = D / 64;
#pragma unroll 1
        for (int item = warp % group; item < 2 * NT * kSub; item += group) {
            const int nc = item / kSub, i0 = item % kSub * 4, row = nc / 2 * 8 + 2 * jj + nc % 2, d = r * (D / 8) + i0 * 2;
            float top = kNoMax, sum = 0.0f;
            float2 x[4] = {};
#pragma unroll 4
            for (int k = 0; k < n; k++) top = fmaxf(top, part(k)[R * D + row]);
#pragma unroll 4
            for (int k = 0; k < n; k++) {
                const float *src = part(k);
                const float f = ex2(src[R * D + row] - top);
                sum += f * src[R * D + R + row];
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const float2 v = *reinterpret_cast<const float2 *>(src + part_at<D>(nc, i0 + i, lane));
                    x[i].x += f * v.x;
                    x[i].y += f * v.y;
                }
            }
            if (whole) {
                if (rho0 + row >= j.rows * a.share) continue;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                *reinterpret_cast<uint4 *>((T *)a.out + row_at(a, j, head, rho0 + row, a.out_token, a.out_head) + d) =
                    make_uint4(pack_out<T>(x[0].x * inv, x[0].y * inv), pack_out<T>(x[1].x * inv, x[1].y * inv),
                               pack_out<T>(x[2].x * inv, x[2].y * inv), pack_out<T>(x[3].x * inv, x[3].y * inv));
                if (a.lse && d == 0) a.lse[row_at(a, j, head, rho0 + row, a.q_heads, 1)] = lse_of(top, sum);
            } else {
                float4 *dst = reinterpret_cast<float4 *>(to + row * D + d);
                dst[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
                dst[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
                if (d == 0) {
                    to[R * D + row] = top;
                    to[R * D + R + row] = sum;
                }
            }
        }
    }
}

template <typename S, typename T>
int launch_split(const KvAttend &a, void *workspace, int sms, cudaStream_t st) {
    // A job a CTA where every job has an SM and at most six units a warp: no
    // joining, one launch (32 jobs of 333 tokens: 10 us, dealt out evenly 12).
    const int64_t most_rows = a.q_start ? a.q_tokens : a.rows_each;
    const int64_t jobs = a.c.kv_heads * (a.q_start ? a.batch + (int64_t)a.q_tokens * a.share / S::R
                                                    : a.batch * ((most_rows * a.share + S::R - 1) / S::R));
    int64_t tokens = (int64_t)a.table_pages * a.c.page_tokens;
    if (a.window) tokens = std::min(tokens, a.window + most_rows);
    const bool one_each = jobs <= sms && tokens / 32 + 2 <= 6 * S::NW;
    int shift = 0;  // 25 at most: fewer than 2^30 tokens, and jobs
    while ((double)a.c.kv_heads * (a.batch + (double)a.q_tokens * a.share / S::R) * ((a.most_tokens >> (5 + shift)) + 2) >= 2147483648.0)
        shift++;
    const SplitParams p = {a, (float *)workspace, kv_carries<S::D, S::R>(workspace), one_each ? 0 : 4, shift};
    auto kernel = split_kernel<S, T>;
    static KvOnce once;
    if (!once.set_smem((const void *)kernel, S::kSmem)) return DSQ_ERR_CUDA;
    const int grid = one_each ? (int)jobs : std::min(sms, kMaxCtas);
    const int rc = kv_launch(kernel, grid, S::NW * 32, S::kSmem, st, p);
    return rc != DSQ_OK || one_each ? rc : launch_join<S::D, S::R, T>(a, p.parts, p.carries, grid, jobs, st);
}

template <typename T>
int launch_of(const KvAttend &a, int head_dim, void *workspace, int sms, cudaStream_t st) {
    // Sixteen rows at once when a job has more than eight: the cache is read
    // and unpacked half as often.
    const bool wide = a.q_tokens / a.batch * a.share > 8;
    if (head_dim == 64)
        return wide ? launch_split<Split<64, 2, 12, 4>, T>(a, workspace, sms, st)
                    : launch_split<Split<64, 1, 16, 4>, T>(a, workspace, sms, st);
    if (head_dim == 128)
        return wide ? launch_split<Split<128, 2, 8, 4>, T>(a, workspace, sms, st)
                    : launch_split<Split<128, 1, 16, 4>, T>(a, workspace, sms, st);
    return launch_split<Split<256, 1, 8, 4>, T>(a, workspace, sms, st);
}

}  // namespace

size_t kv_split_workspace() {
    return std::max(std::max(kv_parts_bytes<64, 16>(), kv_parts_bytes<128, 16>()), kv_parts_bytes<256, 8>());
}

int launch_kv_split(const KvAttend &a, int head_dim, int dtype, void *workspace, int sms, cudaStream_t st) {
    if (dtype == DSQ_DTYPE_F16) return launch_of<__half>(a, head_dim, workspace, sms, st);
    return launch_of<__nv_bfloat16>(a, head_dim, workspace, sms, st);
}

}  // namespace dsq
