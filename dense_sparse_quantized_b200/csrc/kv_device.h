// kv_device.h -- what the attention kernels over the 4-bit cache share: fp16
// arithmetic on packed codes, query rows, and the joining of partial results.
#pragma once
#include "kv.h"

namespace dsq {

constexpr float kNoMax = -3.0e38f;  // a maximum of no scores: finite, so that -inf minus it stays -inf
// Numerators are rounded to fp16, which has them down to 2^-25: a running
// maximum is held kLift below the largest score, so that numerators are 2^7 at
// it and small ones that far from the end of the range (2^-32 of the largest;
// 2^20 tokens at 2^-25.2 beside one that attracts a row lost 2.6 % of its
// output without).  kLazy: log2 of how far they may pass 2^7; 2^15 is fp16's
// last power.
constexpr float kLift = 7.0f;
constexpr float kLazy = 8.0f;
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kMaxCtas = 160;  // workspace slots; the kernels run one CTA per SM, at most this many

__device__ __forceinline__ uint32_t lop_magic(uint32_t w, uint32_t mask, uint32_t magic) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "r"(mask), "r"(magic));  // (w & mask) | magic
    return r;
}
__device__ __forceinline__ uint32_t hadd2u(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t hmul2u(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Scale and zero of a pair of codes: two fp16 scales, and minus 1024 plus
// zero (for codes at the bottom of the halves) or minus 64 plus zero.  The
// difference is an integer of four bits and the scale has seven, so the
// product is exact.
struct Decode {
    uint32_t s, z1024, z64;
    __device__ __forceinline__ explicit Decode(uint32_t words) {
        s = words & 0xfff0fff0u;
        z1024 = lop_magic(words, 0x000f000fu, 0xe400e400u);
        z64 = hadd2u(z1024, 0x63806380u);  // + 960
    }
    // Codes 0 and 4 of eight, and codes 1 and 5; of w >> 8, codes 2 and 6, 3 and 7.
    __device__ __forceinline__ uint32_t low(uint32_t w) const {
        return hmul2u(hadd2u(lop_magic(w, 0x000f000fu, 0x64006400u), z1024), s);
    }
    __device__ __forceinline__ uint32_t high(uint32_t w) const {
        return hmul2u(hadd2u(lop_magic(w, 0x00f000f0u, 0x54005400u), z64), s);
    }
};

template <typename T>
__device__ __forceinline__ uint32_t pack_out(float a, float b) {
    if constexpr (std::is_same<T, __half>::value) return pack_h2(a, b);
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}

// Query rows as fp16.  bf16 rows are scaled by a power of two, 2^up, that
// brings the row's largest magnitude to 2^14, so that fp16 holds what bf16
// did; the scores are multiplied by 2^-up.
__device__ __forceinline__ float exponent(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ uint32_t top_bits(uint4 x, uint32_t top) {  // largest magnitude, as bits
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; i++) top = max(top, max(u[i] & 0x7fffu, (u[i] >> 16) & 0x7fffu));
    return top;
}
__device__ __forceinline__ int up_of(uint32_t top) {
    const int e = (int)(top >> 7);  // biased; 0 for zero, 255 for an infinity or a NaN
    return e == 0 || e == 255 ? 0 : min(127 + 14 - e, 120);
}
// N x 8 elements of a row in the order in which codes unpack: (0, 4), (1, 5),
// (2, 6), (3, 7) of every eight.
template <typename T, int N>
__device__ __forceinline__ void query_codes_order(uint4 (&x)[N], int up) {
#pragma unroll
    for (int w = 0; w < N; w++) {
        if constexpr (!std::is_same<T, __half>::value) {
            uint32_t u[4] = {x[w].x, x[w].y, x[w].z, x[w].w};
#pragma unroll
            for (int i = 0; i < 4; i++)
                u[i] = pack_h2(__uint_as_float(u[i] << 16) * exponent(up), __uint_as_float(u[i] & 0xffff0000u) * exponent(up));
            x[w] = make_uint4(u[0], u[1], u[2], u[3]);
        }
        x[w] = make_uint4(prmt(x[w].x, x[w].z, 0x5410), prmt(x[w].x, x[w].z, 0x7632), prmt(x[w].y, x[w].w, 0x5410),
                          prmt(x[w].y, x[w].w, 0x7632));
    }
}

__device__ __forceinline__ int64_t divide(int64_t n, int d) {  // n >= 0, d > 0
    return n >> 32 ? n / d : (int64_t)((uint32_t)n / (uint32_t)d);
}

// Tokens [x, y) that query row `rho` of a kv head (of the sequence's rows
// times the heads of a group) sees.
__device__ __forceinline__ int2 seen_by(const KvAttend &a, const KvSeq &s, int rho) {
    const int pos = s.len - s.rows + a.share_by.div(rho);
    return make_int2(a.window ? max(0, pos - a.window + 1) : 0, a.causal ? min(s.len, pos + 1) : s.len);
}

// Where that row of kv head `head` lies.
__device__ __forceinline__ int64_t row_at(const KvAttend &a, const KvSeq &s, int head, int rho, int64_t token_stride,
                                          int64_t head_stride) {
    const int i = a.share_by.div(rho);
    return (int64_t)(s.row0 + i) * token_stride + (int64_t)(head * a.share + rho - i * a.share) * head_stride;
}

__device__ __forceinline__ float lse_of(float top, float sum) {
    return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.69314718055994531f;
}

// Partial results.  A job (sequence, kv head, tile of R query rows) whose
// tokens span several CTAs' runs leaves R x D sums, R maxima and R sums of
// numerators in each: in the first part of a CTA's two if the job began
// before the CTA's run, else in the second.  A CTA in whose run a job begins
// that goes on in `more` further CTAs says so in its KvCarry.
struct KvCarry {
    int valid, more, b, head, qt, pad[3];
};
template <int D, int R>
__host__ __device__ constexpr size_t kv_part_floats() { return (size_t)R * (D + 2); }
template <int D, int R>
constexpr size_t kv_parts_bytes() { return kMaxCtas * (2 * kv_part_floats<D, R>() * 4 + sizeof(KvCarry)); }
template <int D, int R>
inline KvCarry *kv_carries(void *workspace) {
    return (KvCarry *)((uint8_t *)workspace + kMaxCtas * 2 * kv_part_floats<D, R>() * 4);
}

// Joins them, always in the same order.  A warp takes N rows; or, of short
// tiles, eight warps take one row and share out its parts (37 parts of 8 rows,
// four heads of 7449 tokens: 22 us for the whole attention with one warp's loop
// over them, 12 us so).
template <int D, int R, int N, bool SHARED, typename T>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ KvAttend a, const float *parts,
                                                   const KvCarry *carries) {
    kv_after_previous();
    constexpr int E = D / 32, S = SHARED ? 8 : 1;  // elements of a lane; warps to a row
    static_assert(!SHARED || N == 1, "");
    const KvCarry c = carries[blockIdx.x];
    if (!c.valid) return;
    const KvSeq s = kv_seq(a, c.b);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = SHARED ? warp : 0;
    const int row0 = SHARED ? blockIdx.y : (blockIdx.y * 8 + warp) * N, left = s.rows * a.share - (c.qt * R + row0);
    if (left <= 0) return;  // the whole block, where it shares
    const float *const at = parts + row0 * D + lane * E, *const ends = parts + R * D + row0;
    auto part = [&](int i) { return (2 * (blockIdx.x + i) + (i == 0 ? 1 : 0)) * kv_part_floats<D, R>(); };
    float top[N], sum[N], x[N][E];
#pragma unroll
    for (int n = 0; n < N; n++) {
        top[n] = kNoMax;
        sum[n] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) x[n][e] = 0.0f;
    }
#pragma unroll 8
    for (int i = mine; i <= c.more; i += S)
#pragma unroll
        for (int n = 0; n < N; n++) top[n] = fmaxf(top[n], ends[part(i) + n]);
#pragma unroll(N == 1 ? 8 : 2)
    for (int i = mine; i <= c.more; i += S) {
        const size_t of = part(i);
        float tops[N], sums[N];
        float2 v[N][E / 2];
#pragma unroll
        for (int n = 0; n < N; n++) {  // all of a part's loads are under way together
            tops[n] = ends[of + n];
            sums[n] = ends[of + R + n];
#pragma unroll
            for (int e = 0; e < E; e += 2) v[n][e / 2] = *reinterpret_cast<const float2 *>(at + of + n * D + e);
        }
#pragma unroll
        for (int n = 0; n < N; n++) {
            const float f = ex2(tops[n] - top[n]);
            sum[n] += sums[n] * f;
#pragma unroll
            for (int e = 0; e < E; e += 2) {
                x[n][e] += v[n][e / 2].x * f;
                x[n][e + 1] += v[n][e / 2].y * f;
            }
        }
    }
    if constexpr (SHARED) {
        __shared__ float found[8][D + 2];
#pragma unroll
        for (int e = 0; e < E; e++) found[warp][e * 32 + lane] = x[0][e];
        if (lane == 0) {
            found[warp][D] = top[0];
            found[warp][D + 1] = sum[0];
        }
        __syncthreads();
        if (warp) return;
        top[0] = kNoMax;
        for (int w = 0; w < 8; w++) top[0] = fmaxf(top[0], found[w][D]);
        sum[0] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) x[0][e] = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; w++) {
            const float f = ex2(found[w][D] - top[0]);
            sum[0] += found[w][D + 1] * f;
#pragma unroll
            for (int e = 0; e < E; e++) x[0][e] += found[w][e * 32 + lane] * f;
        }
    }
#pragma unroll
    for (int n = 0; n < N; n++) {
        if (n >= left) continue;
        const int rho = c.qt * R + row0 + n;
        const float inv = sum[n] == 0.0f ? 0.0f : 1.0f / sum[n];
        T *to = (T *)a.out + row_at(a, s, c.head, rho, a.out_token, a.out_head) + lane * E;
#pragma unroll
        for (int e = 0; e < E; e += 2) reinterpret_cast<uint32_t *>(to)[e / 2] = pack_out<T>(x[n][e] * inv, x[n][e + 1] * inv);
        if (a.lse && lane == 0) a.lse[row_at(a, s, c.head, rho, a.q_heads, 1)] = lse_of(top[n], sum[n]);
    }
}

// jobs: at most so many.  Fewer than half the CTAs: each spans several, and a
// warp takes one row and many parts, else four rows and few parts.
template <int D, int R, typename T>
int launch_join(const KvAttend &a, const float *parts, const KvCarry *carries, int ctas, int64_t jobs, cudaStream_t st) {
    if constexpr (R < 32) return kv_launch(join_kernel<D, R, 1, true, T>, dim3(ctas, R), 256, 0, st, a, parts, carries);
    else if (2 * jobs <= ctas)
        return kv_launch(join_kernel<D, R, 1, false, T>, dim3(ctas, R / 8), 256, 0, st, a, parts, carries);
    else return kv_launch(join_kernel<D, R, 4, false, T>, dim3(ctas, R / 32), 256, 0, st, a, parts, carries);
}

}  // namespace dsq
