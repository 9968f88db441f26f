// kv_cache.cu -- writing the 4-bit key/value cache and reading it back.
//
// Both kernels move bytes: a row of D values (2 D bytes at 16 bits) against
// 9 D / 16 bytes of codes and words.  One thread handles eight dimensions of
// one token's head, keys and values both: one 16-byte access of the rows and
// one 4-byte word of codes each, so a warp's accesses are whole 32-byte
// sectors on both sides.  Four neighbouring threads share a group of 32.
//
// Measured on one B200, among other calls (bench.py --op kv): reading 65536
// tokens of 8 heads of 128 to fp16, 344 MB, takes 61 us, 5.6 TB/s (0.86 of a
// copy's rate; 66 us apart): bound by HBM.  Writing 16384 such tokens of bf16, 86
// MB, takes 27 of the 40 us of writing and reading back: bound by issue (80 %) and
// the ALU pipe, about 20 instructions a value for quotient, rounding, clipping
// and packing.  IEEE divisions and fp64 scales took 57 us for the same.
#include "kv_device.h"

namespace dsq {

namespace {

constexpr int kThreads = 256;

// fp16 and bf16 pairs.
template <typename T>
struct Pairs;
template <>
struct Pairs<__half> {
    static __device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float2 floats(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2 *>(&a)); }
};
template <>
struct Pairs<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t min_nan(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ uint32_t max_nan(uint32_t a, uint32_t b) {
        uint32_t r;
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
        return r;
    }
    static __device__ __forceinline__ float2 floats(uint32_t a) {
        return make_float2(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
    }
};

// The scale of a group: the least multiple n u of u that 15 n u >= hi - lo,
// u the last of its seven bits.  fp32 finds n to within one and compares
// 15 n u (12 bits, exact) with the rounded difference: unless the two are
// equal they differ by more than the rounding did, and where they are equal
// fp64 decides.  The approximate quotient's binade may be the one below or
// above the exact one's: below, n comes out as 129, which stands for 65 of
// twice u; above, as 64, the same scale as 128 of half of u.
__device__ __forceinline__ float scale_of(float lo, float hi) {
    const float range = hi - lo, d = range * (1.0f / 15.0f);
    const int e = max((int)(__float_as_uint(d) >> 23) - 127 - 6, -20);  // u = 2^e
    const float u = exponent(e);
    float n = ceilf(d * exponent(-e));
    auto enough = [&](float k) {
        const float t = 15.0f * k * u;
        return t == range ? (double)t >= (double)hi - (double)lo : t > range;
    };
    if (!enough(n)) n += 1.0f;
    else if (n > 1.0f && enough(n - 1.0f)) n -= 1.0f;
    return fmaxf(n == 129.0f ? 130.0f : n, 1.0f) * u;
}

// (lowest, -highest) of a group's values, held eight each by four neighbouring
// lanes; a NaN stays.
template <typename T>
__device__ __forceinline__ uint32_t ends_of(uint4 raw) {
    using P = Pairs<T>;
    const uint32_t lo2 = P::min_nan(P::min_nan(raw.x, raw.y), P::min_nan(raw.z, raw.w));
    const uint32_t hi2 = P::max_nan(P::max_nan(raw.x, raw.y), P::max_nan(raw.z, raw.w)) ^ 0x80008000u;
    uint32_t ends = P::min_nan(prmt(lo2, hi2, 0x5410), prmt(lo2, hi2, 0x7632));
    ends = P::min_nan(ends, __shfl_xor_sync(kFull, ends, 1));
    return P::min_nan(ends, __shfl_xor_sync(kFull, ends, 2));
}

// x / s rounded to an integer, ties to even, as a float above 3 * 2^22: the
// quotient by Markstein's residual correction of x times the rounded
// reciprocal.  (His theorem, IBM J. Res. Dev. 34, 1990, makes the result the
// correctly rounded quotient where y is within an ulp of it and the residual is
// exact; y may be two ulps and a bit off here, so what follows does without.)
//   y = x inv (1 + e), |e| <= 2^-24, and inv = (1 + e') / s, |e'| <= 2^-24: y is
//   less than 2^-22.9 of itself off.  x - y s is a multiple of the product of
//   the last bits of y and of s (7 bits), fewer than 2^10 of them, so the first
//   fused step is exact.  The second rounds x / s with an error of 2^-24 of the
//   correction, 2^-46 of itself.  (An x far below s gives 0, underflow or not.)
// x (11 bits) over s (7 bits) against a border k + 1/2 (5 bits): two numbers of
// 16 bits at most, equal or 2^-16 apart.  Equal, the border is a float and the
// one nearest to what is rounded; else the result lies on the exact quotient's
// side of it.  `most`: an integer not to be passed.
constexpr float kRound = 12582912.0f;
__device__ __forceinline__ float rounded(float x, float s, float inv, float most) {
    const float y = x * inv;
    return fminf(fmaf(fmaf(-y, s, x), inv, y), most) + kRound;
}

struct Group {
    float s, inv;
    uint32_t word;
};
template <typename T>
__device__ __forceinline__ Group group_of(uint32_t ends) {
    const float2 f = Pairs<T>::floats(ends);
    const float lo = fmaxf(fminf(f.x, 0.0f), -kKvClamp), hi = fminf(fmaxf(-f.y, 0.0f), kKvClamp);
    Group g;
    g.s = scale_of(lo, hi);
    g.inv = __frcp_rn(g.s);
    const uint32_t zero = (uint32_t)(__float_as_int(rounded(-lo, g.s, g.inv, 15.0f)) - __float_as_int(kRound));
    g.word = f.x != f.x || f.y != f.y ? 0x7e00u : (uint32_t)__half_as_ushort(__float2half_rn(g.s)) | zero;
    return g;
}

// The codes of this thread's eight values.  lo's is 0 and none is below;
// rounding up can bring one to 16, which becomes 15.  The floats' bits,
// 16^i times the i-th, are added up as they are: what kRound and zero add to
// them is the same for all.
template <typename T>
__device__ __forceinline__ uint32_t codes_of(uint4 raw, const Group &g, bool clamp) {
    if (g.word == 0x7e00u) return 0;
    const uint32_t zero = g.word & 15u, v[4] = {raw.x, raw.y, raw.z, raw.w};
    const float most = 15.0f - (float)zero;
    uint32_t codes = (zero - (uint32_t)__float_as_int(kRound)) * 0x11111111u;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float2 x = Pairs<T>::floats(v[i / 2]);
        if (clamp) {  // infinities have no quotient
            x.x = fminf(fmaxf(x.x, -kKvClamp), kKvClamp);
            x.y = fminf(fmaxf(x.y, -kKvClamp), kKvClamp);
        }
        codes += (uint32_t)__float_as_int(rounded(x.x, g.s, g.inv, most)) << (4 * i);
        codes += (uint32_t)__float_as_int(rounded(x.y, g.s, g.inv, most)) << (4 * i + 4);
    }
    return codes;
}

// Where the slot's token lies: its tile, and its row in it.
struct Place {
    int64_t tile;
    int row;
};
template <int D>
__device__ __forceinline__ Place place_of(const KvView &c, int slot, int head) {
    const int page = c.page_by.div(slot), off = slot - page * c.page_tokens;
    return {kv_tile_at(c, D, page, head, off), off % kKvTile};
}

struct RowsIn {
    const void *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ KvView c, uint8_t *cache,
                                                          const __grid_constant__ RowsIn r, const int64_t *slots,
                                                          int64_t tokens) {
    constexpr int kLanes = D / 8;
    kv_after_previous();
    const int64_t t0 = (int64_t)blockIdx.x * (kThreads / kLanes);  // the block's first token
    const int t = threadIdx.x / kLanes, dim = (threadIdx.x % kLanes) * 8, head = blockIdx.y;
    int64_t slot = -1;
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (t < tokens - t0) {
        k = *reinterpret_cast<const uint4 *>((const T *)r.k + t0 * r.k_token + head * r.k_head + t * r.k_token + dim);
        v = *reinterpret_cast<const uint4 *>((const T *)r.v + t0 * r.v_token + head * r.v_head + t * r.v_token + dim);
        slot = slots[t0 + t];
    }
    // Even lanes work out the key group's scale and zero, odd ones the value
    // group's, for both.
    const uint32_t ke = ends_of<T>(k), ve = ends_of<T>(v);
    const bool odd = threadIdx.x & 1;
    const Group mine = group_of<T>(odd ? ve : ke);
    Group theirs;
    theirs.s = __shfl_xor_sync(kFull, mine.s, 1);
    theirs.inv = __shfl_xor_sync(kFull, mine.inv, 1);
    theirs.word = __shfl_xor_sync(kFull, mine.word, 1);
    const Group kg = odd ? theirs : mine, vg = odd ? mine : theirs;
    const uint32_t kw = kg.word, vw = vg.word;
    auto outside = [](uint32_t ends) {
        const float2 f = Pairs<T>::floats(ends);
        return f.x < -kKvClamp || f.y < -kKvClamp;
    };
    uint32_t kc, vc;
    if (__any_sync(kFull, outside(ke) || outside(ve))) {
        kc = codes_of<T>(k, kg, true);
        vc = codes_of<T>(v, vg, true);
    } else {
        kc = codes_of<T>(k, kg, false);
        vc = codes_of<T>(v, vg, false);
    }
    if ((uint64_t)slot >= (uint64_t)c.slots) return;
    const Place at = place_of<D>(c, (int)slot, head);
    uint8_t *codes = cache + at.tile + at.row * (D / 2) + dim / 2;
    *reinterpret_cast<uint32_t *>(codes + kv_codes(D, 0)) = kc;
    *reinterpret_cast<uint32_t *>(codes + kv_codes(D, 1)) = vc;
    if (dim % kKvGroup == 0) {
        uint8_t *words = cache + at.tile + (dim / kKvGroup * kKvTile + at.row) * 2;
        *reinterpret_cast<uint16_t *>(words + kv_words(D, 0)) = (uint16_t)kw;
        *reinterpret_cast<uint16_t *>(words + kv_words(D, 1)) = (uint16_t)vw;
    }
}

// Eight values of the cache, exact as fp16.
template <typename T>
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t word, T *to) {
    const Decode d(prmt(word, word, 0x1010));
    const uint32_t x[4] = {d.low(codes), d.high(codes), d.low(codes >> 8), d.high(codes >> 8)};  // (0, 4) (1, 5) (2, 6) (3, 7)
    const uint32_t h[4] = {prmt(x[0], x[1], 0x5410), prmt(x[2], x[3], 0x5410), prmt(x[0], x[1], 0x7632), prmt(x[2], x[3], 0x7632)};
    if constexpr (std::is_same<T, __half>::value) {
        *reinterpret_cast<uint4 *>(to) = make_uint4(h[0], h[1], h[2], h[3]);
    } else {
        float2 f[4];
#pragma unroll
        for (int i = 0; i < 4; i++) f[i] = __half22float2(*reinterpret_cast<const __half2 *>(&h[i]));
        if constexpr (sizeof(T) == 4) {
            reinterpret_cast<float4 *>(to)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
            reinterpret_cast<float4 *>(to)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
        } else {
            *reinterpret_cast<uint4 *>(to) = make_uint4(pack_out<T>(f[0].x, f[0].y), pack_out<T>(f[1].x, f[1].y),
                                                        pack_out<T>(f[2].x, f[2].y), pack_out<T>(f[3].x, f[3].y));
        }
    }
}

struct RowsOut {
    void *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};

// N tokens a thread, whose loads are under way together: four where that still
// leaves every SM eight blocks (64k tokens of 8 heads: 61 us against 84 with
// one), one below (777 tokens of 3 heads: 2.4 us against 3.9 with four).
template <int D, int N, typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ KvView c, const __grid_constant__ RowsOut r,
                                                        const int64_t *slots, int64_t tokens) {
    constexpr int kLanes = D / 8, kStep = kThreads / kLanes;
    kv_after_previous();
    const int64_t t0 = (int64_t)blockIdx.x * (kStep * N) + threadIdx.x / kLanes;
    const int dim = (threadIdx.x % kLanes) * 8, head = blockIdx.y;
    int64_t slot[N];
    uint32_t kc[N], vc[N], kw[N], vw[N];
#pragma unroll
    for (int i = 0; i < N; i++) slot[i] = t0 + i * kStep < tokens ? slots[t0 + i * kStep] : -1;
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (slot[i] < 0 || slot[i] >= c.slots) continue;
        const Place at = place_of<D>(c, (int)slot[i], head);
        const uint8_t *codes = c.cache + at.tile + at.row * (D / 2) + dim / 2;
        const uint8_t *words = c.cache + at.tile + (dim / kKvGroup * kKvTile + at.row) * 2;
        kc[i] = *reinterpret_cast<const uint32_t *>(codes + kv_codes(D, 0));
        vc[i] = *reinterpret_cast<const uint32_t *>(codes + kv_codes(D, 1));
        kw[i] = *reinterpret_cast<const uint16_t *>(words + kv_words(D, 0));
        vw[i] = *reinterpret_cast<const uint16_t *>(words + kv_words(D, 1));
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (slot[i] < 0 || slot[i] >= c.slots) continue;
        const int64_t t = t0 + i * kStep;
        if (r.k) decode8(kc[i], kw[i], (T *)r.k + t * r.k_token + head * r.k_head + dim);
        if (r.v) decode8(vc[i], vw[i], (T *)r.v + t * r.v_token + head * r.v_head + dim);
    }
}

int check_rows(const dsq_kv_rows *r, bool both) {
    if (!r || (both ? !r->k || !r->v : !r->k && !r->v)) return DSQ_ERR_INVALID_ARG;
    if (r->dtype < DSQ_DTYPE_F16 || r->dtype > DSQ_DTYPE_F32) return DSQ_ERR_INVALID_ARG;
    if (!kv_aligned(r->k, 16) || !kv_aligned(r->v, 16)) return DSQ_ERR_INVALID_ARG;
    if (!kv_multiple8(r->k_token) || !kv_multiple8(r->k_head) || !kv_multiple8(r->v_token) || !kv_multiple8(r->v_head))
        return DSQ_ERR_INVALID_ARG;
    return DSQ_OK;
}

// The grid of both kernels: `step` tokens a block along x, kv heads along y.
int grid_for(int64_t tokens, int heads, int step, dim3 *grid) {
    const int64_t blocks = (tokens + step - 1) / step;
    if (blocks >= ((int64_t)1 << 31) || heads > 65535) return DSQ_ERR_UNSUPPORTED;
    *grid = dim3((unsigned)blocks, (unsigned)heads);
    return DSQ_OK;
}

template <int D>
int launch_append(dim3 grid, const KvView &c, void *cache, const dsq_kv_rows *r, const int64_t *slots, int64_t tokens,
                  cudaStream_t st) {
    const RowsIn in = {r->k, r->v, r->k_token, r->k_head, r->v_token, r->v_head};
    if (r->dtype == DSQ_DTYPE_F16)
        return kv_launch(append_kernel<D, __half>, grid, kThreads, 0, st, c, (uint8_t *)cache, in, slots, tokens);
    return kv_launch(append_kernel<D, __nv_bfloat16>, grid, kThreads, 0, st, c, (uint8_t *)cache, in, slots, tokens);
}

template <int D, int N>
int launch_read(const KvView &c, const dsq_kv_rows *r, const int64_t *slots, int64_t tokens, cudaStream_t st) {
    dim3 grid;
    const int rc = grid_for(tokens, c.kv_heads, N * kThreads * 8 / D, &grid);
    if (rc != DSQ_OK) return rc;
    const RowsOut out = {r->k, r->v, r->k_token, r->k_head, r->v_token, r->v_head};
    if (r->dtype == DSQ_DTYPE_F16) return kv_launch(read_kernel<D, N, __half>, grid, kThreads, 0, st, c, out, slots, tokens);
    if (r->dtype == DSQ_DTYPE_BF16)
        return kv_launch(read_kernel<D, N, __nv_bfloat16>, grid, kThreads, 0, st, c, out, slots, tokens);
    return kv_launch(read_kernel<D, N, float>, grid, kThreads, 0, st, c, out, slots, tokens);
}

}  // namespace

}  // namespace dsq

using namespace dsq;

extern "C" int dsq_kv_bytes(const dsq_kv_desc *d, size_t *bytes) {
    if (!bytes) return DSQ_ERR_INVALID_ARG;
    const int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    *bytes = (size_t)d->pages * d->kv_heads * (d->page_tokens / kKvTile) * kv_tile_bytes(d->head_dim);
    return DSQ_OK;
}

extern "C" int dsq_kv_append(const dsq_kv_desc *d, void *cache, const dsq_kv_rows *rows, const int64_t *slots,
                             int64_t tokens, void *stream) {
    int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    if (tokens < 0) return DSQ_ERR_INVALID_ARG;
    if (tokens == 0 || d->pages == 0) return DSQ_OK;
    if (!cache || !slots || !kv_aligned(cache, 128) || !kv_aligned(slots, 8)) return DSQ_ERR_INVALID_ARG;
    if ((rc = check_rows(rows, true)) != DSQ_OK) return rc;
    if (rows->dtype == DSQ_DTYPE_F32) return DSQ_ERR_UNSUPPORTED;
    dim3 grid;
    if ((rc = grid_for(tokens, d->kv_heads, kThreads * 8 / d->head_dim, &grid)) != DSQ_OK) return rc;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    const KvView c = kv_view(d, cache);
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->head_dim == 64) return launch_append<64>(grid, c, cache, rows, slots, tokens, st);
    if (d->head_dim == 128) return launch_append<128>(grid, c, cache, rows, slots, tokens, st);
    return launch_append<256>(grid, c, cache, rows, slots, tokens, st);
}

extern "C" int dsq_kv_read(const dsq_kv_desc *d, const void *cache, const dsq_kv_rows *rows, const int64_t *slots,
                           int64_t tokens, void *stream) {
    int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    if (tokens < 0) return DSQ_ERR_INVALID_ARG;
    if (tokens == 0 || d->pages == 0) return DSQ_OK;
    if (!cache || !slots || !kv_aligned(cache, 128) || !kv_aligned(slots, 8)) return DSQ_ERR_INVALID_ARG;
    if ((rc = check_rows(rows, false)) != DSQ_OK) return rc;
    if ((rows->k && !kv_rows_apart(tokens, d->kv_heads, rows->k_token, rows->k_head, d->head_dim)) ||
        (rows->v && !kv_rows_apart(tokens, d->kv_heads, rows->v_token, rows->v_head, d->head_dim)))
        return DSQ_ERR_INVALID_ARG;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    const KvView c = kv_view(d, cache);
    const cudaStream_t st = (cudaStream_t)stream;
    const int sms = kv_sm_count(d->device);
    if (sms < 1) return DSQ_ERR_CUDA;
    const bool many = (double)tokens * d->kv_heads * d->head_dim / 8 >= 4.0 * 8 * sms * kThreads;
    if (d->head_dim == 64)
        return many ? launch_read<64, 4>(c, rows, slots, tokens, st) : launch_read<64, 1>(c, rows, slots, tokens, st);
    if (d->head_dim == 128)
        return many ? launch_read<128, 4>(c, rows, slots, tokens, st) : launch_read<128, 1>(c, rows, slots, tokens, st);
    return many ? launch_read<256, 4>(c, rows, slots, tokens, st) : launch_read<256, 1>(c, rows, slots, tokens, st);
}
