// kv_cache.cu -- writing the 4-bit key/value cache and reading it back.
//
// Both kernels move bytes: a row of D values (2 D bytes at 16 bits) against
// 9 D / 16 bytes of codes and words.  One thread handles eight dimensions of
// one token's head, keys and values both: one 16-byte access of the rows and
// one 4-byte word of codes each, so a warp's accesses are whole 32-byte
// sectors on both sides.  Four neighbouring threads share a group of 32.
#include "kv.h"

namespace dsq {

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8]) {
    const uint4 u = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float2 f;
        if constexpr (sizeof(T) == 2 && std::is_same<T, __half>::value)
            f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        else
            f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Quantises this thread's eight values of a group held by four neighbouring
// lanes; returns the eight codes, and the group's word in `word`.
__device__ __forceinline__ uint32_t encode8(float (&x)[8], uint32_t &word) {
    bool nan = false;
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        nan |= x[i] != x[i];
        x[i] = fminf(fmaxf(x[i], -kKvClamp), kKvClamp);
        lo = fminf(lo, x[i]);
        hi = fmaxf(hi, x[i]);
    }
#pragma unroll
    for (int m = 1; m <= 2; m <<= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
    }
    const uint32_t votes = __ballot_sync(0xffffffffu, nan);
    nan = (votes >> (threadIdx.x & 28)) & 15u;

    // The scale: the least n * u with 15 n u >= hi - lo, u the last of seven
    // bits.  fp32 finds n to within one; fp64 decides, since hi - lo of two
    // 16-bit floats takes up to 40 bits.  d32 of the rounded difference lies
    // in the same binade as the exact quotient or on its upper border, where
    // 64 * 2u and 128 * u are the same scale.
    const double range = (double)hi - (double)lo;
    const float d32 = (float)range / 15.0f;
    const int e = max((int)(__float_as_uint(d32) >> 23) - 127 - 6, -20);  // u = 2^e
    const float u = __uint_as_float((uint32_t)(e + 127) << 23);
    float n = ceilf(d32 * __uint_as_float((uint32_t)(127 - e) << 23));
    if ((double)(15.0f * n * u) < range) n += 1.0f;
    else if (n > 1.0f && (double)(15.0f * (n - 1.0f) * u) >= range) n -= 1.0f;
    const float s = fmaxf(n, 1.0f) * u;

    // x (11 bits) over s (7 bits) against a border k + 1/2 (5 bits): two
    // numbers of 16 bits at most that are equal or 2^-16 apart, so the
    // rounded fp32 quotient lies on the same side as the exact one.
    const float z = rintf(-lo / s);
    uint32_t codes = 0;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float q = fminf(fmaxf(rintf(x[i] / s) + z, 0.0f), 15.0f);
        codes |= (uint32_t)q << (4 * i);
    }
    word = (uint32_t)__half_as_ushort(__float2half_rn(s)) | (uint32_t)z;
    if (nan) {
        word = 0x7e00u;
        codes = 0;
    }
    return codes;
}

struct RowsIn {
    const void *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) append_kernel(KvView c, uint8_t *__restrict__ cache, RowsIn r,
                                                          const int64_t *__restrict__ slots, int64_t tokens) {
    constexpr int kLanes = D / 8;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const int dim = (threadIdx.x % kLanes) * 8, head = blockIdx.y;
    const int64_t slot = t < tokens ? slots[t] : -1;
    const bool there = slot >= 0 && slot < c.slots;
    float k[8] = {}, v[8] = {};
    if (there) {
        load8((const T *)r.k + t * r.k_token + head * r.k_head + dim, k);
        load8((const T *)r.v + t * r.v_token + head * r.v_head + dim, v);
    }
    uint32_t kw, vw;
    const uint32_t kc = encode8(k, kw), vc = encode8(v, vw);
    if (!there) return;
    const int page = (int)slot / c.page_tokens, off = (int)slot % c.page_tokens, row = off % kKvTile;
    uint8_t *tile = cache + kv_tile_at(c, D, page, head, off);
    *reinterpret_cast<uint32_t *>(tile + kv_codes(D, 0) + row * (D / 2) + dim / 2) = kc;
    *reinterpret_cast<uint32_t *>(tile + kv_codes(D, 1) + row * (D / 2) + dim / 2) = vc;
    if (dim % kKvGroup == 0) {
        const int at = (dim / kKvGroup * kKvTile + row) * 2;
        *reinterpret_cast<uint16_t *>(tile + kv_words(D, 0) + at) = (uint16_t)kw;
        *reinterpret_cast<uint16_t *>(tile + kv_words(D, 1) + at) = (uint16_t)vw;
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, const __half *) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, const __nv_bfloat16 *) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Eight values of the cache: each product is exact in fp32.
template <typename T>
__device__ __forceinline__ void decode8(uint32_t codes, uint32_t word, T *to) {
    const float s = kv_scale(word), z = (float)(word & 15u);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; i++) x[i] = s * ((float)((codes >> (4 * i)) & 15u) - z);
    if constexpr (sizeof(T) == 4) {
        float4 *f = reinterpret_cast<float4 *>(to);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    } else {
        *reinterpret_cast<uint4 *>(to) =
            make_uint4(pack2(x[0], x[1], to), pack2(x[2], x[3], to), pack2(x[4], x[5], to), pack2(x[6], x[7], to));
    }
}

struct RowsOut {
    void *k, *v;
    int64_t k_token, k_head, v_token, v_head;
};

template <int D, typename T>
__global__ void __launch_bounds__(kThreads) read_kernel(KvView c, RowsOut r, const int64_t *__restrict__ slots,
                                                        int64_t tokens) {
    constexpr int kLanes = D / 8;
    const int64_t t = (int64_t)blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    const int dim = (threadIdx.x % kLanes) * 8, head = blockIdx.y;
    const int64_t slot = t < tokens ? slots[t] : -1;
    if (slot < 0 || slot >= c.slots) return;
    const int page = (int)slot / c.page_tokens, off = (int)slot % c.page_tokens, row = off % kKvTile;
    const uint8_t *tile = c.cache + kv_tile_at(c, D, page, head, off);
    const int code_at = row * (D / 2) + dim / 2, word_at = (dim / kKvGroup * kKvTile + row) * 2;
    if (r.k)
        decode8(*reinterpret_cast<const uint32_t *>(tile + kv_codes(D, 0) + code_at),
                *reinterpret_cast<const uint16_t *>(tile + kv_words(D, 0) + word_at),
                (T *)r.k + t * r.k_token + head * r.k_head + dim);
    if (r.v)
        decode8(*reinterpret_cast<const uint32_t *>(tile + kv_codes(D, 1) + code_at),
                *reinterpret_cast<const uint16_t *>(tile + kv_words(D, 1) + word_at),
                (T *)r.v + t * r.v_token + head * r.v_head + dim);
}

int check_rows(const dsq_kv_rows *r, bool both) {
    if (!r || (both ? !r->k || !r->v : !r->k && !r->v)) return DSQ_ERR_INVALID_ARG;
    if (r->dtype < DSQ_DTYPE_F16 || r->dtype > DSQ_DTYPE_F32) return DSQ_ERR_INVALID_ARG;
    if (!kv_aligned(r->k, 16) || !kv_aligned(r->v, 16)) return DSQ_ERR_INVALID_ARG;
    if (!kv_multiple8(r->k_token) || !kv_multiple8(r->k_head) || !kv_multiple8(r->v_token) || !kv_multiple8(r->v_head))
        return DSQ_ERR_INVALID_ARG;
    return DSQ_OK;
}

// The grid of both kernels: tokens along x, kv heads along y.
int grid_for(int64_t tokens, int heads, int D, dim3 *grid) {
    const int64_t blocks = (tokens + kThreads / (D / 8) - 1) / (kThreads / (D / 8));
    if (blocks >= ((int64_t)1 << 31) || heads > 65535) return DSQ_ERR_UNSUPPORTED;
    *grid = dim3((unsigned)blocks, (unsigned)heads);
    return DSQ_OK;
}

template <int D>
void launch_append(dim3 grid, const KvView &c, void *cache, const dsq_kv_rows *r, const int64_t *slots, int64_t tokens,
                   cudaStream_t st) {
    const RowsIn in = {r->k, r->v, r->k_token, r->k_head, r->v_token, r->v_head};
    if (r->dtype == DSQ_DTYPE_F16)
        append_kernel<D, __half><<<grid, kThreads, 0, st>>>(c, (uint8_t *)cache, in, slots, tokens);
    else
        append_kernel<D, __nv_bfloat16><<<grid, kThreads, 0, st>>>(c, (uint8_t *)cache, in, slots, tokens);
}

template <int D>
void launch_read(dim3 grid, const KvView &c, const dsq_kv_rows *r, const int64_t *slots, int64_t tokens,
                 cudaStream_t st) {
    const RowsOut out = {r->k, r->v, r->k_token, r->k_head, r->v_token, r->v_head};
    if (r->dtype == DSQ_DTYPE_F16)
        read_kernel<D, __half><<<grid, kThreads, 0, st>>>(c, out, slots, tokens);
    else if (r->dtype == DSQ_DTYPE_BF16)
        read_kernel<D, __nv_bfloat16><<<grid, kThreads, 0, st>>>(c, out, slots, tokens);
    else
        read_kernel<D, float><<<grid, kThreads, 0, st>>>(c, out, slots, tokens);
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
    if ((rc = grid_for(tokens, d->kv_heads, d->head_dim, &grid)) != DSQ_OK) return rc;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    const KvView c = kv_view(d, cache);
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->head_dim == 64) launch_append<64>(grid, c, cache, rows, slots, tokens, st);
    else if (d->head_dim == 128) launch_append<128>(grid, c, cache, rows, slots, tokens, st);
    else launch_append<256>(grid, c, cache, rows, slots, tokens, st);
    return cudaGetLastError() == cudaSuccess ? DSQ_OK : DSQ_ERR_CUDA;
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
    dim3 grid;
    if ((rc = grid_for(tokens, d->kv_heads, d->head_dim, &grid)) != DSQ_OK) return rc;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    const KvView c = kv_view(d, cache);
    const cudaStream_t st = (cudaStream_t)stream;
    if (d->head_dim == 64) launch_read<64>(grid, c, rows, slots, tokens, st);
    else if (d->head_dim == 128) launch_read<128>(grid, c, rows, slots, tokens, st);
    else launch_read<256>(grid, c, rows, slots, tokens, st);
    return cudaGetLastError() == cudaSuccess ? DSQ_OK : DSQ_ERR_CUDA;
}
