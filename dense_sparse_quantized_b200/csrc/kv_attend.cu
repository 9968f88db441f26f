// kv_attend.cu -- attention over the 4-bit key/value cache.
//
// One warp per (query row, query head): the lanes hold D / 32 dimensions each
// and walk the tokens the query sees with a running maximum and sum.
#include "kv.h"

namespace dsq {

namespace {

template <typename T>
__device__ __forceinline__ float to_float(T x) { return (float)x; }

template <int D, typename T>
__global__ void __launch_bounds__(128) attend_rows_kernel(KvAttend a) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
    const int64_t row = item / a.q_heads;
    const int head = (int)(item % a.q_heads), kv_head = head / a.share;
    if (row >= a.q_tokens) return;
    int b = -1;
    KvSeq s;
    for (int i = 0; i < a.batch; i++) {
        s = kv_seq(a, i);
        if (row >= s.row0 && row < s.row0 + s.rows) {
            b = i;
            break;
        }
    }
    if (b < 0) return;
    const int pos = s.len - s.rows + (int)(row - s.row0);
    const int hi = a.causal ? min(s.len, pos + 1) : s.len;
    const int lo = a.window ? max(0, pos - a.window + 1) : 0;
    float q[E], o[E] = {};
    const T *qp = (const T *)a.q + row * a.q_token + head * a.q_head + lane * E;
#pragma unroll
    for (int i = 0; i < E; i++) q[i] = to_float(qp[i]);
    float m = -INFINITY, l = 0.0f;
    for (int t = lo; t < hi; t++) {
        const int page = a.page_table[(int64_t)b * a.table_pages + t / a.c.page_tokens];
        if (page < 0 || page >= a.c.pages) continue;
        const int off = t % a.c.page_tokens, r = off % kKvTile;
        const uint8_t *tile = a.c.cache + kv_tile_at(a.c, D, page, kv_head, off);
        float x[2][E];
#pragma unroll
        for (int which = 0; which < 2; which++) {
            const uint32_t w = *(const uint16_t *)(tile + kv_words(D, which) + (lane * E / kKvGroup * kKvTile + r) * 2);
            const float sc = kv_scale(w), z = (float)(w & 15u);
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                const uint8_t c = tile[kv_codes(D, which) + r * (D / 2) + (lane * E + i) / 2];
                x[which][i] = sc * ((float)(c & 15) - z);
                x[which][i + 1] = sc * ((float)(c >> 4) - z);
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int i = 0; i < E; i++) dot += q[i] * x[0][i];
#pragma unroll
        for (int k = 16; k; k >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, k);
        const float y = dot * a.scale_log2, top = fmaxf(m, y);
        const float keep = m == top ? 1.0f : exp2f(m - top), p = exp2f(y - top);
        l = l * keep + p;
#pragma unroll
        for (int i = 0; i < E; i++) o[i] = o[i] * keep + p * x[1][i];
        m = top;
    }
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    T *op = (T *)a.out + row * a.out_token + head * a.out_head + lane * E;
#pragma unroll
    for (int i = 0; i < E; i++) op[i] = (T)(o[i] * inv);
    if (a.lse && lane == 0) a.lse[row * a.q_heads + head] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

template <int D>
int launch(const KvAttend &a, int dtype, cudaStream_t st) {
    const unsigned blocks = (unsigned)((a.q_tokens * a.q_heads + 3) / 4);
    if (dtype == DSQ_DTYPE_F16) attend_rows_kernel<D, __half><<<blocks, 128, 0, st>>>(a);
    else attend_rows_kernel<D, __nv_bfloat16><<<blocks, 128, 0, st>>>(a);
    return cudaGetLastError() == cudaSuccess ? DSQ_OK : DSQ_ERR_CUDA;
}

}  // namespace

size_t kv_attend_workspace(const dsq_kv_desc *, const dsq_kv_queries *, int) { return 256; }

int launch_kv_attend(const KvAttend &a, int head_dim, int dtype, void *, int, cudaStream_t st) {
    if (head_dim == 64) return launch<64>(a, dtype, st);
    if (head_dim == 128) return launch<128>(a, dtype, st);
    return launch<256>(a, dtype, st);
}

}  // namespace dsq
