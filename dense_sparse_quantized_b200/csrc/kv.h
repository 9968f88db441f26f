// kv.h -- the 4-bit key/value cache: its layout, argument checks and the
// launchers behind dsq_kv_append, dsq_kv_read and dsq_kv_attend.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "device_guard.h"
#include "internal.h"

namespace dsq {

constexpr int kKvGroup = 32;  // dimensions that share a scale and a zero
constexpr int kKvTile = 16;   // tokens of a tile: the k extent of one fp16 matrix instruction
constexpr float kKvClamp = 57344.0f;

// Byte offsets inside a tile of head dimension D.
__host__ __device__ constexpr int kv_tile_bytes(int D) { return kKvTile * (D + D / 8); }
__host__ __device__ constexpr int kv_codes(int D, int which) { return which * kKvTile * D / 2; }
__host__ __device__ constexpr int kv_words(int D, int which) { return kKvTile * D + which * kKvTile * D / 16; }

// Division of 0 <= n < 2^31 by a number the host knows: with l = ceil(log2 d)
// and mul = ceil(2^(31 + l) / d), n mul / 2^(31 + l) exceeds n / d by less than
// n / 2^(31 + l) < 1 / d.
struct KvDivisor {
    uint32_t mul, shift;
    __device__ __forceinline__ int div(int n) const { return (int)(((uint64_t)(uint32_t)n * mul) >> shift); }
};
inline KvDivisor kv_divisor(int d) {
    uint32_t l = 0;
    while ((1ll << l) < d) l++;
    return {(uint32_t)(((1ull << (31 + l)) + d - 1) / d), 31 + l};
}

struct KvView {
    const uint8_t *cache;
    int kv_heads, page_tokens, page_tiles, pages;
    int slots;          // pages * page_tokens < 2^31
    KvDivisor page_by;  // by tokens of a page
};

inline int kv_check_desc(const dsq_kv_desc *d) {
    if (!d || d->kv_heads < 1 || d->page_tokens < 1 || d->page_tokens % kKvTile || d->pages < 0 || d->device < 0)
        return DSQ_ERR_INVALID_ARG;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return DSQ_ERR_UNSUPPORTED;
    const int64_t slots = (int64_t)d->pages * d->page_tokens;
    if (slots >= ((int64_t)1 << 31) || slots / kKvTile * d->kv_heads >= ((int64_t)1 << 31)) return DSQ_ERR_UNSUPPORTED;
    return DSQ_OK;
}

inline KvView kv_view(const dsq_kv_desc *d, const void *cache) {
    return {(const uint8_t *)cache, d->kv_heads, d->page_tokens, d->page_tokens / kKvTile, d->pages,
            d->pages * d->page_tokens, kv_divisor(d->page_tokens)};
}

// Where the tile with token offset `off` of (page, head) starts.
__device__ __forceinline__ int64_t kv_tile_at(const KvView &c, int D, int page, int head, int off) {
    return (int64_t)((page * c.kv_heads + head) * c.page_tiles + off / kKvTile) * kv_tile_bytes(D);  // fewer than 2^31 tiles
}

struct KvAttend {
    KvView c;
    KvDivisor share_by, tiles_by;  // by heads of a group, by tiles of a page
    const void *q;
    void *out;
    float *lse;
    int64_t q_token, q_head, out_token, out_head;
    int q_tokens, rows_each;  // rows_each: of a sequence, without q_start
    int most_tokens;          // that a sequence's pages hold
    int q_heads, share, batch, table_pages, causal, window;
    float scale_log2;  // scale * log2(e): the softmax runs in powers of two
    const int32_t *page_table, *kv_lens, *q_start;
};

// Rows and cached tokens of sequence b, clamped to what the buffers hold.
// (Rows, and rows times heads, are below 2^31.)
struct KvSeq {
    int row0, rows, len;
};
__device__ __forceinline__ KvSeq kv_seq(const KvAttend &a, int b) {
    KvSeq s;
    if (a.q_start) {
        s.row0 = min(max(a.q_start[b], 0), a.q_tokens);
        s.rows = min(max(a.q_start[b + 1], s.row0), a.q_tokens) - s.row0;
    } else {
        s.row0 = b * a.rows_each;
        s.rows = a.rows_each;
    }
    s.len = min(max(a.kv_lens[b], 0), a.most_tokens);
    return s;
}

inline bool kv_aligned(const void *p, uintptr_t to) { return ((uintptr_t)p & (to - 1)) == 0; }
inline bool kv_multiple8(int64_t s) { return (s & 7) == 0; }

// Whether [tokens][heads] rows of D elements at these strides are apart.
inline bool kv_rows_apart(int64_t tokens, int64_t heads, int64_t token, int64_t head, int D) {
    if (tokens <= 1 && heads <= 1) return true;
    if (tokens <= 1) return head >= D;
    if (heads <= 1) return token >= D;
    return (head >= D && token >= (heads - 1) * head + D) || (token >= D && head >= (tokens - 1) * token + D);
}

// The kernels are launched early, while the one before them in the stream still
// runs (programmatic dependent launch): they touch no memory of the caller's
// before kv_after_previous(), which waits until that one has ended, and let
// the next one be launched as early.  No pointer to what an earlier kernel may
// have written is __restrict__: with it a load counts as one of constant memory,
// which the compiler is free to move up past the wait.
__device__ __forceinline__ void kv_after_previous() {
    asm volatile("griddepcontrol.launch_dependents;\n\tgriddepcontrol.wait;" ::: "memory");
}
template <typename... Params, typename... Args>
int kv_launch(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem, cudaStream_t stream, const Args &...args) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return DSQ_OK;
    cudaGetLastError();  // returned here, not left for the caller's next check
    return DSQ_ERR_CUDA;
}

// Sets a kernel's shared-memory limit once per device (a call per launch
// would cost a microsecond of host time).
struct KvOnce {
    std::atomic<uint64_t> done{0};
    bool set_smem(const void *kernel, int bytes) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return false;
        const uint64_t bit = 1ull << (dev & 63);
        if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return true;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
            cudaGetLastError();
            return false;
        }
        if (dev < 64) done.fetch_or(bit, std::memory_order_release);
        return true;
    }
};

// SMs of a device, asked for once; 0 if CUDA does not say.
inline int kv_sm_count(int device) {
    static std::atomic<int> known[64];
    int n = device < 64 ? known[device].load(std::memory_order_relaxed) : 0;
    if (n) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    if (device < 64) known[device].store(n, std::memory_order_relaxed);
    return n;
}

// Few query rows per sequence (kv_split.cu).
size_t kv_split_workspace();
int launch_kv_split(const KvAttend &a, int head_dim, int dtype, void *workspace, int sms, cudaStream_t stream);

// Many query rows per sequence (kv_prompt.cu).
size_t kv_prompt_workspace(int head_dim);
int launch_kv_prompt(const KvAttend &a, int head_dim, int dtype, void *workspace, int sms, cudaStream_t stream);
int launch_kv_wait_timeout(cudaStream_t stream);  // a kernel whose wait runs out
int kv_take_status(int *word);                    // the current device's status word, cleared; waits for the device

}  // namespace dsq
