// kv_attend.cu -- dsq_kv_attend: argument checks and the choice of kernel; the
// report of waits that ran out.
#include <algorithm>

#include "kv.h"

using namespace dsq;

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kMeasuredSms = 148;  // of the GPU that the estimates below were measured on

// Rows of a job: query tokens of a sequence, on average, times the heads of a group.
double rows_of(const dsq_kv_desc *d, const dsq_kv_queries *a) {
    return a->batch ? (double)a->q_tokens / a->batch * (a->q_heads / d->kv_heads) : 0.0;
}

// Which kernel, by estimates in microseconds of what either takes, for
// sequences of average rows and of as many tokens as the pages hold (or their
// window).  kv_split.cu works on units of 16 rows (8 at 256 dimensions) x 32
// tokens and takes four units' time more for each tile of rows; kv_prompt.cu on
// units of 256 rows (128 at 256 dimensions) x 128 tokens and three units' time
// more for each piece, three quarters of the time for up to 128 rows.
// Measured on kMeasuredSms SMs, fp16, causal, microseconds (kv_split / kv_prompt), of (sequences x
// kv heads, rows, tokens):
//   128 dimensions: (8, 96, 4096) 21 / 26, (8, 96, 16384) 44 / 33,
//     (64, 24, 4096) 35 / 40, (64, 96, 1024) 33 / 26, (64, 96, 256) 20 / 13,
//     (512, 24, 256) 33 / 43, (512, 96, 256) 79 / 48
//   64: (64, 48, 4096) 30 / 38, (64, 96, 256) 16 / 11, (512, 96, 256) 39 / 35
//   256: (64, 16, 4096) 51 / 77, (64, 48, 1024) 47 / 34, (8, 96, 1024) 16 / 31
// All with page tables as wide as the sequences are long.  The lengths are on
// the device: a wider table is taken for longer sequences, and a batch that
// mixes prompts with single tokens for one of average rows.
bool many_rows(const dsq_kv_desc *d, const dsq_kv_queries *a, int sms) {
    const double each = a->batch ? (double)a->q_tokens / a->batch : 0.0, rows = rows_of(d, a);
    if (rows <= 8 || d->pages == 0) return false;
    const double jobs = (double)a->batch * d->kv_heads;
    double tokens = (double)a->table_pages * d->page_tokens;
    if (a->window) tokens = fmin(tokens, a->window + each);
    if (a->causal) tokens = fmax(tokens - each / 2, 1.0);
    const bool wide = d->head_dim == 256;
    const double few_unit = d->head_dim == 64 ? 0.8e-3 : d->head_dim == 128 ? 1.36e-3 : 1.95e-3;
    const double few_tiles = jobs * ceil(rows / (wide ? 8 : 16));
    const double few = (few_tiles <= sms ? 8.0 : 12.0) + few_unit * ((double)kMeasuredSms / sms) * few_tiles * (ceil(tokens / 32) + 4);
    const double many_unit = (d->head_dim == 64 ? 2.0 : d->head_dim == 128 ? 2.7 : 3.7) * (rows <= 128 && !wide ? 0.75 : 1.0);
    const double many_tiles = jobs * ceil(rows / (wide ? 128 : 256)), units = ceil(tokens / 128);
    const double many = many_tiles <= sms && units <= 4
                            ? 7.0 + many_unit * (units + 1)
                            : 12.0 + many_unit * fmax(fmin(units + 3, 7.0), many_tiles * (units + 3) / sms);
    return many < few;
}

// Whether the shape of a call is one there is: what does not need its pointers.
int check_shape(const dsq_kv_desc *d, const dsq_kv_queries *a) {
    const int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    if (!a) return DSQ_ERR_INVALID_ARG;
    if (a->q_heads < 1 || a->q_heads % d->kv_heads || a->batch < 0 || a->q_tokens < 0 || a->table_pages < 0 ||
        a->window < 0 || (a->window > 0 && !a->causal) || !isfinite(a->scale * kLog2e))
        return DSQ_ERR_INVALID_ARG;
    if (a->dtype != DSQ_DTYPE_F16 && a->dtype != DSQ_DTYPE_BF16)
        return a->dtype == DSQ_DTYPE_F32 ? DSQ_ERR_UNSUPPORTED : DSQ_ERR_INVALID_ARG;
    if (!a->q_start && (a->batch == 0 ? a->q_tokens > 0 : a->q_tokens % a->batch != 0)) return DSQ_ERR_INVALID_ARG;
    if ((int64_t)a->table_pages * d->page_tokens >= ((int64_t)1 << 30) ||
        a->q_tokens >= ((int64_t)1 << 30) / a->q_heads ||  // token and row numbers are ints, with room to round up
        (int64_t)a->batch * d->kv_heads >= ((int64_t)1 << 29))  // and so are job numbers (launch_split's shift)
        return DSQ_ERR_UNSUPPORTED;
    return DSQ_OK;
}

}  // namespace

extern "C" int dsq_kv_attend_kernel(const dsq_kv_desc *d, const dsq_kv_queries *a) {
    const int rc = check_shape(d, a);
    if (rc != DSQ_OK) return rc;
    const int sms = kv_sm_count(d->device);
    return many_rows(d, a, sms ? sms : kMeasuredSms) ? 1 : 0;
}

extern "C" int dsq_kv_attend(const dsq_kv_desc *d, const void *cache, const dsq_kv_queries *a, void *workspace,
                             size_t *workspace_bytes, void *stream) {
    const int rc = check_shape(d, a);
    if (rc != DSQ_OK) return rc;
    if (!workspace_bytes) return DSQ_ERR_INVALID_ARG;
    // by the queries' shape alone, so that one workspace does for any lengths
    const size_t need = rows_of(d, a) <= 8 ? kv_split_workspace() : std::max(kv_split_workspace(), kv_prompt_workspace(d->head_dim));
    if (!workspace || *workspace_bytes < need) {
        *workspace_bytes = need;
        return DSQ_ERR_BUFFER_TOO_SMALL;
    }
    if (a->batch == 0 || a->q_tokens == 0) return DSQ_OK;
    if (!a->q || !a->out || !a->kv_lens || (a->table_pages > 0 && !a->page_table) || (d->pages > 0 && !cache))
        return DSQ_ERR_INVALID_ARG;
    if (!kv_aligned(a->q, 16) || !kv_aligned(a->out, 16) || !kv_aligned(a->lse, 4) || !kv_aligned(cache, 128) ||
        !kv_aligned(workspace, 256) || !kv_aligned(a->page_table, 4) || !kv_aligned(a->kv_lens, 4) || !kv_aligned(a->q_start, 4))
        return DSQ_ERR_INVALID_ARG;
    if (!kv_multiple8(a->q_token) || !kv_multiple8(a->q_head) || !kv_multiple8(a->out_token) || !kv_multiple8(a->out_head) ||
        !kv_rows_apart(a->q_tokens, a->q_heads, a->out_token, a->out_head, d->head_dim))
        return DSQ_ERR_INVALID_ARG;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    KvAttend k = {};
    k.c = kv_view(d, cache);
    k.q = a->q;
    k.out = a->out;
    k.lse = a->lse;
    k.q_token = a->q_token;
    k.q_head = a->q_head;
    k.out_token = a->out_token;
    k.out_head = a->out_head;
    k.q_tokens = (int)a->q_tokens;
    k.rows_each = a->q_start ? 0 : (int)(a->q_tokens / a->batch);
    k.most_tokens = (int)((int64_t)a->table_pages * d->page_tokens);
    k.q_heads = a->q_heads;
    k.share = a->q_heads / d->kv_heads;
    k.share_by = kv_divisor(k.share);
    k.tiles_by = kv_divisor(k.c.page_tiles);
    k.batch = a->batch;
    k.table_pages = a->table_pages;
    k.causal = a->causal;
    k.window = std::min(a->window, 1 << 30);  // more than any position; token numbers less it stay ints
    k.scale_log2 = a->scale * kLog2e;
    k.page_table = a->page_table;
    k.kv_lens = a->kv_lens;
    k.q_start = a->q_start;
    const int sms = kv_sm_count(d->device);
    if (sms < 1) return DSQ_ERR_CUDA;
    return many_rows(d, a, sms) ? launch_kv_prompt(k, d->head_dim, a->dtype, workspace, sms, (cudaStream_t)stream)
                           : launch_kv_split(k, d->head_dim, a->dtype, workspace, sms, (cudaStream_t)stream);
}

extern "C" int dsq_kv_check(const dsq_kv_desc *d) {
    int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    int word = 0;
    if ((rc = kv_take_status(&word)) != DSQ_OK) return rc;
    return word == 0 ? DSQ_OK : DSQ_ERR_DEVICE;
}

extern "C" int dsq_kv_selftest_wait_timeout(const dsq_kv_desc *d, void *stream) {
    const int rc = kv_check_desc(d);
    if (rc != DSQ_OK) return rc;
    DeviceGuard guard(d->device);
    if (!guard.ok) return DSQ_ERR_CUDA;
    return launch_kv_wait_timeout((cudaStream_t)stream);
}
