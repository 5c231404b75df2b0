// C ABI of the operators around the attention: argument checks and launches.
// Declarations and the contract live in include/mla.h.
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "launch.h"
#include "layer.h"

namespace mla {

int layer_num_sms() {
    static std::atomic<int> cached[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
    if (dev < 64 && cached[dev].load(std::memory_order_relaxed) > 0) return cached[dev].load(std::memory_order_relaxed);
    int n = 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 2) n = 152;
    if (dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

}  // namespace mla

namespace {

constexpr int kMaxTokens = 65535 * 128;
constexpr int kMaxWidth = 1 << 20;
constexpr unsigned long long kWaitNs = 2000000000ull;  // bound of the products' waits for work unless one is set

bool aligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }

cudaStream_t as_stream(void *s) { return reinterpret_cast<cudaStream_t>(s); }

int result(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// Sizes of a call on B * s_q tokens.
int check_tokens(const mla_dims *d) {
    if (!d) return MLA_ERR_NULL;
    if (d->B < 0 || d->H < 1 || d->s_q < 1) return MLA_ERR_SHAPE;
    if (d->s_q > (1 << 20) || d->B > 65535 || d->H > 65535 || (long long)d->B * d->s_q > kMaxTokens)
        return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

bool good_plan(const mla_rope_plan *p) {
    return p->d_rope >= 16 && p->d_rope <= 64 && p->d_rope % 16 == 0 &&
           (p->layout == MLA_ROPE_INTERLEAVED || p->layout == MLA_ROPE_HALF);
}

// Widths of the latent rows the store and the load take.
int check_widths(const mla_dims *d) {
    if (d->d_c < 1 || d->d_rope < 0) return MLA_ERR_SHAPE;
    if (d->d_c % 64 || d->d_c > 512 || d->d_rope % 16 || d->d_rope > 64) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

// A cache that rows are written to or read back from.
int check_store_cache(const mla_dims *d, const mla_cache *c) {
    if (!c) return MLA_ERR_NULL;
    if (d->B == 0) return MLA_OK;
    if (!c->kv || !c->seq_lens) return MLA_ERR_NULL;
    if (!aligned(c->kv, 16) || !aligned(c->seq_lens, 4)) return MLA_ERR_ALIGN;
    const bool blocks = c->kv_dtype == MLA_KV_E4M3_BLOCKS;
    const long long W = blocks ? mla_latent_row_bytes(d) : d->d_c + d->d_rope;  // of a row, in units of seq_stride
    if (c->kv_dtype != MLA_KV_BF16 && c->kv_dtype != MLA_KV_E4M3 && !blocks) return MLA_ERR_UNSUPPORTED;
    if (blocks && !c->block_table && c->seq_stride % 16) return MLA_ERR_ALIGN;
    if (c->kv_dtype == MLA_KV_E4M3) {
        if (!(c->kv_scale > 0.f) || c->kv_scale > 3.0e38f) return MLA_ERR_SHAPE;
        if (c->kv_scale < 1.1754944e-38f) return MLA_ERR_UNSUPPORTED;  // 1 / kv_scale has to be finite
        if (W % 16 || (!c->block_table && c->seq_stride % 16)) return MLA_ERR_ALIGN;
    }
    if (c->block_table) {
        if (!aligned(c->block_table, 4)) return MLA_ERR_ALIGN;
        if (c->max_pages < 1 || c->page_size < 1 || c->num_pages < 1) return MLA_ERR_SHAPE;
        if (c->page_size % 64) return MLA_ERR_UNSUPPORTED;
        if ((long long)c->max_pages * c->page_size > (1ll << 30)) return MLA_ERR_UNSUPPORTED;
    } else {
        if (c->capacity < 1 || c->seq_stride < (long long)c->capacity * W) return MLA_ERR_SHAPE;
        if (c->seq_stride % 8) return MLA_ERR_ALIGN;
        if (c->capacity > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    }
    return MLA_OK;
}

void fill_cache(const mla_dims &d, const mla_cache &c, mla::AttnParams &p) {
    p.B = d.B;
    p.s_q = d.s_q;
    p.kv = c.kv;
    p.kv_fp8 = c.kv_dtype == MLA_KV_E4M3;
    p.kv_scale = p.kv_fp8 ? c.kv_scale : 1.f;
    p.seq_stride = c.seq_stride;
    p.capacity = c.block_table ? c.max_pages * c.page_size : c.capacity;
    p.block_table = c.block_table;
    p.max_pages = c.max_pages;
    p.page_size = c.page_size;
    p.num_pages = c.num_pages;
    p.seq_lens = c.seq_lens;
}

int check_pool(const mla_page_pool *p, int max_tokens) {
    if (!p) return MLA_ERR_NULL;
    if (p->B < 0 || p->page_size < 1 || p->max_pages < 1 || p->num_pages < 1 || max_tokens < 0) return MLA_ERR_SHAPE;
    if (p->page_size % 64 || p->B > 65535 || max_tokens > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    if ((long long)p->max_pages * p->page_size > (1ll << 30)) return MLA_ERR_UNSUPPORTED;
    if ((long long)p->num_pages * p->page_size > 0x7fffffffll) return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

int check_quantize(const mla_quantize_desc *d) {
    if (!d) return MLA_ERR_NULL;
    if (d->M < 0 || d->K < 1) return MLA_ERR_SHAPE;
    if (d->block_rows != 1 && d->block_rows != 128) return MLA_ERR_UNSUPPORTED;
    if (d->M > kMaxTokens || d->K > kMaxWidth) return MLA_ERR_UNSUPPORTED;
    if (d->K % 16) return MLA_ERR_ALIGN;
    if (d->x_stride < d->K || d->code_stride < d->K) return MLA_ERR_SHAPE;
    if (d->scale_stride < (d->block_rows == 1 ? d->M : (d->K + 127) / 128)) return MLA_ERR_SHAPE;
    if (d->x_stride % 8 || d->code_stride % 16) return MLA_ERR_ALIGN;
    return MLA_OK;
}

int check_linear_fp8(const mla_linear_fp8_desc *d, bool residual) {
    if (!d) return MLA_ERR_NULL;
    if (d->M < 0 || d->K < 1 || d->N < 1) return MLA_ERR_SHAPE;
    if (d->act < MLA_ACT_NONE || d->act > MLA_ACT_GELU_TANH) return MLA_ERR_UNSUPPORTED;
    if (d->M > kMaxTokens || d->K > kMaxWidth || d->N > kMaxWidth) return MLA_ERR_UNSUPPORTED;
    if (d->K % 16 || d->N % 8) return MLA_ERR_ALIGN;
    if (d->x_stride < d->K || d->x_scale_stride < d->M || d->out_stride < d->N || (residual && d->residual_stride < d->N))
        return MLA_ERR_SHAPE;
    if (d->x_stride % 16 || d->out_stride % 8 || (residual && d->residual_stride % 8)) return MLA_ERR_ALIGN;
    // a tensor map's strides stay below 2^40 bytes
    if (d->x_stride > (1ll << 39) || d->out_stride > (1ll << 38) || (residual && d->residual_stride > (1ll << 38)))
        return MLA_ERR_UNSUPPORTED;
    return MLA_OK;
}

unsigned long long wait_ns() {
    const unsigned long long ns = mla::wait_limit_ns();
    return ns == 0 ? kWaitNs : ns < (1ull << 61) ? ns : 1ull << 61;  // twice that are cycles
}

int check_linear(const mla_linear_desc *d, bool residual) {
    if (!d) return MLA_ERR_NULL;
    if (d->M < 0 || d->K < 1 || d->N < 1) return MLA_ERR_SHAPE;
    if (d->act < MLA_ACT_NONE || d->act > MLA_ACT_GELU_TANH) return MLA_ERR_UNSUPPORTED;
    if (d->M > kMaxTokens || d->K > kMaxWidth || d->N > kMaxWidth) return MLA_ERR_UNSUPPORTED;
    if (d->K % 8 || d->N % 8) return MLA_ERR_ALIGN;
    if (d->x_stride < d->K || d->out_stride < d->N || (residual && d->residual_stride < d->N)) return MLA_ERR_SHAPE;
    if (d->x_stride % 8 || d->out_stride % 8 || (residual && d->residual_stride % 8)) return MLA_ERR_ALIGN;
    if (d->x_stride > (1ll << 38)) return MLA_ERR_UNSUPPORTED;  // a tensor map's strides stay below 2^40 bytes
    return MLA_OK;
}

}  // namespace

extern "C" {

MLA_API int mla_rope_init(const mla_rope_config *cfg, mla_rope_plan *plan) {
    if (!cfg || !plan) return MLA_ERR_NULL;
    const int d = cfg->d_rope;
    if (d < 16 || d > 64 || d % 16) return MLA_ERR_UNSUPPORTED;
    if (cfg->layout != MLA_ROPE_INTERLEAVED && cfg->layout != MLA_ROPE_HALF) return MLA_ERR_UNSUPPORTED;
    if (!(cfg->mscale > 0.0) || !isfinite((float)cfg->mscale) || !((float)cfg->mscale > 0.f)) return MLA_ERR_SHAPE;
    const double pi = 3.14159265358979323846;
    double base = cfg->base, low = 0.0, high = 0.0;
    const double s = cfg->factor;
    if (!cfg->inv_freq) {
        if (cfg->scaling < MLA_ROPE_PLAIN || cfg->scaling > MLA_ROPE_YARN) return MLA_ERR_UNSUPPORTED;
        if (!(base > 1.0) || !isfinite(base)) return MLA_ERR_SHAPE;
        if (cfg->scaling != MLA_ROPE_PLAIN && (!(s > 0.0) || !isfinite(s))) return MLA_ERR_SHAPE;
        if (cfg->scaling == MLA_ROPE_NTK) {
            base *= pow(s, d / (d - 2.0));
            if (!(base > 0.0) || !isfinite(base)) return MLA_ERR_SHAPE;
        }
        if (cfg->scaling == MLA_ROPE_YARN) {
            if (cfg->original_len < 1 || !(cfg->beta_fast > 0.0) || !isfinite(cfg->beta_fast) || !(cfg->beta_slow > 0.0) ||
                !isfinite(cfg->beta_slow))
                return MLA_ERR_SHAPE;
            low = floor(d * log(cfg->original_len / (2.0 * pi * cfg->beta_fast)) / (2.0 * log(base)));
            high = ceil(d * log(cfg->original_len / (2.0 * pi * cfg->beta_slow)) / (2.0 * log(base)));
            if (low < 0.0) low = 0.0;
            if (high > d - 1.0) high = d - 1.0;
            if (high - low < 0.001) high = low + 0.001;
        }
    }
    mla_rope_plan p;
    memset(&p, 0, sizeof p);
    p.d_rope = d;
    p.layout = cfg->layout;
    p.mscale = (float)cfg->mscale;
    for (int i = 0; i < d / 2; ++i) {
        double f;
        if (cfg->inv_freq) {
            f = cfg->inv_freq[i];
            if (!isfinite(f)) return MLA_ERR_SHAPE;
        } else {
            f = pow(base, -2.0 * i / d);
            if (cfg->scaling == MLA_ROPE_LINEAR) f /= s;
            if (cfg->scaling == MLA_ROPE_YARN) {
                double ramp = (i - low) / (high - low);
                ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
                f = f / s * ramp + f * (1.0 - ramp);
            }
        }
        double turns = f / (2.0 * pi);
        turns -= floor(turns);  // whole turns a position change nothing
        if (turns >= 1.0) turns = 0.0;
        p.turn[i] = (unsigned long long)rint(ldexp(turns, 64));
    }
    *plan = p;
    return MLA_OK;
}

MLA_API int mla_rope(const mla_dims *dims, const mla_rope_plan *plan, const void *x, long long token_stride,
                     long long head_stride, const int *positions, const int *seq_lens, void *pass_out, void *rope_out,
                     int transpose, void *stream) {
    int s = check_tokens(dims);
    if (s) return s;
    if (!plan) return MLA_ERR_NULL;
    if (!good_plan(plan)) return MLA_ERR_UNSUPPORTED;
    if (dims->d_rope != plan->d_rope) return MLA_ERR_SHAPE;
    const int d_pass = pass_out ? dims->d_nope : 0;
    if (pass_out && dims->d_nope < 1) return MLA_ERR_SHAPE;
    if (pass_out && (dims->d_nope % 16 || dims->d_nope > 256)) return MLA_ERR_UNSUPPORTED;
    const long long width = d_pass + dims->d_rope;
    if (dims->H == 1) head_stride = width;
    if (head_stride < width || token_stride < (dims->H - 1) * head_stride + width) return MLA_ERR_SHAPE;
    if (head_stride % 8 || token_stride % 8) return MLA_ERR_ALIGN;
    if (dims->B == 0) return MLA_OK;
    if (!x || !rope_out || (!positions && !seq_lens)) return MLA_ERR_NULL;
    if (!aligned(x, 16) || !aligned(rope_out, 16) || !aligned(pass_out, 16) || !aligned(positions, 4) ||
        !aligned(seq_lens, 4))
        return MLA_ERR_ALIGN;
    // x may be turned in place where every value is written by the thread that read it
    if (pass_out == x || pass_out == rope_out) return MLA_ERR_UNSUPPORTED;
    if (rope_out == x && (pass_out || (dims->H > 1 && head_stride != width) ||
                          ((long long)dims->B * dims->s_q > 1 && token_stride != dims->H * width)))
        return MLA_ERR_UNSUPPORTED;
    mla::RopeArgs a;
    a.x = (const __nv_bfloat16 *)x;
    a.token_stride = token_stride;
    a.head_stride = head_stride;
    a.tokens = dims->B * dims->s_q;
    a.s_q = dims->s_q;
    a.H = dims->H;
    a.d_pass = d_pass;
    a.d_rope = dims->d_rope;
    a.positions = positions;
    a.seq_lens = seq_lens;
    a.pass_out = (__nv_bfloat16 *)pass_out;
    a.rope_out = (__nv_bfloat16 *)rope_out;
    a.sign = transpose ? -1.f : 1.f;
    a.plan = *plan;
    return result(mla::launch_rope(a, as_stream(stream)));
}

MLA_API int mla_pages_update(const mla_page_pool *pool, const int *old_lens, const int *new_lens, int max_tokens,
                             int *seq_lens, int *token_start, int *positions, int *slots, int *status,
                             void *stream) {
    int s = check_pool(pool, max_tokens);
    if (s) return s;
    if (!pool->free_ring || !pool->state || !pool->state_out || !token_start) return MLA_ERR_NULL;
    if (pool->B > 0 && (!pool->block_table || !old_lens || !new_lens || !seq_lens)) return MLA_ERR_NULL;
    if (max_tokens > 0 && (!positions || !slots)) return MLA_ERR_NULL;
    const void *all[] = {pool->block_table, pool->free_ring, pool->state, pool->state_out, old_lens, new_lens,
                         seq_lens, token_start, positions, slots, status};
    for (const void *p : all)
        if (!aligned(p, 4)) return MLA_ERR_ALIGN;
    // outputs of their own: the inputs are read by every CTA while they are written
    if (pool->state_out == pool->state || (pool->B > 0 && (seq_lens == old_lens || seq_lens == new_lens)))
        return MLA_ERR_UNSUPPORTED;
    mla::PagesArgs a{pool->B, pool->page_size, pool->max_pages, pool->num_pages, max_tokens, pool->block_table,
                     pool->free_ring, pool->state, pool->state_out, old_lens, new_lens, seq_lens, token_start,
                     positions, slots, status, 0, 25};
    const unsigned long long units = (unsigned)pool->page_size / 64;
    while ((1ull << (a.div_shift - 25)) < units) ++a.div_shift;
    a.div_magic = (unsigned)(((1ull << a.div_shift) + units - 1) / units);
    return result(mla::launch_pages_update(a, as_stream(stream)));
}

MLA_API int mla_latent_store(const mla_dims *dims, const mla_rope_plan *plan, const void *x, long long token_stride,
                             const void *norm_weight, float eps, const int *positions, const int *slots,
                             const mla_cache *cache, int *status, void *stream) {
    int s = check_tokens(dims);
    if (s) return s;
    if ((s = check_widths(dims))) return s;
    if (plan && !good_plan(plan)) return MLA_ERR_UNSUPPORTED;
    if (plan && plan->d_rope != dims->d_rope) return MLA_ERR_SHAPE;
    if (norm_weight && (!(eps >= 0.f) || !isfinite(eps))) return MLA_ERR_SHAPE;
    if ((s = check_store_cache(dims, cache))) return s;
    const long long W = dims->d_c + dims->d_rope;
    if (token_stride < W) return MLA_ERR_SHAPE;
    if (token_stride % 8) return MLA_ERR_ALIGN;
    if (dims->B == 0) return MLA_OK;
    if (slots && !cache->block_table) return MLA_ERR_UNSUPPORTED;
    if (slots && (long long)cache->num_pages * cache->page_size > 0x7fffffffll) return MLA_ERR_UNSUPPORTED;
    if (!x) return MLA_ERR_NULL;
    if (!aligned(x, 16) || !aligned(norm_weight, 16) || !aligned(positions, 4) || !aligned(slots, 4) ||
        !aligned(status, 4))
        return MLA_ERR_ALIGN;
    mla::StoreArgs a;
    memset(&a, 0, sizeof a);
    a.x = (const __nv_bfloat16 *)x;
    a.token_stride = token_stride;
    a.tokens = dims->B * dims->s_q;
    a.s_q = dims->s_q;
    a.d_c = dims->d_c;
    a.d_rope = dims->d_rope;
    a.weight = (const __nv_bfloat16 *)norm_weight;
    a.eps = eps;
    a.rotate = plan != nullptr;
    a.positions = positions;
    a.slots = slots;
    a.status = status;
    if (plan) a.plan = *plan;
    a.dtype = cache->kv_dtype;
    fill_cache(*dims, *cache, a.cache);
    return result(mla::launch_latent_store(a, as_stream(stream)));
}

MLA_API int mla_linear_query_cut(const mla_linear_desc *d, mla_linear_cut *cut) {
    const int s = check_linear(d, false);
    if (s) return s;
    if (!cut) return MLA_ERR_NULL;
    if (d->M == 0) return MLA_ERR_SHAPE;
    const mla::LinearPlan p = mla::linear_plan(d->M, d->K, d->N, mla::layer_num_sms());
    *cut = mla_linear_cut{p.bt, p.pair ? 256 : 128, p.cluster, !p.whole, p.grid};
    return MLA_OK;
}

MLA_API size_t mla_linear_workspace_size(const mla_linear_desc *d) {
    if (check_linear(d, false)) return 0;
    return d->M == 0 ? 256 : mla::linear_workspace_bytes(mla::linear_plan(d->M, d->K, d->N, mla::layer_num_sms()));
}

MLA_API int mla_linear(const mla_linear_desc *d, const void *x, const void *w, const void *bias, const void *residual,
                       void *out, void *workspace, size_t ws_bytes, void *stream) {
    return mla_linear_status(d, x, w, bias, residual, out, workspace, ws_bytes, nullptr, stream);
}

MLA_API int mla_linear_status(const mla_linear_desc *d, const void *x, const void *w, const void *bias,
                              const void *residual, void *out, void *workspace, size_t ws_bytes, int *status,
                              void *stream) {
    int s = check_linear(d, residual != nullptr);
    if (s) return s;
    if (!aligned(workspace, 16)) return MLA_ERR_ALIGN;
    if (d->M == 0) return ws_bytes < 256 ? MLA_ERR_WORKSPACE : MLA_OK;
    const mla::LinearPlan plan = mla::linear_plan(d->M, d->K, d->N, mla::layer_num_sms());
    const size_t need = mla::linear_workspace_bytes(plan);
    if (ws_bytes < need) return MLA_ERR_WORKSPACE;
    if (!workspace && need > 256) return MLA_ERR_NULL;
    if (!x || !w || !out) return MLA_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
        !aligned(status, 4))
        return MLA_ERR_ALIGN;
    if (out == x || out == w || (out == residual && d->M > 1 && d->out_stride != d->residual_stride))
        return MLA_ERR_UNSUPPORTED;
    mla::LinearArgs a;
    a.M = d->M;
    a.K = d->K;
    a.N = d->N;
    a.act = d->act;
    a.x = (const __nv_bfloat16 *)x;
    a.w = (const __nv_bfloat16 *)w;
    a.bias = (const __nv_bfloat16 *)bias;
    a.residual = (const __nv_bfloat16 *)residual;
    a.out = (__nv_bfloat16 *)out;
    a.x_stride = d->x_stride;
    a.out_stride = d->out_stride;
    a.residual_stride = d->residual_stride;
    a.part = (float *)workspace;
    a.status = status;
    a.wait_ns = wait_ns();
    return result(mla::launch_linear(a, plan, as_stream(stream)));
}

MLA_API long long mla_latent_row_bytes(const mla_dims *dims) {
    if (!dims || check_widths(dims)) return 0;
    return dims->d_c + 16 + 2 * dims->d_rope;
}

MLA_API int mla_latent_load(const mla_dims *dims, const mla_cache *cache, int rows, const int *positions, void *out,
                            long long out_stride, int *status, void *stream) {
    if (!dims) return MLA_ERR_NULL;
    if (dims->B < 0) return MLA_ERR_SHAPE;
    if (dims->B > 65535) return MLA_ERR_UNSUPPORTED;
    int s = check_widths(dims);
    if (s) return s;
    if ((s = check_store_cache(dims, cache))) return s;
    const long long W = dims->d_c + dims->d_rope;
    if (rows < 0 || out_stride < rows * W) return MLA_ERR_SHAPE;
    if (rows > (1 << 30)) return MLA_ERR_UNSUPPORTED;
    if (out_stride % 8) return MLA_ERR_ALIGN;
    if (dims->B == 0 || rows == 0) return MLA_OK;
    if (!out) return MLA_ERR_NULL;
    if (!aligned(out, 16) || !aligned(positions, 4) || !aligned(status, 4)) return MLA_ERR_ALIGN;
    if (out == cache->kv) return MLA_ERR_UNSUPPORTED;
    mla::LoadArgs a;
    memset(&a, 0, sizeof a);
    a.rows = rows;
    a.d_c = dims->d_c;
    a.width = (int)W;
    a.dtype = cache->kv_dtype;
    a.positions = positions;
    a.out = (__nv_bfloat16 *)out;
    a.out_stride = out_stride;
    a.row_bytes = a.dtype == MLA_KV_BF16 ? 2 * W : a.dtype == MLA_KV_E4M3 ? W : mla_latent_row_bytes(dims);
    a.seq_bytes = cache->seq_stride * (a.dtype == MLA_KV_BF16 ? 2 : 1);
    fill_cache(*dims, *cache, a.cache);
    a.status = status;
    return result(mla::launch_latent_load(a, as_stream(stream)));
}

MLA_API int mla_quantize(const mla_quantize_desc *d, const void *x, const void *norm_weight, float eps, void *codes,
                         float *scales, void *stream) {
    const int s = check_quantize(d);
    if (s) return s;
    if (norm_weight && d->block_rows != 1) return MLA_ERR_UNSUPPORTED;
    if (norm_weight && (!(eps >= 0.f) || !isfinite(eps))) return MLA_ERR_SHAPE;
    if (d->M == 0) return MLA_OK;
    if (!x || !codes || !scales) return MLA_ERR_NULL;
    if (!aligned(x, 16) || !aligned(norm_weight, 16) || !aligned(codes, 16) || !aligned(scales, 4)) return MLA_ERR_ALIGN;
    if (codes == x || scales == x || (const void *)scales == codes) return MLA_ERR_UNSUPPORTED;
    const mla::QuantizeArgs a{d->M, d->K, d->block_rows, (const __nv_bfloat16 *)x, d->x_stride,
                              (const __nv_bfloat16 *)norm_weight, eps, (uint8_t *)codes, d->code_stride, scales,
                              d->scale_stride};
    return result(mla::launch_quantize(a, as_stream(stream)));
}

MLA_API int mla_linear_fp8_query_cut(const mla_linear_fp8_desc *d, mla_linear_cut *cut) {
    const int s = check_linear_fp8(d, false);
    if (s) return s;
    if (!cut) return MLA_ERR_NULL;
    if (d->M == 0) return MLA_ERR_SHAPE;
    const mla::LinearFp8Plan p = mla::linear_fp8_plan(d->M, d->K, d->N, mla::layer_num_sms());
    *cut = mla_linear_cut{p.pair ? 256 : 128, p.columns, p.cluster, 0, p.grid};
    return MLA_OK;
}

MLA_API int mla_linear_fp8(const mla_linear_fp8_desc *d, const void *x, const float *x_scale, const void *w,
                           const float *w_scale, const void *bias, const void *residual, void *out, int *status,
                           void *stream) {
    const int s = check_linear_fp8(d, residual != nullptr);
    if (s) return s;
    if (d->M == 0) return MLA_OK;
    if (!x || !x_scale || !w || !w_scale || !out) return MLA_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 16) || !aligned(residual, 16) || !aligned(out, 16) ||
        !aligned(x_scale, 4) || !aligned(w_scale, 4) || !aligned(status, 4))
        return MLA_ERR_ALIGN;
    if (out == x || out == w || (out == residual && d->M > 1 && d->out_stride != d->residual_stride))
        return MLA_ERR_UNSUPPORTED;
    mla::LinearFp8Args a;
    memset(&a, 0, sizeof a);
    a.M = d->M;
    a.K = d->K;
    a.N = d->N;
    a.act = d->act;
    a.x = (const __nv_bfloat16 *)x;
    a.w = (const __nv_bfloat16 *)w;
    a.bias = (const __nv_bfloat16 *)bias;
    a.residual = (const __nv_bfloat16 *)residual;
    a.out = (__nv_bfloat16 *)out;
    a.x_stride = d->x_stride;
    a.out_stride = d->out_stride;
    a.residual_stride = d->residual_stride;
    a.status = status;
    a.wait_ns = wait_ns();
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.x_scale_stride = d->x_scale_stride;
    const mla::LinearFp8Plan plan = mla::linear_fp8_plan(d->M, d->K, d->N, mla::layer_num_sms());
    if (plan.grid == 0) return MLA_ERR_UNSUPPORTED;
    return result(mla::launch_linear_fp8(a, plan, as_stream(stream)));
}

}  // extern "C"
