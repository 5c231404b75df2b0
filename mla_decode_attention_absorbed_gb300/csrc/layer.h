// Launchers of the operators around the attention (rotary positions, page
// tables, latent store, matrix product with epilogue) and what they share.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {

struct RopeArgs {
    const __nv_bfloat16 *x;
    long long token_stride, head_stride;
    int tokens, s_q, H, d_pass, d_rope;
    const int *positions;  // [tokens], or NULL: seq_lens[t / s_q] - s_q + t % s_q
    const int *seq_lens;
    __nv_bfloat16 *pass_out, *rope_out;
    float sign;  // -1: the transposed rotation
    mla_rope_plan plan;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t st);

struct StoreArgs {
    const __nv_bfloat16 *x;
    long long token_stride;
    int tokens, s_q, d_c, d_rope;
    const __nv_bfloat16 *weight;  // NULL: no norm
    float eps;
    int rotate;
    const int *positions, *slots;
    int dtype;         // mla_kv_dtype
    AttnParams cache;  // the cache's fields and the lengths
    int *status;
    mla_rope_plan plan;
};
cudaError_t launch_latent_store(const StoreArgs &a, cudaStream_t st);

struct LoadArgs {
    int rows, d_c, width;  // rows a sequence; width: d_c + d_rope
    int dtype;             // mla_kv_dtype
    const int *positions;  // [B][rows], or NULL: row i is token i
    __nv_bfloat16 *out;
    long long out_stride;  // elements between sequences
    long long row_bytes, seq_bytes;
    AttnParams cache;  // the cache's fields and the lengths
    int *status;
};
cudaError_t launch_latent_load(const LoadArgs &a, cudaStream_t st);

struct QuantizeArgs {
    int M, K, block_rows;
    const __nv_bfloat16 *x;
    long long x_stride;
    const __nv_bfloat16 *weight;  // NULL: no norm
    float eps;
    uint8_t *codes;
    long long code_stride;
    float *scales;
    long long scale_stride;
};
cudaError_t launch_quantize(const QuantizeArgs &a, cudaStream_t st);

struct PagesArgs {
    int B, page_size, max_pages, num_pages, max_tokens;
    int *table, *ring;
    const int *state;
    int *state_out;
    const int *old_lens, *new_lens;
    int *seq_lens, *token_start, *positions, *slots, *status;
    unsigned div_magic;  // division by page_size / 64, see pages.cu
    int div_shift;
};
cudaError_t launch_pages_update(const PagesArgs &a, cudaStream_t st);

struct LinearArgs {
    int M, K, N, act;
    const __nv_bfloat16 *x, *w, *bias, *residual;
    __nv_bfloat16 *out;
    long long x_stride, out_stride, residual_stride;
    float *part;  // workspace: fp32 tiles of the pieces of tiles that are cut along K
    int *status;
    unsigned long long wait_ns;  // bound of the waits for work
};
// How a product is cut (see linear.cu).
struct LinearPlan {
    int bt;                // tokens a tile
    int tiles_m, tiles_n;  // tile t: tokens (t % tiles_m) * bt, columns (t / tiles_m) * 128 (pair: 256)
    int nk;                // chunks a tile
    int grid;
    int cluster;           // CTAs that share a tile's K (1: none)
    bool whole;            // whole tiles, CTA g the tiles g, g + grid, ...; else runs of chunks
    bool pair;             // a tile is 256 columns, taken by a pair of CTAs
};
LinearPlan linear_plan(int M, int K, int N, int sms);
size_t linear_workspace_bytes(const LinearPlan &p);
cudaError_t launch_linear(const LinearArgs &a, const LinearPlan &p, cudaStream_t st);

// x and w hold codes
struct LinearFp8Args : LinearArgs {
    const float *x_scale, *w_scale;  // [K / 128][x_scale_stride], [N / 128][K / 128]
    long long x_scale_stride;
};
// How a product of codes is cut (see linear_fp8.cu).
struct LinearFp8Plan {
    int columns;           // of a tile a CTA accumulates, for 128 tokens
    int tiles_m, tiles_n;  // of tokens, of columns
    int nk;                // blocks of K
    int grid;
    int whole;             // tiles that a CTA (or pair) takes whole, one after another; of the others,
    int cluster;           // the CTAs (or pairs) of a cluster share one's K (1: there are none)
    int x_rows;            // of a copy of x: as many as there are, up to 128
    bool pair;             // a tile is 256 tokens high, taken by a pair of CTAs
};
LinearFp8Plan linear_fp8_plan(int M, int K, int N, int sms);
cudaError_t launch_linear_fp8(const LinearFp8Args &a, const LinearFp8Plan &p, cudaStream_t st);

// SMs of the current device (work plans only), looked up once per device.
int layer_num_sms();

}  // namespace mla
