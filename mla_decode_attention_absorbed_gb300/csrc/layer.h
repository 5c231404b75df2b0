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
    AttnParams cache;  // the cache's fields and the lengths
    int *status;
    mla_rope_plan plan;
};
cudaError_t launch_latent_store(const StoreArgs &a, cudaStream_t st);

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

// SMs of the current device (work plans only), looked up once per device.
int layer_num_sms();

}  // namespace mla
