// Cached latents read back as bf16 rows: whole histories or listed tokens, from any of the cache's
// formats, contiguous or paged.
//
// A warp takes 4 rows at a time: it works out where they lie (length, position, page: a chain of
// loads that the 4 rows share), has all their values under way, converts (fp32, one rounding) and
// writes whole rows, 16 bytes a lane.
#include "quantize.cuh"

namespace mla {
namespace {

using namespace quant;

constexpr int kWarps = 8;
constexpr int kRows = 4;    // a warp's rows
constexpr int kParts = 3;   // chunks of 8 values a lane and row: d_c + d_rope <= 576

template <int kDtype>
__global__ void __launch_bounds__(32 * kWarps) latent_values(const LoadArgs a) {
    const int lane = threadIdx.x % 32, b = blockIdx.y, i0 = (blockIdx.x * kWarps + threadIdx.x / 32) * kRows;
    const AttnParams &c = a.cache;
    if (i0 >= a.rows) return;
    const int L = __ldg(c.seq_lens + b);
    if (L < 0 || L > c.capacity) {
        if (lane == 0 && i0 == 0) set_status(a.status, MLA_ERR_SEQLEN);
        return;
    }
    // lane r works out where row r lies (bytes), -1: left as it is
    long long at = -1;
    if (lane < kRows && i0 + lane < a.rows) {
        const int j = a.positions ? __ldg(a.positions + (long long)b * a.rows + i0 + lane) : i0 + lane;
        if (j >= 0 && j < L) {
            if (c.block_table == nullptr) {
                at = b * a.seq_bytes + (long long)j * a.row_bytes;
            } else {
                const int col = j / c.page_size, page = __ldg(c.block_table + (long long)b * c.max_pages + col);
                if (page < 0 || page >= c.num_pages) set_status(a.status, MLA_ERR_PAGE);
                else at = ((long long)page * c.page_size + (j - col * c.page_size)) * a.row_bytes;
            }
        }
    }
    const uint8_t *kv = static_cast<const uint8_t *>(c.kv);
    const int n_codes = kDtype == MLA_KV_E4M3 ? a.width / 8 : a.d_c / 8, n = a.width / 8;
    uint4 v[kRows][kParts];
    float scale[kRows][2];
    long long from[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        from[r] = __shfl_sync(~0u, at, r);
        if (from[r] < 0) continue;
        const uint8_t *row = kv + from[r];
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const int chunk = lane + 32 * p;
            if (chunk >= n) continue;
            if (kDtype == MLA_KV_BF16) {
                v[r][p] = __ldg(reinterpret_cast<const uint4 *>(row) + chunk);
            } else if (chunk < n_codes) {
                const uint2 w = __ldg(reinterpret_cast<const uint2 *>(row) + chunk);
                v[r][p].x = w.x;
                v[r][p].y = w.y;
            } else {  // a key of a row of blocks
                v[r][p] = __ldg(reinterpret_cast<const uint4 *>(row + a.d_c + kScaleBytes) + chunk - n_codes);
            }
            if (kDtype == MLA_KV_E4M3_BLOCKS && p < 2 && chunk < n_codes)
                scale[r][p] = __ldg(reinterpret_cast<const float *>(row + a.d_c) + chunk / 16);
        }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
        if (from[r] < 0) continue;
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + b * a.out_stride + (long long)(i0 + r) * a.width);
#pragma unroll
        for (int p = 0; p < kParts; ++p) {
            const int chunk = lane + 32 * p;
            if (chunk >= n) continue;
            uint4 y = v[r][p];
            if (kDtype != MLA_KV_BF16 && chunk < n_codes) {
                const float s = kDtype == MLA_KV_E4M3 ? c.kv_scale : scale[r][p < 2 ? p : 1];
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t w = e < 2 ? v[r][p].x : v[r][p].y;
                    const float2 f = from_e4m3x2((e & 1 ? w >> 16 : w) & 0xffffu);
                    o[e] = sm100::pack_bf16x2(f.x * s, f.y * s);
                }
                y = make_uint4(o[0], o[1], o[2], o[3]);
            }
            dst[chunk] = y;
        }
    }
}

}  // namespace

cudaError_t launch_latent_load(const LoadArgs &a, cudaStream_t st) {
    const dim3 grid((a.rows + kWarps * kRows - 1) / (kWarps * kRows), a.cache.B);
    if (a.dtype == MLA_KV_BF16) latent_values<MLA_KV_BF16><<<grid, 32 * kWarps, 0, st>>>(a);
    else if (a.dtype == MLA_KV_E4M3) latent_values<MLA_KV_E4M3><<<grid, 32 * kWarps, 0, st>>>(a);
    else latent_values<MLA_KV_E4M3_BLOCKS><<<grid, 32 * kWarps, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace mla
