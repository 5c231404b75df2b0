// Cached latents read back as bf16 rows: whole histories or listed tokens, from any of the cache's
// formats, contiguous or paged.
//
// A warp takes kRows rows at a time: it works out where they lie (length, position, page: a chain of
// loads that the rows go through side by side), has all their values under way, converts (fp32, one rounding)
// and writes whole rows.  Of a row of blocks a lane takes 16 codes, one load, and writes 32 bytes at once
// (8 codes a load and two turns: histories 64.1 us, so 55.4).
//
// Measured (device time): histories of 64 sequences, three quarters of 4096 tokens on average, in blocks 55.4 us = 0.94 of the
// measured copy rate (a row of 656 bytes spans 21 sectors of 32), as codes with one scale 53.3 = 0.94, as
// bf16 68.5 = 0.97; 65536 listed tokens in blocks 21.2 us = 0.82, position, page and row one after another;
// 3 x 333 rows 2.6 us, a launch and four round trips.  Two rows a warp 21.8, eight 23.6 (listed tokens).
#include "quantize.cuh"

namespace mla {
namespace {

using namespace quant;

constexpr int kWarps = 4;
constexpr int kRows = 4;  // a warp's rows

struct Piece {  // 16 values of the output
    uint4 lo, hi;
};

// 32 bytes at once where the address allows it.
__device__ __forceinline__ void store_piece(__nv_bfloat16 *to, const Piece &p, bool aligned) {
    if (aligned) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(p.lo.x), "r"(p.lo.y), "r"(p.lo.z),
                     "r"(p.lo.w), "r"(p.hi.x), "r"(p.hi.y), "r"(p.hi.z), "r"(p.hi.w)
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(to)[0] = p.lo;
        reinterpret_cast<uint4 *>(to)[1] = p.hi;
    }
}

__device__ __forceinline__ uint4 values8(uint2 codes, float scale) {
    uint32_t o[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t w = e < 2 ? codes.x : codes.y;
        const float2 f = from_e4m3x2((e & 1 ? w >> 16 : w) & 0xffffu);
        o[e] = sm100::pack_bf16x2(f.x * scale, f.y * scale);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int kDtype>
__global__ void __launch_bounds__(32 * kWarps, 8) latent_values(const LoadArgs a) {
    const int lane = threadIdx.x % 32, b = blockIdx.y, i0 = (blockIdx.x * kWarps + threadIdx.x / 32) * kRows;
    const AttnParams &c = a.cache;
    if (i0 >= a.rows) return;
    // lane r works out where row r lies (bytes), -1: left as it is
    int j = i0 + lane;
    if (a.positions && lane < kRows && j < a.rows) j = __ldg(a.positions + (long long)b * a.rows + j);
    const int L = __ldg(c.seq_lens + b);
    if (L < 0 || L > c.capacity) {
        if (lane == 0 && i0 == 0) set_status(a.status, MLA_ERR_SEQLEN);
        return;
    }
    long long at = -1;
    if (lane < kRows && i0 + lane < a.rows && j >= 0 && j < L) {
        if (c.block_table == nullptr) {
            at = b * a.seq_bytes + (long long)j * a.row_bytes;
        } else {
            const int col = j / c.page_size, page = __ldg(c.block_table + (long long)b * c.max_pages + col);
            if (page < 0 || page >= c.num_pages) set_status(a.status, MLA_ERR_PAGE);
            else at = ((long long)page * c.page_size + (j - col * c.page_size)) * a.row_bytes;
        }
    }
    const uint8_t *kv = static_cast<const uint8_t *>(c.kv);
    __nv_bfloat16 *out = a.out + b * a.out_stride + (long long)i0 * a.width;
    const bool aligned = (reinterpret_cast<uintptr_t>(out) & 31) == 0;  // rows are multiples of 32 bytes
    const int n = a.width / 16;  // pieces of 16 values a row, at most 36
    long long from[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) from[r] = __shfl_sync(~0u, at, r);
    if (kDtype == MLA_KV_E4M3_BLOCKS) {
        // a lane's 16 codes (d_c <= 512), and the keys behind them, two pieces' halves a lane
        const int n_codes = a.d_c / 16, n_keys = 2 * (n - n_codes);
        uint4 v[kRows], key[kRows];
        float scale[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const uint8_t *row = kv + from[r];
            v[r] = key[r] = make_uint4(0, 0, 0, 0);
            scale[r] = 0.f;
            if (from[r] < 0) continue;
            if (lane < n_codes) {
                v[r] = __ldg(reinterpret_cast<const uint4 *>(row) + lane);
                scale[r] = __ldg(reinterpret_cast<const float *>(row + a.d_c) + lane / 8);
            }
            if (lane < n_keys) key[r] = __ldg(reinterpret_cast<const uint4 *>(row + a.d_c + kScaleBytes) + lane);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (from[r] < 0) continue;
            if (lane < n_codes) store_piece(out + r * a.width + 16 * lane,
                                           Piece{values8(make_uint2(v[r].x, v[r].y), scale[r]), values8(make_uint2(v[r].z, v[r].w), scale[r])},
                                           aligned);
            if (lane < n_keys) reinterpret_cast<uint4 *>(out + r * a.width + a.d_c)[lane] = key[r];
        }
    } else {
        // 8 values a lane and turn (32-byte pieces took histories of bf16 rows 68.4 -> 75.8 us, of codes 53.3 ->
        // 61.0: their rows are not whole turns of a warp either way)
        uint4 v[kRows][3];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (from[r] < 0) continue;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int p = lane + 32 * i;
                if (p >= 2 * n) continue;
                if (kDtype == MLA_KV_BF16) {
                    v[r][i] = __ldg(reinterpret_cast<const uint4 *>(kv + from[r]) + p);
                } else {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(kv + from[r]) + p);
                    v[r][i].x = w.x;
                    v[r][i].y = w.y;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            if (from[r] < 0) continue;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const int p = lane + 32 * i;
                if (p >= 2 * n) continue;
                reinterpret_cast<uint4 *>(out + r * a.width)[p] =
                    kDtype == MLA_KV_BF16 ? v[r][i] : values8(make_uint2(v[r][i].x, v[r][i].y), c.kv_scale);
            }
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
