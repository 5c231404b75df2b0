// Block tables, lengths, positions and slots of a batch from its requests' old
// and new lengths; pages from a ring of free ones.
//
// Three sums run over the requests in order: new tokens, pages taken, pages given
// back.  They are sums of non-negative integers that stop at 2^31 - 1, which keeps
// them associative, so every CTA forms all of them by itself (a batch's lengths are
// a few hundred KB at most and come from L2): one launch, no exchange between CTAs
// and no counters to clear.  A CTA keeps the sums before every group of requests in
// shared memory (1024 groups); a token, a page taken or a page given back is then
// found by bisection over the groups and a walk inside one.
//
// A step of 64 requests takes 2.9 us and a turn of 512 (1,300 tokens) 4.0: a launch, the
// lengths, the sums, and one round trip for the pages.  8,191 requests with 2.9 M tokens'
// entries take 19 us against 3.5 for the 24 MB it writes: 5 us for the sums, that every CTA
// repeats, the rest for finding requests and pages: bound by instructions.
#include "layer.h"

namespace mla {
namespace {

constexpr int kGroups = 1024;
constexpr int kBig = 0x7fffffff;

__device__ __forceinline__ int sat_add(int x, int y) { return (int)min((uint32_t)x + (uint32_t)y, (uint32_t)kBig); }

struct Sums {
    int tokens, taken, given;
};
__device__ __forceinline__ Sums add(const Sums &x, const Sums &y) {
    return Sums{sat_add(x.tokens, y.tokens), sat_add(x.taken, y.taken), sat_add(x.given, y.given)};
}

struct Request {
    int old_len, new_len, had, has;  // lengths, and the pages they fill
    bool valid;
    Sums n;  // its own tokens, pages taken, pages given back
};

// m / units for the pool's page size of 64 units tokens, m < 2^25: with l the bits of
// units - 1, ceil(2^(25 + l) / units) is off by less than 1, that is by less than 2^-25 of a
// quotient's step, so the product's integer part is the quotient.
__device__ __forceinline__ int div_units(const PagesArgs &a, int m) {
    return (int)((unsigned long long)(unsigned)m * a.div_magic >> a.div_shift);
}

__device__ __forceinline__ Request make_request(const PagesArgs &a, int old_len, int new_len) {
    Request r;
    r.old_len = old_len;
    r.new_len = new_len;
    const int most = a.max_pages * a.page_size;  // at most 2^30
    r.valid = r.old_len >= 0 && r.new_len >= 0 && r.old_len <= most && r.new_len <= most;
    r.had = r.has = 0;
    r.n = Sums{0, 0, 0};
    if (r.valid) {
        r.had = div_units(a, ((r.old_len + 63) >> 6) + (a.page_size >> 6) - 1);
        r.has = div_units(a, ((r.new_len + 63) >> 6) + (a.page_size >> 6) - 1);
        r.n = Sums{max(r.new_len - r.old_len, 0), max(r.has - r.had, 0), max(r.had - r.has, 0)};
    }
    return r;
}

__device__ __forceinline__ Request load_request(const PagesArgs &a, int b) {
    return make_request(a, __ldg(a.old_lens + b), __ldg(a.new_lens + b));
}

// f(b, request) of requests [b0, b1), four at a time where the lengths allow it.
template <class F>
__device__ __forceinline__ void each_request(const PagesArgs &a, int b0, int b1, bool aligned, F f) {
    int b = b0;
    for (; aligned && b + 4 <= b1; b += 4) {
        const int4 o = __ldg(reinterpret_cast<const int4 *>(a.old_lens + b)), n = __ldg(reinterpret_cast<const int4 *>(a.new_lens + b));
        f(b, make_request(a, o.x, n.x));
        f(b + 1, make_request(a, o.y, n.y));
        f(b + 2, make_request(a, o.z, n.z));
        f(b + 3, make_request(a, o.w, n.w));
    }
    for (; b < b1; ++b) f(b, load_request(a, b));
}

struct Ring {
    int head, count;
    bool ok;
};

// Whether a request whose sums end at `end` (itself included) is served.
__device__ __forceinline__ bool served(const PagesArgs &a, const Ring &ring, const Request &r, const Sums &end) {
    return r.valid && (r.n.taken == 0 || end.taken <= ring.count) && (r.n.tokens == 0 || end.tokens <= a.max_tokens) &&
           (ring.ok || (r.n.taken == 0 && r.n.given == 0));
}

__device__ __forceinline__ int ring_at(const PagesArgs &a, int from, int k) {  // from < num_pages, k <= num_pages
    const unsigned i = (unsigned)from + (unsigned)k;
    return (int)(i >= (unsigned)a.num_pages ? i - a.num_pages : i);
}

// The last group whose sum of member `which` is at most k (groups' first sums are
// non-decreasing and begin at 0).
template <int Sums::*which>
__device__ __forceinline__ int find_group(const Sums *first, int groups, int k) {
    int lo = 0, hi = groups - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (first[mid].*which <= k) lo = mid;
        else hi = mid - 1;
    }
    return lo;
}

// The request that holds item k of member `which`, and the sums before it.
template <int Sums::*which>
__device__ __forceinline__ Request find_request(const PagesArgs &a, const Sums *first, int groups, int per, int k, int &b,
                                                Sums &before) {
    const int g = find_group<which>(first, groups, k);
    b = g * per;
    before = first[g];
    Request r = load_request(a, b);
    // item k lies before the sums of all requests (the callers' bound), so the walk ends
    // inside the batch
    while (sat_add(before.*which, r.n.*which) <= k && b + 1 < a.B) {
        before = add(before, r.n);
        r = load_request(a, ++b);
    }
    return r;
}

// The page that column col of served request b will hold, or -1 with the error recorded.
__device__ __forceinline__ int page_at(const PagesArgs &a, const Ring &ring, const Request &r, const Sums &before, int b, int col) {
    const int page = col < r.had ? a.table[(long long)b * a.max_pages + col]
                                 : __ldg(a.ring + ring_at(a, ring.head, before.taken + col - r.had));
    if (page >= 0 && page < a.num_pages) return page;
    set_status(a.status, MLA_ERR_PAGE);
    return -1;
}

// A thread's place among the tokens: a request, and in it tokens [begin, end) that lie in one
// page (or the rest of a request that is not served, or what lies behind the last token:
// pos -1).
struct TokenRun {
    int b, begin, end, pos, slot;
    Sums before;
    Request r;

    __device__ __forceinline__ TokenRun() : b(-1), begin(0), end(0), pos(-1), slot(-1) {}

    // moves on to the run of token k (not before the last one asked for)
    __device__ __forceinline__ void to(const PagesArgs &a, const Ring &ring, const Sums *first, int groups, int per, int total,
                                       int k) {
        begin = k;
        pos = slot = -1;
        if (k >= total) {
            end = kBig;
            return;
        }
        // the same request, one of the next few, else by bisection
        for (int steps = 0; b >= 0 && sat_add(before.tokens, r.n.tokens) <= k; ++steps) {
            if (steps == 4 || b + 1 >= a.B) {
                b = -1;
            } else {
                before = add(before, r.n);
                r = load_request(a, ++b);
            }
        }
        if (b < 0) r = find_request<&Sums::tokens>(a, first, groups, per, k, b, before);
        end = sat_add(before.tokens, r.n.tokens);
        if (!served(a, ring, r, add(before, r.n))) return;
        pos = r.old_len + (k - before.tokens);
        const int col = div_units(a, pos >> 6), row = pos - col * a.page_size;
        end = min(end, k + a.page_size - row);
        const int page = page_at(a, ring, r, before, b, col);
        if (page >= 0) slot = page * a.page_size + row;
    }
};

__global__ void __launch_bounds__(kGroups) pages_update(const __grid_constant__ PagesArgs a, int per, int quads) {
    __shared__ Sums first[kGroups];
    __shared__ Sums warp_sums[32];
    __shared__ Sums total_s;
    __shared__ int taken_s;
    const int tid = threadIdx.x, lane = tid % 32, warp = tid / 32, groups = (a.B + per - 1) / per;
    Ring ring{__ldg(a.state), __ldg(a.state + 1), true};
    if (ring.head < 0 || ring.head >= a.num_pages || ring.count < 0 || ring.count > a.num_pages) ring.ok = false;

    // sums before every group
    Sums mine{0, 0, 0};
    const bool aligned = per % 4 == 0 && (((uintptr_t)a.old_lens | (uintptr_t)a.new_lens) & 15) == 0;
    const int b0 = min(a.B, tid * per), b1 = min(a.B, b0 + per);
    each_request(a, b0, b1, aligned, [&](int, const Request &r) { mine = add(mine, r.n); });
    Sums run = mine;
    for (int o = 1; o < 32; o <<= 1) {
        Sums up{__shfl_up_sync(~0u, run.tokens, o), __shfl_up_sync(~0u, run.taken, o), __shfl_up_sync(~0u, run.given, o)};
        if (lane >= o) run = add(run, up);
    }
    if (lane == 31) warp_sums[warp] = run;
    if (tid == 0) taken_s = 0;
    __syncthreads();
    if (warp == 0) {
        Sums w = lane < (int)blockDim.x / 32 ? warp_sums[lane] : Sums{0, 0, 0};
        for (int o = 1; o < 32; o <<= 1) {
            Sums up{__shfl_up_sync(~0u, w.tokens, o), __shfl_up_sync(~0u, w.taken, o), __shfl_up_sync(~0u, w.given, o)};
            if (lane >= o) w = add(w, up);
        }
        if (lane < (int)blockDim.x / 32) warp_sums[lane] = w;  // sums up to and with warp `lane`
        if (lane == 31) total_s = w;
    }
    __syncthreads();
    const Sums total = total_s;
    // room for everybody: every valid request is served
    const bool plenty = ring.ok && total.taken <= ring.count && total.tokens <= a.max_tokens;
    {
        // sums before this thread's group: before its warp, and before it within the warp
        Sums before = warp > 0 ? warp_sums[warp - 1] : Sums{0, 0, 0};
        Sums up{__shfl_up_sync(~0u, run.tokens, 1), __shfl_up_sync(~0u, run.taken, 1), __shfl_up_sync(~0u, run.given, 1)};
        if (lane > 0) before = add(before, up);
        if (tid < groups) first[tid] = before;
        // the group's requests: lengths, starts, and what the whole batch takes
        const bool writes = tid % (int)gridDim.x == (int)blockIdx.x;
        int most = 0;
        if (writes || !plenty) each_request(a, b0, b1, aligned, [&](int b, const Request &r) {
            const Sums end = add(before, r.n);
            const bool fits = served(a, ring, r, end);
            if (fits && r.n.taken > 0) most = end.taken;
            if (writes) {
                a.seq_lens[b] = fits ? r.new_len : r.old_len;
                a.token_start[b] = before.tokens;
                if (!fits)
                    set_status(a.status, !r.valid ? MLA_ERR_SEQLEN
                                         : !ring.ok || (r.n.taken > 0 && end.taken > ring.count) ? MLA_ERR_PAGE
                                                                                                 : MLA_ERR_SHAPE);
            }
            before = end;
        });
        if (most > 0) atomicMax(&taken_s, most);
    }
    __syncthreads();
    const int taken = plenty ? total.taken : taken_s;  // served takers are the first ones: their sums do not exceed the ring's count
    // pages given back that the ring has room for (all of them, in a consistent pool)
    const int given = ring.ok ? min(total.given, a.num_pages - ring.count) : 0;
    const int gsize = gridDim.x * blockDim.x, gid = blockIdx.x * blockDim.x + tid;
    if (gid == 0) {
        a.token_start[a.B] = total.tokens;
        a.state_out[0] = ring.ok ? ring_at(a, ring.head, taken) : ring.head;
        a.state_out[1] = ring.ok ? ring.count - taken + given : ring.count;
        if (!ring.ok || given < total.given) set_status(a.status, MLA_ERR_PAGE);
    }

    // The three kinds of items begin a third of the grid apart, so that a small batch's run
    // beside one another, not one after another.
    const int rotated = gid + gsize / 3 < gsize ? gid + gsize / 3 : gid + gsize / 3 - gsize;
    for (int k = gid; k < taken; k += gsize) {
        int b;
        Sums before;
        const Request r = find_request<&Sums::taken>(a, first, groups, per, k, b, before);
        int page = __ldg(a.ring + ring_at(a, ring.head, k));
        if (page < 0 || page >= a.num_pages) {
            set_status(a.status, MLA_ERR_PAGE);
            page = -1;
        }
        a.table[(long long)b * a.max_pages + r.had + (k - before.taken)] = page;
    }
    const int tail = ring.ok ? ring_at(a, ring.head, ring.count) : 0;
    for (int k = rotated; k < given; k += gsize) {
        int b;
        Sums before;
        const Request r = find_request<&Sums::given>(a, first, groups, per, k, b, before);
        a.ring[ring_at(a, tail, k)] = a.table[(long long)b * a.max_pages + r.has + (k - before.given)];
    }

    TokenRun run_of;
    if (!quads) {
        for (int k = gid - gsize / 3 >= 0 ? gid - gsize / 3 : gid - gsize / 3 + gsize; k < a.max_tokens; k += gsize) {
            run_of.to(a, ring, first, groups, per, total.tokens, k);
            a.positions[k] = run_of.pos;
            a.slots[k] = run_of.slot;
        }
        return;
    }
    // Four neighbours a thread, a warp's in a contiguous run of 128-token chunks, so that a
    // thread walks on where it is.
    const bool wide = (((uintptr_t)a.positions | (uintptr_t)a.slots) & 15) == 0;
    const int warps = gsize / 32, w = gid / 32;
    const long long chunks = ((long long)a.max_tokens + 127) / 128, c1 = chunks * (w + 1) / warps;
    for (long long c = chunks * w / warps; c < c1; ++c) {
        const long long k0 = c * 128 + lane * 4;
        const int k1 = (int)min(k0 + 4, (long long)a.max_tokens);
#pragma unroll 1
        for (int k = (int)k0, n; k < k1; k += n) {
            if (k >= run_of.end) run_of.to(a, ring, first, groups, per, total.tokens, k);
            n = min(k1, run_of.end) - k;
            const int dp = run_of.pos >= 0 ? 1 : 0, ds = run_of.slot >= 0 ? 1 : 0;  // -1 stays
            const int pos = run_of.pos + dp * (k - run_of.begin), slot = run_of.slot + ds * (k - run_of.begin);
            if (n == 4 && wide) {
                *reinterpret_cast<int4 *>(a.positions + k) = make_int4(pos, pos + dp, pos + 2 * dp, pos + 3 * dp);
                *reinterpret_cast<int4 *>(a.slots + k) = make_int4(slot, slot + ds, slot + 2 * ds, slot + 3 * ds);
            } else {
#pragma unroll 1
                for (int e = 0; e < n; ++e) {
                    a.positions[k + e] = pos + e * dp;
                    a.slots[k + e] = slot + e * ds;
                }
            }
        }
    }
}

}  // namespace

cudaError_t launch_pages_update(const PagesArgs &a, cudaStream_t st) {
    // requests a group: one, or fours (loaded as 16 bytes)
    const int per = a.B <= kGroups ? 1 : (a.B + 4 * kGroups - 1) / (4 * kGroups) * 4;
    const int groups = (a.B + per - 1) / per;
    // Enough threads for the groups' sums.  Few tokens: one a thread, on at least 12 CTAs, so
    // that the items' loads run side by side (512 requests, 1,300 tokens: 10.8 us on one CTA,
    // 8.4 on 3, 7.4 on 12).  Many, more than two rounds of that: four a thread (7,929 requests,
    // 0.7 M tokens: 15.1 us, one a thread 21.0; 2,997 and 0.1 M: 9.2 us, one a thread 7.2).
    int threads = groups > 0 ? (groups + 31) / 32 * 32 : 32;
    if (threads < 256 && a.max_tokens > threads) threads = 256;
    const int sms = layer_num_sms();
    const int quads = a.max_tokens / 2 > sms * threads ? 1 : 0;
    const long long want = ((long long)a.max_tokens + threads - 1) / threads;
    const int grid = want < 12 ? 12 : want > sms ? sms : (int)want;
    pages_update<<<grid, threads, 0, st>>>(a, per, quads);
    return cudaGetLastError();
}

}  // namespace mla
