// sv_commit_paged.hip -- commit of a verified draft tree's accepted path inside a
// paged KV cache.
//
// The rows of the accepted nodes, depth 1 first, move in place into consecutive
// slots, as in the commit of a contiguous cache.  In place with commit_base <=
// tree_base + 1 a write can only land on the source row of the same or an earlier
// path node (node ids grow by at least one per level).
//
// A slot of request b lies in page page_table[b][slot / page_size], where each
// head's rows are consecutive; a unit is one head's rows of one array g.  One
// wave per request and run of units: it checks the request, looks the source and
// destination rows of up to kWave path nodes up once (lane k holds node k's),
// and then moves the rows of all its units, taken as one list of (unit, node)
// pairs in that order, kPagedVecs instructions' worth at a time.  Rows of
// different units never meet, and a unit's rows are moved in increasing path
// order, each chunk loaded before any of it is stored, so the order argument
// above holds.
//
// Bound by the latency of the lookups (a request's length, path and pages are
// four loads that wait for each other) where there is little to move: 4.2 us for
// one request.  At 64 requests in 72 arrays of 8 heads, rows of 256 bytes (65 MB
// read and written): a wave per unit 91 us; about kCommitWaves waves, here 9
// units each, 31 us; and with non-temporal stores 12.8 us (5.1 TB/s).  The rows
// are read only in the next pass, and as ordinary stores they cost more than
// twice the time of the rest.  2048, 8192 and 16384 waves: 37, 36 and 37 us where
// 4096 took 32; non-temporal loads beside the stores: 17 us.
#include <algorithm>

#include "sv_paged.hpp"
#include "sv_paged_internal.hpp"

namespace sv {
namespace {

constexpr int kPagedVecs = 4;       // 16-byte vectors per lane per chunk
constexpr int kCommitWaves = 4096;  // waves a commit aims for

// Row of `slot` in head 0's arrays (in units of rows), or -1 for a slot outside
// the table or a page outside the cache.
__device__ __forceinline__ long long paged_row(const int32_t *__restrict__ pages, int P, int page_shift,
                                               int num_pages, int Hkv, long long slot) {
    if (slot < 0 || (slot >> page_shift) >= P) return -1;
    const int page = pages[slot >> page_shift];
    if (page < 0 || page >= num_pages) return -1;
    return ((static_cast<long long>(page) * Hkv) << page_shift) + (slot & ((1 << page_shift) - 1));
}

// n / d for n d < 2^32: the product with 2^32 / d rounded up.
struct Divide {
    unsigned d, magic;
    __device__ __forceinline__ explicit Divide(unsigned by)
        : d(by), magic(static_cast<unsigned>(((1ull << 32) + by - 1) / by)) {}
    __device__ __forceinline__ unsigned operator()(unsigned n) const { return d == 1 ? n : __umulhi(n, magic); }
};

__global__ __launch_bounds__(kBlock) void k_commit_paged(
    u32x4 *pages, float *scales, int G, int B, int Hkv, int num_pages, int page_shift, int vec_shift,
    int units_per_wave, int runs, const int32_t *__restrict__ page_table, int P,
    const int32_t *__restrict__ tree_base, const int32_t *__restrict__ commit_base,
    const int32_t *__restrict__ accept_len, const int32_t *__restrict__ path_nodes, int N,
    int32_t *__restrict__ status) {
    const int lane = threadIdx.x & (kWave - 1);
    const long long wave = static_cast<long long>(blockIdx.x) * kWavesPerBlock + (threadIdx.x >> 6);
    if (wave >= static_cast<long long>(B) * runs) return;
    const int b = uniform(static_cast<int>(wave / runs)), run = uniform(static_cast<int>(wave % runs));
    const int32_t *path = path_nodes + static_cast<long long>(b) * N;
    const int32_t *table = page_table + static_cast<long long>(b) * P;
    const int d = uniform(accept_len[b]);
    const long long tb = uniform(tree_base[b]), cb = uniform(commit_base[b]);
    const int j0 = lane < N ? path[lane] : 0;  // fetched with the scalars above

    // request check (every wave of the request reaches the same verdict); lane k
    // keeps the rows of node k for paths of up to kWave nodes
    int code = 0;
    long long src = 0, dst = 0;
    if (d < 0 || d > N - 1) {
        code = 2;
    } else if (d > 0) {
        bool bad = false, out = false;
        for (int k = lane; k < d; k += kWave) {
            const int j = k < kWave ? j0 : path[k];
            const int prev = k == 0 ? 0 : path[k - 1];
            if (j < 1 || j >= N || j <= prev) {
                bad = true;
                continue;
            }
            src = paged_row(table, P, page_shift, num_pages, Hkv, tb + j);
            dst = paged_row(table, P, page_shift, num_pages, Hkv, cb + k);
            if (src < 0 || dst < 0) out = true;
        }
        if (ballot(bad) != 0)
            code = 2;
        else if (ballot(out) != 0)
            code = 1;
        else if (cb >= tb + 2 && cb < tb + N)
            code = 3;
    }
    if (run == 0 && lane == 0 && status) status[b] = code;
    if (code != 0 || d == 0) return;

    const int u0 = run * units_per_wave, units = min(units_per_wave, G * Hkv - u0);
    const long long rows = (static_cast<long long>(num_pages) * Hkv) << page_shift;  // rows of one array
    // offset of a unit's rows (Hkv <= 32768, so the quotient's bound holds)
    const int g0 = u0 / Hkv, h0 = u0 - g0 * Hkv;
    const Divide by_head(static_cast<unsigned>(Hkv));
    auto unit_row = [&](unsigned unit) {
        const unsigned g = by_head(h0 + unit), h = h0 + unit - g * Hkv;
        return static_cast<long long>(g0 + g) * rows + (static_cast<long long>(h) << page_shift);
    };
    const int rows_per = kWave >> vec_shift;  // rows one instruction of the wave moves
    const int sub = lane >> vec_shift, v = lane & ((1 << vec_shift) - 1);
    for (int k0 = 0; k0 < d; k0 += kWave) {
        const int nk = min(kWave, d - k0);
        if (d > kWave) {
            const int k = min(lane, nk - 1) + k0;
            src = paged_row(table, P, page_shift, num_pages, Hkv, tb + path[k]);
            dst = paged_row(table, P, page_shift, num_pages, Hkv, cb + k);
        }
        const Divide by_nk(static_cast<unsigned>(nk));
        const int pairs = units * nk;
        for (int p0 = 0; p0 < pairs; p0 += rows_per * kPagedVecs) {
            u32x4 x[kPagedVecs];
            long long to[kPagedVecs];
#pragma unroll
            for (int t = 0; t < kPagedVecs; ++t) {
                const unsigned p = static_cast<unsigned>(min(p0 + t * rows_per + sub, pairs - 1));
                const unsigned unit = by_nk(p), k = p - unit * nk;
                const long long off = unit_row(unit);
                x[t] = pages[((off + __shfl(src, k, kWave)) << vec_shift) + v];
                to[t] = ((off + __shfl(dst, k, kWave)) << vec_shift) + v;
            }
            wait_own_stores();  // every load of the chunk has returned before any store
#pragma unroll
            for (int t = 0; t < kPagedVecs; ++t)
                if (p0 + t * rows_per + sub < pairs) __builtin_nontemporal_store(x[t], pages + to[t]);
        }
        if (!scales) continue;
        for (int p0 = 0; p0 < pairs; p0 += kWave) {
            const unsigned p = static_cast<unsigned>(min(p0 + lane, pairs - 1));
            const unsigned unit = by_nk(p), k = p - unit * nk;
            const long long off = unit_row(unit);
            const float x = scales[off + __shfl(src, k, kWave)];
            const long long at = off + __shfl(dst, k, kWave);
            wait_own_stores();
            if (p0 + lane < pairs) scales[at] = x;
        }
    }
}

}  // namespace

static int units_per_wave(int G, int B, int Hkv) {
    const long long units = static_cast<long long>(G) * Hkv;
    return static_cast<int>(std::min<long long>(64, std::max<long long>(1, (units * B + kCommitWaves - 1) / kCommitWaves)));
}

long long commit_paged_groups(int G, int B, int Hkv) {
    const long long per = units_per_wave(G, B, Hkv), runs = (static_cast<long long>(G) * Hkv + per - 1) / per;
    return (B * runs + kWavesPerBlock - 1) / kWavesPerBlock;
}

hipError_t launch_commit_paged(void *pages, float *scales, int G, int B, int Hkv, int num_pages, int page_shift,
                               int vecs, const int32_t *page_table, int P, const int32_t *tree_base,
                               const int32_t *commit_base, const int32_t *accept_len, const int32_t *path_nodes,
                               int N, int32_t *status, hipStream_t s) {
    const int per = units_per_wave(G, B, Hkv);
    const int runs = static_cast<int>((static_cast<long long>(G) * Hkv + per - 1) / per);
    const unsigned groups = static_cast<unsigned>(commit_paged_groups(G, B, Hkv));
    return launch_kernel(k_commit_paged, dim3(groups), dim3(kBlock), 0, s,
                         static_cast<u32x4 *>(pages), scales, G, B, Hkv, num_pages, page_shift,
                         __builtin_ctz(static_cast<unsigned>(vecs)), per, runs, page_table, P, tree_base, commit_base,
                         accept_len, path_nodes, N, status);
}

}  // namespace sv
