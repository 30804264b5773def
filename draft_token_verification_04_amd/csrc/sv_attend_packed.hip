// sv_attend_packed.hip -- causal attention of packed sequences (whole prompts, or
// their next chunks) over a paged cache that holds them.
//
// Row j of request b (token starts[b] + j) sees the slots s < base[b] + j + 1:
//   w_s = scale q . k_s,  out = sum exp(w_s - m) v_s / l,  lse = m + log l.
//
// The G query heads that share a KV head and a request's tokens form the rows of one
// product, r = j G + g; a workgroup takes 32 of them for each of its four waves (or
// eight), and all walk the same slots, half a tile of 32 at a time:
//   S^T = K Q^T   (32x32x16 MFMAs; lane l holds 16 of the 32 slots' scores of row
//                  l % 32, the other 16 are lane l ^ 32's)
//   online softmax: a row's weights are relative to a reference that moves only where a
//                  score is more than 8 (log2) above it; the sum meets its other half
//                  at the end.  A bf16 cache's sums begin at minus the reference, so
//                  nothing is subtracted
//   O^T += V^T P^T: a lane's weights of 16 slots are, in the order (4 slots, lane
//                  half), the 8 that MFMA's right operand wants from it; the left
//                  operand V^T comes from rows of V through transposing LDS reads.
// Half a tile is what the registers hold twice (O, the queries, two halves' scores):
// one half's weights are made out of its scores while the matrix cores form the next
// half's scores, then its values are mixed while the next half's maximum is taken; each
// phase asks LDS for the first fragments of the one behind it.  K's window of 64 slots
// runs half a tile ahead of V's, so a barrier falls between tiles only.  A bf16 cache's
// rows go straight from memory to LDS, two stages of each; an e4m3 cache's pass through
// registers and are widened to bf16 (exactly) on the way, its scales multiply scores and
// weights.  16-byte chunks of a row are permuted so that the reads of several rows meet
// distinct banks.
//
// Bound by the matrix cores and the exponentials beside them, two waves on a SIMD: a
// half tile is 512 cycles of products and about as many of vector instructions.  8191
// tokens, 32 query heads over 8 of 128, bf16: 560 us, 0.98 PFLOP/s, where large library
// products of bf16 reach 1.43 (64-slot steps with rows staged through registers: 708).
// With short prompts a workgroup's beginning and end, which nothing of its own covers,
// take a quarter: 16 prompts, 17500 tokens in all: 327 us, 0.66 PFLOP/s.
//
// Everything between the loads and the stores is fp32, but the weights, which enter
// the second product rounded to bf16 (at most 2^-9 each, independent of one another);
// their sum l takes them unrounded.
//
// Masked slots: scores are replaced, never added to.  Rows of V behind the last slot
// seen are zeroed; a non-finite value of V at a slot that some row of the workgroup
// does not see is left out of the product and added for the rows that see it.
#include <algorithm>

#include "sv_paged.hpp"
#include "sv_prompt_internal.hpp"

namespace sv {
namespace {

#define SV_LDS __attribute__((address_space(3)))
#define SV_GLOBAL __attribute__((address_space(1)))

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kSlots = 64;         // slots of a tile
constexpr float kSlack = 8.0f;     // weights may reach 2^kSlack before the reference moves
// The reference of a row that has met no score.
constexpr float kNoRef = -3.4028234663852886e38f;

// Natural log of L 2^(m c).
__device__ __forceinline__ float log_sum(float m, float L, float c) {
    return static_cast<float>((static_cast<double>(m) * static_cast<double>(c) + static_cast<double>(log2f(L))) * 0.6931471805599453);
}

// Over the lanes l and l ^ 32 that hold one row.
__device__ __forceinline__ float pair_max(float v) {
    const unsigned u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float pair_sum(float v) {
    const unsigned u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}

__device__ __forceinline__ bf16x8 as_bf16x8(unsigned a, unsigned b, unsigned c, unsigned d) {
    const u32x4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ f32x16 mfma32(const bf16x8 &a, const bf16x8 &b, const f32x16 &c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Whether a word of two bf16 values holds an infinity or NaN, and the word with
// those cleared.
__device__ __forceinline__ bool has_nonfinite(unsigned w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
__device__ __forceinline__ unsigned finite_only(unsigned w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int I>
struct Index {
    static constexpr int value = I;
};
template <int I, int N, typename F>
__device__ __forceinline__ void unrolled(F &&f) {
    if constexpr (I < N) {
        f(Index<I>{});
        unrolled<I + 1, N>(f);
    }
}

// 16 bytes, or a transposed read's 8, at LDS address at + OFF; there once `arrived` has
// named the register.  (With loads into LDS on their way the compiler would wait for all
// of them before each LDS read of its own.)
template <int OFF>
__device__ __forceinline__ u32x4 lds_read(uint32_t at) {
    static_assert(OFF >= 0 && OFF < 65536, "ds offset range");
    u32x4 r;
    asm volatile("ds_read_b128 %0, %1 offset:%2" : "=v"(r) : "v"(at), "i"(OFF));
    return r;
}
template <int OFF>
__device__ __forceinline__ u32x2 lds_read_turned(uint32_t at) {
    static_assert(OFF >= 0 && OFF < 65536, "ds offset range");
    u32x2 r;
    asm volatile("ds_read_b64_tr_b16 %0, %1 offset:%2" : "=v"(r) : "v"(at), "i"(OFF));
    return r;
}
// All but the wave's N youngest LDS reads have arrived, these registers among them.
template <int N>
__device__ __forceinline__ void arrived(u32x4 &a) {
    asm volatile("s_waitcnt lgkmcnt(%1)" : "+v"(a) : "i"(N));
}
template <int N>
__device__ __forceinline__ void arrived(u32x2 &a, u32x2 &b) {
    asm volatile("s_waitcnt lgkmcnt(%2)" : "+v"(a), "+v"(b) : "i"(N));
}

// Keeps a value's computation where it is written.
__device__ __forceinline__ void pin(float &x) { asm volatile("" : "+v"(x)); }

// The row tile a workgroup takes: rows [r0, r0 + rows of a workgroup) of request b.
struct Unit {
    int b, tile, first, count, base;  // request, its tile, first token, tokens, and cached ones before
    bool last;                        // the request's last tile
};
// Row tiles of a request of `count` tokens, or one more than the launch has if that is
// less (so that 64 requests' sum fits).
__device__ __forceinline__ int tiles_of(const PackedArgs &a, int count, int rows) {
    return static_cast<int>(min((static_cast<long long>(count) * a.G + rows - 1) / rows, a.units + 1LL));
}
// Tokens of request i, 0 where its bounds are malformed.
__device__ __forceinline__ int request_tokens(const PackedArgs &a, int i, int *first) {
    const int lo = a.starts[i], hi = a.starts[i + 1];
    *first = lo;
    return lo >= 0 && hi >= lo && hi <= a.T ? hi - lo : 0;
}
// The sum over the wave's lanes up to this one: within rows of 16 lanes, then the rows'
// last lanes to the rows behind.
__device__ __forceinline__ int running_sum(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast 15, 31
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}
// The u-th row tile, requests in order, or b = -1 behind the last.  A wave sums the
// tiles of 64 requests at a time.
__device__ __forceinline__ Unit find_unit(const PackedArgs &a, int u, int rows, int lane) {
    long long before = 0;
    for (int i0 = 0; i0 < a.B; i0 += kWave) {
        int first = 0, count = 0, base = 0;
        if (i0 + lane < a.B) {
            count = request_tokens(a, i0 + lane, &first);
            if (a.base) base = a.base[i0 + lane];
        }
        const int mine = tiles_of(a, count, rows), up = running_sum(mine);
        const uint64_t past = __ballot(before + up > u);
        if (past) {
            const int at = __ffsll(static_cast<long long>(past)) - 1;
            Unit r;
            r.b = i0 + at;
            r.count = uniform(__shfl(count, at, kWave));
            r.first = uniform(__shfl(first, at, kWave));
            r.base = uniform(__shfl(base, at, kWave));
            const int tiles = uniform(__shfl(mine, at, kWave));
            r.tile = uniform(static_cast<int>(u - before - (__shfl(up, at, kWave) - tiles)));
            r.last = r.tile == tiles - 1;
            return r;
        }
        before += __shfl(up, kWave - 1, kWave);
    }
    return Unit{-1, 0, 0, 0, 0, false};
}

// Splits of a row tile whose rows see `tiles` tiles of slots: as many as have a
// least run.
constexpr int kLeastRun = 8;
__device__ __forceinline__ int splits_of(int tiles, int S) { return max(1, min(S, tiles / kLeastRun)); }

// Where 16-byte chunk c of row r lies in its row of LDS.  K is read by rows of one
// chunk (32 rows at once), V by four rows of two or four chunks.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) {
    return D == 64 ? c ^ ((r >> 1) & 7) : c ^ (r & 15);
}
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    return D == 64 ? c ^ (2 * (r & 3)) : c ^ (4 * (r & 3)) ^ (2 * ((r >> 1) & 1));
}

template <int D, bool E4M3, int WAVES>
__global__ __launch_bounds__(WAVES *kWave, D > 128 ? 1 : 2) void k_attend_packed(PackedArgs a) {
    constexpr int kThreads = WAVES * kWave;
    constexpr int kRows = 32 * WAVES;             // of a workgroup
    constexpr int kSteps = D / 16;                // of the first product
    constexpr int kVals = D / 32;                 // 32-value blocks of a row of V
    constexpr int kRowB = D * 2;                  // bytes of a row in LDS
    constexpr int kElem = E4M3 ? 1 : 2;
    constexpr int kRowChunks = D * kElem / 16;    // 16-byte chunks of a row in memory
    __shared__ __align__(1024) char kv[2][2][kSlots * kRowB];  // [K, V][tile's parity]
    __shared__ __align__(16) float scales[2][2][kSlots];       // e4m3: of the tile's slots, likewise
    __shared__ int odd_tile[2];                   // first and last tile where V has a non-finite value
    const int lane = threadIdx.x & (kWave - 1), w = uniform(static_cast<int>(threadIdx.x >> 6));
    const int half = lane >> 5, col = lane & 31;

    // requests without rows, with malformed bounds, or (where bounds overlap) behind the
    // last row tile of the launch
    if (blockIdx.x == 0 && a.status && w == 0) {
        long long before = 0;
        for (int i0 = 0; i0 < a.B; i0 += kWave) {
            const int b = i0 + lane;
            int first = 0;
            const int count = b < a.B ? request_tokens(a, b, &first) : 0;
            const long long up = before + running_sum(tiles_of(a, count, kRows));
            if (b < a.B) {
                if (count == 0)
                    a.status[b] = first == a.starts[b + 1] && first >= 0 && first <= a.T ? 0 : 2;
                else if (up > a.units)
                    a.status[b] = 2;
            }
            before = __shfl(up, kWave - 1, kWave);
        }
    }
    // the rows that see most come first
    const int h = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
    const int split = rest % a.S, u = a.units - 1 - rest / a.S;
    const Unit un = find_unit(a, u, kRows, lane);
    if (un.b < 0) return;
    const int base = un.base;
    const long long r0 = static_cast<long long>(un.tile) * kRows;
    const int rows = static_cast<int>(min(static_cast<long long>(un.count) * a.G - r0, static_cast<long long>(kRows)));
    // slots that exist, and the slots that the tile's first and last row see
    const long long exist = static_cast<long long>(a.P) << a.page_shift;
    const long long want = static_cast<long long>(base) + (r0 + rows - 1) / a.G + 1;
    const bool inside = base >= 0;
    const int total = inside ? static_cast<int>(min(want, exist)) : 0;
    const int least = inside ? static_cast<int>(min(static_cast<long long>(base) + r0 / a.G + 1, exist)) : 0;
    // the first slot that does not exist (before any row's last, where the base is negative)
    int first_bad = inside ? (want > exist ? static_cast<int>(exist) : 0x7fffffff) : -0x7fffffff - 1;

    const int tiles = (total + kSlots - 1) / kSlots;
    const int active = splits_of(tiles, a.S);
    if (split >= active) return;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / active);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / active);

    // this lane's query row and how many slots it sees; the wave's least, and the end of
    // its tiles
    const int r = w * 32 + col;
    const bool live = r < rows;
    const long long at = r0 + (live ? r : 0);
    const int j = static_cast<int>(at / a.G), head = h * a.G + static_cast<int>(at - static_cast<long long>(j) * a.G);
    const int token = un.first + j;
    const int sees = live ? static_cast<int>(min(static_cast<long long>(base) + j + 1, exist + 1)) : 0;
    bf16x8 q[kSteps];
    {
        const uint16_t *p = a.q + token * a.q_stride + static_cast<long long>(head) * D + half * 8;
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
            u32x4 x = {0, 0, 0, 0};
            if (live) x = *reinterpret_cast<const u32x4 *>(p + c * 16);
            q[c] = __builtin_bit_cast(bf16x8, x);
        }
    }
    int wave_least = 0, wave_end = t0;
    {
        const long long ra = r0 + w * 32, rb = min(ra + 32, r0 + rows) - 1;
        if (rb >= ra) {
            wave_least = static_cast<int>(min(base + ra / a.G + 1, exist + 1));
            const long long most = min(base + rb / a.G + 1, exist);
            wave_end = static_cast<int>(min(static_cast<long long>(t1), (most + kSlots - 1) / kSlots));
        }
    }

    f32x16 o[kVals];
    float m = kNoRef, l = 0.0f;  // reference (a score q.k), and the weights' sum
#pragma unroll
    for (int i = 0; i < kVals; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[i][e] = 0.0f;

    // ---- rows from memory to LDS: V's stage holds a tile; K's window j, half a tile
    // earlier, the 64 slots from 64 j - 32 on.  Wave w brings the w-th 16 (of eight waves:
    // 8) of them, which lie in one page; a bf16 cache's straight into LDS, an e4m3 cache's through registers
    const int32_t *table = a.page_table + static_cast<long long>(un.b) * a.P;
    const int page_mask = (1 << a.page_shift) - 1;
    constexpr int kLaneRows = kWave / kRowChunks;  // rows that one load of a wave covers
    constexpr int kWaveRows = kSlots / WAVES, kLoads = kWaveRows / kLaneRows;
    static_assert(kLoads >= 1, "a wave's rows fill its loads");
    constexpr int kTileB = kSlots * kRowB;
    const int row_in = lane / kRowChunks, chunk = lane % kRowChunks;
    struct Stream {
        int ids, end;  // lane i: the page of 16 slots, the i-th of 64 groups before `end`
        u32x4 x[E4M3 ? kLoads : 1];
        float scale;
    } ks, vs;
    ks.end = vs.end = -0x7fffffff;
    auto load = [&](Stream &s, int slot, const void *pages, const float *scale, char *stage, bool is_k) {
        const int group0 = slot / 16 - t0 * 4;  // in groups of 16 slots from the first tile on
        if (group0 >= s.end) {
            s.end = group0 + kWave;
            const int mine = slot + 16 * lane;
            s.ids = mine >= 0 && mine < total ? table[mine >> a.page_shift] : 0;
            if (s.ids < 0 || s.ids >= a.num_pages) {
                if (mine >= t0 * kSlots && mine < t1 * kSlots) first_bad = min(first_bad, mine);
                s.ids = 0;
            }
        }
        const int page = __builtin_amdgcn_readlane(s.ids, group0 + kWaveRows * w / 16 - (s.end - kWave));
        const long long row = ((static_cast<long long>(page) * a.Hkv + h) << a.page_shift) + ((slot + kWaveRows * w) & page_mask);
        const char *from = static_cast<const char *>(pages) + row * (D * kElem);
        if constexpr (E4M3) {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) s.x[i] = *reinterpret_cast<const u32x4 *>(from + (i * kLaneRows + row_in) * (D * kElem) + chunk * 16);
            s.scale = scale[row + lane % kWaveRows];
        } else {
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int r = i * kLaneRows + row_in, at = kWaveRows * w + r;
                const int c = is_k ? k_chunk<D>(at, chunk) : v_chunk<D>(at, chunk);  // what place `chunk` holds
                __builtin_amdgcn_global_load_lds((const SV_GLOBAL void *)(from + r * kRowB + c * 16),
                                                 (SV_LDS void *)(stage + kWaveRows * w * kRowB + i * 1024), 16, 0, 0);
            }
        }
    };
    auto load_k = [&](int window) {
        load(ks, window * kSlots - kSlots / 2, a.k_pages, a.k_scale, kv[0][(window - t0) & 1], true);
    };
    auto load_v = [&](int tile) { load(vs, tile * kSlots, a.v_pages, a.v_scale, kv[1][(tile - t0) & 1], false); };
    auto store = [&](Stream &s, char *stage, float *scale, bool is_k) {  // e4m3: widened
#pragma unroll
        for (int i = 0; i < (E4M3 ? kLoads : 0); ++i) {
            const int r = kWaveRows * w + i * kLaneRows + row_in;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                u32x4 y;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    y[2 * e] = e4m3_to_bf16<false>(s.x[i][2 * p + e]);
                    y[2 * e + 1] = e4m3_to_bf16<true>(s.x[i][2 * p + e]);
                }
                const int c = is_k ? k_chunk<D>(r, chunk * 2 + p) : v_chunk<D>(r, chunk * 2 + p);
                *reinterpret_cast<u32x4 *>(stage + r * kRowB + c * 16) = y;
            }
        }
        if (lane < kWaveRows) scale[kWaveRows * w + lane] = s.scale;
    };
    auto note_odd = [&](int tile) {
        atomicMin(&odd_tile[0], tile);
        atomicMax(&odd_tile[1], tile);
    };
    auto store_k = [&](int window) {
        if constexpr (E4M3) {
            ks.scale *= a.c;
            store(ks, kv[0][(window - t0) & 1], scales[0][(window - t0) & 1], true);
        }
    };
    auto store_v = [&](int tile) {
        if constexpr (E4M3) {
            if ((tile + 1) * kSlots > least && !isfinite(vs.scale)) {  // as a value is, in clean_v
                vs.scale = 0.0f;
                note_odd(tile);
            }
            store(vs, kv[1][(tile - t0) & 1], scales[1][(tile - t0) & 1], false);
        }
    };
    // A tile's values that some row does not see: those behind the last slot zeroed, and
    // what is not finite left out (and noted)
    auto clean_v = [&](int tile) {
        char *stage = kv[1][(tile - t0) & 1];
        bool odd = false;
        for (int i = threadIdx.x; i < kTileB / 16; i += kThreads) {
            u32x4 y = *reinterpret_cast<u32x4 *>(stage + i * 16);
            const bool behind = tile * kSlots + i / (kRowB / 16) >= total;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (behind) y[e] = 0;
                odd |= has_nonfinite(y[e]);
                y[e] = finite_only(y[e]);
            }
            *reinterpret_cast<u32x4 *>(stage + i * 16) = y;
        }
        if (odd) note_odd(tile);
    };

    // ---- the parts of a half tile's work; slot 64 tile + 32 f + 8 (e / 4) + 4 half + e % 4
    // of row col is score s[e] of half f
    uint32_t kp[kSteps], vp[kVals];  // LDS addresses in the stage of even windows and tiles
    const uint32_t k0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((SV_LDS char *)&kv[0][0][0]));
    const uint32_t v0 = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((SV_LDS char *)&kv[1][0][0]));
#pragma unroll
    for (int c = 0; c < kSteps; ++c) kp[c] = k0 + col * kRowB + k_chunk<D>(col, 2 * c + half) * 16;
#pragma unroll
    for (int d = 0; d < kVals; ++d) {
        // lane i of 16 addresses 4 values of row i / 4 and gets value i of the 4 rows
        const int r = 4 * half + (lane & 15) / 4, byte = (d * 32 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;
        vp[d] = v0 + r * kRowB + v_chunk<D>(r, byte / 16) * 16 + byte % 16;
    }
    const SV_LDS f32x4 *kscale = (const SV_LDS f32x4 *)&scales[0][0][0] + half, *vscale = (const SV_LDS f32x4 *)&scales[1][0][0] + half;
    auto k_part = [&](auto par, auto f, auto c) {
        return lds_read<decltype(f)::value * 32 * kRowB + decltype(par)::value * kTileB>(kp[decltype(c)::value]);
    };
    struct Turned {
        u32x2 lo, hi;
    };
    auto v_part = [&](auto par, auto f, auto i) {
        constexpr int g = decltype(i)::value / kVals, d = decltype(i)::value % kVals;
        constexpr int kOff = (decltype(f)::value * 32 + g * 16) * kRowB + decltype(par)::value * kTileB;
        Turned t;
        t.lo = lds_read_turned<kOff>(vp[d]);
        t.hi = lds_read_turned<kOff + 8 * kRowB>(vp[d]);
        return t;
    };
    constexpr int kMixes = 2 * kVals, kAhead = kSteps < 4 ? kSteps - 1 : 3;  // fragments on their way
    // minus the reference, and as what a bf16 cache's sums begin at
    float minus_m = 0.0f;
    f32x16 minus;
#pragma unroll
    for (int e = 0; e < 16; ++e) minus[e] = 0.0f;
    // Fragments on their way: a phase asks for the first of the next while it ends, so none
    // begins with a wait.  Entry n of a phase goes to place n % (kAhead + 1).
    u32x4 kf[kAhead + 1];
    Turned vf[kAhead + 1];
    auto ask_k = [&](auto par, auto f, auto n) {  // of the products that half f's weights run beside
        kf[decltype(n)::value % (kAhead + 1)] = k_part(Index<1 - decltype(par)::value>{}, f, n);
    };
    auto ask_v = [&](auto par, auto f, auto n) { vf[decltype(n)::value % (kAhead + 1)] = v_part(par, f, n); };
    // A half's weights out of its scores (relative to the reference), and the next half's
    // products, a product to a few weights.  The sums of a bf16 cache begin at minus the
    // reference: what leaves them is already relative to it.
    auto weigh = [&](auto par, auto f, f32x16 &s, f32x16 &next, bf16x8 (&p)[2]) {
        constexpr int F = decltype(f)::value;
        float sum[2] = {0, 0};
        f32x4 vs4;
        unrolled<0, kSteps>([&](auto cc) {
            constexpr int c = decltype(cc)::value, kPer = 16 / kSteps;
            constexpr int kLeft = kSteps - 1 - c < kAhead ? kSteps - 1 - c : kAhead;  // K's fragments behind this one
            if constexpr (c + kAhead < kSteps)
                ask_k(par, f, Index<c + kAhead>{});
            else
                ask_v(par, f, Index<c + kAhead - kSteps>{});
            arrived<kLeft + 2 * (kAhead - kLeft)>(kf[c % (kAhead + 1)]);
            next = mfma32(__builtin_bit_cast(bf16x8, kf[c % (kAhead + 1)]), q[c], c == 0 ? minus : next);
            unrolled<0, kPer>([&](auto xx) {
                constexpr int e = c * kPer + decltype(xx)::value;
                if constexpr (E4M3 && e % 4 == 0) vs4 = vscale[decltype(par)::value * (kSlots / 4) + 8 * F + 2 * (e / 4)];
                float y = fast_exp2(E4M3 ? s[e] : s[e] * a.unit);
                sum[e % 2] += y;
                if constexpr (E4M3) y *= vs4[e % 4];
                s[e] = y;
                if constexpr (e % 8 == 7)
                    p[e / 8] = as_bf16x8(pack_bf16(s[e - 7], s[e - 6]), pack_bf16(s[e - 5], s[e - 4]), pack_bf16(s[e - 3], s[e - 2]),
                                         pack_bf16(s[e - 1], s[e]));
            });
            pin(sum[0]);
            pin(sum[1]);
            __builtin_amdgcn_sched_barrier(0);
        });
        l += sum[0] + sum[1];
    };
    // The half's values mixed, and the next half's largest score (an e4m3 cache's scores
    // scaled, into units of log2, and made relative first)
    auto mix = [&](auto par, auto f, const bf16x8 (&p)[2], f32x16 &next) {
        constexpr int F = decltype(f)::value, kWindow = 1 - decltype(par)::value;
        float most = -__builtin_huge_valf();
        f32x4 ks4;
        unrolled<0, kMixes>([&](auto ii) {
            constexpr int i = decltype(ii)::value, g = i / kVals, d = i % kVals;
            constexpr int kLeft = kMixes - 1 - i < kAhead ? kMixes - 1 - i : kAhead;
            if constexpr (i + kAhead < kMixes)
                ask_v(par, f, Index<i + kAhead>{});
            else if constexpr (F == 0)  // the second half's window is there already
                ask_k(par, Index<1>{}, Index<i + kAhead - kMixes>{});
            Turned &v = vf[i % (kAhead + 1)];
            arrived<2 * kLeft + (F == 0 ? kAhead - kLeft : 0)>(v.lo, v.hi);
            o[d] = mfma32(as_bf16x8(v.lo.x, v.lo.y, v.hi.x, v.hi.y), p[g], o[d]);
            if constexpr (i >= kVals) {  // the scores are there by now
                constexpr int kPairs = 8 / kVals;
                unrolled<0, kPairs>([&](auto xx) {
                    constexpr int e = ((i - kVals) * kPairs + decltype(xx)::value) * 2;
                    if constexpr (E4M3) {
                        if constexpr (e % 4 == 0) ks4 = kscale[kWindow * (kSlots / 4) + 8 * F + 2 * (e / 4)];
                        next[e] = fmaf(next[e], ks4[e % 4], minus_m);
                        next[e + 1] = fmaf(next[e + 1], ks4[e % 4 + 1], minus_m);
                    }
                    most = fmaxf(most, fmaxf(next[e], next[e + 1]));
                });
                pin(most);
            }
            __builtin_amdgcn_sched_barrier(0);
        });
        return most;
    };
    // Masks the scores from slot `slot` on; the largest then
    auto masked = [&](int slot, f32x16 &s) {
        float most = -__builtin_huge_valf();
        const int seen = sees - slot - 4 * half;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            if (8 * (e / 4) + e % 4 >= seen) s[e] = -__builtin_huge_valf();
            most = fmaxf(most, s[e]);
        }
        return most;
    };
    // Moves the references where a score is far above its own, and to a row's first score
    auto refer = [&](float most, f32x16 &s) {
        const bool moves = m == kNoRef ? most > -__builtin_huge_valf() : most * a.unit > kSlack;
        if (__ballot(moves) == 0) return;
        const float up = pair_max(most);
        const bool first = m == kNoRef;
        const float by = first ? (up > -__builtin_huge_valf() ? up : 0.0f) : fmaxf(up, 0.0f);
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] -= by;
        const float f = first ? 1.0f : fast_exp2(-by * a.unit);  // a first reference has nothing to turn
        l *= f;
#pragma unroll
        for (int i = 0; i < kVals; ++i) o[i] *= f;
        m = first ? (up > -__builtin_huge_valf() ? up : kNoRef) : m + by;
        minus_m = m == kNoRef ? 0.0f : -m;
        if constexpr (!E4M3) {
#pragma unroll
            for (int e = 0; e < 16; ++e) minus[e] = minus_m;
        }
    };

    if (threadIdx.x < 2) odd_tile[threadIdx.x] = threadIdx.x == 0 ? 0x7fffffff : -1;
    __syncthreads();
    if (t0 < t1) {
        load_k(t0);
        load_v(t0);
        store_k(t0);
        store_v(t0);
        load_k(t0 + 1);
        store_k(t0 + 1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    __syncthreads();
    // Half tiles, one after the other: the weights of one come out of its scores while the
    // next one's are formed (behind the wave's last half, scores that nothing reads), then
    // its values are mixed.
    f32x16 s, next;
    float most = 0.0f;
    if (t0 < wave_end) {
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = 0.0f;
        unrolled<0, kSteps>([&](auto c) {
            u32x4 x = k_part(Index<0>{}, Index<1>{}, c);
            arrived<0>(x);
            s = mfma32(__builtin_bit_cast(bf16x8, x), q[decltype(c)::value], s);
        });
        if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 16; ++e) s[e] *= kscale[8 + 2 * (e / 4)][e % 4];
        }
        most = masked(t0 * kSlots, s);
    }
    auto turn = [&](auto par, int tile) {
        // the next window of K and this tile's V are there; every wave is done with the ones
        // before
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
        __syncthreads();
        if ((tile + 1) * kSlots > least) {
            clean_v(tile);
            __syncthreads();
        }
        const bool more = tile + 1 < t1;
        if (more) {
            load_k(tile + 2);
            load_v(tile + 1);
        }
        if (tile < wave_end) {
            bf16x8 p[2];
            unrolled<0, kAhead>([&](auto n) { ask_k(par, Index<0>{}, n); });
            refer(most, s);
            weigh(par, Index<0>{}, s, next, p);
            most = mix(par, Index<0>{}, p, next);
            if ((tile + 1) * kSlots > wave_least) most = masked(tile * kSlots + 32, next);
            refer(most, next);
            weigh(par, Index<1>{}, next, s, p);
            most = mix(par, Index<1>{}, p, s);
            if ((tile + 2) * kSlots > wave_least) most = masked((tile + 1) * kSlots, s);
        }
        if (more) {
            store_k(tile + 2);
            store_v(tile + 1);
        }
    };
    int tile = t0;
    for (; tile + 1 < t1; tile += 2) {
        turn(Index<0>{}, tile);
        turn(Index<1>{}, tile + 1);
    }
    if (tile < t1) turn(Index<0>{}, tile);

    __syncthreads();
    if (odd_tile[0] <= odd_tile[1]) {
        // the non-finite values of V, one by one, for the rows that see their slot
        const int s1 = min((odd_tile[1] + 1) * kSlots, total);
        for (int slot = odd_tile[0] * kSlots; slot < s1; ++slot) {
            const int page = uniform(table[slot >> a.page_shift]);
            const long long row = (((page < 0 || page >= a.num_pages ? 0LL : page) * a.Hkv + h) << a.page_shift) + (slot & page_mask);
            auto value = [&](const void *pages, int d) {
                if constexpr (E4M3)
                    return __uint_as_float(e4m3_to_bf16<false>(static_cast<const uint8_t *>(pages)[row * D + d]) << 16);
                else
                    return bf16_to_f32(static_cast<const uint16_t *>(pages)[row * D + d]);
            };
            float score = 0.0f;
#pragma unroll
            for (int c = 0; c < kSteps; ++c)
#pragma unroll
                for (int e = 0; e < 8; ++e) score += static_cast<float>(q[c][e]) * value(a.k_pages, 16 * c + 8 * half + e);
            score = pair_sum(score);
            if constexpr (E4M3) score *= a.k_scale[row] * a.c;
            if (slot >= sees) continue;
            const float weight = fast_exp2((score - m) * a.unit), scale = E4M3 ? a.v_scale[row] : 1.0f;
#pragma unroll
            for (int d = 0; d < kVals; ++d)
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float v = value(a.v_pages, d * 32 + 8 * (x / 4) + 4 * half + x % 4) * scale;
                    if (!isfinite(v)) o[d][x] += weight * v;
                }
        }
    }

    // the first slot of a bad page that the workgroup met
#pragma unroll
    for (int x = 32; x > 0; x >>= 1) first_bad = min(first_bad, __shfl_xor(first_bad, x, kWave));
    const bool alone = active == 1;
    const long long unit = (static_cast<long long>(u) * a.Hkv + h) * a.S + split;
    if (threadIdx.x == 0) {
        if (alone) {
            if (un.last && h == 0 && a.status) a.status[un.b] = first_bad != 0x7fffffff;
        } else {
            a.part_bad[unit] = first_bad;
        }
    }
    const float L = pair_sum(l);
    if (alone) {
        const bool none = first_bad < sees;
        const float f = none ? 0.0f : 1.0f / L;
        const long long to = static_cast<long long>(token) * a.H + head;
        if (live && a.lse && half == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(m, L, a.unit);
        // turned in LDS (the wave's own 32 rows of the first stages, chunk c of row r at
        // c ^ r), so that rows leave whole (16 prompts, 143 MB of them: 335 us, and 343 as
        // pieces of 16 bytes of 32 rows)
        constexpr int kChunks = kRowB / 16, kPer = kWave / kChunks;  // of a row; rows a store covers
        char *room = &kv[0][0][0] + w * 32 * kRowB;
#pragma unroll
        for (int d = 0; d < kVals; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = none ? 0.0f : o[d][4 * x + e] * f;
                *reinterpret_cast<u32x2 *>(room + col * kRowB + ((4 * d + x) ^ (col & (kChunks - 1))) * 16 + 8 * half) =
                    u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
            }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        const int place = lane % kChunks;
#pragma unroll
        for (int i = 0; i < 32 / kPer; ++i) {
            const int row = i * kPer + lane / kChunks;  // whose lanes know where it goes
            const long long dst = __shfl(to, row, kWave);
            const u32x4 v = *reinterpret_cast<const u32x4 *>(room + row * kRowB + place * 16);
            if (w * 32 + row < rows)
                *reinterpret_cast<u32x4 *>(a.out + dst * D + (place ^ (row & (kChunks - 1))) * 8) = v;
        }
    } else if (live) {
        const long long row = unit * kRows + r;
        if (half == 0) {
            a.part_ml[row * 2] = m;
            a.part_ml[row * 2 + 1] = L;
        }
        float *dst = a.part_o + row * D + 4 * half;
#pragma unroll
        for (int d = 0; d < kVals; ++d)
#pragma unroll
            for (int x = 0; x < 4; ++x)
                *reinterpret_cast<f32x4 *>(dst + d * 32 + 8 * x) = f32x4{o[d][4 * x], o[d][4 * x + 1], o[d][4 * x + 2], o[d][4 * x + 3]};
    }
}

// Joins the splits of the row tiles that have several: D / 4 lanes a row.
template <int D>
__global__ __launch_bounds__(kBlock) void k_packed_join(PackedArgs a, int rows_per) {
    constexpr int kLanes = D / 4, kPer = kBlock / kLanes;
    const int lane = threadIdx.x & (kWave - 1);
    const int pieces = rows_per / kPer;
    const int piece = blockIdx.x % pieces, rest = blockIdx.x / pieces;
    const int h = rest % a.Hkv, u = rest / a.Hkv;
    const Unit un = find_unit(a, u, rows_per, lane);
    if (un.b < 0) return;
    const int base = un.base;
    const long long r0 = static_cast<long long>(un.tile) * rows_per;
    const int rows = static_cast<int>(min(static_cast<long long>(un.count) * a.G - r0, static_cast<long long>(rows_per)));
    const long long exist = static_cast<long long>(a.P) << a.page_shift;
    const long long want = static_cast<long long>(base) + (r0 + rows - 1) / a.G + 1;
    const int total = base >= 0 ? static_cast<int>(min(want, exist)) : 0;
    const int active = splits_of((total + kSlots - 1) / kSlots, a.S);
    if (active == 1) return;
    const long long unit = (static_cast<long long>(u) * a.Hkv + h) * a.S;
    int first_bad = 0x7fffffff;
    for (int s = 0; s < active; ++s) first_bad = min(first_bad, a.part_bad[unit + s]);
    if (un.last && h == 0 && piece == 0 && threadIdx.x == 0 && a.status) a.status[un.b] = first_bad != 0x7fffffff;
    const int r = piece * kPer + static_cast<int>(threadIdx.x) / kLanes, d = static_cast<int>(threadIdx.x) % kLanes * 4;
    if (r >= rows) return;
    const int j = static_cast<int>((r0 + r) / a.G), g = static_cast<int>(r0 + r - static_cast<long long>(j) * a.G);
    float m = kNoRef;
    for (int s = 0; s < active; ++s) m = fmaxf(m, a.part_ml[((unit + s) * rows_per + r) * 2]);
    float L = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (int s = 0; s < active; ++s) {
        const long long row = (unit + s) * rows_per + r;
        const float ms = a.part_ml[row * 2], ls = a.part_ml[row * 2 + 1];
        const float f = ms == kNoRef ? 0.0f : fast_exp2((ms - m) * a.unit);
        L += ls * f;
        o += *reinterpret_cast<const f32x4 *>(a.part_o + row * D + d) * f;
    }
    const bool none = first_bad < static_cast<long long>(base) + j + 1;
    const long long to = static_cast<long long>(un.first + j) * a.H + h * a.G + g;
    if (a.lse && d == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(m, L, a.unit);
    const float f = none ? 0.0f : 1.0f / L;
    if (none) o = f32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x2 *>(a.out + to * D + d) = u32x2{pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f)};
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int D, bool E4M3>
hipError_t launch_waves(const PackedArgs &a, const PackedPlan &p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(packed_groups(a.Hkv, p)));
    if constexpr (D == 128 && E4M3)
        if (p.rows == 256) return launch_kernel(k_attend_packed<D, E4M3, 8>, grid, dim3(8 * kWave), 0, s, a);
    return launch_kernel(k_attend_packed<D, E4M3, 4>, grid, dim3(4 * kWave), 0, s, a);
}
template <int D>
hipError_t launch_d(const PackedArgs &a, bool e4m3, const PackedPlan &p, hipStream_t s) {
    return e4m3 ? launch_waves<D, true>(a, p, s) : launch_waves<D, false>(a, p, s);
}

constexpr long long kCus = 256;

// Row tiles of `rows` rows and the parts of their slots, with an estimate of a launch.
struct Parts {
    long long units, groups, S;
    double us;
};

// The parts with the least estimate of a row tile that sees the whole table, us: a tile of
// slots takes `alone` while every workgroup has a compute unit to itself, `shared` where two
// have one (with heads of 256 they follow one another; eight waves have one alone), the
// join a launch and its traffic.  1000 tokens over 8 heads of 128: 30 us in one part, 39 in
// two; 100 over 8000 42 in eight, 46 in sixteen; 256 over 16000 122 in three, 105 in seven;
// 200 over 8000 with heads of 256 66 in nine, 85 in eighteen.  The lengths are the device's,
// so a table wider than its requests is planned for as if they filled it: 500 tokens take
// 18 us in a table of 512 slots, and in one of 8192 19 and a join of 4 that has nothing to do.
Parts parts_of(long long all, int B, int Hkv, int D, long long tiles, int rows, bool e4m3) {
    constexpr double kJoin = 5.0, kJoinBytes = 3e6, kEightMore = 3.0;
    const bool eight = rows == 256;
    const double size = D == 64 ? 0.75 : (D == 128 ? 1.0 : 2.5);
    const double alone = size * (eight ? 2.3 : (e4m3 ? 1.95 : 1.25));
    const double shared = D == 256 ? 2 * alone : size * (e4m3 ? 2.7 : 2.2);
    Parts p = {};
    // every request may end in a part of a tile (of one row at least); none has more tiles
    // than rows
    p.units = std::max(1LL, std::min((all + B * (rows - 1LL)) / rows, all));
    p.groups = p.units * Hkv;
    const double bytes = static_cast<double>(p.groups) * rows * (D + 2) * 4;
    const long long most = std::min(kCus * (eight ? 1 : 2) / p.groups, tiles / kLeastRun);
    for (long long n = 1; n <= std::max(1LL, most) && (n == 1 || bytes * n <= 512 << 20); ++n) {
        const double us = static_cast<double>((tiles + n - 1) / n) * (p.groups * n <= kCus ? alone : shared) +
                          (n > 1 ? kJoin + bytes * n / kJoinBytes : 0.0) + (eight ? kEightMore : 0.0);
        if (n > 1 && us >= p.us) continue;
        p.us = us;
        p.S = n;
    }
    return p;
}

}  // namespace

long long packed_groups(int Hkv, const PackedPlan &p) { return static_cast<long long>(p.units) * Hkv * p.S; }

long long packed_join_groups(int Hkv, int D, const PackedPlan &p) {
    return p.S == 1 ? 0 : static_cast<long long>(p.units) * Hkv * (p.rows / (kBlock / (D / 4)));
}

PackedPlan packed_plan(int T, int B, int H, int Hkv, int D, int P, int page_size, bool e4m3) {
    const long long all = static_cast<long long>(T) * (H / Hkv);
    const long long tiles = (static_cast<long long>(P) * page_size + kSlots - 1) / kSlots;
    PackedPlan p = {};
    p.rows = 128;
    Parts use = parts_of(all, B, Hkv, D, tiles, 128, e4m3);
    // An e4m3 cache's rows are widened by each workgroup, so with heads of 128 eight waves
    // share them where there are row tiles for many rounds, or parts that fill the card
    // (8191 tokens: 605 us, 628 with four; 512 over 16000 188 and 197; but 2000 tokens 73 and
    // 64, as a tile's slots are all one workgroup's.  Heads of 64 leave eight waves less
    // than a load each, 256 one wave a SIMD).
    if (e4m3 && D == 128) {
        const Parts eight = parts_of(all, B, Hkv, D, tiles, 256, e4m3);
        if (use.groups >= 4 * kCus || (eight.S > 1 && eight.us < use.us)) {
            p.rows = 256;
            use = eight;
        }
    }
    p.units = static_cast<int>(use.units);
    p.S = static_cast<int>(use.S);
    if (p.S > 1) {
        const size_t parts = static_cast<size_t>(use.groups) * p.S;
        size_t o = 0;
        p.part_o = o;
        o = align_up(o + parts * p.rows * D * 4);
        p.part_ml = o;
        o = align_up(o + parts * p.rows * 2 * 4);
        p.part_bad = o;
        o = align_up(o + parts * 4);
        p.total = o;
    }
    return p;
}

hipError_t launch_attend_packed(const PackedArgs &a, int D, bool e4m3, const PackedPlan &p, hipStream_t s) {
    if (D == 64) return launch_d<64>(a, e4m3, p, s);
    if (D == 128) return launch_d<128>(a, e4m3, p, s);
    return launch_d<256>(a, e4m3, p, s);
}

hipError_t launch_attend_packed_join(const PackedArgs &a, int D, const PackedPlan &p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(packed_join_groups(a.Hkv, D, p)));
    if (D == 64) return launch_kernel(k_packed_join<64>, grid, dim3(kBlock), 0, s, a, p.rows);
    if (D == 128) return launch_kernel(k_packed_join<128>, grid, dim3(kBlock), 0, s, a, p.rows);
    return launch_kernel(k_packed_join<256>, grid, dim3(kBlock), 0, s, a, p.rows);
}

}  // namespace sv
