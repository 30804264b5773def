// sv_attend.hip -- attention of a short window of new tokens (one token, a
// draft chain, a draft tree) over a paged cache.
//
// For every window row (token n, head) with query q, over the request's cached
// slots s < base and the window's own tokens the row may see:
//   w_s = scale q . k_s,  m = max w,  l = sum exp(w_s - m),
//   out = sum exp(w_s - m) v_s / l,  lse = m + log l.
//
// The query heads that share a KV head and all the window's tokens form the
// rows of one product: rows r = n * G + g, 16 to a tile.  A wave walks 32
// slots at a time:
//   S^T = K Q^T   (16x16x32 MFMAs; K is the left operand: its rows are 16
//                  slots, loaded 16 bytes per lane straight from the page)
//   online softmax; lane l holds 8 slots of row l % 16, so the running reference
//                  needs two cross-lane swaps where it moves and the sum none
//                  until the end;
//   O^T += V^T P^T: lane l's 8 weights are exactly the k-slice that MFMA's
//                  right operand wants from it (the contraction runs over the
//                  slots in the order (half, lane group, register)), so the
//                  weights go from the softmax to the product without leaving
//                  the lane.  The left operand V^T wants 8 slots of one value:
//                  lane l loads 16 bytes (8 values) of each of its 8 slots and
//                  transposes the 8 x 8 block in registers (v_perm), which
//                  serves 8 MFMAs, MFMA i holding values d = 8 m + i.
// The weights enter the second product as two bf16 terms, the rounded weight and
// the rounded rest (2^-16 relative): up to two row tiles per wave the products
// that this adds are hidden behind the cache's bytes.  With three (33 to 48 rows per
// KV head where the slots are divided, nine to twelve row tiles of a workgroup where
// the rows are), where they are not and the registers are full, it takes the first
// term alone: at most 2^-8 relative for each weight, independent, averaged over the
// slots.  l sums the weights unrounded, and every accumulator,
// reference and sum is fp32.  An e4m3 cache is widened to bf16 in
// registers (exact); its per-row scales multiply the scores and the weights.
//
// Work split.  Few rows (kCached, kStream): the slots of a (request, KV head) go
// to `active` of S workgroups, each of whose 4 waves takes a run of tiles with
// the next tile's rows in flight, and joins them through LDS.  Many rows
// (kShared): the waves of a workgroup hold different rows and walk the same
// tiles, which come through a ring of four stages in LDS, loaded three ahead
// straight from the pages.  Either way a workgroup writes the result (one active
// split) or a partial (reference, l, O) that k_attend_join joins.  S comes from
// the table's size on the host, the runs from the request's own length on the
// device, so a captured graph replays with other lengths.
//
// Bounds and figures (MI355X, 32 query and 8 KV heads of 128): one token, 64
// requests of 8192: 353 us, 6.1 TB/s of cache, bound by memory; lengths up to 8192:
// 166 us, 5.6 TB/s, the rest the tail of the longest; e4m3: 208 and 103 us, 5.3 and
// 4.7 TB/s, half the bytes in flight per wave; 64 trees of 33 over up to 2048: 97 us,
// all over 2048 130 us (541 TFLOP/s), in e4m3 118 and 141, bound by a tile's chain of
// LDS reads, products and exponentials with two waves per SIMD (registers).  Heads
// of 256 never share: 64 trees of 33, 8 query heads to one KV head, take 131 + 12 us
// where the same bytes as 16 to 2 heads of 128 take 88 + 10.
//
// Masked slots: scores are replaced, never added to; value rows behind the
// last token are zeroed; and a non-finite value of a window token is left to
// the rows that see the token (0 * inf would reach the others).
#include <algorithm>

#include "sv_paged.hpp"
#include "sv_paged_internal.hpp"

namespace sv {
namespace {

#define SV_LDS __attribute__((address_space(3)))
#define SV_GLOBAL __attribute__((address_space(1)))

constexpr int kTile = 32;          // slots a wave takes per step
constexpr float kSlack = 8.0f;     // weights may reach 2^kSlack before the reference moves

// A row's weights are 2^(s c) relative to 2^(m c), m its reference (a score q.k).
// Where |m c| < kNear the exponent is one fma, s c - shift with shift = fp32(m c),
// whose rounding (up to 2^-5) all of the row's weights and their sum share.  It grows
// with |m c|, and from 2^31 on would overflow or lose every weight; there the exponent
// is (s - m) c, and shift is kFar: the fma of any score that is not masked then lies
// above kSlack, which leads to the step that knows m.  m itself waits in LDS (64 ragged
// trees of 33: 94.9 -> 96.5 us a call; 32 chains in e4m3 44.0 -> 45.3, the others equal;
// a branch of its own for near rows, which need not read m: 99 and 45).
constexpr float kNear = 0x1p20f, kFar = -3e38f;
// The reference of a row that has met no score.
constexpr float kNoRef = -3.4028234663852886e38f;

__device__ __forceinline__ float shift_of(float m, float c) {
#pragma clang fp contract(off)
    const float x = m * c;
    return fabsf(x) < kNear ? x : kFar;
}
// The exponent of score s relative to reference m.
__device__ __forceinline__ float relative(float s, float m, float shift, float c) {
    return shift != kFar ? fmaf(s, c, -shift) : (s - m) * c;
}
// log2 of what turns weights relative to one reference into those of another.
__device__ __forceinline__ float rebase(float m, float shift, float to, float to_shift, float c) {
    if (shift == kFar) return relative(m, to, to_shift, c);
    return to_shift == kFar ? fmaf(-to, c, shift) : shift - to_shift;
}

// Natural log of L 2^(m c).
__device__ __forceinline__ float log_sum(float m, float L, float c) {
    const float shift = shift_of(m, c);
    const double x = shift != kFar ? static_cast<double>(shift) : static_cast<double>(m) * static_cast<double>(c);
    return static_cast<float>((x + static_cast<double>(log2f(L))) * 0.6931471805599453);
}

__device__ __forceinline__ f32x4 mfma16(const bf16x8 &a, const bf16x8 &b, const f32x4 &c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Over the four lanes l, l ^ 16, l ^ 32, l ^ 48 that hold one row.
__device__ __forceinline__ float quad_max(float v) {
    const unsigned u = __float_as_uint(v);
    const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    const float x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const unsigned t = __float_as_uint(x);
    const auto b = __builtin_amdgcn_permlane16_swap(t, t, false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float quad_sum(float v) {
    v += __shfl_xor(v, 32, kWave);
    return v + __shfl_xor(v, 16, kWave);
}

// What every workgroup of a request derives from the request's length alike.
struct Span {
    int base, count, total, tiles, active;
    bool ok;  // the window lies inside the table and its parent array is well formed
};
__device__ __forceinline__ Span request_span(const AttendArgs &a, int b, int lane, uint64_t *anc) {
    Span s;
    s.base = uniform(a.base[b]);
    s.count = uniform(window_rows(a.counts, b, a.N));
    const long long total = static_cast<long long>(s.base) + s.count;
    s.ok = s.base >= 0 && total <= (static_cast<long long>(a.P) << a.page_shift);
    if (a.parents) {
        // ancestor masks by pointer doubling: lane t's mask gains that of the
        // ancestor it has reached, which then moves as far again
        int p = lane < s.count ? a.parents[static_cast<long long>(b) * a.N + lane] : -1;
        const bool bad = lane < s.count && (lane == 0 ? p != -1 : p < 0 || p >= lane);
        if (ballot(bad) != 0) {
            s.ok = false;
            p = -1;
        }
        uint64_t m = 1ull << lane;
        if (anc) {
#pragma unroll
            for (int i = 0; i < 6; ++i) {
                const int from = p < 0 ? lane : p;
                const uint64_t up = __shfl(m, from, kWave);
                const int next = __shfl(p, from, kWave);
                if (p >= 0) {
                    m |= up;
                    p = next;
                }
            }
            *anc = m;
        }
    } else if (anc) {
        *anc = (2ull << lane) - 1;  // token t sees tokens 0..t
    }
    s.total = s.ok ? static_cast<int>(total) : 0;
    s.tiles = (s.total + kTile - 1) / kTile;
    // as many splits as have a least run
    s.active = s.tiles == 0 ? 0 : max(1, min(a.S, s.tiles / (a.min_tiles * kWavesPerBlock)));
    return s;
}

// First tile of split i of a request.  Where the workgroups come in many rounds
// (falling), split i's share falls evenly from 3/2 of the mean for the first to
// 1/2 for the last: workgroups start in the order of i, so the last to start are
// short and the card drains evenly.  In one round the shares are equal.
__device__ __forceinline__ int first_tile(const Span &s, int i, bool falling) {
    const long long n = s.active;
    if (!falling || n < 2) return static_cast<int>(s.tiles * static_cast<long long>(i) / n);
    // share of split k: 3 (n - 1) - 2 k of n times 2 (n - 1)
    return static_cast<int>(s.tiles * (3 * (n - 1) * i - static_cast<long long>(i) * (i - 1)) / (2 * n * (n - 1)));
}

// The 8 bf16 values of 16 bytes, or of 8 e4m3 bytes.
__device__ __forceinline__ bf16x8 as_bf16x8(unsigned a, unsigned b, unsigned c, unsigned d) {
    const u32x4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ bf16x8 widen8(unsigned lo, unsigned hi) {
    return as_bf16x8(e4m3_to_bf16<false>(lo), e4m3_to_bf16<true>(lo), e4m3_to_bf16<false>(hi), e4m3_to_bf16<true>(hi));
}

// Whether a word of cached values holds an infinity or NaN, and the word with
// those cleared.
template <bool E4M3>
__device__ __forceinline__ bool has_nonfinite(unsigned w) {
    if constexpr (E4M3) {  // a byte of 0x7f or 0xff: the low 7 bits + 1 carry into bit 7
        return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
    } else {
        return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
}
template <bool E4M3>
__device__ __forceinline__ unsigned finite_only(unsigned w) {
    if constexpr (E4M3) {
        const unsigned m = (((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) >> 7;
        return w & ~(m * 0xffu);
    } else {
        if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
        if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
        return w;
    }
}

// 16, 8 or 4 bytes of the cache; STREAM: past the caches.
template <bool STREAM, typename T>
__device__ __forceinline__ T load_cached(const void *p) {
    if constexpr (STREAM)
        return __builtin_nontemporal_load(static_cast<const T *>(p));
    else
        return *static_cast<const T *>(p);
}

// The cached rows of one tile as they lie in memory: the lane's slices of K (row
// lane % 16 of each half, for the left operand) and its 8 rows of V.
template <int D, bool E4M3, bool STREAM>
struct Tile {
    static constexpr int kElem = E4M3 ? 1 : 2;
    static constexpr int kRowB = D * kElem;
    static constexpr int kKVecs = D * kElem / 64;      // 16-byte loads of a K row per lane
    static constexpr int kVWords = D * kElem / 64;     // words of a V row per lane (D / 16 values)
    static constexpr int kVStep = kVWords < 4 ? kVWords : 4;
    static constexpr int kWordVals = 4 / kElem;        // values per word
    u32x4 k[2][kKVecs];
    unsigned v[2][4][kVWords];
    f32x4 ks[2], vs[2];  // e4m3: the rows' scales, in the order of the scores

    __device__ __forceinline__ void load_k(const AttendArgs &a, const long long (&row)[2], int col, int kg) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const char *p = static_cast<const char *>(a.k_pages) + (row[f] + col) * (D * kElem) + kg * 16;
#pragma unroll
            for (int c = 0; c < kKVecs; ++c) k[f][c] = load_cached<STREAM, u32x4>(p + c * 64);
            if constexpr (E4M3) ks[f] = *reinterpret_cast<const f32x4 *>(a.k_scale + row[f] + kg * 4);
        }
    }
    __device__ __forceinline__ void load_v(const AttendArgs &a, const long long (&row)[2], int col, int kg) {
#pragma unroll
        for (int f = 0; f < 2; ++f) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const unsigned *p = reinterpret_cast<const unsigned *>(
                    static_cast<const char *>(a.v_pages) + (row[f] + kg * 4 + j) * (D * kElem) + col * (kVWords * 4));
#pragma unroll
                for (int i = 0; i < kVWords; i += kVStep) {
                    if constexpr (kVStep == 4) {
                        const u32x4 x = load_cached<STREAM, u32x4>(p + i);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[f][j][i + e] = x[e];
                    } else if constexpr (kVStep == 2) {
                        const u32x2 x = load_cached<STREAM, u32x2>(p + i);
                        v[f][j][i] = x.x;
                        v[f][j][i + 1] = x.y;
                    } else {
                        v[f][j][i] = load_cached<STREAM, unsigned>(p + i);
                    }
                }
            }
            if constexpr (E4M3) vs[f] = *reinterpret_cast<const f32x4 *>(a.v_scale + row[f] + kg * 4);
        }
    }
    // The same from a stage of the ring (below): K from the four addresses ka, V
    // from va, each with the second half's rows 16 rows further.  Each block waits
    // for its own reads, so nothing is used before it has arrived.
    __device__ __forceinline__ void read_k(const uint32_t (&ka)[kKVecs], uint32_t stage) {
        if constexpr (kKVecs == 4)
            asm volatile(
                "ds_read_b128 %0, %8\n\tds_read_b128 %1, %9\n\tds_read_b128 %2, %10\n\tds_read_b128 %3, %11\n\t"
                "ds_read_b128 %4, %8 offset:%12\n\tds_read_b128 %5, %9 offset:%12\n\t"
                "ds_read_b128 %6, %10 offset:%12\n\tds_read_b128 %7, %11 offset:%12\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(k[0][0]), "=&v"(k[0][1]), "=&v"(k[0][2]), "=&v"(k[0][3]), "=&v"(k[1][0]), "=&v"(k[1][1]),
                  "=&v"(k[1][2]), "=&v"(k[1][3])
                : "v"(ka[0] + stage), "v"(ka[1] + stage), "v"(ka[2] + stage), "v"(ka[3] + stage), "i"(16 * kRowB));
        else if constexpr (kKVecs == 2)
            asm volatile(
                "ds_read_b128 %0, %4\n\tds_read_b128 %1, %5\n\tds_read_b128 %2, %4 offset:%6\n\t"
                "ds_read_b128 %3, %5 offset:%6\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(k[0][0]), "=&v"(k[0][1]), "=&v"(k[1][0]), "=&v"(k[1][1])
                : "v"(ka[0] + stage), "v"(ka[1] + stage), "i"(16 * kRowB));
        else
            asm volatile("ds_read_b128 %0, %2\n\tds_read_b128 %1, %2 offset:%3\n\ts_waitcnt lgkmcnt(0)"
                         : "=&v"(k[0][0]), "=&v"(k[1][0])
                         : "v"(ka[0] + stage), "i"(16 * kRowB));
    }
    __device__ __forceinline__ void read_v(const uint32_t (&va)[4], uint32_t stage) {
#define SV_READ_V(OP, X)                                                                                        \
    asm volatile(OP " %0, %8 offset:%12\n\t" OP " %1, %9 offset:%12\n\t" OP " %2, %10 offset:%12\n\t" OP          \
                    " %3, %11 offset:%12\n\t" OP " %4, %8 offset:%13\n\t" OP " %5, %9 offset:%13\n\t" OP          \
                    " %6, %10 offset:%13\n\t" OP " %7, %11 offset:%13\n\ts_waitcnt lgkmcnt(0)"                   \
                 : "=&v"(X[0]), "=&v"(X[1]), "=&v"(X[2]), "=&v"(X[3]), "=&v"(X[4]), "=&v"(X[5]), "=&v"(X[6]),     \
                   "=&v"(X[7])                                                                                   \
                 : "v"(va[0] + stage), "v"(va[1] + stage), "v"(va[2] + stage), "v"(va[3] + stage),                \
                   "i"(32 * kRowB), "i"(48 * kRowB))
        if constexpr (kVWords == 4) {
            u32x4 x[8];
            SV_READ_V("ds_read_b128", x);
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int i = 0; i < 4; ++i) v[e / 4][e % 4][i] = x[e][i];
        } else if constexpr (kVWords == 2) {
            u32x2 x[8];
            SV_READ_V("ds_read_b64", x);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e / 4][e % 4][0] = x[e].x;
                v[e / 4][e % 4][1] = x[e].y;
            }
        } else {
            unsigned x[8];
            SV_READ_V("ds_read_b32", x);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e / 4][e % 4][0] = x[e];
        }
#undef SV_READ_V
    }
    // e4m3: the scales of the scores' rows, 4 kg .. 4 kg + 3 of each half.
    __device__ __forceinline__ void read_scales(uint32_t at) {
        asm volatile(
            "ds_read_b128 %0, %4\n\tds_read_b128 %1, %4 offset:64\n\tds_read_b128 %2, %4 offset:128\n\t"
            "ds_read_b128 %3, %4 offset:192\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(ks[0]), "=&v"(ks[1]), "=&v"(vs[0]), "=&v"(vs[1])
            : "v"(at));
    }
    // The left operand of the 32 values of step c of the first product.
    __device__ __forceinline__ bf16x8 k_slice(int f, int c) const {
        if constexpr (E4M3)
            return c % 2 ? widen8(k[f][c / 2].z, k[f][c / 2].w) : widen8(k[f][c / 2].x, k[f][c / 2].y);
        else
            return __builtin_bit_cast(bf16x8, k[f][c]);
    }
    // V^T of word i: for each of its values the lane's 8 slots, in the order (half, slot).
    __device__ __forceinline__ void transpose(int i, bf16x8 (&vt)[kWordVals]) const {
        unsigned x[kWordVals][4];  // [value][pair of slots]
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const unsigned even = v[f][2 * j][i], odd = v[f][2 * j + 1][i];
                if constexpr (E4M3) {
                    // bytes of two slots side by side, then widened in pairs
                    const unsigned lo = __builtin_amdgcn_perm(odd, even, 0x05010400u);
                    const unsigned hi = __builtin_amdgcn_perm(odd, even, 0x07030602u);
                    x[0][2 * f + j] = e4m3_to_bf16<false>(lo);
                    x[1][2 * f + j] = e4m3_to_bf16<true>(lo);
                    x[2][2 * f + j] = e4m3_to_bf16<false>(hi);
                    x[3][2 * f + j] = e4m3_to_bf16<true>(hi);
                } else {
                    x[0][2 * f + j] = __builtin_amdgcn_perm(odd, even, 0x05040100u);
                    x[1][2 * f + j] = __builtin_amdgcn_perm(odd, even, 0x07060302u);
                }
            }
#pragma unroll
        for (int e = 0; e < kWordVals; ++e) vt[e] = as_bf16x8(x[e][0], x[e][1], x[e][2], x[e][3]);
    }
};

// How a workgroup's waves divide its work and how the cache reaches them.
enum AttendMode {
    kCached,  // the slots are divided; each wave loads its own into registers
    kStream,  // the same, past the caches
    kShared   // the rows are divided; all waves walk the same slots through LDS
};

// The ring of kShared: kStages stages of one tile each, K's 32 rows, V's, and for
// e4m3 a copy of the tile's 64 scales for each wave, written by global-to-LDS
// loads of 16 bytes per lane (4 for the scales).  Chunk c of row r lies at place
// c ^ swizzle(r) of its row, so that the 16 rows of a K slice, a row length
// apart, lie in different banks.
template <int D, bool E4M3>
struct Ring {
    static constexpr int kRowB = D * (E4M3 ? 1 : 2), kRowChunks = kRowB / 16;
    static constexpr int kStages = 4;
    static constexpr int kPieces = 64 * kRowB / 1024;         // 1 KB loads per tile
    static constexpr int kPerWave = kPieces / kWavesPerBlock;
    static constexpr int kLoads = kPerWave + (E4M3 ? 1 : 0);  // a wave's loads per tile
    static constexpr int kStageB = 64 * kRowB + (E4M3 ? kWavesPerBlock * 256 : 0);
    static __device__ __forceinline__ int swizzle(int r) {
        return (r / (16 / kRowChunks)) & (kRowChunks - 1);
    }
};

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the wave's N youngest
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

template <int D, bool E4M3, int QT, AttendMode MODE>
__global__ __launch_bounds__(kBlock, 2) void k_attend(AttendArgs a) {
    constexpr int kChunks = D / 32;       // 32-value steps of the first product
    constexpr int kVals = D / 16;         // values per lane of V: one MFMA each
    constexpr bool kShares = MODE == kShared;
    constexpr bool kQInLds = !kShares && (QT > 1 || D == 256);
    constexpr int kRowsPerGroup = QT * 16 * (kShares ? kWavesPerBlock : 1);
    // where the registers just suffice, loads and widenings stay where they are
    // written: moved ahead, as the compiler likes to, they spill (64 requests of 33
    // rows, QT = 3: 203 us, and 120 us in place)
    constexpr bool kTight = QT * D > 256 || D == 256 || kShares;
    constexpr bool kTwoTerms = QT < 3;  // weights as two bf16 terms, where the registers allow
    constexpr int kPad = 4;
    // the queries during the walk, the four waves' rows at the end
    __shared__ __align__(1024) union {
        u32x4 q[kQInLds ? QT : 1][kChunks][kWave];
        float o[kShares ? 1 : kWavesPerBlock][16][D + kPad];
        char ring[kShares ? Ring<D, E4M3>::kStages * Ring<D, E4M3>::kStageB : 16];
    } lds;
    // the rows' reference scores; the walk itself needs only their shifts
    __shared__ float refs[QT][kBlock];
    __shared__ float sm[kWavesPerBlock][16], sl[kWavesPerBlock][16];
    __shared__ int sbad;
    const int lane = threadIdx.x & (kWave - 1), w = uniform(static_cast<int>(threadIdx.x >> 6));
    const int col = lane & 15, kg = lane >> 4;

    // workgroups that read the same slots (the row blocks of one split) are
    // 8 apart: consecutive workgroups go to consecutive XCDs, so they share an L2
    const int octet = blockIdx.x / (8 * a.QB), in = blockIdx.x % (8 * a.QB);
    const int qb = in / 8;
    const int rest = octet * 8 + in % 8;
    if (rest >= a.S * a.B * a.Hkv) return;
    const int h = rest % a.Hkv, b = rest / a.Hkv % a.B, split = rest / a.Hkv / a.B;

    uint64_t anc;
    const Span sp = request_span(a, b, lane, &anc);
    const bool speaks = h == 0 && qb == 0 && split == 0 && threadIdx.x == 0 && a.status;
    const int rows = sp.count * a.G, group0 = qb * kRowsPerGroup;
    // this wave's row tiles: every fourth of them where the waves divide the rows.  A
    // wave skips a QT-th tile it lacks: 9 tiles are 3, 2, 2, 2 (105 us for 64 ragged
    // trees of 33, and 109 as 3, 3, 3, 0), 5 are 2, 1, 1, 1 (115 and 124 us)
    auto tile_row = [&](int t) { return group0 + (kShares ? t * kWavesPerBlock + w : t) * 16; };
    const bool last = !kShares || QT == 1 || tile_row(QT - 1) < rows;
    if (!sp.ok || rows == 0) {
        if (split == 0) {  // a malformed request reads as zeros
            for (int i = threadIdx.x; i < kRowsPerGroup * D; i += kBlock) {
                const int r = group0 + i / D;
                if (r >= rows) break;
                const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
                a.out[to * D + i % D] = 0;
                if (a.lse && i % D == 0) a.lse[to] = -__builtin_huge_valf();
            }
            if (speaks) a.status[b] = sp.ok ? 0 : 2 - (a.base[b] < 0 || static_cast<long long>(a.base[b]) + sp.count >
                                                                            (static_cast<long long>(a.P) << a.page_shift));
        }
        return;
    }
    if (split >= sp.active) return;

    // this lane's query rows: the right operand's column `col` of each row tile.
    // One row tile's slices stay in registers; more of them are shared by the
    // workgroup's waves through LDS, [row tile][step][lane]
    uint64_t sees[QT];
    u32x4 qr[kQInLds ? 1 : QT][kChunks];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = tile_row(t) + col;
        const bool live = r < rows;
        const int n = live ? r / a.G : 0, g = live ? r % a.G : 0;
        sees[t] = __shfl(anc, n, kWave);
        const uint16_t *q = a.q + (static_cast<long long>(b) * a.N + n) * a.q_stride + static_cast<long long>(h * a.G + g) * D;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (kQInLds && (t * kChunks + c) % kWavesPerBlock != w) continue;
            // e4m3 rows are read 16 values per lane, which are two steps' slices
            const int d = E4M3 ? (c / 2) * 64 + kg * 16 + (c % 2) * 8 : c * 32 + kg * 8;
            u32x4 x = {0, 0, 0, 0};
            if (live) x = *reinterpret_cast<const u32x4 *>(q + d);
            if constexpr (kQInLds)
                lds.q[t][c][lane] = x;
            else
                qr[t][c] = x;
        }
    }
    if constexpr (kQInLds) __syncthreads();
    auto q_slice = [&](int t, int c) {
        if constexpr (kQInLds)
            return __builtin_bit_cast(bf16x8, lds.q[t][c][lane]);
        else
            return __builtin_bit_cast(bf16x8, qr[t][c]);
    };

    f32x4 o[QT][kVals];
    float shift[QT], l[QT];  // of the reference, and the weights' sum
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        refs[t][threadIdx.x] = kNoRef;
        shift[t] = shift_of(kNoRef, a.c);
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < kVals; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    }

    const int32_t *table = a.page_table + static_cast<long long>(b) * a.P;
    const int page_mask = (1 << a.page_shift) - 1;
    bool bad = false;
    const int c0 = first_tile(sp, split, a.falling), c1 = first_tile(sp, split + 1, a.falling);
    const int run = kShares ? c1 - c0 : (c1 - c0 + kWavesPerBlock - 1) / kWavesPerBlock;
    const int t0 = c0 + (kShares ? 0 : w * run), t1 = min(t0 + run, c1);
    int ids = 0;  // lane i: the page of the i-th 16 slots of 32 tiles
    // rows (in units of rows) of the first slots of a tile's two 16-slot halves;
    // tiles are asked for in order
    auto find_rows = [&](int tile, long long (&row)[2]) {
        const int half0 = ((tile - t0) & 31) * 2;
        if (half0 == 0) {
            const int s = tile * kTile + 16 * lane;
            ids = s < sp.total ? table[s >> a.page_shift] : 0;
            asm volatile("" : "+v"(ids));  // waited for here, once in 32 tiles, not where it is used
            const bool out = ids < 0 || ids >= a.num_pages;
            bad |= out && s < t1 * kTile;
            if (out) ids = 0;
        }
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            // a half behind the last slot reads the first half's rows
            const bool there = tile * kTile + 16 * f < sp.total;
            const int s = tile * kTile + (there ? 16 * f : 0);
            const int page = __builtin_amdgcn_readlane(ids, half0 + (there ? f : 0));
            row[f] = ((static_cast<long long>(page) * a.Hkv + h) << a.page_shift) + (s & page_mask);
        }
    };
    Tile<D, E4M3, MODE == kStream> kv;
    // kCached, kStream: a tile's K is replaced by the next tile's as soon as the
    // scores are formed, its V once it is transposed, so a wave always has loads in
    // flight.  kShared: every wave loads its pieces of the tile kStages - 1 ahead.
    long long next[2];
    using R = Ring<D == 256 ? 128 : D, E4M3>;
    const uint32_t ring = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((SV_LDS char *)lds.ring));
    uint32_t ka[kv.kKVecs], va[4];
    auto issue = [&](int tile) {
        long long next[2];
        find_rows(tile, next);
        // opaque: as elements of `next`, picked by an index, they would pass through memory
        long long row0 = next[0], row1 = next[1];
        asm volatile("" : "+s"(row0), "+s"(row1));
        char *stage = lds.ring + (tile - t0) % R::kStages * R::kStageB;
#pragma unroll
        for (int i = 0; i < R::kPerWave; ++i) {
            const int piece = i * kWavesPerBlock + w, of = piece % (R::kPieces / 2);
            const int r = of * (1024 / R::kRowB) + lane / R::kRowChunks;  // the row this lane loads from
            const char *from = static_cast<const char *>(piece < R::kPieces / 2 ? a.k_pages : a.v_pages) +
                               (of < R::kPieces / 4 ? row0 : row1) * R::kRowB + (r & 15) * R::kRowB +
                               ((lane % R::kRowChunks) ^ R::swizzle(r)) * 16;
            __builtin_amdgcn_global_load_lds((const SV_GLOBAL void *)from, (SV_LDS void *)(stage + piece * 1024), 16, 0, 0);
        }
        if constexpr (E4M3) {
            const float *from = (lane < 32 ? a.k_scale : a.v_scale) + ((lane & 16) ? row1 : row0) + col;
            __builtin_amdgcn_global_load_lds((const SV_GLOBAL void *)from, (SV_LDS void *)(stage + 64 * R::kRowB + w * 256), 4, 0, 0);
        }
    };
    if constexpr (kShares) {
        const int fk = R::swizzle(col);
#pragma unroll
        for (int c = 0; c < kv.kKVecs; ++c) ka[c] = ring + col * R::kRowB + ((4 * c + kg) ^ fk) * 16;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = 4 * kg + j, byte = col * kv.kVWords * 4;
            va[j] = ring + r * R::kRowB + ((byte / 16) ^ R::swizzle(r)) * 16 + byte % 16;
        }
        // the queries have arrived before the ring's loads are counted
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int c = 0; c < kChunks; ++c) asm volatile("" : "+v"(qr[t][c]));
#pragma unroll
        for (int i = 0; i < R::kStages - 1; ++i)
            if (t0 + i < t1) issue(t0 + i);
    } else if (t0 < t1) {
        find_rows(t0, next);
        kv.load_k(a, next, col, kg);
        kv.load_v(a, next, col, kg);
    }
    for (int tile = t0; tile < t1; ++tile) {
        const int s0 = tile * kTile;
        const bool more = tile + 1 < t1;
        uint32_t stage = 0;
        if constexpr (kShares) {
            // this wave's pieces of the tile have arrived, then everybody's; the
            // barrier also says that the stage of the tile before is free
            if (t1 - 1 - tile >= R::kStages - 2)
                wait_loads<R::kLoads *(R::kStages - 2)>();
            else
                wait_loads<0>();
            asm volatile("s_barrier" ::: "memory");
            if (tile + R::kStages - 1 < t1) issue(tile + R::kStages - 1);
            if (tile_row(0) >= rows) continue;  // a wave without rows only loads
            stage = static_cast<uint32_t>((tile - t0) % R::kStages * R::kStageB);
            kv.read_k(ka, stage);
            if constexpr (E4M3) kv.read_scales(ring + stage + 64 * R::kRowB + w * 256 + kg * 16);
        } else if (more) {
            find_rows(tile + 1, next);
        }

        // kShared: while a wave has products to issue it goes before its SIMD's other
        // wave, whose exponentials fill the gaps (64 ragged trees of 33: 101 us against
        // 105, in e4m3 at equal lengths 153 and 157)
        if constexpr (kShares) __builtin_amdgcn_s_setprio(1);
        // scores: slot s0 + 16 f + 4 kg + j of row col
        f32x4 sc[QT][2];
#pragma unroll
        for (int t = 0; t < QT; ++t) sc[t][0] = sc[t][1] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);  // no slice read long before its use
            const bf16x8 k0 = kv.k_slice(0, c), k1 = kv.k_slice(1, c);
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                if (kShares && t == QT - 1 && !last) continue;
                const bf16x8 q = q_slice(t, c);
                sc[t][0] = mfma16(k0, q, sc[t][0]);
                sc[t][1] = mfma16(k1, q, sc[t][1]);
            }
        }
        if constexpr (E4M3) {
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                sc[t][0] *= kv.ks[0];
                sc[t][1] *= kv.ks[1];
            }
        }
        if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);
        if constexpr (kShares)
            kv.read_v(va, stage);
        else if (more)
            kv.load_k(a, next, col, kg);
        if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);
        const bool edge = s0 + kTile > sp.base;  // slots of the window, or behind it
        bool odd = false;                        // a window token has a non-finite value
        if (edge) {
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int s = s0 + 16 * f + 4 * kg + j;
                    if (s >= sp.base) {
#pragma unroll
                        for (int i = 0; i < kv.kVWords; ++i) {
                            if (s >= sp.total) kv.v[f][j][i] = 0;
                            odd |= has_nonfinite<E4M3>(kv.v[f][j][i]);
                            kv.v[f][j][i] = finite_only<E4M3>(kv.v[f][j][i]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        if (!(s < sp.base || (s < sp.total && ((sees[t] >> (s - sp.base)) & 1))))
                            sc[t][f][j] = -__builtin_huge_valf();
                }
            odd = ballot(odd) != 0;
        }

        if constexpr (kShares) __builtin_amdgcn_s_setprio(0);
        bf16x8 pf[QT], pl[kTwoTerms ? QT : 1];
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);
            if (kShares && t == QT - 1 && !last) continue;
            // weights relative to the reference, which stays while none exceeds
            // 2^kSlack: a few exponents more cost fp32 sums and bf16 weights nothing
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = fmaf(sc[t][e / 4][e % 4], a.c, -shift[t]);
            const float top = fmaxf(fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3])), fmaxf(fmaxf(p[4], p[5]), fmaxf(p[6], p[7])));
            if (ballot(top > kSlack) != 0) {
                float most = sc[t][0][0];
#pragma unroll
                for (int e = 1; e < 8; ++e) most = fmaxf(most, sc[t][e / 4][e % 4]);
                const float from = refs[t][threadIdx.x], to = fmaxf(from, quad_max(most)), now = shift_of(to, a.c);
                const float f = fast_exp2(rebase(from, shift[t], to, now, a.c));
                l[t] *= f;
#pragma unroll
                for (int i = 0; i < kVals; ++i) o[t][i] *= f;
                refs[t][threadIdx.x] = to;
                shift[t] = now;
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = relative(sc[t][e / 4][e % 4], to, now, a.c);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = fast_exp2(p[e]);
            l[t] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
            if constexpr (E4M3) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = p[e] * kv.vs[e / 4][e % 4];
                    p[e] = edge && sc[t][e / 4][e % 4] == -__builtin_huge_valf() ? 0.0f : x;
                }
            }
            pf[t] = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
            if constexpr (kTwoTerms) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] -= static_cast<float>(pf[t][e]);
                pl[t] = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]), pack_bf16(p[6], p[7]));
            }
        }
        if constexpr (kShares) __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int i = 0; i < kv.kVWords; ++i) {
            if constexpr (kTight) __builtin_amdgcn_sched_barrier(0);
            bf16x8 vt[kv.kWordVals];
            kv.transpose(i, vt);
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                if (kShares && t == QT - 1 && !last) continue;
#pragma unroll
                for (int e = 0; e < kv.kWordVals; ++e) {
                    f32x4 &x = o[t][i * kv.kWordVals + e];
                    x = mfma16(vt[e], pf[t], x);
                    if constexpr (kTwoTerms) x = mfma16(vt[e], pl[t], x);
                }
            }
        }
        if constexpr (kShares) __builtin_amdgcn_s_setprio(0);
        if (!kShares && more) kv.load_v(a, next, col, kg);
        if (odd) {
            // the non-finite values, one by one, for the rows that see their token
            for (int s = max(s0, sp.base); s < min(s0 + kTile, sp.total); ++s) {
                const int e = s - s0;
                const int page = uniform(table[s >> a.page_shift]);
                const long long at = ((((page < 0 || page >= a.num_pages ? 0LL : page) * a.Hkv + h) << a.page_shift) +
                                      (s & page_mask)) * D;
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                    if (kShares && t == QT - 1 && !last) continue;
                    float mine = 0.0f;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x == (e / 16) * 4 + e % 4) mine = static_cast<float>(pf[t][x]);
                    const float weight = __shfl(mine, (e % 16) / 4 * 16 + col, kWave);
                    if (!((sees[t] >> (s - sp.base)) & 1)) continue;
#pragma unroll
                    for (int i = 0; i < kVals; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int d = (kg * 4 + j) * kVals + i;
                            float v;
                            if constexpr (E4M3)
                                v = __uint_as_float(e4m3_to_bf16<false>(static_cast<const uint8_t *>(a.v_pages)[at + d]) << 16);
                            else
                                v = bf16_to_f32(static_cast<const uint16_t *>(a.v_pages)[at + d]);
                            if (!isfinite(v)) o[t][i][j] += weight * v;
                        }
                }
            }
        }
    }

    const long long unit = ((static_cast<long long>(b) * a.Hkv + h) * a.QB + qb) * a.S + split;
    if constexpr (kShares) {
        // every wave has its rows' whole result; each has seen every page
        const int any = ballot(bad) != 0;
#pragma unroll
        for (int t = 0; t < QT; ++t) {
            const int r = tile_row(t) + col;
            const float L = quad_sum(l[t]);
            if (r >= rows) continue;
            if (sp.active == 1) {
                const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
                const bool none = any || L == 0.0f;
                const float f = none ? 0.0f : 1.0f / L;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < kVals; i += 4) {
                        uint2 y = make_uint2(0, 0);
                        if (!none)
                            y = make_uint2(pack_bf16(o[t][i][j] * f, o[t][i + 1][j] * f),
                                           pack_bf16(o[t][i + 2][j] * f, o[t][i + 3][j] * f));
                        *reinterpret_cast<uint2 *>(a.out + to * D + (kg * 4 + j) * kVals + i) = y;
                    }
                if (a.lse && kg == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(refs[t][threadIdx.x], L, a.c);
            } else {
                const long long at = unit * kRowsPerGroup + (t * kWavesPerBlock + w) * 16 + col;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int i = 0; i < kVals; i += 4)
                        *reinterpret_cast<float4 *>(a.part_o + at * D + (kg * 4 + j) * kVals + i) =
                            make_float4(o[t][i][j], o[t][i + 1][j], o[t][i + 2][j], o[t][i + 3][j]);
                if (kg == 0) {
                    a.part_ml[at * 2] = refs[t][threadIdx.x];
                    a.part_ml[at * 2 + 1] = L;
                }
            }
        }
        if (threadIdx.x == 0) {
            if (sp.active > 1) a.part_bad[unit] = any;
            if (speaks && sp.active == 1) a.status[b] = any;
        }
        return;
    }

    // join the four waves' rows through LDS, one row tile at a time
    if (threadIdx.x == 0) sbad = 0;
    __syncthreads();
    if (bad) sbad = 1;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if (t > 0) __syncthreads();
        const float ll = quad_sum(l[t]);
        if (kg == 0) {
            sm[w][col] = refs[t][threadIdx.x];
            sl[w][col] = ll;
        }
        // the lane's values: d = (4 kg + j) kVals + i
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < kVals; i += 4)
                *reinterpret_cast<float4 *>(&lds.o[w][col][(kg * 4 + j) * kVals + i]) =
                    make_float4(o[t][i][j], o[t][i + 1][j], o[t][i + 2][j], o[t][i + 3][j]);
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * (D / 4); i += kBlock) {
            const int rr = i / (D / 4), d = i % (D / 4) * 4;
            const int r = tile_row(t) + rr;
            if (r >= rows) break;
            float M = sm[0][rr];
#pragma unroll
            for (int v = 1; v < kWavesPerBlock; ++v) M = fmaxf(M, sm[v][rr]);
            const float shift_M = shift_of(M, a.c);
            float L = 0.0f;
            float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < kWavesPerBlock; ++v) {
                const float m = sm[v][rr], f = fast_exp2(rebase(m, shift_of(m, a.c), M, shift_M, a.c));
                L += sl[v][rr] * f;
                const float4 y = *reinterpret_cast<const float4 *>(&lds.o[v][rr][d]);
                x.x += y.x * f;
                x.y += y.y * f;
                x.z += y.z * f;
                x.w += y.w * f;
            }
            if (sp.active == 1) {
                const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
                const bool none = sbad || L == 0.0f;
                const float f = none ? 0.0f : 1.0f / L;
                uint2 y = make_uint2(0, 0);
                if (!none) y = make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
                *reinterpret_cast<uint2 *>(a.out + to * D + d) = y;
                if (a.lse && d == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(M, L, a.c);
            } else {
                const long long at = unit * kRowsPerGroup + t * 16 + rr;
                *reinterpret_cast<float4 *>(a.part_o + at * D + d) = x;
                if (d == 0) {
                    a.part_ml[at * 2] = M;
                    a.part_ml[at * 2 + 1] = L;
                }
            }
        }
    }
    if (threadIdx.x == 0) {
        if (sp.active > 1) a.part_bad[unit] = sbad;
        if (speaks && sp.active == 1) a.status[b] = sbad;
    }
}

// The active splits' partials of a row joined by JW waves, each taking every JW-th.
template <int D, int JW>
__global__ __launch_bounds__(kBlock) void k_attend_join(AttendArgs a, int group_rows) {
    constexpr int kPer = D / kWave;
    constexpr int kAhead = 4;  // partials a wave loads before it uses one
    __shared__ float so[JW][D], sl[JW];
    const int lane = threadIdx.x & (kWave - 1), w = uniform(static_cast<int>(threadIdx.x >> 6));
    const int all = a.N * a.G, wj = w % JW;
    const long long unit_row = static_cast<long long>(blockIdx.x) * (kWavesPerBlock / JW) + w / JW;
    if (unit_row >= static_cast<long long>(a.B) * a.Hkv * all) return;  // JW > 1: a workgroup has one row
    const int r = static_cast<int>(unit_row % all);
    const int h = static_cast<int>(unit_row / all % a.Hkv), b = static_cast<int>(unit_row / all / a.Hkv);
    const Span sp = request_span(a, b, lane, nullptr);
    if (!sp.ok || sp.active <= 1 || r >= sp.count * a.G) return;
    const int qb = r / group_rows;
    const long long unit = ((static_cast<long long>(b) * a.Hkv + h) * a.QB + qb) * a.S;
    const float *ml = a.part_ml + (unit * group_rows + r % group_rows) * 2;
    const float *po = a.part_o + (unit * group_rows + r % group_rows) * D + lane * kPer;
    const float ninf = -__builtin_huge_valf();
    bool bad = false;
    float M = kNoRef;
    for (int s = lane; s < sp.active; s += kWave) {
        bad |= a.part_bad[unit + s] != 0;
        M = fmaxf(M, ml[static_cast<long long>(s) * group_rows * 2]);
    }
    bad = ballot(bad) != 0;
    M = wave_max(M);
    const float shift_M = shift_of(M, a.c);
    float L = 0.0f, x[kPer] = {};
    for (int s0 = wj; s0 < sp.active; s0 += kAhead * JW) {
        float y[kAhead][kPer], ms[kAhead], ls[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const long long at = static_cast<long long>(min(s0 + i * JW, sp.active - 1)) * group_rows;
            ms[i] = ml[at * 2];
            ls[i] = ml[at * 2 + 1];
#pragma unroll
            for (int e = 0; e < kPer; ++e) y[i][e] = po[at * D + e];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            if (s0 + i * JW >= sp.active) continue;
            const float f = fast_exp2(rebase(ms[i], shift_of(ms[i], a.c), M, shift_M, a.c));
            L += ls[i] * f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] += y[i][e] * f;
        }
    }
    if constexpr (JW > 1) {
#pragma unroll
        for (int e = 0; e < kPer; ++e) so[w][lane * kPer + e] = x[e];
        if (lane == 0) sl[w] = L;
        __syncthreads();
        if (w != 0) return;
        L = (sl[0] + sl[1]) + (sl[2] + sl[3]);
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
            const int d = lane * kPer + e;
            x[e] = (so[0][d] + so[1][d]) + (so[2][d] + so[3][d]);
        }
    }
    const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
    const bool none = bad || L == 0.0f;
    const float f = none ? 0.0f : 1.0f / L;
    uint16_t *out = a.out + to * D + lane * kPer;
    if constexpr (kPer == 1) {
        *out = none ? 0 : static_cast<uint16_t>(pack_bf16(x[0] * f, 0.0f) & 0xffffu);
    } else {
#pragma unroll
        for (int e = 0; e < kPer; e += 2)
            *reinterpret_cast<unsigned *>(out + e) = none ? 0 : pack_bf16(x[e] * f, x[e + 1] * f);
    }
    if (lane == 0) {
        if (a.lse) a.lse[to] = none ? ninf : log_sum(M, L, a.c);
        if (a.status && h == 0 && r == 0) a.status[b] = bad ? 1 : 0;
    }
}

template <int D, bool E4M3, int QT>
hipError_t launch_shape(const AttendArgs &a, bool shares, dim3 grid, hipStream_t s) {
    if constexpr (D <= 128)
        if (shares) return launch_kernel(k_attend<D, E4M3, QT, kShared>, grid, dim3(kBlock), 0, s, a);
    // A cache whose rows one workgroup reads is read past the caches: 346 us
    // against 375 for 64 requests of one token over 8k (bf16; e4m3 210 and 210, and
    // plain loads are kept there).
    if constexpr (!E4M3)
        if (a.QB == 1) return launch_kernel(k_attend<D, E4M3, QT, kStream>, grid, dim3(kBlock), 0, s, a);
    if constexpr (E4M3 || D == 256) return launch_kernel(k_attend<D, E4M3, QT, kCached>, grid, dim3(kBlock), 0, s, a);
    return hipErrorInvalidValue;  // D <= 128 has one row block, or shares
}

template <int D, bool E4M3>
hipError_t launch_qt(const AttendArgs &a, int QT, bool shares, dim3 grid, hipStream_t s) {
    if constexpr (D <= 128) {
        if (QT == 2) return launch_shape<D, E4M3, 2>(a, shares, grid, s);
        if (QT == 3) return launch_shape<D, E4M3, 3>(a, shares, grid, s);
    }
    return launch_shape<D, E4M3, 1>(a, shares, grid, s);
}

}  // namespace

// The rows.  Up to three row tiles (D = 256: one) a wave holds them all, and the
// slots are divided.  With more, the workgroup's waves divide the rows and walk
// the same slots, up to 12 row tiles per workgroup: 64 trees of 33 (9 row tiles,
// lengths up to 2048) took 114 us as three row blocks that each read the cache,
// 104 us sharing it; 64 chains of 16 (4 row tiles) over 2k 121 and 109 us.
//
// The slots.  A wave that holds all rows runs over at most kRun tiles per row
// tile (1024 slots per workgroup and row tile: its 2.4 us of preparation are then
// 6% of its time, and a partial is a small part of what it read), and over fewer
// where that leaves the card without kTargetGroups workgroups (two per compute
// unit, what the registers of two row tiles admit: 1024 took one chain of 5 over
// 128k 97 + 10 us where 512 take 90 + 6, and 64 chains of 8 over 2k 103 + 13 where
// one split takes 91), but not below a least run.  Waves that share the slots make
// partials as large as what the workgroup reads in 500 slots, so they are split
// only past kSharedRun tiles or for want of workgroups: splits of 1024 slots took
// the trees 99 + 24 us where none took 104.
//
// Two or three row tiles of several requests that have to be split anyway get
// kFineRun, and shares that fall (first_tile) from two rounds of the card on, since
// a batch's lengths seldom agree: 32 chains of 8 over lengths up to 4096 took 54 us
// so and 70 otherwise (e4m3 36 and 43), where all are 4096 long 102 and 93.  With
// kTargetGroups pairs or more the join takes back what it gains (64 chains of 8
// over lengths up to 2048: 57 + 9 against 69, all 2048 long 99 + 11 against 91).
//
// The splits are counted from the table's width, and a request is cut into as many of
// them as have a least run.  A table much wider than its requests therefore cuts them
// finer than the runs above (tables of 131072 slots: one token of 64 requests up to
// 8192 245 us against 169, 32 e4m3 chains 59 against 36, 64 trees 97 + 19 against 97)
// and takes workspace for splits that stay unused, in all at most kMaxPartials: 256
// trees of 64 over tables of 2^20 slots would ask for 618 GB.
AttendPlan attend_plan(int B, int N, int H, int Hkv, int D, int P, int page_size) {
    constexpr int kTargetGroups = 512, kRun = 8, kFineRun = 6, kSharedRun = 96;
    constexpr long long kMaxPartials = 512LL << 20;
    AttendPlan p;
    const int rows = N * (H / Hkv), tiles = (rows + 15) / 16;
    p.shares = D <= 128 && tiles > 3;
    const int most = D == 256 ? 1 : (p.shares ? 12 : 3);  // row tiles per workgroup
    p.QB = (tiles + most - 1) / most;
    const int each = (tiles + p.QB - 1) / p.QB;
    p.QT = p.shares ? (each + kWavesPerBlock - 1) / kWavesPerBlock : each;
    p.group_rows = p.QT * 16 * (p.shares ? kWavesPerBlock : 1);
    p.min_tiles = p.shares ? 8 : (p.QT == 1 ? 2 : 4);
    const long long slots = static_cast<long long>(P) * page_size;
    const long long all = (slots + kTile - 1) / kTile, groups = static_cast<long long>(B) * Hkv * p.QB;
    const long long cap = (all + kWavesPerBlock * p.min_tiles - 1) / (kWavesPerBlock * p.min_tiles);
    const bool fine = B > 1 && p.QT > 1 && !p.shares && groups < kTargetGroups;
    const long long run = p.shares ? kSharedRun : kWavesPerBlock * (fine ? kFineRun : kRun) * p.QT;
    long long want = std::max((kTargetGroups + groups - 1) / groups, (all + run - 1) / run);
    if (groups * want < 4 * kTargetGroups)  // whole rounds of the card: a part of one takes as long
        want = std::max(want, (groups * want + kTargetGroups - 1) / kTargetGroups * kTargetGroups / groups);
    const long long split_bytes = groups * p.group_rows * (D + 2) * 4;  // partials of one split of everything
    p.S = static_cast<int>(std::max(1LL, std::min({want, cap, 1024LL, kMaxPartials / split_bytes})));
    p.falling = groups * p.S >= (fine ? 2 : 4) * kTargetGroups;
    const size_t units = static_cast<size_t>(groups) * p.S, n = units * p.group_rows;
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    p.part_o = 0;
    p.part_ml = up(p.S > 1 ? n * D * sizeof(float) : 0);
    p.part_bad = p.part_ml + up(p.S > 1 ? n * 2 * sizeof(float) : 0);
    p.total = p.part_bad + up(p.S > 1 ? units * sizeof(int32_t) : 0);
    return p;
}

long long attend_groups(int B, int Hkv, const AttendPlan &p) {
    return (static_cast<long long>(p.S) * B * Hkv + 7) / 8 * 8 * p.QB;
}

hipError_t launch_attend(const AttendArgs &a, int D, bool e4m3, const AttendPlan &p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(attend_groups(a.B, a.Hkv, p)));
    const int QT = p.QT;
    const bool sh = p.shares;
    if (D == 64) return e4m3 ? launch_qt<64, true>(a, QT, sh, grid, s) : launch_qt<64, false>(a, QT, sh, grid, s);
    if (D == 128) return e4m3 ? launch_qt<128, true>(a, QT, sh, grid, s) : launch_qt<128, false>(a, QT, sh, grid, s);
    return e4m3 ? launch_qt<256, true>(a, QT, sh, grid, s) : launch_qt<256, false>(a, QT, sh, grid, s);
}

namespace {
template <int D>
hipError_t launch_join(const AttendArgs &a, int group_rows, hipStream_t s) {
    const long long rows = static_cast<long long>(a.B) * a.Hkv * a.N * a.G;
    // few rows, of many splits each as a rule: four waves a row (160 rows of 128
    // splits 9 us against 17); many: a wave a row (8192 rows of 2 splits 7 against 19)
    if (rows <= 2048)
        return launch_kernel(k_attend_join<D, 4>, dim3(static_cast<unsigned>(rows)), dim3(kBlock), 0, s, a, group_rows);
    return launch_kernel(k_attend_join<D, 1>, dim3(static_cast<unsigned>((rows + kWavesPerBlock - 1) / kWavesPerBlock)),
                         dim3(kBlock), 0, s, a, group_rows);
}
}  // namespace

hipError_t launch_attend_join(const AttendArgs &a, int D, const AttendPlan &p, hipStream_t s) {
    if (D == 64) return launch_join<64>(a, p.group_rows, s);
    if (D == 128) return launch_join<128>(a, p.group_rows, s);
    return launch_join<256>(a, p.group_rows, s);
}

}  // namespace sv
