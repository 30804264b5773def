// sv_attend_packed.hip -- causal attention of packed sequences (whole prompts, or
// their next chunks) over a paged cache that holds them.
//
// Row j of request b (token starts[b] + j) sees the slots s < base[b] + j + 1:
//   w_s = scale q . k_s,  out = sum exp(w_s - m) v_s / l,  lse = m + log l.
//
// The G query heads that share a KV head and a request's tokens form the rows of one
// product, r = j G + g; a workgroup of four waves takes 128 QT of them, a wave
// 32 QT, and all walk the same tiles of 64 slots:
//   S^T = K Q^T   (32x32x16 MFMAs; lane l holds 16 of a tile's 32 slots of row
//                  l % 32, the other 16 are lane l ^ 32's)
//   online softmax: a maximum needs one cross-lane swap, the sum none until the end
//   O^T += V^T P^T: a lane's weights of 16 slots are, in the order (4 slots, lane
//                  half), the 8 that MFMA's right operand wants from it; the left
//                  operand V^T comes from rows of V through transposing LDS reads.
// A tile's rows are loaded into registers while the tile before is worked on, then
// written to one of two LDS stages (an e4m3 cache is widened to bf16 there, exactly;
// its scales multiply scores and weights).  16-byte chunks of a row are permuted so
// that the reads of several rows meet distinct banks.
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

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kSlots = 64;         // slots of a tile
constexpr float kSlack = 8.0f;     // weights may reach 2^kSlack before the reference moves
// Where a row's reference m (a score q.k) has |m c| < kNear, exponents are one fma
// against its rounded product; beyond, differences of scores.
constexpr float kNear = 0x1p20f, kFar = -3e38f;
constexpr float kNoRef = -3.4028234663852886e38f;  // the reference of a row that has met no score

__device__ __forceinline__ float shift_of(float m, float c) {
#pragma clang fp contract(off)
    const float x = m * c;
    return fabsf(x) < kNear ? x : kFar;
}
__device__ __forceinline__ float relative(float s, float m, float shift, float c) {
    return shift != kFar ? fmaf(s, c, -shift) : (s - m) * c;
}
// log2 of what turns weights relative to one reference into those of another.
__device__ __forceinline__ float rebase(float m, float shift, float to, float to_shift, float c) {
    if (shift == kFar) return relative(m, to, to_shift, c);
    return to_shift == kFar ? fmaf(-to, c, shift) : shift - to_shift;
}
__device__ __forceinline__ float log_sum(float m, float L, float c) {
    const float shift = shift_of(m, c);
    const double x = shift != kFar ? static_cast<double>(shift) : static_cast<double>(m) * static_cast<double>(c);
    return static_cast<float>((x + static_cast<double>(log2f(L))) * 0.6931471805599453);
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

// The row tile a workgroup takes: rows [r0, r0 + rows of a workgroup) of request b.
struct Unit {
    int b, tile, first, count;  // request, its tile, its first token and its tokens
    bool last;                  // the request's last tile
};
// Row tiles of a request of `count` tokens.
__device__ __forceinline__ int tiles_of(int count, int G, int rows) {
    return static_cast<int>((static_cast<long long>(count) * G + rows - 1) / rows);
}
// Tokens of request i, 0 where its bounds are malformed.
__device__ __forceinline__ int request_tokens(const PackedArgs &a, int i, int *first) {
    const int lo = a.starts[i], hi = a.starts[i + 1];
    *first = lo;
    return lo >= 0 && hi >= lo && hi <= a.T ? hi - lo : 0;
}
// The u-th row tile, requests in order, or b = -1 behind the last.  A wave sums the
// tiles of 64 requests at a time.
__device__ __forceinline__ Unit find_unit(const PackedArgs &a, int u, int rows, int lane) {
    long long before = 0;
    for (int i0 = 0; i0 < a.B; i0 += kWave) {
        int first = 0, count = 0;
        if (i0 + lane < a.B) count = request_tokens(a, i0 + lane, &first);
        const int mine = tiles_of(count, a.G, rows);
        long long up = mine;
#pragma unroll
        for (int o = 1; o < kWave; o <<= 1) {
            const long long y = __shfl_up(up, o, kWave);
            if (lane >= o) up += y;
        }
        const uint64_t past = __ballot(before + up > u);
        if (past) {
            const int at = __ffsll(static_cast<long long>(past)) - 1;
            Unit r;
            r.b = i0 + at;
            r.count = uniform(__shfl(count, at, kWave));
            r.first = uniform(__shfl(first, at, kWave));
            const int tiles = uniform(__shfl(mine, at, kWave));
            r.tile = uniform(static_cast<int>(u - before - (__shfl(up, at, kWave) - tiles)));
            r.last = r.tile == tiles - 1;
            return r;
        }
        before += __shfl(up, kWave - 1, kWave);
    }
    return Unit{-1, 0, 0, 0, false};
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

template <int D, bool E4M3, int QT>
__global__ __launch_bounds__(kBlock, QT * D > 128 ? 1 : 2) void k_attend_packed(PackedArgs a) {
    constexpr int kRows = 128 * QT;               // of a workgroup
    constexpr int kSteps = D / 16;                // of the first product
    constexpr int kVals = D / 32;                 // 32-value blocks of a row of V
    constexpr int kRowB = D * 2;                  // bytes of a row in LDS
    constexpr int kElem = E4M3 ? 1 : 2;
    constexpr int kRowChunks = D * kElem / 16;    // 16-byte chunks of a row in memory
    constexpr int kLoads = kSlots * kRowChunks / kBlock;  // of a lane, for K and for V
    constexpr int kStep = kBlock / kRowChunks;    // rows that one load of the workgroup covers
    __shared__ __align__(1024) char kv[2][2][kSlots * kRowB];  // [stage][K, V]
    __shared__ __align__(16) float scales[2][2][kSlots];       // e4m3: of the tile's slots
    __shared__ int odd_tile[2];                   // the tile of a stage where V has a non-finite value
    const int lane = threadIdx.x & (kWave - 1), w = uniform(static_cast<int>(threadIdx.x >> 6));
    const int half = lane >> 5, col = lane & 31;

    if (blockIdx.x == 0 && a.status) {  // requests without rows, or with malformed bounds
        for (int b = threadIdx.x; b < a.B; b += kBlock) {
            int first;
            if (request_tokens(a, b, &first) == 0) a.status[b] = first == a.starts[b + 1] && first >= 0 && first <= a.T ? 0 : 2;
        }
    }
    // the rows that see most come first
    const int h = blockIdx.x % a.Hkv, rest = blockIdx.x / a.Hkv;
    const int split = rest % a.S, u = a.units - 1 - rest / a.S;
    const Unit un = find_unit(a, u, kRows, lane);
    if (un.b < 0) return;
    const int base = a.base ? uniform(a.base[un.b]) : 0;
    const int rows = static_cast<int>(min(static_cast<long long>(un.count) * a.G - static_cast<long long>(un.tile) * kRows, static_cast<long long>(kRows)));
    const long long r0 = static_cast<long long>(un.tile) * kRows;
    // slots that exist, and the slots that the tile's first and last row see
    const long long exist = static_cast<long long>(a.P) << a.page_shift;
    const long long want = static_cast<long long>(base) + (r0 + rows - 1) / a.G + 1;
    const bool inside = base >= 0;
    const int total = inside ? static_cast<int>(min(want, exist)) : 0;
    const int least = inside ? static_cast<int>(min(static_cast<long long>(base) + r0 / a.G + 1, exist)) : 0;
    int first_bad = inside ? (want > exist ? static_cast<int>(exist) : 0x7fffffff) : -0x7fffffff;

    const int tiles = (total + kSlots - 1) / kSlots;
    const int active = splits_of(tiles, a.S);
    if (split >= active) return;
    const int t0 = static_cast<int>(static_cast<long long>(tiles) * split / active);
    const int t1 = static_cast<int>(static_cast<long long>(tiles) * (split + 1) / active);

    // this lane's query rows and how many slots they see
    bf16x8 q[QT][kSteps];
    int sees[QT], token[QT], head[QT];
    int wave_least = 0x7fffffff, wave_most = 0;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = w * 32 * QT + t * 32 + col;
        const bool live = r < rows;
        const long long at = r0 + (live ? r : 0);
        const int j = static_cast<int>(at / a.G), g = static_cast<int>(at - static_cast<long long>(j) * a.G);
        token[t] = live ? un.first + j : -1;
        head[t] = h * a.G + g;
        sees[t] = live ? static_cast<int>(min(static_cast<long long>(base) + j + 1, exist + 1)) : 0;
        const uint16_t *p = a.q + (un.first + j) * a.q_stride + static_cast<long long>(head[t]) * D + half * 8;
#pragma unroll
        for (int c = 0; c < kSteps; ++c) {
            u32x4 x = {0, 0, 0, 0};
            if (live) x = *reinterpret_cast<const u32x4 *>(p + c * 16);
            q[t][c] = __builtin_bit_cast(bf16x8, x);
        }
    }
    {
        const long long ra = r0 + w * 32 * QT, rb = min(ra + 32 * QT, r0 + rows) - 1;
        if (rb >= ra) {
            wave_least = static_cast<int>(min(base + ra / a.G + 1, exist + 1));
            wave_most = static_cast<int>(min(base + rb / a.G + 1, exist + 1));
        }
    }

    f32x16 o[QT][kVals];
    float m[QT], shift[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = kNoRef;
        shift[t] = kFar;
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < kVals; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[t][i][e] = 0.0f;
    }
    bool far = false;  // a row of the wave has a reference too large for the fma

    // ---- a tile's rows, from memory to registers to LDS
    const int32_t *table = a.page_table + static_cast<long long>(un.b) * a.P;
    const int page_mask = (1 << a.page_shift) - 1;
    int ids = 0;  // lane i: the page of the i-th 16 slots of 16 tiles
    const int row_in = static_cast<int>(threadIdx.x) / kRowChunks, chunk = static_cast<int>(threadIdx.x) % kRowChunks;
    u32x4 kr[kLoads], vr[kLoads];
    float sr = 0.0f;
    auto load = [&](int tile) {
        const int in = (tile - t0) & 15;
        if (in == 0) {
            const int s = tile * kSlots + 16 * lane;
            const bool there = s < total;
            ids = there ? table[s >> a.page_shift] : 0;
            const bool bad = ids < 0 || ids >= a.num_pages;
            if (bad) {
                if (s < t1 * kSlots) first_bad = min(first_bad, s);
                ids = 0;
            }
        }
        auto row_of = [&](int group) {  // the row of the cache where 16 slots of the tile begin
            const int page = __builtin_amdgcn_readlane(ids, in * 4 + group);
            const int s = tile * kSlots + 16 * group;
            return ((static_cast<long long>(page) * a.Hkv + h) << a.page_shift) + (s & page_mask);
        };
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            // a wave's rows lie in one group of 16 slots
            const int r = i * kStep + row_in, group = uniform((i * kStep + w * (kStep / 4)) / 16);
            const long long at = (row_of(group) + (r & 15)) * (D * kElem) + chunk * 16;
            kr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.k_pages) + at);
            vr[i] = *reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.v_pages) + at);
        }
        if constexpr (E4M3) {
            // waves 0 and 1: lane i the scale of slot i, of K and of V
            if (w < 2) {
                long long at = 0;
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const long long x = row_of(g) + (lane & 15);
                    if (lane / 16 == g) at = x;
                }
                sr = (w == 0 ? a.k_scale : a.v_scale)[at];
            }
        }
    };
    auto store = [&](int tile) {
        const int st = (tile - t0) & 1;
        const bool edge = (tile + 1) * kSlots > least;  // some row does not see all of it
        bool odd = false;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int r = i * kStep + row_in;
            constexpr int kParts = E4M3 ? 2 : 1;
            u32x4 kp[kParts], vp[kParts];
            if constexpr (E4M3) {
#pragma unroll
                for (int p = 0; p < 2; ++p)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        kp[p][2 * e] = e4m3_to_bf16<false>(kr[i][2 * p + e]);
                        kp[p][2 * e + 1] = e4m3_to_bf16<true>(kr[i][2 * p + e]);
                        vp[p][2 * e] = e4m3_to_bf16<false>(vr[i][2 * p + e]);
                        vp[p][2 * e + 1] = e4m3_to_bf16<true>(vr[i][2 * p + e]);
                    }
            } else {
                kp[0] = kr[i];
                vp[0] = vr[i];
            }
            if (edge) {
                const bool behind = tile * kSlots + r >= total;
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (behind) vp[p][e] = 0;
                        odd |= has_nonfinite(vp[p][e]);
                        vp[p][e] = finite_only(vp[p][e]);
                    }
            }
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const int c = chunk * kParts + p;
                *reinterpret_cast<u32x4 *>(&kv[st][0][r * kRowB + k_chunk<D>(r, c) * 16]) = kp[p];
                *reinterpret_cast<u32x4 *>(&kv[st][1][r * kRowB + v_chunk<D>(r, c) * 16]) = vp[p];
            }
        }
        if (odd) odd_tile[st] = tile;
        if constexpr (E4M3) {
            if (w < 2) scales[st][w][lane] = sr;
        }
    };

    if (threadIdx.x < 2) odd_tile[threadIdx.x] = -1;
    __syncthreads();
    if (t0 < t1) {
        load(t0);
        store(t0);
    }
    for (int tile = t0; tile < t1; ++tile) {
        __syncthreads();  // the tile is there, and the other stage free
        const bool more = tile + 1 < t1;
        if (more) load(tile + 1);
        const int st = (tile - t0) & 1, s0 = tile * kSlots;
        if (s0 < wave_most) {
            // scores: slot s0 + 32 f + 8 (e / 4) + 4 half + e % 4 of row col
            f32x16 s[QT][2];
#pragma unroll
            for (int f = 0; f < 2; ++f) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[t][f][e] = 0.0f;
#pragma unroll
                for (int c = 0; c < kSteps; ++c) {
                    const bf16x8 kf = *reinterpret_cast<const bf16x8 *>(
                        &kv[st][0][(32 * f + col) * kRowB + k_chunk<D>(32 * f + col, 2 * c + half) * 16]);
#pragma unroll
                    for (int t = 0; t < QT; ++t) s[t][f] = mfma32(kf, q[t][c], s[t][f]);
                }
            }
            if constexpr (E4M3) {
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        const f32x4 ks = *reinterpret_cast<const f32x4 *>(&scales[st][0][32 * f + 8 * x + 4 * half]);
#pragma unroll
                        for (int t = 0; t < QT; ++t)
#pragma unroll
                            for (int e = 0; e < 4; ++e) s[t][f][4 * x + e] *= ks[e];
                    }
            }
            const bool edge = s0 + kSlots > wave_least;
            if (edge) {
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const int slot = s0 + 32 * f + 8 * (e / 4) + 4 * half + e % 4;
                            if (slot >= sees[t]) s[t][f][e] = -__builtin_huge_valf();
                        }
            }
            bf16x8 p[QT][4];
#pragma unroll
            for (int t = 0; t < QT; ++t) {
                float most = fmaxf(s[t][0][0], s[t][1][0]);
#pragma unroll
                for (int e = 1; e < 16; ++e) most = fmaxf(most, fmaxf(s[t][0][e], s[t][1][e]));
                const float top = relative(most, m[t], shift[t], a.c);
                if (__ballot(top > kSlack) != 0) {
                    const float to = fmaxf(m[t], pair_max(most)), now = shift_of(to, a.c);
                    const float f = fast_exp2(rebase(m[t], shift[t], to, now, a.c));
                    l[t] *= f;
#pragma unroll
                    for (int i = 0; i < kVals; ++i) o[t][i] *= f;
                    m[t] = to;
                    shift[t] = now;
                    far = false;
#pragma unroll
                    for (int x = 0; x < QT; ++x) far |= shift[x] == kFar && m[x] != kNoRef;
                    far = __ballot(far) != 0;
                }
                float sum = 0.0f;
                if (!far) {
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[t][f][e] = fast_exp2(fmaf(s[t][f][e], a.c, -shift[t]));
                } else {
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int e = 0; e < 16; ++e) s[t][f][e] = fast_exp2(relative(s[t][f][e], m[t], shift[t], a.c));
                }
#pragma unroll
                for (int f = 0; f < 2; ++f)
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum += s[t][f][e];
                l[t] += sum;
                if constexpr (E4M3) {
#pragma unroll
                    for (int f = 0; f < 2; ++f)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const f32x4 vs = *reinterpret_cast<const f32x4 *>(&scales[st][1][32 * f + 8 * x + 4 * half]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const int slot = s0 + 32 * f + 8 * x + 4 * half + e;
                                const float y = s[t][f][4 * x + e] * vs[e];
                                s[t][f][4 * x + e] = edge && slot >= sees[t] ? 0.0f : y;
                            }
                        }
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int f = i / 2, e = 8 * (i % 2);
                    p[t][i] = as_bf16x8(pack_bf16(s[t][f][e], s[t][f][e + 1]), pack_bf16(s[t][f][e + 2], s[t][f][e + 3]),
                                        pack_bf16(s[t][f][e + 4], s[t][f][e + 5]), pack_bf16(s[t][f][e + 6], s[t][f][e + 7]));
                }
            }
            // lane i of 16 addresses 4 values of row i / 4 and gets value i of the 4 rows
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int d = 0; d < kVals; ++d) {
                    bf16x4 part[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int r = 16 * i + 8 * x + 4 * half + (lane & 15) / 4;
                        const int byte = (d * 32 + ((lane >> 4) & 1) * 16 + (lane & 3) * 4) * 2;
                        part[x] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                            (SV_LDS bf16x4 *)&kv[st][1][r * kRowB + v_chunk<D>(r, byte / 16) * 16 + byte % 16]);
                    }
                    const bf16x8 vt = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
                    for (int t = 0; t < QT; ++t) o[t][d] = mfma32(vt, p[t][i], o[t][d]);
                }
            if (uniform(odd_tile[st]) == tile) {
                // the non-finite values, one by one, for the rows that see their slot
                for (int e = 0; e < kSlots && s0 + e < total; ++e) {
                    const int page = uniform(table[(s0 + e) >> a.page_shift]);
                    const long long at = (((page < 0 || page >= a.num_pages ? 0LL : page) * a.Hkv + h) << a.page_shift) +
                                         ((s0 + e) & page_mask);
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                        float mine = 0.0f;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
#pragma unroll
                            for (int x = 0; x < 8; ++x)
                                if (16 * i + 8 * (x / 4) + 4 * half + x % 4 == e) mine = static_cast<float>(p[t][i][x]);
                        const float weight = __shfl(mine, ((e >> 2) & 1) * 32 + col, kWave);
                        if (s0 + e >= sees[t]) continue;
#pragma unroll
                        for (int d = 0; d < kVals; ++d)
#pragma unroll
                            for (int x = 0; x < 16; ++x) {
                                const long long i = at * D + d * 32 + 8 * (x / 4) + 4 * half + x % 4;
                                float v;
                                if constexpr (E4M3)
                                    v = __uint_as_float(e4m3_to_bf16<false>(static_cast<const uint8_t *>(a.v_pages)[i]) << 16);
                                else
                                    v = bf16_to_f32(static_cast<const uint16_t *>(a.v_pages)[i]);
                                if (!isfinite(v)) o[t][d][x] += weight * v;
                            }
                    }
                }
            }
        }
        if (more) store(tile + 1);
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
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const float L = pair_sum(l[t]);
        if (token[t] < 0) continue;
        if (alone) {
            const bool none = first_bad < sees[t];
            const float f = none ? 0.0f : 1.0f / L;
            const long long to = static_cast<long long>(token[t]) * a.H + head[t];
            if (a.lse && half == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(m[t], L, a.c);
            uint16_t *dst = a.out + to * D + 4 * half;
#pragma unroll
            for (int d = 0; d < kVals; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = none ? 0.0f : o[t][d][4 * x + e] * f;
                    *reinterpret_cast<u32x2 *>(dst + d * 32 + 8 * x) = u32x2{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
                }
        } else {
            const long long row = unit * kRows + w * 32 * QT + t * 32 + col;
            if (half == 0) {
                a.part_ml[row * 2] = m[t];
                a.part_ml[row * 2 + 1] = L;
            }
            float *dst = a.part_o + row * D + 4 * half;
#pragma unroll
            for (int d = 0; d < kVals; ++d)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    *reinterpret_cast<f32x4 *>(dst + d * 32 + 8 * x) =
                        f32x4{o[t][d][4 * x], o[t][d][4 * x + 1], o[t][d][4 * x + 2], o[t][d][4 * x + 3]};
        }
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
    const int base = a.base ? uniform(a.base[un.b]) : 0;
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
    const float shift = shift_of(m, a.c);
    float L = 0.0f;
    f32x4 o = {0, 0, 0, 0};
    for (int s = 0; s < active; ++s) {
        const long long row = (unit + s) * rows_per + r;
        const float ms = a.part_ml[row * 2], ls = a.part_ml[row * 2 + 1];
        const float f = ls == 0.0f ? 0.0f : fast_exp2(rebase(ms, shift_of(ms, a.c), m, shift, a.c));
        L += ls * f;
        o += *reinterpret_cast<const f32x4 *>(a.part_o + row * D + d) * f;
    }
    const bool none = first_bad < static_cast<long long>(base) + j + 1;
    const long long to = static_cast<long long>(un.first + j) * a.H + h * a.G + g;
    if (a.lse && d == 0) a.lse[to] = none ? -__builtin_huge_valf() : log_sum(m, L, a.c);
    const float f = none ? 0.0f : 1.0f / L;
    if (none) o = f32x4{0, 0, 0, 0};
    *reinterpret_cast<u32x2 *>(a.out + to * D + d) = u32x2{pack_bf16(o.x * f, o.y * f), pack_bf16(o.z * f, o.w * f)};
}

size_t align_up(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

template <int D, bool E4M3>
hipError_t launch_qt(const PackedArgs &a, const PackedPlan &p, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(packed_groups(a.Hkv, p)));
    if constexpr (D < 256)
        if (p.QT == 2) return launch_kernel(k_attend_packed<D, E4M3, 2>, grid, dim3(kBlock), 0, s, a);
    return launch_kernel(k_attend_packed<D, E4M3, 1>, grid, dim3(kBlock), 0, s, a);
}
template <int D>
hipError_t launch_d(const PackedArgs &a, bool e4m3, const PackedPlan &p, hipStream_t s) {
    return e4m3 ? launch_qt<D, true>(a, p, s) : launch_qt<D, false>(a, p, s);
}

}  // namespace

long long packed_groups(int Hkv, const PackedPlan &p) { return static_cast<long long>(p.units) * Hkv * p.S; }

long long packed_join_groups(int Hkv, int D, const PackedPlan &p) {
    return p.S == 1 ? 0 : static_cast<long long>(p.units) * Hkv * (p.rows / (kBlock / (D / 4)));
}

PackedPlan packed_plan(int T, int B, int H, int Hkv, int D, int P, int page_size) {
    PackedPlan p = {};
    const long long all = static_cast<long long>(T) * (H / Hkv);
    p.QT = 1;
    p.rows = 128 * p.QT;
    // every request may end in a part of a tile; none has more tiles than rows
    p.units = static_cast<int>(std::max(1LL, std::min(all / p.rows + B, all)));
    const long long tiles = (static_cast<long long>(P) * page_size + kSlots - 1) / kSlots;
    const long long groups = static_cast<long long>(p.units) * Hkv;
    long long S = std::max(1LL, 512 / std::max(1LL, groups));
    S = std::min(S, std::max(1LL, tiles / kLeastRun));
    const size_t per = static_cast<size_t>(groups) * p.rows * (D + 2) * 4;
    while (S > 1 && per * S > (size_t{512} << 20)) --S;
    p.S = static_cast<int>(S);
    if (S > 1) {
        size_t o = 0;
        p.part_o = o;
        o = align_up(o + static_cast<size_t>(groups) * S * p.rows * D * 4);
        p.part_ml = o;
        o = align_up(o + static_cast<size_t>(groups) * S * p.rows * 2 * 4);
        p.part_bad = o;
        o = align_up(o + static_cast<size_t>(groups) * S * 4);
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
