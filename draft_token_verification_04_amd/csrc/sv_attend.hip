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
// slots at a time, with nothing in LDS:
//   S^T = K Q^T   (16x16x32 MFMAs; K is the left operand: its rows are 16
//                  slots, loaded 16 bytes per lane straight from the page)
//   online softmax; lane l holds 8 slots of row l % 16, so the running maximum
//                  needs two cross-lane swaps and the sum none until the end;
//   O^T += V^T P^T: lane l's 8 weights are exactly the k-slice that MFMA's
//                  right operand wants from it (the contraction runs over the
//                  slots in the order (half, lane group, register)), so the
//                  weights go from the softmax to the product without leaving
//                  the lane.  The left operand V^T wants 8 slots of one value:
//                  lane l loads 16 bytes (8 values) of each of its 8 slots and
//                  transposes the 8 x 8 block in registers (v_perm), which
//                  serves 8 MFMAs, MFMA i holding values d = 8 m + i.
// The weights are rounded to bf16 for the second product (relative 2^-9 each,
// independent, averaged over the slots); l sums them unrounded, and every
// accumulator, maximum and sum is fp32.  An e4m3 cache is widened to bf16 in
// registers (exact); its per-row scales multiply the scores and the weights.
//
// Work split: the slots of a (request, KV head) go to `active` of S
// workgroups, each of whose 4 waves takes a run of tiles; a workgroup joins
// its waves through LDS and writes either the result (one active split) or a
// partial (m, l, O) that k_attend_join joins.  S comes from the table's size
// on the host, the runs from the request's own length on the device, so a
// captured graph replays with other lengths.
//
// Masked slots: scores are replaced, never added to; value rows behind the
// last token are zeroed; and a non-finite value of a window token is left to
// the rows that see the token (0 * inf would reach the others).
#include <algorithm>

#include "sv_internal.hpp"
#include "sv_paged.hpp"

namespace sv {
namespace {

constexpr int kTile = 32;  // slots a wave takes per step

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
    int base, count, total, tiles, per_wave, active;
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
    const int most = a.S * kWavesPerBlock;
    s.per_wave = max(a.min_tiles, (s.tiles + most - 1) / most);
    const int per_split = s.per_wave * kWavesPerBlock;
    s.active = (s.tiles + per_split - 1) / per_split;
    return s;
}

// The 8 bf16 values of 16 bytes, or of 8 e4m3 bytes.
__device__ __forceinline__ bf16x8 as_bf16x8(unsigned a, unsigned b, unsigned c, unsigned d) {
    const u32x4 v = {a, b, c, d};
    return __builtin_bit_cast(bf16x8, v);
}
__device__ __forceinline__ bf16x8 widen8(unsigned lo, unsigned hi) {
    return as_bf16x8(e4m3_to_bf16<false>(lo), e4m3_to_bf16<true>(lo), e4m3_to_bf16<false>(hi), e4m3_to_bf16<true>(hi));
}

__device__ __forceinline__ bool has_nonfinite(unsigned w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}
// The word with its non-finite halves cleared.
__device__ __forceinline__ unsigned finite_only(unsigned w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int D, bool E4M3, int QT>
__global__ __launch_bounds__(kBlock) void k_attend(AttendArgs a) {
    constexpr int kChunks = D / 32;       // 32-value steps of the first product
    constexpr int kVals = D / 16;         // values per lane of V: one MFMA each
    constexpr int kWords = kVals / 2;     // packed pairs
    constexpr int kElem = E4M3 ? 1 : 2;
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
    const int rows = sp.count * a.G, row0 = qb * QT * 16;
    if (!sp.ok || rows == 0) {
        if (split == 0) {  // a malformed request reads as zeros
            for (int i = threadIdx.x; i < QT * 16 * D; i += kBlock) {
                const int r = row0 + i / D;
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

    // this lane's query rows: the right operand's column `col` of each row tile
    bf16x8 qf[QT][kChunks];
    uint64_t sees[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        const int r = row0 + t * 16 + col;
        const bool live = r < rows;
        const int n = live ? r / a.G : 0, g = live ? r % a.G : 0;
        sees[t] = __shfl(anc, n, kWave);
        const uint16_t *q = a.q + (static_cast<long long>(b) * a.N + n) * a.q_stride + static_cast<long long>(h * a.G + g) * D;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            // e4m3 rows are read 16 values per lane, which are two chunks' slices
            const int d = E4M3 ? (c / 2) * 64 + kg * 16 + (c % 2) * 8 : c * 32 + kg * 8;
            uint4 x = make_uint4(0, 0, 0, 0);
            if (live) x = *reinterpret_cast<const uint4 *>(q + d);
            qf[t][c] = as_bf16x8(x.x, x.y, x.z, x.w);
        }
    }

    f32x4 o[QT][kVals];
    float m[QT], l[QT];
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        m[t] = -__builtin_huge_valf();
        l[t] = 0.0f;
#pragma unroll
        for (int i = 0; i < kVals; ++i) o[t][i] = f32x4{0, 0, 0, 0};
    }

    const int32_t *table = a.page_table + static_cast<long long>(b) * a.P;
    const int page_mask = (1 << a.page_shift) - 1;
    const char *kp = static_cast<const char *>(a.k_pages), *vp = static_cast<const char *>(a.v_pages);
    bool bad = false;
    const int t0 = (split * kWavesPerBlock + w) * sp.per_wave;
    const int t1 = min(t0 + sp.per_wave, sp.tiles);
    for (int tile = t0; tile < t1; ++tile) {
        const int s0 = tile * kTile;
        // row (in units of rows) of the first slot of each 16-slot half
        long long row[2];
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const int s = s0 + 16 * f < sp.total ? s0 + 16 * f : s0;
            int page = uniform(table[s >> a.page_shift]);
            if (page < 0 || page >= a.num_pages) {
                bad = true;
                page = 0;
            }
            row[f] = ((static_cast<long long>(page) * a.Hkv + h) << a.page_shift) + (s & page_mask);
        }
        bf16x8 kf[2][kChunks];
        unsigned vw[2][4][kWords];  // [half][slot][pair of values]
#pragma unroll
        for (int f = 0; f < 2; ++f) {
            const char *p = kp + (row[f] + col) * (D * kElem);
            if constexpr (E4M3) {
#pragma unroll
                for (int c = 0; c < kChunks; c += 2) {
                    const u32x4 x = *reinterpret_cast<const u32x4 *>(p + c * 32 + kg * 16);
                    kf[f][c] = widen8(x.x, x.y);
                    kf[f][c + 1] = widen8(x.z, x.w);
                }
            } else {
#pragma unroll
                for (int c = 0; c < kChunks; ++c)
                    kf[f][c] = *reinterpret_cast<const bf16x8 *>(p + (c * 32 + kg * 8) * 2);
            }
        }
#pragma unroll
        for (int f = 0; f < 2; ++f)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const char *p = vp + (row[f] + kg * 4 + j) * (D * kElem) + col * (kVals * kElem);
                if constexpr (E4M3) {
#pragma unroll
                    for (int i = 0; i < kVals / 4; ++i) {
                        const unsigned x = reinterpret_cast<const unsigned *>(p)[i];
                        vw[f][j][2 * i] = e4m3_to_bf16<false>(x);
                        vw[f][j][2 * i + 1] = e4m3_to_bf16<true>(x);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < kWords; ++i) vw[f][j][i] = reinterpret_cast<const unsigned *>(p)[i];
                }
            }
        f32x4 ks[2], vs[2];
        if constexpr (E4M3) {
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                ks[f] = *reinterpret_cast<const f32x4 *>(a.k_scale + row[f] + kg * 4);
                vs[f] = *reinterpret_cast<const f32x4 *>(a.v_scale + row[f] + kg * 4);
            }
        }

        // scores: slot s0 + 16 f + 4 kg + j of row col
        f32x4 sc[QT][2];
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
                f32x4 x = {0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < kChunks; ++c) x = mfma16(kf[f][c], qf[t][c], x);
                if constexpr (E4M3) x *= ks[f];
                sc[t][f] = x;
            }
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
                        for (int i = 0; i < kWords; ++i) {
                            if (s >= sp.total) vw[f][j][i] = 0;
                            odd |= has_nonfinite(vw[f][j][i]);
                            vw[f][j][i] = finite_only(vw[f][j][i]);
                        }
                    }
#pragma unroll
                    for (int t = 0; t < QT; ++t)
                        if (!(s < sp.base || (s < sp.total && ((sees[t] >> (s - sp.base)) & 1))))
                            sc[t][f][j] = -__builtin_huge_valf();
                }
            odd = ballot(odd) != 0;
        }

        // V^T: for each of the lane's values its 8 slots, in the order (half, slot)
        bf16x8 vt[kVals];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            unsigned lo[4], hi[4];
#pragma unroll
            for (int f = 0; f < 2; ++f)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    lo[2 * f + j] = __builtin_amdgcn_perm(vw[f][2 * j + 1][i], vw[f][2 * j][i], 0x05040100u);
                    hi[2 * f + j] = __builtin_amdgcn_perm(vw[f][2 * j + 1][i], vw[f][2 * j][i], 0x07060302u);
                }
            vt[2 * i] = as_bf16x8(lo[0], lo[1], lo[2], lo[3]);
            vt[2 * i + 1] = as_bf16x8(hi[0], hi[1], hi[2], hi[3]);
        }

#pragma unroll
        for (int t = 0; t < QT; ++t) {
            float top = fmaxf(fmaxf(sc[t][0][0], sc[t][0][1]), fmaxf(sc[t][0][2], sc[t][0][3]));
            top = fmaxf(top, fmaxf(fmaxf(sc[t][1][0], sc[t][1][1]), fmaxf(sc[t][1][2], sc[t][1][3])));
            top = fmaxf(m[t], quad_max(top));
            if (ballot(top > m[t]) != 0) {
                const float f = m[t] == -__builtin_huge_valf() ? 0.0f : fast_exp2((m[t] - top) * a.c);
                l[t] *= f;
#pragma unroll
                for (int i = 0; i < kVals; ++i) o[t][i] *= f;
                m[t] = top;
            }
            const float ref = m[t] == -__builtin_huge_valf() ? 0.0f : m[t] * a.c;
            float p[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                p[e] = fast_exp2(fmaf(sc[t][e / 4][e % 4], a.c, -ref));
                l[t] += p[e];
            }
            if constexpr (E4M3) {
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float x = p[e] * vs[e / 4][e % 4];
                    p[e] = edge && sc[t][e / 4][e % 4] == -__builtin_huge_valf() ? 0.0f : x;
                }
            }
            const bf16x8 pf = as_bf16x8(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]), pack_bf16(p[4], p[5]),
                                        pack_bf16(p[6], p[7]));
#pragma unroll
            for (int i = 0; i < kVals; ++i) o[t][i] = mfma16(vt[i], pf, o[t][i]);
            if (odd) {
                // the non-finite values, one by one, for the rows that see their token
                for (int s = max(s0, sp.base); s < min(s0 + kTile, sp.total); ++s) {
                    const int e = s - s0;
                    float mine = 0.0f;
#pragma unroll
                    for (int x = 0; x < 8; ++x)
                        if (x == (e / 16) * 4 + e % 4) mine = p[x];
                    const float weight = __shfl(mine, (e % 16) / 4 * 16 + col, kWave);
                    if (!((sees[t] >> (s - sp.base)) & 1)) continue;
                    const long long at = (row[e / 16] + e % 16) * D;
#pragma unroll
                    for (int i = 0; i < kVals; ++i)
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int d = (kg * 4 + j) * kVals + i;
                            float v;
                            if constexpr (E4M3)
                                v = __uint_as_float(e4m3_to_bf16<false>(reinterpret_cast<const uint8_t *>(vp)[at + d]) << 16);
                            else
                                v = bf16_to_f32(reinterpret_cast<const uint16_t *>(vp)[at + d]);
                            if (!isfinite(v)) o[t][i][j] += weight * v;
                        }
                }
            }
        }
    }

    // join the four waves' rows through LDS, one row tile at a time
    constexpr int kPad = 4;
    __shared__ float so[kWavesPerBlock][16][D + kPad];
    __shared__ float sm[kWavesPerBlock][16], sl[kWavesPerBlock][16];
    __shared__ int sbad;
    if (threadIdx.x == 0) sbad = 0;
    __syncthreads();
    if (bad) sbad = 1;
    const long long unit = ((static_cast<long long>(b) * a.Hkv + h) * a.QB + qb) * a.S + split;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
        if (t > 0) __syncthreads();
        const float ll = quad_sum(l[t]);
        if (kg == 0) {
            sm[w][col] = m[t];
            sl[w][col] = ll;
        }
        // the lane's values: d = (4 kg + j) kVals + i
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int i = 0; i < kVals; i += 4)
                *reinterpret_cast<float4 *>(&so[w][col][(kg * 4 + j) * kVals + i]) =
                    make_float4(o[t][i][j], o[t][i + 1][j], o[t][i + 2][j], o[t][i + 3][j]);
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * (D / 4); i += kBlock) {
            const int rr = i / (D / 4), d = i % (D / 4) * 4;
            const int r = row0 + t * 16 + rr;
            if (r >= rows) break;
            const float M = fmaxf(fmaxf(sm[0][rr], sm[1][rr]), fmaxf(sm[2][rr], sm[3][rr]));
            float L = 0.0f;
            float4 x = make_float4(0, 0, 0, 0);
#pragma unroll
            for (int v = 0; v < kWavesPerBlock; ++v) {
                if (sm[v][rr] == -__builtin_huge_valf()) continue;
                const float f = fast_exp2((sm[v][rr] - M) * a.c);
                L += sl[v][rr] * f;
                const float4 y = *reinterpret_cast<const float4 *>(&so[v][rr][d]);
                x.x += y.x * f;
                x.y += y.y * f;
                x.z += y.z * f;
                x.w += y.w * f;
            }
            if (sp.active == 1) {
                const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
                const bool none = sbad || M == -__builtin_huge_valf();
                const float f = none ? 0.0f : 1.0f / L;
                uint2 y = make_uint2(0, 0);
                if (!none) y = make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
                *reinterpret_cast<uint2 *>(a.out + to * D + d) = y;
                if (a.lse && d == 0) a.lse[to] = none ? -__builtin_huge_valf() : M * a.scale + logf(L);
            } else {
                const long long at = unit * (QT * 16) + t * 16 + rr;
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

// One wave per row: the active splits' partials joined.
template <int D>
__global__ __launch_bounds__(kBlock) void k_attend_join(AttendArgs a, int tile_rows) {
    const int lane = threadIdx.x & (kWave - 1);
    const long long wave = static_cast<long long>(blockIdx.x) * kWavesPerBlock + (threadIdx.x >> 6);
    const int all = a.N * a.G;
    if (wave >= static_cast<long long>(a.B) * a.Hkv * all) return;
    const int r = static_cast<int>(wave % all);
    const int h = static_cast<int>(wave / all % a.Hkv), b = static_cast<int>(wave / all / a.Hkv);
    const Span sp = request_span(a, b, lane, nullptr);
    if (!sp.ok || sp.active <= 1 || r >= sp.count * a.G) return;
    const int qb = r / tile_rows;
    const long long unit = ((static_cast<long long>(b) * a.Hkv + h) * a.QB + qb) * a.S;
    const float ninf = -__builtin_huge_valf();
    bool bad = false;
    float M = ninf;
    for (int s = lane; s < sp.active; s += kWave) {
        bad |= a.part_bad[unit + s] != 0;
        M = fmaxf(M, a.part_ml[((unit + s) * tile_rows + r % tile_rows) * 2]);
    }
    bad = ballot(bad) != 0;
    M = wave_max(M);
    float L = 0.0f;
    constexpr int kPer = D / kWave;
    float x[kPer] = {};
    if (M != ninf) {
#pragma unroll 4
        for (int s = 0; s < sp.active; ++s) {
            const long long at = (unit + s) * tile_rows + r % tile_rows;
            const float ms = a.part_ml[at * 2];
            const float f = ms == ninf ? 0.0f : fast_exp2((ms - M) * a.c);
            L += a.part_ml[at * 2 + 1] * f;
#pragma unroll
            for (int e = 0; e < kPer; ++e) x[e] += a.part_o[at * D + lane * kPer + e] * f;
        }
    }
    const long long to = (static_cast<long long>(b) * a.N + r / a.G) * a.H + h * a.G + r % a.G;
    const bool none = bad || M == ninf;
    const float f = none ? 0.0f : 1.0f / L;
#pragma unroll
    for (int e = 0; e < kPer; ++e)
        a.out[to * D + lane * kPer + e] =
            none ? 0 : static_cast<uint16_t>(pack_bf16(x[e] * f, 0.0f) & 0xffffu);
    if (lane == 0) {
        if (a.lse) a.lse[to] = none ? ninf : M * a.scale + logf(L);
        if (a.status && h == 0 && r == 0) a.status[b] = bad ? 1 : 0;
    }
}

template <int D, bool E4M3>
hipError_t launch_qt(const AttendArgs &a, int QT, dim3 grid, hipStream_t s) {
    if (QT == 1) return launch_kernel(k_attend<D, E4M3, 1>, grid, dim3(kBlock), 0, s, a);
    if constexpr (D <= 128) {
        if (QT == 3) return launch_kernel(k_attend<D, E4M3, 3>, grid, dim3(kBlock), 0, s, a);
        if (QT == 4) return launch_kernel(k_attend<D, E4M3, 4>, grid, dim3(kBlock), 0, s, a);
    }
    return launch_kernel(k_attend<D, E4M3, 2>, grid, dim3(kBlock), 0, s, a);
}

}  // namespace

AttendPlan attend_plan(int B, int N, int H, int Hkv, int D, int P, int page_size) {
    constexpr int kTargetGroups = 1024;  // workgroups a call aims for
    AttendPlan p;
    const int rows = N * (H / Hkv), tiles = (rows + 15) / 16;
    const int most = D <= 128 ? 4 : 2;  // row tiles whose accumulators a wave holds
    p.QB = (tiles + most - 1) / most;
    p.QT = (tiles + p.QB - 1) / p.QB;
    p.min_tiles = p.QT == 1 ? 2 : 4;
    const long long slots = static_cast<long long>(P) * page_size;
    const long long all = (slots + kTile - 1) / kTile, groups = static_cast<long long>(B) * Hkv * p.QB;
    const long long cap = (all + kWavesPerBlock * p.min_tiles - 1) / (kWavesPerBlock * p.min_tiles);
    long long want = (kTargetGroups + groups - 1) / groups;
    want = std::max(want, (all + kWavesPerBlock * 8 - 1) / (kWavesPerBlock * 8));  // 1024 slots per workgroup
    p.S = static_cast<int>(std::max(1LL, std::min({want, cap, 1024LL})));
    const size_t units = static_cast<size_t>(groups) * p.S, n = units * p.QT * 16;
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    p.part_o = 0;
    p.part_ml = up(p.S > 1 ? n * D * sizeof(float) : 0);
    p.part_bad = p.part_ml + up(p.S > 1 ? n * 2 * sizeof(float) : 0);
    p.total = p.part_bad + up(p.S > 1 ? units * sizeof(int32_t) : 0);
    return p;
}

hipError_t launch_attend(const AttendArgs &a, int D, bool e4m3, int QT, hipStream_t s) {
    const long long rest = static_cast<long long>(a.S) * a.B * a.Hkv;
    const dim3 grid(static_cast<unsigned>((rest + 7) / 8 * 8 * a.QB));
    if (D == 64) return e4m3 ? launch_qt<64, true>(a, QT, grid, s) : launch_qt<64, false>(a, QT, grid, s);
    if (D == 128) return e4m3 ? launch_qt<128, true>(a, QT, grid, s) : launch_qt<128, false>(a, QT, grid, s);
    return e4m3 ? launch_qt<256, true>(a, QT, grid, s) : launch_qt<256, false>(a, QT, grid, s);
}

hipError_t launch_attend_join(const AttendArgs &a, int D, int QT, hipStream_t s) {
    const long long waves = static_cast<long long>(a.B) * a.Hkv * a.N * a.G;
    const dim3 grid(static_cast<unsigned>((waves + kWavesPerBlock - 1) / kWavesPerBlock));
    const int rows = QT * 16;
    if (D == 64) return launch_kernel(k_attend_join<64>, grid, dim3(kBlock), 0, s, a, rows);
    if (D == 128) return launch_kernel(k_attend_join<128>, grid, dim3(kBlock), 0, s, a, rows);
    return launch_kernel(k_attend_join<256>, grid, dim3(kBlock), 0, s, a, rows);
}

}  // namespace sv
