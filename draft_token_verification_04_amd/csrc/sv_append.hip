// sv_append.hip -- a window's keys and values written to a paged cache, with
// the per-head norms and the position rotation of queries and keys.
//
// For every row x of D values (one head of one token):
//   query, key: y = x / sqrt(mean(x^2) + eps) * weight, then the pairs of its
//               first `rot` values turned by the token's angles:
//               (a, b) -> (a cos - b sin, b cos + a sin);
//   value:      y = x.
// Queries go to q_out as bf16; keys and values go to their slot as bf16, or as
// e4m3 with one fp32 scale per row: scale = max|y| / 448 (448: the largest
// e4m3 value), stored y * (448 / max|y|).  Everything between the load and the
// one rounding at the store is fp32.
//
// Bound by memory: a token of 32 + 2 x 8 heads of 128 reads 12 KB and writes
// as much (bf16), and nothing is read twice but the angles.  A row is held by
// D / 8 lanes, 16 bytes each, so a wave holds 64 / (D / 8) rows and the norm,
// the maximum and the half-split rotation's partners move between the lanes of
// a row.  A workgroup takes one token: its lanes keep the token's angles in
// registers over all the rows they walk.
#include "sv_paged.hpp"
#include "sv_paged_internal.hpp"

namespace sv {
namespace {

template <int LANES>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, kWave);
    return v;
}
template <int LANES>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, kWave));
    return v;
}

template <int D, bool E4M3>
__global__ __launch_bounds__(kBlock) void k_append(AppendArgs a) {
    constexpr int kLanes = D / 8;                 // lanes per row
    constexpr int kRows = kBlock / kLanes;        // rows a workgroup holds at once
    const int tok = blockIdx.x;
    const int b = tok / a.N, j = tok - b * a.N;
    const bool first = blockIdx.y == 0 && threadIdx.x == 0;
    if (j >= window_rows(a.counts, b, a.N)) {  // padding: nothing is written
        if (first && a.status) a.status[tok] = 0;
        return;
    }
    // where the token goes; a bad slot, page or position writes nothing
    const long long slot = static_cast<long long>(a.base[b]) + j;
    const int pos = a.rope ? a.positions[tok] : 0;
    int page = -1;
    if (slot >= 0 && (slot >> a.page_shift) < a.P)
        page = a.page_table[static_cast<long long>(b) * a.P + (slot >> a.page_shift)];
    int code = 0;
    if (page < 0 || page >= a.num_pages)
        code = 1;
    else if (a.rope && (pos < 0 || pos >= a.max_pos))
        code = 2;
    if (first && a.status) a.status[tok] = code;
    if (code) return;
    const int in_page = static_cast<int>(slot & ((1 << a.page_shift) - 1));

    const int c = threadIdx.x % kLanes, d0 = c * 8;  // this lane's 8 values of its rows
    const int half = a.rot / 2;
    const bool turned = a.rope && d0 < a.rot;
    // angles of this lane's values.  Half split: values i and i + rot/2 share
    // angle i, so the lane's 8 values have 8 consecutive angles; interleaved:
    // its 4 pairs have 4.
    float cs[8], sn[8];
    const bool upper = d0 >= half;  // half split: holds the second value of its pairs
    if (turned) {
        const float *t = a.rope + static_cast<long long>(pos) * a.rot;
        if (a.interleaved) {
            const float4 x = *reinterpret_cast<const float4 *>(t + d0 / 2);
            const float4 y = *reinterpret_cast<const float4 *>(t + half + d0 / 2);
            cs[0] = cs[1] = x.x, cs[2] = cs[3] = x.y, cs[4] = cs[5] = x.z, cs[6] = cs[7] = x.w;
            sn[0] = sn[1] = y.x, sn[2] = sn[3] = y.y, sn[4] = sn[5] = y.z, sn[6] = sn[7] = y.w;
        } else {
            const int f = upper ? d0 - half : d0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                cs[e] = t[f + e];
                sn[e] = t[half + f + e];
            }
        }
    }
    const int lane = threadIdx.x & (kWave - 1);
    const int partner = upper ? lane - half / 8 : lane + half / 8;

    const int rows = a.H + 2 * a.Hkv;
    for (int r0 = blockIdx.y * kRows; r0 < rows; r0 += gridDim.y * kRows) {
        const int r = r0 + threadIdx.x / kLanes;
        const bool live = r < rows;
        const int kind = r < a.H ? 0 : (r < a.H + a.Hkv ? 1 : 2);  // query, key, value
        const int head = kind == 0 ? r : (kind == 1 ? r - a.H : r - a.H - a.Hkv);
        const uint16_t *src = kind == 0 ? a.q + tok * a.q_stride : (kind == 1 ? a.k + tok * a.k_stride : a.v + tok * a.v_stride);
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live) w = *reinterpret_cast<const uint4 *>(src + static_cast<long long>(head) * D + d0);
        float y[8];
        unpack(w, y);
        const uint16_t *weight = kind == 0 ? a.q_weight : a.k_weight;
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss += y[e] * y[e];
        ss = row_sum<kLanes>(ss);
        if (kind < 2 && weight) {
            const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
            float wt[8];
            unpack(*reinterpret_cast<const uint4 *>(weight + d0), wt);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = y[e] * inv * wt[e];
        }
        if (a.rope) {
            if (a.interleaved) {
                if (turned && kind < 2) {
#pragma unroll
                    for (int e = 0; e < 8; e += 2) {
                        const float u = y[e], t = y[e + 1];
                        y[e] = u * cs[e] - t * sn[e];
                        y[e + 1] = t * cs[e] + u * sn[e];
                    }
                }
            } else {
                float o[8];  // the other value of each pair (every lane takes part)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __shfl(y[e], partner & (kWave - 1), kWave);
                if (turned && kind < 2) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        y[e] = upper ? y[e] * cs[e] + o[e] * sn[e] : y[e] * cs[e] - o[e] * sn[e];
                }
            }
        }
        float inv = 0.0f, top = 0.0f;
        if constexpr (E4M3) {
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
            top = row_max<kLanes>(top);
            inv = top > 0.0f ? 448.0f / fmaxf(top, kMinAmax) : 0.0f;
        }
        if (!live) continue;
        if (kind == 0 || !E4M3) {
            const uint4 o = make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]),
                                       pack_bf16(y[6], y[7]));
            uint16_t *dst;
            if (kind == 0) {
                dst = a.q_out + (static_cast<long long>(tok) * a.H + head) * D;
            } else {
                const long long row =
                    ((static_cast<long long>(page) * a.Hkv + head) << a.page_shift) + in_page;
                dst = static_cast<uint16_t *>(kind == 1 ? a.k_pages : a.v_pages) + row * D;
            }
            __builtin_nontemporal_store(u32x4{o.x, o.y, o.z, o.w}, reinterpret_cast<u32x4 *>(dst + d0));
        } else {
            const long long row = ((static_cast<long long>(page) * a.Hkv + head) << a.page_shift) + in_page;
            uint8_t *dst = static_cast<uint8_t *>(kind == 1 ? a.k_pages : a.v_pages) + row * D;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= inv;
            __builtin_nontemporal_store(u32x2{pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7])},
                                        reinterpret_cast<u32x2 *>(dst + d0));
            if (c == 0) (kind == 1 ? a.k_scale : a.v_scale)[row] = fmaxf(top, top > 0.0f ? kMinAmax : 0.0f) / 448.0f;
        }
    }
}

template <int D>
hipError_t launch_d(const AppendArgs &a, bool e4m3, dim3 grid, hipStream_t s) {
    return e4m3 ? launch_kernel(k_append<D, true>, grid, dim3(kBlock), 0, s, a)
                : launch_kernel(k_append<D, false>, grid, dim3(kBlock), 0, s, a);
}

}  // namespace

// Tokens (padding among them) from which a workgroup takes all of a token's rows, in
// passes, instead of one pass's: lookups and angles are then read once per token.  In
// passes against not, 48 rows of 128 a token, bf16: 256 tokens 5.3 and 4.2 us, 1024
// 7.5 and 8.2, 2112 13.0 and 14.3, 4096 18.9 and 24.1, 8191 33.9 and 46.1 (e4m3 36.9
// and 49.6); 64 windows of up to 33, half of it padding, 9.9 both.  The two cross
// below 1000 tokens; from 4096 on passes gain a fifth and more.
constexpr int kWideTokens = 4096;

hipError_t launch_append(const AppendArgs &a, int D, bool e4m3, int tokens, hipStream_t s) {
    const int rows = a.H + 2 * a.Hkv, per = kBlock / (D / 8);
    const int passes = (rows + per - 1) / per;
    const dim3 grid(static_cast<unsigned>(tokens), static_cast<unsigned>(tokens >= kWideTokens ? 1 : passes));
    if (D == 64) return launch_d<64>(a, e4m3, grid, s);
    if (D == 128) return launch_d<128>(a, e4m3, grid, s);
    return launch_d<256>(a, e4m3, grid, s);
}

}  // namespace sv
