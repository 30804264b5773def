// sv_norm.hip -- RMS norm of rows with the residual's addition, to bf16 or to
// e4m3 with one fp32 scale for each 128 columns.
//
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight,
//   residual_out = bf16(h),  out = bf16(y), or e4m3(y * (448 / a)) with the scale
//   a / 448, a = max |y| over the block of 128 columns.
// Everything between the loads and the one rounding at each store is fp32.
//
// Bound by memory: nothing is read twice.  A row is held in registers by TPR
// lanes, 8 consecutive values (16 bytes) each and V such vectors, so a block of
// 128 columns is 16 consecutive lanes, one row of the DPP network: its maximum
// takes four steps and no LDS.  8191 rows of 4096 with residual to e4m3, 236 MB:
// 46 us, 5.1 TB/s, what a large copy reaches (5.2); one row 4 us, the launch.
#include "sv_paged.hpp"
#include "sv_prompt_internal.hpp"

namespace sv {
namespace {

// v of the lane that DPP control CTRL names, inside rows of 16 lanes.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    const int x = __float_as_int(v);
    return __int_as_float(__builtin_amdgcn_update_dpp(x, x, CTRL, 0xf, 0xf, true));
}
// Over the 16 lanes of a DPP row: quad_perm [1, 0, 3, 2], [2, 3, 0, 1], then the
// mirrors of half a row and of a row.
__device__ __forceinline__ float row16_max(float v) {
    v = fmaxf(v, dpp<0xb1>(v));
    v = fmaxf(v, dpp<0x4e>(v));
    v = fmaxf(v, dpp<0x141>(v));
    return fmaxf(v, dpp<0x140>(v));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xb1>(v);
    v += dpp<0x4e>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}

// A row whose mean square and eps overflow together, or are below kLeastMean together
// (the squares that underflow are 2^-150 off each), is scaled by kFar down or up before it
// is squared: its largest value is above 2^56 (or eps is), or below 2^-43, so scaled
// squares neither overflow nor lose what counts.
constexpr float kLeastMean = 0x1p-100f, kFar = 0x1p80f;

template <int TPR, int V, bool E4M3>
__global__ __launch_bounds__(TPR > kBlock ? TPR : kBlock) void k_rms_norm(NormArgs a) {
    constexpr int kThreads = TPR > kBlock ? TPR : kBlock;
    constexpr int kRows = kThreads / TPR, kWaves = TPR / kWave;
    static_assert(kWaves == 1 || kRows == 1, "rows of several waves have a workgroup each");
    __shared__ float sums[kThreads / kWave];
    const int l = threadIdx.x % TPR;
    const int t = blockIdx.x * kRows + static_cast<int>(threadIdx.x) / TPR;
    const bool live = t < a.T;
    const long long row = static_cast<long long>(live ? t : 0) * a.D;
    float h[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (i * TPR + l) * 8;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (live && d < a.D) w = *reinterpret_cast<const uint4 *>(a.x + t * a.x_stride + d);
        unpack(w, h[i]);
    }
    if (a.residual) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int d = (i * TPR + l) * 8;
            if (live && d < a.D) {
                float r[8];
                unpack(*reinterpret_cast<const uint4 *>(a.residual + row + d), r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[i][e] += r[e];
            }
        }
    }
    // the mean of the row's squares, its values times `by` first; the same in all its lanes
    auto mean_square = [&](float by) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float v = h[i][e] * by;
                ss += v * v;
            }
        ss = wave_sum(ss);
        if constexpr (kWaves > 1) {
            sums[threadIdx.x / kWave] = ss;
            __syncthreads();
            ss = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) ss += sums[w];
        }
        return ss / static_cast<float>(a.D);
    };
    float mean = mean_square(1.0f), eps = a.eps, up = 1.0f, down = 1.0f;
    const bool over = isinf(mean + eps);
    if (over || mean + eps < kLeastMean) {  // the same in all lanes of a row
        if constexpr (kWaves > 1) __syncthreads();  // the sums before have been read
        (over ? down : up) = over ? 1.0f / kFar : kFar;
        mean = mean_square(up * down);
        eps = eps * up * down * up * down;
    }
    const float inv = 1.0f / sqrtf(mean + eps);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int d = (i * TPR + l) * 8;
        const bool in = live && d < a.D;
        if (in && a.residual_out)
            *reinterpret_cast<uint4 *>(a.residual_out + row + d) =
                make_uint4(pack_bf16(h[i][0], h[i][1]), pack_bf16(h[i][2], h[i][3]), pack_bf16(h[i][4], h[i][5]),
                           pack_bf16(h[i][6], h[i][7]));
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = h[i][e] * up * inv * down;
        if (a.weight && in) {
            float w[8];
            unpack(*reinterpret_cast<const uint4 *>(a.weight + d), w);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= w[e];
        }
        if constexpr (E4M3) {
            float top = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(y[e]));
            top = row16_max(top);  // lanes behind the row hold zeros
            const float up = top > 0.0f ? 448.0f / fmaxf(top, kMinAmax) : 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] *= up;
            if (in) {
                *reinterpret_cast<u32x2 *>(static_cast<uint8_t *>(a.out) + row + d) =
                    u32x2{pack_e4m3(y[0], y[1], y[2], y[3]), pack_e4m3(y[4], y[5], y[6], y[7])};
                if (l % 16 == 0)
                    a.out_scale[static_cast<long long>(d / kScaleBlock) * a.T + t] =
                        fmaxf(top, top > 0.0f ? kMinAmax : 0.0f) / 448.0f;
            }
        } else if (in) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + row + d) =
                make_uint4(pack_bf16(y[0], y[1]), pack_bf16(y[2], y[3]), pack_bf16(y[4], y[5]), pack_bf16(y[6], y[7]));
        }
    }
}

template <int TPR, int V>
hipError_t launch_v(const NormArgs &a, bool e4m3, hipStream_t s) {
    constexpr int kThreads = TPR > kBlock ? TPR : kBlock, kRows = kThreads / TPR;
    const dim3 grid(static_cast<unsigned>((a.T + kRows - 1) / kRows));
    return e4m3 ? launch_kernel(k_rms_norm<TPR, V, true>, grid, dim3(kThreads), 0, s, a)
                : launch_kernel(k_rms_norm<TPR, V, false>, grid, dim3(kThreads), 0, s, a);
}
template <int TPR>
hipError_t launch_tpr(const NormArgs &a, int vecs, bool e4m3, hipStream_t s) {
    if (vecs <= 1 * TPR) return launch_v<TPR, 1>(a, e4m3, s);
    if (vecs <= 2 * TPR) return launch_v<TPR, 2>(a, e4m3, s);
    if (vecs <= 4 * TPR) return launch_v<TPR, 4>(a, e4m3, s);
    return launch_v<TPR, 8>(a, e4m3, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs &a, bool e4m3, hipStream_t s) {
    const int vecs = a.D / 8;
    if (vecs <= 128) return launch_tpr<64>(a, vecs, e4m3, s);
    return launch_tpr<256>(a, vecs, e4m3, s);
}

}  // namespace sv
