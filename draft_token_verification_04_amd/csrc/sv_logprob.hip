// sv_logprob.hip -- log probabilities of given tokens, the entropy of each row
// and its most probable alternatives, in one read of the logits.
//
// For a row x of V logits and p = softmax(x / T), with c = log2(e) / T:
//   m = max x, d_v = (x_v - m) c, S = sum 2^d_v, U = sum 2^d_v d_v
//   log p_t  = ln 2 ((x_t - m) c - log2 S)
//   entropy  = ln 2 (log2 S - U / S)
// and the k largest (value, lowest index) pairs.
//
// k_logprob: a wave takes a segment of a row, holds it in registers (one read,
// all loads issued before the first use), and leaves (m, S, U) and the
// segment's k best keys.  k_logprob_merge: a wave per row joins its segments.
// Bound by the read of the logits; the exponentials (one per logit, at a
// quarter of the rate of other instructions) come close to it.
//
// The k best of a segment: the k-th largest of the 64 lanes' maxima is a value
// that at least k logits reach, so only logits at or above it (k + a few) are
// candidates.  They are collected in LDS and ranked by counting, for each, how
// many are larger; keys are distinct (the index is part of them), so the
// result does not depend on the order in which they were collected.  Where
// many logits tie (a masked vocabulary), the list is cut back to the k best
// whenever it fills, which raises the bar to the k-th key so far.
#include <algorithm>

#include "sv_internal.hpp"
#include "sv_paged.hpp"

namespace sv {
namespace {

constexpr double kLn2d = 0.6931471805599453094172321214581766;
constexpr int kListCap = 128;  // keys a wave's list holds between cuts

__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// A wave's list of candidate keys in LDS: the k best seen so far are always in
// it.  `bar` is a key that k distinct keys of the list exceed or equal, once
// known: keys below it cannot be among the k best.
struct KeyList {
    uint64_t *buf;  // kListCap keys
    int n, k;
    uint64_t bar;

    __device__ __forceinline__ void init(uint64_t *b, int kk) {
        buf = b;
        n = 0;
        k = kk;
        bar = 0;
    }
    // Adds the keys of the lanes with `take` (wave-uniform control flow).
    __device__ __forceinline__ void push(uint64_t key, bool take, int lane) {
        const uint64_t m = ballot(take);
        if (m == 0) return;
        if (take) buf[n + __popcll(m & ((1ull << lane) - 1))] = key;
        n += __popcll(m);
        if (n > kListCap - kWave) cut(lane);
    }
    // Sorts the list in descending order and keeps its first k.
    __device__ __forceinline__ void cut(int lane) {
        wave_lds_sync();
        const uint64_t a = lane < n ? buf[lane] : 0, b = lane + kWave < n ? buf[lane + kWave] : 0;
        int ra = 0, rb = 0;
        for (int i = 0; i < n; ++i) {
            const uint64_t x = buf[i];
            ra += x > a;
            rb += x > b;
        }
        wave_lds_sync();
        if (lane < n && ra < k) buf[ra] = a;
        if (lane + kWave < n && rb < k) buf[rb] = b;
        n = n < k ? n : k;
        wave_lds_sync();
        if (n == k) bar = uniform(buf[k - 1]);
    }
};

// A row cut into 16-byte vectors on the address's own 16-byte grid: vector j
// holds elements [j P - off, (j + 1) P - off), off = the elements between the
// grid and the row's start.  Elements outside [0, V) are never read: a vector
// that sticks out is put together from single loads, with -inf outside.
template <typename E>
struct RowVecs {
    const typename E::storage *row;
    int V, off;
    __device__ __forceinline__ RowVecs(const typename E::storage *r, int v) : row(r), V(v) {
        off = static_cast<int>((reinterpret_cast<uintptr_t>(r) & 15) / sizeof(typename E::storage));
    }
    __device__ __forceinline__ int first(int j) const { return j * E::kPerVec - off; }
    __device__ __forceinline__ u32x4 load(int j) const {
        const int i0 = first(j);
        if (i0 >= 0 && i0 + E::kPerVec <= V)
            return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + i0));
        unsigned w[4] = {E::kNegInfWord, E::kNegInfWord, E::kNegInfWord, E::kNegInfWord};
        constexpr int kBits = 8 * sizeof(typename E::storage), kPerWord = 32 / kBits;
#pragma unroll
        for (int e = 0; e < E::kPerVec; ++e)
            if (i0 + e >= 0 && i0 + e < V) {
                const unsigned bits = storage_bits(row[i0 + e]);
                const int sh = (e % kPerWord) * kBits;
                if constexpr (kPerWord == 1)
                    w[e] = bits;
                else
                    w[e / kPerWord] = (w[e / kPerWord] & ~(0xffffu << sh)) | (bits << sh);
            }
        return u32x4{w[0], w[1], w[2], w[3]};
    }
};

__device__ __forceinline__ bool padding(const int32_t *__restrict__ tokens, long long row) {
    return tokens && uniform(tokens[row]) == -1;
}

template <typename E, int U>
__global__ __launch_bounds__(kBlock) void k_logprob(const typename E::storage *__restrict__ logits,
                                                    const int32_t *__restrict__ tokens, long long nwaves, int V,
                                                    int segs, float c, int k, LogprobPart *__restrict__ parts,
                                                    uint64_t *__restrict__ keys) {
    constexpr int P = E::kPerVec;
    __shared__ uint64_t lists[kWavesPerBlock][kListCap];
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x >> 6;
    const long long wave = static_cast<long long>(blockIdx.x) * kWavesPerBlock + w;
    if (wave >= nwaves) return;
    const long long row = wave / segs;
    const int seg = static_cast<int>(wave - row * segs);
    if (padding(tokens, row)) return;
    const RowVecs<E> rv(logits + row * V, V);
    const int j0 = seg * (U * kWave) + lane;
    const float ninf = -__builtin_huge_valf();
    u32x4 x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = rv.load(j0 + u * kWave);
    float vmax[U], m = ninf;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[P];
        unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
        float t = ninf;
#pragma unroll
        for (int e = 0; e < P; ++e) t = fmaxf(t, v[e]);
        vmax[u] = t;
        m = fmaxf(m, t);
    }
    const float lane_max = m;
    m = wave_max(m);
    double S = 0.0, Us = 0.0;
    if (m != ninf) {
        float s = 0.0f, t = 0.0f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[P], d[P];
            unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
#pragma unroll
            for (int e = 0; e < P; ++e) {
                const float dd = (v[e] - m) * c;
                v[e] = fast_exp2(dd);
                d[e] = v[e] * fmaxf(dd, -300.0f);  // 0 for a logit of -inf
            }
            s += pairwise_sum(v);
            t += pairwise_sum(d);
        }
        S = wave_sum(static_cast<double>(s));
        Us = wave_sum(static_cast<double>(t));
    }
    if (lane == 0) parts[wave] = LogprobPart{S, Us, m, 0.0f};
    if (k == 0) return;

    // a value that at least k logits of the segment reach
    float bar = ninf;
    {
        int rank = 0;
        for (int i = 0; i < kWave; ++i) {
            const float o = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lane_max), i));
            rank += o > lane_max || (o == lane_max && i < lane);
        }
        const uint64_t at = ballot(rank == k - 1);
        if (at) bar = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lane_max), first_lane(at)));
    }
    KeyList list;
    list.init(lists[w], k);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (ballot(vmax[u] >= bar) == 0) continue;
        float v[P];
        unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
        const int i0 = rv.first(j0 + u * kWave);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            const bool reach = v[e] >= bar;
            if (ballot(reach) == 0) continue;
            const int i = i0 + e;
            const uint64_t key = argmax_key(v[e], i);
            list.push(key, reach && i >= 0 && i < V && key > list.bar, lane);
        }
    }
    list.cut(lane);
    if (lane < k) keys[wave * k + lane] = lane < list.n ? list.buf[lane] : 0;
}

// The value a key was made from.
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

template <typename E>
__global__ __launch_bounds__(kBlock) void k_logprob_merge(
    const typename E::storage *__restrict__ logits, const int32_t *__restrict__ tokens, int R, int V, int segs,
    float c, int k, const LogprobPart *__restrict__ parts, const uint64_t *__restrict__ keys,
    float *__restrict__ logprob, float *__restrict__ entropy, int32_t *__restrict__ top_ids,
    float *__restrict__ top_logprobs, int32_t *__restrict__ status) {
    __shared__ uint64_t lists[kWavesPerBlock][kListCap];
    const int lane = threadIdx.x & (kWave - 1), w = threadIdx.x >> 6;
    const long long row = static_cast<long long>(blockIdx.x) * kWavesPerBlock + w;
    if (row >= R) return;
    const float ninf = -__builtin_huge_valf();
    const int tok = tokens ? uniform(tokens[row]) : -1;
    if (tokens && tok == -1) {
        if (lane == 0) {
            if (logprob) logprob[row] = 0.0f;
            if (entropy) entropy[row] = 0.0f;
            if (status) status[row] = 0;
        }
        if (lane < k) {
            top_ids[row * k + lane] = -1;
            top_logprobs[row * k + lane] = ninf;
        }
        return;
    }
    const LogprobPart *pp = parts + row * segs;
    float M = ninf;
    for (int s = lane; s < segs; s += kWave) M = fmaxf(M, pp[s].m);
    M = wave_max(M);
    // log2 of 2^(x c) relative to the row's maximum, from the stored value
    auto shifted = [&](float x) { return (static_cast<double>(x) - static_cast<double>(M)) * static_cast<double>(c); };
    double S = 0.0, Us = 0.0;
    if (M != ninf) {
        for (int s = lane; s < segs; s += kWave) {
            const LogprobPart p = pp[s];
            if (p.m == ninf) continue;
            const double g = shifted(p.m), f = exp2(g);
            S += p.S * f;
            Us += f * (p.U + p.S * g);
        }
        S = wave_sum(S);
        Us = wave_sum(Us);
    }
    const double L = log2(S);  // -inf where no logit is finite
    if (lane == 0) {
        const bool in = tok >= 0 && tok < V;
        if (logprob) {
            const float x = tokens && in ? to_f32(logits[row * V + tok]) : ninf;
            logprob[row] = x == ninf ? ninf : static_cast<float>(kLn2d * (shifted(x) - L));
        }
        if (entropy) entropy[row] = M == ninf ? 0.0f : static_cast<float>(kLn2d * (L - Us / S));
        if (status) status[row] = tokens && !in ? 1 : 0;
    }
    if (k == 0) return;
    // the segments' lists are sorted: the first keys of all lists raise the
    // bar at once, and the level at which no key passes it is the last
    KeyList list;
    list.init(lists[w], k);
    const uint64_t *kk = keys + row * segs * k;
    for (int i = 0; i < k; ++i) {
        bool any = false;
        for (int s0 = 0; s0 < segs; s0 += kWave) {
            const int s = s0 + lane;
            const uint64_t key = s < segs ? kk[static_cast<long long>(s) * k + i] : 0;
            const bool take = key > list.bar;
            any |= ballot(take) != 0;
            list.push(key, take, lane);
        }
        if (!any) break;
    }
    list.cut(lane);
    if (lane < k) {
        const uint64_t key = lane < list.n ? list.buf[lane] : 0;
        const float x = key_value(key);
        top_ids[row * k + lane] = key ? argmax_key_index(key) : -1;
        top_logprobs[row * k + lane] = key == 0 || x == ninf ? ninf : static_cast<float>(kLn2d * (shifted(x) - L));
    }
}

}  // namespace

// Vectors per lane of a segment: 16 (8192 bf16 logits) where the rows fill the
// card, 4 where they do not.
static int logprob_vecs(int rows, int V, sv_dtype dt) {
    const long long per = dt == SV_BF16 ? 8 : 4;
    const long long waves = static_cast<long long>(rows) * ((V / per + kWave * 16) / (kWave * 16));
    return waves >= 1024 ? 16 : 4;
}

int logprob_segs(int rows, int V, sv_dtype dt) {
    const int per = dt == SV_BF16 ? 8 : 4;
    // a row may start anywhere on the 16-byte grid: one element of a vector short of a whole vector more
    const int nvec = (V + per - 1 + per - 1) / per;
    const int wave = kWave * logprob_vecs(rows, V, dt);
    return (nvec + wave - 1) / wave;
}

namespace {
template <typename E, int U>
hipError_t launch_segments(const LogprobArgs &a, hipStream_t s) {
    const long long nwaves = static_cast<long long>(a.R) * a.segs;
    return launch_kernel(k_logprob<E, U>, dim3(static_cast<unsigned>((nwaves + kWavesPerBlock - 1) / kWavesPerBlock)),
                         dim3(kBlock), 0, s, static_cast<const typename E::storage *>(a.logits), a.tokens, nwaves,
                         a.V, a.segs, a.c, a.k, a.parts, a.keys);
}
template <typename E>
hipError_t launch_merge(const LogprobArgs &a, hipStream_t s) {
    return launch_kernel(k_logprob_merge<E>, dim3((a.R + kWavesPerBlock - 1) / kWavesPerBlock), dim3(kBlock), 0, s,
                         static_cast<const typename E::storage *>(a.logits), a.tokens, a.R, a.V, a.segs, a.c, a.k,
                         a.parts, a.keys, a.logprob, a.entropy, a.top_ids, a.top_logprobs, a.status);
}
}  // namespace

hipError_t launch_logprob(const LogprobArgs &a, sv_dtype dt, hipStream_t s) {
    const bool wide = logprob_vecs(a.R, a.V, dt) == 16;
    if (dt == SV_BF16) return wide ? launch_segments<BF16, 16>(a, s) : launch_segments<BF16, 4>(a, s);
    return wide ? launch_segments<F32, 16>(a, s) : launch_segments<F32, 4>(a, s);
}

hipError_t launch_logprob_merge(const LogprobArgs &a, sv_dtype dt, hipStream_t s) {
    return dt == SV_BF16 ? launch_merge<BF16>(a, s) : launch_merge<F32>(a, s);
}

}  // namespace sv
