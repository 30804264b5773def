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
// all loads issued before the first use), and leaves (m, S, U) and, where
// alternatives are asked for, the maxima of 64 groups of its logits.  A group is
// U consecutive 16-byte vectors (U = 16: 128 bf16 logits, two cache lines), so
// one that has to be looked into again is a contiguous read.
// k_logprob_merge: a workgroup per row joins its segments and finds the k best.
// Bound by the read of the logits; the exponentials (one per logit, at a
// quarter of the rate of other instructions) come close to it, so the first
// pass keeps to ten instructions per logit and selects nothing.  Measured at
// 2048 rows of 151936 bf16 logits with 20 alternatives: 107 to 117 us (5.9 to 5.3
// TB/s) and 14 to 16 us, at any temperature; selecting the segment's 20 best in the
// first pass took 281 us and 10 us, and a lane's own (strided) logits as the groups
// 106 us and 30 us.
//
// The k best: the k-th largest of 64 column maxima (a column: group l of every
// segment) is a value that at least k logits reach.  Only groups whose maximum
// reaches it can hold one of the k best: k + a few of them, which are read
// again.  What reaches the bar there is collected in LDS and ranked by counting,
// for each, how many are larger; keys are distinct (the index is part of them),
// so the result does not depend on the order in which they were collected.
// Where many logits tie (a masked vocabulary), each wave walks its segments in
// order and its list is cut back to the k best whenever it fills, which raises
// the bar to the k-th key so far, index included, and with it passes over the
// groups whose ties come later.
#include <algorithm>

#include "sv_paged.hpp"
#include "sv_paged_internal.hpp"

namespace sv {
namespace {

constexpr double kLn2d = 0.6931471805599453094172321214581766;
constexpr int kListCap = 128;  // keys a wave's list holds between cuts
constexpr int kGroupCap = 512;  // groups that are looked into at once

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
        // keys behind the list read as 0, below every key
        const int n8 = (n + 7) & ~7;
        if (lane < n8 - n) buf[n + lane] = 0;
        wave_lds_sync();
        int ra = 0, rb = 0;
        for (int i = 0; i < n8; i += 8) {
            uint64_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = buf[i + e];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ra += x[e] > a;
                rb += x[e] > b;
            }
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
    __device__ __forceinline__ u32x4 load_whole(int j) const {
        return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(row + first(j)));
    }
    __device__ __forceinline__ u32x4 load(int j) const {
        const int i0 = first(j);
        if (i0 >= 0 && i0 + E::kPerVec <= V) return load_whole(j);
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

// Keeps a register's value from being derived again from an earlier one.
__device__ __forceinline__ void opaque(u32x4 &x) { asm volatile("" : "+v"(x)); }

// |m| c below which d is formed in one step, as fma(x, c, -fp32(m c)), where
// (x - m) c takes two instructions.  All of a segment's exponents are then off by
// the rounding e of m c, at most 2^-11 here, which its sums take back by two terms
// of the series of 2^e (the third: e^3 / 18 < 2^-37).  The rounding grows with |m c|: at
// 2^24 it is half a step of the exponent itself, and a mask value of -1e10 would make
// a segment's weights 2^328.  Logits within +-2^14 T / log2(e), 11000 T, are below.
constexpr float kOneStep = 0x1p14f;

// Sums of 2^d and 2^d d over a lane's vectors, d in one step or as (x - m) c.
template <typename E, int U, bool ONE_STEP>
__device__ __forceinline__ void lane_sums(u32x4 (&x)[U], float m, float c, float &s, float &t) {
    constexpr int P = E::kPerVec;
    const float R = m * c;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[P], d[P];
        unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
#pragma unroll
        for (int e = 0; e < P; ++e) {
            d[e] = ONE_STEP ? fmaf(v[e], c, -R) : (v[e] - m) * c;
            v[e] = fast_exp2(d[e]);
            d[e] = fmaxf(d[e], -300.0f);  // 2^d d is 0 for a logit of -inf
        }
        // a vector's terms first, so that no addend meets a much longer sum
        float sp = v[0], tp = v[0] * d[0];
#pragma unroll
        for (int e = 1; e < P; ++e) {
            sp += v[e];
            tp = fmaf(v[e], d[e], tp);
        }
        s += sp;
        t += tp;
    }
}

// One step of the group maxima: lanes whose bit of `take` is set keep the odd
// values of pairs and give their partner (the DPP pattern CTRL) the even ones,
// the others the reverse; N values per lane become N / 2 over twice the lanes.
template <int CTRL, int N>
__device__ __forceinline__ void fold_max(float (&v)[N], bool odd) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const float keep = odd ? v[2 * i + 1] : v[2 * i], give = odd ? v[2 * i] : v[2 * i + 1];
        const float got = __int_as_float(
            __builtin_amdgcn_update_dpp(0, __float_as_int(give), CTRL, 0xf, 0xf, false));
        v[i] = fmaxf(keep, got);
    }
}
constexpr int kXor1 = 0xb1, kXor2 = 0x4e, kHalfMirror = 0x141, kMirror = 0x140;  // DPP lane patterns

// v[u]: the lane's maximum of its vector u.  Returns the maximum of the lane's
// group: vector group_vec<U>(lane) of each of the U lanes of lane / U.
__device__ __forceinline__ float group_max(float (&v)[16], int lane) {
    // mirror pairs lanes whose bits 3 differ, half mirror those whose bits 2
    // do, and the lanes met so far, x and its complement in the low 3 bits and
    // bit 3, are completed to 16 by x ^ 2 and x ^ 1
    fold_max<kMirror>(v, lane & 8);
    float a[8], b[4], c[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = v[i];
    fold_max<kHalfMirror>(a, lane & 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = a[i];
    fold_max<kXor2>(b, lane & 2);
    c[0] = b[0];
    c[1] = b[1];
    fold_max<kXor1>(c, lane & 1);
    return c[0];
}
__device__ __forceinline__ float group_max(float (&v)[4], int lane) {
    fold_max<kXor1>(v, lane & 1);
    float a[2] = {v[0], v[1]};
    fold_max<kXor2>(a, lane & 2);
    return a[0];
}
template <int U>
__device__ __forceinline__ int group_vec(int lane) {
    if constexpr (U == 16)
        return ((lane >> 3) & 1) | ((lane >> 1) & 2) | ((lane << 1) & 4) | ((lane << 3) & 8);
    else
        return lane & 3;
}
// First vector of group `lane` of a segment that starts at vector v0.
template <int U>
__device__ __forceinline__ int group_first(int v0, int lane) {
    return v0 + group_vec<U>(lane) * kWave + lane / U * U;
}

template <typename E, int U>
__global__ __launch_bounds__(kBlock, 4) void k_logprob(const typename E::storage *__restrict__ logits,
                                                       const int32_t *__restrict__ tokens, long long nwaves, int V,
                                                       int segs, float c, int k, LogprobPart *__restrict__ parts,
                                                       float *__restrict__ group_maxima) {
    constexpr int P = E::kPerVec;
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
    const int e0 = rv.first(seg * (U * kWave));  // the segment's first element
    if (e0 >= 0 && e0 + U * kWave * P <= V) {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = rv.load_whole(j0 + u * kWave);
    } else {
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = rv.load(j0 + u * kWave);
    }
    float m = ninf, vm[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float v[P];
        unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
        vm[u] = v[0];
#pragma unroll
        for (int e = 1; e < P; ++e) vm[u] = fmaxf(vm[u], v[e]);
        opaque(x[u]);  // the second pass widens the packed values anew: they need half the registers
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m = fmaxf(m, vm[u]);
    if (k) group_maxima[wave * kWave + lane] = group_max(vm, lane);
    m = wave_max(m);
    double S = 0.0, Us = 0.0;
    if (m != ninf) {
        float s = 0.0f, t = 0.0f;
        const bool one_step = fabsf(m) * c < kOneStep;
        if (one_step)
            lane_sums<E, U, true>(x, m, c, s, t);
        else
            lane_sums<E, U, false>(x, m, c, s, t);
        const double v = wave_sum_pair(static_cast<double>(s), static_cast<double>(t));
        // The maximum's own term, 2^0 and 0, is put in exactly: S is then at least 1, no
        // probability exceeds it, and a lone token has logprob 0.  In one step every d
        // is too small by e = -d0, so the other terms gain the factor
        // 2^e = 1 + e ln 2 (1 + e ln 2 / 2)
        const float R = m * c, d0 = one_step ? fmaf(m, c, -R) : 0.0f, own = fast_exp2(d0), own_d = own * d0;
        const double y = -static_cast<double>(d0) * kLn2d, f = 1.0 + y * (1.0 + 0.5 * y);
        const double rest = v - own;
        S = 1.0 + f * rest;
        Us = f * (__shfl(v, 32, kWave) - own_d - d0 * rest);
    } else {
        // nothing but -inf, or NaN, which the maximum passes over and the sums must not
        bool nan = false;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[P];
            unpack(make_uint4(x[u].x, x[u].y, x[u].z, x[u].w), v);
#pragma unroll
            for (int e = 0; e < P; ++e) nan |= v[e] != v[e];
        }
        if (ballot(nan) != 0) S = __builtin_nan("");
    }
    if (lane == 0) parts[wave] = LogprobPart{S, Us, m, 0.0f};
}

// The value a key was made from.
__device__ __forceinline__ float key_value(uint64_t key) {
    const uint32_t b = static_cast<uint32_t>(key >> 32);
    return __uint_as_float((b & 0x80000000u) ? b & 0x7fffffffu : ~b);
}

// A workgroup per row.  U: vectors per lane of a segment.
template <typename E, int U>
__global__ __launch_bounds__(kBlock) void k_logprob_merge(
    const typename E::storage *__restrict__ logits, const int32_t *__restrict__ tokens, int V, int segs, float c,
    int k, const LogprobPart *__restrict__ parts, const float *__restrict__ group_maxima, float *__restrict__ logprob,
    float *__restrict__ entropy, int32_t *__restrict__ top_ids, float *__restrict__ top_logprobs,
    int32_t *__restrict__ status) {
    constexpr int P = E::kPerVec;
    // segments per wave whose group maxima stay in registers, asked for together: few
    // rows have many segments and nothing but this latency (8 rows of 151936 fp32,
    // 38 a wave: 6.5 us against 10 with 6 held and the rest in rounds of 8)
    constexpr int kHeld = U == 4 ? 40 : 6;
    __shared__ __align__(16) uint64_t lists[kWavesPerBlock][kListCap];
    __shared__ float col[kWavesPerBlock][kWave];
    __shared__ float sM[kWavesPerBlock];
    __shared__ double sS[kWavesPerBlock], sU[kWavesPerBlock];
    __shared__ int left[kWavesPerBlock], reach[kGroupCap], ngroups, nkeys;
    const int lane = threadIdx.x & (kWave - 1), w = uniform(static_cast<int>(threadIdx.x >> 6));
    const long long row = blockIdx.x;
    const float ninf = -__builtin_huge_valf();
    // everything the row's own loads can start with is asked for at once
    const LogprobPart *pp = parts + row * segs;
    const float *gm = group_maxima + row * segs * kWave + lane;
    const int tok = tokens ? tokens[row] : 0;
    LogprobPart mine = {0.0, 0.0, ninf, 0.0f};
    if (threadIdx.x < segs) mine = pp[threadIdx.x];
    float held[kHeld];
    if (k) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            held[i] = gm[static_cast<long long>(min(w + i * kWavesPerBlock, segs - 1)) * kWave];
    }
    if (tokens && uniform(tok) == -1) {
        if (threadIdx.x == 0) {
            if (logprob) logprob[row] = 0.0f;
            if (entropy) entropy[row] = 0.0f;
            if (status) status[row] = 0;
        }
        if (threadIdx.x < k) {
            top_ids[row * k + threadIdx.x] = -1;
            top_logprobs[row * k + threadIdx.x] = ninf;
        }
        return;
    }
    const bool in = tokens && tok >= 0 && tok < V;
    const float xt = in ? to_f32(logits[row * V + tok]) : ninf;
    float M = mine.m;
    for (int s = threadIdx.x + kBlock; s < segs; s += kBlock) M = fmaxf(M, pp[s].m);
    float cm = ninf;
    if (k) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) cm = fmaxf(cm, held[i]);  // the last segment twice: no matter
#pragma unroll 8
        for (int s = w + kHeld * kWavesPerBlock; s < segs; s += kWavesPerBlock)
            cm = fmaxf(cm, gm[static_cast<long long>(s) * kWave]);
        col[w][lane] = cm;
    }
    M = wave_max(M);
    if (lane == 0) sM[w] = M;
    if (threadIdx.x == 0) ngroups = nkeys = 0;
    __syncthreads();
    M = fmaxf(fmaxf(sM[0], sM[1]), fmaxf(sM[2], sM[3]));
    // log2 of 2^(x c) relative to the row's maximum, from the stored value
    auto shifted = [&](float x) { return (static_cast<double>(x) - static_cast<double>(M)) * static_cast<double>(c); };
    KeyList list;
    list.init(lists[w], k);
    bool few = true;
    const RowVecs<E> rv(logits + row * V, V);
    float bar = ninf;
    if (k) {
        // the k-th largest column maximum: the least that fewer than k exceed
        cm = fmaxf(fmaxf(col[0][lane], col[1][lane]), fmaxf(col[2][lane], col[3][lane]));
        int above = 0;
#pragma unroll
        for (int i = 0; i < kWave; ++i) above += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(cm), i)) > cm;
        bar = -wave_max(above < k ? -cm : ninf);
        list.bar = argmax_key(bar, -1) & 0xffffffff00000000ull;  // below every key of a value >= bar
        // the groups that reach it, from all segments
        auto reaches = [&](float x, int s) {
            const uint64_t m = ballot(x >= bar);
            if (m == 0) return;
            int at = 0;
            if (lane == 0) at = atomicAdd(&ngroups, __popcll(m));
            at = uniform(at) + __popcll(m & ((1ull << lane) - 1));
            if (x >= bar && at < kGroupCap) reach[at] = s * kWave + lane;
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const int s = w + i * kWavesPerBlock;
            if (s < segs) reaches(held[i], s);
        }
        for (int s0 = w + kHeld * kWavesPerBlock; s0 < segs; s0 += 8 * kWavesPerBlock) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = s0 + i * kWavesPerBlock;
                x[i] = s < segs ? gm[static_cast<long long>(s) * kWave] : ninf;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int s = s0 + i * kWavesPerBlock;
                if (s < segs) reaches(x[i], s);
            }
        }
        __syncthreads();
        const int ng = ngroups;
        few = ng <= kGroupCap;
        if (few) {
            // their vectors spread over the workgroup; what reaches the bar goes to one list
            for (int i0 = 0; i0 < ng * U; i0 += 2 * kBlock) {
                u32x4 x[2];
                int j[2];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = i0 + h * kBlock + threadIdx.x;
                    j[h] = -1;
                    if (i < ng * U) {
                        const int from = reach[i / U];
                        j[h] = group_first<U>(from / kWave * (U * kWave), from % kWave) + i % U;
                        x[h] = rv.load(j[h]);
                    }
                }
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (j[h] < 0) continue;
                    float v[P];
                    unpack(make_uint4(x[h].x, x[h].y, x[h].z, x[h].w), v);
                    const int first = rv.first(j[h]);
#pragma unroll
                    for (int e = 0; e < P; ++e)
                        if (v[e] >= bar && first + e >= 0 && first + e < V) {
                            const int at = atomicAdd(&nkeys, 1);
                            if (at < kListCap) lists[0][at] = argmax_key(v[e], first + e);
                        }
                }
            }
        }
    }
    // the sums, while the groups' logits are on their way
    double S = 0.0, Us = 0.0;
    for (int s = threadIdx.x; s < segs; s += kBlock) {
        if (s >= kBlock) mine = pp[s];
        if (mine.m == ninf) {
            S += mine.S;  // 0, or NaN where the segment holds one
            continue;
        }
        // the factor in fp32: off by 2^-22 (1 + |g|) of a share 2^g of the sum
        const double g = shifted(mine.m), f = fast_exp2(static_cast<float>(g));
        S += mine.S * f;
        Us += f * (mine.U + mine.S * g);
    }
    {
        const double v = wave_sum_pair(S, Us);
        if (lane == 0) sS[w] = v;
        if (lane == 32) sU[w] = v;
    }
    __syncthreads();
    if (k) {
        few = few && nkeys <= kListCap;
        if (few) {
            list.n = nkeys;
        } else {
            // many ties at the bar: each wave walks its segments in order and cuts its list as it fills
            for (int s0 = w; s0 < segs; s0 += kWavesPerBlock) {
                const float mx = gm[static_cast<long long>(s0) * kWave];
                const int j0 = group_first<U>(s0 * (U * kWave), lane);
                // no key of this group is above that of its maximum at its first place
                const uint64_t best = argmax_key(mx, max(rv.first(j0), 0));
                uint64_t todo = ballot(best > list.bar);
                while (todo) {
                    // the next groups' vectors spread over the wave
                    constexpr int kAtOnce = kWave / U;
                    int from = -1;
#pragma unroll
                    for (int i = 0; i < kAtOnce; ++i)
                        if (todo) {
                            if (lane / U == i) from = first_lane(todo);
                            todo &= todo - 1;
                        }
                    const int j = group_first<U>(s0 * (U * kWave), max(from, 0)) + lane % U;
                    u32x4 x = {};
                    if (from >= 0) x = rv.load(j);
                    float v[P];
                    unpack(make_uint4(x.x, x.y, x.z, x.w), v);
                    const int first = rv.first(j);
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const int i = first + e;
                        const uint64_t key = argmax_key(v[e], i);
                        list.push(key, from >= 0 && i >= 0 && i < V && v[e] == v[e] && key > list.bar, lane);
                    }
                    todo &= ballot(best > list.bar);
                }
            }
            list.cut(lane);
            if (lane == 0) left[w] = list.n;
            __syncthreads();
        }
    }
    if (w != 0) return;
    S = sS[0] + sS[1] + sS[2] + sS[3];
    Us = sU[0] + sU[1] + sU[2] + sU[3];
    const double L = log2(S);
    const bool nan = S != S;  // the row holds a NaN, or +inf, whose 2^d is 2^(inf - inf)
    auto log_prob = [&](float x) { return x == ninf ? ninf : static_cast<float>(kLn2d * (shifted(x) - L)); };
    if (lane == 0) {
        if (logprob) logprob[row] = nan && in ? static_cast<float>(S) : log_prob(xt);
        const double h = L - Us / S;  // below 0 only by rounding
        if (entropy) entropy[row] = (M == ninf && !nan) || h < 0.0 ? 0.0f : static_cast<float>(kLn2d * h);
        if (status) status[row] = tokens && !in ? 1 : 0;
    }
    if (k == 0) return;
    for (int i = few ? kWavesPerBlock : 1; i < kWavesPerBlock; ++i) {
        const uint64_t key = lane < left[i] ? lists[i][lane] : 0;
        list.push(key, key > list.bar, lane);
    }
    list.cut(lane);
    if (lane < k) {
        const uint64_t key = lane < list.n ? list.buf[lane] : 0;
        const float x = key_value(key);
        top_ids[row * k + lane] = key ? argmax_key_index(key) : -1;
        top_logprobs[row * k + lane] = key == 0 ? ninf : (nan ? static_cast<float>(S) : log_prob(x));
    }
}

}  // namespace

// Vectors per lane of a segment: 16 (8192 bf16 logits) where the rows fill the
// card (8 take 112 us where 16 take 106: a segment's reductions cost the same),
// 4 where they do not (8 rows of 151936 fp32: 4.2 us against 6.9).
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
                         a.V, a.segs, a.c, a.k, a.parts, a.group_maxima);
}
template <typename E, int U>
hipError_t launch_merge(const LogprobArgs &a, hipStream_t s) {
    return launch_kernel(k_logprob_merge<E, U>, dim3(static_cast<unsigned>(a.R)), dim3(kBlock), 0, s,
                         static_cast<const typename E::storage *>(a.logits), a.tokens, a.V, a.segs, a.c, a.k,
                         a.parts, a.group_maxima, a.logprob, a.entropy, a.top_ids, a.top_logprobs, a.status);
}
}  // namespace

hipError_t launch_logprob(const LogprobArgs &a, sv_dtype dt, hipStream_t s) {
    const bool wide = logprob_vecs(a.R, a.V, dt) == 16;
    if (dt == SV_BF16) return wide ? launch_segments<BF16, 16>(a, s) : launch_segments<BF16, 4>(a, s);
    return wide ? launch_segments<F32, 16>(a, s) : launch_segments<F32, 4>(a, s);
}

hipError_t launch_logprob_merge(const LogprobArgs &a, sv_dtype dt, hipStream_t s) {
    const bool wide = logprob_vecs(a.R, a.V, dt) == 16;
    if (dt == SV_BF16) return wide ? launch_merge<BF16, 16>(a, s) : launch_merge<BF16, 4>(a, s);
    return wide ? launch_merge<F32, 16>(a, s) : launch_merge<F32, 4>(a, s);
}

}  // namespace sv
