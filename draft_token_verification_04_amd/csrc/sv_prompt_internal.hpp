// sv_prompt_internal.hpp -- arguments, workspace plans and launchers of the
// prompt operators (norm, e4m3 projection, attention of packed sequences),
// shared by the C-ABI entry points and the kernel translation units.
#pragma once

#include "sv_paged_internal.hpp"

namespace sv {

constexpr int kScaleBlock = 128;  // columns (and weight rows) that share a scale

struct NormArgs {
    const uint16_t *x;         // bf16, row t at t * x_stride
    long long x_stride;
    const uint16_t *residual;  // bf16 [T][D] or null
    const uint16_t *weight;    // bf16 [D] or null
    float eps;
    int T, D;
    uint16_t *residual_out;    // bf16 [T][D] or null
    void *out;                 // bf16 or e4m3 [T][D]
    float *out_scale;          // [blocks of D][T] (e4m3)
};
hipError_t launch_rms_norm(const NormArgs &a, bool e4m3, hipStream_t s);

struct LinearArgs {
    const uint8_t *x;  // e4m3, row m at m * x_stride
    long long x_stride;
    const float *x_scale;  // block kb of row m at kb * x_scale_stride + m
    long long x_scale_stride;
    const uint8_t *w;      // e4m3 [N][K]
    const float *w_scale;  // [blocks of N][blocks of K]
    int M, N, K;
    void *out;             // bf16 or fp32 [M][N]
    float *part;           // [splits][M][N] (splits > 1)
    int splits;
};
struct LinearPlan {
    int kind;      // which kernel (see sv_linear.hip)
    int splits;    // parts of K, joined by a second launch
    long long groups;  // of 256 work items
    size_t total;  // workspace
};
LinearPlan linear_plan(int M, int N, int K, bool f32);
hipError_t launch_linear(const LinearArgs &a, const LinearPlan &p, bool f32, hipStream_t s);
hipError_t launch_linear_join(const LinearArgs &a, bool f32, hipStream_t s);

struct PackedArgs {
    const uint16_t *q;  // bf16, token t at t * q_stride
    long long q_stride;
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *starts, *base;  // base may be null: no cached tokens
    int T, B, H, Hkv, G, P, page_shift, num_pages;
    float c;            // scale * log2(e)
    float unit;         // log2(e) in the units of the scores that a row's reference is held in
    uint16_t *out;      // [T][H][D]
    float *lse;         // [T][H] or null
    int32_t *status;    // [B] or null
    int S, units;       // splits, row tiles (of all requests, at most)
    float *part_o, *part_ml;  // [units][Hkv][S][rows] x D, x 2
    int32_t *part_bad;        // [units][Hkv][S]
};
struct PackedPlan {
    int rows;           // rows of a workgroup, two work items each
    int units, S;
    size_t part_o, part_ml, part_bad, total;
};
PackedPlan packed_plan(int T, int B, int H, int Hkv, int D, int P, int page_size, bool e4m3);
long long packed_groups(int Hkv, const PackedPlan &p);  // workgroups of the launches
long long packed_join_groups(int Hkv, int D, const PackedPlan &p);
hipError_t launch_attend_packed(const PackedArgs &a, int D, bool e4m3, const PackedPlan &p, hipStream_t s);
hipError_t launch_attend_packed_join(const PackedArgs &a, int D, const PackedPlan &p, hipStream_t s);

}  // namespace sv
