// sv_paged_internal.hpp -- arguments, workspace plans and launchers of the
// paged-cache and log-probability kernels, shared by the C-ABI entry points and
// the kernel translation units.
#pragma once

#include "sv_internal.hpp"

namespace sv {

// Smallest row maximum an e4m3 scale is formed from: the scale (maximum / 448)
// and its inverse are then normal floats.
constexpr float kMinAmax = 448.0f * 0x1p-126f;

// Most workgroups of a launch along x: fewer than 2^32 work items.
constexpr long long kMaxGroups = (1LL << 32) / 256 - 1;

struct AppendArgs {
    const uint16_t *q, *k, *v;              // bf16 rows of token t at t * stride
    long long q_stride, k_stride, v_stride;
    const uint16_t *q_weight, *k_weight;    // [D] or null
    float eps;
    const float *rope;                      // [max_pos][rot]: cosines, then sines; or null
    int rot, max_pos, interleaved;
    const int32_t *positions, *base, *counts, *page_table;
    int N, H, Hkv, P, page_shift, num_pages;
    uint16_t *q_out;
    void *k_pages, *v_pages;
    float *k_scale, *v_scale;
    int32_t *status;
};
hipError_t launch_append(const AppendArgs &a, int D, bool e4m3, int tokens, hipStream_t s);

// (m, S, U) of a segment of a row: m its maximum, d = (x - m) c, S = sum 2^d, U = sum 2^d d.
struct LogprobPart {
    double S, U;
    float m, pad;
};
struct LogprobArgs {
    const void *logits;
    const int32_t *tokens;
    int R, V, segs, k;
    float c;
    LogprobPart *parts;  // [R][segs]
    float *group_maxima;     // [R][segs][64] (k > 0)
    float *logprob, *entropy;
    int32_t *top_ids;
    float *top_logprobs;
    int32_t *status;
};
int logprob_segs(int rows, int V, sv_dtype dt);
hipError_t launch_logprob(const LogprobArgs &a, sv_dtype dt, hipStream_t s);
hipError_t launch_logprob_merge(const LogprobArgs &a, sv_dtype dt, hipStream_t s);

// Moves the accepted path's rows inside the pages: G arrays of pages
// [num_pages][Hkv][page_size] rows of `vecs` (a power of two) 16-byte vectors,
// and as many of one float per row (scales, may be null).
long long commit_paged_groups(int G, int B, int Hkv);  // workgroups of the launch
hipError_t launch_commit_paged(void *pages, float *scales, int G, int B, int Hkv, int num_pages, int page_shift,
                               int vecs, const int32_t *page_table, int P, const int32_t *tree_base,
                               const int32_t *commit_base, const int32_t *accept_len, const int32_t *path_nodes,
                               int N, int32_t *status, hipStream_t s);

struct AttendArgs {
    const uint16_t *q;       // bf16, token t at t * q_stride
    long long q_stride;
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *base, *counts, *parents;
    int B, N, H, Hkv, G, P, page_shift, num_pages;
    float c, scale;          // c = scale * log2(e)
    uint16_t *out;           // [B][N][H][D]
    float *lse;              // [B][N][H] or null
    int32_t *status;         // [B] or null
    int S, QB, min_tiles;    // splits, row blocks, least tiles per wave
    bool falling;            // splits of falling size
    float *part_o, *part_ml; // [B][Hkv][QB][S][rows] x D, x 2
    int32_t *part_bad;       // [B][Hkv][QB][S]
};
struct AttendPlan {
    int QT, QB, S, min_tiles;         // 16-row tiles per wave, row blocks, splits, least tiles per wave
    bool shares;                      // the waves of a workgroup divide its rows, not its slots
    bool falling;                     // splits of falling size
    int group_rows;                   // rows of a workgroup
    size_t part_o, part_ml, part_bad, total;  // workspace
};
AttendPlan attend_plan(int B, int N, int H, int Hkv, int D, int P, int page_size);
hipError_t launch_attend(const AttendArgs &a, int D, bool e4m3, const AttendPlan &p, hipStream_t s);
hipError_t launch_attend_join(const AttendArgs &a, int D, const AttendPlan &p, hipStream_t s);
long long attend_groups(int B, int Hkv, const AttendPlan &p);  // workgroups of the first launch

}  // namespace sv
