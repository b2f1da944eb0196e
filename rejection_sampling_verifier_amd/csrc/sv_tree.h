// Internal structures of the tree round's kernels: attention of drafted trees
// over a paged cache, verification of trees from given random numbers, and
// the commit and fork of cache pages.  Not part of the public C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "sv_internal.h"

namespace sv {

constexpr int kMaxNodes = 64;        // nodes of a tree: one bit each of a 64-bit ancestor set
constexpr int kMaxPages = 1 << 20;   // of a cache whose tables are changed: one bit each in LDS
constexpr int kDTypeF16 = 2;         // after DT_F32 and DT_BF16

// Kernel kinds of the timing interface, after the verify step's.
enum TreeKernelKind : int {
    KK_TREE_ATTN = KK_COUNT,
    KK_TREE_MERGE,
    KK_VERIFY_CLEAR,
    KK_TREE_VERIFY,
    KK_CACHE_PLAN,
    KK_CACHE_COPY,
    KK_LATENT_ATTN,
    KK_LATENT_JOIN,
    KK_PRODUCT,
    KK_PROMPT_PLAN,
    KK_PROMPT_EXPAND,
    KK_PROMPT_SCALE,
    KK_PROMPT_ATTN,
    KK_BEAM_STATS,
    KK_BEAM_SELECT,
    KK_BEAM_REORDER,
    KK_RESERVE_PLAN,
    KK_RESERVE_WRITE,
    KK_CACHE_WRITE,
    KK_ALL
};

// ---- attention ----
struct TreeAttnParams {
    const uint8_t *q, *kt, *vt, *kc, *vc;  // queries, tree K/V, cache K/V
    uint8_t* out;
    uint32_t qs[3], os[3];                 // strides in 16-byte units: sequence, node, head
    uint32_t kts[3], vts[3];
    uint32_t kcs[3], vcs[3];               // page, slot, head
    const int32_t *table, *len, *parent, *n_nodes;  // n_nodes may be null
    int64_t table_stride;
    int B, N, Hkv, G, D;                   // G = query heads per key head
    int pages, width, ps_shift;            // page size 1 << ps_shift
    int window, sinks;
    float scale2;                          // |scale| log2(e), a normal number
    int flip;                              // scale < 0: the queries' signs are flipped
    int MT;                                // row tiles per (sequence, key head)
    int clusters;                          // parts the work is cut into
    int merge;                             // 0: every (sequence, key head) is one part
    int64_t* start;                        // [B + 1] workspace: first tile of each sequence, over the key heads
    float* part;                           // [clusters, 2, MT, rows, D32 + 2] workspace: partial results
};

// What a workgroup of four waves takes at a time, by the N * G query rows that
// share a key head.  A wave always has 32 rows: up to 32 rows, the waves take a
// quarter of 128 keys each; up to 64, two waves over rows and two over 64 keys;
// else four waves over 128 rows, all on the same 64 keys.
struct TreeAttnShape {
    int rows;  // 32, 64 or 128
    int keys;
    int dp;    // head dimension rounded up to 64 or 128
};

hipError_t launch_tree_attn(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                            const LaunchEvents& ev);
hipError_t launch_tree_merge(const TreeAttnParams& p, const TreeAttnShape& s, int dtype, hipStream_t st,
                             const LaunchEvents& ev);

// ---- verification ----
struct TreeVerifyParams {
    const uint8_t *tgt, *dft;     // probabilities [B, N, V], [B, P, V] (dft may be null)
    int64_t tsb, tsp, dsb, dsp;   // strides in elements
    const int32_t *tokens, *parent, *n_nodes;  // [B, N], [B, N], [B] or null
    const float *u_accept, *u_final;           // [B, N], [B]
    int32_t *out_tokens, *out_nodes, *out_n;   // [B, N], [B, N], [B]
    int B, N, P, V;
    int team;                     // workgroups per sequence
    int passes;                   // passes over rows a sequence may need: N + 2
    int looks;                    // times a workgroup looks for another's sum (about a microsecond each)
    uint64_t* rec;                // [B, passes, team * 16] workspace: the ranges' sums (team > 1)
};
constexpr int kMaxTeam = 16;
constexpr int kVerifyWaves = 16;  // waves of a workgroup, ranges of a row per workgroup
hipError_t launch_verify_clear(const TreeVerifyParams& p, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_tree_verify(const TreeVerifyParams& p, int dtype, hipStream_t st, const LaunchEvents& ev);

// ---- cache pages ----
struct CacheParams {
    uint8_t *k, *v;               // [layers, pages, page size, heads, dim]
    int64_t ks[4], vs[4];         // strides in 16-byte units: layer, page, slot, head
    const uint8_t *kt, *vt;       // commit: [layers, B, N, heads, dim]
    int64_t kts[4], vts[4];       // layer, sequence, node, head (16-byte units)
    int layers, pages, ps_shift, heads, vec;  // vec: 16-byte vectors per (row, head)
    const int32_t *table, *len;
    int32_t *out_table, *out_len, *status;
    int64_t table_stride, out_stride;
    int B, N, width;
    const int32_t *nodes, *n_accepted;  // commit
    const int32_t* ancestor;            // fork
    int fork;
    // workspace: what the plan decides and the copies carry out
    int32_t* plan;                // [B, kPlanWords], [kPlanSpare, B], the new pages
};
constexpr int kPlanWords = 4;     // old length, new length, pages kept, place of the new pages
constexpr int kPlanSpare = 4;     // words per sequence the plan itself uses for large batches
hipError_t launch_cache_plan(const CacheParams& p, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_cache_copy(const CacheParams& p, hipStream_t st, const LaunchEvents& ev);

}  // namespace sv
