// Internal structures of the kernels for models with one latent row per token:
// attention on the rows themselves, products per head, attention of prompts
// with expanded keys and values.  Not part of the public C ABI.
#pragma once

#include "sv_tree.h"

namespace sv {

// ---- attention on latent rows ----
struct LatentParams {
    const uint8_t *q, *nw, *kc;            // queries, the nodes' own rows, cache rows
    uint8_t* out;
    uint32_t qs[3], os[3];                 // strides in 16-byte units: sequence, node, head
    uint32_t nws[2], kcs[2];               // sequence, node; page, slot
    const int32_t *table, *len, *parent, *n_nodes;  // parent null: chains; n_nodes may be null
    int64_t table_stride;
    int B, N, H, C, dv;
    int pages, width, ps_shift;            // page size 1 << ps_shift
    float scale2;                          // |scale| log2(e), a normal number
    int flip;                              // scale < 0: the queries' signs are flipped
    int MT;                                // row tiles per sequence
    int clusters;                          // parts the work is cut into
    int merge;                             // 0: every sequence is one part
    int64_t* start;                        // [B + 1] workspace: first tile of each sequence
    float* part;                           // [clusters, 2, MT, rows, dv template + 2] workspace: partial results
};

// Rows of a workgroup's tile, and the kernel's row and value widths.
struct LatentShape {
    int rows;  // 32 or 64
    int wide;  // 1: rows up to 576 and values up to 512 elements; 0: 320 and 256
};
constexpr int latent_dv(int wide) { return wide ? 512 : 256; }

hipError_t launch_latent_attn(const LatentParams& p, const LatentShape& s, int dtype, hipStream_t st,
                              const LaunchEvents& ev);
hipError_t launch_latent_join(const LatentParams& p, const LatentShape& s, int dtype, hipStream_t st,
                              const LaunchEvents& ev);

// ---- products per head ----
struct ProductParams {
    const uint8_t *x, *w;          // [T, H, K], [H, M, K]
    uint8_t* out;                  // [T, H, M]
    int64_t xs[2], ws[2], os[2];   // strides in 16-byte units: token, head; head, row; token, head
    int T, H, M, K;
    int tt;                        // tokens of a workgroup's tile
};
hipError_t launch_product(const ProductParams& p, int dtype, hipStream_t st, const LaunchEvents& ev);

// ---- attention of prompts ----
struct PromptParams {
    const uint8_t *q, *kc, *wk, *wv;  // [T, H, dn + dr], cache rows, [H, dn, R], [H, dv, R]
    uint8_t* out;                     // [T, H, dv]
    int64_t qs[2], os[2];             // strides in 16-byte units: token, head
    int64_t kcs[2];                   // page, slot
    int64_t wks[2], wvs[2];           // head, row
    const int32_t *table, *len, *q_start;
    int64_t table_stride;
    int T, B, H, dn, dr, dv, R;
    int rows;                         // of the line: all sequences' rows one after the other
    int pages, width, ps_shift;
    float scale2;
    int flip;
    int cus;                          // of the device
    // workspace
    int64_t* plan;                    // [B + 1] first row of the line, [B + 1] first query tile
    int32_t* odd;                     // bit 0: an infinity or NaN among the values; 1: a row whose page does not exist;
                                      // 2: a row whose values have a power of two of their own
    int16_t* sizes;                   // [H, kSizeParts, rows] exponent of the largest value in a part of a row
    int16_t* power;                   // [H, rows] the row's power of two
    int32_t* there;                   // [rows rounded up] 1: the row's page exists
    uint8_t *k, *v, *pe;              // [H, rows, dn], [H, rows, dv], [rows, dr]
    int part;                         // outputs of a part: those a wave of the expansion has, 64 or 128
};
constexpr int kSizeParts = 3;         // a head's values lie in that many parts at most
constexpr int kPromptRows = 128;      // queries of a tile
hipError_t launch_prompt_plan(const PromptParams& p, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_prompt_expand(const PromptParams& p, int dtype, bool again, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_prompt_attn(const PromptParams& p, int dtype, hipStream_t st, const LaunchEvents& ev);

}  // namespace sv
