// Internal structures of the beam step and of the reservation of cache rows.
// Not part of the public C ABI.
#pragma once

#include "sv_tree.h"

namespace sv {

constexpr int kMaxBeams = 64;

// ---- selection over beams and vocabulary ----
// What the first kernel leaves of a chunk of a logit row.
struct BeamChunk {
    double sum;    // of e^(x - top)
    float top;
    int32_t n;     // candidates listed; -1: the chunk holds a NaN or +inf
};
struct BeamParams {
    const uint8_t* logits;        // [B, W, V]
    int64_t sb, sw;               // strides in elements
    const float* scores;          // [B, W]
    const int32_t* finished;      // [B, W] or null
    int32_t *out_tokens, *out_ancestor, *out_finished;  // [B, W], [B * W], [B, W]
    float* out_scores;            // [B, W]
    int B, W, V, end;
    int runs;                     // 2048-id runs of a chunk: 1 or 4
    int chunks;                   // per row
    // workspace
    BeamChunk* rec;               // [B * W, chunks]
    uint64_t* list;               // [B * W, chunks, W]: order key << 32 | ~id
};
hipError_t launch_beam_stats(const BeamParams& p, int dtype, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_beam_select(const BeamParams& p, int dtype, hipStream_t st, const LaunchEvents& ev);

struct ReorderParams {
    const uint8_t* src;
    uint8_t* dst;
    const int32_t* ancestor;
    int64_t src_stride, dst_stride, bytes;  // of a row
    int rows;
};
hipError_t launch_reorder(const ReorderParams& p, hipStream_t st, const LaunchEvents& ev);

// ---- rows of a paged cache: their reservation and writing ----
struct ReserveParams {
    const int32_t *table, *len, *n_new;
    int64_t table_stride, out_stride;
    int32_t *out_table, *out_len, *start, *slots, *position, *status;
    int B, width, pages, ps_shift, rows;
    // workspace
    int32_t* plan;                // [B, kReserveWords], then the new pages
};
constexpr int kReserveWords = 8;  // old length, new length, entries kept, place of the new pages, first slot; spare
hipError_t launch_reserve_plan(const ReserveParams& p, hipStream_t st, const LaunchEvents& ev);
hipError_t launch_reserve_write(const ReserveParams& p, hipStream_t st, const LaunchEvents& ev);

struct WriteParams {
    uint8_t* cache;
    int64_t cs[2];                // page, slot, in 16-byte units
    const uint8_t *a, *b;         // [T, va vectors], [T, vb vectors] (null where vb is 0)
    int64_t as, bs;               // strides in 16-byte units
    const int32_t* slots;
    int T, va, vb, ps_shift;
    int64_t all;                  // slots of the cache
};
hipError_t launch_cache_write(const WriteParams& p, hipStream_t st, const LaunchEvents& ev);

}  // namespace sv
