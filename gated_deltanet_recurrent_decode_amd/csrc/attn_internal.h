// attn_internal.h -- parameter blocks and launchers of the paged-attention kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdn {

struct Heads {
    uint16_t *p; // null: absent
    int64_t row, head;
};

struct AttnPrologueParams {
    Heads q, k, v, q_out;
    void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *kv_len, *row, *cu, *positions;
    const double *freqs;
    const uint16_t *q_w, *k_w;
    float eps, add, rope_scale;
    int rot, interleaved;
    int B, T, R, H_q, H_kv, N, page_shift, width;
};

struct AttnParams {
    Heads q, out;
    float *lse;                 // [T][H_q] or null
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *page_table, *kv_len, *row, *cu;
    float *part_o;              // partial outputs [workgroups][2][rows of a tile][d]
    float *part_ml;             // their running maximum and sum [workgroups][2][rows of a tile][2]
    int32_t *cut;               // [workgroups][8] what of the workgroup's piece goes on in the next, see Cut
    float scale;                // in the exponent of 2
    int B, T, R, H_q, H_kv, G, N, page_shift, width, max_new, window;
    int workgroups;
    long long *before;          // tiles: units of the call before each entry, and the sum of all
    int32_t *entry;             // tiles: [entries][8] kv head, tile, the sequence
    int32_t *count;             // tiles: entries, and from [2] on their units in 64 bits
    int capacity;               // tiles: entries that the workspace holds
    int block;                  // tiles: keys of a block
    // a batch that shares prefixes
    const int32_t *cu_groups, *shared_len; // [K + 1], [K]
    int K;
    int least;                  // keys from which a group is taken together; -1: by the plan's rule
    int tile_rows;              // rows of a tile
    int pad;                    // units that an entry counts more than its blocks
    int own_blocks;             // 32-row blocks of a part of a sequence's own keys
    int64_t shared_parts;       // where the parts of shared keys begin, in 32-row blocks
};

struct PageParams {
    int32_t *table, *kv_len, *refs;
    int R, width, N, page_shift;
    uint8_t *k, *v;
    int layers;
    int64_t layer_stride, page_bytes;
    const int32_t *a, *b;       // the call's lists: rows and adds, sources and destinations
    int n;
    int32_t *result, *remap;
    int32_t *owner;             // workspace [R]: first list entry that names the row
    int32_t *plan;              // workspace [4 n + 2 N + 4], see kv_pages.hip
};

hipError_t launch_attn_prologue(const AttnPrologueParams &p, int d, bool e4m3, hipStream_t stream);
// device scratch in bytes; fills the parameter block's pointers when it is given
inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }
size_t attn_paged_layout(int B, int T, int max_new, int H_kv, int G, int d, void *base, AttnParams *p);
// whether attn_paged takes its 16-row tiles
bool attn_few_rows(int max_new, int G);
size_t attn_rows_layout(int d, void *base, AttnParams *p);
size_t attn_tiles_layout(int B, int T, int H_kv, int G, int d, void *base, AttnParams *p);
hipError_t launch_attn_rows(const AttnParams &p, int d, bool e4m3, hipStream_t stream);
hipError_t launch_attn_tiles(const AttnParams &p, int d, bool e4m3, hipStream_t stream);
size_t attn_shared_layout(int B, int T, int K, int max_new, int H_kv, int G, int d, void *base, AttnParams *p);
// the tiles of a plan with shared entries (attn_tiles.hip), and the whole call
hipError_t launch_attn_tiles_shared(const AttnParams &p, int d, bool e4m3, hipStream_t stream);
hipError_t launch_attn_shared(const AttnParams &p, int d, bool e4m3, hipStream_t stream);
hipError_t launch_attn_paged(const AttnParams &p, int d, bool e4m3, hipStream_t stream);
hipError_t launch_kv_reserve(const PageParams &p, hipStream_t stream);
hipError_t launch_kv_fork(const PageParams &p, hipStream_t stream);
hipError_t launch_kv_free(const PageParams &p, hipStream_t stream);
hipError_t launch_kv_copy(const PageParams &p, hipStream_t stream);
hipError_t launch_kv_compact(const PageParams &p, hipStream_t stream);

} // namespace gdn
