// Kernel argument blocks and launchers shared between the .cu files.
#pragma once

#include "common.cuh"

namespace pdattn {

// Layers one multi-layer decode launch serves (its per-layer pointers and
// tensor maps travel as kernel parameters).
constexpr int kMaxLayers = 32;

// Parameter block of the single-layer launches: nothing per layer.
struct NoLayers {};

// Per-layer inputs of a multi-layer prep launch.  Row v of the launch is row
// v % layer_rows of layer v / layer_rows.
struct PrepLayers {
    const void* q[kMaxLayers];
    const void* k_new[kMaxLayers];
    const void* v_new[kMaxLayers];
    void* k_pool[kMaxLayers];
    void* v_pool[kMaxLayers];
    int window[kMaxLayers];
};

// Per-layer pools (as TMA maps), outputs and sinks of a multi-layer
// attention launch.
struct AttendLayers {
    CUtensorMap k[kMaxLayers];
    CUtensorMap v[kMaxLayers];
    void* out[kMaxLayers];
    const void* sinks[kMaxLayers];
    int window[kMaxLayers];
};

struct PrepArgs {
    int rows, heads, kv_heads, head_dim, pages_per_row, num_pages, window;
    int max_pos;            // rows at this position or past it are skipped
    int layer_rows;         // multi-layer launches: rows per layer (rows = layers x layer_rows)
    const void* q;
    const void* k_new;
    const void* v_new;
    const int* positions;
    const int* table;
    const void* rope_cos;   // nullptr: copy without rotation
    const void* rope_sin;
    void* q_out;
    void* k_pool;
    void* v_pool;
    int rope_blocks;        // rows to rotate and write (0: none)
    int do_plan;            // 1: a planner launch builds the split plan first
    int grid_attend;        // persistent CTAs of the attention launch
    int chunk_pages;        // 0: planner's choice
    char* ws;
    WsLayout L;
};

struct AttendArgs {
    int rows, heads, kv_heads, group, head_dim, pages_per_row, num_pages;
    int layer_rows, n_layers;   // multi-layer launches: rows per layer, layers
    int window, chunk_pages;    // as given to the planner (first-wave items are derived from them)
    float scale_log2;       // score scale times log2(e)
    const void* q;          // rotated queries [rows, heads, D]
    const int* positions;   // [rows] (per layer in a multi-layer launch)
    const int* table;
    const void* sinks;      // nullptr, or [heads] of T
    void* out;
    char* ws;
    WsLayout L;
    const float* k_scale;   // coded cache: [num_pages, kv_heads, 64]; q then holds code_kernel's rows
    const float* v_scale;
    int max_pos;            // rows at this position or past it are skipped, as the planner does
};

// Groups of rows whose tables begin with the same pages: rows [start[i],
// start[i + 1]) share their first pages[i] pages.
struct SharedScan {
    int n_groups, rows, kv_heads, tile_tokens, pages_per_row, window, max_pos;
    const int* start;       // [n_groups + 1]
    const int* pages;       // [n_groups]
    const int* positions;
};

// Workspace of a decode over shared prefixes.  Pieces of the shared pages need
// at most tile_tokens partial slots per CTA and 2 per (row, kv head) and one
// per group (csrc/shared.cuh: the units are at most `share` per CTA); the own
// pages two per run, and one per (row, kv head) that no run cuts.
constexpr int kSharedRuns = 8;           // runs of own pages per CTA, at most (a long one and up to 6 short ones)

struct ShLayout {
    WsLayout w;             // ctrl, row_info, part_ml and part_o (own pages), q_rot
    size_t row_pre, pairs, pre_ml, pre_o, total;
    long long pre_slots, own_slots;
};

inline ShLayout shared_layout(int rows, int heads, int kv_heads, int head_dim, int n_groups, int grid) {
    ShLayout S = {};
    WsLayout& L = S.w;
    const int g = heads / kv_heads, tile_tokens = 2 * (kPfRows / g);
    S.pre_slots = (long long)tile_tokens * grid + 2ll * rows * kv_heads + n_groups;
    S.own_slots = 2ll * kSharedRuns * grid + (long long)rows * kv_heads;
    size_t off = 0;
    L.ctrl = off; off += 256;
    L.row_info = off; off = align256(off + sizeof(int4) * (size_t)rows);
    L.part_ml = off; off = align256(off + sizeof(float2) * (size_t)S.own_slots * g);
    L.part_o = off; off = align256(off + sizeof(float) * (size_t)S.own_slots * g * head_dim);
    L.q_rot = off; off = align256(off + (size_t)2 * rows * heads * head_dim);
    S.row_pre = off; off = align256(off + sizeof(int4) * (size_t)rows);
    S.pairs = off; off = align256(off + sizeof(int2) * (size_t)rows * kv_heads);
    S.pre_ml = off; off = align256(off + sizeof(float2) * (size_t)S.pre_slots * g);
    S.pre_o = off; off = align256(off + sizeof(float) * (size_t)S.pre_slots * g * head_dim);
    L.total = S.total = off;
    return S;
}

// Decode attention of the rows' own pages (row_info: position or -1, first own
// page, shared pages).
struct AttendShared {
    size_t pairs;           // int2 per (row, kv head): first run (-1: not cut, -2: output written) and pieces
};

struct SharedArgs {
    SharedScan sc;
    int heads, group, head_dim, num_pages, grid;
    float scale_log2;
    const int* table;
    const void* sinks;
    void* out;
    char* ws;
    ShLayout S;
};

struct PrefillPrepArgs {
    int n_tokens, rows, heads, kv_heads, head_dim, pages_per_row, num_pages, window, rope_len;
    int tile_tokens;        // tokens per tile: two halves of 128 / (heads / kv_heads)
    const void* q;          // [n_tokens, heads, D]
    const void* k_new;      // [n_tokens, kv_heads, D]
    const void* v_new;
    const int* positions;   // [n_tokens]
    const int* row_of;      // [n_tokens] table row of each token (packed: segment id)
    const int* slots;       // [n_tokens] page * 64 + offset (packed: unused)
    const void* rope_cos;   // nullptr: copy without rotation
    const void* rope_sin;
    void* k_pool;
    void* v_pool;
    char* ws;
    PfLayout L;
    int split_grid;         // > 0: also list sub-tiles at `units`, of about a share of this many CTAs each
    size_t units;
};

struct PrefillArgs {
    int n_tokens, heads, kv_heads, group, tile_tokens, head_dim, pages_per_row, num_pages, window;
    int packed;             // 1: packed sequences (keys are the pack's 64-token blocks)
    float scale_log2;
    const int* positions;
    const int* table;
    const void* sinks;      // nullptr, or [heads] of bf16
    void* out;              // [n_tokens, heads, D]
    char* ws;
    PfLayout L;
};

// Rotation, coding and cache write of n tokens (csrc/coded.cu).  With q the
// queries are rotated too, as f16 rows of q_row_bytes: D elements, for f32
// D more that hold what the first round off, and the row's factor (after
// them, or in q_factor).
struct CodeArgs {
    int n_tokens, heads, kv_heads, head_dim, num_pages, pages_per_row;
    int last_pos;           // tokens past this position are skipped
    int after_plan;         // 1: a programmatic dependent of a planner launch
    int q_row_bytes;
    float scale_log2;
    const void* q;          // nullptr: keys and values only
    const void* k_new;
    const void* v_new;
    const int* positions;
    const int* slots;       // [n_tokens] page * 64 + offset; nullptr: through the table at the token's position
    const int* table;
    const void* rope_cos;   // nullptr: no rotation
    const void* rope_sin;
    uint8_t* k;             // codes [num_pages, kv_heads, 64, head_dim]
    uint8_t* v;
    float* k_scale;         // [num_pages, kv_heads, 64]
    float* v_scale;
    uint8_t* q_out;
    float* q_factor;
    int* merge_cnt;         // decode: [rows, kv_heads] counters to clear
    char* ws;
};

struct ReadArgs {
    int n_tokens, kv_heads, head_dim, num_pages;
    int wide;               // 1: both outputs are 32-byte aligned
    const uint8_t* k;
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const int* slots;
    void* k_out;            // [n_tokens, kv_heads, head_dim] of T
    void* v_out;
    char* ws;
};

// Prefill attention over a coded cache (csrc/prefill_coded.cu).
struct CodedPrefillArgs {
    PrefillArgs a;
    const uint8_t* k;       // codes and scales
    const uint8_t* v;
    const float* k_scale;
    const float* v_scale;
    const float* q_factor;  // [n_tokens, heads]
    size_t units;           // offset of the tile list the units come from
    int slot_rows;          // rows of a split piece's partial
    float* part_o;          // [slot, kv head, slot_rows, D]
    float2* part_ml;        // [slot, kv head, slot_rows] (maximum, sum)
};

// Rotary frequencies (csrc/rotary.cu): turns per position of every pair in
// 2^-64, and what cos and sin are multiplied by.
constexpr int kRotaryPairs = 64;

struct RotaryArgs {
    int head_dim, rot_dim, interleaved, inverse, heads, kv_heads;
    float gain;
    const int* positions;   // [n_tokens]
    const void* q;          // token t's heads at q + t * q_stride elements
    const void* k;
    void* q_out;
    void* k_out;
    long long q_stride, k_stride, q_out_stride, k_out_stride;
    char* ws;               // status word only
    uint64_t turns[kRotaryPairs];
};

// Page bookkeeping (csrc/pages.cu).
struct PagesLayout {
    size_t info, table, rows, jobs, a, b, c, d, total;
};

inline PagesLayout pages_layout(int rows, int pages_per_row, int num_pages) {
    PagesLayout L;
    const size_t jobs = rows > num_pages ? rows : num_pages;
    size_t off = 256;                                   // Ctrl
    L.info = off; off += 256;
    L.table = off; off = align256(off + sizeof(int) * (size_t)rows * pages_per_row);
    L.rows = off; off = align256(off + sizeof(int2) * (size_t)rows);
    L.jobs = off; off = align256(off + sizeof(int4) * jobs);
    L.a = off; off = align256(off + sizeof(int) * (size_t)num_pages);
    L.b = off; off = align256(off + sizeof(int) * (size_t)num_pages);
    L.c = off; off = align256(off + sizeof(int) * (size_t)num_pages);
    L.d = off; off = align256(off + sizeof(int) * (size_t)num_pages);
    L.total = off;
    return L;
}

struct PagesArgs {
    int rows, pages_per_row, num_pages;
    const int* table;       // [rows, pages_per_row]
    const int* lengths;     // [rows]
    const int* refs;        // [num_pages]
    const int* parents;     // update: [rows]
    const int* new_lengths; // update: [rows]
    int* table_out;         // may be table
    int* refs_out;          // may be refs
    int* map;               // compact: [num_pages]
    char* ws;
    PagesLayout L;
};

// Pools of one copy launch; pool i's heads are slabs [first[i], first[i + 1]).
constexpr int kPoolsPerLaunch = 128;

struct PoolList {
    int n, slabs;
    void* data[kPoolsPerLaunch];
    int first[kPoolsPerLaunch];
    int row_bytes[kPoolsPerLaunch];
};

cudaError_t launch_rope_tables(float theta, int D, int S, int dtype, void* cos_out, void* sin_out,
                               cudaStream_t stream);
// The split planner (one block, if a.do_plan), then the rope + cache write of
// a.rope_blocks rows (a programmatic dependent of the planner); *launches
// gets the number of launches made.
cudaError_t launch_prep(const PrepArgs& a, int dtype, cudaStream_t stream, int* launches);
// Multi-layer prep: rope + write of every layer's rows, one plan over all.
cudaError_t launch_prep_layers(const PrepArgs& a, const PrepLayers& lay, int dtype, cudaStream_t stream,
                               int* launches);
// Sets the kernel's shared-memory limit (once per device) and launches.
cudaError_t launch_attend(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map,
                          int dtype, int grid, bool programmatic, cudaStream_t stream);
// Multi-layer attention: one persistent launch over every layer's items.
cudaError_t launch_attend_layers(const AttendArgs& a, const AttendLayers& lay, int dtype, int grid,
                                 cudaStream_t stream);
// The same over a coded cache (code 0: e4m3, 1: int8); maps over the codes.
cudaError_t launch_attend_coded(const AttendArgs& a, const CUtensorMap& k_map, const CUtensorMap& v_map, int dtype,
                                int code, int grid, cudaStream_t stream);
// Decode over shared prefixes (bf16): the rope + cache write of its rows with
// what each shares; the attention of shared and of own pages side by side; the
// outputs from their partials.
cudaError_t launch_shared_rope(const PrepArgs& a, const SharedScan& sc, size_t row_pre, cudaStream_t stream);
cudaError_t launch_shared_attend(const SharedArgs& a, const AttendArgs& own, const CUtensorMap& q_map,
                                 const CUtensorMap& k_map, const CUtensorMap& v_map, cudaStream_t stream);
cudaError_t launch_shared_join(const SharedArgs& a, cudaStream_t stream);
size_t attend_smem_bytes(int dtype, int head_dim);
// The tile list (one block), then the rope + write of every token at its
// slot (programmatic launch that ends after the tile list): two launches.
cudaError_t launch_prefill_prep(const PrefillPrepArgs& a, int dtype, cudaStream_t stream);
// Tensor-core attention of the tiles (bf16, head dim 64 or 128).
cudaError_t launch_prefill(const PrefillArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map,
                           const CUtensorMap& v_map, int grid, cudaStream_t stream);
size_t prefill_smem_bytes(int head_dim);
// Packed sequences: tile list and block summaries (one block), then rope of
// q and k into the workspace (programmatic launch ending after the plan).
cudaError_t launch_packed_prep(const PrefillPrepArgs& a, int dtype, cudaStream_t stream);
// Tensor-core attention of the packed tiles: k_map over the rotated keys and
// v_map over v, both [n, kv_heads, D] as 3-D tensors.
cudaError_t launch_packed(const PrefillArgs& a, const CUtensorMap& q_map, const CUtensorMap& k_map,
                          const CUtensorMap& v_map, int grid, cudaStream_t stream);

// The tile list alone, with sub-tiles if a.split_grid > 0 (one block).
cudaError_t launch_prefill_plan(const PrefillPrepArgs& a, cudaStream_t stream);
// Attention of the units, then, where tiles may be split, their merge.
cudaError_t launch_prefill_coded(const CodedPrefillArgs& ca, const CUtensorMap& q_map, int code, int grid, bool merge,
                                 cudaStream_t stream);
// Rotary tables of `length` positions (on a device of `sms` SMs); rotation of n_tokens tokens.
cudaError_t launch_rotary_tables(const RotaryArgs& a, int length, int dtype, void* cos_out, void* sin_out, int sms,
                                 cudaStream_t stream);
cudaError_t launch_rotary(const RotaryArgs& a, int n_tokens, int dtype, cudaStream_t stream);
// The table's part of an update or a compaction (one CTA or one cluster), then the page
// copies it listed (after_plan: a programmatic dependent of it).
cudaError_t launch_pages(const PagesArgs& a, bool compact, cudaStream_t stream);
cudaError_t launch_pages_copy(const PagesArgs& a, const PoolList& pools, int grid, bool after_plan, cudaStream_t stream);
cudaError_t launch_code(const CodeArgs& a, int dtype, int code, cudaStream_t stream);
cudaError_t launch_read(const ReadArgs& a, int dtype, int code, cudaStream_t stream);

}  // namespace pdattn
