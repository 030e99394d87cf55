// kda_linear.h -- host-side interface of the linear-attention and cache-page kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

struct LinearStepParams {
    int N, H, group;                  // group = value heads per query / key head
    const void *q, *k, *v;            // [N, H / group, Dk], [N, H / group, Dk], [N, H, Dv]
    const float *g;                   // [N, H], or [H] when g_per_head
    int g_per_head;
    float scale;
    const int32_t *slots;             // [N] or null
    int n_slots;
    const float *state;               // [n_slots, H, Dk, Dv]
    float *new_state;                 // may equal state
    void *o;                          // [N, H, Dv]
};

hipError_t launch_linear_step(int bf16, int Dk, int Dv, const LinearStepParams &p, hipStream_t stream);

// Whole sequences.  q, k, v name the walk's operands (see kda_linear_chunk.hip).
struct LinearChunkParams {
    const void *q, *k, *v;
    const float *g;                   // [rows, H], or [H] when g_per_head
    int g_per_head;
    float scale;
    const int32_t *cu;                // [N + 1] or null
    int N, T, rows;                   // sequences; tokens per sequence (all rows when cu); rows
    int H, group;                     // value heads; value heads per query / key head
    int seg, n_seg;                   // tokens per segment, segments at most
    // many packed sequences: the sequence of each segment (-1: none) [n_seg], each sequence's first segment and the
    // anchor intervals before it [N]; null: searched
    int32_t *seq_of, *first_seg, *first_anchor;
    const float *h0;                  // [N, H, Dk, Dv] or null
    float *hT;                        // [N, H, Dk, Dv] or null
    void *o;
    float *part, *dec;                // [n_part, H, Dk * Dv] and [n_part, H] of the first pass, or null: no pass
    float *part_tr;                   // backward: part once more, as [Dk][Dv]
    int n_part;
    int summed;                       // backward: the parts have been summed over each sequence
    int defer;                        // entering and resulting states share memory, and there is a first pass
    float *ckpt;                      // [N, ckpt_slots, H, Dk, Dv] or null
    int ckpt_every, ckpt_slots;
    // backward
    const void *q_rows;               // q, for y
    float *y;                         // [rows, H] or null
    float *anchors;                   // [n_anchors (+ N), H, Dk, Dv] or null: states every anchor_tokens
    int anchor_tokens, n_anchors;     // anchor_tokens divides seg
    int anchor_end;                   // the sequences' last states are kept too, behind the others
    int wide;                         // dq, dk as float32 per value head
};

struct LinearBwdParams {
    LinearChunkParams c;
    const void *d_o;
    const float *dhT;
    float *dh0;
    void *dq, *dk, *dv;               // dq, dk: float32 [rows, H, Dk] when c.wide
    void *dq_out, *dk_out;            // then their sums over the value heads of a query / key head
    float *dg;                        // or null
    double *dg_part;                  // [n_seg, H] when g_per_head
    float *part_fwd, *dec_fwd;        // the forward states' first pass (c.part, c.dec: the gradients')
    float *sum_fwd, *sum_rev;         // products of the decays that belong to the summed parts [n_part, H]
};

// Above this many packed sequences a kernel tabulates their segments first (about 5 us
// with its launch); up to it every wave searches 64 of them at a time.  Forward, H = 8, sequences of
// 64 tokens: 64 searched 17 us, tabulated 19 us; 128: 27 and 28 us; 300: 59 and 50 us; 20000 of 16: 46 and 2.2 ms.
constexpr int TABLE_SEQUENCES = 128;

// Threads of the largest workgroup that each direction launches for a segment and head.
constexpr int LINEAR_FWD_THREADS = 256, LINEAR_BWD_THREADS = 512;

hipError_t launch_linear_fwd(int bf16, int Dk, int Dv, const LinearChunkParams &p, hipStream_t stream);
hipError_t launch_linear_bwd(int bf16, int Dk, int Dv, const LinearBwdParams &p, hipStream_t stream);

// One pool of pages; unit: widest access (16, 4, 2 or 1 bytes) that its base
// addresses and page size allow.
struct CachePool {
    char *dst;
    const char *src;
    size_t page_bytes;
    int unit;
    int slices;                       // workgroup-sized pieces of a page
};

constexpr int CACHE_MAX_POOLS = 8;
// Bytes one workgroup copies: eight 16-byte accesses of each of its 256 threads,
// all in flight at once (256 pages of 2.1 MiB: 209 us, 5.3 TB/s; with 16, 64 and 128 KiB
// 203, 212 and 217 us; 237 pages of 135 KiB: 11.2 us, with the others 14.1, 14.6 and 19.3 us).
constexpr size_t CACHE_SLICE = 32768;

struct CachePools {
    CachePool pool[CACHE_MAX_POOLS];
    int n;
    int slices;                       // of a page, over all pools
};

hipError_t launch_cache_copy(const CachePools &pools, int n_dst, int n_src, const int32_t *dst_pages,
                             const int32_t *src_pages, int n, hipStream_t stream);
hipError_t launch_cache_fork(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                             int32_t *refcount, const int32_t *parents, const int32_t *children, int n,
                             int32_t *old_pages, int32_t *new_pages, hipStream_t stream);
hipError_t launch_cache_free(int32_t *table, int rows, int per_row, int32_t *refcount, int n_pages,
                             const int32_t *free_rows, int n, hipStream_t stream);
hipError_t launch_cache_compact(const CachePools &pools, int n_pages, int32_t *table, int rows, int per_row,
                                int32_t *refcount, int32_t *moved_to, int32_t *moves, int32_t *counts,
                                hipStream_t stream);

}  // namespace kda
