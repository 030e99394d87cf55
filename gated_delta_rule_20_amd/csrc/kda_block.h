// kda_block.h -- host-side interface of the gated scan, of the norms around a
// block and of activations in 8 bits.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int ACT_GROUP = 128;        // channels that share a scale
constexpr int NORM_MAX_D = 16384;     // channels of a row

// Block norms backwards: up to norm_row_d channels a workgroup holds whole rows, beyond columns of NORM_COLUMN channels.  In
// float32 a row of 8192 does not fit the registers next to its sums: 4096 x 8192 412 us by rows, 370 by columns, 16 x 8192 48 and 27.
// With bf16 it does: 141 and 230 us, 27 and 28 (next to a float32 stream 231 and 282, but 38 and 27: the rule goes by the blocks' type alone).
constexpr int norm_row_d(bool f32) { return f32 ? 4096 : 8192; }
constexpr int NORM_COLUMN = 1024;

// Rows that the gradients add up in float32 (64 roundings); such sums are joined in float64.
constexpr int NORM_CHAIN = 64;

// Rows that a workgroup holds side by side, and its waves.
constexpr int norm_rows(int D) { return D <= 256 ? 4 : D <= 512 ? 2 : 1; }
constexpr int norm_waves(int D) { return D <= 1024 ? 4 : D <= 2048 ? 8 : 16; }

// Rows of C elements: of a type, or (scales set) int8 codes with their scales.
struct Rows {
    const void *p;
    const float *scales;              // [rows, groups] or null
    int64_t stride;                   // elements from row to row
};

// An 8-bit copy that a kernel also writes.
struct PackedOut {
    int8_t *codes;                    // null: none
    float *scales;
};

// A workgroup of a scan takes SCAN_ROWS rows (a segment) of SCAN_CHANNELS channels.
constexpr int SCAN_ROWS = 64, SCAN_CHANNELS = 128;

// Segments that join their pairs, and blocks of them that join theirs; counters that lie 128 bytes apart.
constexpr int SCAN_BLOCK = 8, SCAN_TICKET_STEP = 32;

// Up to so many packed sequences, segments go through the offsets that fall among their rows and pass on the states of empty sequences
// themselves; of more, they search the offsets and a kernel of its own passes the states on.  (2^16 empty sequences in one place take
// 14 ms of one workgroup, for which the segments behind wait; 2^22 740 ms, longer than they do.)
constexpr int SCAN_MANY = 1 << 16;

// Hand-over between segments, cleared at the start of a call: pairs of decay and state for each segment and each
// SCAN_BLOCK segments [.., C], the state behind every SCAN_BLOCK^2 [.., C]; the tickets of each SCAN_CHANNELS channels;
// whether a wait was given up.
struct ScanChain {
    uint64_t *part, *blocks, *whole;
    uint32_t *tickets, *gave_up;
    size_t words, counters;           // pairs, all three kinds; counters of 4 bytes, the flag among them
    int segments;
};

struct ScanParams {
    int rows, T, C;                   // rows of all sequences; tokens per sequence when cu is null
    const int32_t *cu;                // [N + 1] or null
    int N;
    Rows x, g;                        // backward: x only with complement
    const float *A_log;               // [C] or null: g holds log-decays
    float g_min;
    int complement;
    const float *h0;                  // [N, C] or null
    // forward
    void *h;
    float *hT;
    PackedOut h8;
    // backward
    Rows hs;                          // p null: no dg
    const void *d_h;
    const float *dhT;
    void *dx, *dg;
    int64_t dx_stride, dg_stride;
    float *dA, *dh0;
    float *dA_part;                   // [segments, C]
    // more than one segment: the call's tickets and what the segments hand on
    ScanChain chain;
    float *state_copy;                // of the entering states, where the resulting ones overwrite them, or null
};

struct ScanStepParams {
    int N, C;
    Rows x, g;
    const float *A_log;
    float g_min;
    int complement;
    const int32_t *slots;             // [N] or null
    int n_slots;
    const float *state;
    float *new_state;
    void *h;
};

hipError_t launch_scan_fwd(int bf16, int g_bf16, const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_bwd(int bf16, int g_bf16, const ScanParams &p, hipStream_t stream);
hipError_t launch_scan_step(int bf16, int g_bf16, const ScanStepParams &p, hipStream_t stream);

struct NormParams {
    int R, D;
    Rows x, y, gate;                  // backward: x is the stream behind the block; y.p, gate.p may be null
    const float *post, *res, *pre;    // [D] or null
    float scale, eps;
    // forward
    void *x_out, *n;
    PackedOut x8, y8, gate8;
    // backward
    const void *d_x, *d_n;            // or null
    void *dx, *dy, *dgate;
    int64_t dy_stride, dgate_stride;
    float *dpost, *dres, *dpre;       // [D] or null
    float *part;                      // [3, parts, D]
    float __attribute__((ext_vector_type(4))) *numbers;  // [R], beyond norm_row_d channels
    int parts, groups;                // workgroups (of a column); those that run at a time
};

hipError_t launch_norm_fwd(int bf16, int x_bf16, const NormParams &p, hipStream_t stream);
hipError_t launch_norm_bwd(int bf16, int x_bf16, const NormParams &p, hipStream_t stream);

// rows x D values at a stride to codes and scales, and back.
hipError_t launch_act_pack(int bf16, const Rows &x, long long rows, int D, const PackedOut &out, hipStream_t stream);
hipError_t launch_act_unpack(int bf16, const Rows &x, long long rows, int D, void *out, hipStream_t stream);

}  // namespace kda
