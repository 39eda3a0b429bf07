// msa_ragged.cuh -- parameters of the calls on ragged batches: norm and rotation
// of queries and keys, append to the paged cache, attention of ragged query rows.
#pragma once

#include "msa_cache.cuh"

namespace msa {

// Rows of 128 elements of one kind: `heads` a token, in groups of four.
struct RowSet {
    const uint16_t *x;      // bf16 bits, a token's heads one after another
    const uint16_t *weight; // norm weights (bf16), nullptr: no norm
    // head h of a token goes to y + block * block_step + h * head_step + row * bytes, block and row
    // being the token and 0 (kToOut) or its page and the row there; the scales of NVFP4 rows alike
    uint8_t *y, *scales;
    long long stride;       // elements from a token's rows to the next token's
    long long block_step, scales_block_step;
    int head_step, scales_head_step, bytes;
    int heads, group0;      // group0: the set's first group of the token's
    int where;              // kToOut .. kToIndex
    bool rotated;
    float scale, inverse;   // what stored values are multiplied with, and its reciprocal where that is exact, else 0
};

constexpr int kToOut = 0, kToK = 1, kToV = 2, kToIndex = 3;
constexpr int kMaxSets = 5;

struct AppendParams {
    RowSet set[kMaxSets];
    int sets, groups;           // row sets, and their groups of four rows a token
    int per_warp;               // groups that a warp takes
    const unsigned long long *freqs; // turns a position, in 2^-64, [rotary_dim / 2]
    const int32_t *positions;   // [T], nullptr: by offsets and seq_lens
    const int32_t *offsets;     // [R + 1]
    const int32_t *seq_lens;    // [R]
    const int32_t *block_table; // [R][maxB]
    uint32_t *err;
    int T, R, maxB, num_pages;
    int units;                  // rotary_dim / 16
    bool interleaved, per_head;
    float scale, eps, offset;
};

// A unit cut between CTAs: its first cut is this record's CTA's start (c0 < 0: there is none).
struct AttendJoin {
    int token0, tokens, head; // its first token's row, its tokens, its KV head
    int c0, c1;               // the CTAs that have parts of it
    int idle;                 // there are requests without states, whose outputs are to be written
    int pad[2];
};

struct AttendParams : CacheParams { // (nq is not used)
    uint16_t *out;          // bf16 bits [T][Hq][D]
    float *lse;             // [T][Hq]
    const int32_t *offsets; // [R + 1]
    float *partial;         // 2 slots a CTA
    AttendJoin *joins;      // one a CTA
    float v_scale;
    int T, unit_tokens;
    bool causal;
};

int device_sms(); // SMs of the current device, below 1 if it cannot be read
size_t attend_slot_bytes();
cudaError_t launch_attend(const AttendParams &p, int kv_dtype, int ctas, cudaStream_t stream);
cudaError_t launch_append(const AppendParams &p, cudaStream_t stream);

} // namespace msa
