// dense_attn.cuh -- arguments, workspace and work division of the attention over the whole FP4 cache.
#pragma once

#include "common.cuh"

namespace csa {

constexpr int kDenseRows = 128;          // query rows (token, head) of one row tile
constexpr int kDensePairs = kNumSms / 2; // persistent clusters of two CTAs, one CTA per SM

// What a cluster left unfinished, for the combine: a row tile whose cache pages were shared with the next
// cluster (tail: its first part, in partial slot 2c + 1) and one that an earlier one began (head: slot 2c).
struct DenseShare {
    long long tail_row;   // first row (token * H + head, over the whole call) of the tail's row tile
    int tail_rows;        // its rows, 0 for no tail
    int head;             // 1: slot 2c holds a part of a row tile begun by an earlier cluster
    int head_ends;        // 1: that part is the row tile's last
    int pad;
};

struct DenseArgs {
    const uint8_t *codes;
    const uint8_t *scales;
    int num_pages;
    int B;
    const int32_t *seq_len;
    const int32_t *block_table;
    int max_pages;
    int max_seq_len;
    const int32_t *cu_rows;
    int rows;
    const uint16_t *q;
    int H;
    float sm_scale;
    float softcap;         // 0: none
    const float *slopes;   // float [H] or nullptr
    const int2 *spans;     // [rows] (lo, hi) or nullptr: causal
    uint16_t *out;
    float *lse;
    DenseShare *share;     // [kDensePairs]
    float2 *part_ml;       // [2 kDensePairs][kDenseRows] (running max, running sum)
    float *part_o;         // [2 kDensePairs][kDenseRows][512]
    void *ws;
};

struct DenseWs {
    size_t share, part_ml, part_o, total;
};

inline DenseWs dense_ws_layout()
{
    DenseWs w;
    w.share = kHeaderBytes;
    w.part_ml = align_up(w.share + kDensePairs * sizeof(DenseShare), 256);
    w.part_o = align_up(w.part_ml + (size_t)2 * kDensePairs * kDenseRows * sizeof(float2), 256);
    w.total = w.part_o + (size_t)2 * kDensePairs * kDenseRows * kLatent * sizeof(float);
    return w;
}

cudaError_t launch_dense_attn(const DenseArgs &a, cudaStream_t st);

}  // namespace csa
