// runs.cuh -- ragged runs: the rows of a call that belong to a batch's sequences.
//
// cu_rows[b] .. cu_rows[b + 1] - 1 are the rows of sequence b, which are its last n_b positions: row t
// is position seq_len[b] - n_b + (t - cu_rows[b]).  A decode step (n_b = 1), a few drafted tokens and a
// prefill chunk are the same layout.  Rows outside [cu_rows[0], cu_rows[B]) belong to no sequence.
#pragma once

#include "common.cuh"

namespace csa {

struct Runs {
    int B;
    int rows;                    // rows of the caller's arrays, an upper bound of cu_rows[B]
    const int32_t *cu_rows;      // [B + 1]
    const int32_t *seq_len;
    const int32_t *block_table;
    int max_pages;
    int max_seq_len;
    const int32_t *swa_row;
};

// Where a row's token lives.  seq < 0: the row belongs to no sequence, or its metadata is out of range
// (then `bad` is set).
struct RowPlace {
    int seq;
    int pos;
    int len;         // seq_len of the sequence
    int64_t slot;    // page * 64 + offset
    bool bad;
};

// The sequence of row t: the number of b with cu_rows[b + 1] <= t, found by a 32-way search of the
// whole warp (one round for up to 32 sequences, three for 16,384).  Any cu_rows gives a value in
// [0, B]; the caller checks that the sequence found holds the row.
__device__ __forceinline__ int warp_find_sequence(const int32_t *cu_rows, int B, int t)
{
    const int lane = threadIdx.x & 31;
    int lo = 0, len = B;
    while (len > 32) {
        const int step = (len + 31) >> 5;
        const int at = (lane + 1) * step;
        const int past = __popc(__ballot_sync(0xffffffffu, at <= len && cu_rows[lo + min(at, len)] <= t));
        lo += past * step;
        len = min(step, len - past * step);
    }
    return lo + __popc(__ballot_sync(0xffffffffu, lane < len && cu_rows[lo + min(lane + 1, len)] <= t));
}

// Places of the warp's rows t0 .. t0 + kTok - 1 (every lane gets them): the sequence is looked up again only
// where a row leaves it, and the page ids are loaded together, so a warp waits for one chain of loads, not kTok.
template <int kTok>
__device__ __forceinline__ void warp_place_rows(const Runs &r, int t0, int num_pages, RowPlace *p)
{
    int b = -1, c0 = 0, c1 = 0, L = 0, page[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        const int t = t0 + i;
        p[i].seq = -1;
        p[i].pos = p[i].len = 0;
        p[i].slot = -1;
        p[i].bad = false;
        page[i] = 0;
        if (t >= r.rows) continue;
        if (b < 0 || t < c0 || t >= c1) {
            b = warp_find_sequence(r.cu_rows, r.B, t);
            if (b >= r.B) continue;           // behind the last sequence
            c0 = r.cu_rows[b];
            c1 = r.cu_rows[b + 1];
            L = r.seq_len[b];
        }
        if (t < c0 && b == 0) continue;       // before the first one
        const bool holds = t >= c0 && t < c1 && c0 >= 0 && c1 <= r.rows;
        const int n = holds ? c1 - c0 : 0;
        if (!holds || L > r.max_seq_len || n > L) {
            p[i].bad = true;
            continue;
        }
        p[i].pos = L - n + (t - c0);
        p[i].len = L;
        p[i].seq = b;
        page[i] = r.block_table[(size_t)b * r.max_pages + p[i].pos / kPage];
    }
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        if (p[i].seq < 0) continue;
        if (page[i] < 0 || page[i] >= num_pages) {
            p[i].seq = -1;
            p[i].bad = true;
        } else {
            p[i].slot = (int64_t)page[i] * kPage + p[i].pos % kPage;
        }
    }
}

}  // namespace csa
