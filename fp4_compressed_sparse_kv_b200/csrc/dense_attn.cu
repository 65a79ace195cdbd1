// dense_attn.cu -- attention of ragged query runs over the whole paged FP4 cache, on the sm_100a tensor
// cores (tcgen05, TMEM).
//
// yomxxx.com long-form post on KV-cache compression limits, section 五 (a fixed layout with addresses from
// the token index, dequantised in the kernel, in parallel); rebasdaily article on DeepSeek-V4.1-Flash KV
// compression, section "同一份笔记，多层一起用" (FP4 main KV; the 512-channel latent is key and value).
//
// Row tile: 64 consecutive (token, head) rows of one sequence, token-major, so that 64 heads of one
// decoded token, 16 heads of four drafted tokens or half of a 128-head token fill the same matrix
// operand and any head count works.  Cache tile: one 64-position page.  For every (row tile, page):
//   QK:  S_x[64 rows x 64 entries] = Q_x . V_x^T for the channel halves x = 0, 1 (M = 64; A = Q_x in
//        TMEM, B = V K-major);
//   PV:  O^T[128 ch x 64 rows] (x4) += V^T[128 ch x 64 entries] . P^T  (M = 128; A = V^T MN-major,
//        B = P^T K-major).
// The tile layout, TMEM columns, warp roles and numerics are those of attention_tc.cu (Q in TMEM, three
// 64 KB fp16 V buffers, exact dequantisation, P rounded to fp16 once, fp32 accumulation and sums); Q is
// scaled by a power of two per row, so a row of very large or non-finite values does not touch the
// others of its tile.
//
// Work division: the (row tile, page) pairs of the whole call, row tile by row tile, are one line that
// 148 persistent CTAs (one per SM) cut into equal shares, whatever the batch looks like: one long
// sequence splits over all SMs, a prefill chunk gives each SM whole row tiles.  Every CTA works out the
// division itself from cu_rows, seq_len and the spans (a block scan; no extra launch).  A CTA finishes
// the row tiles it holds whole; the first and last tile of its share may be shared with its neighbours,
// and those leave an fp32 partial (unnormalised O, running maximum and sum) in the workspace, which the
// combine kernel adds in CTA order, so results do not depend on timing.
#include <cuda_bf16.h>

#include "attention_tile.cuh"
#include "convert.cuh"
#include "dense_attn.cuh"

namespace csa {

constexpr int kTile = 64;                        // entries per tile: one page
constexpr int kDnChunks = kLatent / 64;          // 8 chunks of 64 channels
constexpr int kDnStages = 3;                     // tiles in flight
constexpr int kDnProducers = 512;                // warps 0-15
constexpr int kDnSoftmax = 128;                  // warps 16-19
constexpr int kDnSoftmaxWarp = 16;
constexpr int kDnIssuerWarp = 20;                // warps 20-23
constexpr int kDnThreads = 768;
constexpr uint32_t kDnVChunk = kTile * 128;              // 8 KB: 64 rows x 64 fp16
constexpr uint32_t kDnVBuf = kDnChunks * kDnVChunk;      // 64 KB per tile buffer
constexpr uint32_t kDnPBuf = kDenseRows * 128;           // 8 KB: 64 rows x 64 entries fp16
constexpr uint32_t kDnOffP = kDnStages * kDnVBuf;
constexpr uint32_t kDnOffMisc = kDnOffP + kDnStages * kDnPBuf;
constexpr uint32_t kDnTmemCols = 512;
constexpr uint32_t kDnColO = 0;                  // O^T: M-tile m in columns 64m .. 64m+63
constexpr uint32_t kDnColQ = 256;                // Q_x: 128 columns in lane half x
constexpr uint32_t kDnColS = 384;                // S_x of tile g: columns 384 + 64(g%2) in lane half x
constexpr long long kDnMinTiles = 2;             // pages a CTA takes at least
static_assert(kTile == kPage, "a tile is one page");

// One CTA's part of one row tile.
struct DensePiece {
    long long row;       // first row of the row tile over the call (token * H + head)
    uint32_t r0;         // the same within the sequence
    int rows;            // rows of the row tile, 1 .. 64; 0: the CTA has no further piece
    int b, c0, n, L;     // sequence, its first token, tokens and length
    int kv0, kv1;        // pages [kv0, kv1) of this piece; none if no row of the tile sees anything
    int first, last;     // the piece holds the first / last of the row tile's pages
};

// Where a CTA is on the line of (row tile, page) pairs.
struct DenseCursor {
    long long left;      // pairs of its share still to take
    long long off;       // pairs of row tile `tile` before them
    int tile, b;
};

struct DenseMisc {
    uint64_t q_ready;
    uint64_t v_ready[kDnStages], v_free[kDnStages], p_full[kDnStages];
    uint64_t s_full[2], s_free[2];
    uint64_t final_bar[4];
    uint64_t vmask[kDnStages];              // valid entries of the tile in each V buffer
    uint32_t nan_tile[kDnStages];           // tile number + 1 if an entry of the tile has a NaN scale
    uint32_t nan_entry[kDnStages][kTile];   // the same for each entry
    uint32_t tmem_base;
    int abort_flag;
    long long warp_sum[kDnThreads / 32];
    DensePiece piece[2];
    DenseCursor cur;
    DenseShare share;
    uint32_t qmax[kDenseRows];              // bits of each row's largest |q|
    float zs[kDenseRows];                   // accumulated score -> log2 domain, per row
    float alpha[kDenseRows];                // rescale factor of each row at a maximum update
    float inv[kDenseRows];                  // 1 / denominator of a finished row
};

constexpr size_t kDnSmem = kDnOffMisc + sizeof(DenseMisc) + 1024;
constexpr uint32_t kDnIdescQK = umma_idesc_f16(64, kTile, false, false);
constexpr uint32_t kDnIdescPV = umma_idesc_f16(128, kDenseRows, true, false);

// Named barriers: 1 = the softmax warps; 3 = the producers; 4 = every warp.

// ------------------------------------------------------------------------------------------------
// Work division.  Sequence b's row tiles have the numbers tile_base(b) .. tile_base(b + 1) - 1: at least
// ceil(n_b H / 64) of them, the rest empty, without a scan over the batch.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ long long tile_base(int c0, int b, int H) { return (long long)c0 * H / kDenseRows + b; }

// Pages [kv0, kv0 + nk) that rows r0 .. r0 + 63 of a sequence see between them.
__device__ __forceinline__ void tile_pages(const DenseArgs &a, int c0, int n, int L, uint32_t r0, int &kv0, int &nk)
{
    const int ta = (int)(r0 / (uint32_t)a.H);
    const int tb = min((int)((r0 + kDenseRows - 1) / (uint32_t)a.H), n - 1);
    int lo = 0, hi = L - n + tb + 1;
    if (a.spans) {
        lo = L;
        hi = 0;
        for (int t = ta; t <= tb; ++t) {
            const int2 s = a.spans[c0 + t];
            const int sl = max(s.x, 0), sh = min(s.y, L);
            if (sl < sh) {
                lo = min(lo, sl);
                hi = max(hi, sh);
            }
        }
    }
    kv0 = hi > lo ? lo / kPage : 0;
    nk = hi > lo ? (hi + kPage - 1) / kPage - kv0 : 0;
}

// Share of the line that row tile r0 of a sequence takes: its pages, at least one so that a row tile
// that sees nothing is written too; 0 for a tile number without rows or a sequence left out.
__device__ __forceinline__ int tile_weight(const DenseArgs &a, int c0, int n, int L, uint32_t r0)
{
    if (L < n || r0 >= (uint32_t)n * (uint32_t)a.H) return 0;
    int kv0, nk;
    tile_pages(a, c0, n, L, r0, kv0, nk);
    return max(nk, 1);
}

// The next piece of the CTA's share, and what the share leaves unfinished.
__device__ void next_piece(const DenseArgs &a, DenseCursor &cu, DenseShare &share, DensePiece &pc)
{
    pc.rows = 0;
    while (cu.left > 0) {
        const int c0 = a.cu_rows[cu.b], c1 = a.cu_rows[cu.b + 1], n = c1 - c0;
        if (cu.tile >= tile_base(c1, cu.b + 1, a.H)) {
            if (++cu.b >= a.B) return;
            continue;
        }
        int L = a.seq_len[cu.b];
        if (L > a.max_seq_len) L = 0;
        const uint32_t r0 = (uint32_t)(cu.tile - tile_base(c0, cu.b, a.H)) * kDenseRows;
        const int w = tile_weight(a, c0, n, L, r0);
        if (w == 0) {
            ++cu.tile;
            continue;
        }
        int kv0, nk;
        tile_pages(a, c0, n, L, r0, kv0, nk);
        const long long take = min((long long)w - cu.off, cu.left);
        pc.row = (long long)c0 * a.H + r0;
        pc.r0 = r0;
        pc.rows = (int)min((uint32_t)kDenseRows, (uint32_t)n * (uint32_t)a.H - r0);
        pc.b = cu.b;
        pc.c0 = c0;
        pc.n = n;
        pc.L = L;
        pc.kv0 = kv0 + (int)cu.off;
        pc.kv1 = min(kv0 + (int)(cu.off + take), kv0 + nk);
        pc.first = cu.off == 0;
        pc.last = cu.off + take == w;
        if (!pc.first) {
            share.head = 1;
            share.head_ends = pc.last;
        } else if (!pc.last) {
            share.tail_row = pc.row;
            share.tail_rows = pc.rows;
        }
        cu.left -= take;
        cu.off = 0;
        ++cu.tile;
        return;
    }
}

// This CTA's share: block-wide sums of the row tiles' weights, each thread over consecutive tiles, then
// the tile and page where the share begins.  `scratch` holds cu_rows and seq_len of every sequence.
__device__ void plan(const DenseArgs &a, DenseMisc &ms, int32_t *scratch)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int32_t *s_cu = scratch, *s_len = scratch + a.B + 1;
    for (int i = tid; i <= a.B; i += kDnThreads) s_cu[i] = a.cu_rows[i];
    for (int i = tid; i < a.B; i += kDnThreads) s_len[i] = a.seq_len[i];
    if (tid == 0) {
        ms.piece[0].rows = 0;
        ms.cur = DenseCursor{0, 0, 0, 0};
        ms.share = DenseShare{0, 0, 0, 0, 0};
    }
    __syncthreads();
    int bad = 0;
    for (int b = tid; b < a.B; b += kDnThreads) {
        const int c0 = s_cu[b], c1 = s_cu[b + 1];
        if (c0 < 0 || c1 < c0 || c1 > a.rows) {
            bad = 1;
            report(a.ws, CSA_ERR_DEVICE_DATA, b);
        } else if (c1 > c0 && (s_len[b] < c1 - c0 || s_len[b] > a.max_seq_len)) {
            s_len[b] = 0;   // left out
            report(a.ws, CSA_ERR_DEVICE_DATA, b);
        }
    }
    if (__syncthreads_or(bad)) return;   // no row can be placed
    const long long tiles = tile_base(s_cu[a.B], a.B, a.H);
    const long long chunk = (tiles + kDnThreads - 1) / kDnThreads;
    const long long i0 = chunk * tid, i1 = min(tiles, i0 + chunk);
    int b0 = 0;
    if (i0 < i1) {
        int hi = a.B - 1;   // the last sequence that begins at or before tile i0
        while (b0 < hi) {
            const int mid = (b0 + hi + 1) >> 1;
            if (tile_base(s_cu[mid], mid, a.H) <= i0) b0 = mid;
            else hi = mid - 1;
        }
    }
    auto weight = [&](long long i, int &b) {
        while (b + 1 < a.B && tile_base(s_cu[b + 1], b + 1, a.H) <= i) ++b;
        return tile_weight(a, s_cu[b], s_cu[b + 1] - s_cu[b], s_len[b],
                           (uint32_t)(i - tile_base(s_cu[b], b, a.H)) * kDenseRows);
    };
    long long sum = 0;
    int b = b0;
    for (long long i = i0; i < i1; ++i) sum += weight(i, b);
    long long incl = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) ms.warp_sum[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int i = 0; i < kDnThreads / 32; ++i) {
        if (i < warp) before += ms.warp_sum[i];
        total += ms.warp_sum[i];
    }
    const long long excl = before + incl - sum;
    // as many CTAs as leave each kDnMinTiles pages
    const long long ctas = max(1ll, min((long long)gridDim.x, total / kDnMinTiles));
    if (blockIdx.x < ctas) {
        const long long s = total * blockIdx.x / ctas, e = total * (blockIdx.x + 1) / ctas;
        if (s < e && excl <= s && s < excl + sum) {
            long long at = excl;
            b = b0;
            for (long long i = i0; i < i1; ++i) {
                const int w = weight(i, b);
                if (s < at + w) {
                    ms.cur = DenseCursor{e - s, s - at, (int)i, b};
                    break;
                }
                at += w;
            }
            next_piece(a, ms.cur, ms.share, ms.piece[0]);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// A producer thread's share of one page: entry e, channels 64cp .. 64cp+63 (V chunk cp).  The raw bytes
// (32 B of codes, 4 scale bytes) are loaded into registers two tiles ahead and dequantised one tile
// ahead, so that once PV releases the buffer only the stores remain.
// ------------------------------------------------------------------------------------------------
struct PageEntry {
    uint4 code[2];
    uint32_t sc;
    bool valid;

    __device__ __forceinline__ void fetch(const DenseArgs &a, int page, bool ok, int e, int cp)
    {
        valid = ok;
        if (ok) {
            const size_t row = (size_t)page * kPage + e;
            const uint4 *c4 = reinterpret_cast<const uint4 *>(a.codes + row * kCodeBytes + 32 * cp);
            code[0] = c4[0];
            code[1] = c4[1];
            sc = *reinterpret_cast<const uint32_t *>(a.scales + row * kScaleBytes + 4 * cp);
        }
    }

    // One of the four scales is NaN (E4M3 0x7F or 0xFF).
    __device__ __forceinline__ bool has_nan() const
    {
        return valid && (((sc & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
    }

    // Channels 64cp .. 64cp+63 as 32 fp16 pairs; zeros for an invalid or NaN entry.
    __device__ __forceinline__ void dequant(uint32_t *v) const
    {
        if (!valid || has_nan()) {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0u;
            return;
        }
        uint32_t sh[2];   // the four group scales as (s0, s1), (s2, s3)
        e4m3x4_to_f16x2x2(sc, sh);
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) {
            const uint32_t s2 = __byte_perm(sh[gg >> 1], 0u, (gg & 1) ? 0x3232u : 0x1010u);
            const uint4 cw = code[gg >> 1];
            uint32_t c0[4], c1[4];
            e2m1x8_to_f16x2x4((gg & 1) ? cw.z : cw.x, c0);
            e2m1x8_to_f16x2x4((gg & 1) ? cw.w : cw.y, c1);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[8 * gg + q] = hmul2_u32(c0[q], s2);
                v[8 * gg + 4 + q] = hmul2_u32(c1[q], s2);
            }
        }
    }
};

// Q of the row tile into TMEM as the A operand of the QK MMAs, each row scaled by the power of two 2^k
// that puts its largest |q| in [2^13, 2^14); ms.zs gets tau * log2(e) * 2^-k.  Warps 0-15; warp w writes
// TMEM quarter w%4 (rows 16(w%4) .. +15) and channel block w/4 of each half: lane l converts channels
// 256(l/16) + 64(w/4) .. +63 of row 16(w%4) + l%16 into 32 columns of lane 32(w%4) + l.  Rows past the
// row tile's are zeros.
__device__ __forceinline__ void load_q_rows(const DenseArgs &a, DenseMisc &ms, const DensePiece &pc, uint32_t tmem)
{
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, q = w & 3, j = w >> 2;
    const int h = 16 * q + (lane & 15);
    const int c0 = 256 * (lane >> 4) + 64 * j;
    uint4 qw[8];
    const uint4 *src = reinterpret_cast<const uint4 *>(a.q + (size_t)(pc.row + h) * kLatent + c0);
#pragma unroll
    for (int c = 0; c < 8; ++c) qw[c] = h < pc.rows ? src[c] : make_uint4(0u, 0u, 0u, 0u);
    uint32_t top = 0u;   // largest |q| as bf16 bits in the upper half
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t ww[4] = {qw[c].x, qw[c].y, qw[c].z, qw[c].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(ww[k] & 0x7FFF0000u, (ww[k] << 16) & 0x7FFF0000u));
    }
    atomicMax(&ms.qmax[h], top);
    bar_sync(3, kDnProducers);
    top = ms.qmax[h];
    int k = 0;
    if (top != 0u) {
        k = 13 - ((int)(top >> 23) - 127);
        k = k < -120 ? -120 : (k > 120 ? 120 : k);
    }
    const float sc = exp2f((float)k);
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
        uint32_t v[16];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint4 x = qw[4 * hh + c];
            v[4 * c] = pack_f16x2(bf16_lo(x.x) * sc, bf16_hi(x.x) * sc);
            v[4 * c + 1] = pack_f16x2(bf16_lo(x.y) * sc, bf16_hi(x.y) * sc);
            v[4 * c + 2] = pack_f16x2(bf16_lo(x.z) * sc, bf16_hi(x.z) * sc);
            v[4 * c + 3] = pack_f16x2(bf16_lo(x.w) * sc, bf16_hi(x.w) * sc);
        }
        tc_st16_u(tmem + ((uint32_t)(32 * q) << 16) + kDnColQ + 32 * j + 16 * hh, v);
    }
    tc_wait_st();
    tc_fence_before();
    if (j == 0 && lane < 16) ms.zs[h] = a.sm_scale * exp2f((float)-k) * kLog2e;
    warp_arrive(&ms.q_ready);
}

__global__ void __launch_bounds__(kDnThreads, 1) dense_attn_kernel(DenseArgs a)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t *base = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *V = base;
    uint8_t *P = base + kDnOffP;
    DenseMisc &ms = *reinterpret_cast<DenseMisc *>(base + kDnOffMisc);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    grid_dep_launch();   // the combine may be scheduled as CTAs finish

    if (tid == 0) {
        mbar_init(&ms.q_ready, kDnProducers / 32);
        for (int i = 0; i < kDnStages; ++i) {
            mbar_init(&ms.v_ready[i], kDnProducers / 32);
            mbar_init(&ms.v_free[i], 2);
            mbar_init(&ms.p_full[i], kDnSoftmax / 32);
            ms.nan_tile[i] = 0;
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.s_full[i], 2);
            mbar_init(&ms.s_free[i], kDnSoftmax / 32);
        }
        for (int r = 0; r < 4; ++r) mbar_init(&ms.final_bar[r], 1);
        ms.abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < kDenseRows) ms.qmax[tid] = 0u;
    if (tid < kDnStages * kTile) (&ms.nan_entry[0][0])[tid] = 0u;
    if (warp == kDnIssuerWarp) {
        tc_alloc(smem_addr(&ms.tmem_base), kDnTmemCols);
        tc_relinquish();
    }
    grid_dep_wait();   // everything below reads what earlier kernels wrote, or writes what they read
    plan(a, ms, reinterpret_cast<int32_t *>(V));

    bool ok = true;
    uint32_t g0 = 0;      // tiles of the earlier pieces
    uint32_t pieces = 0;  // earlier pieces that had tiles
    for (int pi = 0;; pi ^= 1) {
        // the piece is visible and the previous one is finished with TMEM and shared memory
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        const DensePiece &pc = ms.piece[pi];
        if (pc.rows == 0) break;
        const uint32_t tmem = ms.tmem_base;
        const int nk = pc.kv1 - pc.kv0;

        if (warp >= kDnIssuerWarp) {
            // ------------------------------- MMA issuers -------------------------------
            const int r = warp - kDnIssuerWarp;
            if (r == 3 && lane == 0) next_piece(a, ms.cur, ms.share, ms.piece[pi ^ 1]);
            if (lane == 0 && nk > 0) {
                const uint32_t sV = smem_addr(V), sP = smem_addr(P);
                ok = mbar_wait(&ms.q_ready, pieces & 1u, &ms.abort_flag, a.ws, 1);
                tc_fence_after();
                if (r < 2) {
                    // QK of channel half r into S_r of tile g (lanes of half r, columns of parity g % 2),
                    // once the producers have written the tile and the softmax has read tile g - 2's scores
                    const uint32_t lanes = (uint32_t)(16 * r) << 16;
                    for (int t = 0; ok && t < nk; ++t) {
                        const uint32_t g = g0 + t, p = g % kDnStages, sb = g & 1u;
                        ok = mbar_wait(&ms.v_ready[p], (g / kDnStages) & 1u, &ms.abort_flag, a.ws, 3);
                        if (ok && g >= 2) ok = mbar_wait(&ms.s_free[sb], ((g >> 1) - 1u) & 1u, &ms.abort_flag, a.ws, 10);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const int c = 4 * r + (k >> 2);   // V chunk of channels 256r + 16k ..
                            const uint64_t bd = umma_sdesc_sw128(sV + p * kDnVBuf + c * kDnVChunk + (k & 3) * 32, 16, 1024);
                            tc_mma_f16_ts(tmem + lanes + kDnColS + 64 * sb, tmem + lanes + kDnColQ + 8 * k, bd, kDnIdescQK,
                                          k > 0 ? 1u : 0u);
                        }
                        tc_commit(smem_addr(&ms.s_full[sb]));
                    }
                } else {
                    // PV of M-tiles 2(r-2), 2(r-2)+1 once the softmax has written P of the tile; the commit
                    // releases the tile's V and P buffers
                    const int m0 = 2 * (r - 2);
                    for (int t = 0; ok && t < nk; ++t) {
                        const uint32_t g = g0 + t, p = g % kDnStages;
                        ok = mbar_wait(&ms.p_full[p], (g / kDnStages) & 1u, &ms.abort_flag, a.ws, 2);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int mi = 0; mi < 2; ++mi)
#pragma unroll
                            for (int kk = 0; kk < kTile / 16; ++kk) {
                                const int m = m0 + mi;
                                const uint64_t ad = umma_sdesc_sw128(sV + p * kDnVBuf + 2 * m * kDnVChunk + kk * 2048, kDnVChunk, 1024);
                                const uint64_t bd = umma_sdesc_sw128(sP + p * kDnPBuf + kk * 32, 16, 1024);
                                tc_mma_f16(tmem + kDnColO + 64 * m, ad, bd, kDnIdescPV, (t > 0 || kk > 0) ? 1u : 0u);
                            }
                        tc_commit(smem_addr(&ms.v_free[p]));
                    }
                }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        } else if (warp < kDnSoftmaxWarp) {
            // ------------------------------- producers -------------------------------
            if (nk > 0) {
                const int e = tid & (kTile - 1), cp = tid >> 6;
                const int32_t *bt = a.block_table + (size_t)pc.b * a.max_pages + pc.kv0;
                const int left = pc.L - pc.kv0 * kPage;   // positions of the sequence from the piece's first page on
                auto fetch = [&](PageEntry &en, int page, int t) {
                    const bool page_ok = page >= 0 && page < a.num_pages;
                    if (!page_ok && tid == 0) report(a.ws, CSA_ERR_DEVICE_DATA, pc.kv0 + t);
                    en.fetch(a, page, page_ok && t * kPage + e < left, e, cp);
                };
                PageEntry raw0, raw1;   // tiles of even and of odd index
                fetch(raw0, bt[0], 0);
                if (nk > 1) fetch(raw1, bt[1], 1);
                int page = nk > 2 ? bt[2] : 0;   // the page of the tile fetched next
                load_q_rows(a, ms, pc, tmem);
                uint32_t v[32];   // the next tile's row, dequantised before its buffer is free
                raw0.dequant(v);
                // rw holds tile t, already dequantised into v, so it takes tile t + 2 at once; rn holds t + 1
                auto step = [&](int t, PageEntry &rw, const PageEntry &rn) {
                    const uint32_t g = g0 + t, p = g % kDnStages;
                    const unsigned int vb = __ballot_sync(0xffffffffu, rw.valid);
                    const bool nan = rw.has_nan();
                    if (t + 2 < nk) {
                        fetch(rw, page, t + 2);
                        if (t + 3 < nk) page = bt[t + 3];
                    }
                    if (g >= kDnStages) ok = ok && warp_wait(&ms.v_free[p], (g / kDnStages - 1u) & 1u, &ms.abort_flag, a.ws, 5);
                    if (ok) {
                        uint8_t *dst = V + p * kDnVBuf + cp * kDnVChunk;
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *reinterpret_cast<uint4 *>(dst + swz((uint32_t)e, (uint32_t)u)) =
                                make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
                        if (nan) {
                            ms.nan_entry[p][e] = g + 1u;
                            ms.nan_tile[p] = g + 1u;
                        }
                    }
                    if (cp == 0 && lane == 0) reinterpret_cast<volatile uint32_t *>(&ms.vmask[p])[warp] = vb;
                    fence_async_smem();
                    warp_arrive(&ms.v_ready[p]);
                    if (t + 1 < nk) rn.dequant(v);
                };
#pragma unroll 1
                for (int t = 0; t < nk; t += 2) {
                    step(t, raw0, raw1);
                    if (t + 1 < nk) step(t + 1, raw1, raw0);
                }
            }
        } else {
            // ------------------------------- softmax -------------------------------
            const int q = warp - kDnSoftmaxWarp;     // TMEM quarter: rows 16q .. 16q+15
            const int u = lane >> 4;                 // this thread's entries 32u .. 32u+31 of a tile
            const int hl = 16 * q + (lane & 15);     // this thread's row
            const uint32_t tq = tmem + ((uint32_t)(32 * q) << 16);
            const uint32_t row = pc.r0 + (uint32_t)hl;
            const int tok = (int)(row / (uint32_t)a.H), head = (int)(row % (uint32_t)a.H);
            const int pos = pc.L - pc.n + tok;
            int lo = 0, hi = 0;                      // positions the row sees
            float slope = 0.f;                       // of the distance bias, log2 domain
            if (hl < pc.rows) {
                hi = pos + 1;
                if (a.spans) {
                    const int2 s = a.spans[pc.c0 + tok];
                    lo = max(s.x, 0);
                    hi = min(s.y, pc.L);
                }
                if (a.slopes) slope = a.slopes[head] * kLog2e;
            }
            float m_run = kNoMax;                    // the row's running maximum (log2 domain), as the partner has it
            float lsum = 0.f;                        // this thread's share of the row's denominator
            if (nk > 0) ok = bar_and(1, kDnSoftmax, ok && warp_wait(&ms.q_ready, pieces & 1u, &ms.abort_flag, a.ws, 11));
            const float zs = ms.zs[hl];
            for (int t = 0; t < nk; ++t) {
                const uint32_t g = g0 + t, p = g % kDnStages, sb = g & 1u;
                // v_ready: the producers' valid-entry mask of this tile; s_full: both halves of its scores
                ok = bar_and(1, kDnSoftmax, ok && warp_wait(&ms.v_ready[p], (g / kDnStages) & 1u, &ms.abort_flag, a.ws, 9) &&
                                                warp_wait(&ms.s_full[sb], (g >> 1) & 1u, &ms.abort_flag, a.ws, 6));
                if (!ok) {
                    warp_arrive(&ms.s_free[sb]);
                    warp_arrive(&ms.p_full[p]);
                    continue;
                }
                tc_fence_after();
                // z[j] = S_0 + S_1 of entry 32u + j of row hl (unscaled)
                float z[32];
#pragma unroll
                for (int pcs = 0; pcs < 2; ++pcs) {
                    float s0[16], s1[16];
                    tc_ld16x32bx2_x16_pair(tq + kDnColS + 64 * sb + 16 * pcs,
                                           tq + (16u << 16) + kDnColS + 64 * sb + 16 * pcs, s0, s1);
#pragma unroll
                    for (int i = 0; i < 16; ++i) z[16 * pcs + i] = s0[i] + s1[i];
                }
                tc_fence_before();
                warp_arrive(&ms.s_free[sb]);   // QK of tile g + 2 may overwrite these columns
                const int e0 = (pc.kv0 + t) * kPage + 32 * u;   // position of z[0]
                float zf = zs;                                  // z -> log2 domain
                if (a.softcap > 0.f) {
                    // cap tanh(s / cap) = cap (1 - 2 / (1 + e^(2 s / cap))): absolute error a few 2^-24 cap
                    const float arg = 2.f * zs / a.softcap, cap = a.softcap * kLog2e;
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = cap * (1.f - __fdividef(2.f, 1.f + exp2f(z[i] * arg)));
                    zf = 1.f;
                }
                if (a.slopes) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) z[i] = fmaf(z[i], zf, -slope * fabsf((float)(pos - e0 - i)));
                    zf = 1.f;
                }
                if (ms.nan_tile[p] == g + 1u) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (ms.nan_entry[p][32 * u + i] == g + 1u) z[i] = __int_as_float(0x7FC00000);
                }
                // entries that are valid and that the row sees
                uint32_t seen = (uint32_t)(ms.vmask[p] >> (32 * u));
                if (lo > e0) seen &= lo - e0 < 32 ? 0xFFFFFFFFu << (lo - e0) : 0u;
                if (hi < e0 + 32) seen &= hi > e0 ? 0xFFFFFFFFu >> (32 - (hi - e0)) : 0u;
                if (seen != 0xFFFFFFFFu) {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (!((seen >> i) & 1u)) z[i] = -INFINITY;
                }
                float mt = -INFINITY;
#pragma unroll
                for (int i = 0; i < 32; ++i) mt = fmaxf(mt, z[i]);
                mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16)) * zf;   // zf > 0
                const bool need = mt > m_run + kLazy;
                if (bar_or(1, kDnSoftmax, need)) {
                    // some row's maximum grew: new maxima, and O^T rescaled column by column
                    const float mn = need ? fmaxf(m_run, mt) : m_run;
                    const float al = exp2f(m_run - mn);   // 0 while m_run is kNoMax, 1 if unchanged
                    if (u == 0) ms.alpha[hl] = al;
                    lsum *= al;
                    m_run = mn;
                    bar_sync(1, kDnSoftmax);   // every row's factor visible
                    if (t > 0) {
                        // this warp's lanes of the four O^T M-tiles, once PV of the previous tile has completed
                        const uint32_t gp = g - 1u;
                        ok = warp_wait(&ms.v_free[gp % kDnStages], (gp / kDnStages) & 1u, &ms.abort_flag, a.ws, 7);
                        if (ok) {
                            tc_fence_after();
#pragma unroll 1
                            for (int k = 0; k < 32; ++k) {
                                float o[8];
                                const uint32_t col = kDnColO + 8 * k;   // M-tile k/8, rows 8(k%8) ..
                                tc_ld8_sync(tq + col, o);
#pragma unroll
                                for (int i = 0; i < 8; ++i) o[i] *= ms.alpha[8 * (k & 7) + i];
                                tc_st8(tq + col, o);
                            }
                            tc_wait_st();
                        }
                    }
                }
                // P^T row hl, entries 32u .. 32u+31: four 16-byte units of the 128-byte swizzled row;
                // p = 2^(z zf - m + 7), 0 for a masked entry (z = -inf)
                const float mref = m_run - kPOffset;
                float ls = 0.f;
                uint8_t *Pb = P + p * kDnPBuf;
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    uint32_t pk[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p0 = exp2f(fmaf(z[8 * gq + 2 * i], zf, -mref));
                        const float p1 = exp2f(fmaf(z[8 * gq + 2 * i + 1], zf, -mref));
                        ls += p0 + p1;
                        pk[i] = pack_f16x2(p0, p1);
                    }
                    *reinterpret_cast<uint4 *>(Pb + swz((uint32_t)hl, (uint32_t)(4 * u + gq))) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
                lsum += ls;
                fence_async_smem();
                tc_fence_before();
                warp_arrive(&ms.p_full[p]);
            }
            lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);   // the row's two halves
            if (u == 0 && hl < pc.rows) {
                if (pc.first && pc.last) {
                    // a row that sees nothing: out = 0, lse = -inf (a NaN sum stays NaN)
                    ms.inv[hl] = lsum == 0.f ? 0.f : 1.f / lsum;
                    a.lse[pc.row + hl] = lsum == 0.f ? -INFINITY : (m_run - kPOffset) * kLn2 + logf(lsum);
                } else {
                    const int slot = 2 * (int)blockIdx.x + (pc.first ? 1 : 0);
                    a.part_ml[(size_t)slot * kDenseRows + hl] = make_float2(m_run - kPOffset, lsum);
                }
            }
        }
        // ---- epilogue: O^T, M-tile w/4, quarter w%4, by warps 0-15
        if (nk > 0) {
            const uint32_t gl = g0 + nk - 1;
            ok = ok && warp_wait(&ms.v_free[gl % kDnStages], (gl / kDnStages) & 1u, &ms.abort_flag, a.ws, 8);
        }
        ok = bar_and(4, kDnThreads, ok);
        if (tid < kDenseRows) ms.qmax[tid] = 0u;
        if (ok && warp < 16) {
            tc_fence_after();
            const int m = warp >> 2, qq = warp & 3, ch = 128 * m + 32 * qq + lane;
            const bool whole = pc.first && pc.last;
            float *po = a.part_o + ((size_t)(2 * blockIdx.x + (pc.first ? 1 : 0)) * kDenseRows) * kLatent + ch;
            uint32_t *out = reinterpret_cast<uint32_t *>(a.out + (size_t)pc.row * kLatent + (ch & ~1));
#pragma unroll
            for (int hq = 0; hq < kDenseRows; hq += 16) {
                float o[16];
                if (nk > 0) {
                    tc_ld16_sync(tmem + ((uint32_t)(32 * qq) << 16) + kDnColO + 64 * m + hq, o);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[i] = 0.f;
                }
                if (!whole) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (hq + i < pc.rows) po[(size_t)(hq + i) * kLatent] = o[i];
                } else {
                    // lanes 2l and 2l + 1 exchange one row each, so that both store a channel pair
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        const float x0 = o[i] * ms.inv[hq + i], x1 = o[i + 1] * ms.inv[hq + i + 1];
                        const float other = __shfl_xor_sync(0xffffffffu, (lane & 1) ? x0 : x1, 1);
                        const int r = hq + i + (lane & 1);
                        __nv_bfloat162 v = (lane & 1) ? __floats2bfloat162_rn(other, x1) : __floats2bfloat162_rn(x0, other);
                        if (r < pc.rows) out[(size_t)r * (kLatent / 2)] = *reinterpret_cast<uint32_t *>(&v);
                    }
                }
            }
        }
        if (nk > 0) {
            g0 += nk;
            ++pieces;
        }
    }
    if (tid == 0) a.share[blockIdx.x] = ms.share;
    if (warp >= kDnIssuerWarp && lane == 0) {
        // every MMA this thread issued has completed before TMEM is released
        tc_commit(smem_addr(&ms.final_bar[warp - kDnIssuerWarp]));
        volatile int no_abort = 0;
        mbar_wait(&ms.final_bar[warp - kDnIssuerWarp], 0, &no_abort, a.ws, 4);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kDnIssuerWarp) tc_dealloc(ms.tmem_base, kDnTmemCols);
}

// ------------------------------------------------------------------------------------------------
// Combine: out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i over the parts of a shared row tile, in CTA
// order.  CTA (c, y) takes rows 8y .. 8y+7 of the row tile that CTA c of the attention began and did
// not finish, one warp per row.
// ------------------------------------------------------------------------------------------------
constexpr int kCombineRows = 8;

__global__ void __launch_bounds__(32 * kCombineRows) dense_combine_kernel(DenseArgs a)
{
    __shared__ int slots[kDenseCtas + 1];
    __shared__ int first_end, counts[kCombineRows];
    __shared__ float wgt[kCombineRows][kDenseCtas + 1];
    grid_dep_wait();     // every part
    grid_dep_launch();   // a dependent kernel launched after this one waits for it before reading
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const DenseShare tail = a.share[c];
    const int r = kCombineRows * blockIdx.y + warp;
    if (tail.tail_rows <= kCombineRows * (int)blockIdx.y) return;
    // the parts: the tail of CTA c, then the heads of the CTAs behind it up to the one that ends the tile
    if (tid == 0) first_end = kDenseCtas;
    __syncthreads();
    const int o = c + 1 + tid;
    DenseShare sh{};
    if (o < kDenseCtas) sh = a.share[o];
    if (sh.head && sh.head_ends) atomicMin(&first_end, o);
    __syncthreads();
    const bool part = sh.head && o <= first_end;
    const unsigned vote = __ballot_sync(0xffffffffu, part);
    if (lane == 0) counts[warp] = __popc(vote);
    __syncthreads();
    int at = 1, n = 1;
    for (int w = 0; w < kCombineRows; ++w) {
        if (w < warp) at += counts[w];
        n += counts[w];
    }
    if (tid == 0) slots[0] = 2 * c + 1;
    if (part) slots[at + __popc(vote & ((1u << lane) - 1u))] = 2 * o;
    __syncthreads();
    if (r >= tail.tail_rows) return;
    float M = -INFINITY;
    for (int i = lane; i < n; i += 32) M = fmaxf(M, a.part_ml[(size_t)slots[i] * kDenseRows + r].x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    float den = 0.f;
    for (int i = lane; i < n; i += 32) {
        const float2 ml = a.part_ml[(size_t)slots[i] * kDenseRows + r];
        const float w = exp2f(ml.x - M);
        wgt[warp][i] = w;
        den = fmaf(w, ml.y, den);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) den += __shfl_xor_sync(0xffffffffu, den, d);
    __syncwarp();
    float4 acc[4] = {};
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
        const float4 *po = reinterpret_cast<const float4 *>(a.part_o + ((size_t)slots[i] * kDenseRows + r) * kLatent) + lane;
        const float w = wgt[warp][i];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = po[32 * j];
            acc[j].x = fmaf(w, v.x, acc[j].x);
            acc[j].y = fmaf(w, v.y, acc[j].y);
            acc[j].z = fmaf(w, v.z, acc[j].z);
            acc[j].w = fmaf(w, v.w, acc[j].w);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint2 *out = reinterpret_cast<uint2 *>(a.out + (size_t)(tail.tail_row + r) * kLatent) + lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        __nv_bfloat162 x = __floats2bfloat162_rn(acc[j].x * inv, acc[j].y * inv);
        __nv_bfloat162 y = __floats2bfloat162_rn(acc[j].z * inv, acc[j].w * inv);
        out[32 * j] = make_uint2(*reinterpret_cast<uint32_t *>(&x), *reinterpret_cast<uint32_t *>(&y));
    }
    if (lane == 0) a.lse[tail.tail_row + r] = den == 0.f ? -INFINITY : M * kLn2 + logf(den);
}

cudaError_t launch_dense_attn(const DenseArgs &a, cudaStream_t st)
{
    static_assert(kDnSmem <= 232448, "shared memory budget");
    static_assert(32 * kCombineRows >= kDenseCtas, "one thread per CTA behind the tail");
    cudaError_t e = allow_dynamic_smem(reinterpret_cast<const void *>(dense_attn_kernel), kDnSmem);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(dense_attn_kernel, dim3(kDenseCtas), dim3(kDnThreads), kDnSmem, st, a);
    if (e != cudaSuccess) return e;
    return launch_overlapped(dense_combine_kernel, dim3(kDenseCtas, kDenseRows / kCombineRows), dim3(32 * kCombineRows), 0,
                             st, a);
}

}  // namespace csa
