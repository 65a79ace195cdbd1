// dense_attn.cu -- attention of ragged query runs over the whole paged FP4 cache, on the sm_100a tensor
// cores (tcgen05, TMEM).
//
// yomxxx.com long-form post on KV-cache compression limits, section 五 (a fixed layout with addresses from
// the token index, dequantised in the kernel, in parallel); rebasdaily article on DeepSeek-V4.1-Flash KV
// compression, section "同一份笔记，多层一起用" (FP4 main KV; the 512-channel latent is key and value).
//
// Row tile: 128 consecutive (token, head) rows of one sequence, token-major, so that the 128 heads of one
// token, 16 heads of eight drafted tokens or 64 heads of two prompt tokens fill the same matrix operand and
// any head count works.  Cache tile: one 64-position page.  The fp32 output of 128 rows x 512 channels alone
// would fill a TMEM, so a row tile belongs to a cluster of two CTAs, each with half of the channels: CTA x
// dequantises channels 256x .. 256x+255 of a page (fp16, exact) and for every (row tile, page) computes
//   QK:  S_x[128 rows x 64 entries] = Q_x . V_x^T     (M = 128, N = 64; A = Q_x in TMEM, B = V_x K-major);
//   each CTA adds and exponentiates the two partial scores of half of the rows (half of S_x goes to the other
//   CTA's shared memory, half of P comes back from there);
//   PV:  O_x[128 rows x 256 ch] += P . V_x            (M = 128, N = 256; A = P K-major, B = V_x MN-major).
// Every MMA runs at the tensor cores' full rate (M = 128), a page is dequantised once per 128 rows, and no
// byte of V crosses between the CTAs.
//
// Numerics: fp16 operands (exact for the entries; P rounded to fp16 once), fp32 accumulation and sums.  Q is
// scaled by a power of two per row and channel half, so a row of very large or non-finite values does not
// touch the others of its tile.  O is rescaled only when a row's maximum has grown by 2^8.
//
// Work division: the (row tile, page) pairs of the whole call, row tile by row tile, are one line (on which a row
// tile also takes the length of kDnPieceCost pages) that the 74 persistent clusters, one CTA per SM, cut into equal
// shares, whatever the batch looks like: one long sequence splits over all SMs, a prefill chunk gives each cluster
// whole row tiles.  Every CTA works out the division itself from cu_rows, seq_len and the spans (a block scan; no extra
// launch).  A cluster finishes the row tiles it holds whole; the first and last tile of its share may be shared with
// its neighbours, and those leave an fp32 partial (unnormalised O, running maximum and sum) in the workspace, which
// the combine kernel adds in cluster order, so results do not depend on timing.
//
// What bounds it.  A (row tile, page) pair needs 1,036 tensor cycles (QK 512, PV 524); it takes about 2,300, which is
// half of the softmax's chain (read S, send, receive, maximum, exp2, P to both CTAs, PV, P buffer free: 4,600 cycles):
// two groups of warps take the tiles in turn, and a third does not fit the two S and P buffers that TMEM and shared
// memory leave.  A row tile costs 16,000 cycles more (Q into TMEM, the last tiles' chain, O out), and a call 15 us before
// and after (plan, first pages, partials, combine).  Measured: 2,048 rows of 64 heads behind 14,336 positions 4.3-4.5 ms
// (0.92-0.95 PFLOP/s, at the power limit); one row of each of 8 sequences of 131,072 positions, 64 heads (half of the tensor
// rows idle): 270-279 us; one row of 16 heads over 4,096 positions: 23 us.
#include <cuda_bf16.h>

#include "attention_tile.cuh"
#include "cluster.cuh"
#include "convert.cuh"
#include "dense_attn.cuh"
#include "tensor_map.cuh"

namespace csa {

constexpr int kTile = 64;                        // entries per tile: one page
constexpr int kDnCh = kLatent / 2;               // channels of a CTA
constexpr int kDnStages = 4;                     // V tiles in flight
constexpr int kDnPStages = 2;                    // P tiles
constexpr int kDnRawStages = 3;                  // tiles as the cache holds them
constexpr int kDnFlags = 8;                      // tiles whose page is known to be valid or not
constexpr int kDnGroups = 2;                     // tiles in their softmax at a time
constexpr int kDnProducerWarps = 4;              // warps 0-3
constexpr int kDnScoreWarp = 4;                  // warps 4-11: groups of four, one per TMEM quarter
constexpr int kDnMmaWarp = kDnScoreWarp + 4 * kDnGroups;    // warps 12-15: PV, QK, next piece; each rescales a quarter of O
constexpr int kDnPvWarp = kDnMmaWarp, kDnQkWarp = kDnMmaWarp + 1, kDnPlanWarp = kDnMmaWarp + 2;
constexpr int kDnThreads = 32 * (kDnMmaWarp + 4);          // 128 registers each: a spill is a miss in the 20 KB of L1 left
constexpr uint32_t kDnFailed = 0xFFFFFFFFu;
constexpr uint32_t kDnVChunk = kTile * 128;              // 8 KB: 64 entries x 64 fp16
constexpr uint32_t kDnVBuf = kDnCh / 64 * kDnVChunk;     // 32 KB per tile buffer
constexpr uint32_t kDnPBuf = kDenseRows * 128;           // 16 KB: 128 rows x 64 entries fp16
constexpr uint32_t kDnRBuf = kDenseRows / 2 * kTile * 4; // 16 KB: 64 rows x 64 entries fp32
constexpr uint32_t kDnRawCodes = kTile * kDnCh / 2;      // 8 KB: 64 entries x 256 channels of FP4
constexpr uint32_t kDnRawScales = kTile * kDnCh / 16;    // 1 KB: their scales
constexpr uint32_t kDnOffP = kDnStages * kDnVBuf;
constexpr uint32_t kDnOffR = kDnOffP + kDnPStages * kDnPBuf;
constexpr uint32_t kDnOffC = kDnOffR + kDnGroups * kDnRBuf;
constexpr uint32_t kDnOffSc = kDnOffC + kDnRawStages * kDnRawCodes;
constexpr uint32_t kDnOffMisc = kDnOffSc + kDnRawStages * kDnRawScales;
constexpr uint32_t kDnTmemCols = 512;
constexpr uint32_t kDnColO = 0;                  // O_x: 256 channels
constexpr uint32_t kDnColQ = 256;                // Q_x: 256 channels, two per column
constexpr uint32_t kDnColS = 384;                // S_x of tile g: columns 384 + 64(g%2) ..
constexpr long long kDnMinTiles = 4;             // a cluster's least share of the line, in pages (a row tile's fixed kDnPieceCost
                                                 // counted, so a share inside that has no page: of a tile of 64 pages, 18
                                                 // shares, 16 clusters take pages).  That tile: 23.2 us; 2: 24.6; 8: 25.6
constexpr int kDnPieceCost = 8;                  // what a row tile costs besides its pages, in pages
constexpr float kDnNoMax = -3.402823466e38f;     // reference of a row that has seen nothing: no finite score is below it
static_assert(kTile == kPage, "a tile is one page");
static_assert(kDnStages * kDnVBuf >= kDenseRows * kDnCh * 2, "Q is staged in the V buffers");

// One cluster's part of one row tile.
struct DensePiece {
    long long row;       // first row of the row tile over the call (token * H + head)
    uint32_t r0;         // the same within the sequence
    int rows;            // rows of the row tile, 1 .. 128; 0: the cluster has no further piece
    int b, c0, n, L;     // sequence, its first token, tokens and length
    int kv0, kv1;        // pages [kv0, kv1) of this piece; none if no row of the tile sees anything
    int first, last;     // the piece holds the first / last of the row tile's pages
};

// Where a cluster is on the line of (row tile, page) pairs.
struct DenseCursor {
    long long left;      // pairs of its share still to take
    long long off;       // pairs of row tile `tile` before them
    int tile, b;
};

// Tensor maps of the cache as [num_pages][64 entries][bytes]: boxes of 64 entries x one CTA's channels.
struct DenseMaps {
    CUtensorMap codes, scales;
};

struct DenseMisc {
    DenseArgs args;
    uint64_t raw_full[kDnRawStages], raw_free[kDnRawStages];
    uint64_t v_ready[kDnStages], v_free[kDnStages];
    uint64_t s_full[2], s_free[2];
    uint64_t r_full[kDnGroups][4];          // scores received, by softmax warp
    uint64_t r_free[kDnGroups][4];          // the other CTA has read those sent to it
    uint64_t p_full[kDnPStages], p_free[kDnPStages];
    uint64_t planned;                       // the next piece is known
    uint64_t go, c_done;                    // O is to be rescaled (or the piece is over); it has been
    uint64_t m_full[kDnGroups][4];          // rows' references after a tile, by softmax warp
    uint64_t inv_full;
    uint64_t final_bar[2];
    uint32_t nan_mask[kDnStages][kDnProducerWarps];    // entries with a NaN scale: bits of 32 entries per producer warp
    uint4 flags[kDnStages];                            // entries with a NaN scale (two words), page valid
    uint32_t go_slot;                                  // P buffer of the tile to rescale for, kDnFailed at the end
    int page_ok[kDnFlags];                             // the page id of tile g % 8 is valid
    uint32_t tmem_base;
    uint32_t rescales;                                 // of O so far
    int abort_flag;
    long long warp_sum[kDnThreads / 32];
    DensePiece piece[2];
    DenseCursor cur;
    DenseShare share;
    float zs[kDenseRows];                   // accumulated score -> log2 domain, per row
    float m_row[kDnGroups][kDenseRows / 2]; // the references
    float2 ml[kDnGroups][kDenseRows / 2];   // each group's reference and sum of p at the end of a piece
    alignas(16) float alpha[kDnPStages][kDenseRows];   // rescale factor of each row before a tile
    float inv[kDenseRows];                  // 1 / denominator of a finished row
};

constexpr size_t kDnSmem = kDnOffMisc + sizeof(DenseMisc) + 1024;
constexpr uint32_t kDnIdescQK = umma_idesc_f16(kDenseRows, kTile, false, false);
constexpr uint32_t kDnIdescPV = umma_idesc_f16(kDenseRows, kDnCh, false, true);

// Named barriers: 1 + q = the score warps of quarter q.

// Load of data that is read once: past the L1.
__device__ __forceinline__ uint4 ld_stream16(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void prefetch_l2(const void *p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ------------------------------------------------------------------------------------------------
// Work division.  Sequence b's row tiles have the numbers tile_base(b) .. tile_base(b + 1) - 1: at least
// ceil(n_b H / 128) of them, the rest empty, without a scan over the batch.
// ------------------------------------------------------------------------------------------------
__device__ __forceinline__ long long tile_base(int c0, int b, int H) { return (long long)c0 * H / kDenseRows + b; }

// Pages [kv0, kv0 + nk) that the rows of row tile r0 of a sequence see between them.
__device__ __forceinline__ void tile_pages(const DenseArgs &a, int c0, int n, int L, uint32_t r0, int &kv0, int &nk)
{
    const int ta = (int)(r0 / (uint32_t)a.H);
    const int tb = min((int)((r0 + kDenseRows - 1) / (uint32_t)a.H), n - 1);
    int lo = 0, hi = L - n + tb + 1;
    if (a.spans) {
        lo = L;
        hi = 0;
#pragma unroll 8
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

// Share of the line that row tile r0 of a sequence takes: kDnPieceCost, then its pages; 0 for a tile number
// without rows or a sequence left out.
__device__ __forceinline__ int tile_weight(const DenseArgs &a, int c0, int n, int L, uint32_t r0)
{
    if (L < n || r0 >= (uint32_t)n * (uint32_t)a.H) return 0;
    int kv0, nk;
    tile_pages(a, c0, n, L, r0, kv0, nk);
    return kDnPieceCost + nk;
}

// The next piece of the cluster's share, and what the share leaves unfinished.
__device__ void next_piece(const DenseArgs &a, const int32_t *cu_rows, const int32_t *seq_len, DenseCursor &cu, DenseShare &share,
                           DensePiece &pc)
{
    pc.rows = 0;
    while (cu.left > 0) {
        const int c0 = cu_rows[cu.b], c1 = cu_rows[cu.b + 1], n = c1 - c0;
        if (cu.tile >= tile_base(c1, cu.b + 1, a.H)) {
            if (++cu.b >= a.B) return;
            continue;
        }
        int L = seq_len[cu.b];
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
        const int k0 = (int)max(0ll, cu.off - kDnPieceCost), k1 = (int)max(0ll, cu.off + take - kDnPieceCost);
        const bool last = cu.off + take == w;
        cu.left -= take;
        cu.off = 0;
        ++cu.tile;
        if (k1 == k0 && !(nk == 0 && last)) continue;   // the share ends before the row tile's pages
        pc.row = (long long)c0 * a.H + r0;
        pc.r0 = r0;
        pc.rows = (int)min((uint32_t)kDenseRows, (uint32_t)n * (uint32_t)a.H - r0);
        pc.b = cu.b;
        pc.c0 = c0;
        pc.n = n;
        pc.L = L;
        pc.kv0 = kv0 + k0;
        pc.kv1 = kv0 + k1;
        pc.first = k0 == 0;
        pc.last = last;
        if (!pc.first) {
            share.head = 1;
            share.head_ends = pc.last;
        } else if (!pc.last) {
            share.tail_row = pc.row;
            share.tail_rows = pc.rows;
        }
        return;
    }
}

// This cluster's share: block-wide sums of the row tiles' weights, each thread over consecutive tiles, then
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
    long long sums = lane < kDnThreads / 32 ? ms.warp_sum[lane] : 0;   // inclusive, over the warps
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, sums, d);
        if (lane >= d) sums += o;
    }
    const long long total = __shfl_sync(0xffffffffu, sums, 31);
    const long long excl = (warp > 0 ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0) + incl - sum;
    // as many clusters as leave each kDnMinTiles pages
    const long long pairs = max(1ll, min((long long)gridDim.x / 2, total / kDnMinTiles));
    const int pair = blockIdx.x >> 1;
    if (pair < pairs) {
        // shares of total / pairs, the first total % pairs of them one longer
        const long long each = total / pairs, more = total - each * pairs;
        const long long s = each * pair + min((long long)pair, more), e = s + each + (pair < more ? 1 : 0);
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
            next_piece(a, s_cu, s_len, ms.cur, ms.share, ms.piece[0]);
        }
    }
}

// ------------------------------------------------------------------------------------------------
// A producer thread's share of one page: entry e, 128 channels (half cp of this CTA's).  TMA brings the raw
// bytes, 64 B of codes (16-byte units swizzled as V's) and 8 scale bytes, three tiles ahead.
// ------------------------------------------------------------------------------------------------
struct PageEntry {
    uint4 code[4];
    uint2 sc;
    bool valid;

    __device__ __forceinline__ void read(const uint8_t *codes, const uint8_t *scales, int e, int cp)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) code[i] = *reinterpret_cast<const uint4 *>(codes + swz((uint32_t)e, (uint32_t)(4 * cp + i)));
        sc = *reinterpret_cast<const uint2 *>(scales + 16 * e + 8 * cp);
    }

    // One of the eight scales is NaN (E4M3 0x7F or 0xFF).
    __device__ __forceinline__ bool has_nan() const
    {
        return valid && ((((sc.x & 0x7F7F7F7Fu) + 0x01010101u) | ((sc.y & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u) != 0;
    }

    // Channels 32c .. 32c + 31 as 16 fp16 pairs; zeros for an invalid or NaN entry.
    __device__ __forceinline__ void dequant(int c, bool ok, uint32_t *v) const
    {
        uint32_t sh[2];   // the four group scales of 64 channels as (s0, s1), (s2, s3)
        e4m3x4_to_f16x2x2(c & 2 ? sc.y : sc.x, sh);
        const uint32_t s01 = ok ? sh[c & 1] : 0u;
        const uint4 cw = code[c];
#pragma unroll
        for (int gg = 0; gg < 2; ++gg) {
            const uint32_t s2 = __byte_perm(s01, 0u, gg ? 0x3232u : 0x1010u);
            uint32_t c0[4], c1[4];
            e2m1x8_to_f16x2x4(gg ? cw.z : cw.x, c0);
            e2m1x8_to_f16x2x4(gg ? cw.w : cw.y, c1);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[8 * gg + q] = hmul2_u32(c0[q], s2);
                v[8 * gg + 4 + q] = hmul2_u32(c1[q], s2);
            }
        }
    }
};

// This CTA's channels of the row tile's Q into `stage`, each row scaled by the power of two 2^k that puts its
// largest |q| of these channels in [2^13, 2^14), 16-byte units swizzled; ms.zs gets tau * log2(e) * 2^-k.
// Warp w: the rows of lanes 8w .. 8w+7 (a row per load, 512 contiguous bytes); zeros past the row tile's rows.
template <typename F>
__device__ __forceinline__ void stage_q(const DenseArgs &a, DenseMisc &ms, const DensePiece &pc, int x, uint8_t *stage, F between)
{
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint4 qw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int r = 8 * w + j;
        qw[j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < pc.rows) qw[j] = ld_stream16(a.q + (size_t)(pc.row + r) * kLatent + kDnCh * x + 8 * lane);
    }
    between();   // the rows are on their way
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int i = 8 * w + j;
        const uint32_t ww[4] = {qw[j].x, qw[j].y, qw[j].z, qw[j].w};
        uint32_t top = 0u;   // largest |q| as bf16 bits in the upper half
#pragma unroll
        for (int k = 0; k < 4; ++k) top = max(top, max(ww[k] & 0x7FFF0000u, (ww[k] << 16) & 0x7FFF0000u));
        top = __reduce_max_sync(0xffffffffu, top);
        int k = 0;
        if (top != 0u) {
            k = 13 - ((int)(top >> 23) - 127);
            k = k < -120 ? -120 : (k > 120 ? 120 : k);
        }
        const float sc = __int_as_float((127 + k) << 23);
        uint32_t h[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) h[m] = pack_f16x2(bf16_lo(ww[m]) * sc, bf16_hi(ww[m]) * sc);
        *reinterpret_cast<uint4 *>(stage + i * 512 + ((lane ^ (i & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        // a row of non-finite q is NaN whatever its products are
        if (lane == 0) ms.zs[i] = top >= 0x7F800000u ? __int_as_float(0x7FC00000) : a.sm_scale * __int_as_float((127 - k) << 23) * kLog2e;
    }
}

// The staged rows into TMEM as the A operand of the QK MMAs: warp w stores quarter w%4, channels 64(w/4) ..
__device__ __forceinline__ void store_q(const uint8_t *stage, uint32_t tmem)
{
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int q = w & 3, cg = w >> 2, i = 32 * q + lane;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        uint32_t v[16];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int unit = 8 * cg + 4 * j + k;
            const uint4 y = *reinterpret_cast<const uint4 *>(stage + i * 512 + ((unit ^ (i & 7)) << 4));
            v[4 * k] = y.x;
            v[4 * k + 1] = y.y;
            v[4 * k + 2] = y.z;
            v[4 * k + 3] = y.w;
        }
        tc_st16_u(tmem + ((uint32_t)(32 * q) << 16) + kDnColQ + 32 * cg + 16 * j, v);
    }
    tc_wait_st();
}

__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// c tanh(s / c) in the log2 domain, z = s log2(e), arg = 2 / c, cap = c log2(e).  With x = s / c and w = z arg = 2x log2(e):
//   |x| < 0.25: z (1 + x^2 (-1/3 + x^2 (2/15 - x^2 17/315))), the series of tanh (next term below 2^-21);
//   otherwise cap (1 - 2 / (1 + 2^w)), whose error of a few 2^-23 cap is then below 2^-19 of the result.
// So the error goes by the score, not by the cap: a cap far above the scores leaves them as they are.
constexpr float kCapSmall = 0.72f;   // |w| below it: the series

__device__ __forceinline__ float cap_small(float z, float w)
{
    constexpr float kX2 = kLn2 * kLn2 / 4.f;   // x^2 / w^2
    const float u = w * w;
    return fmaf(z, u * fmaf(u, fmaf(u, -17.f / 315.f * kX2 * kX2 * kX2, 2.f / 15.f * kX2 * kX2), -1.f / 3.f * kX2), z);
}

// The 32 scores of every lane of a warp.  Where all are small, as ordinary caps leave them, the series alone, without the two
// special functions: 23 rows of six sequences of 50,021 positions 128 us (146 where scores pass a quarter of the cap; both
// forms and a choice for every score: 137 and 140).
__device__ __forceinline__ void cap_scores(float *z, float softcap)
{
    const float arg = 2.f / softcap, cap = softcap * kLog2e;
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = fmaxf(top, fabsf(z[i]));   // a NaN passes through either form
    if (__all_sync(0xffffffffu, top * arg < kCapSmall)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = cap_small(z[i], z[i] * arg);
    } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const float w = z[i] * arg;
            z[i] = fabsf(w) < kCapSmall ? cap_small(z[i], w) : fmaf(-2.f * cap, rcp(1.f + ex2(w)), cap);
        }
    }
}

__device__ __forceinline__ uint8_t *dense_smem()
{
    extern __shared__ uint8_t smem_raw[];
    return reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

__device__ __forceinline__ DenseMisc &dense_misc(uint8_t *base) { return *reinterpret_cast<DenseMisc *>(base + kDnOffMisc); }

__device__ __forceinline__ WaitCtx dense_wait(DenseMisc &ms) { return WaitCtx{smem_addr(&ms.abort_flag)}; }

// ------------------------------------------------------------------------------------------------
// Roles of the warps while a piece runs.  Each is a function of its own: the register allocation of one
// does not see what the others keep, and nothing is spilled inside a tile loop (the L1 beside 200 KB of
// shared memory holds no stack: a reload costs an L2 access).  They return false after a failed wait.
// ------------------------------------------------------------------------------------------------
// This warp's quarter of O times the rescale factors of the tile in P buffer pp, PV of the tile before having completed.
__device__ __forceinline__ void dense_rescale(DenseMisc &ms, uint32_t tmem, int q, uint32_t pp)
{
    const float al = ms.alpha[pp][32 * q + (threadIdx.x & 31)];
    const uint32_t to = tmem + ((uint32_t)(32 * q) << 16) + kDnColO;
    tc_fence_after();
#pragma unroll 1
    for (int k = 0; k < kDnCh; k += 32) {
        float o[32];
        tc_ld32_sync(to + k, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= al;
        tc_st32(to + k, o);
    }
    tc_wait_st();
    tc_fence_before();
}

// PV of every tile, once its P has come from both CTAs and O is at its scale; the commits release the tile's V buffer
// and, in both CTAs, its P buffer.  When a row's maximum has grown, the four MMA warps rescale O first.
__device__ __noinline__ bool dense_pv(int pi, uint32_t g0)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DensePiece &pc = ms.piece[pi];
    const int lane = threadIdx.x & 31, nk = pc.kv1 - pc.kv0, rows = pc.rows;
    const WaitCtx cx = dense_wait(ms);
    const uint32_t tmem = ms.tmem_base;
    const uint64_t p_desc = umma_sdesc_sw128(smem_addr(base) + kDnOffP, 16, 1024);
    const uint64_t v_desc = umma_sdesc_sw128(smem_addr(base), kDnVChunk, 1024);
    uint32_t rescales = ms.rescales;
    bool ok = true;
#pragma unroll 1
    for (int t = 0; t < nk; ++t) {
        const uint32_t g = g0 + t, p = g % kDnStages, pp = g % kDnPStages;
        ok = warp_wait_hint(&ms.p_full[pp], (g / kDnPStages) & 1u, cx, 7);
        if (!ok) break;
        if (t > 0) {
            const float4 al = reinterpret_cast<const float4 *>(ms.alpha[pp])[lane];   // rows 4 lane ..
            const bool one = al.x == 1.f && al.y == 1.f && al.z == 1.f && al.w == 1.f;
            if (__any_sync(0xffffffffu, !one && (4 * lane & ~31) < rows)) {
                const uint32_t gp = g - 1u;
                ok = warp_wait_hint(&ms.v_free[gp % kDnStages], (gp / kDnStages) & 1u, cx, 13);
                if (!ok) break;
                if (lane == 0) ms.go_slot = pp;
                __syncwarp();
                lane0_arrive(&ms.go, lane);
                dense_rescale(ms, tmem, kDnPvWarp & 3, pp);
                ok = warp_wait_hint(&ms.c_done, rescales & 1u, cx, 12);
                if (!ok) break;
                ++rescales;
            }
        }
        tc_fence_after();
        // descriptor addresses count 16-byte units
        const uint64_t ad = p_desc + pp * (kDnPBuf >> 4), bd = v_desc + p * (kDnVBuf >> 4);
        if (elect_lane()) {
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
                tc_mma_f16(tmem + kDnColO, ad + 2 * kk, bd + 128 * kk, kDnIdescPV, (t > 0 || kk > 0) ? 1u : 0u);
            tc_commit_both(smem_addr(&ms.p_free[pp]));
            tc_commit(smem_addr(&ms.v_free[p]));
        }
        __syncwarp();
    }
    if (lane == 0) {
        ms.go_slot = kDnFailed;   // the other MMA warps are done too
        ms.rescales = rescales;
    }
    __syncwarp();
    lane0_arrive(&ms.go, lane);
    return ok;
}

// The other MMA warps: QK of every tile and the next piece, by one of them each, and rescaling of their quarter of O
// when the PV warp asks.  n_go counts its requests.
__device__ __noinline__ uint32_t dense_mma(int pi, uint32_t g0, uint32_t n_go)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DensePiece &pc = ms.piece[pi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nk = pc.kv1 - pc.kv0;
    const WaitCtx cx = dense_wait(ms);
    const uint32_t tmem = ms.tmem_base;
    const uint64_t v_desc = umma_sdesc_sw128(smem_addr(base), 16, 1024);
    if (warp == kDnPlanWarp) {
        if (lane == 0) next_piece(ms.args, ms.args.cu_rows, ms.args.seq_len, ms.cur, ms.share, ms.piece[pi ^ 1]);
        __syncwarp();
        lane0_arrive(&ms.planned, lane);
        // its Q rows to the L2: this CTA's half of each is four lines
        const DensePiece &nx = ms.piece[pi ^ 1];
        const uint16_t *src = ms.args.q + (size_t)nx.row * kLatent + kDnCh * (int)cluster_rank() + 64 * (lane & 3);
        for (int r = lane >> 2; r < nx.rows; r += 8) prefetch_l2(src + (size_t)r * kLatent);
    }
    __syncwarp();
    // a request of the PV warp: false at the end of the piece
    auto serve = [&]() {
        ++n_go;
        const uint32_t pp = ms.go_slot;
        if (pp == kDnFailed) return false;
        dense_rescale(ms, tmem, warp & 3, pp);
        __syncwarp();
        lane0_arrive(&ms.c_done, lane);
        return true;
    };
    if (warp == kDnQkWarp) {
        // waits for a barrier and serves requests meanwhile (testing: a try_wait would sleep through them)
        auto wait_serving = [&](uint64_t *bar, uint32_t parity) {
            if (mbar_test_wait(bar, parity)) return true;
            const uint32_t t0 = global_ns_lo();
#pragma unroll 1
            do {
                if (mbar_test_wait(bar, parity)) return true;
                if (mbar_test_wait(&ms.go, n_go & 1u) && !serve()) return false;
                if (*(volatile int *)&ms.abort_flag) return false;
            } while (global_ns_lo() - t0 < (uint32_t)kWaitLimitNs);
            ms.abort_flag = 3;
            return false;
        };
#pragma unroll 1
        for (int t = 0; t < nk; ++t) {
            const uint32_t g = g0 + t, p = g % kDnStages, sb = g & 1u;
            // QK into S of tile g (columns of parity g % 2) once the producers have written the tile and the score warps
            // have read tile g - 2's scores
            if (!wait_serving(&ms.v_ready[p], (g / kDnStages) & 1u)) return kDnFailed;
            if (g >= 2 && !wait_serving(&ms.s_free[sb], ((g >> 1) - 1u) & 1u)) return kDnFailed;
            if (lane == 0) {
                ms.flags[p] = make_uint4(ms.nan_mask[p][0] | ms.nan_mask[p][2], ms.nan_mask[p][1] | ms.nan_mask[p][3],
                                         (uint32_t)ms.page_ok[g % kDnFlags], 0u);
                mbar_arrive(&ms.s_full[sb]);   // the flags; the scores by the commit
            }
            __syncwarp();
            tc_fence_after();
            const uint64_t bd = v_desc + p * (kDnVBuf >> 4);
            const uint32_t sc = tmem + kDnColS + 64 * sb;
            if (elect_lane()) {
#pragma unroll
                for (int k = 0; k < kDnCh / 16; ++k)
                    tc_mma_f16_ts(sc, tmem + kDnColQ + 8 * k, bd + (k >> 2) * (kDnVChunk >> 4) + 2 * (k & 3), kDnIdescQK, k > 0 ? 1u : 0u);
                tc_commit(smem_addr(&ms.s_full[sb]));
            }
            __syncwarp();
        }
    }
    for (;;) {
        if (!warp_wait_hint(&ms.go, n_go & 1u, cx, 10)) return kDnFailed;
        if (!serve()) return n_go;
    }
}

// The order of a piece's pages: with a distance bias from the last to the first, so that the newest positions set the
// rows' references and O is hardly ever rescaled (23 rows of six sequences of 50,021 positions: 129 us, upwards 167);
// otherwise upwards, so that the page that causal rows see in part comes last (no difference beyond the noise: 2,048
// rows behind 14,336 positions 4.44-4.52 ms, downwards 4.53).
struct PageOrder {
    int first, step;
    __device__ __forceinline__ PageOrder(const DenseArgs &a, const DensePiece &pc)
        : first(a.slopes ? pc.kv1 - 1 : pc.kv0), step(a.slopes ? -1 : 1)
    {
    }
    __device__ __forceinline__ int page(int t) const { return first + step * t; }
};

// Page of tile t to shared memory, by warp 0; `ids` holds the page ids of tiles t & ~31 ..
__device__ __forceinline__ void dense_fetch(const DenseArgs &a, DenseMisc &ms, const DenseMaps *maps, uint8_t *base, int ids, int t,
                                            uint32_t g, int where)
{
    const int page = __shfl_sync(0xffffffffu, ids, t & 31);
    if (elect_lane()) {
        const uint32_t st = g % kDnRawStages;
        const bool ok = page >= 0 && page < a.num_pages;
        ms.page_ok[g % kDnFlags] = ok;
        if (ok) {
            mbar_arrive_expect_tx(&ms.raw_full[st], kDnRawCodes + kDnRawScales);
            const int x = (int)cluster_rank();
            tma_load_3d(smem_addr(base + kDnOffC + st * kDnRawCodes), &maps->codes, 128 * x, 0, page, &ms.raw_full[st]);
            tma_load_3d(smem_addr(base + kDnOffSc + st * kDnRawScales), &maps->scales, 16 * x, 0, page, &ms.raw_full[st]);
        } else {
            report(a.ws, CSA_ERR_DEVICE_DATA, where);
            mbar_arrive(&ms.raw_full[st]);
        }
    }
    __syncwarp();
}

// The first two pages of a piece, ahead of everything else (warp 0).
__device__ __forceinline__ bool dense_prefetch(const DenseArgs &a, DenseMisc &ms, const DenseMaps *maps, uint8_t *base,
                                               const DensePiece &pc, uint32_t g0)
{
    const int nk = pc.kv1 - pc.kv0, lane = threadIdx.x & 31;
    const PageOrder po(a, pc);
    const WaitCtx cx = dense_wait(ms);
    const int ids = lane < min(nk, 2) ? a.block_table[(size_t)pc.b * a.max_pages + po.page(lane)] : -1;
    for (int t = 0; t < min(nk, 2); ++t) {
        const uint32_t g = g0 + t;
        if (g >= kDnRawStages && !warp_wait_hint(&ms.raw_free[g % kDnRawStages], (g / kDnRawStages - 1u) & 1u, cx, 23)) return false;
        dense_fetch(a, ms, maps, base, ids, t, g, po.page(t));
    }
    return true;
}

// Pages of the piece, dequantised, into the V buffers.
__device__ __noinline__ bool dense_produce(int pi, uint32_t g0, uint32_t n_planned, const DenseMaps *maps)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DenseArgs &a = ms.args;
    const DensePiece &pc = ms.piece[pi];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const WaitCtx cx = dense_wait(ms);
    const int nk = pc.kv1 - pc.kv0, L = pc.L;
    const PageOrder po(a, pc);
    const int32_t *bt = a.block_table + (size_t)pc.b * a.max_pages;
    const int e = tid & (kTile - 1), cp = tid >> 6;
    int ids = lane < nk ? bt[po.page(lane)] : -1, ids_next = 32 + lane < nk ? bt[po.page(32 + lane)] : -1;
    bool ok = true;
#pragma unroll 1
    for (int t = 0; ok && t < nk; ++t) {
        const uint32_t g = g0 + t, p = g % kDnStages, st = g % kDnRawStages;
        if (warp == 0 && t + 2 < nk) {
            const uint32_t gf = g + 2;
            if (gf >= kDnRawStages) ok = warp_wait_hint(&ms.raw_free[gf % kDnRawStages], (gf / kDnRawStages - 1u) & 1u, cx, 20);
            if (!ok) break;
            if (((t + 2) & 31) == 0) {
                ids = ids_next;
                ids_next = t + 34 + lane < nk ? bt[po.page(t + 34 + lane)] : -1;
            }
            dense_fetch(a, ms, maps, base, ids, t + 2, gf, po.page(t + 2));
        }
        ok = warp_wait_hint(&ms.raw_full[st], (g / kDnRawStages) & 1u, cx, 21);
        if (!ok) break;
        PageEntry raw;
        raw.read(base + kDnOffC + st * kDnRawCodes, base + kDnOffSc + st * kDnRawScales, e, cp);
        raw.valid = ms.page_ok[g % kDnFlags] && po.page(t) * kPage + e < L;
        __syncwarp();
        lane0_arrive(&ms.raw_free[st], lane);
        const bool is_nan = raw.has_nan(), use = raw.valid && !is_nan;
        const unsigned int nan = __ballot_sync(0xffffffffu, is_nan);
        if (g >= kDnStages) ok = warp_wait_hint(&ms.v_free[p], (g / kDnStages - 1u) & 1u, cx, 5);
        if (!ok) break;
        uint8_t *dst = base + p * kDnVBuf + 2 * cp * kDnVChunk;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            uint32_t v[16];
            raw.dequant(c, use, v);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                *reinterpret_cast<uint4 *>(dst + (c >> 1) * kDnVChunk + swz((uint32_t)e, (uint32_t)(4 * (c & 1) + u))) =
                    make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        }
        if (lane == 0) ms.nan_mask[p][warp] = nan;
        fence_async_smem();
        __syncwarp();
        lane0_arrive(&ms.v_ready[p], lane);
    }
    if (warp == 0 && ok) {
        // the next piece's first pages, while this one's last tiles go through the softmax
        ok = warp_wait_hint(&ms.planned, n_planned & 1u, cx, 22);
        if (ok && ms.piece[pi ^ 1].rows > 0) ok = dense_prefetch(a, ms, maps, base, ms.piece[pi ^ 1], g0 + nk);
    }
    return ok;
}

// Scores and softmax.  Warp (group a, quarter q) takes the tiles g with g % kDnGroups == a.  In its TMEM quarter lanes
// 16y .. 16y + 15 are rows of CTA y: it sends the other CTA's 16 rows of partial scores there and does the softmax of
// its own 16, thread i < 16 entries 0-31 of row i, thread 16 + i entries 32-63.  n_sent counts the tiles whose scores
// the warp has sent (and received).
__device__ __noinline__ uint32_t dense_scores(int pi, uint32_t g0, uint32_t n_sent)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DenseArgs &a = ms.args;
    const DensePiece &pc = ms.piece[pi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x = (int)cluster_rank();
    const WaitCtx cx = dense_wait(ms);
    const uint32_t tmem = ms.tmem_base, peer = (uint32_t)(x ^ 1);
    const int nk = pc.kv1 - pc.kv0;
    const PageOrder po(a, pc);
    const int q = warp & 3, grp = (warp - kDnScoreWarp) >> 2, u = lane >> 4;
    const int hl = 32 * q + 16 * x + (lane & 15);   // this thread's TMEM lane and row of the row tile
    const int hr = 16 * q + (lane & 15);            // row among this CTA's
    const bool active = 32 * q < pc.rows;           // the quarter has rows (the same in both CTAs)
    const uint32_t ts = tmem + ((uint32_t)(32 * q + 16 * x) << 16) + kDnColS;
    const uint32_t to = tmem + ((uint32_t)(32 * q + 16 * (x ^ 1)) << 16) + kDnColS;
    const float zs = ms.zs[hl], zo = ms.zs[hl ^ 16];
    const float softcap = a.softcap;
    const bool biased = a.slopes != nullptr;
    const uint32_t row = pc.r0 + (uint32_t)hl;
    const int tok = (int)(row / (uint32_t)a.H);
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
        if (biased) slope = a.slopes[row - (uint32_t)tok * (uint32_t)a.H] * kLog2e;
    }
    __syncwarp();
    const uint32_t rbase = remote_addr(smem_addr(base), peer);   // of this CTA's shared memory in the other one
    const uint32_t r_at = kDnOffR + kDnRBuf * grp + 4096u * q + 16u * lane;
    const uint32_t r_full_there = remote_addr(smem_addr(&ms.r_full[grp][q]), peer);
    const uint32_t r_free_there = remote_addr(smem_addr(&ms.r_free[grp][q]), peer);
    uint32_t sent = n_sent;
    bool ok = true;
    float m_run = kDnNoMax;                    // the reference of this thread's sum (log2 domain)
    float lsum = 0.f;                        // its share of the row's denominator
#pragma unroll 1
    for (int t = (int)((uint32_t)(grp + kDnGroups - (int)(g0 % kDnGroups)) % kDnGroups); t < nk; t += kDnGroups) {
        const uint32_t g = g0 + t, sb = g & 1u, pp = g % kDnPStages;
        if (active) lane0_arrive_expect_tx(&ms.r_full[grp][q], 4096u, lane);
        ok = warp_wait_hint(&ms.s_full[sb], (g >> 1) & 1u, cx, 6);
        if (ok && active && sent > 0) ok = warp_wait_hint(&ms.r_free[grp][q], (sent - 1u) & 1u, cx, 14);
        if (!ok) break;
        const uint4 fl = ms.flags[g % kDnStages];
        const uint32_t nan = u ? fl.y : fl.x;   // entries of this thread with a NaN scale in this CTA's channels
        const bool page_ok = fl.z != 0u;
        float z[32];
        tc_fence_after();
        if (active) {
            tc_ld16x32bx2_x32(to + 64 * sb, z);
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] *= zo;
            if (nan) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if ((nan >> i) & 1u) z[i] = __int_as_float(0x7FC00000);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                st_async16(rbase + r_at + 512u * i,
                           make_uint4(__float_as_uint(z[4 * i]), __float_as_uint(z[4 * i + 1]),
                                      __float_as_uint(z[4 * i + 2]), __float_as_uint(z[4 * i + 3])),
                           r_full_there);
            tc_ld16x32bx2_x32(ts + 64 * sb, z);
        }
        tc_fence_before();
        __syncwarp();
        lane0_arrive(&ms.s_free[sb], lane);   // QK of tile g + 2 may overwrite these columns
        float al = 1.f;
        if (active) {
            ok = warp_wait_hint(&ms.r_full[grp][q], sent & 1u, cx, 15);
            if (!ok) break;
            ++sent;
            // z = both halves of the channels, log2 domain
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint4 o = *reinterpret_cast<const uint4 *>(base + r_at + 512 * i);
                z[4 * i] = fmaf(z[4 * i], zs, __uint_as_float(o.x));
                z[4 * i + 1] = fmaf(z[4 * i + 1], zs, __uint_as_float(o.y));
                z[4 * i + 2] = fmaf(z[4 * i + 2], zs, __uint_as_float(o.z));
                z[4 * i + 3] = fmaf(z[4 * i + 3], zs, __uint_as_float(o.w));
            }
            __syncwarp();
            lane0_arrive_remote(r_free_there, lane);
            const int e0 = po.page(t) * kPage + 32 * u;   // position of z[0]
            if (softcap > 0.f) cap_scores(z, softcap);
            if (biased) {
                const float d = (float)(pos - e0);   // distances are whole numbers below 2^24, exact
#pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = fmaf(-slope, fabsf(d - (float)i), z[i]);
            }
            if (nan) {
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if ((nan >> i) & 1u) z[i] = __int_as_float(0x7FC00000);
            }
            if (lo > e0 || hi < e0 + 32 || !page_ok) {
                // entries of a mapped page that the row sees
                uint32_t seen = page_ok ? 0xFFFFFFFFu : 0u;
                if (lo > e0) seen &= lo - e0 < 32 ? 0xFFFFFFFFu << (lo - e0) : 0u;
                if (hi < e0 + 32) seen &= hi > e0 ? 0xFFFFFFFFu >> (32 - (hi - e0)) : 0u;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (!((seen >> i) & 1u)) z[i] = -INFINITY;
            }
            float mt = z[0];
#pragma unroll
            for (int i = 1; i < 32; ++i) mt = fmaxf(mt, z[i]);
            mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, 16));
            // the row's reference after the previous tile, which another group has; it grows only by more
            // than 2^8 at a time
            float m_old = kDnNoMax;
            if (t > 0) {
                const uint32_t gp = g - 1u;
                ok = warp_wait_hint(&ms.m_full[gp % kDnGroups][q], (gp / kDnGroups) & 1u, cx, 18);
                if (!ok) break;
                m_old = ms.m_row[gp % kDnGroups][hr];
            }
            const float m_new = mt > m_old + kLazy ? fmaxf(m_old, mt) : m_old;
            if (u == 0) ms.m_row[grp][hr] = m_new;
            __syncwarp();
            lane0_arrive(&ms.m_full[grp][q], lane);
            al = ex2(m_old - m_new);        // 0 while m_old is kDnNoMax, 1 if unchanged
            lsum *= ex2(m_run - m_new);
            m_run = m_new;
        } else {                            // the barrier's phases count tiles
            lane0_arrive(&ms.m_full[grp][q], lane);
        }
        if (g >= kDnPStages) ok = warp_wait_hint(&ms.p_free[pp], (g / kDnPStages - 1u) & 1u, cx, 16);
        if (!ok) break;
        if (active) {
            // P row hl, entries 32u .. 32u+31: four 16-byte units of the 128-byte swizzled row; p = 2^(z - m + 7), 0
            // for a masked entry (z = -inf)
            const float mref = m_run - kPOffset;
            float ls = 0.f;
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                uint32_t pk[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float p0 = ex2(z[8 * gq + 2 * i] - mref);
                    const float p1 = ex2(z[8 * gq + 2 * i + 1] - mref);
                    ls += p0 + p1;
                    pk[i] = pack_f16x2(p0, p1);
                }
                *reinterpret_cast<uint4 *>(base + kDnOffP + pp * kDnPBuf + swz((uint32_t)hl, (uint32_t)(4 * u + gq))) =
                    make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
            if (u == 0) ms.alpha[pp][hl] = al;
            lsum += ls;
            fence_async_smem();
            __syncwarp();
            if (elect_lane()) {
                // to the other CTA: the 16 rows are contiguous, one copy of 2 KB (16-byte stores to 16 rows cost twice
                // the time and slow every other access of the shared memory)
                const uint32_t r16 = 32u * q + 16u * x, pf = remote_addr(smem_addr(&ms.p_full[pp]), peer);
                const uint32_t src = kDnOffP + pp * kDnPBuf + 128u * r16, asrc = smem_addr(&ms.alpha[pp][r16]);
                bulk_to_cta(rbase + src, smem_addr(base) + src, 2048u, pf);
                bulk_to_cta(remote_addr(asrc, peer), asrc, 64u, pf);
            }
        }
        __syncwarp();
        if (active) lane0_arrive_expect_tx(&ms.p_full[pp], 2048u + 64u, lane);
        else lane0_arrive(&ms.p_full[pp], lane);
    }
    // the row's denominator from its two threads in every group
    lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
    if (u == 0) ms.ml[grp][hr] = make_float2(m_run, lsum);
    bar_sync(1 + q, 32 * kDnGroups);
    if (grp == 0) {
        float M = kDnNoMax, l = 0.f;
#pragma unroll
        for (int i = 0; i < kDnGroups; ++i) M = fmaxf(M, ms.ml[i][hr].x);
#pragma unroll
        for (int i = 0; i < kDnGroups; ++i) l += ex2(ms.ml[i][hr].x - M) * ms.ml[i][hr].y;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        if (u == 0) {
            if (hl < pc.rows) {
                // a row that sees nothing: out = 0, lse = -inf (a NaN sum stays NaN)
                if (pc.first && pc.last)
                    a.lse[pc.row + hl] = l == 0.f ? -INFINITY : (M - kPOffset) * kLn2 + logf(l);
                else
                    a.part_ml[(size_t)(2 * (blockIdx.x >> 1) + (pc.first ? 1 : 0)) * kDenseRows + hl] = make_float2(M - kPOffset, l);
            }
            // Only quarters with rows send: the scores that came from the other CTA in this piece show that it has
            // stored the last piece's rows and read their inv.  A quarter without rows has waited for nothing of this
            // piece from there, and its inv is of no use.
            if (ok && active) {
                ms.inv[hl] = inv;
                st_async4(remote_addr(smem_addr(&ms.inv[hl]), peer), __float_as_uint(inv),
                          remote_addr(smem_addr(&ms.inv_full), peer));
            }
        }
        __syncwarp();
        if (active) lane0_arrive_expect_tx(&ms.inv_full, 64u, lane);
        else lane0_arrive(&ms.inv_full, lane);
    }
    return ok ? sent : kDnFailed;
}

// A row tile no row of which sees anything (a whole one): lse, and the next piece.
__device__ __noinline__ void dense_nothing_seen(int pi)
{
    DenseMisc &ms = dense_misc(dense_smem());
    const DensePiece &pc = ms.piece[pi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == kDnPlanWarp && lane == 0) next_piece(ms.args, ms.args.cu_rows, ms.args.seq_len, ms.cur, ms.share, ms.piece[pi ^ 1]);
    if (warp == kDnScoreWarp && cluster_rank() == 0)
        for (int i = lane; i < pc.rows; i += 32) ms.args.lse[pc.row + i] = -INFINITY;
}

// The piece's Q into TMEM, and its first pages on their way unless they are already.
__device__ __noinline__ void dense_begin(int pi, uint32_t g0, bool fetch, const DenseMaps *maps)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DensePiece &pc = ms.piece[pi];
    const int warp = threadIdx.x >> 5;
    stage_q(ms.args, ms, pc, (int)cluster_rank(), base, [&]() {
        if (warp == 0 && fetch) dense_prefetch(ms.args, ms, maps, base, pc, g0);   // a failure shows in the role
    });
    __syncthreads();
    store_q(base, ms.tmem_base);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
}

// O of the piece to out or to a partial: quarter w%4, channels 64(w/4) .. of this CTA's, each warp through 4 KB
// of the V buffers so that its stores are whole rows of 128 bytes.
__device__ __noinline__ bool dense_epilogue(int pi, uint32_t g0, uint32_t pieces, bool ok)
{
    uint8_t *base = dense_smem();
    DenseMisc &ms = dense_misc(base);
    const DenseArgs &a = ms.args;
    const DensePiece &pc = ms.piece[pi];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int x = (int)cluster_rank();
    const WaitCtx cx = dense_wait(ms);
    const uint32_t tmem = ms.tmem_base;
    const int nk = pc.kv1 - pc.kv0;
    uint8_t *V = base;
    if (nk > 0) {
        const uint32_t gl = g0 + nk - 1;
        ok = ok && warp_wait_hint(&ms.v_free[gl % kDnStages], (gl / kDnStages) & 1u, cx, 8) &&
             warp_wait_hint(&ms.inv_full, pieces & 1u, cx, 17);
    }
    // the V buffers are free once every warp that reads or writes them has come here
    ok = __syncthreads_and(ok);
    if (ok) {
        tc_fence_after();
        const int q = warp & 3, c0 = 64 * (warp >> 2), r0 = 32 * q;
        const uint32_t to = tmem + ((uint32_t)(32 * q) << 16) + kDnColO + c0;
        uint8_t *st = V + 4096 * warp;
        const bool whole = pc.first && pc.last;
        const float inv = ms.inv[32 * q + lane];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float o[32];
            if (nk > 0) {
                tc_ld32_sync(to + 32 * h, o);
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0.f;
            }
            if (whole) {
                const float sc = nk > 0 ? inv : 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t b[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __nv_bfloat162 y = __floats2bfloat162_rn(o[8 * i + 2 * j] * sc, o[8 * i + 2 * j + 1] * sc);
                        b[j] = *reinterpret_cast<const uint32_t *>(&y);
                    }
                    *reinterpret_cast<uint4 *>(st + swz((uint32_t)lane, (uint32_t)(4 * h + i))) = make_uint4(b[0], b[1], b[2], b[3]);
                }
                if (h == 0) continue;
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(st + swz((uint32_t)lane, (uint32_t)i)) =
                        make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            }
            __syncwarp();
            // row r0 + l of 128 bytes: eight lanes
            const int unit = lane & 7;
            uint8_t *dst = whole ? reinterpret_cast<uint8_t *>(a.out + (size_t)(pc.row + r0) * kLatent + kDnCh * x + c0)
                                 : reinterpret_cast<uint8_t *>(a.part_o +
                                       ((size_t)(2 * (blockIdx.x >> 1) + (pc.first ? 1 : 0)) * kDenseRows + r0) * kLatent +
                                       kDnCh * x + c0 + 32 * h);
            const uint32_t stride = whole ? 2 * kLatent : 4 * kLatent;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int l = 4 * i + (lane >> 3);
                if (r0 + l < pc.rows)
                    *reinterpret_cast<uint4 *>(dst + (size_t)l * stride + 16 * unit) =
                        *reinterpret_cast<const uint4 *>(st + swz((uint32_t)l, (uint32_t)unit));
            }
            __syncwarp();
        }
    }
    return ok;
}

// The end of a CTA's work: its share for the combine, and nothing left on its way.
__device__ __noinline__ void dense_finish(uint32_t g0, uint32_t sent, bool ok)
{
    DenseMisc &ms = dense_misc(dense_smem());
    const int tid = threadIdx.x, warp = tid >> 5, x = (int)cluster_rank();
    const WaitCtx cx = dense_wait(ms);
    if (tid == 0 && x == 0) ms.args.share[blockIdx.x >> 1] = ms.share;
    // nothing is on its way to or from the other CTA when this one ends: what it sent here has been waited
    // for tile by tile, and its last releases are waited for now
    if (warp == kDnPvWarp && ok)
        for (uint32_t i = 1; i <= (uint32_t)kDnPStages && i <= g0; ++i)
            ok = ok && warp_wait_hint(&ms.p_free[(g0 - i) % kDnPStages], ((g0 - i) / kDnPStages) & 1u, cx, 18);
    if (warp >= kDnScoreWarp && warp < kDnMmaWarp && ok && sent > 0)
        warp_wait_hint(&ms.r_free[(warp - kDnScoreWarp) >> 2][warp & 3], (sent - 1u) & 1u, cx, 19);
    if (ms.abort_flag && (warp == kDnQkWarp || warp == kDnPvWarp) && elect_lane()) {
        // every MMA this thread issued has completed before TMEM is released (otherwise the pieces' ends saw to it)
        uint64_t *done = &ms.final_bar[warp == kDnQkWarp ? 0 : 1];
        tc_commit(smem_addr(done));
        volatile int no_abort = 0;
        mbar_wait(done, 0, &no_abort, ms.args.ws, 4);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kDnMmaWarp) tc_dealloc(ms.tmem_base, kDnTmemCols);
    if (ms.abort_flag) {
        if (tid == 0) report(ms.args.ws, CSA_ERR_TIMEOUT, ms.abort_flag);
        // after a failed wait, stores to the other CTA may still be on their way
        const unsigned long long t0 = global_ns();
        while (global_ns() - t0 < 1000000ull) {}
    }
    __syncwarp();
    cluster_arrive();
    cluster_wait();
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDnThreads, 1)
    dense_attn_kernel(const __grid_constant__ DenseMaps maps, DenseArgs a)
{
    uint8_t *V = dense_smem();
    DenseMisc &ms = dense_misc(V);
    const int warp = threadIdx.x >> 5;
    grid_dep_launch();   // the combine may be scheduled as CTAs finish

    if (threadIdx.x == 0) {
        for (int i = 0; i < kDnRawStages; ++i) {
            mbar_init(&ms.raw_full[i], 1);
            mbar_init(&ms.raw_free[i], kDnProducerWarps);
        }
        for (int i = 0; i < kDnStages; ++i) {
            mbar_init(&ms.v_ready[i], kDnProducerWarps);
            mbar_init(&ms.v_free[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.s_full[i], 2);
            mbar_init(&ms.s_free[i], 4);
        }
        for (int i = 0; i < kDnGroups; ++i)
            for (int w = 0; w < 4; ++w) {
                mbar_init(&ms.r_full[i][w], 1);
                mbar_init(&ms.r_free[i][w], 1);
            }
        for (int i = 0; i < kDnPStages; ++i) {
            mbar_init(&ms.p_full[i], 4);
            mbar_init(&ms.p_free[i], 2);
        }
        for (int i = 0; i < kDnGroups; ++i)
            for (int w = 0; w < 4; ++w) mbar_init(&ms.m_full[i][w], 1);
        mbar_init(&ms.planned, 1);
        mbar_init(&ms.go, 1);
        mbar_init(&ms.c_done, 3);
        mbar_init(&ms.inv_full, 4);
        for (int r = 0; r < 2; ++r) mbar_init(&ms.final_bar[r], 1);
        ms.abort_flag = 0;
        ms.rescales = 0;
        ms.args = a;
        fence_mbar_init();
    }
    if (warp == kDnMmaWarp) {
        tc_alloc(smem_addr(&ms.tmem_base), kDnTmemCols);
        tc_relinquish();
    }
    grid_dep_wait();     // everything below reads what earlier kernels wrote, or writes what they read
    plan(a, ms, reinterpret_cast<int32_t *>(V));
    __syncwarp();
    cluster_arrive();
    cluster_wait();      // the other CTA's barriers are there, and it has read its plan from where P goes

    bool ok = true;
    uint32_t g0 = 0;      // tiles of the earlier pieces
    uint32_t pieces = 0;  // earlier pieces that had tiles
    bool prefetched = false;   // this piece's first pages are on their way: the producers of the one before saw to it
    uint32_t sent = 0;    // score warps: tiles whose scores went to the other CTA (and came from there); MMA warps: requests
    for (int pi = 0;; pi ^= 1) {
        // the piece is visible and the previous one is finished with TMEM and shared memory
        tc_fence_before();
        if (__syncthreads_or(!ok)) break;
        tc_fence_after();
        if (ms.piece[pi].rows == 0) break;
        const int nk = ms.piece[pi].kv1 - ms.piece[pi].kv0;
        if (nk > 0) dense_begin(pi, g0, !prefetched, &maps);
        prefetched = nk > 0;
        if (nk > 0) {
            if (warp < kDnProducerWarps) ok = dense_produce(pi, g0, pieces, &maps);
            else if (warp < kDnMmaWarp) sent = dense_scores(pi, g0, sent), ok = sent != kDnFailed;
            else if (warp == kDnPvWarp) ok = dense_pv(pi, g0);
            else sent = dense_mma(pi, g0, sent), ok = sent != kDnFailed;
        } else {
            dense_nothing_seen(pi);
        }
        ok = dense_epilogue(pi, g0, pieces, ok);
        if (nk > 0) {
            g0 += nk;
            ++pieces;
        }
    }
    dense_finish(g0, sent, ok);
}

// ------------------------------------------------------------------------------------------------
// Combine: out = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i over the parts of a shared row tile, in
// cluster order.  CTA (c, y) takes rows 8y .. 8y+7 of the row tile that cluster c began and did not
// finish, two warps per row.
// ------------------------------------------------------------------------------------------------
constexpr int kCombineRows = 8;

__global__ void __launch_bounds__(64 * kCombineRows) dense_combine_kernel(DenseArgs a)
{
    constexpr int kWarps = 2 * kCombineRows;
    __shared__ int slots[kDensePairs + 1];
    __shared__ int first_end, counts[kWarps];
    __shared__ float wgt[kWarps][kDensePairs + 1];
    const int c = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) first_end = kDensePairs;
    grid_dep_wait();     // every part
    grid_dep_launch();   // a dependent kernel launched after this one waits for it before reading
    const DenseShare tail = a.share[c];
    const int o = c + 1 + tid;
    DenseShare sh{};
    if (o < kDensePairs) sh = a.share[o];
    if (tail.tail_rows <= kCombineRows * (int)blockIdx.y) return;
    // the parts: the tail of cluster c, then the heads of the clusters behind it up to the one that ends the tile
    __syncthreads();
    if (sh.head && sh.head_ends) atomicMin(&first_end, o);
    __syncthreads();
    const bool part = sh.head && o <= first_end;
    const unsigned vote = __ballot_sync(0xffffffffu, part);
    if (lane == 0) counts[warp] = __popc(vote);
    __syncthreads();
    int at = 1, n = 1;
    for (int w = 0; w < (kDensePairs + 31) / 32; ++w) {
        if (w < warp) at += counts[w];
        n += counts[w];
    }
    if (tid == 0) slots[0] = 2 * c + 1;
    if (part) slots[at + __popc(vote & ((1u << lane) - 1u))] = 2 * o;
    __syncthreads();
    const int r = kCombineRows * blockIdx.y + (warp >> 1), half = warp & 1;
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
    float4 acc[2] = {};
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
        const float4 *po = reinterpret_cast<const float4 *>(a.part_o + ((size_t)slots[i] * kDenseRows + r) * kLatent) + 64 * half + lane;
        const float w = wgt[warp][i];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float4 v = po[32 * j];
            acc[j].x = fmaf(w, v.x, acc[j].x);
            acc[j].y = fmaf(w, v.y, acc[j].y);
            acc[j].z = fmaf(w, v.z, acc[j].z);
            acc[j].w = fmaf(w, v.w, acc[j].w);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint2 *out = reinterpret_cast<uint2 *>(a.out + (size_t)(tail.tail_row + r) * kLatent) + 64 * half + lane;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        __nv_bfloat162 x = __floats2bfloat162_rn(acc[j].x * inv, acc[j].y * inv);
        __nv_bfloat162 y = __floats2bfloat162_rn(acc[j].z * inv, acc[j].w * inv);
        out[32 * j] = make_uint2(*reinterpret_cast<uint32_t *>(&x), *reinterpret_cast<uint32_t *>(&y));
    }
    if (lane == 0 && half == 0) a.lse[tail.tail_row + r] = den == 0.f ? -INFINITY : M * kLn2 + logf(den);
}

static cudaError_t cache_map(PFN_cuTensorMapEncodeTiled_v12000 encode, const uint8_t *pool, int num_pages, int bytes,
                             CUtensorMapSwizzle swizzle, CUtensorMap *out)
{
    const cuuint64_t dims[3] = {(cuuint64_t)bytes, (cuuint64_t)kPage, (cuuint64_t)num_pages};
    const cuuint64_t strides[2] = {(cuuint64_t)bytes, (cuuint64_t)bytes * kPage};
    const cuuint32_t box[3] = {(cuuint32_t)bytes / 2, (cuuint32_t)kPage, 1}, estr[3] = {1, 1, 1};
    return encode(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t *>(pool), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

cudaError_t launch_dense_attn(const DenseArgs &a, cudaStream_t st)
{
    static_assert(kDnSmem <= 232448, "shared memory budget");
    static_assert(64 * kCombineRows >= kDensePairs, "one thread per cluster behind the tail");
    PFN_cuTensorMapEncodeTiled_v12000 encode;
    cudaError_t e = tensor_map_encoder(&encode);
    if (e != cudaSuccess) return e;
    DenseMaps maps;
    if ((e = cache_map(encode, a.codes, a.num_pages, kCodeBytes, CU_TENSOR_MAP_SWIZZLE_128B, &maps.codes)) != cudaSuccess) return e;
    if ((e = cache_map(encode, a.scales, a.num_pages, kScaleBytes, CU_TENSOR_MAP_SWIZZLE_NONE, &maps.scales)) != cudaSuccess) return e;
    e = allow_dynamic_smem(reinterpret_cast<const void *>(dense_attn_kernel), kDnSmem);
    if (e != cudaSuccess) return e;
    e = launch_overlapped(dense_attn_kernel, dim3(2 * kDensePairs), dim3(kDnThreads), kDnSmem, st, maps, a);
    if (e != cudaSuccess) return e;
    // no row tile has more rows than the call
    const long long most = a.rows * (long long)a.H < kDenseRows ? a.rows * (long long)a.H : kDenseRows;
    return launch_overlapped(dense_combine_kernel, dim3(kDensePairs, (unsigned)((most + kCombineRows - 1) / kCombineRows)),
                             dim3(64 * kCombineRows), 0, st, a);
}

}  // namespace csa
