// kv_runs.cu -- append a ragged run of tokens to the paged FP4 cache by position, and read one back.
//
// rebasdaily article on DeepSeek-V4.1-Flash KV compression, section "同一份笔记，多层一起用" (FP4 main
// KV, FP8 window) and section "先让长输入少走一半路" (the window holds the most recent tokens); yomxxx.com
// long-form post, section 五 (addresses computed from the token index).
//
// Append: one warp per token, with the arithmetic of pack.cu (pack_token.cuh); the token's sequence, page,
// rotation and window slot are worked out from its row number, so the caller builds no slot or angle
// arrays and no pass over the latents comes before the pack.  Unpack: the inverse for the FP4 entries,
// e2m1 * e4m3 in bf16, which is exact (at most 6 significant bits); a lane converts two pieces of 8
// channels so that a warp's stores are 512 contiguous bytes.
//
// Both stream their bytes once.  Long unpacks are bound by HBM (200,003 entries: 44 us, 5.9 TB/s).  Long appends are
// bound by instructions and the latency of the metadata's loads together: 65,536 tokens with norm and rotation 40 us
// (3.3 TB/s, 449 warp instructions a token issued in 68 % of the cycles), 20,001 ready tokens 10.2 us (265 a token in
// 59 %, the commonest stall a global load; its 5,001 CTAs are 3.4 rounds of the SMs).  Short calls are bound by the metadata's loads, one behind
// the other (cu_rows, then the page id, then the entry), which the tokens of an unpacking warp share.  Both are dependent launches,
// in place when the kernel before them ends (8 tokens appended and read back: 10.2 -> 7.5-8.2 us).
#include "pack_token.cuh"
#include "pipeline.cuh"
#include "runs.cuh"

namespace csa {

constexpr int kRunWarps = 4;             // warps per CTA: a CTA's place is free again when its slowest token is done (65,536 normed
                                         // and 20,001 ready tokens appended and read back: 8 warps 57.1 and 17.6 us, 4: 55.3
                                         // and 17.2, 2: 54.9 and 18.1)
constexpr int kUnpackTok = 4;            // tokens per unpacking warp (in CTAs of 8 warps, 200,003 entries: 46 us; 1: 54)
constexpr int kRunLargeFrom = 4096;      // rows from which unpacking warps take several tokens

// 40 warps on an SM hide a token's chain of conversions and shuffles better than several tokens per warp do: 65,536
// tokens 42 us in CTAs of 8 warps (2 tokens per warp, 32 warps: 45; 4 tokens in 98 registers: 66).
template <bool kNorm, bool kRope>
__global__ void __launch_bounds__(32 * kRunWarps, 10) kv_append_kernel(csa_kv_layer layer, Runs r,
                                                                   const uint16_t *__restrict__ latent,
                                                                   const uint16_t *__restrict__ idx_key,
                                                                   const float *__restrict__ norm_w,
                                                                   const float *__restrict__ rope_table,
                                                                   int rope_positions, void *ws)
{
    grid_dep_wait();     // what follows reads and overwrites the data of the kernel before it
    grid_dep_launch();   // only now: a dependent kernel may read at its start what any kernel before this one wrote
    const int t = blockIdx.x * kRunWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (t == 0 && lane == 0 && r.cu_rows[r.B] > r.rows) report(ws, CSA_ERR_DEVICE_DATA, r.B);
    if (t >= r.rows) return;
    PackIn in;
    const uint4 *src = reinterpret_cast<const uint4 *>(latent + (size_t)t * kLatent) + 2 * lane;
    in.a = src[0];
    in.b = src[1];
    in.kw = reinterpret_cast<const uint2 *>(idx_key + (size_t)t * kIdxDim)[lane];
    RowPlace p[1];
    warp_place_rows<1>(r, t, layer.num_pages, p);
    const bool no_rotation = kRope && p[0].pos >= rope_positions;
    if ((p[0].bad || no_rotation) && lane == 0) report(ws, CSA_ERR_DEVICE_DATA, t);
    if (p[0].seq < 0 || no_rotation) return;
    const float *rope_row = kRope ? rope_table + (size_t)p[0].pos * kRopeRow : nullptr;
    // the rotation is needed behind the norm: on its way meanwhile (65,536 tokens: 1 us less)
    if (kRope && lane >= 28) asm volatile("prefetch.global.L2 [%0];" ::"l"(rope_row + 16 * (lane - 28)));
    in.s = p[0].slot;
    in.ss = -1;
    if (layer.swa && p[0].pos >= p[0].len - kWindow) {
        const int row = r.swa_row[p[0].seq];
        if (row >= 0 && row < layer.num_rows) in.ss = row * kWindow + p[0].pos % kWindow;
        else if (row != -1 && lane == 0) report(ws, CSA_ERR_DEVICE_DATA, t);
    }
    pack_token<kNorm, kRope>(layer, in, t, lane, ws, norm_w, rope_row);
}

template <int kTok>
__global__ void __launch_bounds__(32 * kRunWarps) kv_unpack_kernel(csa_kv_layer layer, Runs r,
                                                                   uint16_t *__restrict__ latent, void *ws)
{
    grid_dep_wait();
    grid_dep_launch();
    const int t0 = (blockIdx.x * kRunWarps + (threadIdx.x >> 5)) * kTok;
    const int lane = threadIdx.x & 31;
    if (t0 == 0 && lane == 0 && r.cu_rows[r.B] > r.rows) report(ws, CSA_ERR_DEVICE_DATA, r.B);
    RowPlace p[kTok];
    warp_place_rows<kTok>(r, t0, layer.num_pages, p);
    int64_t slot[kTok];
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
        if (p[i].bad && lane == 0) report(ws, CSA_ERR_DEVICE_DATA, t0 + i);
        slot[i] = p[i].seq >= 0 ? p[i].slot : -1;
    }
    // lane: channels 256 j + 8 lane .. + 7 for j = 0, 1
    uint32_t code[kTok][2];
    uint8_t scale[kTok][2];
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (slot[i] >= 0) {
                code[i][j] = reinterpret_cast<const uint32_t *>(layer.codes + slot[i] * kCodeBytes)[32 * j + lane];
                scale[i][j] = layer.scales[slot[i] * kScaleBytes + 16 * j + (lane >> 1)];
            }
#pragma unroll
    for (int i = 0; i < kTok; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (slot[i] >= 0) {
                uint32_t c[4], o[4];
                e2m1x8_to_f16x2x4(code[i][j], c);
                const float s = e4m3_to_f32(scale[i][j]);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    __nv_bfloat162 v = __floats2bfloat162_rn(h_lo(c[k]) * s, h_hi(c[k]) * s);
                    o[k] = *reinterpret_cast<uint32_t *>(&v);
                }
                reinterpret_cast<uint4 *>(latent + (size_t)(t0 + i) * kLatent)[32 * j + lane] =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
}

template <bool kNorm, bool kRope>
static cudaError_t append(const csa_kv_layer &layer, const Runs &r, const uint16_t *latent, const uint16_t *idx_key,
                          const float *norm_w, const float *rope_table, int rope_positions, void *ws, cudaStream_t st)
{
    return launch_overlapped(kv_append_kernel<kNorm, kRope>, dim3((r.rows + kRunWarps - 1) / kRunWarps), dim3(32 * kRunWarps), 0, st,
                             layer, r, latent, idx_key, norm_w, rope_table, rope_positions, ws);
}

cudaError_t launch_kv_append(const csa_kv_layer &layer, const Runs &r, const uint16_t *latent, const uint16_t *idx_key,
                             const float *norm_w, const float *rope_table, int rope_positions, void *ws,
                             cudaStream_t st)
{
    if (norm_w && rope_table)
        return append<true, true>(layer, r, latent, idx_key, norm_w, rope_table, rope_positions, ws, st);
    if (norm_w) return append<true, false>(layer, r, latent, idx_key, norm_w, rope_table, rope_positions, ws, st);
    if (rope_table) return append<false, true>(layer, r, latent, idx_key, norm_w, rope_table, rope_positions, ws, st);
    return append<false, false>(layer, r, latent, idx_key, norm_w, rope_table, rope_positions, ws, st);
}

cudaError_t launch_kv_unpack(const csa_kv_layer &layer, const Runs &r, uint16_t *latent, void *ws, cudaStream_t st)
{
    const int per = kRunWarps * (r.rows >= kRunLargeFrom ? kUnpackTok : 1);
    return launch_overlapped(r.rows >= kRunLargeFrom ? kv_unpack_kernel<kUnpackTok> : kv_unpack_kernel<1>,
                             dim3((r.rows + per - 1) / per), dim3(32 * kRunWarps), 0, st, layer, r, latent, ws);
}

}  // namespace csa
