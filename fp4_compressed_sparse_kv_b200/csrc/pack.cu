// pack.cu -- step 1: pack new tokens' latents into the FP4 main cache, the E4M3 indexer-key cache
// and the FP8 sliding-window ring.
//
// rebasdaily article on DeepSeek-V4.1-Flash KV compression, section "同一份笔记，多层一起用": the
// main KV is FP4 while the more quantisation-sensitive SWA KV stays FP8.  ailily.cc article
// "每个 token 只占 890 字节", section 二: one E4M3 scale per 16 channels holds the value range.
//
// One warp per token at a time; for long calls, four consecutive tokens per warp with all their loads
// issued first.
// Lane g owns 16-channel group g of the 512-channel latent, which is exactly one E4M3 scale: its amax
// needs no cross-lane step, and its 16 codes are one 8-byte store.  The window entry needs the
// token's amax, a 5-step warp max.  Loads are 2 x 16 B per lane (latent) and 8 B per lane (key), all
// coalesced; long calls are HBM-bound streaming (65,536 tokens, 112 MB: 25.0 us, 4.5 TB/s; 43 us with a
// division per value).
//
// The norm variant starts from the pre-norm latent (ailily.cc article, section 三: the KV latent is
// RMS-normalised, with weights of magnitude about 1, and rotated by RoPE, which keeps its norm): in
// binary32, lane g forms the FMA chain of its 16 squares, an xor butterfly (16, 8, 4, 2, 1) sums the
// lanes, r = 1 / sqrt(sum / 512 + 1e-6) with correctly rounded operations, y = (v * r) * weight; lanes
// 28-31 then rotate their channel pairs (448 + 2i, 449 + 2i) with the caller's (cos_i, sin_i), every
// product and sum rounded on its own; the result is rounded to bf16 and packed as above.
#include "pack_token.cuh"
#include "pipeline.cuh"

namespace csa {

// Each warp packs kTok consecutive tokens: their loads are issued together, then each token's
// arithmetic runs on registers, so every warp keeps several tokens' bytes in flight (prefill chunks);
// a decode batch of a few tokens takes one token per warp, its latency being one token's.
constexpr int kPackTokLarge = 4;
constexpr int kPackLargeFrom = 4096;   // tokens per call from which warps take kPackTokLarge tokens

template <bool kNorm, int kPackTok>
__global__ void __launch_bounds__(256) kv_pack_kernel(csa_kv_layer layer, const uint16_t *__restrict__ latent,
                                                      const uint16_t *__restrict__ idx_key,
                                                      const int64_t *__restrict__ slot,
                                                      const int32_t *__restrict__ swa_slot, int n, void *ws,
                                                      const float *__restrict__ norm_w,
                                                      const float *__restrict__ rope_cs)
{
    // a dependent kernel launched after this one (the indexer's query terms, an attention) may be
    // scheduled now: each waits for this grid before it reads anything this grid writes
    grid_dep_launch();
    const int tok0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kPackTok;
    const int lane = threadIdx.x & 31;
    PackIn in[kPackTok];
#pragma unroll
    for (int i = 0; i < kPackTok; ++i) {
        const int tok = tok0 + i;
        if (tok < n) {
            const uint4 *src = reinterpret_cast<const uint4 *>(latent + (size_t)tok * kLatent) + 2 * lane;
            in[i].a = src[0];
            in[i].b = src[1];
            in[i].kw = reinterpret_cast<const uint2 *>(idx_key + (size_t)tok * kIdxDim)[lane];
            in[i].s = slot[tok];
            in[i].ss = swa_slot ? swa_slot[tok] : -1;
        }
    }
#pragma unroll
    for (int i = 0; i < kPackTok; ++i)
        if (tok0 + i < n)
            pack_token<kNorm, kNorm>(layer, in[i], tok0 + i, lane, ws, norm_w,
                                     kNorm ? rope_cs + (size_t)(tok0 + i) * kRopeRow : nullptr);
}

cudaError_t launch_kv_pack(const csa_kv_layer &layer, const uint16_t *latent, const uint16_t *idx_key,
                           const int64_t *slot, const int32_t *swa_slot, int n, void *ws, cudaStream_t st)
{
    if (n == 0) return cudaSuccess;
    if (n >= kPackLargeFrom)
        kv_pack_kernel<false, kPackTokLarge><<<(n + 8 * kPackTokLarge - 1) / (8 * kPackTokLarge), 256, 0, st>>>(
            layer, latent, idx_key, slot, swa_slot, n, ws, nullptr, nullptr);
    else
        kv_pack_kernel<false, 1><<<(n + 7) / 8, 256, 0, st>>>(layer, latent, idx_key, slot, swa_slot, n, ws, nullptr,
                                                             nullptr);
    return cudaGetLastError();
}

cudaError_t launch_kv_norm_rope_pack(const csa_kv_layer &layer, const uint16_t *latent, const float *norm_w,
                                     const float *rope_cs, const uint16_t *idx_key, const int64_t *slot,
                                     const int32_t *swa_slot, int n, void *ws, cudaStream_t st)
{
    if (n == 0) return cudaSuccess;
    if (n >= kPackLargeFrom)
        kv_pack_kernel<true, kPackTokLarge><<<(n + 8 * kPackTokLarge - 1) / (8 * kPackTokLarge), 256, 0, st>>>(
            layer, latent, idx_key, slot, swa_slot, n, ws, norm_w, rope_cs);
    else
        kv_pack_kernel<true, 1><<<(n + 7) / 8, 256, 0, st>>>(layer, latent, idx_key, slot, swa_slot, n, ws, norm_w,
                                                            rope_cs);
    return cudaGetLastError();
}

}  // namespace csa
