// Internal declarations of the training-side row and vocabulary-loss
// kernels (orthrus_embed_rows .. orthrus_kl_lm_head_grad): they need no
// context, so their scratch is a plan over the caller's workspace.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/orthrus.h"

namespace orthrus {

// Offsets into a caller's workspace, each 256-byte aligned.
struct WsPlan {
    size_t total = 0;
    size_t take(size_t bytes)
    {
        const size_t o = total;
        total += (bytes + 255) & ~(size_t)255;
        return o;
    }
};

// ------------------------------------------------------------- embedding
struct EmbedRowsArgs {
    const void *table;
    const int32_t *ids;
    void *out;
    int dtype, out_dtype, rows, d, vocab;
    float scale;
    unsigned *err;
};
cudaError_t launch_embed_rows(const EmbedRowsArgs &a, cudaStream_t s);

// most rows sorted by counting (16384 rows: 44 us; the radix sort's six launches
// take 45, and no less at fewer)
constexpr int kRankMost = 16384;
constexpr int kSortTile = 2048;    // keys per block of the radix sort
constexpr int kSortDigit = 9;      // widest radix digit

struct EmbedGradPlan {
    size_t total, o_tok[2], o_idx[2], o_hist, o_part;
    int piece;     // sorted rows per piece
    int pieces;
    int digits, digit_bits, tiles;   // radix sort (rows > kRankMost)
};
EmbedGradPlan plan_embed_grad(int rows, int vocab, int d);
struct EmbedGradArgs {
    const void *dout;
    const int32_t *ids;
    void *dtable;
    int dout_dtype, dtable_dtype, rows, d, vocab, accumulate;
    float scale;
    char *ws;
    unsigned *err;
};
cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t s);

// --------------------------------------------------------------- RMSNorm
struct NormArgs {
    const void *x, *gain, *dy;
    void *out;        // y, or dx
    float *dgain;
    int x_dtype, dtype, rows, d;
    float eps;
    char *ws;
};
cudaError_t launch_norm_rows(const NormArgs &a, cudaStream_t s);
size_t norm_grad_workspace(int rows, int d);
cudaError_t launch_norm_grad(const NormArgs &a, cudaStream_t s);

// -------------------------------------------------------- vocabulary loss
// acc += the products of eight bf16 pairs (each exact in fp32)
__device__ __forceinline__ void dot8(uint4 u, uint4 v, float (&acc)[4])
{
    const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, vv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        acc[k] = fmaf(__uint_as_float(uu[k] << 16), __uint_as_float(vv[k] << 16), acc[k]);
        acc[k] = fmaf(__uint_as_float(uu[k] & 0xffff0000u), __uint_as_float(vv[k] & 0xffff0000u), acc[k]);
    }
}
__device__ __forceinline__ double warp_sum_f64(double v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// One loss call: z = h W^T over V ids.  KL: h holds the AR rows, h2 the
// diffusion rows, and lse / lse2 their log-sum-exps.
struct LossArgs {
    const void *h, *h2, *w;
    const int32_t *targets;   // CE: [N], negative = ignored row
    const float *lse_in, *lse2_in, *g;
    float *loss, *lse;        // CE forward outputs
    void *dh, *dw;            // gradients (dw nullable)
    int dtype, N, d, V;
    int kl;
    char *ws;
    unsigned *err;
};

size_t loss_fwd_workspace(int N, int d, int V, int dtype);
size_t loss_grad_workspace(int N, int d, int V, int dtype, int want_dw, int kl);
// the tensor-core path (vocab_loss_tc.cu): bf16, hidden a multiple of 8,
// 16-byte aligned buffers
bool loss_tc_ok(const LossArgs &a);
size_t loss_fwd_workspace_tc(int N, int d, int V);
size_t loss_grad_workspace_tc(int N, int d, int V, int want_dw, int kl);
cudaError_t loss_fwd_tc(const LossArgs &a, cudaStream_t s);
cudaError_t loss_grad_tc(const LossArgs &a, cudaStream_t s);
// shared kernels (vocab_loss.cu)
cudaError_t launch_ce_finalize(const float2 *rec, const float *zt, const LossArgs &a, int n_tiles, int exact,
                               cudaStream_t s);
cudaError_t launch_part_sum(const float *part, int splits, size_t n, void *out, int dtype, cudaStream_t s);
cudaError_t launch_loss_fwd(const LossArgs &a, cudaStream_t s);
cudaError_t launch_loss_grad(const LossArgs &a, cudaStream_t s);

}  // namespace orthrus
