// Losses through the shared LM head without keeping the logits: the cross
// entropy of one token id per row with its gradients, and the gradient of
// the forward KL(p_AR || p_diff) (paper notes §3.3).  With z = W h:
//     CE   lse = log sum_v exp z_v,  loss = lse - z_t = log(1 + sum_{v != t} exp(z_v - z_t)),
//          dz_v = g (exp(z_v - lse) - [v = t])
//     KL   dz_v = g (softmax(W h_diff)_v - softmax(W h_AR)_v)
//     dh = dz W,   dW = dz^T h.
// The forward pass keeps a maximum and a sum of exponentials per (row,
// vocabulary tile).  The gradient goes over the vocabulary in pieces: a
// piece's dz is made from recomputed logits and the row's log-sum-exp, and
// used for its part of dh and its rows of dW before the next piece takes its
// place, so the scratch does not grow with the vocabulary.
//
// This file: the plan over the workspace, the kernels every path shares, and
// the SIMT path (fp32, and bf16 rows that TMA cannot address).  The tensor-core
// path of bf16 is in vocab_loss_tc.cu.
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "train.h"

namespace orthrus {

// ---------------------------------------------------------------- tiles
constexpr int kSt = 64;            // rows and columns of a SIMT tile
constexpr int kStK = 32;           // k per step
constexpr int kStThreads = 256;
constexpr int kStFlush = 4;        // steps per partial sum (128 products)
constexpr int kStLoads = kSt * kStK / kStThreads;
constexpr int kStBufs = 4;         // steps in shared memory

// A strided operand: element (row, k).  With `live`, a k whose byte is zero
// reads as zeros whatever it holds.
template <class T> struct Operand {
    const T *p;
    size_t row_stride, k_stride;
    int rows;
    const unsigned char *live;
};

// One element to shared memory, zero when it is not there: fp32 by an
// asynchronous copy, bf16 converted on the way.
template <class T> __device__ __forceinline__ void st_put(float *dst, const T *src, const T *any, bool ok)
{
    if constexpr (sizeof(T) == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(smem_u32(dst)), "l"(ok ? src : any), "r"(ok ? 4 : 0)
                     : "memory");
    else
        *dst = ok ? to_f<T>(*src) : 0.f;
}

// A thread's elements of an operand's steps.  k contiguous in memory (K): one k
// and every 8th row; 8 k x 4 rows per warp, whole 32-byte sectors, and a warp's
// 32 stores into the transposed tile hit 32 banks.  Otherwise one row and every
// 4th k, lanes along the rows.
template <class T, bool K> struct StLoader {
    const Operand<T> &op;
    const T *p;          // first element of the next step
    size_t stride, step, k, kmax;
    int r, kk, left;     // left: rows from r on
    unsigned char alive[K ? 1 : kStLoads];   // of the next step's k, read a step ahead
    __device__ __forceinline__ StLoader(const Operand<T> &o, int row0, size_t k0, size_t k1) : op(o), kmax(k1)
    {
        const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
        r = K ? (l >> 3) + 4 * (w >> 2) : threadIdx.x % kSt;
        kk = K ? (l & 7) + 8 * (w & 3) : threadIdx.x / kSt;
        k = k0 + kk;
        left = o.rows - row0 - r;
        p = o.p + (size_t)(row0 + r) * o.row_stride + k * o.k_stride;
        stride = K ? 8 * o.row_stride : 4 * o.k_stride;
        step = kStK * o.k_stride;
        peek();
    }
    __device__ __forceinline__ void peek()
    {
        if constexpr (!K) {
#pragma unroll
            for (int q = 0; q < kStLoads; ++q) alive[q] = op.live && k + 4 * q < kmax ? op.live[k + 4 * q] : 1;
        }
    }
    __device__ __forceinline__ void load(float (&s)[kStK][kSt + 4])
    {
#pragma unroll
        for (int q = 0; q < kStLoads; ++q) {
            const bool ok = K ? 8 * q < left && k < kmax : left > 0 && k + 4 * q < kmax && alive[K ? 0 : q];
            st_put(K ? &s[kk][r + 8 * q] : &s[kk + 4 * q][r], p + q * stride, op.p, ok);
        }
        p += step;
        k += kStK;
        peek();
    }
};
static_assert(kStThreads == 8 * 32 && kSt == 64 && kStK == 32, "StLoader's cut of a step");

union StSmem {
    struct {
        float a[kStBufs][kStK][kSt + 4], b[kStBufs][kStK][kSt + 4];   // a step's products run under the next ones' loads
    };
    float z[kSt][kSt + 1];
};

// acc[i][j] = sum over k in [k0, k1) of A(m0 + 4 ty + i, k) B(n0 + 4 tx + j, k).
// Sums of 128 products are added up separately, so the rounding error grows
// with the root of K / 128, not of K.  AK / BK: the operand's k is contiguous.
template <class TA, class TB, bool AK, bool BK>
__device__ void simt_tile(const Operand<TA> &A, const Operand<TB> &B, int m0, int n0, size_t k0, size_t k1,
                          float (&acc)[4][4], StSmem &sm)
{
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float part[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) { acc[i][j] = 0.f; part[i][j] = 0.f; }
    StLoader<TA, AK> la(A, m0, k0, k1);
    StLoader<TB, BK> lb(B, n0, k0, k1);
#pragma unroll
    for (int i = 0; i < kStBufs - 1; ++i) {
        if (k0 + i * kStK < k1) { la.load(sm.a[i]); lb.load(sm.b[i]); }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    int step = 0;
    for (size_t k = k0; k < k1; k += kStK) {
        const int buf = step % kStBufs, next = (step + kStBufs - 1) % kStBufs;
        asm volatile("cp.async.wait_group %0;\n" ::"n"(kStBufs - 2) : "memory");
        __syncthreads();   // (the buffer loaded next was read in the step before)
        if (k + (kStBufs - 1) * kStK < k1) { la.load(sm.a[next]); lb.load(sm.b[next]); }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
#pragma unroll
        for (int kk = 0; kk < kStK; ++kk) {
            const float4 a = *(const float4 *)&sm.a[buf][kk][ty * 4], b = *(const float4 *)&sm.b[buf][kk][tx * 4];
            const float av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(av[i], bv[j], part[i][j]);
        }
        if (++step % kStFlush == 0 || k + kStK >= k1)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) { acc[i][j] += part[i][j]; part[i][j] = 0.f; }
    }
    asm volatile("cp.async.wait_group 0;\n" ::: "memory");
    __syncthreads();
}

// The shift of a sum of exponentials whose maximum is m: 0 where every term is
// exp(-inf) (a NaN among them still makes the sum a NaN).
__device__ __forceinline__ float exp_shift(float m) { return m == -INFINITY ? 0.f : m; }

// Forward: per (64-id tile, row) maximum and sum of exponentials of the ids but
// the row's target, and the target's logit.
template <class T>
__global__ void __launch_bounds__(kStThreads) ce_tile_simt(const T *h, const T *w, const int32_t *targets, int N, int d,
                                                           int V, float2 *rec, float *zt)
{
    extern __shared__ __align__(16) unsigned char st_smem[];
    StSmem &sm = *(StSmem *)st_smem;
    pdl_wait();
    const int m0 = blockIdx.y * kSt, n0 = blockIdx.x * kSt;
    float acc[4][4];
    const Operand<T> A{h, (size_t)d, 1, N, nullptr}, B{w, (size_t)d, 1, V, nullptr};
    simt_tile<T, T, true, true>(A, B, m0, n0, 0, d, acc, sm);
    pdl_trigger();   // (late: blocks that wait for this kernel would crowd its own onto fewer SMs)
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sm.z[ty * 4 + i][tx * 4 + j] = acc[i][j];
    __syncthreads();
    const int r = threadIdx.x >> 2, q = threadIdx.x & 3, row = m0 + r, nv = min(kSt, V - n0);
    const int t = row < N ? targets[row] : -1, tc = t < 0 ? -1 : t - n0;   // the target's column, if below nv
    float m = -INFINITY, s = 0.f;
    for (int c = q; c < nv; c += 4)
        if (c != tc) m = fmaxf(m, sm.z[r][c]);
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const float sh = exp_shift(m);
    for (int c = q; c < nv; c += 4)
        if (c != tc) s += expf(sm.z[r][c] - sh);
    s += __shfl_xor_sync(0xffffffffu, s, 1);
    s += __shfl_xor_sync(0xffffffffu, s, 2);
    if (q == 0 && row < N) {
        rec[(size_t)blockIdx.x * N + row] = make_float2(m, s);
        if (tc >= 0 && tc < nv) zt[row] = sm.z[r][tc];
    }
}

// lse and loss from the tiles' records: rx rows x 1024 / rx strands of tiles
// per block (few rows: many strands, or one row's records would be read one
// after the other).
// The target joins last: with a = log sum_{v != t} exp(z_v) - z_t the loss is
// log(1 + exp a), which keeps its digits where the target is likely (lse - z_t
// would be off by the rounding of lse, 1e-6 at 16, and by that of a sum of tiles
// near 1: at p = 0.9999 5 % of the loss).
// EXACT (tensor-core path): the tensor cores' accumulator truncates, which
// moves a logit by up to ~1e-5 of itself.  Over the vocabulary that averages
// out, but the target's logit enters the loss alone, so it is taken again, in
// fp32 parts and a double sum.
constexpr int kFinThreads = 1024;

template <bool EXACT>
__global__ void __launch_bounds__(kFinThreads) ce_finalize_kernel(const float2 *rec, const float *zt, LossArgs a,
                                                                  int n_tiles, int rx)
{
    __shared__ float sm[kFinThreads], ss[kFinThreads];
    __shared__ double sz[32];
    pdl_trigger();
    pdl_wait();
    const int N = a.N, V = a.V, strands = kFinThreads / rx;
    const int x = threadIdx.x % rx, y = threadIdx.x / rx, row = blockIdx.x * rx + x;
    if (EXACT) {   // one warp per row
        const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, r = blockIdx.x * rx + w;
        if (w < rx && r < N) {
            const int t = a.targets[r];
            if (t >= 0 && t < V) {
                const uint4 *ph = (const uint4 *)((const bf16 *)a.h + (size_t)r * a.d);
                const uint4 *pw = (const uint4 *)((const bf16 *)a.w + (size_t)t * a.d);
                float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
                for (int i = lane; i < a.d / 8; i += 32) dot8(ph[i], pw[i], acc);
                const double z = warp_sum_f64((double)(acc[0] + acc[1]) + (double)(acc[2] + acc[3]));
                if (lane == 0) sz[w] = z;
            }
        }
    }
    float m = -INFINITY, s = 0.f;
    if (row < N) {
#pragma unroll 4
        for (int i = y; i < n_tiles; i += strands) {
            const float2 v = rec[(size_t)i * N + row];
            const float mn = fmaxf(m, v.x);
            const float sh = exp_shift(mn);
            s = (m == mn ? s : s * expf(m - sh)) + v.y * expf(v.x - sh);
            m = mn;
        }
    }
    sm[threadIdx.x] = m;
    ss[threadIdx.x] = s;
    // strands join in pairs, in a fixed order
    for (int o = strands / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (y < o) {
            const int q = threadIdx.x + o * rx;
            const float m2 = sm[q], mn = fmaxf(m, m2), sh = exp_shift(mn);
            s = s * expf(m - sh) + ss[q] * expf(m2 - sh);
            m = mn;
            sm[threadIdx.x] = m;
            ss[threadIdx.x] = s;
        }
    }
    __syncthreads();
    if (y || row >= N) return;
    const int t = a.targets[row];
    const bool live = t >= 0 && t < V;
    if (t >= V && a.err) raise_err(a.err, ORTHRUS_DEVERR_TOKEN);
    const float rest = m + logf(s);   // the ids but the target
    if (!live) {
        a.lse[row] = rest;
        a.loss[row] = 0.f;
        return;
    }
    const double z = EXACT ? sz[x] : (double)zt[row];
    const float x_t = (float)z, d = (float)((double)m - z) + logf(s);
    const float e = log1pf(expf(-fabsf(d)));
    const float L = x_t == -INFINITY ? rest : d > 0.f ? rest + e : (float)(z + (double)e);
    a.lse[row] = L;
    if (!isfinite(L) && a.err) raise_err(a.err, ORTHRUS_DEVERR_NONFINITE);
    a.loss[row] = !isfinite(L) ? L - x_t : d > 0.f ? d + e : e;
}

cudaError_t launch_ce_finalize(const float2 *rec, const float *zt, const LossArgs &a, int n_tiles, int exact,
                               cudaStream_t s)
{
    int rx = 1;
    while (rx < 32 && rx < a.N) rx <<= 1;
    const int grid = (a.N + rx - 1) / rx;
    return exact ? launch_k(ce_finalize_kernel<true>, grid, kFinThreads, 0, s, rec, zt, a, n_tiles, rx)
                 : launch_k(ce_finalize_kernel<false>, grid, kFinThreads, 0, s, rec, zt, a, n_tiles, rx);
}

// dz of one piece [v0, v0 + Vp) of the vocabulary, fp32.  A row whose
// upstream gradient is zero, or that has no target, gets exact zeros
// whatever its hidden row holds.
template <class T, bool KL>
__global__ void __launch_bounds__(kStThreads) dz_tile_simt(LossArgs a, int v0, int Vp, float *dz, unsigned char *alive)
{
    extern __shared__ __align__(16) unsigned char st_smem[];
    StSmem &sm = *(StSmem *)st_smem;
    pdl_wait();
    const int m0 = blockIdx.y * kSt, n0 = v0 + blockIdx.x * kSt, d = a.d;
    const int vend = min(a.V, v0 + Vp);
    float z[4][4], z2[4][4];
    const Operand<T> A{(const T *)a.h, (size_t)d, 1, a.N, nullptr}, B{(const T *)a.w, (size_t)d, 1, a.V, nullptr};
    simt_tile<T, T, true, true>(A, B, m0, n0, 0, d, z, sm);
    if (KL) {
        const Operand<T> A2{(const T *)a.h2, (size_t)d, 1, a.N, nullptr};
        simt_tile<T, T, true, true>(A2, B, m0, n0, 0, d, z2, sm);
    }
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    pdl_trigger();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = m0 + ty * 4 + i;
        if (row >= a.N) continue;
        const float lse = a.lse_in[row];
        float g = a.g[row], lse2 = 0.f;
        int t = -1;
        if (KL) lse2 = a.lse2_in[row];
        else {
            t = a.targets[row];
            if (t >= a.V && tx == 0 && blockIdx.x == 0 && a.err) raise_err(a.err, ORTHRUS_DEVERR_TOKEN);
            if (t < 0 || t >= a.V) g = 0.f;
            if (alive && v0 == 0 && blockIdx.x == 0 && tx == 0) alive[row] = g != 0.f;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int v = n0 + tx * 4 + j;
            if (v >= vend) continue;
            float x;
            if (KL) x = expf(z2[i][j] - lse2) - expf(z[i][j] - lse);
            else x = expf(z[i][j] - lse) - (v == t ? 1.f : 0.f);   // (z's and lse's own half steps are larger than 1's)
            dz[(size_t)row * Vp + (v - v0)] = g == 0.f ? 0.f : g * x;
        }
    }
}

// C = A B^T over k in the split's share of [0, K): dh parts (fp32, added to
// what earlier pieces left) and dW rows (T).
struct GradGemm {
    int M, N, K, splits;      // C is [M][N]
    float *part;              // [splits][M][N], or null: write out
    int add;                  // add to part
    void *out;
};
template <class TA, class TB, bool AK, class TO>
__device__ __forceinline__ void grad_tile(const Operand<TA> &A, const Operand<TB> &B, const GradGemm &g, unsigned block,
                                          StSmem &sm)
{
    const unsigned nt = (g.N + kSt - 1) / kSt, mt = (g.M + kSt - 1) / kSt;
    const int n0 = block % nt * kSt, m0 = block / nt % mt * kSt, sp = block / nt / mt;
    const size_t per = (((size_t)g.K + g.splits - 1) / g.splits + kStK - 1) / kStK * kStK;
    const size_t k0 = min((size_t)g.K, per * sp), k1 = min((size_t)g.K, k0 + per);
    float acc[4][4];
    simt_tile<TA, TB, AK, false>(A, B, m0, n0, k0, k1, acc, sm);
    pdl_trigger();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + ty * 4 + i;
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n >= g.N) continue;
            const size_t o = (size_t)m * g.N + n;
            if (g.part) {
                float *p = g.part + (size_t)sp * g.M * g.N + o;
                *p = g.add ? *p + acc[i][j] : acc[i][j];
            } else {
                ((TO *)g.out)[o] = from_f<TO>(acc[i][j]);
            }
        }
    }
}

// Both products of a piece's dz in one launch (neither fills the GPU at the
// sizes this path serves): blocks below h_blocks make dh, the others dW.
template <class T>
__global__ void __launch_bounds__(kStThreads) grads_simt(Operand<float> dz, Operand<T> w, GradGemm gh, unsigned h_blocks,
                                                         Operand<float> dzt, Operand<T> h, GradGemm gw)
{
    extern __shared__ __align__(16) unsigned char st_smem[];
    StSmem &sm = *(StSmem *)st_smem;
    pdl_wait();
    if (blockIdx.x < h_blocks) grad_tile<float, T, true, T>(dz, w, gh, blockIdx.x, sm);
    else grad_tile<float, T, false, T>(dzt, h, gw, blockIdx.x - h_blocks, sm);
}

// out = sum of the splits' parts, in order, rounded once.
template <class T>
__global__ void __launch_bounds__(256) part_sum_kernel(const float *part, int splits, size_t n, T *out)
{
    pdl_wait();
    for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) {
        float s = part[i];
        for (int k = 1; k < splits; ++k) s += part[(size_t)k * n + i];
        out[i] = from_f<T>(s);
    }
    pdl_trigger();   // (late, as above: the next call's 64 blocks went to the 20 SMs that this kernel left free)
}

cudaError_t launch_part_sum(const float *part, int splits, size_t n, void *out, int dtype, cudaStream_t s)
{
    const int grid = (int)std::min<size_t>((n + 255) / 256, 8 * 148);
    if (dtype == ORTHRUS_BF16) return launch_k(part_sum_kernel<bf16>, grid, 256, 0, s, part, splits, n, (bf16 *)out);
    return launch_k(part_sum_kernel<float>, grid, 256, 0, s, part, splits, n, (float *)out);
}

__global__ void __launch_bounds__(1024) zero_kernel(void *p, size_t bytes)
{
    pdl_trigger();
    pdl_wait();
    const size_t n16 = ((uintptr_t)p & 15) == 0 ? bytes / 16 : 0;
    const size_t t = (size_t)blockIdx.x * 1024 + threadIdx.x, n = (size_t)gridDim.x * 1024;
    for (size_t i = t; i < n16; i += n) ((uint4 *)p)[i] = make_uint4(0, 0, 0, 0);
    for (size_t i = n16 * 16 + t * 2; i < bytes; i += n * 2) *(uint16_t *)((char *)p + i) = 0;
}

// ---------------------------------------------------------------- plans
struct SimtPlan {
    size_t total, o_dz, o_part, o_alive;
    int piece, splits;
};
static SimtPlan plan_simt(int N, int d, int V, int want_dw)
{
    SimtPlan p{};
    WsPlan w;
    // a piece's dz stays within 64 MiB (past 262144 rows, 256 bytes per row: a
    // piece has 64 ids at least)
    const size_t cap = std::max<size_t>(kSt, ((size_t)64 << 20) / (4 * (size_t)std::max(N, 1)) / kSt * kSt);
    p.piece = (int)std::min<size_t>(cap, ((size_t)V + kSt - 1) / kSt * kSt);
    // dh has few tiles at small N and d: its k axis (the piece) is cut until
    // the blocks cover the SMs about twice, in shares of at least 256 ids
    const long tiles = (long)((N + kSt - 1) / kSt) * ((d + kSt - 1) / kSt);
    p.splits = (int)std::max<long>(1, std::min<long>({(2 * 148 + tiles - 1) / tiles, (p.piece + 255) / 256, 32L}));
    p.o_dz = w.take((size_t)N * p.piece * 4);
    p.o_part = w.take((size_t)p.splits * N * d * 4);
    p.o_alive = w.take(want_dw ? (size_t)N : 0);
    p.total = w.total;
    return p;
}

// Room for either path: which one a bf16 call takes depends on its pointers.
size_t loss_fwd_workspace(int N, int d, int V, int dtype)
{
    WsPlan w;
    w.take((size_t)((V + kSt - 1) / kSt) * N * sizeof(float2));
    w.take((size_t)N * 4);
    return dtype == ORTHRUS_BF16 && d % 8 == 0 ? std::max(w.total, loss_fwd_workspace_tc(N, d, V)) : w.total;
}

size_t loss_grad_workspace(int N, int d, int V, int dtype, int want_dw, int kl)
{
    const size_t simt = plan_simt(N, d, V, want_dw).total;
    return dtype == ORTHRUS_BF16 && d % 8 == 0 ? std::max(simt, loss_grad_workspace_tc(N, d, V, want_dw, kl)) : simt;
}

// ---------------------------------------------------------------- launches
template <class... K, class... A>
static cudaError_t st_launch(void (*kernel)(K...), dim3 grid, cudaStream_t s, A... args)
{
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(StSmem));
    return e != cudaSuccess ? e : launch_k(kernel, grid, kStThreads, sizeof(StSmem), s, args...);
}

template <class T> static cudaError_t loss_fwd_simt(const LossArgs &a, cudaStream_t s)
{
    WsPlan w;
    const int nt = (a.V + kSt - 1) / kSt;
    float2 *rec = (float2 *)(a.ws + w.take((size_t)nt * a.N * sizeof(float2)));
    float *zt = (float *)(a.ws + w.take((size_t)a.N * 4));
    cudaError_t e = st_launch(ce_tile_simt<T>, dim3(nt, (a.N + kSt - 1) / kSt), s, (const T *)a.h,
                             (const T *)a.w, a.targets, a.N, a.d, a.V, rec, zt);
    if (e != cudaSuccess) return e;
    return launch_ce_finalize(rec, zt, a, nt, 0, s);
}

template <class T> static cudaError_t loss_grad_simt(const LossArgs &a, cudaStream_t s)
{
    const SimtPlan p = plan_simt(a.N, a.d, a.V, a.dw != nullptr);
    float *dz = (float *)(a.ws + p.o_dz), *part = (float *)(a.ws + p.o_part);
    unsigned char *alive = a.dw ? (unsigned char *)(a.ws + p.o_alive) : nullptr;
    const unsigned mt = (a.N + kSt - 1) / kSt, dt = (a.d + kSt - 1) / kSt;
    const bool direct = p.splits == 1 && p.piece >= a.V;   // dh in one share: no parts
    for (int v0 = 0; v0 < a.V; v0 += p.piece) {
        const int nv = std::min(p.piece, a.V - v0);
        const dim3 gz((nv + kSt - 1) / kSt, mt);
        cudaError_t e = a.kl ? st_launch(dz_tile_simt<T, true>, gz, s, a, v0, p.piece, dz, alive)
                             : st_launch(dz_tile_simt<T, false>, gz, s, a, v0, p.piece, dz, alive);
        if (e != cudaSuccess) return e;
        const Operand<float> A{dz, (size_t)p.piece, 1, a.N, nullptr};
        const Operand<T> B{(const T *)a.w + (size_t)v0 * a.d, 1, (size_t)a.d, a.d, nullptr};
        GradGemm g{};
        g.M = a.N; g.N = a.d; g.K = nv; g.splits = p.splits; g.part = direct ? nullptr : part; g.add = v0 > 0; g.out = a.dh;
        // a padding row's dz is zero, but zero times a NaN or an infinity in its
        // hidden row would not be: dW skips the rows that take no part
        const Operand<float> At{dz, 1, (size_t)p.piece, nv, nullptr};
        const Operand<T> Bh{(const T *)a.h, 1, (size_t)a.d, a.d, alive};
        GradGemm gw{};
        gw.M = nv; gw.N = a.d; gw.K = a.N; gw.splits = 1; gw.out = a.dw ? (T *)a.dw + (size_t)v0 * a.d : nullptr;
        const unsigned hb = dt * mt * p.splits, wb = a.dw ? dt * ((nv + kSt - 1) / kSt) : 0;
        e = st_launch(grads_simt<T>, hb + wb, s, A, B, g, hb, At, Bh, gw);
        if (e != cudaSuccess) return e;
    }
    return direct ? cudaSuccess : launch_part_sum(part, p.splits, (size_t)a.N * a.d, a.dh, a.dtype, s);
}

cudaError_t launch_loss_fwd(const LossArgs &a, cudaStream_t s)
{
    if (a.N == 0) return cudaSuccess;
    if (loss_tc_ok(a)) return loss_fwd_tc(a, s);
    return a.dtype == ORTHRUS_BF16 ? loss_fwd_simt<bf16>(a, s) : loss_fwd_simt<float>(a, s);
}

cudaError_t launch_loss_grad(const LossArgs &a, cudaStream_t s)
{
    if (a.N == 0) {   // no rows: dW is zero
        if (!a.dw) return cudaSuccess;
        return launch_k(zero_kernel, 2 * 148, 1024, 0, s, a.dw,
                        (size_t)a.V * a.d * (a.dtype == ORTHRUS_BF16 ? 2 : 4));
    }
    if (loss_tc_ok(a)) return loss_grad_tc(a, s);
    return a.dtype == ORTHRUS_BF16 ? loss_grad_simt<bf16>(a, s) : loss_grad_simt<float>(a, s);
}

}  // namespace orthrus
