// Row operators of the training side: the token embedding with scaling and
// its gradient by sorted tokens, and RMSNorm with its gradient.  All of them
// are bound by memory traffic (large calls: 16384 embedded rows of 4096 in 63
// us, 6.4 TB/s; the norm's gradient over 8192 rows of 4096 in 61 us, 5.5 TB/s)
// or by the call itself (32 rows of 2048: 3.4 us of kernel in a 10 us call).
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "train.h"

namespace orthrus {

// ---------------------------------------------------------------- vectors
// VEC elements of T as fp32: 8 when all of a kernel's tensors are bf16 (16-byte
// accesses), 4 when one is fp32 (16 bytes of it: with 8, two accesses of half
// a sector each; 16384 embedded rows of 4096 took 73 us with 8, 63 with 4), 1
// for odd row lengths and unaligned buffers.
template <class T, int VEC> struct RowVec;
template <class T> struct RowVec<T, 1> {
    static __device__ __forceinline__ void load(const T *p, float (&v)[1]) { v[0] = to_f<T>(*p); }
    static __device__ __forceinline__ void store(T *p, const float (&v)[1]) { *p = from_f<T>(v[0]); }
};
template <> struct RowVec<float, 8> {
    static __device__ __forceinline__ void load(const float *p, float (&v)[8])
    {
        const float4 a = ((const float4 *)p)[0], b = ((const float4 *)p)[1];
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[8])
    {
        ((float4 *)p)[0] = make_float4(v[0], v[1], v[2], v[3]);
        ((float4 *)p)[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
};
template <> struct RowVec<float, 4> {
    static __device__ __forceinline__ void load(const float *p, float (&v)[4])
    {
        const float4 a = *(const float4 *)p;
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    }
    static __device__ __forceinline__ void store(float *p, const float (&v)[4])
    {
        *(float4 *)p = make_float4(v[0], v[1], v[2], v[3]);
    }
};
template <> struct RowVec<bf16, 4> {
    static __device__ __forceinline__ void load(const bf16 *p, float (&v)[4])
    {
        const uint2 u = *(const uint2 *)p;
        v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    static __device__ __forceinline__ void store(bf16 *p, const float (&v)[4])
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
        *(uint2 *)p = make_uint2(*(const uint32_t *)&a, *(const uint32_t *)&b);
    }
};
template <> struct RowVec<bf16, 8> {
    static __device__ __forceinline__ void load(const bf16 *p, float (&v)[8])
    {
        const uint4 u = *(const uint4 *)p;
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // bf16 -> fp32 is a shift
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void store(bf16 *p, const float (&v)[8])
    {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *(const uint32_t *)&h;
        }
        *(uint4 *)p = make_uint4(w[0], w[1], w[2], w[3]);
    }
};

// A chunk of VEC elements as loaded, not yet converted.
template <class T, int VEC> struct RawVec {
    static constexpr int U = VEC * (int)sizeof(T) / 16;
    uint4 u[U];
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < U; ++i) u[i] = ((const uint4 *)p)[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < U; ++i) u[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void get(float (&v)[VEC]) const
    {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (sizeof(T) == 4) v[(i * 4 + k) % VEC] = __uint_as_float(w[k]);
                else {
                    v[(i * 8 + 2 * k) % VEC] = __uint_as_float(w[k] << 16);
                    v[(i * 8 + 2 * k + 1) % VEC] = __uint_as_float(w[k] & 0xffff0000u);
                }
        }
    }
};
template <> struct RawVec<bf16, 4> {
    uint2 u;
    __device__ __forceinline__ void load(const bf16 *p) { u = *(const uint2 *)p; }
    __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
    __device__ __forceinline__ void get(float (&v)[4]) const
    {
        v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
        v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
    }
};
template <class T> struct RawVec<T, 1> {
    T u;
    __device__ __forceinline__ void load(const T *p) { u = *p; }
    __device__ __forceinline__ void zero() { u = from_f<T>(0.f); }
    __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = to_f<T>(u); }
};

// Zeros in [p, p + bytes) by the n threads t = 0 .. n - 1 (p and bytes even).
__device__ __forceinline__ void zero_span(char *p, size_t bytes, size_t t, size_t n)
{
    char *a = (char *)(((uintptr_t)p + 15) & ~(uintptr_t)15), *e = p + bytes;
    if (a > e) a = e;
    char *b = a + (size_t)(e - a) / 16 * 16;
    for (char *q = p + 2 * t; q < a; q += 2 * n) *(uint16_t *)q = 0;
    for (char *q = a + 16 * t; q < b; q += 16 * n) *(uint4 *)q = make_uint4(0, 0, 0, 0);
    for (char *q = b + 2 * t; q < e; q += 2 * n) *(uint16_t *)q = 0;
}

static bool rows_aligned(const void *p, int d) { return ((uintptr_t)p & 15) == 0 && d % 8 == 0; }

// ---------------------------------------------------------------- embedding
// out[r] = scale * table[ids[r]]; a negative id is padding (a zero row).
constexpr int kEmbThreads = 256;

template <class T, class TO, int VEC>
__global__ void __launch_bounds__(kEmbThreads) embed_rows_kernel(const T *table, const int32_t *ids, TO *out, int d,
                                                                 int vocab, float scale, unsigned *err)
{
    constexpr int Q = VEC == 1 ? 4 : 16 / VEC;   // chunks of a thread in flight
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x;
    const int id = ids[row];
    const bool ok = id >= 0 && id < vocab;
    if (id >= vocab && threadIdx.x == 0 && blockIdx.y == 0 && err) raise_err(err, ORTHRUS_DEVERR_TOKEN);
    const T *src = table + (size_t)(ok ? id : 0) * d;
    TO *dst = out + (size_t)row * d;
    const int nc = d / VEC, step = gridDim.y * Q * kEmbThreads;
    for (int c0 = blockIdx.y * Q * kEmbThreads + threadIdx.x; c0 < nc; c0 += step) {
        float v[Q][VEC];
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = c0 + q * kEmbThreads;
            if (ok && c < nc) RowVec<T, VEC>::load(src + (size_t)c * VEC, v[q]);
            else
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[q][i] = 0.f;
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = c0 + q * kEmbThreads;
            if (c >= nc) continue;
            // (0 * scale stays 0 for a padding row unless the scale is not finite)
            if (ok)
#pragma unroll
                for (int i = 0; i < VEC; ++i) v[q][i] *= scale;
            RowVec<TO, VEC>::store(dst + (size_t)c * VEC, v[q]);
        }
    }
}

template <class T, class TO> static cudaError_t embed_rows_t(const EmbedRowsArgs &a, cudaStream_t s)
{
    const bool vec = rows_aligned(a.table, a.d) && rows_aligned(a.out, a.d);
    constexpr int V = sizeof(T) == 4 || sizeof(TO) == 4 ? 4 : 8;
    const int per = (vec ? 16 : 4) * kEmbThreads;   // elements a block covers per step
    // one block per row and slab of the row, so that every element is in
    // flight at once; rows beyond 64 slabs loop
    const dim3 grid(a.rows, std::min(64, (a.d + per - 1) / per));
    if (vec)
        return launch_k(embed_rows_kernel<T, TO, V>, grid, kEmbThreads, 0, s, (const T *)a.table, a.ids, (TO *)a.out,
                        a.d, a.vocab, a.scale, a.err);
    return launch_k(embed_rows_kernel<T, TO, 1>, grid, kEmbThreads, 0, s, (const T *)a.table, a.ids, (TO *)a.out, a.d,
                    a.vocab, a.scale, a.err);
}

cudaError_t launch_embed_rows(const EmbedRowsArgs &a, cudaStream_t s)
{
    const bool ib = a.dtype == ORTHRUS_BF16, ob = a.out_dtype == ORTHRUS_BF16;
    if (ib) return ob ? embed_rows_t<bf16, bf16>(a, s) : embed_rows_t<bf16, float>(a, s);
    return ob ? embed_rows_t<float, bf16>(a, s) : embed_rows_t<float, float>(a, s);
}

// ------------------------------------------------------- embedding gradient
// dE[v] = scale * sum over the rows r with ids[r] = v of dout[r], summed in
// fp32 in row order: the rows are sorted by token (stable), the sorted list
// is cut into pieces of equal length, a piece sums its runs of equal tokens,
// and a run that crosses pieces leaves one partial sum in each, joined in
// order afterwards.  A draft block's 31 mask tokens make one token 97 % of
// the rows, so a run has to be shared by many blocks; the fixed cut and
// order give the same bits on every call (no floating-point atomics).
// Ids outside [0, vocab) sort behind every token and are left out.
constexpr int kRunThreads = 128;
constexpr int kPieceMost = 4096;     // longest piece

EmbedGradPlan plan_embed_grad(int rows, int vocab, int d)
{
    EmbedGradPlan p{};
    WsPlan w;
    for (int i = 0; i < 2; ++i) {
        p.o_tok[i] = w.take((size_t)rows * 4);
        p.o_idx[i] = w.take((size_t)rows * 4);
    }
    int bits = 1;
    while (bits < 31 && (vocab >> bits) != 0) ++bits;   // keys 0 .. vocab
    p.digits = (bits + kSortDigit - 1) / kSortDigit;
    p.digit_bits = (bits + p.digits - 1) / p.digits;
    p.tiles = (rows + kSortTile - 1) / kSortTile;
    p.o_hist = w.take(rows > kRankMost ? ((size_t)p.tiles << p.digit_bits) * 4 : 0);
    // pieces: short enough that the rows spread over the SMs, long enough that
    // about 1024 blocks, and partials per column, are the most
    const int slabs = (d + 8 * kRunThreads - 1) / (8 * kRunThreads);
    p.piece = 8;
    while (p.piece < kPieceMost && (long)(rows / p.piece) * slabs > 1024) p.piece *= 2;
    p.pieces = (rows + p.piece - 1) / p.piece;
    p.o_part = w.take((size_t)p.pieces * 2 * d * 4);
    p.total = w.total;
    return p;
}

__device__ __forceinline__ int sort_key(const int32_t *ids, int r, int vocab, unsigned *err)
{
    const int id = ids[r];
    if (id >= vocab && err) raise_err(err, ORTHRUS_DEVERR_TOKEN);
    return id < 0 || id >= vocab ? vocab : id;
}

// Up to kRankMost rows: a row's place is the number of rows before it in (token,
// row) order, counted against all of them.  64 rows per block, one per lane, 16
// warps for each 32 rows, every warp over its share of the keys in shared memory
// (four per broadcast read).  The count grows with the square of the rows but is
// spread over all SMs: 15 us at 8192 rows, where a bitonic sort by one block took 37
// (1003 rows of 64 altogether 17.4 -> 9.4 us of kernels, 8000 rows of 100 56 -> 30).
constexpr int kRankThreads = 1024, kRankRows = 64, kRankStrands = kRankThreads / kRankRows;

__global__ void __launch_bounds__(kRankThreads) rank_sort_kernel(const int32_t *ids, int rows, int vocab, int blocks,
                                                                 int32_t *tok, int32_t *idx, char *zero,
                                                                 size_t zero_bytes, unsigned *err)
{
    extern __shared__ __align__(16) int32_t rank_keys[];
    __shared__ int part[kRankStrands][kRankRows];
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x >= blocks) {   // the table's first zeros, for which the memory has time
        zero_span(zero, zero_bytes, (size_t)(blockIdx.x - blocks) * kRankThreads + threadIdx.x,
                  (size_t)(gridDim.x - blocks) * kRankThreads);
        return;
    }
    const int n4 = (rows + 3) / 4;
    for (int i = threadIdx.x; i < 4 * n4; i += kRankThreads) rank_keys[i] = i < rows ? sort_key(ids, i, vocab, err) : INT_MAX;
    __syncthreads();
    const int lane = threadIdx.x & 31, group = (threadIdx.x >> 5) & 1, strand = threadIdx.x >> 6;
    const int first = blockIdx.x * kRankRows + 32 * group, row = first + lane;
    const int key = row < rows ? rank_keys[row] : 0;
    const int per = (n4 + kRankStrands - 1) / kRankStrands, c0 = min(n4, strand * per), c1 = min(n4, c0 + per);
    const int below = min(c1, max(c0, first / 4)), mixed = min(c1, max(c0, first / 4 + 8));
    const int4 *k4 = (const int4 *)rank_keys;
    int count = 0;
    // keys of rows before all of the warp's rows come first when equal, of rows after them when smaller
#pragma unroll 8
    for (int c = c0; c < below; ++c) {
        const int4 k = k4[c];
        count += (k.x <= key) + (k.y <= key) + (k.z <= key) + (k.w <= key);
    }
    for (int c = below; c < mixed; ++c) {
        const int4 k = k4[c];
        const int j = 4 * c;
        count += (k.x < key + (j < row)) + (k.y < key + (j + 1 < row)) + (k.z < key + (j + 2 < row)) +
                 (k.w < key + (j + 3 < row));
    }
#pragma unroll 8
    for (int c = mixed; c < c1; ++c) {
        const int4 k = k4[c];
        count += (k.x < key) + (k.y < key) + (k.z < key) + (k.w < key);
    }
    part[strand][32 * group + lane] = count;
    __syncthreads();
    const int r = blockIdx.x * kRankRows + threadIdx.x;
    if (threadIdx.x >= kRankRows || r >= rows) return;
    int at = 0;
#pragma unroll
    for (int q = 0; q < kRankStrands; ++q) at += part[q][threadIdx.x];
    tok[at] = rank_keys[r];
    idx[at] = r;
}

// More rows: least-significant-digit radix sort, one launch each for a
// digit's histograms (per tile of kSortTile keys), their exclusive scan, and
// the stable scatter.
constexpr int kRadixThreads = 256, kRadixWarps = kRadixThreads / 32, kRadixPer = kSortTile / kRadixThreads;

template <bool FIRST>
__global__ void __launch_bounds__(kRadixThreads) radix_hist_kernel(const int32_t *src, int rows, int vocab, int tiles,
                                                                   int shift, int bits, int *hist, unsigned *err)
{
    __shared__ int h[1 << kSortDigit];
    pdl_trigger();
    pdl_wait();
    for (int i = threadIdx.x; i < (1 << bits); i += kRadixThreads) h[i] = 0;
    __syncthreads();
    const int base = blockIdx.x * kSortTile;
#pragma unroll
    for (int j = 0; j < kRadixPer; ++j) {
        const int i = base + j * kRadixThreads + threadIdx.x;
        const int k = i < rows ? (FIRST ? sort_key(src, i, vocab, err) : src[i]) : -1;
        const int dg = k < 0 ? -1 : (k >> shift) & ((1 << bits) - 1);
        // one atomic per distinct digit of the warp (most rows may share one)
        const unsigned m = __match_any_sync(0xffffffffu, dg);
        if (dg >= 0 && (threadIdx.x & 31) == __ffs(m) - 1) atomicAdd(&h[dg], __popc(m));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < (1 << bits); i += kRadixThreads) hist[(size_t)i * tiles + blockIdx.x] = h[i];
}

// exclusive scan of n ints in place by one block
__global__ void __launch_bounds__(1024) radix_scan_kernel(int *h, int n)
{
    __shared__ int warp_tot[32];
    pdl_trigger();
    pdl_wait();
    int carry = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = 0; b < n; b += 4096) {
        int v[4], t = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = b + threadIdx.x * 4 + j;
            v[j] = i < n ? h[i] : 0;
            t += v[j];
        }
        int x = t;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) warp_tot[warp] = x;
        __syncthreads();
        if (warp == 0) {
            int w = warp_tot[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) w += y;
            }
            warp_tot[lane] = w;
        }
        __syncthreads();
        int e = carry + (warp ? warp_tot[warp - 1] : 0) + x - t;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = b + threadIdx.x * 4 + j;
            if (i < n) h[i] = e;
            e += v[j];
        }
        carry += warp_tot[31];
        __syncthreads();
    }
}

template <bool FIRST>
__global__ void __launch_bounds__(kRadixThreads) radix_scatter_kernel(const int32_t *src_tok, const int32_t *src_idx,
                                                                      int rows, int vocab, int tiles, int shift, int bits,
                                                                      const int *hist, int32_t *tok, int32_t *idx)
{
    __shared__ int cnt[kRadixWarps][1 << kSortDigit];
    pdl_trigger();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nb = 1 << bits;
    for (int i = threadIdx.x; i < kRadixWarps * nb; i += kRadixThreads) cnt[i / nb][i % nb] = 0;
    __syncthreads();
    // a warp owns kRadixPer x 32 consecutive keys, 32 at a time
    const int base = blockIdx.x * kSortTile + warp * 32 * kRadixPer;
    int key[kRadixPer], rank[kRadixPer];
#pragma unroll
    for (int j = 0; j < kRadixPer; ++j) {
        const int i = base + j * 32 + lane;
        key[j] = i < rows ? (FIRST ? sort_key(src_tok, i, vocab, nullptr) : src_tok[i]) : -1;
        const int dg = key[j] < 0 ? nb : (key[j] >> shift) & (nb - 1);
        const unsigned m = __match_any_sync(0xffffffffu, dg);
        const int before = __popc(m & ((1u << lane) - 1));
        int at = 0;
        if (dg < nb) at = cnt[warp][dg];
        __syncwarp();
        if (dg < nb && before == 0) cnt[warp][dg] = at + __popc(m);
        __syncwarp();
        rank[j] = at + before;
    }
    __syncthreads();
    // counts -> first position of (digit, warp) in the output
    for (int dg = threadIdx.x; dg < nb; dg += kRadixThreads) {
        int e = hist[(size_t)dg * tiles + blockIdx.x];
        for (int w = 0; w < kRadixWarps; ++w) {
            const int c = cnt[w][dg];
            cnt[w][dg] = e;
            e += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kRadixPer; ++j) {
        const int i = base + j * 32 + lane;
        if (i >= rows) continue;
        const int pos = cnt[warp][(key[j] >> shift) & (nb - 1)] + rank[j];
        tok[pos] = key[j];
        idx[pos] = FIRST ? i : src_idx[i];
    }
}

// One block per (piece, column slab): runs of equal tokens summed in fp32.
// Blocks from run_blocks on write the rows of zeros of the ids from zero_from on
// that do not occur: a warp takes `unit` table rows, its lanes look them up in
// the sorted tokens, and the absent ones are written.
template <class T, class TG, int VEC>
__global__ void __launch_bounds__(kRunThreads) run_sum_kernel(const T *dout, const int32_t *tok, const int32_t *idx,
                                                              int rows, int d, int vocab, int P, int slabs,
                                                              int run_blocks, int zero_from, int unit, float scale, int accumulate,
                                                              TG *dtable, float *part)
{
    constexpr int J = VEC == 8 ? 1 : 2;                       // column chunks of a thread
    constexpr int U = VEC == 8 && sizeof(T) == 4 ? 8 : 16;    // rows in flight
    // a thread's rows in flight, passed to a rolled loop (unrolled, the flushes
    // are tens of KB of code that each block fetches once)
    __shared__ RawVec<T, VEC> held[U][J][kRunThreads];
    extern __shared__ int run_smem[];
    int *st = run_smem, *si = run_smem + P;
    pdl_trigger();
    pdl_wait();
    if ((int)blockIdx.x >= run_blocks) {
        const size_t row_bytes = (size_t)d * sizeof(TG);
        const int lane = threadIdx.x & 31, step = (gridDim.x - run_blocks) * (kRunThreads / 32) * unit;
        for (int v0 = zero_from + ((blockIdx.x - run_blocks) * (kRunThreads / 32) + (threadIdx.x >> 5)) * unit; v0 < vocab;
             v0 += step) {
            const int v = v0 + lane;
            bool absent = lane < unit && v < vocab;
            if (absent) {
                int lo = 0, hi = rows;   // first place of a token >= v
                while (lo < hi) {
                    const int m = (lo + hi) >> 1;
                    if (tok[m] < v) lo = m + 1;
                    else hi = m;
                }
                absent = lo == rows || tok[lo] != v;
            }
            for (unsigned m = __ballot_sync(0xffffffffu, absent); m;) {   // spans of absent rows
                const int b = __ffs(m) - 1, n = __ffs(~(m >> b)) ? __ffs(~(m >> b)) - 1 : 32;
                zero_span((char *)dtable + (size_t)(v0 + b) * row_bytes, n * row_bytes, lane, 32);
                m = b + n < 32 ? m >> (b + n) << (b + n) : 0;
            }
        }
        return;
    }
    const int piece = blockIdx.x / slabs;
    const int lo = piece * P, hi = min(rows, lo + P), n = hi - lo;
    for (int i = threadIdx.x; i < n; i += kRunThreads) { st[i] = tok[lo + i]; si[i] = idx[lo + i]; }
    const int prev = lo > 0 ? tok[lo - 1] : -1, next = hi < rows ? tok[hi] : -1;
    __syncthreads();
    const int c0 = (blockIdx.x % slabs) * kRunThreads * J;
    float acc[J][VEC];
    auto clear = [&]() {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
            for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
    };
    auto flush = [&](int token, int b, int e) {   // run [b, e) of the piece
        if (token >= vocab) return;
        const bool head = b == 0 && prev == token, tail = e == n && next == token;
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = (c0 + j * kRunThreads + threadIdx.x) * VEC;
            if (c >= d) continue;
            if (head || tail) {
                float *p = part + ((size_t)piece * 2 + (head ? 0 : 1)) * d + c;
                RowVec<float, VEC>::store(p, acc[j]);
            } else {
                TG *o = dtable + (size_t)token * d + c;
                float old[VEC], v[VEC];
                if (accumulate) RowVec<TG, VEC>::load(o, old);
#pragma unroll
                for (int q = 0; q < VEC; ++q) v[q] = accumulate ? fmaf(scale, acc[j][q], old[q]) : scale * acc[j][q];
                RowVec<TG, VEC>::store(o, v);
            }
        }
    };
    clear();
    int cur = st[0], begin = 0;
    for (int r0 = 0; r0 < n; r0 += U) {
        RawVec<T, VEC> v[U][J];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int c = (c0 + j * kRunThreads + threadIdx.x) * VEC;
                if (r0 + u < n && c < d && st[r0 + u] < vocab) v[u][j].load(dout + (size_t)si[r0 + u] * d + c);
                else v[u][j].zero();
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < J; ++j) held[u][j][threadIdx.x] = v[u][j];
        const int m = min(U, n - r0);
#pragma unroll 1
        for (int u = 0; u < m; ++u) {
            const int t = st[r0 + u];
            if (t != cur) {
                flush(cur, begin, r0 + u);
                clear();
                cur = t;
                begin = r0 + u;
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
                float x[VEC];
                held[u][j][threadIdx.x].get(x);
#pragma unroll
                for (int e = 0; e < VEC; ++e) acc[j][e] += x[e];
            }
        }
    }
    flush(cur, begin, n);
}

// Runs that cross pieces: the piece a run starts in adds up its partials in
// order.  A block looks at up to 32 pieces (blockIdx.x, + gridDim.x, ..) for
// runs that start there; 32 threads of VEC columns x 8 strands of pieces add
// up, and the strands join in order too.
constexpr int kJoinLanes = 32, kJoinStrands = 8, kJoinThreads = kJoinLanes * kJoinStrands;
constexpr int kJoinBlocks = 64;

template <class TG, int VEC>
__global__ void __launch_bounds__(kJoinThreads) run_join_kernel(const int32_t *tok, int rows, int d, int vocab, int pieces,
                                                                int P, float scale, int accumulate, TG *dtable,
                                                                const float *part)
{
    __shared__ float red[kJoinStrands][kJoinLanes * VEC];
    __shared__ unsigned starts;
    pdl_trigger();
    pdl_wait();
    const int x = threadIdx.x % kJoinLanes, y = threadIdx.x / kJoinLanes;
    if (y == 0) {
        const int q = blockIdx.x + x * gridDim.x, lo = q * P, hi = lo + P;
        bool s = false;
        if (q < pieces - 1) {   // (the last piece has no successor)
            const int a = tok[hi - 1], b = tok[hi], c = tok[lo], e = lo > 0 ? tok[lo - 1] : -1;
            s = a == b && a < vocab && !(c == a && e == a);   // leaves the piece, and did not enter it
        }
        const unsigned m = __ballot_sync(0xffffffffu, s);
        if (x == 0) starts = m;
    }
    __syncthreads();
    const int c = (blockIdx.y * kJoinLanes + x) * VEC;
    for (unsigned m = starts; m; m &= m - 1) {
        const int piece = blockIdx.x + (__ffs(m) - 1) * gridDim.x, cur = tok[(piece + 1) * P];
        int n = 0;   // pieces after this one that begin with the run
        for (int q0 = piece + 1;; q0 += kJoinThreads) {
            const int q = q0 + threadIdx.x;
            const int k = __syncthreads_count(q < pieces && tok[q * P] == cur);
            n += k;
            if (k < kJoinThreads) break;
        }
        float sum[VEC];
#pragma unroll
        for (int e = 0; e < VEC; ++e) sum[e] = 0.f;
        if (c < d) {
            const float *p = part + (size_t)piece * 2 * d + c;
            auto add = [&](const float *f) {
                if constexpr (VEC == 4) {
                    const float4 v = *(const float4 *)f;
                    sum[0] += v.x; sum[1] += v.y; sum[2] += v.z; sum[3] += v.w;
                } else {
                    sum[0] += *f;
                }
            };
            if (y == 0) add(p + d);
#pragma unroll 8
            for (int q = 1 + y; q <= n; q += kJoinStrands) add(p + (size_t)q * 2 * d);
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) red[y][x * VEC + e] = sum[e];
        __syncthreads();
        for (int i = threadIdx.x; i < kJoinLanes * VEC; i += kJoinThreads) {
            const int col = blockIdx.y * kJoinLanes * VEC + i;
            if (col >= d) continue;
            float t = red[0][i];
#pragma unroll
            for (int k = 1; k < kJoinStrands; ++k) t += red[k][i];
            TG *o = dtable + (size_t)cur * d + col;
            *o = from_f<TG>(accumulate ? fmaf(scale, t, to_f<TG>(*o)) : scale * t);
        }
        __syncthreads();
    }
}

__global__ void __launch_bounds__(1024) fill_zero_kernel(char *p, size_t bytes)
{
    pdl_trigger();
    pdl_wait();
    zero_span(p, bytes, (size_t)blockIdx.x * 1024 + threadIdx.x, (size_t)gridDim.x * 1024);
}

template <class T, class TG>
static cudaError_t run_sums(const EmbedGradArgs &a, const EmbedGradPlan &p, const int32_t *tok, const int32_t *idx,
                            int zero_from, cudaStream_t s)
{
    float *part = (float *)(a.ws + p.o_part);
    const bool vec = rows_aligned(a.dout, a.d) && rows_aligned(a.dtable, a.d);
    const int cols = vec ? 8 * kRunThreads : 2 * kRunThreads, slabs = (a.d + cols - 1) / cols;
    const int run_blocks = p.pieces * slabs;
    // zeros: about 32 KiB of table rows per warp, so that the blocks, started in
    // order, write the table in order (8 blocks per SM that stride over it: 250 us
    // instead of 216 for 8192 rows of 4096, vocabulary 151936, of a floor of 204)
    const size_t row_bytes = (size_t)a.d * sizeof(TG);
    const int unit = (int)std::max<size_t>(1, std::min<size_t>(32, 32768 / row_bytes));
    const int units = (a.vocab - zero_from + unit - 1) / unit, per = kRunThreads / 32;
    const int fill_blocks = (units + per - 1) / per;
    auto sum = [&](auto kernel) {
        // a long piece's tokens beside the rows in flight: more than the 48 KiB of a plain launch (the limit is the
        // process's, so it is set to the most that any call needs: another thread's call may lie between the two)
        if (p.piece > 1024) {
            const cudaError_t ea = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPieceMost * 8);
            if (ea != cudaSuccess) return ea;
        }
        return launch_k(kernel, run_blocks + fill_blocks, kRunThreads, (size_t)p.piece * 8, s, (const T *)a.dout, tok, idx,
                        a.rows, a.d, a.vocab, p.piece, slabs, run_blocks, zero_from, unit, a.scale, a.accumulate, (TG *)a.dtable, part);
    };
    cudaError_t e = vec ? sum(run_sum_kernel<T, TG, 8>) : sum(run_sum_kernel<T, TG, 1>);
    if (e != cudaSuccess || p.pieces < 2) return e;
    auto join = [&](auto kernel, int per) {
        // (few columns: more blocks, each with fewer pieces to look at)
        const int cols = (a.d + per - 1) / per, wide = std::max(kJoinBlocks, 16 * 148 / cols);
        return launch_k(kernel, dim3(std::min(wide, p.pieces - 1), cols), kJoinThreads, 0, s, tok,
                        a.rows, a.d, a.vocab, p.pieces, p.piece, a.scale, a.accumulate, (TG *)a.dtable, (const float *)part);
    };
    return a.d % 4 == 0 ? join(run_join_kernel<TG, 4>, kJoinLanes * 4) : join(run_join_kernel<TG, 1>, kJoinLanes);
}

cudaError_t launch_embed_grad(const EmbedGradArgs &a, cudaStream_t s)
{
    cudaError_t e;
    if (a.rows == 0) {
        if (a.accumulate) return cudaSuccess;
        const size_t bytes = (size_t)a.vocab * a.d * (a.dtable_dtype == ORTHRUS_BF16 ? 2 : 4);
        return launch_k(fill_zero_kernel, (int)std::min<size_t>(2 * 148, (bytes + 16383) / 16384), 1024, 0, s,
                        (char *)a.dtable, bytes);
    }
    const EmbedGradPlan p = plan_embed_grad(a.rows, a.vocab, a.d);
    int32_t *tok[2] = {(int32_t *)(a.ws + p.o_tok[0]), (int32_t *)(a.ws + p.o_tok[1])};
    int32_t *idx[2] = {(int32_t *)(a.ws + p.o_idx[0]), (int32_t *)(a.ws + p.o_idx[1])};
    int cur = 0, zero_from = a.accumulate ? a.vocab : 0;   // the sums' launch writes the zeros from this id on
    if (a.rows <= kRankMost) {
        const size_t smem = (size_t)(a.rows + 3) / 4 * 16;
        if (smem > 40960) {   // (beside the partial counts, within 48 KiB of a plain launch)
            e = cudaFuncSetAttribute(rank_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRankMost * 4);
            if (e != cudaSuccess) return e;
        }
        // beside the sort (4 us, and 15 us at 8192 rows) the memory writes 6 TB/s of zeros
        const int blocks = (a.rows + kRankRows - 1) / kRankRows;
        const size_t row_bytes = (size_t)a.d * (a.dtable_dtype == ORTHRUS_BF16 ? 2 : 4);
        if (!a.accumulate)
            zero_from = (int)std::min<size_t>(a.vocab, (((size_t)16 << 20) + (size_t)a.rows * a.rows) / row_bytes);
        const size_t zero_bytes = a.accumulate ? 0 : zero_from * row_bytes;
        const int fill = (int)std::min<size_t>(148, (zero_bytes + 32767) / 32768);
        e = launch_k(rank_sort_kernel, blocks + fill, kRankThreads, smem, s, a.ids, a.rows, a.vocab, blocks, tok[0], idx[0],
                     (char *)a.dtable, zero_bytes, a.err);
        if (e != cudaSuccess) return e;
    } else {
        int *hist = (int *)(a.ws + p.o_hist);
        const int32_t *st = a.ids, *si = nullptr;
        for (int pass = 0; pass < p.digits; ++pass) {
            const int shift = pass * p.digit_bits;
            if (pass == 0)
                e = launch_k(radix_hist_kernel<true>, p.tiles, kRadixThreads, 0, s, st, a.rows, a.vocab, p.tiles, shift,
                             p.digit_bits, hist, a.err);
            else
                e = launch_k(radix_hist_kernel<false>, p.tiles, kRadixThreads, 0, s, st, a.rows, a.vocab, p.tiles, shift,
                             p.digit_bits, hist, a.err);
            if (e != cudaSuccess) return e;
            e = launch_k(radix_scan_kernel, 1, 1024, 0, s, hist, p.tiles << p.digit_bits);
            if (e != cudaSuccess) return e;
            if (pass == 0)
                e = launch_k(radix_scatter_kernel<true>, p.tiles, kRadixThreads, 0, s, st, si, a.rows, a.vocab, p.tiles,
                             shift, p.digit_bits, (const int *)hist, tok[0], idx[0]);
            else
                e = launch_k(radix_scatter_kernel<false>, p.tiles, kRadixThreads, 0, s, st, si, a.rows, a.vocab, p.tiles,
                             shift, p.digit_bits, (const int *)hist, tok[pass & 1], idx[pass & 1]);
            if (e != cudaSuccess) return e;
            cur = pass & 1;
            st = tok[cur];
            si = idx[cur];
        }
    }
    const bool ib = a.dout_dtype == ORTHRUS_BF16, ob = a.dtable_dtype == ORTHRUS_BF16;
    if (ib)
        return ob ? run_sums<bf16, bf16>(a, p, tok[cur], idx[cur], zero_from, s)
                  : run_sums<bf16, float>(a, p, tok[cur], idx[cur], zero_from, s);
    return ob ? run_sums<float, bf16>(a, p, tok[cur], idx[cur], zero_from, s)
              : run_sums<float, float>(a, p, tok[cur], idx[cur], zero_from, s);
}

// ---------------------------------------------------------------- RMSNorm
// Forward: y = x r g with r = (mean x^2 + eps)^-1/2, in fp32.  G threads per
// row; the first J chunks of a thread stay in registers between the sum and
// the output, longer rows are read again.
constexpr int kNormRowsThreads = 256;

// Sum over the G threads of a row: a warp, or the whole block.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float *red)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (G == 32) return;
    constexpr int W = G / 32;
    const int gi = threadIdx.x / G, w = (threadIdx.x % G) >> 5, lane = threadIdx.x & 31;
    float *r = red + gi * W * N;
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) r[w * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float t = 0.f;
#pragma unroll
        for (int k = 0; k < W; ++k) t += r[k * N + i];
        v[i] = t;
    }
}

template <class TX, class T, int VEC, int G>
__global__ void __launch_bounds__(kNormRowsThreads) norm_rows_kernel(const TX *x, const T *gain, T *y, int rows, int d,
                                                                     float eps)
{
    constexpr int J = VEC == 8 ? 4 : 8;
    __shared__ float red[kNormRowsThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x * (kNormRowsThreads / G) + threadIdx.x / G, t = threadIdx.x % G;
    const TX *xr = x + (size_t)row * d;
    const int nc = row < rows ? d / VEC : 0;   // (no row: no chunks)
    float v[J][VEC], ss[1] = {0.f};
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = t + j * G;
        if (c < nc) RowVec<TX, VEC>::load(xr + (size_t)c * VEC, v[j]);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e) v[j][e] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] = fmaf(v[j][e], v[j][e], ss[0]);
    for (int c = t + J * G; c < nc; c += G) {
        float u[VEC];
        RowVec<TX, VEC>::load(xr + (size_t)c * VEC, u);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss[0] = fmaf(u[e], u[e], ss[0]);
    }
    group_sum<G, 1>(ss, red);
    const float r = 1.0f / sqrtf(ss[0] / (float)d + eps);
    T *yr = y + (size_t)row * d;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = t + j * G;
        if (c >= nc) continue;
        float g[VEC], o[VEC];
        RowVec<T, VEC>::load(gain + (size_t)c * VEC, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = v[j][e] * r * g[e];
        RowVec<T, VEC>::store(yr + (size_t)c * VEC, o);
    }
    for (int c = t + J * G; c < nc; c += G) {
        float u[VEC], g[VEC], o[VEC];
        RowVec<TX, VEC>::load(xr + (size_t)c * VEC, u);
        RowVec<T, VEC>::load(gain + (size_t)c * VEC, g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) o[e] = u[e] * r * g[e];
        RowVec<T, VEC>::store(yr + (size_t)c * VEC, o);
    }
}

template <class TX, class T> static cudaError_t norm_rows_t(const NormArgs &a, cudaStream_t s)
{
    const bool vec = rows_aligned(a.x, a.d) && rows_aligned(a.gain, a.d) && rows_aligned(a.out, a.d);
    auto go = [&](auto kernel, int G) {
        const int per = kNormRowsThreads / G;
        return launch_k(kernel, (a.rows + per - 1) / per, kNormRowsThreads, 0, s, (const TX *)a.x, (const T *)a.gain,
                        (T *)a.out, a.rows, a.d, a.eps);
    };
    // threads per row: as few as hold it in registers, so that each has up to
    // four 16- or 32-byte loads in flight (8192 x 2048, fp32 x: 25.4 us with 256 threads a row, 14.4 us with 64)
    constexpr int V = sizeof(T) == 4 ? 4 : 8;   // (only y is written: 8 bf16 of it are one access)
    if (vec)
        return a.d <= 1024 ? go(norm_rows_kernel<TX, T, V, 32>, 32)
               : a.d <= 2048 ? go(norm_rows_kernel<TX, T, V, 64>, 64)
               : a.d <= 4096 ? go(norm_rows_kernel<TX, T, V, 128>, 128)
                             : go(norm_rows_kernel<TX, T, V, 256>, 256);
    return a.d <= 256 ? go(norm_rows_kernel<TX, T, 1, 32>, 32) : go(norm_rows_kernel<TX, T, 1, 256>, 256);
}

cudaError_t launch_norm_rows(const NormArgs &a, cudaStream_t s)
{
    const bool xb = a.x_dtype == ORTHRUS_BF16, yb = a.dtype == ORTHRUS_BF16;
    if (xb) return yb ? norm_rows_t<bf16, bf16>(a, s) : cudaErrorNotSupported;
    return yb ? norm_rows_t<float, bf16>(a, s) : norm_rows_t<float, float>(a, s);
}

// Gradient.  With u = g dy, A = sum x^2, B = sum u x over a row and
// r = (A/d + eps)^-1/2:
//     dx = r u - k x, k = r^2 (r B / d),     dgain = sum over rows of dy x r.
// k's factors in that order: r^3 leaves fp32 where k does not (rows of 1e-14
// with eps = 0, or of 1e15), r^2 only where the row's sum of squares does too.
// One pass: a row's x and dy are read once into registers, both sums are
// reduced together, dx is written, and dgain's columns stay in the thread's
// registers over all rows the block takes; each block leaves its column sums
// in the workspace and a second kernel adds the blocks up in a fixed order.
// The next row's loads are issued before this row's sums are joined, or the
// memory would idle behind every row's barrier (8192 x 4096, fp32 x: 128 us without, 70 with,
// 61 with 4 fp32 per access, of a floor of 52 us).
constexpr int kNgThreads = 512;
constexpr int kNgMaxCols = 8192;     // longest row the register path holds
constexpr int kNgBlocks = 2 * 148;   // blocks: two per SM

template <class TX, class T, int VEC, int G, int J>
__global__ void __launch_bounds__(kNgThreads, VEC * J == 8 ? 2 : 1)
    norm_grad_kernel(const TX *x, const T *gain, const T *dy, TX *dx, int rows, int d, float eps, float *part)
{
    constexpr int R = kNgThreads / G;   // rows of a block at a time
    __shared__ float red[2][2 * kNgThreads / 32];
    __shared__ float comb[R > 1 ? kNgThreads * VEC : 1];
    pdl_trigger();
    const int gi = threadIdx.x / G, t = threadIdx.x % G, nc = d / VEC;
    pdl_wait();
    RawVec<TX, VEC> rx[J];
    RawVec<T, VEC> ry[J];
    auto fetch = [&](int row) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = t + j * G;
            if (row < rows && c < nc) {
                rx[j].load(x + (size_t)row * d + (size_t)c * VEC);
                ry[j].load(dy + (size_t)row * d + (size_t)c * VEC);
            } else {
                rx[j].zero();
                ry[j].zero();
            }
        }
    };
    fetch(blockIdx.x * R + gi);
    RawVec<T, VEC> rg[J];
    float acc[J][VEC];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = t + j * G;
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[j][e] = 0.f;
        if (c < nc) rg[j].load(gain + (size_t)c * VEC);
        else rg[j].zero();
    }
    int flip = 0;
    for (int r0 = blockIdx.x * R; r0 < rows; r0 += gridDim.x * R, flip ^= 1) {
        const int row = r0 + gi;
        const bool live = row < rows;
        float xv[J][VEC], u[J][VEC], s[2] = {0.f, 0.f};
#pragma unroll
        for (int j = 0; j < J; ++j) { rx[j].get(xv[j]); ry[j].get(u[j]); }
        fetch(row + gridDim.x * R);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            float g[VEC];
            rg[j].get(g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[0] = fmaf(xv[j][e], xv[j][e], s[0]);
                s[1] = fmaf(u[j][e] * g[e], xv[j][e], s[1]);
            }
        }
        // (two buffers: a block reads one while the next row writes the other)
        group_sum<G, 2>(s, red[flip]);
        const float r = 1.0f / sqrtf(s[0] / (float)d + eps), k = (r * r) * (r * (s[1] / (float)d));
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int c = t + j * G;
            if (!live || c >= nc) continue;
            float o[VEC], g[VEC];
            rg[j].get(g);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                o[e] = r * (u[j][e] * g[e]) - k * xv[j][e];
                acc[j][e] = fmaf(u[j][e] * xv[j][e], r, acc[j][e]);
            }
            RowVec<TX, VEC>::store(dx + (size_t)row * d + (size_t)c * VEC, o);
        }
    }
    float *p = part + (size_t)blockIdx.x * d;
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = t + j * G;
        if (R > 1) {   // the block's row groups, in order
            __syncthreads();
#pragma unroll
            for (int e = 0; e < VEC; ++e) comb[threadIdx.x * VEC + e] = acc[j][e];
            __syncthreads();
            if (gi == 0)
#pragma unroll
                for (int e = 0; e < VEC; ++e)
                    for (int q = 1; q < R; ++q) acc[j][e] += comb[(q * G + t) * VEC + e];
        }
        if (gi == 0 && c < nc) RowVec<float, VEC>::store(p + (size_t)c * VEC, acc[j]);
    }
}

// Rows longer than kNgMaxCols: row statistics and dx by one block per row
// (x and dy are read twice), dgain by blocks of columns over strips of rows.
template <class TX, class T>
__global__ void __launch_bounds__(kNgThreads) norm_grad_long_kernel(const TX *x, const T *gain, const T *dy, TX *dx,
                                                                    int rows, int d, float eps, float *rstd)
{
    __shared__ float red[2 * kNgThreads / 32];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x;
    const TX *xr = x + (size_t)row * d;
    const T *yr = dy + (size_t)row * d;
    float s[2] = {0.f, 0.f};
    for (int c = threadIdx.x; c < d; c += kNgThreads) {
        const float xv = to_f<TX>(xr[c]);
        s[0] = fmaf(xv, xv, s[0]);
        s[1] = fmaf(to_f<T>(yr[c]) * to_f<T>(gain[c]), xv, s[1]);
    }
    group_sum<kNgThreads, 2>(s, red);
    const float r = 1.0f / sqrtf(s[0] / (float)d + eps), k = (r * r) * (r * (s[1] / (float)d));
    if (threadIdx.x == 0) rstd[row] = r;
    for (int c = threadIdx.x; c < d; c += kNgThreads) {
        const float xv = to_f<TX>(xr[c]);
        dx[(size_t)row * d + c] = from_f<TX>(r * (to_f<T>(yr[c]) * to_f<T>(gain[c])) - k * xv);
    }
}

template <class TX, class T>
__global__ void __launch_bounds__(256) norm_grad_cols_kernel(const TX *x, const T *dy, const float *rstd, int rows, int d,
                                                             float *part)
{
    pdl_trigger();
    pdl_wait();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    float acc = 0.f;
    for (int r = blockIdx.y; r < rows; r += gridDim.y)
        acc = fmaf(to_f<T>(dy[(size_t)r * d + c]) * to_f<TX>(x[(size_t)r * d + c]), rstd[r], acc);
    part[(size_t)blockIdx.y * d + c] = acc;
}

// dgain[c] = sum over blocks of part[block][c], 8 strands joined in order
__global__ void __launch_bounds__(256) dgain_kernel(const float *part, int blocks, int d, float *dgain)
{
    __shared__ float red[8][32];
    pdl_trigger();
    pdl_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + x;
    float s = 0.f;
    if (c < d)
#pragma unroll 8
        for (int b = y; b < blocks; b += 8) s += part[(size_t)b * d + c];
    red[y][x] = s;
    __syncthreads();
    if (y == 0 && c < d) {
        float t = red[0][x];
#pragma unroll
        for (int k = 1; k < 8; ++k) t += red[k][x];
        dgain[c] = t;
    }
}

size_t norm_grad_workspace(int rows, int d)
{
    WsPlan w;
    w.take((size_t)kNgBlocks * d * 4);
    w.take(d > kNgMaxCols ? (size_t)rows * 4 : 0);
    return w.total;
}

template <class TX, class T> static cudaError_t norm_grad_t(const NormArgs &a, cudaStream_t s)
{
    const bool vec = rows_aligned(a.x, a.d) && rows_aligned(a.gain, a.d) && rows_aligned(a.dy, a.d) &&
                     rows_aligned(a.out, a.d);
    float *part = (float *)a.ws;
    int blocks = 0;
    cudaError_t e;
    if (a.d > kNgMaxCols) {
        WsPlan w;
        w.take((size_t)kNgBlocks * a.d * 4);
        float *rstd = (float *)(a.ws + w.take((size_t)a.rows * 4));
        e = launch_k(norm_grad_long_kernel<TX, T>, a.rows, kNgThreads, 0, s, (const TX *)a.x, (const T *)a.gain,
                     (const T *)a.dy, (TX *)a.out, a.rows, a.d, a.eps, rstd);
        if (e != cudaSuccess) return e;
        blocks = std::min(32, a.rows);
        e = launch_k(norm_grad_cols_kernel<TX, T>, dim3((a.d + 255) / 256, blocks), 256, 0, s, (const TX *)a.x,
                     (const T *)a.dy, (const float *)rstd, a.rows, a.d, part);
    } else {
        auto go = [&](auto kernel, int G) {
            const int R = kNgThreads / G;
            blocks = std::min(kNgBlocks, (a.rows + R - 1) / R);
            return launch_k(kernel, blocks, kNgThreads, 0, s, (const TX *)a.x, (const T *)a.gain, (const T *)a.dy,
                            (TX *)a.out, a.rows, a.d, a.eps, part);
        };
        // threads per row: as few as hold the row in registers
        constexpr int V = sizeof(TX) == 4 ? 4 : 8, J = 8 / V;
        if (vec)
            e = a.d <= 256 ? go(norm_grad_kernel<TX, T, V, 32, J>, 32)
                : a.d <= 1024 ? go(norm_grad_kernel<TX, T, V, 128, J>, 128)
                : a.d <= 2048 ? go(norm_grad_kernel<TX, T, V, 256, J>, 256)
                : a.d <= 4096 ? go(norm_grad_kernel<TX, T, V, 512, J>, 512)
                              : go(norm_grad_kernel<TX, T, V, 512, 2 * J>, 512);
        else
            e = a.d <= 512 ? go(norm_grad_kernel<TX, T, 1, 32, 16>, 32)
                : a.d <= 2048 ? go(norm_grad_kernel<TX, T, 1, 128, 16>, 128)
                              : go(norm_grad_kernel<TX, T, 1, 512, 16>, 512);
    }
    if (e != cudaSuccess) return e;
    return launch_k(dgain_kernel, (a.d + 31) / 32, 256, 0, s, (const float *)part, blocks, a.d, a.dgain);
}

cudaError_t launch_norm_grad(const NormArgs &a, cudaStream_t s)
{
    if (a.rows == 0) return launch_k(dgain_kernel, (a.d + 31) / 32, 256, 0, s, (const float *)nullptr, 0, a.d, a.dgain);
    const bool xb = a.x_dtype == ORTHRUS_BF16, yb = a.dtype == ORTHRUS_BF16;
    if (xb) return yb ? norm_grad_t<bf16, bf16>(a, s) : cudaErrorNotSupported;
    return yb ? norm_grad_t<float, bf16>(a, s) : norm_grad_t<float, float>(a, s);
}

}  // namespace orthrus
