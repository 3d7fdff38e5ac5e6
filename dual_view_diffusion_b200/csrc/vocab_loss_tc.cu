// The vocabulary losses on the 5th-generation tensor cores (bf16, rows of a
// multiple of 8 elements, 16-byte aligned buffers).
//
// One persistent kernel runs every product of the losses as tiles of 256 x bn
// per pair of SMs (tcgen05.mma.cta_group::2: each CTA of a 2-CTA cluster
// holds 128 rows of A and bn/2 rows of B in shared memory and 128 accumulator
// rows in its TMEM, so a k step reads half the shared memory of two separate
// 128-row tiles, which is what held those back).  What differs between the
// products is the operands' order in memory and the epilogue:
//
//   LSE   z = h W^T          epilogue: (max, sum exp) per (row, tile) of the ids
//                            but the target
//   DZ    z = h W^T          epilogue: dz = g exp(z - lse), the target's from
//                            vl_target_kernel, bf16
//   DZKL  z of interleaved (AR, diffusion) rows: dz = g (p_diff - p_AR), bf16
//   DH    dh += dz W         A = dz rows, B = W read along its rows (MN-major)
//   DW    dW  = dz^T h       both operands MN-major
//
// With few rows these products stream W once and little else.  LSE_T, DZ_T,
// DZKL_T and DH_T then take W as the 256-row operand and the rows as bn
// (32 .. 256) columns: a stage is nearly all weights, so the ring keeps up to
// 192 KB of them in flight per SM instead of 48.
//
//   warp 0      producer: one thread issues the CTA's TMA loads into a ring of
//               shared-memory stages; both CTAs' loads count on the first
//               CTA's mbarrier
//   warp 1      MMA issuer (first CTA of the pair only)
//   warps 4..11 epilogue: one accumulator row per thread, 32 columns at a time;
//               two warps share 32 rows and take every other 32 columns
//
// Two accumulators (2 x 256 TMEM columns) let the next tile's MMAs run under
// an epilogue.  Every wait is bounded: on timeout the kernel raises
// ORTHRUS_DEVERR_TIMEOUT, stops issuing, lets its copies land and still frees
// its TMEM.
//
// Measured: 4096 rows of 4096 over 151936 ids, forward 3.4 to 3.7 ms (1.4 to 1.5
// PFLOP/s, the sustained rate of a library product), both gradients 11.7 to 12.1 ms
// (three products, 1.3 PFLOP/s; tensor pipe 80 to 87 % active, the rest the
// ramps of a launch per product and piece, and L2 waits).  Few rows: forward of one row of 2048, 113 us
// of 97 for W's 622 MB; the gradients read W twice (31 rows: 204 us frozen head,
// 206 to 210 KL, of 193 for that).  A narrow product is close to its own bound there too: each MMA takes
// as long as a 256-column one, which passes W at 52 GB/s per SM.
#include <cuda.h>
#include <string.h>

#include <algorithm>

#include "common.cuh"
#include "train.h"

namespace orthrus {

bool make_tmap_box(CUtensorMap *m, const void *ptr, uint64_t rows, uint64_t cols, uint32_t box_cols, uint32_t box_rows);

constexpr int kVlThreads = 384;
constexpr int kVlEpi = 256;                    // epilogue threads per CTA
constexpr int kVlM = 256;                      // rows of a pair's tile
constexpr int kVlNMax = 256;                   // columns of a pair's tile
constexpr int kVlK = 128;                      // k per stage: eight MMAs for each wait and commit
constexpr uint32_t kVlABytes = 128 * kVlK * 2; // A bytes of a CTA's stage
constexpr int kVlStages = 6;                   // most ring stages (3 at bn = 256)
constexpr uint32_t kVlRing = 221184;           // most bytes of the ring: 3 stages of 64 KiB, or 6 at bn = 32
constexpr uint32_t kVlShared = 229376;         // the ring and what an epilogue keeps behind it
constexpr int kVlPairs = 74;                   // 2-CTA clusters that fit at once on 148 SMs
constexpr long long kVlSpinCycles = 4000000000LL;   // ~2 s at the B200 SM clock
constexpr float kLog2e = 1.4426950408889634f;

enum VlKind : int { VL_LSE = 0, VL_DZ = 1, VL_DZKL = 2, VL_DH = 3, VL_DW = 4, VL_LSE_T = 5, VL_DZ_T = 6, VL_DZKL_T = 7,
                    VL_DH_T = 8 };

// The product of a launch: mt x nt x splits tiles; pair p takes tiles p, p + pairs, ..
struct VlJob {
    CUtensorMap a, b, c;   // c (DZ, DZKL, DW): the result, boxes of 64 columns x a warp's rows
    int kind;
    int M, N;            // valid rows and columns of the result
    int chunks, splits;  // k chunks of kVlK, and the shares they are cut into (DH)
    int kr;              // k of a chunk that are loaded and multiplied: kVlK, or fewer (DW of few rows)
    int bn, mt, nt;
    int a_mn, b_mn;      // operand order in memory: 1 = MN-major
    int a_off, b_off;    // first row (K-major) or k row (MN-major): the piece's offset in W
    int n_fast;          // tile order: 1 = columns first, 0 = rows first
    // epilogue
    const int32_t *targets;
    const float *lse, *lse2, *g;
    const float *et;     // DZ, DZ_T: exp(z - lse) - 1 of the rows' targets
    float2 *rec;         // LSE: [nt][M]; LSE_T: [groups of 32 ids][N]
    bf16 *dz;            // DZ_T: [rows][pitch]
    int v0, V, pitch;    // DZ: the piece's first id, the vocabulary, dz's row length
    float *part;         // DH: [splits][M][N] fp32
    int add, last;       // DH: add to part; the last piece of an unsplit dh: write out
    bf16 *out;           // DH: [M][N]
    int c_off;           // DW: first row of the result
};
struct VlParams {
    VlJob job;
    int pairs, stages;
    uint32_t stage_bytes;
    unsigned *err;
};

// ---------------------------------------------------------------- PTX wrappers
__device__ __forceinline__ void vl_mbar_init(uint64_t *b, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(smem_u32(b)), "r"(count));
}
__device__ __forceinline__ void vl_expect_tx(uint64_t *b, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(smem_u32(b)), "r"(bytes) : "memory");
}
// arrive on the barrier at shared::cluster address a (this CTA's or the peer's)
__device__ __forceinline__ void vl_arrive_at(uint32_t a)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(a) : "memory");
}
__device__ __forceinline__ bool vl_try(uint64_t *b, uint32_t parity)
{
    uint32_t ok;
    asm volatile("{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
                 " selp.u32 %0, 1, 0, p;\n}\n"
                 : "=r"(ok) : "r"(smem_u32(b)), "r"(parity) : "memory");
    return ok != 0;
}
// Bounded wait (about two seconds of SM clock); false on timeout, or when
// another role of the CTA already gave up.
__device__ __forceinline__ bool vl_wait(uint64_t *b, uint32_t parity, volatile int *abort)
{
    if (vl_try(b, parity)) return true;
    const long long t0 = clock64();
    for (long i = 0;; ++i) {
        if (vl_try(b, parity)) return true;
        if ((i & 15) == 15) {   // (a try may itself be suspended for a while)
            if (*abort) return false;
            if (clock64() - t0 > kVlSpinCycles) break;
        }
    }
    *abort = 1;
    return false;
}
__device__ __forceinline__ uint32_t vl_mapa(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
// TMA tile load whose bytes count on a barrier of either CTA of the pair.
__device__ __forceinline__ void vl_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n"
        ::"r"(dst), "l"((uint64_t)map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// Shared-memory descriptors, 128-byte swizzle (layout code 2, version 1).
// K-major: rows of 64 k, 8-row groups 1024 B apart; a k step of 16 is 32 B.
__device__ __forceinline__ uint64_t vl_desc_k(uint32_t a)
{
    return (uint64_t)((a & 0x3FFFF) >> 4) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) |
           ((uint64_t)2 << 61);
}
// MN-major: k rows of 64 elements along M or N; 8-k groups 1024 B apart, the
// next 64 elements along M or N one TMA box (kVlK rows) on; a k step of 16 is
// 2048 B.
__device__ __forceinline__ uint64_t vl_desc_mn(uint32_t a)
{
    return (uint64_t)((a & 0x3FFFF) >> 4) | ((uint64_t)(kVlK * 128 >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void vl_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
                 " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}
// arrive on this barrier of both CTAs once the MMAs issued so far are done
__device__ __forceinline__ void vl_commit(uint64_t *bar)
{
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)3)
                 : "memory");
}
__device__ __forceinline__ void vl_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void vl_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;\n" ::: "memory"); }
__device__ __forceinline__ void vl_cluster_sync()
{
    asm volatile("barrier.cluster.arrive;\nbarrier.cluster.wait;\n" ::: "memory");
}
__device__ __forceinline__ void vl_tmem_ld32(uint32_t taddr, float (&r)[32])
{
    uint32_t u[32];
    __syncwarp();   // (lanes without a row to write skip the previous chunk's stores)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];\n"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7]),
          "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]), "=r"(u[14]), "=r"(u[15]),
          "=r"(u[16]), "=r"(u[17]), "=r"(u[18]), "=r"(u[19]), "=r"(u[20]), "=r"(u[21]), "=r"(u[22]), "=r"(u[23]),
          "=r"(u[24]), "=r"(u[25]), "=r"(u[26]), "=r"(u[27]), "=r"(u[28]), "=r"(u[29]), "=r"(u[30]), "=r"(u[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ float vl_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *(const uint32_t *)&h;
}

// ---------------------------------------------------------------- tiles
struct VlTile {
    int m0, n0, nt, split, c0, dc, nc;   // first row and column, column tile, k chunks c0, c0 + dc, .. (nc of them)
};
__device__ __forceinline__ VlTile vl_tile(const VlJob &jb, int t)
{
    VlTile x;
    int m, n;
    if (jb.n_fast) { n = t % jb.nt; t /= jb.nt; m = t % jb.mt; t /= jb.mt; }
    else { m = t % jb.mt; t /= jb.mt; n = t % jb.nt; t /= jb.nt; }
    x.m0 = m * kVlM;
    x.n0 = n * jb.bn;
    x.nt = n;
    x.split = t;
    // dh walks the ids backwards, all shares together: the rows of W that dz
    // read last are still in L2
    const bool back = jb.kind == VL_DH || jb.kind == VL_DH_T;
    x.c0 = back ? jb.chunks - 1 - t : 0;
    x.dc = back ? -jb.splits : 1;
    x.nc = back ? (jb.chunks - t + jb.splits - 1) / jb.splits : jb.chunks;
    return x;
}

struct VlSmem {
    alignas(8) uint64_t full[kVlStages], empty[kVlStages], tfull[2], tempty[2];
    uint64_t half[2][4];   // LSE: the second warp of a quarter left its part (per accumulator)
    uint32_t tmem_base;
    int abort;
};
// Behind the ring: LSE, the second warps' (maximum, sum) of a tile, per
// accumulator; the transposed kinds, per column (row of h) lse * log2 e,
// upstream gradient, target and its dz; DZ, DZKL and DW, 4 KiB per epilogue warp.
union VlTail {
    float2 half[2][128];
    struct {
        float k[kVlNMax], g[kVlNMax], e[kVlNMax];
        int t[kVlNMax];
    } col;
    unsigned char store[kVlEpi / 32][4096];
};
static_assert(kVlRing + sizeof(((VlTail *)0)->col) <= kVlShared && 3 * 65536 + sizeof(VlTail) <= kVlShared, "shared memory");

// ---------------------------------------------------------------- epilogues
// taddr: the accumulator's first column, this warp's lanes; half: which of the
// two warps of these rows.
// false: the other warp's part did not come (the kernel is giving up)
__device__ __forceinline__ bool vl_epi_lse(const VlJob &jb, const VlTile &x, int row, uint32_t taddr, int half, float2 *other,
                                           uint64_t *bar, uint32_t parity, volatile int *abort)
{
    const int nv = min(jb.bn, jb.N - x.n0);           // ids of this tile below the vocabulary
    const int id = row < jb.M ? jb.targets[row] : -1, t = id < 0 ? -1 : id - x.n0;
    float m = -INFINITY, s = 0.f;
    for (int c = 32 * half; c < nv; c += 64) {
        float r[32];
        vl_tmem_ld32(taddr + c, r);
        if (nv - c < 32)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i >= nv) r[i] = -INFINITY;
        if (t >= c && t < c + 32)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (t == c + i) r[i] = -INFINITY;   // (ce_finalize_kernel adds it)
        float cm = r[0];
#pragma unroll
        for (int i = 1; i < 32; ++i) cm = fmaxf(cm, r[i]);
        const float mn = fmaxf(m, cm), k = (mn == -INFINITY ? 0.f : mn) * kLog2e;   // (a NaN logit makes the sum NaN)
        float a[4] = {s * vl_exp2(fmaf(m, kLog2e, -k)), 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 32; ++i) a[i & 3] += vl_exp2(fmaf(r[i], kLog2e, -k));
        s = (a[0] + a[1]) + (a[2] + a[3]);
        m = mn;
    }
    // (the buffer of this accumulator is free: the MMAs of the tile needed both
    // warps' arrival after its last use)
    if (half) {
        *other = make_float2(m, s);
        __syncwarp();
        if ((threadIdx.x & 31) == 0)
            asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
    } else if (!__all_sync(0xffffffffu, vl_wait(bar, parity, abort))) {
        return false;
    }
    if (row < jb.M && !half) {
        const float2 o = *other;
        const float mn = fmaxf(m, o.x), k = (mn == -INFINITY ? 0.f : mn) * kLog2e;
        s = s * vl_exp2(fmaf(m, kLog2e, -k)) + o.y * vl_exp2(fmaf(o.x, kLog2e, -k));
        jb.rec[(size_t)x.nt * jb.M + row] = make_float2(mn, s);
    }
    return true;
}

// Results in bf16 leave by TMA, a box of 64 columns at a time through the warp's
// 4 KiB of shared memory (rows of 128 bytes, 128-byte swizzle): whole lines
// (16-byte stores of a row per thread took about 310 us for the dW of 31 rows of
// 2048, vocabulary 151936; the boxes take 170 us).  The map clips what lies past
// the last row or column.
//
// the buffer is free again (lane 0 issued the copies; a warp sync follows)
__device__ __forceinline__ void vl_box_free() { asm volatile("cp.async.bulk.wait_group.read 0;\n" ::: "memory"); }
// eight columns of a row: 16-byte piece `piece` of its 128 bytes
__device__ __forceinline__ void vl_box_put(uint32_t buf, int row, int piece, const float *v)
{
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(buf + row * 128 + ((piece ^ (row & 7)) << 4)),
                 "r"(pack_bf16(v[0], v[1])), "r"(pack_bf16(v[2], v[3])), "r"(pack_bf16(v[4], v[5])), "r"(pack_bf16(v[6], v[7]))
                 : "memory");
}
__device__ __forceinline__ void vl_box_send(const CUtensorMap *map, int x, int y, uint32_t buf, int lane)
{
    asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
    __syncwarp();
    if (lane == 0)
        asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n"
                     "cp.async.bulk.commit_group;\n" ::"l"((uint64_t)map), "r"(x), "r"(y), "r"(buf)
                     : "memory");
}

__device__ __forceinline__ void vl_epi_dz(const VlJob &jb, const VlTile &x, int row, uint32_t taddr, int half, int lane,
                                          uint32_t buf, unsigned *err)
{
    float g = 0.f, k = 0.f, et = 0.f;
    int t = -1;
    if (row < jb.M) {
        et = jb.et[row];
        const int id = jb.targets[row];
        if (id >= jb.V && x.n0 == 0 && jb.v0 == 0 && half == 0 && err) raise_err(err, ORTHRUS_DEVERR_TOKEN);
        if (id >= 0 && id < jb.V) { g = jb.g[row]; t = id - jb.v0 - x.n0; }
        k = jb.lse[row] * kLog2e;
    }
    const int nv = jb.N - x.n0;                        // columns of the tile below the piece's end (may exceed bn)
    const int nc = min(jb.bn, jb.pitch - x.n0);        // columns dz has room for
    for (int c = 64 * half; c < nc; c += 128) {
        vl_box_free();
#pragma unroll
        for (int q = 0; q < 64; q += 32) {
            float r[32];
            vl_tmem_ld32(taddr + c + q, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const float e = c + q + i == t ? et : vl_exp2(fmaf(r[i], kLog2e, -k));
                // rows without a share and columns past the vocabulary are exact zeros
                r[i] = g == 0.f || c + q + i >= nv ? 0.f : g * e;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) vl_box_put(buf, lane, q / 8 + i, r + 8 * i);
        }
        vl_box_send(&jb.c, x.n0 + c, row - lane, buf, lane);
    }
}

// Interleaved rows: even lanes hold the AR view's logits of a position, odd
// lanes the diffusion view's.  Each pair of lanes exchanges halves of a chunk
// and puts 16 columns per lane.
__device__ __forceinline__ void vl_epi_dzkl(const VlJob &jb, const VlTile &x, int row, uint32_t taddr, int half, int lane,
                                            uint32_t buf)
{
    const int pos = row >> 1, odd = row & 1;
    const bool live = row < jb.M;
    const float k = live ? (odd ? jb.lse2 : jb.lse)[pos] * kLog2e : 0.f, g = live ? jb.g[pos] : 0.f;
    const int nv = jb.N - x.n0;
    const int nc = min(jb.bn, jb.pitch - x.n0);
    for (int c = 64 * half; c < nc; c += 128) {
        vl_box_free();
#pragma unroll
        for (int q = 0; q < 64; q += 32) {
            float r[32], v[16];
            vl_tmem_ld32(taddr + c + q, r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = vl_exp2(fmaf(r[i], kLog2e, -k));
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const float mine = odd ? r[16 + i] : r[i];
                const float other = __shfl_xor_sync(0xffffffffu, odd ? r[i] : r[16 + i], 1);
                const float e = odd ? mine - other : other - mine;   // p_diff - p_AR
                v[i] = g == 0.f || c + q + 16 * odd + i >= nv ? 0.f : g * e;
            }
            vl_box_put(buf, lane >> 1, q / 8 + 2 * odd, v);
            vl_box_put(buf, lane >> 1, q / 8 + 2 * odd + 1, v + 8);
        }
        vl_box_send(&jb.c, x.n0 + c, (row - lane) >> 1, buf, lane);
    }
}

// dh: this piece's share, added to what earlier pieces left
__device__ __forceinline__ void vl_epi_dh(const VlJob &jb, const VlTile &x, int row, uint32_t taddr, int half)
{
    const int nv = min(jb.bn, jb.N - x.n0);            // (a multiple of 8)
    const bool out = jb.last;
    float *p = jb.part + ((size_t)x.split * jb.M + row) * jb.N + x.n0;
    bf16 *o = jb.out + (size_t)row * jb.N + x.n0;
    for (int c = 32 * half; c < nv; c += 64) {
        float r[32];
        vl_tmem_ld32(taddr + c, r);
        if (row >= jb.M) continue;
#pragma unroll
        for (int q = 0; q < 32; q += 8) {
            if (c + q >= nv) break;
            float4 *f = (float4 *)(p + c + q);
            float4 a = make_float4(r[q], r[q + 1], r[q + 2], r[q + 3]), b = make_float4(r[q + 4], r[q + 5], r[q + 6], r[q + 7]);
            if (jb.add) {
                const float4 u = f[0], w = f[1];
                a.x += u.x; a.y += u.y; a.z += u.z; a.w += u.w;
                b.x += w.x; b.y += w.y; b.z += w.z; b.w += w.w;
            }
            if (out)
                *(uint4 *)(o + c + q) = make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
            else { f[0] = a; f[1] = b; }
        }
    }
}

__device__ __forceinline__ void vl_epi_dw(const VlJob &jb, const VlTile &x, int row, uint32_t taddr, int half, int lane,
                                          uint32_t buf)
{
    const int nv = min(jb.bn, jb.N - x.n0);
    for (int c = 64 * half; c < nv; c += 128) {
        vl_box_free();
#pragma unroll
        for (int q = 0; q < 64; q += 32) {
            float r[32];
            vl_tmem_ld32(taddr + c + q, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) vl_box_put(buf, lane, q / 8 + i, r + 8 * i);
        }
        vl_box_send(&jb.c, x.n0 + c, jb.c_off + row - lane, buf, lane);
    }
}

// ---- transposed: a thread holds one id (or one hidden column), 32 rows at a time
// the columns' constants, one column per thread
__device__ __forceinline__ void vl_columns(const VlJob &jb, VlTail &tail, unsigned *err)
{
    const int c = threadIdx.x;
    if (c >= kVlNMax) return;
    float k = 0.f, g = 0.f, e = 0.f;
    int t = -1;
    if (c < jb.N) {
        if (jb.kind == VL_DZKL_T) {
            k = (c & 1 ? jb.lse2 : jb.lse)[c >> 1] * kLog2e;
            g = jb.g[c >> 1];
        } else {
            k = jb.lse[c] * kLog2e;
            t = jb.targets[c];
            e = jb.et[c];
            if (t >= 0 && t < jb.V) g = jb.g[c];
            if (t >= jb.V && blockIdx.x == 0 && err) raise_err(err, ORTHRUS_DEVERR_TOKEN);
        }
    }
    tail.col.k[c] = k;
    tail.col.g[c] = g;
    tail.col.e[c] = e;
    tail.col.t[c] = t;
}
static_assert(kVlThreads >= kVlNMax, "one column per thread");

__device__ __forceinline__ float warp_max_f32(float v)
{
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;\n" : "=f"(m) : "f"(v));
    return m;
}

// v: this thread's id (the tile's ids are in order, so a warp holds one group
// of 32); a record per (group, row).
__device__ __forceinline__ void vl_epi_lse_t(const VlJob &jb, int v, uint32_t taddr, int half, int lane)
{
    for (int c = 32 * half; c < jb.N; c += 64) {
        float r[32], m = -INFINITY;
        vl_tmem_ld32(taddr + c, r);
        const int tgt = c + lane < jb.N ? jb.targets[c + lane] : -1;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            const int t = __shfl_sync(0xffffffffu, tgt, j);
            if (v >= jb.M || t == v) r[j] = -INFINITY;   // (the target: ce_finalize_kernel adds it)
            const float mj = warp_max_f32(r[j]), k = (mj == -INFINITY ? 0.f : mj) * kLog2e;
            r[j] = vl_exp2(fmaf(r[j], kLog2e, -k));
            if (lane == j) m = mj;
        }
        // lane j ends with the sum of column j
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < o; ++i) {
                const float keep = lane & o ? r[i + o] : r[i], send = lane & o ? r[i] : r[i + o];
                r[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
            }
        if (c + lane < jb.N) jb.rec[(size_t)(v / 32) * jb.N + c + lane] = make_float2(m, r[0]);
    }
}

// i: this thread's id within the piece; jb.M ids of the piece are real, the
// rest of dz's row length gets zeros
__device__ __forceinline__ void vl_epi_dz_t(const VlJob &jb, const VlTail &tail, int i, uint32_t taddr, int half)
{
    const int v = jb.v0 + i;
    const bool live = i < jb.M;
    for (int c = 32 * half; c < jb.N; c += 64) {
        float r[32];
        vl_tmem_ld32(taddr + c, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (c + j >= jb.N) break;
            const float g = tail.col.g[c + j];
            const float e = tail.col.t[c + j] == v ? tail.col.e[c + j] : vl_exp2(fmaf(r[j], kLog2e, -tail.col.k[c + j]));
            jb.dz[(size_t)(c + j) * jb.pitch + i] = __float2bfloat16_rn(g == 0.f || !live ? 0.f : g * e);
        }
    }
}

__device__ __forceinline__ void vl_epi_dzkl_t(const VlJob &jb, const VlTail &tail, int i, uint32_t taddr, int half)
{
    const bool live = i < jb.M;
    for (int c = 32 * half; c < jb.N; c += 64) {
        float r[32];
        vl_tmem_ld32(taddr + c, r);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
            if (c + j >= jb.N) break;
            const float g = tail.col.g[c + j];
            const float pa = vl_exp2(fmaf(r[j], kLog2e, -tail.col.k[c + j]));
            const float pd = vl_exp2(fmaf(r[j + 1], kLog2e, -tail.col.k[c + j + 1]));
            jb.dz[(size_t)((c + j) >> 1) * jb.pitch + i] = __float2bfloat16_rn(g == 0.f || !live ? 0.f : g * (pd - pa));
        }
    }
}

__device__ __forceinline__ void vl_epi_dh_t(const VlJob &jb, const VlTile &x, int i, uint32_t taddr, int half)
{
    for (int c = 32 * half; c < jb.N; c += 64) {
        float r[32];
        vl_tmem_ld32(taddr + c, r);
        if (i >= jb.M) continue;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
            if (c + j >= jb.N) break;
            float *p = jb.part + ((size_t)x.split * jb.N + c + j) * jb.M + i;
            const float s = jb.add ? *p + r[j] : r[j];
            if (jb.last) jb.out[(size_t)(c + j) * jb.M + i] = __float2bfloat16_rn(s);
            else *p = s;
        }
    }
}

// ---------------------------------------------------------------- kernel
__global__ void __launch_bounds__(kVlThreads, 1) vocab_pair_kernel(const __grid_constant__ VlParams prm)
{
    extern __shared__ __align__(1024) unsigned char vl_smem_raw[];
    __shared__ VlSmem sm;
    const uint32_t ring = (smem_u32(vl_smem_raw) + 1023) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = blockIdx.x & 1;               // CTA of the pair
    const int pair = blockIdx.x >> 1;
    volatile int *abort = &sm.abort;
    VlTail &tail = *(VlTail *)(vl_smem_raw + (ring - smem_u32(vl_smem_raw)) + prm.stages * prm.stage_bytes);

    if (threadIdx.x == 0) {
        for (int s = 0; s < kVlStages; ++s) { vl_mbar_init(&sm.full[s], 1); vl_mbar_init(&sm.empty[s], 1); }
        for (int s = 0; s < 2; ++s) { vl_mbar_init(&sm.tfull[s], 1); vl_mbar_init(&sm.tempty[s], 2 * kVlEpi / 32); }
        for (int s = 0; s < 8; ++s) vl_mbar_init(&sm.half[s >> 2][s & 3], 1);
        sm.abort = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    }
    vl_fence_before();
    __syncthreads();
    vl_cluster_sync();                                  // both CTAs' barriers and TMEM are ready
    vl_fence_after();
    const uint32_t tmem = sm.tmem_base;
    pdl_wait();
    const VlJob &jb = prm.job;
    const int tiles = jb.mt * jb.nt * jb.splits;
    if (jb.kind == VL_DZ_T || jb.kind == VL_DZKL_T) {
        vl_columns(jb, tail, prm.err);
        __syncthreads();
    }

    if (warp == 0) {
        if (lane == 0) {   // ------------------------------------------- producer
            uint32_t stage = 0, phase = 0;
            bool stop = false;
            for (int t = pair; t < tiles && !stop; t += prm.pairs) {
                const VlTile x = vl_tile(jb, t);
                const int am = x.m0 + (int)rank * 128, bnh = jb.bn / 2, bx = x.n0 + (int)rank * bnh;
                const uint32_t bytes = 2 * (128 + (uint32_t)bnh) * jb.kr * 2;
                for (int i = 0; i < x.nc; ++i) {
                    if (!vl_wait(&sm.empty[stage], phase ^ 1, abort) || *abort) { stop = true; break; }
                    if (rank == 0) vl_expect_tx(&sm.full[stage], bytes);
                    const uint32_t bar = vl_mapa(smem_u32(&sm.full[stage]), 0);
                    const uint32_t a = ring + stage * prm.stage_bytes, b = a + kVlABytes;
                    const int k = (x.c0 + i * x.dc) * kVlK;
                    // two boxes of 64 elements each: along k (K-major), or along M / N
                    if (jb.a_mn) {
                        vl_load(a, &jb.a, am, jb.a_off + k, bar);
                        vl_load(a + kVlABytes / 2, &jb.a, am + 64, jb.a_off + k, bar);
                    } else {
                        vl_load(a, &jb.a, k, jb.a_off + am, bar);
                        vl_load(a + kVlABytes / 2, &jb.a, k + 64, jb.a_off + am, bar);
                    }
                    if (jb.b_mn) {
                        for (int q = 0; q < bnh; q += 64) vl_load(b + q * kVlK * 2, &jb.b, bx + q, jb.b_off + k, bar);
                    } else {
                        vl_load(b, &jb.b, k, jb.b_off + bx, bar);
                        vl_load(b + bnh * 128, &jb.b, k + 64, jb.b_off + bx, bar);
                    }
                    if (++stage == (uint32_t)prm.stages) { stage = 0; phase ^= 1; }
                }
            }
            pdl_trigger();
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {   // ------------------------------ MMA issuer
            uint32_t stage = 0, phase = 0;
            int local = 0;
            for (int t = pair; t < tiles && !*abort; t += prm.pairs, ++local) {
                const VlTile x = vl_tile(jb, t);
                const int acc = local & 1;
                const bool a_mn = jb.a_mn, b_mn = jb.b_mn;
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) |
                                       ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(jb.bn >> 3) << 17) |
                                       ((uint32_t)(kVlM >> 4) << 24);
                // descriptor steps: 16 k inside a 64-k half of the stage, and the other half
                const uint64_t as = a_mn ? 2048 >> 4 : 32 >> 4, bs = b_mn ? 2048 >> 4 : 32 >> 4;
                const uint64_t ah = a_mn ? 4 * as : kVlABytes / 2 >> 4, bh = b_mn ? 4 * bs : (uint64_t)(jb.bn / 2 * 128 >> 4);
                if (!vl_wait(&sm.tempty[acc], ((local >> 1) & 1) ^ 1, abort)) break;
                vl_fence_after();
                const uint32_t d = tmem + acc * kVlNMax;
                bool ok = true;
                for (int i = 0; i < x.nc; ++i) {
                    if (!vl_wait(&sm.full[stage], phase, abort)) { ok = false; break; }
                    vl_fence_after();
                    const uint32_t a = ring + stage * prm.stage_bytes, b = a + kVlABytes;
                    const uint64_t ad = a_mn ? vl_desc_mn(a) : vl_desc_k(a), bd = b_mn ? vl_desc_mn(b) : vl_desc_k(b);
#pragma unroll
                    for (int k = 0; k < kVlK / 16; ++k)
                        if (k * 16 < jb.kr) vl_mma(d, ad + as * (k & 3) + ah * (k >> 2), bd + bs * (k & 3) + bh * (k >> 2), idesc,
                               (i > 0 || k > 0) ? 1u : 0u);
                    vl_commit(&sm.empty[stage]);
                    if (++stage == (uint32_t)prm.stages) { stage = 0; phase ^= 1; }
                }
                if (!ok) break;
                vl_commit(&sm.tfull[acc]);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {   // ---------------------------------------- epilogue
        const int q = warp & 3;                          // TMEM lane quarter of this warp
        const int r = (int)rank * 128 + q * 32 + lane;   // row in the tile
        const uint32_t free0 = vl_mapa(smem_u32(&sm.tempty[0]), 0), free1 = vl_mapa(smem_u32(&sm.tempty[1]), 0);
        const int half = (warp - 4) >> 2;
        const uint32_t buf = smem_u32(tail.store[warp - 4]);
        int local = 0;
        uint32_t halves = 0;   // phases of sm.half: they count the tiles that this quarter has rows in
        for (int t = pair; t < tiles; t += prm.pairs, ++local) {
            const VlTile x = vl_tile(jb, t);
            const int acc = local & 1, row = x.m0 + r;
            bool ok = vl_wait(&sm.tfull[acc], (local >> 1) & 1, abort);
            if (!__all_sync(0xffffffffu, ok)) break;
            vl_fence_after();
            const uint32_t taddr = tmem + ((uint32_t)(q * 32) << 16) + acc * kVlNMax;
            // (whole warps past the last row have nothing to do, but dz's padding is written)
            const int rows = jb.kind == VL_DZ_T || jb.kind == VL_DZKL_T ? jb.pitch : jb.M;
            if (x.m0 + (int)rank * 128 + q * 32 < rows) {
                switch (jb.kind) {
                case VL_LSE:
                    ok = vl_epi_lse(jb, x, row, taddr, half, &tail.half[acc][q * 32 + lane], &sm.half[acc][q], halves >> acc & 1, abort);
                    halves ^= 1u << acc;
                    break;
                case VL_DZ: vl_epi_dz(jb, x, row, taddr, half, lane, buf, prm.err); break;
                case VL_DZKL: vl_epi_dzkl(jb, x, row, taddr, half, lane, buf); break;
                case VL_DH: vl_epi_dh(jb, x, row, taddr, half); break;
                case VL_DW: vl_epi_dw(jb, x, row, taddr, half, lane, buf); break;
                case VL_LSE_T: vl_epi_lse_t(jb, row, taddr, half, lane); break;
                case VL_DZ_T: vl_epi_dz_t(jb, tail, row, taddr, half); break;
                case VL_DZKL_T: vl_epi_dzkl_t(jb, tail, row, taddr, half); break;
                default: vl_epi_dh_t(jb, x, row, taddr, half); break;
                }
            }
            if (!ok) break;
            vl_fence_before();
            __syncwarp();
            if (lane == 0) vl_arrive_at(acc ? free1 : free0);
        }
        asm volatile("cp.async.bulk.wait_group 0;\n" ::: "memory");
    }

    vl_fence_before();
    __syncthreads();
    if (*abort) {   // let this CTA's copies and MMAs in flight land before the memory goes away
        const long long t0 = clock64();
        while (clock64() - t0 < 20000000LL) {}
        if (threadIdx.x == 0 && prm.err) raise_err(prm.err, ORTHRUS_DEVERR_TIMEOUT);
    }
    vl_cluster_sync();                                  // the peer may still signal this CTA's barriers
    if (warp == 2) {
        vl_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(512u));
    }
}

// rows 2i and 2i + 1 of out: row i of the AR and of the diffusion view; with a
// zero upstream gradient both are zero (so their values cannot matter)
__global__ void __launch_bounds__(256) vl_interleave_kernel(const uint4 *ra, const uint4 *rb, const float *g, uint4 *out,
                                                            int vecs)
{
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.x;
    const bool live = g[r] != 0.f;
    const uint4 z = make_uint4(0, 0, 0, 0);
    for (int i = threadIdx.x; i < vecs; i += 256) {
        out[(size_t)(2 * r) * vecs + i] = live ? ra[(size_t)r * vecs + i] : z;
        out[(size_t)(2 * r + 1) * vecs + i] = live ? rb[(size_t)r * vecs + i] : z;
    }
}

// Per row of the cross entropy, what its target's dz is made of: exp(z_t - lse)
// - 1, with z_t taken again as a dot product in fp32 parts and a double sum.  The
// tensor cores' accumulator truncates, by up to about 1e-5 of a logit: to every
// other id that is 1e-4 of its probability, but of a likely target's 1 - p it
// was most (measured at 600 rows of 4096 over 20000 ids, error of a row's dh:
// 7 % at p = 0.999 and 84 % at p = 0.9999; 0.25 % and 0.5 % so, the latter the
// rounding of a log-sum-exp near 16 to fp32).
// For dW = dz^T h (out), also the hidden rows with the rows that take no part
// zeroed: a padding row's dz is zero, but zero times a NaN or an infinity in
// its hidden row would not be.
__global__ void __launch_bounds__(256) vl_target_kernel(const uint4 *h, const uint4 *w, const int32_t *targets,
                                                        const float *lse, const float *g, int V, float *et, uint4 *out,
                                                        int vecs)
{
    __shared__ double part[8];
    pdl_trigger();
    pdl_wait();
    const int r = blockIdx.x, t = targets[r];
    const bool live = t >= 0 && t < V && g[r] != 0.f;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = threadIdx.x; i < vecs; i += 256) {
        const uint4 u = live ? h[(size_t)r * vecs + i] : make_uint4(0, 0, 0, 0);
        if (live) dot8(u, w[(size_t)t * vecs + i], acc);
        if (out) out[(size_t)r * vecs + i] = u;
    }
    const double z = warp_sum_f64((double)(acc[0] + acc[1]) + (double)(acc[2] + acc[3]));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = z;
    __syncthreads();
    if (threadIdx.x) return;
    double s = part[0];
#pragma unroll
    for (int k = 1; k < 8; ++k) s += part[k];
    et[r] = live ? expm1f((float)(s - (double)lse[r])) : 0.f;
}

// ---------------------------------------------------------------- host
static size_t up(size_t x, size_t m) { return (x + m - 1) / m * m; }

// Up to kVlNMax rows ride as columns beside W's rows: a stage is then mostly
// weights (measured at one row of 2048, vocabulary 151936: the 256-row tile of
// h kept 48 KB of W in flight per SM and ran at 285 us, this one at 113; at 256
// rows of 4096 this one takes 398 us, the 256-row tile at 257 rows 548).
static bool vl_narrow(int rows) { return rows <= kVlNMax; }
static int vl_narrow_bn(int rows) { return (rows + 31) / 32 * 32; }

// Shares of dh's k axis: the smallest count that keeps the rounds of the
// pairs nearly full, each share at least 4 chunks.
static int vl_splits(long tiles, long chunks)
{
    int best = 1;
    double cost = 1e30;
    for (int s = 1; s <= 32 && (s == 1 || chunks / s >= 4); ++s) {
        const double t = (double)((tiles * s + kVlPairs - 1) / kVlPairs) / s * (1.0 + 0.02 * s);
        if (t < cost) { cost = t; best = s; }
    }
    return best;
}

bool loss_tc_ok(const LossArgs &a)
{
    auto al = [](const void *p) { return ((uintptr_t)p & 15) == 0; };
    return a.dtype == ORTHRUS_BF16 && a.d % 8 == 0 && al(a.h) && al(a.h2) && al(a.w) && al(a.dh) && al(a.dw);
}

static cudaError_t vl_launch(VlParams &p, cudaStream_t s)
{
    const VlJob &j = p.job;
    p.pairs = (int)std::min<long>(kVlPairs, (long)j.mt * j.nt * j.splits);
    p.stage_bytes = kVlABytes + (uint32_t)j.bn / 2 * kVlK * 2;
    p.stages = (int)std::min<uint32_t>(kVlStages, kVlRing / p.stage_bytes);
    const size_t smem = 1024 + kVlShared;
    cudaError_t e = cudaFuncSetAttribute(vocab_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * p.pairs);
    cfg.blockDim = dim3(kVlThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, vocab_pair_kernel, p);
}

size_t loss_fwd_workspace_tc(int N, int d, int V)
{
    WsPlan w;
    w.take((size_t)(vl_narrow(N) ? (V + 31) / 32 : (V + kVlNMax - 1) / kVlNMax) * N * sizeof(float2));
    return w.total;
}

cudaError_t loss_fwd_tc(const LossArgs &a, cudaStream_t s)
{
    float2 *rec = (float2 *)a.ws;
    VlParams p;
    memset(&p, 0, sizeof(p));
    VlJob &j = p.job;
    j.kr = kVlK;
    const bool narrow = vl_narrow(a.N);
    const int rows = narrow ? a.V : a.N, cols = narrow ? a.N : a.V;
    j.kind = narrow ? VL_LSE_T : VL_LSE; j.M = rows; j.N = cols; j.chunks = (a.d + kVlK - 1) / kVlK; j.splits = 1;
    j.bn = narrow ? vl_narrow_bn(a.N) : kVlNMax;
    j.mt = (rows + kVlM - 1) / kVlM; j.nt = (cols + j.bn - 1) / j.bn;
    j.targets = a.targets; j.rec = rec;
    if (!make_tmap_box(&j.a, narrow ? a.w : a.h, rows, a.d, 64, 128) ||
        !make_tmap_box(&j.b, narrow ? a.h : a.w, cols, a.d, 64, j.bn / 2))
        return cudaErrorInvalidValue;
    p.err = a.err;
    cudaError_t e = vl_launch(p, s);
    if (e != cudaSuccess) return e;
    return launch_ce_finalize(rec, nullptr, a, narrow ? (a.V + 31) / 32 : j.nt, 1, s);
}

struct VlPlan {
    size_t total, o_dz, o_part, o_h, o_et;
    int piece, splits, zrows;
    bool z_narrow, h_narrow;
};
static VlPlan vl_plan(int N, int d, int V, int want_dw, int kl)
{
    VlPlan p{};
    WsPlan w;
    // a piece's dz stays within 256 MiB (past 524288 rows, 512 bytes per row: a
    // piece has 256 ids at least), whatever the vocabulary, and is large enough
    // that a piece's products fill many rounds of the pairs and dh is added up few
    // times (both gradients, 4096 x 4096 x 151936: 13.3 ms at 64 MiB, 12.8 at 128,
    // 12.4 at 256, 12.3 at 512)
    const size_t cap = std::max<size_t>(256, ((size_t)256 << 20) / (2 * (size_t)N) / 256 * 256);
    p.piece = (int)std::min(cap, up(V, 256));
    p.zrows = kl ? 2 * N : N;
    p.z_narrow = vl_narrow(p.zrows);
    p.h_narrow = vl_narrow(N);
    const long tiles = p.h_narrow ? (d + kVlM - 1) / kVlM : (long)up(N, kVlM) / kVlM * ((d + 255) / 256);
    p.splits = vl_splits(tiles, (std::min(p.piece, V) + kVlK - 1) / kVlK);
    p.o_dz = w.take((size_t)N * p.piece * 2);
    p.o_part = w.take((size_t)p.splits * N * d * 4);
    p.o_h = w.take(kl ? (size_t)2 * N * d * 2 : want_dw ? (size_t)N * d * 2 : 0);
    p.o_et = w.take(kl ? 0 : (size_t)N * 4);
    p.total = w.total;
    return p;
}

size_t loss_grad_workspace_tc(int N, int d, int V, int want_dw, int kl) { return vl_plan(N, d, V, want_dw, kl).total; }

cudaError_t loss_grad_tc(const LossArgs &a, cudaStream_t s)
{
    const int N = a.N, d = a.d;
    const VlPlan pl = vl_plan(N, d, a.V, a.dw != nullptr, a.kl);
    bf16 *dz = (bf16 *)(a.ws + pl.o_dz), *hx = (bf16 *)(a.ws + pl.o_h);
    float *part = (float *)(a.ws + pl.o_part), *et = (float *)(a.ws + pl.o_et);
    cudaError_t e;
    if (a.kl)
        e = launch_k(vl_interleave_kernel, N, 256, 0, s, (const uint4 *)a.h, (const uint4 *)a.h2, a.g, (uint4 *)hx, d / 8);
    else
        e = launch_k(vl_target_kernel, N, 256, 0, s, (const uint4 *)a.h, (const uint4 *)a.w, a.targets, a.lse_in, a.g, a.V,
                     et, a.dw ? (uint4 *)hx : (uint4 *)nullptr, d / 8);
    if (e != cudaSuccess) return e;
    const int zbn = pl.z_narrow ? vl_narrow_bn(pl.zrows) : kVlNMax, hbn = pl.h_narrow ? vl_narrow_bn(N) : kVlNMax;
    const int wk = (int)std::min<size_t>(kVlK, up(N, 16));   // k of dW's chunks
    // zh: hidden rows, zw: head rows (both along k); dzs: dz as it is written, dzk: dz along its ids; wm:
    // head columns; dzm, hm: dz's and h's columns (dW); dwm: dW itself
    CUtensorMap zh, zw, dzs, dzk, dzm, wm, hm, dwm;
    const bool ok = make_tmap_box(&zh, a.kl ? (const void *)hx : a.h, pl.zrows, d, 64, pl.z_narrow ? zbn / 2 : 128) &&
                    make_tmap_box(&zw, a.w, a.V, d, 64, 128) &&
                    make_tmap_box(&dzs, dz, N, pl.piece, 64, a.kl ? 16 : 32) &&
                    make_tmap_box(&dzk, dz, N, pl.piece, 64, pl.h_narrow ? hbn / 2 : 128) &&
                    make_tmap_box(&wm, a.w, a.V, d, 64, kVlK) &&
                    (!a.dw || (make_tmap_box(&dzm, dz, N, pl.piece, 64, wk) && make_tmap_box(&hm, hx, N, d, 64, wk) &&
                                make_tmap_box(&dwm, a.dw, a.V, d, 64, 32)));
    if (!ok) return cudaErrorInvalidValue;
    VlParams p;
    for (int v0 = 0; v0 < a.V; v0 += pl.piece) {
        const int nv = std::min(pl.piece, a.V - v0);
        {
            memset(&p, 0, sizeof(p));
            VlJob &j = p.job;
            j.kr = kVlK;
            j.kind = a.kl ? (pl.z_narrow ? VL_DZKL_T : VL_DZKL) : (pl.z_narrow ? VL_DZ_T : VL_DZ);
            j.M = pl.z_narrow ? nv : pl.zrows; j.N = pl.z_narrow ? pl.zrows : nv;
            j.chunks = (d + kVlK - 1) / kVlK; j.splits = 1; j.bn = zbn;
            j.mt = (j.M + kVlM - 1) / kVlM; j.nt = (j.N + zbn - 1) / zbn;
            (pl.z_narrow ? j.a_off : j.b_off) = v0;
            j.targets = a.targets; j.lse = a.lse_in; j.lse2 = a.lse2_in; j.g = a.g; j.et = et;
            j.dz = dz; j.v0 = v0; j.V = a.V; j.pitch = pl.piece;
            j.a = pl.z_narrow ? zw : zh; j.b = pl.z_narrow ? zh : zw; j.c = dzs;
            p.err = a.err;
            if ((e = vl_launch(p, s)) != cudaSuccess) return e;
        }
        {
            memset(&p, 0, sizeof(p));
            VlJob &j = p.job;
            j.kr = kVlK;
            j.kind = pl.h_narrow ? VL_DH_T : VL_DH;
            j.M = pl.h_narrow ? d : N; j.N = pl.h_narrow ? N : d; j.chunks = (nv + kVlK - 1) / kVlK;
            j.splits = std::min(pl.splits, j.chunks);
            j.bn = hbn; j.mt = (j.M + kVlM - 1) / kVlM; j.nt = (j.N + hbn - 1) / hbn;
            (pl.h_narrow ? j.a_mn : j.b_mn) = 1;
            (pl.h_narrow ? j.a_off : j.b_off) = v0;
            j.part = part; j.add = v0 > 0; j.last = pl.splits == 1 && v0 + pl.piece >= a.V; j.out = (bf16 *)a.dh;
            j.a = pl.h_narrow ? wm : dzk; j.b = pl.h_narrow ? dzk : wm;
            p.err = a.err;
            if ((e = vl_launch(p, s)) != cudaSuccess) return e;
        }
        if (a.dw) {
            memset(&p, 0, sizeof(p));
            VlJob &j = p.job;
            j.kr = kVlK;
            j.kind = VL_DW; j.M = nv; j.N = d; j.chunks = (N + kVlK - 1) / kVlK; j.splits = 1;
            j.bn = 256; j.mt = (nv + kVlM - 1) / kVlM; j.nt = (d + 255) / 256; j.n_fast = 1; j.kr = wk;
            j.a_mn = j.b_mn = 1;
            j.c_off = v0;
            j.a = dzm; j.b = hm; j.c = dwm;
            p.err = a.err;
            if ((e = vl_launch(p, s)) != cudaSuccess) return e;
        }
    }
    if (pl.splits > 1) return launch_part_sum(part, pl.splits, (size_t)N * d, a.dh, ORTHRUS_BF16, s);
    return cudaSuccess;
}

}  // namespace orthrus
