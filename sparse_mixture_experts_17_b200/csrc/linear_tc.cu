// linear_tc.cu -- the products of the linear layers on the 5th-generation
// tensor cores (tcgen05, operands by TMA, accumulators in TMEM):
//   out[c, m] = sum_k A[m, k] B[c, k],   m contiguous in the output.
//
// Orientation. The weight side (or, for dW, the input features) is the M side
// of the MMA and the tokens (for dW the output features) its N side, because N
// is free in steps of 16: a group's rows are cut into near-equal tiles of at
// most 256 and each tile runs MMAs just wide enough, so a ragged group pays for
// at most 31 rows that it does not have, and a single token takes MMAs of the
// smallest N while its weights pass once.
//
// Operands. Every box that the TMA brings is 64 elements (128 bytes) wide,
// 128-byte swizzled. Where the contraction runs along the contiguous axis the
// tile is K-major; where it runs across rows (W for dx; x and dz for dW) the
// same boxes are an MN-major operand, so no operand is transposed in memory.
// W is a three-dimensional map (d_in, d_out, expert): what lies past an edge of
// one expert's matrix reads as zero and never as the next expert's values. For
// dW the contraction runs over a group's rows: the rows of the last block that
// belong to the next group (or to nobody) are zeroed in shared memory, in both
// operands, since they may hold infinities.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "act.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "linear.h"

namespace moe {

namespace {

constexpr int kBox = 64;                    // box width in elements, and the K stage
constexpr int kBoxBytes = kBox * kBox * 2;  // 64 rows of 128 bytes
constexpr int kTileC = 256;                 // widest N

// ---------------------------------------------------------------- PTX

__device__ __forceinline__ void tma_3d(void *dst, const void *tmap, int c0, int c1, int c2,
                                       uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_4d(void *dst, const void *tmap, int c0, int c1, int c2, int c3,
                                       uint64_t *bar)
{
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
                 "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void tma_3d_pair(uint32_t dst, const void *tmap, int c0, int c1, int c2,
                                            uint32_t bar_cluster)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void tma_4d_pair(uint32_t dst, const void *tmap, int c0, int c1, int c2,
                                            int c3, uint32_t bar_cluster)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar_cluster)
        : "memory");
}

__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const void *tmap, int c0, int c1,
                                            uint32_t bar_cluster)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(tmap), "r"(c0), "r"(c1), "r"(bar_cluster)
        : "memory");
}

// Make generic-proxy writes to shared memory visible to the MMAs.
__device__ __forceinline__ void fence_proxy_async()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// Arrive on a barrier of another CTA of the cluster without ordering memory at cluster
// scope: a release there would wait until the warp's stores to global memory are done.
// For hand-overs of tensor memory, which carry no data through memory.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t cluster_addr)
{
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// MN-major operand in 128-byte-swizzled boxes of 64 (MN) x 64 (K): 8 K rows of
// 128 bytes per 1024-byte atom (stride offset 1024 between atoms along K), the
// next 64 MN elements one box further (leading offset 8192).
__device__ __forceinline__ uint64_t smem_desc_mn128(uint32_t smem_addr)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)(kBoxBytes >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

// Operand descriptor of K step kk (16 elements) of a stage.
template <bool MN>
__device__ __forceinline__ uint64_t op_desc(uint32_t base, int kk)
{
    return MN ? smem_desc_mn128(base + kk * 2048) : smem_desc_k128(base + kk * 32);
}

// What a K step of 16 adds to it (its address field counts 16 bytes).
template <bool MN>
__device__ __forceinline__ constexpr uint64_t op_step()
{
    return MN ? 2048 / 16 : 32 / 16;
}

template <LinMode MODE>
__device__ __forceinline__ uint32_t lin_idesc(int M, int N)
{
    return idesc_bf16_f32(M, N) | (MODE != LIN_FWD ? 1u << 15 : 0u)   // A is MN-major
           | (MODE == LIN_DW ? 1u << 16 : 0u);                        // B is MN-major
}

// 16 TMEM lanes (m) x 16 columns (c): in v[4 i + j], j = 0, 1: lane t / 4, column
// 8 i + 2 (t % 4) + j; j = 2, 3: the same columns of lane t / 4 + 8 (t: this thread).
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[8])
{
    uint32_t r[8];
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = __uint_as_float(r[i]);
}

// Four 8 x 8 matrices of bf16 between registers (row t / 4, columns 2 (t % 4) and
// + 1) and shared memory, transposed; lane l gives row l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, const uint32_t (&r)[4])
{
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// ---------------------------------------------------------------- epilogue

struct LinOut {
    const float *bias;
    const uint16_t *residual;
    uint16_t *out, *z;
    float *part;        // LIN_DW in splits: fp32 sums instead of out
    long long ld;       // elements between consecutive c
};

// A warp turns 32 m (its TMEM lanes) x 16 c of an accumulator into rows of out.
// The accumulator has c along its columns and memory has m contiguous: pairs of
// c are packed to bf16 in registers, stmatrix transposes them into 1 KB of the
// warp's own shared memory, and each lane moves two 16-byte pieces (8 m of one
// c) to memory; 1 store for 8 elements, where storing the columns one by one
// took 22 instructions an element and held the gradient of 128 experts'
// weights at 1.3 TB/s. The residual comes in the same way backwards, read by
// the lane that will write it. Piece v of row c lies at v ^ (c / 2 % 4): no bank
// conflict in either direction.
constexpr int kChunk = 16;
constexpr int kStageBytes = kChunk * 64;
constexpr int kEpiWarps = 16;   // of the pair kernel

struct WarpStage {
    uint32_t mat;       // shared address of this lane's row for ldmatrix / stmatrix, c group 0
    uint4 *vec;         // this lane's piece of row lane / 4, c group 0
    __device__ __forceinline__ WarpStage(uint8_t *base, int lane)
    {
        const int c = lane & 7, v = lane & 3;
        mat = smem_u32(base) + c * 64 + (((lane >> 3) ^ (c >> 1)) & 3) * 16;
        vec = reinterpret_cast<uint4 *>(base + (lane >> 2) * 64 + ((v ^ (lane >> 3)) & 3) * 16);
    }
};

// The staged 16 x 32 values to dst + c * ld (dst: this lane's piece of row lane / 4).
__device__ __forceinline__ void copy_out(const WarpStage &w, uint16_t *dst, long long ld8, int rows)
{
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kChunk / 8; ++i) {
        if (8 * i < rows)
            *reinterpret_cast<uint4 *>(dst) = w.vec[i * 32];
        dst += ld8;
    }
    __syncwarp();
}

// 32 lanes x 16 columns of an accumulator; tmem_ld_wait() before v is used.
__device__ __forceinline__ void load_acc(uint32_t taddr, float (&v)[2][8])
{
    tmem_ld16(taddr, v[0]);
    tmem_ld16(taddr + (16u << 16), v[1]);
}

// This lane's pieces of the residual's rows c0 + [0, n), n <= 16 (see store_chunk).
template <LinMode MODE>
__device__ __forceinline__ void load_residual(const LinOut &o, long long c0, int m0, int M, int n,
                                              int lane, uint4 (&res)[kChunk / 8])
{
    if (MODE != LIN_FWD || !o.residual)
        return;
    const int m = m0 + (lane & 3) * 8, rows = m < M ? n - (lane >> 2) : 0;
    const uint16_t *src = o.residual + (c0 + (lane >> 2)) * o.ld + m;
#pragma unroll
    for (int i = 0; i < kChunk / 8; ++i) {
        if (8 * i < rows)
            res[i] = *reinterpret_cast<const uint4 *>(src);
        src += 8 * o.ld;
    }
}

// Columns [0, n) of an accumulator, n <= 16, to rows c0 + [0, n) of m [m0, m0 + 32)
// cut at M. bias[i]: of m0 + 8 i + lane / 4; res: this lane's pieces of the residual.
// `loaded` runs before the first use of v.
template <LinMode MODE, int ACT, class F>
__device__ __forceinline__ void store_chunk(const LinOut &o, float (&v)[2][8],
                                            const float (&bias)[4], const uint4 (&res)[kChunk / 8],
                                            long long c0, int m0, int M, int n, int lane,
                                            const WarpStage &w, F loaded)
{
    const int m = m0 + (lane & 3) * 8;
    // rows this lane moves: c = lane / 4 + 8 i < n, none when its m lie past the end
    const int rows = m < M ? n - (lane >> 2) : 0;
    const long long at = (c0 + (lane >> 2)) * o.ld + m, ld8 = 8 * o.ld;
    loaded();
    if (MODE == LIN_FWD) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            v[i >> 3][i & 7] += bias[(i >> 3) * 2 + ((i >> 1) & 1)];
        if (o.z) {
#pragma unroll
            for (int ci = 0; ci < kChunk / 8; ++ci) {
                uint32_t r[4];
#pragma unroll
                for (int mi = 0; mi < 4; ++mi) {
                    const int k = 4 * ci + 2 * (mi & 1);
                    r[mi] = pack_bf16x2(v[mi >> 1][k], v[mi >> 1][k + 1]);
                }
                stmatrix4_t(w.mat + ci * 512, r);
            }
            copy_out(w, o.z + at, ld8, rows);
        }
        if (o.residual) {
#pragma unroll
            for (int i = 0; i < kChunk / 8; ++i)
                if (8 * i < rows)
                    w.vec[i * 32] = res[i];
            __syncwarp();
        }
    }
#pragma unroll
    for (int ci = 0; ci < kChunk / 8; ++ci) {
        uint32_t r[4];
        if (MODE == LIN_FWD && o.residual)
            ldmatrix4_t(w.mat + ci * 512, r);
        float f[2][4];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i >> 2][i & 3] = v[i >> 2][4 * ci + (i & 3)];
        act_n<ACT>(f[0]);
        act_n<ACT>(f[1]);
#pragma unroll
        for (int mi = 0; mi < 4; ++mi) {
            float a = f[mi >> 1][2 * (mi & 1)], b = f[mi >> 1][2 * (mi & 1) + 1];
            if (MODE == LIN_FWD && o.residual) {
                a += bf16lo(r[mi]);
                b += bf16hi(r[mi]);
            }
            r[mi] = pack_bf16x2(a, b);
        }
        stmatrix4_t(w.mat + ci * 512, r);
    }
    copy_out(w, o.out + at, ld8, rows);
}

// A warp's part of a tile: columns h * 16 + [0, 16), and every 16 NH from there, below
// cn (NH warps share a lane quarter). res: the residual of the first chunk; each next
// one's goes out a chunk ahead. `release` runs as soon as the last value has left the
// accumulator.
template <LinMode MODE, int ACT, int NH, class R>
__device__ __forceinline__ void store_tile(const LinOut &o, uint32_t tb, int h,
                                           const float (&bias)[4], uint4 (&res)[kChunk / 8],
                                           long long c0, int m0, int M, int cn, int lane,
                                           const WarpStage &w, R release)
{
    constexpr int STEP = kChunk * NH;
    const int first = h * kChunk;
    if (m0 >= M || first >= cn) {
        release();
        return;
    }
#pragma unroll 1
    for (int c = first; c < cn; c += STEP) {
        float v[2][8];
        uint4 next[kChunk / 8];
        load_acc(tb + c, v);
        load_residual<MODE>(o, c0 + c + STEP, m0, M, min(kChunk, cn - c - STEP), lane, next);
        store_chunk<MODE, ACT>(o, v, bias, res, c0 + c, m0, M, min(kChunk, cn - c), lane, w, [&] {
            tmem_ld_wait();
            if (c + STEP >= cn)
                release();
        });
#pragma unroll
        for (int i = 0; i < kChunk / 8; ++i)
            res[i] = next[i];
    }
}

// Zeros in place of a tile: the gradient of an empty group's weights. Rows of 256 bytes.
__device__ __forceinline__ void store_zeros(const LinOut &o, int warp, long long c0, int mt, int M, int cn,
                                            int lane)
{
    const int m = mt + (lane & 15) * 8;
    for (int c = 2 * warp + (lane >> 4); c < cn && m < M; c += 2 * kEpiWarps)
        *reinterpret_cast<uint4 *>(o.out + (c0 + c) * o.ld + m) = make_uint4(0, 0, 0, 0);
}

// fp32 partial sums of dW: a lane holds one m of 32 columns, and a warp's store is 128
// contiguous bytes.
__device__ __forceinline__ void store_part(float *part, long long ld, uint32_t taddr, bool zero,
                                           long long c0, int m, int M, int n)
{
    float v[32];
    if (zero) {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            v[j] = 0.f;
    } else {
        tmem_ld32(taddr, v);
        tmem_ld_wait();
    }
    if (m >= M)
        return;
    float *dst = part + c0 * ld + m;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        if (j < n)
            *dst = v[j];
        dst += ld;
    }
}

template <LinMode MODE>
__device__ __forceinline__ void load_bias(const LinOut &o, long long first, int m0, int M, int lane,
                                          float (&bias)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int m = m0 + 8 * i + (lane >> 2);
        bias[i] = (MODE == LIN_FWD && o.bias && m < M) ? o.bias[first + m] : 0.f;
    }
}

// ---------------------------------------------------------------- pair kernel
// Persistent; a cluster of two CTAs computes tiles of 256 (m) x up to 256 (c)
// with cta_group::2 MMAs that the leader issues: each CTA loads its own 128 m
// of A and its own half of the tile's c of B. Two accumulators of 256 TMEM
// columns alternate, so a tile's epilogue overlaps the next tile's main loop.
//   warp 0   producer        warp 1   MMA issue (leader)
//   warp 2   dW: zeroes the rows of a group's last block past its end
//   warps 4-19  epilogue, four per TMEM lane quarter, taking 16 columns in turn. With two
//               per quarter 16384 x 256 -> 4096 took 45 us and 103 with gelu
constexpr int kPairThreads = 128 + 32 * kEpiWarps;
constexpr int kPairABytes = 2 * kBoxBytes;
constexpr int kRingBytes = 24 * kBoxBytes;
constexpr int kPairBars = 768;
constexpr int kPairSmem = 1024 + kRingBytes + kPairBars + kEpiWarps * kStageBytes;

// Stages of the ring for tiles of each class (class 0: up to 256 rows; 1: 128; 2:
// 64): the smaller the tokens' part of a stage, the more stages fit. A stage's round
// trip (copy, MMAs, commit, the producer's wait) takes 1.9 us even on an idle GPU,
// so 6 stages of 16 KB of weights let an SM read 51 GB/s, and 9 half as much again.
// Each class has its own barriers; a CTA passes each class once, and goes to the next only
// when every stage of the last one has been consumed. Class 3 is for double tiles (up to
// 512 rows), in the place of class 0.
__host__ __device__ constexpr int ring_stages(int c) { return c == 0 ? 6 : c == 1 ? 8 : c == 2 ? 9 : 4; }
__host__ __device__ constexpr int ring_stage_bytes(int c)
{
    return kPairABytes +
           (c == 0 ? 2 * kBoxBytes : c == 1 ? kBoxBytes : c == 2 ? kBoxBytes / 2 : 4 * kBoxBytes);
}
__host__ __device__ constexpr int ring_bar(int c) { return c == 0 ? 0 : c == 1 ? 6 : c == 2 ? 14 : 23; }
constexpr int kRingBars = 27;

// A role's place in the ring: its stage's barrier (its index in full and empty), byte
// offset and the parity of the stage's current use. Kept by steps, not by division, and
// with the class's numbers at hand: the producer and the MMA issue are one thread each,
// and what they spend on a stage is not hidden. Divisions by a stage count of 6, 8 or 9
// cost 8% of 16384 x 14336 -> 4096, and numbers chosen by class at every step 57% of
// 73 x 14336 -> 18944 (141 us against 89).
struct Ring {
    int cls, bar, at;
    uint32_t phase;
    bool used;
    int first, end, bytes;
    __device__ __forceinline__ explicit Ring(int c)
        : cls(c), bar(ring_bar(c)), at(0), phase(0), used(false), first(ring_bar(c)),
          end(ring_bar(c) + ring_stages(c)), bytes(ring_stage_bytes(c))
    {
    }
    __device__ __forceinline__ void next()
    {
        used = true;
        ++bar;
        at += bytes;
        if (bar == end) {
            bar = first;
            at = 0;
            phase ^= 1u;
        }
    }
    // the stage before this one
    __device__ __forceinline__ int last() const { return bar == first ? end - 1 : bar - 1; }
    __device__ __forceinline__ uint32_t last_phase() const { return bar == first ? phase ^ 1u : phase; }
};
static_assert(6 * ring_stage_bytes(0) <= kRingBytes && 8 * ring_stage_bytes(1) <= kRingBytes &&
                  9 * ring_stage_bytes(2) <= kRingBytes && 4 * ring_stage_bytes(3) <= kRingBytes,
              "the ring holds every class");
static_assert((2 * kRingBars + 4 + ring_stages(0)) * 8 + 8 <= kPairBars, "room for the barriers");

// n / d for 0 <= n < 2^31 by a multiplication: n (ceil(2^64 / d) / 2^64 - 1 / d) < 2^-32
// cannot reach the next integer.
struct Divisor {
    unsigned long long inv;   // 0: d = 1
    void set(int d) { inv = d == 1 ? 0 : ~0ull / (unsigned)d + 1; }
    __device__ __forceinline__ int div(int n) const
    {
        return inv ? (int)__umul64hi((unsigned long long)n, inv) : n;
    }
};

struct PairArgs {
    const int32_t *offsets;
    int E, rows, d_in, d_out;
    int m_tiles;     // tiles of 256 along m
    int c_tiles;     // LIN_DW: tiles of 256 along d_out
    int kblocks;     // LIN_FWD, LIN_DX
    int band;        // items of a group whose B rows stay in L2 while W passes by
    int splits;      // LIN_DW
    Divisor by_m, by_c, by_split;   // m_tiles, c_tiles, splits
    bool a_wide, b_wide;   // MN-major operands: two boxes in one copy
    bool late;       // see LinArgs
    // Bound of every wait. starve (test only): the second CTA's producer stops before the last
    // K block of its first tile, so that block's stage never fills on either side.
    unsigned long long wait_ns;
    bool starve;
    LinOut o;
    uint32_t *status;
};

// Maps of the tokens' operand with boxes of 16, 32, 64 and 128 rows: a tile takes
// its rows in one copy that is no larger than it has to be. (LIN_DW: box[0] only.)
// Copies are issued by one thread, and their number counts as well as their
// bytes: with two boxes of 64 rows in place of one of 128 the loads alone of
// 16384 x 14336 -> 4096 took 1100 us, with one 835.
struct BMaps {
    CUtensorMap box[4];
};

struct TileAt {
    int e, m0;        // group, first m
    int c0, cn;       // first c (a row, or an output feature) and how many
    int r0;           // LIN_DW: first row of the contraction
    int nkb, tail;    // K blocks; LIN_DW: rows of the last block (0: all 64)
    int split;
    int cn2;          // double tile: rows of its second half, which follow the first's; else 0
};

// Rows of one token tile of a group of n rows: near-equal tiles of at most 256,
// a multiple of 32. Never leaves a tile empty: 256 (tiles - 1) < n.
__device__ __forceinline__ int tile_rows(int n)
{
    const int nt = (n + kTileC - 1) / kTileC;
    return ((n + nt - 1) / nt + 31) & ~31;
}

template <LinMode MODE, bool WIDE>
__device__ __forceinline__ TileAt tile_at(const PairArgs &p, const GroupSmem &G, int t)
{
    TileAt a;
    if (MODE == LIN_DW) {
        const int cg = p.by_m.div(t), g = p.by_c.div(cg);
        a.e = p.by_split.div(g);
        a.split = g - a.e * p.splits;
        a.cn2 = 0;
        a.m0 = (t - cg * p.m_tiles) * 256;
        a.c0 = (cg - g * p.c_tiles) * kTileC;
        a.cn = min(kTileC, p.d_out - a.c0);
        const int first = G.row0[a.e], n = G.row0[a.e + 1] - first;
        const int all = (n + kBox - 1) / kBox, part = p.by_split.div(all + p.splits - 1);
        const int k0 = min(a.split * part, all), k1 = min(k0 + part, all);
        a.nkb = k1 - k0;
        a.r0 = first + k0 * kBox;
        a.tail = (k1 == all && k1 > k0) ? n - (all - 1) * kBox : 0;
        if (a.tail == kBox)
            a.tail = 0;
    } else {
        const int at = item_group(G, p.E, p.by_m.div(t));
        a.e = G.group[at];
        const int f = G.first[at], ni = G.first[at + 1] - f;
        const int local = t - f * p.m_tiles;
        const int per = p.band * p.m_tiles;
        const int b = local / per, r = local - b * per;
        const int in_band = min(p.band, ni - b * p.band);
        const int i = b * p.band + r % in_band;
        a.m0 = (r / in_band) * 256;
        const int first = G.row0[a.e], n = G.row0[a.e + 1] - first;
        const int q = tile_rows(n);
        const int c = (WIDE ? 2 * i : i) * q;
        a.c0 = first + c;
        a.cn = min(q, n - c);
        a.cn2 = WIDE ? max(min(q, n - c - q), 0) : 0;
        a.nkb = p.kblocks;
        a.r0 = 0;
        a.tail = 0;
        a.split = 0;
    }
    return a;
}

// Calls f(tile, ring class) for a pair's tiles in order, until it returns false. The groups
// come by class, so a pair passes each ring once. (Starting half of the pairs with the
// short groups, so that tiles bound by the tensor cores run beside tiles bound by
// reading weights, changed nothing: 2482 us against 2447 for 256 skewed experts.)
template <LinMode MODE, bool WIDE, class F>
__device__ __forceinline__ void walk_tiles(const PairArgs &p, const GroupSmem &G, F f)
{
    const int total = MODE == LIN_DW ? p.E * p.splits * p.m_tiles * p.c_tiles : G.cls[3] * p.m_tiles;
    const int end0 = G.cls[1] * p.m_tiles, end1 = G.cls[2] * p.m_tiles;
    for (int t = blockIdx.x >> 1; t < total; t += gridDim.x >> 1) {
        const int c = MODE == LIN_DW ? 0 : t < end0 ? (WIDE ? 3 : 0) : t < end1 ? 1 : 2;
        if (!f(tile_at<MODE, WIDE>(p, G, t), c))
            return;
    }
}

template <LinMode MODE, int ACT, bool WIDE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    k_linear_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ BMaps tmB,
                  const PairArgs p)
{
    constexpr bool A_MN = MODE != LIN_FWD, B_MN = MODE == LIN_DW;
    extern __shared__ uint8_t smem_raw[];
    __shared__ GroupSmem G;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + kRingBytes);
    uint64_t *empty = full + kRingBars;
    uint64_t *tfull = empty + kRingBars;
    uint64_t *tempty = tfull + 2;
    uint64_t *tailbar = tempty + 2;   // one a stage: several last blocks may be in flight
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(tailbar + ring_stages(0));
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
    uint8_t *stage = smem + kRingBytes + kPairBars;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRingBars; ++s) {
            mbar_init(&full[s], 2);    // the leader's producer twice, or each CTA's warp 2 once
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < ring_stages(0); ++s)
            mbar_init(&tailbar[s], 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(&tfull[b], 1);
            mbar_init(&tempty[b], 2 * kEpiWarps);   // of both CTAs
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0 && lane == 0) {
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB.box[MODE == LIN_DW ? 0 : 3]);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, 512);
        tmem_relinquish_pair();
    }
    if (!p.late)
        pdl_wait();
    pdl_trigger();
    // items of one group: token tiles; LIN_DW needs the groups' rows only
    build_groups<true>(G, p.offsets, p.E, p.rows, WIDE ? 2 * kTileC : kTileC, p.status);
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers exist and TMEM is allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {   // ---------------- producer (both CTAs)
            Ring ring(WIDE ? 3 : 0);
            const uint32_t smem0 = smem_u32(smem), full0 = mapa_shared(smem_u32(full), 0);
            const int skip = p.starve && !leader ? 1 : 0;
            walk_tiles<MODE, WIDE>(p, G, [&](const TileAt &a, int c) {
                const int half = ((a.cn + 31) & ~31) / 2;      // c of this CTA
                const int c0 = a.c0 + (int)rank * half, m0 = a.m0 + 128 * (int)rank;
                const int fit = half <= 16 ? 0 : half <= 32 ? 1 : half <= 64 ? 2 : 3;
                const CUtensorMap *tb = &tmB.box[MODE == LIN_DW ? 0 : fit];
                const int nb = p.b_wide ? 1 : (half + kBox - 1) / kBox;   // LIN_DW: copies of B
                const int half2 = WIDE ? ((a.cn2 + 31) & ~31) / 2 : 0;
                const int c2 = a.c0 + a.cn + (int)rank * half2;
                const int fit2 = half2 <= 16 ? 0 : half2 <= 32 ? 1 : half2 <= 64 ? 2 : 3;
                const uint32_t bytes =
                    kPairABytes + (MODE == LIN_DW ? (p.b_wide ? 2 : nb) * kBoxBytes : 2048 << fit) +
                    (half2 ? 2048 << fit2 : 0);
                if (MODE != LIN_DW && c != ring.cls) {   // another ring over the same memory
                    if (ring.used && !mbar_wait(&empty[ring.last()], ring.last_phase(), abort_flag,
                                                p.status, p.wait_ns))
                        return false;
                    ring = Ring(c);
                }
                for (int kb = 0; kb < a.nkb - skip; ++kb) {
                    if (!mbar_wait(&empty[ring.bar], ring.phase ^ 1u, abort_flag, p.status, p.wait_ns))
                        return false;
                    const uint32_t sa = smem0 + ring.at, sb = sa + kPairABytes;
                    const bool tail = MODE == LIN_DW && a.tail && kb == a.nkb - 1;
                    uint32_t bar = full0 + ring.bar * 8;
                    if (tail) {   // to this CTA's own barrier; warp 2 passes it on
                        mbar_arrive_expect_tx(&tailbar[ring.bar], bytes);
                        bar = mapa_shared(smem_u32(&tailbar[ring.bar]), rank);
                    } else if (leader) {   // for both CTAs' copies: halves are equal
                        mbar_arrive_expect_tx(&full[ring.bar], 2 * bytes);
                        mbar_arrive(&full[ring.bar]);
                    }
                    ring.next();
                    const int k = kb * kBox;
                    if (WIDE && half2)
                        tma_2d_pair(sb + 2 * kBoxBytes, &tmB.box[fit2], k, c2, bar);
                    if (MODE == LIN_FWD) {
                        tma_3d_pair(sa, &tmA, k, m0, a.e, bar);
                        tma_2d_pair(sb, tb, k, c0, bar);
                        continue;
                    }
                    const int ka = MODE == LIN_DX ? k : a.r0 + k, ea = MODE == LIN_DX ? a.e : 0;
                    if (p.a_wide) {
                        tma_4d_pair(sa, &tmA, 0, ka, m0 / kBox, ea, bar);
                    } else {
                        tma_4d_pair(sa, &tmA, m0, ka, 0, ea, bar);
                        tma_4d_pair(sa + kBoxBytes, &tmA, m0 + kBox, ka, 0, ea, bar);
                    }
                    if (MODE == LIN_DX) {
                        tma_2d_pair(sb, tb, k, c0, bar);
                    } else if (p.b_wide) {
                        tma_4d_pair(sb, tb, 0, ka, c0 / kBox, 0, bar);
                    } else {
                        for (int j = 0; j < nb; ++j)
                            tma_4d_pair(sb + j * kBoxBytes, tb, c0 + j * kBox, ka, 0, 0, bar);
                    }
                }
                return skip == 0;
            });
        }
    } else if (warp == 1) {
        if (lane == 0 && leader) {   // ---------------- MMA issue
            uint32_t local = 0;
            Ring ring(WIDE ? 3 : 0);
            const uint32_t smem0 = smem_u32(smem);
            // the K steps of one stage into the accumulator at d; B at boff of the stage
            const auto mma = [&](uint32_t d, uint32_t idesc, const Ring &r, uint32_t boff, bool add,
                                 int rows) {
                const uint64_t da = op_desc<A_MN>(smem0 + r.at, 0);
                const uint64_t db = op_desc<B_MN>(smem0 + r.at + boff, 0);
#pragma unroll
                for (int kk = 0; kk < kBox / 16; ++kk)
                    if (kk * 16 < rows)
                        tc_mma_bf16_pair(d, da + kk * op_step<A_MN>(), db + kk * op_step<B_MN>(), idesc,
                                         add || kk != 0);
            };
            const auto wait_full = [&](const Ring &r) {
                const bool ok = mbar_wait(&full[r.bar], r.phase, abort_flag, p.status, p.wait_ns);
                tc_fence_after();
                return ok;
            };
            walk_tiles<MODE, WIDE>(p, G, [&](const TileAt &a, int c) {
                if (MODE == LIN_DW && a.nkb == 0)
                    return true;         // nothing to add up: the epilogue writes zeros
                if (MODE != LIN_DW && c != ring.cls)
                    ring = Ring(c);
                const uint32_t b = local & 1u, aph = (local >> 1) & 1u;
                ++local;
                const uint32_t idesc = lin_idesc<MODE>(256, (a.cn + 31) & ~31);
                if (!mbar_wait(&tempty[b], aph ^ 1u, abort_flag, p.status, p.wait_ns))
                    return false;
                tc_fence_after();
                const uint32_t d = tmem_base + b * kTileC;
                if (WIDE && a.cn2) {
                    // Both accumulators at work: the first four stages go into the first
                    // one while the epilogue may still read the second, and the last four
                    // finish the first one early.
                    const uint32_t b2 = local & 1u, aph2 = (local >> 1) & 1u;
                    ++local;
                    const uint32_t idesc2 = lin_idesc<MODE>(256, (a.cn2 + 31) & ~31);
                    const uint32_t d2 = tmem_base + b2 * kTileC, boff2 = kPairABytes + 2 * kBoxBytes;
                    const int head = min(a.nkb, ring_stages(3));
                    const int tail = a.nkb >= 2 * ring_stages(3) ? ring_stages(3) : 0;
                    Ring r = ring;
                    for (int kb = 0; kb < head; ++kb, r.next()) {
                        if (!wait_full(r))
                            return false;
                        mma(d, idesc, r, kPairABytes, kb != 0, kBox);
                    }
                    if (!mbar_wait(&tempty[b2], aph2 ^ 1u, abort_flag, p.status, p.wait_ns))
                        return false;
                    tc_fence_after();
                    for (int kb = 0; kb < head; ++kb, ring.next()) {
                        mma(d2, idesc2, ring, boff2, kb != 0, kBox);
                        tc_commit_pair(&empty[ring.bar], 0x3);
                    }
                    for (int kb = head; kb < a.nkb - tail; ++kb, ring.next()) {
                        if (!wait_full(ring))
                            return false;
                        mma(d, idesc, ring, kPairABytes, true, kBox);
                        mma(d2, idesc2, ring, boff2, true, kBox);
                        tc_commit_pair(&empty[ring.bar], 0x3);
                    }
                    r = ring;
                    for (int kb = 0; kb < tail; ++kb, r.next()) {
                        if (!wait_full(r))
                            return false;
                        mma(d, idesc, r, kPairABytes, true, kBox);
                    }
                    tc_commit_pair(&tfull[b], 0x3);
                    for (int kb = 0; kb < tail; ++kb, ring.next()) {
                        mma(d2, idesc2, ring, boff2, true, kBox);
                        tc_commit_pair(&empty[ring.bar], 0x3);
                    }
                    tc_commit_pair(&tfull[b2], 0x3);
                    return true;
                }
                for (int kb = 0; kb < a.nkb; ++kb, ring.next()) {
                    // Copies need no acquire beyond this CTA. One at cluster scope
                    // stalls the issue for longer than a stage's MMAs take, so only
                    // a last block, whose zeros the peer wrote, waits with it.
                    const bool last = MODE == LIN_DW && a.tail && kb == a.nkb - 1;
                    if (last && !mbar_wait_cluster(&full[ring.bar], ring.phase, abort_flag, p.status,
                                                   p.wait_ns))
                        return false;
                    if (!mbar_wait(&full[ring.bar], ring.phase, abort_flag, p.status, p.wait_ns))
                        return false;
                    tc_fence_after();
                    const uint64_t da = op_desc<A_MN>(smem0 + ring.at, 0);
                    const uint64_t db = op_desc<B_MN>(smem0 + ring.at + kPairABytes, 0);
#pragma unroll
                    for (int kk = 0; kk < kBox / 16; ++kk)
                        if (!last || kk * 16 < a.tail)
                            tc_mma_bf16_pair(d, da + kk * op_step<A_MN>(), db + kk * op_step<B_MN>(),
                                             idesc, (kb | kk) != 0);
                    tc_commit_pair(&empty[ring.bar], 0x3);
                }
                tc_commit_pair(&tfull[b], 0x3);
                return true;
            });
        }
    } else if (MODE == LIN_DW && warp == 2) {   // ---------------- last blocks (both CTAs)
        uint32_t it = 0, phases = 0;   // bit s: parity of stage s's next use
        walk_tiles<MODE, WIDE>(p, G, [&](const TileAt &a, int) {
            it += a.nkb;
            if (!a.tail)
                return true;
            const uint32_t s = (it - 1) % ring_stages(0);
            if (!__all_sync(kFullMask, mbar_wait(&tailbar[s], (phases >> s) & 1u, abort_flag, p.status,
                                                 p.wait_ns)))
                return false;
            phases ^= 1u << s;
            // row r of a 64 x 64 box is its bytes [128 r, 128 r + 128): the swizzle
            // only permutes the 16-byte pieces of a row. Rows past the last K step of
            // 16 that the MMAs take need no zeros.
            const int end = (a.tail + 15) & ~15;
            const int boxes = p.b_wide ? 4 : 2 + (((a.cn + 31) & ~31) / 2 + kBox - 1) / kBox;
            for (int r = a.tail + (lane >> 3); r < end; r += 4)
                for (int j = 0; j < boxes; ++j)
                    *reinterpret_cast<uint4 *>(smem + s * ring_stage_bytes(0) + j * kBoxBytes +
                                               r * 128 + (lane & 7) * 16) = make_uint4(0, 0, 0, 0);
            fence_proxy_async();
            __syncwarp();
            if (lane == 0)
                mbar_arrive_cluster(mapa_shared(smem_u32(&full[s]), 0));
            return true;
        });
    } else if (warp >= 4) {   // ---------------- epilogue (both CTAs)
        const int q = warp & 3, h = (warp - 4) >> 2;
        const int M = MODE == LIN_FWD ? p.d_out : p.d_in;
        const WarpStage ws(stage + (warp - 4) * kStageBytes, lane);
        uint32_t local = 0;
        walk_tiles<MODE, WIDE>(p, G, [&](const TileAt &a, int) {
            const int m0 = a.m0 + 128 * (int)rank + q * 32;
            // first row of the output: dW's rows count from expert (and split) 0
            const long long c00 =
                MODE == LIN_DW ? ((long long)(p.o.part ? a.split * p.E : 0) + a.e) * p.d_out : 0;
            const bool none = MODE == LIN_DW && a.nkb == 0;
            float bias[4];
            load_bias<MODE>(p.o, (long long)a.e * p.d_out, m0, M, lane, bias);
            for (int part = 0; part < (WIDE && a.cn2 ? 2 : 1); ++part) {   // one, or the two of a double tile
                const int cn = part ? a.cn2 : a.cn;
                const long long c0 = c00 + a.c0 + (part ? a.cn : 0);
                const uint32_t b = local & 1u, aph = (local >> 1) & 1u;
                uint4 res[kChunk / 8];
                load_residual<MODE>(p.o, c0 + h * kChunk, m0, M, min(kChunk, cn - h * kChunk), lane, res);
                if (!none) {
                    if (!__all_sync(kFullMask, mbar_wait(&tfull[b], aph, abort_flag, p.status,
                                                         p.wait_ns)))
                        return false;
                    ++local;
                    tc_fence_after();
                }
                const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + b * kTileC;
                const auto release = [&] {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive_remote(mapa_shared(smem_u32(&tempty[b]), 0));
                };
                if (MODE == LIN_DW && p.o.part) {
                    for (int c = h * 32; c < cn && m0 < M; c += 32 * (kEpiWarps / 4))
                        store_part(p.o.part, p.o.ld, tb + c, none, c0 + c, m0 + lane, M,
                                   min(32, cn - c));
                    if (!none)
                        release();
                } else if (none) {
                    store_zeros(p.o, warp - 4, c0, a.m0 + 128 * (int)rank, M, cn, lane);
                } else {
                    store_tile<MODE, ACT, kEpiWarps / 4>(p.o, tb, h, bias, res, c0, m0, M, cn, lane,
                                                         ws, release);
                }
            }
            return true;
        });
    }

    __syncthreads();
    if (*abort_flag) {   // a wait ran out: let this CTA's copies in flight land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull)
            ;
        __syncwarp();
    }
    tc_fence_before();
    cluster_sync_all();   // neither CTA leaves while the pair's MMAs may read its memory
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem_base, 512);
    }
    if (p.late)
        pdl_wait();
}

// ---------------------------------------------------------------- split kernel
// For few tiles (one token, small batches, small layers): one CTA per 128 (m) x
// up to BC (c) x a slice of K; the S CTAs of a cluster split K and add their
// accumulators through distributed shared memory in rank order (no atomics, no
// workspace). Not persistent: with BC <= 128 two CTAs share an SM, so one's
// start and end hide behind the other's loads.
template <int BC>
struct SplitCfg {
    static constexpr int BOXROWS = BC < 128 ? BC : 128;
    static constexpr int A_BYTES = 2 * kBoxBytes;
    static constexpr int B_BYTES = BC * 128;
    static constexpr int STAGE = A_BYTES + B_BYTES;
    static constexpr int STAGES = BC == 32 ? 5 : BC == 128 ? 3 : 4;
    static constexpr int SMEM = 1024 + STAGES * STAGE + 256;
    static_assert(BC * 128 * 4 <= STAGES * STAGE, "the partial sums reuse the ring");
};

struct SplitArgs {
    const int32_t *offsets;
    int E, rows, d_in, d_out;
    int S, log_s;
    int kblocks;
    bool a_wide;
    bool late;       // see LinArgs
    // Bound of every wait. starve (test only): the producer of each cluster's last CTA stops
    // before its last K block.
    unsigned long long wait_ns;
    bool starve;
    LinOut o;
    uint32_t *status;
};

template <LinMode MODE, int ACT, int BC>
__global__ void __launch_bounds__(256, BC <= 128 ? 2 : 1)
    k_linear_split(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const SplitArgs p)
{
    using C = SplitCfg<BC>;
    constexpr bool A_MN = MODE == LIN_DX;
    extern __shared__ uint8_t smem_raw[];
    __shared__ GroupSmem G;
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::STAGES * C::STAGE);
    uint64_t *empty = full + C::STAGES;
    uint64_t *done = empty + C::STAGES;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = blockIdx.x % p.S;   // clusters run along x
    const int m0 = (blockIdx.x / p.S) * 128;
    // what needs nothing of the kernel before this one, while that one ends
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(done, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmA);
        tma_prefetch_desc(&tmB);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, BC);
        tmem_relinquish();
    }
    if (!p.late)
        pdl_wait();
    pdl_trigger();
    const int item = blockIdx.y;
    int e = 0, c0 = item * BC, cn = min(BC, p.rows - c0);
    bool any = true;
    if (p.offsets) {
        build_groups(G, p.offsets, p.E, p.rows, BC, p.status);
        any = item < G.first[p.E];   // the same for the whole cluster: it has one blockIdx.y
        if (any) {
            e = item_group(G, p.E, item);
            c0 = G.row0[e] + (item - G.first[e]) * BC;
            cn = min(BC, G.row0[e + 1] - c0);
        }
    }
    const int per = (p.kblocks + p.S - 1) / p.S;
    const int k0 = min(rank * per, p.kblocks), nkb = min(k0 + per, p.kblocks) - k0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    if (!any) {
        if (warp == 1)
            tmem_dealloc(tmem_base, BC);
        if (p.late)
            pdl_wait();
        return;
    }

    if (warp == 0 && lane == 0) {   // ---------------- producer
        const int nb = (cn + C::BOXROWS - 1) / C::BOXROWS;
        const uint32_t bytes = C::A_BYTES + nb * C::BOXROWS * 128;
        const int loads = p.starve && rank == p.S - 1 ? nkb - 1 : nkb;
        for (int i = 0; i < loads; ++i) {
            const int s = i % C::STAGES;
            if (!mbar_wait(&empty[s], ((i / C::STAGES) & 1u) ^ 1u, abort_flag, p.status, p.wait_ns))
                break;
            uint8_t *sa = smem + s * C::STAGE, *sb = sa + C::A_BYTES;
            mbar_arrive_expect_tx(&full[s], bytes);
            const int k = (k0 + i) * kBox;
            if (A_MN && p.a_wide) {
                tma_4d(sa, &tmA, 0, k, m0 / kBox, e, &full[s]);
            } else if (A_MN) {
                tma_4d(sa, &tmA, m0, k, 0, e, &full[s]);
                tma_4d(sa + kBoxBytes, &tmA, m0 + kBox, k, 0, e, &full[s]);
            } else {
                tma_3d(sa, &tmA, k, m0, e, &full[s]);
            }
            for (int j = 0; j < nb; ++j)
                tma_load_2d(sb + j * C::BOXROWS * 128, &tmB, k, c0 + j * C::BOXROWS, &full[s]);
        }
    } else if (warp == 1 && lane == 0) {   // ---------------- MMA issue
        const uint32_t idesc = lin_idesc<MODE>(128, (cn + 15) & ~15);
        bool ok = true;
        for (int i = 0; i < nkb; ++i) {
            const int s = i % C::STAGES;
            if (!mbar_wait(&full[s], (i / C::STAGES) & 1u, abort_flag, p.status, p.wait_ns)) {
                ok = false;
                break;
            }
            tc_fence_after();
            const uint32_t a0 = smem_u32(smem + s * C::STAGE), b0 = a0 + C::A_BYTES;
#pragma unroll
            for (int kk = 0; kk < kBox / 16; ++kk)
                tc_mma_bf16(tmem_base, op_desc<A_MN>(a0, kk), op_desc<false>(b0, kk), idesc,
                            (i | kk) != 0);
            tc_commit(&empty[s]);
        }
        if (ok)
            tc_commit(done);
    }
    __syncwarp();

    // ---------------- epilogue: all eight warps, two per TMEM lane quarter
    const int q = warp & 3, h = warp >> 2, mq = m0 + q * 32;
    const int M = MODE == LIN_FWD ? p.d_out : p.d_in;
    const uint32_t tb = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    float bias[4];
    uint4 res[kChunk / 8];
    if (p.S == 1) {
        load_bias<MODE>(p.o, (long long)e * p.d_out, mq, M, lane, bias);
        load_residual<MODE>(p.o, c0 + h * kChunk, mq, M, min(kChunk, cn - h * kChunk), lane, res);
    }
    const bool got = __all_sync(kFullMask, mbar_wait(done, 0, abort_flag, p.status, p.wait_ns));
    tc_fence_after();
    if (p.S == 1) {
        // the ring, which every copy and MMA has left, holds the rows on their way out
        const WarpStage ws(smem + warp * kStageBytes, lane);
        if (got)
            store_tile<MODE, ACT, 2>(p.o, tb, h, bias, res, c0, mq, M, cn, lane, ws, [] {});
    } else {
        // partial sums [c][128 m] over the ring, which every copy and MMA has left
        float *mine = reinterpret_cast<float *>(smem);
#pragma unroll 1
        for (int c = h * 32; got && c < cn; c += 64) {
            float v[32];
            if (nkb > 0) {
                tmem_ld32(tb + c, v);
                tmem_ld_wait();
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c + j < cn)
                    mine[(c + j) * 128 + q * 32 + lane] = v[j];
        }
        __syncwarp();
        cluster_sync_all();
        // each CTA finishes 128 / S of the m of every token, a thread four of them (S is a
        // power of two, and all sizes are multiples of 8)
        const int quads = 5 - p.log_s;   // log2 of (128 / S) / 4
        uint32_t peer[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            peer[r] = r < p.S ? mapa_shared(smem_u32(mine), r) : 0u;
        if (got)
            for (int i = threadIdx.x; i < cn << quads; i += 256) {
                const int c = i >> quads, ml = (rank << (quads + 2)) + (i & ((1 << quads) - 1)) * 4;
                const int m = m0 + ml;
                if (m >= M)
                    continue;
                float4 part[8];
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (r < p.S)
                        asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                                     : "=f"(part[r].x), "=f"(part[r].y), "=f"(part[r].z), "=f"(part[r].w)
                                     : "r"(peer[r] + (uint32_t)(c * 128 + ml) * 4u));
                const long long at = (long long)(c0 + c) * p.o.ld + m;
                uint2 res = make_uint2(0, 0);
                float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
                if (MODE == LIN_FWD) {
                    if (p.o.residual)
                        res = *reinterpret_cast<const uint2 *>(p.o.residual + at);
                    if (p.o.bias)
                        f = *reinterpret_cast<const float4 *>(p.o.bias + (long long)e * p.d_out + m);
                }
                float4 sum = part[0];
#pragma unroll
                for (int r = 1; r < 8; ++r)
                    if (r < p.S)
                        sum.x += part[r].x, sum.y += part[r].y, sum.z += part[r].z, sum.w += part[r].w;
                if (MODE == LIN_FWD) {
                    sum.x += f.x, sum.y += f.y, sum.z += f.z, sum.w += f.w;
                    if (p.o.z)
                        *reinterpret_cast<uint2 *>(p.o.z + at) =
                            make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
                    float v[4] = {sum.x, sum.y, sum.z, sum.w};
                    act_n<ACT>(v);
                    sum = make_float4(v[0], v[1], v[2], v[3]);
                    if (p.o.residual) {
                        sum.x += bf16lo(res.x), sum.y += bf16hi(res.x);
                        sum.z += bf16lo(res.y), sum.w += bf16hi(res.y);
                    }
                }
                *reinterpret_cast<uint2 *>(p.o.out + at) =
                    make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
            }
        __syncwarp();
        cluster_sync_all();   // no CTA leaves while another reads its sums
    }
    if (*abort_flag) {   // a wait ran out: let this CTA's copies in flight land
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000ull)
            ;
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem_base, BC);
    }
    if (p.late)
        pdl_wait();
}

// dW = bf16(sum over the splits, in order).
__global__ void __launch_bounds__(256)
    k_linear_dw_sum(const float4 *__restrict__ part, uint2 *__restrict__ dW, long long n4, int splits)
{
    pdl_wait();
    pdl_trigger();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= n4)
        return;
    float4 s = part[i];
    for (int k = 1; k < splits; ++k) {
        const float4 v = part[i + k * n4];
        s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    dW[i] = make_uint2(pack_bf16x2(s.x, s.y), pack_bf16x2(s.z, s.w));
}

// ---------------------------------------------------------------- host side

PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

int encode(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims,
           const cuuint64_t *strides, const cuuint32_t *box)
{
    auto fn = encode_fn();
    if (!fn)
        return MOE_ERR_CUDA;
    const cuuint32_t estr[4] = {1u, 1u, 1u, 1u};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims,
                          strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? MOE_OK : MOE_ERR_CUDA;
}

// bf16 [depth, rows, cols] (depth 0: two-dimensional); boxes of 64 x box_rows
// elements, 128-byte swizzle, zero fill outside.
int make_map(CUtensorMap *m, const void *base, long long cols, long long rows, long long depth,
             int box_rows)
{
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)depth};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * rows * 2};
    const cuuint32_t box[3] = {(cuuint32_t)kBox, (cuuint32_t)box_rows, 1u};
    return encode(m, base, depth ? 3 : 2, dims, strides, box);
}

// The same matrices for an MN-major operand, boxes of 64 x 64. `wide` (cols a
// multiple of 64): as [depth, cols / 64, rows, 64], two neighbouring boxes in one copy.
int make_map_mn(CUtensorMap *m, const void *base, long long cols, long long rows, long long depth,
                bool wide)
{
    const cuuint64_t dims[4] = {(cuuint64_t)(wide ? kBox : cols), (cuuint64_t)rows,
                                (cuuint64_t)(wide ? cols / kBox : 1), (cuuint64_t)depth};
    const cuuint64_t strides[3] = {(cuuint64_t)cols * 2, (cuuint64_t)kBox * 2,
                                   (cuuint64_t)cols * rows * 2};
    const cuuint32_t box[4] = {(cuuint32_t)kBox, (cuuint32_t)kBox, wide ? 2u : 1u, 1u};
    return encode(m, base, 4, dims, strides, box);
}

template <class K>
int allow_smem(K kernel, int bytes)
{
    return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
                   cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
}

int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

LinOut out_of(LinMode mode, const LinArgs &a)
{
    LinOut o;
    std::memset(&o, 0, sizeof o);
    o.bias = a.bias;
    o.residual = a.residual;
    o.out = a.out;
    o.z = a.z;
    o.part = (mode == LIN_DW && a.splits > 1) ? a.part : nullptr;
    o.ld = mode == LIN_FWD ? a.d_out : a.d_in;
    return o;
}

// Map of the tokens' operand (LIN_FWD, LIN_DX) with boxes of box_rows rows.
int token_map(LinMode mode, const LinArgs &a, int box_rows, CUtensorMap *B)
{
    return mode == LIN_FWD ? make_map(B, a.x, a.d_in, a.rows, 0, box_rows)
                           : make_map(B, a.dz, a.d_out, a.rows, 0, box_rows);
}

template <LinMode MODE, int ACT, bool WIDE = false>
int launch_pair(const LinArgs &a, cudaStream_t st)
{
    CUtensorMap A;
    BMaps B;
    // a tile's m start at multiples of 128; its two halves of c at multiples of 64
    // where all c come in multiples of 128
    const bool a_wide = a.d_in % kBox == 0, b_wide = MODE == LIN_DW && a.d_out % 128 == 0;
    int rc;
    if (MODE == LIN_FWD)
        rc = make_map(&A, a.W, a.d_in, a.d_out, a.E, 128);
    else if (MODE == LIN_DX)
        rc = make_map_mn(&A, a.W, a.d_in, a.d_out, a.E, a_wide);
    else if (!(rc = make_map_mn(&A, a.x, a.d_in, a.rows, 1, a_wide)))
        rc = make_map_mn(&B.box[0], a.dz, a.d_out, a.rows, 1, b_wide);
    for (int i = 0; i < 4 && !rc && MODE != LIN_DW; ++i)
        rc = token_map(MODE, a, 16 << i, &B.box[i]);
    if (rc || (rc = allow_smem(k_linear_pair<MODE, ACT, WIDE>, kPairSmem)))
        return rc;
    PairArgs p;
    std::memset(&p, 0, sizeof p);
    p.offsets = a.offsets;
    p.E = a.E;
    p.rows = a.rows;
    p.d_in = a.d_in;
    p.d_out = a.d_out;
    p.m_tiles = ceil_div(MODE == LIN_FWD ? a.d_out : a.d_in, 256);
    p.c_tiles = ceil_div(a.d_out, kTileC);
    const int K = MODE == LIN_FWD ? a.d_in : a.d_out;
    p.kblocks = ceil_div(K, kBox);
    // a band's token rows stay in L2 (48 MiB of them) while it sweeps the m tiles
    p.band = (int)std::max<long long>((48LL << 20) / ((long long)(WIDE ? 2 : 1) * kTileC * K * 2), 1);
    p.splits = std::max(a.splits, 1);
    p.by_m.set(p.m_tiles);
    p.by_c.set(p.c_tiles);
    p.by_split.set(p.splits);
    p.a_wide = a_wide;
    p.b_wide = b_wide;
    p.late = a.late;
    p.o = out_of(MODE, a);
    p.wait_ns = a.starve ? kTestWaitLimitNs : kWaitLimitNs;
    p.starve = a.starve;
    p.status = a.status;
    const long long tiles =
        MODE == LIN_DW ? (long long)a.E * p.splits * p.m_tiles * p.c_tiles
                       : (long long)(ceil_div(a.rows, kTileC) + std::min(a.E, a.rows)) * p.m_tiles;
    const int pairs = (int)std::min<long long>(tiles, num_sms() / 2);
    launch_pdl_ex(k_linear_pair<MODE, ACT, WIDE>, dim3(2 * pairs), dim3(kPairThreads), kPairSmem, st, A, B, p);
    if ((rc = launched()))
        return rc;
    if (MODE == LIN_DW && p.splits > 1) {
        const long long n4 = (long long)a.E * a.d_out * a.d_in / 4;
        launch_pdl_ex(k_linear_dw_sum, dim3(ceil_div(n4, 256)), dim3(256), 0, st,
                      reinterpret_cast<const float4 *>(a.part), reinterpret_cast<uint2 *>(a.out), n4,
                      p.splits);
        return launched();
    }
    return MOE_OK;
}

template <LinMode MODE, int ACT, int BC>
int launch_split(const LinArgs &a, int S, cudaStream_t st)
{
    using C = SplitCfg<BC>;
    CUtensorMap A, B;
    const bool a_wide = a.d_in % kBox == 0;
    int rc = MODE == LIN_FWD ? make_map(&A, a.W, a.d_in, a.d_out, a.E, 128)
                             : make_map_mn(&A, a.W, a.d_in, a.d_out, a.E, a_wide);
    if (rc || (rc = token_map(MODE, a, C::BOXROWS, &B)) ||
        (rc = allow_smem(k_linear_split<MODE, ACT, BC>, C::SMEM)))
        return rc;
    SplitArgs p;
    std::memset(&p, 0, sizeof p);
    p.offsets = a.offsets;
    p.E = a.E;
    p.rows = a.rows;
    p.d_in = a.d_in;
    p.d_out = a.d_out;
    p.S = S;
    while (1 << p.log_s < S)
        ++p.log_s;
    p.a_wide = a_wide;
    p.late = a.late;
    p.kblocks = ceil_div(MODE == LIN_FWD ? a.d_in : a.d_out, kBox);
    p.o = out_of(MODE, a);
    p.wait_ns = a.starve ? kTestWaitLimitNs : kWaitLimitNs;
    p.starve = a.starve;
    p.status = a.status;
    const int m_tiles = ceil_div(MODE == LIN_FWD ? a.d_out : a.d_in, 128);
    // a group of n rows has at most n / BC + 1 items, and none when it is empty
    const int items = a.offsets ? a.rows / BC + std::min(a.E, a.rows) : ceil_div(a.rows, BC);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(m_tiles * S, items);
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = S;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaLaunchKernelEx(&cfg, k_linear_split<MODE, ACT, BC>, A, B, p);
    return launched();
}

// Engine and shape of one product over token rows.
template <LinMode MODE, int ACT>
int launch_rows(const LinArgs &a, cudaStream_t st)
{
    const int M = MODE == LIN_FWD ? a.d_out : a.d_in, K = MODE == LIN_FWD ? a.d_in : a.d_out;
    const int groups = std::min(a.E, a.rows);
    const int avg = ceil_div(a.rows, groups);
    const long long pair_tiles = (long long)groups * ceil_div(avg, kTileC) * ceil_div(M, 256);
    const int sms = num_sms();
    // Pairs of SMs where each has a tile and the groups average more than 32 rows; single SMs
    // below, where the weights' stream decides. us single / pair, k = 8 of 256 experts of 4096
    // -> 4096: 16 tokens 515 / 576, 128 tokens 1247 / 1393, 1024 tokens (32 rows a group)
    // 1391 / 1485, the same by a Zipf law of 1.1 (1 to 900 rows) 1533 / 1538. Above: 4096 rows
    // in 64 groups 409 / 411, 1280 x 4096 -> 4096 52 / 47, dx of 4096 x 4096 -> 2048 56 / 49; but 128 x
    // 4096 -> 14336 28.2 / 30.0. Below a tile each: 512 x 4096 -> 4096 21 / 27, 4096 x 2048 -> 1024
    // 14.4 / 17.1. The average does not show how the rows fall, and the sizes are on the
    // device: 8192 rows are 420 / 240 when they all are one of 256 groups, 1683 / 1637 when the
    // other 255 have one row each.
    if (pair_tiles >= sms / 2 && avg > 32) {
        // Double tiles share the weights' part of a stage between 512 rows: a quarter less
        // from L2 for the same products, at the price of an epilogue that overlaps less.
        // us single -> double: 16384 x 14336 -> 4096 1522 -> 1444, 4096 x 8192 -> 4096 in 8
        // groups 263 -> 249, 16384 x 4096 -> 4096 469 -> 454, x 2048 256 -> 254, x 1024 149 ->
        // 148; where the pairs' last round fills up worse (8192 x 2048 -> 4096 in 8) 132 -> 144.
        const long long pairs = sms / 2, half = (pair_tiles + 1) / 2;
        if (avg >= 2 * kTileC && ceil_div(K, kBox) >= 32 &&
            2 * ((half + pairs - 1) / pairs) <= (pair_tiles + pairs - 1) / pairs)
            return launch_pair<MODE, ACT, true>(a, st);
        return launch_pair<MODE, ACT>(a, st);
    }
    // Tiles as wide as the groups (half as much again where those are ragged, so that few
    // are cut in two: 1024 x 1024 -> 1024 in 32 groups 15.2 us against 19.8); narrower
    // where that leaves half the SMs without one (300 x 1024 -> 1024: 6.7 with 32, 9.3 with
    // 128; the weights are then read more than once, but from L2).
    const int kb = ceil_div(K, kBox), need = a.offsets ? avg + avg / 2 : avg;
    int bc = need <= 32 ? 32 : need <= 64 ? 64 : need <= 128 ? 128 : 256;
    const auto tiles_of = [&](int b) {
        const long long items = a.offsets ? a.rows / b + groups : ceil_div(a.rows, b);
        return items * ceil_div(M, 128);
    };
    while (bc > (kb >= 32 ? 64 : 32) && tiles_of(bc) * 2 <= sms)
        bc /= 2;
    const long long tiles = tiles_of(bc);
    // CTAs that split K: enough to fill the SMs, each with eight K stages or more, four for
    // few rows, whose sums are joined sooner (one row, 2048 -> 2048: 4.6 us with four, 5.5
    // with eight, 11.5 unsplit; 1000 x 512 -> 512: 6.2 with four, 4.9 unsplit)
    const int stages = avg <= 16 ? 4 : 8;
    int S = 1;
    while (S < 8 && tiles * S * 2 <= (bc == 256 ? sms : 2 * sms) && kb >= 2 * S * stages)
        S *= 2;
    switch (bc) {
    case 32: return launch_split<MODE, ACT, 32>(a, S, st);
    case 64: return launch_split<MODE, ACT, 64>(a, S, st);
    case 128: return launch_split<MODE, ACT, 128>(a, S, st);
    default: return launch_split<MODE, ACT, 256>(a, S, st);
    }
}

} // namespace

// As many as there are SMs for the tiles, at most 16, none shorter than 512 rows: the sums over
// the rows are one chain of blocks a tile, and few tiles leave most SMs idle. us with 1 / 2 / 4 /
// 8 parts (the rule's own number, where it is another), dense layers:
//   512 -> 512 (4 tiles), 4096 rows 29.5 / 19.9 / 13.3 / 11.1; 16384 rows 94 / 50 / 29 / 19 (16: 22)
//   1024 -> 1024 (16 tiles), 1024 rows 11.2 / 11.1 (2); 4096 rows 29.5 / 20.8 / 15.4 / 18.2 (8: 22.0);
//     16384 rows 97 / 53 / 36 / 45 (9: 44)
//   1536 -> 1536 (36 tiles), 4096 rows 28.0 / 22.0 / 24.9 / 36.1 (4); 16384 rows 102 / 77 / 72 / 92 (4)
//   2048 -> 2048 (64 tiles), 1024 rows 12.3 / 19.2 (2); 4096 rows 31.4 / 41.9 (2: 36.1); 16384 rows
//     126 / 138 (2: 141)
//   2304 -> 2304 (81 tiles, never split), 4096 rows 50.8 / 50.0; 16384 rows 200 / 193
// The tiles run on pairs of SMs, so from 38 tiles on, and for short sums below that, the
// rule takes more parts than pay.
int lin_dw_splits(const moe_linear_t &s)
{
    const long long tiles = (long long)s.E * ceil_div(s.d_in, 256) * ceil_div(s.d_out, kTileC);
    const long long room = num_sms() / std::max<long long>(tiles, 1);
    return (int)std::max<long long>(1, std::min<long long>({room, 16LL, (long long)s.rows / 512}));
}

int launch_linear(LinMode mode, const LinArgs &a, cudaStream_t st)
{
    if (mode == LIN_DX)
        return launch_rows<LIN_DX, MOE_ACT_NONE>(a, st);
    if (mode == LIN_DW)
        return launch_pair<LIN_DW, MOE_ACT_NONE>(a, st);
    switch (a.act) {
    case MOE_ACT_NONE: return launch_rows<LIN_FWD, MOE_ACT_NONE>(a, st);
    case MOE_ACT_RELU: return launch_rows<LIN_FWD, MOE_ACT_RELU>(a, st);
    case MOE_ACT_GELU: return launch_rows<LIN_FWD, MOE_ACT_GELU>(a, st);
    case MOE_ACT_GELU_TANH: return launch_rows<LIN_FWD, MOE_ACT_GELU_TANH>(a, st);
    default: return launch_rows<LIN_FWD, MOE_ACT_SILU>(a, st);
    }
}

} // namespace moe
