// linear.cu -- linear products with bias, activation and residual, dense or
// grouped by expert with ragged sizes, and their gradients:
//   forward   y = act(x W_e^T + b_e) + residual       (z = x W_e^T + b_e kept on request)
//   backward  dz = dy act'(z), dx = dz W_e, dW_e = dz^T x, db_e = sum_r dz_r
// ("Expert FFN" and "Sparse MoE Block" on "MoE Model Architectures" with another
// activation, with biases, or alone.)
//
// This file holds the entry points and the elementwise pass of the backward;
// the products are in linear_tc.cu.
#include <algorithm>
#include <cstring>

#include "act.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "internal.h"
#include "linear.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- elementwise backward
// dz = dy act'(z) in bf16 and the column sums of the unrounded dz over items of
// kDzRows rows of one group. Bound by HBM: dy and z read, dz written once. A
// work unit is 256 columns (a lane 8 of them, 16-byte vectors) of an item; the 8
// warps take its rows in turn, kDzUnroll in flight each, and their sums meet in
// shared memory in warp order, so db repeats bit for bit. Persistent: the groups'
// list is built once a CTA, not once a unit. Measured with the bias sums: 4096 x 4096
// (100 MB) 20 us with silu, 23 with gelu's tanh form, 25 with gelu; a third more with 64 rows
// a unit.
constexpr int kDzRows = 32;
constexpr int kDzCols = 256;
constexpr int kDzUnroll = 4;   // rows of a warp in flight
constexpr int kDzCtasPerSm = 4;

template <int ACT>
__global__ void __launch_bounds__(256, kDzCtasPerSm)
    k_linear_dz(const uint4 *__restrict__ dy, const uint4 *__restrict__ z, uint4 *dz, float *part,
                const int32_t *offsets, int E, int rows, int d_out, uint32_t *status)
{
    __shared__ GroupSmem G;
    __shared__ float red[8][kDzCols];
    pdl_wait();
    pdl_trigger();
    build_groups(G, offsets, E, rows, kDzRows, status);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nv = d_out / 8, tiles = (d_out + kDzCols - 1) / kDzCols;
    const long long units = (long long)G.first[E] * tiles;
    for (long long unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int item = (int)(unit / tiles), tile = (int)(unit - (long long)item * tiles);
        const int e = item_group(G, E, item);
        const int r0 = G.row0[e] + (item - G.first[e]) * kDzRows;
        const int n = min(kDzRows, G.row0[e + 1] - r0);
        const int col = tile * kDzCols + lane * 8;
        float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (col < d_out) {
            const long long at0 = (long long)r0 * nv + col / 8;
            for (int r = warp; r < n; r += 8 * kDzUnroll) {
                uint4 g[kDzUnroll], zz[kDzUnroll];
#pragma unroll
                for (int u = 0; u < kDzUnroll; ++u)
                    if (r + 8 * u < n) {
                        g[u] = ld_stream_v4(dy + at0 + (long long)(r + 8 * u) * nv);
                        if (ACT != MOE_ACT_NONE)
                            zz[u] = ld_stream_v4(z + at0 + (long long)(r + 8 * u) * nv);
                    }
#pragma unroll
                for (int u = 0; u < kDzUnroll; ++u)
                    if (r + 8 * u < n) {
                        const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
                        const uint32_t zw[4] = {zz[u].x, zz[u].y, zz[u].z, zz[u].w};
                        uint32_t ow[4];
                        float slope[2][4];
                        if (ACT != MOE_ACT_NONE) {
#pragma unroll
                            for (int q = 0; q < 2; ++q) {
                                slope[q][0] = bf16lo(zw[2 * q]), slope[q][1] = bf16hi(zw[2 * q]);
                                slope[q][2] = bf16lo(zw[2 * q + 1]), slope[q][3] = bf16hi(zw[2 * q + 1]);
                                act_grad_n<ACT>(slope[q]);
                            }
                        }
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            float a = bf16lo(gw[q]), b = bf16hi(gw[q]);
                            if (ACT != MOE_ACT_NONE) {
                                a *= slope[q >> 1][2 * (q & 1)];
                                b *= slope[q >> 1][2 * (q & 1) + 1];
                            }
                            sum[2 * q] += a;
                            sum[2 * q + 1] += b;
                            ow[q] = pack_bf16x2(a, b);
                        }
                        if (ACT != MOE_ACT_NONE)
                            dz[at0 + (long long)(r + 8 * u) * nv] =
                                make_uint4(ow[0], ow[1], ow[2], ow[3]);
                    }
            }
        }
        if (!part)
            continue;
        // a lane's 8 sums lie 32 columns apart, so that neither side has bank conflicts
#pragma unroll
        for (int i = 0; i < 8; ++i)
            red[warp][i * 32 + lane] = sum[i];
        __syncthreads();
        const int c = tile * kDzCols + (threadIdx.x & 31) * 8 + warp;
        if (c < d_out) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < 8; ++w)
                s += red[w][threadIdx.x];
            part[(long long)item * d_out + c] = s;
        }
        __syncthreads();
    }
}

// db[e] = sum of the group's items (0 for an empty group). A CTA of 32 columns x 8:
// each of the 8 adds every eighth item, and their sums are added in order. In fp64: an item
// is 10 fp32 additions deep, but a group of 2^24 rows has 65,536 items for each of the 8,
// and terms of one sign and size left such a chain 5.5e-4 off in fp32 (2.4e-5 at 2^19 rows).
__global__ void __launch_bounds__(256)
    k_linear_db(const float *__restrict__ part, float *db, const int32_t *offsets, int E, int rows,
                int d_out)
{
    __shared__ GroupSmem G;
    __shared__ double red[8][32];
    pdl_wait();
    pdl_trigger();
    build_groups(G, offsets, E, rows, kDzRows, nullptr);
    const int e = blockIdx.y, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    double s = 0.0;
    if (c < d_out)
#pragma unroll 4
        for (int i = G.first[e] + w; i < G.first[e + 1]; i += 8)
            s += (double)part[(long long)i * d_out + c];
    red[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < d_out) {
#pragma unroll
        for (int k = 1; k < 8; ++k)
            s += red[k][lane];
        db[(long long)e * d_out + c] = (float)s;
    }
}

// ---------------------------------------------------------------- host side

int check_linear(const moe_linear_t *s)
{
    if (!s)
        return MOE_ERR_INVALID_ARG;
    auto dim = [](int v) { return v >= 8 && v <= 65536 && v % 8 == 0; };
    if (s->rows < 0 || s->rows > (1 << 24) || s->E < 1 || s->E > MOE_MAX_E || !dim(s->d_in) ||
        !dim(s->d_out) || s->act < MOE_ACT_NONE || s->act > MOE_ACT_SILU ||
        (s->flags & ~MOE_FLAG_TEST_TIMEOUT) != 0)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

long long dz_items(const moe_linear_t &s)
{
    return (s.rows + kDzRows - 1) / kDzRows + std::min(s.E, s.rows);
}

struct LinWs {
    size_t dz, part, dw_part, total;
    int splits;
};

LinWs lin_ws(const moe_linear_t &s)
{
    LinWs L;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t o = off;
        off += (bytes + 255) & ~static_cast<size_t>(255);
        return o;
    };
    L.dz = take(s.act != MOE_ACT_NONE ? (size_t)s.rows * s.d_out * 2 : 0);
    L.part = take((size_t)dz_items(s) * s.d_out * 4);
    L.splits = lin_dw_splits(s);
    L.dw_part = take(L.splits > 1 ? (size_t)L.splits * s.E * s.d_out * s.d_in * 4 : 0);
    L.total = std::max<size_t>(off, 256);
    return L;
}

template <int ACT>
int launch_dz(const moe_linear_t &s, const uint16_t *dy, const uint16_t *z, uint16_t *dz,
              float *part, const int32_t *offsets, uint32_t *status, cudaStream_t st)
{
    const long long units = dz_items(s) * ((s.d_out + kDzCols - 1) / kDzCols);
    launch_pdl_ex(k_linear_dz<ACT>,
                  dim3((unsigned)std::min<long long>(units, (long long)kDzCtasPerSm * num_sms())),
                  dim3(256), 0, st, reinterpret_cast<const uint4 *>(dy),
                  reinterpret_cast<const uint4 *>(z), reinterpret_cast<uint4 *>(dz), part, offsets,
                  s.E, s.rows, s.d_out, status);
    return launched();
}

int elementwise_backward(const moe_linear_t &s, const uint16_t *dy, const uint16_t *z,
                         uint16_t *dz, float *part, const int32_t *offsets, uint32_t *status,
                         cudaStream_t st)
{
    switch (s.act) {
    case MOE_ACT_NONE: return launch_dz<MOE_ACT_NONE>(s, dy, z, dz, part, offsets, status, st);
    case MOE_ACT_RELU: return launch_dz<MOE_ACT_RELU>(s, dy, z, dz, part, offsets, status, st);
    case MOE_ACT_GELU: return launch_dz<MOE_ACT_GELU>(s, dy, z, dz, part, offsets, status, st);
    case MOE_ACT_GELU_TANH:
        return launch_dz<MOE_ACT_GELU_TANH>(s, dy, z, dz, part, offsets, status, st);
    default: return launch_dz<MOE_ACT_SILU>(s, dy, z, dz, part, offsets, status, st);
    }
}

} // namespace
} // namespace moe

using namespace moe;

extern "C" {

int moe_linear_workspace_size(const moe_linear_t *shape, size_t *bytes)
{
    const int rc = check_linear(shape);
    if (rc)
        return rc;
    if (!bytes)
        return MOE_ERR_INVALID_ARG;
    *bytes = lin_ws(*shape).total;
    return MOE_OK;
}

int moe_linear_forward(const moe_linear_t *shape, const moe_bf16_t *x,
                       const int32_t *expert_offsets, const moe_bf16_t *W, const float *bias,
                       const moe_bf16_t *residual, moe_bf16_t *y, moe_bf16_t *z, uint32_t *status,
                       moe_stream_t stream)
{
    const int rc = check_linear(shape);
    if (rc)
        return rc;
    const moe_linear_t &s = *shape;
    if (!expert_offsets && s.E != 1)
        return MOE_ERR_INVALID_ARG;
    if (s.rows == 0)
        return MOE_OK;
    if (!x || !W || !y || !aligned(x, 16) || !aligned(W, 16) || !aligned(y, 16) ||
        !aligned(z, 16) || !aligned(residual, 16) || !aligned(bias, 16) ||
        !aligned(expert_offsets, 4))
        return MOE_ERR_INVALID_ARG;
    LinArgs p;
    std::memset(&p, 0, sizeof p);
    p.x = x;
    p.W = W;
    p.bias = bias;
    p.residual = residual;
    p.out = y;
    p.z = z;
    p.offsets = expert_offsets;
    p.rows = s.rows;
    p.d_in = s.d_in;
    p.d_out = s.d_out;
    p.E = s.E;
    p.act = s.act;
    p.starve = (s.flags & MOE_FLAG_TEST_TIMEOUT) != 0;
    p.status = status;
    return launch_linear(LIN_FWD, p, reinterpret_cast<cudaStream_t>(stream));
}

int moe_linear_backward(const moe_linear_t *shape, const moe_bf16_t *x,
                        const int32_t *expert_offsets, const moe_bf16_t *W, const moe_bf16_t *z,
                        const moe_bf16_t *dy, moe_bf16_t *dx, moe_bf16_t *dW, float *dbias,
                        uint32_t *status, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    int rc = check_linear(shape);
    if (rc)
        return rc;
    const moe_linear_t &s = *shape;
    if (!expert_offsets && s.E != 1)
        return MOE_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || !aligned(z, 16) || !aligned(dy, 16) ||
        !aligned(dx, 16) || !aligned(dW, 16) || !aligned(dbias, 16) || !aligned(expert_offsets, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (s.rows == 0) {   // no rows: the sums over them are zero
        if (dW && cudaMemsetAsync(dW, 0, (size_t)s.E * s.d_out * s.d_in * 2, st) != cudaSuccess)
            return MOE_ERR_CUDA;
        if (dbias && cudaMemsetAsync(dbias, 0, (size_t)s.E * s.d_out * 4, st) != cudaSuccess)
            return MOE_ERR_CUDA;
        return MOE_OK;
    }
    if (!dy || (!dx && !dW && !dbias) || (dx && !W) || (dW && !x) ||
        (s.act != MOE_ACT_NONE && !z))
        return MOE_ERR_INVALID_ARG;
    const LinWs L = lin_ws(s);
    if (!ws || !aligned(ws, 256) || ws_bytes < L.total)
        return MOE_ERR_WORKSPACE;
    char *w = static_cast<char *>(ws);
    float *part = reinterpret_cast<float *>(w + L.part);
    uint16_t *dz = reinterpret_cast<uint16_t *>(w + L.dz);
    if (s.act != MOE_ACT_NONE || dbias) {
        if ((rc = elementwise_backward(s, dy, z, dz, dbias ? part : nullptr, expert_offsets, status,
                                       st)))
            return rc;
    }
    if (dbias) {
        launch_pdl_ex(k_linear_db, dim3((s.d_out + 31) / 32, s.E), dim3(256), 0, st, part, dbias,
                      expert_offsets, s.E, s.rows, s.d_out);
        if ((rc = launched()))
            return rc;
    }
    LinArgs p;
    std::memset(&p, 0, sizeof p);
    p.x = x;
    p.W = W;
    p.dz = s.act != MOE_ACT_NONE ? dz : dy;
    p.offsets = expert_offsets;
    p.rows = s.rows;
    p.d_in = s.d_in;
    p.d_out = s.d_out;
    p.E = s.E;
    p.starve = (s.flags & MOE_FLAG_TEST_TIMEOUT) != 0;
    p.status = status;
    // The bias sums, dx and dW run beside each other (4096 x 2048 -> 4096: dx and dW are 128
    // tiles each for 74 pairs of SMs, and two rounds of one leave 20 pairs to the other). That
    // is sound because
    //  - the first kernel after dz (the bias sums; without them dx, or dW alone, which is then
    //    not late) lets its successor start only after its own wait: by then dz has
    //    completed, and so has whatever ran before the call;
    //  - a late product lets its successor start at once, waits for nothing, reads nothing
    //    that a kernel of this call behind dz writes, and writes nothing that one reads
    //    (dx, dW, the parts of dW and the bias sums' parts are apart);
    //  - it waits for its predecessor before each of its ways out, so that whatever waits for
    //    the call's last kernel has waited for all of them.
    // A late product thus reads dz, and what came before the call, without a wait of its own:
    // what it rests on is that their kernels had completed, their writes with them, before
    // it was started.
    p.late = dbias != nullptr;
    if (dx) {
        p.out = dx;
        if ((rc = launch_linear(LIN_DX, p, st)))
            return rc;
        p.late = true;
    }
    if (dW) {
        p.out = dW;
        p.splits = L.splits;
        p.part = reinterpret_cast<float *>(w + L.dw_part);
        if ((rc = launch_linear(LIN_DW, p, st)))
            return rc;
    }
    return MOE_OK;
}

} // extern "C"
