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
// CTA of 8 warps covers 256 columns (a lane 8 of them, 16-byte vectors) and
// its warps take the item's rows in turn; their sums meet in shared memory in
// warp order, so db repeats bit for bit.
constexpr int kDzRows = 64;
constexpr int kDzCols = 256;
constexpr int kDzUnroll = 4;   // rows of a warp in flight

template <int ACT>
__global__ void __launch_bounds__(256, 4)
    k_linear_dz(const uint4 *__restrict__ dy, const uint4 *__restrict__ z, uint4 *dz, float *part,
                const int32_t *offsets, int E, int rows, int d_out, uint32_t *status)
{
    __shared__ GroupSmem G;
    __shared__ float red[8][kDzCols];
    pdl_wait();
    pdl_trigger();
    build_groups(G, offsets, E, rows, kDzRows, status);
    const int item = blockIdx.y;
    if (item >= G.first[E])
        return;
    const int e = item_group(G, E, item);
    const int r0 = G.row0[e] + (item - G.first[e]) * kDzRows;
    const int r1 = min(r0 + kDzRows, G.row0[e + 1]);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * kDzCols + lane * 8, nv = d_out / 8;
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (col < d_out) {
        const long long at0 = (long long)r0 * nv + col / 8;
        for (int r = warp; r < r1 - r0; r += 8 * kDzUnroll) {
            uint4 g[kDzUnroll], zz[kDzUnroll];
#pragma unroll
            for (int u = 0; u < kDzUnroll; ++u)
                if (r + 8 * u < r1 - r0) {
                    g[u] = ld_stream_v4(dy + at0 + (long long)(r + 8 * u) * nv);
                    if (ACT != MOE_ACT_NONE)
                        zz[u] = ld_stream_v4(z + at0 + (long long)(r + 8 * u) * nv);
                }
#pragma unroll
            for (int u = 0; u < kDzUnroll; ++u)
                if (r + 8 * u < r1 - r0) {
                    const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
                    const uint32_t zw[4] = {zz[u].x, zz[u].y, zz[u].z, zz[u].w};
                    uint32_t ow[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        float a = bf16lo(gw[q]), b = bf16hi(gw[q]);
                        if (ACT != MOE_ACT_NONE) {
                            a *= act_grad_f<ACT>(bf16lo(zw[q]));
                            b *= act_grad_f<ACT>(bf16hi(zw[q]));
                        }
                        sum[2 * q] += a;
                        sum[2 * q + 1] += b;
                        ow[q] = pack_bf16x2(a, b);
                    }
                    if (ACT != MOE_ACT_NONE)
                        dz[at0 + (long long)(r + 8 * u) * nv] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
                }
        }
    }
    if (!part)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        red[warp][lane * 8 + i] = sum[i];
    __syncthreads();
    const int c = blockIdx.x * kDzCols + threadIdx.x;
    if (c < d_out) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            s += red[w][threadIdx.x];
        part[(long long)item * d_out + c] = s;
    }
}

// db[e] = sum of the group's items in order (0 for an empty group).
__global__ void __launch_bounds__(256)
    k_linear_db(const float *__restrict__ part, float *db, const int32_t *offsets, int E, int rows,
                int d_out)
{
    __shared__ GroupSmem G;
    pdl_wait();
    pdl_trigger();
    build_groups(G, offsets, E, rows, kDzRows, nullptr);
    const int e = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d_out)
        return;
    float s = 0.f;
#pragma unroll 8
    for (int i = G.first[e]; i < G.first[e + 1]; ++i)
        s += part[(long long)i * d_out + c];
    db[(long long)e * d_out + c] = s;
}

// ---------------------------------------------------------------- host side

int check_linear(const moe_linear_t *s)
{
    if (!s)
        return MOE_ERR_INVALID_ARG;
    auto dim = [](int v) { return v >= 8 && v <= 65536 && v % 8 == 0; };
    if (s->rows < 0 || s->rows > (1 << 24) || s->E < 1 || s->E > MOE_MAX_E || !dim(s->d_in) ||
        !dim(s->d_out) || s->act < MOE_ACT_NONE || s->act > MOE_ACT_SILU || s->flags != 0)
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
    launch_pdl_ex(k_linear_dz<ACT>, dim3((s.d_out + kDzCols - 1) / kDzCols, (unsigned)dz_items(s)),
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
        launch_pdl_ex(k_linear_db, dim3((s.d_out + 255) / 256, s.E), dim3(256), 0, st, part, dbias,
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
    p.status = status;
    if (dx) {
        p.out = dx;
        if ((rc = launch_linear(LIN_DX, p, st)))
            return rc;
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
