// linear.cu -- linear products with bias, activation and residual, dense or
// grouped by expert with ragged sizes, and their gradients:
//   forward   y = act(x W_e^T + b_e) + residual       (z = x W_e^T + b_e kept on request)
//   backward  dz = dy act'(z), dx = dz W_e, dW_e = dz^T x, db_e = sum_r dz_r
// ("Expert FFN" and "Sparse MoE Block" on "MoE Model Architectures" with another
// activation, with biases, or alone.)
//
// This file holds the entry points, the elementwise pass of the backward and
// the product kernels.
#include <algorithm>
#include <cstring>

#include "act.cuh"
#include "common.cuh"
#include "groups.cuh"
#include "internal.h"

namespace moe {

namespace {

// ---------------------------------------------------------------- elementwise backward
// dz = dy act'(z) in bf16 and the column sums of the unrounded dz over items of
// kDzRows rows of one group. Bound by HBM: dy and z read, dz written once. A
// CTA of 8 warps covers 256 columns (a lane 8 of them, 16-byte vectors) and
// its warps take the item's rows in turn; their sums meet in shared memory in
// warp order, so db repeats bit for bit.
constexpr int kDzRows = 128;
constexpr int kDzCols = 256;

template <int ACT>
__global__ void __launch_bounds__(256)
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
        for (int r = r0 + warp; r < r1; r += 8) {
            const long long at = (long long)r * nv + col / 8;
            const uint4 g = ld_stream_v4(dy + at);
            const uint32_t gw[4] = {g.x, g.y, g.z, g.w};
            uint32_t ow[4];
            if (ACT != MOE_ACT_NONE) {
                const uint4 zz = ld_stream_v4(z + at);
                const uint32_t zw[4] = {zz.x, zz.y, zz.z, zz.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float a = bf16lo(gw[q]) * act_grad_f<ACT>(bf16lo(zw[q]));
                    const float b = bf16hi(gw[q]) * act_grad_f<ACT>(bf16hi(zw[q]));
                    sum[2 * q] += a;
                    sum[2 * q + 1] += b;
                    ow[q] = pack_bf16x2(a, b);
                }
                dz[at] = make_uint4(ow[0], ow[1], ow[2], ow[3]);
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    sum[2 * q] += bf16lo(gw[q]);
                    sum[2 * q + 1] += bf16hi(gw[q]);
                }
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
    for (int i = G.first[e]; i < G.first[e + 1]; ++i)
        s += part[(long long)i * d_out + c];
    db[(long long)e * d_out + c] = s;
}

// ---------------------------------------------------------------- products (CUDA cores)
// out[c, m] = sum_k A[m, k] B[c, k], 64 x 64 tiles. LIN_FWD: m = d_out, c = rows,
// k = d_in. LIN_DX: m = d_in, c = rows, k = d_out. LIN_DW: m = d_in, c = d_out,
// k = the group's rows.
enum LinMode { LIN_FWD = 0, LIN_DX = 1, LIN_DW = 2 };

struct LinArgs {
    const uint16_t *x, *W, *dz;
    const float *bias;
    const uint16_t *residual;
    uint16_t *out, *z;
    const int32_t *offsets;
    int rows, d_in, d_out, E;
    uint32_t *status;
};

constexpr int kT = 64, kTk = 16;

template <int MODE, int ACT>
__global__ void __launch_bounds__(256) k_linear_simt(const LinArgs p)
{
    __shared__ GroupSmem G;
    __shared__ float sa[kTk][kT + 1], sb[kTk][kT + 1];
    build_groups(G, p.offsets, p.E, p.rows, kT, p.status);
    int e, r0, r1;
    if (MODE == LIN_DW) {
        e = blockIdx.z;
        r0 = G.row0[e];
        r1 = G.row0[e + 1];
    } else {
        const int item = blockIdx.y;
        if (item >= G.first[p.E])
            return;
        e = item_group(G, p.E, item);
        r0 = G.row0[e] + (item - G.first[e]) * kT;
        r1 = min(r0 + kT, G.row0[e + 1]);
    }
    const int M = MODE == LIN_FWD ? p.d_out : p.d_in;
    const int m0 = blockIdx.x * kT;
    const int c0 = MODE == LIN_DW ? blockIdx.y * kT : r0;
    const int c1 = MODE == LIN_DW ? min(c0 + kT, p.d_out) : r1;
    const int K = MODE == LIN_FWD ? p.d_in : MODE == LIN_DX ? p.d_out : r1 - r0;
    const uint16_t *We = p.W + (MODE == LIN_DW ? 0 : (long long)e * p.d_out * p.d_in);
    const int tm = threadIdx.x & 15, tc = threadIdx.x >> 4;
    float acc[4][4] = {};
    auto bf = [](uint16_t v) { return __uint_as_float((uint32_t)v << 16); };
    for (int k0 = 0; k0 < K; k0 += kTk) {
        __syncthreads();
        for (int i = threadIdx.x; i < kTk * kT; i += 256) {
            int kk, mm;
            if (MODE == LIN_FWD)
                kk = i % kTk, mm = i / kTk;
            else
                kk = i / kT, mm = i % kT;
            float a = 0.f, b = 0.f;
            const int k = k0 + kk, m = m0 + mm;
            if (k < K && m < M)
                a = MODE == LIN_FWD  ? bf(We[(long long)m * p.d_in + k])
                    : MODE == LIN_DX ? bf(We[(long long)k * p.d_in + m])
                                     : bf(p.x[(long long)(r0 + k) * p.d_in + m]);
            sa[kk][mm] = a;
            int kb, cc;
            if (MODE == LIN_DW)
                kb = i / kT, cc = i % kT;
            else
                kb = i % kTk, cc = i / kTk;
            if (k0 + kb < K && c0 + cc < c1)
                b = MODE == LIN_FWD  ? bf(p.x[(long long)(c0 + cc) * p.d_in + k0 + kb])
                    : MODE == LIN_DX ? bf(p.dz[(long long)(c0 + cc) * p.d_out + k0 + kb])
                                     : bf(p.dz[(long long)(r0 + k0 + kb) * p.d_out + c0 + cc]);
            sb[kb][cc] = b;
        }
        __syncthreads();
#pragma unroll
        for (int kk = 0; kk < kTk; ++kk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sa[kk][tm + 16 * i], sb[kk][tc + 16 * j], acc[i][j]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + tm + 16 * i, c = c0 + tc + 16 * j;
            if (m >= M || c >= c1)
                continue;
            const long long at = (MODE == LIN_DW ? (long long)e * p.d_out * p.d_in : 0) +
                                 (long long)c * M + m;
            float v = acc[i][j];
            if (MODE == LIN_FWD) {
                if (p.bias)
                    v += p.bias[(long long)e * p.d_out + m];
                if (p.z)
                    p.z[at] = (uint16_t)pack_bf16x2(v, 0.f);
                v = act_f<ACT>(v);
                if (p.residual)
                    v += bf(p.residual[at]);
            }
            p.out[at] = (uint16_t)pack_bf16x2(v, 0.f);
        }
}

template <int MODE, int ACT>
int launch_product(const LinArgs &p, cudaStream_t st)
{
    const int M = MODE == LIN_FWD ? p.d_out : p.d_in;
    const dim3 grid((M + kT - 1) / kT,
                    MODE == LIN_DW ? (p.d_out + kT - 1) / kT
                                   : (p.rows + kT - 1) / kT + std::min(p.E, p.rows),
                    MODE == LIN_DW ? p.E : 1);
    k_linear_simt<MODE, ACT><<<grid, 256, 0, st>>>(p);
    return launched();
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
    size_t dz, part, total;
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

int forward_product(int act, const LinArgs &p, cudaStream_t st)
{
    switch (act) {
    case MOE_ACT_NONE: return launch_product<LIN_FWD, MOE_ACT_NONE>(p, st);
    case MOE_ACT_RELU: return launch_product<LIN_FWD, MOE_ACT_RELU>(p, st);
    case MOE_ACT_GELU: return launch_product<LIN_FWD, MOE_ACT_GELU>(p, st);
    case MOE_ACT_GELU_TANH: return launch_product<LIN_FWD, MOE_ACT_GELU_TANH>(p, st);
    default: return launch_product<LIN_FWD, MOE_ACT_SILU>(p, st);
    }
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
    p.status = status;
    return forward_product(s.act, p, reinterpret_cast<cudaStream_t>(stream));
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
        if ((rc = launch_product<LIN_DX, MOE_ACT_NONE>(p, st)))
            return rc;
    }
    if (dW) {
        p.out = dW;
        if ((rc = launch_product<LIN_DW, MOE_ACT_NONE>(p, st)))
            return rc;
    }
    return MOE_OK;
}

} // extern "C"
