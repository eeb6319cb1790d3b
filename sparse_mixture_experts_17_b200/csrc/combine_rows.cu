// combine_rows.cu -- combine of bf16 expert rows into token order, and its
// gradient ("Sparse MoE Block" on "MoE Model Architectures": scale by the
// routing weight, index_add into token order).
//
//   out[t]       = residual[t] + sum_j w[t,j] y[slot[t,j]]
//   dy[slot[t,j]] = w[t,j] dout[t],   dw[t,j] = <dout[t], y[slot[t,j]]>
//
// Bound by HBM: each kept row is read (and in the backward written) once. A
// token is owned by `lanes` consecutive threads (d / 8 rounded up to a power of
// two, 16 to 256; see lanes_for), each moving 16-byte vectors of 8 columns, all k
// rows' loads of a vector in flight together (four at a time in the backward of
// k = 8). Sums run in fp32 in slot order, so results repeat bit for bit; no atomics.
// Measured: 16384 x 4096, k = 2, with the residual 82 us (537 MB, 6.5 TB/s); backward
// of 4096 x 2048, k = 8, 60% kept, 37 us (179 MB, 4.9 TB/s: latency of the scattered rows).
#include <algorithm>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8])
{
    f[0] = bf16lo(v.x), f[1] = bf16hi(v.x), f[2] = bf16lo(v.y), f[3] = bf16hi(v.y);
    f[4] = bf16lo(v.z), f[5] = bf16hi(v.z), f[6] = bf16lo(v.w), f[7] = bf16hi(v.w);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8])
{
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// The k slots and weights of token t; slots past T*k count as dropped.
template <int K>
__device__ __forceinline__ void load_slots(const int32_t *slot_pos, const float *w, long long t,
                                           int k, long long n, bool flagger, uint32_t *status,
                                           int (&ps)[K], float (&ws)[K])
{
#pragma unroll
    for (int j = 0; j < K; ++j) {
        ps[j] = -1;
        ws[j] = 0.f;
        if (j < k) {
            const int p = slot_pos[t * k + j];
            ws[j] = w ? w[t * k + j] : 1.f;
            if (p >= n) {
                if (flagger)
                    flag_status(status, MOE_ERR_CHECK);
            } else {
                ps[j] = p;
            }
        }
    }
}

template <int K>
__global__ void __launch_bounds__(kThreads)
    k_combine_rows(const uint4 *__restrict__ y, const int32_t *__restrict__ slot_pos,
                   const float *__restrict__ w, const uint4 *residual, uint4 *out, int T, int k,
                   int nv, int lanes, uint32_t *status)
{
    const int lane = threadIdx.x & (lanes - 1);
    const long long t = (long long)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    pdl_wait();
    pdl_trigger();
    if (t >= T)
        return;
    int ps[K];
    float ws[K];
    load_slots<K>(slot_pos, w, t, k, (long long)T * k, lane == 0, status, ps, ws);
    for (int c = lane; c < nv; c += lanes) {
        uint4 v[K];
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (ps[j] >= 0)
                v[j] = ld_stream_v4(y + (long long)ps[j] * nv + c);
        float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (residual) {
            const uint4 r = residual[t * nv + c];
            unpack8(r, acc);
        }
#pragma unroll
        for (int j = 0; j < K; ++j)
            if (ps[j] >= 0) {
                float f[8];
                unpack8(v[j], f);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[i] = fmaf(ws[j], f[i], acc[i]);
            }
        out[t * nv + c] = pack8(acc);
    }
}

template <int K>
__global__ void __launch_bounds__(kThreads, K == 8 ? 4 : 1)
    k_combine_rows_bwd(const uint4 *__restrict__ dout, const uint4 *__restrict__ y,
                       const int32_t *__restrict__ slot_pos, const float *__restrict__ w, uint4 *dy,
                       float *dw, int T, int k, int nv, int lanes, uint32_t *status)
{
    __shared__ float red[kThreads / 32][K];
    const int lane = threadIdx.x & (lanes - 1);
    const long long t = (long long)blockIdx.x * (kThreads / lanes) + threadIdx.x / lanes;
    pdl_wait();
    pdl_trigger();
    const bool live = t < T;   // every thread reaches the barrier of the dot products
    int ps[K];
    float ws[K], dot[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
        ps[j] = -1;
        ws[j] = dot[j] = 0.f;
    }
    if (live) {
        load_slots<K>(slot_pos, w, t, k, (long long)T * k, lane == 0, status, ps, ws);
        // 4 rows in flight at a time, and registers for 4 CTAs an SM (k = 8, 4096 x 2048:
        // 53 us against 55 with all 8 rows and 2 CTAs; 16384 x 512: 57 against 70)
        constexpr int KC = K < 4 ? K : 4;
        for (int c = lane; c < nv; c += lanes) {
            uint4 v[KC];
            float g[8];
#pragma unroll
            for (int j0 = 0; j0 < K; j0 += KC) {
                if (dw) {
#pragma unroll
                    for (int i = 0; i < KC; ++i)
                        if (ps[j0 + i] >= 0)
                            v[i] = ld_stream_v4(y + (long long)ps[j0 + i] * nv + c);
                }
                if (j0 == 0)
                    unpack8(dout[t * nv + c], g);
#pragma unroll
                for (int i = 0; i < KC; ++i) {
                    const int j = j0 + i;
                    if (ps[j] < 0)
                        continue;
                    if (dy) {
                        float o[8];
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            o[q] = ws[j] * g[q];
                        dy[(long long)ps[j] * nv + c] = pack8(o);
                    }
                    if (dw) {
                        float f[8];
                        unpack8(v[i], f);
#pragma unroll
                        for (int q = 0; q < 8; ++q)
                            dot[j] = fmaf(g[q], f[q], dot[j]);
                    }
                }
            }
        }
    }
    if (!dw)
        return;
    // tree over the token's threads: within a half or whole warp by shuffles,
    // then across the token's warps in warp order
    const int span = min(lanes, 32);
#pragma unroll
    for (int j = 0; j < K; ++j)
        for (int off = span >> 1; off > 0; off >>= 1)
            dot[j] += __shfl_xor_sync(kFullMask, dot[j], off);
    if (lanes <= 32) {
        if (live && lane == 0)
#pragma unroll
            for (int j = 0; j < K; ++j)
                if (j < k)
                    dw[t * k + j] = dot[j];
        return;
    }
    const int warp = threadIdx.x >> 5, per = lanes >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int j = 0; j < K; ++j)
            red[warp][j] = dot[j];
    __syncthreads();
    if (live && lane < k) {
        float s = 0.f;
        for (int i = 0; i < per; ++i)
            s += red[warp / per * per + i][lane];
        dw[t * k + lane] = s;
    }
}

// Threads of a token. Many tokens: 64, whose warps of different tokens overlap
// their loads, stores and sums (backward of 4096 x 2048, k = 8, kept rows 100%:
// 60 us against 75 with 256; 16384 x 512: 74 against 220). Few tokens: up to 256
// as long as the GPU is not full (one token, d = 7168, k = 8: 12 us against 25).
int lanes_for(int nv, int T)
{
    int l = 16;
    while (l < nv && l < kThreads)
        l <<= 1;
    while (l > 64 && (long long)T * (l / 2) >= 1024LL * num_sms())
        l >>= 1;
    return l;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Rows of any width that a linear product writes: the fields that the combine does not use
// may hold anything, d is its own rule.
int check_rows_shape(const moe_shape_t *s)
{
    if (!s || s->T < 0 || s->T > (1 << 24) || s->E < 1 || s->E > MOE_MAX_E || s->k < 1 ||
        s->k > std::min(s->E, MOE_MAX_K) || s->d < 8 || s->d > 65536 || s->d % 8 != 0)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

template <int K>
int launch_fwd(const moe_shape_t &s, const uint16_t *y, const int32_t *slot, const float *w,
               const uint16_t *res, uint16_t *out, uint32_t *status, cudaStream_t st)
{
    const int nv = s.d / 8, lanes = lanes_for(nv, s.T), per = kThreads / lanes;
    launch_pdl_ex(k_combine_rows<K>, dim3((s.T + per - 1) / per), dim3(kThreads), 0, st,
                  reinterpret_cast<const uint4 *>(y), slot, w, reinterpret_cast<const uint4 *>(res),
                  reinterpret_cast<uint4 *>(out), s.T, s.k, nv, lanes, status);
    return launched();
}

template <int K>
int launch_bwd(const moe_shape_t &s, const uint16_t *dout, const uint16_t *y, const int32_t *slot,
               const float *w, uint16_t *dy, float *dw, uint32_t *status, cudaStream_t st)
{
    const int nv = s.d / 8, lanes = lanes_for(nv, s.T), per = kThreads / lanes;
    launch_pdl_ex(k_combine_rows_bwd<K>, dim3((s.T + per - 1) / per), dim3(kThreads), 0, st,
                  reinterpret_cast<const uint4 *>(dout), reinterpret_cast<const uint4 *>(y), slot, w,
                  reinterpret_cast<uint4 *>(dy), dw, s.T, s.k, nv, lanes, status);
    return launched();
}

} // namespace
} // namespace moe

using namespace moe;

extern "C" {

int moe_combine_rows(const moe_shape_t *shape, const moe_bf16_t *y_perm, const int32_t *slot_pos,
                     const float *topk_w, const moe_bf16_t *residual, moe_bf16_t *out,
                     uint32_t *status, moe_stream_t stream)
{
    const int rc = check_rows_shape(shape);
    if (rc)
        return rc;
    if (shape->T == 0)
        return MOE_OK;
    if (!y_perm || !slot_pos || !out || !aligned(y_perm, 16) || !aligned(out, 16) ||
        !aligned(slot_pos, 4) || !aligned(topk_w, 4) || !aligned(residual, 16))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    // the slot loop is unrolled: the smallest of 1, 2, 4, 8, 16 that holds k
    const moe_shape_t &s = *shape;
    if (s.k == 1)
        return launch_fwd<1>(s, y_perm, slot_pos, topk_w, residual, out, status, st);
    if (s.k == 2)
        return launch_fwd<2>(s, y_perm, slot_pos, topk_w, residual, out, status, st);
    if (s.k <= 4)
        return launch_fwd<4>(s, y_perm, slot_pos, topk_w, residual, out, status, st);
    if (s.k <= 8)
        return launch_fwd<8>(s, y_perm, slot_pos, topk_w, residual, out, status, st);
    return launch_fwd<16>(s, y_perm, slot_pos, topk_w, residual, out, status, st);
}

int moe_combine_rows_backward(const moe_shape_t *shape, const moe_bf16_t *dout,
                              const moe_bf16_t *y_perm, const int32_t *slot_pos,
                              const float *topk_w, moe_bf16_t *dy_perm, float *dtopk_w,
                              uint32_t *status, moe_stream_t stream)
{
    const int rc = check_rows_shape(shape);
    if (rc)
        return rc;
    if (shape->T == 0)
        return MOE_OK;
    if (!dout || !slot_pos || (!dy_perm && !dtopk_w) || (dtopk_w && !y_perm) ||
        !aligned(dout, 16) || !aligned(y_perm, 16) || !aligned(dy_perm, 16) ||
        !aligned(slot_pos, 4) || !aligned(topk_w, 4) || !aligned(dtopk_w, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const moe_shape_t &s = *shape;
    if (s.k == 1)
        return launch_bwd<1>(s, dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, status, st);
    if (s.k == 2)
        return launch_bwd<2>(s, dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, status, st);
    if (s.k <= 4)
        return launch_bwd<4>(s, dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, status, st);
    if (s.k <= 8)
        return launch_bwd<8>(s, dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, status, st);
    return launch_bwd<16>(s, dout, y_perm, slot_pos, topk_w, dy_perm, dtopk_w, status, st);
}

} // extern "C"
