// grad_clip.cu -- the global gradient norm over many tensors, and clipping:
//   norm = sqrt(sum g^2),  c = min(1, max_norm / (norm + 1e-6)),  out = c g.
//
// Bound by HBM: one read for the norm, and one read and write where something
// is scaled. The tensors of a launch travel in its parameters (no table in
// device memory, nothing to copy, safe to capture). Every tensor is cut into
// chunks of kChunkVecs 16-byte vectors; CTA c takes chunks c, c + G, ... of all
// tensors together and writes one fp64 partial sum, so the order of the sums
// depends on sizes, alignments and the SM count only. The scaling kernel adds the
// partials itself (every CTA the same way), which saves a launch, and walks
// the chunks backwards: the ones read last may still be in L2. Measured: 2.8 GB
// scaled into other buffers 1320 us (8.4 GB moved, 6.4 TB/s; the squares alone 430 us,
// 717 when a slow path indexed the vectors at run time and put them in local memory).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxTensors = 96;       // tensors of one launch (their parameters stay below 4 KB)
constexpr int kChunkVecs = 4096;      // 64 KB of a tensor: 16 vectors a thread
constexpr int kCtasPerSm = 8;
constexpr int kMaxCtas = MOE_GRAD_WS_BYTES / 8;       // an fp64 partial each

struct TensorList {
    const void *p[kMaxTensors];
    long long n[kMaxTensors];
    int first[kMaxTensors + 1];       // first chunk of each tensor
    unsigned bf16[(kMaxTensors + 31) / 32];
    int count;
};

struct OutList {
    void *p[kMaxTensors];
};

__device__ __forceinline__ int tensor_of(const TensorList &L, int chunk)
{
    int lo = 0, hi = L.count - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (L.first[mid] <= chunk)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A chunk of tensor i: its scalar head and tail (elements outside the 16-byte
// vectors) belong to the tensor's first and last chunk.
struct Chunk {
    const char *base;      // first vector of the tensor
    long long v0, v1;      // its vectors
    long long head, tail0, n;   // head elements [0, head) / tail elements [tail0, n), when this chunk has them
    bool bf16;
    int tensor;
};

__device__ __forceinline__ Chunk chunk_of(const TensorList &L, int chunk)
{
    Chunk c;
    const int i = tensor_of(L, chunk);
    c.tensor = i;
    c.bf16 = (L.bf16[i >> 5] >> (i & 31)) & 1u;
    const int es = c.bf16 ? 2 : 4, per = 16 / es;
    const uintptr_t p = reinterpret_cast<uintptr_t>(L.p[i]);
    c.n = L.n[i];
    const long long head = min((long long)((16 - (p & 15)) & 15) / es, c.n);
    const long long nv = (c.n - head) / per;
    c.base = reinterpret_cast<const char *>(p + head * es);
    const int j = chunk - L.first[i];
    c.v0 = (long long)j * kChunkVecs;
    c.v1 = min(c.v0 + kChunkVecs, nv);
    c.head = j == 0 ? head : 0;
    const bool last = chunk + 1 == L.first[i + 1];
    c.tail0 = last ? head + nv * per : c.n;
    return c;
}

__device__ __forceinline__ float elem(const void *p, long long i, bool bf16)
{
    return bf16 ? __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16)
                : static_cast<const float *>(p)[i];
}

__device__ __forceinline__ double sq64(uint32_t bits)
{
    const double v = (double)__uint_as_float(bits);
    return v * v;
}

// Sum of squares of 32 elements held in registers. fp32 has 24 bits and 32
// terms of one sign, so the sum is good to 2^-20; where it leaves [2^-90, inf)
// (an overflow, or terms that may have been lost below 2^-126) the squares are
// formed in fp64. All-zero runs stay on the fast side.
template <int NV, bool BF16>
__device__ __forceinline__ double run_sum(const uint4 (&v)[NV])
{
    float s = 0.f;
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            any |= w[q];
            if (BF16) {
                s = fmaf(bf16lo(w[q]), bf16lo(w[q]), s);
                s = fmaf(bf16hi(w[q]), bf16hi(w[q]), s);
            } else {
                const float f = __uint_as_float(w[q]);
                s = fmaf(f, f, s);
            }
        }
    }
    if (s >= 8.0779356694631609e-28f && s <= 3.402823466e38f)   // 2^-90
        return (double)s;
    if (any == 0)
        return 0.0;
    double d = 0.0;
#pragma unroll   // a loop would index v at run time and put it in local memory, on the fast side too
    for (int u = 0; u < NV; ++u) {
        const uint32_t w[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (BF16)
                d += sq64(w[q] << 16) + sq64(w[q] & 0xffff0000u);
            else
                d += sq64(w[q]);
        }
    }
    return d;
}

template <bool BF16>
__device__ __forceinline__ double chunk_sum(const Chunk &c)
{
    constexpr int NV = BF16 ? 4 : 8;   // 32 elements a run
    const uint4 *p = reinterpret_cast<const uint4 *>(c.base);
    double acc = 0.0;
    for (long long v = c.v0 + threadIdx.x; v < c.v1; v += (long long)NV * kThreads) {
        uint4 r[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const long long at = v + (long long)u * kThreads;
            r[u] = at < c.v1 ? ld_stream_v4(p + at) : make_uint4(0, 0, 0, 0);
        }
        acc += run_sum<NV, BF16>(r);
    }
    return acc;
}

// Sum over the block in a fixed tree; the result is in every thread.
__device__ __forceinline__ double block_sum(double v)
{
    __shared__ double s[kThreads / 32];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v += __shfl_xor_sync(kFullMask, v, off);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        s[threadIdx.x >> 5] = v;
    __syncthreads();
    double t = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        t += s[w];
    return t;
}

// part[CTA] (+)= the CTA's share of the sum of squares.
__global__ void __launch_bounds__(kThreads)
    k_grad_sq(const __grid_constant__ TensorList L, int accumulate, double *part)
{
    pdl_wait();
    pdl_trigger();
    double acc = 0.0;
    const int chunks = L.first[L.count];
    for (int ch = blockIdx.x; ch < chunks; ch += gridDim.x) {
        const Chunk c = chunk_of(L, ch);
        acc += c.bf16 ? chunk_sum<true>(c) : chunk_sum<false>(c);
        const void *p = L.p[c.tensor];
        for (long long i = threadIdx.x; i < c.head; i += kThreads) {
            const double f = (double)elem(p, i, c.bf16);
            acc += f * f;
        }
        for (long long i = c.tail0 + threadIdx.x; i < c.n; i += kThreads) {
            const double f = (double)elem(p, i, c.bf16);
            acc += f * f;
        }
    }
    const double total = block_sum(acc);
    if (threadIdx.x == 0)
        part[blockIdx.x] = accumulate ? part[blockIdx.x] + total : total;
}

__device__ __forceinline__ float total_norm(const double *part, int nparts)
{
    double acc = 0.0;
    for (int i = threadIdx.x; i < nparts; i += kThreads)
        acc += part[i];
    return (float)sqrt(block_sum(acc));
}

__global__ void __launch_bounds__(kThreads)
    k_grad_norm(const double *part, int nparts, float *norm, uint32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const float n = total_norm(part, nparts);
    if (threadIdx.x == 0) {
        norm[0] = n;
        if (!isfinite(n))
            flag_status(status, MOE_ERR_NONFINITE);
    }
}

template <bool BF16>
__device__ __forceinline__ uint4 scale_vec(uint4 v, float c)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q)
        w[q] = BF16 ? pack_bf16x2(c * bf16lo(w[q]), c * bf16hi(w[q]))
                    : __float_as_uint(c * __uint_as_float(w[q]));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void scale_elem(const void *p, void *o, long long i, bool bf16, float c)
{
    // a factor of 1 copies the bits (as integers: a product would change a NaN's payload)
    if (bf16) {
        uint16_t v = static_cast<const uint16_t *>(p)[i];
        if (c != 1.f)
            v = (uint16_t)pack_bf16x2(c * __uint_as_float((uint32_t)v << 16), 0.f);
        static_cast<uint16_t *>(o)[i] = v;
    } else {
        uint32_t v = static_cast<const uint32_t *>(p)[i];
        if (c != 1.f)
            v = __float_as_uint(c * __uint_as_float(v));
        static_cast<uint32_t *>(o)[i] = v;
    }
}

__device__ __forceinline__ void st_stream_v4(uint4 *p, uint4 v)
{
    asm volatile("st.global.cs.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

template <bool BF16>
__device__ __forceinline__ void chunk_scale(const Chunk &c, void *out, const void *in, float f)
{
    constexpr int NV = 8;
    const uint4 *p = reinterpret_cast<const uint4 *>(c.base);
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<char *>(out) +
                                         (c.base - static_cast<const char *>(in)));
    for (long long v = c.v0 + threadIdx.x; v < c.v1; v += (long long)NV * kThreads) {
        uint4 r[NV];
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const long long at = v + (long long)u * kThreads;
            if (at < c.v1)
                r[u] = p[at];
        }
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            const long long at = v + (long long)u * kThreads;
            if (at < c.v1)
                st_stream_v4(o + at, f == 1.f ? r[u] : scale_vec<BF16>(r[u], f));
        }
    }
}

// out = c g for the tensors of one launch; the first launch also writes the norm.
__global__ void __launch_bounds__(kThreads)
    k_grad_scale(const __grid_constant__ TensorList L, const __grid_constant__ OutList O,
                 const double *part, int nparts, float max_norm, float *norm, int write_norm,
                 uint32_t *status)
{
    pdl_wait();
    pdl_trigger();
    const float n = total_norm(part, nparts);
    const bool finite = isfinite(n);
    if (write_norm && blockIdx.x == 0 && threadIdx.x == 0) {
        norm[0] = n;
        if (!finite)
            flag_status(status, MOE_ERR_NONFINITE);
    }
    const float c = finite ? fminf(1.f, max_norm / (n + 1e-6f)) : 1.f;
    const int chunks = L.first[L.count];
    for (int ch = chunks - 1 - (int)blockIdx.x; ch >= 0; ch -= gridDim.x) {
        const Chunk k = chunk_of(L, ch);
        const void *p = L.p[k.tensor];
        void *o = O.p[k.tensor];
        if (c == 1.f && p == o)
            continue;
        if (((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0) {
            if (k.bf16)
                chunk_scale<true>(k, o, p, c);
            else
                chunk_scale<false>(k, o, p, c);
        } else {   // the two are not 16-byte aligned together: element by element
            const int es = k.bf16 ? 2 : 4, per = 16 / es;
            const long long e0 = (k.base - static_cast<const char *>(p)) / es;
            for (long long i = e0 + k.v0 * per + threadIdx.x; i < e0 + k.v1 * per; i += kThreads)
                scale_elem(p, o, i, k.bf16, c);
        }
        for (long long i = threadIdx.x; i < k.head; i += kThreads)
            scale_elem(p, o, i, k.bf16, c);
        for (long long i = k.tail0 + threadIdx.x; i < k.n; i += kThreads)
            scale_elem(p, o, i, k.bf16, c);
    }
}

// ---------------------------------------------------------------- host side

constexpr long long kMaxNumel = 1LL << 40;

int type_size(int t) { return t == MOE_TYPE_BF16 ? 2 : 4; }

int check_list(int n, const void *const *p, const int64_t *numel, const int32_t *types)
{
    if (n < 0 || n > (1 << 20) || (n > 0 && (!p || !numel || !types)))
        return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < n; ++i) {
        if (types[i] != MOE_TYPE_F32 && types[i] != MOE_TYPE_BF16)
            return MOE_ERR_INVALID_ARG;
        if (numel[i] < 0 || numel[i] > kMaxNumel)
            return MOE_ERR_INVALID_ARG;
        if (numel[i] > 0 &&
            (!p[i] || reinterpret_cast<uintptr_t>(p[i]) % (unsigned)type_size(types[i])))
            return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

struct Range {
    uintptr_t a, b;
    bool operator<(const Range &o) const { return a < o.a; }
};

// MOE_OK when no two of the tensors overlap, outs[i] == grads[i] aside.
int check_overlap(int n, const void *const *grads, void *const *outs, const int64_t *numel,
                  const int32_t *types)
{
    constexpr int kLocal = 256;
    Range local[kLocal];
    Range *r = 2LL * n <= kLocal ? local : new (std::nothrow) Range[2 * (size_t)n];
    if (!r)
        return MOE_ERR_UNSUPPORTED;
    size_t m = 0;
    for (int i = 0; i < n; ++i) {
        if (numel[i] == 0)
            continue;
        const uintptr_t bytes = (uintptr_t)numel[i] * type_size(types[i]);
        const uintptr_t g = reinterpret_cast<uintptr_t>(grads[i]);
        const uintptr_t o = reinterpret_cast<uintptr_t>(outs[i]);
        r[m++] = {g, g + bytes};
        if (o != g)
            r[m++] = {o, o + bytes};
    }
    std::sort(r, r + m);
    int rc = MOE_OK;
    for (size_t i = 1; i < m; ++i)
        if (r[i].a < r[i - 1].b)
            rc = MOE_ERR_INVALID_ARG;
    if (r != local)
        delete[] r;
    return rc;
}

int chunks_of(const void *p, int64_t n, int type)
{
    const int es = type_size(type), per = 16 / es;
    const long long head =
        std::min<long long>(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / es, n);
    const long long nv = (n - head) / per;
    return (int)std::max<long long>((nv + kChunkVecs - 1) / kChunkVecs, 1);
}

// The next launch's tensors, from *at on: at most kMaxTensors, and few enough
// chunks for an int.
void fill(TensorList &L, OutList *O, int &at, int n, const void *const *p, void *const *outs,
          const int64_t *numel, const int32_t *types)
{
    std::memset(&L, 0, sizeof L);
    long long chunks = 0;
    for (; at < n && L.count < kMaxTensors; ++at) {
        if (numel[at] == 0)
            continue;
        const int c = chunks_of(p[at], numel[at], types[at]);
        if (chunks + c > (1LL << 30))
            break;
        const int i = L.count++;
        L.p[i] = p[at];
        L.n[i] = numel[at];
        L.first[i] = (int)chunks;
        chunks += c;
        if (types[at] == MOE_TYPE_BF16)
            L.bf16[i >> 5] |= 1u << (i & 31);
        if (O)
            O->p[i] = outs[at];
        L.first[i + 1] = (int)chunks;
    }
}

int grid_for(const TensorList &L)
{
    return std::max(1, std::min(L.first[L.count], std::min(kCtasPerSm * num_sms(), kMaxCtas)));
}

// The partial sums of all tensors; *nparts of them.
int launch_squares(int n, const void *const *grads, const int64_t *numel, const int32_t *types,
                   double *part, int *nparts, cudaStream_t st)
{
    TensorList L;
    int at = 0;
    *nparts = 0;
    do {
        fill(L, nullptr, at, n, grads, nullptr, numel, types);
        const bool more = at < n;
        // several launches add into the same partials, so the first writes them all
        const int grid = *nparts ? *nparts
                         : more  ? std::min(kCtasPerSm * num_sms(), kMaxCtas)
                                 : grid_for(L);
        launch_pdl_ex(k_grad_sq, dim3(grid), dim3(kThreads), 0, st, L, *nparts ? 1 : 0, part);
        const int rc = launched();
        if (rc)
            return rc;
        *nparts = grid;
    } while (at < n);
    return MOE_OK;
}

int check_ws(const void *ws, size_t ws_bytes)
{
    return !ws || (reinterpret_cast<uintptr_t>(ws) & 255u) || ws_bytes < MOE_GRAD_WS_BYTES
               ? MOE_ERR_WORKSPACE
               : MOE_OK;
}

} // namespace
} // namespace moe

using namespace moe;

extern "C" {

int moe_grad_norm(int n, const void *const *grads, const int64_t *numel, const int32_t *types,
                  float *norm, uint32_t *status, void *ws, size_t ws_bytes, moe_stream_t stream)
{
    int rc = check_list(n, grads, numel, types);
    if (rc)
        return rc;
    if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u))
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_ws(ws, ws_bytes)))
        return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(ws);
    int nparts = 0;
    if ((rc = launch_squares(n, grads, numel, types, part, &nparts, st)))
        return rc;
    launch_pdl_ex(k_grad_norm, dim3(1), dim3(kThreads), 0, st, part, nparts, norm, status);
    return launched();
}

int moe_clip_grads(int n, const void *const *grads, void *const *outs, const int64_t *numel,
                   const int32_t *types, float max_norm, float *norm, uint32_t *status, void *ws,
                   size_t ws_bytes, moe_stream_t stream)
{
    int rc = check_list(n, grads, numel, types);
    if (rc)
        return rc;
    // in place: the gradients themselves, which the caller lets the call write
    if (!outs)
        outs = const_cast<void *const *>(grads);
    if ((rc = check_list(n, const_cast<const void *const *>(outs), numel, types)))
        return rc;
    if (!norm || (reinterpret_cast<uintptr_t>(norm) & 3u) || !(max_norm > 0.f))
        return MOE_ERR_INVALID_ARG;
    if ((rc = check_overlap(n, grads, outs, numel, types)))
        return rc;
    if ((rc = check_ws(ws, ws_bytes)))
        return rc;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    double *part = static_cast<double *>(ws);
    int nparts = 0;
    if ((rc = launch_squares(n, grads, numel, types, part, &nparts, st)))
        return rc;
    TensorList L;
    OutList O;
    int at = 0, first = 1;
    do {
        std::memset(&O, 0, sizeof O);
        fill(L, &O, at, n, grads, outs, numel, types);
        launch_pdl_ex(k_grad_scale, dim3(grid_for(L)), dim3(kThreads), 0, st, L, O, part, nparts,
                      max_norm, norm, first, status);
        if ((rc = launched()))
            return rc;
        first = 0;
    } while (at < n);
    return MOE_OK;
}

} // extern "C"
