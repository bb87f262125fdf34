// The global L2 norm of a list of gradient tensors, and the list scaled to a
// largest norm: what a training step does between the layer's backward pass
// and its optimizer.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / norm)
//
// Both are streams: the norm reads every gradient once, clipping reads and
// writes every one once more, so bytes over the HBM rate is the floor and a
// launch per tensor is what a list of many small tensors must not cost.  The
// tensors' addresses and sizes travel in the kernel's argument block (128
// tensors a launch, no copy to the device, so a captured graph holds them);
// blocks take fixed chunks of the list, whatever tensor they lie in.
//
// Squares and sums are taken in fp64: the square of an fp32 value is exact
// there and no gradient is too large or too small to be squared.  A sum of n
// squares is off by at most n 2^-53 of itself, so the norm by that and half a step
// of fp32.  Partial sums are stored per block and added in block order: no
// atomics, the same bits every time.
#include <float.h>
#include <math.h>

#include "common.h"

namespace moe {
namespace {

constexpr int kTensors = 128;                 // tensors of one launch
// One block's work item, of one tensor: the blocks at work together then read
// neighbouring 16 KB pieces.  (Of 16, 32, 64 and 128 KB, 16 was best for small
// lists, 6.1 against 7.4 us with 64 KB for 1 MB in all, and large ones differed
// by 1-2%.)
constexpr int kChunkBytes = 16 << 10;
// Blocks of one launch at most.  The norm of 5.6 GB: 910 us with 1024 (6.2 TB/s),
// 934 with 2048; scaling 1.07 GB: 380 us with 4096 (5.65 TB/s read and written; a
// large copy 5.0), 384 with 2048, 387 with 1024.
constexpr int kNormBlocks = 1024, kScaleBlocks = 4096;
// Up to this many partial sums every block of the scaling adds them itself, which
// saves a launch (1 MB in 4 tensors 10.3 us against 12.6, 128 tensors of 0.25 MB
// 23.4 against 24.5; 1024 sums in 4 launches 36.9 against 35.9).  With more, one
// block adds them for all: the blocks' reading grows with the square of the list
// (256 tensors of 1 MB, 2048 sums, 141 us against 138; 2560 tensors, 20480 sums,
// 2297 against 1523; 5120 tensors 6219 against 3062).
constexpr int kOwnSums = kNormBlocks;
constexpr uint64_t kBf16Flag = 1ull << 63;

// One launch's tensors: tensor i covers chunks first[i] .. first[i+1]-1.
struct GradTable {
    const void* in[kTensors];
    void* out[kTensors];
    uint64_t numel[kTensors];                 // bit 63: bf16
    uint32_t first[kTensors + 1];
    int n;
};

struct Chunk {
    int t;                                    // tensor
    bool bf16;
    uint64_t i0;                              // first element
    int len;                                  // elements
};
template <bool BACK>                          // a tensor's chunks from its last to its first
__device__ __forceinline__ Chunk chunk_of(const GradTable& g, uint32_t c) {
    int lo = 0, hi = g.n;                     // largest t with first[t] <= c
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (g.first[mid] <= c) lo = mid; else hi = mid;
    }
    Chunk k;
    k.t = lo;
    k.bf16 = (g.numel[lo] & kBf16Flag) != 0;
    const uint64_t n = g.numel[lo] & ~kBf16Flag;
    const int per = kChunkBytes / (k.bf16 ? 2 : 4);
    k.i0 = (uint64_t)(BACK ? g.first[lo + 1] - 1 - c : c - g.first[lo]) * per;
    MOE_DASSERT(g.first[lo] <= c && c < g.first[lo + 1] && k.i0 < n);
    k.len = (int)min((uint64_t)per, n - k.i0);
    return k;
}

// 16 bytes at an address aligned to an element only (tensors may be views of
// a flat buffer).
typedef unsigned int u32x4_2_t __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned int u32x4_4_t __attribute__((ext_vector_type(4), aligned(4)));
template <typename T> struct Packed;
template <> struct Packed<bf16_t> { typedef u32x4_2_t type; };
template <> struct Packed<float> { typedef u32x4_4_t type; };

__device__ __forceinline__ double sq(double s, float v) {
    const double d = (double)v;
    return fma(d, d, s);
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* __restrict__ p, int len) {
    typedef typename Packed<T>::type P;
    constexpr int V = Vec16<T>::N, UN = 4;
    const int nvec = len / V;
    double s[2] = {0.0, 0.0};
    int v = threadIdx.x;
    for (; v + 256 * (UN - 1) < nvec; v += 256 * UN) {
        u32x4_t raw[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) raw[u] = *reinterpret_cast<const P*>(p + (v + 256 * u) * V);
#pragma unroll
        for (int u = 0; u < UN; ++u) {
            float o[V];
            unpack16<T>(raw[u], o);
#pragma unroll
            for (int q = 0; q < V; ++q) s[q & 1] = sq(s[q & 1], o[q]);
        }
    }
    for (; v < nvec; v += 256) {
        float o[V];
        unpack16<T>(*reinterpret_cast<const P*>(p + v * V), o);
#pragma unroll
        for (int q = 0; q < V; ++q) s[q & 1] = sq(s[q & 1], o[q]);
    }
    const int i = nvec * V + threadIdx.x;                 // the last len % V elements
    if (i < len) s[0] = sq(s[0], Elem<T>::ld(p + i));
    return s[0] + s[1];
}

// Sum over the block's 256 threads, in a fixed order; every thread gets it.
__device__ __forceinline__ double block_sum(double v, double* sh) {
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    return (sh[0] + sh[1]) + (sh[2] + sh[3]);
}

__global__ __launch_bounds__(256) void grad_squares_kernel(GradTable g,
                                                           double* __restrict__ partial) {
    __shared__ double sh[4];
    double s = 0.0;
    for (uint32_t c = blockIdx.x; c < g.first[g.n]; c += gridDim.x) {
        const Chunk k = chunk_of<false>(g, c);
        s += k.bf16 ? chunk_squares(static_cast<const bf16_t*>(g.in[k.t]) + k.i0, k.len)
                    : chunk_squares(static_cast<const float*>(g.in[k.t]) + k.i0, k.len);
    }
    s = block_sum(s, sh);
    if (threadIdx.x == 0) partial[blockIdx.x] = s;
}

// The norm from all launches' partial sums; every block that calls it gets
// the same bits.
__device__ __forceinline__ float norm_of(const double* __restrict__ partial, int np, double* sh) {
    double s = 0.0;
    for (int i = threadIdx.x; i < np; i += 256) s += partial[i];
    return (float)sqrt(block_sum(s, sh));
}

__global__ __launch_bounds__(256) void grad_norm_kernel(const double* __restrict__ partial,
                                                        int np, float* __restrict__ norm) {
    __shared__ double sh[4];
    const float v = norm_of(partial, np, sh);
    if (threadIdx.x == 0) *norm = v;
}

// WIDE: by a factor below fp32's normal range, which has lost bits there (or is
// 0): factor and product in fp64.
template <typename T, bool WIDE>
__device__ __forceinline__ void chunk_scale(const T* p, T* o, int len, double c) {
    typedef typename Packed<T>::type P;
    constexpr int V = Vec16<T>::N, UN = 4;
    const int nvec = len / V;
    auto times = [&](float a) { return WIDE ? (float)((double)a * c) : a * (float)c; };
    auto scaled = [&](u32x4_t raw) {
        float a[V];
        unpack16<T>(raw, a);
#pragma unroll
        for (int q = 0; q < V; ++q) a[q] = times(a[q]);
        return pack16<T>(a);
    };
    int v = threadIdx.x;
    for (; v + 256 * (UN - 1) < nvec; v += 256 * UN) {
        u32x4_t raw[UN];
#pragma unroll
        for (int u = 0; u < UN; ++u) raw[u] = *reinterpret_cast<const P*>(p + (v + 256 * u) * V);
#pragma unroll
        for (int u = 0; u < UN; ++u)
            __builtin_nontemporal_store(scaled(raw[u]),
                                        reinterpret_cast<P*>(o + (v + 256 * u) * V));
    }
    for (; v < nvec; v += 256)
        *reinterpret_cast<P*>(o + v * V) = scaled(*reinterpret_cast<const P*>(p + v * V));
    const int i = nvec * V + threadIdx.x;
    if (i < len) Elem<T>::st(o + i, times(Elem<T>::ld(p + i)));
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const GradTable& g, const Chunk& k, float c,
                                            double wide) {
    const T* p = static_cast<const T*>(g.in[k.t]) + k.i0;
    T* o = static_cast<T*>(g.out[k.t]) + k.i0;
    if (wide > 0.0) chunk_scale<T, true>(p, o, k.len, wide);
    else chunk_scale<T, false>(p, o, k.len, c);
}

// out = g * (norm > max_norm ? max_norm / norm : 1), the product rounded to fp32
// and a bf16 element then to bf16.  A norm that is not finite scales nothing: the step is the caller's to drop, and
// zeros or NaN in place of the gradients would hide why.  In place a factor
// of 1 leaves nothing to do.
//
// The list is taken from its end to its start: what the norm read last is
// still in the 256 MB cache.  Stores bypass the caches, so that they neither
// evict it nor leave lines to be written back under the next kernel's reads
// (345 MB in 200 tensors, norm and scaling: 224 us with plain stores in list
// order, 210 backwards, 181 with both).
//
// np = 0: *norm is there already; else the launch for the first chunks (first)
// stores it.
__global__ __launch_bounds__(256) void grad_scale_kernel(GradTable g,
                                                         const double* __restrict__ partial,
                                                         int np, float max_norm, bool first,
                                                         float* norm) {
    __shared__ double sh[4];
    const float v = np > 0 ? norm_of(partial, np, sh) : *norm;
    if (np > 0 && first && blockIdx.x == 0 && threadIdx.x == 0) *norm = v;
    const float c = v > max_norm && v < INFINITY ? max_norm / v : 1.0f;
    const double wide = c < FLT_MIN ? (double)max_norm / (double)v : 0.0;
    for (uint32_t q = blockIdx.x; q < g.first[g.n]; q += gridDim.x) {
        const Chunk k = chunk_of<true>(g, q);
        if (c == 1.0f && g.in[k.t] == g.out[k.t]) continue;
        if (k.bf16) chunk_scale<bf16_t>(g, k, c, wide);
        else chunk_scale<float>(g, k, c, wide);
    }
}

// ------------------------------------------------------------------- host
constexpr size_t kMaxNumel = (size_t)1 << 40;          // chunks of a launch stay in 32 bits

bool list_ok(const void* const* grads, void* const* out, const size_t* numel, const int32_t* dt,
             int n, bool clip) {
    if (n < 0 || (n > 0 && (!grads || !numel || !dt || (clip && !out)))) return false;
    for (int i = 0; i < n; ++i) {
        if (dt[i] != MOE_F32 && dt[i] != MOE_BF16) return false;
        if (numel[i] > kMaxNumel) return false;
        if (numel[i] == 0) continue;
        const uintptr_t mask = dt[i] == MOE_BF16 ? 1 : 3;
        if (!grads[i] || (reinterpret_cast<uintptr_t>(grads[i]) & mask)) return false;
        if (clip && (!out[i] || (reinterpret_cast<uintptr_t>(out[i]) & mask))) return false;
    }
    return true;
}

uint64_t chunks_of(size_t numel, int dt) {
    const size_t per = kChunkBytes / (dt == MOE_BF16 ? 2 : 4);
    return (numel + per - 1) / per;
}

// Calls f(table, blocks) for each launch of the list, first tensors first or
// (back) last ones first; stops early when f returns false.  out may be NULL.
template <class F>
void for_launches(const void* const* grads, void* const* out, const size_t* numel,
                  const int32_t* dt, int n, int max_blocks, bool back, F&& f) {
    GradTable g;
    g.n = 0;
    g.first[0] = 0;
    auto flush = [&]() {
        if (g.n == 0) return true;
        const bool ok = f(g, (int)min((uint32_t)max_blocks, g.first[g.n]));
        g.n = 0;
        return ok;
    };
    for (int q = 0; q < n; ++q) {
        const int i = back ? n - 1 - q : q;
        if (numel[i] == 0) continue;
        const uint64_t c = chunks_of(numel[i], dt[i]);
        // a launch's chunk numbers, and a block's next one, stay below 2^32
        if (g.n == kTensors || (g.n > 0 && g.first[g.n] + c >= (1ull << 31)))
            if (!flush()) return;
        if (grads) g.in[g.n] = grads[i];
        g.out[g.n] = out ? out[i] : nullptr;
        g.numel[g.n] = numel[i] | (dt[i] == MOE_BF16 ? kBf16Flag : 0);
        g.first[g.n + 1] = g.first[g.n] + (uint32_t)c;
        ++g.n;
    }
    flush();
}

int partials_of(const size_t* numel, const int32_t* dt, int n) {
    int np = 0;
    for_launches(nullptr, nullptr, numel, dt, n, kNormBlocks, false,
                 [&](const GradTable&, int blocks) {
        np += blocks;
        return true;
    });
    return np;
}

moe_status run_squares(const void* const* grads, const size_t* numel, const int32_t* dt, int n,
                       double* partial, hipStream_t s) {
    int at = 0;
    moe_status st = MOE_OK;
    for_launches(grads, nullptr, numel, dt, n, kNormBlocks, false,
                 [&](const GradTable& g, int blocks) {
        MOE_LAUNCH("grad_squares", s, (grad_squares_kernel<<<blocks, 256, 0, s>>>(g, partial + at)));
        at += blocks;
        st = launch_status();
        return st == MOE_OK;
    });
    return st;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_grad_norm_workspace_bytes(const size_t* numel, const int32_t* dt, int n) {
    if (n < 0 || (n > 0 && (!numel || !dt))) return 0;
    for (int i = 0; i < n; ++i)
        if ((dt[i] != MOE_F32 && dt[i] != MOE_BF16) || numel[i] > kMaxNumel) return 0;
    return align_up(sizeof(double) * ((size_t)partials_of(numel, dt, n) + 1), 256);
}

moe_status moe_grad_norm(const void* const* grads, const size_t* numel, const int32_t* dt, int n,
                         float* norm, void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_CHECK_ARG(list_ok(grads, nullptr, numel, dt, n, false) && norm);
    const int np = partials_of(numel, dt, n);
    if (!ws || ws_bytes < sizeof(double) * (size_t)np) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 7u) == 0);
    MOE_CHECK_DEVICE();
    double* partial = static_cast<double*>(ws);
    const moe_status st = run_squares(grads, numel, dt, n, partial, stream);
    if (st != MOE_OK) return st;
    MOE_LAUNCH("grad_norm", stream,
               (grad_norm_kernel<<<1, 256, 0, stream>>>(partial, np, norm)));
    return launch_status();
}

moe_status moe_clip_grads(const void* const* grads, void* const* out, const size_t* numel,
                          const int32_t* dt, int n, const float* max_norm, float* norm, void* ws,
                          size_t ws_bytes, hipStream_t stream) {
    MOE_CHECK_ARG(list_ok(grads, out, numel, dt, n, true) && norm && max_norm);
    const float mx = *max_norm;
    MOE_CHECK_ARG(mx >= 0.0f);                            // NaN too is refused
    const int np = partials_of(numel, dt, n);
    if (!ws || ws_bytes < sizeof(double) * (size_t)np) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 7u) == 0);
    MOE_CHECK_DEVICE();
    double* partial = static_cast<double*>(ws);
    moe_status st = run_squares(grads, numel, dt, n, partial, stream);
    if (st != MOE_OK) return st;
    const bool ahead = np == 0 || np > kOwnSums;
    if (ahead) {
        MOE_LAUNCH("grad_norm", stream,
                   (grad_norm_kernel<<<1, 256, 0, stream>>>(partial, np, norm)));
        st = launch_status();
        if (st != MOE_OK || np == 0) return st;
    }
    bool first = true;
    for_launches(grads, out, numel, dt, n, kScaleBlocks, true,
                 [&](const GradTable& g, int blocks) {
        MOE_LAUNCH("grad_scale", stream,
                   (grad_scale_kernel<<<blocks, 256, 0, stream>>>(g, partial, ahead ? 0 : np, mx,
                                                                  first, norm)));
        first = false;
        st = launch_status();
        return st == MOE_OK;
    });
    return st;
}

}  // extern "C"
