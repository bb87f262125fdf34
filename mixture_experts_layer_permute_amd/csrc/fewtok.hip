// The whole layer for a few tokens (1 .. 64), forward only: a serving step.
//
// With a handful of rows per expert every product reads a weight matrix once
// and does almost no arithmetic on it, so the layer is a stream of the chosen
// experts' weights from HBM: bytes = hit * P * d * f * b (P = 2 matrices, 3
// for SwiGLU).  The grouped GEMM's 64-256-row tiles, its plan, its saved
// state and its row copies have nothing to give there.
//
// Kernels of a call:
//   few_logits   the gate's logits, one fixed-order fp32 chain per (token,
//                expert): the same bits as moe_gate_topk
//   few_topk     top-k and gate weights, one wave per token
//   few_up       per (expert hit, strip of columns): act(x W1[e]) (* x W3[e])
//   few_down     per (expert hit, strip of columns, chunk of f): h W2[e], fp32
//   few_combine  y[t] = sum_j w[t,j] sum_chunks partial, in slot and chunk order
//
// Weight tiles go straight from HBM into registers, with no LDS: a strip of
// 16 * VW columns is read by 16 lanes of VW columns (16 bytes of a row each),
// and the wave's four groups of 16 lanes take different rows.  As the A
// operand of v_mfma_f32_16x16x32_bf16 a lane needs eight consecutive k of one
// column: its eight row loads hold exactly those for each of its VW columns,
// so one byte permute per pair of rows transposes in registers.  The tokens
// are the B operand's columns, 16 at a time, read from L2.
#include <float.h>

#include <type_traits>

#include "common.h"

namespace moe {
namespace {

constexpr int kFewTokens = 64;          // most tokens of a call
constexpr int kFewPairs = 4096;         // most (token, slot) pairs of a call

// ------------------------------------------------------------ gate logits
// Block: 256 threads, 16 tokens x 16 experts, one chain per thread.  The
// chain's order is fixed (increasing feature index, each sum rounded), so its
// length d sets the time: GK features at a time are staged in LDS as fp32,
// NPF chunks ahead of the chain in registers.
constexpr int GK = 128, GTOK = 16, GEXP = 16, GROW = GK + 4;

template <typename T>
__global__ __launch_bounds__(256) void few_logits_kernel(const T* __restrict__ x,
                                                         const T* __restrict__ Wg,
                                                         const float* __restrict__ bias, int Tn,
                                                         int d, int E,
                                                         float* __restrict__ logits) {
#pragma clang fp contract(off)
    constexpr int V = Vec16<T>::N;
    constexpr int NPF = 4;
    constexpr int WV = GK * GEXP / 256;                 // gate elements per thread and chunk
    constexpr int XV = GTOK * GK / V / 256;             // x vectors per thread and chunk
    static_assert(XV >= 1, "a vector per thread");
    __shared__ __attribute__((aligned(16))) float ws[GEXP * GROW];
    __shared__ __attribute__((aligned(16))) float xs[GTOK * GROW];
    const int tid = threadIdx.x;
    const int e0 = blockIdx.x * GEXP, t0 = blockIdx.y * GTOK;
    const int le = tid % GEXP, lt = tid / GEXP;

    T wr[NPF][WV];
    u32x4_t xr[NPF][XV];
    // loads past the matrix read a valid element instead: features past d are
    // never summed, experts and tokens past the end never stored
    auto fetch = [&](int c, T (&w)[WV], u32x4_t (&xv)[XV]) {
        const int k0 = c * GK;
#pragma unroll
        for (int q = 0; q < WV; ++q) {
            const int kk = min(k0 + (tid + 256 * q) / GEXP, d - 1);
            w[q] = Wg[(long)kk * E + min(e0 + le, E - 1)];
        }
#pragma unroll
        for (int q = 0; q < XV; ++q) {
            const int i = tid + 256 * q;
            const int tok = min(t0 + i / (GK / V), Tn - 1);
            const int k = min(k0 + i % (GK / V) * V, d - V);
            xv[q] = ld16<false>(x + (long)tok * d + k);
        }
    };
    float acc = 0.0f;
    const int nc = (d + GK - 1) / GK;
#pragma unroll
    for (int c = 0; c < NPF; ++c) fetch(c, wr[c], xr[c]);
    for (int cb = 0; cb < nc; cb += NPF) {
#pragma unroll
        for (int u = 0; u < NPF; ++u) {
            const int c = cb + u;
            if (c >= nc) break;
            __syncthreads();
#pragma unroll
            for (int q = 0; q < WV; ++q)
                ws[le * GROW + (tid + 256 * q) / GEXP] = Elem<T>::ld(&wr[u][q]);
#pragma unroll
            for (int q = 0; q < XV; ++q) {
                const int i = tid + 256 * q;
                float o[V];
                unpack16<T>(xr[u][q], o);
                float* p = xs + (i / (GK / V)) * GROW + i % (GK / V) * V;
#pragma unroll
                for (int v = 0; v < V; v += 4)
                    *reinterpret_cast<float4*>(p + v) =
                        make_float4(o[v], o[v + 1], o[v + 2], o[v + 3]);
            }
            __syncthreads();
            fetch(c + NPF, wr[u], xr[u]);
            const int kn = min(GK, d - c * GK);         // a multiple of 64
            const float* wp = ws + le * GROW;
            const float* xp = xs + lt * GROW;
#pragma unroll 4
            for (int k = 0; k < kn; k += 4) {
                const float4 a = *reinterpret_cast<const float4*>(xp + k);
                const float4 b = *reinterpret_cast<const float4*>(wp + k);
                if constexpr (sizeof(T) == 2) {
                    // the product of two bf16 is exact in fp32: one rounding
                    acc = __builtin_fmaf(a.x, b.x, acc);
                    acc = __builtin_fmaf(a.y, b.y, acc);
                    acc = __builtin_fmaf(a.z, b.z, acc);
                    acc = __builtin_fmaf(a.w, b.w, acc);
                } else {
                    acc = acc + a.x * b.x;
                    acc = acc + a.y * b.y;
                    acc = acc + a.z * b.z;
                    acc = acc + a.w * b.w;
                }
            }
        }
    }
    if (e0 + le < E && t0 + lt < Tn) {
        if (bias) acc = acc + bias[e0 + le];
        logits[(long)(t0 + lt) * E + e0 + le] = acc;
    }
}

// ------------------------------------------------------------------ top-k
// One wave per token: k rounds of an arg-max over (value descending, index
// ascending), then the softmax over the selected logits or over all.  A lane
// holds experts lane, lane + 64, ...; `live` marks those not taken yet.
//
// The order is taken on one 64-bit key per expert, so that it is total and
// every lane agrees on the winner whatever the logits hold: the float's bits
// made monotone (both zeros alike, NaN below everything), then the index
// downwards.  A key is never 0, which stands for an expert already taken.
__device__ __forceinline__ uint64_t logit_key(float v, int e) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    const uint32_t m = v != v ? 0u : b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)m << 32) | (uint32_t)(0x7fffffff - e);
}

__device__ __forceinline__ void wave_topk(const float* __restrict__ lt, int E, int k, int renorm,
                                          int32_t* __restrict__ idx, float* __restrict__ w) {
    const int lane = threadIdx.x & 63;
    uint32_t live = 0;
    for (int q = 0; q * 64 + lane < E; ++q) live |= 1u << q;      // E <= 1024
    float best0 = 0.0f, den = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint64_t best = 0;
        for (int q = 0; q * 64 + lane < E; ++q) {
            const int e = q * 64 + lane;
            const uint64_t key = logit_key(lt[e], e);
            if (((live >> q) & 1u) && key > best) best = key;
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const uint64_t o = __shfl_xor((unsigned long long)best, off);
            best = o > best ? o : best;
        }
        const int bi = 0x7fffffff - (int)(uint32_t)best;          // k <= E: always one left
        const float bv = lt[bi];
        if ((bi & 63) == lane) live &= ~(1u << (bi >> 6));
        if (j == 0) best0 = bv;
        const float ex = expf(bv - best0);
        den += ex;
        if (lane == 0) {
            idx[j] = bi;
            w[j] = ex;                                             // scaled below
        }
    }
    if (!renorm) {
        den = 0.0f;
        for (int e = lane; e < E; e += 64) den += expf(lt[e] - best0);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) den += __shfl_xor(den, off);
    }
    const float inv = 1.0f / den;
    if (lane == 0)
        for (int j = 0; j < k; ++j) w[j] *= inv;
}

__global__ __launch_bounds__(256) void few_topk_kernel(const float* __restrict__ logits, int Tn,
                                                       int E, int k, int renorm,
                                                       int32_t* __restrict__ idx,
                                                       float* __restrict__ w) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= Tn) return;
    wave_topk(logits + (long)t * E, E, k, renorm, idx + (long)t * k, w + (long)t * k);
}

// ------------------------------------------------------- experts' row lists
// The rows of the `slot`-th expert (by index) that any token chose, as pair
// numbers t * k + j in increasing order: at most one per token.  Returns the
// expert, or -1 when fewer experts were hit.  Every thread of the block takes
// part; bits: 32 words, rows: kFewTokens ints, res: 2 ints of LDS.
__device__ __forceinline__ int expert_rows(const int32_t* __restrict__ idx, int pairs, int E,
                                           int slot, uint32_t* bits, int* rows, int* res, int* n) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    if (tid < 32) bits[tid] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += nthr) {
        const int e = idx[p];
        if ((unsigned)e < (unsigned)E) atomicOr(&bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (tid < 64) {
        uint32_t b = tid < 32 ? bits[tid] : 0u;
        const int pc = __popc(b);
        const int inc = wave_incl_scan(pc);
        const int exc = inc - pc;
        const bool mine = slot >= exc && slot < inc;
        int e = -1;
        if (mine) {
            for (int q = exc; q < slot; ++q) b &= b - 1;          // drop the lower set bits
            e = tid * 32 + __ffs(b) - 1;
        }
        const uint64_t who = __ballot(mine);
        e = who ? __shfl(e, __ffsll((unsigned long long)who) - 1) : -1;
        int cnt = 0;
        if (e >= 0)
            for (int p0 = 0; p0 < pairs; p0 += 64) {
                const int p = p0 + tid;
                const bool hit = p < pairs && idx[p] == e;
                const uint64_t m = __ballot(hit);
                const int pos = cnt + __popcll(m & ((1ull << tid) - 1));
                if (hit && pos < kFewTokens) rows[pos] = p;
                cnt += __popcll(m);
            }
        if (tid == 0) {
            res[0] = e;
            res[1] = min(cnt, kFewTokens);
        }
    }
    __syncthreads();
    *n = res[1];
    return res[0];
}

// -------------------------------------------------------------- activation
__device__ __forceinline__ float gelu_f(float z) {
    return 0.5f * z * erfcf(z * -0.70710678118654752f);
}
__device__ __forceinline__ float silu_f(float z) { return z / (1.0f + expf(-z)); }

// ----------------------------------------------------- skinny product core
// C[n columns of a strip][16 * NT tokens] += W[K, N]^T x^T over the k-steps
// s0 .. s1 of one wave.  Lane (c = lane % 16, g = lane / 16) loads columns
// n0 + c*VW .. + VW-1; accumulator acc[i][j][r] is column
// n0 + (4 g + r) VW + j of token 16 i + c.
template <typename T> struct Core;

template <> struct Core<bf16_t> {
    static constexpr int KSTEP = 32;                  // rows of W per step
    static constexpr int NL = 8;                      // row loads per lane and step
    template <int VW> struct Raw { uint32_t w[NL][VW / 2]; };
    struct XRaw { u32x4_t v; };

    template <int VW>
    static __device__ __forceinline__ void load(const bf16_t* W, long ldw, int k0, int g,
                                                Raw<VW>& r) {
        const bf16_t* p = W + (long)(k0 + g * 8) * ldw;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if constexpr (VW == 8) {
                const u32x4_t v = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x4_t*>(p + i * ldw));
#pragma unroll
                for (int q = 0; q < 4; ++q) r.w[i][q] = v[q];
            } else {
                typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
                const u32x2_t v = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x2_t*>(p + i * ldw));
                r.w[i][0] = v[0];
                r.w[i][1] = v[1];
            }
        }
    }
    static __device__ __forceinline__ void loadx(const bf16_t* xrow, int k0, int g, XRaw& r) {
        r.v = ld16<false>(xrow + k0 + g * 8);
    }
    template <int VW, int NT>
    static __device__ __forceinline__ void mul(const Raw<VW>& r, const XRaw (&x)[NT], int nt,
                                               f32x4 (&acc)[NT][VW]) {
#pragma unroll
        for (int j = 0; j < VW; ++j) {
            // column j's eight k: the low (j even) or high halves of dword
            // j / 2 of each row, packed in pairs
            u32x4_t a;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                a[q] = __builtin_amdgcn_perm(r.w[2 * q + 1][j / 2], r.w[2 * q][j / 2],
                                             (j & 1) ? 0x07060302u : 0x05040100u);
            const bf16x8 av = __builtin_bit_cast(bf16x8, a);
#pragma unroll
            for (int i = 0; i < NT; ++i)
                if (i < nt)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        av, __builtin_bit_cast(bf16x8, x[i].v), acc[i][j], 0, 0, 0);
        }
    }
};

template <> struct Core<float> {
    static constexpr int KSTEP = 16;
    static constexpr int NL = 4;
    template <int VW> struct Raw { f32x4 w[NL]; };
    struct XRaw { f32x4 v; };

    template <int VW>
    static __device__ __forceinline__ void load(const float* W, long ldw, int k0, int g,
                                                Raw<VW>& r) {
        static_assert(VW == 4, "16 bytes per lane and row");
        const float* p = W + (long)(k0 + g * 4) * ldw;
#pragma unroll
        for (int i = 0; i < NL; ++i)
            r.w[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + i * ldw));
    }
    static __device__ __forceinline__ void loadx(const float* xrow, int k0, int g, XRaw& r) {
        r.v = *reinterpret_cast<const f32x4*>(xrow + k0 + g * 4);
    }
    template <int VW, int NT>
    static __device__ __forceinline__ void mul(const Raw<VW>& r, const XRaw (&x)[NT], int nt,
                                               f32x4 (&acc)[NT][VW]) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j)
#pragma unroll
                for (int m = 0; m < NT; ++m)
                    if (m < nt)
                        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(r.w[i][j], x[m].v[i],
                                                                        acc[m][j], 0, 0, 0);
    }
};

template <typename T, int VW, int NT, bool DUAL>
__device__ __forceinline__ void strip_product(const T* W, const T* W3, long ldw,
                                              const T* const (&xrow)[NT], int nt, int s0, int s1,
                                              f32x4 (&acc)[NT][VW],
                                              f32x4 (&acc3)[DUAL ? NT : 1][DUAL ? VW : 1]) {
    typedef Core<T> C;
    const int g = (threadIdx.x & 63) >> 4;
    typename C::template Raw<VW> wa[2], wb[2];
    typename C::XRaw xa[2][NT];
    auto fetch = [&](int s, int b) {
        C::template load<VW>(W, ldw, s * C::KSTEP, g, wa[b]);
        if constexpr (DUAL) C::template load<VW>(W3, ldw, s * C::KSTEP, g, wb[b]);
#pragma unroll
        for (int i = 0; i < NT; ++i) C::loadx(xrow[i], s * C::KSTEP, g, xa[b][i]);
    };
    auto mul = [&](int b) {
        C::template mul<VW, NT>(wa[b], xa[b], nt, acc);
        if constexpr (DUAL) C::template mul<VW, NT>(wb[b], xa[b], nt, acc3);
    };
    if (s0 >= s1) return;
    fetch(s0, 0);
    int s = s0;
    for (; s + 2 < s1; s += 2) {
        fetch(s + 1, 1);
        mul(0);
        fetch(s + 2, 0);
        mul(1);
    }
    if (s + 1 < s1) {
        fetch(s + 1, 1);
        mul(0);
        mul(1);
    } else {
        mul(0);
    }
}

// One wave's accumulators of 16 tokens into its LDS slab [16][BN + 4].
template <int VW>
__device__ __forceinline__ void slab_store(float* slab, const f32x4 (&acc)[VW]) {
    constexpr int LD = 16 * VW + 4;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    float* p = slab + c * LD + g * 4 * VW;
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < VW; j += 4)
            *reinterpret_cast<float4*>(p + r * VW + j) =
                make_float4(acc[j][r], acc[j + 1][r], acc[j + 2][r], acc[j + 3][r]);
}
template <int VW, int NW>
__device__ __forceinline__ float4 slab_sum(const float* slabs, int row, int col) {
    constexpr int LD = 16 * VW + 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(slabs + (w * 16 + row) * LD + col);
        s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
    }
    return s;
}

__device__ __forceinline__ void store4(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(bf16_t* p, const float* v) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

struct FewArgs {
    const void* x;              // up: tokens [T, K]; down: h [pairs, K]
    const void *W, *W3;         // [E, K, N]
    const int32_t* idx;         // [pairs]
    void* out;                  // up: h [pairs, N]; down: partial [KS][pairs][N] fp32
    int pairs, k, E, K, N;
};

// UP: h[p] = act(x[p / k] W[e]) (DUAL: * x W3[e]) for the expert's pairs p.
// Down (UP = false): partial[ks][p] = h[p] W[e] over the ks-th chunk of K.
// Grid: strips of 16 * VW columns, experts hit, chunks.  The NW waves of a
// block take consecutive parts of the chunk; their sums meet in LDS, in order.
template <typename T, int VW, int NT, int NW, bool UP, bool DUAL>
__global__ __launch_bounds__(64 * NW, 2) void few_product_kernel(FewArgs p) {
    constexpr int BN = 16 * VW, LD = BN + 4;
    constexpr int SLABS = NW * 16 * LD;
    __shared__ __attribute__((aligned(16))) float red[SLABS * (DUAL ? 2 : 1)];
    __shared__ uint32_t bits[32];
    __shared__ int rows[kFewTokens], res[2];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    int n;
    const int e = expert_rows(p.idx, p.pairs, p.E, blockIdx.y, bits, rows, res, &n);
    if (e < 0) return;
    const int nt = (n + 15) >> 4;
    const int n0 = blockIdx.x * BN;
    const int c = lane & 15;
    // columns past N (a multiple of 64) read the last ones of the row instead
    const int col = min(n0 + c * VW, p.N - VW);
    const T* W = static_cast<const T*>(p.W) + (long)e * p.K * p.N + col;
    const T* W3 = DUAL ? static_cast<const T*>(p.W3) + (long)e * p.K * p.N + col : nullptr;
    const T* xrow[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int q = rows[min(i * 16 + c, n - 1)];   // rows past n: the last one's again
        xrow[i] = static_cast<const T*>(p.x) + (long)(UP ? q / p.k : q) * p.K;
    }
    f32x4 acc[NT][VW], acc3[DUAL ? NT : 1][DUAL ? VW : 1];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < VW; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (DUAL) {
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j) acc3[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    const int steps = p.K / Core<T>::KSTEP;
    const int units = gridDim.z * NW, u = blockIdx.z * NW + wv;
    strip_product<T, VW, NT, DUAL>(W, W3, p.N, xrow, nt, (int)((long)steps * u / units),
                                   (int)((long)steps * (u + 1) / units), acc, acc3);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        if (i >= nt) break;
        if (i > 0) __syncthreads();
        slab_store<VW>(red + wv * 16 * LD, acc[i]);
        if constexpr (DUAL) slab_store<VW>(red + SLABS + wv * 16 * LD, acc3[i]);
        __syncthreads();
        for (int q = tid; q < 16 * BN / 4; q += 64 * NW) {
            const int row = q / (BN / 4), cl = q % (BN / 4) * 4;
            if (i * 16 + row >= n || n0 + cl >= p.N) continue;
            const float4 s = slab_sum<VW, NW>(red, row, cl);
            const int pr = rows[i * 16 + row];
            float v[4] = {s.x, s.y, s.z, s.w};
            if constexpr (UP) {
                if constexpr (DUAL) {
                    const float4 h3 = slab_sum<VW, NW>(red + SLABS, row, cl);
                    v[0] = silu_f(v[0]) * h3.x;
                    v[1] = silu_f(v[1]) * h3.y;
                    v[2] = silu_f(v[2]) * h3.z;
                    v[3] = silu_f(v[3]) * h3.w;
                } else {
#pragma unroll
                    for (int a = 0; a < 4; ++a) v[a] = gelu_f(v[a]);
                }
                // h in the layer's type, as moe_expert_ffn_fwd keeps it
                store4(static_cast<T*>(p.out) + (long)pr * p.N + n0 + cl, v);
            } else {
                store4(static_cast<float*>(p.out) +
                           ((long)blockIdx.z * p.pairs + pr) * p.N + n0 + cl, v);
            }
        }
    }
}

// y[t] = sum_j w[t,j] sum_s partial[s][t k + j], rounded once.
template <typename T>
__global__ __launch_bounds__(256) void few_combine_kernel(const float* __restrict__ partial,
                                                          const float* __restrict__ w, int Tn,
                                                          int k, int d, int ks,
                                                          T* __restrict__ y) {
    const int q = blockIdx.x * 256 + threadIdx.x;
    const int per = d / 4;
    if (q >= Tn * per) return;
    const int t = q / per, c = q % per * 4;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j = 0; j < k; ++j) {
        float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int z = 0; z < ks; ++z) {
            const float4 a = *reinterpret_cast<const float4*>(
                partial + ((long)z * Tn * k + t * k + j) * d + c);
            s.x += a.x; s.y += a.y; s.z += a.z; s.w += a.w;
        }
        const float wj = w[t * k + j];
        v[0] = fmaf(wj, s.x, v[0]);
        v[1] = fmaf(wj, s.y, v[1]);
        v[2] = fmaf(wj, s.z, v[2]);
        v[3] = fmaf(wj, s.w, v[3]);
    }
    store4(y + (long)t * d + c, v);
}

// ------------------------------------------------------------------- plan
struct FewPlan {
    int slots;                   // experts hit at most
    int up_vw, down_vw, up_strips, down_strips, ks;
    size_t logits, idx, w, h, partial, total;
};

bool few_sizes_ok(int T, int d, int f, int E, int k, moe_act act, moe_dtype dt) {
    return T >= 0 && d >= 64 && d % 64 == 0 && f >= 64 && f % 64 == 0 && E >= 1 && E <= 1024 &&
           k >= 1 && k <= E && (act == MOE_ACT_GELU || act == MOE_ACT_SWIGLU) &&
           (dt == MOE_F32 || dt == MOE_BF16);
}
bool few_limits_ok(int T, int k) { return T <= kFewTokens && (long)T * k <= kFewPairs; }

FewPlan few_plan(int T, int d, int f, int E, int k, moe_act act, moe_dtype dt) {
    FewPlan p;
    const int pairs = T * k;
    p.slots = min(E, pairs);
    // 16 VW columns a strip.  Two weights at once over more than 16 tokens
    // would not fit the registers at VW = 8
    p.up_vw = dt == MOE_BF16 && !(act == MOE_ACT_SWIGLU && T > 16) ? 8 : 4;
    p.down_vw = dt == MOE_BF16 ? 8 : 4;
    p.up_strips = cdiv(f, 16 * p.up_vw);
    p.down_strips = cdiv(d, 16 * p.down_vw);
    const int steps = f / (dt == MOE_BF16 ? 32 : 16);
    int ks = 1;
    while (ks < 16 && p.down_strips * p.slots * ks < 512 && steps >= ks * 2 * 4 * 2) ks *= 2;
    p.ks = ks;
    const size_t es = dt == MOE_BF16 ? 2 : 4;
    p.logits = 0;
    p.idx = align_up(sizeof(float) * (size_t)T * E, 256);
    p.w = align_up(p.idx + sizeof(int32_t) * pairs, 256);
    p.h = align_up(p.w + sizeof(float) * pairs, 256);
    p.partial = align_up(p.h + es * pairs * f, 256);
    p.total = align_up(p.partial + sizeof(float) * (size_t)ks * pairs * d, 256);
    return p;
}

template <typename T, int NT>
moe_status few_run(const void* x, const void* Wg, const float* bias, const void* W1,
                   const void* W3, const void* W2, int Tn, int d, int f, int E, int k, int renorm,
                   moe_act act, const FewPlan& p, float* logits, int32_t* idx, float* w, void* y,
                   char* ws, hipStream_t s) {
    MOE_LAUNCH("few_logits", s,
               (few_logits_kernel<T><<<dim3(cdiv(E, GEXP), cdiv(Tn, GTOK)), 256, 0, s>>>(
                   static_cast<const T*>(x), static_cast<const T*>(Wg), bias, Tn, d, E,
                   logits)));
    MOE_LAUNCH("few_topk", s,
               (few_topk_kernel<<<cdiv(Tn, 4), 256, 0, s>>>(logits, Tn, E, k, renorm, idx, w)));
    const int pairs = Tn * k;
    FewArgs u{x, W1, W3, idx, ws + p.h, pairs, k, E, d, f};
    const dim3 gu(p.up_strips, p.slots, 1), gd(p.down_strips, p.slots, p.ks);
    constexpr int VW = sizeof(T) == 2 ? 8 : 4;
    constexpr int VWD = NT == 1 ? VW : 4;
    if (act == MOE_ACT_SWIGLU)
        MOE_LAUNCH("few_up_swiglu", s,
                   (few_product_kernel<T, VWD, NT, 4, true, true><<<gu, 256, 0, s>>>(u)));
    else
        MOE_LAUNCH("few_up_gelu", s,
                   (few_product_kernel<T, VW, NT, 4, true, false><<<gu, 256, 0, s>>>(u)));
    FewArgs v{ws + p.h, W2, nullptr, idx, ws + p.partial, pairs, k, E, f, d};
    MOE_LAUNCH("few_down", s,
               (few_product_kernel<T, VW, NT, 4, false, false><<<gd, 256, 0, s>>>(v)));
    MOE_LAUNCH("few_combine", s,
               (few_combine_kernel<T><<<cdiv((long)Tn * d / 4, 256), 256, 0, s>>>(
                   reinterpret_cast<const float*>(ws + p.partial), w, Tn, k, d, p.ks,
                   static_cast<T*>(y))));
    return launch_status();
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_layer_few_workspace_bytes(int T, int d, int f, int E, int k, moe_act act,
                                     moe_dtype dt) {
    if (!few_sizes_ok(T, d, f, E, k, act, dt) || !few_limits_ok(T, k)) return 0;
    return few_plan(T, d, f, E, k, act, dt).total;
}

moe_status moe_layer_fwd_few(const void* x, const void* Wg, const float* logit_bias,
                             const void* W1, const void* W3, const void* W2, int T, int d, int f,
                             int E, int k, int renorm, moe_act act, moe_dtype dt, float* logits,
                             int32_t* topk_idx, float* topk_w, void* y, void* ws,
                             size_t ws_bytes, hipStream_t stream) {
    MOE_CHECK_ARG(few_sizes_ok(T, d, f, E, k, act, dt));
    if (!few_limits_ok(T, k)) return MOE_ERR_UNSUPPORTED;
    if (T == 0) return MOE_OK;
    MOE_CHECK_ARG(x && Wg && W1 && W2 && y && (act != MOE_ACT_SWIGLU || W3));
    MOE_CHECK_ARG(aligned16(x) && aligned16(W1) && aligned16(W2) && aligned16(y) &&
                  (act != MOE_ACT_SWIGLU || aligned16(W3)));
    const FewPlan p = few_plan(T, d, f, E, k, act, dt);
    if (!ws || ws_bytes < p.total) return MOE_ERR_WORKSPACE;
    MOE_CHECK_ARG((reinterpret_cast<uintptr_t>(ws) & 15u) == 0);
    MOE_CHECK_DEVICE();
    char* base = static_cast<char*>(ws);
    float* lg = logits ? logits : reinterpret_cast<float*>(base + p.logits);
    int32_t* ix = topk_idx ? topk_idx : reinterpret_cast<int32_t*>(base + p.idx);
    float* wt = topk_w ? topk_w : reinterpret_cast<float*>(base + p.w);
    auto go = [&](auto tag, auto nt) {
        return few_run<decltype(tag), decltype(nt)::value>(
            x, Wg, logit_bias, W1, W3, W2, T, d, f, E, k, renorm, act, p, lg, ix, wt, y, base,
            stream);
    };
    auto by_tokens = [&](auto tag) {
        using std::integral_constant;
        if (T <= 16) return go(tag, integral_constant<int, 1>{});
        if (T <= 32) return go(tag, integral_constant<int, 2>{});
        return go(tag, integral_constant<int, 4>{});
    };
    return dt == MOE_BF16 ? by_tokens(bf16_t{}) : by_tokens(float{});
}

}  // extern "C"
