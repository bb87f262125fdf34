// The whole layer for a few tokens (1 .. 64), forward only: a serving step.
//
// With a handful of rows per expert every product reads a weight matrix once
// and does almost no arithmetic on it, so the layer is a stream of the chosen
// experts' weights from HBM: bytes = hit * P * d * f * b (P = 2 matrices, 3
// for SwiGLU).  The grouped GEMM's 64-256-row tiles, its plan, its saved
// state and its row copies have nothing to give there.
//
// Kernels of a call:
//   few_gate     the gate's logits, one fixed-order fp32 chain per (token,
//                expert): the bits of moe_gate_topk (bf16: while each product
//                is zero or a normal fp32 number); then top-k and gate
//                weights, one wave per token (few_topk, with many experts)
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
#include <math.h>

#include <algorithm>
#include <type_traits>
#include <utility>

#include "common.h"

namespace moe {
namespace {

constexpr int kFewTokens = 64;          // most tokens of a call
constexpr int kFewSlots = 64;           // most experts per token

// ------------------------------------------------------------------- gate
// Maximum / minimum over the 64 lanes of a wave, by DPP moves as in
// wave_incl_scan (a lane without a source keeps its own value); all lanes
// active, the result in every lane.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
    auto step = [&](auto ctrl, auto rows) {
        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(
            (int)v, (int)v, decltype(ctrl)::value, decltype(rows)::value, 0xf, false);
        v = o > v ? o : v;
    };
    using std::integral_constant;
    step(integral_constant<int, 0x111>{}, integral_constant<int, 0xf>{});   // row_shr:1
    step(integral_constant<int, 0x112>{}, integral_constant<int, 0xf>{});   // row_shr:2
    step(integral_constant<int, 0x114>{}, integral_constant<int, 0xf>{});   // row_shr:4
    step(integral_constant<int, 0x118>{}, integral_constant<int, 0xf>{});   // row_shr:8
    step(integral_constant<int, 0x142>{}, integral_constant<int, 0xa>{});   // row_bcast:15
    step(integral_constant<int, 0x143>{}, integral_constant<int, 0xc>{});   // row_bcast:31
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Top-k and gate weights of one token by one wave: k rounds of an arg-max
// over (value descending, index ascending), then the softmax over the
// selected logits (renorm) or over all.  Lane l holds experts l, l + 64, ...
// (NQ of them); lane j gets the j-th choice and its weight.  k <= 64.
//
// The order is taken on the float's bits made monotone (both zeros alike, NaN
// below every number, 0 for an expert that is taken or does not exist), so
// that it is total and every lane agrees on the winner whatever x holds.
template <int NQ>
__device__ __forceinline__ void wave_topk(const float* lt, int E, int k, int renorm, int& idx,
                                          float& w) {
    const int lane = threadIdx.x & 63;
    float v[NQ];
    uint32_t key[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
        const int e = q * 64 + lane;
        v[q] = e < E ? lt[e] : 0.0f;
        const uint32_t b = __float_as_uint(v[q] + 0.0f);
        const uint32_t m = b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
        key[q] = e >= E ? 0u : v[q] != v[q] ? 1u : m;
    }
    float first = 0.0f, den = 0.0f;
    idx = 0;
    w = 0.0f;
    for (int j = 0; j < k; ++j) {
        uint32_t best = key[0];
        int bq = 0;
#pragma unroll
        for (int q = 1; q < NQ; ++q)
            if (key[q] > best) best = key[q], bq = q;      // the lane's lowest index on a tie
        const uint32_t top = wave_max_u32(best);
        // of the lanes that hold it, the one with the lowest expert index
        const int cand = best == top ? bq * 64 + lane : 0x7fffffff;
        const int e = NQ == 1 ? __ffsll((unsigned long long)__ballot(best == top)) - 1
                              : (int)~wave_max_u32(~(uint32_t)cand);
        const int src = e & 63, sq = e >> 6;
        float ev = v[0];
#pragma unroll
        for (int q = 1; q < NQ; ++q) ev = sq == q ? v[q] : ev;
        ev = __shfl(ev, src);
        if (lane == src) {
#pragma unroll
            for (int q = 0; q < NQ; ++q)
                if (sq == q) key[q] = 0u;
        }
        if (j == 0) first = ev;
        const float ex = expf(ev - first);
        den += ex;
        if (lane == j) idx = e, w = ex;
    }
    if (!renorm) {
        den = 0.0f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
            if (q * 64 + lane < E) den += expf(v[q] - first);
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) den += __shfl_xor(den, off);
    }
    w /= den;
}

// Logits of TB = 64 / EB tokens x EB experts per block, one chain per lane of
// wave 0.
//
// A chain's order is fixed (increasing feature index, each product and each
// sum rounded), so with few tokens its d dependent additions are the kernel's
// time and all else stays out of their way: wave 0 does nothing but read
// products from LDS, 32 features ahead of their use, and add.  Waves 1, 2, 3
// and 5 form the products, half a gate row per thread: they load x and the
// row NPF chunks of GK features ahead, multiply in fp32 (exactly, for bf16)
// and store them transposed, one row per chain, in a ring of three chunks:
// the chunk after the one being added is complete, so the reads ahead cross
// from chunk to chunk without a wait.
// Wave 4 does neither: waves go round the four SIMDs, and a second wave on the
// chain's SIMD would take issue slots from it.  Further waves only meet the
// barriers.  One token, 16 experts: 3.1 ns per feature (12 us at d 4096)
// after 3 us to start; additions alone would take 1.9 ns, the rest is the
// LDS reads, which hold the wave for about 10 clocks each.
// PACKED: gate rows of any length and alignment, loaded 16 bytes at a time all
// the same; what a row's last load finds behind it belongs to no expert.
constexpr int GK = 128, GROW = GK + 4;
struct GateLds {
    alignas(16) float ps[3][64 * GROW];
    float lg[64];
};

// Chunks in flight: eight take 0.3 us each, more than the latency of HBM.
constexpr int kGateAhead = 8;

typedef unsigned int u32x4_2_t __attribute__((ext_vector_type(4), aligned(2)));

// The logits of tokens t0 .. t0 + TB - 1 and experts e0 .. e0 + EB - 1 into
// s.lg [TB][EB], and into logits [T, E] when not NULL.
template <typename T, int EB, bool PACKED>
__device__ __forceinline__ void gate_block(GateLds& s, const T* __restrict__ x,
                                           const T* __restrict__ Wg,
                                           const float* __restrict__ bias, int Tn, int d, int E,
                                           int e0, int t0, float* __restrict__ logits) {
#pragma clang fp contract(off)
    constexpr int TB = 64 / EB, NPF = kGateAhead;
    static_assert(EB * sizeof(T) <= 128, "half a gate row of each chunk is held in registers");
    constexpr int VE = 16 / sizeof(T);
    constexpr int WL = EB / 2 / VE;                   // loads of half a gate row
    constexpr int G = 32;                             // features read ahead
    const int tid = threadIdx.x;
    // the wave number as a scalar: the roles are a uniform branch, and each
    // side meets the other's barriers, one per chunk
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nc = (d + GK - 1) / GK;

    if (wv == 4 || wv > 5) {
        for (int c = 0; c < nc; ++c) __syncthreads();
    } else if (wv > 0) {
        const int st = (tid - (wv == 5 ? 128 : 64)) % GK;             // feature of a chunk
        const int el = (tid - (wv == 5 ? 128 : 64)) / GK * (EB / 2);  // first expert
        u32x4_t wr[NPF][WL];
        T xr[NPF][TB];
        // Loads past the matrix read a valid element instead: features past d
        // are never summed, experts and tokens past the end never stored.
        // place: a load's element offset.  A packed one that would end behind
        // the last row starts earlier, and its value is shifted down by as much.
        const long last = (long)d * E - VE;
        auto place = [&](int c, int q, int& shift) {
            const long row = (long)min(c * GK + st, d - 1) * E;
            const int e = e0 + el + q * VE;
            if constexpr (!PACKED) return row + min(e, E - VE);
            const long off = row + (e < E ? e : 0);
            shift = (int)max(off - last, 0l);
            return off - shift;
        };
        auto fetch = [&](int c, u32x4_t (&w)[WL], T (&xv)[TB]) {
            int shift;
#pragma unroll
            for (int q = 0; q < WL; ++q) {
                const T* p = Wg + place(c, q, shift);
                if constexpr (PACKED) w[q] = *reinterpret_cast<const u32x4_2_t*>(p);
                else w[q] = *reinterpret_cast<const u32x4_t*>(p);
            }
#pragma unroll
            for (int t = 0; t < TB; ++t)
                xv[t] = x[(long)min(t0 + t, Tn - 1) * d + min(c * GK + st, d - 1)];
        };
        auto stash = [&](int c, int b, const u32x4_t (&w)[WL], const T (&xv)[TB]) {
            float xf[TB];
#pragma unroll
            for (int t = 0; t < TB; ++t) xf[t] = Elem<T>::ld(&xv[t]);
#pragma unroll
            for (int q = 0; q < WL; ++q) {
                u32x4_t raw = w[q];
                if (PACKED && c == nc - 1) {
                    int shift;
                    place(c, q, shift);
                    const unsigned __int128 v = __builtin_bit_cast(unsigned __int128, raw);
                    raw = __builtin_bit_cast(u32x4_t, v >> (shift * 8 * (int)sizeof(T)));
                }
                float o[VE];
                unpack16<T>(raw, o);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    if (t > 0 && t0 + t >= Tn) break;
#pragma unroll
                    for (int a = 0; a < VE; ++a)
                        s.ps[b][(t * EB + el + q * VE + a) * GROW + st] = xf[t] * o[a];
                }
            }
        };
#pragma unroll
        for (int c = 0; c < NPF; ++c) fetch(c, wr[c], xr[c]);
        // chunk c goes to LDS while the chains add chunk c - 2, over chunk c - 3
        int b = 0;
        for (int cb = 0; cb < nc; cb += NPF) {
#pragma unroll
            for (int u = 0; u < NPF; ++u) {
                const int c = cb + u;
                if (c >= nc) break;
                stash(c, b, wr[u], xr[u]);
                b = b == 2 ? 0 : b + 1;
                fetch(c + NPF, wr[u], xr[u]);
                __syncthreads();
            }
        }
    } else {
        float acc = 0.0f;
        float4 pv[2][G / 4];
        // Reads the next group, at p, then adds group b.  The fences keep the
        // compiler from moving the reads behind the additions; one wait for the
        // whole group (all but the G / 4 reads just issued) stands for the one
        // per read that it would place.
        static_assert(G / 4 == 8, "the wait below leaves 8 reads in flight");
        auto group = [&](const float* p, int b, bool add) {
#pragma unroll
            for (int q = 0; q < G / 4; ++q)
                pv[1 - b][q] = *reinterpret_cast<const float4*>(p + 4 * q);
            asm volatile("" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            if (!add) return;
            __builtin_amdgcn_s_waitcnt(0xc87f);                   // lgkmcnt(8)
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < G / 4; ++q) {
                acc = acc + pv[b][q].x;
                acc = acc + pv[b][q].y;
                acc = acc + pv[b][q].z;
                acc = acc + pv[b][q].w;
            }
            __builtin_amdgcn_sched_barrier(0);
        };
        __syncthreads();                                          // chunk 0 is in LDS
        group(s.ps[0] + tid * GROW, 1, false);
        int b = 0;
        for (int c = 0; c < nc; ++c) {
            if (c + 1 < nc) __syncthreads();                      // chunk c + 1 is in LDS
            const float* p = s.ps[b] + tid * GROW;
            b = b == 2 ? 0 : b + 1;
            const float* pn = s.ps[b] + tid * GROW;
            const int kn = min(GK, d - c * GK);                   // a multiple of 2 G
            for (int k0 = 0; k0 < kn; k0 += 2 * G) {
                group(p + k0 + G, 0, true);
                group(k0 + 2 * G < kn ? p + k0 + 2 * G : pn, 1, true);   // (the last: unused)
            }
        }
        const int e = e0 + tid % EB, t = t0 + tid / EB;
        if (bias) acc = acc + bias[min(e, E - 1)];
        s.lg[tid] = acc;
        if (logits && e < E && t < Tn) logits[(long)t * E + e] = acc;
    }
    __syncthreads();
}

template <typename T, int EB, bool PACKED>
__global__ __launch_bounds__(384) void few_gate_kernel(
    const T* __restrict__ x, const T* __restrict__ Wg, const float* __restrict__ bias, int Tn,
    int d, int E, int k, int renorm, float* __restrict__ logits, int32_t* __restrict__ topk_idx,
    float* __restrict__ topk_w) {
    constexpr int TB = 64 / EB;
    __shared__ GateLds s;
    const int t0 = blockIdx.y * TB;
    gate_block<T, EB, PACKED>(s, x, Wg, bias, Tn, d, E, blockIdx.x * EB, t0, logits);
    if (E > EB) return;                                           // few_topk follows
    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wv < TB && t0 + wv < Tn) {
        int e;
        float w;
        wave_topk<1>(s.lg + wv * EB, E, k, renorm, e, w);
        if (lane < k) {
            topk_idx[(long)(t0 + wv) * k + lane] = e;
            topk_w[(long)(t0 + wv) * k + lane] = w;
        }
    }
}

__global__ __launch_bounds__(256) void few_topk_kernel(const float* __restrict__ logits, int Tn,
                                                       int E, int k, int renorm,
                                                       int32_t* __restrict__ idx,
                                                       float* __restrict__ w) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (t >= Tn) return;
    int e;
    float we;
    wave_topk<16>(logits + (long)t * E, E, k, renorm, e, we);
    const int lane = threadIdx.x & 63;
    if (lane < k) {
        idx[(long)t * k + lane] = e;
        w[(long)t * k + lane] = we;
    }
}

template <typename T>
bool gate_rows_aligned(const void* Wg, int E) {
    return E % (int)(16 / sizeof(T)) == 0 && aligned16(Wg);
}

template <typename T, int EB>
void few_gate_go(const T* x, const T* Wg, const float* bias, int Tn, int d, int E, int k,
                 int renorm, float* logits, int32_t* idx, float* w, hipStream_t s) {
    const dim3 grid(cdiv(E, EB), cdiv(Tn, 64 / EB));
    if (EB > 32 || gate_rows_aligned<T>(Wg, E))
        MOE_LAUNCH("few_gate", s,
                   (few_gate_kernel<T, EB, false><<<grid, 384, 0, s>>>(x, Wg, bias, Tn, d, E, k,
                                                                       renorm, logits, idx, w)));
    else if constexpr (EB <= 32)
        MOE_LAUNCH("few_gate", s,
                   (few_gate_kernel<T, EB, true><<<grid, 384, 0, s>>>(x, Wg, bias, Tn, d, E, k,
                                                                      renorm, logits, idx, w)));
    if (E > EB)
        MOE_LAUNCH("few_topk", s,
                   (few_topk_kernel<<<cdiv(Tn, 4), 256, 0, s>>>(logits, Tn, E, k, renorm, idx,
                                                                w)));
}

template <typename T>
void few_gate(const T* x, const T* Wg, const float* bias, int Tn, int d, int E, int k, int renorm,
              float* logits, int32_t* idx, float* w, hipStream_t s) {
    // Up to 64 experts go in one block, which then also has the choice to make
    // (32 in fp32, whose rows are as long, or packed).  More go in blocks of 16,
    // whose loads are the least in the way of their chains, with the choice in a
    // launch of its own, about 3 us (one token, d 4096, 128 experts: bf16 18.5 us
    // against 24.3 in blocks of 64, fp32 19.8 against 34.8; 49 experts, packed:
    // 24.3 against 35.0).
    if constexpr (sizeof(T) == 2)
        if (E > 32 && E <= 64 && gate_rows_aligned<T>(Wg, E))
            return few_gate_go<T, 64>(x, Wg, bias, Tn, d, E, k, renorm, logits, idx, w, s);
    if (E > 16 && E <= 32)
        return few_gate_go<T, 32>(x, Wg, bias, Tn, d, E, k, renorm, logits, idx, w, s);
    few_gate_go<T, 16>(x, Wg, bias, Tn, d, E, k, renorm, logits, idx, w, s);
}

// ------------------------------------------------------- experts' row lists
struct RowsLds {
    uint32_t bits[32];
    int rows[kFewTokens], res[3];
};

// The rows of the `slot`-th expert (by index) that any token chose, as pair
// numbers t * k + j in increasing order (at most one per token) in r.rows, their
// number in *n and the pairs of the experts before it in *base.  Returns the
// expert, or -1 when fewer experts were hit.  Every thread of the block takes
// part.
__device__ __forceinline__ int expert_rows(const int32_t* __restrict__ idx, int pairs, int E,
                                           int slot, RowsLds& r, int* n, int* base) {
    const int tid = threadIdx.x, nthr = blockDim.x;
    if (tid < 32) r.bits[tid] = 0;
    __syncthreads();
    for (int p = tid; p < pairs; p += nthr) {
        const int e = idx[p];
        MOE_DASSERT((unsigned)e < (unsigned)E);
        if ((unsigned)e < (unsigned)E) atomicOr(&r.bits[e >> 5], 1u << (e & 31));
    }
    __syncthreads();
    if (tid < 64) {
        uint32_t b = tid < 32 ? r.bits[tid] : 0u;
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
        int cnt = 0, before = 0;
        if (e >= 0)
            for (int p0 = 0; p0 < pairs; p0 += 64) {
                const int p = p0 + tid;
                const int ep = p < pairs ? idx[p] : E;
                const uint64_t m = __ballot(ep == e);
                const int pos = cnt + __popcll(m & ((1ull << tid) - 1));
                if (ep == e && pos < kFewTokens) r.rows[pos] = p;
                cnt += __popcll(m);
                before += __popcll(__ballot(ep < e));
            }
        MOE_DASSERT(e < 0 || (cnt > 0 && cnt <= kFewTokens && before + cnt <= pairs));
        if (tid == 0) {
            r.res[0] = e;
            r.res[1] = min(cnt, kFewTokens);
            r.res[2] = before;
        }
    }
    __syncthreads();
    *n = r.res[1];
    *base = r.res[2];
    return r.res[0];
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
    // eight k of a token; LO: as the sum of two bf16
    template <bool LO> struct XRaw { u32x4_t v[LO ? 2 : 1]; };

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
            } else if constexpr (VW == 2) {
                r.w[i][0] = __builtin_nontemporal_load(
                    reinterpret_cast<const uint32_t*>(p + i * ldw));
            } else {
                typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
                const u32x2_t v = __builtin_nontemporal_load(
                    reinterpret_cast<const u32x2_t*>(p + i * ldw));
                r.w[i][0] = v[0];
                r.w[i][1] = v[1];
            }
        }
    }
    template <bool LO>
    static __device__ __forceinline__ void loadx(const bf16_t* x, long lo, int g, XRaw<LO>& r) {
        r.v[0] = ld16<false>(x + g * 8);
        if constexpr (LO) r.v[1] = ld16<false>(x + lo + g * 8);
    }
    template <int VW, int NT, bool LO>
    static __device__ __forceinline__ void mul(const Raw<VW>& r, const XRaw<LO> (&x)[NT],
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
            for (int i = 0; i < NT; ++i) {
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    av, __builtin_bit_cast(bf16x8, x[i].v[0]), acc[i][j], 0, 0, 0);
                if constexpr (LO)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        av, __builtin_bit_cast(bf16x8, x[i].v[1]), acc[i][j], 0, 0, 0);
            }
        }
    }
};

template <> struct Core<float> {
    static constexpr int KSTEP = 16;
    static constexpr int NL = 4;
    template <int VW> struct Raw { float w[NL][VW]; };
    template <bool LO> struct XRaw { f32x4 v; };

    template <int VW>
    static __device__ __forceinline__ void load(const float* W, long ldw, int k0, int g,
                                                Raw<VW>& r) {
        typedef float vec_t __attribute__((ext_vector_type(VW)));
        const float* p = W + (long)(k0 + g * 4) * ldw;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const vec_t v = __builtin_nontemporal_load(reinterpret_cast<const vec_t*>(p + i * ldw));
#pragma unroll
            for (int j = 0; j < VW; ++j) r.w[i][j] = v[j];
        }
    }
    template <bool LO>
    static __device__ __forceinline__ void loadx(const float* x, long, int g, XRaw<LO>& r) {
        r.v = *reinterpret_cast<const f32x4*>(x + g * 4);
    }
    template <int VW, int NT, bool LO>
    static __device__ __forceinline__ void mul(const Raw<VW>& r, const XRaw<LO> (&x)[NT],
                                               f32x4 (&acc)[NT][VW]) {
#pragma unroll
        for (int i = 0; i < NL; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j)
#pragma unroll
                for (int m = 0; m < NT; ++m)
                    acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(r.w[i][j], x[m].v[i],
                                                                    acc[m][j], 0, 0, 0);
    }
};

// x + xoff: each tile's token of this lane, its next step xstep elements on; lo:
// from a value to its rest.  NB - 1 steps are in flight while one is multiplied.
template <typename T, int VW, int NT, int NB, bool LO, typename Off>
__device__ __forceinline__ void strip_product(const T* W, long ldw, const T* x,
                                              const Off (&xoff)[NT], long xstep, long lo, int s0,
                                              int s1, f32x4 (&acc)[NT][VW]) {
    typedef Core<T> C;
    const int g = (threadIdx.x & 63) >> 4;
    typename C::template Raw<VW> wr[NB];
    typename C::template XRaw<LO> xr[NB][NT];
    auto fetch = [&](int s, int b) {
        C::template load<VW>(W, ldw, s * C::KSTEP, g, wr[b]);
#pragma unroll
        for (int i = 0; i < NT; ++i) 
            C::template loadx<LO>(x + s * xstep + xoff[i], lo, g, xr[b][i]);
    };
#pragma unroll
    for (int u = 0; u < NB - 1; ++u)
        if (s0 + u < s1) fetch(s0 + u, u);
    int s = s0;
    for (; s + 2 * NB - 1 <= s1; s += NB) {            // no branch between the loads
#pragma unroll
        for (int u = 0; u < NB; ++u) {
            fetch(s + u + NB - 1, (u + NB - 1) % NB);
            C::template mul<VW, NT, LO>(wr[u], xr[u], acc);
        }
    }
#pragma unroll
    for (int u = 0; u < 2 * NB - 2; ++u) {             // the last steps
        if (s + u >= s1) break;
        if (s + u + NB - 1 < s1) fetch(s + u + NB - 1, (u + NB - 1) % NB);
        C::template mul<VW, NT, LO>(wr[u % NB], xr[u % NB], acc);
    }
}

// The same for three and four tiles of bf16, whose accumulators leave registers
// for two steps of W and one of x: x of a step is asked for before W of the next,
// so that waiting for it leaves those weights in flight.  The order of the loads
// is the point, so it is held (left to the compiler's scheduling, which spills:
// 1194 us against 746, the down product of 34 rows for each of 32 experts, d 4096,
// f 14336).
template <typename T, int VW, int NT, bool LO, typename Off>
__device__ __forceinline__ void strip_tall(const T* W, long ldw, const T* x,
                                           const Off (&xoff)[NT], long xstep, long lo, int s0,
                                           int s1, f32x4 (&acc)[NT][VW]) {
    typedef Core<T> C;
    const int g = (threadIdx.x & 63) >> 4;
    typename C::template Raw<VW> wr[2];
    auto loadw = [&](int s, int b) { C::template load<VW>(W, ldw, s * C::KSTEP, g, wr[b]); };
    auto step = [&](int s, int b, bool more) {
        typename C::template XRaw<LO> xr[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) C::template loadx<LO>(x + s * xstep + xoff[i], lo, g, xr[i]);
        __builtin_amdgcn_sched_barrier(0);
        if (more) loadw(s + 1, b ^ 1);
        __builtin_amdgcn_sched_barrier(0);
        C::template mul<VW, NT, LO>(wr[b], xr, acc);
        __builtin_amdgcn_sched_barrier(0);
    };
    if (s0 < s1) loadw(s0, 0);
    int s = s0;
    for (; s + 3 <= s1; s += 2) {
        step(s, 0, true);
        step(s + 1, 1, true);
    }
    if (s < s1) step(s, 0, s + 1 < s1);
    if (s + 1 < s1) step(s + 1, 1, false);
}

// One wave's accumulators of 16 tokens into its LDS slab [16][BN + 4].
template <int VW>
__device__ __forceinline__ void slab_store(float* slab, const f32x4 (&acc)[VW]) {
    constexpr int LD = 16 * VW + 4;
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    float* p = slab + c * LD + g * 4 * VW;
#pragma unroll
    for (int q = 0; q < 4 * VW; q += 4)               // column q of the lane: row q / VW, j q % VW
        *reinterpret_cast<float4*>(p + q) =
            make_float4(acc[q % VW][q / VW], acc[(q + 1) % VW][(q + 1) / VW],
                        acc[(q + 2) % VW][(q + 2) / VW], acc[(q + 3) % VW][(q + 3) / VW]);
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
    const void* x;              // up: tokens [T, K]; down: h (bf16: and h_lo)
    const void *W, *W3;         // [E, K, N]
    const int32_t* idx;         // [pairs]
    void* out;                  // up: h [N / KSTEP][pairs][KSTEP] (bf16: and h_lo);
                                // down: partial [KS][pairs][N] fp32
    int pairs, k, E, K, N;
};
// The block's expert (the blockIdx.z-th that any pair chose) and its rows, or
// -1.  With one token the pairs' experts differ: the slot's own, and no search.
__device__ __forceinline__ int block_expert(const FewArgs& p, const int32_t* idx, RowsLds& r,
                                            int* n, int* base) {
    const int slot = blockIdx.z;
    if (p.pairs == p.k) {
        const int e = idx[slot];
        MOE_DASSERT((unsigned)e < (unsigned)p.E);
        // every wave writes the one row and reads what it wrote itself
        if ((threadIdx.x & 63) == 0) r.rows[0] = slot;
        __builtin_amdgcn_wave_barrier();
        *n = 1;
        *base = slot;
        return (unsigned)e < (unsigned)p.E ? e : -1;
    }
    return expert_rows(idx, p.pairs, p.E, slot, r, n, base);
}

// UP: h of pair p = act(x[p / k] W[e]) (DUAL: * x W3[e]) for the expert's pairs.
// Down (UP = false): partial[ks][p] = h[p] W[e] over the ks-th chunk of K.
// Grid: strips of 16 * VW columns, chunks, experts hit, in this order, so that the
// slots that no token filled come last (64 slots with 15 filled: the down product
// 30.0 us against 31.0 with the chunks last).  The NW waves of a block take
// consecutive parts of the chunk (DUAL: one half of them W, the other W3, which
// keeps the accumulators of a wave to one product); their sums meet in LDS (red:
// NW * 16 * (16 VW + 4) floats), in order.
//
// h is laid out for its one reader: the rows in the order of their experts, in
// blocks of KSTEP columns (64 bytes), so that the 16 tokens' 64 bytes of one
// step are eight whole cache lines; by token they were 16 half ones, and with
// few registers' worth of loads in flight the number of lines asked for is what
// bounds these kernels (T 64, d 4096, f 14336, 32 experts, two tiles to a wave: 768
// us against 825; as it is now, 662, 5.7 TB/s).
// h in bf16 is kept as the sum of two (h_lo, the rest that the first rounding
// left, follows h): the matrix cores wait for memory here anyway, and one
// rounding of h was the largest part of y's error (0.0024 of |y| against
// 0.0017 for y's own rounding).
template <typename T, int VW, int NTM, int NW, bool UP, bool DUAL>
__device__ __forceinline__ void product_block(const FewArgs& p, int e, int n, int base,
                                              const int* rows, float* red) {
    constexpr int KW = DUAL ? NW / 2 : NW;             // waves that share a product's chunk
    constexpr bool LO = !UP && sizeof(T) == 2;
    constexpr int KSTEP = Core<T>::KSTEP;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15;
    MOE_DASSERT(n > 0 && n <= 16 * NTM && base >= 0 && base + n <= p.pairs);
    const T* We = static_cast<const T*>(DUAL && wv >= KW ? p.W3 : p.W) + (long)e * p.K * p.N;
    const int n0 = blockIdx.x * 16 * VW;
    // NT tiles of 16 rows per wave, depth steps of registers
    auto body = [&](auto tiles, auto depth) {
        constexpr int NT = decltype(tiles)::value;
        constexpr int BN = 16 * VW, LD = BN + 4;
        const int steps = p.K / KSTEP;
        const int units = gridDim.y * KW, u = blockIdx.y * KW + wv % KW;
        const int s0 = (int)((long)steps * u / units), s1 = (int)((long)steps * (u + 1) / units);
        const T* x = static_cast<const T*>(p.x) + (UP ? 0 : (long)base * KSTEP);
        std::conditional_t<UP, long, int> xoff[NT];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int q = min(i * 16 + c, n - 1);          // rows past n: the last one's again
            if constexpr (UP) xoff[i] = (long)(rows[q] / p.k) * p.K;
            else xoff[i] = q * KSTEP;
        }
        f32x4 acc[NT][VW];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < VW; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // columns past N (a multiple of 64) read the last ones of the row instead
        const T* Wn = We + min(n0 + c * VW, p.N - VW);
        const long xstep = UP ? KSTEP : (long)p.pairs * KSTEP, lo = (long)p.pairs * p.K;
        if constexpr (sizeof(T) == 2 && NT > 2)
            strip_tall<T, VW, NT, LO>(Wn, p.N, x, xoff, xstep, lo, s0, s1, acc);
        else
            strip_product<T, VW, NT, decltype(depth)::value, LO>(Wn, p.N, x, xoff, xstep, lo, s0,
                                                                 s1, acc);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            if (i * 16 >= n) break;
            if (i > 0) __syncthreads();
            slab_store<VW>(red + wv * 16 * LD, acc[i]);
            __syncthreads();
            for (int q = tid; q < 16 * BN / 4; q += 64 * NW) {
                const int row = q / (BN / 4), cl = q % (BN / 4) * 4, r = i * 16 + row;
                if (r >= n || n0 + cl >= p.N) continue;
                const float4 s = slab_sum<VW, KW>(red, row, cl);
                float v[4] = {s.x, s.y, s.z, s.w};
                if constexpr (UP) {
                    if constexpr (DUAL) {
                        const float4 h3 = slab_sum<VW, KW>(red + KW * 16 * LD, row, cl);
                        v[0] = silu_f(v[0]) * h3.x;
                        v[1] = silu_f(v[1]) * h3.y;
                        v[2] = silu_f(v[2]) * h3.z;
                        v[3] = silu_f(v[3]) * h3.w;
                    } else {
#pragma unroll
                        for (int a = 0; a < 4; ++a) v[a] = gelu_f(v[a]);
                    }
                    const int hc = n0 + cl;
                    T* h = static_cast<T*>(p.out) +
                           ((long)(hc / KSTEP) * p.pairs + base + r) * KSTEP + hc % KSTEP;
                    store4(h, v);
                    if constexpr (sizeof(T) == 2) {
#pragma unroll
                        for (int a = 0; a < 4; ++a) {
                            const float hi = bf16_to_f32(f32_to_bf16(v[a]));
                            v[a] = fabsf(hi) < INFINITY ? v[a] - hi : 0.0f;   // NaN, infinity: hi
                        }
                        store4(h + (long)p.pairs * p.N, v);
                    }
                } else {
                    store4(static_cast<float*>(p.out) +
                               ((long)blockIdx.y * p.pairs + rows[r]) * p.N + n0 + cl, v);
                }
            }
        }
    };
    // The expert's rows in tiles of 16, one to four of them to a wave (34 rows for
    // each of 32 experts, down: three tiles 701 us, four 746)
    using std::integral_constant;
    constexpr integral_constant<int, 2> two{};
    if constexpr (NTM >= 4) {
        if (n > 48) return body(integral_constant<int, 4>{}, two);
        if (n > 32) return body(integral_constant<int, 3>{}, two);
    }
    if constexpr (NTM >= 2) {
        if (n > 16) return body(two, two);
    }
    // (one tile, fp32: three steps deep 151 us against 158 with four, one token
    // of d 4096, f 14336, 2 of 8 experts; bf16, half-width strips: four)
    body(integral_constant<int, 1>{},
         integral_constant<int, (VW == 8 || sizeof(T) == 4 ? 3 : 4)>{});
}

template <typename T, int VW, int NTM, int NW, bool UP, bool DUAL>
__global__ __launch_bounds__(64 * NW, 2) void few_product_kernel(FewArgs p) {
    __shared__ __attribute__((aligned(16))) float red[NW * 16 * (16 * VW + 4)];
    __shared__ RowsLds r;
    int n, base;
    const int e = block_expert(p, p.idx, r, &n, &base);
    if (e < 0) return;
    product_block<T, VW, NTM, NW, UP, DUAL>(p, e, n, base, r.rows, red);
}

// The gate and the up product in one launch, for a gate that one block of
// gate_block covers (E <= 16, T <= 4): every block works the same logits and
// choice out for itself, and the first one stores them.  That costs a read of
// the gate's matrix from L2 per block and saves a launch and the round trip
// of the choice through memory.
struct GateArgs {
    const void *x, *Wg;
    const float* bias;
    int T, d, renorm;
    float* logits;
    int32_t* idx;
    float* w;
};
template <typename T, bool PACKED, bool DUAL>
__global__ __launch_bounds__(512, 2) void few_gate_up_kernel(GateArgs g, FewArgs p) {
    constexpr int EB = 16, TB = 4, VW = 4, NW = 8;
    // the product's slabs take the gate's place once the choice is made
    __shared__ union {
        GateLds gate;
        alignas(16) float red[NW * 16 * (16 * VW + 4)];
    } s;
    __shared__ RowsLds r;
    __shared__ int32_t idx[TB * EB];                              // k <= E <= 16
    const bool first = blockIdx.x == 0 && blockIdx.z == 0;
    gate_block<T, EB, PACKED>(
        s.gate, static_cast<const T*>(g.x), static_cast<const T*>(g.Wg), g.bias, g.T, g.d, p.E, 0,
        0, first ? g.logits : nullptr);
    const int wv = threadIdx.x >> 6, lane = threadIdx.x & 63;
    if (wv < g.T) {
        int e;
        float w;
        wave_topk<1>(s.gate.lg + wv * EB, p.E, p.k, g.renorm, e, w);
        if (lane < p.k) {
            idx[wv * p.k + lane] = e;
            if (first) {
                g.idx[wv * p.k + lane] = e;
                g.w[wv * p.k + lane] = w;
            }
        }
    }
    __syncthreads();
    int n, base;
    const int e = block_expert(p, idx, r, &n, &base);
    if (e < 0) return;
    product_block<T, VW, 1, NW, true, DUAL>(p, e, n, base, r.rows, s.red);
}

// y[t] = sum over a token's k slots and ks chunks of w[t,j] partial[s][t k + j],
// rounded once.  A block takes 128 columns of one token; eight groups of 32
// threads take every eighth (slot, chunk) each, and meet in LDS, in order.  It is
// a launch and one round trip to memory long (3 to 5 us).  The down product's last
// block of a strip could take these sums over, in the same order, by a counter per
// strip; whether making the partial sums visible to a block of another XCD costs
// less than the launch is not measured.
constexpr int kCombineCols = 128;
template <typename T>
__global__ __launch_bounds__(256) void few_combine_kernel(const float* __restrict__ partial,
                                                          const float* __restrict__ w, int Tn,
                                                          int k, int d, int ks,
                                                          T* __restrict__ y) {
    __shared__ __attribute__((aligned(16))) float sums[8][kCombineCols];
    const int t = blockIdx.y, part = threadIdx.x >> 5;
    const int c = blockIdx.x * kCombineCols + (threadIdx.x & 31) * 4;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (c < d) {
        const float* p = partial + (long)t * k * d + c;
        const int n = k * ks;
#pragma unroll 4
        for (int q = part; q < n; q += 8) {
            const int z = q / k, j = q - z * k;
            const float4 a =
                *reinterpret_cast<const float4*>(p + ((long)z * Tn * k + j) * d);
            const float wj = w[t * k + j];
            v.x = fmaf(wj, a.x, v.x);
            v.y = fmaf(wj, a.y, v.y);
            v.z = fmaf(wj, a.z, v.z);
            v.w = fmaf(wj, a.w, v.w);
        }
    }
    *reinterpret_cast<float4*>(&sums[part][(threadIdx.x & 31) * 4]) = v;
    __syncthreads();
    if (part > 0 || c >= d) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) {
        const float4 a = *reinterpret_cast<const float4*>(&sums[q][threadIdx.x * 4]);
        v.x += a.x; v.y += a.y; v.z += a.z; v.w += a.w;
    }
    const float o[4] = {v.x, v.y, v.z, v.w};
    store4(y + (long)t * d + c, o);
}

// ------------------------------------------------------------------- plan
struct FewPlan {
    int slots;                   // experts hit at most
    bool fuse_gate;
    int up_vw, up_nw, up_strips, down_vw, down_nw, down_strips, ks;
    size_t logits, idx, w, h, partial, total;
};

constexpr double kFewWaves = 600, kChunkWaves = 6000;    // bf16, see few_plan
constexpr int kFewChunks = 16;

bool few_sizes_ok(int T, int d, int f, int E, int k, moe_act act, moe_dtype dt) {
    return T >= 0 && d >= 64 && d % 64 == 0 && f >= 64 && f % 64 == 0 && E >= 1 && E <= 1024 &&
           k >= 1 && k <= E && (act == MOE_ACT_GELU || act == MOE_ACT_SWIGLU) &&
           (dt == MOE_F32 || dt == MOE_BF16);
}
bool few_limits_ok(int T, int k) { return T <= kFewTokens && k <= kFewSlots; }

FewPlan few_plan(int T, int d, int f, int E, int k, moe_act act, moe_dtype dt) {
    FewPlan p;
    const int pairs = T * k;
    p.slots = min(E, pairs);
    const int wide = dt == MOE_BF16 ? 8 : 4;
    // Waves of a product over n columns, from the experts that T tokens hit
    // when the gate prefers none.  A skewed gate hits fewer, and then fewer waves
    // run than are aimed at: the choice is not known when the launch is made (T 48,
    // top-2 of 64 with popularity 1 / rank: 50 expected, 15 to 20 hit, and the down
    // product runs 1920 waves).
    const double hit = E * (1.0 - pow(1.0 - (double)k / E, T));
    auto waves = [&](int n, int vw, int nw) { return cdiv(n, 16 * vw) * hit * nw; };
    // Strips of 16 wide columns and 4 waves stream best (bf16: 256-byte pieces
    // of a row; one token of d 4096, f 14336, 8 of 32 experts: 476 us against
    // 503 with strips of half the width).  Below kFewWaves such waves there is
    // not enough in flight to cover the latency of HBM, and strips of half the
    // width with 8 waves are faster (d 4096, f 1536, 8 of 128 experts: 100
    // against 117 us; d 1024, f 4096, 2 of 8: 22.1 against 22.9).
    // fp32 has 64-column strips either way and half the bytes per wave and step:
    // 4 waves a block, or 8 below twice that number (same shape: 76 against 102).
    const double few = dt == MOE_BF16 ? kFewWaves : 2 * kFewWaves;
    p.up_vw = wide;
    p.up_nw = 4;
    // The gate's fusion: what one gate_block covers, in one round of blocks
    // (two rounds would work the gate out twice).  One token, d 1024, 8
    // experts: 21.4 us against 23.4 with a launch of its own.
    p.fuse_gate = E <= 16 && T <= 4 && cdiv(f, 64) * p.slots <= 256;
    if (p.fuse_gate || waves(f, wide, 4) < few) p.up_vw = 4, p.up_nw = 8;
    // Too few even of those (small f): half the width again, for twice the
    // compute units (two tokens, d 2368, f 832, 2 of 48 experts: bf16 15.6 us
    // against 17.6, fp32 23 against 31; more waves a block gained nothing.  With
    // 512 waves, bf16, one token, d 4096, f 512, 8 of 64: 19.0 against 18.4).
    if (!p.fuse_gate && T <= 16 && waves(f, 4, 8) < 0.75 * few) p.up_vw = 2;
    p.up_strips = cdiv(f, 16 * p.up_vw);
    // The down product's reduction f is long and its columns are few: chunks
    // of it until kChunkWaves waves run, each with at least 8 (narrow strips: 2)
    // steps to go: short blocks, since the experts with the most rows take
    // longest and may come last.  (T 48, d 1024, f 4096, 64 experts, this product:
    // 31 us with 6000 or 12000, 38 with 3000; T 64, d 4096, f 14336, 32 experts:
    // 662 with 6000, 668 with 3000, 694 with 12000; T 16, f 1024, whole pass: 78
    // unsplit, 81 in chunks of 4 steps.)
    const int steps = f / (dt == MOE_BF16 ? 32 : 16);
    auto chunks = [&](int vw, int nw, int least) {
        int ks = 1;
        while (ks < kFewChunks && waves(d, vw, nw) * ks < kChunkWaves &&
               steps >= ks * 2 * nw * least)
            ks *= 2;
        return ks;
    };
    p.down_vw = wide;
    p.down_nw = 4;
    int ks = chunks(wide, 4, 8);
    if (waves(d, wide, 4) * ks < few) {
        p.down_vw = 4;
        p.down_nw = 8;
        ks = chunks(4, 8, 2);
    }
    p.down_strips = cdiv(d, 16 * p.down_vw);
    p.ks = ks;
    const size_t es = dt == MOE_BF16 ? 2 : 4;
    p.logits = 0;
    p.idx = align_up(sizeof(float) * (size_t)T * E, 256);
    p.w = align_up(p.idx + sizeof(int32_t) * pairs, 256);
    p.h = align_up(p.w + sizeof(float) * pairs, 256);
    p.partial = align_up(p.h + (dt == MOE_BF16 ? 2 : 1) * es * pairs * f, 256);   // h, h_lo
    p.total = align_up(p.partial + sizeof(float) * (size_t)ks * pairs * d, 256);
    return p;
}

template <typename T, int NT>
moe_status few_run(const void* x, const void* Wg, const float* bias, const void* W1,
                   const void* W3, const void* W2, int Tn, int d, int f, int E, int k, int renorm,
                   moe_act act, const FewPlan& p, float* logits, int32_t* idx, float* w, void* y,
                   char* ws, hipStream_t s) {
    const int pairs = Tn * k;
    FewArgs u{x, W1, W3, idx, ws + p.h, pairs, k, E, d, f};
    const dim3 gu(p.up_strips, 1, p.slots), gd(p.down_strips, p.ks, p.slots);
    const bool sw = act == MOE_ACT_SWIGLU;
    if (!p.fuse_gate)
        few_gate<T>(static_cast<const T*>(x), static_cast<const T*>(Wg), bias, Tn, d, E, k, renorm,
                    logits, idx, w, s);
    auto product = [&](const char* name, auto up, auto dual, int vw, int nw, dim3 grid,
                       const FewArgs& a) {
        using std::integral_constant;
        auto go = [&](auto vwc, auto nwc) {
            constexpr int NWC = decltype(nwc)::value;
            MOE_LAUNCH(name, s,
                       (few_product_kernel<T, decltype(vwc)::value, NT, NWC, decltype(up)::value,
                                           decltype(dual)::value><<<grid, 64 * NWC, 0, s>>>(a)));
        };
        // few_plan's: the type's wide strips with 4 waves, narrower ones with 8
        constexpr integral_constant<int, sizeof(T) == 2 ? 8 : 4> wide{};
        if (nw == 4) return go(wide, integral_constant<int, 4>{});
        if constexpr (decltype(up)::value && NT == 1)
            if (vw == 2) return go(integral_constant<int, 2>{}, integral_constant<int, 8>{});
        go(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    };
    if (p.fuse_gate) {
        if constexpr (NT == 1) {
            const GateArgs g{x, Wg, bias, Tn, d, renorm, logits, idx, w};
            auto go = [&](auto packed, auto dual) {
                MOE_LAUNCH("few_gate_up", s,
                           (few_gate_up_kernel<T, decltype(packed)::value, decltype(dual)::value>
                            <<<gu, 512, 0, s>>>(g, u)));
            };
            if (gate_rows_aligned<T>(Wg, E)) {
                if (sw) go(std::false_type{}, std::true_type{});
                else go(std::false_type{}, std::false_type{});
            } else {
                if (sw) go(std::true_type{}, std::true_type{});
                else go(std::true_type{}, std::false_type{});
            }
        }
    } else if (sw) {
        product("few_up_swiglu", std::true_type{}, std::true_type{}, p.up_vw, p.up_nw, gu, u);
    } else {
        product("few_up_gelu", std::true_type{}, std::false_type{}, p.up_vw, p.up_nw, gu, u);
    }
    FewArgs v{ws + p.h, W2, nullptr, idx, ws + p.partial, pairs, k, E, f, d};
    product("few_down", std::false_type{}, std::false_type{}, p.down_vw, p.down_nw, gd, v);
    MOE_LAUNCH("few_combine", s,
               (few_combine_kernel<T><<<dim3(cdiv(d, kCombineCols), Tn), 256, 0, s>>>(
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
    // for every smaller step too: fewer tokens may cut the reduction into more chunks
    size_t most = 0;
    for (int t = 1; t <= T; ++t) most = std::max(most, few_plan(t, d, f, E, k, act, dt).total);
    return most;
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
    auto whole = [](const void* q, unsigned bytes) {       // at an element, or NULL
        return (reinterpret_cast<uintptr_t>(q) & (bytes - 1)) == 0;
    };
    MOE_CHECK_ARG(whole(Wg, dt == MOE_BF16 ? 2 : 4) && whole(logit_bias, 4) && whole(logits, 4) &&
                  whole(topk_idx, 4) && whole(topk_w, 4));
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
