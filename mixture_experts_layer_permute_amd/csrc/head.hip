// Losses over a vocabulary head: softmax cross entropy and distillation from
// a teacher's top scores, with the gradients of x and of the head.
//
//   z[t,v] = sum_i x[t,i] Wv[v,i]
//   lse_t  = ln sum_v exp z[t,v],  loss_t = lse_t - z[t,label_t]
//   q      = softmax over the teacher's slots of s / tau
//   kd_t   = tau^2 sum_j q_j (ln q_j - z[t,i_j] / tau + ln sum_v exp(z[t,v] / tau))
//   dz     = w_t (softmax(z_t) - [label]) + u_t tau (softmax(z_t / tau) - q)
//   dx = dz Wv,  dWv = dz^T x
//
// The tokens without a loss are left out first (a stable compaction, one
// index list); the rest goes in pieces of tokens whose scores fit the
// workspace.  A piece is three matrix products of 2 n d V operations and one
// pass over its scores:
//  head_scores  z of a 256 x 256 tile in the matrix cores; the epilogue
//               reduces every row's 128 columns to (max, sum of exp) from the
//               fp32 accumulators, so the normaliser needs no second look at
//               z, and z is stored (in fp32) only when something reads it;
//  head_dz      z -> dz in place, one wave a row: no barriers, as a wave's
//               stores at half the element size stay behind its loads;
//  head_product dx = dz Wv (split over the vocabulary when the tiles are few)
//               and dWv = dz^T x, summed over the pieces in fp32.
// Nothing is computed twice: 6 n d V operations, the least there is with z
// not kept beyond its piece.  The other way, keeping no scores and computing
// them again for dz, costs 8 n d V.
//
// Roundings (bf16): dz is rounded once to bf16 as an operand of the matrix
// cores; every sum is fp32; dx and dWv are rounded once.
#include <algorithm>

#include "common.h"
#include "mfma_tile.h"

namespace moe {
namespace {

constexpr int kMaxK = 256;              // teacher slots of a token
constexpr int kRowAlign = 256;          // tokens of a piece: whole row tiles

// A wave's lane reads and writes ordered as written: the reads before it have
// returned, the writes before it are done.
__device__ __forceinline__ void wave_mem_sync() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Sum or maximum over groups of 8 or 16 neighbouring lanes, in every lane of
// the group: quad swaps, then the mirror of 8, then the mirror of 16 lanes
// (mirrors, since the smaller groups' lanes agree by then).  Every lane of the
// wave must be active.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ float group_max(float v) {
    v = fmaxf(v, dpp<0xB1>(v));                    // quad_perm 1,0,3,2
    v = fmaxf(v, dpp<0x4E>(v));                    // quad_perm 2,3,0,1
    v = fmaxf(v, dpp<0x141>(v));                   // row_half_mirror
    if constexpr (N == 16) v = fmaxf(v, dpp<0x140>(v));   // row_mirror
    return v;
}
template <int N>
__device__ __forceinline__ float group_sum(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    if constexpr (N == 16) v += dpp<0x140>(v);
    return v;
}
__device__ __forceinline__ float wave_max(float v) {
    v = group_max<16>(v);
    v = fmaxf(v, __shfl_xor(v, 16));
    return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float wave_sum(float v) {
    v = group_sum<16>(v);
    v += __shfl_xor(v, 16);
    return v + __shfl_xor(v, 32);
}

// ------------------------------------------------------- tokens with a loss

__device__ __forceinline__ bool in_vocab(int v, int V) { return (unsigned)v < (unsigned)V; }

// act[t]: whether token t has a label or a teacher's slot (one wave a token).
__global__ __launch_bounds__(256) void head_active_kernel(const int32_t* __restrict__ labels,
                                                          const int32_t* __restrict__ tidx,
                                                          int T, int K, int V,
                                                          int32_t* __restrict__ act) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (t >= T) return;
    bool on = labels && in_vocab(labels[t], V);
    for (int j = lane; j < K && !on; j += 64) on = in_vocab(tidx[(long)t * K + j], V);
    const bool any = __ballot(on) != 0;
    if (lane == 0) act[t] = any ? 1 : -1;
}

// rows[0..n) = the tokens that have a loss, in order; *count = n; the outputs
// of the others are zero.  act: labels (limit V) or head_active's (limit 2).
// One block: each round takes 4096 tokens, four a thread.
__global__ __launch_bounds__(1024) void head_compact_kernel(const int32_t* __restrict__ act,
                                                            int T, int limit,
                                                            int32_t* __restrict__ rows,
                                                            int32_t* __restrict__ count,
                                                            float* __restrict__ o0,
                                                            float* __restrict__ o1,
                                                            float* __restrict__ o2) {
    __shared__ int sh[16];
    int base = 0;
    for (int t0 = 0; t0 < T; t0 += 4096) {
        const int t = t0 + threadIdx.x * 4;
        bool on[4];
        int c = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            on[q] = t + q < T && in_vocab(act[min(t + q, T - 1)], limit);
            c += on[q];
        }
        int total;
        int at = base + block_excl_scan<1024>(c, sh, &total);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (on[q]) {
                MOE_DASSERT(at >= 0 && at < T);
                rows[at++] = t + q;
            } else if (t + q < T) {
                if (o0) o0[t + q] = 0.0f;
                if (o1) o1[t + q] = 0.0f;
                if (o2) o2[t + q] = 0.0f;
            }
        }
        base += total;
    }
    if (threadIdx.x == 0) *count = base;
}

// The active rows of one piece (of `piece` rows from compacted row p0 on).
__device__ __forceinline__ int piece_rows(const int32_t* count, int p0, int piece, int fixed) {
    const int n = count ? *count : fixed;
    return max(0, min(n - p0, piece));
}

// xc[r] = x[rows[p0 + r]] for the piece's rows; with dx (first piece) also
// dx[t] = 0 for the tokens without a loss.  vpr: 16-byte vectors of a row.
__global__ __launch_bounds__(256) void head_gather_kernel(
    const u32x4_t* __restrict__ x, const int32_t* __restrict__ rows,
    const int32_t* __restrict__ count, int p0, int piece, int vpr, u32x4_t* __restrict__ xc,
    const int32_t* __restrict__ act, int T, int limit, u32x4_t* __restrict__ dx) {
    const int n = piece_rows(count, p0, piece, 0);
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    const long r = i / vpr;
    const int c = (int)(i - r * vpr);
    if (r < n) {
        const int t = rows[p0 + r];
        MOE_DASSERT(t >= 0 && t < T);
        xc[r * vpr + c] = x[(long)t * vpr + c];
    }
    if (dx && r < T && !in_vocab(act[r], limit)) dx[r * vpr + c] = u32x4_t{0, 0, 0, 0};
}

__global__ __launch_bounds__(256) void head_zero_kernel(u32x4_t* __restrict__ p, long n) {
    const long i = (long)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = u32x4_t{0, 0, 0, 0};
}

// ------------------------------------------------------- matrix products

// C [M,N] = A . B over K, in `splits` parts of the reduction.  Of M and K one
// may be the piece's rows, known on the device only (dyn).
template <typename T>
struct HeadGemm {
    const T* A;
    long lda;
    const T* B;
    long ldb;
    int M, N, K;
    int dyn;                 // 1: M, 2: K is the piece's rows (0: neither)
    const int32_t* count;
    int p0, piece;
    int splits;
    int xcd_run;
};

struct HeadTile {
    int m0, n0, rows, cols;  // tile origin, valid rows and columns
    int M;
    int k0, k1;              // this part of the reduction
    int split;
    bool live;
};

// Tiles in groups of 8 row tiles, every column tile of a group before the
// next group, row tiles fastest: a run of 32 on one XCD is 8 x 4 tiles, which
// share their operands in its L2.  The parts of the reduction go one after the other.
template <int BM, int BN, typename T>
__device__ __forceinline__ HeadTile head_tile(const HeadGemm<T>& p) {
    HeadTile t;
    const int n = p.dyn ? piece_rows(p.count, p.p0, p.piece, p.piece) : 0;
    t.M = p.dyn == 1 ? n : p.M;
    const int K = p.dyn == 2 ? n : p.K;
    const int nM = (t.M + BM - 1) / BM, nN = (p.N + BN - 1) / BN;
    const int L = xcd_logical(blockIdx.x, p.xcd_run);
    t.live = L < nM * nN * p.splits;
    if (!t.live) return t;
    t.split = L / (nM * nN);
    const int w0 = L - t.split * (nM * nN);
    const int first = (w0 / (8 * nN)) * 8;
    const int gm = min(8, nM - first);
    const int w = w0 - first * nN;
    t.m0 = (first + w % gm) * BM;
    t.n0 = (w / gm) * BN;
    t.rows = min(BM, t.M - t.m0);
    t.cols = min(BN, p.N - t.n0);
    const int kc = ((K + p.splits - 1) / p.splits + 63) / 64 * 64;
    t.k0 = min(K, t.split * kc);
    t.k1 = min(K, t.k0 + kc);
    return t;
}

// Epilogue: each wave stages 16-row slabs of its accumulators (32 x 32
// fragments of the matrix instructions: column = lane % 32, row by register
// and lane / 32) in its own part of LDS and hands rows of 8 neighbouring
// columns to epi.row8(tile, row, col, v).  Every lane takes part in every
// call; rows and columns past the tile are up to the functor.
template <int WTM, int WTN, int FM, int FN, class Epi>
__device__ __forceinline__ void head_epilogue(float* slab, const HeadTile& ti, int wr, int wc,
                                              const f32x16 (&acc)[FM][FN], const Epi& epi) {
    constexpr int LDW = WTN + 4;
    constexpr int LPR = WTN / 8;                   // lanes of a row
    constexpr int RPP = 64 / LPR;
    const int lane = threadIdx.x & 63;
    const int c0 = (lane % LPR) * 8;
#pragma unroll
    for (int q = 0; q < 2 * FM; ++q) {
        const int i = q >> 1, h = q & 1;
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int vv = 0; vv < 8; ++vv) {
                const int r = (vv >> 2) * 8 + (lane >> 5) * 4 + (vv & 3);
                slab[r * LDW + j * 32 + (lane & 31)] = acc[i][j][h * 8 + vv];
            }
        wave_lds_sync();
#pragma unroll 1
        for (int ps = 0; ps < 16 / RPP; ++ps) {
            const int rl = ps * RPP + lane / LPR;
            const float* src = &slab[rl * LDW + c0];
            float v[8];
            *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(src);
            *reinterpret_cast<float4*>(v + 4) = *reinterpret_cast<const float4*>(src + 4);
            epi.template row8<LPR>(ti, wr + i * 32 + h * 16 + rl, wc + c0, v);
        }
        wave_lds_sync();
    }
}

// Scores: per row and 128 (64 in fp32) columns the maximum m and the sums of
// exp(z - m) and exp((z - m) / tau); the label's score; z itself if kept.
struct EpiScores {
    int V;
    float2* stat;            // [parts][ldr] (m, sum)
    float* tstat;            // [parts][ldr] sum at the temperature, or NULL
    float inv_tau;
    long ldr;
    const int32_t* labels;   // or NULL
    const int32_t* rows;     // compacted row -> token, or NULL: the row itself
    int p0;
    float* zl;               // [rows] label's score
    float* Z;                // or NULL
    long ldz;                // a multiple of 64

    template <int LPR>
    __device__ __forceinline__ void row8(const HeadTile& ti, int rl, int cl,
                                         const float* v) const {
        const int col = ti.n0 + cl;
        const bool in = rl < ti.rows;
        const long r = (long)ti.m0 + rl;
        float m = -INFINITY;
#pragma unroll
        for (int q = 0; q < 8; ++q) m = fmaxf(m, col + q < V ? v[q] : -INFINITY);
        m = group_max<LPR>(m);
        const float ref = m == -INFINITY ? 0.0f : m;   // no column here, or none finite
        float s = 0.0f, st = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += col + q < V ? expf(v[q] - ref) : 0.0f;
        s = group_sum<LPR>(s);
        if (tstat) {
#pragma unroll
            for (int q = 0; q < 8; ++q) st += col + q < V ? expf((v[q] - ref) * inv_tau) : 0.0f;
            st = group_sum<LPR>(st);
        }
        if (!in) return;
        if ((threadIdx.x & (LPR - 1)) == 0) {
            const long at = (long)(col / (LPR * 8)) * ldr + r;
            stat[at] = make_float2(m, s);
            if (tstat) tstat[at] = st;
        }
        if (labels) {
            const int t = rows ? rows[p0 + r] : (int)r;
            const int y = labels[t] - col;
            if ((unsigned)y < 8u && col + y < V) {
                uint32_t z = 0;                    // (not an indexed read: v stays in registers)
#pragma unroll
                for (int q = 0; q < 8; ++q) z |= y == q ? __float_as_uint(v[q]) : 0u;
                zl[r] = __uint_as_float(z);
            }
        }
        if (Z && col < ldz) {
            float4* q = reinterpret_cast<float4*>(Z + r * ldz + col);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
    }
};

template <typename T>
__device__ __forceinline__ void st8(T* p, const float* v) {
    Vec16<T>::st(p, v);
    if constexpr (sizeof(T) == 4) Vec16<T>::st(p + 4, v + 4);
}
template <typename T>
__device__ __forceinline__ void ld8(const T* p, float* v) {
    Vec16<T>::ld(p, v);
    if constexpr (sizeof(T) == 4) Vec16<T>::ld(p + 4, v + 4);
}

// dx rows, back at their tokens.
template <typename T>
struct EpiRows {
    T* out;
    long ldo;
    const int32_t* rows;
    int p0;
    template <int LPR>
    __device__ __forceinline__ void row8(const HeadTile& ti, int rl, int cl,
                                         const float* v) const {
        if (rl < ti.rows && cl < ti.cols)
            st8(out + (long)rows[p0 + ti.m0 + rl] * ldo + ti.n0 + cl, v);
    }
};

// One part of a split reduction, fp32.
struct EpiPart {
    float* part;
    long ldo, stride;
    template <int LPR>
    __device__ __forceinline__ void row8(const HeadTile& ti, int rl, int cl,
                                         const float* v) const {
        if (rl < ti.rows && cl < ti.cols)
            st8(part + ti.split * stride + (long)(ti.m0 + rl) * ldo + ti.n0 + cl, v);
    }
};

// dWv over the pieces: the running sum in fp32, the last piece rounds it.
template <typename T>
struct EpiSum {
    T* out;
    float* acc;
    long ldo;
    const int32_t* count;
    int p0, piece;
    template <int LPR>
    __device__ __forceinline__ void row8(const HeadTile& ti, int rl, int cl, float* v) const {
        if (rl >= ti.rows || cl >= ti.cols) return;
        const long at = (long)(ti.m0 + rl) * ldo + ti.n0 + cl;
        if (p0 > 0) {
            float a[8];
            ld8(acc + at, a);
#pragma unroll
            for (int q = 0; q < 8; ++q) v[q] += a[q];
        }
        if (*count <= p0 + piece) st8(out + at, v);
        else st8(acc + at, v);
    }
};

// A piece past the last token adds nothing to dWv (the first always runs: it
// writes the zeros of a batch without a loss).
template <typename T>
__device__ __forceinline__ bool piece_done(const HeadGemm<T>& p) {
    return p.dyn == 2 && p.p0 > 0 && *p.count <= p.p0;
}

// bf16: BM x BN tiles, WM x WN waves, operands straight from HBM into a ring
// of NSTG stages of BK steps, fragments double-buffered over the stages (the
// main loop of the expert products, ggemm_bf16_dma_kernel).
template <int BM, int BN, int WM, int WN, int NSTG, int BK, int ALAY, int BLAY, class Epi>
__global__ __launch_bounds__(64 * WM * WN, 2) void head_product_kernel(HeadGemm<bf16_t> p,
                                                                       Epi epi) {
    constexpr int NT = 64 * WM * WN;
    constexpr int WTM = BM / WM, WTN = BN / WN;
    constexpr int FM = WTM / 32, FN = WTN / 32;
    constexpr int A_BYTES = BM * BK * 2, B_BYTES = BN * BK * 2;
    constexpr int STAGE = A_BYTES + B_BYTES;
    constexpr int SLAB = 16 * (WTN + 4) * 4;
    static_assert(NSTG * STAGE <= 160 * 1024 && WM * WN * SLAB <= NSTG * STAGE, "LDS");
    __shared__ __attribute__((aligned(1024))) uint8_t ringbuf[NSTG * STAGE];
    if (piece_done(p)) return;
    const HeadTile ti = head_tile<BM, BN>(p);
    if (!ti.live) return;
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    const int wm = wv / WN, wn = wv % WN;

    DmaOperand<BM, ALAY, NT, BK> opA;
    DmaOperand<BN, BLAY, NT, BK> opB;
    opA.init(p.A + (ALAY == KMAJ ? (long)ti.m0 * p.lda : (long)ti.m0), p.lda, ti.rows, ti.k1);
    opB.init(p.B + (BLAY == KMAJ ? (long)ti.n0 * p.ldb : (long)ti.n0), p.ldb, ti.cols, ti.k1);
    constexpr int NL = DmaOperand<BM, ALAY, NT, BK>::NLOAD + DmaOperand<BN, BLAY, NT, BK>::NLOAD;
    static_assert(NL * (NSTG - 1) <= 63, "vmcnt counts at most 63 loads");

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    constexpr int KS = BK / 16;
    static_assert(KS % 2 == 0, "fragment buffer parity assumes an even count");
    bf16x8 af[2][FM], bfr[2][FN];
    auto issue = [&](uint8_t* stg, int j) {
        const long k = (long)ti.k0 + (long)j * BK;
        opA.dma(k, stg);
        opB.dma(k, stg + A_BYTES);
    };
    auto read_frags = [&](const uint8_t* stg, int ks, int buf) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
            af[buf][i] = dma_frag<BM, ALAY, BK>(stg, wm * WTM + i * 32, ks, lane);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            bfr[buf][j] = dma_frag<BN, BLAY, BK>(stg + A_BYTES, wn * WTN + j * 32, ks, lane);
    };
    auto mfmas = [&](int buf) {
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
            for (int j = 0; j < FN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[buf][i], bfr[buf][j],
                                                                   acc[i][j], 0, 0, 0);
    };
    auto ring = [&](int q) -> uint8_t* { return ringbuf + q * STAGE; };
    const int nj = (ti.k1 - ti.k0 + BK - 1) / BK;
    constexpr int NP = ALAY == KMAJ && BLAY == KMAJ ? NSTG : NSTG - 1;
#pragma unroll
    for (int q = 0; q < NP; ++q)
        if (q < nj) issue(ring(q), q);
    stage_barrier_ahead<NL, NP - 1>(min(nj - 1, NP - 1));   // stage 0 landed
    if (nj > 0) read_frags(ring(0), 0, 0);
    int qc = 0;                                        // ring slot of stage j
#pragma unroll 1
    for (int j = 0; j + 1 < nj; ++j) {
        const uint8_t* cur = ring(qc);
        const int qn = qc + 1 == NSTG ? 0 : qc + 1;    // slot of stage j+1
        const int qf = qc == 0 ? NSTG - 1 : qc - 1;    // slot of stage j-1 = j+NSTG-1
        // every read of stage j-1 returned before the barrier that opened stage j
        if ((NP < NSTG || j > 0) && j + NSTG - 1 < nj) issue(ring(qf), j + NSTG - 1);
#pragma unroll
        for (int ks = 0; ks + 1 < KS; ++ks) {
            read_frags(cur, ks + 1, (ks + 1) & 1);
            mfmas(ks & 1);
        }
        stage_barrier_ahead<NL, NSTG - 2>(min(nj - 2 - j, NSTG - 2));  // stage j+1 landed
        read_frags(ring(qn), 0, 0);
        mfmas((KS - 1) & 1);
        qc = qn;
    }
    if (nj > 0) {
        const uint8_t* cur = ring(qc);
#pragma unroll
        for (int ks = 0; ks + 1 < KS; ++ks) {
            read_frags(cur, ks + 1, (ks + 1) & 1);
            mfmas(ks & 1);
        }
        mfmas((KS - 1) & 1);
    }
    __syncthreads();
    head_epilogue<WTM, WTN>(reinterpret_cast<float*>(ringbuf + wv * SLAB), ti, wm * WTM,
                            wn * WTN, acc, epi);
}

// fp32: 128 x 128 tiles, 4 waves of 64 x 64, v_mfma_f32_32x32x2_f32; tiles
// staged through registers into k-major LDS, the next ones loaded during the
// products of these.
constexpr int FBM = 128, FBK = 16;
template <int ALAY, int BLAY, class Epi>
__global__ __launch_bounds__(256, 2) void head_product_f32_kernel(HeadGemm<float> p, Epi epi) {
    constexpr int LDT = FBM + 4;
    constexpr int SLABF = 16 * (64 + 4);
    __shared__ __attribute__((aligned(16))) float lds[2 * 2 * FBK * LDT];
    static_assert(4 * SLABF <= 4 * FBK * LDT, "epilogue slabs");
    if (piece_done(p)) return;
    const HeadTile ti = head_tile<FBM, FBM>(p);
    if (!ti.live) return;
    const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
    const int wm = wv >> 1, wn = wv & 1;
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    // two 16-byte vectors of each operand's stage a thread
    float4 ra[2], rb[2];
    auto load = [&](const float* P, long ld, int lay, int lim, int k, float4* r) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = tid + 256 * u;
            float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (lay == KMAJ) {
                const int row = i >> 2, kk = k + (i & 3) * 4;
                if (row < lim && kk < ti.k1) {
                    const float4 v = *reinterpret_cast<const float4*>(P + row * ld + kk);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                }
            } else {
                const int kk = k + (i >> 5), c = (i & 31) * 4;
                if (kk < ti.k1 && c < lim) {
                    const float4 v = *reinterpret_cast<const float4*>(P + kk * ld + c);
                    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
                }
            }
            r[u] = make_float4(w[0], w[1], w[2], w[3]);
        }
    };
    auto store = [&](float* s, int lay, const float4* r) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int i = tid + 256 * u;
            if (lay == KMAJ) {
                const int row = i >> 2, kk = (i & 3) * 4;
                s[(kk + 0) * LDT + row] = r[u].x;
                s[(kk + 1) * LDT + row] = r[u].y;
                s[(kk + 2) * LDT + row] = r[u].z;
                s[(kk + 3) * LDT + row] = r[u].w;
            } else {
                *reinterpret_cast<float4*>(s + (i >> 5) * LDT + (i & 31) * 4) = r[u];
            }
        }
    };
    const float* A = p.A + (ALAY == KMAJ ? (long)ti.m0 * p.lda : (long)ti.m0);
    const float* B = p.B + (BLAY == KMAJ ? (long)ti.n0 * p.ldb : (long)ti.n0);
    const int nj = (ti.k1 - ti.k0 + FBK - 1) / FBK;
    auto bufA = [&](int b) { return lds + b * 2 * FBK * LDT; };
    auto bufB = [&](int b) { return lds + (b * 2 + 1) * FBK * LDT; };
    if (nj > 0) {
        load(A, p.lda, ALAY, ti.rows, ti.k0, ra);
        load(B, p.ldb, BLAY, ti.cols, ti.k0, rb);
        store(bufA(0), ALAY, ra);
        store(bufB(0), BLAY, rb);
        __syncthreads();
    }
#pragma unroll 1
    for (int j = 0; j < nj; ++j) {
        const bool more = j + 1 < nj;
        if (more) {
            load(A, p.lda, ALAY, ti.rows, ti.k0 + (j + 1) * FBK, ra);
            load(B, p.ldb, BLAY, ti.cols, ti.k0 + (j + 1) * FBK, rb);
        }
        const float* sa = bufA(j & 1) + wm * 64 + (lane & 31);
        const float* sb = bufB(j & 1) + wn * 64 + (lane & 31);
#pragma unroll
        for (int kk = 0; kk < FBK; kk += 2) {
            const int o = (kk + (lane >> 5)) * LDT;
            const float a0 = sa[o], a1 = sa[o + 32], b0 = sb[o], b1 = sb[o + 32];
            acc[0][0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a0, b0, acc[0][0], 0, 0, 0);
            acc[0][1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a0, b1, acc[0][1], 0, 0, 0);
            acc[1][0] = __builtin_amdgcn_mfma_f32_32x32x2f32(a1, b0, acc[1][0], 0, 0, 0);
            acc[1][1] = __builtin_amdgcn_mfma_f32_32x32x2f32(a1, b1, acc[1][1], 0, 0, 0);
        }
        if (more) {                    // the other buffer: read two stages ago
            store(bufA((j + 1) & 1), ALAY, ra);
            store(bufB((j + 1) & 1), BLAY, rb);
        }
        __syncthreads();
    }
    head_epilogue<64, 64>(lds + wv * SLABF, ti, wm * 64, wn * 64, acc, epi);
}

// out = the parts of a split reduction added in order, for dx (rows != NULL:
// row r goes to token rows[p0 + r]) or dWv (the pieces' running sum as in
// EpiSum).  8 elements a thread; n8 = M * N / 8, N a multiple of 8.
template <typename T>
__global__ __launch_bounds__(256) void head_join_kernel(const float* __restrict__ part, int splits,
                                                        long stride, long n8, int N,
                                                        T* __restrict__ out,
                                                        const int32_t* __restrict__ rows,
                                                        float* __restrict__ acc,
                                                        const int32_t* __restrict__ count, int p0,
                                                        int piece) {
    const long i = ((long)blockIdx.x * 256 + threadIdx.x) * 8;
    if (i >= n8 * 8) return;
    const int have = *count;
    const long r = i / N;
    if (rows ? r >= have - p0 : (p0 > 0 && have <= p0)) return;
    float v[8];
    ld8(part + i, v);
    for (int s = 1; s < splits; ++s) {
        float a[8];
        ld8(part + s * stride + i, a);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += a[q];
    }
    if (rows) {
        st8(out + (long)rows[p0 + r] * N + (i - r * N), v);
        return;
    }
    if (p0 > 0) {
        float a[8];
        ld8(acc + i, a);
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] += a[q];
    }
    if (have <= p0 + piece) st8(out + i, v);
    else st8(acc + i, v);
}

// --------------------------------------------------------- normalisers

// lse (and that at the temperature, relative to the same maximum) of a
// piece's rows from the parts: 64 rows a block, its 16 waves share the parts.
// The loss of a labelled row goes to its token.
__global__ __launch_bounds__(1024) void head_lse_kernel(
    const float2* __restrict__ stat, const float* __restrict__ tstat, int parts, long ldr,
    float inv_tau, const float* __restrict__ zl, const int32_t* __restrict__ labels, int V,
    const int32_t* __restrict__ rows, const int32_t* __restrict__ count, int fixed, int p0,
    int piece, float* __restrict__ row_lse, float* __restrict__ row_tlse,
    float* __restrict__ loss, float* __restrict__ lse) {
    __shared__ float sm[16][64], ss[16][64], st[16][64];
    const int n = piece_rows(count, p0, piece, fixed);
    if (blockIdx.x * 64 >= n) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const long r = (long)blockIdx.x * 64 + lane;
    float m = -INFINITY, s = 0.0f, t = 0.0f;
    if (r < n) {
        for (int q = w; q < parts; q += 16) {
            const float2 a = stat[q * ldr + r];
            if (a.x == -INFINITY) {
                s += a.y, t += tstat ? tstat[q * ldr + r] : 0.0f;   // no column: 0 (or a NaN)
                continue;
            }
            const float mx = fmaxf(m, a.x);
            const float k0 = m == -INFINITY ? 0.0f : expf(m - mx), k1 = expf(a.x - mx);
            s = s * k0 + a.y * k1;
            if (tstat) {
                const float j0 = m == -INFINITY ? 0.0f : expf((m - mx) * inv_tau);
                t = t * j0 + tstat[q * ldr + r] * expf((a.x - mx) * inv_tau);
            }
            m = mx;
        }
    }
    sm[w][lane] = m, ss[w][lane] = s, st[w][lane] = t;
    __syncthreads();
    if (w != 0 || r >= n) return;
    for (int q = 1; q < 16; ++q) m = fmaxf(m, sm[q][lane]);
    s = 0.0f, t = 0.0f;
    for (int q = 0; q < 16; ++q) {
        const float d = sm[q][lane] == -INFINITY ? 0.0f : sm[q][lane] - m;
        s += ss[q][lane] * expf(d);
        t += st[q][lane] * expf(d * inv_tau);
    }
    const float l = m + logf(s);
    if (row_lse) row_lse[r] = l;
    if (row_tlse) row_tlse[r] = m * inv_tau + logf(t);
    const int tok = rows ? rows[p0 + r] : (int)r;
    if (labels) {
        const bool on = in_vocab(labels[tok], V);
        if (loss) loss[tok] = on ? l - zl[r] : 0.0f;
        if (lse) lse[tok] = on ? l : 0.0f;
    }
}

// ----------------------------------------------------------------- dz

struct HeadDz {
    float* Z;                // [piece][ldz]; dz takes its place, from each row's start
    long ldz;
    int V;
    const int32_t* rows;
    const int32_t* count;
    int p0, piece;
    const float* lse;        // of the row, and at the temperature
    const float* tlse;
    const int32_t* labels;   // or NULL
    const float* weight;     // [T] or NULL: 1
    const int32_t* tidx;     // [T,K] or NULL
    const float* tlogit;
    const float* tweight;    // [T] or NULL: 1
    int K;
    float tau, inv_tau;
    float* kd;               // [T] or NULL
    int grad;
};

// One wave a row.  The scores at the label and the teacher's slots are read
// first and their dz is written last (an entry named twice by its first slot,
// with the slots' q added in order), the rest streams: chunk c of the row's
// dz is stored after chunk c of z has been read, and lies in front of every
// chunk still to be read (half the element size; in fp32 at the same place).
template <typename T>
__global__ __launch_bounds__(256) void head_dz_kernel(HeadDz p) {
    __shared__ int s_idx[4][kMaxK + 1];
    __shared__ float s_q[4][kMaxK + 1];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int n = piece_rows(p.count, p.p0, p.piece, 0);
    const int r = blockIdx.x * 4 + w;
    if (r >= n) return;                       // whole waves; no block barrier below
    const int t = p.rows[p.p0 + r];
    float* z = p.Z + (long)r * p.ldz;
    int label = p.labels ? p.labels[t] : -1;
    if (!in_vocab(label, p.V)) label = -1;
    const float wce = label >= 0 ? (p.weight ? p.weight[t] : 1.0f) : 0.0f;
    const float lse = p.lse[r];

    // the teacher's distribution; slot K is the label
    constexpr int PL = (kMaxK + 63) / 64;
    int idx[PL];
    float q[PL], zt[PL];
    float wkd = 0.0f, tlse = 0.0f;
    if (p.tidx) {
        tlse = p.tlse[r];
        float hi = -INFINITY;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int j = lane + 64 * u;
            idx[u] = -1;
            q[u] = -INFINITY;
            if (j < p.K) {
                const int v = p.tidx[(long)t * p.K + j];
                if (in_vocab(v, p.V)) {
                    idx[u] = v;
                    q[u] = p.tlogit[(long)t * p.K + j] * p.inv_tau;
                    hi = fmaxf(hi, q[u]);
                }
            }
        }
        hi = wave_max(hi);
        const bool any = hi > -INFINITY;
        const float ref = any ? hi : 0.0f;
        float tot = 0.0f;
        float lq[PL];
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            lq[u] = q[u] - ref;
            q[u] = expf(lq[u]);               // 0 for a slot left out
            tot += q[u];
        }
        tot = wave_sum(tot);
        const float inv = any ? 1.0f / tot : 0.0f, ltot = any ? logf(tot) : 0.0f;
        float kd = 0.0f;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int j = lane + 64 * u;
            q[u] *= inv;
            zt[u] = idx[u] >= 0 ? z[idx[u]] : 0.0f;
            if (q[u] != 0.0f) kd += q[u] * (lq[u] - ltot - (zt[u] * p.inv_tau - tlse));
            if (j < p.K) s_idx[w][j] = idx[u], s_q[w][j] = q[u];
        }
        kd = wave_sum(kd);
        if (lane == 0 && p.kd) p.kd[t] = any ? kd * p.tau * p.tau : 0.0f;
        wkd = any ? p.tau * (p.tweight ? p.tweight[t] : 1.0f) : 0.0f;
    }
    if (!p.grad) return;
    const float zy = label >= 0 ? z[label] : 0.0f;
    wave_lds_sync();
    wave_mem_sync();                          // those reads are back before any store

    T* g = reinterpret_cast<T*>(z);
    auto dense = [&](float v) {
        float o = wce != 0.0f ? wce * expf(v - lse) : 0.0f;
        if (wkd != 0.0f) o += wkd * expf(v * p.inv_tau - tlse);
        return o;
    };
    for (long c = lane * 8; c < p.ldz; c += 512) {
        float v[8];
        ld8(z + c, v);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = c + u < p.V ? dense(v[u]) : 0.0f;
        st8(g + c, v);
    }
    wave_mem_sync();
    // the label and the teacher's slots
    bool label_named = false;
    if (p.tidx) {
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int j = lane + 64 * u;
            if (j >= p.K || idx[u] < 0) continue;
            float sum = 0.0f;
            bool first = true;
            for (int k = 0; k < p.K; ++k)
                if (s_idx[w][k] == idx[u]) {
                    first = first && k >= j;
                    sum += s_q[w][k];
                }
            if (idx[u] == label) label_named = true;
            if (first)
                Elem<T>::st(g + idx[u], dense(zt[u]) - wkd * sum - (idx[u] == label ? wce : 0.0f));
        }
    }
    if (label >= 0 && __ballot(label_named) == 0 && lane == 0)
        Elem<T>::st(g + label, dense(zy) - wce);
}

// ------------------------------------------------------------- the calls

inline bool head_sizes_ok(int T, int d, int V, int K, moe_dtype dt) {
    return T >= 0 && T <= (1 << 24) && d >= 64 && d <= 65536 && d % 64 == 0 && V >= 1 &&
           V <= (1 << 20) && K >= 0 && K <= kMaxK && (dt == MOE_F32 || dt == MOE_BF16);
}

constexpr size_t kHeadLimit = (size_t)4 << 30;

struct HeadPlan {
    int piece, pieces, parts;
    long ldz;
    int dx_splits, dw_splits;
    size_t rows, count, act, xc, zl, lse, tlse, stat, tstat, z, dxp, acc, dwp, total;
};

// Parts of the reduction of a product with `tiles` output tiles over K:
// enough for two rounds of the compute units, each at least 512 long.
inline int head_splits(long tiles, long K) {
    if (tiles >= 256 || tiles == 0) return 1;
    return (int)std::max(1l, std::min((512 + tiles - 1) / tiles, K / 512));
}

HeadPlan head_layout(int T, int d, int V, int K, moe_dtype dt, int grad, int piece) {
    HeadPlan p;
    const size_t b = dt == MOE_BF16 ? 2 : 4;
    const bool store = grad || K > 0;
    const int bm = dt == MOE_BF16 ? 256 : 128, pc = dt == MOE_BF16 ? 128 : 64;
    p.piece = piece;
    p.pieces = T == 0 ? 0 : cdiv(T, piece);
    p.ldz = (long)align_up(V, 64);
    p.parts = cdiv(V, bm) * (bm / pc);
    p.dx_splits = head_splits((long)cdiv(piece, bm) * cdiv(d, bm), V);
    p.dw_splits = head_splits((long)cdiv(V, bm) * cdiv(d, bm), piece);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    p.rows = take((size_t)T * 4);
    p.count = take(4);
    p.act = take(K > 0 ? (size_t)T * 4 : 0);
    p.xc = take((size_t)piece * d * b);
    p.zl = take((size_t)piece * 4);
    p.lse = take((size_t)piece * 4);
    p.tlse = take(K > 0 ? (size_t)piece * 4 : 0);
    p.stat = take((size_t)p.parts * piece * 8);
    p.tstat = take(K > 0 ? (size_t)p.parts * piece * 4 : 0);
    p.z = take(store ? (size_t)piece * p.ldz * 4 : 0);
    // the partial sums of dx: room for any smaller piece too (fewer tiles, more
    // parts), so that a workspace for T tokens serves every smaller batch
    size_t dxp = 0;
    const int cols = cdiv(d, bm);
    for (int u = 1; u <= cdiv(piece, bm) && u * cols < 256; ++u) {
        const int sp = head_splits((long)u * cols, V);
        if (sp > 1) dxp = std::max(dxp, (size_t)sp * std::min(u * bm, piece) * d * 4);
    }
    p.dxp = take(grad ? dxp : 0);
    p.acc = take(grad && p.pieces > 1 ? (size_t)V * d * 4 : 0);
    p.dwp = take(grad && p.dw_splits > 1 ? (size_t)p.dw_splits * V * d * 4 : 0);
    p.total = o;
    return p;
}

// The plan with the largest piece whose workspace stays within `limit`, or
// the one with the smallest workspace if none does.  The fewest pieces of equal size (in whole row
// tiles), so that the last one is not a small rest.
HeadPlan head_plan(int T, int d, int V, int K, moe_dtype dt, int grad, size_t limit) {
    const int units = std::max(1, cdiv(T, kRowAlign));
    int lo = 1, hi = units;              // pieces: the fewest that fit
    auto of = [&](int pieces) {
        const int u = cdiv(units, pieces);
        return head_layout(T, d, V, K, dt, grad,
                           T <= kRowAlign ? std::max(T, 1) : u * kRowAlign);
    };
    const HeadPlan whole = of(1);        // (no running sum of dWv: it may be the smallest)
    if (whole.total <= limit) return whole;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (of(mid).total <= limit) hi = mid; else lo = mid + 1;
    }
    const HeadPlan p = of(lo);
    return p.total > limit && whole.total < p.total ? whole : p;
}

struct HeadCall {
    const void *x, *Wv;
    const int32_t* labels;
    const float* weight;
    const int32_t* tidx;
    const float* tlogit;
    const float* tweight;
    int K;
    float tau;
    int T, d, V, grad;
    float *loss, *lse, *kd;
    void *dx, *dWv;
};

template <int BMT, int BNT, typename T>
int head_grid(HeadGemm<T>& g, long m) {
    const long tiles = (long)cdiv(m, BMT) * cdiv(g.N, BNT) * g.splits;
    g.xcd_run = 32;
    const long pad = NXCD * g.xcd_run;
    return (int)((tiles + pad - 1) / pad * pad);
}

template <int ALAY, int BLAY, typename T, class Epi>
void head_product(HeadGemm<T> g, long m, const Epi& epi, hipStream_t s, const char* name) {
    if constexpr (sizeof(T) == 2) {
        const int grid = head_grid<256, 256>(g, m);
        MOE_LAUNCH(name, s, head_product_kernel<256, 256, 4, 2, 2, 64, ALAY, BLAY, Epi>
                   <<<grid, 512, 0, s>>>(g, epi));
    } else {
        const int grid = head_grid<FBM, FBM>(g, m);
        MOE_LAUNCH(name, s, head_product_f32_kernel<ALAY, BLAY, Epi><<<grid, 256, 0, s>>>(g, epi));
    }
}

template <typename T>
moe_status head_run(const HeadCall& c, const HeadPlan& p, char* ws, hipStream_t s) {
    const bool teacher = c.K > 0, store = c.grad || teacher;
    int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
    int32_t* count = reinterpret_cast<int32_t*>(ws + p.count);
    float2* stat = reinterpret_cast<float2*>(ws + p.stat);
    float* tstat = teacher ? reinterpret_cast<float*>(ws + p.tstat) : nullptr;
    float* zl = reinterpret_cast<float*>(ws + p.zl);
    float* rlse = reinterpret_cast<float*>(ws + p.lse);
    float* rtlse = teacher ? reinterpret_cast<float*>(ws + p.tlse) : nullptr;
    float* Z = store ? reinterpret_cast<float*>(ws + p.z) : nullptr;
    T* xc = reinterpret_cast<T*>(ws + p.xc);
    const float inv_tau = 1.0f / c.tau;
    const int vpr = c.d * (int)sizeof(T) / 16;
    const int32_t* act = c.labels;
    int limit = c.V;
    if (teacher) {
        int32_t* a = reinterpret_cast<int32_t*>(ws + p.act);
        MOE_LAUNCH("head_active", s, head_active_kernel<<<cdiv(c.T, 4), 256, 0, s>>>(
                       c.labels, c.tidx, c.T, c.K, c.V, a));
        act = a;
        limit = 2;
    }
    MOE_LAUNCH("head_compact", s, head_compact_kernel<<<1, 1024, 0, s>>>(
                   act, c.T, limit, rows, count, c.loss, c.lse, c.kd));
    for (int i = 0; i < p.pieces; ++i) {
        const int p0 = i * p.piece, bound = std::min(p.piece, c.T - p0);
        u32x4_t* zero_dx = c.grad && c.dx && i == 0 ? static_cast<u32x4_t*>(c.dx) : nullptr;
        MOE_LAUNCH("head_gather", s,
                   head_gather_kernel<<<cdiv((long)(zero_dx ? c.T : bound) * vpr, 256), 256, 0, s>>>(
                       static_cast<const u32x4_t*>(c.x), rows, count, p0, p.piece, vpr,
                       reinterpret_cast<u32x4_t*>(xc), act, c.T, limit, zero_dx));
        HeadGemm<T> g;
        g.count = count, g.p0 = p0, g.piece = p.piece;
        g.A = xc, g.lda = c.d, g.B = static_cast<const T*>(c.Wv), g.ldb = c.d;
        g.M = bound, g.N = c.V, g.K = c.d, g.dyn = 1, g.splits = 1;
        const EpiScores es = {c.V, stat, tstat, inv_tau, p.piece, c.labels, rows, p0, zl, Z, p.ldz};
        head_product<KMAJ, KMAJ>(g, bound, es, s, "head_scores");
        MOE_LAUNCH("head_lse", s, head_lse_kernel<<<cdiv(bound, 64), 1024, 0, s>>>(
                       stat, tstat, p.parts, p.piece, inv_tau, zl, c.labels, c.V, rows, count, 0, p0,
                       p.piece, rlse, rtlse, c.loss, c.lse));
        if (!store) continue;
        const HeadDz dz = {Z, p.ldz, c.V, rows, count, p0, p.piece, rlse, rtlse, c.labels, c.weight,
                           c.tidx, c.tlogit, c.tweight, c.K, c.tau, inv_tau, c.kd, c.grad};
        MOE_LAUNCH("head_dz", s, head_dz_kernel<T><<<cdiv(bound, 4), 256, 0, s>>>(dz));
        if (!c.grad) continue;
        const T* G = reinterpret_cast<const T*>(Z);
        const long ldg = p.ldz * (4 / (long)sizeof(T));
        if (c.dx) {
            g.A = G, g.lda = ldg, g.B = static_cast<const T*>(c.Wv), g.ldb = c.d;
            g.M = bound, g.N = c.d, g.K = c.V, g.dyn = 1, g.splits = p.dx_splits;
            T* dx = static_cast<T*>(c.dx);
            if (p.dx_splits > 1) {
                float* part = reinterpret_cast<float*>(ws + p.dxp);
                const long stride = (long)p.piece * c.d;
                head_product<KMAJ, MNMAJ>(g, bound, EpiPart{part, c.d, stride}, s, "head_dx");
                const long n8 = (long)bound * c.d / 8;
                MOE_LAUNCH("head_dx_join", s, head_join_kernel<T><<<cdiv(n8, 256), 256, 0, s>>>(
                               part, p.dx_splits, stride, n8, c.d, dx, rows, nullptr, count, p0,
                               p.piece));
            } else {
                head_product<KMAJ, MNMAJ>(g, bound, EpiRows<T>{dx, c.d, rows, p0}, s, "head_dx");
            }
        }
        if (c.dWv) {
            g.A = G, g.lda = ldg, g.B = xc, g.ldb = c.d;
            g.M = c.V, g.N = c.d, g.K = bound, g.dyn = 2, g.splits = p.dw_splits;
            T* dW = static_cast<T*>(c.dWv);
            float* acc = p.pieces > 1 ? reinterpret_cast<float*>(ws + p.acc) : nullptr;
            if (p.dw_splits > 1) {
                float* part = reinterpret_cast<float*>(ws + p.dwp);
                const long stride = (long)c.V * c.d;
                head_product<MNMAJ, MNMAJ>(g, c.V, EpiPart{part, c.d, stride}, s, "head_dW");
                const long n8 = stride / 8;
                MOE_LAUNCH("head_dW_join", s, head_join_kernel<T><<<cdiv(n8, 256), 256, 0, s>>>(
                               part, p.dw_splits, stride, n8, c.d, dW, nullptr, acc, count, p0,
                               p.piece));
            } else {
                head_product<MNMAJ, MNMAJ>(g, c.V, EpiSum<T>{dW, acc, c.d, count, p0, p.piece}, s,
                                           "head_dW");
            }
        }
    }
    return launch_status();
}

bool head_overlaps(const void* a, size_t an, const void* b, size_t bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && an && bn && x < y + bn && y < x + an;
}

moe_status head_call(const HeadCall& c, moe_dtype dt, void* ws, size_t ws_bytes, hipStream_t s) {
    auto whole4 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0; };
    MOE_CHECK_ARG(head_sizes_ok(c.T, c.d, c.V, c.K, dt));
    MOE_CHECK_ARG(c.Wv || (c.T == 0 && !c.grad));
    MOE_CHECK_ARG(aligned16(c.x) && aligned16(c.Wv) && aligned16(c.dx) && aligned16(c.dWv));
    MOE_CHECK_ARG(whole4(c.labels) && whole4(c.weight) && whole4(c.tidx) && whole4(c.tlogit) &&
                  whole4(c.tweight) && whole4(c.loss) && whole4(c.lse) && whole4(c.kd));
    const size_t b = dt == MOE_BF16 ? 2 : 4;
    const size_t nx = (size_t)c.T * c.d * b, nw = (size_t)c.V * c.d * b;
    MOE_CHECK_ARG(!head_overlaps(c.dx, nx, c.x, nx) && !head_overlaps(c.dx, nx, c.Wv, nw) &&
                  !head_overlaps(c.dWv, nw, c.x, nx) && !head_overlaps(c.dWv, nw, c.Wv, nw) &&
                  !head_overlaps(c.dx, nx, c.dWv, nw));
    if (c.T > 0) {
        MOE_CHECK_ARG(c.x && (c.labels || c.K > 0));
        MOE_CHECK_ARG(!c.labels || c.loss);
        MOE_CHECK_ARG(c.K == 0 || (c.tidx && c.tlogit && c.kd));
        if (!ws || ws_bytes < head_plan(c.T, c.d, c.V, c.K, dt, c.grad, ws_bytes).total)
            return MOE_ERR_WORKSPACE;
        MOE_CHECK_ARG(aligned16(ws));
    }
    MOE_CHECK_DEVICE();
    if (c.T == 0) {
        if (!c.grad || !c.dWv) return MOE_OK;
        const long n = (long)(nw / 16);
        MOE_LAUNCH("head_zero", s, head_zero_kernel<<<cdiv(n, 256), 256, 0, s>>>(
                       static_cast<u32x4_t*>(c.dWv), n));
        return launch_status();
    }
    const HeadPlan p = head_plan(c.T, c.d, c.V, c.K, dt, c.grad, ws_bytes);
    return dt == MOE_BF16 ? head_run<bf16_t>(c, p, static_cast<char*>(ws), s)
                          : head_run<float>(c, p, static_cast<char*>(ws), s);
}

}  // namespace
}  // namespace moe

extern "C" {

size_t moe_head_workspace_bytes(int T, int d, int V, int K, moe_dtype dt, int grad, size_t limit) {
    using namespace moe;
    if (!head_sizes_ok(T, d, V, K, dt)) return 0;
    return head_plan(T, d, V, K, dt, grad != 0, limit ? limit : kHeadLimit).total;
}

moe_status moe_head_xent(const void* x, const void* Wv, const int32_t* labels, int T, int d, int V,
                         moe_dtype dt, float* loss, float* lse, void* ws, size_t ws_bytes,
                         hipStream_t stream) {
    const moe::HeadCall c = {x, Wv, labels, nullptr, nullptr, nullptr, nullptr, 0, 1.0f, T, d, V, 0,
                             loss, lse, nullptr, nullptr, nullptr};
    return moe::head_call(c, dt, ws, ws_bytes, stream);
}

moe_status moe_head_xent_grad(const void* x, const void* Wv, const int32_t* labels,
                              const float* weight, int T, int d, int V, moe_dtype dt, float* loss,
                              float* lse, void* dx, void* dWv, void* ws, size_t ws_bytes,
                              hipStream_t stream) {
    const moe::HeadCall c = {x, Wv, labels, weight, nullptr, nullptr, nullptr, 0, 1.0f, T, d, V, 1,
                             loss, lse, nullptr, dx, dWv};
    MOE_CHECK_ARG(dx || dWv);
    return moe::head_call(c, dt, ws, ws_bytes, stream);
}

static bool head_tau_ok(const float* tau) {
    return tau && *tau >= 1e-3f && *tau <= 1e3f;
}

moe_status moe_head_distill(const void* x, const void* Wv, const int32_t* t_idx,
                            const float* t_score, int K, const float* tau, const int32_t* labels,
                            int T, int d, int V, moe_dtype dt, float* kd, float* loss, float* lse,
                            void* ws, size_t ws_bytes, hipStream_t stream) {
    MOE_CHECK_ARG(K >= 1 && head_tau_ok(tau));
    const moe::HeadCall c = {x, Wv, labels, nullptr, t_idx, t_score, nullptr, K, *tau, T, d, V, 0,
                             labels ? loss : nullptr, labels ? lse : nullptr, kd, nullptr, nullptr};
    return moe::head_call(c, dt, ws, ws_bytes, stream);
}

moe_status moe_head_distill_grad(const void* x, const void* Wv, const int32_t* t_idx,
                                 const float* t_score, const float* t_weight, int K,
                                 const float* tau, const int32_t* labels, const float* weight,
                                 int T, int d, int V, moe_dtype dt, float* kd, float* loss,
                                 float* lse, void* dx, void* dWv, void* ws, size_t ws_bytes,
                                 hipStream_t stream) {
    MOE_CHECK_ARG(K >= 1 && head_tau_ok(tau) && (dx || dWv));
    const moe::HeadCall c = {x, Wv, labels, weight, t_idx, t_score, t_weight, K, *tau, T, d, V, 1,
                             labels ? loss : nullptr, labels ? lse : nullptr, kd, dx, dWv};
    return moe::head_call(c, dt, ws, ws_bytes, stream);
}

}  // extern "C"
