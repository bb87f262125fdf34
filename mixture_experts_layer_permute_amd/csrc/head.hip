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
//               z, and z is stored only when something reads it;
//  head_dz      z -> dz, a stream; the scores are held for a few row tiles at a
//               time (they share a column tile's weights), dz for the piece;
//  head_product dx = dz Wv and dWv = dz^T x, the tiles after the last full round
//               of the compute units split over the reduction; dWv is summed over the
//               pieces in fp32.
// Nothing is computed twice: 6 n d V operations, the least there is with z
// not kept beyond its piece.  The other way, keeping no scores and computing
// them again for dz, costs 8 n d V.
//
// Roundings (bf16): dz is rounded once to bf16 as an operand of the matrix
// cores (the cross entropy's from scores kept within 3.4e-4 of exp(z), see
// code_pair); every sum is fp32; dx and dWv are rounded once.  A row of dz mostly is
// its label's entry, or a teacher's first one, whose rounding alone would be as
// large as that of the results: what it loses stays in fp32 (HeadTop) and is added
// to the row of dx.  In dWv the roundings of many tokens average out, with few
// tokens they do not: up to 128 tokens dz is two bf16 terms there (HeadGemm::terms).
#include <algorithm>
#include <type_traits>

#include "common.h"
#include "mfma_tile.h"

namespace moe {
namespace {

constexpr int kMaxK = 256;              // teacher slots of a token
constexpr int kRowAlign = 256;          // tokens of a piece: whole row tiles
constexpr int kTermTokens = 128;        // up to so many, dz is two terms in dWv

// What bf16 took from the largest of a row's named entries of dz (the label, the
// teacher's slots): dz there is the rounded value plus `lost`.
struct HeadTop {
    int col;
    float lost;
};

// The wave's stores before it are done: a later one of another lane to the same
// place comes behind them.
__device__ __forceinline__ void wave_mem_sync() {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// Sums and maxima over lanes, in every lane of the group; every lane of the wave
// must be active.  16 neighbouring lanes: quad swaps, then the mirror of 8, then
// that of 16 (mirrors, since the smaller groups' lanes agree by then).  Lanes 16
// and 32 apart: the swap of a register's halves with its own copy's.
template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
    return __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
struct F2 {
    float a, b;
};
__device__ __forceinline__ F2 swap16(float v) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return {__uint_as_float(s[0]), __uint_as_float(s[1])};
}
__device__ __forceinline__ F2 swap32(float v) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                    false);
    return {__uint_as_float(s[0]), __uint_as_float(s[1])};
}
__device__ __forceinline__ float max16(float v) { const F2 s = swap16(v); return fmaxf(s.a, s.b); }
__device__ __forceinline__ float max32(float v) { const F2 s = swap32(v); return fmaxf(s.a, s.b); }
__device__ __forceinline__ float sum16(float v) { const F2 s = swap16(v); return s.a + s.b; }
__device__ __forceinline__ float sum32(float v) { const F2 s = swap32(v); return s.a + s.b; }
__device__ __forceinline__ float wave_max(float v) {
    v = fmaxf(v, dpp<0xB1>(v));                    // quad_perm 1,0,3,2
    v = fmaxf(v, dpp<0x4E>(v));                    // quad_perm 2,3,0,1
    v = fmaxf(v, dpp<0x141>(v));                   // row_half_mirror
    v = fmaxf(v, dpp<0x140>(v));                   // row_mirror
    return max32(max16(v));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += dpp<0xB1>(v);
    v += dpp<0x4E>(v);
    v += dpp<0x141>(v);
    v += dpp<0x140>(v);
    return sum32(sum16(v));
}

// f(0), f(1), ... f(N - 1) with constants.
template <int N, int I = 0, class F>
__device__ __forceinline__ void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, I + 1>(f);
    }
}

// ------------------------------------------------------- tokens with a loss

__device__ __forceinline__ bool in_vocab(int v, int V) { return (unsigned)v < (unsigned)V; }
// Whether a teacher's slot counts: its entry is one, its score not -infinity (a NaN
// counts, and shows in the results).
__device__ __forceinline__ bool slot_on(const int32_t* tidx, const float* tlogit, long at, int V) {
    return in_vocab(tidx[at], V) && !(tlogit[at] == -INFINITY);
}

// act[t]: whether token t has a label or a teacher's slot (one wave a token).
__global__ __launch_bounds__(256) void head_active_kernel(const int32_t* __restrict__ labels,
                                                          const int32_t* __restrict__ tidx,
                                                          const float* __restrict__ tlogit,
                                                          int T, int K, int V,
                                                          int32_t* __restrict__ act) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (t >= T) return;
    bool on = labels && in_vocab(labels[t], V);
    for (int j = lane; j < K && !on; j += 64) on = slot_on(tidx, tlogit, (long)t * K + j, V);
    const bool any = __ballot(on) != 0;
    if (lane == 0) act[t] = any ? 1 : -1;
}

constexpr int kXcdRun = 32;             // neighbouring tiles on one XCD
constexpr int kRound = 256;             // compute units
constexpr int kMaxParts = 32;           // of a tile
constexpr int kMaxSlots = 768;          // rest tiles times parts
constexpr long kScoreSlots = 128;       // the scores' tiles times parts, where they are split

// Parts of each of R rest tiles whose reduction has nj stages of 64 steps: the
// fewest stage times over the rounds they take, with `ends` of them for a tile's
// start and end and `slot` for writing and adding up a part.  bf16: 6 (10 us
// against 1.2 a stage) and a twelfth (512 KB at about 4.5 TB/s); fp32: 1 and a
// hundredth (128 KB against 3.4 us a stage).  One wave: lane i looks at i + 1.
__device__ __forceinline__ int rest_parts(int R, int nj, bool f32) {
    const float ends = f32 ? 1.0f : 6.0f, slot = f32 ? 0.01f : 0.085f;
    const int S = (threadIdx.x & 63) + 1;
    const bool can = S == 1 || (S <= kMaxParts && (f32 ? S <= nj : S * 4 <= nj + 3) &&
                               R * S <= kMaxSlots);
    const int rounds = (R * S + kRound - 1) / kRound;
    const float t = can ? rounds * ((nj + S - 1) / S + ends) + (S > 1 ? ends + R * S * slot : 0.0f)
                        : INFINITY;
    const float least = -wave_max(-t);
    return __ffsll((long long)__ballot(t == least));      // the fewest parts of equals
}

// plan[2 piece + {0: dx, 1: dWv}] = the parts of the product's rest tiles.
struct HeadParts {
    int32_t* plan;
    int pieces, piece, d, V, bm;
    int terms;               // of dz in dWv
};

// Whether token t has a loss: by its label, by its teacher's slots, or as
// head_active_kernel found (tidx NULL, act then its flags with limit 2).
struct HeadTokens {
    const int32_t* act;      // labels (limit V) or flags (limit 2), or NULL
    int limit;
    const int32_t* tidx;     // or NULL
    const float* tlogit;
    int K, V, T;
    __device__ __forceinline__ bool has_loss(int t) const {
        bool on = act && in_vocab(act[t], limit);
        if (tidx)
            for (int j = 0; j < K && !on; ++j) on = slot_on(tidx, tlogit, (long)t * K + j, V);
        return on;
    }
};
// What the compaction leaves besides the list: the count, zeros in the outputs
// of the tokens without a loss, the split of the products.
struct HeadStart {
    int32_t* rows;
    int32_t* clab;           // the rows' labels, or NULL
    int32_t* count;
    float* out[3];
    HeadParts parts;
    __device__ __forceinline__ void place(const HeadTokens& tk, int t, int at) const {
        MOE_DASSERT(at >= 0 && at < tk.T);
        rows[at] = t;
        if (clab) clab[at] = tk.act[t];
    }
    __device__ __forceinline__ void skip(int t) const {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (out[i]) out[i][t] = 0.0f;
    }
    __device__ __forceinline__ void finish(int n) const {
        if (threadIdx.x == 0) *count = n;
        for (int i = threadIdx.x >> 6; i < parts.pieces * 2; i += 16) {    // a wave each
            const int k = max(0, min(n - (i >> 1) * parts.piece, parts.piece));
            const int nM = ((i & 1) ? parts.V + parts.bm - 1 : k + parts.bm - 1) / parts.bm;
            const int tiles = nM * ((parts.d + parts.bm - 1) / parts.bm);
            const int best = rest_parts(tiles % kRound,
                                        ((i & 1) ? k * parts.terms + 63 : parts.V + 63) / 64,
                                        parts.bm == 128);
            if ((threadIdx.x & 63) == 0) parts.plan[i] = best;
        }
    }
};
constexpr int kStartTokens = 4096;      // of a block's round: four a thread
// One round of the compaction: f(t, place) for the tokens t0 .. t0 + 4095 with a
// loss, skip(t) for the others; returns the places used so far.
template <class F, class G>
__device__ __forceinline__ int compact_round(const HeadTokens& tk, int t0, int base, int* sh,
                                             F&& f, G&& skip) {
    const int t = t0 + threadIdx.x * 4;
    bool on[4];
    int c = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        on[q] = t + q < tk.T && tk.has_loss(t + q);
        c += on[q];
    }
    int total;
    int at = base + block_excl_scan<1024>(c, sh, &total);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        if (on[q]) f(t + q, at++);
        else if (t + q < tk.T) skip(t + q);
    }
    return base + total;
}

// rows[0..n) = the tokens that have a loss, in order.  One block.
__global__ __launch_bounds__(1024) void head_compact_kernel(HeadTokens tk, HeadStart st) {
    __shared__ int sh[16];
    int n = 0;
    for (int t0 = 0; t0 < tk.T; t0 += kStartTokens)
        n = compact_round(tk, t0, n, sh, [&](int t, int at) { st.place(tk, t, at); },
                          [&](int t) { st.skip(t); });
    st.finish(n);
}

// For up to 4096 tokens: the same and the row copies (head_gather) in one launch.
// Every block makes the whole list, in LDS; block 0 writes it out.  copies: of a row,
// one behind the other (one per term of dz).
__global__ __launch_bounds__(1024) void head_start_kernel(HeadTokens tk, HeadStart st,
                                                          const u32x4_t* __restrict__ x, int vpr,
                                                          u32x4_t* __restrict__ xc, int copies,
                                                          u32x4_t* __restrict__ dx) {
    __shared__ int sh[16];
    __shared__ int list[kStartTokens];
    const bool first = blockIdx.x == 0;
    const int n = compact_round(tk, 0, 0, sh, [&](int t, int at) {
        list[at] = t;
        if (first) st.place(tk, t, at);
    }, [&](int t) { if (first) st.skip(t); });
    __syncthreads();
    if (first) st.finish(n);
    const int step = gridDim.x * 1024;
    for (int i = blockIdx.x * 1024 + threadIdx.x; i < n * vpr; i += step) {
        const int r = i / vpr, c = i - r * vpr;
        const u32x4_t v = x[(long)list[r] * vpr + c];
        for (int k = 0; k < copies; ++k) xc[((long)r * copies + k) * vpr + c] = v;
    }
    if (!dx || n == tk.T) return;
    for (int i = blockIdx.x * 1024 + threadIdx.x; i < tk.T * vpr; i += step)
        if (!tk.has_loss(i / vpr)) dx[i] = u32x4_t{0, 0, 0, 0};
}

// Both copies are bound by launch and bandwidth: 8192 rows of 1024 bf16, list 10 us
// (one block), copy 9 us (3.6 TB/s); 777 rows in one launch 5 us.

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
    HeadTokens tk, u32x4_t* __restrict__ dx) {
    const int n = piece_rows(count, p0, piece, 0);
    const long end = (long)(dx ? tk.T : n) * vpr;
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < end; i += (long)gridDim.x * 256) {
        const long r = i / vpr;
        const int c = (int)(i - r * vpr);
        if (r < n) {
            const int t = rows[p0 + r];
            MOE_DASSERT(t >= 0 && t < tk.T);
            xc[i] = x[(long)t * vpr + c];
        }
        if (dx && !tk.has_loss((int)r)) dx[i] = u32x4_t{0, 0, 0, 0};
    }
}

__global__ __launch_bounds__(256) void head_zero_kernel(u32x4_t* __restrict__ p, long n) {
    for (long i = (long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long)gridDim.x * 256)
        p[i] = u32x4_t{0, 0, 0, 0};
}
// Blocks of 256 threads for n items, by those kernels' strides: a launch has fewer
// than 2^32 threads.
inline int head_blocks(long n) { return (int)std::min((n + 255) / 256, 1l << 22); }

// ------------------------------------------------------- matrix products

// C [M,N] = A . B over K.  Of M and K one may be the piece's rows, known on the
// device only (dyn).  The compute units take the output tiles in rounds of 256;
// the rest of the tiles, after the last full round, may be split over the
// reduction (plan: in how many parts), each part's product stored in fp32 in a slot of
// its own for head_join to add up.
template <typename T>
struct HeadGemm {
    const T* A;
    long lda;
    const T* B;
    long ldb;
    int M, N, K;
    int dyn;                 // 1: M, 2: K is the piece's rows (0: neither)
    int terms;               // reduction rows of a piece's row (dyn 2)
    const int32_t* count;
    int p0, piece;
    const int32_t* plan;     // parts of a rest tile (NULL: split)
    int split;               // of every tile of a product with fewer than 256, known to the host
    float* part;             // [slot][BM][BN]
};

struct HeadTile {
    int m0, n0, rows, cols;  // tile origin, valid rows and columns
    int k0, k1;              // this part of the reduction
    int slot;                // >= 0: a part, stored there
    bool live;
};

// Tile w of nM x nN: in groups of 8 row tiles, every column tile of a group before
// the next group, row tiles fastest: a run of 32 on one XCD is 8 x 4 tiles,
// which share their operands in its L2.
template <int BM, int BN>
__device__ __forceinline__ void head_origin(int w, int nM, int nN, int& m0, int& n0) {
    const int first = (w / (8 * nN)) * 8;
    const int gm = min(8, nM - first);
    w -= first * nN;
    m0 = (first + w % gm) * BM;
    n0 = (w / gm) * BN;
}

template <int BM, int BN, typename T>
__device__ __forceinline__ HeadTile head_tile(const HeadGemm<T>& p, int block) {
    HeadTile t;
    const int n = p.dyn ? piece_rows(p.count, p.p0, p.piece, p.piece) : 0;
    const int M = p.dyn == 1 ? n : p.M, K = p.dyn == 2 ? n * p.terms : p.K;
    const int nM = (M + BM - 1) / BM, nN = (p.N + BN - 1) / BN, tiles = nM * nN;
    const int S = p.plan ? *p.plan : p.split;
    const int full = S > 1 ? tiles / kRound * kRound : tiles;
    int L = xcd_logical(block, kXcdRun);
    t.slot = -1;
    t.k0 = 0, t.k1 = K;
    if (L >= full) {
        const int R = tiles - full, item = L - full;
        t.live = item < R * S;
        if (!t.live) return t;
        const int s = item / R;
        const int kc = ((K + S - 1) / S + 63) / 64 * 64;
        t.k0 = min(K, s * kc);
        t.k1 = min(K, t.k0 + kc);
        t.slot = item;
        L = full + item - s * R;
    }
    t.live = true;
    head_origin<BM, BN>(L, nM, nN, t.m0, t.n0);
    t.rows = min(BM, M - t.m0);
    t.cols = min(BN, p.N - t.n0);
    return t;
}

// Epilogues.  The products are made with the operands swapped, so that a lane's
// four accumulators of a fragment are four neighbouring columns of one row: the
// wave hands over row by row (rl: this lane's row in the tile), with the lane's
// quads v[q] at the columns Lanes::col(q) from cl on.  No LDS, no barrier.
//  Quads16: 16 x 16 fragments, 8 quads of 128 columns, 4 lanes (16 apart) a row;
//  Quads32: 32 x 32 fragments, 8 quads of 64 columns, 2 lanes (32 apart) a row.
struct Quads16 {
    static constexpr int WIDTH = 128;
    static __device__ __forceinline__ int col(int q) { return q * 16 + ((threadIdx.x >> 4) & 3) * 4; }
    static __device__ __forceinline__ bool first() { return (threadIdx.x & 48) == 0; }
    static __device__ __forceinline__ float max(float v) { return max32(max16(v)); }
    static __device__ __forceinline__ float sum(float v) { return sum32(sum16(v)); }
};
struct Quads32 {
    static constexpr int WIDTH = 64;
    static __device__ __forceinline__ int col(int q) {
        return (q >> 2) * 32 + (q & 3) * 8 + ((threadIdx.x >> 5) & 1) * 4;
    }
    static __device__ __forceinline__ bool first() { return (threadIdx.x & 32) == 0; }
    static __device__ __forceinline__ float max(float v) { return max32(v); }
    static __device__ __forceinline__ float sum(float v) { return sum32(v); }
};

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
__device__ __forceinline__ float exp2_hw(float v) { return __builtin_amdgcn_exp2f(v); }

// Coded scores.  Where only the cross entropy's dz needs them (which bf16 rounds
// to 2^-9), a score is kept in 16 bits, as how far below the largest of its 128
// columns it lies, in steps of 64 / 65535 of log2: exp(z) comes back within 2^-11 ln 2 =
// 3.4e-4, a sixth of that rounding, at half the bytes of fp32 (8192 x 50257
// scores: writing them 1.65 GB to 0.82, the pass that reads them 466 us to 298).  What lies 64
// or more below (2^-64 of that maximum) counts as 64 below.  The label's own score and the
// statistics stay fp32.
// The coding is the hardware's conversion of [0, 1] to 0 .. 65535, clamped and rounded,
// of what z L lies below m L itself: x, relative to m' = m L rounded, less rho = m L - m',
// which is as large as a step of the code for scores above 4000.
constexpr float kCodeRange = 64.0f, kCodeStep = 64.0f / 65535.0f;
__device__ __forceinline__ uint32_t code_pair(float lo, float hi, float rho) {
    constexpr float k = -1.0f / kCodeRange;
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pknorm_u16(fmaf(lo, k, -k * rho),
                                                                       fmaf(hi, k, -k * rho)));
}

// (fmaxf would first turn signalling NaNs into quiet ones, an instruction each)
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Quads16 of 16-bit elements (pairs w) in 16-byte stores: two lanes 16 apart
// trade halves of two neighbouring fragments.  After the swap of X's odd 16-lane
// rows with Y's even ones a lane of an even row holds 8 columns of fragment q, of
// an odd one of fragment q + 1.
template <bool EDGE>
__device__ __forceinline__ void store_pairs(void* out, bool in, int cols,
                                            const uint32_t (&w)[8][2]) {
    const int g = (threadIdx.x >> 4) & 3;
    const int c0 = (g & 1) * 16 + (g >> 1) * 8;
#pragma unroll
    for (int q = 0; q < 8; q += 2) {
        u32x4_t x;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const auto sw = __builtin_amdgcn_permlane16_swap(w[q][u], w[q + 1][u], false, false);
            x[u] = sw[0];
            x[2 + u] = sw[1];
        }
        const int c = c0 + q * 16;
        if (in && (!EDGE || c < cols))
            *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(out) + c) = x;
    }
}

// Scores: per row and 128 (64 in fp32) columns the maximum m and the sums of
// exp(z - m) and exp((z - m) / tau); the label's score; z itself if kept.
// exp(z - m) = 2^(z L - m'), L = log2 e, m' = m L rounded: one fused multiply-add
// before the hardware's 2^x, the same m' wherever the sum is used.
struct EpiScores {
    static constexpr bool kSplits = false;
    typedef int Ask;
    int V;
    float2* stat;            // (m, sum) of a row's part: part * sp + row * sr
    float* tstat;            // the sum at the temperature likewise, or NULL
    long sp, sr;
    float l2t;               // L / tau
    const int32_t* labels;   // [rows] or NULL
    float* zl;               // [rows] label's score
    float* Z;                // z, or NULL
    uint16_t* code;          // z coded (bf16 products only), or NULL
    long ldz;                // a multiple of 64

    // what row() needs of a row from memory, asked for before the products
    __device__ __forceinline__ int ask(const HeadTile& ti, int rl) const {
        return labels && rl < ti.rows ? labels[ti.m0 + rl] : -1;
    }
    template <class Lanes>
    __device__ __forceinline__ void row(const HeadTile& ti, int rl, int cl, const f32x4 (&acc)[8],
                                        int label) const {
        // (the wave's columns all inside the vocabulary: nothing to test)
        if (ti.n0 + cl + Lanes::WIDTH <= V) row_of<Lanes, false>(ti, rl, cl, acc, label);
        else row_of<Lanes, true>(ti, rl, cl, acc, label);
    }
    template <class Lanes, bool EDGE>
    __device__ __forceinline__ void row_of(const HeadTile& ti, int rl, int cl,
                                           const f32x4 (&acc)[8], int label) const {
        constexpr bool kCodes = Lanes::WIDTH == 128;
        const int col = ti.n0 + cl, left = V - col, room = (int)ldz - col;
        const bool in = rl < ti.rows;
        const long r = (long)ti.m0 + rl;
        f32x4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = acc[q];
        if (Z && in) {
            float* z = Z + r * ldz + col;
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (!EDGE || Lanes::col(q) < room) *reinterpret_cast<f32x4*>(z + Lanes::col(q)) = v[q];
        }
        const int y = label - col;
        if (label >= 0 && (unsigned)y < (unsigned)Lanes::WIDTH && y < left) {
            // this lane's quad with column y, if it has it
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if ((y & ~3) == Lanes::col(q)) {
                    const float lo = y & 1 ? v[q][1] : v[q][0], hi = y & 1 ? v[q][3] : v[q][2];
                    zl[r] = y & 2 ? hi : lo;
                }
        }
        if (EDGE) {                                    // the vocabulary's end
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    v[q][u] = Lanes::col(q) + u < left ? v[q][u] : -INFINITY;
        }
        float m = fmaxf(v[0][0], v[0][1]);
        m = max3(m, v[0][2], v[0][3]);
#pragma unroll
        for (int q = 1; q < 8; ++q) m = max3(max3(m, v[q][0], v[q][1]), v[q][2], v[q][3]);
        m = Lanes::max(m);
        const float ref = m == -INFINITY ? 0.0f : m;   // no column here, or none finite
        const float m2 = ref * kLog2e, rho = fmaf(ref, kLog2e, -m2);
        float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        uint32_t w[8][2];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            float x[4], e[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u] = fmaf(v[q][u], kLog2e, -m2);
#pragma unroll
            for (int u = 0; u < 4; ++u) e[u] = exp2_hw(x[u]);
#pragma unroll
            for (int u = 0; u < 4; ++u) s[u] += e[u];
            if (kCodes)
#pragma unroll
                for (int u = 0; u < 2; ++u) w[q][u] = code_pair(x[2 * u], x[2 * u + 1], rho);
        }
        if (kCodes && code) store_pairs<EDGE>(code + r * ldz + col, in, room, w);
        const float sum = Lanes::sum((s[0] + s[1]) + (s[2] + s[3]));
        const long at = (long)(col / Lanes::WIDTH) * sp + r * sr;
        if (tstat) {
            const float mt = ref * l2t;
            float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < 8; ++q)
#pragma unroll
                for (int u = 0; u < 4; ++u) t[u] += exp2_hw(fmaf(v[q][u], l2t, -mt));
            const float tsum = Lanes::sum((t[0] + t[1]) + (t[2] + t[3]));
            if (in && Lanes::first()) tstat[at] = tsum;
        }
        if (in && Lanes::first()) stat[at] = make_float2(m, sum);
    }
};

// Scores whose product was split: only parts are stored.
struct EpiParts {
    static constexpr bool kSplits = true;
    typedef int Ask;
    __device__ __forceinline__ int ask(const HeadTile&, int) const { return 0; }
    template <class Lanes>
    __device__ __forceinline__ void row(const HeadTile&, int, int, const f32x4 (&)[8], int) const {}
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

// A row's quads to out (row start).
template <class Lanes, typename T>
__device__ __forceinline__ void store_row(T* out, bool in, int cl, int cols, const f32x4 (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        out += cl;
        cols -= cl;
        if (cols >= Lanes::WIDTH) {
            if (in)
#pragma unroll
                for (int q = 0; q < 8; ++q) *reinterpret_cast<f32x4*>(out + Lanes::col(q)) = v[q];
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                if (in && Lanes::col(q) < cols)
                    *reinterpret_cast<f32x4*>(out + Lanes::col(q)) = v[q];
        }
    } else {
        uint32_t w[8][2];
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int u = 0; u < 2; ++u) w[q][u] = pack_bf16x2(v[q][2 * u], v[q][2 * u + 1]);
        if (cols - cl >= Lanes::WIDTH) store_pairs<false>(out + cl, in, cols - cl, w);
        else store_pairs<true>(out + cl, in, cols - cl, w);
    }
}

// dx rows, back at their tokens, with what dz lost in bf16: lost * Wv[col].
template <typename T>
struct EpiRows {
    static constexpr bool kSplits = true;
    T* out;
    long ldo;
    const int32_t* rows;
    int p0;
    const HeadTop* top;      // [piece] (bf16)
    const T* Wv;             // [V][ldo]
    // a piece's row: its token, and what it lost (fp32: nothing)
    struct Ask {
        int token;
        HeadTop lost;
    };
    __device__ __forceinline__ Ask of(int r) const {
        if constexpr (sizeof(T) == 2) return {rows[p0 + r], top[r]};
        else return {rows[p0 + r], {0, 0.0f}};
    }
    __device__ __forceinline__ Ask ask(const HeadTile& ti, int rl) const {
        return rl < ti.rows ? of(ti.m0 + rl) : Ask{0, {0, 0.0f}};
    }
    template <class Lanes>
    __device__ __forceinline__ void row(const HeadTile& ti, int rl, int cl, f32x4 (&v)[8],
                                        const Ask& k) const {
        const bool in = rl < ti.rows;
        if constexpr (sizeof(T) == 2) {
            const HeadTop a = k.lost;
            if (a.lost != 0.0f) {
                const T* w = Wv + (long)a.col * ldo + ti.n0 + cl;
                uint2 b[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    b[q] = cl + Lanes::col(q) < ti.cols
                               ? *reinterpret_cast<const uint2*>(w + Lanes::col(q)) : uint2{0, 0};
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    v[q][0] = fmaf(a.lost, __uint_as_float(b[q].x << 16), v[q][0]);
                    v[q][1] = fmaf(a.lost, __uint_as_float(b[q].x & 0xffff0000u), v[q][1]);
                    v[q][2] = fmaf(a.lost, __uint_as_float(b[q].y << 16), v[q][2]);
                    v[q][3] = fmaf(a.lost, __uint_as_float(b[q].y & 0xffff0000u), v[q][3]);
                }
            }
        }
        store_row<Lanes>(out + (long)k.token * ldo + ti.n0, in, cl, ti.cols, v);
    }
    __device__ __forceinline__ void put8(int r, int c, float* v) const {
        const Ask k = of(r);
        if (sizeof(T) == 2 && k.lost.lost != 0.0f) {
            float w[8];
            ld8(Wv + (long)k.lost.col * ldo + c, w);
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = fmaf(k.lost.lost, w[u], v[u]);
        }
        st8(out + (long)k.token * ldo + c, v);
    }
};

// dWv over the pieces: the running sum in fp32, the last piece rounds it.
template <typename T>
struct EpiSum {
    static constexpr bool kSplits = true;
    typedef int Ask;
    T* out;
    float* acc;
    long ldo;
    const int32_t* count;
    int p0, piece;
    __device__ __forceinline__ int ask(const HeadTile&, int) const { return 0; }
    template <class Lanes>
    __device__ __forceinline__ void row(const HeadTile& ti, int rl, int cl, f32x4 (&v)[8],
                                        int) const {
        const bool in = rl < ti.rows;
        const long at = (long)(ti.m0 + rl) * ldo + ti.n0;
        if (p0 > 0) {
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int c = cl + Lanes::col(q);
                if (in && c < ti.cols) v[q] += *reinterpret_cast<const f32x4*>(acc + at + c);
            }
        }
        if (*count <= p0 + piece) store_row<Lanes>(out + at, in, cl, ti.cols, v);
        else store_row<Lanes>(acc + at, in, cl, ti.cols, v);
    }
    __device__ __forceinline__ void put8(int r, int c, float* v) const {
        const long at = (long)r * ldo + c;
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

// One row of a part into its slot.
template <class Lanes, int BM, int BN>
__device__ __forceinline__ void store_part(float* part, const HeadTile& ti, int rl, int cl,
                                           const f32x4 (&v)[8]) {
    store_row<Lanes>(part + (long)ti.slot * (BM * BN) + rl * BN, rl < ti.rows, cl, ti.cols, v);
}

// A piece past the last token adds nothing to dWv (the first always runs: it
// writes the zeros of a batch without a loss).
template <typename T>
__device__ __forceinline__ bool piece_done(const HeadGemm<T>& p) {
    return p.dyn == 2 && p.p0 > 0 && *p.count <= p.p0;
}

// One operand of a bf16 product: 256 rows of a stage of BK reduction steps go
// from HBM straight into LDS (a unit of 256 * BK * 2 bytes, 1 KB a wave and load),
// and fragments of v_mfma_f32_16x16x32_bf16 come out of it: row = lane % 16,
// eight reduction steps from 8 * (lane / 16) on.
//  K-major: rows of BK elements in 16-byte chunks, chunk c of row r at c ^ ((r ^
//    r/CH) mod CH): the 16 rows of a read lie in distinct banks.
//  M/N-major: BK rows of 256 elements, read with the transposing LDS read, which
//    takes 4 reduction steps x 16 columns per 16 lanes; chunk c of step k at c ^
//    4 (k mod 4) ^ 2 (k/8 mod 2): the four steps of a group and the two groups
//    of half a wave lie in distinct banks.
template <int LAY, int BK, int NW, int ROWS = 256>
struct HeadOperand {
    static_assert(LAY == KMAJ || ROWS == 256, "32 chunks a row of M/N-major units");
    static constexpr int CH = BK / 8;
    static constexpr int UNIT = ROWS * BK * 2;
    static constexpr int NLOAD = UNIT / 1024 / NW;
    const bf16_t* P;
    long ld, span;
    int k_lim;
    uint32_t off[NLOAD];
    uint32_t frag[LAY == KMAJ ? BK / 32 : 1];    // this lane's offsets in a unit, see read

    static __device__ __forceinline__ int mn_swz(int k, int c) {
        return c ^ ((k & 3) << 2) ^ ((k >> 3 & 1) << 1);
    }
    // P_: the tile's first row (K-major) or column; rows: valid ones; k_lim: end of
    // the reduction; w0: the wave's first row in the tile
    __device__ __forceinline__ void init(const bf16_t* P_, long ld_, int rows, int k_lim_, int w0) {
        P = P_, ld = ld_, k_lim = k_lim_;
        span = (long)rows * ld * 2;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) {
            const int blk = w + NW * i;                    // 1 KB block of the unit
            if constexpr (LAY == KMAJ) {
                const int row = blk * (64 / CH) + lane / CH;
                const int c = (lane % CH) ^ ((row ^ (row / CH)) & (CH - 1));
                off[i] = (uint32_t)(row * ld * 2 + c * 16);
            } else {
                const int k = blk * 2 + lane / 32;
                const int c = mn_swz(k, lane % 32);
                off[i] = c * 8 < rows ? (uint32_t)(k * ld * 2 + c * 16) : OOB;
            }
        }
        if constexpr (LAY == KMAJ) {
            const int row = w0 + (lane & 15);
#pragma unroll
            for (int s = 0; s < BK / 32; ++s)
                frag[s] = row * BK * 2 +
                          (((s * 4 + (lane >> 4)) ^ ((row ^ (row / CH)) & (CH - 1))) << 4);
        } else {
            // step (lane / 16) * 8 + (lane % 16) / 4 of 32, columns 4 (lane % 4) on
            const int k = (lane >> 4) * 8 + ((lane & 15) >> 2);
            const int c = (w0 >> 3) + ((lane & 3) >> 1);
            frag[0] = k * ROWS * 2 + (mn_swz(k, c) << 4) + (lane & 1) * 8;
        }
    }
    // The descriptor of the unit at k0, whose loads outside the valid rows, the end
    // of the reduction or (!some) altogether give zeros and read nothing.
    __device__ __forceinline__ i32x4_t words(long k0, bool some) const {
        const bf16_t* base = LAY == KMAJ ? P + k0 : P + k0 * ld;
        const long n = LAY == KMAJ ? span - k0 * 2 : min((long)BK, k_lim - k0) * ld * 2;
        return rsrc_words(base, some ? n : 0);
    }
    // wlds: the unit's LDS address + 1 KB times the wave, in a scalar register
    template <int I>
    __device__ __forceinline__ void load(i32x4_t rs, uint32_t wlds) const {
        // One wait state between writing m0 and the load that reads it.  A vector
        // instruction that writes a scalar register (the descriptor may come out of
        // v_readfirstlane) stands five wait states before a load that reads it, and
        // the compiler does not count them into inline assembly: the first load of a
        // unit, the nearest to its descriptor, waits for all five itself.
        asm volatile(
            "s_add_u32 m0, %0, %1\n\t"
            "s_nop %4\n\t"
            "buffer_load_dwordx4 %2, %3, 0 offen lds"
            :
            : "s"(wlds), "n"(NW * I * 1024), "v"(off[I]), "s"(rs), "n"(I == 0 ? 3 : 0)
            : "memory", "m0", "scc");
    }
    // Fragment I (rows 16 I on of the wave's) of the 32 steps S of the unit at
    // LDS address u (aligned to its size, so that the swizzle can be applied to the sum,
    // which keeps the eight addresses out of registers between the steps).
    typedef __attribute__((address_space(3))) const u32x4_t lds_u32x4_t;
    template <int I, int S>
    __device__ __forceinline__ bf16x8 read(uint32_t u) const {
        if constexpr (LAY == KMAJ) {
            // 16 rows further: the swizzle of BK = 64 changes by (2 I) mod 8 chunks
            constexpr uint32_t X = CH == 8 ? ((I * 2) & 7) << 4 : 0;
            const u32x4_t v = *reinterpret_cast<lds_u32x4_t*>(((u + frag[S]) ^ X) + I * 16 * BK * 2);
            return __builtin_bit_cast(bf16x8, v);
        } else {
            // 16 columns further: two chunks, under the swizzle
            const uint32_t o = ((u + frag[0]) ^ (I << 5)) + S * 32 * ROWS * 2;
            const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<lds_v4i16_t*>(o));
            const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                reinterpret_cast<lds_v4i16_t*>(o + 4 * ROWS * 2));
            typedef short v8i16_t __attribute__((ext_vector_type(8)));
            const v8i16_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
            return __builtin_bit_cast(bf16x8, v);
        }
    }
};

// c += a b, the accumulators kept in the accumulation registers: 64 fragments
// fill all 256 of them, and the compiler, left to choose, moves some of them to
// the others and back in every step.  The compiler does not see the waits that
// go with it (behind it a read of the result, before it a vector instruction that
// writes an operand), so it stands only in the loop, where its operands come
// from LDS and its results go to the next one; a tile's last stage is made with
// the compiler's own form.
__device__ __forceinline__ void mfma16(f32x4& c, const bf16x8& a, const bf16x8& b) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
}
// bf16: 256 x 256 tiles, four waves of 128 x 128 (one a SIMD), operands straight
// from HBM into a ring of NU units (a unit: one operand's 256 rows of a stage of
// BK reduction steps, 32 KB; A's and B's take turns, unit u in slot u mod NU).
//
// The order of the instructions is the kernel: the matrix pipe takes one
// 16x16x32 product every 16 cycles, and between two of them a wave issues at
// most one fragment read or one load.  A step of 32 is 64 products on one set of
// fragments, with the reads of the next step's set behind every second of the
// first 32 and the loads spread between them; sched_barrier keeps that order.  One
// barrier a stage, at the start of its last step: by then every wave has read the
// whole stage (its two slots are free for the loads that follow) and the next
// stage, which that step reads from, has landed.
constexpr int BK = 64, NU = 5, UNIT = 256 * BK * 2;
constexpr int kRingBytes = NU * UNIT;
template <int ALAY, int BLAY, class Epi>
__device__ __forceinline__ void head_product_body(const HeadGemm<bf16_t>& p, const Epi& epi,
                                                  int block, uint8_t* ringbuf) {
    static_assert(kRingBytes <= 160 * 1024, "LDS");
    if (piece_done(p)) return;
    const HeadTile ti = head_tile<256, 256>(p, block);
    if (!ti.live) return;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);    // (uniform, for the branches)
    const int wm = wv >> 1, wn = wv & 1;

    typename Epi::Ask asked[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) asked[i] = epi.ask(ti, wm * 128 + i * 16 + (lane & 15));
    typedef HeadOperand<ALAY, BK, 4> OpA;
    typedef HeadOperand<BLAY, BK, 4> OpB;
    constexpr int NL = OpA::NLOAD;                     // loads of a unit
    OpA opA;
    OpB opB;
    opA.init(p.A + (ALAY == KMAJ ? (long)ti.m0 * p.lda : (long)ti.m0), p.lda, ti.rows, ti.k1,
             wm * 128);
    opB.init(p.B + (BLAY == KMAJ ? (long)ti.n0 * p.ldb : (long)ti.n0), p.ldb, ti.cols, ti.k1,
             wn * 128);

    f32x4 acc[8][8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    bf16x8 af[2][8], bfr[2][8];

    // stages past the end are loaded too, from an empty range: no memory is
    // read, and the counts of loads in flight stay the same to the end (an empty
    // reduction is one such stage: zeros)
    const int some = (ti.k1 - ti.k0 + BK - 1) / BK, nj = max(some, 1);
    auto rsA = [&](int j) { return opA.words((long)ti.k0 + (long)j * BK, j < some); };
    auto rsB = [&](int j) { return opB.words((long)ti.k0 + (long)j * BK, j < some); };
    auto wrap = [](int q) { return q >= NU ? q - NU : q; };
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(ringbuf) + wv * 1024);
    auto slot = [&](int q) { return lds0 + (uint32_t)(q * UNIT); };
    const uint32_t ring0 = lds_addr(ringbuf);
    auto unit = [&](int q) { return ring0 + (uint32_t)(q * UNIT); };

    // fragment r of step s of a stage, in the order in which the products take them
    auto read1 = [&](auto R, auto S, auto BUF, uint32_t ua, uint32_t ub) {
        constexpr int r = decltype(R)::value, s = decltype(S)::value, buf = decltype(BUF)::value;
        if constexpr (r == 0) af[buf][0] = opA.template read<0, s>(ua);
        else if constexpr (r <= 8) bfr[buf][r - 1] = opB.template read<r - 1, s>(ub);
        else af[buf][r - 8] = opA.template read<r - 8, s>(ua);
    };
    // one step: products on set BUF; reads of the set of step S in (ua, ub); loads
    // L(0..n-1) from product first on, every gap-th
    auto step = [&](auto BUF, auto S, uint32_t ua, uint32_t ub, auto FIRST, auto GAP,
                    auto COUNT, auto&& load) {
        constexpr int buf = decltype(BUF)::value, first = decltype(FIRST)::value,
                      gap = decltype(GAP)::value, n = decltype(COUNT)::value;
        constexpr bool last = n == 0;          // (a tile's last stage, which loads nothing)
        static_assert(n == 0 || first + gap * (n - 1) < 64, "loads behind the products");
        unroll<64>([&](auto Q) {
            constexpr int q = decltype(Q)::value;
            if constexpr (last)                // (columns as rows)
                acc[q / 8][q % 8] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    bfr[buf][q % 8], af[buf][q / 8], acc[q / 8][q % 8], 0, 0, 0);
            else
                mfma16(acc[q / 8][q % 8], bfr[buf][q % 8], af[buf][q / 8]);
            if constexpr (q % 2 == 0 && q < 32 && !(last && buf == 1))
                read1(std::integral_constant<int, q / 2>{}, S, std::integral_constant<int, 1 - buf>{},
                      ua, ub);
            if constexpr (q >= first && (q - first) % gap == 0 && (q - first) / gap < n)
                load(std::integral_constant<int, (q - first) / gap>{});
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    typedef std::integral_constant<int, 0> I0;
    typedef std::integral_constant<int, 1> I1;

    // units 0 .. 3: stages 0 and 1
    unroll<4>([&](auto U) {
        constexpr int u = decltype(U)::value;
        const i32x4_t rs = u % 2 ? rsB(u / 2) : rsA(u / 2);
        unroll<NL>([&](auto I) {
            if constexpr (u % 2) opB.template load<decltype(I)::value>(rs, slot(u));
            else opA.template load<decltype(I)::value>(rs, slot(u));
        });
    });
    stage_barrier<NL * 2>();                           // stage 0 landed
    unroll<16>([&](auto R) { read1(R, I0{}, I0{}, unit(0), unit(1)); });
    int qa = 0;                                        // slot of A's unit of stage j
    // stage j: units 2j, 2j+1; A of stage j+2 is loaded in its first step, B of stage
    // j+2 right behind its barrier
    typedef std::integral_constant<int, 32 / NL> GAP;
    typedef std::integral_constant<int, NL> CNT;
#pragma unroll 1
    for (int j = 0; j + 1 < nj; ++j) {
        const uint32_t ua = unit(qa), ub = unit(wrap(qa + 1));
        const i32x4_t ra = rsA(j + 2);
        step(I0{}, I1{}, ua, ub, std::integral_constant<int, 33>{}, GAP{}, CNT{}, [&](auto I) {
            opA.template load<decltype(I)::value>(ra, slot(wrap(qa + 4)));
        });
        stage_barrier<NL>();                           // stage j read, stage j+1 landed
        const i32x4_t rb = rsB(j + 2);
        const int qn = wrap(qa + 2);
        step(I1{}, I0{}, unit(qn), unit(wrap(qn + 1)), I1{}, GAP{}, CNT{}, [&](auto I) {
            opB.template load<decltype(I)::value>(rb, slot(qa));
        });
        qa = qn;
    }
    step(I0{}, I1{}, unit(qa), unit(wrap(qa + 1)), I1{}, I1{}, I0{}, [](auto) {});
    step(I1{}, I0{}, 0u, 0u, I1{}, I1{}, I0{}, [](auto) {});
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");    // (loads of the empty stages)
    // (a row of fragments at a time, so that the others stay where they are)
    const bool part = Epi::kSplits && ti.slot >= 0;
    unroll<8>([&](auto I) {
        const int rl = wm * 128 + I * 16 + (lane & 15);
        if (part) store_part<Quads16, 256, 256>(p.part, ti, rl, wn * 128, acc[I]);
        else epi.template row<Quads16>(ti, rl, wn * 128, acc[I], asked[I]);
        __builtin_amdgcn_sched_barrier(0);
    });
}

// The scores, on two cards: 8192 x 50257 from d 1024 900 and 935 us with 16-bit scores
// stored (935 and 900 TFLOP/s; 16 stages and a 10 us epilogue a tile, pipes busy 42%), a
// tenth masked and the loss alone 620 and 645; 16 tokens, d 4096, 128000 entries 228-236
// us (Wv at 4.6 TB/s).
template <int ALAY, int BLAY, class Epi>
__global__ __launch_bounds__(256, 1) void head_product_kernel(HeadGemm<bf16_t> p, Epi epi) {
    __shared__ __attribute__((aligned(UNIT))) uint8_t ringbuf[kRingBytes];
    head_product_body<ALAY, BLAY>(p, epi, blockIdx.x, ringbuf);
}

// fp32: 128 x 128 tiles, 4 waves of 64 x 64, v_mfma_f32_32x32x2_f32, two
// workgroups a compute unit.  The operands' units are those of the bf16 products
// with an element as two: K-major 128 rows of 32 steps (128 bytes), M/N-major 32
// steps of 128 elements.  A matrix instruction takes one step from each half of
// the wave; the halves take steps 0-3 and 4-7 of every eight, so that K-major
// operands are read four steps at a time.  The matrix pipe is busy for 4096 cycles a
// stage of 32 KB: two stages in LDS, the compiler's order of instructions.
constexpr int FBM = 128, FBK = 32;
template <int LAY>
struct HeadOperandF32 : HeadOperand<LAY, LAY == KMAJ ? 64 : 32, 4, LAY == KMAJ ? 128 : 256> {
    typedef HeadOperand<LAY, LAY == KMAJ ? 64 : 32, 4, LAY == KMAJ ? 128 : 256> Base;
    int w0;
    __device__ __forceinline__ void init(const float* P, long ld, int rows, int k_lim, int w0_) {
        Base::init(reinterpret_cast<const bf16_t*>(P), ld * 2, LAY == KMAJ ? rows : rows * 2, k_lim,
                   0);
        w0 = w0_;
    }
    __device__ __forceinline__ i32x4_t words32(int k0, bool some) const {
        return Base::words(LAY == KMAJ ? (long)k0 * 2 : (long)k0, some);
    }
    // four steps (4 (lane / 32) on of the eight 8 b on) of row 32 i + lane % 32
    __device__ __forceinline__ f32x4 read4(uint32_t u, int i, int b) const {
        const int lane = threadIdx.x & 63, h = lane >> 5, r = w0 + i * 32 + (lane & 31);
        if constexpr (LAY == KMAJ) {
            const uint32_t o = u + r * 128 + (((2 * b + h) ^ ((r ^ (r >> 3)) & 7)) << 4);
            return __builtin_bit_cast(f32x4, *reinterpret_cast<typename Base::lds_u32x4_t*>(o));
        } else {
            typedef __attribute__((address_space(3))) const float lds_f32_t;
            f32x4 v;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int k = 8 * b + 4 * h + e;
                v[e] = *reinterpret_cast<lds_f32_t*>(u + k * 512 + (Base::mn_swz(k, r >> 2) << 4) +
                                                     (r & 3) * 4);
            }
            return v;
        }
    }
};

constexpr int kRingBytesF32 = 65536;
constexpr int kSumStages = 2;
template <int ALAY, int BLAY, class Epi>
__device__ __forceinline__ void head_product_body(const HeadGemm<float>& p, const Epi& epi,
                                                  int block, uint8_t* ringbuf) {
    constexpr int UNIT = 16384, STAGE = 2 * UNIT;
    static_assert(2 * STAGE <= kRingBytesF32, "LDS");
    if (piece_done(p)) return;
    const HeadTile ti = head_tile<FBM, FBM>(p, block);
    if (!ti.live) return;
    const int lane = threadIdx.x & 63;
    const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wv >> 1, wn = wv & 1;
    typename Epi::Ask asked[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) asked[i] = epi.ask(ti, wm * 64 + i * 32 + (lane & 31));
    typedef HeadOperandF32<ALAY> OpA;
    typedef HeadOperandF32<BLAY> OpB;
    constexpr int NL = OpA::NLOAD;
    static_assert(NL == 4 && OpB::NLOAD == 4, "16 KB units");
    OpA opA;
    OpB opB;
    opA.init(p.A + (ALAY == KMAJ ? (long)ti.m0 * p.lda : (long)ti.m0), p.lda, ti.rows, ti.k1,
             wm * 64);
    opB.init(p.B + (BLAY == KMAJ ? (long)ti.n0 * p.ldb : (long)ti.n0), p.ldb, ti.cols, ti.k1,
             wn * 64);
    f32x16 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
    const int nj = (ti.k1 - ti.k0 + FBK - 1) / FBK;
    const uint32_t ring0 = lds_addr(ringbuf);
    const uint32_t lds0 = __builtin_amdgcn_readfirstlane(ring0 + wv * 1024);
    auto issue = [&](int j) {
        const i32x4_t ra = opA.words32(ti.k0 + j * FBK, true);
        const i32x4_t rb = opB.words32(ti.k0 + j * FBK, true);
        const uint32_t at = lds0 + (uint32_t)((j & 1) * STAGE);
        unroll<NL>([&](auto I) { opA.template load<decltype(I)::value>(ra, at); });
        unroll<NL>([&](auto I) { opB.template load<decltype(I)::value>(rb, at + UNIT); });
    };
    if (nj > 0) issue(0);
    // the sums of kSumStages stages are made by themselves and then added: a chain of
    // hundreds of additions, each rounded at the size of the whole, would lose more than
    // the rounding of z that the loss shows
    // NI: the wave's row fragments that have rows; up to 32 tokens half of the waves
    // then have none and the others one of two (1 token, d 1600, 101207 entries: 970 us
    // to 640; 24, 512, 5000: 90 to 69; full tiles the same)
    auto products = [&](auto NI) {
        constexpr int ni = decltype(NI)::value;
#pragma unroll 1
        for (int j0 = 0; j0 < nj; j0 += kSumStages) {
            f32x16 sum[2][2] = {};
#pragma unroll
            for (int k = 0; k < kSumStages; ++k) {
                const int j = j0 + k;
                if (k > 0 && j >= nj) break;
                stage_barrier<0>();        // stage j landed, stage j - 1 read by every wave
                if (j + 1 < nj) issue(j + 1);
                uint32_t u = ring0 + (uint32_t)((j & 1) * STAGE);
                asm volatile("" : "+s"(u));    // (addresses of both stages would not fit the registers)
                f32x4 fa[2][2], fc[2][2];
                auto read = [&](int b) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (i < ni) fa[b & 1][i] = opA.read4(u, i, b);
                        if (ni > 0) fc[b & 1][i] = opB.read4(u + UNIT, i, b);
                    }
                };
                read(0);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    if (b < 3) read(b + 1);
                    __builtin_amdgcn_sched_barrier(0);     // (those reads before these products)
                    const f32x4(&a)[2] = fa[b & 1], (&c)[2] = fc[b & 1];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < ni; ++i)
#pragma unroll
                            for (int n = 0; n < 2; ++n)    // (columns as rows)
                                sum[i][n] = __builtin_amdgcn_mfma_f32_32x32x2f32(
                                    c[n][e], a[i][e], sum[i][n], 0, 0, 0);
                }
            }
#pragma unroll
            for (int i = 0; i < ni; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n) acc[i][n] += sum[i][n];
        }
    };
    const int some = (ti.rows - wm * 64 + 31) / 32;
    if (some >= 2) products(std::integral_constant<int, 2>{});
    else if (some == 1) products(std::integral_constant<int, 1>{});
    else products(std::integral_constant<int, 0>{});
    // 32 x 32 fragments: row = lane % 32, four columns by register and lane / 32
    unroll<2>([&](auto I) {
        f32x4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q)
#pragma unroll
            for (int u = 0; u < 4; ++u) v[q][u] = acc[I][q >> 2][(q & 3) * 4 + u];
        const int rl = wm * 64 + I * 32 + (lane & 31);
        if (Epi::kSplits && ti.slot >= 0)
            store_part<Quads32, FBM, FBM>(p.part, ti, rl, wn * 64, v);
        else
            epi.template row<Quads32>(ti, rl, wn * 64, v, asked[I]);
    });
}

template <int ALAY, int BLAY, class Epi>
__global__ __launch_bounds__(256, 2) void head_product_f32_kernel(HeadGemm<float> p, Epi epi) {
    __shared__ __attribute__((aligned(16384))) uint8_t ringbuf[kRingBytesF32];
    head_product_body<ALAY, BLAY>(p, epi, blockIdx.x, ringbuf);
}

// Bound by the matrix pipes and the power they draw: 68% of their cycles busy at
// 1.9 GHz; on two cards 8192 tokens, d 1024, 50257 entries 1200 and 1267 us (1405 and
// 1331 TFLOP/s), 16384, 4096, 128000 23.7 and 24.8 ms (1450 and 1384); fp32 1999, 1088,
// 8191 618-650 us (104-110).
// Both gradients' products in one launch: blocks 0 .. nx - 1 make dx = dz Wv, the
// others dWv = dz^T x, so that the second fills the rounds that the first leaves.
__global__ __launch_bounds__(256, 1) void head_grads_kernel(HeadGemm<bf16_t> gx,
                                                            EpiRows<bf16_t> ex,
                                                            HeadGemm<bf16_t> gw,
                                                            EpiSum<bf16_t> ew, int nx) {
    __shared__ __attribute__((aligned(UNIT))) uint8_t ringbuf[kRingBytes];
    const int b = blockIdx.x;
    if (b < nx) head_product_body<KMAJ, MNMAJ>(gx, ex, b, ringbuf);
    else head_product_body<MNMAJ, MNMAJ>(gw, ew, b - nx, ringbuf);
}
__global__ __launch_bounds__(256, 2) void head_grads_kernel(HeadGemm<float> gx, EpiRows<float> ex,
                                                            HeadGemm<float> gw, EpiSum<float> ew,
                                                            int nx) {
    __shared__ __attribute__((aligned(16384))) uint8_t ringbuf[kRingBytesF32];
    const int b = blockIdx.x;
    if (b < nx) head_product_body<KMAJ, MNMAJ>(gx, ex, b, ringbuf);
    else head_product_body<MNMAJ, MNMAJ>(gw, ew, b - nx, ringbuf);
}

// The rest tiles of a product whose reduction was split: their parts added in
// order and put where the product's epilogue puts them.  8 elements a thread.
template <int BM, int BN, typename T, class Epi>
__device__ __forceinline__ void head_join_body(const HeadGemm<T>& p, const Epi& epi, int block) {
    constexpr int PER = BM * BN / 8192;               // blocks of a tile
    const int S = *p.plan;
    if (S == 1 || piece_done(p)) return;
    const int n = piece_rows(p.count, p.p0, p.piece, p.piece);
    const int M = p.dyn == 1 ? n : p.M;
    const int nM = (M + BM - 1) / BM, nN = (p.N + BN - 1) / BN;
    const int full = nM * nN / kRound * kRound, R = nM * nN - full;
    const int tile = block / PER;
    if (tile >= R) return;
    int m0, n0;
    head_origin<BM, BN>(full + tile, nM, nN, m0, n0);
    const int e = ((block % PER) * 1024 + threadIdx.x) * 8;
    const int r = m0 + e / BN, c = n0 + e % BN;
    if (r >= M || c >= p.N) return;
    const float* q = p.part + (long)tile * (BM * BN) + e;
    const long stride = (long)R * (BM * BN);
    float v[8];
    ld8(q, v);
#pragma unroll 4
    for (int s = 1; s < S; ++s) {
        float a[8];
        ld8(q + s * stride, a);
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] += a[u];
    }
    epi.put8(r, c, v);
}
template <int BM, typename T>
__global__ __launch_bounds__(1024) void head_join_kernel(HeadGemm<T> gx, EpiRows<T> ex,
                                                         HeadGemm<T> gw, EpiSum<T> ew, int nx) {
    const int b = blockIdx.x;
    if (b < nx) head_join_body<BM, BM>(gx, ex, b);
    else head_join_body<BM, BM>(gw, ew, b - nx);
}

// The scores of a product that was split: their parts added in order, then what
// EpiScores does.  8 columns a thread, the W columns of a statistic in W / 8 lanes.
template <int BM, int W, typename T>
__global__ __launch_bounds__(1024) void head_scores_join_kernel(HeadGemm<T> p, EpiScores es) {
    constexpr int PER = BM * BM / 8192;               // blocks of a tile
    const int n = piece_rows(p.count, p.p0, p.piece, p.piece);
    const int nM = (n + BM - 1) / BM, nN = (p.N + BM - 1) / BM, R = nM * nN;
    const int tile = blockIdx.x / PER;
    if (tile >= R) return;
    int m0, n0;
    head_origin<BM, BM>(tile, nM, nN, m0, n0);
    const int e = ((blockIdx.x % PER) * 1024 + threadIdx.x) * 8;
    const long r = m0 + e / BM;
    const int c = n0 + e % BM, left = es.V - c;
    const bool in = r < n;                            // (all lanes stay, for the exchanges)
    float v[8] = {};
    const float* q = p.part + (long)tile * (BM * BM) + e;
    for (int k = 0; k < p.split; ++k) {
        const float* a = q + (long)k * R * (BM * BM);
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (in && left > 4 * h) {                 // quads that were stored
                const f32x4 b = *reinterpret_cast<const f32x4*>(a + 4 * h);
#pragma unroll
                for (int u = 0; u < 4; ++u) v[4 * h + u] += b[u];
            }
    }
    const int y = in && es.labels ? es.labels[r] - c : -1;
#pragma unroll
    for (int u = 0; u < 8; ++u)
        if (u == y && u < left) es.zl[r] = v[u];
    if (es.Z && in && c < es.ldz) st8(es.Z + r * es.ldz + c, v);
    float m = -INFINITY;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        v[u] = u < left ? v[u] : -INFINITY;
        m = fmaxf(m, v[u]);
    }
#pragma unroll
    for (int k = 1; k < W / 8; k *= 2) m = fmaxf(m, __shfl_xor(m, k));
    const float ref = m == -INFINITY ? 0.0f : m, m2 = ref * kLog2e, mt = ref * es.l2t;
    const float rho = fmaf(ref, kLog2e, -m2);
    float x[8], s = 0.0f, t = 0.0f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
        x[u] = fmaf(v[u], kLog2e, -m2);
        s += exp2_hw(x[u]);
        if (es.tstat) t += exp2_hw(fmaf(v[u], es.l2t, -mt));
    }
    if (W == 128 && es.code && in && c < es.ldz)
        *reinterpret_cast<u32x4_t*>(es.code + r * es.ldz + c) =
            u32x4_t{code_pair(x[0], x[1], rho), code_pair(x[2], x[3], rho),
                    code_pair(x[4], x[5], rho), code_pair(x[6], x[7], rho)};
#pragma unroll
    for (int k = 1; k < W / 8; k *= 2) {
        s += __shfl_xor(s, k);
        if (es.tstat) t += __shfl_xor(t, k);
    }
    if (!in || (threadIdx.x & (W / 8 - 1))) return;
    const long at = (long)(c / W) * es.sp + r * es.sr;
    es.stat[at] = make_float2(m, s);
    if (es.tstat) es.tstat[at] = t;
}

// --------------------------------------------------------- normalisers

// The normaliser of a row in units of log2: 2^(a + b) = sum_v e^z, a = the maximum
// times L, rounded (the m' of the sums), b = log2 of the sum relative to it.
struct Norm2 {
    float a, b;
};
// ln of the sum: m + ln 2 (b - (m L - a)), the bracket's m L - a exact in a fused
// multiply-add, so that the rounding of a does not reach the result.
__device__ __forceinline__ float norm_ln(Norm2 n, float m, float scale, float l2) {
    return fmaf(kLn2, n.b - fmaf(m, l2, -n.a), m * scale);
}
// p = e^(z - lse) (l2 = L, or L / tau at the temperature)
__device__ __forceinline__ float norm_p(Norm2 n, float z, float l2) {
    return exp2_hw(fmaf(z, l2, -n.a) - n.b);
}

// A part's factor relative to the maximum mx: 2^(m' - mx'), m' as in the sums; a
// part without a column (m = -inf) adds its sum as it is: 0, or the NaN of a score.
// Both products are rounded by themselves: fused with the difference one of them
// would not be, and the factor of the part that holds the maximum not 1 but off by
// the rounding of m L, once for every merge (lse up to 127: 2.3e-5).
__device__ __forceinline__ float part_factor(float m, float mx, float l2) {
#pragma clang fp contract(off)
    return m == -INFINITY ? 1.0f : exp2_hw(m * l2 - mx * l2);
}

// 8192 rows of 393 parts: 7 us (26 MB, 3.7 TB/s); 16 rows of 1000: 6.6, latency.
// A loss without gradient: lse of every row from its parts, 16 rows a block, 64
// threads share a row's parts; loss and lse go to the row's token.
__global__ __launch_bounds__(1024) void head_lse_kernel(
    const float2* __restrict__ stat, int parts, long ldr, const float* __restrict__ zl,
    const int32_t* __restrict__ labels, int V, const int32_t* __restrict__ rows,
    const int32_t* __restrict__ count, int p0, int piece, float* __restrict__ loss,
    float* __restrict__ lse) {
    __shared__ float sm[16][16], ss[16][16];
    const int n = piece_rows(count, p0, piece, piece);
    if (blockIdx.x * 16 >= n) return;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, k = lane & 15;
    const long r = (long)blockIdx.x * 16 + k;
    float m = -INFINITY, s = 0.0f;
    auto add = [&](float m1, float s1) {
        const float mx = fmaxf(m, m1);
        s = s * part_factor(m, mx, kLog2e) + s1 * part_factor(m1, mx, kLog2e);
        m = mx;
    };
    if (r < n) {
#pragma unroll 4
        for (int q = w * 4 + (lane >> 4); q < parts; q += 64) {
            const float2 a = stat[q * ldr + r];
            add(a.x, a.y);
        }
    }
    {
        const F2 m1 = swap16(m), s1 = swap16(s);
        m = m1.a, s = s1.a;
        add(m1.b, s1.b);
    }
    {
        const F2 m1 = swap32(m), s1 = swap32(s);
        m = m1.a, s = s1.a;
        add(m1.b, s1.b);
    }
    if (lane < 16) sm[w][k] = m, ss[w][k] = s;
    __syncthreads();
    if (threadIdx.x >= 16 || r >= n) return;
    for (int q = 1; q < 16; ++q) add(sm[q][k], ss[q][k]);
    const int tok = rows ? rows[p0 + r] : (int)r;
    const bool on = in_vocab(labels[tok], V);
    const float l = norm_ln({m * kLog2e, __builtin_amdgcn_logf(s)}, m, 1.0f, kLog2e);
    loss[tok] = on ? l - zl[r] : 0.0f;
    if (lse) lse[tok] = on ? l : 0.0f;
}

// ----------------------------------------------------------------- dz

// The second bf16 terms of two values whose first ones are `hi`.
__device__ __forceinline__ uint32_t second_terms(float a, float b, uint32_t hi) {
    return pack_bf16x2(a - __uint_as_float(hi << 16), b - __uint_as_float(hi & 0xffff0000u));
}
// What a value loses as an element of T (exact in fp32); 0 if it is not finite there.
template <typename T>
__device__ __forceinline__ float lost_of(float v) {
    if constexpr (sizeof(T) == 4) {
        return 0.0f;
    } else {
        const float lost = v - bf16_to_f32(f32_to_bf16(v));
        return fabsf(lost) < INFINITY ? lost : 0.0f;
    }
}
// One element of dz, in one or two terms.
template <bool TERMS, typename T>
__device__ __forceinline__ float put_dz(T* g, long second, float v) {
    const float lost = lost_of<T>(v);
    Elem<T>::st(g, v);
    if (TERMS) Elem<T>::st(g + second, lost);
    return lost;
}

struct HeadDz {
    const float* Z;          // [piece][ldz] scores, or
    const uint16_t* code;    // coded ones and the labels' scores
    const float* zl;         // [piece]
    long ldz;
    void* G;                 // [piece][ldg] dz, its second term (if any) ldz further
    long ldg;
    HeadTop* top;            // [piece] (bf16)
    int segs, seg;           // segments of a row, their length (a multiple of 256)
    int V;
    const int32_t* rows;
    const int32_t* count;
    int p0, piece;
    const float2* stat;      // [piece][parts] the scores' statistics
    const float* tstat;
    int parts;
    float *loss, *lse;       // [T] or NULL
    const int32_t* labels;   // or NULL
    const float* weight;     // [T] or NULL: 1
    const int32_t* tidx;     // [T,K] or NULL
    const float* tlogit;
    const float* tweight;    // [T] or NULL: 1
    int K;
    float tau, inv_tau, l2t;
    float* kd;               // [T] or NULL
    int grad;
};

// Bound by HBM: 8192 x 50257 in bf16 from coded scores 298 us (1.65 GB, 5.5 TB/s), with
// a teacher from fp32 ones 533 us (2.5 GB, 4.7 TB/s; two exponentials an entry).
// One wave a row, or a segment of one when the rows are few.  The dz of the label
// and the teacher's slots are written behind the others (an entry named twice by
// its first slot, with the slots' q added in order).
template <typename T, bool CODED, bool TERMS>
__global__ __launch_bounds__(256) void head_dz_kernel(HeadDz p) {
    static_assert((!CODED && !TERMS) || sizeof(T) == 2, "coded scores, two terms: bf16 dz");
    __shared__ int s_idx[CODED ? 1 : 4][kMaxK];
    __shared__ float s_q[CODED ? 1 : 4][kMaxK];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int n = piece_rows(p.count, p.p0, p.piece, 0);
    const int item = blockIdx.x * 4 + w;
    const int r = item / p.segs, part = item - r * p.segs;
    if (r >= n) return;                       // whole waves; no block barrier below
    const int t = p.rows[p.p0 + r];
    const float* z = CODED ? nullptr : p.Z + (long)r * p.ldz;
    const int c0 = part * p.seg, c1 = (int)min(p.ldz, (long)c0 + p.seg);
    int label = p.labels ? p.labels[t] : -1;
    if (!in_vocab(label, p.V)) label = -1;
    const float wce = label >= 0 ? (p.weight ? p.weight[t] : 1.0f) : 0.0f;
    // the row's normaliser (and that at the temperature) from its parts
    float m = -INFINITY;
    const float2* sp = p.stat + (long)r * p.parts;
    for (int j = lane; j < p.parts; j += 64) m = fmaxf(m, sp[j].x);
    m = wave_max(m);
    float s = 0.0f, st = 0.0f;
    for (int j = lane; j < p.parts; j += 64) {
        const float2 a = sp[j];
        s += a.y * part_factor(a.x, m, kLog2e);
        if (p.tstat) st += p.tstat[(long)r * p.parts + j] * part_factor(a.x, m, p.l2t);
    }
    const Norm2 nm = {m * kLog2e, __builtin_amdgcn_logf(wave_sum(s))};
    const Norm2 tn = {m * p.l2t, p.tstat ? __builtin_amdgcn_logf(wave_sum(st)) : 0.0f};
    if (p.loss && part == 0 && lane == 0) {
        const float l = norm_ln(nm, m, 1.0f, kLog2e);
        p.loss[t] = label >= 0 ? l - (CODED ? p.zl[r] : z[label]) : 0.0f;
        if (p.lse) p.lse[t] = label >= 0 ? l : 0.0f;
    }
    if constexpr (CODED) {
        // every row has a label; dz = w 2^(m L - step * code - log2 of the sum), m the part's
        bf16_t* g = static_cast<bf16_t*>(p.G) + (long)r * p.ldg;
        const uint16_t* cr = p.code + (long)r * p.ldz;
        constexpr int U = 4;                  // units of 512 in flight
        for (int c = c0 + lane * 8; c < c1; c += 512 * U) {
            u32x4_t w[U];
            float top[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + 512 * u < c1) {       // read once: not kept
                    w[u] = __builtin_nontemporal_load(
                        reinterpret_cast<const u32x4_t*>(cr + c + 512 * u));
                    top[u] = sp[(c + 512 * u) >> 7].x;
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int cu = c + 512 * u;
                if (cu >= c1) break;
                const float b = fmaf(top[u], kLog2e, -nm.a) - nm.b;
                u32x4_t o, o2;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float lo = (float)(w[u][e] & 0xffffu), hi = (float)(w[u][e] >> 16);
                    const float vl = wce * exp2_hw(fmaf(lo, -kCodeStep, b));
                    const float vh = wce * exp2_hw(fmaf(hi, -kCodeStep, b));
                    const float a = cu + 2 * e < p.V ? vl : 0.0f;
                    const float b2 = cu + 2 * e + 1 < p.V ? vh : 0.0f;
                    o[e] = pack_bf16x2(a, b2);
                    if (TERMS) o2[e] = second_terms(a, b2, o[e]);
                }
                const bool on = wce != 0.0f;
                *reinterpret_cast<u32x4_t*>(g + cu) = on ? o : u32x4_t{0, 0, 0, 0};
                if (TERMS)
                    *reinterpret_cast<u32x4_t*>(g + p.ldz + cu) = on ? o2 : u32x4_t{0, 0, 0, 0};
            }
        }
        wave_mem_sync();
        if (lane == 0 && label >= c0 && label < c1) {
            const float v = wce != 0.0f ? wce * norm_p(nm, p.zl[r], kLog2e) - wce : 0.0f;
            const float lost = put_dz<TERMS>(g + label, p.ldz, v);
            p.top[r] = {label, lost};
        }
        return;
    }

    // the teacher's distribution
    constexpr int PL = kMaxK / 64;
    int idx[PL];
    float q[PL], zt[PL];
    float wkd = 0.0f;
    if (p.tidx) {
        float hi = -INFINITY;
        bool some = false;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int j = lane + 64 * u;
            idx[u] = -1;
            q[u] = -INFINITY;
            if (j < p.K && slot_on(p.tidx, p.tlogit, (long)t * p.K + j, p.V)) {
                some = true;
                idx[u] = p.tidx[(long)t * p.K + j];
                q[u] = p.tlogit[(long)t * p.K + j];
                hi = fmaxf(hi, q[u]);
            }
        }
        hi = wave_max(hi);
        const bool any = __ballot(some) != 0;
        const float ref = hi > -INFINITY ? hi : 0.0f;      // (NaNs alone: they show)
        float tot = 0.0f;
        float lq[PL];
        // the difference first: rounded, s / tau would be off by 2^-24 of itself, which at
        // a low temperature is much in q (1e-3 for a score of 16 at 0.001)
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            lq[u] = (q[u] - ref) * p.inv_tau;
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
            if (q[u] != 0.0f)                 // ln p = ln 2 log2 p
                kd += q[u] * (lq[u] - ltot - kLn2 * (fmaf(zt[u], p.l2t, -tn.a) - tn.b));
            if (j < p.K) s_idx[w][j] = idx[u], s_q[w][j] = q[u];
        }
        kd = wave_sum(kd);
        if (part == 0 && lane == 0 && p.kd) p.kd[t] = any ? kd * p.tau * p.tau : 0.0f;
        wkd = any ? p.tau * (p.tweight ? p.tweight[t] : 1.0f) : 0.0f;
    }
    if (!p.grad) return;
    const float zy = label >= 0 ? z[label] : 0.0f;
    wave_lds_sync();

    T* g = static_cast<T*>(p.G) + (long)r * p.ldg;
    auto ce = [&](float v) { return wce * norm_p(nm, v, kLog2e); };
    auto kl = [&](float v) { return wkd * norm_p(tn, v, p.l2t); };
    auto stream = [&](auto&& dense) {
        constexpr int U = 4;                  // units in flight
        for (int c = c0 + lane * 4; c < c1; c += 256 * U) {
            f32x4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (c + 256 * u < c1)          // read once: not kept (565 us to 466, 8192 x 50257)
                    v[u] = __builtin_nontemporal_load(
                        reinterpret_cast<const f32x4*>(z + c + 256 * u));
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int cu = c + 256 * u;
                if (cu >= c1) break;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[u][e] = cu + e < p.V ? dense(v[u][e]) : 0.0f;
                if constexpr (sizeof(T) == 4) {
                    *reinterpret_cast<f32x4*>(g + cu) = v[u];
                } else {
                    const uint2 o =
                        make_uint2(pack_bf16x2(v[u][0], v[u][1]), pack_bf16x2(v[u][2], v[u][3]));
                    *reinterpret_cast<uint2*>(g + cu) = o;
                    if (TERMS)
                        *reinterpret_cast<uint2*>(g + p.ldz + cu) =
                            make_uint2(second_terms(v[u][0], v[u][1], o.x),
                                       second_terms(v[u][2], v[u][3], o.y));
                }
            }
        }
    };
    // a weight of zero leaves its term out (no 0 times infinity)
    auto at = [&](float v) { return (wce != 0.0f ? ce(v) : 0.0f) + (wkd != 0.0f ? kl(v) : 0.0f); };
    if (wkd == 0.0f && wce != 0.0f) stream(ce);
    else if (wce == 0.0f && wkd != 0.0f) stream(kl);
    else stream(at);
    wave_mem_sync();
    // the label and the teacher's slots: written by the segment that has them; the
    // first segment finds which of them loses most in bf16
    auto mine = [&](int v) { return v >= c0 && v < c1; };
    bool label_named = false;
    HeadTop top = {0, 0.0f};
    auto put = [&](int v, float dz) {
        const float lost = lost_of<T>(dz);
        if (fabsf(lost) > fabsf(top.lost)) top = {v, lost};
        if (mine(v)) put_dz<TERMS>(g + v, p.ldz, dz);
    };
    if (p.tidx) {
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int j = lane + 64 * u;
            if (j >= p.K || idx[u] < 0) continue;
            if (idx[u] == label) label_named = true;
            if (part > 0 && !mine(idx[u])) continue;
            float sum = 0.0f;
            bool first = true;
            for (int k = 0; k < p.K; ++k)
                if (s_idx[w][k] == idx[u]) {
                    first = first && k >= j;
                    sum += s_q[w][k];
                }
            if (first) put(idx[u], at(zt[u]) - wkd * sum - (idx[u] == label ? wce : 0.0f));
        }
    }
    if (label >= 0 && __ballot(label_named) == 0 && lane == 0) put(label, at(zy) - wce);
    if (sizeof(T) == 2 && part == 0) {
        const float most = wave_max(fabsf(top.lost));
        const int from = __ffsll((long long)__ballot(fabsf(top.lost) == most)) - 1;
        if (lane == from) p.top[r] = top;
    }
}

// ------------------------------------------------------------- the calls

inline bool head_sizes_ok(int T, int d, int V, int K, moe_dtype dt) {
    return T >= 0 && T <= (1 << 24) && d >= 64 && d <= 65536 && d % 64 == 0 && V >= 1 &&
           V <= (1 << 20) && K >= 0 && K <= kMaxK && (dt == MOE_F32 || dt == MOE_BF16);
}

constexpr size_t kHeadLimit = (size_t)8 << 30;
constexpr int kSubUnits = 11;          // row tiles whose scores are held at a time, at most
// scores of a piece: its score product's blocks (a thread for 64 of them, in fp32)
// stay below a launch's 2^32 threads
constexpr long kPieceScores = 1l << 37;

// A call takes its tokens in `pieces` of `piece` rows, whose dz (or x alone, for a
// loss without gradient) is held at a time, and a piece in steps of `sub`
// rows, whose scores are: 4 (coded: 2) bytes a score, 2 (fp32: 4) for dz.
struct HeadPlan {
    int piece, pieces, sub, parts;
    long ldz;
    int segs, seg;                     // of a row of dz
    size_t rows, clab, count, plan, act, xc, zl, top, stat, tstat, z, g, part_dx, part_dw, acc, total;
    bool direct, coded;                // x as it is; scores in 16 bits
    bool slots_dx, slots_dw;           // products that may be split
    int terms;                         // of dz in dWv
};

// Slots that a product with up to `tiles` tiles and K reduction steps can use
// (no fewer for more of either, so that a workspace serves every smaller batch).
inline long head_slots(long tiles, long K, bool f32) {
    const long parts = std::min((long)kMaxParts, f32 ? (long)cdiv(K, 64) : (cdiv(K, 64) + 3) / 4l);
    return parts > 1 ? std::min((long)kMaxSlots, std::min(tiles, (long)kRound - 1) * parts) : 0;
}

// Parts of the scores' tiles: few tiles with a long reduction would leave most
// compute units idle.  A stage takes 1.2 us (fp32: 1.7), the parts' way through memory and the
// second launch about 12 (scores, one part / split: fp32 12 tokens, d 3712, 587
// entries 145 us / 29; 500, 1536, 2000 120 / 74; bf16 12, 3968, 2151 82 / 28; 1000, 2048,
// 2000 55 / 43; 16, 1536, 16000 40 / 30).
inline int head_score_split(long rows, int d, int V, bool f32) {
    const int bm = f32 ? 128 : 256, stages = cdiv(d, f32 ? 32 : 64);
    const long tiles = (long)cdiv(rows, bm) * cdiv(V, bm);
    if (tiles == 0 || tiles > kScoreSlots / 2 || stages < 24) return 1;
    return (int)std::min(kScoreSlots / tiles, (long)stages / 8);
}
// Their slots, for any number of rows up to `rows`.
inline long head_score_slots(long rows, int d, int V, bool f32) {
    const int bm = f32 ? 128 : 256;
    long most = 0;
    for (long k = 1; k <= std::min((long)cdiv(rows, bm), kScoreSlots / 2); ++k) {
        const int s = head_score_split(k * bm, d, V, f32);
        if (s > 1) most = std::max(most, k * cdiv(V, bm) * s);
    }
    return most;
}

HeadPlan head_layout(int T, int d, int V, int K, moe_dtype dt, int grad, int piece) {
    HeadPlan p;
    const size_t b = dt == MOE_BF16 ? 2 : 4;
    const bool store = grad || K > 0;
    const int bm = dt == MOE_BF16 ? 256 : 128, pc = dt == MOE_BF16 ? 128 : 64;
    p.coded = grad && K == 0 && dt == MOE_BF16;
    p.piece = piece;
    p.pieces = T == 0 ? 0 : cdiv(T, piece);
    // steps of 6 to 11 row tiles, of those the ones that leave the fewest rounds of
    // tiles partly empty (8192 tokens, 50257 entries: 9 row tiles 25 rounds, 8 28)
    const int units = cdiv(piece, kRowAlign), most = std::min(units, kSubUnits);
    int su = most;
    auto rounds = [&](int u) {
        auto of = [&](int n) {
            return cdiv((long)cdiv((long)n * kRowAlign, bm) * cdiv(V, bm), kRound);
        };
        return units / u * of(u) + (units % u ? of(units % u) : 0);
    };
    for (int u = most - 1; u >= 6; --u)
        if (rounds(u) < rounds(su)) su = u;
    p.sub = store ? std::min(piece, su * kRowAlign) : piece;
    // buffers for the longest step, as a smaller batch may choose it
    const size_t rmax = store ? std::min(piece, kSubUnits * kRowAlign) : piece;
    p.ldz = (long)align_up(V, 64);
    const bool bgrad = grad && dt == MOE_BF16;
    p.terms = bgrad && T <= kTermTokens ? 2 : 1;
    // rows of dz: for any smaller batch too
    const size_t gmax = bgrad ? std::max(piece, 2 * kTermTokens) : piece;
    p.parts = cdiv(V, bm) * (bm / pc);
    // about 8192 waves for a step's rows, each 2048 elements at least
    p.seg = std::max(2048, (int)align_up(cdiv(p.ldz * p.sub, 8192), 256));
    p.segs = cdiv(p.ldz, p.seg);
    size_t o = 0;
    auto take = [&](size_t bytes) {
        const size_t at = o;
        o = align_up(o + bytes, 256);
        return at;
    };
    p.rows = take((size_t)T * 4);
    p.clab = take(K == 0 ? (size_t)T * 4 : 0);
    p.count = take(4);
    p.plan = take(grad ? (size_t)p.pieces * 8 : 0);
    p.act = take(K > 0 ? (size_t)T * 4 : 0);
    // a row tile's worth of tokens and no gradient: every token is scored
    p.direct = !store && T <= kRowAlign;
    p.xc = take(p.direct ? 0 : gmax * d * b);
    p.zl = take(rmax * 4);
    p.top = take(bgrad ? (size_t)piece * 8 : 0);
    p.stat = take(rmax * p.parts * 8);
    p.tstat = take(K > 0 ? rmax * p.parts * 4 : 0);
    p.z = take(store ? rmax * p.ldz * (p.coded ? 2 : 4) : 0);
    p.g = take(grad ? gmax * p.ldz * b : 0);
    const long cols = cdiv(d, bm);
    const long sx = head_slots(cdiv(piece, bm) * cols, V, dt == MOE_F32);
    const long sw = head_slots(cdiv(V, bm) * cols, gmax, dt == MOE_F32);
    p.slots_dx = sx > 0, p.slots_dw = sw > 0;
    // (the scores' parts are done with before the gradients' come)
    const long ss = head_score_slots(rmax, d, V, dt == MOE_F32);
    p.part_dx = take((size_t)std::max(grad ? sx : 0l, ss) * bm * bm * 4);
    p.part_dw = take(grad ? (size_t)sw * bm * bm * 4 : 0);
    p.acc = take(grad && p.pieces > 1 ? (size_t)V * d * 4 : 0);
    p.total = o;
    return p;
}

// The plan with the largest piece whose workspace stays within `limit`, or the
// one with the smallest workspace if none does.  The fewest pieces of equal size
// (in whole row tiles), so that the last one is not a small rest.
HeadPlan head_plan(int T, int d, int V, int K, moe_dtype dt, int grad, size_t limit) {
    const int units = std::max(1, cdiv(T, kRowAlign));
    const int most = (int)std::min((long)units, std::max(1l, kPieceScores / kRowAlign / V));
    int lo = cdiv(units, most), hi = units;              // pieces: the fewest that fit
    auto of = [&](int pieces) {
        const int u = cdiv(units, pieces);
        return head_layout(T, d, V, K, dt, grad,
                           T <= kRowAlign ? std::max(T, 1) : u * kRowAlign);
    };
    const HeadPlan whole = of(lo);       // (often no running sum of dWv: it may be the smallest)
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

// Blocks of a product with up to m rows: its tiles, and the slots of its rest.
template <int BM, typename T>
int head_grid(const HeadGemm<T>& g, long m) {
    const long tiles = (long)cdiv(m, BM) * cdiv(g.N, BM);
    const long blocks = g.plan ? std::max(tiles, tiles / kRound * kRound + kMaxSlots)
                               : tiles * g.split;
    const long pad = NXCD * kXcdRun;
    return (int)((blocks + pad - 1) / pad * pad);
}
// Blocks that add up its rest tiles.
template <int BM, typename T>
int head_join_grid(const HeadGemm<T>& g, long m) {
    const long rest = std::min((long)kRound - 1, (long)cdiv(m, BM) * cdiv(g.N, BM));
    return g.plan ? (int)(rest * (BM * BM / 8192)) : 0;
}

template <class Epi>
void head_scores(const HeadGemm<bf16_t>& g, long m, const Epi& e, hipStream_t s) {
    MOE_LAUNCH("head_scores", s, head_product_kernel<KMAJ, KMAJ, Epi>
               <<<head_grid<256>(g, m), 256, 0, s>>>(g, e));
}
template <class Epi>
void head_scores(const HeadGemm<float>& g, long m, const Epi& e, hipStream_t s) {
    MOE_LAUNCH("head_scores", s, head_product_f32_kernel<KMAJ, KMAJ, Epi>
               <<<head_grid<FBM>(g, m), 256, 0, s>>>(g, e));
}

template <typename T>
moe_status head_run(const HeadCall& c, const HeadPlan& p, char* ws, hipStream_t s) {
    const bool teacher = c.K > 0, store = c.grad || teacher;
    int32_t* rows = reinterpret_cast<int32_t*>(ws + p.rows);
    int32_t* count = reinterpret_cast<int32_t*>(ws + p.count);
    int32_t* plan = c.grad ? reinterpret_cast<int32_t*>(ws + p.plan) : nullptr;
    int32_t* clab = teacher ? nullptr : reinterpret_cast<int32_t*>(ws + p.clab);
    float2* stat = reinterpret_cast<float2*>(ws + p.stat);
    float* tstat = teacher ? reinterpret_cast<float*>(ws + p.tstat) : nullptr;
    float* zl = reinterpret_cast<float*>(ws + p.zl);
    float* Z = store && !p.coded ? reinterpret_cast<float*>(ws + p.z) : nullptr;
    uint16_t* code = p.coded ? reinterpret_cast<uint16_t*>(ws + p.z) : nullptr;
    T* G = reinterpret_cast<T*>(ws + p.g);
    T* xc = reinterpret_cast<T*>(ws + p.xc);
    HeadTop* top = reinterpret_cast<HeadTop*>(ws + p.top);
    const long ldx = (long)c.d * p.terms, ldg = p.ldz * p.terms;
    const float inv_tau = 1.0f / c.tau, l2t = (float)(1.4426950408889634 / (double)c.tau);
    const int vpr = c.d * (int)sizeof(T) / 16;
    constexpr int BM = sizeof(T) == 2 ? 256 : FBM;
    HeadGemm<T> g;
    g.count = p.direct ? nullptr : count;
    if (!p.direct) {
        HeadTokens tk = {c.labels, c.V, teacher ? c.tidx : nullptr, c.tlogit, c.K, c.V, c.T};
        const HeadParts hp = {plan, plan ? p.pieces : 0, p.piece, c.d, c.V, BM, p.terms};
        const HeadStart st = {rows, clab, count, {c.loss, c.lse, c.kd}, hp};
        u32x4_t* dx0 = c.grad ? static_cast<u32x4_t*>(c.dx) : nullptr;
        // (a thread of the compaction looks at its tokens' slots itself: few)
        if (teacher && (long)c.T * c.K > 16384) {
            int32_t* a = reinterpret_cast<int32_t*>(ws + p.act);
            MOE_LAUNCH("head_active", s, head_active_kernel<<<cdiv(c.T, 4), 256, 0, s>>>(
                           c.labels, c.tidx, c.tlogit, c.T, c.K, c.V, a));
            tk.act = a, tk.limit = 2, tk.tidx = nullptr;
        }
        if (c.T <= kStartTokens && p.pieces == 1) {
            const int blocks = std::max(1, std::min(256, cdiv((long)c.T * vpr, 1024)));
            MOE_LAUNCH("head_start", s, head_start_kernel<<<blocks, 1024, 0, s>>>(
                           tk, st, static_cast<const u32x4_t*>(c.x), vpr,
                           reinterpret_cast<u32x4_t*>(xc), p.terms, dx0));
        } else {
            MOE_LAUNCH("head_compact", s, head_compact_kernel<<<1, 1024, 0, s>>>(tk, st));
        }
    }
    for (int i = 0; i < p.pieces; ++i) {
        const int p0 = i * p.piece, bound = std::min(p.piece, c.T - p0);
        if (!p.direct && (c.T > kStartTokens || p.pieces > 1)) {
            u32x4_t* dx0 = c.grad && i == 0 ? static_cast<u32x4_t*>(c.dx) : nullptr;
            HeadTokens tk = {c.labels, c.V, teacher ? c.tidx : nullptr, c.tlogit, c.K, c.V, c.T};
            if (teacher && (long)c.T * c.K > 16384) {
                tk.act = reinterpret_cast<int32_t*>(ws + p.act);
                tk.limit = 2, tk.tidx = nullptr;
            }
            MOE_LAUNCH("head_gather", s,
                       head_gather_kernel<<<head_blocks((long)(dx0 ? c.T : bound) * vpr), 256, 0, s>>>(
                           static_cast<const u32x4_t*>(c.x), rows, count, p0, p.piece, vpr,
                           reinterpret_cast<u32x4_t*>(xc), tk, dx0));
        }
        for (int q0 = 0; q0 < bound; q0 += p.sub) {
            const int s0 = p0 + q0, sn = std::min(p.sub, bound - q0);
            g.A = p.direct ? static_cast<const T*>(c.x) : xc + (long)q0 * ldx;
            g.lda = p.direct ? c.d : ldx, g.B = static_cast<const T*>(c.Wv), g.ldb = c.d;
            g.M = sn, g.N = c.V, g.K = c.d, g.dyn = 1, g.terms = 1, g.p0 = s0, g.piece = sn;
            g.plan = nullptr, g.part = reinterpret_cast<float*>(ws + p.part_dx);
            g.split = head_score_split(sn, c.d, c.V, sizeof(T) == 4);
            // statistics by row for head_dz, by part for head_lse; the label's score
            // comes from z where that is kept
            const EpiScores es = {c.V, stat, tstat, store ? 1 : (long)p.sub, store ? p.parts : 1, l2t,
                                  teacher ? nullptr : p.direct ? c.labels : clab + s0, zl, Z, code,
                                  p.ldz};
            if (g.split == 1) {
                head_scores(g, sn, es, s);
            } else {
                head_scores(g, sn, EpiParts{}, s);
                const int blocks = cdiv(sn, BM) * cdiv(c.V, BM) * (BM * BM / 8192);
                MOE_LAUNCH("head_scores_join", s,
                           head_scores_join_kernel<BM, (sizeof(T) == 2 ? 128 : 64), T>
                           <<<blocks, 1024, 0, s>>>(g, es));
            }
            if (!store) {
                MOE_LAUNCH("head_lse", s, head_lse_kernel<<<cdiv(sn, 16), 1024, 0, s>>>(
                               stat, p.parts, p.sub, zl, c.labels, c.V, p.direct ? nullptr : rows,
                               g.count, s0, sn, c.loss, c.lse));
                continue;
            }
            const int segs = c.grad ? p.segs : 1;
            const HeadDz dz = {Z, code, zl, p.ldz, G + (long)q0 * ldg, ldg,
                               top + q0, segs, p.seg, c.V, rows, count, s0, sn,
                               stat, tstat, p.parts, c.loss, c.lse, c.labels, c.weight, c.tidx,
                               c.tlogit, c.tweight, c.K, c.tau, inv_tau, l2t, c.kd, c.grad};
            const int blocks = cdiv((long)sn * segs, 4);
            auto launch = [&](auto CODED, auto TERMS) {
                MOE_LAUNCH("head_dz", s,
                           head_dz_kernel<T, decltype(CODED)::value, decltype(TERMS)::value>
                           <<<blocks, 256, 0, s>>>(dz));
            };
            typedef std::true_type Yes;
            typedef std::false_type No;
            if constexpr (sizeof(T) == 4) launch(No{}, No{});
            else if (p.coded && p.terms == 2) launch(Yes{}, Yes{});
            else if (p.coded) launch(Yes{}, No{});
            else if (p.terms == 2) launch(No{}, Yes{});
            else launch(No{}, No{});
        }
        if (!c.grad) continue;
        HeadGemm<T> gx = g, gw = g;
        gx.split = gw.split = 1;
        gx.p0 = gw.p0 = p0, gx.piece = gw.piece = p.piece;
        gx.A = gw.A = G, gx.lda = ldg, gw.lda = p.ldz;
        gx.B = static_cast<const T*>(c.Wv), gx.ldb = c.d;
        gx.M = bound, gx.N = c.d, gx.K = c.V, gx.dyn = 1;
        gx.plan = p.slots_dx ? plan + 2 * i : nullptr;
        gx.part = reinterpret_cast<float*>(ws + p.part_dx);
        gw.B = xc, gw.ldb = c.d;
        gw.M = c.V, gw.N = c.d, gw.K = bound * p.terms, gw.dyn = 2, gw.terms = p.terms;
        gw.plan = p.slots_dw ? plan + 2 * i + 1 : nullptr;
        gw.part = reinterpret_cast<float*>(ws + p.part_dw);
        const EpiRows<T> ex = {static_cast<T*>(c.dx), c.d, rows, p0, top, static_cast<const T*>(c.Wv)};
        float* acc = p.pieces > 1 ? reinterpret_cast<float*>(ws + p.acc) : nullptr;
        const EpiSum<T> ew = {static_cast<T*>(c.dWv), acc, c.d, count, p0, p.piece};
        const int nx = c.dx ? head_grid<BM>(gx, bound) : 0;
        const int nw = c.dWv ? head_grid<BM>(gw, c.V) : 0;
        MOE_LAUNCH("head_grads", s, head_grads_kernel<<<nx + nw, 256, 0, s>>>(gx, ex, gw, ew, nx));
        const int jx = c.dx ? head_join_grid<BM>(gx, bound) : 0;
        const int jw = c.dWv ? head_join_grid<BM>(gw, c.V) : 0;
        if (jx + jw)
            MOE_LAUNCH("head_join", s,
                       head_join_kernel<BM, T><<<jx + jw, 1024, 0, s>>>(gx, ex, gw, ew, jx));
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
        MOE_LAUNCH("head_zero", s, head_zero_kernel<<<head_blocks(n), 256, 0, s>>>(
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
