// Building blocks of the bf16 matrix kernels (gfx950): operand tiles loaded
// from HBM straight into a ring of LDS stages, the fragments of
// v_mfma_f32_32x32x16_bf16 read from them, the barrier between stages, and the
// block -> tile order that gives each XCD runs of neighbouring tiles.
#pragma once

#include "common.h"

namespace moe {

// Workgroups are dealt to the 8 XCDs round-robin (block b runs on XCD b % 8);
// block -> logical tile such that each XCD receives runs of `run` consecutive
// logical tiles.  Grids are padded to a multiple of NXCD * run.
constexpr int NXCD = 8;

__device__ __forceinline__ int xcd_logical(int b, int run) {
    const int x = b % NXCD, j = b / NXCD;
    return ((j / run) * NXCD + x) * run + (j % run);
}

// Operand tiles go from HBM straight into LDS with buffer_load_dwordx4 ...
// lds (each wave instruction fills 1 KB: lane l's 16 bytes land at base +
// 16*l), through a ring of NSTG stages of BK reduction steps, with no
// register staging.  The descriptor's byte range covers exactly the valid
// part of the tile, so lanes past a ragged segment end, the end of the
// reduction, a partial tile or the allocation read zeros, with no branch.
constexpr uint32_t OOB = 0x80000000u;    // an offset past any descriptor range
// Rows of the reduction-row gather map held in LDS at a time (RAGGED_K); a
// power of two.
constexpr int KG_CHUNK = 4096;
enum { KMAJ = 0, MNMAJ = 1 };   // operand storage: row-of-K contiguous or M/N contiguous

typedef short v4i16_t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16_t lds_v4i16_t;


// K-major stage tile: rows of BK bf16 (CH = BK/8 chunks of 16 B), chunk c of
// row r stored at chunk c ^ ((r ^ r/CH) mod CH), so that the rows one
// fragment read touches spread over distinct banks.
template <int CH>
__device__ __forceinline__ int swzk(int r, int c) {
    constexpr int L = CH == 4 ? 2 : 3;
    static_assert(CH == 4 || CH == 8, "32 or 64 reduction steps per stage");
    return r * (CH * 16) + ((c ^ ((r ^ (r >> L)) & (CH - 1))) << 4);
}
// M/N-major stage tile: BK rows of ROWS elements; chunk c of row k is
// stored at chunk c ^ 4*(k mod 4), which spreads the four rows a transposing
// read touches over distinct banks.
template <int ROWS>
__device__ __forceinline__ int mnoff(int k, int c) {
    return k * ROWS * 2 + ((c ^ ((k & 3) << 2)) << 4);
}

typedef __attribute__((address_space(3))) void lds_void_t;
typedef int i32x4_t __attribute__((ext_vector_type(4)));

// The four words of a raw buffer resource: base address, stride 0,
// num_records = nbytes (clamped at 0), and word 3 = 0x00020000 (data format
// 32 bits, no swizzle), the usual raw-access setting on gfx9 parts.  Reads at
// offsets >= nbytes return zero.
__device__ __forceinline__ i32x4_t rsrc_words(const bf16_t* base, long nbytes) {
    const uint64_t a = (uint64_t)base;
    const uint32_t n = nbytes <= 0 ? 0u : (uint32_t)nbytes;
    // the words are wave-uniform; readfirstlane states it where the
    // compiler cannot see it (operand fields set on two paths)
    return i32x4_t{__builtin_amdgcn_readfirstlane((int)(uint32_t)a),
                   __builtin_amdgcn_readfirstlane((int)((uint32_t)(a >> 32) & 0xFFFFu)),
                   __builtin_amdgcn_readfirstlane((int)n), 0x00020000};
}
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
    return (uint32_t)(uintptr_t)(const lds_void_t*)p;
}
// One wave-wide 16-byte-per-lane load from a buffer straight into LDS: lane
// l's bytes at voff land at lds + 16*l.  Issued from inline assembly so that
// the compiler does not tie every later LDS read to its completion; callers
// wait on vmcnt themselves (stage_barrier) before reading the stage.
// The compiler counts no wait states into inline assembly: one between writing
// m0 and the load that reads it, and five between a vector instruction that
// writes a scalar register (v_readfirstlane, in rsrc_words) and a load that reads
// it, which the first load behind a descriptor (FIRST) waits for itself.
template <bool FIRST>
__device__ __forceinline__ void lds_dma16(i32x4_t rs, uint32_t voff, uint32_t lds) {
    asm volatile(
        "s_mov_b32 m0, %0\n\t"
        "s_nop %3\n\t"
        "buffer_load_dwordx4 %1, %2, 0 offen lds"
        :
        : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rs), "n"(FIRST ? 3 : 0)
        : "memory", "m0");
}
__device__ __forceinline__ void lds_dma16(bool first, i32x4_t rs, uint32_t voff, uint32_t lds) {
    if (first) lds_dma16<true>(rs, voff, lds);      // (a constant in an unrolled loop)
    else lds_dma16<false>(rs, voff, lds);
}

template <int ROWS, int LAY, int NT, int BK>
struct DmaOperand {
    static constexpr int NW = NT / 64;
    static constexpr int CH = BK / 8;                     // K-major: chunks per row
    static constexpr int TILE = ROWS * BK * 2;            // bytes per stage
    static constexpr int NLOAD = TILE / 1024 / NW;        // 1 KB loads per wave
    static_assert(TILE % (1024 * NW) == 0, "tile/wave mismatch");
    static_assert(LAY == KMAJ || ROWS >= 128, "M/N-major swizzle needs 16 chunks per row");
    static_assert(TILE >= 1024 * NW, "every wave loads at least 1 KB per stage");
    const bf16_t* P;
    long ld;
    int row_lim;
    long k_lim;
    long span;               // K-major: bytes from P that hold valid rows
    uint32_t off[NLOAD];

    __device__ __forceinline__ void init(const bf16_t* P_, long ld_, int row_lim_,
                                         long k_lim_) {
        P = P_;
        ld = ld_;
        row_lim = row_lim_;
        k_lim = k_lim_;
        span = (long)row_lim_ * ld_ * 2;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) {
            const int blk = w + NW * i;                    // 1 KB block of the stage
            if (LAY == KMAJ) {
                constexpr int L = CH == 4 ? 2 : 3;
                const int row = blk * (64 / CH) + lane / CH;
                const int c = (lane % CH) ^ ((row ^ (row >> L)) & (CH - 1));
                off[i] = (uint32_t)(row * ld * 2 + c * 16);
            } else {
                constexpr int NC = ROWS / 8;               // chunks per row
                constexpr int RB = 1024 / (ROWS * 2);      // rows per block
                const int k = blk * RB + lane / NC;
                const int c = (lane % NC) ^ ((k & 3) << 2);
                off[i] = c * 8 < row_lim ? (uint32_t)(k * ld * 2 + c * 16) : OOB;
            }
        }
    }

    // K-major operand whose tile row r (< row_lim) is source row map[r] of a
    // source of src_rows rows at P; the byte range then covers the whole
    // source (under 2^31 bytes, checked on the host) and rows past row_lim
    // get an offset past it.
    __device__ __forceinline__ void init_gather(const bf16_t* P_, long ld_, int row_lim_,
                                                const int32_t* map, long src_rows) {
        static_assert(LAY == KMAJ, "row gather of a K-major operand");
        P = P_;
        ld = ld_;
        row_lim = row_lim_;
        k_lim = 0;
        span = src_rows * ld_ * 2;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        constexpr int L = CH == 4 ? 2 : 3;
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) {
            const int row = (w + NW * i) * (64 / CH) + lane / CH;
            const int c = (lane % CH) ^ ((row ^ (row >> L)) & (CH - 1));
            off[i] = row < row_lim ? (uint32_t)((long)map[row] * ld * 2 + c * 16) : OOB;
        }
    }

    // M/N-major operand whose reduction row k (< k_lim) is a gathered row of
    // a source with src_rows rows; P points at the tile's first column (of
    // row_lim valid ones).  off[] holds each load's chunk offset in a row.
    __device__ __forceinline__ void init_kgather(const bf16_t* P_, long ld_, int row_lim_,
                                                 long k_lim_, long src_rows, int m0) {
        static_assert(LAY != KMAJ, "reduction-row gather of an M/N-major operand");
        P = P_;
        ld = ld_;
        row_lim = row_lim_;
        k_lim = k_lim_;
        span = src_rows * ld_ * 2 - (long)m0 * 2;
        constexpr int NC = ROWS / 8;
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) {
            const int k = (w + NW * i) * (1024 / (ROWS * 2)) + lane / NC;
            const int c = (lane % NC) ^ ((k & 3) << 2);
            off[i] = c * 8 < row_lim ? (uint32_t)(c * 16) : OOB;
        }
    }
    // Source rows of the loads of the stage of reduction rows k0 .. k0+BK-1:
    // row k is source row lmap[k - kmap] (lmap in LDS; k - kmap lies inside
    // the map chunk for a stage of it, so the read is unconditional and the
    // value is only looked at when the stage is issued: the LDS wait of
    // this read-ahead stays off the issue path).
    __device__ __forceinline__ void rows_of(long k0, const int32_t* lmap, long kmap,
                                            int32_t* rows) const {
        constexpr int NC = ROWS / 8;
        constexpr int RB = 1024 / (ROWS * 2);
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
        for (int i = 0; i < NLOAD; ++i)
            rows[i] = lmap[(k0 + (w + NW * i) * RB + lane / NC - kmap) & (KG_CHUNK - 1)];
    }
    // Issue the stage at k0, given rows_of's result; loads past the segment
    // or the tile's columns get an offset past the source.
    __device__ __forceinline__ void dma_rows(long k0, uint8_t* stage, const int32_t* rows) const {
        constexpr int NC = ROWS / 8;
        constexpr int RB = 1024 / (ROWS * 2);
        const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
        const i32x4_t rs = rsrc_words(P, span);
        const uint32_t lds0 = lds_addr(stage) + (uint32_t)(w * 1024);
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) {
            // branch-free: a source row offset is below 2^31 (host check),
            // so setting bit 31 (a column past the tile: off[i] = OOB, or a
            // row past the segment) sends the load past the descriptor range
            const long k = k0 + (w + NW * i) * RB + lane / NC;
            const uint32_t o = ((uint32_t)rows[i] * (uint32_t)(ld * 2) + off[i]) |
                               ((uint32_t)(k >= k_lim) << 31);
            lds_dma16(i == 0, rs, o, lds0 + NW * i * 1024);
        }
    }

    __device__ __forceinline__ void dma(long k0, uint8_t* stage) const {
        const bf16_t* base;
        long nbytes;
        if (LAY == KMAJ) {
            base = P + k0;
            nbytes = span - k0 * 2;
        } else {
            base = P + k0 * ld;
            nbytes = min((long)BK, k_lim - k0) * ld * 2;
        }
        const i32x4_t rs = rsrc_words(base, nbytes);
        const uint32_t lds0 = lds_addr(stage) + (uint32_t)((threadIdx.x >> 6) * 1024);
#pragma unroll
        for (int i = 0; i < NLOAD; ++i) lds_dma16(i == 0, rs, off[i], lds0 + NW * i * 1024);
    }
};

template <int ROWS, int LAY, int BK>
__device__ __forceinline__ bf16x8 dma_frag(const uint8_t* lds, int row0, int ks, int lane) {
    if constexpr (LAY == KMAJ) {
        const uint4 v = *reinterpret_cast<const uint4*>(
            lds + swzk<BK / 8>(row0 + (lane & 31), ks * 2 + (lane >> 5)));
        return __builtin_bit_cast(bf16x8, v);
    } else {
        const int k = ks * 16 + (lane >> 5) * 8 + ((lane & 15) >> 2);
        const int col = row0 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
        const uint8_t* p0 = lds + mnoff<ROWS>(k, col >> 3) + (col & 7) * 2;
        const uint8_t* p1 = lds + mnoff<ROWS>(k + 4, col >> 3) + (col & 7) * 2;
        const v4i16_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)p0);
        const v4i16_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16_t*)p1);
        typedef short v8i16_t __attribute__((ext_vector_type(8)));
        const v8i16_t v = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        return __builtin_bit_cast(bf16x8, v);
    }
}

// Order a wave's LDS writes before its later LDS reads (and reads before
// later writes) of data other lanes of the same wave touch: one wave's LDS
// instructions execute in order, so only the compiler must not move them.
__device__ __forceinline__ void wave_lds_sync() {
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
}

// Wait until at most N direct-to-LDS loads of this wave are in flight and
// its LDS reads have returned, then meet the other waves of the block.  The
// compiler does not read the wait inside the asm; the lgkmcnt(0) after it
// (which then costs nothing) tells it that no LDS read is outstanding, so
// its own waits for the next fragments count only the reads issued after
// the barrier instead of draining them all (dW products 2-3% faster).
template <int N>
__device__ __forceinline__ void stage_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
    __builtin_amdgcn_s_waitcnt(0xc07f);                // lgkmcnt(0), no vmcnt wait
}
// stage_barrier with `ahead` (0..MAXA, wave-uniform) later stages of NL loads
// each allowed to stay in flight
template <int NL, int MAXA>
__device__ __forceinline__ void stage_barrier_ahead(int ahead) {
    if constexpr (MAXA <= 0) {
        stage_barrier<0>();
    } else {
        if (ahead >= MAXA) stage_barrier<NL * MAXA>();
        else stage_barrier_ahead<NL, MAXA - 1>(ahead);
    }
}

}  // namespace moe
