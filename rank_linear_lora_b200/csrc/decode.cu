// decode.cu -- the gated and the epilogue projections of a few tokens (generating text):
//
//   acc[n, m] = sum_k W[n, k] x[m, k] + sum_j B[n, j] (s.xa)[m, j],   then the epilogue
//
// Bound by reading W once.  A 256 x 256 tensor-core tile per CTA pair would put only
// d_out / 256 pairs of SMs on that stream, so here one persistent CTA an SM takes groups of 16 or
// 32 weight rows (16 of the gate and 16 of the up projection, when gated), every CTA the same
// number:
//
//   product warps    a group's rows are cut along K into stages of two 2 KB boxes (128 bytes of
//                    16 rows: both of a group's, or two in a row); the warps take the CTA's
//                    stages in turn.  Each streams its own by TMA into a private ring
//                    in shared memory, several ahead and on into the next groups, and at a
//                    group's end leaves its sums in one of two buffers.
//   finishing warps  finish a group while the others go on: the warps' sums in a fixed order,
//                    the low-rank term (products on B's rows and s.xa), the epilogue.
//
// The products run on mma.sync m16n8k16: weight rows are its 16-row side, tokens its 8-column
// side (M <= 8 NT).  tcgen05 would want its weight operand decoded back into shared memory;
// here a tile goes from shared memory into fragment registers once, and at a few tokens the
// tensor pipe has nothing to do either way.  Both operands may order k in any one way, so a
// lane's fragment registers are 8 or 16 consecutive weights of one row, and x is laid out to
// match, in shared memory.  TMA's 128-byte swizzle and the order in which fragment rows take
// tile rows keep those reads free of bank conflicts.
//
// Where x does not fit into shared memory whole, batches of 2 or 4 groups share its segments: the
// product warps go through all groups of a batch with one segment before the next one, their
// sums of each group waiting in shared memory, while a finishing warp brings the segment after
// it (28672 -> 8192 in bf16: 74 us for 8 tokens, the weight's 470 MB at 6.4 TB/s, 89 us for 16;
// with x's fragments read from L2 stage by stage it was 151 and 170).
//
// Codes are widened in registers, and no decoded weight is rounded.  A 4-bit code under the
// exponent of 128 is 128 + q, and stands for q - 8: the products take 128 + q and start from -136
// times the block's sum of x (8192 -> 2 x 28672, four tokens: 64.3 us, with an addition
// afterwards 65.5; 621 instructions a stage, 0.56 issued a cycle and scheduler).  A 4-bit sum that
// is not finite is formed again from the codes by the finishing warps: an infinite x (or a finite
// one that 128 + q takes past fp32) keeps the sign of its product, where 128 + q and the offset give
// inf - inf.  E4M3 codes enter with their exact values.  The scale (one a row, or one a row and
// 64 k, fetched a tile ahead) multiplies the fp32 sums.  Codebook values are rounded once to bf16
// and looked up two codes at a time in a table of a byte's 256 pairs, a copy in every bank.
//
// s.xa comes from k_decode_xa just before; this kernel starts its stream beside it and waits
// for it only before the low-rank term (programmatic dependent launch: that kernel lets this
// one start only once all its own CTAs have seen their predecessor complete, so x is final).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "act.cuh"
#include "decode.h"
#include "ptx.cuh"
#include "tc_gemm.cuh"
#include "tmap.h"

namespace {

using namespace lora;
using lora_host::DecodeArgs;

constexpr int ROWS = 16;        // weight rows per m-tile
constexpr int TILE_BYTES = 128;  // of a row per tile
constexpr int BOX = ROWS * TILE_BYTES;
constexpr int TILE = 128;       // values of an m-tile x n-tile
constexpr int FIN_WARPS = 4;     // finishing warps: a thread for each value of an n-tile
enum DecodeOp { D_ACT = 1, D_GLU = 2 };
enum DecodeFmt { F_BF16 = LORA_W_BF16, F_Q4 = LORA_W_Q4, F_FP8 = LORA_W_FP8, F_CB = LORA_W_NF4 };

template <int FMT, int OP, int NT, bool SEG, int MT>
struct Cfg {
    static constexpr bool NIBBLE = FMT == F_Q4 || FMT == F_CB;
    static constexpr int GROUP_ROWS = OP == D_GLU ? ROWS : MT * ROWS;  // of each projection
    // Widening 4-bit codes is bound by instructions, not by memory: more warps, and the ring they
    // leave room for (8192 -> 2 x 28672, four tokens: 64 us; 8 warps x 4 stages 78, 16 x 2, which
    // spill, 94).  The other formats stream at 8 x 4 (4096 -> 2 x 11008 in bf16, one token: 30 us).
    // With x in segments a 4-bit stage is one box, so that a short segment still has stages for all
    // warps, and 12 warps pay only where their sums leave the segments room (28672 -> 8192 in groups
    // of 16 rows, 8 tokens: 12 x 2 56 us, 8 x 4 66; 16 tokens: 12 x 2 stages of two boxes 113, 97).
    static constexpr int WARPS = NIBBLE && (!SEG || MT * NT == 1) ? 12 : 8;
    static constexpr int BOXES = MT == 2 || !(NIBBLE && SEG) ? 2 : 1;  // of a stage
    static constexpr int STAGE = BOXES * BOX;
    static constexpr int STAGES = NIBBLE && (WARPS == 12 || BOXES == 2) ? 2 : 4;
    static constexpr int THREADS = (WARPS + FIN_WARPS) * 32;
    static constexpr int BOX_K = FMT == F_BF16 ? 64 : FMT == F_FP8 ? 128 : 256;  // k of a box
    static constexpr int STAGE_K = MT == 2 ? BOX_K : BOXES * BOX_K;
    static constexpr int BLOCKS = STAGE_K / 64;                // 64-wide blocks of k
    static constexpr int BOX_BLOCKS = BOX_K / 64;
    static constexpr int RING = WARPS * STAGES * STAGE;
    static constexpr int OUT = MT * NT * TILE;                 // fp32 sums of a group
    // Groups of a batch, which share each segment of x: their sums take room from the segments.
    static constexpr int GROUPS = !SEG ? 1 : MT * NT == 4 && !NIBBLE ? 2 : 4;
    static constexpr int SLOTS = SEG ? GROUPS : 2;             // groups' sums kept
    static constexpr int RED = SLOTS * WARPS * OUT * 4;
    static constexpr int TABLE = FMT == F_CB ? 256 * 32 * 4 : 0;
    static constexpr int BARS = (WARPS * STAGES + 2 * SLOTS + 4) * 8;
    static constexpr int FIXED = 1024 + RING + RED + OUT * 4 + TABLE + BARS + 16 + 128;
    static constexpr int X_PAD = SEG && FMT != F_BF16 ? 16 : 64;  // behind a token of x: reads of tokens side by side share no bank
    static constexpr int X_MAX = (232448 - FIXED) / 64 * 64;   // room for x
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from C = 0.
__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
// From C = (lo, hi) in both rows.
__device__ __forceinline__ void mma_bf16_from(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1, float lo, float hi) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%10,%11};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(lo), "f"(hi));
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}
// Shared-memory loads by 32-bit address, in program order with the waits and the copies.
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }

// Tile row (0..7) of fragment row g: 8 lanes (16-byte reads) or 16 (8-byte reads) that are
// served together then read all 32 banks of the swizzled rows.
template <bool NIBBLE>
__device__ __forceinline__ int tile_row(int g) {
    return NIBBLE ? ((g & 3) << 1) | (g >> 2) : (g >> 1) | ((g & 1) << 2);
}

// Four E4M3 codes to two pairs of bf16, exactly.
__device__ __forceinline__ void widen_fp8(uint32_t q, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 c0, c1, a0, a1, a2, a3;\n\t.reg .b32 h0, h1;\n\t.reg .f32 f0, f1, f2, f3;\n\t"
        "mov.b32 {c0, c1}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 h0, c0;\n\t"
        "cvt.rn.f16x2.e4m3x2 h1, c1;\n\t"
        "mov.b32 {a0, a1}, h0;\n\t"
        "mov.b32 {a2, a3}, h1;\n\t"
        "cvt.f32.f16 f0, a0;\n\tcvt.f32.f16 f1, a1;\n\tcvt.f32.f16 f2, a2;\n\tcvt.f32.f16 f3, a3;\n\t"
        "cvt.rn.bf16x2.f32 %0, f1, f0;\n\t"
        "cvt.rn.bf16x2.f32 %1, f3, f2;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(q));
}
// 128 + q of the codes (e, e + 4) of a word's 8 is and_or(word >> 4 e, 0x000F000F, 0x43004300), a
// pair of bf16.  The masks come in registers: one LOP3 then ands and ors (immediates take two).
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits) {
    uint32_t d;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(v), "r"(mask), "r"(bits));
    return d;
}
// The table's pair of a byte of codes.
__device__ __forceinline__ uint32_t cb_pair(uint32_t table_lane, uint32_t v, int byte) {
    uint32_t w;
    asm("ld.shared.u32 %0, [%1];" : "=r"(w) : "r"(table_lane + ((v >> (8 * byte)) & 0xFFu) * 128u));
    return w;
}

// sum_k (q - 8) scale / 7 x of one row and token, from memory: for the few sums that products with
// 128 + q cannot give.
__device__ __forceinline__ float q4_sum(const DecodeArgs &a, int64_t row, int token) {
    const uint8_t *codes = a.w + row * (a.K / 2);
    const uint16_t *scales = a.wscale + row * (a.K / 64), *x = a.x + static_cast<int64_t>(token) * a.K;
    float v = 0.0f;
#pragma unroll 1
    for (int k0 = 0; k0 < a.K && v == v; k0 += 64) {  // a NaN stays one: the usual case ends early
        float sum = 0.0f;
#pragma unroll 4
        for (int k = k0; k < k0 + 64; k += 8) {
            const uint32_t q = __ldg(reinterpret_cast<const uint32_t *>(codes + k / 2));
            const uint4 u = __ldcg(reinterpret_cast<const uint4 *>(x + k));
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int e = 0; e < 8; ++e)
                sum = fmaf(static_cast<float>(static_cast<int>((q >> (4 * e)) & 15u) - 8),
                           __uint_as_float(e & 1 ? w[e / 2] & 0xFFFF0000u : w[e / 2] << 16), sum);
        }
        v = fmaf(bf16_f32(__ldg(scales + k0 / 64)), sum, v);
    }
    return v * (1.0f / 7.0f);
}

// Barrier of the finishing warps; true where any of their threads brings true.
__device__ __forceinline__ bool fin_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.or.pred q, 1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(r) : "r"(static_cast<uint32_t>(v)), "n"(FIN_WARPS * 32) : "memory");
    return r != 0;
}

// SEG: x does not fit into shared memory whole.
template <int FMT, int OP, int NT, bool SEG, int MT>
__global__ void __launch_bounds__(Cfg<FMT, OP, NT, SEG, MT>::THREADS, 1) k_decode(const __grid_constant__ DecodeArgs a) {
    using C_ = Cfg<FMT, OP, NT, SEG, MT>;
    constexpr int SLOTS = C_::SLOTS, GROUPS = C_::GROUPS;
    constexpr int GROUP_ROWS = C_::GROUP_ROWS, WARPS = C_::WARPS, STAGES = C_::STAGES, STAGE = C_::STAGE, OUT = C_::OUT, BLOCKS = C_::BLOCKS;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *red = reinterpret_cast<float *>(smem + C_::RING);  // [SLOTS][WARPS][OUT]
    float *tail = red + SLOTS * WARPS * OUT;                  // [OUT] the low-rank term
    uint32_t *table = reinterpret_cast<uint32_t *>(tail + OUT);
    uint64_t *bars = reinterpret_cast<uint64_t *>(reinterpret_cast<uint8_t *>(table) + C_::TABLE);  // [WARPS][STAGES]
    uint64_t *red_full = bars + WARPS * STAGES, *red_empty = red_full + SLOTS;
    uint64_t *x_full = red_empty + SLOTS, *x_empty = x_full + 2;      // SEG: of the two segments
    volatile int *abort_flag = reinterpret_cast<volatile int *>(x_empty + 2);
    uint8_t *zero = reinterpret_cast<uint8_t *>(x_empty + 2) + 16;    // 128 bytes: a block of a token behind M
    uint8_t *xs = zero + 128;                                         // x, rows x_stride bytes (SEG: two segments)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, j = lane & 3;
    const int S = (a.K + C_::STAGE_K - 1) / C_::STAGE_K;      // stages of a group
    const int groups = (a.N + GROUP_ROWS - 1) / GROUP_ROWS;
    // row of m-tile m of a group in W, and in what has a value a row of it; rows behind N read the last
    auto w_row = [&](int u, int m, int row) {
        return OP == D_GLU ? min(u * ROWS + row, a.N - 1) + m * a.N : min(u * GROUP_ROWS + m * ROWS + row, a.N - 1);
    };
    const int u0 = blockIdx.x, u_step = gridDim.x;
    const int mine = (groups - u0 + u_step - 1) / u_step;     // groups of this CTA: u0 + i u_step
    const int SS = SEG ? a.seg_stages : S, n_seg = SEG ? (S + SS - 1) / SS : 1;
    auto seg_len = [&](int seg) { return SEG ? min(SS, S - seg * SS) : S; };
    const int row_in = tile_row<C_::NIBBLE>(g);  // tile rows of the lane: row_in, row_in + 8

    if (warp < WARPS && lane == 0)
        for (int s = 0; s < STAGES; ++s) mbar_init(smem_u32(&bars[warp * STAGES + s]), 1);
    if (threadIdx.x == WARPS * 32) {
        for (int b = 0; b < SLOTS; ++b) {
            mbar_init(smem_u32(&red_full[b]), WARPS);
            mbar_init(smem_u32(&red_empty[b]), FIN_WARPS);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(smem_u32(&x_full[b]), 1);
            mbar_init(smem_u32(&x_empty[b]), WARPS);
        }
        *abort_flag = 0;
    }
    fence_mbar_init();
    __syncwarp();
    grid_dep_launch_dependents();

    // x: 64-wide blocks laid out as the fragments take them, zero behind K.  Its loads go out
    // before the stream's, which would hold them up by the whole ring.
    const int x_stride = SS * C_::STAGE_K * 2 + C_::X_PAD, x_buf = a.M * x_stride;
    const int x_cols8 = S * (C_::STAGE_K / 8), x_chunks = SEG ? 0 : a.M * x_cols8;
    constexpr int X_AHEAD = 8;
    uint4 xv[X_AHEAD];
    auto x_load = [&](int c) {
        const int m = c / x_cols8, k = (c - m * x_cols8) * 8;
        return k < a.K ? __ldcg(reinterpret_cast<const uint4 *>(a.x + static_cast<int64_t>(m) * a.K + k)) : make_uint4(0, 0, 0, 0);
    };
    auto x_store = [&](int c, uint4 v) {
        const int m = c / x_cols8, k = (c - m * x_cols8) * 8;
        int at = k;
        if (FMT != F_BF16) at = (k & ~63) + ((k >> 3) & 1) * 32 + ((k >> 4) & 3) * 8;  // 16 in a row per lane
        if (FMT == F_Q4)
            v = make_uint4(prmt(v.x, v.z, 0x5410), prmt(v.x, v.z, 0x7632), prmt(v.y, v.w, 0x5410), prmt(v.y, v.w, 0x7632));
        *reinterpret_cast<uint4 *>(xs + m * x_stride + at * 2) = v;
    };
    // SEG: segment `seg` of x to buffer `buf` by bulk copies, as it is, zero behind K; one warp
    auto x_fill = [&](int seg, int buf) {
        const int k0 = seg * SS * C_::STAGE_K, width = seg_len(seg) * C_::STAGE_K, cols = min(width, a.K - k0);
        uint8_t *dst = xs + buf * x_buf;
        const int behind = (width - cols) / 8;
        for (int c = lane; c < a.M * behind; c += 32)
            *reinterpret_cast<uint4 *>(dst + c / behind * x_stride + cols * 2 + c % behind * 16) = make_uint4(0, 0, 0, 0);
        __syncwarp();
        const uint32_t bar = smem_u32(&x_full[buf]);
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(a.M * cols * 2));
        __syncwarp();
        if (lane < a.M) bulk_load(smem_u32(dst + lane * x_stride), a.x + static_cast<int64_t>(lane) * a.K + k0, cols * 2, bar);
        __syncwarp();
    };
    if constexpr (SEG) {
        if (warp == WARPS) x_fill(0, 0);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < X_AHEAD; ++i)
        if (static_cast<int>(threadIdx.x) + i * C_::THREADS < x_chunks) xv[i] = x_load(threadIdx.x + i * C_::THREADS);

    // A product warp's stages are the CTA's warp, warp + WARPS, ..., of all batches, their segments, the
    // segments' groups and the groups' stages, in that order.
    struct Cursor {
        int u, st;         // group, stage of the segment
        int base, seg, i;  // SEG: the batch's first group (of `mine`), segment, group of the batch
    };
    auto settle = [&](Cursor &c) {
        while (c.st >= seg_len(c.seg) && (!SEG || c.base < mine)) {
            c.st -= seg_len(c.seg);
            c.u += u_step;
            if constexpr (SEG) {
                const int n = min(GROUPS, mine - c.base);
                if (++c.i < n) continue;
                c.i = 0;
                if (++c.seg < n_seg) {
                    c.u -= n * u_step;
                    continue;
                }
                c.seg = 0;
                c.base += GROUPS;
            }
        }
    };
    auto more = [&](const Cursor &c) { return SEG ? c.base < mine : c.u < groups; };
    // Its requests run STAGES ahead of the stage in use.
    uint8_t *ring = smem + warp * (STAGES * STAGE);  // (product warps only)
    Cursor rq{u0, warp, 0, 0, 0};
    int requested = 0;
    auto advance = [&]() {
        if (!more(rq)) return;
        if (lane == 0) {
            const int s = requested & (STAGES - 1);
            const uint32_t bar = smem_u32(&bars[warp * STAGES + s]), dst = smem_u32(ring + s * STAGE);
            mbar_arrive_expect_tx(bar, static_cast<uint32_t>(STAGE));
            const int byte = (rq.seg * SS + rq.st) * (MT == 2 ? 1 : C_::BOXES) * TILE_BYTES, row = rq.u * GROUP_ROWS;
            tma_load_2d(dst, &a.tmW, bar, byte, row);
            if (C_::BOXES == 2) tma_load_2d(dst + BOX, &a.tmW, bar, MT == 2 ? byte : byte + TILE_BYTES, OP == D_GLU ? a.N + row : MT == 2 ? row + ROWS : row);
        }
        ++requested;
        rq.st += WARPS;
        settle(rq);
    };
    static_assert((STAGES & (STAGES - 1)) == 0, "stages are counted by masks");
    if (warp < WARPS) {
        settle(rq);
        for (int s = 0; s < STAGES; ++s) advance();
    }

#pragma unroll
    for (int i = 0; i < X_AHEAD; ++i)
        if (static_cast<int>(threadIdx.x) + i * C_::THREADS < x_chunks) x_store(threadIdx.x + i * C_::THREADS, xv[i]);
    for (int c = threadIdx.x + X_AHEAD * C_::THREADS; c < x_chunks; c += C_::THREADS) x_store(c, x_load(c));
    if (threadIdx.x < 32) reinterpret_cast<uint32_t *>(zero)[threadIdx.x] = 0;
    // 4-bit codes: -136 times each block's sum of x, [block][token] (zero behind M), behind x
    float *xsum = reinterpret_cast<float *>(xs + x_buf);
    if constexpr (!SEG && FMT == F_Q4) {
        __syncthreads();
        const int nb = S * BLOCKS;
        for (int c = threadIdx.x; c < nb * 8 * NT; c += C_::THREADS) {
            const int b = c / (8 * NT), m = c % (8 * NT);
            float v = 0.0f;
            if (m < a.M) {
                const uint4 *p = reinterpret_cast<const uint4 *>(xs + m * x_stride + b * 128);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint4 q = p[i];
                    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) v += __uint_as_float(w[e] << 16) + __uint_as_float(w[e] & 0xFFFF0000u);
                }
            }
            xsum[c] = -136.0f * v;
        }
    }
    if constexpr (FMT == F_CB) {
        for (int i = threadIdx.x; i < 256 * 32; i += C_::THREADS) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(a.cb[(i >> 5) & 15], a.cb[i >> 9]);
            table[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    __syncthreads();

    if (warp < WARPS) {
        // ------------------------------------------------------------------ products
        const uint32_t table_lane = smem_u32(table) + lane * 4;
        const uint32_t ring0 = smem_u32(ring) + row_in * TILE_BYTES;
        uint32_t q4_mask = 0x000F000Fu, q4_bits = 0x43004300u;  // kept in registers
        asm volatile("" : "+r"(q4_mask), "+r"(q4_bits));
        uint32_t chunk[4];  // byte of the lane's weights of block b of a box in its (swizzled) row
#pragma unroll
        for (int b = 0; b < 4; ++b)
            chunk[b] = C_::NIBBLE ? (((2 * b + (j >> 1)) ^ row_in) << 4) + (j & 1) * 8 : ((4 * (b & 1) + j) ^ row_in) << 4;
        // the fragments of a 64-wide block of x, token n*8 + g; tokens behind M read zeros
        const uint32_t xsum0 = smem_u32(xsum) + j * 8;
        uint32_t xp[NT], x_step[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const bool in = n * 8 + g < a.M;
            xp[n] = smem_u32(in ? xs + (n * 8 + g) * x_stride : zero) + j * (SEG && FMT != F_BF16 ? 32 : 16);
            x_step[n] = in ? 128u : 0u;
        }
        uint32_t x_at = 0;  // byte of the segment's buffer
        auto load_x = [&](int n, int block, uint32_t (&v)[8]) {
            const uint32_t p = xp[n] + block * x_step[n] + (SEG && x_step[n] ? x_at : 0);
            uint4 u = lds16(p), w = lds16(p + (SEG && FMT != F_BF16 ? 16 : 64));
            if (SEG && FMT == F_Q4) {
                u = make_uint4(prmt(u.x, u.z, 0x5410), prmt(u.x, u.z, 0x7632), prmt(u.y, u.w, 0x5410), prmt(u.y, u.w, 0x7632));
                w = make_uint4(prmt(w.x, w.z, 0x5410), prmt(w.x, w.z, 0x7632), prmt(w.y, w.w, 0x5410), prmt(w.y, w.w, 0x7632));
            }
            v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w, v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
        };
        // 4-bit scales of a stage, as loaded: 4 blocks of k of each of the lane's rows of a box.  The
        // rows' pointers are the group's.
        const int n_kb = a.K / 64;
        const uint16_t *sc_row[MT][2];
        auto scale_rows = [&](int u) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    sc_row[m][h] = a.wscale + static_cast<int64_t>(w_row(u, m, row_in + 8 * h)) * n_kb;
        };
        const bool sc_aligned = n_kb % 4 == 0;  // four scales are 8 aligned bytes
        auto load_scales = [&](int s, uint2 (&sc)[2][2]) {
#pragma unroll
            for (int x = 0; x < C_::BOXES; ++x) {
                const int kb = MT == 2 ? s * 4 : (s * C_::BOXES + x) * 4;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint16_t *p = sc_row[MT == 2 ? x : 0][h] + kb;
                    if (sc_aligned) {
                        sc[x][h] = kb < n_kb ? __ldg(reinterpret_cast<const uint2 *>(p)) : make_uint2(0, 0);
                    } else {
                        uint32_t q[4];
#pragma unroll
                        for (int b = 0; b < 4; ++b) q[b] = kb + b < n_kb ? __ldg(p + b) : 0;
                        sc[x][h] = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
                    }
                }
            }
        };
        bool ok = true;
        int used = 0, fill = 0;
        Cursor at{u0, warp, 0, 0, 0};  // the warp's next stage
        settle(at);
        uint2 sc[2][2], sc_next[2][2];
        int sc_u = at.u;  // the group of sc_row
        if constexpr (C_::NIBBLE)
            if (more(at)) {
                scale_rows(sc_u);
                load_scales(at.seg * SS + at.st, sc_next);
            }
        for (int base = 0; ok && (SEG ? base < mine : u0 + base * u_step < groups); base += GROUPS)
        for (int seg = 0; ok && seg < n_seg; ++seg, ++fill) {
        if constexpr (SEG) {
            ok = wait_bounded(smem_u32(&x_full[fill & 1]), static_cast<uint32_t>(fill >> 1) & 1u, abort_flag, a.err,
                              DERR_WAIT_FULL);
            ok = __all_sync(0xffffffffu, ok);
            x_at = static_cast<uint32_t>((fill & 1) * x_buf);
        }
        for (int i = 0; ok && i < (SEG ? min(GROUPS, mine - base) : 1); ++i) {
            const int gu = u0 + (base + i) * u_step;
            const int sums = SEG ? i : base & 1;  // slot of the group's sums
            float acc[MT][NT][4] = {};
            if (SEG && seg > 0)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const float4 v = *reinterpret_cast<const float4 *>(&red[(sums * WARPS + warp) * OUT + (m * NT + n) * TILE + lane * 4]);
                        acc[m][n][0] = v.x, acc[m][n][1] = v.y, acc[m][n][2] = v.z, acc[m][n][3] = v.w;
                    }
            const bool last = seg == n_seg - 1;
            float row_scale[MT][2] = {};
            if (FMT == F_FP8 && last) {
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        row_scale[m][h] = bf16_f32(__ldg(a.wscale + w_row(gu, m, row_in + 8 * h)));
            }
            while (SEG ? at.base == base && at.seg == seg && at.i == i : at.u == gu) {
                const int slot = used & (STAGES - 1), s = at.st;
                at.st += WARPS;
                settle(at);
                if constexpr (C_::NIBBLE) {
#pragma unroll
                    for (int x = 0; x < C_::BOXES; ++x) sc[x][0] = sc_next[x][0], sc[x][1] = sc_next[x][1];
                    if (more(at)) {
                        if (at.u != sc_u) scale_rows(sc_u = at.u);
                        load_scales(at.seg * SS + at.st, sc_next);
                    }
                }
                if (ok) ok = wait_bounded(smem_u32(&bars[warp * STAGES + slot]), static_cast<uint32_t>(used / STAGES) & 1u,
                                          abort_flag, a.err, DERR_WAIT_FULL);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t box0 = ring0 + slot * STAGE;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    uint32_t xb[NT][8];
#pragma unroll
                    for (int n = 0; n < NT; ++n) load_x(n, s * BLOCKS + b, xb[n]);
                    const int bb = b % C_::BOX_BLOCKS;  // block of its box
                    // the lane's weights of the block, as loaded: two rows of each m-tile
                    uint4 q[MT][2][FMT == F_BF16 ? 2 : 1];
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t p = box0 + (MT == 2 ? m : b / C_::BOX_BLOCKS) * BOX + h * 1024 + chunk[bb];
                            if constexpr (C_::NIBBLE) {
                                const uint2 c = lds8(p);
                                q[m][h][0] = make_uint4(c.x, c.y, 0, 0);
                            } else {
                                q[m][h][0] = lds16(p);
                                if constexpr (FMT == F_BF16) q[m][h][1] = lds16(box0 + (MT == 2 ? m : b / C_::BOX_BLOCKS) * BOX + h * 1024 + chunk[1]);
                            }
                        }
                    // pairs 2 i, 2 i + 1 of a row: its operand of the i-th product
                    auto pairs = [&](const uint4 (&c)[FMT == F_BF16 ? 2 : 1], int i, uint32_t &lo, uint32_t &hi) {
                        if constexpr (FMT == F_BF16) {
                            const uint4 &v = c[i >> 1];
                            lo = i & 1 ? v.z : v.x;
                            hi = i & 1 ? v.w : v.y;
                        } else if constexpr (FMT == F_FP8) {
                            widen_fp8(i == 0 ? c[0].x : i == 1 ? c[0].y : i == 2 ? c[0].z : c[0].w, lo, hi);
                        } else if constexpr (FMT == F_Q4) {
                            const uint32_t v = i < 2 ? c[0].x : c[0].y;
                            lo = and_or(v >> (i & 1 ? 8 : 0), q4_mask, q4_bits);
                            hi = and_or(v >> (i & 1 ? 12 : 4), q4_mask, q4_bits);
                        } else {
                            const uint32_t v = i < 2 ? c[0].x : c[0].y;
                            lo = cb_pair(table_lane, v, (i & 1) * 2);
                            hi = cb_pair(table_lane, v, (i & 1) * 2 + 1);
                        }
                    };
                    // Widening alternates with the products of the m-tiles, so that a product's latency is spent
                    // on the next one's operands.
                    float p4[MT][NT][4], xo[NT][4];  // xo: -136 times the sum of x, of the lane's tokens
                    if constexpr (FMT == F_Q4 && !SEG) {
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 v = lds8(xsum0 + ((s * BLOCKS + b) * 8 * NT + n * 8) * 4);
                            xo[n][0] = __uint_as_float(v.x), xo[n][1] = __uint_as_float(v.y);
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            uint32_t a0, a1, a2, a3;
                            pairs(q[m][0], i, a0, a2);
                            pairs(q[m][1], i, a1, a3);
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if constexpr (C_::NIBBLE) {
                                    if (i == 0 && FMT == F_Q4 && !SEG)
                                        mma_bf16_from(p4[m][n], a0, a1, a2, a3, xb[n][0], xb[n][1], xo[n][0], xo[n][1]);
                                    else if (i == 0) mma_bf16_zero(p4[m][n], a0, a1, a2, a3, xb[n][0], xb[n][1]);
                                    else mma_bf16(p4[m][n], a0, a1, a2, a3, xb[n][2 * i], xb[n][2 * i + 1]);
                                } else {
                                    mma_bf16(acc[m][n], a0, a1, a2, a3, xb[n][2 * i], xb[n][2 * i + 1]);
                                }
                            }
                        }
                        if constexpr (FMT == F_Q4 && SEG) {  // one more product, with -136 for the weights
                            constexpr uint32_t off = 0xC308C308u;
#pragma unroll
                            for (int n = 0; n < NT; ++n) {
                                if (i == 0) mma_bf16_zero(xo[n], off, off, off, off, xb[n][0], xb[n][1]);
                                else mma_bf16(xo[n], off, off, off, off, xb[n][2 * i], xb[n][2 * i + 1]);
                            }
                        }
                    }
                    if constexpr (C_::NIBBLE) {
                        // the block's sums times the scale of each of the lane's rows; a 4-bit code stands for
                        // q - 8 = (128 + q) - 136
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            const int x_ = MT == 2 ? m : b / C_::BOX_BLOCKS;
                            const uint32_t q0 = bb < 2 ? sc[x_][0].x : sc[x_][0].y, q1 = bb < 2 ? sc[x_][1].x : sc[x_][1].y;
                            const float s0 = __uint_as_float(bb & 1 ? q0 & 0xFFFF0000u : q0 << 16);
                            const float s1 = __uint_as_float(bb & 1 ? q1 & 0xFFFF0000u : q1 << 16);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float v = FMT == F_Q4 && SEG ? p4[m][n][e] + xo[n][e & 1] : p4[m][n][e];
                                    acc[m][n][e] = fmaf(e < 2 ? s0 : s1, v, acc[m][n][e]);
                                }
                        }
                    }
                }
                __syncwarp();  // every lane has read the stage
                ++used;
                advance();
            }
            // the group's sums of this warp, once the slot's last group is finished
            const uint32_t round = static_cast<uint32_t>(SEG ? base / GROUPS : base >> 1);  // of the slot
            if (ok && seg == 0) ok = wait_bounded(smem_u32(&red_empty[sums]), (round & 1u) ^ 1u, abort_flag, a.err,
                                                  DERR_WAIT_TMEM_EMPTY);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float v[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[e] = acc[m][n][e];
                        if (FMT == F_FP8 && last) v[e] *= row_scale[m][e >> 1];
                        if (FMT == F_Q4 && last) v[e] *= 1.0f / 7.0f;
                    }
                    *reinterpret_cast<float4 *>(&red[(sums * WARPS + warp) * OUT + (m * NT + n) * TILE + lane * 4]) =
                        make_float4(v[0], v[1], v[2], v[3]);
                }
            __syncwarp();
            if (last && lane == 0) mbar_arrive(smem_u32(&red_full[sums]));
        }
        if constexpr (SEG) {
            __syncwarp();  // every lane has read the segment
            if (lane == 0) mbar_arrive(smem_u32(&x_empty[fill & 1]));
        }
        }
        // After a wait that ran out: copies still in flight land before the CTA leaves.
        if (!ok && lane == 0)
            for (int q = used; q < requested; ++q) {
                volatile int never = 0;
                wait_bounded(smem_u32(&bars[warp * STAGES + (q & (STAGES - 1))]), static_cast<uint32_t>(q / STAGES) & 1u, &never,
                             a.err, DERR_WAIT_DRAIN);
            }
        return;
    }

    // ---------------------------------------------------------------------- finish
    const int fw = warp - WARPS, o = threadIdx.x - WARPS * 32;  // a thread: value o of each n-tile
    const int l = o >> 2, oi = o & 3;
    // s.xa and the fragments of B run through the same products; warp fw takes tile fw of MT x NT
    auto low_rank = [&](int u) {
        if (fw < MT * NT) {
            const int m = fw / NT, n = fw % NT;
            const int64_t r0 = w_row(u, m, row_in), r1 = w_row(u, m, row_in + 8);
            const uint4 zero = make_uint4(0, 0, 0, 0);
            float c[4] = {};
#pragma unroll 2
            for (int k = 8 * j; k < (a.r + 31) / 32 * 32; k += 32) {
                const bool in = k < a.r;
                const uint4 b0 = in ? __ldcg(reinterpret_cast<const uint4 *>(a.B + r0 * a.r + k)) : zero;
                const uint4 b1 = in ? __ldcg(reinterpret_cast<const uint4 *>(a.B + r1 * a.r + k)) : zero;
                const uint4 v = in && n * 8 + g < a.M
                                    ? __ldcg(reinterpret_cast<const uint4 *>(a.xa + static_cast<int64_t>(n * 8 + g) * a.r + k)) : zero;
                __syncwarp();
                mma_bf16(c, b0.x, b1.x, b0.y, b1.y, v.x, v.y);
                mma_bf16(c, b0.z, b1.z, b0.w, b1.w, v.z, v.w);
            }
            *reinterpret_cast<float4 *>(&tail[fw * TILE + lane * 4]) = make_float4(c[0], c[1], c[2], c[3]);
        }
    };
    // this thread's value of n-tile n and m-tile m of group u: its token, and its row in W (gated: the
    // m-th projection's), up to the projection's last
    auto token_of = [&](int n) { return n * 8 + 2 * (l & 3) + (oi & 1); };
    auto row_of = [&](int u, int m) {
        return u * GROUP_ROWS + tile_row<C_::NIBBLE>(l >> 2) + 8 * (oi >> 1) + m * (OP == D_GLU ? a.N : ROWS);
    };
    auto epilogue = [&](int u, int n, const float (&v)[MT]) {
        const int col0 = row_of(u, 0), token = token_of(n);
        if (token >= a.M) return;
        const int64_t row = static_cast<int64_t>(token) * a.N;
        if constexpr (OP == D_GLU) {
            if (col0 >= a.N) return;
            if (a.save) {
                a.save[2 * row + col0] = f32_bf16(v[0]);
                a.save[2 * row + col0 + a.N] = f32_bf16(v[1]);
            }
            float y = 0.0f;
            act_dispatch(a.act, [&](auto A) { y = act_value<A.value>(v[0]); });
            a.out[row + col0] = f32_bf16(y * v[1]);
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int col = col0 + m * ROWS;
                if (col >= a.N) break;
                float y = v[m];
                if (a.bias) y += bf16_f32(__ldcg(a.bias + col));
                if (a.save) a.save[row + col] = f32_bf16(y);
                act_dispatch(a.act, [&](auto A) { y = act_value<A.value>(y); });
                if (a.residual) y += bf16_f32(__ldcg(a.residual + row + col));
                a.out[row + col] = f32_bf16(y);
            }
        }
    };
    const int fills = (mine + GROUPS - 1) / GROUPS * n_seg;
    int filled = 1;  // segments asked for, by warp fw == 0
    bool ok = true;
    for (int base = 0; ok && base < mine; base += GROUPS) {
        // segments of x: each while the products use the one before, the next batch's first at the end
        if (SEG && fw == 0)
            for (int f = base / GROUPS * n_seg + 1, seg = 1; ok && seg <= n_seg && f < fills; ++f, ++seg) {
                if (f >= 2)
                    ok = wait_bounded(smem_u32(&x_empty[f & 1]), static_cast<uint32_t>((f >> 1) - 1) & 1u, abort_flag, a.err,
                                      DERR_WAIT_EMPTY);
                ok = __all_sync(0xffffffffu, ok);
                if (ok) {
                    x_fill(seg < n_seg ? seg : 0, f & 1);
                    filled = f + 1;
                }
            }
        if (base == 0) grid_dep_wait();  // s.xa is there, and no earlier kernel still reads what is stored here
        for (int i = 0; i < min(GROUPS, mine - base); ++i) {
        const int u = u0 + (base + i) * u_step, sums = SEG ? i : base & 1;
        const uint32_t round = static_cast<uint32_t>(SEG ? base / GROUPS : base >> 1);
        low_rank(u);
        // the low-rank term of all four warps is there, and all four agree on how the wait ended
        ok = !fin_any(!ok || !wait_bounded(smem_u32(&red_full[sums]), round & 1u, abort_flag, a.err, DERR_WAIT_TMEM_FULL));
        if (!ok) break;
        float v[NT][MT];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                v[n][m] = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w) v[n][m] += red[(sums * WARPS + w) * OUT + (m * NT + n) * TILE + o];
                if (FMT == F_Q4 && __builtin_expect(!(fabsf(v[n][m]) < INFINITY), 0)) {
                    // 128 + q or the offset went past fp32 (an infinite x: inf - inf, which is NaN where
                    // (q - 8) x is not), or the sum itself is not finite: formed again from the codes
                    const int token = token_of(n), row = row_of(u, m);
                    if (token < a.M && row < (OP == D_GLU ? m + 1 : 1) * a.N) v[n][m] = q4_sum(a, row, token);
                }
                v[n][m] += tail[(m * NT + n) * TILE + o];
            }
        named_bar_sync(1, FIN_WARPS * 32);  // read by all before the next group's low-rank term
        if (lane == 0) mbar_arrive(smem_u32(&red_empty[sums]));
#pragma unroll
        for (int n = 0; n < NT; ++n) epilogue(u, n, v[n]);
        }
    }
    // After a wait that ran out: the last copy into each buffer lands before the CTA leaves (product
    // warps that gave up no longer wait for it).
    if (SEG && !ok && fw == 0 && lane == 0)
        for (int f = max(0, filled - 2); f < filled; ++f) {
            volatile int never = 0;
            wait_bounded(smem_u32(&x_full[f & 1]), static_cast<uint32_t>(f >> 1) & 1u, &never, a.err, DERR_WAIT_DRAIN);
        }
}

// ------------------------------------------------------------------ s.xa = bf16(s . x.A^T)
// The same products on A's rows, few and short: no ring, each lane loads its weights straight
// from memory, the CTAs of a cluster split K.
constexpr int XA_WARPS = 8;

template <int NT>
__global__ void __launch_bounds__(XA_WARPS * 32) k_decode_xa(const uint16_t *x, const uint16_t *A, uint16_t *xa, int M,
                                                             int K, int r, float scale, int C) {
    __shared__ float red[XA_WARPS][NT * TILE];
    __shared__ float sums[NT * TILE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, j = lane & 3;
    const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row0 = static_cast<int>(blockIdx.x) / C * ROWS;
    grid_dep_wait();
    grid_dep_launch_dependents();  // only now: k_decode reads x without waiting for this kernel
    const uint4 zero = make_uint4(0, 0, 0, 0);
    auto at = [&](const uint16_t *p, int64_t row, int k) {
        return k < K ? __ldcg(reinterpret_cast<const uint4 *>(p + row * K + k)) : zero;
    };
    const int64_t a0 = min(row0 + g, r - 1), a1 = min(row0 + g + 8, r - 1);  // rows behind r are not stored
    float acc[NT][4] = {};
    const int steps = (K + 31) / 32;
    const int s_lo = steps * rank / C, s_hi = steps * (rank + 1) / C;
#pragma unroll 2
    for (int s = s_lo + warp; s < s_hi; s += XA_WARPS) {
        const int k = s * 32 + 8 * j;
        const uint4 w0 = at(A, a0, k), w1 = at(A, a1, k);
        uint4 v[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) v[t] = t * 8 + g < M ? at(x, t * 8 + g, k) : zero;
        __syncwarp();
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            mma_bf16(acc[t], w0.x, w1.x, w0.y, w1.y, v[t].x, v[t].y);
            mma_bf16(acc[t], w0.z, w1.z, w0.w, w1.w, v[t].z, v[t].w);
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
        *reinterpret_cast<float4 *>(&red[warp][t * TILE + lane * 4]) = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    for (int o = threadIdx.x; o < NT * TILE; o += XA_WARPS * 32) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < XA_WARPS; ++w) v += red[w][o];
        sums[o] = v;
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0)
        for (int o = threadIdx.x; o < NT * TILE; o += XA_WARPS * 32) {
            float v = sums[o];
            for (int c = 1; c < C; ++c) {
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];"
                             : "=f"(f) : "r"(mapa_shared(smem_u32(&sums[o]), static_cast<uint32_t>(c))) : "memory");
                v += f;
            }
            const int l = (o & (TILE - 1)) >> 2, i = o & 3;
            const int n = row0 + (l >> 2) + 8 * (i >> 1), token = o / TILE * 8 + 2 * (l & 3) + (i & 1);
            if (n < r && token < M) xa[static_cast<int64_t>(token) * r + n] = f32_bf16(v * scale);
        }
    if (C > 1) cluster_sync();  // no CTA leaves while its sums may still be read
}

// ------------------------------------------------------------------ host
void launch_config(cudaLaunchConfig_t *cfg, cudaLaunchAttribute (&attr)[2], int grid, int threads, size_t smem, int cluster,
                   cudaStream_t st) {
    std::memset(cfg, 0, sizeof(*cfg));
    cfg->gridDim = dim3(static_cast<unsigned>(grid));
    cfg->blockDim = dim3(static_cast<unsigned>(threads));
    cfg->dynamicSmemBytes = smem;
    cfg->stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg->attrs = attr;
    cfg->numAttrs = lora_host::programmatic_launch() ? 2 : 1;
}

std::mutex g_mu;

// Raise an instantiation's shared-memory limit, once a device.
template <int FMT, int OP, int NT, bool SEG, int MT>
cudaError_t launch(const DecodeArgs &a, int grid, int64_t x_bytes, cudaStream_t st) {
    using C_ = Cfg<FMT, OP, NT, SEG, MT>;
    static bool done[64] = {};  // shared-memory limit raised, once a device
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    {
        std::lock_guard<std::mutex> lk(g_mu);
        if (!done[d]) {
            e = cudaFuncSetAttribute(k_decode<FMT, OP, NT, SEG, MT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     C_::FIXED + C_::X_MAX);
            if (e != cudaSuccess) return e;
            done[d] = true;
        }
    }
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config(&cfg, attr, grid, C_::THREADS, C_::FIXED + static_cast<size_t>(x_bytes), 1, st);
    e = cudaLaunchKernelEx(&cfg, k_decode<FMT, OP, NT, SEG, MT>, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    lora_host::count_launch();
    return e;
}

template <int FMT, int OP, int NT, int MT>
cudaError_t launch_x(const DecodeArgs &a, int sms, cudaStream_t st) {
    using C_ = Cfg<FMT, OP, NT, false, MT>;
    // One CTA an SM, each with as many groups as the fullest has to have: fewer SMs than all of
    // them still draw the whole bandwidth, and none waits for a last one.
    const int groups = (a.N + C_::GROUP_ROWS - 1) / C_::GROUP_ROWS, rounds = (groups + sms - 1) / sms;
    const int grid = (groups + rounds - 1) / rounds;
    const int64_t S = (a.K + C_::STAGE_K - 1) / C_::STAGE_K;
    // all of x, with 4-bit codes and its blocks' sums
    const int64_t x_bytes = a.M * (S * C_::STAGE_K * 2 + C_::X_PAD) + (FMT == F_Q4 ? S * C_::BLOCKS * 8 * NT * 4 : 0);
    if (x_bytes <= C_::X_MAX) return launch<FMT, OP, NT, false, MT>(a, grid, x_bytes, st);
    // The longest segments of which two fit.
    using G_ = Cfg<FMT, OP, NT, true, MT>;
    static_assert(G_::X_MAX / 2 >= 8 * NT * (G_::STAGE_K * 2 + G_::X_PAD), "one stage of x");
    const int64_t seg_S = (a.K + G_::STAGE_K - 1) / G_::STAGE_K;
    const int64_t most = (G_::X_MAX / 2 / a.M - G_::X_PAD) / (G_::STAGE_K * 2), n_seg = (seg_S + most - 1) / most;
    DecodeArgs seg = a;
    seg.seg_stages = static_cast<int>((seg_S + n_seg - 1) / n_seg);
    return launch<FMT, OP, NT, true, MT>(seg, grid, 2 * a.M * (int64_t(seg.seg_stages) * G_::STAGE_K * 2 + G_::X_PAD), st);
}

// The s.xa kernel asks for the shared-memory split that k_decode needs, so that an SM it runs on
// does not have to empty before a CTA of k_decode can join it; once a device.
cudaError_t prepare_xa() {
    static bool done[64] = {};
    int d = 0;
    cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(g_mu);
    if (!done[d]) {
        for (auto kern : {k_decode_xa<1>, k_decode_xa<2>}) {
            e = cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
            if (e != cudaSuccess) return e;
        }
        done[d] = true;
    }
    return cudaSuccess;
}

// Groups of 32 rows (two m-tiles) read x once for both.  The gated projections' are such by nature;
// plain ones take them where the products weigh more than the stream and the fullest CTA has at
// most a fifth more rows to do: 28672 -> 8192, 8 tokens in FP8 66 -> 60 us and 4-bit 56 -> 50, 16
// tokens in bf16 106 -> 89 us.  2048 -> 2048, where they leave half the CTAs, 7.1 us -> 7.4 (4-bit, 8
// tokens); in bf16 up to 8 tokens (11008 -> 4096, one token) 18.0 -> 18.6; codebook, 16 tokens
// of 11008 -> 4096, 24 -> 31.
template <int FMT, int OP, int NT>
cudaError_t launch_mt(const DecodeArgs &a, int sms, cudaStream_t st) {
    if constexpr (OP == D_GLU) {
        return launch_x<FMT, OP, NT, 2>(a, sms, st);
    } else {
        if constexpr (NT == 1 ? FMT != F_BF16 : FMT != F_CB) {
            auto rounds = [&](int rows) { return ((a.N + rows - 1) / rows + sms - 1) / sms; };
            if (2 * rounds(2 * ROWS) * 5 <= 6 * rounds(ROWS)) return launch_x<FMT, OP, NT, 2>(a, sms, st);
        }
        return launch_x<FMT, OP, NT, 1>(a, sms, st);
    }
}

template <int FMT, int OP>
cudaError_t launch_nt(const DecodeArgs &a, int sms, cudaStream_t st) {
    return a.M <= 8 ? launch_mt<FMT, OP, 1>(a, sms, st) : launch_mt<FMT, OP, 2>(a, sms, st);
}

template <int OP>
cudaError_t launch_fmt(int fmt, const DecodeArgs &a, int sms, cudaStream_t st) {
    switch (fmt) {
        case F_Q4: return launch_nt<F_Q4, OP>(a, sms, st);
        case F_FP8: return launch_nt<F_FP8, OP>(a, sms, st);
        case F_CB: return launch_nt<F_CB, OP>(a, sms, st);
        default: return launch_nt<F_BF16, OP>(a, sms, st);
    }
}

}  // namespace

namespace lora_host {

cudaError_t launch_decode(const uint16_t *A, uint16_t *xa, float s, int format, bool glu, DecodeArgs a, const void *w,
                          int sms, cudaStream_t st) {
    const uint64_t rows = static_cast<uint64_t>(a.N) * (glu ? 2 : 1);
    const uint64_t row_bytes = format == F_BF16 ? uint64_t(a.K) * 2 : format == F_FP8 ? uint64_t(a.K) : uint64_t(a.K) / 2;
    if (!tmap_2d(&a.tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w, row_bytes, rows, TILE_BYTES, ROWS, CU_TENSOR_MAP_SWIZZLE_128B))
        return cudaErrorInvalidValue;
    // s.xa: clusters of up to 8 CTAs, as long as each warp keeps a 32-wide step
    int C = 1;
    while (C < 8 && (a.K + 31) / 32 >= 2 * C * XA_WARPS) C *= 2;
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute attr[2];
    launch_config(&cfg, attr, (a.r + ROWS - 1) / ROWS * C, XA_WARPS * 32, 0, C, st);
    cudaError_t e = prepare_xa();
    if (e != cudaSuccess) return e;
    e = cudaLaunchKernelEx(&cfg, a.M <= 8 ? k_decode_xa<1> : k_decode_xa<2>, a.x, A, xa, a.M, a.K, a.r, s, C);
    if (e == cudaSuccess) e = cudaGetLastError();
    count_launch();
    if (e != cudaSuccess) return e;
    a.xa = xa;
    a.w = static_cast<const uint8_t *>(w);
    return glu ? launch_fmt<D_GLU>(format, a, sms, st) : launch_fmt<D_ACT>(format, a, sms, st);
}

}  // namespace lora_host
