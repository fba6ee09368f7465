// decode.cu -- the gated and the epilogue projections of a few tokens (generating text):
//
//   acc[n, m] = sum_k W[n, k] x[m, k] + sum_j B[n, j] (s.xa)[m, j],   then the epilogue
//
// Bound by reading W once.  A 256 x 256 tensor-core tile per CTA pair would put only
// d_out / 256 pairs of SMs on that stream, so here a cluster of CTAs takes 16 weight rows (the
// gate's and the up projection's 16, when gated), its warps split K, and each lane loads the
// weight straight from memory into the registers of mma.sync m16n8k16: weight rows are the
// 16-row side, tokens the 8-column side (M <= 8 NT).  A lane's 16-byte load holds 8
// consecutive k of one row; since both operands may order k in any one way, those are the k of
// the lane's fragment registers of two products, and x is loaded by the same rule: no shared
// memory, no shuffles, no layout of W other than its own.
//
// Codes are widened in registers.  4-bit codes enter the products as the exact integers q - 8,
// E4M3 codes as their exact values; the scale (one a row, or one a row and 64 k) multiplies
// the fp32 sums, so no decoded weight is rounded.  Codebook values are rounded once to bf16
// and looked up two codes at a time in a shared table of a byte's 256 pairs, one copy for
// each lane's bank.
//
// The sums of the CTA's warps, then of the cluster's CTAs, are added in a fixed order; the
// low-rank term is one warp's extra products on the rows of B.  s.xa comes from the same
// kernel run on A's rows just before; this kernel starts its stream of W beside it and waits
// for it only before the low-rank term (programmatic dependent launch: the s.xa kernel lets
// it start only once all its own CTAs have seen their predecessor complete, so x is final).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "act.cuh"
#include "decode.h"
#include "ptx.cuh"

namespace {

using namespace lora;
using lora_host::DecodeArgs;

constexpr int WARPS = 8;
constexpr int ROWS = 16;  // weight rows per m-tile
enum DecodeOp { D_XA = 0, D_ACT = 1, D_GLU = 2 };
enum DecodeFmt { F_BF16 = LORA_W_BF16, F_Q4 = LORA_W_Q4, F_FP8 = LORA_W_FP8, F_CB = LORA_W_NF4 };

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Weights are read once: past L1, and 256 bytes at a time into L2.
__device__ __forceinline__ uint4 ld_stream16(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ld_stream8(const void *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.L2::256B.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t d;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(sel));
    return d;
}

// One row's 64-wide step as loaded by a lane (16 weights), and its scale.
template <int FMT>
struct RowLoad {
    uint4 v[FMT == F_BF16 ? 2 : 1];
    uint16_t sc;
};

// Lane's weights of one row in a 64-wide step: bf16, k0 + 8 j and k0 + 32 + 8 j (8 each);
// codes, the 16 from k0 + 16 j.  Nothing is read at or behind K.
template <int FMT>
__device__ __forceinline__ void load_row(RowLoad<FMT> &r, const DecodeArgs &a, int64_t row, int k0, int j) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if constexpr (FMT == F_BF16) {
        const uint16_t *p = static_cast<const uint16_t *>(a.w) + row * a.K + k0 + 8 * j;
        r.v[0] = k0 + 8 * j < a.K ? ld_stream16(p) : zero;
        r.v[1] = k0 + 32 + 8 * j < a.K ? ld_stream16(p + 32) : zero;
    } else if constexpr (FMT == F_FP8) {
        r.v[0] = k0 + 16 * j < a.K ? ld_stream16(static_cast<const uint8_t *>(a.w) + row * a.K + k0 + 16 * j) : zero;
    } else {  // K % 64 == 0
        const uint2 q = ld_stream8(static_cast<const uint8_t *>(a.w) + row * (a.K / 2) + k0 / 2 + 8 * j);
        r.v[0] = make_uint4(q.x, q.y, 0, 0);
        r.sc = __ldg(a.wscale + row * (a.K / 64) + k0 / 64);
    }
}

// The lane's 16 weights as 8 bf16 pairs, in the order of the x pairs that load_x gives.
template <int FMT>
__device__ __forceinline__ void decode_row(const RowLoad<FMT> &r, const uint32_t *table, int lane, uint32_t (&w)[8]) {
    if constexpr (FMT == F_BF16) {
        w[0] = r.v[0].x, w[1] = r.v[0].y, w[2] = r.v[0].z, w[3] = r.v[0].w;
        w[4] = r.v[1].x, w[5] = r.v[1].y, w[6] = r.v[1].z, w[7] = r.v[1].w;
    } else if constexpr (FMT == F_FP8) {
        const uint32_t q[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            asm("{\n\t.reg .b16 c0, c1, a0, a1, a2, a3;\n\t.reg .b32 h0, h1;\n\t.reg .f32 f0, f1, f2, f3;\n\t"
                "mov.b32 {c0, c1}, %2;\n\t"
                "cvt.rn.f16x2.e4m3x2 h0, c0;\n\t"
                "cvt.rn.f16x2.e4m3x2 h1, c1;\n\t"
                "mov.b32 {a0, a1}, h0;\n\t"
                "mov.b32 {a2, a3}, h1;\n\t"
                "cvt.f32.f16 f0, a0;\n\tcvt.f32.f16 f1, a1;\n\tcvt.f32.f16 f2, a2;\n\tcvt.f32.f16 f3, a3;\n\t"
                "cvt.rn.bf16x2.f32 %0, f1, f0;\n\t"
                "cvt.rn.bf16x2.f32 %1, f3, f2;\n\t}"
                : "=r"(w[2 * i]), "=r"(w[2 * i + 1])
                : "r"(q[i]));
    } else if constexpr (FMT == F_Q4) {
        // pairs (e, e + 4) of each word's 8 codes: a nibble under the exponent of 128 is
        // 128 + q, less 136 it is q - 8, both exact
        const uint32_t q[2] = {r.v[0].x, r.v[0].y};
        const __nv_bfloat162 off = __floats2bfloat162_rn(136.0f, 136.0f);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t u = ((q[i] >> (4 * e)) & 0x000F000Fu) | 0x43004300u;
                const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&u), off);
                w[4 * i + e] = *reinterpret_cast<const uint32_t *>(&d);
            }
    } else {
        const uint32_t q[2] = {r.v[0].x, r.v[0].y};
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int b = 0; b < 4; ++b) w[4 * i + b] = table[((q[i] >> (8 * b)) & 0xFFu) * 32 + lane];
    }
}

// The x pairs of token n that belong to the lane's weights of a step (zero behind M and K).
template <int FMT>
__device__ __forceinline__ void load_x(uint32_t (&v)[8], const DecodeArgs &a, int n, int k0, int j) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int ka = FMT == F_BF16 ? k0 + 8 * j : k0 + 16 * j, kb = FMT == F_BF16 ? ka + 32 : ka + 8;
    const uint16_t *p = a.x + static_cast<int64_t>(n) * a.K;
    const uint4 u = n < a.M && ka < a.K ? __ldcg(reinterpret_cast<const uint4 *>(p + ka)) : zero;
    const uint4 w = n < a.M && kb < a.K ? __ldcg(reinterpret_cast<const uint4 *>(p + kb)) : zero;
    if constexpr (FMT == F_Q4) {
        v[0] = prmt(u.x, u.z, 0x5410), v[1] = prmt(u.x, u.z, 0x7632);
        v[2] = prmt(u.y, u.w, 0x5410), v[3] = prmt(u.y, u.w, 0x7632);
        v[4] = prmt(w.x, w.z, 0x5410), v[5] = prmt(w.x, w.z, 0x7632);
        v[6] = prmt(w.y, w.w, 0x5410), v[7] = prmt(w.y, w.w, 0x7632);
    } else {
        v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
        v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
    }
}

template <int FMT, int OP, int NT>
__global__ void __launch_bounds__(WARPS * 32) k_decode(const __grid_constant__ DecodeArgs a) {
    constexpr int MT = OP == D_GLU ? 2 : 1;
    constexpr int TILE = 128;                 // values of an m-tile x n-tile
    constexpr int PER_STEP = MT == 2 ? 1 : 2;  // steps in flight together
    extern __shared__ uint32_t table[];        // F_CB: [256][32]
    __shared__ float red[WARPS][MT * NT * TILE];
    __shared__ float sums[MT * NT * TILE];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, j = lane & 3;
    const int C = a.cluster, rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int row0 = static_cast<int>(blockIdx.x) / C * ROWS;
    if (OP == D_XA) grid_dep_wait();
    grid_dep_launch_dependents();
    if constexpr (FMT == F_CB) {
        for (int i = threadIdx.x; i < 256 * 32; i += WARPS * 32) {
            const int b = i >> 5;
            const __nv_bfloat162 v = __floats2bfloat162_rn(a.cb[b & 15], a.cb[b >> 4]);
            table[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        __syncthreads();
    }
    // the lane's rows (those behind the output repeat the last one and are not stored)
    int64_t row[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) row[m][h] = static_cast<int64_t>(m) * a.N + min(row0 + g + 8 * h, a.N - 1);
    float acc[MT][NT][4] = {};
    const int steps = (a.K + 63) / 64;
    const int s_lo = steps * rank / C, s_hi = steps * (rank + 1) / C;
    for (int s = s_lo + warp; s < s_hi; s += WARPS * PER_STEP) {
        RowLoad<FMT> ld[PER_STEP][MT][2];
        uint32_t xv[PER_STEP][NT][8];
#pragma unroll
        for (int u = 0; u < PER_STEP; ++u) {
            const int k0 = (s + u * WARPS) * 64;
            if (u > 0 && s + u * WARPS >= s_hi) break;
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int h = 0; h < 2; ++h) load_row<FMT>(ld[u][m][h], a, row[m][h], k0, j);
#pragma unroll
            for (int t = 0; t < NT; ++t) load_x<FMT>(xv[u][t], a, t * 8 + g, k0, j);
        }
#pragma unroll
        for (int u = 0; u < PER_STEP; ++u) {
            if (u > 0 && s + u * WARPS >= s_hi) break;
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                uint32_t w0[8], w1[8];
                decode_row<FMT>(ld[u][m][0], table, lane, w0);
                decode_row<FMT>(ld[u][m][1], table, lane, w1);
                if constexpr (FMT == F_Q4 || FMT == F_CB) {
                    // the step is one scale block: its sums times the scale
                    const float f = FMT == F_Q4 ? 1.0f / 7.0f : 1.0f;
                    const float s0 = __uint_as_float(static_cast<uint32_t>(ld[u][m][0].sc) << 16) * f;
                    const float s1 = __uint_as_float(static_cast<uint32_t>(ld[u][m][1].sc) << 16) * f;
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        float part[4] = {};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(part, w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1], xv[u][t][2 * i],
                                     xv[u][t][2 * i + 1]);
                        acc[m][t][0] += s0 * part[0];
                        acc[m][t][1] += s0 * part[1];
                        acc[m][t][2] += s1 * part[2];
                        acc[m][t][3] += s1 * part[3];
                    }
                } else {
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            mma_bf16(acc[m][t], w0[2 * i], w1[2 * i], w0[2 * i + 1], w1[2 * i + 1], xv[u][t][2 * i],
                                     xv[u][t][2 * i + 1]);
                }
            }
        }
    }
    if constexpr (FMT == F_FP8) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const float s0 = __uint_as_float(static_cast<uint32_t>(__ldg(a.wscale + row[m][0])) << 16);
            const float s1 = __uint_as_float(static_cast<uint32_t>(__ldg(a.wscale + row[m][1])) << 16);
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                acc[m][t][0] *= s0;
                acc[m][t][1] *= s0;
                acc[m][t][2] *= s1;
                acc[m][t][3] *= s1;
            }
        }
    }
    if (OP != D_XA && rank == 0) {
        // every thread of the storing CTA waits: what it stores may still be read by an earlier
        // kernel, and s.xa is the predecessor's
        grid_dep_wait();
        if (warp == WARPS - 1)
            for (int k0 = 0; k0 < a.r; k0 += 32) {
                const bool in = k0 + 8 * j < a.r;
                const uint4 zero = make_uint4(0, 0, 0, 0);
                uint4 xa[NT];
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    xa[t] = in && t * 8 + g < a.M
                                ? __ldcg(reinterpret_cast<const uint4 *>(a.xa + static_cast<int64_t>(t * 8 + g) * a.r + k0 + 8 * j))
                                : zero;
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const uint4 b0 = in ? __ldcg(reinterpret_cast<const uint4 *>(a.B + row[m][0] * a.r + k0 + 8 * j)) : zero;
                    const uint4 b1 = in ? __ldcg(reinterpret_cast<const uint4 *>(a.B + row[m][1] * a.r + k0 + 8 * j)) : zero;
                    __syncwarp();
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        mma_bf16(acc[m][t], b0.x, b1.x, b0.y, b1.y, xa[t].x, xa[t].y);
                        mma_bf16(acc[m][t], b0.z, b1.z, b0.w, b1.w, xa[t].z, xa[t].w);
                    }
                }
            }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t)
            *reinterpret_cast<float4 *>(&red[warp][(m * NT + t) * TILE + lane * 4]) =
                make_float4(acc[m][t][0], acc[m][t][1], acc[m][t][2], acc[m][t][3]);
    __syncthreads();
    for (int o = threadIdx.x; o < MT * NT * TILE; o += WARPS * 32) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) v += red[w][o];
        sums[o] = v;
    }
    if (C > 1) cluster_sync();
    else __syncthreads();
    if (rank == 0) {
        for (int o = threadIdx.x; o < NT * TILE; o += WARPS * 32) {
            float v[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int at = m * NT * TILE + o;
                v[m] = sums[at];
                for (int c = 1; c < C; ++c) {
                    float f;
                    asm volatile("ld.shared::cluster.f32 %0, [%1];"
                                 : "=f"(f)
                                 : "r"(mapa_shared(smem_u32(&sums[at]), static_cast<uint32_t>(c))));
                    v[m] += f;
                }
            }
            const int l = (o & (TILE - 1)) >> 2, i = o & 3;
            const int n = row0 + (l >> 2) + 8 * (i >> 1), token = o / TILE * 8 + 2 * (l & 3) + (i & 1);
            if (n >= a.N || token >= a.M) continue;
            const int64_t at = static_cast<int64_t>(token) * a.N + n;
            if constexpr (OP == D_XA) {
                a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0] * a.scale));
            } else if constexpr (OP == D_GLU) {
                if (a.save) {
                    const int64_t s = static_cast<int64_t>(token) * 2 * a.N + n;
                    a.save[s] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
                    a.save[s + a.N] = __bfloat16_as_ushort(__float2bfloat16_rn(v[1]));
                }
                float y = 0.0f;
                act_dispatch(a.act, [&](auto A) { y = act_value<A.value>(v[0]); });
                a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y * v[1]));
            } else {
                float y = v[0];
                if (a.bias) y += __uint_as_float(static_cast<uint32_t>(__ldcg(a.bias + n)) << 16);
                if (a.save) a.save[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
                act_dispatch(a.act, [&](auto A) { y = act_value<A.value>(y); });
                if (a.residual) y += __uint_as_float(static_cast<uint32_t>(__ldcg(a.residual + at)) << 16);
                a.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
            }
        }
    }
    if (C > 1) cluster_sync();  // no CTA leaves while its sums may still be read
}

template <int FMT, int OP, int NT>
cudaError_t launch(const DecodeArgs &a, cudaStream_t st) {
    auto kern = k_decode<FMT, OP, NT>;
    constexpr size_t smem = FMT == F_CB ? 256 * 32 * sizeof(uint32_t) : 0;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3(static_cast<unsigned>((a.N + ROWS - 1) / ROWS * a.cluster));
    cfg.blockDim = dim3(WARPS * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = a.cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = lora_host::programmatic_launch() ? 2 : 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    lora_host::count_launch();
    return e;
}

template <int FMT, int OP>
cudaError_t launch_nt(const DecodeArgs &a, cudaStream_t st) {
    if (a.M <= 8) return launch<FMT, OP, 1>(a, st);
    return launch<FMT, OP, 2>(a, st);
}

template <int OP>
cudaError_t launch_fmt(int fmt, const DecodeArgs &a, cudaStream_t st) {
    switch (fmt) {
        case F_Q4: return launch_nt<F_Q4, OP>(a, st);
        case F_FP8: return launch_nt<F_FP8, OP>(a, st);
        case F_CB: return launch_nt<F_CB, OP>(a, st);
        default: return launch_nt<F_BF16, OP>(a, st);
    }
}

// CTAs that share 16 rows, splitting K: enough for four CTAs an SM, while each warp keeps two
// steps of 64 (a quarter of that for s.xa, whose whole stream is short: latency counts there).
int choose_cluster(int64_t units, int K, int sms, int steps_per_warp) {
    int c = 1;
    while (c < 8 && units * c < 4 * sms && (K + 63) / 64 >= 2 * c * WARPS * steps_per_warp) c *= 2;
    return c;
}

}  // namespace

namespace lora_host {

cudaError_t launch_decode(const uint16_t *A, uint16_t *xa, float s, int format, bool glu, DecodeArgs a, int sms,
                          cudaStream_t st) {
    DecodeArgs p = a;
    p.w = A;
    p.N = a.r;
    p.out = xa;
    p.scale = s;
    p.cluster = choose_cluster((a.r + ROWS - 1) / ROWS, a.K, sms, 1);
    cudaError_t e = launch_nt<F_BF16, D_XA>(p, st);
    if (e != cudaSuccess) return e;
    a.xa = xa;
    a.cluster = choose_cluster((a.N + ROWS - 1) / ROWS, a.K, sms, 2);
    return glu ? launch_fmt<D_GLU>(format, a, st) : launch_fmt<D_ACT>(format, a, st);
}

}  // namespace lora_host
