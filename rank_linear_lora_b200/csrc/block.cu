// block.cu -- the elementwise halves of the gated and the epilogue projections' backward:
//
//   gated     [dg | du] = [dP * u * act'(g) | dP * act(g)] from dP [M, f] and [g | u] [M, 2f]
//   epilogue  dPre = dOut * act'(pre), and the bias gradient sum_m dPre[m, :]
//
// Both are bound by HBM: each input is read once and each output written once, 16 bytes
// (8 bf16) a load; arithmetic in fp32, one rounding.  What follows (the rank-r products
// and dX of the layer) reads the result through TMA.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "act.cuh"
#include "block.h"
#include "ptx.cuh"

namespace {

using namespace lora;

constexpr int THREADS = 256;

__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[8]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(w[e] << 16);
        f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
        w[e] = *reinterpret_cast<const uint32_t *>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// ------------------------------------------------------------------ gated backward
constexpr int GLU_VECS = 2;  // 8-column vectors per thread: 96 bytes of loads in flight each

// CTA b takes the vectors b * THREADS * GLU_VECS .. of the M * f / 8 of dP.
template <int ACT>
__global__ void __launch_bounds__(THREADS) k_glu_bwd(const uint4 *__restrict__ dP, const uint4 *__restrict__ gu,
                                                     uint4 *__restrict__ dGU, int64_t total, int nv) {
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (THREADS * GLU_VECS);
    const int64_t row0 = base / nv;                        // the CTA's first row; offsets from it are 32-bit
    const uint32_t off0 = static_cast<uint32_t>(base - row0 * nv) + threadIdx.x;
    uint4 d[GLU_VECS], g[GLU_VECS], u[GLU_VECS];
    int64_t at[GLU_VECS];  // vector index of the gate half in gu and dGU
#pragma unroll
    for (int k = 0; k < GLU_VECS; ++k) {
        const uint32_t off = off0 + k * THREADS;
        const int64_t i = base + threadIdx.x + k * THREADS;
        const uint32_t r = off / static_cast<uint32_t>(nv);
        at[k] = (row0 + r) * 2 * nv + (off - r * static_cast<uint32_t>(nv));
        if (i < total) {
            d[k] = __ldcs(dP + i);
            g[k] = __ldcs(gu + at[k]);
            u[k] = __ldcs(gu + at[k] + nv);
        }
    }
#pragma unroll
    for (int k = 0; k < GLU_VECS; ++k) {
        if (base + threadIdx.x + k * THREADS >= total) break;
        float fd[8], fg[8], fu[8];
        unpack8(d[k], fd);
        unpack8(g[k], fg);
        unpack8(u[k], fu);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float y, dy;
            act_both<ACT>(fg[e], y, dy);
            fg[e] = fd[e] * fu[e] * dy;
            fu[e] = fd[e] * y;
        }
        dGU[at[k]] = pack8(fg);
        dGU[at[k] + nv] = pack8(fu);
    }
}

// ------------------------------------------------------------------ epilogue backward
// CTA (x = column block of 256, y = row chunk): a warp takes every 8th row of the chunk, a
// lane 8 columns.  The column sums of dPre stay in registers over the chunk, are added
// over the 8 warps in shared memory, and the chunk's partial goes to the workspace; the
// column block's last CTA to arrive adds the partials in chunk order, so that the result
// does not depend on who was last.
constexpr int ACT_ROWS = 4;  // rows per warp in flight

template <int ACT, bool BIAS>
__global__ void __launch_bounds__(THREADS)
    k_act_bwd(const uint16_t *__restrict__ dOut, const uint16_t *__restrict__ pre, uint16_t *__restrict__ dPre,
              float *__restrict__ dbias, float *__restrict__ partials, int *__restrict__ counters, int64_t M, int N,
              int64_t rows_per_chunk) {
    __shared__ float red[8][256 + 8];
    __shared__ int last;
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int col = blockIdx.x * 256 + lane * 8;
    const int64_t r0 = blockIdx.y * rows_per_chunk, r1 = min(M, r0 + rows_per_chunk);
    float sum[8] = {};
    if (col < N) {
        for (int64_t r = r0 + warp; r < r1; r += 8 * ACT_ROWS) {
            uint4 d[ACT_ROWS], h[ACT_ROWS];
#pragma unroll
            for (int k = 0; k < ACT_ROWS; ++k)
                if (r + 8 * k < r1) {
                    d[k] = __ldcs(reinterpret_cast<const uint4 *>(dOut + (r + 8 * k) * N + col));
                    if (ACT != LORA_ACT_NONE)
                        h[k] = __ldcs(reinterpret_cast<const uint4 *>(pre + (r + 8 * k) * N + col));
                }
#pragma unroll
            for (int k = 0; k < ACT_ROWS; ++k)
                if (r + 8 * k < r1) {
                    float fd[8];
                    unpack8(d[k], fd);
                    if constexpr (ACT != LORA_ACT_NONE) {
                        float fh[8];
                        unpack8(h[k], fh);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            float y, dy;
                            act_both<ACT>(fh[e], y, dy);
                            fd[e] *= dy;
                        }
                        *reinterpret_cast<uint4 *>(dPre + (r + 8 * k) * N + col) = pack8(fd);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) sum[e] += fd[e];
                }
        }
    }
    if constexpr (BIAS) {
#pragma unroll
        for (int e = 0; e < 8; ++e) red[warp][lane * 8 + e] = sum[e];
        __syncthreads();
        const int c = blockIdx.x * 256 + threadIdx.x;
        float s = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += red[w][threadIdx.x];
        if (c < N) __stcg(partials + static_cast<int64_t>(blockIdx.y) * N + c, s);
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            last = atomicAdd(counters + blockIdx.x, 1) == static_cast<int>(gridDim.y) - 1;
            if (last) counters[blockIdx.x] = 0;  // zero again for the next call
        }
        __syncthreads();
        if (last && c < N) {
            __threadfence();
            float t = 0.0f;
#pragma unroll 8
            for (int y = 0; y < static_cast<int>(gridDim.y); ++y) t += __ldcg(partials + static_cast<int64_t>(y) * N + c);
            dbias[c] = t;
        }
    }
}

template <class F>
cudaError_t with_act(int act, F &&f) {
    switch (act) {
        case LORA_ACT_RELU: return f(ActCode<LORA_ACT_RELU>());
        case LORA_ACT_SILU: return f(ActCode<LORA_ACT_SILU>());
        case LORA_ACT_GELU: return f(ActCode<LORA_ACT_GELU>());
        case LORA_ACT_GELU_TANH: return f(ActCode<LORA_ACT_GELU_TANH>());
        default: return f(ActCode<LORA_ACT_NONE>());
    }
}

}  // namespace

namespace lora_host {

cudaError_t launch_glu_bwd(const uint16_t *dP, const uint16_t *gu, uint16_t *dGU, int64_t M, int64_t f, int act,
                           cudaStream_t st) {
    const int64_t total = M * (f / 8);
    const int64_t grid = (total + THREADS * GLU_VECS - 1) / (THREADS * GLU_VECS);
    if (grid > INT32_MAX) return cudaErrorInvalidValue;
    return with_act(act, [&](auto A) {
        return launch_pdl(k_glu_bwd<A.value>, dim3(static_cast<unsigned>(grid)), dim3(THREADS), 0, st,
                          reinterpret_cast<const uint4 *>(dP), reinterpret_cast<const uint4 *>(gu),
                          reinterpret_cast<uint4 *>(dGU), total, static_cast<int>(f / 8));
    });
}

// Four CTAs an SM's worth of chunks over all column blocks, at least 32 rows each (a warp's
// four rows in flight).
BiasPlan bias_plan(int64_t M, int64_t N, int sms) {
    BiasPlan b;
    b.col_blocks = static_cast<int>((N + 255) / 256);
    const int64_t want = std::max<int64_t>(1, (4 * sms + b.col_blocks - 1) / b.col_blocks);
    const int64_t most = (M + 31) / 32;
    const int64_t chunks = std::min(want, most);
    b.rows_per_chunk = (M + chunks - 1) / chunks;
    b.chunks = static_cast<int>((M + b.rows_per_chunk - 1) / b.rows_per_chunk);
    return b;
}

cudaError_t launch_act_bwd(const uint16_t *dOut, const uint16_t *pre, uint16_t *dPre, float *dbias, float *partials,
                           int *counters, int64_t M, int64_t N, int act, const BiasPlan &bp, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(bp.col_blocks), static_cast<unsigned>(bp.chunks));
    return with_act(act, [&](auto A) {
        auto kern = dbias ? k_act_bwd<A.value, true> : k_act_bwd<A.value, false>;
        return launch_pdl(kern, grid, dim3(THREADS), 0, st, dOut, pre, dPre, dbias, partials, counters, M,
                          static_cast<int>(N), bp.rows_per_chunk);
    });
}

}  // namespace lora_host
