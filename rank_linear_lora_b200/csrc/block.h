// block.h -- internal: launches of the kernels around the layer (block.cu, heads.cu), and
// what they share with the layer's host code (lora_linear.cu).  Arguments are validated by
// the callers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>

namespace lora_host {

void count_launch();          // one more kernel of this library launched
bool programmatic_launch();   // programmatic dependent launch is on
bool device_supported();      // the current device is one the kernels are built for

// Launch with programmatic dependent launch: the kernel must call grid_dep_wait() before
// it touches memory.
template <class... Params, class... Args>
cudaError_t launch_pdl(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, Args &&...args) {
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = programmatic_launch() ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Params>(args)...);
    if (e == cudaSuccess) e = cudaGetLastError();
    count_launch();
    return e;
}

// dGU = [dP * u * act'(g) | dP * act(g)] with gu = [g | u]; f % 8 == 0.
cudaError_t launch_glu_bwd(const uint16_t *dP, const uint16_t *gu, uint16_t *dGU, int64_t M, int64_t f, int act,
                           cudaStream_t st);

// Split of the bias gradient's column sums: col_blocks x chunks CTAs, a chunk a range of
// rows_per_chunk rows.
struct BiasPlan {
    int col_blocks = 0, chunks = 0;
    int64_t rows_per_chunk = 0;
};
BiasPlan bias_plan(int64_t M, int64_t N, int sms);

// dPre = dOut * act'(pre) (skipped if dPre is null: act none) and dbias = its column sums
// (skipped if dbias is null), through `partials` [chunks][N] and arrival `counters`
// [col_blocks] (zero on entry and on exit); N % 8 == 0.
cudaError_t launch_act_bwd(const uint16_t *dOut, const uint16_t *pre, uint16_t *dPre, float *dbias, float *partials,
                           int *counters, int64_t M, int64_t N, int act, const BiasPlan &bp, cudaStream_t st);

}  // namespace lora_host
