// decode.h -- internal: the projections of a few tokens (decode.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/lora_linear.h"
#include "block.h"

namespace lora_host {

// Tokens up to which the gated and the epilogue projections run here.
constexpr int64_t DECODE_MAX_M = 16;

struct DecodeArgs {
    const uint16_t *x;        // [M, K]
    const void *w;            // the weight or its codes, [N or 2 N, K]
    const uint16_t *wscale;
    float cb[16];             // LORA_W_NF4
    const uint16_t *B;        // [N or 2 N, r]
    const uint16_t *xa;       // s.xa [M, r]
    uint16_t *out;            // [M, N]
    uint16_t *save;           // pre-activations [M, N], or [M, 2 N] when gated; or null
    const uint16_t *bias, *residual;
    int M, N, K, r;
    int act;
    int cluster;              // CTAs that split K
    float scale;              // s.xa: s
};

// s.xa = bf16(s . x.A^T) into xa [M, r], then the projection: p = act(g) * u (`glu`) or
// act(acc + bias) + residual.  a.x .. a.act set by the caller, M <= DECODE_MAX_M.
cudaError_t launch_decode(const uint16_t *A, uint16_t *xa, float s, int format, bool glu, DecodeArgs a, int sms,
                          cudaStream_t st);

}  // namespace lora_host
