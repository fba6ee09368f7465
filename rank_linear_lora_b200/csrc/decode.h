// decode.h -- internal: the projections of a few tokens (decode.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/lora_linear.h"
#include "block.h"

namespace lora_host {

// Tokens up to which the gated and the epilogue projections run here.
constexpr int64_t DECODE_MAX_M = 16;

struct DecodeArgs {
    CUtensorMap tmW;          // set by launch_decode
    const uint16_t *x;        // [M, K]
    const uint8_t *w;         // the weight, or its codes; set by launch_decode
    const uint16_t *wscale;
    float cb[16];             // LORA_W_NF4
    const uint16_t *B;        // [N or 2 N, r]
    const uint16_t *xa;       // s.xa [M, r]; set by launch_decode
    uint16_t *out;            // [M, N]
    uint16_t *save;           // pre-activations [M, N], or [M, 2 N] when gated; or null
    const uint16_t *bias, *residual;
    int *err;                 // device error word
    int M, N, K, r;
    int act;
    int seg_stages;           // stages of a segment of x; set by launch_decode
};

// s.xa = bf16(s . x.A^T) into xa [M, r], then the projection with the weight (or its codes) w
// [N or 2 N, K]: p = act(g) * u (`glu`) or act(acc + bias) + residual.  M <= DECODE_MAX_M.
cudaError_t launch_decode(const uint16_t *A, uint16_t *xa, float s, int format, bool glu, DecodeArgs a, const void *w,
                          int sms, cudaStream_t st);

}  // namespace lora_host
