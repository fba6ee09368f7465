// heads.cu -- norms of queries and keys for each head with the rotation of their positions,
// forward and backward, in one pass over the data.
//
//   n = v i w,  i = 1 / sqrt(mean v^2 + eps)          y = R(position) n
//   dn = R^T dy,  e = v i,  dw = sum dn e,  dv = i (dn w - e mean(e dn w))
//                                              = i (dn w - v i^2 mean(v dn w))
//
// Bound by HBM: forward reads and writes each element once, backward reads two and writes
// one.  Layout of the work: a group of L lanes holds one head (one or two 16-byte vectors a
// lane: the vector with dimension j and the one with its partner j + rot/2, so the rotation
// needs no exchange), a warp holds 32 / L heads of one token at a time and goes through the
// token's heads (or a range of them, where tokens are few) with several heads' loads in
// flight; the token's cos and sin stay in registers over its heads, so the fp32 tables,
// as wide as a head itself, are read once a token instead of once a head.  The backward
// forms sum v^2 and sum v dn w in the same shuffles.
//
// The weight gradients are summed per lane over a CTA's whole share in fp32, over the CTA
// in shared memory, and over the CTAs by a second kernel, each in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/lora_linear.h"
#include "block.h"
#include "ptx.cuh"

namespace {

using namespace lora;

constexpr int WARPS = 8;
constexpr int FWD_HEADS = 4;  // heads per group in flight, forward
constexpr int BWD_HEADS = 2;  // backward (two inputs)
constexpr int SMS = 148;

// One of q and k.
struct HeadTensor {
    const void *in, *dy;
    void *out;
    int64_t in_ts, in_hs, dy_ts, dy_hs, out_ts, out_hs;
    const void *weight;
    int heads;
    int per_unit;   // heads a warp takes of one token
    int splits;     // units a token has
    int64_t units;  // M * splits
    int ctas;       // backward: CTAs of this tensor
};

struct HeadArgs {
    HeadTensor t[2];  // q, k (heads 0: absent)
    const float *cos, *sin;
    const int64_t *pos;
    int64_t n_pos;
    int D, rot;
    int log_l;        // lanes per head
    int norm;
    float eps, inv_d;
    float *partials;  // backward: [CTAs][D], or null
};

// ------------------------------------------------------------------ element types
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ float get(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __nv_bfloat16 put(float f) { return __float2bfloat16_rn(f); }
};
template <>
struct Elem<__half> {
    static __device__ float get(__half v) { return __half2float(v); }
    static __device__ __half put(float f) { return __float2half_rn(f); }
};
template <>
struct Elem<float> {
    static __device__ float get(float v) { return v; }
    static __device__ float put(float f) { return f; }
};

template <int BYTES>
struct Raw;
template <>
struct Raw<16> {
    using type = uint4;
};
template <>
struct Raw<8> {
    using type = uint2;
};

// A vector of V elements as loaded.
template <class T, int V>
struct Vec {
    typename Raw<V * sizeof(T)>::type raw;
    __device__ void load(const T *p) { raw = __ldcs(reinterpret_cast<const decltype(raw) *>(p)); }
    __device__ void load_kept(const T *p) { raw = __ldg(reinterpret_cast<const decltype(raw) *>(p)); }
    __device__ void clear() { raw = decltype(raw)(); }
    __device__ void get(float (&f)[V]) const {
        const T *e = reinterpret_cast<const T *>(&raw);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = Elem<T>::get(e[i]);
    }
    __device__ void put(const float (&f)[V]) {
        T *e = reinterpret_cast<T *>(&raw);
#pragma unroll
        for (int i = 0; i < V; ++i) e[i] = Elem<T>::put(f[i]);
    }
    __device__ void store(T *p) const { *reinterpret_cast<decltype(raw) *>(p) = raw; }
};

// ------------------------------------------------------------------ a lane's share of a head
// Slots of V elements.  Halves: slot 0 is vector p of the first rot/2 dimensions, slot 1
// its partner, slots 2.. (NS of them) the dimensions behind the rotation.  INTER: two slots
// over all of D, pairs inside a vector.
template <int V, bool INTER, int NS>
struct Lane {
    static constexpr int SLOTS = INTER ? 2 : 2 + NS;
    int off[SLOTS];   // first dimension
    bool has[SLOTS];
    float c[V], s[V];  // halves: of the vector's dimensions; INTER: V/2 pairs per slot

    __device__ void place(int D, int rot, int p, int L) {
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                off[i] = (p + i * L) * V;
                has[i] = off[i] < D;
            }
        } else {
            off[0] = p * V;
            off[1] = rot / 2 + p * V;
            has[0] = has[1] = p * V < rot / 2;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                off[2 + i] = rot + (p + i * L) * V;
                has[2 + i] = off[2 + i] < D;
            }
        }
    }
    // cos and sin of a token; a position outside the table makes the rotated dimensions NaN
    __device__ void angles(const HeadArgs &a, int64_t token) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            c[e] = 1.0f;
            s[e] = 0.0f;
        }
        if (a.rot == 0) return;
        const int64_t pos = __ldg(a.pos + token);
        const bool ok = pos >= 0 && pos < a.n_pos;
        const int64_t row = ok ? pos * (a.rot / 2) : 0;
        constexpr int N = INTER ? V / 2 : V;  // table entries of a slot
#pragma unroll
        for (int i = 0; i < (INTER ? 2 : 1); ++i) {
            if (!has[i] || (INTER && off[i] >= a.rot)) continue;
            const int64_t at = row + (INTER ? off[i] / 2 : off[i]);
#pragma unroll
            for (int e = 0; e < N; e += (N < 4 ? 2 : 4)) {
                if constexpr (N < 4) {
                    const float2 fc = __ldg(reinterpret_cast<const float2 *>(a.cos + at + e));
                    const float2 fs = __ldg(reinterpret_cast<const float2 *>(a.sin + at + e));
                    c[i * N + e] = fc.x, c[i * N + e + 1] = fc.y;
                    s[i * N + e] = fs.x, s[i * N + e + 1] = fs.y;
                } else {
                    const float4 fc = __ldg(reinterpret_cast<const float4 *>(a.cos + at + e));
                    const float4 fs = __ldg(reinterpret_cast<const float4 *>(a.sin + at + e));
                    c[i * N + e] = fc.x, c[i * N + e + 1] = fc.y, c[i * N + e + 2] = fc.z, c[i * N + e + 3] = fc.w;
                    s[i * N + e] = fs.x, s[i * N + e + 1] = fs.y, s[i * N + e + 2] = fs.z, s[i * N + e + 3] = fs.w;
                }
            }
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (!ok) c[i * N + e] = s[i * N + e] = __int_as_float(0x7fc00000);
        }
    }
    // rotate by the angles (sign 1) or back (sign -1)
    template <int SIGN>
    __device__ void rotate(float (&v)[SLOTS][V]) const {
        if constexpr (INTER) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < V / 2; ++e) {
                    const float x = v[i][2 * e], y = v[i][2 * e + 1];
                    const float cc = c[i * (V / 2) + e], ss = SIGN * s[i * (V / 2) + e];
                    v[i][2 * e] = x * cc - y * ss;
                    v[i][2 * e + 1] = y * cc + x * ss;
                }
        } else {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                const float x = v[0][e], y = v[1][e], ss = SIGN * s[e];
                v[0][e] = x * c[e] - y * ss;
                v[1][e] = y * c[e] + x * ss;
            }
        }
    }
};

// Sum over the L lanes of a head (all 32 lanes take part).
__device__ __forceinline__ float sum_head(float v, int log_l) {
    for (int i = 0; i < log_l; ++i) v += __shfl_xor_sync(0xffffffffu, v, 1 << i);
    return v;
}

// The weight of a lane's slots, as loaded (ones without a weight).
template <class T, int V, class LaneT>
__device__ __forceinline__ void load_weight(const HeadTensor &t, const LaneT &ln, Vec<T, V> (&w)[LaneT::SLOTS]) {
#pragma unroll
    for (int i = 0; i < LaneT::SLOTS; ++i) {
        if (t.weight && ln.has[i]) {
            w[i].load_kept(static_cast<const T *>(t.weight) + ln.off[i]);
        } else {
            float one[V];
#pragma unroll
            for (int e = 0; e < V; ++e) one[e] = 1.0f;
            w[i].put(one);
        }
    }
}

// ------------------------------------------------------------------ forward
template <class T, int V, bool INTER, int NS>
__global__ void __launch_bounds__(WARPS * 32) k_heads_fwd(const __grid_constant__ HeadArgs a) {
    using LaneT = Lane<V, INTER, NS>;
    constexpr int SL = LaneT::SLOTS;
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31;
    int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int which = u >= a.t[0].units;
    if (which) u -= a.t[0].units;
    const HeadTensor &t = a.t[which];
    if (u >= t.units) return;
    const int64_t token = u / t.splits;
    const int h_lo = static_cast<int>(u - token * t.splits) * t.per_unit;
    const int h_hi = min(t.heads, h_lo + t.per_unit);
    const int L = 1 << a.log_l, G = 32 >> a.log_l, g = lane >> a.log_l;
    LaneT ln;
    ln.place(a.D, a.rot, lane & (L - 1), L);
    const T *in = static_cast<const T *>(t.in) + token * t.in_ts;
    T *out = static_cast<T *>(t.out) + token * t.out_ts;
    Vec<T, V> w[SL];
    for (int h0 = h_lo + g; h0 - g < h_hi; h0 += G * FWD_HEADS) {
        Vec<T, V> x[FWD_HEADS][SL];
#pragma unroll
        for (int j = 0; j < FWD_HEADS; ++j)
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                x[j][i].clear();
                if (h0 + j * G < h_hi && ln.has[i]) x[j][i].load(in + (h0 + j * G) * t.in_hs + ln.off[i]);
            }
        if (h0 - g == h_lo) {  // behind the first heads' loads
            ln.angles(a, token);
            load_weight<T, V>(t, ln, w);
        }
#pragma unroll
        for (int j = 0; j < FWD_HEADS; ++j) {
            float v[SL][V], ss = 0.0f;
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                x[j][i].get(v[i]);
#pragma unroll
                for (int e = 0; e < V; ++e) ss += v[i][e] * v[i][e];
            }
            ss = sum_head(ss, a.log_l);
            const float inv = a.norm ? rsqrtf(ss * a.inv_d + a.eps) : 1.0f;
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                float f[V];
                w[i].get(f);
#pragma unroll
                for (int e = 0; e < V; ++e) v[i][e] = v[i][e] * inv * f[e];
            }
            ln.template rotate<1>(v);
            if (h0 + j * G < h_hi) {
#pragma unroll
                for (int i = 0; i < SL; ++i)
                    if (ln.has[i]) {
                        Vec<T, V> y;
                        y.put(v[i]);
                        y.store(out + (h0 + j * G) * t.out_hs + ln.off[i]);
                    }
            }
        }
    }
}

// ------------------------------------------------------------------ backward
template <class T, int V, bool INTER, int NS>
__global__ void __launch_bounds__(WARPS * 32) k_heads_bwd(const __grid_constant__ HeadArgs a) {
    using LaneT = Lane<V, INTER, NS>;
    constexpr int SL = LaneT::SLOTS;
    __shared__ float red[WARPS][256];
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = static_cast<int>(blockIdx.x) >= a.t[0].ctas;
    const HeadTensor &t = a.t[which];
    const int cta = static_cast<int>(blockIdx.x) - (which ? a.t[0].ctas : 0);
    const int L = 1 << a.log_l, G = 32 >> a.log_l, g = lane >> a.log_l;
    LaneT ln;
    ln.place(a.D, a.rot, lane & (L - 1), L);
    Vec<T, V> w[SL];
    load_weight<T, V>(t, ln, w);
    float dw[SL][V] = {};
    for (int64_t u = static_cast<int64_t>(cta) * WARPS + warp; u < t.units; u += static_cast<int64_t>(t.ctas) * WARPS) {
        const int64_t token = u / t.splits;
        const int h_lo = static_cast<int>(u - token * t.splits) * t.per_unit;
        const int h_hi = min(t.heads, h_lo + t.per_unit);
        const T *in = static_cast<const T *>(t.in) + token * t.in_ts;
        const T *dy = static_cast<const T *>(t.dy) + token * t.dy_ts;
        T *out = static_cast<T *>(t.out) + token * t.out_ts;
        for (int h0 = h_lo + g; h0 - g < h_hi; h0 += G * BWD_HEADS) {
            Vec<T, V> x[BWD_HEADS][SL], d[BWD_HEADS][SL];
#pragma unroll
            for (int j = 0; j < BWD_HEADS; ++j)
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    x[j][i].clear();
                    d[j][i].clear();
                    if (h0 + j * G < h_hi && ln.has[i]) {
                        x[j][i].load(in + (h0 + j * G) * t.in_hs + ln.off[i]);
                        d[j][i].load(dy + (h0 + j * G) * t.dy_hs + ln.off[i]);
                    }
                }
            if (h0 - g == h_lo) ln.angles(a, token);
#pragma unroll
            for (int j = 0; j < BWD_HEADS; ++j) {
                float v[SL][V], dn[SL][V], ss = 0.0f, st = 0.0f;
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    x[j][i].get(v[i]);
                    d[j][i].get(dn[i]);
                }
                ln.template rotate<-1>(dn);
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    float f[V];
                    w[i].get(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        ss += v[i][e] * v[i][e];
                        st += v[i][e] * dn[i][e] * f[e];
                    }
                }
                ss = sum_head(ss, a.log_l);
                st = sum_head(st, a.log_l);
                const float inv = a.norm ? rsqrtf(ss * a.inv_d + a.eps) : 1.0f;
                const float m = a.norm ? inv * inv * st * a.inv_d : 0.0f;  // v m = e mean(e dn w)
                const bool mine = h0 + j * G < h_hi;
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    if (!mine || !ln.has[i]) continue;
                    float f[V];
                    w[i].get(f);
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        dw[i][e] += dn[i][e] * (v[i][e] * inv);
                        f[e] = inv * (dn[i][e] * f[e] - v[i][e] * m);
                    }
                    Vec<T, V> y;
                    y.put(f);
                    y.store(out + (h0 + j * G) * t.out_hs + ln.off[i]);
                }
            }
        }
    }
    if (!a.partials) return;
    // over the warp's groups, then over the CTA's warps
#pragma unroll
    for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            float v = dw[i][e];
            for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (g == 0 && ln.has[i]) red[warp][ln.off[i] + e] = v;
        }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.D) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v += red[k][threadIdx.x];
        __stcg(a.partials + static_cast<int64_t>(blockIdx.x) * a.D + threadIdx.x, v);
    }
}

// dw[j] = the sum of the CTAs' partials: 32 columns x 32 row lanes a CTA (y: q or k).
__global__ void __launch_bounds__(1024) k_heads_dw(const float *partials, float *dwq, float *dwk, int q_ctas, int k_ctas,
                                                   int D) {
    __shared__ float red[32][33];
    grid_dep_wait();
    grid_dep_launch_dependents();
    float *dst = blockIdx.y ? dwk : dwq;
    if (!dst) return;
    const int n = blockIdx.y ? k_ctas : q_ctas;
    const float *src = partials + (blockIdx.y ? static_cast<int64_t>(q_ctas) * D : 0);
    const int col = blockIdx.x * 32 + threadIdx.x;
    float v = 0.0f;
    if (col < D)
#pragma unroll 8
        for (int r = threadIdx.y; r < n; r += 32) v += __ldcg(src + static_cast<int64_t>(r) * D + col);
    red[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    if (threadIdx.y == 0 && col < D) {
        v = 0.0f;
#pragma unroll
        for (int r = 0; r < 32; ++r) v += red[r][threadIdx.x];
        dst[col] = v;
    }
}

// ------------------------------------------------------------------ host
// How vectors and lanes cover a head.
struct HeadShape {
    int V = 0;      // elements of a vector
    int ns = 0;     // 0 or 2 slots behind the rotation (halves)
    int log_l = 0;
};

HeadShape head_shape(int dtype, int D, int rot, bool inter) {
    HeadShape s;
    s.V = dtype == LORA_T_FP32 ? 4 : 8;
    if (!inter && (rot / 2) % s.V) s.V = 4;  // 8-byte vectors where the halves split a 16-byte one
    int need;
    if (inter) {
        need = (D / s.V + 1) / 2;
    } else {
        const int rest = (D - rot) / s.V;
        s.ns = rest > 0 ? 2 : 0;
        need = std::max(rot / 2 / s.V, (rest + 1) / 2);
    }
    while ((1 << s.log_l) < need) ++s.log_l;
    return s;
}

constexpr int BWD_CTAS = 2 * SMS;  // persistent: two CTAs of eight warps an SM

// CTAs of q and k in the backward, in proportion to their heads.
void split_ctas(int q_heads, int k_heads, int *q, int *k) {
    *q = q_heads ? std::max(1, static_cast<int>(static_cast<int64_t>(BWD_CTAS) * q_heads / (q_heads + k_heads))) : 0;
    *k = k_heads ? std::max(1, BWD_CTAS - *q) : 0;
}

size_t dw_bytes(int D) { return (static_cast<size_t>(BWD_CTAS) + 2) * D * sizeof(float); }

bool aligned(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A tensor's checks: 0 or a status.
lora_status_t check_heads(const lora_heads_t *t, int heads, int esize, int vec_bytes, int64_t M, int D) {
    if (!t->data || t->heads < 1 || t->heads > 4096 || t->heads != heads) return LORA_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 40;  // keeps every offset far inside 63 bits
    if (t->token_stride < 0 || t->head_stride < 0 || t->token_stride > most || t->head_stride > most)
        return LORA_ERR_INVALID_ARG;
    // no element twice: tokens outside heads, or heads outside tokens
    const bool tokens_outside = M == 1 || t->token_stride >= (heads - 1) * t->head_stride + D;
    const bool heads_outside = heads == 1 || t->head_stride >= (M - 1) * t->token_stride + D;
    if ((M > 1 && t->token_stride < D) || (heads > 1 && t->head_stride < D) || (!tokens_outside && !heads_outside))
        return LORA_ERR_INVALID_ARG;
    if (!aligned(t->data, 16) || (t->token_stride * esize) % vec_bytes || (t->head_stride * esize) % vec_bytes)
        return LORA_ERR_MISALIGNED;
    return LORA_OK;
}

// Heads a warp takes of one token: all of them, halved while the warps are too few to fill
// the device (eight an SM), down to one round of the warp's groups.
void fill_units(HeadTensor &t, int64_t M, int group_heads, int all_heads) {
    int per = t.heads;
    while (per > group_heads && M * ((all_heads + per - 1) / per) < int64_t(SMS) * 8) per = (per + 1) / 2;
    per = std::min(t.heads, (per + group_heads - 1) / group_heads * group_heads);
    t.per_unit = per;
    t.splits = (t.heads + per - 1) / per;
    t.units = M * t.splits;
}

template <class T, int V, bool INTER, int NS>
cudaError_t launch(const HeadArgs &a, bool bwd, cudaStream_t st) {
    if (bwd)
        return lora_host::launch_pdl(k_heads_bwd<T, V, INTER, NS>, dim3(a.t[0].ctas + a.t[1].ctas), dim3(WARPS * 32), 0,
                                     st, a);
    const int64_t ctas = (a.t[0].units + a.t[1].units + WARPS - 1) / WARPS;
    if (ctas > INT32_MAX) return cudaErrorInvalidValue;
    return lora_host::launch_pdl(k_heads_fwd<T, V, INTER, NS>, dim3(static_cast<unsigned>(ctas)), dim3(WARPS * 32), 0,
                                 st, a);
}

template <class T>
cudaError_t launch_type(const HeadArgs &a, const HeadShape &s, bool inter, bool bwd, cudaStream_t st) {
    constexpr int FULL = 16 / sizeof(T);
    if (inter) return launch<T, FULL, true, 0>(a, bwd, st);
    if (s.V == FULL) return s.ns ? launch<T, FULL, false, 2>(a, bwd, st) : launch<T, FULL, false, 0>(a, bwd, st);
    return s.ns ? launch<T, 4, false, 2>(a, bwd, st) : launch<T, 4, false, 0>(a, bwd, st);
}

// Both directions: dy null for the forward.
lora_status_t run(int dtype, const lora_heads_t *const in[2], const lora_heads_t *const dy[2],
                  const lora_heads_t *const out[2], const void *const weight[2], const float *cos, const float *sin,
                  const int64_t *positions, int64_t n_pos, float *const dw[2], int64_t M, int D, int rot,
                  int interleaved, int norm, float eps, bool bwd, void *ws, size_t ws_bytes, void *stream) {
    if (dtype < LORA_T_BF16 || dtype > LORA_T_FP32) return LORA_ERR_INVALID_ARG;
    if (M < 1 || M > (int64_t(1) << 30) || D < 8 || D > 256 || D % 8 || rot < 0 || rot > D || rot % 8)
        return LORA_ERR_INVALID_ARG;
    if (!std::isfinite(eps) || eps < 0) return LORA_ERR_INVALID_ARG;
    if (!in[0] && !in[1]) return LORA_ERR_INVALID_ARG;
    if (rot > 0 && (!cos || !sin || !positions || n_pos < 1 || n_pos > (int64_t(1) << 40))) return LORA_ERR_INVALID_ARG;
    const HeadShape shape = head_shape(dtype, D, rot, interleaved != 0);
    const int esize = dtype == LORA_T_FP32 ? 4 : 2, vb = shape.V * esize;
    HeadArgs a;
    std::memset(&a, 0, sizeof(a));
    bool want_dw = false;
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) {
            if (out[i] || dy[i] || dw[i]) return LORA_ERR_INVALID_ARG;
            continue;
        }
        if (!out[i] || (bwd && !dy[i])) return LORA_ERR_INVALID_ARG;
        for (const lora_heads_t *t : {in[i], out[i], bwd ? dy[i] : in[i]}) {
            const lora_status_t s = check_heads(t, in[i]->heads, esize, vb, M, D);
            if (s != LORA_OK) return s;
        }
        if (weight[i] && !aligned(weight[i], 16)) return LORA_ERR_MISALIGNED;
        if (dw[i] && !aligned(dw[i], 16)) return LORA_ERR_MISALIGNED;
        want_dw |= dw[i] != nullptr;
    }
    if (rot > 0 && (!aligned(cos, 16) || !aligned(sin, 16) || !aligned(positions, 8))) return LORA_ERR_MISALIGNED;
    if (want_dw) {
        if (!ws || ws_bytes < dw_bytes(D)) return LORA_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return LORA_ERR_MISALIGNED;
    }
    if (!lora_host::device_supported()) return LORA_ERR_UNSUPPORTED;
    a.cos = cos;
    a.sin = sin;
    a.pos = positions;
    a.n_pos = n_pos;
    a.D = D;
    a.rot = rot;
    a.log_l = shape.log_l;
    a.norm = norm != 0;
    a.eps = eps;
    a.inv_d = 1.0f / static_cast<float>(D);
    a.partials = want_dw ? static_cast<float *>(ws) : nullptr;
    const int group_heads = 32 >> shape.log_l;
    const int all = (in[0] ? in[0]->heads : 0) + (in[1] ? in[1]->heads : 0);
    split_ctas(in[0] ? in[0]->heads : 0, in[1] ? in[1]->heads : 0, &a.t[0].ctas, &a.t[1].ctas);
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        HeadTensor &t = a.t[i];
        t.in = in[i]->data;
        t.in_ts = in[i]->token_stride;
        t.in_hs = in[i]->head_stride;
        t.out = out[i]->data;
        t.out_ts = out[i]->token_stride;
        t.out_hs = out[i]->head_stride;
        if (bwd) {
            t.dy = dy[i]->data;
            t.dy_ts = dy[i]->token_stride;
            t.dy_hs = dy[i]->head_stride;
        }
        t.weight = weight[i];
        t.heads = in[i]->heads;
        fill_units(t, M, group_heads, all);
        t.ctas = static_cast<int>(std::min<int64_t>(t.ctas, (t.units + WARPS - 1) / WARPS));
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case LORA_T_BF16: e = launch_type<__nv_bfloat16>(a, shape, interleaved != 0, bwd, st); break;
        case LORA_T_FP16: e = launch_type<__half>(a, shape, interleaved != 0, bwd, st); break;
        default: e = launch_type<float>(a, shape, interleaved != 0, bwd, st); break;
    }
    if (e == cudaSuccess && want_dw)
        e = lora_host::launch_pdl(k_heads_dw, dim3((D + 31) / 32, 2), dim3(32, 32), 0, st, a.partials, dw[0], dw[1],
                                  a.t[0].ctas, a.t[1].ctas, D);
    return e == cudaSuccess ? LORA_OK : LORA_ERR_CUDA;
}

}  // namespace

extern "C" {

lora_status_t lora_qk_norm_rope_fwd(int dtype, const lora_heads_t *q, const lora_heads_t *k, const void *q_weight,
                                    const void *k_weight, const float *cos, const float *sin, const int64_t *positions,
                                    int64_t n_pos, const lora_heads_t *q_out, const lora_heads_t *k_out, int64_t M,
                                    int D, int rot, int interleaved, int norm, float eps, void *stream) {
    const lora_heads_t *in[2] = {q, k}, *none[2] = {nullptr, nullptr}, *out[2] = {q_out, k_out};
    const void *w[2] = {q_weight, k_weight};
    float *dw[2] = {nullptr, nullptr};
    return run(dtype, in, none, out, w, cos, sin, positions, n_pos, dw, M, D, rot, interleaved, norm, eps, false,
               nullptr, 0, stream);
}

lora_status_t lora_qk_norm_rope_bwd(int dtype, const lora_heads_t *dq_out, const lora_heads_t *dk_out,
                                    const lora_heads_t *q, const lora_heads_t *k, const void *q_weight,
                                    const void *k_weight, const float *cos, const float *sin, const int64_t *positions,
                                    int64_t n_pos, const lora_heads_t *dq, const lora_heads_t *dk, float *dq_weight,
                                    float *dk_weight, int64_t M, int D, int rot, int interleaved, int norm, float eps,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    const lora_heads_t *in[2] = {q, k}, *dy[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
    const void *w[2] = {q_weight, k_weight};
    float *dw[2] = {dq_weight, dk_weight};
    return run(dtype, in, dy, out, w, cos, sin, positions, n_pos, dw, M, D, rot, interleaved, norm, eps, true, workspace,
               workspace_bytes, stream);
}

size_t lora_qk_norm_rope_workspace_size(int64_t M, int heads, int D) {
    if (M < 1 || heads < 1 || heads > 8192 || D < 8 || D > 256 || D % 8) return 0;
    return (dw_bytes(D) + 255) & ~size_t(255);
}

}  // extern "C"
