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
// flight (forward in registers; the backward, whose registers the two inputs and the weight
// gradients fill, through shared memory by asynchronous copies, each lane its own: 8192 tokens of
// 40 heads of 128 in bf16 61 -> 55 us, 252 MB at 4.6 TB/s); the token's cos and sin stay in
// registers over its heads, so the fp32 tables, as wide as a head itself, are read once a
// token instead of once a head.  The backward forms sum v^2 and sum v dn w in the same
// shuffles.
//
// The weight gradients are summed per lane over a CTA's whole share in fp32, over the CTA
// in shared memory, and over the CTAs by a second kernel, each in a fixed order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/lora_linear.h"
#include "block.h"
#include "ptx.cuh"

namespace {

using namespace lora;

constexpr int WARPS = 8;
// Heads of a group at a time.  Forward: two, at three CTAs an SM (16384 tokens of 40 heads of
// 128 in bf16: 61 us; three heads at three CTAs 69, two at four 68, four at two 72, registers
// spilling or loads too few).  Backward, whose loads run ahead through shared memory: one, three
// steps of it, where a vector holds 8 elements (8192 tokens: 55 us; with loads to registers
// 61); two, two steps, where it holds 4.
constexpr int FWD_HEADS = 2;
__host__ __device__ constexpr int bwd_heads(int V) { return V == 4 ? 2 : 1; }
__host__ __device__ constexpr int bwd_stages(int V) { return V == 4 ? 2 : 3; }
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

// ------------------------------------------------------------------ pairs of fp32
// Arithmetic runs on pairs of neighbouring elements (the packed fp32 instructions), which
// halves the instructions of a kernel that issue would bound otherwise.
typedef uint64_t f2;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(f2 v, float &lo, float &hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 swap2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return pack2(hi, lo);
}
__device__ __forceinline__ float hsum2(f2 v) {
    float lo, hi;
    unpack2(v, lo, hi);
    return lo + hi;
}

// ------------------------------------------------------------------ element types
// A 32-bit word of two 16-bit elements to a pair and back (one rounding).
template <class T>
struct Elem;
template <>
struct Elem<__nv_bfloat16> {
    static __device__ f2 get(uint32_t w) { return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
    static __device__ uint32_t put(f2 v) {
        float lo, hi;
        unpack2(v, lo, hi);
        const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&b);
    }
};
template <>
struct Elem<__half> {
    static __device__ f2 get(uint32_t w) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return pack2(f.x, f.y);
    }
    static __device__ uint32_t put(f2 v) {
        float lo, hi;
        unpack2(v, lo, hi);
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// A vector of V elements as loaded: V * sizeof(T) is 16 or 8 bytes.
template <class T, int V>
struct Vec {
    static constexpr int W = V * sizeof(T) / 4;  // 32-bit words
    uint32_t w[W];
    __device__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ void load(const T *p) {  // read once: past L1
        if constexpr (W == 4)
            asm volatile("ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                         : "l"(p));
        else
            asm volatile("ld.global.L1::no_allocate.L2::256B.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    }
    __device__ void load_kept(const T *p) {
        if constexpr (W == 4) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
            w[0] = v.x, w[1] = v.y;
        }
    }
    __device__ void load_shared(const uint8_t *p) {
        if constexpr (W == 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x, w[1] = v.y;
        }
    }
    __device__ void store(T *p) const {
        // written once: streaming stores keep them from evicting what is still to be read
        // (16384 tokens of 40 heads of 128 in bf16: 65.7 -> 62.5 us)
        if constexpr (W == 4) __stcs(reinterpret_cast<uint4 *>(p), make_uint4(w[0], w[1], w[2], w[3]));
        else __stcs(reinterpret_cast<uint2 *>(p), make_uint2(w[0], w[1]));
    }
    __device__ f2 get(int i) const {  // elements 2 i, 2 i + 1
        if constexpr (sizeof(T) == 4) return pack2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        else return Elem<T>::get(w[i]);
    }
    __device__ void put(int i, f2 v) {
        if constexpr (sizeof(T) == 4) {
            float lo, hi;
            unpack2(v, lo, hi);
            w[2 * i] = __float_as_uint(lo);
            w[2 * i + 1] = __float_as_uint(hi);
        } else {
            w[i] = Elem<T>::put(v);
        }
    }
};

// ------------------------------------------------------------------ a lane's share of a head
// Slots of V elements.  Halves: slot 0 is vector p of the first rot/2 dimensions, slot 1
// its partner, slots 2.. (NS of them) the dimensions behind the rotation.  INTER: two slots
// over all of D, partners next to each other.  So in either layout a rotated pair of
// elements is  own * c + partner * (+-s)  with the partner in the other slot, or swapped.
template <int V, bool INTER, int NS>
struct Lane {
    static constexpr int SLOTS = INTER ? 2 : 2 + NS;
    static constexpr int P = V / 2;  // pairs of a slot
    int off[SLOTS];   // first dimension
    bool has[SLOTS];

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

    // cos and sin of a token's position: halves, of the vector's dimensions (they serve slots 0
    // and 1); INTER, of each slot's pairs, an angle twice.  Without a rotation 1 and 0; a
    // position outside the table reads nothing and gives NaN.
    static constexpr int TURNS = INTER ? 2 : 1;
    static constexpr int FLOATS = INTER ? V / 2 : V;   // angles of a turn
    __device__ bool turns(int rot, int i) const { return rot > 0 && has[i] && (!INTER || off[i] < rot); }
    __device__ int first_angle(int i) const { return INTER ? off[i] / 2 : off[0]; }

    // from the turns' angles, cos and sin: read(i, e, sine) gives angles e, e + 1 of turn i
    template <class Read>
    __device__ void angles(int rot, float bad, f2 (&c)[TURNS][P], f2 (&s)[TURNS][P], Read read) const {
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
#pragma unroll
            for (int e = 0; e < P; ++e) {
                c[i][e] = pack2(1.0f, 1.0f);
                s[i][e] = 0;
            }
            if (!turns(rot, i)) continue;
#pragma unroll
            for (int e = 0; e < FLOATS; e += 2) {
                const float2 fc = read(i, e, 0), fs = read(i, e, 1);
                if constexpr (INTER) {  // angle e belongs to the elements 2 e, 2 e + 1
                    c[i][e] = pack2(fc.x + bad, fc.x + bad);
                    c[i][e + 1] = pack2(fc.y + bad, fc.y + bad);
                    s[i][e] = pack2(fs.x, fs.x);
                    s[i][e + 1] = pack2(fs.y, fs.y);
                } else {
                    c[i][e / 2] = pack2(fc.x + bad, fc.y + bad);
                    s[i][e / 2] = pack2(fs.x, fs.y);
                }
            }
        }
    }
    __device__ void angles(const HeadArgs &a, int64_t pos, f2 (&c)[TURNS][P], f2 (&s)[TURNS][P]) const {
        const bool ok = pos >= 0 && pos < a.n_pos;
        const int64_t at = a.rot && ok ? pos * (a.rot / 2) : 0;
        const float *cr = a.cos + at, *sr = a.sin + at;
        angles(a.rot, ok ? 0.0f : __int_as_float(0x7fc00000), c, s, [&](int i, int e, int sine) {
            return __ldg(reinterpret_cast<const float2 *>((sine ? sr : cr) + first_angle(i) + e));
        });
    }
    static __device__ f2 partner(const f2 (&v)[SLOTS][P], int i, int e) { return INTER ? swap2(v[i][e]) : v[1 - i][e]; }
};

// v rotated back by the angles, in place:  v_a c + v_b s,  v_b c - v_a s.  `turned`: INTER, the
// slots inside the rotation.
template <int V, bool INTER, int NS>
__device__ __forceinline__ void rotate_back(f2 (&v)[Lane<V, INTER, NS>::SLOTS][V / 2],
                                            const f2 (&c)[INTER ? 2 : 1][V / 2], const f2 (&s)[INTER ? 2 : 1][V / 2],
                                            const bool (&turned)[2]) {
#pragma unroll
    for (int e = 0; e < V / 2; ++e) {
        if constexpr (INTER) {
            const f2 sign = pack2(1.0f, -1.0f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (turned[i]) v[i][e] = fma2(swap2(v[i][e]), mul2(s[i][e], sign), mul2(v[i][e], c[i][e]));
        } else {
            const f2 a = v[0][e], b = v[1][e];
            v[0][e] = fma2(b, s[0][e], mul2(a, c[0][e]));
            v[1][e] = fma2(mul2(a, s[0][e]), pack2(-1.0f, -1.0f), mul2(b, c[0][e]));
        }
    }
}

// Each of N values summed over the L lanes of a head (all 32 lanes take part); together, so
// that their shuffles overlap.
template <int N>
__device__ __forceinline__ void sum_head(float (&v)[N], int log_l) {
#pragma unroll 1
    for (int m = 1; m < (1 << log_l); m <<= 1) {
        float o[N];
#pragma unroll
        for (int n = 0; n < N; ++n) o[n] = __shfl_xor_sync(0xffffffffu, v[n], m);
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += o[n];
    }
}

// The weight of a lane's slots as loaded (ones without a weight).
template <class T, int V, class LaneT>
__device__ __forceinline__ void load_weight(const HeadTensor &t, const LaneT &ln, Vec<T, V> (&w)[LaneT::SLOTS]) {
#pragma unroll
    for (int i = 0; i < LaneT::SLOTS; ++i) {
        w[i].clear();
        if (t.weight && ln.has[i]) w[i].load_kept(static_cast<const T *>(t.weight) + ln.off[i]);
#pragma unroll
        for (int e = 0; e < V / 2; ++e)
            if (!t.weight) w[i].put(e, pack2(1.0f, 1.0f));
    }
}

// Unit u of a tensor: its token and the first of its heads.
__device__ __forceinline__ int64_t unit_token(const HeadTensor &t, int64_t u, int &h_lo) {
    if (t.splits == 1) {
        h_lo = 0;
        return u;
    }
    const int64_t token = u / t.splits;
    h_lo = static_cast<int>(u - token * t.splits) * t.per_unit;
    return token;
}

__device__ __forceinline__ int64_t position(const HeadArgs &a, int64_t token) { return a.rot ? __ldg(a.pos + token) : 0; }

// ------------------------------------------------------------------ forward
// The weight goes into the rotation's coefficients once a token:
//   y = i (own * (w c) + partner * (w_partner q))
template <class T, int V, bool INTER, int NS>
__global__ void __launch_bounds__(WARPS * 32, NS ? 2 : 3) k_heads_fwd(const __grid_constant__ HeadArgs a) {
    using LaneT = Lane<V, INTER, NS>;
    constexpr int SL = LaneT::SLOTS, P = V / 2;
    grid_dep_wait();
    grid_dep_launch_dependents();
    const int lane = threadIdx.x & 31;
    int64_t u = static_cast<int64_t>(blockIdx.x) * WARPS + (threadIdx.x >> 5);
    const int which = u >= a.t[0].units;
    if (which) u -= a.t[0].units;
    const HeadTensor &t = a.t[which];
    if (u >= t.units) return;
    int h_lo;
    const int64_t token = unit_token(t, u, h_lo);
    const int64_t pos = position(a, token);
    const int h_hi = min(t.heads, h_lo + t.per_unit);
    const int L = 1 << a.log_l, G = 32 >> a.log_l, g = lane >> a.log_l;
    LaneT ln;
    ln.place(a.D, a.rot, lane & (L - 1), L);
    const T *in = static_cast<const T *>(t.in) + token * t.in_ts + (h_lo + g) * t.in_hs;
    T *out = static_cast<T *>(t.out) + token * t.out_ts + (h_lo + g) * t.out_hs;
    const int64_t in_step = G * t.in_hs, out_step = G * t.out_hs;
    f2 c[2][P], q[2][P], w[SL][P];
    // INTER: a slot behind the rotation has partners that it must not see, not even times zero (an
    // infinity times zero is NaN)
    bool turned[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) turned[i] = !INTER || ln.turns(a.rot, i);
    for (int h0 = h_lo; h0 < h_hi; h0 += G * FWD_HEADS) {
        Vec<T, V> x[FWD_HEADS][SL];
#pragma unroll
        for (int j = 0; j < FWD_HEADS; ++j) {
            const bool mine = h0 + g + j * G < h_hi;
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                x[j][i].clear();
                if (mine && ln.has[i]) x[j][i].load(in + ln.off[i]);
            }
            in += in_step;
        }
        if (h0 == h_lo) {  // behind the first heads' loads
            f2 co[LaneT::TURNS][P], si[LaneT::TURNS][P];
            ln.angles(a, pos, co, si);
            Vec<T, V> raw[SL];
            load_weight<T, V>(t, ln, raw);
#pragma unroll
            for (int i = 0; i < SL; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) w[i][e] = raw[i].get(e);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const f2 sign = INTER ? pack2(-1.0f, 1.0f) : i ? pack2(1.0f, 1.0f) : pack2(-1.0f, -1.0f);
                    c[i][e] = mul2(co[INTER ? i : 0][e], w[i][e]);
                    q[i][e] = mul2(mul2(si[INTER ? i : 0][e], sign), LaneT::partner(w, i, e));
                }
        }
        float ss[FWD_HEADS];
#pragma unroll
        for (int j = 0; j < FWD_HEADS; ++j) {
            f2 sq = 0;
#pragma unroll
            for (int i = 0; i < SL; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    const f2 v = x[j][i].get(e);
                    sq = fma2(v, v, sq);
                }
            ss[j] = hsum2(sq);
        }
        sum_head(ss, a.log_l);
#pragma unroll
        for (int j = 0; j < FWD_HEADS; ++j) {
            f2 v[SL][P];
#pragma unroll
            for (int i = 0; i < SL; ++i)
#pragma unroll
                for (int e = 0; e < P; ++e) v[i][e] = x[j][i].get(e);
            const float inv = a.norm ? rsqrtf(ss[j] * a.inv_d + a.eps) : 1.0f;
            const f2 inv2 = pack2(inv, inv);
            const bool mine = h0 + g + j * G < h_hi;
#pragma unroll
            for (int i = 0; i < SL; ++i) {
                Vec<T, V> y;
#pragma unroll
                for (int e = 0; e < P; ++e) {
                    f2 r = mul2(v[i][e], i < 2 ? c[i < 2 ? i : 0][e] : w[i][e]);
                    if (i < 2 && turned[i < 2 ? i : 0]) r = fma2(LaneT::partner(v, i, e), q[i < 2 ? i : 0][e], r);
                    y.put(e, mul2(r, inv2));
                }
                if (mine && ln.has[i]) y.store(out + ln.off[i]);
            }
            out += out_step;
        }
    }
}

// ------------------------------------------------------------------ backward
// Each lane copies its own part of the heads ahead of their use to shared memory (and reads it back
// itself: no barrier), a ring of BWD_STAGES steps, and with a unit's first step its angles.
template <class T, int V, int SL>
struct BwdRing {
    static constexpr int VEC = V * sizeof(T);            // bytes of a vector
    static constexpr int HEADS = bwd_heads(V), STAGES = bwd_stages(V);
    static constexpr int HEAD = 2 * SL * VEC * 32;        // a warp's x and dy of a head a group
    static constexpr int STEP = HEADS * HEAD;
    static constexpr int TURN = 2 * V * 4 * 32;           // and cos and sin of a unit
    static constexpr int WARP = STAGES * (STEP + TURN);
    static constexpr int BYTES = WARPS * WARP;
};
template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global.L2::256B [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

template <class T, int V, bool INTER, int NS>
__global__ void __launch_bounds__(WARPS * 32, NS ? 1 : 2) k_heads_bwd(const __grid_constant__ HeadArgs a) {
    using LaneT = Lane<V, INTER, NS>;
    constexpr int SL = LaneT::SLOTS, P = V / 2;
    using R = BwdRing<T, V, SL>;
    constexpr int S = R::STAGES, H = R::HEADS;
    extern __shared__ __align__(16) uint8_t ring_all[];
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
    const int64_t in_step = G * t.in_hs, dy_step = G * t.dy_hs, out_step = G * t.out_hs;
    bool turned[2];  // as in the forward
#pragma unroll
    for (int i = 0; i < 2; ++i) turned[i] = !INTER || ln.turns(a.rot, i);
    Vec<T, V> w[SL];  // as loaded: half the registers
    f2 dw[SL][P];
    load_weight<T, V>(t, ln, w);
#pragma unroll
    for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) dw[i][e] = 0;
    uint8_t *ring = ring_all + warp * R::WARP + lane * R::VEC;         // slots of a lane: 32 vectors apart
    uint8_t *turn = ring_all + warp * R::WARP + S * R::STEP;            // [S][cos, sin][lane][V]
    // this warp's units: u0, u0 + stride, ..., as (token, split) without a division each
    const int stride = t.ctas * WARPS, u0 = cta * WARPS + warp;
    const int d_token = stride / t.splits, d_split = stride - d_token * t.splits;
    struct Unit {
        int64_t token;
        int split;
    };
    const int64_t M = t.units / t.splits;
    const Unit first{u0 / t.splits, u0 % t.splits};
    auto step = [&](Unit &v) {
        v.token += d_token;
        v.split += d_split;
        if (v.split >= t.splits) {
            v.split -= t.splits;
            ++v.token;
        }
    };

    // the copies' cursor: a step is one head a group of lanes
    Unit fu = first;
    int64_t f_pos = 0, f_next = fu.token < M ? position(a, fu.token) : 0;  // a position is loaded a unit ahead
    int f_lo = 0, f_h = 0, f_hi = 0, f_slot = 0, f_turn = 0;
    const T *f_in = nullptr, *f_dy = nullptr;
    auto enter = [&]() {
        const int64_t token = fu.token;
        if (token >= M) return;
        f_lo = fu.split * t.per_unit;
        f_h = f_lo;
        f_hi = min(t.heads, f_lo + t.per_unit);
        f_in = static_cast<const T *>(t.in) + token * t.in_ts + (f_lo + g) * t.in_hs;
        f_dy = static_cast<const T *>(t.dy) + token * t.dy_ts + (f_lo + g) * t.dy_hs;
        f_pos = f_next;
        Unit next = fu;
        step(next);
        if (next.token < M) f_next = position(a, next.token);
    };
    auto fetch = [&]() {
        if (fu.token < M) {
            const bool first_step = f_h == f_lo;
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const uint32_t dst = smem_u32(ring + f_slot * R::STEP + j * R::HEAD);
                if (f_h + g < f_hi)
#pragma unroll
                    for (int i = 0; i < SL; ++i)
                        if (ln.has[i]) {
                            copy_async<R::VEC>(dst + 2 * i * 32 * R::VEC, f_in + ln.off[i]);
                            copy_async<R::VEC>(dst + (2 * i + 1) * 32 * R::VEC, f_dy + ln.off[i]);
                        }
                f_h += G;
                f_in += in_step;
                f_dy += dy_step;
            }
            if (first_step && a.rot) {
                const bool ok = f_pos >= 0 && f_pos < a.n_pos;
                float *to = reinterpret_cast<float *>(turn + f_turn * R::TURN) + lane * V;
#pragma unroll
                for (int i = 0; i < LaneT::TURNS; ++i) {
                    if (!ln.turns(a.rot, i)) continue;
                    constexpr int F = LaneT::FLOATS, B = F % 4 ? 8 : 16;
                    const int64_t at = ok ? f_pos * (a.rot / 2) + ln.first_angle(i) : 0;
#pragma unroll
                    for (int e = 0; e < F; e += B / 4) {
                        if (ok) {
                            copy_async<B>(smem_u32(to + i * F + e), a.cos + at + e);
                            copy_async<B>(smem_u32(to + 32 * V + i * F + e), a.sin + at + e);
                        } else {
#pragma unroll
                            for (int k = 0; k < B / 4; ++k) to[i * F + e + k] = __int_as_float(0x7fc00000);
                        }
                    }
                }
                f_turn = f_turn + 1 == S ? 0 : f_turn + 1;
            }
            f_slot = f_slot + 1 == S ? 0 : f_slot + 1;
            if (f_h >= f_hi) {
                step(fu);
                enter();
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    enter();
#pragma unroll
    for (int k = 0; k < S - 1; ++k) fetch();

    int slot = 0, used_turn = 0;
    for (Unit u = first; u.token < M; step(u)) {
        const int64_t token = u.token;
        const int h_lo = u.split * t.per_unit, h_hi = min(t.heads, h_lo + t.per_unit);
        T *out = static_cast<T *>(t.out) + token * t.out_ts + (h_lo + g) * t.out_hs;
        f2 c[LaneT::TURNS][P], s[LaneT::TURNS][P];
        for (int h0 = h_lo; h0 < h_hi; h0 += G * H) {
            asm volatile("cp.async.wait_group %0;" ::"n"(S - 2) : "memory");
            Vec<T, V> x[H][SL], d[H][SL];
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const uint8_t *from = ring + slot * R::STEP + j * R::HEAD;
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    x[j][i].clear();
                    d[j][i].clear();
                    if (h0 + g + j * G < h_hi && ln.has[i]) {
                        x[j][i].load_shared(from + 2 * i * 32 * R::VEC);
                        d[j][i].load_shared(from + (2 * i + 1) * 32 * R::VEC);
                    }
                }
            }
            slot = slot + 1 == S ? 0 : slot + 1;
            if (h0 == h_lo) {
                const float *cs = reinterpret_cast<const float *>(turn + used_turn * R::TURN) + lane * V;
                ln.angles(a.rot, 0.0f, c, s, [&](int i, int e, int sine) {
                    return *reinterpret_cast<const float2 *>(cs + sine * 32 * V + i * LaneT::FLOATS + e);
                });
                if (a.rot) used_turn = used_turn + 1 == S ? 0 : used_turn + 1;
            }
            fetch();  // into the slots of the step before, which has been read
            f2 dn[H][SL][P];         // the gradient rotated back
            float sums[2 * H];       // of v^2 and of v dn w
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f2 sq = 0, st = 0;
#pragma unroll
                for (int i = 0; i < SL; ++i)
#pragma unroll
                    for (int e = 0; e < P; ++e) dn[j][i][e] = d[j][i].get(e);
                rotate_back<V, INTER, NS>(dn[j], c, s, turned);
#pragma unroll
                for (int i = 0; i < SL; ++i)
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const f2 v = x[j][i].get(e);
                        sq = fma2(v, v, sq);
                        st = fma2(v, mul2(dn[j][i][e], w[i].get(e)), st);
                    }
                sums[2 * j] = hsum2(sq);
                sums[2 * j + 1] = hsum2(st);
            }
            sum_head(sums, a.log_l);
#pragma unroll
            for (int j = 0; j < H; ++j) {
                const float inv = a.norm ? rsqrtf(sums[2 * j] * a.inv_d + a.eps) : 1.0f;
                // i (dn w - v i^2 mean(v dn w)) = i dn w + v k
                const float k = a.norm ? -(inv * inv) * (sums[2 * j + 1] * a.inv_d) * inv : 0.0f;
                const f2 inv2 = pack2(inv, inv), k2 = pack2(k, k);
                const bool mine = h0 + g + j * G < h_hi;
#pragma unroll
                for (int i = 0; i < SL; ++i) {
                    Vec<T, V> y;
                    if (!mine || !ln.has[i]) continue;
#pragma unroll
                    for (int e = 0; e < P; ++e) {
                        const f2 v = x[j][i].get(e), di = mul2(dn[j][i][e], inv2);
                        dw[i][e] = fma2(di, v, dw[i][e]);
                        y.put(e, fma2(v, k2, mul2(di, w[i].get(e))));
                    }
                    y.store(out + ln.off[i]);
                }
                out += out_step;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (!a.partials) return;
    // over the warp's groups, then over the CTA's warps
#pragma unroll
    for (int i = 0; i < SL; ++i)
#pragma unroll
        for (int e = 0; e < P; ++e) {
            float v[2];
            unpack2(dw[i][e], v[0], v[1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                for (int o = L; o < 32; o <<= 1) v[h] += __shfl_xor_sync(0xffffffffu, v[h], o);
                if (g == 0 && ln.has[i]) red[warp][ln.off[i] + 2 * e + h] = v[h];
            }
        }
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < a.D) {
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < WARPS; ++k) v += red[k][threadIdx.x];
        __stcg(a.partials + static_cast<int64_t>(blockIdx.x) * a.D + threadIdx.x, v);
    }
}

// dw[j] = the sum of the CTAs' partials, rounded once to T: 32 columns x 32 row lanes a CTA (y:
// q or k).
template <class T>
__global__ void __launch_bounds__(1024) k_heads_dw(const float *partials, T *dwq, T *dwk, int q_ctas, int k_ctas, int D) {
    __shared__ float red[32][33];
    grid_dep_wait();
    grid_dep_launch_dependents();
    T *dst = blockIdx.y ? dwk : dwq;
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
        dst[col] = T(v);
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

// The strides of a tensor as the kernels take them: one over a single token or head leads nowhere,
// whatever it is.
int64_t token_stride(const lora_heads_t &t, int64_t M) { return M > 1 ? t.token_stride : 0; }
int64_t head_stride(const lora_heads_t &t) { return t.heads > 1 ? t.head_stride : 0; }

// A tensor's checks: 0 or a status.
lora_status_t check_heads(const lora_heads_t *t, int heads, int esize, int vec_bytes, int64_t M, int D) {
    if (!t->data || t->heads < 1 || t->heads > 4096 || t->heads != heads) return LORA_ERR_INVALID_ARG;
    const int64_t most = int64_t(1) << 40, ts = token_stride(*t, M), hs = head_stride(*t);
    if (ts < 0 || hs < 0 || ts > most || hs > most) return LORA_ERR_INVALID_ARG;
    // no element twice: tokens outside heads, or heads outside tokens
    const __int128 over_tokens = __int128(M - 1) * ts + D, over_heads = __int128(heads - 1) * hs + D;
    if (over_tokens + over_heads > (__int128(1) << 58)) return LORA_ERR_INVALID_ARG;  // bytes in 63 bits
    const bool tokens_outside = M == 1 || ts >= over_heads;
    const bool heads_outside = heads == 1 || hs >= over_tokens;
    if ((M > 1 && ts < D) || (heads > 1 && hs < D) || (!tokens_outside && !heads_outside)) return LORA_ERR_INVALID_ARG;
    if (!aligned(t->data, 16) || (ts * esize) % vec_bytes || (hs * esize) % vec_bytes) return LORA_ERR_MISALIGNED;
    return LORA_OK;
}

// Heads a warp takes of one token: all of them, halved while the tensor has fewer than `want`
// units, down to one batch of the warp's groups; then, while the units are too few to fill
// the device (eight an SM), down to one head a group.
void fill_units(HeadTensor &t, int64_t M, int group_heads, int batch, int64_t want) {
    int per = t.heads;
    auto units = [&] { return M * ((t.heads + per - 1) / per); };
    while (per > group_heads * batch && units() < want) per = (per + 1) / 2;
    while (per > group_heads && units() < int64_t(SMS) * 8) per = (per + 1) / 2;
    per = std::min(t.heads, (per + group_heads - 1) / group_heads * group_heads);
    t.per_unit = per;
    t.splits = (t.heads + per - 1) / per;
    t.units = M * t.splits;
}

// A kernel's limit of dynamic shared memory raised, once a device.
template <auto *KERNEL>
cudaError_t allow_shared(int bytes) {
    static std::mutex mu;
    static bool done[64] = {};
    int d = 0;
    const cudaError_t e = cudaGetDevice(&d);
    if (e != cudaSuccess || d < 0 || d >= 64) return cudaErrorInvalidDevice;
    const std::lock_guard<std::mutex> lk(mu);
    if (done[d]) return cudaSuccess;
    const cudaError_t s = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    done[d] = s == cudaSuccess;
    return s;
}

template <class T, int V, bool INTER, int NS>
cudaError_t launch(const HeadArgs &a, bool bwd, cudaStream_t st) {
    if (bwd) {
        constexpr int BYTES = BwdRing<T, V, Lane<V, INTER, NS>::SLOTS>::BYTES;
        const cudaError_t e = allow_shared<k_heads_bwd<T, V, INTER, NS>>(BYTES);
        if (e != cudaSuccess) return e;
        return lora_host::launch_pdl(k_heads_bwd<T, V, INTER, NS>, dim3(a.t[0].ctas + a.t[1].ctas), dim3(WARPS * 32), BYTES,
                                     st, a);
    }
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

template <class T>
cudaError_t launch_dw(const HeadArgs &a, void *const dw[2], cudaStream_t st) {
    return lora_host::launch_pdl(k_heads_dw<T>, dim3((a.D + 31) / 32, 2), dim3(32, 32), 0, st,
                                 static_cast<const float *>(a.partials), static_cast<T *>(dw[0]), static_cast<T *>(dw[1]),
                                 a.t[0].ctas, a.t[1].ctas, a.D);
}

// Both directions: dy null for the forward.
lora_status_t run(int dtype, const lora_heads_t *const in[2], const lora_heads_t *const dy[2],
                  const lora_heads_t *const out[2], const void *const weight[2], const float *cos, const float *sin,
                  const int64_t *positions, int64_t n_pos, void *const dw[2], bool dw_typed, int64_t M, int D, int rot,
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
    split_ctas(in[0] ? in[0]->heads : 0, in[1] ? in[1]->heads : 0, &a.t[0].ctas, &a.t[1].ctas);
    for (int i = 0; i < 2; ++i) {
        if (!in[i]) continue;
        HeadTensor &t = a.t[i];
        t.in = in[i]->data;
        t.in_ts = token_stride(*in[i], M);
        t.in_hs = head_stride(*in[i]);
        t.out = out[i]->data;
        t.out_ts = token_stride(*out[i], M);
        t.out_hs = head_stride(*out[i]);
        if (bwd) {
            t.dy = dy[i]->data;
            t.dy_ts = token_stride(*dy[i], M);
            t.dy_hs = head_stride(*dy[i]);
        }
        t.weight = weight[i];
        t.heads = in[i]->heads;
        // backward: eight units or more for each of the tensor's resident warps, so that the last
        // round, which not all of them have, is a small part
        if (bwd) fill_units(t, M, group_heads, bwd_heads(shape.V), int64_t(t.ctas) * WARPS * 8);
        else fill_units(t, M, group_heads, FWD_HEADS, int64_t(SMS) * 8);
        t.ctas = static_cast<int>(std::min<int64_t>(t.ctas, (t.units + WARPS - 1) / WARPS));
    }
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (dtype) {
        case LORA_T_BF16: e = launch_type<__nv_bfloat16>(a, shape, interleaved != 0, bwd, st); break;
        case LORA_T_FP16: e = launch_type<__half>(a, shape, interleaved != 0, bwd, st); break;
        default: e = launch_type<float>(a, shape, interleaved != 0, bwd, st); break;
    }
    if (e == cudaSuccess && want_dw) {
        if (!dw_typed || dtype == LORA_T_FP32) e = launch_dw<float>(a, dw, st);
        else if (dtype == LORA_T_BF16) e = launch_dw<__nv_bfloat16>(a, dw, st);
        else e = launch_dw<__half>(a, dw, st);
    }
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
    void *dw[2] = {nullptr, nullptr};
    return run(dtype, in, none, out, w, cos, sin, positions, n_pos, dw, false, M, D, rot, interleaved, norm, eps, false,
               nullptr, 0, stream);
}

lora_status_t lora_qk_norm_rope_bwd(int dtype, const lora_heads_t *dq_out, const lora_heads_t *dk_out,
                                    const lora_heads_t *q, const lora_heads_t *k, const void *q_weight,
                                    const void *k_weight, const float *cos, const float *sin, const int64_t *positions,
                                    int64_t n_pos, const lora_heads_t *dq, const lora_heads_t *dk, void *dq_weight,
                                    void *dk_weight, int64_t M, int D, int rot, int interleaved, int norm, float eps,
                                    void *workspace, size_t workspace_bytes, void *stream) {
    const lora_heads_t *in[2] = {q, k}, *dy[2] = {dq_out, dk_out}, *out[2] = {dq, dk};
    const void *w[2] = {q_weight, k_weight};
    void *dw[2] = {dq_weight, dk_weight};
    const bool typed = (dtype & LORA_T_WEIGHT_GRADS) != 0;
    dtype &= ~static_cast<int>(LORA_T_WEIGHT_GRADS);
    return run(dtype, in, dy, out, w, cos, sin, positions, n_pos, dw, typed, M, D, rot, interleaved, norm, eps, true, workspace,
               workspace_bytes, stream);
}

size_t lora_qk_norm_rope_workspace_size(int64_t M, int heads, int D) {
    if (M < 1 || heads < 1 || heads > 8192 || D < 8 || D > 256 || D % 8) return 0;
    return (dw_bytes(D) + 255) & ~size_t(255);
}

}  // extern "C"
