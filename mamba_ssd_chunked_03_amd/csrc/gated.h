// gated.h -- the gated recurrence and the 8-bit checkpoints: arguments, launchers and the
// element arithmetic that their kernels share.  Not part of the public ABI.
#pragma once

#include "ssd_internal.h"

namespace ssd {

constexpr int kGatedChunk = SSD_GATED_CHUNK;

// ---- the gate --------------------------------------------------------------------------
// With z = (g + bias) log2 e, formed as fma(g, log2 e, bias log2 e): q = 1 / (1 + 2^z) and
// a = 1 - q = 2^z q, each to a few fp32 ulps of ITSELF: where the state keeps nearly
// everything q is tiny, and where it keeps nearly nothing a is, and 1 - q would lose either.
// The roundings of z cost |z| 2^-24 relative, under 3e-6 for every |g + bias| < 30.  z above
// 128 gives 2^z = inf and q = 0 (true value below 2^-127), z below -126 gives q = 1, a = 0;
// NaN stays NaN in both.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float gate_q(float z) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z));
}
struct Gate {
    float q, a;
    __device__ __forceinline__ explicit Gate(float z) {
        const float e = __builtin_amdgcn_exp2f(z);
        q = __builtin_amdgcn_rcpf(1.f + e);
        a = z > 126.f ? 1.f : e * q;  // inf * 0 beyond
    }
};

// One step.  The form h + q (x - h) takes the decay as exactly 1 - q for the rounded q: with
// a separately rounded a = 1 - q, a slow channel's decay would be off by up to 2^-25 / q of
// its rate, the same way at every step.
__device__ __forceinline__ float gate_step(float q, float x, float h) {
    return fmaf(q, x - h, h);
}

// ---- 8-bit groups ----------------------------------------------------------------------
// bits of a group's largest |v| -> its scale and inverse.  As unsigned integers NaN and
// infinities lie above every finite value, so one integer maximum finds either.
struct CkptScale {
    float scale, inverse;
    __device__ __forceinline__ explicit CkptScale(uint32_t most) {
        const float m = __uint_as_float(most);
        const bool tiny = most < 0x0d800000u;        // below 2^-100: 127 / m could overflow
        const bool finite = most < 0x7f800000u;
        // at most the largest fp32 value that 127 times stays finite
        scale = tiny     ? 0.f
                : finite ? fminf(m / 127.f, 0x1.020406p+121f)
                         : __uint_as_float(0x7fc00000u);
        inverse = tiny || !finite ? 0.f : 127.f / m;
    }
};

// The codes of four neighbouring channels: the integers nearest to the exact products
// v * inverse, ties to even, in the low 8 bits of one fused multiply-add each onto 1.5 * 2^23,
// whose unit in the last place is 1.  A group that is not finite has inverse 0, and its codes
// are 0 whatever v is.
__device__ __forceinline__ uint32_t ckpt_codes(const float* v, const CkptScale& s) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(fmaf(v[i], s.inverse, 12582912.f));
    const uint32_t lo = __builtin_amdgcn_perm(w[1], w[0], 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(w[3], w[2], 0x04000c0cu);
    return s.inverse == 0.f ? 0u : lo | hi;
}

// The maximum over the LANES (8 or 16) neighbouring lanes of a group, in all of them.
template <int CTRL> __device__ __forceinline__ uint32_t dpp_move(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int LANES> __device__ __forceinline__ uint32_t ckpt_group_max(uint32_t v) {
    v = max(v, dpp_move<0xb1>(v));                    // quad_perm [1,0,3,2]
    v = max(v, dpp_move<0x4e>(v));                    // quad_perm [2,3,0,1]
    v = max(v, dpp_move<0x141>(v));                   // row_half_mirror: the other quad of 8
    if (LANES == 16) v = max(v, dpp_move<0x140>(v));  // row_mirror: the other 8 of 16
    return v;
}

// V codes of neighbouring channels (4 or 8 bytes at any alignment).
template <int V> struct CkptPiece {
    struct __attribute__((packed, aligned(1))) Any { uint32_t w[V / 4]; };
    uint32_t w[V / 4];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) w[k] = 0;
    }
    __device__ __forceinline__ void load(const int8_t* p) {
        const Any b = *(const Any*)p;
#pragma unroll
        for (int k = 0; k < V / 4; ++k) w[k] = b.w[k];
    }
    // the first n < V, zeros behind them
    __device__ __forceinline__ void load_part(const int8_t* p, int n) {
        clear();
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) w[i / 4] |= (uint32_t)(uint8_t)p[i] << (8 * (i % 4));
    }
    // elements lo to hi
    __device__ __forceinline__ void store(int8_t* p, int lo, int hi) const {
        if (hi - lo == V) {
            Any b;
#pragma unroll
            for (int k = 0; k < V / 4; ++k) b.w[k] = w[k];
            *(Any*)p = b;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i >= lo && i < hi) p[i] = (int8_t)(w[i / 4] >> (8 * (i % 4)));
        }
    }
    __device__ __forceinline__ float get(int i) const {
        return (float)(int8_t)(w[i / 4] >> (8 * (i % 4)));
    }
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int k = 0; k < V / 4; ++k) asm volatile("" : "+v"(w[k]));
    }
};
template <int V>
__device__ __forceinline__ void ckpt_store(int8_t* p, const float (&v)[V], const CkptScale& s,
                                           int lo, int hi) {
    CkptPiece<V> c;
#pragma unroll
    for (int k = 0; k < V / 4; ++k) c.w[k] = ckpt_codes(&v[4 * k], s);
    c.store(p, lo, hi);
}

// ---- launchers -------------------------------------------------------------------------
struct GatedFwdArgs {
    int B, T, D;
    const void *x, *g;               // rows in dtype
    long long x_stride, g_stride;
    const float* bias;               // [D] or null
    const int* cu;                   // packed row: [nseq + 1], or null
    int nseq;
    const float* init;               // [B][D] or null
    void* h;                         // [B][T][D], dtype
    float* final_state;              // [B or nseq][D] or null
    float* entry;                    // [B][nC][D] or null
    int8_t *x_codes, *g_codes;       // all four, or null
    float *x_scales, *g_scales;
};
struct GatedBwdArgs {
    int B, T, D;
    const void *x, *g;               // rows in dtype, or null: take the codes
    long long x_stride, g_stride;
    const int8_t *x_codes, *g_codes;
    const float *x_scales, *g_scales;
    const float* bias;
    const int* cu;
    int nseq;
    const float* entry;
    const void* dh;
    long long dh_stride;
    const float* d_final;            // [B or nseq][D] or null
    void *dx, *dg;
    long long dx_stride, dg_stride;
    float *d_bias, *d_init;          // [D], [B][D], or null
};
struct GatedStepArgs {
    int B, D;
    const void *x, *g;
    long long x_stride, g_stride;
    const float* bias;
    float* state;                    // [B][D]
    void* h;                         // [B][D], dtype
};
// workspace either pass needs (16-byte aligned)
size_t gated_workspace_bytes(int B, int T, int D);
// sizes as checked by the API; B, D >= 1
hipError_t launch_gated_fwd(ssd_dtype dtype, const GatedFwdArgs& a, void* ws, hipStream_t st);
hipError_t launch_gated_bwd(ssd_dtype dtype, const GatedBwdArgs& a, void* ws, hipStream_t st);
hipError_t launch_gated_step(ssd_dtype dtype, const GatedStepArgs& a, hipStream_t st);

// rows, width >= 1
hipError_t launch_ckpt_pack(long long rows, int width, ssd_dtype dtype, const void* src,
                            long long src_stride, int8_t* codes, float* scales, hipStream_t st);
hipError_t launch_ckpt_unpack(long long rows, int width, ssd_dtype dtype, const int8_t* codes,
                              const float* scales, void* dst, long long dst_stride,
                              hipStream_t st);

}  // namespace ssd
