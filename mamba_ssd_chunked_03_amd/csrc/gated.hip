// gated.hip -- the gated recurrence: forward, backward and single step.
//
// Per batch element and channel, with s = g + bias and q = 1 / (1 + exp(s)), a = 1 - q:
//     h_t = h_{t-1} + q_t (x_t - h_{t-1}),     G_t = dh_t + a_{t+1} G_{t+1},
//     dx_t = q_t G_t,   dg_t = G_t (h_{t-1} - x_t) q_t a_t     (dq/ds = -q a).
//
// Both recursions are affine in what they carry: over a span of steps the carry v becomes
// H + P v, with P the product of the span's a and H its result from zero, and two spans
// combine to (P2 P1, H2 + P2 H1).  A workgroup owns a tile of 64 channels and 32 runs of S
// steps; one pass over HBM:
//   1. every thread loads its run (S steps of 4 neighbouring channels) into registers and
//      forms the run's (P, H);
//   2. one wave, a lane per channel, scans the 32 runs through LDS into prefixes and the
//      tile's own (P, H), and finds the carry into the tile: the tiles of one chain (batch
//      element and 64 channels) publish their (P, H), every 16th also the carry out of it,
//      and a tile combines the last such carry with the spans behind it;
//   3. every thread takes its run's carry and goes through the run again, from registers.
// The backward does this for h from the saved entry states (no waiting) and, last step
// first, for G.  Bound by HBM: 3 (forward) or 5 (backward) values per element in and out.
//
// Waiting ends: tiles are numbered so that a chain's tiles follow in carry order, and a
// workgroup takes its number from a counter when it starts, so every tile that it waits for
// was taken by a workgroup that already runs; that one publishes its (P, H) before it
// waits itself, and the carry out of a 16th tile waits for earlier tiles only.  A published
// word holds the value and a tag in one 64-bit atomic store, so a reader that sees the tag
// has the value, whatever the order of other stores.
#include "gated.h"

namespace ssd {
namespace {

constexpr int kTileThreads = 512;
constexpr int kRuns = 32;      // runs of a tile; 16 lanes of 4 channels each
constexpr int kCols = 64;      // channels of a tile
// Steps of a run, so that what a thread holds of it (raw x and g, the backward's dh too) is
// 32 to 64 registers: more would halve the waves in flight.
constexpr int kFwdSteps = 8;
constexpr int bwd_steps(ssd_dtype t) { return t == SSD_F32 ? 4 : 8; }

// ---- quads: four neighbouring channels of a row ------------------------------------------
// Rows need only element alignment, so quads are loaded and stored as unaligned vectors
// (one 8- or 16-byte access each; the hardware takes any alignment).
template <typename T> struct Quad;
template <> struct Quad<__bf16> {
    uint2 v;
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = i < 2 ? v.x : v.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    __device__ __forceinline__ void clear() { v = make_uint2(0, 0); }
};
template <> struct Quad<float> {
    float4 v;
    __device__ __forceinline__ float get(int i) const {
        return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
    }
    __device__ __forceinline__ void clear() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
};
struct __attribute__((packed, aligned(2))) Bytes8 { uint32_t x, y; };
struct __attribute__((packed, aligned(4))) Bytes16 { float x, y, z, w; };
struct __attribute__((packed, aligned(1))) Bytes4 { uint32_t x; };

__device__ __forceinline__ void load(Quad<__bf16>& q, const __bf16* p) {
    const Bytes8 b = *(const Bytes8*)p;
    q.v = make_uint2(b.x, b.y);
}
__device__ __forceinline__ void load(Quad<float>& q, const float* p) {
    const Bytes16 b = *(const Bytes16*)p;
    q.v = make_float4(b.x, b.y, b.z, b.w);
}
__device__ __forceinline__ void load_part(Quad<__bf16>& q, const __bf16* p, int n) {
    const uint16_t* w = (const uint16_t*)p;
    q.v = make_uint2(0, 0);
    if (n > 0) q.v.x = w[0];
    if (n > 1) q.v.x |= (uint32_t)w[1] << 16;
    if (n > 2) q.v.y = w[2];
}
__device__ __forceinline__ void load_part(Quad<float>& q, const float* p, int n) {
    q.v = make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, 0.f);
}
// n: channels of the row from p on; four or more: the whole quad
__device__ __forceinline__ void store(__bf16* p, const float (&v)[4], int n) {
    typedef __bf16 pair __attribute__((ext_vector_type(2)));
    union { pair h[2]; uint32_t w[2]; } u;
    u.h[0] = pair{(__bf16)v[0], (__bf16)v[1]};
    u.h[1] = pair{(__bf16)v[2], (__bf16)v[3]};
    if (n >= 4) {
        *(Bytes8*)p = Bytes8{u.w[0], u.w[1]};
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) p[i] = u.h[i / 2][i % 2];
    }
}
__device__ __forceinline__ void store(float* p, const float (&v)[4], int n) {
    if (n >= 4) {
        *(Bytes16*)p = Bytes16{v[0], v[1], v[2], v[3]};
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < n) p[i] = v[i];
    }
}
__device__ __forceinline__ void load4(float (&v)[4], const float* p, int n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = p && i < n ? p[i] : 0.f;
}
__device__ __forceinline__ float4 lds4(const float* p) { return *(const float4*)p; }
__device__ __forceinline__ void put4(float* p, const float (&v)[4]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
}

// ---- tiles, and the carry between them ----------------------------------------------------
constexpr int kBlockTiles = 16;  // tiles of a block of a chain
constexpr int kLook = 4;         // spans looked at together

struct Tiles {
    unsigned* ticket;                  // counter of tiles taken (null: one tile per chain)
    unsigned long long* span;          // [tile][2][64] the tile's P and H
    unsigned long long* carry;         // [k / 16][chain][64] carry out of every 16th tile
    const uint8_t* starts;             // packed rows: bit t: a sequence starts at step t
    int chains, blocks, nk;            // B * blocks, channel blocks, tiles of a chain
};

// tag 1; 2: a sequence starts inside the span, so nothing from before reaches its end
__device__ __forceinline__ void publish(unsigned long long* p, float v, unsigned tag) {
    __hip_atomic_store(p, (unsigned long long)tag << 32 | __float_as_uint(v), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ unsigned long long look(const unsigned long long* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ bool there(unsigned long long w) { return (w >> 32) != 0; }
__device__ __forceinline__ float value(unsigned long long w) {
    return __uint_as_float((unsigned)w);
}

// One wave, a lane per channel.  (P, H): the tile's span; cut: a sequence starts inside;
// first: the carry into the chain's first tile.  Returns the carry into this tile.  The
// order of combining is fixed by the tile's place alone (the carry into its block, then the
// block's earlier spans from first to last), never by what happens to be ready, so results
// are the same bits on every run.
__device__ float carry_in(const Tiles& tl, unsigned tile, int k, float P, float H, bool cut,
                          float first) {
    if (tl.nk == 1) return first;
    const int lane = threadIdx.x & 63;
    const int i = k % kBlockTiles;
    const bool last = k == tl.nk - 1;
    if (!last && i < kBlockTiles - 1) {
        unsigned long long* s = tl.span + (size_t)tile * 2 * kCols + lane;
        publish(s, P, cut ? 2 : 1);
        publish(s + kCols, H, 1);
    }
    float accP = 1.f, accH = 0.f;
    bool accCut = false;
    const unsigned long long* s =
        tl.span + (size_t)(tile - (unsigned)i * tl.chains) * 2 * kCols + lane;
    const size_t step = (size_t)tl.chains * 2 * kCols;
    for (int m0 = 0; m0 < i; m0 += kLook, s += kLook * step) {
        unsigned long long p[kLook], h[kLook];
        for (;;) {
            bool all = true;
#pragma unroll
            for (int m = 0; m < kLook; ++m)
                if (m0 + m < i) {
                    p[m] = look(s + m * step);
                    h[m] = look(s + m * step + kCols);
                }
#pragma unroll
            for (int m = 0; m < kLook; ++m)
                if (m0 + m < i) all = all && there(p[m]) && there(h[m]);
            if (__all(all)) break;
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int m = 0; m < kLook; ++m)
            if (m0 + m < i) {
                const bool c = __builtin_amdgcn_readfirstlane((unsigned)(p[m] >> 32)) == 2;
                accH = c ? value(h[m]) : fmaf(value(p[m]), accH, value(h[m]));
                accP *= value(p[m]);
                accCut = accCut || c;
            }
    }
    float in = first;
    if (k >= kBlockTiles && !accCut) {
        const unsigned long long* c =
            tl.carry + ((size_t)(k / kBlockTiles - 1) * tl.chains + tile % tl.chains) * kCols + lane;
        unsigned long long v;
        while (!__all(there(v = look(c)))) __builtin_amdgcn_s_sleep(1);
        in = value(v);
    }
    in = accCut ? accH : fmaf(accP, in, accH);
    if (!last && i == kBlockTiles - 1)
        publish(tl.carry + ((size_t)(k / kBlockTiles) * tl.chains + tile % tl.chains) * kCols + lane,
                cut ? H : fmaf(P, in, H), 1);
    return in;
}

// The sequence of a packed row whose last step is t.
__device__ int sequence_ending(const int* cu, int nseq, int t) {
    int lo = 0, hi = nseq - 1;  // first s with cu[s + 1] > t
    while (lo < hi) {
        const int m = (lo + hi) / 2;
        if (cu[m + 1] > t) hi = m; else lo = m + 1;
    }
    return lo;
}

// Which tile, and where this thread stands in it.
struct Place {
    unsigned tile;
    int k, b, cb, cq, r, c0, n;  // n: channels of the row from c0 on (may be <= 0)
};
__device__ __forceinline__ Place place(const Tiles& tl, int D, unsigned* shared) {
    Place p;
    unsigned tile = blockIdx.x;
    if (tl.ticket) {
        if (threadIdx.x == 0) *shared = atomicAdd(tl.ticket, 1u);
        __syncthreads();
        tile = *shared;
    }
    p.tile = __builtin_amdgcn_readfirstlane(tile);
    p.k = p.tile / tl.chains;
    const int chain = p.tile % tl.chains;
    p.b = chain / tl.blocks;
    p.cb = chain % tl.blocks;
    p.cq = threadIdx.x & 15;
    p.r = threadIdx.x >> 4;
    p.c0 = p.cb * kCols + 4 * p.cq;
    p.n = D - p.c0;
    return p;
}

// Bits of a run's steps: starts (a sequence starts there) and ends (one ends there).
template <int S>
__device__ __forceinline__ void run_bits(const uint8_t* bits, int ts, int T, unsigned* starts,
                                         unsigned* ends) {
    const unsigned w = (bits[ts >> 3] | (unsigned)bits[(ts >> 3) + 1] << 8) >> (ts & 7);
    constexpr unsigned mask = (1u << S) - 1;
    *starts = w & mask;
    *ends = (w >> 1) & mask;
    if (T - 1 >= ts && T - 1 < ts + S) *ends |= 1u << (T - 1 - ts);
}

// Load a run's quads of rows b*T + ts + j (steps behind T repeat the last one; the caller
// clears them).
template <typename T, int S>
__device__ __forceinline__ void load_run(Quad<T> (&q)[S], const void* base, long long stride,
                                         long long row0, int ts, int steps, int c0, int n) {
    const T* p = (const T*)base + c0;
    if (n >= 4) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            load(q[j], p + (row0 + min(ts + j, steps - 1)) * stride);
    } else {
#pragma unroll
        for (int j = 0; j < S; ++j)
            load_part(q[j], p + (row0 + min(ts + j, steps - 1)) * stride, n);
    }
}

// ---- forward ------------------------------------------------------------------------------
template <typename T, int S, bool PACKED>
__global__ __launch_bounds__(kTileThreads) void gated_fwd_kernel(GatedFwdArgs a, Tiles tl) {
    constexpr int kTile = kRuns * S;
    __shared__ __align__(16) float sP[kRuns * kCols], sH[kRuns * kCols], sE[kCols];
    __shared__ unsigned sTile, sCut[kRuns];
    const Place w = place(tl, a.D, &sTile);
    const int t0 = w.k * kTile, ts = t0 + w.r * S;
    const long long row0 = (long long)w.b * a.T;
    Quad<T> x[S], g[S];
    load_run<T, S>(g, a.g, a.g_stride, row0, ts, a.T, w.c0, w.n);
    load_run<T, S>(x, a.x, a.x_stride, row0, ts, a.T, w.c0, w.n);
    float bias[4];
    load4(bias, a.bias ? a.bias + w.c0 : nullptr, w.n);
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] *= kLog2e;
    unsigned starts = 0, ends = 0;
    if (PACKED) {
        run_bits<S>(tl.starts, ts, a.T, &starts, &ends);
        if (w.cq == 0) sCut[w.r] = starts;
    }
    const bool whole = t0 + kTile <= a.T;

    float q[S][4], P[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < S; ++j) {
#pragma unroll
        for (int i = 0; i < 4; ++i) q[j][i] = gate_q(fmaf(g[j].get(i), kLog2e, bias[i]));
    }
    if (!whole) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (ts + j >= a.T) {
                x[j].clear();
                q[j][0] = q[j][1] = q[j][2] = q[j][3] = 0.f;
            }
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
        if (PACKED && (starts >> j & 1)) {
#pragma unroll
            for (int i = 0; i < 4; ++i) P[i] = H[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            H[i] = gate_step(q[j][i], x[j].get(i), H[i]);
            P[i] = fmaf(-q[j][i], P[i], P[i]);
        }
    }
    put4(&sP[w.r * kCols + 4 * w.cq], P);
    put4(&sH[w.r * kCols + 4 * w.cq], H);
    __syncthreads();
    unsigned cuts = 0;
    if (PACKED) cuts = (unsigned)__ballot(sCut[threadIdx.x & 31] != 0);
    if (threadIdx.x < kCols) {
        const int lane = threadIdx.x, c = w.cb * kCols + lane;
        float accP = 1.f, accH = 0.f;
#pragma unroll
        for (int r0 = 0; r0 < kRuns; r0 += 8) {
            float p[8], h[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                p[r] = sP[(r0 + r) * kCols + lane];
                h[r] = sH[(r0 + r) * kCols + lane];
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                sP[(r0 + r) * kCols + lane] = accP;
                sH[(r0 + r) * kCols + lane] = accH;
                const bool cut = PACKED && (cuts >> (r0 + r) & 1);
                accH = cut ? h[r] : fmaf(p[r], accH, h[r]);
                accP *= p[r];
            }
        }
        const float first =
            w.k < kBlockTiles && a.init && c < a.D ? a.init[(long long)w.b * a.D + c] : 0.f;
        sE[lane] = carry_in(tl, w.tile, w.k, accP, accH, cuts != 0, first);
    }
    __syncthreads();
    float h[4];
    {
        const float4 p = lds4(&sP[w.r * kCols + 4 * w.cq]), v = lds4(&sH[w.r * kCols + 4 * w.cq]);
        const float4 e = lds4(&sE[4 * w.cq]);
        const bool cut = PACKED && (cuts & ((1u << w.r) - 1));
        h[0] = cut ? v.x : fmaf(p.x, e.x, v.x);
        h[1] = cut ? v.y : fmaf(p.y, e.y, v.y);
        h[2] = cut ? v.z : fmaf(p.z, e.z, v.z);
        h[3] = cut ? v.w : fmaf(p.w, e.w, v.w);
    }
    if (w.n <= 0) return;
    if (a.entry && ts % kGatedChunk == 0 && ts < a.T) {
        const long long nC = (a.T + kGatedChunk - 1) / kGatedChunk;
        store(a.entry + (w.b * nC + ts / kGatedChunk) * a.D + w.c0, h, w.n);
    }
#pragma unroll
    for (int j = 0; j < S; ++j) {
        if (PACKED && (starts >> j & 1)) h[0] = h[1] = h[2] = h[3] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) h[i] = gate_step(q[j][i], x[j].get(i), h[i]);
        if (whole || ts + j < a.T)
            store((T*)a.h + (row0 + ts + j) * a.D + w.c0, h, w.n);
        if (PACKED && a.final_state && (ends >> j & 1))
            store(a.final_state + (long long)sequence_ending(a.cu, a.nseq, ts + j) * a.D + w.c0, h,
                  w.n);
    }
    if (!PACKED && a.final_state && ts <= a.T - 1 && a.T - 1 < ts + S)
        store(a.final_state + (long long)w.b * a.D + w.c0, h, w.n);
}

// Values that a later pass computes from again: without this the compiler keeps the first
// pass' gates in registers instead (205 against 128 and fewer, which halves the waves).
__device__ __forceinline__ void renew(uint32_t& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void renew(Quad<__bf16>& q) { renew(q.v.x); renew(q.v.y); }
__device__ __forceinline__ void renew(float& v) { asm volatile("" : "+v"(v)); }
__device__ __forceinline__ void renew(Quad<float>& q) {
    renew(q.v.x); renew(q.v.y); renew(q.v.z); renew(q.v.w);
}

// ---- backward -----------------------------------------------------------------------------
// x and g of a run, from rows in T or from 8-bit codes and their scales (the tile's 64
// channels are one group).
template <typename T, int S, bool CODES> struct RunIn;
template <typename T, int S> struct RunIn<T, S, false> {
    Quad<T> v[S];
    __device__ __forceinline__ void load(const void* rows, long long stride, const int8_t*,
                                         const float*, long long row0, int ts, const Place& w,
                                         const GatedBwdArgs& a) {
        load_run<T, S>(v, rows, stride, row0, ts, a.T, w.c0, w.n);
    }
    __device__ __forceinline__ float get(int j, int i) const { return v[j].get(i); }
    __device__ __forceinline__ void clear(int j) { v[j].clear(); }
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int j = 0; j < S; ++j) renew(v[j]);
    }
};
template <typename T, int S> struct RunIn<T, S, true> {
    uint32_t v[S];
    float s[S];
    __device__ __forceinline__ void load(const void*, long long, const int8_t* codes,
                                         const float* scales, long long row0, int ts,
                                         const Place& w, const GatedBwdArgs& a) {
        const int groups = (a.D + kCols - 1) / kCols;
#pragma unroll
        for (int j = 0; j < S; ++j) {
            const long long row = row0 + min(ts + j, a.T - 1);
            const int8_t* p = codes + row * a.D + w.c0;
            v[j] = 0;
            if (w.n >= 4) {
                v[j] = ((const Bytes4*)p)->x;
            } else {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < w.n) v[j] |= (uint32_t)(uint8_t)p[i] << (8 * i);
            }
            s[j] = scales[row * groups + w.cb];
        }
    }
    __device__ __forceinline__ float get(int j, int i) const {
        return (float)(int8_t)(v[j] >> (8 * i)) * s[j];
    }
    __device__ __forceinline__ void clear(int j) { v[j] = 0; s[j] = 0.f; }
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int j = 0; j < S; ++j) renew(v[j]);
    }
};

template <typename T, int S, bool PACKED, bool CODES>
__global__ __launch_bounds__(kTileThreads) void gated_bwd_kernel(GatedBwdArgs a, Tiles tl,
                                                                 float* part) {
    constexpr int kTile = kRuns * S;
    constexpr int kChunkRuns = kGatedChunk / S;
    __shared__ __align__(16) float sP[kRuns * kCols], sH[kRuns * kCols], sC[kRuns * kCols],
        sR[kRuns * kCols], sE[kCols];
    __shared__ unsigned sTile, sCut[kRuns];
    const Place w = place(tl, a.D, &sTile);
    const int kt = tl.nk - 1 - w.k;  // last tile first
    const int t0 = kt * kTile, ts = t0 + w.r * S;
    const long long row0 = (long long)w.b * a.T;
    RunIn<T, S, CODES> x, g;
    Quad<T> dh[S];
    g.load(a.g, a.g_stride, a.g_codes, a.g_scales, row0, ts, w, a);
    x.load(a.x, a.x_stride, a.x_codes, a.x_scales, row0, ts, w, a);
    load_run<T, S>(dh, a.dh, a.dh_stride, row0, ts, a.T, w.c0, w.n);
    float bias[4];
    load4(bias, a.bias ? a.bias + w.c0 : nullptr, w.n);
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] *= kLog2e;
    unsigned starts = 0, ends = 0;
    if (PACKED) {
        run_bits<S>(tl.starts, ts, a.T, &starts, &ends);
        if (w.cq == 0) sCut[w.r] = starts;
    }
    const bool whole = t0 + kTile <= a.T;
    if (!whole) {
#pragma unroll
        for (int j = 0; j < S; ++j)
            if (ts + j >= a.T) {
                x.clear(j);
                dh[j].clear();
            }
    }
    // d_final of a packed sequence that ends at step j of this run
    auto ending = [&](int j, float (&v)[4]) {
        load4(v,
              a.d_final ? a.d_final +
                              (long long)sequence_ending(a.cu, a.nseq, ts + j) * a.D + w.c0
                        : nullptr,
              w.n);
    };
    {
        float P[4] = {1.f, 1.f, 1.f, 1.f}, H[4] = {0.f, 0.f, 0.f, 0.f}, C[4];
        float q[S][4];
#pragma unroll
        for (int j = 0; j < S; ++j) {
            if (PACKED && (starts >> j & 1)) {
#pragma unroll
                for (int i = 0; i < 4; ++i) P[i] = H[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                q[j][i] = gate_q(fmaf(g.get(j, i), kLog2e, bias[i]));
                if (!whole && ts + j >= a.T) q[j][i] = 0.f;
                H[i] = gate_step(q[j][i], x.get(j, i), H[i]);
                P[i] = fmaf(-q[j][i], P[i], P[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) C[i] = 0.f;
#pragma unroll
        for (int j = S - 1; j >= 0; --j) {
            if (PACKED && (ends >> j & 1)) ending(j, C);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float G = dh[j].get(i) + C[i];
                C[i] = fmaf(-q[j][i], G, G);
            }
            if (PACKED && (starts >> j & 1)) C[0] = C[1] = C[2] = C[3] = 0.f;
        }
        put4(&sP[w.r * kCols + 4 * w.cq], P);
        put4(&sH[w.r * kCols + 4 * w.cq], H);
        put4(&sC[w.r * kCols + 4 * w.cq], C);
    }
    __syncthreads();
    unsigned cuts = 0;
    if (PACKED) cuts = (unsigned)__ballot(sCut[threadIdx.x & 31] != 0);
    if (threadIdx.x < kCols) {  // the first wave: G, last run first
        const int lane = threadIdx.x, c = w.cb * kCols + lane;
        float accP = 1.f, accC = 0.f;
#pragma unroll
        for (int r0 = kRuns - 8; r0 >= 0; r0 -= 8) {
            float p[8], v[8];
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                p[r] = sP[(r0 + r) * kCols + lane];
                v[r] = sC[(r0 + r) * kCols + lane];
            }
#pragma unroll
            for (int r = 7; r >= 0; --r) {
                sR[(r0 + r) * kCols + lane] = accP;
                sC[(r0 + r) * kCols + lane] = accC;
                const bool cut = PACKED && (cuts >> (r0 + r) & 1);
                accC = cut ? v[r] : fmaf(p[r], accC, v[r]);
                accP *= p[r];
            }
        }
        const float first = !PACKED && w.k < kBlockTiles && a.d_final && c < a.D
                                ? a.d_final[(long long)w.b * a.D + c]
                                : 0.f;
        sE[lane] = carry_in(tl, w.tile, w.k, accP, accC, cuts != 0, first);
    } else if (threadIdx.x < 2 * kCols) {  // the second: h, from every chunk's entry state
        const int lane = threadIdx.x - kCols, c = w.cb * kCols + lane;
        const int nC = (a.T + kGatedChunk - 1) / kGatedChunk;
        float E[kTile / kGatedChunk];
#pragma unroll
        for (int k = 0; k < kTile / kGatedChunk; ++k) {
            const int chunk = t0 / kGatedChunk + k;
            E[k] = chunk < nC && c < a.D ? a.entry[((long long)w.b * nC + chunk) * a.D + c] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kTile / kGatedChunk; ++k) {
            float e = E[k];
#pragma unroll
            for (int r = k * kChunkRuns; r < (k + 1) * kChunkRuns; ++r) {
                const float p = sP[r * kCols + lane], v = sH[r * kCols + lane];
                sH[r * kCols + lane] = e;
                e = PACKED && (cuts >> r & 1) ? v : fmaf(p, e, v);
            }
        }
    }
    __syncthreads();
    float h[4], C[4], db[4] = {0.f, 0.f, 0.f, 0.f};
    {
        const int at = w.r * kCols + 4 * w.cq;
        const float4 e = lds4(&sH[at]), p = lds4(&sR[at]), v = lds4(&sC[at]);
        const float4 in = lds4(&sE[4 * w.cq]);
        h[0] = e.x; h[1] = e.y; h[2] = e.z; h[3] = e.w;
        const bool cut = PACKED && w.r < 31 && (cuts >> (w.r + 1));
        C[0] = cut ? v.x : fmaf(p.x, in.x, v.x);
        C[1] = cut ? v.y : fmaf(p.y, in.y, v.y);
        C[2] = cut ? v.z : fmaf(p.z, in.z, v.z);
        C[3] = cut ? v.w : fmaf(p.w, in.w, v.w);
    }
    g.again();
    x.again();
#pragma unroll
    for (int j = 0; j < S; ++j) renew(dh[j]);
    float off[S][4];  // h_{t-1} - x_t
#pragma unroll
    for (int j = 0; j < S; ++j) {
        if (PACKED && (starts >> j & 1)) h[0] = h[1] = h[2] = h[3] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            off[j][i] = h[i] - x.get(j, i);
            if (j < S - 1) {
                const float q = gate_q(fmaf(g.get(j, i), kLog2e, bias[i]));
                h[i] = fmaf(-q, off[j][i], h[i]);
            }
        }
    }
    g.again();
#pragma unroll
    for (int j = S - 1; j >= 0; --j) {
        if (PACKED && (ends >> j & 1)) ending(j, C);
        if (whole || ts + j < a.T) {
            float dx[4], dg[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const Gate e(fmaf(g.get(j, i), kLog2e, bias[i]));
                const float G = dh[j].get(i) + C[i];
                dx[i] = e.q * G;
                dg[i] = dx[i] * e.a * off[j][i];
                db[i] += dg[i];
                C[i] = fmaf(-e.q, G, G);
            }
            const long long row = row0 + ts + j;
            store((T*)a.dx + row * a.dx_stride + w.c0, dx, w.n);
            store((T*)a.dg + row * a.dg_stride + w.c0, dg, w.n);
        }
        if (PACKED && (starts >> j & 1)) C[0] = C[1] = C[2] = C[3] = 0.f;
    }
    if (!PACKED && a.d_init && ts == 0) store(a.d_init + (long long)w.b * a.D + w.c0, C, w.n);
    if (!part) return;
    put4(&sP[w.r * kCols + 4 * w.cq], db);  // the scans are done with sP
    __syncthreads();
    if (threadIdx.x < kCols && w.cb * kCols + (int)threadIdx.x < a.D) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRuns; ++r) s += sP[r * kCols + threadIdx.x];
        part[((long long)w.b * tl.nk + kt) * a.D + w.cb * kCols + threadIdx.x] = s;
    }
}

// ---- small kernels ------------------------------------------------------------------------
constexpr int kThreads = 256;

// Before a pass: the counter and the tags cleared, the start bits of a packed row, and zero
// final states for its empty sequences.
struct Prep {
    unsigned* clear;       // ticket and tags: words to clear
    long long words;
    uint8_t* starts;       // null: not a packed row
    int bytes;             // of starts
    const int* cu;
    int nseq, T, D;
    float* final_state;    // null: none
};
__global__ __launch_bounds__(kThreads) void gated_prep_kernel(Prep p) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long all = (long long)gridDim.x * kThreads;
    for (long long i = id; i < p.words / 4; i += all)
        reinterpret_cast<uint4*>(p.clear)[i] = make_uint4(0, 0, 0, 0);
    if (!p.starts) return;
    for (long long i = id; i < p.bytes; i += all) {
        int lo = 0, hi = p.nseq;  // first s with cu[s] >= 8 i
        while (lo < hi) {
            const int m = (lo + hi) / 2;
            if (p.cu[m] >= 8 * i) hi = m; else lo = m + 1;
        }
        unsigned bits = 0;
        for (int s = lo; s < p.nseq && p.cu[s] < 8 * i + 8; ++s)
            if (p.cu[s + 1] > p.cu[s]) bits |= 1u << (p.cu[s] - 8 * i);
        p.starts[i] = (uint8_t)bits;
    }
    if (!p.final_state) return;
    for (long long i = id; i < (long long)p.nseq * p.D; i += all) {
        const int s = (int)(i / p.D);
        if (p.cu[s + 1] <= p.cu[s]) p.final_state[i] = 0.f;
    }
}

// d_bias from the tiles' sums: a workgroup per 64 channels, 16 threads per channel; fixed
// order.
__global__ __launch_bounds__(1024) void gated_dbias_kernel(const float* part, float* d_bias,
                                                           int rows, int D) {
    __shared__ float s[16][kCols];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int c = blockIdx.x * kCols + lane;
    float v = 0.f;
    if (c < D)
        for (int r = w; r < rows; r += 16) v += part[(long long)r * D + c];
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || c >= D) return;
    for (int i = 1; i < 16; ++i) v += s[i][lane];
    d_bias[c] = v;
}

__global__ __launch_bounds__(kThreads) void gated_carry_kernel(const float* src, float* dst,
                                                               long long n) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id < n) dst[id] = src ? src[id] : 0.f;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedStepArgs a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)a.B * a.D) return;
    const long long b = id / a.D;
    const int d = (int)(id % a.D);
    const float q = gate_q(fmaf(to_f32(((const T*)a.g)[b * a.g_stride + d]), kLog2e,
                                (a.bias ? a.bias[d] : 0.f) * kLog2e));
    const float h = gate_step(q, to_f32(((const T*)a.x)[b * a.x_stride + d]), a.state[id]);
    a.state[id] = h;
    ((T*)a.h)[id] = from_f32<T>(h);
}

unsigned blocks_of(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

// ---- workspace: ticket and tags | start bits | d_bias' sums ---------------------------------
struct Layout {
    int nk, blocks;
    long long tiles, carries;
    size_t clear, starts, part, bytes;  // sizes of the first two; offset of the third; total
};
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
Layout layout(int B, int T, int D, int steps) {
    Layout l;
    const int kTile = kRuns * steps;
    l.nk = (T + kTile - 1) / kTile;
    l.blocks = (D + kCols - 1) / kCols;
    l.tiles = (long long)B * l.blocks * l.nk;
    l.carries = l.nk / kBlockTiles * (l.tiles / l.nk);
    l.clear = l.nk > 1 ? 256 + ((size_t)l.tiles * 2 + l.carries) * kCols * 8 : 0;
    l.starts = up256((size_t)l.nk * (kTile / 8) + 1);
    l.part = l.clear + l.starts;
    l.bytes = l.part + (size_t)B * l.nk * D * sizeof(float);
    return l;
}
Tiles tiles_of(const Layout& l, int B, char* ws, bool packed) {
    Tiles t = {};
    t.blocks = l.blocks;
    t.chains = B * l.blocks;
    t.nk = l.nk;
    if (l.nk > 1) {
        t.ticket = (unsigned*)ws;
        t.span = (unsigned long long*)(ws + 256);
        t.carry = t.span + l.tiles * 2 * kCols;
    }
    if (packed) t.starts = (const uint8_t*)(ws + l.clear);
    return t;
}
hipError_t prepare(const Layout& l, char* ws, const int* cu, int nseq, int T, int D,
                   float* final_state, hipStream_t st) {
    if (l.nk <= 1 && !cu) return hipSuccess;
    Prep p = {};
    p.clear = (unsigned*)ws;
    p.words = (long long)(l.clear / 4);
    long long work = p.words / 4;
    if (cu) {
        p.starts = (uint8_t*)(ws + l.clear);
        p.bytes = (int)l.starts;
        p.cu = cu; p.nseq = nseq; p.T = T; p.D = D;
        p.final_state = final_state;
        if (p.bytes > work) work = p.bytes;
        if (final_state && (long long)nseq * D > work) work = (long long)nseq * D;
    }
    unsigned blocks = blocks_of(work);
    if (blocks > 2048) blocks = 2048;
    gated_prep_kernel<<<blocks, kThreads, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

size_t gated_workspace_bytes(int B, int T, int D) {
    if (B == 0 || T == 0 || D == 0) return 0;
    const size_t fwd = layout(B, T, D, kFwdSteps).bytes;
    const size_t bwd = layout(B, T, D, bwd_steps(SSD_F32)).bytes;  // the shorter tiles
    return fwd > bwd ? fwd : bwd;
}

hipError_t launch_gated_fwd(ssd_dtype dtype, const GatedFwdArgs& a, void* ws, hipStream_t st) {
    if (a.T == 0) {
        if (!a.final_state) return hipSuccess;
        const long long n = (long long)(a.cu ? a.nseq : a.B) * a.D;
        gated_carry_kernel<<<blocks_of(n), kThreads, 0, st>>>(a.init, a.final_state, n);
        return hipGetLastError();
    }
    const Layout l = layout(a.B, a.T, a.D, kFwdSteps);
    hipError_t e = prepare(l, (char*)ws, a.cu, a.nseq, a.T, a.D, a.final_state, st);
    if (e != hipSuccess) return e;
    const Tiles tl = tiles_of(l, a.B, (char*)ws, a.cu != nullptr);
    const dim3 grid((unsigned)l.tiles), block(kTileThreads);
    constexpr int S = kFwdSteps;
    if (dtype == SSD_F32)
        a.cu ? gated_fwd_kernel<float, S, true><<<grid, block, 0, st>>>(a, tl)
             : gated_fwd_kernel<float, S, false><<<grid, block, 0, st>>>(a, tl);
    else
        a.cu ? gated_fwd_kernel<__bf16, S, true><<<grid, block, 0, st>>>(a, tl)
             : gated_fwd_kernel<__bf16, S, false><<<grid, block, 0, st>>>(a, tl);
    e = hipGetLastError();
    if (e != hipSuccess || !a.x_codes) return e;
    const long long rows = (long long)a.B * a.T;
    e = launch_ckpt_pack(rows, a.D, dtype, a.x, a.x_stride, a.x_codes, a.x_scales, st);
    if (e != hipSuccess) return e;
    return launch_ckpt_pack(rows, a.D, dtype, a.g, a.g_stride, a.g_codes, a.g_scales, st);
}

hipError_t launch_gated_bwd(ssd_dtype dtype, const GatedBwdArgs& a, void* ws, hipStream_t st) {
    if (a.T == 0 || a.B == 0) {
        const long long n = (long long)a.B * a.D;
        if (a.d_init && n > 0)
            gated_carry_kernel<<<blocks_of(n), kThreads, 0, st>>>(a.d_final, a.d_init, n);
        if (a.d_bias)
            gated_carry_kernel<<<blocks_of(a.D), kThreads, 0, st>>>(nullptr, a.d_bias, a.D);
        return hipGetLastError();
    }
    const Layout l = layout(a.B, a.T, a.D, bwd_steps(dtype));
    hipError_t e = prepare(l, (char*)ws, a.cu, a.nseq, a.T, a.D, nullptr, st);
    if (e != hipSuccess) return e;
    const Tiles tl = tiles_of(l, a.B, (char*)ws, a.cu != nullptr);
    const dim3 grid((unsigned)l.tiles), block(kTileThreads);
    const int rows = a.B * l.nk;
    float* part = !a.d_bias ? nullptr : rows == 1 ? a.d_bias : (float*)((char*)ws + l.part);
#define SSD_GATED_BWD(T, DT, PACKED, CODES) \
    gated_bwd_kernel<T, bwd_steps(DT), PACKED, CODES><<<grid, block, 0, st>>>(a, tl, part)
    const bool codes = a.x_codes != nullptr, packed = a.cu != nullptr;
    if (dtype == SSD_F32) {
        if (packed) codes ? SSD_GATED_BWD(float, SSD_F32, true, true) : SSD_GATED_BWD(float, SSD_F32, true, false);
        else codes ? SSD_GATED_BWD(float, SSD_F32, false, true) : SSD_GATED_BWD(float, SSD_F32, false, false);
    } else {
        if (packed) codes ? SSD_GATED_BWD(__bf16, SSD_BF16, true, true) : SSD_GATED_BWD(__bf16, SSD_BF16, true, false);
        else codes ? SSD_GATED_BWD(__bf16, SSD_BF16, false, true) : SSD_GATED_BWD(__bf16, SSD_BF16, false, false);
    }
#undef SSD_GATED_BWD
    e = hipGetLastError();
    if (e != hipSuccess || !a.d_bias || rows == 1) return e;
    gated_dbias_kernel<<<(unsigned)l.blocks, 1024, 0, st>>>(part, a.d_bias, rows, a.D);
    return hipGetLastError();
}

hipError_t launch_gated_step(ssd_dtype dtype, const GatedStepArgs& a, hipStream_t st) {
    const unsigned blocks = blocks_of((long long)a.B * a.D);
    if (dtype == SSD_F32)
        gated_step_kernel<float><<<blocks, kThreads, 0, st>>>(a);
    else
        gated_step_kernel<__bf16><<<blocks, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace ssd
