// gated.hip -- the gated recurrence: forward, backward and single step.
//
// Per batch element and channel, with s = g + bias and q = 1 / (1 + exp(s)), a = 1 - q:
//     h_t = h_{t-1} + q_t (x_t - h_{t-1}),     G_t = dh_t + a_{t+1} G_{t+1},
//     dx_t = q_t G_t,   dg_t = G_t (h_{t-1} - x_t) q_t a_t     (dq/ds = -q a).
//
// Both recursions are affine in what they carry: over a span of steps the carry v becomes
// H + P v, with P the product of the span's a and H its result from zero, and two spans
// combine to (P2 P1, H2 + P2 H1).  A workgroup works on a tile of 16 lanes' pieces of a row
// (64 or 128 channels) by 32 runs of S steps, in one pass over HBM:
//   1. every thread loads its run (S steps of its piece) into registers and forms the run's
//      (P, H);
//   2. a lane per channel scans the 32 runs through LDS into prefixes and the tile's own
//      (P, H), publishes that, and finds the carry into the tile from what the tiles before
//      it in its chain (batch element and channels) have published;
//   3. every thread takes its run's carry and goes through the run again, from registers.
// The backward does this for h from the saved entry states (no waiting) and, last step
// first, for G.
//
// Bound by HBM: 3 (forward) or 5 (backward) values per element in and out.  At 4 x 4096 x 5120
// in bf16 the forward takes 99 us (503 MB, 5.1 TB/s: what a large copy reaches here) and the
// backward 182 us (844 MB, 4.6 TB/s); a forward in three kernels would read x and g twice, 5
// values per element.  One tile alone takes 5.5 us from launch to end; what lies between
// that and HBM's time at medium sizes is the wait for the carry and the prep launch (2 us).
//
// Waiting ends: tiles are numbered so that a chain's tiles follow in carry order, and a
// workgroup takes numbers from a counter, the next one while it works on a tile.  Of all
// tiles not finished the one with the lowest number in its counter is being worked on (a
// workgroup works on its numbers in order), and what it waits for was published by finished
// tiles, or by later parts of none: a tile publishes its own (P, H) before it waits.  So it
// ends, whatever share of the workgroups is on the device.
#include <initializer_list>

#include "gated.h"

namespace ssd {
namespace {

constexpr int kLanes = 16;  // lanes along a row of a tile
constexpr int kRuns = 32;   // runs of a tile: 512 threads, two workgroups to a CU
constexpr int kLook = 8;    // published spans looked at together
constexpr int kScan = 8;    // runs that a scan reads together

// V channels by S steps of a lane.  16 or 32 elements a lane in 16 or 8 byte pieces were
// measured, at 4 x 4096 x 5120 (backward, and forward with codes at 8 x 2048 x 1536), at one
// row of 65536 x 5120 (forward) and of 65536 x 256 (thin; non-temporal loads):
//   bf16 forward  4 x 8: 99, 393, thin 31 us;    8 x 4: 100, 414, 36;   4 x 4: 122, 531, 43
//   with codes    8 x 4: 114 us for the training pass;  4 x 8: 124: the 8-bit scales' two
//                 divisions come once per step and lane
//   bf16 backward 4 x 8: 183 us;  4 x 4: 200;  8 x 4: 228 (more registers than there are)
//   fp32          4 x 8 forward, 4 x 4 backward: the same bytes a lane as in bf16
constexpr int fwd_vec(ssd_dtype t, bool codes) { return t == SSD_BF16 && codes ? 8 : 4; }
constexpr int fwd_steps(ssd_dtype t, bool codes) { return t == SSD_BF16 && codes ? 4 : 8; }
constexpr int kBwdVec = 4;
constexpr int bwd_steps(ssd_dtype t) { return t == SSD_BF16 ? 8 : 4; }

// ---- pieces: a lane's V neighbouring channels of a row -------------------------------------
// Rows need only element alignment, so pieces are loaded and stored as unaligned vectors (one
// access each; the hardware takes any alignment).
// Stores of rows are non-temporal, since every row is written once: at 4 x 4096 x 5120 in bf16
// the forward takes 99 us so and 101 us with cached stores, the backward 184 and 193.  Loads of
// rows are non-temporal where the call's rows are large (kCachedBytes).
template <int WORDS> using Words = uint32_t __attribute__((ext_vector_type(WORDS)));
template <typename T, int WORDS> struct AnyWords {
    typedef Words<WORDS> Any __attribute__((aligned(sizeof(T))));
};
struct __attribute__((packed, aligned(4))) Floats4 { float v[4]; };

template <typename T, int V> struct Piece {
    static constexpr int W = V * (int)sizeof(T) / 4;
    uint32_t w[W];
    __device__ __forceinline__ float get(int i) const {
        if (sizeof(T) == 4) return __uint_as_float(w[i % W]);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const T* p) {
        const Words<W> b =
            __builtin_nontemporal_load((const typename AnyWords<T, W>::Any*)p);
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = b[i];
    }
    __device__ __forceinline__ void load_cached(const T* p) {
        const Words<W> b = *(const typename AnyWords<T, W>::Any*)p;
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = b[i];
    }
    // the first n < V channels, zeros behind them
    __device__ __forceinline__ void load_part(const T* p, int n) {
        clear();
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) {
                if (sizeof(T) == 4) w[i % W] = ((const uint32_t*)p)[i];
                else w[i / 2] |= (uint32_t)((const uint16_t*)p)[i] << (16 * (i & 1));
            }
    }
    // Values that a later pass computes from again: without this the compiler keeps the
    // first pass' gates in registers instead, which halves the waves in flight.
    __device__ __forceinline__ void renew() {
#pragma unroll
        for (int i = 0; i < W; ++i) asm volatile("" : "+v"(w[i]));
    }
};

// Which channels a lane has.  Its piece starts at channel c0; it owns elements lo to hi of it.
// A row's last piece is moved back to end with the row, so that every load is a whole piece
// inside the row: a lane there computes channels that its neighbour owns too and stores its
// own alone, and a lane behind the row's end owns none.  Rows narrower than a piece (NARROW)
// have one lane, which loads element by element.
struct Own {
    int c0, lo, hi;
    __device__ __forceinline__ bool any() const { return lo < hi; }
    __device__ __forceinline__ bool has(int i) const { return i >= lo && i < hi; }
};
template <int V, bool NARROW> __device__ __forceinline__ Own own_of(int piece, int D) {
    const int c = piece * V;
    if (NARROW) return Own{0, 0, piece == 0 ? D : 0};
    const int n = D - c;  // channels from c on
    return Own{min(c, D - V), n >= V ? 0 : n > 0 ? V - n : V, V};
}

template <typename T, int V, bool CACHED = false>
__device__ __forceinline__ void store(T* p, const float (&v)[V], const Own& o) {
    constexpr int W = V * (int)sizeof(T) / 4;
    union { T t[V]; Words<W> b; } u;
#pragma unroll
    for (int i = 0; i < V; ++i) u.t[i] = from_f32<T>(v[i]);
    if (o.hi - o.lo == V) {
        if (CACHED) *(typename AnyWords<T, W>::Any*)p = u.b;
        else __builtin_nontemporal_store(u.b, (typename AnyWords<T, W>::Any*)p);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
            if (o.has(i)) p[i] = u.t[i];
    }
}
template <int V, bool NARROW>
__device__ __forceinline__ void load_f32(float (&v)[V], const float* p, const Own& o) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    } else if (NARROW) {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < o.hi ? p[i] : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const Floats4 f = *(const Floats4*)(p + i);
            v[i] = f.v[0]; v[i + 1] = f.v[1]; v[i + 2] = f.v[2]; v[i + 3] = f.v[3];
        }
    }
}

// A run's values of a tile's C = 16 V channels in LDS: column 64 (i / 4) + 4 lane + i % 4
// holds channel V lane + i, so a lane's accesses are 16-byte vectors and neighbouring lanes'
// lie side by side.
template <int V> __device__ __forceinline__ void put(float* row, int cq, const float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4)
        *(float4*)(row + 16 * i + 4 * cq) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
}
template <int V> __device__ __forceinline__ void get(const float* row, int cq, float (&v)[V]) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const float4 f = *(const float4*)(row + 16 * i + 4 * cq);
        v[i] = f.x; v[i + 1] = f.y; v[i + 2] = f.z; v[i + 3] = f.w;
    }
}
// the channel of a column of tile column block cb, and whether its lane owns it
template <int V, bool NARROW>
__device__ __forceinline__ int channel_of(int cb, int col, int D, bool* owned) {
    const Own o = own_of<V, NARROW>(cb * kLanes + col % 64 / 4, D);
    const int i = col / 64 * 4 + col % 4;
    *owned = o.has(i);
    return o.c0 + i;  // inside the row, if not NARROW
}

// ---- tiles, and the carry between them ----------------------------------------------------
constexpr int kBlockTiles = 16;  // tiles of a block of a chain, and blocks of a larger one
// Counters of tiles taken, each for a range of neighbouring chains and on a cache line of its
// own.  A counter serves one workgroup in about 9 ns: with one for all, the 512 workgroups
// that start together wait 5 us for their first number (8 x 1024 x 1536 in bf16: forward 24
// us, 17 with eight counters; backward 42 and 32).
constexpr unsigned kCounters = 8, kCounterWords = 64;

struct Tiles {
    unsigned* ticket;                  // the counters (null: one tile per chain)
    unsigned long long* span;          // [tile][C] the tile's P (low word) and H
    unsigned long long* block;         // [k / 16][chain][C] the same of 16 tiles
    unsigned* carry;                   // [k / 256][chain][C] carry out of 256 tiles
    const uint8_t* starts;             // packed rows: bit t: a sequence starts at step t
    const int* from;                   // and per byte of these: the first s with cu[s] >= 8 i
    int chains, blocks, nk;            // B * blocks, channel blocks, tiles of a chain
    unsigned groups;                   // counters in use
    unsigned* done;                    // d_bias: tiles of a channel block that are through
};

// A word not yet published has all bits set: a NaN that no published value can be, since a
// NaN is published as the one below.  A span is one 64-bit store, so it is seen whole, and
// nothing rests on the order of two stores.  All of these words are read and written at the
// device's scope, past the XCDs' own L2 caches.
constexpr unsigned kNotYet = 0xffffffffu;
__device__ __forceinline__ unsigned bits_of(float v) {
    return v == v ? __float_as_uint(v) : 0x7fc00000u;
}
// P is a product of values in [0, 1]; kCut: a sequence starts inside the span, so nothing from
// before reaches its end.
constexpr float kCut = -1.f;
__device__ __forceinline__ void publish(unsigned long long* p, float P, float H) {
    __hip_atomic_store(p, (unsigned long long)bits_of(H) << 32 | bits_of(P), __ATOMIC_RELAXED,
                       __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void extend(float& P, float& H, float p, float h) {
    H = p == kCut ? h : fmaf(p, H, h);
    P = p == kCut || P == kCut ? kCut : P * p;
}

// Fold n published spans, `step` words apart from s on, into (P, H), first to last.  A round of
// loads for kLook of them, and further rounds for those that were not there yet.
__device__ __forceinline__ void fold(const unsigned long long* s, size_t step, int n, float& P,
                                     float& H) {
    for (int m0 = 0; m0 < n; m0 += kLook, s += kLook * step) {
        unsigned long long w[kLook];
        unsigned missing = (1u << min(kLook, n - m0)) - 1;
        for (;;) {
#pragma unroll
            for (int m = 0; m < kLook; ++m)
                if (missing >> m & 1)
                    w[m] = __hip_atomic_load(s + m * step, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
            for (int m = 0; m < kLook; ++m)
                if ((missing >> m & 1) && __all((unsigned)w[m] != kNotYet)) missing &= ~(1u << m);
            if (!missing) break;
            __builtin_amdgcn_s_sleep(1);
        }
#pragma unroll
        for (int m = 0; m < kLook; ++m)
            if (m0 + m < n)
                extend(P, H, __uint_as_float((unsigned)w[m]),
                       __uint_as_float((unsigned)(w[m] >> 32)));
    }
}

// One wave, a lane for column col of the tile's C; (P, H): the tile's span (P = kCut where a
// sequence starts inside); first: the carry into the chain's first tile.  Publishes the
// tile's span, behind 16 tiles what those amount to, and behind 256 the carry out of them;
// returns the carry into this tile.  The order of combining is fixed by the tile's place
// alone (the carry into its 256 tiles, the blocks of 16 before its own, the tiles of its own
// block before it), never by what happens to be ready, so results are the same bits on every
// run.
template <int C>
__device__ __forceinline__ float carry_in(const Tiles& tl, unsigned tile, int k, int col, float P,
                                          float H, float first) {
    if (tl.nk == 1) return first;
    const bool last = k == tl.nk - 1;  // nobody looks at what it publishes
    const int i = k % kBlockTiles, nb = k / kBlockTiles % kBlockTiles;
    const int big = k / (kBlockTiles * kBlockTiles);
    const size_t step = (size_t)tl.chains * C;
    const size_t at = (size_t)(tile - (unsigned)k * tl.chains) * C + col;
    if (!last && i < kBlockTiles - 1) publish(tl.span + k * step + at, P, H);
    float bP = 1.f, bH = 0.f;  // the block up to this tile
    fold(tl.span + (k - i) * step + at, step, i, bP, bH);
    if (!last && i == kBlockTiles - 1 && nb < kBlockTiles - 1) {
        float p = bP, h = bH;
        extend(p, h, P, H);
        publish(tl.block + (k / kBlockTiles) * step + at, p, h);
    }
    float in = first;
    if (big > 0) {
        const unsigned* c = tl.carry + (big - 1) * step + at;
        unsigned v;
        while (!__all((v = __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)) !=
                      kNotYet))
            __builtin_amdgcn_s_sleep(1);
        in = __uint_as_float(v);
    }
    if (nb > 0) {
        float P16 = 1.f, H16 = 0.f;
        fold(tl.block + (k / kBlockTiles - nb) * step + at, step, nb, P16, H16);
        in = P16 == kCut ? H16 : fmaf(P16, in, H16);
    }
    in = bP == kCut ? bH : fmaf(bP, in, bH);
    if (!last && i == kBlockTiles - 1 && nb == kBlockTiles - 1)
        __hip_atomic_store(tl.carry + big * step + at, bits_of(P == kCut ? H : fmaf(P, in, H)),
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return in;
}

// The sequence of a packed row whose last step is t; from: any s up to it with cu[s] <= t + 1.
__device__ __forceinline__ int sequence_ending(const int* cu, int nseq, int from, int t) {
    int s = from;  // to the first with cu[s] = t + 1: empty sequences lie behind it
    while (s < nseq && cu[s] <= t) ++s;
    return max(s - 1, 0);
}

// Tiles are taken from the counter of the workgroup's group; a workgroup takes its next
// number while it works on a tile.
struct Group {
    unsigned* counter;
    unsigned first, chains, tiles;  // the group's chains, and their tiles
};
__device__ __forceinline__ Group group_of(const Tiles& tl) {
    const unsigned g = blockIdx.x % tl.groups, q = tl.chains / tl.groups,
                   rem = tl.chains % tl.groups;
    Group r;
    r.counter = tl.ticket + g * kCounterWords;
    r.first = g * q + min(g, rem);
    r.chains = q + (g < rem ? 1 : 0);
    r.tiles = r.chains * tl.nk;
    return r;
}

// The workgroup's first number, and the number after t (in thread 0; without a counter, where
// no tile waits for another, in all of them).
__device__ __forceinline__ unsigned first_number(const Tiles& tl, const Group& g, unsigned* sh) {
    if (!tl.ticket) return blockIdx.x / tl.groups;
    if (threadIdx.x == 0) *sh = g.tiles ? atomicAdd(g.counter, 1u) : 0u;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(*sh);
}
__device__ __forceinline__ unsigned take_number(const Tiles& tl, const Group& g, unsigned t) {
    if (!tl.ticket) return t + gridDim.x / tl.groups;
    return threadIdx.x == 0 ? atomicAdd(g.counter, 1u) : 0u;
}

// Which tile, and where this thread stands in it.
struct Place {
    unsigned tile;
    int k, b, cb, cq, r;
    Own o;
};
// t: the number taken (uniform)
template <int V, bool NARROW>
__device__ __forceinline__ Place place(const Tiles& tl, const Group& g, unsigned t, int D) {
    Place p;
    p.k = t / g.chains;
    const unsigned chain = g.first + t % g.chains;
    p.tile = p.k * tl.chains + chain;
    p.b = chain / tl.blocks;
    p.cb = chain % tl.blocks;
    p.cq = threadIdx.x % kLanes;
    p.r = threadIdx.x / kLanes;
    p.o = own_of<V, NARROW>(p.cb * kLanes + p.cq, D);
    return p;
}

// Where sequences of a packed row start and end among a run's steps.
struct RunSeqs {
    unsigned bits;  // of the starts, from the byte of the run's first step on
    int from;       // first sequence that starts in that byte or behind
    __device__ __forceinline__ void load(const Tiles& tl, int ts) {
        bits = tl.starts[ts >> 3] | (unsigned)tl.starts[(ts >> 3) + 1] << 8;
        from = tl.from[ts >> 3];
    }
    template <int S> __device__ __forceinline__ unsigned starts(int ts) const {
        return bits >> (ts & 7) & ((1u << S) - 1);
    }
    template <int S> __device__ __forceinline__ unsigned ends(int ts, int T) const {
        const unsigned e = bits >> (ts & 7) >> 1 & ((1u << S) - 1);
        return T - 1 >= ts && T - 1 < ts + S ? e | 1u << (T - 1 - ts) : e;
    }
};

// Byte offset of row `row` (of a tile) and channel c0 in rows `stride` elements apart: a
// tile's rows lie within 2^31 bytes, so an address is a scalar base plus 32 bits per lane.
template <typename T>
__device__ __forceinline__ uint32_t row_offset(int row, long long stride, int c0) {
    return ((uint32_t)row * (uint32_t)stride + (uint32_t)c0) * (uint32_t)sizeof(T);
}

// Load a run's pieces: step ts + j is the tile's row `run * S + j`; base: the tile's first
// row; rows: the tile's rows that exist (steps behind repeat the last one; the caller clears
// them).  No branch: one would make the loads of x wait for those of g.
template <typename T, int V, int S, bool NARROW, bool CACHED>
__device__ __forceinline__ void load_run(Piece<T, V> (&q)[S], const void* base, long long stride,
                                         int run, int rows, const Own& o) {
    const uint32_t last = row_offset<T>(rows - 1, stride, o.c0);
    uint32_t off = row_offset<T>(run * S, stride, o.c0);
    const uint32_t step = (uint32_t)stride * (uint32_t)sizeof(T);
#pragma unroll
    for (int j = 0; j < S; ++j, off += step) {
        const T* p = (const T*)((const char*)base + min(off, last));
        if (NARROW) q[j].load_part(p, o.hi);
        else if (CACHED) q[j].load_cached(p);
        else q[j].load(p);
    }
}

// Codes and scales of a run's pieces: the 64 channels of a group are 64 / V neighbouring
// lanes.  All of a wave's lanes take part.  row0: the tile's first row.
template <typename T, int V, int S>
__device__ __forceinline__ void pack_run(const Piece<T, V> (&v)[S], int8_t* codes, float* scales,
                                         const GatedFwdArgs& a, const Place& w, long long row0,
                                         int rows) {
    const int groups = (a.D + SSD_CKPT_GROUP - 1) / SSD_CKPT_GROUP;
    codes += row0 * a.D;
    scales += row0 * groups;
    const int piece = w.cb * kLanes + w.cq;
    const uint32_t at = (uint32_t)(w.r * S) * (uint32_t)a.D + (uint32_t)w.o.c0;
    const uint32_t sat =
        (uint32_t)(w.r * S) * (uint32_t)groups + (uint32_t)(piece * V / SSD_CKPT_GROUP);
#pragma unroll
    for (int j = 0; j < S; ++j) {
        float f[V];
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = v[j].get(i);
        if (w.o.hi - w.o.lo != V) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (!w.o.has(i)) f[i] = 0.f;  // another group's
        }
#pragma unroll
        for (int i = 0; i < V; ++i) most = max(most, __float_as_uint(f[i]) & 0x7fffffffu);
        const CkptScale s(ckpt_group_max<SSD_CKPT_GROUP / V>(most));
        if (w.r * S + j >= rows || !w.o.any()) continue;
        if (piece * V % SSD_CKPT_GROUP == 0) (scales + j * groups)[sat] = s.scale;
        ckpt_store<V>(codes + (long long)j * a.D + at, f, s, w.o.lo, w.o.hi);
    }
}

// A kernel's one argument.  FRESH: read anew where it is asked for, from the start of the
// segment that kernel arguments lie in.  Kept over a whole tile, its fields and what is made
// of them take more scalar registers than there are, and those that do not fit cost vector
// instructions and registers; read anew, the next access waits for a scalar load.
// In us, kept and read anew:
//   FRESH  forward with codes: the training pass from codes at 8 x 2048 x 1536 in bf16 118, 113;
//          backward in bf16: 4 x 4096 x 5120 equal, a packed row of 16384 x 2048 102, 100
//   not    forward without codes: 4 x 4096 x 5120 in bf16 99, 113; backward in fp32: a packed
//          row of 5001 x 1280 40, 42
template <bool FRESH, typename A> __device__ __forceinline__ A args(const A& in) {
    if (!FRESH) return in;
    static_assert(sizeof(A) % 8 == 0, "copied in words of 64 bits");
    typedef const uint64_t __attribute__((address_space(4))) Word;
    Word* p = (Word*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    union { A a; uint64_t w[sizeof(A) / 8]; } u;
#pragma unroll
    for (unsigned i = 0; i < sizeof(A) / 8; ++i) u.w[i] = p[i];
    return u.a;
}
struct FwdParams {
    GatedFwdArgs a;
    Tiles tl;
};
struct BwdParams {
    GatedBwdArgs a;
    Tiles tl;
    float* part;  // d_bias' sums of the tiles, or null
};

// threadIdx.x, computed anew in every iteration: the addresses that follow from it would
// otherwise be kept over the whole loop, in more registers than there are.
__device__ __forceinline__ int fresh_thread() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// ---- forward ------------------------------------------------------------------------------
template <typename T, int V, int S, bool PACKED, bool CODES, bool NARROW, bool CACHED>
__global__ __launch_bounds__(kRuns * kLanes, 4) void gated_fwd_kernel(FwdParams in) {
    constexpr bool FRESH = CODES;
    constexpr int C = kLanes * V, kTile = kRuns * S;
    __shared__ __align__(16) float sP[kRuns * C], sH[kRuns * C], sE[C];
    __shared__ unsigned sFirst, sNext, sCut[kRuns];
    Group group;
    unsigned t;
    {
        const Tiles tl = args<FRESH>(in).tl;
        group = group_of(tl);
        t = first_number(tl, group, &sFirst);
    }
    if (t >= group.tiles) return;
    Place w;
    Piece<T, V> x[S], g[S];
    float bias[V];
    RunSeqs seqs;
    auto fetch = [&]() {
        const FwdParams p = args<FRESH>(in);
        const GatedFwdArgs& a = p.a;
        const Tiles& tl = p.tl;
        w = place<V, NARROW>(tl, group, t, a.D);
        const int t0 = w.k * kTile, rows = min(kTile, a.T - t0);
        if (PACKED) seqs.load(tl, t0 + w.r * S);
        const long long row0 = (long long)w.b * a.T + t0;
        load_f32<V, NARROW>(bias, a.bias ? a.bias + w.o.c0 : nullptr, w.o);
        load_run<T, V, S, NARROW, CACHED>(g, (const T*)a.g + row0 * a.g_stride, a.g_stride,
                                          w.r, rows, w.o);
        load_run<T, V, S, NARROW, CACHED>(x, (const T*)a.x + row0 * a.x_stride, a.x_stride,
                                          w.r, rows, w.o);
    };
    fetch();
    for (;;) {
        const int tid = fresh_thread();
        const FwdParams p1 = args<FRESH>(in);
        const GatedFwdArgs& a = p1.a;
        const Tiles& tl = p1.tl;
        const int t0 = w.k * kTile, ts = t0 + w.r * S;
        const int rows = min(kTile, a.T - t0);
        const bool whole = rows == kTile;
        const long long row0 = (long long)w.b * a.T + t0;  // of the tile
        const unsigned taken = take_number(tl, group, t);
        unsigned starts = 0, ends = 0;
        const int from = PACKED ? seqs.from : 0;
        if (PACKED) {
            starts = seqs.template starts<S>(ts);
            ends = seqs.template ends<S>(ts, a.T);
            if (w.cq == 0) sCut[w.r] = starts;
        }
        float q[S][V];
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] *= kLog2e;
#pragma unroll
        for (int j = 0; j < S; ++j) {
#pragma unroll
            for (int i = 0; i < V; ++i) q[j][i] = gate_q(fmaf(g[j].get(i), kLog2e, bias[i]));
        }
        if (CODES) pack_run<T, V, S>(g, a.g_codes, a.g_scales, a, w, row0, rows);
        if (!whole) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (ts + j >= a.T) {
                    x[j].clear();
#pragma unroll
                    for (int i = 0; i < V; ++i) q[j][i] = 0.f;
                }
        }
        {
            float P[V], H[V];
#pragma unroll
            for (int i = 0; i < V; ++i) P[i] = 1.f, H[i] = 0.f;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                if (PACKED && (starts >> j & 1)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) P[i] = H[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    H[i] = gate_step(q[j][i], x[j].get(i), H[i]);
                    P[i] = fmaf(-q[j][i], P[i], P[i]);
                }
            }
            put<V>(&sP[w.r * C], w.cq, P);
            put<V>(&sH[w.r * C], w.cq, H);
        }
        if (tid == 0) sNext = taken;
        __syncthreads();
        const unsigned next = __builtin_amdgcn_readfirstlane(sNext);
        unsigned cuts = 0;
        if (PACKED)
            cuts = (unsigned)__ballot((tid & 63) < kRuns && sCut[tid % kRuns] != 0);
        if (tid < C) {
            const int col = tid;
            float accP = 1.f, accH = 0.f;
#pragma unroll
            for (int r0 = 0; r0 < kRuns; r0 += kScan) {
                float p[kScan], h[kScan];
#pragma unroll
                for (int r = 0; r < kScan; ++r) {
                    p[r] = sP[(r0 + r) * C + col];
                    h[r] = sH[(r0 + r) * C + col];
                }
#pragma unroll
                for (int r = 0; r < kScan; ++r) {
                    sP[(r0 + r) * C + col] = accP;
                    sH[(r0 + r) * C + col] = accH;
                    const bool cut = PACKED && (cuts >> (r0 + r) & 1);
                    accH = cut ? h[r] : fmaf(p[r], accH, h[r]);
                    accP *= p[r];
                }
            }
            const FwdParams p2 = args<FRESH>(in);
            const GatedFwdArgs& a = p2.a;
            const Tiles& tl = p2.tl;
            bool owned;
            const int c = channel_of<V, NARROW>(w.cb, col, a.D, &owned);
            const float first =
                a.init && w.k < kBlockTiles * kBlockTiles && c < a.D
                    ? a.init[(long long)w.b * a.D + c]
                    : 0.f;
            sE[col] = carry_in<C>(tl, w.tile, w.k, col, cuts ? kCut : accP, accH, first);
        } else if (CODES) {  // meanwhile
            pack_run<T, V, S>(x, a.x_codes, a.x_scales, a, w, row0, rows);
        }
        __syncthreads();
        if (CODES && tid < C)
            pack_run<T, V, S>(x, a.x_codes, a.x_scales, a, w, row0, rows);
        float h[V];
        {
            float p[V], e[V];
            get<V>(&sH[w.r * C], w.cq, h);
            get<V>(&sP[w.r * C], w.cq, p);
            get<V>(sE, w.cq, e);
            const bool cut = PACKED && (cuts & ((1u << w.r) - 1));
#pragma unroll
            for (int i = 0; i < V; ++i) h[i] = cut ? h[i] : fmaf(p[i], e[i], h[i]);
        }
        if (w.o.any()) {
            const FwdParams p3 = args<FRESH>(in);
            const GatedFwdArgs& a = p3.a;
            if (a.entry && ts % kGatedChunk == 0 && ts < a.T) {
                const long long nC = (a.T + kGatedChunk - 1) / kGatedChunk;
                store<float, V>(a.entry + (w.b * nC + ts / kGatedChunk) * a.D + w.o.c0, h, w.o);
            }
            char* const out = (char*)((T*)a.h + row0 * a.D);
            uint32_t off = row_offset<T>(w.r * S, a.D, w.o.c0);
#pragma unroll
            for (int j = 0; j < S; ++j, off += a.D * (uint32_t)sizeof(T)) {
                if (PACKED && (starts >> j & 1)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) h[i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) h[i] = gate_step(q[j][i], x[j].get(i), h[i]);
                if (whole || ts + j < a.T) store<T, V>((T*)(out + off), h, w.o);
                if (PACKED && a.final_state && (ends >> j & 1)) {
                    const long long seq = sequence_ending(a.cu, a.nseq, from, ts + j);
                    store<float, V>(a.final_state + seq * a.D + w.o.c0, h, w.o);
                }
            }
            if (!PACKED && a.final_state && ts <= a.T - 1 && a.T - 1 < ts + S)
                store<float, V>(a.final_state + (long long)w.b * a.D + w.o.c0, h, w.o);
        }
        t = next;
        if (t >= group.tiles) break;
        fetch();
        __syncthreads();  // LDS is free again
    }
}

// ---- backward -----------------------------------------------------------------------------
// the sum over the four rows of 16 lanes of a wave, in all of them
__device__ __forceinline__ float row_sum(float v) {
    unsigned u = __float_as_uint(v);
    auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    u = __float_as_uint(__uint_as_float(p[0]) + __uint_as_float(p[1]));
    p = __builtin_amdgcn_permlane32_swap(u, u, false, false);
    return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

// x and g of a run, from rows in T or from 8-bit codes and their scales.
template <typename T, int V, int S, bool CODES, bool NARROW, bool CACHED> struct RunIn;
template <typename T, int V, int S, bool NARROW, bool CACHED>
struct RunIn<T, V, S, false, NARROW, CACHED> {
    Piece<T, V> v[S];
    __device__ __forceinline__ void load(const void* from, long long stride, const int8_t*,
                                         const float*, long long row0, int rows, const Place& w,
                                         int) {
        load_run<T, V, S, NARROW, CACHED>(v, (const T*)from + row0 * stride, stride, w.r, rows,
                                          w.o);
    }
    __device__ __forceinline__ float get(int j, int i) const { return v[j].get(i); }
    __device__ __forceinline__ void clear(int j) { v[j].clear(); }
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int j = 0; j < S; ++j) v[j].renew();
    }
};
template <typename T, int V, int S, bool NARROW, bool CACHED>
struct RunIn<T, V, S, true, NARROW, CACHED> {
    CkptPiece<V> v[S];
    float s[S];
    __device__ __forceinline__ void load(const void*, long long, const int8_t* codes,
                                         const float* scales, long long row0, int rows,
                                         const Place& w, int D) {
        const int groups = (D + SSD_CKPT_GROUP - 1) / SSD_CKPT_GROUP;
        codes += row0 * D;
        scales += row0 * groups;
        const uint32_t group =
            min((w.cb * kLanes + w.cq) * V / SSD_CKPT_GROUP, groups - 1);
        const uint32_t last = (uint32_t)(rows - 1) * (uint32_t)D + (uint32_t)w.o.c0;
        const uint32_t slast = (uint32_t)(rows - 1) * (uint32_t)groups + group;
        uint32_t at = (uint32_t)(w.r * S) * (uint32_t)D + (uint32_t)w.o.c0;
        uint32_t sat = (uint32_t)(w.r * S) * (uint32_t)groups + group;
#pragma unroll
        for (int j = 0; j < S; ++j, at += D, sat += groups) {
            const int8_t* p = codes + min(at, last);
            if (NARROW) v[j].load_part(p, w.o.hi);
            else v[j].load(p);
            s[j] = scales[min(sat, slast)];
        }
    }
    __device__ __forceinline__ float get(int j, int i) const { return v[j].get(i) * s[j]; }
    __device__ __forceinline__ void clear(int j) { v[j].clear(); s[j] = 0.f; }
    __device__ __forceinline__ void again() {
#pragma unroll
        for (int j = 0; j < S; ++j) v[j].renew();
    }
};

template <typename T, int V, int S, bool PACKED, bool CODES, bool NARROW, bool CACHED>
__global__ __launch_bounds__(kRuns * kLanes, 4) void gated_bwd_kernel(BwdParams in) {
    constexpr bool FRESH = sizeof(T) == 2;
    constexpr int C = kLanes * V, kTile = kRuns * S;
    constexpr int kChunkRuns = kGatedChunk / S;
    static_assert(kTile % kGatedChunk == 0 && kRuns * kLanes >= 3 * C, "tiles hold whole chunks");
    constexpr int kWaves = kRuns * kLanes / 64;
    __shared__ __align__(16) float sP[kRuns * C], sH[kRuns * C], sC[kRuns * C], sR[kRuns * C];
    __shared__ __align__(16) float sE[C];
    __shared__ __align__(16) float sD[kWaves * C];  // d_bias' share of every wave
    __shared__ unsigned sFirst, sNext, sCut[kRuns];
    Group group;
    unsigned t;
    bool sums;  // d_bias is wanted
    {
        const BwdParams p = args<FRESH>(in);
        sums = p.part != nullptr;
        group = group_of(p.tl);
        t = first_number(p.tl, group, &sFirst);
    }
    if (t >= group.tiles) return;
    Place w;
    RunIn<T, V, S, CODES, NARROW, CACHED> x, g;
    Piece<T, V> dh[S];
    float bias[V];
    RunSeqs seqs;
    auto fetch = [&]() {
        const BwdParams p = args<FRESH>(in);
        const GatedBwdArgs& a = p.a;
        const Tiles& tl = p.tl;
        w = place<V, NARROW>(tl, group, t, a.D);
        const int t0 = (tl.nk - 1 - w.k) * kTile, rows = min(kTile, a.T - t0);  // last tile first
        if (PACKED) seqs.load(tl, t0 + w.r * S);
        const long long row0 = (long long)w.b * a.T + t0;
        load_f32<V, NARROW>(bias, a.bias ? a.bias + w.o.c0 : nullptr, w.o);
        g.load(a.g, a.g_stride, a.g_codes, a.g_scales, row0, rows, w, a.D);
        x.load(a.x, a.x_stride, a.x_codes, a.x_scales, row0, rows, w, a.D);
        load_run<T, V, S, NARROW, CACHED>(dh, (const T*)a.dh + row0 * a.dh_stride, a.dh_stride,
                                          w.r, rows, w.o);
    };
    Place before;  // the tile whose shares of d_bias are in sD
    before.k = -1;
    // one wave; with tl.done the last tile of the channel block adds up all of them
    auto sum_up = [&](int col) {
        const BwdParams p = args<FRESH>(in);
        const GatedBwdArgs& a = p.a;
        const Tiles& tl = p.tl;
        float* const part = p.part;
        bool owned;
        const int c = channel_of<V, NARROW>(before.cb, col, a.D, &owned);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) s += sD[i * C + col];
        const int tiles = a.B * tl.nk;
        unsigned* to = (unsigned*)part + ((long long)before.b * tl.nk + tl.nk - 1 - before.k) * a.D;
        if (!tl.done) {
            if (owned) to[c] = __float_as_uint(s);
            return;
        }
        if (owned)
            __hip_atomic_store(to + c, bits_of(s), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        unsigned through = 0;
        if (col == 0) through = atomicAdd(tl.done + before.cb, 1u);
        if ((int)__builtin_amdgcn_readfirstlane(through) != tiles - 1) return;
        // the others' sums are there, or stored and on their way
        const unsigned* from = (const unsigned*)part + c;
        s = 0.f;
        for (int r0 = 0; r0 < tiles; r0 += 8) {
            unsigned v[8];
            for (;;) {
                bool all = true;
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    v[r] = owned && r0 + r < tiles
                               ? __hip_atomic_load(from + (long long)(r0 + r) * a.D,
                                                   __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT)
                               : 0u;
#pragma unroll
                for (int r = 0; r < 8; ++r) all = all && v[r] != kNotYet;
                if (__all(all)) break;
                __builtin_amdgcn_s_sleep(1);
            }
#pragma unroll
            for (int r = 0; r < 8; ++r) s += __uint_as_float(v[r]);
        }
        if (owned) a.d_bias[c] = s;
    };
    fetch();
    for (;;) {
        const int tid = fresh_thread();
        const BwdParams p1 = args<FRESH>(in);
        const GatedBwdArgs& a = p1.a;
        const Tiles& tl = p1.tl;
        const int kt = tl.nk - 1 - w.k;
        const int t0 = kt * kTile, ts = t0 + w.r * S;
        const int rows = min(kTile, a.T - t0);
        const bool whole = rows == kTile;
        const long long row0 = (long long)w.b * a.T + t0;  // of the tile
        const unsigned taken = take_number(tl, group, t);
#pragma unroll
        for (int i = 0; i < V; ++i) bias[i] *= kLog2e;
        unsigned starts = 0, ends = 0;
        const int from = PACKED ? seqs.from : 0;
        if (PACKED) {
            starts = seqs.template starts<S>(ts);
            ends = seqs.template ends<S>(ts, a.T);
            if (w.cq == 0) sCut[w.r] = starts;
        }
        if (!whole) {
#pragma unroll
            for (int j = 0; j < S; ++j)
                if (ts + j >= a.T) {
                    x.clear(j);
                    dh[j].clear();
                }
        }
        // d_final of a packed sequence that ends at step j of this run
        auto ending = [&](int j, float (&v)[V]) {
            const BwdParams p = args<FRESH>(in);
            const GatedBwdArgs& a = p.a;
            const float* d = nullptr;
            if (a.d_final) {
                const long long seq = sequence_ending(a.cu, a.nseq, from, ts + j);
                d = a.d_final + seq * a.D + w.o.c0;
            }
            load_f32<V, NARROW>(v, d, w.o);
        };
        {
            // G's carry out of the run in the same sweep: dh_j reaches it through the product
            // of a up to j; behind the run's first start nothing does
            float P[V], H[V], G[V], kept[V];
            bool cut = false;
#pragma unroll
            for (int i = 0; i < V; ++i) P[i] = 1.f, H[i] = G[i] = 0.f;
#pragma unroll
            for (int j = 0; j < S; ++j) {
                if (PACKED && (starts >> j & 1)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        kept[i] = cut ? kept[i] : G[i];
                        H[i] = 0.f;
                    }
                    cut = true;
                }
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    float q = gate_q(fmaf(g.get(j, i), kLog2e, bias[i]));
                    if (!whole && ts + j >= a.T) q = 0.f;
                    H[i] = gate_step(q, x.get(j, i), H[i]);
                    P[i] = fmaf(-q, P[i], P[i]);
                    G[i] = fmaf(P[i], dh[j].get(i), G[i]);
                }
                if (PACKED && !cut && (ends >> j & 1)) {
                    float v[V];
                    ending(j, v);
#pragma unroll
                    for (int i = 0; i < V; ++i) G[i] = fmaf(P[i], v[i], G[i]);
                }
            }
            if (PACKED && cut) {
#pragma unroll
                for (int i = 0; i < V; ++i) G[i] = kept[i];
            }
            put<V>(&sP[w.r * C], w.cq, P);
            put<V>(&sH[w.r * C], w.cq, H);
            put<V>(&sC[w.r * C], w.cq, G);
        }
        if (tid == 0) sNext = taken;
        __syncthreads();
        const unsigned next = __builtin_amdgcn_readfirstlane(sNext);
        unsigned cuts = 0;
        if (PACKED)
            cuts = (unsigned)__ballot((tid & 63) < kRuns && sCut[tid % kRuns] != 0);
        if (tid < C) {  // the first waves: G, last run first
            const int col = tid;
            float accP = 1.f, accC = 0.f;
#pragma unroll
            for (int r0 = kRuns - kScan; r0 >= 0; r0 -= kScan) {
                float p[kScan], v[kScan];
#pragma unroll
                for (int r = 0; r < kScan; ++r) {
                    p[r] = sP[(r0 + r) * C + col];
                    v[r] = sC[(r0 + r) * C + col];
                }
#pragma unroll
                for (int r = kScan - 1; r >= 0; --r) {
                    sR[(r0 + r) * C + col] = accP;
                    sC[(r0 + r) * C + col] = accC;
                    const bool cut = PACKED && (cuts >> (r0 + r) & 1);
                    accC = cut ? v[r] : fmaf(p[r], accC, v[r]);
                    accP *= p[r];
                }
            }
            const BwdParams p2 = args<FRESH>(in);
            const GatedBwdArgs& a = p2.a;
            const Tiles& tl = p2.tl;
            bool owned;
            const int c = channel_of<V, NARROW>(w.cb, col, a.D, &owned);
            const float first =
                !PACKED && a.d_final && w.k < kBlockTiles * kBlockTiles && c < a.D
                    ? a.d_final[(long long)w.b * a.D + c]
                    : 0.f;
            sE[col] = carry_in<C>(tl, w.tile, w.k, col, cuts ? kCut : accP, accC, first);
        } else if (tid < 2 * C) {  // the next: h, from every chunk's entry state
            const int col = tid - C;
            const BwdParams p2 = args<FRESH>(in);
            const GatedBwdArgs& a = p2.a;
            bool owned;
            const int c = channel_of<V, NARROW>(w.cb, col, a.D, &owned);
            const int nC = (a.T + kGatedChunk - 1) / kGatedChunk;
            float E[kTile / kGatedChunk];
#pragma unroll
            for (int k = 0; k < kTile / kGatedChunk; ++k) {
                const int chunk = t0 / kGatedChunk + k;
                E[k] = chunk < nC && c < a.D ? a.entry[((long long)w.b * nC + chunk) * a.D + c]
                                             : 0.f;
            }
#pragma unroll
            for (int k = 0; k < kTile / kGatedChunk; ++k) {
                float e = E[k];
#pragma unroll
                for (int r = k * kChunkRuns; r < (k + 1) * kChunkRuns; ++r) {
                    const float p = sP[r * C + col], v = sH[r * C + col];
                    sH[r * C + col] = e;
                    e = PACKED && (cuts >> r & 1) ? v : fmaf(p, e, v);
                }
            }
        } else if (tid < 3 * C) {
            if (sums && before.k >= 0) sum_up(tid - 2 * C);
        }
        __syncthreads();
        float h[V], G[V], db[V];
        {
            float p[V], in[V];
            get<V>(&sH[w.r * C], w.cq, h);
            get<V>(&sC[w.r * C], w.cq, G);
            get<V>(&sR[w.r * C], w.cq, p);
            get<V>(sE, w.cq, in);
            const bool cut = PACKED && w.r < kRuns - 1 && (cuts >> (w.r + 1));
#pragma unroll
            for (int i = 0; i < V; ++i) {
                G[i] = cut ? G[i] : fmaf(p[i], in[i], G[i]);
                db[i] = 0.f;
            }
        }
        g.again();
        x.again();
#pragma unroll
        for (int j = 0; j < S; ++j) dh[j].renew();
        float off[S][V];  // h_{t-1} - x_t
#pragma unroll
        for (int j = 0; j < S; ++j) {
            if (PACKED && (starts >> j & 1)) {
#pragma unroll
                for (int i = 0; i < V; ++i) h[i] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
                off[j][i] = h[i] - x.get(j, i);
                if (j < S - 1) {
                    const float q = gate_q(fmaf(g.get(j, i), kLog2e, bias[i]));
                    h[i] = fmaf(-q, off[j][i], h[i]);
                }
            }
        }
        g.again();
        const BwdParams p3 = args<FRESH>(in);
        const uint32_t dx_step = (uint32_t)p3.a.dx_stride * (uint32_t)sizeof(T);
        const uint32_t dg_step = (uint32_t)p3.a.dg_stride * (uint32_t)sizeof(T);
        char* const to_dx = (char*)((T*)p3.a.dx + row0 * p3.a.dx_stride);
        char* const to_dg = (char*)((T*)p3.a.dg + row0 * p3.a.dg_stride);
        uint32_t dx_off = row_offset<T>(w.r * S + S - 1, p3.a.dx_stride, w.o.c0);
        uint32_t dg_off = row_offset<T>(w.r * S + S - 1, p3.a.dg_stride, w.o.c0);
#pragma unroll
        for (int j = S - 1; j >= 0; --j, dx_off -= dx_step, dg_off -= dg_step) {
            if (PACKED && (ends >> j & 1)) ending(j, G);
            if (whole || ts + j < a.T) {
                float dx[V], dg[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const Gate e(fmaf(g.get(j, i), kLog2e, bias[i]));
                    const float v = dh[j].get(i) + G[i];
                    dx[i] = e.q * v;
                    dg[i] = dx[i] * e.a * off[j][i];
                    db[i] += dg[i];
                    G[i] = fmaf(-e.q, v, v);
                }
                store<T, V>((T*)(to_dx + dx_off), dx, w.o);
                store<T, V>((T*)(to_dg + dg_off), dg, w.o);
                if (PACKED && (starts >> j & 1)) {
#pragma unroll
                    for (int i = 0; i < V; ++i) G[i] = 0.f;
                }
            }
        }
        if (!PACKED && p3.a.d_init && ts == 0)
            store<float, V>(p3.a.d_init + (long long)w.b * p3.a.D + w.o.c0, G, w.o);
        if (sums) {  // the wave's four runs; summed up during the next tile's scan
#pragma unroll
            for (int i = 0; i < V; ++i) db[i] = row_sum(db[i]);
            if (tid % 64 < kLanes) put<V>(&sD[tid / 64 * C], w.cq, db);
            before = w;
        }
        t = next;
        if (t >= group.tiles) break;
        fetch();
        __syncthreads();  // LDS is free again
    }
    if (sums) {
        __syncthreads();
        if (threadIdx.x < C) sum_up(threadIdx.x);
    }
}

// ---- small kernels ------------------------------------------------------------------------
constexpr int kThreads = 256;
constexpr int kStepVec = 4;
constexpr int kPrepSeqs = 2048;

// Before a pass: the counters cleared, spans and carries marked missing, the start bits of a
// packed row, and zero final states for its empty sequences.
// Cached stores: non-temporal ones took 1 us longer (4 x 4096 x 5120, 2.8 MB).
struct Prep {
    unsigned* clear;       // counters, then spans and carries: words to set
    long long zeros, words;  // the first to 0, the others to kNotYet
    uint8_t* starts;       // null: not a packed row
    int* from;
    int bytes;             // of starts; words of from
    const int* cu;
    int nseq, T, D;
    float* final_state;    // null: none
};
__global__ __launch_bounds__(kThreads) void gated_prep_kernel(Prep p) {
    __shared__ int sCu[kPrepSeqs];
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long all = (long long)gridDim.x * kThreads;
    for (long long i = id; i < p.words / 4; i += all)
        reinterpret_cast<Words<4>*>(p.clear)[i] =
            i < p.zeros / 4 ? Words<4>{0, 0, 0, 0} : Words<4>{~0u, ~0u, ~0u, ~0u};
    if (!p.starts) return;
    auto mark = [&](const int* cu) {
        for (long long i = id; i < p.bytes; i += all) {
            int lo = 0, hi = p.nseq;  // first s with cu[s] >= 8 i
            while (lo < hi) {
                const int m = (lo + hi) / 2;
                if (cu[m] >= 8 * i) hi = m; else lo = m + 1;
            }
            unsigned bits = 0;
            for (int s = lo; s < p.nseq && cu[s] < 8 * i + 8; ++s)
                if (cu[s + 1] > cu[s]) bits |= 1u << (cu[s] - 8 * i);
            p.starts[i] = (uint8_t)bits;
            p.from[i] = lo;
        }
    };
    if (p.nseq < kPrepSeqs) {  // the search's steps wait for LDS then, not for memory
        for (int i = threadIdx.x; i <= p.nseq; i += kThreads) sCu[i] = p.cu[i];
        __syncthreads();
        mark(sCu);
    } else {
        mark(p.cu);
    }
    if (!p.final_state) return;
    for (long long i = id; i < (long long)p.nseq * p.D; i += all) {
        const int s = (int)(i / p.D);
        if (p.cu[s + 1] <= p.cu[s]) p.final_state[i] = 0.f;
    }
}

// d_bias from the tiles' sums, where there are many: a workgroup per 32 channels, 8 threads
// per channel; fixed order.
__global__ __launch_bounds__(kThreads) void gated_dbias_kernel(const float* part, float* d_bias,
                                                               int rows, int D) {
    __shared__ float s[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    float v = 0.f;
    if (c < D)
#pragma unroll 8
        for (int r = w; r < rows; r += 8) v += part[(long long)r * D + c];
    s[w][lane] = v;
    __syncthreads();
    if (w != 0 || c >= D) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) v += s[i][lane];
    d_bias[c] = v;
}

__global__ __launch_bounds__(kThreads) void gated_carry_kernel(const float* src, float* dst,
                                                               long long n) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id < n) dst[id] = src ? src[id] : 0.f;
}

// One thread per piece of four channels of a row.  Cached accesses: the state comes back at
// the next step.
template <typename T, bool NARROW>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedStepArgs a, unsigned pieces) {
    constexpr int V = kStepVec;
    const unsigned id = blockIdx.x * kThreads + threadIdx.x;
    const unsigned b = id / pieces;
    if (b >= (unsigned)a.B) return;
    const Own o = own_of<V, NARROW>(id % pieces, a.D);
    const T* xp = (const T*)a.x + b * a.x_stride + o.c0;
    const T* gp = (const T*)a.g + b * a.g_stride + o.c0;
    float* sp = a.state + (long long)b * a.D + o.c0;
    T* hp = (T*)a.h + (long long)b * a.D + o.c0;
    Piece<T, V> x, g;
    if (NARROW) {
        x.load_part(xp, o.hi);
        g.load_part(gp, o.hi);
    } else {
        x.load_cached(xp);
        g.load_cached(gp);
    }
    float bias[V], s[V];
    load_f32<V, NARROW>(bias, a.bias ? a.bias + o.c0 : nullptr, o);
    load_f32<V, NARROW>(s, sp, o);
#pragma unroll
    for (int i = 0; i < V; ++i)
        s[i] = gate_step(gate_q(fmaf(g.get(i), kLog2e, bias[i] * kLog2e)), x.get(i), s[i]);
    store<float, V, true>(sp, s, o);
    store<T, V, true>(hp, s, o);
}

unsigned blocks_of(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

// ---- workspace: counters | spans (and d_bias' sums) | start bits, sequences | (d_bias' sums) --
struct Layout {
    int nk, blocks;
    bool fused;                        // the last tile of a channel block makes d_bias
    long long tiles, spans, carries;  // tiles; spans of one and of 16; carries
    // sizes of what prep clears to zero, of all that it sets, of the start bits; offset of
    // d_bias' sums; total
    size_t zeros, clear, starts, part, bytes;
};
constexpr size_t kCounterBytes = kCounters * kCounterWords * 4;
// d_bias from its tiles' sums: with so many tiles to a channel block or fewer the last one adds
// them up (2 x 1003 x 1001 in fp32, 16 tiles: 17.0 us, 19.1 with a kernel of its own), behind
// that a kernel of its own does (4 x 4096 x 5120, 64 tiles: 188 and 183; 32 tiles: equal).
constexpr long long kFusedTiles = 16;
size_t up256(size_t v) { return (v + 255) / 256 * 256; }
// tiles of `steps` steps and `cols` channels
Layout layout(int B, int T, int D, int steps, int cols, bool bwd) {
    Layout l;
    l.nk = (T + steps - 1) / steps;
    l.blocks = (D + cols - 1) / cols;
    l.tiles = (long long)B * l.blocks * l.nk;
    const long long chains = (long long)B * l.blocks, rows = (long long)B * l.nk;
    l.spans = l.tiles + chains * (l.nk / kBlockTiles);
    l.carries = (chains * (l.nk / (kBlockTiles * kBlockTiles)) + 3) / 4 * 4;
    l.fused = bwd && l.nk > 1 && rows <= kFusedTiles;
    l.zeros = kCounterBytes + (l.fused ? up256((size_t)l.blocks * sizeof(unsigned)) : 0);
    const size_t sums = up256((size_t)rows * D * sizeof(float));
    l.clear = l.zeros + (l.nk > 1 ? up256((size_t)(l.spans * 2 + l.carries) * cols * 4) : 0);
    l.part = l.clear;
    if (l.fused) l.clear += sums;
    l.starts = up256((size_t)l.nk * ((steps + 7) / 8) + 1);
    if (!l.fused) l.part = l.clear + l.starts * 5;
    l.bytes = l.clear + l.starts * 5 + (bwd && !l.fused ? sums : 0);
    return l;
}
Layout fwd_layout(ssd_dtype t, bool codes, int B, int T, int D) {
    return layout(B, T, D, kRuns * fwd_steps(t, codes), kLanes * fwd_vec(t, codes), false);
}
Layout bwd_layout(ssd_dtype t, int B, int T, int D) {
    return layout(B, T, D, kRuns * bwd_steps(t), kLanes * kBwdVec, true);
}
Tiles tiles_of(const Layout& l, int B, int cols, char* ws, bool packed) {
    Tiles t = {};
    t.blocks = l.blocks;
    t.chains = B * l.blocks;
    t.nk = l.nk;
    // as many counters as share the chains out evenly, or nearly so
    t.groups = kCounters;
    while (t.chains % t.groups != 0 && t.chains < 8 * (int)t.groups) --t.groups;
    if (l.nk > 1) t.ticket = (unsigned*)ws;
    if (l.fused) t.done = (unsigned*)(ws + kCounterBytes);
    t.span = (unsigned long long*)(ws + l.zeros);
    t.block = t.span + l.tiles * cols;
    t.carry = (unsigned*)(t.span + l.spans * cols);
    if (packed) {
        t.starts = (const uint8_t*)(ws + l.clear);
        t.from = (const int*)(ws + l.clear + l.starts);
    }
    return t;
}
hipError_t prepare(const Layout& l, char* ws, const int* cu, int nseq, int T, int D,
                   float* final_state, hipStream_t st) {
    if (l.nk <= 1 && !cu) return hipSuccess;
    Prep p = {};
    p.clear = (unsigned*)ws;
    p.zeros = (long long)(l.zeros / 4);
    p.words = (long long)(l.clear / 4);
    long long work = p.words / 4;
    if (cu) {
        p.starts = (uint8_t*)(ws + l.clear);
        p.bytes = (int)l.starts;
        p.from = (int*)(ws + l.clear + l.starts);
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
    size_t most = 0;
    for (ssd_dtype t : {SSD_F32, SSD_BF16})
        for (const Layout& l : {fwd_layout(t, false, B, T, D), fwd_layout(t, true, B, T, D),
                                bwd_layout(t, B, T, D)})
            if (l.bytes > most) most = l.bytes;
    return most;
}

namespace {
// As many workgroups as are resident at once, and no more per counter than its tiles.
template <auto kern, typename Params>
hipError_t launch_tiles(const Params& p, hipStream_t st) {
    const Tiles& tl = p.tl;
    static DeviceSlots slots;
    int grid = 0;
    const hipError_t e =
        resident_grid((const void*)kern, kRuns * kLanes, 0, slots, &grid);
    if (e != hipSuccess) return e;
    const long long most =
        ((long long)tl.chains + tl.groups - 1) / tl.groups * tl.nk * tl.groups;
    if (grid > most) grid = (int)most;
    grid -= grid % tl.groups;
    kern<<<grid, kRuns * kLanes, 0, st>>>(p);
    return hipGetLastError();
}

// Cached loads where all rows of the call (`tensors` of them) take at most half of the 256 MB
// cache between the L2s and HBM: its inputs were often made just before, and are there still.
// In bf16, cached and non-temporal: 8 x 1024 x 1536 (75 MB) forward 17.3 and 21.2 us, (126 MB)
// backward 32.4 and 36.7; 16384 x 2048 (336 MB) packed backward 103 and 101; 4 x 4096 x 5120
// (503, 839 MB) forward 101.6 and 99.4, backward 194 and 184.
constexpr long long kCachedBytes = 128ll << 20;
template <typename T, bool NARROW>
bool cached_rows(long long B, long long T_, long long D, int tensors) {
    return !NARROW && B * T_ * D <= kCachedBytes / (long long)sizeof(T) / tensors;
}

template <typename T, ssd_dtype DT, bool CODES, bool NARROW>
hipError_t run_fwd(const GatedFwdArgs& a, char* ws, hipStream_t st) {
    constexpr int V = fwd_vec(DT, CODES), S = fwd_steps(DT, CODES);
    const Layout l = fwd_layout(DT, CODES, a.B, a.T, a.D);
    const hipError_t e = prepare(l, ws, a.cu, a.nseq, a.T, a.D, a.final_state, st);
    if (e != hipSuccess) return e;
    const Tiles tl = tiles_of(l, a.B, kLanes * V, ws, a.cu != nullptr);
    const FwdParams p{a, tl};
    const bool cached = cached_rows<T, NARROW>(a.B, a.T, a.D, 3);
#define SSD_GATED_FWD(PACKED, CACHED) \
    launch_tiles<gated_fwd_kernel<T, V, S, PACKED, CODES, NARROW, CACHED && !NARROW>>(p, st)
    if (a.cu) return cached ? SSD_GATED_FWD(true, true) : SSD_GATED_FWD(true, false);
    return cached ? SSD_GATED_FWD(false, true) : SSD_GATED_FWD(false, false);
#undef SSD_GATED_FWD
}

template <typename T, ssd_dtype DT, bool CODES, bool NARROW>
hipError_t run_bwd(const GatedBwdArgs& a, char* ws, hipStream_t st) {
    constexpr int V = kBwdVec, S = bwd_steps(DT);
    const Layout l = bwd_layout(DT, a.B, a.T, a.D);
    hipError_t e = prepare(l, ws, a.cu, a.nseq, a.T, a.D, nullptr, st);
    if (e != hipSuccess) return e;
    const Tiles tl = tiles_of(l, a.B, kLanes * V, ws, a.cu != nullptr);
    const int rows = a.B * l.nk;
    float* part = !a.d_bias ? nullptr : rows == 1 ? a.d_bias : (float*)(ws + l.part);
    const BwdParams p{a, tl, part};
    const bool cached = cached_rows<T, NARROW>(a.B, a.T, a.D, CODES ? 3 : 5);
#define SSD_GATED_BWD(PACKED, CACHED) \
    launch_tiles<gated_bwd_kernel<T, V, S, PACKED, CODES, NARROW, CACHED && !NARROW>>(p, st)
    if (a.cu) e = cached ? SSD_GATED_BWD(true, true) : SSD_GATED_BWD(true, false);
    else e = cached ? SSD_GATED_BWD(false, true) : SSD_GATED_BWD(false, false);
#undef SSD_GATED_BWD
    if (e != hipSuccess || !a.d_bias || rows == 1 || l.fused) return e;
    gated_dbias_kernel<<<(unsigned)((a.D + 31) / 32), kThreads, 0, st>>>(part, a.d_bias, rows,
                                                                         a.D);
    return hipGetLastError();
}

// run<T, dtype, CODES, NARROW>(a, ws, st): rows narrower than a piece have forms of their own
#define SSD_GATED_RUN(run, T, DT, vec)                                                       \
    (a.x_codes ? (a.D < vec(DT, true) ? run<T, DT, true, true>(a, (char*)ws, st)             \
                                      : run<T, DT, true, false>(a, (char*)ws, st))           \
               : (a.D < vec(DT, false) ? run<T, DT, false, true>(a, (char*)ws, st)           \
                                       : run<T, DT, false, false>(a, (char*)ws, st)))
constexpr int bwd_vec(ssd_dtype, bool) { return kBwdVec; }
}  // namespace

hipError_t launch_gated_fwd(ssd_dtype dtype, const GatedFwdArgs& a, void* ws, hipStream_t st) {
    if (a.T > 0)
        return dtype == SSD_F32 ? SSD_GATED_RUN(run_fwd, float, SSD_F32, fwd_vec)
                                : SSD_GATED_RUN(run_fwd, __bf16, SSD_BF16, fwd_vec);
    if (!a.final_state) return hipSuccess;
    const long long n = (long long)(a.cu ? a.nseq : a.B) * a.D;
    gated_carry_kernel<<<blocks_of(n), kThreads, 0, st>>>(a.init, a.final_state, n);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(ssd_dtype dtype, const GatedBwdArgs& a, void* ws, hipStream_t st) {
    if (a.T > 0 && a.B > 0)
        return dtype == SSD_F32 ? SSD_GATED_RUN(run_bwd, float, SSD_F32, bwd_vec)
                                : SSD_GATED_RUN(run_bwd, __bf16, SSD_BF16, bwd_vec);
    const long long n = (long long)a.B * a.D;
    if (a.d_init && n > 0)
        gated_carry_kernel<<<blocks_of(n), kThreads, 0, st>>>(a.d_final, a.d_init, n);
    if (a.d_bias)
        gated_carry_kernel<<<blocks_of(a.D), kThreads, 0, st>>>(nullptr, a.d_bias, a.D);
    return hipGetLastError();
}

hipError_t launch_gated_step(ssd_dtype dtype, const GatedStepArgs& a, hipStream_t st) {
    const unsigned pieces = (a.D + kStepVec - 1) / kStepVec;
    const unsigned blocks = blocks_of((long long)a.B * pieces);
    const bool narrow = a.D < kStepVec;
    if (dtype == SSD_F32)
        narrow ? gated_step_kernel<float, true><<<blocks, kThreads, 0, st>>>(a, pieces)
               : gated_step_kernel<float, false><<<blocks, kThreads, 0, st>>>(a, pieces);
    else
        narrow ? gated_step_kernel<__bf16, true><<<blocks, kThreads, 0, st>>>(a, pieces)
               : gated_step_kernel<__bf16, false><<<blocks, kThreads, 0, st>>>(a, pieces);
    return hipGetLastError();
}

}  // namespace ssd
