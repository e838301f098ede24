// ckpt.hip -- activations held in 8 bits: pack and unpack.
//
// Every 64 neighbouring channels of a row share a scale (m / 127, m the largest |v|); a
// code is the integer nearest to v * (127 / m).  Bound by HBM: pack reads 2 or 4 bytes a
// value and writes 1 + 1/16, unpack the reverse.  A lane holds one 16-byte piece of a row (8
// bf16 or 4 fp32), so a group is 8 or 16 neighbouring lanes and its maximum a few DPP steps
// inside them.  The wide rows are read and written once: non-temporal (16384 x 5376 in bf16,
// packed and unpacked again: 118 us cached with 4 rows a thread in flight, 91 non-temporal; 86
// with 2 rows, 98 with 8).
#include "gated.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = SSD_CKPT_GROUP;
constexpr int kRows = 2;  // rows of a thread

// Pieces of a row are a power of two of neighbouring threads (at most a whole workgroup):
// block -> (rows, columns), thread -> (row, piece).
struct Grid {
    long long rows;
    int width, groups;
    int shift;        // log2 of the threads along a row
    unsigned cols;    // workgroups along a row
};

template <typename T> constexpr int kVec = 16 / sizeof(T);

typedef uint32_t Words4 __attribute__((ext_vector_type(4)));
typedef Words4 AnyWords4 __attribute__((aligned(2)));

// rows need only element alignment: pieces are unaligned 16-byte accesses
template <typename T>
__device__ __forceinline__ void load_piece(float (&v)[kVec<T>], const T* p, int n) {
    constexpr int V = kVec<T>;
    if (n >= V) {
        const Words4 b = __builtin_nontemporal_load((const AnyWords4*)p);
#pragma unroll
        for (int i = 0; i < V; ++i)
            v[i] = sizeof(T) == 4
                       ? __uint_as_float(b[i % 4])
                       : __uint_as_float(i & 1 ? b[i / 2] & 0xffff0000u : b[i / 2] << 16);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = i < n ? to_f32(p[i]) : 0.f;
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void ckpt_pack_kernel(const T* src, long long stride,
                                                             Grid g, int8_t* codes,
                                                             float* scales) {
    constexpr int V = kVec<T>, L = kGroup / V;
    const int per = kThreads >> g.shift;  // rows of a workgroup at a time
    const unsigned rb = blockIdx.x / g.cols, cb = blockIdx.x % g.cols;
    const int c0 = ((int)(cb << g.shift) + (threadIdx.x & ((1 << g.shift) - 1))) * V;
    const int n = g.width - c0;
    const long long row0 = (long long)rb * per * kRows + (threadIdx.x >> g.shift);
    float v[kRows][V];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = row0 + u * per;
        load_piece<T>(v[u], src + row * stride + c0, row < g.rows ? n : 0);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = row0 + u * per;
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < V; ++i) most = max(most, __float_as_uint(v[u][i]) & 0x7fffffffu);
        most = ckpt_group_max<L>(most);  // every lane of the wave takes part
        const CkptScale s(most);
        if (row >= g.rows || n <= 0) continue;
        if (c0 % kGroup == 0) scales[row * g.groups + c0 / kGroup] = s.scale;
        ckpt_store<V>(codes + row * g.width + c0, v[u], s, 0, min(n, V));
    }
}

template <typename T>
__global__ __launch_bounds__(kThreads) void ckpt_unpack_kernel(const int8_t* codes,
                                                               const float* scales, Grid g,
                                                               T* dst, long long stride) {
    constexpr int V = kVec<T>;
    const int per = kThreads >> g.shift;
    const unsigned rb = blockIdx.x / g.cols, cb = blockIdx.x % g.cols;
    const int c0 = ((int)(cb << g.shift) + (threadIdx.x & ((1 << g.shift) - 1))) * V;
    const int n = g.width - c0;
    if (n <= 0) return;
    const long long row0 = (long long)rb * per * kRows + (threadIdx.x >> g.shift);
    CkptPiece<V> b[kRows];
    float s[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = row0 + u * per;
        if (row >= g.rows) continue;
        const int8_t* p = codes + row * g.width + c0;
        s[u] = scales[row * g.groups + c0 / kGroup];
        if (n >= V) b[u].load(p);
        else b[u].load_part(p, n);
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const long long row = row0 + u * per;
        if (row >= g.rows) continue;
        T* p = dst + row * stride + c0;
        union { T t[V]; Words4 a; } o;
#pragma unroll
        for (int i = 0; i < V; ++i)
            o.t[i] = from_f32<T>(b[u].get(i) * s[u]);
        if (n >= V) {
            __builtin_nontemporal_store(o.a, (AnyWords4*)p);
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < n) p[i] = o.t[i];
        }
    }
}

template <typename T> Grid grid_of(long long rows, int width, unsigned* blocks) {
    Grid g;
    g.rows = rows;
    g.width = width;
    g.groups = (width + kGroup - 1) / kGroup;
    const int lanes = kGroup / kVec<T>;  // a group's lanes stay together
    g.shift = lanes == 8 ? 3 : 4;
    while ((1 << g.shift) < kThreads && ((long long)kVec<T> << g.shift) < width) ++g.shift;
    g.cols = (unsigned)((width + ((long long)kVec<T> << g.shift) - 1) /
                        ((long long)kVec<T> << g.shift));
    const long long per = (long long)(kThreads >> g.shift) * kRows;
    *blocks = (unsigned)((rows + per - 1) / per * g.cols);
    return g;
}

}  // namespace

hipError_t launch_ckpt_pack(long long rows, int width, ssd_dtype dtype, const void* src,
                            long long src_stride, int8_t* codes, float* scales, hipStream_t st) {
    unsigned blocks;
    if (dtype == SSD_F32) {
        const Grid g = grid_of<float>(rows, width, &blocks);
        ckpt_pack_kernel<float>
            <<<blocks, kThreads, 0, st>>>((const float*)src, src_stride, g, codes, scales);
    } else {
        const Grid g = grid_of<__bf16>(rows, width, &blocks);
        ckpt_pack_kernel<__bf16>
            <<<blocks, kThreads, 0, st>>>((const __bf16*)src, src_stride, g, codes, scales);
    }
    return hipGetLastError();
}

hipError_t launch_ckpt_unpack(long long rows, int width, ssd_dtype dtype, const int8_t* codes,
                              const float* scales, void* dst, long long dst_stride,
                              hipStream_t st) {
    unsigned blocks;
    if (dtype == SSD_F32) {
        const Grid g = grid_of<float>(rows, width, &blocks);
        ckpt_unpack_kernel<float>
            <<<blocks, kThreads, 0, st>>>(codes, scales, g, (float*)dst, dst_stride);
    } else {
        const Grid g = grid_of<__bf16>(rows, width, &blocks);
        ckpt_unpack_kernel<__bf16>
            <<<blocks, kThreads, 0, st>>>(codes, scales, g, (__bf16*)dst, dst_stride);
    }
    return hipGetLastError();
}

}  // namespace ssd
