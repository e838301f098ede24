// ckpt.hip -- activations held in 8 bits: pack and unpack.
//
// Every 64 neighbouring channels of a row share a scale (m / 127, m the largest |v|); a
// code is the integer nearest to v * (127 / m).  One thread per group.
#include "gated.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = SSD_CKPT_GROUP;

template <typename T>
__global__ __launch_bounds__(kThreads) void ckpt_pack_kernel(const T* src, long long stride,
                                                             long long groups, int per_row,
                                                             int width, int8_t* codes,
                                                             float* scales) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= groups) return;
    const long long row = id / per_row;
    const int c0 = (int)(id % per_row) * kGroup, n = min(kGroup, width - c0);
    const T* v = src + row * stride + c0;
    uint32_t most = 0;
    for (int i = 0; i < n; ++i)
        most = max(most, __float_as_uint(to_f32(v[i])) & 0x7fffffffu);
    const CkptScale s(most);
    scales[id] = s.scale;
    for (int i = 0; i < n; ++i)
        codes[row * width + c0 + i] =
            most < 0x7f800000u ? (int8_t)ckpt_code(to_f32(v[i]), s.inverse) : 0;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void ckpt_unpack_kernel(const int8_t* codes,
                                                               const float* scales,
                                                               long long groups, int per_row,
                                                               int width, T* dst,
                                                               long long stride) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= groups) return;
    const long long row = id / per_row;
    const int c0 = (int)(id % per_row) * kGroup, n = min(kGroup, width - c0);
    const float s = scales[id];
    for (int i = 0; i < n; ++i)
        dst[row * stride + c0 + i] = from_f32<T>((float)codes[row * width + c0 + i] * s);
}

}  // namespace

hipError_t launch_ckpt_pack(long long rows, int width, ssd_dtype dtype, const void* src,
                            long long src_stride, int8_t* codes, float* scales, hipStream_t st) {
    const int per_row = (width + kGroup - 1) / kGroup;
    const long long groups = rows * per_row;
    const unsigned blocks = (unsigned)((groups + kThreads - 1) / kThreads);
    if (dtype == SSD_F32)
        ckpt_pack_kernel<float><<<blocks, kThreads, 0, st>>>(
            (const float*)src, src_stride, groups, per_row, width, codes, scales);
    else
        ckpt_pack_kernel<__bf16><<<blocks, kThreads, 0, st>>>(
            (const __bf16*)src, src_stride, groups, per_row, width, codes, scales);
    return hipGetLastError();
}

hipError_t launch_ckpt_unpack(long long rows, int width, ssd_dtype dtype, const int8_t* codes,
                              const float* scales, void* dst, long long dst_stride,
                              hipStream_t st) {
    const int per_row = (width + kGroup - 1) / kGroup;
    const long long groups = rows * per_row;
    const unsigned blocks = (unsigned)((groups + kThreads - 1) / kThreads);
    if (dtype == SSD_F32)
        ckpt_unpack_kernel<float><<<blocks, kThreads, 0, st>>>(
            codes, scales, groups, per_row, width, (float*)dst, dst_stride);
    else
        ckpt_unpack_kernel<__bf16><<<blocks, kThreads, 0, st>>>(
            codes, scales, groups, per_row, width, (__bf16*)dst, dst_stride);
    return hipGetLastError();
}

}  // namespace ssd
