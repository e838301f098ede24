// gated.hip -- the gated recurrence: forward, backward and single step.
//
// Per batch element and channel, with s = g + bias and q = 1 / (1 + exp(s)), a = 1 - q:
//     h_t = h_{t-1} + q_t (x_t - h_{t-1}),     G_t = dh_t + a_{t+1} G_{t+1},
//     dx_t = q_t G_t,   dg_t = G_t (h_{t-1} - x_t) q_t a_t     (dq/ds = -q a).
// One thread per channel walks the steps: the backward runs over the chunks from the last
// to the first, recomputes a chunk's 64 states from its entry state and then goes through
// them in reverse.
#include "gated.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_fwd_kernel(GatedFwdArgs a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)a.B * a.D) return;
    const int b = (int)(id / a.D), d = (int)(id % a.D);
    const float bias = a.bias ? a.bias[d] : 0.f;
    const int nC = (a.T + kGatedChunk - 1) / kGatedChunk;
    float h = a.init ? a.init[id] : 0.f;
    int seq = 0;  // packed rows: the sequence that the next step belongs to, or one before
    for (int t = 0; t < a.T; ++t) {
        const long long row = (long long)b * a.T + t;
        if (t % kGatedChunk == 0 && a.entry)
            a.entry[((long long)b * nC + t / kGatedChunk) * a.D + d] = h;
        if (a.cu) {
            while (seq < a.nseq - 1 && a.cu[seq + 1] <= t) ++seq;
            if (a.cu[seq] == t) h = 0.f;
        }
        const Gate q(to_f32(((const T*)a.g)[row * a.g_stride + d]) + bias);
        h = gate_step(q.q, to_f32(((const T*)a.x)[row * a.x_stride + d]), h);
        ((T*)a.h)[row * a.D + d] = from_f32<T>(h);
        if (a.cu && a.final_state && a.cu[seq + 1] == t + 1)
            a.final_state[(long long)seq * a.D + d] = h;
    }
    if (!a.final_state) return;
    if (!a.cu) {
        a.final_state[id] = h;
        return;
    }
    for (int s = 0; s < a.nseq; ++s)  // empty sequences end in their zero state
        if (a.cu[s] == a.cu[s + 1]) a.final_state[(long long)s * a.D + d] = 0.f;
}

// d_bias' share of every batch element goes to part [B][D]
template <typename T, bool CODES>
__global__ __launch_bounds__(kThreads) void gated_bwd_kernel(GatedBwdArgs a, float* part) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)a.B * a.D) return;
    const int b = (int)(id / a.D), d = (int)(id % a.D);
    const float bias = a.bias ? a.bias[d] : 0.f;
    const int nC = (a.T + kGatedChunk - 1) / kGatedChunk;
    const long long groups = (a.D + SSD_CKPT_GROUP - 1) / SSD_CKPT_GROUP;
    auto load = [&](const void* v, long long stride, const int8_t* codes, const float* scales,
                    int t) {
        const long long row = (long long)b * a.T + t;
        if (CODES)
            return (float)codes[row * a.D + d] * scales[row * groups + d / SSD_CKPT_GROUP];
        return to_f32(((const T*)v)[row * stride + d]);
    };
    float G = a.cu ? 0.f : (a.d_final ? a.d_final[id] : 0.f);  // carried into step t
    float db = 0.f;
    int seq = a.nseq - 1;
    float before[kGatedChunk];
    for (int c = nC - 1; c >= 0; --c) {
        const int t0 = c * kGatedChunk;
        const int t1 = min(a.T, t0 + kGatedChunk);
        float h = a.entry[((long long)b * nC + c) * a.D + d];
        int s = 0;
        for (int t = t0; t < t1; ++t) {
            if (a.cu) {
                while (s < a.nseq - 1 && a.cu[s + 1] <= t) ++s;
                if (a.cu[s] == t) h = 0.f;
            }
            before[t - t0] = h;
            const Gate q(load(a.g, a.g_stride, a.g_codes, a.g_scales, t) + bias);
            h = gate_step(q.q, load(a.x, a.x_stride, a.x_codes, a.x_scales, t), h);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const long long row = (long long)b * a.T + t;
            bool first = false;
            if (a.cu) {
                while (seq > 0 && a.cu[seq] > t) --seq;
                first = a.cu[seq] == t;
                if (a.cu[seq + 1] == t + 1)
                    G = a.d_final ? a.d_final[(long long)seq * a.D + d] : 0.f;
            }
            const Gate q(load(a.g, a.g_stride, a.g_codes, a.g_scales, t) + bias);
            const float x = load(a.x, a.x_stride, a.x_codes, a.x_scales, t);
            G += to_f32(((const T*)a.dh)[row * a.dh_stride + d]);
            const float dg = G * (before[t - t0] - x) * q.q * q.a;
            ((T*)a.dx)[row * a.dx_stride + d] = from_f32<T>(q.q * G);
            ((T*)a.dg)[row * a.dg_stride + d] = from_f32<T>(dg);
            db += dg;
            G = first ? 0.f : fmaf(-q.q, G, G);
        }
    }
    if (a.d_init) a.d_init[id] = G;
    part[id] = db;
}

__global__ __launch_bounds__(kThreads) void gated_dbias_kernel(const float* part, float* d_bias,
                                                               int rows, int D) {
    const int d = blockIdx.x * kThreads + threadIdx.x;
    if (d >= D) return;
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += part[(long long)r * D + d];
    d_bias[d] = s;
}

template <typename T>
__global__ __launch_bounds__(kThreads) void gated_step_kernel(GatedStepArgs a) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id >= (long long)a.B * a.D) return;
    const long long b = id / a.D;
    const int d = (int)(id % a.D);
    const Gate q(to_f32(((const T*)a.g)[b * a.g_stride + d]) + (a.bias ? a.bias[d] : 0.f));
    const float h = gate_step(q.q, to_f32(((const T*)a.x)[b * a.x_stride + d]), a.state[id]);
    a.state[id] = h;
    ((T*)a.h)[id] = from_f32<T>(h);
}

__global__ __launch_bounds__(kThreads) void gated_carry_kernel(const float* src, float* dst,
                                                               long long n) {
    const long long id = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (id < n) dst[id] = src ? src[id] : 0.f;
}

unsigned blocks_of(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace

size_t gated_workspace_bytes(int B, int T, int D) {
    return T > 0 ? (size_t)B * D * sizeof(float) : 0;
}

hipError_t launch_gated_fwd(ssd_dtype dtype, const GatedFwdArgs& a, void*, hipStream_t st) {
    const unsigned blocks = blocks_of((long long)a.B * a.D);
    if (dtype == SSD_F32)
        gated_fwd_kernel<float><<<blocks, kThreads, 0, st>>>(a);
    else
        gated_fwd_kernel<__bf16><<<blocks, kThreads, 0, st>>>(a);
    if (!a.x_codes || a.T == 0) return hipGetLastError();
    const long long rows = (long long)a.B * a.T;
    const hipError_t e = launch_ckpt_pack(rows, a.D, dtype, a.x, a.x_stride, a.x_codes,
                                          a.x_scales, st);
    if (e != hipSuccess) return e;
    return launch_ckpt_pack(rows, a.D, dtype, a.g, a.g_stride, a.g_codes, a.g_scales, st);
}

hipError_t launch_gated_step(ssd_dtype dtype, const GatedStepArgs& a, hipStream_t st) {
    const unsigned blocks = blocks_of((long long)a.B * a.D);
    if (dtype == SSD_F32)
        gated_step_kernel<float><<<blocks, kThreads, 0, st>>>(a);
    else
        gated_step_kernel<__bf16><<<blocks, kThreads, 0, st>>>(a);
    return hipGetLastError();
}

hipError_t launch_gated_bwd(ssd_dtype dtype, const GatedBwdArgs& a, void* ws, hipStream_t st) {
    const unsigned blocks = blocks_of((long long)a.B * a.D);
    float* part = (float*)ws;
    if (a.T > 0 && a.B > 0) {
        const bool codes = a.x_codes != nullptr;
        if (dtype == SSD_F32)
            codes ? gated_bwd_kernel<float, true><<<blocks, kThreads, 0, st>>>(a, part)
                  : gated_bwd_kernel<float, false><<<blocks, kThreads, 0, st>>>(a, part);
        else
            codes ? gated_bwd_kernel<__bf16, true><<<blocks, kThreads, 0, st>>>(a, part)
                  : gated_bwd_kernel<__bf16, false><<<blocks, kThreads, 0, st>>>(a, part);
    } else if (a.d_init && a.B > 0) {
        gated_carry_kernel<<<blocks, kThreads, 0, st>>>(a.cu ? nullptr : a.d_final, a.d_init,
                                                        (long long)a.B * a.D);
    }
    if (a.d_bias)
        gated_dbias_kernel<<<blocks_of(a.D), kThreads, 0, st>>>(part, a.d_bias,
                                                                a.T > 0 ? a.B : 0, a.D);
    return hipGetLastError();
}

}  // namespace ssd
