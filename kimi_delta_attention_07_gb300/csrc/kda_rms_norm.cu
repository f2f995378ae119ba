// RMS norm with the residual's addition and an optional e4m3 output:
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight
//   e4m3: s = max(amax |y|, 1e-30) / 448 over the row or 128 channels, y / s
//
// HBM bound: x and the residual are read once, h and y written once.  One CTA
// per row; the row stays in registers between the sum of squares and the
// outputs, so that nothing is read twice.  h, the statistics and y are fp32;
// h is rounded once into residual_out, y once into its output.
#include <cuda_fp8.h>

#include "kda_hybrid.cuh"

namespace kda {
namespace {

constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 1e-30f;  // an all-zero group still gets a normal, invertible scale
constexpr int kMaxThreads = 512;

// the larger of two values, NaN if either is (fmaxf would drop it)
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int WIDTH>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int o = WIDTH / 2; o > 0; o >>= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

__device__ __forceinline__ uint2 to_e4m3(const float (&y)[8], float inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(
            make_float2(y[4 * i] * inv, y[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(
            make_float2(y[4 * i + 2] * inv, y[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
        w[i] = lo | (hi << 16);
    }
    return make_uint2(w[0], w[1]);
}

// NV: vectors of 8 channels per thread
template <typename T, int QUANT, int NV>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(const RmsNormArgs a) {
    __shared__ float part[2][kMaxThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5, warps = blockDim.x >> 5;
    const int nvec = a.D >> 3;
    const int64_t row = blockIdx.x;
    const T *x = (const T *)a.x + row * a.D;
    const T *res = a.residual ? (const T *)a.residual + row * a.D : nullptr;

    griddep_wait();
    griddep_launch_dependents();
    float h[NV][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        if (v < nvec) {
            load8(x + 8 * v, h[i]);
            if (res) {
                float r[8];
                load8(res + 8 * v, r);
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] += r[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum += h[i][j] * h[i][j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
        }
    }
    sum = warp_sum(sum);
    if (lane == 0) part[0][wid] = sum;
    __syncthreads();
    sum = warp_sum(lane < warps ? part[0][lane] : 0.0f);
    const float rn = 1.0f / sqrtf(sum / (float)a.D + a.eps);

    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = tid + i * blockDim.x;
        if (v < nvec) {
            if (a.residual_out) store8((T *)a.residual_out + row * a.D + 8 * v, h[i]);
            float w[8];
            if (a.weight) load8(a.weight + 8 * v, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[i][j] *= a.weight ? rn * w[j] : rn;
            if (QUANT == KDA_QUANT_NONE) store8((T *)a.y + row * a.D + 8 * v, h[i]);
        }
        if (QUANT != KDA_QUANT_NONE) {
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = max_nan(m, fabsf(h[i][j]));
            if (QUANT == KDA_QUANT_ROW) {
                amax = max_nan(amax, m);
            } else {
                // 128 channels are 16 neighbouring vectors: half a warp
                const float s = max_nan(lanes_max<16>(m), kAmaxFloor) / kE4m3Max;
                if (v < nvec) {
                    *(uint2 *)((uint8_t *)a.y + row * a.D + 8 * v) = to_e4m3(h[i], 1.0f / s);
                    if ((lane & 15) == 0) a.scales[row * (a.D >> 7) + (v >> 4)] = s;
                }
            }
        }
    }
    if (QUANT == KDA_QUANT_ROW) {
        amax = lanes_max<32>(amax);
        if (lane == 0) part[1][wid] = amax;
        __syncthreads();
        amax = lanes_max<32>(lane < warps ? part[1][lane] : 0.0f);
        const float s = max_nan(amax, kAmaxFloor) / kE4m3Max, inv = 1.0f / s;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * blockDim.x;
            if (v < nvec) *(uint2 *)((uint8_t *)a.y + row * a.D + 8 * v) = to_e4m3(h[i], inv);
        }
        if (tid == 0) a.scales[row] = s;
    }
}

template <typename T, int QUANT>
cudaError_t launch(const RmsNormArgs &a, cudaStream_t stream) {
    const int nvec = a.D / 8;
    const int nv = (nvec + kMaxThreads - 1) / kMaxThreads;
    const int threads = nv > 1 ? kMaxThreads : (nvec + 31) / 32 * 32;
    auto kern = nv <= 1   ? rms_norm_kernel<T, QUANT, 1>
                : nv <= 2 ? rms_norm_kernel<T, QUANT, 2>
                : nv <= 4 ? rms_norm_kernel<T, QUANT, 4>
                          : rms_norm_kernel<T, QUANT, 8>;
    const cudaError_t e = launch_dependent(kern, dim3((unsigned)a.rows), dim3(threads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T>
cudaError_t launch(const RmsNormArgs &a, int quant, cudaStream_t stream) {
    return quant == KDA_QUANT_NONE  ? launch<T, KDA_QUANT_NONE>(a, stream)
           : quant == KDA_QUANT_ROW ? launch<T, KDA_QUANT_ROW>(a, stream)
                                    : launch<T, KDA_QUANT_BLOCK>(a, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs &a, int quant, int dtype, cudaStream_t stream) {
    return dtype == KDA_BF16 ? launch<__nv_bfloat16>(a, quant, stream) : launch<float>(a, quant, stream);
}

}  // namespace kda
