// RMS norm with the residual's addition and an optional e4m3 output:
//   h = x + residual,  y = h / sqrt(mean(h^2) + eps) * weight
//   e4m3: s = max(amax |y|, 1e-30) / 448 over the row or 128 channels, y / s
//
// HBM bound: x and the residual are read once, h and y written once.  A CTA, or for
// short rows a warp, takes a row; the row stays in registers between the sum of squares
// and the outputs, so that nothing is read twice, and the next row is requested
// before this one's reduction, so that loads stay in flight across it (4096 x
// 4096 bf16 to e4m3: 20.4 us, 5.7 TB/s, against 23.2 us with a CTA per row and
// nothing requested ahead).  h, the statistics and y are fp32; h is rounded once
// into residual_out, y once into its output.
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

// Eight channels as they lie in memory.
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *p) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)(sizeof(T) / 2); ++i) r.v[i] = reinterpret_cast<const uint4 *>(p)[i];
    return r;
}
__device__ __forceinline__ void unpack(const Raw<float> &r, float (&x)[8]) {
    load8(reinterpret_cast<const float *>(&r), x);
}
__device__ __forceinline__ void unpack(const Raw<__nv_bfloat16> &r, float (&x)[8]) {
    load8(reinterpret_cast<const __nv_bfloat16 *>(&r), x);
}

// NV: vectors of 8 channels per thread; WARP: a warp per row, else the CTA
template <typename T, int QUANT, int NV, bool WARP>
__global__ void __launch_bounds__(kMaxThreads) rms_norm_kernel(const RmsNormArgs a) {
    __shared__ float part[2][2][kMaxThreads / 32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int tid = WARP ? lane : threadIdx.x, threads = WARP ? 32 : blockDim.x;  // of the row
    const int nvec = a.D >> 3;
    const int64_t row0 = WARP ? (int64_t)blockIdx.x * warps + wid : blockIdx.x;
    const int64_t step = WARP ? (int64_t)gridDim.x * warps : gridDim.x;

    griddep_wait();
    griddep_launch_dependents();
    Raw<T> x[NV], r[NV];
    auto request = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * threads;
            if (v < nvec) {
                x[i] = load_raw((const T *)a.x + row * a.D + 8 * v);
                if (a.residual) r[i] = load_raw((const T *)a.residual + row * a.D + 8 * v);
            }
        }
    };
    if (row0 < a.rows) request(row0);
    int flip = 0;  // the reductions' buffers alternate, so that a barrier each is enough
    for (int64_t row = row0; row < a.rows; row += step, flip ^= 1) {
        float h[NV][8];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * threads;
            if (v < nvec) {
                unpack(x[i], h[i]);
                if (a.residual) {
                    float e[8];
                    unpack(r[i], e);
#pragma unroll
                    for (int j = 0; j < 8; ++j) h[i][j] += e[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sum += h[i][j] * h[i][j];
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) h[i][j] = 0.0f;
            }
        }
        if (row + step < a.rows) request(row + step);
        sum = warp_sum(sum);
        if (!WARP) {
            if (lane == 0) part[flip][0][wid] = sum;
            __syncthreads();
            sum = warp_sum(lane < warps ? part[flip][0][lane] : 0.0f);
        }
        const float rn = 1.0f / sqrtf(sum / (float)a.D + a.eps);

        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = tid + i * threads;
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
            if (!WARP) {
                if (lane == 0) part[flip][1][wid] = amax;
                __syncthreads();
                amax = lanes_max<32>(lane < warps ? part[flip][1][lane] : 0.0f);
            }
            const float s = max_nan(amax, kAmaxFloor) / kE4m3Max, inv = 1.0f / s;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = tid + i * threads;
                if (v < nvec) *(uint2 *)((uint8_t *)a.y + row * a.D + 8 * v) = to_e4m3(h[i], inv);
            }
            if (tid == 0) a.scales[row] = s;
        }
    }
}

template <typename T, int QUANT, int NV, bool WARP>
cudaError_t launch(const RmsNormArgs &a, int threads, int rows_per_cta, cudaStream_t stream) {
    auto kern = rms_norm_kernel<T, QUANT, NV, WARP>;
    const int64_t want = (a.rows + rows_per_cta - 1) / rows_per_cta;
    int64_t most = sm_count();
    if (want > most) {  // (a query that few rows do without)
        int per_sm = 0;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kern, threads, 0) != cudaSuccess || per_sm < 1) {
            cudaGetLastError();
            per_sm = 1;
        }
        most *= per_sm;
    }
    const cudaError_t e =
        launch_dependent(kern, dim3((unsigned)(want < most ? want : most)), dim3(threads), 0, stream, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int QUANT>
cudaError_t launch(const RmsNormArgs &a, cudaStream_t stream) {
    const int nvec = a.D / 8, nv = (nvec + kMaxThreads - 1) / kMaxThreads;
    // 65536 rows of 128: 16.7 us with a warp per row, 19.8 us with a CTA of one warp per row; at 512 channels
    // (two vectors a lane) the CTA per row is the faster one, 11.1 against 12.1 us for 16384 rows
    if (nvec <= 32) return launch<T, QUANT, 1, true>(a, 256, 8, stream);
    const int threads = nv > 1 ? kMaxThreads : (nvec + 31) / 32 * 32;
    if (nv <= 1) return launch<T, QUANT, 1, false>(a, threads, 1, stream);
    if (nv <= 2) return launch<T, QUANT, 2, false>(a, threads, 1, stream);
    if (nv <= 4) return launch<T, QUANT, 4, false>(a, threads, 1, stream);
    return launch<T, QUANT, 8, false>(a, threads, 1, stream);
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
