// w8a8.cu -- the 8-bit linear: Y = X W^T with X and W of 8-bit codes,
//
//   Y[m][n] = x_scales[m] w_scales[n] sum_k x_q[m][k] (w_q[n][k] - z[n]) + bias[n]
//           = x_scales[m] w_scales[n] (sum_k x_q w_q - z[n] S[m]) + bias[n],
//
// S[m] = sum_k x_q[m][k].  The integer sums are exact in 32 bits for K <=
// 65536 (|x_q| <= 128, |w_q - z| <= 255: at most 2139095040 < 2^31), also
// where the two terms of the difference are not: it is taken modulo 2^32.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gptq {

namespace {

constexpr int kTile = 64;
constexpr int kWords = 16;   // 4-code words of K per step

__device__ __forceinline__ void store_rounded(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_rounded(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_rounded(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The 4 codes k .. k+3 of a row, zero where k is past K.
__device__ __forceinline__ int codes4(const int8_t* row, int k, int K)
{
    if (k >= K) return 0;
    const uint32_t v = *reinterpret_cast<const uint32_t*>(row + k);
    return static_cast<int>(K - k >= 4 ? v : v & (0xffffffffu >> (8 * (4 - (K - k)))));
}

// 64 x 64 outputs a block, 4 x 4 a thread, four products an instruction.
template <typename T>
__global__ void __launch_bounds__(256) w8a8_simt_kernel(W8A8Args a)
{
    __shared__ int xs[kWords][kTile + 1], ws[kWords][kTile + 1];
    const int64_t m0 = static_cast<int64_t>(blockIdx.x) * kTile;
    const int64_t n0 = static_cast<int64_t>(blockIdx.y) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const int K = static_cast<int>(a.K);
    int acc[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 4 * kWords) {
        for (int i = threadIdx.x; i < kTile * kWords; i += 256) {
            const int r = i / kWords, w = i % kWords;
            xs[w][r] = m0 + r < a.M ? codes4(a.Xq + (m0 + r) * a.ldx, k0 + 4 * w, K) : 0;
            ws[w][r] = n0 + r < a.N ? codes4(a.Wq + (n0 + r) * a.ldw, k0 + 4 * w, K) : 0;
        }
        __syncthreads();
        for (int w = 0; w < kWords; ++w)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) acc[i][j] = __dp4a(xs[w][ty + 16 * i], ws[w][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m >= a.M || n >= a.N) continue;
            uint32_t v = static_cast<uint32_t>(acc[i][j]);
            if (a.w_zeros) v -= static_cast<uint32_t>(a.w_zeros[n]) * static_cast<uint32_t>(a.x_sums[m]);
            const float y = static_cast<float>(static_cast<int>(v)) * a.w_scales[n] * a.x_scales[m];
            store_rounded(static_cast<T*>(a.Y) + m * a.ldy + n, a.bias ? y + a.bias[n] : y);
        }
}

}  // namespace

int run_w8a8(const W8A8Args& a, int y_type, cudaStream_t stream)
{
    const dim3 grid(static_cast<unsigned>((a.M + kTile - 1) / kTile), static_cast<unsigned>((a.N + kTile - 1) / kTile));
    if (y_type == GPTQ_F32)
        w8a8_simt_kernel<float><<<grid, 256, 0, stream>>>(a);
    else if (y_type == GPTQ_F16)
        w8a8_simt_kernel<__half><<<grid, 256, 0, stream>>>(a);
    else
        w8a8_simt_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
