// tokens.cu -- 8-bit tokens: the quantization of activation rows, the norm
// between two blocks (whose output may be 8-bit tokens), and the layout of
// 8-bit weight codes for the product of w8a8.cu.
//
//   quantize_tokens  v = x  or  silu(a) x;  t = max_k |v_k|;
//                    q_k = rint(127 v_k / t), s = t / 127, S = sum_k q_k,
//                    hat_k = s q_k.
//   block_norm       h' = h  or  h rsqrt(mean h^2 + eps) w_post;
//                    r' = r + scale g h';  out = r' rsqrt(mean r'^2 + eps)
//                    w_pre, and its 8-bit tokens.
//
// One block per row, the row read once for each pass over it.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace gptq {

namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ float load_as_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_as_f32(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load_as_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_rounded(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_rounded(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_rounded(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float silu(float a) { return a / (1.f + expf(-a)); }

// Sum / unsigned maximum over the block; every thread gets the result.
template <typename T, typename Op>
__device__ __forceinline__ T block_reduce(T v, Op op)
{
    __shared__ T part[kRowThreads / 32];
    __syncthreads();
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    v = part[0];
    for (int i = 1; i < kRowThreads / 32; ++i) v = op(v, part[i]);
    return v;
}

struct Add {
    template <typename T>
    __device__ T operator()(T a, T b) const { return a + b; }
};
struct Max {
    __device__ uint32_t operator()(uint32_t a, uint32_t b) const { return a > b ? a : b; }
};

// The grid of one row from t = max |v|, given as the bits of t (as unsigned
// integers the magnitudes' bits keep their order, with infinities and then
// NaN above every finite value).
struct TokenGrid {
    float scale;   // t / 127; 0 for a row of zeros, NaN for a row with an infinite or NaN value
    float c127;    // 127 c, c = 2^+-100 where t is so small or large that 127 v or 1 / t would leave fp32's range
    float b;       // c t
    float rb;      // 1 / b
    float top;     // t
    bool ok;       // codes are not all 0
};

__device__ __forceinline__ TokenGrid token_grid(uint32_t top_bits)
{
    TokenGrid g;
    g.top = __uint_as_float(top_bits);
    g.ok = top_bits != 0 && top_bits < 0x7f800000u;
    g.scale = top_bits < 0x7f800000u ? __fdiv_rn(g.top, 127.f) : __uint_as_float(0x7fffffffu);
    const float c = g.top < 0x1p-100f ? 0x1p100f : g.top > 0x1p100f ? 0x1p-100f : 1.f;
    g.c127 = 127.f * c;
    g.b = g.top * c;
    g.rb = __frcp_rn(g.b);
    return g;
}

// rint(127 v / t).  One correction step on the product with the rounded
// reciprocal gives the quotient of (127 c v) / (c t) rounded to nearest
// (Markstein; the exception, a divisor whose significand is all ones, has 24
// significant bits).  For v and t of at most 11 significant bits 127 v is
// exact, a quotient that is no tie lies at least 2^-19 (relative) from one
// and a tie is representable, so the code is the exact one.  EXACT (v of 24
// bits): the quotient is within 127 * 2^-22 of 127 v / t, and one that near
// to a tie is decided in double (127 v is exact there, and a quotient that is
// no tie lies 2^-33 from one).
template <bool EXACT>
__device__ __forceinline__ int token_code(float v, const TokenGrid& g)
{
    const float a = v * g.c127;
    const float t0 = a * g.rb;
    const float t = fmaf(fmaf(-t0, g.b, a), g.rb, t0);
    const float q = rintf(t);
    if (EXACT && fabsf(fabsf(t - q) - 0.5f) < 1e-4f)
        return static_cast<int>(rint(127.0 * static_cast<double>(v) / static_cast<double>(g.top)));
    return static_cast<int>(q);
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    quantize_tokens_kernel(int8_t* Xq, int64_t ldq, float* x_scales, int32_t* x_sums, T* hat,
                           int64_t ldh, const T* X, int64_t ldx, const T* gate, int64_t ldg, int K)
{
    const int64_t m = blockIdx.x;
    auto value = [&](int k) {
        const float x = load_as_f32(X + m * ldx + k);
        return gate ? silu(load_as_f32(gate + m * ldg + k)) * x : x;
    };
    uint32_t top = 0;
    for (int k = threadIdx.x; k < K; k += kRowThreads)
        top = max(top, __float_as_uint(value(k)) & 0x7fffffffu);
    const TokenGrid g = token_grid(block_reduce(top, Max()));
    int sum = 0;
    for (int k = threadIdx.x; k < K; k += kRowThreads) {
        const int q = !g.ok ? 0 : gate ? token_code<false>(value(k), g) : token_code<sizeof(T) == 4>(value(k), g);
        sum += q;
        if (Xq) Xq[m * ldq + k] = static_cast<int8_t>(q);
        if (hat) store_rounded(hat + m * ldh + k, g.scale * static_cast<float>(q));
    }
    if (x_sums) {
        sum = block_reduce(sum, Add());
        if (threadIdx.x == 0) x_sums[m] = sum;
    }
    if (x_scales && threadIdx.x == 0) x_scales[m] = g.scale;
}

template <typename T>
__global__ void __launch_bounds__(kRowThreads)
    block_norm_kernel(BlockNormArgs a)
{
    const int64_t m = blockIdx.x;
    const int D = static_cast<int>(a.D);
    const T* block = static_cast<const T*>(a.block);
    const T* residual = static_cast<const T*>(a.residual);
    const T* gate = static_cast<const T*>(a.gate);
    float post = 1.f;
    if (block && a.post_norm) {
        float s = 0.f;
        for (int k = threadIdx.x; k < D; k += kRowThreads) {
            const float h = load_as_f32(block + m * a.ldb + k);
            s = fmaf(h, h, s);
        }
        post = rsqrtf(block_reduce(s, Add()) / static_cast<float>(D) + a.eps);
    }
    const int64_t grow = gate ? (m / a.gate_rows) * a.ldg : 0;
    auto value = [&](int k) {
        float r = residual ? load_as_f32(residual + m * a.ldr + k) : 0.f;
        if (!block) return r;
        float h = load_as_f32(block + m * a.ldb + k) * post;
        if (a.post_norm && a.post_weight) h *= a.post_weight[k];
        if (gate) h *= load_as_f32(gate + grow + k);
        return fmaf(a.scale, h, r);
    };
    float s = 0.f;
    uint32_t top = 0;
    for (int k = threadIdx.x; k < D; k += kRowThreads) {
        const float r = value(k);
        s = fmaf(r, r, s);
        top = max(top, __float_as_uint(a.pre_weight ? r * a.pre_weight[k] : r) & 0x7fffffffu);
    }
    const float pre = rsqrtf(block_reduce(s, Add()) / static_cast<float>(D) + a.eps);
    // the codes are those of r w: the factor rsqrt(...) of the row cancels in 127 v / t
    TokenGrid g = token_grid(block_reduce(top, Max()));
    int sum = 0;
    for (int k = threadIdx.x; k < D; k += kRowThreads) {
        const float r = value(k);
        const float v = a.pre_weight ? r * a.pre_weight[k] : r;
        if (a.out) store_rounded(static_cast<T*>(a.out) + m * a.ldo + k, v * pre);
        if (a.q) {
            const int q = g.ok ? token_code<false>(v, g) : 0;
            sum += q;
            a.q[m * a.ldq + k] = static_cast<int8_t>(q);
        }
        if (a.stream_out) store_rounded(static_cast<T*>(a.stream_out) + m * a.lds + k, r);
    }
    if (a.q && a.q_sums) {
        sum = block_reduce(sum, Add());
        if (threadIdx.x == 0) a.q_sums[m] = sum;
    }
    if (a.q && threadIdx.x == 0) a.q_scales[m] = g.scale * pre;
}

__global__ void w8a8_pack_kernel(int8_t* Wq, int64_t ldw, int32_t* w_zeros, const uint8_t* codes,
                                 const float* zeros, int64_t N, int64_t K)
{
    const int64_t n = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
    if (n >= N) return;
    for (int64_t k = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; k < ldw;
         k += static_cast<int64_t>(gridDim.x) * blockDim.x)
        Wq[n * ldw + k] = k < K ? static_cast<int8_t>(codes[n * K + k] ^ 0x80) : int8_t(0);
    if (blockIdx.x == 0 && threadIdx.x == 0) w_zeros[n] = static_cast<int32_t>(zeros[n]) - 128;
}

}  // namespace

int run_quantize_tokens(int8_t* Xq, int64_t ldq, float* x_scales, int32_t* x_sums, void* hat,
                        int64_t ldh, const void* X, int64_t ldx, const void* gate, int64_t ldg,
                        int type, int64_t M, int64_t K, cudaStream_t stream)
{
    const unsigned blocks = static_cast<unsigned>(M);
    const int k = static_cast<int>(K);
    if (type == GPTQ_F32)
        quantize_tokens_kernel<<<blocks, kRowThreads, 0, stream>>>(
            Xq, ldq, x_scales, x_sums, static_cast<float*>(hat), ldh, static_cast<const float*>(X),
            ldx, static_cast<const float*>(gate), ldg, k);
    else if (type == GPTQ_F16)
        quantize_tokens_kernel<<<blocks, kRowThreads, 0, stream>>>(
            Xq, ldq, x_scales, x_sums, static_cast<__half*>(hat), ldh, static_cast<const __half*>(X),
            ldx, static_cast<const __half*>(gate), ldg, k);
    else
        quantize_tokens_kernel<<<blocks, kRowThreads, 0, stream>>>(
            Xq, ldq, x_scales, x_sums, static_cast<__nv_bfloat16*>(hat), ldh,
            static_cast<const __nv_bfloat16*>(X), ldx, static_cast<const __nv_bfloat16*>(gate), ldg, k);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

int run_block_norm(const BlockNormArgs& a, int type, cudaStream_t stream)
{
    const unsigned blocks = static_cast<unsigned>(a.M);
    if (type == GPTQ_F32)
        block_norm_kernel<float><<<blocks, kRowThreads, 0, stream>>>(a);
    else if (type == GPTQ_F16)
        block_norm_kernel<__half><<<blocks, kRowThreads, 0, stream>>>(a);
    else
        block_norm_kernel<__nv_bfloat16><<<blocks, kRowThreads, 0, stream>>>(a);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

int run_w8a8_pack(int8_t* Wq, int64_t ldw, int32_t* w_zeros, const uint8_t* codes, const float* zeros,
                  int64_t N, int64_t K, cudaStream_t stream)
{
    const unsigned y = static_cast<unsigned>(std::min<int64_t>(N, 32768));
    const unsigned z = static_cast<unsigned>((N + y - 1) / y);
    w8a8_pack_kernel<<<dim3(static_cast<unsigned>(std::min<int64_t>((ldw + 255) / 256, 64)), y, z), 256, 0, stream>>>(
        Wq, ldw, w_zeros, codes, zeros, N, K);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
