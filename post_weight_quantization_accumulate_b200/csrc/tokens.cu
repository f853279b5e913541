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
// All of these are bound by memory: a row is read once, kept in registers
// through its reductions and written once.  A row belongs to as many threads as
// give each CH chunks of 16 bytes.  Chunks lie on 16-byte boundaries of
// the row that is written; where its rows do not begin on one (an odd width),
// a row's first and last chunk are partial, and what lies at other alignments
// is read in two aligned pieces and shifted into place.  Element-wise accesses
// instead cost about 90 instructions an element, with the issue slots and not
// memory as the bound.  Rows pass L1 by, so that the float32 weights stay in it,
// and each row asks for a later one (two an SM ahead) to be brought into L2.
// The kernels are programmatic dependent launches: set up while the kernel
// before ends, waiting for its results before the first global access.
//
// B200: tokens of 8192 x 11008 bf16 with values 67 us (6.7 TB/s), without 48
// (5.6), of a gated activation 77 (5.9; 20 instructions a value); norm of 16384 x
// 4096 bf16 84 us (6.4 TB/s), with norm and gate after the block 89 (6.0), to
// tokens 75 (6.2); 8192 x 4096 f32 81 (6.7); 16384 x 5003 f16 139 (4.7: the rows of
// one tensor and its neighbours lie alike and need no shifts, but every row's float32
// weights are moved into place, and first and last chunks are partial); one row of
// 4096 1.9 and 2.9.
#include "common.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

namespace gptq {

namespace {

constexpr int kWideThreads = 1024;

__device__ __forceinline__ float load_as_f32(const float* p) { return *p; }
__device__ __forceinline__ float load_as_f32(const __half* p) { return __half2float(*p); }
__device__ __forceinline__ float load_as_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_rounded(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_rounded(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_rounded(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

__device__ __forceinline__ float2 widen(uint32_t w, const __half*)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
__device__ __forceinline__ float2 widen(uint32_t w, const __nv_bfloat16*)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t narrow(float a, float b, const __half*)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t narrow(float a, float b, const __nv_bfloat16*)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Two neighbouring values at a time: one instruction for both.
__device__ __forceinline__ uint64_t bits_of(float2 v)
{
    return static_cast<uint64_t>(__float_as_uint(v.y)) << 32 | __float_as_uint(v.x);
}
__device__ __forceinline__ float2 pair_of(uint64_t b)
{
    return make_float2(__uint_as_float(static_cast<uint32_t>(b)), __uint_as_float(static_cast<uint32_t>(b >> 32)));
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)), "l"(bits_of(c)));
    return pair_of(d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return pair_of(d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits_of(a)), "l"(bits_of(b)));
    return pair_of(d);
}

// ---------------------------------------------------------------- chunks
// 16 bytes of a row as they lie in memory, and how many elements that is.
// Loads stand apart from what is computed with them: a thread's loads are all
// on their way before the first is used.
template <typename T>
constexpr int kVec = 16 / static_cast<int>(sizeof(T));

// The longest row kept in registers: four chunks a thread.
template <typename T>
constexpr int kHeldCols = 4 * kWideThreads * kVec<T>;

// A row and a chunk of it: elements k .. k + kVec<T> - 1, of which those in
// 0 .. K - 1 are there.  SHIFT: the row may begin off a 16-byte boundary (k
// may then be negative, and the last chunk partial); else every chunk is whole.
template <typename T>
__device__ __forceinline__ bool whole(int k, int K) { return k >= 0 && k + kVec<T> <= K; }

// Elements of a chunk that are not there become 0.
template <typename T>
__device__ __forceinline__ uint4 only_there(uint4 u, int k, int K)
{
    uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            if (k + i < 0 || k + i >= K) w[i] = 0u;
        } else {
            if (k + 2 * i < 0 || k + 2 * i >= K) w[i] &= 0xffff0000u;
            if (k + 2 * i + 1 < 0 || k + 2 * i + 1 >= K) w[i] &= 0x0000ffffu;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes at byte offset `o` (0 .. 15, a multiple of 2) of 32.
__device__ __forceinline__ uint4 shifted(uint4 a, uint4 b, int o)
{
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = (o & 8) ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = (o & 4) ? w[i + 1] : w[i];
    const int bits = 8 * (o & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], bits);
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// 16 bytes, or four times `other` where they are not there (a predicate, no
// branch: with 8 values a chunk, the branches around its loads and stores were
// a sixth of the instructions).  Rows pass the L1 cache by, so that what every
// row reads (KEEP) stays in it.  Not by the read-only path: a row may be
// written in place, and a kernel that was started early was there before its
// inputs were.
template <bool KEEP>
__device__ __forceinline__ uint4 load16(const void* p, bool there, uint32_t other = 0u)
{
    uint4 u;
    if constexpr (KEEP)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b32 %0, %6;\n\tmov.b32 %1, %6;\n\tmov.b32 %2, %6;\n\tmov.b32 %3, %6;\n\t"
            "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
            : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
            : "l"(p), "r"(static_cast<uint32_t>(there)), "r"(other));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %5, 0;\n\t"
            "mov.b32 %0, %6;\n\tmov.b32 %1, %6;\n\tmov.b32 %2, %6;\n\tmov.b32 %3, %6;\n\t"
            "@p ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}\n"
            : "=&r"(u.x), "=&r"(u.y), "=&r"(u.z), "=&r"(u.w)
            : "l"(p), "r"(static_cast<uint32_t>(there)), "r"(other));
    return u;
}

// The aligned 16 bytes at p, where one of them is between lo and hi: no byte
// of another 16 is touched.
__device__ __forceinline__ uint4 piece(uintptr_t p, uintptr_t lo, uintptr_t hi)
{
    return load16<true>(reinterpret_cast<const void*>(p), p + 16 > lo && p < hi);
}

template <typename T, bool SHIFT, bool KEEP = false>
__device__ __forceinline__ uint4 load_chunk(const T* row, int k, int K, bool live)
{
    if constexpr (!SHIFT) {
        return load16<KEEP>(row + k, live && k < K);
    } else {
        if (!live || k >= K) return make_uint4(0u, 0u, 0u, 0u);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(row), hi = lo + K * sizeof(T);
        const uintptr_t at = lo + static_cast<int64_t>(k) * static_cast<int64_t>(sizeof(T));
        const int o = static_cast<int>(at & 15);
        uint4 u = piece(at - o, lo, hi);
        if (o) u = shifted(u, piece(at - o + 16, lo, hi), o);
        return whole<T>(k, K) ? u : only_there<T>(u, k, K);
    }
}

// A chunk in float32, as pairs.
template <typename T>
struct Chunk {
    float2 v[kVec<T> / 2];
};

template <typename T>
__device__ __forceinline__ Chunk<T> widen_chunk(uint4 u)
{
    Chunk<T> c;
    if constexpr (sizeof(T) == 4) {
        c.v[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        c.v[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    } else {
        const T* t = nullptr;
        c.v[0] = widen(u.x, t);
        c.v[1] = widen(u.y, t);
        c.v[2] = widen(u.z, t);
        c.v[3] = widen(u.w, t);
    }
    return c;
}

template <typename T, bool SHIFT>
__device__ __forceinline__ void store_chunk(T* row, int k, int K, const Chunk<T>& c)
{
    if (!SHIFT || (whole<T>(k, K) && reinterpret_cast<uintptr_t>(row + k) % 16 == 0)) {
        uint4 u;
        if constexpr (sizeof(T) == 4)
            u = make_uint4(__float_as_uint(c.v[0].x), __float_as_uint(c.v[0].y), __float_as_uint(c.v[1].x), __float_as_uint(c.v[1].y));
        else
            u = make_uint4(narrow(c.v[0].x, c.v[0].y, row), narrow(c.v[1].x, c.v[1].y, row), narrow(c.v[2].x, c.v[2].y, row),
                           narrow(c.v[3].x, c.v[3].y, row));
        *reinterpret_cast<uint4*>(row + k) = u;
    } else {
#pragma unroll
        for (int j = 0; j < kVec<T>; ++j)
            if (k + j >= 0 && k + j < K) store_rounded(row + k + j, j % 2 ? c.v[j / 2].y : c.v[j / 2].x);
    }
}

// c *= the float32 weights of the chunk's elements, where there are any.  Off
// the boundaries: the aligned pieces that hold them, moved by whole words (the
// same for all of a row), and 0 for elements that are not there, so that
// nothing of what lies behind the weights meets the row's zeros.
template <typename T, bool SHIFT>
__device__ __forceinline__ void times_weights(Chunk<T>& c, const float* w, int k, int K, bool any)
{
    constexpr int VEC = kVec<T>;
    if constexpr (!SHIFT) {
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) {
            const Chunk<float> f = widen_chunk<float>(load16<true>(w + k + 4 * i, any && k < K, 0x3f800000u));
            c.v[2 * i] = mul2(c.v[2 * i], f.v[0]);
            c.v[2 * i + 1] = mul2(c.v[2 * i + 1], f.v[1]);
        }
    } else {
        if (!any || k >= K) return;
        float f[VEC + 4];
        if (reinterpret_cast<uintptr_t>(w) % 16 == 0) {
            const int first = k & ~3;
#pragma unroll
            for (int i = 0; i < VEC + 4; i += 4) {
                const uint4 u = load16<true>(w + first + i, first + i >= 0 && first + i < K);
                f[i] = __uint_as_float(u.x);
                f[i + 1] = __uint_as_float(u.y);
                f[i + 2] = __uint_as_float(u.z);
                f[i + 3] = __uint_as_float(u.w);
            }
#pragma unroll
            for (int i = 0; i < VEC + 2; ++i) f[i] = (k & 2) ? f[i + 2] : f[i];
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = (k & 1) ? f[i + 1] : f[i];
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i) f[i] = k + i >= 0 && k + i < K ? w[k + i] : 0.f;
        }
        if (!whole<T>(k, K)) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                if (k + i < 0 || k + i >= K) f[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VEC / 2; ++i) c.v[i] = mul2(c.v[i], make_float2(f[2 * i], f[2 * i + 1]));
    }
}

// Elements of the row before the first 16-byte boundary's chunk: chunk c is
// at k = kVec c - lead.
template <typename T>
__device__ __forceinline__ int lead_of(const void* row)
{
    return static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(T));
}

// ------------------------------------------------------------- reductions
// silu(a) = a / (1 + exp(-a)).  Rounding -a log2(e) costs exp |a| half steps
// of float32, the two approximations (2 steps and 1) and the rest 9.  Where
// exp(-a) passes 2^126 (a below -87.3) the reciprocal would be subnormal and is 0,
// and so is silu; an infinite negative a gives NaN.
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float reciprocal_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 silu(float2 a)
{
    const float2 x = mul2(a, both(-1.44269504f));
    const float2 d = add2(make_float2(exp2_approx(x.x), exp2_approx(x.y)), both(1.f));
    return mul2(a, make_float2(reciprocal_approx(d.x), reciprocal_approx(d.y)));
}

// The threads of a row: whole warps, or (SHORT) 8 or 16 neighbouring lanes.
template <bool SHORT>
struct RowThreads {
    int threads;   // of a row
    int tid;       // this thread's place among them
    int row;       // the block's row

    __device__ explicit RowThreads(int threads_)
        : threads(threads_), tid(threadIdx.x % threads_), row(threadIdx.x / threads_) {}
    __device__ int warps() const { return SHORT ? 1 : threads / 32; }
    __device__ int width() const { return SHORT ? threads : 32; }
    __device__ int lane() const { return tid & (width() - 1); }
    __device__ uint32_t lanes() const
    {
        return SHORT ? ((1u << threads) - 1u) << ((threadIdx.x & 31) & ~(threads - 1)) : 0xffffffffu;
    }
};

__device__ __forceinline__ float warp_sum(float v, int width = 32)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < width) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Over the threads of a row.  Each reduction of a kernel has slots of its own,
// so that one barrier each is enough.  A block has several rows only where
// they have four warps at most.
template <bool SHORT>
__device__ __forceinline__ int row_slot(const RowThreads<SHORT>& r) { return r.warps() <= 4 ? 4 * r.row : 0; }

template <bool SHORT>
__device__ __forceinline__ float row_sum(float v, float (&part)[32], const RowThreads<SHORT>& r)
{
    v = warp_sum(v, r.width());
    const int warps = r.warps();
    if (warps == 1) return v;
    const float* p = part + row_slot(r);
    if (r.lane() == 0) part[row_slot(r) + (r.tid >> 5)] = v;
    __syncthreads();
    if (warps <= 4) return (p[0] + p[1]) + (warps > 2 ? p[2] + (warps > 3 ? p[3] : 0.f) : 0.f);
    return warp_sum(r.lane() < warps ? p[r.lane()] : 0.f);
}

template <bool SHORT>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t (&part)[32], const RowThreads<SHORT>& r)
{
    v = __reduce_max_sync(r.lanes(), v);
    if (r.warps() == 1) return v;
    if (r.lane() == 0) part[row_slot(r) + (r.tid >> 5)] = v;
    __syncthreads();
    return __reduce_max_sync(0xffffffffu, r.lane() < r.warps() ? part[row_slot(r) + r.lane()] : 0u);
}

// The sum ends up with the row's first warp.
template <bool SHORT>
__device__ __forceinline__ int row_sum_first(int v, int (&part)[32], const RowThreads<SHORT>& r)
{
    v = __reduce_add_sync(r.lanes(), v);
    if (r.warps() == 1) return v;
    if (r.lane() == 0) part[row_slot(r) + (r.tid >> 5)] = v;
    __syncthreads();
    return r.tid < 32 ? __reduce_add_sync(0xffffffffu, r.lane() < r.warps() ? part[row_slot(r) + r.lane()] : 0) : 0;
}

// ------------------------------------------------------------------ codes
// A row's codes: q = rint(127 v / t), t = max |v|.
//
// One multiply-add: rint(v r), r = 127 / t rounded up, by adding kRound (1.5 *
// 2^23): the sum's only rounding is to a whole number, and a code's two's
// complement is its low byte.  Where t is so small or large that r would leave
// the normal numbers, v and t are taken times c = 2^+-100 first.
//
// This gives the exact codes of values of 8 or 11 significant bits: a quotient
// below 2^(8-p) that is no tie lies 2^-(12+p) or more from one, and v r within
// 2^-(15+p) of the quotient.  Of a tie, 254 v / t is an odd number; 127 being a
// prime, t's odd part then is a multiple of 127 or 2 |v| = t.  In the second
// case the tie is 63.5, and r being no less than 127 / t it goes to 64, as it
// should.  In the first r is a power of two and v r exact if the odd part is
// 127 itself; rows of other multiples (11 bits: 7 of 1024 significands) divide:
// the product with the rounded reciprocal of t and one correction step give
// the quotient of 127 v (18 bits, exact) and t rounded to nearest (Markstein;
// the exception, a divisor whose significand is all ones, has 24 bits), and a
// tie is representable.
//
// Values of 24 bits (EXACT): a quotient within 2^-13 of a tie h is decided by
// the sign of 254 v - 2 h t: the product 254 v in two parts, 2 h t from the
// first part without a rounding, since the two are so near.
constexpr float kRound = 12582912.f;

enum CodeKind { kZeros, kMultiply, kDivide };

struct TokenGrid {
    __device__ bool plain() const { return kind == kMultiply && c == 1.f; }

    CodeKind kind;   // kZeros: a row of zeros, or one that holds an infinity or NaN
    float scale;     // t / 127; NaN for a row that is not finite
    float c, t, r;   // 2^0 or 2^+-100; c times the maximum; 127 / t rounded up
};

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// The row's maximum is given by its bits: as unsigned integers the magnitudes'
// bits keep their order, with infinities and then NaN above every finite value.
template <bool ELEVEN>
__device__ __forceinline__ TokenGrid token_grid(uint32_t top_bits)
{
    TokenGrid g;
    const float top = __uint_as_float(top_bits);
    const bool finite = top_bits < 0x7f800000u;
    g.scale = finite ? __fdiv_rn(top, 127.f) : __uint_as_float(0x7fffffffu);
    g.c = top < 0x1p-100f ? 0x1p100f : top > 0x1p100f ? 0x1p-100f : 1.f;
    g.t = top * g.c;
    g.r = __fdiv_ru(127.f, g.t);
    const bool ties = ELEVEN && (((top_bits & 0x7fffffu) | 0x800000u) >> 13) % 127u == 0u;
    g.kind = top_bits == 0u || !finite ? kZeros : ties ? kDivide : kMultiply;
    return g;
}

// kRound + the code of v, whose quotient is next to a tie: c is one side's.
__device__ __forceinline__ float beside_tie(float v, float c, const TokenGrid& g)
{
    const float q = c - kRound;
    const float side = copysignf(1.f, fmaf(v, g.r, -q));
    const float h2 = 2.f * q + side;
    const float p = 254.f * v;
    const float d = fmaf(-h2, g.t, p) + fmaf(254.f, v, -p);
    // over the tie, or on it and q odd
    const bool over = d * side > 0.f || (d == 0.f && (static_cast<int>(q) & 1));
    return over ? c + side : c;
}

// A pair becomes kRound + its codes.
template <bool EXACT>
__device__ __forceinline__ float2 multiplied(float2 v, const TokenGrid& g)
{
    float2 c = fma2(v, both(g.r), both(kRound));
    if (EXACT) {
        const float2 f = fma2(v, both(g.r), make_float2(kRound - c.x, kRound - c.y));
        if (fabsf(f.x) > 0.5f - 0x1p-13f) c.x = beside_tie(v.x, c.x, g);
        if (fabsf(f.y) > 0.5f - 0x1p-13f) c.y = beside_tie(v.y, c.y, g);
    }
    return c;
}

template <bool ELEVEN, bool EXACT>
__device__ __forceinline__ float2 code_pair(float2 v, const TokenGrid& g)
{
    if (g.kind == kZeros) return both(kRound);
    if (g.c != 1.f) v = mul2(v, both(g.c));
    if (!ELEVEN || g.kind == kMultiply) return multiplied<EXACT>(v, g);
    const float rt = __frcp_rn(g.t);
    auto code = [&](float x) {
        const float a = 127.f * x, q = a * rt;
        return kRound + fmaf(fmaf(-q, g.t, a), rt, q);
    };
    return make_float2(code(v.x), code(v.y));
}

// A chunk's; PLAIN: a row of kind kMultiply with c = 1.
template <typename T, bool ELEVEN, bool EXACT, bool PLAIN>
__device__ __forceinline__ void code_chunk(Chunk<T>& c, const TokenGrid& g)
{
#pragma unroll
    for (int j = 0; j < kVec<T> / 2; ++j)
        c.v[j] = PLAIN ? multiplied<EXACT>(c.v[j], g) : code_pair<ELEVEN, EXACT>(c.v[j], g);
}

__device__ __forceinline__ uint32_t pack4(float2 a, float2 b)
{
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

// Stores the codes of the chunk at k (elements not there have code 0) and
// returns their sum.  Off the boundaries of the codes' row a whole chunk goes
// in up to four aligned pieces, the same for all of a row.
template <typename T, bool SHIFT>
__device__ __forceinline__ int store_codes(int8_t* row, int k, int K, bool live, const Chunk<T>& c)
{
    constexpr int VEC = kVec<T>;
    uint32_t w[VEC / 4];
    int sum = 0;
#pragma unroll
    for (int j = 0; j < VEC / 4; ++j) {
        w[j] = pack4(c.v[2 * j], c.v[2 * j + 1]);
        sum = __dp4a(static_cast<int>(w[j]), 0x01010101, sum);
    }
    if (!row || !live || k >= K) return sum;
    if (!SHIFT || (k >= 0 && k % VEC == 0 && k + VEC <= K)) {
        if constexpr (VEC == 8)
            *reinterpret_cast<uint2*>(row + k) = make_uint2(w[0], w[VEC / 4 - 1]);
        else
            *reinterpret_cast<uint32_t*>(row + k) = w[0];
        return sum;
    }
    uint64_t codes = VEC == 8 ? static_cast<uint64_t>(w[VEC / 4 - 1]) << 32 | w[0] : w[0];
    int8_t* p = row + k;
    if (whole<T>(k, K)) {
        int left = VEC;
        if (k & 1) {
            *p = static_cast<int8_t>(codes);
            codes >>= 8;
            p += 1;
            left -= 1;
        }
        if (reinterpret_cast<uintptr_t>(p) & 2) {
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(codes);
            codes >>= 16;
            p += 2;
            left -= 2;
        }
        if (left >= 4) {
            *reinterpret_cast<uint32_t*>(p) = static_cast<uint32_t>(codes);
            codes >>= 32;
            p += 4;
            left -= 4;
        }
        if (left & 4) {   // only where two pieces of 4 follow each other
            *reinterpret_cast<uint32_t*>(p) = static_cast<uint32_t>(codes);
            return sum;
        }
        if (left & 2) {
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(codes);
            codes >>= 16;
            p += 2;
        }
        if (left & 1) *p = static_cast<int8_t>(codes);
    } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            if (k + j >= 0 && k + j < K) p[j] = static_cast<int8_t>(codes >> (8 * j));
    }
    return sum;
}

// Asks for row `m` of `cols` elements to be brought into L2 (its whole 16-byte
// pieces).
template <typename T>
__device__ __forceinline__ void prefetch_row(const T* rows, int64_t ld, int64_t m, int cols)
{
    const uintptr_t lo = (reinterpret_cast<uintptr_t>(rows + m * ld) + 15) & ~uintptr_t(15);
    const uintptr_t hi = reinterpret_cast<uintptr_t>(rows + m * ld + cols) & ~uintptr_t(15);
    if (hi > lo)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"(static_cast<uint32_t>(hi - lo)) : "memory");
}

// ---------------------------------------------------------------- kernels
struct TokenArgs {
    int8_t* Xq;
    int64_t ldq;
    float* x_scales;
    int32_t* x_sums;
    void* hat;
    int64_t ldh;
    const void* X;
    int64_t ldx;
    const void* gate;
    int64_t ldg;
    int64_t M;
    int K;
    int64_t ahead;
};

template <typename T, int CH, bool SHIFT, bool GATE, bool SHORT, bool THREE = false>
__global__ void __launch_bounds__(THREE ? 384 : kWideThreads, THREE ? 3 : 1) quantize_tokens_kernel(const TokenArgs a, int threads)
{
    constexpr int VEC = kVec<T>;
    __shared__ uint32_t part_top[32];
    __shared__ int part_sum[32];
    pdl_trigger();
    pdl_wait();
    const RowThreads<SHORT> row(threads);
    const int tid = row.tid;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (blockDim.x / threads) + row.row;
    const bool live = m < a.M;
    const T* x = static_cast<const T*>(a.X) + m * a.ldx;
    const T* gate = static_cast<const T*>(a.gate) + m * a.ldg;
    T* hat = static_cast<T*>(a.hat) + m * a.ldh;
    const int k0 = tid * VEC - (SHIFT ? lead_of<T>(a.hat ? hat : x) : 0);
    if (tid == 0 && a.ahead && m + a.ahead < a.M) {
        prefetch_row(static_cast<const T*>(a.X), a.ldx, m + a.ahead, a.K);
        if (GATE) prefetch_row(static_cast<const T*>(a.gate), a.ldg, m + a.ahead, a.K);
    }
    uint4 xr[CH], gr[GATE ? CH : 1];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        xr[i] = load_chunk<T, SHIFT>(x, k0 + i * threads * VEC, a.K, live);
        if (GATE) gr[i] = load_chunk<T, SHIFT>(gate, k0 + i * threads * VEC, a.K, live);
    }
    // what is kept through the reduction: 16-bit values as they are, else float32
    constexpr bool PACKED = !GATE && sizeof(T) == 2;
    Chunk<T> v[PACKED ? 1 : CH];
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        if constexpr (PACKED) {   // two magnitudes at a time
            const uint32_t mask = 0x7fff7fffu;
            top = __vmaxu2(__vmaxu2(top, xr[i].x & mask),
                           __vmaxu2(xr[i].y & mask, __vmaxu2(xr[i].z & mask, xr[i].w & mask)));
        } else {
            v[i] = widen_chunk<T>(xr[i]);
            if (GATE) {
                const Chunk<T> s = widen_chunk<T>(gr[i]);
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) v[i].v[j] = mul2(v[i].v[j], silu(s.v[j]));
            }
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) top = max(max(top, magnitude(v[i].v[j].x)), magnitude(v[i].v[j].y));
        }
    }
    if constexpr (PACKED) {
        const float2 two = widen(top, x);
        top = max(__float_as_uint(two.x), __float_as_uint(two.y));
    }
    constexpr bool ELEVEN = PACKED && std::is_same<T, __half>::value;
    const TokenGrid g = token_grid<ELEVEN>(row_max(top, part_top, row));
    int sum = 0;
    int8_t* q = a.Xq ? a.Xq + m * a.ldq : nullptr;
    auto finish = [&](auto plain) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = k0 + i * threads * VEC;
            Chunk<T>& w = v[PACKED ? 0 : i];
            if constexpr (PACKED) w = widen_chunk<T>(xr[i]);
            code_chunk<T, ELEVEN, !GATE && sizeof(T) == 4, decltype(plain)::value>(w, g);
            sum += store_codes<T, SHIFT>(q, k, a.K, live, w);
            if (a.hat && live && k < a.K) {
#pragma unroll
                for (int j = 0; j < VEC / 2; ++j) w.v[j] = mul2(add2(w.v[j], both(-kRound)), both(g.scale));
                store_chunk<T, SHIFT>(hat, k, a.K, w);
            }
        }
    };
    if (g.plain())
        finish(std::true_type());
    else
        finish(std::false_type());
    if (a.x_sums) {
        sum = row_sum_first(sum, part_sum, row);
        if (live && tid == 0) a.x_sums[m] = sum;
    }
    if (live && tid == 0) a.x_scales[m] = g.scale;
}

template <typename T, int CH, bool SHIFT, bool GATE, bool SHORT, bool THREE = false>
__global__ void __launch_bounds__(THREE ? 384 : kWideThreads, THREE ? 3 : 1) block_norm_kernel(const BlockNormArgs a, int threads)
{
    constexpr int VEC = kVec<T>;
    __shared__ float part_post[32], part_pre[32];
    __shared__ uint32_t part_top[32];
    __shared__ int part_sum[32];
    pdl_trigger();
    pdl_wait();
    const RowThreads<SHORT> row(threads);
    const int tid = row.tid;
    const int64_t m = static_cast<int64_t>(blockIdx.x) * (blockDim.x / threads) + row.row;
    const bool live = m < a.M;
    const int D = static_cast<int>(a.D);
    const T* block = static_cast<const T*>(a.block) + m * a.ldb;
    const T* residual = static_cast<const T*>(a.residual) + m * a.ldr;
    const T* gate = static_cast<const T*>(a.gate) + (GATE && live ? m / a.gate_rows : 0) * a.ldg;
    T* stream_out = static_cast<T*>(a.stream_out) + m * a.lds;
    T* out = static_cast<T*>(a.out) + m * a.ldo;
    const int k0 = tid * VEC - (SHIFT ? lead_of<T>(a.stream_out ? stream_out : a.out ? out : a.block ? block : residual) : 0);
    const int step = threads * VEC;
    if (tid == 0 && a.ahead && m + a.ahead < a.M) {
        if (a.block) prefetch_row(static_cast<const T*>(a.block), a.ldb, m + a.ahead, D);
        if (a.residual) prefetch_row(static_cast<const T*>(a.residual), a.ldr, m + a.ahead, D);
        if (GATE && a.gate_rows == 1) prefetch_row(static_cast<const T*>(a.gate), a.ldg, m + a.ahead, D);
    }
    uint4 br[CH], rr[CH], gr[GATE ? CH : 1];
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        br[i] = load_chunk<T, SHIFT>(block, k0 + i * step, D, live && a.block);
        rr[i] = load_chunk<T, SHIFT>(residual, k0 + i * step, D, live && a.residual);
        if (GATE) gr[i] = load_chunk<T, SHIFT, true>(gate, k0 + i * step, D, live);
    }
    float scale = a.block ? a.scale : 0.f;
    if (a.block && a.post_norm) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const Chunk<T> c = widen_chunk<T>(br[i]);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) s = fma2(c.v[j], c.v[j], s);
        }
        scale *= rsqrtf(row_sum(s.x + s.y, part_post, row) / static_cast<float>(D) + a.eps);
    }
    const bool weighted = a.post_norm && a.post_weight, store_stream = a.stream_out && live;
    Chunk<T> h[CH];
    float2 s = both(0.f);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int k = k0 + i * step;
        h[i] = widen_chunk<T>(br[i]);
        times_weights<T, SHIFT>(h[i], a.post_weight, k, D, weighted);
        if (GATE) {
            const Chunk<T> f = widen_chunk<T>(gr[i]);
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) h[i].v[j] = mul2(h[i].v[j], f.v[j]);
        }
        const Chunk<T> r = widen_chunk<T>(rr[i]);
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
            h[i].v[j] = fma2(both(scale), h[i].v[j], r.v[j]);
            s = fma2(h[i].v[j], h[i].v[j], s);
        }
        if (store_stream && k < D) store_chunk<T, SHIFT>(stream_out, k, D, h[i]);
        times_weights<T, SHIFT>(h[i], a.pre_weight, k, D, a.pre_weight);
        if (a.q) {
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) top = max(max(top, magnitude(h[i].v[j].x)), magnitude(h[i].v[j].y));
        }
    }
    if (!a.out && !a.q) return;
    const float pre = rsqrtf(row_sum(s.x + s.y, part_pre, row) / static_cast<float>(D) + a.eps);
    if (a.out) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int k = k0 + i * step;
            Chunk<T> f;
#pragma unroll
            for (int j = 0; j < VEC / 2; ++j) f.v[j] = mul2(h[i].v[j], both(pre));
            if (live && k < D) store_chunk<T, SHIFT>(out, k, D, f);
        }
    }
    if (!a.q) return;
    // the codes are those of r' w: the factor rsqrt(...) of the row cancels in 127 v / t
    const TokenGrid g = token_grid<false>(row_max(top, part_top, row));
    int sum = 0;
    auto finish = [&](auto plain) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            code_chunk<T, false, false, decltype(plain)::value>(h[i], g);
            sum += store_codes<T, SHIFT>(a.q + m * a.ldq, k0 + i * step, D, live, h[i]);
        }
    };
    if (g.plain())
        finish(std::true_type());
    else
        finish(std::false_type());
    if (a.q_sums) {
        sum = row_sum_first(sum, part_sum, row);
        if (live && tid == 0) a.q_sums[m] = sum;
    }
    if (live && tid == 0) a.q_scales[m] = g.scale * pre;
}

// -- rows longer than kHeldCols: one block a row, which reads it again (from
// L2) for each pass over it, element by element.  Right, not fast: tokens of
// 2048 x 53248 bf16 122 us (2.7 TB/s), gated 218 (2.5), 2048 x 28672 f32 93
// (3.2); norm of 2048 x 40000 bf16 645 (1.0), of 2048 x 53248 to tokens 901 (0.8)

template <typename T>
__global__ void __launch_bounds__(kWideThreads) quantize_wide_tokens_kernel(const TokenArgs a)
{
    __shared__ uint32_t part_top[32];
    __shared__ int part_sum[32];
    const int64_t m = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    const RowThreads<false> row(kWideThreads);
    const T* x = static_cast<const T*>(a.X) + m * a.ldx;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + m * a.ldg : nullptr;
    auto value = [&](int k) {
        const float v = load_as_f32(x + k);
        return gate ? v * silu(both(load_as_f32(gate + k))).x : v;
    };
    uint32_t top = 0;
    for (int k = threadIdx.x; k < a.K; k += kWideThreads) top = max(top, magnitude(value(k)));
    top = row_max(top, part_top, row);
    const TokenGrid g = gate ? token_grid<false>(top) : token_grid<std::is_same<T, __half>::value>(top);
    int sum = 0;
    for (int k = threadIdx.x; k < a.K; k += kWideThreads) {
        const float2 v = both(value(k));
        const float q =
            (gate ? code_pair<false, false>(v, g) : code_pair<std::is_same<T, __half>::value, sizeof(T) == 4>(v, g)).x - kRound;
        sum += static_cast<int>(q);
        if (a.Xq) a.Xq[m * a.ldq + k] = static_cast<int8_t>(q);
        if (a.hat) store_rounded(static_cast<T*>(a.hat) + m * a.ldh + k, q * g.scale);
    }
    if (a.x_sums) {
        sum = row_sum_first(sum, part_sum, row);
        if (threadIdx.x == 0) a.x_sums[m] = sum;
    }
    if (threadIdx.x == 0) a.x_scales[m] = g.scale;
}

template <typename T>
__global__ void __launch_bounds__(kWideThreads) block_norm_wide_kernel(const BlockNormArgs a)
{
    __shared__ float part_post[32], part_pre[32];
    __shared__ uint32_t part_top[32];
    __shared__ int part_sum[32];
    const int64_t m = blockIdx.x;
    pdl_trigger();
    pdl_wait();
    const RowThreads<false> row(kWideThreads);
    const int D = static_cast<int>(a.D);
    const T* block = a.block ? static_cast<const T*>(a.block) + m * a.ldb : nullptr;
    const T* residual = a.residual ? static_cast<const T*>(a.residual) + m * a.ldr : nullptr;
    const T* gate = a.gate ? static_cast<const T*>(a.gate) + (m / a.gate_rows) * a.ldg : nullptr;
    float scale = a.scale;
    if (block && a.post_norm) {
        float s = 0.f;
        for (int k = threadIdx.x; k < D; k += kWideThreads) {
            const float h = load_as_f32(block + k);
            s = fmaf(h, h, s);
        }
        scale *= rsqrtf(row_sum(s, part_post, row) / static_cast<float>(D) + a.eps);
    }
    auto value = [&](int k) {
        const float r = residual ? load_as_f32(residual + k) : 0.f;
        if (!block) return r;
        float h = load_as_f32(block + k);
        if (a.post_norm && a.post_weight) h *= a.post_weight[k];
        if (gate) h *= load_as_f32(gate + k);
        return fmaf(scale, h, r);
    };
    auto weighted = [&](float r, int k) { return a.pre_weight ? r * a.pre_weight[k] : r; };
    float s = 0.f;
    uint32_t top = 0;
    for (int k = threadIdx.x; k < D; k += kWideThreads) {
        const float r = value(k);
        s = fmaf(r, r, s);
        top = max(top, magnitude(weighted(r, k)));
    }
    const float pre = rsqrtf(row_sum(s, part_pre, row) / static_cast<float>(D) + a.eps);
    const TokenGrid g = token_grid<false>(row_max(top, part_top, row));
    int sum = 0;
    for (int k = threadIdx.x; k < D; k += kWideThreads) {
        const float r = value(k);
        const float v = weighted(r, k);
        if (a.out) store_rounded(static_cast<T*>(a.out) + m * a.ldo + k, v * pre);
        if (a.stream_out) store_rounded(static_cast<T*>(a.stream_out) + m * a.lds + k, r);
        if (a.q) {
            const float q = code_pair<false, false>(both(v), g).x - kRound;
            sum += static_cast<int>(q);
            a.q[m * a.ldq + k] = static_cast<int8_t>(q);
        }
    }
    if (!a.q) return;
    if (a.q_sums) {
        sum = row_sum_first(sum, part_sum, row);
        if (threadIdx.x == 0) a.q_sums[m] = sum;
    }
    if (threadIdx.x == 0) a.q_scales[m] = g.scale * pre;
}

// -- the product's weights: 16 codes a thread, one pass at memory's rate (once
// a layer)

template <bool WHOLE>
__global__ void w8a8_pack_kernel(int8_t* Wq, int64_t ldw, int32_t* w_zeros, const uint8_t* codes, const float* zeros, int64_t N,
                                 int64_t K)
{
    const int64_t pieces = ldw / 16;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i < N) w_zeros[i] = static_cast<int32_t>(zeros[i]) - 128;
    for (int64_t p = i; p < N * pieces; p += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        const int64_t n = p / pieces, k = 16 * (p % pieces);
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (WHOLE) {   // rows of whole, aligned pieces
            if (k < K) {
                u = *reinterpret_cast<const uint4*>(codes + n * K + k);
                u = make_uint4(u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u);
            }
        } else {
            uint8_t c[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) c[j] = k + j < K ? codes[n * K + k + j] ^ 0x80 : 0;
            memcpy(&u, c, 16);
        }
        *reinterpret_cast<uint4*>(Wq + n * ldw + k) = u;
    }
}

// ------------------------------------------------------------------- host
// Rows of whole, aligned 16-byte chunks (what is absent passes).
template <typename T>
bool chunks_ok(const void* p, int64_t ld)
{
    return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * sizeof(T) % 16 == 0);
}

// Launches kernel(args, threads of a row): `chunks` 16-byte pieces a row, CH a
// thread.  A block has as many rows as fit into 128 threads, one at least: rows of
// 8, 16, 32 or 64 threads share blocks of 128, one of 96 has a block to itself.
template <int CH, bool SHORT, typename Args>
int launch_rows(void (*kernel)(Args, int), const Args& args, int64_t M, int64_t chunks, cudaStream_t stream)
{
    const int threads = SHORT ? (chunks <= 8 ? 8 : 16) : static_cast<int>((chunks + 32 * CH - 1) / (32 * CH)) * 32;
    const int rows = std::max(1, 128 / threads);
    const cudaError_t e = launch_k(kernel, dim3(static_cast<unsigned>((M + rows - 1) / rows)), dim3(threads * rows), 0, stream, true,
                                   args, threads);
    if (e != cudaSuccess) return cuda_fail(e);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

// Chunks a thread, 1, 2 or 4: the fewest from `least` on with which the SMs hold
// all rows at once (at 64 registers 1024 threads each), since then the latency of
// a row counts, else `most`, which keep more bytes on their way a thread and need
// fewer warps to meet (norm of 16384 x 4096: 91 us with four, 119 with two, 167
// with one; of 444 x 4096 8.8, 6.2, 7.7; of 64 x 4096 5.1, 4.0, 3.7).  0: one, and
// part of a warp a row (norm of 500000 x 128: 91 us against 157 with a warp a row).
int chunks_a_thread(int64_t M, int64_t chunks, int least, int most)
{
    if (chunks <= 16) return 0;
    if (chunks <= 32) return 1;
    for (int n = least; n < most; n *= 2) {
        const int64_t threads = (chunks + 32 * n - 1) / (32 * n) * 32;
        if (threads <= kWideThreads && M <= kWideThreads / threads * sm_count()) return n;
    }
    return chunks <= 64 ? 2 : most;
}

template <typename T, bool SHIFT>
int64_t chunks_of(int64_t cols) { return (cols + (SHIFT ? kVec<T> - 1 : 0) + kVec<T> - 1) / kVec<T>; }

// Rows of 352 or 384 threads with four chunks each: at 64 registers a thread an
// SM holds two of them, at 56 three (tokens of a gated activation of 8192 x
// 11008: 77 us against 96; norm of 4096 x 11008 to tokens 57 against 66).  Not
// for the norm with a gate or off its boundaries, which keep a third row's
// chunks or shifts and would spill (96 against 88, 119 against 116).
bool three_blocks(int64_t chunks) { return chunks > 4 * 320 && chunks <= 4 * 384; }

template <typename T, bool SHIFT, bool GATE>
int tokens_chunked(const TokenArgs& a, cudaStream_t stream)
{
    const int64_t chunks = chunks_of<T, SHIFT>(a.K);
    // Their warps meet once: more warps with a chunk each pay only where a row has
    // two to four of them, or to eight where each has shifts to do (64 x 4096:
    // 2.0 us with two chunks, 2.4 with one; 64 x 1003 in float32 2.6 and 2.3).
    const int least = chunks > 64 && chunks < (SHIFT ? 256 : 129) ? 1 : 2;
    switch (chunks_a_thread(a.M, chunks, least, 4)) {
        case 0: return launch_rows<1, true>(quantize_tokens_kernel<T, 1, SHIFT, GATE, true>, a, a.M, chunks, stream);
        case 1: return launch_rows<1, false>(quantize_tokens_kernel<T, 1, SHIFT, GATE, false>, a, a.M, chunks, stream);
        case 2: return launch_rows<2, false>(quantize_tokens_kernel<T, 2, SHIFT, GATE, false>, a, a.M, chunks, stream);
        default: break;
    }
    if (three_blocks(chunks))
        return launch_rows<4, false>(quantize_tokens_kernel<T, 4, SHIFT, GATE, false, true>, a, a.M, chunks, stream);
    return launch_rows<4, false>(quantize_tokens_kernel<T, 4, SHIFT, GATE, false>, a, a.M, chunks, stream);
}

template <typename T, bool SHIFT, bool GATE>
int norm_chunked(const BlockNormArgs& a, cudaStream_t stream)
{
    const int64_t chunks = chunks_of<T, SHIFT>(a.D);
    // The norm with a gate keeps a third row's chunks: two of each are better for
    // short rows (8192 x 2048 27 us against 31), and off the boundaries, where
    // four spill most, while an SM holds three such rows (2048 x 5003 32 us
    // against 43; but 2048 x 8190 75 against 67).
    const int most = GATE && chunks <= (SHIFT && sizeof(T) == 2 ? 640 : 256) ? 2 : 4;
    switch (chunks_a_thread(a.M, chunks, 1, most)) {
        case 0: return launch_rows<1, true>(block_norm_kernel<T, 1, SHIFT, GATE, true>, a, a.M, chunks, stream);
        case 1: return launch_rows<1, false>(block_norm_kernel<T, 1, SHIFT, GATE, false>, a, a.M, chunks, stream);
        case 2: return launch_rows<2, false>(block_norm_kernel<T, 2, SHIFT, GATE, false>, a, a.M, chunks, stream);
        default: break;
    }
    if constexpr (!SHIFT && !GATE)
        if (three_blocks(chunks))
            return launch_rows<4, false>(block_norm_kernel<T, 4, SHIFT, GATE, false, true>, a, a.M, chunks, stream);
    return launch_rows<4, false>(block_norm_kernel<T, 4, SHIFT, GATE, false>, a, a.M, chunks, stream);
}

template <typename T>
int tokens_typed(const TokenArgs& a, cudaStream_t stream)
{
    const bool whole = a.K % kVec<T> == 0 && chunks_ok<T>(a.X, a.ldx) && chunks_ok<T>(a.gate, a.ldg) && chunks_ok<T>(a.hat, a.ldh);
    if (a.K + (whole ? 0 : kVec<T> - 1) > kHeldCols<T>) {
        const cudaError_t e = launch_k(quantize_wide_tokens_kernel<T>, dim3(static_cast<unsigned>(a.M)), dim3(kWideThreads), 0, stream, true, a);
        if (e != cudaSuccess) return cuda_fail(e);
        GPTQ_LAUNCH_CHECK();
        return GPTQ_OK;
    }
    if (whole) return a.gate ? tokens_chunked<T, false, true>(a, stream) : tokens_chunked<T, false, false>(a, stream);
    return a.gate ? tokens_chunked<T, true, true>(a, stream) : tokens_chunked<T, true, false>(a, stream);
}

template <typename T>
int norm_typed(const BlockNormArgs& a, cudaStream_t stream)
{
    const bool whole = a.D % kVec<T> == 0 && chunks_ok<T>(a.block, a.ldb) && chunks_ok<T>(a.residual, a.ldr) &&
                       chunks_ok<T>(a.gate, a.ldg) && chunks_ok<T>(a.out, a.ldo) && chunks_ok<T>(a.stream_out, a.lds) &&
                       chunks_ok<float>(a.post_weight, 4) && chunks_ok<float>(a.pre_weight, 4);
    if (a.D + (whole ? 0 : kVec<T> - 1) > kHeldCols<T>) {
        const cudaError_t e = launch_k(block_norm_wide_kernel<T>, dim3(static_cast<unsigned>(a.M)), dim3(kWideThreads), 0, stream, true, a);
        if (e != cudaSuccess) return cuda_fail(e);
        GPTQ_LAUNCH_CHECK();
        return GPTQ_OK;
    }
    if (whole) return a.gate ? norm_chunked<T, false, true>(a, stream) : norm_chunked<T, false, false>(a, stream);
    return a.gate ? norm_chunked<T, true, true>(a, stream) : norm_chunked<T, true, false>(a, stream);
}

}  // namespace

int run_quantize_tokens(int8_t* Xq, int64_t ldq, float* x_scales, int32_t* x_sums, void* hat,
                        int64_t ldh, const void* X, int64_t ldx, const void* gate, int64_t ldg,
                        int type, int64_t M, int64_t K, cudaStream_t stream)
{
    const TokenArgs a{Xq, ldq, x_scales, x_sums, hat, ldh, X, ldx, gate, ldg, M, static_cast<int>(K), 2 * sm_count()};
    if (type == GPTQ_F32) return tokens_typed<float>(a, stream);
    if (type == GPTQ_F16) return tokens_typed<__half>(a, stream);
    return tokens_typed<__nv_bfloat16>(a, stream);
}

int run_block_norm(const BlockNormArgs& a0, int type, cudaStream_t stream)
{
    BlockNormArgs a = a0;
    a.ahead = 2 * sm_count();
    if (!a.block) {   // its term is 0, whatever it would be multiplied with
        a.post_norm = 0;
        a.post_weight = nullptr;
        a.gate = nullptr;
    }
    if (type == GPTQ_F32) return norm_typed<float>(a, stream);
    if (type == GPTQ_F16) return norm_typed<__half>(a, stream);
    return norm_typed<__nv_bfloat16>(a, stream);
}

int run_w8a8_pack(int8_t* Wq, int64_t ldw, int32_t* w_zeros, const uint8_t* codes, const float* zeros,
                  int64_t N, int64_t K, cudaStream_t stream)
{
    // every zero has a thread of its own; the pieces go round
    const int64_t want = std::max(N, std::min(N * (ldw / 16), int64_t(sm_count()) * 2048 * 4));
    const unsigned blocks = static_cast<unsigned>((want + 255) / 256);
    if (K % 16 == 0 && reinterpret_cast<uintptr_t>(codes) % 16 == 0)
        w8a8_pack_kernel<true><<<blocks, 256, 0, stream>>>(Wq, ldw, w_zeros, codes, zeros, N, K);
    else
        w8a8_pack_kernel<false><<<blocks, 256, 0, stream>>>(Wq, ldw, w_zeros, codes, zeros, N, K);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

}  // namespace gptq
