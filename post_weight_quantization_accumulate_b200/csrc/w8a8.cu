// w8a8.cu -- the 8-bit linear: Y = X W^T with X and W of 8-bit codes,
//
//   Y[m][n] = x_scales[m] w_scales[n] sum_k x_q[m][k] (w_q[n][k] - z[n]) + bias[n]
//           = x_scales[m] w_scales[n] (sum_k x_q w_q - z[n] S[m]) + bias[n],
//
// S[m] = sum_k x_q[m][k].  The integer sums are exact in 32 bits for K <=
// 65536 (|x_q| <= 128, |w_q - z| <= 255: at most 2139095040 < 2^31), also
// where the two terms of the difference are not: it is taken modulo 2^32.
// Integer sums have no order, so every variant gives the same bits.
//
// tcgen05 kind::i8 with the weights' rows as the M operand and the tokens as
// the N operand: a tile's tokens can then be as few as 16, and a warp's 32
// accumulator lanes are 32 neighbouring outputs of one token, so the results
// go from registers to memory in whole sectors without a transpose, at any
// pitch and alignment of Y.  Both operands are K-major rows of 128 codes
// under the 128-byte swizzle; TMA fills what lies past K, M or N with zeros.
//
//  * pair kernel: 256 weight rows x NT tokens by a pair of CTAs (cta_group::2),
//    persistent, double-buffered accumulators, so that the scaling and the
//    stores of a tile overlap the products of the next.  Bound by the tensor
//    cores and, at full load, by the card's power: 8192 x 4096 x 11008 232 us
//    back to back (3180 TOP/s), 205 us alone (3600).
//  * split kernel: 128 weight rows x NT tokens by a cluster of CTAs that share
//    K and add their partial sums through distributed shared memory: for few
//    tokens, where the weights' way from memory is what counts and one tile a
//    CTA would leave SMs without work.  24 x 11008 x 4096 10.9 us (4.2 TB/s; 7
//    of them the weights' bytes, 3.8 a call of one stage).
//  * few kernel (8 tokens, or a few more of small weights): 16 weight rows a
//    block, the warps take turns along K and feed mma.sync straight from
//    global loads.  Nothing but the weights' bytes counts there, and the set-up
//    of tensor memory, barriers and clusters costs more than the products.
//    1 x 4096 x 4096 3.4 us (5.0 TB/s), 1 x 28672 x 8192 36.4 us (6.5 TB/s).
//
// All kernels are programmatic dependent launches: they may start while the
// kernel before them ends, set themselves up, and wait for its results
// (pdl_wait) before their first global access; for few tokens they ask for their
// first weights to be brought into L2 before that.  They let the next kernel start
// once they hold their tensor memory, never before.  A decoder layer's chain of
// such kernels: one token 46 us (50 without the requests), 24 tokens
// 59 (63 without them, 68 without early starts).
//
// The two threads of a CTA that issue loads and MMAs are the elected ones of
// their warps: under a plain lane test every such instruction took about 110
// cycles to issue instead of 45, and with that the issue bound the kernels
// (24 x 4096 x 4096 8.2 us against 6.1, 8192 x 11008 x 4096 270 against 245).
#include "pair.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <mutex>

namespace gptq {

namespace {

constexpr int kRows = 128;      // weight rows of a CTA
constexpr int kBK = 128;        // codes of K a stage
constexpr int kStep = 32;       // codes of K an MMA
constexpr int kWBytes = kRows * kBK;

__device__ __forceinline__ void store_rounded(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_rounded(__half* p, float v) { *p = __float2half_rn(v); }
__device__ __forceinline__ void store_rounded(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// The first `left` (at most 4) of four neighbouring outputs.
__device__ __forceinline__ void store4(float* p, int64_t left, float a, float b, float c, float d)
{
    if (left >= 4 && reinterpret_cast<uintptr_t>(p) % 16 == 0) {
        *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
        return;
    }
    if (left > 0) p[0] = a;
    if (left > 1) p[1] = b;
    if (left > 2) p[2] = c;
    if (left > 3) p[3] = d;
}
template <typename T>
__device__ __forceinline__ void store4(T* p, int64_t left, float a, float b, float c, float d)
{
    T v[4];
    store_rounded(v, a);
    store_rounded(v + 1, b);
    store_rounded(v + 2, c);
    store_rounded(v + 3, d);
    if (left >= 4 && reinterpret_cast<uintptr_t>(p) % 8 == 0) {
        uint2 u;
        memcpy(&u, v, 8);
        *reinterpret_cast<uint2*>(p) = u;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < left) p[j] = v[j];
}

// Instruction descriptor of kind::i8: 32-bit integer sums of signed 8-bit
// operands, both K-major.
__host__ __device__ constexpr uint32_t idesc_i8(uint32_t M, uint32_t N)
{
    return (2u << 4) | (1u << 7) | (1u << 10) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

template <int GROUP>
__device__ __forceinline__ void umma_i8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    if constexpr (GROUP == 2)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
            "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
            : "memory");
}

// The MMAs of one stage: `codes` codes of K (or all of them) from the
// descriptors of its two operands.
template <int GROUP>
__device__ __forceinline__ void stage_mmas(uint32_t d, uint64_t wd, uint64_t xd, uint32_t idesc, int codes, bool first)
{
    umma_i8<GROUP>(d, wd, xd, idesc, first ? 0u : 1u);
    if (codes >= kBK) {
#pragma unroll
        for (int k = 1; k < kBK / kStep; ++k) umma_i8<GROUP>(d, wd + k * (kStep >> 4), xd + k * (kStep >> 4), idesc, 1u);
    } else {
        for (int k = 1; k * kStep < codes; ++k) umma_i8<GROUP>(d, wd + k * (kStep >> 4), xd + k * (kStep >> 4), idesc, 1u);
    }
}

// True for one lane of a converged warp.  The compiler knows that one thread
// runs what it guards and issues tcgen05 instructions there straight.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(one));
    return one != 0;
}

// The accumulators of a lane, 16 or 32 columns.
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, int (&v)[16])
{
    float f[16];
    tmem_ld_32x32b_x16(taddr, f);
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __float_as_int(f[i]);
}
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, int (&v)[32])
{
    float f[32];
    tmem_ld_32x32b_x32(taddr, f);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __float_as_int(f[i]);
}

// What the outputs of one weight row n share.
struct RowScale {
    float scale, bias;
    uint32_t zero;
};

__device__ __forceinline__ RowScale row_scale(const W8A8Args& a, int64_t n)
{
    RowScale r{0.f, 0.f, 0u};
    if (n < a.N) {
        r.scale = a.w_scales[n];
        if (a.bias) r.bias = a.bias[n];
        if (a.w_zeros) r.zero = static_cast<uint32_t>(a.w_zeros[n]);
    }
    return r;
}

// A token's scale and sum, as bits.
__device__ __forceinline__ uint2 token_scale(const W8A8Args& a, int64_t m)
{
    if (m >= a.M) return make_uint2(0u, 0u);
    return make_uint2(__float_as_uint(a.x_scales[m]), a.w_zeros ? static_cast<uint32_t>(a.x_sums[m]) : 0u);
}

__device__ __forceinline__ float output(int acc, const RowScale& r, uint2 t)
{
    const int sum = static_cast<int>(static_cast<uint32_t>(acc) - r.zero * t.y);
    return __fadd_rn(__fmul_rn(__fmul_rn(static_cast<float>(sum), r.scale), __uint_as_float(t.x)), r.bias);
}

// Asks for a box of the weights to be brought into L2, before the kernel before
// has ended: nothing is read yet, and L2 sees what is written later too.  In the
// split kernel 24 x 11008 x 4096 in a row 11.2 -> 10.9 us and a layer's chain
// 63 -> 60, for 5.8 -> 6.3 where a product of 16 MB follows the like of itself; in
// the pair kernel, with more tokens for each weight, it does not pay (512 x 4096 x
// 4096 12.8 -> 13.5).
__device__ __forceinline__ void prefetch_box(const CUtensorMap* map, int x, int y)
{
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];" ::"l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y)
                 : "memory");
}

// ------------------------------------------------------------- pair kernel
constexpr int kEpiWarps = 16;
constexpr int kPairThreads = 128 + 32 * kEpiWarps;
// Between its looks at a barrier a waiting epilogue warp sleeps this long (ns):
// sixteen polling warps slow the two threads that issue the loads and MMAs.
constexpr unsigned kNap = 100;

template <int NT>
struct alignas(1024) PairSmem {
    static constexpr int kXBytes = NT / 2 * kBK;    // this CTA's half of the tokens
    static constexpr int kStageBytes = kWBytes + kXBytes;
    static constexpr int kStages = 192 * 1024 / kStageBytes;
    uint8_t stage[kStages][kStageBytes];
    uint2 token[2][NT];
    uint64_t full[kStages];    // first CTA: the bytes of both CTAs have landed
    uint64_t empty[kStages];   // the MMAs have read the stage (both CTAs)
    uint64_t tfull[2];         // tile complete (both CTAs)
    uint64_t tempty[2];        // first CTA: both epilogues have read the accumulators
    uint32_t tmem_base;
    int abort;
};

// Tile number -> (weight tile, token tile).  Bands of kBand weight tiles,
// walked token tile by token tile: the pairs that run at one time then cover
// a compact block of tiles and share both operands in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_of(int t, int n_tiles, int m_tiles, int& tn, int& tm)
{
    const int band = t / (kBand * m_tiles);
    const int width = min(kBand, n_tiles - band * kBand);
    const int i = t - band * kBand * m_tiles;
    tm = i / width;
    tn = band * kBand + i % width;
}

template <int NT, typename T>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    w8a8_pair_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX, const W8A8Args a,
                     int n_tiles, int m_tiles, int* status)
{
    using Smem = PairSmem<NT>;
    constexpr int kStages = Smem::kStages;
    extern __shared__ uint8_t smem_raw[];
    Smem& S = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster::cta_rank();
    const int pair = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const int K = static_cast<int>(a.K);
    const int nk = (K + kBK - 1) / kBK;
    const int tiles = n_tiles * m_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.tfull[b], 1);
            mbar_init(&S.tempty[b], 2 * kEpiWarps);
        }
        S.abort = 0;
        fence_mbar_init();
        prefetch_tmap(&mapW);
        prefetch_tmap(&mapX);
    }
    if (warp == 1) {
        cluster::pair_tmem_alloc(&S.tmem_base, 2 * NT);
        cluster::pair_tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    cluster::sync();   // both CTAs' barriers and tensor memory exist before any use
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    const uint32_t tbase = S.tmem_base;
    volatile int* abort = &S.abort;

    if (warp == 0) {
        if (elect_one()) {
            uint32_t it = 0, phase = 1;
            int s = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += n_pairs) {
                int tn, tm;
                tile_of(t, n_tiles, m_tiles, tn, tm);
                const int n0 = tn * 2 * kRows + static_cast<int>(rank) * kRows;
                const int m0 = tm * NT + static_cast<int>(rank) * (NT / 2);
                for (int k = 0; k < nk; ++k, ++it) {
                    if (!mbar_wait_bounded(&S.empty[s], phase, abort, status)) { ok = false; break; }
                    if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 2 * Smem::kStageBytes);
                    const uint32_t bar = cluster::map_address(&S.full[s], 0);
                    cluster::pair_tma_load_2d(S.stage[s], &mapW, bar, k * kBK, n0);
                    cluster::pair_tma_load_2d(S.stage[s] + kWBytes, &mapX, bar, k * kBK, m0);
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
            }
            // copies in flight land before the shared memory goes away: every
            // one that was issued was waited for by the MMAs, unless a wait
            // ran out; then the stages' own barriers are waited for here
            int none = 0;
            if (*abort && rank == 0)
                for (uint32_t i = it > kStages ? it - kStages : 0; i < it; ++i)
                    mbar_wait_bounded(&S.full[i % kStages], (i / kStages) & 1, &none, nullptr, kWaitLimitCycles / 16);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            const uint64_t wd0 = sdesc_sw128(smem_u32(S.stage[0]), 16, 1024);
            const uint64_t xd0 = sdesc_sw128(smem_u32(S.stage[0] + kWBytes), 16, 1024);
            uint32_t i = 0, phase = 0;
            int s = 0;
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += n_pairs, ++i) {
                const int b = i & 1;
                if (!mbar_wait_bounded(&S.tempty[b], ((i >> 1) & 1) ^ 1, abort, status)) break;
                tc_fence_after();
                for (int k = 0; k < nk; ++k) {
                    if (!mbar_wait_bounded(&S.full[s], phase, abort, status)) { ok = false; break; }
                    tc_fence_after();
                    stage_mmas<2>(tbase + b * NT, wd0 + s * (Smem::kStageBytes >> 4), xd0 + s * (Smem::kStageBytes >> 4),
                                  idesc_i8(2 * kRows, NT), K - k * kBK, k == 0);
                    cluster::pair_commit(&S.empty[s]);
                    if (++s == kStages) { s = 0; phase ^= 1; }
                }
                if (ok) cluster::pair_commit(&S.tfull[b]);
            }
        }
        __syncwarp();
    } else if (warp >= 4) {
        // epilogue: warp w reads TMEM lanes 32 (w % 4) .. +31, token quarter h
        constexpr int kPart = 4 * NT / kEpiWarps;
        constexpr int kCols = kPart < 32 ? kPart : 32;
        const int q = warp & 3;
        const int h = (warp - 4) >> 2;
        const int et = threadIdx.x - 128;
        uint32_t i = 0;
        bool ok = true;
        for (int t = pair; t < tiles; t += n_pairs, ++i) {
            const int b = i & 1;
            int tn, tm;
            tile_of(t, n_tiles, m_tiles, tn, tm);
            const int64_t n = static_cast<int64_t>(tn) * 2 * kRows + rank * kRows + q * 32 + lane;
            const int64_t m0 = static_cast<int64_t>(tm) * NT;
            // the buffer's readers, two tiles ago, are past the last barrier
            if (et < NT) S.token[b][et] = token_scale(a, m0 + et);
            const RowScale r = row_scale(a, n);
            asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory");
            // after a wait that ran out every warp still takes part in the barriers of the tiles left
            ok = ok && mbar_wait_warp(&S.tfull[b], (i >> 1) & 1, abort, status, kWaitLimitCycles, kNap);
            if (!ok) continue;
            tc_fence_after();
            const uint32_t taddr = tbase + (static_cast<uint32_t>(q * 32) << 16) + b * NT + h * kPart;
            T* y = static_cast<T*>(a.Y) + (m0 + h * kPart) * a.ldy + n;
#pragma unroll 1
            for (int c = 0; c < kPart; c += kCols) {
                int v[kCols];
                tmem_ld_cols(taddr + c, v);
                tmem_ld_wait();
                const int64_t left = a.M - (m0 + h * kPart + c);
                if (n < a.N) {
#pragma unroll
                    for (int j = 0; j < kCols; ++j)
                        if (j < left) {
                            store_rounded(y, output(v[j], r, S.token[b][h * kPart + c + j]));
                            y += a.ldy;
                        }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster::arrive_on(cluster::map_address(&S.tempty[b], 0));
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster::sync();   // no MMA, commit or remote arrive of the pair is still in flight
    if (warp == 1) {
        tc_fence_after();
        cluster::pair_tmem_dealloc(tbase, 2 * NT);
    }
}

// ------------------------------------------------------------ split kernel
constexpr int kSplitThreads = 192;   // loads, MMAs, four epilogue warps
constexpr int kMaxStages = 12;
constexpr int kMaxSplits = 8;

struct SplitShared {
    uint64_t full[kMaxStages], empty[kMaxStages], done;
    uint2 token[128];
    uint32_t tmem_base;
    int abort;
};

template <int NT, typename T>
__global__ void __launch_bounds__(kSplitThreads)
    w8a8_split_kernel(const __grid_constant__ CUtensorMap mapW, const __grid_constant__ CUtensorMap mapX, const W8A8Args a,
                      int splits, int stages, int* status)
{
    constexpr int kStageBytes = kWBytes + NT * kBK;
    constexpr uint32_t kCols = NT < 32 ? 32 : NT;
    __shared__ SplitShared S;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster::cta_rank());
    const int n0 = static_cast<int>(blockIdx.x) / splits * kRows;   // a cluster is one tile
    const int m0 = blockIdx.y * NT;
    const int K = static_cast<int>(a.K);
    const int blocks = (K + kBK - 1) / kBK;
    const int k_begin = blocks * rank / splits, k_end = blocks * (rank + 1) / splits;
    const int nk = k_end - k_begin;

    auto load = [&](int k, int s) {
        uint8_t* st = base + s * kStageBytes;
        mbar_arrive_expect_tx(&S.full[s], kStageBytes);
        tma_load_2d(st, &mapW, &S.full[s], (k_begin + k) * kBK, n0);
        tma_load_2d(st + kWBytes, &mapX, &S.full[s], (k_begin + k) * kBK, m0);
    };
    const int first = min(stages, nk);
    if (warp == 0 && elect_one()) {
        for (int s = 0; s < stages; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        mbar_init(&S.done, 1);
        S.abort = 0;
        fence_mbar_init();
        for (int k = 0; k < first; ++k) prefetch_box(&mapW, (k_begin + k) * kBK, n0);
        pdl_wait();
        // the first loads are on their way before the block has met
        for (int k = 0; k < first; ++k) load(k, k);
    }
    if (warp == 1) {
        tmem_alloc(&S.tmem_base, kCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();
    pdl_wait();
    const uint32_t tbase = S.tmem_base;
    volatile int* abort = &S.abort;

    // This thread's outputs of the shared epilogue: four neighbouring weight
    // rows, every sixth token of this CTA's part.  What they need is loaded
    // before it is wanted.
    const int64_t n = n0 + 4 * lane;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(NT), a.M - m0));
    const int t_end = tokens * (rank + 1) / splits;
    RowScale rows[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) rows[j] = row_scale(a, n + j);

    if (warp == 0) {
        if (elect_one()) {
            int k = first, s = 0;
            uint32_t phase = 0;
            for (; k < nk; ++k) {
                if (!mbar_wait_bounded(&S.empty[s], phase, abort, status)) break;
                load(k, s);
                if (++s == stages) { s = 0; phase ^= 1; }
            }
            // after a wait that ran out: the copies issued land before the shared memory goes away
            int none = 0;
            if (*abort)
                for (int i = max(0, k - stages); i < k; ++i)
                    mbar_wait_bounded(&S.full[i % stages], (i / stages) & 1, &none, nullptr, kWaitLimitCycles / 16);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint64_t wd0 = sdesc_sw128(smem_u32(base), 16, 1024);
            const uint64_t xd0 = sdesc_sw128(smem_u32(base + kWBytes), 16, 1024);
            bool ok = true;
            int s = 0;
            uint32_t phase = 0;
            for (int k = 0; k < nk; ++k) {
                if (!mbar_wait_bounded(&S.full[s], phase, abort, status)) { ok = false; break; }
                tc_fence_after();
                stage_mmas<1>(tbase, wd0 + s * (kStageBytes >> 4), xd0 + s * (kStageBytes >> 4), idesc_i8(kRows, NT),
                              K - (k_begin + k) * kBK, k == 0);
                umma_commit(&S.empty[s]);
                if (++s == stages) { s = 0; phase ^= 1; }
            }
            if (ok) umma_commit(&S.done);
        }
        __syncwarp();
    } else {
        // the partial sums to shared memory (the stages' place: they have
        // been read), token by token
        const int q = warp & 3;
        int* part = reinterpret_cast<int*>(base);
        const int row = q * 32 + lane;
        if (row < NT) S.token[row] = token_scale(a, m0 + row);
        if (mbar_wait_warp(&S.done, 0, abort, status)) {
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < NT; c += 16) {
                int v[16];
                tmem_ld_cols(tbase + (static_cast<uint32_t>(q * 32) << 16) + c, v);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) part[(c + j) * kRows + row] = v[j];
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster::arrive();
    // freed before the cluster meets: a CTA that waits for others holds no
    // tensor memory that they, or another kernel on their SMs, may wait for
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tbase, kCols);
    }
    cluster::wait();
    for (int t0 = tokens * rank / splits + warp; t0 < t_end; t0 += 2 * (kSplitThreads / 32)) {
        // two tokens at a time: the loads of both are on their way together
        int4 sum[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + i * (kSplitThreads / 32);
            int4 v[kMaxSplits];
#pragma unroll
            for (int p = 0; p < kMaxSplits; ++p)
                if (p < splits && t < t_end) v[p] = cluster::load_int4(cluster::map_address(base + 4 * (t * kRows + 4 * lane), p));
            sum[i] = v[0];
#pragma unroll
            for (int p = 1; p < kMaxSplits; ++p)
                if (p < splits && t < t_end) {
                    sum[i].x += v[p].x;
                    sum[i].y += v[p].y;
                    sum[i].z += v[p].z;
                    sum[i].w += v[p].w;
                }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = t0 + i * (kSplitThreads / 32);
            if (t >= t_end) continue;
            const uint2 token = S.token[t];
            store4(static_cast<T*>(a.Y) + (m0 + t) * a.ldy + n, a.N - n, output(sum[i].x, rows[0], token),
                   output(sum[i].y, rows[1], token), output(sum[i].z, rows[2], token), output(sum[i].w, rows[3], token));
        }
    }
    cluster::sync();   // no CTA leaves while another reads its sums
}

// -------------------------------------------------------------- few tokens
// Lane (g, t) of a warp holds rows g and g + 8 of the weights and row g of the
// tokens at 16 codes 16 t .. of each 64: two 8-code operands of two MMAs, the
// same (permuted) order of K on both sides.  A row's 128 codes a step are read
// in whole lines, U steps in flight a warp.
constexpr int kFewRows = 16;
// What a block asks into L2 of each of its weight rows before it waits for the
// kernel before: enough to bridge that kernel's end, no more, since requests for
// whole rows stand in the way of the reads themselves.  In a row, of nothing,
// 2048 and 8192 bytes: 1 x 4096 x 11008 10.0, 9.1, 8.3 us; 1 x 14336 x 4096 10.5,
// 8.9, 9.9; 1 x 28672 x 8192 37.5, 36.6, 45.3.
constexpr int64_t kAhead = 2048;

// Not by the read-only path: the kernel may have started before its inputs
// were there.
__device__ __forceinline__ uint4 load_tokens(const void* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 load_once(const void* p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// The first `valid` of 16 codes, the others zero.
__device__ __forceinline__ uint4 first_codes(uint4 v, int valid)
{
    if (valid >= 16) return v;
    auto word = [valid](uint32_t w, int at) {
        const int n = valid - at;
        return n >= 4 ? w : n <= 0 ? 0u : w & (0xffffffffu >> (8 * (4 - n)));
    };
    return make_uint4(word(v.x, 0), word(v.y, 4), word(v.z, 8), word(v.w, 12));
}

// Sums of 16 weight rows x 8 tokens over 32 codes, signed.
__device__ __forceinline__ void mma_i8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int MT, int U, int W, typename T>
__global__ void __launch_bounds__(W * 32) w8a8_few_kernel(const W8A8Args a)
{
    __shared__ int part[W][8 * MT][kFewRows];
    pdl_trigger();
    if (threadIdx.x < kFewRows) {
        const int64_t r = static_cast<int64_t>(blockIdx.x) * kFewRows + threadIdx.x;
        if (r < a.N) {
            const uint32_t bytes = static_cast<uint32_t>(min((a.K + 15) / 16 * 16, kAhead));
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.Wq + r * a.ldw), "r"(bytes) : "memory");
        }
    }
    pdl_wait();
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kFewRows;
    const int K = static_cast<int>(a.K);
    const int steps = (K + kBK - 1) / kBK;
    // rows past the end repeat the last one; what they give is not stored
    const int8_t* w0 = a.Wq + min(n0 + g, a.N - 1) * a.ldw;
    const int8_t* w1 = a.Wq + min(n0 + g + 8, a.N - 1) * a.ldw;
    const int8_t* x[MT];
#pragma unroll
    for (int j = 0; j < MT; ++j) x[j] = a.Xq + min(static_cast<int64_t>(8 * j + g), a.M - 1) * a.ldx;
    int acc[MT][4] = {};
    for (int s = warp; s < steps; s += W * U) {
        uint4 w[U][2][2], xb[U][2][MT];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (s + W * u) * kBK + 64 * h + 16 * t;
                const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
                w[u][h][0] = k < K ? load_once(w0 + k) : zero;
                w[u][h][1] = k < K ? load_once(w1 + k) : zero;
#pragma unroll
                for (int j = 0; j < MT; ++j)
                    xb[u][h][j] = k < K ? first_codes(load_tokens(x[j] + k), K - k) : zero;
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    mma_i8(acc[j], w[u][h][0].x, w[u][h][1].x, w[u][h][0].y, w[u][h][1].y, xb[u][h][j].x, xb[u][h][j].y);
                    mma_i8(acc[j], w[u][h][0].z, w[u][h][1].z, w[u][h][0].w, w[u][h][1].w, xb[u][h][j].z, xb[u][h][j].w);
                }
    }
#pragma unroll
    for (int j = 0; j < MT; ++j) {
        part[warp][8 * j + 2 * t][g] = acc[j][0];
        part[warp][8 * j + 2 * t + 1][g] = acc[j][1];
        part[warp][8 * j + 2 * t][g + 8] = acc[j][2];
        part[warp][8 * j + 2 * t + 1][g + 8] = acc[j][3];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 8 * MT * kFewRows; e += W * 32) {
        const int64_t m = e / kFewRows, n = n0 + e % kFewRows;
        if (m >= a.M || n >= a.N) continue;
        int sum = 0;
#pragma unroll
        for (int p = 0; p < W; ++p) sum += part[p][m][e % kFewRows];
        store_rounded(static_cast<T*>(a.Y) + m * a.ldy + n, output(sum, row_scale(a, n), token_scale(a, m)));
    }
}

// ------------------------------------------------------------------- host
using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(p);
    });
    return fn;
}

// 8-bit rows in boxes of kBK codes x box_rows rows, 128-byte swizzle.
int make_map(CUtensorMap* map, const int8_t* p, int64_t cols, int64_t rows, int64_t pitch, int box_rows)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return cuda_fail(cudaErrorNotSupported);
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(pitch)};
    cuuint32_t box[2] = {kBK, static_cast<cuuint32_t>(box_rows)};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(p), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return cuda_fail_msg("w8a8: tensor map encoding", cudaErrorInvalidValue);
    return GPTQ_OK;
}

// Sets a kernel's shared-memory limit, once per device: to the most that any of
// its launches asks for, so that calls which set it at the same time set the
// same value and none lowers what another goes by.
template <typename K>
int allow_smem(K kernel, std::atomic<bool> (&done)[64], int most)
{
    int dev = 0;
    GPTQ_CUDA_CHECK(cudaGetDevice(&dev));
    if (dev < 64 && done[dev].load(std::memory_order_acquire)) return GPTQ_OK;
    GPTQ_CUDA_CHECK(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most));
    if (dev < 64) done[dev].store(true, std::memory_order_release);
    return GPTQ_OK;
}

template <int NT, typename T>
int launch_pair(const W8A8Args& a, cudaStream_t stream)
{
    constexpr int smem = sizeof(PairSmem<NT>) + 1024;
    static_assert(smem <= 227 * 1024, "one CTA per SM");
    static std::atomic<bool> smem_set[64] = {};
    int rc = allow_smem(w8a8_pair_kernel<NT, T>, smem_set, smem);
    if (rc) return rc;
    CUtensorMap mapW, mapX;
    rc = make_map(&mapW, a.Wq, a.K, a.N, a.ldw, kRows);
    if (rc) return rc;
    rc = make_map(&mapX, a.Xq, a.K, a.M, a.ldx, NT / 2);
    if (rc) return rc;
    const int64_t n_tiles = (a.N + 2 * kRows - 1) / (2 * kRows), m_tiles = (a.M + NT - 1) / NT;
    const int pairs = static_cast<int>(std::min<int64_t>(n_tiles * m_tiles, sm_count() / 2));
    const cudaError_t e = launch_k(w8a8_pair_kernel<NT, T>, dim3(2 * pairs), dim3(kPairThreads), smem, stream, true, mapW, mapX, a,
                                   static_cast<int>(n_tiles), static_cast<int>(m_tiles), device_status_ptr());
    if (e != cudaSuccess) return cuda_fail(e);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int NT, typename T>
int launch_split(const W8A8Args& a, int splits, cudaStream_t stream)
{
    constexpr int stage_bytes = kWBytes + NT * kBK;
    const int n_tiles = static_cast<int>((a.N + kRows - 1) / kRows), m_tiles = static_cast<int>((a.M + NT - 1) / NT);
    const int blocks = static_cast<int>((a.K + kBK - 1) / kBK);
    // all of an SM's shared memory where each has one CTA at most, else half
    // (clusters of more than 4 such CTAs do not all find their SMs in one GPC)
    const bool alone = static_cast<int64_t>(n_tiles) * m_tiles * splits <= sm_count() && splits <= 4;
    constexpr int most_alone = std::min(kMaxStages, 200 * 1024 / stage_bytes), most_shared = std::min(kMaxStages, 104 * 1024 / stage_bytes);
    const int stages = std::min(alone ? most_alone : most_shared, (blocks + splits - 1) / splits);
    auto bytes = [](int n) constexpr { return std::max(n * stage_bytes, NT * kRows * 4) + 1024; };
    const int smem = bytes(stages);
    static std::atomic<bool> smem_set[64] = {};
    int rc = allow_smem(w8a8_split_kernel<NT, T>, smem_set, bytes(most_alone));
    if (rc) return rc;
    CUtensorMap mapW, mapX;
    rc = make_map(&mapW, a.Wq, a.K, a.N, a.ldw, kRows);
    if (rc) return rc;
    rc = make_map(&mapX, a.Xq, a.K, a.M, a.ldx, NT);
    if (rc) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(splits * n_tiles, m_tiles);
    cfg.blockDim = dim3(kSplitThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = splits;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaError_t e = cudaLaunchKernelEx(&cfg, w8a8_split_kernel<NT, T>, mapW, mapX, a, splits, stages, device_status_ptr());
    if (e != cudaSuccess) return cuda_fail_msg("w8a8: cluster launch", e);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

template <int MT, int U, int W, typename T>
int launch_few(const W8A8Args& a, cudaStream_t stream)
{
    const unsigned blocks = static_cast<unsigned>((a.N + kFewRows - 1) / kFewRows);
    const cudaError_t e = launch_k(w8a8_few_kernel<MT, U, W, T>, dim3(blocks), dim3(W * 32), 0, stream, 1, a);
    if (e != cudaSuccess) return cuda_fail(e);
    GPTQ_LAUNCH_CHECK();
    return GPTQ_OK;
}

// Which kernel, and how it is cut.  The times are a model of what was measured
// on B200 (us; M x N x K with bf16 out):
//   few tokens: a block reads 16 weight rows and, again, every token's row.
//     8 x 4096 x 4096 4.2 against 5.9 by the split kernel, 16 x 4096 x 4096 5.4
//     against 6.3, 16 x 4096 x 11008 12.7 against 12.2, 24 x 1000 x 1003 3.8
//     against 5.1, 24 x 1024 x 4096 5.2 against 5.5, 24 x 4096 x 4096 9.2
//     against 6.3;
//   tiles: a start and an end (longer for more tokens a tile and more CTAs than
//     SMs), then whichever is longest of the issue of a CTA's stages, the operands' way from L2 (14
//     bytes a ps over all SMs) and the weights' from memory (6.2, less with few CTAs).  128 x 4096 x 4096:
//     split 128 9.3, split 64 9.7 (which the model takes), pair 64 12.9; 256 x 4096 x 11008: split 128
//     19.9, pair 128 24.0; 512 x 4096 x 4096: pair 128 14.2, pair 256 17.2,
//     split 128 16.4; 1024 x 4096 x 4096: pair 256 18.1, pair 128 20.6;
//     256 x 11008 x 4096: pair 256 19.1, pair 128 22.8, split 128 23.5;
//     2048 x 1024 x 4096: pair 128 14.4, split 128 16.0.
struct Choice {
    int tokens;   // a tile's
    int splits;   // CTAs that share a tile's K; 0: the pair kernel
};

Choice choose_tiles(int64_t M, int64_t N, int64_t K)
{
    const double sms = sm_count(), blocks = static_cast<double>((K + kBK - 1) / kBK);
    Choice best{256, 0};
    double best_time = 1e30;
    auto consider = [&](Choice c, double ctas, double ends, double issue, double bytes) {
        const double memory = static_cast<double>(N) * K / std::min(6.2e6, 0.056e6 * ctas);
        const double t = ends + std::max({issue, bytes / 14e6, memory});
        if (t < best_time) {
            best_time = t;
            best = c;
        }
    };
    for (int nt : {32, 64, 128}) {
        if (nt > 32 && nt / 2 >= M) break;   // half the tile would be empty
        if ((M + nt - 1) / nt > 65535) continue;   // the grid's second dimension
        const int64_t tiles = (N + kRows - 1) / kRows * ((M + nt - 1) / nt);
        // one CTA an SM while each keeps 2 stages of K, two while it keeps 8;
        // large clusters only where they are few (500 x 512 x 4096: 6.9 us by
        // 4, 9.4 by 8: they do not spread over all SMs)
        const int64_t one = std::min<int64_t>(sm_count() / tiles, static_cast<int64_t>(blocks) / 2);
        const int64_t two = std::min<int64_t>(2 * sm_count() / tiles, static_cast<int64_t>(blocks) / 8);
        const int64_t most = tiles <= 8 ? kMaxSplits : tiles <= 24 ? 6 : 4;
        const int splits = static_cast<int>(std::min(most, std::max<int64_t>({1, one, two})));
        const double own = std::ceil(blocks / splits);
        const double rounds = std::ceil(static_cast<double>(tiles) * splits / (2 * sms));
        const double ends = 3.5 + 0.008 * nt + 0.03 * nt / splits + 0.012 * std::max(0.0, tiles * splits - sms);
        const double ctas = static_cast<double>(tiles) * splits;
        consider({nt, splits}, ctas, ends, rounds * own * 0.2, ctas * own * (kRows + nt) * kBK / std::min(1.0, ctas / sms / 1.5));
    }
    const struct { int nt; double ends, stage; } pairs[] = {{64, 4.9, 0.24}, {128, 5.6, 0.235}, {256, 7.5, 0.285}};
    for (const auto& p : pairs) {
        if (p.nt > 64 && p.nt / 2 >= M) break;
        const int64_t tiles = (N + 2 * kRows - 1) / (2 * kRows) * ((M + p.nt - 1) / p.nt);
        consider({p.nt, 0}, 2.0 * tiles, p.ends, std::ceil(2.0 * tiles / sms) * blocks * p.stage,
                 static_cast<double>(tiles) * blocks * (2 * kRows + p.nt) * kBK);
    }
    return best;
}

template <typename T>
int run_typed(const W8A8Args& a, cudaStream_t stream)
{
    const int64_t weights = a.N * a.K;
    if (a.M <= 8) {
        // many blocks: four warps each and more blocks an SM, whose loads and
        // reductions overlap (1 x 11008 x 4096 9.1 us against 10.8 as plain launches); else eight
        // warps a block, each with more on its way (1 x 4096 x 4096 3.6 against 5.2)
        if (a.N >= int64_t(3) * kFewRows * sm_count()) return launch_few<1, 2, 4, T>(a, stream);
        return launch_few<1, 4, 8, T>(a, stream);
    }
    if (a.M <= 16 && weights <= (int64_t(1) << 25)) return launch_few<2, 2, 8, T>(a, stream);
    if (a.M <= 32 && weights <= (int64_t(1) << 22)) return launch_few<4, 2, 8, T>(a, stream);
    const Choice c = choose_tiles(a.M, a.N, a.K);
    if (c.splits) {
        if (c.tokens == 32) return launch_split<32, T>(a, c.splits, stream);
        if (c.tokens == 64) return launch_split<64, T>(a, c.splits, stream);
        return launch_split<128, T>(a, c.splits, stream);
    }
    if (c.tokens == 64) return launch_pair<64, T>(a, stream);
    if (c.tokens == 128) return launch_pair<128, T>(a, stream);
    return launch_pair<256, T>(a, stream);
}

}  // namespace

int run_w8a8(const W8A8Args& a, int y_type, cudaStream_t stream)
{
    if (y_type == GPTQ_F32) return run_typed<float>(a, stream);
    if (y_type == GPTQ_F16) return run_typed<__half>(a, stream);
    return run_typed<__nv_bfloat16>(a, stream);
}

}  // namespace gptq
