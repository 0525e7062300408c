// Dense product with its epilogue: y = act(x w^T + b) + r, or with SwiGLU
// y = silu(x wg^T + bg) (x wu^T + bu) + r, w holding the N gate rows and
// then the N up rows. bf16 or fp16 operands, fp32 accumulation on the matrix
// cores, everything after the product in fp32, one rounding to y's type.
//
// Up to kSkinnyTokens tokens the weights' bytes bound it: they are streamed
// once, straight into MFMA operands (linear_skinny_kernel) or through each
// wave's own LDS ring (linear_stream_kernel). Beyond, tiles of both operands
// meet in LDS: linear_phased_kernel (large products), linear_ring_kernel
// (smaller ones), linear_any_kernel (rows of any alignment).
#include <hip/hip_runtime.h>

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pw_internal.h"

namespace pw {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

// 16 x 16 x 32 product: lane (r = lane % 16, g = lane / 16) holds the 8
// K-slots 8 g .. 8 g + 7 of row r of a and of column r of b; it gets rows
// 4 g .. 4 g + 3 of column r of the product.
template <class T>
__device__ __forceinline__ f32x4 mma(const u32x4& a, const u32x4& b, const f32x4& c) {
    if constexpr (std::is_same<T, _Float16>::value)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// ---- epilogue ----

// The native exponential and reciprocal: z log2(e) is rounded once, so the
// result is off by about |z| 2^-24 of itself and a few 2^-24 more (below a step of
// fp32 at 1 in absolute terms everywhere; far below what bf16 or fp16 keep).
__device__ __forceinline__ float sigmoid_of(float z) {
    constexpr float kLog2e = 1.4426950408889634f;
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

__device__ __forceinline__ float silu_of(float z) { return z * sigmoid_of(z); }

__device__ __forceinline__ float load_out(const void* p, int64_t i, int dtype) {
    if (dtype == PW_F32) return reinterpret_cast<const float*>(p)[i];
    if (dtype == PW_BF16) return (float)reinterpret_cast<const __bf16*>(p)[i];
    return (float)reinterpret_cast<const _Float16*>(p)[i];
}
__device__ __forceinline__ void store_out(void* p, int64_t i, int dtype, float v) {
    if (dtype == PW_F32) reinterpret_cast<float*>(p)[i] = v;
    else if (dtype == PW_BF16) reinterpret_cast<__bf16*>(p)[i] = (__bf16)v;
    else reinterpret_cast<_Float16*>(p)[i] = (_Float16)v;
}

// Four consecutive values: residual bits, their addition, the store.
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
template <int DT>
struct QuadOf {
    typedef uint2 bits;
    typedef typename std::conditional<DT == PW_BF16, bf16x4, f16x4>::type vec;
    typedef typename std::conditional<DT == PW_BF16, __bf16, _Float16>::type elem;
};
template <>
struct QuadOf<PW_F32> {
    typedef u32x4 bits;
    typedef f32x4 vec;
    typedef float elem;
};
template <int DT>
__device__ __forceinline__ typename QuadOf<DT>::bits load_quad(const void* p, int64_t i) {
    return *reinterpret_cast<const typename QuadOf<DT>::bits*>(reinterpret_cast<const typename QuadOf<DT>::elem*>(p) + i);
}
template <int DT>
__device__ __forceinline__ void add_quad(float (&v)[4], const typename QuadOf<DT>::bits& r) {
    const auto f = __builtin_bit_cast(typename QuadOf<DT>::vec, r);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] += (float)f[e];
}
template <int DT>
__device__ __forceinline__ void store_quad(void* p, int64_t i, const float (&v)[4]) {
    typedef typename QuadOf<DT>::elem E;
    *reinterpret_cast<typename QuadOf<DT>::vec*>(reinterpret_cast<E*>(p) + i) =
        typename QuadOf<DT>::vec{(E)v[0], (E)v[1], (E)v[2], (E)v[3]};
}

// The activation of n quads (one branch for all of them).
template <int N>
__device__ __forceinline__ void act_all(float (&v)[N][4], int act) {
    auto each = [&](auto f) {
#pragma unroll
        for (int t = 0; t < N; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) v[t][e] = f(v[t][e]);
    };
    switch (act) {
        case PW_ACT_RELU: each([](float z) { return z > 0.0f || z != z ? z : 0.0f; }); break;
        case PW_ACT_SILU: each([](float z) { return silu_of(z); }); break;
        case PW_ACT_SIGMOID: each([](float z) { return sigmoid_of(z); }); break;
        case PW_ACT_GELU: each([](float z) { return 0.5f * z * erfcf(-0.70710678118654752f * z); }); break;
        case PW_ACT_GELU_TANH:
            // (1 + tanh u) / 2 = sigmoid(2 u)
            each([](float z) { return z * sigmoid_of(1.5957691216057308f * (z + 0.044715f * z * z * z)); });
            break;
        default: break;
    }
}

// Outputs n .. n + 3 of token m from their sums.
template <int DT, bool GLU>
__device__ __forceinline__ void put4_t(const LinearArgs& a, int64_t m, int n, f32x4 z, f32x4 up) {
    const bool vec = a.vec_out && n + 3 < a.N;
    typename QuadOf<DT>::bits res{};
    if (a.residual && vec) res = load_quad<DT>(a.residual, m * a.ldr + n);
    float v[1][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (a.bias && n + e < a.N) {
            z[e] += a.bias[n + e];
            if (GLU) up[e] += a.bias[a.N + n + e];
        }
        v[0][e] = GLU ? silu_of(z[e]) * up[e] : z[e];
    }
    if constexpr (!GLU) act_all(v, a.act);
    if (vec) {
        if (a.residual) add_quad<DT>(v[0], res);
        store_quad<DT>(a.y, m * a.ldy + n, v[0]);
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        if (n + e >= a.N) break;
        float o = v[0][e];
        if (a.residual) o += load_out(a.residual, m * a.ldr + n + e, DT);
        store_out(a.y, m * a.ldy + n + e, DT, o);
    }
}
template <bool GLU>
__device__ __forceinline__ void put4(const LinearArgs& a, int64_t m, int n, const f32x4& z, const f32x4& up) {
    if (a.out_dtype == PW_F32) put4_t<PW_F32, GLU>(a, m, n, z, up);
    else if (a.out_dtype == PW_BF16) put4_t<PW_BF16, GLU>(a, m, n, z, up);
    else put4_t<PW_F16, GLU>(a, m, n, z, up);
}

// ---- operands ----

// 8 consecutive K values from p, which need not be aligned (the loads are
// declared with the element's alignment); left: values of the row from p on,
// zeros past them
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));
__device__ __forceinline__ u32x4 load_chunk(const uint16_t* p, int left) {
    if (left >= 8) return *reinterpret_cast<const u32x4_any*>(p);
    u32x4 u = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) u[i >> 1] |= (uint32_t)p[i] << (16 * (i & 1));
    return u;
}

constexpr int BK = 64;   // K values per step: 128-byte rows in LDS
constexpr uint32_t kOutside = 0x80000000u;   // buffer offset past every record: reads 0

__device__ __forceinline__ __amdgpu_buffer_rsrc_t make_rsrc(const void* p) {
    const uint64_t a = reinterpret_cast<uint64_t>(p);
    const uint64_t u = ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(a >> 32)) << 32) |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)a);
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), (short)0, 0x7fffffff, 0x00020000);
}

// 16 bytes per lane from the buffer to LDS, lane i's to dst + 16 i (device
// pass only: the host pass does not know the builtin)
__device__ __forceinline__ void copy_to_lds(const __amdgpu_buffer_rsrc_t& rsrc, uint16_t* dst, uint32_t off, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)dst, 16, (int)off, soff, 0, 0);
#endif
}

// 4 bytes per lane, likewise (64 of them at dst).
__device__ __forceinline__ void touch_to_lds(const __amdgpu_buffer_rsrc_t& rsrc, uint16_t* dst, uint32_t off, int soff) {
#if defined(__HIP_DEVICE_COMPILE__)
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc, (__attribute__((address_space(3))) void*)dst, 4, (int)off, soff, 0, 0);
#endif
}

// Waits count copies in the order in which they were issued (s_waitcnt vmcnt):
// where they tell older from younger ones, no memory access may change sides.
__device__ __forceinline__ void keep_order() { asm volatile("" ::: "memory"); }

// byte offset of K value k0, 0 past the end (the lanes are out of bounds there)
__device__ __forceinline__ int in_bytes(int k0, int K) { return k0 < K ? 2 * k0 : 0; }

// ---- few tokens ----

// The sums of a workgroup's waves (each over its own pieces of K) through
// LDS, added in wave order, and out.
template <int RB, int MB, bool GLU>
__device__ __forceinline__ void join_waves(const LinearArgs& a, const f32x4 (&acc)[RB][MB], float* part, int n0, int m0) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    f32x4* mine = reinterpret_cast<f32x4*>(part) + (int64_t)wave * RB * MB * 64 + lane;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) mine[(i * MB + j) * 64] = acc[i][j];
    __syncthreads();
    // one (row block, token block, lane) per thread and round, the waves'
    // sums in order
    constexpr int kBlocks = kRowsOut / 16;
    for (int i = threadIdx.x; i < kBlocks * MB * 64; i += blockDim.x) {
        const int ln = i & 63, q = i >> 6, blk = q / MB, j = q - blk * MB;
        const f32x4* src = reinterpret_cast<const f32x4*>(part) + ln;
        f32x4 z = {0.f, 0.f, 0.f, 0.f}, up = z;
        for (int w = 0; w < waves; ++w) {
            if (GLU) {
                z += src[((w * RB + 2 * blk) * MB + j) * 64];
                up += src[((w * RB + 2 * blk + 1) * MB + j) * 64];
            } else {
                z += src[((w * RB + blk) * MB + j) * 64];
            }
        }
        const int m = m0 + 16 * j + (ln & 15), n = n0 + 16 * blk + 4 * (ln >> 4);
        if (m < a.M && n < a.N) put4<GLU>(a, m, n, z, up);
    }
}

// Workgroup: RB blocks of 16 weight rows (with SwiGLU the same RB / 2 blocks
// of gate and of up rows), MB blocks of 16 tokens, the K range dealt to its
// waves in pieces of 64: neighbouring waves read neighbouring 128 bytes of
// every row, straight into MFMA operands, D pieces in flight per wave. The
// waves' sums meet in LDS. (A lane's K values are 32 contiguous bytes, so that
// its two loads come from one 128-byte line: 50 us for 16 x 14336 x 4096
// SwiGLU, 62 with 64-byte halves of the lines and non-temporal loads.)
template <class T, int RB, int MB, int D, bool GLU>
__global__ __launch_bounds__(RB * MB > 4 ? 256 : 1024) void linear_skinny_kernel(LinearArgs a) {
    extern __shared__ __attribute__((aligned(16))) float part[];   // [waves][RB][MB][64 lanes][4]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const int n0 = blockIdx.x * kRowsOut, m0 = blockIdx.y * 16 * MB;
    // rows past the end repeat the last one; their sums are dropped
    const uint16_t* wp[RB];
    const uint16_t* xp[MB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int blk = GLU ? b >> 1 : b;
        const int64_t row = min(n0 + 16 * blk + r, a.N - 1) + (GLU && (b & 1) ? (int64_t)a.N : 0);
        wp[b] = reinterpret_cast<const uint16_t*>(a.w) + row * a.ldw + 16 * g;
    }
#pragma unroll
    for (int b = 0; b < MB; ++b)
        xp[b] = reinterpret_cast<const uint16_t*>(a.x) + (int64_t)min(m0 + 16 * b + r, a.M - 1) * a.ldx + 16 * g;
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Piece {
        u32x4 w[RB][2], x[MB][2];
    };
    auto load = [&](Piece& p, int i) {   // the wave's i-th piece, a whole one
        const int k = 64 * (wave + waves * i);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < RB; ++b)
                p.w[b][h] = *reinterpret_cast<const u32x4_any*>(wp[b] + k + 8 * h);
#pragma unroll
            for (int b = 0; b < MB; ++b) p.x[b][h] = *reinterpret_cast<const u32x4_any*>(xp[b] + k + 8 * h);
        }
    };
    auto multiply = [&](const Piece& p) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(p.w[i][h], p.x[j][h], acc[i][j]);
    };
    const int whole = a.K >> 6;   // whole pieces, dealt in turn
    const int n = whole > wave ? (whole - wave + waves - 1) / waves : 0;
    Piece ring[D];
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load(ring[j], j);
    int i = 0;
    for (; i + 2 * D <= n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            multiply(ring[j]);
            load(ring[j], i + D + j);
        }
    }
#pragma unroll
    for (int j = 0; j < D; ++j) {
        if (i + j < n) multiply(ring[j]);
        if (i + D + j < n) load(ring[j], i + D + j);
    }
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (i + D + j < n) multiply(ring[j]);
    if ((a.K & 63) && whole % waves == wave) {   // the last, partial piece
        Piece p;
        const int k = 64 * whole;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int left = a.K - (k + 8 * h + 16 * g);
#pragma unroll
            for (int b = 0; b < RB; ++b) p.w[b][h] = load_chunk(wp[b] + k + 8 * h, left);
#pragma unroll
            for (int b = 0; b < MB; ++b) p.x[b][h] = load_chunk(xp[b] + k + 8 * h, left);
        }
        multiply(p);
    }
    join_waves<RB, MB, GLU>(a, acc, part, n0, m0);
}

// The same product for 16-byte aligned rows, the pieces through LDS: a wave
// copies its own pieces (8 whole 128-byte row parts per instruction) into a
// ring of D slots that no other wave touches, so nothing but its own counter
// of copies is waited for, and what is in flight takes no registers.
template <class T, int RB, int MB, int D, bool GLU>
__global__ __launch_bounds__(1024) void linear_stream_kernel(LinearArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint16_t ring_lds[];   // [waves][D][RB + MB][16 rows][64]
    constexpr int kBlock = 16 * BK, kSlot = (RB + MB) * kBlock;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const int n0 = blockIdx.x * kRowsOut, m0 = blockIdx.y * 16 * MB;
    const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
    const uint16_t* wbase = reinterpret_cast<const uint16_t*>(a.w) + (int64_t)n0 * a.ldw;
    const auto rw = make_rsrc(wbase), ru = make_rsrc(wbase + (GLU ? (int64_t)a.N * a.ldw : 0));
    const auto rx = make_rsrc(reinterpret_cast<const uint16_t*>(a.x) + (int64_t)m0 * a.ldx);
    uint32_t off[RB + MB][2];
#pragma unroll
    for (int b = 0; b < RB + MB; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int row = 16 * (b >= RB ? b - RB : GLU ? b >> 1 : b) + 8 * h + crow;
            const bool in = b >= RB ? m0 + row < a.M : n0 + row < a.N;
            off[b][h] = in ? (uint32_t)(row * (b >= RB ? a.ldx : a.ldw) + 8 * chunk) * 2u : kOutside;
        }
    const int total = (a.K + BK - 1) / BK;
    const int n = total > wave ? (total - wave + waves - 1) / waves : 0;
    uint16_t* ring = ring_lds + wave * D * kSlot;
    auto copy = [&](int i, int slot) {   // piece i of this wave (past the last: zeros, no memory touched)
        const int k0 = BK * (wave + waves * i);
        const bool in = k0 + 8 * chunk < a.K;
#pragma unroll
        for (int b = 0; b < RB + MB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h)
                copy_to_lds(b >= RB ? rx : GLU && (b & 1) ? ru : rw, ring + slot * kSlot + b * kBlock + 8 * h * BK,
                            in ? off[b][h] : kOutside, in_bytes(k0, a.K));
    };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < D; ++j) {
        copy(j, j);
        keep_order();
    }
    int slot = 0;
    for (int i = 0; i < n; ++i) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (RB + MB) * (D - 1)) : "memory");
        const u32x4* base = reinterpret_cast<const u32x4*>(ring + slot * kSlot) + r * 8;
        u32x4 f[RB + MB][2];
#pragma unroll
        for (int b = 0; b < RB + MB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) f[b][h] = base[b * 128 + ((4 * h + g) ^ (r & 7))];
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read, before the slot is written again
        __builtin_amdgcn_sched_barrier(0);
        copy(i + D, slot);
        slot = slot + 1 == D ? 0 : slot + 1;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int p = 0; p < RB; ++p)
#pragma unroll
                for (int q = 0; q < MB; ++q) acc[p][q] = mma<T>(f[p][h], f[RB + q][h], acc[p][q]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();   // the rings are done with
    join_waves<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(ring_lds), n0, m0);
}

// ---- many tokens ----


// Epilogue of a wave's tile: the sums of 16 tokens at a time through the
// wave's own part of the (free) LDS, out as whole rows of its 16 RB weight
// rows. n0, m0: the wave's first output column and token.
template <int RB>
__host__ __device__ constexpr int out_stage_floats() { return 16 * (16 * RB + 4); }   // the padding spreads the tokens over the banks

template <int DT, int RB, int MB, bool GLU>
__device__ __forceinline__ void put_tile_t(const LinearArgs& a, const f32x4 (&acc)[RB][MB], float* os, int n0, int64_t m0) {
    constexpr int kStride = 16 * RB + 4;
    constexpr int kQuads = (GLU ? RB / 2 : RB) * 4;   // four outputs each, per token
    // tokens at a time, a power of two (RB = 6 leaves 16 lanes idle)
    constexpr int kStep = 64 / kQuads >= 16 ? 16 : 64 / kQuads >= 8 ? 8 : 64 / kQuads >= 4 ? 4 : 64 / kQuads >= 2 ? 2 : 1;
    constexpr int kRounds = 16 / kStep;                // for 16 tokens
    constexpr int kIter = kRounds < 4 ? kRounds : 4;   // of them in one part
    constexpr int kParts = kRounds / kIter;
    static_assert(kStep * kRounds == 16 && kIter * kParts == kRounds, "16 tokens in whole parts");
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int q = lane % kQuads, tok = lane / kQuads;
    const bool mine = tok < kStep;
    const int col = GLU ? (q >> 2) * 32 + (q & 3) * 4 : q * 4;
    const int n = n0 + q * 4;   // the lane's four columns, for every token
    const bool whole = a.vec_out && n0 + (GLU ? RB / 2 : RB) * 16 <= a.N && m0 + MB * 16 <= a.M;
    const bool ahead = whole && a.residual && mine;
    f32x4 bz = {0.f, 0.f, 0.f, 0.f}, bu = bz;
    if (a.bias) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (n + e < a.N) {
                bz[e] = a.bias[n + e];
                if (GLU) bu[e] = a.bias[a.N + n + e];
            }
        }
    }
    // a part's residual is loaded a part ahead, before the stores of the one
    // between (a wait for a load is a wait for every older store)
    typename QuadOf<DT>::bits res[kIter], next[kIter];
    auto fetch = [&](int c) {
        const int64_t m = m0 + (c / kParts) * 16 + (c % kParts) * kIter * kStep + tok;
        const int64_t at = m * a.ldr + n;
#pragma unroll
        for (int t = 0; t < kIter; ++t) next[t] = load_quad<DT>(a.residual, at + (int64_t)(t * kStep) * a.ldr);
    };
    if (ahead) fetch(0);
    // the loop runs over parts of 16 tokens, so that the code of the
    // activations is there once
#pragma unroll 1
    for (int c = 0; c < MB * kParts; ++c) {
        if (c % kParts == 0) {
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the former tokens are read
            __builtin_amdgcn_wave_barrier();
#pragma unroll
            for (int J = 0; J < MB; ++J) {
                if (J * kParts != c) continue;
#pragma unroll
                for (int i = 0; i < RB; ++i) *reinterpret_cast<f32x4*>(os + r * kStride + 16 * i + 4 * g) = acc[i][J];
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        if (ahead) {
#pragma unroll
            for (int t = 0; t < kIter; ++t) res[t] = next[t];
            if (c + 1 < MB * kParts) fetch(c + 1);
        }
        const int t0 = (c % kParts) * kIter * kStep + tok;
        float v[kIter][4];
#pragma unroll
        for (int t = 0; t < kIter; ++t) {
            const float* row = os + min(t0 + t * kStep, 15) * kStride + col;
            const f32x4 z = *reinterpret_cast<const f32x4*>(row) + bz;
            if constexpr (GLU) {
                const f32x4 up = *reinterpret_cast<const f32x4*>(row + 16) + bu;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[t][e] = silu_of(z[e]) * up[e];
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[t][e] = z[e];
            }
        }
        if constexpr (!GLU) act_all(v, a.act);
        if (!mine) continue;
        const int64_t m1 = m0 + (c / kParts) * 16 + t0;
        if (whole) {
            if (ahead) {
#pragma unroll
                for (int t = 0; t < kIter; ++t) add_quad<DT>(v[t], res[t]);
            }
            const int64_t at = m1 * a.ldy + n;
#pragma unroll
            for (int t = 0; t < kIter; ++t) store_quad<DT>(a.y, at + (int64_t)(t * kStep) * a.ldy, v[t]);
        } else {
            // ragged or unaligned: value by value, the residual's loads
            // together
            float add[kIter][4];
#pragma unroll
            for (int t = 0; t < kIter; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    add[t][e] = a.residual && m1 + t * kStep < a.M && n + e < a.N
                                    ? load_out(a.residual, (m1 + t * kStep) * a.ldr + n + e, DT) : 0.0f;
#pragma unroll
            for (int t = 0; t < kIter; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (m1 + t * kStep < a.M && n + e < a.N)
                        store_out(a.y, (m1 + t * kStep) * a.ldy + n + e, DT, a.residual ? v[t][e] + add[t][e] : v[t][e]);
        }
    }
}

template <int RB, int MB, bool GLU>
__device__ __forceinline__ void put_tile(const LinearArgs& a, const f32x4 (&acc)[RB][MB], float* os, int n0, int64_t m0) {
    if (a.out_dtype == PW_F32) put_tile_t<PW_F32, RB, MB, GLU>(a, acc, os, n0, m0);
    else if (a.out_dtype == PW_BF16) put_tile_t<PW_BF16, RB, MB, GLU>(a, acc, os, n0, m0);
    else put_tile_t<PW_F16, RB, MB, GLU>(a, acc, os, n0, m0);
}

// Tile of this workgroup, or false past the last. Each XCD (every eighth
// workgroup) walks one contiguous eighth of the tiles, in bands of kBand
// token tiles with the band's token tiles fastest: the 32 workgroups that
// run together on an XCD share 8 token and 4 weight tiles through its L2.
constexpr int kBand = 8;
__device__ __forceinline__ bool tile_of(int tn, int tm, int& nt, int& mt) {
    const int64_t used = (int64_t)tn * tm, share = (used + 7) >> 3;
    const int64_t at = blockIdx.x >> 3, li = (int64_t)(blockIdx.x & 7) * share + at;
    if (at >= share || li >= used) return false;
    const int band = (int)(li / ((int64_t)kBand * tn));
    const int in = (int)(li - (int64_t)band * kBand * tn);
    const int wide = min(kBand, tm - band * kBand);
    nt = in / wide;
    mt = band * kBand + in - nt * wide;
    return true;
}

// Large products: 32 RB weight rows x 64 MB tokens (256 x 256 at most), 8
// waves (2 x 4) of 16 RB x 16 MB each, K in stages of 64 (128-byte LDS rows)
// through two LDS slots.
//
// The two waves of a SIMD take turns. Half a stage is a phase of operand
// reads (RB + MB of 16 bytes a lane) and a phase of RB MB matrix
// instructions; waves 4 .. 7 run one phase behind waves 0 .. 3, so that one
// wave of each SIMD multiplies while the other reads. Phases end at
// barriers. Stage s is read in phases 4 s .. 4 s + 3; the other slot, read up
// to phase 4 s - 1, takes the copies of stage s + 1 meanwhile: each wave
// starts its own among its first matrix instructions of the stage (issued
// with the reads they delayed these: 177k cycles for 64 stages of a 256 x 256
// tile, 163k so; the matrix instructions alone take 131k) and waits for them
// by the end of phase 4 s + 3 (the first four waves multiply there, the
// others read). Copies past the last stage read zeros (out of the buffer's
// bounds).
//
// A layer's weights come from memory each time it runs, 1 to 2 us away where
// a stage takes 1: each of the 8 token tiles that share a weight tile on an
// XCD asks for an eighth of its rows kAhead stages ahead (four bytes of each
// 128-byte row part, into LDS that nobody reads), which brings them into the
// L2 (8192 x 4096 x 4096 from memory: 255 -> 238 us; the tokens too: 231, but
// 3% slower where they were written just before).
//
// A row's 16-byte chunk c lies at position c ^ (row % 8): the rows of an
// operand read fall on different banks (no conflicts counted; 64-byte rows
// had one cycle in three).
constexpr int kAhead = 4;
template <class T, int RB, int MB, bool GLU>
__global__ __launch_bounds__(512) void linear_phased_kernel(LinearArgs a) {
    constexpr int BN = 32 * RB, BM = 64 * MB, kRows = BN + BM;
    constexpr int kOutN = GLU ? BN / 2 : BN;
    constexpr int QW = BN / 64, QX = BM / 64;   // copies per thread and stage
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    int nt, mt;
    if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + BM - 1) / BM, nt, mt)) return;
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * BM;
    // a wave's copy covers 8 rows: 64 j + 8 wave + lane / 8 of the weights,
    // then of the tokens
    const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
    const uint16_t* wbase = reinterpret_cast<const uint16_t*>(a.w) + (int64_t)n0 * a.ldw;
    const uint16_t* xbase = reinterpret_cast<const uint16_t*>(a.x) + m0 * a.ldx;
    // SwiGLU: the tile's blocks of 16 rows are gate and up rows in turn (a
    // wave copies one kind)
    const bool up = GLU && (wave & 2);
    const auto rw = make_rsrc(wbase + (up ? (int64_t)a.N * a.ldw : 0)), rx = make_rsrc(xbase);
    uint32_t off[QW + QX];
#pragma unroll
    for (int j = 0; j < QW; ++j) {
        const int lr = 64 * j + 8 * wave + crow;
        const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
        off[j] = n0 + wr < a.N ? (uint32_t)(wr * a.ldw + 8 * chunk) * 2u : kOutside;
    }
#pragma unroll
    for (int j = 0; j < QX; ++j) {
        const int lr = 64 * j + 8 * wave + crow;
        off[QW + j] = m0 + lr < a.M ? (uint32_t)(lr * a.ldx + 8 * chunk) * 2u : kOutside;
    }
    auto copy = [&](int s) {
        const int k0 = s * BK;
        const bool in = k0 + 8 * chunk < a.K;
        uint16_t* dst = tile_lds + (s & 1) * kRows * BK + 8 * wave * BK;
#pragma unroll
        for (int j = 0; j < QW + QX; ++j)
            copy_to_lds(j < QW ? rw : rx, dst + 64 * j * BK, in ? off[j] : kOutside, in_bytes(k0, a.K));
    };
    // the row this lane asks for early, if any: four of a wave, which lie in
    // one block of 16 and so are of one kind with SwiGLU
    const int lr0 = (mt & 7) * (BN / 8) + 4 * wave;
    uint32_t ahead = kOutside;
    if (lane < 4 && 4 * wave < BN / 8) {
        const int lr = lr0 + lane;
        const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
        if (n0 + wr < a.N) ahead = (uint32_t)(wr * a.ldw) * 2u;
    }
    const auto ra = make_rsrc(wbase + (GLU && ((lr0 >> 4) & 1) ? (int64_t)a.N * a.ldw : 0));
    auto touch = [&](int s) {
        touch_to_lds(ra, tile_lds + 2 * kRows * BK + wave * 128, s * BK < a.K ? ahead : kOutside, in_bytes(s * BK, a.K));
    };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wn = wave & 1, wm = wave >> 1;
    const bool late = wave >= 4;
    const int S = (a.K + BK - 1) / BK;
    copy(0);
    keep_order();
#pragma unroll
    for (int s = 1; s < kAhead; ++s) touch(s);
    // the copies are older than the touches
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kAhead - 1) : "memory");
    if (late) asm volatile("s_barrier" ::: "memory");
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + (s & 1) * kRows * BK) + r * 8 +
                                ((4 * h + g) ^ (r & 7));
            u32x4 fw[RB], fx[MB];
#pragma unroll
            for (int j = 0; j < MB; ++j) fx[j] = base[(BN + (wm * MB + j) * 16) * 8];
#pragma unroll
            for (int i = 0; i < RB; ++i) fw[i] = base[(wn * RB + i) * 128];
            __builtin_amdgcn_sched_barrier(0);
            if (h == 1 && late) asm volatile("s_waitcnt vmcnt(1)" ::: "memory");   // all but the last touch
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_setprio(1);
            if (h == 0) {
                copy(s + 1);
                keep_order();
                touch(s + kAhead);   // the last: the waits below count on it
            }
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[i], fx[j], acc[i][j]);
            if (h == 0) {
                // a copy after every second matrix instruction
#pragma unroll
                for (int q = 0; q < QW + QX + 1; ++q) {
                    __builtin_amdgcn_sched_group_barrier(0x8, 2, 0);
                    __builtin_amdgcn_sched_group_barrier(0x10, 1, 0);
                }
            }
            __builtin_amdgcn_s_setprio(0);
            __builtin_amdgcn_sched_barrier(0);
            if (h == 1 && !late) asm volatile("s_waitcnt vmcnt(1)" ::: "memory");
            asm volatile("s_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    // the early waves' last barrier pairs with the late ones' last phase;
    // every copy has landed before the LDS is used again
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (!late) asm volatile("s_barrier" ::: "memory");
    __syncthreads();
    static_assert(8 * out_stage_floats<RB>() * 4 <= 2 * kRows * BK * 2, "the sums fit the slots");
    put_tile<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

// Workgroups of one launch, in whole eighths for the XCDs; 0 if they would
// have 2^32 threads or more, which no launch takes.
unsigned groups_of(int64_t tiles, int threads) {
    const int64_t groups = (tiles + 7) / 8 * 8;
    return groups < ((int64_t)1 << 32) / threads ? (unsigned)groups : 0u;
}

template <class T, int RB, int MB, bool GLU>
hipError_t launch_phased(const LinearArgs& a, hipStream_t s) {
    constexpr int kOutN = GLU ? 16 * RB : 32 * RB, BM = 64 * MB;
    const int64_t tiles = (int64_t)((a.N + kOutN - 1) / kOutN) * ((a.M + BM - 1) / BM);
    const unsigned groups = groups_of(tiles, 512);
    if (!groups) return hipErrorInvalidConfiguration;
    linear_phased_kernel<T, RB, MB, GLU>
        <<<groups, 512, (size_t)2 * (32 * RB + BM) * BK * 2 + 8 * 256, s>>>(a);
    return hipGetLastError();
}

// Products too small to fill the GPU with those tiles: BN weight rows x BM
// tokens, WN x WM waves, K in steps of 64 through a ring of D LDS slots, one
// barrier a step, so that D - 2 steps' copies are on their way while one is
// multiplied. Rows, chunks and copies as above.
template <class T, int BM, int BN, int WM, int WN, int D, bool GLU>
__global__ __launch_bounds__(64 * WM * WN) void linear_ring_kernel(LinearArgs a) {
    constexpr int kWaves = WM * WN, kRows = BN + BM;
    constexpr int RB = BN / WN / 16, MB = BM / WM / 16;   // blocks of a wave's tile
    constexpr int kOutN = GLU ? BN / 2 : BN;
    constexpr int QW = BN / 8 / kWaves, QX = BM / 8 / kWaves;   // copies per thread and step
    static_assert(BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole copies");
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    int nt, mt;
    if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + BM - 1) / BM, nt, mt)) return;
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * BM;
    const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
    const uint16_t* wbase = reinterpret_cast<const uint16_t*>(a.w) + (int64_t)n0 * a.ldw;
    const auto rw = make_rsrc(wbase), ru = make_rsrc(wbase + (GLU ? (int64_t)a.N * a.ldw : 0));
    const auto rx = make_rsrc(reinterpret_cast<const uint16_t*>(a.x) + m0 * a.ldx);
    uint32_t off[QW + QX];
#pragma unroll
    for (int j = 0; j < QW; ++j) {
        const int lr = (j * kWaves + wave) * 8 + crow;
        const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
        off[j] = n0 + wr < a.N ? (uint32_t)(wr * a.ldw + 8 * chunk) * 2u : kOutside;
    }
#pragma unroll
    for (int j = 0; j < QX; ++j) {
        const int lr = (j * kWaves + wave) * 8 + crow;
        off[QW + j] = m0 + lr < a.M ? (uint32_t)(lr * a.ldx + 8 * chunk) * 2u : kOutside;
    }
    auto copy = [&](int s, int slot) {
        const int k0 = s * BK;
        const bool in = k0 + 8 * chunk < a.K;
        uint16_t* dst = tile_lds + slot * kRows * BK;
#pragma unroll
        for (int j = 0; j < QW; ++j) {
            const bool up = GLU && ((((j * kWaves + wave) * 8) >> 4) & 1);
            copy_to_lds(up ? ru : rw, dst + (j * kWaves + wave) * 8 * BK, in ? off[j] : kOutside, in_bytes(k0, a.K));
        }
#pragma unroll
        for (int j = 0; j < QX; ++j)
            copy_to_lds(rx, dst + (BN + (j * kWaves + wave) * 8) * BK, in ? off[QW + j] : kOutside, in_bytes(k0, a.K));
    };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wn = wave % WN, wm = wave / WN;
    const int S = (a.K + BK - 1) / BK;
#pragma unroll
    for (int j = 0; j < D - 1; ++j) {
        copy(j, j);
        keep_order();
    }
    int slot = 0;
    for (int s = 0; s < S; ++s) {
        // step s is whole (this wave's part, then everyone's), and everyone
        // has read the slot before it, which takes step s + D - 1
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((QW + QX) * (D - 2)) : "memory");
        copy(s + D - 1, slot == 0 ? D - 1 : slot - 1);
        const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + slot * kRows * BK) + r * 8;
        u32x4 fw[2][RB], fx[2][MB];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = (4 * h + g) ^ (r & 7);
#pragma unroll
            for (int j = 0; j < MB; ++j) fx[h][j] = base[(BN + (wm * MB + j) * 16) * 8 + pos];
#pragma unroll
            for (int i = 0; i < RB; ++i) fw[h][i] = base[(wn * RB + i) * 128 + pos];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[h][i], fx[h][j], acc[i][j]);
        slot = slot + 1 == D ? 0 : slot + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();   // every wave is done with the slots
    static_assert(kWaves * out_stage_floats<RB>() * 4 <= D * kRows * BK * 2, "the sums fit the slots");
    put_tile<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

template <class T, int BM, int BN, int WM, int WN, int D, bool GLU>
hipError_t launch_ring(const LinearArgs& a, hipStream_t s) {
    constexpr int kOutN = GLU ? BN / 2 : BN;
    const int64_t tiles = (int64_t)((a.N + kOutN - 1) / kOutN) * ((a.M + BM - 1) / BM);
    const unsigned groups = groups_of(tiles, 64 * WM * WN);
    if (!groups) return hipErrorInvalidConfiguration;
    linear_ring_kernel<T, BM, BN, WM, WN, D, GLU>
        <<<groups, 64 * WM * WN, (size_t)D * (BN + BM) * BK * 2, s>>>(a);
    return hipGetLastError();
}

// Rows of any alignment: 64 weight rows x 64 tokens, WN x WM waves, K in
// steps of 64 through two LDS buffers; the rows go through registers, loaded
// two steps ahead with unaligned loads. LDS layout as above.
constexpr int kAnyWN = 2, kAnyWM = 4;
template <class T, bool GLU>
__global__ __launch_bounds__(64 * kAnyWN * kAnyWM) void linear_any_kernel(LinearArgs a) {
    constexpr int kWaves = kAnyWN * kAnyWM, kRows = 128;
    constexpr int RB = 4 / kAnyWN, MB = 4 / kAnyWM, Q = kRows / 8 / kWaves;
    constexpr int kOutN = GLU ? 32 : 64;
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    int nt, mt;
    if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + 63) / 64, nt, mt)) return;
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * 64;
    // this thread's chunks: LDS rows 8 (kWaves j + wave) + lane / 8 (64 of the
    // weights, then the tokens), position lane % 8
    const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
    const uint16_t* src[Q];
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        const int lr = 8 * (kWaves * j + wave) + crow, xr = lr - 64;
        if (lr < 64) {
            const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
            const int64_t row = (GLU && ((lr >> 4) & 1) ? (int64_t)a.N : 0) + n0 + wr;
            src[j] = n0 + wr < a.N ? reinterpret_cast<const uint16_t*>(a.w) + row * a.ldw + 8 * chunk : nullptr;
        } else {
            src[j] = m0 + xr < a.M ? reinterpret_cast<const uint16_t*>(a.x) + (m0 + xr) * a.ldx + 8 * chunk : nullptr;
        }
    }
    const int S = (a.K + BK - 1) / BK;
    u32x4 even[Q], odd[Q];   // the rows of an even and of an odd step
    auto fetch = [&](int s, u32x4 (&reg)[Q]) {
        const int left = a.K - (s * BK + 8 * chunk);
#pragma unroll
        for (int j = 0; j < Q; ++j)
            reg[j] = src[j] && left > 0 ? load_chunk(src[j] + s * BK, left) : u32x4{0u, 0u, 0u, 0u};
    };
    auto settle = [&](int s, const u32x4 (&reg)[Q]) {   // registers to LDS
        u32x4* dst = reinterpret_cast<u32x4*>(tile_lds + (s & 1) * kRows * BK) + lane;
#pragma unroll
        for (int j = 0; j < Q; ++j) dst[(kWaves * j + wave) * 64] = reg[j];
    };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wn = wave % kAnyWN, wm = wave / kAnyWN;
    auto step = [&](int s, u32x4 (&mine)[Q], const u32x4 (&other)[Q]) {
        __syncthreads();   // step s is in LDS; everyone is done with the other buffer
        if (s + 2 < S) fetch(s + 2, mine);
        const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + (s & 1) * kRows * BK) + r * 8;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = (4 * h + g) ^ (r & 7);
            u32x4 fw[RB], fx[MB];
#pragma unroll
            for (int j = 0; j < MB; ++j) fx[j] = base[(64 + (wm * MB + j) * 16) * 8 + pos];
#pragma unroll
            for (int i = 0; i < RB; ++i) fw[i] = base[(wn * RB + i) * 128 + pos];
#pragma unroll
            for (int i = 0; i < RB; ++i)
#pragma unroll
                for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[i], fx[j], acc[i][j]);
        }
        if (s + 1 < S) settle(s + 1, other);
    };
    if (S > 0) {
        fetch(0, even);
        if (S > 1) fetch(1, odd);
        settle(0, even);
    }
    for (int s = 0; s < S; s += 2) {
        step(s, even, odd);
        if (s + 1 < S) step(s + 1, odd, even);
    }
    __syncthreads();   // every wave is done with the buffers
    static_assert(kWaves * out_stage_floats<RB>() * 4 <= 2 * kRows * BK * 2, "the sums fit the buffers");
    put_tile<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

template <class T, int RB, int MB, int D, bool GLU>
hipError_t launch_stream(const LinearArgs& a, int waves, hipStream_t s) {
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const dim3 grid((unsigned)((a.N + kRowsOut - 1) / kRowsOut), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
    if (!groups_of(grid.x, 64 * waves)) return hipErrorInvalidConfiguration;
    const size_t lds = std::max((size_t)waves * D * (RB + MB) * 2048, (size_t)waves * RB * MB * 1024);
    linear_stream_kernel<T, RB, MB, D, GLU><<<grid, 64 * waves, lds, s>>>(a);
    return hipGetLastError();
}

template <class T, int RB, int MB, int D, bool GLU>
hipError_t launch_skinny(const LinearArgs& a, int waves, hipStream_t s) {
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const dim3 grid((unsigned)((a.N + kRowsOut - 1) / kRowsOut), (unsigned)((a.M + 16 * MB - 1) / (16 * MB)));
    if (!groups_of(grid.x, 64 * waves)) return hipErrorInvalidConfiguration;
    const size_t lds = (size_t)waves * RB * MB * 1024;
    linear_skinny_kernel<T, RB, MB, D, GLU><<<grid, 64 * waves, lds, s>>>(a);
    return hipGetLastError();
}

constexpr int kSkinnyTokens = 64;

template <class T, bool GLU>
hipError_t launch_linear_t(const LinearArgs& a, hipStream_t s) {
    if (a.M <= kSkinnyTokens) {
        const int mb = (a.M + 15) / 16;
        const int64_t b32 = ((GLU ? 2ll * a.N : a.N) + 31) / 32;   // blocks of 32 weight rows
        auto waves_for = [&](int64_t blocks) {
            int w = 4;
            while (w < 16 && blocks * w < 3000 && w * BK < a.K) w *= 2;
            return w;
        };
        // few rows: a workgroup per 16 of them and per 16 tokens, up to 16
        // waves along K (64 x 128 x 2048: 6.9 us; 32 rows each 8.5 us. 1 x
        // 4096 x 14336: 22.5 us, through LDS 23.3 us)
        if (b32 * mb < 256) {
            if constexpr (GLU) return launch_skinny<T, 2, 1, 3, GLU>(a, waves_for(b32 * mb), s);
            else return launch_skinny<T, 1, 1, 4, GLU>(a, waves_for(2 * b32 * mb), s);
        }
        if (!a.aligned) {
            if (mb == 1) return launch_skinny<T, 2, 1, 3, GLU>(a, waves_for(b32), s);
            if (mb == 2) return launch_skinny<T, 4, 2, 2, GLU>(a, 4, s);
            return launch_skinny<T, 4, 4, 2, GLU>(a, 4, s);
        }
        // through LDS: 16 x 14336 x 4096 SwiGLU 44.7 us (straight into
        // registers 49.9 us), 32 tokens 49.6 (54.6), 64 tokens 65.3 (71.9).
        // More than 32 tokens share a workgroup's weights only where the rows
        // fill the GPU (64 x 4096 x 14336: 38.8 us, 51.4 us shared), up to 32
        // take 16 rows where 32 do not (17 x 4096 x 14336: 28.4 and 34.3 us).
        const int w = std::min(4, std::max(1, (a.K + BK - 1) / BK));
        if (mb == 1) return launch_stream<T, 2, 1, 2, GLU>(a, w, s);
        if constexpr (!GLU)
            if (mb == 2 && b32 <= 256) return launch_stream<T, 1, 2, 2, GLU>(a, w, s);
        if (mb == 2 || b32 <= 256) return launch_stream<T, 2, 2, 2, GLU>(a, w, s);
        return launch_stream<T, 2, 4, 2, GLU>(a, w, s);
    }
    const int64_t cols = GLU ? 2ll * a.N : a.N;
    auto tiles = [&](int64_t bn, int64_t bm) { return (cols + bn - 1) / bn * ((a.M + bm - 1) / bm); };
    if (!a.aligned) {
        const unsigned groups = groups_of(tiles(64, 64), 64 * kAnyWN * kAnyWM);
        if (!groups) return hipErrorInvalidConfiguration;
        linear_any_kernel<T, GLU><<<groups, 64 * kAnyWN * kAnyWM, 2 * 128 * BK * 2, s>>>(a);
        return hipGetLastError();
    }
    // The tile whose rounds (one workgroup per CU; two of the 64 x 64 tile)
    // take least, by a full round's time for K = 4096, measured in us: small
    // tiles fill the GPU, large ones read less per product. 256 x 4096 rows:
    // 21 us with 64 x 64 tiles, 34 with 128 x 128; 1024 x 4096: 55, 39 and 55
    // with 256 x 128; 2048 x 4096: 80, 67 and 85 with 256 x 256; 4096 x 4096:
    // 127 with 256 x 128, 102 with 256 x 256.
    auto rounds = [&](int64_t bn, int64_t bm, int64_t at_once) { return (tiles(bn, bm) + at_once - 1) / at_once; };
    const int64_t cost[5] = {rounds(64, 64, 256) == 1 ? 21 : 28 * rounds(64, 64, 512), 39 * rounds(128, 128, 256),
                             66 * rounds(128, 256, 256), 80 * rounds(192, 256, 256), 100 * rounds(256, 256, 256)};
    switch (std::min_element(cost, cost + 5) - cost) {
        case 0: return launch_ring<T, 64, 64, 2, 2, 4, GLU>(a, s);
        case 1: return launch_ring<T, 128, 128, 2, 4, 4, GLU>(a, s);
        case 2: return launch_ring<T, 256, 128, 4, 2, 3, GLU>(a, s);
        case 3: return launch_phased<T, 6, 4, GLU>(a, s);
        default: return launch_phased<T, 8, 4, GLU>(a, s);
    }
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t s) {
    const bool glu = a.act == PW_ACT_SWIGLU;
    if (a.in_dtype == PW_BF16) return glu ? launch_linear_t<__bf16, true>(a, s) : launch_linear_t<__bf16, false>(a, s);
    return glu ? launch_linear_t<_Float16, true>(a, s) : launch_linear_t<_Float16, false>(a, s);
}

}  // namespace pw
