// Root-mean-square norm of rows, with the addition of a residual before it
// and, if asked for, e4m3 values with a scale for each 128 columns after it;
// and the e4m3 quantizer of given rows or weights.
//
// Norm of a row: h = x + residual, rounded to the residual's type, which is
// written; r = 1 / sqrt(mean(h^2) + eps); y = h w r, in fp32 from the written
// h on (as (h r) w: h r is at most sqrt(n), so no product leaves fp32's range
// before y does) and rounded once. In 8 bits: z = h w in fp32 (exact for 16-bit h
// and w), m = max |z| over 128 columns, codes 448 z / m and the scale r m / 448: r
// cancels from the codes, so they do not hang on its rounding. Rows whose sum of
// squares leaves fp32's range, and blocks whose z do, go through fp64.
//
// Bound by the bytes: each element is read once, held in registers over the
// reduction, and written once. 16384 x 4096 bf16 with a bf16 residual and e4m3
// out 84 us, 5.6 TB/s (a large copy reaches 5.1); quantized in rows, bf16 24576 x
// 1408, and in tiles, fp32 28672 x 4096: 21 and 102 us, 5.0 and 5.8 TB/s. One
// row of 4096 takes 3.2 us: a trip to memory, the waves' joined sums, a store.
#include "pw_internal.h"

#include <algorithm>
#include <type_traits>

#include "e4m3.h"

namespace pw {
namespace {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x2_byte __attribute__((ext_vector_type(2), aligned(1)));

// Eight consecutive elements as they lie in memory.
template <class T>
struct Eight {
    typedef T vec __attribute__((ext_vector_type(8), aligned(16)));
    vec v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const vec*>(p); }
    // rows of any alignment (the loads are declared with the element's), and
    // their ends
    typedef T any __attribute__((ext_vector_type(8), aligned(sizeof(T))));
    __device__ __forceinline__ void load_some(const T* p, int left) {
        if (left >= 8) {
            v = *reinterpret_cast<const any*>(p);
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? p[i] : (T)0.0f;
    }
    __device__ __forceinline__ float operator[](int i) const { return (float)v[i]; }
};

template <class T>
__device__ __forceinline__ void store8(T* p, const float (&f)[8]) {
    typename Eight<T>::vec v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (T)f[i];
    *reinterpret_cast<typename Eight<T>::vec*>(p) = v;
}
template <class T>
__device__ __forceinline__ void store_some(T* p, int left, const float (&f)[8]) {
    if (left >= 8) {
        typename Eight<T>::any v;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = (T)f[i];
        *reinterpret_cast<typename Eight<T>::any*>(p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = (T)f[i];
}
template <bool VEC, class T>
__device__ __forceinline__ void put8(T* p, int left, const float (&f)[8]) {
    if (VEC) store8(p, f);
    else store_some(p, left, f);
}

// Eight columns of 16 neighbouring lanes are a block: its largest magnitude,
// the codes (of t = 448 z / m), and (the first lane) the scale.
__device__ __forceinline__ void quotients(float (&t)[8], const float (&z)[8], const E4m3Factor& f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e] = e4m3_scaled(z[e], f);
}
template <bool VEC>
__device__ __forceinline__ void put_codes(uint8_t* p, int left, const float (&t)[8]) {
    const uint32_t a = e4m3_pack(t[0], t[1], t[2], t[3]);
    const uint32_t b = e4m3_pack(t[4], t[5], t[6], t[7]);
    if (VEC) {
        *reinterpret_cast<u32x2*>(p) = u32x2{a, b};
        return;
    }
    if (left >= 8) {
        *reinterpret_cast<u32x2_byte*>(p) = u32x2{a, b};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = (uint8_t)((i < 4 ? a : b) >> (8 * (i & 3)));
}
__device__ __forceinline__ float largest(const float (&z)[8]) {
    float m = fabsf(z[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = fmaxf(m, fabsf(z[i]));
    return m;
}

// ---- norm ----

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The quotients 448 h w / m and the scale r m / 448 of a block whose h w, or
// whose row's r, fp32 does not hold (h comes times 2^-shift). NaN counts no more
// here than there.
__device__ __forceinline__ void wide_block(const float (&h)[8], const float (&w)[8], float r, int shift, float (&q)[8], float& scale) {
    double m = ldexp((double)kE4m3Least, -shift);
#pragma unroll
    for (int e = 0; e < 8; ++e) m = fmax(m, fabs((double)h[e] * (double)w[e]));
#pragma unroll
    for (int d = 8; d; d >>= 1) m = fmax(m, __shfl_xor(m, d));
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = (float)((double)kE4m3Top * ((double)h[e] * (double)w[e]) / m);
    scale = (float)(m * (double)r / (double)kE4m3Top);
}

// blockDim.x / 64 waves a row, V pieces of 8 elements a lane: piece i of lane
// l of wave w starts at column 8 (64 (i waves + w) + l). R: the residual's
// type (void: none). A workgroup a row, so that rows of any length up to 65536
// stay in registers: a lane has as few pieces as 16 waves allow, but two of a
// row longer than one wave's (us with 1, 2, 8 pieces, bf16 with residual and
// e4m3 out: 65536 x 512 42, 44, 79; 16384 x 2048 44, 42, 45; 8192 x 7168 86, 76,
// 82; 4096 x 16384 two 93, eight 95; 2048 x 32768 eight 101).
template <class X, class R, int V, bool VEC>
__global__ __launch_bounds__(1024) void rms_norm_kernel(NormArgs a) {
    constexpr bool kAdd = !std::is_same<R, void>::value;
    typedef typename std::conditional<kAdd, R, X>::type H;   // what is normalised
    __shared__ float part[16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int64_t t = blockIdx.x;
    const X* x = reinterpret_cast<const X*>(a.x) + t * a.ldx;
    const H* res = reinterpret_cast<const H*>(a.residual) + t * a.ldr;
    Eight<X> xv[V];
    Eight<H> rv[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (64 * (i * waves + wave) + lane);
        if (c < a.n) {
            if (VEC) xv[i].load(x + c);
            else xv[i].load_some(x + c, a.n - c);
            if (kAdd) {
                if (VEC) rv[i].load(res + c);
                else rv[i].load_some(res + c, a.n - c);
            }
        } else {
            xv[i].v = 0;
            if (kAdd) rv[i].v = 0;
        }
    }
    float h[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (64 * (i * waves + wave) + lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            h[i][e] = xv[i][e];
            if (kAdd) h[i][e] = (float)(H)(h[i][e] + rv[i][e]);
            sum = __builtin_fmaf(h[i][e], h[i][e], sum);
        }
        if (kAdd && c < a.n) put8<VEC>(reinterpret_cast<H*>(a.h) + t * a.ldh + c, a.n - c, h[i]);
    }
    auto over_row = [&](float v, auto join, auto in_wave) {
        v = in_wave(v);
        if (waves == 1) return v;
        __syncthreads();
        if (lane == 0) part[wave] = v;
        __syncthreads();
        v = part[0];
        for (int w = 1; w < waves; ++w) v = join(v, part[w]);
        return v;
    };
    auto add = [](float p, float q) { return p + q; };
    sum = over_row(sum, add, wave_sum);
    float r;
    int shift = 0;   // h is held times 2^-shift
    const bool wide = !(sum < 0x1p+120f && sum > 0x1p-90f);
    if (!wide) {
        r = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    } else {
        // squares that overflow, or vanish beside a small eps: again in fp64,
        // whose range holds the square of every fp32 value
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) s += (double)h[i][e] * (double)h[i][e];
        __shared__ double wide[16];
#pragma unroll
        for (int d = 32; d; d >>= 1) s += __shfl_xor(s, d);
        if (waves > 1) {
            __syncthreads();
            if (lane == 0) wide[wave] = s;
            __syncthreads();
            s = 0.0;
            for (int w = 0; w < waves; ++w) s += wide[w];
        }
        // r itself may leave fp32's range: its power of two goes to h
        const double r64 = 1.0 / sqrt(s / a.n + (double)a.eps);
        const bool usual = r64 > 0.0 && r64 < (double)INFINITY;
        shift = usual ? -__builtin_amdgcn_readfirstlane(ilogb(r64)) : 0;
        r = (float)ldexp(r64, shift);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = ldexpf(h[i][e], -shift);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int c = 8 * (64 * (i * waves + wave) + lane);
        float w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = 1.0f;
        if (a.weight && c < a.n) {
            auto take = [&](auto v, auto type) {
                typedef decltype(type) W;
                if (VEC) v.load(reinterpret_cast<const W*>(a.weight) + c);
                else v.load_some(reinterpret_cast<const W*>(a.weight) + c, a.n - c);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = v[e];
            };
            if (a.w_dtype == PW_F32) take(Eight<float>{}, 0.0f);
            else if (a.w_dtype == PW_BF16) take(Eight<__bf16>{}, (__bf16)0.0f);
            else take(Eight<_Float16>{}, (_Float16)0.0f);
        }
        if (a.y_dtype == PW_E4M3) {
            float z[8], q[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = h[i][e] * w[e];
            const float m = fmaxf(row_max(largest(z)), kE4m3Least);
            float scale = m * r / kE4m3Top;
            if (!wide && m < INFINITY) quotients(q, z, e4m3_factor(m));
            else wide_block(h[i], w, r, shift, q, scale);   // (the same for a block's 16 lanes)
            if (c >= a.n) continue;
            put_codes<VEC>(reinterpret_cast<uint8_t*>(a.y) + t * a.ldy + c, a.n - c, q);
            if (!(lane & 15)) a.scale[t * a.s_row + (c / kScaleBlock) * a.s_block] = scale;
            continue;
        }
        if (c >= a.n) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * r * w[e];
        const int64_t at = t * a.ldy + c;
        if (a.y_dtype == PW_F32) put8<VEC>(reinterpret_cast<float*>(a.y) + at, a.n - c, h[i]);
        else if (a.y_dtype == PW_BF16) put8<VEC>(reinterpret_cast<__bf16*>(a.y) + at, a.n - c, h[i]);
        else put8<VEC>(reinterpret_cast<_Float16*>(a.y) + at, a.n - c, h[i]);
    }
}

bool rows_aligned(const void* p, int64_t ld, int dtype, int bytes) {
    const int64_t e = dtype == PW_F32 ? 4 : dtype == PW_E4M3 ? 1 : 2;
    return (uintptr_t)p % bytes == 0 && ld * e % bytes == 0;
}

template <class X, class R>
hipError_t launch_norm_t(const NormArgs& a, hipStream_t s) {
    auto ok = [&](const void* p, int64_t ld, int dtype) {
        return !p || rows_aligned(p, a.T > 1 ? ld : 0, dtype, dtype == PW_E4M3 ? 8 : 16);
    };
    const bool vec = a.n % 8 == 0 && ok(a.x, a.ldx, a.x_dtype) && ok(a.residual, a.ldr, a.r_dtype) &&
                     ok(a.h, a.ldh, a.r_dtype) && ok(a.y, a.ldy, a.y_dtype) && ok(a.weight, 0, a.w_dtype);
    const int pieces = (a.n + 511) / 512;   // of a wave
    auto go = [&](auto kernel, int v) {
        int waves = 1;
        while (waves * v < pieces) waves *= 2;
        if ((int64_t)a.T * 64 * waves >= (int64_t)1 << 32) return hipErrorInvalidConfiguration;
        kernel<<<(unsigned)a.T, 64 * waves, 0, s>>>(a);
        return hipGetLastError();
    };
    if (pieces <= 1) return vec ? go(rms_norm_kernel<X, R, 1, true>, 1) : go(rms_norm_kernel<X, R, 1, false>, 1);
    if (pieces <= 32) return vec ? go(rms_norm_kernel<X, R, 2, true>, 2) : go(rms_norm_kernel<X, R, 2, false>, 2);
    return vec ? go(rms_norm_kernel<X, R, 8, true>, 8) : go(rms_norm_kernel<X, R, 8, false>, 8);
}

// ---- quantizer ----

// Workgroup: 128 rows x 128 columns; 16 lanes and 8 columns each to a row.
template <class X, bool TILE, bool VEC>
__global__ __launch_bounds__(256) void quantize_kernel(QuantizeArgs a) {
    __shared__ float part[4];
    const int tid = threadIdx.x;
    const int cols = (a.K + kScaleBlock - 1) / kScaleBlock, down = (a.M + kScaleBlock - 1) / kScaleBlock;
    const int kb = blockIdx.x % cols;
    const int64_t q = blockIdx.x / cols;
    const int mb = (int)(q % down);
    const int64_t e = q / down;
    const int c = kb * kScaleBlock + 8 * (tid & 15);
    const X* x = reinterpret_cast<const X*>(a.x) + e * a.x_batch;
    uint8_t* out = a.q + e * a.q_batch;
    float* scale = a.scale + e * a.s_batch;
    Eight<X> v[8];
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = mb * kScaleBlock + 16 * i + (tid >> 4);
        v[i].v = 0;
        if (row < a.M && c < a.K) {
            if (VEC) v[i].load(x + (int64_t)row * a.ldx + c);
            else v[i].load_some(x + (int64_t)row * a.ldx + c, a.K - c);
        }
    }
    float f[8], t[8];
    auto values = [&](int i) {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = v[i][j];
    };
    if (TILE) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            values(i);
            m = fmaxf(m, largest(f));
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
        if ((tid & 63) == 0) part[tid >> 6] = m;
        __syncthreads();
        m = fmaxf(fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3])), kE4m3Least);
        if (tid == 0) scale[mb * a.s_row + kb * a.s_block] = m / kE4m3Top;
    }
    E4m3Factor factor = TILE ? e4m3_factor(m) : E4m3Factor{0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = mb * kScaleBlock + 16 * i + (tid >> 4);
        values(i);
        if (!TILE) {
            m = fmaxf(row_max(largest(f)), kE4m3Least);
            factor = e4m3_factor(m);
        }
        if (row >= a.M || c >= a.K) continue;
        quotients(t, f, factor);
        put_codes<VEC>(out + (int64_t)row * a.ldq + c, a.K - c, t);
        if (!TILE && !(tid & 15)) scale[row * a.s_row + kb * a.s_block] = m / kE4m3Top;
    }
}

template <class X>
hipError_t launch_quantize_t(const QuantizeArgs& a, hipStream_t s) {
    const bool vec = a.K % 8 == 0 && rows_aligned(a.x, a.M > 1 ? a.ldx : 0, a.dtype, 16) &&
                     rows_aligned(a.x, a.E > 1 ? a.x_batch : 0, a.dtype, 16) &&
                     rows_aligned(a.q, a.M > 1 ? a.ldq : 0, PW_E4M3, 8) && rows_aligned(a.q, a.E > 1 ? a.q_batch : 0, PW_E4M3, 8);
    const int64_t groups = (int64_t)((a.K + kScaleBlock - 1) / kScaleBlock) * ((a.M + kScaleBlock - 1) / kScaleBlock) * a.E;
    if (groups >= ((int64_t)1 << 32) / 256) return hipErrorInvalidConfiguration;
    auto go = [&](auto kernel) {
        kernel<<<(unsigned)groups, 256, 0, s>>>(a);
        return hipGetLastError();
    };
    if (a.tile) return vec ? go(quantize_kernel<X, true, true>) : go(quantize_kernel<X, true, false>);
    return vec ? go(quantize_kernel<X, false, true>) : go(quantize_kernel<X, false, false>);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
    auto with = [&](auto x) {
        typedef decltype(x) X;
        if (!a.residual) return launch_norm_t<X, void>(a, s);
        if (a.r_dtype == PW_F32) return launch_norm_t<X, float>(a, s);
        return launch_norm_t<X, X>(a, s);
    };
    if (a.x_dtype == PW_F32) return with(0.0f);
    if (a.x_dtype == PW_BF16) return with((__bf16)0.0f);
    return with((_Float16)0.0f);
}

hipError_t launch_quantize_fp8(const QuantizeArgs& a, hipStream_t s) {
    if (a.dtype == PW_F32) return launch_quantize_t<float>(a, s);
    if (a.dtype == PW_BF16) return launch_quantize_t<__bf16>(a, s);
    return launch_quantize_t<_Float16>(a, s);
}

}  // namespace pw
