// Dense product of e4m3 operands with block scales: T is E4M3 or E4M3Full
// (product_dev.h).
#pragma once

#include "product_dev.h"

namespace pw {
namespace {

// Few rows of any alignment: RB blocks of 16 weight rows (with SwiGLU gate and
// up rows of the same 16) and 16 rows of x a workgroup, K dealt to its waves in
// pieces of 128 bytes, each straight into matrix operands with unaligned loads
// (two of 16 bytes a lane and row), D pieces in flight a wave. The waves' sums
// meet in LDS, in wave order. (Such a load takes a CU 55 to 130 cycles, twice
// and more what an aligned one does, which bounds it: 44 x 60 x 7168 with rows
// 7171 apart 21 us with 4, 8 and 16 waves alike, 30 through 64 x 64 tiles; 4 x
// 4096 x 5109 13 and 23, 38 x 1303 x 5284 16 and 25; 53 x 2989 x 2438, past the
// rule's 512 workgroups, 20 and 15.)
template <class T, int RB, int D, bool GLU>
__global__ __launch_bounds__(512) void fp8_skinny_kernel(ProductArgs a) {
    extern __shared__ __attribute__((aligned(16))) float part[];   // [waves][RB][64 lanes][4]
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16 * (GLU ? RB / 2 : RB), m0 = blockIdx.y * 16;
    const int total = (a.K + 127) >> 7, whole = a.K >> 7;   // pieces, whole ones
    const int n = whole > wave ? (whole - wave + waves - 1) / waves : 0;
    // rows past the end repeat the last one; their sums are dropped
    const uint8_t* wp[RB];
#pragma unroll
    for (int b = 0; b < RB; ++b) {
        const int64_t row = min(n0 + 16 * (GLU ? b >> 1 : b) + r, a.N - 1) + (GLU && (b & 1) ? (int64_t)a.N : 0);
        wp[b] = reinterpret_cast<const uint8_t*>(a.w) + row * a.ldw + 16 * g;
    }
    const int64_t m = min(m0 + r, a.M - 1);
    const uint8_t* xp = reinterpret_cast<const uint8_t*>(a.x) + m * a.ldx + 16 * g;
    const float* xs = a.xs + m * a.xs_row;
    const float *wg = scale_row<GLU>(a, min(n0, a.N - 1), 0), *wu = scale_row<GLU>(a, min(n0, a.N - 1), 1);
    f32x4 acc[RB][1];
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    struct Piece {
        u32x4 w[RB][2], x[1][2];
        float sx, sg, su;
    };
    auto scales = [&](Piece& p, int k) {
        p.sg = wg[k * a.ws_block];
        p.su = GLU ? wu[k * a.ws_block] : 0.0f;
        p.sx = xs[k * a.xs_block];
    };
    auto load = [&](Piece& p, int i) {   // the wave's i-th whole piece
        const int k = wave + waves * i;
        scales(p, k);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int b = 0; b < RB; ++b) p.w[b][h] = *reinterpret_cast<const u32x4_byte*>(wp[b] + 128 * (int64_t)k + 64 * h);
            p.x[0][h] = *reinterpret_cast<const u32x4_byte*>(xp + 128 * (int64_t)k + 64 * h);
        }
    };
    auto multiply = [&](const Piece& p) {
        const float f[2][1] = {{p.sx * p.sg}, {p.sx * p.su}};
        scaled_blocks<T, RB, 1, GLU>(acc, p.w, p.x, f);
    };
    Piece ring[D];
#pragma unroll
    for (int j = 0; j < D; ++j)
        if (j < n) load(ring[j], j);
    for (int i = 0; i < n; i += D) {
#pragma unroll
        for (int j = 0; j < D; ++j) {
            if (i + j < n) multiply(ring[j]);
            if (i + D + j < n) load(ring[j], i + D + j);
        }
    }
    if (total > whole && whole % waves == wave) {   // the last, partial piece
        Piece p;
        scales(p, whole);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int left = a.K - (128 * whole + 16 * g + 64 * h);
#pragma unroll
            for (int b = 0; b < RB; ++b) p.w[b][h] = load_bytes(wp[b] + 128 * (int64_t)whole + 64 * h, left);
            p.x[0][h] = load_bytes(xp + 128 * (int64_t)whole + 64 * h, left);
        }
        multiply(p);
    }
    join_waves<RB, 1, GLU>(a, acc, part, n0, m0);
}

template <class T, bool GLU>
hipError_t launch_skinny(const ProductArgs& a, hipStream_t s) {
    constexpr int RB = GLU ? 2 : 1;
    const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 15) / 16));
    const int waves = a.K >= 2048 ? 8 : 4;
    fp8_skinny_kernel<T, RB, 3, GLU><<<grid, 64 * waves, (size_t)waves * RB * 1024, s>>>(a);
    return hipGetLastError();
}

// Streamed weights or tiles, whichever takes less by times measured (us):
// 64 x 4096 x 4096 7.7 with blocks of 32 rows of x, 9.0 with 16, 9.3 with 64, 14.5
// with 64 x 64 tiles; 128 rows 11.4, 13.7, 9.7 and 14.8; 256 rows 18.9, 23.1, 17.1
// and 15.4; 128 x 4096 x 14336 25, 37, 20 and 42. 64 x 14336 x 4096 SwiGLU 49, 87,
// 42 and 30 (every block of rows reads the weights again). E4M3Full, in this
// order: 64 x 4096 x 4096 8.5, 10.1, 11.7, 19.5; 128 rows 12.9, 15.7, 12.3, 19.8;
// 256 rows 20.8, 24.8, 21.4, 20.0; 64 x 14336 x 4096 SwiGLU 50, 88, 46, 34.
template <class T, bool GLU>
hipError_t launch_fp8_t(const ProductArgs& a, hipStream_t s) {
    if (!a.aligned) {
        const int64_t blocks = (((int64_t)a.N + 15) / 16) * (((int64_t)a.M + 15) / 16);
        return blocks <= (GLU ? 256 : 512) ? launch_skinny<T, GLU>(a, s) : launch_any<T, GLU, false>(a, s);
    }
    const int64_t b32 = ((GLU ? 2ll * a.N : a.N) + 31) / 32;   // blocks of 32 weight rows
    const int pieces = std::max(1, (a.K + 127) / 128);
    const auto by = [&](int rows) { return ((int64_t)a.M + rows - 1) / rows; };
    // little to do: 16 weight rows and 16 of x a workgroup, up to 16 waves along
    // K (16 x 4096 x 14336: 11.6 us, 32 weight rows and four waves 12.8)
    if (b32 * by(16) < 256) {
        int w = 4;
        while (w < 16 && b32 * by(16) * w < 3000 && w < pieces) w *= 2;
        if constexpr (GLU) return launch_stream<T, 2, 1, 2, GLU, false>(a, std::min(w, 8), s);
        else return launch_stream<T, 1, 1, 2, GLU, false>(a, w, s);
    }
    const TileChoice tile = choose_tile<T, GLU, false>(a);
    // P pieces a wave: a workgroup alone on its CU, then what each further one adds
    const double P = (pieces + 3) / 4;
    const double l1 = b32 * by(16) / 256.0, l2 = b32 * by(32) / 256.0, l4 = b32 * by(64) / 256.0;
    const double t1 = (kFull<T> ? 1.07 : 1.0) * (3.6 + 0.32 * P) * (1.0 + 0.6 * std::max(0.0, l1 - 1.0));
    const double t2 = (kFull<T> ? 1.1 : 1.0) * (3.6 + 0.37 * P) * (1.0 + 0.85 * std::max(0.0, l2 - 1.0));
    const double t4 = (kFull<T> ? 1.25 : 1.0) * (5.4 + 0.51 * P) * ceil(l4);
    const double least = std::min(std::min(t1, t2), t4);
    // (a grid has at most 65535 blocks of rows)
    if (tile.time <= least || by(16) > 65535) return launch_tiles<T, GLU, false>(a, tile.tile, s);
    const int w = std::min(4, pieces);
    if (t1 == least) return launch_stream<T, 2, 1, 2, GLU, false>(a, w, s);
    if (t2 == least) return launch_stream<T, 2, 2, 2, GLU, false>(a, w, s);
    return launch_stream<T, 2, 4, 2, GLU, false>(a, w, s);
}

}  // namespace
}  // namespace pw
