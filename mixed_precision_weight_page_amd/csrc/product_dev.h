// Products with an epilogue beyond kernels_linear.hip: of e4m3 operands with
// fp32 scales, and grouped by expert with ragged sizes (16-bit or e4m3).
//
// e4m3: y = f(sum over blocks b of 128 K values of xs[t, b] ws[n / 128, b]
// (sum over b's values of xq wq) + bias) + residual. The inner sum runs on the
// matrix cores (16 x 16 x 128 products, fp32), from zero for each block; its
// result times both scales is added to the fp32 sum in vector registers.
// Measured: an 8-bit matrix instruction (this one, and the 16 x 16 x 32 and 32 x 32 x
// 64 ones alike) cuts each product off, towards zero, at 2^(E - 13), E the
// largest sum of the two codes' exponents (-6 for those below 2^-6) among the
// eight products, not zero, whose K values share 8 bytes. That is 1.5e-5 of the
// norm of the sum for normally distributed operands, where e4m3 has rounded
// each by up to 2^-4 (rows with a few channels twenty times the others: 3.5e-5).
// A 16-bit y rounds by far more; for an fp32 y the same kernels run with
// E4M3Full operands, whose products are exact, on 16-bit instructions of half
// the rate.
// With SwiGLU the gate and the up rows have row blocks of their own, each from
// its first row.
//
// Grouped: rows offsets[e] .. offsets[e + 1] - 1 of x by the weights of expert
// e. The offsets are read on the device only: a launch has workgroups for any
// split of the rows, each finds its tile by a scan over the experts, and the
// ones left over end. Offsets are taken within [0, M] and a group not before
// its start, so that no value of theirs reaches outside the tensors.
#pragma once

#include "linear_dev.h"

namespace pw {
namespace {

struct E4M3 {   // one OCP e4m3 value
    uint8_t bits;
};
struct E4M3Full {   // the same, for products of which nothing may be lost
    uint8_t bits;
};
template <class T>
constexpr bool kFull = std::is_same<T, E4M3Full>::value;
template <class T>
constexpr bool kEight = std::is_same<T, E4M3>::value || kFull<T>;
template <class T>
constexpr int kStage = 128 / (int)sizeof(T);   // K values per step: 128-byte rows in LDS

typedef int i32x8 __attribute__((ext_vector_type(8)));

// 16 x 16 x 128 product of e4m3 rows from zero; lane (r, g) holds 32 K-slots
// of row r of a and of column r of b (the same slots in both), and gets rows
// 4 g .. 4 g + 3 of column r. Without scale operands: the unscaled form.
__device__ __forceinline__ f32x4 mma8(const u32x4& a0, const u32x4& a1, const u32x4& b0, const u32x4& b1) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
        __builtin_bit_cast(i32x8, __builtin_shufflevector(a0, a1, 0, 1, 2, 3, 4, 5, 6, 7)),
        __builtin_bit_cast(i32x8, __builtin_shufflevector(b0, b1, 0, 1, 2, 3, 4, 5, 6, 7)), f32x4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// 32 codes as fp16, which holds every e4m3 value (and their products are exact
// in fp32): 8 to each of four 16 x 16 x 32 products, which together cover a
// lane's K-slots as mma8 does.
struct Halves {
    u32x4 v[4];
};
__device__ __forceinline__ Halves halves_of(const u32x4& a0, const u32x4& a1) {
    Halves h;
#if defined(__HIP_DEVICE_COMPILE__)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t word = i < 4 ? a0[i & 3] : a1[i & 3];
        h.v[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, false));
        h.v[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(word, 1.0f, true));
    }
#endif
    return h;
}

// 16 bytes from p, of any alignment; left: bytes of the row from p on, zeros
// past them
typedef unsigned int u32x4_byte __attribute__((ext_vector_type(4), aligned(1)));
typedef unsigned int u32x4_word __attribute__((ext_vector_type(4), aligned(4)));
__device__ __forceinline__ u32x4 load_bytes(const uint8_t* p, int left) {
    if (left >= 16) return *reinterpret_cast<const u32x4_byte*>(p);
    u32x4 u = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < left) u[i >> 2] |= (uint32_t)p[i] << (8 * (i & 3));
    return u;
}

// acc += (fw fx^T) f, block by block; f[h][j]: the scales' product for token
// block j and the gate (or only) and up rows.
template <class T, int RB, int MB, bool GLU>
__device__ __forceinline__ void scaled_blocks(f32x4 (&acc)[RB][MB], const u32x4 (&fw)[RB][2], const u32x4 (&fx)[MB][2],
                                              const float (&f)[2][MB]) {
    auto join = [&](int i, int j, const f32x4& p) {
        const float s = f[GLU ? i & 1 : 0][j];
        acc[i][j] = __builtin_elementwise_fma(p, f32x4{s, s, s, s}, acc[i][j]);
    };
    if constexpr (kFull<T>) {
        Halves x[MB];
#pragma unroll
        for (int j = 0; j < MB; ++j) x[j] = halves_of(fx[j][0], fx[j][1]);
#pragma unroll
        for (int i = 0; i < RB; ++i) {
            const Halves w = halves_of(fw[i][0], fw[i][1]);
            f32x4 p[MB];
#pragma unroll
            for (int j = 0; j < MB; ++j) p[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int j = 0; j < MB; ++j) p[j] = mma<_Float16>(w.v[q], x[j].v[q], p[j]);
#pragma unroll
            for (int j = 0; j < MB; ++j) join(i, j, p[j]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) join(i, j, mma8(fw[i][0], fw[i][1], fx[j][0], fx[j][1]));
    }
}

// ---- groups ----

struct Group {
    int e, start, cnt;   // expert, its first row, its rows
};

// Experts base .. base + 63, one a lane.
__device__ __forceinline__ Group lane_group(const ProductArgs& a, int base) {
    const int e = base + (threadIdx.x & 63);
    Group g{e, 0, 0};
    if (e < a.E) {
        g.start = min(max(a.offsets[e], 0), a.M);
        g.cnt = max(min(a.offsets[e + 1], a.M), g.start) - g.start;
    }
    return g;
}
__device__ __forceinline__ int scan_lanes(int v) {   // inclusive
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// This workgroup's tile of BM rows: its group, the tile within it and the
// column tile; false if there is none. Each XCD takes one contiguous eighth
// of the tiles: expert by expert, the row tiles of an expert (in bands of
// kBand) fastest.
template <int BM>
__device__ __forceinline__ bool group_tile(const ProductArgs& a, int tn, Group& g, int& nt, int& mt) {
    int total = 0;
    for (int base = 0; base < a.E; base += 64) {
        int t = (lane_group(a, base).cnt + BM - 1) / BM;
#pragma unroll
        for (int d = 32; d; d >>= 1) t += __shfl_xor(t, d);
        total += t;
    }
    total = __builtin_amdgcn_readfirstlane(total);
    const int64_t used = (int64_t)tn * total, share = (used + 7) >> 3;
    const int64_t at = blockIdx.x >> 3, li = (int64_t)(blockIdx.x & 7) * share + at;
    if (at >= share || li >= used) return false;
    const int row_tile = (int)(li / tn);   // an expert's tiles lie together: the expert is that of any of them
    int before = 0;
    for (int base = 0; base < a.E; base += 64) {
        const Group mine = lane_group(a, base);
        const int t = (mine.cnt + BM - 1) / BM;
        const int upto = before + scan_lanes(t);
        const uint64_t hit = __ballot(upto > row_tile);
        if (hit) {
            const int l = __ffsll((unsigned long long)hit) - 1;
            g.e = base + l;
            g.start = __builtin_amdgcn_readlane(mine.start, l);
            g.cnt = __builtin_amdgcn_readlane(mine.cnt, l);
            const int tiles = (g.cnt + BM - 1) / BM;
            const int64_t first = (int64_t)(__builtin_amdgcn_readlane(upto, l) - tiles) * tn;
            const int in_e = (int)(li - first);
            const int band = in_e / (kBand * tn), in = in_e - band * kBand * tn;
            const int wide = min(kBand, tiles - band * kBand);
            nt = in / wide;
            mt = band * kBand + in - nt * wide;
            return true;
        }
        before = __builtin_amdgcn_readlane(upto, 63);
    }
    return false;
}

// The arguments of a group's own product: its rows (unless they are gathered)
// and its expert's weights.
template <class T>
__device__ __forceinline__ void narrow(ProductArgs& a, const Group& g, bool glu) {
    const int64_t ob = a.out_dtype == PW_F32 ? 4 : 2, rows = glu ? 2 * (int64_t)a.N : a.N;
    if (a.rows) {
        a.rows += g.start;
    } else {
        a.x = reinterpret_cast<const uint8_t*>(a.x) + (int64_t)g.start * a.ldx * (int64_t)sizeof(T);
        if (kEight<T>) a.xs += (int64_t)g.start * a.xs_row;
    }
    a.w = reinterpret_cast<const uint8_t*>(a.w) + g.e * a.w_expert * (int64_t)sizeof(T);
    if (kEight<T>) a.ws += g.e * a.ws_expert;
    if (a.bias) a.bias += g.e * rows;
    if (a.residual) a.residual = reinterpret_cast<const uint8_t*>(a.residual) + (int64_t)g.start * a.ldr * ob;
    a.y = reinterpret_cast<uint8_t*>(a.y) + (int64_t)g.start * a.ldy * ob;
    a.M = g.cnt;
}

// The row of x behind row m of the product, -1 if there is none.
template <bool GRP>
__device__ __forceinline__ int x_row(const ProductArgs& a, int64_t m) {
    if (m >= a.M) return -1;
    if (!GRP || !a.rows) return (int)m;
    const int r = a.rows[m];
    return r >= 0 && r < a.x_rows ? r : -1;
}

// Row block of the scales of weight row n (of the gate's or the up half).
template <bool GLU>
__device__ __forceinline__ const float* scale_row(const ProductArgs& a, int n, int half) {
    return a.ws + (int64_t)((n >> 7) + (GLU ? half * ((a.N + 127) >> 7) : 0)) * a.ws_row;
}

// ---- rows of any alignment ----

// kTile weight rows x kTile rows of x (64 or 128), WN x WM waves, K in steps
// of 128 bytes through two LDS buffers; the rows go through registers, loaded two steps
// ahead. A row's 16-byte chunk c lies at position c ^ (row % 8). Loads start at
// the 4-byte word of a chunk's first byte (a wave's 1 KB from there takes a CU
// about 34 cycles, from an odd byte 55 to 130), and the bytes are moved on the
// way to LDS: the word behind a chunk is the next lane's first, that behind a
// step's last chunk is loaded too. (Against loads from the bytes themselves: 8192
// x 4096 x 4095 e4m3 449 -> 397 us, 1000 x 2000 x 2001 20.6 -> 16.1, 1400 x 316 x
// 4013 27.6 -> 22.0, 777 x 1001 x 700 10.2 -> 9.2, and 11.6 with gelu, bias and
// residual; 4096 rows of 64 experts the same. Codes with more bits set draw more
// power and take longer: 8192 x 4096 x 4095 451.)
constexpr int kAnyWN = 2, kAnyWM = 4;
template <class T, int kTile, bool GLU, bool GRP>
__global__ __launch_bounds__(64 * kAnyWN * kAnyWM) void product_any_kernel(ProductArgs a) {
    constexpr int kWaves = kAnyWN * kAnyWM, kRows = 2 * kTile, kB = (int)sizeof(T);
    constexpr int RB = kTile / 16 / kAnyWN, MB = kTile / 16 / kAnyWM, Q = kRows / 8 / kWaves;
    constexpr int kOutN = GLU ? kTile / 2 : kTile;
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int r = lane & 15, g = lane >> 4;
    int nt, mt;
    if constexpr (GRP) {
        Group grp;
        if (!group_tile<kTile>(a, (a.N + kOutN - 1) / kOutN, grp, nt, mt)) return;
        narrow<T>(a, grp, GLU);
    } else {
        if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + kTile - 1) / kTile, nt, mt)) return;
    }
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * kTile;
    const int crow = lane >> 3, chunk = lane & 7;
    const bool gather = GRP && a.rows;
    const uint8_t* from[2];   // the first weight row (gate and up rows are different waves'), the first row of x
    from[0] = reinterpret_cast<const uint8_t*>(a.w) + (n0 + (GLU && (wave & 2) ? (int64_t)a.N : 0)) * a.ldw * kB;
    from[1] = reinterpret_cast<const uint8_t*>(a.x) + (gather ? 0 : m0 * a.ldx * kB);
    uint32_t off[Q];   // of this lane's bytes behind the word that holds from's
#pragma unroll
    for (int j = 0; j < Q; ++j) {
        const int lr = 8 * (kWaves * j + wave) + crow, of_x = 2 * j >= Q;
        int64_t at = -1;
        if (!of_x) {
            const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
            if (n0 + wr < a.N) at = wr * a.ldw;
        } else {
            const int xr = x_row<GRP>(a, m0 + lr - kTile);
            if (xr >= 0) at = (gather ? xr : lr - kTile) * a.ldx;
        }
        off[j] = at >= 0 ? (uint32_t)(at * kB) + 16 * chunk + ((uint32_t)(uintptr_t)from[of_x] & 3) : kOutside;
    }
    const auto rw = make_rsrc(from[0] - ((uintptr_t)from[0] & 3)), rx = make_rsrc(from[1] - ((uintptr_t)from[1] & 3));
    const int S = (a.K + kStage<T> - 1) / kStage<T>;
    const int row_bytes = a.K * kB;
    struct Rows {
        u32x4 at[Q];
        uint32_t behind[Q];   // of the last chunk
    };
    Rows even, odd;   // of an even and of an odd step
    auto fetch = [&](int s, Rows& to) {
        if ((s + 1) * 128 <= row_bytes) {
#pragma unroll
            for (int j = 0; j < Q; ++j) {
                const uint32_t word = off[j] & ~3u;
                to.at[j] = load_words<u32x4>(2 * j < Q ? rw : rx, word, s * 128);
                to.behind[j] = load_words<uint32_t>(2 * j < Q ? rw : rx, chunk == 7 && word != off[j] ? word + 16 : kOutside, s * 128);
            }
            return;
        }
        const int left = row_bytes - (s * 128 + 16 * chunk);   // the last, partial step as it lies
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const uint8_t* first = from[2 * j < Q ? 0 : 1];
            to.at[j] = off[j] != kOutside && left > 0 ? load_bytes(first - ((uintptr_t)first & 3) + off[j] + s * 128, left) : u32x4{0u, 0u, 0u, 0u};
            to.behind[j] = 0u;
        }
    };
    auto settle = [&](int s, const Rows& rows) {   // registers to LDS
        u32x4* dst = reinterpret_cast<u32x4*>(tile_lds + (s & 1) * kRows * 64) + crow * 8 + (chunk ^ crow);
        const bool whole = (s + 1) * 128 <= row_bytes;
#pragma unroll
        for (int j = 0; j < Q; ++j) {
            const u32x4 v = rows.at[j];
            uint32_t next = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v[0], 0x101, 0xf, 0xf, true);   // row_shl:1, the next lane's
            if (chunk == 7) next = rows.behind[j];
            const uint32_t by = whole ? off[j] & 3 : 0u;
            dst[(kWaves * j + wave) * 64] = u32x4{__builtin_amdgcn_alignbyte(v[1], v[0], by), __builtin_amdgcn_alignbyte(v[2], v[1], by),
                                                  __builtin_amdgcn_alignbyte(v[3], v[2], by), __builtin_amdgcn_alignbyte(next, v[3], by)};
        }
    };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wn = wave % kAnyWN, wm = wave / kAnyWN;
    // scales: of this lane's rows of x (0 where there is none), of the wave's
    // weight rows
    const float* xs[MB];
    const float *wg = nullptr, *wu = nullptr;
    if constexpr (kEight<T>) {
#pragma unroll
        for (int j = 0; j < MB; ++j) {
            const int row = x_row<GRP>(a, m0 + (wm * MB + j) * 16 + r);
            xs[j] = row < 0 ? nullptr : a.xs + (int64_t)row * a.xs_row;
        }
        const int n = n0 + wn * (GLU ? 8 : 16) * RB;
        wg = scale_row<GLU>(a, min(n, a.N - 1), 0);
        wu = scale_row<GLU>(a, min(n, a.N - 1), 1);
    }
    auto step = [&](int s, Rows& mine, const Rows& other) {
        __syncthreads();   // step s is in LDS; everyone is done with the other buffer
        if (s + 2 < S) fetch(s + 2, mine);
        const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + (s & 1) * kRows * 64) + r * 8;
        u32x4 fw[RB][2], fx[MB][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int pos = (4 * h + g) ^ (r & 7);
#pragma unroll
            for (int j = 0; j < MB; ++j) fx[j][h] = base[(kTile + (wm * MB + j) * 16) * 8 + pos];
#pragma unroll
            for (int i = 0; i < RB; ++i) fw[i][h] = base[(wn * RB + i) * 128 + pos];
        }
        if constexpr (kEight<T>) {
            const float sg = wg[s * a.ws_block], su = GLU ? wu[s * a.ws_block] : 0.0f;
            if constexpr (kFull<T>) {
                float f[2][MB];
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    const float sx = xs[j] ? xs[j][s * a.xs_block] : 0.0f;
                    f[0][j] = sx * sg;
                    f[1][j] = sx * su;
                }
                scaled_blocks<T, RB, MB, GLU>(acc, fw, fx, f);
            } else {
                // (a block of rows of x at a time: 8192 x 4096 x 4095 449 us,
                // as scaled_blocks goes 472)
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    const float sx = xs[j] ? xs[j][s * a.xs_block] : 0.0f;
#pragma unroll
                    for (int i = 0; i < RB; ++i) {
                        const float f = sx * (GLU && (i & 1) ? su : sg);
                        const f32x4 p = mma8(fw[i][0], fw[i][1], fx[j][0], fx[j][1]);
                        acc[i][j] = __builtin_elementwise_fma(p, f32x4{f, f, f, f}, acc[i][j]);
                    }
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < RB; ++i)
#pragma unroll
                    for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[i][h], fx[j][h], acc[i][j]);
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
    static_assert(kWaves * out_stage_floats<RB>() * 4 <= 2 * kRows * 128, "the sums fit the buffers");
    put_tile<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

// ---- 16-byte aligned rows: copies straight to LDS ----

// What a tile of BM rows of x and BN weight rows (with SwiGLU blocks of 16
// gate and up rows in turn) copies for each step of 128 bytes: a wave's
// copy covers 8 rows, 16 bytes a lane, row % 8 = lane / 8, chunk c of a row at
// position c ^ (row % 8), so that operand reads fall on different banks.
// Steps past the last, rows and columns outside read zeros (out of the
// buffer's bounds, no memory is touched).
template <class T, int BM, int BN, int kWaves, bool GLU, bool GRP>
struct TileCopies {
    static constexpr int kB = (int)sizeof(T);
    static constexpr int QW = BN / 8 / kWaves, QX = BM / 8 / kWaves;   // copies of a wave and step
    static_assert(BN % (8 * kWaves) == 0 && BM % (8 * kWaves) == 0, "whole copies");
    static_assert(kWaves % 4 == 0, "a wave's weight rows are of one kind");
    __amdgpu_buffer_rsrc_t rw, rx;
    uint32_t off[QW + QX];
    int row_bytes, in_row;   // of K values; this lane's byte in a step
    int wave;

    __device__ __forceinline__ TileCopies(const ProductArgs& a, int n0, int wave_) : row_bytes(a.K * kB), wave(wave_) {
        const int lane = threadIdx.x & 63, crow = lane >> 3, chunk = (lane & 7) ^ crow;
        in_row = 16 * chunk;
        const uint8_t* wbase = reinterpret_cast<const uint8_t*>(a.w) + (int64_t)n0 * a.ldw * kB;
        rw = make_rsrc(wbase + (GLU && (wave & 2) ? (int64_t)a.N * a.ldw * kB : 0));
#pragma unroll
        for (int j = 0; j < QW; ++j) {
            const int lr = (j * kWaves + wave) * 8 + crow;
            const int wr = GLU ? (lr >> 5) * 16 + (lr & 15) : lr;
            off[j] = n0 + wr < a.N ? (uint32_t)(wr * a.ldw * kB) + in_row : kOutside;
        }
    }
    // the rows of x, after the first weights are on their way: rows that are
    // gathered are looked up first
    __device__ __forceinline__ void rows_of_x(const ProductArgs& a, int64_t m0) {
        const int crow = (threadIdx.x & 63) >> 3;
        const bool gather = GRP && a.rows;
        rx = make_rsrc(reinterpret_cast<const uint8_t*>(a.x) + (gather ? 0 : m0 * a.ldx * kB));
#pragma unroll
        for (int j = 0; j < QX; ++j) {
            const int lr = (j * kWaves + wave) * 8 + crow;
            const int row = x_row<GRP>(a, m0 + lr);
            off[QW + j] = row >= 0 ? (uint32_t)((gather ? row : lr) * a.ldx * kB) + in_row : kOutside;
        }
    }
    // the q-th of them; dst: the slot's weight rows, then its rows of x
    __device__ __forceinline__ void one(int q, int s, uint16_t* dst) const {
        const bool in = s * 128 + in_row < row_bytes;
        copy_to_lds(q < QW ? rw : rx, dst + (q * kWaves + wave) * 512,
                    in ? off[q] : kOutside, s * 128 < row_bytes ? s * 128 : 0);
    }
    __device__ __forceinline__ void operator()(int s, uint16_t* dst) const {
#pragma unroll
        for (int q = 0; q < QW + QX; ++q) one(q, s, dst);
    }
};

// The scales of a tile and step, one 4-byte copy a wave: BM of the rows of x
// (64 a wave, from wave 0 on), then by the next wave those of the weight rows
// of each of WN columns of waves (gate's, then up's); the other waves' copies
// touch nothing and land past them. kScaleFloats in all.
template <int BM, int BN, int WN, int kWaves, bool GLU, bool GRP>
struct ScaleCopies {
    static constexpr int kX = BM / 64;
    static_assert(kX < kWaves && BM % 64 == 0, "a wave for the weights' scales");
    static constexpr int kFloats = 64 * kWaves;
    __amdgpu_buffer_rsrc_t rs;
    uint32_t off;
    int step, steps, wave;

    __device__ __forceinline__ ScaleCopies(const ProductArgs& a, int n0, int64_t m0, int S, int wave_) : steps(S), wave(wave_) {
        const int lane = threadIdx.x & 63;
        const bool gather = GRP && a.rows;
        off = kOutside;
        rs = make_rsrc(wave < kX ? a.xs + (gather ? 0 : m0 * a.xs_row) : a.ws);
        step = (int)((wave < kX ? a.xs_block : a.ws_block) * 4);
        if (wave < kX) {
            const int lr = 64 * wave + lane, row = x_row<GRP>(a, m0 + lr);
            if (row >= 0) off = (uint32_t)((gather ? row : lr) * a.xs_row) * 4u;
        } else {
            const int n = n0 + (lane % WN) * (GLU ? BN / WN / 2 : BN / WN);
            if (wave == kX && lane < (GLU ? 2 : 1) * WN && n < a.N) off = (uint32_t)(scale_row<GLU>(a, n, lane / WN) - a.ws) * 4u;
        }
    }
    __device__ __forceinline__ void operator()(int s, uint16_t* dst) const {
        touch_to_lds(rs, dst + wave * 128, s < steps ? off : kOutside, s < steps ? s * step : 0);
    }
};

// BN weight rows x BM rows of x, WN x WM waves, K in steps of 128 bytes
// through a ring of D LDS slots, one barrier a step, so that D - 2 steps'
// copies are on their way while one is multiplied. Bound by those copies, and
// by the end of a tile, which nothing overlaps: 24576 rows of 64 experts with
// popularity ~ rank^-0.3, 1408 -> 4096 bf16 400 us, 710 TFLOP/s, with an fp32 y 425
// (384 rows each 358 and 378, with one expert's weights for all 327).
template <class T, int BM, int BN, int WM, int WN, int D, bool GLU, bool GRP>
__global__ __launch_bounds__(64 * WM * WN) void product_ring_kernel(ProductArgs a) {
    constexpr int kWaves = WM * WN, kRows = BN + BM;
    constexpr int RB = BN / WN / 16, MB = BM / WM / 16;   // blocks of a wave's tile
    constexpr int kOutN = GLU ? BN / 2 : BN;
    typedef TileCopies<T, BM, BN, kWaves, GLU, GRP> Copies;
    typedef ScaleCopies<BM, BN, WN, kWaves, GLU, GRP> Scales;
    constexpr int kSlot = kRows * 64 + (kEight<T> ? Scales::kFloats * 2 : 0);   // in 16-bit units
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    int nt, mt;
    if constexpr (GRP) {
        Group grp;
        if (!group_tile<BM>(a, (a.N + kOutN - 1) / kOutN, grp, nt, mt)) return;
        narrow<T>(a, grp, GLU);
    } else {
        if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + BM - 1) / BM, nt, mt)) return;
    }
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * BM;
    const int S = (a.K + kStage<T> - 1) / kStage<T>;
    Copies copies(a, n0, wave);
    copies.rows_of_x(a, m0);
    auto copy = [&](int s, int slot) { copies(s, tile_lds + slot * kSlot); };
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const int wn = wave % WN, wm = wave / WN;
    constexpr int kEach = Copies::QW + Copies::QX + (kEight<T> ? 1 : 0);   // copies a step
    auto loop = [&](auto scale) {
#pragma unroll
        for (int j = 0; j < D - 1; ++j) {
            copy(j, j);
            if constexpr (kEight<T>) scale(j, j);
            keep_order();
        }
        int slot = 0;
        for (int s = 0; s < S; ++s) {
            // step s is whole (this wave's part, then everyone's), and everyone
            // has read the slot before it, which takes step s + D - 1
            asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kEach * (D - 2)) : "memory");
            const int next = slot == 0 ? D - 1 : slot - 1;
            copy(s + D - 1, next);
            if constexpr (kEight<T>) scale(s + D - 1, next);
            keep_order();
            const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + slot * kSlot) + r * 8;
            u32x4 fw[RB][2], fx[MB][2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pos = (4 * h + g) ^ (r & 7);
#pragma unroll
                for (int j = 0; j < MB; ++j) fx[j][h] = base[(BN + (wm * MB + j) * 16) * 8 + pos];
#pragma unroll
                for (int i = 0; i < RB; ++i) fw[i][h] = base[(wn * RB + i) * 128 + pos];
            }
            if constexpr (kEight<T>) {
                const float* sc = reinterpret_cast<const float*>(tile_lds + slot * kSlot + kRows * 64);
                const float sg = sc[BM + wn], su = GLU ? sc[BM + WN + wn] : 0.0f;
                float f[2][MB];
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    const float sx = sc[(wm * MB + j) * 16 + r];
                    f[0][j] = sx * sg;
                    f[1][j] = sx * su;
                }
                scaled_blocks<T, RB, MB, GLU>(acc, fw, fx, f);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[i][h], fx[j][h], acc[i][j]);
            }
            slot = slot + 1 == D ? 0 : slot + 1;
        }
    };
    if constexpr (kEight<T>) {
        const Scales scales(a, n0, m0, S, wave);
        loop([&](int s, int slot) { scales(s, tile_lds + slot * kSlot + kRows * 64); });
    } else {
        loop(0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();   // every wave is done with the slots
    static_assert(kWaves * out_stage_floats<RB>() * 4 <= D * kSlot * 2, "the sums fit the slots");
    put_tile<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

// Large products: 256 weight rows x 256 rows of x, 8 waves (2 x 4) of 128 x 64
// each, K in steps of 128 bytes through two LDS slots. The two waves of a
// SIMD take turns: half a step is a phase of operand reads and a phase of
// matrix instructions, and waves 4 .. 7 run one phase behind waves 0 .. 3, so
// that one wave of each SIMD multiplies while the other reads. Phases end at
// barriers. Step s is read in phases 4 s .. 4 s + 3; the other slot takes the
// copies of step s + 1 meanwhile, each wave's started among its first matrix
// instructions of the step and waited for by the end of phase 4 s + 3. A
// half step is half of K for 16-bit operands; for e4m3 (whose instruction
// takes the whole step) half of the weight rows.
//
// Bound by the matrix cores and the clock they leave: 8192 x 8192 x 8192 e4m3
// 475 to 510 us, 2.2 to 2.3 PFLOP/s. The last tile of a group (or of all rows)
// has only the rows it needs, in 64s, but 128 of them take three quarters of
// the time of 256 (64 experts, 4096 -> 2 x 1408 e4m3, 256, 384 and 512 rows
// each: 239, 383, 432 us; with one expert's weights for all, which stay in
// the caches, 176, 325, 366). Weights asked for two to four steps early, as
// in linear_phased_kernel, gained nothing: 382, 24576 ragged rows, became
// 391 with a 128-byte row part at a time, 391 and 400 with two neighbouring
// ones; 16-bit 399, became 409.
template <class T, int MB, bool GLU, bool GRP>
__device__ __forceinline__ void phased_tile(const ProductArgs& a, uint16_t* tile_lds, int nt, int mt) {
    constexpr int RB = 8, BN = 256, BM = 64 * MB, kRows = BN + BM;
    constexpr int kOutN = GLU ? BN / 2 : BN;
    typedef TileCopies<T, BM, BN, 8, GLU, GRP> Copies;
    typedef ScaleCopies<BM, BN, 2, 8, GLU, GRP> Scales;
    constexpr int kSlot = kRows * 64 + (kEight<T> ? Scales::kFloats * 2 : 0);
    constexpr int kEach = Copies::QW + Copies::QX + (kEight<T> ? 1 : 0);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, g = lane >> 4;
    const int n0 = nt * kOutN;
    const int64_t m0 = (int64_t)mt * 256;
    const int S = (a.K + kStage<T> - 1) / kStage<T>;
    Copies copies(a, n0, wave);
#pragma unroll
    for (int q = 0; q < Copies::QW; ++q) copies.one(q, 0, tile_lds);
    const int wn = wave & 1, wm = wave >> 1;
    const bool late = wave >= 4;
    copies.rows_of_x(a, m0);
    f32x4 acc[RB][MB];
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    auto loop = [&](auto scale) {
        auto copy = [&](int s) {
            copies(s, tile_lds + (s & 1) * kSlot);
            if constexpr (kEight<T>) scale(s);
            keep_order();
        };
#pragma unroll
        for (int q = Copies::QW; q < Copies::QW + Copies::QX; ++q) copies.one(q, 0, tile_lds);
        if constexpr (kEight<T>) scale(0);
        keep_order();
        asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
        if (late) asm volatile("s_barrier" ::: "memory");
        if constexpr (kEight<T>) {
            // Block i of the wave's 8 MB: its sum over the step's K values
            // goes to p[i % 4] and joins the whole three blocks later, a
            // half's last three in the next phase: 11 other instructions
            // have to lie between (two blocks later the compiler adds up to
            // as many idle ones, and the matrix cores were busy 53% of the
            // time).
            constexpr int kLag = 3;
            constexpr int kHalf = RB / 2 * MB;   // blocks of half a step
            static_assert(kLag == 3 && kLag <= kHalf, "a half's last blocks");
            constexpr int kPer = (kEach + kHalf - 1) / kHalf;   // copies with each block of the first half
            f32x4 p[4] = {};
            float f[2][MB] = {};
            u32x4 fw[RB / 2][2], fx[MB][2];
            auto join = [&](int i) {
                const float v = f[GLU ? (i / MB) & 1 : 0][i % MB];
                f32x4& sum = acc[i / MB][i % MB];
                sum = __builtin_elementwise_fma(p[i & 3], f32x4{v, v, v, v}, sum);
                asm volatile("" : "+v"(sum));   // here, not where the sum is used next
            };
            for (int s = 0; s < S; ++s) {
                const uint16_t* slot = tile_lds + (s & 1) * kSlot;
                const u32x4* base = reinterpret_cast<const u32x4*>(slot) + r * 8;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float sg = 0.f, su = 0.f, sx[MB];
                    if (h == 0) {
                        const float* sc = reinterpret_cast<const float*>(slot + kRows * 64);
                        sg = sc[BM + wn];
                        if (GLU) su = sc[BM + 2 + wn];
#pragma unroll
                        for (int j = 0; j < MB; ++j) sx[j] = sc[(wm * MB + j) * 16 + r];
#pragma unroll
                        for (int j = 0; j < MB; ++j)
#pragma unroll
                            for (int q = 0; q < 2; ++q) fx[j][q] = base[(BN + (wm * MB + j) * 16) * 8 + ((4 * q + g) ^ (r & 7))];
                    }
#pragma unroll
                    for (int i = 0; i < RB / 2; ++i)
#pragma unroll
                        for (int q = 0; q < 2; ++q) fw[i][q] = base[(wn * RB + h * (RB / 2) + i) * 128 + ((4 * q + g) ^ (r & 7))];
                    // (one by one: as a loop they kept these sums in scratch
                    // memory, whose loads wait for every copy on its way)
                    join((h == 0 ? 2 : 1) * kHalf - 3);
                    join((h == 0 ? 2 : 1) * kHalf - 2);
                    join((h == 0 ? 2 : 1) * kHalf - 1);
                    if (h == 0) {
#pragma unroll
                        for (int j = 0; j < MB; ++j) {
                            f[0][j] = sx[j] * sg;
                            if (GLU) f[1][j] = sx[j] * su;
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                    if (h == 1 && late) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_setprio(1);
#pragma unroll
                    for (int k = 0; k < kHalf; ++k) {
                        const int i = kHalf * h + k;
                        p[i & 3] = mma8(fw[k / MB][0], fw[k / MB][1], fx[k % MB][0], fx[k % MB][1]);
                        if (h == 0) {   // the next step's copies
                            uint16_t* dst = tile_lds + ((s + 1) & 1) * kSlot;
#pragma unroll
                            for (int q = k * kPer; q < (k + 1) * kPer; ++q) {
                                if (q < kEach - 1) copies.one(q, s + 1, dst);
                                if (q == kEach - 1) scale(s + 1);
                            }
                        }
                        if (k >= kLag) join(i - kLag);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    __builtin_amdgcn_s_setprio(0);
                    if (h == 1 && !late) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
            join(2 * kHalf - 3);
            join(2 * kHalf - 2);
            join(2 * kHalf - 1);
        } else {
            for (int s = 0; s < S; ++s) {
                const u32x4* base = reinterpret_cast<const u32x4*>(tile_lds + (s & 1) * kSlot) + r * 8;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    u32x4 fw[RB], fx[MB];
                    const int pos = (4 * h + g) ^ (r & 7);
#pragma unroll
                    for (int j = 0; j < MB; ++j) fx[j] = base[(BN + (wm * MB + j) * 16) * 8 + pos];
#pragma unroll
                    for (int i = 0; i < RB; ++i) fw[i] = base[(wn * RB + i) * 128 + pos];
                    __builtin_amdgcn_sched_barrier(0);
                    if (h == 1 && late) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                    __builtin_amdgcn_s_setprio(1);
                    if (h == 0) copy(s + 1);
#pragma unroll
                    for (int i = 0; i < RB; ++i)
#pragma unroll
                        for (int j = 0; j < MB; ++j) acc[i][j] = mma<T>(fw[i], fx[j], acc[i][j]);
                    if (h == 0) {
                        // copies among the matrix instructions
#pragma unroll
                        for (int q = 0; q < kEach; ++q) {
                            __builtin_amdgcn_sched_group_barrier(0x8, MB > 2 ? 2 : 1, 0);
                            __builtin_amdgcn_sched_group_barrier(0x10, 1, 0);
                        }
                    }
                    __builtin_amdgcn_s_setprio(0);
                    __builtin_amdgcn_sched_barrier(0);
                    if (h == 1 && !late) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                    asm volatile("s_barrier" ::: "memory");
                    __builtin_amdgcn_sched_barrier(0);
                }
            }
        }
    };
    if constexpr (kEight<T>) {
        const Scales scales(a, n0, m0, S, wave);
        loop([&](int s) { scales(s, tile_lds + (s & 1) * kSlot + kRows * 64); });
    } else {
        loop(0);
    }
    // the early waves' last barrier pairs with the late ones' last phase;
    // every copy has landed before the LDS is used again
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (!late) asm volatile("s_barrier" ::: "memory");
    __syncthreads();
    static_assert(8 * out_stage_floats<RB>() * 4 <= 2 * kSlot * 2, "the sums fit the slots");
    // stores that do not keep y in the caches, which a product of this size
    // leaves anyway (8192 x 4096 x 4096 with gelu, bias and residual 168 -> 158 us)
    put_tile<RB, MB, GLU, true>(a, acc, reinterpret_cast<float*>(tile_lds) + wave * out_stage_floats<RB>(),
                          n0 + wn * (GLU ? RB / 2 : RB) * 16, m0 + wm * MB * 16);
}

template <class T, bool GLU, bool GRP>
__global__ __launch_bounds__(512) void product_phased_kernel(ProductArgs a) {
    constexpr int kOutN = GLU ? 128 : 256;
    extern __shared__ __attribute__((aligned(16))) uint16_t tile_lds[];
    int nt, mt;
    if constexpr (GRP) {
        Group grp;
        if (!group_tile<256>(a, (a.N + kOutN - 1) / kOutN, grp, nt, mt)) return;
        narrow<T>(a, grp, GLU);
    } else {
        if (!tile_of((a.N + kOutN - 1) / kOutN, (a.M + 255) / 256, nt, mt)) return;
    }
    const int64_t left = a.M - (int64_t)mt * 256;
    if (left > 192) phased_tile<T, 4, GLU, GRP>(a, tile_lds, nt, mt);
    else if (left > 128) phased_tile<T, 3, GLU, GRP>(a, tile_lds, nt, mt);
    else if (left > 64) phased_tile<T, 2, GLU, GRP>(a, tile_lds, nt, mt);
    else phased_tile<T, 1, GLU, GRP>(a, tile_lds, nt, mt);
}

// Few rows of x: the weights' bytes bound it, they are streamed once. A
// workgroup has RB blocks of 16 weight rows (with SwiGLU the same RB / 2
// blocks of gate and of up rows) and blocks of 16 MB rows of x, K dealt to its
// waves in pieces of 128 bytes: a wave copies its own pieces (8 whole 128-byte
// row parts per instruction) into a ring of D slots that no other wave
// touches, so nothing but its own counter of copies is waited for, and what is
// in flight takes no registers. The waves' sums meet in LDS, in wave order.
// 16 x 14336 x 4096 e4m3 SwiGLU 28 us, 4.2 TB/s of weights; 512 rows of 128
// experts, 2048 -> 2 x 768 bf16 117 us, 5.3 TB/s.
// Grouped: blockIdx.y is the expert, its rows are taken 16 MB at a time.
template <class T, int RB, int MB, int D, bool GLU, bool GRP>
__global__ __launch_bounds__(kFull<T> && MB == 4 ? 256 : 1024) void product_stream_kernel(ProductArgs a) {
    extern __shared__ __attribute__((aligned(16))) uint16_t ring_lds[];   // [waves][D][slot]
    constexpr int kBlock = 16 * 64, kB = (int)sizeof(T);
    constexpr int kSC = kEight<T> ? 2 : 0;   // copies of scales, 64 floats each: of the rows of x, of the weights (gate, up)
    constexpr int kSlot = (RB + MB) * kBlock + kSC * 128;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
    const int r = lane & 15, g = lane >> 4;
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const int n0 = blockIdx.x * kRowsOut;
    if constexpr (GRP) {
        Group grp;
        grp.e = blockIdx.y;
        grp.start = min(max(a.offsets[grp.e], 0), a.M);
        grp.cnt = max(min(a.offsets[grp.e + 1], a.M), grp.start) - grp.start;
        if (grp.cnt == 0) return;
        narrow<T>(a, grp, GLU);
    }
    const bool gather = GRP && a.rows;
    const int crow = lane >> 3, chunk = (lane & 7) ^ crow;
    const uint8_t* wbase = reinterpret_cast<const uint8_t*>(a.w) + (int64_t)n0 * a.ldw * kB;
    const auto rw = make_rsrc(wbase), ru = make_rsrc(wbase + (GLU ? (int64_t)a.N * a.ldw * kB : 0));
    const int total = (a.K + kStage<T> - 1) / kStage<T>, row_bytes = a.K * kB;
    const int n = total > wave ? (total - wave + waves - 1) / waves : 0;
    uint16_t* ring = ring_lds + wave * D * kSlot;
    for (int m0 = GRP ? 0 : (int)blockIdx.y * 16 * MB; m0 < a.M; m0 += 16 * MB) {
        const auto rx = make_rsrc(reinterpret_cast<const uint8_t*>(a.x) + (gather ? 0 : (int64_t)m0 * a.ldx * kB));
        uint32_t off[RB + MB][2];
#pragma unroll
        for (int b = 0; b < RB + MB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int lr = 16 * (b >= RB ? b - RB : GLU ? b >> 1 : b) + 8 * h + crow;
                if (b < RB) {
                    off[b][h] = n0 + lr < a.N ? (uint32_t)(lr * a.ldw * kB) + 16 * chunk : kOutside;
                } else {
                    const int row = x_row<GRP>(a, m0 + lr);
                    off[b][h] = row >= 0 ? (uint32_t)((gather ? row : lr) * a.ldx * kB) + 16 * chunk : kOutside;
                }
            }
        // scales: this lane's of a row of x, and of the weights
        uint32_t xoff = kOutside, woff = kOutside;
        if constexpr (kEight<T>) {
            if (lane < 16 * MB) {
                const int row = x_row<GRP>(a, m0 + lane);
                if (row >= 0) xoff = (uint32_t)((gather ? row : lane) * a.xs_row) * 4u;
            }
            if (lane < (GLU ? 2 : 1)) woff = (uint32_t)(scale_row<GLU>(a, n0, lane) - a.ws) * 4u;
        }
        const auto rxs = make_rsrc(kEight<T> ? a.xs + (gather ? 0 : m0 * a.xs_row) : nullptr);
        const auto rws = make_rsrc(kEight<T> ? a.ws : nullptr);
        (void)rxs;
        (void)rws;
        auto copy = [&](int i, int slot) {   // piece i of this wave (past the last: zeros, no memory touched)
            const int s = wave + waves * i;
            const bool in = s * 128 + 16 * chunk < row_bytes;
            const int at = s * 128 < row_bytes ? s * 128 : 0;
            uint16_t* dst = ring + slot * kSlot;
#pragma unroll
            for (int b = 0; b < RB + MB; ++b)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    copy_to_lds(b >= RB ? rx : GLU && (b & 1) ? ru : rw, dst + b * kBlock + 512 * h, in ? off[b][h] : kOutside, at);
            if constexpr (kEight<T>) {
                const bool live = s < total;
                uint16_t* sc = dst + (RB + MB) * kBlock;
                const uint32_t xo = live && xoff != kOutside ? xoff + (uint32_t)(s * (int)(a.xs_block * 4)) : kOutside;
                const uint32_t wo = live && woff != kOutside ? woff + (uint32_t)(s * (int)(a.ws_block * 4)) : kOutside;
                touch_to_lds(rxs, sc, xo, 0);
                touch_to_lds(rws, sc + 128, wo, 0);
            }
            keep_order();
        };
        f32x4 acc[RB][MB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
            for (int j = 0; j < MB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < D; ++j) copy(j, j);
        int slot = 0;
        for (int i = 0; i < n; ++i) {
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"((2 * (RB + MB) + kSC) * (D - 1)) : "memory");
            const u32x4* base = reinterpret_cast<const u32x4*>(ring + slot * kSlot) + r * 8;
            u32x4 fw[RB][2], fx[MB][2];
            float f[2][MB];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int pos = (4 * h + g) ^ (r & 7);
#pragma unroll
                for (int b = 0; b < RB; ++b) fw[b][h] = base[b * 128 + pos];
#pragma unroll
                for (int b = 0; b < MB; ++b) fx[b][h] = base[(RB + b) * 128 + pos];
            }
            if constexpr (kEight<T>) {
                const float* sc = reinterpret_cast<const float*>(ring + slot * kSlot + (RB + MB) * kBlock);
                const float sg = sc[64], su = GLU ? sc[65] : 0.0f;
#pragma unroll
                for (int j = 0; j < MB; ++j) {
                    const float sx = sc[16 * j + r];
                    f[0][j] = sx * sg;
                    f[1][j] = sx * su;
                }
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read, before the slot is written again
            __builtin_amdgcn_sched_barrier(0);
            copy(i + D, slot);
            slot = slot + 1 == D ? 0 : slot + 1;
            if constexpr (kEight<T>) {
                scaled_blocks<T, RB, MB, GLU>(acc, fw, fx, f);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int p = 0; p < RB; ++p)
#pragma unroll
                        for (int q = 0; q < MB; ++q) acc[p][q] = mma<T>(fw[p][h], fx[q][h], acc[p][q]);
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();   // the rings are done with
        join_waves<RB, MB, GLU>(a, acc, reinterpret_cast<float*>(ring_lds), n0, m0);
        if constexpr (!GRP) return;
        __syncthreads();   // and so are the sums, before the next rows' copies
    }
}

// ---- launches ----

// Row tiles of bm rows that M rows in E groups may have, at most.
inline int64_t most_tiles(const ProductArgs& a, int bm, bool grouped) {
    if (!grouped) return (a.M + bm - 1) / bm;
    const int64_t groups = std::min<int64_t>(a.E, a.M);   // with a row
    return (a.M + groups * (bm - 1)) / bm;
}

template <class T, int kTile, bool GLU, bool GRP>
hipError_t launch_any_tile(const ProductArgs& a, hipStream_t s) {
    constexpr int kOutN = GLU ? kTile / 2 : kTile;
    const unsigned groups = groups_of((a.N + kOutN - 1) / kOutN * most_tiles(a, kTile, GRP), 64 * kAnyWN * kAnyWM);
    if (!groups) return hipErrorInvalidConfiguration;
    product_any_kernel<T, kTile, GLU, GRP><<<groups, 64 * kAnyWN * kAnyWM, 2 * 2 * kTile * 128, s>>>(a);
    return hipGetLastError();
}
template <class T, bool GLU, bool GRP>
hipError_t launch_any(const ProductArgs& a, hipStream_t s) {
    // larger tiles where they still fill the GPU (us with 64 x 64, 128 x 128: 8192
    // x 4096 x 4095 e4m3 436, 397; 2000 x 2000 x 2001, 256 large ones, 34, 25; 1600 x
    // 2048 x 1001, 208, 19, 16; 637 x 4049 x 6142, 160, 66, 70), and groups do (8192 rows
    // of 8 experts, 2047 -> 2048 bf16 186, 166; of 64, 4095 -> 1408 325, 375)
    const int64_t large = ((int64_t)a.M + 127) / 128 * (((GLU ? 2ll * a.N : a.N) + 127) / 128);
    if (large >= 192 && (!GRP || a.M / std::min(a.E, a.M) >= 1024)) return launch_any_tile<T, 128, GLU, GRP>(a, s);
    return launch_any_tile<T, 64, GLU, GRP>(a, s);
}

template <class T, int BM, int BN, int WM, int WN, int D, bool GLU, bool GRP>
hipError_t launch_ring(const ProductArgs& a, hipStream_t s) {
    constexpr int kOutN = GLU ? BN / 2 : BN;
    const unsigned groups = groups_of((a.N + kOutN - 1) / kOutN * most_tiles(a, BM, GRP), 64 * WM * WN);
    if (!groups) return hipErrorInvalidConfiguration;
    const size_t slot = (size_t)(BN + BM) * 128 + (kEight<T> ? 256 * WM * WN : 0);
    product_ring_kernel<T, BM, BN, WM, WN, D, GLU, GRP><<<groups, 64 * WM * WN, D * slot, s>>>(a);
    return hipGetLastError();
}

template <class T, bool GLU, bool GRP>
hipError_t launch_phased(const ProductArgs& a, hipStream_t s) {
    constexpr int kOutN = GLU ? 128 : 256;
    const unsigned groups = groups_of((a.N + kOutN - 1) / kOutN * most_tiles(a, 256, GRP), 512);
    if (!groups) return hipErrorInvalidConfiguration;
    const size_t slot = (size_t)512 * 128 + (kEight<T> ? 256 * 8 : 0);
    product_phased_kernel<T, GLU, GRP><<<groups, 512, 2 * slot, s>>>(a);
    return hipGetLastError();
}

template <class T, int RB, int MB, int D, bool GLU, bool GRP>
hipError_t launch_stream(const ProductArgs& a, int waves, hipStream_t s) {
    constexpr int kRowsOut = 16 * (GLU ? RB / 2 : RB);
    const dim3 grid((unsigned)((a.N + kRowsOut - 1) / kRowsOut), (unsigned)(GRP ? a.E : (a.M + 16 * MB - 1) / (16 * MB)));
    if (!groups_of(grid.x, 64 * waves)) return hipErrorInvalidConfiguration;
    const size_t slot = (RB + MB) * 2048 + (kEight<T> ? 512 : 0);
    const size_t lds = std::max((size_t)waves * D * slot, (size_t)waves * RB * MB * 1024);
    product_stream_kernel<T, RB, MB, D, GLU, GRP><<<grid, 64 * waves, lds, s>>>(a);
    return hipGetLastError();
}

// The tile whose workgroups take least, by times measured (us; S steps of K
// over a CU's one or two workgroups): small tiles fill the GPU and have the
// shorter steps, large ones read less per product. 1000 x 2048 x 2048 bf16: 18
// us with 64 x 64 tiles, 22 with 128 x 128, 48 with 256 x 256; 8192 rows of 8
// experts, 4096 -> 2048 bf16: 262, 197, 218, and 186 with 128 rows x 256; in
// e4m3 158, 96 (two workgroups on a CU), 113; 24576 rows of 64 experts, 4096
// -> 2816 e4m3: 770, 470, 435; of one: 4096 -> 4096 bf16 775 (128 x 256) and
// 668 (256 x 256). E4M3Full has no 256 x 256 tile (its operands as fp16 leave
// no registers for one): 8192 x 4096 x 4096 385, 318, 263 (two workgroups on a
// CU), 254; 1024 x 4096 x 4096 57, 44, 43, 62.
struct TileCost {
    int bm, bn, at_once;           // rows of x, weight rows; workgroups on a CU
    double fixed, alone, shared;   // time of a tile: fixed + S times alone, or shared where a CU has two
};
template <class T>
constexpr int kTileKinds = kFull<T> ? 4 : 5;
template <class T>
constexpr TileCost kTiles[5] = {
    {64, 64, 2, 3.0, kFull<T> ? 0.52 : kEight<T> ? 0.44 : 0.33, kFull<T> ? 0.66 : kEight<T> ? 0.53 : 0.50},
    {128, 128, 1, 4.0, kFull<T> ? 1.10 : kEight<T> ? 0.66 : 0.65, 0.0},
    {128, 128, 2, 4.0, kFull<T> ? 1.12 : kEight<T> ? 0.68 : 0.90, kFull<T> ? 1.93 : kEight<T> ? 1.25 : 1.35},
    {128, 256, 1, 5.0, kFull<T> ? 1.80 : kEight<T> ? 1.15 : 0.95, 0.0},
    {256, 256, 1, kEight<T> ? 8.0 : 10.0, 1.6, 0.0},
};

struct TileChoice {
    int tile;      // of kTiles
    double time;
};
template <class T, bool GLU, bool GRP>
TileChoice choose_tile(const ProductArgs& a) {
    const int64_t cols = GLU ? 2ll * a.N : a.N;
    const double S = (a.K + kStage<T> - 1) / kStage<T>;
    const double groups = GRP ? std::min(a.E, a.M) : 1, mean = a.M / groups;
    TileChoice best{0, 0.0};
    for (int i = 0; i < kTileKinds<T>; ++i) {
        const TileCost& t = kTiles<T>[i];
        // an expert's rows are not known here: on average half a tile more than they fill
        const double rows = GRP && groups > 1 ? groups * std::max(1.0, mean / t.bm + 0.5) : (double)(((int64_t)a.M + t.bm - 1) / t.bm);
        const double load = rows * (double)((cols + t.bn - 1) / t.bn) / 256;   // workgroups of a CU
        double time;
        if (load <= 1.0) time = t.fixed + t.alone * S;
        else if (t.at_once == 1) time = (load < 4.0 ? ceil(load) : load + 0.5) * (t.fixed + t.alone * S);
        else time = (load <= 2.0 ? t.alone + (t.shared - t.alone) * (load - 1.0) : t.shared * load / 2) * S + t.fixed * std::max(1.0, load / 2);
        if (i == 0 || time < best.time) best = {i, time};
    }
    return best;
}

template <class T, bool GLU, bool GRP>
hipError_t launch_tiles(const ProductArgs& a, int tile, hipStream_t s) {
    switch (tile) {
        case 0: return launch_ring<T, 64, 64, 2, 2, 4, GLU, GRP>(a, s);
        case 1: return launch_ring<T, 128, 128, 2, 4, 4, GLU, GRP>(a, s);
        case 2: return launch_ring<T, 128, 128, 2, 4, 2, GLU, GRP>(a, s);
        case 3: return launch_ring<T, 128, 256, 2, 4, 3, GLU, GRP>(a, s);
        default: break;
    }
    if constexpr (kTileKinds<T> == 5) return launch_phased<T, GLU, GRP>(a, s);
    return hipErrorInvalidValue;   // choose_tile names no such tile
}

// Few rows an expert (on average): the weights are streamed. 512 rows of 64
// experts, 2048 -> 768: bf16 41 us (16-row blocks of x, four weight blocks a
// workgroup; two 43; 64 x 64 tiles 51), e4m3 19 (four blocks 20 to 24; tiles
// 22); 1024 rows: 45 and 24 with blocks of 32 rows (56 and 28 with 16, tiles 49
// and 22). With few steps of K two waves: 512 rows of 128 experts, 768 -> 2048
// e4m3 33 us, 44 with four.
// The rule knows the mean only. Rows that gather on one expert are passes, 16
// or 32 rows at a time, of that expert's workgroups over its weights: 128 experts,
// 768 -> 2048 e4m3, 512 rows spread evenly, by popularity ~ 1/rank, half of them
// on one expert, all on one: 40, 33, 54, 58 us (128 x 128 tiles 60, 42, 63, 10);
// 2048 rows 58, 65, 114, 175 (60, 65, 65, 14).
template <class T, bool GLU>
hipError_t launch_grouped_any_size(const ProductArgs& a, hipStream_t s) {
    const int pieces = (a.K + kStage<T> - 1) / kStage<T>;
    const int waves = pieces > 8 ? 4 : pieces > 1 ? 2 : 1;
    const int mean = a.M / std::min(a.E, a.M);
    if (!a.aligned) return launch_any<T, GLU, true>(a, s);
    if (mean > 16) return launch_tiles<T, GLU, true>(a, choose_tile<T, GLU, true>(a).tile, s);
    if (mean > 8) return launch_stream<T, 2, 2, 2, GLU, true>(a, waves, s);
    if constexpr (!kEight<T>)
        if (waves == 4) return launch_stream<T, 4, 1, 2, GLU, true>(a, 4, s);
    return launch_stream<T, 2, 1, 2, GLU, true>(a, waves, s);
}

}  // namespace
}  // namespace pw
