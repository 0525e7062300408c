// Gated router: scores, groups, biased top-k choice and weights.
//
// Per token, over the experts that are to be had (logit finite or +inf and
// above the type's lowest value; NaN, -inf and the lowest value are not):
//   s_e = 1 / (1 + e^-l_e)  or  e^(l_e - m) / sum e^(l - m)
//   c_e = s_e + b_e (b absent: c orders like the logit itself)
//   groups of E / G consecutive experts, scored by their largest c or by the
//   sum of their two largest; the topk_group best stay (ties: lower group);
//   the k largest c of the groups that stay (ties: lower expert);
//   g_j = scale s_j, or scale s_j / sum of the chosen s. Slots without an
//   expert: id -1, weight 0.
//
// The choice is that of the exact scores. Where c is the logit (no bias, and
// groups by their largest) it is exact as it stands. Otherwise c is taken in
// fp64 with a short exponential (about 2^-36 of a score; 20 instructions per
// expert), every comparison that decides something is checked against a
// bound on its error, and a token with a nearer pair is chosen again from
// full fp64 scores. (With fp32 scores and the same check one token in a
// thousand had to be: its wave took 10 us longer, and with it the launch.)
//
// Keys: c as a double with the expert id in its low 10 bits (a converted
// fp32 logit leaves 29 empty), so one v_max_f64 orders (c, lower id first).
//
// A token is routed by L lanes of a wave, lane l holding experts l, l + L,
// ...: 16 lanes (four tokens a wave, reductions inside a DPP row) for
// throughput, 64 lanes for the latency of few tokens and for more than 256
// experts.
#include <hip/hip_runtime.h>

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "pw_internal.h"
#include "route_dev.h"

namespace pw {
namespace {

using namespace rdev;

constexpr int kGateBlock = 256;
constexpr double kGone = -0x1p300;      // key of an expert that is not to be had
constexpr double kGoneBelow = -0x1p250; // keys below: none left
constexpr double kMost = 0x1p200;       // key of c = +inf (above every fp32 value)
// How far two choice scores can be from their exact difference, as a
// multiple of (|c| + S), S = 1 (sigmoid) or the largest score (softmax): the
// exponential is off by at most 2^-36 of itself (exp_short), so a score by
// 2^-35 of S, and a key by the 10 bits the id takes, 2^-42 |c|; for two 2^-34
// S + 2^-41 |c|, twice that for sums of two scores (taken with 2 S and the
// sum of their |c|).
constexpr double kTol = 0x1p-33;

__device__ __forceinline__ double max_f64(double a, double b) {
    double d;
    asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}
__device__ __forceinline__ double min_f64(double a, double b) {
    double d;
    asm("v_min_f64 %0, %1, %2" : "=v"(d) : "v"(a), "v"(b));
    return d;
}

// The result over the L lanes of a token, in each of them.
template <int L>
__device__ __forceinline__ double lanes_max(double x) {
    x = max_f64(x, dpp_d<kQuadXor1>(x));
    x = max_f64(x, dpp_d<kQuadXor2>(x));
    x = max_f64(x, dpp_d<kRowHalfMirror>(x));
    x = max_f64(x, dpp_d<kRowMirror>(x));
    if constexpr (L == 64) {
        auto rows = [&](auto ctrl, auto mask) {
            const uint64_t u = __builtin_bit_cast(uint64_t, x);
            const int lo = dpp_rows_i<decltype(ctrl)::value, decltype(mask)::value>((int)(uint32_t)u);
            const int hi = dpp_rows_i<decltype(ctrl)::value, decltype(mask)::value>((int)(uint32_t)(u >> 32));
            x = max_f64(x, __builtin_bit_cast(double, ((uint64_t)(uint32_t)hi << 32) | (uint32_t)lo));
        };
        rows(std::integral_constant<int, kRowBcast15>{}, std::integral_constant<int, 0xa>{});
        rows(std::integral_constant<int, kRowBcast31>{}, std::integral_constant<int, 0xc>{});
        const uint64_t u = __builtin_bit_cast(uint64_t, x);
        const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, 63);
        const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
        x = __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
    }
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
    if constexpr (L == 64) return wave_sum(x);
    return row_sum(x);
}
template <int L>
__device__ __forceinline__ double lanes_sum(double x) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) x += __shfl_xor(x, o);
    return x;
}
template <int L>
__device__ __forceinline__ float lanes_fmax(float x) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}

// c (fp32, -inf: not to be had) and the expert id as one key: the id, its
// bits turned for positive c so that lower ids are larger either way, in the
// low bits that a converted fp32 number leaves empty
__device__ __forceinline__ double make_key(float c, int e) {
    const double d = max_f64(min_f64((double)(c + 0.0f), kMost), kGone);   // -0 as +0
    const uint64_t u = __builtin_bit_cast(uint64_t, d);
    const int neg = (int)(u >> 32) >> 31;
    const uint32_t lo = (uint32_t)u | (uint32_t)((neg & 1023) ^ (e ^ 1023));
    return __builtin_bit_cast(double, (u & 0xffffffff00000000ull) | lo);
}
__device__ __forceinline__ int key_id(double k) {
    const uint64_t u = __builtin_bit_cast(uint64_t, k);
    const int i = (int)(u & 1023u);
    return (u >> 63) ? i : 1023 - i;
}

// The same for fp64 scores (their low 10 bits go).
__device__ __forceinline__ double make_key(double c, int e) {
    const double d = max_f64(min_f64(c + 0.0, kMost), kGone);   // -inf: kGone (c is not NaN)
    const uint64_t u = __builtin_bit_cast(uint64_t, d);
    const int neg = (int)(u >> 32) >> 31;
    const uint32_t lo = ((uint32_t)u & ~1023u) | (uint32_t)((neg & 1023) ^ (e ^ 1023));
    return __builtin_bit_cast(double, (u & 0xffffffff00000000ull) | lo);
}

// A constant that stays in a pair of scalar registers, where the compiler would
// move it into vector registers for each use (16384 x 256, top-8, both builds in
// turn: sigmoid with bias 15.4 -> 15.1 us, with groups 19.65 -> 19.5)
__device__ __forceinline__ double scalar_f64(double c) {
    asm("" : "+s"(c));
    return c;
}
// e^x for x <= 0 in fp64: x = n ln 2 + r, |r| <= 0.3466, the Taylor polynomial
// of degree 9 (remainder r^10 / 10! < 2^-37) and 2^n; r is off by n ln2 2^-53
// and the sums by a few 2^-53, so the whole by less than 2^-36.
__device__ __forceinline__ double exp_short(double x) {
    x = max_f64(x, -800.0);
    const double n = rint(x * scalar_f64(1.4426950408889634));
    const double r = fma(-n, scalar_f64(0.69314718055994531), x);
    double p = scalar_f64(1.0 / 362880.0);
    p = fma(p, r, scalar_f64(1.0 / 40320.0));
    p = fma(p, r, scalar_f64(1.0 / 5040.0));
    p = fma(p, r, scalar_f64(1.0 / 720.0));
    p = fma(p, r, scalar_f64(1.0 / 120.0));
    p = fma(p, r, scalar_f64(1.0 / 24.0));
    p = fma(p, r, scalar_f64(1.0 / 6.0));
    p = fma(p, r, 0.5);
    p = fma(p, r, 1.0);
    p = fma(p, r, 1.0);
    return ldexp(p, (int)n);
}
// 1 / d for 1 <= d <= 2048: the instruction's estimate and one Newton step
// (an estimate good to 2^-20 already gives 2^-40)
__device__ __forceinline__ double rcp_short(double d) {
    const double y = __builtin_amdgcn_rcp(d);
    return fma(y, fma(-d, y, 1.0), y);
}

// e^x for x <= 0 with the rounding of x log2(e) carried along: within 3
// 2^-24 of the value wherever that is a normal number
__device__ __forceinline__ float exp_neg(float x) {
    constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLo = 1.92596299e-8f, kLn2 = 0.693147180559945f;
    if (!(x > -104.0f)) return 0.0f;
    const float t = x * kLog2e;
    const float r = fmaf(x, kLog2eLo, fmaf(x, kLog2e, -t));
    const float e = __builtin_amdgcn_exp2f(t);
    return fmaf(e, r * kLn2, e);
}

template <class T>
__device__ __forceinline__ float to_f32(T v) { return (float)v; }
template <>
__device__ __forceinline__ float to_f32<uint16_t>(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
// the type's lowest finite value: logits at or below it are masked
template <class T> __device__ __forceinline__ constexpr float lowest_of();
template <> __device__ __forceinline__ constexpr float lowest_of<float>() { return -3.402823466385288598e38f; }
template <> __device__ __forceinline__ constexpr float lowest_of<uint16_t>() { return -3.38953138925153547590e38f; }
template <> __device__ __forceinline__ constexpr float lowest_of<_Float16>() { return -65504.0f; }

// LDS of a wave is read in order after what it wrote: only the compiler has
// to keep the order
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// The groups that stay, as a bit mask (G <= 64), of experts scored c[i] (below
// kGoneBelow: not to be had; scores or keys, whose id bits order equal groups
// like their numbers); tol > 0: the scores are approximate, near is set
// where they do not decide. c goes through the token's LDS row (E doubles),
// the groups' scores through gs_row (2 G doubles).
template <int L, int PER>
__device__ __forceinline__ uint64_t keep_groups(const GateArgs& a, const double (&c)[PER], double* row, double* gs_row,
                                                double tol, double top_s, bool& near) {
    const int l = threadIdx.x & (L - 1);
    const int G = a.n_group, gs = a.E / G;
    wave_fence();   // the row's former readers are done
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (l + L * i < a.E) row[l + L * i] = c[i];
    wave_fence();
    // p lanes per group, the largest power of two that lets all groups go at
    // once (one lane, and several rounds, if there are more groups than lanes)
    const int p = a.group_lanes;
    for (int q0 = 0; q0 < G; q0 += L / p) {
        const int q = q0 + l / p, sub = l & (p - 1);
        double m1 = kGone, m2 = kGone;
        if (q < G) {
            // each group starts at another place: groups of 32 experts
            // would otherwise read one LDS bank
            int at = sub + q % gs;
            const double* src = row + q * gs;
#pragma unroll 4
            for (int i = sub; i < gs; i += p) {
                at = at >= gs ? at - gs : at;
                const double v = src[at];
                m2 = max_f64(m2, min_f64(m1, v));
                m1 = max_f64(m1, v);
                at += p;
            }
        }
        for (int o = 1; o < p; o <<= 1) {
            const double n1 = __shfl_xor(m1, o), n2 = __shfl_xor(m2, o);
            m2 = max_f64(max_f64(m2, n2), min_f64(m1, n1));
            m1 = max_f64(m1, n1);
        }
        double score = kGone, size = 0.0;
        if (m1 > kGoneBelow) {
            score = m1;
            size = fabs(m1);
            if (a.group_top2 && m2 > kGoneBelow) {
                score = min_f64(score + m2, kMost);   // inf + inf is not above inf
                size += fabs(m2);
            }
        }
        if (q < G && sub == 0) {
            gs_row[q] = score;
            gs_row[G + q] = size;
        }
    }
    wave_fence();
    uint64_t kept = 0;
    double low_kept = kMost * 4.0, high_out = kGone, size = 0.0;
    for (int q0 = 0; q0 < G; q0 += L) {
        const int q = q0 + l;
        bool keep = false;
        if (q < G) {
            const double mine = gs_row[q];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < G; ++j) {
                const double v = gs_row[j];
                rank += (v > mine || (v == mine && j < q)) ? 1 : 0;
            }
            keep = rank < a.topk_group;
            if (keep) low_kept = min_f64(low_kept, mine);
            else high_out = max_f64(high_out, mine);
            size = max_f64(size, gs_row[G + q]);
        }
        const uint64_t b = __ballot(keep);
        const uint64_t mine_bits = L == 64 ? b : (b >> ((threadIdx.x & 63) & ~(L - 1))) & 0xffffull;
        kept |= mine_bits << q0;
    }
    if (tol > 0.0) {
        low_kept = -lanes_max<L>(-low_kept);
        high_out = lanes_max<L>(high_out);
        size = lanes_max<L>(size);
        if (high_out > kGoneBelow && low_kept - high_out <= tol * (size + 2.0 * top_s)) near = true;
    }
    return kept;
}

// The k largest keys: lane l gets choice l in id0 and, with 16 lanes, choice
// l + 16 in id1 (-1: none). near as above.
template <int L, int PER>
__device__ __forceinline__ void choose(const GateArgs& a, double (&key)[PER], double tol, double top_s, int& id0,
                                       int& id1, bool& near) {
    const int l = threadIdx.x & (L - 1);
    id0 = id1 = -1;
    double prev = kMost * 4.0;
    for (int j = 0;; ++j) {
        if (j == a.k && tol == 0.0) break;
        double m[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) m[i] = key[i];
#pragma unroll
        for (int h = 1; h < PER; h *= 2)
#pragma unroll
            for (int i = 0; i + h < PER; i += 2 * h) m[i] = max_f64(m[i], m[i + h]);
        const double best = lanes_max<L>(m[0]);
        const bool any = best > kGoneBelow;
        if (tol > 0.0 && any && prev - best <= tol * (fabs(best) + top_s)) near = true;
        if (j == a.k) break;
        prev = best;
        const int e = any ? key_id(best) : -1;
        if (j == l) id0 = e;
        if (L == 16 && j == l + 16) id1 = e;
        // the chosen expert leaves its lane (the high word alone makes its
        // key smaller than every other)
        const int d = e - l;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint64_t u = __builtin_bit_cast(uint64_t, key[i]);
            const uint32_t hi = d == L * i ? 0xd2b00000u : (uint32_t)(u >> 32);
            key[i] = __builtin_bit_cast(double, ((uint64_t)hi << 32) | (uint32_t)u);
        }
    }
}

// The same choice from whole fp64 scores (kGone: none): the largest, of equal
// ones the lowest expert.
template <int L, int PER>
__device__ __forceinline__ void choose_exact(const GateArgs& a, double (&c)[PER], int& id0, int& id1) {
    const int l = threadIdx.x & (L - 1);
    id0 = id1 = -1;
    for (int j = 0; j < a.k; ++j) {
        double m = c[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = max_f64(m, c[i]);
        const double best = lanes_max<L>(m);
        int e = kMaxExperts;
#pragma unroll
        for (int i = PER - 1; i >= 0; --i)
            if (c[i] == best) e = l + L * i;
#pragma unroll
        for (int o = 1; o < L; o <<= 1) e = min(e, __shfl_xor(e, o));
        if (!(best > kGoneBelow)) e = -1;
        if (j == l) id0 = e;
        if (L == 16 && j == l + 16) id1 = e;
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (l + L * i == e) c[i] = kGone;
    }
}

template <int L, int PER, class TL>
__device__ __forceinline__ void gate_token(const GateArgs& a, int t, bool valid, double* row, double* gs_row, int* hist) {
    const int l = threadIdx.x & (L - 1);
    const TL* src = reinterpret_cast<const TL*>(a.logits) + (int64_t)t * a.ld;
    const bool live = valid && (!a.mask || a.mask[t] != 0);
    float v[PER];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = l + L * i;
        v[i] = (live && e < a.E) ? to_f32(src[e]) : -INFINITY;
        if (!(v[i] > lowest_of<TL>())) v[i] = -INFINITY;   // NaN too
    }
    // with 64 lanes (few tokens) the bias is loaded with the logits; 16 lanes
    // load it where it is used (its registers would cost a wave per SIMD:
    // 16384 x 256 took 28 us instead of 23)
    auto bias_of = [&](int i) { return a.bias && l + L * i < a.E ? a.bias[l + L * i] : 0.0f; };
    float b[L == 64 ? PER : 1];
    if constexpr (L == 64) {
#pragma unroll
        for (int i = 0; i < PER; ++i) b[i] = bias_of(i);
    }
    auto bias = [&](int i) { return (double)(L == 64 ? b[L == 64 ? i : 0] : bias_of(i)); };
    const bool softmax = a.score == PW_SCORE_SOFTMAX;
    const bool by_logit = !a.bias && !(a.n_group > 1 && a.group_top2);
    // softmax: the largest logit and the sum of the exponentials, where the
    // scores themselves are needed
    float m = 0.0f, den = 1.0f;
    if (softmax && (!by_logit || !a.renorm)) {
        m = v[0];
#pragma unroll
        for (int i = 1; i < PER; ++i) m = fmaxf(m, v[i]);
        m = lanes_fmax<L>(m);
    }
    if (softmax && by_logit && !a.renorm) {
        den = 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) den += v[i] == -INFINITY ? 0.0f : (v[i] == m ? 1.0f : exp_neg(v[i] - m));
        den = lanes_sum<L>(den);
    }
    double key[PER], top_s = 1.0;
    if (by_logit) {
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = make_key(v[i], l + L * i);
    } else {
        double inv = 1.0;
        if (softmax) {
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                key[i] = v[i] == -INFINITY ? 0.0 : (v[i] == m ? 1.0 : exp_short((double)v[i] - (double)m));
                sum += key[i];
            }
            sum = lanes_sum<L>(sum);
            den = (float)sum;
            inv = top_s = sum > 0.0 ? rcp_short(sum) : 0.0;
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = l + L * i;
            double sc;
            if (softmax) {
                sc = key[i] * inv;
            } else {
                const double ex = exp_short(-fabs((double)v[i]));
                sc = (v[i] < 0.0f ? ex : 1.0) * rcp_short(1.0 + ex);
            }
            sc += bias(i);
            key[i] = make_key(v[i] > -INFINITY && sc == sc ? sc : -INFINITY, e);
        }
    }
    bool near = false;
    int id0, id1;
    if (a.n_group > 1) {
        const uint64_t kept = keep_groups<L, PER>(a, key, row, gs_row, by_logit ? 0.0 : kTol, top_s, near);
        // without a bias the logits give the order within the groups that stay
        if (!by_logit && !a.bias) {
#pragma unroll
            for (int i = 0; i < PER; ++i) key[i] = make_key(v[i], l + L * i);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int q = (int)(((uint32_t)(l + L * i) * a.group_magic) >> 20);
            if (!((kept >> (q & 63)) & 1)) key[i] = kGone;
        }
    }
    choose<L, PER>(a, key, a.bias ? kTol : 0.0, top_s, id0, id1, near);
    if (!by_logit && __any(near)) {
        // scores in fp64 (the whole wave; tokens that were decided keep
        // their choice)
        double den64 = 1.0;
        if (softmax) {
            den64 = 0.0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                den64 += v[i] == -INFINITY ? 0.0 : (v[i] == m ? 1.0 : exp((double)v[i] - (double)m));
            den64 = lanes_sum<L>(den64);
        }
        double s64[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            double sc = kGone;
            if (v[i] > -INFINITY) {
                const double x = (double)v[i];
                if (softmax) sc = (v[i] == m ? 1.0 : exp(x - (double)m)) / den64;
                else sc = 1.0 / (1.0 + exp(-x));
                sc += bias(i);
                // a NaN c is not chosen (v_min_f64 would make it kMost)
                sc = sc == sc ? max_f64(min_f64(sc, kMost), kGone) : kGone;
            }
            s64[i] = sc;
        }
        bool none = false;
        int i0, i1;
        if (a.n_group > 1) {
            const uint64_t kept = keep_groups<L, PER>(a, s64, row, gs_row, 0.0, top_s, none);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int q = (int)(((uint32_t)(l + L * i) * a.group_magic) >> 20);
                if (!a.bias) s64[i] = v[i] > -INFINITY ? min_f64((double)v[i], kMost) : kGone;
                if (!((kept >> (q & 63)) & 1)) s64[i] = kGone;
            }
        }
        choose_exact<L, PER>(a, s64, i0, i1);
        if (near) {
            id0 = i0;
            id1 = i1;
        }
    }
    // weights of the chosen, from their own logits
    auto logit_of = [&](int id) { return id >= 0 ? to_f32(src[id]) : -INFINITY; };
    const float x0 = logit_of(id0), x1 = L == 16 ? logit_of(id1) : -INFINITY;
    float w0, w1;
    if (softmax) {
        const float top = a.renorm ? lanes_fmax<L>(fmaxf(x0, x1)) : m;
        w0 = id0 < 0 ? 0.0f : (x0 == top ? 1.0f : exp_neg(x0 - top));
        w1 = id1 < 0 ? 0.0f : (x1 == top ? 1.0f : exp_neg(x1 - top));
        // beside an infinite logit that is not chosen every score is 0, and so
        // is their sum (m is not taken where the largest logit is always chosen)
        if (a.renorm && m == INFINITY && top < INFINITY) w0 = w1 = 0.0f;
    } else {
        // s = e^min(x, 0) / (1 + e^-|x|); renormalised weights leave out the
        // common power of e, so that they are right where every s underflows
        const float z0 = fminf(x0, 0.0f), z1 = fminf(x1, 0.0f);
        const float top = a.renorm ? lanes_fmax<L>(fmaxf(z0, z1)) : 0.0f;
        w0 = id0 < 0 ? 0.0f : exp_neg(z0 - top) / (1.0f + exp_neg(-fabsf(x0)));
        w1 = id1 < 0 ? 0.0f : exp_neg(z1 - top) / (1.0f + exp_neg(-fabsf(x1)));
    }
    const float total = a.renorm ? lanes_sum<L>(w0 + w1) : (softmax ? den : 1.0f);
    const float f = total > 0.0f ? a.scale / total : 0.0f;
    if (!valid) return;
    auto put = [&](int j, int id, float w) {
        if (j >= a.k) return;
        a.ids[(int64_t)t * a.k + j] = id;
        a.g[(int64_t)t * a.k + j] = id < 0 ? 0.0f : w * f;
        if (hist && id >= 0) atomicAdd(&hist[id], 1);
    };
    put(l, id0, w0);
    if (L == 16) put(l + 16, id1, w1);
}

// ONE: the whole batch in one workgroup, L lanes per token, which also counts
// the pairs of each expert in LDS; else a token per L lanes over the grid
// (workgroup 0 clears the counts for the kernel that follows).
constexpr int one_threads(int per) { return per > 8 ? 512 : 1024; }   // what their registers allow

template <int L, int PER, class TL, bool ONE>
__global__ __launch_bounds__(ONE ? one_threads(PER) : kGateBlock) void gate_kernel(GateArgs a) {
    extern __shared__ __attribute__((aligned(16))) double gate_lds[];
    __shared__ int hist[ONE ? kMaxExperts : 1];
    const int slot = threadIdx.x / L;
    double* row = gate_lds + (int64_t)slot * (a.E + 2 * a.n_group);
    if constexpr (ONE) {
        for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
        __syncthreads();
        gate_token<L, PER, TL>(a, slot < a.T ? slot : 0, slot < a.T, row, row + a.E, a.counts ? hist : nullptr);
        __syncthreads();
        if (a.counts)
            for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[e] = hist[e];
    } else {
        if (a.counts && blockIdx.x == 0)
            for (int e = threadIdx.x; e < a.E; e += kGateBlock) a.counts[e] = 0;
        const int64_t t = (int64_t)blockIdx.x * (kGateBlock / L) + slot;
        gate_token<L, PER, TL>(a, t < a.T ? (int)t : 0, t < a.T, row, row + a.E, nullptr);
    }
}

// Pairs of each expert (counts cleared by the kernel before): LDS counters
// per workgroup, then one atomic per expert.
__global__ __launch_bounds__(1024) void gate_count_kernel(const int32_t* ids, int64_t P, int E, int32_t* counts) {
    __shared__ int hist[kMaxExperts];
    for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
    __syncthreads();
    const int64_t step = (int64_t)gridDim.x * 1024;
    for (int64_t p0 = (int64_t)blockIdx.x * 1024 + threadIdx.x; p0 < P; p0 += 8 * step) {
        int e[8];   // their loads together
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = p0 + i * step < P ? ids[p0 + i * step] : -1;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (e[i] >= 0) atomicAdd(&hist[e[i]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += 1024)
        if (hist[e]) atomicAdd(&counts[e], hist[e]);
}

// 64 lanes per token up to this many tokens (they spread over the GPU)
constexpr int kWaveTokens = 1024;

template <int L, int PER, class TL>
hipError_t launch_gate_t(const GateArgs& a0, hipStream_t s) {
    GateArgs a = a0;
    a.group_lanes = 1;
    while (2 * a.group_lanes * a.n_group <= L) a.group_lanes *= 2;
    const size_t row = a.n_group > 1 ? ((size_t)a.E + 2 * a.n_group) * sizeof(double) : 0;
    const int64_t threads = ((int64_t)a.T * L + 63) / 64 * 64;
    if (threads <= one_threads(PER) && (size_t)(threads / L) * row <= 64 * 1024) {
        gate_kernel<L, PER, TL, true><<<1, (unsigned)threads, row * (size_t)(threads / L), s>>>(a);
        return hipGetLastError();
    }
    const int per = kGateBlock / L;
    gate_kernel<L, PER, TL, false><<<(unsigned)((a.T + per - 1) / per), kGateBlock, row * per, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.counts) return e;
    const int64_t P = (int64_t)a.T * a.k;
    const unsigned blocks = (unsigned)std::min<int64_t>((P + 8191) / 8192, 64);
    gate_count_kernel<<<blocks, 1024, 0, s>>>(a.ids, P, a.E, a.counts);
    return hipGetLastError();
}

template <class TL>
hipError_t launch_gate_d(const GateArgs& a, hipStream_t s) {
    // one workgroup up to 64 tokens if 16 lanes can take one (to 16 at 64
    // lanes each)
    const bool rows = a.E <= 256 && (a.T > kWaveTokens || (a.counts && a.T > 16 && a.T <= (a.E <= 128 ? 64 : 32)));
    if (!rows) {
        const int per = (a.E + 63) / 64;
        if (per == 1) return launch_gate_t<64, 1, TL>(a, s);
        if (per == 2) return launch_gate_t<64, 2, TL>(a, s);
        if (per <= 4) return launch_gate_t<64, 4, TL>(a, s);
        if (per <= 8) return launch_gate_t<64, 8, TL>(a, s);
        return launch_gate_t<64, 16, TL>(a, s);
    }
    const int per = (a.E + 15) / 16;
    if (per <= 2) return launch_gate_t<16, 2, TL>(a, s);
    if (per <= 4) return launch_gate_t<16, 4, TL>(a, s);
    if (per <= 8) return launch_gate_t<16, 8, TL>(a, s);
    return launch_gate_t<16, 16, TL>(a, s);
}

}  // namespace

hipError_t launch_gate(const GateArgs& a0, hipStream_t s) {
    GateArgs a = a0;
    // e / (E / G) for e < 1024 as a multiplication: the error e / 2^20 stays
    // below 1 / (E / G)
    const uint32_t gs = (uint32_t)(a.E / a.n_group);
    a.group_magic = ((1u << 20) + gs - 1) / gs;
    if (a.dtype == PW_F32) return launch_gate_d<float>(a, s);
    if (a.dtype == PW_BF16) return launch_gate_d<uint16_t>(a, s);
    return launch_gate_d<_Float16>(a, s);
}

}  // namespace pw
