// Rotary positions of rows of D channels, and rows held in 4 bits (device side).
//
// Rotation.  Pair i of a row at position t turns by t theta_i.  theta_i comes as
// a 64-bit fraction of a turn, f_i = 2^64 theta_i / 2 pi: the product t f_i is
// taken modulo 2^64 by the integer multiplier, so the angle is as good at
// position 2^31 as at 0 (an fp32 product is off by half a radian at position
// 10^7).  What is left is the quarter turn and a rest of at most an eighth.
//
// The angles of a tile of tokens are computed once, into shared memory, whatever
// the number of heads that turn by them.
#pragma once

#include "common.cuh"
#include "ptx.cuh"

namespace attn {

// cos and sin of pos * f / 2^64 turns, times m
__device__ __forceinline__ void turn_by(int pos, uint64_t f, float m, float &c, float &s) {
    const uint32_t h = uint32_t((uint64_t(int64_t(pos)) * f) >> 32);
    const uint32_t quarter = (h + 0x20000000u) >> 30;
    const int rest = int(h - (quarter << 30));         // [-1/8, 1/8) turn
    float sr, cr;
    sincospif(float(rest) * 0x1p-31f, &sr, &cr);
    const float x = quarter & 1u ? -sr : cr, y = quarter & 1u ? cr : sr;
    c = (quarter & 2u ? -x : x) * m;
    s = (quarter & 2u ? -y : y) * m;
}

struct Rotation {
    const uint64_t *freq;                              // [rot / 2]; rot 0: no rotation
    int rot;                                           // rotated channels, a multiple of 16
    int interleaved;                                   // pairs (2i, 2i + 1), else (i, i + rot / 2)
    int inverse;
    float mscale;
};

// Where (cos, sin) of a pair stands among its token's rot / 2: the pairs 8 j .. 8 j + 7
// of neighbouring lanes j side by side, two pairs (16 bytes) at a time.
__device__ __forceinline__ int turn_at(int rot, int pair) {
    return (((pair & 7) >> 1) * (rot >> 4) + (pair >> 3)) * 2 + (pair & 1);
}

// (cos, sin) of every pair of the tile's tokens, for the positions pos(token).  All
// threads of the CTA; a barrier must follow.
template <typename F>
__device__ __forceinline__ void fill_turns(const Rotation &r, float2 *tab, int tokens, F pos) {
    const int pairs = r.rot / 2, dt = int(blockDim.x) / pairs, dp = int(blockDim.x) - dt * pairs;
    int t = int(threadIdx.x) / pairs, pair = int(threadIdx.x) - t * pairs;
    while (t < tokens) {
        float c, s;
        turn_by(pos(t), r.freq[pair], r.mscale, c, s);
        tab[t * pairs + turn_at(r.rot, pair)] = make_float2(c, r.inverse ? -s : s);
        t += dt;
        pair += dp;
        if (pair >= pairs) {
            pair -= pairs;
            ++t;
        }
    }
}

// Eight channels of a row as they lie in memory.
template <typename T> struct Row8;
template <> struct Row8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float *p) {
        a = reinterpret_cast<const float4 *>(p)[0];
        b = reinterpret_cast<const float4 *>(p)[1];
    }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        a = make_float4(x[0], x[1], x[2], x[3]);
        b = make_float4(x[4], x[5], x[6], x[7]);
    }
    __device__ __forceinline__ void store(float *p) const {
        reinterpret_cast<float4 *>(p)[0] = a;
        reinterpret_cast<float4 *>(p)[1] = b;
    }
};
template <bool F16> struct Row8H {
    uint4 u;
    __device__ __forceinline__ void load(const void *p) { u = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void get(float (&x)[8]) const {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = H16<F16>::lo(w[i]);
            x[2 * i + 1] = H16<F16>::hi(w[i]);
        }
    }
    __device__ __forceinline__ void set(const float (&x)[8]) {
        u = make_uint4(H16<F16>::pack(x[0], x[1]), H16<F16>::pack(x[2], x[3]), H16<F16>::pack(x[4], x[5]),
                       H16<F16>::pack(x[6], x[7]));
    }
    __device__ __forceinline__ void store(void *p) const { *reinterpret_cast<uint4 *>(p) = u; }
};
template <> struct Row8<__nv_bfloat16> : Row8H<false> {};
template <> struct Row8<__half> : Row8H<true> {};

// Two times eight channels: eight pairs, (a_i, b_i) or interleaved (a_2i, a_2i+1) and
// (b_2i, b_2i+1).  tab: the lane's first (cos, sin), `step` float4s from one two to the
// next.
template <typename T>
__device__ __forceinline__ void rotate16(const float4 *tab, int step, bool interleaved, Row8<T> &a, Row8<T> &b) {
    float x[8], y[8];
    a.get(x);
    b.get(y);
    auto turn = [](float &u, float &v, float c, float s) {
        const float u0 = u;
        u = fmaf(-v, s, u0 * c);
        v = fmaf(u0, s, v * c);
    };
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 p = tab[i * step], q = tab[(i + 2) * step];
            turn(x[4 * i], x[4 * i + 1], p.x, p.y);
            turn(x[4 * i + 2], x[4 * i + 3], p.z, p.w);
            turn(y[4 * i], y[4 * i + 1], q.x, q.y);
            turn(y[4 * i + 2], y[4 * i + 3], q.z, q.w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 p = tab[i * step];
            turn(x[2 * i], y[2 * i], p.x, p.y);
            turn(x[2 * i + 1], y[2 * i + 1], p.z, p.w);
        }
    }
    a.set(x);
    b.set(y);
}

// ------------------------------------------------------- rows held in 4 bits
//
// A group of 32 channels is s (n - 8): s in the 16-bit type, n in [0, 15].  With
// x* the group's largest or least value, whichever is further from zero (the
// largest if both are), s = -x* / 8 rounded, so that x* itself is the code 0 and
// the 16 codes span the group; n = rint(x / s) + 8, held to [0, 15].  A group with
// an infinite or NaN value has s = NaN.
//
// A row of one token and KV head is D + D / 8 bytes: the codes of K, those of V,
// the scales of K's groups, those of V's.  Four codes make a 16-bit word, code i
// at bit 4 i, rotated right by two bits: so a reader gets codes 1 and 2 of two
// words at once by masking bits 2-5 and 6-9 into the mantissas of two f16 numbers
// (256 + n and 16 + n), and 0 and 3 the same way after swapping bytes.  K's words
// for channels 32 g + 8 p .. + 7 lie at p D / 8 + 4 g, V's word for channels
// 32 g + 4 q .. + 3 at D / 2 + q D / 16 + 2 g: what one lane of a decode warp
// multiplies lies together (decode_paged_q4.cu).

__device__ __forceinline__ int q4_row_bytes(int D) { return D + D / 8; }

// Pairs of the 16-bit types.
template <typename T> struct H16F;
template <> struct H16F<__half> {
    static constexpr bool f16 = true;
    using P = __half2;
    static __device__ __forceinline__ P pair(uint32_t x) { return *reinterpret_cast<P *>(&x); }
    static __device__ __forceinline__ P same(__half x) { return __half2half2(x); }
    static __device__ __forceinline__ P same(float x) { return __floats2half2_rn(x, x); }
};
template <> struct H16F<__nv_bfloat16> {
    static constexpr bool f16 = false;
    using P = __nv_bfloat162;
    static __device__ __forceinline__ P pair(uint32_t x) { return *reinterpret_cast<P *>(&x); }
    static __device__ __forceinline__ P same(__nv_bfloat16 x) { return __bfloat162bfloat162(x); }
    static __device__ __forceinline__ P same(float x) { return __floats2bfloat162_rn(x, x); }
};
template <typename P> __device__ __forceinline__ uint32_t pair_bits(P x) { return *reinterpret_cast<uint32_t *>(&x); }

// Largest and least, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b, float c) {
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// x* of the group whose values 4 neighbouring lanes hold, 8 each; NaN if one of them is,
// infinite if one is.
__device__ __forceinline__ float q4_best(const float (&x)[8]) {
    float hi = max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[7]));
    float lo = min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[7]));
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        hi = max_nan(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        lo = min_nan(lo, __shfl_xor_sync(0xffffffffu, lo, off));
    }
    return hi >= -lo ? hi : lo;
}

// The same of values as they lie in memory: pairs, and then the largest and the negative
// of the least side by side.
template <typename T>
__device__ __forceinline__ float q4_best(const uint4 &u) {
    using H = H16F<T>;
    const auto a = H::pair(u.x), b = H::pair(u.y), c = H::pair(u.z), d = H::pair(u.w);
    const uint32_t hi = pair_bits(__hmax2_nan(__hmax2_nan(a, b), __hmax2_nan(c, d)));
    const uint32_t lo = pair_bits(__hmin2_nan(__hmin2_nan(a, b), __hmin2_nan(c, d))) ^ 0x80008000u;
    auto m = __hmax2_nan(H::pair(__byte_perm(hi, lo, 0x5410)), H::pair(__byte_perm(hi, lo, 0x7632)));
#pragma unroll
    for (int off = 1; off < 4; off <<= 1)
        m = __hmax2_nan(m, H::pair(__shfl_xor_sync(0xffffffffu, pair_bits(m), off)));
    const uint32_t w = pair_bits(m);
    const float x = H16<H::f16>::lo(w), y = H16<H::f16>::hi(w);
    return x >= y ? x : -y;
}

// The scale of a group with that x*, and the factor that turns values into codes.
template <typename T>
__device__ __forceinline__ T q4_scale(float best, float &inv) {
    T s;
    Elem<T>::store(&s, best * -0.125f);
    float f = Elem<T>::load(&s);
    if (!(fabsf(f) < INFINITY)) {
        f = NAN;
        Elem<T>::store(&s, f);
    }
    if (fabsf(f) < 0x1p-126f) {                        // a subnormal bf16 has no reciprocal
        f = 0.f;
        Elem<T>::store(&s, f);
    }
    inv = f == 0.f ? 0.f : 1.f / f;
    return s;
}

// The two 16-bit words of 8 channels' codes, the first in the low half.  1.5 2^23 + 8
// is added so that rint(x inv) + 8 stands in the sum's last bits.
template <bool F16>
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        float a, b;
        ptx::ffma2(a, b, x[i], x[i + 1], inv, inv, -0.f, -0.f);
        a = fminf(a, 7.f);
        b = fminf(b, 7.f);
        if (F16) {                                     // (a normal s leaves nothing below -8.5)
            a = fmaxf(a, -8.f);
            b = fmaxf(b, -8.f);
        }
        ptx::fadd2(a, b, a, b, 12582920.f, 12582920.f);
        w += (__float_as_uint(a) << (4 * i)) + (__float_as_uint(b) << (4 * i + 4));
    }
    w -= 0x4b400000u * 0x11111111u;
    w = inv == inv ? w : 0u;                           // a group of NaN
    return ((w >> 2) & 0x3fff3fffu) | ((w << 14) & 0xc000c000u);
}

// The values of 8 codes in the 16-bit type: n - 8 is exact in either, so one product
// rounds once.
template <typename T>
__device__ __forceinline__ uint4 q4_values(uint32_t w, T scale) {
    using H = H16F<T>;
    const uint32_t y = __byte_perm(w, 0, 0x2301);
    uint32_t c[4];                                     // channels (i, i + 4) as 16 + n (f16), 32 + n (bf16)
    if constexpr (H::f16) {
        c[0] = ptx::and_or(y, 0x03c003c0u, 0x4c004c00u);
        c[1] = ptx::and_or(w << 4, 0x03c003c0u, 0x4c004c00u);
        c[2] = ptx::and_or(w, 0x03c003c0u, 0x4c004c00u);
        c[3] = ptx::and_or(y << 4, 0x03c003c0u, 0x4c004c00u);
    } else {
        c[0] = ptx::and_or(y >> 4, 0x003c003cu, 0x42004200u);
        c[1] = ptx::and_or(w, 0x003c003cu, 0x42004200u);
        c[2] = ptx::and_or(w >> 4, 0x003c003cu, 0x42004200u);
        c[3] = ptx::and_or(y, 0x003c003cu, 0x42004200u);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = pair_bits(__hmul2(__hsub2(H::pair(c[i]), H::same(H::f16 ? 24.f : 40.f)), H::same(scale)));
    return make_uint4(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410),
                      __byte_perm(c[0], c[1], 0x7632), __byte_perm(c[2], c[3], 0x7632));
}

}  // namespace attn
