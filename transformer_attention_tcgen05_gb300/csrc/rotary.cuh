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
    const int pairs = r.rot / 2;
    for (int e = threadIdx.x; e < tokens * pairs; e += blockDim.x) {
        const int t = e / pairs, pair = e - t * pairs;
        float c, s;
        turn_by(pos(t), r.freq[pair], r.mscale, c, s);
        tab[t * pairs + turn_at(r.rot, pair)] = make_float2(c, r.inverse ? -s : s);
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

// The scale of the group whose values 4 neighbouring lanes hold, 8 each; the
// factor that turns values into codes.
template <typename T>
__device__ __forceinline__ T q4_scale(const float (&x)[8], float &inv) {
    float hi = x[0], lo = x[0], z = 0.f * x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) {
        hi = fmaxf(hi, x[i]);
        lo = fminf(lo, x[i]);
        z = fmaf(0.f, x[i], z);                        // NaN if a value is infinite or NaN
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
        z += __shfl_xor_sync(0xffffffffu, z, off);
    }
    T s;
    Elem<T>::store(&s, (hi >= -lo ? hi : lo) * -0.125f + z);
    float f = Elem<T>::load(&s);
    if (fabsf(f) < 0x1p-126f) {                        // a subnormal bf16 has no reciprocal
        Elem<T>::store(&s, 0.f);
        f = 0.f;
    }
    inv = f == 0.f ? 0.f : 1.f / f;
    return s;
}

// Pairs of the 16-bit types.
template <typename T> struct H16F;
template <> struct H16F<__half> {
    static constexpr bool f16 = true;
    static __device__ __forceinline__ uint32_t minus24(uint32_t x) {
        const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&x), __floats2half2_rn(24.f, 24.f));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ uint32_t mul(uint32_t x, __half s) {
        const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&x), __half2half2(s));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};
template <> struct H16F<__nv_bfloat16> {
    static constexpr bool f16 = false;
    static __device__ __forceinline__ uint32_t minus24(uint32_t x) {
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&x), __floats2bfloat162_rn(24.f, 24.f));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ uint32_t mul(uint32_t x, __nv_bfloat16 s) {
        const __nv_bfloat162 r = __hmul2(*reinterpret_cast<__nv_bfloat162 *>(&x), __bfloat162bfloat162(s));
        return *reinterpret_cast<const uint32_t *>(&r);
    }
};

// The two 16-bit words of 8 channels' codes, the first in the low half.  1.5 2^23 + 8
// is added so that rint(x inv) + 8 stands in the sum's last bits.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float n = fminf(fmaxf(x[i] * inv, -8.f), 7.f);       // NaN: -8
        w += __float_as_uint(n + 12582920.f) << (4 * i);
    }
    w -= 0x4b400000u * 0x11111111u;
    return ((w >> 2) & 0x3fff3fffu) | ((w << 14) & 0xc000c000u);
}

// The values of 8 codes in the 16-bit type: n - 8 is exact in either, so one product
// rounds once.
template <typename T>
__device__ __forceinline__ uint4 q4_values(uint32_t w, T scale) {
    const uint32_t y = __byte_perm(w, 0, 0x2301);
    uint32_t c[4];                                     // channels (i, i + 4) as 16 + n
    if constexpr (H16F<T>::f16) {
        c[0] = (y & 0x03c003c0u) | 0x4c004c00u;
        c[1] = ((w << 4) & 0x03c003c0u) | 0x4c004c00u;
        c[2] = (w & 0x03c003c0u) | 0x4c004c00u;
        c[3] = ((y << 4) & 0x03c003c0u) | 0x4c004c00u;
    } else {
        c[0] = ((y >> 3) & 0x00780078u) | 0x41804180u;
        c[1] = ((w << 1) & 0x00780078u) | 0x41804180u;
        c[2] = ((w >> 3) & 0x00780078u) | 0x41804180u;
        c[3] = ((y << 1) & 0x00780078u) | 0x41804180u;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = H16F<T>::mul(H16F<T>::minus24(c[i]), scale);
    return make_uint4(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410),
                      __byte_perm(c[0], c[1], 0x7632), __byte_perm(c[2], c[3], 0x7632));
}

}  // namespace attn
