// Rotary positions of rows of D channels, and rows held in 4 bits (device side).
//
// Rotation.  Pair i of a row at position t turns by t theta_i.  theta_i comes as
// a 64-bit fraction of a turn, f_i = 2^64 theta_i / 2 pi: the product t f_i is
// taken modulo 2^64 by the integer multiplier, so the angle is as good at
// position 2^31 as at 0 (an fp32 product is off by half a radian at position
// 10^7).  What is left is the quarter turn and a rest of at most an eighth.
//
// Every thread owns 8 consecutive channels of a row, so a group of 32 channels
// belongs to 4 neighbouring lanes and a row to D / 8.
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

// What a thread needs to rotate its channels [c0, c0 + 8): y = x cs + partner sn.
struct Turn {
    float cs[8], sn[8];
    int partner;                                       // first channel of the partners (interleaved: c0)
};

__device__ __forceinline__ void make_turn(const Rotation &r, int pos, int c0, Turn &t) {
    if (r.interleaved) {
        t.partner = c0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float c, s;
            turn_by(pos, r.freq[c0 / 2 + i], r.mscale, c, s);
            s = r.inverse ? -s : s;
            t.cs[2 * i] = t.cs[2 * i + 1] = c;
            t.sn[2 * i] = -s;
            t.sn[2 * i + 1] = s;
        }
    } else {
        const bool upper = c0 >= r.rot / 2;
        t.partner = upper ? c0 - r.rot / 2 : c0 + r.rot / 2;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float c, s;
            turn_by(pos, r.freq[(upper ? t.partner : c0) + i], r.mscale, c, s);
            t.cs[i] = c;
            t.sn[i] = upper != bool(r.inverse) ? s : -s;
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

// The rotated channels in fp32 (x: the thread's own, y: its partners').
template <typename T>
__device__ __forceinline__ void rotate8(const Turn &t, const Row8<T> &x, const Row8<T> &y, bool interleaved,
                                        float (&out)[8]) {
    float a[8], b[8];
    x.get(a);
    y.get(b);
#pragma unroll
    for (int i = 0; i < 8; ++i)
        out[i] = fmaf(interleaved ? a[i ^ 1] : b[i], t.sn[i], a[i] * t.cs[i]);
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

// The two 16-bit words of 8 channels' codes, the first in the low half.
__device__ __forceinline__ uint32_t q4_codes(const float (&x)[8], float inv) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int n = int(fminf(fmaxf(rintf(x[i] * inv) + 8.f, 0.f), 15.f));
        w |= uint32_t(n) << (4 * i);
    }
    return ((w >> 2) & 0x3fff3fffu) | ((w << 14) & 0xc000c000u);
}

// The values of 8 codes.
__device__ __forceinline__ void q4_values(uint32_t w, float s, float (&x)[8]) {
    w = ((w << 2) & 0xfffcfffcu) | ((w >> 14) & 0x00030003u);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = float(int((w >> (4 * i)) & 15u) - 8) * s;
}

}  // namespace attn
