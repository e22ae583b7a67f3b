// Device helpers shared by the layer operators' kernels.
#pragma once

#include "layer_internal.hpp"

namespace muon {
namespace layer {

typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

#ifndef GMEM   // a host build for bounds checking defines it empty
#define GMEM __attribute__((address_space(1)))
#endif
template <class T>
__device__ __forceinline__ GMEM T* gm(T* p) { return (GMEM T*)p; }

__device__ __forceinline__ float bf16_bits_to_f32(uint32_t b) { return __uint_as_float(b << 16); }
__device__ __forceinline__ uint32_t f32_to_bf16_bits(float f) {   // round to nearest even
    __bf16 h = (__bf16)f;
    return uint32_t(__builtin_bit_cast(uint16_t, h));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    return f32_to_bf16_bits(lo) | (f32_to_bf16_bits(hi) << 16);
}

// dt 0 = bf16, 1 = f32
__device__ __forceinline__ float load1(const void* p, int64_t i, int dt) {
    return dt == 0 ? bf16_bits_to_f32(gm(static_cast<const uint16_t*>(p))[i]) : gm(static_cast<const float*>(p))[i];
}
__device__ __forceinline__ void store1(void* p, int64_t i, int dt, float v) {
    if (dt == 0) gm(static_cast<uint16_t*>(p))[i] = uint16_t(f32_to_bf16_bits(v));
    else gm(static_cast<float*>(p))[i] = v;
}

__device__ __forceinline__ void unpack_bf16x8(u32x4_t w, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// 8 consecutive elements from element i on, of which the first n exist (the
// rest read as 0); vec: the address allows 16-byte vectors.
__device__ __forceinline__ void load8(const void* p, int64_t i, int dt, bool vec, int n, float (&v)[8]) {
    if (vec && n >= 8) {
        if (dt == 0) {
            unpack_bf16x8(*gm(reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + i)), v);
        } else {
            const f32x4_t a = *gm(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i));
            const f32x4_t b = *gm(reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + i + 4));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = a[k];
                v[4 + k] = b[k];
            }
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = k < n ? load1(p, i + k, dt) : 0.f;
}

// 16 bytes; STREAM: past the caches where that can be (each XCD's L2 writes its
// dirty lines back at the kernel's end, and a streamed line has left by then).
template <bool STREAM, class V>
__device__ __forceinline__ void put16(GMEM void* p, V w) {
    GMEM V* q = reinterpret_cast<GMEM V*>(p);
    if constexpr (STREAM) __builtin_nontemporal_store(w, q);
    else *q = w;
}
__device__ __forceinline__ void store8(void* p, int64_t i, int dt, bool vec, int n, const float (&v)[8]) {
    if (vec && n >= 8) {
        if (dt == 0) {
            *gm(reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + i)) =
                u32x4_t{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
        } else {
            *gm(reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i)) = f32x4_t{v[0], v[1], v[2], v[3]};
            *gm(reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + i + 4)) = f32x4_t{v[4], v[5], v[6], v[7]};
        }
        return;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (k < n) store1(p, i + k, dt, v[k]);
}

// ---- 8-bit checkpoints ----
// A group's step is the smallest power of two 2^k with amax <= 127 * 2^k, and
// at least 2^-126; the exponent byte is k + 127.  From the bits of amax =
// (1 + f) 2^E: k = E - 6 while 1 + f <= 127 / 64 (f <= 0x7E0000 / 2^23), else
// E - 5.  A group that holds an infinity or a NaN gets byte 255 and codes 0,
// which decode to 0 * inf = NaN.
__device__ __forceinline__ uint32_t act8_exp(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = int(b >> 23) - 6 + ((b & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return b >= 0x7F800000u ? 255u : uint32_t(e < 1 ? 1 : e);
}
// Maximum of magnitudes that keeps a NaN (as bits: NaN > inf > finite).
__device__ __forceinline__ float max_mag(float a, float b) {
    const uint32_t x = __float_as_uint(a) & 0x7FFFFFFFu, y = __float_as_uint(b) & 0x7FFFFFFFu;
    return __uint_as_float(x > y ? x : y);
}
// 2^(127 - byte): the exact multiplier of the encoding (byte 1 .. 249).
__device__ __forceinline__ float act8_inv(uint32_t e) { return __uint_as_float((254u - e) << 23); }
__device__ __forceinline__ float act8_step(uint32_t e) { return __uint_as_float(e << 23); }
__device__ __forceinline__ uint32_t act8_code(float v, uint32_t e) {   // round to nearest even, as a byte
    return e == 255u ? 0u : uint32_t(int(__builtin_rintf(v * act8_inv(e)))) & 0xFFu;
}
// The four codes of a word times the step.
__device__ __forceinline__ void act8_dec4(uint32_t w, float step, float* v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = float(int(int8_t(w >> (8 * k)))) * step;
}

// ---- activations ----
// GELU in the tanh form, z s(u) with u = 2 sqrt(2/pi) (z + 0.044715 z^3) and
// the logistic s (0.5 (1 + tanh(u / 2)) = s(u)).  exp and the reciprocal are
// the hardware's, good to a unit in the last place; s(1 - s)|u| <= 0.23 keeps
// the rounding of u out of the result.
constexpr float kGeluU = 1.5957691216057308f;      // 2 sqrt(2 / pi)
constexpr float kGeluC = 0.044715f;

// exp(-u(z)) as 2^x: x = -log2(e) u, its constants folded.
constexpr float kGeluE1 = -2.302208198144325f;     // -2 sqrt(2 / pi) log2(e)
constexpr float kGeluE3 = -0.10294323958002269f;   // and times 0.044715
__device__ __forceinline__ float gelu_exp(float z) {
    return __builtin_amdgcn_exp2f(z * fmaf(kGeluE3 * z, z, kGeluE1));
}
// The product of which a factor 0 makes 0, also beside an infinity: GELU's
// limit at -infinity, where the logistic is 0, without an instruction more (a
// maximum of z with a bound cost the 8192 x 4096 forward epilogue 1.0 us of
// 75.7).  A NaN z stays: its logistic is NaN too.
#ifdef __HIP__
extern "C" __device__ float muon_fmul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");   // v_mul_legacy_f32
__device__ __forceinline__ float mul_zero(float a, float b) { return muon_fmul_legacy(a, b); }
#else   // a host build for checking
inline float mul_zero(float a, float b) { return a == 0.f || b == 0.f ? 0.f : a * b; }
#endif
__device__ __forceinline__ float act_value(float z, int act) {
    if (act == ACT_GELU) return mul_zero(z, __builtin_amdgcn_rcpf(1.f + gelu_exp(z)));
    if (act == ACT_RELU_SQ) return z <= 0.f ? 0.f : z * z;   // a NaN stays one
    return z;
}
// Value and derivative.  With e = exp(-u), s = 1 / (1 + e) and 1 - s = e s (no
// cancellation).  Beyond |z| = 9 the logistic is 0 or 1 to float32 (e^66 or
// e^-66 away): z is held there, by a minimum and a maximum that keep a NaN, so
// that nothing can overflow, and under -9 s is set to 0.  So infinities give
// the limits, as in act_value.
__device__ __forceinline__ void act_both(float z, int act, float& v, float& d) {
    if (act == ACT_GELU) {
        const float c = __builtin_elementwise_maximum(__builtin_elementwise_minimum(z, 9.f), -9.f), c2 = c * c;
        const float e = __builtin_amdgcn_exp2f(c * fmaf(kGeluE3, c2, kGeluE1));
        const float s = z < -9.f ? 0.f : __builtin_amdgcn_rcpf(1.f + e);
        v = mul_zero(z, s);
        d = fmaf((c * s) * (e * s), fmaf(3.f * kGeluC * kGeluU, c2, kGeluU), s);
    } else if (act == ACT_RELU_SQ) {
        v = z <= 0.f ? 0.f : z * z;
        d = z <= 0.f ? 0.f : 2.f * z;
    } else {
        v = z;
        d = 1.f;
    }
}

__device__ __forceinline__ float wave_add(float v) {
#pragma unroll
    for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
    return v;
}

}  // namespace layer
}  // namespace muon
