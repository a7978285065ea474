// act8.cuh -- the 8-bit activation checkpoint format (muon_act8 in muon.h):
// device code shared by the kernels that write it (act8.cu, seam.cu) and read
// it (act8.cu, act8_grad.cu, seam.cu), and the host checks of its arguments.
//
// A block of 32 columns of one row holds x as q 2^e, e the smallest exponent
// in [kActExpMin, kActExpMax] with max|x| <= 127 2^e and q = rne(x 2^-e).  The
// scale is a power of two so that q 2^e has 7 significant bits: exact as a
// bfloat16 tensor-core operand, where a general fp32 scale would round every
// value a second time (2^-9 relative) or need the scale outside the sum over
// tokens, which a scale per token and block cannot have.  It costs at most one
// bit of resolution against the general scale.
#pragma once

#include "muon_internal.cuh"

namespace muon {

constexpr int kActBlock = 32;
constexpr int kActExpMin = -120, kActExpMax = 119;
constexpr int kActMaxDim = 1 << 30; // rows, columns, outputs: sums of a few of them with tile sizes stay ints
constexpr int kActBad = 255;        // exponent byte of a block that stands for NaNs

__host__ __device__ inline int act8_blocks(int cols) { return (cols + kActBlock - 1) / kActBlock; }

// Exponent byte of a block whose largest magnitude has the bits m: with
// max = f 2^E (1 <= f < 2), 127 2^(E-6) = (127/64) 2^E holds it unless f > 127/64.
__device__ __forceinline__ int act8_exp_byte(uint32_t m) {
    const int e = (int)(m >> 23) - 127 - 6 + ((m & 0x7FFFFFu) > 0x7E0000u ? 1 : 0);
    return e > kActExpMax ? kActBad : max(e, kActExpMin) + 127;
}

// 2^e and 2^-e of a valid exponent byte.
__device__ __forceinline__ float act8_scale(int byte) { return __uint_as_float((uint32_t)byte << 23); }
__device__ __forceinline__ float act8_inv(int byte) { return __uint_as_float((uint32_t)(254 - byte) << 23); }

// Codes of four values.  x 2^-e is exact, so the fused multiply-add onto 1.5 2^23
// rounds once, to the nearest whole number (ties to even), whose two's
// complement is the sum's low byte.
__device__ __forceinline__ uint32_t act8_codes4(float a, float b, float c, float d, float inv) {
    const float magic = 12582912.f;
    const uint32_t ua = __float_as_uint(__fmaf_rn(a, inv, magic)), ub = __float_as_uint(__fmaf_rn(b, inv, magic));
    const uint32_t uc = __float_as_uint(__fmaf_rn(c, inv, magic)), ud = __float_as_uint(__fmaf_rn(d, inv, magic));
    return __byte_perm(__byte_perm(ua, ub, 0x0040), __byte_perm(uc, ud, 0x0040), 0x5410);
}

// 32 bytes in one store: a whole sector, where two stores of 16 write it half by half.
__device__ __forceinline__ void st_global_v8(void* p, const uint4& a, const uint4& b) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
                 "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w) : "memory");
}

// Eight consecutive elements as they lie in memory (16-byte aligned): loaded without
// a branch (zeros where not `ok`), so that loads can be in flight together, and
// turned into floats where they are used.
template <int DT> struct Raw8 {
    static constexpr int N = DT == DT_FP32 ? 2 : 1;
    uint4 w[N];
    __device__ __forceinline__ void load(const void* p, bool ok) {
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = ok ? static_cast<const uint4*>(p)[i] : make_uint4(0u, 0u, 0u, 0u);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const {
        if constexpr (DT == DT_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v[4 * i] = __uint_as_float(w[i].x); v[4 * i + 1] = __uint_as_float(w[i].y);
                v[4 * i + 2] = __uint_as_float(w[i].z); v[4 * i + 3] = __uint_as_float(w[i].w);
            }
        } else {
            const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (DT == DT_BF16) {
                    v[2 * i] = __uint_as_float(u[i] << 16);
                    v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                } else {
                    v[2 * i] = unpack_lo<__half>(u[i]);
                    v[2 * i + 1] = unpack_hi<__half>(u[i]);
                }
            }
        }
    }
    __device__ __forceinline__ void set(const float (&v)[8]) {
        if constexpr (DT == DT_FP32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                w[i] = make_uint4(__float_as_uint(v[4 * i]), __float_as_uint(v[4 * i + 1]), __float_as_uint(v[4 * i + 2]),
                                  __float_as_uint(v[4 * i + 3]));
        } else {
            uint32_t u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = DT == DT_BF16 ? pack2<__nv_bfloat16>(v[2 * i], v[2 * i + 1]) : pack2<__half>(v[2 * i], v[2 * i + 1]);
            w[0] = make_uint4(u[0], u[1], u[2], u[3]);
        }
    }
    // wide: p is 32-byte aligned, and fp32 is stored in whole sectors
    __device__ __forceinline__ void store(void* p, bool ok, bool wide = false) const {
        if (!ok) return;
        if constexpr (DT == DT_FP32) {
            if (wide) {
                st_global_v8(p, w[0], w[1]);
                return;
            }
        }
#pragma unroll
        for (int i = 0; i < N; ++i) static_cast<uint4*>(p)[i] = w[i];
    }
};

// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max3_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}

// Exponent byte and codes (two words) of eight columns of a block, its four lanes in step (every lane of
// the warp takes part; columns past the row given as 0): the block's largest
// magnitude by two shuffles.
__device__ __forceinline__ int act8_quantise8(const float (&x)[8], uint2& w) {
    float m = fabsf(x[0]);
    m = max3_abs(m, x[1], x[2]);
    m = max3_abs(m, x[3], x[4]);
    m = max3_abs(m, x[5], x[6]);
    m = max3_abs(m, x[7], x[7]);
    m = max3_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1), 0.f);
    m = max3_abs(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2), 0.f);
    const int byte = act8_exp_byte(__float_as_uint(m));
    const float inv = act8_inv(byte);
    w.x = act8_codes4(x[0], x[1], x[2], x[3], inv);
    w.y = act8_codes4(x[4], x[5], x[6], x[7], inv);
    if (byte == kActBad) w = make_uint2(0u, 0u);
    return byte;
}

// The same, stored: the codes at qrow + col, and by the block's first lane the
// exponent byte.  Returns false for a block that cannot be held.
__device__ __forceinline__ bool act8_encode8(const float (&x)[8], int col, int nvalid, signed char* qrow,
                                             unsigned char* erow, int lane) {
    uint2 w;
    const int byte = act8_quantise8(x, w);
    if (nvalid >= 8) {
        *reinterpret_cast<uint2*>(qrow + col) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < nvalid) qrow[col + i] = (signed char)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
    }
    if ((lane & 3) == 0 && nvalid > 0) erow[col / kActBlock] = (unsigned char)byte;
    return byte != kActBad;
}

// Eight codes (two words) as whole floats.  A code's byte with the sign bit flipped is
// q + 128, as the low bits of a float 2^23 + 128 + q; the difference is q (a conversion
// instruction per code would take four times the issue time).
__device__ __forceinline__ void act8_whole8(uint2 w, float (&q)[8]) {
    const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        q[i] = __uint_as_float(__byte_perm(u[i >> 2], 0x4B000000u, 0x7440 + (i & 3))) - 8388736.f;
}

// 2^e of an exponent byte, NaN for a bad block's.
__device__ __forceinline__ float act8_step(int byte) {
    return byte == kActBad ? __uint_as_float(0x7FC00000u) : act8_scale(byte);
}

// The values of eight codes under an exponent byte.
__device__ __forceinline__ void act8_decode8(uint2 w, int byte, float (&v)[8]) {
    const float s = act8_step(byte);
    act8_whole8(w, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= s;
}

// A checkpoint's value as fp16 takes it.  fp16 values from 65024 on lie in a block of e = 10 and
// are held as 64 2^10 = 65536, which rounds to infinity; fp16's largest value, 65504, is as close to what
// 65536 stands for (half a step, 512, around it).  65536 is the only value of an fp16 tensor's checkpoint beyond that range.
constexpr int kActFp16Top = 127 + 10;   // smallest exponent byte under which it occurs
__device__ __forceinline__ float act8_fp16(float v) { return fabsf(v) == 65536.f ? copysignf(65504.f, v) : v; }

// Host: whether a checkpoint's fields can be used (an empty one needs no pointers).
inline bool act8_valid(const muon_act8& c) {
    if (c.rows < 0 || c.rows > kActMaxDim || c.cols < 1 || c.cols > kActMaxDim || c.ldq < c.cols || c.ldq % 16 != 0 || c.lde < act8_blocks(c.cols)) return false;
    if (c.rows == 0) return true;
    return c.q && c.e && (reinterpret_cast<uintptr_t>(c.q) & 15) == 0;
}

// Host: 16-byte accesses of rows of `esz`-byte elements are allowed.
inline bool rows_aligned(const void* p, long long ld, int esz) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (ld * esz) % 16 == 0;
}

muon_status check_device();     // muon_api.cu: the current device runs sm_100 code

}  // namespace muon
