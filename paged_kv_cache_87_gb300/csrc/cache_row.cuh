// cache_row.cuh -- eight consecutive head dims of one cached row, for every cache type.
//
// The kernels that write the cache (reshape_and_cache into 4 bits, the fused norm +
// rotary + write) and the one that reads it back give a lane eight consecutive dims, 8j ..
// 8j + 7, of a row: one 16-byte access of a 16-bit source, one 4-byte word of 4-bit codes.
// CacheRow<KT> moves those eight between registers (fp32) and the (block, kv head) tile.
#pragma once

#include <type_traits>

#include "common.cuh"

namespace pkv {

// 4-bit cache: e2m1 codes with an e4m3 scale for every 16 dims (pagedkv.h has the layout).
struct E2M1 {
    static constexpr pkv_dtype code = PKV_FP4_E2M1;
};

// Bytes of one row of a cache of the given type (scales included).
inline int64_t cache_row_bytes(pkv_dtype t, int head_dim) {
    switch (t) {
    case PKV_F32: return (int64_t)head_dim * 4;
    case PKV_F16: case PKV_BF16: return (int64_t)head_dim * 2;
    case PKV_FP8_E4M3: return head_dim;
    case PKV_FP4_E2M1: return head_dim / 2 + head_dim / 16;
    default: return 0;
    }
}

template <typename KT>
constexpr bool is_quantised() {
    return std::is_same<KT, E4M3>::value || std::is_same<KT, E2M1>::value;
}

template <typename KT>
__host__ __device__ constexpr int cache_row_bytes_of(int head_dim) {
    if constexpr (std::is_same<KT, E2M1>::value) return head_dim / 2 + head_dim / 16;
    else return head_dim * KT::bytes;
}

// Two fp32 values -> two e4m3 codes (round to nearest even, saturate to
// +-448, NaN -> NaN), packed little-endian: `lo` lands in the lower byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low byte first) -> f16x2 (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_codes) {
    __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two_codes),
                                               __NV_E4M3);
    return *reinterpret_cast<uint32_t*>(&h);
}

// The same of the low (HALF = 0) or high half of a word of four codes.
template <int HALF>
__device__ __forceinline__ uint32_t e4m3x2_of(uint32_t w) {
    uint32_t r;
    if constexpr (HALF == 0)
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}"
            : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}"
            : "=r"(r) : "r"(w));
    return r;
}

// Element-wise product of two f16x2.
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The low (k = 0) or high half of an f16x2 in both halves (an operand modifier, not an operation).
__device__ __forceinline__ uint32_t half_twice(uint32_t x, int k) {
    const __half2 h = *reinterpret_cast<const __half2*>(&x);
    const __half2 t = k ? __high2half2(h) : __low2half2(h);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// Eight fp32 values -> e2m1 codes (round to nearest even, saturate to +-6), the first in the
// lowest nibble.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float (&q)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
    return r;
}

// Byte 0..3 of a word of e2m1 codes -> f16x2 (exact), the low nibble in the low half.
template <int BYTE>
__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t w) {
    uint32_t r;
    if constexpr (BYTE == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (BYTE == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (BYTE == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\t"
            "cvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// max of |a| and b, NaN if either is (fmaxf would drop it)
__device__ __forceinline__ float absmax_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(b));
    return r;
}

// Eight consecutive source elements (16 bytes of a 16-bit type, 32 of fp32) <-> fp32.
template <typename ST>
__device__ __forceinline__ void load8(const void* src, float (&f)[8]) {
    const uint4* s = static_cast<const uint4*>(src);
    Chunk<ST>::to_float(s[0], f);
    if constexpr (ST::bytes == 4) Chunk<ST>::to_float(s[1], f + 4);
}

template <typename ST>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    static_assert(ST::bytes == 2, "16-bit types");
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<ST, F16>::value) {
            __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        } else {
            __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<uint32_t*>(&h);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename ST>
__device__ __forceinline__ void store8(void* dst, const float (&f)[8]) {
    uint4* d = static_cast<uint4*>(dst);
    if constexpr (ST::bytes == 4) {
        d[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                          __float_as_uint(f[3]));
        d[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]),
                          __float_as_uint(f[7]));
    } else {
        d[0] = pack8<ST>(f);
    }
}

// One row of a cache of type KT: dims 8j .. 8j + 7 of row `row` of the (block, kv head)
// tile at `tile` (B rows, d dims).  Of the quantised types, store() is called by all 32 lanes of a
// warp together, lanes 2i and 2i + 1 holding the two halves of one 16-dim group; only `live` lanes
// write; values() are chunk c's eight values, before kv_scale.
// A cache of the rows' own type takes them as they are stored: put() and copy() move bits, which
// a way through fp32 would not (a 16-bit NaN comes back from it without its sign and payload).
template <typename KT>
struct CacheRow {
    static constexpr int N16 = KT::bytes / 2;      // 16-byte pieces of eight dims
    __device__ __forceinline__ static void put(uint8_t* tile, int d, int row, int j, const uint4 (&x)[N16]) {
        uint4* to = reinterpret_cast<uint4*>(tile + ((int64_t)row * d + 8 * j) * KT::bytes);
#pragma unroll
        for (int i = 0; i < N16; ++i) to[i] = x[i];
    }
    // a quarter of a row: dims 32c + 8w .. + 7 of every 32-dim chunk c, as stored
    template <int HD>
    struct Raw {
        uint4 x[HD / 32 * N16];
    };
    template <int HD>
    __device__ __forceinline__ static void fetch(const uint8_t* tile, int B, int row, int w,
                                                 Raw<HD>& r) {
        const uint4* s = reinterpret_cast<const uint4*>(tile + ((int64_t)row * HD + 8 * w) * KT::bytes);
#pragma unroll
        for (int c = 0; c < HD / 32; ++c)
#pragma unroll
            for (int i = 0; i < N16; ++i) r.x[N16 * c + i] = s[4 * N16 * c + i];
    }
    // the quarter into a row of the same type
    template <int HD>
    __device__ __forceinline__ static void copy(const Raw<HD>& r, int w, uint8_t* row) {
        uint4* to = reinterpret_cast<uint4*>(row + 8 * w * KT::bytes);
#pragma unroll
        for (int c = 0; c < HD / 32; ++c)
#pragma unroll
            for (int i = 0; i < N16; ++i) to[4 * N16 * c + i] = r.x[N16 * c + i];
    }
};

template <>
struct CacheRow<E4M3> {
    __device__ __forceinline__ static void store(uint8_t* tile, int B, int d, int row, int j,
                                                 const float (&f)[8], float kv_scale, bool live) {
        uint32_t w[2];
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = cvt_e4m3x2(__fdiv_rn(f[4 * i], kv_scale), __fdiv_rn(f[4 * i + 1], kv_scale)) |
                   (cvt_e4m3x2(__fdiv_rn(f[4 * i + 2], kv_scale),
                               __fdiv_rn(f[4 * i + 3], kv_scale)) << 16);
        if (live) *reinterpret_cast<uint2*>(tile + (int64_t)row * d + 8 * j) = make_uint2(w[0], w[1]);
    }
    template <int HD>
    struct Raw {
        uint2 x[HD / 32];
    };
    template <int HD>
    __device__ __forceinline__ static void fetch(const uint8_t* tile, int B, int row, int w,
                                                 Raw<HD>& r) {
#pragma unroll
        for (int c = 0; c < HD / 32; ++c)
            r.x[c] = *reinterpret_cast<const uint2*>(tile + (int64_t)row * HD + 32 * c + 8 * w);
    }
    template <int HD>
    __device__ __forceinline__ static void values(const Raw<HD>& r, int c, int, float (&f)[8]) {
        const uint32_t w[2] = {r.x[c].x, r.x[c].y};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t h = e4m3x2_to_f16x2((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
            f[2 * i] = v.x;
            f[2 * i + 1] = v.y;
        }
    }
};

template <>
struct CacheRow<E2M1> {
    __device__ __forceinline__ static int code_at(int B, int row, int j) {
        return ((j >> 2) * B + row) * 16 + (j & 3) * 4;
    }
    __device__ __forceinline__ static int scale_at(int B, int d, int row, int j) {
        return B * (d / 2) + row * (d / 16) + (j >> 1);
    }
    // The scale of a group whose largest magnitude is amax (NaN if it holds one): its e4m3 code,
    // and what its codes' quotients need.
    struct Scale {
        uint32_t code;
        float step, inverse;    // scale * kv_scale, and its correctly rounded reciprocal
        bool near;              // every term of a quotient below stays in the normal range
        __device__ __forceinline__ Scale(float amax, float kv_scale) {
            code = cvt_e4m3x2(__fdiv_rn(amax, 6.0f * kv_scale), 0.f) & 0xffu;
            const uint32_t h = e4m3x2_to_f16x2(code);
            step = __low2float(*reinterpret_cast<const __half2*>(&h)) * kv_scale;
            inverse = __frcp_rn(step);
            near = step > 0x1p-100f && step < 0x1p100f && amax * inverse < 0x1p20f;
        }
    };
    // Eight codes: e2m1(x / step), zeros for a scale of 0 or NaN.  x / step is correctly rounded,
    // from the correctly rounded reciprocal y: q = x y, r = q step - x (exact in a fused
    // multiply-add), q - r y (P. Markstein, IBM J. Res. Dev. 34, 1990); with r of this sign a zero
    // keeps its own.  Three operations instead of a division each; where a term could leave the
    // normal range (a saturated group, far scales) the division.
    __device__ __forceinline__ static uint32_t codes8(const float* f, const Scale& s) {
        float q[8];
        if (s.near) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = f[i] * s.inverse;
                q[i] = fmaf(-fmaf(t, s.step, -f[i]), s.inverse, t);
            }
        } else if (s.step > 0.f) {
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(f[i], s.step);
        } else {
            return 0u;
        }
        return cvt_e2m1x8(q);
    }
    __device__ __forceinline__ static void store(uint8_t* tile, int B, int d, int row, int j,
                                                 const float (&f)[8], float kv_scale, bool live) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = absmax_nan(f[i], amax);
        amax = absmax_nan(__shfl_xor_sync(0xffffffffu, amax, 1), amax);
        const Scale s(amax, kv_scale);
        const uint32_t w = codes8(f, s);
        if (live) {
            *reinterpret_cast<uint32_t*>(tile + code_at(B, row, j)) = w;
            if ((j & 1) == 0) tile[scale_at(B, d, row, j)] = (uint8_t)s.code;
        }
    }
    // A whole group, dims 16g .. 16g + 15, by one lane: the same bytes.
    __device__ __forceinline__ static void store_group(uint8_t* tile, int B, int d, int row, int g,
                                                       const float (&f)[16], float kv_scale) {
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = absmax_nan(f[i], amax);
        const Scale s(amax, kv_scale);
        *reinterpret_cast<uint2*>(tile + code_at(B, row, 2 * g)) =
            make_uint2(codes8(f, s), codes8(f + 8, s));
        tile[scale_at(B, d, row, 2 * g)] = (uint8_t)s.code;
    }
    template <int HD>
    struct Raw {
        uint32_t w[HD / 32], scales[HD / 64];       // this lane's words, the row's scales
    };
    template <int HD>
    __device__ __forceinline__ static void fetch(const uint8_t* tile, int B, int row, int w,
                                                 Raw<HD>& r) {
#pragma unroll
        for (int c = 0; c < HD / 32; ++c)
            r.w[c] = *reinterpret_cast<const uint32_t*>(tile + (c * B + row) * 16 + 4 * w);
        const uint8_t* s = tile + B * (HD / 2) + row * (HD / 16);
        if constexpr (HD == 128) {
            const uint2 v = *reinterpret_cast<const uint2*>(s);
            r.scales[0] = v.x;
            r.scales[1] = v.y;
        } else {
            r.scales[0] = *reinterpret_cast<const uint32_t*>(s);
        }
    }
    template <int HD>
    __device__ __forceinline__ static void values(const Raw<HD>& r, int c, int w, float (&f)[8]) {
        const int byte = 2 * c + (w >> 1);
        const uint32_t sh = e4m3x2_to_f16x2((r.scales[c >> 1] >> (8 * (byte & 3))) & 0xffu);
        const float s = __low2float(*reinterpret_cast<const __half2*>(&sh));
        const uint32_t x = r.w[c];
        const uint32_t h[4] = {e2m1x2_to_f16x2<0>(x), e2m1x2_to_f16x2<1>(x),
                               e2m1x2_to_f16x2<2>(x), e2m1x2_to_f16x2<3>(x)};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
            f[2 * i] = v.x * s;       // exact: 2 + 4 significant bits
            f[2 * i + 1] = v.y * s;
        }
    }
};

}  // namespace pkv
