// Microscaled 4-bit floats (MXFP4, the OCP MX format): E2M1 codes, element 2j
// in the low nibble of byte j, and one E8M0 scale byte per 32 consecutive
// values of a row, an element being code * 2^(byte - 127); byte 255 is NaN.
//
// From values x the scale is e = floor(log2 max|x|) - 2 (the largest code, 6,
// has the exponent 2), at least -127, and the codes are x * 2^-e rounded to
// nearest even, those above 6 saturated: v_cvt_scalef32_pk_fp4_f32 does just
// that, for every scale and every tie (compared on the borders between all
// codes and their neighbours, scales 2^-127 to 2^127).  A block with an
// infinity or a NaN gets the scale byte 255 and codes 0, so that it stays visible.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace qmm {

constexpr int KV_MX4 = 4;  // QMM_KV_MXFP4
enum : int { MX_F32 = 0, MX_F16 = 1, MX_BF16 = 2 };  // qmm_mx_type

__device__ __forceinline__ uint32_t mx_magnitude(float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t mx_larger(uint32_t x, uint32_t y) { return x > y ? x : y; }

// The scale byte of a block whose largest magnitude has these bits (an
// infinity and then NaN are the largest of all).
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t bits) {
    const uint32_t e = bits >> 23;
    return e == 255 ? 255u : e > 2 ? e - 2 : 0u;
}
// A scale byte as the scaled conversions take it: they read an f32's exponent
// field alone (compared over all 256 with other signs and mantissas), 0 being
// 2^-127 and 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }
// The codes of four values over their block's scale, element 0 lowest.
__device__ __forceinline__ uint32_t mx_codes4(f32x4 x, uint32_t byte) {
    const float s = mx_scale(byte);
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x.x, x.y, s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x.z, x.w, s, 1);
    return byte == 255 ? 0u : c;
}
__device__ __forceinline__ uint32_t mx_codes8(f32x4 lo, f32x4 hi, uint32_t byte) {
    const float s = mx_scale(byte);
    uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, lo.x, lo.y, s, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, lo.z, lo.w, s, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, hi.x, hi.y, s, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, hi.z, hi.w, s, 3);
    return byte == 255 ? 0u : c;
}
// The largest of the four lanes of a quad, in each of them.
__device__ __forceinline__ uint32_t mx_quad_max(uint32_t v) {
    v = mx_larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xb1, 0xf, 0xf, true));  // quad_perm [1, 0, 3, 2]
    return mx_larger(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4e, 0xf, 0xf, true));  // [2, 3, 0, 1]
}
__device__ __forceinline__ uint32_t mx_max8(f32x4 lo, f32x4 hi) {
    uint32_t b = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) b = mx_larger(b, mx_larger(mx_magnitude(lo[j]), mx_magnitude(hi[j])));
    return b;
}

// Rows of k values, ldx elements apart, to codes and scales, and back.
void launch_quantize_mxfp4(uint8_t* q, uint8_t* e, const void* x, int type, int64_t ldx, int64_t rows, int64_t k,
                           hipStream_t st);
void launch_dequantize_mxfp4(float* x, const uint8_t* q, const uint8_t* e, int64_t elems, hipStream_t st);

// dst[j*ldd + i] = s[j] * sum_c W[i][c] X[j][c] (s null: 1)
struct MxGemmArgs {
    float* dst;
    const uint8_t *wq, *we, *xq, *xe;
    const float* s;
    int64_t ldd;
    int m, n, k;
};
// forced: the kernel to take where it can (tests and sweeps), or -1.
void launch_gemm_mxfp4(const MxGemmArgs& a, int forced, int num_cu, hipStream_t st);
int gemm_mxfp4_kernels();  // how many there are

// The norm to MXFP4: codes of h * weight in q, their scales in e, 1/rms in d.
struct NormMxArgs : NormArgs {
    uint8_t* e;
};
void launch_add_rmsnorm_mxfp4(const NormMxArgs& a, int num_cu, hipStream_t st);

}  // namespace qmm
