// Rows of values to MXFP4 and back (the format: mxfp4.hpp).
//
// Both read and write each byte once (4 or 2 and 0.53 bytes per element) and
// do next to nothing with it: HBM bounds large arrays, launch latency small ones.
// Measured: 2048 x 14336 f32 to MXFP4 (133 MB) 25.6 us, 5.2 TB/s, and back 21.0
// us, 6.3 TB/s; a row of 1024 1.4 us.
#include "mxfp4.hpp"

namespace qmm {

namespace {

constexpr int THREADS = 256;

template <int TYPE>
__device__ __forceinline__ void load8(const char* x, int64_t at, f32x4* lo, f32x4* hi) {
    if constexpr (TYPE == MX_F32) {
        *lo = *(const f32x4*)(x + 4 * at);
        *hi = *(const f32x4*)(x + 4 * at + 16);
    } else {
        const u32x4 v = *(const u32x4*)(x + 2 * at);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = v[j];
            float a, b;
            if constexpr (TYPE == MX_F16) {
                a = f16lo(w);
                b = f16hi(w);
            } else {
                a = __builtin_bit_cast(float, w << 16);
                b = __builtin_bit_cast(float, w & 0xffff0000u);
            }
            f32x4* t = j < 2 ? lo : hi;
            (*t)[2 * (j & 1)] = a;
            (*t)[2 * (j & 1) + 1] = b;
        }
    }
}

// A thread takes eight values, four lanes a block.
template <int TYPE>
__global__ __launch_bounds__(THREADS) void quantize_mxfp4_kernel(uint8_t* q, uint8_t* e, const char* x, int64_t ldx,
                                                                 int64_t items, int per_row) {
    for (int64_t it = (int64_t)blockIdx.x * THREADS + threadIdx.x; it < items; it += (int64_t)gridDim.x * THREADS) {
        const int64_t row = items <= UINT32_MAX ? (uint32_t)it / (uint32_t)per_row : it / per_row;
        f32x4 lo, hi;
        load8<TYPE>(x, row * ldx + 8 * (it - row * per_row), &lo, &hi);
        const uint32_t byte = mx_scale_byte(mx_quad_max(mx_max8(lo, hi)));
        ((uint32_t*)q)[it] = mx_codes8(lo, hi, byte);
        if ((it & 3) == 0) e[it >> 2] = (uint8_t)byte;
    }
}

// A thread takes four values, so that a wave's stores are whole lines.
__global__ __launch_bounds__(THREADS) void dequantize_mxfp4_kernel(float* x, const uint8_t* q, const uint8_t* e,
                                                                   int64_t items) {
    for (int64_t it = (int64_t)blockIdx.x * THREADS + threadIdx.x; it < items; it += (int64_t)gridDim.x * THREADS) {
        const uint32_t c = ((const uint16_t*)q)[it];
        const float s = mx_scale(e[it >> 3]);
        const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
        ((f32x4*)x)[it] = f32x4{a.x, a.y, b.x, b.y};
    }
}

unsigned blocks_for(int64_t items) {
    const int64_t b = (items + THREADS - 1) / THREADS;
    return (unsigned)(b < (1 << 22) ? b : 1 << 22);  // fewer than 2^32 threads; more items: several each
}

}  // namespace

void launch_quantize_mxfp4(uint8_t* q, uint8_t* e, const void* x, int type, int64_t ldx, int64_t rows, int64_t k,
                           hipStream_t st) {
    const int64_t items = rows * (k / 8);
    const int per_row = (int)(k / 8);
    const unsigned grid = blocks_for(items);
    if (type == MX_F32)
        quantize_mxfp4_kernel<MX_F32><<<grid, THREADS, 0, st>>>(q, e, (const char*)x, ldx, items, per_row);
    else if (type == MX_F16)
        quantize_mxfp4_kernel<MX_F16><<<grid, THREADS, 0, st>>>(q, e, (const char*)x, ldx, items, per_row);
    else
        quantize_mxfp4_kernel<MX_BF16><<<grid, THREADS, 0, st>>>(q, e, (const char*)x, ldx, items, per_row);
}

void launch_dequantize_mxfp4(float* x, const uint8_t* q, const uint8_t* e, int64_t elems, hipStream_t st) {
    dequantize_mxfp4_kernel<<<blocks_for(elems / 4), THREADS, 0, st>>>(x, q, e, elems / 4);
}

}  // namespace qmm
