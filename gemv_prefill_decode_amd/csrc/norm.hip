// RMS norm with the residual's addition, to f32 or to Q8_1 activations.
//
//     h = x + r,  y = h * w / sqrt(mean(h^2) + eps)
//
// One pass: a row's elements stay in registers between the sum of squares and
// the output, so each input is read once and each output written once (16
// bytes per element with a residual and f32 output, 13.1 with Q8_1): HBM
// bounds many rows, launch and load latency few.
//
// Q8_1 output: 1/rms is one factor of a whole row, so a block's codes are
// those of z = h * w, d0 = max|z| / 127, q = round(z * (1/d0)) (halves away
// from zero, every step in f32 as qmm_quantize_q8_1), and its scale is d0/rms:
// the codes do not depend on the order in which the squares were added.
#include <type_traits>

#include "common.hpp"
#include "kernels.hpp"

namespace qmm {

namespace {

// Sum over T consecutive lanes (a power of two up to 64), the same in each.
template <int T>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int s = 1; s < T; s <<= 1) v += __shfl_xor(v, s);
    return v;
}

__device__ __forceinline__ float dot4(f32x4 v) { return v.x * v.x + v.y * v.y + v.z * v.z + v.w * v.w; }

// The Q8_1 codes of a block held by eight consecutive lanes, four values each.
__device__ __forceinline__ uint32_t codes4(f32x4 z, float* d0) {
    float top = fmaxf(fmaxf(fabsf(z.x), fabsf(z.y)), fmaxf(fabsf(z.z), fabsf(z.w)));
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
    float dd = top / 127.0f;
    if (dd < 1.17549435e-38f) dd = 0.0f;  // its inverse would overflow
    const float id = dd != 0.0f ? 1.0f / dd : 0.0f;
    *d0 = dd;
    return (uint32_t)(uint8_t)(int8_t)(int)roundf(z.x * id) | ((uint32_t)(uint8_t)(int8_t)(int)roundf(z.y * id) << 8) |
           ((uint32_t)(uint8_t)(int8_t)(int)roundf(z.z * id) << 16) | ((uint32_t)(uint8_t)(int8_t)(int)roundf(z.w * id) << 24);
}

// THREADS threads per work group, T of them per row, V float4 per thread: a
// row of up to 4*T*V elements.  LOOP: longer rows, read a second time.
template <int THREADS, int T, int V, bool Q8, bool LOOP>
__global__ __launch_bounds__(THREADS) void add_rmsnorm_kernel(const NormArgs a) {
    constexpr int ROWS = THREADS / T;
    __shared__ float wave_sum[THREADS / 64];
    const int tid = threadIdx.x, at = tid % T, nv = a.k / 4;
    const int64_t row = (int64_t)blockIdx.x * ROWS + tid / T;
    const bool live = row < a.n;
    const f32x4* x = (const f32x4*)(a.x + (live ? row : 0) * a.x_stride);
    const f32x4* r = a.r ? (const f32x4*)(a.r + (live ? row : 0) * a.r_stride) : nullptr;
    const f32x4* w = (const f32x4*)a.w;
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 h[V], wt[V];
    float sum = 0.0f;
    const int span = LOOP ? (nv + T * V - 1) / (T * V) * (T * V) : T * V;
    for (int base = 0; base < span; base += T * V) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = base + i * T + at;
            h[i] = live && e < nv ? x[e] : zero;
            if (r) h[i] += live && e < nv ? r[e] : zero;
            if constexpr (!LOOP) wt[i] = e < nv ? w[e] : zero;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = base + i * T + at;
            if (a.h && live && e < nv) ((f32x4*)(a.h + row * a.h_stride))[e] = h[i];
            sum += dot4(h[i]);
        }
    }
    if constexpr (T <= 64) {
        sum = lanes_sum<T>(sum);
    } else {
        sum = lanes_sum<64>(sum);
        if ((tid & 63) == 0) wave_sum[tid >> 6] = sum;
        __syncthreads();
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < THREADS / 64; ++i) sum += wave_sum[i];
    }
    const float inv = 1.0f / sqrtf(sum * a.inv_k + a.eps);
    for (int base = 0; base < span; base += T * V) {
        if constexpr (LOOP) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const int e = base + i * T + at;
                h[i] = live && e < nv ? x[e] : zero;
                if (r) h[i] += live && e < nv ? r[e] : zero;
                wt[i] = e < nv ? w[e] : zero;
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = base + i * T + at;
            if constexpr (Q8) {
                float d0;
                const uint32_t c = codes4(h[i] * wt[i], &d0);
                if (live && e < nv) {
                    ((uint32_t*)a.q)[row * nv + e] = c;
                    if ((e & 7) == 0) a.d[(row * nv + e) / 8] = d0 * inv;
                }
            } else if (live && e < nv) {
                ((f32x4*)(a.y + row * a.y_stride))[e] = h[i] * inv * wt[i];
            }
        }
    }
}

template <int THREADS, int T, int V, bool LOOP = false>
void launch(const NormArgs& a, hipStream_t st) {
    constexpr int ROWS = THREADS / T;
    const dim3 grid((unsigned)((a.n + ROWS - 1) / ROWS));
    if (a.q)
        add_rmsnorm_kernel<THREADS, T, V, true, LOOP><<<grid, THREADS, 0, st>>>(a);
    else
        add_rmsnorm_kernel<THREADS, T, V, false, LOOP><<<grid, THREADS, 0, st>>>(a);
}

}  // namespace

void launch_add_rmsnorm(const NormArgs& a, hipStream_t st) {
    const int nv = a.k / 4;
    if (nv <= 8)
        launch<256, 8, 1>(a, st);
    else if (nv <= 16)
        launch<256, 16, 1>(a, st);
    else if (nv <= 32)
        launch<256, 32, 1>(a, st);
    else if (nv <= 64)
        launch<256, 64, 1>(a, st);
    else if (nv <= 256)
        launch<256, 256, 1>(a, st);
    else if (nv <= 512)
        launch<256, 256, 2>(a, st);
    else if (nv <= 1024)
        launch<256, 256, 4>(a, st);
    else if (nv <= 2048)
        launch<512, 512, 4>(a, st);
    else if (nv <= 4096)
        launch<1024, 1024, 4>(a, st);
    else
        launch<1024, 1024, 4, true>(a, st);
}

}  // namespace qmm
