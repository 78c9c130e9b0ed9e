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

__device__ __forceinline__ uint32_t code(float z, float id) { return (uint32_t)(uint8_t)(int8_t)(int)roundf(z * id); }

// The Q8_1 codes of a block held by eight consecutive lanes, four values each.
// The largest magnitude is taken as bits: an infinity and then NaN are the
// largest of all, so that a block with either has it as its scale and codes 0.
__device__ __forceinline__ uint32_t codes4(f32x4 z, float* d0) {
    auto magnitude = [](float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; };
    auto larger = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
    uint32_t bits = larger(larger(magnitude(z.x), magnitude(z.y)), larger(magnitude(z.z), magnitude(z.w)));
#pragma unroll
    for (int s = 1; s < 8; s <<= 1) bits = larger(bits, (uint32_t)__shfl_xor((int)bits, s));
    float dd = __builtin_bit_cast(float, bits) / 127.0f;
    if (dd < 1.17549435e-38f) dd = 0.0f;  // its inverse would overflow
    *d0 = dd;
    const float id = dd != 0.0f ? 1.0f / dd : 0.0f;
    const uint32_t codes = code(z.x, id) | code(z.y, id) << 8 | code(z.z, id) << 16 | code(z.w, id) << 24;
    return bits < 0x7f800000u ? codes : 0;
}

template <bool NT>
__device__ __forceinline__ f32x4 ld(const f32x4* p) {
    return NT ? __builtin_nontemporal_load(p) : *p;
}

// THREADS threads per work group, T of them per row, V float4 per thread: a
// row of up to 4*T*V elements.  NT: rows read past the caches.  LOOP: longer
// rows, read a second time.
template <int THREADS, int T, int V, bool Q8, bool NT, bool LOOP>
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
            h[i] = live && e < nv ? ld<NT>(x + e) : zero;
            if (r) h[i] += live && e < nv ? ld<NT>(r + e) : zero;
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
void launch(const NormArgs& all, hipStream_t st) {
    constexpr int ROWS = THREADS / T;
    // Large inputs are read past the caches.  Kernel times so (and through them)
    // with x and the residual just written, with x just written, and with neither,
    // behind 640 MB of other writes: 2048 x 4096 19.0 us (19.2), 20.3 (24.8), 23.0
    // (35.0); 512 x 14336 16.8 (17.2), 18.1 (23.0), 20.0 (31.5); 8192 x 4096 83.9
    // (101.7), 81.9 (99.4), 101.4 (123.9); Q8_1 the same within 10%.  Below 48 MB
    // it gains from HBM and loses a little where the 256 MB cache behind the L2s
    // holds all: 1000 x 4608 13.6 (13.0), 12.4 (14.9), 13.4 (20.3).
    const bool nt = !LOOP && all.n * all.k * (all.r ? 8 : 4) > ((int64_t)48 << 20);
    // a launch has fewer than 2^32 threads
    constexpr int64_t MOST = ((int64_t)1 << 31) / THREADS * ROWS;
    for (int64_t first = 0; first < all.n; first += MOST) {
        NormArgs a = all;
        a.n = all.n - first < MOST ? all.n - first : MOST;
        a.x += first * a.x_stride;
        if (a.r) a.r += first * a.r_stride;
        if (a.h) a.h += first * a.h_stride;
        if (a.y) a.y += first * a.y_stride;
        if (a.q) {
            a.q += first * a.k;
            a.d += first * (a.k / 32);
        }
        const dim3 grid((unsigned)((a.n + ROWS - 1) / ROWS));
        if (a.q && nt)
            add_rmsnorm_kernel<THREADS, T, V, true, !LOOP, LOOP><<<grid, THREADS, 0, st>>>(a);
        else if (a.q)
            add_rmsnorm_kernel<THREADS, T, V, true, false, LOOP><<<grid, THREADS, 0, st>>>(a);
        else if (nt)
            add_rmsnorm_kernel<THREADS, T, V, false, !LOOP, LOOP><<<grid, THREADS, 0, st>>>(a);
        else
            add_rmsnorm_kernel<THREADS, T, V, false, false, LOOP><<<grid, THREADS, 0, st>>>(a);
    }
}

}  // namespace

void launch_add_rmsnorm(const NormArgs& a, int num_cu, hipStream_t st) {
    const int nv = a.k / 4;
    if (nv <= 8) return launch<256, 8, 1>(a, st);
    if (nv <= 16) return launch<256, 16, 1>(a, st);
    if (nv <= 32) return launch<256, 32, 1>(a, st);
    if (nv <= 64) return launch<256, 64, 1>(a, st);
    if (nv <= 256) return launch<256, 256, 1>(a, st);
    // few rows: as many threads as a row has work for (16 x 4096 4.1 -> 3.3 us)
    if (a.n <= num_cu && nv <= 1024) return launch<1024, 1024, 1>(a, st);
    if (a.n <= num_cu && nv <= 2048) return launch<1024, 1024, 2>(a, st);
    switch ((nv + 255) / 256) {
        case 2: return launch<256, 256, 2>(a, st);
        case 3: return launch<256, 256, 3>(a, st);
        case 4: return launch<256, 256, 4>(a, st);
        case 5: return launch<256, 256, 5>(a, st);
        case 6: return launch<256, 256, 6>(a, st);
        case 7: return launch<256, 256, 7>(a, st);
        case 8: return launch<256, 256, 8>(a, st);
    }
    if (nv <= 4096) return launch<1024, 1024, 4>(a, st);
    launch<1024, 1024, 4, true>(a, st);
}

}  // namespace qmm
