// Product of two MXFP4 matrices (the format: mxfp4.hpp),
//     dst[j*ldd + i] = s[j] * sum_c W[i][c] X[j][c],
// on v_mfma_scale_f32_16x16x128_f8f6f4, which takes E2M1 codes and a scale per
// 32 of them from each side and sums in f32: the products are exact.
//
// Lanes.  Lane (c, i) = (lane / 16, lane % 16) holds one block of 32 codes (16
// bytes) of operand row i, any block, as long as both operands' lanes c hold the
// same one; and rows 4c .. 4c + 3 of output column i.
#include "mxfp4.hpp"

namespace qmm {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t ld8(rsrc_t r, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b8(r, off, 0, 0); }

// acc += A B^T for 16 rows of each side and four blocks; byte S of the scale words.
template <int S>
__device__ __forceinline__ f32x4 mx_mfma(u32x4 a, uint32_t sa, u32x4 b, uint32_t sb, f32x4 acc) {
    const i32x8 x = {(int)a.x, (int)a.y, (int)a.z, (int)a.w, 0, 0, 0, 0}, y = {(int)b.x, (int)b.y, (int)b.z, (int)b.w, 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, acc, 4, 4, S, (int)sa, S, (int)sb);
}
template <int S>
__device__ __forceinline__ void mx_steps(const u32x4* a, uint32_t sa, const u32x4* b, uint32_t sb, f32x4& acc) {
    acc = mx_mfma<0>(a[0], sa, b[0], sb, acc);
    if constexpr (S > 1) acc = mx_mfma<1>(a[1], sa, b[1], sb, acc);
    if constexpr (S > 2) acc = mx_mfma<2>(a[2], sa, b[2], sb, acc);
    if constexpr (S > 3) acc = mx_mfma<3>(a[3], sa, b[3], sb, acc);
}

// Rows [row0, row0 + 16*T) of a matrix of n rows: S blocks per lane and row.
template <int T, int S>
struct MxRows {
    rsrc_t codes, scales;
    uint32_t row_codes, row_scales;  // bytes between rows
    __device__ __forceinline__ MxRows(const uint8_t* q, const uint8_t* e, int64_t row0, int n, int blocks) {
        const int64_t left = n - row0, rows = left < 16 * T ? left : 16 * T;
        row_codes = 16u * (uint32_t)blocks;
        row_scales = (uint32_t)blocks;
        codes = make_rsrc(q + row0 * row_codes, (uint32_t)rows * row_codes);
        scales = make_rsrc(e + row0 * row_scales, (uint32_t)rows * row_scales);
    }
    // blocks [blk, blk + S) of row 16 t + i; none past the row's end (dead)
    __device__ __forceinline__ void load(u32x4 (&x)[T][S], uint32_t (&s)[T], int i, uint32_t blk, uint32_t dead) const {
#pragma unroll
        for (int t = 0; t < T; ++t) {
            const uint32_t row = 16u * (uint32_t)t + (uint32_t)i;
#pragma unroll
            for (int j = 0; j < S; ++j) x[t][j] = ld128(codes, (row * row_codes + 16u * (blk + (uint32_t)j)) | dead);
            const uint32_t at = (row * row_scales + blk) | dead;
            s[t] = S == 4 ? ld32(scales, at) : ld8(scales, at);
        }
    }
};

// A work group takes 16 RT weight rows and 16 NT tokens, its KW waves every
// KW-th group of 4 S blocks, straight from memory into operands.  S = 4: k a
// multiple of 128 (a lane's four scales are one aligned word).
template <int RT, int NT, int KW, int S>
__global__ __launch_bounds__(64 * KW) void gemm_mx_stream_kernel(const MxGemmArgs a) {
    __shared__ f32x4 red[KW][RT * NT][64];
    const int tid = threadIdx.x, lane = tid & 63, w = wave_id(), i = lane & 15, c = lane >> 4;
    const int64_t row0 = (int64_t)blockIdx.x * (16 * RT), tok0 = (int64_t)blockIdx.y * (16 * NT);
    const int blocks = a.k / 32;
    const MxRows<RT, S> wr(a.wq, a.we, row0, a.m, blocks);
    const MxRows<NT, S> xr(a.xq, a.xe, tok0, a.n, blocks);
    f32x4 acc[RT][NT] = {};
    for (int g = w; g * (4 * S) < blocks; g += KW) {
        const uint32_t blk = (uint32_t)(g * (4 * S) + c * S), dead = blk < (uint32_t)blocks ? 0u : OOB_OFF;
        u32x4 aw[RT][S], bx[NT][S];
        uint32_t sw[RT], sx[NT];
        wr.load(aw, sw, i, blk, dead);
        xr.load(bx, sx, i, blk, dead);
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int t = 0; t < NT; ++t) mx_steps<S>(aw[r], sw[r], bx[t], sx[t], acc[r][t]);
    }
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) red[w][r * NT + t][lane] = acc[r][t];
    __syncthreads();
    const bool wide = (a.m & 3) == 0 && (a.ldd & 3) == 0 && ((uintptr_t)a.dst & 15) == 0;
    for (int x = tid; x < RT * NT * 64; x += 64 * KW) {
        const int part = x >> 6, l = x & 63;
        f32x4 v = red[0][part][l];
#pragma unroll
        for (int z = 1; z < KW; ++z) v += red[z][part][l];
        const int64_t tok = tok0 + 16 * (part % NT) + (l & 15), row = row0 + 16 * (part / NT) + 4 * (l >> 4);
        if (tok >= a.n || row >= a.m) continue;
        if (a.s) v *= a.s[tok];
        float* d = a.dst + tok * a.ldd + row;
        if (wide) {
            *(f32x4*)d = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (row + r < a.m) d[r] = v[r];
        }
    }
}

template <int RT, int NT, int KW, int S>
void stream(const MxGemmArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.m + 16 * RT - 1) / (16 * RT)), (unsigned)((a.n + 16 * NT - 1) / (16 * NT)));
    gemm_mx_stream_kernel<RT, NT, KW, S><<<grid, 64 * KW, 0, st>>>(a);
}

}  // namespace

void launch_gemm_mxfp4(const MxGemmArgs& a, int num_cu, hipStream_t st) {
    if (a.k % 128 == 0)
        a.n <= 16 ? stream<1, 1, 8, 4>(a, st) : stream<2, 2, 4, 4>(a, st);
    else
        a.n <= 16 ? stream<1, 1, 8, 1>(a, st) : stream<2, 2, 4, 1>(a, st);
}

}  // namespace qmm
