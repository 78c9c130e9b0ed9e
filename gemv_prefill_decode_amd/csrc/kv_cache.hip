// The paged key-value cache's bookkeeping and its writer.
#include "common.hpp"
#include "kernels.hpp"

namespace qmm {

namespace {

// ------------------------------------------------------------------ page tables
// Per sequence i with c cached and n new tokens and pages of P tokens:
//     have = ceil(c / P), need = ceil((c + n) / P) - have,
//     first = sum of need over the sequences before it, table[have + r] = free[first + r];
// row R + r (R = sum of n before it): position c + r, slot = page of the position * P + its place.
// A few thousand integers: launch and memory latency bound it.  One kernel
// without communication between work groups: each scans all sequences in
// passes of THREADS (two sums), and writes its own range of rows and its
// stride of new table entries, which it finds in the pass by bisection.
// Measured: 64 sequences of one new token 3.7 us (1024 threads instead of 256:
// 6.1); 512 prompts with 88600 rows 7.0 us (4096 rows per work group instead of
// 1024: 10.4).
template <int THREADS, typename T>
__device__ __forceinline__ T block_inclusive(T v, T* waves, T* total) {
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
#pragma unroll
    for (int s = 1; s < 64; s <<= 1) {
        const T u = __shfl_up(v, s);
        if (lane >= s) v += u;
    }
    if (lane == 63) waves[w] = v;
    __syncthreads();
    T t = 0;
    for (int i = 0; i < THREADS / 64; ++i) {
        if (i < w) v += waves[i];
        t += waves[i];
    }
    *total = t;
    return v;
}

// First index whose inclusive sum exceeds x (sums do not decrease).
template <int THREADS, typename T>
__device__ __forceinline__ int bisect(const T* sums, T x) {
    int lo = 0, hi = THREADS - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (sums[mid] > x)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void paged_extend_kernel(const ExtendArgs a, int rows_per_group) {
    __shared__ int64_t row_end[THREADS], row_waves[THREADS / 64];
    __shared__ int need_end[THREADS], need_waves[THREADS / 64];
    __shared__ int cached[THREADS], fresh[THREADS];
    __shared__ bool taken[THREADS];
    const int tid = threadIdx.x;
    const int64_t lo = (int64_t)blockIdx.x * rows_per_group;
    const int64_t hi = lo + rows_per_group < a.n_rows ? lo + rows_per_group : a.n_rows;
    const int mask = (1 << a.page_log2) - 1;
    auto pages = [&](int64_t tokens) { return (int)((tokens + mask) >> a.page_log2); };
    int64_t rows_before = 0;
    int need_before = 0;
    for (int base = 0, pass = 0; base < a.batch; base += THREADS, ++pass) {
        const int b = base + tid;
        const int c = b < a.batch ? a.cached[b] : 0, n = b < a.batch ? a.fresh[b] : 0;
        bool ok = c >= 0 && n >= 0 && (int64_t)c + n <= a.capacity;
        const int need = ok ? pages((int64_t)c + n) - pages(c) : 0;
        int64_t rows_total;
        int need_total;
        const int64_t rows_incl = rows_before + block_inclusive<THREADS, int64_t>(n > 0 ? n : 0, row_waves, &rows_total);
        const int need_incl = need_before + block_inclusive<THREADS, int>(need, need_waves, &need_total);
        ok = ok && (need == 0 || need_incl <= a.n_free);
        row_end[tid] = rows_incl;
        need_end[tid] = need_incl;
        cached[tid] = c;
        fresh[tid] = n > 0 ? n : 0;
        taken[tid] = ok;
        if (b < a.batch && pass % gridDim.x == blockIdx.x) a.seq_lens[b] = ok ? c + n : c;
        __syncthreads();

        // new table entries
        for (int e = need_before + blockIdx.x * THREADS + tid; e < need_before + need_total && e < a.n_free;
             e += gridDim.x * THREADS) {
            const int s = bisect<THREADS>(need_end, e);
            const int begin = s ? need_end[s - 1] : need_before;
            if (taken[s]) a.table[(int64_t)(base + s) * a.table_stride + pages(cached[s]) + (e - begin)] = a.free_pages[e];
        }
        // this work group's rows that belong to the pass
        const int64_t r_lo = lo > rows_before ? lo : rows_before;
        const int64_t r_hi = hi < rows_before + rows_total ? hi : rows_before + rows_total;
        for (int64_t r = r_lo + tid; r < r_hi; r += THREADS) {
            const int s = bisect<THREADS>(row_end, r);
            const int pos = (int)(cached[s] + (r - (row_end[s] - fresh[s])));
            int slot = -1;
            if (taken[s]) {
                const int col = pos >> a.page_log2, have = pages(cached[s]);
                const int page = col < have ? a.table[(int64_t)(base + s) * a.table_stride + col]
                                            : a.free_pages[(s ? need_end[s - 1] : need_before) + col - have];
                const int64_t at = ((int64_t)page << a.page_log2) + (pos & mask);
                slot = page >= 0 && at <= INT32_MAX ? (int)at : -1;
            }
            a.slots[r] = slot;
            a.positions[r] = pos;
        }
        rows_before += rows_total;
        need_before += need_total;
        __syncthreads();
    }
    for (int64_t r = (lo > rows_before ? lo : rows_before) + tid; r < hi; r += THREADS) {
        a.slots[r] = -1;
        a.positions[r] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) *a.pages_used = need_before;
}

// ------------------------------------------------------------------ append
// One thread takes eight consecutive elements of a row (two 16-byte loads; a
// 16-byte store to a 16-bit cache).  Reads 4 bytes per element and writes 2
// (1): HBM bounds many tokens, launch latency few.  8-bit rows: the thread's
// row is shared by LANES consecutive lanes, a power of two, some idle where
// head_dim / 8 is none, which find the row's largest magnitude together.
// Measured: 8192 tokens of 8 heads of 128 from f32 to bf16, 100.7 MB, 18.6 us
// where the projection's output is still in the 256 MB cache (5.4 TB/s), 22 us
// from HBM (4.5; a copy reaches 4.7); 16 tokens 2.0 us.  Non-temporal loads
// gain 1 us of the 22 and lose 4 of the others: not used.
constexpr int APP_THREADS = 256;

template <int KIND, int NB>
__global__ __launch_bounds__(APP_THREADS) void kv_append_kernel(const AppendArgs a) {
    constexpr int VEC = 4 * NB;  // threads' shares of a row
    constexpr int LANES = KIND != KV_Q8 ? VEC : NB == 1 ? 4 : NB == 2 ? 8 : NB <= 4 ? 16 : 32;
    const bool second = blockIdx.y != 0;
    const float* src = second ? a.v : a.k;
    const int64_t src_stride = second ? a.v_stride : a.k_stride;
    const int64_t rows = a.n * a.n_kv;  // (token, head)
    constexpr int RPB = APP_THREADS / LANES;
    const int e = threadIdx.x % LANES;
    for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / LANES; row < rows; row += (int64_t)gridDim.x * RPB) {
        if (threadIdx.x >= RPB * LANES) return;
        const int64_t tok = rows <= UINT32_MAX ? (uint32_t)row / (uint32_t)a.n_kv : row / a.n_kv;
        const int head = (int)(row - tok * a.n_kv);
        const int slot = a.slots[tok];
        f32x4 lo = {0, 0, 0, 0}, hi = {0, 0, 0, 0};
        if (e < VEC) {  // whether or not the row goes anywhere: the loads do not wait for its slot
            const f32x4* p = (const f32x4*)(src + tok * src_stride + (int64_t)head * (32 * NB) + 8 * e);
            lo = p[0];
            hi = p[1];
        }
        const bool live = e < VEC && slot >= 0 && slot < a.n_slots;
        const int64_t page = slot >> a.page_log2, in_page = slot & ((1 << a.page_log2) - 1);
        const int64_t at = page * a.page_stride + head * a.head_stride + in_page * a.slot_stride + 8 * e;
        if constexpr (KIND == KV_Q8) {
            float top = 0.0f;
#pragma unroll
            for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(lo[j]), fabsf(hi[j])));
#pragma unroll
            for (int s = 1; s < LANES; s <<= 1) top = fmaxf(top, __shfl_xor(top, s));
            float d = top / 127.0f;
            if (d < 1.17549435e-38f) d = 0.0f;  // its inverse would overflow
            const float id = d != 0.0f ? 1.0f / d : 0.0f;
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[0] |= (uint32_t)(uint8_t)(int8_t)(int)roundf(lo[j] * id) << (8 * j);
                w[1] |= (uint32_t)(uint8_t)(int8_t)(int)roundf(hi[j] * id) << (8 * j);
            }
            if (live) {
                *(u32x2*)((int8_t*)(second ? a.vc : a.kc) + at) = u32x2{w[0], w[1]};
                if (e == 0)
                    (second ? a.vs : a.ks)[page * a.scale_page + head * a.scale_head + in_page * a.scale_slot] = d;
            }
        } else if (live) {
            u32x4 w;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = j < 2 ? lo[2 * j] : hi[2 * j - 4], v = j < 2 ? lo[2 * j + 1] : hi[2 * j - 3];
                if constexpr (KIND == KV_F16) {
                    w[j] = pack_f2h(u, v);
                } else {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    w[j] = __builtin_bit_cast(uint32_t, bf16x2{(__bf16)u, (__bf16)v});
                }
            }
            *(u32x4*)((uint16_t*)(second ? a.vc : a.kc) + at) = w;
        }
    }
}

template <int KIND, int NB>
void append(const AppendArgs& a, hipStream_t st) {
    constexpr int LANES = KIND != KV_Q8 ? 4 * NB : NB == 1 ? 4 : NB == 2 ? 8 : NB <= 4 ? 16 : 32;
    const int64_t rows = a.n * a.n_kv, rpb = APP_THREADS / LANES;
    int64_t blocks = (rows + rpb - 1) / rpb;
    if (blocks > 65536) blocks = 65536;
    kv_append_kernel<KIND, NB><<<dim3((unsigned)blocks, 2), APP_THREADS, 0, st>>>(a);
}

template <int KIND>
void append_kind(const AppendArgs& a, int head_dim, hipStream_t st) {
    switch (head_dim / 32) {
        case 1: append<KIND, 1>(a, st); break;
        case 2: append<KIND, 2>(a, st); break;
        case 3: append<KIND, 3>(a, st); break;
        case 4: append<KIND, 4>(a, st); break;
        case 5: append<KIND, 5>(a, st); break;
        case 6: append<KIND, 6>(a, st); break;
        case 7: append<KIND, 7>(a, st); break;
        case 8: append<KIND, 8>(a, st); break;
    }
}

}  // namespace

void launch_paged_extend(const ExtendArgs& a, hipStream_t st) {
    // a row per thread, in at most 512 work groups (each scans all sequences)
    const int threads = a.batch <= 256 ? 256 : 1024;
    int64_t rows = ((int64_t)a.n_rows + 511) / 512;
    if (rows < threads) rows = threads;
    int64_t groups = ((int64_t)a.n_rows + rows - 1) / rows;
    if (groups < 1) groups = 1;
    if (threads == 256)
        paged_extend_kernel<256><<<dim3((unsigned)groups), 256, 0, st>>>(a, (int)rows);
    else
        paged_extend_kernel<1024><<<dim3((unsigned)groups), 1024, 0, st>>>(a, (int)rows);
}

void launch_kv_append(const AppendArgs& a, int kind, int head_dim, hipStream_t st) {
    if (kind == KV_F16)
        append_kind<KV_F16>(a, head_dim, st);
    else if (kind == KV_BF16)
        append_kind<KV_BF16>(a, head_dim, st);
    else
        append_kind<KV_Q8>(a, head_dim, st);
}

}  // namespace qmm
