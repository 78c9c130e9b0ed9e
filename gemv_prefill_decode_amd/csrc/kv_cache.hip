// The paged key-value cache's bookkeeping and its writer.
#include "common.hpp"
#include "kernels.hpp"
#include "mxfp4.hpp"

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
// Measured: 64 sequences of one new token 2.9 us, 512 prompts with 88600 rows
// 3.9, 1024 prompts on pages of one token 5.2 (with 64-bit sums, LDS shuffles
// and a branching bisection 4.0, 7.0 and 13.0; a launch alone 1.6).
//
// Sums of rows saturate at 2^32 - 1, far behind any row that is written
// (saturating addition is associative, so the scan may take it in any order).
__device__ __forceinline__ uint32_t add_sat(uint32_t a, uint32_t b) { return __builtin_elementwise_add_sat(a, b); }

// Inclusive sums over the wave's lanes: row shifts within 16 lanes, then the
// rows' last lanes handed on.
template <bool SAT>
__device__ __forceinline__ uint32_t wave_inclusive(uint32_t v) {
    auto add = [](uint32_t a, uint32_t b) { return SAT ? add_sat(a, b) : a + b; };
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, true));   // row_shr:1
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, true));   // row_shr:2
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, true));   // row_shr:4
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, true));   // row_shr:8
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));  // row_bcast:15
    v = add(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));  // row_bcast:31
    return v;
}

// First index whose inclusive sum exceeds x (sums do not decrease).
template <int THREADS>
__device__ __forceinline__ int bisect(const uint32_t* sums, uint32_t x) {
    int lo = 0;
#pragma unroll
    for (int step = THREADS / 2; step > 0; step >>= 1)
        if (sums[lo + step - 1] <= x) lo += step;
    return lo;
}

template <int THREADS>
__global__ __launch_bounds__(THREADS) void paged_extend_kernel(const ExtendArgs a, int rows_per_group) {
    constexpr int WAVES = THREADS / 64;
    __shared__ uint32_t row_end[THREADS], need_end[THREADS];
    __shared__ uint32_t row_waves[WAVES], need_waves[WAVES];
    __shared__ int cached[THREADS];
    __shared__ bool taken[THREADS];
    const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t lo = blockIdx.x * (uint32_t)rows_per_group, n_rows = (uint32_t)a.n_rows;
    const uint32_t hi = lo + rows_per_group < n_rows ? lo + rows_per_group : n_rows;
    const int mask = (1 << a.page_log2) - 1;
    auto pages = [&](int64_t tokens) { return (int)((tokens + mask) >> a.page_log2); };
    uint32_t rows_before = 0, need_before = 0;
    for (int base = 0, pass = 0; base < a.batch; base += THREADS, ++pass) {
        const int b = base + tid;
        const int c = b < a.batch ? a.cached[b] : 0, n = b < a.batch ? a.fresh[b] : 0;
        bool ok = c >= 0 && n >= 0 && (int64_t)c + n <= a.capacity;
        const int need = ok ? pages((int64_t)c + n) - pages(c) : 0;
        uint32_t rows = wave_inclusive<true>(n > 0 ? (uint32_t)n : 0u), needs = wave_inclusive<false>((uint32_t)need);
        if (lane == 63) {
            row_waves[w] = rows;
            need_waves[w] = needs;
        }
        cached[tid] = c;
        __syncthreads();
        // the waves before this one, and the whole pass
        const uint32_t rw = wave_inclusive<true>(lane < WAVES ? row_waves[lane] : 0u);
        const uint32_t nw = wave_inclusive<false>(lane < WAVES ? need_waves[lane] : 0u);
        if (w > 0) {
            rows = add_sat(rows, __builtin_amdgcn_readlane(rw, w - 1));
            needs += __builtin_amdgcn_readlane(nw, w - 1);
        }
        rows = add_sat(rows, rows_before);
        needs += need_before;
        const uint32_t rows_after = add_sat(rows_before, __builtin_amdgcn_readlane(rw, 63));
        const uint32_t need_after = need_before + __builtin_amdgcn_readlane(nw, 63);
        ok = ok && (need == 0 || needs <= (uint32_t)a.n_free);
        row_end[tid] = rows;
        need_end[tid] = needs;
        taken[tid] = ok;
        if (b < a.batch && pass % gridDim.x == blockIdx.x) a.seq_lens[b] = ok ? c + n : c;
        __syncthreads();

        // new table entries
        for (uint32_t e = need_before + blockIdx.x * THREADS + tid; e < need_after && e < (uint32_t)a.n_free;
             e += gridDim.x * THREADS) {
            const int page = a.free_pages[e], s = bisect<THREADS>(need_end, e);
            const uint32_t begin = s ? need_end[s - 1] : need_before;
            if (taken[s]) a.table[(int64_t)(base + s) * a.table_stride + pages(cached[s]) + (e - begin)] = page;
        }
        // this work group's rows that belong to the pass
        const uint32_t r_lo = lo > rows_before ? lo : rows_before, r_hi = hi < rows_after ? hi : rows_after;
        for (uint32_t r = r_lo + tid; r < r_hi; r += THREADS) {
            const int s = bisect<THREADS>(row_end, r);
            const int pos = (int)((int64_t)cached[s] + (r - (s ? row_end[s - 1] : rows_before)));
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
        rows_before = rows_after;
        need_before = need_after;
        if (base + THREADS < a.batch) __syncthreads();
    }
    for (uint32_t r = (lo > rows_before ? lo : rows_before) + tid; r < hi; r += THREADS) {
        a.slots[r] = -1;
        a.positions[r] = -1;
    }
    if (blockIdx.x == 0 && tid == 0) *a.pages_used = (int)need_before;
}

// ------------------------------------------------------------------ append
// One thread takes eight consecutive elements of a row (two 16-byte loads; a
// 16-byte store to a 16-bit cache).  Reads 4 bytes per element and writes 2
// (1): HBM bounds many tokens, launch latency few.  8-bit rows: the thread's
// row is shared by LANES consecutive lanes, a power of two, some idle where
// head_dim / 8 is none, which find the row's largest magnitude together.
// Measured: 8192 tokens of 8 heads of 128 from f32 to bf16, 100.7 MB, 18.6 us
// where the projection's output is still in the 256 MB cache (5.4 TB/s), 22 us
// from HBM (4.5; a copy reaches 4.7); 16 tokens 2.8 us.  To 8 bits 17.6 us (84.4
// MB, 4.8 TB/s) and 3.2.  Non-temporal loads gain 1 us of the 22 and lose 4 of
// the others: not used.  MXFP4 (four lanes a block): 76 MB from HBM 20.5 us (3.7
// TB/s, nearly all of it reading) and 3.0.
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
            // The largest magnitude as bits: an infinity and then NaN are the largest of all, so
            // that a row with either gets it as its scale and stays visible.
            auto magnitude = [](float x) { return __builtin_bit_cast(uint32_t, x) & 0x7fffffffu; };
            auto larger = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
            uint32_t bits = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) bits = larger(bits, larger(magnitude(lo[j]), magnitude(hi[j])));
#pragma unroll
            for (int s = 1; s < LANES; s <<= 1) bits = larger(bits, (uint32_t)__shfl_xor((int)bits, s));
            float d = __builtin_bit_cast(float, bits) / 127.0f;
            if (d < 1.17549435e-38f) d = 0.0f;  // its inverse would overflow
            const bool finite = bits < 0x7f800000u;
            const float id = finite && d != 0.0f ? 1.0f / d : 0.0f;
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                w[0] |= (uint32_t)(uint8_t)(int8_t)(int)roundf(finite ? lo[j] * id : 0.0f) << (8 * j);
                w[1] |= (uint32_t)(uint8_t)(int8_t)(int)roundf(finite ? hi[j] * id : 0.0f) << (8 * j);
            }
            if (live) {
                *(u32x2*)((int8_t*)(second ? a.vc : a.kc) + at) = u32x2{w[0], w[1]};
                if (e == 0)
                    (second ? a.vs : a.ks)[page * a.scale_page + head * a.scale_head + in_page * a.scale_slot] = d;
            }
        } else if constexpr (KIND == KV_MX4) {
            const uint32_t byte = mx_scale_byte(mx_quad_max(mx_max8(lo, hi)));  // a quad of lanes holds a block
            const uint32_t codes = mx_codes8(lo, hi, byte);
            if (live) {
                *(uint32_t*)((uint8_t*)(second ? a.vc : a.kc) + at / 2) = codes;
                if ((e & 3) == 0)
                    ((uint8_t*)(second ? a.vs : a.ks))[page * a.scale_page + head * a.scale_head + in_page * a.scale_slot +
                                                       e / 4] = (uint8_t)byte;
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
    else if (kind == KV_MX4)
        append_kind<KV_MX4>(a, head_dim, st);
    else
        append_kind<KV_Q8>(a, head_dim, st);
}

}  // namespace qmm
