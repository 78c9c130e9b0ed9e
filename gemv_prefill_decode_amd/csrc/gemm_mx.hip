// Product of two MXFP4 matrices (the format: mxfp4.hpp),
//     dst[j*ldd + i] = s[j] * sum_c W[i][c] X[j][c],
// on v_mfma_scale_f32_16x16x128_f8f6f4, which takes E2M1 codes and a scale per
// 32 of them from each side and sums in f32: the products are exact.
//
// Lanes.  Lane (c, i) = (lane / 16, lane % 16) holds one block of 32 codes (16
// bytes) of operand row i, any block, as long as both operands' lanes c hold the
// same one; and rows 4c .. 4c + 3 of output column i.
//
// Bounds and measured times (MI355X).  Few tokens: the weights' bytes, 14336 x
// 4096 with 16 tokens (32 MB) 8.9 us from HBM, 3.6 TB/s, 7.6 where the 256 MB cache
// holds them; or latency, 4608 x 1024 with one 3.2 us, 1024 x 4608 with 512 6.8
// us.  In between, 4096 x 4096 with 512, 13.9: 128 tiles of 128 x 128 for 256 CUs, or
// 64 x 64 ones, which read twice the bytes.  Many, 14336 x 4096 with 2048: 76.0 us,
// 3.16 PFLOP/s, where the matrix instructions alone take 44 to 51 us (the clock falls
// with the data), the loads into LDS alone 54 us (L2 gives about 15 TB/s of whole
// lines) and the outputs, behind which no loads go on, 13 to 19 us; operands' reads
// from LDS and the loads' writes keep it as busy as the matrix cores are.
// In turn: operands straight from memory 656 us; 128 x 128 tiles through LDS 126;
// scales as 16 bytes a row 98; whole lines of outputs past the caches 90; lines of
// 128 bytes with operands read ahead 85; outputs through LDS and 256 x 256 tiles 79.5;
// the tokens' factors out of the stores' way 78.6; the tokens' loads ahead of the
// stage's end 76.0.  Rings of more and shorter stages
// (64 bytes a row) lost more on half lines than they hid; loads that warm L2 ahead
// gained nothing.
#include <type_traits>
#include <utility>

#include "mxfp4.hpp"

namespace qmm {

namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ uint32_t ld16(rsrc_t r, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0); }
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
            s[t] = S == 2 ? ld16(scales, at) : ld8(scales, at);
        }
    }
};

// Few rows and tokens, or a short k: a work group takes 16 RT weight rows and 16
// NT tokens, its KW waves every KW-th group of 4 S blocks, straight from memory
// into operands, and adds their sums in order.  S = 2: k a multiple of 64 (a
// lane's two scales are one aligned half word; with four blocks a lane, whose
// loads touch every line four times, 14336 x 4096 n = 16 takes 13.8 us for 12.6).
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

// ------------------------------------------------------------------ tiles
// s_waitcnt with vmcnt(VM) and lgkmcnt(0) (gfx9 encoding)
template <int VM>
__device__ __forceinline__ void wait_vm() {
    static_assert(VM >= 0 && VM < 64, "waitcnt range");
    __builtin_amdgcn_s_waitcnt((VM & 15) | ((VM >> 4) << 14) | (7 << 4));
}

typedef __attribute__((address_space(3))) void lds_void_t;

// A work group of WM x WN waves takes BM = 16 RI WM weight rows x BN = 16 NJ WN
// tokens.  Codes go in stages of 256 k, a 128-byte line of each row, from memory
// straight into NR stages of LDS; chunk p of row r holds chunk p ^ (r / 2 % 8), so
// that the 16 rows a wave reads at a time lie in different banks.  Scales, 16
// bytes a row for 512 k, go through registers, where they are turned so that a
// lane's four steps are the bytes of one word.
template <int RI, int NJ, int WM, int WN, int NR>
struct MxTile {
    static constexpr int WAVES = WM * WN, THREADS = 64 * WAVES, BM = 16 * RI * WM, BN = 16 * NJ * WN;
    static constexpr int LOADS = (BM + BN) / 8, D = (LOADS + WAVES - 1) / WAVES;  // 8 rows each: of a stage, of a wave
    static constexpr int B_THREAD = (BM + 63) / 64 * 64;                          // the thread that loads token 0's scales
    static constexpr int E = (B_THREAD + BN + THREADS - 1) / THREADS;             // rows of scales of a thread
    static constexpr int STAGE = (BM + BN) * 128, SCALES = (BM + BN) * 16;
    static constexpr int LDS = NR * STAGE + SCALES;
    static_assert(RI >= 2 && NJ <= 4 && LDS <= 160 * 1024, "tile");
};

template <typename F, int... Q>
__device__ __forceinline__ void for_each(F&& f, std::integer_sequence<int, Q...>) {
    (f(std::integral_constant<int, Q>{}), ...);
}

template <int RI, int NJ, int WM, int WN, int NR, int KG>
__global__ __launch_bounds__(64 * WM * WN * KG) void gemm_mx_tile_kernel(const MxGemmArgs a, int n_mb, int n_nb) {
    using T = MxTile<RI, NJ, WM, WN, NR>;
    constexpr int BM = T::BM, BN = T::BN;
    extern __shared__ __attribute__((aligned(1024))) uint8_t all_lds[];
    const int lane = threadIdx.x & 63, i = lane & 15, c = lane >> 4;
    const int kg = KG == 1 ? 0 : wave_id() / T::WAVES, w = KG == 1 ? wave_id() : wave_id() % T::WAVES, wm = w / WN, wn = w % WN;
    uint8_t *const lds = all_lds + kg * T::LDS, *const sc = lds + NR * T::STAGE;

    // Work groups are dealt round-robin to the 8 XCDs; each takes a contiguous
    // run of tiles, in bands of 8 weight tiles, so that those that run together on
    // an XCD share weight and token rows in its L2.
    const int total = n_mb * n_nb, L = blockIdx.x;
    const int xcd = L & 7, idx = L >> 3, per = total >> 3, rem = total & 7;
    const int item = xcd < rem ? xcd * (per + 1) + idx : rem * (per + 1) + (xcd - rem) * per + idx;
    const int band = item / (8 * n_nb), in_band = item - band * (8 * n_nb);
    const int height = n_mb - 8 * band < 8 ? n_mb - 8 * band : 8;
    const int nb = in_band / height, mb = 8 * band + in_band - nb * height;
    const int64_t m0 = (int64_t)mb * BM, n0 = (int64_t)nb * BN;

    // k group kg of KG takes every KG-th pair of stages: its stage s is stage_of(s) (past the end: zeros)
    const int blocks = a.k / 32, stages = KG == 1 ? (blocks + 7) / 8 : ((blocks + 15) / 16 + KG - 1) / KG * 2;
    auto stage_of = [&](int s) { return KG == 1 ? s : 2 * KG * (s / 2) + 2 * kg + (s & 1); };
    const uint32_t row_codes = 16u * (uint32_t)blocks;
    const uint32_t m_left = (uint32_t)imin64(a.m - m0, BM), n_left = (uint32_t)imin64(a.n - n0, BN);
    const rsrc_t wr = make_rsrc(a.wq + m0 * row_codes, m_left * row_codes);
    const rsrc_t xr = make_rsrc(a.xq + n0 * row_codes, n_left * row_codes);

    // A load takes 8 rows of eight chunks.  (Where the loads do not divide, the last waves
    // load the last rows once more.)
    auto issue = [&](int s, int slot, auto first, auto last) {
        uint8_t* st = lds + slot * T::STAGE;
#pragma unroll
        for (int u = first; u < last; ++u) {
            const int l = T::D * T::WAVES == T::LOADS || u * T::WAVES + w < T::LOADS ? u * T::WAVES + w : T::LOADS - 1;
            const bool of_w = l < BM / 8;
            const int blk = 8 * stage_of(s) + ((lane & 7) ^ (4 * (l & 1) + (lane >> 4)));
            const uint32_t at = (uint32_t)(of_w ? 8 * l : 8 * l - BM) * row_codes + (uint32_t)(lane >> 3) * row_codes + 16u * (uint32_t)blk;
            const uint32_t dead = blk < blocks ? 0u : OOB_OFF;
            if (of_w)
                __builtin_amdgcn_raw_ptr_buffer_load_lds(wr, (lds_void_t*)(st + l * 1024), 16, at | dead, 0, 0, 0);
            else
                __builtin_amdgcn_raw_ptr_buffer_load_lds(xr, (lds_void_t*)(st + l * 1024), 16, at | dead, 0, 0, 0);
        }
    };

    // Scales: a thread loads those of E rows.  (m0 and n0 are multiples of 16 rows, so the first
    // row's lie at a multiple of 16 bytes; the last word may be read to its end.)
    const bool odd = (blocks & 3) != 0;  // rows of scales that are not whole words
    struct Row {
        rsrc_t r;
        uint32_t at, dead;
        int place;  // in LDS
    };
    auto row_of = [&](int j) {
        const int r0 = T::THREADS * j + 64 * w;  // of the wave's first thread
        const bool of_w = r0 < T::B_THREAD;
        const int row = r0 + lane - (of_w ? 0 : T::B_THREAD);
        const rsrc_t r = make_rsrc(of_w ? a.we + m0 * blocks : a.xe + n0 * blocks,
                                   ((of_w ? m_left : n_left) * (uint32_t)blocks + 3u) & ~3u);
        const bool in = row < (of_w ? BM : BN);
        return Row{r, (uint32_t)row * (uint32_t)blocks, in ? 0u : OOB_OFF, in ? of_w ? row : BM + row : -1};
    };
    u32x4 e4[T::E];
    uint32_t e1[T::E] = {};
    auto load_scales = [&](int g) {
#pragma unroll
        for (int j = 0; j < T::E; ++j) {
            const Row r = row_of(j);
            const uint32_t at = ((r.at + 16u * (uint32_t)(KG * g + kg)) & ~3u) | r.dead;
            e4[j] = ld128(r.r, at);
            if (odd) e1[j] = ld32(r.r, at + 16u);
        }
    };
    auto store_scales = [&](int g) {
        const int valid = blocks - 16 * (KG * g + kg);  // scales of a row from here on
#pragma unroll
        for (int z = 0; z < T::E; ++z) {
            const Row r = row_of(z);
            const uint32_t sh = r.at & 3u;
            const uint32_t d[5] = {e4[z].x, e4[z].y, e4[z].z, e4[z].w, e1[z]};
            uint32_t x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int n = valid - 4 * j;
                x[j] = __builtin_amdgcn_alignbyte(d[j + 1], d[j], sh);
                x[j] = n >= 4 ? x[j] : n <= 0 ? 0u : x[j] & ((1u << (8 * n)) - 1u);
            }
            // byte c of words 0..3 (blocks 4 t + c) to bytes 0..3 of word c
            const uint32_t p01 = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u), q01 = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);
            const uint32_t p23 = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u), q23 = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
            const u32x4 out = {__builtin_amdgcn_perm(p23, p01, 0x05040100u), __builtin_amdgcn_perm(p23, p01, 0x07060302u),
                               __builtin_amdgcn_perm(q23, q01, 0x05040100u), __builtin_amdgcn_perm(q23, q01, 0x07060302u)};
            if (r.place >= 0) *(u32x4*)(sc + r.place * 16) = out;
        }
    };

    f32x4 acc[RI][NJ] = {};
    // operands of a stage's half h: chunk 4 h + c of the wave's rows
    const int arow = wm * (16 * RI) + i, brow = BM + wn * (16 * NJ) + i, p0 = 16 * (c ^ ((i >> 1) & 7));
    auto operand = [&](const uint8_t* st, int row, int h) { return *(const u32x4*)(st + row * 128 + (p0 ^ (64 * h))); };
    constexpr int PF = 3;  // row tiles whose operands are read ahead
    u32x4 fa[PF], fb[NJ];
    uint32_t sa[RI], sb[NJ];
    auto row_scales = [&](int row) { return *(const uint32_t*)(sc + row * 16 + 4 * c); };
    auto wait_lds = [&]() {
        __builtin_amdgcn_s_waitcnt(15 | (3 << 14) | (7 << 4));  // lgkmcnt(0)
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    // this wave's loads have landed and its LDS reads and writes are done; then every wave's
    auto wait = [&](auto n) {
        wait_vm<n>();
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };

    // Large tiles: the tokens' share of a stage is in registers long before the weights', and its place
    // takes loads then: there are some on their way all the time, not only after the stage's end.
    constexpr int MID = 6, LAST = 2 * RI - PF;
    constexpr bool SPLIT = MID + 2 < LAST;
    constexpr int OF_W = SPLIT ? BM / 8 / T::WAVES : T::D;  // a wave's loads of weights
    static_assert(!SPLIT || (BM / 8 % T::WAVES == 0 && BN / 8 % T::WAVES == 0 && MID < RI && NJ <= 4), "loads");
    const std::integral_constant<int, 0> none{};
    const std::integral_constant<int, OF_W> of_w{};
    const std::integral_constant<int, T::D> all{};
    load_scales(0);
#pragma unroll
    for (int p = 0; p < NR - 1; ++p) issue(p, p, none, all);
    store_scales(0);
    wait(std::integral_constant<int, (NR - 2) * T::D>{});
    if constexpr (RI <= 4) load_scales(1);
    issue(NR - 1, NR - 1, none, all);
#pragma unroll
    for (int q = 0; q < PF; ++q) fa[q] = operand(lds, arow + 16 * (q % RI), q / RI);
#pragma unroll
    for (int y = 0; y < NJ; ++y) fb[y] = operand(lds, brow + 16 * y, 0);
#pragma unroll
    for (int x = 0; x < RI; ++x) sa[x] = row_scales(arow + 16 * x);
#pragma unroll
    for (int y = 0; y < NJ; ++y) sb[y] = row_scales(brow + 16 * y);
    // Stage s: 2 RI row tiles q (half, tile), each NJ matrix instructions, with the operands of
    // tile q + PF read behind them.  Before tile LAST, where the stage's last operands are in
    // registers, one barrier: the next stage is whole, and this one's place takes the loads of the
    // one after.
    int place = 0;
    auto stage = [&](int s, auto odd_stage) {
        constexpr int O = odd_stage;
        const int here = place;
        place = here == NR - 1 ? 0 : here + 1;
        const uint8_t *st = lds + here * T::STAGE, *next = lds + place * T::STAGE;
        u32x4 fa_stage[PF], fb_half[NJ], fb_stage[NJ];  // of the next stage, of the second half
        if constexpr (O == 0 && RI > 4)
            load_scales(s / 2 + 1);
        if constexpr (O == 1)
            store_scales(s / 2 + 1);  // every wave has read this group's: before the last barrier
        auto tile = [&](auto at) {
            constexpr int q = at, h = q / RI, x = q % RI;
            const u32x4 f = fa[q % PF];
            if constexpr (q < LAST) fa[q % PF] = operand(st, arow + 16 * ((q + PF) % RI), (q + PF) / RI);
            if constexpr (!SPLIT && h == 0 && x < NJ) fb_half[x] = operand(st, brow + 16 * x, 1);
            if constexpr (SPLIT && q < (NJ + 1) / 2) {
                fb_half[2 * q] = operand(st, brow + 32 * q, 1);
                if constexpr (2 * q + 1 < NJ) fb_half[2 * q + 1] = operand(st, brow + 32 * q + 16, 1);
            }
            if constexpr (SPLIT && q == MID) {
                // LDS answers in order: tile MID - 1 had its operands, read in tile MID - 1 - PF, behind
                // the tokens' in tiles 0 and 1
                static_assert(MID - 1 - PF >= (NJ + 1) / 2, "tokens read");
                asm volatile("" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                issue(s + NR, here, of_w, all);
            }
            if constexpr (q == LAST) {
                wait(std::integral_constant<int, (NR - 2) * T::D + T::D - OF_W>{});
                if constexpr (O == 1 && RI <= 4) load_scales(s / 2 + 2);
                issue(s + NR, here, none, of_w);
            }
            if constexpr (q >= LAST) {
                constexpr int z = q - LAST;
                fa_stage[z] = operand(next, arow + 16 * (z % RI), z / RI);
                if constexpr (2 * z < NJ) fb_stage[2 * z] = operand(next, brow + 16 * (2 * z), 0);
                if constexpr (2 * z + 1 < NJ) fb_stage[2 * z + 1] = operand(next, brow + 16 * (2 * z + 1), 0);
                if constexpr (O == 1) {
                    // the next group's scales, each behind the last use of this one's
#pragma unroll
                    for (int r = 0; r < RI; ++r)
                        if (q == (LAST > RI + r + 1 ? LAST : RI + r + 1)) sa[r] = row_scales(arow + 16 * r);
                }
            }
#pragma unroll
            for (int y = 0; y < NJ; ++y) acc[x][y] = mx_mfma<2 * O + h>(f, sa[x], fb[y], sb[y], acc[x][y]);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (q == RI - 1) {
#pragma unroll
                for (int y = 0; y < NJ; ++y) fb[y] = fb_half[y];
            }
        };
        for_each(tile, std::make_integer_sequence<int, 2 * RI>{});
#pragma unroll
        for (int z = 0; z < PF; ++z) fa[z] = fa_stage[z];
#pragma unroll
        for (int y = 0; y < NJ; ++y) fb[y] = fb_stage[y];
        if constexpr (O == 1) {
            sa[RI - 1] = row_scales(arow + 16 * (RI - 1));
#pragma unroll
            for (int y = 0; y < NJ; ++y) sb[y] = row_scales(brow + 16 * y);
        }
    };
    for (int s = 0; s < stages; s += 2) {
        stage(s, std::integral_constant<int, 0>{});
        if (s + 1 < stages) stage(s + 1, std::integral_constant<int, 1>{});
    }
    // Outputs through LDS, 16 WN tokens at a time in two places, so that a store writes whole lines of
    // a token; the k groups' sums are added in order.
    wait(std::integral_constant<int, 0>{});
    constexpr int ROW = 4 * BM + 16, PLACE = 16 * WN * ROW;  // 16 bytes apart: the tokens of a wave's write in different banks
    static_assert(2 * PLACE + 4 * BN <= T::LDS, "outputs");
    // the tokens' scales too: a load of one would wait for the stores before it
    float* const tok_scale = (float*)(all_lds + 2 * PLACE);
    for (int t = threadIdx.x; t < BN; t += T::THREADS * KG) tok_scale[t] = a.s && n0 + t < a.n ? a.s[n0 + t] : 1.0f;
    const bool wide = (a.m & 3) == 0 && (a.ldd & 3) == 0 && ((uintptr_t)a.dst & 15) == 0;
    auto write = [&](auto at) {
        constexpr int y = at;
        uint8_t* place = lds + (y & 1) * PLACE;
#pragma unroll
        for (int x = 0; x < RI; ++x) *(f32x4*)(place + (16 * wn + i) * ROW + 4 * (wm * (16 * RI) + 16 * x + 4 * c)) = acc[x][y];
        wait_lds();
#pragma unroll 1
        for (int e = threadIdx.x; e < 16 * WN * (BM / 4); e += T::THREADS * KG) {
            const int t = e / (BM / 4), r = 4 * (e % (BM / 4));
            const int of_tile = (t / 16) * (16 * NJ) + 16 * y + t % 16;
            const int64_t tok = n0 + of_tile, row = m0 + r;
            if (tok >= a.n || row >= a.m) continue;
            const uint8_t* sum = all_lds + (y & 1) * PLACE + t * ROW + 4 * r;
            f32x4 v = *(const f32x4*)sum;
#pragma unroll
            for (int z = 1; z < KG; ++z) v += *(const f32x4*)(sum + z * T::LDS);
            v *= tok_scale[of_tile];
            float* d = a.dst + tok * a.ldd + row;
            if (wide) {
                __builtin_nontemporal_store(v, (f32x4*)d);
            } else {
#pragma unroll
                for (int z = 0; z < 4; ++z)
                    if (row + z < a.m) d[z] = v[z];
            }
        }
    };
    for_each(write, std::make_integer_sequence<int, NJ>{});
}

template <int RI, int NJ, int WM, int WN, int NR, int KG>
void tiles(const MxGemmArgs& a, hipStream_t st) {
    using T = MxTile<RI, NJ, WM, WN, NR>;
    const int n_mb = (a.m + T::BM - 1) / T::BM, n_nb = (a.n + T::BN - 1) / T::BN;
    if (T::LDS * KG > 64 * 1024)
        (void)hipFuncSetAttribute((const void*)gemm_mx_tile_kernel<RI, NJ, WM, WN, NR, KG>,
                                  hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS * KG);
    gemm_mx_tile_kernel<RI, NJ, WM, WN, NR, KG><<<(unsigned)((int64_t)n_mb * n_nb), T::THREADS * KG, T::LDS * KG, st>>>(a, n_mb, n_nb);
}

template <int RT, int NT, int KW, int S>
void stream(const MxGemmArgs& a, hipStream_t st) {
    const dim3 grid((unsigned)((a.m + 16 * RT - 1) / (16 * RT)), (unsigned)((a.n + 16 * NT - 1) / (16 * NT)));
    gemm_mx_stream_kernel<RT, NT, KW, S><<<grid, 64 * KW, 0, st>>>(a);
}

// The kernels a product may take, and what each takes in microseconds:
//     start + groups * (step * rounds + step_per * load) + end_per * load
// for `groups` passes of its k loop (of one k group's `pass` k each), `rounds` of
// work groups one after another on a CU that holds `per_cu` at a time, and a
// load of work groups per CU (at least 1; whole where one fits a CU).  The four
// are fitted to the times of 522 products, m 16 .. 14336, k 64 .. 14336, n 1 ..
// 4096, in graphs with the operands in HBM.  On 520 products timed since, most of
// them in the 256 MB cache, they are 11 to 26% off (rms; the last three, from
// memory, up to 37%) where a kernel is within 1.7 of the fastest; the kernel with
// the least takes 0.7% longer than the fastest of all on 90 projections, 22% at
// worst, and 2.4% on 430 sizes spread over their logarithms, 51% at worst.
struct Kernel {
    void (*launch)(const MxGemmArgs&, hipStream_t);
    int rows, tokens, k_groups, per_cu, pass;
    bool even;  // k a multiple of 64 only
    float start, step, step_per, end_per;
};
constexpr Kernel KERNELS[] = {
    {tiles<8, 4, 2, 4, 2, 1>, 256, 256, 1, 1, 512, false, 0.0f, 1.611f, 1.611f, 11.247f},
    {tiles<4, 4, 2, 2, 2, 1>, 128, 128, 1, 2, 512, false, 1.964f, 1.312f, 0.467f, 3.382f},
    {tiles<2, 2, 2, 2, 3, 1>, 64, 64, 1, 3, 512, false, 2.674f, 0.337f, 0.395f, 0.802f},
    {tiles<2, 2, 2, 2, 3, 2>, 64, 64, 2, 1, 512, false, 1.114f, 0.960f, 0.157f, 2.586f},
    {tiles<2, 2, 2, 1, 3, 2>, 64, 32, 2, 2, 512, false, 2.435f, 0.0f, 0.766f, 1.118f},
    {tiles<2, 1, 2, 1, 3, 2>, 64, 16, 2, 2, 512, false, 2.828f, 0.0f, 0.706f, 0.442f},
    {tiles<2, 2, 1, 1, 3, 4>, 32, 32, 4, 1, 512, false, 0.866f, 0.925f, 0.163f, 2.735f},
    {tiles<2, 1, 1, 1, 3, 4>, 32, 16, 4, 2, 512, false, 2.602f, 0.0f, 0.996f, 0.689f},
    {stream<1, 1, 4, 2>, 16, 16, 4, 8, 256, true, 2.290f, 0.031f, 0.562f, 0.0f},
    {stream<2, 2, 4, 2>, 32, 32, 4, 8, 256, true, 2.421f, 0.049f, 1.108f, 0.0f},
    {stream<1, 1, 8, 1>, 16, 16, 8, 4, 128, false, 2.781f, 0.315f, 0.314f, 0.0f},
};

}  // namespace

int gemm_mxfp4_kernels() { return (int)(sizeof(KERNELS) / sizeof(KERNELS[0])); }

void launch_gemm_mxfp4(const MxGemmArgs& a, int forced, int num_cu, hipStream_t st) {
    auto work_groups_of = [&](const Kernel& x) {
        return (int64_t)((a.m + x.rows - 1) / x.rows) * ((a.n + x.tokens - 1) / x.tokens);
    };
    // a launch has fewer than 2^32 threads, a grid's second axis fewer than 2^16 work groups
    // (2^37 outputs, the most there are, are 2^21 tiles of 256 x 256, and 2^13 more at the ends)
    auto runs = [&](const Kernel& x) {
        return !(x.even && a.k % 64 != 0) && work_groups_of(x) <= 1 << 22 && (a.n + x.tokens - 1) / x.tokens < 1 << 16;
    };
    if (forced >= 0 && runs(KERNELS[forced])) return KERNELS[forced].launch(a, st);
    const Kernel* best = nullptr;
    double least = 0;
    for (const Kernel& x : KERNELS) {
        if (!runs(x)) continue;
        const int64_t work_groups = work_groups_of(x);
        const int64_t rounds = (work_groups + (int64_t)num_cu * x.per_cu - 1) / ((int64_t)num_cu * x.per_cu);
        const int groups = ((a.k + x.pass - 1) / x.pass + x.k_groups - 1) / x.k_groups;
        const double each = (double)work_groups / num_cu;
        const double load = x.per_cu == 1 ? (double)((work_groups + num_cu - 1) / num_cu) : each > 1 ? each : 1;
        const double t = x.start + groups * (x.step * (double)rounds + x.step_per * load) + x.end_per * load;
        if (!best || t < least) {
            best = &x;
            least = t;
        }
    }
    best->launch(a, st);
}

}  // namespace qmm
