// Attention of one new token per sequence over a paged key-value cache.
//
// For query head h of sequence b, over the sequence's cached tokens t:
//     s_t = scale * q . k_t,  M = max s_t,  p_t = exp(s_t - M),
//     out = sum p_t v_t / sum p_t,  lse = M + log(sum p_t)
// in one pass over the cache with a running maximum (all exponentials are
// powers of two: scale * log2(e) is folded into the scores).
//
// Bound.  Each cached row is read once for the whole group of query heads
// that share it: 4 flops per element and query head on 2 (or 1) bytes, so
// HBM bounds every group size the matrix cores keep up with.
//
// Precision.  q and out are f32, and the arithmetic is f32's: an f32 operand
// (q, p) is split into f16 parts (high and low, 22 bits; for a bf16 cache into
// three bf16 parts, 24 bits), each multiplied with the cache's own 16-bit
// values on v_mfma_f32_16x16x32 into the same f32 sum.  f16 parts keep their
// bits because q is scaled to [2^13, 2^14) per head and p to (0, 2^14], powers
// of two that cancel at the end; bf16 parts have f32's exponents and only stay
// clear of its ends, keys and values reaching as far as f32's.  8-bit rows are
// exact as f16 codes; a key's scale multiplies its score, a value's scale its
// probability.
//
// Tiles.  A wave takes 32 tokens at a time: scores as K q^T (two 16-token
// tiles: lane (c, i) = (lane / 16, lane % 16) gets head i's scores of tokens
// 4c..4c+3 and 16+4c..16+4c+3), then out^T += V^T p^T with exactly those eight
// tokens as lane (c, i)'s k index, so neither p nor its running maximum ever
// changes lanes.  K and V rows go from memory straight into registers, K in
// operand layout; V's 16-bit transpose is one byte permute per operand dword.
// Loads of the next tile are issued as soon as the present one's registers
// are read, page ids one tile further ahead.
//
// Split.  A head space's units' tiles, and what a unit costs beside them, form
// one axis that is cut into equal chunks, one per work group and a quarter of
// it per wave, whatever the lengths are: every wave scans the lengths by
// itself, so no host plan or length is needed.  All head spaces are cut alike,
// so that heads whose rows lie side by side are read at the same time (8-bit
// heads of 96, tokens outermost, which share lines: 62 us, 79 where the cuts
// drift).  A unit inside one wave is finished there; parts of a unit are joined
// in LDS, or, where it spans work groups, by a second kernel from the
// workspace, always in the same order, so results do not vary between calls.
// (Joining in the first kernel by the last of a unit's work groups was no
// faster: release fences write back whole L2s, 171 us for 96; device-scope
// stores and a counter took the 9 us that the second kernel had taken.)
//
// Measured (MI355X, 8 kv heads of 128; both kernels): 131071 tokens of f16, 537
// MB, 89 us (6.0 TB/s; a kernel that only reads reaches 7.0); 51 sequences of up
// to 16384 tokens of bf16, tokens outermost, 1109 MB, 188 us (5.9 TB/s); 64
// sequences of up to 8192 8-bit tokens, 382 MB, 72 us (5.3 TB/s; vector ALUs
// about half busy, most of it the codes' conversion); one sequence of 97 tokens,
// heads of 64, 5.1 us (launch and four dependent loads).
#include "common.hpp"
#include "kernels.hpp"

namespace qmm {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr int TILE = 32;      // tokens per wave step
constexpr int HEADS = 16;     // query heads per pass over a unit's rows
// Work groups per CU that the registers are shared between.  Two hold 128 KB
// (8-bit: 64 KB) of loads in flight on a CU, and more read no faster: with
// three or four, where the registers allow it, 8-bit heads of 128 went from
// 103 to 121 us and f16 heads of 64 from 92 to 97 us (64 sequences of 4096).
constexpr int occupancy(int kind, int nb) { return nb <= (kind == KV_Q8 ? 6 : 5) ? 2 : 1; }
// What a unit's start and end cost its wave, in tiles: its loads are not ahead
// of it, and its sums are written.  Counted where a wave has at least
// START_MIN tiles, so that the waves with many short units are not the last
// (64 sequences of up to 8192 8-bit tokens, sorted: 87.7 -> 72.1 us; of 0, 1,
// 2 and 3 the second was 74.0, the last 72.7).  With few tiles the cuts would
// only move off the units' ends.
constexpr int UNIT_START = 2, START_MIN = 6;
constexpr float PBITS = 14.0f;
constexpr float P_UNIT = 6.103515625e-05f;  // 2^-14
constexpr float LN2 = 0.6931471805599453f, LOG2E = 1.4426950408889634f;

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ float fbits(uint32_t u) { return __builtin_bit_cast(float, u); }
__device__ __forceinline__ uint32_t ubits(float f) { return __builtin_bit_cast(uint32_t, f); }
__device__ __forceinline__ float from_lane(float v, int lane) {
    return fbits(__builtin_amdgcn_ds_bpermute(4 * lane, (int)ubits(v)));
}

// The maximum (sum) over the four lanes that differ in lane / 16, in each of
// them: row exchanges (v_permlane16_swap, v_permlane32_swap), no LDS.
__device__ __forceinline__ void swap16(float v, float* x, float* y) {
    const auto r = __builtin_amdgcn_permlane16_swap(ubits(v), ubits(v), false, false);
    *x = fbits(r[0]);
    *y = fbits(r[1]);
}
__device__ __forceinline__ void swap32(float v, float* x, float* y) {
    const auto r = __builtin_amdgcn_permlane32_swap(ubits(v), ubits(v), false, false);
    *x = fbits(r[0]);
    *y = fbits(r[1]);
}
__device__ __forceinline__ float max_c(float v) {
    float x, y;
    swap16(v, &x, &y);
    swap32(fmaxf(x, y), &x, &y);
    return fmaxf(x, y);
}
__device__ __forceinline__ float sum_c(float v) {
    float x, y;
    swap16(v, &x, &y);
    swap32(x + y, &x, &y);
    return x + y;
}

// Tokens of a sequence: -1 for a length the table cannot hold (its outputs
// become NaN, nothing is read).
__device__ __forceinline__ int seq_len(const AttnArgs& a, int b) {
    const int n = a.lens[b];
    return (n < 0 || n > a.capacity) ? -1 : n;
}
// One over what the weight of a head's largest score counts in its sums (m, l
// and acc, in registers and in parts).  f16: 2^14, sums of values of at most
// 65504 stay far inside f32.  bf16 and 8-bit elements reach as far as f32: 2^-b
// for up to 2^b tokens, so that a sum of weights times values is no larger than
// the largest value.
__device__ __forceinline__ int log2_up(int len) { return len > 1 ? 32 - __builtin_clz(len - 1) : 0; }
__device__ __forceinline__ float one_weight(int kind, int len) {
    return kind == KV_F16 ? P_UNIT : fbits((uint32_t)(127 + log2_up(len)) << 23);
}
// A unit without tokens still takes one tile, whose wave writes its outputs.
__device__ __forceinline__ int seq_tiles(int len) { return len <= TILE ? 1 : (len + TILE - 1) / TILE; }

template <bool NT, typename T>
__device__ __forceinline__ T ldx(const char* p) {
    if constexpr (NT) return __builtin_nontemporal_load((const T*)p);
    return *(const T*)p;
}
template <bool NT, int N>
__device__ __forceinline__ void ldg(uint32_t (&dst)[N], int at, const char* p, int bytes) {
    if (bytes == 16) {
        const u32x4 v = ldx<NT, u32x4>(p);
        dst[at] = v.x; dst[at + 1] = v.y; dst[at + 2] = v.z; dst[at + 3] = v.w;
    } else if (bytes == 8) {
        const u32x2 v = ldx<NT, u32x2>(p);
        dst[at] = v.x; dst[at + 1] = v.y;
    } else if (bytes == 4) {
        dst[at] = ldx<NT, uint32_t>(p);
    } else {
        dst[at] = ldx<NT, uint16_t>(p);
    }
}

// Eight f32 as f16 (bf16) parts: x = part 0 + part 1 (+ part 2) up to 2^-22
// (2^-24) of |x|.
template <int KIND>
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&part)[KIND == KV_BF16 ? 3 : 2]) {
    constexpr int NS = KIND == KV_BF16 ? 3 : 2;
    float rest[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) rest[j] = x[j];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        if constexpr (KIND == KV_BF16) {
            bf16x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = (__bf16)rest[j];
                rest[j] -= (float)v[j];
            }
            part[s] = __builtin_bit_cast(u32x4, v);
        } else {
            f16x8 v;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = (_Float16)rest[j];
                rest[j] -= (float)v[j];
            }
            part[s] = __builtin_bit_cast(u32x4, v);
        }
    }
}

template <int KIND>
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    if constexpr (KIND == KV_BF16)
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
}

// Codes as f16.  A dword of codes with their sign bits flipped holds code +
// 128 per byte; put under the byte 0x64 it is the f16 value 1024 + 128 + code.
constexpr uint32_t SIGNS = 0x80808080u, B64 = 0x64646464u;
__device__ __forceinline__ uint32_t codes2(uint32_t bytes, bool high) {
    const uint32_t p = __builtin_amdgcn_perm(B64, bytes, high ? 0x04030402u : 0x04010400u);
    const f16x2 v = __builtin_bit_cast(f16x2, p) - f16x2{(_Float16)1152.0f, (_Float16)1152.0f};
    return __builtin_bit_cast(uint32_t, v);
}

// One wave's state over a segment (some tiles of one unit), head i = lane % 16:
// acc[o][r] belongs to the value dimension of operand o that lane 4c + r loads.
template <int KIND, int NB>
struct Segment {
    static constexpr int D = 32 * NB;
    static constexpr bool Q8 = KIND == KV_Q8;
    static constexpr int NS = KIND == KV_BF16 ? 3 : 2;
    static constexpr int ES = Q8 ? 1 : 2;          // bytes per element
    static constexpr int KW = Q8 ? 2 * NB : 4 * NB;  // dwords of a lane's share of a key tile row
    static constexpr int VW = Q8 ? (NB + 1) / 2 : NB;
    // A value row is read by 16 lanes in runs of 8 elements per lane (128
    // dimensions), then 4 (64) and 2 (32) as head_dim leaves them.
    static constexpr int N8 = NB / 4;
    static constexpr bool N4 = (NB & 2) != 0, N2 = (NB & 1) != 0;

    f32x4 acc[2 * NB];
    float m, l;
    // 8-bit values: the largest weight times value scale so far, against the
    // present maximum, and the exponent of a power of two above it, which acc's
    // sums are relative to
    float vtop;
    int vexp;

    // Rows of whole lines are read once and past the caches (non-temporal: 131071
    // tokens of f16 heads of 128 94.9 -> 91.1 us); rows that share lines are not
    // (2048 tokens x 64 of 8-bit heads of 96: 63 us, non-temporal 84).
    static constexpr bool STREAM = D * ES % 128 == 0;

    // A key row's 128-byte lines, then what is left: 64 and 32 bytes.
    static constexpr int LINES = D * ES / 128;
    static constexpr bool REST64 = (D * ES & 64) != 0, REST32 = (D * ES & 32) != 0;

    // The lane's share of 16 rows: row i (its operand row), which needs the
    // 16-byte chunks 2c and 2c + 1 of every line.  A load instruction takes
    // whole lines, of eight rows: even and odd lanes read chunk 2c and 2c + 1
    // first of the even row, then of the odd one (odd: rows of the pair), and
    // settle() swaps what the other one needs.
    static __device__ __forceinline__ void load_k(uint32_t (&kr)[KW], const char* even, const char* odd, const char* own,
                                                  int c, int i) {
#pragma unroll
        for (int n = 0; n < LINES; ++n) {
            const int at = 128 * n + 32 * c + 16 * (i & 1);
            ldg<STREAM>(kr, 8 * n, even + at, 16);
            ldg<STREAM>(kr, 8 * n + 4, odd + at, 16);
        }
        if constexpr (REST64) ldg<STREAM>(kr, 8 * LINES, own + 128 * LINES + 16 * c, 16);
        if constexpr (REST32) ldg<STREAM>(kr, 8 * LINES + (REST64 ? 4 : 0), own + D * ES - 32 + 8 * c, 8);
    }
    static __device__ __forceinline__ void settle(uint32_t (&kr)[KW], int i) {
        const bool odd = i & 1;
#pragma unroll
        for (int n = 0; n < LINES; ++n)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t x = kr[8 * n + j], y = kr[8 * n + 4 + j];
                // quad_perm [1, 0, 3, 2]: the neighbour's
                const uint32_t px = __builtin_amdgcn_update_dpp(0, x, 0xb1, 0xf, 0xf, true);
                const uint32_t py = __builtin_amdgcn_update_dpp(0, y, 0xb1, 0xf, 0xf, true);
                kr[8 * n + j] = odd ? py : x;
                kr[8 * n + 4 + j] = odd ? y : px;
            }
    }
    static __device__ __forceinline__ void load_v(uint32_t (&vr)[VW], const char* row, int i) {
#pragma unroll
        for (int n = 0; n < N8; ++n) ldg<STREAM>(vr, n * 2 * ES, row + ES * (128 * n + 8 * i), 8 * ES);
        if constexpr (N4) ldg<STREAM>(vr, N8 * 2 * ES, row + ES * (128 * N8 + 4 * i), 4 * ES);
        if constexpr (N2) ldg<STREAM>(vr, (N8 * 2 + (N4 ? 1 : 0)) * ES, row + ES * (128 * N8 + (N4 ? 64 : 0) + 2 * i), 2 * ES);
    }
    // first dimension of the eight that lane c's share of step s holds
    static __device__ __forceinline__ int kdim(int s, int c) {
        constexpr int CH = 16 / ES, PER = 32 / ES / 8;  // dimensions in a chunk; steps of a line
        if (s < PER * LINES) return 128 / ES * (s / PER) + 2 * CH * c + 8 * (s % PER);
        s -= PER * LINES;
        if (REST64 && s < PER / 2) return 128 / ES * LINES + CH * c + 8 * s;
        return D - 32 + 8 * c;  // 32 bytes: 8-bit rows
    }
    // the key operand of step s
    static __device__ __forceinline__ u32x4 key(const uint32_t (&kr)[KW], int s) {
        if constexpr (Q8) {
            const uint32_t x = kr[2 * s] ^ SIGNS, y = kr[2 * s + 1] ^ SIGNS;
            return u32x4{codes2(x, false), codes2(x, true), codes2(y, false), codes2(y, true)};
        } else {
            return u32x4{kr[4 * s], kr[4 * s + 1], kr[4 * s + 2], kr[4 * s + 3]};
        }
    }
    // the value operand o: its element of the lane's eight rows
    static __device__ __forceinline__ u32x4 value(const uint32_t (&vr)[8][VW], int o) {
        uint32_t out[4];
        if constexpr (Q8) {
            const int w = o / 4, x = o % 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t two = __builtin_amdgcn_perm(vr[2 * j + 1][w] ^ SIGNS, vr[2 * j][w] ^ SIGNS,
                                                           x < 2 ? 0x05010400u : 0x07030602u);
                out[j] = codes2(two, x & 1);
            }
        } else {
            const int w = o / 2;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                out[j] = __builtin_amdgcn_perm(vr[2 * j + 1][w], vr[2 * j][w], (o & 1) ? 0x07060302u : 0x05040100u);
        }
        return u32x4{out[0], out[1], out[2], out[3]};
    }

    // Tiles [t, t + n) of sequence b (len tokens) for `rows` heads from query head head0.
    __device__ __forceinline__ void run(const AttnArgs& a, int b, int len, int kvh, int head0, int rows, int t, int n) {
        const int lane = threadIdx.x & 63, c = lane >> 4, i = lane & 15;
        m = -INFINITY;
        l = 0.0f;
        vtop = 0.0f;
        vexp = 0;
#pragma unroll
        for (int o = 0; o < 2 * NB; ++o) acc[o] = f32x4{0, 0, 0, 0};
        if (len <= 0) {
            l = len < 0 ? NAN : 0.0f;
            return;
        }
        const char* kb = (const char*)a.k + (int64_t)kvh * a.head_bytes;
        const char* vb = (const char*)a.v + (int64_t)kvh * a.head_bytes;
        const float* sb = Q8 ? ((lane & 32) ? a.v_scale : a.k_scale) + (int64_t)kvh * a.scale_head : nullptr;
        const int* table = a.table + (int64_t)b * a.table_stride;
        bool bad = false;
        const float pbits = KIND == KV_BF16 ? (float)-log2_up(len) : Q8 ? 0.0f : PBITS;

        // page id of the lane's token (lane % 32) of tile tt; tokens behind the last read as the last
        auto token = [&](int tt) {
            const int tok = TILE * tt + (lane & 31);
            return tok < len ? tok : len - 1;
        };
        auto page_id = [&](int tt) { return table[token(tt) >> a.page_log2]; };
        uint32_t off;        // the row of the lane's token, in 16-byte units from the head's first
        float sc = 0.0f;     // its key (lanes 0..31) or value scale
        auto locate = [&](int id, int tt) {
            const bool out = (uint32_t)id >= (uint32_t)a.n_pages;
            bad |= out;
            const uint32_t pg = out ? 0u : (uint32_t)id, slot = (uint32_t)token(tt) & (uint32_t)(a.page_size - 1);
            off = pg * a.page_units + slot * a.slot_units;
            if constexpr (Q8) sc = sb[(int64_t)pg * a.scale_page + (int64_t)slot * a.scale_slot];
        };
        auto row_of = [&](const char* base, int src) {
            return base + ((uint64_t)(uint32_t)__builtin_amdgcn_ds_bpermute(4 * src, (int)off) << 4);
        };
        uint32_t kr[2][KW], vr[8][VW];
        auto load_keys = [&]() {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                load_k(kr[h], row_of(kb, 16 * h + (i & ~1)), row_of(kb, 16 * h + (i | 1)),
                       REST64 || REST32 ? row_of(kb, 16 * h + i) : kb, c, i);
        };
        auto tok_of = [&](int j) { return (j < 4 ? 0 : 12) + 4 * c + j; };  // token of the lane's k index j
        auto load_values = [&]() {
#pragma unroll
            for (int j = 0; j < 8; ++j) load_v(vr[j], row_of(vb, tok_of(j)), i);
        };

        int id = page_id(t);
        // the query heads, split; lanes past the last head hold zeros
        u32x4 qp[NB][NS];
        float qs;
        {
            const float* qrow = a.q + (int64_t)b * a.q_stride + (int64_t)(head0 + (i < rows ? i : 0)) * D;
            float x[NB][8];
            float top = 0.0f;
#pragma unroll
            for (int s = 0; s < NB; ++s) {
                const f32x4 lo = *(const f32x4*)(qrow + kdim(s, c)), hi = *(const f32x4*)(qrow + kdim(s, c) + 4);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[s][j] = i < rows ? lo[j] : 0.0f;
                    x[s][4 + j] = i < rows ? hi[j] : 0.0f;
                    top = fmaxf(top, fmaxf(fabsf(x[s][j]), fabsf(x[s][4 + j])));
                }
            }
            locate(id, t);
            load_keys();
            if (n > 1) id = page_id(t + 1);
            load_values();
            top = max_c(top);
            // q's factor, a power of two: its exponent field
            int e;
            if constexpr (KIND == KV_BF16) {
                // 2^-12, so that the sum of products passes f32 no sooner than the score, but at
                // least what takes the largest to 2^-60: its parts are normal numbers
                e = 194 - (int)(ubits(top) >> 23);
                e = e < 115 ? 115 : e;
            } else {
                // 2^(13 - floor(log2 top)), kept normal with its inverse
                e = 267 - (int)(ubits(top) >> 23);
                e = e > 253 ? 253 : (e < 1 ? 1 : e);
            }
            const float f = fbits((uint32_t)e << 23);
            qs = fbits((uint32_t)(254 - e) << 23) * a.scale * LOG2E;  // scale * log2(e) may pass f32
#pragma unroll
            for (int s = 0; s < NB; ++s) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[s][j] *= f;
                split8<KIND>(x[s], qp[s]);
            }
        }

        for (int it = 0; it < n; ++it) {
            const int tt = t + it;
            const bool more = it + 1 < n;
            f32x4 s4[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
            settle(kr[0], i);
            settle(kr[1], i);
#pragma unroll
            for (int s = 0; s < NB; ++s)
#pragma unroll
                for (int p = 0; p < NS; ++p)
#pragma unroll
                    for (int h = 0; h < 2; ++h) s4[h] = mfma<KIND>(key(kr[h], s), qp[s][p], s4[h]);
            float s[8], vs[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if constexpr (Q8) {
                    s[j] = s4[j / 4][j % 4] * (qs * from_lane(sc, tok_of(j)));  // the factors alone may leave f32
                    vs[j] = from_lane(sc, 32 + tok_of(j));
                } else {
                    s[j] = s4[j / 4][j % 4] * qs;
                }
            }
            if (TILE * (tt + 1) > len) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (TILE * tt + tok_of(j) >= len) s[j] = -INFINITY;
            }
            if (more) {
                locate(id, tt + 1);
                load_keys();
                if (it + 2 < n) id = page_id(tt + 2);
            }
            float top = s[0];
#pragma unroll
            for (int j = 1; j < 8; ++j) top = fmaxf(top, s[j]);
            top = fmaxf(m, max_c(top));
            const float base = top == -INFINITY ? 0.0f : top;
            const float shift = base - pbits;
            float alpha = __builtin_amdgcn_exp2f(m - base);
            m = top;
            float p[8], sum = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                // f16's offset apart from the maximum
                p[j] = __builtin_amdgcn_exp2f(KIND == KV_F16 ? s[j] - base + pbits : s[j] - shift);
                sum += p[j];
            }
            l = l * alpha + sum;
            if constexpr (Q8) {
                // A value's scale multiplies its probability.  The products are taken relative to
                // a power of two above the head's largest so far, as that has faded since: a far
                // larger scale of a token that weighs nothing takes no bits from the others
                // (relative to the largest scale alone, 1e12 beside a weight of e^-60 lost them all).
                float big = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] *= vs[j];
                    big = fmaxf(big, fabsf(p[j]));
                }
                vtop = fmaxf(vtop * alpha, max_c(big));
                const int e = __builtin_amdgcn_frexp_expf(vtop);
                alpha = __builtin_amdgcn_ldexpf(alpha, vexp - e);
                vexp = e;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    p[j] = __builtin_amdgcn_ldexpf(p[j], 14 - e);
                    // The product as one f32 value: the compiler otherwise rounds it to f16 for the
                    // high part straight from its factors (v_fma_mixlo_f16), which near a tie is not
                    // the f16 that the low part was taken against (2^-11 off, seen about once in 10^4).
                    asm("" : "+v"(p[j]));
                }
            }
            if (__any(alpha != 1.0f)) {
#pragma unroll
                for (int o = 0; o < 2 * NB; ++o) acc[o] *= alpha;
            }
            u32x4 pp[NS];
            split8<KIND>(p, pp);
#pragma unroll
            for (int o = 0; o < 2 * NB; ++o) {
                const u32x4 v = value(vr, o);
#pragma unroll
                for (int q = 0; q < NS; ++q) acc[o] = mfma<KIND>(v, pp[q], acc[o]);
            }
            if (more) load_values();
        }
        if (__any(bad)) l = NAN;
        l = sum_c(l);
        if constexpr (Q8) {
            const float u = 1.0f / one_weight(KIND, len);
#pragma unroll
            for (int o = 0; o < 2 * NB; ++o)
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[o][r] = __builtin_amdgcn_ldexpf(acc[o][r] * (P_UNIT * u), vexp);
            l *= u;
        }
    }

    // f(dimension, the sums of it and the next one or three, times w) over the lane's sums
    template <typename F>
    __device__ __forceinline__ void each(float w, F f) const {
        const int rho = 4 * ((threadIdx.x >> 4) & 3);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int o = 0; o < 8 * N8; o += 4)
                f(128 * (o / 8) + 8 * (rho + r) + o % 8,
                  f32x4{acc[o][r] * w, acc[o + 1][r] * w, acc[o + 2][r] * w, acc[o + 3][r] * w});
            if constexpr (N4) {
                constexpr int o = 8 * N8;
                f(128 * N8 + 4 * (rho + r), f32x4{acc[o][r] * w, acc[o + 1][r] * w, acc[o + 2][r] * w, acc[o + 3][r] * w});
            }
            if constexpr (N2) {
                constexpr int o = 2 * NB - 2;
                f(D - 32 + 2 * (rho + r), f32x2{acc[o][r] * w, acc[o + 1][r] * w});
            }
        }
    }
};

// unit: one_weight of the sequence
__device__ __forceinline__ float lse_of(float m, float l, float unit) {
    return (m + __builtin_amdgcn_logf(l * unit)) * LN2;
}

// A unit: (kv head, block of at most HEADS of its query heads, sequence).
struct Unit {
    int b, kvh, head0, rows;
};
__device__ __forceinline__ Unit unit_of(const AttnArgs& a, int hs, int b) {
    Unit u;
    u.b = b;
    u.kvh = hs / a.blocks_per_kv;
    const int blk = hs - u.kvh * a.blocks_per_kv;
    u.head0 = u.kvh * a.group + blk * a.heads_per_block;
    u.rows = a.group - blk * a.heads_per_block;
    if (u.rows > a.heads_per_block) u.rows = a.heads_per_block;
    return u;
}

// A part: heads_per_block rows of D sums, then (m, l) per row, in whole 16-byte units.
__host__ __device__ __forceinline__ int part_floats(int heads_per_block, int d) {
    return heads_per_block * d + ((2 * heads_per_block + 3) & ~3);
}

// Sum over the wave's lanes up to this one: row shifts within 16 lanes, then
// the rows' last lanes handed on (no LDS).
__device__ __forceinline__ int wave_inclusive(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

// A wave's run [pos, end) of its head space's axis, and where it begins:
// sequence, offset in it.  A unit takes `start` places, for what its start and
// end cost a wave, and then one per tile.
struct Run {
    int pos, end, b, at, start;
};

// Cuts a head space's axis into a.cuts equal chunks, a quarter per wave; *run:
// wave w's of chunk j.  Every wave scans the lengths by itself, its lanes a run
// of consecutive sequences each.  Returns the places of a chunk.
__device__ __forceinline__ int cut(const AttnArgs& a, int j, int w, Run* run) {
    const int lane = threadIdx.x & 63, per = (a.batch + 63) / 64;
    const int b_lo = lane * per, b_hi = b_lo + per < a.batch ? b_lo + per : a.batch;
    int mine = 0;
#pragma unroll 8
    for (int b = b_lo; b < b_hi; ++b) mine += seq_tiles(seq_len(a, b));
    const int incl = wave_inclusive(mine);
    int total = __builtin_amdgcn_readlane(incl, 63);
    const int start = total / 4 / START_MIN >= a.cuts ? UNIT_START : 0;
    const int places = incl + start * b_hi;  // up to the lane's last sequence, and up to its first
    const int before = places - mine - (b_hi > b_lo ? start * (b_hi - b_lo) : 0);
    total += start * a.batch;
    int chunk = (int)(((uint32_t)total + a.cuts - 1) / (uint32_t)a.cuts);
    if (chunk < 4) chunk = 4;  // a place per wave
    const int quarter = (chunk + 3) >> 2;
    const int64_t lo = (int64_t)j * chunk, pos = lo + w * quarter;
    int64_t end = pos + quarter < lo + chunk ? pos + quarter : lo + chunk;
    if (end > total) end = total;
    run->start = start;
    run->pos = run->end = 0;
    if (pos >= end) return chunk;
    run->pos = (int)pos;
    run->end = (int)end;
    const int src = __builtin_ctzll(__ballot(run->pos >= before && run->pos < places));
    int at = __builtin_amdgcn_readlane(before, src), b = src * per;
    if (per > 1)
        for (;; ++b) {
            const int n = seq_tiles(seq_len(a, b)) + start;
            if (run->pos < at + n) break;
            at += n;
        }
    run->b = b;
    run->at = run->pos - at;
    return chunk;
}

template <int KIND, int NB>
__global__ __launch_bounds__(256, occupancy(KIND, NB)) void paged_attn_kernel(const AttnArgs a) {
    constexpr int D = 32 * NB;
    extern __shared__ __attribute__((aligned(16))) float parts[];  // [wave][2] parts
    __shared__ int part_unit[4][2], part_ends[4][2], part_len[4][2];
    __shared__ int2 out_unit;  // the unit that starts here and goes on in the next work groups, and in how many
    const int tid = threadIdx.x, w = uni(tid >> 6), lane = tid & 63;
    const int g = blockIdx.x;

    int chunk = 0, hs, j = 0;
    Run run;
    if (a.per_unit) {
        const int nt = seq_tiles(seq_len(a, g)), quarter = (nt + 3) / 4;
        hs = blockIdx.y;
        run.b = g;
        run.start = 0;
        run.pos = run.at = w * quarter;
        run.end = run.pos + quarter < nt ? run.pos + quarter : nt;
    } else {
        hs = g / a.cuts;
        j = g - hs * a.cuts;
        chunk = cut(a, j, w, &run);
    }
    if (lane < 2) part_unit[w][lane] = -1;
    if (tid == 0) out_unit = make_int2(0, 0);
    if (!a.per_unit && !a.meta_by_unit) __syncthreads();

    const int pf = part_floats(a.heads_per_block, D);
    while (run.pos < run.end) {
        const int b = uni(run.b), at = uni(run.at);
        const int len = uni(seq_len(a, b)), nt = seq_tiles(len);
        const int t = at > run.start ? at - run.start : 0;
        const int left = run.end - run.pos + at - run.start;  // tiles of the unit up to the run's end
        const int n = (left < nt ? left : nt) - t;
        if (n <= 0) break;  // the run ends in the unit's first places: the next one starts it
        const Unit u = unit_of(a, hs, b);
        Segment<KIND, NB> seg;
        seg.run(a, b, len, u.kvh, u.head0, u.rows, t, n);
        const int i = lane & 15;
        if (n == nt) {  // the whole unit: its outputs
            if (i < u.rows) {
                const float inv = len == 0 ? 0.0f : 1.0f / seg.l;
                float* o = a.out + (int64_t)b * a.out_stride + (int64_t)(u.head0 + i) * D;
                seg.each(inv, [&](int d, auto v) { *(decltype(v)*)(o + d) = v; });
                if (a.lse && lane < 16)
                    a.lse[(int64_t)b * a.n_q + u.head0 + i] = len == 0 ? -INFINITY : lse_of(seg.m, seg.l, one_weight(KIND, len));
            }
        } else {
            const int slot = t == 0 ? 1 : 0;  // the unit starts in this wave, or came in from the one before
            float* o = parts + (w * 2 + slot) * pf;
            if (i < a.heads_per_block) {
                float* row = o + i * D;
                seg.each(1.0f, [&](int d, auto v) { *(decltype(v)*)(row + d) = v; });
                if (lane < 16) *(f32x2*)(o + a.heads_per_block * D + 2 * i) = f32x2{seg.m, seg.l};
            }
            if (lane == 0) {
                part_unit[w][slot] = hs * a.batch + b;
                part_ends[w][slot] = t + n == nt;
                part_len[w][slot] = len;
            }
        }
        if (t == 0 && !a.per_unit) {  // work groups after this one that share the unit
            const int follow = n == nt ? 0 : (run.pos - at + run.start + nt - 1) / chunk - j;
            if (a.meta_by_unit) {
                if (lane == 0) a.meta[hs * a.batch + b] = make_int2(g, follow);
            } else if (follow && lane == 0) {
                out_unit = make_int2(hs * a.batch + b, follow);
            }
        }
        run.pos += run.start + nt - at;
        run.at = 0;
        run.b = b + 1;
    }
    __syncthreads();

    // Join the parts of each unit, in token order: a unit that starts here
    // (slot 1 of some wave) or came in from the previous work group (slot 0 of
    // wave 0), and the slots 0 of the following waves up to its end.
    // (Unrolled: left to itself the compiler rolls it for bf16 and 8-bit rows, 0.1
    // us more per call for 97 tokens, 0.6 for 64 sequences of 2048.)
#pragma unroll
    for (int first = -1; first < 4; ++first) {
        const int w0 = first < 0 ? 0 : first, s0 = first < 0 ? 0 : 1;
        const int unit = part_unit[w0][s0];
        if (unit < 0) continue;
        int last = w0;
        bool ends = part_ends[w0][s0];
        while (!ends && last < 3 && part_unit[last + 1][0] == unit) ends = part_ends[++last][0];
        const Unit u = unit_of(a, unit / a.batch, unit % a.batch);
        const bool whole = s0 == 1 && ends;
        float* ws = whole ? nullptr : a.parts + (int64_t)(2 * g + s0) * pf;
        for (int x = tid; x < u.rows * (D / 4); x += 256) {
            const int row = x / (D / 4), d = 4 * (x % (D / 4));
            const float* ml = parts + a.heads_per_block * D + 2 * row;
            float top = -INFINITY;
            for (int v = w0; v <= last; ++v) top = fmaxf(top, ml[(v * 2 + (v == w0 ? s0 : 0)) * pf]);
            const float base = top == -INFINITY ? 0.0f : top;
            f32x4 o = {0, 0, 0, 0};
            float l = 0.0f;
            for (int v = w0; v <= last; ++v) {
                const int p = (v * 2 + (v == w0 ? s0 : 0)) * pf;
                const float f = __builtin_amdgcn_exp2f(ml[p] - base);
                o += *(const f32x4*)(parts + p + row * D + d) * f;
                l += ml[p + 1] * f;
            }
            if (whole) {
                *(f32x4*)(a.out + (int64_t)u.b * a.out_stride + (int64_t)(u.head0 + row) * D + d) = o * (1.0f / l);
                if (a.lse && d == 0) a.lse[(int64_t)u.b * a.n_q + u.head0 + row] = lse_of(top, l, one_weight(KIND, part_len[w0][s0]));
            } else {
                *(f32x4*)(ws + row * D + d) = o;
                if (d == 0) *(f32x2*)(ws + a.heads_per_block * D + 2 * row) = f32x2{top, l};
            }
        }
    }
    if (tid == 0 && !a.per_unit && !a.meta_by_unit) a.meta[g] = out_unit;
}

// The units that span work groups.  A unit's parts are part 1 of the work group it
// starts in and part 0 of the following ones; meta says where and how many.
// An entry per unit, or per work group where the units are more (a work group
// starts at most one such unit): {work group or unit, following work groups}.
struct Split {
    Unit u;
    int g, n;    // first work group, parts
    float unit;  // one_weight of its parts
};
__device__ __forceinline__ Split split_of(const AttnArgs& a) {
    const int2 info = a.meta[blockIdx.x];
    const int unit = a.meta_by_unit ? blockIdx.x : info.x;
    Split s;
    s.g = a.meta_by_unit ? info.x : blockIdx.x;
    s.n = info.y == 0 ? 0 : info.y + 1;
    if (s.n) {
        s.u = unit_of(a, unit / a.batch, unit % a.batch);
        s.unit = one_weight(a.kind, a.kind == KV_F16 ? 1 : seq_len(a, s.u.b));
    }
    return s;
}

struct Sum {
    f32x4 o = {0, 0, 0, 0};
    float m = -INFINITY, l = 0.0f;
    __device__ __forceinline__ void add(f32x4 v, float m2, float l2) {
        const float top = fmaxf(m, m2), base = top == -INFINITY ? 0.0f : top;
        const float f = __builtin_amdgcn_exp2f(m - base), f2 = __builtin_amdgcn_exp2f(m2 - base);
        o = o * f + v * f2;
        l = l * f + l2 * f2;
        m = top;
    }
    // parts p0, p0 + step, .. of a split unit, eight in flight
    __device__ __forceinline__ void parts(const AttnArgs& a, const Split& s, int dim, int row, int d, int p0, int step) {
        const int pf = part_floats(a.heads_per_block, dim), ml0 = a.heads_per_block * dim + 2 * row;
        for (; p0 < s.n; p0 += 8 * step) {
            f32x4 v[8];
            f32x2 ml[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int p = p0 + j * step < s.n ? p0 + j * step : p0;
                const float* at = a.parts + (int64_t)(2 * (s.g + p) + (p == 0 ? 1 : 0)) * pf;
                v[j] = *(const f32x4*)(at + row * dim + d);
                ml[j] = *(const f32x2*)(at + ml0);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (p0 + j * step < s.n) add(v[j], ml[j].x, ml[j].y);
        }
    }
    __device__ __forceinline__ void write(const AttnArgs& a, const Split& s, int dim, int row, int d) const {
        const Unit& u = s.u;
        *(f32x4*)(a.out + (int64_t)u.b * a.out_stride + (int64_t)(u.head0 + row) * dim + d) = o * (1.0f / l);
        if (a.lse && d == 0) a.lse[(int64_t)u.b * a.n_q + u.head0 + row] = lse_of(m, l, s.unit);
    }
};

// Few units of many parts: a work group per unit, query head and 32
// dimensions.  Eight lanes take four dimensions each, 32 lane groups the parts;
// the groups' sums are added within the waves, then across them.  (One CU has
// few enough lines under way at a time that 64 parts of 512 bytes took it 4 us
// more than a line of each; one wave instead of four takes 6 us more for 512
// parts, one kv head of 16 query heads over 131071 tokens 29.0 us for 23.1, and
// 0.1 us less for 64.)
template <int D>
__global__ __launch_bounds__(256) void paged_attn_join_wide_kernel(const AttnArgs a) {
    __shared__ f32x4 so[4][8];
    __shared__ f32x2 sml[4];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int row = blockIdx.y, d = 32 * blockIdx.z + 4 * (lane & 7), pg = threadIdx.x >> 3;
    const Split s = split_of(a);
    if (s.n == 0 || row >= s.u.rows) return;
    Sum x;
    x.parts(a, s, D, row, d, pg, 32);
#pragma unroll
    for (int i = 8; i < 64; i <<= 1) {
        const f32x4 v = {__shfl_xor(x.o.x, i), __shfl_xor(x.o.y, i), __shfl_xor(x.o.z, i), __shfl_xor(x.o.w, i)};
        const float m2 = __shfl_xor(x.m, i), l2 = __shfl_xor(x.l, i);
        x.add(v, m2, l2);
    }
    if (lane < 8) so[w][lane] = x.o;
    if (lane == 0) sml[w] = f32x2{x.m, x.l};
    __syncthreads();
    if (threadIdx.x >= 8) return;
#pragma unroll
    for (int i = 1; i < 4; ++i) x.add(so[i][lane], sml[i].x, sml[i].y);
    x.write(a, s, D, row, d);
}

// Many units: one work group each (its start alone costs 0.5 ns of the whole
// device, so that one per unit, head and 32 dimensions took 12 us for 512
// units of 8 heads).  Threads take (row, four dimensions), and where that
// leaves some over, the parts in groups whose sums are added in order.
template <int D>
__global__ __launch_bounds__(256) void paged_attn_join_kernel(const AttnArgs a) {
    constexpr int DL = D / 4;
    __shared__ f32x4 so[256];
    __shared__ f32x2 sml[256];
    const Split s = split_of(a);
    if (s.n == 0) return;
    const int tid = threadIdx.x, items = s.u.rows * DL;
    for (int base = 0; base < items; base += 256) {
        const int span = items - base < 256 ? items - base : 256;
        int groups = 256 / span;
        if (groups > s.n) groups = s.n;
        const int pg = tid / span, item = base + tid % span, row = item / DL, d = 4 * (item % DL);
        Sum x;
        if (pg < groups) x.parts(a, s, D, row, d, pg, groups);
        if (groups > 1) {
            so[tid] = x.o;
            sml[tid] = f32x2{x.m, x.l};
            __syncthreads();
            if (pg == 0)
                for (int p = 1; p < groups; ++p) x.add(so[p * span + tid], sml[p * span + tid].x, sml[p * span + tid].y);
            __syncthreads();
        }
        if (pg == 0) x.write(a, s, D, row, d);
    }
}

template <int KIND, int NB>
void launch(const AttnArgs& a, hipStream_t st) {
    const size_t lds = (size_t)8 * part_floats(a.heads_per_block, 32 * NB) * sizeof(float);
    if (lds > 64 * 1024)
        (void)hipFuncSetAttribute((const void*)paged_attn_kernel<KIND, NB>, hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    const dim3 grid = a.per_unit ? dim3((unsigned)a.batch, (unsigned)a.head_spaces) : dim3((unsigned)a.groups);
    paged_attn_kernel<KIND, NB><<<grid, 256, lds, st>>>(a);
    if (a.per_unit) return;
    const int64_t units = a.head_spaces * a.batch;
    if (units * 8 <= a.groups)
        paged_attn_join_wide_kernel<32 * NB><<<dim3((unsigned)units, (unsigned)a.heads_per_block, NB), 256, 0, st>>>(a);
    else
        paged_attn_join_kernel<32 * NB><<<dim3((unsigned)(a.meta_by_unit ? units : a.groups)), 256, 0, st>>>(a);
}

template <int KIND>
void launch_kind(const AttnArgs& a, int head_dim, hipStream_t st) {
    switch (head_dim / 32) {
        case 1: launch<KIND, 1>(a, st); break;
        case 2: launch<KIND, 2>(a, st); break;
        case 3: launch<KIND, 3>(a, st); break;
        case 4: launch<KIND, 4>(a, st); break;
        case 5: launch<KIND, 5>(a, st); break;
        case 6: launch<KIND, 6>(a, st); break;
        case 7: launch<KIND, 7>(a, st); break;
        case 8: launch<KIND, 8>(a, st); break;
    }
}

}  // namespace

AttnPlan plan_paged_attention(int64_t batch, int64_t n_q, int64_t n_kv, int64_t head_dim, int64_t capacity, int num_cu) {
    AttnPlan p;
    const int64_t group = n_q / n_kv;
    p.blocks_per_kv = (int)((group + HEADS - 1) / HEADS);
    p.heads_per_block = (int)((group + p.blocks_per_kv - 1) / p.blocks_per_kv);
    p.head_spaces = n_kv * p.blocks_per_kv;
    // work groups: two per CU, or as many as the tables' tiles give a tile per wave
    const int64_t tiles = (capacity + TILE - 1) / TILE;
    const int64_t most = (batch * tiles + 3) / 4;
    const int64_t want = (int64_t)num_cu * 2;
    // Short tables: a work group per unit saves the scan of the lengths and the
    // join, up to a length at which its waves' own tiles take longer, which few
    // units reach sooner than many (8 kv heads of 128, f16, this way against
    // the split: one sequence of 256 tokens 6.9 and 9.1 us, 384 8.9 / 9.6, 512
    // 10.6 / 9.6; 32 sequences of 512 14.6 / 18.7).  Longer, only even lengths
    // gain (32 sequences of 1024 24.7 / 28.4, one of 1024 and 31 of 64 16.7 /
    // 12.2).  Not where the units are many more than fit the device at a time
    // (256 sequences of 64: 22.9 / 18.5).
    const int64_t units = batch * p.head_spaces;
    p.per_unit = tiles <= (2 * units >= num_cu ? 16 : 12) && units <= 4 * (int64_t)num_cu;
    int64_t cuts = want / p.head_spaces;
    if (cuts > most) cuts = most;
    p.cuts = cuts < 1 ? 1 : (int)cuts;
    p.groups = (int)(p.cuts * p.head_spaces);
    p.meta_by_unit = units <= p.groups;
    p.meta_bytes = ((int64_t)p.groups * 8 + 255) / 256 * 256;
    const int64_t part = (int64_t)part_floats(p.heads_per_block, (int)head_dim) * 4;
    p.ws_bytes = !p.per_unit ? p.meta_bytes + (2 * p.groups * part + 255) / 256 * 256 : 0;
    return p;
}

void launch_paged_attention(const AttnArgs& a, int head_dim, hipStream_t st) {
    if (a.kind == KV_F16)
        launch_kind<KV_F16>(a, head_dim, st);
    else if (a.kind == KV_BF16)
        launch_kind<KV_BF16>(a, head_dim, st);
    else
        launch_kind<KV_Q8>(a, head_dim, st);
}

}  // namespace qmm
