// bk_lora.hpp -- low-rank adapters of many requests beside a shared projection (included once for each type of
// adapters, so that the kernels compile side by side).
//
// Token t names an adapter a (or none); with A_a (r x n), B_a (m x r):
//   u_tk = xs_t sum_j x_tj A_a[k][j],   y_ti = base_ti + s_a sum_k u_tk B_a[i][k].
//
// Few tokens: one launch (k_lora). A workgroup takes up to 16 tokens of one adapter and a range of rows of B. It forms u
// for them first (each workgroup of a range anew: r n elements of A, which the caches hold), then its outputs, so
// that nothing passes through memory in between. Its first rows of B and of the base are on their way meanwhile.
// More: u through memory in fp32 (k_lora_down: 32 tokens and a part of the columns a workgroup), then the outputs
// (k_lora_up: 64 tokens and a range of rows), which stream the base and y.
//
// Both products run on the matrix cores in the adapter's type with fp32 sums (x in 8 bits is converted to it without loss); u
// stays fp32 on its way and enters the second in pieces (see pieces()).
#pragma once

#include <algorithm>
#include <type_traits>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

struct LoraArgs {
    const char* x;
    const float* xs;
    const char* a;
    const char* b;
    const float* scales;
    const int32_t* ids;
    const void* base;
    void* y;
    int64_t T, n, m, r, R;
    int64_t ldx, ldb, ldy;
    int btype, ytype;
    int slots, row_blocks;     // workgroups of a token tile: adapters (each takes every slots-th), ranges of rows
    int64_t rows_each;         // rows of a range, a multiple of 64
    // more tokens
    float* u;                  // [split][T][rp]
    int splits, rp, up_slots;  // parts of the columns; r rounded up to 16; slots of k_lora_up
};

// The operands of the first product. A block is the columns of one operand read: a row's share is its 4 lanes'
// kElems contiguous elements each, so columns are multiplied in another order than they lie in, the same for both.
template <typename X, typename W> struct First {
    static constexpr int kElems = 16, kBlock = 64;  // of a lane, of a block
    typedef W op __attribute__((ext_vector_type(8)));
    struct Part { op p[2]; };
    static __device__ __forceinline__ f32x4 mma(const Part& a, const Part& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if constexpr (std::is_same_v<W, __bf16>)
                c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.p[i], b.p[i], c, 0, 0, 0);
            else
                c = __builtin_amdgcn_mfma_f32_16x16x32_f16(a.p[i], b.p[i], c, 0, 0, 0);
        }
        return c;
    }
};
template <> struct First<float, float> {
    static constexpr int kElems = 8, kBlock = 32;
    struct Part { f32x8 p; };
    static __device__ __forceinline__ f32x4 mma(const Part& a, const Part& b, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 8; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.p[i], b.p[i], c, 0, 0, 0);
        return c;
    }
};

template <typename W> struct Vec8 { typedef W type __attribute__((ext_vector_type(8))); };

struct i8 { int8_t v; };
struct e4m3 { uint8_t v; };

// kElems elements of type S from p on, as an operand's part; no alignment beyond the element's is needed.
template <typename F, typename S, typename W>
__device__ __forceinline__ typename F::Part convert(const uint32_t (&w)[F::kElems * sizeof(S) / 4]) {
    typename F::Part out;
    if constexpr (std::is_same_v<S, W>) {
        __builtin_memcpy(&out, w, sizeof out);
    } else {
        W v[16];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            if constexpr (std::is_same_v<S, i8>) {
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * d + e] = (W)(float)(int8_t)(w[d] >> (8 * e));
            } else if constexpr (std::is_same_v<W, __bf16>) {
                const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[d], 1.0f, false);
                const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[d], 1.0f, true);
                v[4 * d] = lo[0], v[4 * d + 1] = lo[1], v[4 * d + 2] = hi[0], v[4 * d + 3] = hi[1];
            } else {
                const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[d], 1.0f, false);
                const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[d], 1.0f, true);
                v[4 * d] = lo[0], v[4 * d + 1] = lo[1], v[4 * d + 2] = hi[0], v[4 * d + 3] = hi[1];
            }
        }
        __builtin_memcpy(&out, v, sizeof out);
    }
    return out;
}
// A lane's elements as they lie in memory, converted where they are used, so that the loads stay in flight until then.
template <typename F, typename S> struct Words {
    uint32_t w[F::kElems * sizeof(S) / 4];
};
template <typename F, typename S>
__device__ __forceinline__ Words<F, S> whole_words(const S* p) {
    Words<F, S> r;
    __builtin_memcpy(r.w, p, sizeof r.w);
    return r;
}
// the first `count` elements (zeros behind them)
template <typename F, typename S, typename W>
__device__ __forceinline__ typename F::Part cut_part(const S* p, int count) {
    S v[F::kElems];
#pragma unroll
    for (int e = 0; e < F::kElems; ++e) {
        S z = {};
        if (e < count) z = p[e];
        v[e] = z;
    }
    uint32_t w[F::kElems * sizeof(S) / 4];
    __builtin_memcpy(w, v, sizeof w);
    return convert<F, S, W>(w);
}

// k_lora (and k_lora_up behind whole row blocks) takes 64 rows of B as four operand tiles; which row is which is free. Lane
// group q's sums of tile j are the four rows from tile_row(j, q) on: 16 bytes of y (fp32: of a tile; 16 bits: of two) lie
// together, and next to them those of the next group, so that an access of 16 bytes a lane covers 64 bytes of a token's
// row.
template <bool kWideY>
__device__ __forceinline__ int tile_row(int j, int q) {
    return kWideY ? 16 * j + 4 * q : 32 * (j >> 1) + 8 * q + 4 * (j & 1);
}
__device__ __forceinline__ f32x4 value4(u32x2 w, int type) {
    f32x4 f;
    if (type == BAKRON_F16) {
        typedef _Float16 h4 __attribute__((ext_vector_type(4)));
        const h4 h = __builtin_bit_cast(h4, w);
#pragma unroll
        for (int e = 0; e < 4; ++e) f[e] = (float)h[e];
    } else {
        f[0] = __uint_as_float(w[0] << 16);
        f[1] = __uint_as_float(w[0] & 0xFFFF0000u);
        f[2] = __uint_as_float(w[1] << 16);
        f[3] = __uint_as_float(w[1] & 0xFFFF0000u);
    }
    return f;
}
// A lane's 16 values of the base in flight (fp32: kWide), `row` the 64 rows' first element.
template <bool kWide, bool kWideY> struct Raw16;
template <bool kWideY> struct Raw16<true, kWideY> {
    u32x4 v[4];
    __device__ __forceinline__ void fetch(const void* base, int64_t row, int q) {
#pragma unroll
        for (int j = 0; j < 4; ++j) __builtin_memcpy(&v[j], (const float*)base + row + tile_row<kWideY>(j, q), 16);
    }
    __device__ __forceinline__ f32x4 value(int j, int) const { return __builtin_bit_cast(f32x4, v[j]); }
};
template <> struct Raw16<false, false> {
    u32x4 v[2];
    __device__ __forceinline__ void fetch(const void* base, int64_t row, int q) {
#pragma unroll
        for (int j = 0; j < 2; ++j) __builtin_memcpy(&v[j], (const uint16_t*)base + row + tile_row<false>(2 * j, q), 16);
    }
    __device__ __forceinline__ f32x4 value(int j, int type) const {
        const u32x4 w = v[j / 2];
        return value4(j % 2 ? u32x2{w[2], w[3]} : u32x2{w[0], w[1]}, type);
    }
};
template <> struct Raw16<false, true> {
    u32x2 v[4];
    __device__ __forceinline__ void fetch(const void* base, int64_t row, int q) {
#pragma unroll
        for (int j = 0; j < 4; ++j) __builtin_memcpy(&v[j], (const uint16_t*)base + row + tile_row<true>(j, q), 8);
    }
    __device__ __forceinline__ f32x4 value(int j, int type) const { return value4(v[j], type); }
};
// The sum of a token without an adapter: -0, which leaves every base as it is, -0 too; 0 where there is no base.
__device__ __forceinline__ f32x4 no_sum(const void* base) {
    const float v = base ? -0.0f : 0.0f;
    return f32x4{v, v, v, v};
}
// y = base + g * sum for a lane's 16 rows of 64 whole ones of a token; raw holds the base.
template <bool kWide, bool kWideY>
__device__ __forceinline__ void finish16(bool based, int btype, const Raw16<kWide, kWideY>& raw, float g, const f32x4 (&sum)[4],
                                         void* y, int ytype, int64_t row, int q) {
    f32x4 v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f32x4 b = {};
        if (based) b = raw.value(j, btype);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] = fmaf(g, sum[j][e], b[e]);
    }
    if constexpr (kWideY) {
#pragma unroll
        for (int j = 0; j < 4; ++j) __builtin_memcpy((float*)y + row + tile_row<true>(j, q), &v[j], 16);
    } else {
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            uint16_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = v[j + e / 4][e % 4];
                h[e] = ytype == BAKRON_F16 ? __builtin_bit_cast(uint16_t, (_Float16)x) : __builtin_bit_cast(uint16_t, (__bf16)x);
            }
            __builtin_memcpy((uint16_t*)y + row + tile_row<false>(j, q), h, 16);
        }
    }
}
// The same for 16 tokens by the 64 rows from i0 on of which the range's end cuts some: through kBox floats of LDS of
// the wave's own, so that one short loop serves every type. `live` lanes' columns are stored; t is lane c's token.
constexpr int kBox = 16 * 68;
template <bool kWideY>
__device__ __forceinline__ void finish_cut(const LoraArgs& a, float* box, int64_t i0, int64_t row1, bool live, int64_t t, float g,
                                           const f32x4 (&sum)[4], int lane) {
    const uint32_t columns = (uint32_t)__ballot(live && lane < 16);
    wave_fence();
#pragma unroll
    for (int j = 0; j < 4; ++j)
        *reinterpret_cast<f32x4*>(box + (lane & 15) * 68 + tile_row<kWideY>(j, lane >> 4)) = g * sum[j];
    wave_fence();
#pragma unroll 1
    for (int col = 0; col < 16; ++col) {
        const int64_t row = i0 + lane, tt = __shfl(t, col);
        if ((columns >> col & 1) && row < row1) {
            float v = box[col * 68 + lane];
            if (a.base) v += load_elem(a.base, a.btype, tt * a.ldb + row);
            store_elem(a.y, a.ytype, tt * a.ldy + row, v);
        }
    }
}

// The first product of RT rank tiles from rank k0 on by the NT column tiles of tokens xr over blocks first, first + step, ..
// of a row and, for the last of them, the block that its end cuts. The lane's sums: ranks 16 j + 4 q .. of column c. Whole
// blocks are counted from `turn` on, and around: rows a power of two apart fall on one memory channel, column by column,
// and tiles of tokens that start in different columns use different ones. (The splits of a tile share its turn.)
template <typename X, typename W, int RT, int NT, int PF>
__device__ __forceinline__ void first_product(const X* const (&xr)[NT], const bool (&live)[NT], const W* ar, int64_t r, int64_t n, int k0, int first,
                                              int step, int turn, int q, int c, f32x4 (&acc)[RT][NT]) {
    using F = First<X, W>;
    using Part = typename F::Part;
    const int blocks = (int)(n / F::kBlock);  // whole ones
    const W* row[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) row[j] = ar + min<int64_t>(k0 + 16 * j + c, r - 1) * n;
    if (first < blocks) {
        // PF blocks in flight (past the last one, the last again); columns past the last token are not read
        Words<F, X> xp[PF][NT];
        Words<F, W> ap[PF][RT];
        const auto fetch = [&](int s, int b) __attribute__((always_inline)) {
            int k = min(b, blocks - 1) + turn;
            k -= k >= blocks ? blocks : 0;
            const int64_t at = (int64_t)k * F::kBlock + q * F::kElems;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                xp[s][t] = Words<F, X>{};
                if (live[t]) xp[s][t] = whole_words<F, X>(xr[t] + at);
            }
#pragma unroll
            for (int j = 0; j < RT; ++j) ap[s][j] = whole_words<F, W>(row[j] + at);
        };
        const auto product = [&](int s) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const Part x = convert<F, X, W>(xp[s][t].w);
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[j][t] = F::mma(convert<F, W, W>(ap[s][j].w), x, acc[j][t]);
            }
        };
        int b = first;
#pragma unroll
        for (int s = 0; s < PF; ++s) fetch(s, b + s * step);
        for (; b + PF * step < blocks; b += PF * step)
#pragma unroll
            for (int s = 0; s < PF; ++s) {
                product(s);
                fetch(s, b + (s + PF) * step);
            }
#pragma unroll
        for (int s = 0; s < PF; ++s)
            if (b + s * step < blocks) product(s);
    }
    if (n % F::kBlock != 0 && first == blocks % step) {  // the block that the row's end cuts
        const int64_t at = (int64_t)blocks * F::kBlock + q * F::kElems;
        const int cut = (int)max<int64_t>(0, min<int64_t>(F::kElems, n - at));
        Part xc[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) xc[t] = cut_part<F, X, W>(xr[t] + min(at, n), cut);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            const Part ac = cut_part<F, W, W>(row[j] + min(at, n), cut);
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[j][t] = F::mma(ac, xc[t], acc[j][t]);
        }
    }
}

// The second product. u, with the token's and the adapter's factors, lies in LDS as operand: in three pieces of the
// adapter's type, of which all but the last are cut off and the last is rounded, so that they hold all 24 bits of u: bf16 has 8 in
// each; fp16 11, of u times the power of two that takes the token's largest value to 2^14 (undone in fp32). fp32: one,
// on the fp32 matrix cores. (fp32 products for all types cost a 64-token batch 3.8 us of 18.)
template <typename W>
constexpr int pieces() {
    return std::is_same_v<W, float> ? 1 : 3;
}
template <typename W>
__device__ __forceinline__ f32x4 second_mma(typename Vec8<W>::type a, typename Vec8<W>::type b, f32x4 c) {
    if constexpr (std::is_same_v<W, __bf16>) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    else if constexpr (std::is_same_v<W, _Float16>) return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    else {
#pragma unroll
        for (int e = 0; e < 8; ++e) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[e], b[e], c, 0, 0, 0);
        return c;
    }
}
// What a value counts for the largest of its token: its magnitude, an infinity or NaN (which stays what it is) nothing.
__device__ __forceinline__ float finite_magnitude(float v) { return fabsf(v) < INFINITY ? fabsf(v) : 0.0f; }
// The power of two for fp16 pieces of values up to `top`, as the exponent; both it and its inverse are normal.
__device__ __forceinline__ int piece_exponent(float top) {
    return top > 0.0f ? min(max(14 - (int)((__float_as_uint(top) >> 23) - 127), -126), 126) : 0;
}
__device__ __forceinline__ float power(int ex) { return __uint_as_float((uint32_t)(127 + ex) << 23); }
// Cuts the next piece off x (the last one: rounds it).
template <typename W, bool kLast>
__device__ __forceinline__ W cut_piece(float& x) {
    W h;
    if constexpr (std::is_same_v<W, float> || kLast) h = (W)x;
    else {
        x = __builtin_canonicalizef(x);
        if constexpr (std::is_same_v<W, __bf16>) h = __builtin_bit_cast(__bf16, (uint16_t)(__float_as_uint(x) >> 16));
        else h = (_Float16)__uint_as_float(x == x ? __float_as_uint(x) & 0xFFFFE000u : __float_as_uint(x));
    }
    const float rest = x - (float)h;
    x = rest == rest ? rest : 0.0f;
    return h;
}

// A lane's 8 ranks from `at` on of the rows of B that tile_row gives it (rows past the last: the last again), 0 from rank
// r on. kEven: r is a multiple of 8, so that all are there or none. Else a read of 8 goes past the row's end, into the
// next row, and what it finds there is dropped; where B itself ends, elements are read one by one.
template <typename W, bool kEven, bool kWideY>
__device__ __forceinline__ void load_rows_of_b(typename Vec8<W>::type (&v)[4], const LoraArgs& a, int64_t adapter, int64_t i0, int at,
                                                int c) {
    const W* b = (const W*)a.b;
    int64_t pos[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        pos[j] = (adapter * a.m + min(i0 + tile_row<kWideY>(j, c >> 2) + (c & 3), a.m - 1)) * a.r + (kEven && at >= a.r ? 0 : at);
    if constexpr (kEven) {
#pragma unroll
        for (int j = 0; j < 4; ++j) __builtin_memcpy(&v[j], b + pos[j], sizeof v[j]);
    } else {
        const int64_t last = a.R * a.m * a.r - 8;
        const bool cut = max(max(pos[0], pos[1]), max(pos[2], pos[3])) > last;
        if (__ballot(cut)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 8; ++e) v[j][e] = at + e < a.r ? b[pos[j] + e] : (W)0.0f;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) __builtin_memcpy(&v[j], b + pos[j], sizeof v[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) v[j][e] = at + e < a.r ? v[j][e] : (W)0.0f;
    }
}

// ---------------------------------------------------------------- few tokens
// Bound by latency: ids, x and A, their sums through LDS, the operands, then y (one token, rank 16, 4096 x 4096: 8.1 us of
// GPU time; 64 tokens of 43 adapters, rank 16, 4096 -> 14336: 16.3). B's first rows and the base, which need nothing of the
// first product, are fetched in front of it, and columns past an adapter's last token are not read (33 -> 25 us for that
// batch). RT: tiles of 16 ranks of a pass of the first product, S: steps of 32 ranks of the second; kPasses: r may be more
// than they take; kEven: a lane's 8 ranks of a step are all there, or none is; kWide, kWideY: the base, and y, is fp32.
// (Branches around loads, and loops around the whole, make the compiler wait for all that is in flight.)
constexpr int kLoraWaves = 8;

template <typename X, typename W, int RT, int S, bool kPasses, bool kEven, bool kWide, bool kWideY>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora(LoraArgs a) {
    using Op = typename Vec8<W>::type;
    constexpr int NW = kLoraWaves, PF = 8 / RT, RP = 16 * RT, NP = pieces<W>();
    constexpr bool kScaled = std::is_same_v<W, _Float16>;
    extern __shared__ __align__(16) char lds[];
    const int steps = kPasses ? (int)((a.r + 31) / 32) : S, pitch = 32 * steps + 4;
    W* ops = (W*)lds;                                // [piece][step][lane][8]
    float* u = (float*)(ops + NP * steps * 512);     // [16 tokens][pitch]
    float* factor = u + 16 * pitch;                  // [16 tokens]
    float* undo = factor + 16;                       // [16 tokens]
    float* red = undo + 16;                          // [wave][RP ranks][17]
    float* box = red + NW * RP * 17;                 // of the wave with a cut row block: at most one of a range
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    // workgroups 8 apart share an XCD: the ranges of one group of tokens run there, for the A that they share
    const int span = blockIdx.x / (8 * a.row_blocks), off = blockIdx.x % (8 * a.row_blocks);
    // (slots outermost: often only the first have work)
    const int group = span * 8 + off % 8, rb = off / 8, tiles = (int)((a.T + 15) / 16), slot = group / tiles;
    const int64_t t0 = (int64_t)(group % tiles) * 16;
    if (slot >= a.slots) return;
    const int64_t row0 = rb * a.rows_each, row1 = min(a.m, row0 + a.rows_each);
    const int tokens = (int)min<int64_t>(16, a.T - t0);
    // the adapter of token c (-1: none); this workgroup's is the slot-th of those that the tile names
    int mine = c < tokens ? a.ids[t0 + c] : 0;
    if (mine < 0 || mine >= a.R) mine = -1;
    uint32_t left = ((uint32_t)1 << tokens) - 1, members = 0;
    int ad = -1;
    for (int i = 0; i <= slot; ++i) {
        if (left == 0) return;
        ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        members = (uint32_t)__ballot(lane < tokens && mine == ad);
        left &= ~members;
    }
    // column c of the products is the c-th token of the adapter (the first again past the last)
    const int count = __popc(members);
    int tok = __builtin_ctz(members);
    {
        uint32_t s = members;
        for (int k = 1; k < count; ++k) {
            s &= s - 1;
            if (c == k) tok = __builtin_ctz(s);
        }
    }
    const int64_t t = t0 + tok;
    const bool live = c < count;
    const int64_t whole = row1 - (row1 - row0) % 64;  // row blocks up to here are whole
    struct Rows {
        Op b[S][4];
        Raw16<kWide, kWideY> raw;
    };
    const auto load_rows = [&](Rows& r, int64_t i0) __attribute__((always_inline)) {
#pragma unroll
        for (int s = 0; s < S; ++s) load_rows_of_b<W, kEven, kWideY>(r.b[s], a, max(ad, 0), min(i0, a.m - 1), 32 * s + 8 * q, c);
        if (a.base && whole > row0) r.raw.fetch(a.base, t * a.ldb + min(i0, whole - 64), q);
    };
    Rows next = {};
    if constexpr (kEven) load_rows(next, row0 + 64 * w);
    if (ad >= 0) {
        if (w == 0 && lane < 16) factor[c] = (a.scales ? a.scales[ad] : 1.0f) * (a.xs ? a.xs[t] : 1.0f);
        const X* const xr[1] = {(const X*)a.x + t * a.ldx};
        const bool lv[1] = {live};
        int k0 = 0;
        do {
            f32x4 acc[RT][1] = {};
            first_product<X, W, RT, 1, PF>(xr, lv, (const W*)a.a + (int64_t)ad * a.r * a.n, a.r, a.n, k0, w, NW, 0, q, c, acc);
            // sums of the waves, in their order
            if (kPasses) __syncthreads();
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int v = 0; v < 4; ++v) red[(w * RP + 16 * j + 4 * q + v) * 17 + c] = acc[j][0][v];
            __syncthreads();
            for (int e = threadIdx.x; e < 16 * RP; e += 64 * NW) {
                const int k = e >> 4, tk = e & 15;
                float s = 0.0f;
#pragma unroll
                for (int i2 = 0; i2 < NW; ++i2) s += red[(i2 * RP + k) * 17 + tk];
                if (k0 + k < 32 * steps) u[tk * pitch + k0 + k] = k0 + k < a.r ? s * factor[tk] : 0.0f;
            }
            k0 += RP;
        } while (kPasses && k0 < 32 * steps);
        if (RP < 32 && !kPasses)
            for (int e = threadIdx.x; e < 16 * 16; e += 64 * NW) u[(e & 15) * pitch + 16 + (e >> 4)] = 0.0f;
        __syncthreads();
        // operands: 32 threads a token
        const int tk = threadIdx.x >> 5, part = threadIdx.x & 31;
        float up = 1.0f;
        if constexpr (kScaled) {
            float top = 0.0f;
            for (int s = 0; s < steps; ++s) top = fmaxf(top, finite_magnitude(u[tk * pitch + 32 * s + part]));
#pragma unroll
            for (int d = 1; d < 32; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
            const int ex = piece_exponent(top);
            up = power(ex);
            if (part == 0) undo[tk] = power(-ex);
        }
        for (int s = 0; s < steps; ++s) {
            float x = u[tk * pitch + 32 * s + part] * up;
#pragma unroll
            for (int p = 0; p < NP; ++p)
                ops[((p * steps + s) * 64 + part / 8 * 16 + tk) * 8 + part % 8] = p == NP - 1 ? cut_piece<W, true>(x) : cut_piece<W, false>(x);
        }
        __syncthreads();
    }
    if constexpr (!kEven) load_rows(next, row0 + 64 * w);
    const float g = kScaled && ad >= 0 ? undo[c] : 1.0f;
    const auto step_product = [&](int s, Op (&b)[4], f32x4 (&acc)[4]) __attribute__((always_inline)) {
        if (kEven && 32 * s + 8 * q >= a.r)
#pragma unroll
            for (int j = 0; j < 4; ++j) b[j] = Op{};
#pragma unroll
        for (int p = NP - 1; p >= 0; --p) {  // the smallest piece first into the sum
            const Op uo = *reinterpret_cast<const Op*>(ops + ((p * steps + s) * 64 + lane) * 8);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = second_mma<W>(b[j], uo, acc[j]);
        }
    };
    const auto product = [&](int64_t i0, Rows& r, f32x4 (&acc)[4]) __attribute__((always_inline)) {
        if (ad < 0) {
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j] = no_sum(a.base);
            return;
        }
#pragma unroll
        for (int s = 0; s < S; ++s) step_product(s, r.b[s], acc);
        if constexpr (kPasses)
            for (int s = S; s < steps; ++s) {
                load_rows_of_b<W, kEven, kWideY>(r.b[0], a, ad, i0, 32 * s + 8 * q, c);
                step_product(s, r.b[0], acc);
            }
    };
    int64_t i0 = row0 + 64 * w;
    for (; i0 < whole; i0 += 64 * NW) {
        Rows cur = next;
        if constexpr (kEven) load_rows(next, i0 + 64 * NW);
        f32x4 acc[4] = {};
        product(i0, cur, acc);
        if (live) finish16<kWide, kWideY>(a.base != nullptr, a.btype, cur.raw, g, acc, a.y, a.ytype, t * a.ldy + i0, q);
        if constexpr (!kEven) load_rows(next, i0 + 64 * NW);
    }
    if (i0 < row1) {
        f32x4 acc[4] = {};
        product(i0, next, acc);
        finish_cut<kWideY>(a, box, i0, row1, live, t, g, acc, lane);
    }
}

// ---------------------------------------------------------------- more tokens
// In one launch, each range of rows would form u anew: 4096 tokens, rank 64, 4096 -> 14336 took 334 us, 88 in two.
constexpr int kDownWaves = 8, kDownTokens = 32, kUpTokens = 64, kUpWaves = 4, kUpRows = 128;

// u of 32 tokens over a part of the columns: [split][token][rp], 0 behind r. A token without an adapter has none.
// Bound by the loads of x and A, which every wave takes straight from memory as operands: 25 us at 4096 tokens, rank 64, 4096
// columns (2.2 GFLOP; x's 34 MB would be 7). One block of loads ahead for 4 rank tiles, two for fewer: with 4 tiles two are
// 33 to 36 us, since a unit then holds fewer waves.
template <typename X, typename W, int RT>
__global__ __launch_bounds__(64 * kDownWaves) void k_lora_down(LoraArgs a) {
    constexpr int NW = kDownWaves, RP = 16 * RT;
    extern __shared__ __align__(16) char lds[];
    float* red = (float*)lds;  // [wave][RP ranks][33]
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15, tk = lane & 31;
    // slots outermost: often only the first has work, and its workgroups are to spread over all XCDs
    const uint32_t tiles = (uint32_t)((a.T + kDownTokens - 1) / kDownTokens);
    const int split = blockIdx.x % a.splits, slot = blockIdx.x / a.splits / tiles;
    const int64_t t0 = (int64_t)(blockIdx.x / a.splits % tiles) * kDownTokens;
    const int tokens = (int)min<int64_t>(kDownTokens, a.T - t0);
    int mine = tk < tokens ? a.ids[t0 + tk] : 0;
    if (mine < 0 || mine >= a.R) mine = -1;
    uint32_t left = (uint32_t)__ballot(lane < tokens && mine >= 0);
    for (int i = 0; left; ++i) {
        const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        const uint32_t members = (uint32_t)__ballot(lane < tokens && mine == ad);
        left &= ~members;
        if (i % a.slots != slot) continue;
        const int count = __popc(members);
        int tok = __builtin_ctz(members);  // lane k < 32: the k-th member (the first again past the last)
        {
            uint32_t s = members;
            for (int k = 1; k < count; ++k) {
                s &= s - 1;
                if (tk == k) tok = __builtin_ctz(s);
            }
        }
        const W* ar = (const W*)a.a + (int64_t)ad * a.r * a.n;
        const int blocks = (int)(a.n / First<X, W>::kBlock), turn = blocks ? (int)(t0 / kDownTokens) * 2 % blocks : 0;
        const X* const x0 = (const X*)a.x + (t0 + __shfl(tok, c)) * a.ldx;
        const X* const x1 = (const X*)a.x + (t0 + __shfl(tok, c + 16)) * a.ldx;
        for (int k0 = 0; k0 < a.rp; k0 += RP) {
            f32x4 acc[RT][2] = {};
            if (count > 16) {
                const X* const xr[2] = {x0, x1};
                const bool lv[2] = {true, c + 16 < count};
                first_product<X, W, RT, 2, RT == 4 ? 1 : 2>(xr, lv, ar, a.r, a.n, k0, split * NW + w, a.splits * NW, turn, q, c, acc);
            } else {
                const X* const xr[1] = {x0};
                const bool lv[1] = {c < count};
                f32x4 one[RT][1] = {};
                first_product<X, W, RT, 1, RT == 4 ? 1 : 2>(xr, lv, ar, a.r, a.n, k0, split * NW + w, a.splits * NW, turn, q, c, one);
#pragma unroll
                for (int j = 0; j < RT; ++j) acc[j][0] = one[j][0];
            }
            __syncthreads();
#pragma unroll
            for (int j = 0; j < RT; ++j)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int v = 0; v < 4; ++v) red[(w * RP + 16 * j + 4 * q + v) * 33 + 16 * t + c] = acc[j][t][v];
            __syncthreads();
            for (int e = threadIdx.x; e < RP * kDownTokens; e += 64 * NW) {
                const int k = e % RP, col = e / RP;
                if (col >= count || k0 + k >= a.rp) continue;
                float s = 0.0f;
#pragma unroll
                for (int i2 = 0; i2 < NW; ++i2) s += red[(i2 * RP + k) * 33 + col];
                uint32_t m = members;  // the col-th member
                for (int k2 = 0; k2 < col; ++k2) m &= m - 1;
                a.u[((int64_t)split * a.T + t0 + __builtin_ctz(m)) * a.rp + k0 + k] = k0 + k < a.r ? s : 0.0f;
            }
        }
    }
}

// k_lora_up takes tokens as the rows of its products and 128 rows of B as the columns, eight tiles: lane c of a tile has 8
// rows of y that lie together (fp32: twice 4), so that 16 lanes cover 256 bytes of a token's row. With B's rows as the
// products' rows, 4 lanes cover 64 bytes, and to read and write no more than base and y in such pieces takes 76 us where a
// copy takes 45 (4096 tokens of 14336 rows in bf16).
template <bool kWideY>
__device__ __forceinline__ int up_row(int j, int c) {
    return kWideY ? 64 * (j >> 2) + 4 * c + (j & 3) : 8 * c + j;
}
// A lane's 8 values of the base in flight, `row` the 128 rows' first element.
template <bool kWide, bool kWideY> struct Raw8 {
    typedef std::conditional_t<kWide, u32x4, u32x2> Four;
    Four v[2];
    __device__ __forceinline__ void fetch(const void* base, int64_t row, int c) {
        typedef std::conditional_t<kWide, float, uint16_t> E;
        if constexpr (!kWideY && !kWide) {
            __builtin_memcpy(v, (const E*)base + row + up_row<kWideY>(0, c), 16);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) __builtin_memcpy(&v[h], (const E*)base + row + up_row<kWideY>(4 * h, c), sizeof(Four));
        }
    }
    __device__ __forceinline__ f32x4 value(int h, int type) const {
        if constexpr (kWide) return __builtin_bit_cast(f32x4, v[h]);
        else return value4(v[h], type);
    }
};
// y = base + g * sum for a lane's 8 rows of 128 whole ones of a token.
template <bool kWide, bool kWideY>
__device__ __forceinline__ void finish8(bool based, int btype, const Raw8<kWide, kWideY>& raw, float g, const float (&sum)[8], void* y,
                                        int ytype, int64_t row, int c) {
    float v[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        f32x4 b = {};
        if (based) b = raw.value(h, btype);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * h + e] = fmaf(g, sum[4 * h + e], b[e]);
    }
    if constexpr (kWideY) {
#pragma unroll
        for (int h = 0; h < 2; ++h) __builtin_memcpy((float*)y + row + up_row<true>(4 * h, c), v + 4 * h, 16);
    } else {
        uint16_t o[8];
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = ytype == BAKRON_F16 ? __builtin_bit_cast(uint16_t, (_Float16)v[e]) : __builtin_bit_cast(uint16_t, (__bf16)v[e]);
        __builtin_memcpy((uint16_t*)y + row + up_row<false>(0, c), o, 16);
    }
}

// y of 64 tokens by a range of rows. Base and y are read and written once (4096 tokens of 14336 rows in bf16: 235 MB, 45 us
// as a copy, and in this kernel without its products; with them 68, 3.5 TB/s; vector instructions 36 % of it, matrix cores
// 13 %, 1.3 waves a SIMD). The rest is the row block's B on its way
// through LDS and a barrier a turn. With each wave reading B as operands for itself it took 111 (16 lanes at 16 lines),
// with 64 rows of B as the products' rows, each wave all 64 tokens, 76. S: steps of 32 ranks.
template <typename W, int S> struct UpShape {
    static constexpr int kBlock = kUpRows * 32 * S;                                 // elements of B in LDS at a time
    static constexpr int kBuffers = kBlock * sizeof(W) <= 16384 ? 2 : 1;            // (two leave room for two workgroups a unit)
    static constexpr size_t kBytes = std::max(kBuffers * kBlock * sizeof(W), kUpWaves * kBox * sizeof(float));
};

template <typename W, int S, bool kEven, bool kWide, bool kWideY>
__global__ __launch_bounds__(64 * kUpWaves) __attribute__((amdgpu_waves_per_eu(2))) void k_lora_up(LoraArgs a) {
    using Op = typename Vec8<W>::type;
    constexpr int NT = kUpTokens / 16, NP = pieces<W>();
    constexpr bool kScaled = std::is_same_v<W, _Float16>;
    extern __shared__ __align__(16) char lds[];
    W* blocks = (W*)lds;                                       // [buffer][kBlock]
    float* box = (float*)lds;                                  // [wave][kBox], where no blocks are
    W* ops = (W*)(lds + UpShape<W, S>::kBytes);                // [piece][step][tile][lane][8]
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const uint32_t tiles = (uint32_t)((a.T + kUpTokens - 1) / kUpTokens);
    const int slot = blockIdx.x / a.row_blocks / tiles;  // outermost: often only the first has work
    const int64_t t0 = (int64_t)(blockIdx.x / a.row_blocks % tiles) * kUpTokens;
    // whole row blocks first; the last range is that of the rows behind them
    const int64_t whole = a.m / kUpRows * kUpRows, row0 = min((blockIdx.x % a.row_blocks) * a.rows_each, whole);
    const int64_t row1 = row0 < whole ? min(whole, row0 + a.rows_each) : a.m;
    const int tokens = (int)min<int64_t>(kUpTokens, a.T - t0);
    int mine = lane < tokens ? a.ids[t0 + lane] : -1;
    if (mine < 0 || mine >= a.R) mine = -1;
    // the tokens of this slot's adapters (no adapter counts as one): every slots-th of those that the tile names
    uint64_t ours = 0;
    {
        uint64_t left = __ballot(lane < tokens);
        for (int i = 0; left; ++i) {
            const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            const uint64_t members = __ballot(lane < tokens && mine == ad);
            left &= ~members;
            if (i % a.up_slots == slot) ours |= members;
        }
    }
    if (ours == 0) return;
    // four threads a token, ranks 4 part .., 16 apart
    const int ut = threadIdx.x >> 2, part = threadIdx.x & 3, uad = __shfl(mine, ut & 63);
    float undo = 1.0f;  // of token ut; the wave's token j is its lanes' 4 j ..
    if (ut < kUpTokens) {
        const int t = ut, ad = uad;
        const float f = ad < 0 ? 0.0f : (a.scales ? a.scales[ad] : 1.0f) * (a.xs ? a.xs[t0 + t] : 1.0f);
        f32x4 v[2 * S];
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * S; ++i) {
            const int k = 16 * i + 4 * part;
            v[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (ad >= 0 && k < a.rp && (ours >> t & 1)) {
                for (int s = 0; s < a.splits; ++s)
                    v[i] += *reinterpret_cast<const f32x4*>(a.u + ((int64_t)s * a.T + t0 + t) * a.rp + k);
                v[i] *= f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, finite_magnitude(v[i][e]));
        }
        if constexpr (kScaled) {
            top = fmaxf(top, __shfl_xor(top, 1));
            top = fmaxf(top, __shfl_xor(top, 2));
            const int ex = piece_exponent(top);
            const float up = power(ex);
#pragma unroll
            for (int i = 0; i < 2 * S; ++i) v[i] *= up;
            undo = power(-ex);
        }
#pragma unroll
        for (int i = 0; i < 2 * S; ++i) {
            const int k = 16 * i + 4 * part;
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                W h[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float x = v[i][e];
                    h[e] = p == NP - 1 ? cut_piece<W, true>(x) : cut_piece<W, false>(x);
                    v[i][e] = x;
                }
                __builtin_memcpy(ops + ((((p * S + k / 32) * NT + (t >> 4)) * 64 + k % 32 / 8 * 16 + (t & 15)) * 8 + k % 8), h, sizeof h);
            }
        }
    }
    __syncthreads();
    if (row0 == whole) {  // a wave for 16 tokens
        uint64_t left = ours & ((uint64_t)0xFFFF << (16 * w));
        while (left) {
            const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
            const uint64_t members = __ballot(lane < tokens && lane >> 4 == w && mine == ad);
            left &= ~members;
#pragma unroll 1
            for (int64_t i0 = row0; i0 < row1; i0 += 64) {
                f32x4 sum[4] = {};
                if (ad < 0)
#pragma unroll
                    for (int j = 0; j < 4; ++j) sum[j] = no_sum(a.base);
#pragma unroll 1
                for (int s = 0; s < S && 32 * s < a.r && ad >= 0; ++s) {
                    Op b[4];
                    load_rows_of_b<W, kEven, kWideY>(b, a, ad, i0, 32 * s + 8 * q, c);
                    if (kEven && 32 * s + 8 * q >= a.r)
#pragma unroll
                        for (int j = 0; j < 4; ++j) b[j] = Op{};
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p) {
                        const Op uo = *reinterpret_cast<const Op*>(ops + (((p * S + s) * NT + w) * 64 + lane) * 8);
#pragma unroll
                        for (int j = 0; j < 4; ++j) sum[j] = second_mma<W>(b[j], uo, sum[j]);
                    }
                }
                finish_cut<kWideY>(a, box + w * kBox, i0, row1, members >> (16 * w) >> c & 1, t0 + min(16 * w + c, tokens - 1),
                                   kScaled ? __shfl(undo, 4 * c) : 1.0f, sum, lane);
            }
        }
        return;
    }
    // a wave: 16 of the tokens by 128 rows at a time, whose B the waves bring to LDS together, in the order of the operands:
    // [step][tile][lane][8], 2 S pieces of 8 ranks a thread
    const uint64_t own = ours & ((uint64_t)0xFFFF << (16 * w)), some = own ? own : ours;
    const auto token = [&](int v) __attribute__((always_inline)) { return 16 * w + 4 * q + v; };
    const auto piece = [&](int i, int* row) __attribute__((always_inline)) {
        const int u = threadIdx.x + 64 * kUpWaves * i;
        *row = u / (4 * S);
        return u % (4 * S);
    };
    const auto load_b = [&](Op (&b)[2 * S], int ad, int64_t i0) __attribute__((always_inline)) {
        int64_t pos[2 * S], top = 0;
#pragma unroll
        for (int i = 0; i < 2 * S; ++i) {
            int row;
            const int at = 8 * piece(i, &row);
            pos[i] = (ad * a.m + i0 + row) * a.r + (kEven && at >= a.r ? 0 : at);
            top = max(top, pos[i]);
        }
        if (kEven || __ballot(top > a.R * a.m * a.r - 8) == 0) {  // (as load_rows_of_b)
#pragma unroll
            for (int i = 0; i < 2 * S; ++i) __builtin_memcpy(&b[i], (const W*)a.b + pos[i], sizeof b[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 2 * S; ++i) {
                int row;
                const int at = 8 * piece(i, &row);
#pragma unroll
                for (int e = 0; e < 8; ++e) b[i][e] = at + e < a.r ? ((const W*)a.b)[pos[i] + e] : (W)0.0f;
            }
        }
    };
    const auto put_b = [&](const Op (&b)[2 * S], W* to) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 2 * S; ++i) {
            int row;
            const int k = piece(i, &row), tile = kWideY ? row / 64 * 4 + row % 4 : row % 8, col = kWideY ? row % 64 / 4 : row / 8;
            Op o = b[i];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 8 * k + (kEven ? 0 : e) < a.r ? o[e] : (W)0.0f;
            *reinterpret_cast<Op*>(to + (((k / 4) * 8 + tile) * 64 + k % 4 * 16 + col) * 8) = o;
        }
    };
    // a base of 16 bits is one row block ahead
    constexpr bool kAhead = !kWide;
    typedef Raw8<kWide, kWideY> Raw;
    // (of tokens of other slots, or past the last, the base is not read: the first of ours again)
    const auto load_base = [&](Raw (&raw)[4], int64_t i0) __attribute__((always_inline)) {
        if (a.base)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                raw[v].fetch(a.base, (t0 + (own >> token(v) & 1 ? token(v) : (int)__builtin_ctzll(some))) * a.ldb + i0, c);
    };
    float g[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) g[v] = kScaled ? __shfl(undo, 4 * (4 * q + v)) : 1.0f;
    // turns: the adapters of a row block, then those of the next, for all waves alike
    struct Turn {
        int64_t i0;
        uint64_t left, members;
        int ad;
    };
    const auto pick = [&](Turn& t) __attribute__((always_inline)) {
        t.ad = __builtin_amdgcn_readlane(mine, __builtin_ctzll(t.left));
        t.members = __ballot(lane < tokens && mine == t.ad);
        t.left &= ~t.members;
    };
    Turn cur = {row0, ours, 0, 0};
    pick(cur);
    Op stage[2 * S];
    load_b(stage, max(cur.ad, 0), cur.i0);
    Raw raw[4], next[4] = {};
    if (kAhead) load_base(next, cur.i0);
    bool fresh = true;  // the first turn of its row block
    for (int buffer = 0;; buffer = (buffer + 1) % UpShape<W, S>::kBuffers) {
        W* const block = blocks + buffer * UpShape<W, S>::kBlock;
        put_b(stage, block);
        const bool began = fresh;
        Turn then = cur;
        fresh = cur.left == 0;
        if (fresh) {
            then.i0 += kUpRows;
            then.left = ours;
        }
        const bool more = then.i0 < row1;
        pick(then);
        if (more) load_b(stage, max(then.ad, 0), then.i0);
        if (began) {
            if (!kAhead) {
                load_base(raw, cur.i0);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) raw[v] = next[v];
                if (cur.i0 + kUpRows < row1) load_base(next, cur.i0 + kUpRows);
            }
        }
        __syncthreads();
        const uint64_t members = cur.members & own;
        if (members) {
            f32x4 acc[8] = {};
            if (cur.ad < 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[j] = no_sum(a.base);
            } else {
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int p = NP - 1; p >= 0; --p) {  // the smallest piece first into the sum
                        const Op uo = *reinterpret_cast<const Op*>(ops + (((p * S + s) * NT + w) * 64 + lane) * 8);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            acc[j] = second_mma<W>(uo, *reinterpret_cast<const Op*>(block + ((s * 8 + j) * 64 + lane) * 8), acc[j]);
                    }
            }
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (members >> token(v) & 1) {
                    float f[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] = acc[j][v];
                    finish8<kWide, kWideY>(a.base != nullptr, a.btype, raw[v], kScaled ? g[v] : 1.0f, f, a.y, a.ytype,
                                           (t0 + token(v)) * a.ldy + cur.i0, c);
                }
        }
        if (!more) break;
        if (UpShape<W, S>::kBuffers == 1) __syncthreads();
        cur = then;
    }
}

template <typename X, typename W, int RT, int S, bool kPasses, bool kEven>
void launch_few(const LoraArgs& a, hipStream_t stream) {
    constexpr int NW = kLoraWaves;
    const bool wide = a.base && a.btype == BAKRON_F32, wide_y = a.ytype == BAKRON_F32;
    const size_t steps = kPasses ? (size_t)(a.r + 31) / 32 : S, np = pieces<W>();
    const size_t lds = np * steps * 512 * sizeof(W) + sizeof(float) * (16 * (32 * steps + 4) + 32 + NW * 16 * RT * 17 + kBox);
    const int64_t groups = (a.T + 15) / 16 * a.slots;
    const dim3 grid((unsigned)((groups + 7) / 8 * 8 * a.row_blocks)), threads(64 * NW);
    if (wide_y) {
        if (wide) hipLaunchKernelGGL((k_lora<X, W, RT, S, kPasses, kEven, true, true>), grid, threads, lds, stream, a);
        else hipLaunchKernelGGL((k_lora<X, W, RT, S, kPasses, kEven, false, true>), grid, threads, lds, stream, a);
    } else {
        if (wide) hipLaunchKernelGGL((k_lora<X, W, RT, S, kPasses, kEven, true, false>), grid, threads, lds, stream, a);
        else hipLaunchKernelGGL((k_lora<X, W, RT, S, kPasses, kEven, false, false>), grid, threads, lds, stream, a);
    }
}

template <typename X, typename W, int RT>
void launch_down(const LoraArgs& a, hipStream_t stream) {
    const int64_t tiles = (a.T + kDownTokens - 1) / kDownTokens;
    hipLaunchKernelGGL((k_lora_down<X, W, RT>), dim3((unsigned)(tiles * a.slots * a.splits)), dim3(64 * kDownWaves),
                       sizeof(float) * kDownWaves * 16 * RT * 33, stream, a);
}

template <typename W, int S, bool kEven, bool kWideY>
void launch_up(const LoraArgs& a, hipStream_t stream) {
    const int64_t tiles = (a.T + kUpTokens - 1) / kUpTokens;
    constexpr size_t lds = UpShape<W, S>::kBytes + pieces<W>() * S * (kUpTokens / 16) * 512 * sizeof(W);
    const dim3 grid((unsigned)(tiles * a.row_blocks * a.up_slots)), threads(64 * kUpWaves);
    if (a.base && a.btype == BAKRON_F32) hipLaunchKernelGGL((k_lora_up<W, S, kEven, true, kWideY>), grid, threads, lds, stream, a);
    else hipLaunchKernelGGL((k_lora_up<W, S, kEven, false, kWideY>), grid, threads, lds, stream, a);
}
template <typename W, bool kWideY>
void launch_up_ranks(const LoraArgs& a, hipStream_t stream) {
    if (a.r % 8 != 0 && a.r <= 32) launch_up<W, 1, false, kWideY>(a, stream);
    else if (a.r % 8 != 0) launch_up<W, 4, false, kWideY>(a, stream);
    else if (a.r <= 32) launch_up<W, 1, true, kWideY>(a, stream);
    else if (a.r <= 64) launch_up<W, 2, true, kWideY>(a, stream);
    else launch_up<W, 4, true, kWideY>(a, stream);
}

// One launch or two, us of a call, one and two. In one launch every range of rows forms u anew, in two a tile takes a turn an
// adapter; ids lie on the device, so the rule cannot see whether adapters are mixed, and its sizes are those that the
// workspace's size is asked for by, T and r.
//   r = 16, bf16, mixed adapters (one adapter):
//     4096 x 4096:  16 tokens 9.1 12.8; 64 10.6 19.8 (12.9 14.8); 128 13.2 22.3 (15.2 15.0); 192 17.8 31.8 (19.5 15.1)
//     4096 -> 14336: 64 tokens 16.4 25.8 (18.7 15.0); 128 24.4 39.0 (26.2 15.2); 192 39.5 53.2 (41.1 15.6); 256 39.9 69.7
//   Up to 128 tokens one launch is ahead by more where adapters are mixed than it is behind where there is one; above, behind by
//   more, up to 2.6 times.
//   fp32 and long rows, whose u takes longer, would rather have two where tokens are few: fp32, r = 16, 4096 x 4096, one token
//     15.0 13.0, 64 18.6 28.8 (24.0 18.6); 8192 -> 4096, one token 23.5 13.3, 64 27.5 29.9 (37.8 19.0); bf16, 11008 -> 4096, one token
//     16.6 11.2, 64 19.8 24.4 (26.4 17.0). (256 KB of an adapter's A are the border for up to 16 tokens, 512 KB for more.)
//   Rank 64, one token, bf16, 4096 x 4096: one launch 21.7, two 15.2. Above 128, u's pieces pass k_lora_up's LDS and registers.
inline bool lora_few(int64_t T, int64_t r) { return (T <= 128 && r <= 32) || r > 128; }

template <typename X, typename W>
void launch_lora_types(const LoraArgs& a, hipStream_t stream) {
    if (lora_few(a.T, a.r)) {
        if (a.r % 8 != 0 && a.r <= 16) launch_few<X, W, 1, 1, false, false>(a, stream);
        else if (a.r % 8 != 0) launch_few<X, W, 4, 1, true, false>(a, stream);
        else if (a.r <= 16) launch_few<X, W, 1, 1, false, true>(a, stream);
        else if (a.r <= 32) launch_few<X, W, 2, 1, false, true>(a, stream);
        else launch_few<X, W, 4, sizeof(W) == 4 ? 1 : 2, true, true>(a, stream);
        return;
    }
    if (a.r <= 16) launch_down<X, W, 1>(a, stream);
    else if (a.r <= 32) launch_down<X, W, 2>(a, stream);
    else launch_down<X, W, 4>(a, stream);
    if (a.ytype == BAKRON_F32) launch_up_ranks<W, true>(a, stream);
    else launch_up_ranks<W, false>(a, stream);
}

// by the type of x; W that of the adapters
template <typename W>
void launch_lora_adapters(const LoraArgs& a, int xtype, hipStream_t stream) {
    if constexpr (std::is_same_v<W, float>) launch_lora_types<float, float>(a, stream);
    else if (xtype == BAKRON_I8) launch_lora_types<i8, W>(a, stream);
    else if (xtype == BAKRON_E4M3) launch_lora_types<e4m3, W>(a, stream);
    else launch_lora_types<W, W>(a, stream);
}

}  // namespace bk
