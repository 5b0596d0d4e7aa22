// bk_matvec.hpp -- products of token rows with packed low-bit weights (included once for
// each type of x, so that the kernels compile side by side).
//
// The solve leaves a layer as codes c_ij in {0..Lq}, Lq = 2^bits - 1, and scales; the
// weight it stands for is w_ij = s_i,g(j) v_ij with v_ij = c_ij - Lq/2. For T tokens
//   y_ti = a_t sum_g s_ig sum_{j in group g} x_tj v_ij.
// v is a half-integer of at most 4 bits, so it is exact in bf16, fp16, e4m3 and (times a
// power of two) int8: the inner sums run on the matrix cores with exact products and
// fp32 (int8: exact int32) accumulation, and only the group's scale is applied to the
// sum, in fp32. Nothing is rounded below 32 bits before the output.
//
// Packed layout (k_pack). Storage width W = 2 for bits <= 2, else 4; a code of fewer bits
// is moved to the middle of the wider grid, c' = c + (2^W - 2^bits) / 2, which leaves v
// as it is, so the products know W only. A tile is 16 rows, a chunk 128 columns; the
// 256 W bytes of (tile, chunk) are contiguous, chunks of a tile follow each other, and
// lane l of a wave owns 4 W of the bytes: row l % 16 and, of each of the chunk's four
// 32-column steps, the 8 columns 8 (l / 16) + 0..7, which is its share of the B operand of
// a 16x16x32 MFMA. So a wave streams its weights in whole contiguous loads and no value
// moves between lanes. A weight is kept as sign and magnitude: s = (v < 0), k = |v| - 1/2.
//   W = 4: dword j is step j; low nibbles of its bytes are columns 0..3, high ones 4..7;
//          nibble = s k2 k1 k0.
//   W = 2: dword j is steps 2j (a) and 2j + 1 (b); nibble i is column i of both:
//          s_a s_b k_a k_b.
// Behind the codes: the scales as float [tile][group][16], zero where padded.
#pragma once

#include <algorithm>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowTile = 16;
constexpr int kStep = 32;         // columns of one MFMA
constexpr int kChunk = 128;       // columns of a chunk
constexpr int kSteps = kChunk / kStep;
constexpr int kWaves = 8;         // waves of a product workgroup that split the columns
constexpr int kMvThreads = 64 * kWaves;
constexpr int kFew = 4;           // tokens that the kernel with x in LDS takes
constexpr int kFewLds = 65536;    // bytes of x that it stages at a time

struct MvArgs {
    const char* codes;
    const float* scales;
    const char* x;
    const float* xs;
    void* y;
    int64_t m, n, T, ldx, ldy;
    int64_t nc, ngp;   // chunks, and groups as stored
    uint32_t tiles;
    int gshift;        // the group of scale unit u (a chunk, or a step where groups are shorter) is u >> gshift
    int ytype;
};

// ---------------------------------------------------------------- operands
enum Math { kBF16, kF16, kF8, kI8, kF32 };

template <int MATH> struct Mt;
template <> struct Mt<kBF16> {
    using Op = bf16x8;
    using Acc = f32x4;
    static constexpr int kBytes = 2, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mt<kF32> : Mt<kBF16> {
    static constexpr int kBytes = 4, kPieces = 3;
};
template <> struct Mt<kF16> {
    using Op = f16x8;
    using Acc = f32x4;
    static constexpr int kBytes = 2, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mt<kF8> {
    using Op = u32x2;
    using Acc = f32x4;
    static constexpr int kBytes = 1, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_fp8_fp8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c,
                                                          0, 0, 0);
    }
};
template <> struct Mt<kI8> {
    using Op = u32x2;
    using Acc = i32x4;
    static constexpr int kBytes = 1, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0,
                                                     0);
    }
};

// What the weight operand holds, as a multiple of v: e4m3 bytes hold 2 |v| in the three
// low mantissa bits of the subnormal range and the first binade, where e4m3 is linear
// (value = bits * 2^-9, so v 2^-8); int8 holds 16 v (W = 4) or 64 v (W = 2); bf16 and
// fp16 hold v. `unit` undoes it on the finished sum; powers of two, exact.
template <int MATH, int W>
constexpr float unit() {
    return MATH == kF8 ? 256.0f : MATH == kI8 ? (W == 4 ? 1.0f / 16 : 1.0f / 64) : 1.0f;
}

// 4 weights of W = 4 as e4m3 bytes: sign to bit 7, k to bits 3..1, bit 0 set.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
    return ((w << 1) & 0x0E0E0E0Eu) | 0x01010101u | ((w << 4) & 0x80808080u);
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
    return ((w >> 3) & 0x0E0E0E0Eu) | 0x01010101u | (w & 0x80808080u);
}

__device__ __forceinline__ bf16x8 from_e4m3(uint32_t lo, uint32_t hi, bf16x8) {
    const bf16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 256.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 256.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 256.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 256.0f, true)};
    return __builtin_bit_cast(bf16x8, p);
}
__device__ __forceinline__ f16x8 from_e4m3(uint32_t lo, uint32_t hi, f16x8) {
    const f16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 256.0f, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 256.0f, true),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 256.0f, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 256.0f, true)};
    return __builtin_bit_cast(f16x8, p);
}
// 8 weights of W = 2 as e2m1 nibbles s 0 k 1: e2m1 holds 0.5 and 1.5 there, which is |v|.
__device__ __forceinline__ bf16x8 from_e2m1(uint32_t q, bf16x8) {
    const bf16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 0),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 1),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 2),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, 1.0f, 3)};
    return __builtin_bit_cast(bf16x8, p);
}
__device__ __forceinline__ f16x8 from_e2m1(uint32_t q, f16x8) {
    const f16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3)};
    return __builtin_bit_cast(f16x8, p);
}

// A lane's share of a chunk.
template <int W> struct Share;
template <> struct Share<4> { using T = u32x4; };
template <> struct Share<2> { using T = u32x2; };

// The B operand of step `st` of a chunk.
template <int MATH, int W>
__device__ __forceinline__ typename Mt<MATH>::Op weights(typename Share<W>::T d, int st) {
    using Op = typename Mt<MATH>::Op;
    if constexpr (W == 4) {
        uint32_t w = d[st];
        if constexpr (MATH == kF8) {
            return Op{e4m3_lo(w), e4m3_hi(w)};
        } else if constexpr (MATH == kI8) {
            // to two's complement: k -> 7 - k under a sign, then 16 (-8 s + k) + 8 = 16 v
            const uint32_t n = w & 0x88888888u;
            w ^= n - (n >> 3);
            return Op{((w << 4) & 0xF0F0F0F0u) | 0x08080808u, (w & 0xF0F0F0F0u) | 0x08080808u};
        } else {
            return from_e4m3(e4m3_lo(w), e4m3_hi(w), Op{});
        }
    } else {
        uint32_t w = d[st >> 1];
        if constexpr (MATH == kF8 || MATH == kI8) {
            // even nibbles give columns 0 2 4 6, odd ones 1 3 5 7 (even_odd does the same to x)
            if constexpr (MATH == kI8) w ^= (w >> 2) & 0x33333333u;
            if (st & 1) w <<= 1;  // step b into the places of step a: sign at bit 3, k at bit 1
            if constexpr (MATH == kF8)
                return Op{((w << 4) & 0x80808080u) | (w & 0x02020202u) | 0x01010101u,
                          (w & 0x80808080u) | ((w >> 4) & 0x02020202u) | 0x01010101u};
            else
                return Op{((w << 4) & 0x80808080u) | ((w << 5) & 0x40404040u) | 0x20202020u,
                          (w & 0x80808080u) | ((w << 1) & 0x40404040u) | 0x20202020u};
        } else {
            if (st & 1) w <<= 1;
            return from_e2m1((w & 0xAAAAAAAAu) | 0x11111111u, Op{});
        }
    }
}

// 8 bytes of x in the order of the 8-bit operands of W = 2.
__device__ __forceinline__ u32x2 even_odd(u32x2 x) {
    return u32x2{__builtin_amdgcn_perm(x[1], x[0], 0x06040200u), __builtin_amdgcn_perm(x[1], x[0], 0x07050301u)};
}

// fp32 as three bf16 pieces, cut by truncation: 8 significant bits each, their sum is x
// exactly. An infinity or NaN stays in the first piece (the others would be NaN).
__device__ __forceinline__ void split3(const float (&x)[8], bf16x8 (&p)[3]) {
    uint32_t h[8], m[8], l[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t b = __builtin_bit_cast(uint32_t, x[e]);
        const bool special = (b & 0x7F800000u) == 0x7F800000u;
        h[e] = (b & 0xFFFF0000u) | ((special && (b & 0x7FFFFFu)) ? 0x00400000u : 0u);
        const float r = x[e] - __builtin_bit_cast(float, b & 0xFFFF0000u);
        m[e] = special ? 0u : __builtin_bit_cast(uint32_t, r) & 0xFFFF0000u;
        l[e] = special ? 0u : __builtin_bit_cast(uint32_t, r - __builtin_bit_cast(float, m[e]));
    }
    const auto pack = [](const uint32_t (&a)[8]) {
        u32x4 d;
#pragma unroll
        for (int e = 0; e < 4; ++e) d[e] = __builtin_amdgcn_perm(a[2 * e + 1], a[2 * e], 0x07060302u);
        return __builtin_bit_cast(bf16x8, d);
    };
    p[0] = pack(l);
    p[1] = pack(m);
    p[2] = pack(h);
}

// The A operand from 8 elements of x at `src` (in LDS or in registers).
template <int MATH, int W>
__device__ __forceinline__ void operand(const char* src, typename Mt<MATH>::Op (&p)[Mt<MATH>::kPieces]) {
    constexpr int kB = Mt<MATH>::kBytes;
    if constexpr (MATH == kF32) {
        float x[8];
        __builtin_memcpy(x, __builtin_assume_aligned(src, 16), sizeof x);
        split3(x, p);
    } else {
        __builtin_memcpy(&p[0], __builtin_assume_aligned(src, 8 * kB), 8 * kB);
        if constexpr (W == 2 && kB == 1) p[0] = even_odd(p[0]);
    }
}

// ---------------------------------------------------------------- the products
// In all of them A = x (rows are tokens) and B = the weights, so a lane's four sums are
// four tokens of one weight row and share its scale. The sums are scaled every FS steps: a
// chunk (FS = 4), or a step where groups are shorter than a chunk (FS = 1).

// A wave's chunks of R row tiles with their scales, PF chunks ahead of their use.
template <int W, int FS, int R, int PF>
struct Stream {
    using Sh = typename Share<W>::T;
    static constexpr int kUnits = kSteps / FS;
    const Sh* wp[R];
    const float* sp[R];
    int gshift;
    Sh d[PF][R];
    float s[PF][R][kUnits];
    __device__ __forceinline__ Stream(const MvArgs& a, int64_t tile0, int lane) : gshift(a.gshift) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tile = min(tile0 + r, (int64_t)a.tiles - 1);
            wp[r] = reinterpret_cast<const Sh*>(a.codes) + tile * a.nc * 64 + lane;
            sp[r] = a.scales + tile * a.ngp * 16 + (lane & 15);
        }
    }
    __device__ __forceinline__ void fetch(int slot, int64_t c) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            d[slot][r] = wp[r][c * 64];
#pragma unroll
            for (int f = 0; f < kUnits; ++f) s[slot][r][f] = sp[r][((c * kUnits + f) >> gshift) * 16];
        }
    }
};

// Few tokens (T <= 4): the lanes of an A operand that stand for tokens past the last would
// each fetch x again, and the address units, not HBM, would set the pace. So x is staged
// in LDS, `slab` columns at a time (all of them up to 64 KB), where lanes share a read.
// The 8 waves split the columns (wave w takes chunks w, w + 8, ...); their sums meet in
// LDS and are added in a fixed order.
template <int MATH, int W, int FS, int R>
__global__ __launch_bounds__(kMvThreads) void k_matvec_few(MvArgs a, int64_t slab, int pitch) {
    using M = Mt<MATH>;
    constexpr int kB = M::kBytes, PF = 16 / (W * R);  // 4 KB of weights in flight per wave
    using St = Stream<W, FS, R, PF>;
    extern __shared__ __align__(16) char xs[];
    __shared__ float red[kWaves][R][kFew][16];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t tile0 = (int64_t)blockIdx.x * R;
    St st(a, tile0, lane);
    const int mine = a.nc > w ? (int)((a.nc - w + kWaves - 1) / kWaves) : 0;  // this wave's chunks
#pragma unroll
    for (int p = 0; p < PF; ++p)
        if (p < mine) st.fetch(p, w + p * kWaves);
    float sum[R][4] = {};
    const char* xl = xs + min((lane & 15), (int)a.T - 1) * pitch + (lane >> 4) * 8 * kB;
    int i = 0;
    for (int64_t k0 = 0; k0 < a.n; k0 += slab) {
        if (k0) __syncthreads();
        const int units = (int)(slab * kB / 16);
        const int64_t left = (a.n - k0) * kB;
        for (int t = 0; t < (int)a.T; ++t) {
            const char* row = a.x + ((int64_t)t * a.ldx + k0) * kB;
            for (int u = threadIdx.x; u < units; u += kMvThreads) {
                u32x4 v = {0, 0, 0, 0};
                if (u * 16 + 16 <= left) {
                    __builtin_memcpy(&v, row + u * 16, 16);
                } else {  // zeros from column n on
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        if (u * 16 + e < left) v[e / 4] |= (uint32_t)(uint8_t)row[u * 16 + e] << (8 * (e & 3));
                }
                *reinterpret_cast<u32x4*>(xs + t * pitch + u * 16) = v;
            }
        }
        __syncthreads();
        const int end = (int)min<int64_t>(mine, ((k0 + slab) / kChunk - w + kWaves - 1) / kWaves);
        const char* xk = xl - k0 * kB;
        for (; i < end; i += PF) {  // slabs are whole multiples of PF chunks per wave, or the last
#pragma unroll
            for (int p = 0; p < PF; ++p) {
                if (i + p >= end) break;
                const int64_t c = w + (int64_t)(i + p) * kWaves;
#pragma unroll
                for (int f = 0; f < St::kUnits; ++f) {
                    typename M::Acc acc[R] = {};
#pragma unroll
                    for (int j = 0; j < FS; ++j) {
                        typename M::Op x[M::kPieces];
                        operand<MATH, W>(xk + (c * kChunk + (f * FS + j) * kStep) * kB, x);
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const typename M::Op b = weights<MATH, W>(st.d[p][r], f * FS + j);
#pragma unroll
                            for (int q = 0; q < M::kPieces; ++q) acc[r] = M::mma(x[q], b, acc[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int v = 0; v < 4; ++v) sum[r][v] = fmaf(st.s[p][r][f], (float)acc[r][v], sum[r][v]);
                }
                if (i + p + PF < mine) st.fetch(p, c + PF * kWaves);
            }
        }
    }
    if (lane < 16)
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < kFew; ++v) red[w][r][v][lane] = sum[r][v];
    __syncthreads();
    if (threadIdx.x < R * kFew * 16) {
        const int r = threadIdx.x / (kFew * 16), t = (threadIdx.x >> 4) % kFew;
        const int64_t row = (tile0 + r) * 16 + (threadIdx.x & 15);
        if (t < a.T && row < a.m) {
            float y = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) y += red[k][r][t][threadIdx.x & 15];
            y *= unit<MATH, W>();
            if (a.xs) y *= a.xs[t];
            store_elem(a.y, a.ytype, t * a.ldy + row, y);
        }
    }
}

// More tokens: workgroup (R row tiles, block of 16 NT tokens), columns split over the
// waves as above, x straight from memory in operand form; an operand of x serves R tiles.
template <int MATH, int W, int FS, int NT, int R>
__global__ __launch_bounds__(kMvThreads) void k_matvec(MvArgs a) {
    using M = Mt<MATH>;
    constexpr int PF = 2;
    using St = Stream<W, FS, R, PF>;
    constexpr int kB = M::kBytes;
    __shared__ float red[kWaves][16][17];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t groups = (a.tiles + R - 1) / R;
    const int64_t tile0 = blockIdx.x % groups * R, t0 = (int64_t)(blockIdx.x / groups) * 16 * NT;
    const char* row[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
        row[t] = a.x + (min(t0 + 16 * t + (lane & 15), a.T - 1) * a.ldx + 8 * (lane >> 4)) * kB;
    St st(a, tile0, lane);
    const int mine = a.nc > w ? (int)((a.nc - w + kWaves - 1) / kWaves) : 0;
    const int64_t whole = a.n / kChunk;  // chunks without padding
#pragma unroll
    for (int p = 0; p < PF; ++p)
        if (p < mine) st.fetch(p, w + p * kWaves);
    float sum[R][NT][4] = {};
    for (int i = 0; i < mine; i += PF) {
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            const int64_t c = w + (int64_t)(i + p) * kWaves;
            if (c >= whole) break;
#pragma unroll
            for (int f = 0; f < St::kUnits; ++f) {
                typename M::Acc acc[R][NT] = {};
#pragma unroll
                for (int j = 0; j < FS; ++j) {
                    const int step = f * FS + j;
                    typename M::Op b[R];
#pragma unroll
                    for (int r = 0; r < R; ++r) b[r] = weights<MATH, W>(st.d[p][r], step);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        struct alignas(16) { char d[8 * kB]; } raw;
                        __builtin_memcpy(&raw, row[t] + (c * kChunk + step * kStep) * kB, 8 * kB);
                        typename M::Op x[M::kPieces];
                        operand<MATH, W>(raw.d, x);
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int q = 0; q < M::kPieces; ++q) acc[r][t] = M::mma(x[q], b[r], acc[r][t]);
                    }
                }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int t = 0; t < NT; ++t)
#pragma unroll
                        for (int v = 0; v < 4; ++v)
                            sum[r][t][v] = fmaf(st.s[p][r][f], (float)acc[r][t][v], sum[r][t][v]);
            }
            if (i + p + PF < mine) st.fetch(p, c + PF * kWaves);
        }
    }
    if (whole < a.nc && whole % kWaves == w) {  // the chunk that the row ends in
        st.fetch(0, whole);
#pragma unroll 1
        for (int step = 0; step < kSteps; ++step) {
            const int k = (int)(a.n - whole * kChunk) - step * kStep - 8 * (lane >> 4);  // columns left
            float s[R];
            typename M::Op b[R];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                s[r] = st.s[0][r][0];
#pragma unroll
                for (int f = 1; f < St::kUnits; ++f) s[r] = f == step ? st.s[0][r][f] : s[r];
                auto d = st.d[0][r];
                constexpr int kPer = 4 / W;  // steps of a dword, less one
#pragma unroll
                for (int q = 1; q < W; ++q)
                    if (step >> (kPer - 1) == q) d[0] = d[q];
                b[r] = W == 2 && (step & 1) ? weights<MATH, W>(d, 1) : weights<MATH, W>(d, 0);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                struct alignas(16) { char d[8 * kB]; } raw;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const char* src = row[t] + (whole * kChunk + step * kStep + e) * kB;
                    if constexpr (kB == 4) reinterpret_cast<uint32_t*>(raw.d)[e] = e < k ? *(const uint32_t*)src : 0;
                    else if constexpr (kB == 2) reinterpret_cast<uint16_t*>(raw.d)[e] = e < k ? *(const uint16_t*)src : 0;
                    else raw.d[e] = e < k ? *src : 0;
                }
                typename M::Op x[M::kPieces];
                operand<MATH, W>(raw.d, x);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    typename M::Acc acc = {0, 0, 0, 0};
#pragma unroll
                    for (int q = 0; q < M::kPieces; ++q) acc = M::mma(x[q], b[r], acc);
#pragma unroll
                    for (int v = 0; v < 4; ++v) sum[r][t][v] = fmaf(s[r], (float)acc[v], sum[r][t][v]);
                }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (r + t) __syncthreads();
#pragma unroll
            for (int v = 0; v < 4; ++v) red[w][4 * (lane >> 4) + v][lane & 15] = sum[r][t][v];
            __syncthreads();
            if (threadIdx.x < 256) {
                const int64_t tt = t0 + 16 * t + (threadIdx.x >> 4), o = (tile0 + r) * 16 + (threadIdx.x & 15);
                if (tt < a.T && o < a.m) {
                    float y = 0.0f;
#pragma unroll
                    for (int k = 0; k < kWaves; ++k) y += red[k][threadIdx.x >> 4][threadIdx.x & 15];
                    y *= unit<MATH, W>();
                    if (a.xs) y *= a.xs[tt];
                    store_elem(a.y, a.ytype, tt * a.ldy + o, y);
                }
            }
        }
}

template <int MATH, int W, int FS, int NT, int R>
void launch_many(const MvArgs& a, hipStream_t stream) {
    const dim3 grid((unsigned)((a.tiles + R - 1) / R) * (unsigned)((a.T + 16 * NT - 1) / (16 * NT)));
    hipLaunchKernelGGL((k_matvec<MATH, W, FS, NT, R>), grid, dim3(kMvThreads), 0, stream, a);
}

template <int MATH, int W, int FS, int R>
void launch_few(const MvArgs& a, hipStream_t stream) {
    constexpr int kB = Mt<MATH>::kBytes, kAll = kChunk * kWaves * (16 / (W * R));
    // whole rounds of every wave's chunks in flight, unless the row ends first
    int64_t slab = kFewLds / (a.T * kB) / kAll * kAll;
    if (slab == 0) slab = kAll;
    slab = std::min<int64_t>(slab, a.nc * kChunk);
    const int pitch = (int)(slab * kB) + 16;
    const dim3 grid((unsigned)((a.tiles + R - 1) / R));
    hipLaunchKernelGGL((k_matvec_few<MATH, W, FS, R>), grid, dim3(kMvThreads), (size_t)(a.T * pitch), stream, a, slab,
                       pitch);
}

template <int MATH, int W, int FS>
void launch_mv(const MvArgs& a, hipStream_t stream) {
    if (a.T <= kFew) {
        if (a.tiles >= 1024) launch_few<MATH, W, FS, 2>(a, stream);
        else launch_few<MATH, W, FS, 1>(a, stream);
    } else if (a.T <= 16) {
        if (a.tiles >= 512) launch_many<MATH, W, FS, 1, 2>(a, stream);
        else launch_many<MATH, W, FS, 1, 1>(a, stream);
    } else if (a.T <= 32 || MATH == kF32 || FS == 1) {
        launch_many<MATH, W, FS, 2, 2>(a, stream);
    } else {
        if constexpr (MATH != kF32 && FS != 1) launch_many<MATH, W, FS, 4, 2>(a, stream);
    }
}

template <int MATH>
void launch_products(const MvArgs& a, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_mv<MATH, 4, 1>(a, stream);
        else launch_mv<MATH, 4, 4>(a, stream);
    } else {
        if (fs == 1) launch_mv<MATH, 2, 1>(a, stream);
        else launch_mv<MATH, 2, 4>(a, stream);
    }
}

}  // namespace bk
