// bk_matvec.hpp -- products of token rows with packed low-bit weights (included once for
// each type of x, so that the kernels compile side by side).
//
// The solve leaves a layer as codes c_ij in {0..Lq}, Lq = 2^bits - 1, and scales; the
// weight it stands for is w_ij = s_i,g(j) v_ij with v_ij = c_ij - Lq/2. For T tokens
//   y_ti = a_t sum_g s_ig sum_{j in group g} x_tj v_ij.
// v is a half-integer of at most 4 bits, so it is exact in bf16, fp16 and (times a power
// of two) int8: the inner sums run on the matrix cores with exact products and fp32
// (int8: exact int32) accumulation, and only the group's scale is applied to the sum, in
// fp32. Nothing is rounded below 32 bits before the output. e4m3 tokens are converted to
// fp16, which holds them all, on their way into LDS: the matrix cores' e4m3 operations do
// not keep 32 bits (448 and 127 times 2^-9 lose most of the small ones; activations with a
// few large channels came out 2e-5 to 2e-4 off in the 2-norm, in fp16 1e-7).
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
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowTile = 16;
constexpr int kStep = 32;         // columns of one MFMA
constexpr int kChunk = 128;       // columns of a chunk
constexpr int kSteps = kChunk / kStep;
constexpr int kWaves = 8;         // waves of a product workgroup that split the columns
constexpr int kMvThreads = 64 * kWaves;

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

// kBytes: of an element of x in memory; kLds: of one (fp32: of a piece of one) in LDS.
template <int MATH> struct Mt;
template <> struct Mt<kBF16> {
    using Op = bf16x8;
    using Acc = f32x4;
    static constexpr int kBytes = 2, kLds = 2, kPieces = 1;
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
    static constexpr int kBytes = 2, kLds = 2, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
};
template <> struct Mt<kF8> : Mt<kF16> {
    static constexpr int kBytes = 1;
};
template <> struct Mt<kI8> {
    using Op = u32x2;
    using Acc = i32x4;
    static constexpr int kBytes = 1, kLds = 1, kPieces = 1;
    static __device__ __forceinline__ Acc mma(Op a, Op b, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x32_i8(__builtin_bit_cast(long, a), __builtin_bit_cast(long, b), c, 0, 0,
                                                     0);
    }
};

// What the weight operand holds, as a multiple of v: int8 holds 16 v (W = 4) or 64 v (W = 2); bf16 and
// fp16 hold v. `unit` undoes it on the finished sum; powers of two, exact.
template <int MATH, int W>
constexpr float unit() {
    return MATH == kI8 ? (W == 4 ? 1.0f / 16 : 1.0f / 64) : 1.0f;
}

// 4 weights of W = 4 as e4m3 bytes, on their way to bf16 or fp16: sign to bit 7, k to bits 3..1, bit 0 set.
// That is 2 |v| in the low bits of the subnormal range and the first binade, where e4m3 is linear (value =
// bits * 2^-9, so v 2^-8), and the conversions' scale undoes the 2^-8.
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
        if constexpr (MATH == kI8) {
            // to two's complement: k -> 7 - k under a sign, then 16 (-8 s + k) + 8 = 16 v
            const uint32_t n = w & 0x88888888u;
            w ^= n - (n >> 3);
            return Op{((w << 4) & 0xF0F0F0F0u) | 0x08080808u, (w & 0xF0F0F0F0u) | 0x08080808u};
        } else {
            return from_e4m3(e4m3_lo(w), e4m3_hi(w), Op{});
        }
    } else {
        uint32_t w = d[st >> 1];
        if constexpr (MATH == kI8) {
            // even nibbles give columns 0 2 4 6, odd ones 1 3 5 7 (even_odd does the same to x)
            w ^= (w >> 2) & 0x33333333u;
            if (st & 1) w <<= 1;  // step b into the places of step a: sign at bit 3, k at bit 1
            return Op{((w << 4) & 0x80808080u) | ((w << 5) & 0x40404040u) | 0x20202020u,
                      (w & 0x80808080u) | ((w << 1) & 0x40404040u) | 0x20202020u};
        } else {
            if (st & 1) w <<= 1;
            return from_e2m1((w & 0xAAAAAAAAu) | 0x11111111u, Op{});
        }
    }
}

// 8 bytes of x in the order of the int8 operands of W = 2.
__device__ __forceinline__ u32x2 even_odd(u32x2 x) {
    return u32x2{__builtin_amdgcn_perm(x[1], x[0], 0x06040200u), __builtin_amdgcn_perm(x[1], x[0], 0x07050301u)};
}

// 8 e4m3 values as fp16 (NaN stays NaN).
__device__ __forceinline__ u32x4 f16_of_e4m3(uint32_t lo, uint32_t hi) {
    const f16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false),
                        __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true)};
    return __builtin_bit_cast(u32x4, p);
}

// Four fp32 values as three bf16 pieces each, largest first, cut by truncation: 8 significant
// bits each, their sum is x exactly, but for bits below 2^-133, the smallest bf16, which no
// value of 2^-110 or more has. An infinity or NaN, whose remainder is NaN, stays in the
// first piece; a NaN is quieted first, so that it does not lose its whole payload to the cut.
// (Pieces rounded to nearest take fewer instructions but a branch for what rounds up to
// infinity: 16 tokens by 8192 x 8192 22.9 us with it, 20.1 so.)
__device__ __forceinline__ void split4(u32x4 x, u32x2 (&p)[3]) {
    u32x4 h, m, l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float v = __uint_as_float(x[e]);
        h[e] = __float_as_uint(__builtin_canonicalizef(v));
        float r = v - __uint_as_float(x[e] & 0xFFFF0000u);
        r = r == r ? r : 0.0f;
        m[e] = __float_as_uint(r);
        l[e] = __float_as_uint(r - __uint_as_float(m[e] & 0xFFFF0000u));
    }
    const auto pack = [](u32x4 a) {
        return u32x2{__builtin_amdgcn_perm(a[1], a[0], 0x07060302u), __builtin_amdgcn_perm(a[3], a[2], 0x07060302u)};
    };
    p[0] = pack(h);
    p[1] = pack(m);
    p[2] = pack(l);
}

// The A operand from 8 elements of a staged row of x at `src`, pieces `piece` bytes apart.
template <int MATH, int W>
__device__ __forceinline__ void operand(const char* src, int piece, typename Mt<MATH>::Op (&p)[Mt<MATH>::kPieces]) {
    using Op = typename Mt<MATH>::Op;
#pragma unroll
    for (int i = 0; i < Mt<MATH>::kPieces; ++i)  // the smallest piece first into the sum
        p[i] = *reinterpret_cast<const Op*>(src + (Mt<MATH>::kPieces - 1 - i) * piece);
    if constexpr (W == 2 && MATH == kI8) p[0] = even_odd(p[0]);
}

// The 16 bytes of a row of x from byte `at` on that the row's end, byte `end`, cuts: zeros
// from there on. (All other units are whole, or past the end.)
template <int kB>
__device__ __forceinline__ u32x4 cut_unit(const char* __restrict__ row, int at, int end) {
    u32x4 v = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < 16; e += kB)
        if (at + e < end) {
            uint32_t w = 0;
            __builtin_memcpy(&w, row + at + e, kB);
            v[e / 4] |= w << (8 * (e & 3));
        }
    return v;
}

// ---------------------------------------------------------------- the products
// In all of them A = x (rows are tokens) and B = the weights, so a lane's four sums are
// four tokens of one weight row and share its scale. The sums are scaled every FS steps: a
// chunk (FS = 4), or a step where groups are shorter than a chunk (FS = 1).

// A wave's chunks of R row tiles with their scales, PF chunks ahead of their use. A chunk
// past the last fetches the last again: the loads of the loops below are all unconditional
// (clamped, not branched around), because behind a branch the compiler no longer knows how
// many are in flight and waits for all of them before it uses the first.
template <int W, int FS, int R, int PF>
struct Stream {
    using Sh = typename Share<W>::T;
    static constexpr int kUnits = kSteps / FS;
    const Sh* wp[R];
    const float* sp[R];
    int64_t nc;
    int gshift, lane;
    Sh d[PF][R];
    float s[PF][R][kUnits];
    // tile0 and c are uniform over the wave (and known to be): addresses but for the lane's part are scalar
    __device__ __forceinline__ Stream(const MvArgs& a, int64_t tile0, int lane_) : nc(a.nc), gshift(a.gshift), lane(lane_) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tile = min(tile0 + r, (int64_t)a.tiles - 1);
            wp[r] = reinterpret_cast<const Sh*>(a.codes) + tile * a.nc * 64;
            sp[r] = a.scales + tile * a.ngp * 16;
        }
    }
    __device__ __forceinline__ void fetch(int slot, int64_t c) {
        c = min(c, nc - 1);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            d[slot][r] = (wp[r] + c * 64)[lane];
#pragma unroll
            for (int f = 0; f < kUnits; ++f) s[slot][r][f] = (sp[r] + ((c * kUnits + f) >> gshift) * 16)[lane & 15];
        }
    }
};

// Few tokens (T <= TB): the lanes of an A operand that stand for tokens past the last would
// fetch x again, and rows a power of two apart fall on one memory channel, if operands came
// straight from memory: the address units, not HBM, would set the pace. So each wave stages
// x for its next PF chunks by rows in an LDS area of its own, where the surplus lanes share
// a read: loads of a set are in flight while the set before is multiplied, and no wave
// waits for another. The 8 waves split the columns (wave w takes chunks w, w + 8, ...);
// their sums meet in LDS at the end and are added in a fixed order. Bound by HBM for large
// layers (28672 x 8192, one bf16 token: 4 bits 25 to 28 us, 4.4 to 4.9 TB/s; 2 bits 14.5 us, where the
// LDS reads of x weigh as much), by latency for small ones (4096 x 4096 4.3 us, an empty
// kernel 2.4), by the pieces' instructions for fp32 (16 tokens by 8192 x 8192 20 us; 16 bf16
// tokens by 14336 x 4096 10).
template <int MATH, int PF, int TB>
struct FewShape {
    static constexpr int kB = Mt<MATH>::kBytes;
    static constexpr int kRowUnits = PF * kChunk * kB / 16;           // 16-byte units of a token row in a set
    static constexpr int kUnits = (TB * kRowUnits + 63) / 64;         // units of a lane
    static constexpr int kPieces = Mt<MATH>::kPieces;
    static constexpr int kL = Mt<MATH>::kLds;
    static constexpr int kPiece = PF * kChunk * kL;                   // from piece to piece of a token
    static constexpr int kPitch = kPieces * kPiece + 16;              // from token to token: 4 banks
    static constexpr int kBytes = TB * kPitch;                        // of a wave
};

template <int MATH, int W, int FS, int R, int PF, int TB, int NW>
__global__ __launch_bounds__(64 * NW) void k_matvec_few(MvArgs a) {
    using M = Mt<MATH>;
    using St = Stream<W, FS, R, PF>;
    using Sh = FewShape<MATH, PF, TB>;
    constexpr int kB = M::kBytes;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char* xs = lds + w * Sh::kBytes;
    const int64_t tile0 = (int64_t)blockIdx.x * R;
    const int T = (int)a.T, end = (int)a.n * kB;  // bytes of a row
    const int mine = a.nc > w ? (int)((a.nc - w + NW - 1) / NW) : 0;  // this wave's chunks
    u32x4 x[Sh::kUnits];
    // unit i of this lane in the set from chunk i0 on: token, place in the token's LDS row, byte in the row of x
    const auto token_of = [&](int i) { return (lane + i * 64) / Sh::kRowUnits; };
    const auto place_of = [&](int i) { return (lane + i * 64) % Sh::kRowUnits; };
    const auto byte_of = [&](int i, int i0) {
        constexpr int kPer = kChunk * kB / 16;
        const int u = place_of(i);
        return ((i0 + u / kPer) * NW + w) * kChunk * kB + u % kPer * 16;
    };
    // a row below 16 bytes has no whole unit: the loads, whose values are then not used, go elsewhere
    const char* xb = end >= 16 ? a.x : a.codes;
    const int64_t ldb = end >= 16 ? a.ldx * kB : 0;
    const int most = max(end - 16, 0);
    const auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < Sh::kUnits; ++i)
            __builtin_memcpy(&x[i], xb + min(token_of(i), T - 1) * ldb + min(byte_of(i, i0), most), 16);
    };
    St st(a, tile0, lane);
    load(0);
#pragma unroll
    for (int p = 0; p < PF; ++p) st.fetch(p, w + p * NW);
    float sum[R][4] = {};
    const char* xl = xs + min((lane & 15), T - 1) * Sh::kPitch + (lane >> 4) * 8 * Sh::kL;
    // 0, but known to the compiler only as made from every operand read so far: a set's writes, whose addresses it is
    // part of, cannot move in front of other lanes' reads of the set before. (A fence there would keep global loads
    // in place too: 4096 x 14336 int8 8.8 -> 9.9 us. This costs nothing.)
    int after = 0;
    const auto put = [&](int token, int place, u32x4 v) __attribute__((always_inline)) {  // unit `place` of a token
        char* dst = xs + token * Sh::kPitch + after;
        if constexpr (kB == 4) {
            u32x2 p[3];
            split4(v, p);
#pragma unroll
            for (int i = 0; i < 3; ++i) *reinterpret_cast<u32x2*>(dst + i * Sh::kPiece + place * 8) = p[i];
        } else if constexpr (MATH == kF8) {
            *reinterpret_cast<u32x4*>(dst + place * 32) = f16_of_e4m3(v[0], v[1]);
            *reinterpret_cast<u32x4*>(dst + place * 32 + 16) = f16_of_e4m3(v[2], v[3]);
        } else {
            *reinterpret_cast<u32x4*>(dst + place * 16) = v;
        }
    };
    for (int i0 = 0; i0 < mine; i0 += PF) {
        if (((i0 + PF - 1) * NW + w + 1) * kChunk * kB > end)  // the set passes the row's end: zeros from there on
#pragma unroll
            for (int i = 0; i < Sh::kUnits; ++i)
                if (byte_of(i, i0) + 16 > end) x[i] = u32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < Sh::kUnits; ++i)
            if (token_of(i) < TB) put(token_of(i), place_of(i), x[i]);
        if (end % 16 != 0) {  // the unit that the row ends in, if it is in this set
            const int at = end & ~15, c = at / (kChunk * kB), p = c / NW - i0;
            wave_fence();  // behind the zeros that another lane wrote there
            if (c % NW == w && p >= 0 && p < PF && lane < T)
                put(lane, ((p - c) * kChunk * kB + at) / 16, cut_unit<kB>(a.x + lane * a.ldx * kB, at, end));
        }
        // this wave alone reads what it staged
        wave_fence();
        load(i0 + PF);
#pragma unroll
        for (int p = 0; p < PF; ++p) {
            const char* xk = xl + p * kChunk * Sh::kL;
            if (i0 + p < mine)
#pragma unroll
                for (int f = 0; f < St::kUnits; ++f) {
                    typename M::Acc acc[R] = {};
#pragma unroll
                    for (int j = 0; j < FS; ++j) {
                        typename M::Op v[M::kPieces];
                        operand<MATH, W>(xk + (f * FS + j) * kStep * Sh::kL, Sh::kPiece, v);
#pragma unroll
                        for (int q = 0; q < M::kPieces; ++q) asm("" : "+v"(after) : "v"(v[q]));
#pragma unroll
                        for (int r = 0; r < R; ++r) {
                            const typename M::Op b = weights<MATH, W>(st.d[p][r], f * FS + j);
#pragma unroll
                            for (int q = 0; q < M::kPieces; ++q) acc[r] = M::mma(v[q], b, acc[r]);
                        }
                    }
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int v = 0; v < 4; ++v) sum[r][v] = fmaf(st.s[p][r][f], (float)acc[r][v], sum[r][v]);
                }
            st.fetch(p, w + (int64_t)(i0 + p + PF) * NW);
        }
        if constexpr (PF == 1) asm volatile("" ::: "memory");  // or all loads move over the loop's edge, to their use
    }
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);  // [wave][tile][token][16 rows + 1]
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[((w * R + r) * 16 + 4 * (lane >> 4) + v) * 17 + (lane & 15)] = sum[r][v];
    __syncthreads();
    for (int i = threadIdx.x; i < T * R * 16; i += (64 * NW)) {
        const int t = i / (R * 16), r = i / 16 % R;
        const int64_t row = (tile0 + r) * 16 + (i & 15);
        if (row < a.m) {
            float y = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) y += red[((k * R + r) * 16 + t) * 17 + (i & 15)];
            y *= unit<MATH, W>();
            if (a.xs) y *= a.xs[t];
            store_elem(a.y, a.ytype, t * a.ldy + row, y);
        }
    }
}

// More tokens: x tiles shared in LDS.
//
// A workgroup has KS x RW waves: wave (kg, rg) multiplies the R row tiles of row group rg
// with the 16 NT tokens of the block over the chunks kg, kg + KS, ...; per iteration the
// workgroup stages KS CH chunks of x, double buffered, one barrier an iteration. With many
// workgroups at hand KS = 1 and all waves share the chunk; with few, the waves split the
// columns and their sums meet in LDS at the end, in the order of kg.
//
// x lies in LDS in operand form, 1 KB for 64 lanes of 16 bytes, so an operand is one
// conflict-free read. A thread stages 16 bytes of a row (u-th of the row's chunk); the
// lane slot is (q, t ^ u) for token t, which spreads a row's units over the banks. fp32 is
// cut into its three pieces on the way in, e4m3 becomes fp16. Of int8, 16 bytes of a lane
// are its columns of two steps.
//
// Bound by vector instructions beside the MFMAs: dequantisation (11 for 8 bf16 weights, 7 for
// int8), spread over the NT tiles that use a weight, and scaling (for int8 two a sum and chunk).
// 14336 x 4096, groups of 128, 2048 tokens: int8 182 us (1.32 PFLOP/s), e4m3 240, bf16 261;
// 48 bf16 tokens 17 us.
//
// MmOp: the MFMA of kSub steps, its operands from a share of weights and from LDS. Whole
// chunks (FS = 4) take int8 two steps at a time, at twice the rate.
template <int MATH, int FS>
struct MmOp {
    using M = Mt<MATH>;
    static constexpr int kSub = FS == 4 && MATH == kI8 ? 2 : 1;
    using Op = std::conditional_t<kSub == 2, u32x4, typename M::Op>;
    template <int W>
    static __device__ __forceinline__ Op weight(typename Share<W>::T d, int step) {
        if constexpr (kSub == 1) {
            return weights<MATH, W>(d, step);
        } else {
            Op b;
#pragma unroll
            for (int h = 0; h < kSub; ++h) {
                const u32x2 w = weights<MATH, W>(d, step + h);
                b[2 * h] = w[0];
                b[2 * h + 1] = w[1];
            }
            return b;
        }
    }
    static __device__ __forceinline__ void read(Op (&x)[M::kPieces], const char* buf, int step, int q, int t) {
        if constexpr (MATH == kI8) {
            const int pair = step >> 1;
            const char* p = buf + pair * 1024 + ((t ^ (4 * pair + q)) & 15) * 16;
            x[0] = *reinterpret_cast<const Op*>(kSub == 1 ? p + (step & 1) * 8 : p);
        } else {
#pragma unroll
            for (int p = 0; p < M::kPieces; ++p)
                x[p] = *reinterpret_cast<const Op*>(buf + (p * 4 + step) * 1024 + ((t ^ (4 * step + q)) & 15) * 16);
        }
    }
    static __device__ __forceinline__ typename M::Acc mma(Op a, Op b, typename M::Acc c) {
        if constexpr (kSub == 1) {
            return M::mma(a, b, c);
        } else {
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c,
                                                         0, 0, 0);
        }
    }
};

template <int MATH, int NT, int KC>
struct MmTile {
    // bytes of x in LDS a buffer: [chunk][token tile][piece or not][4 steps or 2 pairs][64 lanes][16 bytes]
    static constexpr int kSlabs = 2 * Mt<MATH>::kLds * Mt<MATH>::kPieces;  // of 1 KB a chunk and tile
    static constexpr int kBytes = KC * NT * kSlabs * 1024;
};

// Token tiles of an output pass: as many as `room` bytes of LDS hold at `each`.
constexpr int mm_pass(int tiles, int each, int room) {
    int n = tiles;
    while (n > 1 && n * each > room) n = (n + 1) / 2;
    return n;
}

template <int MATH, int W, int FS, int NT, int R, int KS, int RW, int CH>
__global__ __launch_bounds__(64 * KS * RW) __attribute__((amdgpu_waves_per_eu(2)))
void k_matmul(MvArgs a, int token_blocks) {
    using M = Mt<MATH>;
    using St = Stream<W, FS, R, 2>;
    constexpr int KC = KS * CH;  // chunks of an iteration
    using Tile = MmTile<MATH, NT, KC>;
    constexpr int kB = M::kBytes, kThreads = 64 * KS * RW, kRows = 16 * R * RW, kPitch = kRows + 4;
    constexpr int kUnitCols = 16 / (kB == 4 ? 2 : kB);        // columns of a staged unit: 16 bytes of x, fp32 32
    constexpr int kRowUnits = KC * kChunk / kUnitCols;        // units of a token row in an iteration
    constexpr int kUnits = 16 * NT * kRowUnits / kThreads;    // units a thread stages
    static_assert(16 * NT * kRowUnits % kThreads == 0, "units divide over the threads");
    extern __shared__ __align__(16) char lds[];
    float* red = reinterpret_cast<float*>(lds);               // [KS][16][kPitch], after the loop

    // workgroups 8 apart share an XCD: give each XCD a run of row blocks, token blocks innermost, so that those
    // that read the same weights run side by side
    const uint32_t total = gridDim.x, per = total / 8, extra = total % 8;
    const uint32_t xcd = blockIdx.x % 8, id = xcd * per + min(xcd, extra) + blockIdx.x / 8;
    const int64_t tile_b = (int64_t)(id / token_blocks) * R * RW, t0 = (int64_t)(id % token_blocks) * 16 * NT;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave / RW, rg = wave % RW;
    const int q = lane >> 4, t = lane & 15;

    constexpr int kParts = kB == 4 ? 2 : 1;  // 16-byte parts of a unit
    constexpr int kAhead = KS > 1 && kUnits * kParts <= 6 ? 2 : 1;  // iterations that x is fetched ahead: few
                                                                   // workgroups hide less, and registers allow
    u32x4 raw[kAhead][kUnits][kParts];
    // this thread stages unit `un` of the token rows row0 + i kRowStep
    constexpr int kRowStep = kThreads / kRowUnits;
    static_assert(kThreads % kRowUnits == 0, "a thread keeps its unit");
    const int row0 = threadIdx.x / kRowUnits, un = threadIdx.x % kRowUnits;
    const int end = (int)a.n * kB;  // bytes of a row
    const int64_t ldb = a.ldx * kB;
    const char* x0 = a.x + t0 * ldb;
    const int last_row = (int)min<int64_t>(16 * NT, a.T - t0) - 1;
    // rows past the last token repeat it, units past the row's end its last one; a row shorter than a unit has no
    // whole one: the loads, whose values are then not used, go elsewhere
    const bool some = end >= 16 * kParts;
    const char* rows[kUnits];
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
        rows[i] = some ? x0 + min(row0 + i * kRowStep, last_row) * ldb : a.codes;
    const auto load = [&](int it, u32x4 (&to)[kUnits][kParts]) __attribute__((always_inline)) {
        const int at = min((it * KC * kChunk + un * kUnitCols) * kB, some ? end - 16 * kParts : 0);
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
#pragma unroll
            for (int h = 0; h < kParts; ++h) __builtin_memcpy(&to[i][h], rows[i] + at + 16 * h, 16);
    };
    // unit `ru` of a token row's iteration, into its operands' slots
    const auto put = [&](char* buf, int row, int ru, const u32x4 (&v)[kParts]) __attribute__((always_inline)) {
        const int u = ru % (kChunk / kUnitCols), ck = ru / (kChunk / kUnitCols);
        char* dst = buf + (ck * NT + (row >> 4)) * Tile::kSlabs * 1024;
        if constexpr (MATH == kI8) {  // columns 16 u ..: step u / 2, lanes of q = 2 (u % 2) and the next
            const u32x2 lo = {v[0][0], v[0][1]}, hi = {v[0][2], v[0][3]};
            const int step = u >> 1, pair = step >> 1;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int qq = 2 * (u & 1) + h;
                const u32x2 w = h ? hi : lo;
                *reinterpret_cast<u32x2*>(dst + pair * 1024 + (qq * 16 + ((row ^ (4 * pair + qq)) & 15)) * 16 +
                                          (step & 1) * 8) = W == 2 ? even_odd(w) : w;
            }
        } else if constexpr (MATH == kF8) {  // columns 16 u ..: 8 of them as below, and the next 8
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int o = 2 * u + h;
                *reinterpret_cast<u32x4*>(dst + (o >> 2) * 1024 + ((o & 3) * 16 + ((row ^ o) & 15)) * 16) =
                    f16_of_e4m3(v[0][2 * h], v[0][2 * h + 1]);
            }
        } else {  // columns 8 u ..: step u / 4, lanes of q = u % 4
            const int at = (u >> 2) * 1024 + ((u & 3) * 16 + ((row ^ u) & 15)) * 16;
            if constexpr (kB == 4) {
                u32x2 lo[3], hi[3];
                split4(v[0], lo);
                split4(v[kParts - 1], hi);
#pragma unroll
                for (int c = 0; c < 3; ++c)  // the smallest piece first into the sum
                    *reinterpret_cast<u32x4*>(dst + (2 - c) * 4096 + at) = u32x4{lo[c][0], lo[c][1], hi[c][0], hi[c][1]};
            } else {
                *reinterpret_cast<u32x4*>(dst + at) = v[0];
            }
        }
    };
    const auto store = [&](int it, char* buf, const u32x4 (&from)[kUnits][kParts]) __attribute__((always_inline)) {
        // the unit that a row's end cuts, if there is one in this iteration (else -1)
        const int first = it * KC * kChunk * kB, last = end / (16 * kParts) * 16 * kParts;
        const int cut = end != last && last >= first && last < first + KC * kChunk * kB ? (last - first) / (16 * kParts) : -1;
        if (first + (un + 1) * 16 * kParts <= end) {
#pragma unroll
            for (int i = 0; i < kUnits; ++i) put(buf, row0 + i * kRowStep, un, from[i]);
        } else if (un != cut) {  // past the end
            const u32x4 zero[kParts] = {};
#pragma unroll
            for (int i = 0; i < kUnits; ++i) put(buf, row0 + i * kRowStep, un, zero);
        }
        if (cut >= 0)
            for (int row = threadIdx.x; row < 16 * NT; row += kThreads) {
                const char* src = a.x + min(t0 + row, a.T - 1) * a.ldx * kB;
                u32x4 v[kParts];
#pragma unroll
                for (int h = 0; h < kParts; ++h) v[h] = cut_unit<kB>(src, last + 16 * h, end);
                put(buf, row, cut, v);
            }
    };

    St st(a, tile_b + rg * R, lane);
    const int iters = (int)((a.nc + KC - 1) / KC);
    load(0, raw[0]);
    st.fetch(0, kg);
    if (kAhead == 2) load(1, raw[kAhead - 1]);
    st.fetch(1, kg + KS);
    store(0, lds, raw[0]);
    __syncthreads();

    float sum[R][NT][4] = {};
    const auto body = [&](int it, int parity) __attribute__((always_inline)) {
        load(it + kAhead, raw[kAhead == 2 ? parity : 0]);
#pragma unroll
        for (int ch = 0; ch < CH; ++ch) {
            const int64_t c = (int64_t)it * KC + ch * KS + kg;
            const char* buf = lds + (it & 1) * Tile::kBytes + (ch * KS + kg) * NT * Tile::kSlabs * 1024 + q * 256;
            const int slot = CH == 2 ? ch : parity;
            using Mm = MmOp<MATH, FS>;
            constexpr int kMfma = FS / Mm::kSub;  // MFMAs of a sum
            typename Mm::Op b[St::kUnits][kMfma][R];
            float s[St::kUnits][R];
#pragma unroll
            for (int f = 0; f < St::kUnits; ++f)
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    s[f][r] = st.s[slot][r][f];
#pragma unroll
                    for (int j = 0; j < kMfma; ++j)
                        b[f][j][r] = Mm::template weight<W>(st.d[slot][r], f * FS + j * Mm::kSub);
                }
            st.fetch(slot, c + 2 * KS);
            if (c >= a.nc) continue;
            // token tiles one after the other, each behind the reads of the next one's x and in front of the scaling
            // of the last one's sums, so that neither waits for the matrix core
            constexpr int kSums = NT * St::kUnits;  // sum i: token tile i / kUnits, scale unit i % kUnits
            constexpr int kRead = M::kPieces == 1 ? 2 : 1;  // three pieces leave no registers for the next tile's
            typename Mm::Op x[kRead][kMfma][M::kPieces];
            typename M::Acc acc[2][R];
            const auto read = [&](int i) {
#pragma unroll
                for (int j = 0; j < kMfma; ++j)
                    Mm::read(x[i % kRead][j], buf + i / St::kUnits * Tile::kSlabs * 1024,
                             i % St::kUnits * FS + j * Mm::kSub, q, t);
            };
            const auto flush = [&](int i) {
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int v = 0; v < 4; ++v)
                        sum[r][i / St::kUnits][v] =
                            fmaf(s[i % St::kUnits][r], (float)acc[i & 1][r][v], sum[r][i / St::kUnits][v]);
            };
            if (kRead == 2) read(0);
#pragma unroll
            for (int i = 0; i < kSums; ++i) {
                if (kRead == 1) read(i);
                else if (i + 1 < kSums) read(i + 1);
#pragma unroll
                for (int r = 0; r < R; ++r) acc[i & 1][r] = typename M::Acc{0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < kMfma; ++j)
#pragma unroll
                    for (int p = 0; p < M::kPieces; ++p)
#pragma unroll
                        for (int r = 0; r < R; ++r)
                            acc[i & 1][r] = Mm::mma(x[i % kRead][j][p], b[i % St::kUnits][j][r], acc[i & 1][r]);
                if (i > 0) flush(i - 1);
                __builtin_amdgcn_sched_barrier(0);
            }
            flush(kSums - 1);
        }
        if (it + 1 < iters) store(it + 1, lds + (~it & 1) * Tile::kBytes, raw[kAhead == 2 ? parity ^ 1 : 0]);
        __syncthreads();
    };
    for (int it = 0; it < iters; it += 2) {
        body(it, 0);
        if (it + 1 < iters) body(it + 1, 1);
    }

    // the sums through LDS, NP token tiles at a time, so that a thread stores 4 rows of a token together
    constexpr int NP = mm_pass(NT, KS * 16 * kPitch * 4, 2 * Tile::kBytes);
#pragma unroll
    for (int n0 = 0; n0 < NT; n0 += NP) {
        if (n0) __syncthreads();
#pragma unroll
        for (int n = n0; n < n0 + NP && n < NT; ++n)
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    red[(kg * 16 * NP + (n - n0) * 16 + 4 * q + v) * kPitch + (rg * R + r) * 16 + t] = sum[r][n][v];
        __syncthreads();
        const int toks = 16 * (NP < NT - n0 ? NP : NT - n0);
        for (int i = threadIdx.x; i < toks * (kRows / 4); i += kThreads) {
            const int tok = i / (kRows / 4), row = i % (kRows / 4) * 4;
            const int64_t tt = t0 + 16 * n0 + tok, o = tile_b * 16 + row;
            if (tt < a.T && o < a.m) {
                f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k) y += *reinterpret_cast<const f32x4*>(red + (k * 16 * NP + tok) * kPitch + row);
                y *= unit<MATH, W>();
                if (a.xs) y *= a.xs[tt];
                store4(a.y, a.ytype, tt * a.ldy + o, y, (int)min<int64_t>(4, a.m - o));
            }
        }
    }
}

template <int MATH, int W, int FS, int NT, int R, int KS, int RW, int CH = 1>
void launch_mm(const MvArgs& a, hipStream_t stream) {
    const unsigned rows = (unsigned)((a.tiles + R * RW - 1) / (R * RW));
    const unsigned blocks = (unsigned)((a.T + 16 * NT - 1) / (16 * NT));
    constexpr size_t red = sizeof(float) * KS * 16 * (16 * R * RW + 4);
    constexpr size_t lds = std::max<size_t>(2 * (size_t)MmTile<MATH, NT, KS * CH>::kBytes, red);
    hipLaunchKernelGGL((k_matmul<MATH, W, FS, NT, R, KS, RW, CH>), dim3(rows * blocks), dim3(64 * KS * RW), lds, stream, a,
                       (int)blocks);
}

template <int MATH, int W, int FS, int R, int PF, int TB, int NW>
void launch_few(const MvArgs& a, hipStream_t stream) {
    constexpr size_t red = sizeof(float) * NW * R * 16 * 17;
    constexpr size_t lds = std::max<size_t>((size_t)NW * FewShape<MATH, PF, TB>::kBytes, red);
    const dim3 grid((unsigned)((a.tiles + R - 1) / R));
    hipLaunchKernelGGL((k_matvec_few<MATH, W, FS, R, PF, TB, NW>), grid, dim3(64 * NW), lds, stream, a);
}

// Chunks ahead of their use (PF): 2 KB of weights in flight per wave, 1 KB for fp32 from 5 tokens on, whose pieces fill
// LDS. 14336 x 4096, 16 bf16 tokens 10.6 us, with half 10.6, with twice as many 15.0; one token 8.5, 8.7 and 9.2.
// Tiles that share an operand of x (R): two, from 5 tokens on, where that still makes a workgroup for every compute
// unit: 16 tokens by 8176 x 4096 (256 workgroups of two tiles) bf16 7.4 us, one tile 8.2, fp32 11.7 and 17.5; by 4096 x
// 4096 (128) 6.7 and 5.5. Up to 4 tokens two tiles gain nothing but for fp32 (14336 x 4096: bf16 9.1 and 9.1, int8 8.1
// and 8.2, fp32 12.0 and 14.3).
template <int MATH, int W, int FS, int TB>
void launch_tokens(const MvArgs& a, hipStream_t stream) {
    constexpr int PF = TB <= 4 ? 8 / W : MATH == kF32 ? 1 : 2;
    constexpr int R = TB <= 4 ? 1 : 2;
    if (R > 1 && (int)a.tiles >= 2 * device_info().cus) launch_few<MATH, W, FS, R, PF, TB, 8>(a, stream);
    else launch_few<MATH, W, FS, 1, PF, TB, 8>(a, stream);
}

// Up to 16 tokens k_matvec_few, by the tokens that its LDS holds (fp32, 4096 x 4096, one token 5.0 us, with room for 4
// 6.1, 8 7.5, 16 9.6; bf16 4.45, 4.5, 4.7, 5.3): 16 bf16 tokens by 14336 x 4096 10.9 us, the smallest k_matmul 14.7.
// More than 16 tokens: k_matmul with the first of these tiles whose workgroups all run at once (two of the first on a
// compute unit, one of the others), so that a call is one round of them; us of each side by the number of workgroups:
//   rows x tokens  (16-bit types and int8)
//   16 x 32  64 bf16 tokens by 4096 x 4096 (512 workgroups) 12.7, 64 x 32 13.8; 80 tokens (768) 19.2 and 13.9
//   64 x 32  64 tokens by 8192 x 8192 (256) 24.1, 64 x 48 30.3; 80 tokens (384) 44.2 and 30.7
//   64 x 48  80 tokens by 8192 x 8192 (256) 30.7, 64 x 64 34.9; 100 tokens (384) 55.8 and 34.5
//   64 x 64  columns split over 4 waves: 128 tokens by 8192 x 8192 (256) 34.5, over 2 40.7; 200 tokens (512) 64.3, 54.9
// else, up to 32 tokens, 64 x 32 in rounds (32 tokens by 28672 x 4096 26.9, 64 x 64 29.1); 128 x 128 with a workgroup
// for every unit (512 tokens by 8192 x 8192 (256): bf16 98.7, 64 x 64 108, int8 73 and 79; 512 tokens by 4096 x 14336
// (128) 164 and 95), for which 64 tokens are too few; 64 x 64 over 2 waves for the rest.
// 128 x 128 takes two chunks an iteration for int8 (2048 tokens by 14336 x 4096 209, one 217), and half the tokens
// where 16-bit types scale every step, for the registers (with whole chunks half the tokens cost 303 -> 354).
// fp32: 64 x 32 while its workgroups make two rounds at most, else 256 x 32 (n = 8192, 128 tokens by 8192 rows (512
// workgroups) 125, 256 x 32 131; 200 tokens (896) 239 and 128; n = 4096, 64 tokens by 14336 rows (448) 66 and 68).
template <int MATH, int W, int FS>
void launch_mv(const MvArgs& a, hipStream_t stream) {
    if (a.T == 1) return launch_tokens<MATH, W, FS, 1>(a, stream);
    if (a.T <= 4) return launch_tokens<MATH, W, FS, 4>(a, stream);
    if (a.T <= 8) return launch_tokens<MATH, W, FS, 8>(a, stream);
    if (a.T <= 16) return launch_tokens<MATH, W, FS, 16>(a, stream);
    const int64_t cus = device_info().cus;
    const auto blocks = [&](int tiles, int tokens) {
        return (int64_t)((a.tiles + tiles - 1) / tiles) * ((a.T + tokens - 1) / tokens);
    };
    if constexpr (MATH == kF32) {
        if constexpr (FS == 4) {
            if (blocks(4, 32) > 2 * cus) return launch_mm<MATH, W, FS, 2, 4, 1, 4>(a, stream);
        }
        launch_mm<MATH, W, FS, 2, 2, 2, 2>(a, stream);
    } else {
        constexpr bool kByte = MATH == kI8;
        if (blocks(1, 32) <= 2 * cus) launch_mm<MATH, W, FS, 2, 1, 4, 1>(a, stream);
        else if (a.T <= 32 || blocks(4, 32) <= cus) launch_mm<MATH, W, FS, 2, 2, 4, 2>(a, stream);
        else if (blocks(4, 48) <= cus) launch_mm<MATH, W, FS, 3, 2, 4, 2>(a, stream);
        else if (blocks(4, 64) <= cus) launch_mm<MATH, W, FS, 4, 2, 4, 2>(a, stream);
        else if (a.T > 64 && blocks(8, 128) >= cus)
            launch_mm<MATH, W, FS, kByte || FS == 4 ? 8 : 4, 2, 1, 4, kByte ? 2 : 1>(a, stream);
        else launch_mm<MATH, W, FS, 4, 2, 2, 2>(a, stream);
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
