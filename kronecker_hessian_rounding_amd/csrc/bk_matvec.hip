// bk_matvec.hip -- products with packed low-bit weights: the solve's codes put to use.
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
// as it is, so the products know W only. A tile is 16 rows, a chunk 512 / W columns; the
// 1024 bytes of (tile, chunk) are contiguous, chunks of a tile follow each other, and
// lane l of a wave owns 16 of the bytes: row l % 16 and, of each of the chunk's 32-column
// steps, the 8 columns 8 (l / 16) + 0..7, which is its share of the B operand of a
// 16x16x32 MFMA. So a wave streams its weights in whole 1 KB loads and no value moves
// between lanes. A weight is kept as sign and magnitude: s = (v < 0), k = |v| - 1/2.
//   W = 4: dword j is step j; low nibbles of its bytes are columns 0..3, high ones 4..7;
//          nibble = s k2 k1 k0.
//   W = 2: dword j is steps 2j (a) and 2j + 1 (b); nibble i is column i of both:
//          s_a s_b k_a k_b.
// Behind the codes: the scales as float [tile][group][16], zero where padded.
#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRowTile = 16;
constexpr int kStep = 32;         // columns of one MFMA
constexpr int kWaves = 8;         // waves of a product workgroup: they split the columns
constexpr int kMvThreads = 64 * kWaves;

// ---------------------------------------------------------------- pack
// One thread per 16-byte unit: it gathers its 128 / W codes. Bound by HBM (reads m n bytes).
template <int W>
__global__ __launch_bounds__(256) void k_pack(const uint8_t* __restrict__ codes, int64_t m, int64_t n,
                                              int64_t ldc, int shift, int64_t nc, int64_t units,
                                              u32x4* __restrict__ out) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= units) return;
    const int lane = (int)(u & 63);
    const int64_t chunk = (u >> 6) % nc, tile = (u >> 6) / nc;
    const int64_t row = tile * kRowTile + (lane & 15);
    constexpr int kTop = (1 << W) - 1, kHalf = 1 << (W - 1);
    u32x4 d;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 32 / W; ++e) {
            // W = 4: e is the column; W = 2: e >> 3 picks step a or b
            const int step = W == 4 ? j : 2 * j + (e >> 3);
            const int64_t col = chunk * (512 / W) + step * kStep + 8 * (lane >> 4) + (e & 7);
            int c = row < m && col < n ? codes[row * ldc + col] + shift : kHalf;
            c = min(c, kTop);
            const uint32_t s = c < kHalf, k = s ? kHalf - 1 - c : c - kHalf;
            if (W == 4)
                w |= (s << 3 | k) << (8 * (e & 3) + 4 * (e >> 2));
            else
                w |= (s << 3 | k << 1) >> (e >> 3) << (4 * (e & 7));
        }
        d[j] = w;
    }
    out[u] = d;
}

__global__ __launch_bounds__(256) void k_pack_scales(const float* __restrict__ s, int64_t m, int64_t lds, int64_t ng,
                                                     int64_t ngp, int64_t total, float* __restrict__ out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int64_t r = i & 15, g = (i >> 4) % ngp, row = (i >> 4) / ngp * kRowTile + r;
    out[i] = row < m && g < ng ? s[row * lds + g] : 0.0f;
}

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

// The B operand of step `st` of a chunk from a lane's 16 bytes.
template <int MATH, int W>
__device__ __forceinline__ typename Mt<MATH>::Op weights(u32x4 d, int st) {
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

// 8 consecutive elements of a row of x from column k on, zeros from column n on. The
// loads need no alignment beyond the element's.
template <int MATH, int W>
__device__ __forceinline__ void load_x(const char* __restrict__ row, int64_t k, int64_t n,
                                       typename Mt<MATH>::Op (&p)[Mt<MATH>::kPieces]) {
    constexpr int kB = Mt<MATH>::kBytes;
    struct { uint32_t d[2 * kB]; } raw;
    if (k + 8 <= n) {
        __builtin_memcpy(&raw, row + k * kB, 8 * kB);
    } else {
        unsigned char b[8 * kB];
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int c = 0; c < kB; ++c) b[e * kB + c] = k + e < n ? row[(k + e) * kB + c] : 0;
        __builtin_memcpy(&raw, b, sizeof raw);
    }
    if constexpr (MATH == kF32) {
        float x[8];
        __builtin_memcpy(x, &raw, sizeof x);
        split3(x, p);
    } else {
        __builtin_memcpy(&p[0], &raw, sizeof raw);
        if constexpr (W == 2 && kB == 1) p[0] = even_odd(p[0]);
    }
}

struct MvArgs {
    const u32x4* codes;
    const float* scales;
    const char* x;
    const float* xs;
    void* y;
    int64_t m, n, T, ldx, ldy;
    int64_t nc, ngp;
    uint32_t tiles;
    int gshift;  // groups of whole chunks: chunk >> gshift is the group
    int ytype;
};

// ---------------------------------------------------------------- the product
// Workgroup (tile, token block of 16); wave w takes chunks w, w + 8, ...; A = x (rows
// are tokens), B = the weights, so a lane's four sums are four tokens of one weight row
// and share its scale. The sum is scaled every FS steps: a group, or a chunk of a longer
// one. The waves' sums meet in LDS and are added in a fixed order.
template <int MATH, int W, int FS>
__global__ __launch_bounds__(kMvThreads) void k_matvec(MvArgs a) {
    using M = Mt<MATH>;
    constexpr int kSteps = 16 / W;  // steps of a chunk
    __shared__ float red[kWaves][16][17];
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int64_t tile = blockIdx.x % a.tiles, t0 = (int64_t)(blockIdx.x / a.tiles) * 16;
    const int64_t t = min(t0 + (lane & 15), a.T - 1);
    const char* row = a.x + t * a.ldx * M::kBytes;
    const u32x4* wp = a.codes + tile * a.nc * 64 + lane;
    const float* sp = a.scales + tile * a.ngp * 16 + (lane & 15);
    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t c = w; c < a.nc; c += kWaves) {
        const u32x4 d = wp[c * 64];
#pragma unroll
        for (int f = 0; f < kSteps / FS; ++f) {
            typename M::Acc acc = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < FS; ++j) {
                const int st = f * FS + j;
                typename M::Op p[M::kPieces];
                load_x<MATH, W>(row, c * (512 / W) + st * kStep + 8 * (lane >> 4), a.n, p);
                const typename M::Op b = weights<MATH, W>(d, st);
#pragma unroll
                for (int i = 0; i < M::kPieces; ++i) acc = M::mma(p[i], b, acc);
            }
            const int64_t g = FS == kSteps ? c >> a.gshift : c * (kSteps / FS) + f;
            const float s = sp[g * 16];
#pragma unroll
            for (int v = 0; v < 4; ++v) sum[v] = fmaf(s, (float)acc[v], sum[v]);
        }
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) red[w][4 * (lane >> 4) + v][lane & 15] = sum[v];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int64_t tt = t0 + (threadIdx.x >> 4), i = tile * 16 + (threadIdx.x & 15);
        if (tt < a.T && i < a.m) {
            float y = 0.0f;
#pragma unroll
            for (int k = 0; k < kWaves; ++k) y += red[k][threadIdx.x >> 4][threadIdx.x & 15];
            y *= unit<MATH, W>();
            if (a.xs) y *= a.xs[tt];
            store_elem(a.y, a.ytype, tt * a.ldy + i, y);
        }
    }
}

template <int MATH, int W, int FS>
void launch_mv(const MvArgs& a, hipStream_t stream) {
    const dim3 grid(a.tiles * (unsigned)((a.T + 15) / 16));
    hipLaunchKernelGGL((k_matvec<MATH, W, FS>), grid, dim3(kMvThreads), 0, stream, a);
}

template <int MATH, int W>
void launch_mv_fs(const MvArgs& a, int fs, hipStream_t stream) {
    switch (fs) {
        case 1: launch_mv<MATH, W, 1>(a, stream); break;
        case 2: launch_mv<MATH, W, 2>(a, stream); break;
        case 4: launch_mv<MATH, W, 4>(a, stream); break;
        default:
            if constexpr (W == 2) launch_mv<MATH, W, 8>(a, stream);
            break;
    }
}

template <int MATH>
void launch_mv_w(const MvArgs& a, int W, int fs, hipStream_t stream) {
    if (W == 4) launch_mv_fs<MATH, 4>(a, fs, stream);
    else launch_mv_fs<MATH, 2>(a, fs, stream);
}

}  // namespace

PackShape pack_shape(int64_t m, int64_t n, int bits, int64_t group) {
    PackShape p;
    p.W = bits <= 2 ? 2 : 4;
    p.tiles = (m + kRowTile - 1) / kRowTile;
    const int64_t ck = 512 / p.W;
    p.chunks = (n + ck - 1) / ck;
    p.groups = group ? (n + group - 1) / group : 1;
    p.groups_padded = group && group < ck ? p.chunks * (ck / group) : p.groups;
    p.scale_offset = (size_t)p.tiles * p.chunks * 1024;
    p.bytes = p.scale_offset + (size_t)p.tiles * p.groups_padded * kRowTile * sizeof(float);
    return p;
}

int launch_pack(const uint8_t* codes, int64_t m, int64_t n, int64_t ldc, int bits, const float* scales, int64_t lds,
                int64_t group, void* packed, hipStream_t stream) {
    const PackShape p = pack_shape(m, n, bits, group);
    const int64_t units = p.tiles * p.chunks * 64, total = p.tiles * p.groups_padded * kRowTile;
    const int shift = ((1 << p.W) - (1 << bits)) / 2;
    const dim3 grid((unsigned)((units + 255) / 256)), sgrid((unsigned)((total + 255) / 256));
    u32x4* out = (u32x4*)packed;
    if (p.W == 4)
        hipLaunchKernelGGL(k_pack<4>, grid, dim3(256), 0, stream, codes, m, n, ldc, shift, p.chunks, units, out);
    else
        hipLaunchKernelGGL(k_pack<2>, grid, dim3(256), 0, stream, codes, m, n, ldc, shift, p.chunks, units, out);
    hipLaunchKernelGGL(k_pack_scales, sgrid, dim3(256), 0, stream, scales, m, lds, p.groups, p.groups_padded, total,
                       (float*)((char*)packed + p.scale_offset));
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

int launch_matvec(const void* packed, int64_t m, int64_t n, int bits, int64_t group, const void* x, int xtype,
                  int64_t T, int64_t ldx, const float* xs, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    const PackShape p = pack_shape(m, n, bits, group);
    const int64_t ck = 512 / p.W;
    MvArgs a;
    a.codes = (const u32x4*)packed;
    a.scales = (const float*)((const char*)packed + p.scale_offset);
    a.x = (const char*)x;
    a.xs = xs;
    a.y = y;
    a.m = m;
    a.n = n;
    a.T = T;
    a.ldx = ldx;
    a.ldy = ldy;
    a.tiles = (uint32_t)p.tiles;
    a.nc = p.chunks;
    a.ngp = p.groups_padded;
    a.ytype = ytype;
    a.gshift = 62;  // one group
    int fs = (int)(ck / kStep);
    if (group && group < ck) {
        fs = (int)(group / kStep);
    } else if (group) {
        a.gshift = 0;
        while ((ck << a.gshift) < group) ++a.gshift;
    }
    switch (xtype) {
        case BAKRON_F32: launch_mv_w<kF32>(a, p.W, fs, stream); break;
        case BAKRON_F16: launch_mv_w<kF16>(a, p.W, fs, stream); break;
        case BAKRON_BF16: launch_mv_w<kBF16>(a, p.W, fs, stream); break;
        case BAKRON_I8: launch_mv_w<kI8>(a, p.W, fs, stream); break;
        default: launch_mv_w<kF8>(a, p.W, fs, stream); break;
    }
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
