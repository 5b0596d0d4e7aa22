// bk_lora.hip -- low-rank adapters of many requests beside a shared projection.
//
// Token t names an adapter a (or none); with A_a (r x n), B_a (m x r):
//   u_tk = xs_t sum_j x_tj A_a[k][j],   y_ti = base_ti + s_a sum_k u_tk B_a[i][k].
// One launch: a workgroup takes up to 16 tokens of one adapter and a range of rows of B. It forms u for
// them first (each workgroup of a range anew: r n elements of A, which the caches hold), then its outputs,
// so that nothing passes through memory in between and no workspace is needed.
//
// The first product runs on the matrix cores in the adapter's type (x in 8 bits is converted to it without
// loss) with fp32 sums; u stays fp32, and the second product runs on the fp32 matrix cores.
#include <algorithm>
#include <type_traits>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
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
    int slots, row_blocks;     // workgroups of a token tile: adapters, ranges of rows
    int64_t rows_each;         // rows of a range, a multiple of 64
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
template <typename F, typename S, typename W>
__device__ __forceinline__ typename F::Part whole_part(const S* p) {
    uint32_t w[F::kElems * sizeof(S) / 4];
    __builtin_memcpy(w, p, sizeof w);
    return convert<F, S, W>(w);
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

// 16 elements of a row of `type`, the first `count` of them.
__device__ __forceinline__ void load16(const void* p, int type, int64_t i, int count, float (&f)[16]) {
    if (count < 16) {
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = e < count ? load_elem(p, type, i + e) : 0.0f;
    } else if (type == BAKRON_F32) {
        __builtin_memcpy(f, (const float*)p + i, 64);
    } else if (type == BAKRON_F16) {
        _Float16 h[16];
        __builtin_memcpy(h, (const _Float16*)p + i, 32);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = (float)h[e];
    } else {
        __bf16 h[16];
        __builtin_memcpy(h, (const __bf16*)p + i, 32);
#pragma unroll
        for (int e = 0; e < 16; ++e) f[e] = (float)h[e];
    }
}

constexpr int kLoraWaves = 8;

// RT: tiles of 16 ranks of a pass.
template <typename X, typename W, int RT>
__global__ __launch_bounds__(64 * kLoraWaves) void k_lora(LoraArgs a) {
    using F = First<X, W>;
    using Part = typename F::Part;
    constexpr int NW = kLoraWaves, PF = RT == 4 ? 2 : 4;
    extern __shared__ __align__(16) char lds[];
    const int rp = (int)((a.r + 15) / 16 * 16), pitch = rp + 4;
    float* u = (float*)lds;                  // [16 tokens][pitch]
    float* red = u + 16 * pitch;             // [wave][16 RT ranks][17]
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int q = lane >> 4, c = lane & 15;
    const int64_t id = blockIdx.x;
    const int rb = (int)(id % a.row_blocks), slot = (int)(id / a.row_blocks % a.slots);
    const int64_t t0 = id / a.row_blocks / a.slots * 16;
    const int64_t row0 = rb * a.rows_each, row1 = min(a.m, row0 + a.rows_each);
    const int tokens = (int)min<int64_t>(16, a.T - t0);
    // the adapter of token c (-1: none), and the lanes whose token is the first of its adapter
    int mine = c < tokens ? a.ids[t0 + c] : 0;
    if (mine < 0 || mine >= a.R) mine = -1;
    bool leads = lane < tokens;
#pragma unroll
    for (int i = 0; i < 15; ++i) leads = leads && !(i < lane && __builtin_amdgcn_readlane(mine, i) == mine);
    uint32_t left = (uint32_t)__ballot(leads);
    for (int i = 0; left; left &= left - 1, ++i) {
        if (i % a.slots != slot) continue;
        const int ad = __builtin_amdgcn_readlane(mine, __builtin_ctz(left));
        const uint32_t members = (uint32_t)__ballot(lane < tokens && mine == ad);
        // column c of the products is the c-th token of the adapter (the first again past the last)
        const int count = __popc(members);
        int tok = __builtin_ctz(members);
        {
            uint32_t s = members;
            for (int k = 0; k < 15 && k < count - 1; ++k) {
                s &= s - 1;
                if (c == k + 1) tok = __builtin_ctz(s);
            }
        }
        const int64_t t = t0 + tok;
        const bool live = c < count;
        if (ad >= 0) {
            const X* xr = (const X*)a.x + t * a.ldx;
            const W* ar = (const W*)a.a + (int64_t)ad * a.r * a.n;
            const int blocks = (int)(a.n / F::kBlock);  // whole ones
            for (int k0 = 0; k0 < rp; k0 += 16 * RT) {
                const W* row[RT];
#pragma unroll
                for (int j = 0; j < RT; ++j) row[j] = ar + min<int64_t>(k0 + 16 * j + c, a.r - 1) * a.n;
                f32x4 acc[RT] = {};
                if (blocks > 0) {
                    // each wave takes blocks w, w + NW, ..; PF of them in flight (past the last one, the last again)
                    Part xp[PF], ap[PF][RT];
                    const auto fetch = [&](int s, int b) __attribute__((always_inline)) {
                        const int64_t at = (int64_t)min(b, blocks - 1) * F::kBlock + q * F::kElems;
                        xp[s] = whole_part<F, X, W>(xr + at);
#pragma unroll
                        for (int j = 0; j < RT; ++j) ap[s][j] = whole_part<F, W, W>(row[j] + at);
                    };
#pragma unroll
                    for (int s = 0; s < PF; ++s) fetch(s, w + s * NW);
                    for (int b = w; b < blocks; b += PF * NW) {
#pragma unroll
                        for (int s = 0; s < PF; ++s) {
                            if (b + s * NW < blocks)
#pragma unroll
                                for (int j = 0; j < RT; ++j) acc[j] = F::mma(ap[s][j], xp[s], acc[j]);
                            fetch(s, b + (s + PF) * NW);
                        }
                    }
                }
                if (a.n % F::kBlock != 0 && w == blocks % NW) {  // the block that the row's end cuts
                    const int64_t at = (int64_t)blocks * F::kBlock + q * F::kElems;
                    const int cut = (int)max<int64_t>(0, min<int64_t>(F::kElems, a.n - at));
                    const Part xc = cut_part<F, X, W>(xr + min(at, a.n), cut);
#pragma unroll
                    for (int j = 0; j < RT; ++j) acc[j] = F::mma(cut_part<F, W, W>(row[j] + min(at, a.n), cut), xc, acc[j]);
                }
                // sums of the waves, in their order
                __syncthreads();
#pragma unroll
                for (int j = 0; j < RT; ++j)
#pragma unroll
                    for (int v = 0; v < 4; ++v) red[(w * 16 * RT + 16 * j + 4 * q + v) * 17 + c] = acc[j][v];
                __syncthreads();
                for (int e = threadIdx.x; e < 256 * RT; e += 64 * NW) {
                    const int k = e >> 4, tk = e & 15;
                    float s = 0.0f;
#pragma unroll
                    for (int i2 = 0; i2 < NW; ++i2) s += red[(i2 * 16 * RT + k) * 17 + tk];
                    if (k0 + k < rp) u[tk * pitch + k0 + k] = k0 + k < a.r ? s : 0.0f;
                }
            }
            __syncthreads();
        }
        const float f = ad < 0 ? 0.0f : (a.scales ? a.scales[ad] : 1.0f) * (a.xs ? a.xs[t] : 1.0f);
        // the second product: 64 rows of B a wave and turn. Row of tile j: 16 (c / 4) + 4 j + c % 4 as operand, so
        // that a lane's sums are 16 consecutive rows, 16 q .., of token c; of the ranks, lane group q has its own quarter.
        const int quarter = rp / 4;
        for (int64_t i0 = row0 + 64 * w; i0 < row1; i0 += 64 * NW) {
            f32x4 acc[4] = {};
            if (ad >= 0) {
                const W* br = (const W*)a.b + (int64_t)ad * a.m * a.r;
                const float* ur = u + c * pitch + q * quarter;
                for (int k = 0; k < quarter; k += 4) {
                    const f32x4 uk = *reinterpret_cast<const f32x4*>(ur + k);
                    const int at = q * quarter + k;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int64_t i1 = min(i0 + 16 * (c >> 2) + 4 * j + (c & 3), a.m - 1);
                        const W* p = br + i1 * a.r + at;
                        float b[4];
                        if (at + 4 <= a.r) {
                            W h[4];
                            __builtin_memcpy(h, p, sizeof h);
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[e] = (float)h[e];
                        } else {
#pragma unroll
                            for (int e = 0; e < 4; ++e) b[e] = at + e < a.r ? (float)p[e] : 0.0f;
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[e], uk[e], acc[j], 0, 0, 0);
                    }
                }
            }
            const int64_t i1 = i0 + 16 * q;
            const int rows = (int)max<int64_t>(0, min<int64_t>(16, row1 - i1));
            if (live && rows > 0) {
                float y[16] = {};
                if (a.base) load16(a.base, a.btype, t * a.ldb + i1, rows, y);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f4 v;
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = ad < 0 ? y[4 * j + e] : fmaf(f, acc[j][e], y[4 * j + e]);
                    if (4 * j < rows) store4(a.y, a.ytype, t * a.ldy + i1 + 4 * j, v, min(4, rows - 4 * j));
                }
            }
        }
        __syncthreads();  // u is read
    }
}

template <typename X, typename W, int RT>
void launch_rt(const LoraArgs& a, unsigned grid, hipStream_t stream) {
    const size_t lds = sizeof(float) * (16 * ((size_t)(a.r + 15) / 16 * 16 + 4) + kLoraWaves * 16 * RT * 17);
    hipLaunchKernelGGL((k_lora<X, W, RT>), dim3(grid), dim3(64 * kLoraWaves), lds, stream, a);
}

template <typename X, typename W>
void launch_types(const LoraArgs& a, unsigned grid, hipStream_t stream) {
    if (a.r <= 16) launch_rt<X, W, 1>(a, grid, stream);
    else if (a.r <= 32) launch_rt<X, W, 2>(a, grid, stream);
    else launch_rt<X, W, 4>(a, grid, stream);
}

}  // namespace

int launch_lora(const void* x, int xtype, int64_t T, int64_t n, int64_t ldx, const float* xs, const void* A, const void* B,
                int wtype, int64_t R, int64_t r, int64_t m, const float* scales, const int32_t* ids, const void* base,
                int btype, int64_t ldb, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    LoraArgs a;
    a.xs = xs;
    a.a = (const char*)A;
    a.b = (const char*)B;
    a.scales = scales;
    a.n = n;
    a.m = m;
    a.r = r;
    a.R = R;
    a.ldx = ldx;
    a.ldb = ldb;
    a.ldy = ldy;
    a.btype = btype;
    a.ytype = ytype;
    const int64_t xb = xtype == BAKRON_F32 ? 4 : xtype == BAKRON_I8 || xtype == BAKRON_E4M3 ? 1 : 2;
    const auto wide = [](int type) { return type == BAKRON_F32 ? 4 : 2; };
    const int64_t cus = device_info().cus, most = (int64_t)1 << 22;  // tokens of a launch
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        a.T = std::min(most, T - t0);
        a.x = (const char*)x + t0 * ldx * xb;
        a.xs = xs ? xs + t0 : nullptr;
        a.ids = ids + t0;
        a.base = base ? (const char*)base + t0 * ldb * wide(btype) : nullptr;
        a.y = (char*)y + t0 * ldy * wide(ytype);
        const int64_t tiles = (a.T + 15) / 16;
        a.slots = (int)(tiles >= cus ? 1 : std::min<int64_t>({16, a.T, R + 1}));
        const int64_t ranges = std::max<int64_t>(1, std::min((m + 511) / 512, 2 * cus / (tiles * a.slots)));
        a.rows_each = ((m + ranges - 1) / ranges + 63) / 64 * 64;
        a.row_blocks = (int)((m + a.rows_each - 1) / a.rows_each);
        const unsigned grid = (unsigned)(tiles * a.slots * a.row_blocks);
        if (wtype == BAKRON_F32) launch_types<float, float>(a, grid, stream);
        else if (wtype == BAKRON_F16) {
            if (xtype == BAKRON_F16) launch_types<_Float16, _Float16>(a, grid, stream);
            else if (xtype == BAKRON_I8) launch_types<i8, _Float16>(a, grid, stream);
            else launch_types<e4m3, _Float16>(a, grid, stream);
        } else {
            if (xtype == BAKRON_BF16) launch_types<__bf16, __bf16>(a, grid, stream);
            else if (xtype == BAKRON_I8) launch_types<i8, __bf16>(a, grid, stream);
            else launch_types<e4m3, __bf16>(a, grid, stream);
        }
    }
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
