// bk_norm.hip -- the norm in front of a quantised layer: residual, root mean square,
// rotation, and rounding to 8 bits, in one pass over a token's row.
//
//   h = x + r,  v = U (gain * h / sqrt(mean(h^2) + eps)),
// U the randomised Hadamard matrix that bk_rotate.hip applies to the layer's weights and
// factors (or none), and out: v in fp32, fp16 or bf16, or codes q = round(v / s) in int8
// or e4m3 with one scale a token, s = max|v| / 127 or / 448. Everything between the loads
// and the stores is fp32; h is stored rounded, but the norm is that of the unrounded sum.
//
// u = H (signs * gain * h) is formed first and the row's factor f = 1 / (sqrt(b) rms) is
// applied last, so a value is rounded once for the gain, once a butterfly and once for f;
// the codes are u * (127 / max|u|), which f does not enter.
//
// Bound by HBM for many rows (x, r, h and y are touched once: the row stays in registers):
// 4096 bf16 rows of 8192 with residual 50 us, 5.3 TB/s. With the rotation its vector
// instructions and LDS passes come close (e4m3 out: 62 us, 3.8 TB/s). By latency for few: one
// row of 4096 3.2 us, rotated to int8 4.4 (an empty kernel 2.4).
#include <cmath>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

struct NormArgs {
    const void* x;
    const void* r;
    void* h;
    const void* gain;
    void* y;
    float* ys;
    int64_t T, n, ldx, ldr, ldh, ldy;
    int gfloat;   // gain is fp32 (else x's type)
    int xtype, ytype;
    float eps;
    int rotate, kbits;
    uint64_t seed;
    float rscale;
};

template <typename T> struct Vec { typedef T type __attribute__((ext_vector_type(8))); };

// 8 elements from column c on of a row of `type` T, zeros from column n on; no alignment
// beyond the element's is assumed.
// kWhole: n is a multiple of 8 (and c < n), so there is no tail.
template <bool kWhole, typename T>
__device__ __forceinline__ typename Vec<T>::type load8(const T* row, int c, int n) {
    typename Vec<T>::type v;
    if (kWhole || c + 8 <= n) {
        __builtin_memcpy(&v, row + c, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < n ? row[c + e] : (T)0.0f;
    }
    return v;
}
template <bool kWhole, typename T>
__device__ __forceinline__ void store8(T* row, int c, int n, typename Vec<T>::type v) {
    if (kWhole || c + 8 <= n) {
        __builtin_memcpy(row + c, &v, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < n) row[c + e] = v[e];
    }
}
template <bool kWhole, typename T>
__device__ __forceinline__ void store8f(void* row, int c, int n, const float (&f)[8]) {
    typename Vec<T>::type v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (T)f[e];
    store8<kWhole>((T*)row, c, n, v);
}

constexpr float kMaxFinite = 3.402823466e38f;

// Over a wave: within 16 lanes by DPP (quad permutations, half-row and row mirrors), then
// two exchanges; over the workgroup through `red`, whose values 16 lanes reduce again.
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false);
}
template <typename F>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, F op) {
    v = op(v, dpp<0xB1>(v));
    v = op(v, dpp<0x4E>(v));
    v = op(v, dpp<0x141>(v));
    return op(v, dpp<0x140>(v));
}
template <typename F>  // op(v, 0) is v
__device__ __forceinline__ uint32_t block_reduce(uint32_t v, uint32_t* red, F op) {
    v = row_reduce(v, op);
    v = op(v, (uint32_t)__shfl_xor((int)v, 16));
    v = op(v, (uint32_t)__shfl_xor((int)v, 32));
    const int waves = blockDim.x >> 6;  // at most 16
    if (waves == 1) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    const int i = threadIdx.x & 15;
    return row_reduce(i < waves ? red[i] : 0u, op);
}
__device__ __forceinline__ float block_sum(float v, uint32_t* red) {
    return __uint_as_float(block_reduce(__float_as_uint(v), red, [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    }));
}
// The largest magnitude, as the bits of |v|: their order as integers is that of the values,
// infinity and then NaN above all others.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ float block_max(uint32_t v, uint32_t* red) {
    return __uint_as_float(block_reduce(v, red, [](uint32_t x, uint32_t y) { return max(x, y); }));
}

// The codes of a row with maximum mx = max|u| and factor f are (u * up) * inv, and its scale
// is mx f / top. `up` is 2^64 for a maximum whose reciprocal fp32 may not hold. A row of
// zeros: scale 0; a row that is not finite: scale NaN; inv 0 and codes 0 in both. A code
// needs no clamping: |u| <= mx, so |u up inv| <= top (1 + 2^-22), which rounds to top.
struct Coder {
    float up, inv, scale;
    __device__ __forceinline__ Coder(float mx, float f, bool i8) {
        const float top = i8 ? 127.0f : 448.0f;
        scale = mx * f / top;
        if (!(mx <= kMaxFinite) || !(scale <= kMaxFinite)) scale = NAN;
        up = mx < 0x1p-64f ? 0x1p64f : 1.0f;
        inv = scale >= 0.0f && mx > 0.0f ? top / (mx * up) : 0.0f;
    }
};
// Four codes of u. int8: behind 1.5 * 2^23 a float's low byte is the integer it was rounded to.
__device__ __forceinline__ uint32_t e4m3_4(const float* u, float inv) {
    const int w = __builtin_amdgcn_cvt_pk_fp8_f32(u[0] * inv, u[1] * inv, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(u[2] * inv, u[3] * inv, w, true);
}
__device__ __forceinline__ uint32_t int8_4(const float* u, float inv) {
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = __float_as_uint(fmaf(u[e], inv, 12582912.0f));
    return __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[3], q[2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u), 0x05040100u);
}

// LDS address of element e of a row in floats: 8 floats of padding behind 64, so that the
// strided reads of the lowest pass fall on all banks. Additive over disjoint bits of e.
__device__ __forceinline__ int at(int e) { return e + ((e >> 6) << 3); }

// The butterflies of index bits [w0 + skip, w0 + 3) among the 8 values of a thread.
__device__ __forceinline__ void butterflies(float (&v)[8], int skip, int end) {
#pragma unroll
    for (int s = 0; s < 3; ++s)
        if (s >= skip && s < end)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if ((j & (1 << s)) == 0) {
                    const float a = v[j], b = v[j | (1 << s)];
                    v[j] = a + b;
                    v[j | (1 << s)] = a - b;
                }
}

// h = x + r of 8 columns from c on, in fp32.
template <bool kWhole, typename TX>
__device__ __forceinline__ void load_sum(const NormArgs& a, int64_t row, int c, int n, float (&v)[8]) {
    const auto x = load8<kWhole>((const TX*)a.x + row * a.ldx, c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
    if (a.r) {
        const auto r = load8<kWhole>((const TX*)a.r + row * a.ldr, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += (float)r[e];
    }
}
template <bool kWhole, typename TX>
__device__ __forceinline__ void load_gain(const NormArgs& a, int c, int n, float (&g)[8]) {
    if (!a.gain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.0f;
    } else if (a.gfloat) {
        const auto w = load8<kWhole>((const float*)a.gain, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = w[e];
    } else {
        const auto w = load8<kWhole>((const TX*)a.gain, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (float)w[e];
    }
}
// The signs of columns c .. c + 7, a bit each: bit 63 of SplitMix64's outputs c .. c + 7
// (splitmix64_out; its last step, z ^ z >> 31, leaves that bit as it is).
__device__ __forceinline__ uint32_t sign_bits(uint64_t seed, int c) {
    constexpr uint64_t kStep = 0x9E3779B97F4A7C15ull;
    const uint64_t first = seed + (uint64_t)(c + 1) * kStep;
    uint32_t neg = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        uint64_t z = first + e * kStep;
        z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
        z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
        neg |= (uint32_t)(z >> 63) << e;
    }
    return neg;
}
__device__ __forceinline__ float signed_gain(float g, uint32_t bit) {
    return __uint_as_float(__float_as_uint(g) ^ (bit << 31));
}
// The outputs of columns c .. c + 7: u f, or the codes of u.
template <bool kWhole>
__device__ __forceinline__ void store_row(const NormArgs& a, int64_t row, int c, int n, float (&u)[8], float f,
                                          const Coder& code) {
    if (a.ys) {
        uint32_t d[2] = {0, 0};
        if (code.inv > 0.0f) {
            if (code.up != 1.0f)
#pragma unroll
                for (int e = 0; e < 8; ++e) u[e] *= code.up;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                d[k] = a.ytype == BAKRON_I8 ? int8_4(u + 4 * k, code.inv) : e4m3_4(u + 4 * k, code.inv);
        }
        Vec<uint8_t>::type w;
        __builtin_memcpy(&w, d, 8);
        store8<kWhole>((uint8_t*)a.y + row * a.ldy, c, n, w);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= f;
    if (a.ytype == BAKRON_F32) store8f<kWhole, float>((float*)a.y + row * a.ldy, c, n, u);
    else if (a.ytype == BAKRON_F16) store8f<kWhole, _Float16>((_Float16*)a.y + row * a.ldy, c, n, u);
    else store8f<kWhole, __bf16>((__bf16*)a.y + row * a.ldy, c, n, u);
}

// A row per workgroup at a time, in registers: thread t holds columns 8 q .. 8 q + 7 of
// the groups q = t + i threads. Without rotation (kRot) a workgroup per row; with it,
// workgroups take rows blockIdx.x, + gridDim.x, ... and keep the signs in registers.
// Rotation: index bits 0..2 in registers, then passes over three bits each through LDS
// (n % 8 == 0 whenever there are any): group q of a pass with window w0 holds the elements
// that differ in bits w0..w0+2. Bits below 9 stay within a wave's 512 columns. The order
// 2^kbits is a template argument: the passes' bounds and offsets are then constants, which
// as run-time values overflowed the scalar registers (4096 rows of 8192: 68 us, with it 62).
template <typename TX, int NV, int kbits>
__global__ __launch_bounds__(1024) __attribute__((amdgpu_waves_per_eu(NV == 1 ? 8 : 4))) void k_norm_rows(NormArgs a) {
    constexpr bool kRot = kbits >= 0, kWhole = kbits >= 3;
    extern __shared__ __align__(16) float buf[];
    __shared__ uint32_t red[2][16];
    const int n = (int)a.n, threads = blockDim.x;
    uint32_t neg = 0;  // 8 bits a group
    // the first row's loads, before the signs are drawn (about 1 us of multiplications): 16-bit types, whose
    // registers allow it
    using V = typename Vec<TX>::type;
    constexpr bool kFirst = kRot && kWhole && sizeof(TX) == 2;
    V fx[NV], fr[NV];
    if (kFirst)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = min(8 * ((int)threadIdx.x + i * threads), n - 8);
            fx[i] = load8<kWhole>((const TX*)a.x + blockIdx.x * a.ldx, c, n);
            fr[i] = load8<kWhole>((const TX*)(a.r ? a.r : a.x) + blockIdx.x * (a.r ? a.ldr : a.ldx), c, n);
        }
    if (kRot)
#pragma unroll 1
        for (int i = 0; i < NV; ++i) neg |= sign_bits(a.seed, 8 * ((int)threadIdx.x + i * threads)) << (8 * i);
    // one group a thread: its gain, signs applied, stays in registers too. Addresses are computed in each
    // row (from an opaque thread index), with more groups where they are used, instead of held in registers
    constexpr bool kKeep = NV == 1;
    float g0[8] = {};
    if (kKeep && 8 * (int)threadIdx.x < n) {
        load_gain<kWhole, TX>(a, 8 * (int)threadIdx.x, n, g0);
        if (kRot)
#pragma unroll
            for (int e = 0; e < 8; ++e) g0[e] = signed_gain(g0[e], neg >> e);
    }
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const int t0 = tid_opaque();
        const auto tid = [&] { return kKeep ? t0 : tid_opaque(); };
        float v[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid() + i * threads);
            if (c < n) {
                float g[8];
                if (kFirst && row == blockIdx.x) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) v[i][e] = a.r ? (float)fx[i][e] + (float)fr[i][e] : (float)fx[i][e];
                } else {
                    load_sum<kWhole, TX>(a, row, c, n, v[i]);
                }
                if (!kKeep) load_gain<kWhole, TX>(a, c, n, g);
                if (a.h) store8f<kWhole, TX>((TX*)a.h + row * a.ldh, c, n, v[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(v[i][e], v[i][e], ss);
                    v[i][e] *= kKeep ? g0[e] : kRot ? signed_gain(g[e], neg >> (8 * i + e)) : g[e];
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
            }
            if (NV > 1) __builtin_amdgcn_sched_barrier(0);  // one group's loads at a time: registers
        }
        ss = block_sum(ss, red[0]);
        const float f = (kRot ? a.rscale : 1.0f) / sqrtf(ss / (float)n + a.eps);
        if (kRot) {
#pragma unroll
            for (int i = 0; i < NV; ++i) butterflies(v[i], 0, kbits);
            if (kbits > 3) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = tid() + i * threads;
                    if (8 * q < n) {
                        float* p = buf + at(8 * q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] = v[i][e];
                    }
                }
                const auto pass = [&](int w0, int skip) {
                    if (w0 + 3 > 9) __syncthreads();
                    else wave_fence();
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int q = tid() + i * threads;
                        if (8 * q < n) {
                            float* p = buf + at((q >> w0 << (w0 + 3)) | (q & ((1 << w0) - 1)));
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[i][j] = p[at(j << w0)];
                            butterflies(v[i], skip, 3);
#pragma unroll
                            for (int j = 0; j < 8; ++j) p[at(j << w0)] = v[i][j];
                        }
                        if (NV > 1) __builtin_amdgcn_sched_barrier(0);
                    }
                };
                // whole windows, then one that ends at the top bit and skips the stages that are done
                if (kbits >= 6) pass(3, 0);
                if (kbits >= 9) pass(6, 0);
                if (kbits >= 12) pass(9, 0);
                if (kbits % 3 != 0) pass(kbits - 3, 3 - kbits % 3);
                if (kbits > 9) __syncthreads();
                else wave_fence();
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = tid() + i * threads;
                    if (8 * q < n) {
                        const float* p = buf + at(8 * q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) v[i][e] = p[e];
                    }
                }
            }
        }
        float mx = 0.0f;
        if (a.ys) {
            uint32_t top = 0;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, mag(v[i][e]));
            mx = block_max(top, red[1]);
        }
        const Coder code(mx, f, a.ytype == BAKRON_I8);
        if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid() + i * threads);
            if (c < n) store_row<kWhole>(a, row, c, n, v[i], f, code);
            if (NV > 1) __builtin_amdgcn_sched_barrier(0);
        }
        if (row + gridDim.x >= a.T) break;
        if (threads > 64) __syncthreads();  // the next row writes red and buf again
        else wave_fence();
    }
}

// Rows of 16385 to 32768 columns: a workgroup's registers would not hold them beside their
// addresses, so u is kept in LDS (128 KB) and every step is a loop over its groups.
constexpr int kLongThreads = 1024;
template <typename TX>
__global__ __launch_bounds__(kLongThreads) void k_norm_lds(NormArgs a) {
    extern __shared__ __align__(16) float buf[];
    __shared__ uint32_t red[2][kLongThreads / 64];
    const int n = (int)a.n, groups = (n + 7) / 8;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        float ss = 0.0f;
#pragma unroll 1
        for (int q = threadIdx.x; q < groups; q += kLongThreads) {
            float v[8], g[8];
            load_sum<false, TX>(a, row, 8 * q, n, v);
            if (a.h) store8f<false, TX>((TX*)a.h + row * a.ldh, 8 * q, n, v);
            load_gain<false, TX>(a, 8 * q, n, g);
            const uint32_t neg = a.rotate ? sign_bits(a.seed, 8 * q) : 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(v[e], v[e], ss);
                v[e] *= signed_gain(g[e], neg >> e);
            }
            if (a.rotate) butterflies(v, 0, a.kbits);
            float* p = buf + at(8 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e) p[e] = v[e];
        }
        ss = block_sum(ss, red[0]);
        const float f = (a.rotate ? a.rscale : 1.0f) / sqrtf(ss / (float)n + a.eps);
        if (a.rotate)
            for (int done = 3; done < a.kbits;) {
                const int w0 = min(done, a.kbits - 3);
                __syncthreads();
#pragma unroll 1
                for (int q = threadIdx.x; q < groups; q += kLongThreads) {
                    float* p = buf + at((q >> w0 << (w0 + 3)) | (q & ((1 << w0) - 1)));
                    float v[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = p[at(j << w0)];
                    butterflies(v, done - w0, 3);
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[at(j << w0)] = v[j];
                }
                done = w0 + 3;
            }
        __syncthreads();
        float mx = 0.0f;
        if (a.ys) {
            uint32_t top = 0;
#pragma unroll 1
            for (int q = threadIdx.x; q < groups; q += kLongThreads) {
                const float* p = buf + at(8 * q);
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, mag(p[e]));  // zeros from column n on
            }
            mx = block_max(top, red[1]);
        }
        const Coder code(mx, f, a.ytype == BAKRON_I8);
        if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
#pragma unroll 1
        for (int q = threadIdx.x; q < groups; q += kLongThreads) {
            float v[8];
            const float* p = buf + at(8 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = p[e];
            store_row<false>(a, row, 8 * q, n, v, f, code);
        }
        __syncthreads();  // the next row writes red and buf again
    }
}

// Rows too long for registers (no rotation): x and r are read again from cache, and each
// element's loads precede its stores in the same thread, so in-place calls hold.
__global__ __launch_bounds__(kLongThreads) void k_norm_long(NormArgs a) {
    __shared__ uint32_t red[2][kLongThreads / 64];
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const auto h_of = [&](int64_t i) {
            float h = load_elem(a.x, a.xtype, row * a.ldx + i);
            if (a.r) h += load_elem(a.r, a.xtype, row * a.ldr + i);
            return h;
        };
        const auto u_of = [&](int64_t i) {
            const float h = h_of(i);
            return a.gain ? h * load_elem(a.gain, a.gfloat ? BAKRON_F32 : a.xtype, i) : h;
        };
        float ss = 0.0f;
        for (int64_t i = threadIdx.x; i < a.n; i += kLongThreads) {
            const float h = h_of(i);
            ss = fmaf(h, h, ss);
        }
        const float f = 1.0f / sqrtf(block_sum(ss, red[0]) / (float)a.n + a.eps);
        const bool i8 = a.ytype == BAKRON_I8;
        float mx = 0.0f;
        if (a.ys) {
            uint32_t top = 0;
            for (int64_t i = threadIdx.x; i < a.n; i += kLongThreads) top = max(top, mag(u_of(i)));
            mx = block_max(top, red[1]);
        }
        const Coder code(mx, f, i8);
        if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
        for (int64_t i = threadIdx.x; i < a.n; i += kLongThreads) {
            const float h = h_of(i), u = u_of(i);
            if (a.h) store_elem(a.h, a.xtype, row * a.ldh + i, h);
            if (!a.ys) {
                store_elem(a.y, a.ytype, row * a.ldy + i, u * f);
            } else {
                const float w[4] = {u * code.up, 0.0f, 0.0f, 0.0f};
                const uint32_t q = i8 ? int8_4(w, code.inv) : e4m3_4(w, code.inv);
                ((uint8_t*)a.y)[row * a.ldy + i] = code.inv > 0.0f ? (uint8_t)q : (uint8_t)0;
            }
        }
        __syncthreads();  // the next row writes red again
    }
}

constexpr int64_t kMaxRowGrid = 1 << 21;  // a grid has fewer than 2^32 threads

template <typename TX, int NV, int kbits>
void launch_rows(const NormArgs& a, hipStream_t stream) {
    const int threads = (int)((a.n + 512 * NV - 1) / (512 * NV)) * 64;
    // enough workgroups to fill the chip; each then keeps its signs and gain over its rows
    const int64_t most = (int64_t)device_info().cus * (2048 / threads);
    // rows of a workgroup, as even as possible; without rotation one, but for more rows than a grid has
    const int64_t per = (a.T + (kbits >= 0 ? most : kMaxRowGrid) - 1) / (kbits >= 0 ? most : kMaxRowGrid);
    const unsigned grid = (unsigned)((a.T + per - 1) / per);
    const size_t lds = kbits > 3 ? sizeof(float) * (a.n + (a.n >> 6 << 3)) : 0;
    hipLaunchKernelGGL((k_norm_rows<TX, NV, kbits>), dim3(grid), dim3(threads), lds, stream, a);
}

template <typename TX, int NV, int kbits>
void launch_order(const NormArgs& a, hipStream_t stream) {
    if (!a.rotate) launch_rows<TX, NV, -1>(a, stream);
    else if (a.kbits == kbits) launch_rows<TX, NV, kbits>(a, stream);
    else if constexpr (kbits > 0) launch_order<TX, NV, kbits - 1>(a, stream);
}

template <typename TX>
void launch_type(const NormArgs& a, hipStream_t stream) {
    if (a.n <= 8192) launch_order<TX, 1, 13>(a, stream);
    else if (a.n <= 16384) launch_order<TX, 2, 14>(a, stream);
    else
        hipLaunchKernelGGL(k_norm_lds<TX>, dim3((unsigned)std::min(a.T, kMaxRowGrid)), dim3(kLongThreads),
                           sizeof(float) * (a.n + 8 + ((a.n + 7) >> 6 << 3)), stream, a);
}

}  // namespace

int launch_rmsnorm(const void* x, int xtype, int64_t T, int64_t n, int64_t ldx, const void* r, int64_t ldr, void* h,
                   int64_t ldh, const void* gain, int gtype, float eps, int rotate, uint64_t seed, void* y, int ytype,
                   int64_t ldy, float* ys, hipStream_t stream) {
    NormArgs a;
    a.x = x;
    a.r = r;
    a.h = h;
    a.gain = gain;
    a.y = y;
    a.ys = ytype == BAKRON_I8 || ytype == BAKRON_E4M3 ? ys : nullptr;
    a.T = T;
    a.n = n;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.gfloat = gtype == BAKRON_F32;
    a.xtype = xtype;
    a.ytype = ytype;
    a.eps = eps;
    a.rotate = rotate;
    a.kbits = 0;
    while (((n >> a.kbits) & 1) == 0) ++a.kbits;
    a.seed = seed;
    a.rscale = (float)(1.0 / std::sqrt((double)((int64_t)1 << a.kbits)));
    if (n > kNormMaxBuffered)
        hipLaunchKernelGGL(k_norm_long, dim3((unsigned)std::min(T, kMaxRowGrid)), dim3(kLongThreads), 0, stream, a);
    else if (xtype == BAKRON_F32)
        launch_type<float>(a, stream);
    else if (xtype == BAKRON_F16)
        launch_type<_Float16>(a, stream);
    else
        launch_type<__bf16>(a, stream);
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
