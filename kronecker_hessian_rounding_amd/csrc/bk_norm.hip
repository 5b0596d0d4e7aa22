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
// Bound by HBM for many rows (x, r, h and y are touched once: the row stays in registers),
// by latency for few.
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
template <typename T>
__device__ __forceinline__ typename Vec<T>::type load8(const T* row, int c, int n) {
    typename Vec<T>::type v;
    if (c + 8 <= n) {
        __builtin_memcpy(&v, row + c, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = c + e < n ? row[c + e] : (T)0.0f;
    }
    return v;
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int n, typename Vec<T>::type v) {
    if (c + 8 <= n) {
        __builtin_memcpy(row + c, &v, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (c + e < n) row[c + e] = v[e];
    }
}
template <typename T>
__device__ __forceinline__ void store8f(void* row, int c, int n, const float (&f)[8]) {
    typename Vec<T>::type v;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (T)f[e];
    store8((T*)row, c, n, v);
}

constexpr float kMaxFinite = 3.402823466e38f;

// |v| for the row's maximum: a value that is not finite counts as infinity.
__device__ __forceinline__ float mag(float v) {
    const float a = fabsf(v);
    return a <= kMaxFinite ? a : INFINITY;
}

template <int THREADS>
__device__ __forceinline__ float block_reduce(float v, float* red, bool max) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
        const float w = __shfl_xor(v, o);
        v = max ? fmaxf(v, w) : v + w;
    }
    if (THREADS == 64) return v;
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < THREADS / 64; ++i) s = max ? fmaxf(s, red[i]) : s + red[i];
    return s;
}

// The codes of a row with maximum mx = max|u| and factor f are (u * up) * inv, and its scale
// is mx f / top. `up` is 2^64 for a maximum whose reciprocal fp32 may not hold. A row of
// zeros: scale 0; a row that is not finite: scale NaN; codes 0 in both.
struct Coder {
    float top, up, inv, scale;
    __device__ __forceinline__ Coder(float mx, float f, bool i8) {
        top = i8 ? 127.0f : 448.0f;
        scale = mx * f / top;
        if (!(mx <= kMaxFinite) || !(scale <= kMaxFinite)) scale = NAN;
        up = mx < 0x1p-64f ? 0x1p64f : 1.0f;
        inv = scale >= 0.0f && mx > 0.0f ? top / (mx * up) : 0.0f;
    }
    __device__ __forceinline__ float operator()(float u) const {
        const float q = fminf(fmaxf(u * up * inv, -top), top);
        return inv > 0.0f ? q : 0.0f;  // u may be infinite or NaN where inv is 0
    }
};
__device__ __forceinline__ uint32_t e4m3_4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}
__device__ __forceinline__ uint32_t int8_4(float a, float b, float c, float d) {
    const auto q = [](float v) { return (uint32_t)(int)rintf(v) & 255u; };
    return q(a) | q(b) << 8 | q(c) << 16 | q(d) << 24;
}

// LDS address of element e of a row in floats: 8 floats of padding behind 64, so that the
// strided reads of the lowest pass fall on all banks.
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
template <typename TX>
__device__ __forceinline__ void load_sum(const NormArgs& a, int64_t row, int c, int n, float (&v)[8]) {
    const auto x = load8((const TX*)a.x + row * a.ldx, c, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
    if (a.r) {
        const auto r = load8((const TX*)a.r + row * a.ldr, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += (float)r[e];
    }
}
template <typename TX>
__device__ __forceinline__ void load_gain(const NormArgs& a, int c, int n, float (&g)[8]) {
    if (!a.gain) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 1.0f;
    } else if (a.gfloat) {
        const auto w = load8((const float*)a.gain, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = w[e];
    } else {
        const auto w = load8((const TX*)a.gain, c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (float)w[e];
    }
}
// The signs of columns c .. c + 7, a bit each.
__device__ __forceinline__ uint32_t sign_bits(uint64_t seed, int c) {
    uint32_t neg = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) neg |= (uint32_t)(splitmix64_out(seed, (uint64_t)(c + e)) >> 63) << e;
    return neg;
}
__device__ __forceinline__ float signed_gain(float g, uint32_t bit) {
    return __uint_as_float(__float_as_uint(g) ^ (bit << 31));
}
// The outputs of columns c .. c + 7: u f, or the codes of u.
__device__ __forceinline__ void store_row(const NormArgs& a, int64_t row, int c, int n, float (&u)[8], float f,
                                          const Coder& code) {
    if (a.ys) {
        float q[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) q[e] = code(u[e]);
        uint32_t d[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
            d[k] = a.ytype == BAKRON_I8 ? int8_4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3])
                                        : e4m3_4(q[4 * k], q[4 * k + 1], q[4 * k + 2], q[4 * k + 3]);
        Vec<uint8_t>::type w;
        __builtin_memcpy(&w, d, 8);
        store8((uint8_t*)a.y + row * a.ldy, c, n, w);
        return;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= f;
    if (a.ytype == BAKRON_F32) store8f<float>((float*)a.y + row * a.ldy, c, n, u);
    else if (a.ytype == BAKRON_F16) store8f<_Float16>((_Float16*)a.y + row * a.ldy, c, n, u);
    else store8f<__bf16>((__bf16*)a.y + row * a.ldy, c, n, u);
}

// A row per workgroup at a time, in registers: thread t holds columns 8 q .. 8 q + 7 of
// the groups q = t + i THREADS. Workgroups take rows blockIdx.x, + gridDim.x, ...; the
// signs stay in registers over them, and with one group a thread so does the gain, and the
// next row's x and r are on the way while a row is worked on.
// Rotation: index bits 0..2 in registers, then passes over three bits each through LDS
// (n % 8 == 0 whenever there are any): group q of a pass with window w0 holds the elements
// that differ in bits w0..w0+2. Bits below 9 stay within a wave's 512 columns.
template <typename TX, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void k_norm_rows(NormArgs a) {
    using V = typename Vec<TX>::type;
    extern __shared__ float buf[];
    __shared__ float red[2][THREADS / 64];
    const int n = (int)a.n;
    constexpr bool kKeep = NV == 1;
    // opaque where a thread holds several groups: their addresses are then computed where they are used
    // instead of held in registers over the row and the loop
    const auto tid = [] { return kKeep ? (int)threadIdx.x : tid_opaque(); };
    const int c0 = 8 * (int)threadIdx.x;
    V xv, rv;
    const auto fetch = [&](int64_t row) {
        xv = load8((const TX*)a.x + row * a.ldx, c0, n);
        if (a.r) rv = load8((const TX*)a.r + row * a.ldr, c0, n);
    };
    float g0[8];
    if (kKeep && c0 < n) {
        fetch(blockIdx.x);
        load_gain<TX>(a, c0, n, g0);
    }
    uint32_t neg = 0;  // 8 bits a group
    if (a.rotate)
#pragma unroll 1
        for (int i = 0; i < NV; ++i) neg |= sign_bits(a.seed, 8 * ((int)threadIdx.x + i * THREADS)) << (8 * i);
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        float v[NV][8];
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid() + i * THREADS);
            if (c < n) {
                float g[8];
                if (kKeep) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        g[e] = g0[e];
                        v[i][e] = a.r ? (float)xv[e] + (float)rv[e] : (float)xv[e];
                    }
                } else {
                    load_sum<TX>(a, row, c, n, v[i]);
                    load_gain<TX>(a, c, n, g);
                }
                if (a.h) store8f<TX>((TX*)a.h + row * a.ldh, c, n, v[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(v[i][e], v[i][e], ss);
                    v[i][e] *= signed_gain(g[e], neg >> (8 * i + e));
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] = 0.0f;
            }
            if (!kKeep) __builtin_amdgcn_sched_barrier(0);  // one group's loads at a time: registers
        }
        if (kKeep && c0 < n && row + gridDim.x < a.T) fetch(row + gridDim.x);
        ss = block_reduce<THREADS>(ss, red[0], false);
        const float f = (a.rotate ? a.rscale : 1.0f) / sqrtf(ss / (float)n + a.eps);
        if (a.rotate) {
#pragma unroll
            for (int i = 0; i < NV; ++i) butterflies(v[i], 0, a.kbits);
            if (a.kbits > 3) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = tid() + i * THREADS;
                    if (8 * q < n) {
                        float* p = buf + at(8 * q);
#pragma unroll
                        for (int e = 0; e < 8; ++e) p[e] = v[i][e];
                    }
                }
                for (int done = 3; done < a.kbits;) {
                    const int w0 = min(done, a.kbits - 3);
                    if (w0 + 3 > 9) __syncthreads();
#pragma unroll
                    for (int i = 0; i < NV; ++i) {
                        const int q = tid() + i * THREADS;
                        if (8 * q < n) {
                            const int e0 = (q >> w0 << (w0 + 3)) | (q & ((1 << w0) - 1));
#pragma unroll
                            for (int j = 0; j < 8; ++j) v[i][j] = buf[at(e0 + (j << w0))];
                            butterflies(v[i], done - w0, 3);
#pragma unroll
                            for (int j = 0; j < 8; ++j) buf[at(e0 + (j << w0))] = v[i][j];
                        }
                        if (!kKeep) __builtin_amdgcn_sched_barrier(0);
                    }
                    done = w0 + 3;
                }
                if (a.kbits > 9) __syncthreads();
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int q = tid() + i * THREADS;
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
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) mx = fmaxf(mx, mag(v[i][e]));
            mx = block_reduce<THREADS>(mx, red[1], true);
        }
        const Coder code(mx, f, a.ytype == BAKRON_I8);
        if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = 8 * (tid() + i * THREADS);
            if (c < n) store_row(a, row, c, n, v[i], f, code);
            if (!kKeep) __builtin_amdgcn_sched_barrier(0);
        }
        // the next row writes red and buf again
        if (THREADS > 64) __syncthreads();
    }
}

// Rows of 16385 to 32768 columns: a workgroup's registers would not hold them beside their
// addresses, so u is kept in LDS (128 KB) and every step is a loop over its groups.
constexpr int kLongThreads = 1024;
template <typename TX>
__global__ __launch_bounds__(kLongThreads) void k_norm_lds(NormArgs a) {
    extern __shared__ float buf[];
    __shared__ float red[2][kLongThreads / 64];
    const int n = (int)a.n, groups = (n + 7) / 8;
    const int64_t row = blockIdx.x;
    float ss = 0.0f;
#pragma unroll 1
    for (int q = threadIdx.x; q < groups; q += kLongThreads) {
        float v[8], g[8];
        load_sum<TX>(a, row, 8 * q, n, v);
        if (a.h) store8f<TX>((TX*)a.h + row * a.ldh, 8 * q, n, v);
        load_gain<TX>(a, 8 * q, n, g);
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
    ss = block_reduce<kLongThreads>(ss, red[0], false);
    const float f = (a.rotate ? a.rscale : 1.0f) / sqrtf(ss / (float)n + a.eps);
    if (a.rotate)
        for (int done = 3; done < a.kbits;) {
            const int w0 = min(done, a.kbits - 3);
            __syncthreads();
#pragma unroll 1
            for (int q = threadIdx.x; q < groups; q += kLongThreads) {
                const int e0 = (q >> w0 << (w0 + 3)) | (q & ((1 << w0) - 1));
                float v[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = buf[at(e0 + (j << w0))];
                butterflies(v, done - w0, 3);
#pragma unroll
                for (int j = 0; j < 8; ++j) buf[at(e0 + (j << w0))] = v[j];
            }
            done = w0 + 3;
        }
    __syncthreads();
    float mx = 0.0f;
    if (a.ys) {
#pragma unroll 1
        for (int q = threadIdx.x; q < groups; q += kLongThreads) {
            const float* p = buf + at(8 * q);
#pragma unroll
            for (int e = 0; e < 8; ++e) mx = fmaxf(mx, mag(p[e]));  // zeros from column n on
        }
        mx = block_reduce<kLongThreads>(mx, red[1], true);
    }
    const Coder code(mx, f, a.ytype == BAKRON_I8);
    if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
#pragma unroll 1
    for (int q = threadIdx.x; q < groups; q += kLongThreads) {
        float v[8];
        const float* p = buf + at(8 * q);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = p[e];
        store_row(a, row, 8 * q, n, v, f, code);
    }
}

// Rows too long for registers (no rotation): x and r are read again from cache, and each
// element's loads precede its stores in the same thread, so in-place calls hold.
__global__ __launch_bounds__(kLongThreads) void k_norm_long(NormArgs a) {
    __shared__ float red[2][kLongThreads / 64];
    const int64_t row = blockIdx.x;
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
    const float f = 1.0f / sqrtf(block_reduce<kLongThreads>(ss, red[0], false) / (float)a.n + a.eps);
    const bool i8 = a.ytype == BAKRON_I8;
    float mx = 0.0f;
    if (a.ys) {
        for (int64_t i = threadIdx.x; i < a.n; i += kLongThreads) mx = fmaxf(mx, mag(u_of(i)));
        mx = block_reduce<kLongThreads>(mx, red[1], true);
    }
    const Coder code(mx, f, i8);
    if (a.ys && threadIdx.x == 0) a.ys[row] = code.scale;
    for (int64_t i = threadIdx.x; i < a.n; i += kLongThreads) {
        const float h = h_of(i), u = u_of(i);
        if (a.h) store_elem(a.h, a.xtype, row * a.ldh + i, h);
        if (!a.ys) {
            store_elem(a.y, a.ytype, row * a.ldy + i, u * f);
        } else {
            const float q = code(u);
            ((uint8_t*)a.y)[row * a.ldy + i] = (uint8_t)(i8 ? int8_4(q, 0, 0, 0) : e4m3_4(q, 0, 0, 0));
        }
    }
}

template <typename TX, int THREADS, int NV>
void launch_rows(const NormArgs& a, hipStream_t stream) {
    // enough workgroups to fill the chip; each then keeps its signs and gain over its rows
    const int per_cu = std::max(1, 2048 / THREADS / 2) * 2;
    const unsigned grid = (unsigned)std::min<int64_t>(a.T, (int64_t)device_info().cus * per_cu);
    const size_t lds = a.rotate && a.kbits > 3 ? sizeof(float) * (a.n + (a.n >> 6 << 3)) : 0;
    hipLaunchKernelGGL((k_norm_rows<TX, THREADS, NV>), dim3(grid), dim3(THREADS), lds, stream, a);
}

template <typename TX>
void launch_type(const NormArgs& a, hipStream_t stream) {
    if (a.n <= 512) launch_rows<TX, 64, 1>(a, stream);
    else if (a.n <= 2048) launch_rows<TX, 256, 1>(a, stream);
    else if (a.n <= 4096) launch_rows<TX, 512, 1>(a, stream);
    else if (a.n <= 8192) launch_rows<TX, 1024, 1>(a, stream);
    else if (a.n <= 16384) launch_rows<TX, 1024, 2>(a, stream);
    else
        hipLaunchKernelGGL(k_norm_lds<TX>, dim3((unsigned)a.T), dim3(kLongThreads),
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
        hipLaunchKernelGGL(k_norm_long, dim3((unsigned)T), dim3(kLongThreads), 0, stream, a);
    else if (xtype == BAKRON_F32)
        launch_type<float>(a, stream);
    else if (xtype == BAKRON_F16)
        launch_type<_Float16>(a, stream);
    else
        launch_type<__bf16>(a, stream);
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
