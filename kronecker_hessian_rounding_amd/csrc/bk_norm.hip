// bk_norm.hip -- the norm in front of a quantised layer: residual, root mean square,
// rotation, and rounding to 8 bits, in one pass over a token's row.
//
//   h = x + r,  v = U (gain * h / sqrt(mean(h^2) + eps)),
// U the randomised Hadamard matrix that bk_rotate.hip applies to the layer's weights and
// factors (or none), and out: v in fp32, fp16 or bf16, or codes q = round(v / s) in int8
// or e4m3 with one scale a token, s = max|v| / 127 or / 448. Everything between the loads
// and the stores is fp32; h is stored rounded, but the norm is that of the unrounded sum.
#include <cmath>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

constexpr int kNormThreads = 256;

struct NormArgs {
    const void* x;
    const void* r;
    void* h;
    const void* gain;
    void* y;
    float* ys;
    int64_t n, ldx, ldr, ldh, ldy;
    int xtype, gtype, ytype;
    float eps;
    int rotate, kbits;
    uint64_t seed;
    float rscale;
};

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kNormThreads / 64; ++i) s += red[i];
    return s;
}
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = red[0];
#pragma unroll
    for (int i = 1; i < kNormThreads / 64; ++i) s = fmaxf(s, red[i]);
    return s;
}

// |v| for the row's maximum: a value that is not finite counts as infinity.
__device__ __forceinline__ float mag(float v) {
    const float a = fabsf(v);
    return a <= 3.402823466e38f ? a : INFINITY;
}

__device__ __forceinline__ void store_code(void* y, int type, int64_t i, float v, float s) {
    // s is 0 for a row of zeros and NaN for a row that is not finite: codes 0
    float q = s > 0.0f ? v / s : 0.0f;
    if (type == BAKRON_I8) {
        ((int8_t*)y)[i] = (int8_t)(int)fminf(fmaxf(rintf(q), -127.0f), 127.0f);
    } else {
        q = fminf(fmaxf(q, -448.0f), 448.0f);
        ((uint8_t*)y)[i] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false);
    }
}

// One workgroup per row. kBuf: the row is kept in LDS; without (long rows, no rotation)
// x and r are read again, and each element's loads precede its stores in the same thread.
template <bool kBuf>
__global__ __launch_bounds__(kNormThreads) void k_norm(NormArgs a) {
    extern __shared__ float buf[];
    __shared__ float red[kNormThreads / 64];
    const int64_t row = blockIdx.x;
    const auto h_of = [&](int64_t i) {
        float h = load_elem(a.x, a.xtype, row * a.ldx + i);
        if (a.r) h += load_elem(a.r, a.xtype, row * a.ldr + i);
        return h;
    };
    float ss = 0.0f;
    for (int64_t i = threadIdx.x; i < a.n; i += kNormThreads) {
        const float h = h_of(i);
        ss = fmaf(h, h, ss);
        if (kBuf) {
            buf[i] = h;
            if (a.h) store_elem(a.h, a.xtype, row * a.ldh + i, h);
        }
    }
    const float rs = 1.0f / sqrtf(block_sum(ss, red) / (float)a.n + a.eps);
    const auto v_of = [&](int64_t i) {
        const float v = (kBuf ? buf[i] : h_of(i)) * rs;
        return a.gain ? v * load_elem(a.gain, a.gtype, i) : v;
    };
    if (kBuf) {
        for (int64_t i = threadIdx.x; i < a.n; i += kNormThreads) {
            float v = v_of(i);
            if (a.rotate && (splitmix64_out(a.seed, (uint64_t)i) >> 63)) v = -v;
            buf[i] = v;
        }
        __syncthreads();
        if (a.rotate) {
            for (int s = 0; s < a.kbits; ++s) {
                const int hs = 1 << s;
                for (int q = threadIdx.x; q < a.n / 2; q += kNormThreads) {
                    const int lo = ((q >> s) << (s + 1)) | (q & (hs - 1));
                    const float u = buf[lo], w = buf[lo + hs];
                    buf[lo] = u + w;
                    buf[lo + hs] = u - w;
                }
                __syncthreads();
            }
        }
    }
    const float rscale = a.rotate ? a.rscale : 1.0f;
    const auto out_of = [&](int64_t i) { return kBuf ? buf[i] * rscale : v_of(i); };
    float s = 0.0f;
    if (a.ys) {
        float mx = 0.0f;
        for (int64_t i = threadIdx.x; i < a.n; i += kNormThreads) mx = fmaxf(mx, mag(out_of(i)));
        mx = block_max(mx, red);
        s = mx <= 3.402823466e38f ? mx / (a.ytype == BAKRON_I8 ? 127.0f : 448.0f) : NAN;
        if (threadIdx.x == 0) a.ys[row] = s;
    }
    for (int64_t i = threadIdx.x; i < a.n; i += kNormThreads) {
        const float v = out_of(i);
        if (!kBuf && a.h) store_elem(a.h, a.xtype, row * a.ldh + i, h_of(i));
        if (a.ys) store_code(a.y, a.ytype, row * a.ldy + i, v, s);
        else store_elem(a.y, a.ytype, row * a.ldy + i, v);
    }
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
    a.n = n;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldh = ldh;
    a.ldy = ldy;
    a.xtype = xtype;
    a.gtype = gtype;
    a.ytype = ytype;
    a.eps = eps;
    a.rotate = rotate;
    a.kbits = 0;
    while (((n >> a.kbits) & 1) == 0) ++a.kbits;
    a.seed = seed;
    a.rscale = (float)(1.0 / std::sqrt((double)((int64_t)1 << a.kbits)));
    if (n <= kNormMaxBuffered)
        hipLaunchKernelGGL(k_norm<true>, dim3((unsigned)T), dim3(kNormThreads), sizeof(float) * n, stream, a);
    else
        hipLaunchKernelGGL(k_norm<false>, dim3((unsigned)T), dim3(kNormThreads), 0, stream, a);
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
