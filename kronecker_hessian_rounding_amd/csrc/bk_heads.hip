// bk_heads.hip -- the norm of each query and key head with the position rotation, one pass.
//
// For every token t and head h (a row x of d elements, of the queries or of the keys)
//   v = gain * x / sqrt(mean(x^2) + eps)          (or v = x, without the norm)
// and the first `rot` elements of v are turned in pairs (a, b) by the angle pos_t freq_i,
//   (a cos - b sin, b cos + a sin),
// where pair i is (v_i, v_{i + rot/2}) or (v_2i, v_2i+1). fp32 throughout, one rounding at the end.
//
// Angles. pos freq is formed in 64 bits (exact below 2^29), as turns its fraction is taken there too,
// so what is left of a position's angle is within 2^-52 of its number of turns, and sine and cosine are
// fp32 functions of half a turn at most. One set of angles serves all heads of a token through LDS.
//
// Bound by HBM for prompts (each element is read and written once): 8192 tokens of 32 + 8 heads of 128, bf16, 168 MB of which
// part may stay in the caches, take 31 to 35 us, 4.75 to 5.5 TB/s; by latency and the launch for single tokens (3.5 us, of
// which 1.1 beyond an empty kernel). A workgroup of up to 512 threads holds one token's heads, so that sines and cosines,
// 64-bit products each, are formed once a token and not once a head.
#include <algorithm>
#include <cmath>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

struct HeadArgs {
    const void* x[2];  // queries, keys
    void* y[2];
    const void* gain[2];
    int64_t xt[2], xh[2], yt[2], yh[2];  // strides of tokens and of heads, in elements
    int64_t T;
    const void* pos;
    const float* freq;
    int heads[2];
    int d, rot;
    int lanes;        // lanes of a head, a power of two
    int gfloat, pos32, interleaved, norm;
    float eps;
};

typedef float f8 __attribute__((ext_vector_type(8)));
template <typename T> struct V8 { typedef T type __attribute__((ext_vector_type(8))); };

// The first `count` of 8 elements (zeros behind them); no alignment beyond the element's is needed.
template <bool kWhole, typename T>
__device__ __forceinline__ f8 get8(const T* p, int count) {
    f8 f = {};
    if (kWhole || count >= 8) {
        typename V8<T>::type v;
        __builtin_memcpy(&v, p, sizeof v);
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = (float)v[e];
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < count) f[e] = (float)p[e];
    }
    return f;
}
template <bool kWhole, typename T>
__device__ __forceinline__ void put8(T* p, int count, f8 f) {
    if (kWhole || count >= 8) {
        typename V8<T>::type v;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = (T)f[e];
        __builtin_memcpy(p, &v, sizeof v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (e < count) p[e] = (T)f[e];
    }
}

// A head is cut into items of two vectors of 8 elements: 8 pairs of the rotated part, or 16 elements of the
// rest. One lane holds one item, so no value moves between lanes but the sum of squares. A workgroup serves
// one token at a time. kWhole: every vector is whole.
template <typename T, bool kWhole>
__global__ __launch_bounds__(512) void k_head_norm(HeadArgs a) {
    extern __shared__ float trig[];  // [rot / 2] cosines, [rot / 2] sines
    const int pairs = a.rot / 2, pair_items = (pairs + 7) / 8;
    const int item = threadIdx.x & (a.lanes - 1), first = threadIdx.x / a.lanes, step = blockDim.x / a.lanes;
    const bool turned = item < pair_items;
    // the item's vectors: places and element counts
    int o1, o2, n1, n2;
    if (turned) {
        if (a.interleaved) {
            o1 = 16 * item;
            o2 = o1 + 8;
            n1 = min(8, a.rot - o1);
            n2 = min(8, a.rot - o2);
        } else {
            o1 = 8 * item;
            o2 = pairs + o1;
            n1 = n2 = min(8, pairs - o1);
        }
    } else {
        o1 = a.rot + 16 * (item - pair_items);
        o2 = o1 + 8;
        n1 = min(8, a.d - o1);
        n2 = min(8, a.d - o2);
    }
    n1 = max(n1, 0);
    n2 = max(n2, 0);
    const int heads = a.heads[0] + a.heads[1];
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        if (pairs) {
            const double p = a.pos32 ? (double)((const int32_t*)a.pos)[t] : (double)((const int64_t*)a.pos)[t];
            if (t != blockIdx.x) __syncthreads();
            for (int i = threadIdx.x; i < pairs; i += blockDim.x) {
                const double turns = p * (double)a.freq[i] * 0.15915494309189533577;  // 1 / 2 pi
                float s, c;
                sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
                trig[i] = c;
                trig[pairs + i] = s;
            }
            __syncthreads();
        }
        for (int h = first; h < heads; h += step) {
            const int k = h >= a.heads[0], head = k ? h - a.heads[0] : h;
            const T* x = (const T*)(k ? a.x[1] : a.x[0]) + t * (k ? a.xt[1] : a.xt[0]) + head * (k ? a.xh[1] : a.xh[0]);
            T* y = (T*)(k ? a.y[1] : a.y[0]) + t * (k ? a.yt[1] : a.yt[0]) + head * (k ? a.yh[1] : a.yh[0]);
            const void* gain = k ? a.gain[1] : a.gain[0];
            f8 u = get8<kWhole>(x + (n1 ? o1 : 0), kWhole ? 8 : n1), v = get8<kWhole>(x + (n2 ? o2 : 0), kWhole ? 8 : n2);
            if (a.norm) {
                float s = 0.0f;
                if (!kWhole || n1)
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(u[e], u[e], fmaf(v[e], v[e], s));
                for (int w = 1; w < a.lanes; w *= 2) s += __shfl_xor(s, w);
                const float f = 1.0f / sqrtf(s / (float)a.d + a.eps);
                u *= f;
                v *= f;
                if (gain) {
                    f8 g1, g2;
                    if (a.gfloat) {
                        g1 = get8<kWhole>((const float*)gain + (n1 ? o1 : 0), kWhole ? 8 : n1);
                        g2 = get8<kWhole>((const float*)gain + (n2 ? o2 : 0), kWhole ? 8 : n2);
                    } else {
                        g1 = get8<kWhole>((const T*)gain + (n1 ? o1 : 0), kWhole ? 8 : n1);
                        g2 = get8<kWhole>((const T*)gain + (n2 ? o2 : 0), kWhole ? 8 : n2);
                    }
                    u *= g1;
                    v *= g2;
                }
            }
            if (turned) {
                const float* c = trig + 8 * item;
                const float* s = c + pairs;
                if (a.interleaved) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (kWhole || 2 * e < n1) {
                            const float p = u[2 * e], q = u[2 * e + 1];
                            u[2 * e] = p * c[e] - q * s[e];
                            u[2 * e + 1] = q * c[e] + p * s[e];
                        }
                        if (kWhole || 2 * e < n2) {
                            const float p = v[2 * e], q = v[2 * e + 1];
                            v[2 * e] = p * c[4 + e] - q * s[4 + e];
                            v[2 * e + 1] = q * c[4 + e] + p * s[4 + e];
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (kWhole || e < n1) {
                            const float p = u[e], q = v[e];
                            u[e] = p * c[e] - q * s[e];
                            v[e] = q * c[e] + p * s[e];
                        }
                }
            }
            if (n1) put8<kWhole>(y + o1, n1, u);
            if (n2) put8<kWhole>(y + o2, n2, v);
        }
    }
}

template <typename T>
void launch_type(const HeadArgs& a, int threads, unsigned grid, hipStream_t stream) {
    const size_t lds = sizeof(float) * 2 * (size_t)(a.rot / 2);
    const bool whole = a.rot % 16 == 0 && (a.d - a.rot) % 16 == 0;
    if (whole)
        hipLaunchKernelGGL((k_head_norm<T, true>), dim3(grid), dim3(threads), lds, stream, a);
    else
        hipLaunchKernelGGL((k_head_norm<T, false>), dim3(grid), dim3(threads), lds, stream, a);
}

}  // namespace

int launch_head_norm(const HeadRows& q, const HeadRows& k, int type, int64_t T, int64_t d, int gtype, float eps, int norm,
                     const void* pos, int pos32, const float* freq, int64_t rot, int interleaved, hipStream_t stream) {
    HeadArgs a;
    const HeadRows* rows[2] = {&q, &k};
    for (int i = 0; i < 2; ++i) {
        a.x[i] = rows[i]->x;
        a.y[i] = rows[i]->y;
        a.gain[i] = rows[i]->gain;
        a.heads[i] = (int)rows[i]->heads;
        a.xt[i] = rows[i]->xt;
        a.xh[i] = rows[i]->xh;
        a.yt[i] = rows[i]->yt;
        a.yh[i] = rows[i]->yh;
    }
    a.T = T;
    a.pos = pos;
    a.freq = freq;
    a.d = (int)d;
    a.rot = (int)rot;
    a.gfloat = gtype == BAKRON_F32;
    a.pos32 = pos32;
    a.interleaved = interleaved;
    a.norm = norm;
    a.eps = eps;
    const int items = (a.rot / 2 + 7) / 8 + (a.d - a.rot + 15) / 16;  // at most 33
    a.lanes = 1;
    while (a.lanes < items) a.lanes *= 2;
    const int64_t want = (int64_t)a.lanes * (a.heads[0] + a.heads[1]);
    const int threads = (int)std::min<int64_t>(512, (want + 63) / 64 * 64);
    const unsigned grid = (unsigned)std::min<int64_t>(T, (int64_t)1 << 22);
    if (type == BAKRON_F32) launch_type<float>(a, threads, grid, stream);
    else if (type == BAKRON_F16) launch_type<_Float16>(a, threads, grid, stream);
    else launch_type<__bf16>(a, threads, grid, stream);
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
