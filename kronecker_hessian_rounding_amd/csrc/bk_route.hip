// bk_route.hip -- a router's logits to the experts of each token and their weights.
//
//   softmax: score_e = exp(l_e - max) / sum over all experts, chosen by l_e
//   sigmoid: score_e = 1 / (1 + exp(-l_e)), chosen by score_e + bias_e
// The k largest are taken one after the other, the lowest index first among equals, which softmax's order
// decides on the logits themselves and sigmoid's on 64-bit scores: sigmoids crowd below 1, where 32 bits
// would make many of them equal.
//
// One wave a row, expert 64 i + lane in register i of a lane. Keys are integers whose order is that of the values (0 for
// what is never chosen). A round is a maximum over the wave, by DPP within rows of 16 lanes and by scalars over the four;
// the lane that owns it (the lowest index, where several do) looks for its next one.
// Bytes are few (8192 x 256 bf16 logits are 1 us of HBM); what a call takes is the chain of k rounds of
// dependent instructions, and with sigmoid the 64-bit exponentials, 4 a lane for 256 experts. 1 x 128, k = 8: 3.5 us of GPU
// time, 1.1 above an empty kernel; 8192 x 256 bf16, k = 8, sigmoid: 14.8 us. With shuffles through LDS and comparisons of
// (value, index) pairs in place of DPP and integers the same took 6.6 and 21.8.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "bk_common.hpp"
#include "bk_internal.hpp"
#include "bk_rows.hpp"

namespace bk {

namespace {

struct RouteArgs {
    const void* logits;
    const float* bias;
    int32_t* ids;
    float* weights;
    int64_t T, ldl;
    int type, E, k, renorm;
    float scale;
};

template <typename T>
__device__ __forceinline__ T wave_add(T v) {
#pragma unroll
    for (int w = 1; w < 64; w *= 2) v += __shfl_xor(v, w);
    return v;
}

template <int kCtrl>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
    return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, kCtrl, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    v = max_dpp<0xB1>(v);   // neighbours, pairs, half rows, rows
    v = max_dpp<0x4E>(v);
    v = max_dpp<0x141>(v);
    v = max_dpp<0x140>(v);
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    return max(max(a, b), max(c, d));
}

// Integers in the order of the values, both zeros alike; above 0 for every value but -infinity and NaN, which get 0.
__device__ __forceinline__ uint32_t order(float v) {
    const uint32_t b = __float_as_uint(v + 0.0f);
    return v > -INFINITY ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0;
}
__device__ __forceinline__ uint64_t order(double v) {
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);
    return v > -INFINITY ? b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000u) : 0;
}

template <int NV, bool kSigmoid>
__global__ __launch_bounds__(256) void k_route(RouteArgs a) {
    using Key = std::conditional_t<kSigmoid, uint64_t, uint32_t>;
    const int lane = threadIdx.x & 63;
    const int64_t waves = (int64_t)gridDim.x * 4;
    for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.T; t += waves) {
        Key key[NV];
        float l[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            l[i] = e < a.E ? load_elem(a.logits, a.type, t * a.ldl + e) : -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = 64 * i + lane;
            if constexpr (kSigmoid) {
                const double v = 1.0 / (1.0 + exp(-(double)l[i])) + (a.bias && e < a.E ? (double)a.bias[e] : 0.0);
                key[i] = l[i] > -INFINITY ? order(v) : 0;
            } else {
                key[i] = order(l[i]);
            }
        }
        // the lane's own best, the lowest index among equals
        Key best;
        int at;
        const auto look = [&]() __attribute__((always_inline)) {
            best = key[0];
            at = 0;
#pragma unroll
            for (int i = 1; i < NV; ++i)
                if (key[i] > best) {
                    best = key[i];
                    at = i;
                }
        };
        look();
        float mx = -INFINITY, chosen_l = 0.0f;
        int chosen = -1;
        for (int j = 0; j < a.k; ++j) {
            uint64_t owners;
            if constexpr (kSigmoid) {
                const uint32_t hi = wave_max((uint32_t)(best >> 32));
                if (hi == 0) break;  // nothing left to choose
                const bool top = (uint32_t)(best >> 32) == hi;
                owners = __ballot(top);
                if (owners & (owners - 1)) {
                    const uint32_t lo = wave_max(top ? (uint32_t)best : 0);
                    owners = __ballot(top && (uint32_t)best == lo);
                }
            } else {
                const uint32_t b = wave_max(best);
                if (b == 0) break;
                owners = __ballot(best == b);
            }
            // the lowest register, then the lowest lane
            int owner = __builtin_ctzll(owners), reg = __builtin_amdgcn_readlane(at, owner);
            for (owners &= owners - 1; owners; owners &= owners - 1) {
                const int o = __builtin_ctzll(owners), r = __builtin_amdgcn_readlane(at, o);
                owner = r < reg ? o : owner;
                reg = min(r, reg);
            }
            float v = 0.0f;
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (i == reg) {
                    v = l[i];
                    if (lane == owner) key[i] = 0;
                }
            v = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), owner));
            if (j == 0) mx = v;
            if (lane == j) {
                chosen = 64 * reg + owner;
                chosen_l = v;
            }
            if (lane == owner) look();
        }
        float w = 0.0f;
        if constexpr (kSigmoid) {
            double p = chosen >= 0 ? 1.0 / (1.0 + exp(-(double)chosen_l)) : 0.0;
            if (a.renorm) {
                const double s = wave_add(p);
                p = s > 0.0 ? p / s : 0.0;
            }
            w = (float)(p * (double)a.scale);  // the one rounding
        } else {
            // l - mx, 0 where both are infinite
            const auto term = [&](float v) { return v == mx ? 1.0f : expf(v - mx); };
            w = chosen >= 0 ? term(chosen_l) : 0.0f;
            float s;
            if (a.renorm) {
                s = w;
            } else {
                s = 0.0f;
#pragma unroll
                for (int i = 0; i < NV; ++i) s += l[i] > -INFINITY ? term(l[i]) : 0.0f;
            }
            s = wave_add(s);
            w = (s > 0.0f ? w / s : 0.0f) * a.scale;
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = chosen;
            a.weights[t * a.k + lane] = w;
        }
    }
}

template <int NV>
void launch_nv(const RouteArgs& a, int sigmoid, unsigned grid, hipStream_t stream) {
    if (sigmoid) hipLaunchKernelGGL((k_route<NV, true>), dim3(grid), dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_route<NV, false>), dim3(grid), dim3(256), 0, stream, a);
}

}  // namespace

int launch_route(const void* logits, int type, int64_t T, int64_t E, int64_t ldl, int64_t k, int sigmoid,
                 const float* bias, int renorm, float scale, int32_t* ids, float* weights, hipStream_t stream) {
    RouteArgs a;
    a.logits = logits;
    a.bias = bias;
    a.ids = ids;
    a.weights = weights;
    a.T = T;
    a.ldl = ldl;
    a.type = type;
    a.E = (int)E;
    a.k = (int)k;
    a.renorm = renorm;
    a.scale = scale;
    const unsigned grid = (unsigned)std::min<int64_t>((T + 3) / 4, (int64_t)1 << 22);
    if (E <= 64) launch_nv<1>(a, sigmoid, grid, stream);
    else if (E <= 128) launch_nv<2>(a, sigmoid, grid, stream);
    else if (E <= 256) launch_nv<4>(a, sigmoid, grid, stream);
    else if (E <= 512) launch_nv<8>(a, sigmoid, grid, stream);
    else launch_nv<16>(a, sigmoid, grid, stream);
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
