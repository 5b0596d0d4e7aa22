// bk_experts.hpp -- the products of a mixture of rounded experts (included once for each type of x).
//
//   y_t = sum_j w_tj D_e (act(G_e x_t) * (U_e x_t)),  e = ids_tj,
// G_e, U_e (I x n) and D_e (n x I) packed as bk_matvec.hpp says, the experts of a matrix one behind the other.
//
// A pair is (token, slot); a leader is a pair whose expert no earlier slot of its token names, and it carries the
// weights of those that repeat it. The plan lists the leaders by expert, cut into tiles of tokens of one expert.
// The first product takes a tile of G and the same one of U by a tile of tokens and leaves h = w act(g) u in fp32,
// a row for each leader; the second leaves w D h in fp32 by leaders, and the sum over a token's leaders, in the
// order of its slots, is y. No result depends on the order within a list.
#pragma once

#include "bk_matvec.hpp"

namespace bk {

struct ExpertTile {
    int32_t expert, begin, count, pad;
};

struct ExpertArgs {
    MvArgs first, second;         // of the first product (x) and the second (h); codes and scales of expert 0
    const char* up_codes;         // of U, the shape of G
    const float* up_scales;
    int64_t first_stride, second_stride;  // bytes from expert to expert
    // the plan
    const int32_t* tiles_used;
    const ExpertTile* list;
    const int32_t* tokens;        // of each leader, in the order of the list
    const int32_t* pairs;
    const float* weights;
    float* h;                     // [pair][ldh]
    int64_t ldh;
    float* part;                  // [pair][n]
    int64_t n, I;
    int act;
    int most_tiles;               // the list's bound
};

struct Listed {  // token t is row list[t]
    const int32_t* list;
    __device__ __forceinline__ int64_t operator()(int64_t t) const { return list[t]; }
};

__device__ __forceinline__ float activation(float v, int act) {
    // v sigmoid(v), or gelu's tanh form v sigmoid(2 z), z = sqrt(2 / pi) (v + 0.044715 v^3)
    const float z = act == BAKRON_ACT_SILU ? v : 1.5957691216057308f * fmaf(0.044715f * v * v, v, v);
    return v / (1.0f + expf(-z));
}

template <int MATH, int W, int FS, int PF, int TB, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_first(ExpertArgs e) {
    extern __shared__ __align__(16) char lds[];
    const uint32_t li = blockIdx.x / e.first.tiles, tile = blockIdx.x % e.first.tiles;
    if ((int)li >= *e.tiles_used) return;
    const ExpertTile l = e.list[li];
    MvArgs a = e.first, b = e.first;
    a.codes += l.expert * e.first_stride;
    a.scales = (const float*)((const char*)a.scales + l.expert * e.first_stride);
    b.codes = e.up_codes + l.expert * e.first_stride;
    b.scales = (const float*)((const char*)e.up_scales + l.expert * e.first_stride);
    a.T = l.count;
    few_products<MATH, W, FS, 2, PF, TB, NW>(a, Stream<W, FS, 2, PF>(a, b, tile, threadIdx.x & 63),
                                             Listed{e.tokens + l.begin}, lds);
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i = threadIdx.x; i < l.count * 16; i += 64 * NW) {
        const int t = i >> 4, r = i & 15;
        const int64_t row = (int64_t)tile * 16 + r;
        if (row >= e.I) continue;
        float g = 0.0f, u = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) {
            g += red[((k * 2) * 16 + t) * 17 + r];
            u += red[((k * 2 + 1) * 16 + t) * 17 + r];
        }
        const float s = unit<MATH, W>() * (a.xs ? a.xs[e.tokens[l.begin + t]] : 1.0f);
        g *= s;
        u *= s;
        e.h[(int64_t)e.pairs[l.begin + t] * e.ldh + row] = e.weights[l.begin + t] * (activation(g, e.act) * u);
    }
}

template <int MATH, int W, int FS, int R, int PF, int TB, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_second(ExpertArgs e) {
    extern __shared__ __align__(16) char lds[];
    const uint32_t blocks = (e.second.tiles + R - 1) / R;
    const uint32_t li = blockIdx.x / blocks;
    const int64_t tile0 = (int64_t)(blockIdx.x % blocks) * R;
    if ((int)li >= *e.tiles_used) return;
    const ExpertTile l = e.list[li];
    MvArgs a = e.second;
    a.codes += l.expert * e.second_stride;
    a.scales = (const float*)((const char*)a.scales + l.expert * e.second_stride);
    a.T = l.count;
    few_products<MATH, W, FS, R, PF, TB, NW>(a, Stream<W, FS, R, PF>(a, tile0, threadIdx.x & 63),
                                             Listed{e.pairs + l.begin}, lds);
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i = threadIdx.x; i < l.count * R * 16; i += 64 * NW) {
        const int t = i / (R * 16), r = i / 16 % R;
        const int64_t row = (tile0 + r) * 16 + (i & 15);
        if (row >= e.n) continue;
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) y += red[((k * R + r) * 16 + t) * 17 + (i & 15)];
        e.part[(int64_t)e.pairs[l.begin + t] * e.n + row] = y * unit<MATH, W>();
    }
}

constexpr int kExpertTokens = 16;  // tokens of a list's tile

template <int MATH, int W, int FS>
void launch_first_shape(const ExpertArgs& e, hipStream_t stream) {
    constexpr int NW = 8, TB = kExpertTokens, PF = MATH == kF32 ? 1 : 2;
    constexpr size_t red = sizeof(float) * NW * 2 * 16 * 17;
    constexpr size_t lds = std::max<size_t>((size_t)NW * FewShape<MATH, PF, TB>::kBytes, red);
    hipLaunchKernelGGL((k_experts_first<MATH, W, FS, PF, TB, NW>), dim3(e.first.tiles * (unsigned)e.most_tiles), dim3(64 * NW),
                       lds, stream, e);
}

template <int MATH>
void launch_experts_first(const ExpertArgs& e, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_first_shape<MATH, 4, 1>(e, stream);
        else launch_first_shape<MATH, 4, 4>(e, stream);
    } else {
        if (fs == 1) launch_first_shape<MATH, 2, 1>(e, stream);
        else launch_first_shape<MATH, 2, 4>(e, stream);
    }
}

template <int MATH, int W, int FS>
void launch_second_shape(const ExpertArgs& e, hipStream_t stream) {
    constexpr int NW = 8, TB = kExpertTokens, PF = MATH == kF32 ? 1 : 2, R = 2;
    constexpr size_t red = sizeof(float) * NW * R * 16 * 17;
    constexpr size_t lds = std::max<size_t>((size_t)NW * FewShape<MATH, PF, TB>::kBytes, red);
    hipLaunchKernelGGL((k_experts_second<MATH, W, FS, R, PF, TB, NW>),
                       dim3((e.second.tiles + R - 1) / R * (unsigned)e.most_tiles), dim3(64 * NW), lds, stream, e);
}

template <int MATH>
void launch_experts_second(const ExpertArgs& e, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_second_shape<MATH, 4, 1>(e, stream);
        else launch_second_shape<MATH, 4, 4>(e, stream);
    } else {
        if (fs == 1) launch_second_shape<MATH, 2, 1>(e, stream);
        else launch_second_shape<MATH, 2, 4>(e, stream);
    }
}

}  // namespace bk
