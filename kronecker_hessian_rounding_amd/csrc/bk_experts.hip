// bk_experts.hip -- plan, sum and dispatch of the experts' products (bk_experts.hpp has the rest).
#include "bk_experts.hpp"

namespace bk {

// compiled in bk_experts_*.hip, one file for each type of x
extern template void launch_experts_first<kF32>(const ExpertArgs&, int, int, int, hipStream_t);
extern template void launch_experts_first_few<kF32>(const FewArgs&, int, int, hipStream_t);
extern template void launch_experts_first<kF16>(const ExpertArgs&, int, int, int, hipStream_t);
extern template void launch_experts_first_few<kF16>(const FewArgs&, int, int, hipStream_t);
extern template void launch_experts_first<kBF16>(const ExpertArgs&, int, int, int, hipStream_t);
extern template void launch_experts_first_few<kBF16>(const FewArgs&, int, int, hipStream_t);
extern template void launch_experts_first<kI8>(const ExpertArgs&, int, int, int, hipStream_t);
extern template void launch_experts_first_few<kI8>(const FewArgs&, int, int, hipStream_t);
extern template void launch_experts_first<kF8>(const ExpertArgs&, int, int, int, hipStream_t);
extern template void launch_experts_first_few<kF8>(const FewArgs&, int, int, hipStream_t);

namespace {

// Whether pair p = t k + j leads: its id is an expert and no earlier slot of its token has it.
__device__ __forceinline__ bool leads(const int32_t* ids, int64_t p, int k, int E) {
    const int e = ids[p];
    if (e < 0 || e >= E) return false;
    for (int64_t i = p / k * k; i < p; ++i)
        if (ids[i] == e) return false;
    return true;
}

struct PlanArgs {
    const int32_t* ids;
    const float* weights;
    int64_t pairs;
    int k, E, tile;
    int32_t* tiles_used;
    ExpertTile* list;
    int32_t* tokens;
    int32_t* pair;
    float* weight;
};

// One workgroup: leaders counted by expert, the counts' running sums, then each leader to its place (the order
// within an expert's list is that in which they come, and nothing depends on it). Ids pass through LDS, read once (7 us for
// 2048 pairs, all of it latency).
constexpr int64_t kRoundPairs = 1 << 14;
__global__ __launch_bounds__(1024) void k_experts_plan(PlanArgs a) {
    __shared__ int16_t id[kRoundPairs];
    __shared__ int count[1024], next[1024], sums[2][16];
    const int e = threadIdx.x, lane = e & 63, wave = e >> 6, pairs = (int)a.pairs;
    count[e] = 0;
    for (int p = e; p < pairs; p += 1024) {
        const int x = a.ids[p];
        id[p] = (int16_t)(x >= 0 && x < a.E ? x : -1);
    }
    __syncthreads();
    const auto leader = [&](int p) {
        if (id[p] < 0) return false;
        for (int i = p / a.k * a.k; i < p; ++i)
            if (id[i] == id[p]) return false;
        return true;
    };
    for (int p = e; p < pairs; p += 1024)
        if (leader(p)) atomicAdd(&count[id[p]], 1);
    __syncthreads();
    const int mine = count[e], mine_tiles = (mine + a.tile - 1) / a.tile;
    int upto = mine, upto_tiles = mine_tiles;  // sums up to this expert
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int b = __shfl_up(upto, d), t = __shfl_up(upto_tiles, d);
        upto += lane >= d ? b : 0;
        upto_tiles += lane >= d ? t : 0;
    }
    if (lane == 63) {
        sums[0][wave] = upto;
        sums[1][wave] = upto_tiles;
    }
    __syncthreads();
    for (int i = 0; i < wave; ++i) {
        upto += sums[0][i];
        upto_tiles += sums[1][i];
    }
    const int first = upto - mine, first_tile = upto_tiles - mine_tiles;
    next[e] = first;
    for (int i = 0; i < mine_tiles; ++i)
        a.list[first_tile + i] = ExpertTile{e, first + i * a.tile, min(a.tile, mine - i * a.tile), 0};
    if (e == 1023) *a.tiles_used = upto_tiles;
    __syncthreads();
    for (int p = e; p < pairs; p += 1024)
        if (leader(p)) {
            const int at = atomicAdd(&next[id[p]], 1);
            float w = a.weights[p];
            for (int i = p + 1; i < (p / a.k + 1) * a.k; ++i)
                if (id[i] == id[p]) w += a.weights[i];
            a.tokens[at] = p / a.k;
            a.pair[at] = p;
            a.weight[at] = w;
        }
}

struct SumArgs {
    const int32_t* ids;
    const float* part;
    void* y;
    int64_t T, n, ldy;
    int k, E, ytype;
};

// y_t: the rows of a token's leaders, in the order of its slots. 4 columns a thread.
__global__ __launch_bounds__(256) void k_experts_sum(SumArgs a) {
    const int64_t per = (a.n + 1023) / 1024, t = blockIdx.x / per;
    const int64_t i = (blockIdx.x % per) * 1024 + threadIdx.x * 4;
    const int lane = threadIdx.x & 63;
    const uint64_t lead = __ballot(lane < a.k && leads(a.ids, t * a.k + min(lane, a.k - 1), a.k, a.E));
    if (i >= a.n) return;
    const int count = (int)min<int64_t>(4, a.n - i);
    f4 y = {};
    for (uint64_t m = lead; m; m &= m - 1) {
        const float* p = a.part + (t * a.k + __builtin_ctzll(m)) * a.n + i;
        f4 v = {};
        if (count == 4) __builtin_memcpy(&v, p, 16);
        else
            for (int e = 0; e < 4; ++e) v[e] = e < count ? p[e] : 0.0f;
        y += v;
    }
    store4(a.y, a.ytype, t * a.ldy + i, y, count);
}

// y of few tokens whose second product was split.
__global__ __launch_bounds__(256) void k_experts_splits(const float* part, int splits, int64_t T, int64_t n, void* y, int ytype,
                                                        int64_t ldy) {
    const int64_t per = (n + 1023) / 1024, t = blockIdx.x / per, i = (blockIdx.x % per) * 1024 + threadIdx.x * 4;
    if (i >= n) return;
    const int count = (int)min<int64_t>(4, n - i);
    f4 v = {};
    for (int s = 0; s < splits; ++s) {
        const float* p = part + (s * T + t) * n + i;
        f4 u = {};
        if (count == 4) __builtin_memcpy(&u, p, 16);
        else
            for (int e = 0; e < 4; ++e) u[e] = e < count ? p[e] : 0.0f;
        v += u;
    }
    store4(y, ytype, t * ldy + i, v, count);
}

// Grid of the few tokens' second product: workgroups that share the columns of a row block, and row tiles of a block. LDS holds one
// workgroup a unit, so there are at most as many as units where that is possible: first with four splits, which cost a
// launch for their sum, and few tiles, which cost h's way into LDS the more often. us of a call at 16 (8) tokens as chosen, and
// the next best of 1, 2, 4 splits by 1, 2, 4 tiles, 2 of 8 experts unless said:
//   1024 x 8192: 4 by 1 48 (36), 4 by 2 51 (40), 1 by 1 105 (71)       2048 x 5632: 4 by 2 46 (37), 4 by 4 53 (44), 1 by 1 81 (57)
//   4096 x 14336: 4 by 4 175 (139), 2 by 2 199 (152), 1 by 1 254       7168 x 2048, 4 of 64: 2 by 4 212 (137), 4 by 4 234, 1 by 1 324
//   16384 x 1024: 1 by 4 52 (47), 2 by 4 58 (53), 1 by 1 81 (53)       24576 x 1024: 1 by 4 98 (83), 2 by 4 97 (86)
// 2 to 4 tokens take one tile (their waves have no room for more): 4 tokens, 2048 x 1408, 6 of 64, 2 splits 38, 1 44, 4 45; 1024 x
// 3584, 2 of 16, 4 splits 20, 1 24; 4096 x 14336 none 144, 2 148. One token alone is waits in a row, which splits lengthen.
// With fewer than 64 chunks of columns there is too little for the launch to pay: 4096 x 2048, 2 of 4 (64 chunks), 4 by 4 23
// (21), 1 by 1 25 (21); 4096 x 1024, 2 of 4 (32), 4 by 4 18 (16), 1 by 1 17 (15).
struct SecondGrid {
    int splits, tiles;
};
constexpr int kMostSplits = 4;
SecondGrid second_grid(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) {
    const int64_t tiles = (n + kRowTile - 1) / kRowTile, chunks = (I + kChunk - 1) / kChunk * std::min(E, T * k);
    if (T == 1) return {1, 1};
    const int64_t units = device_info().cus;
    const int most = T <= 4 ? 1 : 4;
    for (int splits = chunks >= 64 ? kMostSplits : 1; splits >= 1; splits /= 2)
        for (int r = 1; r <= most; r *= 2)
            if ((tiles + r - 1) / r * splits <= units) return {splits, r};
    return {1, most};
}

// Tokens of one round of launches: the plan and the workspace hold 2^14 pairs at most, and a grid fewer than 2^32 threads.
int64_t round_tokens(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) {
    int64_t t = std::max<int64_t>(1, std::min(T, kRoundPairs / k));
    const int64_t tiles = (std::max(n, I) + kRowTile - 1) / kRowTile;
    while (t > 1 && (tiles + 8) * (std::min(E, t * k) + t * k / kListFew) * 256 >= (int64_t)1 << 32) t /= 2;
    return t;
}

// List tiles of 16 tokens up to this many of an expert on average, else of 64. us of a call in tiles of 16 and of 64 with 16, 24
// and 32 tokens an expert, bf16 tokens: 4 of 32 experts 2048 x 1408 66 86, 74 87, 91 95; 2 of 8, 1024 x 3584, 31 59, 40 60, 45
// 61; 2 of 8, 4096 x 14336, 266 335, 332 340, 434 346; 4 of 16, 7168 x 2048, 133 142, 170 154, 201 163. int8: the same borders (the
// third 244 284, 296 288, 393 295); fp32, whose pieces cost the wide tiles more: 4096 x 14336 412 745, 551 748, 708 752.
constexpr int kFewEach = 24;

struct Layout {
    size_t planes, part;
    size_t used, list, tokens, pair, weight;  // more tokens
    size_t named;                             // few
    size_t bytes;
    int64_t plane, most;
};
Layout layout(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) {
    const int64_t t = round_tokens(T, k, E, n, I), p = t * k;
    Layout l = {};
    l.plane = (I + kChunk - 1) / kChunk * kChunk * 2;
    l.most = std::min(E, p) + p / kListFew;
    size_t at = 0;
    const auto take = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    if (few_tokens(T, k)) {
        l.named = take(4 * (1 + 17 * std::min(E, T * k)));
        l.planes = take(kPieces * l.plane * T * k);
        if (T > 1) l.part = take(4 * kMostSplits * T * n);
        l.bytes = at;
        return l;
    }
    l.used = take(4);
    l.list = take(sizeof(ExpertTile) * l.most);
    l.tokens = take(4 * p);
    l.pair = take(4 * p);
    l.weight = take(4 * p);
    l.planes = take(kPieces * l.plane * p);
    l.part = take(4 * p * n);
    l.bytes = at;
    return l;
}

MvArgs layer_args(const void* packed, const PackShape& p, int64_t m, int64_t n, int64_t group, int* fs) {
    MvArgs a = {};
    a.codes = (const char*)packed;
    a.scales = (const float*)((const char*)packed + p.scale_offset);
    a.m = m;
    a.n = n;
    a.tiles = (uint32_t)p.tiles;
    a.nc = p.chunks;
    a.ngp = p.groups_padded;
    // units of scaling: steps where groups are shorter than a chunk, else chunks
    *fs = group && group < kChunk ? 1 : kSteps;
    a.gshift = 62;  // one group
    if (group) {
        a.gshift = 0;
        while (((int64_t)*fs * kStep << a.gshift) < group) ++a.gshift;
    }
    return a;
}

void launch_first(const ExpertArgs& e, int tile, int xtype, int W, int fs, hipStream_t stream) {
    switch (xtype) {
        case BAKRON_F32: launch_experts_first<kF32>(e, tile, W, fs, stream); break;
        case BAKRON_F16: launch_experts_first<kF16>(e, tile, W, fs, stream); break;
        case BAKRON_BF16: launch_experts_first<kBF16>(e, tile, W, fs, stream); break;
        case BAKRON_I8: launch_experts_first<kI8>(e, tile, W, fs, stream); break;
        default: launch_experts_first<kF8>(e, tile, W, fs, stream); break;
    }
}

}  // namespace

size_t experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) { return layout(T, k, E, n, I).bytes; }

int launch_experts(const void* gate, const void* up, int bits, int64_t group, const void* down, int dbits, int64_t dgroup,
                   int64_t E, int64_t n, int64_t I, const void* x, int xtype, int64_t T, int64_t ldx, const float* xs,
                   const int32_t* ids, const float* weights, int64_t k, int act, void* y, int ytype, int64_t ldy, void* ws,
                   hipStream_t stream) {
    const PackShape p1 = pack_shape(I, n, bits, group), p2 = pack_shape(n, I, dbits, dgroup);
    const Layout l = layout(T, k, E, n, I);
    char* w = (char*)ws;
    if (few_tokens(T, k)) {
        int fs;
        FewArgs f = {};
        f.ids = ids;
        f.weights = weights;
        f.xs = xs;
        f.named = (int32_t*)(w + l.named);
        f.planes = w + l.planes;
        f.plane = (int32_t)l.plane;
        f.part = (float*)(w + l.part);
        f.T = (int32_t)T;
        f.k = (int32_t)k;
        f.E = (int32_t)E;
        f.slots = (int32_t)std::min(E, T * k);
        f.act = act;
        const auto product = [&](const void* packed, const PackShape& p, int64_t m, int64_t cols, int64_t g) {
            const MvArgs a = layer_args(packed, p, m, cols, g, &fs);
            f.gate = a.codes;
            f.stride = (int64_t)p.bytes;
            f.scale_offset = (int64_t)p.scale_offset;
            f.m = (int32_t)m;
            f.n = (int32_t)cols;
            f.tiles = (int32_t)a.tiles;
            f.nc = (int32_t)a.nc;
            f.ngp = (int32_t)a.ngp;
            f.gshift = a.gshift;
        };
        product(gate, p1, I, n, group);
        f.up = (const char*)up;
        f.x = (const char*)x;
        f.ldx = ldx;
        switch (xtype) {
            case BAKRON_F32: launch_experts_first_few<kF32>(f, p1.W, fs, stream); break;
            case BAKRON_F16: launch_experts_first_few<kF16>(f, p1.W, fs, stream); break;
            case BAKRON_BF16: launch_experts_first_few<kBF16>(f, p1.W, fs, stream); break;
            case BAKRON_I8: launch_experts_first_few<kI8>(f, p1.W, fs, stream); break;
            default: launch_experts_first_few<kF8>(f, p1.W, fs, stream); break;
        }
        product(down, p2, n, I, dgroup);
        const SecondGrid grid = second_grid(T, k, E, n, I);
        launch_experts_second_few(f, p2.W, fs, grid.splits, grid.tiles, y, ytype, ldy, stream);
        if (grid.splits > 1)
            hipLaunchKernelGGL(k_experts_splits, dim3((unsigned)(T * ((n + 1023) / 1024))), dim3(256), 0, stream, f.part, grid.splits,
                               T, n, y, ytype, ldy);
        return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
    }
    ExpertArgs e = {};
    int fs1, fs2;
    e.first = layer_args(gate, p1, I, n, group, &fs1);
    e.second = layer_args(down, p2, n, I, dgroup, &fs2);
    e.up_codes = (const char*)up;
    e.up_scales = (const float*)((const char*)up + p1.scale_offset);
    e.first_stride = (int64_t)p1.bytes;
    e.second_stride = (int64_t)p2.bytes;
    e.tiles_used = (const int32_t*)(w + l.used);
    e.list = (const ExpertTile*)(w + l.list);
    e.tokens = (const int32_t*)(w + l.tokens);
    e.pairs = (const int32_t*)(w + l.pair);
    e.weights = (const float*)(w + l.weight);
    e.planes = w + l.planes;
    e.plane = l.plane;
    e.part = (float*)(w + l.part);
    e.n = n;
    e.I = I;
    e.act = act;
    e.first.ldx = ldx;
    e.second.x = e.planes;
    e.second.n = l.plane / 2;  // zeros behind I
    e.second.ldx = kPieces * l.plane / 2;
    const int64_t xb = xtype == BAKRON_F32 ? 4 : xtype == BAKRON_I8 || xtype == BAKRON_E4M3 ? 1 : 2;
    const int64_t round = round_tokens(T, k, E, n, I);
    for (int64_t t0 = 0; t0 < T; t0 += round) {
        const int64_t tokens = std::min(round, T - t0), pairs = tokens * k;
        e.first.x = (const char*)x + t0 * ldx * xb;
        e.first.xs = xs ? xs + t0 : nullptr;
        const int tile = pairs > kFewEach * std::min(E, pairs) ? kListMany : kListFew;
        e.most_tiles = (int)(std::min(E, pairs) + pairs / tile);
        PlanArgs p = {ids + t0 * k, weights + t0 * k, pairs, (int)k, (int)E, tile, (int32_t*)(w + l.used),
                      (ExpertTile*)(w + l.list), (int32_t*)(w + l.tokens), (int32_t*)(w + l.pair), (float*)(w + l.weight)};
        hipLaunchKernelGGL(k_experts_plan, dim3(1), dim3(1024), 0, stream, p);
        launch_first(e, tile, xtype, p1.W, fs1, stream);
        launch_experts_second(e, tile, p2.W, fs2, stream);
        SumArgs s = {ids + t0 * k, e.part, (char*)y + t0 * ldy * (ytype == BAKRON_F32 ? 4 : 2), tokens, n, ldy, (int)k, (int)E, ytype};
        hipLaunchKernelGGL(k_experts_sum, dim3((unsigned)(tokens * ((n + 1023) / 1024))), dim3(256), 0, stream, s);
    }
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
