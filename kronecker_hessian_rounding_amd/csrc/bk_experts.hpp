// bk_experts.hpp -- the products of a mixture of rounded experts (included once for each type of x).
//
//   y_t = sum_j w_tj D_e (act(G_e x_t) * (U_e x_t)),  e = ids_tj,
// G_e, U_e (I x n) and D_e (n x I) packed as bk_matvec.hpp says, the experts of a matrix one behind the other.
//
// A pair is (token, slot); a leader is a pair whose expert no earlier slot of its token names, and it carries the
// weights of those that repeat it. The first product takes a row tile of G and the same one of U by tokens of one expert
// and leaves h = w act(g) u, a row for each leader.
//
// Few tokens (T <= 16, and at most 512 pairs): two launches, three where the second product is split. A workgroup of the
// first finds its expert's tokens in the ids by itself, and one more lists the experts that are named, with their tokens,
// for the second, in which a workgroup takes row tiles of all named experts' D: their columns follow each other as if they
// were one long layer's, so that its sums are y.
// More: a plan lists the leaders by expert, cut into tiles of tokens of one expert; the second product leaves w D h by
// leaders, and the sum over a token's leaders, in the order of its slots, is y.
// No result depends on the order within a list.
//
// Few tokens are bound by the codes' way from HBM: 16 tokens through all of 8 experts of 4096 x 14336 (4 bits, 0.74 GB with
// scales) take 179 us, 4.1 TB/s; one token through 6 experts of 2048 x 1408 (26 MB) 16.5 with the router's choice, most of
// it waits in a row (ids, codes, sums; the same again for the second product). By way of the plan that took 36. Many are bound
// by vector instructions (codes to operands, scaling) beside the matrix cores: see the kernels.
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
    char* planes;                 // h as bf16 pieces, largest first: [pair][piece][plane] bytes
    int64_t plane;
    float* part;                  // [pair][n]
    int64_t n, I;
    int act;
    int most_tiles;               // the list's bound
};

// Of few tokens: what a workgroup reads first of all, in as few lines as it takes (each is a miss).
struct FewArgs {
    const int32_t* ids;
    const float* weights;
    const char* gate;             // packed, of expert 0; of the second product its only layer
    const char* up;
    const char* x;
    const float* xs;
    int32_t* named;               // the experts that are named: how many, which, and [slot][16] pairs of their tokens or -1
    char* planes;                 // h as bf16 pieces: [pair][piece][plane] bytes
    int64_t stride, scale_offset; // bytes from expert to expert, and from a layer's codes to its scales
    int64_t ldx;
    int32_t T, k, E, slots;       // slots: experts, or pairs where they are fewer
    int32_t m, n, tiles, nc, ngp, gshift;
    int32_t plane, act;
    float* part;                  // [split][token][m] of the second product
};

__device__ __forceinline__ MvArgs layer_of(const FewArgs& e, const char* packed, int expert) {
    MvArgs a;
    a.codes = packed + expert * e.stride;
    a.scales = (const float*)(a.codes + e.scale_offset);
    a.x = e.x;
    a.xs = nullptr;
    a.y = nullptr;
    a.m = e.m;
    a.n = e.n;
    a.T = 0;
    a.ldx = e.ldx;
    a.ldy = 0;
    a.nc = e.nc;
    a.ngp = e.ngp;
    a.tiles = (uint32_t)e.tiles;
    a.gshift = e.gshift;
    a.ytype = 0;
    return a;
}

struct Listed {  // token t is row list[t]
    const int32_t* list;
    __device__ __forceinline__ int64_t operator()(int64_t t) const { return list[t]; }
};

__device__ __forceinline__ float activation(float v, int act) {
    // v sigmoid(v), or gelu's tanh form v sigmoid(2 z), z = sqrt(2 / pi) (v + 0.044715 v^3)
    const float z = act == BAKRON_ACT_SILU ? v : 1.5957691216057308f * fmaf(0.044715f * v * v, v, v);
    // (exponential and quotient of full fp32 accuracy: the hardware's exponential alone is off by some |z| steps)
    return v / (1.0f + expf(-z));
}

// h between the products: three bf16 pieces, the largest first, which hold all 24 bits of it (the first two are cut off, the
// last is rounded). An infinity or NaN stays in the first.
constexpr int kPieces = Mt<kH>::kPieces;
template <int N>
__device__ __forceinline__ void store_pieces(char* row, int64_t plane, int64_t i, const float (&h)[N]) {
    float r[N];
#pragma unroll
    for (int e = 0; e < N; ++e) r[e] = h[e];
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
        uint16_t b[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
            if (p == kPieces - 1) b[e] = __builtin_bit_cast(uint16_t, (__bf16)r[e]);
            else b[e] = (uint16_t)(__float_as_uint(__builtin_canonicalizef(r[e])) >> 16);
            const float left = r[e] - __uint_as_float((uint32_t)b[e] << 16);
            r[e] = left == left ? left : 0.0f;
        }
        __builtin_memcpy(__builtin_assume_aligned(row + p * plane + 2 * i, 2 * N), b, 2 * N);
    }
}

// ---------------------------------------------------------------- few tokens
constexpr int kFewTokens = 16, kFewPairs = 512;  // of the few tokens' path: what LDS holds of the map
inline bool few_tokens(int64_t T, int64_t k) { return T <= kFewTokens && T * k <= kFewPairs; }

// The named experts, by one workgroup, in the order of their numbers. Row `slot` of the map: the leader of each token that
// names the expert, or -1.
__device__ __forceinline__ void list_named(const FewArgs& e, char* lds) {
    constexpr int kWords = (int)(kMaxExperts / 32);
    const int pairs = e.T * e.k, threads = blockDim.x;
    int* id = reinterpret_cast<int*>(lds);                               // [pairs]
    uint32_t* some = reinterpret_cast<uint32_t*>(id + kFewPairs);        // a bit an expert
    int* before = reinterpret_cast<int*>(some + kWords);                 // experts of the words in front
    if (threadIdx.x < kWords) some[threadIdx.x] = 0;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const int x = e.ids[p];
        const bool named = x >= 0 && x < e.E;
        id[p] = named ? x : -1;
        if (named) atomicOr(&some[x >> 5], 1u << (x & 31));
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        const int lane = threadIdx.x, mine = lane < kWords ? __popc(some[lane]) : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < kWords; d *= 2) {
            const int v = __shfl_up(upto, d);
            upto += lane >= d ? v : 0;
        }
        if (lane < kWords) before[lane] = upto - mine;
        if (lane == kWords - 1) e.named[0] = upto;
    }
    int32_t* map = e.named + 1 + e.slots;
    for (int i = threadIdx.x; i < e.slots * 16; i += threads) map[i] = -1;
    __syncthreads();  // (the map's own lines: written and then overwritten by this workgroup)
    const auto slot = [&](int x) { return before[x >> 5] + __popc(some[x >> 5] & ((1u << (x & 31)) - 1)); };
    for (int x = threadIdx.x; x < e.E; x += threads)
        if (some[x >> 5] >> (x & 31) & 1) e.named[1 + slot(x)] = x;
    for (int p = threadIdx.x; p < pairs; p += threads)
        if (id[p] >= 0) {
            bool leader = true;
            for (int i = p / e.k * e.k; i < p; ++i) leader = leader && id[i] != id[p];
            if (leader) map[slot(id[p]) * 16 + p / e.k] = p;
        }
}

// The first product: a row tile of G and of U for one expert's tokens. Ids come first, then codes, so that the codes' first
// chunks leave before the expert's tokens are worked out. 16 tokens, 8 experts of 4096 x 14336: 105 us for 0.5 GB
// (4.75 TB/s).
template <int MATH, int W, int FS, int PF, int TB, int NW, int kWords>  // kWords: words of 64 pairs at most
__global__ __launch_bounds__(64 * NW) void k_experts_first_few(FewArgs e) {
    extern __shared__ __align__(16) char lds[];
    if (blockIdx.x == gridDim.x - 1) return list_named(e, lds);
    const int tiles = e.plane / 32, lane = threadIdx.x & 63;  // with those that pad h
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = blockIdx.x / tiles;
    const int64_t tile = blockIdx.x % tiles;
    // lane p of word v holds pair 64 v + p: its id (-1: no expert) and weight
    const int pairs = e.T * e.k, words = (pairs + 63) / 64;
    int id[kWords];
    float wt[kWords];
#pragma unroll
    for (int v = 0; v < kWords; ++v) {
        id[v] = -1;
        wt[v] = 0.0f;
        if (v < words) {
            const int p = min(64 * v + lane, pairs - 1);
            id[v] = e.ids[p];
            wt[v] = e.weights[p];
            if (64 * v + lane >= pairs || id[v] >= e.E) id[v] = -1;
        }
    }
    // the expert: the slot itself, or the id of a pair that is the first to name it
    int expert = slot;
    if (e.slots < e.E) {
#pragma unroll
        for (int v = 0; v < kWords; ++v)
            if (v == slot >> 6) expert = __builtin_amdgcn_readlane(id[v], slot & 63);
        if (expert < 0) return;
    }
    // the weights' first chunks are on their way before the tokens are known
    MvArgs a = layer_of(e, e.gate, expert), b = layer_of(e, e.up, expert);
    Stream<W, FS, 2, PF> st(a, b, tile, lane);
#pragma unroll
    for (int p = 0; p < PF; ++p) st.fetch(p, wave + p * NW);
    uint64_t named[kWords + 1];
#pragma unroll
    for (int v = 0; v < kWords; ++v) {
        named[v] = v < words ? __ballot(id[v] == expert) : 0;
        if (e.slots < e.E && ((v < slot >> 6 && named[v]) ||
                              (v == slot >> 6 && (named[v] & (((uint64_t)1 << (slot & 63)) - 1)))))
            return;
    }
    named[kWords] = 0;
    // lane t < T: token t's leader and weight for this expert, from the k bits of its pairs
    int pair = -1;
    float weight = 0.0f;
    {
        const int at = lane * e.k;
        uint64_t lo = 0, hi = 0;
#pragma unroll
        for (int v = 0; v < kWords; ++v)
            if (v < words) {
                lo = at >> 6 == v ? named[v] : lo;
                hi = at >> 6 == v ? named[v + 1] : hi;
            }
        uint64_t bits = (at & 63 ? lo >> (at & 63) | hi << (64 - (at & 63)) : lo) & (~(uint64_t)0 >> (64 - e.k));
        if (lane >= e.T) bits = 0;
        if (bits) pair = at + __builtin_ctzll(bits);
        while (__ballot(bits != 0)) {  // once, but for an expert that comes twice in a row
            const int p = bits ? at + __builtin_ctzll(bits) : 0;
#pragma unroll
            for (int v = 0; v < kWords; ++v)
                if (v < words) {
                    const float x = __shfl(wt[v], p & 63);
                    weight += bits && p >> 6 == v ? x : 0.0f;
                }
            bits &= bits - 1;
        }
    }
    const uint32_t members = (uint32_t)__ballot(pair >= 0);
    const int count = __popc(members);
    if (count == 0) return;
    // lane c: the c-th of them
    int token = 0;
    {
        uint32_t m = members;
        for (int c = 0; c < count; ++c, m &= m - 1)
            if (lane == c) token = __builtin_ctz(m);
    }
    pair = __shfl(pair, token);
    weight = __shfl(weight, token);
    float xs = e.xs && lane < count ? e.xs[token] : 1.0f;
    const bool real = tile < e.tiles;
    if (real) {
        a.T = count;
        const auto rows = [&](int64_t t) { return (int64_t)__shfl(token, (int)t); };
        few_products<MATH, W, FS, 2, PF, TB, NW, true>(a, st, rows, lds);
    }
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i0 = 0; i0 < count * 16; i0 += 64 * NW) {
        const int i = i0 + threadIdx.x, t = i >> 4, r = i & 15;
        const int64_t row = tile * 16 + r;
        const int64_t to = __shfl(pair, t & 63);
        const float w = __shfl(weight, t & 63), s = unit<MATH, W>() * __shfl(xs, t & 63);
        if (i >= count * 16) continue;
        float h = 0.0f;
        if (row < e.m) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                g += red[((k * 2) * 16 + t) * 17 + r];
                u += red[((k * 2 + 1) * 16 + t) * 17 + r];
            }
            h = w * (activation(g * s, e.act) * (u * s));
        }
        const float hh[1] = {h};
        store_pieces<1>(e.planes + to * kPieces * e.plane, e.plane, row, hh);
    }
}

// The second product of few tokens. A workgroup takes R row tiles of every named expert's D; its waves (and with `splits`
// those of as many workgroups: `all` together, a power of two) share the chunks. Chunk c of expert i is wave (i nc + c) % all's, and
// a wave takes the experts in the order of their numbers, so that a token's sums do not depend on what other tokens name. (One token
// alone: slot in place of i, which spreads the chunks evenly.) Each wave stages h's pieces for its next PF chunks in LDS of its own,
// as few_products does x: a token that does not name the expert has zeros there. 16 tokens, 8 experts of 4096 x 14336: 76
// us for 0.25 GB, 3.3 TB/s (vector instructions 46 % of it, matrix cores 24 %); one token, 6 of 2048 x 1408: 6.5 us.
template <int PF, int TB>
struct SecondShape {
    static constexpr int NP = kPieces;
    static constexpr int kUnits = (TB * PF * NP * 16 + 63) / 64;  // 16-byte units of a lane in a set
    static constexpr int kPiece = PF * 256;                       // from piece to piece of a token
    static constexpr int kPitch = NP * kPiece + 16;               // from token to token: 4 banks
    static constexpr int kBytes = TB * kPitch;                    // of a wave
};

template <int W, int FS, int R, int PF, int TB, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_second_few(FewArgs e, int splits, void* y, int ytype, int64_t ldy) {
    using M = Mt<kH>;
    using Sh = SecondShape<PF, TB>;
    constexpr int NP = kPieces;
    using Wd = typename Share<W>::T;
    constexpr int kScales = kSteps / FS;
    extern __shared__ __align__(16) char lds[];
    const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int split = blockIdx.x % splits, wave = split * NW + w, all = splits * NW;
    const int64_t tile0 = (int64_t)(blockIdx.x / splits) * R;
    const int nc = e.nc;
    int16_t* map = reinterpret_cast<int16_t*>(lds + NW * Sh::kBytes);  // [slots + 1][TB], -1 behind the named ones
    int16_t* ids = map + (e.slots + 1) * TB;                           // [slots] of more than 64
    const int live = __builtin_amdgcn_readfirstlane(e.named[0]);
    int window = e.named[1 + min(lane, e.slots - 1)];  // lane: the expert of slot 64 i + lane, i that of the furthest chunk
    if (TB > 1 && e.slots > 64) {
        for (int i = threadIdx.x; i < e.slots; i += 64 * NW) ids[i] = (int16_t)e.named[1 + i];
        __syncthreads();
    }
    struct At {
        int slot, chunk, id;  // slot == live, chunk 0: behind the last
    };
    const auto enter = [&](At& p) __attribute__((always_inline)) {  // the wave's first chunk of a slot, if it has one
        p.id = __builtin_amdgcn_readlane(window, p.slot & 63);
        p.chunk = (int)(((uint32_t)wave - (uint32_t)p.id * (uint32_t)nc) & (uint32_t)(all - 1));
    };
    const auto settle = [&](At p) __attribute__((always_inline)) {
        if constexpr (TB == 1) {  // (at most 64 slots)
            while (p.chunk >= nc) {
                p.chunk -= nc;
                ++p.slot;
            }
            p.slot = min(p.slot, live);
            p.id = __builtin_amdgcn_readlane(window, min(p.slot, 63));
        } else {
            while (p.chunk >= nc && p.slot < live) {
                ++p.slot;
                if ((p.slot & 63) == 0) window = ids[min(p.slot + lane, e.slots - 1)];
                enter(p);
            }
            if (p.slot >= live) p.chunk = 0;
        }
        return p;
    };
    const auto ahead = [&](At p) __attribute__((always_inline)) {  // the wave's next chunk
        p.chunk += all;
        return settle(p);
    };
    At next[PF];
    {
        At p = {0, wave, 0};
        if (TB > 1) enter(p);
        next[0] = settle(p);
    }
#pragma unroll
    for (int p = 1; p < PF; ++p) next[p] = ahead(next[p - 1]);
    Wd d[PF][R];
    float s[PF][R][kScales];
    // (behind the named experts' last chunk: some expert's, and never used)
    const auto fetch = [&](int p) __attribute__((always_inline)) {
        const char* codes = e.gate + min(max(next[p].id, 0), e.E - 1) * e.stride;
        const float* scales = (const float*)(codes + e.scale_offset);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t tile = min(tile0 + r, (int64_t)e.tiles - 1);
            d[p][r] = (reinterpret_cast<const Wd*>(codes) + (tile * nc + next[p].chunk) * 64)[lane];
#pragma unroll
            for (int f = 0; f < kScales; ++f)
                s[p][r][f] = (scales + (tile * e.ngp + (((int64_t)next[p].chunk * kScales + f) >> e.gshift)) * 16)[lane & 15];
        }
    };
    const int32_t* from = e.named + 1 + e.slots;
#pragma unroll
    for (int p = 0; p < PF; ++p) fetch(p);
    for (int i = threadIdx.x; i < (e.slots + 1) * TB; i += 64 * NW) {
        const int pair = from[min(i / TB, e.slots - 1) * 16 + i % TB];
        map[i] = (int16_t)(i / TB < live ? pair : -1);
    }
    __syncthreads();
    float sum[R][4] = {};
    if (next[0].slot < live) {
        char* xs = lds + w * Sh::kBytes;
        u32x4 x[Sh::kUnits];
        // unit of this lane: 16 bytes `u` of a piece of a token's row in chunk p of the set. A buffer load past the buffer's end
        // reads nothing and gives zeros: those of the tokens that do not name the expert. (All of h is below 2^31 bytes.)
        const auto planes = __builtin_amdgcn_make_buffer_rsrc(e.planes, 0, NP * e.plane * e.T * e.k, 0x00027000);
        const auto load = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int i = 0; i < Sh::kUnits; ++i) {
                const int v = lane + 64 * i, u = v % 16, piece = v / 16 % NP, p = v / (16 * NP) % PF;
                const int token = min(v / (16 * NP * PF), TB - 1);
                At c = next[0];
#pragma unroll
                for (int k = 1; k < PF; ++k) {
                    c.slot = p == k ? next[k].slot : c.slot;
                    c.chunk = p == k ? next[k].chunk : c.chunk;
                }
                const int pair = map[c.slot * TB + token];
                const uint32_t at = (uint32_t)((pair * NP + piece) * e.plane + c.chunk * 256 + u * 16);
                x[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(planes, pair >= 0 ? at : 0x80000000u, 0, 0));
            }
        };
        load();
        const char* xl = xs + min(lane & 15, TB - 1) * Sh::kPitch + (lane >> 4) * 16;
        int after = 0;  // as in few_products: keeps a set's writes behind the reads of the set before
        while (next[0].slot < live) {
#pragma unroll
            for (int i = 0; i < Sh::kUnits; ++i) {
                const int v = lane + 64 * i, u = v % 16, piece = v / 16 % NP, p = v / (16 * NP) % PF, token = v / (16 * NP * PF);
                if (token < TB)
                    *reinterpret_cast<u32x4*>(xs + token * Sh::kPitch + piece * Sh::kPiece + p * 256 + u * 16 + after) = x[i];
            }
            wave_fence();
            At now[PF];
            {
                At p = next[PF - 1];
#pragma unroll
                for (int k = 0; k < PF; ++k) {
                    now[k] = next[k];
                    next[k] = p = ahead(p);
                }
            }
            load();
#pragma unroll
            for (int p = 0; p < PF; ++p) {
                // which of the lane's tokens name the expert: the others' sums stay, whatever its scales hold
                int16_t own[4] = {0, 0, 0, 0};
                if constexpr (TB >= 4)
                    __builtin_memcpy(own, __builtin_assume_aligned(map + now[p].slot * TB + min(4 * (lane >> 4), TB - 4), 8), 8);
                if (now[p].slot < live)
#pragma unroll
                    for (int f = 0; f < kScales; ++f) {
                        f32x4 acc[R] = {};
#pragma unroll
                        for (int j = 0; j < FS; ++j) {
                            bf16x8 v[NP];
#pragma unroll
                            for (int q = 0; q < NP; ++q) {  // the smallest piece first into the sum
                                v[q] = *reinterpret_cast<const bf16x8*>(xl + (NP - 1 - q) * Sh::kPiece + p * 256 + (f * FS + j) * 64);
                                asm("" : "+v"(after) : "v"(v[q]));
                            }
#pragma unroll
                            for (int r = 0; r < R; ++r) {
                                const bf16x8 b = weights<kBF16, W>(d[p][r], f * FS + j);
#pragma unroll
                                for (int q = 0; q < NP; ++q) acc[r] = M::mma(v[q], b, acc[r]);
                            }
                        }
#pragma unroll
                        for (int r = 0; r < R; ++r)
#pragma unroll
                            for (int v = 0; v < 4; ++v) sum[r][v] = own[v] >= 0 ? fmaf(s[p][r][f], acc[r][v], sum[r][v]) : sum[r][v];
                    }
                fetch(p);
            }
            if constexpr (PF == 1) asm volatile("" ::: "memory");  // or all loads move over the loop's edge, to their use
        }
    }
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);  // [wave][tile][token][16 rows + 1]
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[((w * R + r) * 16 + 4 * (lane >> 4) + v) * 17 + (lane & 15)] = sum[r][v];
    __syncthreads();
    for (int i = threadIdx.x; i < e.T * R * 16; i += 64 * NW) {
        const int t = i / (R * 16), r = i / 16 % R;
        const int64_t row = (tile0 + r) * 16 + (i & 15);
        if (row >= e.m) continue;
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) v += red[((k * R + r) * 16 + t) * 17 + (i & 15)];
        if (splits > 1) e.part[((int64_t)split * e.T + t) * e.m + row] = v;
        else store_elem(y, ytype, t * ldy + row, v);
    }
}

template <int MATH, int W, int FS, int TB>
void launch_first_tokens(const FewArgs& e, hipStream_t stream) {
    // 4 waves: 16 tokens, 8 experts of 4096 x 14336, 171 us for the call where 8 took 200 (a tile is short, and twice as
    // many fit side by side). Few tokens have registers for 64 bytes of codes ahead a lane; with more tokens x's pieces
    // have them.
    constexpr int NW = 4, PF = TB <= 4 ? 16 / W : 1;
    constexpr size_t red = sizeof(float) * NW * 2 * 16 * 17, list = sizeof(int) * (kFewPairs + kMaxExperts / 16);
    constexpr size_t lds = std::max<size_t>({(size_t)NW * FewShape<MATH, PF, TB>::kBytes, red, list});
    const unsigned grid = (unsigned)(e.slots * (e.plane / 32) + 1);
    if constexpr (TB > 1) {
        if (e.T * e.k > 64) {
            hipLaunchKernelGGL((k_experts_first_few<MATH, W, FS, PF, TB, NW, kFewPairs / 64>), dim3(grid), dim3(64 * NW), lds,
                               stream, e);
            return;
        }
    }
    hipLaunchKernelGGL((k_experts_first_few<MATH, W, FS, PF, TB, NW, 1>), dim3(grid), dim3(64 * NW), lds, stream, e);
}
template <int MATH, int W, int FS>
void launch_first_few(const FewArgs& e, hipStream_t stream) {
    if (e.T == 1) launch_first_tokens<MATH, W, FS, 1>(e, stream);
    else if (e.T <= 4) launch_first_tokens<MATH, W, FS, 4>(e, stream);
    else if (e.T <= 8) launch_first_tokens<MATH, W, FS, 8>(e, stream);
    else launch_first_tokens<MATH, W, FS, 16>(e, stream);
}
template <int MATH>
void launch_experts_first_few(const FewArgs& e, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_first_few<MATH, 4, 1>(e, stream);
        else launch_first_few<MATH, 4, 4>(e, stream);
    } else {
        if (fs == 1) launch_first_few<MATH, 2, 1>(e, stream);
        else launch_first_few<MATH, 2, 4>(e, stream);
    }
}

template <int W, int FS, int TB>
void launch_second_tokens(const FewArgs& e, int splits, int tiles, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    // Up to 4 tokens are waits in a row, which 16 waves shorten; above, LDS for h's pieces leaves 8, with one chunk ahead.
    constexpr int NW = TB <= 4 ? 16 : 8, PF = TB <= 4 ? 2 : 1;
    const auto launch = [&](auto r) {
        constexpr int R = decltype(r)::value;
        const size_t red = sizeof(float) * NW * R * 16 * 17;
        const size_t lds = std::max(red, (size_t)NW * SecondShape<PF, TB>::kBytes + sizeof(int16_t) * ((e.slots + 1) * TB + e.slots));
        hipLaunchKernelGGL((k_experts_second_few<W, FS, R, PF, TB, NW>), dim3((unsigned)((e.tiles + R - 1) / R * splits)),
                           dim3(64 * NW), lds, stream, e, splits, y, ytype, ldy);
    };
    if constexpr (TB > 4) {
        if (tiles == 4) return launch(std::integral_constant<int, 4>());
        if (tiles == 2) return launch(std::integral_constant<int, 2>());
    }
    launch(std::integral_constant<int, 1>());
}
template <int W, int FS>
void launch_second_few(const FewArgs& e, int splits, int tiles, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    if (e.T == 1) launch_second_tokens<W, FS, 1>(e, splits, tiles, y, ytype, ldy, stream);
    else if (e.T <= 4) launch_second_tokens<W, FS, 4>(e, splits, tiles, y, ytype, ldy, stream);
    else if (e.T <= 8) launch_second_tokens<W, FS, 8>(e, splits, tiles, y, ytype, ldy, stream);
    else launch_second_tokens<W, FS, 16>(e, splits, tiles, y, ytype, ldy, stream);
}

// ---------------------------------------------------------------- more tokens
// The list's tiles hold at most 16 tokens where an expert has about as few (few_products), else as many as a workgroup of
// mm_products takes.
constexpr int kListFew = 16, kListMany = 64;  // tokens of a list's tile

struct FirstTile {
    MvArgs a, b;
    ExpertTile l;
};
__device__ __forceinline__ FirstTile first_tile(const ExpertArgs& e, uint32_t li) {
    FirstTile f;
    f.l = e.list[li];
    f.a = f.b = e.first;
    f.a.codes += f.l.expert * e.first_stride;
    f.a.scales = (const float*)((const char*)f.a.scales + f.l.expert * e.first_stride);
    f.b.codes = e.up_codes + f.l.expert * e.first_stride;
    f.b.scales = (const float*)((const char*)e.up_scales + f.l.expert * e.first_stride);
    f.a.T = f.l.count;
    return f;
}
__device__ __forceinline__ MvArgs second_tile(const ExpertArgs& e, const ExpertTile& l) {
    MvArgs a = e.second;
    a.codes += l.expert * e.second_stride;
    a.scales = (const float*)((const char*)a.scales + l.expert * e.second_stride);
    a.T = l.count;
    return a;
}

template <int MATH, int W, int FS, int PF, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_first(ExpertArgs e) {
    extern __shared__ __align__(16) char lds[];
    const uint32_t tiles = (uint32_t)(e.plane / 32);  // with those that pad h
    const uint32_t li = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    if ((int)li >= *e.tiles_used) return;
    const FirstTile f = first_tile(e, li);
    if (tile < e.first.tiles)
        few_products<MATH, W, FS, 2, PF, 16, NW>(f.a, Stream<W, FS, 2, PF>(f.a, f.b, tile, threadIdx.x & 63),
                                                 Listed{e.tokens + f.l.begin}, lds);
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i = threadIdx.x; i < f.l.count * 16; i += 64 * NW) {
        const int t = i >> 4, r = i & 15, at = f.l.begin + t;
        const int64_t row = (int64_t)tile * 16 + r;
        float h[1] = {0.0f};
        if (row < e.I) {
            float g = 0.0f, u = 0.0f;
#pragma unroll
            for (int k = 0; k < NW; ++k) {
                g += red[((k * 2) * 16 + t) * 17 + r];
                u += red[((k * 2 + 1) * 16 + t) * 17 + r];
            }
            const float s = unit<MATH, W>() * (f.a.xs ? f.a.xs[e.tokens[at]] : 1.0f);
            h[0] = e.weights[at] * (activation(g * s, e.act) * (u * s));
        }
        store_pieces<1>(e.planes + (int64_t)e.pairs[at] * kPieces * e.plane, e.plane, row, h);
    }
}

template <int W, int FS, int R, int PF, int NW>
__global__ __launch_bounds__(64 * NW) void k_experts_second(ExpertArgs e) {
    extern __shared__ __align__(16) char lds[];
    const uint32_t blocks = (e.second.tiles + R - 1) / R;
    const uint32_t li = blockIdx.x / blocks;
    const int64_t tile0 = (int64_t)(blockIdx.x % blocks) * R;
    if ((int)li >= *e.tiles_used) return;
    const ExpertTile l = e.list[li];
    const MvArgs a = second_tile(e, l);
    few_products<kH, W, FS, R, PF, 16, NW>(a, Stream<W, FS, R, PF>(a, tile0, threadIdx.x & 63), Listed{e.pairs + l.begin}, lds);
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i = threadIdx.x; i < l.count * R * 16; i += 64 * NW) {
        const int t = i / (R * 16), r = i / 16 % R;
        const int64_t row = (tile0 + r) * 16 + (i & 15);
        if (row >= e.n) continue;
        float y = 0.0f;
#pragma unroll
        for (int k = 0; k < NW; ++k) y += red[((k * R + r) * 16 + t) * 17 + (i & 15)];
        e.part[(int64_t)e.pairs[l.begin + t] * e.n + row] = y;
    }
}

// 16 RW rows of G and of U (and so of h) by 16 NT tokens. int8, 512 tokens of 4 in 32 experts of 2048 x 1408: 50 us with 64
// rows by 64 tokens (0.47 PFLOP/s); with 128 rows 68, 32 rows 61, columns split over waves 67 to 79, 128 tokens 58 to 64.
// Vector instructions are busy 46 % of it, the matrix cores 13 %, with 1.8 waves a SIMD.
template <int MATH, int W, int FS, int NT, int KS, int RW, int CH>
__global__ __launch_bounds__(64 * KS * RW) __attribute__((amdgpu_waves_per_eu(2))) void k_experts_first_mm(ExpertArgs e) {
    constexpr int kThreads = 64 * KS * RW, kRows = 16 * RW, kPitch = 2 * kRows + 4;
    extern __shared__ __align__(16) char lds[];
    const uint32_t blocks = (uint32_t)((e.plane / 2 + kRows - 1) / kRows);
    const uint32_t li = blockIdx.x / blocks;
    const int64_t tile_b = (int64_t)(blockIdx.x % blocks) * RW;
    if ((int)li >= *e.tiles_used) return;
    const FirstTile f = first_tile(e, li);
    const auto stream = [&](int rg, int lane) __attribute__((always_inline)) {
        return Stream<W, FS, 2, 2>(f.a, f.b, tile_b + rg, lane);
    };
    const auto sink = [&](int n0, int toks, const float* red, int pass) __attribute__((always_inline)) {
        for (int i = threadIdx.x; i < toks * (kRows / 4); i += kThreads) {
            const int tok = i / (kRows / 4), r = i % (kRows / 4) * 4;
            const int t = 16 * n0 + tok, at = f.l.begin + t;
            const int64_t row = tile_b * 16 + r;
            if (t >= f.l.count || 2 * row >= e.plane) continue;
            f32x4 g = {}, u = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const float* p = red + (k * pass + tok) * kPitch + r / 16 * 32 + r % 16;
                g += *reinterpret_cast<const f32x4*>(p);
                u += *reinterpret_cast<const f32x4*>(p + 16);
            }
            const float s = unit<MATH, W>() * (f.a.xs ? f.a.xs[e.tokens[at]] : 1.0f), w = e.weights[at];
            float h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = row + k < e.I ? w * (activation(g[k] * s, e.act) * (u[k] * s)) : 0.0f;
            store_pieces<4>(e.planes + (int64_t)e.pairs[at] * kPieces * e.plane, e.plane, row, h);
        }
    };
    mm_products<MATH, W, FS, NT, 2, KS, RW, CH>(f.a, 0, Listed{e.tokens + f.l.begin}, stream, lds, sink);
}

// 16 R RW rows of D by 16 NT tokens. At the sizes above, int8 tokens: 110 us for the call with 128 rows by 32 tokens; 256 rows 116,
// 64 rows 137; 64 tokens by 128 rows 141, by 256 rows 124; 16 tokens by 128 rows 111; 64 rows a wave spill. Alone 62 us: vector
// instructions 38 %, matrix cores 30 %, 1.8 waves a SIMD.
template <int W, int FS, int NT, int R, int KS, int RW, int CH>
__global__ __launch_bounds__(64 * KS * RW) __attribute__((amdgpu_waves_per_eu(2))) void k_experts_second_mm(ExpertArgs e) {
    constexpr int kThreads = 64 * KS * RW, kRows = 16 * R * RW, kPitch = kRows + 4;
    extern __shared__ __align__(16) char lds[];
    const uint32_t blocks = (e.second.tiles + R * RW - 1) / (R * RW);
    constexpr uint32_t kParts = kListMany / (16 * NT);  // of a list's tile
    const uint32_t li = blockIdx.x / blocks / kParts;
    const int64_t tile_b = (int64_t)(blockIdx.x % blocks) * R * RW;
    const int t0 = (int)(blockIdx.x / blocks % kParts) * 16 * NT;
    if ((int)li >= *e.tiles_used) return;
    const ExpertTile l = e.list[li];
    if (t0 >= l.count) return;
    const MvArgs a = second_tile(e, l);
    const auto stream = [&](int rg, int lane) __attribute__((always_inline)) {
        return Stream<W, FS, R, 2>(a, tile_b + rg * R, lane);
    };
    const auto sink = [&](int n0, int toks, const float* red, int pass) __attribute__((always_inline)) {
        for (int i = threadIdx.x; i < toks * (kRows / 4); i += kThreads) {
            const int tok = i / (kRows / 4), r = i % (kRows / 4) * 4, t = t0 + 16 * n0 + tok;
            const int64_t row = tile_b * 16 + r;
            if (t >= l.count || row >= e.n) continue;
            f32x4 y = {};
#pragma unroll
            for (int k = 0; k < KS; ++k) y += *reinterpret_cast<const f32x4*>(red + (k * pass + tok) * kPitch + r);
            store4(e.part, BAKRON_F32, (int64_t)e.pairs[l.begin + t] * e.n + row, y, (int)min<int64_t>(4, e.n - row));
        }
    };
    mm_products<kH, W, FS, NT, R, KS, RW, CH>(a, t0, Listed{e.pairs + l.begin}, stream, lds, sink);
}

template <int MATH, int W, int FS>
void launch_first_shape(const ExpertArgs& e, int tile, hipStream_t stream) {
    if (tile == kListFew) {
        constexpr int NW = 4, PF = 1;
        constexpr size_t red = sizeof(float) * NW * 2 * 16 * 17;
        constexpr size_t lds = std::max<size_t>((size_t)NW * FewShape<MATH, PF, 16>::kBytes, red);
        hipLaunchKernelGGL((k_experts_first<MATH, W, FS, PF, NW>), dim3((unsigned)(e.plane / 32 * e.most_tiles)), dim3(64 * NW),
                           lds, stream, e);
    } else {
        constexpr int NT = kListMany / 16, KS = 1, RW = 4, CH = MATH == kI8 ? 2 : 1;
        constexpr size_t red = sizeof(float) * KS * 16 * (32 * RW + 4);
        constexpr size_t lds = std::max<size_t>(2 * (size_t)MmTile<MATH, NT, KS * CH>::kBytes, red);
        const int64_t blocks = (e.plane / 2 + 16 * RW - 1) / (16 * RW);
        hipLaunchKernelGGL((k_experts_first_mm<MATH, W, FS, NT, KS, RW, CH>), dim3((unsigned)(blocks * e.most_tiles)), dim3(64 * KS * RW), lds,
                           stream, e);
    }
}
template <int MATH>
void launch_experts_first(const ExpertArgs& e, int tile, int W, int fs, hipStream_t stream) {
    if (W == 4) {
        if (fs == 1) launch_first_shape<MATH, 4, 1>(e, tile, stream);
        else launch_first_shape<MATH, 4, 4>(e, tile, stream);
    } else {
        if (fs == 1) launch_first_shape<MATH, 2, 1>(e, tile, stream);
        else launch_first_shape<MATH, 2, 4>(e, tile, stream);
    }
}

template <int W, int FS>
void launch_second_shape(const ExpertArgs& e, int tile, hipStream_t stream) {
    if (tile == kListFew) {
        // Four row tiles a workgroup: each stages all three pieces of its tokens' h. Two waves where the grid gives a unit more
        // than the three workgroups of four waves that its LDS holds: 64 tokens of 6 in 64 experts 2048 x 1920 112 us for the call,
        // with four 117; 24 of 2 in 16, 4096 x 2816, 69 and 74; on the other side 32 of 2 in 8, 4096 x 14336, 226 and with four 187.
        // Eight where it does not give one to each: 24 of 2 in 8, 1024 x 4096, 30 and with four 34; on the other side 32 of 2 in
        // 8 by 4096 x 14336 again, 192.
        constexpr int PF = 1, R = 4;
        const unsigned blocks = (e.second.tiles + R - 1) / R * (unsigned)e.most_tiles;
        const auto launch = [&](auto waves) {
            constexpr int NW = decltype(waves)::value;
            constexpr size_t red = sizeof(float) * NW * R * 16 * 17;
            constexpr size_t lds = std::max<size_t>((size_t)NW * FewShape<kH, PF, 16>::kBytes, red);
            hipLaunchKernelGGL((k_experts_second<W, FS, R, PF, NW>), dim3(blocks), dim3(64 * NW), lds, stream, e);
        };
        const unsigned units = (unsigned)device_info().cus;
        if (blocks > 3 * units) launch(std::integral_constant<int, 2>());
        else if (blocks <= units) launch(std::integral_constant<int, 8>());
        else launch(std::integral_constant<int, 4>());
    } else {
        constexpr int NT = 2, R = 2, KS = 1, RW = 4, CH = 1;
        constexpr size_t red = sizeof(float) * KS * 16 * (16 * R * RW + 4);
        constexpr size_t lds = std::max<size_t>(2 * (size_t)MmTile<kH, NT, KS * CH>::kBytes, red);
        hipLaunchKernelGGL((k_experts_second_mm<W, FS, NT, R, KS, RW, CH>),
                           dim3((e.second.tiles + R * RW - 1) / (R * RW) * (unsigned)e.most_tiles * (kListMany / (16 * NT))),
                           dim3(64 * KS * RW), lds, stream, e);
    }
}

// in bk_experts_second.hip
void launch_experts_second(const ExpertArgs& e, int tile, int W, int fs, hipStream_t stream);
void launch_experts_second_few(const FewArgs& e, int W, int fs, int splits, int tiles, void* y, int ytype, int64_t ldy, hipStream_t stream);

}  // namespace bk
