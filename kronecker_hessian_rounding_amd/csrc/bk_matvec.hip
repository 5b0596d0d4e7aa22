// bk_matvec.hip -- packing of a rounded layer and dispatch of its products (bk_matvec.hpp
// has the layout and the kernels).
#include "bk_matvec.hpp"

namespace bk {

// compiled in bk_matvec_*.hip, one file for each type of x
extern template void launch_products<kF32>(const MvArgs&, int, int, hipStream_t);
extern template void launch_products<kF16>(const MvArgs&, int, int, hipStream_t);
extern template void launch_products<kBF16>(const MvArgs&, int, int, hipStream_t);
extern template void launch_products<kI8>(const MvArgs&, int, int, hipStream_t);
extern template void launch_products<kF8>(const MvArgs&, int, int, hipStream_t);

namespace {

// ---------------------------------------------------------------- pack
// One thread per lane's share of a chunk: it gathers its 32 codes. Done once a layer; bound by the 8-byte pieces in
// which it reads its m n bytes (14336 x 4096 115 to 125 us, 0.7 TB/s).
template <int W>
__global__ __launch_bounds__(256) void k_pack(const uint8_t* __restrict__ codes, int64_t m, int64_t n,
                                              int64_t ldc, int top, int shift, int64_t nc, int64_t units,
                                              typename Share<W>::T* __restrict__ out) {
    const int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= units) return;
    const int lane = (int)(u & 63);
    const int64_t chunk = (u >> 6) % nc, tile = (u >> 6) / nc;
    const int64_t row = tile * kRowTile + (lane & 15);
    constexpr int kHalf = 1 << (W - 1);
    typename Share<W>::T d;
#pragma unroll
    for (int j = 0; j < W; ++j) {
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < 32 / W; ++e) {
            // W = 4: e is the column; W = 2: e >> 3 picks step a or b
            const int step = W == 4 ? j : 2 * j + (e >> 3);
            const int64_t col = chunk * kChunk + step * kStep + 8 * (lane >> 4) + (e & 7);
            // cut to the layer's own grid, then moved to the middle of the stored one
            const int c = row < m && col < n ? min((int)codes[row * ldc + col], top) + shift : kHalf;
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

}  // namespace

PackShape pack_shape(int64_t m, int64_t n, int bits, int64_t group) {
    PackShape p;
    p.W = bits <= 2 ? 2 : 4;
    p.tiles = (m + kRowTile - 1) / kRowTile;
    p.chunks = (n + kChunk - 1) / kChunk;
    p.groups = group ? (n + group - 1) / group : 1;
    p.groups_padded = group && group < kChunk ? p.chunks * (kChunk / group) : p.groups;
    p.scale_offset = (size_t)p.tiles * p.chunks * 256 * p.W;
    p.bytes = p.scale_offset + (size_t)p.tiles * p.groups_padded * kRowTile * sizeof(float);
    return p;
}

int launch_pack(const uint8_t* codes, int64_t m, int64_t n, int64_t ldc, int bits, const float* scales, int64_t lds,
                int64_t group, void* packed, hipStream_t stream) {
    const PackShape p = pack_shape(m, n, bits, group);
    const int64_t units = p.tiles * p.chunks * 64, total = p.tiles * p.groups_padded * kRowTile;
    const int top = (1 << bits) - 1, shift = ((1 << p.W) - (1 << bits)) / 2;
    const dim3 grid((unsigned)((units + 255) / 256)), sgrid((unsigned)((total + 255) / 256));
    if (p.W == 4)
        hipLaunchKernelGGL(k_pack<4>, grid, dim3(256), 0, stream, codes, m, n, ldc, top, shift, p.chunks, units,
                           (u32x4*)packed);
    else
        hipLaunchKernelGGL(k_pack<2>, grid, dim3(256), 0, stream, codes, m, n, ldc, top, shift, p.chunks, units,
                           (u32x2*)packed);
    hipLaunchKernelGGL(k_pack_scales, sgrid, dim3(256), 0, stream, scales, m, lds, p.groups, p.groups_padded, total,
                       (float*)((char*)packed + p.scale_offset));
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

int launch_matvec(const void* packed, int64_t m, int64_t n, int bits, int64_t group, const void* x, int xtype,
                  int64_t T, int64_t ldx, const float* xs, void* y, int ytype, int64_t ldy, hipStream_t stream) {
    const PackShape p = pack_shape(m, n, bits, group);
    MvArgs a;
    a.codes = (const char*)packed;
    a.scales = (const float*)((const char*)packed + p.scale_offset);
    a.m = m;
    a.n = n;
    a.ldx = ldx;
    a.ldy = ldy;
    a.tiles = (uint32_t)p.tiles;
    a.nc = p.chunks;
    a.ngp = p.groups_padded;
    a.ytype = ytype;
    // units of scaling: steps where groups are shorter than a chunk, else chunks
    const int fs = group && group < kChunk ? 1 : kSteps;
    a.gshift = 62;  // one group
    if (group) {
        a.gshift = 0;
        while (((int64_t)fs * kStep << a.gshift) < group) ++a.gshift;
    }
    // a grid has fewer than 2^32 threads: tokens by ranges, whole blocks of 128 (one range for anything usual; at most
    // 512 threads for 64 rows x 32 tokens, or 16 rows x 16)
    const int64_t most = std::max<int64_t>(16, ((int64_t)1 << 29) / p.tiles / 128 * 128);
    const int64_t xb = xtype == BAKRON_F32 ? 4 : xtype == BAKRON_I8 || xtype == BAKRON_E4M3 ? 1 : 2;
    for (int64_t t0 = 0; t0 < T; t0 += most) {
        a.x = (const char*)x + t0 * ldx * xb;
        a.xs = xs ? xs + t0 : nullptr;
        a.y = (char*)y + t0 * ldy * (ytype == BAKRON_F32 ? 4 : 2);
        a.T = std::min(most, T - t0);
        switch (xtype) {
            case BAKRON_F32: launch_products<kF32>(a, p.W, fs, stream); break;
            case BAKRON_F16: launch_products<kF16>(a, p.W, fs, stream); break;
            case BAKRON_BF16: launch_products<kBF16>(a, p.W, fs, stream); break;
            case BAKRON_I8: launch_products<kI8>(a, p.W, fs, stream); break;
            default: launch_products<kF8>(a, p.W, fs, stream); break;
        }
    }
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
