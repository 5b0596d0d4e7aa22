// bk_lora.hip -- sizes and dispatch of the low-rank adapters (kernels in bk_lora.hpp).
#include "bk_lora.hpp"

namespace bk {

// compiled in bk_lora_*.hip, one file for each type of adapters
extern template void launch_lora_adapters<float>(const LoraArgs&, int, hipStream_t);
extern template void launch_lora_adapters<_Float16>(const LoraArgs&, int, hipStream_t);
extern template void launch_lora_adapters<__bf16>(const LoraArgs&, int, hipStream_t);

namespace {

// Tokens of one round of launches (a grid has fewer than 2^32 threads), and the parts of the columns that u is formed in:
// as many workgroups as compute units, and at most 16 parts, whose sums the second launch adds in their order.
constexpr int64_t kRound = (int64_t)1 << 16;
int most_splits(int64_t T) { return (int)std::max<int64_t>(1, std::min<int64_t>(16, 256 / ((T + kDownTokens - 1) / kDownTokens))); }

}  // namespace

size_t lora_workspace_bytes(int64_t T, int64_t r) {
    const int64_t t = std::min(T, kRound);
    return lora_few(t, r) ? 0 : sizeof(float) * most_splits(t) * t * ((r + 15) / 16 * 16);
}

int launch_lora(const void* x, int xtype, int64_t T, int64_t n, int64_t ldx, const float* xs, const void* A, const void* B,
                int wtype, int64_t R, int64_t r, int64_t m, const float* scales, const int32_t* ids, const void* base,
                int btype, int64_t ldb, void* y, int ytype, int64_t ldy, void* ws, hipStream_t stream) {
    LoraArgs a = {};
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
    const int64_t cus = device_info().cus;
    a.rp = (int)((r + 15) / 16 * 16);
    a.u = (float*)ws;
    for (int64_t t0 = 0; t0 < T; t0 += kRound) {
        a.T = std::min(kRound, T - t0);
        a.x = (const char*)x + t0 * ldx * xb;
        a.xs = xs ? xs + t0 : nullptr;
        a.ids = ids + t0;
        a.base = base ? (const char*)base + t0 * ldb * wide(btype) : nullptr;
        a.y = (char*)y + t0 * ldy * wide(ytype);
        int64_t ranges;
        if (lora_few(a.T, r)) {
            // Ranges of 512 rows at least (a turn of the 8 waves), and a workgroup a unit, since each range forms u again (64
            // tokens, rank 16, 4096 -> 14336: these 18 us, twice as many 25).
            const int64_t tiles = (a.T + 15) / 16;
            a.slots = (int)std::min<int64_t>({16, a.T, R + 1});
            ranges = std::max<int64_t>(1, std::min((m + 511) / 512, cus / (tiles * a.slots)));
            a.rows_each = ((m + ranges - 1) / ranges + 63) / 64 * 64;
            a.row_blocks = (int)((m + a.rows_each - 1) / a.rows_each);
        } else {
            // a wave of a split has a block of columns at least
            const int64_t blocks = n / (wtype == BAKRON_F32 ? 32 : 64);
            a.splits = (int)std::max<int64_t>(1, std::min<int64_t>(most_splits(a.T), blocks / kDownWaves));
            a.slots = (int)std::max<int64_t>(1, std::min<int64_t>({16, R, 4 * cus / ((a.T + kDownTokens - 1) / kDownTokens * a.splits)}));
            const int64_t whole = m / kUpRows * kUpRows;
            // Four workgroups a unit (4096 tokens, 14336 rows, rank 64, with two pieces a value: 66 us, with two workgroups 78, with
            // eight 68), of two row blocks at least, since each forms its tokens' operands (512 tokens: 27.6 us for both launches, with one row block 35).
            // Slots share a tile's adapters over workgroups where ranges alone leave units idle.
            ranges = std::max<int64_t>(1, std::min(4 * cus / ((a.T + kUpTokens - 1) / kUpTokens), whole / (2 * kUpRows)));
            a.rows_each = std::max<int64_t>(1, (whole / kUpRows + ranges - 1) / ranges) * kUpRows;
            a.row_blocks = (int)((whole + a.rows_each - 1) / a.rows_each) + (m > whole);
            const int64_t each = (a.T + kUpTokens - 1) / kUpTokens * a.row_blocks;
            a.up_slots = (int)std::max<int64_t>(1, std::min<int64_t>({16, R + 1, a.T, 2 * cus / each}));
        }
        if (wtype == BAKRON_F32) launch_lora_adapters<float>(a, xtype, stream);
        else if (wtype == BAKRON_F16) launch_lora_adapters<_Float16>(a, xtype, stream);
        else launch_lora_adapters<__bf16>(a, xtype, stream);
    }
    return hipGetLastError() == hipSuccess ? BAKRON_OK : BAKRON_E_DEVICE;
}

}  // namespace bk
