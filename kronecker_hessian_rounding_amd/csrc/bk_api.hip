// bk_api.hip -- the extern "C" entry points of libbakron: argument validation on
// the host, workspace checks, then dispatch to the kernel drivers. Every check
// happens before anything is enqueued, so an invalid call enqueues no work.
#include <algorithm>
#include <mutex>

#include "bk_internal.hpp"

namespace {

bool bad_ld(int64_t ld, int64_t cols) { return ld < cols || ld <= 0; }

// The solve's workspace for callers that cannot allocate (bakron_solve_noalloc):
// one array per device, held from the moment the library is loaded on it. In
// host code `scratch` is only a stand-in for the symbol; its device address is
// taken once per device with hipGetSymbolAddress and used from then on.
__device__ __align__(256) unsigned char scratch[BAKRON_NOALLOC_SCRATCH_BYTES];

constexpr int kMaxDevices = 64;

// The device address of `scratch` on the current device, or nullptr.
void* scratch_address() {
    static std::mutex mu;
    static void* addr[kMaxDevices] = {};
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (addr[dev] == nullptr) {
        void* p = nullptr;
        if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

// Host-side checks of the solve's arguments (shared by both solve entry points).
int check_solve_args(const float* W, int64_t m, int64_t n, int64_t ldw, const float* L_O, int64_t ldlo,
                     const float* L_I, int64_t ldli, const bakron_quantizer* q, const uint8_t* codes,
                     int64_t ldc, const float* scales_out, const float* delta_out, int64_t ldd,
                     const float* D_O, const float* D_I, const double* loss_out) {
    if (!W || !q || !codes || !scales_out) return BAKRON_E_INVALID_ARG;
    if (m <= 0 || n <= 0 || bad_ld(ldw, n) || bad_ld(ldc, n)) return BAKRON_E_INVALID_ARG;
    if (m > (int64_t)1 << 30 || n > (int64_t)1 << 30) return BAKRON_E_INVALID_ARG;
    if (L_O && bad_ld(ldlo, m)) return BAKRON_E_INVALID_ARG;
    if (L_I && bad_ld(ldli, n)) return BAKRON_E_INVALID_ARG;
    if (delta_out && bad_ld(ldd, n)) return BAKRON_E_INVALID_ARG;
    if (q->bits < 1 || q->bits > 8) return BAKRON_E_INVALID_ARG;
    if (q->rounding != BAKRON_ROUND_NEAREST && q->rounding != BAKRON_ROUND_STOCHASTIC)
        return BAKRON_E_INVALID_ARG;
    if (loss_out && (!D_I || (!D_O && L_O))) return BAKRON_E_INVALID_ARG;
    return BAKRON_OK;
}

bk::SolveArgs solve_args(const float* W, int64_t m, int64_t n, int64_t ldw, const float* L_O, int64_t ldlo,
                         const float* L_I, int64_t ldli, const bakron_quantizer* q, uint8_t* codes,
                         int64_t ldc, float* scales_out, float* delta_out, int64_t ldd, const float* D_O,
                         const float* D_I, double* loss_out, int64_t* clamped_out, int32_t* info) {
    bk::SolveArgs a;
    a.W = W;
    a.m = m;
    a.n = n;
    a.ldw = ldw;
    a.LO = L_O;
    a.ldlo = ldlo;
    a.LI = L_I;
    a.ldli = ldli;
    a.bits = q->bits;
    a.stochastic = q->rounding == BAKRON_ROUND_STOCHASTIC;
    a.seed = q->seed;
    a.row_scale = q->row_scale;
    a.codes = codes;
    a.ldc = ldc;
    a.scales = scales_out;
    a.delta = delta_out;
    a.ldd = ldd;
    a.DO = D_O;
    a.DI = D_I;
    a.loss = loss_out;
    a.clamped = clamped_out;
    a.info = info;
    return a;
}

// --- token rows (serving) ---
size_t elem_size(int type) {
    switch (type) {
        case BAKRON_F32: return 4;
        case BAKRON_F16:
        case BAKRON_BF16: return 2;
        case BAKRON_I8:
        case BAKRON_E4M3: return 1;
        default: return 0;
    }
}
bool wide_type(int type) { return type == BAKRON_F32 || type == BAKRON_F16 || type == BAKRON_BF16; }

// rows of `width` bytes, `pitch` bytes apart (what passes 63 bits: 2^63 - 1, further than any address)
typedef __int128 wide_t;
struct Rows {
    const void* p;
    int64_t rows, width, pitch;
};
int64_t bytes_of(int64_t n, int64_t size) {
    int64_t b;
    return __builtin_mul_overflow(n, size, &b) ? INT64_MAX : b;
}
Rows rows_of(const void* p, int64_t rows, int64_t cols, int64_t ld, int type) {
    const int64_t e = (int64_t)elem_size(type);
    return {p, rows, bytes_of(cols, e), bytes_of(ld, e)};
}
template <typename I>
bool cross(const Rows& a, const Rows& b, I a0, I b0) {
    if (a0 + (I)(a.rows - 1) * a.pitch + a.width <= b0 || b0 + (I)(b.rows - 1) * b.pitch + b.width <= a0) return false;
    if (a.pitch != b.pitch) return true;
    const I d = b0 >= a0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;
    return d < a.width || d + b.width > a.pitch;
}
// Whether two arrays share a byte. Rows of one pitch may interleave (columns of one
// buffer); with different pitches, ranges that cross count as overlapping. b_at: bytes from b.p to where b is taken to lie.
// Where a last row's address could pass 64 bits, in 128.
bool overlap(const Rows& a, const Rows& b, wide_t b_at = 0) {
    if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0) return false;
    const uint64_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
    const uint64_t size = (uint64_t)(a.rows | a.width | a.pitch | b.rows | b.width | b.pitch);
    if (b_at == 0 && (size >> 31) == 0 && ((a0 | b0) >> 62) == 0) return cross<int64_t>(a, b, (int64_t)a0, (int64_t)b0);
    return cross<wide_t>(a, b, a0, b0 + b_at);
}
bool same_rows(const Rows& a, const Rows& b) { return a.p == b.p && a.pitch == b.pitch && a.width == b.width; }

constexpr int64_t kMaxDim = (int64_t)1 << 30;

// m below 2^26 and n below 2^28 (so 4 n fits 31 bits), and as many chunks and scales as one grid packs
bool bad_pack_shape(int64_t m, int64_t n, int32_t bits, int64_t group) {
    if (m <= 0 || n <= 0 || m >= (int64_t)1 << 26 || n >= (int64_t)1 << 28 || bits < 1 || bits > 4) return true;
    if (group != 0 && (group < 32 || group > kMaxDim || (group & (group - 1)) != 0)) return true;
    const bk::PackShape p = bk::pack_shape(m, n, bits, group);
    return p.tiles * p.chunks > (int64_t)1 << 25 || p.tiles * p.groups_padded > (int64_t)1 << 27;
}

// Heads of T tokens as rows: tokens that hold heads, or heads that hold tokens (see bakron_head_norm).
bool bad_heads(int64_t T, int64_t H, int64_t d, int64_t st, int64_t sh) {
    if ((H > 1 && sh < d) || (T > 1 && st < d)) return true;
    if (H <= 1 || T <= 1) return false;
    return st < (wide_t)(H - 1) * sh + d && sh < (wide_t)(T - 1) * st + d;
}
struct Heads {
    const void* p;
    int64_t T, H, d, st, sh;
    int type;
};
Rows rows_of_heads(const Heads& a) {
    const auto [p, T, H, d, st, sh, type] = a;
    if (H <= 1) return rows_of(p, T, d, T > 1 ? st : d, type);
    if (T <= 1) return rows_of(p, H, d, sh, type);
    const auto span = [d = d](int64_t n, int64_t stride) { return std::min<wide_t>((wide_t)(n - 1) * stride + d, INT64_MAX); };
    if (st >= sh) return rows_of(p, T, (int64_t)span(H, sh), st, type);
    return rows_of(p, H, (int64_t)span(T, st), sh, type);
}
// Whether two arrays of as many tokens share an element. Where their ranges of heads cross, heads of one stride may still lie
// between each other (queries and keys of one head side by side): a head of the one and the head k further of the other.
bool overlap(const Heads& a, const Heads& b) {
    if (!overlap(rows_of_heads(a), rows_of_heads(b))) return false;
    if ((a.T > 1 && a.st != b.st) || (a.H > 1 && b.H > 1 && a.sh != b.sh)) return true;
    const int64_t st = a.T > 1 ? a.st : a.d;
    const wide_t sh = (wide_t)(a.H > 1 ? a.sh : b.sh) * (wide_t)elem_size(a.type);
    const Rows x = rows_of(a.p, a.T, a.d, st, a.type), y = rows_of(b.p, b.T, b.d, st, b.type);
    for (int64_t k = 1 - a.H; k < b.H; ++k)
        if (overlap(x, y, k * sh)) return true;
    return false;
}

bool bad_experts(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) {
    return T < 0 || T > (int64_t)1 << 40 || k < 1 || k > bk::kMaxChosen || E < 1 || E > bk::kMaxExperts || n < 1 ||
           n > bk::kMaxExpertDim || I < 1 || I > bk::kMaxExpertDim;
}

}  // namespace

extern "C" {

int bakron_abi_version(void) { return BAKRON_ABI_VERSION; }

const char* bakron_status_str(int status) {
    switch (status) {
        case BAKRON_OK: return "ok";
        case BAKRON_E_INVALID_ARG: return "invalid argument";
        case BAKRON_E_NOT_SPD: return "matrix is not positive definite";
        case BAKRON_E_WORKSPACE: return "workspace missing or too small";
        case BAKRON_E_DEVICE: return "HIP runtime or kernel launch failure";
        default: return "unknown status";
    }
}

size_t bakron_hessian_accum_workspace_bytes(int64_t T, int64_t d) {
    if (d <= 0 || T < 0) return 0;
    return bk::hessian_workspace_bytes(T, d);
}

int bakron_hessian_accum(const float* X, int64_t T, int64_t d, int64_t ldx, float alpha,
                         float beta, float* H, int64_t ldh, void* ws, size_t ws_bytes,
                         void* stream) {
    if (!H || d <= 0 || T < 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    if (T > 0 && (!X || bad_ld(ldx, d))) return BAKRON_E_INVALID_ARG;
    return bk::launch_hessian_accum(X, T, d, ldx, alpha, beta, H, ldh, ws, ws_bytes,
                                    (hipStream_t)stream);
}

int bakron_hessian_accum_t(const float* X, int64_t T, int64_t d, int64_t ldx, float alpha,
                           float beta, float* H, int64_t ldh, void* ws, size_t ws_bytes,
                           void* stream) {
    if (!H || d <= 0 || T < 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    if (T > 0 && (!X || bad_ld(ldx, T))) return BAKRON_E_INVALID_ARG;
    if (!ws || ws_bytes < bk::hessian_workspace_bytes(T, d)) return BAKRON_E_WORKSPACE;
    return bk::launch_hessian_accum(X, T, d, ldx, alpha, beta, H, ldh, ws, ws_bytes,
                                    (hipStream_t)stream, true);
}

int bakron_hessian_accum_tb(const float* X, int64_t S, int64_t d, int64_t tin, int64_t ldx, int64_t bs,
                            float alpha, float beta, float* H, int64_t ldh, void* ws, size_t ws_bytes,
                            void* stream) {
    if (!H || d <= 0 || S < 0 || tin < 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    const int64_t T = S * tin;
    if (T > 0 && (!X || bad_ld(ldx, tin) || (S > 1 && bs < d * ldx))) return BAKRON_E_INVALID_ARG;
    if (!ws || ws_bytes < bk::hessian_workspace_bytes(T, d)) return BAKRON_E_WORKSPACE;
    return bk::launch_hessian_accum(X, T, d, ldx, alpha, beta, H, ldh, ws, ws_bytes, (hipStream_t)stream,
                                    true, nullptr, tin, bs);
}

int bakron_hessian_accum_w(const float* X, int64_t T, int64_t d, int64_t ldx, const float* w, float alpha,
                           float beta, float* H, int64_t ldh, void* ws, size_t ws_bytes, void* stream) {
    if (!H || d <= 0 || T < 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    if (T > 0 && (!X || !w || bad_ld(ldx, d))) return BAKRON_E_INVALID_ARG;
    if (!ws || ws_bytes < bk::hessian_workspace_bytes(T, d)) return BAKRON_E_WORKSPACE;
    return bk::launch_hessian_accum(X, T, d, ldx, alpha, beta, H, ldh, ws, ws_bytes, (hipStream_t)stream,
                                    false, w);
}

size_t bakron_token_weights_workspace_bytes(int64_t T, int64_t d) {
    if (d <= 0 || T < 0) return 0;
    return bk::token_weights_workspace_bytes(T, d);
}

int bakron_token_weights(const float* Y, int64_t T, int64_t d, int64_t ldy, const float* H, int64_t ldh,
                         float* w, void* ws, size_t ws_bytes, void* stream) {
    if (d <= 0 || T < 0 || (T > 0 && (!Y || !w || bad_ld(ldy, d))) || (H && bad_ld(ldh, d)))
        return BAKRON_E_INVALID_ARG;
    return bk::launch_token_weights(Y, T, d, ldy, H, ldh, w, ws, ws_bytes, (hipStream_t)stream);
}

size_t bakron_ldl_workspace_bytes(int64_t d) {
    if (d <= 0) return 0;
    return bk::ldl_workspace_bytes(d);
}

int bakron_ldl(float* H, int64_t d, int64_t ldh, double damp_rel, float* D, int64_t* bad_pivot,
               void* ws, size_t ws_bytes, void* stream) {
    if (bad_pivot) *bad_pivot = -1;
    if (!H || d <= 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    if (!(damp_rel >= 0.0) || !(damp_rel < INFINITY)) return BAKRON_E_INVALID_ARG;
    if (!ws || ws_bytes < bk::ldl_workspace_bytes(d)) return BAKRON_E_WORKSPACE;
    return bk::run_ldl(H, d, ldh, damp_rel, D, bad_pivot, ws, (hipStream_t)stream);
}

int bakron_ldl_async(float* H, int64_t d, int64_t ldh, double damp_rel, float* D,
                     int64_t* bad_pivot_dev, void* ws, size_t ws_bytes, void* stream) {
    if (!H || !bad_pivot_dev || d <= 0 || bad_ld(ldh, d)) return BAKRON_E_INVALID_ARG;
    if (!(damp_rel >= 0.0) || !(damp_rel < INFINITY)) return BAKRON_E_INVALID_ARG;
    if (!ws || ws_bytes < bk::ldl_workspace_bytes(d)) return BAKRON_E_WORKSPACE;
    return bk::enqueue_ldl(H, d, ldh, damp_rel, D, ws, (hipStream_t)stream, bad_pivot_dev);
}

int bakron_ldl_pair_async(float* HA, int64_t dA, int64_t ldha, float* DA, int64_t* bad_pivot_dev_A,
                          void* wsA, size_t wsA_bytes, float* HB, int64_t dB, int64_t ldhb, float* DB,
                          int64_t* bad_pivot_dev_B, void* wsB, size_t wsB_bytes, double damp_rel,
                          void* stream_a, void* stream_b) {
    if (!HA || !bad_pivot_dev_A || dA <= 0 || bad_ld(ldha, dA)) return BAKRON_E_INVALID_ARG;
    if (!HB || !bad_pivot_dev_B || dB <= 0 || bad_ld(ldhb, dB)) return BAKRON_E_INVALID_ARG;
    if (!(damp_rel >= 0.0) || !(damp_rel < INFINITY)) return BAKRON_E_INVALID_ARG;
    if (!wsA || wsA_bytes < bk::ldl_workspace_bytes(dA)) return BAKRON_E_WORKSPACE;
    if (!wsB || wsB_bytes < bk::ldl_workspace_bytes(dB)) return BAKRON_E_WORKSPACE;
    return bk::enqueue_ldl_pair(HA, dA, ldha, DA, wsA, bad_pivot_dev_A, HB, dB, ldhb, DB, wsB, bad_pivot_dev_B,
                                damp_rel, (hipStream_t)stream_a, (hipStream_t)stream_b);
}

size_t bakron_solve_workspace_bytes(int64_t m, int64_t n) {
    if (m <= 0 || n <= 0) return 0;
    return bk::solve_workspace_bytes(m, n);
}

int bakron_solve(const float* W, int64_t m, int64_t n, int64_t ldw, const float* L_O, int64_t ldlo,
                 const float* L_I, int64_t ldli, const bakron_quantizer* q, uint8_t* codes,
                 int64_t ldc, float* scales_out, float* delta_out, int64_t ldd, const float* D_O,
                 const float* D_I, double* loss_out, int64_t* clamped_out, int32_t* info,
                 void* ws, size_t ws_bytes, void* stream) {
    const int st = check_solve_args(W, m, n, ldw, L_O, ldlo, L_I, ldli, q, codes, ldc, scales_out, delta_out,
                                    ldd, D_O, D_I, loss_out);
    if (st != BAKRON_OK) return st;
    if (!ws || ws_bytes < bk::solve_workspace_bytes(m, n)) return BAKRON_E_WORKSPACE;
    return bk::run_solve(solve_args(W, m, n, ldw, L_O, ldlo, L_I, ldli, q, codes, ldc, scales_out, delta_out, ldd,
                                    D_O, D_I, loss_out, clamped_out, info),
                         ws, (hipStream_t)stream);
}

int bakron_solve_noalloc(const float* W, int64_t m, int64_t n, int64_t ldw, const float* L_O, int64_t ldlo,
                         const float* L_I, int64_t ldli, const bakron_quantizer* q, uint8_t* codes,
                         int64_t ldc, float* scales_out, float* delta_out, int64_t ldd, const float* D_O,
                         const float* D_I, double* loss_out, int64_t* clamped_out, int32_t* info,
                         void* stream) {
    const int st = check_solve_args(W, m, n, ldw, L_O, ldlo, L_I, ldli, q, codes, ldc, scales_out, delta_out,
                                    ldd, D_O, D_I, loss_out);
    if (st != BAKRON_OK) return st;
    if (bk::solve_workspace_bytes(m, n) > BAKRON_NOALLOC_SCRATCH_BYTES) return BAKRON_E_WORKSPACE;
    void* ws = scratch_address();
    if (ws == nullptr) return BAKRON_E_DEVICE;
    return bk::run_solve(solve_args(W, m, n, ldw, L_O, ldlo, L_I, ldli, q, codes, ldc, scales_out, delta_out, ldd,
                                    D_O, D_I, loss_out, clamped_out, info),
                         ws, (hipStream_t)stream);
}

int bakron_layer_report(int64_t m, int64_t n, const float* D_O, const float* D_I, const float* scales,
                        const float* H_I, int64_t ldhi, const float* H_O, int64_t ldho, double* out,
                        void* stream) {
    if (m <= 0 || n <= 0 || !D_I || !scales || !out) return BAKRON_E_INVALID_ARG;
    if ((H_I && bad_ld(ldhi, n)) || (H_O && bad_ld(ldho, m))) return BAKRON_E_INVALID_ARG;
    return bk::launch_layer_report(m, n, D_O, D_I, scales, H_I, ldhi, H_O, ldho, out, (hipStream_t)stream);
}

int bakron_rht(float* A, int64_t rows, int64_t cols, int64_t lda, int axis, uint64_t seed, int transpose,
               void* stream) {
    if (!A || rows <= 0 || cols <= 0 || bad_ld(lda, cols) || (axis != 0 && axis != 1))
        return BAKRON_E_INVALID_ARG;
    if (axis == 1 && (cols & -cols) > 16384) return BAKRON_E_INVALID_ARG;
    return bk::launch_rht(A, rows, cols, lda, axis, seed, transpose, (hipStream_t)stream);
}

size_t bakron_packed_bytes(int64_t m, int64_t n, int32_t bits, int64_t group) {
    if (bad_pack_shape(m, n, bits, group)) return 0;
    return bk::pack_shape(m, n, bits, group).bytes;
}

int bakron_pack(const uint8_t* codes, int64_t m, int64_t n, int64_t ldc, int32_t bits, const float* scales,
                int64_t lds, int64_t group, void* packed, size_t packed_bytes, void* stream) {
    if (!codes || !scales || !packed || bad_pack_shape(m, n, bits, group) || bad_ld(ldc, n))
        return BAKRON_E_INVALID_ARG;
    const bk::PackShape p = bk::pack_shape(m, n, bits, group);
    if (bad_ld(lds, p.groups) || ((uintptr_t)packed & 15) != 0) return BAKRON_E_INVALID_ARG;
    const Rows out = {packed, 1, (int64_t)p.bytes, (int64_t)p.bytes};
    if (overlap(rows_of(codes, m, n, ldc, BAKRON_I8), out) || overlap(rows_of(scales, m, p.groups, lds, BAKRON_F32), out))
        return BAKRON_E_INVALID_ARG;
    if (packed_bytes < p.bytes) return BAKRON_E_WORKSPACE;
    return bk::launch_pack(codes, m, n, ldc, bits, scales, lds, group, packed, (hipStream_t)stream);
}

int bakron_matvec(const void* packed, size_t packed_bytes, int64_t m, int64_t n, int32_t bits, int64_t group,
                  const void* X, int32_t xtype, int64_t T, int64_t ldx, const float* xscale, void* Y, int32_t ytype,
                  int64_t ldy, void* stream) {
    if (!packed || ((uintptr_t)packed & 15) != 0 || bad_pack_shape(m, n, bits, group) || T < 0)
        return BAKRON_E_INVALID_ARG;
    if (elem_size(xtype) == 0 || !wide_type(ytype)) return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    if (!X || !Y || bad_ld(ldx, n) || bad_ld(ldy, m)) return BAKRON_E_INVALID_ARG;
    if (T > (int64_t)1 << 40) return BAKRON_E_INVALID_ARG;
    const Rows y = rows_of(Y, T, m, ldy, ytype);
    const Rows w = {packed, 1, (int64_t)packed_bytes, (int64_t)packed_bytes};
    const Rows xs = {xscale, 1, 4 * T, 4 * T};
    if (overlap(rows_of(X, T, n, ldx, xtype), y) || overlap(w, y) || overlap(xs, y)) return BAKRON_E_INVALID_ARG;
    if (packed_bytes < bk::pack_shape(m, n, bits, group).bytes) return BAKRON_E_WORKSPACE;
    return bk::launch_matvec(packed, m, n, bits, group, X, xtype, T, ldx, xscale, Y, ytype, ldy, (hipStream_t)stream);
}

int bakron_rmsnorm(const void* X, int32_t xtype, int64_t T, int64_t n, int64_t ldx, const void* R, int64_t ldr,
                   void* H, int64_t ldh, const void* gain, int32_t gtype, float eps, int rotate, uint64_t seed,
                   void* Y, int32_t ytype, int64_t ldy, float* yscale, void* stream) {
    if (n <= 0 || n > kMaxDim || T < 0 || T > 0x7fffffff || !wide_type(xtype) || elem_size(ytype) == 0)
        return BAKRON_E_INVALID_ARG;
    if (gain && gtype != xtype && gtype != BAKRON_F32) return BAKRON_E_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps < INFINITY) || (rotate && n > bk::kNormMaxBuffered)) return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    const bool coded = !wide_type(ytype);
    if (!X || !Y || (coded && !yscale)) return BAKRON_E_INVALID_ARG;
    if (bad_ld(ldx, n) || bad_ld(ldy, n) || (R && bad_ld(ldr, n)) || (H && bad_ld(ldh, n)))
        return BAKRON_E_INVALID_ARG;
    const Rows x = rows_of(X, T, n, ldx, xtype), r = rows_of(R, T, n, ldr, xtype), h = rows_of(H, T, n, ldh, xtype);
    const Rows y = rows_of(Y, T, n, ldy, ytype), s = {coded ? yscale : nullptr, 1, 4 * T, 4 * T};
    const Rows g = rows_of(gain, 1, n, n, gtype);
    const auto clash = [&](const Rows& in, const Rows& out, int in_type, int out_type) {
        return overlap(in, out) && !(same_rows(in, out) && in_type == out_type);
    };
    if (clash(x, h, xtype, xtype) || clash(r, h, xtype, xtype) || clash(x, y, xtype, ytype) ||
        clash(r, y, xtype, ytype))
        return BAKRON_E_INVALID_ARG;
    if (overlap(h, y) || overlap(s, x) || overlap(s, r) || overlap(s, h) || overlap(s, y) || overlap(s, g) ||
        overlap(g, h) || overlap(g, y))
        return BAKRON_E_INVALID_ARG;
    return bk::launch_rmsnorm(X, xtype, T, n, ldx, R, ldr, H, ldh, gain, gtype, eps, rotate != 0, seed, Y, ytype, ldy,
                              yscale, (hipStream_t)stream);
}

size_t bakron_lora_workspace_bytes(int64_t T, int64_t r) {
    return T < 1 || T > (int64_t)1 << 40 || r < 1 || r > bk::kMaxRank ? 0 : bk::lora_workspace_bytes(T, r);
}

int bakron_lora(const void* X, int32_t xtype, int64_t T, int64_t n, int64_t ldx, const float* xscale, const void* A,
                const void* B, int32_t wtype, int64_t R, int64_t r, int64_t m, const float* scales, const int32_t* ids,
                const void* base, int32_t btype, int64_t ldb, void* Y, int32_t ytype, int64_t ldy, void* ws, size_t ws_bytes,
                void* stream) {
    constexpr int64_t kMax = (int64_t)1 << 28;
    if (T < 0 || T > (int64_t)1 << 40 || n < 1 || m < 1 || n >= kMax || m >= kMax || r < 1 || r > bk::kMaxRank || R < 1 ||
        R > 0x7fffffff)
        return BAKRON_E_INVALID_ARG;
    if (elem_size(xtype) == 0 || !wide_type(wtype) || !wide_type(ytype) || (base && !wide_type(btype)))
        return BAKRON_E_INVALID_ARG;
    if (wide_type(xtype) ? wtype != xtype : wtype == BAKRON_F32) return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    if (!X || !A || !B || !ids || !Y || bad_ld(ldx, n) || bad_ld(ldy, m) || (base && bad_ld(ldb, m)))
        return BAKRON_E_INVALID_ARG;
    const Rows y = rows_of(Y, T, m, ldy, ytype), b = rows_of(base, T, m, ldb, btype);
    const Rows in[6] = {rows_of(X, T, n, ldx, xtype), rows_of(A, R, r * n, r * n, wtype), rows_of(B, R, m * r, m * r, wtype),
                        {xscale, 1, 4 * T, 4 * T}, {scales, 1, 4 * R, 4 * R}, {ids, 1, 4 * T, 4 * T}};
    for (const Rows& i : in)
        if (overlap(i, y)) return BAKRON_E_INVALID_ARG;
    if (overlap(b, y) && !(same_rows(b, y) && btype == ytype)) return BAKRON_E_INVALID_ARG;
    const size_t need = bk::lora_workspace_bytes(T, r);
    if (need) {
        const Rows w = {ws, 1, (int64_t)ws_bytes, (int64_t)ws_bytes};
        if (((uintptr_t)ws & 15) != 0 || overlap(w, y) || overlap(w, b)) return BAKRON_E_INVALID_ARG;
        for (const Rows& i : in)
            if (overlap(i, w)) return BAKRON_E_INVALID_ARG;
        if (!ws || ws_bytes < need) return BAKRON_E_WORKSPACE;
    }
    return bk::launch_lora(X, xtype, T, n, ldx, xscale, A, B, wtype, R, r, m, scales, ids, base, btype, ldb, Y, ytype, ldy,
                           ws, (hipStream_t)stream);
}

int bakron_head_norm(const void* Q, int64_t hq, int64_t qt, int64_t qh, const void* K, int64_t hk, int64_t kt, int64_t kh,
                     int32_t type, int64_t T, int64_t d, const void* qgain, const void* kgain, int32_t gtype, float eps,
                     int norm, const void* pos, int pos32, const float* freq, int64_t rot, int interleaved, void* YQ,
                     int64_t yqt, int64_t yqh, void* YK, int64_t ykt, int64_t ykh, void* stream) {
    if (!wide_type(type) || T < 0 || T > 0x7fffffff || hq < 1 || hk < 0 || hq > 65535 || hk > 65535 || d < 1 ||
        d > bk::kMaxHeadDim || rot < 0 || rot > d || (rot & 1))
        return BAKRON_E_INVALID_ARG;
    if (!(eps >= 0.0f) || !(eps < INFINITY)) return BAKRON_E_INVALID_ARG;
    if ((qgain || kgain) && (!norm || (gtype != type && gtype != BAKRON_F32))) return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    if (!Q || !YQ || (hk && (!K || !YK)) || (rot && (!pos || !freq))) return BAKRON_E_INVALID_ARG;
    if (bad_heads(T, hq, d, qt, qh) || bad_heads(T, hq, d, yqt, yqh)) return BAKRON_E_INVALID_ARG;
    if (hk && (bad_heads(T, hk, d, kt, kh) || bad_heads(T, hk, d, ykt, ykh))) return BAKRON_E_INVALID_ARG;
    const Heads in[2] = {{Q, T, hq, d, qt, qh, type}, {hk ? K : nullptr, T, hk, d, kt, kh, type}};
    const Heads out[2] = {{YQ, T, hq, d, yqt, yqh, type}, {hk ? YK : nullptr, T, hk, d, ykt, ykh, type}};
    const bool same[2] = {Q == YQ && (T == 1 || qt == yqt) && (hq == 1 || qh == yqh),
                          K == YK && (T == 1 || kt == ykt) && (hk <= 1 || kh == ykh)};
    const Rows small[4] = {rows_of(qgain, 1, d, d, gtype), rows_of(kgain, 1, d, d, gtype),
                           {rot ? pos : nullptr, 1, (pos32 ? 4 : 8) * T, (pos32 ? 4 : 8) * T},
                           {rot ? freq : nullptr, 1, 2 * rot, 2 * rot}};
    if (overlap(out[0], out[1])) return BAKRON_E_INVALID_ARG;
    for (int o = 0; o < 2; ++o) {
        for (int i = 0; i < 2; ++i)
            if (overlap(in[i], out[o]) && !(i == o && same[i])) return BAKRON_E_INVALID_ARG;
        for (const Rows& r : small)
            if (overlap(r, rows_of_heads(out[o]))) return BAKRON_E_INVALID_ARG;
    }
    const bk::HeadRows q = {Q, YQ, qgain, hq, qt, qh, yqt, yqh}, k = {K, YK, kgain, hk, kt, kh, ykt, ykh};
    return bk::launch_head_norm(q, k, type, T, d, gtype, eps, norm != 0, pos, pos32 != 0, freq, rot, interleaved != 0,
                                (hipStream_t)stream);
}

int bakron_route(const void* logits, int32_t type, int64_t T, int64_t E, int64_t ldl, int64_t k, int scoring,
                 const float* bias, int renorm, float scale, int32_t* ids, float* weights, void* stream) {
    if (!wide_type(type) || T < 0 || T > (int64_t)1 << 40 || E < 1 || E > bk::kMaxExperts || k < 1 ||
        k > bk::kMaxChosen || k > E)
        return BAKRON_E_INVALID_ARG;
    if ((scoring != BAKRON_SCORE_SOFTMAX && scoring != BAKRON_SCORE_SIGMOID) || (bias && scoring == BAKRON_SCORE_SOFTMAX) ||
        !(scale - scale == 0.0f))
        return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    if (!logits || !ids || !weights || bad_ld(ldl, E)) return BAKRON_E_INVALID_ARG;
    const Rows l = rows_of(logits, T, E, ldl, type), b = rows_of(bias, 1, E, E, BAKRON_F32);
    const Rows i = {ids, 1, 4 * T * k, 4 * T * k}, w = {weights, 1, 4 * T * k, 4 * T * k};
    if (overlap(i, w) || overlap(l, i) || overlap(l, w) || overlap(b, i) || overlap(b, w)) return BAKRON_E_INVALID_ARG;
    return bk::launch_route(logits, type, T, E, ldl, k, scoring == BAKRON_SCORE_SIGMOID, bias, renorm != 0, scale, ids,
                            weights, (hipStream_t)stream);
}

size_t bakron_experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I) {
    if (bad_experts(T, k, E, n, I) || T == 0) return 0;
    return bk::experts_workspace_bytes(T, k, E, n, I);
}

int bakron_experts(const void* gate, const void* up, size_t gate_bytes, int32_t bits, int64_t group, const void* down,
                   size_t down_bytes, int32_t dbits, int64_t dgroup, int64_t E, int64_t n, int64_t I, const void* X,
                   int32_t xtype, int64_t T, int64_t ldx, const float* xscale, const int32_t* ids, const float* weights,
                   int64_t k, int act, void* Y, int32_t ytype, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
    if (bad_experts(T, k, E, n, I) || bad_pack_shape(I, n, bits, group) || bad_pack_shape(n, I, dbits, dgroup))
        return BAKRON_E_INVALID_ARG;
    if (elem_size(xtype) == 0 || !wide_type(ytype) || (act != BAKRON_ACT_SILU && act != BAKRON_ACT_GELU))
        return BAKRON_E_INVALID_ARG;
    if (T == 0) return BAKRON_OK;
    if (!gate || !up || !down || !X || !ids || !weights || !Y || bad_ld(ldx, n) || bad_ld(ldy, n))
        return BAKRON_E_INVALID_ARG;
    if ((((uintptr_t)gate | (uintptr_t)up | (uintptr_t)down | (uintptr_t)ws) & 15) != 0) return BAKRON_E_INVALID_ARG;
    const int64_t gb = (int64_t)gate_bytes, db = (int64_t)down_bytes, wb = (int64_t)ws_bytes;
    const Rows y = rows_of(Y, T, n, ldy, ytype), w = {ws, 1, wb, wb};
    const Rows in[7] = {{gate, 1, gb, gb}, {up, 1, gb, gb}, {down, 1, db, db}, rows_of(X, T, n, ldx, xtype),
                        {xscale, 1, 4 * T, 4 * T}, {ids, 1, 4 * T * k, 4 * T * k}, {weights, 1, 4 * T * k, 4 * T * k}};
    if (overlap(y, w)) return BAKRON_E_INVALID_ARG;
    for (const Rows& i : in)
        if (overlap(i, y) || overlap(i, w)) return BAKRON_E_INVALID_ARG;
    if (gate_bytes / E < bk::pack_shape(I, n, bits, group).bytes || down_bytes / E < bk::pack_shape(n, I, dbits, dgroup).bytes)
        return BAKRON_E_WORKSPACE;
    if (!ws || ws_bytes < bk::experts_workspace_bytes(T, k, E, n, I)) return BAKRON_E_WORKSPACE;
    return bk::launch_experts(gate, up, bits, group, down, dbits, dgroup, E, n, I, X, xtype, T, ldx, xscale, ids, weights, k,
                              act, Y, ytype, ldy, ws, (hipStream_t)stream);
}

}  // extern "C"
