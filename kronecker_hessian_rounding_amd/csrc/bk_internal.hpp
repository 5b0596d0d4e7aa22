// bk_internal.hpp -- host-side interfaces between the C ABI layer and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/bakron.h"

namespace bk {

// Round a byte count up to a 256-byte boundary (workspace carving).
inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Compute units and the wall clock of s_memrealtime of the current device, read once per device.
struct DeviceInfo {
    int cus = 0;
    int clock_khz = 0;
};
inline DeviceInfo device_info() {
    static DeviceInfo cache[64];
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
    DeviceInfo& di = cache[dev];
    if (di.cus == 0) {
        int cus = 0, khz = 0;
        if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0)
            cus = 256;
        if (hipDeviceGetAttribute(&khz, hipDeviceAttributeWallClockRate, dev) != hipSuccess || khz <= 0)
            khz = 100000;
        di.clock_khz = khz;
        di.cus = cus;
    }
    return di;
}

// --- Hessian factor accumulation (bk_accum.hip) ---
size_t hessian_workspace_bytes(int64_t T, int64_t d);
// trans: X is stored d x T (H = X X^T); wt: per-token weights (H = sum_k wt_k
// x_k^T x_k); both need the workspace of the piece path
int launch_hessian_accum(const float* X, int64_t T, int64_t d, int64_t ldx, float alpha,
                         float beta, float* H, int64_t ldh, void* ws, size_t ws_bytes,
                         hipStream_t stream, bool trans = false, const float* wt = nullptr,
                         int64_t tin = 0, int64_t bs = 0);

// --- Sketch A token weights (bk_sketch.hip) ---
size_t token_weights_workspace_bytes(int64_t T, int64_t d);
int launch_token_weights(const float* Y, int64_t T, int64_t d, int64_t ldy, const float* H, int64_t ldh,
                         float* w, void* ws, size_t ws_bytes, hipStream_t stream);

// --- LDL factorisation (bk_ldl.hip) ---
size_t ldl_workspace_bytes(int64_t d);
// Enqueues the whole factorisation on `stream` without waiting; with info_dev
// (device int64) non-null, the status (-1, the first failing pivot, or -2 for a
// wait that timed out) lands there. allow_sched false keeps it to the launch chain.
int enqueue_ldl(float* H, int64_t d, int64_t ldh, double damp_rel, float* D, void* ws,
                hipStream_t stream, int64_t* info_dev, bool allow_sched = true);
int run_ldl(float* H, int64_t d, int64_t ldh, double damp_rel, float* D, int64_t* bad_pivot,
            void* ws, hipStream_t stream);
// Two factorisations: in one launch on `stream` when both take the scheduled
// path, else A on `stream` and B on `stream_b`, both by the launch chain.
// info* are device int64, required.
int enqueue_ldl_pair(float* HA, int64_t dA, int64_t ldha, float* DA, void* wsA, int64_t* infoA,
                     float* HB, int64_t dB, int64_t ldhb, float* DB, void* wsB, int64_t* infoB,
                     double damp_rel, hipStream_t stream, hipStream_t stream_b);

// --- incoherence rotation (bk_rotate.hip) ---
int launch_rht(float* A, int64_t rows, int64_t cols, int64_t lda, int axis, uint64_t seed, int transpose,
               hipStream_t stream);

// --- packed layers and their products (bk_matvec.hip) ---
struct PackShape {
    int W;  // bits stored per weight
    int64_t tiles, chunks, groups, groups_padded;
    size_t scale_offset, bytes;
};
PackShape pack_shape(int64_t m, int64_t n, int bits, int64_t group);
int launch_pack(const uint8_t* codes, int64_t m, int64_t n, int64_t ldc, int bits, const float* scales, int64_t lds,
                int64_t group, void* packed, hipStream_t stream);
int launch_matvec(const void* packed, int64_t m, int64_t n, int bits, int64_t group, const void* x, int xtype,
                  int64_t T, int64_t ldx, const float* xs, void* y, int ytype, int64_t ldy, hipStream_t stream);

// --- norm with residual, rotation and 8-bit output (bk_norm.hip) ---
constexpr int64_t kNormMaxBuffered = 32768;  // longest row held in LDS as fp32 (128 KB)
int launch_rmsnorm(const void* x, int xtype, int64_t T, int64_t n, int64_t ldx, const void* r, int64_t ldr, void* h,
                   int64_t ldh, const void* gain, int gtype, float eps, int rotate, uint64_t seed, void* y, int ytype,
                   int64_t ldy, float* ys, hipStream_t stream);

// --- low-rank adapters (bk_lora.hip) ---
constexpr int64_t kMaxRank = 512;
int launch_lora(const void* x, int xtype, int64_t T, int64_t n, int64_t ldx, const float* xs, const void* A, const void* B,
                int wtype, int64_t R, int64_t r, int64_t m, const float* scales, const int32_t* ids, const void* base,
                int btype, int64_t ldb, void* y, int ytype, int64_t ldy, void* ws, hipStream_t stream);
size_t lora_workspace_bytes(int64_t T, int64_t r);

// --- norm and position rotation of heads (bk_heads.hip) ---
constexpr int64_t kMaxHeadDim = 512;
struct HeadRows {
    const void* x;
    void* y;
    const void* gain;
    int64_t heads, xt, xh, yt, yh;  // strides of tokens and heads, in elements
};
int launch_head_norm(const HeadRows& q, const HeadRows& k, int type, int64_t T, int64_t d, int gtype, float eps, int norm,
                     const void* pos, int pos32, const float* freq, int64_t rot, int interleaved, hipStream_t stream);

// --- a router's choice of experts (bk_route.hip) ---
constexpr int64_t kMaxExperts = 1024, kMaxChosen = 64;
int launch_route(const void* logits, int type, int64_t T, int64_t E, int64_t ldl, int64_t k, int sigmoid,
                 const float* bias, int renorm, float scale, int32_t* ids, float* weights, hipStream_t stream);

// --- a mixture of rounded experts (bk_experts.hip) ---
constexpr int64_t kMaxExpertDim = (int64_t)1 << 18;
size_t experts_workspace_bytes(int64_t T, int64_t k, int64_t E, int64_t n, int64_t I);
int launch_experts(const void* gate, const void* up, int bits, int64_t group, const void* down, int dbits, int64_t dgroup,
                   int64_t E, int64_t n, int64_t I, const void* x, int xtype, int64_t T, int64_t ldx, const float* xs,
                   const int32_t* ids, const float* weights, int64_t k, int act, void* y, int ytype, int64_t ldy, void* ws,
                   hipStream_t stream);

// --- bound and sensitivity report (bk_report.hip) ---
int launch_layer_report(int64_t m, int64_t n, const float* DO, const float* DI, const float* scales,
                        const float* HI, int64_t ldhi, const float* HO, int64_t ldho, double* out,
                        hipStream_t stream);

// --- rounding solve (bk_solve.hip) ---
struct SolveArgs {
    const float* W;
    int64_t m, n, ldw;
    const float* LO;
    int64_t ldlo;
    const float* LI;
    int64_t ldli;
    int bits;
    int stochastic;
    uint64_t seed;
    const float* row_scale;
    uint8_t* codes;
    int64_t ldc;
    float* scales;
    float* delta;
    int64_t ldd;
    const float* DO;
    const float* DI;
    double* loss;
    int64_t* clamped;
    int32_t* info;
};
size_t solve_workspace_bytes(int64_t m, int64_t n);
int run_solve(const SolveArgs& a, void* ws, hipStream_t stream);

}  // namespace bk
