"""MI355X-native BaKron: two-sided adaptive rounding under a Kronecker-factored Hessian.

The computation runs in libbakron (HIP kernels for gfx950, C ABI in
include/bakron.h); this package is a thin ctypes binding that takes PyTorch
tensors for device memory and uses the current stream.

  hessian_accum(X)            H <- beta H + alpha X^T X            (fp16 pieces, fp32 accuracy)
  sketch_b(grads)             H_I = E[G^T G]/m, H_O = E[G G^T]/n from per-sequence gradients
  sketch_a(X, G, iters)       alternating factor estimate with per-token weights
  ldl(H, damp_rel)            H + lambda I = (L + I) D (L + I)^T   (fp64, L strictly upper)
  ldl_pair(HA, HB, damp_rel)  two independent factorisations side by side on two streams
  check_ldl_pair(status)      raise for the statuses a non-waiting ldl_pair(..., status=) left
  solve(W, L_O, L_I, bits)    BaKron rounding: codes, scales, error, proxy loss
  solve_noalloc(W, L_O, L_I, bits, out)  the same, allocating nothing (library-held scratch)
  rotate_layer(W, HI, HO, sO, sI) two-sided randomised Hadamard rotation (incoherence processing)
  quantize_layer(W, X, G, b)  the whole per-layer path
  pack(codes, scales, bits)   a rounded layer laid out for matvec (2 or 4 bits a weight, row or group scales)
  matvec(x, packed)           x W^T for tokens x in fp32, fp16, bf16, int8 or e4m3
  rmsnorm(x, gain, residual)  norm with the residual's addition, the layer's rotation and an 8-bit output
  lora(x, a, b, ids, base)    low-rank adapters of many requests beside a shared projection
  head_norm(q, k, ...)        norm of each query and key head with the position rotation
  route(logits, k)            a router's choice of experts and their weights
  pack_experts(codes, scales, bits)  the layers of a mixture of experts laid out for experts
  experts(x, gate, up, down, ids, weights)  the products of a mixture of rounded experts
"""
from ._binding import (  # noqa: F401
    BAKRON_E_DEVICE, BAKRON_E_INVALID_ARG, BAKRON_E_NOT_SPD, BAKRON_E_WORKSPACE, BAKRON_OK,
    EXPORTS, LIB, LIB_PATH, NOALLOC_SCRATCH_BYTES, ROW_TYPES, BakronError, NormResult, PackedExperts, PackedWeight,
    SolveResult,
    abi_version, check_ldl_pair, experts, head_norm, hessian_accum, ldl, ldl_pair, layer_report, lora, matvec, pack, pack_experts, quantize_layer,
    release_workspace, rht, rmsnorm, rotate_layer, route, sketch_a, sketch_b, solve, solve_noalloc, token_weights,
)
