"""MI355X-native (gfx950) owner-side Muon step, AdamW tail, Shampoo and SOAP steps,
and the operators that write the gradients these steps read.

Under owner-shaped ZeRO-3 placement ("MatrixFSDP: communication-free matrix
optimizers under ZeRO-3 parameter sharding", §3) each 2D weight is whole on one
owner, so that owner runs Muon locally on its whole matrices and AdamW on its
packed non-2D tail.  This package is that step: hand-written HIP kernels behind
the C ABI in ``include/mo.h`` (``libmo.so``), with this thin ctypes binding.

    from matrix_optimizers_amd import muon_owner_step, adamw_tail_step
    muon_owner_step([(W, G, M), ...], lr=0.02, weight_decay=0.01)
    adamw_tail_step(p, g, m, v, step=10)
    shampoo_owner_step([(W, G, L, R), ...], lr=1e-3, root_iters=20)
    soap_owner_step([(W, G, L, R, M, V), ...], lr=1e-3, step=t)

    Y = embedding_forward(tokens, W);  embedding_backward(tokens, dY, G)
    Y, mean, rstd = layer_norm_forward(X, weight, bias)
    dX, dweight, dbias = layer_norm_backward(dY, X, mean, rstd, weight)
    Y, h, rstd = rms_norm_forward(X, weight, residual=R)
    q, scales, h, rstd = rms_norm_quantize(X, weight, residual=R)
    dX, dweight = rms_norm_backward(dY, h, rstd, weight, dH=dH)
    wq, ws, wqt, wst = fp8_quantize_weight(W)
    Y = fp8_matmul(q, scales, wq, ws)
    dX = fp8_matmul(*fp8_quantize(dY), wqt, wst)
    fp8_weight_grad(dY, q, scales, G);  X = fp8_dequantize(*fp8_quantize(X))
    loss, lse = softmax_xent_forward(H, W, labels)
    dH, dW = softmax_xent_backward(H, W, labels, loss, lse, dloss)
    loss, lse, z = topk_distill_forward(H, W, ids, logits, temperature=T)
    dH, dW = topk_distill_backward(H, W, ids, logits, lse, z, dloss, temperature=T)

The library is loaded on first use; if it has not been built
(``python -m matrix_optimizers_amd.build``) every entry point raises.
"""
from ._binding import (  # noqa: F401
    PLAN_POLICIES, ROLE_MATRIX, ROLE_TAIL, MoError, MoMatrix, MoMuonHParams, MoRole, MuonOwnerStep,
    MoShampooHParams, MoShampooMatrix, ShampooOwnerStep, shampoo_descriptor, shampoo_hparams,
    shampoo_owner_step, shampoo_tensor_descriptor, shampoo_workspace_bytes,
    MoSoapHParams, MoSoapMatrix, SoapOwnerStep, soap_descriptor, soap_hparams, soap_owner_step,
    soap_converged, soap_tensor_descriptor, soap_workspace_bytes,
    PHASES, adamw_tail_step, build_worklist, descriptor, device_copy, hparams, load_library,
    mo_status_string, muon_build_worklist, muon_owner_step, muon_owner_step_noalloc, muon_workspace_bytes,
    NOALLOC_SCRATCH_BYTES, plan_layout,
    plan_owners, plan_score, profile_enable, profile_read, status_string, tensor_descriptor,
    workspace_bytes,
)

_OPERATORS = (
    "TOPK_MAX", "embedding_backward", "embedding_forward", "embedding_workspace_bytes",
    "layer_norm_backward", "layer_norm_forward", "layer_norm_workspace_bytes", "rms_norm_backward",
    "rms_norm_forward", "rms_norm_quantize", "rms_norm_workspace_bytes", "softmax_xent_backward",
    "softmax_xent_forward", "softmax_xent_workspace_bytes", "topk_distill_backward", "topk_distill_forward",
    "topk_distill_workspace_bytes",
)
_FP8 = (
    "fp8_dequantize", "fp8_matmul", "fp8_matmul_workspace_bytes", "fp8_quantize", "fp8_quantize_weight",
    "fp8_weight_grad", "fp8_weight_grad_workspace_bytes",
)


def __getattr__(name):
    """The operators, imported with torch on first use (the rest of the package
    imports without it)."""
    if name in _OPERATORS or name in _FP8:
        from . import fp8, operators
        globals().update({n: getattr(operators, n) for n in _OPERATORS})
        globals().update({n: getattr(fp8, n) for n in _FP8})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(set(globals()) | set(_OPERATORS) | set(_FP8))
