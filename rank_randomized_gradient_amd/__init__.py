"""Randomized low-rank gradient sketching on MI355X (gfx950).

The hot path of a linear layer W (d x k) trained from a rank-r sketch of its
gradient, as hand-written HIP kernels behind the C ABI in include/rgc.h:
projection sampling, XP = X P, C += D^T (X P), and the normalized update
with stochastic rounding to bf16. `rgc` is the thin ctypes binding;
`sketched_linear` wraps a bf16 linear layer whose backward feeds the sketch.
"""
from .rgc import (  # noqa: F401
    RgcError,
    Workspace,
    abi_version,
    load_library,
    rgc_accumulate,
    rgc_accumulate_batch,
    rgc_accumulate_batch_deferred,
    rgc_apply,
    rgc_apply_batch,
    rgc_apply_carried,
    rgc_apply_carried_batch,
    rgc_apply_from_seed,
    rgc_apply_scaled,
    rgc_apply_scaled_batch,
    rgc_project,
    rgc_project_batch,
    rgc_project_shared,
    rgc_linear_forward,
    rgc_linear_forward_batch,
    rgc_linear_backward,
    rgc_linear_cross_entropy_forward,
    rgc_linear_cross_entropy_backward,
    rgc_layer_norm_forward,
    rgc_layer_norm_backward,
    rgc_add_norm_forward,
    rgc_add_norm_backward,
    rgc_linear_log_prob_forward,
    rgc_linear_log_prob_backward,
    rgc_log_prob_forward,
    rgc_log_prob_backward,
    rgc_grad_norm_batch,
    rgc_scale_batch,
    rgc_adamw_batch,
    rgc_sample_projection,
    rgc_sample_projections,
    rgc_test_philox,
    rgc_test_reconstruct,
    rgc_test_stochastic_round,
)
from .sketched_linear import SketchedLinear, SketchedLinearFunction  # noqa: F401,E402
from .sketched_head import SketchedCrossEntropy, SketchedCrossEntropyFunction, SketchedLogProbFunction  # noqa: F401,E402
from .layer_norm import AddNormFunction, LayerNorm, LayerNormFunction  # noqa: F401,E402
from .logits import LogProbFunction, log_prob  # noqa: F401,E402
from .clip import clip_grad_norm  # noqa: F401,E402
from .adamw import AdamW  # noqa: F401,E402
