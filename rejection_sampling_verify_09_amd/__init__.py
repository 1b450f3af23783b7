"""MI355X (gfx950) speculative-sampling verification.

The computation runs in libspecverify.so (hand-written HIP kernels behind the
C ABI of include/specverify.h); this package is its Python binding.
"""
from ._lib import (  # noqa: F401
    SV_BF16,
    SV_F32,
    SV_MAX_K,
    DraftLengthController,
    SpecVerifyError,
    adjust_logits,
    distill_loss,
    filtered_probs,
    init,
    layer_norm,
    layer_norm_backward,
    lib,
    linear,
    lm_logits,
    profile_start,
    profile_stop,
    read_floor,
    release,
    rms_norm,
    rms_norm_backward,
    scratch_bytes,
    stream_release,
    sample,
    spec_verify,
    spec_verify_noalloc,
    spec_verify_lmhead,
    spec_verify_probs,
    spec_verify_ragged,
    status_string,
    top_logits,
)

__all__ = ["spec_verify", "spec_verify_noalloc", "spec_verify_lmhead", "lm_logits", "rms_norm", "linear", "adjust_logits", "layer_norm", "layer_norm_backward", "rms_norm_backward", "top_logits", "distill_loss", "spec_verify_probs", "spec_verify_ragged", "DraftLengthController", "sample", "filtered_probs", "profile_start", "profile_stop", "read_floor", "release", "init", "stream_release", "scratch_bytes", "status_string", "lib",
           "SpecVerifyError"]
