"""Parallel evaluation of recurrences (diagonal GRU / LSTM by Newton iterations, gated linear ones by one scan) on AMD MI355X.

The compute lives in libprn.so (HIP, gfx950; C ABI in include/prn.h).
``binding`` marshals torch tensors into that ABI under the same names;
``api`` adds allocation, contiguity, K schedules, the residual gate and the
agreement check; ``lm`` has the operators of a token model around the
recurrence (embedding lookup, block-boundary norms, vocabulary loss, gated
feed-forward product, dropout).
"""
from .binding import (  # noqa: F401
    EXPORTS, PrnError, PrnUnsupportedError, lib, prn_backward_workspace_bytes, prn_input_proj, prn_last_error, prn_newton_backward,
    prn_newton_forward, prn_newton_forward_fused, prn_sequential_forward, prn_validate_cu_seqlens, prn_version,
    prn_workspace_bytes,
)
from .api import (  # noqa: F401
    AGREEMENT_ATOL, AgreementError, AgreementReport, LookbackTimeoutError, NewtonDivergenceError, RESIDUAL_FAIL,
    RESIDUAL_WARN,
    forward, forward_fused, gate_residual, input_proj, input_proj_apply, newton_apply, newton_forward, resolve_k,
    sequential_forward, validate_cu_seqlens, verify_agreement,
    check_waits, gated_scan, gated_scan_apply, gated_scan_backward,
)
from .lm import (  # noqa: F401
    block_norm, block_norm_apply, block_norm_backward, embed, embed_apply, embed_backward, vocab_loss,
    vocab_loss_apply, vocab_loss_backward,
    dropout, dropout_apply, dropout_backward, gated_ffn, gated_ffn_apply, gated_ffn_backward,
)
