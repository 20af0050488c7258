"""Fused MaxSim late-interaction scoring for AMD MI355X (gfx950).

The operator lives in liblik.so (hand-written HIP kernels behind a C ABI,
declared in include/lik.h), and beside it the losses over rows of logits that
train on its scores (lik_ce_rows, and those of include/lik_rows.h), and the
steps of generation that make what they train on: drafted tokens verified
(lik_verify_rows) over a paged cache in 8 bits (include/lik_cache.h).  This
package holds the thin ctypes binding (``_lib``), the build script (``build``)
and the seeded synthetic workloads (``workloads``).
"""

from ._lib import (  # noqa: F401
    LikError,
    lik_maxsim_fwd,
    lik_maxsim_bwd,
    lik_maxsim_pairwise_fwd,
    lik_maxsim_pairwise_bwd,
    lik_maxsim_kd_fwd,
    lik_maxsim_kd_bwd,
    lik_ce_rows,
    lik_logprob_rows_fwd,
    lik_logprob_rows_bwd,
    lik_distill_rows,
    lik_policy_rows,
    lik_preference_rows,
    lik_verify_rows,
    lik_cache_tables,
    lik_cache_append,
    lik_cache_attention,
    LIK_PREF_SIGMOID,
    LIK_PREF_HINGE,
    LIK_PREF_SQUARE,
)
