"""GB300 (sm_103a) recurrent KDA training forward + backward behind a C ABI.

``kda_fwd`` / ``kda_bwd`` (and the aliases ``recurrent_kda_training_forward`` /
``recurrent_kda_training_backward``), the standalone ``recurrent_kda_backward``
(with a reusable ``RecurrentKDABackwardWorkspace``), the inference
``kda_prefill`` and the single-token ``kda_decode`` call libkda.so; ``HostStep`` runs whole training
steps from and to host memory (``kda_step_host``). Linear attention with a decay for each head:
``kda_decay_attn_fwd`` / ``_bwd`` / ``_prefill`` / ``_decode``, and the norm and position rotation of its
queries and keys, ``kda_qk_norm_rope_fwd`` / ``_bwd``. The gated delta rule with a decay for each token and head:
``kda_gated_delta_fwd`` / ``_bwd`` / ``_prefill`` / ``_decode``. Layer norm: ``kda_layer_norm_fwd`` / ``_bwd``.
See include/kda.h.
"""

from .decay import (  # noqa: F401
    DecayContext,
    decay_workspace_bytes,
    kda_decay_attn_bwd,
    kda_decay_attn_decode,
    kda_decay_attn_fwd,
    kda_decay_attn_prefill,
    kda_qk_norm_rope_bwd,
    kda_qk_norm_rope_fwd,
)

from .delta import (  # noqa: F401
    DeltaContext,
    gated_delta_workspace_bytes,
    kda_gated_delta_bwd,
    kda_gated_delta_decode,
    kda_gated_delta_fwd,
    kda_gated_delta_prefill,
)

from .norm import (  # noqa: F401
    kda_layer_norm_bwd,
    kda_layer_norm_fwd,
)

from .kda import (  # noqa: F401
    EXPORTED,
    GRAD_NAMES,
    HostStep,
    KdaContext,
    KdaError,
    RecurrentKDABackwardWorkspace,
    kda_bwd,
    kda_bwd_noalloc,
    kda_decode,
    kda_fwd,
    kda_prefill,
    load_library,
    noalloc_status,
    recurrent_kda_backward,
    recurrent_kda_training_backward,
    recurrent_kda_training_forward,
    workspace_bytes,
)
