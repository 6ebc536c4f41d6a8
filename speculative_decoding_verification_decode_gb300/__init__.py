"""GB300-native verification step of speculative decoding.

Greedy verification and Leviathan/Chen rejection sampling for B sequences in
one kernel launch (libsv.so, C ABI in include/sv.h); this package is the thin
PyTorch binding.  See the spec-verify model card, sections "Method" and
"Correctness", for what is computed.
"""

from ._lib import (  # noqa: F401
    FLAG_EXPIRE_EXCHANGE,
    FLAG_FORCE_EXACT,
    FLAG_PLAN_CHAIN,
    FLAG_PLAN_ROWS,
    SEQ_BAD_LAYOUT,
    SEQ_BAD_TOKEN,
    SEQ_BAD_VALUE,
    SEQ_EXACT_PATH,
    SEQ_NEAR_BOUNDARY,
    SEQ_NO_PAGES,
    SEQ_TIMEOUT,
    SEQ_ZERO_MASS,
    load as load_library,
)
from .api import (  # noqa: F401
    BeamCandidates,
    GateResult,
    LMHeadResult,
    PagedCache,
    Q4Projection,
    SVError,
    TreeAttention,
    TreeResult,
    VerifyResult,
    accept,
    accept_from_logits,
    apply_penalties,
    beam_reorder,
    beam_select,
    beam_select_workspace,
    cache_append,
    cache_fork,
    cache_truncate,
    gate_draft_lengths,
    gate_update,
    lm_head_logits,
    lm_head_verify,
    lm_head_verify_static,
    lm_head_workspace,
    paged_cache,
    q4_quantize,
    sampler_floors,
    tree_attention,
    verify_greedy,
    verify_tree,
    verify_tree_greedy,
)
from ._build import build  # noqa: F401
from .decoder import BeamDecoder, SpeculativeDecoder, TreeDecoder  # noqa: F401,E402
