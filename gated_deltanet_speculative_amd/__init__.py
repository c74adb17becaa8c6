"""MI355X-native speculative-verify Gated DeltaNet route.

Three calls over one caller stream, each a thin binding of the C ABI in
include/gdn_verify.h (libgdnverify.so, hand-written gfx950 HIP kernels):

    conv_tree_step  -> conv_out, commit_win
    tree_verify     -> out, replay_log          (persistent state read-only)
    conv_tree_verify -> out, replay_log, commit_win  (the two above fused)
    replay_commit   -> advances state_pool / conv_hist of accepting slots
    replay_commit_layers -> the same for every layer of a round, one launch

and, for a step without a draft (plain decode), two calls that advance the slots
directly:

    conv_step       -> conv_out; writes each slot's conv history in place
    decode_step     -> out; applies one token to each slot's state in place
    conv_decode_step -> out; the two above for one token, fused in one launch

and a prompt fills a slot with conv_step over its tokens followed by

    prefill         -> out; the recurrence over the prompt, each slot's state in place
                       (prefill_workspace_size: the scratch bytes it needs;
                       prefill_noalloc: the same with the library's static scratch,
                       for callers that cannot allocate)

Around the recurrence (include/gdn_round.h), the attention layers' part of a round over a
paged key/value cache and the acceptance of the draft:

    rope_kv_write    -> q_out; rotary positions, k and v written behind the committed rows
    paged_attention  -> out; the round's tokens over the cache and their own ancestors
    draft_accept     -> accept_node, n_accept, next_token (what the commits take)
    kv_commit_layers -> new_len; the accepted paths' cache rows moved together, every layer

and the same over a cache held in 4 bits (include/gdn_kv4.h):

    rope_kv4_write   -> q_out; k and v written as 4-bit numbers with a power of two for every 32
    paged_attention_kv4 -> out
    kv4_commit_layers -> new_len
    kv4_read_layers  -> rows of every layer's cache as values
    kv4_cache        -> a cache of zeros

and between the target's logits and the acceptance (include/gdn_logits.h):

    adjust_logits    -> penalties for repeated tokens, biases, grammar masks; with temperatures, the
                        probabilities that draft_accept takes

The library is loaded on first use and must have been built
(`python -m gated_deltanet_speculative_amd.build`); there is no fallback path.
"""

from ._lib import (  # noqa: F401
    EXPORTED,
    GdnError,
    LIB_PATH,
    MAX_CHAIN,
    MAX_LAYERS,
    Shape,
    STATUS_ACCEPT,
    STATUS_NODES,
    STATUS_PARENT,
    STATUS_SLOT_DUP,
    STATUS_SLOT_RANGE,
    SYNC_STRIDE,
    conv_decode_step,
    conv_step,
    conv_tree_step,
    conv_tree_verify,
    decode_step,
    STATIC_SCRATCH_BYTES,
    prefill,
    prefill_noalloc,
    prefill_workspace_size,
    load_library,
    replay_commit,
    replay_commit_layers,
    strerror,
    tree_verify,
)
from ._round import (  # noqa: F401
    AcceptShape,
    AttnShape,
    ROUND_EXPORTED,
    STATUS_AXIS,
    STATUS_LENGTH,
    STATUS_PAGE,
    STATUS_TOKEN,
    draft_accept,
    draft_accept_workspace_size,
    kv_commit_layers,
    paged_attention,
    paged_attention_workspace_size,
    rope_kv_write,
)
from ._kv4 import (  # noqa: F401
    KV4_EXPORTED,
    Kv4Cache,
    kv4_cache,
    kv4_commit_layers,
    kv4_read_layers,
    paged_attention_kv4,
    paged_attention_kv4_workspace_size,
    rope_kv4_write,
)
from ._logits import (  # noqa: F401
    LOGITS_EXPORTED,
    LogitsShape,
    STATUS_RULE,
    adjust_logits,
    adjust_logits_workspace_size,
)
