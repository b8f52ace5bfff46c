"""GB300-native path-conditioned draft-tree construction (libdtree + binding)."""
from .dtree import (  # noqa: F401
    DraftTreeBuilder,
    DtreeError,
    bf16_tensor,
    check_config,
    load_library,
    node_count,
    status_string,
    workspace_bytes,
)
from .kvcache import (  # noqa: F401
    AttentionWorkspace,
    KvCache,
    cache_attention,
    kv_append,
    kv_plan,
    prompt_attention,
)
from .layer import (  # noqa: F401
    Rotary,
    linear,
    qk_norm_rope,
    token_logprobs,
)
