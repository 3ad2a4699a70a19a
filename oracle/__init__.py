"""CPU oracle for exact attention (test infrastructure only; see attention.py)."""
from .attention import (  # noqa: F401
    attention,
    attention_rows,
    bf16_round,
    flash_fa1,
    flash_fa2,
    naive_bf16_attention,
    safe_softmax,
)
from .backward import (  # noqa: F401
    attention_bwd,
    attention_bwd_heads,
    attention_bwd_recompute,
    naive_bf16_attention_bwd,
)
from .packed import (  # noqa: F401
    attention_packed,
    attention_packed_bwd,
    attention_prefix,
    masked_head,
)
from .cache import (  # noqa: F401
    append_pages,
    attention_paged,
    least_scale,
    rotate,
    round_e4m3,
)
from .gqa import (  # noqa: F401
    attention_gqa,
    attention_gqa_rows,
    attention_split,
    merge_partials,
)
