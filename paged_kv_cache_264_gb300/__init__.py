"""GB300 (sm_103a) PagedAttention decode: a C-ABI library of hand-written CUDA kernels
(``include/pagedkv.h``, sources in ``csrc/``) and this thin Python binding.

The library is loaded on first use; importing the package does not need a GPU.
"""

from .api import (  # noqa: F401
    BlockManager,
    PagedKVPool,
    copy_blocks,
    decode_plan,
    decode_workspace_bytes,
    gather_cache,
    get_device_error,
    launch_count,
    norm_rope_and_cache,
    paged_attention_decode,
    paged_attention_prefill,
    pool_bytes,
    pool_create,
    pool_destroy,
    prefill_workspace_bytes,
    prompt_attention,
    reserve_slots,
    reshape_and_cache,
    rope_table,
    selftest_bounded_wait,
    shared_prefix_decode,
    shared_prefix_workspace_bytes,
    version,
)
from ._lib import (  # noqa: F401
    BLOCK_SIZE,
    DEVERR_BLOCK_ID,
    DEVERR_CAPACITY,
    DEVERR_CONTEXT_LEN,
    DEVERR_POSITION,
    DEVERR_PREFIX,
    DEVERR_QUERY,
    DEVERR_SLOT,
    DEVERR_TIMEOUT,
    PagedKVError,
)
