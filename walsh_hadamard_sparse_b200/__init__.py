"""B200 (sm_100a) Walsh-Hadamard adapter layer: Python binding of libqwha.

The arithmetic runs in the CUDA kernels of libqwha.so; this package only
marshals torch tensors (device memory and the current stream) into the C ABI
of include/qwha.h. Import fails if the library is not built.
"""

from ._lib import QwhaError, lib  # noqa: F401
from .api import (  # noqa: F401
    DECODE_MAX_T,
    Adapter,
    PageTable,
    QCache,
    QWeight,
    adapter_bwd,
    adapter_decode,
    adapter_fwd,
    cache_alloc,
    cache_attention,
    cache_compact,
    cache_copy_pages,
    cache_read,
    cache_write,
    calib_hessian,
    check_stream_status,
    dp_backward,
    dp_step,
    energy_stats,
    fwht,
    init_alloc,
    init_alloc_sharded,
    init_budgets,
    init_norms,
    init_select,
    init_select_global,
    page_table,
    pages_fork,
    pages_resize,
    pattern_stats,
    plan_build,
    plan_tiles,
    qgemv,
    refine_values,
    rotary,
    rotary_frequencies,
    shard_rows,
    stage_report,
    stage_timing,
    validate_plan,
    validate_slots,
    workspace_size,
)

lib()  # fail loudly at import when libqwha.so is missing
