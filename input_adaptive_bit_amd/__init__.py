"""MI355X-native decode-phase GEMV of GRINQH (input-adaptive bit widths).

The product is libgrinqh.so (HIP kernels for gfx950 behind the C ABI in
include/grinqh.h); this package holds its sources (csrc/), the in-tree build
script (build.py) and the ctypes binding (grinqh.py).
"""

from .grinqh import (  # noqa: F401
    GRINQH_BF16, GRINQH_F32, GrinqhError, Layout, EXPORTS, load, status_string,
    grinqh_layout_init, grinqh_packed_bytes, grinqh_gemv_workspace_bytes,
    grinqh_pack, grinqh_assign_bits, grinqh_gemv, grinqh_debug_codes,
    grinqh_debug_force_launch, force_launch_shape, grinqh_gemv_noalloc, NOALLOC_SCRATCH_BYTES,
    grinqh_gemv_group_workspace_bytes, grinqh_gemv_group, Operands, MAX_GROUP,
    new_workspace, new_group_workspace, pack, assign_bits, gemv, debug_codes,
    grinqh_calibrate_workspace_bytes, grinqh_calibrate_thresholds, calibrate_thresholds,
    grinqh_quantize_rtn, quantize_rtn,
    grinqh_prefill_workspace_bytes, grinqh_prefill_gemm, prefill_gemm,
)
from .attention import (  # noqa: F401
    KVLayout, KVCache, grinqh_kv_layout_init, grinqh_kv_code_bytes, grinqh_kv_grid_bytes, grinqh_kv_write,
    grinqh_kv_read, grinqh_debug_kv_row, grinqh_debug_page_row, grinqh_attention_workspace_bytes, grinqh_decode_attention,
    grinqh_prefill_attention, grinqh_prefill_attention_workspace_bytes, new_kv_cache, new_attention_workspace, kv_write, kv_read, decode_attention,
    prefill_attention,
)
from .fourbit import (  # noqa: F401
    FourbitLayout, FourbitWeight, grinqh_fourbit_layout_init, grinqh_fourbit_code_bytes, grinqh_fourbit_grid_bytes,
    grinqh_fourbit_pack, grinqh_fourbit_linear, grinqh_expert_linear, fourbit_pack, fourbit_quantize, fourbit_linear,
    expert_linear,
)
from .rope import grinqh_qk_rope, qk_rope  # noqa: F401
from .pages import (  # noqa: F401
    Step, grinqh_kv_extend_workspace_bytes, grinqh_kv_extend, grinqh_kv_release, new_page_list, kv_extend, kv_release,
)
