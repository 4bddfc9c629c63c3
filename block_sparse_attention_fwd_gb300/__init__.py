"""GB300-native BackLite attention: exact forward with per-tile LSE statistics,
tile selection (mask_from_stats) and a block-sparse backward.

The compute lives in ``libbl_attn.so`` (hand-written sm_103a CUDA behind the C
ABI in ``include/bl_attn.h``); this package only marshals arguments.  The
library is loaded on first use and a missing library raises.
"""
from . import _lib  # noqa: F401
from ._lib import (BLError, alloc_lists, attn_bwd, attn_fwd, bwd_check_status,  # noqa: F401
                   bwd_workspace_bytes, make_shape, mask_from_stats, tile_stats_elems, tiles)
from .api import (BLAttention, BLDropout, BLLayerNorm, BLLinear8, BLRMSNorm,  # noqa: F401
                  Rotary)
from .linear import (Cols8, Weight8, act_save_both, dropout, dropout_next,  # noqa: F401
                     layer_norm_bwd, layer_norm_fwd, layer_norm_fwd_8bit, matmul8, matmul8_gw,
                     matmul8_gx, weight_save)
from .ops import (Act8, RopePlan, act_load, act_save, attn_bwd_act8,  # noqa: F401
                  attn_bwd_act8_workspace_bytes, grid_positions, rms_norm_bwd, rms_norm_fwd,
                  rms_norm_fwd_8bit, rope)
