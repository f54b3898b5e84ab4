"""HiSparse swap-in path for MI355X (gfx950): HIP kernels behind a C ABI, with a thin Python binding.

Importing the package loads the built HIP library and raises ImportError if it is missing; nothing here
falls back to another implementation.
"""
from .hisparse import (EXPORTED, HS_EVICT_FIFO, HS_EVICT_LRU, HS_E_HIP, HS_E_INVALID, HS_E_NOMEM, HS_E_STATE, HS_OK, HS_STATUS_BAD_ID,
                       HS_STATUS_BAD_STATE, HS_STATUS_DUP_ID, HS_STATUS_STALE, HiSparseError, HsConfig, HsDeviceViews, HsSizes, SwapIn,
                       config, config_from_hisparse_json, hs_bind_device, hs_create, hs_destroy, hs_gather,
                       hs_host_pool, hs_last_error, hs_plan, hs_step_static, HS_STATIC_PLAN_BYTES, hs_export_state, hs_import_state, HS_STATE_TABLES, HS_STATE_ROWS, hs_copy, hs_trial, hs_commit, hs_offload, hs_advance_tail, hs_rebuild_order, hs_required_sizes, hs_reset, hs_resolve, lib,
                       library_path, HS_ROW_BF16, HS_ROW_MXFP8, HS_ROPE_PAIRS, HS_ROPE_HALVES, HsRowFormat, row_format,
                       hs_row_bytes, hs_map_tokens, hs_store_rows, hs_attend_work_bytes, hs_attend, hs_attend_prompt_work_bytes, hs_attend_prompt,
                       HS_NORM_NONE, HS_NORM_RMS, HS_NORM_LAYER, HS_KEY_MXFP8, HS_KEY_MXFP4, HsHeadFormat, HsKeyFormat, head_format,
                       key_format, key_parts, hs_norm_rotate, hs_key_bytes, hs_store_keys, hs_score_keys, hs_select_work_bytes, hs_select)

lib()
