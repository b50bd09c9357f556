"""MI355X (gfx950) chunked gated delta rule with dynamic state/W fake QDQ.

The computation runs in hand-written HIP kernels (csrc/) behind the C ABI in
include/gdn.h; binding.py marshals torch device tensors into that ABI.
"""
from .binding import (GDN_BF16, GDN_F32, QDQ_E4M3, QDQ_INT8, QDQ_OFF, READOUT_AFTER_WRITE,  # noqa: F401
                      READOUT_BEFORE_WRITE, SCALE_DIVIDE, SCALE_RECIPROCAL, GdnError, StatePool, device_errors,
                      gdn_beam_advance, gdn_beam_select, gdn_chunk_bwd, gdn_chunk_fwd, gdn_decode_bwd,
                      gdn_decode_fwd, gdn_pool_copy, gdn_pool_prefill, gdn_pool_read,
                      gdn_pool_reorder, gdn_pool_step, gdn_pool_write, gdn_prefill_decode_bwd,
                      gdn_prefill_decode_fwd, gdn_qdq_state, load_library, make_fwd_args,
                      saved_layout)
