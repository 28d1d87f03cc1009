"""MI355X (gfx950) HIP library for the Mamba-2 SSD hot path.

Behind a C ABI (``include/ssd_mi355x.h``):

* ``ssd_chunk_scan_fwd`` -- the SSD chunked selective scan (four-step block
  decomposition of the semiseparable sequence map).
* ``ssd_verify_step`` -- the K-token recurrent update a target model runs when it
  verifies speculative-decoding drafts, keeping the state at the accepted
  position (and optionally at every position).
* ``ssd_gated_delta_step`` / ``_fwd`` / ``_bwd`` -- the gated delta rule, a recurrence of
  the same layout, token by token and in chunks, with its gradients.
* ``ssd_gated_scan_step`` / ``_fwd`` / ``_bwd`` -- the gated scan, a recurrence of one number
  per channel with a gate per token, likewise.
* ``ssd_norm_gate_*`` / ``ssd_norm_add_*`` -- the norms after and before a mixer block,
  fused with its gate and with the residual sum, with their gradients; the latter also with
  dropout (``ssd_norm_add_drop_*``) and with an 8-bit output (``ssd_norm_add_q8_fwd``).

The Python binding (``selective_state_space_ssd_amd.binding``) only marshals
torch tensors into the C calls; every step runs in the HIP kernels.  Importing
this package loads nothing; the shared library is opened on first use and a
missing library is an error, never a fallback.
"""

__version__ = "0.1.0"
