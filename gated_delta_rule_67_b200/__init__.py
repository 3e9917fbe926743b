"""B200-native Kimi Delta Attention (KDA): C-ABI CUDA library + thin Python binding.

    kda_chunk_fwd(q, k, v, g, beta, scale, initial_state) -> (o, final_state)
    kda_recurrent_step(q, k, v, g, beta, state, scale) -> o   (state updated in place)
    kda_backward(q, k, v, g, beta, grad_o, scale, initial_state, grad_final_state) -> gradients
    kda_scan_fwd(x, g, initial_state) -> (h, final_state)     the elementwise gated linear recurrence
    kda_scan_step(x, g, state) -> h                           (state updated in place)
    kda_scan_backward(x, g, h, grad_h, ...), kda_scan_backward_ckpt(checkpoint, grad_h, ...) -> gradients

The compiled library (libkda.so, built by ``build.build()``) does all the
work; the binding only marshals arguments.  It is loaded on first use.
"""
from .binding import (KDAError, kda_backward, kda_chunk_fwd, kda_chunk_fwd_check, kda_chunk_fwd_launch_count,
                      kda_chunk_fwd_workspace_size, kda_recurrent_step, kda_scan_backward, kda_scan_backward_ckpt,
                      kda_scan_checkpoint_size, kda_scan_fwd, kda_scan_step, kda_scan_workspace_size, load,
                      status_string, version)

__all__ = ["KDAError", "kda_backward", "kda_chunk_fwd", "kda_chunk_fwd_check", "kda_chunk_fwd_launch_count",
           "kda_chunk_fwd_workspace_size", "kda_recurrent_step", "kda_scan_backward", "kda_scan_backward_ckpt",
           "kda_scan_checkpoint_size", "kda_scan_fwd", "kda_scan_step", "kda_scan_workspace_size", "load",
           "status_string", "version"]
