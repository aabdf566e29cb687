"""fp64 CPU oracle of the Flash-dLLM fused KV-cache step (test infrastructure only).

Only `tests/`, `__graft_entry__.smoke()` and the benchmark's CPU-baseline and
reference legs may import this package.  The CUDA library never does.
"""
from .fdllm_oracle import (FLAG_ACCEPT, FLAG_COMMIT, FLAG_PASS, accept, attend,
                           attention_mass, bf16_bits, bf16_bits_to_f64, fused_step,
                           project_qkv, rope, round_bf16, round_to, to_f64,
                           track_select, verify_step, verify_visibility)

from .draft_oracle import (ancestors, chain_verify, draw, e4m3_to_f64, quantise_rows,
                           round_e4m3, tree_attend, tree_verify)

__all__ = ["FLAG_ACCEPT", "FLAG_COMMIT", "FLAG_PASS", "accept", "attend", "attention_mass",
           "bf16_bits", "bf16_bits_to_f64", "fused_step", "project_qkv", "rope",
           "round_bf16", "round_to", "to_f64", "track_select", "verify_step",
           "verify_visibility", "ancestors", "chain_verify", "draw", "e4m3_to_f64",
           "quantise_rows", "round_e4m3", "tree_attend", "tree_verify"]
