"""Float64 CPU oracle of the routed-expert layer (test infrastructure only).

Importable by ``tests/``, ``__graft_entry__.smoke()`` and the CPU-baseline
leg of ``bench.py``; never by the library.
"""
from .moe_oracle import (  # noqa: F401
    bf16_to_f64, f16_to_f64, q3_fields, q3_pack, q3_dequant, expert_matrices,
    router_logits, route_topk, expert_histogram, permute, silu, expert_ffn, grouped_ffn,
    combine, moe_layer, dense_layer, rel_max_err,
    e4m3_to_f64, f64_to_e4m3, fp8_block_scale, quantize_fp8, fp8_values, fp8_expert_ffn,
    balance_loss, softmax_row, route_backward, combine_backward,
)
