"""The README's Python lines use nothing that neither they nor their user makes (CPU)."""

import ast
import builtins

import readme_code

# what a user has in hand: matrices, activations, the router's logits, and a training step's gradients
GIVEN = {"x_fp16", "w_q4_0", "w_q6_k", "topk_ids", "w13", "w2", "s13", "s2", "x_bf16", "router_logits", "bias", "I", "shared_expert_row",
         "a", "b", "s", "offsets", "dy", "g", "a1", "b1", "request_adapter"}


def test_every_name_is_made_or_given():
    known = set(GIVEN) | set(dir(builtins))
    for node in ast.parse(readme_code.block()).body:
        if isinstance(node, ast.Import):
            known |= {a.asname or a.name for a in node.names}
            continue
        used = {n.id for n in ast.walk(node) if isinstance(n, ast.Name) and isinstance(n.ctx, ast.Load)}
        assert used <= known, f"line {node.lineno}: {sorted(used - known)}"
        known |= {n.id for n in ast.walk(node) if isinstance(n, ast.Name) and isinstance(n.ctx, ast.Store)}


def test_the_router_is_differentiated_as_it_was_called():
    calls = {}
    for node in ast.walk(ast.parse(readme_code.part("FP8") + readme_code.part("adapters"))):
        if isinstance(node, ast.Call) and isinstance(node.func, ast.Attribute):
            calls.setdefault(node.func.attr, {k.arg: ast.dump(k.value) for k in node.keywords})
    gate = calls["moe_gate"]
    for name in ("score", "renormalize", "scale"):
        assert calls["moe_gate_backward"].get(name) == gate.get(name), name
    assert calls["moe_balance_loss"].get("score") == gate.get("score")
