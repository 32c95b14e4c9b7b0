"""The dense layer's two appends are called alike."""
import inspect

import pytest


def test_both_appends_take_the_same_arguments_in_the_same_order():
    import deepseek_sparse_mla_gb300 as dsa
    kinds = [[(p.name, p.kind, p.default) for p in inspect.signature(f).parameters.values()] for f in (dsa.kv8_append, dsa.kv4_append)]
    assert kinds[0] == kinds[1]
    assert [name for name, kind, _ in kinds[0] if kind is inspect.Parameter.POSITIONAL_OR_KEYWORD] == ["cache", "batch", "k", "v", "stream"]


@pytest.mark.parametrize("name", ["kv8_append", "kv4_append"])
def test_a_rope_and_queries_go_by_name(name):
    """What stands fifth is a stream in both: nothing else is taken for one."""
    import deepseek_sparse_mla_gb300 as dsa
    from types import SimpleNamespace
    import torch
    cache = SimpleNamespace(k_codes=torch.zeros(1), kv_heads=1)
    rope = dsa.RotaryTable.__new__(dsa.RotaryTable)
    with pytest.raises(AttributeError, match="RotaryTable"):
        getattr(dsa, name)(cache, None, None, None, rope)
    with pytest.raises(TypeError):
        getattr(dsa, name)(cache, None, None, None, None, rope)
