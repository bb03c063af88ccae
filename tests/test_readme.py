"""The README's examples."""
import os
import re

import pytest

import grouped_nf4_w4a16_b200 as gnf4

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def serving_example():
    with open(README) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    return next(b for b in blocks if "gnf4_moe_experts(" in b)


@pytest.mark.parametrize("T,k,H,F,E", [(4, 2, 4096, 14336, 8), (1, 8, 2048, 1024, 64), (32, 4, 2048, 1024, 64),
                                       (32, 1, 4096, 64, 8), (1, 1, 64, 64, 1)])
def test_the_decode_step_s_workspace_serves_each_of_its_calls(T, k, H, F, E, monkeypatch):
    """The statements before the first call size one workspace for all of them."""
    monkeypatch.setattr(gnf4, "make_workspace", lambda nbytes: nbytes)
    names = dict(T=T, k=k, H=H, F=F, E=E, gnf4=gnf4)
    exec(serving_example().split("hidden =")[0], names)
    assert names["ws"] >= gnf4.gnf4_workspace_bytes(gnf4.GNF4_OP_GEMV, T, H)
    assert names["ws"] >= gnf4.gnf4_workspace_bytes(gnf4.GNF4_OP_MOE_ROUTE, T)
    assert names["ws"] >= gnf4.gnf4_workspace_bytes(gnf4.GNF4_OP_MOE_EXPERTS, T * k, 2 * F, H, E)
