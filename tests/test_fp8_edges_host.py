"""Block-128 FP8 operators and block norms on the host: constants, buffers, workspaces and plans at their edges."""
import ctypes

import pytest
import torch

B = pytest.importorskip("mxfp4_routed_expert_amd.binding", reason="libmoe.so not built (python mxfp4_routed_expert_amd/build.py)")
lib = B.lib


# ------------------------------------------------------------------ constants of the norms

@pytest.mark.parametrize("name", ["eps", "residual_scale", "dropout"])
def test_norm_constants_are_read_at_each_call(name):
    """A tensor (or parameter) may change between calls: its value counts, not the object."""
    for value in (torch.tensor(0.5), torch.nn.Parameter(torch.tensor(0.5)), torch.tensor([0.5], dtype=torch.float64)):
        kw = dict(eps=1e-6, residual_scale=1.0, dropout=0.0)
        kw[name] = value
        got = []
        for v in (0.5, 0.125):
            with torch.no_grad():
                value.fill_(v)
            got.append(getattr(B._norm_desc(4, 64, 0, 0, 0, **kw)[0]._obj, name))
        assert got == [0.5, 0.125]


def test_norm_constants_of_every_kind():
    d = B._norm_desc(4, 64, 0, 0, 0, 1e-6, -0.0, 0.0)[0]._obj
    assert str(d.residual_scale) == "0.0" and d.eps == ctypes.c_float(1e-6).value
    assert B._norm_desc(4, 64, 0, 0, 0, 1, True, 0)[0]._obj.residual_scale == 1.0
    for bad in ("0.5", None, torch.tensor([1.0, 2.0])):
        with pytest.raises((TypeError, ValueError)):
            B._norm_desc(4, 64, 0, 0, 0, 1e-6, bad, 0.0)
