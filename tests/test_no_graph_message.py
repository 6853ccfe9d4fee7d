"""What a caller reads who gives an operator an operand that requires a gradient (CPU only)."""
import pytest
import torch

import nvfp4_block_scaled_elem_amd as nv
from nvfp4_block_scaled_elem_amd.layer import _no_graph


def test_refusal_names_every_gradient_that_there_is():
    """Each operator's gradient by its own name, and which have none."""
    t = torch.ones(2, requires_grad=True)
    with pytest.raises(nv.NVFP4Error, match="no autograd graph") as e:
        _no_graph(None, t)
    for name in ("rms_norm_grad", "linear_grad", "rotary", "inverse=True", "attention", "kv_append", "moe"):
        assert name in str(e.value)
        assert "=" in name or hasattr(nv, name)
    with torch.no_grad():
        _no_graph(t)
    _no_graph(t.detach())
