"""The cache's wrappers refuse tensors whose memory is not what their shape says (no GPU needed)."""
import pytest
import torch

import ternary_weight_fwd_b200 as tw
from test_kv_host import cpu_args


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 30),
                                       torch.zeros(1 << 16, dtype=torch.uint8)[::2]], ids=["expanded", "every other"])
def test_workspace_must_be_contiguous(monkeypatch, workspace):
    (k, v, ks, vs), (table, lens, starts) = cpu_args()
    q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(tw, "_kv_views", lambda *a: (tw.bitnet_kv_cache_t(), tw.bitnet_kv_batch_t()))
    with pytest.raises(ValueError, match="contiguous"):
        tw.bitnet_attention((k, v, ks, vs), table, lens, starts, q, 1, out=torch.zeros_like(q), workspace=workspace)
