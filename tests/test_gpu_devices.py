"""Calls of the delta rule with another device current: refused, nothing is
launched."""

import pytest

torch = pytest.importorskip("torch")

from linear_attention_sequence_chunked_gb300 import gdn  # noqa: E402

pytestmark = pytest.mark.gpu


def test_every_wrapper_refuses_another_device(monkeypatch):
    q, v = (torch.zeros(1, 64, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g, beta = torch.zeros(1, 64, 2, device="cuda"), torch.zeros(1, 64, 2, dtype=torch.bfloat16, device="cuda")
    gk = torch.zeros(1, 64, 2, 64, device="cuda")
    monkeypatch.setattr(gdn, "_device", lambda: 1)
    launches = gdn.gdn_kernel_launches()
    for call in (lambda: gdn.chunk_gated_delta_rule_fwd(q, q, v, g, beta),
                 lambda: gdn.chunk_gated_delta_rule_bwd(q, q, v, g, beta, v),
                 lambda: gdn.chunk_gated_delta_rule_fwd_split(q, q, v, g, beta, 1),
                 lambda: gdn.chunk_kda_fwd(q, q, v, gk, beta), lambda: gdn.chunk_kda_bwd(q, q, v, gk, beta, v),
                 lambda: gdn.chunk_gated_delta_rule(q, q, v, g, beta)):
        with pytest.raises(ValueError, match="current device is cuda:1"):
            call()
    assert gdn.gdn_kernel_launches() == launches
