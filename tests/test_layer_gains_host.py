"""A layer's q / k gains come together, and the backward takes those of its forward: a call that would
drop one, or differentiate another layer than the forward's, is refused before anything runs."""
import pytest
import torch

from shared_prefix_grouped_gb300 import layer, rollout

KW = dict(heads_q=2, heads_kv=1, head_dim=64, rope_theta=1e4, eps=1e-5)
X, G = torch.zeros((3, 8)), torch.ones(64)
W = (None,) * 6


@pytest.mark.parametrize("gains", [dict(g_q=G), dict(g_k=G)], ids=["q", "k"])
def test_one_gain_is_refused(gains):
    calls = [lambda: layer.layer_fwd(None, X, *W, **KW, **gains),
             lambda: layer.layer_bwd(None, X, *W, dict(q_in=X, k_in=X), X, **KW, **gains),
             lambda: rollout.layer_prefill(None, None, X, *W, None, None, rope_theta=1e4, eps=1e-5, **gains),
             lambda: rollout.layer_decode(None, X, *W, None, None, rope_theta=1e4, eps=1e-5, **gains)]
    for call in calls:
        with pytest.raises(ValueError, match="g_q and g_k come together"):
            call()


def test_gains_of_another_forward_are_refused():
    with pytest.raises(ValueError, match="forward"):      # the forward normed, the backward would not
        layer.layer_bwd(None, X, *W, dict(q_in=X, k_in=X), X, **KW)
    for saved in (dict(q_in=None, k_in=None), {}):        # and the other way round
        with pytest.raises(ValueError, match="forward"):
            layer.layer_bwd(None, X, *W, saved, X, **KW, g_q=G, g_k=G)
