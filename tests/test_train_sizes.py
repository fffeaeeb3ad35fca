"""A training step's operators on the host: what the binding keeps, and the sizes
of workspaces."""
from bit_quantized_routed_router_amd import ds4moe as D


def test_the_optimizer_keeps_decays_of_its_own():
    """set_grads lays the table out anew, with the decays that it was made with."""
    given = [0.25]
    opt = D.AdamW([], [], [], [], weight_decay=given)
    given[0] = 9.0
    assert opt.weight_decay.tolist() == [0.25]
    assert D.AdamW([], [], [], [], weight_decay=0.5).weight_decay == 0.5
