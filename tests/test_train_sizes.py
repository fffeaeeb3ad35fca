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


def test_xent_workspace_of_the_most_rows():
    """ds of 2048 words, beside rows of h's size and fp32 sums of dh's, and 256 MB
    of w's parts: what the header says of a call of many rows."""
    d = 256
    for dt, size in ((D.DT_BF16, 2), (D.DT_F32, 6)):  # fp32 in three parts
        for T in (1 << 18, 1 << 20):
            ds, rows = 2048 * T * size, (size + 4 + 1) * T * d
            assert ds <= D.xent_workspace_bytes(dt, T, 1 << 20, d, True) <= ds + rows + (1 << 28)
            # a vocabulary below a piece has no more than its own
            assert D.xent_workspace_bytes(dt, T, 300, d, True) <= 512 * T * size + rows + (1 << 28)
    # up to so many rows ds stays within 256 MB
    for dt, size, T in ((D.DT_BF16, 2, 65536), (D.DT_F32, 6, 21845)):
        most = (1 << 28) + (size + 4 * 32) * T * d + (1 << 28) * (size == 6)
        assert D.xent_workspace_bytes(dt, T, 1 << 20, d, True) <= most
