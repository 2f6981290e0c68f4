"""Which continuation of two the small model's preference steps prefer (no GPU)."""
import torch


def test_the_better_one_first_and_equal_ones_left_out(pk):
    from streaming_selection_primitive_gb300.mixture import preferred
    tokens = torch.arange(24) + 100
    inputs = torch.arange(24)
    reward = torch.tensor([[1, 1, 0], [0, 1, 0],  # the first is better
                           [0, 0, 1], [1, 1, 1],  # the second
                           [1, 0, 1], [0, 1, 1],  # the same score
                           [0, 0, 0], [0, 0, 0]]).float().flatten()
    got_inputs, got_tokens, apart = preferred(inputs, tokens, reward, 4, 3)
    order = [0, 1, 2, 3, 4, 5, 9, 10, 11, 6, 7, 8]
    assert got_tokens.tolist() == [100 + i for i in order] + [-1] * 12 and got_inputs[:12].tolist() == order
    assert apart.tolist() == [True, True, False, False]
