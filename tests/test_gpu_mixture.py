"""The small mixture-of-experts model learns its table with the library's routing and follows it when sampled."""
import math

import pytest

pytestmark = pytest.mark.gpu


def test_a_model_learns_and_answers(pk, cuda_device):
    from streaming_selection_primitive_gb300 import mixture
    vocab = 256
    got = mixture.run(steps=150, batch=1024, vocab=vocab, width=32, experts=8, k=2, sequences=16, length=16)
    # The table's entropy: 0.9 of one token, and 0.1 spread over all.
    one = 0.9 + 0.1 / vocab
    entropy = -one * math.log(one) - (vocab - 1) * 0.1 / vocab * math.log(0.1 / vocab)
    assert got["loss"][0] > 4 and got["loss"][1] < entropy + 0.5
    # 1: an even choice; 4: always the same two experts of eight, evenly.
    assert 0.99 < got["balance_loss"][1] < 1.5
    # Trained, the table's token has nearly all of the mass that the filters leave.
    assert got["followed"] > 0.8 and got["mean_logprob"] > -0.5
