"""Balance loss over more sequences than two rounds of the search for a window's
first sequence cover (64 places a round: 4096), most of them empty."""
import pytest
import torch

from test_gpu_balance_loss import check, draw

pytestmark = pytest.mark.gpu


# three rounds from 4097 sequences on, four from 262145 on
@pytest.mark.parametrize("n_seq,T,E", [(4096, 3000, 16), (4097, 3000, 16), (6000, 20000, 5),
                                       (300000, 900, 4)])
def test_more_sequences_than_two_rounds_cover(n_seq, T, E):
    g = torch.Generator().manual_seed(90)
    cuts = torch.randint(0, T - 20, (n_seq - 1,), generator=g).sort().values
    # a long run of empty sequences inside a window, and tokens in no sequence at both ends
    cuts[n_seq // 3:n_seq // 2] = cuts[n_seq // 3].item()
    offsets = [3] + cuts.clamp(min=3).tolist() + [T - 7]
    assert offsets == sorted(offsets) and len(offsets) == n_seq + 1
    check(*draw(T, E, 2, 91, 0.6, 0.2), offsets)
