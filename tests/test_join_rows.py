"""``KANJoin`` takes rows of its own width alone (no GPU: the refusal comes first)."""

import pytest
import torch

import kolmogorov_arnold_network_amd as kan


@pytest.mark.parametrize("features,shape", [(6, (5, 4, 12)), (12, (4, 6)), (6, (5, 18)), (4, (3, 4, 1)), (5, (5,) * 0),
                                            (1, (7, 3)), (6, (0, 12))])
@pytest.mark.parametrize("pre", [True, False])
def test_rows_of_another_width_are_refused(features, shape, pre):
    join = kan.KANJoin(features, pre=pre)
    h = torch.zeros(shape)
    with pytest.raises(ValueError, match="features"):
        join(h)
    with pytest.raises(ValueError, match="features"):
        join(h, residual=h.clone(), gate=h.clone())
