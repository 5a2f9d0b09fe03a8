"""The distillation's workspace: few long rows need one in the step alone."""

import pytest

from kan_testutil import ensure_built


def test_only_a_step_of_few_long_rows_needs_one():
    ensure_built()
    from kolmogorov_arnold_network_amd import _lib as L

    def size(N, V):
        return L.lib().kan_distill_workspace_size(L.kan_distill_desc_t(N, V, 8, V, V, 0, 0, 1, 0, 1.0))

    assert size(4, 131072) >= 4 * 2 * 8 and size(65, 131072) == 0 and size(4, 32003) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 4, 64])
def test_forward_of_long_rows_without_a_workspace(N):
    ensure_built()
    import torch
    from kolmogorov_arnold_network_amd import _lib as L
    from kolmogorov_arnold_network_amd import functional as F
    V = 131072
    torch.manual_seed(N)
    z, t = torch.randn(N, V, device="cuda:0"), torch.randn(N, 8, device="cuda:0")
    ids = torch.randint(0, V, (N, 8), device="cuda:0")
    desc = F.distill_desc(z, ids, t, 1.0)
    n = F.kan_distill_workspace_size(desc)
    assert n > 0
    want = F.kan_distill_forward(z, ids, t)
    loss, lse = torch.empty(N, device="cuda:0"), torch.empty(N, device="cuda:0")
    stream = torch.cuda.current_stream().cuda_stream
    args = [desc, z.data_ptr(), ids.data_ptr(), t.data_ptr(), None, loss.data_ptr(), lse.data_ptr(), None, 0, stream]
    assert L.lib().kan_distill_forward(*args) == L.KAN_OK
    torch.cuda.synchronize()
    assert torch.equal(loss, want[0]) and torch.equal(lse, want[1])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda:0"), n          # one that is given stays untouched
    ws[0].fill_(77)
    assert torch.equal(F.kan_distill_forward(z, ids, t, ws=ws)[0], loss) and bool((ws[0] == 77).all())
    dz = torch.empty(N, V, device="cuda:0")
    args[5:8] = loss.data_ptr(), dz.data_ptr(), None
    assert L.lib().kan_distill_step(*args) == L.KAN_ERR_WORKSPACE
