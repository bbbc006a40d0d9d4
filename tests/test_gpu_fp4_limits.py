"""A matrix of one row has a pitch that leads nowhere: any number that the header allows gives what
the row's own length does."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda"


@pytest.mark.parametrize("m,n,k", [(1, 8200, 4100), (700, 1, 600), (1, 1, 5000), (1, 40, 96)])
def test_the_pitch_of_a_single_row(m, n, k):
    from dlrm_embedding_bag_b200 import fp4, optim

    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    (xq, xs), (wq, ws) = (fp4.quantize_rows(torch.empty((r, k), device=DEV).normal_(0, 1, generator=g))
                          for r in (m, n))
    want = fp4.linear_fp4(xq, xs, wq, ws)
    for pitch in (1 << 20, 1 << 40, 1 << 61):
        y = torch.full((m, n), 9.0, device=DEV)
        rc = optim._lib.dlrm_linear_fp4(
            xq.data_ptr(), pitch if m == 1 else xq.stride(0), xs.data_ptr(), wq.data_ptr(),
            pitch if n == 1 else wq.stride(0), ws.data_ptr(), None, m, n, k, 0, y.data_ptr(), 0,
            pitch if m == 1 else n, None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0, pitch
        torch.cuda.synchronize()
        assert torch.equal(y, want), pitch
