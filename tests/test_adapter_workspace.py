"""moe_adapter_workspace_bytes on the host: empty batches."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.cpu


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


@pytest.mark.parametrize("d_in,d_out,n,rank", [(256, 256, 2, 16), (8, 1, 1, 8),
                                               (4096, 1 << 20, 5, 128)])
def test_no_rows_need_a_workspace_all_the_same(moe, d_in, d_out, n, rank):
    sh = moe.make_adapter_shape(0, d_in, d_out, n, rank)
    assert moe.moe_adapter_workspace_bytes(sh) == 256
    assert moe.adapter_workspace(sh, "cpu").numel() == 256


@pytest.mark.parametrize("few", [False, True])
def test_layer_of_no_tokens_with_adapters(moe, few):
    ad = dict(A=torch.zeros(2, 16, 64, dtype=torch.bfloat16),
              B=torch.zeros(2, 64, 16, dtype=torch.bfloat16), scales=torch.zeros(2))
    layer = moe.MoELayer(0, 64, 4, 2, 128, W_g=None, weights={}, device="cpu", pack_router=False,
                         few=few, adapters=ad)
    assert layer.adapter_ws.numel() == 256 and layer.y.shape == (0, 64)
