"""moe_adapter_workspace_bytes on the host, and what a layer with adapters refuses there."""
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


def sizes(moe, rows, **kw):
    return [moe.moe_adapter_workspace_bytes(moe.make_adapter_shape(T, **kw)) for T in rows]


@pytest.mark.parametrize("kw", [
    dict(d_in=4096, d_out=4096, n_adapters=8, rank=16),
    dict(d_in=4096, d_out=14336, n_adapters=8, rank=16),
    dict(d_in=7168, d_out=2048, n_adapters=8, rank=64, w_dtype=4),
    dict(d_in=512, d_out=100, n_adapters=3, rank=128),
    dict(d_in=8, d_out=1, n_adapters=1, rank=8),
    dict(d_in=8192, d_out=1 << 15, n_adapters=1, rank=8)])
def test_workspace_serves_smaller_batches(moe, kw):
    """Never smaller for more rows: a workspace for the largest batch is enough for every
    smaller one, whatever parts the products of those are cut into."""
    rows = [*range(0, 1100), *range(1100, 9000, 37), *range(9000, 1 << 20, 4999), 1 << 20]
    rows = [T for T in rows if T * kw["d_out"] <= 1 << 37]
    got = sizes(moe, rows, **kw)
    assert got[0] > 0
    down = [(a, b) for a, b, x, y in zip(rows, rows[1:], got, got[1:]) if y < x]
    assert not down, down[:5]


def test_layer_refuses_adapters_of_another_device(moe):
    """A kernel would follow their addresses."""
    ok = dict(A=torch.zeros(2, 16, 64, dtype=torch.bfloat16),
              B=torch.zeros(2, 64, 16, dtype=torch.bfloat16), scales=torch.zeros(2),
              ranks=torch.zeros(2, dtype=torch.int32))

    def layer(**kw):
        return moe.MoELayer(3, 64, 4, 2, 128, W_g=None, weights={}, device="cpu",
                            pack_router=False, adapters={**ok, **kw})

    for name in ok:
        with pytest.raises(ValueError, match="device"):
            layer(**{name: ok[name].to("meta")})
    with pytest.raises(ValueError, match="device"):
        layer()(torch.zeros(3, 64, dtype=torch.bfloat16),
                adapter_idx=torch.zeros(3, dtype=torch.int32, device="meta"))
    assert layer(ranks=None).adapters["ranks"] is None
