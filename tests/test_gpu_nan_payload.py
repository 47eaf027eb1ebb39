"""A NaN of any bits in a scale or a bias is a NaN in the outputs it belongs to: the
terms that fp32 values are split into must not lose it (a NaN whose fraction is all ones
carries out of the exponent when it is rounded as a number)."""
import numpy as np
import pytest

from moe_synth import Workload, custom_config
from tests.test_gpu_adapter import Case
from tests.test_gpu_few import few_layer, needs_gpu, outputs, poison
from tests.test_gpu_few_edges import fill

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

NANS = [0xFFFFFFFF, 0x7FFFFFFF, 0x7FC00000, 0xFF800001]


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("T,w", [(1, "bf16"), (40, "bf16"), (40, None), (100, "bf16"),
                                 (100, None), (2600, "bf16")])
def test_adapter_scale(moe, T, w, bits):
    needs_gpu()
    print(f"[adapter NaN] T={T} {w} {bits:x}", flush=True)
    c = Case(T, 320, 4096 if T > 1000 else 200, 4, 16, w=w, y="f32")
    c.idx[0] = 2
    clean = c.run(moe)
    fill(c.scales[2], bits)
    got = c.run(moe)
    hit = (c.idx == 2).numpy()
    assert np.isnan(got[hit]).all()
    assert np.array_equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("T", [5, 16, 33])
@pytest.mark.parametrize("which", ["s1", "s3", "s2"])
def test_few_scale(moe, T, bits, which):
    needs_gpu()
    print(f"[few NaN] T={T} {which} {bits:x}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, 256, 8, 2, 256, w="int8", seed=T))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev)
    layer(dev["x"])
    idx = outputs(layer)["idx"]
    fill(dev["weights"][which][int(idx[0, 1])], bits)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    hit = (idx == idx[0, 1]).any(1)
    assert np.isnan(out["y"][hit]).all() and np.isfinite(out["y"][~hit]).all()


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("T", [5, 16, 33])
def test_few_router_bias(moe, T, bits):
    """Every routing weight is NaN, so is y; the experts are still experts."""
    needs_gpu()
    print(f"[few NaN bias] T={T} {bits:x}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, 256, 8, 2, 256, router_bias="zipf1.5", seed=T))
    dev = upload(wl)
    fill(dev["b_g"], bits)
    layer = few_layer(moe, wl, dev)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    assert np.isnan(out["w"]).all() and np.isnan(out["y"]).all()
    assert ((out["idx"] >= 0) & (out["idx"] < 8)).all() and out["counts"].sum() == 2 * T


@pytest.mark.parametrize("bits", NANS)
@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("T", [7, 33])
def test_few_gate(moe, T, pack, bits):
    """One NaN in the gate, packed or as it is: that expert's logits are NaN."""
    needs_gpu()
    print(f"[few NaN gate] T={T} pack={pack} {bits:x}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, 256, 4, 4, 256, seed=3))
    dev = upload(wl)
    fill(dev["W_g"][17, 2], bits)
    layer = few_layer(moe, wl, dev, pack_router=pack)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    assert np.isnan(out["w"]).all() and np.isnan(out["y"]).all()
