"""moe_forward_few where numbers end: what one expert's weights or one token hold does
not reach the tokens of others."""
import numpy as np
import pytest

from moe_synth import Workload, custom_config
from tests.test_gpu_few import few_layer, needs_gpu, outputs, poison

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-5  # of test_gpu_few.py


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


def fill(t, bits):
    """Fill with fp32 (or, by their upper half, bf16) bits."""
    if t.dtype == torch.float32:
        t.view(torch.int32).fill_(bits - (1 << 32) if bits >> 31 else bits)
    else:
        b = bits >> 16
        t.view(torch.int16).fill_(b - (1 << 16) if b >> 15 else b)


INF, NAN = 0x7F800000, 0x7FC00000

APART = [
    # T, d, E, k, d_ff, w, shared
    (1, 256, 8, 2, 128, "bf16", False),
    (13, 256, 16, 2, 256, "bf16", True),
    (16, 512, 8, 2, 4096, "bf16", False),
    (16, 768, 8, 3, 1408, "fp8_e4m3", True),
    (11, 256, 32, 4, 256, "int8", False),
    (7, 256, 8, 2, 4096, "int4", True),
    (40, 256, 16, 2, 256, "bf16", False),
    (64, 512, 8, 2, 384, "int4", True),
]


@pytest.mark.parametrize("value", [INF, NAN])
@pytest.mark.parametrize("T,d,E,k,d_ff,w,shared", APART)
@pytest.mark.parametrize("which", ["1", "3", "2"])
def test_an_expert_reaches_its_own_tokens_only(moe, T, d, E, k, d_ff, w, shared, value, which):
    """One chosen expert's W1, W3 or W2 (quantised: its scales) is not finite: the tokens
    that chose it are not finite, the others keep their bits."""
    needs_gpu()
    print(f"[few apart] T={T} E={E} {w} W{which} {value:x}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, d, E, k, d_ff, w=w, shared=shared, seed=T + d + E))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev)
    layer(dev["x"])
    ref = outputs(layer)
    e = int(ref["idx"][0, 0])
    fill(dev["weights"][("W" if w == "bf16" else "s") + which][e], value)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    hit = (ref["idx"] == e).any(1)
    assert np.array_equal(out["y"][~hit], ref["y"][~hit])
    assert not np.isfinite(out["y"][hit]).any()
    for n in ("idx", "w", "counts", "offsets"):
        assert np.array_equal(out[n], ref[n]), n


@pytest.mark.parametrize("T,w", [(9, "bf16"), (16, "int4"), (50, "fp8_e4m3")])
def test_a_token_reaches_itself_only(moe, T, w):
    """A token of NaN (its routing is anything) changes nothing beyond a rounding for the
    others: with other experts touched, sums may be cut elsewhere."""
    needs_gpu()
    print(f"[few token apart] T={T} {w}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, 256, 16, 2, 384, w=w, shared=True, seed=T))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev)
    layer(dev["x"])
    ref = outputs(layer)
    fill(dev["x"][T // 2], NAN)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    rest = np.arange(T) != T // 2
    assert np.isnan(out["y"][T // 2]).all()
    assert np.array_equal(out["idx"][rest], ref["idx"][rest])
    rms = np.sqrt((ref["y"].astype(np.float64) ** 2).mean())
    assert np.abs(out["y"][rest] - ref["y"][rest]).max() <= 2 * TOL * rms
