"""moe_forward_few's own selection (up to 16 tokens) and the route it takes above, at the
edges of the rules: equal logits, equal groups, signed zeros, infinities; and whole
layers at their full widths against the float64 oracle.

The logits are set exactly: x is zero, so l = b_g whatever the gate."""
import numpy as np
import pytest

import oracle
from moe_synth import Workload, custom_config
from perf import operators as cases
from tests.test_gpu_few import few_layer, needs_gpu, outputs, poison

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 2e-5  # of test_gpu_few.py


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


def select(moe, logits, T, k, groups=0, topk_groups=0):
    """The routing of T tokens that all have these logits."""
    E = len(logits)
    wl = Workload(custom_config(T, 64, E, k, 128, seed=E))
    from moe_synth.device import upload
    dev = upload(wl)
    dev["b_g"] = torch.tensor(np.asarray(logits, np.float32), device="cuda")
    layer = few_layer(moe, wl, dev, n_groups=groups, topk_groups=topk_groups)
    poison(layer)
    layer(torch.zeros_like(dev["x"]))
    return outputs(layer)


def logits_of(kind, E, rng):
    if kind == "equal":
        return np.full(E, 0.25)
    if kind == "zeros":          # -0 equals +0
        return np.where(rng.random(E) < 0.5, -0.0, 0.0)
    if kind == "few values":     # many ties, in every lane and register
        return rng.integers(-2, 3, E) * 0.5
    if kind == "tie at the end":
        v = -np.arange(E, dtype=np.float64)
        v[E // 2:] = v[E // 2]
        return v
    v = rng.standard_normal(E)   # some at the type's lowest value, some at minus infinity
    v[rng.random(E) < 0.3] = np.finfo(np.float32).min
    v[rng.random(E) < 0.3] = -np.inf
    v[E - 1] = 1.0
    return v


@pytest.mark.parametrize("kind", ["equal", "zeros", "few values", "tie at the end", "masked"])
@pytest.mark.parametrize("E,k,G,M", [(1, 1, 0, 0), (8, 2, 0, 0), (64, 8, 8, 3), (65, 7, 0, 0),
                                     (256, 8, 8, 4), (300, 32, 0, 0), (1024, 16, 64, 5),
                                     (1000, 3, 0, 0)])
@pytest.mark.parametrize("T", [1, 16, 33])
def test_few_takes_the_lowest_of_equals(moe, T, E, k, G, M, kind):
    needs_gpu()
    print(f"[few ties] T={T} E={E} k={k} G={G} {kind}", flush=True)
    l = logits_of(kind, E, np.random.default_rng(E + k)).astype(np.float32)
    out = select(moe, l, T, k, G, M)
    # largest first, equal values by index; groups by their largest, equal groups by index
    pick = l.astype(np.float64) + 0.0
    if G:
        best = pick.reshape(G, -1).max(1)
        kept = sorted(range(G), key=lambda g: (-best[g], g))[:M]
        allowed = [e for e in range(E) if e // (E // G) in kept]
    else:
        allowed = range(E)
    want = sorted(allowed, key=lambda e: (-pick[e], e))[:k]
    o_idx, o_w = oracle.route(l[None].astype(np.float64), k, G, M)
    assert o_idx[0].tolist() == want
    assert (out["idx"] == np.array(want)).all(), (out["idx"][0], want)
    assert np.abs(out["w"] - o_w).max() <= 1e-6
    assert np.array_equal(out["counts"], T * np.bincount(want, minlength=E))
    assert np.array_equal(out["offsets"], np.concatenate([[0], np.cumsum(out["counts"])]))
    assert not out["y"].any()  # x = 0


@pytest.mark.parametrize("T", [2, 40])
def test_few_all_logits_minus_infinity(moe, T):
    """No weights (NaN, as the definition gives), but a selection all the same."""
    needs_gpu()
    print(f"[few -inf] T={T}", flush=True)
    out = select(moe, np.full(32, -np.inf), T, 4)
    assert (out["idx"] == np.arange(4)).all() and np.isnan(out["w"]).all()
    assert out["counts"].sum() == 4 * T


def full(name, T, d, E, k, d_ff, w, **kw):
    return cases._few(name, T, d, E, k, d_ff, w, **kw)


@pytest.mark.parametrize("c", [
    full("mixtral", 16, 4096, 8, 2, 14336, "bf16"),
    full("mixtral", 1, 4096, 8, 2, 14336, "int4"),
    full("mixtral", 64, 4096, 8, 2, 14336, "bf16"),
    full("mixtral", 64, 4096, 8, 2, 14336, "int4"),
    full("mixtral", 17, 4096, 8, 2, 14336, "fp8_e4m3"),
    full("64 experts", 16, 4096, 64, 2, 1408, "bf16", bias=True, cf=1.25),
    full("64 experts", 64, 4096, 64, 2, 1408, "int8", bias=True, cf=1.25),
    full("fine", 16, 7168, 256, 8, 2048, "int4", shared=True, groups=8, topk_groups=4),
    full("fine", 40, 7168, 256, 8, 2048, "int4", shared=True, groups=8, topk_groups=4, cf=1.25,
         overflow="shared"),
], ids=lambda c: f"{c['name']}-{c['T']}-{c['w']}")
def test_few_at_full_widths(moe, c, monkeypatch):
    """Whole layers at their full widths against their definition in float64."""
    needs_gpu()
    print(f"[few full] {c}", flush=True)
    monkeypatch.setattr(cases, "own", True)
    st = cases.prepare(c, 11)
    for n in ("y", "topk_w"):
        st[n].fill_(float("nan"))
    st["ws"].fill_(0xFF)
    out = cases.run(st)
    torch.cuda.synchronize()
    want = cases.exact(c, 11)
    for n in ("topk_idx", "counts", "offsets"):
        assert torch.equal(out[n], want[n]), n
    # (the logits' fp32 sums, 4 sqrt(d / 32) 2^-24 of their size, move a weight by as much)
    assert (out["topk_w"].double() - want["topk_w"]).abs().max() <= 1e-5
    rms = want["y"].pow(2).mean().sqrt()
    err = float((out["y"].double() - want["y"]).abs().max() / rms)
    print(f"  err={err:.2e}", flush=True)
    assert err <= TOL
