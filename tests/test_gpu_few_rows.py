"""moe_forward_few for 17 to 64 tokens (the layer's route and dispatch, the experts as
two weight streams over grouped rows, the grouped combine) against the float64 oracle,
its limits, and its use on streams and in graphs.

Tolerance on max-abs error / RMS(y): the arithmetic of test_gpu_few.py (exact products,
fp32 sums split over eight waves, h in three bf16 terms) and one more fp32 sum of at
most 33 weighted rows in the combine: 2e-5, as there."""
import numpy as np
import pytest

from moe_synth import Workload, custom_config
from tests.parity import check_forward
from tests.test_gpu_few import few_layer, gpu_logits_of, needs_gpu, outputs, poison

torch = pytest.importorskip("torch")

TOL = 2e-5


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


CASES = [
    # T, d, E, k, d_ff, w, shared, cf, bias, overflow
    (17, 256, 4, 2, 256, "bf16", False, None, "zipf1.5", "drop"),
    (33, 320, 2, 1, 384, "bf16", False, None, None, "drop"),
    (64, 4096, 8, 2, 256, "bf16", False, None, None, "drop"),
    (64, 256, 1, 1, 4096, "bf16", False, None, None, "drop"),
    (49, 768, 32, 8, 256, "bf16", True, 0.5, None, "drop"),
    (64, 256, 1024, 8, 128, "bf16", False, 1.0, None, "drop"),
    (64, 64, 700, 32, 128, "bf16", True, None, None, "drop"),
    (32, 64, 1, 1, 128, "bf16", True, None, None, "drop"),
    (40, 256, 8, 2, 256, "bf16", True, 0.75, "zipf1.5", "shared"),
    (64, 512, 8, 2, 1408, "fp8_e4m3", False, None, "zipf1.5", "drop"),
    (27, 768, 16, 4, 256, "fp8_e4m3", True, 0.5, None, "shared"),
    (61, 640, 8, 3, 384, "int8", True, None, "zipf1.5", "drop"),
    (30, 512, 16, 2, 640, "int8", True, 0.75, None, "shared"),
    (20, 512, 8, 2, 384, "int4", True, None, None, "drop"),
    (64, 640, 4, 2, 256, "int4", True, None, "zipf1.5", "drop"),
    (31, 256, 256, 8, 2048, "int4", False, None, None, "drop"),
]


@pytest.mark.gpu
@pytest.mark.parametrize("pack", [True, False])
@pytest.mark.parametrize("T,d,E,k,d_ff,w,shared,cf,bias,overflow", CASES)
def test_few_rows_match_oracle(moe, T, d, E, k, d_ff, w, shared, cf, bias, overflow, pack):
    needs_gpu()
    print(f"[few rows] T={T} d={d} E={E} k={k} d_ff={d_ff} {w} shared={shared} cf={cf} "
          f"{overflow} pack={pack}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, d, E, k, d_ff, w=w, shared=shared, cf=cf, router_bias=bias,
                                seed=T + d + E))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev, overflow=overflow, pack_router=pack)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    rep = check_forward(wl, out, tol=TOL, overflow=overflow)
    print(f"  err={rep['err']:.2e}", flush=True)
    layer(dev["x"])  # equal calls, equal bits
    again = outputs(layer)
    assert all(np.array_equal(out[n], again[n]) for n in out)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E,k,G,M", [(50, 256, 8, 8, 4), (19, 32, 4, 8, 2), (64, 128, 2, 64, 1)])
def test_few_rows_group_limited(moe, T, E, k, G, M):
    needs_gpu()
    print(f"[few rows groups] T={T} E={E} k={k} G={G} M={M}", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(T, 256, E, k, 128, shared=True, seed=T + E))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev, n_groups=G, topk_groups=M)
    poison(layer)
    layer(dev["x"])
    check_forward(wl, outputs(layer), tol=TOL, decide_on=gpu_logits_of(moe, wl, dev, G, M),
                  groups=G, topk_groups=M)


@pytest.mark.gpu
@pytest.mark.parametrize("shared", [False, True])
def test_few_rows_capacity_zero(moe, shared):
    """No room anywhere: y is zero, or the shared expert's alone."""
    needs_gpu()
    print(f"[few rows] capacity 0 shared={shared}", flush=True)
    from moe_synth import bf16_bits_to_f32
    from moe_synth.device import upload
    wl = Workload(custom_config(35, 256, 8, 2, 256, shared=shared, seed=5))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev, capacity=0)
    poison(layer)
    layer(dev["x"])
    out = outputs(layer)
    assert not out["offsets"].any() and out["counts"].sum() == 70
    if not shared:
        assert not out["y"].any()
        return
    s = wl.shared()
    x = bf16_bits_to_f32(wl.x()).astype(np.float64)
    W = {n: bf16_bits_to_f32(s[n]).astype(np.float64) for n in ("W1", "W3", "W2")}
    a = x @ W["W1"].T
    ref = (a / (1 + np.exp(-a)) * (x @ W["W3"].T)) @ W["W2"].T
    assert np.abs(out["y"] - ref).max() <= TOL * np.sqrt((ref ** 2).mean())


@pytest.mark.gpu
def test_few_rows_keep_to_their_outputs(moe):
    """Weights of unrouted experts may hold anything, and nothing around the outputs
    and the workspace is written."""
    needs_gpu()
    print("[few rows] outputs", flush=True)
    from moe_synth.device import upload
    wl = Workload(custom_config(18, 256, 200, 2, 256, w="fp8_e4m3", shared=True, seed=77))
    dev = upload(wl)
    layer = few_layer(moe, wl, dev)
    layer(dev["x"])
    ref = outputs(layer)
    free = torch.as_tensor(np.setdiff1d(np.arange(200), ref["idx"]), device="cuda")
    for n in ("s1", "s3", "s2"):
        dev["weights"][n][free] = float("nan")
    guard = {}
    for name in ("y", "topk_w", "topk_idx", "counts", "offsets", "ws"):
        t = getattr(layer, name)
        pad = 256 // t.element_size()
        big = torch.full((t.numel() + 2 * pad,), 77, dtype=t.dtype, device="cuda")
        guard[name] = (big, pad)
        setattr(layer, name, big[pad:pad + t.numel()].view(t.shape))
    layer(dev["x"])
    out = outputs(layer)
    for key in ref:
        assert np.array_equal(ref[key], out[key]), key
    for name, (big, pad) in guard.items():
        assert (big[:pad] == 77).all() and (big[-pad:] == 77).all(), name


@pytest.mark.gpu
def test_few_rows_on_streams_and_in_graphs(moe):
    """Equal calls give equal bits: two streams at once, and two graphs that share the
    workspace of the larger batch, 60 and 16 tokens."""
    needs_gpu()
    print("[few rows] streams and graphs", flush=True)
    from moe_synth.device import upload
    layers = []
    for T, w, seed in ((60, "int4", 21), (16, "bf16", 22)):
        wl = Workload(custom_config(T, 512, 16, 4, 1408, w=w, shared=True, seed=seed))
        dev = upload(wl)
        layer = few_layer(moe, wl, dev)
        layer(dev["x"])
        layers.append((layer, dev["x"], outputs(layer)))
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(10):
        for (layer, x, _), s in zip(layers, streams):
            with torch.cuda.stream(s):
                layer(x)
    for layer, x, ref in layers:
        out = outputs(layer)
        assert all(np.array_equal(out[n], ref[n]) for n in ref)
    graphs = []
    for layer, x, _ in layers:
        layer.ws = layers[0][0].ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer(x)
        graphs.append(g)
    for rep in range(3):
        for (layer, x, ref), g in zip(layers, graphs):
            for t in (layer.y, layer.topk_w):
                t.fill_(float("nan"))
            _ = (torch.randn(1 << 16, device="cuda") * 2).sum().item()
            g.replay()
            out = outputs(layer)
            assert all(np.array_equal(out[n], ref[n]) for n in ref), rep


@pytest.mark.cpu
@pytest.mark.parametrize("T", [17, 37, 63, 64])
def test_few_takes_up_to_64_tokens(moe, T):
    """Their shapes are taken; what is wrong is refused before anything is launched."""
    sh = moe.make_shape(T, 256, 8, 2, 128)
    assert moe.moe_few_workspace_bytes(sh) > 0
    ok = dict(x=256, W_g=256, y=256, idx=256, w=256, counts=256, offsets=256, ws=256, W2=256)
    for bad, needle in ((dict(x=None), "x is NULL"), (dict(x=264), "x is not 16"),
                        (dict(y=None), "y is NULL"), (dict(ws=128), "ws is not 256"),
                        (dict(counts=None), "counts is NULL"), (dict(W2=264), "W2 is not 16")):
        a = {**ok, **bad}
        with pytest.raises(moe.MoEError, match=needle):
            moe.moe_forward_few(sh, a["x"], a["W_g"], None,
                                moe.make_weights(W1=256, W3=256, W2=a["W2"]), a["y"], a["idx"],
                                a["w"], a["counts"], a["offsets"], a["ws"], stream=0)


@pytest.mark.cpu
def test_few_refuses_past_64_tokens(moe):
    for T in (65, 1 << 20):
        sh = moe.make_shape(T, 256, 8, 2, 128)
        assert moe.moe_few_workspace_bytes(sh) == 0
        with pytest.raises(moe.MoEError, match="at most 64"):
            moe.few_workspace(sh, "cpu")
    assert moe.FEW_MAX_TOKENS == 64
    # a batch whose hidden rows cannot be addressed
    assert moe.moe_few_workspace_bytes(moe.make_shape(40, 64, 8, 2, 1 << 23, w_dtype=1)) > 0
    assert moe.moe_few_workspace_bytes(moe.make_shape(43, 64, 8, 2, 1 << 23, w_dtype=1)) == 0


@pytest.mark.cpu
def test_few_workspace_serves_smaller_batches(moe):
    """A workspace of the largest batch is enough for every smaller one."""
    for kw in (dict(d=4096, E=8, top_k=2, d_ff=14336),
               dict(d=4096, E=4, top_k=1, d_ff=4096, w_dtype=2),
               dict(d=7168, E=256, top_k=8, d_ff=2048, w_dtype=4, has_shared=1, capacity=3),
               dict(d=256, E=1024, top_k=32, d_ff=128)):
        sizes = [moe.moe_few_workspace_bytes(moe.make_shape(T=T, **kw)) for T in range(65)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), kw
