"""moe_adapter_linear on its 256 x 256 tiles (from 150 of them on) where adapters are
absent, clamped or apart, adapters far into B, and one workspace for batches of all sizes.
Tolerances are those of test_gpu_adapter.py."""
import numpy as np
import pytest

from tests.test_gpu_adapter import Case, needs_gpu

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

T_TILES = 2600  # 11 x 16 tiles of 256 x 256 with 4096 outputs


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_layer_bincount_amd as m
    return m


def test_rows_without_any(moe):
    needs_gpu()
    print("[adapter none] tiles", flush=True)
    c = Case(T_TILES, 264, 4096, 3, 16, bias=True)
    c.idx.fill_(-1)
    c.A.fill_(float("nan"))
    c.B.fill_(float("nan"))
    c.check(c.run(moe))
    c.idx[:] = torch.tensor([2 ** 31 - 1, -2 ** 31, 3, -1, 3]).repeat(T_TILES // 5 + 1)[:T_TILES].int()
    c.check(c.run(moe))


def test_ranks_are_clamped(moe):
    needs_gpu()
    print("[adapter clamp] tiles", flush=True)
    c = Case(T_TILES, 264, 4096, 3, 24, ragged=True, garbage=False)
    c.ranks[:] = torch.tensor([-5, 2 ** 31 - 1, 11], dtype=torch.int32)
    c.A[0] = float("nan")
    c.check(c.run(moe))


@pytest.mark.parametrize("w", ["fp8_e4m3", "int8", "int4"])
def test_rows_are_apart(moe, w):
    needs_gpu()
    print(f"[adapter apart] tiles {w}", flush=True)
    c = Case(T_TILES, 320, 4096, 4, 16, w=w, y="f32", base=True)
    clean = c.run(moe)
    c.A[2, 3] = float("inf")
    c.B[2, :, 1] = float("nan")
    c.x[T_TILES // 3] = float("nan")
    got = c.run(moe)
    hit = (c.idx == 2).numpy()
    hit[T_TILES // 3] = True
    assert np.array_equal(got[~hit], clean[~hit]) and np.isnan(got[hit]).all()


@pytest.mark.parametrize("T", [3, 90, 400])
def test_adapters_far_into_B(moe, T):
    """B of more than 2^31 elements and 2^32 bytes; the joins by rows, by blocks and by tiles."""
    needs_gpu()
    print(f"[adapter far B] T={T}", flush=True)
    n, R, d_out = 600, 128, 32768
    small = Case(T, 16, d_out, 2, R, y="f32")
    A = torch.zeros(n, R, 16, dtype=torch.bfloat16, device="cuda")
    B = torch.zeros(n, d_out, R, dtype=torch.bfloat16, device="cuda")
    far = (17, n - 1)
    for i, a in enumerate(far):
        A[a], B[a] = small.A[i].cuda(), small.B[i].cuda()
    scales = torch.zeros(n, device="cuda")
    scales[torch.tensor(far)] = small.scales.cuda()
    idx = torch.tensor([far[i] if 0 <= i < 2 else -1 for i in small.idx.tolist()],
                       dtype=torch.int32, device="cuda")
    sh = moe.make_adapter_shape(T, 16, d_out, n, R, y_dtype=moe.DT_F32)
    y = torch.full((T, d_out), float("nan"), device="cuda")
    moe.moe_adapter_linear(sh, small.x.cuda(), small.W.cuda(), None, None, A, B, None, scales, idx,
                           None, y, moe.adapter_workspace(sh))
    torch.cuda.synchronize()
    small.check(y.double().cpu().numpy())


@pytest.mark.parametrize("w", ["bf16", "int4", None])
def test_one_workspace_for_all_batches(moe, w):
    """The workspace of the largest batch, and nothing behind it is written by smaller ones."""
    needs_gpu()
    print(f"[adapter workspace] {w}", flush=True)
    kw = dict(d_in=2048, d_out=2048, n=6, R=32, w=w, y="f32")
    most = moe.moe_adapter_workspace_bytes(Case(6000, **kw).shape(moe))
    big = torch.full((most + (64 << 20),), 77, dtype=torch.uint8, device="cuda")
    for T in (1, 16, 64, 65, 256, 333, 2048):
        c = Case(T, **kw)
        y = torch.full((T, 2048), float("nan"), device="cuda")
        moe.moe_adapter_linear(c.shape(moe), *c.args(), y, big[:most])
        torch.cuda.synchronize()
        c.check(y.double().cpu().numpy())
        assert bool((big[most:] == 77).all()), T
