"""The 64-bit reference forms of the block operators: gradients against autograd through the forward as it is
written and against central differences, the random numbers against published values (CPU)."""
import pytest
import torch

from tests import block_ref as ref


def rnd(*shape, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + 7 * len(shape) + sum(shape)), dtype=torch.float64)


def against(loss, leaves, grads):
    """loss(*leaves) -> scalar: its autograd gradients, and central differences of it, against grads."""
    for t in leaves:
        t.requires_grad_(True)
    auto = torch.autograd.grad(loss(*leaves), leaves)
    for t, g, got in zip(leaves, auto, grads):
        assert torch.allclose(g, got, rtol=1e-9, atol=1e-11)
        with torch.no_grad():
            flat, step = t.view(-1), 1e-5
            for k in range(0, flat.numel(), max(1, flat.numel() // 5)):
                old = flat[k].item()
                flat[k] = old + step
                up = loss(*leaves).item()
                flat[k] = old - step
                down = loss(*leaves).item()
                flat[k] = old
                assert abs((up - down) / (2 * step) - got.reshape(-1)[k].item()) < 1e-6 * (1 + abs(got.reshape(-1)[k].item()))


@pytest.mark.parametrize("form", ["lru", "unit"])
@pytest.mark.parametrize("packed", [False, True])
def test_gated_gradients(form, packed):
    b, L, d = 2, 9, 3
    x, r, i, h0, dout, dh = rnd(b, L, d), rnd(b, L, d, seed=1), rnd(b, L, d, seed=2), rnd(b, d), rnd(b, L, d, seed=3), rnd(b, d, seed=4)
    A = -torch.rand(d, dtype=torch.float64) - 0.01
    reset = (rnd(b, L, seed=5) > 0.8) if packed else None
    lru = form == "lru"
    leaves = [x, r, h0] + ([i, A] if lru else [])

    def loss(x, r, h0, i=None, A=None):
        y, h = ref.gated_forward(x, r, i, A, reset, h0)
        return (dout * y).sum() + (dh * h).sum()

    val, _ = ref.gated(x, r, i if lru else None, A if lru else None, reset, h0, dout, dh)
    y, h = ref.gated_forward(x, r, i if lru else None, A if lru else None, reset, h0)
    assert torch.allclose(val["y"], y, rtol=1e-12) and torch.allclose(val["h_final"], h, rtol=1e-12)
    against(loss, leaves, [val["dx"], val["dr"], val["dh0"]] + ([val["di"], val["dA"]] if lru else []))


@pytest.mark.parametrize("L,W,silu", [(7, 4, True), (2, 4, True), (5, 3, False), (4, 1, True)])
def test_conv_gradients(L, W, silu):
    b, d = 2, 3
    x, w, bias, st, dout, ds = rnd(b, L, d), rnd(d, W), rnd(d), rnd(b, d, W - 1), rnd(b, L, d, seed=1), rnd(b, d, W - 1, seed=2)

    def loss(x, w, bias, st):
        out, state = ref.conv_forward(x, w, bias, st, silu)
        return (dout * out).sum() + (ds * state).sum()

    val, _ = ref.conv_bwd(x, w, dout, bias, st, silu, ds)
    against(loss, [x, w, bias, st], [val["dx"], val["dweight"], val["dbias"], val["dstate_in"]])


@pytest.mark.parametrize("parts", ["zrpsn", "rn", "zp", "s", "rpn", "zrps"])
@pytest.mark.parametrize("drop", [False, True])
def test_norm_gradients(parts, drop):
    rows, dim = 3, 10
    y = rnd(rows, dim)
    opt = dict(z=rnd(rows, dim, seed=1), residual=rnd(rows, dim, seed=2), w_post=rnd(dim), scale=rnd(dim, seed=1), w_pre=rnd(dim, seed=2))
    on = dict(zip("zrpsn", opt))
    opt = {k: v for k, v in opt.items() if k in [on[c] for c in parts]}
    dres = rnd(rows, dim, seed=3)
    dout = rnd(rows, dim, seed=4) if "n" in parts else None
    keep = ref.keep_factors(rows, dim, 0.3, (5, 6)) if drop else None
    names = list(opt)

    def loss(y, *vals):
        R, out = ref.norm_forward(y, keep=keep, **dict(zip(names, vals)))
        return (dres * R).sum() + (0 if out is None else (dout * out).sum())

    val, _ = ref.norm(y, dres, dout, keep=keep, **opt)
    key = dict(z="dz", residual="dresidual", w_post="dw_post", scale="dscale", w_pre="dw_pre")
    against(loss, [y] + [opt[n] for n in names], [val["dy"]] + [val[key[n]] for n in names])


def test_philox_known_answers():
    # the three known-answer vectors that the generator's authors publish with it
    ones = 0xFFFFFFFF
    assert ref.philox(0, 0, 0) == [0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8]
    assert ref.philox(2 ** 64 - 1, 2 ** 64 - 1, 2 ** 64 - 1) == [0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD]
    c = [0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344]
    k = [0xA4093822, 0x299F31D0]
    assert ref.philox(c[0] | c[1] << 32, k[0] | k[1] << 32, c[2] | c[3] << 32) == [0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1]
    assert all(0 <= w <= ones for w in ref.philox(12345, 99, 7))


def test_keep_factors_rate_and_scale():
    k = ref.keep_factors(64, 128, 0.25, (1, 2))
    assert set(k.unique().tolist()) == {0.0, 65536 / (65536 - 16384)}
    n = k.numel()
    kept = float((k > 0).double().mean())
    assert abs(kept - 0.75) < 5 * (0.25 * 0.75 / n) ** 0.5   # five standard deviations
