"""GPU parity of the block norm and its gradient with their 64-bit form (tests/block_ref.py)."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
T = {"bf16": torch.bfloat16, "f32": torch.float32}
RNG = (0x1234567890ABCDEF, 77)


@pytest.fixture(scope="module")
def ssm():
    import __graft_entry__
    __graft_entry__._ensure_built()
    import selective_state_space_58_amd as m
    m.load_library()
    torch.cuda.set_device(0)
    return m


NAMES = dict(z="z", r="residual", p="w_post", s="scale", n="w_pre")


def inputs(rows, dim, parts="zrpsn", act="bf16", res="f32", seed=0):
    """Inputs named by letters: z gate, r residual, p norm after, s scale, n norm before the next block."""
    g = torch.Generator().manual_seed(seed + 3 * rows + dim)
    rn = lambda *s, t=T[act]: torch.randn(*s, generator=g).to(t)  # noqa: E731
    w = lambda: 1 + 0.2 * torch.randn(dim, generator=g)  # noqa: E731
    s = dict(y=rn(rows, dim), z=rn(rows, dim), residual=2 * rn(rows, dim, t=T[res]), w_post=w(), scale=0.5 * w(), w_pre=w())
    s = {k: v for k, v in s.items() if k == "y" or k in [NAMES[c] for c in parts]}
    return s, rn(rows, dim, t=T[res]), rn(rows, dim) if "n" in parts else None


def run(ssm, s, dres, dout, p=0.0, res="f32", **kw):
    t = {k: v.to(DEV) for k, v in s.items()}
    y = t.pop("y")
    rng = torch.tensor(RNG, dtype=torch.int64, device=DEV) if p else None
    o = ssm.ssm_block_norm_fwd(y, p=p, rng=rng, res_dtype=T[res], **t, **kw)
    got = dict(zip(("res_out", "out"), o)) if isinstance(o, tuple) else {"res_out": o}
    got.update(ssm.ssm_block_norm_bwd(y, None if dres is None else dres.to(DEV), None if dout is None else dout.to(DEV),
                                      p=p, rng=rng, res_dtype=T[res], **t, **kw))
    torch.cuda.synchronize()
    return got


def compare(ssm, s, dres, dout, p=0.0, res="f32"):
    got = run(ssm, s, dres, dout, p, res)
    keep = ref.keep_factors(*s["y"].shape, p, RNG) if p else None
    val, bnd = ref.norm(s["y"], dres, dout, keep=keep, **{k: v for k, v in s.items() if k != "y"})
    assert set(got) == set(val)
    for k in val:
        ref.check(got[k], val[k], bnd[k], k)
    return got


@pytest.mark.parametrize("act,res", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 2), (2, 8), (5, 40), (33, 64), (7, 129), (9, 256), (2, 520), (130, 72),
                                      (3, 1000), (2, 1001), (2, 1032), (3, 4104), (2, 4999)])
def test_sizes(ssm, rows, dim, act, res):
    print("block norm", act, res, (rows, dim), flush=True)
    compare(ssm, *inputs(rows, dim, act=act, res=res), p=0.25 if rows * dim < 10000 else 0.0, res=res)


@pytest.mark.parametrize("dim", [8192, 8200, 16384, 16383])
def test_widest_rows(ssm, dim):
    for act in ("bf16", "f32"):
        compare(ssm, *inputs(2, dim, act=act), res="f32")


@pytest.mark.parametrize("parts", ["", "n", "p", "s", "z", "r", "rn", "zp", "zpn", "rps", "zr", "rpn", "zs", "psn", "zrpsn"])
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_parts(ssm, parts, p):
    for dim in (24, 13):
        for act in ("bf16", "f32"):
            compare(ssm, *inputs(6, dim, parts, act), p=p)


def test_only_one_of_the_gradients_given(ssm):
    s, dres, dout = inputs(5, 48)
    compare(ssm, s, None, dout)
    s, dres, dout = inputs(5, 48, "zrps")
    compare(ssm, s, dres, None)


def test_many_rows_and_fixed_order(ssm):
    s, dres, dout = inputs(3000, 40)
    a = compare(ssm, s, dres, dout)
    b = run(ssm, s, dres, dout)
    for k in a:
        assert torch.equal(a[k], b[k]), k
    s, dres, dout = inputs(1100, 600, "zrpsn", "bf16", "bf16")
    compare(ssm, s, dres, dout, res="bf16")


@pytest.mark.parametrize("dim", [64, 77, 600])
def test_dropped_elements_are_the_generators(ssm, dim):
    # ones through dropout alone: the kept elements are exactly those of the published generator, at both layouts
    rows, p = 9, 0.4
    y = torch.ones(rows, dim, device=DEV)
    for rng in (RNG, (0, 0), (-1, -1), (5, 1 << 40)):
        t = torch.tensor(rng, dtype=torch.int64, device=DEV)
        R = ssm.ssm_block_norm_fwd(y, p=p, rng=t)
        k = ref.keep_factors(rows, dim, p, rng)
        ref.check(R, k, torch.zeros_like(k), "keep")
        g = ssm.ssm_block_norm_bwd(y, y, p=p, rng=t)
        assert torch.equal(g["dy"], R)


def test_rows_dropped_whole(ssm):
    # nearly everything dropped: rows with nothing left are norms of zero, finite
    s, dres, dout = inputs(40, 8, "zpsn")
    got = compare(ssm, s, dres, dout, p=0.9)
    empty = (got["res_out"] == 0).all(-1)
    assert bool(empty.any()) and not got["out"][empty].any()


def test_huge_and_tiny_values(ssm):
    s, dres, dout = inputs(4, 64, "zrpsn", "f32")
    s["y"] *= 1e-12
    compare(ssm, s, dres, dout)
    s, dres, dout = inputs(4, 64, "zrpsn", "f32")
    s["residual"] *= 1e6
    compare(ssm, s, dres, dout)
    s, dres, dout = inputs(4, 64, "rpsn", "f32")
    s["y"] *= 1e8
    compare(ssm, s, dres, dout)


def test_nan_stays_in_its_row(ssm):
    s, dres, dout = inputs(6, 40, "zrps")
    clean = run(ssm, s, dres, dout)
    s["y"][2, 5] = float("nan")
    got = run(ssm, s, dres, dout)
    keep = [0, 1, 3, 4, 5]
    for k in ("res_out", "dy", "dz", "dresidual"):
        assert torch.equal(got[k][keep], clean[k][keep]), k
    assert bool(torch.isnan(got["res_out"][2]).all())


def test_what_is_dropped_is_not_looked_at(ssm):
    # without a norm after the block, a NaN or infinity in a dropped place is gone: value and every gradient
    rows, dim, p = 6, 40, 0.5
    keep = ref.keep_factors(rows, dim, p, RNG)
    for parts in ("zrs", "rs", "zrsn"):
        s, dres, dout = inputs(rows, dim, parts, "f32")
        s["y"][keep == 0] = 0.0
        clean = run(ssm, s, dres, dout, p=p)
        s["y"][keep == 0] = torch.tensor([float("nan"), float("inf")]).repeat(rows * dim)[:int((keep == 0).sum())]
        got = run(ssm, s, dres, dout, p=p)
        for k in clean:
            assert torch.equal(got[k], clean[k]), (parts, k)


def test_residual_updated_in_place_and_leading_shapes(ssm):
    s, dres, dout = inputs(6, 40)
    t = {k: v.to(DEV) for k, v in s.items()}
    y = t.pop("y")
    want, want_out = ssm.ssm_block_norm_fwd(y, **t)
    view = {k: v.view(2, 3, 40) if v.dim() == 2 else v for k, v in t.items()}
    res = view["residual"].clone()
    got, out = ssm.ssm_block_norm_fwd(y.view(2, 3, 40), **{**view, "residual": res}, res_out=res)
    assert got.data_ptr() == res.data_ptr() and torch.equal(got.view(6, 40), want) and torch.equal(out.view(6, 40), want_out)


def test_unaligned_rows(ssm):
    s, dres, dout = inputs(4, 48)
    keep = ref.keep_factors(4, 48, 0.25, RNG)
    val, bnd = ref.norm(s["y"], dres, dout, keep=keep, **{k: v for k, v in s.items() if k != "y"})
    y = torch.empty(4 * 48 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(4, 48)
    y.copy_(s["y"])
    s["y"] = y
    for k, v in run(ssm, s, dres, dout, p=0.25).items():
        ref.check(v, val[k], bnd[k], k)


def test_empty(ssm):
    s, dres, dout = inputs(0, 40)
    got = run(ssm, s, dres, dout)
    assert got["out"].shape == (0, 40)
    for k in ("dw_post", "dscale", "dw_pre"):
        assert got[k].shape == (40,) and not got[k].any()


def test_refusals_of_the_binding(ssm):
    s, dres, dout = inputs(4, 40)
    t = {k: v.to(DEV) for k, v in s.items()}
    y = t.pop("y")
    with pytest.raises(ValueError, match="rng"):
        ssm.ssm_block_norm_fwd(y, p=0.1, **t)
    with pytest.raises(TypeError):
        ssm.ssm_block_norm_fwd(y, p=0.1, rng=torch.zeros(2, device=DEV), **t)
    with pytest.raises(ssm.SSMError, match="p must"):
        ssm.ssm_block_norm_fwd(y, p=1.0, rng=torch.zeros(2, dtype=torch.int64, device=DEV), **t)
    with pytest.raises(ValueError, match="contiguous"):
        ssm.ssm_block_norm_fwd(y.t())
    with pytest.raises(ValueError):
        ssm.ssm_block_norm_bwd(y, dres.to(DEV), None, **t)
    with pytest.raises(TypeError):
        ssm.ssm_block_norm_fwd(y, residual=t["residual"], res_dtype=torch.bfloat16)
    with pytest.raises(ssm.SSMError, match="dim"):
        ssm.ssm_block_norm_fwd(torch.zeros(1, 16392, device=DEV))
