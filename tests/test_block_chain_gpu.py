"""The block operators together, as a recurrent block's training step and decoding use them, against the same steps in 64
bits; and captured in HIP graphs, on other streams, two at once (GPU)."""
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
f32, bf16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def ssm():
    import __graft_entry__
    __graft_entry__._ensure_built()
    import selective_state_space_58_amd as m
    m.load_library()
    torch.cuda.set_device(0)
    return m


def layer(dim, W=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(conv_w=rn(dim, W) / 2, conv_b=rn(dim) / 4, A=torch.log(torch.rand(dim, generator=g) * 0.2 + 0.75),
                w_post=1 + rn(dim) / 5, scale=rn(dim) / 3, w_pre=1 + rn(dim) / 5)


def forward(ssm, p, u, r, i, z, res, reset, rng):
    """One block from the normed input u: conv + silu, gated scan, gate + norm + scale + dropout + residual + next norm."""
    c = ssm.ssm_causal_conv1d_fwd(u, p["conv_w"], bias=p["conv_b"])
    y, states = ssm.ssm_gated_scan_fwd_train(c, r, i=i, A=p["A"], reset=reset)
    R, out = ssm.ssm_block_norm_fwd(y, z=z, residual=res, w_post=p["w_post"], scale=p["scale"], w_pre=p["w_pre"], p=0.2, rng=rng)
    return c, y, states, R, out


def backward(ssm, p, u, r, i, z, res, reset, rng, c, y, states, dR, dout):
    n = ssm.ssm_block_norm_bwd(y, dR, dout, z=z, residual=res, w_post=p["w_post"], scale=p["scale"], w_pre=p["w_pre"], p=0.2, rng=rng)
    s = ssm.ssm_gated_scan_bwd(c, r, n["dy"], i=i, A=p["A"], reset=reset, states=states)
    v = ssm.ssm_causal_conv1d_bwd(u, p["conv_w"], s["dx"], bias=p["conv_b"])
    return {"du": v["dx"], "dconv_w": v["dweight"], "dconv_b": v["dbias"], "dr": s["dr"], "di": s["di"], "dA": s["dA"],
            "dz": n["dz"], "dres": n["dresidual"], "dw_post": n["dw_post"], "dscale": n["dscale"], "dw_pre": n["dw_pre"]}


def test_training_step_of_a_block(ssm):
    b, L, d = 2, 150, 24
    g = torch.Generator().manual_seed(3)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    p = layer(d)
    u, r, i, z, res, dR, dout = (rn(b, L, d) for _ in range(7))
    reset = torch.rand(b, L, generator=g) < 0.03
    key = (11, 5)
    P = {k: v.to(DEV) for k, v in p.items()}
    T = [t.to(DEV) for t in (u, r, i, z, res)]
    rng = torch.tensor(key, device=DEV)
    c, y, states, R, out = forward(ssm, P, *T, reset.to(DEV), rng)
    got = {"R": R, "out": out, **backward(ssm, P, *T, reset.to(DEV), rng, c, y, states, dR.to(DEV), dout.to(DEV))}
    # the same block in 64 bits, gradients by autograd
    D = {k: v.double().requires_grad_() for k, v in p.items()}
    U, Rr, I, Z, Res = (t.double().requires_grad_() for t in (u, r, i, z, res))
    keep = ref.keep_factors(b * L, d, 0.2, key).view(b, L, d)
    c64, _ = ref.conv_forward(U, D["conv_w"], D["conv_b"])
    y64, _ = ref.gated_forward(c64, Rr, I, D["A"], reset)
    R64, out64 = ref.norm_forward(y64, Z, Res, D["w_post"], D["scale"], D["w_pre"], keep)
    loss = (R64 * dR.double()).sum() + (out64 * dout.double()).sum()
    names = ["du", "dconv_w", "dconv_b", "dr", "di", "dA", "dz", "dres", "dw_post", "dscale", "dw_pre"]
    grads = torch.autograd.grad(loss, [U, D["conv_w"], D["conv_b"], Rr, I, D["A"], Z, Res, D["w_post"], D["scale"], D["w_pre"]])
    want = dict(zip(names, grads), R=R64.detach(), out=out64.detach())
    # fp32 through four operators: each is held to its own bound elsewhere; here a sum of up to b L = 300 terms, each
    # of at most about 200 roundings, all of one sign: 300 * 200 * 2^-24 of the largest value is 3.6e-3, and random
    # signs leave its root, 3.6e-3 / sqrt(300 * 200) = 1.5e-5.  1e-4 of the largest value lies between.
    assert set(got) == set(want)
    for k in want:
        off = float((got[k].cpu().double() - want[k]).abs().max() / want[k].abs().max())
        assert off <= 1e-4, (k, off)


def test_training_step_in_bf16_is_near(ssm):
    # the same step in bf16: activations rounded between the operators (half a step, 2^-8, each), gates and weights not
    b, L, d = 2, 130, 64
    g = torch.Generator().manual_seed(4)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    P = {k: v.to(DEV) for k, v in layer(d, seed=1).items()}
    base = [rn(b, L, d).to(bf16) for _ in range(7)]
    rng = torch.tensor((2, 9), device=DEV)
    outs = []
    for t in (f32, bf16):
        u, r, i, z, res, dR, dout = (x.to(DEV).to(t) for x in base)
        c, y, states, R, out = forward(ssm, P, u, r, i, z, res, None, rng)
        outs.append({"R": R, "out": out, **backward(ssm, P, u, r, i, z, res, None, rng, c, y, states, dR, dout)})
    # conv, scan, norm forward and norm, scan, conv backward round six times on the way to du; a value carries the
    # roundings of its neighbours in time, which the decays average: eight half steps in the 2-norm
    for k in outs[0]:
        a, e = outs[1][k].double(), outs[0][k].double()
        assert float((a - e).norm() / e.norm()) <= 8 * 2 ** -8, k


def test_decoding_step_by_step(ssm):
    # conv update, gated update and norm a token at a time give the sequence's outputs
    b, L, d = 3, 40, 16
    g = torch.Generator().manual_seed(5)
    P = {k: v.to(DEV) for k, v in layer(d, seed=2).items()}
    u, r, i, z, res = (torch.randn(b, L, d, generator=g).to(DEV) for _ in range(5))
    c = ssm.ssm_causal_conv1d_fwd(u, P["conv_w"], bias=P["conv_b"])
    y = ssm.ssm_gated_scan_fwd(c, r, i=i, A=P["A"])
    norm = lambda y, z, res: ssm.ssm_block_norm_fwd(y, z=z, residual=res, w_post=P["w_post"], w_pre=P["w_pre"])  # noqa: E731
    R, out = norm(y, z, res)
    conv_state, state = torch.zeros(b, d, 3, device=DEV), torch.zeros(b, d, device=DEV)
    for t in range(L):
        at = lambda x: x[:, t].contiguous()  # noqa: E731
        ct = ssm.ssm_causal_conv1d_fwd(u[:, t:t + 1].contiguous(), P["conv_w"], bias=P["conv_b"], state_in=conv_state,
                                       state_out=conv_state)[0][:, 0]
        yt = ssm.ssm_gated_state_update(ct.contiguous(), at(r), state, i=at(i), A=P["A"])
        Rt, ot = norm(yt, at(z), at(res))
        # at most 40 steps of some 30 roundings each between the two orders of the sums
        for a, e in ((yt, y[:, t]), (Rt, R[:, t]), (ot, out[:, t])):
            assert float((a - e).abs().max()) <= 1200 * 2 ** -24 * float(e.abs().max())


def capture(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = fn()
    return g, out


def test_captured_training_step_with_new_random_numbers(ssm):
    b, L, d = 2, 700, 40   # several tiles of the gated scan in either direction
    gen = torch.Generator().manual_seed(6)
    P = {k: v.to(DEV) for k, v in layer(d, seed=3).items()}
    T = [torch.randn(b, L, d, generator=gen).to(DEV).to(bf16) for _ in range(7)]
    reset = (torch.rand(b, L, generator=gen) < 0.01).to(DEV)
    rng = torch.tensor([7, 0], device=DEV)

    def step():
        c, y, states, R, out = forward(ssm, P, *T[:5], reset, rng)
        return {"R": R, "out": out, **backward(ssm, P, *T[:5], reset, rng, c, y, states, *T[5:])}

    g, out = capture(step)
    seen = []
    for k in range(4):
        for t in T:   # new inputs and numbers in the captured tensors
            t.copy_(torch.randn(b, L, d, generator=gen).to(bf16))
        rng[1] += 1
        g.replay()
        torch.cuda.synchronize()
        got = {n: v.clone() for n, v in out.items()}
        want = step()   # eager work between the replays
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(got[n], want[n]), (k, n)
        seen.append(got["R"])
    assert not torch.equal(seen[0], seen[1])


def test_two_graphs_share_a_workspace_in_turn(ssm):
    # calls that share a workspace are ordered on one stream; whatever one leaves in it, the other clears
    b, d = 1, 8
    nbytes = max(ssm.ssm_gated_scan_bwd_workspace_bytes(b, L, d, bf16, False) for L in (9000, 5000))
    ws = torch.full((nbytes,), 255, dtype=torch.uint8, device=DEV)
    runs = []
    for L in (9000, 5000):
        x, r, i, dy = (torch.randn(b, L, d, device=DEV).to(bf16) for _ in range(4))
        A = -torch.rand(d, device=DEV) / 10

        def fn(x=x, r=r, i=i, dy=dy, A=A):
            y = ssm.ssm_gated_scan_fwd(x, r, i=i, A=A, workspace=ws)
            return [y] + list(ssm.ssm_gated_scan_bwd(x, r, dy, i=i, A=A, workspace=ws).values())

        want = [t.clone() for t in fn()]
        runs.append((*capture(fn), want, fn))   # (fn holds the inputs that the graph reads)
    for k in (0, 1, 1, 0, 0, 1):
        g, out, want, _ = runs[k]
        ws.fill_(k)
        g.replay()
        torch.cuda.synchronize()
        for a, e in zip(out, want):
            assert torch.equal(a, e)


def test_two_streams_at_once(ssm):
    # calls with workspaces of their own run side by side
    b, L, d = 1, 20000, 64
    sets, want = [], []
    for k in range(2):
        x, r, i, dy = (torch.randn(b, L, d, device=DEV).to(bf16) for _ in range(4))
        A = -torch.rand(d, device=DEV) / 10
        sets.append((x, r, i, dy, A))
        y, st = ssm.ssm_gated_scan_fwd_train(x, r, i=i, A=A)
        want.append([y] + list(ssm.ssm_gated_scan_bwd(x, r, dy, i=i, A=A, states=st).values()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for rep in range(5):
        got = []
        for k, s in enumerate(streams):
            x, r, i, dy, A = sets[k]
            with torch.cuda.stream(s):
                y, st = ssm.ssm_gated_scan_fwd_train(x, r, i=i, A=A)
                got.append([y] + list(ssm.ssm_gated_scan_bwd(x, r, dy, i=i, A=A, states=st).values()))
        torch.cuda.synchronize()
        for a, e in zip(got, want):
            for u, v in zip(a, e):
                assert torch.equal(u, v), rep


def test_rows_past_the_end_are_left_alone(ssm):
    # outputs that are the front of a larger buffer: what lies behind them stays
    b, L, d = 1, 77, 6
    x, r, i = (torch.randn(b, L, d, device=DEV).to(bf16) for _ in range(3))
    A = -torch.rand(d, device=DEV) / 10
    for dt in (bf16,):
        buf = torch.full((b * L * d + 4096,), 3.0, device=DEV, dtype=dt)
        ssm.ssm_gated_scan_fwd(x, r, i=i, A=A, y=buf[:b * L * d].view(b, L, d))
        assert bool((buf[b * L * d:] == 3.0).all())
        buf.fill_(3.0)
        ssm.ssm_block_norm_fwd(x.view(L, d), w_post=torch.ones(d, device=DEV), res_out=buf[:L * d].view(L, d))
        assert bool((buf[L * d:] == 3.0).all())


def test_long_offsets(ssm):
    # more than 2^31 elements: the last rows of a batch lie past 32-bit offsets
    b, L, d = 3, 192, 1 << 22
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GiB")
    x = torch.zeros(b, L, d, dtype=bf16, device=DEV)
    r = torch.zeros(b, L, d, dtype=bf16, device=DEV)
    part = torch.randn(L, 8).to(bf16)
    x[2, :, d - 8:] = part.to(DEV)
    with pytest.raises(ssm.SSMError):   # a tile of so wide a row is past its 32-bit places: refused
        ssm.ssm_gated_scan_fwd(x, r)
    x, r = x.view(1, b * L * 64, d // 64), r.view(1, b * L * 64, d // 64)
    y, h = ssm.ssm_gated_scan_fwd(x, r, return_final_state=True)
    # gates of 1/2: the last token's state is the sum of x_t 2^-(age + 1)
    tail = x[0, -32:].double()
    want = (tail * 0.5 ** torch.arange(32, 0, -1, device=DEV).double()[:, None]).sum(0)
    assert float((h[0].double() - want).abs().max()) <= 2.0 ** -22 * 4
    assert torch.equal(y[0, -1], h[0].to(bf16))
