"""The training and serving operators around a recurrent block: what they compute, and the cases they are timed on.

Three operators, each in its plain form (elementary torch operations in 32 bits) and as calls of this
repository's package:

* the gated scan, h_t = a_t h_{t-1} + b_t, in the form with a decay and two gates ("lru": a = exp(A sigmoid(r)),
  b = sqrt(1 - a^2) sigmoid(i) x) and in the form with one gate ("unit": a = sigmoid(r), b = (1 - a) x); a token
  with a reset flag has a = 0.  Forward, forward and backward, and the single-token update in place;
* the gradient of the causal depthwise conv1d + SiLU;
* the block norm, R = residual + dropout(scale * rmsnorm(y silu(z)) w_post), out = rmsnorm(R) w_pre, whose
  dropout takes its keep bits from Philox4x32-10.  Forward, and forward and backward.
"""
import math

import numpy as np
import torch

own = False   # False: run() computes the plain form; True: run() calls the package


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a wide layer at a serving batch: a launch and 1.3 MB of gates, latency counts
        dict(name="gated_step_b128_d5120", op="gated_step", form="lru", dtype="bf16", batch=128, dim=5120),
        # the forward pass of an ordinary layer (evaluation, prefill)
        dict(name="gated_fwd_b8_l2048_d1536", op="gated_fwd", form="lru", dtype="bf16", batch=8, seqlen=2048, dim=1536,
             packed=False, carried=False),
        # prefill of one very long sequence: few channels, all parallelism is in time
        dict(name="gated_fwd_b1_l131072_d2048", op="gated_fwd", form="lru", dtype="bf16", batch=1, seqlen=131072,
             dim=2048, packed=False, carried=True),
        # packed documents of uneven length, odd channel count, 32-bit inputs
        dict(name="gated_fwd_unit_f32_b3_l1000_d777", op="gated_fwd", form="unit", dtype="f32", batch=3, seqlen=1000,
             dim=777, packed=True, carried=True),
        # a training step of an ordinary layer
        dict(name="gated_train_b8_l2048_d1536", op="gated_train", form="lru", dtype="bf16", batch=8, seqlen=2048,
             dim=1536, packed=False, carried=False),
        # a training step on one very long sequence
        dict(name="gated_train_b1_l131072_d2048", op="gated_train", form="lru", dtype="bf16", batch=1, seqlen=131072,
             dim=2048, packed=False, carried=False),
        # a training step of a wide layer on packed documents, one gate
        dict(name="gated_train_unit_b4_l4096_d5120", op="gated_train", form="unit", dtype="bf16", batch=4, seqlen=4096,
             dim=5120, packed=True, carried=True),
        # the gradient of an ordinary layer's convolution
        dict(name="conv_bwd_b8_l2048_d1536_w4", op="conv_bwd", dtype="bf16", batch=8, seqlen=2048, dim=1536, width=4,
             silu=True, carried=False),
        # a segment of a longer sequence (state carried in and out), odd length, 32-bit inputs
        dict(name="conv_bwd_f32_b2_l777_d100_w3", op="conv_bwd", dtype="f32", batch=2, seqlen=777, dim=100, width=3,
             silu=True, carried=True),
        # between two blocks of a decoding step at a serving batch
        dict(name="norm_fwd_r128_d5120", op="norm_fwd", dtype="bf16", res="bf16", rows=128, dim=5120, gate=False, p=0.0),
        # between two blocks of a training step, gated, with dropout and a 32-bit residual stream
        dict(name="norm_train_r16384_d5120", op="norm_train", dtype="bf16", res="f32", rows=16384, dim=5120, gate=True,
             p=0.1),
        # an odd width, 32-bit inputs
        dict(name="norm_train_f32_r999_d1001", op="norm_train", dtype="f32", res="f32", rows=999, dim=1001, gate=True,
             p=0.25),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated_step", "gated_fwd", "gated_fwd", "gated_train", "gated_train", "conv_bwd", "conv_bwd",
                     "norm_fwd", "norm_train", "norm_train"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    dim = _log(rng, 16, 8192)
    if rng.random() < 0.7:
        dim = max(8, dim // 8 * 8)
    most = 1 << 26   # elements of one tensor: a quarter of the largest listed case
    if op == "gated_step":
        return dict(op=op, form=rng.choice(["lru", "unit"]), dtype=dtype, batch=_log(rng, 1, 512), dim=dim)
    if op.startswith("norm"):
        return dict(op=op, dtype=dtype, res=rng.choice([dtype, "f32"]), rows=_log(rng, 1, min(65536, most // dim)),
                    dim=dim, gate=rng.random() < 0.5, p=rng.choice([0.0, 0.1, 0.3]))
    batch = _log(rng, 1, 16)
    seqlen = _log(rng, 1, min(65536, max(1, most // (batch * dim))))
    if op == "conv_bwd":
        return dict(op=op, dtype=dtype, batch=batch, seqlen=seqlen, dim=dim, width=rng.choice([2, 3, 4, 4]),
                    silu=rng.random() < 0.8, carried=rng.random() < 0.5)
    return dict(op=op, form=rng.choice(["lru", "lru", "unit"]), dtype=dtype, batch=batch, seqlen=seqlen, dim=dim,
                packed=rng.random() < 0.4, carried=rng.random() < 0.5)


def work(case):
    """Each input read once, each output written once; multiplies, adds and elementary functions as one operation each."""
    op, e = case["op"], 2 if case["dtype"] == "bf16" else 4
    d = case["dim"]
    if op.startswith("norm"):
        n, er = case["rows"] * d, 2 if case["res"] == "bf16" else 4
        gate = 1 if case["gate"] else 0
        total = n * (e * (2 + gate) + 2 * er) + 12 * d
        flops = n * (10 + 6 * gate + (2 if case["p"] else 0))
        if op == "norm_train":
            total += n * (e * (3 + 2 * gate) + 3 * er) + 24 * d
            flops += n * (24 + 12 * gate)
        return {"bytes": total, "flops": flops}
    if op == "gated_step":
        n, lru = case["batch"] * d, case["form"] == "lru"
        return {"bytes": n * (e * (4 if lru else 3) + 8) + (4 * d if lru else 0), "flops": n * (16 if lru else 7)}
    b, n = case["batch"], case["batch"] * case["seqlen"] * d
    if op == "conv_bwd":
        w = case["width"]
        state = 3 * b * d * (w - 1) * e if case["carried"] else 0
        return {"bytes": 3 * n * e + 8 * d * (w + 1) + state, "flops": n * (6 * w + (8 if case["silu"] else 0))}
    lru = case["form"] == "lru"
    total = n * e * (4 if lru else 3) + 4 * b * d * (2 if case["carried"] else 1) + (4 * d if lru else 0)
    total += b * case["seqlen"] if case["packed"] else 0
    flops = n * (16 if lru else 7)
    if op == "gated_train":
        total += n * e * (7 if lru else 5) + 4 * b * d * (3 if case["carried"] else 2) + (8 * d if lru else 0)
        flops += n * (40 if lru else 18)
    return {"bytes": total, "flops": flops}


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)
    act = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    f32 = torch.float32

    def randn(*shape, dtype=act, mean=0.0, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda", dtype=f32).mul_(std).add_(mean).to(dtype)

    def rand(*shape, lo, hi):
        return torch.rand(*shape, generator=g, device="cuda", dtype=f32).mul_(hi - lo).add_(lo)

    s, d = dict(case=case), case["dim"]
    if case["op"].startswith("norm"):
        rows, res = case["rows"], torch.bfloat16 if case["res"] == "bf16" else f32
        s.update(y=randn(rows, d), residual=randn(rows, d, dtype=res, std=2.0), z=randn(rows, d) if case["gate"] else None,
                 w_post=randn(d, dtype=f32, mean=1.0, std=0.1), w_pre=randn(d, dtype=f32, mean=1.0, std=0.1),
                 scale=rand(d, lo=0.1, hi=1.0), p=case["p"], eps=1e-5,
                 rng=torch.randint(0, 1 << 62, (2,), generator=g, device="cuda") if case["p"] else None)
        if case["op"] == "norm_train":
            s.update(dres=randn(rows, d, dtype=res), dout=randn(rows, d))
        return s
    b = case["batch"]
    if case["op"] == "conv_bwd":
        w, bound = case["width"], 1.0 / math.sqrt(case["width"])
        s.update(x=randn(b, case["seqlen"], d), weight=rand(d, w, lo=-bound, hi=bound), bias=rand(d, lo=-bound, hi=bound),
                 dout=randn(b, case["seqlen"], d), silu=case["silu"],
                 state_in=randn(b, d, w - 1) if case["carried"] else None,
                 dstate_out=randn(b, d, w - 1) if case["carried"] else None)
        return s
    shape = (b, d) if case["op"] == "gated_step" else (b, case["seqlen"], d)
    lru = case["form"] == "lru"
    # the decay of a token with an open gate is uniform in [0.9, 0.999] (lru), its gate open at 0.88 on average (unit)
    s.update(x=randn(*shape), r=randn(*shape, mean=0.0 if lru else 2.0), i=randn(*shape) if lru else None,
             A=rand(d, lo=0.9, hi=0.999).log_() if lru else None)
    if case["op"] == "gated_step":
        s["state"] = randn(b, d, dtype=f32)
        return s
    # packed documents: about eight a row, the first starting anywhere
    s["reset"] = (rand(b, case["seqlen"], lo=0.0, hi=1.0) < 8.0 / case["seqlen"]) if case["packed"] else None
    s["h0"] = randn(b, d, dtype=f32) if case["carried"] else None
    if case["op"] == "gated_train":
        s.update(dout=randn(*shape), dh_final=randn(b, d, dtype=f32))
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    op = s["case"]["op"]
    if op == "gated_step":
        return _gated_step(s)
    if op == "gated_fwd":
        return _gated_fwd(s)
    if op == "gated_train":
        return _gated_train(s)
    if op == "conv_bwd":
        return _conv_bwd(s)
    return _norm(s)


def _package():
    import selective_state_space_58_amd as package
    return package


def _gates(s, x, r, i, reset):
    """a_t, the factor of x's contribution and its parts, in 32 bits."""
    if s["A"] is not None:
        g = torch.sigmoid(r)
        la = s["A"] * g
        # a is near 1 and taken to the power of thousands of tokens: a bias of a fraction of 2^-24 would be seen in dA
        a, sq, gi = torch.exp(la.double()).float(), torch.sqrt(-torch.expm1(2 * la)), torch.sigmoid(i)
        if reset is not None:
            a, sq = a.masked_fill(reset, 0.0), sq.masked_fill(reset, 1.0)
        return a, sq * gi, (g, sq, gi)
    a, rest = torch.sigmoid(r), torch.sigmoid(-r)
    if reset is not None:
        a, rest = a.masked_fill(reset, 0.0), rest.masked_fill(reset, 1.0)
    return a, rest, None


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t along dim 1 from h = 0, by doubling: after the step with distance n, (a, b) take
    the state 2n tokens before to the one at t (no elementary operation of torch does this in one)."""
    n, length = 1, a.shape[1]
    while n < length:
        b = torch.cat([b[:, :n], b[:, n:] + a[:, n:] * b[:, :-n]], 1)
        a = torch.cat([a[:, :n], a[:, n:] * a[:, :-n]], 1)
        n *= 2
    return b


def _gated_step(s):
    if own:
        y = _package().ssm_gated_state_update(s["x"], s["r"], s["state"], i=s["i"], A=s["A"])
        return {"y": y, "state": s["state"]}
    x, r, i = s["x"].float(), s["r"].float(), None if s["i"] is None else s["i"].float()
    a, c, _ = _gates(s, x, r, i, None)
    s["state"].copy_(a * s["state"] + c * x)
    return {"y": s["state"].to(s["x"].dtype), "state": s["state"]}


def _states(s):
    """The pass over the sequence in 32 bits: gates, their parts and h."""
    x, r, i = s["x"].float(), s["r"].float(), None if s["i"] is None else s["i"].float()
    reset = None if s["reset"] is None else s["reset"][:, :, None]
    a, c, parts = _gates(s, x, r, i, reset)
    b = c * x
    if s["h0"] is not None:
        b[:, 0] += a[:, 0] * s["h0"]
    return x, a, c, parts, _recurrence(a, b)


def _gated_fwd(s):
    if own:
        y, h_final = _package().ssm_gated_scan_fwd(s["x"], s["r"], i=s["i"], A=s["A"], reset=s["reset"], h0=s["h0"],
                                                   return_final_state=True)
        return {"y": y, "h_final": h_final}
    h = _states(s)[4]
    return {"y": h.to(s["x"].dtype), "h_final": h[:, -1].clone()}


def _gated_train(s):
    if own:
        p = _package()
        y, h_final, states = p.ssm_gated_scan_fwd_train(s["x"], s["r"], i=s["i"], A=s["A"], reset=s["reset"],
                                                        h0=s["h0"], return_final_state=True)
        grads = p.ssm_gated_scan_bwd(s["x"], s["r"], s["dout"], i=s["i"], A=s["A"], reset=s["reset"], h0=s["h0"],
                                     dh_final=s["dh_final"], states=states)
        return {"y": y, "h_final": h_final, **grads}
    act = s["x"].dtype
    x, a, c, parts, h = _states(s)
    out = {"y": h.to(act), "h_final": h[:, -1].clone()}
    first = torch.zeros_like(h[:, :1]) if s["h0"] is None else s["h0"][:, None]
    before = torch.cat([first, h[:, :-1]], 1)
    # lam_t = dout_t + a_{t+1} lam_{t+1}: the same recurrence over the flipped sequence
    dy = s["dout"].float()
    dy[:, -1] += s["dh_final"]
    later = torch.cat([a[:, 1:], torch.zeros_like(a[:, :1])], 1)
    lam = _recurrence(later.flip(1), dy.flip(1)).flip(1)
    out["dx"] = (lam * c).to(act)
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    if parts is None:
        out["dr"] = (lam * (before - x) * a * c).to(act)
    else:
        g, sq, gi = parts
        dla = lam * a * (before - torch.where(sq > 0, gi * x * a / sq, 0.0))
        out["dr"] = (dla * s["A"] * g * (1 - g)).to(act)
        out["dA"] = (dla * g).sum((0, 1), dtype=torch.float64).float()
        out["di"] = (lam * c * x * (1 - gi)).to(act)
    return out


def _conv_bwd(s):
    if own:
        return _package().ssm_causal_conv1d_bwd(s["x"], s["weight"], s["dout"], bias=s["bias"], state_in=s["state_in"],
                                                silu=s["silu"], dstate_out=s["dstate_out"])
    act, w = s["x"].dtype, s["weight"].shape[1]
    x, dpre, L = s["x"].float(), s["dout"].float(), s["x"].shape[1]
    before = (torch.zeros_like(x[:, :1]).expand(-1, w - 1, -1) if s["state_in"] is None
              else s["state_in"].float().transpose(1, 2))
    taps = torch.cat([before, x], 1).unfold(1, w, 1)            # (batch, token, channel, tap)
    if s["silu"]:
        pre = (taps * s["weight"]).sum(-1) + s["bias"]
        gate = torch.sigmoid(pre)
        dpre = dpre * gate * (1 + pre * (1 - gate))
    # input position p (the w - 1 carried ones first) is tap k of token p - k
    pad = torch.nn.functional.pad(dpre, (0, 0, w - 1, w - 1))
    dxx = (pad.unfold(1, w, 1) * s["weight"].flip(1)).sum(-1)
    out = {"dweight": (taps * dpre[..., None]).sum((0, 1), dtype=torch.float64).float(),
           "dbias": dpre.sum((0, 1), dtype=torch.float64).float()}
    if s["dstate_out"] is not None:
        dxx[:, L:] += s["dstate_out"].float().transpose(1, 2)
    if s["state_in"] is not None:
        out["dstate_in"] = dxx[:, :w - 1].transpose(1, 2).to(act).contiguous()
    out["dx"] = dxx[:, w - 1:].to(act)
    return out


def _philox(block, key, offset):
    """Philox4x32-10 (Salmon, Moraes, Dror, Shaw: Parallel random numbers, as easy as 1, 2, 3; 2011) of the counters
    (block, offset): four 32-bit words each.  64-bit products wrap, and their halves are taken as unsigned."""
    low = 0xFFFFFFFF
    c0, c1 = block & low, (block >> 32) & low
    c2, c3 = (offset & low).expand_as(c0), ((offset >> 32) & low).expand_as(c0)
    k0, k1 = key & low, (key >> 32) & low
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((p1 >> 32) & low) ^ c1 ^ k0, p1 & low, ((p0 >> 32) & low) ^ c3 ^ k1, p0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack([c0, c1, c2, c3], -1)


def _keep(s, rows, d):
    """1 / (1 - p) where an element is kept, 0 where it is dropped: eight elements take the 16-bit halves of one block."""
    if not s["p"]:
        return None
    t = math.floor(s["p"] * 65536 + 0.5)
    words = _philox(torch.arange((rows * d + 7) // 8, device="cuda"), s["rng"][0], s["rng"][1])
    halves = torch.stack([words & 0xFFFF, words >> 16], -1).reshape(-1)[:rows * d].reshape(rows, d)
    return (halves >= t).float() * (65536.0 / (65536 - t))


def _norm(s):
    args = dict(z=s["z"], residual=s["residual"], w_post=s["w_post"], scale=s["scale"], w_pre=s["w_pre"], p=s["p"],
                rng=s["rng"], eps=s["eps"])
    if own:
        p = _package()
        res_out, out = p.ssm_block_norm_fwd(s["y"], **args)
        if "dout" not in s:
            return {"res_out": res_out, "out": out}
        return {"res_out": res_out, "out": out,
                **p.ssm_block_norm_bwd(s["y"], dres=s["dres"], dout=s["dout"], **args)}
    y, eps = s["y"].float(), s["eps"]
    act, res = s["y"].dtype, s["residual"].dtype
    v = y
    if s["z"] is not None:
        z = s["z"].float()
        sig = torch.sigmoid(z)
        v = y * z * sig
    r1 = torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)
    vhat = v * r1
    n = vhat * s["w_post"]
    m = n * s["scale"]
    keep = _keep(s, *y.shape)
    R = s["residual"].float() + (m if keep is None else m * keep)
    r2 = torch.rsqrt((R * R).mean(-1, keepdim=True) + eps)
    Rhat = R * r2
    out = {"res_out": R.to(res), "out": (Rhat * s["w_pre"]).to(act)}
    if "dout" not in s:
        return out
    dout = s["dout"].float()
    q = dout * s["w_pre"]
    dR = s["dres"].float() + r2 * (q - Rhat * (q * Rhat).mean(-1, keepdim=True))
    dm = dR if keep is None else dR * keep
    dn = dm * s["scale"]
    q = dn * s["w_post"]
    dv = r1 * (q - vhat * (q * vhat).mean(-1, keepdim=True))
    out["dw_pre"] = (dout * Rhat).sum(0, dtype=torch.float64).float()
    out["dscale"] = (dm * n).sum(0, dtype=torch.float64).float()
    out["dw_post"] = (dn * vhat).sum(0, dtype=torch.float64).float()
    out["dresidual"] = dR.to(res)
    if s["z"] is None:
        out["dy"] = dv.to(act)
    else:
        out["dy"] = (dv * z * sig).to(act)
        out["dz"] = (dv * y * sig * (1 + z * (1 - sig))).to(act)
    return out


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    w = {k: v.double() if isinstance(v, torch.Tensor) and v.is_floating_point() else v for k, v in s.items()}
    if case["op"].startswith("norm"):
        return _exact_norm(case, w)
    if case["op"] == "conv_bwd":
        return _exact_conv(case, w)
    return _exact_gated(case, w)


def _exact_gated(case, w):
    """Token after token, as the recurrence is written."""
    step, lru = case["op"] == "gated_step", case["form"] == "lru"
    x, r, i = (None if v is None else v[:, None] if step else v for v in (w["x"], w["r"], w["i"]))
    reset = None if step else w["reset"]
    g = 1 / (1 + torch.exp(-r))
    a = torch.exp(w["A"] * g) if lru else g
    fresh = torch.sqrt(-torch.expm1(2 * w["A"] * g)) if lru else 1 / (1 + torch.exp(r))
    if reset is not None:
        a[reset], fresh[reset] = 0.0, 1.0
    gate = 1 / (1 + torch.exp(-i)) if lru else None
    u = gate * x if lru else x
    b = fresh * u
    L = x.shape[1]
    h0 = w["state"] if step else w["h0"] if w["h0"] is not None else torch.zeros_like(x[:, 0])
    h = torch.empty_like(x)
    prev = h0
    for t in range(L):
        prev = torch.addcmul(b[:, t], a[:, t], prev)
        h[:, t] = prev
    if step:
        return {"y": h[:, 0], "state": h[:, 0]}
    out = {"y": h, "h_final": h[:, -1]}
    if case["op"] == "gated_fwd":
        return out
    lam = torch.empty_like(x)
    cur = w["dout"][:, L - 1] + w["dh_final"]
    lam[:, L - 1] = cur
    for t in range(L - 2, -1, -1):
        cur = torch.addcmul(w["dout"][:, t], a[:, t + 1], cur)
        lam[:, t] = cur
    da = lam * torch.cat([h0[:, None], h[:, :-1]], 1)
    if lru:
        # b = sqrt(1 - a^2) u: d sqrt(1 - a^2) / da = -a / sqrt(1 - a^2); a = exp(A g)
        da = da - torch.where(fresh > 0, lam * u * a / fresh, torch.zeros_like(a))
        dg = da * a * w["A"]
        out["dA"] = (da * a * g).sum((0, 1))
        out["dr"] = dg * g * (1 - g)
        out["dx"] = lam * fresh * gate
        out["di"] = lam * fresh * x * gate * (1 - gate)
        if reset is not None:
            out["dr"][reset] = 0.0
    else:
        out["dr"] = (da - lam * x) * a * (1 - a)
        out["dx"] = lam * fresh
    if w["h0"] is not None:
        out["dh0"] = a[:, 0] * lam[:, 0]
    return out


def _exact_conv(case, w):
    """Tap by tap."""
    x, W, L = w["x"], case["width"], case["seqlen"]
    b, _, d = x.shape
    xx = torch.zeros(b, L + W - 1, d, dtype=torch.float64, device=x.device)
    xx[:, W - 1:] = x
    if w["state_in"] is not None:
        xx[:, :W - 1] = w["state_in"].transpose(1, 2)
    pre = w["bias"].expand(b, L, d).clone()
    for k in range(W):
        pre += w["weight"][:, k] * xx[:, k:k + L]
    dpre = w["dout"]
    if case["silu"]:
        e = torch.exp(-pre)
        dpre = dpre * (1 + e + pre * e) / (1 + e) ** 2
    dxx = torch.zeros_like(xx)
    dweight = torch.zeros_like(w["weight"])
    for k in range(W):
        dxx[:, k:k + L] += w["weight"][:, k] * dpre
        dweight[:, k] = (dpre * xx[:, k:k + L]).sum((0, 1))
    if w["dstate_out"] is not None:
        dxx[:, L:] += w["dstate_out"].transpose(1, 2)
    out = {"dweight": dweight, "dbias": dpre.sum((0, 1)), "dx": dxx[:, W - 1:].contiguous()}
    if w["state_in"] is not None:
        out["dstate_in"] = dxx[:, :W - 1].transpose(1, 2).contiguous()
    return out


def _exact_keep(case, seed, offset):
    """The keep factors from numpy's unsigned arithmetic."""
    n = case["rows"] * case["dim"]
    u32, u64 = np.uint32, np.uint64
    block = np.arange((n + 7) // 8, dtype=u64)
    split = lambda v: (u32(v & 0xFFFFFFFF), u32((v >> 32) & 0xFFFFFFFF))  # noqa: E731
    c = [block.astype(u32), (block >> u64(32)).astype(u32)] + [np.full(block.shape, v, u32) for v in split(offset)]
    k = list(split(seed))
    with np.errstate(over="ignore"):
        for _ in range(10):
            p0, p1 = c[0].astype(u64) * u64(0xD2511F53), c[2].astype(u64) * u64(0xCD9E8D57)
            c = [(p1 >> u64(32)).astype(u32) ^ c[1] ^ k[0], p1.astype(u32), (p0 >> u64(32)).astype(u32) ^ c[3] ^ k[1],
                 p0.astype(u32)]
            k = [u32((int(k[0]) + 0x9E3779B9) & 0xFFFFFFFF), u32((int(k[1]) + 0xBB67AE85) & 0xFFFFFFFF)]
    halves = np.stack(c, -1).astype("<u4").view("<u2").reshape(-1)[:n]
    t = math.floor(case["p"] * 65536 + 0.5)
    return np.where(halves >= t, 65536.0 / (65536 - t), 0.0).reshape(case["rows"], case["dim"])


def _exact_norm(case, w):
    """The forward as written, the gradients by the chain rule through each step of it."""
    y, d, eps = w["y"], case["dim"], w["eps"]
    silu = w["z"] / (1 + torch.exp(-w["z"])) if case["gate"] else None
    v = y * silu if case["gate"] else y
    var1 = v.square().sum(-1, keepdim=True) / d + eps
    n = v / var1.sqrt() * w["w_post"]
    k = 1.0
    if case["p"]:
        seed, offset = (int(x) for x in w["rng"].tolist())
        k = torch.from_numpy(_exact_keep(case, seed, offset)).to(y.device)
    R = w["residual"] + k * w["scale"] * n
    var2 = R.square().sum(-1, keepdim=True) / d + eps
    out = {"res_out": R, "out": R / var2.sqrt() * w["w_pre"]}
    if case["op"] == "norm_fwd":
        return out
    dRhat = w["dout"] * w["w_pre"]
    # d(R / sqrt(var2)): through the numerator and through var2
    dvar2 = -0.5 * (dRhat * R).sum(-1, keepdim=True) / var2 ** 1.5
    dR = w["dres"] + dRhat / var2.sqrt() + 2 * R * dvar2 / d
    dm = k * dR
    dvhat = dm * w["scale"] * w["w_post"]
    dvar1 = -0.5 * (dvhat * v).sum(-1, keepdim=True) / var1 ** 1.5
    dv = dvhat / var1.sqrt() + 2 * v * dvar1 / d
    out.update(dw_pre=(w["dout"] * R / var2.sqrt()).sum(0), dscale=(dm * n).sum(0),
               dw_post=(dm * w["scale"] * v / var1.sqrt()).sum(0), dresidual=dR)
    if case["gate"]:
        sig = 1 / (1 + torch.exp(-w["z"]))
        out.update(dy=dv * silu, dz=dv * y * (sig + w["z"] * sig * (1 - sig)))
    else:
        out["dy"] = dv
    return out
