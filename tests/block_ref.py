"""Plain 64-bit forms of the operators around a recurrent block, with error bounds (CPU, torch float64).

Each function returns (values, bounds): what the operator returns, and how far a computation in fp32 may be off
before its output is rounded.  A bound is c * U * majorant: U = 2^-24 is half a step of fp32, the majorant the same
formula with every term's absolute value, and c the number of roundings on the longest path to the value, counting
one for each multiply, add and conversion and two for the hardware's exp2, rcp, rsq (1 ulp each).  sigma(v) =
rcp(1 + exp2(-v log2 e)) is relatively off by |v| + 6 of them: the argument's rounding is |v| log2(e) U, which exp2
turns into |v| U.  check() adds the rounding of the output's own type, half a step.  No value is taken from the
package."""
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}   # torch.finfo(t).eps / 2


def check(got, value, bound, what=""):
    """got (any dtype) against value within bound and the rounding of got's type; NaN and infinities must agree."""
    g = got.detach().cpu().double()
    assert g.shape == value.shape, (what, g.shape, value.shape)
    if g.numel() == 0:
        return 0.0
    fine = torch.isfinite(value)
    assert torch.equal(torch.isnan(g), torch.isnan(value)), "%s: NaN in other places" % what
    other = ~fine & ~torch.isnan(value)
    assert torch.equal(g[other], value[other]), "%s: infinities differ" % what
    tiny = 2.0 ** -120   # what flushing a subnormal intermediate may cost
    tol = (HALF[got.dtype] * value.abs() + (1 + HALF[got.dtype]) * bound + tiny)[fine]
    off = (g - value).abs()[fine]
    worst = float((off / tol).max()) if off.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g of the bound (off %.3g)" % (what, worst, float(off.max()))
    return worst


def d64(t):
    return None if t is None else t.detach().cpu().double()


# ---------------------------------------------------------------- gated scan

def _sig(v):
    """sigma(v) and its relative error in U."""
    return torch.sigmoid(v), v.abs() + 6


def gated_forward(x, r, i=None, A=None, reset=None, h0=None):
    """The recurrence token after token; autograd goes through it.  Returns y and h_final."""
    if A is not None:
        la = A * torch.sigmoid(r)
        a, s = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
        u = torch.sigmoid(i) * x
    else:
        a, s, u = torch.sigmoid(r), torch.sigmoid(-r), x
    h = torch.zeros_like(x[:, 0]) if h0 is None else h0
    ys = []
    for t in range(x.shape[1]):
        n = a[:, t] * h + s[:, t] * u[:, t]
        h = n if reset is None else torch.where(reset[:, t, None], u[:, t], n)
        ys.append(h)
    y = torch.stack(ys, 1) if ys else torch.zeros_like(x)
    return y, h


def gated(x, r, i=None, A=None, reset=None, h0=None, dout=None, dh_final=None):
    """Values and bounds: y, h_final and, with dout, dx, dr, di, dA, dh0."""
    x, r, i, A, h0, dout, dh_final = (d64(t) for t in (x, r, i, A, h0, dout, dh_final))
    reset = None if reset is None else reset.cpu().bool()
    b, L, d = x.shape
    g, cg = _sig(r)
    if A is not None:
        la = A * g
        a, m2 = torch.exp(la), -torch.expm1(2 * la)
        s = torch.sqrt(m2)
        gi, ci = _sig(i)
        u = gi * x
        ea = a * la.abs() * (cg + 1) + 4          # of a, absolute, in U: through la, and from 1 - m
        es = 0.5 * (cg + 10) + 3                  # of s, relative: m, 1 + a and their product halved by the root
        eu = ci + 2
        inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    else:
        a, s, u, inv = g, torch.sigmoid(-r), x, None
        ea, es, eu = a * cg, cg, torch.zeros_like(x)
    if reset is not None:
        rs = reset[..., None].expand_as(a)
        a, s = a.masked_fill(rs, 0.0), s.masked_fill(rs, 1.0)
        ea, es = ea.masked_fill(rs, 0.0), es.masked_fill(rs, 0.0)
    bb, eb = s * u, (s * u).abs() * (es + eu + 2)
    # h, a majorant of |h| over any order of the sums, and the error that the steps pile up
    h = torch.zeros(b, d, dtype=torch.float64) if h0 is None else h0
    hm, he = h.abs(), torch.zeros_like(h)
    H, HM, HE, HP, HPM, HPE = ([] for _ in range(6))
    for t in range(L):
        HP.append(h); HPM.append(hm); HPE.append(he)
        cut = (lambda v: v) if reset is None else (lambda v: torch.where(rs[:, t], torch.zeros_like(v), v))
        he = cut(a[:, t] * he + ea[:, t] * hm) + eb[:, t]
        h, hm = cut(a[:, t] * h) + bb[:, t], cut(a[:, t] * hm) + bb[:, t].abs()
        he = he + 3 * hm
        H.append(h); HM.append(hm); HE.append(he)
    if L == 0:
        z = torch.zeros_like(x)
        H, HM, HE, HP, HPM, HPE = (z for _ in range(6))
    else:
        H, HM, HE, HP, HPM, HPE = (torch.stack(v, 1) for v in (H, HM, HE, HP, HPM, HPE))
    # the maps of runs are combined over the rows of a wave, its workgroup's waves and the chunks: 24 roundings more
    val, bnd = {"y": H, "h_final": h}, {"y": U * (HE + 24 * HM), "h_final": U * (he + 24 * hm)}
    if dout is None:
        return val, bnd
    HPE = HPE + 24 * HPM
    mu = torch.zeros(b, d, dtype=torch.float64) if dh_final is None else dh_final
    mm, me = mu.abs(), torch.zeros_like(mu)
    LAM, LM, LE = ([None] * L for _ in range(3))
    for t in range(L - 1, -1, -1):
        lam, lm = dout[:, t] + mu, dout[:, t].abs() + mm
        le = me + 2 * lm
        LAM[t], LM[t], LE[t] = lam, lm, le
        cut = (lambda v: v) if reset is None else (lambda v: torch.where(rs[:, t], torch.zeros_like(v), v))
        mu, mm, me = cut(a[:, t] * lam), cut(a[:, t] * lm), cut(a[:, t] * le + (ea[:, t] + 1) * lm)
    if L == 0:
        LAM = LM = LE = torch.zeros_like(x)
    else:
        LAM, LM, LE = (torch.stack(v, 1) for v in (LAM, LM, LE))
    LE = LE + 24 * LM
    if dh_final is not None or h0 is not None:
        val["dh0"], bnd["dh0"] = mu, U * (me + 24 * mm)
    keep = torch.ones_like(x) if reset is None else (~rs).double()
    if A is not None:
        f = (HP - u * a * inv) * a * keep
        fm = (HPM + u.abs() * a * inv) * a * keep
        fe = (HPE * a + HPM * (ea + 2 * a) + u.abs() * inv * a * (2 * ea + a * (eu + es + 4))) * keep
        dla, dlm, dle = LAM * f, LM * fm, LE * fm + LM * (fe + 2 * fm)
        q = A * g * (1 - g)
        val["dr"] = dla * q
        bnd["dr"] = U * (A.abs() * g * ((1 - g) * (dle + dlm * (cg + 4)) + dlm * (g * cg + 2)))
        term, tm, te = dla * g, dlm * g, (dle + dlm * (cg + 2)) * g
        val["dA"] = term.sum((0, 1))
        # a lane's runs of every tile, its wave's rows, its waves, then the rows of the batch and the chunks
        bnd["dA"] = U * (te.sum((0, 1)) + (L / 64 + 64 + b + 40) * tm.sum((0, 1)))
        val["dx"], bnd["dx"] = LAM * s * gi, U * (s * gi * (LE + LM * (es + ci + 3)))
        val["di"] = LAM * s * u * (1 - gi)
        bnd["di"] = U * (s * u.abs() * ((1 - gi) * (LE + LM * (es + eu + 4)) + LM * (gi * ci + 2)))
    else:
        val["dx"], bnd["dx"] = LAM * s, U * (s * (LE + LM * (es + 2)))
        val["dr"] = LAM * s * a * (HP - x) * keep
        bnd["dr"] = U * keep * s * a * ((HPM + x.abs()) * (LE + LM * (es + cg + 6)) + LM * HPE)
    return val, bnd


# ---------------------------------------------------------------- conv1d

def conv_forward(x, weight, bias=None, state_in=None, silu=True):
    """out and state_out; autograd goes through it."""
    b, L, d = x.shape
    W = weight.shape[1]
    before = torch.zeros(b, W - 1, d, dtype=x.dtype) if state_in is None else state_in.transpose(1, 2)
    xx = torch.cat([before, x], 1)
    pre = sum(weight[:, k] * xx[:, k:k + L] for k in range(W)) + (0 if bias is None else bias)
    return (pre * torch.sigmoid(pre) if silu else pre), xx[:, L:].transpose(1, 2)


def conv_bwd(x, weight, dout, bias=None, state_in=None, silu=True, dstate_out=None):
    """Values and bounds: dx, dweight, dbias, dstate_in."""
    x, weight, dout, bias, state_in, dstate_out = (d64(t) for t in (x, weight, dout, bias, state_in, dstate_out))
    b, L, d = x.shape
    W = weight.shape[1]
    xx = torch.zeros(b, L + W - 1, d, dtype=torch.float64)
    xx[:, W - 1:] = x
    if state_in is not None:
        xx[:, :W - 1] = state_in.transpose(1, 2)
    dpre, de = dout, torch.zeros_like(dout)
    if silu:
        pre = sum(weight[:, k] * xx[:, k:k + L] for k in range(W)) + (0 if bias is None else bias)
        pm = sum((weight[:, k] * xx[:, k:k + L]).abs() for k in range(W)) + (0 if bias is None else bias.abs())
        s = torch.sigmoid(pre)
        dpre = dout * s * (1 + pre * (1 - s))
        # |silu''| <= 1/2 times the error of pre, and the roundings of s (1 + pre (1 - s)), whose terms are below
        # s (1 + |pre|)
        de = dout.abs() * (0.5 * (W + 1) * pm + s * (1 + pre.abs()) * (2 * (pre.abs() + 6) + 6))
    val, bnd = {}, {}
    dxx, dxe = torch.zeros_like(xx), torch.zeros_like(xx)
    dw, dwe = torch.zeros_like(weight), torch.zeros_like(weight)
    depth = 32 * max(1, L * b // 1024) + 120   # a run, the workgroup's blocks, its runs, the parts
    for k in range(W):
        dxx[:, k:k + L] += weight[:, k] * dpre
        dxe[:, k:k + L] += weight[:, k].abs() * (de + (W + 2) * dpre.abs())
        dw[:, k] = (dpre * xx[:, k:k + L]).sum((0, 1))
        dwe[:, k] = (xx[:, k:k + L].abs() * (de + depth * dpre.abs())).sum((0, 1))
    if dstate_out is not None and W > 1:
        dxx[:, L:] += dstate_out.transpose(1, 2)
        dxe[:, L:] += dstate_out.transpose(1, 2).abs() + dxx[:, L:].abs()
    val["dx"], bnd["dx"] = dxx[:, W - 1:], U * dxe[:, W - 1:]
    val["dweight"], bnd["dweight"] = dw, U * dwe
    val["dbias"], bnd["dbias"] = dpre.sum((0, 1)), U * (de + depth * dpre.abs()).sum((0, 1))
    val["dstate_in"], bnd["dstate_in"] = dxx[:, :W - 1].transpose(1, 2), U * dxe[:, :W - 1].transpose(1, 2)
    return val, bnd


# ---------------------------------------------------------------- block norm

def philox(block, seed, offset):
    """Philox4x32-10 of counter (block, offset), key seed, in Python's whole numbers: four words."""
    lo = 0xFFFFFFFF
    c = [block & lo, (block >> 32) & lo, offset & lo, (offset >> 32) & lo]
    k = [seed & lo, (seed >> 32) & lo]
    for _ in range(10):
        p0, p1 = 0xD2511F53 * c[0], 0xCD9E8D57 * c[2]
        c = [(p1 >> 32) ^ c[1] ^ k[0], p1 & lo, (p0 >> 32) ^ c[3] ^ k[1], p0 & lo]
        k = [(k[0] + 0x9E3779B9) & lo, (k[1] + 0xBB67AE85) & lo]
    return c


def keep_factors(rows, dim, p, rng):
    """1 / (1 - q / 65536) where kept, 0 where dropped."""
    q = int(p * 65536 + 0.5)
    seed, offset = (int(v) & (2 ** 64 - 1) for v in rng)
    n = rows * dim
    halves = []
    for block in range((n + 7) // 8):
        for w in philox(block, seed, offset):
            halves += [w & 0xFFFF, w >> 16]
    keep = torch.tensor(halves[:n], dtype=torch.int64).reshape(rows, dim) >= q
    return keep.double() * (65536.0 / (65536 - q))


def norm_forward(y, z=None, residual=None, w_post=None, scale=None, w_pre=None, keep=None, eps=1e-5):
    """R and out (None without w_pre); autograd goes through it."""
    v = y if z is None else y * z * torch.sigmoid(z)
    n = v if w_post is None else v / torch.sqrt((v * v).mean(-1, keepdim=True) + eps) * w_post
    m = n if scale is None else scale * n
    k = m if keep is None else m * keep
    R = k if residual is None else residual + k
    return R, None if w_pre is None else R / torch.sqrt((R * R).mean(-1, keepdim=True) + eps) * w_pre


def norm(y, dres=None, dout=None, z=None, residual=None, w_post=None, scale=None, w_pre=None, keep=None, eps=1e-5,
         grads=True):
    """Values and bounds for rows x dim inputs: res_out, out and the gradients."""
    y, dres, dout, z, residual, w_post, scale, w_pre = (d64(t) for t in (y, dres, dout, z, residual, w_post, scale, w_pre))
    rows, dim = y.shape
    one = torch.ones(dim, dtype=torch.float64)
    depth = 8 * 2 + 6 + 16          # a thread's values, its wave, the waves of a row
    if z is None:
        f, fd, cz = torch.ones_like(y), None, torch.zeros_like(y)
    else:
        sg = torch.sigmoid(z)
        f, cz = z * sg, z.abs() + 9
    v = y * f
    ev = v.abs() * cz
    mean = lambda t: t.mean(-1, keepdim=True)  # noqa: E731
    if w_post is None:
        r1, e1 = torch.ones(rows, 1, dtype=torch.float64), torch.zeros(rows, 1, dtype=torch.float64)
    else:
        r1 = 1 / torch.sqrt(mean(v * v) + eps)
        e1 = r1 * r1 * mean(v.abs() * ev) + depth / 2 + 4      # relative
    w = (one if w_post is None else w_post) * (one if scale is None else scale)
    k = torch.ones_like(y) if keep is None else keep
    m = v * r1 * w * k
    em = w.abs() * k * r1 * (ev + v.abs() * (e1 + 7))
    R = m if residual is None else residual + m
    eR = em + 2 * R.abs()
    val, bnd = {"res_out": R}, {"res_out": U * eR}
    dR, edR = (torch.zeros_like(y), torch.zeros_like(y)) if dres is None else (dres, dres.abs())
    if w_pre is not None:
        r2 = 1 / torch.sqrt(mean(R * R) + eps)
        e2 = r2 * r2 * mean(R.abs() * eR) + depth / 2 + 4
        val["out"] = R * r2 * w_pre
        bnd["out"] = U * w_pre.abs() * r2 * (eR + R.abs() * (e2 + 4))
        if grads:
            q = dout * w_pre
            Rh, eRh = R * r2, r2 * (eR + R.abs() * (e2 + 2))
            c, cm = mean(q * Rh), mean((q * Rh).abs())
            ec = mean(q.abs() * eRh) + (depth + 4) * cm
            val["dw_pre"] = (dout * Rh).sum(0)
            bnd["dw_pre"] = U * (dout.abs() * (eRh + (rows / 64 + 90) * Rh.abs())).sum(0)
            dR = dR + r2 * (q - Rh * c)
            edR = edR + r2 * (q.abs() * (e2 + 5) + eRh * c.abs() + Rh.abs() * (ec + (e2 + 6) * c.abs())) + 2 * dR.abs()
    if not grads:
        return val, bnd
    dm, edm = dR * k, (edR + 2 * dR.abs()) * k
    vh, evh = v * r1, r1 * (ev + v.abs() * (e1 + 2))
    S, eS = (dm * vh).sum(0), (edm * vh.abs() + dm.abs() * (evh + (rows / 64 + 90) * vh.abs())).sum(0)
    if w_post is not None:
        f2 = one if scale is None else scale
        val["dw_post"], bnd["dw_post"] = S * f2, U * f2.abs() * (eS + S.abs())
    if scale is not None:
        f2 = one if w_post is None else w_post
        val["dscale"], bnd["dscale"] = S * f2, U * f2.abs() * (eS + S.abs())
    dn, edn = dm * w, (edm + 2 * dm.abs()) * w.abs()
    if w_post is None:
        dv, edv = dn, edn + dn.abs()
    else:
        c, cm = mean(dn * vh), mean((dn * vh).abs())
        ec = mean(edn * vh.abs() + dn.abs() * evh) + (depth + 4) * cm
        dv = r1 * (dn - vh * c)
        edv = r1 * (edn + dn.abs() * (e1 + 4) + evh * c.abs() + vh.abs() * (ec + (e1 + 6) * c.abs()))
    val["dy"], bnd["dy"] = dv * f, U * (f.abs() * (edv + dv.abs() * (cz + 2)))
    if z is not None:
        t = sg * (1 + z * (1 - sg))
        tm = sg * (1 + z.abs())
        val["dz"] = dv * y * t
        bnd["dz"] = U * y.abs() * (edv * tm + dv.abs() * tm * (2 * cz + 6))
    if residual is not None:
        val["dresidual"], bnd["dresidual"] = dR, U * edR
    return val, bnd
