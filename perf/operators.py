"""What a sublayer of the network is wrapped in, as measured calls: the norms
before and after a block with its gate and residual scale, rotary positions,
and dropout whose mask is never stored.

Activations are [B, H, L, d]: token (b, l) has D = H d features, its H head
rows side by side. "head" layout is that array, contiguous; "token" layout is
[B, L, H, d] in memory, seen as [B, H, L, d].

  norm      h = xhat w + b, xhat = (x - m) r, r = 1 / sqrt(mean (x - m)^2 + eps)
            over a token's D features; m = mean x ("layer") or 0 ("rms").
  residual  y = beta x + alpha drop(gate * post(f)), h = norm(y as stored);
            post = a norm or the identity; gate: none, a learned vector ([D],
            or [B, D] with "gate_batch"), or sigmoid(z) with z like f.
  dropout   element c of row (b H + h) L + l takes 16-bit lane c mod 8 of
            Philox4x32-10 (Salmon et al. 2011) with key = seed and counter =
            (row ceil(d / 8) + c / 8, offset); it is kept when that lane is at
            least t = round(65536 p), and then multiplied by 65536 / (65536 - t).
  rope      the first `rot` features of every head row turn in pairs, (2i,
            2i + 1) or (i, i + rot / 2), by the angle position * freq_i, and
            are multiplied by amp; the rest of the row is copied.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
MASK32 = 0xFFFFFFFF


# ------------------------------------------------------------------ the cases
def _norm(name, B, H, L, dtype, do, kind, layout="head", bias=True):
    return dict(name=name, op="norm", B=B, H=H, L=L, d=64, dtype=dtype, do=do, kind=kind,
                layout=layout, bias=bias)


def _residual(name, B, H, L, dtype, do, post="", norm="", gate="", gate_batch=False, p=0.0,
              alpha=1.0, beta=1.0, layout="head"):
    return dict(name=name, op="residual", B=B, H=H, L=L, d=64, dtype=dtype, do=do, post=post,
                norm=norm, gate=gate, gate_batch=gate_batch, p=p, alpha=alpha, beta=beta,
                layout=layout)


def _rope(name, B, H, L, dtype, do, rot=64, interleaved=False, scaling="", factor=1.0, far=False,
          layout="head"):
    return dict(name=name, op="rope", B=B, H=H, L=L, d=64, dtype=dtype, do=do, rot=rot,
                interleaved=interleaved, scaling=scaling, factor=factor, far=far, layout=layout)


def _dropout(name, B, H, L, dtype, do, p):
    return dict(name=name, op="dropout", B=B, H=H, L=L, d=64, dtype=dtype, do=do, p=p,
                layout="head")


def listed():
    return [
        # one token each of four sequences, before a block while generating
        _norm("norm-decode", 4, 8, 1, "bf16", "fwd", "rms", bias=False),
        # the 64K-token training step: norm before the attention, with its gradients
        _norm("norm-64k-train", 1, 8, 65536, "bf16", "train", "layer"),
        # a wide model in token layout, the largest call here
        _norm("norm-wide-train", 4, 64, 8192, "bf16", "train", "rms", layout="token", bias=False),
        # one token each of sixteen sequences: add, norm after the block, norm before the next
        _residual("residual-decode", 16, 16, 1, "bf16", "fwd", post="rms", norm="rms"),
        # the 12K-token image batch, forward: dropout, add, next norm
        _residual("residual-12k-fwd", 4, 8, 12288, "bf16", "fwd", norm="layer", p=0.1),
        # the 64K-token training step with every part on
        _residual("residual-64k-train", 1, 8, 65536, "bf16", "train", post="layer", norm="layer",
                  gate="vector", p=0.1, alpha=0.5),
        # ragged batch in 32 bits, elementwise gate computed by the network
        _residual("residual-gated-f32", 3, 5, 1001, "f32", "train", norm="rms", gate="sigmoid",
                  p=0.05),
        # one token each of 64 sequences, far into a long context
        _rope("rope-decode", 64, 8, 1, "bf16", "fwd", far=True),
        # the 64K-token training step, forward and backward
        _rope("rope-64k-train", 1, 8, 65536, "bf16", "train"),
        # half a million tokens, half of each head, scaled for the long context
        _rope("rope-halfmillion", 1, 2, 524288, "bf16", "fwd", rot=32, interleaved=True,
              scaling="yarn", factor=8.0),
        # the 64K-token training step, both directions with one seed
        _dropout("dropout-64k-train", 1, 8, 65536, "bf16", "train", 0.1),
        # an odd batch in 32 bits
        _dropout("dropout-ragged-f32", 7, 3, 4001, "f32", "fwd", 0.25),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "residual", "residual", "rope", "dropout"))
    H = _log_int(rng, 1, 64)
    B = _log_int(rng, 1, 64)
    L = 1 if rng.random() < 0.2 else _log_int(rng, 2, 262144)
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    layout = rng.choice(("head", "token"))
    do = rng.choice(("fwd", "train"))
    if op == "norm":
        c = _norm("", B, H, L, dtype, do, rng.choice(("layer", "rms")), layout,
                  rng.random() < 0.5)
    elif op == "residual":
        gate = rng.choice(("", "vector", "sigmoid"))
        c = _residual("", B, H, L, dtype, do, rng.choice(("", "layer", "rms")),
                      rng.choice(("", "layer", "rms")), gate,
                      gate == "vector" and rng.random() < 0.3, rng.choice((0.0, 0.1, 0.3)),
                      rng.choice((1.0, 0.5)), rng.choice((1.0, 1.5)), layout)
    elif op == "rope":
        scaling = rng.choice(("", "linear", "ntk", "yarn"))
        c = _rope("", B, H, L, dtype, do, rng.choice((64, 64, 48, 32, 20)), rng.random() < 0.5,
                  scaling, rng.choice((2.0, 8.0)) if scaling else 1.0, rng.random() < 0.3, layout)
    else:
        c = _dropout("", B, H, L, dtype, do, rng.choice((0.05, 0.1, 0.5)))
    while work(c)["bytes"] > 1.2e9:
        c["B"], c["L"] = max(1, c["B"] // 2), c["L"] if c["B"] > 1 else c["L"] // 2 + 1
    del c["name"]
    return c


def work(c):
    n = c["B"] * c["H"] * c["L"] * c["d"]
    e = 4 if c["dtype"] == "f32" else 2
    train = c["do"] == "train"
    if c["op"] == "norm":            # x -> h;  x, dh, dres -> dx
        units, flops = (6, 24) if train else (2, 8)
    elif c["op"] == "residual":      # x, f -> y, h;  dy, dh, y, f -> dx, df  (+ z, dz)
        gated, normed = c["gate"] == "sigmoid", bool(c["norm"])
        units = 3 + normed + gated
        flops = 6 + 8 * normed + 8 * bool(c["post"])
        if train:
            # without a norm dx is beta dy, a scaling that is written all the same
            units += 4 + 2 * normed + 2 * gated
            flops *= 3
    elif c["op"] == "rope":
        units, flops = (4, 6) if train else (2, 3)
    else:
        units, flops = (4, 2) if train else (2, 1)
    # parameters and their gradients (32 bits), positions and frequencies
    D, more = c["H"] * c["d"], 0
    if c["op"] == "norm":
        more = 4 * D * (1 + c["bias"])
    elif c["op"] == "residual":
        more = 4 * D * sum({"": 0, "rms": 1, "layer": 2}[c[k]] for k in ("post", "norm"))
        if c["gate"] == "vector":
            more += 4 * D * (c["B"] if c["gate_batch"] else 1)
    elif c["op"] == "rope":
        return {"bytes": float(n * e * units + 4 * c["B"] * c["L"] * c["far"] + 4 * c["rot"]),
                "flops": float(n * flops)}
    more *= 3 if train else 1      # read in both directions, gradients written
    return {"bytes": float(n * e * units + more), "flops": float(n * flops)}


# ------------------------------------------------------------------ the inputs
_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _act(c, g, scale=1.0, shift=0.0):
    B, H, L, d = c["B"], c["H"], c["L"], c["d"]
    shape = (B, L, H, d) if c["layout"] == "token" else (B, H, L, d)
    t = torch.empty(shape, dtype=_DT[c["dtype"]], device="cuda").normal_(shift, scale, generator=g)
    return t.transpose(1, 2) if c["layout"] == "token" else t


def _vec(n, g, scale, shift):
    return torch.empty(n, dtype=torch.float32, device="cuda").normal_(shift, scale, generator=g)


def _freqs(rot, scaling, factor):
    """Radians a position, in 64 bits, and the multiplier of the turned features
    (linear: Chen et al. 2023; ntk: a larger base; yarn: Peng et al. 2023)."""
    base = 10000.0
    if scaling == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    amp = 1.0
    if scaling == "linear":
        f = [v / factor for v in f]
    elif scaling == "yarn":
        turns = [65536 * v / (2 * math.pi) for v in f]     # trained on 65536 positions
        ramp = [min(1.0, max(0.0, (r - 1.0) / (32.0 - 1.0))) for r in turns]
        f = [v * k + v / factor * (1.0 - k) for v, k in zip(f, ramp)]
        amp = 0.1 * math.log(factor) + 1.0
    return f, amp


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    D = c["H"] * c["d"]
    train = c["do"] == "train"
    s = {"case": c}
    if c["op"] == "norm":
        s["x"] = _act(c, g, 1.5, 0.2)
        s["w"] = _vec(D, g, 0.1, 1.0)
        s["b"] = _vec(D, g, 0.1, 0.0) if c["bias"] else None
        if train:
            s["dh"], s["dres"] = _act(c, g), _act(c, g)
    elif c["op"] == "residual":
        s["x"], s["f"] = _act(c, g), _act(c, g, 0.8, 0.1)
        s["gate"] = None
        if c["gate"] == "vector":
            s["gate"] = _vec(D * (c["B"] if c["gate_batch"] else 1), g, 0.2, 0.7)
            if c["gate_batch"]:
                s["gate"] = s["gate"].view(c["B"], D)
        elif c["gate"] == "sigmoid":
            s["gate"] = _act(c, g)
        s["w_post"] = _vec(D, g, 0.1, 1.0) if c["post"] else None
        s["b_post"] = _vec(D, g, 0.1, 0.0) if c["post"] == "layer" else None
        s["w"] = _vec(D, g, 0.1, 1.0) if c["norm"] else None
        s["b"] = _vec(D, g, 0.1, 0.0) if c["norm"] == "layer" else None
        if train:
            s["dy"] = _act(c, g)
            s["dh"] = _act(c, g) if c["norm"] else None
            # the backward comes after the rest of the network: its y is a stored
            # (or, in a reversible layer, rebuilt) array that the program has in hand
            s["y"] = _act(c, g, 1.2) if c["norm"] else None
    elif c["op"] == "rope":
        s["x"] = _act(c, g)
        f, s["amp"] = _freqs(c["rot"], c["scaling"], c["factor"])
        s["freqs"] = torch.tensor(f, dtype=torch.float64, device="cuda")
        s["pos"] = None
        if c["far"]:
            s["pos"] = torch.randint(0, 1 << 20, (c["B"], c["L"]), generator=g, device="cuda",
                                     dtype=torch.int32)
        if train:
            s["dy"] = _act(c, g)
    else:
        s["x"] = _act(c, g)
        if train:
            s["dy"] = _act(c, g)
    s["seed"] = (seed * 0x9E3779B97F4A7C15 + 12345) % (1 << 64)
    s["offset"] = seed % 1000003
    if own:
        from efficient_transformer_lsh_b200 import sublayer
        kw = dict(dtype=c["dtype"], d=c["d"])
        dims = (c["B"], c["H"], c["L"])
        lay = c["layout"]
        if c["op"] == "norm":
            s["runner"] = sublayer.Norm(*dims, kind=c["kind"], eps=EPS, x_layout=lay,
                                        h_layout=lay, **kw)
        elif c["op"] == "residual":
            s["runner"] = sublayer.Residual(*dims, post=c["post"] or None, norm=c["norm"] or None,
                                            gate=c["gate"] or None, gate_batch=c["gate_batch"],
                                            p=c["p"], alpha=c["alpha"], beta=c["beta"], eps=EPS,
                                            x_layout=lay, f_layout=lay, **kw)
        elif c["op"] == "rope":
            scaling = None
            if c["scaling"]:
                scaling = (c["scaling"], c["factor"]) + ((65536,) if c["scaling"] == "yarn" else ())
            s["runner"] = sublayer.Rotary(*dims, rot=c["rot"], interleaved=c["interleaved"],
                                          scaling=scaling, x_layout=lay, y_layout=lay, **kw)
        else:
            s["runner"] = sublayer.Dropout(*dims, c["p"], x_layout=lay, y_layout=lay, **kw)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    c, r = s["case"], s["runner"]
    train = c["do"] == "train"
    if c["op"] == "norm":
        out = {"h": r.forward(s["x"], s["w"], s["b"])}
        if train:
            out["dx"], out["dw"], out["db"] = r.backward(s["x"], s["dh"], s["w"], s["b"],
                                                         dres=s["dres"])
    elif c["op"] == "residual":
        par = dict(gate=s["gate"], w_post=s["w_post"], b_post=s["b_post"], w=s["w"], b=s["b"],
                   seed=s["seed"], offset=s["offset"])
        out = {}
        out["y"], out["h"] = r.forward(s["x"], s["f"], **par)
        if train:
            g = r.backward(s["dy"], s["f"], y=s["y"], dh=s["dh"], **par)
            out.update(zip(("dx", "df", "dgate", "dw_post", "db_post", "dw", "db"), g))
    elif c["op"] == "rope":
        out = {"y": r.forward(s["x"], s["pos"])}
        if train:
            out["dx"] = r.backward(s["dy"], s["pos"])
    else:
        out = {"y": r.forward(s["x"], s["seed"], s["offset"])}
        if train:
            out["dx"] = r.backward(s["dy"], s["seed"], s["offset"])
    return {k: v for k, v in out.items() if v is not None}


def _row(v):
    """A [D] or [B, D] vector against [B, L, D]."""
    return v[:, None, :] if v.dim() == 2 else v


def _tokens(t):
    """[B, H, L, d] as [B, L, H d] in 32 bits."""
    B, H, L, d = t.shape
    return t.transpose(1, 2).reshape(B, L, H * d).float()


def _heads(t, c):
    """[B, L, D] in 32 bits as [B, H, L, d] in the case's type."""
    return t.reshape(c["B"], c["L"], c["H"], c["d"]).transpose(1, 2).to(_DT[c["dtype"]])


def _stats(x, kind):
    """(xhat, r)"""
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _norm_back(a, xhat, r, kind):
    t = a - xhat * (a * xhat).mean(-1, keepdim=True)
    if kind == "layer":
        t = t - a.mean(-1, keepdim=True)
    return t * r


def _mul_hi_lo(a, m):
    p = a * m                          # wraps modulo 2^64: the bits are those of the product
    return (p >> 32) & MASK32, p & MASK32


def _keep(c, seed, offset):
    """Truth values [B, H, L, d]."""
    rows, groups = c["B"] * c["H"] * c["L"], (c["d"] + 7) // 8
    n = torch.arange(rows * groups, dtype=torch.int64, device="cuda")
    x0, x1 = n & MASK32, n >> 32
    x2 = torch.full_like(n, offset & MASK32)
    x3 = torch.full_like(n, offset >> 32)
    k0, k1 = seed & MASK32, seed >> 32
    for _ in range(10):
        h0, l0 = _mul_hi_lo(x0, 0xD2511F53)
        h1, l1 = _mul_hi_lo(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ k0, l1, h0 ^ x3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & MASK32, (k1 + 0xBB67AE85) & MASK32
    w = torch.stack((x0, x1, x2, x3), -1)
    lanes = torch.stack((w & 0xFFFF, w >> 16), -1).reshape(rows, groups * 8)[:, :c["d"]]
    t = int(round(c["p"] * 65536))
    return (lanes >= t).reshape(c["B"], c["H"], c["L"], c["d"])


def _drop_scale(p):
    t = int(round(p * 65536))
    return 65536.0 / (65536 - t) if t < 65536 else 0.0


def _run_plain(s):
    c = s["case"]
    train = c["do"] == "train"
    if c["op"] == "norm":
        x = _tokens(s["x"])
        xhat, r = _stats(x, c["kind"])
        h = xhat * s["w"]
        if c["bias"]:
            h = h + s["b"]
        out = {"h": _heads(h, c)}
        if train:
            dh = _tokens(s["dh"])
            out["dx"] = _heads(_tokens(s["dres"]) + _norm_back(dh * s["w"], xhat, r, c["kind"]), c)
            out["dw"] = (dh * xhat).sum((0, 1))
            if c["bias"]:
                out["db"] = dh.sum((0, 1))
        return out
    if c["op"] == "residual":
        return _residual_plain(s, c, train)
    if c["op"] == "rope":
        pos = s["pos"] if s["pos"] is not None else torch.arange(c["L"], device="cuda")
        # in 64 bits: at position 2^20 an angle in 32 bits is off by up to 0.03
        a = pos.double()[..., None] * s["freqs"]
        cos, sin = (s["amp"] * torch.cos(a)).float(), (s["amp"] * torch.sin(a)).float()
        if cos.dim() == 3:
            cos, sin = cos[:, None], sin[:, None]
        out = {"y": _turn(s["x"], cos, sin, c)}
        if train:
            out["dx"] = _turn(s["dy"], cos, -sin, c)
        return out
    keep, k = _keep(c, s["seed"], s["offset"]), _drop_scale(c["p"])
    zero = torch.zeros((), dtype=torch.float32, device="cuda")
    out = {"y": torch.where(keep, s["x"].float() * k, zero).to(s["x"].dtype)}
    if train:
        out["dx"] = torch.where(keep, s["dy"].float() * k, zero).to(s["dy"].dtype)
    return out


def _turn(x, cos, sin, c):
    r = c["rot"]
    v = x[..., :r].float()
    if c["interleaved"]:
        p, q = v[..., 0::2], v[..., 1::2]
        v = torch.stack((p * cos - q * sin, q * cos + p * sin), -1).flatten(-2)
    else:
        p, q = v[..., :r // 2], v[..., r // 2:]
        v = torch.cat((p * cos - q * sin, q * cos + p * sin), -1)
    return torch.cat((v.to(x.dtype), x[..., r:]), -1)


def _residual_plain(s, c, train):
    f = _tokens(s["f"])
    if c["post"]:
        fhat, rf = _stats(f, c["post"])
        u = fhat * s["w_post"]
        if s["b_post"] is not None:
            u = u + s["b_post"]
    else:
        u = f
    g = None
    if c["gate"] == "vector":
        g = _row(s["gate"])
    elif c["gate"] == "sigmoid":
        g = 1.0 / (1.0 + torch.exp(-_tokens(s["gate"])))
    v = u if g is None else g * u
    keep, k = None, 1.0
    if c["p"] > 0:
        keep = _keep(c, s["seed"], s["offset"]).transpose(1, 2).reshape(v.shape)
        k = _drop_scale(c["p"])
        v = torch.where(keep, v * k, torch.zeros((), device="cuda"))
    out = {"y": _heads(c["beta"] * _tokens(s["x"]) + c["alpha"] * v, c)}
    if c["norm"]:
        yhat, ry = _stats(_tokens(out["y"]), c["norm"])
        h = yhat * s["w"]
        if s["b"] is not None:
            h = h + s["b"]
        out["h"] = _heads(h, c)
    if not train:
        return out
    t = _tokens(s["dy"])
    if c["norm"]:
        dh = _tokens(s["dh"])
        yhat, ry = _stats(_tokens(s["y"]), c["norm"])
        t = t + _norm_back(dh * s["w"], yhat, ry, c["norm"])
        out["dw"] = (dh * yhat).sum((0, 1))
        if s["b"] is not None:
            out["db"] = dh.sum((0, 1))
    out["dx"] = _heads(c["beta"] * t, c)
    q = c["alpha"] * t
    if keep is not None:
        q = torch.where(keep, q * k, torch.zeros((), device="cuda"))
    du = q if g is None else q * g
    if c["gate"] == "vector":
        out["dgate"] = (q * u).sum(1) if c["gate_batch"] else (q * u).sum((0, 1))
    elif c["gate"] == "sigmoid":
        out["dgate"] = _heads(q * u * g * (1.0 - g), c)
    if c["post"]:
        out["dw_post"] = (du * fhat).sum((0, 1))
        if s["b_post"] is not None:
            out["db_post"] = du.sum((0, 1))
        du = _norm_back(du * s["w_post"], fhat, rf, c["post"])
    out["df"] = _heads(du, c)
    return out


# ------------------------------------------------------------------ 64 bits
def _mask64(c, seed, offset):
    """The dropout's multiplier [B, H, L, d] in 64 bits, from numpy's unsigned integers."""
    rows, groups = c["B"] * c["H"] * c["L"], -(-c["d"] // 8)
    u = np.uint64
    low = u(0xFFFFFFFF)
    ctr = np.arange(rows * groups, dtype=u)
    words = [ctr & low, ctr >> u(32), np.full_like(ctr, offset & MASK32),
             np.full_like(ctr, offset >> 32)]
    key = [seed & MASK32, seed >> 32]
    for i in range(10):
        k = [u((key[0] + i * 0x9E3779B9) & MASK32), u((key[1] + i * 0xBB67AE85) & MASK32)]
        a, b = words[0] * u(0xD2511F53), words[2] * u(0xCD9E8D57)
        words = [(b >> u(32)) ^ words[1] ^ k[0], b & low, (a >> u(32)) ^ words[3] ^ k[1], a & low]
    bits = np.empty((rows * groups, 8), dtype=np.uint16)
    for j in range(8):
        bits[:, j] = ((words[j // 2] >> u(16 * (j % 2))) & u(0xFFFF)).astype(np.uint16)
    bits = bits.reshape(rows, groups * 8)[:, :c["d"]]
    t = round(65536 * c["p"])
    kept = torch.from_numpy(bits.astype(np.int32)).to("cuda") >= t
    m = kept.double() * (65536.0 / (65536 - t) if t < 65536 else 0.0)
    return m.view(c["B"], c["H"], c["L"], c["d"])


def _norm64(x, kind, w, b):
    """[B, H, L, d] in 64 bits, over heads and features."""
    B, H, L, d = x.shape
    mean = x.mean((1, 3), keepdim=True) if kind == "layer" else 0.0
    z = x - mean
    z = z / torch.sqrt(z.pow(2).mean((1, 3), keepdim=True) + EPS)
    z = z * w.view(1, H, 1, d)
    return z if b is None else z + b.view(1, H, 1, d)


def _leaf(t):
    return None if t is None else t.detach().double().requires_grad_(True)


def _exact_rope(c, x, pos, sign):
    """Pairs as complex numbers, turned by exp(i angle)."""
    f, amp = _freqs(c["rot"], c["scaling"], c["factor"])
    z = x.double()
    r = c["rot"]
    pos = torch.arange(c["L"], device="cuda") if pos is None else pos
    ang = sign * torch.einsum("...l,i->...li", pos.to(torch.float64),
                              torch.tensor(f, dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.full_like(ang, amp), ang)
    turn = turn.unsqueeze(1) if turn.dim() == 3 else turn
    first = torch.arange(0, r, 2) if c["interleaved"] else torch.arange(r // 2)
    second = first + (1 if c["interleaved"] else r // 2)
    w = torch.complex(z[..., first], z[..., second]) * turn
    z = z.clone()
    z[..., first], z[..., second] = w.real, w.imag
    return z


def exact(case, seed):
    """64 bits throughout, gradients by differentiating the formulas above."""
    c = dict(case)
    if c["B"] * c["H"] * c["L"] * c["d"] > 1 << 28:
        return None
    s = prepare(case, seed)
    train = c["do"] == "train"
    if c["op"] == "rope":
        out = {"y": _exact_rope(c, s["x"], s["pos"], 1.0)}
        if train:
            out["dx"] = _exact_rope(c, s["dy"], s["pos"], -1.0)
        return out
    if c["op"] == "dropout":
        m = _mask64(c, s["seed"], s["offset"])
        out = {"y": s["x"].double() * m}
        if train:
            out["dx"] = s["dy"].double() * m
        return out
    with torch.enable_grad():
        x, w, b = _leaf(s["x"]), _leaf(s["w"]), _leaf(s["b"])
        if c["op"] == "norm":
            h = _norm64(x, c["kind"], w, b)
            out = {"h": h.detach()}
            if train:
                have = [(k, v) for k, v in (("dx", x), ("dw", w), ("db", b)) if v is not None]
                got = torch.autograd.grad(h, [v for _, v in have], s["dh"].double())
                out.update((k, v) for (k, _), v in zip(have, got))
                out["dx"] = out["dx"] + s["dres"].double()
            return out
        f, gate, wp, bp = (_leaf(s[k]) for k in ("f", "gate", "w_post", "b_post"))
        v = _norm64(f, c["post"], wp, bp) if c["post"] else f
        if c["gate"] == "vector":
            v = v * gate.view(-1, c["H"], 1, c["d"])
        elif c["gate"] == "sigmoid":
            v = v * torch.special.expit(gate)
        if c["p"] > 0:
            v = v * _mask64(c, s["seed"], s["offset"])
        y = c["beta"] * x + c["alpha"] * v
        out = {"y": y.detach()}
        if c["norm"]:
            out["h"] = _norm64(y, c["norm"], w, b).detach()
        if train:
            ends, grads = [y], [s["dy"].double()]
            if c["norm"]:
                # the backward's y, with the derivative of the formula's
                at = y + (s["y"].double() - y).detach()
                ends.append(_norm64(at, c["norm"], w, b))
                grads.append(s["dh"].double())
            have = [(k, t) for k, t in (("dx", x), ("df", f), ("dgate", gate), ("dw_post", wp),
                                        ("db_post", bp), ("dw", w), ("db", b)) if t is not None]
            got = torch.autograd.grad(ends, [t for _, t in have], grads)
            out.update((k, t) for (k, _), t in zip(have, got))
        return out
