"""The end of a residual block and its 8-bit activation checkpoints, measured operator by operator.

* ``store``  a matrix as an 8-bit checkpoint: e4m3 values with one power-of-two scale per group of columns or per row.
* ``load``   a checkpoint back in bf16 or fp32, or a norm's output again from the checkpoint of its input
  (y = value * scale * rstd_row * gain_column).
* ``fwd``    the norms after and before a block with its gate and residual scale:
  n = x rstd_post g_post,  s = a r + b gate n,  h = s rstd_pre g_pre;  x and s are kept as checkpoints where the
  case says so.  A row of the gate serves a span of rows (one sequence), or all of them.
* ``bwd``    the gradients of r, x, both gains and the gate, from full or 8-bit x and s.
* ``wgrad``  the weight gradient of a linear layer whose input was kept as a checkpoint: dW (+)= dY^T X.

Checkpoints: per group, scale = 2^k with the smallest k >= -126 for which max |v| <= 448 2^k over the finite
values, kept as the 8-bit code k + 127; a value is v / 2^k rounded to the nearest e4m3 value (ties to even).
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-5
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a short prompt's activations, odd in both sizes: launch latency
        dict(name="store_37x1021", op="store", rows=37, cols=1021, act="bf16", group=32, pad=0),
        # the activations of a 4 x 4096-token batch at hidden size 4096
        dict(name="store_16384x4096", op="store", rows=16384, cols=4096, act="bf16", group=128, pad=0),
        # odd rows inside a wider buffer, a scale per row, back in fp32
        dict(name="load_1501x2003", op="load", rows=1501, cols=2003, act="fp32", group=0, pad=5, norm=False),
        # the norm's output of a 4 x 4096-token batch again, for the recomputation of a block
        dict(name="load_norm_16384x4096", op="load", rows=16384, cols=4096, act="bf16", group=128, pad=0, norm=True),
        # one token at hidden size 4096
        dict(name="fwd_1x4096", op="fwd", rows=1, cols=4096, act="bf16", stream="bf16", gates=1, post=True, group=-1,
             pad=0, a=1.0, b=1.0),
        # a 4 x 4096-token batch, one gate vector per sequence, both checkpoints written
        dict(name="fwd8_16384x4096", op="fwd", rows=16384, cols=4096, act="bf16", stream="bf16", gates=4, post=True,
             group=128, pad=0, a=1.0, b=0.25),
        # hidden size 12288 with an fp32 stream, no gate and no checkpoints
        dict(name="fwd_8192x12288", op="fwd", rows=8192, cols=12288, act="bf16", stream="fp32", gates=0, post=True,
             group=-1, pad=0, a=1.0, b=1.0),
        # the backward pass of a short batch at hidden size 2048
        dict(name="bwd_64x2048", op="bwd", rows=64, cols=2048, act="bf16", stream="bf16", gates=1, post=True, group=-1,
             pad=0, a=1.0, b=1.0),
        # the backward pass of the 4 x 4096-token batch from its checkpoints
        dict(name="bwd8_16384x4096", op="bwd", rows=16384, cols=4096, act="bf16", stream="bf16", gates=4, post=True,
             group=128, pad=0, a=1.0, b=0.25),
        # the backward pass over odd rows, a gate vector for each of 21 sequences, from bf16 tensors
        dict(name="bwd_5003x2003", op="bwd", rows=5003, cols=2003, act="bf16", stream="bf16", gates=21, post=True,
             group=-1, pad=0, a=1.0, b=0.5),
        # a projection of hidden size 1024 over an odd number of tokens, added to an fp32 gradient
        dict(name="wgrad_1003x1024x1000", op="wgrad", tokens=1003, cin=1024, cout=1000, group=32, acc=True),
        # the up projection 4096 -> 11008 over 8192 tokens, bf16 gradient for the update
        dict(name="wgrad_8192x4096x11008", op="wgrad", tokens=8192, cin=4096, cout=11008, group=128, acc=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "load", "fwd", "bwd", "wgrad"])
    if op == "wgrad":
        while True:
            c = dict(op=op, tokens=_log(rng, 1, 16384), cin=16 * _log(rng, 4, 768), cout=8 * _log(rng, 8, 1536),
                     group=rng.choice([0, 32, 64, 128]), acc=rng.random() < 0.4)
            if c["tokens"] * c["cin"] * c["cout"] <= 8192 * 4096 * 11008:
                return c
    cols = _log(rng, 64, 16384)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    rows = min(_log(rng, 1, 65536), (16384 * 4096) // cols)
    c = dict(op=op, rows=rows, cols=cols, act=rng.choice(["bf16", "bf16", "fp32"]), pad=rng.choice([0, 0, 0, 8, 3]))
    if op in ("store", "load"):
        c["group"] = rng.choice([0, 32, 64, 128])
        if op == "load":
            c["norm"] = rng.random() < 0.5
        return c
    c["stream"] = rng.choice(["bf16", "bf16", "fp32"])
    c["gates"] = min(rows, rng.choice([0, 1, 1, 4, _log(rng, 2, 600)]))
    c["post"] = c["gates"] == 0 or rng.random() < 0.7
    c["group"] = rng.choice([-1, -1, 0, 32, 64, 128])
    c["a"], c["b"] = rng.choice([1.0, 0.8]), rng.choice([1.0, 0.25])
    return c


# ----------------------------------------------------------------- inputs ----

def _rows(rows, cols, pad, dtype, v=None):
    """A [rows, cols] view of a buffer with `pad` more columns a row, filled with v where given."""
    t = torch.empty(rows, cols + pad, dtype=DT.get(dtype, dtype), device="cuda")[:, :cols]
    if v is not None:
        t.copy_(v)
    return t


def _groups(cols, group):
    return 1 if group == 0 else -(-cols // group)


def _span(case):
    """Rows that one row of the gate serves."""
    return -(-case["rows"] // case["gates"])


def _gate_rows(case):
    return -(-case["rows"] // _span(case)) if case["gates"] else 0


def _kept(v, group, pad):
    """An 8-bit checkpoint of v in a buffer with `pad` more columns a row: values and scales."""
    q, scale = _quantize(v.float(), group)
    return _rows(v.shape[0], v.shape[1], pad, E4M3, q), scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if case["op"] == "wgrad":
        n, i, o = case["tokens"], case["cin"], case["cout"]
        x = normal(n, i) * torch.exp(0.5 * normal(i))
        s["q"], s["scale"] = _kept(x.to(torch.bfloat16), case["group"], 0)
        s["dy"] = (1e-3 * normal(n, o)).to(torch.bfloat16)
        # a micro-batch adds to the fp32 gradient of the ones before
        s["before"] = 1e-2 * normal(o, i) if case["acc"] else None
        s["dw"] = torch.empty(o, i, dtype=torch.float32 if case["acc"] else torch.bfloat16, device="cuda")
        return s
    rows, cols, pad, act = case["rows"], case["cols"], case["pad"], case["act"]
    # residual streams have channels of very different size
    wide = torch.exp(0.5 * normal(cols))
    gain = lambda: (1.0 + 0.1 * normal(cols)).to(DT[act])  # noqa: E731
    x = _rows(rows, cols, pad, act, normal(rows, cols) * wide)
    if case["op"] == "store":
        s["x"] = x
        s["q"] = _rows(rows, cols, pad, E4M3)
        s["scale"] = torch.empty(rows, _groups(cols, case["group"]), dtype=E8M0, device="cuda")
        return s
    if case["op"] == "load":
        s["q"], s["scale"] = _kept(x, case["group"], pad)
        s["rstd"] = torch.rsqrt(x.float().square().mean(dim=1) + EPS) if case["norm"] else None
        s["gain"] = gain() if case["norm"] else None
        s["y"] = _rows(rows, cols, pad, act)
        return s
    stream, n8 = case["stream"], _groups(cols, max(case["group"], 0))
    s["gain_post"] = gain() if case["post"] else None
    s["gain_pre"] = gain()
    s["gate"] = (0.5 + 0.2 * normal(_gate_rows(case), cols)).to(DT[act]) if case["gates"] else None
    if case["op"] == "fwd":
        s["x"] = x
        s["residual"] = _rows(rows, cols, pad, stream, normal(rows, cols) * wide)
        s["sum"], s["h"] = _rows(rows, cols, pad, stream), _rows(rows, cols, pad, act)
        s["rstd_post"], s["rstd_pre"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if case["group"] >= 0:
            s["x8"], s["sum8"] = _rows(rows, cols, pad, E4M3), _rows(rows, cols, pad, E4M3)
            s["x8_scale"], s["sum8_scale"] = (torch.empty(rows, n8, dtype=E8M0, device="cuda") for _ in range(2))
        return s
    total = _rows(rows, cols, pad, stream, normal(rows, cols) * wide)
    s["dh"] = _rows(rows, cols, pad, act, 1e-3 * normal(rows, cols))
    s["dsum"] = _rows(rows, cols, pad, stream, 1e-3 * normal(rows, cols))
    s["rstd_post"] = torch.rsqrt(x.float().square().mean(dim=1) + EPS)
    s["rstd_pre"] = torch.rsqrt(total.float().square().mean(dim=1) + EPS)
    if case["group"] >= 0:
        s["x8"], s["x8_scale"] = _kept(x, case["group"], pad)
        s["sum8"], s["sum8_scale"] = _kept(total, case["group"], pad)
    else:
        s["x"], s["sum"] = x, total
    s["dresidual"], s["dx"] = _rows(rows, cols, pad, stream), _rows(rows, cols, pad, act)
    s["dgain_pre"] = torch.empty(cols, device="cuda")
    s["dgain_post"] = torch.empty(cols, device="cuda") if case["post"] else None
    s["dgate"] = torch.empty(_gate_rows(case), cols, device="cuda") if case["gates"] else None
    return s


# ------------------------------------------------------------- plain form ----

def _power(k):
    """2^k in fp32 for integers -126 <= k <= 127, by its bits."""
    return ((k + 127) << 23).to(torch.int32).view(torch.float32)


def _quantize(v, group):
    """fp32 v as e4m3 values and e8m0 scales."""
    rows, cols = v.shape
    n = _groups(cols, group)
    width = cols if group == 0 else group
    padded = torch.nn.functional.pad(v, (0, n * width - cols)).reshape(rows, n, width)
    top = torch.where(torch.isfinite(padded), padded.abs(), 0.0).amax(dim=2)
    fraction, e = torch.frexp(top.double() / 448.0)      # top / 448 = fraction 2^e, fraction in [0.5, 1)
    k = torch.where(fraction > 0.5, e, e - 1)
    k = torch.where(top > 0, k, -126).clamp_min(-126)
    q = (padded * _power(-k)[:, :, None]).reshape(rows, n * width)[:, :cols].to(E4M3)
    return q, (k + 127).to(torch.uint8).view(E8M0)


def _restored(q, scale, group):
    """A checkpoint's values in fp32."""
    factor = scale.float()
    return q.float() * (factor if group == 0 else factor.repeat_interleave(group, dim=1)[:, :q.shape[1]])


def _gates(s):
    """The gate of each row in fp32; 1 without one."""
    c = s["case"]
    if s["gate"] is None:
        return 1.0
    return s["gate"].float().repeat_interleave(_span(c), dim=0)[:c["rows"]]


def _plain(s):
    c = s["case"]
    if c["op"] == "store":
        q, scale = _quantize(s["x"].float(), c["group"])
        return dict(q=q, scale=scale)
    if c["op"] == "load":
        y = _restored(s["q"], s["scale"], c["group"])
        if c["norm"]:
            y = y * s["rstd"][:, None] * s["gain"].float()
        return dict(y=y.to(s["y"].dtype))
    if c["op"] == "wgrad":
        dw = s["dy"].float().t() @ _restored(s["q"], s["scale"], c["group"])
        return dict(dw=s["before"] + dw if c["acc"] else dw.to(s["dw"].dtype))
    if c["op"] == "fwd":
        x = s["x"].float()
        rstd_post = torch.rsqrt(x.square().mean(dim=1) + EPS)
        n = x * rstd_post[:, None] * s["gain_post"].float() if c["post"] else x
        total = c["a"] * s["residual"].float() + c["b"] * (_gates(s) * n)
        rstd_pre = torch.rsqrt(total.square().mean(dim=1) + EPS)
        h = total * rstd_pre[:, None] * s["gain_pre"].float()
        out = dict(sum=total.to(s["sum"].dtype), h=h.to(s["h"].dtype), rstd_pre=rstd_pre)
        if c["post"]:
            out["rstd_post"] = rstd_post
        if c["group"] >= 0:
            out["x8"], out["x8_scale"] = _quantize(x, c["group"])
            out["sum8"], out["sum8_scale"] = _quantize(total, c["group"])
        return out
    if c["group"] >= 0:
        x, total = _restored(s["x8"], s["x8_scale"], c["group"]), _restored(s["sum8"], s["sum8_scale"], c["group"])
    else:
        x, total = s["x"].float(), s["sum"].float()
    dh, rp = s["dh"].float(), s["rstd_pre"][:, None]
    hat = total * rp
    dn = dh * s["gain_pre"].float()
    d = s["dsum"].float() + rp * (dn - hat * (dn * hat).mean(dim=1, keepdim=True))
    out = dict(dresidual=(c["a"] * d).to(s["dresidual"].dtype), dgain_pre=(dh * hat).sum(dim=0))
    branch = x * s["rstd_post"][:, None] if c["post"] else x
    du = c["b"] * d
    dn = du * _gates(s)
    if c["post"]:
        out["dgain_post"] = (dn * branch).sum(dim=0)
        dx = dn * s["gain_post"].float()
        dx = s["rstd_post"][:, None] * (dx - branch * (dx * branch).mean(dim=1, keepdim=True))
    else:
        dx = dn
    out["dx"] = dx.to(s["dx"].dtype)
    if c["gates"]:
        t = du * branch * s["gain_post"].float() if c["post"] else du * branch
        rows, span = _gate_rows(c), _span(c)
        t = torch.nn.functional.pad(t, (0, 0, 0, rows * span - c["rows"]))
        out["dgate"] = t.reshape(rows, span, c["cols"]).sum(dim=1)
    return out


def run(state):
    if not own:
        return _plain(state)
    from layer_optimizer_gb300 import native
    s, c = state, state["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "store":
        native.sf_checkpoint_store(s["x"], native.checkpoint(s["q"], s["scale"], c["group"]), stream=stream)
        return dict(q=s["q"], scale=s["scale"])
    if c["op"] == "load":
        native.sf_checkpoint_load(native.checkpoint(s["q"], s["scale"], c["group"]), s["y"], row_factor=s["rstd"],
                                  gain=s["gain"], stream=stream)
        return dict(y=s["y"])
    if c["op"] == "wgrad":
        if "ws" not in s:
            s["ws"] = torch.empty(native.sf_checkpoint_wgrad_workspace_bytes(c["tokens"], c["cout"], c["cin"]),
                                  dtype=torch.uint8, device="cuda")
        native.sf_checkpoint_wgrad(s["dy"], native.checkpoint(s["q"], s["scale"], c["group"]), s["dw"],
                                   base=s["before"], ws=s["ws"], stream=stream)
        return dict(dw=s["dw"])
    if "plan" not in s:
        s["plan"] = native.sandwich(EPS, residual_scale=c["a"], block_scale=c["b"],
                                    gate_span=_span(c) if c["gates"] else 0)
    keeps = c["group"] >= 0
    x8 = native.checkpoint(s["x8"], s["x8_scale"], c["group"]) if keeps else None
    sum8 = native.checkpoint(s["sum8"], s["sum8_scale"], c["group"]) if keeps else None
    if c["op"] == "fwd":
        native.sf_sandwich_norm_forward(s["plan"], s["x"], s["residual"], gain_post=s["gain_post"],
                                        gain_pre=s["gain_pre"], gate=s["gate"], sum=s["sum"], h=s["h"], x8=x8,
                                        sum8=sum8, rstd_post=s["rstd_post"] if c["post"] else None,
                                        rstd_pre=s["rstd_pre"], stream=stream)
        out = dict(sum=s["sum"], h=s["h"], rstd_pre=s["rstd_pre"])
        if c["post"]:
            out["rstd_post"] = s["rstd_post"]
        if keeps:
            out.update(x8=s["x8"], x8_scale=s["x8_scale"], sum8=s["sum8"], sum8_scale=s["sum8_scale"])
        return out
    if "ws" not in s:
        s["ws"] = torch.empty(native.sf_sandwich_norm_workspace_bytes(c["rows"], c["cols"]), dtype=torch.uint8,
                              device="cuda")
    native.sf_sandwich_norm_backward(s["plan"], dh=s["dh"], dsum=s["dsum"], x=x8 if keeps else s["x"],
                                     sum=sum8 if keeps else s["sum"], gain_post=s["gain_post"],
                                     gain_pre=s["gain_pre"], gate=s["gate"],
                                     rstd_post=s["rstd_post"] if c["post"] else None, rstd_pre=s["rstd_pre"],
                                     dresidual=s["dresidual"], dx=s["dx"], dgain_post=s["dgain_post"],
                                     dgain_pre=s["dgain_pre"], dgate=s["dgate"], ws=s["ws"], stream=stream)
    out = dict(dresidual=s["dresidual"], dgain_pre=s["dgain_pre"], dx=s["dx"])
    if c["post"]:
        out["dgain_post"] = s["dgain_post"]
    if c["gates"]:
        out["dgate"] = s["dgate"]
    return out


# ------------------------------------------------------------------- work ----

def work(case):
    if case["op"] == "wgrad":
        # dY and the checkpoint read, dW written (and read where it is added to)
        n, i, o = case["tokens"], case["cin"], case["cout"]
        return dict(bytes=2 * n * o + n * i + n * _groups(i, case["group"]) + (8 if case["acc"] else 2) * o * i,
                    flops=2 * n * i * o)
    rows, cols, a = case["rows"], case["cols"], SIZE[case["act"]]
    e, scales = rows * cols, rows * _groups(cols, max(case["group"], 0))
    if case["op"] == "store":
        return dict(bytes=e * (a + 1) + scales, flops=2 * e)
    if case["op"] == "load":
        return dict(bytes=e * (1 + a) + scales + (4 * rows + a * cols if case["norm"] else 0),
                    flops=e * (3 if case["norm"] else 1))
    st = SIZE[case["stream"]]
    small = a * cols * (1 + case["post"] + _gate_rows(case)) + 4 * rows * (1 + case["post"])
    if case["op"] == "fwd":
        return dict(bytes=e * (2 * a + 2 * st) + small + (2 * (e + scales) if case["group"] >= 0 else 0), flops=12 * e)
    kept = 2 * (e + scales) if case["group"] >= 0 else e * (a + st)
    return dict(bytes=e * (2 * a + 2 * st) + kept + small + 4 * cols * (1 + case["post"] + _gate_rows(case)),
                flops=24 * e)


# ------------------------------------------------------- 64-bit definition ----

def _power64(k):
    """2^k in 64 bits for whole k, by its bits."""
    return ((k.long() + 1023) << 52).view(torch.float64)


def _e4m3_64(v):
    """The nearest e4m3 values (4 significant bits, quantum 2^-9 below 2^-6, ties to even), |v| <= 448."""
    _, e = torch.frexp(v)
    quantum = _power64(torch.clamp(e - 4, min=-9))
    return torch.round(v / quantum) * quantum


def _quantize64(v, group):
    at = (torch.arange(v.shape[1], device="cuda") // (group or v.shape[1])).expand_as(v)
    top = torch.zeros(v.shape[0], _groups(v.shape[1], group), dtype=torch.float64, device="cuda")
    top.scatter_reduce_(1, at, v.abs(), "amax")
    k = torch.ceil(torch.log2(top / 448.0)).clamp(min=-126.0)
    # the logarithm may round across a whole number
    k = torch.where((top <= 448.0 * _power64(k - 1.0)) & (k > -126.0), k - 1.0, k)
    scale = _power64(torch.where(top > 448.0 * _power64(k), k + 1.0, k))
    return _e4m3_64(v / scale.gather(1, at)), scale


def _back64(q, scale, group):
    at = torch.arange(q.shape[1], device="cuda") // (group or q.shape[1])
    return q.double() * scale.double()[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    group = case["group"]
    if case["op"] == "store":
        q, scale = _quantize64(s["x"].double(), group)
        return dict(q=q, scale=scale)
    if case["op"] == "load":
        y = _back64(s["q"], s["scale"], group)
        if case["norm"]:
            y = s["gain"].double() * (s["rstd"].double()[:, None] * y)
        return dict(y=y)
    if case["op"] == "wgrad":
        x, out = _back64(s["q"], s["scale"], group), []
        for o in range(0, case["cout"], 2048):
            out.append(s["dy"][:, o:o + 2048].double().t() @ x)
        dw = torch.cat(out)
        return dict(dw=dw + s["before"].double() if case["acc"] else dw)
    rows, cols = case["rows"], case["cols"]
    at = torch.arange(rows, device="cuda") // _span(case) if case["gates"] else None
    gate = s["gate"].double()[at] if case["gates"] else torch.ones(1, 1, dtype=torch.float64, device="cuda")
    g_post = s["gain_post"].double() if case["post"] else torch.ones(cols, dtype=torch.float64, device="cuda")
    g_pre = s["gain_pre"].double()
    if case["op"] == "fwd":
        x = s["x"].double()
        r_post = 1.0 / torch.sqrt((x * x).sum(dim=1) / cols + EPS)
        n = g_post * (x * r_post[:, None]) if case["post"] else x
        total = s["residual"].double() * case["a"] + n * gate * case["b"]
        r_pre = 1.0 / torch.sqrt((total * total).sum(dim=1) / cols + EPS)
        out = dict(sum=total, h=g_pre * (total * r_pre[:, None]), rstd_pre=r_pre)
        if case["post"]:
            out["rstd_post"] = r_post
        if group >= 0:
            out["x8"], out["x8_scale"] = _quantize64(x, group)
            out["sum8"], out["sum8_scale"] = _quantize64(total, group)
        return out
    if group >= 0:
        x, total = _back64(s["x8"], s["x8_scale"], group), _back64(s["sum8"], s["sum8_scale"], group)
    else:
        x, total = s["x"].double(), s["sum"].double()
    dh, r_pre = s["dh"].double(), s["rstd_pre"].double()[:, None]
    inner = (dh * g_pre * total).sum(dim=1, keepdim=True) / cols
    d = s["dsum"].double() + r_pre * dh * g_pre - r_pre ** 3 * total * inner
    out = dict(dresidual=case["a"] * d, dgain_pre=(dh * total * r_pre).sum(dim=0))
    r_post = s["rstd_post"].double()[:, None] if case["post"] else torch.ones(1, 1, dtype=torch.float64, device="cuda")
    weight = case["b"] * d * gate * g_post
    out["dx"] = weight
    if case["post"]:
        inner = (weight * x).sum(dim=1, keepdim=True) / cols
        out["dx"] = r_post * weight - r_post ** 3 * x * inner
        out["dgain_post"] = (case["b"] * d * gate * x * r_post).sum(dim=0)
    if case["gates"]:
        out["dgate"] = torch.zeros(_gate_rows(case), cols, dtype=torch.float64, device="cuda")
        out["dgate"].index_add_(0, at, case["b"] * d * g_post * x * r_post)
    return out
