"""The output end of a training step, measured operator by operator.

Four operators take a fine-tuning step from the last block's output to the
loss and back to the residual stream:

* ``dropout``  y = r + m o x / (1 - p): dropout with the residual's addition
  (or alone, which is also its backward pass).  The mask m comes from a
  counter-based generator and is never stored.
* ``norm``     s = r + dropout(x), h = s * rsqrt(mean(s^2) + eps) * g: the
  residual's addition and the root-mean-square norm, h in bf16 or fp32, or in
  8 bits (e4m3) with one fp32 scale per group of columns or per row.
* ``norm_bwd`` its gradients: of the stream, of x (through the mask) and of g.
* ``lce``      softmax cross-entropy of a linear output layer over the
  vocabulary in pieces: loss, per-token losses, dH and dW, without keeping
  the logits.

The generator: Philox-4x32 with 10 rounds (Salmon et al., "Parallel random
numbers: as easy as 1, 2, 3", 2011).  Eight columns of a row share one
counter (b mod 2^32, b / 2^32, offset mod 2^32, offset / 2^32) with
b = row * ceil(cols / 8) + col / 8 and the key (seed mod 2^32, seed / 2^32);
word j's low and high halves belong to the columns 8 (col / 8) + 2 j and + 1.
A column is kept where its 16 bits are at least t = round(65536 p), and kept
values are divided by 1 - t / 65536.

e4m3 outputs: per group, scale = max(max |h| / 448, 2^-126) and q = h / scale
rounded to the nearest e4m3 value; q is returned as a float8 tensor beside
its scales.
"""

import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}
EPS = 1e-5
IGNORE = -100


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # a short prompt's activations, odd in both sizes: launch latency
        dict(name="dropout_37x1021", op="dropout", rows=37, cols=1021, act="bf16", stream="bf16", residual=False,
             p=0.1, pad=0),
        # residual dropout of a 4 x 4096-token batch at hidden size 4096
        dict(name="dropout_add_16384x4096", op="dropout", rows=16384, cols=4096, act="bf16", stream="bf16",
             residual=True, p=0.1, pad=0),
        # one decoded token at hidden size 4096
        dict(name="norm_1x4096", op="norm", rows=1, cols=4096, act="bf16", stream="bf16", p=0.0, group=-1, pad=0),
        # the norm of a 4 x 4096-token batch, bf16 stream
        dict(name="norm_16384x4096", op="norm", rows=16384, cols=4096, act="bf16", stream="bf16", p=0.0, group=-1,
             pad=0),
        # hidden size 12288 (the Mistral-Large layer), fp32 stream, 8-bit output with a scale per 128 columns
        dict(name="norm8_8192x12288", op="norm", rows=8192, cols=12288, act="bf16", stream="fp32", p=0.0, group=128,
             pad=0),
        # odd rows and columns inside a wider buffer, dropout on, a scale per row
        dict(name="norm8_dropout_1501x2003", op="norm", rows=1501, cols=2003, act="bf16", stream="bf16", p=0.2,
             group=0, pad=5),
        # the backward pass of a short batch at hidden size 2048
        dict(name="norm_bwd_64x2048", op="norm_bwd", rows=64, cols=2048, act="bf16", stream="bf16", p=0.0, pad=0),
        # the backward pass of a 4 x 4096-token batch with dropout before the addition
        dict(name="norm_bwd_16384x4096", op="norm_bwd", rows=16384, cols=4096, act="bf16", stream="bf16", p=0.1,
             pad=0),
        # a few labelled tokens against a small vocabulary: latency of the whole chain
        dict(name="lce_16x1024x8000", op="lce", tokens=16, d=1024, vocab=8000),
        # odd token count and vocabulary
        dict(name="lce_1003x2048x50001", op="lce", tokens=1003, d=2048, vocab=50001),
        # the LLaMA-2-7B output layer on one sequence
        dict(name="lce_2048x4096x32000", op="lce", tokens=2048, d=4096, vocab=32000),
        # the Llama-3.1-8B output layer on 8192 tokens
        dict(name="lce_8192x4096x128256", op="lce", tokens=8192, d=4096, vocab=128256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm_bwd", "lce"])
    if op == "lce":
        tokens, vocab = _log(rng, 1, 8192), _log(rng, 1000, 128256)
        d = 8 * _log(rng, 8, 512)
        return dict(op=op, tokens=tokens, d=d, vocab=vocab)
    cols = _log(rng, 64, 16384)
    if rng.random() < 0.6:
        cols = max(64, cols // 64 * 64)
    rows = min(_log(rng, 1, 65536), (16384 * 4096) // cols)
    c = dict(op=op, rows=rows, cols=cols, act=rng.choice(["bf16", "bf16", "fp32"]),
             stream=rng.choice(["bf16", "bf16", "fp32"]), p=rng.choice([0.0, 0.05, 0.1, 0.25]),
             pad=rng.choice([0, 0, 0, 8, 3]))
    if op == "dropout":
        c["p"] = rng.choice([0.05, 0.1, 0.25, 0.5])
        c["residual"] = rng.random() < 0.6
    if op == "norm":
        c["group"] = rng.choice([-1, -1, 0, 32, 64, 128])
    return c


# ----------------------------------------------------------------- inputs ----

def _rows(rows, cols, pad, dtype, g=None, scale=None):
    """A [rows, cols] view of a buffer with `pad` more columns a row; normal values where a generator is given."""
    t = torch.empty(rows, cols + pad, dtype=DT.get(dtype, dtype), device="cuda")[:, :cols]
    if g is not None:
        v = torch.randn(rows, cols, generator=g, device="cuda")
        t.copy_(v if scale is None else v * scale)
    return t


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "lce":
        n, d, v = case["tokens"], case["d"], case["vocab"]
        s["H"] = torch.randn(n, d, generator=g, device="cuda", dtype=torch.bfloat16)
        s["W"] = (torch.randn(v, d, generator=g, device="cuda", dtype=torch.bfloat16) * 0.02)
        y = torch.randint(0, v, (n,), generator=g, device="cuda", dtype=torch.int32)
        # about one token in ten carries no label (padding, prompts); the first always does
        off = torch.rand(n, generator=g, device="cuda") < 0.1
        off[0] = False
        s["labels"] = torch.where(off, torch.full_like(y, IGNORE), y)
        s["loss"] = torch.empty(1, device="cuda")
        s["token_loss"] = torch.empty(n, device="cuda")
        s["dH"], s["dW"] = torch.empty_like(s["H"]), torch.empty_like(s["W"])
        return s
    rows, cols, pad, act, stream = case["rows"], case["cols"], case["pad"], case["act"], case["stream"]
    s["seed"] = int(torch.randint(0, 1 << 62, (1,), generator=g, device="cuda").item())
    s["offset"] = int(torch.randint(0, 1 << 40, (1,), generator=g, device="cuda").item())
    # residual streams have channels of very different size
    wide = torch.exp(0.5 * torch.randn(cols, generator=g, device="cuda"))
    gain = (1.0 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(DT[act])
    if case["op"] == "dropout":
        s["x"] = _rows(rows, cols, pad, act, g)
        s["residual"] = _rows(rows, cols, pad, stream, g, wide) if case["residual"] else None
        s["y"] = _rows(rows, cols, pad, stream if case["residual"] else act)
    elif case["op"] == "norm":
        s["x"] = _rows(rows, cols, pad, act, g)
        s["residual"] = _rows(rows, cols, pad, stream, g, wide)
        s["gain"] = gain
        s["sum"] = _rows(rows, cols, pad, stream)
        s["rstd"] = torch.empty(rows, device="cuda")
        if case["group"] < 0:
            s["h"] = _rows(rows, cols, pad, act)
        else:
            s["h8"] = _rows(rows, cols, pad, torch.float8_e4m3fn)
            s["scale"] = torch.empty(rows, _groups(case), device="cuda")
    else:
        s["dh"] = _rows(rows, cols, pad, act, g, 1e-3)
        s["dsum"] = _rows(rows, cols, pad, stream, g, 1e-3)
        s["sum"] = _rows(rows, cols, pad, stream, g, wide)
        s["gain"] = gain
        s["rstd"] = torch.rsqrt(s["sum"].float().square().mean(dim=1) + EPS)
        s["dresidual"] = _rows(rows, cols, pad, stream)
        s["dx"] = _rows(rows, cols, pad, act)
        s["dgain"] = torch.empty(cols, device="cuda")
    return s


def _groups(case):
    return 1 if case["group"] == 0 else -(-case["cols"] // case["group"])


# ------------------------------------------------------------- plain form ----

def _keep(rows, cols, p, seed, offset):
    """The mask [rows, cols] of the counter-based generator, and the factor of the kept values."""
    low = 0xFFFFFFFF
    nv = -(-cols // 8)
    b = torch.arange(rows * nv, device="cuda", dtype=torch.int64)
    c0, c1 = b & low, b >> 32
    c2, c3 = torch.full_like(b, offset & low), torch.full_like(b, offset >> 32)
    k0, k1 = seed & low, seed >> 32
    for _ in range(10):
        m0, m1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((m1 >> 32) & low) ^ c1 ^ k0, m1 & low, ((m0 >> 32) & low) ^ c3 ^ k1, m0 & low)
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack([c0, c1, c2, c3], dim=1)
    bits = torch.stack([words & 0xFFFF, words >> 16], dim=2).reshape(rows, nv * 8)[:, :cols]
    t = _threshold(p)
    return bits >= t, 65536.0 / (65536 - t)


def _threshold(p):
    return int(math.floor(p * 65536 + 0.5))


def _dropped(x, p, seed, offset):
    if p == 0.0:
        return x
    keep, factor = _keep(x.shape[0], x.shape[1], p, seed, offset)
    return torch.where(keep, x * factor, torch.zeros_like(x))


def _plain(s):
    c = s["case"]
    if c["op"] == "lce":
        H, W, y = s["H"].float(), s["W"].float(), s["labels"].long()
        on = y != IGNORE
        n = on.sum()
        at = torch.where(on, y, 0)[:, None]
        z = H @ W.t()
        top = z.amax(dim=1, keepdim=True)
        lse = top + torch.exp(z - top).sum(dim=1, keepdim=True).log()
        token_loss = torch.where(on, (lse - z.gather(1, at))[:, 0], 0.0)
        loss = (token_loss.sum() / n).reshape(1)
        z.sub_(lse).exp_()
        z.scatter_add_(1, at, torch.full_like(lse, -1.0))
        z.mul_((on / n)[:, None])
        return dict(loss=loss, token_loss=token_loss, dH=(z @ W).to(s["dH"].dtype), dW=(z.t() @ H).to(s["dW"].dtype))
    if c["op"] == "dropout":
        y = _dropped(s["x"].float(), c["p"], s["seed"], s["offset"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return dict(y=y.to(s["y"].dtype))
    if c["op"] == "norm":
        a = s["residual"].float() + _dropped(s["x"].float(), c["p"], s["seed"], s["offset"])
        rstd = torch.rsqrt(a.square().mean(dim=1) + EPS)
        h = a * rstd[:, None] * s["gain"].float()
        out = dict(sum=a.to(s["sum"].dtype), rstd=rstd)
        if c["group"] < 0:
            return dict(out, h=h.to(s["h"].dtype))
        rows, cols, n = c["rows"], c["cols"], _groups(c)
        width = cols if c["group"] == 0 else c["group"]
        padded = torch.nn.functional.pad(h, (0, n * width - cols)).reshape(rows, n, width)
        scale = (padded.abs().amax(dim=2) / 448.0).clamp_min(2.0 ** -126)
        q = (padded / scale[:, :, None]).clamp(-448.0, 448.0).reshape(rows, n * width)[:, :cols]
        return dict(out, h8=q.to(torch.float8_e4m3fn), scale=scale)
    dh, a, gain, rstd = s["dh"].float(), s["sum"].float(), s["gain"].float(), s["rstd"][:, None]
    hat = a * rstd
    dn = dh * gain
    ds = s["dsum"].float() + rstd * (dn - hat * (dn * hat).mean(dim=1, keepdim=True))
    dx = _dropped(ds, c["p"], s["seed"], s["offset"])
    return dict(dresidual=ds.to(s["dresidual"].dtype), dx=dx.to(s["dx"].dtype), dgain=(dh * hat).sum(dim=0))


def run(state):
    if not own:
        return _plain(state)
    from layer_optimizer_gb300 import native
    s, c = state, state["case"]
    stream = torch.cuda.current_stream()
    if c["op"] == "lce":
        n, d, v = c["tokens"], c["d"], c["vocab"]
        if "ws" not in s:
            s["ws"] = torch.empty(native.lce_vocab_workspace_bytes(n, d, v), dtype=torch.uint8, device="cuda")
        native.lce_vocab_forward_backward(s["H"], s["W"], s["labels"], loss=s["loss"], token_loss=s["token_loss"],
                                          dH=s["dH"], dW=s["dW"], ws=s["ws"], ignore_index=IGNORE, stream=stream)
        return dict(loss=s["loss"], token_loss=s["token_loss"], dH=s["dH"], dW=s["dW"])
    rng = native.rng(s["seed"], s["offset"]) if c["p"] > 0 else None
    if c["op"] == "dropout":
        native.sf_dropout(s["x"], s["y"], p=c["p"], rng=rng, residual=s["residual"], stream=stream)
        return dict(y=s["y"])
    if c["op"] == "norm":
        if c["group"] < 0:
            native.sf_add_rmsnorm_forward(s["x"], s["residual"], s["gain"], EPS, sum=s["sum"], h=s["h"],
                                          rstd=s["rstd"], p=c["p"], rng=rng, stream=stream)
            return dict(sum=s["sum"], rstd=s["rstd"], h=s["h"])
        native.sf_add_rmsnorm_forward(s["x"], s["residual"], s["gain"], EPS, sum=s["sum"], h8=s["h8"],
                                      h8_scale=s["scale"], group=c["group"], rstd=s["rstd"], p=c["p"], rng=rng,
                                      stream=stream)
        return dict(sum=s["sum"], rstd=s["rstd"], h8=s["h8"], scale=s["scale"])
    if "ws" not in s:
        s["ws"] = torch.empty(native.sf_add_rmsnorm_workspace_bytes(c["rows"], c["cols"]), dtype=torch.uint8,
                              device="cuda")
    native.sf_add_rmsnorm_backward(s["dh"], s["sum"], s["gain"], s["rstd"], dsum=s["dsum"], dresidual=s["dresidual"],
                                   dx=s["dx"], dgain=s["dgain"], p=c["p"], rng=rng, ws=s["ws"], stream=stream)
    return dict(dresidual=s["dresidual"], dx=s["dx"], dgain=s["dgain"])


# ------------------------------------------------------------------- work ----

def work(case):
    if case["op"] == "lce":
        # H, W and the labels read, dH, dW and the losses written; the logits and the two gradient products
        n, d, v = case["tokens"], case["d"], case["vocab"]
        return dict(bytes=2 * (2 * n * d + 2 * v * d) + 8 * n + 4, flops=6 * n * d * v)
    rows, cols, a, st = case["rows"], case["cols"], SIZE[case["act"]], SIZE[case["stream"]]
    e = rows * cols
    if case["op"] == "dropout":
        return dict(bytes=e * (a + 2 * st if case["residual"] else 2 * a), flops=2 * e)
    if case["op"] == "norm":
        out = e * a if case["group"] < 0 else e + 4 * rows * _groups(case)
        return dict(bytes=e * (a + 2 * st) + out + cols * a + 4 * rows, flops=6 * e)
    return dict(bytes=e * (2 * a + 3 * st) + cols * (a + 4) + 4 * rows, flops=12 * e)


# ------------------------------------------------------- 64-bit definition ----

def _mask64(rows, cols, p, seed, offset):
    """The kept elements by the generator's definition, in numpy on the host, 2^20 counters at a time."""
    u = np.uint64
    per_row = (cols + 7) // 8
    out = np.empty((rows * per_row, 8), dtype=bool)
    threshold = _threshold(p)
    for lo in range(0, rows * per_row, 1 << 20):
        b = np.arange(lo, min(rows * per_row, lo + (1 << 20)), dtype=np.uint64)
        x = [b % u(1 << 32), b // u(1 << 32), np.full_like(b, offset % (1 << 32)), np.full_like(b, offset // (1 << 32))]
        for r in range(10):
            key0, key1 = u((seed % (1 << 32) + r * 0x9E3779B9) % (1 << 32)), u((seed // (1 << 32) + r * 0xBB67AE85) % (1 << 32))
            left, right = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
            x = [(right // u(1 << 32)) ^ x[1] ^ key0, right % u(1 << 32), (left // u(1 << 32)) ^ x[3] ^ key1, left % u(1 << 32)]
        for j in range(4):
            out[lo:lo + b.size, 2 * j] = x[j] % u(1 << 16) >= threshold
            out[lo:lo + b.size, 2 * j + 1] = x[j] // u(1 << 16) >= threshold
    return out.reshape(rows, per_row * 8)[:, :cols]


def _drop64(v, case, s):
    if case["p"] == 0.0:
        return v
    keep = torch.from_numpy(_mask64(case["rows"], case["cols"], case["p"], s["seed"], s["offset"])).to(v.device)
    return torch.where(keep, v / (1.0 - _threshold(case["p"]) / 65536), 0.0)


def _e4m3_64(v):
    """The nearest e4m3 values (4 significant bits, quantum 2^-9 below 2^-6, ties to even), |v| <= 448."""
    _, e = torch.frexp(v)
    quantum = torch.ldexp(torch.ones_like(v), torch.clamp(e - 4, min=-9))
    return torch.clamp(torch.round(v / quantum) * quantum, -448.0, 448.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lce":
        n, d, v = case["tokens"], case["d"], case["vocab"]
        grads = 6.0 * n * d * v < 4e12   # the products' time in 64 bits
        H, y = s["H"].double(), s["labels"].long()
        labelled = torch.nonzero(y >= 0)[:, 0]
        count = int(labelled.numel())
        step = 4096
        best, total = torch.full((n,), -math.inf, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
        for v0 in range(0, v, step):
            z = H @ s["W"][v0:v0 + step].double().t()
            new = torch.maximum(best, z.max(dim=1).values)
            total = total * torch.exp(best - new) + torch.exp(z - new[:, None]).sum(dim=1)
            best = new
        lse = best + torch.log(total)
        own_w = s["W"][y[labelled]].double()
        losses = torch.zeros(n, dtype=torch.float64, device="cuda")
        losses[labelled] = lse[labelled] - (H[labelled] * own_w).sum(dim=1)
        dH = dW = None
        if grads:
            dH, dW = torch.zeros_like(H), torch.zeros(v, d, dtype=torch.float64, device="cuda")
            dH[labelled] -= own_w / count
            dW.index_add_(0, y[labelled], -H[labelled] / count)
            for v0 in range(0, v, step):
                w = s["W"][v0:v0 + step].double()
                prob = torch.exp(H[labelled] @ w.t() - lse[labelled][:, None]) / count
                dH[labelled] += prob @ w
                dW[v0:v0 + step] += prob.t() @ H[labelled]
        return dict(loss=losses.sum().reshape(1) / count, token_loss=losses, dH=dH, dW=dW)
    if case["op"] == "dropout":
        y = _drop64(s["x"].double(), case, s)
        return dict(y=y if s["residual"] is None else y + s["residual"].double())
    if case["op"] == "norm":
        a = s["residual"].double() + _drop64(s["x"].double(), case, s)
        rstd = 1.0 / torch.sqrt((a * a).sum(dim=1) / case["cols"] + EPS)
        h = s["gain"].double() * (a * rstd[:, None])
        if case["group"] < 0:
            return dict(sum=a, rstd=rstd, h=h)
        width = case["group"] or case["cols"]
        scales, q = [], torch.empty_like(h)
        for c0 in range(0, case["cols"], width):
            block = h[:, c0:c0 + width]
            scales.append(torch.clamp(block.abs().max(dim=1).values / 448.0, min=2.0 ** -126))
            q[:, c0:c0 + width] = _e4m3_64(block / scales[-1][:, None])
        return dict(sum=a, rstd=rstd, h8=q, scale=torch.stack(scales, dim=1))
    dh, a, gain, rstd = s["dh"].double(), s["sum"].double(), s["gain"].double(), s["rstd"].double()[:, None]
    inner = (dh * gain * a).sum(dim=1, keepdim=True) / case["cols"]
    ds = s["dsum"].double() + rstd * dh * gain - rstd ** 3 * a * inner
    return dict(dresidual=ds, dx=_drop64(ds, case, s), dgain=(dh * a * rstd).sum(dim=0))
