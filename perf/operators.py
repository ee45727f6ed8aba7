"""What the layer-norm and dropout operators are timed on: cases, inputs, the plain form of each operator and its value in 64 bits.

Rows are the active token slots of one call: a token slot holds a logical token (or padding, which no operator reads
or writes), and every value goes by the logical row, so the plain forms gather the active rows, compute, and put the
results back.  The dropout mask is Philox4x32-10 of (column / 8, logical row, offset) under a seed, 16 bits an element.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
M0, M1, W0, W1 = 0xD2511F53, 0xCD9E8D57, 0x9E3779B9, 0xBB67AE85      # Philox4x32 (Salmon et al., SC 2011)
M32 = 0xFFFFFFFF


def listed():
    def case(name, op, dtype, hidden, samples, longest, **more):
        c = {"name": name, "op": op, "dtype": dtype, "params": "same", "hidden": hidden, "heads": 1, "samples": samples,
             "longest": longest, "even": False, "layout": "packed", "p": 0.0}
        c.update(more)
        return c

    return [
        # decoding: one new token through one norm
        case("ln_fwd_one_token", "layernorm_fwd", "bf16", 4096, 1, 1),
        # prefill or a training step's forward pass over packed samples
        case("ln_fwd_4096", "layernorm_fwd", "bf16", 4096, 8, 4096),
        # an FP32 stream of an odd width, samples in fixed slots: half of the slots are padding
        case("ln_fwd_f32_1000_padded", "layernorm_fwd", "fp32", 1000, 33, 1009, layout="padded_right"),
        # the smallest training call
        case("ln_bwd_46x8", "layernorm_bwd", "bf16", 8, 8, 10),
        # a training step's backward pass with both parameter gradients
        case("ln_bwd_4096", "layernorm_bwd", "bf16", 4096, 8, 4096),
        # norms of query heads (width 128, 32 heads a token) in FP16, FP32 parameters
        case("ln_bwd_heads_128", "layernorm_bwd", "fp16", 128, 16, 1000, heads=32, params="fp32"),
        # decoding a batch of seven: residual add and norm in one call
        case("add_fwd_seven_tokens", "layernorm_add_fwd", "bf16", 5120, 7, 1),
        # a training step's block boundary: dropout, residual add, norm, over left-padded samples
        case("add_fwd_5120_padded", "layernorm_add_fwd", "bf16", 5120, 8, 4096, layout="padded_left", p=0.1),
        # its backward pass at a wide hidden size, samples in a permuted order
        case("add_bwd_8192_permuted", "layernorm_add_bwd", "bf16", 8192, 8, 4096, layout="permuted", p=0.1),
        # the same over an FP32 stream without dropout, a ragged small batch
        case("add_bwd_f32_1000", "layernorm_add_bwd", "fp32", 1000, 13, 333),
        # dropout alone, as behind an embedding: the largest call
        case("dropout_fwd_5120", "dropout_fwd", "bf16", 5120, 16, 4096, p=0.1),
        # its backward pass on a small padded batch
        case("dropout_bwd_264_padded", "dropout_bwd", "fp16", 264, 5, 257, layout="padded_right", p=0.25),
    ]


OPS = ("layernorm_fwd", "layernorm_bwd", "layernorm_add_fwd", "layernorm_add_bwd", "dropout_fwd", "dropout_bwd")


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp16", "fp32"))
    hidden = 8 * max(1, round(_log(rng, 1, (8192 if dtype == "fp32" else 16384) / 8)))
    heads = rng.choice((1, 1, 3, 8, 32)) if hidden <= 256 else 1
    most = (48 if dtype == "fp32" else 96) * 2 ** 20                  # elements in all slots
    slots = int(_log(rng, 1, max(2, min(2 ** 18, most // (hidden * heads)))))
    samples = min(slots, int(_log(rng, 1, 300)))
    p = rng.choice((0.0, 0.1, 0.5, round(rng.uniform(0.001, 0.9), 3))) if "add" in op else \
        rng.choice((0.1, 0.5, round(rng.uniform(0.001, 0.9), 3))) if "dropout" in op else 0.0
    return {"op": op, "dtype": dtype, "params": rng.choice(("same", "fp32")), "hidden": hidden, "heads": heads,
            "samples": samples, "longest": max(1, slots // samples), "even": rng.random() < 0.25,
            "layout": rng.choice(("packed", "padded_right", "padded_left", "permuted")), "p": p}


def _lengths(case):
    """Token counts of the samples: the first one has the longest, the others spread over 1 .. longest."""
    i = np.arange(case["samples"], dtype=np.int64)
    n = case["longest"]
    return np.full(i.size, n) if case["even"] else 1 + (n - 1 + i * (int(0.618 * n) | 1)) % n


def _slots(case):
    """Token id of every slot of the call, -1 in padding, and the number of logical tokens."""
    n = _lengths(case)
    off = np.cumsum(n) - n
    total = int(n.sum())
    if case["layout"] == "packed":
        ids = np.arange(total)
    elif case["layout"] == "permuted":
        order = np.arange(n.size)[::-1]
        start = np.cumsum(n[order]) - n[order]
        ids = np.arange(total) - np.repeat(start, n[order]) + np.repeat(off[order], n[order])
    else:
        pos = np.arange(case["longest"])[None, :]
        if case["layout"] == "padded_left":
            pos = pos - (case["longest"] - n)[:, None]
        ids = np.where((pos >= 0) & (pos < n[:, None]), off[:, None] + pos, -1).reshape(-1)
    return ids.astype(np.int32), total


def _inputs(case, seed):
    """Tensors of the call on the GPU: padding slots hold NaN."""
    ids, total = _slots(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, H, heads = DTYPES[case["dtype"]], case["hidden"], case["heads"]
    param = torch.float32 if case["params"] == "fp32" else dtype
    tok = torch.from_numpy(ids).to("cuda")
    padding = (tok < 0).view(-1, 1, 1) if bool((ids < 0).any()) else None

    def rows(scale, stream):
        t = torch.randn(ids.size, heads, H, generator=gen, device="cuda")
        if stream:                                                    # a residual stream: an offset and a scale of its own a row
            t = t * torch.rand(ids.size, heads, 1, generator=gen, device="cuda").mul_(4).add_(0.25)
            t = t + torch.randn(ids.size, heads, 1, generator=gen, device="cuda")
        t = (t * scale).to(dtype)
        return t if padding is None else t.masked_fill_(padding, float("nan"))

    op = case["op"]
    s = {"ids": ids, "n_logical": total, "tok": tok, "x": rows(1.0, "dropout" not in op)}
    if "layernorm" in op:
        s["weight"] = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(param)
        s["bias"] = (0.1 * torch.randn(H, generator=gen, device="cuda")).to(param)
    if op.endswith("_bwd") and "layernorm" in op:
        s["dy"] = rows(0.01, False)
    if "add" in op:
        s["res"] = rows(1.0, True) if op.endswith("fwd") else rows(0.01, False)
    s["rng"] = torch.randint(-2 ** 62, 2 ** 62, (2,), generator=gen, device="cuda", dtype=torch.int64)
    return s


def _buffers(case, s):
    """Outputs that a program keeps from step to step: padding in them stays as it is."""
    op, x = case["op"], s["x"]
    new = lambda: torch.zeros_like(x)                                 # noqa: E731
    stat = lambda: torch.zeros(x.shape[0] * x.shape[1], device="cuda")  # noqa: E731
    col = lambda: torch.zeros(x.shape[2], device="cuda")              # noqa: E731
    if op == "layernorm_fwd":
        return {"y": new(), "mean": stat(), "rstd": stat()}
    if op == "layernorm_bwd":
        return {"dx": new(), "dweight": col(), "dbias": col()}
    if op == "layernorm_add_fwd":
        return {"h": new(), "y": new(), "mean": stat(), "rstd": stat()}
    if op == "layernorm_add_bwd":
        return {"dh": new(), "dweight": col(), "dbias": col(), **({"dx": new()} if case["p"] else {})}
    return {"y" if op == "dropout_fwd" else "dx": new()}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"], s["out"] = case, _buffers(case, s)
    s["active"] = torch.nonzero(s["tok"] >= 0).reshape(-1)
    s["whole"] = bool((s["ids"] >= 0).all())
    if own:
        import invariant_rmsnorm_fwd_gb300 as rb
        grads = "layernorm" in case["op"] and case["op"].endswith("_bwd")
        s["layout"] = rb.call_layout(s["ids"], case["heads"], s["n_logical"], with_plan=grads)
        if grads:
            s["workspace"] = rb.LayerNormWorkspace(s["n_logical"] * case["heads"], case["hidden"])
        s["dropout"] = rb.Dropout(case["p"], s["rng"]) if case["p"] else None
    return s


def _own(s):
    import invariant_rmsnorm_fwd_gb300 as rb
    op, o, lay, drop = s["case"]["op"], s["out"], s["layout"], s["dropout"]
    if op == "layernorm_fwd":
        rb.layernorm_fwd(s["x"], s["weight"], s["bias"], lay, EPS, y=o["y"], mean=o["mean"], rstd=o["rstd"])
    elif op == "layernorm_add_fwd":
        rb.layernorm_add_fwd(s["x"], s["res"], s["weight"], s["bias"], lay, EPS, h=o["h"], y=o["y"], mean=o["mean"],
                             rstd=o["rstd"], dropout=drop)
    elif op == "dropout_fwd":
        rb.dropout_fwd(s["x"], lay, drop, y=o["y"])
    elif op == "dropout_bwd":
        rb.dropout_bwd(s["x"], lay, drop, dx=o["dx"])
    else:
        ws = s["workspace"]
        ws.begin()
        if op == "layernorm_bwd":
            rb.layernorm_bwd(s["x"], s["weight"], s["dy"], lay, EPS, dx=o["dx"], workspace=ws)
        else:
            rb.layernorm_add_bwd(s["x"], s["weight"], s["dy"], lay, EPS, dres=s["res"], dropout=drop, dh=o["dh"],
                                 dx=o.get("dx"), workspace=ws)
        ws.finalize(dweight=o["dweight"], dbias=o["dbias"])
    return o


def _product(a, m):
    """High and low 32 bits of a * m for a in 0 .. 2^32 - 1 (int64 lanes), in two halves of 16 bits."""
    low = (a & 0xFFFF) * m
    high = (a >> 16) * m + (low >> 16)
    return high >> 16, ((high & 0xFFFF) << 16) | (low & 0xFFFF)


def _keep(rng, rows, hidden, p):
    """The dropout mask of the logical rows, and the factor of what is kept."""
    t = int(round(p * 65536))
    k0, k1 = rng[0] & M32, (rng[0] >> 32) & M32
    shape = (rows.numel(), hidden // 8)
    a = torch.arange(shape[1], device=rows.device).expand(shape)
    b = rows.reshape(-1, 1).expand(shape)
    c, d = (rng[1] & M32).expand(shape), ((rng[1] >> 32) & M32).expand(shape)
    for i in range(10):
        (h0, l0), (h1, l1) = _product(a, M0), _product(c, M1)
        a, b, c, d = h1 ^ b ^ k0, l1, h0 ^ d ^ k1, l0
        k0, k1 = (k0 + W0) & M32, (k1 + W1) & M32
    u = torch.stack((a & 0xFFFF, a >> 16, b & 0xFFFF, b >> 16, c & 0xFFFF, c >> 16, d & 0xFFFF, d >> 16), dim=-1)
    return (u >= t).reshape(rows.numel(), hidden), (65536.0 / (65536 - t) if t < 65536 else 0.0)


def run(state):
    return _own(state) if own else _plain(state)


def _plain(s):
    case, o, act = s["case"], s["out"], s["active"]
    op, H, heads, dtype = case["op"], case["hidden"], case["heads"], DTYPES[case["dtype"]]

    def rows(t):                                                      # the active rows, in 32 bits
        return (t if s["whole"] else t[act]).reshape(-1, H).float()

    def put(name, v):
        v = v.to(o[name].dtype).reshape(act.numel(), heads, *v.shape[1:])
        to = o[name].view(-1, heads, *v.shape[2:])
        to.copy_(v) if s["whole"] else to.index_copy_(0, act, v)

    x = rows(s["x"])
    if case["p"]:
        tok = s["tok"].long() if s["whole"] else s["tok"][act].long()
        logical = (tok.reshape(-1, 1) * heads + torch.arange(heads, device=tok.device)).reshape(-1)
        keep, factor = _keep(s["rng"], logical, H, case["p"])
        drop = lambda v: torch.where(keep, v * factor, 0.0)           # noqa: E731
    else:
        drop = lambda v: v                                            # noqa: E731
    if "dropout" in op:
        put("y" if op == "dropout_fwd" else "dx", drop(x))
        return o
    if op == "layernorm_add_fwd":
        x = (drop(x) + rows(s["res"])).to(dtype)
        put("h", x)
        x = x.float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(1, keepdim=True) + EPS)
    xhat, w = d * rstd, s["weight"].float()
    if op.endswith("fwd"):
        put("y", xhat * w + s["bias"].float())
        put("mean", mean.reshape(-1))
        put("rstd", rstd.reshape(-1))
        return o
    dy = rows(s["dy"])
    g = dy * w
    dx = rstd * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    o["dweight"].copy_((dy * xhat).sum(0))
    o["dbias"].copy_(dy.sum(0))
    if op == "layernorm_bwd":
        put("dx", dx)
    else:
        dh = dx + rows(s["res"])
        put("dh", dh)
        if case["p"]:
            put("dx", drop(dh))
    return o


def _words(case):
    """Active slots and active rows of the call."""
    n = int(_lengths(case).sum())
    return n, n * case["heads"]


def work(case):
    tokens, rows = _words(case)
    slots = tokens if case["layout"] in ("packed", "permuted") else case["samples"] * case["longest"]
    op, H = case["op"], case["hidden"]
    size = 4 if case["dtype"] == "fp32" else 2
    tensors = {"layernorm_fwd": 2, "layernorm_bwd": 3, "layernorm_add_fwd": 4,
               "layernorm_add_bwd": 5 if case["p"] else 4, "dropout_fwd": 2, "dropout_bwd": 2}[op]
    param = 4 if case["params"] == "fp32" else size
    extra = 0 if "dropout" in op else 2 * H * param + 8 * rows if op.endswith("fwd") else H * param + 8 * H
    each = {"layernorm_fwd": 8, "layernorm_bwd": 16, "layernorm_add_fwd": 9, "layernorm_add_bwd": 18, "dropout_fwd": 1, "dropout_bwd": 1}[op]
    return {"bytes": float(tensors * rows * H * size + 4 * slots + extra), "flops": float(each * rows * H)}


def _kept64(seed, offset, rows, hidden, p):
    """The mask again, on host integers of 64 bits."""
    u64 = np.uint64
    low, sh = u64(M32), u64(32)
    seed, offset = u64(seed % 2 ** 64), u64(offset % 2 ** 64)
    ctr = [np.broadcast_to(np.arange(hidden // 8, dtype=u64), (rows.size, hidden // 8)),
           np.broadcast_to(rows.astype(u64)[:, None], (rows.size, hidden // 8)), offset & low, offset >> sh]
    key = [seed & low, seed >> sh]
    for i in range(10):
        p0, p1 = ctr[0] * u64(M0), ctr[2] * u64(M1)
        ctr = [(p1 >> sh) ^ ctr[1] ^ key[0], p1 & low, (p0 >> sh) ^ ctr[3] ^ key[1], p0 & low]
        key = [(key[0] + u64(W0)) & low, (key[1] + u64(W1)) & low]
    words = np.stack(ctr, axis=-1).astype(np.uint32).view(np.uint16)  # little-endian: low half first
    return words.reshape(rows.size, hidden) >= int(round(p * 65536))


def exact(case, seed):
    s = _inputs(case, seed)
    op, H, heads = case["op"], case["hidden"], case["heads"]
    tok = torch.from_numpy(s["ids"].astype(np.int64)).cuda()
    act = tok >= 0
    logical = (tok[act][:, None] * heads + torch.arange(heads, device="cuda")).reshape(-1)
    pick = lambda t: t[act].reshape(-1, H).double()                   # noqa: E731

    def full(v):
        out = torch.zeros(tok.numel(), heads, *v.shape[1:], dtype=torch.float64, device="cuda")
        out[act] = v.reshape(-1, heads, *v.shape[1:])
        return out if v.dim() > 1 else out.reshape(-1)

    mask = None
    if case["p"]:
        seed64, offset64 = (int(v) for v in s["rng"].cpu())
        mask = torch.from_numpy(_kept64(seed64, offset64, logical.cpu().numpy(), H, case["p"])).cuda()
        t = int(round(case["p"] * 65536))
        scale = 65536 / (65536 - t) if t < 65536 else 0.0
    kept = (lambda v: torch.zeros_like(v).masked_scatter_(mask, (v * scale)[mask])) if mask is not None else (lambda v: v)
    x = pick(s["x"])
    if op == "dropout_fwd":
        return {"y": full(kept(x))}
    if op == "dropout_bwd":
        return {"dx": full(kept(x))}
    out = {}
    if op == "layernorm_add_fwd":
        x = kept(x) + pick(s["res"])
        out["h"] = full(x)
        x = x.to(s["x"].dtype).double()                               # the norm takes the stored sum
    var, mu = torch.var_mean(x, dim=1, unbiased=False, keepdim=True)
    r = torch.rsqrt(var + EPS)
    w = s["weight"].double()
    if op.endswith("fwd"):
        return {**out, "y": full((x - mu) * (r * w) + s["bias"].double()), "mean": full(mu[:, 0]), "rstd": full(r[:, 0])}
    dy = pick(s["dy"])
    xh = (x - mu) * r
    a = dy * w
    dx = r * (a - (a.sum(1, keepdim=True) + xh * (a * xh).sum(1, keepdim=True)) / H)
    out = {"dweight": torch.einsum("gh,gh->h", dy, xh), "dbias": dy.sum(0)}
    if op == "layernorm_bwd":
        return {"dx": full(dx), **out}
    dh = dx + pick(s["res"])
    return {"dh": full(dh), **out, **({"dx": full(kept(dh))} if case["p"] else {})}
