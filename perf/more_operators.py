"""What the rotary operators are timed on: cases, inputs, the plain form of each operator and its value in 64 bits.

Rotary positions turn the pairs of columns of a head by angles that grow with the token's position; in front of them
stands, in the fused operators, an RMS norm of every head of the queries and of the keys.  Queries and keys are the
heads of the token slots of one call: a slot holds a logical token (or padding, which no operator reads or writes).
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    def case(name, op, dtype, q_heads, k_heads, head_dim, samples, longest, **more):
        c = {"name": name, "op": op, "dtype": dtype, "params": "same", "q_heads": q_heads, "k_heads": k_heads,
             "head_dim": head_dim, "rotary_dim": head_dim, "first": 0, "pairs": "half", "base": 10000.0, "factor": 1.0,
             "ramp": 0, "scale": 1.0, "samples": samples, "longest": longest, "even": False, "context": 0,
             "layout": "packed", "joined": False}
        c.update(more)
        return c

    return [
        # decoding one token far into its context, queries and keys as they come out of one joined projection
        case("rot_fwd_one_token", "rotary_fwd", "bf16", 32, 8, 128, 1, 1, context=100000, joined=True),
        # prefill of packed samples from a joined projection
        case("rot_fwd_prefill", "rotary_fwd", "bf16", 32, 8, 128, 8, 4096, joined=True),
        # part of the head in interleaved pairs, frequencies stretched for a long context, half of the slots padding
        case("rot_fwd_part_interleaved", "rotary_fwd", "fp16", 16, 16, 64, 33, 1009, rotary_dim=32, pairs="interleaved",
             factor=8.0, ramp=8192, scale=1.2, context=65536, layout="padded_right"),
        # a training step's backward pass, samples in a permuted order: the largest rotation
        case("rot_bwd_permuted", "rotary_bwd", "bf16", 32, 8, 128, 16, 4096, layout="permuted"),
        # an FP32 stream with odd sizes: seven query heads share a key head of 80 columns, of which 20 turn
        case("rot_bwd_f32_odd", "rotary_bwd", "fp32", 7, 1, 80, 13, 333, rotary_dim=20, layout="padded_left"),
        # decoding one token: norm and rotation in one call
        case("qk_fwd_one_token", "qk_norm_rotary_fwd", "bf16", 32, 8, 128, 1, 1, context=100000, joined=True),
        # decoding a batch of 64 samples, each at a position of its own
        case("qk_fwd_batch", "qk_norm_rotary_fwd", "fp16", 28, 4, 128, 64, 1, context=32768, base=500000.0, joined=True),
        # prefill of packed samples from a joined projection
        case("qk_fwd_prefill", "qk_norm_rotary_fwd", "bf16", 32, 8, 128, 16, 4096, joined=True),
        # an FP32 stream of an odd head width in interleaved pairs, half of the slots padding
        case("qk_fwd_f32_odd", "qk_norm_rotary_fwd", "fp32", 9, 3, 72, 33, 1009, pairs="interleaved", layout="padded_right"),
        # the smallest training call
        case("qk_bwd_46_tokens", "qk_norm_rotary_bwd", "bf16", 4, 2, 16, 8, 10),
        # a training step's backward pass with both weight gradients: the largest call
        case("qk_bwd_prefill", "qk_norm_rotary_bwd", "bf16", 32, 8, 128, 16, 4096),
        # one key head for all queries, wide heads of which the last quarter turns, FP32 weights, a permuted order
        case("qk_bwd_shared_key", "qk_norm_rotary_bwd", "fp16", 16, 1, 256, 8, 4096, rotary_dim=64, first=192,
             pairs="interleaved", params="fp32", layout="permuted"),
    ]


OPS = ("rotary_fwd", "rotary_bwd", "qk_norm_rotary_fwd", "qk_norm_rotary_bwd")


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(OPS)
    dtype = rng.choice(("bf16", "bf16", "bf16", "fp16", "fp32"))
    D = rng.choice((64, 80, 96, 128, 128, 192, 256, 8 * max(2, round(_log(rng, 2, 64)))))
    q_heads = max(1, round(_log(rng, 1, 64)))
    k_heads = rng.choice((1, q_heads, max(1, q_heads // 4), max(1, q_heads // 8)))
    pairs = rng.choice(("half", "interleaved"))
    r = max(4, rng.choice((D, D, D // 2, D // 4, rng.randint(4, D))) // 4 * 4)
    most = (64 if dtype == "fp32" else 128) * 2 ** 20                 # elements in all slots
    slots = int(_log(rng, 1, max(2, min(2 ** 18, most // ((q_heads + k_heads) * D)))))
    samples = min(slots, int(_log(rng, 1, 300)))
    factor = rng.choice((1.0, 1.0, 4.0, round(rng.uniform(1.5, 32), 2)))
    return {"op": op, "dtype": dtype, "params": rng.choice(("same", "fp32")), "q_heads": q_heads, "k_heads": k_heads,
            "head_dim": D, "rotary_dim": r, "first": rng.choice((0, 0, D - r, 2 * rng.randint(0, (D - r) // 2))),
            "pairs": pairs, "base": rng.choice((10000.0, 500000.0)), "factor": factor,
            "ramp": rng.choice((0, 8192)) if factor > 1 else 0, "scale": rng.choice((1.0, round(rng.uniform(0.8, 1.5), 3))),
            "samples": samples, "longest": max(1, slots // samples), "even": rng.random() < 0.25,
            "context": rng.choice((0, int(_log(rng, 1, 2 ** 20)))),
            "layout": rng.choice(("packed", "padded_right", "padded_left", "permuted")),
            "joined": rng.random() < 0.5 and op.endswith("fwd")}


def _lengths(case):
    """Token counts of the samples: the first one has the longest, the others spread over 1 .. longest."""
    i = np.arange(case["samples"], dtype=np.int64)
    n = case["longest"]
    return np.full(i.size, n) if case["even"] else 1 + (n - 1 + i * (int(0.618 * n) | 1)) % n


def _slots(case, seed):
    """Token id (-1 in padding) and position of every slot of the call, and the number of logical tokens.  A sample's
    positions start where its context ends: at 0, or somewhere up to case["context"]."""
    n = _lengths(case)
    off = np.cumsum(n) - n
    total = int(n.sum())
    start = np.random.default_rng(seed).integers(0, case["context"] + 1, n.size)
    order = np.arange(n.size)
    if case["layout"] in ("packed", "permuted"):
        order = order[::-1] if case["layout"] == "permuted" else order
        at = np.cumsum(n[order]) - n[order]
        pos = np.arange(total) - np.repeat(at, n[order])
        ids = pos + np.repeat(off[order], n[order])
        pos = pos + np.repeat(start[order], n[order])
    else:
        pos = np.broadcast_to(np.arange(case["longest"]), (n.size, case["longest"]))
        if case["layout"] == "padded_left":
            pos = pos - (case["longest"] - n)[:, None]
        on = (pos >= 0) & (pos < n[:, None])
        ids = np.where(on, off[:, None] + pos, -1).reshape(-1)
        pos = np.where(on, start[:, None] + pos, 0).reshape(-1)
    return ids.astype(np.int32), pos.astype(np.int32), total


def _inputs(case, seed):
    """Tensors of the call on the GPU: padding slots hold NaN."""
    ids, pos, total = _slots(case, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, D, hq, hk = DTYPES[case["dtype"]], case["head_dim"], case["q_heads"], case["k_heads"]
    param = torch.float32 if case["params"] == "fp32" else dtype
    tok = torch.from_numpy(ids).to("cuda")
    padding = (tok < 0).view(-1, 1, 1) if bool((ids < 0).any()) else None

    def heads(count, scale):
        t = (torch.randn(ids.size, count, D, generator=gen, device="cuda") * scale).to(dtype)
        return t if padding is None else t.masked_fill_(padding, float("nan"))

    op = case["op"]
    s = {"ids": ids, "n_logical": total, "tok": tok, "pos": torch.from_numpy(pos).to("cuda")}
    if op != "rotary_bwd":
        if case["joined"]:                                            # queries, keys and values of a token side by side
            qkv = heads(hq + 2 * hk, 1.5)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = heads(hq, 1.5), heads(hk, 1.5)
    if op.endswith("_bwd"):
        s["dq_out"], s["dk_out"] = heads(hq, 0.01), heads(hk, 0.01)
    if op.startswith("qk"):
        s["q_weight"], s["k_weight"] = ((1 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(param) for _ in "qk")
    return s


def _frequencies(case):
    """Angles per position, in 64 bits: base^(-2i/r), stretched by the factor; with a ramp (the context that the model
    was trained on) pairs that turn more than 32 times over that context keep their speed, below one turn they are
    stretched in full."""
    r = case["rotary_dim"]
    f = case["base"] ** (-np.arange(0, r, 2, dtype=np.float64) / r)
    if case["ramp"]:
        keep = np.clip((case["ramp"] * f / (2 * np.pi) - 1) / (32 - 1), 0, 1)
        return f * keep + f * (1 - keep) / case["factor"]
    return f / case["factor"]


def prepare(case, seed):
    s = _inputs(case, seed)
    D, n = case["head_dim"], s["ids"].size
    like = DTYPES[case["dtype"]]
    new = lambda count: torch.zeros(n, count, D, dtype=like, device="cuda")   # noqa: E731
    names = ("dq", "dk") if case["op"].endswith("_bwd") else ("q", "k")
    # outputs that a program keeps from step to step: padding in them stays as it is
    s["case"], s["out"] = case, {names[0]: new(case["q_heads"]), names[1]: new(case["k_heads"])}
    if case["op"] == "qk_norm_rotary_bwd":
        s["out"].update({w: torch.zeros(D, device="cuda") for w in ("dq_weight", "dk_weight")})
    s["active"] = torch.nonzero(s["tok"] >= 0).reshape(-1)
    s["whole"] = bool((s["ids"] >= 0).all())
    s["freq"] = torch.from_numpy(_frequencies(case)).cuda()
    if own:
        import invariant_rmsnorm_fwd_gb300 as rb
        s["layout"] = rb.call_layout(s["ids"], 1, s["n_logical"], with_plan=False)
        s["rotary"] = rb.Rotary(case["rotary_dim"], interleaved=case["pairs"] == "interleaved", first=case["first"],
                                scale=case["scale"],
                                inv_freq=rb.rotary_frequencies(case["rotary_dim"], case["base"], case["factor"],
                                                               original_length=case["ramp"] or None))
        if case["op"] == "qk_norm_rotary_bwd":
            s["workspace"] = rb.QkNormWorkspace(s["n_logical"], case["q_heads"], case["k_heads"], D)
    return s


def _own(s):
    import invariant_rmsnorm_fwd_gb300 as rb
    op, o, lay, pos, rot = s["case"]["op"], s["out"], s["layout"], s["pos"], s["rotary"]
    if op == "rotary_fwd":
        rb.rotary_fwd(s["q"], s["k"], lay, pos, rot, q_out=o["q"], k_out=o["k"])
    elif op == "rotary_bwd":
        rb.rotary_bwd(s["dq_out"], s["dk_out"], lay, pos, rot, dq=o["dq"], dk=o["dk"])
    elif op == "qk_norm_rotary_fwd":
        rb.qk_norm_rotary_fwd(s["q"], s["k"], s["q_weight"], s["k_weight"], lay, pos, rot, EPS, q_out=o["q"], k_out=o["k"])
    else:
        ws = s["workspace"]
        ws.begin()
        rb.qk_norm_rotary_bwd(s["q"], s["k"], s["q_weight"], s["k_weight"], s["dq_out"], s["dk_out"], lay, pos, rot, EPS,
                              dq=o["dq"], dk=o["dk"], workspace=ws)
        ws.finalize(dq_weight=o["dq_weight"], dk_weight=o["dk_weight"])
    return o


def run(state):
    return _own(state) if own else _plain(state)


def _plain(s):
    case, o, act, whole = s["case"], s["out"], s["active"], s["whole"]
    op, r, first = case["op"], case["rotary_dim"], case["first"]
    pos = s["pos"] if whole else s["pos"][act]
    angle = pos.double()[:, None] * s["freq"]                         # far positions: 64 bits
    cos = (torch.cos(angle).float() * case["scale"])[:, None]
    sin = (torch.sin(angle).float() * case["scale"])[:, None]

    def turn(x, sin):
        out = x.clone()
        part = x[..., first:first + r]
        if case["pairs"] == "half":
            a, b = part[..., :r // 2], part[..., r // 2:]
            out[..., first:first + r // 2] = a * cos - b * sin
            out[..., first + r // 2:first + r] = b * cos + a * sin
        else:
            a, b = part[..., ::2], part[..., 1::2]
            out[..., first:first + r:2] = a * cos - b * sin
            out[..., first + 1:first + r:2] = b * cos + a * sin
        return out

    def rows(t):                                                      # the active tokens, in 32 bits
        return (t if whole else t[act]).float()

    def put(name, v):
        v = v.to(o[name].dtype)
        o[name].copy_(v) if whole else o[name].index_copy_(0, act, v)

    for n in ("q", "k"):
        if op == "rotary_fwd":
            put(n, turn(rows(s[n]), sin))
        elif op == "rotary_bwd":
            put("d" + n, turn(rows(s[f"d{n}_out"]), -sin))
        else:
            x, w = rows(s[n]), s[n + "_weight"].float()
            rstd = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            if op == "qk_norm_rotary_fwd":
                put(n, turn(x * rstd * w, sin))
            else:
                g, xhat = turn(rows(s[f"d{n}_out"]), -sin), x * rstd
                o[f"d{n}_weight"].copy_((g * xhat).sum((0, 1)))
                a = g * w
                put("d" + n, rstd * (a - xhat * (a * xhat).mean(-1, keepdim=True)))
    return o


def work(case):
    tokens = int(_lengths(case).sum())
    slots = tokens if case["layout"] in ("packed", "permuted") else case["samples"] * case["longest"]
    size = 4 if case["dtype"] == "fp32" else 2
    param = 4 if case["params"] == "fp32" else size
    heads, D, r, op = case["q_heads"] + case["k_heads"], case["head_dim"], case["rotary_dim"], case["op"]
    tensors = 3 if op == "qk_norm_rotary_bwd" else 2
    extra = {"qk_norm_rotary_fwd": 2 * D * param, "qk_norm_rotary_bwd": 2 * D * (param + 4)}.get(op, 0)
    each = {"qk_norm_rotary_fwd": 4, "qk_norm_rotary_bwd": 10}.get(op, 0)
    return {"bytes": float(tensors * tokens * heads * D * size + 4 * slots + 4 * tokens + extra),
            "flops": float(tokens * heads * (3 * r + each * D) + tokens * r)}


def exact(case, seed):
    s = _inputs(case, seed)
    r, D, op = case["rotary_dim"], case["head_dim"], case["op"]
    act = torch.from_numpy(s["ids"] >= 0).cuda()
    pos = s["pos"][act].to(torch.float64)
    # each pair is a complex number, turned by scale * e^(i angle)
    i = torch.arange(r // 2, device="cuda")
    a = case["first"] + (i if case["pairs"] == "half" else 2 * i)
    b = a + (r // 2 if case["pairs"] == "half" else 1)
    turn = torch.polar(torch.full((), case["scale"], dtype=torch.float64, device="cuda"),
                       torch.outer(pos, torch.from_numpy(_frequencies(case)).cuda()))[:, None, :]
    turn = turn.conj() if op.endswith("_bwd") else turn

    def rotated(v):
        z = torch.complex(v[:, :, a], v[:, :, b]) * turn
        v = v.clone()
        v[:, :, a], v[:, :, b] = z.real, z.imag
        return v

    def full(v, heads):
        out = torch.zeros(act.numel(), heads, D, dtype=torch.float64, device="cuda")
        out[act] = v
        return out

    out, grads = {}, {}
    for n, heads in (("q", case["q_heads"]), ("k", case["k_heads"])):
        if op == "rotary_fwd":
            out[n] = full(rotated(s[n][act].double()), heads)
            continue
        if op == "rotary_bwd":
            out["d" + n] = full(rotated(s[f"d{n}_out"][act].double()), heads)
            continue
        x, w = s[n][act].double(), s[n + "_weight"].double()
        length = torch.sqrt(torch.einsum("thd,thd->th", x, x) / D + EPS)[..., None]
        unit = x / length
        if op == "qk_norm_rotary_fwd":
            out[n] = full(rotated(unit * w), heads)
        else:
            g = rotated(s[f"d{n}_out"][act].double())
            grads[f"d{n}_weight"] = torch.einsum("thd,thd->d", g, unit)
            along = torch.einsum("thd,thd->th", g * w, unit)[..., None] / D
            out["d" + n] = full((g * w - unit * along) / length, heads)
    return {**out, **grads}
