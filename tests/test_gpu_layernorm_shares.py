"""GPU: layer-norm calls that give a CTA many rows.

With few rows every CTA has one group; the fold of a block's groups, its cut at a share's
end, the second list of a CTA (more than 256 rows) and a team's further groups only come
with more rows than the resident CTAs take at once.  The sizes are counted from the launch
rules: 16 warps an SM on 152 SMs in the streaming backward pass (20 at 257 to 320 threads),
24 in the team kernel (16 above 256 columns).

Rows of +-2^k (mean 0, variance 4^k, eps 0) have exact xhat = +-1, so the gradients' terms
are exact; dy spans 2^-9 .. 2^15, so nearly every order of additions gives another sum, and
the replay of the documented order has to be met bit for bit.
"""
import numpy as np
import pytest
import torch

from oracle import layernorm as O
import invariant_rmsnorm_fwd_gb300 as rb

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

BF, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


def _same(a, b):
    word = torch.int32 if a.element_size() == 4 else torch.int16
    return torch.equal(a.contiguous().view(word), b.contiguous().view(word))


def _state():
    return torch.tensor([77, 5], dtype=torch.int64, device="cuda")


def _exact_terms(n, H, dtype):
    """(x, dy, sign of xhat) with exact statistics, on the GPU."""
    g = torch.Generator("cuda").manual_seed(n + H)
    rnd = lambda *s: torch.rand(*s, generator=g, device="cuda")              # noqa: E731
    sign = torch.where(torch.arange(H, device="cuda") % 2 == 0, 1.0, -1.0) * torch.where(rnd(n, 1) < 0.5, 1.0, -1.0)
    x = sign * 2.0 ** torch.randint(-3, 4, (n, 1), generator=g, device="cuda")
    e = torch.where(rnd(n, H) < 0.5, 0, torch.randint(0, 25, (n, H), generator=g, device="cuda"))
    dy = torch.where(rnd(n, H) < 0.5, 1.0, -1.0) * 2.0 ** (e - 9)
    return x.to(dtype), dy.to(dtype), sign


# hidden, type, rows: groups a CTA (streaming) or a team
SHARES = [(520, BF, 30011),         # 1216 CTAs: 3 groups
          (1040, BF, 49003),        # 760: 8
          (2048, FP16, 29301),      # 608: 6
          (5120, FP16, 10001),      # 304: 4
          (5128, BF, 41005),        # 152: 34, more than one list
          (8192, F32, 6101),        # 152: 5
          (8200, BF, 6101),         # 152: 5
          (16384, BF, 3205),        # 152: 2 or 3
          (24, BF, 520003),         # 29184 teams: 2 or 3
          (128, FP16, 150011),      # 7296 teams: 2 or 3
          (256, F32, 70001),        # 3648 teams: 2 or 3
          (512, BF, 50021)]         # 2432 teams: 2 or 3


@pytest.mark.parametrize("H,dtype,n", SHARES, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("chain", [False, True])
def test_gradients_of_large_shares_keep_the_documented_order(H, dtype, n, chain):
    x, dy, sign = _exact_terms(n, H, dtype)
    cols = torch.unique(torch.cat([torch.arange(0, H, max(1, H // 40)), torch.tensor([1, 7, 8 % H, H // 2, H - 8, H - 1])]))
    dy_cols, sign_cols = (t[:, cols.cuda()].double().cpu().numpy() for t in (dy, sign))
    want = O.grad_replay(dy_cols, sign_cols), O.grad_replay(dy_cols)
    drop = rb.Dropout(0.25, _state()) if chain else None
    half = n // 2 + 13
    layouts = {"full": [np.arange(n)],
               "backwards": [np.arange(n)[::-1]],
               "two calls": [np.arange(half, n), np.arange(half)],
               "three calls": [np.arange(37), np.arange(37, n - 100), np.arange(n - 100, n)],
               "padded": [np.insert(np.arange(n), np.arange(0, n, 501), -1)]}
    first = None
    for name, calls in layouts.items():
        ws = rb.LayerNormWorkspace(n, H)
        ws.begin()
        for ids in calls:
            cl = rb.call_layout(ids.astype(np.int32), 1, n)
            at = cl.tok_id.long().clamp(min=0)
            if len(calls) == 1 and name == "full":
                xs, ds = x, dy
            else:
                xs, ds = x[at], dy[at]
                xs[cl.tok_id < 0] = float("nan")
            if chain:
                rb.layernorm_add_bwd(xs, None, ds, cl, 0.0, dres=ds, dropout=drop, workspace=ws)
            else:
                rb.layernorm_bwd(xs, None, ds, cl, 0.0, workspace=ws, write_dx=H % 16 == 0)
        got = ws.finalize()
        assert ws.status() == 0, name
        for g, v, what in zip(got, want, ("dweight", "dbias")):
            assert np.array_equal(g[cols.cuda()].cpu().numpy(), v), (name, what)
        if first is None:
            first = got
        assert all(_same(u, v) for u, v in zip(first, got)), name
        del ws, xs, ds


# rows of a CTA (streaming) or groups of a team beyond the first ones
ROWS = [(5128, BF, 42003), (5128, F32, 42003), (1040, FP16, 60007), (512, BF, 50021), (128, F32, 150011), (24, FP16, 520003)]


@pytest.mark.parametrize("H,dtype,n", ROWS, ids=lambda v: str(v).replace("torch.", ""))
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_rows_of_large_calls_are_those_of_small_ones(H, dtype, n, p):
    """Every output row of a large, padded call, bit for bit, next to calls of 150 slots."""
    g = torch.Generator("cuda").manual_seed(n + H)
    ids = np.insert(np.arange(n), np.arange(0, n, 97), -1)
    ids = np.concatenate([ids[:n // 3], np.full(700, -1), ids[n // 3:]]).astype(np.int32)   # a long run of padding too
    T = ids.size
    rnd = lambda s: (torch.randn(T, H, generator=g, device="cuda") * s).to(dtype)           # noqa: E731
    x, res, dy, dres = rnd(1.0), rnd(1.0), rnd(0.01), rnd(0.01)
    w, b = (torch.randn(H, generator=g, device="cuda").to(dtype) for _ in range(2))
    drop = rb.Dropout(p, _state()) if p else None

    def run(lo, hi, plan):
        cl = rb.call_layout(ids[lo:hi], 1, n, with_plan=plan)
        v = [t[lo:hi] for t in (x, res, dy, dres)]
        stat = lambda: torch.full((hi - lo,), 7.0, device="cuda")                            # noqa: E731
        out = {k: torch.full((hi - lo, H), 7.0, dtype=dtype, device="cuda") for k in ("h", "y", "y2", "dh", "dx", "dx2", "z")}
        out.update({k: stat() for k in ("mean", "rstd", "mean2", "rstd2")})
        rb.layernorm_fwd(v[0], w, b, cl, 1e-5, y=out["y2"], mean=out["mean2"], rstd=out["rstd2"])
        rb.layernorm_add_fwd(v[0], v[1], w, b, cl, 1e-5, h=out["h"], y=out["y"], mean=out["mean"], rstd=out["rstd"], dropout=drop)
        ws = rb.LayerNormWorkspace(n, H) if plan else None
        if plan:
            ws.begin()
        rb.layernorm_add_bwd(out["h"], w, v[2], cl, 1e-5, dres=v[3], dropout=drop, dh=out["dh"], dx=out["dx"] if p else None,
                             workspace=ws)
        rb.layernorm_bwd(v[0], w, v[2], cl, 1e-5, dx=out["dx2"])
        if p:
            rb.dropout_fwd(v[0], cl, drop, y=out["z"])
        assert ws is None or ws.status() == 0
        return out

    large = run(0, T, True)
    again = run(0, T, False)                             # the backward passes without gradients: the same rows
    pad = torch.from_numpy(ids < 0).cuda()
    for k in large:
        assert _same(large[k], again[k]), k
        assert bool((large[k][pad] == 7).all()), k
        if not (p == 0 and k in ("dx", "z")):
            assert bool(torch.isfinite(large[k]).all()) and not bool((large[k] == 7).reshape(T, -1).all(1)[~pad].any()), k
    for lo in (0, 149, T // 3, T // 2 + 1, T - 1000, T - 150):
        small = run(lo, lo + 150, False)
        for k in small:
            assert _same(small[k], large[k][lo:lo + 150]), (k, lo)
