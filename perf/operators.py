"""What is measured of the operators for long user histories and drafted candidates: rotary positions
with several axes, causal attention with a sliding window and first tokens that stay visible
(training forward and backward, and one new token over a cache), and attention of a tree of drafted
tokens over a cache. Each case says which operator it runs and at which sizes; `run` is one pass,
in elementary torch operations or through the library."""

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------------------
# Cases
# ------------------------------------------------------------------------------------------------

def listed():
    return [
        # The three-user batch of the tests, rotated before a layer: latency.
        dict(name="rope three users", op="rope", dtype="bf16", users=3, median=100, longest=1000, prefix=2,
             lengths_seed=0, pad_to=1, H=4, Hkv=4, d=64, axes=3, per_axis=False),
        # Queries and keys of the 256-user batch, three axes (order, time, session).
        dict(name="rope 256 users", op="rope", dtype="bf16", users=256, median=280, longest=4096, prefix=68,
             lengths_seed=0, pad_to=1, H=8, Hkv=8, d=128, axes=3, per_axis=False),
        # The gradient of the rotation, shared key heads, 32-bit gradients.
        dict(name="rope gradient 64 users fp32", op="rope_bwd", dtype="fp32", users=64, median=280, longest=4096,
             prefix=4, lengths_seed=1, pad_to=1, H=16, Hkv=4, d=64, axes=2, per_axis=True),
        # One layer of the three-user batch, its rows padded to a multiple of 8: latency.
        dict(name="window three users", op="window", users=3, median=100, longest=1000, prefix=2, lengths_seed=0,
             pad_to=8, H=4, Hkv=4, d=64, window=128, sinks=2),
        # The 256-user batch, the four prefix tokens stay visible.
        dict(name="window 256 users", op="window", users=256, median=280, longest=4096, prefix=68, lengths_seed=0,
             pad_to=1, H=8, Hkv=8, d=128, window=256, sinks=4),
        # Few long histories with shared key heads.
        dict(name="window 12 long users", op="window", users=12, median=4096, longest=8192, prefix=16,
             lengths_seed=2, pad_to=1, H=16, Hkv=4, d=64, window=1024, sinks=16),
        # Training on a small padded batch.
        dict(name="window gradient 16 users", op="window_bwd", users=16, median=100, longest=1000, prefix=4,
             lengths_seed=3, pad_to=8, H=4, Hkv=2, d=64, window=128, sinks=4),
        # Training on the 256-user batch.
        dict(name="window gradient 256 users", op="window_bwd", users=256, median=280, longest=4096, prefix=68,
             lengths_seed=0, pad_to=1, H=8, Hkv=8, d=128, window=256, sinks=4),
        # One request, one new token over its cached history: latency.
        dict(name="decode 1 user", op="decode", users=1, longest=4096, lengths_seed=4, H=8, Hkv=8, d=128,
             window=4096, sinks=4),
        # 256 requests in a padded batch, shared key heads, window of the training runs.
        dict(name="decode 256 users", op="decode", users=256, longest=2048, lengths_seed=5, H=16, Hkv=4, d=128,
             window=1024, sinks=4),
        # A few requests with small trees of drafted tokens.
        dict(name="tree 4 users", op="tree", users=4, median=280, longest=1000, prefix=4, lengths_seed=6, H=8,
             Hkv=2, d=64, drafts=17),
        # The 256 histories with 64 drafted tokens each.
        dict(name="tree 256 users", op="tree", users=256, median=280, longest=4096, prefix=4, lengths_seed=0, H=8,
             Hkv=8, d=128, drafts=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "window", "window", "window_bwd", "window_bwd", "decode", "decode", "tree",
                     "tree"])
    d = rng.choice([32, 64, 128, 128])
    Hkv, G = rng.choice([(1, 4), (2, 2), (2, 4), (4, 1), (4, 2), (8, 1)])
    c = dict(op=op, users=_log(rng, 1, 200), lengths_seed=rng.randrange(1 << 20), H=Hkv * G, Hkv=Hkv, d=d)
    if op in ("rope", "rope_bwd"):
        c.update(dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), median=_log(rng, 4, 280),
                 longest=_log(rng, 300, 4096), prefix=rng.randrange(0, 9), pad_to=1, axes=rng.randrange(1, 5),
                 per_axis=rng.random() < 0.5)
    elif op in ("window", "window_bwd"):
        c.update(median=_log(rng, 4, 280), longest=_log(rng, 300, 4096), prefix=rng.randrange(1, 9),
                 pad_to=rng.choice([1, 1, 8]), window=_log(rng, 1, 700), sinks=rng.randrange(0, 17))
    elif op == "decode":
        c.update(longest=_log(rng, 40, 4096), window=_log(rng, 1, 4096), sinks=rng.randrange(0, 17))
    else:
        c.update(median=_log(rng, 20, 280), longest=_log(rng, 300, 2048), prefix=rng.randrange(0, 9),
                 drafts=_log(rng, 1, 64))
    return c


# ------------------------------------------------------------------------------------------------
# Lengths and counts of a case (host, from the case alone)
# ------------------------------------------------------------------------------------------------

def _lengths(c):
    """Rows of each user before padding: prefix plus a lognormal history, one user at the longest
    and, in larger batches, one with none."""
    r = np.random.default_rng(c["lengths_seed"])
    n = np.floor(r.lognormal(math.log(c["median"]), 1.0, c["users"])).astype(np.int64)
    n = np.clip(n, 0, c["longest"])
    if c["users"] > 2:
        n[1] = c["longest"]
    if c["users"] > 3:
        n[0] = 0
    n = n + c["prefix"]
    return np.maximum(n, 1) if int(n.sum()) == 0 else n


def _layout(c):
    """(real rows, rows with padding) of each user."""
    real = _lengths(c)
    m = c["pad_to"]
    return real, (real + m - 1) // m * m


def _cached(c):
    """Tokens in each user's cache and the rows of its region; -1 marks an empty slot of the batch."""
    r = np.random.default_rng(c["lengths_seed"])
    n = r.integers(0, c["longest"], c["users"])
    if c["users"] == 1:
        n[0] = c["longest"] - 1
    cap = n + 1 + r.integers(0, 16, c["users"])
    if c["users"] > 8:
        n[5] = -1
    return n, cap


def _drafts(c):
    r = np.random.default_rng(c["lengths_seed"] + 1)
    n = r.integers(max(1, c["drafts"] // 2), c["drafts"] + 1, c["users"])
    n[-1] = c["drafts"]
    if c["users"] > 8:
        n[3] = 0
    return n


def _sections(c):
    """Rotated pairs of each axis; with two axes or more the last pairs of a head stay unrotated."""
    half, a = c["d"] // 2, c["axes"]
    if a == 1:
        return [half]
    base = max(1, (half - 1) // a)
    return [half - 1 - base * (a - 1)] + [base] * (a - 1)


def _window_pairs(n, w, s):
    """Visible (query, key) pairs of causal rows 0..n-1 with a window of w and s first tokens."""
    total = 0
    for x in np.unique(n):
        p = np.arange(int(x))
        total += int((np.minimum(p + 1, w) + np.minimum(s, np.maximum(0, p + 1 - w))).sum()) * int((n == x).sum())
    return total


def work(c):
    H, Hkv, d, op = c["H"], c["Hkv"], c["d"], c["op"]
    if op in ("rope", "rope_bwd"):
        T = int(_layout(c)[1].sum())
        size = TYPES[c["dtype"]].itemsize
        return {"bytes": 2 * T * (H + Hkv) * d * size + 8 * T * c["axes"], "flops": 3 * T * (H + Hkv) * d}
    if op in ("window", "window_bwd"):
        real, rows = _layout(c)
        T, pairs = int(rows.sum()), _window_pairs(real, c["window"], c["sinks"])
        if op == "window":
            return {"bytes": T * (2 * d * (2 * H + 2 * Hkv) + 4 * H), "flops": 4 * pairs * H * d}
        # q, out, dout, dq; k, v, dk, dv; five products of each pair
        return {"bytes": T * (2 * d * (4 * H + 4 * Hkv) + 4 * H), "flops": 10 * pairs * H * d}
    if op == "decode":
        n, _ = _cached(c)
        p = n[n >= 0]
        seen = int((np.minimum(p + 1, c["window"]) + np.minimum(c["sinks"], np.maximum(0, p + 1 - c["window"]))).sum())
        B = c["users"]
        return {"bytes": 2 * d * (2 * seen * Hkv + 2 * B * H + 2 * len(p) * Hkv), "flops": 4 * seen * H * d}
    h, n = _lengths(c), _drafts(c)
    N = int(n.sum())
    used = int(h[n > 0].sum())
    return {"bytes": 2 * d * (2 * used * Hkv + N * (2 * H + 2 * Hkv)), "flops": 4 * H * d * int((h * n + n).sum())}


# ------------------------------------------------------------------------------------------------
# Inputs
# ------------------------------------------------------------------------------------------------

def _normal(g, shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32).to(dtype)


def _offsets(n):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int64)).to(DEV)


def prepare(c, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    H, Hkv, d, op = c["H"], c["Hkv"], c["d"], c["op"]
    s = {"case": c, "scale": 1.0 / math.sqrt(d)}
    if op in ("rope", "rope_bwd"):
        n = _layout(c)[1]
        T, t = int(n.sum()), TYPES[c["dtype"]]
        s["q"], s["k"] = _normal(g, (T, H, d), t), _normal(g, (T, Hkv, d), t)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        # order in the row, minutes of the event, and small counters (session, place in it)
        order = torch.cat([torch.arange(int(x), device=DEV) for x in n])
        other = [torch.randint(0, hi, (T,), generator=g, device=DEV) for hi in (525600, 512, 64)]
        s["positions"] = torch.stack(([order] + other)[: c["axes"]], 1).to(torch.int64).contiguous()
        s["sections"] = _sections(c)
    elif op in ("window", "window_bwd"):
        real, rows = _layout(c)
        T = int(rows.sum())
        s["q"], s["k"], s["v"] = _normal(g, (T, H, d)), _normal(g, (T, Hkv, d)), _normal(g, (T, Hkv, d))
        s["offsets"] = _offsets(rows)
        s["valid"] = None
        if c["pad_to"] > 1:
            start, end = s["offsets"][:-1], torch.from_numpy(real).to(DEV)
            user = torch.searchsorted(s["offsets"], torch.arange(T, device=DEV), right=True) - 1
            s["valid"] = (torch.arange(T, device=DEV) - start[user] < end[user]).to(torch.uint8)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(T, H, device=DEV)
        if op == "window_bwd":
            o, s["lse"] = _plain_window(s)
            s["out"] = o
            s["dout"] = _normal(g, (T, H, d))
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
    elif op == "decode":
        n, cap = _cached(c)
        R = int(cap.sum())
        s["q"] = _normal(g, (c["users"], H, d))
        s["k_new"], s["v_new"] = _normal(g, (c["users"], Hkv, d)), _normal(g, (c["users"], Hkv, d))
        s["k_cache"], s["v_cache"] = _normal(g, (R, Hkv, d)), _normal(g, (R, Hkv, d))
        s["offsets"], s["cached"] = _offsets(cap), torch.from_numpy(n).to(DEV)
        s["out"] = torch.empty_like(s["q"])
    else:
        h, n = _lengths(c), _drafts(c)
        N, R = int(n.sum()), int(h.sum())
        s["q"], s["k"], s["v"] = _normal(g, (N, H, d)), _normal(g, (N, Hkv, d)), _normal(g, (N, Hkv, d))
        s["k_cache"], s["v_cache"] = _normal(g, (R, Hkv, d)), _normal(g, (R, Hkv, d))
        s["offsets"], s["hist_offsets"] = _offsets(n), _offsets(h)
        # each token hangs on the history or on one of the last few before it
        i = torch.cat([torch.arange(int(x), device=DEV) for x in n])
        back = torch.randint(0, 6, (N,), generator=g, device=DEV)
        s["parent"] = torch.clamp(i - 1 - back, min=-1).to(torch.int32)
        s["slot"] = torch.cat([u * c["drafts"] + torch.arange(int(x), device=DEV) for u, x in enumerate(n)])
        s["out"] = torch.empty_like(s["q"])
    return s


# ------------------------------------------------------------------------------------------------
# Plain forms
# ------------------------------------------------------------------------------------------------

def _angles(s):
    """Angle of each row and pair, in 64 bits; pairs past the sections keep angle 0."""
    c, half = s["case"], s["case"]["d"] // 2
    axis = np.repeat(np.arange(len(s["sections"])), s["sections"])
    if c["per_axis"]:
        freq = np.concatenate([10000.0 ** (-np.arange(m) / m) for m in s["sections"]])
    else:
        freq = 10000.0 ** (-np.arange(len(axis)) / half)
    freq = torch.from_numpy(freq).to(DEV)
    turned = s["positions"][:, torch.from_numpy(axis).to(DEV)].double() * freq
    return torch.nn.functional.pad(turned, (0, half - len(axis)))


def _plain_rope(s, sign):
    a = _angles(s)
    cos, sin = torch.cos(a).float()[:, None], (sign * torch.sin(a)).float()[:, None]

    def turn(x):
        lo, hi = x.float().chunk(2, -1)
        return torch.cat([lo * cos - hi * sin, lo * sin + hi * cos], -1).to(x.dtype)

    return turn(s["q"]), turn(s["k"])


class _Band:
    """Keys of a packed batch laid out for blocks of queries: each block of C rows sees its own
    block and the one before it (C >= window), and the first tokens of its users."""

    def __init__(self, s):
        c = s["case"]
        self.T, self.Hkv, self.S = s["q"].shape[0], s["k"].shape[1], max(1, c["sinks"])
        self.G = s["q"].shape[1] // self.Hkv
        self.C = C = min(max(c["window"], 16), self.T)
        self.nb = -(-self.T // C)
        row = torch.arange(self.T, device=DEV)
        user = torch.searchsorted(s["offsets"], row, right=True) - 1
        start = s["offsets"][user]
        lo = torch.maximum(start, row - c["window"] + 1)
        real = torch.ones(self.T, dtype=torch.bool, device=DEV) if s["valid"] is None else s["valid"].bool()
        self.real = real
        j = (torch.arange(self.nb, device=DEV)[:, None] - 1) * C + torch.arange(2 * C, device=DEV)
        i = torch.arange(self.nb * C, device=DEV).view(self.nb, C)
        in_batch = (j >= 0) & (j < self.T)
        key = (in_batch & real[j.clamp(0, self.T - 1)])[:, None, :]
        lo_i = torch.nn.functional.pad(lo, (0, self.nb * C - self.T)).view(self.nb, C)
        self.band = key & (j[:, None, :] >= lo_i[:, :, None]) & (j[:, None, :] <= i[:, :, None])
        first = start[:, None] + torch.arange(self.S, device=DEV)
        self.first = first.clamp(max=self.T - 1)
        self.seen = (first < lo[:, None]) & (first < start[:, None] + c["sinks"]) & real[self.first]

    def queries(self, x):  # [T, H, d] -> [nb, Hkv, G, C, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, self.nb * self.C - self.T))
        return x.view(self.nb, self.C, self.Hkv, self.G, -1).permute(0, 2, 3, 1, 4)

    def rows(self, x):  # and back
        return x.permute(0, 3, 1, 2, 4).reshape(self.nb * self.C, self.Hkv * self.G, -1)[: self.T]

    def keys(self, x):  # [T, Hkv, d] -> [nb, Hkv, 1, 2C, d]
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, self.C, self.nb * self.C - self.T))
        x = x.view(self.nb + 1, self.C, self.Hkv, -1)
        return torch.cat([x[:-1], x[1:]], 1).permute(0, 2, 1, 3)[:, :, None]

    def key_rows(self, x):  # [nb, Hkv, 2C, d] -> [T, Hkv, d], the two blocks of a key added
        a, b = x.permute(0, 2, 1, 3).split(self.C, 1)
        b = b + torch.cat([a[1:], torch.zeros_like(a[:1])])
        return b.reshape(self.nb * self.C, self.Hkv, -1)[: self.T]

    def first_keys(self, x):  # [T, Hkv, d] -> [T, Hkv, S, d]
        return x.float()[self.first].permute(0, 2, 1, 3)

    def scores(self, s):
        q = s["q"].float() * s["scale"]
        band = torch.matmul(self.queries(q), self.keys(s["k"]).transpose(-1, -2))
        band = band.masked_fill(~self.band[:, None, None], -math.inf)
        first = torch.matmul(q.view(self.T, self.Hkv, self.G, -1), self.first_keys(s["k"]).transpose(-1, -2))
        return band, first.masked_fill(~self.seen[:, None, None], -math.inf)


def _plain_window(s):
    b = _Band(s)
    band, first = b.scores(s)
    top = torch.maximum(b.rows(band.amax(-1, keepdim=True)), first.reshape(b.T, -1, b.S).amax(-1, keepdim=True))
    base = torch.where(torch.isfinite(top), top, 0.0)
    band = torch.exp(band - b.queries(base))
    first = torch.exp(first - base.view(b.T, b.Hkv, b.G, 1))
    total = b.rows(band.sum(-1, keepdim=True)) + first.reshape(b.T, -1, b.S).sum(-1, keepdim=True)
    out = b.rows(torch.matmul(band, b.keys(s["v"])))
    out = out + torch.matmul(first, b.first_keys(s["v"])).reshape(out.shape)
    live = b.real[:, None, None] & (total > 0)
    out = torch.where(live, out / total, 0.0)
    lse = torch.where(live, base + torch.log(total), -math.inf)
    return out.to(torch.bfloat16), lse[..., 0].contiguous()


def _plain_window_bwd(s):
    b = _Band(s)
    band, first = b.scores(s)
    real = b.real[:, None, None]
    lse = torch.where(torch.isfinite(s["lse"]), s["lse"], math.inf)[..., None]
    dout = torch.where(real, s["dout"].float(), 0.0)
    delta = (dout * s["out"].float()).sum(-1, keepdim=True)
    grouped = (b.T, b.Hkv, b.G, -1)
    p, p1 = torch.exp(band - b.queries(lse)), torch.exp(first - lse.view(grouped))
    do, do1 = b.queries(dout), dout.view(grouped)
    ds = p * (torch.matmul(do, b.keys(s["v"]).transpose(-1, -2)) - b.queries(delta))
    ds1 = p1 * (torch.matmul(do1, b.first_keys(s["v"]).transpose(-1, -2)) - delta.view(grouped))
    q = s["q"].float() * s["scale"]
    qb, q1 = b.queries(q), q.view(grouped)
    dq = b.rows(torch.matmul(ds, b.keys(s["k"])))
    dq = (dq + torch.matmul(ds1, b.first_keys(s["k"])).reshape(dq.shape)) * s["scale"]
    dk = b.key_rows(torch.matmul(ds.transpose(-1, -2), qb).sum(2))
    dv = b.key_rows(torch.matmul(p.transpose(-1, -2), do).sum(2))
    at = b.first.reshape(-1)
    for grad, w, x in ((dk, ds1, q1), (dv, p1, do1)):
        grad.index_add_(0, at, torch.matmul(w.transpose(-1, -2), x).transpose(1, 2).reshape(len(at), b.Hkv, -1))
    return dq.to(torch.bfloat16), dk.to(torch.bfloat16), dv.to(torch.bfloat16)


def _plain_cached(q, k, v, seen, scale):
    """Softmax of q [B, n, H, d] over k, v [B, m, Hkv, d] where seen [B, n, m]."""
    B, n, H, d = q.shape
    Hkv = k.shape[2]
    q = (q.float() * scale).view(B, n, Hkv, H // Hkv, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q, k.float().permute(0, 2, 3, 1)[:, :, None])
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(torch.isfinite(top), top, 0.0))
    total = x.sum(-1, keepdim=True)
    out = torch.matmul(x, v.float().masked_fill(~seen.any(1)[..., None, None], 0.0).permute(0, 2, 1, 3)[:, :, None])
    out = torch.where(total > 0, out / total, 0.0)
    return out.permute(0, 3, 1, 2, 4).reshape(B, n, H, d).to(torch.bfloat16)


def _plain_decode(s):
    c, p = s["case"], s["cached"]
    live = p >= 0
    at = s["offsets"][:-1] + p.clamp(min=0)
    for cache, new in ((s["k_cache"], s["k_new"]), (s["v_cache"], s["v_new"])):
        cache[at] = torch.where(live[:, None, None], new, cache[at])
    w = min(c["window"], c["longest"])
    near = p[:, None] - w + 1 + torch.arange(w, device=DEV)
    first = torch.arange(c["sinks"], device=DEV).expand(len(p), -1)
    seen = torch.cat([near >= 0, first < (p[:, None] - w + 1)], 1) & live[:, None]
    at = torch.where(seen, s["offsets"][:-1, None] + torch.cat([near, first], 1), 0)
    out = _plain_cached(s["q"][:, None], s["k_cache"][at], s["v_cache"][at], seen[:, None], s["scale"])
    return out[:, 0], s["k_cache"], s["v_cache"]


def _ancestors(parent):
    """[B, n, n]: which tokens a token descends from, itself included; parent -1 is the history."""
    n = parent.shape[1]
    reach = torch.eye(n, device=DEV) + torch.nn.functional.one_hot(parent.long() + 1, n + 1)[..., 1:].float()
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length each time
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0


def _plain_tree(s):
    c, off, hist = s["case"], s["offsets"], s["hist_offsets"]
    n, m = c["drafts"], int(_lengths(c).max())
    i, j = torch.arange(n, device=DEV), torch.arange(m, device=DEV)
    count, cached = off[1:] - off[:-1], hist[1:] - hist[:-1]
    draft, old = i < count[:, None], j < cached[:, None]
    at = torch.where(draft, off[:-1, None] + i, 0)
    then = torch.where(old, hist[:-1, None] + j, 0)
    tree = _ancestors(torch.where(draft, s["parent"][at], -1)) & draft[:, None]
    seen = torch.cat([old[:, None].expand(-1, n, -1), tree], 2)
    k = torch.cat([s["k_cache"][then], s["k"][at]], 1)
    v = torch.cat([s["v_cache"][then], s["v"][at]], 1)
    return _plain_cached(s["q"][at], k, v, seen, s["scale"]).flatten(0, 1)[s["slot"]]


# ------------------------------------------------------------------------------------------------
# One pass
# ------------------------------------------------------------------------------------------------

def _own(s):
    from candidate_isolated_jagged_b200 import jca
    c, op = s["case"], s["case"]["op"]
    if "status" not in s:
        s["status"] = jca.new_status(DEV)
    if op == "rope":
        jca.jca_rope_axes_fwd(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["sections"],
                              per_axis=c["per_axis"])
        return s["q_out"], s["k_out"]
    if op == "rope_bwd":
        jca.jca_rope_axes_bwd(s["q"], s["k"], s["q_out"], s["k_out"], s["positions"], s["sections"],
                              per_axis=c["per_axis"])
        return s["q_out"], s["k_out"]
    if op in ("window", "window_bwd") and "workspace" not in s:
        size = jca.jca_window_workspace_bytes if op == "window" else jca.jca_window_bwd_workspace_bytes
        n = size(c["users"], s["q"].shape[0], c["H"], c["Hkv"], c["d"], c["sinks"])
        s["workspace"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    if op == "window":
        jca.jagged_window_attn_fwd(s["q"], s["k"], s["v"], s["out"], s["offsets"], c["window"], c["sinks"],
                                   valid=s["valid"], lse=s["lse"], workspace=s["workspace"], status=s["status"])
        return s["out"], s["lse"]
    if op == "window_bwd":
        jca.jagged_window_attn_bwd(s["q"], s["k"], s["v"], s["out"], s["dout"], s["lse"], s["dq"], s["dk"], s["dv"],
                                   s["offsets"], c["window"], c["sinks"], valid=s["valid"],
                                   workspace=s["workspace"], status=s["status"])
        return s["dq"], s["dk"], s["dv"]
    if op == "decode":
        jca.jagged_window_decode_fwd(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["out"],
                                     s["offsets"], s["cached"], c["window"], c["sinks"], status=s["status"])
        return s["out"], s["k_cache"], s["v_cache"]
    jca.cand_tree_attn_fwd(s["q"], s["k"], s["v"], s["offsets"], s["parent"], s["k_cache"], s["v_cache"],
                           s["hist_offsets"], s["out"], max_cand=c["drafts"], status=s["status"])
    return s["out"]


def run(s):
    if own:
        return _own(s)
    return {"rope": lambda s: _plain_rope(s, 1.0), "rope_bwd": lambda s: _plain_rope(s, -1.0),
            "window": _plain_window, "window_bwd": _plain_window_bwd, "decode": _plain_decode,
            "tree": _plain_tree}[s["case"]["op"]](s)


# ------------------------------------------------------------------------------------------------
# The definitions in 64 bits, user by user
# ------------------------------------------------------------------------------------------------

def _exact_softmax(q, k, v, seen, scale):
    """q [n, H, d], k, v [m, Hkv, d], seen [n, m] -> (probabilities [H, n, m], out [n, H, d], lse [n, H])."""
    g = q.shape[1] // k.shape[1]
    kk, vv = k.double().repeat_interleave(g, 1), v.double().repeat_interleave(g, 1)
    x = torch.einsum("nhd,mhd->hnm", q.double(), kk) * scale
    x.masked_fill_(~seen, -math.inf)
    lse = torch.logsumexp(x, -1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0))
    return p, torch.einsum("hnm,mhd->nhd", p, vv), lse[..., 0].t()


def _exact_users(c, s):
    """(first row, last row, mask of what each row sees) of each user of a windowed batch."""
    off = s["offsets"].tolist()
    for a, b in zip(off, off[1:]):
        if a == b:
            continue
        i = torch.arange(b - a, device=DEV)
        seen = (i[None] <= i[:, None]) & ((i[None] > i[:, None] - c["window"]) | (i[None] < c["sinks"]))
        if s["valid"] is not None:
            real = s["valid"][a:b].bool()
            seen &= real[None] & real[:, None]
        yield a, b, seen


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op in ("rope", "rope_bwd"):
        sign = 1.0 if op == "rope" else -1.0
        half = c["d"] // 2
        got = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            j = 0
            for axis, m in enumerate(s["sections"]):
                for t in range(m):
                    angle = s["positions"][:, axis].double() * 10000.0 ** (-(t / m if c["per_axis"] else j / half))
                    z = torch.polar(torch.ones_like(angle), sign * angle)[:, None]
                    z = torch.complex(x[..., j].double(), x[..., j + half].double()) * z
                    y[..., j], y[..., j + half] = z.real, z.imag
                    j += 1
            got.append(y)
        return got
    if op == "window":
        out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
        lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=DEV)
        for a, b, seen in _exact_users(c, s):
            _, out[a:b], lse[a:b] = _exact_softmax(s["q"][a:b], s["k"][a:b], s["v"][a:b], seen, s["scale"])
        return out, lse
    if op == "window_bwd":
        dq, dk, dv = (torch.zeros(s[x].shape, dtype=torch.float64, device=DEV) for x in "qkv")
        g = c["H"] // c["Hkv"]
        for a, b, seen in _exact_users(c, s):
            q, k, v = s["q"][a:b], s["k"][a:b], s["v"][a:b]
            p, o, _ = _exact_softmax(q, k, v, seen, s["scale"])
            do = s["dout"][a:b].double()
            do = do * seen.any(1)[:, None, None]
            ds = torch.einsum("nhd,mhd->hnm", do, v.double().repeat_interleave(g, 1))
            ds.sub_((do * o).sum(-1).t()[..., None]).mul_(p).mul_(s["scale"])
            dq[a:b] = torch.einsum("hnm,mhd->nhd", ds, k.double().repeat_interleave(g, 1))
            shared = (b - a, c["Hkv"], g, c["d"])
            dk[a:b] = torch.einsum("hnm,nhd->mhd", ds, q.double()).view(shared).sum(2)
            dv[a:b] = torch.einsum("hnm,nhd->mhd", p, do).view(shared).sum(2)
        return dq, dk, dv
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    off = s["offsets"].tolist()
    if op == "decode":
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        for u, p in enumerate(s["cached"].tolist()):
            if p < 0:
                continue
            kc[off[u] + p], vc[off[u] + p] = s["k_new"][u].double(), s["v_new"][u].double()
            at = [off[u] + j for j in range(p + 1) if j > p - c["window"] or j < c["sinks"]]
            at = torch.tensor(at, device=DEV)
            seen = torch.ones(1, len(at), dtype=torch.bool, device=DEV)
            out[u] = _exact_softmax(s["q"][u: u + 1], kc[at], vc[at], seen, s["scale"])[1][0]
        return out, kc, vc
    hist, parent = s["hist_offsets"].tolist(), s["parent"].tolist()
    for u, (a, b) in enumerate(zip(off, off[1:])):
        if a == b:
            continue
        h0, h1 = hist[u], hist[u + 1]
        seen = np.zeros((b - a, h1 - h0 + b - a), dtype=bool)
        seen[:, : h1 - h0] = True
        for i in range(b - a):
            j = i
            while j >= 0:
                seen[i, h1 - h0 + j] = True
                j = parent[a + j]
        k, v = (torch.cat([s[x + "_cache"][h0:h1], s[x][a:b]]) for x in "kv")
        out[a:b] = _exact_softmax(s["q"][a:b], k, v, torch.from_numpy(seen).to(DEV), s["scale"])[1]
    return out
