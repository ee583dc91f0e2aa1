"""Work of a paged K/V cache with grouped heads: the rotary write that fills it and the attention that reads it.

A speculative step checks drafts on the latent cache; the model that drafts keeps keys and values per group of heads, over the
same block tables and slot maps.  Four calls, each a form of its own:

* ``rotary``: rotary positions of one or several axes (time, height, width) on the rotated part of queries and keys, into the
  places of a wider row (the latent form: 64 of 576);
* ``write``: the same on grouped heads, the rotated keys and the values written to the cache rows that a slot map names;
* ``grouped``: attention of one or a few new tokens per request over that cache, a run of query heads to each key head;
* ``differential``: the difference of two softmax maps over shared values, with a learned weight and a norm per head.

With ``own`` false ``run`` computes them in elementary torch operations, otherwise through the package's calls.
Request lengths follow from the case alone; values, block ids, positions and queries from the seed.
"""
import math

import numpy as np
import torch

own = False

LATENT, ROPE = 512, 64  # the latent cache's row: 512 values that are not rotated, then 64 that are
EPS = 1e-5


# ------------------------------------------------------------------ cases

def listed():
    return [
        # two short requests, one drafted token each: the smallest attention call (latency)
        dict(name="grouped_draft_b2", op="grouped", B=2, lo=256, hi=256, qmin=1, qmax=1, H=16, Hkv=4, D=128, bs=16, window=0,
             joint=False, lens=1),
        # the drafting step of a batch, as ordinary decode
        dict(name="grouped_decode_b32", op="grouped", B=32, lo=1024, hi=8192, qmin=1, qmax=1, H=32, Hkv=8, D=128, bs=16,
             window=0, joint=False, lens=2),
        # ragged lengths and rows, three heads to a group, narrow heads, keys and values in one pool
        dict(name="grouped_ragged_b64", op="grouped", B=64, lo=512, hi=32768, qmin=1, qmax=3, H=12, Hkv=4, D=64, bs=64,
             window=0, joint=True, lens=3),
        # long contexts, sixteen heads to a group, four verify rows: 64 query rows to a key head
        dict(name="grouped_verify_b4", op="grouped", B=4, lo=131072, hi=131072, qmin=4, qmax=4, H=64, Hkv=4, D=128, bs=64,
             window=0, joint=False, lens=4),
        # a layer of a sliding window, wide heads, two rows a request
        dict(name="grouped_window_b48", op="grouped", B=48, lo=2048, hi=16384, qmin=2, qmax=2, H=16, Hkv=2, D=256, bs=256,
             window=1024, joint=True, lens=5),
        # a few short requests (latency)
        dict(name="differential_b3", op="differential", B=3, lo=100, hi=900, qmin=1, qmax=1, H=8, Hkv=4, D=64, bs=16, window=0,
             norm=True, lens=6),
        # decode of a batch, two maps of 64 over values of 128
        dict(name="differential_b40", op="differential", B=40, lo=1024, hi=8192, qmin=1, qmax=1, H=16, Hkv=8, D=64, bs=32,
             window=0, norm=True, lens=7),
        # verify rows over longer contexts, two maps of 128 over values of 256, the difference without its norm
        dict(name="differential_verify_b6", op="differential", B=6, lo=16384, hi=40000, qmin=4, qmax=4, H=12, Hkv=4, D=128,
             bs=64, window=0, norm=False, lens=8),
        # a verify step's queries and keys of the latent form
        dict(name="rotary_latent_t128", op="rotary", T=128, H=16, R=64, axes=1, split="sections", neighbours=True, far=131072),
        # a prompt chunk of the latent form, positions far out
        dict(name="rotary_latent_t9001", op="rotary", T=9001, H=64, R=64, axes=1, split="sections", neighbours=True,
             far=1000000),
        # a decode step of a batch on one of two shards: half of the rows are not this shard's
        dict(name="write_step_b250", op="write", B=250, lo=512, hi=4096, qmin=1, qmax=4, H=32, Hkv=8, D=128, Dv=128, R=128,
             axes=3, split="sections", neighbours=False, bs=16, W=2, rank=1, far=4096, lens=9),
        # a prompt of images and text: positions of three axes
        dict(name="write_image_b3", op="write", B=3, lo=5000, hi=6000, qmin=0, qmax=0, H=32, Hkv=8, D=128, Dv=128, R=128,
             axes=3, split="cycle", neighbours=False, bs=64, W=1, rank=0, far=8192, lens=10),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "differential", "rotary", "write"])
    bs = rng.choice([8, 16, 32, 64, 96, 128, 256])
    lens = rng.randrange(1000, 1 << 20)
    far = _log_int(rng, 64, 1 << 20)
    axes = rng.choice([1, 2, 3])
    how = dict(axes=axes, split=rng.choice(["sections", "cycle"]), neighbours=rng.random() < 0.5, far=far)
    if op == "rotary":
        H, R = rng.choice([1, 7, 12, 16, 64, 128]), rng.choice([32, 64, 64, 96, 128])
        return dict(op=op, T=_log_int(rng, 1, 9000 * 64 * 64 // (H * R) // 2), H=H, R=R, **how)
    qmin, qmax = rng.choice([(1, 1), (1, 1), (4, 4), (1, 3), (1, 8)])
    if op == "write":
        if rng.random() < 0.4:
            qmin = qmax = 0
        Hkv = rng.choice([1, 2, 3, 4, 8])
        H = Hkv * rng.choice([1, 2, 4, 5, 8])
        D = rng.choice([64, 80, 128, 256])
        rows = 14000 * 24576 // ((2 * H + 4 * Hkv) * D * 2)
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 32, min(16384, rows // B if qmax == 0 else 400_000 // B))
        W = rng.choice([1, 1, 2, 5])
        return dict(op=op, B=B, lo=max(8, hi // rng.choice([1, 4])), hi=hi, qmin=qmin, qmax=qmax, H=H, Hkv=Hkv, D=D,
                    Dv=rng.choice([D, D, 64]), R=rng.choice([D, D, D // 2]), bs=bs, W=W, rank=rng.randrange(W), lens=lens,
                    **how)
    D = rng.choice([64, 128, 128, 256] if op == "grouped" else [64, 128])
    wide = D if op == "grouped" else 2 * D
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    B = _log_int(rng, 1, 256)
    hi = _log_int(rng, 64, min(131072, 200_000_000 // (B * Hkv * wide), 130_000_000 // (B * H * qmax)))
    c = dict(op=op, B=B, lo=max(8, hi // rng.choice([1, 4, 16])), hi=hi, qmin=qmin, qmax=qmax, H=H, Hkv=Hkv, D=D, bs=bs,
             window=rng.choice([0, 0, 0, _log_int(rng, 16, 4096)]), lens=lens)
    return dict(c, joint=rng.random() < 0.5) if op == "grouped" else dict(c, norm=rng.random() < 0.6)


# ------------------------------------------------------------------ lengths (from the case alone)

def _lengths(c):
    """(length, new tokens) per request."""
    r = np.random.default_rng(c["lens"])
    B = c["B"]
    span = np.exp(r.uniform(math.log(c["lo"]), math.log(c["hi"] + 1), B)) if c["hi"] > 4 * c["lo"] and c["hi"] > 8192 \
        else r.integers(c["lo"], c["hi"] + 1, B)
    L = np.clip(np.asarray(span).astype(np.int64), c["lo"], c["hi"])
    return L, (L.copy() if c["qmax"] == 0 else np.minimum(L, r.integers(c["qmin"], c["qmax"] + 1, B)))


def _indptr(ql):
    return np.concatenate([[0], np.cumsum(ql)])


def _rows(ql):
    """(request, row within the request) of every new-token row."""
    req = np.repeat(np.arange(len(ql)), ql)
    return req, np.arange(int(ql.sum())) - _indptr(ql)[:-1][req]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(shape, g):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def _tables(blocks, g):
    """A table of shuffled block ids (unused entries -1) and the pool's size, a tenth more than is in use."""
    n = int(blocks.sum())
    pool = n + max(1, n // 10)
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    b = torch.as_tensor(blocks).cuda()
    col = torch.arange(max(1, int(blocks.max())), device="cuda")
    at = (torch.cumsum(b, 0) - b)[:, None] + col[None, :]
    table = torch.where(col[None, :] < b[:, None], perm[at.clamp_max(pool - 1)], torch.full_like(at, -1, dtype=torch.int32))
    return table.to(torch.int32).contiguous(), pool


# ------------------------------------------------------------------ prepare

def prepare(case, seed):
    return {"rotary": _prepare_rotary, "write": _prepare_write}.get(case["op"], _prepare_attention)(case, seed)


def _frequencies(c, s):
    """Radians per position of every pair, and the axis whose position turns it."""
    pairs = c["R"] // 2
    s["freq"] = torch.as_tensor(10000.0 ** (-np.arange(pairs) / pairs), dtype=torch.float64).cuda()
    i = np.arange(pairs)
    s["axis"] = _i32(i % c["axes"] if c["split"] == "cycle" else i * c["axes"] // pairs)
    if own:
        from mla_decode_speculative_gb300 import mla
        s["turns"] = mla.rotary_turns(s["freq"])


def _positions(c, T, g):
    """[axes, T]: runs of text, whose axes go together, and of image patches on a grid, from a far start."""
    start = int(torch.randint(0, c["far"], (1,), generator=g, device="cuda"))
    t = torch.arange(T, device="cuda")
    grid = torch.stack([t // 1024, t // 32 % 32, t % 32])
    text = (t // 256) % 3 == 0
    return torch.where(text, start + t, start + grid)[:c["axes"]].to(torch.int32).contiguous() if c["axes"] > 1 else \
        (start + t).to(torch.int32)[None].contiguous()


def _prepare_rotary(c, seed):
    g = _gen(seed)
    T, H, R = c["T"], c["H"], c["R"]
    s = dict(c=c, pos=_positions(c, T, g), q=_normal((T, H, 128 + R), g)[:, :, 128:], k=_normal((T, 1, LATENT + R), g)[..., LATENT:])
    # where the rotated parts go: the last values of the absorbed queries and of the new latent rows
    s["q_out"] = torch.zeros((T, H, LATENT + R), dtype=torch.bfloat16, device="cuda")[:, :, LATENT:]
    s["k_out"] = torch.zeros((T, 1, LATENT + R), dtype=torch.bfloat16, device="cuda")[:, :, LATENT:]
    _frequencies(c, s)
    return s


def _prepare_write(c, seed):
    g = _gen(seed)
    L, ql = _lengths(c)
    H, Hkv, D, Dv, bs, W = c["H"], c["Hkv"], c["D"], c["Dv"], c["bs"], c["W"]
    table, pool = _tables(-(-(-(-L // W)) // bs), g)
    req, t = _rows(ql)
    at = (L - ql)[req] + t  # global position; round-robin over the shards
    T = len(at)
    mine, j = torch.as_tensor(at % W == c["rank"]).cuda(), torch.as_tensor(at // W).cuda()
    ids = table[torch.as_tensor(req).cuda(), j // bs].long()
    fused = _normal((T, H * D + Hkv * (D + Dv)), g)  # one projection's rows
    q, k, v = fused.split([H * D, Hkv * D, Hkv * Dv], 1)
    s = dict(c=c, pos=_positions(c, T, g), q=q.view(T, H, D), k=k.view(T, Hkv, D), v=v.view(T, Hkv, Dv),
             q_out=torch.zeros((T, H, D), dtype=torch.bfloat16, device="cuda"),
             slots=torch.where(mine, ids * bs + j % bs, -1).to(torch.int32),
             k_cache=_normal((pool * bs, Hkv, D), g), v_cache=_normal((pool * bs, Hkv, Dv), g))
    _frequencies(c, s)
    return s


def _prepare_attention(c, seed):
    g = _gen(seed)
    L, ql = _lengths(c)
    H, Hkv, D, bs = c["H"], c["Hkv"], c["D"], c["bs"]
    table, pool = _tables(-(-L // bs), g)
    rows, T, qmax = pool * bs, int(ql.sum()), int(ql.max())
    req, t = _rows(ql)
    s = dict(c=c, T=T, qmax=qmax, scale=1.0 / math.sqrt(D), ind=_i32(_indptr(ql)), row_len=_i32((L - ql)[req] + t + 1),
             row_req=torch.as_tensor(req).cuda(), row_t=torch.as_tensor(t).cuda())
    # the sub-page table a program holds: pages of the largest power of two in a block, 128 at most
    P = s["P"] = min(128, bs & -bs)
    pages = -(-L // P)
    col = torch.arange(int(pages.max()), device="cuda")
    sub = table.long()[:, (col * P) // bs] * (bs // P) + (col % (bs // P))
    s["sub"] = torch.where(col[None, :] < torch.as_tensor(pages).cuda()[:, None], sub, -1).to(torch.int32).contiguous()
    if c["op"] == "grouped":
        s["q"] = _normal((T, H, D), g)
        if c["joint"]:
            pool_kv = _normal((rows, 2, Hkv, D), g)
            s["k"], s["v"] = pool_kv[:, 0], pool_kv[:, 1]
        else:
            s["k"], s["v"] = _normal((rows, Hkv, D), g), _normal((rows, Hkv, D), g)
        s["out"], s["lse"] = torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"), torch.empty((T, H), device="cuda")
    else:
        s["q"], s["k"], s["v"] = _normal((T, H, 2, D), g), _normal((rows, Hkv, 2, D), g), _normal((rows, Hkv, 2 * D), g)
        s["lam"] = 0.2 + 0.6 * torch.rand(H, generator=g, device="cuda")
        s["gain"] = 0.2 * (1.0 + 0.1 * torch.randn(2 * D, generator=g, device="cuda")) if c["norm"] else None
        s["out"] = torch.empty((T, H, 2 * D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty((T, H, 2), device="cuda")
    if own:
        from mla_decode_speculative_gb300 import mla
        need = mla.decode_grouped_workspace_bytes(H, Hkv, qmax, D, differential=c["op"] == "differential")
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ run

def run(state):
    op = state["c"]["op"]
    if own:
        return {"rotary": _own_rotary, "write": _own_write, "grouped": _own_grouped, "differential": _own_differential}[op](state)
    return {"rotary": _plain_rotary, "write": _plain_write, "grouped": _plain_grouped, "differential": _plain_differential}[op](state)


def _own_rotary(s):
    from mla_decode_speculative_gb300 import mla
    mla.rotary(s["q"], s["k"], s["pos"], s["turns"], s["axis"], neighbours=s["c"]["neighbours"], q_out=s["q_out"],
               k_out=s["k_out"])
    return s["q_out"], s["k_out"]


def _own_write(s):
    from mla_decode_speculative_gb300 import mla
    mla.rotary_write(s["q"], s["k"], s["v"], s["pos"], s["turns"], s["slots"], s["k_cache"], s["v_cache"], s["axis"],
                     neighbours=s["c"]["neighbours"], q_out=s["q_out"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _own_grouped(s):
    from mla_decode_speculative_gb300 import mla
    mla.decode_grouped(s["q"], s["k"], s["v"], s["ind"], s["row_len"], s["sub"], s["P"], s["qmax"], s["scale"],
                       window=s["c"]["window"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _own_differential(s):
    from mla_decode_speculative_gb300 import mla
    mla.decode_differential(s["q"], s["k"], s["v"], s["lam"], s["ind"], s["row_len"], s["sub"], s["P"], s["qmax"], s["scale"],
                            gain=s["gain"], eps=EPS, window=s["c"]["window"], out=s["out"], lse=s["lse"],
                            workspace=s["workspace"])
    return s["out"], s["lse"]


def _plain_turn(x, s):
    """x with its first R values of the last dimension rotated, float32."""
    c = s["c"]
    R = c["R"]
    angle = s["pos"].double()[s["axis"].long()].T * s["freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    y = x.float()
    a, b = (y[..., 0:R:2], y[..., 1:R:2]) if c["neighbours"] else (y[..., :R // 2], y[..., R // 2:R])
    a, b = a * cos - b * sin, b * cos + a * sin
    if c["neighbours"]:
        return torch.cat([torch.stack([a, b], -1).flatten(-2), y[..., R:]], -1)
    return torch.cat([a, b, y[..., R:]], -1)


def _plain_rotary(s):
    s["q_out"].copy_(_plain_turn(s["q"], s))
    s["k_out"].copy_(_plain_turn(s["k"], s))
    return s["q_out"], s["k_out"]


def _plain_write(s):
    s["q_out"].copy_(_plain_turn(s["q"], s))
    mine = s["slots"] >= 0
    at = s["slots"][mine].long()
    s["k_cache"][at] = _plain_turn(s["k"], s)[mine].to(torch.bfloat16)
    s["v_cache"][at] = s["v"][mine]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _plain_map(s, q, k, v):
    """One softmax map: q [T, H, D] over k [N, Hkv, D], v [N, Hkv, Dv]; (outputs [T, H, Dv], log sums [T, H]) in float32."""
    c = s["c"]
    B, Hkv, P, qmax = c["B"], c["Hkv"], s["P"], s["qmax"]
    G = c["H"] // Hkv
    sub = s["sub"].long()
    pos = torch.arange(sub.shape[1] * P, device=sub.device)
    at = (sub[:, pos // P] * P + pos % P).clamp_min(0)
    rows = torch.zeros((B, qmax, Hkv, G, q.shape[-1]), device=sub.device)
    rows[s["row_req"], s["row_t"]] = q.float().view(-1, Hkv, G, q.shape[-1])
    rows = rows.permute(0, 2, 1, 3, 4).reshape(B, Hkv, qmax * G, -1)
    seen = torch.zeros((B, qmax), dtype=torch.int32, device=sub.device)
    seen[s["row_req"], s["row_t"]] = s["row_len"]
    gone = pos[None, None, :] >= seen[:, :, None]
    if c["window"]:
        gone |= pos[None, None, :] < seen[:, :, None] - c["window"]
    score = rows @ k[at].float().permute(0, 2, 3, 1) * s["scale"]
    score = score.view(B, Hkv, qmax, G, -1).masked_fill_(gone[:, None, :, None, :], -math.inf)
    top = score.amax(4, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    total = p.sum(4, keepdim=True)
    out = p.view(B, Hkv, qmax * G, -1) @ v[at].float().permute(0, 2, 1, 3)
    out = out.view(B, Hkv, qmax, G, -1) / total.clamp_min(1e-30)
    lse = (top + torch.log(total))[..., 0]
    out, lse = out.permute(0, 2, 1, 3, 4).flatten(2, 3), lse.permute(0, 2, 1, 3).flatten(2, 3)
    return out[s["row_req"], s["row_t"]], lse[s["row_req"], s["row_t"]]


def _plain_grouped(s):
    out, lse = _plain_map(s, s["q"], s["k"], s["v"])
    s["out"].copy_(out)
    s["lse"].copy_(lse)
    return s["out"], s["lse"]


def _plain_differential(s):
    (a, la), (b, lb) = (_plain_map(s, s["q"][:, :, m], s["k"][:, :, m], s["v"]) for m in (0, 1))
    y = a - s["lam"][None, :, None] * b
    if s["gain"] is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * s["gain"]
    s["out"].copy_(y)
    s["lse"].copy_(torch.stack([la, lb], -1))
    return s["out"], s["lse"]


# ------------------------------------------------------------------ work

def work(case):
    c = case
    if c["op"] == "rotary":
        n = c["T"] * (c["H"] + 1) * c["R"]
        return {"bytes": 4 * n + c["T"] * c["axes"] * 4 + c["R"] * 6, "flops": 3 * n}
    L, ql = _lengths(c)
    T, H, Hkv, D = int(ql.sum()), c["H"], c["Hkv"], c["D"]
    if c["op"] == "write":
        req, t = _rows(ql)
        mine = int((((L - ql)[req] + t) % c["W"] == c["rank"]).sum())
        return {"bytes": 4 * T * H * D + 4 * mine * Hkv * (D + c["Dv"]) + T * (4 + 4 * c["axes"]),
                "flops": 3 * (T * H + mine * Hkv) * c["R"]}
    lo = np.maximum(L - ql + 1 - c["window"], 0) if c["window"] else 0 * L
    tokens = int((L - lo).sum())
    req, t = _rows(ql)
    n = (L - ql)[req] + t + 1
    seen = int(np.minimum(n, c["window"]).sum() if c["window"] else n.sum())
    maps, Dv = (1, D) if c["op"] == "grouped" else (2, 2 * D)
    return {"bytes": 2 * tokens * Hkv * (maps * D + Dv) + T * H * (2 * maps * D + 2 * Dv + 4 * maps),
            "flops": 2 * seen * H * maps * (D + Dv)}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_turn(s["q"], s), _exact_turn(s["k"], s)
    if case["op"] == "write":
        k, v = s["k_cache"].double(), s["v_cache"].double()
        rows = torch.nonzero(s["slots"] >= 0).view(-1)
        at = s["slots"][rows].long()
        k[at], v[at] = _exact_turn(s["k"], s)[rows], s["v"][rows].double()
        return _exact_turn(s["q"], s), k, v
    return _exact_attention(s)


def _exact_turn(x, s):
    """Every pair as a complex number, times e^(i angle)."""
    c = s["c"]
    R = c["R"]
    y = x.double()
    pos = s["pos"].double()
    angle = torch.stack([pos[a] * f for a, f in zip(s["axis"].tolist(), s["freq"].tolist())], 1)
    head = y[..., :R].reshape(*y.shape[:-1], R // 2, 2) if c["neighbours"] else \
        y[..., :R].reshape(*y.shape[:-1], 2, R // 2).transpose(-1, -2)
    z = torch.view_as_complex(head.contiguous()) * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    z = torch.view_as_real(z)
    z = z.flatten(-2) if c["neighbours"] else z.transpose(-1, -2).flatten(-2)
    return torch.cat([z, y[..., R:]], -1)


def _exact_attention(s):
    c = s["c"]
    G, maps = c["H"] // c["Hkv"], 1 if c["op"] == "grouped" else 2
    ind, seen = s["ind"].tolist(), s["row_len"].tolist()
    q = s["q"].view(s["T"], c["H"], maps, c["D"])
    key = s["k"].unflatten(1, (c["Hkv"], 1)) if maps == 1 else s["k"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["T"], c["H"], maps), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        r = slice(ind[b], ind[b + 1])
        n = torch.as_tensor(seen[r], device="cuda")
        first = max(0, min(seen[r]) - c["window"]) if c["window"] else 0
        j = torch.arange(first, max(seen[r]), device="cuda")
        at = s["sub"][b].long()[j // s["P"]] * s["P"] + j % s["P"]
        hidden = (j[None, :] >= n[:, None]) | ((j[None, :] < n[:, None] - c["window"]) if c["window"] else False)
        for g in range(c["Hkv"]):
            h = slice(g * G, (g + 1) * G)
            val = s["v"][at, g].double()
            y = []
            for m in range(maps):
                score = torch.einsum("thd,nd->thn", q[r, h, m].double(), key[at, g, m].double()) * s["scale"]
                score = score.masked_fill(hidden[:, None, :], -math.inf)
                lse[r, h, m] = torch.logsumexp(score, 2)
                y.append(torch.exp(score - lse[r, h, m][..., None]) @ val)
            out[r, h] = y[0] if maps == 1 else y[0] - s["lam"][h].double()[None, :, None] * y[1]
    if maps == 2 and s["gain"] is not None:
        out = out / torch.sqrt((out ** 2).mean(-1, keepdim=True) + EPS) * s["gain"].double()
    return out, (lse[..., 0] if maps == 1 else lse)
