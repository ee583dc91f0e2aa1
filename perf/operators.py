"""Work of the paged 8-bit latent cache: its block tables, its quantising write and the attention over it.

Three operators, as a serving step calls them one after the other:

* ``tables``: block tables and slot map of a batch from the requests' lengths (blocks come from and go
  back to a ring of free blocks);
* ``write``: new latent rows quantised to e4m3 into the rows a slot map names, one power-of-two scale per
  block of ``G`` tokens;
* ``attention``: absorbed-form MLA decode / causal verify over that cache.

With ``own`` false ``run`` computes them in elementary torch operations, otherwise through the package's calls.
Request lengths follow from the case alone; values, block ids and queries from the seed.
"""
import math

import numpy as np
import torch

own = False

D_K, D_V = 576, 512
SM_SCALE = 1.0 / math.sqrt(192.0)
MIN_EXP = -100  # smallest scale the write chooses: 2^-100


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one speculative step of a small batch: every request grows by four tokens, few of them into a new block
        dict(name="tables_verify_b32", op="tables", B=32, lo=1024, hi=8192, qmin=4, qmax=4, bs=64, W=1, rank=0, I=1,
             back=4, new=0.0, gone=0.0, lens=1),
        # one shard of eight, small blocks, long contexts: drafts taken back, a tenth of the requests finished or new
        dict(name="tables_shard_b256", op="tables", B=256, lo=4096, hi=135168, qmin=1, qmax=8, bs=16, W=8, rank=3, I=1,
             back=8, new=0.1, gone=0.1, lens=2),
        # admission of a batch of prompts: every block is new and every prompt token needs its slot
        dict(name="tables_admit_b200", op="tables", B=200, lo=512, hi=16384, qmin=0, qmax=0, bs=16, W=1, rank=0, I=1,
             back=0, new=1.0, gone=0.0, lens=3),
        # appending a speculative step's tokens to partly filled scale blocks
        dict(name="write_verify_b32_g64", op="write", B=32, lo=1024, hi=8192, qmin=4, qmax=4, bs=64, G=64, W=1, rank=0, I=1,
             lens=4),
        # the same for a large batch on one of four shards: three rows of four belong to other shards
        dict(name="write_shard_b256_g16", op="write", B=256, lo=512, hi=4096, qmin=1, qmax=8, bs=16, G=16, W=4, rank=2, I=1,
             lens=5),
        # a chunk of prompts, one scale per token; odd lengths
        dict(name="write_prompt_g1", op="write", B=5, lo=2100, hi=6300, qmin=0, qmax=0, bs=16, G=1, W=1, rank=0, I=1, lens=6),
        # the largest prompt chunk of a prefill step, one scale per 64 tokens
        dict(name="write_prompt_g64", op="write", B=16, lo=6144, hi=10240, qmin=0, qmax=0, bs=64, G=64, W=1, rank=0, I=1,
             lens=7),
        # the smallest decode: two short requests, one token each (latency)
        dict(name="attention_decode_b2", op="attention", B=2, lo=256, hi=256, H=16, qmin=1, qmax=1, bs=16, G=16, S=1, lens=8),
        # multi-token verify of a medium batch
        dict(name="attention_verify_b32", op="attention", B=32, lo=1024, hi=8192, H=16, qmin=4, qmax=4, bs=64, G=64, S=16,
             lens=9),
        # ragged lengths and verify rows, twelve heads, small pages
        dict(name="attention_ragged_b64", op="attention", B=64, lo=512, hi=32768, H=12, qmin=1, qmax=3, bs=16, G=8, S=16,
             lens=10),
        # long contexts, where the cache's bytes decide
        dict(name="attention_long_b16", op="attention", B=16, lo=131072, hi=131072, H=16, qmin=4, qmax=4, bs=64, G=32, S=16,
             lens=11),
        # unsplit heads: many query rows per request
        dict(name="attention_h128_b8", op="attention", B=8, lo=4096, hi=16384, H=128, qmin=2, qmax=2, bs=256, G=64, S=16,
             lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "write", "attention", "attention"])
    bs = rng.choice([8, 16, 32, 64, 96, 128, 256])
    lens = rng.randrange(1000, 1 << 20)
    if op == "tables":
        B = _log_int(rng, 1, 400)
        hi = _log_int(rng, 64, min(135168, 4_000_000 // B))
        qmin, qmax = rng.choice([(1, 1), (4, 4), (1, 8), (0, 0)])
        if qmax == 0:
            hi = min(hi, 1_600_000 // B)
        W = rng.choice([1, 1, 2, 3, 8])
        return dict(op=op, B=B, lo=max(16, hi // rng.choice([2, 8, 32])), hi=hi, qmin=qmin, qmax=qmax, bs=bs, W=W,
                    rank=rng.randrange(W), I=rng.choice([1, 1, 4]), back=rng.choice([0, 8, 40]),
                    new=1.0 if qmax == 0 else rng.choice([0.0, 0.1, 0.3]), gone=rng.choice([0.0, 0.1, 0.2]), lens=lens)
    page = min(128, bs & -bs)
    G = rng.choice([g for g in (1, 2, 4, 8, 16, 32, 64) if g <= page])
    if op == "write":
        qmin, qmax = rng.choice([(1, 1), (4, 4), (1, 8), (0, 0)])
        B = _log_int(rng, 1, 256)
        hi = _log_int(rng, 64, (120_000 if qmax == 0 else 400_000) // B)
        W = rng.choice([1, 1, 2, 5])
        return dict(op=op, B=B, lo=max(16, hi // rng.choice([2, 8])), hi=hi, qmin=qmin, qmax=qmax, bs=bs, G=G, W=W,
                    rank=rng.randrange(W), I=rng.choice([1, 1, 4]), lens=lens)
    H = rng.choice([12, 16, 16, 64, 128, rng.randrange(1, 129)])
    qmax = rng.choice([1, 2, 3, 4, 8])
    B = _log_int(rng, 1, 256)
    hi = _log_int(rng, 64, min(135168, 2_000_000 // B, 100_000_000 // (B * H * qmax)))
    return dict(op=op, B=B, lo=max(16, hi // rng.choice([1, 4, 16])), hi=hi, H=H, qmin=rng.randrange(1, qmax + 1), qmax=qmax,
                bs=bs, G=G, S=rng.choice([1, 4, 16]), lens=lens)


# ------------------------------------------------------------------ lengths (from the case alone)

def _owner_index(g, W, I):
    """(rank, local index) of global position g: runs of I positions dealt to W ranks in turn."""
    return (g // I) % W, (g // (I * W)) * I + g % I


def _local_len(n, W, rank, I):
    """Positions g < n that a rank holds."""
    return (n // (I * W)) * I + np.clip(n % (I * W) - rank * I, 0, I)


def _lengths(c):
    """(prev, length, qlen) per request: tokens whose blocks are held, tokens after the step, new ones among them."""
    r = np.random.default_rng(c["lens"])
    B = c["B"]
    span = np.exp(r.uniform(math.log(c["lo"]), math.log(c["hi"] + 1), B)) if c["hi"] > 4 * c["lo"] \
        else r.integers(c["lo"], c["hi"] + 1, B)
    L = np.clip(np.asarray(span).astype(np.int64), c["lo"], c["hi"])
    ql = L.copy() if c["qmax"] == 0 else np.minimum(L, r.integers(c["qmin"], c["qmax"] + 1, B))
    prev = L - ql
    if c["op"] == "tables":
        prev = prev + r.integers(0, c["back"] + 1, B)  # drafts of the last step that were not accepted
        state = r.random(B)
        fresh = state < c["new"]
        prev[fresh] = 0
        ql[fresh] = np.minimum(L[fresh], 2048) if c["qmax"] else L[fresh]
        gone = state > 1.0 - c["gone"]
        L[gone], ql[gone] = 0, 0
    return prev, L, ql


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


def _pow2(e):
    """2^e in float32 (e within the normal range), exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def _tables(blocks, g, spare=0.1):
    """A table of shuffled block ids (unused entries -1), the ids left over, and the pool's size."""
    n = int(blocks.sum())
    pool = max(1, int(math.ceil(n * (1.0 + spare))))
    perm = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    width = max(1, int(blocks.max()))
    b = torch.as_tensor(blocks).cuda()
    col = torch.arange(width, device="cuda")
    used = col[None, :] < b[:, None]
    at = (torch.cumsum(b, 0) - b)[:, None] + col[None, :]
    table = torch.where(used, perm[at.clamp_max(pool - 1)], torch.full_like(at, -1, dtype=torch.int32))
    return table.to(torch.int32).contiguous(), perm[n:], pool


# ------------------------------------------------------------------ prepare

def prepare(case, seed):
    return {"tables": _prepare_tables, "write": _prepare_write, "attention": _prepare_attention}[case["op"]](case, seed)


def _prepare_tables(c, seed):
    g = _gen(seed)
    prev, L, ql = _lengths(c)
    W, rank, I, bs = c["W"], c["rank"], c["I"], c["bs"]
    held, need = (-(-_local_len(n, W, rank, I) // bs) for n in (prev, L))
    take = int(np.maximum(need - held, 0).sum())
    table, spare, pool = _tables(np.maximum(held, 0), g, spare=0.0)
    # a pool with the blocks in use, those the step will take, and a tenth more; the free ones in a ring
    pool_all = int(held.sum()) + take + max(8, (int(held.sum()) + take) // 10)
    ids = torch.randperm(pool_all, generator=g, device="cuda").to(torch.int32)
    width = max(1, int(max(held.max(), need.max())))
    wide = torch.full((c["B"], width), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = torch.where(table >= 0, ids[table.clamp_min(0).long()], table)
    n_free = pool_all - int(held.sum())
    head = int(torch.randint(0, pool_all, (1,), generator=g, device="cuda"))
    ring = torch.full((pool_all,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(n_free, device="cuda")) % pool_all] = ids[int(held.sum()):]
    T = int(ql.sum())
    return dict(c=c, T=T, prev=_i32(prev), seq=_i32(L), ind=_i32(_indptr(ql)), table=wide, ring=ring,
                ring_in=_i32([head, n_free]), ring_out=torch.zeros(2, dtype=torch.int32, device="cuda"),
                slots=torch.empty(T, dtype=torch.int32, device="cuda"))


def _write_slots(c, table):
    """Slot of every new row on the case's rank (-1: another rank's)."""
    _, L, ql = _lengths(c)
    req, t = _rows(ql)
    g = (L - ql)[req] + t
    own_rank, j = _owner_index(g, c["W"], c["I"])
    req, j = torch.as_tensor(req).cuda(), torch.as_tensor(j).cuda()
    ids = table[req, torch.clamp(j // c["bs"], max=table.shape[1] - 1)].long()
    return torch.where(torch.as_tensor(own_rank == c["rank"]).cuda(), ids * c["bs"] + j % c["bs"], -1).to(torch.int32)


def _prepare_write(c, seed):
    g = _gen(seed)
    _, L, ql = _lengths(c)
    table, _, pool = _tables(-(-_local_len(L, c["W"], c["rank"], c["I"]) // c["bs"]), g)
    rows, G = pool * c["bs"], c["G"]
    T = int(ql.sum())
    # latents after a norm: about N(0, 1), tokens of different magnitude, some channels much larger
    x = torch.randn((T, D_K), generator=g, device="cuda")
    x *= torch.exp2(torch.randn((T, 1), generator=g, device="cuda"))
    x[:, ::97] *= 6.0
    cache = (torch.randn((rows, D_K), generator=g, device="cuda") * 60).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scales = _pow2(torch.randint(-7, -2, (rows // G,), generator=g, device="cuda"))
    return dict(c=c, x=x.to(torch.bfloat16), slots=_write_slots(c, table), cache=cache.view(torch.uint8), scales=scales)


def _prepare_attention(c, seed):
    g = _gen(seed)
    _, L, ql = _lengths(c)
    bs, G, H = c["bs"], c["G"], c["H"]
    table, _, pool = _tables(-(-L // bs), g)
    rows, T = pool * bs, int(ql.sum())
    codes = torch.empty((rows, D_K), dtype=torch.uint8, device="cuda")
    scales = torch.empty(rows // G, device="cuda")
    step = (1 << 18) // G * G
    for at in range(0, rows, step):  # N(0, 1) rows, blocks of different magnitude, quantised as the write does
        x = torch.randn((min(step, rows - at) // G, G * D_K), generator=g, device="cuda")
        x *= torch.exp2(0.7 * torch.randn((x.shape[0], 1), generator=g, device="cuda"))
        m, e = torch.frexp(x.abs().amax(1))
        s = _pow2(e - 9 + (m > 0.875))
        codes[at:at + x.shape[0] * G] = (x / s[:, None]).to(torch.float8_e4m3fn).view(torch.uint8).view(-1, D_K)
        scales[at // G:at // G + x.shape[0]] = s
    q = torch.randn((T, H, D_K), generator=g, device="cuda").to(torch.bfloat16)
    # the row plan a program holds: visible tokens of every row, sub-page table
    req, t = _rows(ql)
    P = min(128, bs & -bs)
    pages = -(-L // P)
    width = int(pages.max())
    col = torch.arange(width, device="cuda")
    sub = table[:, :].long()[:, (col * P) // bs] * (bs // P) + (col % (bs // P))
    sub = torch.where(col[None, :] < torch.as_tensor(pages).cuda()[:, None], sub, -1).to(torch.int32).contiguous()
    a256 = lambda n: (n + 255) & ~255  # noqa: E731
    S, qmax = c["S"], int(ql.max())
    units = c["B"] * (-(-qmax * H // 64))
    space = 256 + (0 if S == 1 else a256(units * S * 65536) + 2 * a256(T * H * S * 4) + a256(units * 4))
    return dict(c=c, T=T, P=P, qmax=qmax, q=q, cache=codes, scales=scales, ind=_i32(_indptr(ql)),
                row_len=_i32((L - ql)[req] + t + 1), row_req=torch.as_tensor(req).cuda(), row_t=torch.as_tensor(t).cuda(),
                sub=sub, workspace=torch.empty(space, dtype=torch.uint8, device="cuda"),
                out=torch.empty((T, H, D_V), dtype=torch.bfloat16, device="cuda"),
                lse=torch.empty((T, H), device="cuda"))


# ------------------------------------------------------------------ run

def run(state):
    op = state["c"]["op"]
    if own:
        return {"tables": _own_tables, "write": _own_write, "attention": _own_attention}[op](state)
    return {"tables": _plain_tables, "write": _plain_write, "attention": _plain_attention}[op](state)


def _own_tables(s):
    from mla_decode_speculative_gb300 import mla
    c = s["c"]
    mla.update_block_tables(s["prev"], s["seq"], s["ind"], s["table"], s["ring"], s["ring_in"], c["bs"], s["T"],
                            ring_out=s["ring_out"], slot_map=s["slots"], world_size=c["W"], rank=c["rank"],
                            interleave=c["I"])
    return s["table"], s["ring"], s["ring_out"], s["slots"]


def _own_write(s):
    from mla_decode_speculative_gb300 import mla
    mla.write_kv_scaled(s["x"], s["slots"], s["cache"], s["scales"], s["c"]["G"])
    return s["cache"].view(torch.float8_e4m3fn), s["scales"]


def _own_attention(s):
    from mla_decode_speculative_gb300 import mla
    c = s["c"]
    mla.decode_verify_scaled(s["q"], s["cache"], s["scales"], c["G"], s["ind"], s["row_len"], s["sub"], s["P"], c["S"],
                             s["qmax"], SM_SCALE, out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return s["out"], s["lse"]


def _plain_tables(s):
    c = s["c"]
    W, rank, I, bs = c["W"], c["rank"], c["I"], c["bs"]
    table, ring = s["table"], s["ring"]
    pool = ring.shape[0]
    cycle = I * W
    prev, L, ind = s["prev"].long(), s["seq"].long(), s["ind"].long()
    held, need = ((n // cycle * I + (n % cycle - rank * I).clamp(0, I) + bs - 1) // bs for n in (prev, L))
    take, rel = (need - held).clamp_min(0), (held - need).clamp_min(0)
    off, roff = torch.cumsum(take, 0) - take, torch.cumsum(rel, 0) - rel
    head, count = s["ring_in"].long()
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    k = off[:, None] + col - held[:, None]
    dealt = torch.where(k < count, ring[(head + k) % pool], -1)
    new = (col >= held[:, None]) & (col < need[:, None])
    freed = (col >= need[:, None]) & (col < held[:, None])
    back = (head + count + roff[:, None] + col - need[:, None]) % pool
    ids = torch.where(freed, table, -1)
    table.copy_(torch.where(new, dealt, table))
    # freed ids go to their places; every other cell writes past the end of a longer copy
    longer = torch.cat([ring, ring.new_zeros(1)])
    longer.scatter_(0, torch.where(freed, back, pool).view(-1), ids.view(-1))
    ring.copy_(longer[:pool])
    took = torch.minimum(take.sum(), count)
    s["ring_out"].copy_(torch.stack([(head + took) % pool, count - took + rel.sum()]))
    r = torch.arange(s["T"], device=table.device)
    b = torch.searchsorted(ind, r, right=True) - 1
    g = L[b] - (ind[b + 1] - ind[b]) + r - ind[b]
    j = g // cycle * I + g % I
    block = table[b, (j // bs).clamp_max(table.shape[1] - 1)].long()
    mine = ((g // I) % W == rank) & (block >= 0)
    s["slots"].copy_(torch.where(mine, block * bs + j % bs, -1))
    return table, ring, s["ring_out"], s["slots"]


def _plain_write(s):
    x, slots, cache, scales, G = s["x"].float(), s["slots"].long(), s["cache"], s["scales"], s["c"]["G"]
    n = scales.shape[0]
    mine = slots >= 0
    block = torch.where(mine, slots // G, n)
    fresh = torch.zeros(n + 1, device=x.device).scatter_reduce(0, block, x.abs().amax(1), "amax")[:n]
    first = torch.full((n + 1,), G, device=x.device).scatter_reduce(0, block, slots % G, "amin")[:n]
    m, e = torch.frexp(fresh)
    want = _pow2((e - 9 + (m > 0.875)).clamp_min(MIN_EXP))
    want = torch.where(fresh > 0, want, 2.0 ** MIN_EXP)
    scale = torch.where(first == 0, want, torch.where(first < G, torch.maximum(scales, want), scales))
    # earlier tokens of the blocks whose scale grew
    grown = torch.nonzero((first > 0) & (first < G) & (scale > scales)).view(-1)
    rows = grown[:, None] * G + torch.arange(G, device=x.device)[None, :]
    old = cache[rows].view(torch.float8_e4m3fn)
    again = (old.float() * (scales[grown] / scale[grown])[:, None, None]).to(torch.float8_e4m3fn)
    keep = torch.arange(G, device=x.device)[None, :] < first[grown][:, None]
    cache[rows] = torch.where(keep[:, :, None], again.view(torch.uint8), old.view(torch.uint8))
    scales.copy_(scale)
    code = (x / scale[block.clamp_max(n - 1)][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache[slots[mine]] = code[mine]
    return cache.view(torch.float8_e4m3fn), scales


def _plain_attention(s):
    c = s["c"]
    B, H, G, P, qmax = c["B"], c["H"], c["G"], s["P"], s["qmax"]
    sub = s["sub"].long()
    pos = torch.arange(sub.shape[1] * P, device=sub.device)
    at = (sub[:, pos // P] * P + pos % P).clamp_min(0)
    k = s["cache"][at].view(torch.float8_e4m3fn).float() * s["scales"][at // G][:, :, None]
    q = torch.zeros((B, qmax, H, D_K), device=sub.device)
    q[s["row_req"], s["row_t"]] = s["q"].float()
    seen = torch.zeros((B, qmax), dtype=torch.int32, device=sub.device)
    seen[s["row_req"], s["row_t"]] = s["row_len"]
    score = (q.view(B, qmax * H, D_K) @ k.transpose(1, 2)).view(B, qmax, H, -1) * SM_SCALE
    score.masked_fill_(pos[None, None, None, :] >= seen[:, :, None, None], -math.inf)
    top = score.amax(3, keepdim=True).clamp_min(-1e30)
    p = torch.exp(score - top)
    total = p.sum(3, keepdim=True)
    out = (p.view(B, qmax * H, -1) @ k[:, :, :D_V]).view(B, qmax, H, D_V) / total.clamp_min(1e-30)
    lse = (top + torch.log(total))[..., 0]
    s["out"].copy_(out[s["row_req"], s["row_t"]])
    s["lse"].copy_(lse[s["row_req"], s["row_t"]])
    return s["out"], s["lse"]


# ------------------------------------------------------------------ work

def work(case):
    c = case
    prev, L, ql = _lengths(c)
    T = int(ql.sum())
    if c["op"] == "tables":
        held, need = (-(-_local_len(n, c["W"], c["rank"], c["I"]) // c["bs"]) for n in (prev, L))
        moved = int(np.abs(need - held).sum())
        return {"bytes": 12 * c["B"] + 20 + 8 * moved + 4 * T, "flops": 0}
    if c["op"] == "write":
        mine = -(-T // c["W"])
        return {"bytes": 4 * T + mine * (2 * D_K + D_K) + 8 * (-(-mine // c["G"])), "flops": 2 * mine * D_K}
    H = c["H"]
    seen = int((ql * (L - ql) + ql * (ql + 1) // 2).sum())
    tokens = int(L.sum())
    return {"bytes": tokens * D_K + 4 * (-(-tokens // c["G"])) + T * H * (2 * D_K + 2 * D_V + 4),
            "flops": 2 * seen * H * (D_K + D_V)}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    if case["op"] == "tables":
        return None  # whole numbers only
    s = prepare(case, seed)
    return _exact_write(s) if case["op"] == "write" else _exact_attention(s)


def _power(e):
    """2^e in float64, from the exponent's bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _e4m3(y):
    """The e4m3 value nearest to y (ties to even), float64: three mantissa bits down to 2^-6, then steps of 2^-9."""
    y = y.clamp(-448.0, 448.0)
    _, e = torch.frexp(y)
    step = _power((e - 1).clamp_min(-6) - 3)
    return torch.round(y / step) * step


def _exact_write(s):
    G, slots = s["c"]["G"], s["slots"].long()
    value = s["cache"].view(torch.float8_e4m3fn).double()
    scales = s["scales"].double()
    rows = torch.nonzero(slots >= 0).view(-1)
    at, x = slots[rows], s["x"][rows].double()
    touched, unit = torch.unique(at // G, return_inverse=True)
    amax = torch.zeros(touched.shape[0], dtype=torch.float64, device=x.device)
    amax.index_reduce_(0, unit, x.abs().amax(1), "amax")
    first = torch.full((touched.shape[0],), G, device=x.device).index_reduce_(0, unit, at % G, "amin")
    m, e = torch.frexp(amax / 448.0)  # the smallest power of two that is not below amax / 448
    want = _power(torch.where(m > 0.5, e, e - 1).clamp_min(MIN_EXP))
    want = torch.where(amax > 0, want, 2.0 ** MIN_EXP)
    old = scales[touched]
    scale = torch.where(first > 0, torch.maximum(old, want), want)
    cells = touched[:, None] * G + torch.arange(G, device=x.device)
    before = value[cells]
    earlier = torch.arange(G, device=x.device)[None, :] < first[:, None]
    value[cells] = torch.where(earlier[:, :, None], _e4m3(before * (old / scale)[:, None, None]), before)
    value[at] = _e4m3(x / scale[unit][:, None])
    scales[touched] = scale
    return value, scales


def _exact_attention(s):
    c = s["c"]
    ind = s["ind"].tolist()
    seen = s["row_len"].tolist()
    out = torch.zeros((s["T"], c["H"], D_V), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["T"], c["H"]), dtype=torch.float64, device="cuda")
    for b in range(c["B"]):
        n = max(seen[ind[b]:ind[b + 1]])
        j = torch.arange(n, device="cuda")
        at = s["sub"][b].long()[j // s["P"]] * s["P"] + j % s["P"]
        key = s["cache"][at].view(torch.float8_e4m3fn).double() * s["scales"].double()[at // c["G"], None]
        for r in range(ind[b], ind[b + 1]):
            score = s["q"][r].double() @ key[:seen[r]].T * SM_SCALE
            lse[r] = torch.logsumexp(score, 1)
            out[r] = torch.exp(score - lse[r][:, None]) @ key[:seen[r], :D_V]
    return out, lse
