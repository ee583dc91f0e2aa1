"""The paged 8-bit cache on the GPU: block tables and slot map, quantising write, and the decode
over the block-scaled codes, each against its float64 / integer reference, and a run of them
together.  Whole numbers, codes and scales must be equal; outputs are held to the bound that
scaled_reference.out_bound derives and to the framework's bar for the path."""
import math

import numpy as np
import pytest
import torch

import scaled_reference as ref
from parity import LSE_TOL
from mla_decode_speculative_gb300 import mla, runner

pytestmark = pytest.mark.gpu
SM = 1.0 / math.sqrt(192.0)


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def indptr(ql):
    return np.concatenate([[0], np.cumsum(ql)]).astype(np.int64)


# ------------------------------------------------------------------ block tables

def table_state(prev, pool, width, bs, W=1, rank=0, I=1, head=0, seed=0):
    """A consistent state: shuffled ids in the tables, the others in the ring from `head` on."""
    ids = np.random.default_rng(seed).permutation(pool).astype(np.int32)
    table = np.full((len(prev), width), -7, np.int32)
    at = 0
    for b, n in enumerate(prev):
        k = -(-ref.local_len(int(n), W, rank, I) // bs)
        table[b, :k] = ids[at:at + k]
        at += k
    ring = np.full(pool, -9, np.int32)
    ring[(head + np.arange(pool - at)) % pool] = ids[at:]
    return table, ring, (head, pool - at)


def run_tables(prev, seq, ql, table, ring, state, bs, T=None, **shard):
    ind = indptr(ql)
    T = int(ind[-1]) if T is None else T
    d_table, d_ring = i32(table), i32(ring)
    slots, out = mla.update_block_tables(i32(prev), i32(seq), i32(ind), d_table, d_ring, i32(state), bs, T, **shard)
    return d_table.cpu().numpy(), d_ring.cpu().numpy(), tuple(out.tolist()), slots.cpu().numpy()


@pytest.mark.parametrize("B,bs,W,rank,I,seed", [
    (1, 16, 1, 0, 1, 0), (5, 1, 1, 0, 1, 1), (37, 8, 3, 2, 1, 2), (300, 16, 1, 0, 1, 3), (64, 96, 8, 5, 4, 4),
    (700, 4, 2, 1, 16, 5), (256, 256, 1, 0, 1, 6)])
def test_tables_match_reference(B, bs, W, rank, I, seed):
    r = np.random.default_rng(seed)
    prev = r.integers(0, 700, B)
    ql = r.integers(0, 9, B)
    seq = np.maximum(prev - r.integers(0, 12, B) + ql, ql)   # drafts taken back, then the new rows
    gone, fresh, chunk = (r.random(B) < p for p in (0.1, 0.1, 0.1))
    seq[gone], ql[gone] = 0, 0
    prev[fresh] = 0
    ql[chunk] = r.integers(0, 1 + seq[chunk])
    width = -(-1000 // bs)
    held = sum(-(-ref.local_len(int(n), W, rank, I) // bs) for n in np.maximum(prev, seq))
    pool = held + int(r.integers(0, 50)) + 1
    table, ring, state = table_state(prev, pool, width, bs, W, rank, I, head=int(r.integers(0, pool)), seed=seed)
    T = int(ql.sum()) + 5   # rows behind the last request get no slot
    want = ref.update_tables(prev, seq, indptr(ql), table, ring, state, bs, T, W, rank, I)
    got = run_tables(prev, seq, ql, table, ring, state, bs, T, world_size=W, rank=rank, interleave=I)
    assert mla.get_device_error() == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_tables_of_many_requests_and_many_rows():
    """16384 requests (the most), then one request of 300,001 new tokens."""
    r = np.random.default_rng(9)
    prev = r.integers(0, 40, 16384)
    seq = r.integers(0, 40, 16384)
    ql = np.minimum(seq, r.integers(0, 3, 16384))
    table, ring, state = table_state(prev, 16384 * 5, 5, 8, head=16384 * 5 - 3, seed=1)
    want = ref.update_tables(prev, seq, indptr(ql), table, ring, state, 8, int(ql.sum()))
    for g, w in zip(run_tables(prev, seq, ql, table, ring, state, 8), want):
        assert np.array_equal(g, w)
    table, ring, state = table_state([77], 20000, 18760, 16, seed=2)
    want = ref.update_tables([77], [300078], [0, 300001], table, ring, state, 16, 300001)
    for g, w in zip(run_tables([77], [300078], [300001], table, ring, state, 16), want):
        assert np.array_equal(g, w)
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("W,rank,I,at", [(1, 0, 1, 0), (1, 0, 1, 1), (2, 1, 3, 0), (5, 0, 16, 1)])
def test_tables_of_many_rows(W, rank, I, at):
    """More rows than a thread each: several requests, some short, shards, rows behind the last one, and a
    slot map that starts off a 16-byte boundary."""
    ql = np.array([30001, 3, 0, 1, 40000, 2, 5])
    prev = np.array([5, 90, 33, 0, 0, 17, 1000])
    seq = prev + ql - np.array([2, 40, 30, 0, 0, 0, 1])
    bs, width = 24, 2000
    pool = sum(-(-ref.local_len(int(n), W, rank, I) // bs) for n in np.maximum(prev, seq)) + 3
    table, ring, state = table_state(prev, pool, width, bs, W, rank, I, head=pool - 2, seed=4)
    T = int(ql.sum()) + 7
    assert T > 65536
    want = ref.update_tables(prev, seq, indptr(ql), table, ring, state, bs, T, W, rank, I)
    room = torch.full((T + 8,), 77, dtype=torch.int32, device="cuda")
    d_table, d_ring = i32(table), i32(ring)
    slots, out = mla.update_block_tables(i32(prev), i32(seq), i32(indptr(ql)), d_table, d_ring, i32(state), bs, T,
                                         slot_map=room[at:at + T], world_size=W, rank=rank, interleave=I)
    assert mla.get_device_error() == 0
    got = d_table.cpu().numpy(), d_ring.cpu().numpy(), tuple(out.tolist()), slots.cpu().numpy()
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
    assert (room[:at] == 77).all() and (room[at + T:] == 77).all()


def test_tables_are_the_same_when_called_again():
    prev, seq, ql = [20, 40, 0, 9], [24, 10, 33, 0], [4, 2, 33, 0]
    table, ring, state = table_state(prev, 24, 6, 8, head=20)
    d = [i32(table), i32(ring)]
    first = None
    for _ in range(3):
        slots, out = mla.update_block_tables(i32(prev), i32(seq), i32(indptr(ql)), *d, i32(state), 8, 39)
        now = [t.cpu().numpy() for t in (*d, slots, out)]
        assert first is None or all(np.array_equal(a, b) for a, b in zip(first, now))
        first = now


def test_tables_without_requests_or_rows():
    z = torch.zeros(0, dtype=torch.int32, device="cuda")
    slots, out = mla.update_block_tables(z, z, i32([0]), torch.zeros((0, 4), dtype=torch.int32, device="cuda"),
                                         i32([0, 1, 2]), i32([2, 1]), 16, 3)
    assert out.tolist() == [2, 1] and slots.tolist() == [-1, -1, -1]
    assert mla.get_device_error() == 0


def test_tables_device_checks():
    """Bad inputs are recorded and nothing out of range is touched."""
    prev, seq, ql = [10, 3], [26, 20], [4, 17]
    table, ring, state = table_state(prev, 8, 4, 8, head=6)

    def run(code, prev=prev, seq=seq, ind=None, ring=ring, state=state, width=4):
        d_table, d_ring = i32(table[:, :width]), i32(ring)
        slots, out = mla.update_block_tables(i32(prev), i32(seq), i32(indptr(ql) if ind is None else ind), d_table,
                                             d_ring, i32(state), 8, 21)
        assert mla.get_device_error() == code
        return d_table.cpu().numpy(), d_ring.cpu().numpy(), out.tolist(), slots.cpu().numpy()

    for bad in ([1, 4, 21], [0, 5, 4], [0, 4, 22]):
        t, g, out, slots = run(1, ind=bad)
        assert np.array_equal(t, table) and np.array_equal(g, ring) and out == list(state) and (slots == -1).all()
    for bad in ((-1, 5), (8, 5), (0, 9), (0, -1)):
        t, g, out, slots = run(8, state=bad)
        assert np.array_equal(t, table) and np.array_equal(g, ring) and out == list(bad) and (slots == -1).all()
    t, g, out, slots = run(8, seq=[0, 0], ind=[0, 0, 0], state=(6, 6))   # three returned to a ring of six of eight
    assert np.array_equal(t, table) and np.array_equal(g, ring)
    _, _, _, slots = run(2, seq=[3, 20])                                 # four new rows of three tokens
    assert (slots[:4] == -1).all() and (slots[4:] >= 0).all()
    t, _, out, slots = run(4, width=3)                                   # 26 tokens in three blocks of eight
    assert (slots[:4] == [t[0, 2] * 8 + 6, t[0, 2] * 8 + 7, -1, -1]).all()
    t, g, out, slots = run(7, state=(6, 2))                              # two free blocks, four needed
    want = ref.update_tables(prev, seq, indptr(ql), table, ring, (6, 2), 8, 21)
    assert np.array_equal(t, want[0]) and out == list(want[2]) == [0, 0] and np.array_equal(slots, want[3])
    foreign = ring.copy()
    foreign[6] = 8
    t, _, _, slots = run(3, ring=foreign)                                # an id past the pool
    assert t[0, 2] == -1 and (slots[:2] >= 0).sum() == 0


def test_tables_return_bad_entries_as_minus_one():
    """Table entries outside the pool go back to the ring as -1, flagged, and are dealt as -1; the good
    ones among them keep their places."""
    prev, seq = [40, 24], [10, 0]
    table, ring, state = table_state(prev, 12, 6, 8, head=9)
    table[0, 3], table[1, 1], table[1, 2] = 12, -1, 1 << 30
    d_table, d_ring = i32(table), i32(ring)
    slots, out = mla.update_block_tables(i32(prev), i32(seq), i32([0, 0, 0]), d_table, d_ring, i32(state), 8, 0)
    assert mla.get_device_error() == 3 and out.tolist() == [9, 10]
    want = ring.copy()
    want[(9 + 4 + np.arange(6)) % 12] = [table[0, 2], -1, table[0, 4], table[1, 0], -1, -1]
    assert np.array_equal(d_ring.cpu().numpy(), want) and np.array_equal(d_table.cpu().numpy(), table)
    slots, out = mla.update_block_tables(i32(seq), i32([10, 48]), i32([0, 0, 48]), d_table, d_ring, out, 8, 48)
    assert mla.get_device_error() == 3 and out.tolist() == [3, 4]
    got = d_table.cpu().numpy()
    assert np.array_equal(got[1], [*ring[(9 + np.arange(4)) % 12], table[0, 2], -1])
    assert np.array_equal(slots.cpu().numpy(), np.where(got[1] < 0, -1, got[1] * 8).repeat(8)
                          + np.where(got[1] < 0, 0, 1).repeat(8) * np.tile(np.arange(8), 6))


# ------------------------------------------------------------------ quantising write

def slots_of(L, ql, bs, W, rank, I, seed):
    """Tables of shuffled blocks for requests of L tokens and the new rows' slots."""
    r = np.random.default_rng(seed)
    nb = [-(-ref.local_len(int(n), W, rank, I) // bs) for n in L]
    pool = sum(nb) + 2
    ids, at, slots = r.permutation(pool), 0, []
    for b, n in enumerate(L):
        mine = ids[at:at + nb[b]]
        at += nb[b]
        for g in range(int(n) - int(ql[b]), int(n)):
            owner, j = ref.local_index(g, W, I)
            slots.append(mine[j // bs] * bs + j % bs if owner == rank else -1)
    return np.array(slots, np.int32), pool * bs


def new_rows(T, seed):
    r = np.random.default_rng(seed)
    x = r.standard_normal((T, 576)) * 2.0 ** r.integers(-6, 7, (T, 1))
    return torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)


def check_write(x, slots, rows, G, seed, scales=None):
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (rows, 576)).astype(np.uint8)
    codes[(codes & 127) == 127] = 5
    scales = (2.0 ** r.integers(-9, 4, rows // G)).astype(np.float32) if scales is None else scales
    d_codes, d_scales = torch.tensor(codes).cuda(), torch.tensor(scales).cuda()
    mla.write_kv_scaled(x.cuda(), i32(slots), d_codes, d_scales, G)
    want_c, want_s = ref.write_scaled(x.float().numpy().astype(np.float64), slots, codes, scales, G)
    assert mla.get_device_error() == 0
    assert np.array_equal(d_scales.cpu().numpy().astype(np.float64), want_s)
    diff = (d_codes.cpu().numpy() != want_c).any(1)
    assert not diff.any(), f"{diff.sum()} rows differ, first {np.flatnonzero(diff)[:5]}"
    return d_codes, d_scales


@pytest.mark.parametrize("G,bs,W,rank,I", [
    (1, 16, 1, 0, 1), (2, 8, 2, 1, 1), (4, 4, 1, 0, 1), (8, 8, 3, 2, 4), (16, 16, 1, 0, 1), (16, 32, 4, 3, 1),
    (32, 96, 1, 0, 1), (64, 64, 1, 0, 1), (64, 128, 5, 1, 64), (64, 64, 2, 0, 3)])
def test_write_matches_reference(G, bs, W, rank, I):
    L = np.array([300, 1, 77, 512, 64, 129, 40, 5])
    ql = np.array([4, 1, 77, 200, 64, 3, 0, 5])
    slots, rows = slots_of(L, ql, bs, W, rank, I, G + W)
    check_write(new_rows(len(slots), G), slots, rows, G, G)


@pytest.mark.parametrize("G,T", [(1, 1), (8, 40001), (16, 30000), (64, 20011), (64, 1), (1, 20000)])
def test_write_sizes(G, T):
    """One row, and more rows than there are teams at once."""
    rows = -(-(T + 7) // G) * G
    slots = np.arange(7, T + 7, dtype=np.int32)
    check_write(new_rows(T, 3), slots, rows, G, 3)


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("T", [700, 9000, 40003])
def test_write_of_rows_far_apart(G, T):
    """Rows of one scale block with any number of rows without a slot before, between and behind them: a few
    next to each other, some hundreds or thousands apart, the blocks entered at any offset."""
    r = np.random.default_rng(G + T)
    slots, row, block = np.full(T, -1, np.int32), int(r.integers(0, 300)), 0
    while row < T - 200:
        f = int(r.integers(0, G))
        for i in range(int(r.integers(1, G - f + 1))):
            if row >= T - 200:
                break
            slots[row] = block * G + f + i
            row += 1 + int(r.choice([0, 0, 0, 0, 1, 7, 31, 32, 40, 200, 1500, 5000], p=[.2, .2, .2, .1, .08, .08] + 4 * [.03] + 2 * [.01]))
        block += int(r.integers(1, 3))
    assert (slots >= 0).any()
    check_write(new_rows(T, G), slots, (block + 2) * G, G, G)


@pytest.mark.parametrize("G", [2, 16, 64])
def test_write_of_a_few_rows_in_a_large_capacity(G):
    """A step's few rows in front of a capacity sized for prompts: the call does not look over the rest slot
    by slot (131,072 slots are 512 KB; read 32 at a time, one after another, they take 1.2 ms or more)."""
    T = 131072
    slots = np.full(T, -1, np.int32)
    slots[:9] = [5, 6, 70, 71, 72, 73, 130, 131, 132]
    x = new_rows(1, 1).expand(T, 576).contiguous()
    codes, scales = check_write(x, slots, 192, G, G)
    x, s = x.cuda(), i32(slots)
    best = 1e9
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(10):
            mla.write_kv_scaled(x, s, codes, scales, G)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 100)
    print(f"G = {G}: {best:.1f} us")
    assert best < 300


def test_write_of_a_foreign_scale_divides():
    """Scales that are no powers of two (another writer's) stay where they are larger."""
    slots = np.concatenate([np.arange(3, 9), np.arange(40, 48)]).astype(np.int32)
    scales = np.array([0.3, 1.0, 0.7], np.float32)
    scales[1:] *= 3
    check_write(new_rows(14, 1) / 64, slots, 48, 16, 2, scales)


def test_write_of_zeros_infinities_and_nan():
    x = new_rows(40, 2)
    x[0:16] = 0
    x[16, 5], x[17, 100], x[18, 575], x[30, 0] = math.inf, -math.inf, math.nan, -math.nan
    x[33:40] = 0
    x[33, 1] = 3e38
    x[39, 3] = 1e-38
    slots = np.arange(40, dtype=np.int32)
    codes, scales = check_write(x, slots, 48, 8, 4)
    assert codes[16, 5] == 0x7E and codes[17, 100] == 0xFE and codes[18, 575] == 0x7F
    assert scales[0] == 2.0 ** -100 and scales[4] > 2.0 ** 100


@pytest.mark.parametrize("G", [1, 8, 64])
def test_write_token_by_token_is_the_write_at_once(G):
    """Powers of two: a block filled by single rows ends like one filled at once, but for codes that
    went through the subnormal range (two roundings there; values below 2^-6 of the scale)."""
    x = new_rows(128, 7)
    one = torch.zeros((128, 576), dtype=torch.uint8, device="cuda"), torch.ones(128 // G, device="cuda")
    for t in range(128):
        mla.write_kv_scaled(x[t:t + 1].cuda(), i32([t]), *one, G)
    many = torch.zeros_like(one[0]), torch.ones_like(one[1])
    mla.write_kv_scaled(x.cuda(), i32(np.arange(128)), *many, G)
    assert torch.equal(one[1], many[1])
    a, b = (torch.tensor(ref.CODE_VALUE[c.cpu().numpy()]) for c in (one[0], many[0]))
    normal = b.abs() >= 2.0 ** -6
    assert torch.equal(a[normal], b[normal])
    # a second rounding moves a subnormal by one step of 2^-9 at most
    assert (a - b).abs().max() <= 2.0 ** -9


def test_write_bad_slots_are_skipped():
    x = new_rows(6, 5)
    codes, scales = torch.zeros((32, 576), dtype=torch.uint8, device="cuda"), torch.ones(2, device="cuda")
    mla.write_kv_scaled(x.cuda(), i32([3, 32, -2, 4, -1, 1 << 30]), codes, scales, 16)
    assert mla.get_device_error() == 3
    assert (codes.cpu().numpy().any(1) == np.isin(np.arange(32), [3, 4])).all()


@pytest.mark.parametrize("G,slots,good", [
    (16, [3, 5, 6, 40], 1), (16, [3, 4, 4, 5, 40], 2), (16, [7, 6, 40], 1), (16, [3, -1, 4, -1, 6, 7, 40], 3),
    (2, [4, 4, 40], 1), (4, [5, 7, 40], 1), (64, [3, 4, 5, 7, 8, 70], 3), (8, [1, 2, 3, 0, 40], 3),
    (64, [9] + 300 * [-1] + [10, 12, 70], 302), (4, [4] + 50 * [-1] + [5, 7, 40], 52)])
def test_write_of_rows_out_of_order_is_refused(G, slots, good):
    """A row that is not the next one of its scale block: the block's rows before it are written, it and the
    rest are not, and the next block is; nothing goes to a row that the map does not name."""
    x = new_rows(len(slots), G)
    codes = np.full((128, 576), 3, np.uint8)
    scales = np.ones(128 // G, np.float32)
    d = torch.tensor(codes).cuda(), torch.tensor(scales).cuda()
    mla.write_kv_scaled(x.cuda(), i32(slots), *d, G)
    assert mla.get_device_error() == 3
    kept = np.array(slots)
    kept[good:-1] = -1
    want_c, want_s = ref.write_scaled(x.float().numpy().astype(np.float64), kept, codes, scales, G)
    assert np.array_equal(d[0].cpu().numpy(), want_c) and np.array_equal(d[1].cpu().numpy().astype(np.float64), want_s)


# ------------------------------------------------------------------ attention

def attention_inputs(L, ql, H, bs, G, seed, mag=0.7, views=1):
    """q, codes, scales, tables and lengths; views > 1 repeats the row plan with other lengths."""
    g = torch.Generator().manual_seed(seed)
    r = np.random.default_rng(seed)
    P = min(128, bs & -bs)
    nb = [max(1, -(-int(n) // bs)) for n in L]
    pool = sum(nb) * views + 2
    ids = r.permutation(pool)
    codes = (torch.randn((pool * bs, 576), generator=g) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    scales = torch.exp2(torch.round(mag * torch.randn(pool * bs // G, generator=g)) - 6)
    T = int(np.sum(ql))
    q = torch.randn((T, H, 576), generator=g).to(torch.bfloat16)
    width = max(-(-int(n) // P) for n in L) + 1
    sub = np.full((views, len(L), width), -1, np.int32)
    row_len = np.zeros((views, T), np.int32)
    ind, at = indptr(ql), 0
    for v in range(views):
        for b, n in enumerate(L):
            mine = ids[at:at + nb[b]]
            at += nb[b]
            n = max(int(n) - 37 * v, 0)
            for p in range(-(-n // P)):
                sub[v, b, p] = mine[p * P // bs] * (bs // P) + p % (bs // P)
            for t in range(int(ql[b])):
                row_len[v, ind[b] + t] = max(n - int(ql[b]) + t + 1, 0)
    return q, codes.view(torch.uint8), scales, ind, row_len, sub, P


def run_attention(q, codes, scales, G, ind, row_len, sub, P, S, qmax, **kw):
    V = row_len.shape[0]
    kw.update(num_views=V)
    squeeze = (lambda a: a[0]) if V == 1 else (lambda a: a)
    out, lse, ws = mla.decode_verify_scaled(q.cuda(), codes.cuda(), scales.cuda(), G, i32(ind), i32(squeeze(row_len)),
                                            i32(squeeze(sub)), P, S, qmax, SM, **kw)
    return out, lse, ws


def check_rows(out, lse, args, G, nan_rows=None):
    q, codes, scales, ind, row_len, sub, P = args
    V, T = row_len.shape
    out = out.float().cpu().numpy().reshape(V, T, q.shape[1], 512)
    lse = lse.cpu().numpy().reshape(V, T, q.shape[1])
    worst = 0.0
    for v in range(V):
        o, l, mass, far = ref.attention(q.double().numpy(), codes.numpy(), scales.numpy(), G, ind, row_len[v],
                                        sub[v], P, SM)
        if nan_rows is not None:
            assert np.array_equal(np.isnan(out[v]).any(2), nan_rows), "rows that see a NaN"
            assert np.array_equal(np.isnan(lse[v]), nan_rows)
            o, l, mass, far, out_v, lse_v = (np.where(nan_rows[..., None] if a.ndim == 3 else nan_rows, 0, a)
                                             for a in (o, l, mass, far, out[v], lse[v]))
        else:
            out_v, lse_v = out[v], lse[v]
        empty = np.isneginf(l)
        assert np.array_equal(np.isneginf(lse_v), empty) and not out_v[empty].any()
        assert np.abs(np.where(empty, 0, lse_v) - np.where(empty, 0, l)).max() <= LSE_TOL
        err = np.abs(out_v - o)
        over = (err / ref.out_bound(o, mass, far)).max()
        assert over <= 1, f"{over:.3g} times the bound"
        top = np.abs(o).max(2)
        worst = max(worst, (err.max(2) / np.maximum(top, 1e-30))[top > 0].max(initial=0.0))
    return worst


@pytest.mark.parametrize("bs,G", [(8, 1), (8, 8), (16, 16), (32, 4), (96, 32), (64, 64), (128, 64), (256, 2)])
@pytest.mark.parametrize("S", [1, 5])
def test_attention_pages_and_scale_blocks(bs, G, S):
    L = np.array([1, 700, 95, 96, 97, 33, 260])
    ql = np.array([1, 3, 2, 4, 1, 4, 2])
    args = attention_inputs(L, ql, 16, bs, G, bs + S)
    out, lse, _ = run_attention(*args[:3], G, *args[3:], S, 4)
    assert mla.get_device_error() == 0
    assert check_rows(out, lse, args, G) <= 1e-2


@pytest.mark.parametrize("H,qmax", [(1, 1), (1, 8), (3, 5), (12, 3), (16, 8), (33, 1), (64, 2), (128, 3)])
def test_attention_heads_and_rows(H, qmax):
    """From one row to seven row blocks per request, rows not a multiple of anything."""
    L = np.array([400, 131, 64, 9])
    ql = np.minimum(L, [qmax, 1, qmax, max(1, qmax - 1)])
    args = attention_inputs(L, ql, H, 32, 16, H)
    out, lse, _ = run_attention(*args[:3], 16, *args[3:], 3, qmax)
    assert mla.get_device_error() == 0
    assert check_rows(out, lse, args, 16) <= 1e-2


@pytest.mark.parametrize("S", [1, 2, 16, 300])
def test_attention_long_and_short_together(S):
    """Requests from one token to 20,000, more requests than one pass over them takes, any split."""
    r = np.random.default_rng(S)
    L = np.concatenate([[20000, 1, 5000, 2], r.integers(1, 200, 400)])
    ql = np.minimum(L, r.integers(1, 3, len(L)))
    args = attention_inputs(L, ql, 4, 16, 8, 40 + S)
    out, lse, _ = run_attention(*args[:3], 8, *args[3:], S, 2)
    assert mla.get_device_error() == 0
    assert check_rows(out, lse, args, 8) <= 1e-2


@pytest.mark.parametrize("S", [1, 4])
def test_attention_views_and_empty_rows(S):
    """Three row views in one launch; short requests lose every token in the later ones, a padded row
    capacity leaves the rows behind the last request as they were."""
    L, ql = np.array([300, 40, 74, 1, 500]), np.array([4, 4, 2, 1, 3])
    args = list(attention_inputs(L, ql, 12, 16, 16, 3, views=3))
    assert (args[4] == 0).any() and (args[4][2] > 0).any()
    pad = 3
    q = torch.cat([args[0], torch.full((pad, 12, 576), float("nan"), dtype=torch.bfloat16)])
    T = q.shape[0]
    row_len = np.concatenate([args[4], np.full((3, pad), 9, np.int32)], 1)
    out = torch.full((3, T, 12, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, T, 12), 7.0, device="cuda")
    run_attention(q, args[1], args[2], 16, args[3], row_len, *args[5:], S, 4, out=out, lse=lse)
    assert mla.get_device_error() == 0
    assert (out[:, T - pad:] == 7).all() and (lse[:, T - pad:] == 7).all()
    assert check_rows(out[:, :T - pad], lse[:, :T - pad], args, 16) <= 1e-2


def test_attention_only_empty_rows():
    L, ql = np.array([3, 2]), np.array([3, 2])
    args = list(attention_inputs(L, ql, 16, 16, 16, 5))
    args[4][:] = 0
    for S in (1, 4):
        out, lse, _ = run_attention(*args[:3], 16, *args[3:], S, 3)
        assert not out.any() and torch.isneginf(lse).all()
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("S", [1, 6])
def test_attention_scales_far_apart(S):
    """Neighbouring scale blocks differ by up to 2^40 either way, with scores kept moderate by a
    small softmax scale elsewhere: no overflow, no lost block."""
    L, ql = np.array([900, 350]), np.array([2, 1])
    args = list(attention_inputs(L, ql, 16, 64, 16, 8))
    r = np.random.default_rng(1)
    args[2] = torch.tensor(2.0 ** r.integers(-45, -5, len(args[2])) * 1.37, dtype=torch.float32)
    args[2][3] = 1e-38   # counts as 2^-100
    args[2][4] = 0.0
    out, lse, _ = run_attention(*args[:3], 16, *args[3:], S, 2)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 16)


def test_attention_queries_of_every_magnitude():
    """Query rows from 2^-60 to 2^30 of each other in one row block, zeros and single large elements."""
    L, ql = np.array([500, 120]), np.array([4, 2])
    args = list(attention_inputs(L, ql, 16, 64, 64, 9))
    q = args[0].float()
    q *= torch.exp2(torch.linspace(-60, 1, q.shape[1]))[None, :, None]
    q[0, 3] = 0
    q[1, 4, :] = 0
    q[1, 4, 77] = 30.0
    q[2, 5, 570] = -20.0
    args[0] = q.to(torch.bfloat16)
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], 3, 4)
    assert mla.get_device_error() == 0
    assert check_rows(out, lse, args, 64) <= 1e-2


@pytest.mark.parametrize("S", [1, 3])
def test_attention_nan_stays_with_its_rows(S):
    """A NaN code reaches exactly the rows that see its token (here the last token, which only the last
    verify row sees, and one in another request's masked tail); a NaN query spoils its own rows only."""
    L, ql = np.array([200, 333, 150, 100]), np.array([4, 3, 2, 1])
    args = list(attention_inputs(L, ql, 16, 16, 16, 11))
    codes, sub, P = args[1], args[5][0], args[6]
    at = lambda b, j: int(sub[b, j // P]) * P + j % P
    codes[at(0, 199), 300] = 0x7F      # a latent value of request 0's last token
    codes[at(1, 331), 570] = 0xFF      # a rope value of request 1's last but one
    args[0][7, 2, 10] = float("nan")   # one head of request 2's first row
    args[0][8, 3, 10] = float("inf")
    # stale rows past request 3's end, in its last page
    for j in range(100, 112):
        codes[at(3, j)] = 0x7F
    nan_rows = np.zeros((10, 16), bool)
    nan_rows[3], nan_rows[5], nan_rows[6] = True, True, True
    nan_rows[7, 2] = nan_rows[8, 3] = True
    out, lse, _ = run_attention(*args[:3], 16, *args[3:], S, 4)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 16, nan_rows)


@pytest.mark.parametrize("H,S", [(64, 1), (64, 4), (128, 1), (128, 3), (24, 2)])
def test_attention_nan_of_a_later_draft(H, S):
    """A NaN code in the last drafts' tokens, with row blocks whose rows all end before them."""
    L, ql = np.array([300, 97, 193]), np.array([6, 3, 4])
    args = list(attention_inputs(L, ql, H, 32, 32, 17 + H))
    codes, sub, P = args[1], args[5][0], args[6]
    at = lambda b, j: int(sub[b, j // P]) * P + j % P
    codes[at(0, 298), 3] = 0x7F
    codes[at(1, 96), 511] = 0xFF       # the only token of a tile
    codes[at(2, 191), 575] = 0x7F      # rope, the last token of a tile
    nan_rows = np.zeros((13, H), bool)
    nan_rows[[4, 5, 8, 11, 12]] = True
    out, lse, _ = run_attention(*args[:3], 32, *args[3:], S, 6)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 32, nan_rows)


@pytest.mark.parametrize("S", [1, 4])
def test_attention_scores_beyond_float32_spoil_their_row_only(S):
    """A query of +-3e38, whose scores have no float32 value, beside ordinary ones in its row block."""
    L, ql = np.array([400, 130]), np.array([3, 1])
    args = list(attention_inputs(L, ql, 16, 16, 16, 18))
    args[2] = torch.ones_like(args[2])
    sign = torch.where(torch.randn(576, generator=torch.Generator().manual_seed(3)) < 0, -1.0, 1.0)
    args[0][1, 5] = (3e38 * sign).to(torch.bfloat16)
    args[0][:, :5] *= 0.02
    args[0][:, 6:] *= 0.02
    nan_rows = np.zeros((4, 16), bool)
    nan_rows[1, 5] = True
    out, lse, _ = run_attention(*args[:3], 16, *args[3:], S, 3)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 16, nan_rows)


@pytest.mark.parametrize("B", [2, 500])
def test_attention_queries_off_a_32_byte_boundary(B):
    """Few row blocks (the first of a CTA each) and many (several per CTA, read another way)."""
    r = np.random.default_rng(B)
    L, ql = (np.array([260, 500]), np.array([3, 5])) if B == 2 else (r.integers(5, 110, B), r.integers(1, 6, B))
    args = attention_inputs(L, ql, 20, 32, 16, 19)
    first = run_attention(*args[:3], 16, *args[3:], 3, 5)
    room = torch.empty(args[0].numel() + 8, dtype=torch.bfloat16, device="cuda")
    q = room[8:].view(args[0].shape)
    q.copy_(args[0])
    assert q.data_ptr() % 32 == 16
    out, lse, _ = mla.decode_verify_scaled(q, args[1].cuda(), args[2].cuda(), 16, i32(args[3]), i32(args[4][0]),
                                           i32(args[5][0]), args[6], 3, 5, SM)
    assert mla.get_device_error() == 0
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    check_rows(out, lse, args, 16)


@pytest.mark.parametrize("H,rows,S", [(16, 2, 1), (16, 2, 3), (32, 2, 3), (20, 1, 1)])
def test_attention_of_many_parts_per_cta_repeats_itself(H, rows, S):
    """Many parts in every CTA, of one tile or three, so that either softmax group starts a part while the
    other may still read the outputs of the one before; with up to 32 rows the second group has none to read.
    Every launch gives the same bits, and the first is checked."""
    r = np.random.default_rng(7 * H + S)
    B = 1400
    L = np.where(r.random(B) < 0.5, r.integers(rows, 97, B), r.integers(193, 289, B))
    args = attention_inputs(L, np.full(B, rows), H, 32, 16, H + S)
    dev = [t.cuda() for t in args[:3]] + [i32(args[3]), i32(args[4][0]), i32(args[5][0])]
    call = lambda **kw: mla.decode_verify_scaled(*dev[:3], 16, *dev[3:], args[6], S, rows, SM, **kw)
    first, lse, ws = call()
    check_rows(first, lse, args, 16)
    out, l2 = torch.empty_like(first), torch.empty_like(lse)
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for _ in range(400):
        out.fill_(7.0)
        call(out=out, lse=l2, workspace=ws)
        same &= (out.view(torch.int16) == first.view(torch.int16)).all() & (l2 == lse).all()
    assert mla.get_device_error() == 0 and same.item()


@pytest.mark.parametrize("G", [4, 64])
def test_cache_past_32_bit_offsets(G):
    """Rows on both sides of byte 2^32 of the codes: written through the slot map, then read."""
    bs, L, H = 64, 900, 16
    edge = (1 << 32) // 576 // bs      # the block that byte 2^32 lies in
    blocks = edge + 10
    codes = torch.zeros((blocks * bs, 576), dtype=torch.uint8, device="cuda")
    scales = torch.ones(blocks * bs // G, device="cuda")
    mine = np.array([edge - 3, blocks - 1, edge, 0, edge + 1, 5, edge - 1, edge + 3, edge + 7, 1, edge + 2, 9, edge + 5,
                     2, edge + 4])
    j = np.arange(L)
    slots = mine[j // bs] * bs + j % bs
    x = new_rows(L, G)
    mla.write_kv_scaled(x.cuda(), i32(slots), codes, scales, G)
    small_c, small_s = ref.write_scaled(x.double().numpy(), j, np.zeros((15 * bs, 576), np.uint8),
                                        np.ones(15 * bs // G), G)
    pick = torch.as_tensor(mine).cuda()
    assert np.array_equal(codes.view(blocks, bs, 576)[pick].view(-1, 576).cpu().numpy(), small_c)
    assert np.array_equal(scales.view(blocks, bs // G)[pick].view(-1).cpu().numpy(), small_s)
    g = torch.Generator().manual_seed(4)
    q = (torch.randn((2, H, 576), generator=g) * 0.05).to(torch.bfloat16)
    ind, row_len = np.array([0, 2]), np.array([[L - 1, L]], np.int32)
    out, lse, _ = mla.decode_verify_scaled(q.cuda(), codes, scales, G, i32(ind), i32(row_len[0]),
                                           i32(mine[None]), bs, 4, 2, SM)
    assert mla.get_device_error() == 0
    args = (q, torch.tensor(small_c), torch.tensor(small_s, dtype=torch.float32), ind, row_len,
            np.arange(15, dtype=np.int32)[None, None], bs)
    check_rows(out, lse, args, G)


def test_attention_outliers():
    """Peaked rows (one token holds almost everything), flat rows, and a row of a hundred far tokens
    under one large one: probabilities keep their relative precision."""
    L, ql = np.array([2000, 2000]), np.array([1, 1])
    args = list(attention_inputs(L, ql, 8, 64, 64, 12, mag=0.0))
    q = args[0].float()
    q[:, :2] *= 8.0
    q[:, 2:4] *= 0.001
    args[0] = q.to(torch.bfloat16)
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], 4, 1)
    assert check_rows(out, lse, args, 64) <= 1e-2
    # a sink: token 0 scores about 2^18 times any other's weight, and 60,000 others share the rest
    n = 60000
    codes = torch.zeros((n, 576), dtype=torch.float32)
    codes[:, 5] = 1.0
    codes[0, 0] = 16.0
    codes[0, 5] = -1.0
    q = torch.zeros((1, 1, 576))
    q[0, 0, 0] = 11.0
    sub = np.arange(n // 32, dtype=np.int32)[None, None]
    args = (q.to(torch.bfloat16), codes.to(torch.float8_e4m3fn).view(torch.uint8), torch.ones(n // 32),
            np.array([0, 1]), np.array([[n]], np.int32), sub, 32)
    for S in (1, 16):
        out, lse, _ = run_attention(*args[:3], 32, *args[3:], S, 1)
        assert check_rows(out, lse, args, 32) <= 1e-2


@pytest.mark.parametrize("S", [1, 4])
def test_attention_wait_timeout_then_a_correct_call(S):
    """A wait budget of 1000 cycles makes the CTAs give up without a hang; the next call is correct."""
    L, ql = np.array([2500, 3100, 1800]), np.array([4, 4, 2])
    args = attention_inputs(L, ql, 16, 64, 64, 16)
    for _ in range(2):
        run_attention(*args[:3], 64, *args[3:], S, 4, wait_cycles=1000)
        assert mla.get_device_error() == 6
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], S, 4)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 64)


def test_attention_device_checks():
    """A page outside the cache is read as zeros, a row past the bound is clipped; both recorded."""
    L, ql = np.array([300, 90]), np.array([2, 1])
    args = list(attention_inputs(L, ql, 16, 64, 64, 14))
    sub = args[5].copy()
    sub[0, 0, 1] = 1 << 24
    args[5] = sub
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], 3, 2)
    assert mla.get_device_error() == 5 and mla.get_device_error() == 0
    pool = args[1].shape[0]
    zero = sub.copy()
    zero[0, 0, 1] = pool // 64
    args[1] = torch.cat([args[1], torch.zeros((64, 576), dtype=torch.uint8)])
    args[2] = torch.cat([args[2], torch.ones(1)])
    args[5] = zero
    check_rows(out, lse, args, 64)
    args = list(attention_inputs(L, ql, 16, 64, 64, 14))
    args[5] = np.ascontiguousarray(args[5][:, :, :2])
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], 3, 2)
    assert mla.get_device_error() == 4
    args[4] = np.minimum(args[4], 128)
    check_rows(out, lse, args, 64)


def test_attention_inconsistent_rows_are_refused_on_the_device():
    L, ql = np.array([300, 90]), np.array([2, 1])
    args = attention_inputs(L, ql, 16, 64, 64, 15)
    bad = np.array([0, 4, 3])
    for S in (1, 4):
        run_attention(*args[:3], 64, bad, *args[4:], S, 2)
        assert mla.get_device_error() == 1
    out, lse, _ = run_attention(*args[:3], 64, *args[3:], 4, 2)
    assert mla.get_device_error() == 0
    check_rows(out, lse, args, 64)


# ------------------------------------------------------------------ together

def serve(cache, step, q, x, seq, ind, bt):
    cache.append(x, seq, ind)
    return step(q, cache.codes, seq, ind, bt, SM, kv_scales=cache.scales)


@pytest.mark.parametrize("W,graph", [(1, False), (1, True), (3, False)])
def test_serving_steps(W, graph):
    """Prompts, then speculative steps with drafts taken back, a request finished and its place
    given to a new one: tables, slots, codes, scales and outputs after every step.  Captured once
    and replayed with new lengths, and for three shards whose states are merged."""
    bs, G, H, B, T = 16, 8, 4, 3, 96
    caches = [runner.PagedLatentCache(num_reqs=B, num_rows=T, num_blocks=40, block_size=bs, max_kv_len=320,
                                      scale_block=G, world_size=W, rank=r) for r in range(W)]
    steps = [runner.VerifyStep(num_reqs=B, num_rows=T, num_heads=H, max_qlen=T, block_size=bs, num_blocks=40,
                               block_table_width=20, max_kv_len=320, num_segments=4, scale_block=G) for _ in range(W)]
    q, x = (torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in ((T, H, 576), (T, 576)))
    seq, ind = i32(np.zeros(B)), i32(np.zeros(B + 1))
    history = [np.zeros((0, 576)) for _ in range(B)]
    model = [dict(table=c.block_table.cpu().numpy(), ring=c.free_ring.cpu().numpy(), state=(0, 40),
                  codes=c.codes.cpu().numpy(), scales=c.scales.cpu().numpy()) for c in caches]
    prev = np.zeros(B, np.int64)
    g = None
    plan = [([50, 3, 30], [50, 3, 30]), ([53, 7, 34], [4, 4, 4]), ([55, 8, 36], [4, 2, 3]), ([57, 1, 60], [3, 1, 60]),
            ([61, 5, 62], [4, 4, 2])]
    for n, (L, ql) in enumerate(plan):
        rng = np.random.default_rng(n)
        rows = indptr(ql)
        xs, qs = new_rows(T, n), torch.tensor(rng.standard_normal((T, H, 576)), dtype=torch.float32).to(torch.bfloat16)
        x.copy_(xs), q.copy_(qs), seq.copy_(i32(L)), ind.copy_(i32(rows))
        if W == 1:
            if graph and g is None and n == 1:
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g):
                    res = serve(caches[0], steps[0], q, x, seq, ind, caches[0].block_table[None])
            if g is not None:
                g.replay()
            else:
                res = serve(caches[0], steps[0], q, x, seq, ind, caches[0].block_table[None])
            out, lse = res
        else:
            lens = mla.plan_rows(seq, ind, T)[0]
            parts = []
            for r in range(W):
                caches[r].append(x, seq, ind)
                local, sub = mla.shard_row_view(ind, lens, W, r, 1, caches[r].block_table, 40, bs, 20)
                parts.append(mla.decode_verify_scaled(q, caches[r].codes, caches[r].scales, G, ind, local, sub, bs,
                                                      4, T, SM)[:2])
            out, lse = mla.merge_states(*(torch.stack(p) for p in zip(*parts)))
        assert mla.get_device_error() == 0
        for r, m in enumerate(model):
            m["table"], m["ring"], m["state"], slots = ref.update_tables(prev, L, rows, m["table"], m["ring"],
                                                                         m["state"], bs, T, W, r)
            m["codes"], m["scales"] = ref.write_scaled(xs.double().numpy(), slots, m["codes"], m["scales"], G)
            c = caches[r]
            assert np.array_equal(c.block_table.cpu().numpy(), m["table"])
            assert np.array_equal(c.free_ring.cpu().numpy(), m["ring"]) and tuple(c.ring.tolist()) == m["state"]
            assert np.array_equal(c.slot_map.cpu().numpy(), slots)
            assert np.array_equal(c.codes.cpu().numpy(), m["codes"])
            assert np.array_equal(c.scales.cpu().numpy().astype(np.float64), m["scales"])
        prev = np.array(L)
        # every shard's tokens gathered into one cache, request after request
        table = np.full((B, 320), -1, np.int32)
        flat = np.zeros((B * 320, 576), np.uint8)
        scl = np.ones(B * 320)
        for b in range(B):
            for pos in range(L[b]):
                r, j = ref.local_index(pos, W, 1)
                s = model[r]["table"][b, j // bs] * bs + j % bs
                flat[b * 320 + pos], scl[b * 320 + pos] = model[r]["codes"][s], model[r]["scales"][s // G]
                table[b, pos] = b * 320 + pos
        row_len = np.zeros(T, np.int64)
        for b in range(B):
            row_len[rows[b]:rows[b + 1]] = np.arange(L[b] - ql[b] + 1, L[b] + 1)
        n_rows = rows[-1]
        o, l, mass, far = ref.attention(qs.double().numpy()[:n_rows], flat, scl, 1, rows, row_len, table, 1, SM)
        err = np.abs(out.float().cpu().numpy()[:n_rows] - o)
        # one more rounding of each shard's state to bf16 when states are merged
        assert (err <= ref.out_bound(o, mass, far) + (W > 1) * 2.0 ** -8 * mass).all()
        assert np.abs(lse.cpu().numpy()[:n_rows] - l).max() <= LSE_TOL


@pytest.mark.parametrize("S", [1, 4])
def test_verify_step_with_a_finished_request(S):
    """A request that was finished keeps its place in the batch without tokens or rows: the plan records it
    (MLA_DEV_BAD_QLEN), and the others' rows are what they are without it.  On a stream that is not the
    current one."""
    cfg = dict(num_rows=24, block_size=16, num_blocks=40, max_kv_len=320)
    s = torch.cuda.Stream()
    x, q = new_rows(24, 5).cuda(), torch.randn((24, 8, 576), generator=torch.Generator().manual_seed(1)).cuda()
    q = q.to(torch.bfloat16)
    outs = []
    for L, ql in ((([9, 12, 0, 3]), [9, 12, 0, 3]), ([9, 12, 3], [9, 12, 3])):
        B = len(L)
        c = runner.PagedLatentCache(num_reqs=B, scale_block=8, **cfg)
        step = runner.VerifyStep(num_reqs=B, num_heads=8, max_qlen=12, block_table_width=20, num_segments=S,
                                 scale_block=8, **cfg)
        seq, ind = i32(L), i32(indptr(ql))
        s.wait_stream(torch.cuda.current_stream())
        c.append(x, seq, ind, stream=s)
        out, lse = step(q, c.codes, seq, ind, c.block_table[None], SM, kv_scales=c.scales, stream=s)
        s.synchronize()
        assert mla.get_device_error() == (2 if 0 in L else 0)
        outs.append((out.clone(), lse.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("W,I,S", [(3, 1, 4), (2, 4, 1), (8, 1, 16)])
def test_verify_step_over_shard_views(W, I, S):
    """VerifyStep with every shard's view in one launch of the block-scaled decode, requests too short for
    some shards among them: the merged states against the whole sequences."""
    bs, G, H, L, ql = 32, 16, 8, np.array([700, 5, 131, 1]), np.array([4, 3, 2, 1])
    B, T, width = len(L), int(ql.sum()) + 2, 24
    g = torch.Generator().manual_seed(W)
    table = np.random.default_rng(W).permutation(W * B * width).astype(np.int32).reshape(W, B, width)
    pool = table.size
    codes = (torch.randn((pool * bs, 576), generator=g) * 100).clamp_(-448, 448).to(torch.float8_e4m3fn)
    codes = codes.view(torch.uint8)
    scales = torch.exp2(torch.round(torch.randn(pool * bs // G, generator=g)) - 6) * 1.25
    q = torch.randn((T, H, 576), generator=g).to(torch.bfloat16)
    ind = indptr(ql)
    step = runner.VerifyStep(num_reqs=B, num_rows=T, num_heads=H, max_qlen=4, block_size=bs, num_blocks=pool,
                             block_table_width=width, max_kv_len=700, num_segments=S, world_size=W, interleave=I,
                             scale_block=G)
    dev = q.cuda(), codes.cuda(), i32(L), i32(ind), i32(table), scales.cuda()
    out, lse = step(*dev[:5], SM, kv_scales=dev[5])
    assert mla.get_device_error() == 0
    n, flat = int(ql.sum()), np.full((B, int(L.max())), -1, np.int64)
    for b in range(B):
        for pos in range(L[b]):
            r, j = ref.local_index(pos, W, I)
            flat[b, pos] = table[r, b, j // bs] * bs + j % bs
    row_len = np.concatenate([np.arange(L[b] - ql[b] + 1, L[b] + 1) for b in range(B)])
    row_scale = scales.numpy().repeat(G)
    o, l, mass, far = ref.attention(q[:n].double().numpy(), codes.numpy(), row_scale, 1, ind, row_len, flat, 1, SM)
    err = np.abs(out[:n].float().cpu().numpy() - o)
    # one more rounding of each shard's state to bf16 when states are merged
    assert (err <= ref.out_bound(o, mass, far) + 2.0 ** -8 * mass).all()
    assert np.abs(lse[:n].cpu().numpy() - l).max() <= LSE_TOL


def test_append_that_ran_out_of_blocks_is_undone():
    """Too few free blocks: the error, blocks and lengths back as before, then a smaller step, and every
    block returned in the end.  A refused call changes nothing either."""
    c = runner.PagedLatentCache(num_reqs=2, num_rows=64, num_blocks=6, block_size=16, max_kv_len=96, scale_block=16)
    x = new_rows(64, 1).cuda()
    c.append(x, i32([40, 10]), i32([0, 40, 50]))
    held = c.block_table.clone(), c.ring.clone(), c.lens.clone()
    codes = c.codes.clone()
    assert mla.get_device_error() == 0 and held[1].tolist() == [4, 2]
    c.append(x, i32([70, 40]), i32([0, 30, 60]))
    assert mla.get_device_error() == 7
    c.undo()
    assert torch.equal(c.ring, held[1]) and torch.equal(c.lens, held[2])
    for bad in (lambda: c.append(x.float(), i32([41, 10]), i32([0, 1, 1])),
                lambda: c.append(x, i32([41, 10]).float(), i32([0, 1, 1])),
                lambda: c.append(x, i32([41]), i32([0, 1]))):
        with pytest.raises((TypeError, ValueError)):
            bad()
        assert torch.equal(c.ring, held[1]) and torch.equal(c.lens, held[2])
    slots = c.append(x, i32([41, 40]), i32([0, 1, 31])).cpu().numpy()
    assert mla.get_device_error() == 0 and c.ring.tolist() == [0, 0]
    table = c.block_table.cpu().numpy()
    assert slots[0] == table[0, 2] * 16 + 8 and (slots[31:] == -1).all()
    assert list(slots[1:31]) == [table[1, n // 16] * 16 + n % 16 for n in range(10, 40)]
    for b, n in ((0, 40), (1, 10)):   # the tokens before are where they were
        at = held[0][b].cpu().numpy()[np.arange(n) // 16] * 16 + np.arange(n) % 16
        assert np.array_equal(table[b, :-(-n // 16)], held[0][b, :-(-n // 16)].cpu().numpy())
        whole = torch.as_tensor(at[:n // 16 * 16]).cuda()
        assert torch.equal(c.codes[whole], codes[whole])
    c.append(x, i32([0, 0]), i32([0, 0, 0]))
    assert mla.get_device_error() == 0 and c.ring[1].item() == 6
    assert sorted(c.free_ring.tolist()) == list(range(6))


@pytest.mark.parametrize("graph", [False, True])
def test_append_that_the_tables_refuse_changes_nothing(graph):
    """An inconsistent qo_indptr, then a ring state outside the pool: lengths, blocks and codes as before,
    and the next step is dealt as if the refused one had not been."""
    c = runner.PagedLatentCache(num_reqs=3, num_rows=64, num_blocks=12, block_size=16, max_kv_len=96, scale_block=16)
    x, seq, ind = new_rows(64, 1).cuda(), i32([40, 10, 14]), i32([0, 40, 50, 64])
    g = None

    def step(L, rows):
        nonlocal g
        seq.copy_(i32(L)), ind.copy_(i32(rows))
        if graph and g is None:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                c.append(x, seq, ind)
        g.replay() if graph else c.append(x, seq, ind)
        return mla.get_device_error()

    assert step([40, 10, 14], [0, 40, 50, 64]) == 0
    keep = lambda: [t.clone() for t in (c.ring, c.lens, c.block_table, c.free_ring, c.codes, c.scales)]
    same = lambda a: all(torch.equal(u, v) for u, v in zip(a, keep()))
    before = keep()
    assert before[1].tolist() == [40, 10, 14]
    for bad in ([0, 30, 20, 44], [1, 30, 40, 44], [0, 30, 40, 65]):
        assert step([70, 40, 30], bad) == 1 and same(before) and (c.slot_map == -1).all()
    count = int(c.ring[1])
    c.ring[1] = 13
    assert step([70, 40, 30], [0, 30, 40, 44]) == 8 and c.lens.tolist() == [40, 10, 14]
    c.ring[1] = count
    assert same(before)
    m = ref.update_tables([40, 10, 14], [42, 0, 33], [0, 2, 2, 21], before[2].cpu().numpy(), before[3].cpu().numpy(),
                          tuple(before[0].tolist()), 16, 64)
    assert step([42, 0, 33], [0, 2, 2, 21]) == 0
    assert np.array_equal(c.block_table.cpu().numpy(), m[0]) and np.array_equal(c.free_ring.cpu().numpy(), m[1])
    assert tuple(c.ring.tolist()) == m[2] and np.array_equal(c.slot_map.cpu().numpy(), m[3])
    assert c.lens.tolist() == [42, 0, 33]


def test_append_with_the_caches_own_lengths_and_a_negative_one():
    """The cache's own lens as the new lengths (nothing changes); a negative length counts as 0, flagged."""
    c = runner.PagedLatentCache(num_reqs=2, num_rows=32, num_blocks=6, block_size=16, max_kv_len=48, scale_block=16)
    x = new_rows(32, 1).cuda()
    c.append(x, i32([20, 10]), i32([0, 20, 30]))
    state = c.ring.tolist(), c.block_table.clone()
    c.append(x, c.lens, i32([0, 0, 0]))
    assert mla.get_device_error() == 0
    assert c.lens.tolist() == [20, 10] and c.ring.tolist() == state[0] and torch.equal(c.block_table, state[1])
    c.append(x, i32([-5, 10]), i32([0, 0, 0]))
    assert mla.get_device_error() == 2 and c.lens.tolist() == [0, 10] and c.ring[1].item() == 5
    c.append(x, i32([0, 10]), i32([0, 0, 0]))
    assert mla.get_device_error() == 0 and c.ring[1].item() == 5


def test_two_streams_and_two_graphs_at_once():
    """Two captured graphs with a workspace each, replayed on two streams together, and an eager call
    on a third: the same outputs as alone."""
    L, ql = np.array([5000, 3000, 700]), np.array([4, 4, 4])
    runs = []
    for seed in (21, 22, 23):
        args = attention_inputs(L, ql, 16, 64, 64, seed)
        dev = [a.cuda() for a in args[:3]], i32(args[3]), i32(args[4][0]), i32(args[5][0])
        alone, lse, ws = mla.decode_verify_scaled(dev[0][0], dev[0][1], dev[0][2], 64, *dev[1:], 64, 8, 4, SM)
        runs.append((dev, alone.clone(), lse.clone(), torch.empty_like(ws), torch.empty_like(alone),
                     torch.empty_like(lse)))
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream() for _ in range(3)]
    call = lambda r: mla.decode_verify_scaled(r[0][0][0], r[0][0][1], r[0][0][2], 64, *r[0][1:], 64, 8, 4, SM, out=r[4],
                                              lse=r[5], workspace=r[3])
    for r in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(r)
        graphs.append(g)
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        with torch.cuda.stream(streams[2]):
            call(runs[2])
    torch.cuda.synchronize()
    assert mla.get_device_error() == 0
    for r in runs:
        assert torch.equal(r[4], r[1]) and torch.equal(r[5], r[2])


def test_binding_refusals():
    cache, scales = torch.zeros((64, 576), dtype=torch.uint8, device="cuda"), torch.ones(4, device="cuda")
    x, slots = torch.zeros((2, 576), dtype=torch.bfloat16, device="cuda"), i32([0, 1])
    for call in (lambda: mla.write_kv_scaled(x, slots[:1], cache, scales, 16),
                 lambda: mla.write_kv_scaled(x[:, :512], slots, cache, scales, 16),
                 lambda: mla.write_kv_scaled(x, slots, cache, scales, 32),
                 lambda: mla.write_kv_scaled(x.cpu(), slots, cache, scales, 16),
                 lambda: mla.update_block_tables(i32([0]), i32([1, 2]), i32([0, 1, 2]), i32([[0], [0]]), i32([1]),
                                                 i32([0, 1]), 16, 2)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        mla.write_kv_scaled(x.float(), slots, cache, scales, 16)
    with pytest.raises(mla.MLAError) as e:
        mla.write_kv_scaled(x, slots, cache[:63 // 3 * 3], torch.ones(21, device="cuda"), 3)
    assert e.value.status == mla.MLA_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        runner.VerifyStep(num_reqs=1, num_rows=1, num_heads=1, max_qlen=1, block_size=16, num_blocks=1,
                          block_table_width=1, max_kv_len=16, scale_block=16, fused_merge=True)
    with pytest.raises(ValueError):
        runner.PagedLatentCache(num_reqs=1, num_rows=1, num_blocks=1, block_size=24, max_kv_len=24, scale_block=16)
