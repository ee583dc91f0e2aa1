"""Rotary positions, the rotary write and grouped / differential attention over the K/V cache it fills, each
against its float64 reference with the bound derived in grouped_reference.py, and a run of them together."""
import math

import numpy as np
import pytest
import torch

import grouped_reference as ref
from mla_decode_speculative_gb300 import mla, runner

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def f64(t):
    return t.double().cpu().numpy()


def rand(shape, seed):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(BF).cuda()


def freqs(pairs, base=10000.0):
    return base ** (-np.arange(pairs) / pairs)


def close(got, want, tol, what=""):
    """|got - want| <= tol, NaN only where it is wanted."""
    got = f64(got) if isinstance(got, torch.Tensor) else got
    both = np.isnan(want) | (np.isinf(want) & (got == want))
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN elsewhere"
    off = np.where(both, 0.0, np.abs(np.where(both, 0.0, got) - np.where(both, 0.0, want)) - np.where(both, 0.0, tol))
    assert off.max(initial=0.0) <= 0.0, f"{what}: {off.max():.3e} above the bound at {np.unravel_index(off.argmax(), off.shape)}"


# ------------------------------------------------------------------ rotary

@pytest.mark.parametrize("T,H,Hk,D,R,A,neighbours,seed", [
    (1, 1, 1, 64, 64, 1, False, 0), (5, 16, 1, 64, 64, 1, True, 1), (33, 12, 3, 128, 128, 3, False, 2),
    (257, 7, 7, 80, 40, 2, True, 3), (64, 40, 8, 128, 64, 3, True, 4), (19, 3, 1, 70, 6, 3, False, 5),
    (600, 33, 2, 256, 256, 1, False, 6), (4, 2, 1, 2, 2, 1, False, 7), (7, 2, 2, 512, 512, 2, False, 8),
    (2000, 64, 1, 64, 64, 3, True, 9), (9, 5, 1, 96, 36, 1, False, 10)])
def test_rotary_matches_reference(T, H, Hk, D, R, A, neighbours, seed):
    """Into other tensors, and in place; positions negative and at both ends of int32."""
    r = np.random.default_rng(seed)
    q, k = rand((T, H, D), seed), rand((T, Hk, D), seed + 100)
    pos = r.integers(-1000, 1 << 20, (A, T)).astype(np.int32)
    pos[0, 0], pos[-1, -1] = 2 ** 31 - 1, -2 ** 31
    f = freqs(R // 2)
    axes = r.integers(0, A, R // 2)
    turns = mla.rotary_turns(f)
    q_out, k_out = torch.zeros_like(q), torch.zeros_like(k)
    # the angle of the reference in float64 is off by 2^-53 of up to 2^31 radians
    args = (i32(pos if A > 1 else pos[0]), turns, i32(axes) if A > 1 else None)
    mla.rotary(q, k, *args, neighbours=neighbours, q_out=q_out, k_out=k_out)
    for x, y, name in ((q, q_out, "q"), (k, k_out, "k")):
        want, tol = ref.rotate(f64(x), pos, f, axes if A > 1 else 0 * axes, neighbours)
        close(y, want, tol + 2.0 ** -21 * np.abs(f64(x)).max(), name)
        assert torch.equal(y[..., R:], x[..., R:])
    mla.rotary(q, k, *args, neighbours=neighbours)
    assert torch.equal(q, q_out) and torch.equal(k, k_out)
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("order", ["latent", "heads_first", "odd", "one_missing"])
def test_rotary_strides(order):
    """The latent form's slices, heads before rows, an address that is only 2-byte aligned, q or k alone."""
    T, H, R = 37, 6, 64
    pos, f = i32(np.arange(T) * 977), freqs(R // 2)
    turns = mla.rotary_turns(f)
    q, k = rand((T, H, 192), 1)[..., 128:], rand((T, 1, 576), 2)[..., 512:]
    if order == "latent":
        q_out, k_out = torch.full((T, H, 576), 7.0, dtype=BF).cuda(), torch.full((T, 1, 576), 7.0, dtype=BF).cuda()
        a, b = q_out[..., 512:], k_out[..., 512:]
    elif order == "heads_first":
        q, k = rand((H, T, R), 3).transpose(0, 1), rand((1, T, R), 4).transpose(0, 1)
        q_out = torch.full((H, T, R), 7.0, dtype=BF).cuda()
        a, b = q_out.transpose(0, 1), torch.empty((1, T, R), dtype=BF).cuda().transpose(0, 1)
    elif order == "odd":
        q, k = rand(1 + T * H * (R + 1), 5)[1:].view(T, H, R + 1)[..., :R], rand(3 + T * R, 6)[3:].view(T, 1, R)
        q_out = torch.full((T, H, R + 3), 7.0, dtype=BF).cuda()
        a, b = q_out[..., :R], torch.empty((T, 1, R), dtype=BF).cuda()
    else:
        got = mla.rotary(None, k.contiguous(), pos, turns)
        assert got[0] is None
        both = mla.rotary(q.contiguous(), k.contiguous(), pos, turns)
        assert torch.equal(got[1], both[1])
        assert torch.equal(mla.rotary(q.contiguous(), None, pos, turns)[0], both[0])
        return
    mla.rotary(q, k, pos, turns, neighbours=True, q_out=a, k_out=b)
    for x, y in ((q, a), (k, b)):
        want, tol = ref.rotate(f64(x), f64(pos)[None], f, [0] * (R // 2), True)
        close(y, want, tol, order)
    if order == "latent":
        assert (q_out[..., :512] == 7).all() and (k_out[..., :512] == 7).all()
    if order == "odd":
        assert (q_out[..., R:] == 7).all()


def test_rotary_angles_add_up_and_far_positions_are_exact():
    """Rotating by a then by b is rotating by a + b, and a position 10^6 further on, whose turns are whole
    numbers for a frequency of 2 pi k / 10^6, is the same position bit for bit."""
    T, R = 50, 32
    f = 2 * math.pi * np.arange(1, R // 2 + 1) / 2.0 ** 20   # 2^20 positions: k turns, exactly
    turns = mla.rotary_turns(f)
    x, pos = rand((T, 2, R), 1), np.arange(T)
    near = mla.rotary(x.clone(), None, i32(pos), turns)[0]
    far = mla.rotary(x.clone(), None, i32(pos + (1000 << 20)), turns)[0]
    # freq is k * 2 pi / 2^20 to 2^-53 of itself: after 1000 * 2^20 positions 1000 k 2 pi 2^-53 radians
    assert (near.float() - far.float()).abs().max() <= 2.0 ** -7 * near.float().abs().max()
    assert (near != far).float().mean() < 0.01
    want, tol = ref.rotate(f64(near), (7 * pos)[None], f, [0] * (R // 2), False)
    close(mla.rotary(near.clone(), None, i32(7 * pos), turns)[0], want, tol)


@pytest.mark.parametrize("T,H,Hk,D,Dk,R,neighbours,inplace", [
    (130, 200, 9, 128, 128, 128, False, False),   # a row is more than a block
    (700, 65, 1, 64, 64, 64, True, False),        # a row is a little more than a round of threads
    (5001, 1, 1, 128, 128, 128, True, True),      # sines enough for half a block
    (900, 24, 3, 70, 128, 64, False, False),      # q and k of different alignment
    (3001, 130, 6, 128, 128, 64, False, False),   # larger than L2: the values past R with the rotated ones
    (5003, 96, 8, 80, 80, 40, True, False), (3001, 190, 10, 70, 70, 6, False, False),
    (3001, 150, 6, 128, 96, 32, True, False),     # the same of q and k with unequal tails
    (3001, 140, 10, 72, 72, 64, False, False)])   # that do not divide so
def test_rotary_in_one_call_is_rotary_in_many(T, H, Hk, D, Dk, R, neighbours, inplace):
    """q and k together, in whichever way they share their blocks, are q and k by themselves some rows at a
    time, bit for bit; and that is the reference."""
    r = np.random.default_rng(T + H)
    q, k = rand((T, H, D), 1), rand((T, Hk, Dk), 2)
    pos, axes, f = r.integers(0, 1 << 20, (3, T)), r.integers(0, 3, R // 2), freqs(R // 2)
    turns, ax = mla.rotary_turns(f), i32(axes)
    some = [0, T // 3, T - 1]
    parts = []
    for x in (q, k):
        out = torch.zeros_like(x)
        for t in range(0, T, 97):
            rows = slice(t, min(t + 97, T))
            mla.rotary(x[rows], None, i32(pos[:, rows]), turns, ax, neighbours=neighbours, q_out=out[rows])
        want, tol = ref.rotate(f64(x[some]), pos[:, some], f, axes, neighbours)
        close(out[some], want, tol)
        parts.append(out)
    if inplace:
        got = mla.rotary(q, k, i32(pos), turns, ax, neighbours=neighbours)
    else:
        got = mla.rotary(q, k, i32(pos), turns, ax, neighbours=neighbours, q_out=torch.zeros_like(q), k_out=torch.zeros_like(k))
    assert torch.equal(got[0], parts[0]) and torch.equal(got[1], parts[1])
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("T,H,Hkv,D,R", [(4100, 64, 8, 80, 40), (2500, 90, 6, 128, 64), (6000, 2, 2, 128, 128)])
def test_rotary_write_of_many_rows(T, H, Hkv, D, R):
    """The keys and values of a call are the rotary's, in the rows that the slots name; the others stay."""
    r = np.random.default_rng(T)
    q, k, v = rand((T, H, D), 1), rand((T, Hkv, D), 2), rand((T, Hkv, D), 3)
    pos, turns = i32(r.integers(0, 1 << 17, T)), mla.rotary_turns(freqs(R // 2))
    slots = r.permutation(2 * T)[:T].astype(np.int32)
    slots[::7] = -1
    kc, vc = (torch.full((2 * T, Hkv, D), 7.0, dtype=BF).cuda() for _ in range(2))
    want_q, want_k = mla.rotary(q.clone(), k.clone(), pos, turns)
    got = mla.rotary_write(q, k, v, pos, turns, i32(slots), kc, vc, q_out=torch.zeros_like(q))
    at = torch.as_tensor(slots[slots >= 0].astype(np.int64)).cuda()
    there = torch.as_tensor(slots >= 0).cuda()
    assert torch.equal(got, want_q)
    assert torch.equal(kc[at], want_k[there]) and torch.equal(vc[at], v[there])
    rest = torch.ones(2 * T, dtype=torch.bool).cuda()
    rest[at] = False
    assert (kc[rest] == 7).all() and (vc[rest] == 7).all()
    assert mla.get_device_error() == 0


def test_rotary_bad_axis_is_recorded():
    x, f = rand((3, 1, 8), 1), freqs(4)
    mla.rotary(x, None, i32(np.zeros((2, 3))), mla.rotary_turns(f), i32([0, 1, 2, -1]))
    assert mla.get_device_error() == 9 and mla.DEVICE_ERRORS[9] == "MLA_DEV_BAD_AXIS"


def test_rotary_of_nothing():
    x = torch.empty((0, 4, 64), dtype=BF).cuda()
    mla.rotary(x, x.clone(), torch.empty(0, dtype=torch.int32).cuda(), mla.rotary_turns(freqs(32)))
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("T,H,Hkv,D,Dv,R,joint,seed", [
    (1, 4, 1, 64, 64, 64, False, 0), (45, 12, 3, 128, 128, 128, True, 1), (300, 8, 4, 80, 64, 40, False, 2),
    (7, 0, 2, 128, 256, 64, False, 3), (1111, 32, 8, 128, 128, 128, False, 4), (20, 5, 5, 36, 7, 12, False, 5)])
def test_rotary_write_matches_reference(T, H, Hkv, D, Dv, R, joint, seed):
    """Rows without a slot, and cache rows that no slot names, stay as they were."""
    r = np.random.default_rng(seed)
    N = 2 * T + 8
    slots = r.permutation(N)[:T].astype(np.int32)
    slots[r.random(T) < 0.3] = -1
    q = rand((T, max(H, 1), D), seed) if H else None
    fused = rand((T, Hkv * (D + Dv)), seed + 1)
    k, v = fused[:, :Hkv * D].unflatten(1, (Hkv, D)), fused[:, Hkv * D:].unflatten(1, (Hkv, Dv))
    if joint:
        pool = rand((N, 2, Hkv, D), seed + 2)
        kc, vc = pool[:, 0], pool[:, 1]
    else:
        kc, vc = rand((N, Hkv, D), seed + 2), rand((N, Hkv, Dv), seed + 3)
    k0, v0 = kc.clone(), vc.clone()
    pos, f, axes = r.integers(0, 5000, (3, T)), freqs(R // 2), np.arange(R // 2) % 3
    out = mla.rotary_write(q, k, v, i32(pos), mla.rotary_turns(f), i32(slots), kc, vc, i32(axes))
    assert mla.get_device_error() == 0
    mine = slots >= 0
    want, tol = ref.rotate(f64(k), pos, f, axes, False)
    at = torch.as_tensor(slots[mine].astype(np.int64)).cuda()
    close(kc[at], want[mine], tol[mine], "keys")
    assert torch.equal(vc[at], v[torch.as_tensor(mine).cuda()])
    rest = torch.ones(N, dtype=torch.bool).cuda()
    rest[at] = False
    assert torch.equal(kc[rest], k0[rest]) and torch.equal(vc[rest], v0[rest])
    if H:
        assert out.data_ptr() == q.data_ptr()
        want, tol = ref.rotate(f64(rand((T, H, D), seed)), pos, f, axes, False)
        close(out, want, tol, "queries")
    else:
        assert out is None


def test_rotary_write_bad_slots_are_recorded_and_not_written():
    k, kc = rand((4, 2, 64), 1), torch.zeros((16, 2, 64), dtype=BF).cuda()
    vc = kc.clone()
    mla.rotary_write(None, k, k, i32(np.zeros(4)), mla.rotary_turns(freqs(32)), i32([3, 16, -2, 2 ** 31 - 1]), kc, vc)
    assert mla.get_device_error() == 3
    assert torch.equal(vc[3], k[0]) and torch.equal(kc[3], k[0])
    assert int((vc != 0).any(2).any(1).sum()) == 1 and int((kc != 0).any(2).any(1).sum()) == 1


# ------------------------------------------------------------------ attention

class State:
    """A cache whose unused rows are NaN, its page table, queries and row lengths."""

    def __init__(self, L, ql, H, Hkv, D, bs, maps=1, joint=False, seed=0, spare=0):
        r = np.random.default_rng(seed)
        L, ql = np.asarray(L), np.asarray(ql)
        self.maps, self.P = maps, mla.page_size(bs)
        blocks = -(-np.maximum(L, 0) // bs)
        pool = int(blocks.sum()) + 3
        perm = r.permutation(pool)
        R = bs // self.P
        width = max(1, int(blocks.max()) * R)
        self.table = np.full((len(L), width), -1, np.int32)
        at, used = 0, np.zeros(pool * bs, bool)
        for b, n in enumerate(blocks):
            ids = perm[at:at + n]
            at += n
            pages = (ids[:, None] * R + np.arange(R)).reshape(-1)
            self.table[b, :len(pages)] = pages
            rows = (pages[:, None].astype(np.int64) * self.P + np.arange(self.P)).reshape(-1)[:max(L[b], 0)]
            used[rows] = True
        N = pool * bs
        pair = (2,) if maps == 2 else ()
        if joint:
            kv = rand((N, 2, Hkv, D), seed + 1)
            self.k, self.v = kv[:, 0], kv[:, 1]
        else:
            self.k, self.v = rand((N, Hkv) + pair + (D,), seed + 1), rand((N, Hkv, maps * D), seed + 2)
        gone = torch.as_tensor(~used).cuda()
        self.k[gone], self.v[gone] = math.nan, math.nan
        self.ind = np.concatenate([[0], np.cumsum(ql)])
        self.T = int(self.ind[-1]) + spare
        self.q = rand((self.T, H) + pair + (D,), seed + 3)
        self.row_len = np.zeros(self.T, np.int64)
        for b in range(len(L)):
            n = ql[b]
            self.row_len[self.ind[b]:self.ind[b + 1]] = L[b] - n + 1 + np.arange(n)
        self.qmax = max(1, int(ql.max()))
        self.scale = 1.0 / math.sqrt(D)
        self.lam = torch.linspace(0.2, 0.8, H).cuda()
        self.gain = None

    def run(self, window=0, **kw):
        args = (i32(self.ind), i32(self.row_len), i32(self.table), self.P, self.qmax, self.scale)
        if self.maps == 1:
            out, lse, _ = mla.decode_grouped(self.q, self.k, self.v, *args, window=window, **kw)
        else:
            out, lse, _ = mla.decode_differential(self.q, self.k, self.v, self.lam, *args, gain=self.gain, window=window, **kw)
        return out, lse

    def want(self, window=0):
        N, Hkv = self.k.shape[:2]
        q = f64(self.q).reshape(self.T, self.q.shape[1], self.maps, -1)
        return ref.attention(q, f64(self.k).reshape(N, Hkv, self.maps, -1), f64(self.v), self.scale, self.ind, self.row_len,
                             self.table, self.P, window, f64(self.lam), None if self.gain is None else f64(self.gain))

    def check(self, window=0, **kw):
        out, lse = self.run(window, **kw)
        n = self.ind[-1]
        o, tol, l, ltol = self.want(window)
        close(out[:n], o[:n], tol[:n], "out")
        close(lse[:n].reshape(l[:n].shape), l[:n], ltol[:n], "lse")
        # the framework's bar for the path: 1e-2 of a row's largest value
        top = np.abs(o[:n]).max(-1)
        err = np.abs(np.nan_to_num(f64(out[:n])) - np.nan_to_num(o[:n])).max(-1)
        assert (err <= 1e-2 * np.nan_to_num(top) + 1e-30).all()
        assert mla.get_device_error() == 0
        return out, lse


SHAPES = [  # L, qlen, H, Hkv, D, bs, window, joint
    ([1], [1], 1, 1, 64, 8, 0, False), ([1, 2, 7, 8, 9], [1, 2, 1, 3, 1], 6, 2, 128, 8, 0, False),
    ([127, 128, 129, 130], [1, 1, 1, 2], 8, 8, 64, 16, 0, True), ([256, 256], [1, 1], 16, 4, 128, 16, 0, False),
    ([700, 45, 1300], [4, 4, 4], 32, 2, 128, 64, 0, False), ([333, 900], [3, 1], 12, 4, 64, 96, 0, True),
    ([500, 2049], [2, 2], 16, 2, 256, 256, 0, True), ([3000], [1], 4, 4, 256, 32, 0, False),
    ([4000, 31], [8, 8], 5, 1, 128, 128, 0, False), ([650], [8], 64, 4, 128, 16, 0, False),
    ([900, 17], [5, 2], 128, 1, 64, 64, 0, False), ([777], [3], 70, 1, 128, 16, 0, False),
    ([2000, 130, 5], [4, 2, 5], 8, 2, 128, 16, 100, False), ([1500, 640], [1, 8], 12, 3, 64, 64, 257, False),
    ([1025, 129], [2, 1], 16, 2, 256, 256, 1, True), ([300] * 40, [1] * 40, 14, 2, 128, 16, 0, False),
    (list(range(1, 90)), [1] * 89, 6, 3, 64, 8, 0, False), ([20000], [1], 8, 1, 128, 64, 0, False),
    ([9000, 9], [4, 1], 28, 4, 128, 16, 4096, False)]


@pytest.mark.parametrize("i", range(len(SHAPES)))
def test_grouped_matches_reference(i):
    L, ql, H, Hkv, D, bs, window, joint = SHAPES[i]
    State(L, ql, H, Hkv, D, bs, joint=joint, seed=i).check(window)


DIFF = [  # L, qlen, H, Hkv, D, bs, window, gain
    ([1], [1], 1, 1, 64, 8, 0, True), ([1, 2, 17, 128, 129], [1, 2, 3, 1, 4], 4, 2, 64, 16, 0, False),
    ([700, 45, 1300], [4, 4, 4], 16, 4, 128, 64, 0, True), ([333, 900], [3, 1], 12, 4, 64, 96, 0, True),
    ([5000], [1], 8, 8, 128, 32, 0, False), ([640, 9], [8, 8], 10, 2, 64, 16, 0, True),
    ([2000, 130], [4, 2], 48, 1, 128, 128, 0, True), ([1500, 640], [1, 8], 12, 3, 64, 64, 257, False),
    ([300] * 40, [1] * 40, 14, 2, 64, 16, 0, True), ([12000, 60], [2, 2], 4, 1, 64, 64, 0, True)]


@pytest.mark.parametrize("i", range(len(DIFF)))
def test_differential_matches_reference(i):
    L, ql, H, Hkv, D, bs, window, norm = DIFF[i]
    s = State(L, ql, H, Hkv, D, bs, maps=2, seed=100 + i)
    if norm:
        s.gain = 0.2 + 0.1 * torch.randn(2 * D, generator=torch.Generator().manual_seed(i)).cuda()
    s.check(window)


@pytest.mark.parametrize("maps", [1, 2])
def test_rows_that_see_nothing_and_rows_behind_the_last(maps):
    """Row lengths of zero and below; rows from qo_indptr[B] on are left as they were; a request without rows."""
    s = State([200, 100, 300, 64], [3, 0, 2, 1], 6, 2, 64, 16, maps=maps, seed=5, spare=4)
    s.row_len[[0, 3]], s.row_len[5] = 0, -7
    out = torch.full((s.T, 6, maps * 64), 3.0, dtype=BF).cuda()
    lse = torch.full((s.T, 6) + (2,) * (maps - 1), 5.0).cuda()
    s.check(out=out, lse=lse)
    assert (out[s.ind[-1]:] == 3).all() and (lse[s.ind[-1]:] == 5).all()
    for r in (0, 3, 5):
        assert (out[r] == 0).all() and (lse[r] == -math.inf).all()


@pytest.mark.parametrize("maps", [1, 2])
def test_rows_of_unequal_lengths_in_one_request(maps):
    """Row lengths in any order, far apart: every row sees its own tokens."""
    s = State([2000], [6], 4, 2, 128, 32, maps=maps, seed=6)
    s.row_len[:] = [2000, 1, 700, 128, 0, 1999]
    s.check()
    s.check(window=300)


@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("what", ["key", "value"])
def test_nan_reaches_the_rows_that_see_its_token(what, window):
    """A draft's token that is not finite: rows before it are as they were without it, rows that see it are
    NaN; with a window the same at its far end."""
    s = State([300, 140], [4, 3], 8, 2, 128, 16, seed=7)
    clean, clean_lse = s.run(window)
    at = lambda b, j: int(s.table[b][j // s.P]) * s.P + j % s.P  # noqa: E731
    # (an infinite key may rightly end as a weight of zero)
    hit = [(0, 298, math.nan), (1, 138, math.nan if what == "key" else math.inf)]
    if window:
        hit.append((0, 300 - 4 + 1 - window, math.nan))   # the first token of row 0's window only
    for b, j, x in hit:
        (s.k if what == "key" else s.v)[at(b, j), 1, 5] = x
    out, lse = s.run(window)
    sees = np.zeros(7, bool)
    for b, j, _ in hit:
        for r in range(s.ind[b], s.ind[b + 1]):
            n = s.row_len[r]
            sees[r] |= j < n and (not window or j >= n - window)
    for r in range(7):
        for h in range(8):
            if sees[r] and h >= 4:
                assert not torch.isfinite(out[r, h]).all()
            else:
                assert torch.equal(out[r, h], clean[r, h]) and torch.equal(lse[r, h], clean_lse[r, h]), (r, h)


@pytest.mark.parametrize("what", ["seen_by_all", "seen_by_some", "infinite"])
@pytest.mark.parametrize("copies", [1, 150])
@pytest.mark.parametrize("maps", [1, 2])
def test_value_that_is_not_finite_in_a_part_of_vanishing_weight(maps, copies, what):
    """The later half of the keys scores 160 e-folds (230 powers of two) above the earlier one, whose parts'
    weights are zero in float32; a value of the earlier half that is not finite still reaches the rows that see
    it, wherever the split falls: one request (every unit cut), and 150 copies of it (most units whole)."""
    n, j, D = 6000, 1000, 64
    s = State([n], [2], 4, 2, D, 16, maps=maps, seed=30)
    if what == "seen_by_some":
        s.row_len[0] = 940                     # inside the token's tile
    at = s.table[0][np.arange(n) // s.P].astype(np.int64) * s.P + np.arange(n) % s.P
    rows = torch.as_tensor(at).cuda()
    s.k[rows] = (0.1 * s.k[rows].float()).to(BF)
    s.k[rows[3000:]] = 5.0
    s.q[:] = 4.0                               # scores: 8^-1 * 64 * 4 * 5 = 160
    s.table, s.row_len = np.repeat(s.table, copies, 0), np.tile(s.row_len, copies)
    s.q, s.ind, s.T = s.q.repeat(copies, *([1] * (s.q.dim() - 1))), np.arange(copies + 1) * 2, 2 * copies
    clean, clean_lse = s.run()
    assert torch.isfinite(clean).all()
    s.v[rows[j], 1, 5] = math.inf if what == "infinite" else math.nan
    out, lse = s.run()
    assert torch.equal(lse, clean_lse)
    for r in range(s.T):
        assert torch.equal(out[r, :2], clean[r, :2])
        if s.row_len[r] <= j:
            assert torch.equal(out[r], clean[r])
        elif what == "seen_by_some":
            assert torch.isnan(out[r, 2:]).all()
        else:
            assert not torch.isfinite(out[r, 2:, 5]).any()
            keep = [d for d in range(maps * D) if d != 5]
            assert torch.equal(out[r, 2:, keep], clean[r, 2:, keep])
    assert mla.get_device_error() == 0


@pytest.mark.parametrize("L,ql,H,Hkv,D,bs", [
    ([700], [3], 8, 2, 64, 16), ([900, 30], [1, 4], 16, 4, 128, 64), ([400], [8], 64, 4, 128, 16),
    ([500, 60], [2, 2], 8, 1, 256, 32), ([20000], [2], 8, 2, 128, 16)])
def test_infinite_value_is_infinite_in_its_dim(L, ql, H, Hkv, D, bs):
    """A value of plus or minus infinity at tokens that all rows of the request see: infinite in that dim, as the
    weighted sum is; both in one dim: NaN; every other number as it was.  In units that are cut and whole ones."""
    s = State(L, ql, H, Hkv, D, bs, seed=32)
    s.q *= 0.5                                 # no weight that rounds to zero
    clean, clean_lse = s.run()
    at = lambda b, j: int(s.table[b][j // s.P]) * s.P + j % s.P  # noqa: E731
    g = Hkv - 1
    for j, d, x in ((3, 5, math.inf), (L[0] // 2, D - 1, -math.inf), (L[0] - ql[0] - 1, 5, math.inf),
                    (7, 11, math.inf), (L[0] // 2 + 1, 11, -math.inf)):
        s.v[at(0, j), g, d] = x
    out, lse = s.run()
    assert torch.equal(lse, clean_lse)
    want, per = clean.clone(), H // Hkv
    want[:ql[0], g * per:, 5], want[:ql[0], g * per:, D - 1] = math.inf, -math.inf
    want[:ql[0], g * per:, 11] = math.nan
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(out.nan_to_num(nan=0.0, posinf=1e9, neginf=-1e9), want.nan_to_num(nan=0.0, posinf=1e9, neginf=-1e9))
    o, tol, l, ltol = s.want()
    close(out, o, tol, "out")
    close(lse, l.reshape(lse.shape), ltol.reshape(lse.shape), "lse")
    assert mla.get_device_error() == 0


def test_query_that_is_not_finite_spoils_its_own_row():
    s = State([300], [4], 8, 2, 128, 16, seed=8)
    clean, _ = s.run()
    s.q[1, 3, 7], s.q[2, 6, 0] = math.nan, math.inf
    out, _ = s.run()
    for r in range(4):
        for h in range(8):
            if (r, h) in ((1, 3), (2, 6)):
                assert torch.isnan(out[r, h]).any()
            else:
                assert torch.equal(out[r, h], clean[r, h])


@pytest.mark.parametrize("maps", [1, 2])
def test_large_scores_move_the_maximum_late(maps):
    """Scores that grow by hundreds from tile to tile: every tile rescales what came before."""
    s = State([1000], [1], 4, 1, 64, 16, maps=maps, seed=9)
    rows = s.table[0][np.arange(1000) // s.P].astype(np.int64) * s.P + np.arange(1000) % s.P
    ramp = torch.linspace(0.1, 6.0, 1000).cuda().view(-1, *([1] * (s.k.dim() - 1)))
    s.k[torch.as_tensor(rows).cuda()] = (ramp * s.q[0, 0].float().sign() * torch.ones_like(s.k[:1].float())).to(BF)
    s.q *= 4
    s.check()


def test_strides_of_queries_and_caches():
    """q as a slice of a fused projection, a cache row wider than its heads."""
    s = State([500, 70], [2, 3], 8, 2, 128, 16, seed=10)
    want, lse = s.check()
    fused = torch.zeros((s.T, 12 * 128 + 8), dtype=BF).cuda()
    fused[:, 8:8 + 1024] = s.q.flatten(1)
    s.q = fused[:, 8:8 + 1024].unflatten(1, (8, 128))
    wide = torch.full((s.k.shape[0], 2 * 128 + 24), math.nan, dtype=BF).cuda()
    wide[:, 16:272] = s.k.flatten(1)
    s.k = wide[:, 16:272].unflatten(1, (2, 128))
    out, lse2 = s.run()
    assert torch.equal(out, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("maps", [1, 2])
def test_single_row_of_any_stride(maps):
    """One row of queries as it comes out of a transpose, a row stride of one head."""
    s = State([300], [1], 8, 2, 64, 16, maps=maps, seed=34)
    want, lse = s.check()
    by_head = torch.empty((8, 1) + tuple(s.q.shape[2:]), dtype=BF).cuda()
    s.q = by_head.copy_(s.q.transpose(0, 1)).transpose(0, 1)
    assert s.q.stride(0) == maps * 64
    out, lse2 = s.run()
    assert torch.equal(out, want) and torch.equal(lse, lse2)


@pytest.mark.parametrize("maps,L,ql,H,Hkv,D,bs,window", [
    (1, [700] * 6, [8] * 6, 64, 4, 128, 16, 0),                    # two row blocks each
    (1, [9000, 20, 300, 5000, 64, 1], [8, 8, 8, 8, 8, 1], 64, 4, 64, 64, 0),   # and one with one
    (1, [130, 1500] * 9, [8, 8] * 8 + [3, 8], 64, 4, 64, 32, 100),
    (1, [2500] * 3, [1] * 3, 128, 1, 128, 128, 0),                 # a row's heads in two blocks
    (1, [400] * 5, [3] * 5, 100, 1, 256, 8, 0),                    # in two of unequal size
    (1, [3000] * 2, [11] * 2, 64, 1, 64, 16, 0),                   # eleven blocks: the last one alone
    (1, [3000] * 3, [3] * 3, 64, 1, 64, 16, 0),                    # three: not in twos
    (2, [1800] * 4, [8] * 4, 16, 2, 64, 64, 0), (2, [900, 4000, 77], [16, 16, 16], 8, 2, 128, 16, 300)])
def test_row_blocks_that_share_their_keys(maps, L, ql, H, Hkv, D, bs, window):
    """More rows of a group than a product holds, cut into several parts, with rows that see nothing."""
    s = State(L, ql, H, Hkv, D, bs, maps=maps, joint=False, seed=len(L) + H, spare=2)
    for k in range(0, s.ind[-1], 13):
        s.row_len[k] = 0
    s.check(window)


@pytest.mark.parametrize("maps,D,H,Hkv,L,n", [
    (1, 64, 16, 4, [5000, 120, 1, 2222], 2), (2, 64, 16, 4, [5000, 120, 1, 2222], 2), (1, 256, 12, 4, [623] * 60, 1),
    (1, 256, 24, 4, [562] * 35, 4), (1, 256, 40, 4, [562] * 35, 4), (2, 128, 56, 8, [562] * 35, 4), (2, 128, 7, 1, [100 + 37 * i for i in range(60)], 3),
    (1, 128, 64, 2, [300 + 11 * i for i in range(40)], 2)])
def test_repeats_itself_bit_by_bit(maps, D, H, Hkv, L, n):
    """Many units that end inside a tile, so that their last values are cleared while the tile before is still
    being multiplied."""
    s = State(L, [min(n, x) for x in L], H, Hkv, D, 32, maps=maps, seed=11)
    first, lse = s.run()
    for _ in range(100):
        out, l = s.run()
        assert torch.equal(out, first) and torch.equal(l, lse)
    s.check()


def test_device_checks():
    """A page outside the cache reads as zeros, a length beyond the table is clipped, a request whose
    offsets are wrong is left as it was; each is recorded."""
    s = State([100, 100], [1, 1], 4, 2, 64, 16, seed=12)
    good, _ = s.run()
    s.table[0, 2] = 10 ** 6
    out, _ = s.run()
    assert mla.get_device_error() == 5 and torch.equal(out[1], good[1])
    row = s.table[0, 2] = min(set(range(s.k.shape[0] // s.P)) - set(s.table.reshape(-1).tolist()))   # a spare page
    rows = slice(row * s.P, (row + 1) * s.P)
    s.k[rows], s.v[rows] = 0, 0
    assert torch.equal(s.run()[0], out) and mla.get_device_error() == 0
    s.row_len[0] = 10 ** 9
    s.table[0, 6:] = s.table[0, 0]
    out, _ = s.run()
    assert mla.get_device_error() == 4 and torch.equal(out[1], good[1])
    s.row_len[0] = s.table.shape[1] * s.P
    assert torch.equal(s.run()[0], out) and mla.get_device_error() == 0
    for ind in ([0, 2, 1], [0, 1, 9], [-1, 1, 2]):
        s.ind = np.array(ind)
        keep = torch.full((2, 4, 64), 3.0, dtype=BF).cuda()
        s.run(out=keep)
        assert mla.get_device_error() == 1


@pytest.mark.parametrize("maps", [1, 2])
@pytest.mark.parametrize("ind,good", [([0, 2, 1], None), ([0, 1, 9], 0), ([-1, 1, 2], 1), ([0, 1, 2], 1)])
def test_requests_with_wrong_offsets_leave_their_rows(maps, ind, good):
    """The rows of a request that the device checks refuse hold what they held, outputs and sums; the other
    request's are right."""
    s = State([100, 100], [1, 1], 4, 2, 64, 16, maps=maps, seed=33)
    full, full_lse = s.run()
    s.ind = np.array(ind)
    out = torch.full((2, 4, maps * 64), 3.0, dtype=BF).cuda()
    lse = torch.full((2, 4) + (2,) * (maps - 1), 5.0).cuda()
    if ind == [0, 2, 1]:
        s.qmax = 1                             # two rows are above the bound of one, and the next offset goes back
    s.run(out=out, lse=lse)
    assert mla.get_device_error() == (0 if ind == [0, 1, 2] else 1)
    for r in range(2):
        if ind == [0, 1, 2] or r == good:
            assert torch.equal(out[r], full[r]) and torch.equal(lse[r], full_lse[r])
        else:
            assert (out[r] == 3).all() and (lse[r] == 5).all()


def test_another_stream_and_its_own_workspace():
    s = State([900, 20], [2, 2], 8, 2, 128, 16, seed=13)
    want, lse = s.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out, l = s.run(stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(l, lse)


@pytest.mark.parametrize("maps", [1, 2])
def test_more_requests_than_one_launch_tabulates(maps):
    """1,300 requests, some without rows, some that see nothing."""
    r = np.random.default_rng(14)
    L, ql = r.integers(3, 40, 1300), r.integers(0, 4, 1300)
    L[::100], ql[::100] = 400, 2
    s = State(L, ql, 4, 2, 64, 8, maps=maps, seed=14)
    s.row_len[::37] = 0
    s.check()


@pytest.mark.parametrize("maps,H,Hkv,window", [(1, 6, 2, 0), (1, 6, 2, 70), (2, 4, 1, 0), (1, 40, 1, 0)])
def test_many_rows_per_request(maps, H, Hkv, window):
    """Prompts as one causal call: many row blocks, tiles that only some rows see."""
    State([300, 77, 140], [300, 77, 9], H, Hkv, 64, 16, maps=maps, seed=15).check(window)


@pytest.mark.parametrize("bs", [8, 64, 128])
def test_cache_of_one_block_and_of_less_than_a_page(bs):
    s = State([5], [2], 4, 2, 128, bs, seed=16)
    s.check()
    s.table[:] = 0
    s.k, s.v = s.k[:8].clone(), s.v[:8].clone()   # eight rows: no whole page of 64 or 128
    s.k[:], s.v[:] = 1, 1
    out, lse = s.run()
    if bs == 8:
        assert (out == 1).all() and mla.get_device_error() == 0
    else:
        assert (out == 0).all() and mla.get_device_error() == 5


def test_window_does_not_read_pages_before_it():
    """Pages that have left every row's window may have gone back to the pool; a table wider than the
    requests need."""
    s = State([1500, 300], [3, 2], 8, 2, 128, 16, seed=17)
    want, lse = s.check(window=200)
    wide = np.full((2, 4 * s.table.shape[1]), -1, np.int32)
    wide[:, :s.table.shape[1]] = s.table
    wide[0, :(1500 - 3 + 1 - 200) // 16] = -1
    wide[1, :(300 - 2 + 1 - 200) // 16] = 10 ** 8
    s.table = wide
    out, l = s.run(200)
    assert torch.equal(out, want) and torch.equal(l, lse) and mla.get_device_error() == 0


@pytest.mark.parametrize("maps,D", [(1, 64), (1, 128), (1, 256), (2, 64), (2, 128)])
def test_waits_that_run_out_are_recorded(maps, D):
    """A budget that no copy can meet: every CTA gives up, the next call is right."""
    s = State([3000, 200, 1000], [4, 1, 2], 16, 4, D, 16, maps=maps, seed=18)
    want, lse = s.run()
    for _ in range(2):
        s.run(wait_cycles=1)
        assert mla.get_device_error() == 6
    out, l = s.run()
    assert torch.equal(out, want) and torch.equal(l, lse) and mla.get_device_error() == 0


@pytest.mark.parametrize("maps,L,ql,H,Hkv,D", [
    (1, [3000, 200, 1000], [4, 1, 2], 16, 4, 64), (1, [9000, 40, 300, 5000], [1, 2, 1, 1], 8, 4, 256),
    (1, [2500] * 6, [8] * 6, 64, 4, 128), (1, [300 + 90 * i for i in range(64)], [1] * 64, 16, 8, 128),
    (2, [3000, 200, 1000], [4, 1, 2], 16, 4, 64), (2, [120 + 90 * i for i in range(64)], [2] * 64, 16, 8, 64),
    (2, [20000, 900], [4, 4], 32, 4, 128)])
def test_waits_that_run_out_leave_rows_as_they_were_or_right(maps, L, ql, H, Hkv, D):
    """Wait budgets from one that no copy meets to one that some do: every row and head is what it was before
    the call or what a call that ran through gives, output and sum alike."""
    s = State(L, ql, H, Hkv, D, 16, maps=maps, seed=31)
    want, want_lse = s.run()
    gave_up = 0
    for cycles in (1, 1, 500, 2000, 4000, 8000, 16000, 32000):
        out = torch.full((s.T, H, maps * D), 3.0, dtype=BF).cuda()
        lse = torch.full((s.T, H) + (2,) * (maps - 1), 5.0).cuda()
        s.run(out=out, lse=lse, wait_cycles=cycles)
        code = mla.get_device_error()
        assert code in (0, 6)
        same = (out == want).all(-1) & (lse == want_lse).reshape(s.T, H, -1).all(-1)
        kept = (out == 3).all(-1) & (lse == 5).reshape(s.T, H, -1).all(-1)
        assert (same | kept).all(), f"{cycles} cycles: {int((~(same | kept)).sum())} of {s.T * H} rows and heads"
        assert code == 6 or same.all()
        gave_up += code == 6
    assert gave_up >= 2
    out, lse = s.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and mla.get_device_error() == 0


def test_two_captured_graphs_with_a_workspace_each():
    """Two calls captured apart, replayed at the same time on two streams, over and over."""
    states = [State([4000, 700], [2, 2], 16, 4, 128, 32, seed=20), State([3000, 2500, 10], [1, 1, 1], 8, 2, 64, 16, maps=2, seed=21)]
    want = [s.run() for s in states]
    graphs = []
    for s in states:
        args = (i32(s.ind), i32(s.row_len), i32(s.table), s.P, s.qmax, s.scale)
        H, D = s.q.shape[1], s.q.shape[-1]
        ws = torch.empty(mla.decode_grouped_workspace_bytes(H, s.k.shape[1], s.qmax, D, s.maps == 2), dtype=torch.uint8).cuda()
        out = torch.zeros((s.T, H, s.maps * D), dtype=BF).cuda()
        lse = torch.zeros((s.T, H) + (2,) * (s.maps - 1)).cuda()
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g):
            if s.maps == 1:
                mla.decode_grouped(s.q, s.k, s.v, *args, out=out, lse=lse, workspace=ws)
            else:
                mla.decode_differential(s.q, s.k, s.v, s.lam, *args, out=out, lse=lse, workspace=ws)
        graphs.append((g, out, lse, args))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(30):
        for (g, *_), stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                g.replay()
    torch.cuda.synchronize()
    for (_, out, lse, _), (o, l) in zip(graphs, want):
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert mla.get_device_error() == 0


def test_workspace_that_is_too_small_is_refused():
    s = State([100], [1], 4, 2, 64, 16, seed=22)
    with pytest.raises(mla.MLAError) as e:
        s.run(workspace=torch.empty(64, dtype=torch.uint8).cuda())
    assert e.value.status == mla.MLA_ERR_WORKSPACE


def test_cache_past_32_bit_offsets():
    """A pool of more than 2^31 elements, the request's pages at its end."""
    bs, Hkv, D = 64, 8, 128
    N = (1 << 22) + 64 * 40
    k, v = torch.zeros((N, Hkv, D), dtype=BF, device="cuda"), torch.zeros((N, Hkv, D), dtype=BF, device="cuda")
    n = 1000
    first = N // bs - 20
    rows = slice(first * bs, first * bs + n)
    pos, turns = i32(np.arange(n)), mla.rotary_turns(freqs(64))
    kn, vn, q = rand((n, Hkv, D), 1), rand((n, Hkv, D), 2), rand((1, 16, D), 3)
    mla.rotary_write(None, kn, vn, pos, turns, i32(first * bs + np.arange(n)), k, v)
    want, tol = ref.rotate(f64(kn), np.arange(n)[None], freqs(64), [0] * 64, False)
    close(k[rows], want, tol)
    table = i32((first + np.arange(16))[None])
    out, lse, _ = mla.decode_grouped(q, k, v, i32([0, 1]), i32([n]), table, 64, 1, 0.09)
    small_k, small_v = k[first * bs:].clone(), v[first * bs:].clone()
    out2, lse2, _ = mla.decode_grouped(q, small_k, small_v, i32([0, 1]), i32([n]), i32(np.arange(16)[None]), 64, 1, 0.09)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and mla.get_device_error() == 0


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("differential", [False, True])
def test_drafting_steps(differential):
    """A prompt, then drafting steps with drafts taken back and a request that finishes, each appended and
    attended to in a captured graph, against a history kept in float64."""
    r = np.random.default_rng(3)
    B, H, Hkv, D, bs, maps, cap = 3, 6, 2, 64, 16, 2 if differential else 1, 64
    f, axes = freqs(D // 2), np.arange(D // 2) % 3
    turns, ax = mla.rotary_turns(f), i32(axes)
    cache = runner.PagedKVCache(num_reqs=B, num_rows=cap, num_blocks=40, block_size=bs, max_kv_len=160, num_kv_heads=Hkv,
                                head_dim=D, differential=differential)
    step = runner.GroupedStep(num_reqs=B, num_rows=cap, num_heads=H, num_kv_heads=Hkv, head_dim=D, max_qlen=cap,
                              block_size=bs, num_blocks=40, max_kv_len=160, differential=differential, window=50)
    pair = (2,) if differential else ()
    q, k = torch.zeros((cap, H) + pair + (D,), dtype=BF).cuda(), torch.zeros((cap, Hkv) + pair + (D,), dtype=BF).cuda()
    v, pos = torch.zeros((cap, Hkv, maps * D), dtype=BF).cuda(), torch.zeros((3, cap), dtype=torch.int32).cuda()
    q_out, seq, ind = torch.zeros_like(q), torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B + 1, dtype=torch.int32).cuda()
    lam, gain = torch.linspace(0.1, 0.9, H).cuda(), torch.full((maps * D,), 0.3).cuda()
    weights = dict(lam=lam, gain=gain) if differential else {}

    def body():
        cache.append(q, k, v, pos, turns, seq, ind, ax, q_out=q_out)
        return step(q_out, cache.k, cache.v, seq, ind, cache.block_table, 0.11, **weights)

    graph, hist = None, [[] for _ in range(B)]
    for n, (lens, new) in enumerate([([20, 31, 5], [20, 31, 5]), ([24, 35, 9], [4, 4, 4]), ([26, 37, 10], [4, 4, 3]),
                                     ([40, 0, 13], [15, 0, 3]), ([41, 60, 16], [1, 60, 3]), ([44, 64, 20], [4, 4, 4])]):
        T = sum(new)
        q.copy_(rand(q.shape, 50 + n)), k.copy_(rand(k.shape, 60 + n)), v.copy_(rand(v.shape, 70 + n))
        p = r.integers(0, 3000, (3, cap))
        pos.copy_(i32(p)), seq.copy_(i32(lens)), ind.copy_(i32(np.concatenate([[0], np.cumsum(new)])))
        if graph is None:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                body()
            torch.cuda.current_stream().wait_stream(side)
        elif n == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                body()
        if n == 0:
            graph = False
        else:
            graph.replay()
        code = mla.get_device_error()
        assert code == (2 if 0 in new else 0)   # the plan records the finished request
        # the written rows, held to the rotation's bound; the attention's reference then takes them as they are
        slot = cache.slot_map[:T].long()
        want, tol = ref.rotate(f64(k).reshape(cap, Hkv * maps, D), p, f, axes, False)
        close(cache.k[slot].reshape(T, Hkv * maps, D), want[:T], tol[:T], "keys")
        want, tol = ref.rotate(f64(q).reshape(cap, H * maps, D), p, f, axes, False)
        close(q_out.reshape(cap, H * maps, D), want, tol, "queries")
        assert torch.equal(cache.v[slot], v[:T])
        kr, vr = f64(cache.k[slot]).reshape(T, Hkv, maps, D), f64(cache.v[slot])
        qr, at = f64(q_out).reshape(cap, H, maps, D), np.cumsum([0] + new)
        out, lse = f64(step.out), f64(step.lse).reshape(cap, H, maps)
        for b in range(B):
            hist[b] = hist[b][:lens[b] - new[b]] + [(kr[i], vr[i]) for i in range(at[b], at[b + 1])]
            assert len(hist[b]) == lens[b]
            if not new[b]:
                continue
            K, V = np.stack([x for x, _ in hist[b]]), np.stack([x for _, x in hist[b]])
            want, tol, l, ltol = ref.attention(qr[at[b]:at[b + 1]], K, V, 0.11, [0, new[b]], lens[b] - new[b] + 1 + np.arange(new[b]),
                                               np.arange(160)[None], 1, 50, f64(lam), f64(gain) if differential else None)
            close(out[at[b]:at[b + 1]], want, tol, f"step {n}")
            close(lse[at[b]:at[b + 1]], l, ltol, f"step {n}")


@pytest.mark.parametrize("differential", [False, True])
def test_kv_append_that_ran_out_of_blocks_is_undone_and_made_again(differential):
    """Too few free blocks, undone, then appended again with the same queries: with q_out they and the keys are
    those of a step that never failed."""
    maps, D = 2 if differential else 1, 64
    make = lambda: runner.PagedKVCache(num_reqs=2, num_rows=64, num_blocks=6, block_size=16, max_kv_len=96,  # noqa: E731
                                       num_kv_heads=2, head_dim=D, differential=differential)
    pair = (2,) if differential else ()
    q, k = rand((64, 4) + pair + (D,), 1), rand((64, 2) + pair + (D,), 2)
    v, pos, turns = rand((64, 2, maps * D), 3), i32(np.arange(64) * 31), mla.rotary_turns(freqs(D // 2))
    q0, rest = q.clone(), (k, v, pos, turns)
    c, never = make(), make()
    for x in (c, never):
        x.append(q, *rest, i32([40, 10]), i32([0, 40, 50]), q_out=torch.empty_like(q))
    assert mla.get_device_error() == 0
    held = c.ring.clone(), c.lens.clone()
    q_out = torch.empty_like(q)
    c.append(q, *rest, i32([70, 40]), i32([0, 30, 60]), q_out=q_out)
    assert mla.get_device_error() == 7
    c.undo()
    assert torch.equal(c.ring, held[0]) and torch.equal(c.lens, held[1]) and torch.equal(q, q0)
    got = c.append(q, *rest, i32([41, 40]), i32([0, 1, 31]), q_out=q_out)
    want = never.append(q, *rest, i32([41, 40]), i32([0, 1, 31]), q_out=torch.empty_like(q))
    assert mla.get_device_error() == 0 and torch.equal(got, want) and torch.equal(q, q0)
    for x, y in ((c.slot_map, never.slot_map), (c.lens, never.lens)):
        assert torch.equal(x, y)
    at = c.slot_map[:31].long()
    assert torch.equal(c.k[at], never.k[at]) and torch.equal(c.v[at], never.v[at])
