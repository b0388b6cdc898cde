"""qsa_pages_update and qsa_pages_compact against a sequential model of their rules, and
the property they exist for: whatever the steps, every sequence reads its own tokens."""

import random

import pytest
import torch

import block_sparse_attention_key_b200 as qsa

import gpu_util as gu

pytestmark = pytest.mark.gpu

BAD_SEQ, BAD_LEN, BAD_PAGE = (getattr(qsa.qsa, n) for n in ("QSA_DEV_BAD_SEQ", "QSA_DEV_BAD_LEN", "QSA_DEV_BAD_PAGE"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gu.ensure_built()


class Model:
    """The rules of include/qsa.h, one step after the other, on lists."""

    def __init__(self, batch, per_seq, n_pages, page):
        self.table = [[-1] * per_seq for _ in range(batch)]
        self.ref = [0] * n_pages
        self.page, self.cap = page, per_seq * page

    def update(self, free, forks, before, after):
        t, ref, flags, n = self.table, self.ref, 0, len(self.table)
        for s in free:
            if not 0 <= s < n:
                flags |= BAD_SEQ
                continue
            for i, e in enumerate(t[s]):
                if 0 <= e < len(ref):
                    ref[e] -= 1
                t[s][i] = -1
        named = [(a, b) for a, b in forks if 0 <= a < n and 0 <= b < n and a != b]
        sources, taken, holds = {a for a, _ in named}, set(), {b for _, b in named if any(e >= 0 for e in t[b])}
        for a, b in forks:
            if (a, b) not in named or b in sources or b in taken or b in holds:
                flags |= BAD_SEQ
                continue
            taken.add(b)
            t[b] = list(t[a])
            for e in t[a]:
                if e >= 0:
                    ref[e] += 1
        snap, free_ids = list(ref), [p for p, r in enumerate(ref) if r == 0]
        moves = []
        for s in range(n):
            lo, hi = before[s], after[s]
            if lo < 0 or hi < lo or hi > self.cap:
                flags |= BAD_LEN
                continue
            for i in range(lo // self.page, -(-hi // self.page)) if hi > lo else ():
                e = t[s][i]
                if e >= 0 and snap[e] <= 1:
                    continue
                if not free_ids:
                    flags |= BAD_PAGE
                    continue
                new = free_ids.pop(0)
                ref[new] = 1
                if e >= 0:
                    ref[e] -= 1
                    if i * self.page < lo:
                        moves.append((e, new))
                t[s][i] = new
        return flags, moves

    def compact(self):
        live = [p for p, r in enumerate(self.ref) if r > 0]
        n = len(live)
        holes = [p for p in range(n) if self.ref[p] == 0]
        moves = list(zip([p for p in live if p >= n], holes))
        new = dict(moves)
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.table = [[new.get(e, e) for e in row] for row in self.table]
        return n, moves


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Pool:
    """The library's state beside the model's."""

    def __init__(self, batch, per_seq, n_pages, page, widths=(48, 16), offset=0):
        self.m = Model(batch, per_seq, n_pages, page)
        self.dims = qsa.make_dims(batch, 1, 1, per_seq * page, block_size=1 if page % 4 else 4)
        self.table = torch.full((batch, per_seq), -1, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        self.data = [torch.randint(0, 256, (n_pages, page, w), dtype=torch.uint8, device="cuda") for w in widths]
        self.pools = qsa.page_pools(self.data, page, n_pages)
        self.ws = gu.new_workspace(qsa.qsa_pages_workspace_bytes(self.dims, page, n_pages))

    def update(self, free, forks, before, after):
        want = [d.clone() for d in self.data]
        flags, moves = self.m.update(free, forks, before, after)
        for d in want:
            for a, b in moves:
                d[b] = d[a].clone()
        qsa.qsa_pages_update(self.dims, self.pools, self.table, self.ref, _i32(before), _i32(after), self.ws,
                             free_seq=_i32(free), n_free=len(free), fork_src=_i32([a for a, _ in forks]),
                             fork_dst=_i32([b for _, b in forks]), n_fork=len(forks))
        assert qsa.qsa_read_device_status(self.ws) == flags
        self.same(want)
        return flags

    def compact(self):
        want = [d.clone() for d in self.data]
        n, moves = self.m.compact()
        for d in want:
            for a, b in moves:
                d[b] = d[a].clone()
        n_live = _i32([-7])
        qsa.qsa_pages_compact(self.dims, self.pools, self.table, self.ref, n_live, self.ws)
        assert n_live.item() == n
        self.same(want)

    def same(self, want):
        assert self.table.tolist() == self.m.table
        assert self.ref.tolist() == self.m.ref
        for d, w in zip(self.data, want):
            assert torch.equal(d, w)


@pytest.mark.parametrize("batch,per_seq,page,seed", [(1, 3, 16, 0), (7, 5, 4, 1), (40, 9, 16, 2), (300, 4, 8, 3), (3, 70, 1, 4),
                                                     (33, 33, 3, 5)])
def test_random_steps_keep_the_rules_and_every_sequences_tokens(batch, per_seq, page, seed):
    rng = random.Random(seed)
    n_pages = batch * per_seq // 2 + 2 * batch + 3
    p = Pool(batch, per_seq, n_pages, page)
    text = [[] for _ in range(batch)]                    # what each sequence's tokens should read
    stamp = 0
    for step in range(14):
        free = [s for s in range(batch) if rng.random() < (0.25 if text[s] else 0.02)]
        free += rng.sample(free, min(len(free), 1))      # one of them twice
        for s in free:
            text[s] = []
        empty = [s for s in range(batch) if not text[s]]
        full = [s for s in range(batch) if text[s]]
        forks = [(rng.choice(full), d) for d in rng.sample(empty, len(empty) // 2)] if full else []
        for a, b in forks:
            text[b] = list(text[a])
        before = [len(x) for x in text]
        after = [min(n + rng.choice((0, 1, 1, page, 2 * page + 1)), per_seq * page) for n in before]
        if p.update(free, forks, before, after):         # out of pages: nothing is appended
            after = before
        rows, places = [], []
        for s in range(batch):
            for t in range(before[s], after[s]):
                stamp = stamp % 250 + 1
                text[s].append(stamp)
                rows.append(stamp)
                places.append((p.m.table[s][t // page], t % page))
        if rows:
            at = torch.tensor(places, device="cuda")
            assert len(set(places)) == len(places)       # no two tokens in one place
            for d in p.data:
                d[at[:, 0], at[:, 1]] = torch.tensor(rows, dtype=torch.uint8, device="cuda")[:, None]
        if step % 4 == 3:
            p.compact()
        for d in p.data:
            got = d[..., -1].cpu()
            for s in range(batch):
                assert [int(got[p.m.table[s][t // page], t % page]) for t in range(len(text[s]))] == text[s]


def test_out_of_pages_serves_the_first_and_may_be_repeated():
    p = Pool(4, 4, 5, 8)
    assert p.update([], [], [0] * 4, [16, 16, 16, 0]) == BAD_PAGE      # six wanted, five there
    assert p.m.table[2] == [4, -1, -1, -1]
    assert p.update([0], [], [0, 16, 0, 0], [0, 16, 16, 0]) == 0       # room again: the rest is served
    assert p.update([1], [(2, 3)], [0] * 4, [0] * 4) == 0
    # both holders of the shared partial page append at once with one page free for two requests
    p.update([], [], [0] * 4, [16, 0, 0, 0])
    assert p.update([], [], [16, 0, 12, 12], [16, 0, 13, 13]) == BAD_PAGE
    assert p.update([0], [], [0, 0, 12, 12], [0, 0, 13, 13]) == 0


def test_bad_names_and_lengths_are_reported_and_skipped():
    p = Pool(5, 4, 20, 4)
    assert p.update([], [], [0] * 5, [9, 3, 0, 0, 0]) == 0
    assert p.update([-1, 5], [], [0] * 5, [0] * 5) == BAD_SEQ
    for forks in ([(0, 0)], [(0, 1)], [(0, 7)], [(-2, 2)], [(0, 2), (1, 2)], [(0, 3), (3, 4)]):
        p.update([2, 3, 4], [], [0] * 5, [0] * 5)
        assert p.update([], forks, [0] * 5, [0] * 5) == BAD_SEQ, forks
    for lens in (([-1, 0, 0, 0, 0], [4, 0, 0, 0, 0]), ([5, 0, 0, 0, 0], [4, 0, 0, 0, 0]), ([0] * 5, [17, 0, 2, 0, 0])):
        assert p.update([], [], *lens) == BAD_LEN
    p.table[1, 2] = 1 << 20                              # an entry no pool has: taken for none
    p.m.table[1][2] = -1
    qsa.qsa_pages_update(p.dims, p.pools, p.table, p.ref, _i32([0, 3, 0, 0, 0]), _i32([0, 12, 0, 0, 0]), p.ws)
    assert qsa.qsa_read_device_status(p.ws) == 0
    p.m.update([], [], [0, 3, 0, 0, 0], [0, 12, 0, 0, 0])
    p.same(p.data)


def test_entries_past_the_pool_are_reported_where_tokens_should_be():
    """Freed, forked, or appended to behind earlier tokens: taken for none and reported."""
    none = [0] * 4

    def step(p, before, after, free=(), forks=(), want=BAD_PAGE):
        data = [d.clone() for d in p.data]
        flags, moves = p.m.update(free, forks, before, after)
        assert flags == 0 and not moves                  # the model has -1 for an entry that the call looks at
        qsa.qsa_pages_update(p.dims, p.pools, p.table, p.ref, _i32(before), _i32(after), p.ws,
                             free_seq=_i32(free), n_free=len(free), fork_src=_i32([a for a, _ in forks]),
                             fork_dst=_i32([b for _, b in forks]), n_fork=len(forks))
        assert qsa.qsa_read_device_status(p.ws) == want
        p.same(data)

    for entry in (20, 1 << 20, (1 << 31) - 1):
        p = Pool(4, 4, 20, 4)
        assert p.update([], [], none, [10, 7, 0, 0]) == 0
        p.table[1, 1] = p.m.table[1][1] = entry          # its page stays counted: nothing names it any more
        step(p, [10, 7, 0, 0], [11, 7, 0, 0], want=0)    # nobody looks at it
        p.m.table[1][1] = -1
        step(p, [11, 7, 0, 0], [11, 9, 0, 0])            # tokens 4 to 6 should be in the place of token 7
        p.table[0, 2], p.m.table[0][2] = entry, -1
        p.m.table[2] = list(p.m.table[0])
        for e in p.m.table[2]:
            if e >= 0:
                p.m.ref[e] += 1
        data = [d.clone() for d in p.data]
        qsa.qsa_pages_update(p.dims, p.pools, p.table, p.ref, _i32(none), _i32(none), p.ws, fork_src=_i32([0]),
                             fork_dst=_i32([2]), n_fork=1)
        assert qsa.qsa_read_device_status(p.ws) == BAD_PAGE
        assert p.table[0, 2] == entry                    # the source keeps its entry
        p.table[0, 2] = -1
        p.same(data)
        p.table[2, 3] = entry
        step(p, none, none, free=[2])
        step(p, none, none, free=[2], want=0)            # emptied: not reported twice
        p.table[0, 3] = entry
        step(p, [12, 0, 0, 0], [13, 0, 0, 0], want=0)    # a place without tokens just gets a page


def test_a_rolled_back_sequence_leaves_its_siblings_pages_alone():
    """Speculation went past a page and is taken back into a shared one: the append copies it."""
    p = Pool(2, 4, 12, 4)
    p.update([], [], [0, 0], [10, 0])
    p.update([], [(0, 1)], [0, 0], [0, 0])
    assert p.update([], [], [0, 6], [0, 9]) == 0         # sequence 1 back to 6 tokens, appends three
    assert p.m.table[0][0] == p.m.table[1][0]
    assert len({*p.m.table[0][1:3], *p.m.table[1][1:3]}) == 4


def test_full_empty_and_single_page_pools_compact():
    p = Pool(2, 4, 8, 4, widths=(64,))
    p.compact()
    p.update([], [], [0, 0], [16, 16])
    p.compact()
    p.update([0], [], [0, 0], [0, 0])
    p.compact()
    p.update([1], [], [0, 0], [0, 0])
    p.compact()
    one = Pool(1, 1, 1, 4)
    one.update([], [], [0], [1])
    one.compact()


def test_more_sequences_and_longer_ranges_than_a_pass_covers():
    """1,500 sequences (scanned 1,024 at a time), one of them reserving 2,900 pages at once."""
    p = Pool(1500, 3000, 6000, 1, widths=(16,))
    after = [2] * 1500
    after[1200] = 2900
    assert p.update([], [], [0] * 1500, after) == 0
    free = [s for s in range(1500) if s % 3 == 0]
    assert p.update(free, [(1, 0), (1200, 3)], [0] * 1500, [0] * 1500) == 0
    before = [0 if s % 3 == 0 else 2 for s in range(1500)]
    before[0], before[3], before[1200] = 2, 2900, 0
    assert p.update([], [], before, [min(n + 1, 3000) if n else 0 for n in before]) == 0
    p.compact()


def test_large_pools_and_odd_page_sizes_move_whole():
    """Pages of 33,168 bytes (not a whole number of steps) beside ones of 16, over 20,000 pages."""
    p = Pool(64, 500, 20000, 1, widths=(16,))
    big = torch.randint(0, 256, (20000, 33168), dtype=torch.uint8, device="cuda")
    p.data.append(big)
    p.pools = qsa.page_pools(p.data, 1, 20000)
    p.update([], [], [0] * 64, [300] * 64)
    p.update([*range(0, 64, 2)], [], [0] * 64, [0] * 64)
    p.compact()


def test_captured_step_replays_on_the_state_it_finds():
    p = Pool(3, 8, 30, 4)
    p.update([], [], [0, 0, 0], [6, 9, 0])
    before, after = _i32([6, 9, 0]), _i32([7, 12, 0])
    n_live = _i32([0])
    # warm up on a copy of the state
    t, r = p.table.clone(), p.ref.clone()
    qsa.qsa_pages_update(p.dims, p.pools, t, r, before, before, p.ws)
    qsa.qsa_pages_compact(p.dims, p.pools, t, r, n_live, p.ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    free = _i32([2])
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        qsa.qsa_pages_update(p.dims, p.pools, p.table, p.ref, before, after, p.ws, free_seq=free, n_free=1)
        qsa.qsa_pages_compact(p.dims, p.pools, p.table, p.ref, n_live, p.ws)
    for lens in (([6, 9, 0], [7, 12, 0]), ([7, 12, 0], [20, 13, 3]), ([20, 13, 0], [21, 14, 0])):
        before.copy_(_i32(lens[0])), after.copy_(_i32(lens[1]))
        want = [d.clone() for d in p.data]
        for moves in (p.m.update([2], [], *lens)[1], p.m.compact()[1]):
            for d in want:
                for a, b in moves:
                    d[b] = d[a].clone()
        graph.replay()
        torch.cuda.synchronize()
        p.same(want)
        assert n_live.item() == sum(x > 0 for x in p.m.ref)


def test_a_forked_sequence_attends_its_own_continuation():
    """Fork, append to both into 4-bit pages, attend: each sequence sees its own tokens."""
    hkv, hq, page, cap = 2, 8, 16, 64
    dims = qsa.make_dims(3, hq, hkv, cap)
    n_pages = 12
    t = [torch.zeros((n_pages, hkv, page, w), dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    table = torch.full((3, cap // page), -1, dtype=torch.int32, device="cuda")
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    pools, cache = qsa.page_pools(t, page, n_pages), qsa.kv4_cache(*t, table, page, n_pages)
    ws = gu.new_workspace(max(qsa.qsa_pages_workspace_bytes(dims, page, n_pages),
                              qsa.qsa_workspace_bytes(dims, 3, cap // 4, qsa.QSA_MODE_DECODE)))
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    k, v = rnd(23, hkv, 128), rnd(23, hkv, 128)

    def append(lens, new, **kw):
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        qsa.qsa_pages_update(dims, pools, table, ref, _i32(lens), _i32([a + b for a, b in zip(lens, new)]), ws, **kw)
        return cu

    cu = append([0, 0, 0], [21, 0, 0])
    qsa.qsa_kv4_append(dims, cache, k[:21].contiguous(), v[:21].contiguous(), _i32(cu), _i32([0, 0, 0]), 21, ws)
    cu = append([21, 21, 0], [1, 1, 0], fork_src=_i32([0]), fork_dst=_i32([1]), n_fork=1)
    qsa.qsa_kv4_append(dims, cache, k[21:].contiguous(), v[21:].contiguous(), _i32(cu), _i32([21, 21, 0]), 2, ws)
    n_live = _i32([0])
    qsa.qsa_pages_update(dims, pools, table, ref, _i32([0, 22, 0]), _i32([0, 22, 0]), ws, free_seq=_i32([2, 2]), n_free=2)
    qsa.qsa_pages_compact(dims, pools, table, ref, n_live, ws)
    assert n_live.item() == 3                             # one whole page shared, a partial one each
    q = rnd(2, hq, 128)
    sel = torch.full((2, 512), -1, dtype=torch.int32, device="cuda")
    sel[:, :5] = torch.arange(5)
    out = torch.empty_like(q)
    qsa.qsa_sparse_attn_kv4(dims, cache, q, _i32([0, 1]), _i32([21, 21]), sel, _i32([5, 5]), 2, out, ws)
    assert qsa.qsa_read_device_status(ws) == 0
    # the same tokens in a dense cache
    flat = [torch.zeros((3, hkv, cap, w), dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    dense = qsa.kv4_cache(*flat)
    for s in range(2):
        rows = torch.cat((k[:21], k[21 + s:22 + s])), torch.cat((v[:21], v[21 + s:22 + s]))
        qsa.qsa_kv4_append(dims, dense, *rows, _i32([0] * (s + 1) + [22] * (3 - s)), _i32([0, 0, 0]), 22, ws)
    want = torch.empty_like(q)
    qsa.qsa_sparse_attn_kv4(dims, dense, q, _i32([0, 1]), _i32([21, 21]), sel, _i32([5, 5]), 2, want, ws)
    assert qsa.qsa_read_device_status(ws) == 0
    assert torch.equal(out, want) and not torch.equal(out[0], out[1])
