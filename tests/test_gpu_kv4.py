"""4-bit K/V caches: qsa_kv4_append bit by bit against its definition in 64 bits, and
qsa_sparse_attn_kv4 against attention in 64 bits over the values the cache stands for.

Attention tolerance per value: the output's bf16 rounding, 2^-8 |o|; the fp16 rounding
of each probability, 2^-11 sum_j p_j |v_j|; fp32 logits of 128 products (128 x 2^-24 x
log2(e) x scale x sum |q_d k_d|, at most 2^-12 for the inputs here, whose sums stay
below 20) and their exponentials, 2^-11 sum p |v| together with the sums.  K, V and the
queries enter exactly (products of 2 and 4 significant bits; queries keep 31 bits below
their row's largest).  A probability below 2^-27 of the largest lies in fp16's
subnormals after its factor 2^13: off by at most 2^-25 / 2^13 = 2^-38 of the largest,
for up to 2^11 tokens of |v| <= 11.25 together below 2^-23.
"""

import math

import pytest
import torch

import block_sparse_attention_key_b200 as qsa

import gpu_util as gu

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gu.ensure_built()


# ---------------------------------------------------------------- definition in 64 bits (CPU)

def _nearest(x, grid, first):
    """Index of the grid value nearest to x, of two as near the one whose code is even; what lies
    above the grid goes to its end (and is cut first: 64 bits cannot tell distances of 10^38 apart)."""
    x = x.clamp(max=2 * float(grid[-1]))
    off = (x[..., None] - grid).abs()
    odd = (torch.arange(len(grid)) + first) % 2
    return torch.where(off == off.amin(-1, keepdim=True), odd, 2).argmin(-1)


def _quantise(x):
    """bf16 rows of 128 -> (codes u8 [..., 64], scales u8 [..., 8])."""
    x = x.double().cpu().unflatten(-1, (8, 16))
    grid = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0.0)
    idx = _nearest(x.abs().amax(-1) / 6, grid, 1)
    code = _nearest((x / grid[idx][..., None]).abs(), E2M1.double(), 0)
    code = (code + 8 * torch.signbit(x)).to(torch.uint8)
    code = torch.where(finite[..., None], code, 0).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), torch.where(finite, idx + 1, 127).to(torch.uint8)


def _values(codes, scales):
    """What codes and scales stand for, fp64, same device."""
    lut = torch.cat((E2M1, -E2M1)).double().to(codes.device)
    x = torch.stack((lut[(codes & 15).long()], lut[(codes >> 4).long()]), -1).flatten(-2)
    return x * scales.view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)


# ---------------------------------------------------------------- append

def _cache(batch, hkv, cap, page=0, seed=0, spare=3):
    """Zero-filled cache with marks (0xEE) where nothing may be written; paged: pages in random order."""
    g = torch.Generator().manual_seed(seed)
    n = batch * (cap // page) + spare if page else batch
    shape = (n, hkv, page or cap)
    t = [torch.full((*shape, w), 0xEE, dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    table = None
    if page:
        table = torch.randperm(n, generator=g)[: batch * (cap // page)].view(batch, -1).to(torch.int32).cuda()
    return qsa.kv4_cache(*t, table, page, n if page else 0), t, table


def _row(table, page, seq, pos):
    return (int(table[seq, pos // page]), pos % page) if page else (seq, pos)


def _append(dims, cache, k, v, cu, start, n, ws=None):
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    qsa.qsa_kv4_append(dims, cache, k, v, i32(cu), i32(start), n, ws)


@pytest.mark.parametrize("hkv,page", [(1, 0), (4, 16), (3, 0), (8, 64)])
def test_append_writes_the_rounded_rows_and_nothing_else(hkv, page):
    batch, cap = 4, 192
    lens, start = [5, 0, 130, 1], [0, 7, 62, 191]
    cu = [2]
    for n in lens:
        cu.append(cu[-1] + n)
    n_tok = cu[-1] + 4                                   # rows before and behind belong to nobody
    g = torch.Generator(device="cuda").manual_seed(hkv)
    x = torch.empty((n_tok, 3, hkv, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    k, v = x[:, 0], x[:, 2]                              # strided, as a projection's slices
    dims = qsa.make_dims(batch, hkv, hkv, cap)
    cache, (kc, ks, vc, vs), table = _cache(batch, hkv, cap, page, seed=hkv)
    ws = gu.new_workspace(256)
    _append(dims, cache, k, v, cu, start, n_tok, ws)
    assert qsa.qsa_read_device_status(ws) == 0
    want = [torch.full_like(t, 0xEE).cpu() for t in (kc, ks, vc, vs)]
    for s in range(batch):
        for i in range(lens[s]):
            p, r = _row(table, page, s, start[s] + i)
            want[0][p, :, r], want[1][p, :, r] = _quantise(k[cu[s] + i])
            want[2][p, :, r], want[3][p, :, r] = _quantise(v[cu[s] + i])
    for got, w in zip((kc, ks, vc, vs), want):
        assert torch.equal(got.cpu(), w)


def test_append_rounds_borders_ties_and_extremes_as_defined():
    bf = torch.bfloat16
    rows = [torch.zeros(128), torch.full((128,), -0.0), torch.full((128,), 3.3e38), torch.full((128,), 2.0 ** -133)]
    rows.append(torch.linspace(-1, 1, 128) * 2.0 ** -11)          # scales at their lower end
    rows.append(torch.linspace(-3000, 3000, 128))                 # and at their upper end
    g = torch.Generator().manual_seed(1)
    for s in (1.0, 0.8125, 2.0 ** -9, 3 * 2.0 ** -9, 448.0):
        # every border of two codes times the scale, with 6 s in each block
        t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0, 0.26])
        blk = torch.cat((t, torch.tensor([6.0]))) * s
        rows += [torch.cat([blk * (1 if i % 2 else -1) for i in range(8)])]
    for s in range(1, 120):                                       # block maxima around the borders of two scales
        a = torch.tensor([s], dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        b = torch.tensor([s + 1], dtype=torch.uint8).view(torch.float8_e4m3fn).float()
        top = ((a + b) / 2 * 6).to(bf).float()
        steps = torch.tensor([0, -1, 1, -2, 2, 3, -3, 4]) * top * 2.0 ** -8
        x = torch.randn((8, 16), generator=g) * 0.2 * top
        x[:, 5] = top + steps
        rows.append(x.flatten())
    x = torch.stack(rows).to(bf)
    bad = x[:4].clone()
    bad[0, 3], bad[0, 40], bad[1, 127], bad[2, 16] = math.nan, math.inf, -math.inf, math.nan
    x = torch.cat((x, bad)).cuda()[:, None, :].contiguous()
    n = x.shape[0]
    dims = qsa.make_dims(1, 1, 1, 256)
    cache, (kc, ks, vc, vs), _ = _cache(1, 1, 256)
    _append(dims, cache, x, x, [0, n], [0], n)
    codes, scales = _quantise(x[:, 0])
    for c, s in ((kc, ks), (vc, vs)):
        assert torch.equal(s[0, 0, :n].cpu(), scales)
        assert torch.equal(c[0, 0, :n].cpu(), codes)


def test_append_reports_and_skips_bad_lengths_and_pages():
    dims = qsa.make_dims(2, 2, 2, 64)
    k = torch.ones((40, 2, 128), dtype=torch.bfloat16, device="cuda")
    ws = gu.new_workspace(256)
    for cu, start, seqs in (([0, 30, 20], [0, 0], [0]), ([0, 20, 41], [0, 0], [0]), ([0, 20, 40], [0, 45], [0]),
                            ([0, 20, 40], [-1, 0], [1]), ([-3, 20, 40], [0, 0], [1])):
        cache, t, _ = _cache(2, 2, 64)
        _append(dims, cache, k, k, cu, start, 40, ws)
        assert qsa.qsa_read_device_status(ws) == qsa.qsa.QSA_DEV_BAD_LEN, (cu, start)
        for s in range(2):
            touched = (t[1][s] != 0xEE).any().item()
            assert touched == (s in seqs), (cu, start)
    cache, t, table = _cache(2, 2, 64, page=16)
    table[0, 1], table[1, 0] = -1, 99
    _append(dims, cache, k, k, [0, 20, 40], [0, 10], 40, ws)
    assert qsa.qsa_read_device_status(ws) == qsa.qsa.QSA_DEV_BAD_PAGE
    written = (t[1] != 0xEE).all(-1).sum().item()
    assert written == 2 * (16 + 14)


def test_append_finds_sequences_among_many():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 3, (2100,), generator=g)
    cu = [0, *lens.cumsum(0).tolist()]
    n = cu[-1]
    start = torch.randint(0, 14, (2100,), generator=g).tolist()
    dims = qsa.make_dims(2100, 1, 1, 16)
    x = torch.empty((n, 1, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    cache, (kc, ks, vc, vs), _ = _cache(2100, 1, 16)
    _append(dims, cache, x, x, cu, start, n)
    codes, scales = _quantise(x[:, 0])
    want_c, want_s = torch.full((2100, 16, 64), 0xEE, dtype=torch.uint8), torch.full((2100, 16, 8), 0xEE, dtype=torch.uint8)
    for s in range(2100):
        for i in range(lens[s]):
            want_c[s, start[s] + i], want_s[s, start[s] + i] = codes[cu[s] + i], scales[cu[s] + i]
    assert torch.equal(kc[:, 0].cpu(), want_c) and torch.equal(vs[:, 0].cpu(), want_s)


# ---------------------------------------------------------------- attention

def _fill(t, seed):
    """Random codes under scales of 2^-3 to 2^0.8 (values of either sign up to about 10)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    for i, x in enumerate(t):
        lo, hi = ((0, 256), (0x20, 0x3F))[i % 2]
        x.copy_(torch.randint(lo, hi, x.shape, generator=g, device="cuda", dtype=torch.uint8))


def _case(batch, hq, hkv, cap, page, bs, topk, group, t0s, seed):
    """Cache, queries and selections: for each group, blocks drawn below its first position."""
    g = torch.Generator().manual_seed(seed)
    dims = qsa.make_dims(batch, hq, hkv, cap, block_size=bs, top_k=topk)
    cache, t, table = _cache(batch, hkv, cap, page, seed)
    _fill(t, seed)
    q_seq, q_pos, sel, cnt = [], [], [], []
    for i, t0 in enumerate(t0s):
        n_c = (t0 + 1) // bs
        n = min(topk, n_c)
        pick = torch.randperm(max(n_c, 1), generator=g)[:n].sort().values if n else torch.zeros(0, dtype=torch.long)
        sel.append(torch.cat((pick, torch.full((512 - n,), -1))))
        cnt.append(n)
        for j in range(group):
            q_seq.append(i % batch)
            q_pos.append(min(t0 + j, bs * n_c + 2 * bs - 1))
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32).cuda()  # noqa: E731
    q = torch.empty((len(q_pos), hq, 128), dtype=torch.bfloat16, device="cuda").normal_(
        0, 0.25, generator=torch.Generator(device="cuda").manual_seed(seed))
    return dict(dims=dims, cache=cache, t=t, table=table, page=page, bs=bs, group=group, q=q, q_seq=i32(q_seq),
                q_pos=i32(q_pos), sel=i32(torch.stack(sel)), cnt=i32(cnt), hkv=hkv, hq=hq)


def _attend(c, flags=0, **kw):
    n = c["q"].shape[0]
    out = torch.full((n, c["hq"], 128), 55.0, dtype=torch.bfloat16, device="cuda")
    ws = gu.new_workspace(256)
    qsa.qsa_sparse_attn_kv4(c["dims"], c["cache"], c["q"], c["q_seq"], c["q_pos"], c["sel"], c["cnt"], n, out, ws,
                            group_q=c["group"], **kw)
    assert qsa.qsa_read_device_status(ws) == flags
    return out


def _tokens(c, i):
    grp = i // c["group"]
    first = (int(c["q_pos"][grp * c["group"]]) + 1) // c["bs"] * c["bs"]
    blocks = c["sel"][grp, : int(c["cnt"][grp])].cpu().long()
    tok = (blocks[:, None] * c["bs"] + torch.arange(c["bs"])).flatten()
    return torch.cat((tok, torch.arange(first, max(first, int(c["q_pos"][i]) + 1)))).cuda()


def _exact(c, i):
    """(output, sum p |v|) of query i in 64 bits."""
    tok, s = _tokens(c, i), int(c["q_seq"][i])
    out = torch.zeros((c["hq"], 128), dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    if not len(tok):
        return out, mag
    if c["page"]:
        page, row = c["table"][s].long()[tok // c["page"]], tok % c["page"]
    else:
        page, row = torch.full_like(tok, s), tok
    kc, ks, vc, vs = (t[page, :, row] for t in c["t"])
    k, v = _values(kc, ks), _values(vc, vs)
    per = c["hq"] // c["hkv"]
    for h in range(c["hq"]):
        p = torch.softmax(k[:, h // per] @ c["q"][i, h].double() * 128 ** -0.5, 0)
        out[h], mag[h] = p @ v[:, h // per], p @ v[:, h // per].abs()
    return out, mag


def _compare(c, out, rows=None):
    for i in rows if rows is not None else range(out.shape[0]):
        want, mag = _exact(c, i)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -11) * mag + 2.0 ** -23
        err = (out[i].double() - want).abs()
        assert (err <= tol).all(), f"query {i}: worst {(err / tol).max().item():.3f} of the tolerance"


T0S = [0, 2, 3, 1200, 2047, 4001, 777]


@pytest.mark.parametrize("hq,hkv,group", [(8, 1, 1), (32, 4, 1), (16, 16, 1), (32, 4, 4), (16, 4, 3), (12, 2, 2), (32, 1, 1),
                                          (14, 2, 2), (5, 5, 8)])
@pytest.mark.parametrize("page", [0, 16, 256])
def test_head_layouts_drafts_and_pages(hq, hkv, group, page):
    c = _case(3, hq, hkv, 4096 + 256, page, 4, 512, group, T0S, hq + group)
    _compare(c, _attend(c))


@pytest.mark.parametrize("bs,topk", [(1, 512), (1, 3), (2, 100), (8, 512), (16, 64), (16, 512), (4, 1)])
def test_block_sizes_and_budgets(bs, topk):
    c = _case(2, 8, 2, 8448, 0, bs, topk, 2, [8190, 31, 5000, 1], bs * 7 + topk)
    _compare(c, _attend(c))


@pytest.mark.parametrize("n,hq,hkv", [(1, 8, 1), (37, 16, 4), (148, 8, 1), (200, 32, 2), (300, 16, 1)])
def test_query_counts_from_split_rows_to_chunks(n, hq, hkv):
    """One query up to a chunk: split lists merged in a cluster, then one CTA per pair."""
    g = torch.Generator().manual_seed(n)
    t0s = torch.randint(0, 3000, (n,), generator=g).tolist()
    c = _case(2, hq, hkv, 3200, 0, 4, 512, 1, t0s, n)
    _compare(c, _attend(c), rows=range(0, n, max(1, n // 25)))


@pytest.mark.parametrize("lists", [148, 149, 296, 297])
@pytest.mark.parametrize("hq,group", [(4, 2), (16, 1), (16, 2), (11, 2)])
def test_every_launch_shape(hq, group, lists):
    """Row tiles of 8, 16 and 32 in the CTAs of few, of some and of many lists."""
    g = torch.Generator().manual_seed(lists + hq)
    t0s = torch.randint(0, 2300, (lists,), generator=g).tolist()
    c = _case(2, hq, 1, 2304, 16, 4, 512, group, t0s, lists * hq)
    _compare(c, _attend(c), rows=range(0, lists * group, 13))


def test_every_code_and_scale_reads_as_its_value():
    """One visible token: the output is V's value exactly (6 significant bits fit bf16)."""
    n = 256 * 8
    dims = qsa.make_dims(1, 1, 1, n, block_size=1)
    cache, (kc, ks, vc, vs), _ = _cache(1, 1, n)
    kc.zero_(), ks.fill_(0x38)
    tok = torch.arange(n, device="cuda")
    scale = (tok[:, None] // 16 + torch.arange(8, device="cuda")) % 128          # every e4m3 scale of either...
    vs.copy_((scale + 128 * (tok[:, None] % 2)).to(torch.uint8)[None, None])     # ...sign
    byte = (tok[:, None] * 37 + torch.arange(64, device="cuda") * 5) % 256
    vc.copy_(byte.to(torch.uint8)[None, None])
    pos = tok.to(torch.int32)
    sel = torch.full((n, 512), -1, dtype=torch.int32, device="cuda")
    sel[:, 0] = pos
    q = torch.zeros((n, 1, 128), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    qsa.qsa_sparse_attn_kv4(dims, cache, q, torch.zeros_like(pos), pos, sel, torch.ones_like(pos), n, out)
    want = _values(vc, vs)[0]
    got = out[:, 0].double()
    assert torch.equal(got.isnan(), want[0].isnan())
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want[0]))


def test_queries_of_any_magnitude():
    c = _case(1, 8, 1, 1024, 0, 4, 512, 1, [1000, 900], 3)
    c["q"][0, 0] *= 2.0 ** 9                               # beyond fp16's range after the logits' scale
    c["q"][0, 1] = 0
    c["q"][0, 2] *= 2.0 ** -90
    c["q"][0, 3] *= 2.0 ** -126
    c["q"][0, 4, ::2] *= 2.0 ** -30
    out = _attend(c)
    for i in range(2):
        want, mag = _exact(c, i)
        # row 0 of query 0: sum |q_d k_d| scale up to 2^14 puts 2^14 x 128 x 2^-24 x 1.44 = 0.18 into an exponent
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * mag + 2.0 ** -23
        if i == 0:
            tol[0] += 0.2 * mag[0]
        assert ((out[i].double() - want).abs() <= tol).all()
    c["q"][1, 5, 7] = math.nan
    c["q"][1, 6, 7] = math.inf
    c["t"][0][..., 3] = 0x22                               # dims 6, 7 of K: 1.0 times its scale
    out = _attend(c)
    assert out[1, 5].isnan().all() and out[1, 6].isnan().all()
    assert torch.isfinite(out[1, [0, 1, 2, 3, 4, 7]]).all()


def test_rows_that_attend_nothing_are_zero():
    c = _case(2, 8, 2, 512, 0, 4, 512, 1, [3, 7, 400], 4)
    c["cnt"][:2] = 0                                       # position 3 and 7 end a block: no tail either
    out = _attend(c)
    assert (out[:2] == 0).all()
    _compare(c, out)


def test_bad_indices_are_reported_and_skipped():
    c = _case(2, 8, 2, 512, 16, 4, 512, 1, [400, 300, 200, 100], 5)
    good = _attend(c)
    f = qsa.qsa
    for field, i, val, bit in (("q_seq", 1, 2, f.QSA_DEV_BAD_SEQ), ("q_seq", 1, -1, f.QSA_DEV_BAD_SEQ),
                               ("q_pos", 1, 512, f.QSA_DEV_BAD_POS), ("q_pos", 1, -5, f.QSA_DEV_BAD_POS),
                               ("cnt", 1, 513, f.QSA_DEV_BAD_SEL), ("cnt", 1, -1, f.QSA_DEV_BAD_SEL)):
        keep = c[field].clone()
        c[field][i] = val
        out = _attend(c, bit)
        c[field] = keep
        assert torch.equal(out[[0, 2, 3]], good[[0, 2, 3]])
    keep = c["sel"].clone()
    c["sel"][1, 3], c["sel"][1, 7] = 1 << 30, -9           # blocks that do not exist
    out = _attend(c, f.QSA_DEV_BAD_SEL)
    c["sel"] = torch.cat((keep[:, :3], keep[:, 4:7], keep[:, 8:], torch.full((4, 2), -1, device="cuda", dtype=torch.int32)), 1)
    want = c["sel"].clone()
    c["sel"][[0, 2, 3]] = keep[[0, 2, 3]]
    c["sel"] = c["sel"].contiguous()
    c["cnt"][1] -= 2
    _compare(c, out, rows=[1])
    assert torch.equal(want[1], c["sel"][1])
    c["table"][int(c["q_seq"][2]), 0] = 1 << 20
    c["sel"] = keep
    c["cnt"][1] += 2
    _attend(c, f.QSA_DEV_BAD_PAGE)


def test_skipped_drafts_are_zero_and_leave_the_others_alone():
    """A draft of another sequence, before its group or too far behind it, beside valid ones."""
    f = qsa.qsa
    for ns, t0s in ((1, [1501]), (40, [1501] * 40)):       # split over a cluster, one CTA per pair
        c = _case(2, 16, 4, 2048, 0, 4, 512, 4, t0s, 13)
        good = _attend(c)
        _compare(c, good, rows=range(4))
        for field, val, bit in (("q_seq", 1, f.QSA_DEV_BAD_SEQ), ("q_pos", 1500, f.QSA_DEV_BAD_POS),
                                ("q_pos", 1508, f.QSA_DEV_BAD_POS)):
            keep = c[field].clone()
            c[field][2] = val
            out = _attend(c, bit)
            c[field] = keep
            assert (out[2] == 0).all()
            rest = [i for i in range(out.shape[0]) if i != 2]
            assert torch.equal(out[rest], good[rest])


def test_two_streams_and_a_graph_at_once():
    """Calls that overlap on the GPU share nothing."""
    cases = [_case(3, 32, 4, 2304, page, 4, 512, 1, [2000, 900, 2200], 20 + page) for page in (0, 16)]
    want = [_attend(c) for c in cases]
    outs = [torch.empty_like(w) for w in want]

    def call(i, **kw):
        c = cases[i]
        qsa.qsa_sparse_attn_kv4(c["dims"], c["cache"], c["q"], c["q_seq"], c["q_pos"], c["sel"], c["cnt"], 3, outs[i], **kw)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(0)
    side = torch.cuda.Stream()
    for _ in range(50):
        graph.replay()
        call(1, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_drafts_do_not_see_what_lies_behind_them():
    """A tail token that is not finite reaches the drafts at and behind it only."""
    c = _case(1, 8, 2, 512, 0, 4, 512, 4, [301], 6)        # drafts at 301..304, tail from 300
    clean = _attend(c)
    for what in (1, 3):
        kept = c["t"][what].clone()
        c["t"][what][0, 0, 303, 2] = 0x7F                  # KV head 0, token 303, dims 32..47
        c["t"][what][0, 1, 305, 0] = 0xFF                  # a token no draft sees
        out = _attend(c)
        c["t"][what].copy_(kept)
        assert torch.equal(out[:2], clean[:2])
        assert torch.equal(out[2:, 4:], clean[2:, 4:])
        if what == 1:
            assert out[2:, :4].isnan().all()
        else:
            assert out[2:, :4, 32:48].isnan().all()
            assert torch.equal(out[2:, :4, :32], clean[2:, :4, :32])
            assert torch.equal(out[2:, :4, 48:], clean[2:, :4, 48:])


def test_a_cache_whose_offsets_pass_32_bits():
    """Codes beyond 4 GiB: the last pages of a pool of 4.3 GiB, and the last rows of a dense cache."""
    hkv, page = 8, 256
    n_pages = (1 << 32) // (hkv * page * 64) + 200
    t = [torch.zeros((n_pages, hkv, page, w), dtype=torch.uint8, device="cuda") for w in (64, 8, 64, 8)]
    table = torch.arange(n_pages - 4, n_pages, dtype=torch.int32, device="cuda").view(1, 4)
    c = _case(1, 8, hkv, 1024, 0, 4, 512, 1, [1000], 7)
    c.update(cache=qsa.kv4_cache(*t, table, page, n_pages), t=t, table=table, page=page)
    for x in t:
        tail = x[n_pages - 4:]
        _fill([tail] if x.shape[-1] == 64 else [torch.empty(0, dtype=torch.uint8, device="cuda"), tail], 9)
    _compare(c, _attend(c))
    k = torch.ones((1, hkv, 128), dtype=torch.bfloat16, device="cuda")
    _append(c["dims"], c["cache"], k, k, [0, 1], [1001], 1)
    codes, scales = _quantise(k[0, 0])
    assert torch.equal(t[0][n_pages - 1, 3, 1001 - 768].cpu(), codes)
    assert torch.equal(t[3][n_pages - 1, 7, 1001 - 768].cpu(), scales)
    assert not t[0][: n_pages - 4].any()


def test_append_select_attend_run_together_and_replay():
    """A decode step as a server runs it: append the new rows, pool, select, attend; as a graph
    replayed with other rows, on another stream."""
    batch, hq, hkv, cap = 3, 16, 2, 1024
    dims = qsa.make_dims(batch, hq, hkv, cap)
    cache, t, table = _cache(batch, hkv, cap, 64, 8)
    g = torch.Generator(device="cuda").manual_seed(8)
    rnd = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=g)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    hist = [900, 37, 1000]
    cu = [0, 900, 937, 1937]
    _append(dims, cache, rnd(1937, hkv, 128), rnd(1937, hkv, 128), cu, [0, 0, 0], 1937)
    idx_k, pooled = rnd(batch, cap, 64), torch.zeros((batch, cap // 4, 64), dtype=torch.bfloat16, device="cuda")
    qsa.qsa_pool_block_keys(dims, idx_k, pooled, i32([0, 0, 0]), i32(hist), cap)
    k, v, q, q_idx = rnd(3, hkv, 128), rnd(3, hkv, 128), rnd(3, hq, 128), rnd(3, 4, 64)
    w = torch.ones((3, 4), device="cuda")
    before, pos, seq, one = i32(hist), i32(hist), i32([0, 1, 2]), i32([0, 1, 2, 3])
    after = before + 1
    sel, cnt = torch.empty((3, 512), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")
    out = torch.empty((3, hq, 128), dtype=torch.bfloat16, device="cuda")
    ws = gu.new_workspace(qsa.qsa_workspace_bytes(dims, 3, cap // 4, qsa.QSA_MODE_DECODE))

    def step():
        qsa.qsa_kv4_append(dims, cache, k, v, one, before, 3, ws)
        qsa.qsa_pool_block_keys(dims, idx_k, pooled, before, after, 1, ws)
        qsa.qsa_select_blocks(dims, q_idx, w, pooled, seq, pos, 3, cap // 4, qsa.QSA_MODE_DECODE, sel, cnt, ws)
        qsa.qsa_sparse_attn_kv4(dims, cache, q, seq, pos, sel, cnt, 3, out, ws)

    def check():
        assert qsa.qsa_read_device_status(ws) == 0
        c = dict(dims=dims, cache=cache, t=t, table=table, page=64, bs=4, group=1, q=q, q_seq=seq, q_pos=pos, sel=sel,
                 cnt=cnt, hkv=hkv, hq=hq)
        for s in range(3):
            p, r = _row(table, 64, s, int(pos[s]))
            assert torch.equal(t[0][p, :, r].cpu(), _quantise(k[s])[0])
        _compare(c, out)

    step()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        step()
    for x in (k, v, q, q_idx):
        x.copy_(rnd(*x.shape))
    before.add_(1), after.add_(1), pos.add_(1)
    graph.replay()
    torch.cuda.synchronize()
    check()


@pytest.mark.parametrize("n,hq,hkv,group", [(1, 8, 1, 1), (1, 16, 2, 4), (160, 16, 1, 1), (300, 8, 1, 1)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_of_any_size(n, hq, hkv, group, sign):
    """Logits from 2^4 to 2^80, two values of them per row: all weight on the larger one's tokens, in
    equal parts.  Equal K rows give equal fp32 sums, so the expected output needs no tolerance for logits."""
    c = _case(2, hq, hkv, 1280, 16, 4, 512, group, [1201] * n, 31)
    kc, ks = c["t"][:2]
    kc.fill_(0x22), ks.fill_(0x38)                         # every K value 1
    half = torch.rand(ks.shape[:-1], generator=torch.Generator(device="cuda").manual_seed(4), device="cuda") < 0.5
    ks[half] = 0x30                                        # or 1/2
    mag = 2.0 ** torch.linspace(4, 80, n * group * hq, device="cuda").round().view(n * group, hq)
    c["q"] = (sign * mag[..., None]).expand(-1, -1, 128).to(torch.bfloat16).contiguous()
    out = _attend(c)
    for i in range(0, n * group, max(1, n // 20)):
        tok, s = _tokens(c, i), int(c["q_seq"][i])
        page, row = c["table"][s].long()[tok // 16], tok % 16
        v = _values(c["t"][2][page, :, row], c["t"][3][page, :, row])
        for h in range(hq):
            low = half[page, h // (hq // hkv), row]
            # 2^4: the logits differ by 2^3 x 128 x 128^-0.5 = 90, of which exp leaves nothing
            keep = v[low if sign < 0 else ~low, h // (hq // hkv)]
            want, size = keep.mean(0), keep.abs().mean(0)
            # equal probabilities 2^13 and fp32 sums (2^-24 a token) below the output's rounding
            tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * size + 2.0 ** -23
            assert ((out[i, h].double() - want).abs() <= tol).all(), (i, h)


@pytest.mark.parametrize("scale", [1e-10, 1e-18, 1e-38])
def test_logit_scales_next_to_nothing(scale):
    """Rows of zeros and of tiny values under a tiny scale: all logits are 0, masked places stay out."""
    c = _case(2, 8, 2, 512, 16, 4, 512, 2, [301, 7, 130], 32)
    c["dims"].softmax_scale = scale
    c["q"][:, ::2] = 0
    c["q"][:, 1::2] *= 2.0 ** -100
    out = _attend(c)
    for i in range(out.shape[0]):
        tok, s = _tokens(c, i), int(c["q_seq"][i])
        page, row = c["table"][s].long()[tok // 16], tok % 16
        v = _values(c["t"][2][page, :, row], c["t"][3][page, :, row]).repeat_interleave(4, 1)
        want, size = v.mean(0), v.abs().mean(0)
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -11 * size + 2.0 ** -23
        assert ((out[i].double() - want).abs() <= tol).all(), i


@pytest.mark.parametrize("n_seq", [10, 40, 300])
@pytest.mark.parametrize("bound", ["raised", "lowered", "past the rows", "negative"])
def test_append_with_one_bad_bound_among_many_writes_only_what_some_sequence_names(n_seq, bound):
    """BAD_LEN, and every row is its old one or that of a sequence whose own bounds are in order."""
    g = torch.Generator().manual_seed(n_seq)
    cap = 64
    lens = torch.randint(1, 6, (n_seq,), generator=g).tolist()
    start = torch.randint(0, 8, (n_seq,), generator=g).tolist()
    cu, at = [2], n_seq // 2
    for x in lens:
        cu.append(cu[-1] + x)
    n = cu[-1] + 3
    cu[at] = {"raised": min(cu[-2], cu[at] + 40), "lowered": cu[at // 2], "past the rows": n + 1, "negative": -7}[bound]
    x = torch.empty((n, 2, 128), dtype=torch.bfloat16, device="cuda").normal_(generator=torch.Generator(device="cuda").manual_seed(3))
    dims = qsa.make_dims(n_seq, 2, 2, cap)
    cache, t, _ = _cache(n_seq, 2, cap)
    ws = gu.new_workspace(256)
    _append(dims, cache, x, x, cu, start, n, ws)
    assert qsa.qsa_read_device_status(ws) == qsa.qsa.QSA_DEV_BAD_LEN
    rows = _quantise(x)
    for i, got in enumerate(t):
        got, want = got.cpu(), rows[i % 2]
        fine = (got == 0xEE).all(-1)
        for s, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
            if 0 <= a <= b <= n and start[s] + b - a <= cap:
                to = slice(start[s], start[s] + b - a)
                fine[s, :, to] |= (got[s, :, to] == want[a:b].transpose(0, 1)).all(-1)
        assert fine.all()


def _exact_over(c, i, tok):
    """_exact over given tokens of query i's sequence (paged)."""
    s = int(c["q_seq"][i])
    page, row = c["table"][s].long()[tok // c["page"]], tok % c["page"]
    kc, ks, vc, vs = (t[page, :, row] for t in c["t"])
    per = c["hq"] // c["hkv"]
    k, v = _values(kc, ks).repeat_interleave(per, 1), _values(vc, vs).repeat_interleave(per, 1)
    p = torch.softmax(torch.einsum("thd,hd->ht", k, c["q"][i].double()) * 128 ** -0.5, 1)
    return torch.einsum("ht,thd->hd", p, v), torch.einsum("ht,thd->hd", p, v.abs())


@pytest.mark.parametrize("group", [1, 3])
@pytest.mark.parametrize("entry", [-1, 1 << 20, -(1 << 31)])
@pytest.mark.parametrize("place", [0, 18])
def test_tokens_of_a_page_that_is_not_there_are_left_out(place, entry, group):
    """A selected page, or the one of the tail: the sequence's queries attend their other tokens, the other
    sequences' give the same bits."""
    c = _case(2, 8, 2, 512, 16, 4, 512, group, [297, 290, 299, 120], 33)
    good = _attend(c)
    c["table"][0, place] = entry
    out = _attend(c, qsa.qsa.QSA_DEV_BAD_PAGE)
    for i in range(out.shape[0]):
        if int(c["q_seq"][i]) == 1:
            assert torch.equal(out[i], good[i])
            continue
        tok = _tokens(c, i)
        tok = tok[tok // 16 != place]
        want, mag = _exact_over(c, i, tok)
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -11) * mag + 2.0 ** -23
        assert ((out[i].double() - want).abs() <= tol).all(), i


@pytest.mark.parametrize("batch,group,hq,hkv", [(1, 1, 8, 1), (6, 2, 16, 2), (16, 1, 32, 4), (64, 1, 32, 4), (200, 3, 8, 2)])
def test_same_inputs_give_the_same_bits_whatever_runs_beside(batch, group, hq, hkv):
    """A cache per sequence, from split lists to many; the calls of two streams overlap."""
    g = torch.Generator().manual_seed(batch)
    t0s = torch.randint(200, 2400, (batch,), generator=g).tolist()
    c = _case(batch, hq, hkv, 2560, 64, 4, 512, group, t0s, batch)
    first = _attend(c)
    _compare(c, first, rows=range(0, batch * group, max(1, batch * group // 12)))
    outs = [torch.empty_like(first) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for out, st in zip(outs, streams):
            qsa.qsa_sparse_attn_kv4(c["dims"], c["cache"], c["q"], c["q_seq"], c["q_pos"], c["sel"], c["cnt"],
                                    first.shape[0], out, group_q=group, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)
