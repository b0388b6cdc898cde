"""The serving operators around the sparse layer, as measured cases: their inputs, their
plain forms in elementary torch operations, and the library's calls.

prompt   qsa_prompt_attn: causal attention over whole prompts of different lengths, packed
append   qsa_kv4_append: K/V rows of new tokens rounded to 4 bits into a (paged) cache
attend   qsa_sparse_attn_kv4: attention over the selected blocks of such a cache
update   qsa_pages_update: a scheduler's step on a paged cache (free, fork, reserve with
         copy-on-write)
compact  qsa_pages_compact: live pages moved to the front of their pools

A 4-bit row of 128 values is 64 bytes of e2m1 codes (value 2i in the low half of byte i)
and 8 e4m3 scales, one for each 16 values.
"""

import math

import torch

own = False

D = 128
CAP = 512                        # entries of a selection row
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
HEADS = ((8, 1), (32, 4), (16, 16), (4, 2), (64, 8), (12, 4))


# ---------------------------------------------------------------- cases

def listed():
    return [
        # four short chat turns admitted together: the launch's latency counts
        dict(name="prompt_short", op="prompt", lens="1,17,64,40", hq=8, hkv=1),
        # sixteen requests of different lengths packed into one prefill batch, one KV head per query head
        dict(name="prompt_packed", op="prompt", hq=16, hkv=16,
             lens="1021,37,512,260,3,799,128,129,640,1,345,77,911,256,190,515"),
        # one long document, the head layout of the 64K decode workload
        dict(name="prompt_8k", op="prompt", lens="8192", hq=32, hkv=4),
        # the K/V of one decode step of 16 sequences; of their pages of 256 tokens, the last ones
        dict(name="append_decode", op="append", batch=16, new=1, cap=256, hkv=4, page=256),
        # a prefill chunk of four prompts written at once, dense caches
        dict(name="append_prompt", op="append", batch=4, new=2048, cap=2304, hkv=8, page=0),
        # one sequence at 8K, two draft tokens sharing a selection
        dict(name="attend_8k_b1", op="attend", batch=1, nq=2, group=2, ctx=8192, hq=8, hkv=1, bs=4, topk=512, page=0),
        # the headline decode step over a 4-bit cache in pages
        dict(name="attend_64k_b16", op="attend", batch=16, nq=16, group=1, ctx=65536, hq=32, hkv=4, bs=4, topk=512,
             page=256),
        # a prefill chunk over a 4-bit cache
        dict(name="attend_prefill", op="attend", batch=1, nq=1024, group=1, ctx=32768, hq=32, hkv=4, bs=4, topk=512,
             page=0),
        # a decode step of a small server: one request ends, one is forked into its slot
        dict(name="update_b16", op="update", batch=16, ctx=8192, page=256, hkv=1, free=1, fork=1, new=1),
        # a large server on small pages: a quarter of the slots turn over, half of those by forks
        dict(name="update_b128", op="update", batch=128, ctx=8192, page=32, hkv=4, free=32, fork=16, new=33),
        # a small pool with holes
        dict(name="compact_small", op="compact", batch=8, ctx=4096, page=64, hkv=2, live=0.5),
        # half of a pool's pages died; the cache gives the upper half back
        dict(name="compact_large", op="compact", batch=64, ctx=16384, page=128, hkv=8, live=0.5),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append", "attend", "attend", "update", "compact"))
    hq, hkv = rng.choice(HEADS)
    if op == "prompt":
        left = _log(rng, 1, 8192 * 32 // hq if hq > 32 else 8192)
        lens = []
        while left > 0 and len(lens) < 24:
            n = min(left, _log(rng, 1, left))
            lens.append(n)
            left -= n
        rng.shuffle(lens)
        return dict(op=op, lens=",".join(map(str, lens)), hq=hq, hkv=hkv)
    if op == "append":
        batch, new = _log(rng, 1, 64), _log(rng, 1, 2048)
        new = max(1, min(new, 65536 // (batch * hkv)))
        page = rng.choice((0, 16, 256))
        return dict(op=op, batch=batch, new=new, cap=-(-(new + rng.randint(0, 300)) // 256) * 256, hkv=hkv, page=page)
    if op == "attend":
        bs = rng.choice((1, 2, 4, 4, 4, 8, 16))
        group = rng.choice([g for g in (1, 1, 2, 3, 4) if g * (hq // hkv) <= 32])
        many = rng.random() < 0.3
        batch = 1 if many else _log(rng, 1, 16)
        nq = group * (_log(rng, 40, 1024 * 4 // max(hkv, 4) // group) if many else batch)
        ctx = max(64, _log(rng, 64, 32768) // 16 * 16)
        topk = rng.choice((512, 512, 100, 7)) if bs < 8 else rng.choice((256, 64))
        return dict(op=op, batch=batch, nq=nq, group=group, ctx=ctx, hq=hq, hkv=hkv, bs=bs, topk=topk,
                    page=rng.choice((0, 16, 256) if ctx % 256 == 0 else (0, 16)))
    if op == "update":
        batch, page = _log(rng, 2, 128), rng.choice((16, 32, 64, 256))
        free = rng.randint(0, batch // 2)
        return dict(op=op, batch=batch, ctx=_log(rng, page, 8192 // page * page) // page * page + page, page=page,
                    hkv=rng.choice((1, 2, 4)), free=free, fork=rng.randint(0, free), new=rng.choice((1, 1, 5, 40)))
    page = rng.choice((16, 64, 128))
    return dict(op=op, batch=_log(rng, 1, 64), ctx=max(page, _log(rng, page, 16384) // page * page), page=page,
                hkv=rng.choice((1, 2, 8)), live=rng.choice((0.05, 0.5, 0.9)))


# ---------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _rand_table(g, batch, per_seq, n_pages):
    """Distinct pages of a pool for every place of a table, in random order."""
    return torch.randperm(n_pages, generator=g, device="cuda")[: batch * per_seq].view(batch, per_seq).to(torch.int32)


def _kv4_random(g, rows_shape):
    """Codes and scales of normal rows, rounded by the plain form."""
    codes = torch.empty((*rows_shape, D // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((*rows_shape, D // 16), dtype=torch.uint8, device="cuda")
    c, s = codes.view(-1, D // 2), scales.view(-1, D // 16)
    step = 1 << 21
    base = torch.randn((min(step, c.shape[0]), D), generator=g, device="cuda")
    pc, ps = _kv4_quantise(base)
    at = 0
    while at < c.shape[0]:      # one drawn stretch of rows, its order turned for each further stretch
        n = min(step, c.shape[0] - at)
        c[at:at + n], s[at:at + n] = pc[:n].roll(at // step, 0), ps[:n].roll(at // step, 0)
        at += n
    return codes, scales


def _prepare_prompt(c, g):
    lens = [int(x) for x in c["lens"].split(",")]
    n, hq, hkv = sum(lens), c["hq"], c["hkv"]
    qkv = _normal(g, n, (hq + 2 * hkv) * D, std=1.3)     # the fused projection's output
    q, k, v = qkv.split([hq * D, hkv * D, hkv * D], dim=1)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens, dtype=torch.int32).cumsum(0)
    return dict(q=q.unflatten(1, (hq, D)), k=k.unflatten(1, (hkv, D)), v=v.unflatten(1, (hkv, D)), cu=cu.cuda(), n=n)


def _prepare_append(c, g):
    b, hkv, page = c["batch"], c["hkv"], c["page"]
    start = torch.randint(0, c["cap"] - c["new"] + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(max(1, c["new"] // 2), c["new"] + 1, (b,), generator=g, device="cuda")
    lens[0] = c["new"]
    n = c["new"] * b                                     # the chunk's buffer; what lies behind the last sequence is padding
    cu = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
    cu[1:] = lens.cumsum(0)
    per_seq = c["cap"] // page if page else 1
    n_pages = b * per_seq + 3 if page else b
    shape = (2, n_pages, hkv, page or c["cap"])          # K and V in one allocation
    return dict(k=_normal(g, n, hkv, D), v=_normal(g, n, hkv, D, std=0.6), cu=cu, start=start, n=n,
                codes=torch.zeros((*shape, D // 2), dtype=torch.uint8, device="cuda"),
                scales=torch.zeros((*shape, D // 16), dtype=torch.uint8, device="cuda"),
                table=_rand_table(g, b, per_seq, n_pages) if page else None, page=page, n_pages=n_pages,
                lut=torch.tensor([[E2M1[i & 15], E2M1[i >> 4]] for i in range(256)], dtype=torch.float16, device="cuda"))


def _prepare_attend(c, g):
    b, nq, group, ctx, hq, hkv, bs = (c[k] for k in ("batch", "nq", "group", "ctx", "hq", "hkv", "bs"))
    cap = -(-(ctx + 2 * bs) // 256) * 256
    page = c["page"]
    per_seq = cap // page if page else 1
    n_pages = b * per_seq + 5 if page else b
    shape = (n_pages, hkv, page or cap)
    kc, ks = _kv4_random(g, shape)
    vc, vs = _kv4_random(g, shape)
    groups = nq // group
    # queries of a chunk follow each other up to the context's end; decode queries sit at it, or anywhere below
    if groups > b:
        seq = torch.zeros(groups, dtype=torch.int64, device="cuda")
        pos = torch.arange(groups, device="cuda") * group + max(0, ctx - nq)
    else:
        seq = torch.arange(groups, device="cuda") % b
        pos = torch.full((groups,), ctx - 1, device="cuda")
        low = torch.randint(0, ctx, (groups,), generator=g, device="cuda")
        pos = torch.where(torch.rand(groups, generator=g, device="cuda") < 0.25, low, pos)
    pos = pos.clamp(max=ctx - 1)
    n_c = (pos + 1) // bs
    drafts = torch.arange(group, device="cuda").clamp(max=bs)      # a draft stays within the two blocks behind
    q_seq = seq.repeat_interleave(group)
    q_pos = (pos[:, None] + drafts).flatten()
    sel = torch.full((groups, CAP), -1, dtype=torch.int32, device="cuda")
    cnt = n_c.clamp(max=c["topk"])
    n_blk = ctx // bs
    at = 0
    while at < groups:                                   # random blocks, ascending, a stretch of rows at a time
        r = slice(at, min(groups, at + 256))
        key = torch.rand((r.stop - at, max(n_blk, CAP)), generator=g, device="cuda")
        blk = torch.arange(key.shape[1], device="cuda")
        key = torch.where(blk < n_c[r, None], key, 2.0 + blk / key.shape[1])
        pick = key.topk(CAP, dim=1, largest=False, sorted=True).indices
        keep = torch.arange(CAP, device="cuda") < cnt[r, None]
        pick = torch.where(keep, pick, 1 << 40).sort(dim=1).values
        sel[r] = torch.where(keep, pick, -1).to(torch.int32)
        at = r.stop
    return dict(q=_normal(g, nq, hq, D, std=1.5), kc=kc, ks=ks, vc=vc, vs=vs, q_seq=q_seq.to(torch.int32),
                q_pos=q_pos.to(torch.int32), sel=sel, cnt=cnt.to(torch.int32), cap=cap,
                table=_rand_table(g, b, per_seq, n_pages) if page else None, n_pages=n_pages)


def _prepare_update(c, g):
    b, page, hkv = c["batch"], c["page"], c["hkv"]
    per_seq = -(-(c["ctx"] + c["new"]) // page)
    lens = torch.randint(1, c["ctx"] + 1, (b,), generator=g, device="cuda")
    spare = b * (2 + c["new"] // page)                   # what this step may take
    n_pages = b * per_seq // 2 + b + spare
    want = -(-lens // page)
    fits = want.cumsum(0) <= n_pages - spare             # the rest of the slots are empty
    lens, want = torch.where(fits, lens, 0), torch.where(fits, want, 0)
    place = torch.arange(per_seq, device="cuda")
    held = place < want[:, None]
    perm = torch.randperm(n_pages, generator=g, device="cuda")
    table = torch.where(held, perm[(held.flatten().cumsum(0) - 1).clamp(min=0)].view(b, per_seq), -1)
    ref = torch.zeros(n_pages, dtype=torch.int64, device="cuda")
    ref.index_add_(0, table.flatten().clamp(min=0), (table.flatten() >= 0).to(torch.int64))
    seqs = torch.randperm(b, generator=g, device="cuda")
    free, rest = seqs[: c["free"]], seqs[c["free"]:]
    src = rest[torch.arange(c["fork"], device="cuda") % rest.numel()]
    dst = free[: c["fork"]]
    before = lens.clone()
    before[free] = 0
    before[dst] = lens[src]
    after = torch.where(before > 0, before + c["new"], 0)
    after = torch.minimum(after, torch.tensor(per_seq * page, device="cuda"))
    pools = [torch.empty((n_pages, hkv, page, D), dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in "kv"]
    return dict(table=table.to(torch.int32), ref=ref.to(torch.int32), free=free.to(torch.int32), src=src.to(torch.int32),
                dst=dst.to(torch.int32), before=before.to(torch.int32), after=after.to(torch.int32), pools=pools,
                per_seq=per_seq, n_pages=n_pages)


def _prepare_compact(c, g):
    b, page, hkv = c["batch"], c["page"], c["hkv"]
    per_seq = c["ctx"] // page
    n_pages = b * per_seq
    table = _rand_table(g, b, per_seq, n_pages)
    table = torch.where(torch.rand((b, per_seq), generator=g, device="cuda") < c["live"], table, -1)
    if b > 1:
        table[b - 1] = torch.where(table[b - 1] >= 0, table[b - 1], table[0])    # two sequences with a common part
    ref = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    ref.index_add_(0, table.flatten().clamp(min=0), (table.flatten() >= 0).to(torch.int32))
    bits = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda").random_(generator=g)  # noqa: E731
    pools = []
    for _ in "kv":                                       # codes and scales of a 4-bit cache
        pools += [bits(n_pages, hkv, page, D // 8).view(torch.uint8), bits(n_pages, hkv, page, D // 64).view(torch.uint8)]
    return dict(table=table, ref=ref, pools=pools, per_seq=per_seq, n_pages=n_pages)


def prepare(case, seed):
    g = _gen(seed)
    prep = {"prompt": _prepare_prompt, "append": _prepare_append, "attend": _prepare_attend, "update": _prepare_update,
            "compact": _prepare_compact}[case["op"]]
    return dict(prep(case, g), case=dict(case))


# ---------------------------------------------------------------- plain forms

def _plain_prompt(s):
    """softmax(q k^T / sqrt(128)) v over the keys of the same sequence up to the query's own."""
    q, k, v = s["q"].float(), s["k"].float(), s["v"].float()
    n, hq, hkv = q.shape[0], q.shape[1], k.shape[1]
    place = torch.arange(n, device=q.device)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), place.to(torch.int32), right=True)
    seen = (seq[:, None] == seq[None, :]) & (place[None, :] <= place[:, None])
    q = q.view(n, hkv, hq // hkv, D).permute(1, 2, 0, 3).reshape(hkv, hq // hkv * n, D)
    x = torch.matmul(q, k.permute(1, 2, 0)).mul_(1.0 / math.sqrt(D)).view(hq, n, n)
    x = x.masked_fill_(~seen, float("-inf"))
    x = x.sub_(x.amax(dim=-1, keepdim=True)).exp_()
    total = x.sum(dim=-1)
    o = torch.matmul(x.view(hkv, hq // hkv * n, n), v.permute(1, 0, 2)).view(hq, n, D) / total[..., None]
    return o.permute(1, 0, 2).to(torch.bfloat16).contiguous()


def _kv4_quantise(x):
    """Rows of 128 values to codes and scale bytes: a scale is the group's largest
    magnitude over 6 rounded to e4m3 (2^-9 to 448), a code the nearest e2m1 value of
    x / scale, ties to even; a group with a value that is not finite has the scale NaN."""
    x = x.float().unflatten(-1, (D // 16, 16))
    top = x.abs().amax(dim=-1)
    top = torch.where(torch.isfinite(x).all(dim=-1), (top / 6.0).clamp(2.0 ** -9, 448.0), float("nan"))
    scale = top.to(torch.float8_e4m3fn)
    y = (x / scale.float()[..., None]).abs()
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    code = code + 8 * (torch.signbit(x) & torch.isfinite(top)[..., None]).to(torch.uint8)
    code = code.flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale.view(torch.uint8)


def _kv4_values(codes, scales):
    lut = torch.tensor(E2M1, dtype=torch.float32, device=codes.device)
    pairs = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2)
    x = lut[pairs.int()].unflatten(-1, (D // 16, 16))
    return (x * scales.view(torch.float8_e4m3fn).float()[..., None]).flatten(-2)


def _row_of(s, seq, pos, page):
    """Page (or sequence) and row in it of each token."""
    if page:
        return s["table"][seq, pos // page].long(), pos % page
    return seq, pos


def _read_append(s):
    """What the cache holds: its e2m1 values and its e4m3 scales."""
    values = torch.index_select(s["lut"], 0, s["codes"].flatten().int()).view(*s["codes"].shape[:-1], D)
    return [values, s["scales"].view(torch.float8_e4m3fn)]


def _plain_append(s):
    c = s["case"]
    place = torch.arange(s["n"], device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(s["cu"][1:].contiguous(), place, right=True)
    live = seq < c["batch"]
    seq = seq[live]
    pos = (s["start"][seq] + place[live] - s["cu"][seq]).long()
    page, row = _row_of(s, seq, pos, c["page"])
    x = torch.stack((s["k"][live], s["v"][live]))        # [2][tokens][heads][128]
    codes, scales = _kv4_quantise(x)
    s["codes"][:, page, :, row] = codes.transpose(0, 1)
    s["scales"][:, page, :, row] = scales.transpose(0, 1)
    return _read_append(s)


def _plain_attend(s):
    c = s["case"]
    group, hq, hkv, bs = c["group"], c["hq"], c["hkv"], c["bs"]
    nq, groups, dev = c["nq"], c["nq"] // group, s["q"].device
    seq = s["q_seq"][::group].long()
    t = s["q_pos"].view(groups, group).long()
    tail = (t[:, :1] + 1) // bs * bs                     # first token behind the complete blocks
    blocks = s["sel"][:, : c["topk"]].long()
    tok = (blocks[..., None] * bs + torch.arange(bs, device=dev)).flatten(1)
    live = (torch.arange(c["topk"], device=dev) < s["cnt"][:, None]).repeat_interleave(bs, dim=1)
    tok = torch.cat((tok, tail + torch.arange(2 * bs, device=dev)), dim=1)
    seen = torch.cat((live, torch.ones_like(live[:, :1]).expand(-1, 2 * bs)), dim=1)[:, None, :]
    in_tail = torch.arange(tok.shape[1], device=dev) >= live.shape[1]
    seen = seen & (~in_tail | (tok[:, None, :] <= t[..., None]))           # [groups][drafts][tokens]
    at = torch.where(seen.any(dim=1), tok, 0)
    page, row = _row_of(s, seq[:, None], at, c["page"])
    k = _kv4_values(s["kc"][page, :, row], s["ks"][page, :, row])          # [groups][tokens][heads][128]
    v = _kv4_values(s["vc"][page, :, row], s["vs"][page, :, row])
    q = s["q"].float().view(groups, group, hkv, hq // hkv, D)
    x = torch.einsum("ajhrd,athd->ajhrt", q, k) / math.sqrt(D)
    x = x.masked_fill(~seen[:, :, None, None, :], float("-inf"))
    p = torch.exp(x - x.amax(dim=-1, keepdim=True).clamp(min=-3e38))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.einsum("ajhrt,athd->ajhrd", p, v) / torch.where(total > 0, total, 1.0)
    return o.reshape(nq, hq, D).to(torch.bfloat16)


def _plain_update(s):
    c = s["case"]
    page, n_pages = c["page"], s["n_pages"]
    table, ref = s["table"].clone(), torch.cat((s["ref"], s["ref"].new_zeros(1)))     # the last count takes absent pages
    slot = lambda e: torch.where(e >= 0, e, n_pages).flatten().long()  # noqa: E731
    free, src, dst = s["free"].long(), s["src"].long(), s["dst"].long()
    gone = slot(table[free])
    ref.index_add_(0, gone, torch.full_like(gone, -1, dtype=torch.int32))
    table[free] = -1
    rows = table[src]
    table[dst] = rows
    shared = slot(rows)
    ref.index_add_(0, shared, torch.ones_like(shared, dtype=torch.int32))
    place = torch.arange(s["per_seq"], device=table.device)
    lo, hi = s["before"][:, None], s["after"][:, None]
    due = (place >= lo // page) & (place < (hi + page - 1) // page) & (hi > lo)
    ref[n_pages] = 0
    common = (table >= 0) & (ref[slot(table)].view_as(table) > 1)
    want = due & ((table < 0) | common)
    rank = want.flatten().cumsum(0).view_as(table) - 1
    order = torch.argsort((ref[:n_pages] > 0).to(torch.int32), stable=True).to(torch.int32)     # free pages, lowest first
    got = want & (rank < (ref[:n_pages] == 0).sum())
    new = torch.where(got, order[rank.clamp(0, n_pages - 1)], table)
    left = slot(torch.where(got & common, table, -1))
    ref.index_add_(0, left, torch.full_like(left, -1, dtype=torch.int32))
    ref[slot(torch.where(got, new, -1))] = 1
    copy = got & common & (place * page < lo)
    old, to = table[copy].long(), new[copy].long()
    kp, vp = s["pools"]
    kp[to] = kp[old]
    vp[to] = vp[old]
    return [new, ref[:n_pages], kp, vp]


def _plain_compact(s):
    n_pages = s["n_pages"]
    live = s["ref"] > 0
    page = torch.arange(n_pages, device=live.device)
    n_live = live.sum()
    frm = page[live & (page >= n_live)]
    to = page[~live & (page < n_live)]
    where = page.to(torch.int32)
    where[frm] = to.to(torch.int32)
    ref = s["ref"].clone()
    ref[to] = ref[frm]
    ref[frm] = 0
    table = torch.where(s["table"] >= 0, where[s["table"].clamp(min=0).long()], -1)
    kc, ks, vc, vs = s["pools"]
    kc[to] = kc[frm]
    ks[to] = ks[frm]
    vc[to] = vc[frm]
    vs[to] = vs[frm]
    return [table, ref, n_live.to(torch.int32).view(1), kc, ks, vc, vs]


# ---------------------------------------------------------------- the library's calls

def _kept(s, make):
    """What a user's program keeps between calls: dims, workspace, cache handle."""
    if "kept" not in s:
        import block_sparse_attention_key_b200 as qsa
        s["kept"] = make(qsa)
    return s["kept"]


def _workspace(qsa, n):
    ws = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    qsa.qsa_workspace_init(ws)
    return ws


def _own_prompt(s):
    c = s["case"]
    qsa, dims = _kept(s, lambda m: (m, m.make_dims(s["cu"].numel() - 1, c["hq"], c["hkv"], 8192)))
    out = torch.empty((s["n"], c["hq"], D), dtype=torch.bfloat16, device="cuda")
    qsa.qsa_prompt_attn(dims, s["q"], s["k"], s["v"], s["cu"], s["n"], out)
    return out


def _own_append(s):
    c = s["case"]
    qsa, dims, cache = _kept(s, lambda m: (
        m, m.make_dims(c["batch"], c["hkv"], c["hkv"], c["cap"]),
        m.kv4_cache(s["codes"][0], s["scales"][0], s["codes"][1], s["scales"][1], s["table"], c["page"],
                    s["n_pages"] if c["page"] else 0)))
    qsa.qsa_kv4_append(dims, cache, s["k"], s["v"], s["cu"], s["start"], s["n"])
    return _read_append(s)


def _own_attend(s):
    c = s["case"]

    def make(m):
        dims = m.make_dims(c["batch"], c["hq"], c["hkv"], s["cap"], block_size=c["bs"], top_k=c["topk"])
        return (m, dims, _workspace(m, m.qsa_workspace_bytes(dims, c["nq"], 0, m.QSA_MODE_DECODE)),
                m.kv4_cache(s["kc"], s["ks"], s["vc"], s["vs"], s["table"], c["page"], s["n_pages"] if c["page"] else 0))

    qsa, dims, ws, cache = _kept(s, make)
    out = torch.empty((c["nq"], c["hq"], D), dtype=torch.bfloat16, device="cuda")
    qsa.qsa_sparse_attn_kv4(dims, cache, s["q"], s["q_seq"], s["q_pos"], s["sel"], s["cnt"], c["nq"], out, ws,
                            group_q=c["group"])
    return out


def _make_pages(s):
    c = s["case"]

    def make(m):
        dims = m.make_dims(c["batch"], c["hkv"], c["hkv"], s["per_seq"] * c["page"])
        return (m, dims, _workspace(m, m.qsa_pages_workspace_bytes(dims, c["page"], s["n_pages"])),
                m.page_pools(s["pools"], c["page"], s["n_pages"]))

    return _kept(s, make)


def _own_update(s):
    c = s["case"]
    qsa, dims, ws, pools = _make_pages(s)
    table, ref = s["table"].clone(), s["ref"].clone()    # the call works in place; a pass starts from the same state
    qsa.qsa_pages_update(dims, pools, table, ref, s["before"], s["after"], ws, free_seq=s["free"], n_free=c["free"],
                         fork_src=s["src"], fork_dst=s["dst"], n_fork=c["fork"])
    return [table, ref, *s["pools"]]


def _own_compact(s):
    qsa, dims, ws, pools = _make_pages(s)
    table, ref = s["table"].clone(), s["ref"].clone()
    n_live = torch.empty(1, dtype=torch.int32, device="cuda")
    qsa.qsa_pages_compact(dims, pools, table, ref, n_live, ws)
    return [table, ref, n_live, *s["pools"]]


def run(state):
    op = state["case"]["op"]
    if own:
        return {"prompt": _own_prompt, "append": _own_append, "attend": _own_attend, "update": _own_update,
                "compact": _own_compact}[op](state)
    return {"prompt": _plain_prompt, "append": _plain_append, "attend": _plain_attend, "update": _plain_update,
            "compact": _plain_compact}[op](state)


# ---------------------------------------------------------------- work of one pass

def work(case):
    c = case
    if c["op"] == "prompt":
        lens = [int(x) for x in c["lens"].split(",")]
        pairs = sum(n * (n + 1) // 2 for n in lens)
        return {"bytes": sum(lens) * D * 2 * (2 * c["hq"] + 2 * c["hkv"]), "flops": 4 * D * c["hq"] * pairs}
    if c["op"] == "append":
        rows = 2 * c["hkv"] * c["batch"] * c["new"] * (0.75 if c["new"] > 1 and c["batch"] > 1 else 1.0)
        held = 2 * c["hkv"] * c["batch"] * c["cap"]      # what is read back of the cache
        return {"bytes": rows * (D * 2 + 72) + held * (64 + 256), "flops": rows * D * 4}
    if c["op"] == "attend":
        groups = c["nq"] // c["group"]
        tok = min(c["topk"], c["ctx"] // c["bs"]) * c["bs"] + c["bs"]
        read = groups * c["hkv"] * tok * 144
        if groups > c["batch"]:                          # a chunk's queries read a cache at most once
            read = min(read, c["hkv"] * c["ctx"] * 144)
        return {"bytes": read + c["nq"] * c["hq"] * D * 4 + groups * CAP * 4,
                "flops": 4 * D * c["nq"] * c["hq"] * tok}
    table = c["batch"] * (c["ctx"] // c["page"]) * 4
    if c["op"] == "update":
        pages = c["batch"] * (c["ctx"] // c["page"]) // 2
        moved = 2 * c["fork"] * 2 * c["hkv"] * c["page"] * D * 2
        return {"bytes": 2 * moved + 2 * table + 8 * pages, "flops": 0}
    pages = c["batch"] * (c["ctx"] // c["page"])
    moved = pages * c["live"] * (1 - c["live"]) * c["hkv"] * c["page"] * 144
    return {"bytes": 2 * moved + 2 * table + 8 * pages, "flops": 0}


# ---------------------------------------------------------------- in 64 bits

def _exact_prompt(c, s):
    out = torch.zeros((s["n"], c["hq"], D), dtype=torch.float64, device="cuda")
    per = c["hq"] // c["hkv"]
    cu = s["cu"].tolist()
    for a, b in zip(cu[:-1], cu[1:]):
        future = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
        for h in range(c["hq"]):
            q, k, v = s["q"][a:b, h].double(), s["k"][a:b, h // per].double(), s["v"][a:b, h // per].double()
            logits = (q @ k.T * D ** -0.5).masked_fill(future, -math.inf)
            out[a:b, h] = torch.softmax(logits, dim=-1) @ v
    return out


def _exact_append(c, s):
    """Every row by itself: a scale is the nearest e4m3 number, a code the nearest e2m1 one,
    found among all of them; where two are as near, the one with the even last bit."""
    e4m3 = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().cuda()
    e2m1 = torch.tensor(E2M1[:8], dtype=torch.float64, device="cuda")

    def nearest(x, grid, first):
        off = (x[..., None] - grid).abs()
        odd = (torch.arange(len(grid), device="cuda") + first) % 2
        return torch.where(off == off.amin(dim=-1, keepdim=True), odd, 2).argmin(dim=-1)

    values = torch.zeros((*s["codes"].shape[:-1], D), dtype=torch.float64, device="cuda")
    scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
    cu, start = s["cu"].tolist(), s["start"].tolist()
    for which, x in enumerate((s["k"], s["v"])):
        for b in range(c["batch"]):
            rows = x[cu[b]:cu[b + 1]].double().unflatten(-1, (8, 16))
            scale = e4m3[nearest(rows.abs().amax(dim=-1) / 6, e4m3, 1)]
            y = rows / scale[..., None]
            y = (e2m1[nearest(y.abs(), e2m1, 0)] * y.sign()).flatten(-2)
            pos = torch.arange(start[b], start[b] + len(rows), device="cuda")
            page, row = (s["table"][b].long()[pos // c["page"]], pos % c["page"]) if c["page"] else (torch.full_like(pos, b), pos)
            values[which, page, :, row] = y
            scales[which, page, :, row] = scale
    return [values, scales]


def _exact_attend(c, s):
    if c["nq"] > 1100:
        return None
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device="cuda")
    out = torch.zeros((c["nq"], c["hq"], D), dtype=torch.float64, device="cuda")
    per, bs = c["hq"] // c["hkv"], c["bs"]
    sel, cnt, q_seq, q_pos = s["sel"].cpu(), s["cnt"].tolist(), s["q_seq"].tolist(), s["q_pos"].tolist()
    for i in range(c["nq"]):
        g = i // c["group"]
        first = (q_pos[g * c["group"]] + 1) // bs * bs
        tok = (sel[g, : cnt[g], None] * bs + torch.arange(bs)).flatten()
        tok = torch.cat((tok, torch.arange(first, max(first, q_pos[i] + 1)))).long().cuda()
        if not len(tok):
            continue
        if c["page"]:
            page, row = s["table"][q_seq[i]].long()[tok // c["page"]], tok % c["page"]
        else:
            page, row = torch.full_like(tok, q_seq[i]), tok

        def values(codes, scales):
            b = codes[page, :, row].long()
            x = torch.stack((e2m1[b % 16], e2m1[b // 16]), dim=-1).flatten(-2)
            return x * scales[page, :, row].view(torch.float8_e4m3fn).double().repeat_interleave(16, dim=-1)

        k, v = values(s["kc"], s["ks"]), values(s["vc"], s["vs"])
        for h in range(c["hkv"]):
            q = s["q"][i, h * per:(h + 1) * per].double()
            out[i, h * per:(h + 1) * per] = torch.softmax(q @ k[:, h].T * D ** -0.5, dim=-1) @ v[:, h]
    return out


def exact(case, seed):
    if case["op"] in ("update", "compact"):
        return None                                      # whole numbers and copies
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "append": _exact_append, "attend": _exact_attend}[case["op"]](case, s)
