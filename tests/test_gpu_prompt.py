"""qsa_prompt_attn against softmax attention in 64 bits, sequence by sequence.

Tolerance per value, from the kernel's roundings (a bf16 rounding is off by at most
2^-8 of the value): the output's own, 2^-8 |o|, and that of every probability before
the product with V, 2^-8 sum_j p_j |v_j|.  fp32 logits of 128 bf16 products (relative
error below 128 x 2^-24 of sum |q_d k_d| <= 200 here, so below 2^-9.3 x 0.09 in the
exponent), exp2 and the fp32 sums stay below another 2^-10 sum_j p_j |v_j|.
"""

import math

import pytest
import torch

import block_sparse_attention_key_b200 as qsa

import gpu_util as gu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    gu.ensure_built()


def _cu(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def _inputs(n, hq, hkv, seed, fused=False, std=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.empty((n, (hq + 2 * hkv) * 128), dtype=torch.bfloat16, device="cuda").normal_(0, std, generator=g)
    q, k, v = (t.unflatten(1, (-1, 128)) for t in x.split([hq * 128, hkv * 128, hkv * 128], dim=1))
    return (q, k, v) if fused else (q.contiguous(), k.contiguous(), v.contiguous())


def _exact(q, k, v, cu, scale=128 ** -0.5):
    """(outputs, sum_j p_j |v_j|) in 64 bits; rows of no sequence stay 0."""
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(out)
    per = q.shape[1] // k.shape[1]
    for a, b in zip(cu[:-1], cu[1:]):
        future = torch.ones((b - a, b - a), dtype=torch.bool, device="cuda").triu(1)
        for h in range(q.shape[1]):
            kk, vv = k[a:b, h // per].double(), v[a:b, h // per].double()
            p = torch.softmax((q[a:b, h].double() @ kk.T * scale).masked_fill(future, -math.inf), dim=-1)
            out[a:b, h] = p @ vv
            mag[a:b, h] = p @ vv.abs()
    return out, mag


def _run(q, k, v, cu, n=None, out=None, scale=0.0, ws=True, **kw):
    n = q.shape[0] if n is None else n
    dims = qsa.make_dims(len(cu) - 1, q.shape[1], k.shape[1], 8192, softmax_scale=scale)
    out = torch.full((n, q.shape[1], 128), 77.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    w = gu.new_workspace(256) if ws else None
    qsa.qsa_prompt_attn(dims, q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), n, out, w, **kw)
    flags = qsa.qsa_read_device_status(w) if ws else 0
    return out, flags


def _check(out, q, k, v, cu, scale=128 ** -0.5):
    want, mag = _exact(q, k, v, cu, scale)
    a, b = cu[0], cu[-1]
    err = (out[a:b].double() - want[a:b]).abs()
    tol = 2.0 ** -8 * want[a:b].abs() + (2.0 ** -8 + 2.0 ** -10) * mag[a:b] + 1e-30
    assert torch.isfinite(out[a:b]).all()
    assert (err <= tol).all(), f"worst {(err / tol).max().item():.3f} of the tolerance"


@pytest.mark.parametrize("hq,hkv", [(8, 1), (32, 4), (16, 16), (4, 2), (12, 4), (10, 2), (7, 1), (32, 1), (20, 1)])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3], [15, 17, 16], [127, 128, 129], [257, 0, 511, 384], [700]])
def test_lengths_and_head_layouts(hq, hkv, lens):
    q, k, v = _inputs(sum(lens), hq, hkv, hq * 100 + len(lens))
    out, flags = _run(q, k, v, _cu(lens))
    assert flags == 0
    _check(out, q, k, v, _cu(lens))


@pytest.mark.parametrize("hq,hkv,lens", [(8, 1, [4100]), (2, 2, [2049, 1023]), (16, 4, [3000, 77, 1])])
def test_long_prompts(hq, hkv, lens):
    q, k, v = _inputs(sum(lens), hq, hkv, 5, fused=True)
    out, flags = _run(q, k, v, _cu(lens))
    assert flags == 0
    _check(out, q, k, v, _cu(lens))


def test_many_sequences_are_found():
    """More sequences than one search round covers, most of them empty or of a few tokens."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(0, 6, (1500,), generator=g)]
    q, k, v = _inputs(sum(lens), 4, 2, 6)
    out, flags = _run(q, k, v, _cu(lens))
    assert flags == 0
    _check(out, q, k, v, _cu(lens))


@pytest.mark.parametrize("hq,hkv", [(16, 16), (8, 1)])
def test_many_launches_of_prompts_with_and_without_second_tiles(hq, hkv):
    """Items whose second query tile is absent, in a row and between long ones, launched back to
    back: no wait runs out, and every launch gives the same bits."""
    lens = [2, 359, 2, 6, 2, 18, 8, 6, 3, 9, 22, 3, 1951, 2, 147, 43, 6, 3, 6, 1, 54, 1]
    q, k, v = _inputs(sum(lens), hq, hkv, 15)
    first, flags = _run(q, k, v, _cu(lens))
    assert flags == 0
    _check(first, q, k, v, _cu(lens))
    dims = qsa.make_dims(len(lens), hq, hkv, 8192)
    cu = torch.tensor(_cu(lens), dtype=torch.int32, device="cuda")
    outs = [torch.empty_like(first) for _ in range(4)]
    ws = gu.new_workspace(256)
    for i in range(4000):
        qsa.qsa_prompt_attn(dims, q, k, v, cu, sum(lens), outs[i % 4], ws)
    assert qsa.qsa_read_device_status(ws) == 0
    for out in outs:
        assert torch.equal(out, first)


def test_fused_projection_slices_and_scale():
    q, k, v = _inputs(333, 8, 2, 7, fused=True)
    assert q.stride(0) == 12 * 128
    out, _ = _run(q, k, v, [0, 100, 333], scale=0.03)
    _check(out, q, k, v, [0, 100, 333], scale=0.03)


def test_large_logits_move_the_running_maximum():
    """Row maxima that keep growing over the key tiles: every step rescales the sums."""
    n = 900
    q, k, v = _inputs(n, 4, 1, 8, std=1.0)
    ramp = torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None]
    k = (q[:, :1].float() * ramp).to(torch.bfloat16).contiguous()      # logits up to 6 |q|^2 / sqrt(128), rising
    out, _ = _run(q, k, v, [0, n])
    want, mag = _exact(q, k, v, [0, n])
    # logits reach 70: sum |q_d k_d| * scale <= 110, times 128 x 2^-24 in the exponent: 2^-10
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -8) * mag + 1e-30
    assert ((out.double() - want).abs() <= tol).all()


def test_rows_of_no_sequence_are_left_alone():
    q, k, v = _inputs(300, 8, 1, 9)
    cu = [20, 90, 90, 250]
    out, flags = _run(q, k, v, cu)
    assert flags == 0
    _check(out, q, k, v, cu)
    assert (out[:20] == 77).all() and (out[250:] == 77).all()


@pytest.mark.parametrize("hq,hkv", [(8, 1), (2, 2), (6, 2)])
def test_values_that_are_not_finite_stay_with_the_rows_that_see_them(hq, hkv):
    lens = [150, 140, 64]
    cu = _cu(lens)
    q, k, v = _inputs(sum(lens), hq, hkv, 10)
    clean, _ = _run(q, k, v, cu)
    v2, k2 = v.clone(), k.clone()
    v2[130, 0, 3] = math.inf           # first sequence, token 130, dim 3
    v2[140, 0, 3] = -math.inf          # then both signs: NaN from token 140 on
    v2[135, 0, 70] = math.nan
    v2[137, 0, 127] = -math.inf
    k2[cu[2] + 5, 0, 9] = math.nan     # third sequence
    out, flags = _run(q, k2, v2, cu)
    assert flags == 0
    per = hq // hkv
    seen = torch.zeros_like(out, dtype=torch.bool)
    seen[130:150, :per, 3] = True
    seen[135:150, :per, 70] = True
    seen[137:150, :per, 127] = True
    seen[cu[2] + 5:, :per] = True
    assert torch.equal(out[~seen], clean[~seen])       # nothing else moved, other sequences included
    assert (out[130:140, :per, 3] == math.inf).all() and out[140:150, :per, 3].isnan().all()
    assert out[135:150, :per, 70].isnan().all()
    assert (out[137:150, :per, 127] == -math.inf).all()
    assert out[cu[2] + 5:, :per].isnan().all()


def test_bad_lengths_are_reported_and_skipped():
    q, k, v = _inputs(200, 8, 1, 11)
    for cu in ([0, 50, 40, 200], [0, 100, 300], [-4, 100, 200]):
        out, flags = _run(q, k, v, cu)
        assert flags == qsa.qsa.QSA_DEV_BAD_LEN, cu
    out, flags = _run(q, k, v, [0, 100, 300])
    _check(out[:100], q[:100], k[:100], v[:100], [0, 100])
    assert (out[100:] == 77).all()


def test_captured_and_replayed_on_another_stream_with_new_lengths():
    q, k, v = _inputs(400, 8, 2, 12)
    dims = qsa.make_dims(2, 8, 2, 8192)
    cu = torch.tensor([0, 150, 400], dtype=torch.int32, device="cuda")
    out = torch.zeros((400, 8, 128), dtype=torch.bfloat16, device="cuda")
    qsa.qsa_prompt_attn(dims, q, k, v, cu, 400, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        qsa.qsa_prompt_attn(dims, q, k, v, cu, 400, out)
    cu.copy_(torch.tensor([0, 31, 390], dtype=torch.int32))
    out.fill_(77)
    graph.replay()
    torch.cuda.synchronize()
    _check(out, q, k, v, [0, 31, 390])
    assert (out[390:] == 77).all()


def test_two_streams_at_once():
    data = [_inputs(900, 8, 2, 30 + i) for i in range(2)]
    cu = torch.tensor([0, 300, 900], dtype=torch.int32, device="cuda")
    dims = qsa.make_dims(2, 8, 2, 8192)
    want = [_run(*d, [0, 300, 900])[0] for d in data]
    outs = [torch.empty_like(w) for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(50):
        for d, out, st in zip(data, outs, streams):
            qsa.qsa_prompt_attn(dims, *d, cu, 900, out, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_output_that_is_aligned_to_16_bytes_only():
    q, k, v = _inputs(150, 8, 1, 16)
    want, _ = _run(q, k, v, [0, 150])
    flat = torch.full((150 * 8 * 128 + 16,), 77.0, dtype=torch.bfloat16, device="cuda")
    out = flat[8:-8].view(150, 8, 128)
    assert out.data_ptr() % 32 == 16
    got, flags = _run(q, k, v, [0, 150], out=out)
    assert flags == 0 and torch.equal(got, want)
    assert (flat[:8] == 77).all() and (flat[-8:] == 77).all()


def test_same_inputs_give_the_same_bits():
    q, k, v = _inputs(1000, 16, 2, 13)
    a, _ = _run(q, k, v, [0, 400, 1000])
    b, _ = _run(q, k, v, [0, 400, 1000])
    assert torch.equal(a, b)


def test_equals_the_sparse_layer_below_its_budget():
    """A prompt of at most 512 blocks: the sparse attention over every block is this."""
    n, hq, hkv = 515, 8, 2
    q, k, v = _inputs(n, hq, hkv, 14)
    out, _ = _run(q, k, v, [0, n])
    cap = 768
    dims = qsa.make_dims(1, hq, hkv, cap)
    kc = torch.zeros((1, hkv, cap, 128), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    kc[0, :, :n], vc[0, :, :n] = k.transpose(0, 1), v.transpose(0, 1)
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    cnt = (pos + 1) // 4
    idx = torch.arange(512, device="cuda", dtype=torch.int32)
    sel = torch.where(idx < cnt[:, None], idx, -1).to(torch.int32).contiguous()
    ws = gu.new_workspace(qsa.qsa_workspace_bytes(dims, n, 0, qsa.QSA_MODE_DECODE))
    sparse = torch.empty_like(out)
    qsa.qsa_sparse_attn(dims, q, kc, vc, torch.zeros_like(pos), pos, sel, cnt, n, sparse, ws)
    assert qsa.qsa_read_device_status(ws) == 0
    _, mag = _exact(q, k, v, [0, n])
    # both within the tolerance above of the same value
    tol = 2 * (2.0 ** -8 * out.double().abs() + (2.0 ** -8 + 2.0 ** -10) * mag)
    assert ((sparse.double() - out.double()).abs() <= tol).all()


@pytest.mark.parametrize("hq,hkv,n_seq,longest", [(16, 16, 400, 160), (16, 2, 30, 700), (4, 4, 300, 300)])
def test_values_that_are_not_finite_in_many_items(hq, hkv, n_seq, longest):
    """Dozens of items per CTA, in most of them V values that are not finite under the mask: the marks
    of one item are gone before the next, in both halves of the dims, and every launch gives the same bits."""
    g = torch.Generator().manual_seed(hq + n_seq)
    lens = torch.randint(1, longest + 1, (n_seq,), generator=g).tolist()
    cu, n = _cu(lens), sum(lens)
    q, k, v = _inputs(n, hq, hkv, 17)
    bad = torch.rand((n, hkv, 128), generator=torch.Generator(device="cuda").manual_seed(18), device="cuda")
    kinds = ((math.inf, (0.0, 2e-4)), (-math.inf, (2e-4, 4e-4)), (math.nan, (4e-4, 5e-4)))
    v0, v1 = v.clone(), v.clone()
    seen = []
    for value, (lo, hi) in kinds:
        here = (bad >= lo) & (bad < hi)
        v0[here], v1[here] = 0.0, value
        past = torch.cat([here[a:b].cumsum(0) > 0 for a, b in zip(cu[:-1], cu[1:])])
        seen.append(past.repeat_interleave(hq // hkv, 1))
    clean, flags = _run(q, k, v0, cu)
    assert flags == 0
    _check(clean, q, k, v0, cu)
    up, dn, nan = seen
    nan = nan | (up & dn)
    want = clean.masked_fill(up, math.inf).masked_fill(dn, -math.inf)
    dims = qsa.make_dims(n_seq, hq, hkv, 8192)
    cu_t = torch.tensor(cu, dtype=torch.int32, device="cuda")
    ws, out = gu.new_workspace(256), torch.empty_like(clean)
    for _ in range(40):
        out.fill_(77.0)
        qsa.qsa_prompt_attn(dims, q, k, v1, cu_t, n, out, ws)
        assert qsa.qsa_read_device_status(ws) == 0
        assert torch.equal(out.isnan(), nan)
        assert torch.equal(out[~nan], want[~nan])


@pytest.mark.parametrize("hq,hkv", [(8, 1), (2, 2)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_logits_of_any_size(hq, hkv, sign):
    """Logits from 2^4 to 2^81, two values of them per row (203 / 128 times a power of two: their scaled
    values are rounded): all weight on the larger one's tokens, in equal parts.  Equal K rows give equal fp32 sums, so the expected output needs no tolerance for logits."""
    n = 700
    q, _, v = _inputs(n, hq, hkv, 19)
    g = torch.Generator(device="cuda").manual_seed(20)
    low = torch.rand((n, hkv), generator=g, device="cuda") < 0.5
    k = torch.where(low, 0.5, 1.0)[..., None].expand(-1, -1, 128).to(torch.bfloat16).contiguous()
    mag = 2.0 ** torch.randint(4, 81, (n, hq), generator=g, device="cuda")
    q = (203 / 128 * sign * mag[..., None]).expand(-1, -1, 128).to(torch.bfloat16).contiguous()
    out, flags = _run(q, k, v, [0, n])
    assert flags == 0
    for h in range(hq):
        vv, is_low = v[:, h // (hq // hkv)].double(), low[:, h // (hq // hkv), None]
        win = is_low if sign < 0 else ~is_low              # of two tokens that are both seen
        some = win.cumsum(0) > 0                           # else the others are all there is
        # 2^4: the logits differ by 2^3 x 128 x 128^-0.5 = 90, of which exp leaves nothing
        part = lambda x: torch.where(some, (x * win).cumsum(0) / win.cumsum(0).clamp(min=1),  # noqa: E731
                                     x.cumsum(0) / torch.arange(1, n + 1, device="cuda")[:, None])
        want, size = part(vv), part(vv.abs())
        # equal probabilities (each off by at most 2^-8, all alike) and fp32 sums: below the output's rounding
        tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * size
        assert ((out[:, h].double() - want).abs() <= tol).all(), h


@pytest.mark.parametrize("n_seq", [10, 40, 300])
@pytest.mark.parametrize("bound", ["raised", "lowered", "past the rows", "negative"])
def test_one_bad_bound_among_many_writes_only_what_some_sequence_names(n_seq, bound):
    """BAD_LEN, and every value is its old one or that of a sequence whose own bounds are in order."""
    g = torch.Generator().manual_seed(n_seq)
    lens = torch.randint(1, 30, (n_seq,), generator=g).tolist()
    cu, at = _cu(lens, first=3), n_seq // 2
    n = cu[-1] + 5
    cu[at] = {"raised": cu[-2], "lowered": cu[at // 2], "past the rows": n + 1, "negative": -7}[bound]
    q, k, v = _inputs(n, 4, 2, 21)
    out, flags = _run(q, k, v, cu)
    assert flags == qsa.qsa.QSA_DEV_BAD_LEN
    fine = out == 77
    for a, b in zip(cu[:-1], cu[1:]):
        if 0 <= a <= b <= n:
            want, mag = _exact(q[a:b], k[a:b], v[a:b], [0, b - a])
            tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * mag + 1e-30
            fine[a:b] |= (out[a:b].double() - want).abs() <= tol
    assert fine.all()
