"""GPU parity of dsa_attn_mass against the fp64 oracle.

Tolerance per listed entry. A logit z = scale q.c: the tensor core sums 576 products in
fp32, off by at most 2 * 576 * 2^-24 sum |q_d c_d| scale (the order and inner rounding of the
sum are not specified, hence the 2); scale, log2 e and the LSE are rounded once each and the
difference once more: (|z| + |lse|) * 2^-22. A head's weight a is off by a times that, plus
2^-21 a for the exponential; the head sum adds 128 roundings of 2^-24, the mean two. With many
rows a weight is rounded to 2^-41. The sum into fp32 mass adds half a step (2^-24) per row."""

import numpy as np
import pytest
import torch

from oracle import attn_weight, resolve_kv_rows, sparse_mla
from sparse_attention_05_b200 import dsa, synth
from tests.helpers import oracle_args

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _reference(a, T, q_seq, q_pos, idx, lse, scale, mass0, rows, bt, page):
    mass = mass0.astype(np.float64).copy()
    tol = np.zeros_like(mass)
    count = np.zeros_like(mass)
    for t in rows:
        b, pos = int(q_seq[t]), int(q_pos[t])
        sel = [int(s) for s in idx[t] if 0 <= s <= pos]
        if not sel:
            continue
        c = np.asarray(resolve_kv_rows(a["kv"], b, sel, bt, page), np.float64)
        q = np.asarray(a["q"][t], np.float64)
        p, terms = attn_weight(q, c, scale, lse[t])
        z = np.abs(scale * (q @ c.T))
        dz = 2 * 576 * 2.0 ** -24 * scale * (np.abs(q) @ np.abs(c).T) + \
            (z + np.abs(lse[t])[:, None]) * 2.0 ** -22 + 2.0 ** -21
        e = (terms * np.expm1(dz)).mean(0) + p * 130 * 2.0 ** -24 + 2.0 ** -41
        for s, v, w in zip(sel, p, e):
            mass[b, s] += v
            tol[b, s] += w
            count[b, s] += 1
    tol += (count + 1) * 2.0 ** -24 * np.abs(mass)
    return mass, tol


def _lists(T, q_pos, k, seed, dup=False):
    r = np.random.default_rng(seed)
    idx = np.full((T, k), -1, np.int32)
    for t in range(T):
        n = min(k, int(q_pos[t]) + 1)
        idx[t, :n] = np.sort(r.permutation(int(q_pos[t]) + 1)[:n])
    return idx


def _check(p, idx, window=None, seed=0, workspace=None):
    a = oracle_args(p)
    T = p.num_q
    q_seq, q_pos = a["q_seq"], a["q_pos"]
    lens = p.q_lens().numpy()
    start = np.concatenate([[0], np.cumsum(lens)])
    w0, wc = window if window else (0, 0)
    rows = [t for t in range(T) if w0 <= t - start[q_seq[t]] and
            (not wc or t - start[q_seq[t]] < w0 + wc)]
    _, lse = sparse_mla(a["q"], a["kv"], q_seq, q_pos, idx, p.scale, 512,
                        block_table=a["block_table"], page_size=p.page_size)
    lse = lse.astype(np.float32)
    mass0 = np.random.default_rng(seed).random((p.batch, p.max_ctx + 5)).astype(np.float32)
    g = p.to(DEV)
    mass = torch.from_numpy(mass0).cuda()
    args = (g.q, g.kv, dsa.KvLayout.of(g), p.q_per_seq, torch.from_numpy(idx).cuda(), p.scale,
            torch.from_numpy(lse).cuda())
    got = dsa.dsa_attn_mass(*args, mass, workspace, rows=window, q_start=g.q_start)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0 and got is mass
    ref, tol = _reference(a, T, q_seq, q_pos, idx, lse, p.scale, mass0, rows, a["block_table"],
                          p.page_size)
    err = np.abs(mass.double().cpu().numpy() - ref)
    assert np.all(err <= tol), f"max excess {np.max(err - tol):.3e}, max err {err.max():.3e}"
    assert np.array_equal(mass.cpu().numpy()[tol == 0], mass0[tol == 0])
    # the same bits again
    again = torch.from_numpy(mass0).cuda()
    dsa.dsa_attn_mass(*args, again, rows=window, q_start=g.q_start)
    assert torch.equal(again, mass)
    return mass0, mass


def _idx(p, k, seed):
    return _lists(p.num_q, oracle_args(p)["q_pos"], k, seed)


@pytest.mark.parametrize("k", [1, 100, 128, 129, 225, 512, 700, 2000])
def test_decode(k):
    p = synth.decode(batch=3, ctx=900, q_per_seq=1, seed=70 + k)
    mass0, mass = _check(p, _idx(p, k, k))
    # every row spreads a weight of one: 900 roundings of 2^-24 in the difference
    spread = (mass.double().cpu().numpy() - mass0).sum(1)
    assert np.all(np.abs(spread - 1) <= 1e-3)


def test_paged_two_rows_and_short_context():
    p = synth.paged_decode(batch=4, q_per_seq=2, min_ctx=3, max_ctx=700, page_size=64, seed=81)
    _check(p, _idx(p, 256, 1))


@pytest.mark.parametrize("rows", [2, 3, 8, 40])
def test_few_and_many_rows_of_a_sequence(rows):
    """On both sides of the border between the two ways of summing."""
    p = synth.ragged([300, 200], [rows, rows // 2], seed=82 + rows)
    _check(p, _idx(p, 150, rows))


def test_ragged_rows_with_an_empty_sequence_and_a_window():
    p = synth.ragged([400, 50, 130], [30, 0, 12], seed=83)
    idx = _idx(p, 64, 3)
    _check(p, idx)
    _check(p, idx, window=(3, 5))
    _check(p, idx, window=(1, 0))


def test_listed_as_it_comes():
    """Unordered lists, padding in the middle, entries past the row's position, the same
    entry twice (it counts twice), a row without any entry."""
    p = synth.decode(batch=4, ctx=300, q_per_seq=1, seed=84)
    r = np.random.default_rng(5)
    idx = r.integers(-3, 330, size=(4, 200)).astype(np.int32)
    idx[1] = -1
    idx[2, :100] = 7
    _check(p, idx)


@pytest.mark.parametrize("L,k", [(200, 128), (330, 256)])
def test_prefill_rows_shorter_than_the_list(L, k):
    """The second: as many entries as the widest tile, every tile full but for the padding."""
    p = synth.prefill(L=L, seed=85)
    _check(p, _idx(p, k, 6))


def test_nan_only_where_it_is_listed():
    p = synth.decode(batch=2, ctx=200, q_per_seq=1, seed=86)
    idx = _idx(p, 50, 7)
    free = sorted(set(range(200)) - set(idx[0].tolist()))
    for rows, T in ((1, 2), (10, 20)):
        g = p.to(DEV)
        q = g.q if rows == 1 else g.q.repeat_interleave(rows, 0)
        li = np.repeat(idx, rows, 0)
        lse = torch.zeros(T, 128, device=DEV)
        kv = g.kv.clone()
        kv[0, free] = float("nan")               # not listed by any row
        kv[1, int(idx[1, 0])] = float("nan")     # listed
        mass = torch.zeros(2, 200, device=DEV)
        lay = dsa.KvLayout(2, 200, torch.tensor([200, 200], dtype=torch.int32, device=DEV))
        dsa.dsa_attn_mass(q, kv, lay, rows, torch.from_numpy(li).cuda(), p.scale, lse + 3.0, mass)
        assert dsa.dsa_get_device_error() == 0
        bad = torch.isnan(mass).nonzero().cpu().tolist()
        assert bad == [[1, int(idx[1, 0])]]


def test_bad_page_and_bad_rows_are_reported():
    p = synth.paged_decode(batch=3, q_per_seq=2, min_ctx=200, max_ctx=256, page_size=64, seed=87)
    idx = _idx(p, 100, 8)
    g = p.to(DEV)
    lse = torch.zeros(6, 128, device=DEV)
    mass = torch.zeros(3, 256, device=DEV)
    lay = dsa.KvLayout.of(g)
    lay.block_table = lay.block_table.clone()
    lay.block_table[1, 0] = 1 << 20
    dsa.dsa_attn_mass(g.q, g.kv, lay, 2, torch.from_numpy(idx).cuda(), p.scale, lse, mass)
    assert dsa.dsa_get_device_error() == 5
    lay = dsa.KvLayout.of(g)
    lay.seqlens = lay.seqlens.clone()
    lay.seqlens[2] = 1                            # shorter than its two rows
    mass.zero_()
    dsa.dsa_attn_mass(g.q, g.kv, lay, 2, torch.from_numpy(idx).cuda(), p.scale, lse, mass)
    assert dsa.dsa_get_device_error() == 5
    assert torch.all(mass[2] == 0) and torch.any(mass[0] != 0)


def test_own_workspace_other_stream_and_graph():
    p = synth.decode(batch=2, ctx=400, q_per_seq=1, seed=88)
    idx = _idx(p, 200, 9)
    two = synth.decode(batch=2, ctx=400, q_per_seq=2, seed=91)
    n = dsa.dsa_attn_mass_workspace_size(dsa.KvLayout(2, 400), 4, 2, 200)
    _check(two, _idx(two, 200, 12), workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    g = p.to(DEV)
    for rows in (1, 2, 12):
        q = g.q.repeat_interleave(rows, 0)
        li = torch.from_numpy(np.repeat(idx, rows, 0)).cuda()
        lse = torch.full((2 * rows, 128), 6.0, device=DEV)
        lay = dsa.KvLayout(2, 400, g.seqlens)
        want = dsa.dsa_attn_mass(q, g.kv, lay, rows, li, p.scale, lse, torch.zeros(2, 400, device=DEV))
        s = torch.cuda.Stream()
        mass = torch.zeros(2, 400, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        dsa.dsa_attn_mass(q, g.kv, lay, rows, li, p.scale, lse, mass, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(mass, want)
        graph = torch.cuda.CUDAGraph()
        mass.zero_()
        with torch.cuda.graph(graph):
            dsa.dsa_attn_mass(q, g.kv, lay, rows, li, p.scale, lse, mass)
        graph.replay()
        assert torch.equal(mass, want)


def test_the_ways_of_summing_agree():
    """One batch three ways: the window of all its rows at once (integers), two rows and one row
    a call (fp32): apart by at most 2^-41 and one fp32 step per entry."""
    p = synth.ragged([300, 200], [12, 12], seed=89)
    idx = _idx(p, 100, 11)
    g = p.to(DEV)
    li = torch.from_numpy(idx).cuda()
    lay = dsa.KvLayout.of(g)
    lse = torch.full((p.num_q, 128), 6.0, device=DEV)
    sizes = [dsa.dsa_attn_mass_workspace_size(lay, p.num_q, 12, 100, rows=w, q_start=g.q_start)
             for w in (None, (0, 2), (0, 1))]
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert sizes == [up(2 * p.max_ctx * 8), up(2 * 2 * 100 * 4), 0]  # the three ways
    got = []
    for step in (12, 2, 1):
        mass = torch.zeros(2, p.max_ctx, device=DEV)
        for i in range(0, 12, step):
            dsa.dsa_attn_mass(g.q, g.kv, lay, 12, li, p.scale, lse, mass, rows=(i, step),
                              q_start=g.q_start)
        got.append(mass)
    assert torch.all((got[0] - got[1]).abs() <= 12 * 2.0 ** -41 + 13 * 2.0 ** -24 * got[1])
    assert torch.equal(got[1], got[2])      # the same additions in the same order


@pytest.mark.parametrize("k", [300, 512])
def test_long_prefill_agrees_with_its_windows(k):
    """So many rows that a CTA takes whole ones in turn, some of them with tiles without an
    entry, against windows of a hundred rows (runs of tiles): integer sums of the same weights,
    added to fp32 once and 25 times."""
    L = 2500
    g = torch.Generator(device=DEV).manual_seed(90)
    q = (torch.randn(L, 128, 576, device=DEV, generator=g) * 2).bfloat16()
    kv = (torch.randn(1, L, 576, device=DEV, generator=g) * 0.5).bfloat16()
    r = torch.rand(L, L, device=DEV, generator=g)
    at = torch.arange(L, device=DEV)
    v, i = r.masked_fill(at > at[:, None], -1.0).topk(k, dim=1)
    i = torch.where(v >= 0, i, L).sort(dim=1).values
    idx = torch.where(i < L, i, -1).int()
    lay = dsa.KvLayout(1, L)
    out, lse = dsa.dsa_sparse_mla_fwd(q, kv, lay, L, idx, 576 ** -0.5)
    whole, parts = torch.zeros(1, L, device=DEV), torch.zeros(1, L, device=DEV)
    dsa.dsa_attn_mass(q, kv, lay, L, idx, 576 ** -0.5, lse, whole)
    for w in range(0, L, 100):
        dsa.dsa_attn_mass(q, kv, lay, L, idx, 576 ** -0.5, lse, parts, rows=(w, 100))
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0
    assert torch.all((whole - parts).abs() <= 27 * 2.0 ** -24 * parts)
    assert abs(float(whole.double().sum()) - L) <= L * 1e-4   # the LSE's tolerance a row


@pytest.mark.parametrize("rows", [16, 100])
def test_many_rows_keep_small_weights(rows):
    """Every weight of the window below 2^-41 (an LSE far above the logits): summed as integers in
    units of 2^-56 times the rows, rounded up to a power of two. Half a unit an entry, beside what
    test_gpu_attn_mass's header gives for the weight itself."""
    ctx, k = 400, 150
    p = synth.ragged([ctx], [rows], seed=92)
    idx = _idx(p, k, 13)
    g = p.to(DEV)
    lay = dsa.KvLayout.of(g)
    assert dsa.dsa_attn_mass_workspace_size(lay, rows, rows, k, q_start=g.q_start) == 256 * -(-ctx * 8 // 256)
    a = oracle_args(p)
    q = np.asarray(a["q"], np.float64)
    c = np.asarray(resolve_kv_rows(a["kv"], 0, list(range(ctx)), a["block_table"], p.page_size),
                   np.float64)
    z = p.scale * np.einsum("thd,sd->ths", q, c)
    lse = (z.max(2) + 27.0).astype(np.float32)
    unit = 2.0 ** (np.ceil(np.log2(rows)) - 56)
    want, tol = np.zeros(ctx), np.zeros(ctx)
    for t in range(rows):
        sel = idx[t][idx[t] >= 0]
        w = np.exp(z[t][:, sel] - lse[t][:, None].astype(np.float64))
        dz = 2 * 576 * 2.0 ** -24 * p.scale * (np.abs(q[t]) @ np.abs(c[sel]).T) + \
            (np.abs(z[t][:, sel]) + np.abs(lse[t])[:, None]) * 2.0 ** -22 + 2.0 ** -21
        want[sel] += w.mean(0)
        tol[sel] += (w * np.expm1(dz)).mean(0) + w.mean(0) * 130 * 2.0 ** -24 + unit / 2
        assert w.mean(0).max() < 2.0 ** -41
    mass = torch.zeros(1, p.max_ctx, device=DEV)
    dsa.dsa_attn_mass(g.q, g.kv, lay, rows, torch.from_numpy(idx).cuda(), p.scale,
                      torch.from_numpy(lse).cuda(), mass, q_start=g.q_start)
    assert dsa.dsa_get_device_error() == 0
    got = mass[0, :ctx].double().cpu().numpy()
    assert np.all(np.abs(got - want) <= tol + np.abs(want) * 2.0 ** -23)
    assert np.count_nonzero(got) > ctx // 2


@pytest.mark.parametrize("kind", ["spread", "positive", "negative", "large"])
def test_mean_error_of_the_weights(kind):
    """The tensor core truncates a logit's running sum, so without a correction every weight would
    be off the same way: by 2^-21 z as measured (z its logit), in the mean over a row 2^-21 of the
    weights' mean logit. At most half of that may be left, beside 2^-23 for the LSE, the difference
    and the exponential, whose roundings have no such direction. For an exactly rounded LSE and
    for the forward's own: the formula takes the LSE as it is given."""
    B, ctx, k, scale = 16, 3000, 2048, 576 ** -0.5
    g = torch.Generator(device=DEV).manual_seed(93)
    q = torch.randn(B, 128, 576, device=DEV, generator=g) * (12.0 if kind == "large" else 3.0)
    kv = torch.randn(B, ctx, 576, device=DEV, generator=g) * 0.5
    if kind in ("positive", "negative"):
        q = q + (0.5 if kind == "positive" else -0.5)
        kv = kv + 0.3
    q, kv = q.bfloat16(), kv.bfloat16()
    idx = torch.rand(B, ctx, device=DEV, generator=g).topk(k, dim=1).indices.sort(dim=1).values.int()
    lay = dsa.KvLayout(B, ctx)
    _, own = dsa.dsa_sparse_mla_fwd(q, kv, lay, 1, idx, scale)
    z = torch.stack([q[b].double() @ kv[b][idx[b].long()].double().T for b in range(B)]) * scale
    exact = torch.logsumexp(z, 2)
    mean_z = float((torch.exp(z - exact[..., None]) * z).sum(2).mean())
    for lse in (exact.float(), own):
        mass = torch.zeros(B, ctx, device=DEV)
        dsa.dsa_attn_mass(q, kv, lay, 1, idx, scale, lse, mass)
        got = mass.gather(1, idx.long()).double()
        want = torch.exp(z - lse.double()[..., None]).mean(1)
        off = float((got.sum() - want.sum()) / want.sum())
        assert abs(off) <= 2.0 ** -22 * abs(mean_z) + 2.0 ** -23
        # the forward's logits are truncated too, in sums of their own
        rows = got.sum(1) - 1
        assert float(rows.mean().abs()) <= 2.0 ** -20 * abs(mean_z) + 2.0 ** -22
    assert abs(mean_z) > 1
    assert dsa.dsa_get_device_error() == 0


def test_weights_of_cancelling_logits():
    """Partial sums far above the logit they end at: what is lost goes with the partial sums. 36
    steps of at most 2^-23 of the largest."""
    B, ctx, k, scale = 4, 600, 512, 576 ** -0.5
    g = torch.Generator(device=DEV).manual_seed(94)
    up = torch.cat([torch.ones(288, device=DEV), -torch.ones(288, device=DEV)])
    q = (torch.randn(B, 128, 576, device=DEV, generator=g) + 2.0).bfloat16()
    kv = (torch.randn(B, ctx, 576, device=DEV, generator=g) * 0.5 + up).bfloat16()
    idx = torch.rand(B, ctx, device=DEV, generator=g).topk(k, dim=1).indices.sort(dim=1).values.int()
    rows = torch.stack([kv[b][idx[b].long()] for b in range(B)]).double()
    z = torch.einsum("bhd,bsd->bhs", q.double(), rows) * scale
    part = torch.einsum("bhd,bsd->bhs", q[..., :288].double(), rows[..., :288]).abs() * scale
    lse = torch.logsumexp(z, 2).float()
    mass = torch.zeros(B, ctx, device=DEV)
    dsa.dsa_attn_mass(q, kv, dsa.KvLayout(B, ctx), 1, idx, scale, lse, mass)
    terms = torch.exp(z - lse.double()[..., None])
    want = terms.mean(1)
    off = (36 * 2.0 ** -23 * 1.25 * part.amax() + z.abs() * 2.0 ** -21 + lse.abs()[..., None] * 2.0 ** -22
           + 2.0 ** -21)
    tol = (terms * torch.expm1(off)).mean(1) + want * 131 * 2.0 ** -24
    err = (mass.gather(1, idx.long()).double() - want).abs()
    assert float(part.mean()) > 5 * float(z.abs().mean()) and torch.all(err <= tol)


@pytest.mark.parametrize("lens,rows,k", [([1300, 1250], [1300, 1250], 40),
                                         ([900, 700, 1000], [900, 0, 1000], 300)])
def test_whole_prompts_against_the_formula(lens, rows, k):
    """Rows enough for CTAs to take whole ones in turn (sixteen an SM: 2368 on 148), ragged, in fp64
    on the GPU; in test_gpu_attn_mass's bounds."""
    batch, ctx, scale = len(lens), max(lens), 576 ** -0.5
    per = max(rows)
    g = torch.Generator(device=DEV).manual_seed(95)
    T = sum(rows)
    start = np.concatenate([[0], np.cumsum(rows)])
    q = (torch.randn(T, 128, 576, device=DEV, generator=g) * 2).bfloat16()
    kv = (torch.randn(batch, ctx, 576, device=DEV, generator=g) * 0.5).bfloat16()
    idx = torch.full((T, k), -1, device=DEV, dtype=torch.int32)
    lse = torch.zeros(T, 128, device=DEV)
    want = torch.zeros(batch, ctx, device=DEV, dtype=torch.float64)
    tol, count = torch.zeros_like(want), torch.zeros_like(want)
    for b in range(batch):
        c = kv[b].double()
        for t in range(start[b], start[b + 1]):
            pos = lens[b] - rows[b] + t - int(start[b])
            n = min(k, pos + 1)
            s = torch.randperm(pos + 1, device=DEV, generator=g)[:n].sort().values
            idx[t, :n] = s.int()
            z = q[t].double() @ c[s].T * scale
            lse[t] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[t].double()[:, None])
            dz = 2 * 576 * 2.0 ** -24 * scale * (q[t].double().abs() @ c[s].abs().T) + \
                (z.abs() + lse[t].double().abs()[:, None]) * 2.0 ** -22 + 2.0 ** -21
            want[b, s] += w.mean(0)
            tol[b, s] += (w * torch.expm1(dz)).mean(0) + w.mean(0) * 130 * 2.0 ** -24 + 2.0 ** -41
    mass = torch.zeros(batch, ctx, device=DEV)
    lay = dsa.KvLayout(batch, ctx, torch.tensor(lens, device=DEV, dtype=torch.int32))
    starts = torch.tensor(start.tolist(), device=DEV, dtype=torch.int32)
    dsa.dsa_attn_mass(q, kv, lay, per, idx, scale, lse, mass, q_start=starts)
    assert dsa.dsa_get_device_error() == 0
    assert batch * per >= 16 * torch.cuda.get_device_properties(0).multi_processor_count
    assert torch.all((mass.double() - want).abs() <= tol + 2.0 ** -23 * want)
    assert float((mass.double().sum() - T).abs()) <= T * 1e-5
