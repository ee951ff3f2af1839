"""GPU parity of dsa_cache_append, dsa_evict_select and dsa_cache_compact.

Append tolerances: latent dims that pass through and keys that are not rotated are exact
(bits and codes). A rotated value is within 2^-21 (|a| + |b|) m of the formula's (see
test_gpu_rope), so its bf16 value within that and half a step, 2^-8 relative;
the key's scale, amax / 448, within 2^-21 * 2 amax' / 448 + 2^-23 relative; a code's value
within half an E4M3 step of the key: 2^-4 relative, 2^-10 scales below the normal range,
widened by the 2^-20 by which key and scale may be off. Selections and moves are exact."""

import numpy as np
import pytest
import torch

from oracle import append_token, bf16_round, cache_at, e4m3_decode, evict_select, key_codes
from sparse_attention_05_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _caches(batch, ctx, paged, page=64, seed=0, extra=1):
    """Cache arrays with recognisable contents, and their layout."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    if paged:
        per = -(-ctx // page)
        n = batch * per + extra
        table = torch.randperm(n, generator=g, device=DEV)[:batch * per].int().view(batch, per)
        shape = (n, page)
    else:
        table, shape, n = None, (batch, ctx), 0
    kv = torch.randn(*shape, 576, generator=g, device=DEV).bfloat16()
    codes = torch.randint(0, 256, (*shape, 128), generator=g, device=DEV, dtype=torch.uint8)
    scale = torch.rand(*shape, generator=g, device=DEV)

    def layout(lens):
        if not paged:
            return dsa.KvLayout(batch, ctx, lens)
        return dsa.KvLayout(batch, ctx, lens, table, page, n)
    return kv, codes, scale, table, layout


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _check_append(lens, q_lens, ctx, paged, ragged, page=64, positions=None, interleaved=True,
                  idx_interleaved=False, m=1.25, window=None, seed=1):
    batch, T = len(lens), sum(q_lens)
    kv, codes, scale, table, layout = _caches(batch, ctx, paged, page, seed)
    g = torch.Generator(device=DEV).manual_seed(seed + 100)
    lat = torch.randn(T, 640, generator=g, device=DEV).bfloat16()[:, 64:]
    key = (torch.randn(T, 136, generator=g, device=DEV) * 3).bfloat16()[:, 8:]
    f, _ = dsa.rope_freqs(64, device=DEV)
    pos = None if positions is None else positions(T)
    before = [t.clone() for t in (kv, codes, scale)]
    start = np.concatenate([[0], np.cumsum(q_lens)])
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(_i32(lens)), max(q_lens), f, pos,
                         interleaved=interleaved, idx_interleaved=idx_interleaved, magnitude=m,
                         rows=window, q_start=_i32(start.tolist()) if ragged else None)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0
    tb = None if table is None else table.cpu().numpy()
    fn = f.cpu().numpy()
    got = [t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
           for t in (kv, codes, scale)]
    old = [t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy()
           for t in before]
    latn, keyn = lat.double().cpu().numpy(), key.double().cpu().numpy()
    for b in range(batch):
        for i in range(q_lens[b]):
            if window and not window[0] <= i < window[0] + (window[1] or max(q_lens)):
                continue
            t, slot = start[b] + i, lens[b] - q_lens[b] + i
            at = cache_at(b, slot, tb, page)
            p = slot if pos is None else int(pos[t])
            y, k, s = append_token(latn[t], keyn[t], p, fn, m, interleaved=interleaved,
                                   idx_interleaved=idx_interleaved)
            row = got[0][at]
            assert np.array_equal(row[:512], latn[t][:512])
            pair = np.abs(latn[t][512:]).max() * 2 * m * 2.0 ** -21
            assert np.all(np.abs(row[512:] - y[512:]) <= pair * 1.01 + np.abs(y[512:]) * 2.0 ** -8)
            gs, gc = got[2][at], got[1][at]
            if idx_interleaved is None:
                assert gs == s and np.array_equal(gc, key_codes(k.astype(np.float32), s))
            else:
                off = 2 * np.abs(keyn[t]).max() * m * 2.0 ** -21
                assert abs(gs - float(s)) <= off / 448 + float(s) * 2.0 ** -23
                v = e4m3_decode(gc).astype(np.float64) * gs
                assert np.all(np.abs(v - k) <= np.abs(k) * 2.0 ** -4 * (1 + 2.0 ** -18)
                              + gs * 2.0 ** -10 * (1 + 2.0 ** -18) + 2 * off)
                # the dims that are not rotated: the codes for the scale it wrote
                assert np.array_equal(gc[64:], key_codes(keyn[t][64:].astype(np.float32), gs))
            for a, o in zip(got, old):
                a[at] = o[at]
    for a, o in zip(got, old):   # every other row is as it was
        assert np.array_equal(a, o)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("interleaved,idx_interleaved", [(True, False), (False, True), (True, None)])
def test_append_decode(paged, interleaved, idx_interleaved):
    """Two tokens of each sequence; one pair ends and starts a page, one fills the cache."""
    _check_append([2, 65, 200, 131], [2] * 4, 200, paged, False, interleaved=interleaved,
                  idx_interleaved=idx_interleaved)


def test_append_ragged_with_positions_and_empty_rows():
    _check_append([70, 5, 300, 1], [70, 0, 33, 1], 300, True, True, page=128,
                  positions=lambda T: torch.arange(T, device=DEV, dtype=torch.int32) * 9001 - 50)


def test_append_window_of_rows():
    _check_append([40, 60], [20, 20], 64, False, False, window=(5, 7))
    _check_append([40, 60, 9], [20, 3, 0], 64, True, True, window=(2, 0), seed=5)


def test_append_special_keys():
    """A zero key, a NaN, an infinity: floor scale, NaN codes and scale, saturation."""
    kv, codes, scale, _, layout = _caches(1, 8, False)
    lat = torch.zeros(3, 576, device=DEV, dtype=torch.bfloat16)
    key = torch.zeros(3, 128, device=DEV, dtype=torch.bfloat16)
    key[1, 100], key[2, 70], key[2, 3] = float("nan"), float("inf"), 1.0
    f, _ = dsa.rope_freqs(64, device=DEV)
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(_i32([3])), 3, f)
    assert float(scale[0, 0]) == float(np.float32(2.0 ** -120) / np.float32(448))
    assert torch.all(codes[0, 0] == 0)
    assert torch.isnan(scale[0, 1]) and torch.all(codes[0, 1] & 0x7F == 0x7F)
    assert torch.isinf(scale[0, 2]) and int(codes[0, 2, 70]) & 0x7F == 0x7F
    assert torch.all(codes[0, 2, 71:] == 0)


def test_append_reports_bad_pages_and_rows():
    """The token of a page outside the cache and of a sequence shorter than its rows are
    skipped and reported; the others are written."""
    kv, codes, scale, table, layout = _caches(3, 128, True)
    before = kv.clone()
    f, _ = dsa.rope_freqs(64, device=DEV)
    lat = torch.ones(6, 576, device=DEV, dtype=torch.bfloat16)
    key = torch.ones(6, 128, device=DEV, dtype=torch.bfloat16)
    good = table[0].clone()
    table[1, 1] = 1 << 20
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(_i32([70, 66, 1])), 2, f)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 5
    changed = (kv != before).any(-1).nonzero().cpu().tolist()
    assert changed == [[int(good[1]), 4], [int(good[1]), 5]]
    table[1, 1] = -1
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(_i32([70, 66, 66])), 2, f)
    assert dsa.dsa_get_device_error() == 5


def test_append_bits_of_the_documented_rounding():
    """Sine and cosine times the magnitude from fp64 rounded once, the products and their sum
    rounded to fp32 each, then scale and codes by IEEE divisions: the same in numpy gives the same
    bits. (At positions below 256 an fp64 angle is off by at most 2^-45; that moves one of the
    131072 sines and cosines across a rounding border, 2^-24 apart at the most frequent, with a
    probability of 1/16 in all.)"""
    T, m = 2048, 1.25
    g = torch.Generator(device=DEV).manual_seed(21)
    lat = torch.randn(T, 576, generator=g, device=DEV).bfloat16()
    key = torch.randn(T, 128, generator=g, device=DEV).bfloat16()
    pos = torch.randint(0, 256, (T,), generator=g, device=DEV, dtype=torch.int32)
    f, _ = dsa.rope_freqs(64, device=DEV)
    kv, codes, scale, _, layout = _caches(1, T, False)
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(None), T, f, pos, magnitude=m)
    angle = pos.cpu().numpy().astype(np.float64)[:, None] * f.cpu().numpy()
    c, s = (np.cos(angle) * m).astype(np.float32), (np.sin(angle) * m).astype(np.float32)
    ln, kn = lat.float().cpu().numpy(), key.float().cpu().numpy()
    a, b = ln[:, 512::2], ln[:, 513::2]
    ln[:, 512::2], ln[:, 513::2] = a * c - b * s, a * s + b * c
    assert torch.equal(kv[0].cpu(), torch.from_numpy(ln).bfloat16())
    a, b = kn[:, :32].copy(), kn[:, 32:64].copy()
    kn[:, :32], kn[:, 32:64] = a * c - b * s, a * s + b * c
    want = np.abs(kn).max(1) / np.float32(448)
    assert np.array_equal(scale[0].cpu().numpy(), want)
    assert np.array_equal(codes[0].cpu().numpy(), key_codes(kn, want[:, None]))


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_writes_what_rope_gives(interleaved):
    """A token's rope dims are dsa_rope's, and its key's scale and codes those of dsa_rope's fp32
    result, bit for bit, wherever it lies."""
    T = 3000
    g = torch.Generator(device=DEV).manual_seed(22)
    lat = torch.randn(T, 576, generator=g, device=DEV).bfloat16()
    key = (torch.randn(T, 128, generator=g, device=DEV) * 5).bfloat16()
    pos = torch.randint(-1000, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32)
    f, m = dsa.rope_freqs(64, scaling="yarn", factor=16.0, device=DEV)
    kv, codes, scale, _, layout = _caches(1, T, False)
    dsa.dsa_cache_append(lat, key, kv, codes, scale, layout(None), T, f, pos, magnitude=m,
                         interleaved=interleaved, idx_interleaved=interleaved)
    want = dsa.dsa_rope(lat, pos, f, rot_begin=512, interleaved=interleaved, magnitude=m)
    assert torch.equal(kv[0], want)
    k = dsa.dsa_rope(key.float(), pos, f, interleaved=interleaved, magnitude=m).cpu().numpy()
    s = np.abs(k).max(1) / np.float32(448)
    assert np.array_equal(scale[0].cpu().numpy(), s)
    assert np.array_equal(codes[0].cpu().numpy(), key_codes(k, s[:, None]))


# ---- selection -----------------------------------------------------------------------


def _check_select(mass, lens, keep, sink, recent):
    batch, ctx = mass.shape
    kept, new = dsa.dsa_evict_select(mass, dsa.KvLayout(batch, ctx - 3, _i32(lens)), keep, sink,
                                     recent)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0
    m, k = mass.cpu().numpy(), kept.cpu().numpy()
    for b, n in enumerate(lens):
        want = evict_select(m[b], n, keep, sink, recent)
        assert int(new[b]) == len(want)
        assert k[b].tolist() == want + [-1] * (keep - len(want)), f"sequence {b}"


@pytest.mark.parametrize("kind", ["spread", "ties", "equal", "special"])
@pytest.mark.parametrize("ctx,keep,sink,recent", [
    (40, 1, 0, 0), (1000, 500, 4, 64), (5000, 37, 0, 0), (5000, 4990, 1, 2), (3000, 100, 60, 40),
    (70001, 20000, 16, 3000),
])
def test_select_against_a_sort(kind, ctx, keep, sink, recent):
    g = torch.Generator(device=DEV).manual_seed(ctx + keep)
    lens = [0, 1, keep, keep + 1, ctx - 7, ctx]
    lens = [min(n, ctx) for n in lens]
    m = torch.rand(len(lens), ctx + 3, generator=g, device=DEV)
    if kind == "spread":
        m = torch.exp((m - 0.5) * 60) * torch.where(m > 0.5, 1.0, -1.0)
    elif kind == "ties":
        m = (m * 5).round()
    elif kind == "equal":
        m = torch.zeros_like(m)
    else:
        v = torch.tensor([float("nan"), -float("inf"), float("inf"), 0.0, -0.0, 1e-45, -1.0],
                         device=DEV)
        m = v[(m * 6.99).long()]
    _check_select(m.contiguous(), lens, keep, sink, recent)


@pytest.mark.parametrize("ctx", [400001, 1 << 22])
def test_select_from_very_long_contexts(ctx):
    """Beyond the keys that shared memory holds, up to the longest context; many ties."""
    g = torch.Generator(device=DEV).manual_seed(ctx)
    m = (torch.rand(2, ctx, generator=g, device=DEV) * 1000).round()
    lens, keep, sink, recent = [ctx, ctx - 12345], 150000, 7, 1001
    kept, new = dsa.dsa_evict_select(m, dsa.KvLayout(2, ctx, _i32(lens)), keep, sink, recent)
    assert dsa.dsa_get_device_error() == 0 and new.tolist() == [keep, keep]
    for b, n in enumerate(lens):
        middle = m[b, sink:n - recent]
        best = middle.sort(descending=True, stable=True).indices[:keep - sink - recent].sort().values
        at = torch.arange(ctx, device=DEV)
        want = torch.cat([at[:sink], best + sink, at[n - recent:n]])
        assert torch.equal(kept[b].long(), want)


@pytest.mark.parametrize("batch,ctx,keep", [(150, 30001, 9000), (300, 8200, 1000), (80, 100000, 30001),
                                            (150, 600001, 200000)])
@pytest.mark.parametrize("kind", ["spread", "zeros", "ties", "infinities", "nan", "negative"])
def test_select_in_large_batches(batch, ctx, keep, kind):
    """More sequences than SMs: few CTAs each, whose keys shared memory does not always hold;
    borders among zeros of both signs (and of the tiniest numbers), among equal masses, among
    infinities of either sign and among NaN."""
    g = torch.Generator(device=DEV).manual_seed(batch + ctx)
    m = torch.rand(batch, ctx, generator=g, device=DEV)
    if kind == "zeros":   # more is kept than is not zero; every other sequence also has denormals
        small = torch.where(m < 0.6, torch.tensor(-0.0, device=DEV), torch.tensor(0.0, device=DEV))
        small[::2] = torch.where(m[::2] < 0.3, torch.tensor(1e-45, device=DEV), small[::2])
        m = torch.where(m > 0.95, m, small)
    elif kind == "ties":
        m = torch.ones_like(m)
    elif kind == "infinities":   # the border among the lower ones, or the upper ones
        inf = float("inf")
        m = torch.where(m < 0.7, torch.tensor(-inf, device=DEV), m - 2)
        m[::2] = -m[::2]
    elif kind == "nan":
        m = torch.where(m < 0.8, torch.tensor(float("nan"), device=DEV),
                        torch.where(m < 0.85, torch.tensor(-float("inf"), device=DEV), m - 0.9))
    elif kind == "negative":
        m = -torch.exp(m * 100 - 50)
    sink, recent = 5, 70
    lens = torch.randint(ctx // 2, ctx + 1, (batch,), generator=g, device=DEV).int()
    lens[0], lens[1] = ctx, keep
    kept, new = dsa.dsa_evict_select(m, dsa.KvLayout(batch, ctx, lens), keep, sink, recent)
    assert dsa.dsa_get_device_error() == 0
    assert torch.equal(new, lens.clamp(max=keep))
    for b in [0, 1, 2, 3, batch // 2, batch - 2, batch - 1]:
        n = int(lens[b])
        at = torch.arange(n, device=DEV)
        want = at
        if n > keep:
            middle = m[b, sink:n - recent].double()       # NaN below -inf, here both finite
            middle = middle.clamp(min=-1e300).nan_to_num(nan=-1e301, posinf=1e300)
            order = middle.sort(descending=True, stable=True).indices   # -0 equals +0
            best = order[:keep - sink - recent].sort().values
            want = torch.cat([at[:sink], best + sink, at[n - recent:]])
        assert torch.equal(kept[b, :len(want)].long(), want), f"sequence {b}"
        assert torch.all(kept[b, len(want):] == -1)


def test_keep_at_the_end_of_int32():
    """kept of 8 GB, nearly all of it padding: its last places are counted in 64 bits."""
    keep = 2**31 - 1
    kept = torch.zeros(1, keep, dtype=torch.int32, device=DEV)
    kv, codes, scale, _, layout = _caches(1, 600, False)
    lay = layout(_i32([500]))
    mass = torch.rand(1, 600, device=DEV)
    _, new = dsa.dsa_evict_select(mass, lay, keep, sink=3, recent=5, kept=kept)
    assert new.tolist() == [500] and kept[0, :500].tolist() == list(range(500))
    assert int(kept[0, 500:].max()) == -1 and int(kept[0, 500:].min()) == -1
    kept[0, :4] = _i32([7, 8, 11, 499])
    before = [t.clone() for t in (kv, codes, scale, mass)]
    dsa.dsa_cache_compact(kv, codes, scale, lay, kept, _i32([4]), mass=mass)
    assert dsa.dsa_get_device_error() == 0
    for a, b in zip((kv, codes, scale, mass), before):
        assert torch.equal(a[0, :4], b[0, [7, 8, 11, 499]])


def test_select_reports_a_length_out_of_range():
    m = torch.rand(3, 100, device=DEV)
    kept, new = dsa.dsa_evict_select(m, dsa.KvLayout(3, 100, _i32([101, -1, 90])), 10)
    assert dsa.dsa_get_device_error() == 5
    assert new.tolist() == [0, 0, 10] and torch.all(kept[:2] == -1)


# ---- compaction ----------------------------------------------------------------------


def _lists(lens, keep, seed):
    """Random kept lists: an unmoved beginning, gaps, the last slot."""
    r = np.random.default_rng(seed)
    kept = np.full((len(lens), keep), -1, np.int32)
    new = []
    for b, n in enumerate(lens):
        k = min(n, keep)
        s = np.sort(r.permutation(n)[:k]) if b % 2 == 0 or n == 0 else np.r_[
            np.arange(k // 2), np.sort(r.permutation(np.arange(k // 2, n))[:k - k // 2])]
        kept[b, :k] = s
        new.append(k)
    return torch.from_numpy(kept).cuda(), _i32(new)


def _rows(cache, table, page, b, slots):
    if table is None:
        return cache[b, slots]
    s = torch.as_tensor(slots, device=DEV)
    return cache[table[b].long()[s // page], s % page]


@pytest.mark.parametrize("paged,page", [(False, 64), (True, 64), (True, 128)])
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,keep", [([9], 4), ([0, 1, 700, 333, 700], 300), ([5000, 4100], 2600),
                                       ([12345], 9001)])
def test_compact_moves_every_bit(paged, page, in_place, lens, keep):
    ctx = max(lens) + 5
    kv, codes, scale, table, layout = _caches(len(lens), ctx, paged, page, seed=keep)
    mass = torch.rand(len(lens), ctx + 11, device=DEV)
    kept, new = _lists(lens, keep, keep)
    src = [t.clone() for t in (kv, codes, scale, mass)]
    if in_place:
        tkv, tcodes, tscale, ttable, tmass, tctx = kv, codes, scale, table, mass, ctx
        want = [t.clone() for t in src]
        dsa.dsa_cache_compact(kv, codes, scale, layout(_i32(lens)), kept, new, mass=mass)
    else:
        tkv, tcodes, tscale, ttable, tlayout = _caches(len(lens), keep, paged, page, seed=3)
        tmass, tctx = torch.rand(len(lens), keep + 2, device=DEV), keep
        want = [t.clone() for t in (tkv, tcodes, tscale, tmass)]
        dsa.dsa_cache_compact(kv, codes, scale, layout(_i32(lens)), kept, new, mass=mass,
                              dst=tlayout(None), dst_kv_cache=tkv, dst_k_idx=tcodes,
                              dst_k_scale=tscale, dst_mass=tmass)
        for a, b in zip((kv, codes, scale, mass), src):
            assert torch.equal(a, b)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0
    for b, n in enumerate(lens):
        k = int(new[b])
        s = kept[b, :k].long()
        for w, x in zip(want[:3], src[:3]):
            v = _rows(x, table, page, b, s)
            i = torch.arange(k, device=DEV)
            if ttable is None:
                w[b, :k] = v
            else:
                w[ttable[b].long()[i // page], i % page] = v
        want[3][b, k:min(n, tctx)] = 0
        want[3][b, :k] = src[3][b, s]
    for a, w in zip((tkv, tcodes, tscale, tmass), want):
        assert torch.equal(a, w)


@pytest.mark.parametrize("batch,n,keep,paged,in_place", [
    # in place, most tokens kept, so that what one chunk's rows are moved over is another's source;
    # on 148 SMs: one CTA a slice and 20 chunks; clusters of two, four and eight and several chunks
    (100, 5200, 5001, True, True), (100, 700, 513, False, True), (48, 6000, 5777, False, True),
    (20, 9000, 8500, True, True), (4, 20000, 19500, False, True), (2, 30000, 29000, True, True),
    (1, 40000, 39001, True, True),
    # into other pages, two to four steps of a warp
    (20, 1400, 1003, True, False), (20, 1300, 1150, False, False), (40, 1700, 1501, True, False),
])
def test_compact_many_sequences_and_chunks(batch, n, keep, paged, in_place):
    kv, codes, scale, table, layout = _caches(batch, n, paged, 64, seed=batch)
    mass = torch.rand(batch, n, device=DEV)
    lens = [n - 3 * (b % 7) for b in range(batch)]
    r = np.random.default_rng(keep)
    kept = np.stack([np.sort(np.r_[0:5, 5 + r.permutation(m - 5)[:keep - 5]]) for m in lens])
    kept, new = torch.from_numpy(kept.astype(np.int32)).cuda(), _i32([keep] * batch)
    src = [t.clone() for t in (kv, codes, scale, mass)]
    if in_place:
        ttable, to = table, (kv, codes, scale, mass)
        dsa.dsa_cache_compact(kv, codes, scale, layout(_i32(lens)), kept, new, mass=mass)
    else:
        tkv, tcodes, tscale, ttable, tlayout = _caches(batch, keep, paged, 64, seed=3)
        to = (tkv, tcodes, tscale, torch.rand(batch, keep, device=DEV))
        dsa.dsa_cache_compact(kv, codes, scale, layout(_i32(lens)), kept, new, mass, tlayout(None),
                              *to)
    torch.cuda.synchronize()
    assert dsa.dsa_get_device_error() == 0
    i = torch.arange(keep, device=DEV)
    for b, m in enumerate(lens):
        s = kept[b].long()
        for x, y in zip(src[:3], to[:3]):
            assert torch.equal(_rows(y, ttable, 64, b, i), _rows(x, table, 64, b, s)), f"sequence {b}"
        assert torch.equal(to[3][b, :keep], src[3][b, s])
        if in_place:
            assert not to[3][b, keep:m].any() and torch.equal(to[3][b, m:], src[3][b, m:])
            rest = torch.arange(keep, n, device=DEV)    # slots behind the new length as they were
            for x, y in zip(src[:3], to[:3]):
                assert torch.equal(_rows(y, table, 64, b, rest), _rows(x, table, 64, b, rest))


def test_compact_into_fresh_pages_of_the_same_cache_without_mass():
    kv, codes, scale, table, layout = _caches(2, 300, True, 64, seed=9, extra=6)
    used = set(table.flatten().tolist())
    free = torch.tensor([p for p in range(kv.shape[0]) if p not in used][:4], device=DEV)
    to = dsa.KvLayout(2, 128, None, free.int().view(2, 2), 64, kv.shape[0])
    kept, new = _lists([300, 250], 128, 4)
    want = [torch.stack([_rows(x, table, 64, b, kept[b].long()) for b in range(2)])
            for x in (kv, codes, scale)]
    dsa.dsa_cache_compact(kv, codes, scale, layout(_i32([300, 250])), kept, new, dst=to,
                          dst_kv_cache=kv, dst_k_idx=codes, dst_k_scale=scale)
    for x, w in zip((kv, codes, scale), want):
        assert torch.equal(x[free].reshape(2, 128, *x.shape[2:]), w)


def test_compact_reports_bad_lists():
    """Descending, repeated, too large and negative slots, lengths out of range: reported,
    skipped, and the other sequences moved."""
    kv, codes, scale, _, layout = _caches(4, 64, False)
    before = kv.clone()
    kept = _i32([[5, 4, 7, 8], [1, 1, 63, 64], [2, -1, 9, 10], [3, 9, 11, 13]])
    dsa.dsa_cache_compact(kv, codes, scale, layout(_i32([64, 64, 64, 64])), kept, _i32([4, 4, 4, 4]))
    assert dsa.dsa_get_device_error() == 5
    assert torch.equal(kv[3, :4], before[3, [3, 9, 11, 13]])
    assert torch.equal(kv[:, 4:], before[:, 4:])
    for lens, new in (([64] * 4, [5, 4, 4, 4]), ([65, 64, 64, 64], [4] * 4), ([3, 64, 64, 64], [4] * 4),
                      ([64] * 4, [-1, 4, 4, 4])):
        kv.copy_(before)
        good = _i32([[3, 9, 11, 13]] * 4)
        dsa.dsa_cache_compact(kv, codes, scale, layout(_i32(lens)), good, _i32(new))
        assert dsa.dsa_get_device_error() == 5
        assert torch.equal(kv[0], before[0])
        assert torch.equal(kv[1, :4], before[1, [3, 9, 11, 13]])


def test_caches_past_32_bits():
    """Appending to, weighing, choosing from and moving out of the last slots of a cache whose
    latent rows span 4.6 GB."""
    ctx = 4_000_000
    kv = torch.zeros(1, ctx, 576, device=DEV, dtype=torch.bfloat16)
    codes = torch.zeros(1, ctx, 128, device=DEV, dtype=torch.uint8)
    scale = torch.zeros(1, ctx, device=DEV)
    lay = dsa.KvLayout(1, ctx)
    lat = torch.randn(3, 576, device=DEV).bfloat16()
    key = torch.randn(3, 128, device=DEV).bfloat16()
    f, _ = dsa.rope_freqs(64, device=DEV)
    dsa.dsa_cache_append(lat, key, kv, codes, scale, lay, 3, f, idx_interleaved=None)
    assert torch.equal(kv[0, -3:, :512], lat[:, :512]) and torch.all(scale[0, -3:] > 0)
    assert not kv[0, :-3].any() and not scale[0, :-3].any()
    q = torch.randn(3, 128, 576, device=DEV).bfloat16()
    idx = _i32([[0, ctx - 3, -1], [5, ctx - 3, ctx - 2], [7, ctx - 2, ctx - 1]])
    out, lse = dsa.dsa_sparse_mla_fwd(q, kv, lay, 3, idx, 576 ** -0.5)
    mass = torch.zeros(1, ctx, device=DEV)
    dsa.dsa_attn_mass(q, kv, lay, 3, idx, 576 ** -0.5, lse, mass)
    assert abs(float(mass.double().sum()) - 3) < 3e-4
    assert set(mass[0].nonzero().flatten().tolist()) == {0, 5, 7, ctx - 3, ctx - 2, ctx - 1}
    kept, new = dsa.dsa_evict_select(mass, lay, 6)
    assert kept.tolist() == [[0, 5, 7, ctx - 3, ctx - 2, ctx - 1]]
    last = [t[0, -3:].clone() for t in (kv, codes, scale, mass)]
    dsa.dsa_cache_compact(kv, codes, scale, lay, kept, new, mass=mass)
    assert dsa.dsa_get_device_error() == 0
    for t, w in zip((kv, codes, scale, mass), last):
        assert torch.equal(t[0, 3:6], w)
    assert not mass[0, 6:].any() and torch.equal(kv[0, -3:], last[0])


def test_trimming_twice_and_captured():
    """Select and compact captured into one graph and replayed: the second replay trims what
    the first left (nothing moves any more)."""
    kv, codes, scale, _, layout = _caches(3, 1000, False)
    mass = torch.rand(3, 1000, device=DEV)
    lens = _i32([1000, 640, 100])
    lay = layout(lens)
    kept = torch.empty(3, 200, dtype=torch.int32, device=DEV)
    new = torch.empty(3, dtype=torch.int32, device=DEV)
    start = [t.clone() for t in (kv, codes, scale, mass)]
    graph = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        dsa.dsa_evict_select(mass, lay, 200, 4, 32, kept, new, stream=s)
        dsa.dsa_cache_compact(kv, codes, scale, lay, kept, new, mass=mass, stream=s)
        lens.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    assert lens.tolist() == [200, 200, 100]
    after = [t.clone() for t in (kv, codes, scale, mass)]
    for b, n in enumerate((1000, 640, 100)):
        want = evict_select(start[3][b].cpu().numpy(), n, 200, 4, 32)
        assert torch.equal(kv[b, :len(want)], start[0][b, want])
        assert torch.equal(mass[b, :len(want)], start[3][b, want])
    assert torch.all(mass[0, 200:] == 0) and torch.all(mass[1, 200:640] == 0)
    graph.replay()
    torch.cuda.synchronize()
    for a, w in zip((kv, codes, scale, mass), after):
        assert torch.equal(a, w)
