"""The calls around the caches run together as a decoding program uses them: prompts are
appended to empty paged caches, then step by step the newest token's queries are rotated,
its cache rows appended, the forward runs, the attention mass accumulates, and every few
steps the caches are trimmed in place; rotary positions run on while slots are reused.

At three of the steps the caches are read back and the newest row, the forward over the GPU's
own selection and the masses are compared with the fp64 oracle, at every trim the choice.
Outputs are held to the forward's tolerances; a mass grows by weights that sum to one per
row, to the 1e-4 the LSE may be off (twice that a row covers the exponential of it)."""

import numpy as np
import pytest
import torch

from oracle import attn_weight, evict_select, rope_rows, sparse_mla_token
from sparse_attention_05_b200 import dsa
from tests.helpers import LSE_ATOL, OUT_ATOL, OUT_RTOL

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_decode_with_trimming():
    batch, page, ctx, k, keep = 2, 64, 192, 48, 100
    g = torch.Generator(device=DEV).manual_seed(7)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * std).bfloat16()

    per = ctx // page
    n_pages = batch * per + 2
    table = torch.randperm(n_pages, generator=g, device=DEV)[:batch * per].int().view(batch, per)
    kv_cache = torch.zeros(n_pages, page, 576, device=DEV, dtype=torch.bfloat16)
    k_idx = torch.zeros(n_pages, page, 128, device=DEV, dtype=torch.uint8)
    k_scale = torch.zeros(n_pages, page, device=DEV)
    mass = torch.zeros(batch, ctx, device=DEV)
    lens = torch.tensor([130, 101], dtype=torch.int32, device=DEV)
    seen = lens.clone()                     # tokens of the text: the next rotary position
    lay = dsa.KvLayout(batch, ctx, lens, table, page, n_pages)
    freqs, mag = dsa.rope_freqs(64, scaling="yarn", factor=8.0, original_ctx=64, device=DEV)
    fn = freqs.cpu().numpy()
    scale = 576 ** -0.5

    # the prompts, a ragged batch into empty caches
    start = torch.tensor([0, 130, 231], dtype=torch.int32, device=DEV)
    dsa.dsa_cache_append(normal(231, 576, std=0.5), normal(231, 128), kv_cache, k_idx, k_scale, lay,
                         130, freqs, magnitude=mag, q_start=start)
    position = [list(range(130)), list(range(101))]   # rotary position of every slot
    sums = np.zeros(batch)
    trims = 0
    for step in range(40):
        lens += 1
        pos = seen.clone()
        seen += 1
        lat, key = normal(batch, 576, std=0.5), normal(batch, 128)
        dsa.dsa_cache_append(lat, key, kv_cache, k_idx, k_scale, lay, 1, freqs, pos, magnitude=mag)
        for b in range(batch):
            position[b].append(int(pos[b]))
        # queries: the rope part rotated into the absorbed queries, the indexer's in place
        q = torch.empty(batch, 128, 576, device=DEV, dtype=torch.bfloat16)
        q[..., :512] = normal(batch, 128, 512)
        rope_part = normal(batch, 128, 192)[..., 128:]
        dsa.dsa_rope(rope_part, pos, freqs, q[..., 512:], interleaved=True, magnitude=mag)
        q_idx = normal(batch, 64, 128)
        dsa.dsa_rope(q_idx, pos, freqs, q_idx, magnitude=mag)
        w = torch.rand(batch, 64, generator=g, device=DEV)
        idx = torch.empty(batch, k, dtype=torch.int32, device=DEV)
        out, lse, _ = dsa.dsa_forward(q_idx, w, k_idx, k_scale, q, kv_cache, lay, 1, k, scale,
                                      idx_out=idx)
        dsa.dsa_attn_mass(q, kv_cache, lay, 1, idx, scale, lse, mass)
        torch.cuda.synchronize()
        assert dsa.dsa_get_device_error() == 0
        sums += 1
        if step in (0, 17, 39):
            m = mass.double().cpu().numpy()
            for b in range(batch):
                n = int(lens[b])
                assert len(position[b]) == n
                rows = kv_cache[table[b].long()].reshape(-1, 576)[:n].double().cpu().numpy()
                # the newest token's row: its latent, and its rope dims at its text position
                want = rope_rows(lat[b].double().cpu().numpy()[None, None], [position[b][-1]], fn,
                                 mag, rot_begin=512, interleaved=True)[0, 0]
                assert np.all(np.abs(rows[n - 1] - want) <= np.abs(want) * 2.0 ** -8 + 2.0 ** -16)
                sel = idx[b].cpu().numpy()
                sel = sel[sel >= 0]
                assert len(sel) == min(k, n) and sel.max() < n
                o, l = sparse_mla_token(q[b].double().cpu().numpy(), rows[sel], scale, 512)
                err = np.abs(out[b].double().cpu().numpy() - o)
                assert np.all((err <= OUT_ATOL) | (err <= OUT_RTOL * np.abs(o)))
                assert np.all(np.abs(lse[b].double().cpu().numpy() - l) <= LSE_ATOL)
                qn, ln = q[b].double().cpu().numpy(), lse[b].double().cpu().numpy()
                p, terms = attn_weight(qn, rows[sel], scale, ln)
                if step == 0:   # the mass is this step's weights, within test_gpu_attn_mass's bound
                    dz = 2 * 576 * 2.0 ** -24 * scale * (np.abs(qn) @ np.abs(rows[sel]).T) + \
                        (np.abs(scale * (qn @ rows[sel].T)) + np.abs(ln)[:, None]) * 2.0 ** -22 + \
                        2.0 ** -21
                    e = (terms * np.expm1(dz)).mean(0) + p * 131 * 2.0 ** -24
                    assert np.all(np.abs(m[b, sel] - p) <= e)
                    assert np.all(np.delete(m[b], sel) == 0)
                # a row adds weights that sum to one (to the LSE's 1e-4 a row)
                assert abs(m[b].sum() - sums[b]) <= 2e-4 * (step + 1)
        if step % 10 == 9 and step < 39:
            before = mass.cpu().numpy().copy()
            n_before = lens.tolist()
            kept, new = dsa.dsa_evict_select(mass, lay, keep, sink=4, recent=16)
            dsa.dsa_cache_compact(kv_cache, k_idx, k_scale, lay, kept, new, mass=mass)
            lens.copy_(new)
            torch.cuda.synchronize()
            assert dsa.dsa_get_device_error() == 0
            for b in range(batch):
                want = evict_select(before[b], n_before[b], keep, 4, 16)
                assert kept[b, :int(new[b])].tolist() == want
                position[b] = [position[b][s] for s in want]
                sums[b] = before[b][want].astype(np.float64).sum()
                trims += n_before[b] > keep
    assert trims >= 6                       # every trim had something to trim
    assert int(seen[0]) == 170 and max(position[0]) == 169


def test_two_streams_at_once():
    """The masses of two caches and their trims, each on a stream of its own at the same time,
    against the same calls one after another: bit for bit."""
    batch, ctx, k, keep = 3, 4096, 1024, 1500
    g = torch.Generator(device=DEV).manual_seed(11)
    sets = []
    for i in range(2):
        lens = torch.tensor([ctx, 3000 + i, 2000], dtype=torch.int32, device=DEV)
        n = 2                                  # rows a sequence: through the workspace
        q = torch.randn(batch * n, 128, 576, generator=g, device=DEV).bfloat16()
        kvc = (torch.randn(batch, ctx, 576, generator=g, device=DEV) * 0.5).bfloat16()
        idx = torch.stack([torch.randperm(1900, generator=g, device=DEV)[:k]
                           for _ in range(batch * n)]).int()
        lse = torch.full((batch * n, 128), 8.0, device=DEV)
        codes = torch.randint(0, 127, (batch, ctx, 128), generator=g, device=DEV).to(torch.uint8)
        sc = torch.rand(batch, ctx, generator=g, device=DEV)
        sets.append((dsa.KvLayout(batch, ctx, lens), n, q, kvc, idx, lse, codes, sc))
    streams = [torch.cuda.Stream() for _ in sets]

    def run(concurrent):
        out = []
        state = [(s[3].clone(), s[6].clone(), s[7].clone(), torch.zeros(batch, ctx, device=DEV))
                 for s in sets]
        torch.cuda.synchronize()
        for _ in range(3):
            for s, st, (kvc, codes, sc, mass) in zip(sets, streams, state):
                with torch.cuda.stream(st):
                    lay, n, q, _, idx, lse, _, _ = s
                    dsa.dsa_attn_mass(q, kvc, lay, n, idx, 0.04, lse, mass)
                    kept, new = dsa.dsa_evict_select(mass, lay, keep, sink=4, recent=100)
                    to = dsa.KvLayout(batch, keep)
                    dst = (torch.zeros(batch, keep, 576, device=DEV, dtype=torch.bfloat16),
                           torch.zeros(batch, keep, 128, device=DEV, dtype=torch.uint8),
                           torch.zeros(batch, keep, device=DEV))
                    dm = torch.zeros(batch, keep, device=DEV)
                    dsa.dsa_cache_compact(kvc, codes, sc, lay, kept, new, mass, to, *dst, dm)
                    out += [kept, new, *dst, dm]
                if not concurrent:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert dsa.dsa_get_device_error() == 0
        return out + [m for *_, m in state]

    for a, b in zip(run(False), run(True)):
        assert torch.equal(a, b)


def test_yarn_scales_the_whole_logit():
    """A decode step under YaRN as ``rope_freqs`` says: only 64 of a logit's 576 dims rotate, so
    its factor goes into the scale. The same factor on the rotated dims is another attention."""
    n = 90
    g = torch.Generator(device=DEV).manual_seed(12)
    freqs, m = dsa.rope_freqs(64, scaling="yarn", factor=40.0, device=DEV)
    scale = 192 ** -0.5
    lat = (torch.randn(n, 576, generator=g, device=DEV) * 0.5).bfloat16()
    key = torch.randn(n, 128, generator=g, device=DEV).bfloat16()
    raw = torch.randn(1, 128, 576, generator=g, device=DEV).bfloat16()
    lay, at = dsa.KvLayout(1, n), torch.tensor([n - 1], device=DEV, dtype=torch.int32)
    idx = torch.arange(n, device=DEV, dtype=torch.int32)[None]
    fn = freqs.cpu().numpy()
    # the definition: rotate without a factor, multiply the logits by m^2
    rows = rope_rows(lat.double().cpu().numpy()[:, None], range(n), fn, rot_begin=512,
                     interleaved=True)[:, 0]
    q64 = rope_rows(raw.double().cpu().numpy(), [n - 1], fn, rot_begin=512, interleaved=True)
    want, lse64 = sparse_mla_token(q64[0], rows, scale * m * m, 512)
    lses = []
    for magnitude, factor in ((1.0, m * m), (m, 1.0)):
        kv = torch.zeros(1, n, 576, device=DEV, dtype=torch.bfloat16)
        codes = torch.zeros(1, n, 128, device=DEV, dtype=torch.uint8)
        dsa.dsa_cache_append(lat, key, kv, codes, torch.zeros(1, n, device=DEV), lay, n, freqs,
                             magnitude=magnitude)
        q = dsa.dsa_rope(raw, at, freqs, rot_begin=512, interleaved=True, magnitude=magnitude)
        out, lse = dsa.dsa_sparse_mla_fwd(q, kv, lay, 1, idx, scale * factor)
        assert dsa.dsa_get_device_error() == 0
        lses.append(lse[0].double().cpu().numpy())
        if magnitude == 1.0:
            # beside the kernel's own tolerances: the 64 rotated dims rounded to bf16 on both
            # sides move a logit by at most 2 * 2^-8 (1 + 2^-8) sum |q_d c_d|
            d = 2.0 ** -7 * 1.01 * scale * m * m * (np.abs(q64[0, :, 512:]) @ np.abs(rows[:, 512:]).T).max(1)
            assert np.all(np.abs(lses[0] - lse64) <= LSE_ATOL + d)
            err = np.abs(out[0].double().cpu().numpy() - want)
            spread = np.abs(rows[:, :512]).max()
            assert np.all(err <= OUT_ATOL + np.expm1(2 * d)[:, None] * spread)
    d = 2.0 ** -7 * 1.01 * scale * m * m * (np.abs(q64[0, :, 512:]) @ np.abs(rows[:, 512:]).T).max(1)
    assert np.abs(lses[1] - lse64).max() > 5 * d.max()
