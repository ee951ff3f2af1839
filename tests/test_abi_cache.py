"""CPU checks of the calls around the caches: struct layout and the host-side refusals
(nothing is launched: every call here fails its checks first)."""

import ctypes
import os
import subprocess
import tempfile

import pytest
import torch

from sparse_attention_05_b200 import dsa
from tests.test_abi import HEADER, _kv

by = ctypes.byref
FAKE = ctypes.c_void_p(0x100000)   # never dereferenced
OTHER = ctypes.c_void_p(0x900000)


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_05_b200.build import build
    build()
    return dsa.lib()


def test_rope_struct_layout_matches_c():
    src = r"""
    #include <stdio.h>
    #include <stddef.h>
    #include "dsa.h"
    int main(void) {
      printf("%zu %zu %zu %zu\n", sizeof(dsa_rope_desc_t), offsetof(dsa_rope_desc_t, magnitude),
             offsetof(dsa_rope_desc_t, num_rows), offsetof(dsa_rope_desc_t, out_head_stride));
      return 0;
    }
    """
    with tempfile.TemporaryDirectory() as d:
        c, exe = os.path.join(d, "l.c"), os.path.join(d, "l")
        open(c, "w").write(src)
        subprocess.run(["gcc", "-I", os.path.dirname(HEADER), c, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True).stdout.split()]
    D = dsa.RopeDescC
    assert got == [ctypes.sizeof(D), D.magnitude.offset, D.num_rows.offset,
                   D.out_head_stride.offset]


def _rope(**kw):
    d = dict(dtype=0, layout=1, heads=4, dim=96, rot_begin=32, rot_dim=64, magnitude=1.0,
             num_rows=3, x_row_stride=384, x_head_stride=96, out_row_stride=384,
             out_head_stride=96)
    d.update(kw)
    return dsa.RopeDescC(**d)


def _call_rope(lib, d, x=FAKE, out=OTHER, pos=FAKE, f=FAKE):
    a = lib.dsa_rope(x, pos, f, by(d), out, None)
    assert a == lib.dsa_rope_bwd(x, pos, f, by(d), out, None)
    return a


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=3), 1), (dict(layout=2), 1), (dict(heads=0), 1), (dict(dim=0), 1),
    (dict(rot_dim=0), 1), (dict(rot_dim=63), 1), (dict(rot_begin=-1), 1), (dict(rot_begin=33), 1),
    (dict(num_rows=-1), 1), (dict(magnitude=float("nan")), 1), (dict(magnitude=float("inf")), 1),
    (dict(x_row_stride=-1), 1), (dict(num_rows=1 << 31), 2),
    (dict(dim=1024, rot_begin=0, rot_dim=514, x_head_stride=1024, out_head_stride=1024), 2),
    (dict(heads=65536), 2), (dict(dim=32769, x_head_stride=1 << 17, out_head_stride=1 << 17), 2),
    (dict(out_head_stride=95), 1),      # heads of the output overlap
    (dict(out_head_stride=0), 1),
    (dict(out_row_stride=383), 1),      # rows of the output overlap
])
def test_rope_refusals(lib, bad, status):
    assert _call_rope(lib, _rope(**bad)) == status


def test_rope_refuses_null_unaligned_and_overlapping(lib):
    d = _rope()
    assert _call_rope(lib, d, x=None) == 1 and _call_rope(lib, d, out=None) == 1
    assert _call_rope(lib, d, pos=None) == 1 and _call_rope(lib, d, f=None) == 1
    assert _call_rope(lib, d, x=ctypes.c_void_p(0x100001)) == 1
    assert _call_rope(lib, d, f=ctypes.c_void_p(0x100004)) == 1
    # out one head into x: neither in place nor apart
    assert _call_rope(lib, d, out=ctypes.c_void_p(0x100000 + 96 * 2)) == 1
    # the same start with other strides, and a broadcast input written over itself
    assert _call_rope(lib, _rope(out_head_stride=128, out_row_stride=512), out=FAKE) == 1
    assert _call_rope(lib, _rope(x_head_stride=0), out=FAKE) == 1
    # no rows: nothing to do, whatever the pointers
    assert _call_rope(lib, _rope(num_rows=0), x=None, out=None, pos=None, f=None) == 0


def _append(lib, kv=None, q=None, lat=OTHER, ls=576, key=OTHER, ks=128, pos=None, f=FAKE, m=1.0,
            ll=1, kl=0, kvc=FAKE, ki=FAKE, sc=FAKE):
    return lib.dsa_cache_append(lat, ls, key, ks, pos, f, m, ll, kl, by(kv or _kv()),
                                by(q or dsa.QDescC(2, 1, 0, 0)), kvc, ki, sc, None)


def test_append_refusals(lib):
    for name in ("lat", "key", "f", "kvc", "ki", "sc"):
        assert _append(lib, **{name: None}) == 1, name
    for name in ("lat", "key", "kvc", "ki"):
        assert _append(lib, **{name: ctypes.c_void_p(0x100008)}) == 1, name
    assert _append(lib, sc=ctypes.c_void_p(0x100002)) == 1
    assert _append(lib, ls=568) == 1 and _append(lib, ls=580) == 1
    assert _append(lib, ks=120) == 1 and _append(lib, ks=129) == 1
    assert _append(lib, ls=(1 << 30) + 8) == 1 and _append(lib, ks=(1 << 30) + 8) == 1
    # new rows inside the caches: 1024 rows of 1152 and of 128 bytes
    assert _append(lib, lat=FAKE) == 1 and _append(lib, key=FAKE) == 1
    assert _append(lib, lat=ctypes.c_void_p(FAKE.value + 1023 * 1152)) == 1
    assert _append(lib, key=ctypes.c_void_p(FAKE.value + 1023 * 128)) == 1
    assert _append(lib, lat=ctypes.c_void_p(FAKE.value - 1152 - 16)) == 1   # its second row
    assert _append(lib, ll=2) == 1 and _append(lib, kl=3) == 1
    assert _append(lib, m=float("nan")) == 1
    assert _append(lib, q=dsa.QDescC(3, 1, 0, 0)) == 1
    assert _append(lib, kv=_kv(layout=1, page=48, pages=4, max_pages=16, bt=0x2000)) == 2
    # more window rows (batch * q_per_seq) than a grid takes
    many = _kv(batch=1 << 16, max_ctx=1 << 16, layout=1, page=64, pages=1024, max_pages=1024, bt=0x2000)
    assert _append(lib, kv=many, q=dsa.QDescC(5, 1 << 16, 0, 0, 0x3000)) == 2
    # a ragged batch without a single new token
    assert _append(lib, q=dsa.QDescC(0, 1, 0, 0, 0x3000), lat=None, key=None) == 0


def _mass(lib, kv=None, q=None, qp=FAKE, kvc=FAKE, idx=FAKE, k=16, scale=0.04, lse=FAKE,
          mass=FAKE, ld=512, ws=FAKE, nb=1 << 20):
    return lib.dsa_attn_mass(qp, kvc, by(kv or _kv()), by(q or dsa.QDescC(2, 1, 0, 0)), idx, k,
                             scale, lse, mass, ld, ws, nb, None)


def test_attn_mass_refusals(lib):
    for name in ("qp", "kvc", "idx", "lse", "mass"):
        assert _mass(lib, **{name: None}) == 1, name
    assert _mass(lib, k=0) == 2 and _mass(lib, k=(1 << 20) + 1) == 2
    assert _mass(lib, scale=0.0) == 1 and _mass(lib, scale=float("nan")) == 1
    assert _mass(lib, ld=511) == 1
    two = dsa.QDescC(4, 2, 0, 0)    # with one row a sequence there is no workspace
    assert _mass(lib, q=two, ws=None) == 6 and _mass(lib, q=two, ws=ctypes.c_void_p(0x100080)) == 6
    assert _mass(lib, q=two, nb=100) == 6
    assert lib.dsa_attn_mass_workspace_size(by(_kv()), by(dsa.QDescC(2, 1, 0, 0)), 16) == 0
    assert lib.dsa_attn_mass_workspace_size(by(_kv()), by(two), 16) == 256
    assert lib.dsa_attn_mass_workspace_size(by(_kv()), by(dsa.QDescC(2, 1, 0, 0)), 0) == 0
    assert lib.dsa_attn_mass_workspace_size(by(_kv()), by(dsa.QDescC(3, 1, 0, 0)), 16) == 0
    many = _kv(batch=65535, max_ctx=1 << 16, layout=1, page=64, pages=1024, max_pages=1024, bt=0x2000)
    assert _mass(lib, kv=many, q=dsa.QDescC(5, 1 << 16, 0, 0, 0x3000), ld=1 << 16) == 2
    assert _mass(lib, kv=_kv(batch=65536, max_ctx=16), q=dsa.QDescC(65536, 1, 0, 0), ld=16) == 2


def test_evict_and_compact_refusals(lib):
    kv = _kv()

    def sel(mass=FAKE, ld=512, keep=8, sink=2, recent=3, kept=FAKE, lens=FAKE):
        return lib.dsa_evict_select(mass, ld, by(kv), keep, sink, recent, kept, lens, None)
    for name in ("mass", "kept", "lens"):
        assert sel(**{name: None}) == 1, name
    assert sel(ld=511) == 1 and sel(keep=0, sink=0, recent=0) == 1
    assert sel(sink=-1) == 1 and sel(recent=-1) == 1 and sel(keep=4) == 1
    kv.seqlens = FAKE.value
    assert sel() == 1                             # new_lens over the lengths it reads
    kv = _kv(batch=1, max_ctx=(1 << 22) + 1)
    assert sel(ld=1 << 23) == 2
    kv = _kv()

    def com(a=FAKE, b=FAKE, c=FAKE, mass=FAKE, ld=512, kept=FAKE, keep=8, lens=FAKE, dst=None,
            ta=None, tb=None, tc=None, tm=None, tld=0):
        return lib.dsa_cache_compact(a, b, c, mass, ld, by(kv), kept, keep, lens,
                                     by(dst) if dst else None, ta, tb, tc, tm, tld, None)
    for name in ("a", "b", "c", "kept", "lens"):
        assert com(**{name: None}) == 1, name
    assert com(keep=0) == 1 and com(ld=511) == 1
    assert com(ta=FAKE) == 1                      # destination arrays without a geometry
    to = dict(dst=_kv(max_ctx=64), ta=OTHER, tb=OTHER, tc=OTHER, tm=OTHER, tld=64)
    assert com(**dict(to, tb=None)) == 1
    assert com(**dict(to, tm=None)) == 1          # mass without a place for it
    assert com(**dict(to, tld=63)) == 1
    assert com(**dict(to, dst=_kv(batch=3, max_ctx=64))) == 1
    assert com(**dict(to, ta=FAKE)) == 1          # contiguous into itself
    assert com(**dict(to, tb=FAKE)) == 1 and com(**dict(to, tc=FAKE)) == 1
    assert com(**dict(to, ta=ctypes.c_void_p(FAKE.value + 1023 * 1152))) == 1
    assert com(**dict(to, tb=ctypes.c_void_p(FAKE.value - 127 * 128))) == 1
    assert com(**dict(to, tc=ctypes.c_void_p(FAKE.value + 1023 * 4))) == 1
    assert com(**dict(to, tm=ctypes.c_void_p(FAKE.value + 512 * 4))) == 1   # mass into its second row
    kv = _kv(layout=1, page=64, pages=64, max_pages=8, bt=0x2000)
    same = _kv(max_ctx=64, layout=1, page=64, pages=64, max_pages=8, bt=0x2000)
    assert com(**dict(to, dst=same, ta=FAKE)) == 1  # the same pages
    kv = _kv()
    assert com(**dict(to, dst=_kv(layout=1, page=32, pages=4, max_pages=16, bt=0x2000))) == 2


ODD = 0x700002   # on no 4-byte boundary


def test_four_byte_pointers_are_refused_off_their_boundary(lib):
    odd = ctypes.c_void_p(ODD)
    for name in ("idx", "lse", "mass"):
        assert _mass(lib, **{name: odd}) == 1, name
    kv = _kv()

    def sel(mass=FAKE, kept=OTHER, lens=FAKE):
        return lib.dsa_evict_select(mass, 512, by(kv), 8, 2, 3, kept, lens, None)
    for name in ("mass", "kept", "lens"):
        assert sel(**{name: odd}) == 1, name

    def com(c=FAKE, mass=OTHER, kept=OTHER, lens=OTHER, dst=None, tc=None, tm=None):
        to = None if dst is None else ctypes.c_void_p(0x1900000)
        return lib.dsa_cache_compact(FAKE, FAKE, c, mass, 512, by(kv), kept, 8, lens,
                                     by(dst) if dst else None, to, to, tc, tm, 512, None)
    for name in ("c", "mass", "kept", "lens"):
        assert com(**{name: odd}) == 1, name
    far = ctypes.c_void_p(0x2900000)
    for name in ("tc", "tm"):
        assert com(**dict(dict(dst=_kv(), tc=far, tm=far), **{name: ctypes.c_void_p(0x2900002)})) == 1
    # lengths, block table and row starts of any call
    lens = _kv()
    lens.seqlens = ODD
    for name, desc in (("seqlens", lens),
                       ("table", _kv(layout=1, page=64, pages=64, max_pages=8, bt=ODD))):
        assert _append(lib, kv=desc) == 1 and _mass(lib, kv=desc) == 1, name
    assert _append(lib, q=dsa.QDescC(2, 1, 0, 0, ODD)) == 1
    assert _mass(lib, q=dsa.QDescC(2, 1, 0, 0, ODD)) == 1


def _at(v):
    return ctypes.c_void_p(v)


def test_outputs_that_overlap_what_is_read_are_refused(lib):
    """One byte range into another, at both ends (the library writes some of its outputs before it
    has read all of its inputs)."""
    kv = _kv()
    kv.seqlens = 0x50000
    paged = _kv(layout=1, page=64, pages=16, max_pages=8, bt=0x60000)

    def sel(mass=0x1000000, kept=0x2000000, lens=0x3000000):
        return lib.dsa_evict_select(_at(mass), 600, by(kv), 8, 2, 3, _at(kept), _at(lens), None)
    size = (600 + 512) * 4                              # two rows, the second to max_ctx
    assert sel(kept=0x1000000) == 1 and sel(kept=0x1000000 + size - 4) == 1
    assert sel(kept=0x1000000 - 2 * 8 * 4 + 4) == 1
    assert sel(lens=0x1000000 + size - 4) == 1
    assert sel(lens=0x50004) == 1 and sel(lens=0x50000 - 4) == 1   # shifted against the lengths
    assert sel(kept=0x50004) == 1
    assert sel(kept=0x3000000 - 8 * 4) == 1 and sel(lens=0x2000000 + 2 * 8 * 4 - 4) == 1
    # what does not overlap is not refused for it (there is no GPU: the launch fails, or the GPU
    # of a GPU machine is not asked)
    if not torch.cuda.is_available():
        assert sel(kept=0x1000000 + size) == 3 and sel(lens=0x50008) == 3

    # append: any of the three caches over any input
    caches = dict(kvc=_at(0x1000000), ki=_at(0x2000000), sc=_at(0x3000000))
    ins = dict(lat=_at(0x4000000), key=_at(0x5000000), pos=_at(0x6000000), f=_at(0x7000000))

    def app(desc=None, q=None, **kw):
        return _append(lib, kv=desc or _kv(), q=q, **dict(dict(caches, **ins), **kw))
    ends = dict(kvc=1024 * 1152, ki=1024 * 128, sc=1024 * 4)
    for c, n in ends.items():
        for i in ins:
            assert app(**{i: _at(caches[c].value + n - 16)}) == 1, (c, i)
        other = [o for o in ends if o != c][0]
        assert app(**{other: _at(caches[c].value + n - 16)}) == 1, c
    lens = _kv()
    lens.seqlens = 0x3000000 + 1024 * 4 - 4
    assert app(lens) == 1
    assert app(_kv(layout=1, page=64, pages=16, max_pages=8, bt=0x3000000 - 60)) == 1
    assert app(q=dsa.QDescC(2, 1, 0, 0, 0x3000000 - 8)) == 1

    # mass and workspace over the inputs and each other
    far = dict(qp=_at(0x10000000), kvc=_at(0x20000000), idx=_at(0x30000000), lse=_at(0x40000000),
               mass=_at(0x50000000), ws=_at(0x60000000), q=dsa.QDescC(4, 2, 0, 0))
    ends = dict(qp=4 * 147456, kvc=1024 * 1152, idx=4 * 16 * 4, lse=4 * 512)
    for name, n in ends.items():
        assert _mass(lib, **dict(far, mass=_at(far[name].value + n - 4))) == 1, name
        assert _mass(lib, **dict(far, ws=_at(far[name].value))) == 1, name
    assert _mass(lib, **dict(far, mass=_at(0x60000000))) == 1
    assert _mass(lib, **dict(far, kv=lens, mass=_at(lens.seqlens - 4))) == 1

    # rope: the output over positions and frequencies
    d = _rope()
    assert _call_rope(lib, d, pos=_at(OTHER.value + 3 * 384 * 2 - 4)) == 1
    assert _call_rope(lib, d, f=OTHER) == 1

    # compact: what is moved to over the lists, the lengths, the tables and the other arrays
    def com(a=0x1000000, b=0x2000000, c=0x3000000, mass=0x4000000, kept=0x5000000, lens=0x6000000,
            geometry=None, dst=None, to=(None,) * 4):
        return lib.dsa_cache_compact(_at(a), _at(b), _at(c), _at(mass), 512, by(geometry or kv),
                                     _at(kept), 8, _at(lens), by(dst) if dst else None,
                                     *(_at(t) for t in to), 512, None)
    ends = (0x1000000 + 1024 * 1152, 0x2000000 + 1024 * 128, 0x3000000 + 1024 * 4,
            0x4000000 + 1024 * 4)
    for end in ends:
        assert com(kept=end - 4) == 1 and com(lens=end - 4) == 1
        moved = _kv()
        moved.seqlens = end - 4
        assert com(geometry=moved) == 1
        assert com(geometry=_kv(layout=1, page=64, pages=16, max_pages=8, bt=end - 4)) == 1
    assert com(b=ends[0] - 16) == 1 and com(c=ends[1] - 4) == 1 and com(mass=ends[2] - 4) == 1
    to = (0x11000000, 0x12000000, 0x13000000, 0x14000000)
    other = _kv(layout=1, page=64, pages=16, max_pages=8, bt=0x70000)
    for i, start in enumerate(to):
        assert com(geometry=paged, dst=other, to=to, kept=start) == 1
        assert com(geometry=paged, dst=other, to=to, lens=start + 4) == 1
        for j, end in enumerate(ends):     # into its own arrays only as they are
            cross = to[:i] + (end - 16,) + to[i + 1:]
            assert com(geometry=paged, dst=other, to=cross) == 1, (i, j)
    table = _kv(layout=1, page=64, pages=16, max_pages=8, bt=to[2] + 64)
    assert com(geometry=paged, dst=table, to=to) == 1


def test_binding_refuses_wrong_tensors():
    """Types, shapes and devices the pointers alone would not show."""
    x = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        dsa.dsa_rope(torch.zeros(4), None, None)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x.double(), None, None)
    kv = dsa.KvLayout(2, 64)
    with pytest.raises(ValueError):
        dsa.dsa_evict_select(torch.zeros(2, 63), kv, 8)
    with pytest.raises(ValueError):
        dsa.dsa_evict_select(torch.zeros(2, 64), kv, 8)  # not on a GPU


def test_rope_refuses_to_drop_a_gradient():
    x = torch.zeros(2, 4, 64, requires_grad=True)
    args = (torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64))
    for call in (dsa.dsa_rope, dsa.dsa_rope_bwd):
        with pytest.raises(ValueError, match="gradient"):
            call(x, *args)
        with pytest.raises(ValueError, match="gradient"):
            call(x.detach(), *args, x)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(x, *args)
