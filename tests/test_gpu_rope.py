"""GPU parity of dsa_rope / dsa_rope_bwd against the fp64 oracle.

Tolerance per output (a, b the pair, m the magnitude). At positions up to 2^20 the angle in
turns is exact to 2^-34 before it is rounded to fp32 at |turns| <= 1/2 (2^-26 turns, 2^-23.3
rad); the sine and cosine add at most 2 ulp of 1 (2^-22), their product with m, the two products and
the sum five roundings of 2^-24. Together below 2^-21 (|a| + |b|) m; then one rounding to the
output type, half a step: eps/2 relative (for fp16 at least 2^-25 absolute)."""

import numpy as np
import pytest
import torch

from oracle import rope_rows
from sparse_attention_05_b200 import dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _bound(x, ref, half, rot_begin, interleaved, m, dtype, angle):
    mag = np.zeros_like(ref)
    for i in range(half):
        d0 = rot_begin + (2 * i if interleaved else i)
        d1 = rot_begin + (2 * i + 1 if interleaved else i + half)
        s = (np.abs(x[:, :, d0]) + np.abs(x[:, :, d1])) * abs(m) * (2.0 ** -21 + angle)
        mag[:, :, d0] = mag[:, :, d1] = s + 2.0 ** -140
    e = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0
    return np.where(mag > 0, mag * (1 + e) + np.abs(ref) * e + tiny, 0.0)


def _check(x, positions, freqs, m, got, angle=0.0, **kw):
    half = len(freqs)
    xn = x.double().cpu().numpy().reshape(x.shape[0], -1, x.shape[-1])
    ref = rope_rows(xn, positions.cpu().numpy(), freqs.cpu().numpy(), m, **kw)
    kw.pop("backward", None)
    tol = _bound(xn, ref, half, kw.get("rot_begin", 0), kw.get("interleaved", False), m, x.dtype,
                 angle)
    err = np.abs(got.double().cpu().numpy().reshape(ref.shape) - ref)
    assert np.all(err <= tol), f"max excess {np.max(err - tol):.3e}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rows,heads,before,rot,after", [
    (1, 1, 0, 64, 0), (2, 128, 512, 64, 0), (67, 3, 16, 32, 8), (300, 1, 0, 2, 0),
    (5, 7, 3, 10, 1), (33, 64, 0, 64, 64), (3, 2, 0, 512, 0), (2, 3, 1, 64, 7),
    (3, 2, 4000, 64, 1000), (2, 2, 8, 32, 24), (1000, 16, 8, 64, 0), (2, 1, 700, 6, 301),
])
def test_forward_and_backward(dtype, interleaved, rows, heads, before, rot, after):
    g = torch.Generator(device=DEV).manual_seed(rows * 131 + heads)
    x = torch.randn(rows, heads, before + rot + after, device=DEV, generator=g).to(dtype)
    pos = torch.randint(-5, 1 << 20, (rows,), device=DEV, generator=g, dtype=torch.int32)
    f, m = dsa.rope_freqs(rot, scaling="yarn" if rot > 2 else None, factor=32.0, device=DEV)
    kw = dict(rot_begin=before, interleaved=interleaved)
    y = dsa.dsa_rope(x, pos, f, magnitude=m, **kw)
    _check(x, pos, f, m, y, **kw)
    dx = dsa.dsa_rope_bwd(x, pos, f, magnitude=m, **kw)
    _check(x, pos, f, m, dx, backward=True, **kw)
    # in place: the same bits, and two-dimensional x as one head
    z = x.clone()
    assert dsa.dsa_rope(z, pos, f, z, magnitude=m, **kw) is z and torch.equal(z, y)
    if heads == 1:
        assert torch.equal(dsa.dsa_rope(x[:, 0], pos, f, magnitude=m, **kw), y[:, 0])
    assert dsa.dsa_get_device_error() == 0


def test_far_positions_keep_their_angle():
    """At the end of the int32 range an fp32 angle would be wrong by whole turns."""
    pos = torch.tensor([2**31 - 1, -2**31, 2**30 + 1, 16777217], device=DEV, dtype=torch.int32)
    x = torch.randn(4, 2, 64, device=DEV)
    f, m = dsa.rope_freqs(64, device=DEV)
    # below 2^28.4 turns in fp64: two roundings of 2^-53 are 2^-21 rad; the oracle's own angle
    # of up to 2^31 rad is rounded once, 2^-22
    _check(x, pos, f, m, dsa.dsa_rope(x, pos, f), angle=2.0 ** -20)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strided_views_and_untouched_neighbours(dtype):
    """The rope part of a projection's output into the last dims of the absorbed queries,
    heads-major storage, odd offsets, a broadcast key, interleaved views of one buffer."""
    f, m = dsa.rope_freqs(64, device=DEV)
    pos = torch.arange(6, device=DEV, dtype=torch.int32) * 1000
    src = torch.randn(6, 128, 192, device=DEV).to(dtype)
    dst = torch.full((6, 128, 576), 7.0, device=DEV, dtype=dtype)
    out = dsa.dsa_rope(src[..., 128:], pos, f, dst[..., 512:], interleaved=True)
    _check(src[..., 128:], pos, f, m, out, interleaved=True)
    assert torch.all(dst[..., :512] == 7.0)
    t = torch.randn(5, 6, 64, device=DEV).to(dtype).transpose(0, 1)   # head stride > row stride
    o = torch.empty(5, 6, 64, device=DEV, dtype=dtype).transpose(0, 1)
    _check(t, pos, f, m, dsa.dsa_rope(t, pos, f, o))
    odd = torch.randn(6, 3, 67, device=DEV).to(dtype)[..., 3:]        # no 16-byte alignment
    _check(odd, pos, f, m, dsa.dsa_rope(odd, pos, f))
    one = torch.randn(6, 1, 64, device=DEV).to(dtype).expand(6, 9, 64)
    y = dsa.dsa_rope(one, pos, f)
    _check(one, pos, f, m, y)
    assert torch.equal(y[:, 0], y[:, 8])
    buf = torch.randn(6, 4, 128, device=DEV).to(dtype)
    keep = buf[..., :64].clone()
    dsa.dsa_rope(buf[..., :64], pos, f, buf[..., 64:])
    _check(keep, pos, f, m, buf[..., 64:])
    assert torch.equal(buf[..., :64], keep)
    with pytest.raises(dsa.DSAError):                                  # one row into the next
        dsa.dsa_rope(buf.view(-1, 128)[:-1], pos[0].expand(23).contiguous(), f,
                     buf.view(-1, 128)[1:])


def test_many_heads_and_offsets_past_32_bits():
    f, m = dsa.rope_freqs(2, device=DEV)
    x = torch.randn(1, 65535, 2, device=DEV)
    pos = torch.tensor([12345], device=DEV, dtype=torch.int32)
    _check(x, pos, f, m, dsa.dsa_rope(x, pos, f))
    f, m = dsa.rope_freqs(64, device=DEV)
    buf = torch.zeros((1 << 32) + 4096, device=DEV, dtype=torch.bfloat16)  # 8 GB
    far = buf.as_strided((3, 2, 64), (1 << 31, 128, 1))
    far.copy_(torch.randn(3, 2, 64, device=DEV))
    pos = torch.tensor([1, 2, 3], device=DEV, dtype=torch.int32)
    out = torch.empty(3, 2, 64, device=DEV, dtype=torch.bfloat16)
    _check(far, pos, f, m, dsa.dsa_rope(far, pos, f, out))
    dsa.dsa_rope(far, pos, f, far)
    assert torch.equal(far, out)


def test_gradient_is_the_transpose_and_matches_differences():
    f, m = dsa.rope_freqs(64, scaling="yarn", factor=4.0, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(9, 3, 96, device=DEV, generator=g)
    dy = torch.randn(9, 3, 96, device=DEV, generator=g)
    pos = torch.randint(0, 4096, (9,), device=DEV, generator=g, dtype=torch.int32)
    kw = dict(rot_begin=16, interleaved=True, magnitude=m)
    dx = dsa.dsa_rope_bwd(dy, pos, f, **kw)
    v = torch.randn(9, 3, 96, device=DEV, generator=g)
    # the map is linear: a difference of step 1 along v has no truncation error; each of the
    # 2592 products carries at most 2^-20 of (|a| + |b|) |dy| m
    lin = (dy.double() * (dsa.dsa_rope(x + v, pos, f, **kw).double()
                          - dsa.dsa_rope(x, pos, f, **kw).double())).sum()
    want = (dx.double() * v.double()).sum()
    tol = 2.0 ** -20 * 4 * m * float((dy.abs() * (x.abs() + v.abs())).sum() + (dx.abs() * v.abs()).sum())
    assert abs(float(lin - want)) <= tol
    # turning back: R^T R = m^2 on the rotated part, twice the bound of one turn
    back = dsa.dsa_rope_bwd(dsa.dsa_rope(x, pos, f, **kw), pos, f, **kw)
    part = slice(16, 80)
    assert torch.all((back[..., part] - m * m * x[..., part]).abs()
                     <= 2.0 ** -19 * m * m * x[..., part].abs().amax())
    assert torch.equal(back[..., :16], x[..., :16]) and torch.equal(back[..., 80:], x[..., 80:])


def test_broadcast_input_gradient_sums_over_the_heads():
    f, m = dsa.rope_freqs(64, device=DEV)
    pos = torch.arange(5, device=DEV, dtype=torch.int32) * 77
    dy = torch.randn(5, 16, 64, device=DEV)
    dx = dsa.dsa_rope_bwd(dy, pos, f).sum(1)
    ref = rope_rows(dy.double().cpu().numpy(), pos.cpu().numpy(), f.cpu().numpy(),
                    backward=True).sum(1)
    tol = 2.0 ** -20 * dy.abs().sum(1).max().item() * 2
    assert np.all(np.abs(dx.double().cpu().numpy() - ref) <= tol)


def test_no_rows_special_values_streams_and_graphs():
    f, _ = dsa.rope_freqs(64, device=DEV)
    assert dsa.dsa_rope(torch.zeros(0, 4, 64, device=DEV), torch.zeros(0, device=DEV,
                        dtype=torch.int32), f).shape == (0, 4, 64)
    x = torch.zeros(2, 1, 64, device=DEV)
    x[0, 0, 3], x[1, 0, 5] = float("nan"), float("inf")
    pos = torch.tensor([3, 4], device=DEV, dtype=torch.int32)
    y = dsa.dsa_rope(x, pos, f)
    assert torch.isnan(y[0, 0, [3, 35]]).all() and not torch.isfinite(y[1, 0, [5, 37]]).any()
    y[0, 0, [3, 35]] = 0
    y[1, 0, [5, 37]] = 0
    assert torch.all(y == 0)
    # another stream, and a graph replayed on new contents of the same buffers
    x = torch.randn(300, 8, 64, device=DEV)
    pos = torch.arange(300, device=DEV, dtype=torch.int32)
    want = dsa.dsa_rope(x, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = dsa.dsa_rope(x, pos, f, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)
    out, dx = torch.empty_like(x), torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dsa.dsa_rope(x, pos, f, out)
        dsa.dsa_rope_bwd(out, pos, f, dx)
    x.copy_(x.flip(0))
    graph.replay()
    assert torch.equal(out, dsa.dsa_rope(x, pos, f))
    assert torch.equal(dx, dsa.dsa_rope_bwd(out, pos, f))


@pytest.mark.parametrize("dtype,interleaved,rows,heads,dim,rot_begin,rot,offset", [
    # on 148 SMs, calls that give a thread eight heads: 2.4 million units and more, in place too
    (torch.bfloat16, False, 9600, 64, 128, 0, 64, 0),
    (torch.float32, True, 1201, 128, 192, 128, 64, 0),
    (torch.bfloat16, True, 8192, 61, 64, 0, 64, 0),    # heads past the last eight of a thread
    (torch.float16, True, 3001, 131, 128, 16, 96, 0),
    (torch.float16, False, 2200, 37, 67, 3, 64, 3),    # no 16-byte alignment
    (torch.float32, True, 721, 107, 65, 1, 64, 1),
    (torch.float32, False, 40, 250, 520, 1, 512, 0),   # a row's units over several blocks
])
def test_large_calls_equal_small_ones(dtype, interleaved, rows, heads, dim, rot_begin, rot, offset):
    """Forward, backward and in place, bit for bit what calls of few rows give (a thread then takes
    one head), and a sample of rows against the oracle."""
    g = torch.Generator(device=DEV).manual_seed(rows + heads)
    x = torch.empty(rows, heads, offset + dim, device=DEV, dtype=dtype)
    x = x.normal_(generator=g)[..., offset:]
    pos = torch.randint(-5, 1 << 20, (rows,), device=DEV, generator=g, dtype=torch.int32)
    f, m = dsa.rope_freqs(rot, scaling="yarn", factor=32.0, device=DEV)
    kw = dict(rot_begin=rot_begin, interleaved=interleaved, magnitude=m)
    y, dx = dsa.dsa_rope(x, pos, f, **kw), dsa.dsa_rope_bwd(x, pos, f, **kw)
    few = max(1, 100000 // (heads * dim))
    for r in range(0, rows, few):
        part = slice(r, r + few)
        assert torch.equal(y[part], dsa.dsa_rope(x[part], pos[part], f, **kw))
        assert torch.equal(dx[part], dsa.dsa_rope_bwd(x[part], pos[part], f, **kw))
    at = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device=DEV)
    kw.pop("magnitude")
    _check(x[at], pos[at], f, m, y[at], **kw)
    _check(x[at], pos[at], f, m, dx[at], backward=True, **kw)
    dsa.dsa_rope(x, pos, f, x, magnitude=m, **kw)
    assert torch.equal(x, y)
    assert dsa.dsa_get_device_error() == 0


def test_written_tensors_are_known_to_autograd():
    """A tensor that autograd saved and rope then wrote: its backward pass says so instead of
    using the new values. dsa_rope_bwd inside a torch.autograd.Function, as a training program
    would have it, gives the transposed turn."""
    f, m = dsa.rope_freqs(64, device=DEV)
    pos = torch.arange(6, device=DEV, dtype=torch.int32)
    x = torch.randn(6, 2, 64, device=DEV)
    w = torch.randn(6, 2, 64, device=DEV, requires_grad=True)
    y = (w * x).sum()
    dsa.dsa_rope(x, pos, f, x)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()
    with torch.inference_mode():
        z = torch.randn(6, 2, 64, device=DEV)
        dsa.dsa_rope(z, pos, f, z)

    class Rope(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return dsa.dsa_rope(x, pos, f)

        @staticmethod
        def backward(ctx, dy):
            return dsa.dsa_rope_bwd(dy, pos, f)
    (Rope.apply(w) * x).sum().backward()
    assert torch.equal(w.grad, dsa.dsa_rope_bwd(x, pos, f))
