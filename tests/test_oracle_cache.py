"""Pins of the cache oracle: closed forms, invariants and brute force (no GPU), and the
frequency schedules the package computes on the host."""

import math

import numpy as np
import pytest
import torch

from oracle import (append_token, attn_weight, e4m3_decode, evict_select, key_codes, rope_rows,
                    sparse_mla_token)
from sparse_attention_05_b200 import dsa

RNG = np.random.default_rng


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_complex_multiplication(interleaved):
    r = RNG(1)
    x, pos, f = r.normal(size=(5, 3, 20)), np.array([0, 1, -7, 1000, 123456]), r.random(4)
    y = rope_rows(x, pos, f, 1.5, rot_begin=8, interleaved=interleaved)
    part = x[..., 8:16]
    z = part[..., 0::2] + 1j * part[..., 1::2] if interleaved else part[..., :4] + 1j * part[..., 4:]
    z = z * 1.5 * np.exp(1j * pos[:, None, None] * f)
    w = np.stack([z.real, z.imag], -1).reshape(5, 3, 8) if interleaved else \
        np.concatenate([z.real, z.imag], -1)
    assert np.allclose(y[..., 8:16], w, atol=1e-9)
    assert np.array_equal(y[..., :8], x[..., :8]) and np.array_equal(y[..., 16:], x[..., 16:])


def test_scores_depend_on_the_distance_only_and_backward_is_the_transpose():
    r = RNG(2)
    q, k, f = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8)), r.random(4)
    dot = [np.sum(rope_rows(q, [a], f) * rope_rows(k, [a - 9], f)) for a in (9, 500, 7777)]
    assert np.allclose(dot, dot[0], atol=1e-9)
    x, dy = r.normal(size=(3, 2, 12)), r.normal(size=(3, 2, 12))
    kw = dict(rot_begin=2, interleaved=True)
    dx = rope_rows(dy, [5, 0, 31], f, 1.3, backward=True, **kw)
    # <dy, R x> = <R^T dy, x> up to the dims that pass through unchanged in both
    assert np.isclose(np.sum(dy * rope_rows(x, [5, 0, 31], f, 1.3, **kw)), np.sum(dx * x))


def test_append_token_keeps_the_latent_and_spans_the_e4m3_range():
    r = RNG(3)
    lat, key = r.normal(size=576), r.normal(size=128)
    f = r.random(32)
    y, k, s = append_token(lat, key, 17, f)
    assert np.array_equal(y[:512], lat[:512]) and not np.allclose(y[512:], lat[512:])
    codes = key_codes(k, s)
    assert np.max(np.abs(e4m3_decode(codes))) == 448.0
    assert np.max(np.abs(e4m3_decode(codes) * s - k)) <= np.max(np.abs(k)) * 2.0 ** -4 * 1.01
    assert append_token(lat, np.zeros(128), 17, f)[2] == np.float32(2.0 ** -120) / np.float32(448)


def test_weights_of_a_row_sum_to_one_for_the_forwards_lse():
    r = RNG(4)
    q, c = r.normal(size=(4, 576)), r.normal(size=(9, 576))
    _, lse = sparse_mla_token(q, c, 0.05, 512)
    p, _ = attn_weight(q, c, 0.05, lse)
    assert np.isclose(p.sum(), 1.0) and np.all(p > 0)


def test_eviction_against_a_sort():
    r = RNG(5)
    for trial in range(50):
        n = int(r.integers(1, 60))
        m = r.integers(0, 6, size=n).astype(np.float32) / 4  # many ties
        sink, recent = int(r.integers(0, 3)), int(r.integers(0, 4))
        keep = sink + recent + int(r.integers(0 if sink + recent else 1, 20))
        got = evict_select(m, n, keep, sink, recent)
        assert len(got) == min(n, keep) and got == sorted(set(got))
        if n > keep:
            assert set(range(sink)) <= set(got) and set(range(n - recent, n)) <= set(got)
            mid = [s for s in range(sink, n - recent)]
            out = [s for s in mid if s not in got]
            inn = [s for s in mid if s in got]
            for a in inn:
                for b in out:
                    assert (m[a], -a) > (m[b], -b)


def test_eviction_order_of_special_values():
    m = np.array([np.nan, -np.inf, -0.0, 0.0, np.inf, -1.0], np.float32)
    assert evict_select(m, 6, 1, 0, 0) == [4]
    assert evict_select(m, 6, 2, 0, 0) == [2, 4]      # -0 ties with +0: the lower slot
    assert evict_select(m, 6, 5, 0, 0) == [1, 2, 3, 4, 5]  # the NaN goes first


def test_frequency_schedules():
    f, m = dsa.rope_freqs(64)
    assert f.dtype == torch.float64 and f.shape == (32,) and m == 1.0
    assert f[0] == 1.0 and abs(float(f[-1]) - 10000 ** (-62 / 64)) < 1e-18
    lin, m = dsa.rope_freqs(64, scaling="linear", factor=8.0)
    assert torch.allclose(lin, f / 8, rtol=1e-15) and m == 1.0
    ntk, m = dsa.rope_freqs(64, scaling="ntk", factor=8.0)
    # the slowest pair is slowed by the factor, the fastest not at all
    assert ntk[0] == 1.0 and abs(float(ntk[-1] * 8 / f[-1]) - 1) < 1e-12 and m == 1.0
    yarn, m = dsa.rope_freqs(64, scaling="yarn", factor=40.0)
    assert m == 0.1 * math.log(40.0) + 1.0
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns > 32], f[turns > 32])
    assert torch.allclose(yarn[turns < 1], f[turns < 1] / 40, rtol=1e-15)
    assert torch.all(yarn <= f) and torch.all(yarn >= f / 40)
    for bad in (dict(rot_dim=7), dict(rot_dim=64, factor=0.0), dict(rot_dim=64, scaling="x"),
                dict(rot_dim=64, scaling="yarn", beta_fast=1.0, beta_slow=1.0),
                dict(rot_dim=2, scaling="ntk", factor=2.0)):
        with pytest.raises(ValueError):
            dsa.rope_freqs(**bad)
