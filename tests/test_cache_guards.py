"""Layouts and arguments that the cache calls' host side has to refuse before
a pointer crosses the C ABI (no GPU)."""

import os
import re

import pytest
import torch

from bwd_flashattention_fwd_gb300 import gbattn


def test_row_pitch_refuses_caches_without_a_row_per_head():
    """An expanded cache has one head's storage behind the shape of many: its
    strides say pitch 0, which the C ABI reads as "contiguous"."""
    k = torch.zeros(1, 1, 30, 64, dtype=torch.bfloat16)
    for shape in ((2, 3, 30, 64), (1, 3, 30, 64), (2, 1, 30, 64)):
        e = k.expand(shape)
        with pytest.raises(ValueError, match="not a slice"):
            gbattn.kv_row_pitch(e, e)
    # heads that overlap: fewer rows between them than each has
    for rows in (1, 29):
        o = torch.zeros(400 * 64, dtype=torch.bfloat16).as_strided((2, 3, 30, 64), (3 * rows * 64, rows * 64, 64, 1))
        with pytest.raises(ValueError, match="not a slice"):
            gbattn.kv_row_pitch(o, o)
    # one head alone, and heads that follow one another, are contiguous
    assert gbattn.kv_row_pitch(k, k) == 0
    assert gbattn.kv_row_pitch(k.expand(1, 1, 30, 64), k) == 0
    # a single row per head, and slices of one sequence or head
    c = torch.zeros(2, 3, 40, 64, dtype=torch.bfloat16)
    assert gbattn.kv_row_pitch(c[:, :, :1], c[:, :, :1]) == 40
    assert gbattn.kv_row_pitch(c[1:, :, 5:30], c[1:, :, :25]) == 40


def test_histograms_read_in_vectors_are_aligned_for_them():
    """Shared arrays that the eviction kernels read through int2* or as 16-byte
    pieces declare that alignment; the layout next to other arrays is the
    compiler's choice.  (The build has the same as a static_assert.)"""
    path = os.path.join(os.path.dirname(gbattn.__file__), "csrc", "cache_kernel.cuh")
    arrays = re.findall(r"__shared__ (.*?)int4? (hist|quad_sum)\[", open(path).read())
    assert sorted(n for _, n in arrays) == ["hist", "hist", "quad_sum"]
    assert all("__align__(16)" in how for how, _ in arrays), arrays


def test_explicit_pitch_stays_inside_the_tensors():
    """kv_pitch of the cache calls: what the strides say, or for heads that
    follow one another Lk or 0; a larger one would reach past the tensors.  A
    smaller one is left to the C ABI, which refuses it."""
    pitch = gbattn._cache_pitch
    k = torch.zeros(2, 3, 40, 64, dtype=torch.bfloat16)
    s = k[:, :, :25]
    assert pitch("call", k, k, 40) == 40 and pitch("call", k, k, 0) == 0 and pitch("call", s, s, 40) == 40
    for t, bad in ((k, 41), (k, 1 << 30), (s, 41), (s, 0), (s, 25), (s, 30)):
        with pytest.raises(ValueError, match="kv_pitch"):
            pitch("call", t, t, bad)
    for below in (39, 1, -1):
        assert pitch("call", k, k, below) == below
    one = k[:1, :1]  # nothing lies a pitch away from a single head
    assert pitch("call", one, one, 1000) == 1000
    with pytest.raises(ValueError):  # other layouts, whatever the pitch
        pitch("call", k.transpose(1, 2), k.transpose(1, 2), 40)
    e = k[:1, :1].expand(2, 3, 40, 64)
    with pytest.raises(ValueError):
        pitch("call", e, e, 40)
