"""Layouts and arguments that the cache calls' host side has to refuse before
a pointer crosses the C ABI (no GPU)."""

import ctypes
import os
import re

import pytest
import torch

from bwd_flashattention_fwd_gb300 import build, gbattn


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


# Addresses 16 MB apart that are never dereferenced: every call below is refused on the host.
A = [0x1000000 * (i + 1) for i in range(16)]


@pytest.fixture(scope="module")
def lib():
    build.build()
    return gbattn.load_library()


def append(lib, B=2, Hkv=2, T=8, Lk=100, D=128, **over):
    a = dict(zip(("k_new", "v_new", "path", "accept_len", "cache_len", "seen", "k", "v", "pos", "cache_len_out",
                  "seen_out", "limit"), A))
    a.update(over)
    return lib.attn_cache_append(*a.values(), 0, B, Hkv, T, Lk, D, 1, None)


def evict(lib, B=2, Hkv=2, Lk=100, D=128, **over):
    a = dict(zip(("k", "v", "weight", "pos", "cache_len", "seen", "weight_out", "pos_out", "cache_len_out", "ws"), A))
    a.update(over)
    return lib.attn_cache_evict(*a.values(), 1 << 40, 0, B, Hkv, Lk, D, 50, 10, 1, None)


def tree(lib, B=2, Hq=8, Hkv=2, T=8, Lk=100, D=128, **over):
    a = dict(zip(("q", "k", "v", "k_new", "v_new", "tree_mask", "cache_len", "tree_len", "o", "lse", "ws"), A))
    a.update(over)
    return lib.attn_fwd_tree(*a.values(), 1 << 40, 0, B, Hq, Hkv, T, Lk, D, ctypes.c_float(0.1), 1, None)


def weight(lib, B=2, Hq=8, Hkv=2, Lq=8, Lk=100, D=128, **over):
    a = dict(zip(("q", "k", "lse", "limit", "weight", "weight_out", "ws"), A))
    a.update(over)
    return lib.attn_key_weight(*a.values(), 1 << 40, 0, B, Hq, Hkv, Lq, Lk, D, ctypes.c_float(0.1), 0, 1, None)


def refused(call, outputs, others, sizes):
    """Every output over each other array, at its start, over its last element and from below."""
    names = {n: A[i] for i, n in enumerate(call.names)}
    for o in outputs:
        for x in others:
            if x == o:
                continue
            for at in (names[x], names[x] + sizes[x] - 16, names[x] - sizes[o] + 16):
                assert call(**{o: at}) == gbattn.ATTN_ERR_INVALID_ARG, (o, x, at - names[x])


def named(fn, lib, names):
    def call(**over):
        return fn(lib, **over)

    call.names = names
    return call


def test_outputs_over_inputs_or_one_another_are_refused(lib):
    """Blocks read lengths, paths and weights while others write their outputs,
    so no output may share storage with any of them."""
    B, Hq, Hkv, T, Lk, D = 8, 8, 2, 8, 100, 128
    n = dict(B=B, Hkv=Hkv, Lk=Lk, D=D)
    ints = 4 * B
    call = named(lambda lib, **k: append(lib, T=T, **n, **k), lib,
                 ("k_new", "v_new", "path", "accept_len", "cache_len", "seen", "k", "v", "pos", "cache_len_out",
                  "seen_out", "limit"))
    sizes = dict(path=ints * T, accept_len=ints, cache_len=ints, seen=ints, pos=4 * B * Hkv * Lk, cache_len_out=ints,
                 seen_out=ints, limit=ints * T)
    refused(call, ("pos", "cache_len_out", "seen_out", "limit"), sizes, sizes)
    call = named(lambda lib, **k: evict(lib, **n, **k), lib,
                 ("k", "v", "weight", "pos", "cache_len", "seen", "weight_out", "pos_out", "cache_len_out"))
    slots = 4 * B * Hkv * Lk
    sizes = dict(weight=slots, pos=slots, cache_len=ints, seen=ints, weight_out=slots, pos_out=slots, cache_len_out=ints)
    refused(call, ("weight_out", "pos_out", "cache_len_out"), sizes, sizes)
    call = named(lambda lib, **k: tree(lib, Hq=Hq, T=T, **n, **k), lib,
                 ("q", "k", "v", "k_new", "v_new", "tree_mask", "cache_len", "tree_len", "o", "lse"))
    sizes = dict(q=B * Hq * T * D * 2, k_new=B * Hkv * T * D * 2, v_new=B * Hkv * T * D * 2, tree_mask=B * T * T,
                 cache_len=ints, tree_len=ints, o=B * Hq * T * D * 2, lse=B * Hq * T * 4)
    refused(call, ("o", "lse"), sizes, sizes)
    call = named(lambda lib, **k: weight(lib, Hq=Hq, Lq=T, **n, **k), lib,
                 ("q", "k", "lse", "limit", "weight", "weight_out"))
    sizes = dict(q=B * Hq * T * D * 2, lse=B * Hq * T * 4, limit=ints * T, weight=slots, weight_out=slots)
    refused(call, ("weight_out",), ("q", "lse", "limit"), sizes)
    for shift in (16, -16, slots - 16, 16 - slots):  # the same array is fine, a shifted one is not
        assert call(weight_out=A[4] + shift) == gbattn.ATTN_ERR_INVALID_ARG, shift


# Global arrays of the cache kernels that are indexed by something computed on
# the device, and how far above the access its check may stand (in lines).
CHECKED = {
    "cache_kernel.cuh": (r"[^_]freed\[.*\] = i", r"[^_]moving\[.*\] = i", r"evict_move\(p, bh, freed", r"path\[i\] [<>]",
                         r"limit\[t\] =", r"p\.weight\[row", r"p\.weight_out\[row", r"\(w\[j\], pos\[j\]", r"kd\[x\] =",
                         r"p\.pos\[at", r"= w\[i"),
    "key_weight_kernel.cuh": (r"p\.limit\[", r"p\.weight\[o\]", r"p\.weight_out\[o\] =", r"p\.part\[", r"p\.lse\["),
    "tree_kernel.cuh": (r"p\.part_lse\[", r"p\.lse\[grow\]", r"tree_mask_bits<", r"p\.part \+ r \*"),
}


@pytest.mark.parametrize("name", CHECKED)
def test_debug_build_checks_computed_indices(name):
    lines = open(os.path.join(os.path.dirname(gbattn.__file__), "csrc", name)).read().split("\n")
    check = re.compile(r"dbg_in_range|evict_slot_ok|list_ok\(|\bon\[u\]|\bmine\b")
    for access in CHECKED[name]:
        hits = [i for i, s in enumerate(lines) if re.search(access, s) and not s.lstrip().startswith("//")]
        assert hits, f"{name}: no line matches {access}"
        for i in hits:
            assert any(check.search(s) for s in lines[max(0, i - 12):i + 1]), f"{name}:{i + 1}: {lines[i].strip()}"


def test_debug_check_sites_are_unique():
    """A recorded site names one check."""
    sites = {}
    for name in CHECKED:
        text = open(os.path.join(os.path.dirname(gbattn.__file__), "csrc", name)).read()
        for n in re.findall(r"dbg_in_range\((?:[^;{]|\n)*?status,\s*(\d+)\)", text) + re.findall(r"evict_slot_ok\(p, [^;]*?, (\d+)\)", text):
            assert n not in sites, f"site {n}: {sites[n]} and {name}"
            sites[n] = name
    assert len(sites) >= 25
