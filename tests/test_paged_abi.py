"""The paged-cache entry points without a GPU: every declared symbol is
exported, bad arguments are refused with the documented status before any
launch, the frequency tables follow their formulas, and the workspace covers
every window and shorter key axis."""
import ctypes
import math
import os
import re

import numpy as np
import pytest
import torch

import dit_token_b200 as dit
from dit_token_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, ALIGN, UNSUP = 0, 1, 2, 3, 4
P = 0x10000  # an aligned, never dereferenced fake device address


@pytest.fixture(scope="module")
def L():
    build.build()
    return dit.library()


def test_every_declared_symbol_is_exported(L):
    text = open(os.path.join(ROOT, "include", "dit_paged.h")).read()
    names = sorted(set(re.findall(r"DIT_API\s+[\w\s\*]+?\b(dit_\w+)\s*\(", text)))
    assert names == ["dit_paged_attention", "dit_paged_attention_workspace", "dit_qk_rope_scaled",
                     "dit_qkv_rope_append", "dit_rope_frequencies"]
    for n in names:
        assert hasattr(L, n) and hasattr(dit, n) and n in dit.__all__


# ------------------------------------------------------------ frequencies

def table(n, **kw):
    f, gain = dit.dit_rope_frequencies(n, device="cpu", **kw)
    return f.numpy(), gain


def test_frequencies_without_scaling():
    f, gain = table(8, theta=10000.0)
    assert np.allclose(f, [1.0, 0.1, 0.01, 0.001], rtol=1e-15) and gain == 1.0


def test_linear_and_ntk():
    plain, _ = table(64)
    assert np.array_equal(table(64, scaling="linear", factor=4.0)[0], plain / 4.0)
    ntk, gain = table(64, scaling="ntk", factor=8.0)
    assert gain == 1.0 and ntk[0] == 1.0  # the fastest pair is kept, the slowest slowed by exactly the factor
    assert math.isclose(ntk[-1], plain[-1] / 8.0, rel_tol=1e-13)
    assert table(2, scaling="ntk", factor=8.0)[0].tolist() == [1.0]
    for kind in ("linear", "ntk", "yarn"):
        assert np.allclose(table(64, scaling=kind, factor=1.0, original_len=4096)[0], plain, rtol=1e-15)


def test_yarn_bands():
    plain, _ = table(128)
    f, gain = table(128, scaling="yarn", factor=8.0, original_len=4096)
    assert gain == np.float32(0.1 * math.log(8.0) + 1.0)
    turns = 4096 * plain / (2 * math.pi)  # turns a pair makes over the trained context
    assert np.allclose(f[turns > 40], plain[turns > 40], rtol=1e-15)        # many turns: kept
    assert np.allclose(f[turns < 0.8], plain[turns < 0.8] / 8, rtol=1e-15)  # less than one: compressed
    ratio = f / plain
    assert (np.diff(ratio) <= 1e-15).all() and ((ratio > 0.125 - 1e-12) & (ratio < 1 + 1e-12)).all()
    # a context so short that no pair makes 32 turns, and so long that every pair makes one
    assert np.isfinite(table(16, scaling="yarn", factor=4.0, original_len=2)[0]).all()
    assert np.isfinite(table(16, scaling="yarn", factor=4.0, original_len=10**9)[0]).all()


def test_frequency_refusals(L):
    out, gain = (ctypes.c_double * 64)(), ctypes.c_float()

    def call(n=64, theta=1e4, kind=0, factor=2.0, length=4096, fast=32.0, slow=1.0, out=out, gain=ctypes.byref(gain)):
        return L.dit_rope_frequencies(n, theta, kind, factor, length, fast, slow, out, gain)
    assert call() == OK
    assert call(n=0) == SHAPE and call(n=-2) == SHAPE and call(n=7) == SHAPE
    assert call(theta=0.0) == SHAPE and call(theta=math.inf) == SHAPE and call(theta=math.nan) == SHAPE
    assert call(kind=4) == UNSUP and call(kind=-1) == UNSUP
    assert call(kind=1, factor=0.5) == SHAPE and call(kind=2, factor=math.nan) == SHAPE
    assert call(kind=0, factor=0.0) == OK  # not read
    assert call(kind=3, length=0) == SHAPE and call(kind=3, theta=1.0) == SHAPE
    assert call(kind=3, slow=0.0) == SHAPE and call(kind=3, fast=0.5) == SHAPE
    assert call(out=None) == NULL and call(gain=None) == NULL
    with pytest.raises(dit.DitError):
        dit.dit_rope_frequencies(7, device="cpu")
    with pytest.raises(KeyError):
        dit.dit_rope_frequencies(8, scaling="other", device="cpu")


# ------------------------------------------------------------ refusals

def rope(L, **kw):
    a = dict(q=P, qs=256, k=P, ks=256, qo=P, qos=256, ko=P, kos=256, wq=P, wk=P, cs=P, cp=P, B=1, rows=16, hq=2, hk=2,
             d=128, f=P, r=64, grid=None, gf=None, st=0, sh=0, sw=0, po=None, gain=1.0, eps=1e-6, mode=0)
    a.update(kw)
    return L.dit_qk_rope_scaled(a["q"], a["qs"], a["k"], a["ks"], a["qo"], a["qos"], a["ko"], a["kos"], a["wq"],
                                a["wk"], a["cs"], a["cp"], a["B"], a["rows"], a["hq"], a["hk"], a["d"], a["f"],
                                a["r"], a["grid"], a["gf"], a["st"], a["sh"], a["sw"], a["po"], a["gain"], a["eps"],
                                a["mode"], None)


def test_rope_refusals(L):
    for k in ("q", "k", "cs", "cp", "f", "wq", "wk"):
        assert rope(L, **{k: None}) == NULL, k
    for k in ("q", "k", "qo", "ko", "wq", "wk", "f"):
        assert rope(L, **{k: P + 8}) == ALIGN, k
    for k in ("qs", "ks", "qos", "kos"):
        assert rope(L, **{k: 248}) == SHAPE, k
        assert rope(L, **{k: 260}) == ALIGN, k
    assert rope(L, r=0) == SHAPE and rope(L, r=136) == SHAPE and rope(L, r=60) == SHAPE and rope(L, r=-8) == SHAPE
    assert rope(L, d=96, qs=512, ks=512) == UNSUP and rope(L, d=0) == SHAPE and rope(L, mode=3) == UNSUP
    assert rope(L, B=-1) == SHAPE and rope(L, rows=1 << 31) == SHAPE and rope(L, hq=-1) == SHAPE
    assert rope(L, gain=math.inf) == SHAPE and rope(L, eps=-1.0) == SHAPE and rope(L, eps=math.nan) == SHAPE
    assert rope(L, grid=P, gf=P, st=24, sh=20, sw=18) == SHAPE and rope(L, grid=P, gf=P, st=22, sh=21, sw=21) == SHAPE
    assert rope(L, grid=P, st=24, sh=20, sw=20) == NULL          # the grid's own table is missing
    assert rope(L, grid=P, gf=P + 4, st=24, sh=20, sw=20) == ALIGN
    assert rope(L, po=P + 2) == ALIGN and rope(L, grid=P + 2, gf=P, st=24, sh=20, sw=20) == ALIGN
    assert rope(L, B=0, q=None) == OK and rope(L, rows=0, k=None) == OK and rope(L, hq=0, hk=0, q=None, k=None) == OK
    assert rope(L, qo=None, qos=0, ko=None, kos=0, q=None) == NULL  # in place: their strides are not read


def append(L, **kw):
    a = dict(q=P, qs=256, k=P, ks=256, v=P, vs=256, qo=P, qos=256, wq=None, wk=None, kc=P, vc=P, ps=4096, ss=256,
             hs=128, np=4, page=16, t=P, ts=8, mp=8, cl=P, cs=P, cp=P, B=1, rows=16, hq=2, hk=2, d=128, f=P, r=64,
             grid=None, gf=None, st=0, sh=0, sw=0, po=None, gain=1.0, eps=1e-6, mode=0)
    a.update(kw)
    return L.dit_qkv_rope_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qo"], a["qos"], a["wq"],
                                 a["wk"], a["kc"], a["vc"], a["ps"], a["ss"], a["hs"], a["np"], a["page"], a["t"],
                                 a["ts"], a["mp"], a["cl"], a["cs"], a["cp"], a["B"], a["rows"], a["hq"], a["hk"],
                                 a["d"], a["f"], a["r"], a["grid"], a["gf"], a["st"], a["sh"], a["sw"], a["po"],
                                 a["gain"], a["eps"], a["mode"], None)


def test_append_refusals(L):
    for k in ("q", "k", "v", "kc", "vc", "t", "cl", "cs", "cp", "f"):
        assert append(L, **{k: None}) == NULL, k
    for k in ("q", "k", "v", "qo", "kc", "vc", "f"):
        assert append(L, **{k: P + 8}) == ALIGN, k
    for k in ("qs", "ks", "vs", "qos"):
        assert append(L, **{k: 248}) == SHAPE, k
        assert append(L, **{k: 260}) == ALIGN, k
    assert append(L, wq=P) == NULL and append(L, wk=P) == NULL
    assert append(L, page=0) == SHAPE and append(L, np=-1) == SHAPE and append(L, mp=9) == SHAPE
    assert append(L, ss=120) == SHAPE and append(L, hs=64) == SHAPE and append(L, ps=-8) == SHAPE
    assert append(L, ps=4100) == ALIGN and append(L, ss=260) == ALIGN and append(L, hs=132) == ALIGN
    assert append(L, t=P + 2) == ALIGN and append(L, cl=P + 1) == ALIGN
    assert append(L, hk=0) == SHAPE and append(L, d=96, qs=512) == UNSUP and append(L, mode=7) == UNSUP
    assert append(L, B=0, k=None) == OK and append(L, rows=0, t=None) == OK


def attend(L, **kw):
    a = dict(q=P, qs=512, kc=P, vc=P, ps=4096, ss=256, hs=128, np=4, page=16, t=P, ts=8, mp=8, kl=P, cs=P, cp=P, B=1,
             rows=16, hq=4, hk=2, d=128, scale=0.1, causal=1, window=0, mc=0, mk=0, out=P, os=512, lse=None, ws=P,
             wb=1 << 30)
    a.update(kw)
    return L.dit_paged_attention(a["q"], a["qs"], a["kc"], a["vc"], a["ps"], a["ss"], a["hs"], a["np"], a["page"],
                                 a["t"], a["ts"], a["mp"], a["kl"], a["cs"], a["cp"], a["B"], a["rows"], a["hq"],
                                 a["hk"], a["d"], a["scale"], a["causal"], a["window"], a["mc"], a["mk"], a["out"],
                                 a["os"], a["lse"], a["ws"], a["wb"], None)


def test_attention_refusals(L):
    for k in ("q", "kc", "vc", "t", "kl", "cs", "cp", "out"):
        assert attend(L, **{k: None}) == NULL, k
    for k in ("q", "kc", "vc", "out", "ws"):
        assert attend(L, **{k: P + 8}) == ALIGN, k
    assert attend(L, qs=504) == SHAPE and attend(L, os=504) == SHAPE and attend(L, qs=516) == ALIGN
    assert attend(L, hq=3) == SHAPE and attend(L, hq=0) == SHAPE and attend(L, hk=0) == SHAPE
    assert attend(L, d=96) == UNSUP and attend(L, hk=65536, hq=65536, qs=65536 * 128, os=65536 * 128) == UNSUP
    assert attend(L, scale=0.0) == SHAPE and attend(L, scale=math.nan) == SHAPE and attend(L, scale=math.inf) == SHAPE
    assert attend(L, mp=1 << 27, ts=1 << 27) == UNSUP  # 2^31 keys
    assert attend(L, window=-1) == SHAPE and attend(L, wb=-1) == SHAPE and attend(L, page=0) == SHAPE
    assert attend(L, lse=P + 2) == ALIGN and attend(L, kl=P + 2) == ALIGN
    assert attend(L, B=0, q=None) == OK and attend(L, rows=0, out=None) == OK


def workspace(L, rows=16, B=1, hq=4, hk=2, d=128, mc=0, mk=100000, out=True):
    n = ctypes.c_int64(-1)
    st = L.dit_paged_attention_workspace(rows, B, hq, hk, d, mc, mk, ctypes.byref(n) if out else None)
    return st, n.value


def test_workspace(L):
    assert workspace(L, rows=-1)[0] == SHAPE and workspace(L, hq=3)[0] == SHAPE and workspace(L, mk=0)[0] == SHAPE
    assert workspace(L, d=80)[0] == UNSUP and workspace(L, out=False)[0] == NULL
    assert workspace(L, rows=0) == (OK, 0) and workspace(L, B=0) == (OK, 0)
    st, n = workspace(L)  # 8 pages of 16 in attend(): a longer key axis there
    assert st == OK and n > 0
    # one row over 100,000 keys is split; too small a workspace, or none, is refused
    long = dict(rows=1, B=1, np=7000, mp=7000, ts=7000)
    assert attend(L, wb=0, ws=None, **long) == SHAPE
    assert attend(L, wb=1 << 30, ws=None, **long) == NULL


def test_workspace_grows_with_the_keys(L):
    """The workspace of a length serves every shorter one, and (as a window
    only shortens the axis) every window."""
    rng = np.random.default_rng(0)
    for _ in range(300):
        rows, B = int(rng.integers(1, 3000)), int(rng.integers(1, 70))
        hk = int(rng.integers(1, 41))
        hq = hk * int(rng.integers(1, 9))
        d, mc = int(rng.choice([64, 128, 256])), int(rng.integers(0, 5000))
        keys = sorted(int(v) for v in np.exp(rng.uniform(0, np.log(2**31 - 1), 6)))
        sizes = [workspace(L, rows, B, hq, hk, d, mc, k)[1] for k in keys]
        assert sizes == sorted(sizes)


def test_python_refusals():
    t = torch.zeros(16, 256, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        dit.dit_qk_rope_scaled(t, t, i, i, num_q_heads=2, num_k_heads=2, head_dim=128, freqs=None)
    with pytest.raises(ValueError, match="CUDA"):
        dit.dit_paged_attention(t, t, t, i, i, i, i, num_q_heads=2, num_kv_heads=2, head_dim=128)
