"""Serving operators without a GPU: index arithmetic on hostile lengths and
page tables, argument refusals of the C ABI (fake pointers; nothing is
dereferenced or enqueued), and pins of the oracle's own definitions."""
import ctypes
import math
import os
import re
import shutil
import subprocess
import tempfile

import numpy as np
import pytest
import torch

import weight_only_mixed_amd as slq
from oracle import serve as orc
from weight_only_mixed_amd import serve

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = [0x10000000 * i for i in range(1, 16)]     # fake, 256-byte aligned addresses far apart
INVAL, NOTSUP, OK = slq.SLQ_EINVAL, slq.SLQ_ENOTSUP, slq.SLQ_OK


def cache(fmt=0, heads=8, dim=128, page=64, pages=100, ps=None, hs=None, ts=None, k=P[0], v=P[1], ks=P[2], vs=P[3]):
    ts = dim if ts is None else ts
    hs = page * ts if hs is None else hs
    ps = heads * hs if ps is None else ps
    return serve._Cache(fmt, heads, dim, page, pages, ps, hs, ts, k, v, ks, vs)


def seqs(batch=4, width=10, stride=None, table=P[4], lens=P[5], cu=P[6]):
    return serve._Seqs(batch, width, width if stride is None else stride, table, lens, cu)


def write(c=None, s=None, k=P[7], v=P[8], dtype=1, rows=4, st=(1024, 128, 1024, 128), max_new=1):
    c, s = c or cache(), s or seqs()
    return slq.lib().slq_kv_write(ctypes.addressof(c), ctypes.addressof(s), k, v, dtype, rows, *st, max_new, None)


def read(c=None, s=None, k=P[7], v=P[8], dtype=1, rows=4, max_rows=4):
    c, s = c or cache(), s or seqs()
    return slq.lib().slq_kv_read(ctypes.addressof(c), ctypes.addressof(s), k, v, dtype, rows, max_rows, None)


def attn(c=None, s=None, q=P[7], dtype=1, rows=4, hq=32, st=(4096, 128), scale=0.1, window=0, mq=1, ml=100000,
         out=P[8], lse=P[9], ws=P[10]):
    c, s = c or cache(), s or seqs(width=2000)     # long enough to be split: a workspace is needed
    return slq.lib().slq_kv_attention(ctypes.addressof(c), ctypes.addressof(s), q, dtype, rows, hq, *st, scale,
                                      window, mq, ml, out, lse, ws, None)


def sample(logits=P[0], dtype=0, rows=2, vocab=1000, stride=1000, u=P[1], t=P[2], k=P[3], p=P[4], m=P[5], tok=P[6],
           lp=P[7], ws=P[8]):
    return slq.lib().slq_sample(logits, dtype, rows, vocab, stride, u, t, k, p, m, tok, lp, ws, None)


def test_exports_every_declared_symbol():
    text = open(os.path.join(ROOT, "include", "slq_serve.h")).read()
    names = set(re.findall(r"\b(slq_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"slq_kv_write", "slq_kv_read", "slq_kv_attention_workspace_bytes", "slq_kv_attention",
                     "slq_sample_workspace_bytes", "slq_sample"}
    for n in names:
        assert hasattr(slq.lib(), n), n


@pytest.mark.parametrize("bad,want", [
    (dict(fmt=2), INVAL), (dict(heads=0), INVAL), (dict(heads=1025), INVAL), (dict(dim=96), NOTSUP),
    (dict(dim=0), INVAL), (dict(page=8), NOTSUP), (dict(page=48), NOTSUP), (dict(page=512), NOTSUP),
    (dict(pages=-1), INVAL), (dict(ts=120), INVAL), (dict(ts=112), INVAL), (dict(hs=64), INVAL),
    (dict(ps=65536 - 16), INVAL), (dict(ps=-65536), INVAL), (dict(hs=-8192), INVAL), (dict(ts=0), INVAL),
    (dict(ps=0), INVAL), (dict(k=None), INVAL), (dict(vs=None), INVAL), (dict(k=P[0] + 8), INVAL),
    (dict(ks=P[2] + 2), INVAL), (dict(v=P[0] + 65536), INVAL), (dict(v=P[0]), INVAL), (dict(ks=P[0] + 64), INVAL),
    (dict(vs=P[2] + 16), INVAL),
])
def test_cache_refusals(bad, want):
    assert write(c=cache(**bad)) == want
    assert read(c=cache(**bad)) == want
    assert attn(c=cache(**bad)) == want
    c, s = cache(**bad), seqs()
    assert slq.lib().slq_kv_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(s), 4, 32, 0, 1, 640) == 0


def test_cache_layouts_that_are_accepted():
    """rows = 0 validates everything and enqueues nothing."""
    for c in (cache(), cache(ts=1024, hs=128, ps=65536),                  # slots outside heads
              cache(ps=131072, v=P[0] + 65536),                           # K and V alternate page by page
              cache(heads=1, hs=0, ps=8192), cache(pages=1, ps=0), cache(dim=256), cache(dim=64, page=16)):
        assert write(c=c, rows=0) == OK and read(c=c, rows=0) == OK and attn(c=c, rows=0, hq=c.heads) == OK
    assert write(c=cache(pages=0, k=None, v=None, ks=None, vs=None)) == OK


@pytest.mark.parametrize("bad", [
    dict(batch=-1), dict(batch=65537), dict(width=0), dict(stride=9), dict(table=None), dict(lens=None), dict(cu=None),
    dict(table=P[4] + 2), dict(width=1 << 25), dict(table=P[0])])
def test_batch_refusals(bad):
    assert write(s=seqs(**bad)) == INVAL
    if bad != dict(table=P[0]):                # only outputs may not overlap the table
        assert read(s=seqs(**bad)) == INVAL and attn(s=seqs(**bad)) == INVAL


def test_write_and_read_refusals():
    assert write(s=seqs(batch=0)) == OK and read(s=seqs(batch=0)) == OK
    for kw in (dict(dtype=3), dict(dtype=-1), dict(rows=-1), dict(rows=1 << 27), dict(max_new=0), dict(k=None),
               dict(v=None), dict(k=P[7] + 8), dict(st=(1020, 128, 1024, 128)), dict(st=(1024, 4, 1024, 128)),
               dict(st=(1024, 128, -1024, 128)), dict(k=P[0]), dict(v=P[3])):
        assert write(**kw) == INVAL, kw
    for kw in (dict(dtype=3), dict(rows=-1), dict(max_rows=0), dict(k=None), dict(v=P[8] + 4), dict(v=P[7]), dict(k=P[1]),
               dict(v=P[2]), dict(k=P[4])):
        assert read(**kw) == INVAL, kw


def test_attention_refusals():
    assert attn(dtype=0) == NOTSUP
    for kw in (dict(dtype=3), dict(rows=-1), dict(rows=1 << 25), dict(hq=0), dict(hq=12), dict(window=-1), dict(mq=0),
               dict(ml=0), dict(scale=math.inf), dict(scale=math.nan), dict(q=None), dict(q=P[7] + 2), dict(out=None),
               dict(out=P[7]), dict(out=P[0]), dict(lse=P[9] + 1), dict(lse=P[8]), dict(st=(4095, 128)),
               dict(out=P[4]), dict(ws=None), dict(ws=P[10] + 16), dict(ws=P[8])):
        assert attn(**kw) == INVAL, kw
    assert attn(s=seqs(batch=0)) == OK and attn(rows=0, ws=None) == OK


def test_attention_workspace_sizes():
    """A few rows split over long tokens need one; a hint that contradicts the rows
    does not make it large; short and wide calls need none."""
    def size(rows, mq, ml, batch=1, hq=32):
        c, s = cache(), seqs(batch=batch, width=1 << 14)
        return slq.lib().slq_kv_attention_workspace_bytes(ctypes.addressof(c), ctypes.addressof(s), rows, hq, 0, mq, ml)
    assert 0 < size(1, 1, 1 << 20) <= 256 * 32 * 129 * 4
    assert size(1, 1, 100) == 0 and size(64, 1, 4000, batch=64) > 0 and size(1000, 1, 10 ** 6, batch=1000) == 0
    assert size(1 << 20, 1, 1 << 20) == 0 and size(1 << 20, 1 << 20, 1 << 20) == 0


def test_sample_refusals():
    for kw in (dict(dtype=3), dict(rows=-1), dict(rows=1 << 22), dict(vocab=0), dict(vocab=(1 << 24) + 1), dict(stride=-1),
               dict(logits=None), dict(u=None), dict(tok=None), dict(logits=P[0] + 2), dict(u=P[1] + 1), dict(t=P[2] + 2),
               dict(tok=P[6] + 3), dict(tok=P[0]), dict(lp=P[6]), dict(tok=P[1]), dict(lp=P[4])):
        assert sample(**kw) == INVAL, kw
    assert sample(rows=0, logits=None) == OK


def test_python_refusals():
    """The binding refuses before it touches the library or the GPU."""
    codes, scales = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1)
    with pytest.raises(slq.SlqError):
        slq.KvCache(codes, codes.clone(), scales, scales.clone(), 0)            # not on a GPU
    with pytest.raises(slq.SlqError):
        slq.KvCache(codes.float(), codes, scales, scales, 0)
    with pytest.raises(slq.SlqError):
        slq.KvCache(codes, codes[:1], scales, scales, 0)
    with pytest.raises(slq.SlqError):
        slq.KvSeqs(torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))
    with pytest.raises(slq.SlqError) as e:
        slq.slq_sample(torch.zeros(2, 8), torch.zeros(2))
    assert e.value.status == INVAL


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ is not available")
def test_index_arithmetic_under_sanitizers():
    with tempfile.TemporaryDirectory() as tmp:
        exe = os.path.join(tmp, "kv_view_driver")
        subprocess.run(["g++", "-std=c++17", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g", "-O1",
                        os.path.join(ROOT, "tests", "sanitize", "kv_view_driver.cpp"), "-o", exe], check=True)
        r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and "0 failing checks" in r.stdout, (r.stdout + r.stderr)[-3000:]


# ---- pins of the definitions

def test_e4m3_codes():
    """The value table and the encoder against torch's type on the CPU."""
    codes = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    v = orc.decode(codes, orc.E4M3)
    assert np.array_equal(np.isnan(t), np.isnan(v)) and np.array_equal(t[~np.isnan(t)], v[~np.isnan(v)])
    g = np.random.default_rng(3)
    y = np.concatenate([v[~np.isnan(v)], (v[:126] + v[1:127]) / 2, g.standard_normal(20000) * 50,
                        g.standard_normal(5000) * 0.01]).astype(np.float32)
    y = np.clip(y, -448, 448)
    assert np.array_equal(orc.encode(y, orc.E4M3),
                          torch.from_numpy(y).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("fmt", [0, 1])
def test_oracle_cache_round_trip(fmt):
    """One write of whole sequences: every value within half a step of its page's
    scale; token by token the scale is the running maximum."""
    g = np.random.default_rng(fmt)
    page, heads, dim = 16, 2, 64
    x = g.standard_normal((37, heads, dim)).astype(np.float32)
    table, lens, cu = np.array([[2, 0, 3]]), np.array([37]), np.array([0, 37])
    codes, scales = np.full((4, heads, page, dim), 0x55, np.uint8), np.full((4, heads), np.nan, np.float32)
    orc.kv_write(codes, scales, table, lens, cu, x, fmt)
    y = orc.kv_rows(codes, scales, table, lens, cu, 37, fmt)
    s = np.repeat(scales[[2, 0, 3]], page, 0)[:37][:, :, None]
    bound = 0.5001 * s if fmt == 0 else np.maximum(np.abs(x) / 16, s * 2.0 ** -10) * 1.0001
    assert np.all(np.abs(y - x) <= bound)
    assert np.all(codes[1] == 0x55) and np.all(codes[3, :, 5:] == 0x55) and np.isnan(scales[1]).all()
    c2, s2 = codes.copy(), np.full_like(scales, np.nan)
    for t in range(37):
        orc.kv_write(c2, s2, table, np.array([t + 1]), np.array([0, 1]), x[t:t + 1], fmt)
    assert np.array_equal(s2[[2, 0, 3]], scales[[2, 0, 3]])
    y2 = orc.kv_rows(c2, s2, table, lens, cu, 37, fmt)
    assert np.all(np.abs(y2 - x) <= 6 * bound)


def test_oracle_attention_closed_forms():
    g = np.random.default_rng(1)
    kc, vc = (g.integers(-127, 128, (3, 1, 16, 64)).astype(np.int8).view(np.uint8) for _ in range(2))
    one = np.ones((3, 1), np.float32)
    table, lens, cu = np.array([[1, 2, 0]]), np.array([40]), np.array([0, 2])
    q = np.zeros((2, 3, 64))
    o, lse, _, _ = orc.kv_attention(kc, one, vc, one, table, lens, cu, q, 0, 0.3)
    V = orc.decode(vc[[1, 2, 0], 0], 0).reshape(48, 64)
    assert np.allclose(o[1], V[:40].mean(0)) and np.allclose(o[0], V[:39].mean(0)) and np.allclose(lse, np.log([[39], [40]]))
    o, lse, _, _ = orc.kv_attention(kc, one, vc, one, table, lens, cu, q, 0, 0.3, window=1)
    assert np.allclose(o[1], V[39]) and np.allclose(lse, 0)
    o, lse, _, _ = orc.kv_attention(kc, one, vc, one, table, np.array([1]), cu, q, 0, 0.3)
    assert np.all(o[0] == 0) and np.all(np.isneginf(lse[0])) and np.allclose(o[1], V[0])


def test_oracle_sample_by_hand():
    l = np.log(np.array([[0.1, 0.4, 0.2, 0.3]] * 8))
    u = np.array([0.05, 0.1000001, 0.49, 0.51, 0.69, 0.71, 0.99, 0.0], np.float32)
    t, lp, n = orc.sample(l, u)
    assert t.tolist() == [0, 1, 1, 2, 2, 3, 3, 0] and np.allclose(lp, l[0][t])
    t, lp, n = orc.sample(l, u, top_k=np.full(8, 2))
    assert set(t) == {1, 3} and np.all(n == 2) and np.allclose(np.exp(lp), np.where(t == 1, 4 / 7, 3 / 7))
    assert np.all(orc.sample(l, u, top_p=np.full(8, 0.69))[2] == 2)
    assert np.all(orc.sample(l, u, top_p=np.full(8, 0.71))[2] == 3)
    assert np.all(orc.sample(l, u, top_p=np.zeros(8))[2] == 1)
    assert np.all(orc.sample(l, u, min_p=np.full(8, 0.51))[2] == 2)
    assert np.all(orc.sample(l, u, temperature=np.zeros(8))[0] == 1)
    tie = np.zeros((1, 6))
    t, _, n = orc.sample(tie, np.array([0.99]), top_k=np.array([2]))
    assert t[0] == 1 and n[0] == 2
    assert orc.sample(np.full((1, 3), -np.inf), np.array([0.5]))[0][0] == -1
