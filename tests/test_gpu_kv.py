"""The paged 8-bit cache on the GPU against oracle/serve.py: codes, scales and
rows read back bit for bit, attention within bounds derived from the arithmetic.

Bounds of attention, per output (R = rounding of the output type, eps / 2):
  score error  e = 2^-24 (dim + 8) S + 2^-22 |lse| + 2^-20, S = max_j scale sum |q||k_j|
    (fp32 accumulation of exact products, one rounding of the factors, of the
    shift by the running maximum and of the base-2 exponential each);
  |out - ref| <= (2^-11 + 2.5 e) A + R (|ref| + (2^-11 + 2.5 e) A) + 2^-24 max|v|, A = sum_j p_j |v_j|
    (2^-11: a probability in binary16; p / sum p moves by at most 2 e relative;
    2^-24: probabilities are held times 2^11 in binary16, whose subnormals are
    2^-24 apart, so each of n <= 4096 loses at most 2^-25 / 2^11 = 2^-36 of a weight
    of 1, in units of the largest page scale times the largest code);
    (an output below 2^-14 is a binary16 subnormal, whose spacing is 2^-24 whatever
    its size: rounding to fp16 adds up to 2^-25 there, beside the relative R);
  |lse - ref| <= e."""
import numpy as np
import pytest
import torch

import weight_only_mixed_amd as slq
from oracle import serve as orc
from tests.gpu_util import DEV, say

pytestmark = pytest.mark.gpu
FMT = {"int8": slq.SLQ_KV_INT8, "e4m3": slq.SLQ_KV_E4M3}
T = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Box:
    """A cache on the GPU and its twin on the host."""

    def __init__(self, pages, heads, dim, page, fmt, order="hsd", seed=0, fill=None):
        g = np.random.default_rng(seed)
        self.fmt, self.page, self.dim, self.heads, self.pages = FMT[fmt], page, dim, heads, pages
        shape = (pages, heads, page, dim)
        if fill == "values":       # a cache in use
            self.codes = [self._codes(g, shape) for _ in range(2)]
            self.scales = [(g.uniform(0.2, 2.0, (pages, heads)) / (127 if fmt == "int8" else 448)).astype(np.float32)
                           for _ in range(2)]
        else:                      # unset memory: the worst bytes and scales
            self.codes = [np.full(shape, 0x7F if fmt == "e4m3" else 0x80, np.uint8) for _ in range(2)]
            self.scales = [np.full((pages, heads), np.nan, np.float32) for _ in range(2)]
        dev = []
        for c in self.codes:
            if order == "shd":
                dev.append(torch.from_numpy(c).permute(0, 2, 1, 3).contiguous().to(DEV).permute(0, 2, 1, 3))
            elif order == "both":   # K and V alternate in one allocation
                if not dev:
                    both = torch.from_numpy(np.stack(self.codes, 1)).to(DEV)
                dev.append(both[:, len(dev)])
            else:
                dev.append(torch.from_numpy(c).to(DEV))
        self.dev = slq.KvCache(*dev, *[torch.from_numpy(s).to(DEV) for s in self.scales], self.fmt)

    def _codes(self, g, shape):
        c = g.integers(0, 256, shape).astype(np.uint8)
        if self.fmt == slq.SLQ_KV_E4M3:
            c[(c & 0x7F) == 0x7F] = 0x38
        else:
            c[c == 0x80] = 0
        return c

    def host(self):
        torch.cuda.synchronize()
        return [t.cpu().numpy() for t in (self.dev.k_codes, self.dev.k_scales, self.dev.v_codes, self.dev.v_scales)]

    def same(self, what=""):
        kc, ks, vc, vs = self.host()
        for got, ref in ((ks, self.scales[0]), (vs, self.scales[1])):
            assert np.array_equal(got.view(np.uint32), ref.view(np.uint32)), what
        for got, ref in ((kc, self.codes[0]), (vc, self.codes[1])):
            assert np.array_equal(got, ref), (what, int((got != ref).sum()))

    def write(self, table, lens, cu, k, v, **kw):
        t = [torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV) for a in (table, lens, cu)]
        slq.slq_kv_write(self.dev, slq.KvSeqs(*t), k, v, **kw)
        for i, x in enumerate((k, v)):
            orc.kv_write(self.codes[i], self.scales[i], table, lens, cu, x.float().cpu().numpy(), self.fmt)


def gseqs(table, lens, cu):
    return slq.KvSeqs(*[torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV) for a in (table, lens, cu)])


def tables(g, lens, page, spare=2, width=None):
    held = [-(-int(n) // page) for n in lens]
    ids = g.permutation(sum(held) + spare)
    w = max(1, max(held)) if width is None else width
    table, at = np.full((len(lens), w), -1, np.int64), 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, sum(held) + spare


def rand(g, shape, dtype, scale=1.0):
    return torch.from_numpy((g.standard_normal(shape) * scale).astype(np.float32)).to(T[dtype]).to(DEV)


# ---------------------------------------------------------------- write and read

@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("page,dim,heads,order", [(16, 64, 3, "hsd"), (32, 128, 2, "shd"), (64, 256, 1, "hsd"),
                                                  (256, 64, 5, "both"), (128, 128, 8, "shd")])
def test_write_and_read(fmt, dtype, page, dim, heads, order):
    g = np.random.default_rng(page + dim + heads)
    lens = np.array([1, page, page + 1, 3 * page + 5, 0, 2 * page - 1])
    new = np.array([1, page, 1, 2 * page + 7, 0, page])
    table, pages = tables(g, lens, page)
    cu = np.concatenate([[0], np.cumsum(new)])
    box = Box(pages, heads, dim, page, fmt, order, seed=3)
    # what was there before this step
    past = lens - new
    pcu = np.concatenate([[0], np.cumsum(past)])
    box.write(table, past, pcu, rand(g, (pcu[-1], heads, dim), dtype, 0.5), rand(g, (pcu[-1], heads, dim), dtype))
    box.same("past")
    rows = int(cu[-1])
    k, v = rand(g, (rows + 3, heads, dim), dtype, 2.0), rand(g, (rows + 3, heads, dim), dtype)   # 3 rows behind the last
    k[0], v[1] = 0, 0
    box.write(table, lens, cu, k, v, max_new=None if page == 16 else int(new.max()))
    box.same("step")
    for out_t in ("fp32", "bf16", "fp16"):
        out = [torch.full((rows + 3, heads, dim), 7.0, dtype=T[out_t], device=DEV) for _ in range(2)]
        kk, vv = slq.slq_kv_read(box.dev, gseqs(table, lens, cu), rows + 3, T[out_t], out=out)
        for i, got in enumerate((kk, vv)):
            ref = torch.from_numpy(orc.kv_rows(box.codes[i], box.scales[i], table, lens, cu, rows + 3, box.fmt)).to(T[out_t])
            assert torch.equal(got[:rows].cpu(), ref[:rows]) and bool((got[rows:] == 7.0).all())
    # every token of every sequence
    full = np.concatenate([[0], np.cumsum(lens)])
    kk, vv = slq.slq_kv_read(box.dev, gseqs(table, lens, full), int(full[-1]), torch.float32, max_rows=1)
    for i, got in enumerate((kk, vv)):
        assert np.array_equal(got.cpu().numpy(), orc.kv_rows(box.codes[i], box.scales[i], table, lens, full, int(full[-1]), box.fmt))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("page", [16, 64])
def test_token_by_token_with_growing_scales(fmt, page):
    """Rows that grow and shrink: older codes move to each new scale."""
    g = np.random.default_rng(5)
    box = Box(8, 2, 64, page, fmt)
    table = np.array([[5, 1, 7], [2, 0, 3]])
    loud = 10.0 ** g.uniform(-3, 3, 2 * page + 3)
    for t in range(2 * page + 3):
        x, y = rand(g, (2, 2, 64), "bf16", loud[t]), rand(g, (2, 2, 64), "bf16", loud[-1 - t])
        box.write(table, np.array([t + 1, t + 1]), np.array([0, 1, 2]), x, y, max_new=1)
    box.same()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_unusual_values(fmt):
    """Zeros, infinities, NaN, the smallest and largest numbers, ties between codes."""
    box = Box(9, 1, 64, 16, fmt)
    x = torch.zeros(8 * 16, 1, 64)
    x[16:32] = torch.linspace(-1, 1, 1024).view(16, 1, 64)
    x[32, 0, 3], x[33, 0, 1], x[34, 0, 0] = float("inf"), float("-inf"), float("nan")
    x[48:64] = 1e-42 * torch.randn(16, 1, 64, generator=torch.Generator().manual_seed(1))
    x[64:80] = 3e38 * torch.rand(16, 1, 64, generator=torch.Generator().manual_seed(2))
    q = 127 if fmt == "int8" else 448
    x[80:96] = ((torch.arange(1024) % (2 * q)).float() / 2 - q / 2).view(16, 1, 64)      # multiples of half a step
    x[80, 0, 0] = float(q)
    x[96:112, :, :5] = float("nan")
    x[112] = 1e-45
    box.write(np.arange(8)[None], np.array([128]), np.array([0, 128]), x.to(DEV), (-x).to(DEV))
    box.same()
    # a page that held nothing but zeros takes the scale of what follows
    box2 = Box(2, 1, 64, 16, fmt)
    box2.write(np.array([[1]]), np.array([3]), np.array([0, 3]), torch.zeros(3, 1, 64, device=DEV), torch.zeros(3, 1, 64, device=DEV))
    box2.write(np.array([[1]]), np.array([4]), np.array([0, 1]), torch.ones(1, 1, 64, device=DEV), torch.ones(1, 1, 64, device=DEV))
    box2.same()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_codes_are_of_rounded_quotients(fmt):
    """Many mantissas at many scales, and values within an ulp of the border between
    two codes: the quotient is the IEEE one whichever way it is computed."""
    g = np.random.default_rng(21)
    pages, page = 200, 256
    box = Box(pages, 1, 256, page, fmt)
    x = g.standard_normal((pages, page, 256)) * 2.0 ** g.uniform(-70, 70, (pages, 1, 1))
    x = x.astype(np.float32)
    for p in range(pages):
        s = np.abs(x[p]).max() * (np.float32(1) / np.float32(127 if fmt == "int8" else 448))
        edge = (g.integers(-126, 126, 30000) + 0.5).astype(np.float32) * s
        at = 1 + g.permutation(page * 256 - 1)[:30000]
        flat = x[p].reshape(-1)
        top = np.abs(flat).argmax()
        near = edge * (1 + np.float32(2.0 ** -23) * g.integers(-1, 2, 30000).astype(np.float32))
        flat[at[at != top]] = near[at != top]
    x = torch.from_numpy(x.reshape(pages * page, 1, 256)).to(DEV)
    box.write(np.arange(pages)[None], np.array([pages * page]), np.array([0, pages * page]), x, -x)
    box.same()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_positions_and_pages_that_do_not_exist(fmt):
    """Negative positions, pages out of range, lengths behind the table, offsets
    behind the rows: not written, read as 0, the rest as usual."""
    g = np.random.default_rng(8)
    box = Box(6, 2, 64, 16, fmt)
    table = np.array([[0, 1], [6, 2], [3, -1], [4, 2 ** 31 - 1]])
    lens = np.array([5, 20, 32, 40])
    cu = np.array([0, 9, 25, 45, 60])          # 9 rows for 5 tokens; 16 on a bad first page; 20 into page -1; 15, 8 of them behind the table
    k, v = rand(g, (60, 2, 64), "fp32"), rand(g, (60, 2, 64), "fp32")
    box.write(table, lens, cu, k, v)
    box.same()
    out = [torch.full((60, 2, 64), 9.0, device=DEV) for _ in range(2)]
    got = slq.slq_kv_read(box.dev, gseqs(table, lens, cu), 60, torch.float32, out=out)
    for i in range(2):
        assert np.array_equal(got[i].cpu().numpy(), orc.kv_rows(box.codes[i], box.scales[i], table, lens, cu, 60, box.fmt))
    bad = np.array([0, 70, -5, 45, 50])
    box.write(table, np.array([5, -3, 32, 2 ** 31 - 1]), bad, k, v, max_new=3)
    box.same()


def test_strided_rows_and_broadcasts():
    """K and V as slices of one projection output, and one row for all heads."""
    g = np.random.default_rng(2)
    box = Box(3, 4, 64, 16, "int8")
    qkv = rand(g, (20, 6 * 64 + 2 * 4 * 64), "bf16")
    k, v = qkv[:, 6 * 64:10 * 64].unflatten(1, (4, 64)), qkv[:, 10 * 64:].unflatten(1, (4, 64))
    table = np.array([[2, 0]])
    box.write(table, np.array([20]), np.array([0, 20]), k, v)
    box.same()
    one = rand(g, (7, 1, 64), "bf16").expand(7, 4, 64)
    box.write(table, np.array([27]), np.array([0, 7]), one, one)
    box.same()


# ---------------------------------------------------------------- attention

def check_attention(box, table, lens, cu, q, window=0, scale=None, max_q=None, max_len=None, what="", oracle=None):
    """A call against the oracle; rows behind the last sequence stay."""
    dim, rows = box.dim, q.shape[0]
    sc = float(np.float32(1.0 / np.sqrt(dim) if scale is None else scale))
    out = torch.full(q.shape, 3.0, dtype=q.dtype, device=DEV)
    o, lse = slq.slq_kv_attention(box.dev, gseqs(table, lens, cu), q, scale=sc, window=window, max_q=max_q, max_len=max_len,
                                  out=out, with_lse=True)
    torch.cuda.synchronize()
    ro, rl, A, S = oracle or orc.kv_attention(box.codes[0], box.scales[0], box.codes[1], box.scales[1], table, lens, cu,
                                              q.float().cpu().numpy(), box.fmt, sc, window)
    got, gl = o.double().cpu().numpy(), lse.double().cpu().numpy()
    mine = ~np.isnan(rl)
    assert np.all(got[~mine] == 3.0), "rows of no sequence"
    empty = mine & np.isneginf(rl)
    assert np.all(got[empty] == 0) and np.all(np.isneginf(gl[empty]))
    on = mine & ~empty
    if on.any():
        with np.errstate(invalid="ignore"):
            e = 2.0 ** -24 * (dim + 8) * S + 2.0 ** -22 * np.abs(rl) + 2.0 ** -20
        rel = 2.0 ** -11 + 2.5 * e[on][:, None]
        R = torch.finfo(q.dtype).eps / 2
        vmax = 448 * np.nanmax(np.abs(box.scales[1]))
        bound = rel * A[on] + R * (np.abs(ro[on]) + rel * A[on]) + 2.0 ** -24 * vmax
        if q.dtype == torch.float16:
            bound += 2.0 ** -25
        err = np.abs(got[on] - ro[on])
        worst, wl = float((err / bound).max()), float((np.abs(gl[on] - rl[on]) / e[on]).max())
        say(f"attention {what}: out err/bound {worst:.3f}, lse err/bound {wl:.3f}")
        assert worst <= 1 and wl <= 1, what
    return o, lse


SHAPES = [
    # page, dim, heads, group, order, lens, new
    (16, 64, 2, 1, "hsd", [1], [1]),
    (16, 64, 1, 3, "shd", [17, 33, 1, 0, 100], [1, 1, 1, 0, 1]),
    (64, 128, 2, 4, "hsd", [700, 5, 64, 65], [1, 1, 1, 1]),
    (128, 128, 1, 8, "both", [129, 500], [1, 2]),
    (32, 128, 2, 5, "hsd", [200, 90], [7, 90]),
    (64, 128, 1, 7, "shd", [333], [130]),
    (256, 256, 1, 4, "hsd", [300, 513], [1, 1]),
    (16, 256, 2, 2, "shd", [100, 40], [33, 40]),
    (32, 64, 1, 40, "hsd", [90, 31], [1, 2]),
    (64, 64, 3, 1, "hsd", [260, 64, 63], [260, 64, 1]),
    (16, 128, 1, 1, "hsd", [150, 16, 15], [100, 16, 15]),
    (64, 128, 1, 16, "hsd", [257, 128], [64, 3]),
]


@pytest.mark.parametrize("fmt,dtype", [("int8", "bf16"), ("int8", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16")])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_attention(fmt, dtype, case):
    page, dim, heads, group, order, lens, new = SHAPES[case]
    g = np.random.default_rng(case)
    lens, new = np.array(lens), np.array(new)
    table, pages = tables(g, lens, page)
    cu = np.concatenate([[0], np.cumsum(new)])
    box = Box(pages, heads, dim, page, fmt, order, seed=case, fill="values")
    q = rand(g, (int(cu[-1]) + 2, heads * group, dim), dtype, 1.5)
    for window in (0, 1, 20):
        o, l = check_attention(box, table, lens, cu, q, window, max_q=int(new.max()), max_len=int(lens.max()),
                               what=f"{case} {fmt} {dtype} window {window}")
        # the hints change the grid, not the answer's validity
        check_attention(box, table, lens, cu, q, window, what="no hints")
        check_attention(box, table, lens, cu, q, window, max_q=1, max_len=1, what="hints too small")
        o2, l2 = slq.slq_kv_attention(box.dev, gseqs(table, lens, cu), q, window=window, max_q=int(new.max()),
                                      max_len=int(lens.max()), with_lse=True)
        n = int(cu[-1])
        assert torch.equal(o2[:n].view(torch.int16), o[:n].view(torch.int16)) and torch.equal(l2[:n], l[:n])


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 3, 70])
def test_attention_over_unset_and_foreign_slots(fmt, new):
    """Slots behind a sequence's end and pages in front of its window hold NaN
    codes and NaN scales; positions and pages that do not exist are masked."""
    g = np.random.default_rng(new)
    page, heads, dim = 16, 2, 128
    lens = np.array([71, 90, 75, 200])
    table, pages = tables(g, lens, page)
    box = Box(pages, heads, dim, page, fmt)                    # unset
    full = np.concatenate([[0], np.cumsum(lens)])
    box.write(table, lens, full, rand(g, (full[-1], heads, dim), "bf16"), rand(g, (full[-1], heads, dim), "bf16"))
    cu = np.arange(5) * new
    q = rand(g, (4 * new, heads * 2, dim), "bf16")
    check_attention(box, table, lens, cu, q, max_q=new, what="unset slots")
    check_attention(box, table, np.array([0, 1, 2, 0]), cu, q, what="almost nothing there")
    t2 = table.copy()
    t2[1, 2], t2[3, 0], t2[3, 5] = -1, pages, 2 ** 31 - 1
    check_attention(box, t2, lens, cu, q, what="pages that do not exist")
    check_attention(box, t2, lens, np.array([0, new, new, 3 * new, 4 * new + 50]), q, what="offsets")
    # a window: the pages before it are unset again
    win = 20
    for b in range(4):
        for p in range(max(0, lens[b] - new - win + 1) // page):
            for i in range(2):
                box.codes[i][table[b, p]] = 0x7F
                box.scales[i][table[b, p]] = np.nan
    box.dev.k_codes.copy_(torch.from_numpy(box.codes[0]))
    box.dev.v_codes.copy_(torch.from_numpy(box.codes[1]))
    box.dev.k_scales.copy_(torch.from_numpy(box.scales[0]))
    box.dev.v_scales.copy_(torch.from_numpy(box.scales[1]))
    check_attention(box, table, lens, cu, q, window=win, max_q=new, what="window")
    check_attention(box, table, lens, cu, q, window=win, what="window, no hints")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_attention_ranges(dtype):
    """Queries of very different sizes, steep softmaxes, page scales far apart."""
    g = np.random.default_rng(4)
    box = Box(20, 1, 128, 16, "int8", seed=1, fill="values")
    box.scales[1][:] = (10.0 ** g.uniform(-4, 0, (20, 1))).astype(np.float32)
    box.dev.v_scales.copy_(torch.from_numpy(box.scales[1]))
    table, lens, cu = np.arange(20)[None], np.array([311]), np.array([0, 9])
    q = rand(g, (9, 4, 128), "fp32") * torch.tensor([0, 1e-6, 1e-3, 0.1, 1, 5, 20, 50, 100.0], device=DEV)[:, None, None]
    check_attention(box, table, lens, cu, q.to(T[dtype]), what="sizes of q")
    if dtype == "bf16":
        big = rand(g, (9, 4, 128), "fp32") * torch.tensor(2.0 ** np.array([-120, -60, -30, -8, 0, 40, 60, 90, 110]),
                                                         dtype=torch.float32, device=DEV)[:, None, None]
        check_attention(box, table, lens, cu, big.to(T[dtype]), scale=2.0 ** -8, what="exponents of q")
    flat = torch.zeros(9, 4, 128, dtype=T[dtype], device=DEV)
    check_attention(box, table, lens, cu, flat, scale=-1.0, what="flat")
    zero = Box(20, 1, 128, 16, "int8", seed=1, fill="values")
    zero.scales[1][3:] = 0
    zero.dev.v_scales.copy_(torch.from_numpy(zero.scales[1]))
    check_attention(zero, table, lens, cu, q.to(T[dtype]), what="zero scales")


@pytest.mark.parametrize("new", [1, 40])
def test_attention_not_a_number(new):
    """A query of NaN gives NaN in its own row and head only, split or not."""
    g = np.random.default_rng(3)
    box = Box(40, 1, 128, 16, "int8", seed=2, fill="values")
    q = rand(g, (new, 4, 128), "bf16")
    q[0, 1, 5] = float("nan")
    for max_len in (1, 600):
        o, lse = slq.slq_kv_attention(box.dev, gseqs(np.arange(40)[None], [600], [0, new]), q, max_q=new, max_len=max_len,
                                      with_lse=True)
        bad = torch.isnan(o.float()).all(2)
        assert bool(bad[0, 1]) and int(bad.sum()) == 1 and not bool(torch.isnan(o.float()).any(2)[~bad].any())
        assert bool(torch.isnan(lse[0, 1])) and int(torch.isnan(lse).sum()) == 1


MORE = [
    # page, dim, heads, group, lens, new, window: many short sequences; many kv heads; a
    # group wider than any tile; long contexts under few prompt rows; lens behind the table
    (16, 64, 2, 3, list(range(0, 310)), [1] * 310, 0),
    (16, 64, 300, 1, [40, 7], [1, 7], 0),
    (32, 64, 1, 300, [65, 33], [2, 1], 16),
    (64, 128, 1, 4, [3000, 2900], [40, 33], 0),
    (64, 128, 1, 4, [3000, 2900], [40, 33], 2500),
    (16, 256, 1, 5, [1500], [50], 700),
    (16, 64, 1, 20, [2000, 1], [1, 1], 5000),
]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("case", range(len(MORE)))
def test_attention_unusual_batches(fmt, case):
    page, dim, heads, group, lens, new, window = MORE[case]
    g = np.random.default_rng(100 + case)
    lens, new = np.array(lens), np.minimum(np.array(new), lens)
    table, pages = tables(g, lens, page)
    cu = np.concatenate([[0], np.cumsum(new)])
    box = Box(pages, heads, dim, page, fmt, seed=case, fill="values")
    q = rand(g, (int(cu[-1]), heads * group, dim), "bf16", 1.5)
    sc = float(np.float32(1 / np.sqrt(dim)))
    ref = orc.kv_attention(box.codes[0], box.scales[0], box.codes[1], box.scales[1], table, lens, cu,
                           q.float().cpu().numpy(), box.fmt, sc, window)
    for kw in (dict(max_q=int(new.max()), max_len=int(lens.max())), {}, dict(max_q=1, max_len=1), dict(max_len=10 ** 12)):
        check_attention(box, table, lens, cu, q, window, what=f"unusual {case} {kw}", oracle=ref, **kw)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_more_tiles_than_the_grid(fmt, dim):
    """Every width of the decode kernel's query tile, and sequences with more rows
    than its grid covers in one pass (a batch whose other sequences are empty)."""
    g = np.random.default_rng(dim)
    box = Box(30, 1, dim, 16, fmt, seed=1, fill="values")
    for new, hint in ((17, 17), (33, 33), (45, 45), (64, 64), (100, 45), (130, 64), (100, 20), (70, 30), (100, 10)):
        batch = -(-new // hint)
        table = np.concatenate([g.permutation(30)[None]] * batch)
        lens, cu = np.array([170] + [0] * (batch - 1)), np.array([0] + [new] * batch)
        q = rand(g, (new, 1, dim), "bf16", 1.5)
        for max_len in (1, 480):
            check_attention(box, table, lens, cu, q, max_q=hint, max_len=max_len, what=f"{dim} {new} rows, {hint} expected")


@pytest.mark.parametrize("new", [1, 90])
def test_attention_lengths_behind_the_table(new):
    """A length that the table has no pages for: what the table holds is seen, by
    queries whose positions lie behind it too."""
    g = np.random.default_rng(new)
    box = Box(6, 1, 64, 16, "int8", fill="values")
    table = np.array([[0, 1, 2], [3, 4, 5]])
    q = rand(g, (2 * new, 2, 64), "bf16")
    for lens in ([60, 48], [1000, 2 ** 31 - 1], [-5, 47]):
        check_attention(box, table, np.array(lens), np.array([0, new, 2 * new]), q, max_q=new, what=f"lens {lens}")
        check_attention(box, table, np.array(lens), np.array([0, new, 2 * new]), q, window=30, what=f"lens {lens} window")


def test_two_streams_at_once():
    """Calls of different shapes in flight on two streams, each with its own workspace."""
    g = np.random.default_rng(33)
    jobs = []
    for n, new in ((3000, 1), (1500, 80)):
        box = Box(200, 2, 128, 16, "int8", seed=n, fill="values")
        s = gseqs(g.permutation(188)[None], [n], [0, new])
        q = rand(g, (new, 8, 128), "bf16")
        jobs.append((box, s, q, slq.slq_kv_attention(box.dev, s, q, max_q=new, max_len=n, with_lse=True), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for box, s, q, _, stream in jobs:
            with torch.cuda.stream(stream):
                got.append(slq.slq_kv_attention(box.dev, s, q, max_q=q.shape[0], max_len=3008, with_lse=True))
        torch.cuda.synchronize()
        for (box, s, q, ref, _), (o, lse) in zip(jobs, got):
            assert float((o.float() - ref[0].float()).abs().max()) <= 2.0 ** -6 * float(ref[0].float().abs().max())
            assert float((lse - ref[1]).abs().max()) <= 1e-4


def test_attention_strided_queries():
    g = np.random.default_rng(6)
    box = Box(4, 2, 64, 32, "e4m3", seed=2, fill="values")
    qkv = rand(g, (10, 8 * 64), "bf16")
    table, lens, cu = np.array([[3, 1], [0, 2]]), np.array([50, 33]), np.array([0, 6, 10])
    check_attention(box, table, lens, cu, qkv[:, :6 * 64].unflatten(1, (6, 64)), what="slice of a projection")
    check_attention(box, table, lens, cu, qkv[:, None, :64].expand(10, 4, 64), what="one query for all heads")


def test_attention_far_offsets():
    """Pages behind 4 GiB of codes, a long table, a long sequence split many times."""
    page, dim = 256, 256
    pages = 66000                                           # 4.3e9 bytes of codes
    kc = torch.empty(pages, 1, page, dim, dtype=torch.uint8, device=DEV)
    vc = torch.empty(pages, 1, page, dim, dtype=torch.uint8, device=DEV)
    ks, vs = torch.empty(pages, 1, device=DEV), torch.empty(pages, 1, device=DEV)
    cache = slq.KvCache(kc, vc, ks, vs, slq.SLQ_KV_INT8)
    g = np.random.default_rng(9)
    n = 5000
    used = np.sort(g.choice(np.arange(65600, pages), 20, replace=False))
    box = Box(20, 1, dim, page, "int8", fill="values")
    at = torch.from_numpy(used).to(DEV)
    kc[at], vc[at] = (torch.from_numpy(c).to(DEV) for c in box.codes)
    ks[at], vs[at] = (torch.from_numpy(s).to(DEV) for s in box.scales)
    q = rand(g, (1, 2, dim), "bf16")
    ref = orc.kv_attention(box.codes[0], box.scales[0], box.codes[1], box.scales[1], np.arange(20)[None], np.array([n]),
                           np.array([0, 1]), q.float().cpu().numpy(), box.fmt, float(np.float32(1 / 16)))
    box.dev = cache
    check_attention(box, used[None], np.array([n]), np.array([0, 1]), q, scale=1 / 16, max_q=1, max_len=n, what="far", oracle=ref)
    k = rand(g, (1, 1, dim), "bf16", 9.0)
    slq.slq_kv_write(cache, gseqs(used[None], [n + 1], [0, 1]), k, k)
    kk, _ = slq.slq_kv_read(cache, gseqs(used[None], [n + 1], [0, 1]), 1, torch.float32)
    assert float((kk - k.float()).abs().max()) <= 0.51 * float(k.abs().max()) / 127


def test_streams_and_graph_replays():
    """A step captured once and replayed with other lengths, tables and inputs, with
    eager work on another stream in between; every replay against the eager call."""
    g = np.random.default_rng(12)
    page, heads, dim, B = 16, 2, 64, 3
    table = torch.from_numpy(g.permutation(30).reshape(3, 10).astype(np.int32)).to(DEV)
    lens, cu = torch.full((B,), 40, dtype=torch.int32, device=DEV), torch.arange(B + 1, dtype=torch.int32, device=DEV)
    k, v = torch.zeros(B, heads, dim, device=DEV), torch.zeros(B, heads, dim, device=DEV)
    q = torch.zeros(B, heads * 4, dim, dtype=torch.bfloat16, device=DEV)
    a, b = Box(30, heads, dim, page, "int8", fill="values"), Box(30, heads, dim, page, "int8", fill="values")
    out, lse = torch.empty_like(q), None

    def step(box, t, n, o):
        s = slq.KvSeqs(t, n, cu)
        slq.slq_kv_write(box.dev, s, k, v, max_new=1)
        return slq.slq_kv_attention(box.dev, s, q, max_q=1, max_len=160, out=o, with_lse=True)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(a, table, lens, out)                           # loads the kernels; a's cache is reset below
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _, lse = step(a, table, lens, out)
    torch.cuda.synchronize()
    a.dev.k_codes.copy_(b.dev.k_codes), a.dev.v_codes.copy_(b.dev.v_codes)
    a.dev.k_scales.copy_(b.dev.k_scales), a.dev.v_scales.copy_(b.dev.v_scales)
    for r in range(6):
        lens.fill_(40 + 7 * r)
        k.copy_(rand(g, k.shape, "fp32")), v.copy_(rand(g, v.shape, "fp32")), q.copy_(rand(g, q.shape, "bf16"))
        torch.cuda.synchronize()
        graph.replay()
        with torch.cuda.stream(side):
            o2, l2 = step(b, table.clone(), lens.clone(), torch.empty_like(q))
        torch.cuda.synchronize()
        assert torch.equal(out, o2) and torch.equal(lse, l2)
        assert torch.equal(a.dev.k_codes, b.dev.k_codes) and torch.equal(a.dev.v_scales, b.dev.v_scales)


def test_binding_refusals():
    box = Box(4, 2, 64, 16, "int8", fill="values")
    s = gseqs([[0, 1]], [20], [0, 20])
    x = torch.zeros(20, 2, 64, device=DEV)
    for bad in (x[:, :1], x.double(), x.cpu(), x.transpose(1, 2), x[0]):
        with pytest.raises(slq.SlqError):
            slq.slq_kv_write(box.dev, s, bad, bad)
    with pytest.raises(slq.SlqError):
        slq.slq_kv_attention(box.dev, s, x)                  # fp32 queries
    with pytest.raises(slq.SlqError):
        slq.slq_kv_attention(box.dev, s, x[:, :, :64].bfloat16()[:, :1])   # one query head for two kv heads
    with pytest.raises(slq.SlqError):
        slq.slq_kv_read(box.dev, s, 20, torch.float64)
    with pytest.raises(slq.SlqError):
        slq.slq_kv_read(box.dev, s, 20, torch.float32, out=(x, x))
    with pytest.raises(slq.SlqError):
        slq.slq_kv_write(box.dev, s, x[:, :, 1:], x[:, :, 1:])
    with pytest.raises(slq.SlqError):
        slq.KvSeqs(s.table.long(), s.lens, s.cu)
    with pytest.raises(slq.SlqError):
        slq.KvSeqs(s.table, s.lens, s.cu[:1])
    torch.cuda.synchronize()
    box.same("nothing was written")
