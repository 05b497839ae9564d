"""The serving operators as they are used: a prompt and then single tokens through
one small attention layer -- weight-only products for q, k and v, the cache write,
attention, the output product, and sampling -- with every stage checked against
its oracle on the stage's own inputs, eagerly and as a replayed graph."""
import numpy as np
import pytest
import torch

import slq_synth as S
import weight_only_mixed_amd as slq
from oracle import serve as orc
from tests.gpu_util import DEV, gpu, say
from tests.test_gpu_kv import FMT, Box, check_attention, gseqs

pytestmark = pytest.mark.gpu
HID, HEADS, GROUP, DIM, VOCAB, PAGE = 512, 2, 4, 64, 1280, 16


class Layer:
    def __init__(self, seed=0):
        hq = HEADS * GROUP
        self.w = {n: slq.slq_quantize_pack(gpu(S.skewed_weights(o, i, seed + j) * np.float32(2.0)), b)
                  for j, (n, o, i, b) in enumerate((("q", hq * DIM, HID, 5), ("k", HEADS * DIM, HID, 8),
                                                    ("v", HEADS * DIM, HID, 7), ("o", HID, hq * DIM, 6),
                                                    ("head", VOCAB, HID, 4)))}
        g = np.random.default_rng(seed)
        self.embed = gpu(g.standard_normal((VOCAB, HID)).astype(np.float32)).bfloat16()

    def mul(self, n, x, ws):
        y = torch.empty((x.shape[0], self.w[n].n), dtype=torch.float32, device=DEV)
        return slq.slq_dequant_gemm(x, self.w[n], y, ws)

    def step(self, cache, seqs, tokens, last, u, top_p, max_q, max_len, ws):
        x = self.embed[tokens]
        q = self.mul("q", x, ws).bfloat16().view(-1, HEADS * GROUP, DIM)
        k, v = self.mul("k", x, ws).view(-1, HEADS, DIM), self.mul("v", x, ws).view(-1, HEADS, DIM)
        slq.slq_kv_write(cache, seqs, k, v, max_new=max_q)
        a = slq.slq_kv_attention(cache, seqs, q, max_q=max_q, max_len=max_len)
        h = x[last] + self.mul("o", a.view(-1, HEADS * GROUP * DIM)[last], ws).bfloat16()
        logits = self.mul("head", h, ws)
        t, lp = slq.slq_sample(logits, u, top_p=top_p)
        return dict(q=q, k=k, v=v, a=a, logits=logits, tokens=t, logprobs=lp)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_prompt_then_tokens(fmt):
    g = np.random.default_rng(7)
    layer, B = Layer(), 3
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    box = Box(24, HEADS, DIM, PAGE, fmt)
    table = g.permutation(24)[:B * 6].reshape(B, 6)
    lens = np.array([30, 17, 1])
    tokens = torch.from_numpy(g.integers(0, VOCAB, lens.sum())).to(DEV)
    cu = np.concatenate([[0], np.cumsum(lens)])
    for n in range(6):
        top_p = np.full(B, 0.8, np.float32)
        u = g.random(B).astype(np.float32)
        s = gseqs(table, lens, cu)
        last = torch.from_numpy(cu[1:] - 1).to(DEV)
        r = layer.step(box.dev, s, tokens, last, gpu(u), gpu(top_p), int((cu[1:] - cu[:-1]).max()), 96, ws)
        for i, x in enumerate((r["k"], r["v"])):
            orc.kv_write(box.codes[i], box.scales[i], table, lens, cu, x.cpu().numpy(), box.fmt)
        box.same(f"step {n}")
        o, _ = check_attention(box, table, lens, cu, r["q"], max_q=int((cu[1:] - cu[:-1]).max()), max_len=96, what=f"step {n}")
        assert torch.equal(o, r["a"])
        t, lp, kept = orc.sample(r["logits"].cpu().numpy(), u, top_p=top_p)
        assert np.array_equal(t, r["tokens"].cpu().numpy())
        say(f"step {n}: tokens {t.tolist()} of {kept.tolist()} kept")
        tokens, cu, lens = r["tokens"].long(), np.arange(B + 1), lens + 1


def test_captured_step():
    """Decode steps replayed from one graph, lengths and tokens moving on the device,
    against the same steps run eagerly on a second cache."""
    g = np.random.default_rng(9)
    layer, B = Layer(5), 4
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    boxes = [Box(24, HEADS, DIM, PAGE, "int8", seed=1, fill="values") for _ in range(2)]
    table = gpu(g.permutation(24).reshape(B, 6).astype(np.int32))
    cu, last = torch.arange(B + 1, dtype=torch.int32, device=DEV), torch.arange(B, device=DEV)
    top_p = torch.full((B,), 0.9, device=DEV)

    class State:
        def __init__(self):
            self.lens = torch.tensor([20, 3, 41, 16], dtype=torch.int32, device=DEV)
            self.tokens = torch.tensor([1, 2, 3, 4], device=DEV)
            self.u = torch.zeros(B, device=DEV)

    def advance(box, st):
        r = layer.step(box.dev, slq.KvSeqs(table, st.lens, cu), st.tokens, last, st.u, top_p, 1, 96, ws)
        st.tokens.copy_(r["tokens"])
        st.lens.add_(1)
        return r

    warm = torch.cuda.Stream()
    with torch.cuda.stream(warm):
        advance(Box(24, HEADS, DIM, PAGE, "int8", seed=1, fill="values"), State())
    warm.synchronize()
    a, b = State(), State()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ra = advance(boxes[0], a)
    torch.cuda.synchronize()
    for n in range(8):
        u = gpu(g.random(B).astype(np.float32))
        a.u.copy_(u), b.u.copy_(u)
        graph.replay()
        torch.cuda.synchronize()
        rb = advance(boxes[1], b)
        torch.cuda.synchronize()
        for name in ("a", "logits", "tokens", "logprobs"):
            assert torch.equal(ra[name], rb[name]), (n, name)
        assert torch.equal(boxes[0].dev.k_codes, boxes[1].dev.k_codes)
        assert torch.equal(boxes[0].dev.v_scales, boxes[1].dev.v_scales) and torch.equal(a.lens, b.lens)
