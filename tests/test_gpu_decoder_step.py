"""The example's decoder step, its operators together, against a plain evaluation in 64 bits that
takes over at each rounding the step makes on purpose."""
import importlib.util
import os

import pytest
import torch

import int4_weight_only_gemm_amd as w4
from conftest import ROOT
from gpu_helpers import log

pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("decoder_step", os.path.join(ROOT, "examples", "decoder_step.py"))
    m = importlib.util.module_from_spec(spec)
    import sys
    sys.modules["decoder_step"] = m
    spec.loader.exec_module(m)
    return m


def weights(lin):
    """The 64-bit [K, N] values of a 4-bit linear layer."""
    q = torch.stack([(lin.q >> (4 * j)) & 15 for j in range(8)], 1).reshape(-1, lin.q.shape[1]).double()
    return (q - lin.z.double().repeat_interleave(128, 0)) * lin.s.double().repeat_interleave(128, 0)


@pytest.mark.parametrize("batch,tokens,context", [(1, 1, 40), (2, 5, 100), (3, 24, 130)])
def test_step_against_plain(batch, tokens, context):
    ex = example()
    s = ex.Shape(hidden=512, heads=8, kv_heads=2, head_dim=64, ffn=768, vocab=1000, layers=2, page=16)
    d = ex.Decoder(s, batch * -(-context // s.page), seed=3)
    b = ex.batch_of(d, batch, tokens, context)
    log(f"decoder step batch={batch} tokens={tokens} context={context}")
    token, prob, logits = d.step(**b)

    T, bf = batch * tokens, torch.bfloat16
    norm = lambda r, w: r / (r.square().mean(1, keepdim=True) + s.eps).sqrt() * w.double()  # noqa: E731
    x, add = b["x"].double(), 0
    for layer in d.layers:
        x = x + add
        qkv = (norm(x, layer["norm1"]) @ weights(layer["qkv"])).view(T, -1, s.head_dim)
        c, si = d.cos[b["positions"]].double()[:, None], d.sin[b["positions"]].double()[:, None]
        h1, h2 = qkv[:, :s.heads + s.kv_heads].chunk(2, -1)
        q = torch.cat([h1 * c - h2 * si, h2 * c + h1 * si], -1)[:, :s.heads]
        o = torch.zeros(T, s.heads, s.head_dim, dtype=torch.float64, device="cuda")
        for i in range(batch):
            at = torch.arange(context, device="cuda")
            slots = b["block_table"][i, at // s.page].long() * s.page + at % s.page
            k, v = (y.double() for y in w4.kv_read(slots, layer["k"], layer["v"], layer["ks"], layer["vs"], dtype=torch.float32))
            for h in range(s.heads):
                rows = slice(i * tokens, (i + 1) * tokens)
                score = q[rows, h] @ k[:, h // 4].t().contiguous() / s.head_dim ** 0.5
                hidden = torch.arange(context, device="cuda")[None] > torch.arange(context - tokens, context, device="cuda")[:, None]
                o[rows, h] = torch.softmax(score.masked_fill(hidden, float("-inf")), 1) @ v[:, h // 4].contiguous()
        x = x + o.view(T, -1) @ weights(layer["o"])
        gate, up = (norm(x, layer["norm2"]) @ weights(layer["gate_up"])).chunk(2, -1)
        add = (torch.nn.functional.silu(gate) * up) @ weights(layer["down"])
    want = norm(x + add, d.norm) @ weights(d.head)
    # Roundings to bfloat16 along the way (7 a layer of 2^-8 at most, half a step each, independent: of a
    # result's size about 2^-8 * sqrt(2 * 7) / sqrt(3) at one standard deviation), through layers that
    # may double them: 2 * 2^-8 * sqrt(14 / 3) of the logits' norm.
    off = (logits.double() - want).norm() / want.norm()
    assert off <= 2 * 2.0 ** -8 * (14 / 3) ** 0.5, float(off)
    # the draw is the sampling operator's on these logits
    t2, p2 = w4.sample(logits, b["u"], temperature=b["temperature"], top_k=b["top_k"], top_p=b["top_p"])
    assert torch.equal(token, t2) and torch.equal(prob, p2) and ((prob > 0) & (prob <= 1)).all()
    assert d.step(**b)[0].dtype == torch.int32 and bf == b["x"].dtype
