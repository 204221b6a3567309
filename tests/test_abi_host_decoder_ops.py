"""Refusals of the decoder-step operators (norm, cache, attention, sampling) through the C ABI:
each call fails validation on the host, before any HIP call, so no GPU is needed."""
import pytest
import torch

import int4_weight_only_gemm_amd as w4

F32, BF16 = 0, 1
P = [0x10000 * (i + 1) for i in range(16)]  # never dereferenced
OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3


def call(fn, base, **change):
    args = dict(base)
    args.update(change)
    return getattr(w4.lib(), fn)(*args.values())


NORM = dict(x=P[0], x_type=F32, x_stride=256, res=P[1], res_type=BF16, res_stride=256, w=P[2], w_type=BF16, eps=1e-6,
            y=P[3], bits=16, scales=None, res_out=P[4], M=4, H=256, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), NULL), (dict(w=None), NULL), (dict(y=None), NULL), (dict(res_out=None), NULL),
    (dict(bits=8), NULL), (dict(bits=4), NULL),
    (dict(x_type=2), SHAPE), (dict(w_type=-1), SHAPE), (dict(res_type=7), SHAPE), (dict(bits=5), SHAPE),
    (dict(M=-1), SHAPE), (dict(M=1 << 31), SHAPE), (dict(M=1 << 22), SHAPE), (dict(H=0), SHAPE), (dict(H=32769, x_stride=40000, res_stride=40000), SHAPE),
    (dict(H=200, bits=8, scales=P[5]), SHAPE), (dict(H=200, bits=4, scales=P[5]), SHAPE),
    (dict(x_stride=255), SHAPE), (dict(res_stride=255), SHAPE), (dict(x_stride=1 << 41), SHAPE),
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE),
    (dict(x=P[0] + 2), ALIGN), (dict(w=P[2] + 1), ALIGN), (dict(y=P[3] + 1), ALIGN), (dict(res=P[1] + 1), ALIGN),
    (dict(res_out=P[4] + 1), ALIGN), (dict(y=P[3] + 4, bits=8, scales=P[5]), ALIGN),
    (dict(y=P[3] + 2, bits=4, scales=P[5]), ALIGN), (dict(bits=8, scales=P[5] + 2), ALIGN),
    (dict(M=0, x=None, w=None, y=None, res_out=None), OK)])
def test_rms_norm_refusals(change, status):
    assert call("w4_rms_norm", NORM, **change) == status
    if status:
        assert w4.lib().w4_last_error()


DEQ = dict(codes=P[0], scales=P[1], out=P[2], M=3, K=256, bits=8, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(out=None), NULL), (dict(bits=16), SHAPE),
    (dict(M=-1), SHAPE), (dict(K=64), SHAPE), (dict(K=200), SHAPE), (dict(codes=P[0] + 4), ALIGN),
    (dict(codes=P[0] + 2, bits=4), ALIGN), (dict(out=P[2] + 8), ALIGN), (dict(scales=P[1] + 2), ALIGN), (dict(M=0), OK)])
def test_act_dequantize_refusals(change, status):
    assert call("w4_act_dequantize", DEQ, **change) == status


WRITE = dict(k=P[0], v=P[1], src_type=F32, kt=512, kh=128, vt=512, vh=128, slots=P[2], kc=P[3], vc=P[4], ks=P[5],
             vs=P[6], bits=8, T=5, heads=4, D=128, pages=10, page_size=64, stream=None)
READ = dict(slots=P[2], kc=P[3], vc=P[4], ks=P[5], vs=P[6], bits=8, k=P[0], v=P[1], out_type=F32, T=5, heads=4, D=128,
            pages=10, page_size=64, stream=None)
CACHE = [
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(slots=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL),
    (dict(ks=None), NULL), (dict(vs=None), NULL), (dict(bits=4), SHAPE), (dict(T=-1), SHAPE), (dict(T=1 << 27), SHAPE), (dict(heads=0), SHAPE),
    (dict(heads=65536), SHAPE), (dict(D=96), SHAPE), (dict(D=256), SHAPE), (dict(pages=0), SHAPE),
    (dict(page_size=0), SHAPE), (dict(page_size=65537), SHAPE), (dict(pages=1 << 40), SHAPE),
    (dict(slots=P[2] + 4), ALIGN), (dict(kc=P[3] + 8), ALIGN), (dict(vc=P[4] + 8), ALIGN), (dict(ks=P[5] + 2), ALIGN),
    (dict(vs=P[6] + 2), ALIGN), (dict(T=0), OK)]


@pytest.mark.parametrize("change,status", CACHE + [
    (dict(src_type=3), SHAPE), (dict(kt=-1), SHAPE), (dict(vh=1 << 33), SHAPE), (dict(k=P[0] + 2), ALIGN),
    (dict(v=P[1] + 1, src_type=BF16), ALIGN)])
def test_kv_write_refusals(change, status):
    assert call("w4_kv_write", WRITE, **change) == status


@pytest.mark.parametrize("change,status", CACHE + [(dict(out_type=3), SHAPE), (dict(k=P[0] + 8), ALIGN),
                                                   (dict(v=P[1] + 4), ALIGN)])
def test_kv_read_refusals(change, status):
    assert call("w4_kv_read", READ, **change) == status


ATTN = dict(q=P[0], qt=3584, qh=128, kc=P[1], vc=P[2], ks=P[3], vs=P[4], bits=8, table=P[5], ts=16, width=16,
            q_start=P[6], kv_len=P[7], out=P[8], scale=0.1, T=10, B=2, hq=28, hkv=4, D=128, pages=40, page_size=64,
            max_q=5, max_kv=1000, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(q=None), NULL), (dict(kc=None), NULL), (dict(vc=None), NULL), (dict(ks=None), NULL), (dict(vs=None), NULL),
    (dict(table=None), NULL), (dict(q_start=None), NULL), (dict(kv_len=None), NULL), (dict(out=None), NULL),
    (dict(bits=4), SHAPE), (dict(D=96), SHAPE), (dict(T=-1), SHAPE), (dict(B=-1), SHAPE), (dict(B=65536), SHAPE),
    (dict(hkv=0), SHAPE), (dict(hq=27), SHAPE), (dict(hq=2), SHAPE), (dict(T=1 << 30), SHAPE), (dict(pages=0), SHAPE),
    (dict(page_size=8), SHAPE), (dict(page_size=24), SHAPE), (dict(page_size=8192), SHAPE), (dict(pages=1 << 38), SHAPE),
    (dict(width=-1), SHAPE), (dict(ts=15), SHAPE), (dict(max_q=11), SHAPE), (dict(max_q=-1), SHAPE),
    (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(max_kv=-1), SHAPE), (dict(qt=-1), SHAPE), (dict(qh=1 << 33), SHAPE),
    (dict(q=P[0] + 1), ALIGN), (dict(kc=P[1] + 8), ALIGN), (dict(vc=P[2] + 8), ALIGN), (dict(ks=P[3] + 4), ALIGN),
    (dict(vs=P[4] + 4), ALIGN), (dict(table=P[5] + 2), ALIGN), (dict(q_start=P[6] + 2), ALIGN),
    (dict(kv_len=P[7] + 1), ALIGN), (dict(out=P[8] + 8), ALIGN),
    (dict(T=0, max_q=0, q=None, out=None), OK), (dict(B=0), OK), (dict(max_q=0), OK)])
def test_paged_attention_refusals(change, status):
    assert call("w4_paged_attention", ATTN, **change) == status


SAMPLE = dict(logits=P[0], kind=F32, stride=32000, u=P[1], t=P[2], k=P[3], p=P[4], mp=P[5], token=P[6], prob=P[7], B=4,
              V=32000, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), NULL), (dict(u=None), NULL), (dict(token=None), NULL), (dict(kind=2), SHAPE),
    (dict(B=-1), SHAPE), (dict(B=65536), SHAPE), (dict(V=0), SHAPE), (dict(V=(1 << 19) + 1, stride=1 << 20), SHAPE),
    (dict(stride=31999), SHAPE), (dict(stride=1 << 33), SHAPE), (dict(logits=P[0] + 2), ALIGN),
    (dict(logits=P[0] + 1, kind=BF16), ALIGN), (dict(u=P[1] + 2), ALIGN), (dict(t=P[2] + 2), ALIGN),
    (dict(k=P[3] + 2), ALIGN), (dict(p=P[4] + 1), ALIGN), (dict(mp=P[5] + 2), ALIGN), (dict(token=P[6] + 2), ALIGN),
    (dict(prob=P[7] + 2), ALIGN), (dict(B=0, logits=None, u=None, token=None), OK)])
def test_sample_refusals(change, status):
    assert call("w4_sample", SAMPLE, **change) == status


def test_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(2, 128)
    with pytest.raises(ValueError):
        w4.rms_norm(x, torch.ones(128))
    with pytest.raises(TypeError):
        w4.rms_norm([1.0], torch.ones(128))
    with pytest.raises(ValueError):
        w4.sample(x, torch.zeros(2))
    with pytest.raises(ValueError):
        w4.dequantize_activations(torch.zeros(2, 128, dtype=torch.int8), torch.zeros(2, 1), bits=8)
    with pytest.raises(ValueError):
        w4.dequantize_activations(torch.zeros(2, 128, dtype=torch.int8), torch.zeros(2, 1), bits=3)
    c = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        w4.kv_write(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int64), c, c)
    with pytest.raises(TypeError):
        w4.kv_read(torch.zeros(1, dtype=torch.int64), c.float(), c.float())
    with pytest.raises(ValueError):
        w4.paged_attention(torch.zeros(1, 1, 64, dtype=torch.bfloat16), c, c, torch.zeros(1, 1, dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), 1, 1)


def test_new_symbols_are_declared():
    assert set(w4.header_functions()) >= {"w4_rms_norm", "w4_act_dequantize", "w4_kv_write", "w4_kv_read",
                                          "w4_paged_attention", "w4_sample"}
