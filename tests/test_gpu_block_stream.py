"""Streams given as handles: a call's workspace is memory of the stream that the call runs on, the default stream's
handle 0 too."""
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def test_workspace_for_the_default_streams_handle():
    torch.cuda.empty_cache()
    n, device = 24 << 20, torch.cuda.current_device()
    held = torch.empty(n, dtype=torch.uint8, device="cuda")  # memory of the default stream, let go of
    at = held.data_ptr()
    del held
    for stream in (None, 0, torch.cuda.default_stream(), torch.cuda.default_stream().cuda_stream):
        assert pkv._scratch(None, n, device, stream)[0] == at
    other = torch.cuda.Stream()
    with torch.cuda.stream(other):  # another current stream does not matter
        assert pkv._scratch(None, n, device, 0)[0] == at
        assert pkv._scratch(None, n, device, None)[0] != at


def test_a_call_on_the_default_streams_handle():
    b = ref.Batch([700, 31], [1, 1], 2, 128, 16, seed=51, g=4)
    t = [torch.from_numpy(x).cuda() for x in (b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx)]
    q = b.q.cuda()
    outs = [torch.full_like(q, float("nan")) for _ in range(3)]
    for out, stream in zip(outs, (None, 0, torch.cuda.default_stream())):
        pkv.paged_attn_decode_fp8_block(q, *t, b.scale, 2, out, 700, stream=stream)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    want = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx, b.scale, 16,
                      v_scales=b.vs)
    ref.assert_attention(outs[0], want, 2.0 ** -11)
    no_device_error()


@pytest.mark.parametrize("call", ["decode", "decode_fp8", "prefill"])
def test_every_attention_call_takes_its_workspace_from_its_stream(call, monkeypatch):
    taken, scratch, stream = [], pkv._scratch, torch.cuda.Stream()

    def spy(workspace, nbytes, index, on):
        taken.append(on)
        return scratch(workspace, nbytes, index, on)

    monkeypatch.setattr(pkv, "_scratch", spy)
    b = ref.Batch([64], [1], 2, 128, 16, seed=52, g=2)
    q, tables, ctx = b.q.cuda(), torch.from_numpy(b.tables).cuda(), torch.from_numpy(b.ctx).cuda()
    k, v = (x.cuda() for x in b.bf16_pool())
    codes, scale = torch.from_numpy(b.kc).cuda(), torch.ones(2, device="cuda")
    start, out = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.empty_like(q)
    torch.cuda.synchronize()
    for on in (None, stream):
        if call == "decode":
            pkv.paged_attn_decode(q, k, v, tables, ctx, b.scale, 2, out, 64, stream=on)
        elif call == "decode_fp8":
            pkv.paged_attn_decode_fp8(q, codes, codes, scale, scale, tables, ctx, b.scale, 2, out, 64, stream=on)
        else:
            pkv.paged_attn_prefill(q, k, v, tables, ctx, start, b.scale, 2, out, 1, 64, stream=on)
        torch.cuda.synchronize()
    assert taken == [None, stream]
    no_device_error()
