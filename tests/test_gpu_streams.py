"""Calls on a stream given by argument, while the current stream still has work to do on
memory that was freed there: the outputs and the workspace that a call allocates are not
that memory."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    o.device_status(clear=True)
    torch.cuda._sleep(1000)  # loads the kernels that the tests keep the stream busy with
    torch.zeros(8, dtype=torch.uint8, device="cuda").fill_(255)
    torch.cuda.synchronize()
    return o


def i32(a):
    return torch.tensor(np.asarray(a, dtype=np.int32)).cuda()


def make(ops, name):
    """(call(stream) -> outputs, byte sizes of what it allocates)."""
    gen = torch.Generator(device="cuda").manual_seed(5)

    def rand(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    if name == "quantize_row_q8":
        x = rand(64, 2048)
        return lambda st: ops.quantize_row_q8(x, stream=st), [64 * 2048, 256, 256]
    if name == "linear_q4":
        xq, sx, _ = ops.quantize_row_q8(rand(300, 512))
        w, sw = ops.quantize_matrix_q4(rand(256, 512))
        need = ops.workspace_bytes(ops.OP_LINEAR_Q4, 300, 256, 512)
        assert need > 0
        return lambda st: [ops.linear_q4(xq, sx, w, sw, K=512, stream=st)], [300 * 256 * 4, need]
    if name == "quantize_mxfp4":
        x = rand(300, 2048)
        return lambda st: ops.quantize_mxfp4(x, stream=st), [300 * 1024, 300 * 64]
    if name == "dequantize_mxfp4":
        c, s = ops.quantize_mxfp4(rand(300, 2048))
        return lambda st: [ops.dequantize_mxfp4(c, s, 2048, stream=st)], [300 * 2048 * 4]
    if name == "linear_mxfp4":
        x, (w, sw) = rand(5, 512).bfloat16(), ops.quantize_mxfp4(rand(4096, 512))
        return lambda st: [ops.linear_mxfp4(x, w, sw, stream=st)], [5 * 4096 * 4]
    if name == "linear_mxfp4_a4":
        (x, sx), (w, sw) = ops.quantize_mxfp4(rand(200, 512)), ops.quantize_mxfp4(rand(4096, 512))
        return lambda st: [ops.linear_mxfp4_a4(x, sx, w, sw, 512, stream=st)], [200 * 4096 * 4]
    if name == "draft_plan":
        ctx, new, table, free = i32([40] * 64), i32([64] * 64), i32(np.arange(64 * 8).reshape(64, 8)), i32(np.arange(900))
        return (lambda st: ops.draft_plan(ctx, new, None, free, table, 16, max_tokens=4096, stream=st),
                [65 * 4, 4096 * 8, 4096 * 4, 4096 * 16, 4])
    T, Hq, Hkv, D, page = 200, 8, 2, 128, 16
    k, v = rand(40, page, Hkv, D).bfloat16(), rand(40, page, Hkv, D).bfloat16()
    if name == "qk_norm_rope":
        qkv, pos = rand(T, (Hq + 2 * Hkv) * D), torch.arange(T, device="cuda", dtype=torch.int32)
        cs, slots = rand(T, D), torch.arange(T, device="cuda")
        return lambda st: [ops.qk_norm_rope(qkv, Hq, None, None, pos, cs, slots, k, v, stream=st)], [T * Hq * D * 2]
    assert name == "tree_attention"
    q, table = rand(60, Hq, D).bfloat16(), i32(np.arange(40).reshape(2, 20))
    ctx, new = [250, 270], [30, 30]
    cu, _, _, mask, _ = ops.draft_plan(i32(ctx), i32(new), None, i32([]), table, page, max_tokens=60)
    c = i32(ctx)
    need = ops.tree_attention_workspace_bytes(2, Hq, Hkv, D, 300, 30)
    assert need > 0
    return (lambda st: [ops.tree_attention(q, k, v, table, c, cu, mask, 0.09, 300, 30, stream=st)],
            [60 * Hq * D * 2, need])


@pytest.mark.parametrize("name", ["quantize_row_q8", "linear_q4", "quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4",
                                  "linear_mxfp4_a4", "draft_plan", "qk_norm_rope", "tree_attention"])
def test_allocations_belong_to_the_calls_stream(ops, name):
    call, sizes = make(ops, name)
    want = [t.clone() for t in call(None)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    junk = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda._sleep(200_000_000)  # about 0.1 s
    for j in junk:
        j.fill_(255)
    del j, junk
    got = call(st)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert ops.device_status() == 0
