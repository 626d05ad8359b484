"""GPU tests of MXFP4 matrices cut out of stacked tensors: their scale bytes
start at any byte, as N K / 32 is any number."""
import pytest
import torch

pytestmark = pytest.mark.gpu
mx = pytest.importorskip("mxfp4_moe_expert_amd")
DEV = "cuda"
E_, N, K = 3, 101, 96  # 303 scale bytes a matrix


def _stack():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    w = torch.randn(E_, N, K, generator=g, device=DEV)
    return mx.quantize_mxfp4(w) + (g,)


def test_dequantize_a_slice():
    c, s, _ = _stack()
    whole = mx.dequantize_mxfp4(c, s)
    for e in range(E_):
        assert torch.equal(mx.dequantize_mxfp4(c[e], s[e]), whole[e])
    assert torch.equal(mx.dequantize_mxfp4(c[1, 1:], s[1, 1:], dtype=torch.float32), whole[1, 1:].float())


@pytest.mark.parametrize("act", ["bf16", "mxfp4"])
@pytest.mark.parametrize("T", [1, 20, 70, 2100])
def test_products_with_a_slice(T, act):
    c, s, g = _stack()
    x = torch.randn(T, K, generator=g, device=DEV).to(torch.bfloat16)
    dy = torch.randn(T, N, generator=g, device=DEV).to(torch.bfloat16)
    assert s[1].data_ptr() % 16 and s[2].data_ptr() % 4
    for e in range(E_):
        apart = s[e].clone()
        assert torch.equal(mx.linear_mxfp4(x, c[e], s[e], act=act), mx.linear_mxfp4(x, c[e], apart, act=act))
        assert torch.equal(mx.linear_mxfp4_dx(dy, c[e], s[e]), mx.linear_mxfp4_dx(dy, c[e], apart))


def test_a_slice_in_a_graph_and_on_a_stream():
    """The aligned copy is the call's own: it is made in the call's stream and, captured, anew in every replay."""
    c, s, g = _stack()
    s = s.clone()
    x = torch.randn(300, K, generator=g, device=DEV).to(torch.bfloat16)
    graph = torch.cuda.CUDAGraph()
    mx.linear_mxfp4(x, c[1], s[1])
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = mx.linear_mxfp4(x, c[1], s[1]), mx.linear_mxfp4(x, c[1], s[1], act="mxfp4")
    for rep in range(3):
        s.add_(rep)  # other weights
        for o in out:
            o.zero_()
        graph.replay()
        want = mx.linear_mxfp4(x, c[1], s[1].clone()), mx.linear_mxfp4(x, c[1], s[1].clone(), act="mxfp4")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), rep
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = [mx.linear_mxfp4(x, c[1], s[1]) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) for a in got)


def test_refusals_name_the_argument():
    """What the library has to have at 16-byte borders (workspaces: 256) and is not copied."""
    c, s, g = _stack()
    flat = torch.zeros(1 + 64 * K, dtype=torch.bfloat16, device=DEV)
    x = flat[1:].view(64, K)
    w13, w2 = flat[:64 * K].view(64, K), flat[:32 * K].view(K, 32)
    good = flat[:64 * K].view(64, K)
    dy = torch.zeros(1 + 64 * N, dtype=torch.bfloat16, device=DEV)[1:].view(64, N)
    calls = {
        "x": [lambda: mx.linear_mxfp4(x, c[0], s[0]), lambda: mx.quantize_mxfp4(x), lambda: mx.gated_ffn(x, w13, w2)],
        "dy": [lambda: mx.linear_mxfp4_dx(dy, c[0], s[0])],
        "w13": [lambda: mx.gated_ffn(good, x, w2)],
        "scales": [lambda: mx.quantize_mxfp4(good, out=(torch.empty(64, K // 2, dtype=torch.uint8, device=DEV),
                                                        torch.empty(1 + 64 * K // 32, dtype=torch.uint8,
                                                                    device=DEV)[1:].view(64, K // 32)))],
        "ws": [lambda: mx.gated_ffn(good, w13, w2, ws=torch.empty(1 << 20, dtype=torch.uint8, device=DEV)[16:])],
    }
    for name, fs in calls.items():
        for f in fs:
            with pytest.raises(mx.MoEError, match=rf"\b{name}: .*aligned") as e:
                f()
            assert e.value.status == mx.MOE_EINVAL


def test_what_a_call_does_not_use_is_not_refused():
    """A workspace at any address where none is used, and empty batches beside misaligned tensors."""
    c, s, g = _stack()
    x = torch.randn(5, K, generator=g, device=DEV).to(torch.bfloat16)
    odd = torch.empty(4096, dtype=torch.uint8, device=DEV)[1:]
    for n in (1, 5):
        assert torch.equal(mx.linear_mxfp4(x[:n], c[0], s[0], ws=odd), mx.linear_mxfp4(x[:n], c[0], s[0]))
    assert mx.linear_mxfp4(x[:0], c[1], s[1], ws=odd).shape == (0, N)
    w = torch.zeros(1 + 64 * K, dtype=torch.bfloat16, device=DEV)[1:]
    assert mx.gated_ffn(x[:0], w.view(64, K), w[:32 * K].view(K, 32)).shape == (0, K)
