"""The latent-attention layer object's state: refused calls, its own copies of
the weights, kept drafts, streams, and the choice of form where the expanded
one cannot run."""
import numpy as np
import pytest

from tests.test_latent_layer_gpu import DC, DN, DR, DV, H, close, definition, layer, tokens  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


def causal(n):
    return np.tril(np.ones((n, n), bool))


def state(L):
    return dict(L._len), {s: list(p) for s, p in L._pages.items()}, list(L._free)


def test_calls_refused_after_the_pages_are_taken_leave_the_sequences(layer):
    """What the entry points refuse (types, shapes, strides, limits) comes back as it was, and the next call is right."""
    a, b = layer.new_sequence(), layer.new_sequence()
    q, kv = tokens(40, 120)
    layer.forward([a], [30], q[:30], kv[:30])
    before = state(layer)

    def refused(error, *args, **kw):
        with pytest.raises(error):
            layer.forward(*args, **kw)
        assert state(layer) == before

    for n in (2, 90):  # absorbed and expanded
        x, y = q[30:30 + n], kv[30:30 + n]
        refused(TypeError, [a], [n], x.float(), y)
        refused(TypeError, [a], [n], x, y.float())
        refused(TypeError, [a, b], [n - 1, 1], x.cpu(), y)
        refused(ValueError, [a], [n], x[:, :H - 1], y)
        refused(ValueError, [a], [n], x[..., :DN + DR - 8], y)
        refused(ValueError, [a], [n], x.transpose(1, 2).contiguous().transpose(1, 2), y)
        refused(ValueError, [a], [n], x, y[:, :DC])
        wide = torch.zeros((n, DC + DR + 4), dtype=torch.float16, device="cuda")
        refused(RuntimeError, [a], [n], x, wide[:, :DC + DR])  # rows no multiple of 8 apart
    many = [layer.new_sequence() for _ in range(1024)]
    before = state(layer)
    refused(RuntimeError, [a] + many, [2] + [0] * 1024, q[30:32], kv[30:32])  # 1025 sequences
    for s in many:
        layer.drop_sequence(s)
    out = layer.forward([a], [2], q[30:32], kv[30:32])
    layer.ctx.check()
    close(out, definition(layer, q[:32], kv[:32], np.arange(32), causal(32))[30:])
    layer.drop_sequence(a)
    layer.drop_sequence(b)


@pytest.mark.parametrize("word", [1 << 64, (1 << 64) + 1, -1])
def test_words_beyond_64_bits_are_refused(layer, word):
    s = layer.new_sequence()
    q, kv = tokens(41, 3)
    layer.forward([s], [1], q[:1], kv[:1])
    before = state(layer)
    with pytest.raises(ValueError):
        layer.forward([s], [2], q[1:], kv[1:], tree=[1, word], depth=[0, 1])
    assert state(layer) == before
    layer.drop_sequence(s)


def test_the_layer_has_its_own_weights():
    """Tensors that already have the layer's type and place may be overwritten after set_weights, in both forms."""
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.latent import LatentAttention
    ctx = moe.MoeCtx(0)
    L = LatentAttention(ctx, H, DC, DR, DN, DV, n_pages=40, page_size=16, max_positions=400, dtype=torch.float16)
    g = torch.Generator().manual_seed(2)
    w = (torch.randn((H, DN + DV, DC), generator=g) * DC ** -0.5).half().cuda()
    norm = (1 + 0.1 * torch.randn((DC,), generator=g)).cuda()
    w_then, norm_then = w.clone(), norm.clone()
    L.set_weights(w, norm)
    w.zero_()
    norm.zero_()
    assert torch.equal(L.w_kv, w_then) and torch.equal(L.norm_w, norm_then)
    q, kv = tokens(42, 102)
    s = L.new_sequence()
    assert L.expands([100], [100]) and not L.expands([2], [102])
    out = torch.cat([L.forward([s], [100], q[:100], kv[:100]), L.forward([s], [2], q[100:], kv[100:])])
    ctx.check()
    close(out, definition(L, q, kv, np.arange(102), causal(102)))

    # shapes are checked, and a refused call leaves the weights
    for bad in ((w_then[:, :DN + DV - 1], None), (w_then[:H - 1], norm_then), (w_then.flatten(0, 1), None),
                (w_then, norm_then[:-1]), (w_then, norm_then[None])):
        with pytest.raises(ValueError):
            L.set_weights(*bad)
    assert torch.equal(L.w_kv, w_then) and torch.equal(L.norm_w, norm_then)
    assert torch.equal(L.w_kt, w_then[:, :DN].transpose(1, 2))
    ctx.close()


def test_weights_of_a_trained_module_are_values_only(layer):
    """Parameters are taken by value: nothing of them is held by the layer's copies."""
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.latent import LatentAttention
    ctx = moe.MoeCtx(0)
    L = LatentAttention(ctx, H, DC, DR, DN, DV, n_pages=4, page_size=16, max_positions=64, dtype=torch.float16)
    L.set_weights(torch.nn.Parameter(layer.w_kv.float()), torch.nn.Parameter(layer.norm_w.clone()))
    assert torch.equal(L.w_kv, layer.w_kv) and torch.equal(L.norm_w, layer.norm_w)
    assert not any(t.requires_grad for t in (L.w_kv, L.w_kt, L.norm_w))
    ctx.close()


@pytest.mark.parametrize("n_own", [31, 47, 1000, -1])
def test_keep_takes_no_more_tokens_than_there_are(layer, n_own):
    s = layer.new_sequence()
    q, kv = tokens(43, 31)
    layer.forward([s], [30], q[:30], kv[:30])
    before, rows = state(layer), layer.cache.clone()
    for nodes in ([], [0], [0, 20]):
        with pytest.raises(ValueError):
            layer.keep(s, n_own, nodes)
        assert state(layer) == before
    assert torch.equal(layer.cache, rows)
    out = layer.forward([s], [1], q[30:], kv[30:])
    layer.ctx.check()
    close(out, definition(layer, q, kv, np.arange(31), causal(31))[30:])
    layer.drop_sequence(s)


def test_calls_are_ordered_with_the_callers_stream(layer):
    """A context on a stream of its own, nothing synchronised: q and kv are still being made when forward is called,
    are overwritten and freed right after it, and its result is read at once."""
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.latent import LatentAttention
    ctx = moe.MoeCtx(0, torch.cuda.Stream())
    L = LatentAttention(ctx, H, DC, DR, DN, DV, n_pages=40, page_size=16, max_positions=400, dtype=torch.float16)
    L.set_weights(layer.w_kv, layer.norm_w)
    data, caller = tokens(45, 130), torch.cuda.Stream()
    busy = torch.randn((4096, 4096), device="cuda")
    torch.cuda.synchronize()
    counts, outs = [120, 1, 1, 8], []
    with torch.cuda.stream(caller):
        s, at = L.new_sequence(), 0
        for n in counts:
            x = busy
            for _ in range(40):  # about 100 ms before the inputs are there
                x = torch.mm(x, busy).mul_(2.0 ** -6)
            q, kv = [torch.full_like(d[at:at + n], float("nan")) for d in data]
            q.copy_(data[0][at:at + n]).add_(x[0, 0] * 0)
            kv.copy_(data[1][at:at + n]).add_(x[0, 0] * 0)
            out = L.forward([s], [n], q, kv)
            q.fill_(float("nan"))
            kv.fill_(float("nan"))
            outs.append(out * 1)
            out.fill_(float("nan"))
            del q, kv, out
            at += n
        got = torch.cat(outs)
    caller.synchronize()
    ctx.check()
    close(got, definition(layer, *data, np.arange(130), causal(130)))
    ctx.close()


def test_prompts_beyond_the_expanded_form_are_absorbed(layer, monkeypatch):
    """More cached rows than moe_latent_prompt takes, or no memory for its workspace: the other form of the same function."""
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd import latent
    assert layer.expands([4096], [1 << 24])
    assert not layer.expands([4096], [(1 << 24) + 1])
    assert not layer.expands([4096, 1], [1 << 23, (1 << 23) + 1])

    q, kv = tokens(44, 100)
    want = definition(layer, q, kv, np.arange(100), causal(100))
    asked = []

    def full(*args):
        asked.append(args[-2])
        raise moe.MoeError(moe.MOE_ENOMEM, "hipMalloc: out of memory")

    monkeypatch.setattr(latent, "moe_latent_prompt", full)
    s = layer.new_sequence()
    out = layer.forward([s], [100], q, kv)
    layer.ctx.check()
    assert asked == [100]
    close(out, want)
    layer.drop_sequence(s)

    def wrong(*args):
        raise moe.MoeError(moe.MOE_EINVAL, "another error")

    monkeypatch.setattr(latent, "moe_latent_prompt", wrong)
    s = layer.new_sequence()
    before = state(layer)
    with pytest.raises(moe.MoeError):
        layer.forward([s], [100], q, kv)
    assert state(layer) == before
    layer.drop_sequence(s)
