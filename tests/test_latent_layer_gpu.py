"""The latent-attention layer object (norm, rotation, cache pages, the choice of
form, drafts) against the definition in 64 bits, and the decoder-layer example."""
import importlib.util
import os

import numpy as np
import pytest

from tests.gpu_util import log

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

H, DC, DR, DN, DV = 6, 128, 32, 64, 64
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def layer():
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.latent import LatentAttention
    ctx = moe.MoeCtx(0)
    L = LatentAttention(ctx, H, DC, DR, DN, DV, n_pages=40, page_size=16, max_positions=400, dtype=torch.float16)
    g = torch.Generator().manual_seed(1)
    L.set_weights(torch.randn((H, DN + DV, DC), generator=g) * DC ** -0.5, 1 + 0.1 * torch.randn((DC,), generator=g))
    yield L
    ctx.close()


def definition(L, q, kv, pos, seen):
    """One sequence: q [n][H][DN + DR], kv [n][DC + DR] of all its tokens, their positions, seen [n][n]."""
    q, kv = q.double().cpu().numpy(), kv.double().cpu().numpy()
    w, norm = L.w_kv.double().cpu().numpy(), L.norm_w.double().cpu().numpy()
    angle = np.asarray(pos, dtype=np.float64)[:, None] * 10000.0 ** (-np.arange(DR // 2) * 2 / DR)
    turn = np.exp(1j * angle)

    def rotate(x):
        z = (x[..., 0::2] + 1j * x[..., 1::2]) * turn.reshape(turn.shape[:1] + (1,) * (x.ndim - 2) + turn.shape[1:])
        return np.stack([z.real, z.imag], axis=-1).reshape(x.shape)

    c = kv[:, :DC] / np.sqrt((kv[:, :DC] ** 2).mean(1, keepdims=True) + L.eps) * norm
    k, qr = rotate(kv[:, DC:]), rotate(q[..., DN:])
    out = np.zeros((len(pos), H, DV))
    for h in range(H):
        z = (q[:, h, :DN] @ (c @ w[h, :DN].T).T + qr[:, h] @ k.T) * L.cfg.scale
        z = np.where(seen, z, -np.inf)
        p = np.exp(z - z.max(1, keepdims=True))
        out[:, h] = p / p.sum(1, keepdims=True) @ (c @ w[h, DN:].T)
    return out


def close(got, want):
    """2-norm: fp16 roundings (u = 2^-11) of the cached latent and key, the rotated query and the four of the kernels,
    each below u / sqrt(3) of what it rounds, with scores of rms below 1.5: under 2.1 u; 4 u is accepted."""
    rel = np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want)
    log(f"  relative error {rel * 2 ** 11:.2f} u")
    assert rel <= 4 * 2.0 ** -11


def tokens(seed, n):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((n, H, DN + DR), generator=g).half().cuda(), torch.randn((n, DC + DR), generator=g).half().cuda())


def test_prompt_steps_and_pieces(layer):
    n = [90, 33]
    data = [tokens(10 + i, n[i]) for i in range(2)]
    want = [definition(layer, *data[i], np.arange(n[i]), np.tril(np.ones((n[i], n[i]), bool))) for i in range(2)]
    seqs = [layer.new_sequence() for _ in range(2)]
    at = [0, 0]
    forms = set()
    for counts in ([70, 1], [1, 1], [1, 20], [0, 1], [18, 10]):
        q = torch.cat([data[i][0][at[i]:at[i] + c] for i, c in enumerate(counts)])
        kv = torch.cat([data[i][1][at[i]:at[i] + c] for i, c in enumerate(counts)])
        forms.add(layer.expands(counts, [a + c for a, c in zip(at, counts)]))
        out = layer.forward(seqs, counts, q, kv)
        layer.ctx.check()
        log("counts", counts)
        close(out, np.concatenate([want[i][at[i]:at[i] + c] for i, c in enumerate(counts)]))
        at = [a + c for a, c in zip(at, counts)]
    assert at == n and forms == {True, False}
    assert [layer.length(s) for s in seqs] == n
    free = len(layer._free)
    for s in seqs:
        layer.drop_sequence(s)
    assert len(layer._free) == free + 6 + 3


def test_draft_and_keep(layer):
    """A prompt, a draft of five nodes, of which the path 0 - 2 - 4 stays, then a token."""
    q, kv = tokens(20, 26)
    s = layer.new_sequence()
    layer.forward([s], [20], q[:20], kv[:20])
    tree, depth = [0b00001, 0b00011, 0b00101, 0b01011, 0b10101], [0, 1, 1, 2, 2]
    out = layer.forward([s], [5], q[20:25], kv[20:25], tree=tree, depth=depth)
    layer.ctx.check()
    pos = list(range(20)) + [20 + d for d in depth]
    seen = np.zeros((25, 25), bool)
    seen[:20, :20] = np.tril(np.ones((20, 20), bool))
    for i, w in enumerate(tree):
        seen[20 + i, :20] = True
        seen[20 + i, 20:] = [(w >> j) & 1 for j in range(5)]
    close(out, definition(layer, q[:25], kv[:25], pos, seen)[20:])
    layer.keep(s, 5, [0, 2, 4])
    assert layer.length(s) == 23
    path = list(range(20)) + [20, 22, 24, 25]
    out = layer.forward([s], [1], q[25:], kv[25:])
    layer.ctx.check()
    close(out, definition(layer, q[path], kv[path], np.arange(24), np.tril(np.ones((24, 24), bool)))[23:])
    layer.keep(s, 1, [])
    assert layer.length(s) == 23
    layer.drop_sequence(s)


def test_refusals(layer):
    q, kv = tokens(30, 4)
    s = layer.new_sequence()
    with pytest.raises(ValueError):
        layer.forward([s], [3], q, kv)
    with pytest.raises(ValueError):
        layer.forward([s, s], [2, 2], q, kv)
    with pytest.raises(ValueError):
        layer.forward([s], [4], q, kv, tree=[1] * 4)
    with pytest.raises(RuntimeError):
        layer._resize(s, 41 * 16)
    layer.forward([s], [4], q, kv)
    with pytest.raises(ValueError):
        layer.keep(s, 4, [2, 1])
    with pytest.raises(ValueError):
        layer.keep(s, 4, [4])
    layer.drop_sequence(s)


def test_refused_calls_leave_the_sequences_as_they_were(layer):
    a, b = layer.new_sequence(), layer.new_sequence()
    q, kv = tokens(31, 700)
    layer.forward([a], [20], q[:20], kv[:20])
    free = len(layer._free)

    def refused(error, *args, **kw):
        with pytest.raises(error):
            layer.forward(*args, **kw)
        assert (layer.length(a), layer.length(b), len(layer._free)) == (20, 0, free)

    refused(RuntimeError, [a, b], [20, 680], q, kv)  # room for the first, not for both
    refused(ValueError, [a, b], [3, 401], q[:404], kv[:404])  # a position behind the table's
    refused(ValueError, [a], [2], q[:2], kv[:2], tree=[1, 3], depth=[0, 380])
    refused(ValueError, [a], [2], q[:2], kv[:2], tree=[1, 3], depth=[-1, 0])
    refused(ValueError, [a], [2], q[:2], kv[:2], tree=[1], depth=[0])
    refused(ValueError, [a], [65], q[:65], kv[:65], tree=[1] * 65, depth=[0] * 65)
    refused(ValueError, [a, b], [3, -1], q[:2], kv[:2])
    layer.drop_sequence(a)
    layer.drop_sequence(b)


def test_layer_on_a_stream_of_its_own(layer):
    """The same bits as on the default stream, weights and drafts included."""
    import quantized_moe_expert_sigmoid_amd as moe
    from quantized_moe_expert_sigmoid_amd.latent import LatentAttention
    q, kv = tokens(32, 30)

    def steps(L):
        s = L.new_sequence()
        outs = [L.forward([s], [20], q[:20], kv[:20]),
                L.forward([s], [4], q[20:24], kv[20:24], tree=[1, 3, 5, 13], depth=[0, 1, 1, 2])]
        L.keep(s, 4, [0, 2, 3])
        outs.append(L.forward([s], [6], q[24:], kv[24:]))
        L.ctx.check()
        L.drop_sequence(s)
        return outs

    want = steps(layer)
    torch.cuda.synchronize()
    ctx = moe.MoeCtx(0, torch.cuda.Stream())
    L = LatentAttention(ctx, H, DC, DR, DN, DV, n_pages=40, page_size=16, max_positions=400, dtype=torch.float16)
    L.set_weights(layer.w_kv * 1, layer.norm_w * 1)
    got = steps(L)
    ctx.stream.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    ctx.close()


def test_decoder_layer_example():
    """Prompt, single tokens and a verified draft give what one pass over all tokens gives, up to the roundings of the
    two forms (bf16, u = 2^-8: 4 u of the attention's share of each output is accepted) and the experts' int8
    activations, whose codes may differ by one step of 1/127 of the row's largest value where an input moved."""
    spec = importlib.util.spec_from_file_location("decoder_layer", os.path.join(ROOT, "examples", "decoder_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    errs = m.run()
    log(errs)
    assert all(e <= 4 * 2.0 ** -8 + 1 / 127 for e in errs)
