"""A decoder layer: latent attention over its paged cache, then the routed
experts. Two sequences take a prompt, generate single tokens, and verify a
drafted tree, of which one path is kept.

    python examples/decoder_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import quantized_moe_expert_sigmoid_amd as moe  # noqa: E402
from quantized_moe_expert_sigmoid_amd.latent import LatentAttention  # noqa: E402
from quantized_moe_expert_sigmoid_amd.layer import MoeLayer  # noqa: E402

HIDDEN, HEADS, LATENT, ROPE, NOPE, VALUE = 128, 4, 128, 32, 64, 64


def unit(x):
    return x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()


class DecoderLayer:
    """x + attention(norm x), then x + experts(norm x); fp32 hidden states, bf16 attention, int4 experts."""

    def __init__(self, ctx, gen):
        def w(*shape):
            return torch.randn(shape, generator=gen) * shape[-1] ** -0.5

        self.attention = LatentAttention(ctx, HEADS, LATENT, ROPE, NOPE, VALUE, n_pages=64, page_size=16,
                                         max_positions=512)
        self.attention.set_weights(w(HEADS, NOPE + VALUE, LATENT), torch.ones(LATENT))
        self.w_q = w(HEADS * (NOPE + ROPE), HIDDEN).cuda()
        self.w_kv = w(LATENT + ROPE, HIDDEN).cuda()
        self.w_o = w(HIDDEN, HEADS * VALUE).cuda()
        self.experts = MoeLayer(ctx, HIDDEN, 64, 8, 2)
        for e in range(8):
            self.experts.set_expert_fp32(e, w(64, HIDDEN), w(64, HIDDEN), w(HIDDEN, 64))
        self.experts.set_shared_fp32(w(64, HIDDEN), w(64, HIDDEN), w(HIDDEN, 64))
        self.experts.set_router(w(8, HIDDEN), torch.zeros(8))

    def forward(self, seqs, counts, x, **draft):
        y = unit(x)
        q = (y @ self.w_q.t()).bfloat16().view(-1, HEADS, NOPE + ROPE)
        kv = (y @ self.w_kv.t()).bfloat16()
        o = self.attention.forward(seqs, counts, q, kv, **draft)
        x = x + o.flatten(1).float() @ self.w_o.t()
        return x + self.experts.forward(unit(x).contiguous())["out"]


def run():
    gen = torch.Generator().manual_seed(0)
    ctx = moe.MoeCtx(0)
    try:
        layer = DecoderLayer(ctx, gen)
        tokens = [torch.randn((60, HIDDEN), generator=gen).cuda(), torch.randn((45, HIDDEN), generator=gen).cuda()]
        a, b = layer.attention.new_sequence(), layer.attention.new_sequence()
        whole = layer.forward([a, b], [60, 45], torch.cat(tokens))
        layer.attention.drop_sequence(a)
        layer.attention.drop_sequence(b)

        # the same tokens: a prompt each, single tokens, then a draft of which the path 0 - 2 is the true text
        a, b = layer.attention.new_sequence(), layer.attention.new_sequence()
        got = [layer.forward([a, b], [50, 40], torch.cat([tokens[0][:50], tokens[1][:40]]))]
        for i in range(3):
            got.append(layer.forward([a, b], [1, 1], torch.stack([tokens[0][50 + i], tokens[1][40 + i]])))
        wrong = torch.randn((2, HIDDEN), generator=gen).cuda()
        draft = torch.stack([tokens[0][53], wrong[0], tokens[0][54], tokens[1][43], wrong[1], tokens[1][44]])
        verified = layer.forward([a, b], [3, 3], draft, tree=[0b001, 0b011, 0b101] * 2, depth=[0, 1, 1] * 2)
        for s in (a, b):
            layer.attention.keep(s, 3, [0, 2])
        last = layer.forward([a], [5], tokens[0][55:])
        ctx.check()

        want = torch.cat([whole[:50], whole[60:100]])
        pairs = [(got[0], want)] + [(got[1 + i], whole[[50 + i, 100 + i]]) for i in range(3)]
        pairs += [(verified[[0, 2, 3, 5]], whole[[53, 54, 103, 104]]), (last, whole[55:60])]
        return [float((g - w).norm() / w.norm()) for g, w in pairs]
    finally:
        ctx.close()


if __name__ == "__main__":
    names = ["prompts", "token 1", "token 2", "token 3", "verified path", "after the draft"]
    for name, err in zip(names, run()):
        print(f"{name}: relative difference to one pass over all tokens {err:.2e}")
