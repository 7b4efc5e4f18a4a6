"""Learns the token embedding of a mixed text / visual sequence.

Synthetic features are tokenised (rvq_encode); the per-level embedding tables
and a text table are then trained so that the normed embedding of each
token points the way of a target: for a visual token a fixed random map of
its features, for a text token a fixed random vector of its ID.  One step is
embed -> RMS norm -> loss -> RMS norm gradient -> tables' gradients -> AdamW
(8-bit or 32-bit states, clipped).  At the end the rows are normed once more
with an 8-bit output, the form in which a served model takes them.

  python examples/learn_token_embedding.py [--steps 100] [--bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import residual_vector_quantization_rvq_amd as rvq  # noqa: E402


def sequence(dev, L=4, K=256, d=64, D=512, V=500, images=4, patches=400, text=100):
    """(ids, is_visual, targets): images of `patches` visual tokens, each after `text` text tokens."""
    g = torch.Generator(device=dev).manual_seed(0)
    n = images * patches
    x = torch.randn((n, d), generator=g, device=dev)
    codebooks = torch.randn((L, K, d), generator=g, device=dev)
    codebooks *= (0.7 ** torch.arange(L, device=dev))[:, None, None]
    visual_ids = rvq.rvq_encode(x, codebooks).view(images, patches, L)
    features = rvq.rvq_decode(visual_ids.view(n, L), codebooks)
    text_ids = torch.zeros((images, text, L), dtype=torch.int32, device=dev)
    text_ids[:, :, 0] = torch.randint(0, V, (images, text), generator=g, device=dev).int()
    ids = torch.cat([text_ids, visual_ids], 1).view(-1, L).contiguous()
    vis = torch.cat([torch.zeros(images, text), torch.ones(images, patches)], 1).view(-1).to(dev, torch.uint8)
    target = torch.empty((ids.shape[0], D), device=dev)
    target[vis == 1] = features @ torch.randn((d, D), generator=g, device=dev)
    target[vis == 0] = torch.randn((V, D), generator=g, device=dev)[ids[vis == 0, 0].long()]
    target /= target.square().mean(1, keepdim=True).sqrt()
    return ids, vis, target.to(torch.bfloat16)


def train(steps=100, state_bits=8, lr=0.02, quiet=True):
    """(first loss, last loss): mean squared distance of the normed rows from their targets."""
    dev = torch.device("cuda:0")
    L, K, V, D = 4, 256, 500, 512
    ids, vis, target = sequence(dev, L, K, 64, D, V)
    g = torch.Generator(device=dev).manual_seed(1)
    masters = [0.02 * torch.randn((L, K, D), generator=g, device=dev),
               0.02 * torch.randn((V, D), generator=g, device=dev), torch.ones(D, device=dev)]
    level, text, weight = (p.to(torch.bfloat16) for p in masters)   # what the forward pass reads
    state = rvq.rvq_adamw_init(masters, state_bits, weight_decay=[0.0, 0.0, 0.0], copies=[level, text, weight])
    first = loss = None
    for step in range(1, steps + 1):
        x = rvq.rvq_embed_tokens(ids, level, vis, text, out_dtype=torch.bfloat16)
        y = rvq.rvq_rms_norm(x, weight, need_rstd=True)
        diff = y.y.float() - target.float()
        dy = (2.0 / diff.numel() * diff).to(torch.bfloat16)
        dx, dweight = rvq.rvq_rms_norm_backward(dy, x, y.rstd, weight)
        dlevel, dtext = rvq.rvq_embed_tokens_backward(dx, ids, K, vis, V)
        rvq.rvq_adamw_step(state, [dlevel, dtext, dweight], step, lr, max_norm=1.0, seed=step)
        if step in (1, steps) or step % 20 == 0:
            loss = diff.square().mean().item()
            first = loss if first is None else first
            if not quiet:
                print(f"step {step}: loss {loss:.4f}", flush=True)
    x = rvq.rvq_embed_tokens(ids, level, vis, text, out_dtype=torch.bfloat16)
    served = rvq.rvq_rms_norm(x, weight, out_dtype=torch.float8_e4m3fn)
    if not quiet:
        off = (served.y.float() * served.scale[:, None] - target.float()).square().mean().item()
        print(f"with 8-bit rows: loss {off:.4f}")
    return first, loss


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--bits", type=int, default=8, choices=(8, 32))
    a = ap.parse_args()
    train(a.steps, a.bits, quiet=False)
