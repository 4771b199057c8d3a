"""GPU: examples/streaming_decoder.py, frame by frame, against the same decoder
written in plain float64 torch on the host over the whole sequence at once:
the cache and its eviction, both attentions, the seams and the streaming
transposed convolution together."""

import importlib.util
import os

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    path = os.path.join(ROOT, "examples", "streaming_decoder.py")
    spec = importlib.util.spec_from_file_location("streaming_decoder", path)
    m = importlib.util.module_from_spec(spec)
    import sys

    sys.modules["streaming_decoder"] = m
    spec.loader.exec_module(m)
    return m


def reference(E, c, w, encoder, enc_lengths, inputs):
    """[streams, channels, frames * hop] in float64; the cache is a list of rows
    per head, cut back by the same rule."""
    import torch

    w = {k: v.double().cpu() for k, v in w.items()}
    enc, inputs = encoder.double().cpu(), inputs.double().cpu()
    B, Hq, H, D, W = c.streams, c.heads, c.kv_heads, c.head, c.width
    G = Hq // H
    kv = (enc @ w["cross_kv"]).view(B, -1, 2, H, D)

    def norm(x, n):
        return torch.nn.functional.layer_norm(x, (W,), w["norm_" + n], w["bias_" + n], 1e-5)

    cache = [[[] for _ in range(H)] for _ in range(B)]  # [position, k, v, weight]
    out = []
    for f in range(inputs.shape[0]):
        x = w["start"] + w["scale_last"] * (inputs[f] @ w["in"])
        y = norm(x, "self")
        qkv = y @ w["qkv"]
        q, k, v = qkv[:, :W].view(B, Hq, D), *(t.view(B, H, D) for t in qkv[:, W:].chunk(2, -1))
        a = torch.zeros(B, Hq, D, dtype=torch.float64)
        for b in range(B):
            for h in range(H):
                rows = cache[b][h]
                rows.append([f, k[b, h], v[b, h], 0.0])
                K, V = torch.stack([r[1] for r in rows]), torch.stack([r[2] for r in rows])
                p = torch.softmax(q[b, h * G:(h + 1) * G] @ K.T * D ** -0.5, -1)
                a[b, h * G:(h + 1) * G] = p @ V
                for r, s in zip(rows, p.sum(0).tolist()):
                    r[3] += s
                if len(rows) == c.keep + c.slack:
                    safe = [r for r in rows if r[0] < c.sink or r[0] >= f + 1 - c.recent]
                    rest = sorted((r for r in rows if not (r[0] < c.sink or r[0] >= f + 1 - c.recent)),
                                  key=lambda r: -r[3])
                    cache[b][h] = safe + rest[:c.keep - len(safe)]
        x = x + w["scale_self"] * (a.view(B, -1) @ w["out"])
        y = norm(x, "cross")
        q = (y @ w["cross_q"]).view(B, Hq, D)
        for b in range(B):
            n = int(enc_lengths[b])
            for i in range(Hq):
                p = torch.softmax(q[b, i] @ kv[b, :n, 0, i // G].T * D ** -0.5, -1)
                a[b, i] = p @ kv[b, :n, 1, i // G]
        x = x + w["scale_cross"] * (a.view(B, -1) @ w["cross_out"])
        y = norm(x, "mlp")
        m = torch.nn.functional.gelu(y @ w["up"]) @ w["down"]
        x = x + w["scale_mlp"] * torch.sigmoid(y @ w["gate"]) * m
        out.append(norm(x, "last"))
    y = torch.stack(out, -1)  # [B, W, frames]
    full = torch.nn.functional.conv_transpose1d(y, w["conv"], stride=c.hop)
    return full[..., :inputs.shape[0] * c.hop]


@pytest.mark.parametrize("evicts", [False, True])
def test_streaming_decoder_example(evicts):
    import torch

    E = load_example()
    c = E.Config(streams=2, width=64, heads=4, kv_heads=2, encoder_rows=37, keep=24, slack=8,
                 recent=8, channels=16, hop=4, dtype=torch.float32)
    frames = 60 if evicts else 28
    say(f"example frames={frames}")
    g = torch.Generator().manual_seed(3)
    enc = torch.randn(c.streams, c.encoder_rows, c.width, generator=g).cuda()
    lengths = torch.tensor([c.encoder_rows, 20], dtype=torch.int32).cuda()
    inputs = torch.randn(frames, c.streams, c.width, generator=g).cuda()
    w = E.make_weights(c)
    dec = E.Decoder(c, w, enc, lengths)
    got = [o for o in (dec.step(inputs[f]) for f in range(frames)) if o is not None]
    got = torch.cat(got, -1).double().cpu()
    torch.cuda.synchronize()
    ref = reference(E, c, w, enc, lengths, inputs)
    # fp32 throughout: about a hundred roundings of 2^-24 in depth, sums of up
    # to 256 terms; a row kept or given up wrongly is off by more than 1e-2
    err = float((got - ref).abs().max() / ref.abs().max())
    say(f"  max |err| / max |ref| = {err:.2e}")
    assert err < 1e-4
    assert dec.rows == (24 + (60 - 32) % 8 if evicts else 28)
