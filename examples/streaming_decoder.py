"""A streaming audio decoder's step with ctconv: one transformer block over a
bounded paged cache, then the first transposed convolution of its upsampler.

    python examples/streaming_decoder.py            # 400 frames of 4 streams

Per frame and stream, one new row
  - is appended to the cache and attends to what the cache holds
    (cache_append, paged_attention), the softmax weights being added up;
  - attends to the text encoder's states (cross_attention);
  - passes the seams between the blocks: residual, layer scale, gate and the
    next block's norm in one pass (norm_residual);
  - becomes `hop` rows by a streaming ConvTranspose1d, a few frames per call
    (ctconv_stream_step).
When the cache has grown by `slack` rows past `keep`, it is cut back to the
first rows, the latest ones and those that drew the most attention
(cache_evict).  Each operator is a plan, whose sizes are marshalled once, called
with pointers into buffers that live as long as the decoder; the module's
functions of the same names take tensors and make the plan themselves, at some
20 us a call.  Matrix products with the weights are torch's.  Weights are
random: this shows the calls, it does not speak."""

from __future__ import annotations

import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from vision_upsampler_decoders_amd import ctconv as C  # noqa: E402


@dataclass
class Config:
    streams: int = 4
    width: int = 256
    heads: int = 8
    kv_heads: int = 4
    encoder_rows: int = 120
    page: int = 16
    keep: int = 128
    slack: int = 32
    sink: int = 4
    recent: int = 48
    channels: int = 64  # of the first upsampled layer
    hop: int = 8
    chunk: int = 4  # frames per convolution: rows of 8 bytes take its matrix route
    dtype: torch.dtype = torch.bfloat16
    seed: int = 0

    @property
    def head(self) -> int:
        return self.width // self.heads


def make_weights(c: Config, device="cuda"):
    g = torch.Generator().manual_seed(c.seed)

    def mat(*shape, scale=None):
        w = torch.randn(shape, generator=g) * (shape[0] ** -0.5 if scale is None else scale)
        return w.to(c.dtype).to(device)

    kv = c.kv_heads * c.head
    w = {"in": mat(c.width, c.width), "start": mat(c.width, scale=0.1),
         "qkv": mat(c.width, c.width + 2 * kv), "out": mat(c.width, c.width),
         "cross_q": mat(c.width, c.width), "cross_kv": mat(c.width, 2 * kv),
         "cross_out": mat(c.width, c.width), "gate": mat(c.width, c.width),
         "up": mat(c.width, 4 * c.width), "down": mat(4 * c.width, c.width),
         "conv": mat(c.width, c.channels, 2 * c.hop, scale=(2 * c.width) ** -0.5)}
    for n in ("self", "cross", "mlp", "last"):  # a norm before each block and before the conv
        w["norm_" + n], w["bias_" + n] = 1 + mat(c.width, scale=0.1), mat(c.width, scale=0.1)
        w["scale_" + n] = mat(c.width, scale=0.1) + 0.3
    return w


class Decoder:
    """The state of `streams` streams that run in step."""

    def __init__(self, c: Config, weights, encoder, encoder_lengths=None):
        self.c, self.w = c, weights
        B, H, D = c.streams, c.kv_heads, c.head
        dev = encoder.device
        self.cols = -(-(c.keep + c.slack) // c.page)
        slots = self.cols * c.page
        pool = B * self.cols
        self.k = torch.zeros(pool, H, c.page, D, dtype=c.dtype, device=dev)
        self.v = torch.zeros_like(self.k)
        self.table = torch.randperm(pool).int().view(B, self.cols).to(dev)
        self.lengths = torch.zeros(B, dtype=torch.int32, device=dev)
        self.now = torch.zeros_like(self.lengths)
        self.positions = torch.zeros(B, H, slots, dtype=torch.int32, device=dev)
        self.weight_sum = torch.zeros(B, H, slots, device=dev)
        self.rows = 0
        kv = (encoder @ weights["cross_kv"]).view(B, -1, 2, H, D)
        self.enc_k, self.enc_v, self.enc_n = kv[:, :, 0], kv[:, :, 1], encoder_lengths
        self.packed = C.prepack(weights["conv"], (c.hop,))
        self.tail = [torch.zeros(B, c.channels, c.hop, device=dev) for _ in range(2)]
        code = C.dtype_code(encoder)
        _, _, nb = C.ctconv_stream_sizes(B, c.channels, c.chunk, 2 * c.hop, c.hop, code)
        self.conv_ws = torch.empty(nb, dtype=torch.uint8, device=dev)
        self.pending = torch.empty(B, c.width, c.chunk, dtype=c.dtype, device=dev)
        self.held = 0
        # plans
        pages = dict(num_pages=pool, page_size=c.page, max_pages=self.cols, dtype=code)
        row = c.width + 2 * H * D  # q, k and v of a row lie behind each other
        self.append = C.CacheAppend(B, 1, H, D, new_strides=(row, row, D), **pages)
        self.attend = C.PagedAttention(B, c.heads, H, D, weights=True, q_strides=(row, D), **pages)
        self.evict = C.CacheEvict(B, H, D, keep=c.keep, sink=c.sink, recent=c.recent,
                                  out_slot_strides=(H * slots, slots), **pages)
        Lk = encoder.shape[1]
        kvs = tuple(self.enc_k.stride()[:3])
        self.cross = C.CrossAttention(B, 1, Lk, c.heads, H, D, dtype=code, k_strides=kvs,
                                      v_strides=kvs)
        self.first = C.NormResidual(B, c.width, dtype=code, strides=(0,) + (c.width,) * 4)
        self.plain = C.NormResidual(B, c.width, dtype=code)
        self.gated = C.NormResidual(B, c.width, gate=C.GATE_SIGMOID, dtype=code)
        need = max(self.attend.workspace_bytes, self.cross.workspace_bytes, 16)
        self.ws = torch.empty(need, dtype=torch.uint8, device=dev)
        self.x, self.y, self.a = (torch.empty(B, c.width, dtype=c.dtype, device=dev)
                                  for _ in range(3))
        self.source = torch.empty(B, H, c.keep, dtype=torch.int32, device=dev)
        self.code = code

    def seam(self, plan, x, h, block: str, scale: str, gate=None):
        """self.x, self.y = x + scale * gate * h, its norm before `block`."""
        w = self.w
        plan(x.data_ptr(), h.data_ptr(), None, None, w["scale_" + scale].data_ptr(),
             None if gate is None else gate.data_ptr(), w["norm_" + block].data_ptr(),
             w["bias_" + block].data_ptr(), self.x.data_ptr(), self.y.data_ptr(), self.stream)

    def step(self, frame):
        """One frame [streams, width].  Every `chunk` frames: their rows
        [streams, channels, chunk * hop]; else None."""
        c, w = self.c, self.w
        B, H, D = c.streams, c.kv_heads, c.head
        x, y, a = self.x, self.y, self.a
        self.stream = torch.cuda.current_stream().cuda_stream
        k, v, table = self.k.data_ptr(), self.v.data_ptr(), self.table.data_ptr()
        lengths, now = self.lengths.data_ptr(), self.now.data_ptr()
        positions, weights = self.positions.data_ptr(), self.weight_sum.data_ptr()
        ws, nb = self.ws.data_ptr(), self.ws.numel()

        self.seam(self.first, w["start"], frame @ w["in"], "self", "last")
        qkv = y @ w["qkv"]
        q = qkv.data_ptr()
        new = q + c.width * qkv.element_size()
        self.rows += 1
        self.lengths += 1
        self.now += 1
        self.append(new, new + H * D * qkv.element_size(), k, v, table, lengths, None, now,
                    positions, weights, self.stream)
        self.attend(q, k, v, table, lengths, a.data_ptr(), None, weights, ws, nb, self.stream)
        self.seam(self.plain, x, a @ w["out"], "cross", "self")
        q = y @ w["cross_q"]
        self.cross(q.data_ptr(), self.enc_k.data_ptr(), self.enc_v.data_ptr(),
                   None if self.enc_n is None else self.enc_n.data_ptr(), None, a.data_ptr(), None,
                   ws, nb, self.stream)
        self.seam(self.plain, x, a @ w["cross_out"], "mlp", "cross")
        h = torch.nn.functional.gelu(y @ w["up"]) @ w["down"]
        self.seam(self.gated, x, h, "last", "mlp", gate=y @ w["gate"])
        if self.rows == c.keep + c.slack:
            self.evict(k, v, table, lengths, now, weights, positions, weights, positions, lengths,
                       self.source.data_ptr(), self.stream)
            self.rows = c.keep
        self.pending[:, :, self.held].copy_(y)
        self.held = (self.held + 1) % c.chunk
        if self.held:
            return None
        rows = torch.empty(B, c.channels, c.chunk * c.hop, dtype=c.dtype, device=y.device)
        C.ctconv_stream_step(self.pending.data_ptr(), self.packed.data_ptr(), None, rows.data_ptr(),
                             self.tail[0].data_ptr(), self.tail[1].data_ptr(),
                             self.conv_ws.data_ptr(), B, c.width, c.channels, c.chunk, 2 * c.hop,
                             c.hop, self.code, C.ACT_NONE, self.stream)
        self.tail.reverse()
        return rows


def main(frames: int = 400):
    c = Config()
    g = torch.Generator(device="cuda").manual_seed(1)
    encoder = torch.randn(c.streams, c.encoder_rows, c.width, generator=g, device="cuda").to(c.dtype)
    lengths = torch.tensor([c.encoder_rows - 7 * b for b in range(c.streams)], dtype=torch.int32,
                           device="cuda")
    dec = Decoder(c, make_weights(c), encoder, lengths)
    inputs = torch.randn(frames, c.streams, c.width, generator=g, device="cuda").to(c.dtype)
    out = [dec.step(inputs[f]) for f in range(min(8, frames - 1))]  # the first frames load kernels
    torch.cuda.synchronize()
    start = time.perf_counter()
    done = len(out)
    for f in range(done, frames):
        out.append(dec.step(inputs[f]))
    torch.cuda.synchronize()
    per = (time.perf_counter() - start) / (frames - done)
    wave = torch.cat([o for o in out if o is not None], -1).float()
    print(f"{frames} frames of {c.streams} streams: {per * 1e6:.0f} us a frame, "
          f"{dec.rows} rows cached per stream, rms {wave.square().mean().sqrt():.3f}, "
          f"finite: {bool(torch.isfinite(wave).all())}")
    return wave


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 400)
