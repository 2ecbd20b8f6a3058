"""One decoder block on the library: a prompt in chunks, then single tokens.

The attention half (norm, projections, rotation and append, paged attention)
and the routed-expert half (norm, router, experts: on Q8_K rows where they are
few, on fp32 rows where they are many) of a block with random weights.  The projections are plain matrix products of
the caller's; everything between them is a call of the library.

    python examples/decoder_block.py            # a cache of 16-bit values
    python examples/decoder_block.py --codes    # of 8-bit codes, a window with sinks, and drafted trees
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from quantized_routed_expert_02_gb300 import moeq4k as m  # noqa: E402
from quantized_routed_expert_02_gb300 import synth  # noqa: E402

EPS = 1e-6


class Block:
    """Weights and cache of one block for up to ``B`` sequences of up to ``max_len`` tokens; ``codes``: the
    cache in 8 bits; ``window``, ``sinks``: what a token sees."""

    def __init__(self, H=2048, Hq=32, Hkv=4, D=128, E=8, k=2, I=768, B=2, max_len=512, page=16,  # noqa: E741
                 dtype=torch.bfloat16, device="cuda", seed=0, codes=False, window=0, sinks=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, std=1.0, t=torch.float32):
            return (torch.randn(shape, generator=g, device=device) * std).to(t)

        self.H, self.Hq, self.Hkv, self.D, self.E, self.k, self.I = H, Hq, Hkv, D, E, k, I
        self.dtype, self.device, self.B = dtype, device, B
        self.w_qkv = normal(H, (Hq + 2 * Hkv) * D, std=H ** -0.5, t=dtype)
        self.w_o = normal(Hq * D, H, std=(Hq * D) ** -0.5, t=dtype)
        self.norm1, self.norm2 = 1 + 0.1 * normal(H), 1 + 0.1 * normal(H)
        self.q_norm, self.k_norm = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        self.w_router = normal(E, H, std=0.02)
        blobs = synth.expert_blobs(synth.custom_shape(1, H, E, k, I, cfg_id=seed), 0)
        self.gate, self.up, self.down = (torch.from_numpy(blobs[n]).to(device) for n in ("gate", "up", "down"))
        self.inv_freq = 1e6 ** (-torch.arange(0, D, 2, device=device, dtype=torch.float64) / D)
        # the cache: pages of every sequence, handed out here in reverse order
        self.max_pages = -(-max_len // page)
        P = B * self.max_pages
        self.window, self.sinks = window, sinks
        self.k_pages = torch.zeros(P, Hkv, page, D, dtype=torch.int8 if codes else dtype, device=device)
        self.v_pages = torch.zeros_like(self.k_pages)
        self.k_scales = torch.zeros(P, Hkv, page, device=device) if codes else None
        self.v_scales = torch.zeros_like(self.k_scales) if codes else None
        self.table = torch.arange(P - 1, -1, -1, dtype=torch.int32, device=device).view(B, self.max_pages)
        self.lens = [0] * B
        self.attn_ws = m.alloc_attention_workspace(Hq, Hkv, D, device=device)
        self.ffn_ws = None

    def step(self, hidden: torch.Tensor, new: list[int], paths: list[list[int]] | None = None) -> torch.Tensor:
        """``hidden`` [N, H] fp32: the residual stream of new[b] tokens of each sequence, one after
        the other.  Returns it after the block (the input is updated in place on the way).  ``paths``:
        the new tokens are drafted trees; for each its path from the root among its sequence's new tokens,
        itself included."""
        N, dev, t = hidden.shape[0], self.device, self.dtype
        before = list(self.lens)
        self.lens = [a + n for a, n in zip(self.lens, new)]
        offs = torch.tensor([sum(new[:b]) for b in range(self.B + 1)], dtype=torch.int32, device=dev)
        lens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        starts = [a for a, n in zip(before, new) for _ in range(n)]
        if paths is None:
            tree, place = None, [p for a, n in zip(before, new) for p in range(a, a + n)]
        else:
            place = [a + len(p) - 1 for a, p in zip(starts, paths)]
            words = -(-max(new) // 32)
            bits = b"".join(sum(1 << i for i in p).to_bytes(4 * words, "little") for p in paths)
            tree = torch.frombuffer(bytearray(bits), dtype=torch.int32).view(N, words).to(dev)
        pos = torch.tensor([place], dtype=torch.int32, device=dev)

        # attention half
        x = torch.empty(N, self.H, dtype=t, device=dev)
        m.moe_add_rmsnorm(hidden, None, self.norm1, EPS, y=x)
        qkv = x @ self.w_qkv
        q = torch.empty(N, self.Hq, self.D, dtype=t, device=dev)
        cache, scales = (self.k_pages, self.v_pages), (self.k_scales, self.v_scales)
        if self.k_scales is not None:
            m.moe_rope_append_q8(qkv, pos, self.inv_freq, q, *cache, *scales, self.table, offs, lens, self.attn_ws,
                                 q_norm_w=self.q_norm, k_norm_w=self.k_norm, eps=EPS)
        else:
            m.moe_rope_append(qkv, pos, self.inv_freq, q, *cache, self.table, offs, lens, self.attn_ws,
                              q_norm_w=self.q_norm, k_norm_w=self.k_norm, eps=EPS)
        o = torch.empty_like(q)
        m.moe_attention_cache(q, *cache, self.table, offs, lens, max(new), self.D ** -0.5, o, self.attn_ws,
                              k_scales=scales[0], v_scales=scales[1], tree=tree, window=self.window, sinks=self.sinks)
        self.last = offs, lens
        branch = o.view(N, -1) @ self.w_o

        # routed-expert half: fp32 rows for the router and, where they are many, for the experts;
        # the norm's Q8_K rows for few (norm, router and experts of 2048 x 128 x 8, I 768: 8 rows 71
        # against 262 us, 24 170 against 766; from 32 rows on the fp32 rows: 164 against 217, a
        # prompt of 4096 0.6 ms against 29)
        few = N < 32
        y = torch.empty(N, self.H, device=dev)
        codes = (torch.empty(N, self.H, dtype=torch.int8, device=dev),
                 torch.empty(N, self.H // 256, device=dev),
                 torch.empty(N, self.H // 32, dtype=torch.int32, device=dev)) if few else None
        m.moe_add_rmsnorm(branch, hidden, self.norm2, EPS, sum_out=hidden, y=y, q8k=codes)
        need = m.moe_workspace_bytes(N, self.H, self.E, self.k, self.I)
        if self.ffn_ws is None or self.ffn_ws.numel() < need:
            self.ffn_ws = m.alloc_workspace(N, self.H, self.E, self.k, self.I, device=dev)
        idx = torch.empty(N, self.k, dtype=torch.int32, device=dev)
        w = torch.empty(N, self.k, device=dev)
        m.moe_router(y, self.w_router, None, self.k, idx, w, self.ffn_ws)
        ffn = torch.empty(N, self.H, device=dev)
        if few:
            m.moe_ffn_q8k_codes(*codes, idx, w, self.gate, self.up, self.down, self.E, self.I, ffn, self.ffn_ws)
        else:
            m.moe_ffn(y, idx, w, self.gate, self.up, self.down, self.E, self.I, ffn, self.ffn_ws)
        # the next block's first norm would add this branch on its way
        return hidden + ffn

    def keep(self, accepted: list[list[int]]) -> None:
        """Of the last step's new tokens of each sequence only these stay, a path of its tree."""
        offs, lens = self.last
        new = (offs[1:] - offs[:-1]).tolist()
        most = max(1, max(map(len, accepted)))
        keep = torch.tensor([a + [0] * (most - len(a)) for a in accepted], dtype=torch.int32, device=self.device)
        kept = torch.tensor([len(a) for a in accepted], dtype=torch.int32, device=self.device)
        m.moe_cache_keep(self.k_pages, self.v_pages, self.table, offs, lens, keep, kept, self.attn_ws,
                         k_scales=self.k_scales, v_scales=self.v_scales)
        self.lens = [n - d + len(a) for n, d, a in zip(self.lens, new, accepted)]

    def check(self) -> None:
        """Raises when the device recorded an error."""
        for ws in (self.attn_ws, self.ffn_ws):
            code, detail = m.moe_read_device_status(ws)
            if code:
                raise RuntimeError(f"device status {m.status_str(code)} ({detail})")


def main(codes: bool = False) -> None:
    torch.manual_seed(1)
    block = Block(codes=codes, **(dict(window=200, sinks=4) if codes else {}))
    prompt = torch.randn(300 + 40, 2048, device="cuda")
    # two prompts of 300 and 40 tokens: a first chunk of both, the rest of the longer one
    first = torch.cat([prompt[:128], prompt[300:]])
    out = [block.step(first.clone(), [128, 40]), block.step(prompt[128:300].clone(), [172, 0])]
    for _ in range(8):  # then a token of each at a time
        out.append(block.step(torch.randn(2, 2048, device="cuda"), [1, 1]))
    if codes:  # five drafts a sequence: a root, two children, a child of each; the second branch is accepted
        tree = [[0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4]]
        out.append(block.step(torch.randn(10, 2048, device="cuda"), [5, 5], paths=tree * 2))
        block.keep([[0, 2, 4]] * 2)
        out.append(block.step(torch.randn(2, 2048, device="cuda"), [1, 1]))
    block.check()
    print(f"cached tokens {block.lens}; last rows' norm {out[-1].norm(dim=1).tolist()}")


if __name__ == "__main__":
    main(codes="--codes" in sys.argv[1:])
