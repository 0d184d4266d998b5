"""Greedy decoding of a batch through one transformer block on one GPU: the operators of the
decode step around the routed-expert MoE layer, used together.

Per step and token:  q/k/v projection (w4_linear) -> rotation and append to the paged cache
(kv_append_rope) -> attention behind the batch's shared prompt (attn_shared_prefix) -> output
projection (w4_linear) -> MoE layer (dsv4_moe_forward) -> vocabulary projection (w4_linear) ->
log probabilities, entropy and the best alternatives (token_logprobs), the best of which is the
next token.  Weights are random; norms, residual sums and the embedding lookup are torch's.

    python examples/decode_block.py [--batch 8] [--prompt 300] [--steps 16] [--fp8-cache]
"""
from __future__ import annotations

import argparse
import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_expert_ffn_moe_amd as moe  # noqa: E402

DEV = "cuda:0"


@dataclass
class Config:
    hidden: int = 512
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    inter: int = 256
    experts: int = 16
    top_k: int = 4
    vocab: int = 5003
    page: int = 16
    fp8_cache: bool = False
    alternatives: int = 5


class Block:
    """The weights of one block and of the vocabulary, in the library's formats."""

    def __init__(self, cfg: Config, seed: int = 0):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        c = self.cfg = cfg
        self.kept = []

        def fp4(n_out, n_in):      # FP4 codes, power-of-two scales around 2^-7
            q = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device=DEV, dtype=torch.uint8)
            s = torch.randint(118, 121, (n_out, n_in // 32), generator=g, device=DEV,
                              dtype=torch.uint8)
            return moe.make_w4(moe.MOE_W_FP4_E2M1_UE8M0_K32, n_out, n_in, 32, q, s)

        def int4(n_out, n_in):     # 4-bit codes, scale and zero point per 128 inputs
            n_g = -(-n_in // 128)
            q = torch.randint(0, 256, (n_out, n_in // 2), generator=g, device=DEV, dtype=torch.uint8)
            s = (0.005 * (0.5 + torch.rand((n_out, n_g), generator=g, device=DEV))).to(torch.bfloat16)
            z = torch.randint(6, 10, (n_out, n_g), generator=g, device=DEV, dtype=torch.uint8)
            return moe.make_w4(moe.MOE_W_INT4_BF16_GROUP, n_out, n_in, 128, q, s, z)

        heads = c.q_heads + 2 * c.kv_heads
        self.qkv = int4(heads * c.head_dim, c.hidden)
        self.out = int4(c.hidden, c.q_heads * c.head_dim)
        self.vocab = fp4(c.vocab, c.hidden)
        self.embed = torch.randn((c.vocab, c.hidden), generator=g, device=DEV).to(torch.bfloat16)

        def experts(rows, cols):
            q = torch.randint(0, 256, (c.experts + 1, rows, cols // 2), generator=g, device=DEV,
                              dtype=torch.uint8)
            s = torch.randint(117, 120, (c.experts + 1, rows, cols // 32), generator=g, device=DEV,
                              dtype=torch.uint8)
            return q, s
        gate, up = experts(c.inter, c.hidden), experts(c.inter, c.hidden)
        self.moe = moe.make_weights(moe.MOE_W_FP4_E2M1_UE8M0_K32, c.experts, c.hidden, c.inter,
                                    *gate, *up, *experts(c.hidden, c.inter))
        self.router = (0.02 * torch.randn((c.hidden, c.experts), generator=g,
                                          device=DEV)).to(torch.bfloat16)


def rms_norm(x):
    x = x.float()
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Session:
    """A batch behind one shared prompt: cache, page tables, workspaces and step buffers.
    The prompt's keys are read through its own page list, the page in which it ends too;
    each sequence's tokens go to pages of its own from that page's place in its table on."""

    def __init__(self, block: Block, prompt: torch.Tensor, batch: int, max_new: int):
        c = self.cfg = block.cfg
        self.block, self.B, self.P = block, batch, prompt.numel()
        self.max_keys = self.P + max_new
        cols = -(-self.max_keys // c.page)
        pre = -(-self.P // c.page)
        shared = self.P // c.page
        n_pages = pre + batch * (cols - shared)
        shape = (n_pages, c.kv_heads, c.page, c.head_dim)
        if c.fp8_cache:
            self.k, self.v = (torch.zeros(shape, device=DEV, dtype=torch.uint8) for _ in range(2))
            self.ks, self.vs = (torch.zeros(shape[:3], device=DEV) for _ in range(2))
        else:
            self.k, self.v = (torch.zeros(shape, device=DEV, dtype=torch.bfloat16) for _ in range(2))
            self.ks = self.vs = None
        self.cache = moe.make_kv_cache(moe.MOE_DT_FP8_E4M3 if c.fp8_cache else moe.MOE_DT_BF16, n_pages,
                                       c.page, c.kv_heads, c.head_dim, self.k, self.v, self.ks,
                                       self.vs)
        i32 = dict(device=DEV, dtype=torch.int32)
        self.prefix_pages = torch.arange(pre, **i32)
        own = pre + torch.arange(batch * (cols - shared), **i32).view(batch, cols - shared)
        self.table = torch.cat([self.prefix_pages[:shared].expand(batch, shared), own], 1).contiguous()
        a = torch.arange(self.max_keys, device=DEV, dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, c.head_dim, 2, device=DEV, dtype=torch.float64) / c.head_dim)
        self.rope = torch.cat([a.cos(), a.sin()], 1).float().contiguous()
        self.status = torch.zeros(1, **i32)

        B, bf = batch, dict(device=DEV, dtype=torch.bfloat16)
        self.token = torch.full((B,), int(prompt[-1]), **i32)
        self.pos = torch.full((B,), self.P, **i32)
        self.seq = torch.arange(B, **i32)
        self.row = (c.q_heads + 2 * c.kv_heads) * c.head_dim
        self.qkv = torch.empty((B, self.row), **bf)
        self.q = torch.empty((B, c.q_heads, c.head_dim), **bf)
        self.att = torch.empty_like(self.q)
        self.lse = torch.empty((B, c.q_heads), device=DEV)
        self.o = torch.empty((B, c.hidden), **bf)
        self.ffn = torch.empty((B, c.hidden), **bf)
        self.logits = torch.empty((B, c.vocab), device=DEV)
        self.logprob = torch.empty(B, device=DEV)
        self.entropy = torch.empty(B, device=DEV)
        self.top_ids = torch.empty((B, c.alternatives), **i32)
        self.top_lp = torch.empty((B, c.alternatives), device=DEV)
        self.attn_bytes = moe.attn_workspace_bytes(self.cache, B, 1, c.q_heads, self.P, self.max_keys)
        self.attn_ws = torch.empty(self.attn_bytes, device=DEV, dtype=torch.uint8)
        self.moe_bytes = moe.moe_workspace_bytes(block.moe, B, c.top_k)
        self.moe_ws = torch.empty(self.moe_bytes, device=DEV, dtype=torch.uint8)
        moe.moe_workspace_init(self.moe_ws, self.moe_bytes)
        self.lp_bytes = moe.token_logprobs_workspace_bytes(B, c.vocab, c.alternatives)
        self.lp_ws = torch.empty(self.lp_bytes, device=DEV, dtype=torch.uint8)
        self._prefill(prompt)

    def _append(self, qkv, T, seq, pos, table, q_out):
        c, at = self.cfg, qkv.data_ptr()
        kv = 2 * c.q_heads * c.head_dim
        moe.kv_append_rope(self.cache, at, self.row, c.q_heads, at + kv, self.row,
                           at + kv + 2 * c.kv_heads * c.head_dim, self.row, T, self.rope,
                           self.max_keys, c.head_dim, moe.ROPE_HALF, seq, pos, table,
                           table.shape[0], table.shape[1], q_out, self.status)

    def _prefill(self, prompt):
        """The prompt's keys and values (one block: they depend on the embeddings alone)."""
        c = self.cfg
        x = rms_norm(self.block.embed[prompt.to(DEV)])
        qkv = torch.empty((self.P, self.row), device=DEV, dtype=torch.bfloat16)
        moe.w4_linear(self.block.qkv, x, c.hidden, self.P, qkv, self.row, moe.MOE_DT_BF16)
        q = torch.empty((self.P, c.q_heads, c.head_dim), device=DEV, dtype=torch.bfloat16)
        pos = torch.arange(self.P, device=DEV, dtype=torch.int32)
        self._append(qkv, self.P, torch.zeros_like(pos), pos, self.prefix_pages[None], q)

    def step(self):
        """One token for every sequence; everything is enqueued on the current stream, and the
        next step's inputs are left in place (so a captured step can be replayed)."""
        c, b, B = self.cfg, self.block, self.B
        x = b.embed[self.token]
        moe.w4_linear(b.qkv, rms_norm(x), c.hidden, B, self.qkv, self.row, moe.MOE_DT_BF16)
        self._append(self.qkv, B, self.seq, self.pos, self.table, self.q)
        moe.attn_shared_prefix(self.cache, self.q, c.q_heads * c.head_dim, B, 1, c.q_heads,
                               self.pos, self.prefix_pages, self.P, self.table,
                               self.table.shape[1], self.max_keys, c.head_dim ** -0.5, self.att,
                               self.lse, self.status, self.attn_ws, self.attn_bytes)
        moe.w4_linear(b.out, self.att, c.q_heads * c.head_dim, B, self.o, c.hidden, moe.MOE_DT_BF16)
        x = x + self.o
        moe.dsv4_moe_forward(b.moe, b.router, rms_norm(x), B, c.top_k, None, None, self.ffn,
                             moe.MOE_DT_BF16, self.moe_ws, self.moe_bytes)
        x = rms_norm(x + self.ffn)
        moe.w4_linear(b.vocab, x, c.hidden, B, self.logits, c.vocab, moe.MOE_DT_F32)
        moe.token_logprobs(self.logits, moe.MOE_DT_F32, c.vocab, B, c.vocab, None, c.alternatives,
                           None, self.entropy, self.top_ids, self.top_lp, self.status, self.lp_ws,
                           self.lp_bytes)
        self.token.copy_(self.top_ids[:, 0])
        self.pos.add_(1)


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--batch", type=int, default=8)
    p.add_argument("--prompt", type=int, default=300)
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--fp8-cache", action="store_true")
    a = p.parse_args()
    cfg = Config(fp8_cache=a.fp8_cache)
    block = Block(cfg)
    prompt = torch.randint(0, cfg.vocab, (a.prompt,), generator=torch.Generator().manual_seed(1))
    s = Session(block, prompt, a.batch, a.steps + 4)
    # different first tokens, so that the sequences part
    s.token.copy_(torch.arange(a.batch, device=DEV, dtype=torch.int32) * 7 % cfg.vocab)
    for _ in range(2):
        s.step()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        s.step()
    torch.cuda.synchronize()
    t = time.perf_counter()
    for i in range(a.steps):
        graph.replay()
    torch.cuda.synchronize()
    dt = (time.perf_counter() - t) / a.steps
    assert int(s.status.item()) == 0
    print("last step: tokens %s" % s.token.tolist())
    print("           log probabilities %s" % [round(v, 3) for v in s.top_lp[:, 0].tolist()])
    print("           entropies %s" % [round(v, 3) for v in s.entropy.tolist()])
    print("%.1f us a step of %d tokens (graph replay)" % (dt * 1e6, a.batch))


if __name__ == "__main__":
    main()
