"""Speculative decoding over one unified pool: adapters and KV pages side by side.

A small random transformer serves a few requests, each with its own LoRA adapter.
Per step, the first layers of the model propose `n_drafts` tokens per request, the
whole model checks them in one pass, and lora_spec_verify decides how many stand:

    per layer:  q, k, v = x W          (torch)
                q, v += s B_a (A_a x)  (lora_bgmv_apply, one launch for both slices)
                lora_kv_write          (k, v to the request's pages)
                lora_kv_attend         (the new tokens over the request's cache)
    per step:   lora_spec_verify       (accepted drafts and the token after them)

Refused drafts leave nothing to undo: the next step's kv_len ends before them and
its write goes over them.  Blocks are taken from the pool as requests grow and
given back when they end.

    python examples/speculative_serving.py [--drafts 4] [--tokens 48] [--fp8]
"""
import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gather_lora_matmul_amd as L  # noqa: E402


class Server:
    HIDDEN, HEADS, KV_HEADS, DIM, LAYERS, VOCAB = 256, 8, 2, 64, 4, 512
    DRAFT_LAYERS = 2          # the first layers are the draft model: their cache is the model's own
    PAGE = 2048               # elements of a page: 32 tokens of one head (64 with --fp8)
    MAX_TOKENS = 1024         # of one request

    def __init__(self, prompts, adapters, fp8=False, seed=0):
        self.gen = torch.Generator("cuda").manual_seed(seed)
        hid, qd, kd = self.HIDDEN, self.HEADS * self.DIM, self.KV_HEADS * self.DIM
        rnd = lambda *s: torch.randn(*s, generator=self.gen, device="cuda")
        self.embed = rnd(self.VOCAB, hid).bfloat16()
        # logits of a few units between tokens, so that drafts are often right
        self.head = (rnd(hid, self.VOCAB) * 4 / hid ** 0.5).bfloat16()
        self.layers = [dict(qkv=(rnd(hid, qd + 2 * kd) / hid ** 0.5).bfloat16(),
                            o=(rnd(qd, hid) * 0.3 / qd ** 0.5).bfloat16()) for _ in range(self.LAYERS)]
        self.adapters = list(adapters)                  # per request, -1: none
        n_adapters, slices = max(self.adapters) + 1, []
        for _ in range(self.LAYERS):
            slices += [(hid, qd), (hid, kd)]            # of each layer: q and v
        self.pool = L.lora_pool_create(self.PAGE, L.LORA_BF16, 4096, max(1, n_adapters), 16, slices)
        self.lora = {}
        for a in range(n_adapters):
            for s, (d_in, d_out) in enumerate(slices):
                rank = 4 * (1 + a % 4)
                A = (rnd(rank, d_in) / d_in ** 0.5).bfloat16()
                B = (rnd(d_out, rank) / rank ** 0.5).bfloat16()
                bits = [t.view(torch.int16).cpu().numpy().view(np.uint16) for t in (A, B)]
                L.lora_pool_upload(self.pool, a, s, rank, 0.5, *bits)
                self.lora[a, s] = (A, B, 0.5)
        L.lora_page_table_build(self.pool)

        dtype = L.LORA_FP8_E4M3 if fp8 else L.LORA_BF16
        self.T, self.per_block, n_scales = L.lora_kv_layout(self.pool, self.KV_HEADS, self.DIM, dtype)
        scales = torch.zeros(n_scales, dtype=torch.uint8, device="cuda") if fp8 else None
        self.cache = L.KvCache(self.pool, self.KV_HEADS, self.DIM, dtype, scales=scales)
        n, nb = len(prompts), -(-self.MAX_TOKENS // self.T)
        self.table = np.full((self.LAYERS, n, 2, self.KV_HEADS, nb), -1, np.int32)
        self.table_dev = torch.from_numpy(self.table).cuda()
        self.blocks = [0] * n
        self.tokens = [list(p) for p in prompts]        # of which all but the last are cached
        self.accepted = self.proposed = 0

    def close(self):
        used = self.table[self.table >= 0]
        torch.cuda.synchronize()
        L.lora_pool_free_pages(self.pool, used)
        free = L.lora_pool_info(self.pool)[0]
        L.lora_pool_destroy(self.pool)
        return free

    def grow(self, kv_len):
        """Blocks for kv_len[s] tokens of every request, in all layers."""
        dirty = False
        for s, n in enumerate(kv_len):
            while self.blocks[s] * self.T < n:
                ids = L.lora_pool_alloc_pages(self.pool, self.LAYERS * self.per_block)
                self.table[:, s, :, :, self.blocks[s]] = ids.reshape(self.LAYERS, 2, self.KV_HEADS)
                self.blocks[s] += 1
                dirty = True
        if dirty:
            self.table_dev.copy_(torch.from_numpy(self.table))

    def forward(self, rows, q_len, kv_len, n_layers):
        """Logits [n_tokens][VOCAB] of the new tokens `rows` (device ids, request by
        request), the last q_len[s] of kv_len[s]."""
        self.grow(kv_len)
        n, dev = len(rows), "cuda"
        q_start = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32, device=dev)
        lens = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        ids = torch.tensor(np.repeat(self.adapters, q_len), dtype=torch.int32, device=dev)
        H, KH, D = self.HEADS, self.KV_HEADS, self.DIM
        x = self.embed[rows.long()]
        out = torch.zeros(n, H, D, dtype=torch.bfloat16, device=dev)
        ws = None
        for i in range(n_layers):
            h = norm(x)
            qkv = h @ self.layers[i]["qkv"]
            q, k, v = (t.contiguous() for t in qkv.split([H * D, KH * D, KH * D], 1))
            L.lora_bgmv_apply(self.pool, [(2 * i, h, q, 1), (2 * i + 1, h, v, 1)], ids, L.LORA_BF16)
            batch = L.KvBatch(q_start, lens, self.table_dev[i], n, max(q_len))
            if ws is None:
                ws = torch.empty(L.lora_kv_attend_workspace_size(self.cache, batch, H), dtype=torch.uint8, device=dev)
            L.lora_kv_write(self.cache, batch, k.view(n, KH, D), v.view(n, KH, D))
            L.lora_kv_attend(self.cache, batch, q.view(n, H, D), out, D ** -0.5, workspace=ws)
            x = x + out.view(n, H * D) @ self.layers[i]["o"]
        return norm(x).float() @ self.head.float()

    def probs(self, logits, temperature):
        if temperature > 0:
            return torch.softmax(logits / temperature, 1)
        return torch.nn.functional.one_hot(logits.argmax(1), self.VOCAB).float()   # the best token, surely

    def uniform(self, n):
        return torch.rand(n, generator=self.gen, device="cuda")

    def prefill(self, temperature):
        lens = [len(t) for t in self.tokens]
        rows = torch.tensor([t for seq in self.tokens for t in seq], device="cuda")
        logits = self.forward(rows, lens, lens, self.LAYERS)[np.cumsum(lens) - 1]
        first = torch.multinomial(self.probs(logits, temperature), 1, generator=self.gen)
        for seq, t in zip(self.tokens, first.flatten().tolist()):
            seq.append(t)

    def step(self, n_drafts, temperature):
        """One step of every request: 1 to n_drafts + 1 new tokens each."""
        n = len(self.tokens)
        cached = [len(t) - 1 for t in self.tokens]
        rows = [torch.tensor([t[-1] for t in self.tokens], device="cuda")]
        draft = []
        for j in range(n_drafts):
            p = self.probs(self.forward(rows[-1], [1] * n, [c + j + 1 for c in cached], self.DRAFT_LAYERS), temperature)
            rows.append(torch.multinomial(p, 1, generator=self.gen).flatten())
            draft.append(p)
        k = n_drafts + 1
        target = self.probs(self.forward(torch.stack(rows, 1).flatten(), [k] * n, [c + k for c in cached],
                                         self.LAYERS), temperature)
        i32 = dict(dtype=torch.int32, device="cuda")
        tokens, n_out = torch.empty(n * k, **i32), torch.empty(n, **i32)
        drafted = torch.stack(rows[1:], 1).flatten().to(torch.int32) if n_drafts else torch.empty(0, **i32)
        q = torch.stack(draft, 1).view(-1, self.VOCAB) if n_drafts else None
        L.lora_spec_verify(torch.arange(0, n * k + 1, k, **i32), drafted, target, q, self.uniform(n * n_drafts),
                           self.uniform(n), tokens, n_out,
                           torch.empty(L.lora_spec_verify_workspace_size(n, self.VOCAB), dtype=torch.uint8,
                                       device="cuda"))
        for seq, new, m in zip(self.tokens, tokens.view(n, k).tolist(), n_out.tolist()):
            seq += new[:m]
            self.accepted += m - 1
        self.proposed += n * n_drafts

    def generate(self, n_tokens, n_drafts, temperature=0.0):
        end = [len(t) + n_tokens for t in self.tokens]
        self.prefill(temperature)
        while any(len(t) < e for t, e in zip(self.tokens, end)):
            self.step(n_drafts, temperature)
        return [t[:e] for t, e in zip(self.tokens, end)]


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(1, keepdim=True) + 1e-5)).to(x.dtype)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--tokens", type=int, default=48)
    ap.add_argument("--temperature", type=float, default=0.0)
    ap.add_argument("--fp8", action="store_true", help="cache in FP8 E4M3")
    a = ap.parse_args()
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, Server.VOCAB, n).tolist() for n in (1, 17, 80, 300)]
    s = Server(prompts, adapters=[0, 3, -1, 5], fp8=a.fp8)
    for i, seq in enumerate(s.generate(a.tokens, a.drafts, a.temperature)):
        print("request %d: %d tokens, the last %s" % (i, len(seq), seq[-6:]))
    print("drafts accepted: %d of %d" % (s.accepted, s.proposed))
    s.close()


if __name__ == "__main__":
    main()
