"""Sequence-level distillation in miniature: a teacher's beam search writes the targets, the fused loss trains on them.

A small random decoder (embedding, layers of attention and a gated product, a vocabulary head)
generates with beams over a paged key-value cache: every decoding call of the package is used the
way a decoding loop uses it, with buffers and workspaces kept across steps and nothing read back
until the search ends.  The hypotheses then become the targets of lossk_ce_fwd_bwd, with the head
as its weight.

    python examples/beam_decode.py [--beams 4] [--steps 24]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import output_projection_cross_gb300 as L  # noqa: E402


class Decoder:
    """Random weights of a small decoder; attention is left to the caller."""

    def __init__(self, vocab=1003, d=128, layers=2, q_heads=8, kv_heads=2, head_dim=32, seed=0):
        self.vocab, self.d, self.layers = vocab, d, layers
        self.hq, self.kv, self.hd = q_heads, kv_heads, head_dim
        g = torch.Generator().manual_seed(seed)

        def w(rows, cols, scale=1.0):
            return (torch.randn(rows, cols, generator=g) * scale / cols ** 0.5).cuda().bfloat16()
        self.embed = w(vocab, d, d ** 0.5)
        self.qkv = [w((q_heads + 2 * kv_heads) * head_dim, d, 2.0) for _ in range(layers)]
        self.out = [w(d, q_heads * head_dim) for _ in range(layers)]
        self.up, self.down = [w(2 * d, d) for _ in range(layers)], [w(d, d) for _ in range(layers)]
        self.head = w(vocab, d, 3.0)

    def run(self, tokens, attend):
        """Hidden rows of one token per sequence; attend(layer, q, k, v) -> [n, hq, hd]."""
        x = self.embed[tokens]
        for i in range(self.layers):
            qkv = (self.norm(x) @ self.qkv[i].T).view(-1, self.hq + 2 * self.kv, self.hd)
            q, k, v = qkv[:, :self.hq], qkv[:, self.hq:self.hq + self.kv], qkv[:, self.hq + self.kv:]
            x = x + attend(i, q, k, v).flatten(1) @ self.out[i].T
            a, b = (self.norm(x) @ self.up[i].T).chunk(2, 1)
            x = x + (torch.nn.functional.silu(a) * b) @ self.down[i].T
        return self.norm(x)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).bfloat16()


class BeamSearch:
    """Beams over a paged cache.  The cache holds `planes` = 2 per layer (keys, values)."""

    def __init__(self, model, prompts, beams, steps, end_token, page=16, length_alpha=0.0):
        self.m, self.beams, self.end, self.page, self.alpha = model, beams, end_token, page, length_alpha
        self.batch, n = prompts.shape
        self.prompts = prompts
        rows = self.batch * beams
        self.max_pages = -(-(n + steps) // page)
        n_pages = self.batch * (-(-n // page)) + rows * (-(-steps // page) + 2)
        self.pool = torch.empty((2 * model.layers, n_pages, page, model.kv, model.hd), device="cuda", dtype=torch.bfloat16)
        self.ref = torch.zeros(n_pages, device="cuda", dtype=torch.int32)
        self.table = torch.full((self.batch, self.max_pages), -1, device="cuda", dtype=torch.int32)
        self.lens = torch.zeros(self.batch, device="cuda", dtype=torch.int32)
        self.ws_cache = L.decode_workspace(L.KIND_CACHE, rows, n_pages)
        self.ws_attn = L.decode_workspace(L.KIND_PAGED_ATTN, rows, model.hq, model.kv, model.hd)
        self.ws_beam = L.decode_workspace(L.KIND_BEAM_SELECT, self.batch, beams, model.vocab, beams)
        self.history = torch.zeros((self.batch, beams, steps), device="cuda", dtype=torch.int64)

    def step(self, tokens, share):
        """One token per sequence through the model and into the cache; returns the hidden rows."""
        L.lossk_cache_reserve(self.table, self.lens, self.ref, self.pool, self.page, ws=self.ws_cache)
        after = self.lens + 1

        def attend(i, q, k, v):
            pages = self.pool[2 * i], self.pool[2 * i + 1]
            L.lossk_cache_write(k, v, *pages, self.table, self.lens, ws=self.ws_cache)
            return L.lossk_paged_attn(q, *pages, self.table, after, share=share, ws=self.ws_attn)
        h = self.m.run(tokens, attend)
        self.lens = after
        return h

    def run(self, steps):
        """(tokens [batch, beams, steps], lengths, scores), best first."""
        for i in range(self.prompts.shape[1]):
            h = self.step(self.prompts[:, i], 1)
        # every beam starts as its prompt; all but the first are dead until the first selection
        first = torch.zeros((self.batch, self.beams), device="cuda", dtype=torch.int32)
        self.fork(first)
        h = h.repeat_interleave(self.beams, 0)
        score = torch.full((self.batch, self.beams), -float("inf"), device="cuda")
        score[:, 0] = 0.0
        finished = torch.zeros((self.batch, self.beams), device="cuda", dtype=torch.uint8)
        length = torch.zeros((self.batch, self.beams), device="cuda", dtype=torch.int32)
        for t in range(steps):
            o = L.lossk_beam_select(h @ self.m.head.T, score, self.beams, finished=finished, end_token=self.end,
                                    lengths=length, length_alpha=self.alpha, ws=self.ws_beam)
            score, finished, length = o["score"], o["finished"], o["length"]
            self.history = L.lossk_beam_gather(self.history, o["parent"], ws=self.ws_cache)
            self.history[:, :, t] = o["token"]
            if t + 1 < steps:
                self.fork(o["parent"])
                h = self.step(o["token"].flatten().clamp(min=0), self.beams)
        for ws in (self.ws_cache, self.ws_attn, self.ws_beam):
            status = L.lossk_device_status(ws)
            if status != 580:
                raise L.LosskError(status, "beam search")
        L.lossk_cache_free(self.table, self.lens, self.ref, self.page, ws=self.ws_cache)
        return self.history, length, score

    def fork(self, parent):
        self.table, self.lens = L.lossk_cache_fork(parent, self.table, self.lens, self.ref, self.page, ws=self.ws_cache)


def plain_log_probs(model, tokens, n_prompt):
    """log p of each token after the prompt, one sequence at a time with its whole history at hand."""
    past = [([], []) for _ in range(model.layers)]
    logp = []

    def attend(i, q, k, v):
        past[i][0].append(k[0])
        past[i][1].append(v[0])
        kk = torch.stack(past[i][0]).float().repeat_interleave(model.hq // model.kv, 1)
        vv = torch.stack(past[i][1]).float().repeat_interleave(model.hq // model.kv, 1)
        p = torch.softmax(torch.einsum("hd,nhd->hn", q[0].float(), kk) * model.hd ** -0.5, -1)
        return torch.einsum("hn,nhd->hd", p, vv)[None].bfloat16()
    for j in range(len(tokens) - 1):
        h = model.run(tokens[j:j + 1], attend)
        if j + 1 >= n_prompt:
            logp.append(torch.log_softmax((h @ model.head.T).double(), -1)[0, tokens[j + 1]])
    return torch.stack(logp)


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--beams", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--batch", type=int, default=8)
    args = ap.parse_args()
    teacher = Decoder(seed=0)
    prompts = torch.randint(0, teacher.vocab, (args.batch, 21), generator=torch.Generator().manual_seed(1)).cuda()
    search = BeamSearch(teacher, prompts, args.beams, args.steps, end_token=5, length_alpha=0.6)
    tokens, length, score = search.run(args.steps)
    best = tokens[:, 0]
    print("best hypotheses:", best[:, :8].tolist())
    print("scores", [round(x, 3) for x in score[:, 0].tolist()], "lengths", length[:, 0].tolist())

    # the student's loss on the teacher's sequences: rows of hidden state against the fused head
    student = Decoder(seed=2)
    hidden = student.norm(student.embed[best.flatten()])
    mask = torch.arange(args.steps, device="cuda")[None] < length[:, :1]
    step = L.lossk_ce_fwd_bwd(hidden.contiguous(), student.head, best.flatten().clamp(min=0),
                              loss_mask=mask.flatten().to(torch.uint8).contiguous(), chunk=64)
    print("student's loss on them: %.4f" % step["scalars"][0].item())


if __name__ == "__main__":
    main()
