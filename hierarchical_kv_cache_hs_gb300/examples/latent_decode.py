"""A latent-attention layer served from the hierarchical cache, end to end.

For a few requests: the prompt's cache rows are written by the norm (8-bit rows
of 592 bytes, or bf16 rows of 1152), the prompt's attention runs in the expanded
form over them, and the rows go to the pinned host pool.  Each decode step then
appends its token's row to the device tail, resolves the step's top-k indices
(missing rows come from the host pool into the hot buffer) and attends over the
slots in the absorbed form.  Weights are random; the indices are recent tokens
plus random ones, in the indexer's place.

    python -m hierarchical_kv_cache_hs_gb300.examples.latent_decode [--bf16]

prints how far each part is from the same arithmetic in 64 bits over the same rows.
"""
from __future__ import annotations

import sys

import numpy as np
import torch

from .. import hs

B, H, K = 4, 16, 256              # requests, heads, indices a step
PROMPT, TAIL, SLOTS, STEPS = 1792, 256, 512, 6
HIDDEN, EPS = 1024, 1e-6
LATENT, ROPE, ROW, HEAD = hs.HS_LATENT_DIM, hs.HS_ROPE_DIM, hs.HS_ROW_DIM, hs.HS_HEAD_DIM
SCALE = (HEAD + ROPE) ** -0.5


class Layer:
    """Weights of one layer and the calls that a serving loop makes."""

    def __init__(self, e4m3: bool, gen: torch.Generator):
        def weight(*shape):
            w = torch.randn(shape, generator=gen, device="cuda") * shape[-1] ** -0.5
            return w.to(torch.bfloat16)
        self.e4m3 = e4m3
        self.norm_in = torch.ones(HIDDEN, dtype=torch.bfloat16, device="cuda")
        self.norm_latent = torch.ones(LATENT, dtype=torch.bfloat16, device="cuda")
        self.w_q = weight(H * (HEAD + ROPE), HIDDEN)
        self.w_kv = weight(ROW, HIDDEN)
        self.w_uk, self.w_uv = weight(H, HEAD, LATENT), weight(H, HEAD, LATENT)
        self.row_bytes = hs.HS_ROW8_BYTES if e4m3 else 2 * ROW
        self.row_format = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT

    def project(self, x, residual):
        """Queries [n][H][192] and cache rows [n][row_bytes] of tokens with inputs x."""
        y = torch.empty_like(x)
        hs.hs_rms_norm(x, self.norm_in, y, EPS, residual=residual, residual_out=residual,
                       stream=torch.cuda.current_stream())
        q = (y @ self.w_q.t()).view(-1, H, HEAD + ROPE)
        kv = y @ self.w_kv.t()       # the rotation of the last 64 channels belongs here
        rows = torch.zeros((x.shape[0], self.row_bytes), dtype=torch.uint8, device="cuda")
        if self.e4m3:
            hs.hs_rms_norm(kv, self.norm_latent, rows[:, :ROW], EPS, carry=ROPE,
                           scales=rows[:, ROW:ROW + 4].view(torch.float32),
                           stream=torch.cuda.current_stream())
        else:
            hs.hs_rms_norm(kv, self.norm_latent, rows.view(torch.bfloat16), EPS, carry=ROPE,
                           stream=torch.cuda.current_stream())
        return q, rows

    def absorb(self, q):
        """Queries with the key projection absorbed: [n][H][576]."""
        latent = torch.einsum("nhd,hdl->nhl", q[..., :HEAD], self.w_uk)
        return torch.cat([latent, q[..., HEAD:]], -1)

    def rows64(self, rows):
        if not self.e4m3:
            return rows.view(torch.bfloat16).double()
        scale = rows[..., ROW:ROW + 4].contiguous().view(torch.float32).double()
        return rows[..., :ROW].contiguous().view(torch.float8_e4m3fn).double() * scale


def _off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


def run(e4m3: bool = True, seed: int = 0) -> dict:
    """One prompt and STEPS decode steps; the relative errors of both attentions."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    layer = Layer(e4m3, gen)
    stream = torch.cuda.current_stream()

    def hidden(n):
        return torch.randn((n, HIDDEN), generator=gen, device="cuda").to(torch.bfloat16)

    # The prompts, taken together.
    n = B * PROMPT
    q, rows = layer.project(hidden(n), hidden(n))
    start = torch.arange(B + 1, device="cuda", dtype=torch.int32) * PROMPT
    out = torch.empty((n, H, HEAD), dtype=torch.bfloat16, device="cuda")
    space = torch.empty(hs.hs_latent_prefill_workspace(n, H), dtype=torch.uint8, device="cuda")
    hs.hs_workspace_clear(space)
    hs.hs_latent_prefill(q, rows, layer.w_uk, layer.w_uv, start, start, out, SCALE,
                         row_format=layer.row_format, workspace=space, stream=stream)
    late = hs.hs_workspace_error(space)
    wide = layer.rows64(rows.view(B, PROMPT, -1))
    k0 = torch.cat([wide[0, :, :LATENT] @ layer.w_uk[0].double().t(), wide[0, :, LATENT:]], 1)
    s = SCALE * (q[:PROMPT, 0].double() @ k0.t())
    s = s.masked_fill(~torch.ones_like(s, dtype=torch.bool).tril(), -torch.inf)
    prompt = _off(out[:PROMPT, 0], torch.softmax(s, -1) @ (wide[0, :, :LATENT] @ layer.w_uv[0].double().t()))

    # Decode over the hierarchical cache: prompt rows in the host pool, new ones in the device tail.
    cap = PROMPT + TAIL
    worst = 0.0
    with hs.Handle(B, cap, layer.row_bytes, SLOTS, -(-PROMPT // SLOTS), TAIL) as h:
        h.host_pool()[:, :PROMPT] = rows.view(B, PROMPT, -1).cpu().numpy()
        hs.hs_set_lengths(h.h, np.full(B, PROMPT, dtype=np.int32))
        slots = torch.empty((B, 1, K), dtype=torch.int32, device="cuda")
        out = torch.empty((B, 1, H, LATENT), dtype=torch.bfloat16, device="cuda")
        space = torch.empty(hs.hs_latent_attend_workspace(B, 1, H, K), dtype=torch.uint8, device="cuda")
        hs.hs_workspace_clear(space)
        every = layer.rows64(rows.view(B, PROMPT, -1))
        for step in range(STEPS):
            q, row = layer.project(hidden(B), hidden(B))
            hs.hs_append(h.h, row, stream)
            every = torch.cat([every, layer.rows64(row)[:, None]], 1)
            length = PROMPT + step + 1
            picked = np.stack([np.concatenate([
                np.arange(length - 64, length), rng.choice(length - 64, K - 64, replace=False)])
                for _ in range(B)]).astype(np.int32)
            topk = torch.from_numpy(picked).cuda()
            h.resolve(topk, K, slots, stream)
            qa = layer.absorb(q)[:, None]
            h.attend(qa, slots, out, SCALE, row_format=layer.row_format, workspace=space, stream=stream)
            result = torch.einsum("bhl,hdl->bhd", out[:, 0], layer.w_uv)  # the value projection
            assert result.shape == (B, H, HEAD)
            k = torch.gather(every, 1, topk.long()[..., None].expand(-1, -1, ROW))
            p = torch.softmax(SCALE * torch.einsum("bhc,bkc->bhk", qa[:, 0].double(), k), -1)
            worst = max(worst, _off(out[:, 0], torch.einsum("bhk,bkl->bhl", p, k[..., :LATENT])))
        stats = h.stats()
        late |= hs.hs_workspace_error(space)
    return {"prompt": prompt, "decode": worst, "misses": stats["misses"], "hits": stats["hits"],
            "errors": stats["err_bits"], "waits_ran_out": late}


if __name__ == "__main__":
    got = run(e4m3="--bf16" not in sys.argv[1:])
    if got["errors"] or got["waits_ran_out"]:
        sys.exit("device errors %#x, waits that ran out %d" % (got["errors"], got["waits_ran_out"]))
    print("prompt attention: %.2e off 64 bits; decode steps: %.2e; %d misses, %d hits" %
          (got["prompt"], got["decode"], got["misses"], got["hits"]))
