"""The attention half of a decoder layer, served to a batch that mixes adapters.

One layer, as a server runs it each step, over static buffers with the valid token count in device
memory:

    z, x, (x8)  = lora_add_rmsnorm(h, residual)         the norm in front of the layer's product
    y           = x W_qkv                               the base product (a library GEMM)
    y          += LoRA_qkv(x)                           prepare once a batch, then shrink_expand
    q, cache   <- lora_kv4_append(rotate(q), k, v)      rotation, 4-bit pages
    o           = lora_kv4_attention(q, cache)          decode and prefill rows in one call
    h           = o W_o + LoRA_o(o)

Run it (on a GPU): ``python examples/decoder_layer.py`` prefills a few prompts in chunks, decodes a
few tokens, and compares the layer's output with the same steps in plain PyTorch.
"""
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from gathered_rank_gemm_gb300 import binding as B  # noqa: E402

K_SCALE, V_SCALE = 1.0 / 32, 1.0 / 32


def rope_table(positions, dim, device):
    """fp32 [positions][dim]: the cosines, then the sines, of each position's angles."""
    angle = torch.arange(positions, device=device).float()[:, None] / 10000.0 ** (
        torch.arange(0, dim, 2, device=device).float() / dim)
    return torch.cat([angle.cos(), angle.sin()], 1)


class Layer:
    """Weights, adapters and static buffers of one layer."""

    def __init__(self, hidden=512, q_heads=8, kv_heads=2, head_dim=64, max_tokens=256, max_seqs=8, max_loras=4,
                 rank=16, page_size=16, num_pages=64, device="cuda", seed=0):
        g = torch.Generator(device).manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=g, device=device) * std).bfloat16()

        self.q_heads, self.kv_heads, self.d, self.page_size = q_heads, kv_heads, head_dim, page_size
        self.widths = (q_heads * head_dim, kv_heads * head_dim, kv_heads * head_dim)
        self.norm = 1 + normal(hidden, std=0.1)
        self.w_qkv = normal(hidden, sum(self.widths), std=hidden ** -0.5)
        self.w_o = normal(q_heads * head_dim, hidden, std=(q_heads * head_dim) ** -0.5)
        self.a_qkv = [normal(max_loras, rank, hidden, std=0.05) for _ in self.widths]
        self.b_qkv = [normal(max_loras, rank, w, std=0.05) for w in self.widths]
        self.a_o = [normal(max_loras, rank, q_heads * head_dim, std=0.05)]
        self.b_o = [normal(max_loras, rank, hidden, std=0.05)]
        self.rope = rope_table(4096, head_dim, device)
        self.cache = torch.zeros(num_pages, kv_heads, page_size // 16, 18 * head_dim, dtype=torch.uint8, device=device)

        def buffer(*shape, dtype=torch.bfloat16):
            return torch.zeros(*shape, dtype=dtype, device=device)

        self.x, self.x8 = buffer(max_tokens, hidden), buffer(max_tokens, hidden, dtype=torch.float8_e4m3fn)
        self.x8_scale = buffer(max_tokens, 1, dtype=torch.float32)
        self.y = buffer(max_tokens, sum(self.widths))
        self.o = buffer(max_tokens, q_heads, head_dim)
        self.held = [buffer(max_tokens, kv_heads, head_dim) for _ in range(2)]
        self.u = buffer(3, max_tokens, rank, dtype=torch.float32)
        self.u_o = buffer(1, max_tokens, rank, dtype=torch.float32)
        self.n = buffer(1, dtype=torch.int32)
        self.meta = B.LoraMetadata(max_tokens, max_loras, device, workspace_bytes=max(
            B.lora_shrink_expand_workspace_size(max_tokens, max_loras, hidden, self.widths, rank),
            B.lora_shrink_expand_workspace_size(max_tokens, max_loras, q_heads * head_dim, (hidden,), rank)))
        self.workspace = buffer(B.lora_kv4_attention_workspace_size(max_seqs, max_tokens, max_tokens, q_heads, kv_heads,
                                                                    head_dim), dtype=torch.uint8)
        self.status = buffer(4, dtype=torch.int32)

    def step(self, h, residual, mapping, positions, slots, q_start, kv_len, page_table, max_q_len):
        """h, residual [max_tokens][hidden] -> the layer's output; residual takes h + residual."""
        B.lora_add_rmsnorm(h, self.norm, 1e-5, self.n, residual=residual, residual_out=residual, y=self.x, y8=self.x8,
                           y8_scale=self.x8_scale, status=self.status)
        self.meta.prepare(mapping, self.n)
        torch.matmul(self.x, self.w_qkv, out=self.y)
        self.meta.shrink_expand(self.x, self.a_qkv, self.b_qkv, 1.0, self.u, self.y)
        q, k, v = (a.unflatten(1, (-1, self.d)) for a in self.y.split(self.widths, 1))
        B.lora_kv4_append(self.cache, k, v, slots, self.n, q=q, q_out=q, positions=positions, rope=self.rope,
                          k_scale=K_SCALE, v_scale=V_SCALE, k_held=self.held[0], v_held=self.held[1],
                          status=self.status)
        B.lora_kv4_attention(self.cache, q, self.o, q_start, kv_len, page_table, max_q_len, 1 / math.sqrt(self.d),
                             self.workspace, k_scale=K_SCALE, v_scale=V_SCALE, status=self.status)
        o = self.o.flatten(1)
        out = o @ self.w_o
        self.meta.shrink_expand(o, self.a_o, self.b_o, 1.0, self.u_o, out)
        return out


def serve(layer, prompts, chunk, new_tokens, seed=1):
    """Prefills the prompts `chunk` tokens a step, then decodes; yields each step's inputs (as plain
    PyTorch needs them) with the layer's output."""
    dev = layer.cache.device
    g = torch.Generator(dev).manual_seed(seed)
    rows, hidden = layer.x.shape
    seqs = len(prompts)
    per = -(-(max(prompts) + new_tokens) // layer.page_size)
    order = torch.randperm(layer.cache.shape[0], generator=torch.Generator().manual_seed(seed))[:seqs * per]
    table = order.view(seqs, per).to(dev, torch.int32)
    loras = [i % (layer.meta.max_loras + 1) - 1 for i in range(seqs)]  # adapters, and none
    done = [0] * seqs
    total = [p + new_tokens for p in prompts]
    i32 = dict(dtype=torch.int32, device=dev)
    while min(t - d for t, d in zip(total, done)) > 0 or any(d < t for d, t in zip(done, total)):
        take = [min(chunk, p - d) if d < p else min(1, t - d) for d, p, t in zip(done, prompts, total)]
        start, pos, slot, lora = [0], [], [], []
        for b, m in enumerate(take):
            at = torch.arange(done[b], done[b] + m)
            pos.append(at)
            slot.append(order.view(seqs, per)[b][at // layer.page_size] * layer.page_size + at % layer.page_size)
            lora += [loras[b]] * m
            start.append(start[-1] + m)
        n = start[-1]
        pad = rows - n

        def column(v, fill):
            return torch.cat([v, torch.full((pad,), fill)]).to(**i32)

        h = torch.randn(rows, hidden, generator=g, device=dev).bfloat16()
        residual = torch.randn(rows, hidden, generator=g, device=dev).bfloat16()
        layer.n.fill_(n)
        kv = torch.tensor([d + m for d, m in zip(done, take)], **i32)
        before = residual.clone()
        out = layer.step(h, residual, column(torch.tensor(lora), -1), column(torch.cat(pos), 0),
                         column(torch.cat(slot), -1), torch.tensor(start, **i32), kv, table, max(take))
        yield dict(h=h[:n], residual=before[:n], residual_out=residual[:n], loras=lora, positions=torch.cat(pos),
                   start=start, done=list(done), out=out[:n], x=layer.x[:n].clone(),
                   held=[a[:n].clone() for a in layer.held])
        done = [d + m for d, m in zip(done, take)]


def plain_step(layer, s, history):
    """The same step in plain PyTorch (fp32), over the values that the cache holds."""
    z = s["h"].float() + s["residual"].float()
    x = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-5) * layer.norm.float()

    def product(x, w, a, b):
        y = x @ w.float()
        parts = list(y.split([t.shape[2] for t in b], 1))
        for i, (aa, bb) in enumerate(zip(a, b)):
            for t, lora in enumerate(s["loras"]):
                if lora >= 0:
                    parts[i][t] += (x[t] @ aa[lora].float().T) @ bb[lora].float()
        return parts

    q = product(x, layer.w_qkv, layer.a_qkv, layer.b_qkv)[0].unflatten(1, (-1, layer.d))
    cos, sin = layer.rope[s["positions"].to(q.device)].chunk(2, -1)
    lo, hi = q.chunk(2, -1)
    q = torch.cat([lo * cos[:, None] - hi * sin[:, None], hi * cos[:, None] + lo * sin[:, None]], -1)
    o = torch.empty_like(q)
    group = layer.q_heads // layer.kv_heads
    for b, done in enumerate(s["done"]):
        rows = slice(s["start"][b], s["start"][b + 1])
        history[b] = [torch.cat([old, new[rows].float()]) for old, new in zip(history[b], s["held"])]
        k, v = (t.repeat_interleave(group, 1) for t in history[b])
        score = torch.einsum("rhd,khd->hrk", q[rows], k) / math.sqrt(layer.d)
        hidden = torch.arange(k.shape[0], device=q.device) > torch.arange(
            done, done + rows.stop - rows.start, device=q.device)[:, None]
        p = torch.softmax(score.masked_fill(hidden, -math.inf), -1)
        o[rows] = torch.einsum("hrk,khd->rhd", p, v)
    return torch.cat(product(o.flatten(1), layer.w_o, layer.a_o, layer.b_o), 1)


def check(layer, prompts, chunk, new_tokens):
    """Largest relative error (2-norms) of the layer's steps against the plain ones."""
    history = [[torch.zeros(0, layer.kv_heads, layer.d, device=layer.cache.device)] * 2 for _ in prompts]
    worst, steps = 0.0, 0
    for s in serve(layer, prompts, chunk, new_tokens):
        want = plain_step(layer, s, history)
        worst = max(worst, float((s["out"].float() - want).norm() / want.norm()))
        steps += 1
    return worst, steps, B.lora_read_status(layer.status)


def main():
    layer = Layer()
    worst, steps, status = check(layer, prompts=[37, 100, 5, 64], chunk=48, new_tokens=6)
    print(f"{steps} steps, largest relative error against plain PyTorch {worst:.2e}, status {status}")


if __name__ == "__main__":
    main()
