"""The attention half of a decoder layer, fine-tuned with NF4 base weights and LoRA adapters, on one GPU:

    h = x + residual;  n = rmsnorm(h) w                 (n also kept as an 8-bit checkpoint)
    q, k, v = adapted linears of n                      (one group: they share n and its checkpoint)
    q, k = heads normed and rotated by their positions  (where the block is given a Rope)
    a = attention(q, k, v) over packed sequences        (a also kept as an 8-bit checkpoint)
    out = adapted linear of a

``AttentionBlock.forward`` and ``.backward`` run it with the library's calls; the adapters are updated by
clipped AdamW. ``.decode`` adds one token to a key/value cache, of bf16 tensors or in 4 bits, and attends to it.

Usage: python examples/attention_block.py [--steps N]   (needs the built library and a GPU)
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_nf4_quantised_amd as nf4  # noqa: E402

EPS = 1e-5


class AttentionBlock:
    def __init__(self, hidden=512, heads=8, kv_heads=2, d=64, rank=16, alpha=32.0, seed=0, device="cuda:0", rope=None):
        """rope: a Rope to rotate the query and key heads by, which are normed first; None: neither."""
        g = torch.Generator(device=device).manual_seed(seed)
        self.hidden, self.heads, self.kv_heads, self.d, self.device = hidden, heads, kv_heads, d, device
        self.scale = alpha / rank
        rows = [heads * d, kv_heads * d, kv_heads * d, hidden]            # q, k, v, o
        cols = [hidden, hidden, hidden, heads * d]
        rand = lambda *s: torch.randn(*s, generator=g, device=device)  # noqa: E731
        self.norm_weight = (1 + 0.1 * rand(hidden)).to(torch.bfloat16)
        self.weights = [nf4.quantize_weight(0.04 * rand(n, k)) for n, k in zip(rows, cols)]
        # adapters: fp32 masters, gradients and moments; bf16 copies for the linears. B starts small, not at zero,
        # so that the gradients of A are there from the first step.
        self.masters = [t for n, k in zip(rows, cols) for t in (0.05 * rand(rank, k), 0.01 * rand(n, rank))]
        self.grads = [torch.zeros_like(t) for t in self.masters]
        self.copies = [t.to(torch.bfloat16) for t in self.masters]
        self.plan = nf4.AdamWPlan(self.masters, self.grads, [torch.zeros_like(t) for t in self.masters],
                                  [torch.zeros_like(t) for t in self.masters], self.copies,
                                  nf4.AdamWConfig(lr=2e-3, weight_decay=0.0))
        self.A, self.B = self.copies[0::2], self.copies[1::2]
        self.rope = rope
        if rope is not None:    # the heads' weights are frozen here, as the norm's is
            self.q_weight, self.k_weight = ((1 + 0.1 * rand(d)).to(torch.bfloat16) for _ in range(2))

    def _empty(self, *shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device=self.device)

    def _rotated(self, positions, q, k):
        """q and k as the attention takes them: normed and rotated, or as they are."""
        if self.rope is None:
            return q, k
        qr, kr = torch.empty_like(q), torch.empty_like(k)
        nf4.qlora_rope_fwd(self.rope, positions, q, k, qr, kr, q_weight=self.q_weight, k_weight=self.k_weight, eps=EPS)
        return qr, kr

    def forward(self, x, residual, seqs: nf4.AttnSeqs, positions=None):
        """x, residual: bf16 [tokens, hidden]; positions: int64 [tokens], with a Rope. Returns (out, h) and keeps what
        the backward needs: h, rstd, the 8-bit checkpoints of n and a, u of every linear, q and k before and after they
        are rotated, v, a and lse."""
        M, r = x.shape[0], self.A[0].shape[0]
        h, n = torch.empty_like(x), torch.empty_like(x)
        rstd = self._empty(M, dtype=torch.float32)
        n8 = nf4.empty_act8(M, self.hidden, self.device)
        nf4.qlora_rmsnorm_fwd(x, self.norm_weight, EPS, n, residual=residual, h=h, rstd=rstd, act8=n8)
        u = [self._empty(M, r, dtype=torch.float32) for _ in range(4)]
        qkv = [self._empty(M, w.N) for w in self.weights[:3]]
        nf4.qlora_linear_fwd_group(self.weights[:3], n, self.A[:3], self.B[:3], self.scale, qkv, u[:3])
        q0, k0, v = (t.view(M, -1, self.d) for t in qkv)
        q, k = self._rotated(positions, q0, k0)
        a = torch.empty_like(q)
        lse = self._empty(self.heads, M, dtype=torch.float32)
        nf4.qlora_attn_fwd(seqs, q, k, v, a, lse)
        flat = a.view(M, -1)
        a8 = nf4.empty_act8(M, flat.shape[1], self.device)
        nf4.qlora_act8_pack(flat, a8)
        out = self._empty(M, self.hidden)
        nf4.qlora_linear_fwd(self.weights[3], flat, self.A[3], self.B[3], self.scale, out, u[3])
        self.kept = (seqs, h, rstd, n8, a8, u, q, k, v, a, lse)
        self.turned = (positions, q0, k0)
        return out, h

    def backward(self, dout, dh):
        """dout: gradient of out; dh: what flows into h from the rest of the residual stream. Adds nothing
        up over calls: the adapters' gradients are written. Returns the gradient of x (and of residual)."""
        seqs, h, rstd, n8, a8, u, q, k, v, a, lse = self.kept
        M = dout.shape[0]
        dA, dB = self.grads[0::2], self.grads[1::2]
        da = torch.empty_like(a)
        nf4.qlora_linear_bwd_act8(self.weights[3:], a8, [dout], self.A[3:], self.B[3:], self.scale, u[3:],
                                  [da.view(M, -1)], dA[3:], dB[3:])
        dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
        nf4.qlora_attn_bwd(seqs, q, k, v, a, lse, da, dq, dk, dv)
        if self.rope is not None:   # back through the rotation and the heads' norms, in place
            positions, q0, k0 = self.turned
            nf4.qlora_rope_bwd(self.rope, positions, dq, dk, dq, dk, q=q0, k=k0, q_weight=self.q_weight, k_weight=self.k_weight,
                               eps=EPS)
        dn = [self._empty(M, self.hidden) for _ in range(3)]
        nf4.qlora_linear_bwd_act8(self.weights[:3], n8, [t.view(M, -1) for t in (dq, dk, dv)], self.A[:3], self.B[:3],
                                  self.scale, u[:3], dn, dA[:3], dB[:3])
        dn = (dn[0].float() + dn[1].float() + dn[2].float()).to(torch.bfloat16)
        dx = torch.empty_like(dn)
        nf4.qlora_rmsnorm_bwd(dn, h, self.norm_weight, rstd, dx, dh=dh)   # the norm's weight is frozen
        return dx

    def decode(self, x, residual, k_cache, v_cache, lengths):
        """One new token of every sequence: x, residual [batch, hidden]; caches [batch, room, kv_heads, d], or a pair
        of Kv4 with batch * room tokens, of which sequence i holds lengths[i] tokens; its new keys and values are written
        behind them."""
        batch = x.shape[0]
        four = isinstance(k_cache, nf4.Kv4)
        room = k_cache.shape[0] // batch if four else k_cache.shape[1]
        n = torch.empty_like(x)
        nf4.qlora_rmsnorm_fwd(x, self.norm_weight, EPS, n, residual=residual)
        qkv = [self._empty(batch, w.N) for w in self.weights[:3]]
        nf4.qlora_linear_fwd_group(self.weights[:3], n, self.A[:3], self.B[:3], self.scale, qkv)
        q, k, v = (t.view(batch, -1, self.d) for t in qkv)
        at = torch.tensor(lengths, device=self.device)
        q, k = self._rotated(at, q, k)
        seqs = nf4.AttnSeqs([(i, 1, i * room, n_ + 1) for i, n_ in enumerate(lengths)])
        a = torch.empty_like(q)
        if four:
            nf4.qlora_kv4_write(seqs, k, v, k_cache, v_cache)
            nf4.qlora_attn_kv4_fwd(seqs, q, k_cache, v_cache, a)
        else:
            rows = torch.arange(batch, device=self.device)
            k_cache[rows, at], v_cache[rows, at] = k, v
            nf4.qlora_attn_fwd(seqs, q, k_cache.flatten(0, 1), v_cache.flatten(0, 1), a)
        out = self._empty(batch, self.hidden)
        nf4.qlora_linear_fwd(self.weights[3], a.view(batch, -1), self.A[3], self.B[3], self.scale, out)
        return out


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--steps", type=int, default=40)
    args = p.parse_args()
    block = AttentionBlock(rope=nf4.Rope(64))
    lens = [150, 1, 77, 28]
    M = sum(lens)
    g = torch.Generator(device=block.device).manual_seed(1)
    rand = lambda *s: torch.randn(*s, generator=g, device=block.device).to(torch.bfloat16)  # noqa: E731
    x, residual, target = rand(M, block.hidden), rand(M, block.hidden), rand(M, block.hidden)
    seqs = nf4.AttnSeqs.packed(lens)
    positions = torch.cat([torch.arange(n, device=block.device) for n in lens])
    for step in range(1, args.steps + 1):
        out, h = block.forward(x, residual, seqs, positions)
        diff = out.float() - target.float()
        block.backward((diff / M).to(torch.bfloat16), torch.zeros_like(h))
        block.plan.step(step)
        if step == 1 or step % 10 == 0:
            print(f"step {step:3d}  loss {0.5 * diff.square().sum().item() / M:.3f}", flush=True)
    # the same tokens one by one over a cache give the packed forward's rows; over one in 4 bits, nearly
    n, room = lens[0], 160
    out, _ = block.forward(x, residual, seqs, positions)
    kc = torch.zeros(1, room, block.kv_heads, block.d, dtype=torch.bfloat16, device=block.device)
    k4, v4 = (nf4.empty_kv4(room, block.kv_heads, block.d, block.device) for _ in range(2))
    for name, caches in (("bf16", (kc, torch.zeros_like(kc))), ("4-bit", (k4, v4))):
        one = torch.cat([block.decode(x[i:i + 1], residual[i:i + 1], *caches, [i]) for i in range(n)])
        err = (one.float() - out[:n].float()).norm() / out[:n].float().norm()
        print(f"decoding {n} tokens one by one, {name} cache: {err.item():.2e} from the packed forward", flush=True)


if __name__ == "__main__":
    main()
