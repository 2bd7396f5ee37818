"""A recurrent decoder layer with one decay a head on one GPU: a prompt, then tokens one at a time.

    python examples/linear_layer.py [--prompt 300] [--tokens 16] [--sequences 4] [--check]

The layer is x += W_o linear_attention(W_qkv rms_norm(x)) and x += moe_ffn(rms_norm(x)), with
every matrix in 4-bit blocks: the projections through moe_q4_matvec, the token mixer through
moe_linattn_prefill (prompts) and moe_linattn_step (tokens) on one pool of states, the rest
through moe_ffn_forward_ex with the norm prologue and MOE_RESIDUAL. Random weights of the
Flint-shaped layer (synth.WORKLOADS); the attention's norm is folded into W_qkv's input by torch.

--check runs the same tokens as one longer prompt and compares the outputs.
"""

import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np
import torch

import expert_ffn_decode_gb300 as ffn
from expert_ffn_decode_gb300 import synth

WORKLOAD = "flint_decode_t1"
HEADS, QK_HEADS, DIM = 16, 8, 128


class Layer:
    """One layer's weights and the calls that run it."""

    def __init__(self, seed=0):
        w = self.w = synth.WORKLOADS[WORKLOAD]
        rng = np.random.default_rng(seed)
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
        self.hidden = w["hidden"]
        self.ffn = {k: None if v is None else dev(v) for k, v in synth.make_layer(w, seed).items()}
        self.q_rows, self.v_rows = QK_HEADS * DIM, HEADS * DIM
        rows = 2 * self.q_rows + self.v_rows
        # blocks around 0: Q4_0 of nibbles 0 .. 15 and small scales
        self.w_qkv = dev(synth.any_blocks(rng, synth.Q4_0, rows * self.hidden // 32))
        self.w_out = dev(synth.any_blocks(rng, synth.Q4_0, self.hidden * self.v_rows // 32))
        self.decay = -torch.exp2(-8 * (1 + torch.arange(HEADS)) / HEADS).cuda()
        self.norm = torch.ones(self.hidden, device="cuda")
        self.ws = {}

    def workspace(self, name, nbytes):
        if name not in self.ws or self.ws[name].numel() < nbytes:
            self.ws[name] = torch.zeros(nbytes, dtype=torch.uint8, device="cuda")
        return self.ws[name]

    def __call__(self, x, state, slots, offsets=None):
        """x [tokens][hidden] f32, changed in place. With offsets a batch of prompts, without one
        token of each sequence."""
        st, n, h = torch.cuda.current_stream(), x.shape[0], self.hidden
        # the three projections of all tokens, in one matrix and one buffer
        xn = torch.nn.functional.rms_norm(x, (h,)).to(torch.bfloat16)
        rows = 2 * self.q_rows + self.v_rows
        qkv = torch.empty(n, rows, dtype=torch.bfloat16, device="cuda")
        cfg = ffn.make_matvec_cfg(rows, h, n, qtype=ffn.MOE_Q4_0, x_type=ffn.MOE_BF16, y_type=ffn.MOE_BF16)
        ffn.check(ffn.moe_q4_matvec(xn, self.w_qkv, None, None, None, cfg, qkv, st))
        q, k, v = qkv.split([self.q_rows, self.q_rows, self.v_rows], 1)
        k.copy_(torch.nn.functional.normalize(k.float().unflatten(1, (QK_HEADS, DIM)), dim=-1).flatten(1))
        # the token mixer, on views of that buffer
        o = torch.empty(n, self.v_rows, dtype=torch.bfloat16, device="cuda")
        cfg = ffn.make_linattn_cfg(slots.numel(), n, HEADS, DIM, DIM, n_qk_heads=QK_HEADS, n_states=state.shape[0],
                                   flags=0 if offsets is None else ffn.MOE_FRESH_STATE, q_stride=rows, k_stride=rows,
                                   v_stride=rows)
        if offsets is None:
            ffn.check(ffn.moe_linattn_step(q, k, v, self.decay, slots, cfg, state, o, st))
        else:
            ws = self.workspace("attention", ffn.moe_linattn_workspace_size(cfg))
            ffn.check(ffn.moe_linattn_prefill(q, k, v, self.decay, offsets, slots, cfg, state, o, ws, ws.numel(), st))
        # the output projection, added into the residual stream
        cfg = ffn.make_matvec_cfg(h, self.v_rows, n, qtype=ffn.MOE_Q4_0, x_type=ffn.MOE_BF16, flags=ffn.MOE_ACCUMULATE)
        ffn.check(ffn.moe_q4_matvec(o, self.w_out, None, None, None, cfg, x, st))
        # x + moe_ffn(rms_norm(x))
        cfg = ffn.make_cfg(**{**self.w, "n_tokens": n, "flags": ffn.MOE_RESIDUAL}, rms_eps=1e-6, ffn_norm=self.norm)
        ws = self.workspace("ffn", ffn.moe_workspace_size(cfg))
        out = torch.empty_like(x)
        ffn.check(ffn.moe_ffn_forward_ex(x, self.ffn["router_w"], self.ffn["bias"], self.ffn["expert_blocks"],
                                         self.ffn["shared_blocks"], cfg, out, ws, ws.numel(), st))
        return x.copy_(out)

    def check_status(self):
        for ws in self.ws.values():
            ffn.check(ffn.moe_workspace_status(ws, torch.cuda.current_stream()))


def run(prompt=300, tokens=16, sequences=4, check=False, seed=0):
    """Returns (tokens a second of the decoded part, worst relative difference or None)."""
    layer = Layer(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    lens = [max(1, prompt - 37 * i) for i in range(sequences)]
    total = [n + tokens for n in lens]
    xs = [torch.randn(n, layer.hidden, generator=gen, device="cuda") for n in total]
    slots = torch.randperm(sequences + 2, generator=gen, device="cuda")[:sequences].to(torch.int32)
    state = torch.zeros(sequences + 2, HEADS, DIM, DIM, device="cuda")

    def offsets(n):
        return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device="cuda")

    layer(torch.cat([x[:n] for x, n in zip(xs, lens)]), state, slots, offsets(lens))
    outs = []
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for t in range(tokens):
        if t == min(2, tokens - 1):
            start.record()
        outs.append(layer(torch.stack([x[n + t] for x, n in zip(xs, lens)]), state, slots))
    stop.record()
    torch.cuda.synchronize()
    layer.check_status()
    rate = sequences * (tokens - min(2, tokens - 1)) / (start.elapsed_time(stop) * 1e-3)
    worst = None
    if check:
        full = layer(torch.cat(xs), torch.zeros_like(state), slots, offsets(total))
        layer.check_status()
        worst = 0.0
        for b, n in enumerate(lens):
            want = full[sum(total[:b]) + n:sum(total[:b + 1])]
            got = torch.stack([o[b] for o in outs])
            worst = max(worst, float((got - want).norm() / want.norm()))
    return rate, worst


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--sequences", type=int, default=4)
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args()
    rate, worst = run(a.prompt, a.tokens, a.sequences, a.check)
    print(f"{a.sequences} sequences, prompts up to {a.prompt}, {a.tokens} tokens each: {rate:.0f} tokens/s decoded")
    if worst is not None:
        print(f"against one longer prompt: worst relative difference {worst:.2e}")
        assert math.isfinite(worst) and worst < 2e-2


if __name__ == "__main__":
    main()
