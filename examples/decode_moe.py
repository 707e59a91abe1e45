"""A small decoder of MoE blocks, one CUDA graph replay per step.

Each block adds to a token's state what its routed experts give it
(moe_layer_few, FP8 or 4-bit expert weights) and what a shared expert does: 4-bit
(moe_matvec_w4 twice) or in bf16 (moe_gated, and moe_linear onto the routed output); a
4-bit vocabulary projection picks the next token.
There is no attention: the example shows the decoding calls together, with
random weights.

    python examples/decode_moe.py --tokens 8 --steps 32 --weights w4
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import combine_counting_sort_gb300 as moe  # noqa: E402


def quantise_w4(W, group=128):
    """bf16 [E, N, K] -> the laid-out 4-bit matrices."""
    packed = torch.empty(moe.w4_packed_shape(*W.shape, group), dtype=torch.uint8, device=W.device)
    moe.moe_quant_weights_w4(W, group, packed)
    return packed


def quantise_fp8(W):
    """bf16 [E, N, K] -> e4m3 codes and their 128 x 128 scales."""
    E, N, K = W.shape
    codes = torch.empty(E, N, K, dtype=torch.uint8, device=W.device)
    scale = torch.empty(E, N // 128, K // 128, device=W.device)
    moe.moe_quant_weights(W, codes, scale)
    return codes, scale


class Block:
    def __init__(self, gen, T, H, F, E, k, weights, shared, group, status):
        def rand(*shape):
            return (torch.randn(*shape, generator=gen, device="cuda") * shape[-1] ** -0.5).to(torch.bfloat16)

        self.k, self.group, self.status = k, group, status
        self.router = rand(E, H)
        if weights == "fp8":
            (self.W1, self.s1), (self.W2, self.s2) = quantise_fp8(rand(E, 2 * F, H)), quantise_fp8(rand(E, H, F))
        else:
            self.W1, self.W2, self.s1, self.s2 = quantise_w4(rand(E, 2 * F, H), group), quantise_w4(rand(E, H, F), group), None, None
        self.layer_group = 0 if weights == "fp8" else group
        self.shared = shared
        up, down = rand(1, 2 * F, H), rand(1, H, F)
        self.shared_up, self.shared_down = (up[0], down[0]) if shared == "bf16" else (quantise_w4(up, group)[0], quantise_w4(down, group)[0])
        self.act = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
        # what a call writes, and its workspace: made once
        self.ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
        self.w = torch.empty(T, k, device="cuda")
        self.routed = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        self.up = torch.empty(T, 2 * F, dtype=torch.bfloat16, device="cuda")
        self.down = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        self.ws = torch.zeros(moe.moe_layer_few_ws_bytes(T, k, E, H, F), dtype=torch.uint8, device="cuda")

    def __call__(self, x):
        h = torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(torch.bfloat16)
        moe.moe_layer_few(h, self.W1, self.s1, self.W2, self.s2, self.ids, self.w, self.routed, self.ws, self.status,
                          router=self.router, group=self.layer_group)
        if self.shared == "bf16":
            moe.moe_gated(h, self.shared_up, self.act, self.status)
            moe.moe_linear(self.act, self.shared_down, self.down, self.status, residual=self.routed)
            return x + self.down
        moe.moe_matvec_w4(h, self.shared_up, self.group, self.up, self.status)
        gate, up = self.up.float().chunk(2, -1)
        moe.moe_matvec_w4((torch.nn.functional.silu(gate) * up).to(torch.bfloat16), self.shared_down, self.group, self.down, self.status)
        return x + self.routed + self.down


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=8, help="sequences decoded together (1 to 64)")
    ap.add_argument("--steps", type=int, default=32)
    ap.add_argument("--blocks", type=int, default=2)
    ap.add_argument("--weights", choices=("fp8", "w4"), default="w4")
    ap.add_argument("--shared", choices=("w4", "bf16"), default="w4", help="the shared expert's weights")
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--ffn", type=int, default=1024)
    ap.add_argument("--experts", type=int, default=64)
    ap.add_argument("--topk", type=int, default=8)
    ap.add_argument("--vocab", type=int, default=32000)
    a = ap.parse_args()
    gen = torch.Generator(device="cuda").manual_seed(0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    blocks = [Block(gen, a.tokens, a.hidden, a.ffn, a.experts, a.topk, a.weights, a.shared, 128, status) for _ in range(a.blocks)]
    embedding = torch.randn(a.vocab, a.hidden, generator=gen, device="cuda").to(torch.bfloat16)
    vocabulary = quantise_w4((torch.randn(1, a.vocab, a.hidden, generator=gen, device="cuda") * a.hidden ** -0.5).to(torch.bfloat16))[0]
    logits = torch.empty(a.tokens, a.vocab, dtype=torch.bfloat16, device="cuda")
    token = torch.randint(0, a.vocab, (a.tokens,), generator=gen, device="cuda")

    def step():
        x = embedding[token]
        for block in blocks:
            x = block(x)
        moe.moe_matvec_w4(torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(torch.bfloat16), vocabulary, 128, logits, status)
        token.copy_(logits.argmax(-1))

    side = torch.cuda.Stream()   # warm up off the default stream, then capture
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        start = token.clone()
        step()
        eager = token.clone()
        token.copy_(start)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    token.copy_(start)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(token, eager), "the replayed step differs from the eager one"
    out = []
    t = time.perf_counter()
    for _ in range(a.steps):
        graph.replay()
        out.append(token.clone())
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    if status.item():
        raise SystemExit(moe.status_string(status.item()))
    print(f"{a.weights}: {a.tokens} sequences x {a.steps} steps of {a.blocks} blocks, {a.tokens * a.steps / t:.0f} tokens/s, "
          f"{t / a.steps * 1e6:.0f} us a step; first sequence: {torch.stack(out)[:8, 0].tolist()}")


if __name__ == "__main__":
    main()
