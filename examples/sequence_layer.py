"""A sequence layer on the library's operators, trained and then served.

One layer reads a stream of tokens: queries and keys are normed per head and
turned by their positions (``qk_norm_rotate``), linear attention with a learned
decay for each token and head carries the past (``linear_attention``), and the
result predicts the next token.  It learns to repeat what came `PERIOD` tokens
ago; then it is served one token at a time (``linear_attention_step`` on the
state that the prompt leaves), and the single tokens' predictions are checked
against the whole sequence's.

    python examples/sequence_layer.py [steps]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import element_scan_recurrences_gb300 as es  # noqa: E402
from element_scan_recurrences_gb300 import autograd as ag  # noqa: E402

TOKENS, WIDTH, HEADS, HEAD = 32, 256, 4, 64
PERIOD = 7


class Layer(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(TOKENS, WIDTH)
        # the last two tokens' embeddings side by side: what was said, and what had been said before it
        self.qkv = torch.nn.Linear(2 * WIDTH, 3 * HEADS * HEAD, bias=False)
        self.fade = torch.nn.Linear(WIDTH, HEADS)
        self.out = torch.nn.Linear(HEADS * HEAD, TOKENS)
        self.q_weight = torch.nn.Parameter(torch.ones(HEAD))
        self.k_weight = torch.nn.Parameter(torch.ones(HEAD))
        torch.nn.init.constant_(self.fade.bias, -3.0)
        angle = torch.arange(4096)[:, None] * 100.0 ** (-torch.arange(HEAD // 4) / (HEAD // 4))
        self.register_buffer("cos", angle.cos())
        self.register_buffer("sin", angle.sin())

    def inputs(self, now, before):
        """q, k, v [B, T, heads, HEAD] in bf16 and the log decays [B, T, heads] in f32."""
        x, y = self.embed(now), self.embed(before)
        q, k, v = self.qkv(torch.cat([x, y], -1)).view(*now.shape, 3 * HEADS, HEAD).to(torch.bfloat16).split(HEADS, 2)
        return q, k, v, -torch.nn.functional.softplus(self.fade(x))

    def forward(self, tokens, state=None):
        """Logits [B, T, TOKENS] of whole sequences and the state they leave."""
        before = torch.nn.functional.pad(tokens[:, :-1], (1, 0))
        q, k, v, g = self.inputs(tokens, before)
        w = self.q_weight.to(q.dtype), self.k_weight.to(q.dtype)
        q, k = ag.qk_norm_rotate(q, k, *w, self.cos, self.sin)
        o, state = ag.linear_attention(q, k, v, g, state, final_state=True)
        return self.out(o.flatten(2).float()), state

    @torch.no_grad()
    def step(self, token, before, position, state):
        """Logits [B, TOKENS] of one more token; the state is updated in place."""
        q, k, v, g = self.inputs(token[:, None], before[:, None])
        w = self.q_weight.to(q.dtype), self.k_weight.to(q.dtype)
        q, k = es.qk_norm_rotate(q, k, *w, self.cos, self.sin, positions=position)
        o, _ = es.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], g[:, 0], state)
        return self.out(o.flatten(1).float())


def batch(n, length, gen):
    """Sequences that repeat their first PERIOD tokens."""
    first = torch.randint(0, TOKENS, (n, PERIOD), generator=gen, device="cuda")
    return first.repeat(1, -(-(length + 1) // PERIOD))[:, :length + 1]


def main(steps=150):
    torch.manual_seed(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer = Layer().cuda()
    opt = torch.optim.AdamW(layer.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        tokens = batch(16, 120, gen)
        logits, _ = layer(tokens[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits[:, PERIOD:].flatten(0, 1), tokens[:, 1 + PERIOD:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    # served: a prompt of 50 tokens, then the rest one by one
    with torch.no_grad():
        tokens = batch(4, 80, gen)
        whole, _ = layer(tokens[:, :-1])
        logits, state = layer(tokens[:, :50])
        far = float((logits - whole[:, :50]).abs().max())
        right = total = 0
        for t in range(50, 80):
            position = torch.tensor([t], dtype=torch.int32, device="cuda")
            logits = layer.step(tokens[:, t], tokens[:, t - 1], position, state)
            far = max(far, float((logits - whole[:, t]).abs().max()))
            right += int((logits.argmax(-1) == tokens[:, t + 1]).sum())
            total += len(tokens)
    es.device_status()
    return losses, far / float(whole.abs().max()), right / total


if __name__ == "__main__":
    losses, far, right = main(int(sys.argv[1]) if len(sys.argv) > 1 else 150)
    print("loss %.3f -> %.3f; single tokens against the whole sequence: %.1e of the largest logit; %.0f%% right"
          % (losses[0], losses[-1], far, 100 * right))
