"""A state-space layer on the library's operators, trained and then served.

One layer reads a stream of tokens: a projection gives each channel's input and
gate, the short causal convolution mixes neighbouring tokens (``causal_conv``), a
second projection makes the steps and the selections B and C of what it sees, the
selective scan carries the past and gates its result (``selective_scan``), and the
groups of channels are normed (``group_norm``) before the prediction.  It learns to
say which token came last before the latest marker; then it is served one token at a
time (``causal_conv_step``, ``selective_scan_step`` on the states that the prompt
leaves), and the single tokens' predictions are checked against the whole
sequence's.

    python examples/state_space_layer.py [steps]
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import element_scan_recurrences_gb300 as es  # noqa: E402
from element_scan_recurrences_gb300 import autograd as ag  # noqa: E402

TOKENS, WIDTH, CHANNELS, STATES, TAPS, GROUPS, RANK = 16, 128, 256, 16, 4, 4, 8
MARKER = 0


class Layer(torch.nn.Module):
    def __init__(self):
        super().__init__()
        self.embed = torch.nn.Embedding(TOKENS, WIDTH)
        self.inside = torch.nn.Linear(WIDTH, 2 * CHANNELS, bias=False)
        self.conv_weight = torch.nn.Parameter(torch.randn(CHANNELS, TAPS) / math.sqrt(TAPS))
        self.conv_bias = torch.nn.Parameter(torch.zeros(CHANNELS))
        self.select = torch.nn.Linear(CHANNELS, RANK + 2 * STATES, bias=False)
        self.step_out = torch.nn.Linear(RANK, CHANNELS, bias=False)
        # steps from a thousandth to a tenth, through log(1 + e^bias)
        first = torch.exp(torch.rand(CHANNELS) * math.log(100.0) + math.log(1e-3))
        self.step_bias = torch.nn.Parameter(first + torch.log(-torch.expm1(-first)))
        self.log_a = torch.nn.Parameter(torch.log(torch.arange(1, STATES + 1).float()).repeat(CHANNELS, 1))
        self.skip = torch.nn.Parameter(torch.ones(CHANNELS))
        self.norm_weight = torch.nn.Parameter(torch.ones(GROUPS, CHANNELS // GROUPS))
        self.out = torch.nn.Linear(CHANNELS, TOKENS)

    def halves(self, tokens):
        """The channels' inputs and gates, as halves of one projection's result, in bf16."""
        return self.inside(self.embed(tokens)).to(torch.bfloat16).split(CHANNELS, -1)

    def selections(self, x):
        """Steps before the bias [..., CHANNELS], B and C [..., 1, STATES] of the mixed inputs."""
        rank, b, c = self.select(x.float()).split([RANK, STATES, STATES], -1)
        return self.step_out(rank).to(x.dtype), b.to(x.dtype).unsqueeze(-2), c.to(x.dtype).unsqueeze(-2)

    def forward(self, tokens, lengths=None, states=(None, None)):
        """Logits [B, T, TOKENS] of whole sequences and the states they leave."""
        x, gate = self.halves(tokens)
        x, mixed = ag.causal_conv(x, self.conv_weight.to(x.dtype), self.conv_bias.to(x.dtype), states[0], lengths, final_state=True)
        delta, b, c = self.selections(x)
        y, state = ag.selective_scan(x, delta, -self.log_a.exp(), b, c, self.skip, gate, self.step_bias, initial_state=states[1],
                                     lengths=lengths, final_state=True)
        y = ag.group_norm(y.unflatten(-1, (GROUPS, -1)), self.norm_weight.to(y.dtype), center=False)
        return self.out(y.flatten(2).float()), (mixed, state)

    @torch.no_grad()
    def step(self, token, states):
        """Logits [B, TOKENS] of one more token; the states are updated in place."""
        x, gate = self.halves(token)
        x, _ = es.causal_conv_step(x, self.conv_weight.to(x.dtype), self.conv_bias.to(x.dtype), states[0])
        delta, b, c = self.selections(x)
        y, _ = es.selective_scan_step(x, delta, -self.log_a.exp(), b, c, self.skip, gate, self.step_bias, states[1])
        y = es.group_norm(y.view(len(token), 1, GROUPS, -1), self.norm_weight.to(y.dtype), center=False)
        return self.out(y.flatten(1).float())


def batch(n, length, gen):
    """Random tokens with markers among them, and at each place the token before the latest marker."""
    tokens = torch.randint(1, TOKENS, (n, length), generator=gen, device="cuda")
    tokens[torch.rand(n, length, generator=gen, device="cuda") < 0.15] = MARKER
    before = torch.nn.functional.pad(tokens[:, :-1], (1, 0))
    at = torch.where(tokens == MARKER, torch.arange(length, device="cuda"), 0).cummax(1).values
    return tokens, before.gather(1, at)


def main(steps=300):
    torch.manual_seed(0)
    gen = torch.Generator(device="cuda").manual_seed(0)
    layer = Layer().cuda()
    opt = torch.optim.AdamW(layer.parameters(), lr=3e-3)
    losses = []
    for i in range(steps):
        tokens, said = batch(32, 96, gen)
        logits, _ = layer(tokens)
        loss = torch.nn.functional.cross_entropy(logits[:, 8:].flatten(0, 1), said[:, 8:].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    # served: prompts of different lengths in one batch, then each row's next tokens one by one
    with torch.no_grad():
        tokens, said = batch(4, 80, gen)
        whole, _ = layer(tokens)
        first = torch.tensor([50, 31, 2, 44], dtype=torch.int32, device="cuda")
        _, states = layer(tokens[:, :50], first)
        rows = torch.arange(4, device="cuda")
        far, right, total = 0.0, 0, 0
        for i in range(30):
            at = first.long() + i
            logits = layer.step(tokens[rows, at], states)
            far = max(far, float((logits - whole[rows, at]).abs().max()))
            right += int((logits.argmax(-1) == said[rows, at]).sum())
            total += len(rows)
    es.device_status()
    return losses, far / float(whole.abs().max()), right / total


if __name__ == "__main__":
    losses, far, right = main(int(sys.argv[1]) if len(sys.argv) > 1 else 300)
    print("loss %.3f -> %.3f; single tokens against the whole sequence: %.1e of the largest logit; %.0f%% right"
          % (losses[0], losses[-1], far, 100 * right))
