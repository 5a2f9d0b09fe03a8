"""A spline model over tokens, distilled from a teacher and then run token by token.

The model is an embedding, a gated recurrence over the sequence whose value and
gate come from a spline layer, a residual spline layer, and a spline layer to
the logits.  The teacher is a fixed random table of next-token logits (each
token's successor distribution), so that it can be sampled and its top logits
are known; a student that learns it has nothing left to lose.  Training takes
the loss and its gradient from one call (``kan_distill_step``), or through
autograd with ``--autograd``; generation keeps one state row per sequence and
advances all of them by one token a step.  With ``--mixer delta`` the sequence is
mixed by the gated delta rule instead, whose state is a matrix for each head, and a
join puts the mixed rows onto the embedding and makes the rows of the next layer.

    python examples/token_distillation.py --steps 60
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import kolmogorov_arnold_network_amd as kan  # noqa: E402


class TokenModel(torch.nn.Module):
    def __init__(self, tokens, width, grid_size=5, device=None):
        super().__init__()
        kw = dict(grid_size=grid_size, grid_range=(-3.0, 3.0), device=device, coef_std=0.02)
        self.embed = kan.KANEmbedding(tokens, width, device=device)
        self.mix = kan.KANRecurrence(width, width, **kw)
        self.channels = kan.KANLayer(width, width, **kw)
        self.head = kan.KANLayer(width, tokens, **kw)

    def _rows(self, x, mixed):
        x = x + mixed
        return self.head(x + self.channels(x))

    def state(self, rows):
        """A pool of first states."""
        return torch.zeros(rows, self.mix.out_features, device=self.embed.table.device)

    def forward(self, ids, lengths=None):
        """Logits ``[B, T, tokens]`` of token ids ``[B, T]``."""
        x = self.embed(ids)
        return self._rows(x, self.mix(x, lengths=lengths)[0])

    @torch.no_grad()
    def step(self, ids, state, slots=None):
        """Logits ``[B, tokens]`` after one more token of each sequence."""
        x = self.embed(ids)
        return self._rows(x, self.mix.step(x, state, slots))


class DeltaTokenModel(torch.nn.Module):
    """The same around the gated delta rule, with heads of 16 keys and 16 values."""

    def __init__(self, tokens, width, grid_size=5, device=None):
        super().__init__()
        kw = dict(grid_size=grid_size, grid_range=(-3.0, 3.0), device=device, coef_std=0.02)
        self.embed = kan.KANEmbedding(tokens, width, device=device)
        self.mix = kan.KANDeltaRule(width, width // 16, 16, 16, **kw)
        self.join = kan.KANJoin(width, device=device)
        self.channels = kan.KANLayer(width, width, **kw)
        self.head = kan.KANLayer(width, tokens, **kw)

    def _rows(self, x, mixed):
        x, rows = self.join(mixed, x)
        return self.head(x + self.channels(rows))

    def state(self, rows):
        return torch.zeros(rows, self.mix.heads, 16, 16, device=self.embed.table.device)

    def forward(self, ids, lengths=None):
        x = self.embed(ids)
        return self._rows(x, self.mix(x, lengths=lengths)[0])

    @torch.no_grad()
    def step(self, ids, state, slots=None):
        x = self.embed(ids)
        return self._rows(x, self.mix.step(x, state, slots))


def sample_batch(teacher, batch, length, top, gen):
    """Sequences drawn from the teacher, ragged (padded with -1), and its top logits."""
    dev = teacher.device
    V = teacher.shape[0]
    probs = torch.softmax(teacher, 1)
    ids = torch.empty(batch, length, dtype=torch.int64, device=dev)
    ids[:, 0] = torch.randint(0, V, (batch,), device=dev, generator=gen)
    for t in range(1, length):
        ids[:, t] = torch.multinomial(probs[ids[:, t - 1]], 1, generator=gen)[:, 0]
    lengths = torch.randint(length // 2, length + 1, (batch,), device=dev, generator=gen)
    inside = torch.arange(length, device=dev)[None, :] < lengths[:, None]
    t, top_ids = torch.topk(teacher[ids], top, dim=-1)
    return torch.where(inside, ids, -1), lengths.to(torch.int32), inside, top_ids, t


def main(steps=60, tokens=200, width=64, batch=16, length=48, top=16, temperature=1.0, autograd=False, seed=0,
         device="cuda:0", quiet=False, mixer="recurrence"):
    torch.manual_seed(seed)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    teacher = torch.randn(tokens, tokens, device=device, generator=gen) * 2.0
    model = (DeltaTokenModel if mixer == "delta" else TokenModel)(tokens, width, device=device)
    opt = torch.optim.Adam(model.parameters(), lr=1e-2)
    losses = []
    for it in range(steps):
        ids, lengths, inside, top_ids, t = sample_batch(teacher, batch, length, top, gen)
        weight = inside.float() / inside.sum()
        z = model(ids, lengths)
        if autograd:
            loss = kan.KANDistillLoss(temperature, reduction="sum")(z, top_ids, t, weight)
            loss.backward()
        else:
            rows, dz = kan.kan_distill_step(z.detach().view(-1, tokens), top_ids.view(-1, top), t.view(-1, top),
                                            temperature, weight=weight.view(-1))
            loss = rows.sum()
            z.backward(dz.view_as(z))
        opt.step()
        opt.zero_grad(set_to_none=True)
        losses.append(loss.detach())
        if not quiet and (it % 10 == 0 or it == steps - 1):
            print("step %3d  loss %.4f" % (it, float(losses[-1])), flush=True)
    # four sequences, greedily, in rows 5, 2, 7 and 0 of a pool of eight states
    state = model.state(8)
    slots = torch.tensor([5, 2, 7, 0], dtype=torch.int32, device=device)
    out = [torch.randint(0, tokens, (4,), device=device, generator=gen)]
    for _ in range(12):
        out.append(model.step(out[-1], state, slots).argmax(1))
    out = torch.stack(out, 1)
    if not quiet:
        print("generated\n", out.cpu().numpy())
    return dict(losses=[float(v) for v in losses], generated=out, model=model, state=state, slots=slots)


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=200)
    ap.add_argument("--width", type=int, default=64)
    ap.add_argument("--batch", type=int, default=16)
    ap.add_argument("--length", type=int, default=48)
    ap.add_argument("--temperature", type=float, default=1.0)
    ap.add_argument("--autograd", action="store_true")
    ap.add_argument("--mixer", choices=("recurrence", "delta"), default="recurrence")
    main(**vars(ap.parse_args()))
