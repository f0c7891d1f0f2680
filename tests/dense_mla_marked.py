"""Inputs for long contexts whose outputs show every page's weight, and what they have to be.

Each 64-key page of a request carries one marker dim in its values (1 there, 0 elsewhere), so output d is the
summed weight of the pages marked d; at most a few pages share a dim, so a page that is lost or counted twice moves
its output by a fixed share, however long the context is.  The scores depend on the page only: its level in one
rope dim times the query's value there.

Bound, relative, per output: P is rounded to bf16 (2^-8) and so is the output (2^-8); a score is one product, exact
in fp32 before its scaling (2^-23 |S| with |S| < 4: 2^-21), the exponential 2^-21; l sums up to 2^18 weights in
fp32, a thread at most 2^6 of a key tile and then the tiles' sums, up to 2^11 of them: 2^-24 (2^6 + 2^11) < 2^-12;
only the pages of a dim add anything to its output, at most 8 pages in 32 steps of the products or a little more:
2^-23 2^6; joining of pieces: their log-sum-exps (log2, below 32) carry 2^-19 each: 2^-18.  Together below
2 * 2^-8 + 2^-9.  lse: the sum's 2^-12, plus 2^-18 for logarithms and products.
A page alone in its dim is all of that output; one of m equally heavy ones is 1 / m of it."""
import torch

REL = 2 * 2.0 ** -8 + 2.0 ** -9
LSE = 2.0 ** -12 + 2.0 ** -18


def levels(pages, flat):
    """Level of each page: 0, or 0 / 1 / 2 in a pattern without a short period."""
    i = torch.arange(pages)
    return torch.zeros(pages) if flat else ((i * i + i // 7) % 3).float()


def weights(vis, level, gain):
    """[rows, pages] softmax weights of whole pages and the rows' lse, float64: row r sees its first vis[r] keys."""
    vis = torch.as_tensor(vis, dtype=torch.int64).clamp_min(0)
    first = torch.arange(level.shape[0], dtype=torch.int64) * 64
    keys = (vis[:, None] - first[None]).clamp(0, 64).double()
    w = keys * torch.exp(level.double() * gain)[None]
    return w / w.sum(1, keepdim=True), torch.log(w.sum(1))


def outputs(w, marker, dims):
    """[rows, dims]: the weights summed by marker."""
    out = torch.zeros(w.shape[0], dims, dtype=torch.float64)
    return out.index_add_(1, marker, w)


def check(got, lse, want, want_lse):
    got, lse = got.double().cpu(), lse.double().cpu()
    err = (got - want).abs()
    assert bool((err <= REL * want).all()), f"out: off by {float((err / want.clamp_min(1e-12)).max())} of the value"
    assert bool(((lse - want_lse).abs() <= LSE).all()), f"lse: off by {float((lse - want_lse).abs().max())}"


def gain_of(q_value, scale):
    """What a level adds to the score: scale times the query's bf16 value."""
    return scale * float(torch.tensor(q_value).to(torch.bfloat16))


def marker_of(pages, dims, b=0):
    """The dims (a power of two) over and over, five apart: a permutation of all of them each time."""
    return (torch.arange(pages) * 5 + 11 * b) % dims
