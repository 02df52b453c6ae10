"""Inputs of the decoding operators' tests, for the CPU and the GPU."""
import numpy as np
import torch

from oracle import decode


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def random_tree(g, n, chain=0.3):
    """Parents of a tree of n nodes."""
    out = []
    for i in range(n):
        if i == 0:
            out.append(-1)
        elif torch.rand(1, generator=g).item() < chain:
            out.append(i - 1)
        else:
            out.append(int(torch.randint(0, i, (1,), generator=g)))
    return out


def trees(g, nodes, words=None, chain=0.3):
    """Trees of the given numbers of nodes -> (parents int32 [total], bool
    matrices, mask words [total, words], depths)."""
    parents, see, depths = [], [], []
    words = words or max(1, -(-max(nodes + [1]) // 32))
    masks = [torch.zeros(0, words, dtype=torch.int32)]
    for n in nodes:
        p = random_tree(g, n, chain)
        s, d = decode.ancestors(p)
        parents += p
        depths += d
        see.append(torch.from_numpy(s))
        masks.append(decode.words_of(s, words))
    return torch.tensor(parents, dtype=torch.int32), see, torch.cat(masks), depths


def logits_row(g, vocab, peak, T):
    """A vocabulary's bulk and a few tokens that stand out by up to `peak`."""
    x = torch.randn(vocab, generator=g) * 2
    at = torch.randint(0, vocab, (min(vocab, 40),), generator=g)
    x[at] += torch.rand(len(at), generator=g) * peak
    return x.to(T)


def sample_wants(x, u, t=None, k=None, p=None, m=None):
    """decode.sample row by row: tokens, logprobs, margins."""
    out = []
    for i in range(x.shape[0]):
        pick = lambda v, off: off if v is None else v[i].item()  # noqa: E731
        out.append(decode.sample(x[i].float().numpy(), u[i].item(), pick(t, 1.0), pick(k, 0), pick(p, 1.0), pick(m, 0.0)))
    return [np.array(v) for v in zip(*out)]
