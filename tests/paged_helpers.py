"""Batches over paged caches for the tests of the operators around the sparse
attention: ragged sequences (some without new tokens), permuted pages, and
references in 64 bits on the CPU."""
import numpy as np
import torch

import indexer_top_sparse_lightning_b200 as dsa

PAGE = 64
ROW = 576
DV = 512
EPS32 = 2.0 ** -24      # half a step of fp32, relative
HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative to the value


class Paged:
    """lens and nq per sequence; `pad` query rows behind the last sequence; pages in random order,
    with `spare` pages that belong to nobody."""

    def __init__(self, lens, nq, seed=0, pad=0, spare=2, device="cuda"):
        r = np.random.default_rng(seed)
        self.lens, self.nq = np.asarray(lens, np.int64), np.asarray(nq, np.int64)
        self.B = len(self.lens)
        self.cu = np.concatenate([[0], np.cumsum(self.nq)]).astype(np.int32)
        self.real = int(self.cu[-1])
        self.T = self.real + pad
        nb = -(-self.lens // PAGE)
        self.num_blocks = int(nb.sum()) + spare
        ids = r.permutation(self.num_blocks).astype(np.int32)
        self.free = ids[int(nb.sum()):]                      # pages of nobody
        self.table = np.full((self.B, max(1, int(nb.max())) + 1), -1, np.int32)
        at = 0
        for b in range(self.B):
            self.table[b, :nb[b]] = ids[at:at + nb[b]]
            at += int(nb[b])
        self.device = device

    def seq_pos(self):
        """(sequence, position) of each real token."""
        seq = np.repeat(np.arange(self.B), self.nq)
        off = np.arange(self.real) - self.cu[seq]
        return seq, self.lens[seq] - self.nq[seq] + off

    def rows(self, b):
        """Cache rows of the positions of sequence b."""
        p = np.arange(self.lens[b])
        return self.table[b, p // PAGE].astype(np.int64) * PAGE + p % PAGE

    def batch(self):
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).to(self.device)  # noqa: E731
        return dsa.Batch(t(self.lens), t(self.cu), t(self.table), self.num_blocks, int(self.lens.max()),
                         max(1, int(self.nq.max())))


def randn(seed, *shape, scale=1.0):
    """N(0, scale) rounded to bf16, on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(torch.bfloat16)


def fp8_rows(x):
    """bf16 rows [..., 576] as e4m3 codes, scales, and the values they stand for (64 bits)."""
    v = torch.nn.functional.pad(x.float(), (0, 64)).unflatten(-1, (5, 128))
    a = v.abs().amax(-1)
    s = torch.where(a > 0, a / 448.0, torch.ones_like(a))
    c = (v / s[..., None]).to(torch.float8_e4m3fn)
    val = (c.double() * s.double()[..., None]).flatten(-2)[..., :ROW]
    return c.view(torch.uint8).flatten(-2)[..., :ROW].contiguous(), s.contiguous(), val


def assert_status_ok(ws=None):
    torch.cuda.synchronize()
    st = dsa.get_status(ws if ws is not None else dsa.status_workspace())
    assert st == 0, dsa.status_str(st)
