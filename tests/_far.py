"""A context whose last keys are those of a small problem and lie at the end of 32 bits: under a
window that reaches no further, both give the same results."""
import numpy as np
import torch

from _score import Paged, Rule

SPAN = 384  # keys of the small problem, but for what the far end lacks of whole blocks


class Far:
    """small: a Paged of one sequence; table and length of the far one, which ends at `end`, its
    keys the small one's.  No entry below them names a block."""

    def __init__(self, end, hq, hkv, d, kv, seed=0):
        self.start = end // 128 * 128 - (SPAN - 128)
        self.small = Paged([end - self.start], hq, hkv, d, kv, seed=seed)
        self.end, self.mbps = end, (end + 15) // 16
        self.table = torch.full((1, self.mbps), -1, dtype=torch.int32, device="cuda")
        n = self.mbps - self.start // 16
        self.table[0, self.start // 16:] = self.small.t[0, :n]
        self.len = torch.tensor([end], dtype=torch.int32, device="cuda")
        self.desc = self.small.make_desc(max_blocks_per_seq=self.mbps)

    def rule(self, **kw):
        return Rule(self.small.d, self.small.hq, 1, **kw)


def queries(p, m):
    q, q64 = p.queries(m)
    qo = np.array([0, m], np.int32)
    return qo, torch.from_numpy(qo).to("cuda"), q, q64
