"""A batch over the block-scaled cache for the tests: its pools on host and device, its queries, what is expected."""

import numpy as np
import torch

from oracle import block as OB

SENTINEL = -12288.0


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(torch.bfloat16)


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Batch:
    """Requests of given lengths: codes, exponents a few binades apart (``spread``), block table. Codes that no
    token holds are NaN, exponents of blocks that no token is in are 0 or 255. ``order``: how pages, tokens and heads lie in memory."""

    def __init__(self, lens, *, h_k=2, d=128, page=16, block=16, seed=0, spread=(-10, -3), order="phtd", extra=3):
        rng = np.random.default_rng(seed)
        self.lens, self.h_k, self.d, self.page, self.block = np.array(lens, np.int32), h_k, d, page, block
        self.B, self.rng, self.order = len(lens), rng, order
        per = [-(-int(n) // page) for n in lens]
        self.pages = sum(per) + extra
        ids = rng.permutation(self.pages)
        self.table = np.full((self.B, max(per + [1]) + 1), -1, np.int32)
        at = 0
        held = np.zeros((self.pages, page), bool)
        for b, n in enumerate(lens):
            self.table[b, :per[b]] = ids[at:at + per[b]]
            at += per[b]
            t = np.arange(int(n))
            held[self.table[b][t // page], t % page] = True
        self.codes, self.exps = {}, {}
        for name in "kv":
            x = np.clip(rng.standard_normal((self.pages, page, h_k, d)) * 90, -448, 448).astype(np.float32)
            c = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy().copy()
            c[~held] = 0x7F
            e = rng.integers(127 + spread[0], 128 + spread[1], (self.pages, h_k, page // block)).astype(np.uint8)
            live = held.reshape(self.pages, page // block, block).any(2)
            e[~np.repeat(live[:, None], h_k, 1)] = rng.choice([0, 255])
            self.codes[name], self.exps[name] = c, e
        self._dev = None

    def kv(self):
        import paged_fp8_decode_gb300 as mj

        if self._dev is None:
            def pool(c):
                axes = {"p": 0, "t": 1, "h": 2}
                perm = [axes[x] for x in self.order[:3]] + [3]
                return up(c.transpose(perm)).permute(*[perm.index(i) for i in range(4)])
            self._dev = mj.BlockKV(pool(self.codes["k"]), pool(self.codes["v"]), up(self.exps["k"]), up(self.exps["v"]))
            self.table_dev, self.lens_dev = up(self.table), up(self.lens)
        return self._dev

    def rows(self, name, b, n=None):
        n = int(self.lens[b]) if n is None else n
        if not hasattr(self, "_vals"):
            self._vals = {x: OB.values(self.codes[x], self.exps[x]) for x in "kv"}
        return OB.gather(self._vals[name], self.table[b], n)

    def reload(self):
        """The host's copy after a write on the device."""
        kv = self.kv()
        self.codes = {"k": kv.k_cache.cpu().numpy(), "v": kv.v_cache.cpu().numpy()}
        self.exps = {"k": kv.k_exp.cpu().numpy(), "v": kv.v_exp.cpu().numpy()}
        if hasattr(self, "_vals"):
            del self._vals

    def vmax(self, b):
        """The largest value that V's codes could stand for among the request's blocks."""
        n = int(self.lens[b])
        e = self.exps["v"][self.table[b][np.arange(n) // self.page], :, np.arange(n) % self.page // self.block]
        return 448.0 * 2.0 ** (np.clip(e.astype(int), OB.LOW, OB.HIGH).max() - 127.0)
