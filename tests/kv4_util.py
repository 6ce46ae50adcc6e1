"""A paged 4-bit cache on the GPU with its contents on the host, for the GPU tests."""
import numpy as np

import kv4_ref as ref


def i32(x, dev):
    import torch

    return torch.as_tensor(np.ascontiguousarray(x, np.int32)).to(dev)


class Pool:
    """n_seqs sequences of `rows` rows on pages in an order of no kind, between pages that nobody owns (filled with
    bytes of every kind); rows of the owned pages hold normal values."""

    def __init__(self, dev, n_seqs, rows, n_kv, hd, page=64, seed=0, spare=3, scale=1.0):
        import torch

        from weight_streaming_gemv_gb300 import qlin

        rng = np.random.default_rng(seed)
        per = -(-rows // page)
        n = n_seqs * per + spare
        self.page, self.hd, self.n_kv, self.n_seqs, self.per, self.rows = page, hd, n_kv, n_seqs, per, per * page
        self.table = rng.permutation(n)[: n_seqs * per].reshape(n_seqs, per).astype(np.int32)
        self.codes = rng.integers(0, 256, (2, n, n_kv, page, hd // 2)).astype(np.uint8)
        self.scales = rng.integers(0, 256, (2, n, n_kv, page, hd // 32)).astype(np.uint8)
        x = rng.standard_normal((2, n_seqs * per, n_kv, page, hd), np.float32) * np.float32(scale)
        code, b = ref.quantise(x)
        own = self.table.reshape(-1)
        self.codes[:, own], self.scales[:, own] = ref.pack(code), b
        up = lambda a: torch.from_numpy(a).to(dev)
        self.d_codes, self.d_scales, self.d_table = up(self.codes), up(self.scales), up(self.table)
        self.c = qlin.kv4_cache(self.d_codes[0], self.d_codes[1], self.d_scales[0], self.d_scales[1], self.d_table)

    def set_table(self, table):
        import torch

        self.table = np.asarray(table, np.int32)
        self.d_table.copy_(torch.from_numpy(self.table))

    def host(self, s):
        """(keys, values [rows][n_kv][hd], whether a row's page is in range) of sequence s"""
        ids = self.table[s]
        there = (ids >= 0) & (ids < self.codes.shape[1])
        out = []
        for i in (0, 1):
            x = ref.values(self.codes[i][np.where(there, ids, 0)], self.scales[i][np.where(there, ids, 0)])
            out.append(x.transpose(0, 2, 1, 3).reshape(self.rows, self.n_kv, self.hd))
        return out[0], out[1], np.repeat(there, self.page)

    def refresh(self):
        """the device's bytes to the host's"""
        self.codes, self.scales = self.d_codes.cpu().numpy(), self.d_scales.cpu().numpy()
