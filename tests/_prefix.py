"""Test inputs of requests that share their first pages."""

import numpy as np

from _serving import PagedCase


class SharedCase(PagedCase):
    """Groups of requests: the requests of group i start with the same prefix[i] tokens (whole pages), in the same pages.
    own[r]: tokens of request r behind its prefix, new[r] of them new."""

    def __init__(self, seed, sizes, prefix, new, own, Hq, Hkv, d, page_size, pad_rows=0, value=1.0, spare_entries=0):
        import torch

        self.sizes, self.prefix = np.array(sizes), np.array(prefix, np.int32)
        self.group_indptr = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        mine = np.repeat(np.arange(len(sizes)), sizes)
        super().__init__(seed, new, self.prefix[mine] + np.array(own), Hq, Hkv, d, page_size, spare_entries, pad_rows, value)
        for i, (a, b) in enumerate(zip(self.group_indptr[:-1], self.group_indptr[1:])):
            n, pages = int(self.prefix[i]), int(self.prefix[i]) // page_size
            for r in range(a + 1, b):  # the first request's pages; those that it had hold what nobody may read
                at = self.page_indptr[r]
                old = torch.from_numpy(self.page_indices[at:at + pages].astype(np.int64))
                self.k_pages[old] = float("nan")
                self.v_pages[old] = float("nan")
                self.page_indices[at:at + pages] = self.page_indices[self.page_indptr[a]:self.page_indptr[a] + pages]
                self.k_seq[r][:n], self.v_seq[r][:n] = self.k_seq[a][:n], self.v_seq[a][:n]

    def dev(self, dev):
        return dict(super().dev(dev), group_indptr_host=self.group_indptr, prefix_host=self.prefix)
