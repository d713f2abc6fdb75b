"""Paged KV cache: packing per-sequence caches into fixed-size pages.

A page store is bf16 [num_pages, Hkv, page_size, 128]; ``block_table[b, j]``
names the page that holds tokens j*page_size .. j*page_size + page_size - 1 of
sequence b (the layout kascade_decode_anchor_paged / kascade_decode_reuse_paged
read).  Pages are handed out in a seeded random order, as a serving engine's
allocator would after some churn.

A 4-bit store (q4_store) keeps K and V of a token in one 160-byte row of
uint8 [num_pages, Hkv, page_size, 160]; the block table is the same.
"""
from __future__ import annotations

from typing import List, Optional

import torch

from . import binding


def to_paged(ks: List[torch.Tensor], vs: List[torch.Tensor], page_size: int,
             seed: int = 0, spare_pages: int = 0):
    """Pack per-sequence caches ks[b], vs[b] ([Hkv, T_b, d]) into a page store.

    Returns (k_pages, v_pages, block_table int32 [B, max_pages], num_pages).
    Unused tail slots of a sequence's last page are zero; unused block-table
    entries are -1.
    """
    if page_size < 16 or page_size % 16:
        raise ValueError("page_size must be a positive multiple of 16")
    B = len(ks)
    Hkv, _, d = ks[0].shape
    dev = ks[0].device
    n_pages = [(k.shape[1] + page_size - 1) // page_size for k in ks]
    max_pages = max(1, max(n_pages))
    num_pages = sum(n_pages) + spare_pages
    num_pages = max(num_pages, 1)
    g = torch.Generator(device="cpu").manual_seed(seed)
    order = torch.randperm(num_pages, generator=g).tolist()
    k_pages = torch.zeros(num_pages, Hkv, page_size, d, dtype=ks[0].dtype, device=dev)
    v_pages = torch.zeros_like(k_pages)
    table = torch.full((B, max_pages), -1, dtype=torch.int32)
    nxt = 0
    for b in range(B):
        T = ks[b].shape[1]
        for j in range(n_pages[b]):
            p = order[nxt]
            nxt += 1
            table[b, j] = p
            lo, hi = j * page_size, min(T, (j + 1) * page_size)
            k_pages[p, :, : hi - lo] = ks[b][:, lo:hi]
            v_pages[p, :, : hi - lo] = vs[b][:, lo:hi]
    return k_pages, v_pages, table.to(dev), num_pages


def q4_store(lens: List[int], Hkv: int, page_size: int, device, seed: int = 0, spare_pages: int = 0):
    """An empty 4-bit page store with room for sequences of ``lens`` tokens.

    Returns (kv_pages uint8 [num_pages, Hkv, page_size, 160], block_table int32
    [B, max_pages]): the layout api.kv_write_paged_q4 fills and the _paged_q4
    calls read.  Pages are handed out in a seeded random order; unused
    block-table entries are -1.  Zero bytes stand for zeros.
    """
    if page_size < 16 or page_size % 16:
        raise ValueError("page_size must be a positive multiple of 16")
    n_pages = [(T + page_size - 1) // page_size for T in lens]
    num_pages = max(sum(n_pages) + spare_pages, 1)
    g = torch.Generator(device="cpu").manual_seed(seed)
    order = torch.randperm(num_pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(1, max(n_pages))), -1, dtype=torch.int32)
    nxt = 0
    for b, n in enumerate(n_pages):
        table[b, :n] = order[nxt: nxt + n]
        nxt += n
    kv_pages = torch.zeros(num_pages, Hkv, page_size, binding.Q4_ROW_BYTES, dtype=torch.uint8, device=device)
    return kv_pages, table.to(device)
