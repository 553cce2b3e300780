"""Inputs and state builders shared by the tests of the 4-bit cache and of the
page operations."""

from __future__ import annotations

import numpy as np
import torch

from oracle import kv4_oracle as ko


def f64(t):
    return t.double().cpu().numpy()


def bf16_rows(gen, *shape, channels=0.5):
    """Normal bf16 values, some channels stronger than others."""
    x = torch.randn(*shape, generator=gen)
    return (x * torch.exp(channels * torch.randn(shape[-1], generator=gen))).to(torch.bfloat16)


def random_tables(rng, lens, block_rows, extra=3, most=None):
    """(block table int32 [B, max_blocks], num_blocks): pages in any order;
    entries past a sequence's pages are -1."""
    pages = [-(-n // block_rows) for n in lens]
    most = max(1, max(pages, default=1), most or 0)
    num = sum(pages) + extra
    order = rng.permutation(num).tolist()
    table = np.full((len(lens), most), -1, np.int32)
    for b, n in enumerate(pages):
        for i in range(n):
            table[b, i] = order.pop()
    return table, num


def random_pool(rng, num_blocks, Hkv, block_rows, D, scale=(0.05, 0.6)):
    """A 4-bit pool with random codes and finite parameters."""
    tiles = block_rows // 64
    pool = rng.integers(0, 256, (num_blocks, Hkv, tiles, ko.tile_bytes(D)), dtype=np.uint8)
    gr, nb = D // 64, 32 * D
    for first in (nb, 2 * nb + 256 * gr):
        n = 64 * gr
        sc = ko.bf16_bits(ko.bf16(rng.uniform(*scale, (num_blocks, Hkv, tiles, n))))
        off = ko.bf16_bits(ko.bf16(-7.5 * rng.uniform(*scale, (num_blocks, Hkv, tiles, n))))
        words = np.ascontiguousarray(np.stack((sc, off), -1)).view(np.uint8)
        pool[..., first:first + 4 * n] = words.reshape(num_blocks, Hkv, tiles, 4 * n)
    return pool


def random_slots(rng, B, most, R, share=0.5, extra=10, pins=0):
    """A consistent page state: (lens, table, refs, num_blocks).  Some slots
    share the full pages of an earlier one; `pins` pages are held besides."""
    lens, rows, count = [], [], 0
    for b in range(B):
        n = int(rng.integers(0, most * R + 1)) if rng.random() < 0.9 else 0
        row = []
        if b and rng.random() < share:
            f = int(rng.integers(0, b))
            row = rows[f][:min(lens[f], n) // R]
        while len(row) < -(-n // R):
            row = row + [count]
            count += 1
        lens.append(n)
        rows.append(row)
    num = count + extra + pins
    at = rng.permutation(num).tolist()
    refs = [0] * num
    table = []
    for row in rows:
        for p in row:
            refs[at[p]] += 1
        table.append([at[p] for p in row] + [-1] * (most - len(row)))
    for p in rng.permutation(num)[:pins].tolist():
        refs[p] += 1
    return lens, table, refs, num


def ints(x, device="cuda"):
    return torch.tensor(np.asarray(x, np.int32), dtype=torch.int32, device=device)


def same_pool(got, want):
    """None if two pools are equal byte for byte, else where they first differ."""
    got = got.cpu().numpy()
    at = np.argwhere(got != want)
    if not len(at):
        return None
    page, head, tile, byte = (int(x) for x in at[0])
    D = got.shape[-1] // 72
    for what in ("k", "v"):
        place, _, par = ko._PLACES[D][what]
        for name, where in (("codes of row, dim", np.argwhere(place == byte)),
                            ("params of row, group", np.argwhere(np.abs(par + 1.5 - byte) < 2))):
            if len(where):
                r = int(where[0][0])
                a = ko.read_rows(got[page, head, tile], what, D)
                b = ko.read_rows(want[page, head, tile], what, D)
                return (f"{len(at)} bytes; first: page {page} head {head} tile {tile}, {what} {name} "
                        f"{where[0].tolist()}: {int(got[page, head, tile, byte])} != "
                        f"{int(want[page, head, tile, byte])}; scale, offset "
                        f"{a[1][r]} {a[2][r]} != {b[1][r]} {b[2][r]}")
