"""Calls of kv_attention that reach each of its forms under each mask: the block
size, whether contexts are split, and how split ones are joined."""

from dataclasses import dataclass
from typing import Optional, Tuple

import bit_gemm_amd as nv


@dataclass(frozen=True)
class Call:
    d: int
    rows: int  # of a workgroup: the kernel
    split: bool
    lens: Tuple[int, ...]
    new: Tuple[int, ...]
    hq: int
    hkv: int
    window: int = 0
    causal: bool = True
    pages: Optional[int] = None  # of the table; None: as many as the longest context has
    page: int = 32
    wide_join: Optional[bool] = None  # split contexts of more than 128 sixteens of rows: a wave's lanes all on one part

    @property
    def one_each(self):
        return min(self.new) == max(self.new) == 1

    @property
    def table_pages(self):
        return self.pages or max(-(-n // self.page) for n in self.lens)

    @property
    def sizes(self):
        return (len(self.lens), sum(self.new), self.hq, self.hkv, self.d, self.page, self.table_pages, self.window,
                self.one_each)

    def __str__(self):
        lens = f"{len(self.lens)}x{max(self.lens)}"
        mask = f"w{self.window}" if self.window else "causal" if self.causal else "all"
        return f"{self.d}-{self.rows}-{'split' if self.split else 'whole'}-{lens}-{max(self.new)}-{self.hq}on{self.hkv}-{mask}"


def check_plan(c):
    """The call's form is the one that it names."""
    b, tokens, group = len(c.lens), sum(c.new), c.hq // c.hkv
    assert nv.kv_attention_path(*c.sizes) == c.rows, (c, nv.kv_attention_path(*c.sizes))
    ws = nv.kv_attention_workspace_size(*c.sizes)
    assert (ws > 0) == c.split, c
    if c.wide_join is not None:
        blocks = b * -(-group // c.rows) if c.one_each else (tokens * group + b * (c.rows - 1)) // c.rows
        items = ws // (4 * c.rows * c.hkv * (c.d + 2))  # for each head: row blocks and further parts
        assert items > blocks and (blocks * c.hkv * c.rows // 16 > 128) == c.wide_join, (c, blocks)


ONE = (1,)
# windows: shorter than the contexts, no multiples of 32
WINDOWS = [
    Call(64, 16, False, (900, 700, 20), (200, 3, 20), 4, 2, 301),
    Call(64, 32, False, (2600, 333), (400, 50), 64, 1, 1990),
    Call(64, 16, True, (5000, 300), (2, 3), 8, 1, 3001),
    Call(64, 16, True, (5000, 4000, 2000), ONE * 3, 8, 1, 1501),
    Call(64, 32, True, (6500, 6100), (60, 70), 64, 1, 6001),
    Call(128, 16, False, (900, 700, 20), (200, 3, 20), 4, 2, 301),
    Call(128, 32, False, (2600, 333), (400, 50), 64, 1, 1990),
    Call(128, 256, False, (2600, 333), (2100, 50), 64, 1, 1990),
    Call(128, 16, True, (5000, 300), (2, 3), 8, 1, 3001),
    Call(128, 16, True, (5000, 4000, 2000), ONE * 3, 8, 1, 1501),
    Call(128, 32, True, (6500, 6100), (60, 70), 64, 1, 6001),
    Call(128, 256, True, (6500, 100), (700, 100), 64, 1, 6001),
    Call(256, 16, False, (900, 700, 20), (200, 3, 20), 4, 2, 301),
    Call(256, 128, False, (2600, 333), (1000, 50), 64, 1, 1990),
    Call(256, 16, True, (5000, 300), (2, 3), 8, 1, 3001),
    Call(256, 16, True, (5000, 4000, 2000), ONE * 3, 8, 1, 1501),
    Call(256, 128, True, (6500, 100), (200, 100), 64, 1, 6001),
]
# every token sees the whole context, which is split
BOTH_WAYS = [
    Call(64, 16, True, (3000, 1100), (3, 20), 8, 1, causal=False),
    Call(64, 32, True, (3000, 1100), (50, 20), 8, 1, causal=False, pages=10000),
    Call(128, 16, True, (3000, 1100), ONE * 2, 8, 1, causal=False),
    Call(128, 32, True, (3000, 1100), (50, 20), 8, 1, causal=False, pages=6000),
    Call(128, 256, True, (3000, 1100), (150, 120), 8, 1, causal=False, pages=6000),
    Call(256, 16, True, (3000, 1100), (3, 20), 8, 1, causal=False),
    Call(256, 128, True, (3000, 1100), (150, 120), 8, 1, causal=False, pages=6000),
]
# joined with all lanes on one part, and with eight
_RAGGED = tuple(2300 + (977 * i) % 1900 if i % 5 == 0 else 1 + (331 * i) % 500 for i in range(48))
JOINED = [
    Call(64, 16, True, _RAGGED, ONE * 48, 12, 4, wide_join=True),
    Call(64, 16, True, _RAGGED[:20], ONE * 20, 12, 4, wide_join=False),
    Call(64, 32, True, _RAGGED[:10], (33,) * 10, 32, 4, pages=900, wide_join=True),
    Call(128, 16, True, _RAGGED, ONE * 48, 12, 4, wide_join=True),
    Call(128, 32, True, _RAGGED[:10], (15,) * 10, 32, 4, pages=900, wide_join=True),
    Call(128, 256, True, _RAGGED[:6], (130, 40, 7, 90, 61, 200), 32, 2, pages=20000, wide_join=True),
    Call(256, 16, True, _RAGGED, ONE * 48, 12, 4, wide_join=True),
    Call(256, 16, True, _RAGGED[:20], ONE * 20, 12, 4, wide_join=False),
    Call(256, 128, True, _RAGGED[:6], (130, 40, 7, 90, 61, 200), 32, 2, pages=5000, wide_join=True),
]
# more sequences than a wave has lanes, split
_MANY = tuple(2200 + (977 * i) % 1900 if i % 17 == 0 else (331 * i) % 300 for i in range(200))
MANY = [
    Call(64, 16, True, _MANY, ONE * 200, 4, 2),
    Call(64, 16, True, _MANY[:70], tuple(i % 3 for i in range(70)), 4, 2),
    Call(64, 32, True, _MANY[:100], tuple(7 + i % 9 for i in range(100)), 4, 2, pages=900),
    Call(128, 16, True, _MANY[:130], ONE * 130, 4, 2),
    Call(128, 16, True, _MANY[:129], tuple(i % 4 for i in range(129)), 4, 2),
    Call(128, 256, True, _MANY[:70], tuple(100 + i % 90 for i in range(70)), 2, 1, pages=10000),
    Call(256, 16, True, _MANY[:100], ONE * 100, 4, 2),
    Call(256, 128, True, _MANY[:70], tuple(100 + i % 90 for i in range(70)), 2, 1, pages=4000),
    Call(128, 16, True, _MANY[:90], tuple(1 + i % 2 for i in range(90)), 4, 2, window=2071),
]
CALLS = WINDOWS + BOTH_WAYS + JOINED + MANY
