"""prefix_attention over batches of many groups of unlike sizes (GPU); tolerances as in test_gpu_prefix."""
import math

import pytest
import torch

import bit_quantized_token_gb300 as bq
from test_gpu_prefix import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    bq.build()
    torch.cuda.set_device(0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("short", [100, 37, 127])
def test_small_groups_before_large_ones(hd, short):
    """Groups of at most 128 query rows of a kv head behind long prefixes, each before one of more rows behind a prefix
    that ends inside a key tile: the second half of a CTA's rows has nothing to do for many key tiles, then meets a tile
    of which the rows behind the prefix's end are infinite or NaN. The same bits as with finite ones there, every time."""
    starts = [0]
    for _ in range(6):
        starts += [starts[-1] + 20, starts[-1] + 70]
    p = Problem(starts=tuple(starts), gq=4, hd=hd, Hkv=8, P=2048, plens=(2048, short), own=8, lens=(3, 8, 0), tree=False)
    p.call()
    p.check()
    clean = p.out.clone()
    for g in range(1, p.G, 2):
        for m in (0, 1):
            p.rows["prefix"][m][g, :, short:] = math.nan
            p.rows["prefix"][m][g, :, short + 1::2] = math.inf
    outs = [torch.empty_like(clean) for _ in range(4)]
    for i in range(100):
        p.out = outs[i % 4]
        p.call()
        if i % 4 == 3:
            assert all(torch.equal(o, clean) for o in outs), i
    bq.tree_status()


@pytest.mark.parametrize("hd", [64, 128])
def test_groups_out_of_order_stay_apart(hd):
    """Many rows: a group that would begin inside the ones ahead of it begins where they end, so that no two groups have
    the same rows and all units together stay within the checked number."""
    kw = dict(B=170, gq=4, hd=hd, P=300, plens=(300, 200, 77, 150), lens=(5, 0, 40))
    p, want = Problem(starts=(0, 60, 20, 130, 170), **kw), Problem(starts=(0, 60, 60, 130, 170), **kw)
    assert torch.equal(p.call(), want.call())
    want.check()


MANY = [
    # more groups than a warp has lanes, some without sequences or rows
    dict(starts=tuple(sorted(3 * (i // 4 * 4) + 5 * (i % 4 == 3) for i in range(41))), gq=8, P=200, plens=(200, 0, 131, 64, 1)),
    dict(starts=tuple(range(0, 144, 2)), gq=2, hd=128, P=140, plens=(140, 129, 128, 0)),
    # more groups than the kernel for many rows keeps
    dict(starts=tuple(range(1031)), gq=1, Hkv=1, P=24, plens=(24, 1, 0, 17), own=4, lens=(4, 0, 1)),
    # more than 10240 and 40960 rows of all heads: row tiles in at most four pieces, and whole
    dict(starts=(0, 30, 41, 48), n=14, gq=8, P=1300, plens=(1300, 700, 129), own=20),
    dict(starts=(0, 48), n=14, gq=8, hd=128, P=1300, plens=(1290,), own=20),
    dict(starts=(0, 33, 59, 60), n=44, gq=8, P=900, plens=(900, 650, 0), own=20, counts=(44, 3, 0)),
    dict(starts=(0, 60), n=44, gq=8, hd=128, P=700, plens=(690,), own=20, counts=(44, 3)),
    # nothing but the prefix
    dict(starts=(0, 3), P=200, plens=(190,), own=0, lens=(0,), tree=False),
    dict(starts=(0, 90), P=200, plens=(190,), own=0, lens=(5,), tree=False, gq=4),
    dict(starts=(0, 3), n=6, P=200, plens=(190,), own=0, lens=(0,), tree=False, gq=4, kv="q8", q="f32"),
]


@pytest.mark.parametrize("i", range(len(MANY)))
def test_against_the_formula(i):
    p = Problem(**MANY[i], seed=i)
    p.call()
    p.check()
    assert torch.equal(p.out, p.call())
