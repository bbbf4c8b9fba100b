"""That the products tested on the GPU for their tiles take every tile that products of any size take."""
import ctypes
import math
import random

import pytest

import routed_expert_ffn_moe_amd as moe
from train_shapes import CASES, taken


def test_cases_take_every_tile():
    have = {taken(way, *c) for way, cases in CASES.items() for c in cases}
    rng = random.Random(3)

    def size(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    missing = {}
    for _ in range(60000):
        N, K = size(8, 8192), size(8, 8192)
        if rng.random() < 0.75:
            N, K = -(-N // 8) * 8, -(-K // 8) * 8
        M, G = size(1, 1 << 17), rng.choice([1, size(2, 512), size(513, 4096)])
        for way in CASES:
            t = taken(way, M, N, K, G)
            if t not in have:
                missing.setdefault(t, (M, N, K, G))
    assert not missing, missing


def test_alignment_decides_the_kernel():
    for way in CASES:
        m = moe.make_matmul_bf16(300, 256, 512)
        assert moe.moe_matmul_bf16_tile(m, way)[3] == 1
        assert moe.moe_matmul_bf16_tile(m, way, off16=True)[3] == 0
        assert moe.moe_matmul_bf16_tile(moe.make_matmul_bf16(300, 256, 512, ldx=513, ldy=257), way)[3] == 0
        assert moe.moe_matmul_bf16_tile(moe.make_matmul_bf16(300, 250, 509), way)[3] == 0


@pytest.mark.parametrize("bad", [dict(M=-1), dict(N=0), dict(K=0), dict(G=0), dict(G=65536), dict(out_dtype=2),
                                 dict(ldx=7), dict(ldw=7), dict(ldy=7)])
def test_tile_refusals(bad):
    d = dict(M=4, N=8, K=8, G=1, out_dtype=0, ldx=0, ldw=0, ldy=0)
    d.update(bad)
    with pytest.raises(moe.MoeError, match="moe_matmul_bf16_tile"):
        moe.moe_matmul_bf16_tile(moe.moe_matmul_bf16_t(**d), "y")


def test_tile_refuses_other_ways_and_null():
    lib, tile = moe.load(), (ctypes.c_int32 * 4)()
    m = moe.make_matmul_bf16(4, 8, 8)
    for way, at, what in ((3, tile, ctypes.byref(m)), (-1, tile, ctypes.byref(m)), (0, None, ctypes.byref(m)), (0, tile, None)):
        assert lib.moe_matmul_bf16_tile(what, way, 0, at) == moe.MOE_EINVAL
        assert "moe_matmul_bf16_tile" in moe.moe_last_error()
