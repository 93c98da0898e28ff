"""The plan queries of the experts' operators and of the balance loss (no GPU
needed): the tiles at sizes on both sides of each rule, and the refusals of
the calls themselves."""
import ctypes as C

import pytest

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B


def product(E, mean, n, out=M.BF16):
    p = M.ep_expert_plan_query(M.moedisp_rows.contiguous(E, 1 << 20, mean), n, 256, M.SCALE_FP32, out)
    return p["product_rows"], p["product_cols"]


@pytest.mark.parametrize("E,mean,n,tile", [
    (64, 8, 4096, (32, 128)), (64, 24, 4096, (64, 256)), (64, 48, 4096, (96, 256)), (64, 96, 4096, (128, 256)),
    (64, 128, 4096, (160, 256)), (64, 192, 4096, (256, 256)),
    (33, 64, 1656, (64, 256)), (24, 125, 1000, (64, 256)),                  # few tiles: small ones
    (12, 206, 2216, (128, 256)), (9, 335, 3536, (256, 256)),                # whole rounds of the largest
    (1, 2 ** 31 - 1, 8, (256, 256))])
def test_product_tiles(E, mean, n, tile):
    assert product(E, mean, n) == tile
    assert product(E, mean, n, M.FP32) == (min(tile[0], 128), tile[1])


def test_wgrad_tiles():
    def tile(E, n, k):
        p = M.ep_expert_plan_query(M.moedisp_rows.contiguous(E, 64), n, k, M.SCALE_UE8M0, M.BF16)
        return p["wgrad_cols"], p["wgrad_channels"]
    assert tile(8, 4096, 4096) == (256, 256) and tile(64, 7168, 2048) == (256, 256)
    assert tile(8, 512, 512) == (128, 128) and tile(52, 2008, 128) == (128, 128)
    assert tile(35, 3264, 1536) == (256, 256) and tile(13, 1048, 3328) == (128, 128)

    def exact(E, n, k):
        p = M.ep_expert_plan_query(M.moedisp_rows.contiguous(E, 64), n, k, M.SCALE_FP32, M.FP32)
        return p["wgrad_cols"], p["wgrad_channels"]
    assert exact(8, 4096, 4096) == exact(24, 1000, 640) == (256, 128) and exact(8, 512, 512) == (128, 128)


def test_balance_tiles():
    for S, L, E, k in ((64, 2048, 256, 8), (4, 1024, 256, 8), (1, 1, 1, 1), (3, 5000, 4096, 32), (70000, 2, 8, 1)):
        p = M.ep_balance_plan_query(M.moedisp_balance.make(S, L, E, k))
        assert p["tile_tokens"] == p["passes"] * p["rows_at_once"] and p["rows_at_once"] * p["lanes"] == 256
        assert (p["tiles"] - 1) * p["tile_tokens"] < L <= p["tiles"] * p["tile_tokens"]


def test_refusals():
    rows = M.moedisp_rows.contiguous(4, 16)
    for args, code in (((M.moedisp_rows(0, 16), 8, 128, 0, 0), B.ERR_INVALID_ARG),
                       ((rows, 12, 128, 0, 0), B.ERR_UNSUPPORTED), ((rows, 8, 100, 0, 0), B.ERR_UNSUPPORTED),
                       ((rows, 8, 128, 2, 0), B.ERR_UNSUPPORTED), ((rows, 8, 128, 0, 1), B.ERR_UNSUPPORTED)):
        with pytest.raises(M.MoeDispError) as e:
            M.ep_expert_plan_query(*args)
        assert e.value.code == code
    with pytest.raises(M.MoeDispError) as e:
        M.ep_balance_plan_query(M.moedisp_balance.make(1, 1, 4, 5))
    assert e.value.code == B.ERR_INVALID_ARG
    L = M.load()
    assert L.ep_expert_plan_query(C.byref(rows), 8, 128, 0, 0, None, 64) == B.ERR_INVALID_ARG
    info = B.moedisp_expert_plan_info()
    assert L.ep_expert_plan_query(C.byref(rows), 8, 128, 0, 0, C.byref(info), 8) == B.ERR_INVALID_ARG
    b = M.moedisp_balance.make(1, 1, 4, 1)
    assert L.ep_balance_plan_query(C.byref(b), None, 56) == B.ERR_INVALID_ARG


def test_backward_reads_of_the_token_counts():
    """Every workgroup of the backward pass reads all S token counts: their
    number does not grow with S, so neither do the reads of a sequence."""
    for S, L in ((1, 1), (300, 2), (2048, 7), (4096, 1), (4097, 1), (65536, 16), (1 << 20, 1)):
        p = M.ep_balance_plan_query(M.moedisp_balance.make(S, L, 64, 2))
        assert p["backward_blocks"] <= min(4096, S * p["tiles"])
