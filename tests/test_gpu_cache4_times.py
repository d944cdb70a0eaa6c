"""Which kernels serve a call of the 4-bit cache: a call that has less to do than another takes no longer by much. The
bounds leave room for noise; the wrong kernels take 1.4 to three times as long."""
import pytest
import torch

from kv_cache_quantization_token_gb300 import kvarn

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MUCH = 1.5


def _time(call, calls=10):
    """us of a call, the best of several replays of a graph of them."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            call()
    best = float("inf")
    for _ in range(12):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) / calls * 1e3)
    return best


@pytest.mark.parametrize("D,Hkv,C,n", [(64, 2, 48, 1024), (128, 1, 96, 512), (256, 2, 48, 512)])
def test_a_chunk_over_a_long_table_takes_no_longer_than_a_larger_one(D, Hkv, C, n):
    """Few KV heads and long contexts, where going over the cache once for every eight rows costs most."""
    G, lay = 4, kvarn.layout4(D)
    tiles = torch.zeros(Hkv * n * lay.record_bytes, dtype=torch.uint8, device=DEV)
    table = (torch.arange(Hkv * n, device=DEV) * lay.record_bytes).view(Hkv, n)

    def run(C):
        q = torch.randn(C, Hkv * G, D, device=DEV).bfloat16()
        out, ws = torch.empty_like(q), torch.empty(kvarn.prefill4_workspace_bytes(C, n, Hkv * G, Hkv, D), dtype=torch.uint8, device=DEV)
        return _time(lambda: kvarn.prefill_attention4(q, 128 * n - C, tiles, table, lay, ws=ws, out=out))

    assert run(C) <= MUCH * run(C + C // 2)
    assert kvarn.device_error() == 0


@pytest.mark.parametrize("D,G,n", [(64, 4, 6), (128, 4, 1), (128, 8, 3)])
def test_many_short_tables_take_no_longer_than_the_same_tiles_of_wide_ones(D, G, n):
    """2,048 segments of a few tiles: a block for each would come in rounds that begin and end for themselves."""
    B, Hkv, lay = 256, 8, kvarn.layout4(D)
    tiles = torch.zeros(B * Hkv * n * lay.record_bytes, dtype=torch.uint8, device=DEV)
    table = (torch.arange(B * Hkv * n, device=DEV) * lay.record_bytes).view(B, Hkv, n)
    lens = torch.full((B,), 128 * n - 5, dtype=torch.int32, device=DEV)
    q = torch.randn(B, Hkv * G, D, device=DEV).bfloat16()

    def run(width):  # columns behind a sequence's tiles are not read; a table of 40 columns is shared out
        wide = torch.nn.functional.pad(table, (0, width - n), value=-16).contiguous()
        out, ws = torch.empty_like(q), torch.empty(kvarn.decode4_workspace_bytes(B, Hkv * G, Hkv, D, width), dtype=torch.uint8, device=DEV)
        return _time(lambda: kvarn.decode_attention4(q, tiles, wide, lens, lay, ws=ws, out=out))

    assert run(n) <= 1.2 * run(40)
    assert kvarn.device_error() == 0
