"""The 8-bit attention's launches hold to the rules that choose them: splits merge as clusters, and rows go by
eights, only where the device holds all of the grid at once."""
import pytest
import torch

from launches import kernels

pytestmark = pytest.mark.gpu
FMT = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


@pytest.fixture(scope="module")
def ext():
    from paged_kv_sink_gb300 import build
    build.build()
    import paged_kv_sink_gb300 as ext
    return ext


def launches(ext, fmt, d, hkv, group, batch, new, tokens, causal=True):
    """attend_kernel's launch for `batch` requests of up to `tokens` tokens and `new` rows (captured, not run)."""
    kind = FMT[fmt]
    cache = [torch.zeros(1, 16, hkv, d, dtype=torch.uint8, device="cuda").view(kind) for _ in range(2)]
    cache += [torch.ones(1, 1, hkv, device="cuda") for _ in range(2)]
    table = torch.zeros(batch, -(-tokens // 16), dtype=torch.int32, device="cuda")
    lens = torch.full((batch,), tokens, dtype=torch.int32, device="cuda")
    q = torch.zeros(batch * new, hkv * group, d, dtype=torch.bfloat16, device="cuda")
    cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * new
    if new == 1 and causal:
        call = lambda: ext.attn_sink_decode_paged_q8(q, *cache, table, lens)
    else:
        call = lambda: ext.attn_sink_fwd_paged_q8(q, *cache, table, cu, lens, new, tokens, causal=causal)
    return [k for k in kernels(call) if "attend_kernel" in k["name"]]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,new,causal", [(8, 1, True), (1, 1, True), (20, 1, True), (8, 3, True), (4, 2, True), (4, 16, True), (8, 2, False)])
def test_clusters_and_tiles_of_eight_are_resident(ext, fmt, d, group, new, causal):
    """Batches across the border: whatever a launch merges in clusters, and whatever takes more than 8 rows of a KV
    head in tiles of 8, is resident at once."""
    seen = dict(merged=0, split=0)
    for tokens in (300, 700, 1100, 2000):
        for batch in (1, 2, 5, 9, 12, 16, 19, 22, 23, 24, 25, 28, 30, 33, 36, 38, 40, 45, 47, 50, 55, 57, 63, 76, 90, 95, 100, 114):
            for k in launches(ext, fmt, d, 8, group, batch, new, tokens, causal):
                ctas = k["grid"][0] * k["grid"][1] * k["grid"][2]
                rows, tiles = group * new, k["grid"][1] // 8
                where = (tokens, batch, k)
                if k["cluster"] > 1:
                    seen["merged"] += 1
                    assert ctas <= k["resident"], where
                elif k["grid"][0] > 1:
                    seen["split"] += 1
                if rows > 8 and tiles == -(-rows // 8):
                    assert ctas <= k["resident"], where
    assert seen["merged"] > 0
    assert seen["split"] > 0 or group * new > (64 if d == 64 else 32)  # (so many rows are split only where they merge)
