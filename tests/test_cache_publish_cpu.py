"""Orders in the cache attention's source that the memory model asks for and no run can show the lack of."""
import os
import re

SOURCE = os.path.join(os.path.dirname(__file__), os.pardir, "precision_attention_nvfp4_b200", "csrc", "cache_attn.cu")


def test_what_a_tile_holds_is_written_before_the_arrival_that_publishes_it():
    """The readers of good[] (and of issued[]) wait for the tile's barrier: only what precedes the loading thread's
    arrival there is released to them. Its lanes' later arrivals track copies and release nothing."""
    with open(SOURCE) as f:
        body = f.read().split("void load_tiles(", 1)[1].split("\ntemplate", 1)[0]
    arrive = [m.start() for m in re.finditer(r"mbar_arrive_expect_tx\(", body)]
    stores = [m.start() for m in re.finditer(r"\b(good\[st\]|issued\[is_v\]) = ", body)]
    assert len(arrive) == 1 and len(stores) == 2
    assert max(stores) < arrive[0]
