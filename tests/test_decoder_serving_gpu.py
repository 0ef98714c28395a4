"""The decoder-layer example with planned pages, turned queries and keys and a 4-bit cache: where pages lie changes no bit."""
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decoder_layer", PATH)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    return ex


@pytest.mark.parametrize("rotate", [False, True])
@pytest.mark.parametrize("fmt", ["native", "fp8", "mxfp4"])
def test_planned_pages_change_nothing(example, fmt, rotate):
    apart, planned = (example.compare(fmt, rotate=rotate, pool=pool) for pool in (False, True))
    print(f"[decoder layer] {fmt} rotate {rotate}: {planned}", flush=True)
    assert apart == planned and all(math.isfinite(x) for x in planned)


def test_turned_pieces_agree_with_whole_prompts(example):
    # the same roundings as without turning, and one more of queries and keys: the bound of the pieces without it
    assert all(x <= 0.1 for x in example.compare("native", rotate=True, pool=True))
