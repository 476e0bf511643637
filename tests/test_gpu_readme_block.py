"""The README's second example (the block operators) runs as written."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_block_example_runs():
    kq = pytest.importorskip("w4a4_post_quantization_b200")
    text = open(os.path.join(ROOT, "README.md")).read()
    blocks = re.findall(r"```python\n(.*?)```", text, flags=re.S)
    import torch
    scope = {"torch": torch, "kq": kq}
    exec(compile(blocks[1], "README.md", "exec"), scope)
    assert tuple(scope["out"].shape) == (2, 1024, 16, 72) and tuple(scope["y"].shape) == (2048, 1152)
    assert scope["y"].isfinite().all() and kq.device_status() == 0
