"""README's round of parallel continuations runs as it is written."""
import os

import pytest
import torch

from speculative_decoding_verification_pass_gb300 import binding as sb

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("schedule", ["persistent", "per_step"])
def test_parallel_continuations(schedule, monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    if schedule == "per_step":
        monkeypatch.setenv("SPEC_FORWARD_PERSISTENT", "0")
    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    (code,) = [x.split("```")[0] for x in text.split("```python\n")[1:] if "sb.Pages(kv)" in x]
    cfg = sb.ModelConfig(2, 256, 4, 2, 256, 1000)
    names = dict(torch=torch, sb=sb, cfg=cfg, model=sb.Model(cfg, 7), gamma=4)
    exec(code, names)  # noqa: S102
    assert (names["status"], names["bits"]) == (sb.SPEC_OK, 0)
    assert not names["late"].any()
    n = names["n_acc"].tolist()
    assert names["kv"].len.tolist() == [301 + x for x in n]
    assert [[t >= 0 for t in row] for row in names["out"].tolist()] == [[i <= x for i in range(5)] for x in n]
    assert names["pages"].n_free.item() == 512 - 4 - 4  # four full pages once, and each its own last one
    names["model"].close()
