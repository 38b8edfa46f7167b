"""The README's optimizer example, as it is written there."""
import os
import re
import textwrap

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_two_optimizers_of_one_seed_share_no_random_numbers():
    """Matrices by Muon, the rest by AdamW: with one seed, every element's global
    position (which picks its random bits) is its own."""
    from stochastic_rounding_gb300 import AdamWSR, MuonSR
    with open(os.path.join(ROOT, "README.md")) as f:
        text = f.read()
    block = re.search(r"\n( +# matrices by Muon.*?)\n\n", text, re.S).group(1)
    model = torch.nn.Sequential(torch.nn.Linear(8, 6), torch.nn.LayerNorm(6), torch.nn.Linear(6, 4))
    names = dict(model=model, AdamWSR=AdamWSR, MuonSR=MuonSR)
    exec(textwrap.dedent(block), names)
    taken = []
    for opt in (names["muon"], names["adamw"]):
        assert opt.param_groups[0]["seed"] == 1234
        for p in opt.param_groups[0]["params"]:
            taken.append((opt.base_index(p), opt.base_index(p) + p.numel()))
    assert sum(b - a for a, b in taken) == sum(p.numel() for p in model.parameters())
    taken.sort()
    assert all(b <= c for (_, b), (c, _) in zip(taken, taken[1:]))
