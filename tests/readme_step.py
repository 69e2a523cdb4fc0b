"""The serving step as README.md shows it, run as a server would: a few steps of
a few requests, of which one ends, over a pool that they nearly fill."""
import os

import torch

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def serving_step():
    """The code block's part up to the training lines."""
    text = open(README, encoding="utf-8").read()
    block = next(b for b in text.split("```python\n")[1:] if "diffattn_page_plan" in b)
    code = block.split("```")[0]
    return compile(code[:code.index("# training")], README, "exec")


def run(da, device):
    """Runs three steps; after each, every page is free or one request's, once."""
    page, n_pages, max_pages, Hq, Hkv = 64, 12, 8, 4, 2
    i32 = dict(dtype=torch.int32, device=device)
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(device)
    ns = dict(da=da, lens=torch.zeros(3, **i32), free_count=torch.full((1,), n_pages, **i32),
              free_pages=torch.arange(n_pages, **i32),
              block_table=torch.full((3, max_pages), -1, **i32),
              cache=torch.zeros(n_pages, Hkv, page * 144, dtype=torch.uint8, device=device),
              inv_freq=torch.ones(64, device=device), wq=torch.ones(128, device=device),
              wk=torch.ones(128, device=device), lam_pairs=torch.full((Hq // 2,), 0.5,
                                                                      device=device))
    step = serving_step()
    total = [0, 0, 0]
    for new, gone in (([70, 200, 64], [0, 0, 0]), ([1, 1, 1], [0, 1, 0]), ([65, 300, 1], [0, 0, 0])):
        n = sum(new)
        ns.update(new_lens=torch.tensor(new, **i32), finished=torch.tensor(gone, **i32), n_tokens=n,
                  q=rnd(n, Hq, 128), k=rnd(n, Hkv, 128), v=rnd(n, Hkv, 128))
        exec(step, ns)
        total = [0 if e else t + x for t, x, e in zip(total, new, gone)]
        assert ns["lens"].tolist() == total
        table, free = ns["block_table"].tolist(), ns["free_pages"].tolist()
        held = [row[j] for row, t in zip(table, total) for j in range(-(-t // page))]
        pool = held + free[:int(ns["free_count"])]
        assert sorted(pool) == list(range(n_pages)), (held, pool)
        assert ns["out"].shape == (3, Hq // 2, 128) and torch.isfinite(ns["out"].float()).all()
