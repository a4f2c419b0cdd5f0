"""The small decoder over its paged cache: prompts, single tokens, batches of unequal lengths and drafted trees against the same
model in 64 bits."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import transpose_heroes_gb300 as hf
from test_decoder_gpu import PROMPT, model, reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from transpose_heroes_gb300 import build

    build.build()
    hf.lib()


def close(got, want):
    """As in test_decoder_gpu: the f32 products' errors are about 1e-5 of the logits' size."""
    assert float((got.cpu().double() - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_a_batch_of_unequal_prompts_then_tokens():
    from transpose_heroes_gb300.decoder import PagedCache

    m = model()
    texts = [PROMPT, PROMPT[3:8], [7], PROMPT[::-1] + [250]]
    longest = max(map(len, texts))
    cache = PagedCache(m, len(texts), longest + 3, page=4)
    cache.table = cache.table[:, torch.randperm(cache.table.shape[1])].contiguous()
    tokens = torch.tensor([t + [0] * (longest - len(t)) for t in texts], device="cuda")
    counts = torch.tensor([len(t) for t in texts], dtype=torch.int32, device="cuda")
    y = m.extend(tokens, cache, counts=counts)
    for i, t in enumerate(texts):
        close(y[i, :len(t)] @ m.head, reference(m, t)[0].detach())
    cache.lengths += counts
    for step in range(3):
        texts = [t + [(17 * step + i) % 300] for i, t in enumerate(texts)]
        y = m.extend(torch.tensor([t[-1:] for t in texts], device="cuda"), cache)
        cache.lengths += 1
        for i, t in enumerate(texts):
            close(y[i] @ m.head, reference(m, t)[0].detach()[-1:])


def test_every_node_of_a_tree_is_the_model_on_its_way():
    from transpose_heroes_gb300.decoder import PagedCache

    m = model()
    parents, nodes = [-1, 0, 0, 1, 1, 2, 5, 4], [5, 9, 2, 9, 7, 100, 101, 299]
    cache = PagedCache(m, 1, 40)
    m.extend(torch.tensor([PROMPT[:-1]], device="cuda"), cache)
    cache.lengths += len(PROMPT) - 1
    bits, depths = (torch.from_numpy(x).cuda() for x in hf.tree_mask(parents))
    y = m.extend(torch.tensor([nodes], device="cuda"), cache, mask=bits, depths=depths)[0] @ m.head
    for c in range(len(nodes)):
        way, u = [], c
        while u >= 0:
            way.append(nodes[u])
            u = parents[u]
        close(y[c], reference(m, PROMPT[:-1] + way[::-1])[0].detach()[-1])


@pytest.mark.parametrize("draft", [1, 4, 9])
def test_drafts_do_not_change_what_is_generated(draft):
    m = model()
    for t in m.parameters():
        t.requires_grad_(True)
    opt = torch.optim.Adam(m.parameters(), lr=2e-3)
    text = [3, 1, 4, 1, 5, 9, 2, 6]
    for step in range(30):  # a model that repeats itself, so that drafts are accepted
        opt.zero_grad()
        m.loss(torch.tensor(text * 6, device="cuda")).backward()
        opt.step()
    prompt = text * 2 + text[:3]
    steps = []
    extend = m.extend
    m.extend = lambda *a, **k: steps.append(1) or extend(*a, **k)
    want = m.generate(prompt, 12)
    plain = len(steps)
    assert m.generate(prompt, 12, draft=draft) == want and len(steps) - plain < plain
    for kw in (dict(frequency=0.3), dict(repetition=1.2, presence=0.1)):
        assert m.generate(prompt, 9, draft=draft, **kw) == m.generate(prompt, 9, **kw)
    bits = np.zeros(10, np.uint32)
    for v in (1, 4, 5, 9):
        bits[v // 32] |= np.uint32(1 << (v % 32))
    mask = torch.from_numpy(bits.view(np.int32)).cuda()
    got = m.generate(prompt, 8, mask=mask, draft=draft)
    assert got == m.generate(prompt, 8, mask=mask) and set(got) <= {1, 4, 5, 9}
    assert m.generate(prompt, 8, mask=torch.zeros_like(mask), draft=draft) == []


def test_draft_trees():
    from transpose_heroes_gb300.decoder import draft_tree

    nodes, parents = draft_tree([3, 1, 4, 1, 5, 9, 3, 1, 4, 2, 3, 1], 6)
    assert (nodes, parents) == ([1, 4, 2, 3, 1, 1, 5], [-1, 0, 1, 2, 3, 1, 5])
    assert draft_tree([3], 6) == ([3], [-1]) and draft_tree([1, 2, 3], 6) == ([3], [-1])
    for tokens in ([7, 7, 7, 7], [1, 2, 1, 2, 1, 2, 1]):
        for most in (1, 2, 5):
            nodes, parents = draft_tree(tokens, most)
            assert len(nodes) <= most + 1 and all(p < c for c, p in enumerate(parents)) and nodes[0] == tokens[-1]
            kids = [(p, t) for p, t in zip(parents, nodes)]
            assert len(set(kids)) == len(kids)
