"""Pins for oracle.attention (CPU only): against torch's scaled dot product and its
autograd in float64, against differences, and the page allocator against its own rules."""
import numpy as np
import pytest
import torch

import oracle.attention as OA


@pytest.mark.parametrize("lq,lk,causal", [(1, 1, True), (7, 7, True), (5, 9, True), (6, 6, False), (4, 11, False)])
def test_forward_and_gradients_match_autograd(lq, lk, causal):
    rng = np.random.default_rng(lq * 100 + lk)
    heads, kv, d, scale = 4, 2, 8, 0.3
    q, k, v, g = (rng.standard_normal(s) for s in ((lq, heads, d), (lk, kv, d), (lk, kv, d), (lq, heads, d)))
    t = [torch.tensor(a, requires_grad=True) for a in (q, k, v)]
    mask = torch.ones(lq, lk, dtype=torch.bool) if not causal else torch.ones(lq, lk).tril(lk - lq).bool()
    wide = [t[0].transpose(0, 1)] + [a.transpose(0, 1).repeat_interleave(heads // kv, 0) for a in t[1:]]
    o = torch.nn.functional.scaled_dot_product_attention(*wide, attn_mask=mask, scale=scale).transpose(0, 1)
    (o * torch.tensor(g)).sum().backward()
    cu_q, cu_k = [0, lq], [0, lk]
    got, lse = OA.attention_forward(q, k, v, cu_q, cu_k, scale, causal)
    np.testing.assert_allclose(got, o.detach().numpy(), rtol=1e-10, atol=1e-12)
    z = scale * np.einsum("ihd,jhd->hij", q, np.repeat(k, heads // kv, 1))
    np.testing.assert_allclose(lse, torch.logsumexp(torch.tensor(np.where(mask.numpy(), z, -np.inf)), -1).numpy(), rtol=1e-12)
    grads = OA.attention_backward(g, q, k, v, got, lse, cu_q, cu_k, scale, causal)
    for a, b in zip(grads, t):
        np.testing.assert_allclose(a, b.grad.numpy(), rtol=1e-9, atol=1e-11)


def test_gradients_match_differences_on_packed_sequences():
    rng = np.random.default_rng(5)
    cu_q, cu_k, scale = [0, 3, 3, 8, 9], [0, 5, 7, 11, 11], 0.5   # (a sequence of keys alone, rows without keys)
    q, k, v, g = (rng.standard_normal(s) for s in ((9, 2, 4), (11, 1, 4), (11, 1, 4), (9, 2, 4)))
    o, lse = OA.attention_forward(q, k, v, cu_q, cu_k, scale)
    assert np.all(o[3] == 0) and np.all(np.isinf(lse[:, 3])) and np.all(o[8] == 0)
    grads = OA.attention_backward(g, q, k, v, o, lse, cu_q, cu_k, scale)
    loss = lambda: np.sum(OA.attention_forward(q, k, v, cu_q, cu_k, scale)[0] * g)  # noqa: E731
    for x, dx in zip((q, k, v), grads):
        num = np.zeros(x.shape)
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + 1e-5
            up = loss()
            x[i] = keep - 1e-5
            num[i] = (up - loss()) / 2e-5
            x[i] = keep
        np.testing.assert_allclose(dx, num, rtol=1e-5, atol=1e-8)


def test_page_allocator_keeps_every_page_once():
    rng = np.random.default_rng(7)
    n, page, n_pages, width = 9, 4, 40, 12
    lens, table = [0] * n, [[-7] * width for _ in range(n)]
    ring, state = list(rng.permutation(n_pages)), (0, n_pages)
    for step in range(60):
        new = [(-1 if rng.random() < 0.2 else 0) if c > 30 else int(rng.integers(0, 7)) for c in lens]
        before = list(lens)
        lens, cu, slots, pos, seqs, state, short = OA.kv_tables(lens, new, table, ring, state, page, 64)
        held = [table[b][j] for b in range(n) for j in range(-(-lens[b] // page))]
        free = [ring[i % n_pages] for i in range(*state)]
        assert sorted(held + free) == list(range(n_pages)), step
        for b in range(n):
            mine = slots[cu[b]:cu[b + 1]]
            if new[b] > 0 and lens[b] == before[b]:
                assert short and mine == [-1] * new[b]
            else:
                assert mine == [table[b][p // page] * page + p % page for p in range(before[b], before[b] + max(new[b], 0))]
            assert pos[cu[b]:cu[b + 1]] == list(range(before[b], before[b] + max(new[b], 0)))
            assert seqs[cu[b]:cu[b + 1]] == [b] * max(new[b], 0)
        assert slots[cu[-1]:] == [-1] * (64 - cu[-1])


def test_cache_rows():
    cache = np.arange(5 * 2 * 4 * 3).reshape(5, 2, 4, 3)
    rows = OA.cache_rows(cache, [3, 0], 6)
    assert rows.shape == (6, 2, 3) and np.array_equal(rows[5], cache[0, :, 1]) and np.array_equal(rows[0], cache[3, :, 0])
