"""The operators on 8-bit caches and the sampling of rows together, as a serving loop runs them: prompts
in, a tree verified on filtered rows, the accepted rows moved, one more token decoded and drawn.
Each step's output is compared with a plain computation in 64 bits from what the GPU held before."""
import numpy as np
import pytest
import torch

import chunk_ref as R
import q8_ref as Q

pytestmark = pytest.mark.gpu

B, N, HQ, HKV, BS, V = 3, 6, 8, 2, 16, 1000
PROMPTS = [37, 1, 150]
PARENTS = [[-1, 0, 0, 1, 1, 3], [-1, 0, 1, 2, 3, 4], [-1, 0, 0, 0, 2, 4]]
BLOCKS = 14


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    def __init__(self, tv, d, mode):
        from eagle_speculative_decoding_parent_gb300.pipeline import ChunkStep, VerifyStep
        self.tv, self.d, self.mode = tv, d, mode
        self.g = torch.Generator().manual_seed(d + mode)
        blocks = B * BLOCKS + 2
        codes = lambda: (torch.randn((blocks, HKV, BS, d), generator=self.g) * 90).clamp(-448, 448).to(Q.E4M3).cuda()  # noqa: E731
        scales = lambda: torch.exp2(torch.randint(-12, 8, (blocks, HKV), generator=self.g).float()).cuda()  # noqa: E731
        # (whatever was there before: a block starts anew with its first position)
        self.cache = dict(k_cache=codes(), v_cache=codes(), k_scale=scales(), v_scale=scales())
        self.table = torch.randperm(blocks, generator=self.g)[:B * BLOCKS].reshape(B, BLOCKS).to(torch.int32).cuda()
        self.counts = torch.zeros((B, V), dtype=torch.int32, device="cuda")
        self.draft = torch.randint(0, 8, (B, N), generator=self.g).to(torch.int32).cuda()
        self.raw = (torch.randn((B, N, V), generator=self.g) * 3).cuda()
        self.raw[:, :, :8] += 8.0                                    # some drafts are accepted
        f = lambda *x: torch.tensor(x, device="cuda")  # noqa: E731
        self.sampling = dict(counts=self.counts, presence=f(0.2, 0.4, 0.0), temperature=f(0.7, 1.0, 0.0 if mode else 1.5))
        if mode:
            self.sampling.update(top_k=i32([50, 0, 3]), top_p=f(0.95, 0.9, 1.0), min_p=f(0.0, 0.01, 0.0))
        q = torch.rand((B, N, V), generator=self.g) + 0.01
        self.draft_probs = (q / q.sum(-1, keepdim=True)).float().cuda() if mode else None
        self.rope = tv.rope_table(64, theta=5000.0, interleaved=True)
        sizes = dict(Hq=HQ, Hkv=HKV, d=d, dtype=torch.bfloat16, cache_dtype=torch.float8_e4m3fn)
        self.fill = ChunkStep(T=sum(PROMPTS), B=B, rope=self.rope, window=40, sinks=5, **sizes)
        self.one = ChunkStep(T=B, B=B, rope=self.rope, **sizes)
        self.step = VerifyStep(B=B, N=N, max_blocks=BLOCKS, bs=BS, max_path=N, V=V, mode=mode, process=True,
                               filters=bool(mode), **sizes)
        self.parents, self.prefix, self.ones = i32(PARENTS), i32(PROMPTS), i32(list(range(B + 1)))
        self.starts, self.zero = i32(np.cumsum([0] + PROMPTS).tolist()), i32([0] * B)
        self.act = [torch.randn((n, HQ + 2 * HKV, d), generator=self.g).bfloat16().cuda() for n in (sum(PROMPTS), B * N, B)]
        self.q_tree = torch.zeros((B * N, HQ, d), dtype=torch.bfloat16, device="cuda")
        self.st = torch.full((B,), -9, dtype=torch.int32, device="cuda")
        self.row = (torch.randn((B, 1, V), generator=self.g) * 2).bfloat16().cuda()
        self.uniform = torch.rand((B, 1), generator=self.g).cuda()
        self.token, self.st_token = (torch.full((B, 1), -9, dtype=torch.int32, device="cuda") for _ in range(2))

    def split(self, i):
        x = self.act[i]
        return dict(q=x[:, :HQ], k=x[:, HQ:HQ + HKV], v=x[:, HQ + HKV:], block_table=self.table, **self.cache)

    def prefill(self):
        return dict(q_start=self.starts, prefix_lens=self.zero, **self.split(0))

    def append_tree(self):
        self.tv.tree_mask_build(self.parents, self.step.mask, self.step.depth, self.step.st_mask)
        pos = (self.prefix[:, None] + self.step.depth).reshape(-1).contiguous()
        self.tv.chunk_kv_append_q8(status=self.st, q_start=i32([N * b for b in range(B + 1)]), prefix_lens=self.prefix,
                                   q_out=self.q_tree, rope=self.rope, positions=pos, **self.split(1))

    def verify(self):
        return dict(parents=self.parents, q=self.q_tree.view(B, N, HQ, self.d), prefix_lens=self.prefix, draft_tokens=self.draft,
                    target=self.raw, draft_probs=self.draft_probs, mode=self.mode, seed=11, offset=5, sampling=self.sampling,
                    block_table=self.table, **self.cache)

    def decode(self):
        return dict(q_start=self.ones, prefix_lens=self.step.new_lens, **self.split(2))

    def draw(self, stream=None):
        self.tv.logits_sample(self.row, self.uniform, self.token, self.st_token, top_k=i32([20, 1, 0]), stream=stream)

    def held(self, n, P, q, q_start):
        return dict(n=n, P=P, bs=BS, table=self.table.cpu(), q_start=q_start.cpu(), q=q.cpu().view(-1, HQ, self.d),
                    **{x: y.cpu().clone() for x, y in self.cache.items()})


def attended(c, out, **kw):
    ref, A, S = Q.attention(c, **kw)
    tol = R.attention_tolerance(c, ref, A, S, c["q"].shape[2])
    assert ((out.cpu().view(ref.shape).double() - ref).abs() <= tol).all()


def appended(before, s, n, P, v, q_start):
    """Values exactly (keys have their own tests)."""
    c = dict(before, n=n, P=P, q_start=q_start)
    code, scale = Q.append(c, "v", v.cpu().double())
    assert torch.equal(s.cache["v_cache"].view(torch.uint8).cpu(), code)
    assert torch.equal(s.cache["v_scale"].cpu().double(), scale)


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("mode", [0, 1])
def test_serving_loop(tv, orc, mode, d):
    s = Loop(tv, d, mode)
    before = s.held(PROMPTS, [0] * B, s.fill.q, s.starts)
    s.fill.run(**s.prefill())
    torch.cuda.synchronize()
    assert s.fill.st_append.eq(0).all() and s.fill.st_attn.eq(0).all()
    appended(before, s, PROMPTS, [0] * B, s.act[0][:, HQ + HKV:], s.starts.cpu())
    attended(s.held(PROMPTS, [0] * B, s.fill.q, s.starts), s.fill.out, window=40, sinks=5)
    # the tree
    before = s.held([N] * B, PROMPTS, s.q_tree, torch.arange(B + 1) * N)
    s.append_tree()
    torch.cuda.synchronize()
    assert s.st.eq(0).all()
    appended(before, s, [N] * B, PROMPTS, s.act[1][:, HQ + HKV:], torch.arange(B + 1) * N)
    c = s.held([N] * B, PROMPTS, s.q_tree, torch.arange(B + 1) * N)
    s.step.run(**s.verify())
    torch.cuda.synchronize()
    for st in (s.step.st_mask, s.step.st_attn, s.step.st_process, s.step.st_accept, s.step.st_counts, s.step.st_compact):
        assert st.eq(0).all()
    attended(c, s.step.out, mask=s.step.mask.view(-1).cpu())
    target = s.step.target.cpu()
    if mode:
        assert s.step.st_filter.eq(0).all()
        kw = {k: x.cpu().tolist() for k, x in s.sampling.items() if k != "counts"}
        # the rows before the filters: no temperature yet
        want = R.logits(s.raw.cpu(), mask=s.step.mask.cpu(), tokens=s.draft.cpu(), counts=torch.zeros((B, V), dtype=torch.int32),
                        pres=s.sampling["presence"].cpu())
        assert ((target.double() - want).abs() <= 7 * 2.0 ** -24 * 31).all()
        for b in range(B):
            for i in range(N):
                w, kept, near = Q.sample_sets(target[b, i], kw["temperature"][b], kw["top_k"][b], kw["top_p"][b], kw["min_p"][b])
                p = torch.where(kept, w, 0.0) / w[kept].sum()
                # an exponent of (logit - largest) / temperature <= 60 or so, rounded, and float32 sums
                got = s.step.filtered[b, i].cpu().double()
                assert torch.equal((got > 0)[~near], kept[~near]) and ((got - p).abs() <= p * (2.0 ** -20 + 2.0 ** -23 * 60)).all()
        target = s.step.filtered.cpu()
    args = (np.array(PARENTS, np.int32), s.draft.cpu().numpy(), target.numpy())
    acc = orc.accept_stochastic(*args, s.draft_probs.cpu().numpy(), 11, 5, N) if mode else orc.accept_greedy(*args, N)
    for t, r in zip((s.step.accept_len, s.step.path, s.step.out_tokens), acc):
        assert np.array_equal(t.cpu().numpy(), r)
    lens = [p + int(a) + 1 for p, a in zip(PROMPTS, acc[0])]
    assert s.step.new_lens.cpu().tolist() == lens
    for x in ("k", "v"):
        code, scale = Q.compact(c, x, torch.from_numpy(np.asarray(acc[1])), torch.from_numpy(np.asarray(acc[0])))
        assert torch.equal(s.cache[x + "_scale"].cpu().double(), scale)
        assert torch.equal(s.cache[x + "_cache"].cpu().float(), code.view(Q.E4M3).float())
    # one more token of each sequence, and the next one drawn
    before = s.held([1] * B, lens, s.one.q, s.ones)
    s.one.run(**s.decode())
    s.draw()
    torch.cuda.synchronize()
    assert s.one.st_append.eq(0).all() and s.one.st_attn.eq(0).all() and s.st_token.eq(0).all()
    appended(before, s, [1] * B, lens, s.act[2][:, HQ + HKV:], s.ones.cpu())
    attended(s.held([1] * B, lens, s.one.q, s.ones), s.one.out)
    for b, k in enumerate([20, 1, 0]):
        w, kept, _ = Q.sample_sets(s.row[b, 0].cpu(), 1.0, k, 1.0, 0.0)
        sums = torch.cumsum(torch.where(kept, w, 0.0), 0)
        assert int(s.token[b]) == int((sums > float(s.uniform[b]) * float(sums[-1])).nonzero()[0])


@pytest.mark.parametrize("mode", [0, 1])
def test_captured_loop_is_the_eager_one(tv, mode):
    def outputs(s):
        torch.cuda.synchronize()
        return [t.cpu().clone() for t in (s.fill.out, s.step.out, s.step.target, s.step.out_tokens, s.step.new_lens, s.one.out,
                                          s.counts, s.token, *s.cache.values())]

    a, b = Loop(tv, 128, mode), Loop(tv, 128, mode)
    a.fill.run(**a.prefill())
    a.append_tree()
    a.step.run(**a.verify())
    a.one.run(**a.decode())
    a.draw()
    want = outputs(a)
    state = {x: y.clone() for x, y in b.cache.items()}
    fill = b.fill.capture(**b.prefill())
    b.append_tree()
    verify = b.step.capture(**b.verify())
    one = b.one.capture(**b.decode())
    for _ in range(2):                                               # (and again from the same state)
        for x, y in state.items():
            b.cache[x].copy_(y)
        b.counts.zero_()
        fill.replay()
        b.append_tree()
        verify.replay()
        one.replay()
        b.draw()
        for x, y in zip(want, outputs(b)):
            assert torch.equal(x.view(torch.uint8) if x.dtype == Q.E4M3 else x, y.view(torch.uint8) if y.dtype == Q.E4M3 else y)


def test_refusals(tv):
    from eagle_speculative_decoding_parent_gb300.pipeline import ChunkStep, VerifyStep
    sizes = dict(Hq=HQ, Hkv=HKV, d=128, dtype=torch.bfloat16)
    verify = dict(B=B, N=N, max_blocks=BLOCKS, bs=BS, max_path=N, V=V, **sizes)
    with pytest.raises(ValueError):
        ChunkStep(T=3, B=3, sinks=4, **sizes)
    with pytest.raises(ValueError):
        ChunkStep(T=3, B=3, cache_dtype=torch.float8_e4m3fn, **dict(sizes, dtype=torch.float32))
    with pytest.raises(ValueError):
        VerifyStep(cache_dtype=torch.float8_e5m2, **verify)
    with pytest.raises(ValueError):
        VerifyStep(filters=True, process=True, **verify)
    with pytest.raises(ValueError):
        VerifyStep(filters=True, mode=1, **verify)
    s = Loop(tv, 128, 1)
    with pytest.raises(ValueError):
        s.step.run(**dict(s.verify(), node_counts=i32([N] * B)))
    s.step = VerifyStep(mode=1, process=True, cache_dtype=torch.float8_e4m3fn, **verify)
    with pytest.raises(ValueError):
        s.step.run(**s.verify())
