"""The operators on chunks and on a tree's logits together with the tree's own calls, as a
serving loop runs them: prompts in, a tree verified on sampled rows, the accepted rows moved,
one more token decoded.  Each step's output is compared with a plain computation in 64 bits
from what the GPU held before that step."""
import threading

import numpy as np
import pytest
import torch

import chunk_ref as R
from gpu_util import host_f32

pytestmark = pytest.mark.gpu

B, N, HQ, HKV, D, BS, V = 3, 6, 8, 2, 128, 16, 1000
PROMPTS = [37, 1, 150]
PARENTS = [[-1, 0, 0, 1, 1, 3], [-1, 0, 1, 2, 3, 4], [-1, 0, 0, 0, 2, 4]]
BLOCKS = 14                                     # per sequence: 224 positions


@pytest.fixture(scope="module")
def tv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import eagle_speculative_decoding_parent_gb300 as m
    return m


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Loop:
    """A model's state and made-up activations; every random tensor from one seed."""

    def __init__(self, tv, mode, dtype):
        from eagle_speculative_decoding_parent_gb300.pipeline import ChunkStep, VerifyStep
        self.tv, self.mode, self.dtype = tv, mode, dtype
        self.g = torch.Generator().manual_seed(7 + mode)
        self.rope = dict(dim=64, theta=5000.0, interleaved=True)
        self.k_cache = self.rand(B * BLOCKS + 2, HKV, BS, D)
        self.v_cache = self.rand(B * BLOCKS + 2, HKV, BS, D)
        self.table = torch.randperm(B * BLOCKS + 2, generator=self.g)[:B * BLOCKS].reshape(
            B, BLOCKS).to(torch.int32).cuda()
        self.counts = torch.full((B, V), -5, dtype=torch.int32, device="cuda")
        self.prompt = torch.randint(0, V, (sum(PROMPTS),), generator=self.g).to(torch.int32).cuda()
        # few draft tokens, so that paths repeat tokens and meet the prompt's
        self.draft = torch.randint(0, 8, (B, N), generator=self.g).to(torch.int32).cuda()
        self.raw = (torch.randn((B, N, V), generator=self.g) * 3).cuda()
        self.raw[:, :, :8] += 8.0              # some drafts are accepted
        self.sampling = dict(
            counts=self.counts, repetition=torch.tensor([1.2, 1.0, 0.8], device="cuda"),
            frequency=torch.tensor([0.1, 0.0, 0.3], device="cuda"),
            presence=torch.tensor([0.2, 0.4, 0.0], device="cuda"),
            temperature=torch.tensor([0.7, 1.0, 1.5], device="cuda"),
            grammar=torch.randint(-2**31, 2**31, (B, N, (V + 31) // 32), generator=self.g).to(
                torch.int32).cuda() | 1)
        q = torch.rand((B, N, V), generator=self.g) + 0.01
        self.draft_probs = (q / q.sum(-1, keepdim=True)).float().cuda() if mode else None
        table = tv.rope_table(**self.rope)
        sizes = dict(Hq=HQ, Hkv=HKV, d=D, dtype=dtype)
        self.fill = ChunkStep(T=sum(PROMPTS), B=B, rope=table, **sizes)
        self.one = ChunkStep(T=B, B=B, rope=table, **sizes)
        self.step = VerifyStep(B=B, N=N, max_blocks=BLOCKS, bs=BS, max_path=N, V=V, mode=mode,
                               process=True, **sizes)
        self.parents = i32(PARENTS)
        self.prompt_act, self.tree_act, self.one_act = (
            self.rand(n, HQ + 2 * HKV, D) for n in (sum(PROMPTS), B * N, B))
        self.q_tree = torch.zeros((B * N, HQ, D), dtype=dtype, device="cuda")
        self.st = torch.full((B,), -9, dtype=torch.int32, device="cuda")

    def rand(self, *shape):
        return torch.randn(shape, generator=self.g).to(self.dtype).cuda()

    @staticmethod
    def split(x):
        return dict(q=x[:, :HQ], k=x[:, HQ:HQ + HKV], v=x[:, HQ + HKV:])

    def caches(self):
        return dict(k_cache=self.k_cache, v_cache=self.v_cache, block_table=self.table)

    def prefill_args(self):
        lens = torch.tensor([0] + PROMPTS).cumsum(0).to(torch.int32).cuda()
        self.starts, self.zero = lens, i32([0] * B)
        return dict(q_start=lens, prefix_lens=self.zero, **self.split(self.prompt_act), **self.caches())

    def append_tree(self):
        """The tree's nodes through the chunk call: rows at P + i, rotated by P + depth."""
        self.tv.tree_mask_build(self.parents, self.step.mask, self.step.depth, self.step.st_mask)
        self.positions = (self.prefix[:, None] + self.step.depth).reshape(-1).contiguous()
        self.tv.chunk_kv_append(status=self.st, q_start=i32([N * b for b in range(B + 1)]),
                                prefix_lens=self.prefix, q_out=self.q_tree,
                                rope=self.fill.rope, positions=self.positions,
                                **self.split(self.tree_act), **self.caches())

    def verify_args(self):
        return dict(parents=self.parents, q=self.q_tree.view(B, N, HQ, D), prefix_lens=self.prefix,
                    draft_tokens=self.draft, target=self.raw, draft_probs=self.draft_probs,
                    mode=self.mode, seed=11, offset=5, sampling=self.sampling, **self.caches())

    def decode_args(self):
        return dict(q_start=self.ones, prefix_lens=self.step.new_lens,
                    **self.split(self.one_act), **self.caches())


def rotated(loop, act, pos):
    f, amp = R.frequencies(loop.rope["dim"], loop.rope["theta"], "none", 1.0, 0, 1.0, 4.0)
    q, k, v = (x.double().cpu() for x in Loop.split(act).values())
    pos = pos.cpu()
    return R.rotate(q, pos, f, amp, True), R.rotate(k, pos, f, amp, True), v


def rows_of(loop, cache, b, n):
    """The first n positions of sequence b, [n, Hkv, D]."""
    t = torch.arange(n)
    return cache.cpu()[loop.table.cpu()[b][t // BS].long(), :, t % BS]


def half_step(x, dtype):
    """Float32 rotation (12 roundings of a pair) and the rounding to the cache's type."""
    return x.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24) * 1.01 + 12 * 1.5 * 6 * 2.0 ** -24


def check_append(loop, act, pos, n, P, q_got):
    q, k, v = rotated(loop, act, pos)
    assert (q_got.cpu().double() - q).abs().le(half_step(q, loop.dtype)).all()
    at = 0
    for b in range(B):
        new = slice(P[b], P[b] + n[b])
        kc = rows_of(loop, loop.k_cache, b, P[b] + n[b])[new].double()
        assert (kc - k[at:at + n[b]]).abs().le(half_step(k[at:at + n[b]], loop.dtype)).all()
        assert torch.equal(rows_of(loop, loop.v_cache, b, P[b] + n[b])[new].double(), v[at:at + n[b]])
        at += n[b]


def check_chunk_attention(loop, step, q_start, n, P):
    c = dict(n=n, P=P, bs=BS, table=loop.table.cpu(), q_start=q_start.cpu(), prefix=torch.tensor(P),
             q=step.q.cpu(), k_cache=loop.k_cache.cpu(), v_cache=loop.v_cache.cpu())
    ref, A, S = R.attention(c)
    assert (step.out.cpu().double() - ref).abs().le(R.attention_tolerance(c, ref, A, S, D)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", [0, 1])
def test_serving_loop(tv, orc, mode, dtype):
    s = Loop(tv, mode, dtype)
    # prompts
    s.fill.run(**s.prefill_args())
    tv.token_counts_update(s.counts, s.prompt, s.st, starts=s.starts, clear=True, prompt=True)
    torch.cuda.synchronize()
    for st in (s.fill.st_append, s.fill.st_attn, s.st):
        assert st.eq(0).all()
    pos = torch.cat([torch.arange(n) for n in PROMPTS])
    check_append(s, s.prompt_act, pos, PROMPTS, [0] * B, s.fill.q)
    check_chunk_attention(s, s.fill, s.starts, PROMPTS, [0] * B)
    hist = torch.zeros((B, V), dtype=torch.int64)
    for b in range(B):
        hist[b, s.prompt[s.starts[b]:s.starts[b + 1]].long().cpu()] = -2**31
    assert torch.equal(s.counts.cpu().long(), hist)
    # the tree
    s.prefix = i32(PROMPTS)
    s.append_tree()
    torch.cuda.synchronize()
    assert s.st.eq(0).all()
    check_append(s, s.tree_act, s.positions, [N] * B, PROMPTS, s.q_tree)
    k0, v0 = s.k_cache.cpu().clone(), s.v_cache.cpu().clone()
    s.step.run(**s.verify_args())
    torch.cuda.synchronize()
    for st in (s.step.st_mask, s.step.st_attn, s.step.st_process, s.step.st_accept, s.step.st_counts,
               s.step.st_compact):
        assert st.eq(0).all()
    bf16 = dtype == torch.bfloat16
    raw = (lambda t: t.view(torch.int16).numpy().view(np.uint16)) if bf16 else (lambda t: t.numpy())
    mask, depth, _ = orc.tree_mask(np.array(PARENTS, np.int32))
    ref, _ = orc.attention(raw(s.q_tree.cpu()).reshape(B, N, HQ, D), raw(k0), raw(v0), s.table.cpu().numpy(),
                           s.prefix.cpu().numpy(), mask, bf16=bf16)
    err = np.abs(host_f32(s.step.out).reshape(ref.shape) - ref)
    assert err.max() <= (2e-2 if bf16 else 1e-5)
    kw = {k: v.cpu() for k, v in s.sampling.items()}
    kw["counts"] = hist.to(torch.int32)
    want = R.logits(s.raw.cpu(), mask=torch.from_numpy(mask.view(np.int64)), tokens=s.draft.cpu(),
                    counts=kw["counts"], grammar=kw["grammar"], rep=kw["repetition"],
                    freq=kw["frequency"], pres=kw["presence"], temp=kw["temperature"], probs=bool(mode))
    got = s.step.target.cpu().double()
    inf = want == -float("inf")
    assert torch.equal(inf, got == -float("inf"))
    # a logit: seven float32 roundings of at most 3 * 6 + 8 + 6 * 0.7, times 1.25, over 0.7; a
    # probability moves by twice that, by 2^-20 and by a sum of V terms
    z = 7 * 2.0 ** -24 * 31 * 1.25 / 0.7
    tol = want.abs() * (2 * z + 2.0 ** -20 + V * 2.0 ** -24) + 2.0 ** -126 if mode else z
    assert ((got - want).masked_fill(inf, 0.0).abs() <= tol).all()
    # acceptance of what the GPU held, the history with it, the rows moved
    target = s.step.target.cpu().numpy()
    args = (np.array(PARENTS, np.int32), s.draft.cpu().numpy(), target)
    acc = orc.accept_stochastic(*args, s.draft_probs.cpu().numpy(), 11, 5, N) if mode else \
        orc.accept_greedy(*args, N)
    for t, r in zip((s.step.accept_len, s.step.path, s.step.out_tokens), acc):
        assert np.array_equal(t.cpu().numpy(), r)
    for b in range(B):
        for t in acc[2][b]:
            hist[b, t] += int(t >= 0)
    assert torch.equal(s.counts.cpu().long(), hist)
    lens = s.step.new_lens.cpu().tolist()
    for b in range(B):
        assert lens[b] == PROMPTS[b] + int(acc[0][b]) + 1
        src = torch.tensor(list(range(PROMPTS[b])) + [PROMPTS[b] + int(x) for x in acc[1][b][:int(acc[0][b]) + 1]])
        for now, old in ((s.k_cache, k0), (s.v_cache, v0)):
            blk, row = s.table.cpu()[b][src // BS].long(), src % BS
            assert torch.equal(rows_of(s, now, b, lens[b]), old[blk, :, row])
    # one more token of each sequence
    s.ones = i32(list(range(B + 1)))
    s.one.run(**s.decode_args())
    torch.cuda.synchronize()
    assert s.one.st_append.eq(0).all() and s.one.st_attn.eq(0).all()
    check_append(s, s.one_act, torch.tensor(lens), [1] * B, lens, s.one.q)
    check_chunk_attention(s, s.one, s.ones, [1] * B, lens)


@pytest.mark.parametrize("mode", [0, 1])
def test_captured_loop_is_the_eager_one(tv, mode):
    """Prefill, verification with sampling and decoding as three graphs, replayed one after the
    other on the state that the eager steps began with: every output bit for bit."""
    def outputs(s):
        torch.cuda.synchronize()
        return [t.cpu().clone() for t in (s.fill.out, s.step.out, s.step.target, s.step.out_tokens,
                                          s.step.new_lens, s.one.out, s.counts, s.k_cache, s.v_cache)]

    a = Loop(tv, mode, torch.bfloat16)
    b = Loop(tv, mode, torch.bfloat16)
    for s in (a, b):
        s.prefix = i32(PROMPTS)
        s.ones = i32(list(range(B + 1)))
        s.counts.zero_()
    a.fill.run(**a.prefill_args())
    a.append_tree()
    a.step.run(**a.verify_args())
    a.one.run(**a.decode_args())
    want = outputs(a)

    k0, v0 = b.k_cache.clone(), b.v_cache.clone()
    fill = b.fill.capture(**b.prefill_args())
    b.append_tree()
    verify = b.step.capture(**b.verify_args())
    one = b.one.capture(**b.decode_args())
    b.k_cache.copy_(k0)
    b.v_cache.copy_(v0)
    b.counts.zero_()
    fill.replay()
    b.append_tree()
    verify.replay()
    one.replay()
    for x, y in zip(want, outputs(b)):
        assert torch.equal(x, y)


def test_sampling_needs_its_buffers(tv):
    from eagle_speculative_decoding_parent_gb300.pipeline import VerifyStep
    s = Loop(tv, 0, torch.bfloat16)
    s.prefix = i32(PROMPTS)
    s.step = VerifyStep(B=B, N=N, Hq=HQ, Hkv=HKV, d=D, max_blocks=BLOCKS, bs=BS,
                        dtype=torch.bfloat16, max_path=N, V=V)
    with pytest.raises(ValueError):
        s.step.run(**s.verify_args())


def test_two_host_threads(tv):
    """Two threads, each with its own loop on its own stream, give what one alone gives."""
    def run(s, stream):
        with torch.cuda.stream(stream):
            for _ in range(3):
                s.fill.run(**s.prefill_args())
                tv.token_counts_update(s.counts, s.prompt, s.st, starts=s.starts, clear=True, prompt=True)
                s.prefix, s.ones = i32(PROMPTS), i32(list(range(B + 1)))
                s.append_tree()
                s.step.run(**s.verify_args())
                s.one.run(**s.decode_args())
        stream.synchronize()

    def state(s):
        return [t.cpu() for t in (s.fill.out, s.step.out, s.step.target, s.step.out_tokens, s.one.out, s.counts)]

    want = []
    for mode in (0, 1):
        s = Loop(tv, mode, torch.bfloat16)
        torch.cuda.synchronize()
        run(s, torch.cuda.Stream())
        want.append(state(s))
    loops = [Loop(tv, mode, torch.bfloat16) for mode in (0, 1)]
    torch.cuda.synchronize()
    threads = [threading.Thread(target=run, args=(s, torch.cuda.Stream())) for s in loops]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for s, w in zip(loops, want):
        for x, y in zip(state(s), w):
            assert torch.equal(x, y)
