"""The paged step as it is used, end to end on one GPU (needs a GB300): prompts in chunks, then
draft chains verified and scored, against the same model over the whole sequence in float64."""
import numpy as np
import pytest
import torch

from speculative_decoding_tree_mask_gb300 import binding as G

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


class Model:
    """Embedding, one attention layer with head norms and rotated positions, output head."""

    def __init__(self, V=499, Hq=8, H=2, D=64, dtype=torch.float16):
        g = torch.Generator(device=DEV)
        g.manual_seed(5)

        def weight(n, m):
            return (torch.randn((n, m), generator=g, device=DEV) * m ** -0.5).to(dtype)

        self.Hq, self.H, self.D, W = Hq, H, D, Hq * D
        self.emb = weight(V, W) * W ** 0.5
        self.qkv, self.proj, self.head = weight((Hq + 2 * H) * D, W), weight(W, W), weight(V, W)
        self.w = torch.ones(D, dtype=dtype, device=DEV)
        self.inv_freq = 10000.0 ** (-torch.arange(D // 2, device=DEV).float() / (D // 2))

    def split(self, tokens):
        rows = self.emb[tokens] @ self.qkv.T
        n = [self.Hq * self.D, self.H * self.D, self.H * self.D]
        return [t.unflatten(1, (-1, self.D)) for t in rows.split(n, -1)]

    def logits(self, tokens, out):
        x = self.emb[tokens] + 0.3 * (out.flatten(1) @ self.proj.T)
        return (x @ self.head.T).float()

    def whole(self, tokens, window, sinks):
        """Logits of every position of one sequence, in float64 from the rounded projections."""
        q, k, v = (t.double() for t in self.split(tokens))
        L, G_ = len(tokens), self.Hq // self.H
        pos = torch.arange(L, device=DEV)

        def turn(x):
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6)
            t = (pos[:, None] * self.inv_freq.double()).unsqueeze(1)
            a, b = x.chunk(2, -1)
            return torch.cat((a * t.cos() - b * t.sin(), b * t.cos() + a * t.sin()), -1)

        q, k = turn(q), turn(k).repeat_interleave(G_, 1)
        z = torch.einsum("nhd,lhd->hnl", q, k) * self.D ** -0.5
        see = pos[None] <= pos[:, None]
        if window:
            see = see & ((pos[None] > pos[:, None] - window) | (pos[None] < sinks))
        out = torch.einsum("hnl,lhd->nhd", z.masked_fill(~see, -np.inf).softmax(-1),
                           v.repeat_interleave(G_, 1))
        x = self.emb[tokens].double() + 0.3 * (out.flatten(1) @ self.proj.double().T)
        return x @ self.head.double().T


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 4)])
@pytest.mark.parametrize("kind", [torch.float16, torch.float8_e4m3fn])
def test_prompt_chains_and_scores(kind, window, sinks):
    m = Model()
    rng = np.random.default_rng(9)
    lens, chunk, steps, draft = [37, 150, 5, 96], 64, 4, 6
    B, bs, pages = len(lens), 16, 16
    table = torch.from_numpy(rng.permutation(B * pages).reshape(B, pages).astype(np.int32)).to(DEV)
    scale = torch.tensor([2.0 ** -5], device=DEV) if kind != torch.float16 else None
    cache = G.KvCache.empty(B * pages, bs, m.H, m.D, kind, DEV, G.SPEC_KV_HND, scale, scale)
    seqs = [rng.integers(0, 499, n).tolist() for n in lens]
    pos = torch.zeros(B, dtype=torch.int32, device=DEV)
    st = torch.zeros(B, dtype=torch.int32, device=DEV)
    near, scored = 0.0, 0

    def forward(new):
        """Logits of the new tokens of each request (lists), appended at pos."""
        nonlocal near
        tokens = torch.tensor([t for n in new for t in n], device=DEV)
        start = torch.tensor(np.cumsum([0] + [len(n) for n in new]), dtype=torch.int32, device=DEV)
        q, k, v = m.split(tokens)
        q = G.kv_append(h, q, k, v, cache, table, pos, start, m.inv_freq, m.w, m.w, status=st)
        assert not st.any()
        out, _ = G.paged_attention(h, q, cache, table, pos, m.D ** -0.5, start,
                                   max_new=max(map(len, new)), window=window, sinks=sinks, status=st)
        assert not st.any()
        return m.logits(tokens, out), start.tolist()

    with G.Handle(B, 16, 499, 0) as h:
        for at in range(0, max(lens) - 1, chunk):       # all but each prompt's last token
            new = [s[at:min(at + chunk, len(s) - 1)] for s in seqs]
            forward(new)
            pos += torch.tensor([len(n) for n in new], dtype=torch.int32, device=DEV)
        parent = torch.arange(-1, draft - 1, dtype=torch.int32, device=DEV).repeat(B, 1)
        for step in range(steps):
            # drafts: what the whole model likes best, spoilt here and there
            drafts = []
            for s in seqs:
                d = list(s)
                for i in range(draft - 1):
                    t = int(m.whole(torch.tensor(d, device=DEV), window, sinks)[-1].argmax())
                    d.append(t if rng.random() < 0.8 else int(rng.integers(0, 499)))
                drafts.append(d[len(s) - 1:])
            rows, start = forward(drafts)
            rows = rows.view(B, draft, -1)
            res = G.verify_greedy(h, rows, torch.tensor(drafts, dtype=torch.int32, device=DEV), parent)
            lp = G.token_logprobs(h, rows, res["out_tokens"], res["kv_commit"], top=3)
            assert not res["status"].any() and not lp["flags"].any()
            pos += res["accept_len"] + 1
            for b, n in enumerate(res["accept_len"].tolist()):
                answer = res["out_tokens"][b, :n + 1].tolist()
                exact = m.whole(torch.tensor(seqs[b] + answer, device=DEV), window, sinks)
                want = exact.log_softmax(-1)[len(seqs[b]) - 1:-1]
                got = lp["logprob"][b, :n + 1].double()
                picked = want.gather(1, torch.tensor(answer, device=DEV)[:, None])[:, 0]
                near = max(near, float((got - picked).abs().max()))
                total = float(lp["logprob"][b].sum())
                assert abs(total - float(got.sum())) <= 1e-5 * (1 + abs(total))
                scored += n + 1
                seqs[b] += answer
    # the answers' log probabilities are the whole model's, to the rounding of 16-bit rows (2^-11 of
    # values and weights of about one, sums of 512 of them: a logit to 2^-11 sqrt(2) 5, say 2^-8),
    # or of 8-bit keys and values (2^-4 of each, 0.3 of whose mean is in a logit)
    assert scored > B * steps
    assert near <= (2.0 ** -6 if kind == torch.float16 else 0.3)
