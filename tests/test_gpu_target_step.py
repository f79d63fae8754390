"""The operators together, as a serving step runs them: drafts from the chain, the
scheduler's lengths, the target's rows and pages, rotated keys into the cache, attention,
logits with penalties, greedy verification, and what it accepted into the next step.
The target is one layer whose projections are tables by token, so that every stage can
be computed again on the CPU from what the stage before it left on the GPU."""
import math

import pytest

torch = pytest.importorskip("torch")

import target_ref as ref  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import dspark as D  # noqa: E402
from speculative_decoding_draft_dspark_gb300 import target as T  # noqa: E402
from test_gpu_target_rotary import close  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, I32 = torch.bfloat16, torch.int32
HALF = torch.finfo(BF16).eps / 2
N, K, VOCAB, RANK = 6, 3, 512, 16
HQ, HK, HD, PAGE, MAX_PAGES, PAGES = 8, 2, 64, 16, 12, 60
ROWS, WIDTH = 64, 160
PROMPT, CHUNK = 5, 40            # the request that is still reading its prompt


class Server:
    """Everything that a program keeps on the GPU, and one step over it."""

    def __init__(self):
        g = torch.Generator().manual_seed(4)
        rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        i32 = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")  # noqa: E731
        self.table = rnd(VOCAB, (HQ + 2 * HK) * HD).to(BF16).cuda()
        self.head = (rnd(HQ * HD, VOCAB) * 0.2).to(BF16).cuda()
        self.drafter = (rnd(VOCAB, K, VOCAB) * 2).to(BF16).cuda()
        self.U, self.V = ((rnd(VOCAB, RANK) * 0.5).to(BF16).cuda() for _ in range(2))
        self.conf = torch.full((N, K), 0.9, device="cuda")
        self.conf[1, 1:] = 0.01
        self.mask = torch.ones(N, dtype=torch.uint8, device="cuda")
        self.mask[PROMPT] = 0
        self.chunk_len = i32(N)
        self.chunk_len[PROMPT] = CHUNK
        self.cost = torch.linspace(10.0, 10.5, 256).cuda()
        self.T = torch.tensor([N - 1 + CHUNK], dtype=I32, device="cuda")
        self.tokens = torch.randint(0, VOCAB, (N, WIDTH), generator=g, dtype=I32).cuda()
        self.ctx_len, self.prompt_len = i32(N), i32(N)
        self.page_count, self.free_count, self.block_table = i32(N), i32(1), i32(N, MAX_PAGES)
        self.block_table -= 1
        self.free_pages = torch.randperm(PAGES, generator=g).int().cuda()
        self.free_count += PAGES
        self.k_cache, self.v_cache = (torch.full((PAGES, PAGE, HK, HD), math.nan, dtype=BF16, device="cuda")
                                      for _ in range(2))
        self.turns = T.dspark_rotary_table(HD, 10000.0).cuda()
        self.penalty = {k: torch.full((N,), v, device="cuda") for k, v in
                        (("repetition", 1.2), ("frequency", 0.3), ("presence", 0.1))}
        self.allowed = torch.randint(-(1 << 31), 1 << 31, (2, VOCAB // 32), generator=g).int().cuda()
        self.mask_index = torch.full((ROWS,), -1, dtype=I32, device="cuda")
        self.mask_index[2], self.mask_index[7] = 0, 1
        self.draft = i32(N, K)
        self.draft_len, self.cu_len, self.verify_idx, self.B = i32(N), i32(N + 1), i32(N * K), i32(1)
        self.cu_rows, self.cu_out = i32(N + 1), i32(N + 1)
        for k in ("row_request", "position", "slot", "row_token", "out_row"):
            setattr(self, k, i32(ROWS))
        self.q = torch.zeros(ROWS, HQ, HD, dtype=BF16, device="cuda")
        self.out = torch.zeros(ROWS, HQ, HD, dtype=BF16, device="cuda")
        self.lse = torch.zeros(ROWS, HQ, device="cuda")
        self.raw = torch.zeros(ROWS, VOCAB, dtype=BF16, device="cuda")
        self.logits = torch.zeros(ROWS, VOCAB, dtype=BF16, device="cuda")
        self.argmax, self.accepted, self.bonus = i32(N * (K + 1)), i32(N), i32(N)
        self.ws = T.new_workspace(256)
        self.chain_ws = D.new_workspace(D.dspark_chain_workspace_size(N, K))
        self.select_ws = D.new_workspace(D.dspark_select_workspace_size(N, K, 256))
        self.attention_ws = T.new_workspace(T.dspark_attention_workspace_size(N, CHUNK, HQ, HK, HD))

    def step(self):
        last = self.tokens.gather(1, self.ctx_len.long()[:, None])[:, 0]
        D.dspark_chain_draft(self.drafter[last.long()], self.U, self.V, last, self.draft, None, self.chain_ws)
        D.dspark_select_step(self.conf, self.mask, self.cost, self.T, 0.0, 0, self.draft, None, None, None, None,
                             None, self.B, None, self.draft_len, self.cu_len, self.verify_idx, None, self.select_ws)
        T.dspark_step_rows(self.draft_len, self.mask, self.chunk_len, self.ctx_len, None, self.tokens, self.draft,
                           self.page_count, self.free_pages, self.free_count, self.block_table, self.page_count,
                           self.free_count, self.cu_rows, self.cu_out, self.row_request, self.position, self.slot,
                           self.row_token, self.out_row, self.ws, page_size=PAGE, num_pages=PAGES)
        n_rows = self.cu_rows[N:]
        qkv = self.table[self.row_token.long()]
        q, k, v = (x.view(ROWS, -1, HD) for x in qkv.split([HQ * HD, HK * HD, HK * HD], 1))
        T.dspark_rotary_append(q, k, v, self.position, self.slot, self.turns, self.q, self.k_cache, self.v_cache,
                               n_rows=n_rows)
        T.dspark_tree_attention(self.q, self.k_cache, self.v_cache, self.block_table, self.ctx_len, self.cu_rows,
                                None, self.out, self.lse, self.attention_ws, max_len=CHUNK,
                                scale=1.0 / math.sqrt(HD))
        self.raw.copy_(self.out[self.out_row.long()].view(ROWS, -1) @ self.head)
        T.dspark_adjust_logits(self.raw, self.cu_out, self.tokens, self.ctx_len + 1, self.prompt_len, self.draft,
                               None, self.logits, self.ws, mask=self.allowed, mask_index=self.mask_index,
                               **self.penalty)
        D.dspark_greedy_verify(self.logits, self.draft, self.draft_len, self.cu_len, self.mask, self.argmax,
                               self.accepted, self.bonus, self.select_ws)

    def commit(self):
        """What was accepted, and the token after it, to the end of the text; a prompt
        goes on."""
        samples = self.mask.bool()
        moved = torch.where(samples, self.accepted + 1, self.chunk_len)
        at = torch.arange(K + 1, device="cuda")
        new = torch.cat([self.draft, self.draft[:, :1]], 1)
        new = torch.where(at == self.accepted[:, None], self.bonus[:, None], new)
        index = (self.ctx_len[:, None] + 1 + at).long().clamp(max=WIDTH - 1)
        keep = samples[:, None] & (at <= self.accepted[:, None])
        self.tokens.scatter_(1, index, torch.where(keep, new, self.tokens.gather(1, index)))
        self.ctx_len += moved

    def state(self):
        return [x.clone() for x in (self.draft, self.draft_len, self.cu_rows, self.slot, self.q, self.out, self.lse,
                                    self.logits, self.accepted, self.bonus, self.tokens, self.ctx_len,
                                    self.block_table, self.page_count, self.free_count)]


def check(s, before):
    """Every stage of the step, from what the one before it left."""
    ctx, tokens, page_count, free, table = before
    assert all(D.dspark_read_status(w) == 0 for w in (s.ws, s.chain_ws, s.select_ws, s.attention_ws))
    want = ref.rows(s.draft_len.tolist(), s.mask.tolist(), s.chunk_len.tolist(), ctx, None, tokens.tolist(),
                    s.draft.tolist(), page_count, free, PAGE, MAX_PAGES, PAGES, ROWS, table)
    for k in ("cu_rows", "cu_out"):
        assert getattr(s, k).tolist() == want[k]
    R, O = want["cu_rows"][-1], want["cu_out"][-1]
    for k in ("row_request", "position", "slot", "row_token"):
        assert getattr(s, k).tolist()[:R] == want[k], k
    assert s.out_row.tolist()[:O] == want["out_row"]
    assert s.block_table.tolist() == table and s.page_count.tolist() == want["page_count"]
    # keys and values of the rows
    freq = torch.tensor([10000.0 ** (-2.0 * i / HD) for i in range(HD // 2)], dtype=torch.float64)
    rows = s.table.cpu()[want["row_token"]]
    q, k, v = (x.view(R, -1, HD) for x in rows.split([HQ * HD, HK * HD, HK * HD], 1))
    position = torch.tensor(want["position"])
    slot = torch.tensor(want["slot"])
    close(s.q[:R], ref.rotate(q, position, freq, HD, False), q, BF16)
    flat = lambda c: c.cpu().view(PAGES * PAGE, HK, HD)  # noqa: E731
    close(flat(s.k_cache)[slot], ref.rotate(k, position, freq, HD, False), k, BF16)
    assert torch.equal(flat(s.v_cache)[slot], v)
    # attention: see test_gpu_target_attention for the bounds
    out, lse, size = ref.attention(s.q[:R].cpu(), s.k_cache.cpu(), s.v_cache.cpu(), s.block_table.cpu(), ctx,
                                   want["cu_rows"], None, 1.0 / math.sqrt(HD))
    e = 2.0 ** -17 / math.sqrt(HD) * float(s.q[:R].cpu().double().abs().sum(-1).amax()) * float(
        torch.nan_to_num(s.k_cache.cpu().double(), nan=0.0).abs().amax()) + 2.0 ** -18
    assert ((s.out[:R].cpu().double() - out).abs() <= HALF * out.abs() + size * (HALF + 2 * e)).all()
    assert ((s.lse[:R].cpu().double() - lse).abs() <= e + lse.abs() * 2.0 ** -22).all()
    # logits
    adjusted, size = ref.adjust(s.raw[:O].cpu(), want["cu_out"], tokens, torch.tensor(ctx) + 1,
                                s.prompt_len.cpu(), s.draft.cpu(), None, mask=s.allowed.cpu(),
                                mask_index=s.mask_index.cpu(), **{k: x.cpu() for k, x in s.penalty.items()})
    got = s.logits[:O].cpu().double()
    fine = adjusted.isfinite()
    assert torch.equal(fine, got.isfinite())
    assert ((got - adjusted).abs() <= HALF * adjusted.abs() + 2.0 ** -20 * size)[fine].all()
    # verification, of those logits
    best = got.argmax(1).tolist()
    for n in range(N):
        if n == PROMPT:
            assert s.accepted[n] == s.bonus[n] == -1
            continue
        row, a = want["cu_out"][n], 0
        while a < int(s.draft_len[n]) and int(s.draft[n, a]) == best[row + a]:
            a += 1
        assert int(s.accepted[n]) == a and int(s.bonus[n]) == best[row + a]


def test_steps_of_a_server():
    s = Server()
    for _ in range(4):
        before = (s.ctx_len.tolist(), s.tokens.cpu(), s.page_count.tolist(),
                  s.free_pages.tolist()[:int(s.free_count)], s.block_table.tolist())
        s.step()
        check(s, before)
        s.commit()
        if int(s.ctx_len[PROMPT]) + CHUNK > WIDTH - 10:
            break
    assert int(s.ctx_len.max()) > 2 * CHUNK and len(set(s.ctx_len.tolist())) > 1


def test_a_step_as_a_graph_gives_the_same_bits():
    """Nothing of a step depends on the host: captured once, replayed for every step."""
    eager, replayed = Server(), Server()
    warm = Server()
    warm.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed.step()
        replayed.commit()
    for _ in range(3):
        eager.step()
        eager.commit()
        graph.replay()
        for a, b in zip(eager.state(), replayed.state()):
            assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a,
                               b.nan_to_num(7.0) if b.is_floating_point() else b)
