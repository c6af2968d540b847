"""A prompt's way into the cache and the decode that follows, as an engine runs them (needs a GPU): pages and slots, rotary
positions, the quantised write, attention over the prompts, decode steps in place, a context whose first part is cached
already, and pages given back.  The attention is checked against the oracles on the same bytes."""
import math

import numpy as np
import pytest
import torch

from cache_util import dev, host, word
from gpu_util import compare, compare_lse
from oracle import prompt_ops as C
from paged_fp8_kv_04_gb300 import binding as B

pytestmark = pytest.mark.gpu

G, D = 16, 128


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Engine:
    """A cache of one KV head with its pool, and the calls of a step; requests of one batch."""

    def __init__(self, reqs, page, pages, width, seed=0):
        rng = np.random.default_rng(seed)
        self.page, self.pages, self.reqs = page, pages, reqs
        self.lens, self.table = torch.zeros(reqs, dtype=torch.int32, device="cuda"), torch.full((reqs, width), -1, dtype=torch.int32, device="cuda")
        self.free, self.count = dev(rng.permutation(pages).astype(np.int32)), torch.tensor([pages], dtype=torch.int32, device="cuda")
        self.k, self.v = (torch.zeros(pages, 1, page, D, dtype=torch.uint8, device="cuda") for _ in range(2))
        self.ks, self.vs = (torch.zeros(pages, 1, page, device="cuda") for _ in range(2))
        self.freqs, self.scale = B.rope_frequencies(D, base=500000.0)
        self.status = word()

    def rows(self, g, n):
        """The projections' output for n tokens, and its views."""
        buf = torch.randn(n, (G + 2) * D, generator=g, device="cuda").bfloat16()
        return [x.unflatten(1, (-1, D)) for x in buf.split([G * D, D, D], 1)]

    def admit(self, cu, q, k, v):
        """Slots, turned queries and keys, and the write; the lengths move on."""
        _, slots, pos = B.page_assign(self.lens, cu, self.table, self.free, self.count, page_size=self.page, num_pages=self.pages,
                                      num_rows=q.shape[0], new_lens=self.lens, status=self.status)
        q, k = B.rope(q, k, pos, self.freqs, scale=self.scale, q_out=torch.empty_like(q, memory_format=torch.contiguous_format),
                      k_out=torch.empty_like(k, memory_format=torch.contiguous_format))
        v = v.contiguous()
        B.kv_quantize_write(k, v, slots, self.k, self.v, self.ks, self.vs)
        return q, k, v, slots, pos

    def cached(self, r, n):
        """What the cache holds of request r's first n tokens, in fp64."""
        pages = self.table[r, : -(-n // self.page)].long()
        get = lambda c, s: (c[pages, 0].view(torch.float8_e4m3fn).double() * s[pages, 0].double()[..., None]).reshape(-1, D)[:n]  # noqa: E731
        return get(self.k, self.ks), get(self.v, self.vs)


def _attend(q, k, v):
    """q [G, D] of one token over k, v [n, D], fp64."""
    x = (q.double() @ k.T) / math.sqrt(D)
    z = torch.logsumexp(x, -1)
    return torch.exp(x - z[:, None]) @ v, z


@pytest.mark.parametrize("page", [16, 128])
def test_prompts_then_decode_steps(page):
    g = torch.Generator(device="cuda").manual_seed(page)
    lens = [300, 1, 129, 0, 777]
    e = Engine(len(lens), page, 400, 60)
    cu = torch.tensor(np.r_[0, np.cumsum(lens)], dtype=torch.int32, device="cuda")
    rows = int(cu[-1]) + 6                                    # a padded batch
    q, k, v, slots, pos = e.admit(cu, *e.rows(g, rows))
    assert host(e.lens).tolist() == lens and np.all(host(slots)[-6:] == -1)
    out, lse = B.prompt_attn(q, k, v, cu, out=torch.zeros_like(q), want_lse=True, status=e.status)
    ref, rl, *_ = C.prompt_attn(*(x.double().cpu().numpy() for x in (q, k, v)), host(cu), 1 / math.sqrt(D))
    compare(out.double().cpu().numpy(), ref, "prompts")
    n = int(cu[-1])                                           # (rows of no request are not written)
    compare_lse(lse.cpu().numpy()[:n], rl[:n], "prompts")
    # every request's last token, by the decode over the cache that was written, sees what the prompt saw up to e4m3
    live = [r for r, n in enumerate(lens) if n]
    plan = B.Plan(page_size=page, max_batch=len(lens), max_context_len=1024)
    for step in range(3):
        cu1 = torch.arange(len(lens) + 1, dtype=torch.int32, device="cuda")
        q1, _, _, slots, pos = e.admit(cu1, *e.rows(g, len(lens)))
        assert host(e.lens).tolist() == [n + step + 1 for n in lens] and host(pos).tolist() == [n + step for n in lens]
        out = plan.decode(q1, e.k, e.v, e.table, e.lens, k_scale=e.ks, v_scale=e.vs)
        torch.cuda.synchronize()
        for r in range(len(lens)):
            kk, vv = e.cached(r, lens[r] + step + 1)
            compare(out[r].double().cpu().numpy(), _attend(q1[r], kk, vv)[0].cpu().numpy(), f"step {step} request {r}")
    assert int(e.status) == 0 and plan.device_status() == 0 and live
    # all of it given back
    B.page_release(e.lens, torch.zeros_like(e.lens), e.table, e.free, e.count, page_size=page, num_pages=e.pages, status=e.status)
    assert int(e.count) == e.pages and sorted(host(e.free).tolist()) == list(range(e.pages)) and int(e.status) == 0


def test_decode_steps_from_one_graph():
    """assign, rope, write and decode captured once, lengths and tables updated in place; each replay is a step."""
    reqs, page, steps = 7, 16, 40
    g = torch.Generator(device="cuda").manual_seed(1)
    e = Engine(reqs, page, 64, 8)
    plan = B.Plan(page_size=page, max_batch=reqs, max_context_len=128)
    cu = torch.arange(reqs + 1, dtype=torch.int32, device="cuda")
    q, k, v = e.rows(g, reqs)
    buf = q._base
    qo, ko, vo = torch.empty(reqs, G, D, dtype=torch.bfloat16, device="cuda"), torch.empty(reqs, 1, D, dtype=torch.bfloat16, device="cuda"), torch.empty(
        reqs, 1, D, dtype=torch.bfloat16, device="cuda")
    slots, pos = torch.empty(reqs, dtype=torch.int64, device="cuda"), torch.empty(reqs, dtype=torch.int32, device="cuda")
    out = torch.empty_like(qo)

    def step():
        B.page_assign(e.lens, cu, e.table, e.free, e.count, page_size=page, num_pages=e.pages, new_lens=e.lens, slot_mapping=slots, positions=pos, status=e.status)
        B.rope(q, k, pos, e.freqs, q_out=qo, k_out=ko)
        vo.copy_(v)
        B.kv_quantize_write(ko, vo, slots, e.k, e.v, e.ks, e.vs)
        plan.decode(qo, e.k, e.v, e.table, e.lens, k_scale=e.ks, v_scale=e.vs, out=out)
    B.torch_module()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        step()
    for n in range(steps):
        buf.normal_(generator=g)
        graph.replay()
        torch.cuda.synchronize()
        assert host(e.lens).tolist() == [n + 1] * reqs and host(pos).tolist() == [n] * reqs
        for r in (0, reqs - 1):
            kk, vv = e.cached(r, n + 1)
            compare(out[r].double().cpu().numpy(), _attend(qo[r], kk, vv)[0].cpu().numpy(), f"step {n} request {r}")
    assert int(e.status) == 0 and plan.device_status() == 0
    assert int(e.count) == e.pages - reqs * -(-steps // page)


def test_chunk_over_a_cached_prefix():
    """A chunk of a prompt whose beginning is cached: attention over the chunk's own tokens and a decode of each of its rows
    over the cached pages, joined by their log-sum-exps, against attention over both parts at once."""
    page, prefix, chunk = 128, 640, 301
    g = torch.Generator(device="cuda").manual_seed(2)
    e = Engine(1, page, 20, 10)
    one = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    e.admit(one(prefix), *e.rows(g, prefix))
    cached_k, cached_v = e.cached(0, prefix)
    q, k, v, _, pos = e.admit(one(chunk), *e.rows(g, chunk))
    assert host(pos)[0] == prefix
    parts, lses = torch.empty(2, chunk, G, D, device="cuda"), torch.empty(2, chunk, G, device="cuda")
    B.prompt_attn(q, k, v, one(chunk), out=parts[0], lse=lses[0], status=e.status)
    # every row a request of one token over the prefix's pages
    plan = B.Plan(page_size=page, max_batch=chunk, max_context_len=prefix, out_dtype="f32")
    plan.decode(q, e.k, e.v, e.table.expand(chunk, -1).contiguous(), torch.full((chunk,), prefix, dtype=torch.int32, device="cuda"), k_scale=e.ks, v_scale=e.vs,
                out=parts[1], lse=lses[1])
    out, lse = torch.empty_like(q), torch.empty(chunk, G, device="cuda")
    B.lse_merge(parts, lses, out, lse)
    torch.cuda.synchronize()
    assert int(e.status) == 0 and plan.device_status() == 0
    for t in (0, 1, 127, 128, 255, chunk - 1):
        ref, z = _attend(q[t], torch.cat([cached_k, k[:t + 1, 0].double()]), torch.cat([cached_v, v[:t + 1, 0].double()]))
        compare(out[t].double().cpu().numpy(), ref.cpu().numpy(), f"row {t}")
        compare_lse(lse[t].cpu().numpy(), z.cpu().numpy(), f"row {t}")


def test_eviction_gives_its_pages_back():
    """Contexts cut to a budget in place: the pages behind the new lengths return to the pool and are assigned again."""
    page, budget = 16, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = [200, 64, 150]
    e = Engine(3, page, 32, 14)
    cu = torch.tensor(np.r_[0, np.cumsum(lens)], dtype=torch.int32, device="cuda")
    e.admit(cu, *e.rows(g, int(cu[-1])))
    held = sum(-(-n // page) for n in lens)
    assert int(e.count) == e.pages - held
    mass = torch.rand(3, 1, 224, generator=g, device="cuda")
    before = [e.cached(r, n)[0].clone() for r, n in enumerate(lens)]
    keep, new = B.evict_select(mass, e.lens, budget=budget, first=2, recent=8, status=e.status)
    B.kv_compact(keep, new, e.table, e.k, e.v, k_scale=e.ks, v_scale=e.vs, status=e.status)
    B.page_release(e.lens, new, e.table, e.free, e.count, page_size=page, num_pages=e.pages, status=e.status)
    e.lens = new
    assert host(new).tolist() == [budget] * 3 and int(e.count) == e.pages - 3 * budget // page and int(e.status) == 0
    for r in range(3):
        assert torch.equal(e.cached(r, budget)[0], before[r][keep[r, 0].long()])
    mine = set(host(e.table)[:, :budget // page].ravel().tolist())
    assert not mine & set(host(e.free)[:int(e.count)].tolist())
    # as many new tokens as the pool then holds
    more = torch.tensor([0, 160, 160, 320], dtype=torch.int32, device="cuda")
    _, _, _, slots, _ = e.admit(more, *e.rows(g, 320))
    assert int(e.status) == 0 and int(e.count) == 0 and host(e.lens).tolist() == [224, 64, 224]
    assert len(set(host(slots).tolist())) == 320 and not {int(s) // page for s in host(slots)} & mine
