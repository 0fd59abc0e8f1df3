"""Calls over caches with block scales find what was put in front of them: written by kernels and copies of their own
stream and of another one that was joined, in a captured graph and out of one.

Equal calls give equal bits, so the order is checked for equality with the same calls, each finished before the next."""

import pytest
import torch

import block_sparse_attention_03_gb300 as msa
from _blocks import DIM, KINDS, workspace

pytestmark = pytest.mark.gpu

H, HQ, K, NB = 2, 8, 4, 12


def _inputs(kv, seed):
    """What a step reads: prompts of 1 to NB blocks, their rows, queries and index keys."""
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(1, NB * 128 + 1, (5,), generator=gen)
    lens[seed % 5] = 0
    T = NB * 128 * 5
    off = torch.cumsum(lens, 0) - lens
    place = torch.randperm(5 * NB, generator=gen).reshape(5, NB)
    i = lambda x: x.to(torch.int32).contiguous().cuda()  # noqa: E731
    b = lambda *s: torch.randn(s, generator=gen).bfloat16().cuda()  # noqa: E731
    return dict(lens=i(lens), first=i(torch.zeros(5)), off=i(off), table=i(place), k=b(T, H, DIM), v=b(T, H, DIM), q=b(5, HQ, DIM),
                iq=b(5, H, DIM), idx=b(5 * NB, 128, DIM))


class _Step:
    """The same tensors for every step."""

    def __init__(self, kv):
        self.x = {n: t.clone() for n, t in _inputs(kv, 0).items()}
        x = self.x
        dt = torch.int8 if kv == "int8_block" else torch.uint8
        self.cache = msa.PagedCache(kv_dtype=kv, index_dtype="bf16", num_blocks=5 * NB, num_kv_heads=H, idx=x["idx"],
                                    **{n: torch.zeros((5 * NB, H, 128, DIM), dtype=dt, device="cuda") for n in "kv"},
                                    **{n: torch.zeros((5 * NB, H), device="cuda") for n in ("k_scale", "v_scale")})
        self.spans = msa.Spans(x["first"], x["lens"], x["off"], x["table"])
        self.batch = msa.Batch(x["lens"], x["table"], 1)
        self.cfg = msa.default_config(K)
        self.ws = [workspace(max(msa.msa_dense_workspace_size(self.cache, self.batch, HQ),
                                 msa.msa_workspace_size(self.cache, self.batch, self.cfg, HQ))) for _ in range(4)]
        o = lambda: torch.zeros((5, HQ, DIM), dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.out = dict(dense=o(), sparse=o(), lists=torch.zeros((5, H, K), dtype=torch.int32, device="cuda"),
                        k=torch.zeros_like(x["k"]), v=torch.zeros_like(x["v"]))

    def clear(self):
        for n in ("k", "v", "k_scale", "v_scale"):
            getattr(self.cache, n).zero_()
        for t in self.out.values():
            t.zero_()

    def run(self, new, between):
        """Inputs, insert, both attends, read; between(t): in front of every call, t what it reads next."""
        x, o = self.x, self.out
        q = lambda n: msa.Query(x[n])  # noqa: E731
        for n in ("first", "lens", "off", "table", "k", "v"):
            x[n].copy_(new[n])
        between(("v", "off"), new)
        msa.msa_block_insert(self.cache, self.spans, x["k"], x["v"], self.ws[0])
        between(("q",), new)
        msa.msa_dense_attend(self.cache, self.batch, self.cfg, q("q"), HQ, o["dense"], None, self.ws[1])
        between(("iq", "idx"), new)
        msa.msa_decode(self.cache, self.batch, self.cfg, q("iq"), q("q"), HQ, o["lists"], o["sparse"], None, self.ws[2])
        between(("first", "lens"), new)
        msa.msa_cache_read(self.cache, self.spans, o["k"], o["v"], self.ws[3])


def _check(step, want):
    torch.cuda.synchronize()
    # (msa_decode flags the empty sequence, whose length is below q_per_seq)
    assert [msa.msa_read_device_status(ws)[1] for ws in step.ws] == [0, 0, 2, 0]
    for n, t in step.out.items():
        assert torch.equal(t.view(torch.uint8), want[n].view(torch.uint8)), n


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("captured", [False, True])
def test_calls_wait_for_what_is_in_front_of_them(kv, captured):
    news = [_inputs(kv, s) for s in range(3)]
    step = _Step(kv)
    wants = []
    for new in news:
        step.clear()

        def finish(names, new):
            for n in names:
                step.x[n].copy_(new[n])
            torch.cuda.synchronize()
        step.run(new, finish)
        torch.cuda.synchronize()
        wants.append({n: t.clone() for n, t in step.out.items()})
        assert all(t.any() for t in wants[-1].values())

    other = torch.cuda.Stream()
    busy = torch.zeros(1 << 26, device="cuda")

    def join(names, new):
        # work of this stream and of another one, which takes some time before it writes, both just in front of the call
        here = torch.cuda.current_stream()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            busy.add_(1)
            for n in names:
                step.x[n].copy_(new[n])
        for n in ("table", "k"):
            step.x[n].copy_(new[n])
        here.wait_stream(other)

    main = torch.cuda.Stream()
    if captured:
        source = {n: t.clone() for n, t in news[0].items()}
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=main):
            step.clear()
            step.run(source, join)
    for i in (1, 2, 0, 2, 1, 1, 0):
        if captured:
            for n, t in source.items():
                t.copy_(news[i][n])
            graph.replay()
        else:
            main.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(main):
                step.clear()
                step.run(news[i], join)
        _check(step, wants[i])


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("change", ["lens", "table", "query", "layout", "first", "end", "offsets"])
def test_tensors_that_change_in_place_are_looked_at_again(kv, change):
    # holders that a call has taken before
    step = _Step(kv)
    x, o = step.x, step.out
    q = msa.Query(x["q"])

    def dense():
        msa.msa_dense_attend(step.cache, step.batch, step.cfg, q, HQ, o["dense"], None, step.ws[1])

    def sparse():
        msa.msa_sparse_attend(step.cache, step.batch, step.cfg, q, HQ, o["lists"], o["sparse"], None, step.ws[2])

    def insert():
        msa.msa_block_insert(step.cache, step.spans, x["k"], x["v"], step.ws[0])

    def read():
        msa.msa_cache_read(step.cache, step.spans, o["k"], o["v"], step.ws[3])

    for call in (insert, dense, sparse, read):
        call()
    torch.cuda.synchronize()
    attends, moves = (dense, sparse), (insert, read)
    if change == "lens":
        x["lens"].resize_(4)
        calls = attends + moves
    elif change == "table":
        x["table"].resize_(4, NB)
        calls = attends + moves
    elif change == "query":
        x["q"].resize_(5, HQ - 1, DIM)
        calls = attends
    elif change == "layout":
        x["table"].as_strided_((5, NB), (1, 5))
        calls = attends + moves
    else:
        x[{"first": "first", "end": "lens", "offsets": "off"}[change]].resize_(4)
        calls = moves
    for call in calls:
        with pytest.raises(msa.MsaError) as e:
            call()
        assert e.value.status == 1
